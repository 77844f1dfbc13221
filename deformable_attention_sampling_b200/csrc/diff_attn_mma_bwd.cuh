// Gradients of differential attention on the tensor cores (tcgen05,
// accumulators in TMEM), 16-bit types, heads up to 64 and values up to 128
// channels (sm_100a).  The mathematics is diff_attn.cuh's:
//   dS_0 = P_0 (dP - e_0),  dS_1 = -lambda P_1 (dP - e_1),  e_s = <g, O_s>
//   grad_q_s = scale dS_s K_s, grad_k_s = scale dS_s^T Q_s,
//   grad_v = (P_0 - lambda P_1)^T g.
// Two kernels, one owning query tiles and one owning key tiles, so that no sum
// goes through atomics; the price is that scores and dP are computed twice
// (14 of 10 parts of the products' work at D = 64, Dv = 128).
//
// Both run 20 warps: 16 compute warps (thread = lane of the accumulators, the
// four warpgroups take a quarter of a tile's columns each; a warp's steps wait
// for one another, so it takes four a scheduler to keep it busy), a producer (tensor-map
// loads), a warp that issues the scores and dP of the next tile as soon as the
// compute warps hold this tile's in registers, a warp that issues the gradient
// products once their left operands are written, and one that zeroes the rows
// of keys no token may see (0 times NaN).  The left operands are 16-bit, in
// TMEM (dS) and shared memory (P_0 - lambda P_1).
//
// Roundings.  For grad_q a dS is the sum of two 16-bit parts, its rounding and
// what that left over, each in a product of its own: one part alone added as much
// error as the rounding of the result does (root mean square 1.5 times a single
// rounding, now 1.03; the second part costs 25 us of 141 on the case below).
// grad_k and grad_v keep one part: their operands share TMEM with two more
// accumulators, and 1.4 times a single rounding is what they have.  The row sums
// e_s in grad_q come from the forward's outputs, whose weights were rounded: a
// quarter of a rounding, as the keys' errors average out.  grad_k, grad_v and
// grad_lambda take sums of unrounded weights that the query kernel finds on its way.
//
// fp16 operands are scaled by powers of two: dS by cs with |dS| cs <= 2^15
// (incoming gradients may be of any size), the weights by cp with
// |P_0 - lambda P_1| cp <= 2^15; the results are divided by them.  The query
// kernel's cs is a row's own, from its |g| and lambda and the largest |v| of its
// keys; the key kernel sums over tokens and takes one of an image and key / value
// head, from the largest |g| and |lambda| among them.  So no image, no group of
// heads and, in grad_q, no token loses digits to a larger one beside it; in grad_k
// a dS 2^28 times below the largest that its image and group could have does (fp16
// is subnormal there).  bf16 needs neither.
//
// Bound: a 128 x 64 tile's exponentials take 1024 cycles in either kernel, its
// products about 1360; the scores of a tile wait for the registers of the one
// before, so a tile takes about 2700 (grad_q: 16 more conversions and stores a
// thread for the second parts) and 2300.
// Measured on 2 x 4096 tokens, 8 heads of 64 + 128, causal: grad_q 168 us,
// grad_k and grad_v 158 us.
#pragma once

#include "diff_attn_mma.cuh"

namespace dcnb {

constexpr int kAbThreads = 640;
constexpr int kAbMaxD = 64;
constexpr int kAbMaxDv = 128;
constexpr int kAbRowvBytes = kRowvTile * 4 * 4;

struct AttnBwdArgs {
    CUtensorMap tq;            // [N][Lq][2 M][D]
    CUtensorMap tk;            // [N][Lk][2 Mk][D]
    CUtensorMap tv;            // [N][Lk][Mk][Dv]
    CUtensorMap tg;            // [N][Lq][M][Dv]
    AttnArgs a;
    const float4* scales;      // [N][Mk] cs, cp, largest |v| (fp16)
    const float* gnorm;        // |g|^2 of the rows (fp16)
    float* rowv;               // the row values, whose e_s the first kernel rewrites
    unsigned int* flags;
    int dsteps, vsteps;        // K = 16 steps of a head, of the values
    int stages;
    int negate;
    int heads;                 // N * M (query tiles) or N * Mk (key tiles)
};

__host__ __device__ constexpr int attn_dq_smem(int vch, int stages) {
    return 1024 + (2 + vch) * kAmQBytes + stages * (2 + vch) * kAmKBytes + 1024 + 4096;
}
__host__ __device__ constexpr int attn_dkv_smem(int vch, int stages) {
    return 1024 + (3 + vch) * kAmQBytes + stages * ((2 + vch) * kAmKBytes + kAbRowvBytes) +
           1024;
}

// The products a scores warp issues for one tile: both maps' scores and dP, each
// A [128 rows] B [64 rows]^T, to TMEM columns 0, 64, 128.
struct TileProducts {
    uint32_t tmem, d_hi, id_s, id_p;
    int dsteps, vsteps;
    // a, av: low descriptor words of the resident operands; b, bv of the stage's
    __device__ __forceinline__ void issue(uint32_t a, uint32_t av, uint32_t b, uint32_t bv) const {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (k < dsteps)
                    umma_f16(tmem + 64 * m, umma_desc_of(a + m * (kAmQBytes >> 4) + 2 * k, d_hi),
                             umma_desc_of(b + m * (kAmKBytes >> 4) + 2 * k, d_hi), id_s,
                             k != 0 ? 1u : 0u);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < vsteps)
                umma_f16(tmem + 128,
                         umma_desc_of(av + (k >> 2) * (kAmQBytes >> 4) + 2 * (k & 3), d_hi),
                         umma_desc_of(bv + (k >> 2) * (kAmKBytes >> 4) + 2 * (k & 3), d_hi), id_p,
                         k != 0 ? 1u : 0u);
    }
};

// Zeroes the rows of `chunks` swizzled chunks (64 columns each) whose bit is off,
// rows 32 w .. 32 w + 31 from bits[w]; one warp.
__device__ __forceinline__ void zero_hidden_rows(unsigned char* tile, int chunk_bytes, int chunks,
                                                 const uint32_t* bits, int words, int lane) {
    for (int w = 0; w < words; ++w) {
        const uint32_t hidden = ~bits[w];
        for (int r = lane >> 3; r < 32; r += 4)
            if (hidden >> r & 1)
                for (int c = 0; c < chunks; ++c)
                    *reinterpret_cast<uint4*>(tile + c * chunk_bytes + (w * 32 + r) * 128 +
                                              (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
    }
}

// What the rounding of x to the packed pair `w` left over, rounded itself.
template <typename T>
__device__ __forceinline__ uint32_t rest_of(float2 x, uint32_t w) {
    x = __ffma2_rn(make_float2(Elem<T>::lo(w), Elem<T>::hi(w)), make_float2(-1.f, -1.f), x);
    return Elem<T>::pack2(x.x, x.y);
}

template <typename T>
__global__ void __launch_bounds__(kAbThreads, 1)
    diff_attn_dq_mma_kernel(const __grid_constant__ AttnBwdArgs f) {
    constexpr bool kScaled = std::is_same<T, __half>::value;
    const AttnArgs& a = f.a;
    const int NS = f.stages;
    extern __shared__ __align__(128) unsigned char am_smem[];
    unsigned char* base = am_smem + ((1024u - (smem_u32(am_smem) & 1023u)) & 1023u);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int vch = (a.Dv + 63) >> 6, dn = (a.D + 15) & ~15;

    const int tile = (int)(blockIdx.x / (unsigned)f.heads);
    const int nh = (int)blockIdx.x - tile * f.heads;
    const int n = nh / a.M, head = nh - n * a.M, kv = head / a.G;
    const int q0 = ((int)(gridDim.x / (unsigned)f.heads) - 1 - tile) * kAmRows;
    const int len = attn_len(a, n);
    const int last = min(q0 + kAmRows, a.Lq) - 1;
    const int kmax = a.causal ? max(0, min(len, last + len - a.Lq + 1)) : len;
    const int count = (kmax + kAmKeys - 1) / kAmKeys;

    unsigned char* qs = base;                             // [2] chunks
    unsigned char* gs = qs + 2 * kAmQBytes;               // [vch]
    unsigned char* kvs = gs + vch * kAmQBytes;            // [NS][2 + vch]
    const int kvstage = (2 + vch) * kAmKBytes;
    uint64_t* q_full = reinterpret_cast<uint64_t*>(kvs + NS * kvstage);
    uint64_t* kv_full = q_full + 1;
    uint64_t* kv_empty = kv_full + NS;
    uint64_t* kv_clean = kv_empty + NS;
    uint64_t* s_full = kv_clean + NS;
    uint64_t* s_free = s_full + 1;
    uint64_t* p_full = s_free + 1;
    uint64_t* g_done = p_full + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(g_done + 1);
    uint32_t* vis = tmem_slot + 4;        // [NS][2]
    float2* esum = reinterpret_cast<float2*>(vis + 2 * NS);       // [4][128]

    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        for (int s = 0; s < NS; ++s) {
            mbar_init(&kv_full[s], 1);
            mbar_init(&kv_empty[s], 1);
            mbar_init(&kv_clean[s], 1);
        }
        mbar_init(s_full, 1);
        mbar_init(s_free, 16);
        mbar_init(p_full, 16);
        mbar_init(g_done, 1);
        mbar_fence_init();
    }
    if (warp == 17) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;"
                     :: "r"(smem_u32(tmem_slot)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = *tmem_slot;
    // TMEM columns: scores 0, 64; dP 128; dS [high, low part][2 maps] 32 each from 192;
    // grad_q 64 a map from 320
    const uint32_t d_hi = (uint32_t)(umma_desc128(0, 0) >> 32), lo_k = 16u >> 4 << 16;

    if (warp < 16) {
        // ------------------------------------------------------------- compute
        const int h = warp >> 2, quarter = warp & 3;
        const int row = quarter * 32 + lane, tok = q0 + row;
        const uint32_t t_row = tmem + ((uint32_t)(quarter * 32) << 16);
        const int limit = a.causal ? min(len, tok + len - a.Lq + 1) : len;
        const float lam = Elem<T>::one(static_cast<const T*>(a.lam) + head);
        const float cs = kScaled && tok < a.Lq
                             ? attn_grad_scale(lam, sqrtf(f.gnorm[attn_gnorm(a, n, head, tok)]),
                                               f.scales[n * a.Mk + kv].z)
                             : 1.f;
        float nl[2] = {-INFINITY, -INFINITY}, ne[2] = {0.f, 0.f};
        if (tok < a.Lq) {
            const float* r = a.rowv + attn_rowv(a, n, head, tok);
            const float lc = log2f(cs);
            nl[0] = r[0] + lc;
            nl[1] = r[kRowvTile] + lc;
            ne[0] = r[2 * kRowvTile];
            ne[1] = -lam * r[3 * kRowvTile];
        }
        const float2 sc2 = make_float2(a.scale_log2, a.scale_log2), al2 = make_float2(-lam, -lam);
        const float2 n0 = make_float2(nl[0], nl[0]), n1 = make_float2(nl[1], nl[1]);
        const float2 e0 = make_float2(ne[0], ne[0]), e1 = make_float2(ne[1], ne[1]);
        // sums over the keys of P_s dP, cs-fold: e_s from weights that were not rounded
        float2 es0 = make_float2(0.f, 0.f), es1 = es0;
        bool ok = true;
        Ring v(NS);
        for (int i = 0; i < count; ++i, v.next()) {
            const int j0 = i * kAmKeys + 16 * h;
            if (a.mask) ok = mbar_wait(&kv_full[v.st], v.phase, f.flags);
            ok = ok && mbar_wait(s_full, (uint32_t)(i & 1), f.flags);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tmem_fence_after();
            uint32_t r0[16], r1[16], rp[16];
            tmem_ld16(t_row + 16 * h, r0);
            tmem_ld16(t_row + 64 + 16 * h, r1);
            tmem_ld16(t_row + 128 + 16 * h, rp);
            tmem_wait_ld();
            tmem_fence_before();
            __syncwarp();
            mbar_arrive_if(lane == 0, s_free);
            float* s0 = reinterpret_cast<float*>(r0);
            float* s1 = reinterpret_cast<float*>(r1);
            const float* dp = reinterpret_cast<const float*>(rp);
            const int in = limit - j0;
            if (a.mask || !__all_sync(0xffffffffu, in >= 16)) {
                uint32_t bits = a.mask ? vis[v.st * 2 + (h >> 1)] >> (16 * (h & 1)) : 0xffffu;
                bits = in >= 16 ? bits : in <= 0 ? 0u : bits & ((1u << in) - 1u);
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    s0[c] = bits >> c & 1 ? s0[c] : -INFINITY;
                    s1[c] = bits >> c & 1 ? s1[c] : -INFINITY;
                }
            }
            uint32_t d0[8], d1[8], l0[8], l1[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                float2 p0 = __ffma2_rn(make_float2(s0[2 * c], s0[2 * c + 1]), sc2, n0);
                float2 p1 = __ffma2_rn(make_float2(s1[2 * c], s1[2 * c + 1]), sc2, n1);
                const float2 g = make_float2(dp[2 * c], dp[2 * c + 1]);
                p0 = make_float2(ex2(p0.x), ex2(p0.y));
                p1 = make_float2(ex2(p1.x), ex2(p1.y));
                es0 = __ffma2_rn(p0, g, es0);
                es1 = __ffma2_rn(p1, g, es1);
                p0 = __fmul2_rn(p0, __fadd2_rn(g, e0));
                p1 = __fmul2_rn(p1, __ffma2_rn(g, al2, e1));
                d0[c] = Elem<T>::pack2(p0.x, p0.y);
                d1[c] = Elem<T>::pack2(p1.x, p1.y);
                l0[c] = rest_of<T>(p0, d0[c]);
                l1[c] = rest_of<T>(p1, d1[c]);
            }
            // the products that read the operands of the last tile are done
            if (i > 0) ok = mbar_wait(g_done, (uint32_t)((i - 1) & 1), f.flags);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tmem_fence_after();
            tmem_st8(t_row + 192 + 8 * h, d0);
            tmem_st8(t_row + 224 + 8 * h, d1);
            tmem_st8(t_row + 256 + 8 * h, l0);
            tmem_st8(t_row + 288 + 8 * h, l1);
            tmem_wait_st();
            tmem_fence_before();
            __syncwarp();
            mbar_arrive_if(lane == 0, p_full);
        }
        if (ok && count > 0) ok = mbar_wait(g_done, (uint32_t)((count - 1) & 1), f.flags);
        __syncwarp();
        tmem_fence_after();
        // The saved outputs carry the rounding of the forward's weights; grad_k, grad_v and
        // grad_lambda, computed after this kernel, take the sums found here instead.
        esum[h * kAmRows + row] = make_float2(es0.x + es0.y, es1.x + es1.y);
        named_barrier(1, 512);
        if (h == 0 && tok < a.Lq && ok) {
            float x = 0.f, y = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                x += esum[k * kAmRows + row].x;
                y += esum[k * kAmRows + row].y;
            }
            float* r = f.rowv + attn_rowv(a, n, head, tok);
            r[2 * kRowvTile] = -x / cs;
            r[3 * kRowvTile] = -y / cs;
        }
        const float out_scale = a.scale / cs;
        T* dst = static_cast<T*>(a.gq) + (((long long)n * a.Lq + tok) * a.M + head) * 2 * a.D;
        for (int m = 0; m < 2; ++m)
            for (int c = 16 * h; c < dn; c += 64) {
                uint32_t o[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = 0u;
                if (count > 0) {
                    tmem_ld16(t_row + 320 + 64 * m + c, o);
                    tmem_wait_ld();
                }
                if (tok < a.Lq) {
                    float x[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) x[e] = __uint_as_float(o[e]) * out_scale;
#pragma unroll
                    for (int e = 0; e < 16; e += 8)
                        if (c + e < a.D) st_f32<T, 8>(dst + m * a.D + c + e, x + e);
                }
                __syncwarp();
            }
    } else if (warp == 16) {
        // ------------------------------------------------------------ producer
        bool ok = true;
        int loaded = 0;
        if (count > 0 && lane == 0) {
            mbar_arrive_expect_tx(q_full, (uint32_t)((2 + vch) * kAmQBytes));
            for (int m = 0; m < 2; ++m)
                tma_load_4d(qs + m * kAmQBytes, &f.tq, 0, head * 2 + m, q0, n, q_full);
            for (int c = 0; c < vch; ++c)
                tma_load_4d(gs + c * kAmQBytes, &f.tg, c * 64, head, q0, n, q_full);
        }
        Ring v(NS);
        for (int i = 0; i < count; ++i, v.next()) {
            const int st = v.st, j0 = i * kAmKeys;
            if (i >= NS) ok = mbar_wait(&kv_empty[st], v.phase ^ 1, f.flags);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            for (int w = 0; w < 2; ++w) {
                const uint32_t bits = attn_key_bits(a, n, j0 + 32 * w, len, lane);
                if (lane == 0) vis[st * 2 + w] = bits;
            }
            if (lane == 0) {
                unsigned char* dst = kvs + st * kvstage;
                mbar_arrive_expect_tx(&kv_full[st], (uint32_t)kvstage);
                for (int m = 0; m < 2; ++m)
                    tma_load_4d(dst + m * kAmKBytes, &f.tk, 0, kv * 2 + m, j0, n, &kv_full[st]);
                for (int c = 0; c < vch; ++c)
                    tma_load_4d(dst + (2 + c) * kAmKBytes, &f.tv, c * 64, kv, j0, n, &kv_full[st]);
            }
            __syncwarp();
            loaded = i + 1;
        }
        // leave only once the copies in flight have landed
        if (count > 0) (void)mbar_wait(q_full, 0, f.flags);
        for (int i = max(0, loaded - NS); i < loaded; ++i)
            (void)mbar_wait(&kv_full[i % NS], (uint32_t)((i / NS) & 1), f.flags);
    } else if (warp == 17) {
        // ------------------------------------------------------ scores and dP
        const TileProducts t{tmem, d_hi, umma_idesc<T>(kAmKeys, false, f.negate != 0),
                             umma_idesc<T>(kAmKeys, false, false), f.dsteps, f.vsteps};
        const uint32_t qa = (smem_u32(qs) >> 4) + lo_k, ga = (smem_u32(gs) >> 4) + lo_k;
        const uint32_t k_s = smem_u32(kvs);
        bool ok = count > 0 && mbar_wait(q_full, 0, f.flags);
        Ring v(NS);
        for (int i = 0; i < count; ++i, v.next()) {
            ok = ok && mbar_wait(&kv_clean[v.st], v.phase, f.flags);
            if (i > 0) ok = ok && mbar_wait(s_free, (uint32_t)((i - 1) & 1), f.flags);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (elect_one()) {
                tmem_fence_after();
                const uint32_t kb = ((k_s + v.st * kvstage) >> 4) + lo_k;
                t.issue(qa, ga, kb, kb + 2 * (kAmKBytes >> 4));
                umma_commit(s_full);
            }
            __syncwarp();
        }
    } else if (warp == 18) {
        // ------------------------------------------------------------- grad_q
        const uint32_t id_q = umma_idesc<T>(dn, true, false);
        const uint32_t k_s = smem_u32(kvs);
        bool ok = true;
        Ring v(NS);
        for (int i = 0; i < count; ++i, v.next()) {
            ok = mbar_wait(p_full, (uint32_t)(i & 1), f.flags);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (elect_one()) {
                tmem_fence_after();
                const uint32_t kb = ((k_s + v.st * kvstage) >> 4) + lo_k;
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int k = 0; k < 2 * (kAmKeys / 16); ++k)      // high parts, low parts
                        umma_f16_ta(tmem + 320 + 64 * m,
                                    tmem + 192 + 64 * (k >> 2) + 32 * m + 8 * (k & 3),
                                    umma_desc_of(kb + m * (kAmKBytes >> 4) + (k & 3) * (2048 >> 4),
                                                 d_hi),
                                    id_q, (i | k) != 0 ? 1u : 0u);
                umma_commit(g_done);
                umma_commit(&kv_empty[v.st]);
            }
            __syncwarp();
        }
    } else {
        // ------------------------------------------------------------- cleaner
        Ring v(NS);
        for (int i = 0; i < count; ++i, v.next()) {
            const bool ok = mbar_wait(&kv_full[v.st], v.phase, f.flags);
            if (!__all_sync(0xffffffffu, ok)) break;
            const uint32_t bits[2] = {vis[v.st * 2], vis[v.st * 2 + 1]};
            if ((bits[0] & bits[1]) != 0xffffffffu) {
                zero_hidden_rows(kvs + v.st * kvstage, kAmKBytes, 2 + vch, bits, 2, lane);
                fence_async_shared();
                __syncwarp();
            }
            if (lane == 0) mbar_arrive(&kv_clean[v.st]);
        }
    }
    tmem_fence_before();
    __syncthreads();
    if (warp == 17) {
        tmem_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;"
                     :: "r"(tmem) : "memory");
    }
}

// Key tiles: lanes are keys, columns the 64 tokens of a query tile; the tiles of
// all heads that share the key / value head follow one another.
template <typename T>
__global__ void __launch_bounds__(kAbThreads, 1)
    diff_attn_dkv_mma_kernel(const __grid_constant__ AttnBwdArgs f) {
    constexpr bool kScaled = std::is_same<T, __half>::value;
    const AttnArgs& a = f.a;
    const int NS = f.stages;
    extern __shared__ __align__(128) unsigned char am_smem[];
    unsigned char* base = am_smem + ((1024u - (smem_u32(am_smem) & 1023u)) & 1023u);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int vch = (a.Dv + 63) >> 6, dn = (a.D + 15) & ~15, dvn = (a.Dv + 15) & ~15;

    // the first key tiles see the most tokens in causal order: those of all heads start first
    const int tile = (int)(blockIdx.x / (unsigned)f.heads);
    const int nk = (int)blockIdx.x - tile * f.heads;
    const int n = nk / a.Mk, kv = nk - n * a.Mk;
    const int j0 = tile * kAmRows;
    const int len = attn_len(a, n);
    const int qtiles = (a.Lq + kAmKeys - 1) / kAmKeys;
    // tokens before this one see none of these keys
    const int first = j0 >= len ? qtiles : a.causal ? max(0, j0 - len + a.Lq) / kAmKeys : 0;
    const int per_head = max(0, qtiles - first);
    const int count = per_head * a.G;

    unsigned char* ks = base;                             // [2] chunks
    unsigned char* vs = ks + 2 * kAmQBytes;               // [vch]
    unsigned char* ps = vs + vch * kAmQBytes;             // weights: 128 keys x 64 tokens
    unsigned char* qgs = ps + kAmQBytes;                  // [NS][2 + vch]
    const int qgstage = (2 + vch) * kAmKBytes;
    float* rows = reinterpret_cast<float*>(qgs + NS * qgstage);      // [NS][4][64]
    uint64_t* k_full = reinterpret_cast<uint64_t*>(rows + NS * 4 * kRowvTile);
    uint64_t* k_clean = k_full + 1;
    uint64_t* q_full = k_clean + 1;
    uint64_t* q_empty = q_full + NS;
    uint64_t* s_full = q_empty + NS;
    uint64_t* s_free = s_full + 1;
    uint64_t* p_full = s_free + 1;
    uint64_t* g_done = p_full + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(g_done + 1);

    if (threadIdx.x == 0) {
        mbar_init(k_full, 1);
        mbar_init(k_clean, 1);
        for (int s = 0; s < NS; ++s) {
            mbar_init(&q_full[s], 1);
            mbar_init(&q_empty[s], 1);
        }
        mbar_init(s_full, 1);
        mbar_init(s_free, 16);
        mbar_init(p_full, 16);
        mbar_init(g_done, 1);
        mbar_fence_init();
    }
    if (warp == 17) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;"
                     :: "r"(smem_u32(tmem_slot)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = *tmem_slot;
    // TMEM columns: scores 0, 64; dP 128; dS of either map 192, 224; grad_k 64 a map from
    // 256; grad_v from 384
    const uint32_t d_hi = (uint32_t)(umma_desc128(0, 0) >> 32), lo_k = 16u >> 4 << 16;

    if (warp < 16) {
        // ------------------------------------------------------------- compute
        const int h = warp >> 2, quarter = warp & 3;
        const int row = quarter * 32 + lane, key = j0 + row;
        const uint32_t t_row = tmem + ((uint32_t)(quarter * 32) << 16);
        const bool seen = key < len && !(a.mask && a.mask[(long long)n * a.Lk + key]);
        // tokens from this one on see the key
        const int from = !seen ? 0x7fffffff : a.causal ? key - len + a.Lq : 0;
        const float4 scales = kScaled ? f.scales[nk] : make_float4(1.f, 1.f, 0.f, 0.f);
        const float cs = scales.x, cp = scales.y;
        const float2 sc2 = make_float2(a.scale_log2, a.scale_log2);
        const float2 cp2 = make_float2(cp, cp), cs2 = make_float2(cs, cs);
        const float2 r2 = make_float2(cs / cp, cs / cp);
        unsigned char* prow = ps + row * 128;
        bool ok = true;
        Ring v(NS);
        int head = kv * a.G, t = first;
        for (int i = 0; i < count; ++i, v.next()) {
            const float lam = Elem<T>::one(static_cast<const T*>(a.lam) + head) * cp;
            const float2 lam2 = make_float2(-lam, -lam);
            const int hidden = from - (t * kAmKeys + 16 * h);      // the first columns, hidden
            if (++t == qtiles) {
                t = first;
                ++head;
            }
            ok = mbar_wait(&q_full[v.st], v.phase, f.flags);
            ok = ok && mbar_wait(s_full, (uint32_t)(i & 1), f.flags);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tmem_fence_after();
            uint32_t r0[16], r1[16], rp[16];
            tmem_ld16(t_row + 16 * h, r0);
            tmem_ld16(t_row + 64 + 16 * h, r1);
            tmem_ld16(t_row + 128 + 16 * h, rp);
            tmem_wait_ld();
            tmem_fence_before();
            __syncwarp();
            mbar_arrive_if(lane == 0, s_free);
            float* s0 = reinterpret_cast<float*>(r0);
            float* s1 = reinterpret_cast<float*>(r1);
            const float* dp = reinterpret_cast<const float*>(rp);
            if (__any_sync(0xffffffffu, hidden > 0)) {
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    s0[c] = c >= hidden ? s0[c] : -INFINITY;
                    s1[c] = c >= hidden ? s1[c] : -INFINITY;
                }
            }
            const float* rv = rows + v.st * 4 * kRowvTile + 16 * h;
            uint32_t d0[8], d1[8], w[8];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float4 l0 = *reinterpret_cast<const float4*>(rv + 4 * c);
                const float4 l1 = *reinterpret_cast<const float4*>(rv + kRowvTile + 4 * c);
                const float4 e0 = *reinterpret_cast<const float4*>(rv + 2 * kRowvTile + 4 * c);
                const float4 e1 = *reinterpret_cast<const float4*>(rv + 3 * kRowvTile + 4 * c);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int x = 4 * c + 2 * u;
                    float2 p0 = __ffma2_rn(make_float2(s0[x], s0[x + 1]), sc2,
                                           u ? make_float2(l0.z, l0.w) : make_float2(l0.x, l0.y));
                    float2 p1 = __ffma2_rn(make_float2(s1[x], s1[x + 1]), sc2,
                                           u ? make_float2(l1.z, l1.w) : make_float2(l1.x, l1.y));
                    const float2 g = make_float2(dp[x], dp[x + 1]);
                    float2 g0 = __fadd2_rn(g, u ? make_float2(e0.z, e0.w)
                                                : make_float2(e0.x, e0.y));
                    float2 g1 = __fadd2_rn(g, u ? make_float2(e1.z, e1.w)
                                                : make_float2(e1.x, e1.y));
                    p0 = make_float2(ex2(p0.x), ex2(p0.y));
                    p1 = make_float2(ex2(p1.x), ex2(p1.y));
                    p1 = __fmul2_rn(p1, lam2);                      // -lambda P_1 cp
                    const float2 both = kScaled ? __ffma2_rn(p0, cp2, p1) : __fadd2_rn(p0, p1);
                    if (kScaled) {
                        g0 = __fmul2_rn(g0, cs2);
                        g1 = __fmul2_rn(g1, r2);
                    }
                    p0 = __fmul2_rn(p0, g0);
                    p1 = __fmul2_rn(p1, g1);
                    d0[2 * c + u] = Elem<T>::pack2(p0.x, p0.y);
                    d1[2 * c + u] = Elem<T>::pack2(p1.x, p1.y);
                    w[2 * c + u] = Elem<T>::pack2(both.x, both.y);
                }
            }
            // the products that read the operands of the last tile are done
            if (i > 0) ok = mbar_wait(g_done, (uint32_t)((i - 1) & 1), f.flags);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tmem_fence_after();
            tmem_st8(t_row + 192 + 8 * h, d0);
            tmem_st8(t_row + 224 + 8 * h, d1);
#pragma unroll
            for (int u = 0; u < 2; ++u)
                *reinterpret_cast<uint4*>(prow + (((2 * h + u) ^ (row & 7)) << 4)) =
                    make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
            fence_async_shared();
            tmem_wait_st();
            tmem_fence_before();
            __syncwarp();
            mbar_arrive_if(lane == 0, p_full);
        }
        if (ok && count > 0) ok = mbar_wait(g_done, (uint32_t)((count - 1) & 1), f.flags);
        __syncwarp();
        tmem_fence_after();
        const long long at = ((long long)n * a.Lk + key) * a.Mk + kv;
        const float k_scale = a.scale / cs, v_scale = 1.f / cp;
        // 2 dn + dvn columns from 256: grad_k of either map, grad_v
        for (int m = 0; m < 3; ++m) {
            const int cols = m < 2 ? dn : dvn, real = m < 2 ? a.D : a.Dv;
            T* dst = m < 2 ? static_cast<T*>(a.gk) + (at * 2 + m) * a.D
                           : static_cast<T*>(a.gv) + at * a.Dv;
            const float scale = m < 2 ? k_scale : v_scale;
            for (int c = 16 * h; c < cols; c += 64) {
                uint32_t o[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = 0u;
                if (count > 0) {
                    tmem_ld16(t_row + 256 + 64 * m + c, o);
                    tmem_wait_ld();
                }
                if (key < a.Lk) {
                    float x[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) x[e] = __uint_as_float(o[e]) * scale;
#pragma unroll
                    for (int e = 0; e < 16; e += 8)
                        if (c + e < real) st_f32<T, 8>(dst + c + e, x + e);
                }
                __syncwarp();
            }
        }
    } else if (warp == 16) {
        // ------------------------------------------------------------ producer
        if (lane == 0 && count > 0) {
            mbar_arrive_expect_tx(k_full, (uint32_t)((2 + vch) * kAmQBytes));
            for (int m = 0; m < 2; ++m)
                tma_load_4d(ks + m * kAmQBytes, &f.tk, 0, kv * 2 + m, j0, n, k_full);
            for (int c = 0; c < vch; ++c)
                tma_load_4d(vs + c * kAmQBytes, &f.tv, c * 64, kv, j0, n, k_full);
            bool ok = true;
            int loaded = 0, head = kv * a.G, t = first;
            Ring v(NS);
            for (int i = 0; i < count; ++i, v.next()) {
                const int st = v.st;
                if (i >= NS) ok = mbar_wait(&q_empty[st], v.phase ^ 1, f.flags);
                if (!ok) break;
                unsigned char* dst = qgs + st * qgstage;
                mbar_arrive_expect_tx(&q_full[st], (uint32_t)(qgstage + kAbRowvBytes));
                for (int m = 0; m < 2; ++m)
                    tma_load_4d(dst + m * kAmKBytes, &f.tq, 0, head * 2 + m, t * kAmKeys, n,
                                &q_full[st]);
                for (int c = 0; c < vch; ++c)
                    tma_load_4d(dst + (2 + c) * kAmKBytes, &f.tg, c * 64, head, t * kAmKeys, n,
                                &q_full[st]);
                bulk_g2s(rows + st * 4 * kRowvTile, a.rowv + attn_rowv(a, n, head, t * kAmKeys),
                         kAbRowvBytes, &q_full[st]);
                if (++t == qtiles) {
                    t = first;
                    ++head;
                }
                loaded = i + 1;
            }
            // leave only once the copies in flight have landed
            (void)mbar_wait(k_full, 0, f.flags);
            for (int i = max(0, loaded - NS); i < loaded; ++i)
                (void)mbar_wait(&q_full[i % NS], (uint32_t)((i / NS) & 1), f.flags);
        }
        __syncwarp();
    } else if (warp == 17) {
        // ------------------------------------------------------ scores and dP
        const TileProducts t{tmem, d_hi, umma_idesc<T>(kAmKeys, false, f.negate != 0),
                             umma_idesc<T>(kAmKeys, false, false), f.dsteps, f.vsteps};
        const uint32_t ka = (smem_u32(ks) >> 4) + lo_k, va = (smem_u32(vs) >> 4) + lo_k;
        const uint32_t q_s = smem_u32(qgs);
        bool ok = count > 0 && mbar_wait(k_clean, 0, f.flags);
        Ring v(NS);
        for (int i = 0; i < count; ++i, v.next()) {
            ok = ok && mbar_wait(&q_full[v.st], v.phase, f.flags);
            if (i > 0) ok = ok && mbar_wait(s_free, (uint32_t)((i - 1) & 1), f.flags);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (elect_one()) {
                tmem_fence_after();
                const uint32_t qb = ((q_s + v.st * qgstage) >> 4) + lo_k;
                t.issue(ka, va, qb, qb + 2 * (kAmKBytes >> 4));
                umma_commit(s_full);
            }
            __syncwarp();
        }
    } else if (warp == 18) {
        // ---------------------------------------------------- grad_k and grad_v
        const uint32_t id_k = umma_idesc<T>(dn, true, false);
        const uint32_t id_v = umma_idesc<T>(dvn, true, false);
        const uint32_t q_s = smem_u32(qgs), pa = (smem_u32(ps) >> 4) + lo_k;
        const uint32_t lo_v = (uint32_t)kAmKBytes >> 4 << 16;
        bool ok = true;
        Ring v(NS);
        for (int i = 0; i < count; ++i, v.next()) {
            ok = mbar_wait(p_full, (uint32_t)(i & 1), f.flags);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (elect_one()) {
                tmem_fence_after();
                const uint32_t qb = (q_s + v.st * qgstage) >> 4;
#pragma unroll
                for (int k = 0; k < kAmKeys / 16; ++k)
                    umma_f16(tmem + 384, umma_desc_of(pa + 2 * k, d_hi),
                             umma_desc_of(qb + lo_v + 2 * (kAmKBytes >> 4) + k * (2048 >> 4), d_hi),
                             id_v, (i | k) != 0 ? 1u : 0u);
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int k = 0; k < kAmKeys / 16; ++k)
                        umma_f16_ta(tmem + 256 + 64 * m, tmem + 192 + 32 * m + 8 * k,
                                    umma_desc_of(qb + lo_k + m * (kAmKBytes >> 4) +
                                                     k * (2048 >> 4), d_hi),
                                    id_k, (i | k) != 0 ? 1u : 0u);
                umma_commit(g_done);
                umma_commit(&q_empty[v.st]);
            }
            __syncwarp();
        }
    } else {
        // ------------------------------------------------- cleaner, once a CTA
        if (count > 0) {
            const bool ok = mbar_wait(k_full, 0, f.flags);
            if (__all_sync(0xffffffffu, ok)) {
                uint32_t bits[4];
                for (int w = 0; w < 4; ++w) bits[w] = attn_key_bits(a, n, j0 + 32 * w, len, lane);
                if ((bits[0] & bits[1] & bits[2] & bits[3]) != 0xffffffffu) {
                    zero_hidden_rows(ks, kAmQBytes, 2 + vch, bits, 4, lane);
                    fence_async_shared();
                    __syncwarp();
                }
                if (lane == 0) mbar_arrive(k_clean);
            }
        }
    }
    tmem_fence_before();
    __syncthreads();
    if (warp == 17) {
        tmem_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;"
                     :: "r"(tmem) : "memory");
    }
}

}  // namespace dcnb
