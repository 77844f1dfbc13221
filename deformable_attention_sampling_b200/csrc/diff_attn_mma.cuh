// Differential attention on the tensor cores (tcgen05, accumulators in TMEM),
// forward, 16-bit types (sm_100a).  The mathematics is diff_attn.cuh's.
//
// One CTA owns 128 tokens of one head and walks the keys in tiles of 64, with
// both softmax maps in flight, each with its own issuing warp:
//   producer (one warp)     tensor-map loads of the tokens' two query tiles,
//             then per tile the two key tiles and the value tile (128-byte
//             swizzle, rows past the tensor read as zeros);
//   MMA       (a warp a map)  S_m = Q_m K_m^T (float32, 64 TMEM columns), and
//             O_m += P_m V, P_m as the left operand from TMEM, V from the
//             shared tile as it lies (N-major);
//   softmax   (four warps a map, thread = token) reads its row of S_m, keeps
//             the running maximum and sum, writes P_m in 16 bits;
//   cleaner   (one warp)     zeroes the value rows of hidden keys.
// S_m(i + 1) is computed as soon as the softmax warps hold S_m(i) in registers,
// while they work on it; P_m has two buffers, so that they do not wait for the
// value product either.  TMEM: a map's scores 64 columns and weights 2 x 32,
// O_0, O_1 up to 128 columns each: all 512.
//
// The running maximum is lowered into O only when it has grown by more than
// 2^8 (the weights stay below 2^8 then, or 2^14 with fp16's bias): O_m lives in
// TMEM, and a rescale is a round trip through registers that nearly no tile
// needs.  fp16 weights carry a factor 2^6, so that weights down to 2^-20 of
// the largest stay normal numbers.  Weights enter the product rounded to the
// type (half a step of the type each), their sum is that of the unrounded ones:
// the outputs' root mean square error is 1.35 times that of rounding them once.
//
// Keys that no token may see (past the length, masked) get weight 0, and their
// value rows are zeroed in the tile first: 0 times what lies there must not be
// NaN.
//
// Bound: per 128 x 64 tile and map the exponentials take 512 cycles of the
// special-function units and the products 470 (D = 64, Dv = 128: measured 53
// cycles a 128 x 64 x 16 step from shared memory, 64 a 128 x 128 x 16 step from
// TMEM).  Measured: 477 us on one prompt of 8192 tokens, 16 heads of 64 + 128
// (864 TFLOP/s; the products alone take 249 us at the measured bf16 rate, the
// exponentials 239 us); a pair of tiles takes about 1960 cycles, of which the
// steps of a softmax warp that follow one another (two waits, load, maximum,
// exponentials, store) are the longest chain.
// Tried and slower on that prompt (469 us then): strict turns of the maps at the
// exponentials (502), a third of the exponentials by polynomial on the FMA units
// (512), two sets of softmax warps a map with P in shared memory (549), scores and
// value products of both maps each from one polling warp (517).  128-key tiles with
// P over S were timed only with the first way of issuing (one warp, a descriptor
// built for every product): 655 us, where 64-key tiles took 946.
#pragma once

#include "diff_attn.cuh"
#include "tmem.cuh"

namespace dcnb {

constexpr int kAmRows = 128;                 // tokens of a CTA
constexpr int kAmKeys = 64;                  // keys of a tile
constexpr int kAmThreads = 384;              // 2 x 4 softmax warps, producer, 2 MMA, cleaner
constexpr int kAmQBytes = kAmRows * 128;     // 64 columns of the query tile, of a
constexpr int kAmKBytes = kAmKeys * 128;     // key or value tile (16-bit elements)
constexpr int kAmMaxDv = 128;                // value columns of a CTA
constexpr float kAmLazy = 8.f;

struct AttnMmaArgs {
    CUtensorMap tq;            // [N][Lq][2 M][D], box {64, 1, 128, 1}
    CUtensorMap tk;            // [N][Lk][2 Mk][D], box {64, 1, 64, 1}
    CUtensorMap tv;            // [N][Lk][Mk][Dv], likewise
    AttnArgs a;
    unsigned int* flags;
    int dsteps;                // K = 16 steps of a head
    int dv_parts;              // CTAs that share a head's value columns
    int stages;
    int negate;                // the scale is negative
    int heads;                 // N * M
};

// Position in a ring of stages and the parity of the round.
struct Ring {
    int n, st;
    uint32_t phase;
    __device__ __forceinline__ explicit Ring(int stages) : n(stages), st(0), phase(0) {}
    __device__ __forceinline__ void next() {
        if (++st == n) {
            st = 0;
            phase ^= 1;
        }
    }
};

// Bits of the 32 keys from j on that some token may see.
__device__ __forceinline__ uint32_t attn_key_bits(const AttnArgs& a, int n, int j, int len,
                                                  int lane) {
    const int key = j + lane;
    const bool ok = key < len && !(a.mask && a.mask[(long long)n * a.Lk + key]);
    return __ballot_sync(0xffffffffu, ok);
}

__host__ __device__ constexpr int attn_mma_smem(int dchunks, int vchunks, int stages) {
    return 1024 + 2 * dchunks * kAmQBytes + stages * (2 * dchunks + vchunks) * kAmKBytes + 4096;
}

// DCH: 64-column chunks of a head (the 16-column steps past D are skipped).
template <typename T, int DCH>
__global__ void __launch_bounds__(kAmThreads, 1)
    diff_attn_mma_kernel(const __grid_constant__ AttnMmaArgs f) {
    constexpr float kBias = std::is_same<T, __half>::value ? 6.f : 0.f;
    const AttnArgs& a = f.a;
    const int NS = f.stages;
    extern __shared__ __align__(128) unsigned char am_smem[];
    unsigned char* base = am_smem + ((1024u - (smem_u32(am_smem) & 1023u)) & 1023u);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    const int part = (int)blockIdx.y % f.dv_parts, split = (int)blockIdx.y / f.dv_parts;
    const int c0 = part * kAmMaxDv;
    const int dv = min(a.Dv - c0, kAmMaxDv);         // value columns of this CTA
    const int dvn = (dv + 15) & ~15;                 // N of the value product
    const int vch = (dv + 63) >> 6;
    // in causal order the last tiles see the most keys: those of all heads start first
    const int tile = (int)(blockIdx.x / (unsigned)f.heads);
    const int nh = (int)blockIdx.x - tile * f.heads;
    const int n = nh / a.M, head = nh - n * a.M, kv = head / a.G;
    const int q0 = ((int)(gridDim.x / (unsigned)f.heads) - 1 - tile) * kAmRows;
    const int len = attn_len(a, n);
    const int last = min(q0 + kAmRows, a.Lq) - 1;
    const int kmax = a.causal ? max(0, min(len, last + len - a.Lq + 1)) : len;
    const int tiles = (kmax + kAmKeys - 1) / kAmKeys;
    const int t0 = (int)((long long)tiles * split / a.splits);
    const int t1 = (int)((long long)tiles * (split + 1) / a.splits);
    const int count = t1 - t0;

    unsigned char* qs = base;                                   // [2][DCH] chunks
    unsigned char* ks = qs + 2 * DCH * kAmQBytes;               // [NS][2][DCH]
    unsigned char* vs = ks + NS * 2 * DCH * kAmKBytes;          // [NS][vch of the launch]
    const int vstage = ((min(a.Dv, kAmMaxDv) + 63) >> 6) * kAmKBytes;
    uint64_t* bars = reinterpret_cast<uint64_t*>(vs + NS * vstage);
    uint64_t* q_full = bars;
    uint64_t* k_full = q_full + 1;
    uint64_t* k_empty = k_full + NS;
    uint64_t* v_full = k_empty + NS;
    uint64_t* v_empty = v_full + NS;
    uint64_t* v_clean = v_empty + NS;     // value tile ready, hidden rows zeroed
    uint64_t* s_full = v_clean + NS;      // [map] scores written
    uint64_t* s_free = s_full + 2;        // [map] scores read
    uint64_t* p_full = s_free + 2;        // [map][buffer] weights written
    uint64_t* o_done = p_full + 4;        // [map][buffer] value product done
    uint64_t* lead_off = o_done + 4;      // map 0 has its first weights
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(lead_off + 1);
    uint32_t* vis = tmem_slot + 4;                                // [NS][2] key bits of a tile
    float* inv = reinterpret_cast<float*>(vis + NS * 2);          // [2][128]

    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(lead_off, 4);
        for (int s = 0; s < NS; ++s) {
            mbar_init(&k_full[s], 1);
            mbar_init(&k_empty[s], 2);
            mbar_init(&v_full[s], 1);
            mbar_init(&v_empty[s], 2);
            mbar_init(&v_clean[s], 1);
        }
        for (int m = 0; m < 2; ++m) {
            mbar_init(&s_full[m], 1);
            mbar_init(&s_free[m], 4);
        }
        for (int m = 0; m < 4; ++m) {
            mbar_init(&p_full[m], 4);
            mbar_init(&o_done[m], 1);
        }
        mbar_fence_init();
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;"
                     :: "r"(smem_u32(tmem_slot)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp < 8) {
        // ------------------------------------------------------------- softmax
        const int m = warp >> 2, quarter = warp & 3;
        const int row = quarter * 32 + lane, tok = q0 + row;
        const uint32_t t_row = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t t_s = t_row + m * 128, t_o = t_row + 256 + m * 128;
        const int limit = a.causal ? min(len, tok + len - a.Lq + 1) : len;
        const float sc = a.scale_log2;
        float top = -INFINITY, sum = 0.f;        // reference maximum of the weights, their sum
        bool ok = true;
        uint32_t r[64];
        float* s = reinterpret_cast<float*>(r);
        // The scores of tile i on their way to registers.  Their barrier counts every product
        // that map's warp issued before: the weights of tile i - 2 have been read, too.
        // `early`: found complete before (a wait costs 100 cycles even when it is over).
        auto fetch = [&](int i, bool early) {
            if (!__all_sync(0xffffffffu, early)) {
                ok = mbar_wait(&s_full[m], (uint32_t)(i & 1), f.flags);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) return;
            }
            tmem_fence_after();
            tmem_ld32(t_s, r);
            tmem_ld32(t_s + 32, r + 32);
        };
        if (count > 0) fetch(0, false);
        Ring v(NS);
        for (int i = 0; i < count && ok; ++i, v.next()) {
            const int st = v.st, buf = m * 2 + (i & 1), j0 = (t0 + i) * kAmKeys;
            if (a.mask) {          // its key bits
                ok = mbar_wait(&v_full[st], v.phase, f.flags);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
            }
            tmem_wait_ld();
            tmem_fence_before();
            __syncwarp();
            mbar_arrive_if(lane == 0, &s_free[m]);
            const int cnt = limit - j0;
            if (!__all_sync(0xffffffffu, cnt >= kAmKeys) || a.mask) {
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    uint32_t bits = a.mask ? vis[st * 2 + w] : 0xffffffffu;
                    const int in = cnt - 32 * w;
                    bits = in >= 32 ? bits : in <= 0 ? 0u : bits & ((1u << in) - 1u);
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        s[32 * w + c] = bits >> c & 1 ? s[32 * w + c] : -INFINITY;
                }
            }
            float mx[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) mx[c] = max3(s[3 * c], s[3 * c + 1], s[3 * c + 2]);
#pragma unroll
            for (int c = 12; c + 1 < kAmKeys; c += 2)
                mx[c / 2 & 3] = max3(mx[c / 2 & 3], s[c], s[c + 1]);
            const float hi = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * sc - kBias;
            const bool first = top == -INFINITY;
            const bool grow = !first && hi > top + kAmLazy;
            if (__any_sync(0xffffffffu, grow)) {
                // the last value product has to be in O_m
                ok = mbar_wait(&o_done[buf ^ 1], (uint32_t)(((i - 1) >> 1) & 1), f.flags);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tmem_fence_after();
                const float keep = grow ? ex2(top - hi) : 1.f;
                for (int c = 0; c < dvn; c += 16) {
                    uint32_t o[16];
                    tmem_ld16(t_o + c, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        o[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
                    tmem_st16(t_o + c, o);
                }
                sum *= keep;
                if (grow) top = hi;
            }
            if (first) top = hi;
            const float ref = top == -INFINITY ? 0.f : top;
            const float2 sc2 = make_float2(sc, sc), rf2 = make_float2(-ref, -ref);
            float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            uint32_t p[32];
            bool early = false;
#pragma unroll
            for (int c = 0; c < 32; ++c) {
                if (c == 24) early = mbar_test(&s_full[m], (uint32_t)((i + 1) & 1));
                float2 x = __ffma2_rn(make_float2(s[2 * c], s[2 * c + 1]), sc2, rf2);
                x.x = ex2(x.x);
                x.y = ex2(x.y);
                acc[c & 1] = __fadd2_rn(acc[c & 1], x);
                p[c] = Elem<T>::pack2(x.x, x.y);
            }
            tmem_st32(t_s + 64 + 32 * (i & 1), p);
            if (i + 1 < count) fetch(i + 1, early);
            sum += (acc[0].x + acc[1].x) + (acc[0].y + acc[1].y);
            tmem_wait_st();
            tmem_fence_before();
            __syncwarp();
            mbar_arrive_if(lane == 0, &p_full[buf]);
            if (m == 0 && i == 0) mbar_arrive_if(lane == 0, lead_off);
        }
        // ------------------------------------------------------------ epilogue
        if (count > 0) {
            const int b = (count - 1) & 1;
            const uint32_t ph = (uint32_t)(((count - 1) >> 1) & 1);
            ok = ok && mbar_wait(&o_done[b], ph, f.flags) && mbar_wait(&o_done[2 + b], ph, f.flags);
        }
        __syncwarp();
        tmem_fence_after();
        inv[m * 128 + row] = sum > 0.f ? 1.f / sum : 0.f;
        const bool live = tok < a.Lq;
        const bool lead = part == 0 && live;
        const long long rows_total = (long long)a.N * a.M * a.Lq;
        // packed row of the join kernel: token * G + head within its group
        const long long at = (long long)split * rows_total +
                             ((long long)n * a.Mk + kv) * a.rows + (long long)tok * a.G + head -
                             kv * a.G;
        if (a.splits > 1) {
            if (lead) {
                a.part_ml[(at * 2 + m) * 2] = top;
                a.part_ml[(at * 2 + m) * 2 + 1] = sum;
            }
        } else if (a.lse && lead) {
            a.lse[(((long long)n * a.M + head) * 2 + m) * a.Lq + tok] =
                sum > 0.f ? top + log2f(sum) : INFINITY;
        }
        named_barrier(1, 256);
        const float i0 = inv[row], i1 = inv[128 + row];
        const float lam = Elem<T>::one(static_cast<const T*>(a.lam) + head);
        const long long to = (((long long)n * a.Lq + tok) * a.M + head) * a.Dv + c0;
        for (int c = 16 * m; c < dvn; c += 32) {
            uint32_t o0[16], o1[16];
            if (count > 0) {
                tmem_ld16(t_row + 256 + c, o0);
                tmem_ld16(t_row + 384 + c, o1);
                tmem_wait_ld();
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) o0[e] = o1[e] = 0u;
            }
            if (live && a.splits > 1) {
#pragma unroll
                for (int e = 0; e < 16; e += 4)
                    if (c + e < dv) {
                        float* d = a.part_o + at * 2 * a.Dv + c0 + c + e;
                        *reinterpret_cast<uint4*>(d) =
                            make_uint4(o0[e], o0[e + 1], o0[e + 2], o0[e + 3]);
                        *reinterpret_cast<uint4*>(d + a.Dv) =
                            make_uint4(o1[e], o1[e + 1], o1[e + 2], o1[e + 3]);
                    }
            } else if (live) {
                float x[16], y[16], z[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    x[e] = __fmul_rn(__uint_as_float(o0[e]), i0);
                    y[e] = __fmul_rn(__uint_as_float(o1[e]), i1);
                    z[e] = attn_diff(x[e], lam, y[e]);
                }
#pragma unroll
                for (int e = 0; e < 16; e += 8)
                    if (c + e < dv) {
                        st_f32<T, 8>(static_cast<T*>(a.out) + to + c + e, z + e);
                        if (a.maps) {
                            float* d = a.maps + 2 * to - c0 + c + e;
                            st_f32<float, 4>(d, x + e);
                            st_f32<float, 4>(d + 4, x + e + 4);
                            st_f32<float, 4>(d + a.Dv, y + e);
                            st_f32<float, 4>(d + a.Dv + 4, y + e + 4);
                        }
                    }
            }
            __syncwarp();
        }
    } else if (warp == 8) {
        // ------------------------------------------------------------ producer
        bool ok = true;
        int loaded = 0;
        if (count > 0 && lane == 0) {
            mbar_arrive_expect_tx(q_full, (uint32_t)(2 * DCH * kAmQBytes));
            for (int m = 0; m < 2; ++m)
                for (int c = 0; c < DCH; ++c)
                    tma_load_4d(qs + (m * DCH + c) * kAmQBytes, &f.tq, c * 64, head * 2 + m, q0, n,
                                q_full);
        }
        Ring v(NS);
        for (int i = 0; i < count; ++i, v.next()) {
            const int st = v.st, j0 = (t0 + i) * kAmKeys;
            const uint32_t ph = v.phase ^ 1;
            if (i >= NS) ok = mbar_wait(&k_empty[st], ph, f.flags);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(&k_full[st], (uint32_t)(2 * DCH * kAmKBytes));
                for (int m = 0; m < 2; ++m)
                    for (int c = 0; c < DCH; ++c)
                        tma_load_4d(ks + ((st * 2 + m) * DCH + c) * kAmKBytes, &f.tk, c * 64,
                                    kv * 2 + m, j0, n, &k_full[st]);
            }
            if (i >= NS) ok = mbar_wait(&v_empty[st], ph, f.flags);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            for (int w = 0; w < 2; ++w) {
                const uint32_t bits = attn_key_bits(a, n, j0 + 32 * w, len, lane);
                if (lane == 0) vis[st * 2 + w] = bits;
            }
            if (lane == 0) {
                mbar_arrive_expect_tx(&v_full[st], (uint32_t)(vch * kAmKBytes));
                for (int c = 0; c < vch; ++c)
                    tma_load_4d(vs + st * vstage + c * kAmKBytes, &f.tv, c0 + c * 64, kv, j0, n,
                                &v_full[st]);
            }
            __syncwarp();
            loaded = i + 1;
        }
        // leave only once the copies in flight have landed
        if (count > 0) (void)mbar_wait(q_full, 0, f.flags);
        for (int i = max(0, loaded - NS); i < loaded; ++i) {
            (void)mbar_wait(&k_full[i % NS], (uint32_t)((i / NS) & 1), f.flags);
            (void)mbar_wait(&v_full[i % NS], (uint32_t)((i / NS) & 1), f.flags);
        }
    } else if (warp < 11) {
        // ------------------------------------------------------- MMA of one map
        const int m = warp - 9;
        const uint32_t id_s = umma_idesc<T>(kAmKeys, false, f.negate != 0);
        const uint32_t id_o = umma_idesc<T>(dvn, true, false);
        // descriptors: the start address and the leading offset in the low word
        const uint32_t d_hi = (uint32_t)(umma_desc128(0, 0) >> 32);
        const uint32_t lo_k = 16u >> 4 << 16, lo_v = (uint32_t)kAmKBytes >> 4 << 16;
        const uint32_t qa = ((smem_u32(qs) + m * DCH * kAmQBytes) >> 4) + lo_k;
        const uint32_t k_s = smem_u32(ks), v_s = smem_u32(vs);
        const uint32_t t_s = tmem + m * 128, t_o = tmem + 256 + m * 128;
        auto scores = [&](int st) {
            const uint32_t kb = ((k_s + (st * 2 + m) * DCH * kAmKBytes) >> 4) + lo_k;
#pragma unroll
            for (int k = 0; k < 4 * DCH; ++k)
                if (k < f.dsteps)
                    umma_f16(t_s,
                             umma_desc_of(qa + (k >> 2) * (kAmQBytes >> 4) + 2 * (k & 3), d_hi),
                             umma_desc_of(kb + (k >> 2) * (kAmKBytes >> 4) + 2 * (k & 3), d_hi),
                             id_s, k != 0 ? 1u : 0u);
            umma_commit(&s_full[m]);
            umma_commit(&k_empty[st]);
        };
        Ring kr(NS), v(NS);
        bool ok = count > 0 && mbar_wait(q_full, 0, f.flags) && mbar_wait(&k_full[0], 0, f.flags);
        // half a tile apart, the maps' warps take turns at the exponentials
        if (m == 1) ok = ok && mbar_wait(lead_off, 0, f.flags);
        ok = __all_sync(0xffffffffu, ok);
        if (ok && elect_one()) {
            tmem_fence_after();
            scores(0);
        }
        __syncwarp();
        kr.next();
        for (int i = 0; i < count && ok; ++i, v.next(), kr.next()) {
            const int st = v.st, buf = m * 2 + (i & 1);
            if (i + 1 < count) {
                ok = mbar_wait(&k_full[kr.st], kr.phase, f.flags) &&
                     mbar_wait(&s_free[m], (uint32_t)(i & 1), f.flags);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (elect_one()) {
                    tmem_fence_after();
                    scores(kr.st);
                }
                __syncwarp();
            }
            ok = mbar_wait(&v_clean[st], v.phase, f.flags) &&
                 mbar_wait(&p_full[buf], (uint32_t)((i >> 1) & 1), f.flags);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (elect_one()) {
                tmem_fence_after();
                const uint32_t vb = ((v_s + st * vstage) >> 4) + lo_v;
                const uint32_t t_p = t_s + 64 + 32 * (i & 1);
#pragma unroll
                for (int k = 0; k < kAmKeys / 16; ++k)
                    umma_f16_ta(t_o, t_p + k * 8, umma_desc_of(vb + k * (2048 >> 4), d_hi), id_o,
                                (i | k) != 0 ? 1u : 0u);
                umma_commit(&o_done[buf]);
                umma_commit(&v_empty[st]);
            }
            __syncwarp();
        }
    } else {
        // ------------------------------------------------------------- cleaner
        Ring v(NS);
        for (int i = 0; i < count; ++i, v.next()) {
            const int st = v.st;
            const bool ok = mbar_wait(&v_full[st], v.phase, f.flags);
            if (!__all_sync(0xffffffffu, ok)) break;
            const uint32_t vis0 = vis[st * 2], vis1 = vis[st * 2 + 1];
            if ((vis0 & vis1) != 0xffffffffu) {
                for (int w = 0; w < 2; ++w) {
                    const uint32_t hidden = ~(w ? vis1 : vis0);
                    // 8 lanes a row of a chunk, 4 rows at a time
                    for (int r = lane >> 3; r < 32; r += 4)
                        if (hidden >> r & 1)
                            for (int c = 0; c < vch; ++c)
                                *reinterpret_cast<uint4*>(vs + st * vstage + c * kAmKBytes +
                                                          (w * 32 + r) * 128 + (lane & 7) * 16) =
                                    make_uint4(0, 0, 0, 0);
                }
                fence_async_shared();
                __syncwarp();
            }
            if (lane == 0) mbar_arrive(&v_clean[st]);
        }
    }
    tmem_fence_before();
    __syncthreads();
    if (warp == 9) {
        tmem_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;"
                     :: "r"(tmem) : "memory");
    }
}

}  // namespace dcnb
