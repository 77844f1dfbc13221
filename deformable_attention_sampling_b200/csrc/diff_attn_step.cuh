// Differential attention of a few new tokens over a long cache, 16-bit types
// (sm_100a).  The mathematics is diff_attn.cuh's.
//
// Bound: the key and value bytes.  So every key and value is read once, from
// global memory straight into the registers of matrix instructions
// (mma.sync m16n8k16; tcgen05's 128 rows would be empty), and no lane reads what another loaded.
// A warp owns 8 packed rows (the tokens and heads that share a key / value
// head) and walks blocks of 16 keys.  The two maps sit in one 16-row tile:
//   scores   rows 0-7 = Q_0 K_0^T, rows 8-15 = Q_1 K_1^T: map 0's product has
//            zeros in rows 8-15 of its left operand, map 1's in rows 0-7, and
//            both add into one accumulator;
//   values   the 16 x 16 weights of both maps times one value block.
// A contraction may run over its index in any order, so lane (g, t) = (lane / 4,
// lane % 4) takes every fourth 16-byte piece of key g, whatever channels the
// instruction means by them, and every eighth piece of its four keys' values,
// paired by byte permutes: neighbouring lanes read neighbouring pieces, and no
// sector is fetched twice.
// A warp's next block is on its way to shared memory (cp.async, each lane its own
// pieces, so no barrier) while it works on this one.
// Measured: 49 us for 16 caches of 4096 to 8192 keys, 4 key / value heads of 64 +
// 128 (201 MB: 4.1 TB/s; 31 us at the measured copy rate), 10 us for the join.
// Held by a warp's chain of loads, 8 dependent score products and shuffles: the
// time hardly depends on the split (4 to 27 parts: 57 to 64 us with the join).
// Weights enter the value product rounded to the type, as in diff_attn_mma.cuh.
// The keys are split over CTAs (and the 4 warps of a CTA, which join in shared
// memory); diff_attn_join_kernel adds the CTAs' parts in a fixed order.
#pragma once

#include "diff_attn.cuh"
#include "tmem.cuh"

namespace dcnb {

constexpr int kAsWarps = 4;
constexpr int kAsThreads = 32 * kAsWarps;
constexpr int kAsRows = 8;             // packed rows of a CTA
constexpr int kAsKeys = 16;            // keys of a warp's block

template <typename T>
__device__ __forceinline__ void mma_16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same<T, __half>::value) {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    } else {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    }
}

// W words from p, 16-byte pieces 64 bytes apart; zeros unless ok.
template <int W>
__device__ __forceinline__ void ld_row_words(const void* p, bool ok, uint32_t* w) {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = 0u;
    if (ok) {
#pragma unroll
        for (int i = 0; i < W; i += 4) load_vec<16>(static_cast<const char*>(p) + 16 * i, w + i);
    }
}

// Asynchronous copy of VB bytes to shared memory; zeros unless ok.
template <int VB>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool ok) {
    const int n = ok ? VB : 0;
    if constexpr (VB == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                     :: "r"(dst), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;"
                     :: "r"(dst), "l"(src), "r"(n) : "memory");
}

// Bytes of a warp's block in shared memory: a lane's 16-byte pieces of two keys of
// both maps and of four value rows.
__host__ __device__ constexpr int attn_step_block(int D, int Dv) {
    return (4 * (D / 32) + 4 * (Dv >= 64 ? Dv / 64 : 1)) * 512;
}
constexpr int kAsStages = 2;

// The ring of the warps' blocks; the join of the warps takes its place afterwards.
__host__ __device__ constexpr int attn_step_smem(int D, int Dv) {
    const int ring = kAsWarps * kAsStages * attn_step_block(D, Dv);
    const int join = kAsWarps * 16 * (Dv + 2) * 4;
    return ring > join ? ring : join;
}

template <typename T, int D, int DV>
__global__ void __launch_bounds__(kAsThreads,
                                  D == 128 && DV == 128 ? 2 : DV <= 64 && D <= 64 ? 4 : 3)
    diff_attn_step_kernel(const AttnArgs a) {
    constexpr float kBias = std::is_same<T, __half>::value ? 6.f : 0.f;
    constexpr int KW = D / 8;              // words of a lane's channels of a key
    constexpr int CPG = DV / 8;            // value channels of a lane
    constexpr int VW = CPG / 2;
    constexpr int KS = D / 16;             // steps of 16 of the score product
    extern __shared__ __align__(16) float as_smem[];      // [warps][16][DV + 2]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int n = (int)a.div_Mk.div(blockIdx.y), kv = (int)blockIdx.y - n * a.Mk;
    const int split = blockIdx.z, r0 = (int)blockIdx.x * kAsRows;
    const int len = attn_len(a, n);
    const int last_tok = (int)a.div_G.div((uint32_t)min(r0 + kAsRows - 1, a.rows - 1));
    const int kmax = a.causal ? max(0, min(len, last_tok + len - a.Lq + 1)) : len;
    const int blocks = (kmax + kAsKeys - 1) / kAsKeys;
    const int b0 = (int)((long long)blocks * split / a.splits);
    const int b1 = (int)((long long)blocks * (split + 1) / a.splits);

    // the lane's query channels: row g, both maps
    uint32_t q[2][2 * KS];
    const int row = r0 + g;
    const uint32_t tok = a.div_G.div((uint32_t)min(row, a.rows - 1));
    const int head = kv * a.G + min(row, a.rows - 1) - (int)tok * a.G;
    const int limit = a.causal ? min(len, (int)tok + len - a.Lq + 1) : len;
#pragma unroll
    for (int m = 0; m < 2; ++m)
        ld_row_words<KW>(static_cast<const T*>(a.q) + n * a.q_image + (long long)tok * a.q_row +
                             ((long long)head * 2 + m) * D + t * 8,
                         row < a.rows, q[m]);
    const T* kb = static_cast<const T*>(a.k) + n * a.k_image + (long long)kv * 2 * D + t * 8;
    const T* vb = static_cast<const T*>(a.v) + n * a.v_image + (long long)kv * DV +
                  g * (CPG < 8 ? CPG : 8);
    const unsigned char* mask = a.mask ? a.mask + (long long)n * a.Lk : nullptr;

    float o[CPG][4], top[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < CPG; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    const float sc = a.scale_log2;
    constexpr int KP = KW / 4, VP = VW >= 4 ? VW / 4 : 1;      // 16-byte pieces
    constexpr int VB = VW >= 4 ? 16 : 8;
    const uint32_t ring = smem_u32(as_smem) +
                          (uint32_t)(warp * kAsStages * attn_step_block(D, DV) + lane * 16);
    // which of keys 2t, 2t + 1, 2t + 8, 2t + 9 some token may see
    auto keys_seen = [&](int j0) {
        uint32_t seen = 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int key = j0 + 2 * t + (u & 1) + 8 * (u >> 1);
            seen |= (uint32_t)(key < len && !(mask && mask[key])) << u;
        }
        return seen;
    };
    auto fetch = [&](int b, int stage) {
        if (b < b1) {
            const int j0 = b * kAsKeys;
            uint32_t dst = ring + (uint32_t)(stage * attn_step_block(D, DV));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int key = j0 + 8 * h + g;
                const bool ok = key < len;
                const T* p = kb + (long long)(ok ? key : j0) * a.k_row;
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int i = 0; i < KP; ++i, dst += 512)
                        copy_async<16>(dst, p + m * D + 32 * i, ok);
            }
            const uint32_t seen = keys_seen(j0);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const bool ok = seen >> u & 1;
                const T* p = vb + (long long)(ok ? j0 + 2 * t + (u & 1) + 8 * (u >> 1) : j0) *
                                      a.v_row;
#pragma unroll
                for (int i = 0; i < VP; ++i, dst += 512) copy_async<VB>(dst, p + 64 * i, ok);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    fetch(b0 + warp, 0);
    int stage = 0;
    for (int b = b0 + warp; b < b1; b += kAsWarps, stage ^= 1) {
        const int j0 = b * kAsKeys;
        fetch(b + kAsWarps, stage ^ 1);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        uint32_t kw[2][2][KW], vw[4][VP * 4];
        uint32_t src = ring + (uint32_t)(stage * attn_step_block(D, DV));
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int i = 0; i < KP; ++i, src += 512) lds128(src, kw[h][m] + 4 * i);
        const uint32_t seen = keys_seen(j0);
        float s[2][4];                     // keys 2t, 2t + 1 (+ 8) of map 0's row, map 1's row
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            s[h][0] = s[h][1] = s[h][2] = s[h][3] = 0.f;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                mma_16816<T>(s[h], q[0][2 * k], 0u, q[0][2 * k + 1], 0u, kw[h][0][2 * k],
                             kw[h][0][2 * k + 1]);
                mma_16816<T>(s[h], 0u, q[1][2 * k], 0u, q[1][2 * k + 1], kw[h][1][2 * k],
                             kw[h][1][2 * k + 1]);
            }
        }
        float hi[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const bool ok = (seen >> u & 1) && j0 + 2 * t + (u & 1) + 8 * (u >> 1) < limit;
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                float& x = s[u >> 1][2 * m + (u & 1)];
                x = ok ? x * sc : -INFINITY;
                hi[m] = fmaxf(hi[m], x);
            }
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            hi[m] = fmaxf(hi[m], __shfl_xor_sync(0xffffffffu, hi[m], 1));
            hi[m] = fmaxf(hi[m], __shfl_xor_sync(0xffffffffu, hi[m], 2)) - kBias;
        }
        // the reference moves only when a score has outgrown it by 2^8
        const bool grow0 = hi[0] > top[0] + 8.f, grow1 = hi[1] > top[1] + 8.f;
        const bool none0 = top[0] == -INFINITY, none1 = top[1] == -INFINITY;
        if (__any_sync(0xffffffffu, grow0 || grow1 || none0 || none1)) {
            const float k0 = grow0 && !none0 ? ex2(top[0] - hi[0]) : 1.f;
            const float k1 = grow1 && !none1 ? ex2(top[1] - hi[1]) : 1.f;
            if (grow0 || none0) top[0] = hi[0];
            if (grow1 || none1) top[1] = hi[1];
            sum[0] *= k0;
            sum[1] *= k1;
#pragma unroll
            for (int j = 0; j < CPG; ++j) {
                o[j][0] *= k0;
                o[j][1] *= k0;
                o[j][2] *= k1;
                o[j][3] *= k1;
            }
        }
        const float ref[2] = {top[0] == -INFINITY ? 0.f : top[0],
                              top[1] == -INFINITY ? 0.f : top[1]};
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int i = 0; i < VP; ++i, src += 512) lds128(src, vw[u] + 4 * i);
        uint32_t p[2][2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const float x = ex2(s[h][2 * m] - ref[m]), y = ex2(s[h][2 * m + 1] - ref[m]);
                sum[m] += x + y;
                p[h][m] = Elem<T>::pack2(x, y);
            }
#pragma unroll
        for (int j = 0; j < CPG; ++j) {
            const uint32_t sel = j & 1 ? 0x7632u : 0x5410u;
            mma_16816<T>(o[j], p[0][0], p[0][1], p[1][0], p[1][1],
                         __byte_perm(vw[0][j >> 1], vw[1][j >> 1], sel),
                         __byte_perm(vw[2][j >> 1], vw[3][j >> 1], sel));
        }
    }
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        sum[m] += __shfl_xor_sync(0xffffffffu, sum[m], 1);
        sum[m] += __shfl_xor_sync(0xffffffffu, sum[m], 2);
    }
    __syncthreads();                       // every warp is done with the ring
    // the warps' parts: 16 rows of DV sums, the reference and the sum of weights
    float* mine = as_smem + warp * 16 * (DV + 2);
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        float* r = mine + (8 * m + g) * (DV + 2);
#pragma unroll
        for (int j = 0; j < CPG; ++j) {
            constexpr int PC = CPG < 8 ? CPG : 8;              // channels of a piece
            const int at = (j / PC) * 8 * PC + j % PC;
            r[at + PC * 2 * t] = o[j][2 * m];
            r[at + PC * (2 * t + 1)] = o[j][2 * m + 1];
        }
        if (t == 0) {
            r[DV] = top[m];
            r[DV + 1] = sum[m];
        }
    }
    __syncthreads();
    const long long total = (long long)a.N * a.Mk * a.rows;
    for (int r = warp; r < kAsRows; r += kAsWarps) {
        if (r0 + r >= a.rows) break;
        float w[2][kAsWarps], all[2], peak[2];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const float* x = as_smem + (8 * m + r) * (DV + 2) + DV;
            peak[m] = -INFINITY;
#pragma unroll
            for (int k = 0; k < kAsWarps; ++k) peak[m] = fmaxf(peak[m], x[k * 16 * (DV + 2)]);
            const float base = peak[m] == -INFINITY ? 0.f : peak[m];
            all[m] = 0.f;
#pragma unroll
            for (int k = 0; k < kAsWarps; ++k) {
                w[m][k] = ex2(x[k * 16 * (DV + 2)] - base);
                all[m] += w[m][k] * x[k * 16 * (DV + 2) + 1];
            }
        }
        const uint32_t tk = a.div_G.div((uint32_t)(r0 + r));
        const int hd = kv * a.G + r0 + r - (int)tk * a.G;
        const long long at = (long long)split * total + (long long)blockIdx.y * a.rows + r0 + r;
        const long long to = (((long long)n * a.Lq + tk) * a.M + hd) * DV;
        const float lam = Elem<T>::one(static_cast<const T*>(a.lam) + hd);
        const float i0 = all[0] > 0.f ? 1.f / all[0] : 0.f, i1 = all[1] > 0.f ? 1.f / all[1] : 0.f;
#pragma unroll
        for (int c = lane; c < DV; c += 32) {
            float x = 0.f, y = 0.f;
#pragma unroll
            for (int k = 0; k < kAsWarps; ++k) {
                x += w[0][k] * as_smem[(k * 16 + r) * (DV + 2) + c];
                y += w[1][k] * as_smem[(k * 16 + 8 + r) * (DV + 2) + c];
            }
            if (a.splits > 1) {
                a.part_o[at * 2 * DV + c] = x;
                a.part_o[(at * 2 + 1) * DV + c] = y;
            } else {
                x = __fmul_rn(x, i0);
                y = __fmul_rn(y, i1);
                static_cast<T*>(a.out)[to + c] = Elem<T>::from(attn_diff(x, lam, y));
                if (a.maps) {
                    a.maps[2 * to + c] = x;
                    a.maps[2 * to + DV + c] = y;
                }
            }
        }
        if (lane < 2) {
            const float pk = lane ? peak[1] : peak[0], sm = lane ? all[1] : all[0];
            if (a.splits > 1) {
                a.part_ml[(at * 2 + lane) * 2] = pk;
                a.part_ml[(at * 2 + lane) * 2 + 1] = sm;
            } else if (a.lse) {
                a.lse[(((long long)n * a.M + hd) * 2 + lane) * a.Lq + tk] =
                    sm > 0.f ? pk + log2f(sm) : INFINITY;
            }
        }
    }
}

}  // namespace dcnb
