// Differential attention on the CUDA cores (sm_100a): forward, the join of
// split key ranges, and both gradient kernels, for every type and head size.
//
// For token i of image n, head h of key / value head a = h / G:
//   P_s[i][j] = softmax over the visible keys j of scale * <q[i][h][s], k[j][a][s]>, s = 0, 1
//   out[i][h] = sum_j (P_0[i][j] - lambda[h] P_1[i][j]) v[j][a]
// Key j of image n is visible to token i when j < len_n, it is not masked and,
// in causal order, j <= i + len_n - Lq.  A row that sees no key gives zeros.
//
// The scores are kept in the base-2 domain, t = scale * log2(e) * <q, k>, and a
// row runs over the keys once with its running maximum m and sum of 2^(t - m)
// for each of the two maps; everything is float32.
//
// Rows: the G heads that share a key / value head are stacked, row r = token *
// G + (head in group), so each key and value is read once for all of them; for
// one new token a sequence that is what makes a tile's rows worth its reads.
// Bound: the FMA rate for long inputs (two dot products and two weighted sums,
// 4 D + 4 Dv operations a pair), the key / value bytes for few rows.  A thread
// of the 16 x 16 block holds RT x 4 scores of either map (rows ty + 16 i, keys
// tx + 16 j) and RT x DVT outputs of either map; tiles sit in shared memory as
// float32 rows padded by 16 bytes, so that the 16 rows a half-warp reads fall
// into different banks.  One value tile serves both maps.
// It runs float32 data, head sizes that the tensor-core kernels do not take and
// unaligned tensors: 199 us on float32 heads of 32 + 32 over 2 x 950 cells, 8
// heads (16.6 TFLOP/s, 46 us at the FMA rate; shared-memory reads hold it).
#pragma once

#include "axial_rope.cuh"

namespace dcnb {

constexpr int kAttnThreads = 256;
constexpr int kAttnKeys = 64;          // keys of a forward tile
constexpr int kAttnMaxD = 128;
constexpr int kAttnMaxDv = 256;
constexpr int kAttnMaxSplits = 64;
constexpr int kRowvTile = 64;          // tokens of a tile of row values

struct AttnArgs {
    const void* q;
    const void* k;
    const void* v;
    const void* lam;
    const unsigned char* mask;     // [N][Lk], non-zero = masked, or null
    const int* lengths;            // [N] or null
    void* out;
    float* maps;                   // [N][Lq][M][2][Dv], the maps' own outputs, or null
    float* lse;                    // [N][M][2][Lq], or null
    float* part_ml;                // [splits][N * Mk * rows][2][2]
    float* part_o;                 // [splits][N * Mk * rows][2][Dv]
    // gradient
    const void* go;
    const float* rowv;             // [N][M][tiles of 64 tokens][4][64]: -lse_0, -lse_1, -e_0, -e_1
    void* gq;
    void* gk;
    void* gv;
    int N, Lq, Lk, M, Mk, G, D, Dv;
    int rows;                      // Lq * G
    int splits;
    int causal;
    int vec4;                      // every row of q, k, v (and go) is made of aligned groups of 4
    float scale;                   // scale of the scores
    float scale_log2;              // scale * log2(e)
    long long q_image, q_row, k_image, k_row, v_image, v_row;
    FastDiv div_G, div_Mk;
};

// O_0 - lambda O_1, with the same roundings whether the maps' outputs are stored
// or not (a contraction with the product before would differ).
__device__ __forceinline__ float attn_diff(float o0, float lam, float o1) {
    return fmaf(-lam, o1, o0);
}

__device__ __forceinline__ int attn_len(const AttnArgs& a, int n) {
    return a.lengths ? max(0, min(a.lengths[n], a.Lk)) : a.Lk;
}

// Offset of token tok's first row value (the others follow kRowvTile apart).
__device__ __forceinline__ long long attn_rowv(const AttnArgs& a, int n, int head, int tok) {
    const int tiles = (a.Lq + kRowvTile - 1) / kRowvTile;
    return (((long long)n * a.M + head) * tiles + tok / kRowvTile) * (4 * kRowvTile) +
           tok % kRowvTile;
}

// Place of token tok's |g|^2: tokens of a head side by side, padded to whole tiles.
__device__ __forceinline__ long long attn_gnorm(const AttnArgs& a, int n, int head, int tok) {
    const int tiles = (a.Lq + kRowvTile - 1) / kRowvTile;
    return (((long long)n * a.M + head) * tiles) * kRowvTile + tok;
}

// Four elements of a row at column d (D in all) as float32, zeros past the end.
template <typename T>
__device__ __forceinline__ float4 attn_ld4(const T* row, int d, int D, int vec4) {
    float f[4];
    if (vec4) {
        ld_f32<T, 4>(row + d, f);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = d + e < D ? Elem<T>::one(row + d + e) : 0.f;
    }
    return make_float4(f[0], f[1], f[2], f[3]);
}

__device__ __forceinline__ float dot4(float acc, const float4& a, const float4& b) {
    acc = fmaf(a.x, b.x, acc);
    acc = fmaf(a.y, b.y, acc);
    acc = fmaf(a.z, b.z, acc);
    return fmaf(a.w, b.w, acc);
}

// Element offset of packed row r of key / value head a in a tensor [.][M][inner].
__device__ __forceinline__ long long attn_row(const AttnArgs& a, int kv, uint32_t r,
                                              long long row_stride, int inner, uint32_t* token,
                                              int* head) {
    const uint32_t t = a.div_G.div(r);
    *token = t;
    *head = kv * a.G + (int)(r - t * (uint32_t)a.G);
    return (long long)t * row_stride + (long long)*head * inner;
}

// Copies packed rows [r0, r0 + n) (`parts` parts of D columns each) to
// s[row][part][.], parts `part_ld` floats apart, zeros past `rows`.
template <typename T>
__device__ __forceinline__ void attn_stage_rows(const AttnArgs& a, const T* base, long long stride,
                                                int kv, int r0, int n, int parts, int D, float* s,
                                                int ld, int part_ld) {
    const int D4 = (D + 3) & ~3, chunks = parts * (D4 / 4);
    for (int i = threadIdx.x; i < n * chunks; i += kAttnThreads) {
        const int row = i / chunks, ch = i - row * chunks;
        const int part = ch / (D4 / 4), d = (ch - part * (D4 / 4)) * 4;
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r0 + row < a.rows) {
            uint32_t tok;
            int head;
            const T* p = base + attn_row(a, kv, (uint32_t)(r0 + row), stride, parts * D, &tok,
                                         &head);
            f = attn_ld4<T>(p + part * D, d, D, a.vec4);
        }
        *reinterpret_cast<float4*>(s + row * ld + part * part_ld + d) = f;
    }
}

// Copies key rows [j0, j0 + n) of head kv in the same way; rows whose `ok` flag is 0
// (masked or past the end) are zeros, whatever the memory holds.
template <typename T>
__device__ __forceinline__ void attn_stage_keys(const AttnArgs& a, const T* base, long long stride,
                                                int kv, int j0, int n, int parts, int D, float* s,
                                                int ld, int part_ld, const unsigned char* ok) {
    const int D4 = (D + 3) & ~3, chunks = parts * (D4 / 4);
    for (int i = threadIdx.x; i < n * chunks; i += kAttnThreads) {
        const int row = i / chunks, ch = i - row * chunks;
        const int part = ch / (D4 / 4), d = (ch - part * (D4 / 4)) * 4;
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
        if (ok[row]) {
            const T* p = base + (long long)(j0 + row) * stride + (long long)kv * parts * D;
            f = attn_ld4<T>(p + part * D, d, D, a.vec4);
        }
        *reinterpret_cast<float4*>(s + row * ld + part * part_ld + d) = f;
    }
}

// acc[r][c] (+)= <A row ty + 16 r, B row tx + 16 c> over D4 columns.
template <int RT, int CT>
__device__ __forceinline__ void attn_dots(const float* A, int lda, const float* B, int ldb, int D4,
                                          float (&acc)[RT][CT]) {
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[r][c] = 0.f;
#pragma unroll 2
    for (int d = 0; d < D4; d += 4) {
        float4 av[RT], bv[CT];
#pragma unroll
        for (int r = 0; r < RT; ++r)
            av[r] = *reinterpret_cast<const float4*>(A + (ty + 16 * r) * lda + d);
#pragma unroll
        for (int c = 0; c < CT; ++c)
            bv[c] = *reinterpret_cast<const float4*>(B + (tx + 16 * c) * ldb + d);
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int c = 0; c < CT; ++c) acc[r][c] = dot4(acc[r][c], av[r], bv[c]);
    }
}

// acc[r][.] += sum over i < n of A[ty + 16 r][i] * B[i][columns of tx]: CT
// columns a thread in groups of VW, group j at tx * VW + 16 * VW * j.
template <int RT, int CT>
__device__ __forceinline__ void attn_weighted(const float* A, int lda, const float* B, int ldb,
                                              int n, float (&acc)[RT][CT]) {
    constexpr int VW = CT < 4 ? CT : 4;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int i = 0; i < n; i += 4) {
        float w[RT][4];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const float4 f = *reinterpret_cast<const float4*>(A + (ty + 16 * r) * lda + i);
            w[r][0] = f.x;
            w[r][1] = f.y;
            w[r][2] = f.z;
            w[r][3] = f.w;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
#pragma unroll
            for (int j = 0; j < CT / VW; ++j) {
                float b[VW];
                const float* p = B + (i + e) * ldb + tx * VW + 16 * VW * j;
                if constexpr (VW == 4) {
                    const float4 f = *reinterpret_cast<const float4*>(p);
                    b[0] = f.x;
                    b[1] = f.y;
                    b[2] = f.z;
                    b[3] = f.w;
                } else {
                    const float2 f = *reinterpret_cast<const float2*>(p);
                    b[0] = f.x;
                    b[1] = f.y;
                }
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int c = 0; c < VW; ++c)
                        acc[r][j * VW + c] = fmaf(w[r][e], b[c], acc[r][j * VW + c]);
            }
        }
    }
}

// The tile's sum formed first: acc = acc * keep + sum.  A sum of n terms then takes its
// rounding from n / 64 additions to a large value instead of n (of random signs, sqrt(n)
// errors of the sum's own step: 16384 rows gave grad_k an error of 2.3e-6, now less than
// 1e-6, and 8192 keys an output 1.7e-6).
template <int RT, int CT>
__device__ __forceinline__ void attn_weighted_tile(const float* A, int lda, const float* B,
                                                   int ldb, int n, float (&acc)[RT][CT],
                                                   const float (&keep)[RT]) {
    float part[RT][CT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int c = 0; c < CT; ++c) part[r][c] = 0.f;
    attn_weighted<RT, CT>(A, lda, B, ldb, n, part);
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[r][c] = fmaf(acc[r][c], keep[r], part[r][c]);
}

template <int RT, int CT>
__device__ __forceinline__ void attn_weighted_tile(const float* A, int lda, const float* B,
                                                   int ldb, int n, float (&acc)[RT][CT]) {
    float one[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) one[r] = 1.f;
    attn_weighted_tile<RT, CT>(A, lda, B, ldb, n, acc, one);
}

template <int CT>
__device__ __forceinline__ int attn_col(int c) {
    constexpr int VW = CT < 4 ? CT : 4;
    return (threadIdx.x & 15) * VW + 16 * VW * (c / VW) + c % VW;
}

// Row strides of the shared tiles, in floats.
__host__ __device__ constexpr int attn_ld(int parts, int D) { return parts * ((D + 3) & ~3) + 4; }
// Value rows are read as CT columns of 16 threads: 16 * CT floats are allocated.
__host__ __device__ constexpr int attn_ldv(int CT) { return 16 * CT + 4; }

__host__ __device__ constexpr int attn_fwd_smem(int BQ, int D, int CT) {
    const int kp = 2 * BQ * (kAttnKeys + 4), kk = kAttnKeys * attn_ld(2, D);
    return (BQ * attn_ld(2, D) + (kk > kp ? kk : kp) + kAttnKeys * attn_ldv(CT)) * 4 + kAttnKeys;
}

// Two blocks a multiprocessor for 16 rows and for values up to 32 channels: one block (139
// and 148 registers) took 1258 us against 912 on one float32 token over 16 caches of 8192
// keys, and 260 against 199 on the case above.
template <typename T, int BQ, int CT>
__global__ void __launch_bounds__(kAttnThreads, BQ == 16 || CT == 2 ? 2 : 1)
    diff_attn_kernel(const AttnArgs a) {
    constexpr int RT = BQ / 16, BK = kAttnKeys;
    extern __shared__ __align__(16) float attn_smem[];
    const int D = a.D, D4 = (D + 3) & ~3, Dv = a.Dv;
    const int ldq = attn_ld(2, D), ldv = attn_ldv(CT), ldp = BK + 4;
    float* Qs = attn_smem;
    float* Ks = Qs + BQ * ldq;
    float* Ps = Ks;                       // the scores' tile takes the keys' place
    float* Vs = Ks + max(BK * ldq, 2 * BQ * ldp);
    unsigned char* ok = reinterpret_cast<unsigned char*>(Vs + BK * ldv);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int n = (int)a.div_Mk.div(blockIdx.y), kv = (int)blockIdx.y - n * a.Mk;
    const int split = blockIdx.z;
    // the last tiles see the most keys in causal order: they start first
    const int r0 = (int)(gridDim.x - 1 - blockIdx.x) * BQ;
    const int len = attn_len(a, n);
    const int last_tok = (int)a.div_G.div((uint32_t)min(r0 + BQ - 1, a.rows - 1));
    const int kmax = a.causal ? max(0, min(len, last_tok + len - a.Lq + 1)) : len;
    const int tiles = (kmax + BK - 1) / BK;
    const int t_begin = (int)((long long)tiles * split / a.splits);
    const int t_end = (int)((long long)tiles * (split + 1) / a.splits);

    attn_stage_rows<T>(a, static_cast<const T*>(a.q) + n * a.q_image, a.q_row, kv, r0, BQ, 2, D,
                       Qs, ldq, D4);
    // columns past Dv stay zero (only columns below Dv are staged)
    for (int i = threadIdx.x; i < BK * ldv; i += kAttnThreads) Vs[i] = 0.f;
    float m[2][RT], l[2][RT], o[2][RT][CT];
    int limit[RT];                        // keys below this index are in order for the row
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int row = r0 + ty + 16 * r;
        const int tok = (int)a.div_G.div((uint32_t)min(row, a.rows - 1));
        limit[r] = a.causal ? min(len, tok + len - a.Lq + 1) : len;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            m[s][r] = -INFINITY;
            l[s][r] = 0.f;
#pragma unroll
            for (int c = 0; c < CT; ++c) o[s][r][c] = 0.f;
        }
    }
    const T* kb = static_cast<const T*>(a.k) + n * a.k_image;
    const T* vb = static_cast<const T*>(a.v) + n * a.v_image;
    for (int t = t_begin; t < t_end; ++t) {
        const int j0 = t * BK;
        __syncthreads();                  // the last tile's readers are done
        for (int i = threadIdx.x; i < BK; i += kAttnThreads)
            ok[i] = j0 + i < len && !(a.mask && a.mask[(long long)n * a.Lk + j0 + i]);
        __syncthreads();
        attn_stage_keys<T>(a, kb, a.k_row, kv, j0, BK, 2, D, Ks, ldq, D4, ok);
        attn_stage_keys<T>(a, vb, a.v_row, kv, j0, BK, 1, Dv, Vs, ldv, 0, ok);
        __syncthreads();
        float sc[2][RT][4], kept[2][RT];
        attn_dots<RT, 4>(Qs, ldq, Ks, ldq, D4, sc[0]);
        attn_dots<RT, 4>(Qs + D4, ldq, Ks + D4, ldq, D4, sc[1]);
        __syncthreads();                  // the keys are read: their place takes the scores
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                float top = -INFINITY;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int j = tx + 16 * c;
                    sc[s][r][c] = ok[j] && j0 + j < limit[r] ? sc[s][r][c] * a.scale_log2
                                                            : -INFINITY;
                    top = fmaxf(top, sc[s][r][c]);
                }
#pragma unroll
                for (int w = 8; w > 0; w >>= 1)
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
                const float mn = fmaxf(m[s][r], top);
                const float base = mn == -INFINITY ? 0.f : mn;
                const float keep = exp2f(m[s][r] - base);
                m[s][r] = mn;
                float sum = 0.f;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float p = exp2f(sc[s][r][c] - base);
                    sum += p;
                    Ps[(s * BQ + ty + 16 * r) * ldp + tx + 16 * c] = p;
                }
#pragma unroll
                for (int w = 8; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
                l[s][r] = l[s][r] * keep + sum;
                kept[s][r] = keep;
            }
        }
        __syncthreads();
        attn_weighted_tile<RT, CT>(Ps, ldp, Vs, ldv, BK, o[0], kept[0]);
        attn_weighted_tile<RT, CT>(Ps + BQ * ldp, ldp, Vs, ldv, BK, o[1], kept[1]);
    }
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int row = r0 + ty + 16 * r;
        if (row >= a.rows) continue;
        const uint32_t tok = a.div_G.div((uint32_t)row);
        const int head = kv * a.G + row - (int)tok * a.G;
        if (a.splits > 1) {
            const long long total = (long long)a.N * a.Mk * a.rows;
            const long long at = (long long)split * total + (long long)blockIdx.y * a.rows + row;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                if (tx == 0) {
                    a.part_ml[(at * 2 + s) * 2] = m[s][r];
                    a.part_ml[(at * 2 + s) * 2 + 1] = l[s][r];
                }
#pragma unroll
                for (int c = 0; c < CT; ++c) {
                    const int col = attn_col<CT>(c);
                    if (col < Dv) a.part_o[(at * 2 + s) * Dv + col] = o[s][r][c];
                }
            }
            continue;
        }
        const float lam = Elem<T>::one(static_cast<const T*>(a.lam) + head);
        const float i0 = l[0][r] > 0.f ? 1.f / l[0][r] : 0.f;
        const float i1 = l[1][r] > 0.f ? 1.f / l[1][r] : 0.f;
        const long long at = (((long long)n * a.Lq + tok) * a.M + head) * Dv;
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            const int col = attn_col<CT>(c);
            if (col >= Dv) continue;
            const float one = __fmul_rn(o[0][r][c], i0), second = __fmul_rn(o[1][r][c], i1);
            static_cast<T*>(a.out)[at + col] = Elem<T>::from(attn_diff(one, lam, second));
            if (a.maps) {
                a.maps[2 * at + col] = one;
                a.maps[2 * at + Dv + col] = second;
            }
        }
        if (a.lse && tx < 2) {
            const float ms = tx ? m[1][r] : m[0][r], ls = tx ? l[1][r] : l[0][r];
            a.lse[(((long long)n * a.M + head) * 2 + tx) * a.Lq + tok] =
                ls > 0.f ? ms + log2f(ls) : INFINITY;
        }
    }
}

// Joins the splits of a row: O_s and l_s weighted by 2^(m_s - max), in the order
// of the splits.  One block per row: a warp a map forms the weights, then every
// thread sums its columns (loads of a warp are whole rows, and independent of
// one another).
constexpr int kJoinThreads = 128;

template <typename T>
__global__ void __launch_bounds__(kJoinThreads) diff_attn_join_kernel(const AttnArgs a) {
    __shared__ float weight[2][kAttnMaxSplits], inv[2];
    const long long total = (long long)a.N * a.Mk * a.rows;
    const long long at = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nk = (int)(at / a.rows), row = (int)(at - (long long)nk * a.rows);
    const int n = (int)a.div_Mk.div((uint32_t)nk), kv = nk - n * a.Mk;
    const uint32_t tok = a.div_G.div((uint32_t)row);
    const int head = kv * a.G + row - (int)tok * a.G, Dv = a.Dv;
    if (warp < 2) {
        float m[2], l[2];                 // lane holds splits lane and lane + 32
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int sp = lane + 32 * h;
            const long long p = (((long long)sp * total + at) * 2 + warp) * 2;
            m[h] = sp < a.splits ? a.part_ml[p] : -INFINITY;
            l[h] = sp < a.splits ? a.part_ml[p + 1] : 0.f;
        }
        float top = fmaxf(m[0], m[1]);
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float base = top == -INFINITY ? 0.f : top;
        float w[2], sum = 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            w[h] = exp2f(m[h] - base);
            sum += w[h] * l[h];
            if (lane + 32 * h < kAttnMaxSplits) weight[warp][lane + 32 * h] = w[h];
        }
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) {
            inv[warp] = sum > 0.f ? 1.f / sum : 0.f;
            if (a.lse)
                a.lse[(((long long)n * a.M + head) * 2 + warp) * a.Lq + tok] =
                    sum > 0.f ? base + log2f(sum) : INFINITY;
        }
    }
    __syncthreads();
    const float lam = Elem<T>::one(static_cast<const T*>(a.lam) + head);
    const long long to = (((long long)n * a.Lq + tok) * a.M + head) * Dv;
    const long long step = total * 2 * Dv;
    for (int c = threadIdx.x; c < Dv; c += kJoinThreads) {
        const float* p = a.part_o + at * 2 * Dv + c;
        float x = 0.f, y = 0.f;
#pragma unroll 8
        for (int sp = 0; sp < a.splits; ++sp, p += step) {
            x = fmaf(weight[0][sp], p[0], x);
            y = fmaf(weight[1][sp], p[Dv], y);
        }
        x = __fmul_rn(x, inv[0]);
        y = __fmul_rn(y, inv[1]);
        static_cast<T*>(a.out)[to + c] = Elem<T>::from(attn_diff(x, lam, y));
        if (a.maps) {
            a.maps[2 * to + c] = x;
            a.maps[2 * to + Dv + c] = y;
        }
    }
}

// ---------------------------------------------------------------- gradient --
//
// With O_s the maps' own outputs (out = O_0 - lambda O_1), g = grad_out and
// dP[i][j] = <g[i], v[j]> shared by both maps:
//   dT_0 = P_0 (dP - <g, O_0>),  dT_1 = -lambda P_1 (dP - <g, O_1>)
//   grad_q_s = scale dT_s k_s,  grad_k_s = scale dT_s^T q_s
//   grad_v = (P_0 - lambda P_1)^T g,  grad_lambda = -sum over rows of <g, O_1>
// P_s = 2^(t - lse) comes back from the saved lse.  Query tiles own grad_q and
// key tiles own grad_k and grad_v, each in its own kernel: the scores are
// computed twice, but no sum goes through atomics, so a gradient does not
// depend on the order of blocks.

struct AttnDeltaArgs {
    const float* maps;
    const void* go;
    const void* lam;       // scales kernel
    const float* lse;
    AttnArgs a;            // geometry, visible keys and v
    float* rowv;
    void* glam;            // grad_lambda kernel
    float* gnorm;          // [N][M][tiles * 64] |g|^2 of a row, or null
    float* vnorm;          // [N][Mk][Lk] |v|^2 of a visible key (0 of a hidden one), or null
    float4* scales;        // [N][Mk] cs and cp of the key kernel, the largest |v|
    int g_blocks, v_blocks;
    int vec4;              // rows of the maps and of grad_out are aligned groups of 4
};

// at / d and at % d, in 32 bits where they suffice (a 64-bit division costs more
// than the rest of a row).
__device__ __forceinline__ void attn_split(long long at, int d, long long& q, int& r) {
    if (at <= 0xffffffffLL) {
        const uint32_t t = (uint32_t)at / (uint32_t)d;
        q = t;
        r = (int)((uint32_t)at - t * (uint32_t)d);
    } else {
        q = at / d;
        r = (int)(at - q * d);
    }
}

// One warp per (token, head), tokens padded to whole tiles: e_s = <g, O_s> from
// the maps' own outputs, kept in float32 (with outputs rounded to 16 bits the
// differences dP - e_s, and with them grad_q, grad_k and grad_lambda, carried
// that rounding: grad_lambda was off by up to twice a 16-bit result's own).
// Rows past the end and rows that see no key get -lse = -inf: weights of 0.
// With `gnorm` and `vnorm` also |g|^2 of every row and, in blocks of their own,
// |v|^2 of every key.
template <typename T>
__global__ void __launch_bounds__(256) diff_attn_delta_kernel(const AttnDeltaArgs d) {
    const AttnArgs& a = d.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if ((int)blockIdx.x < d.g_blocks) {
        const int tiles = (a.Lq + kRowvTile - 1) / kRowvTile;
        const long long at = (long long)blockIdx.x * 8 + warp;
        long long tok_all;                              // tokens of all images, padded
        int h, n, i;
        attn_split(at, a.M, tok_all, h);
        {
            long long image;
            attn_split(tok_all, tiles * kRowvTile, image, i);
            n = (int)image;
        }
        if (n < a.N) {
            float s = 0.f, s2 = 0.f, norm = 0.f, lse = INFINITY;
            if (i < a.Lq) {
                const long long row = (((long long)n * a.Lq + i) * a.M + h) * a.Dv;
                const T* g = static_cast<const T*>(d.go) + row;
                const float* o = d.maps + 2 * row;
                // four channels a lane where rows are aligned groups of four
                for (int c = 4 * lane; c < a.Dv; c += 128) {
                    const float4 gv = attn_ld4<T>(g, c, a.Dv, d.vec4);
                    const float4 ov = attn_ld4<float>(o, c, a.Dv, d.vec4);
                    const float4 o2v = attn_ld4<float>(o + a.Dv, c, a.Dv, d.vec4);
                    s = dot4(s, gv, ov);
                    s2 = dot4(s2, gv, o2v);
                    norm = dot4(norm, gv, gv);
                }
                if (lane < 2) lse = d.lse[(((long long)n * a.M + h) * 2 + lane) * a.Lq + i];
            }
            for (int w = 16; w > 0; w >>= 1) {
                s += __shfl_xor_sync(0xffffffffu, s, w);
                s2 += __shfl_xor_sync(0xffffffffu, s2, w);
                norm += __shfl_xor_sync(0xffffffffu, norm, w);
            }
            float* r = d.rowv + attn_rowv(a, n, h, i);
            if (lane < 2) {
                r[lane * kRowvTile] = -lse;
                r[(2 + lane) * kRowvTile] = lane ? -s2 : -s;
            }
            if (d.gnorm && lane == 0) d.gnorm[attn_gnorm(a, n, h, i)] = norm;
        }
    } else {
        const long long at = ((long long)blockIdx.x - d.g_blocks) * 8 + warp;
        long long key_all, image;
        int kv, j;
        attn_split(at, a.Mk, key_all, kv);
        attn_split(key_all, a.Lk, image, j);
        const int n = (int)image;
        if (n >= a.N) return;
        float norm = 0.f;
        if (j < attn_len(a, n) && !(a.mask && a.mask[(long long)n * a.Lk + j])) {
            const T* v = static_cast<const T*>(a.v) + n * a.v_image + (long long)j * a.v_row +
                         (long long)kv * a.Dv;
            for (int c = lane; c < a.Dv; c += 32) {
                const float x = Elem<T>::one(v + c);
                norm = fmaf(x, x, norm);
            }
        }
        for (int w = 16; w > 0; w >>= 1) norm += __shfl_xor_sync(0xffffffffu, norm, w);
        if (lane == 0) d.vnorm[((long long)n * a.Mk + kv) * a.Lk + j] = norm;
    }
}

// The power of two that brings x to (2^14, 2^15]; 1 for 0, infinities and NaN, and
// within 2^-40 .. 2^40.
__device__ __forceinline__ float attn_pow2(float x) {
    if (!(x > 0.f) || x > 1e30f) return 1.f;
    return exp2f(fminf(fmaxf(15.f - ceilf(log2f(x)), -40.f), 40.f));
}

// The power of two for the score gradients of a row or of several:
// |dS| <= 2 max(1, |lambda|) |g| |v| with the largest of each among them.
__device__ __forceinline__ float attn_grad_scale(float lam, float g, float v) {
    return attn_pow2(2.f * fmaxf(1.f, fabsf(lam)) * g * v);
}

// Block (n, a): the scales of the key kernel's fp16 operands, from the rows of
// image n and the heads of key / value head a, and the largest |v| of its keys.
template <typename T>
__global__ void __launch_bounds__(1024) diff_attn_scales_kernel(const AttnDeltaArgs d) {
    __shared__ float part[32][3];
    const AttnArgs& a = d.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n = (int)a.div_Mk.div(blockIdx.x), kv = (int)blockIdx.x - n * a.Mk;
    float x[3] = {0.f, 0.f, 0.f};
    // the rows of a group's heads follow one another
    const float* g = d.gnorm + attn_gnorm(a, n, kv * a.G, 0);
    const long long rows = attn_gnorm(a, 0, a.G, 0);
    for (long long i = threadIdx.x; i < rows; i += 1024) x[0] = fmaxf(x[0], g[i]);
    const float* v = d.vnorm + (long long)blockIdx.x * a.Lk;
    for (int i = threadIdx.x; i < a.Lk; i += 1024) x[1] = fmaxf(x[1], v[i]);
    for (int h = threadIdx.x; h < a.G; h += 1024)
        x[2] = fmaxf(x[2], fabsf(Elem<T>::one(static_cast<const T*>(d.lam) + kv * a.G + h)));
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        for (int w = 16; w > 0; w >>= 1)
            x[k] = fmaxf(x[k], __shfl_xor_sync(0xffffffffu, x[k], w));
        if (lane == 0) part[warp][k] = x[k];
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 32; ++w)
            for (int k = 0; k < 3; ++k) part[0][k] = fmaxf(part[0][k], part[w][k]);
        const float lam = part[0][2], most = sqrtf(part[0][1]);
        // |P_0 - lambda P_1| <= 1 + |lambda|
        d.scales[blockIdx.x] = make_float4(attn_grad_scale(lam, sqrtf(part[0][0]), most),
                                           attn_pow2(1.f + lam), most, 0.f);
    }
}

// Block h: grad_lambda of head h, in a fixed order.
template <typename T>
__global__ void __launch_bounds__(1024) diff_attn_glam_kernel(const AttnDeltaArgs d) {
    __shared__ float part[32];
    const AttnArgs& a = d.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.x;
    float s = 0.f;
    for (int n = 0; n < a.N; ++n)
        for (int i = threadIdx.x; i < a.Lq; i += 1024)
            s += d.rowv[attn_rowv(a, n, h, i) + 3 * kRowvTile];
    for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    if (lane == 0) part[warp] = s;
    __syncthreads();
    if (threadIdx.x < 32) {
        s = part[threadIdx.x];
        for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
        if (threadIdx.x == 0) static_cast<T*>(d.glam)[h] = Elem<T>::from(s);
    }
}

// Shared memory of the gradient kernels: q and k rows (two maps of 16 CD
// columns), v and g rows (16 CT columns), three score tiles, five values a row
// and the key flags.
__host__ __device__ constexpr int attn_bwd_smem(int BT, int CD, int CT) {
    return (2 * BT * (32 * CD + 4) + 2 * BT * attn_ldv(CT) + 3 * BT * (BT + 4) + 5 * BT) * 4 + BT;
}

struct AttnBwdTile {
    float *Qs, *Ks, *Vs, *Gs, *S, *rowv;
    unsigned char* ok;
};

template <int BT, int CD, int CT>
__device__ __forceinline__ AttnBwdTile attn_bwd_tile(float* smem) {
    AttnBwdTile t;
    t.Qs = smem;
    t.Ks = t.Qs + BT * (32 * CD + 4);
    t.Vs = t.Ks + BT * (32 * CD + 4);
    t.Gs = t.Vs + BT * attn_ldv(CT);
    t.S = t.Gs + BT * attn_ldv(CT);
    t.rowv = t.S + 3 * BT * (BT + 4);
    t.ok = reinterpret_cast<unsigned char*>(t.rowv + 5 * BT);
    // columns that no part fills stay zero
    for (float* p = smem + threadIdx.x; p < t.rowv + 5 * BT; p += kAttnThreads) *p = 0.f;
    return t;
}

// Stages q, g and the five values (-lse_0, -lse_1, -e_0, -e_1, lambda) of
// packed rows [r0, r0 + BT).
template <typename T, int BT, int CD, int CT>
__device__ __forceinline__ void attn_bwd_rows(const AttnArgs& a, const AttnBwdTile& t, int n,
                                              int kv, int r0) {
    attn_stage_rows<T>(a, static_cast<const T*>(a.q) + n * a.q_image, a.q_row, kv, r0, BT, 2, a.D,
                       t.Qs, 32 * CD + 4, 16 * CD);
    attn_stage_rows<T>(a, static_cast<const T*>(a.go) + (long long)n * a.Lq * a.M * a.Dv,
                       (long long)a.M * a.Dv, kv, r0, BT, 1, a.Dv, t.Gs, attn_ldv(CT), 0);
    for (int i = threadIdx.x; i < BT; i += kAttnThreads) {
        float v[5] = {-INFINITY, -INFINITY, 0.f, 0.f, 0.f};
        if (r0 + i < a.rows) {
            const uint32_t tok = a.div_G.div((uint32_t)(r0 + i));
            const int head = kv * a.G + r0 + i - (int)tok * a.G;
            const float* r = a.rowv + attn_rowv(a, n, head, (int)tok);
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = r[k * kRowvTile];
            v[4] = Elem<T>::one(static_cast<const T*>(a.lam) + head);
        }
#pragma unroll
        for (int k = 0; k < 5; ++k) t.rowv[k * BT + i] = v[k];
    }
}

template <typename T, int BT, int CD, int CT>
__device__ __forceinline__ void attn_bwd_keys(const AttnArgs& a, const AttnBwdTile& t, int n,
                                              int kv, int j0, int len) {
    for (int i = threadIdx.x; i < BT; i += kAttnThreads)
        t.ok[i] = j0 + i < len && !(a.mask && a.mask[(long long)n * a.Lk + j0 + i]);
    __syncthreads();
    attn_stage_keys<T>(a, static_cast<const T*>(a.k) + n * a.k_image, a.k_row, kv, j0, BT, 2, a.D,
                       t.Ks, 32 * CD + 4, 16 * CD, t.ok);
    attn_stage_keys<T>(a, static_cast<const T*>(a.v) + n * a.v_image, a.v_row, kv, j0, BT, 1, a.Dv,
                       t.Vs, attn_ldv(CT), 0, t.ok);
}

// The tile's score gradients to S[0], S[1] and, with KEYS, P_0 - lambda P_1 to
// S[2]; KEYS stores them transposed (key, row).  Rows past the end have
// -lse = -inf, so their probabilities are 0; hidden pairs are exact zeros.
template <int BT, int CD, int CT, bool KEYS>
__device__ __forceinline__ void attn_bwd_scores(const AttnArgs& a, const AttnBwdTile& t, int r0,
                                                int j0, int len) {
    constexpr int RT = BT / 16, ldq = 32 * CD + 4, ldv = attn_ldv(CT), lds = BT + 4;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int D4 = (a.D + 3) & ~3, Dv4 = (a.Dv + 3) & ~3;
    float dp[RT][RT], t0[RT][RT], t1[RT][RT];
    attn_dots<RT, RT>(t.Gs, ldv, t.Vs, ldv, Dv4, dp);
    attn_dots<RT, RT>(t.Qs, ldq, t.Ks, ldq, D4, t0);
    attn_dots<RT, RT>(t.Qs + 16 * CD, ldq, t.Ks + 16 * CD, ldq, D4, t1);
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int row = ty + 16 * r;
        const int tok = (int)a.div_G.div((uint32_t)min(r0 + row, a.rows - 1));
        const int limit = a.causal ? min(len, tok + len - a.Lq + 1) : len;
        const float l0 = t.rowv[row], l1 = t.rowv[BT + row], e0 = t.rowv[2 * BT + row];
        const float e1 = t.rowv[3 * BT + row], lam = t.rowv[4 * BT + row];
#pragma unroll
        for (int c = 0; c < RT; ++c) {
            const int j = tx + 16 * c;
            const bool see = t.ok[j] && j0 + j < limit;
            const float p0 = see ? exp2f(t0[r][c] * a.scale_log2 + l0) : 0.f;
            const float p1 = see ? lam * exp2f(t1[r][c] * a.scale_log2 + l1) : 0.f;
            const float g0 = see ? p0 * (dp[r][c] + e0) : 0.f;
            const float g1 = see ? -p1 * (dp[r][c] + e1) : 0.f;
            const int at = KEYS ? j * lds + row : row * lds + j;
            t.S[at] = g0;
            t.S[BT * lds + at] = g1;
            if (KEYS) t.S[2 * BT * lds + at] = p0 - p1;
        }
    }
}

template <typename T, int BT, int CD, int CT>
__global__ void __launch_bounds__(kAttnThreads) diff_attn_dq_kernel(const AttnArgs a) {
    constexpr int RT = BT / 16, ldq = 32 * CD + 4, lds = BT + 4;
    extern __shared__ __align__(16) float attn_smem[];
    const AttnBwdTile t = attn_bwd_tile<BT, CD, CT>(attn_smem);
    const int n = (int)a.div_Mk.div(blockIdx.y), kv = (int)blockIdx.y - n * a.Mk;
    const int r0 = (int)(gridDim.x - 1 - blockIdx.x) * BT;
    const int len = attn_len(a, n);
    const int last_tok = (int)a.div_G.div((uint32_t)min(r0 + BT - 1, a.rows - 1));
    const int kmax = a.causal ? max(0, min(len, last_tok + len - a.Lq + 1)) : len;
    __syncthreads();
    attn_bwd_rows<T, BT, CD, CT>(a, t, n, kv, r0);
    float acc[2][RT][CD];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int c = 0; c < CD; ++c) acc[s][r][c] = 0.f;
    for (int j0 = 0; j0 < kmax; j0 += BT) {
        __syncthreads();
        attn_bwd_keys<T, BT, CD, CT>(a, t, n, kv, j0, len);
        __syncthreads();
        attn_bwd_scores<BT, CD, CT, false>(a, t, r0, j0, len);
        __syncthreads();
        attn_weighted_tile<RT, CD>(t.S, lds, t.Ks, ldq, BT, acc[0]);
        attn_weighted_tile<RT, CD>(t.S + BT * lds, lds, t.Ks + 16 * CD, ldq, BT, acc[1]);
    }
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int row = r0 + (threadIdx.x >> 4) + 16 * r;
        if (row >= a.rows) continue;
        const uint32_t tok = a.div_G.div((uint32_t)row);
        const int head = kv * a.G + row - (int)tok * a.G;
        T* out = static_cast<T*>(a.gq) + (((long long)n * a.Lq + tok) * a.M + head) * 2 * a.D;
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int c = 0; c < CD; ++c)
                if (attn_col<CD>(c) < a.D)
                    out[s * a.D + attn_col<CD>(c)] = Elem<T>::from(acc[s][r][c] * a.scale);
    }
}

template <typename T, int BT, int CD, int CT>
__global__ void __launch_bounds__(kAttnThreads) diff_attn_dkv_kernel(const AttnArgs a) {
    constexpr int RT = BT / 16, ldq = 32 * CD + 4, ldv = attn_ldv(CT), lds = BT + 4;
    extern __shared__ __align__(16) float attn_smem[];
    const AttnBwdTile t = attn_bwd_tile<BT, CD, CT>(attn_smem);
    const int n = (int)a.div_Mk.div(blockIdx.y), kv = (int)blockIdx.y - n * a.Mk;
    const int j0 = (int)blockIdx.x * BT;          // the first key tiles see the most rows
    const int len = attn_len(a, n);
    __syncthreads();
    attn_bwd_keys<T, BT, CD, CT>(a, t, n, kv, j0, len);
    float gk[2][RT][CD], gv[RT][CT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int c = 0; c < CD; ++c) gk[s][r][c] = 0.f;
#pragma unroll
        for (int c = 0; c < CT; ++c) gv[r][c] = 0.f;
    }
    // tokens before i0 see none of these keys
    const long long i0 = a.causal ? max(0, j0 - len + a.Lq) : 0;
    const int first = j0 < len ? (int)(i0 * a.G / BT * BT) : a.rows;
    for (int r0 = first; r0 < a.rows; r0 += BT) {
        __syncthreads();
        attn_bwd_rows<T, BT, CD, CT>(a, t, n, kv, r0);
        __syncthreads();
        attn_bwd_scores<BT, CD, CT, true>(a, t, r0, j0, len);
        __syncthreads();
        attn_weighted_tile<RT, CD>(t.S, lds, t.Qs, ldq, BT, gk[0]);
        attn_weighted_tile<RT, CD>(t.S + BT * lds, lds, t.Qs + 16 * CD, ldq, BT, gk[1]);
        attn_weighted_tile<RT, CT>(t.S + 2 * BT * lds, lds, t.Gs, ldv, BT, gv);
    }
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int j = j0 + (threadIdx.x >> 4) + 16 * r;
        if (j >= a.Lk) continue;
        const long long at = ((long long)n * a.Lk + j) * a.Mk + kv;
        T* okey = static_cast<T*>(a.gk) + at * 2 * a.D;
        T* ov = static_cast<T*>(a.gv) + at * a.Dv;
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int c = 0; c < CD; ++c)
                if (attn_col<CD>(c) < a.D)
                    okey[s * a.D + attn_col<CD>(c)] = Elem<T>::from(gk[s][r][c] * a.scale);
#pragma unroll
        for (int c = 0; c < CT; ++c)
            if (attn_col<CT>(c) < a.Dv) ov[attn_col<CT>(c)] = Elem<T>::from(gv[r][c]);
    }
}

}  // namespace dcnb
