// The join of two blocks of a residual network, forward and gradient (sm_100a).
//
//   u = norm(y) * post_weight + post_bias      (or u = y)
//   z = x + scale[c] * gate[n][c] * u
//   h = norm(z) * pre_weight + pre_bias        (or no h)
// norm: layer (subtract the mean, divide by sqrt(variance + eps)) or rms
// (divide by sqrt(mean square + eps)), over the C channels of a row.
//
// Measured: 34 us for 64 x 3136 x 64 in fp16 (103 MB, 16 us at the measured copy
// rate), 85 us forward and 141 + 10 us backward for 8 x 4096 x 1024 in bf16 (268
// and 403 MB): a team's sums, not the bytes, set the step.  Longer rows, 67 MB a
// tensor in bf16 (floors 41 and 61 us): 8192 x 4096 forward 88, backward 178 us; 4096
// x 8192 forward 130, backward 391 us, whose blocks of 1024 threads spill (below).
// Bound: HBM.  One pass over the rows: x and y are read once, z and h written
// once, the rows' statistics stay in registers (two-pass: the mean first, then
// the squared deviations, so that a large mean costs no digits), and h is the
// norm of z before its rounding.  A row belongs to a team of `tpr` threads (a
// power of two), eight consecutive channels a thread; the per-channel factors
// of those channels stay in registers while the team walks its rows.
//
// Gradient, from y, z (as stored), grad_z and grad_h, with n1 = norm(y)'s and
// n2 = norm(z)'s normalised rows, r1 and r2 their reciprocal spreads:
//   g      = grad_z + back(grad_h * pre_weight; n2, r2)       grad_x = g
//   gu     = g * scale * gate
//   grad_y = back(gu * post_weight; n1, r1)                   (or gu)
//   back(v; n, r) = r * (v - mean(v) - n * mean(v * n))       (rms: no mean(v))
// and the factors' gradients from four column sums per image,
//   A = sum_l g * n1, B = sum_l g, E = sum_l grad_h * n2, F = sum_l grad_h:
//   grad_gate = scale * (post_weight * A + post_bias * B), and so on.
// h was the norm of z before its rounding; n2 here is that of z as stored.  That
// costs 16-bit gradients 1.4 times the error of rounding them once; the unrounded z
// would have to be saved in float32, or formed again from x and the first norm.
// Every block sums its rows of one image in registers and writes one partial
// row; a second kernel adds the partials in a fixed order, so the gradients do
// not depend on the order in which blocks run.
#pragma once

#include "axial_rope.cuh"

namespace dcnb {

constexpr int kNormV = 8;               // channels per thread
constexpr int kNormMaxThreads = 1024;
constexpr int kNormMaxC = kNormV * kNormMaxThreads;
constexpr int kNormFinalCols = 32;      // columns of one block of the second kernel
constexpr int kNormFinalRows = 32;

struct NormArgs {
    const void* x;
    const void* y;
    const void* post_w;
    const void* post_b;
    const void* gate;      // [images][C] or null
    const void* scale;     // [C] or null
    const void* pre_w;
    const void* pre_b;
    void* z;               // forward: output; gradient: input
    void* h;
    const void* gz;
    const void* gh;
    void* gx;
    void* gy;
    float* partial;        // [images * blocks_per_image][4][C]
    long long rows_per_image;   // rows that share a gate
    long long images;
    int blocks_per_image;
    int C;
    int tpr;               // threads per row
    int rms, post, pre;
    float eps;
};

// Eight channels of a row as stored, loaded ahead of their use.
template <typename T>
struct NormRaw {
    uint32_t w[2 * sizeof(T)];
};

template <typename T, bool VEC>
__device__ __forceinline__ void norm_fetch(const void* p, long long at, int c, int C, bool live,
                                           NormRaw<T>& r) {
    const T* q = static_cast<const T*>(p) + at + c;
    if constexpr (VEC) {
        if (live && c < C) {
            ld_words<16>(q, r.w);
            if constexpr (sizeof(T) == 4) ld_words<16>(q + 4, r.w + 4);
        } else {
#pragma unroll
            for (int i = 0; i < 2 * (int)sizeof(T); ++i) r.w[i] = 0u;
        }
    } else {
        float f[kNormV];               // widening and rounding back are exact
#pragma unroll
        for (int e = 0; e < kNormV; ++e) f[e] = live && c + e < C ? Elem<T>::one(q + e) : 0.f;
        narrow<T, kNormV>(f, r.w);
    }
}

template <typename T, bool VEC>
__device__ __forceinline__ void norm_load(const void* p, long long at, int c, int C, float* f) {
    const T* q = static_cast<const T*>(p) + at;
    if constexpr (VEC) {
        if (c < C) {
            if constexpr (sizeof(T) == 2) {
                ld_f32<T, 8>(q + c, f);
            } else {
                ld_f32<T, 4>(q + c, f);
                ld_f32<T, 4>(q + c + 4, f + 4);
            }
        } else {
#pragma unroll
            for (int e = 0; e < kNormV; ++e) f[e] = 0.f;
        }
    } else {
#pragma unroll
        for (int e = 0; e < kNormV; ++e) f[e] = c + e < C ? Elem<T>::one(q + c + e) : 0.f;
    }
}

template <typename T, bool VEC>
__device__ __forceinline__ void norm_store(void* p, long long at, int c, int C, const float* f) {
    T* q = static_cast<T*>(p) + at;
    if constexpr (VEC) {
        if (c < C) {
            if constexpr (sizeof(T) == 2) {
                st_f32<T, 8>(q + c, f);
            } else {
                st_f32<T, 4>(q + c, f);
                st_f32<T, 4>(q + c + 4, f + 4);
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < kNormV; ++e)
            if (c + e < C) q[c + e] = Elem<T>::from(f[e]);
    }
}

// A factor of the thread's channels, or `otherwise` where there is none.
template <typename T, bool VEC>
__device__ __forceinline__ void norm_factor(const void* p, long long at, int c, int C,
                                            float otherwise, float* f) {
    if (p) {
        norm_load<T, VEC>(p, at, c, C, f);
    } else {
#pragma unroll
        for (int e = 0; e < kNormV; ++e) f[e] = otherwise;
    }
}

// Sums of two values over the row's team.  Teams up to a warp: shuffles.
// Larger: shuffles, then the team's warps through shared memory; `slot`
// alternates between two buffers, so one barrier a call is enough.  All
// threads of the block call it.
struct TeamSum {
    float2* buf;     // [2][32]
    int slot;
    int tpr;
    __device__ __forceinline__ float2 operator()(float a, float b) {
        const int w = tpr < 32 ? tpr : 32;
        for (int o = w >> 1; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, o);
            b += __shfl_xor_sync(0xffffffffu, b, o);
        }
        if (tpr > 32) {
            float2* s = buf + slot * 32;
            slot ^= 1;
            const int warp = threadIdx.x >> 5;
            if ((threadIdx.x & 31) == 0) s[warp] = make_float2(a, b);
            __syncthreads();
            const int n = tpr >> 5, first = warp & ~(n - 1);
            // every lane of a warp adds the same words in the same order
            a = b = 0.f;
            for (int i = 0; i < n; ++i) {
                const float2 v = s[first + i];
                a += v.x;
                b += v.y;
            }
        }
        return make_float2(a, b);
    }
};

// Blocks of 256 threads (rows of up to 2048 channels) and of 512 (up to 4096)
// have 128 registers a thread, which hold every factor and the next row of 16-bit
// data; float32 rows (32 to 136 bytes) and the element-wise 16-bit gradient (96 or
// 128 bytes) spill a little.  Longer rows take 1024 threads at 64 registers and spill
// 324 to 640 bytes.
constexpr int kNormSmall = 256;
constexpr int kNormMiddle = 512;

// A team works on two rows at a time: one sum over the team serves both, and
// four tensors' loads are in flight beside the next two rows'.
template <typename T, bool VEC, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == kNormSmall ? 2 : 1)
    norm_residual_kernel(const NormArgs a) {
    __shared__ float2 buf[64];
    const int tpr = a.tpr, teams = blockDim.x / tpr;
    const int team = threadIdx.x / tpr, c = (threadIdx.x & (tpr - 1)) * kNormV, C = a.C;
    TeamSum sum{buf, 0, tpr};
    const long long rows = a.rows_per_image * a.images;
    const long long r_begin = rows * blockIdx.x / gridDim.x;
    const long long r_end = rows * (blockIdx.x + 1) / gridDim.x;
    const float inv_c = 1.f / (float)C;
    float pw[kNormV], pb[kNormV], sc[kNormV], qw[kNormV], qb[kNormV];
    norm_factor<T, VEC>(a.post_w, 0, c, C, 1.f, pw);
    norm_factor<T, VEC>(a.post_b, 0, c, C, 0.f, pb);
    norm_factor<T, VEC>(a.scale, 0, c, C, 1.f, sc);
    norm_factor<T, VEC>(a.pre_w, 0, c, C, 1.f, qw);
    norm_factor<T, VEC>(a.pre_b, 0, c, C, 0.f, qb);
    // The normalised rows in place of v, from both rows' sums over the team.
    auto normalise = [&](float (&v)[2][kNormV]) {
        if (!a.rms) {
            float s[2] = {0.f, 0.f};
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int e = 0; e < kNormV; ++e) s[k] += v[k][e];
            const float2 m = sum(s[0], s[1]);
#pragma unroll
            for (int e = 0; e < kNormV; ++e) {
                v[0][e] = c + e < C ? v[0][e] - m.x * inv_c : 0.f;
                v[1][e] = c + e < C ? v[1][e] - m.y * inv_c : 0.f;
            }
        }
        float q[2] = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < kNormV; ++e) q[k] += v[k][e] * v[k][e];
        const float2 t = sum(q[0], q[1]);
        const float r0 = 1.0f / sqrtf(t.x * inv_c + a.eps), r1 = 1.0f / sqrtf(t.y * inv_c + a.eps);
#pragma unroll
        for (int e = 0; e < kNormV; ++e) {
            v[0][e] *= r0;
            v[1][e] *= r1;
        }
    };
    NormRaw<T> ry[2], rx[2];
    auto fetch = [&](long long r) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const long long at = r + k * teams;
            norm_fetch<T, VEC>(a.y, at * C, c, C, at < r_end, ry[k]);
            norm_fetch<T, VEC>(a.x, at * C, c, C, at < r_end, rx[k]);
        }
    };
    fetch(r_begin + team);
    // all teams of a block take the same number of steps (barriers in the sums)
    for (long long r0 = r_begin; r0 < r_end; r0 += 2 * teams) {
        float z[2][kNormV], v[2][kNormV];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            widen<T, kNormV>(rx[k].w, z[k]);
            widen<T, kNormV>(ry[k].w, v[k]);
        }
        fetch(r0 + team + 2 * teams);
        if (a.post) normalise(v);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const long long r = r0 + team + k * teams;
            const bool live = r < r_end;
            float gt[kNormV];
            norm_factor<T, VEC>(live ? a.gate : nullptr, live ? r / a.rows_per_image * C : 0, c, C,
                                1.f, gt);
#pragma unroll
            for (int e = 0; e < kNormV; ++e) {
                const float u = a.post ? v[k][e] * pw[e] + pb[e] : v[k][e];
                z[k][e] = c + e < C ? z[k][e] + sc[e] * gt[e] * u : 0.f;
            }
            if (live) norm_store<T, VEC>(a.z, r * C, c, C, z[k]);
        }
        if (a.pre) {
            normalise(z);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const long long r = r0 + team + k * teams;
#pragma unroll
                for (int e = 0; e < kNormV; ++e) z[k][e] = z[k][e] * qw[e] + qb[e];
                if (r < r_end) norm_store<T, VEC>(a.h, r * C, c, C, z[k]);
            }
        }
    }
}

// Rows' gradients and the blocks' column sums.  Block b sums rows of image
// b / blocks_per_image only.
template <typename T, bool VEC, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == kNormSmall ? 2 : 1)
    norm_residual_grad_kernel(const NormArgs a) {
    __shared__ float2 buf[64];
    extern __shared__ float norm_cols[];       // [teams - 1][tpr * 8] of one sum
    const int tpr = a.tpr, teams = blockDim.x / tpr;
    const int team = threadIdx.x / tpr, c = (threadIdx.x & (tpr - 1)) * kNormV, C = a.C;
    TeamSum sum{buf, 0, tpr};
    const long long image = blockIdx.x / a.blocks_per_image;
    const int part = (int)(blockIdx.x - image * a.blocks_per_image);
    const long long first = image * a.rows_per_image;
    const long long r_begin = first + a.rows_per_image * part / a.blocks_per_image;
    const long long r_end = first + a.rows_per_image * (part + 1) / a.blocks_per_image;
    const float inv_c = 1.f / (float)C;
    float pw[kNormV], fac[kNormV], qw[kNormV];
    float sA[kNormV], sB[kNormV], sE[kNormV], sF[kNormV];
    norm_factor<T, VEC>(a.post_w, 0, c, C, 1.f, pw);
    norm_factor<T, VEC>(a.scale, 0, c, C, 1.f, fac);
    norm_factor<T, VEC>(a.pre_w, 0, c, C, 1.f, qw);
    {
        float gt[kNormV];
        norm_factor<T, VEC>(a.gate, image * C, c, C, 1.f, gt);
#pragma unroll
        for (int e = 0; e < kNormV; ++e) {
            fac[e] *= gt[e];
            sA[e] = sB[e] = sE[e] = sF[e] = 0.f;
        }
    }
    NormRaw<T> ry, rz, rg, rh;
    auto fetch = [&](long long r) {
        const bool live = r < r_end;
        norm_fetch<T, VEC>(a.y, r * C, c, C, live, ry);
        norm_fetch<T, VEC>(a.gz, r * C, c, C, live, rg);
        norm_fetch<T, VEC>(a.z, r * C, c, C, live && a.pre, rz);
        norm_fetch<T, VEC>(a.gh, r * C, c, C, live && a.pre, rh);
    };
    fetch(r_begin + team);
    for (long long r0 = r_begin; r0 < r_end; r0 += teams) {
        const long long r = r0 + team;
        const bool live = r < r_end;
        float yv[kNormV], zv[kNormV], g[kNormV], gh[kNormV];
        widen<T, kNormV>(ry.w, yv);
        widen<T, kNormV>(rz.w, zv);
        widen<T, kNormV>(rg.w, g);
        widen<T, kNormV>(rh.w, gh);
        fetch(r + teams);
        // both norms' statistics, two sums at a time
        float my = 0.f, mz = 0.f, r1 = 0.f, r2 = 0.f;
        if (!a.rms) {
            float p = 0.f, q = 0.f;
#pragma unroll
            for (int e = 0; e < kNormV; ++e) {
                p += yv[e];
                q += zv[e];
            }
            const float2 s = sum(p, q);
            my = a.post ? s.x * inv_c : 0.f;
            mz = s.y * inv_c;
        }
        {
            float p = 0.f, q = 0.f;
#pragma unroll
            for (int e = 0; e < kNormV; ++e) {
                yv[e] = c + e < C ? yv[e] - my : 0.f;
                zv[e] = c + e < C ? zv[e] - mz : 0.f;
                p += yv[e] * yv[e];
                q += zv[e] * zv[e];
            }
            const float2 s = sum(p, q);
            // (a team without a row has zeros here: with eps = 0 their spread is 0 too, and
            // 0 / 0 would go into the column sums)
            r1 = !a.post ? 1.f : live ? 1.0f / sqrtf(s.x * inv_c + a.eps) : 0.f;
            r2 = live ? 1.0f / sqrtf(s.y * inv_c + a.eps) : 0.f;
        }
        if (a.pre) {
            float p = 0.f, q = 0.f;
#pragma unroll
            for (int e = 0; e < kNormV; ++e) {
                zv[e] *= r2;
                sE[e] += gh[e] * zv[e];
                sF[e] += gh[e];
                gh[e] *= qw[e];
                p += gh[e];
                q += gh[e] * zv[e];
            }
            const float2 s = sum(p, q);
            const float m1 = a.rms ? 0.f : s.x * inv_c, m2 = s.y * inv_c;
#pragma unroll
            for (int e = 0; e < kNormV; ++e) g[e] += r2 * (gh[e] - m1 - zv[e] * m2);
        }
        if (live) norm_store<T, VEC>(a.gx, r * C, c, C, g);
        float p = 0.f, q = 0.f;
#pragma unroll
        for (int e = 0; e < kNormV; ++e) {
            if (!live || c + e >= C) g[e] = 0.f;
            yv[e] *= r1;
            sA[e] += g[e] * yv[e];
            sB[e] += g[e];
            g[e] *= fac[e];
            if (a.post) g[e] *= pw[e];
            p += g[e];
            q += g[e] * yv[e];
        }
        if (a.post) {
            const float2 s = sum(p, q);
            const float m1 = a.rms ? 0.f : s.x * inv_c, m2 = s.y * inv_c;
#pragma unroll
            for (int e = 0; e < kNormV; ++e) g[e] = r1 * (g[e] - m1 - yv[e] * m2);
        }
        if (live) norm_store<T, VEC>(a.gy, r * C, c, C, g);
    }
    // the teams' sums, in team order, one of the four at a time
    float* out = a.partial + (long long)blockIdx.x * 4 * C;
    float* s4[4] = {sA, sB, sE, sF};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        __syncthreads();
        if (team > 0) {
#pragma unroll
            for (int e = 0; e < kNormV; ++e)
                norm_cols[(team - 1) * tpr * kNormV + c + e] = s4[k][e];
        }
        __syncthreads();
        if (team == 0) {
#pragma unroll
            for (int e = 0; e < kNormV; ++e) {
                float v = s4[k][e];
                for (int t = 0; t + 1 < teams; ++t) v += norm_cols[t * tpr * kNormV + c + e];
                if (c + e < C) out[(long long)k * C + c + e] = v;
            }
        }
    }
}

struct NormFinalArgs {
    const float* partial;
    const void* scale;
    const void* gate;
    const void* post_w;
    const void* post_b;
    void* gscale;
    void* ggate;
    void* gpost_w;
    void* gpost_b;
    void* gpre_w;
    void* gpre_b;
    long long images;
    int blocks_per_image;
    int C;
    int segments;          // threads that share an image's partials (power of two)
};

// One block: 32 channels x 32 threads.  Thread row t adds segment t % segments
// of the partials of images t / segments, + 32 / segments, ...
template <typename T>
__global__ void __launch_bounds__(kNormFinalCols* kNormFinalRows)
    norm_residual_final_kernel(const NormFinalArgs a) {
    __shared__ float4 part[kNormFinalRows][kNormFinalCols + 1];
    __shared__ float2 part2[kNormFinalRows][kNormFinalCols + 1];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int c = blockIdx.x * kNormFinalCols + tx, C = a.C;
    const bool in = c < C;
    const int seg = ty % a.segments, lane_image = ty / a.segments;
    const int step = kNormFinalRows / a.segments;
    auto one = [&](const void* p, long long at, float otherwise) {
        return p && in ? Elem<T>::one(static_cast<const T*>(p) + at) : otherwise;
    };
    const float sc = one(a.scale, c, 1.f), pw = one(a.post_w, c, 1.f), pb = one(a.post_b, c, 0.f);
    float g_scale = 0.f, g_pw = 0.f, g_pb = 0.f, g_qw = 0.f, g_qb = 0.f;
    const int b0 = (int)((long long)a.blocks_per_image * seg / a.segments);
    const int b1 = (int)((long long)a.blocks_per_image * (seg + 1) / a.segments);
    const long long rounds = (a.images + step - 1) / step;
    for (long long k = 0; k < rounds; ++k) {
        const long long n = k * step + lane_image;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (n < a.images && in) {
            const float* p = a.partial + (n * a.blocks_per_image + b0) * 4LL * C + c;
#pragma unroll 4
            for (int b = b0; b < b1; ++b, p += 4LL * C) {
                v.x += p[0];
                v.y += p[C];
                v.z += p[2LL * C];
                v.w += p[3LL * C];
            }
        }
        if (a.segments > 1) {
            __syncthreads();
            part[ty][tx] = v;
            __syncthreads();
            if (seg == 0) {
                for (int s = 1; s < a.segments; ++s) {
                    const float4 w = part[ty + s][tx];
                    v.x += w.x;
                    v.y += w.y;
                    v.z += w.z;
                    v.w += w.w;
                }
            }
        }
        if (seg == 0 && n < a.images && in) {
            const float gt = one(a.gate, n * C + c, 1.f);
            const float t = pw * v.x + pb * v.y;          // sum over rows of g * u
            if (a.ggate) static_cast<T*>(a.ggate)[n * C + c] = Elem<T>::from(sc * t);
            g_scale += gt * t;
            g_pw += gt * sc * v.x;
            g_pb += gt * sc * v.y;
            g_qw += v.z;
            g_qb += v.w;
        }
    }
    __syncthreads();
    part[ty][tx] = make_float4(g_scale, g_pw, g_pb, g_qw);
    part2[ty][tx] = make_float2(g_qb, 0.f);
    __syncthreads();
    if (ty == 0 && in) {
        for (int t = 1; t < kNormFinalRows; ++t) {
            const float4 w = part[t][tx];
            g_scale += w.x;
            g_pw += w.y;
            g_pb += w.z;
            g_qw += w.w;
            g_qb += part2[t][tx].x;
        }
        if (a.gscale) static_cast<T*>(a.gscale)[c] = Elem<T>::from(g_scale);
        if (a.gpost_w) static_cast<T*>(a.gpost_w)[c] = Elem<T>::from(g_pw);
        if (a.gpost_b) static_cast<T*>(a.gpost_b)[c] = Elem<T>::from(g_pb);
        if (a.gpre_w) static_cast<T*>(a.gpre_w)[c] = Elem<T>::from(g_qw);
        if (a.gpre_b) static_cast<T*>(a.gpre_b)[c] = Elem<T>::from(g_qb);
    }
}

}  // namespace dcnb
