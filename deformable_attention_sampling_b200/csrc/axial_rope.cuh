// Rotary positions over one to four axes, forward and gradient (sm_100a).
//
// Pair i < R of a head's channels turns by th_i = pos[axis(i)] * freqs[i]:
//   (a, b) -> (a cos th - b sin th, a sin th + b cos th),
// with (a, b) channels (2i, 2i + 1) (interleaved) or (i, i + R) (halves);
// channels from 2R on pass through.  The gradient of the channels is the turn
// by -th; that of a position sums, over the heads and the axis's pairs,
//   freqs[i] * (gb * a' - ga * b'),   (a', b') the turned pair.
//
// Measured: 16.5 us for 2 x 15000 tokens of 8 x 32 in float32 (9.4 us at the
// measured copy rate), 47 us for the gradient of 2 x 12136 tokens of 16 x 64 in
// bf16 (23 us): each token's angles (float64, sine and cosine) come before its
// few vectors.  Positions that a batch shares cost its gradient their parallelism: a
// token's team then walks all images (float32, 8 x 32: 64 images of 300 tokens 66 us,
// 13 with positions of their own; 256 of 100 tokens 323 and 16; 2 of 15000 18 and 21).
// Bound: one read of x (and grad_out) and one write, so HBM for many tokens
// and launch latency for few.  The angles are the only other work: R per
// token, shared by its M heads.  A team of `tpt` lanes (a power of two up to a
// warp) owns one token: it forms the token's R (cos, sin) pairs in shared
// memory once and then turns the token's heads with 16-byte accesses.
//
// Angles: the product is formed in float64 as a count of turns and reduced by
// rint there, because float32 holds a position of 1e5 times a frequency of 1
// only to 0.004 rad; what is left (|t| <= 1/2 turn) is exact enough in float32.
#pragma once

#include "common.cuh"

namespace dcnb {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxPairs = 256;
constexpr int kRopeMaxAxes = 4;

struct RopeArgs {
    const void* x;
    const float* pos;
    const float* freqs;
    const void* go;            // gradient kernel: gradient of the turned channels
    void* out;                 // turned channels, or their gradient with respect to x
    float* grad_pos;           // gradient kernel, or null
    int L, M, D, R, A;
    int pair_end[kRopeMaxAxes];   // first pair past axis a
    long long x_image, x_row;  // elements between images / tokens of x
    long long units;           // tokens that teams own
    int images;                // images a unit spans (positions shared by the batch), else 1
    int shared_pos;            // 1: pos has one image for all
    int tpt;                   // lanes per token, a power of two
    int tasks;                 // vector tasks per head
    int jl, hl;                // a team's lanes over a head's tasks, heads side by side
    FastDiv div_jl, div_L;
    float sign;                // -1: turn backwards
};

// VB bytes, cached normally: x may be the output itself (in place), so the
// read-only path is not used.
template <int VB>
__device__ __forceinline__ void ld_words(const void* p, uint32_t* w) {
    if constexpr (VB == 16) {
        const uint4 v = *static_cast<const uint4*>(p);
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else if constexpr (VB == 8) {
        const uint2 v = *static_cast<const uint2*>(p);
        w[0] = v.x; w[1] = v.y;
    } else if constexpr (VB == 4) {
        w[0] = *static_cast<const uint32_t*>(p);
    } else {
        w[0] = *static_cast<const unsigned short*>(p);
    }
}

template <int VB>
__device__ __forceinline__ void st_words(void* p, const uint32_t* w) {
    if constexpr (VB == 16) *static_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (VB == 8) *static_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else if constexpr (VB == 4) *static_cast<uint32_t*>(p) = w[0];
    else *static_cast<unsigned short*>(p) = (unsigned short)w[0];
}

template <typename T, int V>
__device__ __forceinline__ void ld_f32(const T* p, float* f) {
    uint32_t w[(V * (int)sizeof(T) + 3) / 4];
    ld_words<V * (int)sizeof(T)>(p, w);
    widen<T, V>(w, f);
}

template <typename T, int V>
__device__ __forceinline__ void st_f32(T* p, const float* f) {
    uint32_t w[(V * (int)sizeof(T) + 3) / 4];
    narrow<T, V>(f, w);
    st_words<V * (int)sizeof(T)>(p, w);
}

// V elements per access.  INTER with V > 1: a task is one vector of V channels
// (V / 2 pairs, or V channels that pass).  Halves, or V = 1: a task is V pairs
// in two vectors, or one vector that passes.
// A team's lanes lie side by side over a head's tasks (jl of them) and over
// heads: a lane keeps its task, its turns in registers and the sums of its
// pairs' position gradients, and steps over the heads with the next one's loads
// in flight.
template <typename T, int V, bool INTER, bool GRAD>
__global__ void __launch_bounds__(kRopeThreads) axial_rope_kernel(const RopeArgs a) {
    extern __shared__ float2 rope_turns[];       // [teams][R] (cos, sin)
    constexpr bool VINTER = INTER && V > 1;
    constexpr int P = VINTER ? V / 2 : V;        // pairs of a task
    constexpr int NV = VINTER ? 1 : 2;           // vectors of a task
    constexpr int W = (V * (int)sizeof(T) + 3) / 4;
    const int tpt = a.tpt;
    const int team = threadIdx.x / tpt, lane = threadIdx.x & (tpt - 1);
    const long long unit = (long long)blockIdx.x * (kRopeThreads / tpt) + team;
    const bool live = unit < a.units;
    float2* turns = rope_turns + team * a.R;
    const uint32_t u = live ? (uint32_t)unit : 0u;
    const uint32_t img = a.images > 1 ? 0u : a.div_L.div(u);
    const uint32_t l = a.images > 1 ? u : u - img * (uint32_t)a.L;
    const long long prow = a.shared_pos ? (long long)l : (long long)img * a.L + l;
    const int hsub = (int)a.div_jl.div((uint32_t)lane);
    const int j0 = lane - hsub * a.jl;
    const bool want_pos = GRAD && a.grad_pos != nullptr;

    uint32_t src_w[NV][W], x_w[NV][W];           // the next head's vectors
    // first channel of each vector of task j
    auto channel = [&](int j, int v) {
        if (VINTER) return j * V;
        const int i0 = j * V;
        if (i0 >= a.R) return i0 + a.R;          // 2R + (i0 - R): passes, one vector
        return INTER ? 2 * i0 + v : i0 + v * a.R;
    };
    auto fetch = [&](int n, int j, int m) {
        if (m >= a.M) return;
        const long long token = ((long long)img + n) * a.L + l;
        const T* x = static_cast<const T*>(a.x) + ((long long)img + n) * a.x_image +
                     (long long)l * a.x_row + m * a.D;
        const T* src = GRAD ? static_cast<const T*>(a.go) + token * ((long long)a.M * a.D) + m * a.D
                            : x;
        const bool turned = VINTER ? j * V < 2 * a.R : j * V < a.R;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (v == 1 && !turned) break;
            ld_words<V * (int)sizeof(T)>(src + channel(j, v), src_w[v]);
            if (want_pos && turned) ld_words<V * (int)sizeof(T)>(x + channel(j, v), x_w[v]);
        }
    };
    const bool active = live && hsub < a.hl;
    if (active && j0 < a.tasks) fetch(0, j0, hsub);
    if (live) {
        for (int i = lane; i < a.R; i += tpt) {
            int ax = 0;
            while (ax + 1 < a.A && i >= a.pair_end[ax]) ++ax;
            double t = (double)a.pos[prow * a.A + ax] * (double)a.freqs[i] *
                       0.15915494309189533576888376337251436;
            t -= rint(t);
            float s, c;
            sincospif(2.0f * (float)t, &s, &c);
            turns[i] = make_float2(c, s * a.sign);
        }
    }
    __syncwarp();
    float acc[kRopeMaxAxes] = {0.f, 0.f, 0.f, 0.f};
    if (active) {
        for (int j = j0; j < a.tasks; j += a.jl) {
            const bool turned = VINTER ? j * V < 2 * a.R : j * V < a.R;
            float2 cs[P];
            float sums[P];
#pragma unroll
            for (int e = 0; e < P; ++e) {
                cs[e] = turned ? turns[j * P + e] : make_float2(1.f, 0.f);
                sums[e] = 0.f;
            }
            for (int n = 0; n < a.images; ++n) {
                if (j != j0 || n > 0) fetch(n, j, hsub);
                T* out = static_cast<T*>(a.out) +
                         (((long long)img + n) * a.L + l) * ((long long)a.M * a.D);
                for (int m = hsub; m < a.M; m += a.hl) {
                    float f[NV][V], xv[NV][V];
#pragma unroll
                    for (int v = 0; v < NV; ++v) {
                        widen<T, V>(src_w[v], f[v]);
                        if (want_pos) widen<T, V>(x_w[v], xv[v]);
                    }
                    fetch(n, j, m + a.hl);
                    if (turned) {
#pragma unroll
                        for (int e = 0; e < P; ++e) {
                            float& fa = VINTER ? f[0][2 * e] : f[0][e];
                            float& fb = VINTER ? f[0][2 * e + 1] : f[NV - 1][e];
                            // GRAD: the turn by -th of the gradient
                            const float s = GRAD ? -cs[e].y : cs[e].y;
                            if (want_pos) {
                                const float xa = VINTER ? xv[0][2 * e] : xv[0][e];
                                const float xb = VINTER ? xv[0][2 * e + 1] : xv[NV - 1][e];
                                const float oa = xa * cs[e].x - xb * cs[e].y;
                                const float ob = xa * cs[e].y + xb * cs[e].x;
                                sums[e] += fb * oa - fa * ob;
                            }
                            const float ra = fa * cs[e].x - fb * s;
                            fb = fa * s + fb * cs[e].x;
                            fa = ra;
                        }
                    }
#pragma unroll
                    for (int v = 0; v < NV; ++v)
                        if (v == 0 || turned) st_f32<T, V>(out + m * a.D + channel(j, v), f[v]);
                }
            }
            if (want_pos && turned) {
#pragma unroll
                for (int e = 0; e < P; ++e) {
                    const int i = j * P + e;
                    int ax = 0;
                    while (ax + 1 < a.A && i >= a.pair_end[ax]) ++ax;
                    const float d = a.freqs[i] * sums[e];
#pragma unroll
                    for (int k = 0; k < kRopeMaxAxes; ++k) acc[k] += k == ax ? d : 0.f;
                }
            }
        }
    }
    if (want_pos) {       // uniform over the grid: every lane of the warp takes part
#pragma unroll
        for (int k = 0; k < kRopeMaxAxes; ++k)
            for (int o = tpt >> 1; o > 0; o >>= 1)
                acc[k] += __shfl_xor_sync(0xffffffffu, acc[k], o);
        // the inverse turn's angle is -pos * freqs: a.sign is its derivative's sign
        if (live && lane < a.A) {
            float v = acc[0];
#pragma unroll
            for (int k = 1; k < kRopeMaxAxes; ++k) v = lane == k ? acc[k] : v;
            a.grad_pos[prow * a.A + lane] = v * a.sign;
        }
    }
}

}  // namespace dcnb
