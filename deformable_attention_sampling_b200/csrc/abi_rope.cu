// C interface of libdcn_b200.so: axial_rope_forward, axial_rope_backward.
#include "abi_common.cuh"
#include "axial_rope.cuh"

using namespace dcnb_abi;

namespace {

template <typename T, bool INTER, bool GRAD>
const void* rope_kernel_v(int v) {
    switch (v) {
        case 8:
            if constexpr (sizeof(T) == 2 && (INTER || !GRAD))
                return (const void*)dcnb::axial_rope_kernel<T, 8, INTER, GRAD>;
            return nullptr;
        case 4: return (const void*)dcnb::axial_rope_kernel<T, 4, INTER, GRAD>;
        case 2: return (const void*)dcnb::axial_rope_kernel<T, 2, INTER, GRAD>;
        case 1: return (const void*)dcnb::axial_rope_kernel<T, 1, INTER, GRAD>;
        default: return nullptr;
    }
}

template <typename T>
const void* rope_kernel_for(int v, bool inter, bool grad) {
    if (inter) return grad ? rope_kernel_v<T, true, true>(v) : rope_kernel_v<T, true, false>(v);
    return grad ? rope_kernel_v<T, false, true>(v) : rope_kernel_v<T, false, false>(v);
}

// The common part of both directions; `go` null: forward.
int rope_launch(const void* x, const float* pos, const float* freqs, const void* go, void* out,
                float* grad_pos, const int* axis_pairs, int N, int L, int M, int D, int A,
                int pos_images, long long x_image, long long x_row, int interleaved, int inverse,
                int dtype, bool grad, void* stream) {
    const int es = elem_bytes(dtype);
    if (es == 0 || N < 0 || L < 0 || M <= 0 || D <= 0 || A <= 0 || !axis_pairs ||
        (pos_images != 1 && pos_images != N) || (interleaved != 0 && interleaved != 1) ||
        (inverse != 0 && inverse != 1))
        return DCN_ERR_INVALID_ARG;
    if (A > dcnb::kRopeMaxAxes) return DCN_ERR_UNSUPPORTED;
    dcnb::RopeArgs a;
    long long R = 0;
    for (int i = 0; i < A; ++i) {
        if (axis_pairs[i] < 0) return DCN_ERR_INVALID_ARG;
        R += axis_pairs[i];
        if (2 * R > D) return DCN_ERR_INVALID_ARG;
        a.pair_end[i] = (int)R;
    }
    for (int i = A; i < dcnb::kRopeMaxAxes; ++i) a.pair_end[i] = (int)R;
    if (x_row < (long long)M * D || x_image < 0) return DCN_ERR_INVALID_ARG;
    if (R > dcnb::kRopeMaxPairs || (long long)M * D > (1 << 24) || (long long)N * L > kInt31 - 1)
        return DCN_ERR_UNSUPPORTED;
    if (N == 0 || L == 0) return DCN_OK;
    const bool reads_x = !grad || grad_pos != nullptr;
    if ((reads_x && !x) || !pos || !out || (R > 0 && !freqs) || (grad && !go))
        return DCN_ERR_INVALID_ARG;
    if (((reads_x ? (uintptr_t)x : 0) | (uintptr_t)out | (uintptr_t)go) % es != 0 ||
        ((uintptr_t)pos | (uintptr_t)freqs | (uintptr_t)grad_pos) % 4 != 0)
        return DCN_ERR_MISALIGNED;
    const long long dense = (long long)N * L * M * D * es;
    const long long xb = ((N - 1) * x_image + (L - 1) * x_row + (long long)M * D) * es;
    const long long pb = (long long)pos_images * L * A * 4, fb = R * 4;
    // in place: the output may be a dense x itself
    const bool in_place = !grad && out == x && x_row == (long long)M * D &&
                          (N == 1 || x_image == (long long)L * M * D);
    if ((reads_x && !in_place && overlaps(out, dense, x, xb)) || overlaps(out, dense, pos, pb) ||
        (R > 0 && overlaps(out, dense, freqs, fb)) || (grad && overlaps(out, dense, go, dense)))
        return DCN_ERR_INVALID_ARG;
    if (grad_pos &&
        (overlaps(grad_pos, pb, x, xb) || overlaps(grad_pos, pb, pos, pb) ||
         overlaps(grad_pos, pb, go, dense) || overlaps(grad_pos, pb, out, dense) ||
         (R > 0 && overlaps(grad_pos, pb, freqs, fb))))
        return DCN_ERR_INVALID_ARG;

    // widest access that the channel spans, strides and addresses allow
    uintptr_t bits = (uintptr_t)out | (uintptr_t)go;
    if (reads_x) {
        bits |= (uintptr_t)x | (uintptr_t)(x_row * es);
        if (N > 1) bits |= (uintptr_t)(x_image * es);
    }
    const int span = interleaved ? (int)(2 * R) : (int)R;
    // (16-bit gradients of halves take 8 bytes: four 16-byte vectors a lane need 122 registers,
    // and half the warps; 47 us against 58 on 2 x 12136 tokens of 16 x 64)
    int v = grad && !interleaved ? 4 : 16 / es;
    while (v > 1 && (D % v != 0 || span % v != 0 || bits % (uintptr_t)(v * es) != 0)) v >>= 1;

    a.x = reads_x ? x : go;
    a.pos = pos;
    a.freqs = freqs;
    a.go = go;
    a.out = out;
    a.grad_pos = grad_pos;
    a.L = L;
    a.M = M;
    a.D = D;
    a.R = (int)R;
    a.A = A;
    a.x_image = x_image;
    a.x_row = x_row;
    a.shared_pos = pos_images == 1 ? 1 : 0;
    a.images = grad_pos && pos_images == 1 ? N : 1;
    a.units = a.images > 1 ? L : (long long)N * L;
    a.tasks = (interleaved && v > 1) ? D / v : (int)(R / v + (D - 2 * R) / v);
    // lanes per token: about two tasks a lane, at most a warp
    const long long total = (long long)M * a.tasks;
    int tpt = 1;
    while (tpt < 32 && 2 * tpt < total) tpt <<= 1;
    // a team writes its token's A position gradients from as many lanes
    while (tpt < A) tpt <<= 1;
    // a team's turns live in shared memory: at most 48 KB a block
    while (tpt < 32 && (dcnb::kRopeThreads / tpt) * R * 8 > kMaxStageBytes) tpt <<= 1;
    a.tpt = tpt;
    a.jl = std::min(a.tasks, tpt);
    a.hl = tpt / a.jl;
    a.div_jl = make_div((uint32_t)a.jl);
    a.div_L = make_div((uint32_t)L);
    a.sign = inverse ? -1.f : 1.f;

    const void* fn = nullptr;
    switch (dtype) {
        case DCN_F32: fn = rope_kernel_for<float>(v, interleaved != 0, grad); break;
        case DCN_F16: fn = rope_kernel_for<__half>(v, interleaved != 0, grad); break;
        case DCN_BF16: fn = rope_kernel_for<__nv_bfloat16>(v, interleaved != 0, grad); break;
        default: break;
    }
    if (!fn) return DCN_ERR_UNSUPPORTED;
    const int teams = dcnb::kRopeThreads / tpt;
    const long long blocks = (a.units + teams - 1) / teams;
    return launch_grid(fn, a, (int)blocks, dcnb::kRopeThreads, teams * (int)R * 8, stream);
}

}  // namespace

extern "C" {

int axial_rope_forward(const void* x, const float* pos, const float* freqs, void* out,
                       const int* axis_pairs, int N, int L, int M, int D, int A, int pos_images,
                       long long x_image, long long x_row, int interleaved, int inverse, int dtype,
                       void* stream) {
    return rope_launch(x, pos, freqs, nullptr, out, nullptr, axis_pairs, N, L, M, D, A, pos_images,
                       x_image, x_row, interleaved, inverse, dtype, false, stream);
}

int axial_rope_backward(const void* x, const float* pos, const float* freqs, const void* grad_out,
                        void* grad_x, float* grad_pos, const int* axis_pairs, int N, int L, int M,
                        int D, int A, int pos_images, long long x_image, long long x_row,
                        int interleaved, int inverse, int dtype, void* stream) {
    return rope_launch(x, pos, freqs, grad_out, grad_x, grad_pos, axis_pairs, N, L, M, D, A,
                       pos_images, x_image, x_row, interleaved, inverse, dtype, true, stream);
}

}  // extern "C"
