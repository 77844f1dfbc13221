// C interface of libdcn_b200.so: norm_residual_forward,
// norm_residual_backward_workspace_size, norm_residual_backward.
#include "abi_common.cuh"
#include "norm_residual.cuh"

using namespace dcnb_abi;

namespace {

constexpr int kNormBlockThreads = dcnb::kNormSmall;

struct NormShape {
    int es;
    int tpr, threads, teams;
    long long rows;
};

// Threads per row (a power of two, eight channels each) and the block's teams.
NormShape norm_shape(int es, long long rows, int C) {
    NormShape s;
    s.es = es;
    s.rows = rows;
    s.tpr = 1;
    while (s.tpr * dcnb::kNormV < C) s.tpr <<= 1;
    s.threads = std::max(s.tpr, kNormBlockThreads);
    s.teams = s.threads / s.tpr;
    return s;
}

// Blocks that share an image's rows in the gradient: over all images as many as
// a multiprocessor's registers hold, two of 256 threads or one of 512 or 1024
// (more would only add partial rows to sum), at least one team step each.
int grad_blocks_per_image(long long images, long long rows_per_image, int teams, int threads) {
    const long long wanted = (threads <= dcnb::kNormSmall ? 2LL : 1LL) * sm_count();
    long long per = wanted / images;
    per = std::min(per, (rows_per_image + teams - 1) / teams);
    return (int)std::max(per, 1LL);
}

// Rows that share a gate, and how many such groups: without a gate the whole
// batch is one.
void groups(const void* gate, int N, long long L, long long* images, long long* rows) {
    *images = gate ? N : 1;
    *rows = gate ? L : (long long)N * L;
}

int check_sizes(int es, int N, long long L, int C, int flags, float eps) {
    if (es == 0 || N < 0 || L < 0 || C <= 0 || (flags & ~7) != 0 || !(eps >= 0.f))
        return DCN_ERR_INVALID_ARG;
    if (C > dcnb::kNormMaxC || (long long)N * L > kInt31) return DCN_ERR_UNSUPPORTED;
    return DCN_OK;
}

struct Span {
    const void* p;
    long long bytes;
};

// Null spans never overlap.
bool clash(const Span& a, const Span& b) {
    return a.p && b.p && a.bytes > 0 && b.bytes > 0 && overlaps(a.p, a.bytes, b.p, b.bytes);
}

template <typename T, bool VEC>
const void* norm_kernel_threads(int threads, bool grad) {
    if (threads <= dcnb::kNormSmall)
        return grad ? (const void*)dcnb::norm_residual_grad_kernel<T, VEC, dcnb::kNormSmall>
                    : (const void*)dcnb::norm_residual_kernel<T, VEC, dcnb::kNormSmall>;
    if (threads <= dcnb::kNormMiddle)
        return grad ? (const void*)dcnb::norm_residual_grad_kernel<T, VEC, dcnb::kNormMiddle>
                    : (const void*)dcnb::norm_residual_kernel<T, VEC, dcnb::kNormMiddle>;
    return grad ? (const void*)dcnb::norm_residual_grad_kernel<T, VEC, dcnb::kNormMaxThreads>
                : (const void*)dcnb::norm_residual_kernel<T, VEC, dcnb::kNormMaxThreads>;
}

template <typename T>
const void* norm_kernel_for(bool vec, int threads, bool grad) {
    return vec ? norm_kernel_threads<T, true>(threads, grad)
               : norm_kernel_threads<T, false>(threads, grad);
}

const void* norm_kernel(int dtype, bool vec, int threads, bool grad) {
    switch (dtype) {
        case DCN_F32: return norm_kernel_for<float>(vec, threads, grad);
        case DCN_F16: return norm_kernel_for<__half>(vec, threads, grad);
        case DCN_BF16: return norm_kernel_for<__nv_bfloat16>(vec, threads, grad);
        default: return nullptr;
    }
}

const void* final_kernel(int dtype) {
    switch (dtype) {
        case DCN_F32: return (const void*)dcnb::norm_residual_final_kernel<float>;
        case DCN_F16: return (const void*)dcnb::norm_residual_final_kernel<__half>;
        case DCN_BF16: return (const void*)dcnb::norm_residual_final_kernel<__nv_bfloat16>;
        default: return nullptr;
    }
}

}  // namespace

extern "C" {

int norm_residual_forward(const void* x, const void* y, const void* scale, const void* gate,
                          const void* post_weight, const void* post_bias, const void* pre_weight,
                          const void* pre_bias, void* z, void* h, int N, long long L, int C,
                          int flags, float eps, int dtype, void* stream) {
    const int es = elem_bytes(dtype);
    const int st = check_sizes(es, N, L, C, flags, eps);
    if (st != DCN_OK) return st;
    const bool post = flags & DCN_NORM_POST, pre = flags & DCN_NORM_PRE;
    if ((!post && (post_weight || post_bias)) || (!pre && (pre_weight || pre_bias || h)))
        return DCN_ERR_INVALID_ARG;
    if (N == 0 || L == 0) return DCN_OK;
    if (!x || !y || !z || (pre && !h)) return DCN_ERR_INVALID_ARG;
    const uintptr_t bits = (uintptr_t)x | (uintptr_t)y | (uintptr_t)z | (uintptr_t)h |
                           (uintptr_t)scale | (uintptr_t)gate | (uintptr_t)post_weight |
                           (uintptr_t)post_bias | (uintptr_t)pre_weight | (uintptr_t)pre_bias;
    if (bits % es != 0) return DCN_ERR_MISALIGNED;
    const long long rows = (long long)N * L, tb = rows * C * es, cb = (long long)C * es;
    const Span ins[] = {{x, tb}, {y, tb}, {scale, cb}, {gate, cb * N}, {post_weight, cb},
                        {post_bias, cb}, {pre_weight, cb}, {pre_bias, cb}};
    for (const Span& s : ins) {
        // z may be x itself: every row is read before it is written
        if ((!(s.p == x && z == x) && clash({z, tb}, s)) || clash({h, tb}, s))
            return DCN_ERR_INVALID_ARG;
    }
    if (clash({z, tb}, {h, tb})) return DCN_ERR_INVALID_ARG;

    const NormShape s = norm_shape(es, rows, C);
    dcnb::NormArgs a = {};
    a.x = x;
    a.y = y;
    a.post_w = post_weight;
    a.post_b = post_bias;
    a.gate = gate;
    a.scale = scale;
    a.pre_w = pre_weight;
    a.pre_b = pre_bias;
    a.z = z;
    a.h = h;
    groups(gate, N, L, &a.images, &a.rows_per_image);
    a.C = C;
    a.tpr = s.tpr;
    a.rms = (flags & DCN_NORM_RMS) != 0;
    a.post = post;
    a.pre = pre;
    a.eps = eps;
    const bool vec = C % dcnb::kNormV == 0 && bits % 16 == 0;
    const void* fn = norm_kernel(dtype, vec, s.threads, false);
    const long long blocks = (rows + s.teams - 1) / s.teams;
    return launch(fn, a, (int)std::min(blocks, kInt31), s.threads, 0, stream);
}

long long norm_residual_backward_workspace_size(int N, long long L, int C, int gated, int dtype) {
    const int es = elem_bytes(dtype);
    if (gated != 0 && gated != 1) return DCN_ERR_INVALID_ARG;
    const int st = check_sizes(es, N, L, C, 0, 0.f);
    if (st != DCN_OK) return st;
    if (N == 0 || L == 0) return 0;
    const long long images = gated ? N : 1, rows = gated ? L : (long long)N * L;
    const NormShape s = norm_shape(es, (long long)N * L, C);
    return images * grad_blocks_per_image(images, rows, s.teams, s.threads) * 4LL * C * 4;
}

int norm_residual_backward(const void* y, const void* z, const void* grad_z, const void* grad_h,
                           const void* scale, const void* gate, const void* post_weight,
                           const void* post_bias, const void* pre_weight, void* grad_x,
                           void* grad_y, void* grad_scale, void* grad_gate, void* grad_post_weight,
                           void* grad_post_bias, void* grad_pre_weight, void* grad_pre_bias,
                           void* workspace, long long workspace_bytes, int N, long long L, int C,
                           int flags, float eps, int dtype, void* stream) {
    const int es = elem_bytes(dtype);
    const int st = check_sizes(es, N, L, C, flags, eps);
    if (st != DCN_OK) return st;
    const bool post = flags & DCN_NORM_POST, pre = flags & DCN_NORM_PRE;
    if ((!post && (post_weight || post_bias || grad_post_weight || grad_post_bias)) ||
        (!pre && (pre_weight || grad_h || grad_pre_weight || grad_pre_bias)) ||
        (grad_gate && !gate))
        return DCN_ERR_INVALID_ARG;
    const long long rows = (long long)N * L, tb = rows * C * es, cb = (long long)C * es;
    if (rows > 0 && (!y || !grad_z || !grad_x || !grad_y || (pre && (!z || !grad_h)) || !workspace))
        return DCN_ERR_INVALID_ARG;
    const uintptr_t row_bits = (uintptr_t)y | (uintptr_t)z | (uintptr_t)grad_z |
                               (uintptr_t)grad_h | (uintptr_t)grad_x | (uintptr_t)grad_y |
                               (uintptr_t)scale | (uintptr_t)gate | (uintptr_t)post_weight |
                               (uintptr_t)pre_weight;
    const uintptr_t bits = row_bits | (uintptr_t)post_bias | (uintptr_t)grad_scale |
                           (uintptr_t)grad_gate | (uintptr_t)grad_post_weight |
                           (uintptr_t)grad_post_bias | (uintptr_t)grad_pre_weight |
                           (uintptr_t)grad_pre_bias;
    if (bits % es != 0 || (uintptr_t)workspace % 16 != 0) return DCN_ERR_MISALIGNED;
    const long long need = norm_residual_backward_workspace_size(N, L, C, gate ? 1 : 0, dtype);
    if (workspace_bytes < need) return DCN_ERR_INVALID_ARG;
    const Span ins[] = {{y, tb}, {pre ? z : nullptr, tb}, {grad_z, tb}, {grad_h, tb}, {scale, cb},
                        {gate, cb * N}, {post_weight, cb}, {post_bias, cb}, {pre_weight, cb}};
    const Span outs[] = {{grad_x, tb}, {grad_y, tb}, {grad_scale, cb}, {grad_gate, cb * N},
                         {grad_post_weight, cb}, {grad_post_bias, cb}, {grad_pre_weight, cb},
                         {grad_pre_bias, cb}, {workspace, need}};
    const int n_out = (int)(sizeof(outs) / sizeof(outs[0]));
    for (int i = 0; i < n_out; ++i) {
        for (const Span& s : ins)
            if (clash(outs[i], s)) return DCN_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (clash(outs[i], outs[j])) return DCN_ERR_INVALID_ARG;
    }

    dcnb::NormFinalArgs f = {};
    if (rows > 0) {
        const NormShape s = norm_shape(es, rows, C);
        dcnb::NormArgs a = {};
        a.y = y;
        a.post_w = post_weight;
        a.gate = gate;
        a.scale = scale;
        a.pre_w = pre_weight;
        a.z = const_cast<void*>(z);
        a.gz = grad_z;
        a.gh = grad_h;
        a.gx = grad_x;
        a.gy = grad_y;
        a.partial = static_cast<float*>(workspace);
        groups(gate, N, L, &a.images, &a.rows_per_image);
        a.blocks_per_image =
            grad_blocks_per_image(a.images, a.rows_per_image, s.teams, s.threads);
        a.C = C;
        a.tpr = s.tpr;
        a.rms = (flags & DCN_NORM_RMS) != 0;
        a.post = post;
        a.pre = pre;
        a.eps = eps;
        const bool vec = C % dcnb::kNormV == 0 && row_bits % 16 == 0;
        const void* fn = norm_kernel(dtype, vec, s.threads, true);
        const int smem = (s.teams - 1) * s.tpr * dcnb::kNormV * 4;
        const int rc = launch_grid(fn, a, (int)(a.images * a.blocks_per_image), s.threads, smem,
                                   stream);
        if (rc != DCN_OK) return rc;
        f.images = a.images;
        f.blocks_per_image = a.blocks_per_image;
    }
    if (rows == 0) {       // an empty batch's factor gradients are zero: no partials to add
        f.images = gate ? N : 1;
        f.blocks_per_image = 0;
    }
    f.partial = static_cast<const float*>(workspace);
    f.scale = scale;
    f.gate = gate;
    f.post_w = post_weight;
    f.post_b = post_bias;
    f.gscale = grad_scale;
    f.ggate = grad_gate;
    f.gpost_w = grad_post_weight;
    f.gpost_b = grad_post_bias;
    f.gpre_w = grad_pre_weight;
    f.gpre_b = grad_pre_bias;
    f.C = C;
    f.segments = 1;
    while (f.segments < 32 && f.segments * 2 * f.images <= 32) f.segments <<= 1;
    if (!(grad_scale || grad_gate || grad_post_weight || grad_post_bias || grad_pre_weight ||
          grad_pre_bias))
        return DCN_OK;
    return launch_grid(final_kernel(dtype), f, (C + dcnb::kNormFinalCols - 1) / dcnb::kNormFinalCols,
                       dcnb::kNormFinalCols * dcnb::kNormFinalRows, 0, stream);
}

}  // extern "C"
