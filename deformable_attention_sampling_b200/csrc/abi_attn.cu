// C interface of libdcn_b200.so: diff_attn_forward, diff_attn_backward and
// their workspace sizes.
#include "abi_common.cuh"
#include "diff_attn.cuh"
#include "diff_attn_mma.cuh"
#include "diff_attn_mma_bwd.cuh"
#include "diff_attn_step.cuh"

using namespace dcnb_abi;

namespace {

struct AttnPlan {
    int bq;            // packed rows of a tile
    int tiles;         // row tiles of a key / value head
    int splits;        // key ranges a tile is split into
};

// Row tile and key splits.  Few rows (a serving step) take the 16-row tile;
// the keys are split when the tiles alone leave most multiprocessors idle, so
// that about two blocks a multiprocessor run, each with at least two key
// tiles (a shorter range costs more in its join than it saves).
AttnPlan attn_plan(int N, int Lq, int Lk, int M, int Mk) {
    AttnPlan p;
    const long long rows = (long long)Lq * (M / Mk);
    p.bq = rows <= 16 ? 16 : 64;
    p.tiles = (int)((rows + p.bq - 1) / p.bq);
    const long long blocks = (long long)p.tiles * N * Mk;
    const int sms = sm_count();
    const int key_tiles = (Lk + dcnb::kAttnKeys - 1) / dcnb::kAttnKeys;
    long long s = blocks < sms ? (2LL * sms + blocks - 1) / std::max(blocks, 1LL) : 1;
    s = std::min(s, (long long)key_tiles / 2);
    p.splits = (int)std::max(1LL, std::min(s, (long long)dcnb::kAttnMaxSplits));
    return p;
}

template <typename T, int BQ>
const void* fwd_kernel_ct(int ct) {
    switch (ct) {
        case 2: return (const void*)dcnb::diff_attn_kernel<T, BQ, 2>;
        case 4: return (const void*)dcnb::diff_attn_kernel<T, BQ, 4>;
        case 8: return (const void*)dcnb::diff_attn_kernel<T, BQ, 8>;
        case 16: return (const void*)dcnb::diff_attn_kernel<T, BQ, 16>;
        default: return nullptr;
    }
}

template <typename T>
const void* fwd_kernel(int bq, int ct) {
    return bq == 16 ? fwd_kernel_ct<T, 16>(ct) : fwd_kernel_ct<T, 64>(ct);
}

// Columns a thread of 16 owns of a head size: 2, 4, 8 or 16.
int columns(int d) {
    int c = 2;
    while (16 * c < d) c <<= 1;
    return c;
}

// The gradient kernels' tile: 64 where shared memory holds it (heads up to 64
// and values up to 128 channels), else 32.
int bwd_tile(int cd, int ct) { return cd <= 4 && ct <= 8 ? 64 : 32; }

template <typename T, int BT, int CD>
void bwd_kernels_ct(int ct, const void** dq, const void** dkv) {
    switch (ct) {
        case 2:
            *dq = (const void*)dcnb::diff_attn_dq_kernel<T, BT, CD, 2>;
            *dkv = (const void*)dcnb::diff_attn_dkv_kernel<T, BT, CD, 2>;
            break;
        case 4:
            *dq = (const void*)dcnb::diff_attn_dq_kernel<T, BT, CD, 4>;
            *dkv = (const void*)dcnb::diff_attn_dkv_kernel<T, BT, CD, 4>;
            break;
        case 8:
            *dq = (const void*)dcnb::diff_attn_dq_kernel<T, BT, CD, 8>;
            *dkv = (const void*)dcnb::diff_attn_dkv_kernel<T, BT, CD, 8>;
            break;
        case 16:
            if constexpr (BT == 32) {
                *dq = (const void*)dcnb::diff_attn_dq_kernel<T, BT, CD, 16>;
                *dkv = (const void*)dcnb::diff_attn_dkv_kernel<T, BT, CD, 16>;
            }
            break;
        default: break;
    }
}

template <typename T>
void bwd_kernels(int cd, int ct, const void** dq, const void** dkv) {
    const bool big = bwd_tile(cd, ct) == 64;
    switch (cd) {
        case 2:
            if (big) bwd_kernels_ct<T, 64, 2>(ct, dq, dkv);
            else bwd_kernels_ct<T, 32, 2>(16, dq, dkv);
            break;
        case 4:
            if (big) bwd_kernels_ct<T, 64, 4>(ct, dq, dkv);
            else bwd_kernels_ct<T, 32, 4>(16, dq, dkv);
            break;
        case 8: bwd_kernels_ct<T, 32, 8>(ct, dq, dkv); break;
        default: break;
    }
}

// Checks shared by both directions; fills the geometry.  `strides`: image and
// row strides of q, k, v.
int attn_setup(dcnb::AttnArgs* a, const void* q, const void* k, const void* v, const void* lam,
               const unsigned char* mask, const int* lengths, int N, int Lq, int Lk, int M, int Mk,
               int D, int Dv, long long q_image, long long q_row, long long k_image,
               long long k_row, long long v_image, long long v_row, float scale, int causal,
               int dtype) {
    const int es = elem_bytes(dtype);
    if (es == 0 || N < 0 || Lq < 0 || Lk < 0 || M <= 0 || Mk <= 0 || M % Mk != 0 || D <= 0 ||
        Dv <= 0 || (causal != 0 && causal != 1) || !std::isfinite(scale) || q_image < 0 ||
        k_image < 0 || v_image < 0)
        return DCN_ERR_INVALID_ARG;
    if (D > dcnb::kAttnMaxD || Dv > dcnb::kAttnMaxDv || (long long)N * M > 65535 ||
        (long long)Lq * (M / Mk) > kInt31 - 65536 || (long long)Lq + Lk > kInt31 - 65536)
        return DCN_ERR_UNSUPPORTED;
    if (q_row < (long long)M * 2 * D || k_row < (long long)Mk * 2 * D ||
        v_row < (long long)Mk * Dv)
        return DCN_ERR_INVALID_ARG;
    a->q = q;
    a->k = k;
    a->v = v;
    a->lam = lam;
    a->mask = mask;
    a->lengths = lengths;
    a->N = N;
    a->Lq = Lq;
    a->Lk = Lk;
    a->M = M;
    a->Mk = Mk;
    a->G = M / Mk;
    a->D = D;
    a->Dv = Dv;
    a->rows = Lq * a->G;
    a->splits = 1;
    a->causal = causal;
    a->scale = scale;
    a->scale_log2 = (float)((double)scale * 1.4426950408889634074);
    a->q_image = q_image;
    a->q_row = q_row;
    a->k_image = k_image;
    a->k_row = k_row;
    a->v_image = v_image;
    a->v_row = v_row;
    a->div_G = make_div((uint32_t)a->G);
    a->div_Mk = make_div((uint32_t)Mk);
    const uintptr_t bits = (uintptr_t)q | (uintptr_t)k | (uintptr_t)v;
    const long long strides = q_image | q_row | k_image | k_row | v_image | v_row;
    a->vec4 = D % 4 == 0 && Dv % 4 == 0 && strides % 4 == 0 && bits % (uintptr_t)(4 * es) == 0;
    return DCN_OK;
}

// Pointers of a non-empty call: present, aligned.
int attn_pointers(const dcnb::AttnArgs& a, int es) {
    if (!a.q || !a.lam || (a.Lk > 0 && (!a.k || !a.v))) return DCN_ERR_INVALID_ARG;
    if (((uintptr_t)a.q | (uintptr_t)a.k | (uintptr_t)a.v | (uintptr_t)a.lam) % es != 0 ||
        (uintptr_t)a.lengths % 4 != 0)
        return DCN_ERR_MISALIGNED;
    return DCN_OK;
}

struct Span {
    const void* p;
    long long bytes;
};

bool clash(const Span& a, const Span& b) {
    return a.p && b.p && a.bytes > 0 && b.bytes > 0 && overlaps(a.p, a.bytes, b.p, b.bytes);
}

long long strided_bytes(int N, long long image, int L, long long row, long long inner, int es) {
    return N > 0 && L > 0 ? ((N - 1) * image + (L - 1) * row + inner) * es : 0;
}

constexpr int kInputs = 6;

void input_spans(const dcnb::AttnArgs& a, int es, Span* s) {
    s[0] = {a.q, strided_bytes(a.N, a.q_image, a.Lq, a.q_row, 2LL * a.M * a.D, es)};
    s[1] = {a.k, strided_bytes(a.N, a.k_image, a.Lk, a.k_row, 2LL * a.Mk * a.D, es)};
    s[2] = {a.v, strided_bytes(a.N, a.v_image, a.Lk, a.v_row, (long long)a.Mk * a.Dv, es)};
    s[3] = {a.lam, (long long)a.M * es};
    s[4] = {a.mask, (long long)a.N * a.Lk};
    s[5] = {a.lengths, 4LL * a.N};
}

bool any_clash(const Span* outs, int n_out, const Span* ins, int n_in) {
    for (int i = 0; i < n_out; ++i) {
        for (int j = 0; j < n_in; ++j)
            if (clash(outs[i], ins[j])) return true;
        for (int j = 0; j < i; ++j)
            if (clash(outs[i], outs[j])) return true;
    }
    return false;
}

// A grid whose x counts row or key tiles, y the (image, head) pairs and z the
// splits.
template <typename Args>
int launch_attn(const void* fn, const Args& a, dim3 grid, int threads, int smem, void* stream) {
    if (wave_size(fn, threads, smem) <= 0) {
        g_last_cuda_error = (int)cudaGetLastError();
        return DCN_ERR_CUDA;
    }
    void* params[] = {const_cast<Args*>(&a)};
    const cudaError_t err =
        cudaLaunchKernel(fn, grid, dim3(threads), params, (size_t)smem, (cudaStream_t)stream);
    if (err != cudaSuccess) {
        g_last_cuda_error = (int)err;
        (void)cudaGetLastError();
        return DCN_ERR_CUDA;
    }
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return DCN_OK;
}

// The tensor-core kernels take 16-bit data whose rows are 16-byte vectors at
// 16-byte aligned places (what tensor maps can address).
bool mma_sizes(int dtype, int D, int Dv) {
    return dtype != DCN_F32 && D % 8 == 0 && Dv % 8 == 0;
}

bool mma_layout(const dcnb::AttnArgs& a) {
    const uintptr_t bits = (uintptr_t)a.q | (uintptr_t)a.k | (uintptr_t)a.v;
    const long long strides = a.q_image | a.q_row | a.k_image | a.k_row | a.v_image | a.v_row;
    const long long limit = 1LL << 38;       // elements: a tensor map's strides end at 2^40 bytes
    // one image has no use for its stride; 0 (a broadcast image) is no tensor-map stride
    return bits % 16 == 0 && strides % 8 == 0 && a.Lk > 0 && a.q_row < limit && a.k_row < limit &&
           a.v_row < limit && a.q_image < limit && a.k_image < limit && a.v_image < limit &&
           (a.N == 1 || (a.q_image > 0 && a.k_image > 0 && a.v_image > 0));
}

// Tensor map of [N][L][heads][inner] rows, box 64 elements x 1 head x rows tokens.
bool head_map(CUtensorMap* map, const void* p, int dtype, int inner, int heads, int L, int N,
              long long row, long long image, int rows) {
    const uint64_t dims[4] = {(uint64_t)inner, (uint64_t)heads, (uint64_t)L, (uint64_t)N};
    const uint64_t strides[3] = {(uint64_t)inner * 2, (uint64_t)row * 2,
                                 (uint64_t)(N == 1 ? row : image) * 2};   // (of one image: unused)
    const uint32_t box[4] = {64, 1, (uint32_t)rows, 1};
    return encode_tmap_4d(map, p, dtype == DCN_BF16, dims, strides, box);
}

int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Key splits of the tensor-core forward: one CTA a multiprocessor runs, so the
// keys are split when the tiles leave half of them idle or more, at least two
// key tiles each.  Measured in bf16 (split / not, us): 300 tokens of 2 images, 4 heads
// of 32 + 64, over 300 keys 16.0 / 10.3, 512 16.4 / 12.4, 1024 18.9 / 19.3, 4096
// 25.5 / 65.8; 128 tokens of 8 heads of 64 + 128 over 300 keys 16.5 / 11.0, 1024
// 17.5 / 19.8, 4096 22.2 / 62.5.  The join costs more than a split saves below about
// 1000 keys.
int mma_splits(int N, int Lq, int Lk, int M, int Dv) {
    const long long ctas = (long long)ceil_div(Lq, dcnb::kAmRows) * N * M *
                           ceil_div(Dv, dcnb::kAmMaxDv);
    long long s = sm_count() / std::max(ctas, 1LL);
    s = std::min(s, (long long)ceil_div(Lk, dcnb::kAmKeys) / 2);
    return (int)std::max(1LL, std::min(s, (long long)dcnb::kAttnMaxSplits));
}

// The few-token kernel's head and value sizes (D a multiple of 32, so that a
// lane's quarter is a 16-byte vector; Dv of 32 or more).
bool step_sizes(int dtype, int D, int Dv) {
    return dtype != DCN_F32 && (D == 32 || D == 64 || D == 128) &&
           (Dv == 32 || Dv == 64 || Dv == 128);
}

// Key splits of the few-token kernel: 3 CTAs of 4 warps a multiprocessor run, and
// three full rounds of them even out images of different lengths (a fourth,
// nearly empty one would not); a split has at least 256 keys.
int step_splits(int N, int Lq, int Lk, int M, int Mk) {
    const long long ctas = (long long)ceil_div(Lq * (M / Mk), dcnb::kAsRows) * N * Mk;
    long long s = 9LL * sm_count() / std::max(ctas, 1LL);
    s = std::min(s, (long long)ceil_div(Lk, 256));
    return (int)std::max(1LL, std::min(s, (long long)dcnb::kAttnMaxSplits));
}

template <typename T, int D>
const void* step_kernel_dv(int Dv) {
    switch (Dv) {
        case 32: return (const void*)dcnb::diff_attn_step_kernel<T, D, 32>;
        case 64: return (const void*)dcnb::diff_attn_step_kernel<T, D, 64>;
        case 128: return (const void*)dcnb::diff_attn_step_kernel<T, D, 128>;
        default: return nullptr;
    }
}

template <typename T>
const void* step_kernel(int D, int Dv) {
    switch (D) {
        case 32: return step_kernel_dv<T, 32>(Dv);
        case 64: return step_kernel_dv<T, 64>(Dv);
        case 128: return step_kernel_dv<T, 128>(Dv);
        default: return nullptr;
    }
}

// Tokens from which the 128-row tiles of the tensor-core kernels are taken.
// Measured in bf16, heads of 64 + 128 (tensor-core / few-token kernel, us): one image,
// 16 heads of 4 key / value heads, 4096 keys: 8 tokens 18.7 / 16.0, 16 tokens 18.8 /
// 24.6, 17 tokens 19.0 / 27.8, 64 tokens 20.8 / 59.0; over 300 keys the other way
// round, 17 tokens 12.4 / 8.7, 64 tokens 14.2 / 12.0.  16 images of 8 + 8 heads, 4096
// keys: 8 tokens 70 / 69, 16 tokens 70 / 103, 17 tokens 70 / 153.  The gradients take
// the same number, but there the other form is the CUDA cores': at 16 tokens 28 / 142
// over 300 keys, 92 / 1314 over 4096.
constexpr int kMmaMinTokens = 17;

// The gradient kernels' tensor-core form: heads and values that its TMEM holds.
bool mma_bwd_sizes(int dtype, int Lq, int Lk, int D, int Dv) {
    return mma_sizes(dtype, D, Dv) && D <= dcnb::kAbMaxD && Dv <= dcnb::kAbMaxDv &&
           Lq >= kMmaMinTokens && Lk > 0;
}

long long rowv_floats(int N, int Lq, int M) {
    return (long long)N * M * ceil_div(Lq, dcnb::kRowvTile) * 4 * dcnb::kRowvTile;
}

// Row values (and fp16's scales) are set; `glam` sums grad_lambda from the row
// values between the two kernels: the first one refines them.
int mma_backward(const dcnb::AttnArgs& a, const void* glam, const dcnb::AttnDeltaArgs& d,
                 int dtype, void* stream) {
    dcnb::AttnBwdArgs f;
    f.rowv = d.rowv;
    f.a = a;
    f.negate = a.scale < 0.f ? 1 : 0;
    f.a.scale_log2 = std::max(std::fabs(a.scale_log2), 1e-30f);
    f.scales = d.scales;
    f.gnorm = d.gnorm;
    f.flags = device_flags_word();
    f.dsteps = ceil_div(a.D, 16);
    f.vsteps = ceil_div(a.Dv, 16);
    const int vch = ceil_div(a.Dv, 64);
    const bool bf16 = dtype == DCN_BF16;
    const long long g_row = (long long)a.M * a.Dv;
    // query tiles of 128 tokens over key tiles of 64, then the other way round
    for (int pass = 0; pass < 2; ++pass) {
        const int qb = pass == 0 ? dcnb::kAmRows : dcnb::kAmKeys;
        const int kb = pass == 0 ? dcnb::kAmKeys : dcnb::kAmRows;
        if (!head_map(&f.tq, a.q, dtype, a.D, 2 * a.M, a.Lq, a.N, a.q_row, a.q_image, qb) ||
            !head_map(&f.tg, a.go, dtype, a.Dv, a.M, a.Lq, a.N, g_row, g_row * a.Lq, qb) ||
            !head_map(&f.tk, a.k, dtype, a.D, 2 * a.Mk, a.Lk, a.N, a.k_row, a.k_image, kb) ||
            !head_map(&f.tv, a.v, dtype, a.Dv, a.Mk, a.Lk, a.N, a.v_row, a.v_image, kb))
            return DCN_ERR_UNSUPPORTED;
        f.heads = a.N * (pass == 0 ? a.M : a.Mk);
        const long long blocks =
            (long long)ceil_div(pass == 0 ? a.Lq : a.Lk, dcnb::kAmRows) * f.heads;
        if (blocks > kInt31) return DCN_ERR_UNSUPPORTED;
        const void* fn;
        int smem;
        if (pass == 0) {
            f.stages = 4;
            smem = dcnb::attn_dq_smem(vch, f.stages);
            fn = bf16 ? (const void*)dcnb::diff_attn_dq_mma_kernel<__nv_bfloat16>
                      : (const void*)dcnb::diff_attn_dq_mma_kernel<__half>;
        } else {
            f.stages = 3;
            smem = dcnb::attn_dkv_smem(vch, f.stages);
            fn = bf16 ? (const void*)dcnb::diff_attn_dkv_mma_kernel<__nv_bfloat16>
                      : (const void*)dcnb::diff_attn_dkv_mma_kernel<__half>;
        }
        int rc = launch_attn(fn, f, dim3((unsigned)blocks), dcnb::kAbThreads, smem, stream);
        if (rc == DCN_OK && pass == 0) rc = launch_grid(glam, d, a.M, 1024, 0, stream);
        if (rc != DCN_OK) return rc;
    }
    return DCN_OK;
}

template <typename T>
const void* mma_kernel(int dchunks) {
    return dchunks == 1 ? (const void*)dcnb::diff_attn_mma_kernel<T, 1>
                        : (const void*)dcnb::diff_attn_mma_kernel<T, 2>;
}

int mma_forward(const dcnb::AttnArgs& a, int dtype, void* stream) {
    dcnb::AttnMmaArgs f;
    f.a = a;
    f.negate = a.scale < 0.f ? 1 : 0;
    // the kernel takes a positive scale (a negative one turns the product's sign);
    // 0 becomes one that leaves every score 0 to float32 and -inf hidden
    f.a.scale_log2 = std::max(std::fabs(a.scale_log2), 1e-30f);
    const int dchunks = ceil_div(a.D, 64);
    f.dsteps = ceil_div(a.D, 16);
    f.dv_parts = ceil_div(a.Dv, dcnb::kAmMaxDv);
    const int vchunks = ceil_div(std::min(a.Dv, dcnb::kAmMaxDv), 64);
    f.heads = a.N * a.M;
    f.stages = 4;
    while (f.stages > 2 && dcnb::attn_mma_smem(dchunks, vchunks, f.stages) > 227 * 1024)
        --f.stages;
    f.flags = device_flags_word();
    if (!head_map(&f.tq, a.q, dtype, a.D, 2 * a.M, a.Lq, a.N, a.q_row, a.q_image, dcnb::kAmRows) ||
        !head_map(&f.tk, a.k, dtype, a.D, 2 * a.Mk, a.Lk, a.N, a.k_row, a.k_image,
                  dcnb::kAmKeys) ||
        !head_map(&f.tv, a.v, dtype, a.Dv, a.Mk, a.Lk, a.N, a.v_row, a.v_image, dcnb::kAmKeys))
        return DCN_ERR_UNSUPPORTED;
    const void* fn = dtype == DCN_BF16 ? mma_kernel<__nv_bfloat16>(dchunks)
                                       : mma_kernel<__half>(dchunks);
    const long long blocks = (long long)ceil_div(a.Lq, dcnb::kAmRows) * f.heads;
    if (blocks > kInt31) return DCN_ERR_UNSUPPORTED;
    return launch_attn(fn, f, dim3((unsigned)blocks, a.splits * f.dv_parts), dcnb::kAmThreads,
                       dcnb::attn_mma_smem(dchunks, vchunks, f.stages), stream);
}

template <typename T>
const void* join_kernel() { return (const void*)dcnb::diff_attn_join_kernel<T>; }

}  // namespace

extern "C" {

long long diff_attn_forward_workspace_size(int N, int Lq, int Lk, int M, int Mk, int D, int Dv,
                                           int dtype) {
    dcnb::AttnArgs a = {};
    const long long qd = 2LL * M * D, kd = 2LL * Mk * D, vd = (long long)Mk * Dv;
    const int st = attn_setup(&a, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, N, Lq, Lk,
                              M, Mk, D, Dv, 0, qd, 0, kd, 0, vd, 1.f, 0, dtype);
    if (st != DCN_OK) return st;
    if (N == 0 || Lq == 0) return 0;
    // which kernel runs depends on the addresses too: enough for either
    int splits = attn_plan(N, Lq, Lk, M, Mk).splits;
    if (mma_sizes(dtype, D, Dv) && Lq >= kMmaMinTokens)
        splits = std::max(splits, mma_splits(N, Lq, Lk, M, Dv));
    if (step_sizes(dtype, D, Dv) && Lq < kMmaMinTokens)
        splits = std::max(splits, step_splits(N, Lq, Lk, M, Mk));
    if (splits == 1) return 0;
    return (long long)splits * N * M * Lq * 2 * (2 + (long long)Dv) * 4;
}

int diff_attn_forward(const void* q, const void* k, const void* v, const void* lambda,
                      const unsigned char* mask, const int* lengths, void* out, float* maps,
                      float* lse, void* workspace, long long workspace_bytes, int N, int Lq, int Lk,
                      int M, int Mk, int D, int Dv, long long q_image, long long q_row,
                      long long k_image, long long k_row, long long v_image, long long v_row,
                      float scale, int causal, int dtype, void* stream) {
    dcnb::AttnArgs a = {};
    int rc = attn_setup(&a, q, k, v, lambda, mask, lengths, N, Lq, Lk, M, Mk, D, Dv, q_image, q_row,
                        k_image, k_row, v_image, v_row, scale, causal, dtype);
    if (rc != DCN_OK) return rc;
    if (N == 0 || Lq == 0) return DCN_OK;
    const int es = elem_bytes(dtype);
    if ((rc = attn_pointers(a, es)) != DCN_OK) return rc;
    if (!out || (maps == nullptr) != (lse == nullptr)) return DCN_ERR_INVALID_ARG;
    if ((uintptr_t)out % es != 0 || ((uintptr_t)maps | (uintptr_t)lse) % 4 != 0 ||
        (uintptr_t)workspace % 16 != 0)
        return DCN_ERR_MISALIGNED;
    const AttnPlan p = attn_plan(N, Lq, Lk, M, Mk);
    const bool mma = mma_sizes(dtype, D, Dv) && Lq >= kMmaMinTokens && mma_layout(a) &&
                     ((uintptr_t)out | (uintptr_t)maps) % 16 == 0;
    const bool step = step_sizes(dtype, D, Dv) && Lq < kMmaMinTokens && mma_layout(a);
    const long long need = diff_attn_forward_workspace_size(N, Lq, Lk, M, Mk, D, Dv, dtype);
    if (need > 0 && (!workspace || workspace_bytes < need)) return DCN_ERR_INVALID_ARG;
    const long long ob = (long long)N * Lq * M * Dv * es;
    Span ins[kInputs];
    input_spans(a, es, ins);
    const Span outs[] = {{out, ob}, {maps, ob / es * 8}, {lse, (long long)N * M * 2 * Lq * 4},
                         {workspace, need}};
    if (any_clash(outs, 4, ins, kInputs)) return DCN_ERR_INVALID_ARG;
    a.out = out;
    a.maps = maps;
    a.lse = lse;
    a.splits = mma    ? mma_splits(N, Lq, Lk, M, Dv)
               : step ? step_splits(N, Lq, Lk, M, Mk)
                      : p.splits;
    const long long rows_total = (long long)N * M * Lq;
    if (a.splits > 1) {
        a.part_o = static_cast<float*>(workspace);
        a.part_ml = a.part_o + (long long)a.splits * rows_total * 2 * Dv;
    }
    const int ct = columns(Dv);
    const void* fn = nullptr;
    const void* join = nullptr;
    switch (dtype) {
        case DCN_F32: fn = fwd_kernel<float>(p.bq, ct); join = join_kernel<float>(); break;
        case DCN_F16: fn = fwd_kernel<__half>(p.bq, ct); join = join_kernel<__half>(); break;
        case DCN_BF16:
            fn = fwd_kernel<__nv_bfloat16>(p.bq, ct);
            join = join_kernel<__nv_bfloat16>();
            break;
        default: break;
    }
    if (!fn) return DCN_ERR_UNSUPPORTED;
    if (step) {
        fn = dtype == DCN_BF16 ? step_kernel<__nv_bfloat16>(D, Dv) : step_kernel<__half>(D, Dv);
        rc = launch_attn(fn, a, dim3(ceil_div(a.rows, dcnb::kAsRows), N * Mk, a.splits),
                         dcnb::kAsThreads, dcnb::attn_step_smem(D, Dv), stream);
    } else if (mma) {
        rc = mma_forward(a, dtype, stream);
    } else {
        rc = launch_attn(fn, a, dim3(p.tiles, N * Mk, a.splits), dcnb::kAttnThreads,
                         dcnb::attn_fwd_smem(p.bq, D, ct), stream);
    }
    if (rc != DCN_OK || a.splits == 1) return rc;
    return launch_attn(join, a, dim3((unsigned)rows_total), dcnb::kJoinThreads, 0, stream);
}

long long diff_attn_backward_workspace_size(int N, int Lq, int Lk, int M, int Mk, int D, int Dv,
                                            int dtype) {
    dcnb::AttnArgs a = {};
    const long long qd = 2LL * M * D, kd = 2LL * Mk * D, vd = (long long)Mk * Dv;
    const int st = attn_setup(&a, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, N, Lq, Lk,
                              M, Mk, D, Dv, 0, qd, 0, kd, 0, vd, 1.f, 0, dtype);
    if (st != DCN_OK) return st;
    // row values; of the scaled fp16 kernels the scales (16 bytes each), the rows' |g|^2 (one
    // where the row values have four) and the keys' |v|^2
    long long floats = rowv_floats(N, Lq, M);
    if (dtype == DCN_F16 && mma_bwd_sizes(dtype, Lq, Lk, D, Dv))
        floats += 4LL * N * Mk + rowv_floats(N, Lq, M) / 4 + (long long)N * Lk * Mk;
    return floats * 4;
}

int diff_attn_backward(const void* q, const void* k, const void* v, const void* lambda,
                       const unsigned char* mask, const int* lengths, const float* maps,
                       const float* lse, const void* grad_out, void* grad_q,
                       void* grad_k, void* grad_v, void* grad_lambda, void* workspace,
                       long long workspace_bytes, int N, int Lq, int Lk, int M, int Mk, int D,
                       int Dv, long long q_image, long long q_row, long long k_image,
                       long long k_row, long long v_image, long long v_row, float scale, int causal,
                       int dtype, void* stream) {
    dcnb::AttnArgs a = {};
    int rc = attn_setup(&a, q, k, v, lambda, mask, lengths, N, Lq, Lk, M, Mk, D, Dv, q_image, q_row,
                        k_image, k_row, v_image, v_row, scale, causal, dtype);
    if (rc != DCN_OK) return rc;
    const int es = elem_bytes(dtype);
    const long long tokens = (long long)N * Lq, keys = (long long)N * Lk;
    if (!grad_lambda) return DCN_ERR_INVALID_ARG;
    if (tokens > 0) {
        if ((rc = attn_pointers(a, es)) != DCN_OK) return rc;
        if (!maps || !lse || !grad_out || !grad_q || !workspace) return DCN_ERR_INVALID_ARG;
    }
    // the key kernel reads k and v whether or not there are tokens
    if (keys > 0 && (!k || !v || !grad_k || !grad_v)) return DCN_ERR_INVALID_ARG;
    if (((uintptr_t)k | (uintptr_t)v | (uintptr_t)grad_out | (uintptr_t)grad_q |
         (uintptr_t)grad_k | (uintptr_t)grad_v | (uintptr_t)grad_lambda) % es != 0 ||
        ((uintptr_t)lse | (uintptr_t)maps | (uintptr_t)lengths) % 4 != 0 || (uintptr_t)workspace % 16 != 0)
        return DCN_ERR_MISALIGNED;
    const long long need = diff_attn_backward_workspace_size(N, Lq, Lk, M, Mk, D, Dv, dtype);
    if (workspace_bytes < need) return DCN_ERR_INVALID_ARG;
    const long long ob = tokens * M * Dv * es, sb = tokens * M * 2 * 4;
    Span ins[kInputs + 3];
    input_spans(a, es, ins);
    ins[kInputs] = {maps, ob / es * 8};
    ins[kInputs + 1] = {lse, sb};
    ins[kInputs + 2] = {grad_out, ob};
    const Span outs[] = {{grad_q, tokens * M * 2 * D * es}, {grad_k, keys * Mk * 2 * D * es},
                         {grad_v, keys * Mk * Dv * es}, {grad_lambda, (long long)M * es},
                         {workspace, need}};
    if (any_clash(outs, 5, ins, kInputs + 3)) return DCN_ERR_INVALID_ARG;
    a.vec4 = a.vec4 && (uintptr_t)grad_out % (uintptr_t)(4 * es) == 0;
    a.go = grad_out;
    a.lse = const_cast<float*>(lse);
    a.rowv = static_cast<const float*>(workspace);
    a.gq = grad_q;
    a.gk = grad_k;
    a.gv = grad_v;

    const int cd = columns(D), ct = columns(Dv), bt = bwd_tile(cd, ct);
    const void *dq = nullptr, *dkv = nullptr, *delta = nullptr, *glam = nullptr;
    switch (dtype) {
        case DCN_F32:
            bwd_kernels<float>(cd, ct, &dq, &dkv);
            delta = (const void*)dcnb::diff_attn_delta_kernel<float>;
            glam = (const void*)dcnb::diff_attn_glam_kernel<float>;
            break;
        case DCN_F16:
            bwd_kernels<__half>(cd, ct, &dq, &dkv);
            delta = (const void*)dcnb::diff_attn_delta_kernel<__half>;
            glam = (const void*)dcnb::diff_attn_glam_kernel<__half>;
            break;
        case DCN_BF16:
            bwd_kernels<__nv_bfloat16>(cd, ct, &dq, &dkv);
            delta = (const void*)dcnb::diff_attn_delta_kernel<__nv_bfloat16>;
            glam = (const void*)dcnb::diff_attn_glam_kernel<__nv_bfloat16>;
            break;
        default: break;
    }
    if (!dq || !dkv) return DCN_ERR_UNSUPPORTED;
    const bool mma = mma_bwd_sizes(dtype, Lq, Lk, D, Dv) && tokens > 0 && mma_layout(a) &&
                     ((uintptr_t)grad_out | (uintptr_t)grad_q | (uintptr_t)grad_k |
                      (uintptr_t)grad_v) % 16 == 0;
    float* const ws = static_cast<float*>(workspace);
    dcnb::AttnDeltaArgs d = {};
    d.a = a;
    d.maps = maps;
    d.go = grad_out;
    d.lam = lambda;
    d.lse = lse;
    d.rowv = ws;
    d.glam = grad_lambda;
    d.vec4 = Dv % 4 == 0 && (uintptr_t)maps % 16 == 0 &&
             (uintptr_t)grad_out % (uintptr_t)(4 * es) == 0;
    const long long g_blocks = rowv_floats(N, Lq, M) / (4 * 8);
    const long long v_blocks = mma && dtype == DCN_F16 ? (keys * Mk + 7) / 8 : 0;
    if (g_blocks + v_blocks > kInt31) return DCN_ERR_UNSUPPORTED;
    d.g_blocks = (int)g_blocks;
    d.v_blocks = (int)v_blocks;
    if (v_blocks > 0) {
        d.scales = reinterpret_cast<float4*>(ws + rowv_floats(N, Lq, M));
        d.gnorm = ws + rowv_floats(N, Lq, M) + 4LL * N * Mk;
        d.vnorm = d.gnorm + rowv_floats(N, Lq, M) / 4;
    }
    if (tokens > 0) {
        rc = launch_grid(delta, d, (int)(g_blocks + v_blocks), 256, 0, stream);
        if (rc != DCN_OK) return rc;
    }
    if (mma) {
        if (d.scales) {
            rc = launch_grid((const void*)dcnb::diff_attn_scales_kernel<__half>, d, N * Mk, 1024, 0,
                             stream);
            if (rc != DCN_OK) return rc;
        }
        return mma_backward(a, glam, d, dtype, stream);
    }
    rc = launch_grid(glam, d, M, 1024, 0, stream);       // zeros for an empty batch
    if (rc != DCN_OK) return rc;
    const int use_ct = bt == 32 && cd <= 4 ? 16 : ct;
    const int smem = dcnb::attn_bwd_smem(bt, cd, use_ct);
    if (tokens > 0) {
        rc = launch_attn(dq, a, dim3((a.rows + bt - 1) / bt, N * Mk), dcnb::kAttnThreads, smem,
                         stream);
        if (rc != DCN_OK) return rc;
    }
    if (keys > 0)
        rc = launch_attn(dkv, a, dim3((Lk + bt - 1) / bt, N * Mk), dcnb::kAttnThreads, smem,
                         stream);
    return rc;
}

}  // extern "C"
