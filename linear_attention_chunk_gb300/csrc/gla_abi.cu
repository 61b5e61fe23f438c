// gla_abi.cu -- the C ABI of libgla (declared in include/gla.h): host-side
// argument validation, the device status word, and dispatch to the kernels.
//
// The operations are those of "Beyond the KV cache: Training and serving
// i14's Laplace 3B linear attention model on AWS Trainium2 with native
// PyTorch": the Simple GLA recurrence of the "GLA mixer" paragraph, its
// chunked form ("Challenge 1"), its backward through the serial state chain
// ("Challenge 3") and the serving step ("Inference optimization on
// Trainium2"). Every argument error is caught here, before any launch.
#include <cuda_runtime.h>

#include <mutex>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include "gla.h"
#include "common.cuh"
#include "kernels.h"

namespace gla {

// One status word per device that loads the library; kernels set bits in it
// (kDevTimeout, ...) and gla_check() reads and clears it.
static __device__ unsigned int g_status_word;

namespace {

thread_local char t_err[512] = {0};
thread_local int t_launches = 0;

constexpr int kMaxDevices = 64;
std::mutex g_mu;
unsigned int *g_status_ptr[kMaxDevices] = {nullptr};

gla_status fail(gla_status st, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(t_err, sizeof t_err, fmt, ap);
    va_end(ap);
    return st;
}

gla_status cuda_fail(cudaError_t e, const char *where) {
    return fail(GLA_ERR_CUDA, "%s: %s (%s)", where, cudaGetErrorName(e), cudaGetErrorString(e));
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Device address of this device's status word (looked up once per device).
gla_status status_word(unsigned int **out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if (dev < 0 || dev >= kMaxDevices) return fail(GLA_ERR_UNSUPPORTED, "device index %d out of range", dev);
    std::lock_guard<std::mutex> lk(g_mu);
    if (!g_status_ptr[dev]) {
        void *ptr = nullptr;
        e = cudaGetSymbolAddress(&ptr, g_status_word);
        if (e != cudaSuccess) return cuda_fail(e, "cudaGetSymbolAddress(status word)");
        g_status_ptr[dev] = static_cast<unsigned int *>(ptr);
    }
    *out = g_status_ptr[dev];
    return GLA_OK;
}

// Common shape checks of the chunk entry points.
gla_status check_chunk_shape(int B, int T, int H, int dk, int dv, int chunk, gla_dtype dtype) {
    if (dtype != GLA_BF16 && dtype != GLA_FP32) return fail(GLA_ERR_INVALID_ARG, "dtype %d is not GLA_BF16/GLA_FP32", (int)dtype);
    if (B < 0 || T < 0 || H < 0) return fail(GLA_ERR_INVALID_ARG, "negative size B=%d T=%d H=%d", B, T, H);
    if (dk <= 0 || dv <= 0) return fail(GLA_ERR_INVALID_ARG, "dk=%d dv=%d must be positive", dk, dv);
    if (chunk != 64 && chunk != 128) return fail(GLA_ERR_UNSUPPORTED, "chunk %d is not 64 or 128", chunk);
    if (dtype == GLA_BF16 && (dk != 96 || dv != 192))
        return fail(GLA_ERR_UNSUPPORTED, "GLA_BF16 needs dk=96, dv=192 (got %d, %d)", dk, dv);
    if (dtype == GLA_FP32 && (dk > 128 || dv > 256))
        return fail(GLA_ERR_UNSUPPORTED, "GLA_FP32 needs dk <= 128, dv <= 256 (got %d, %d)", dk, dv);
    const long double elems = (long double)B * T * H * (dk > dv ? dk : dv);
    if (elems > (long double)(1ull << 40)) return fail(GLA_ERR_INVALID_ARG, "tensor too large (%Lg elements)", elems);
    if ((long double)B * H > 2147483647.0L) return fail(GLA_ERR_INVALID_ARG, "B*H too large");
    return GLA_OK;
}

#define REQUIRE_PTR(p, name)                                                              \
    do {                                                                                  \
        if (!(p)) return fail(GLA_ERR_INVALID_ARG, "%s is NULL", name);                   \
        if (!aligned16(p)) return fail(GLA_ERR_INVALID_ARG, "%s is not 16-byte aligned", name); \
    } while (0)

#define OPTIONAL_PTR(p, name)                                                             \
    do {                                                                                  \
        if ((p) && !aligned16(p)) return fail(GLA_ERR_INVALID_ARG, "%s is not 16-byte aligned", name); \
    } while (0)

// Device arrays of 4-byte numbers that kernels read one by one (a slice of a longer one passes).
#define REQUIRE_INTS(p, name)                                                             \
    do {                                                                                  \
        if (!(p)) return fail(GLA_ERR_INVALID_ARG, "%s is NULL", name);                   \
        OPTIONAL_INTS(p, name);                                                           \
    } while (0)

#define OPTIONAL_INTS(p, name)                                                            \
    do {                                                                                  \
        if (reinterpret_cast<uintptr_t>(p) & 3u) return fail(GLA_ERR_INVALID_ARG, "%s is not 4-byte aligned", name); \
    } while (0)

// Shape checks of the Conv1d entry points (B sequences of T tokens of D channels).
gla_status check_conv_shape(int B, int T, int D, gla_dtype dtype) {
    if (dtype != GLA_BF16 && dtype != GLA_FP32) return fail(GLA_ERR_INVALID_ARG, "dtype %d is not GLA_BF16/GLA_FP32", (int)dtype);
    if (B < 0 || T < 0) return fail(GLA_ERR_INVALID_ARG, "negative size B=%d T=%d", B, T);
    const int vec = dtype == GLA_BF16 ? 8 : 4;
    if (D <= 0 || D % vec != 0) return fail(GLA_ERR_UNSUPPORTED, "D=%d must be a positive multiple of %d", D, vec);
    if ((long double)B * T * D > (long double)(1ull << 40)) return fail(GLA_ERR_INVALID_ARG, "tensor too large");
    return GLA_OK;
}

gla_status check_conv_bwd_shape(int B, int T, int D, gla_dtype dtype) {
    const gla_status st = check_conv_shape(B, T, D, dtype);
    if (st == GLA_OK && T > 2147483647 - 256)   // the kernel's token numbers, a tile and a step past the end, stay ints
        return fail(GLA_ERR_INVALID_ARG, "T=%d is too long", T);
    return st;
}

// The decode step with or without the mixer epilogue (g == NULL: plain o).
gla_status decode_common(const void *q, const void *k, const void *v, const float *log_lambda, float *S_inout,
                         float scale, const void *g, const float *aug, const float *norm_w, float eps, int N,
                         int H, int dk, int dv, gla_dtype dtype, void *o, void *stream, const char *name,
                         const float *log_decay = nullptr) {
    t_err[0] = 0;
    t_launches = 0;
    if (dtype != GLA_BF16 && dtype != GLA_FP32) return fail(GLA_ERR_INVALID_ARG, "dtype %d invalid", (int)dtype);
    if (N < 0 || H < 0) return fail(GLA_ERR_INVALID_ARG, "negative size N=%d H=%d", N, H);
    if (dk <= 0 || dv <= 0) return fail(GLA_ERR_INVALID_ARG, "dk=%d dv=%d must be positive", dk, dv);
    if (dtype == GLA_BF16 && (dk != 96 || dv != 192))
        return fail(GLA_ERR_UNSUPPORTED, "GLA_BF16 needs dk=96, dv=192 (got %d, %d)", dk, dv);
    if (dtype == GLA_FP32 && (dk > 128 || dv > 256))
        return fail(GLA_ERR_UNSUPPORTED, "GLA_FP32 needs dk <= 128, dv <= 256 (got %d, %d)", dk, dv);
    if ((long double)N * H > 2147483647.0L) return fail(GLA_ERR_INVALID_ARG, "N*H too large");
    if (!(eps >= 0.f)) return fail(GLA_ERR_INVALID_ARG, "eps must be >= 0");
    OPTIONAL_PTR(aug, "aug");
    OPTIONAL_PTR(norm_w, "norm_w");
    if (N == 0 || H == 0) return GLA_OK;
    REQUIRE_PTR(q, "q");
    REQUIRE_PTR(k, "k");
    REQUIRE_PTR(v, "v");
    if (log_decay) {
        REQUIRE_PTR(log_decay, "g");
    } else {
        REQUIRE_PTR(log_lambda, "log_lambda");
    }
    REQUIRE_PTR(S_inout, "S_inout");
    REQUIRE_PTR(o, name);
    unsigned int *status = nullptr;
    gla_status st = status_word(&status);
    if (st != GLA_OK) return st;
    DecodeParams p{q, k, v, log_lambda, S_inout, scale, N, H, dk, dv, o, status, g, aug, norm_w, eps, log_decay};
    int launches = 0;
    cudaError_t e = launch_decode(p, dtype == GLA_BF16, static_cast<cudaStream_t>(stream), &launches);
    t_launches = launches;
    return e == cudaSuccess ? GLA_OK : cuda_fail(e, "decode launch");
}

gla_status check_norm_shape(int64_t rows, int D, gla_dtype dtype) {
    if (dtype != GLA_BF16 && dtype != GLA_FP32) return fail(GLA_ERR_INVALID_ARG, "dtype %d is not GLA_BF16/GLA_FP32", (int)dtype);
    if (rows < 0 || rows > 2147483647ll) return fail(GLA_ERR_INVALID_ARG, "rows=%lld out of range", (long long)rows);
    const int vec = dtype == GLA_BF16 ? 8 : 4;
    if (D <= 0 || D % vec != 0 || D > 8192)
        return fail(GLA_ERR_UNSUPPORTED, "D=%d must be a positive multiple of %d, at most 8192", D, vec);
    if ((long double)rows * D > (long double)(1ull << 40)) return fail(GLA_ERR_INVALID_ARG, "tensor too large");
    return GLA_OK;
}

// A [rows, cols] array of a selective-scan call: pointer, row step, alignment.
gla_status check_rows(const void *ptr, int64_t ld, int cols, int elem, bool vector, const char *name) {
    if (!ptr) return fail(GLA_ERR_INVALID_ARG, "%s is NULL", name);
    const uintptr_t align = vector ? 16 : (uintptr_t)elem;
    if (reinterpret_cast<uintptr_t>(ptr) % align) return fail(GLA_ERR_INVALID_ARG, "%s is not %d-byte aligned", name, (int)align);
    if (ld < cols) return fail(GLA_ERR_INVALID_ARG, "%s has rows of %d elements %lld apart", name, cols, (long long)ld);
    if (vector && (ld * elem) % 16) return fail(GLA_ERR_INVALID_ARG, "%s has rows that are not 16-byte aligned", name);
    if (ld > 2147483647ll) return fail(GLA_ERR_INVALID_ARG, "%s has rows too far apart", name);
    return GLA_OK;
}

gla_status check_ssm_shape(int64_t seqs, int64_t rows, int D, int N, gla_dtype dtype) {
    if (dtype != GLA_BF16 && dtype != GLA_FP32) return fail(GLA_ERR_INVALID_ARG, "dtype %d is not GLA_BF16/GLA_FP32", (int)dtype);
    if (seqs < 0 || rows < 0) return fail(GLA_ERR_INVALID_ARG, "negative size (sequences %lld, tokens %lld)", (long long)seqs, (long long)rows);
    const int vec = dtype == GLA_BF16 ? 8 : 4;
    if (D <= 0 || D % vec != 0) return fail(GLA_ERR_UNSUPPORTED, "D=%d must be a positive multiple of %d", D, vec);
    if (N != 8 && N != 16 && N != 32) return fail(GLA_ERR_UNSUPPORTED, "N=%d is not 8, 16 or 32", N);
    if (D > (1 << 25)) return fail(GLA_ERR_UNSUPPORTED, "D=%d is above 2^25", D);   // D * N and D * 4 fit an int
    // at most one CTA per 16 channels of a sequence or segment: inside a 1-D grid
    if ((long double)(seqs + rows) * ((D + 15) / 16) > 2147483647.0L || (long double)rows * D > (long double)(1ull << 40))
        return fail(GLA_ERR_INVALID_ARG, "tensor too large");
    return GLA_OK;
}

// The arrays every selective-scan call reads.
gla_status check_ssm_inputs(const SsmParams &p, gla_dtype dtype) {
    const int e = dtype == GLA_BF16 ? 2 : 4;
    gla_status st;
    if ((st = check_rows(p.x, p.ldx, p.D, e, true, "x")) != GLA_OK) return st;
    if ((st = check_rows(p.dt, p.ldt, p.D, e, true, "dt")) != GLA_OK) return st;
    if ((st = check_rows(p.Bm, p.ldb, p.N, e, false, "Bm")) != GLA_OK) return st;
    if ((st = check_rows(p.Cm, p.ldc, p.N, e, false, "Cm")) != GLA_OK) return st;
    if (p.z && (st = check_rows(p.z, p.ldz, p.D, e, true, "z")) != GLA_OK) return st;
    REQUIRE_PTR(p.A, "A");
    OPTIONAL_PTR(p.skip, "skip");
    OPTIONAL_PTR(p.dt_bias, "dt_bias");
    return GLA_OK;
}

// Pools, windows and filter of the packed and the single-token calls.
gla_status check_ssm_pools(const SsmParams &p) {
    if (p.n_slots < 0) return fail(GLA_ERR_INVALID_ARG, "negative n_slots=%d", p.n_slots);
    if (!p.slots && p.n_slots < p.nseq)
        return fail(GLA_ERR_INVALID_ARG, "without slots the pool needs nseq=%d slots, has %d", p.nseq, p.n_slots);
    OPTIONAL_PTR(p.slots, "slots");
    REQUIRE_PTR(p.h0, "state_pool");
    OPTIONAL_PTR(p.conv_w, "conv_w");
    OPTIONAL_PTR(p.conv_b, "conv_b");
    OPTIONAL_PTR(p.win, "win_pool");
    if ((p.conv_w != nullptr) != (p.win != nullptr))
        return fail(GLA_ERR_INVALID_ARG, "conv_w and win_pool come together");
    if (p.conv_b && !p.conv_w) return fail(GLA_ERR_INVALID_ARG, "conv_b without conv_w");
    return GLA_OK;
}

// Shape checks of the calls over trees of drafted tokens: the state's part.
gla_status check_tree_shape(int nseq, int total_T, int H, int dk, int dv, gla_dtype dtype) {
    if (dtype != GLA_BF16 && dtype != GLA_FP32) return fail(GLA_ERR_INVALID_ARG, "dtype %d is not GLA_BF16/GLA_FP32", (int)dtype);
    if (nseq < 0 || total_T < 0 || H < 0) return fail(GLA_ERR_INVALID_ARG, "negative size nseq=%d total_T=%d H=%d", nseq, total_T, H);
    if (dk <= 0 || dv <= 0) return fail(GLA_ERR_INVALID_ARG, "dk=%d dv=%d must be positive", dk, dv);
    if (dtype == GLA_BF16 && (dk != 96 || dv != 192))
        return fail(GLA_ERR_UNSUPPORTED, "GLA_BF16 needs dk=96, dv=192 (got %d, %d)", dk, dv);
    if (dtype == GLA_FP32 && (dk > 128 || dv > 256))
        return fail(GLA_ERR_UNSUPPORTED, "GLA_FP32 needs dk <= 128, dv <= 256 (got %d, %d)", dk, dv);
    if ((long double)nseq * H > 2147483647.0L) return fail(GLA_ERR_INVALID_ARG, "nseq*H too large");
    if ((long double)H * (dk > dv ? dk : dv) > 2147483647.0L) return fail(GLA_ERR_INVALID_ARG, "H=%d too large", H);
    return GLA_OK;
}

// The trees and the pool's slots.
gla_status check_trees(const TreeParams &p) {
    if (p.n_slots < 0) return fail(GLA_ERR_INVALID_ARG, "negative n_slots=%d", p.n_slots);
    if (!p.slots && p.n_slots < p.nseq)
        return fail(GLA_ERR_INVALID_ARG, "without slots the pool needs nseq=%d slots, has %d", p.nseq, p.n_slots);
    REQUIRE_INTS(p.cu, "cu_nodes");
    OPTIONAL_INTS(p.slots, "slots");
    if (p.total_T > 0) REQUIRE_INTS(p.parents, "parents");
    return GLA_OK;
}

// An array of [total_T, H, d] rows: 16-byte loads at bf16, single elements at fp32.
gla_status check_heads(const void *ptr, int64_t ld, int H, int d, gla_dtype dtype, const char *name) {
    return check_rows(ptr, ld, H * d, dtype == GLA_BF16 ? 2 : 4, dtype == GLA_BF16, name);
}

// The pools of a call over pages.
gla_status check_pools(PageParams &p, void *const *pools, const int64_t *page_bytes, int n_pools, int n_slots) {
    if (n_pools < 0 || n_slots < 0) return fail(GLA_ERR_INVALID_ARG, "negative size n_pools=%d n_slots=%d", n_pools, n_slots);
    if (n_pools > kMaxPools) return fail(GLA_ERR_UNSUPPORTED, "%d pools in one call, at most %d", n_pools, kMaxPools);
    if (n_pools > 0 && (!pools || !page_bytes)) return fail(GLA_ERR_INVALID_ARG, "pools or page_bytes is NULL");
    long double all = 0;
    for (int i = 0; i < n_pools; ++i) {
        if (n_slots > 0) REQUIRE_PTR(pools[i], "a pool");   // (without pages there is nothing to point at)
        if (page_bytes[i] <= 0 || page_bytes[i] % 4 != 0)
            return fail(GLA_ERR_UNSUPPORTED, "pages of %lld bytes: a positive multiple of 4 is needed", (long long)page_bytes[i]);
        if (page_bytes[i] > (1ll << 36)) return fail(GLA_ERR_INVALID_ARG, "pages of %lld bytes are too large", (long long)page_bytes[i]);
        all += page_bytes[i];
        p.pool[i] = pools[i];
        p.bytes[i] = (long)page_bytes[i];
    }
    if (all * n_slots > (long double)(1ull << 48) || all > (long double)(1ull << 40)) return fail(GLA_ERR_INVALID_ARG, "pools too large");
    p.n_pools = n_pools;
    p.n_slots = n_slots;
    return GLA_OK;
}

// Splits the workspace of a segmented scan; without enough of it, one segment per sequence.
void ssm_workspace(SsmParams &p, SsmPlan plan, void *workspace, size_t bytes, bool varlen) {
    const size_t need = ssm_workspace_bytes(plan, p.nseq, p.D, p.N);
    if (need == 0 || !workspace || bytes < need) plan = SsmPlan{varlen ? p.rows : p.T, p.nseq};
    else {
        p.seg_h = static_cast<float *>(workspace);
        p.seg_sum = p.seg_h + (size_t)plan.slots * p.D * p.N;
    }
    p.L = plan.L;
    p.nseg = varlen ? 0 : (int)((p.T + p.L - 1) / p.L);
}

}  // namespace

void set_error_detail(const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(t_err, sizeof t_err, fmt, ap);
    va_end(ap);
}

void reset_call_state() {
    t_err[0] = 0;
    t_launches = 0;
}

}  // namespace gla

using namespace gla;

extern "C" {

gla_status gla_chunk_fwd(const void *q, const void *k, const void *v, const float *log_lambda,
                         const float *h0, float scale, int B, int T, int H, int dk, int dv, int chunk,
                         gla_dtype dtype, void *o, float *hT, void *workspace, size_t workspace_bytes,
                         void *stream) {
    t_err[0] = 0;
    t_launches = 0;
    gla_status st = check_chunk_shape(B, T, H, dk, dv, chunk, dtype);
    if (st != GLA_OK) return st;
    OPTIONAL_PTR(h0, "h0");
    OPTIONAL_PTR(hT, "hT");
    OPTIONAL_PTR(workspace, "workspace");
    if (B == 0 || H == 0) return GLA_OK;
    REQUIRE_PTR(log_lambda, "log_lambda");
    if (T > 0) {
        REQUIRE_PTR(q, "q");
        REQUIRE_PTR(k, "k");
        REQUIRE_PTR(v, "v");
        REQUIRE_PTR(o, "o");
    }
    unsigned int *status = nullptr;
    if ((st = status_word(&status)) != GLA_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int launches = 0;
    cudaError_t e;
    if (T == 0) {
        e = launch_copy_state(h0, hT, (size_t)B * H * dk * dv, s, &launches);
        t_launches = launches;
        return e == cudaSuccess ? GLA_OK : cuda_fail(e, "gla_chunk_fwd(T=0)");
    }
    FwdParams p{q, k, v, log_lambda, h0, scale, B, T, H, dk, dv, chunk, o, hT,
                workspace, workspace ? workspace_bytes : 0, status};
    if (dtype == GLA_BF16)
        e = launch_fwd_tc(p, s, &launches);
    else
        e = launch_fwd_simt(p, false, s, &launches);
    t_launches = launches;
    return e == cudaSuccess ? GLA_OK : cuda_fail(e, "gla_chunk_fwd launch");
}

gla_status gla_chunk_fwd_gated(const void *q, const void *k, const void *v, const float *g, const float *h0,
                               float scale, int B, int T, int H, int dk, int dv, int chunk, gla_dtype dtype,
                               void *o, float *hT, void *workspace, size_t workspace_bytes, void *stream) {
    t_err[0] = 0;
    t_launches = 0;
    gla_status st = check_chunk_shape(B, T, H, dk, dv, chunk, dtype);
    if (st != GLA_OK) return st;
    OPTIONAL_PTR(h0, "h0");
    OPTIONAL_PTR(hT, "hT");
    OPTIONAL_PTR(workspace, "workspace");
    if (B == 0 || H == 0) return GLA_OK;
    if (T > 0) {
        REQUIRE_PTR(q, "q");
        REQUIRE_PTR(k, "k");
        REQUIRE_PTR(v, "v");
        REQUIRE_PTR(g, "g");
        REQUIRE_PTR(o, "o");
    }
    unsigned int *status = nullptr;
    if ((st = status_word(&status)) != GLA_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int launches = 0;
    cudaError_t e;
    if (T == 0) {
        e = launch_copy_state(h0, hT, (size_t)B * H * dk * dv, s, &launches);
        t_launches = launches;
        return e == cudaSuccess ? GLA_OK : cuda_fail(e, "gla_chunk_fwd_gated(T=0)");
    }
    FwdParams p{q, k, v, nullptr, h0, scale, B, T, H, dk, dv, chunk, o, hT,
                workspace, workspace ? workspace_bytes : 0, status, g};
    if (dtype == GLA_BF16)
        e = launch_fwd_tc(p, s, &launches);
    else
        e = launch_fwd_simt(p, false, s, &launches);
    t_launches = launches;
    return e == cudaSuccess ? GLA_OK : cuda_fail(e, "gla_chunk_fwd_gated launch");
}

size_t gla_chunk_fwd_gated_workspace_size(int B, int T, int H, int dk, int dv, int chunk, gla_dtype dtype) {
    if (check_chunk_shape(B, T, H, dk, dv, chunk, dtype) != GLA_OK) return 0;
    if (dtype != GLA_BF16) return 0;
    return fwd_tc_workspace_size(B, T, H, chunk, true);
}

gla_status gla_decode_step_gated(const void *q, const void *k, const void *v, const float *g, float *S_inout,
                                 float scale, int N, int H, int dk, int dv, gla_dtype dtype, void *o, void *stream) {
    if (N > 0 && H > 0 && !g) return fail(GLA_ERR_INVALID_ARG, "g is NULL");
    return decode_common(q, k, v, nullptr, S_inout, scale, nullptr, nullptr, nullptr, 0.f, N, H, dk, dv, dtype, o,
                         stream, "o", g);
}

gla_status gla_chunk_fwd_mixer(const void *q, const void *k, const void *v, const void *g, const float *log_lambda,
                               const float *h0, float scale, const float *aug, const float *norm_w, float eps, int B,
                               int T, int H, int dk, int dv, int chunk, gla_dtype dtype, void *z, float *hT,
                               void *workspace, size_t workspace_bytes, void *stream) {
    t_err[0] = 0;
    t_launches = 0;
    gla_status st = check_chunk_shape(B, T, H, dk, dv, chunk, dtype);
    if (st != GLA_OK) return st;
    if (dtype != GLA_BF16) return fail(GLA_ERR_UNSUPPORTED, "gla_chunk_fwd_mixer supports GLA_BF16 only");
    if (!(eps >= 0.f)) return fail(GLA_ERR_INVALID_ARG, "eps must be >= 0");
    OPTIONAL_PTR(h0, "h0");
    OPTIONAL_PTR(hT, "hT");
    OPTIONAL_PTR(aug, "aug");
    OPTIONAL_PTR(norm_w, "norm_w");
    OPTIONAL_PTR(workspace, "workspace");
    if (B == 0 || H == 0) return GLA_OK;
    if ((long double)B * T > 2147483647.0L || (long double)B * T * H > 2147483647.0L * 8.0L)
        return fail(GLA_ERR_INVALID_ARG, "B*T or B*T*H too large");
    REQUIRE_PTR(log_lambda, "log_lambda");
    if (T > 0) {
        REQUIRE_PTR(q, "q");
        REQUIRE_PTR(k, "k");
        REQUIRE_PTR(v, "v");
        REQUIRE_PTR(g, "g");
        REQUIRE_PTR(z, "z");
        if (z == q || z == k || z == v || z == g) return fail(GLA_ERR_INVALID_ARG, "z may not alias an input");
    }
    unsigned int *status = nullptr;
    if ((st = status_word(&status)) != GLA_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int launches = 0;
    cudaError_t e;
    if (T == 0) {
        e = launch_copy_state(h0, hT, (size_t)B * H * dk * dv, s, &launches);
        t_launches = launches;
        return e == cudaSuccess ? GLA_OK : cuda_fail(e, "gla_chunk_fwd_mixer(T=0)");
    }
    // The forward writes into z's buffer either the normalised rows, which a
    // second pass multiplies by the norm weight and the SiLU gate (one CTA per
    // chain at chunk 128), or o, which the epilogue then rewrites row by row
    // in place (a warp reads all of a row's inputs before storing it).
    FwdParams p{q, k, v, log_lambda, h0, scale, B, T, H, dk, dv, chunk, z, hT,
                workspace, workspace ? workspace_bytes : 0, status};
    const EpilogueParams ep{z, q, k, v, g, aug, norm_w, eps, B * T, H, dk, dv, z};
    e = launch_fwd_tc(p, s, &launches, &ep);
    t_launches = launches;
    return e == cudaSuccess ? GLA_OK : cuda_fail(e, "gla_chunk_fwd_mixer launch");
}

size_t gla_chunk_fwd_workspace_size(int B, int T, int H, int dk, int dv, int chunk, gla_dtype dtype) {
    if (check_chunk_shape(B, T, H, dk, dv, chunk, dtype) != GLA_OK) return 0;
    if (dtype != GLA_BF16) return 0;
    return fwd_tc_workspace_size(B, T, H, chunk);
}

gla_status gla_chunk_bwd(const void *q, const void *k, const void *v, const float *log_lambda,
                         const float *h0, float scale, const void *do_, const float *dhT, int B, int T,
                         int H, int dk, int dv, int chunk, gla_dtype dtype, void *dq, void *dk_, void *dv_,
                         float *dh0, void *workspace, size_t workspace_bytes, void *stream) {
    t_err[0] = 0;
    t_launches = 0;
    gla_status st = check_chunk_shape(B, T, H, dk, dv, chunk, dtype);
    if (st != GLA_OK) return st;
    OPTIONAL_PTR(h0, "h0");
    OPTIONAL_PTR(dhT, "dhT");
    OPTIONAL_PTR(dh0, "dh0");
    OPTIONAL_PTR(workspace, "workspace");
    if (B == 0 || H == 0) return GLA_OK;
    REQUIRE_PTR(log_lambda, "log_lambda");
    const size_t need = gla_chunk_bwd_workspace_size(B, T, H, dk, dv, chunk, dtype);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need))
        return fail(GLA_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need,
                    workspace ? workspace_bytes : (size_t)0);
    if (T > 0) {
        REQUIRE_PTR(q, "q");
        REQUIRE_PTR(k, "k");
        REQUIRE_PTR(v, "v");
        REQUIRE_PTR(do_, "do");
        REQUIRE_PTR(dq, "dq");
        REQUIRE_PTR(dk_, "dk");
        REQUIRE_PTR(dv_, "dv");
    }
    unsigned int *status = nullptr;
    if ((st = status_word(&status)) != GLA_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int launches = 0;
    cudaError_t e;
    if (T == 0) {
        // No tokens: dh0 = dhT (the state passes through untouched).
        e = launch_copy_state(dhT, dh0, (size_t)B * H * dk * dv, s, &launches);
        t_launches = launches;
        return e == cudaSuccess ? GLA_OK : cuda_fail(e, "gla_chunk_bwd(T=0)");
    }
    BwdParams p{q, k, v, log_lambda, h0, scale, do_, dhT, B, T, H, dk, dv, chunk, dq, dk_, dv_, dh0,
                workspace, workspace ? workspace_bytes : 0, status};
    if (dtype == GLA_BF16)
        e = launch_bwd_tc(p, s, &launches);
    else
        e = launch_bwd_simt(p, false, s, &launches);
    t_launches = launches;
    return e == cudaSuccess ? GLA_OK : cuda_fail(e, "gla_chunk_bwd launch");
}

size_t gla_chunk_bwd_gated_workspace_size(int B, int T, int H, int dk, int dv, int chunk, gla_dtype dtype) {
    if (check_chunk_shape(B, T, H, dk, dv, chunk, dtype) != GLA_OK) return 0;
    if (dtype == GLA_BF16) return bwd_gated_tc_workspace_size(B, T, H, chunk);
    const size_t nck = ((size_t)T + chunk - 1) / chunk;
    return 2 * (size_t)B * H * nck * dk * dv * sizeof(float);
}

gla_status gla_chunk_bwd_gated(const void *q, const void *k, const void *v, const float *g, const float *h0,
                               float scale, const void *do_, const float *dhT, int B, int T, int H, int dk, int dv,
                               int chunk, gla_dtype dtype, void *dq, void *dk_, void *dv_, float *dh0, float *dg,
                               void *workspace, size_t workspace_bytes, void *stream) {
    t_err[0] = 0;
    t_launches = 0;
    gla_status st = check_chunk_shape(B, T, H, dk, dv, chunk, dtype);
    if (st != GLA_OK) return st;
    OPTIONAL_PTR(h0, "h0");
    OPTIONAL_PTR(dhT, "dhT");
    OPTIONAL_PTR(dh0, "dh0");
    OPTIONAL_PTR(workspace, "workspace");
    if (B == 0 || H == 0) return GLA_OK;
    if ((long double)B * H * ((T + (long double)chunk - 1) / chunk) > 2147483647.0L)
        return fail(GLA_ERR_INVALID_ARG, "B*H*chunks too large");
    if (dtype == GLA_FP32 && (T + chunk - 1) / chunk > 65535)
        return fail(GLA_ERR_UNSUPPORTED, "GLA_FP32 gated backward needs at most 65535 chunks");
    if (T > 0) {
        REQUIRE_PTR(q, "q");
        REQUIRE_PTR(k, "k");
        REQUIRE_PTR(v, "v");
        REQUIRE_PTR(g, "g");
        REQUIRE_PTR(do_, "do");
        REQUIRE_PTR(dq, "dq");
        REQUIRE_PTR(dk_, "dk");
        REQUIRE_PTR(dv_, "dv");
        REQUIRE_PTR(dg, "dg");
        const size_t need = gla_chunk_bwd_gated_workspace_size(B, T, H, dk, dv, chunk, dtype);
        if (workspace == nullptr || workspace_bytes < need)
            return fail(GLA_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need,
                        workspace ? workspace_bytes : (size_t)0);
    }
    unsigned int *status = nullptr;
    if ((st = status_word(&status)) != GLA_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int launches = 0;
    cudaError_t e;
    if (T == 0) {
        // No tokens: dh0 = dhT (the state passes through untouched); no gates.
        e = launch_copy_state(dhT, dh0, (size_t)B * H * dk * dv, s, &launches);
        t_launches = launches;
        return e == cudaSuccess ? GLA_OK : cuda_fail(e, "gla_chunk_bwd_gated(T=0)");
    }
    BwdParams p{q, k, v, nullptr, h0, scale, do_, dhT, B, T, H, dk, dv, chunk, dq, dk_, dv_, dh0,
                workspace, workspace_bytes, status, g, dg};
    if (dtype == GLA_BF16)
        e = launch_bwd_gated_tc(p, s, &launches);
    else
        e = launch_bwd_simt(p, false, s, &launches);
    t_launches = launches;
    return e == cudaSuccess ? GLA_OK : cuda_fail(e, "gla_chunk_bwd_gated launch");
}

static gla_status varlen_common(const void *q, const void *k, const void *v, const float *log_lambda, const float *g,
                                float scale,
                                const int *cu_seqlens, const int *slots, float *state_pool, int n_slots, int nseq,
                                int total_T, int H, int dk, int dv, int chunk, gla_dtype dtype, void *o,
                                void *stream, const char *name) {
    t_err[0] = 0;
    t_launches = 0;
    gla_status st = check_chunk_shape(1, total_T, H, dk, dv, chunk, dtype);
    if (st != GLA_OK) return st;
    if (dtype != GLA_BF16) return fail(GLA_ERR_UNSUPPORTED, "%s supports GLA_BF16 only", name);
    if (nseq < 0 || n_slots < 0) return fail(GLA_ERR_INVALID_ARG, "negative nseq=%d or n_slots=%d", nseq, n_slots);
    if ((long double)nseq * H * 2 > 2147483647.0L) return fail(GLA_ERR_INVALID_ARG, "nseq*H too large");
    OPTIONAL_PTR(slots, "slots");
    if (nseq == 0 || H == 0) return GLA_OK;
    if (g) {
        REQUIRE_PTR(g, "g");
    } else {
        REQUIRE_PTR(log_lambda, "log_lambda");
    }
    REQUIRE_PTR(cu_seqlens, "cu_seqlens");
    REQUIRE_PTR(state_pool, "state_pool");
    if (!slots && n_slots < nseq)
        return fail(GLA_ERR_INVALID_ARG, "without slots the pool needs nseq=%d slots, has %d", nseq, n_slots);
    if (total_T > 0) {
        REQUIRE_PTR(q, "q");
        REQUIRE_PTR(k, "k");
        REQUIRE_PTR(v, "v");
        REQUIRE_PTR(o, "o");
    }
    unsigned int *status = nullptr;
    if ((st = status_word(&status)) != GLA_OK) return st;
    if (total_T == 0) return GLA_OK;   // every sequence is empty: no state changes
    VarlenParams p{q, k, v, log_lambda, scale, cu_seqlens, slots, state_pool, n_slots, nseq, total_T, H, dk, dv,
                   chunk, o, status, g};
    int launches = 0;
    const cudaError_t e = launch_fwd_varlen_tc(p, static_cast<cudaStream_t>(stream), &launches);
    t_launches = launches;
    return e == cudaSuccess ? GLA_OK : cuda_fail(e, name);
}

gla_status gla_chunk_fwd_varlen(const void *q, const void *k, const void *v, const float *log_lambda, float scale,
                                const int *cu_seqlens, const int *slots, float *state_pool, int n_slots, int nseq,
                                int total_T, int H, int dk, int dv, int chunk, gla_dtype dtype, void *o,
                                void *stream) {
    return varlen_common(q, k, v, log_lambda, nullptr, scale, cu_seqlens, slots, state_pool, n_slots, nseq, total_T, H,
                         dk, dv, chunk, dtype, o, stream, "gla_chunk_fwd_varlen");
}

gla_status gla_chunk_fwd_varlen_gated(const void *q, const void *k, const void *v, const float *g, float scale,
                                      const int *cu_seqlens, const int *slots, float *state_pool, int n_slots,
                                      int nseq, int total_T, int H, int dk, int dv, int chunk, gla_dtype dtype,
                                      void *o, void *stream) {
    if (nseq > 0 && H > 0 && total_T > 0 && !g) return fail(GLA_ERR_INVALID_ARG, "g is NULL");
    return varlen_common(q, k, v, nullptr, g, scale, cu_seqlens, slots, state_pool, n_slots, nseq, total_T, H, dk,
                         dv, chunk, dtype, o, stream, "gla_chunk_fwd_varlen_gated");
}

size_t gla_chunk_bwd_workspace_size(int B, int T, int H, int dk, int dv, int chunk, gla_dtype dtype) {
    if (check_chunk_shape(B, T, H, dk, dv, chunk, dtype) != GLA_OK) return 0;
    if (dtype != GLA_BF16) return 0;
    return bwd_tc_workspace_size(B, T, H, chunk);
}

gla_status gla_decode_step(const void *q, const void *k, const void *v, const float *log_lambda,
                           float *S_inout, float scale, int N, int H, int dk, int dv, gla_dtype dtype,
                           void *o, void *stream) {
    return decode_common(q, k, v, log_lambda, S_inout, scale, nullptr, nullptr, nullptr, 0.f, N, H, dk, dv, dtype,
                         o, stream, "o");
}

gla_status gla_decode_step_mixer(const void *q, const void *k, const void *v, const float *log_lambda,
                                 float *S_inout, float scale, const void *g, const float *aug,
                                 const float *norm_w, float eps, int N, int H, int dk, int dv, gla_dtype dtype,
                                 void *z, void *stream) {
    if (N > 0 && H > 0) {
        if (!g) return fail(GLA_ERR_INVALID_ARG, "g is NULL");
        if (!aligned16(g)) return fail(GLA_ERR_INVALID_ARG, "g is not 16-byte aligned");
    }
    return decode_common(q, k, v, log_lambda, S_inout, scale, g, aug, norm_w, eps, N, H, dk, dv, dtype, z, stream,
                         "z");
}

gla_status gla_mixer_epilogue(const void *o, const void *q, const void *k, const void *v, const void *g,
                              const float *aug, const float *norm_w, float eps, int NT, int H, int dk, int dv,
                              gla_dtype dtype, void *z, void *stream) {
    t_err[0] = 0;
    t_launches = 0;
    if (dtype != GLA_BF16 && dtype != GLA_FP32) return fail(GLA_ERR_INVALID_ARG, "dtype %d invalid", (int)dtype);
    if (NT < 0 || H < 0) return fail(GLA_ERR_INVALID_ARG, "negative size NT=%d H=%d", NT, H);
    if (dk <= 0 || dv <= 0) return fail(GLA_ERR_INVALID_ARG, "dk=%d dv=%d must be positive", dk, dv);
    if (dk > 1024 || dv > 256) return fail(GLA_ERR_UNSUPPORTED, "needs dk <= 1024, dv <= 256 (got %d, %d)", dk, dv);
    if ((long double)NT * H > 2147483647.0L * 8.0L) return fail(GLA_ERR_INVALID_ARG, "NT*H too large");
    if (!(eps >= 0.f)) return fail(GLA_ERR_INVALID_ARG, "eps must be >= 0");
    OPTIONAL_PTR(aug, "aug");
    OPTIONAL_PTR(norm_w, "norm_w");
    if (NT == 0 || H == 0) return GLA_OK;
    REQUIRE_PTR(o, "o");
    REQUIRE_PTR(q, "q");
    REQUIRE_PTR(k, "k");
    REQUIRE_PTR(v, "v");
    REQUIRE_PTR(g, "g");
    REQUIRE_PTR(z, "z");
    EpilogueParams p{o, q, k, v, g, aug, norm_w, eps, NT, H, dk, dv, z};
    int launches = 0;
    cudaError_t e = launch_mixer_epilogue(p, dtype == GLA_BF16, static_cast<cudaStream_t>(stream), &launches);
    t_launches = launches;
    return e == cudaSuccess ? GLA_OK : cuda_fail(e, "gla_mixer_epilogue launch");
}

gla_status gla_conv1d_fwd(const void *x, const float *w, const float *b, const float *win_in, int B, int T, int D,
                          gla_dtype dtype, void *y, float *win_out, void *stream) {
    t_err[0] = 0;
    t_launches = 0;
    gla_status st = check_conv_shape(B, T, D, dtype);
    if (st != GLA_OK) return st;
    OPTIONAL_PTR(b, "b");
    OPTIONAL_PTR(win_in, "win_in");
    OPTIONAL_PTR(win_out, "win_out");
    if (B == 0 || (T == 0 && !win_out)) return GLA_OK;
    REQUIRE_PTR(w, "w");
    if (T > 0) {
        REQUIRE_PTR(x, "x");
        REQUIRE_PTR(y, "y");
        if (x == y) return fail(GLA_ERR_INVALID_ARG, "y may not alias x");
    }
    unsigned int *status = nullptr;
    if ((st = status_word(&status)) != GLA_OK) return st;
    ConvParams p{x, w, b, nullptr, nullptr, win_in, win_out, B, B, (long)B * T, T, D, y, status};
    int launches = 0;
    const cudaError_t e = launch_conv_fwd(p, false, dtype == GLA_BF16, static_cast<cudaStream_t>(stream), &launches);
    t_launches = launches;
    return e == cudaSuccess ? GLA_OK : cuda_fail(e, "gla_conv1d_fwd launch");
}

gla_status gla_conv1d_varlen(const void *x, const float *w, const float *b, const int *cu_seqlens,
                             const int *slots, float *win_pool, int n_slots, int nseq, int total_T, int D,
                             gla_dtype dtype, void *y, void *stream) {
    t_err[0] = 0;
    t_launches = 0;
    gla_status st = check_conv_shape(1, total_T, D, dtype);
    if (st != GLA_OK) return st;
    if (nseq < 0 || n_slots < 0) return fail(GLA_ERR_INVALID_ARG, "negative nseq=%d or n_slots=%d", nseq, n_slots);
    OPTIONAL_PTR(b, "b");
    OPTIONAL_PTR(slots, "slots");
    if (nseq == 0) return GLA_OK;
    if (!slots && n_slots < nseq)
        return fail(GLA_ERR_INVALID_ARG, "without slots the pool needs nseq=%d slots, has %d", nseq, n_slots);
    REQUIRE_PTR(w, "w");
    REQUIRE_PTR(cu_seqlens, "cu_seqlens");
    REQUIRE_PTR(win_pool, "win_pool");
    if (total_T == 0) return GLA_OK;   // every sequence is empty: no window changes
    REQUIRE_PTR(x, "x");
    REQUIRE_PTR(y, "y");
    if (x == y) return fail(GLA_ERR_INVALID_ARG, "y may not alias x");
    unsigned int *status = nullptr;
    if ((st = status_word(&status)) != GLA_OK) return st;
    ConvParams p{x, w, b, cu_seqlens, slots, win_pool, win_pool, n_slots, nseq, (long)total_T, 0, D, y, status};
    int launches = 0;
    const cudaError_t e = launch_conv_fwd(p, true, dtype == GLA_BF16, static_cast<cudaStream_t>(stream), &launches);
    t_launches = launches;
    return e == cudaSuccess ? GLA_OK : cuda_fail(e, "gla_conv1d_varlen launch");
}

gla_status gla_conv1d_step(const void *x, const float *w, const float *b, float *win, int N, int D,
                           gla_dtype dtype, void *y, void *stream) {
    t_err[0] = 0;
    t_launches = 0;
    gla_status st = check_conv_shape(N, 1, D, dtype);
    if (st != GLA_OK) return st;
    OPTIONAL_PTR(b, "b");
    if (N == 0) return GLA_OK;
    REQUIRE_PTR(x, "x");
    REQUIRE_PTR(w, "w");
    REQUIRE_PTR(win, "win");
    REQUIRE_PTR(y, "y");
    if (x == y) return fail(GLA_ERR_INVALID_ARG, "y may not alias x");
    ConvParams p{x, w, b, nullptr, nullptr, win, win, N, N, (long)N, 1, D, y, nullptr};
    int launches = 0;
    const cudaError_t e = launch_conv_step(p, dtype == GLA_BF16, static_cast<cudaStream_t>(stream), &launches);
    t_launches = launches;
    return e == cudaSuccess ? GLA_OK : cuda_fail(e, "gla_conv1d_step launch");
}

gla_status gla_ssm_fwd(const void *x, int64_t ld_x, const void *dt, int64_t ld_dt, const float *A, const void *Bm,
                       int64_t ld_B, const void *Cm, int64_t ld_C, const float *skip, const void *z, int64_t ld_z,
                       const float *dt_bias, int softplus, const float *h0, int B, int T, int D, int N,
                       gla_dtype dtype, void *y, float *hT, void *workspace, size_t workspace_bytes, void *stream) {
    t_err[0] = 0;
    t_launches = 0;
    gla_status st = check_ssm_shape(B, T < 0 ? -1 : (int64_t)B * T, D, N, dtype);
    if (st != GLA_OK) return st;
    OPTIONAL_PTR(h0, "h0");
    OPTIONAL_PTR(hT, "hT");
    OPTIONAL_PTR(workspace, "workspace");
    if (B == 0) return GLA_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int launches = 0;
    cudaError_t e;
    if (T == 0) {
        if (h0 == hT) return GLA_OK;
        e = launch_copy_state(h0, hT, (size_t)B * D * N, s, &launches);
        t_launches = launches;
        return e == cudaSuccess ? GLA_OK : cuda_fail(e, "gla_ssm_fwd(T=0)");
    }
    SsmParams p{x, dt, z, Bm, Cm, (long)ld_x, (long)ld_dt, (long)ld_z, (long)ld_B, (long)ld_C, A, skip, dt_bias,
                nullptr, nullptr, h0, hT, nullptr, nullptr, nullptr, B, B, T, D, N, softplus, (long)B * T, y};
    if ((st = check_ssm_inputs(p, dtype)) != GLA_OK) return st;
    REQUIRE_PTR(y, "y");
    if (y == x || y == dt || y == z || y == Bm || y == Cm) return fail(GLA_ERR_INVALID_ARG, "y may not alias an input");
    ssm_workspace(p, plan_ssm(B, p.rows, D, false), workspace, workspace_bytes, false);
    e = launch_ssm_scan(p, dtype == GLA_BF16, s, &launches);
    t_launches = launches;
    return e == cudaSuccess ? GLA_OK : cuda_fail(e, "gla_ssm_fwd launch");
}

size_t gla_ssm_fwd_workspace_size(int B, int T, int D, int N, gla_dtype dtype) {
    if (check_ssm_shape(B, T < 0 ? -1 : (int64_t)B * T, D, N, dtype) != GLA_OK || B == 0 || T == 0) return 0;
    return ssm_workspace_bytes(plan_ssm(B, (long)B * T, D, false), B, D, N);
}

gla_status gla_ssm_varlen(const void *x, int64_t ld_x, const void *dt, int64_t ld_dt, const float *A, const void *Bm,
                          int64_t ld_B, const void *Cm, int64_t ld_C, const float *skip, const void *z, int64_t ld_z,
                          const float *dt_bias, int softplus, const float *conv_w, const float *conv_b,
                          const int *cu_seqlens, const int *slots, float *state_pool, float *win_pool, int n_slots,
                          int nseq, int total_T, int D, int N, gla_dtype dtype, void *y, void *workspace,
                          size_t workspace_bytes, void *stream) {
    t_err[0] = 0;
    t_launches = 0;
    gla_status st = check_ssm_shape(nseq, total_T, D, N, dtype);
    if (st != GLA_OK) return st;
    OPTIONAL_PTR(workspace, "workspace");
    if (nseq == 0) return GLA_OK;
    SsmParams p{x, dt, z, Bm, Cm, (long)ld_x, (long)ld_dt, (long)ld_z, (long)ld_B, (long)ld_C, A, skip, dt_bias,
                conv_w, conv_b, state_pool, state_pool, win_pool, cu_seqlens, slots, n_slots, nseq, 0, D, N, softplus,
                (long)total_T, y};
    REQUIRE_PTR(cu_seqlens, "cu_seqlens");
    if ((st = check_ssm_pools(p)) != GLA_OK) return st;
    if (total_T == 0) return GLA_OK;   // every sequence is empty: no state changes
    if ((st = check_ssm_inputs(p, dtype)) != GLA_OK) return st;
    REQUIRE_PTR(y, "y");
    if (y == x || y == dt || y == z || y == Bm || y == Cm) return fail(GLA_ERR_INVALID_ARG, "y may not alias an input");
    if ((st = status_word(&p.status)) != GLA_OK) return st;
    ssm_workspace(p, plan_ssm(nseq, total_T, D, true), workspace, workspace_bytes, true);
    int launches = 0;
    const cudaError_t e = launch_ssm_scan(p, dtype == GLA_BF16, static_cast<cudaStream_t>(stream), &launches);
    t_launches = launches;
    return e == cudaSuccess ? GLA_OK : cuda_fail(e, "gla_ssm_varlen launch");
}

size_t gla_ssm_varlen_workspace_size(int nseq, int total_T, int D, int N, gla_dtype dtype) {
    if (check_ssm_shape(nseq, total_T, D, N, dtype) != GLA_OK || nseq == 0 || total_T == 0) return 0;
    return ssm_workspace_bytes(plan_ssm(nseq, total_T, D, true), nseq, D, N);
}

gla_status gla_ssm_step(const void *x, int64_t ld_x, const void *dt, int64_t ld_dt, const float *A, const void *Bm,
                        int64_t ld_B, const void *Cm, int64_t ld_C, const float *skip, const void *z, int64_t ld_z,
                        const float *dt_bias, int softplus, const float *conv_w, const float *conv_b, const int *slots,
                        float *state_pool, float *win_pool, int n_slots, int nseq, int D, int N, gla_dtype dtype,
                        void *y, void *stream) {
    t_err[0] = 0;
    t_launches = 0;
    gla_status st = check_ssm_shape(nseq, nseq, D, N, dtype);
    if (st != GLA_OK) return st;
    if (nseq == 0) return GLA_OK;
    SsmParams p{x, dt, z, Bm, Cm, (long)ld_x, (long)ld_dt, (long)ld_z, (long)ld_B, (long)ld_C, A, skip, dt_bias,
                conv_w, conv_b, state_pool, state_pool, win_pool, nullptr, slots, n_slots, nseq, 1, D, N, softplus,
                (long)nseq, y};
    if ((st = check_ssm_pools(p)) != GLA_OK) return st;
    if ((st = check_ssm_inputs(p, dtype)) != GLA_OK) return st;
    REQUIRE_PTR(y, "y");
    if (y == x || y == dt || y == z || y == Bm || y == Cm) return fail(GLA_ERR_INVALID_ARG, "y may not alias an input");
    if ((st = status_word(&p.status)) != GLA_OK) return st;
    int launches = 0;
    const cudaError_t e = launch_ssm_step(p, dtype == GLA_BF16, static_cast<cudaStream_t>(stream), &launches);
    t_launches = launches;
    return e == cudaSuccess ? GLA_OK : cuda_fail(e, "gla_ssm_step launch");
}

size_t gla_ssm_bwd_workspace_size(int B, int T, int D, int N, gla_dtype dtype) {
    if (check_ssm_shape(B, T < 0 ? -1 : (int64_t)B * T, D, N, dtype) != GLA_OK || B == 0 || T == 0) return 0;
    SsmBwdParams p{};
    p.B = B;
    p.T = T;
    p.D = D;
    p.N = N;
    return plan_ssm_bwd(p, nullptr) * sizeof(float);
}

gla_status gla_ssm_bwd(const void *x, int64_t ld_x, const void *dt, int64_t ld_dt, const float *A, const void *Bm,
                       int64_t ld_B, const void *Cm, int64_t ld_C, const float *skip, const void *z, int64_t ld_z,
                       const float *dt_bias, int softplus, const float *h0, const void *dy, int64_t ld_dy,
                       const float *dhT, int B, int T, int D, int N, gla_dtype dtype, void *dx, void *ddt, float *dA,
                       void *dB, void *dC, float *dskip, void *dz, float *ddt_bias, float *dh0, void *workspace,
                       size_t workspace_bytes, void *stream) {
    t_err[0] = 0;
    t_launches = 0;
    gla_status st = check_ssm_shape(B, T < 0 ? -1 : (int64_t)B * T, D, N, dtype);
    if (st != GLA_OK) return st;
    OPTIONAL_PTR(h0, "h0");
    OPTIONAL_PTR(dhT, "dhT");
    OPTIONAL_PTR(dh0, "dh0");
    OPTIONAL_PTR(dskip, "dskip");
    OPTIONAL_PTR(ddt_bias, "ddt_bias");
    REQUIRE_PTR(dA, "dA");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int launches = 0;
    cudaError_t e;
    if (B == 0 || T == 0) {   // no tokens: the sums are empty, the state passes through
        e = cudaMemsetAsync(dA, 0, (size_t)D * N * sizeof(float), s);
        if (e == cudaSuccess && dskip) e = cudaMemsetAsync(dskip, 0, (size_t)D * sizeof(float), s);
        if (e == cudaSuccess && ddt_bias) e = cudaMemsetAsync(ddt_bias, 0, (size_t)D * sizeof(float), s);
        if (e == cudaSuccess && B > 0 && dh0 != dhT) e = launch_copy_state(dhT, dh0, (size_t)B * D * N, s, &launches);
        t_launches = launches;
        return e == cudaSuccess ? GLA_OK : cuda_fail(e, "gla_ssm_bwd(no tokens)");
    }
    SsmParams in{x, dt, z, Bm, Cm, (long)ld_x, (long)ld_dt, (long)ld_z, (long)ld_B, (long)ld_C, A, skip, dt_bias};
    in.D = D;
    in.N = N;
    if ((st = check_ssm_inputs(in, dtype)) != GLA_OK) return st;
    if ((st = check_rows(dy, ld_dy, D, dtype == GLA_BF16 ? 2 : 4, true, "dy")) != GLA_OK) return st;
    REQUIRE_PTR(dx, "dx");
    REQUIRE_PTR(ddt, "ddt");
    REQUIRE_PTR(dB, "dB");
    REQUIRE_PTR(dC, "dC");
    if ((z != nullptr) != (dz != nullptr)) return fail(GLA_ERR_INVALID_ARG, "z and dz come together");
    OPTIONAL_PTR(dz, "dz");
    for (const void *out : {(const void *)dx, (const void *)ddt, (const void *)dz, (const void *)dB, (const void *)dC})
        if (out && (out == x || out == dt || out == z || out == dy || out == Bm || out == Cm))
            return fail(GLA_ERR_INVALID_ARG, "an output may not alias an input");
    // every segment of a sequence reads its h0 and dhT, the first writes dh0
    if (dh0 && (dh0 == h0 || dh0 == dhT)) return fail(GLA_ERR_INVALID_ARG, "dh0 may not alias h0 or dhT");
    REQUIRE_PTR(workspace, "workspace");
    const size_t need = gla_ssm_bwd_workspace_size(B, T, D, N, dtype);
    if (workspace_bytes < need)
        return fail(GLA_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace_bytes);
    SsmBwdParams p{x, dt, z, Bm, Cm, dy, (long)ld_x, (long)ld_dt, (long)ld_z, (long)ld_B, (long)ld_C, (long)ld_dy, A, skip,
                   dt_bias, h0, dhT, B, T, D, N, softplus, dx, ddt, dz, dB, dC, dA, dskip, ddt_bias, dh0};
    plan_ssm_bwd(p, static_cast<float *>(workspace));
    e = launch_ssm_bwd(p, dtype == GLA_BF16, s, &launches);
    t_launches = launches;
    return e == cudaSuccess ? GLA_OK : cuda_fail(e, "gla_ssm_bwd launch");
}

size_t gla_conv1d_bwd_workspace_size(int B, int T, int D, gla_dtype dtype) {
    if (check_conv_bwd_shape(B, T, D, dtype) != GLA_OK || B == 0 || T == 0) return 0;
    const int tile = conv_bwd_tile(B, T, D);
    return (size_t)B * ((T + tile - 1) / tile) * 5 * D * sizeof(float);
}

gla_status gla_conv1d_bwd(const void *x, const float *w, const float *b, const void *dy, const float *win_in, int B,
                          int T, int D, gla_dtype dtype, void *dx, float *dw, float *db, void *workspace,
                          size_t workspace_bytes, void *stream) {
    t_err[0] = 0;
    t_launches = 0;
    gla_status st = check_conv_bwd_shape(B, T, D, dtype);
    if (st != GLA_OK) return st;
    OPTIONAL_PTR(b, "b");
    OPTIONAL_PTR(win_in, "win_in");
    OPTIONAL_PTR(db, "db");
    REQUIRE_PTR(dw, "dw");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int launches = 0;
    if (B == 0 || T == 0) {   // no tokens: the sums are empty
        cudaError_t e = cudaMemsetAsync(dw, 0, (size_t)D * 4 * sizeof(float), s);
        if (e == cudaSuccess && db) e = cudaMemsetAsync(db, 0, (size_t)D * sizeof(float), s);
        return e == cudaSuccess ? GLA_OK : cuda_fail(e, "gla_conv1d_bwd(no tokens)");
    }
    REQUIRE_PTR(w, "w");
    REQUIRE_PTR(x, "x");
    REQUIRE_PTR(dy, "dy");
    REQUIRE_PTR(dx, "dx");
    if (dx == x || dx == dy) return fail(GLA_ERR_INVALID_ARG, "dx may not alias x or dy");
    REQUIRE_PTR(workspace, "workspace");
    const size_t need = gla_conv1d_bwd_workspace_size(B, T, D, dtype);
    if (workspace_bytes < need)
        return fail(GLA_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace_bytes);
    ConvBwdParams p{x, dy, w, b, win_in, B, T, D, conv_bwd_tile(B, T, D), dx, dw, db, static_cast<float *>(workspace)};
    const cudaError_t e = launch_conv_bwd(p, dtype == GLA_BF16, s, &launches);
    t_launches = launches;
    return e == cudaSuccess ? GLA_OK : cuda_fail(e, "gla_conv1d_bwd launch");
}

gla_status gla_rmsnorm_fwd(const void *x, const void *res, const float *w, float eps, int64_t rows, int D, int group,
                           gla_dtype dtype, void *s_out, void *y, void *y8, float *scale, void *stream) {
    t_err[0] = 0;
    t_launches = 0;
    gla_status st = check_norm_shape(rows, D, dtype);
    if (st != GLA_OK) return st;
    if (!(eps >= 0.f)) return fail(GLA_ERR_INVALID_ARG, "eps must be >= 0");
    if (group != 0 && group != 32 && group != 64 && group != 128)
        return fail(GLA_ERR_UNSUPPORTED, "group %d is not 0, 32, 64 or 128", group);
    OPTIONAL_PTR(res, "res");
    OPTIONAL_PTR(w, "w");
    OPTIONAL_PTR(s_out, "s_out");
    OPTIONAL_PTR(y, "y");
    OPTIONAL_PTR(y8, "y8");
    OPTIONAL_PTR(scale, "scale");
    if ((y8 != nullptr) != (scale != nullptr)) return fail(GLA_ERR_INVALID_ARG, "y8 and scale come together");
    if (rows == 0 || (!s_out && !y && !y8)) return GLA_OK;
    REQUIRE_PTR(x, "x");
    for (const void *out : {(const void *)y, (const void *)y8})
        if (out && (out == x || out == res || out == s_out)) return fail(GLA_ERR_INVALID_ARG, "y and y8 may not alias x, res or s_out");
    if (y && y == y8) return fail(GLA_ERR_INVALID_ARG, "y8 may not alias y");
    NormParams p{x, res, w, eps, (long)rows, D, group, s_out, y, static_cast<unsigned char *>(y8), scale};
    int launches = 0;
    const cudaError_t e = launch_rmsnorm_fwd(p, dtype == GLA_BF16, static_cast<cudaStream_t>(stream), &launches);
    t_launches = launches;
    return e == cudaSuccess ? GLA_OK : cuda_fail(e, "gla_rmsnorm_fwd launch");
}

size_t gla_rmsnorm_bwd_workspace_size(int64_t rows, int D, gla_dtype dtype) {
    if (check_norm_shape(rows, D, dtype) != GLA_OK || rows == 0) return 0;
    return (size_t)norm_bwd_grid((long)rows, D) * D * sizeof(float);
}

gla_status gla_rmsnorm_bwd(const void *s_in, const float *w, const void *dy, const void *ds, float eps, int64_t rows,
                           int D, gla_dtype dtype, void *dx, float *dw, void *workspace, size_t workspace_bytes,
                           void *stream) {
    t_err[0] = 0;
    t_launches = 0;
    gla_status st = check_norm_shape(rows, D, dtype);
    if (st != GLA_OK) return st;
    if (!(eps >= 0.f)) return fail(GLA_ERR_INVALID_ARG, "eps must be >= 0");
    OPTIONAL_PTR(w, "w");
    OPTIONAL_PTR(ds, "ds");
    OPTIONAL_PTR(dw, "dw");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int launches = 0;
    if (rows == 0) {
        const cudaError_t e = dw ? cudaMemsetAsync(dw, 0, (size_t)D * sizeof(float), s) : cudaSuccess;
        return e == cudaSuccess ? GLA_OK : cuda_fail(e, "gla_rmsnorm_bwd(rows=0)");
    }
    REQUIRE_PTR(s_in, "s");
    REQUIRE_PTR(dy, "dy");
    REQUIRE_PTR(dx, "dx");
    if (dx == s_in) return fail(GLA_ERR_INVALID_ARG, "dx may not alias s");
    if (dw) {
        REQUIRE_PTR(workspace, "workspace");
        const size_t need = gla_rmsnorm_bwd_workspace_size(rows, D, dtype);
        if (workspace_bytes < need)
            return fail(GLA_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace_bytes);
    }
    NormParams p{s_in, nullptr, w, eps, (long)rows, D, 0, nullptr, nullptr, nullptr, nullptr, dy, ds, dx, dw,
                 dw ? static_cast<float *>(workspace) : nullptr};
    const cudaError_t e = launch_rmsnorm_bwd(p, dtype == GLA_BF16, s, &launches);
    t_launches = launches;
    return e == cudaSuccess ? GLA_OK : cuda_fail(e, "gla_rmsnorm_bwd launch");
}

// The readout of every node of the trees; log_lambda or g.
static gla_status tree_common(const void *q, int64_t ld_q, const void *k, int64_t ld_k, const void *v, int64_t ld_v,
                              const float *log_lambda, const float *g, float scale, const int *cu_nodes,
                              const int *parents, const int *slots, const float *state_pool, int n_slots, int nseq,
                              int total_T, int H, int dk, int dv, gla_dtype dtype, void *o, void *stream) {
    t_err[0] = 0;
    t_launches = 0;
    gla_status st = check_tree_shape(nseq, total_T, H, dk, dv, dtype);
    if (st != GLA_OK) return st;
    if (nseq == 0 || H == 0) return GLA_OK;
    TreeParams p{};
    p.q = q, p.k = k, p.v = v, p.ldq = (long)ld_q, p.ldk = (long)ld_k, p.ldv = (long)ld_v;
    p.log_lambda = log_lambda, p.g = g, p.scale = scale;
    p.cu = cu_nodes, p.parents = parents, p.slots = slots, p.pool = const_cast<float *>(state_pool);
    p.n_slots = n_slots, p.nseq = nseq, p.total_T = total_T, p.H = H, p.dk = dk, p.dv = dv, p.o = o;
    if ((st = check_trees(p)) != GLA_OK) return st;
    if (total_T == 0) return GLA_OK;
    REQUIRE_PTR(state_pool, "state_pool");
    OPTIONAL_INTS(log_lambda, "log_lambda");
    OPTIONAL_INTS(g, "g");
    if ((st = check_heads(q, ld_q, H, dk, dtype, "q")) != GLA_OK) return st;
    if ((st = check_heads(k, ld_k, H, dk, dtype, "k")) != GLA_OK) return st;
    if ((st = check_heads(v, ld_v, H, dv, dtype, "v")) != GLA_OK) return st;
    REQUIRE_PTR(o, "o");
    if (o == q || o == k || o == v || o == state_pool) return fail(GLA_ERR_INVALID_ARG, "o may not alias an input");
    if (dtype == GLA_BF16 && (long double)n_slots * H * dk > 2147483647.0L)   // the copies' row numbers are ints
        return fail(GLA_ERR_UNSUPPORTED, "a pool of %d slots with %d heads is too large", n_slots, H);
    if ((st = status_word(&p.status)) != GLA_OK) return st;
    int launches = 0;
    const cudaError_t e = launch_tree_fwd(p, dtype == GLA_BF16, static_cast<cudaStream_t>(stream), &launches);
    t_launches = launches;
    return e == cudaSuccess ? GLA_OK : cuda_fail(e, "gla_tree_fwd launch");
}

gla_status gla_tree_fwd(const void *q, int64_t ld_q, const void *k, int64_t ld_k, const void *v, int64_t ld_v,
                        const float *log_lambda, float scale, const int *cu_nodes, const int *parents,
                        const int *slots, const float *state_pool, int n_slots, int nseq, int total_T, int H, int dk,
                        int dv, gla_dtype dtype, void *o, void *stream) {
    if (nseq > 0 && H > 0 && total_T > 0 && !log_lambda) {
        reset_call_state();
        return fail(GLA_ERR_INVALID_ARG, "log_lambda is NULL");
    }
    return tree_common(q, ld_q, k, ld_k, v, ld_v, log_lambda, nullptr, scale, cu_nodes, parents, slots, state_pool,
                       n_slots, nseq, total_T, H, dk, dv, dtype, o, stream);
}

gla_status gla_tree_fwd_gated(const void *q, int64_t ld_q, const void *k, int64_t ld_k, const void *v, int64_t ld_v,
                              const float *g, float scale, const int *cu_nodes, const int *parents, const int *slots,
                              const float *state_pool, int n_slots, int nseq, int total_T, int H, int dk, int dv,
                              gla_dtype dtype, void *o, void *stream) {
    if (nseq > 0 && H > 0 && total_T > 0 && !g) {
        reset_call_state();
        return fail(GLA_ERR_INVALID_ARG, "g is NULL");
    }
    return tree_common(q, ld_q, k, ld_k, v, ld_v, nullptr, g, scale, cu_nodes, parents, slots, state_pool, n_slots,
                       nseq, total_T, H, dk, dv, dtype, o, stream);
}

// The accepted paths, kept; log_lambda or g.
static gla_status commit_common(const void *k, int64_t ld_k, const void *v, int64_t ld_v, const float *log_lambda,
                                const float *g, const int *cu_nodes, const int *parents, const int *last,
                                const int *slots, float *state_pool, const void *x, int64_t ld_x, float *win_pool,
                                int n_slots, int nseq, int total_T, int H, int dk, int dv, int D, gla_dtype dtype,
                                void *stream) {
    t_err[0] = 0;
    t_launches = 0;
    gla_status st = check_tree_shape(nseq, total_T, H, dk, dv, dtype);
    if (st != GLA_OK) return st;
    if ((x != nullptr) != (win_pool != nullptr)) return fail(GLA_ERR_INVALID_ARG, "x and win_pool come together");
    if (x && (st = check_conv_shape(1, total_T, D, dtype)) != GLA_OK) return st;
    if (nseq == 0) return GLA_OK;
    TreeParams p{};
    p.k = k, p.v = v, p.ldk = (long)ld_k, p.ldv = (long)ld_v, p.log_lambda = log_lambda, p.g = g;
    p.cu = cu_nodes, p.parents = parents, p.slots = slots, p.last = last, p.pool = state_pool;
    p.n_slots = n_slots, p.nseq = nseq, p.total_T = total_T, p.H = H, p.dk = dk, p.dv = dv;
    p.x = x, p.ldx = (long)ld_x, p.win = win_pool, p.D = x ? D : 0;
    if ((st = check_trees(p)) != GLA_OK) return st;
    REQUIRE_INTS(last, "last");
    if (total_T == 0) return GLA_OK;   // every tree is empty: nothing to keep
    if (H > 0) {
        REQUIRE_PTR(state_pool, "state_pool");
        if ((st = check_heads(k, ld_k, H, dk, dtype, "k")) != GLA_OK) return st;
        if ((st = check_heads(v, ld_v, H, dv, dtype, "v")) != GLA_OK) return st;
        REQUIRE_INTS(g ? g : log_lambda, "the decay (log_lambda or g)");
    }
    if (x) {
        if ((st = check_rows(x, ld_x, D, dtype == GLA_BF16 ? 2 : 4, true, "x")) != GLA_OK) return st;
        REQUIRE_PTR(win_pool, "win_pool");
    }
    if (H == 0 && !x) return GLA_OK;
    if ((long double)nseq * ((long double)H + D) > 2147483647.0L) return fail(GLA_ERR_INVALID_ARG, "nseq*(H+D) too large");
    if ((st = status_word(&p.status)) != GLA_OK) return st;
    int launches = 0;
    const cudaError_t e = launch_tree_commit(p, dtype == GLA_BF16, static_cast<cudaStream_t>(stream), &launches);
    t_launches = launches;
    return e == cudaSuccess ? GLA_OK : cuda_fail(e, "gla_tree_commit launch");
}

gla_status gla_tree_commit(const void *k, int64_t ld_k, const void *v, int64_t ld_v, const float *log_lambda,
                           const int *cu_nodes, const int *parents, const int *last, const int *slots,
                           float *state_pool, const void *x, int64_t ld_x, float *win_pool, int n_slots, int nseq,
                           int total_T, int H, int dk, int dv, int D, gla_dtype dtype, void *stream) {
    return commit_common(k, ld_k, v, ld_v, log_lambda, nullptr, cu_nodes, parents, last, slots, state_pool, x, ld_x,
                         win_pool, n_slots, nseq, total_T, H, dk, dv, D, dtype, stream);
}

gla_status gla_tree_commit_gated(const void *k, int64_t ld_k, const void *v, int64_t ld_v, const float *g,
                                 const int *cu_nodes, const int *parents, const int *last, const int *slots,
                                 float *state_pool, const void *x, int64_t ld_x, float *win_pool, int n_slots,
                                 int nseq, int total_T, int H, int dk, int dv, int D, gla_dtype dtype, void *stream) {
    return commit_common(k, ld_k, v, ld_v, nullptr, g, cu_nodes, parents, last, slots, state_pool, x, ld_x, win_pool,
                         n_slots, nseq, total_T, H, dk, dv, D, dtype, stream);
}

gla_status gla_conv1d_tree(const void *x, int64_t ld_x, const float *w, const float *b, const int *cu_nodes,
                           const int *parents, const int *slots, const float *win_pool, int n_slots, int nseq,
                           int total_T, int D, gla_dtype dtype, void *y, void *stream) {
    t_err[0] = 0;
    t_launches = 0;
    gla_status st = check_conv_shape(1, total_T, D, dtype);   // (the trees are packed: total_T rows in all)
    if (st != GLA_OK) return st;
    if (nseq < 0) return fail(GLA_ERR_INVALID_ARG, "negative nseq=%d", nseq);
    OPTIONAL_PTR(b, "b");
    if (nseq == 0) return GLA_OK;
    TreeParams p{};
    p.cu = cu_nodes, p.parents = parents, p.slots = slots, p.n_slots = n_slots, p.nseq = nseq, p.total_T = total_T;
    p.x = x, p.ldx = (long)ld_x, p.w = w, p.b = b, p.win = const_cast<float *>(win_pool), p.D = D, p.y = y;
    if ((st = check_trees(p)) != GLA_OK) return st;
    if (total_T == 0) return GLA_OK;
    if ((st = check_rows(x, ld_x, D, dtype == GLA_BF16 ? 2 : 4, true, "x")) != GLA_OK) return st;
    REQUIRE_PTR(w, "w");
    REQUIRE_PTR(win_pool, "win_pool");
    REQUIRE_PTR(y, "y");
    if (y == x || y == win_pool) return fail(GLA_ERR_INVALID_ARG, "y may not alias x or the windows");
    if ((long double)nseq * D > 2147483647.0L) return fail(GLA_ERR_INVALID_ARG, "nseq*D too large");
    if ((st = status_word(&p.status)) != GLA_OK) return st;
    int launches = 0;
    const cudaError_t e = launch_conv_tree(p, dtype == GLA_BF16, static_cast<cudaStream_t>(stream), &launches);
    t_launches = launches;
    return e == cudaSuccess ? GLA_OK : cuda_fail(e, "gla_conv1d_tree launch");
}

// n page numbers of pools: copied from src, or (src NULL) cleared.
static gla_status pages_common(void *const *pools, const int64_t *page_bytes, int n_pools, int n_slots, bool copy,
                               const int *src, const int *dst, int n, const char *name, void *stream) {
    t_err[0] = 0;
    t_launches = 0;
    PageParams p{};
    gla_status st = check_pools(p, pools, page_bytes, n_pools, n_slots);
    if (st != GLA_OK) return st;
    if (n < 0) return fail(GLA_ERR_INVALID_ARG, "negative n=%d", n);
    if (n == 0 || n_pools == 0) return GLA_OK;
    if (copy) REQUIRE_INTS(src, "src");
    REQUIRE_INTS(dst, copy ? "dst" : "slots");
    p.n = n, p.src = copy ? src : nullptr, p.dst = dst;
    if ((st = status_word(&p.status)) != GLA_OK) return st;
    int launches = 0;
    const cudaError_t e = launch_pages_move(p, static_cast<cudaStream_t>(stream), &launches);
    t_launches = launches;
    return e == cudaSuccess ? GLA_OK : cuda_fail(e, name);
}

gla_status gla_pages_copy(void *const *pools, const int64_t *page_bytes, int n_pools, int n_slots, const int *src,
                          const int *dst, int n, void *stream) {
    return pages_common(pools, page_bytes, n_pools, n_slots, true, src, dst, n, "gla_pages_copy launch", stream);
}

gla_status gla_pages_clear(void *const *pools, const int64_t *page_bytes, int n_pools, int n_slots, const int *slots,
                           int n, void *stream) {
    return pages_common(pools, page_bytes, n_pools, n_slots, false, nullptr, slots, n, "gla_pages_clear launch", stream);
}

size_t gla_pages_compact_workspace_size(int n_slots) {
    return n_slots < 0 || !pages_plan_listed(n_slots) ? 0 : (size_t)(2 * ((long)n_slots / 2 + 1) + 1) * sizeof(int);
}

gla_status gla_pages_compact(void *const *pools, const int64_t *page_bytes, int n_pools, int n_slots,
                             const unsigned char *live, int *map, int *count, void *workspace, size_t workspace_bytes,
                             void *stream) {
    t_err[0] = 0;
    t_launches = 0;
    PageParams p{};
    gla_status st = check_pools(p, pools, page_bytes, n_pools, n_slots);
    if (st != GLA_OK) return st;
    REQUIRE_INTS(count, "count");
    if (n_slots > 0) {
        if (!live) return fail(GLA_ERR_INVALID_ARG, "live is NULL");
        REQUIRE_INTS(map, "map");
    }
    const size_t need = gla_pages_compact_workspace_size(n_slots);
    if (need > 0) {
        REQUIRE_INTS(workspace, "workspace");
        if (workspace_bytes < need)
            return fail(GLA_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace_bytes);
    }
    p.live = live, p.map = map, p.count = count, p.moves = static_cast<int *>(workspace);
    if ((st = status_word(&p.status)) != GLA_OK) return st;
    int launches = 0;
    const cudaError_t e = launch_pages_compact(p, static_cast<cudaStream_t>(stream), &launches);
    t_launches = launches;
    return e == cudaSuccess ? GLA_OK : cuda_fail(e, "gla_pages_compact launch");
}

gla_status gla_layernorm_fwd(const void *x, const void *res, const float *w, const float *b, float eps, int64_t rows,
                             int D, gla_dtype dtype, void *s_out, void *y, void *stream) {
    t_err[0] = 0;
    t_launches = 0;
    gla_status st = check_norm_shape(rows, D, dtype);
    if (st != GLA_OK) return st;
    if (!(eps >= 0.f)) return fail(GLA_ERR_INVALID_ARG, "eps must be >= 0");
    OPTIONAL_PTR(res, "res");
    OPTIONAL_PTR(w, "w");
    OPTIONAL_PTR(b, "b");
    OPTIONAL_PTR(s_out, "s_out");
    if (rows == 0) return GLA_OK;
    REQUIRE_PTR(x, "x");
    REQUIRE_PTR(y, "y");
    if (y == x || y == res || y == s_out) return fail(GLA_ERR_INVALID_ARG, "y may not alias x, res or s_out");
    LayerNormParams p{x, res, w, b, eps, (long)rows, D, s_out, y};
    int launches = 0;
    const cudaError_t e = launch_layernorm_fwd(p, dtype == GLA_BF16, static_cast<cudaStream_t>(stream), &launches);
    t_launches = launches;
    return e == cudaSuccess ? GLA_OK : cuda_fail(e, "gla_layernorm_fwd launch");
}

size_t gla_layernorm_bwd_workspace_size(int64_t rows, int D, gla_dtype dtype) {
    if (check_norm_shape(rows, D, dtype) != GLA_OK || rows == 0) return 0;
    return (size_t)layernorm_bwd_grid((long)rows, D) * 2 * D * sizeof(float);
}

gla_status gla_layernorm_bwd(const void *s_in, const float *w, const void *dy, const void *ds, float eps, int64_t rows,
                             int D, gla_dtype dtype, void *dx, float *dw, float *db, void *workspace,
                             size_t workspace_bytes, void *stream) {
    t_err[0] = 0;
    t_launches = 0;
    gla_status st = check_norm_shape(rows, D, dtype);
    if (st != GLA_OK) return st;
    if (!(eps >= 0.f)) return fail(GLA_ERR_INVALID_ARG, "eps must be >= 0");
    OPTIONAL_PTR(w, "w");
    OPTIONAL_PTR(ds, "ds");
    OPTIONAL_PTR(dw, "dw");
    OPTIONAL_PTR(db, "db");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int launches = 0;
    if (rows == 0) {
        cudaError_t e = dw ? cudaMemsetAsync(dw, 0, (size_t)D * sizeof(float), s) : cudaSuccess;
        if (e == cudaSuccess && db) e = cudaMemsetAsync(db, 0, (size_t)D * sizeof(float), s);
        return e == cudaSuccess ? GLA_OK : cuda_fail(e, "gla_layernorm_bwd(rows=0)");
    }
    REQUIRE_PTR(s_in, "s");
    REQUIRE_PTR(dy, "dy");
    REQUIRE_PTR(dx, "dx");
    if (dx == s_in) return fail(GLA_ERR_INVALID_ARG, "dx may not alias s");
    const bool sums = dw || db;
    if (sums) {
        REQUIRE_PTR(workspace, "workspace");
        const size_t need = gla_layernorm_bwd_workspace_size(rows, D, dtype);
        if (workspace_bytes < need)
            return fail(GLA_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace_bytes);
    }
    LayerNormParams p{s_in, nullptr, w, nullptr, eps, (long)rows, D, nullptr, nullptr, dy, ds, dx, dw, db,
                      sums ? static_cast<float *>(workspace) : nullptr};
    const cudaError_t e = launch_layernorm_bwd(p, dtype == GLA_BF16, s, &launches);
    t_launches = launches;
    return e == cudaSuccess ? GLA_OK : cuda_fail(e, "gla_layernorm_bwd launch");
}

gla_status gla_selftest_wait_timeout(unsigned int limit_us, int *result, void *stream) {
    t_err[0] = 0;
    t_launches = 0;
    if (limit_us == 0 || limit_us > 1000000u) return fail(GLA_ERR_INVALID_ARG, "limit_us must be in 1..1000000");
    REQUIRE_PTR(result, "result");
    unsigned int *status = nullptr;
    gla_status st = status_word(&status);
    if (st != GLA_OK) return st;
    int launches = 0;
    const cudaError_t e = launch_selftest_wait(status, (uint64_t)limit_us * 1000u, result,
                                               static_cast<cudaStream_t>(stream), &launches);
    t_launches = launches;
    return e == cudaSuccess ? GLA_OK : cuda_fail(e, "gla_selftest_wait_timeout launch");
}

gla_status gla_check(void *stream) {
    t_err[0] = 0;
    cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "cudaStreamSynchronize");
    e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "earlier launch");
    unsigned int word = 0;
    e = cudaMemcpyFromSymbol(&word, g_status_word, sizeof word);
    if (e != cudaSuccess) return cuda_fail(e, "read status word");
    if (word != 0) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_status_word, &zero, sizeof zero);
        if (e != cudaSuccess) return cuda_fail(e, "clear status word");
        if (word & kDevTimeout) return fail(GLA_ERR_TIMEOUT, "a device-side wait timed out (status 0x%x)", word);
        if (word & kDevBadState)
            return fail(GLA_ERR_INVALID_ARG, "a sequence had a bad cu_seqlens or slots entry (or a tree's offset, parent "
                                             "or accepted node, or a page number) and was skipped (status 0x%x)", word);
        return fail(GLA_ERR_CUDA, "device reported an internal error (status 0x%x)", word);
    }
    return GLA_OK;
}

const char *gla_status_string(gla_status status) {
    switch (status) {
    case GLA_OK: return "GLA_OK";
    case GLA_ERR_INVALID_ARG: return "GLA_ERR_INVALID_ARG";
    case GLA_ERR_UNSUPPORTED: return "GLA_ERR_UNSUPPORTED";
    case GLA_ERR_CUDA: return "GLA_ERR_CUDA";
    case GLA_ERR_TIMEOUT: return "GLA_ERR_TIMEOUT";
    case GLA_ERR_WORKSPACE: return "GLA_ERR_WORKSPACE";
    }
    return "GLA_ERR_UNKNOWN";
}

const char *gla_last_error(void) { return t_err; }

int gla_last_launch_count(void) { return t_launches; }

const char *gla_version(void) { return "libgla 0.1.0 sm_103a"; }

}  // extern "C"
