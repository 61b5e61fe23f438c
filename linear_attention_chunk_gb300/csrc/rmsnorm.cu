// rmsnorm.cu -- the norm in front of a mixer layer, with the residual's
// addition before it and an 8-bit output behind it, and its gradients:
//     s = x + res,   y = s w / sqrt(mean(s^2) + eps)       per row of D channels
//     scale = max |y| / 448 over the row or a block of channels,  y8 = e4m3(y / scale)
// and, with xn = s / sqrt(mean(s^2) + eps) and g = dy w,
//     dx = ds + (g - xn mean(g xn)) / sqrt(mean(s^2) + eps),  dw = sum over rows of dy xn.
//
// Streams over HBM: forward 7 bytes an element (bf16 x and res in, s and e4m3
// out), backward 8. A CTA walks every G-th row, the rows ahead of it arriving
// by asynchronous copies (a thread copies and reads its own vectors of eight
// channels); one row ahead in registers kept too few bytes in flight (backward
// 63 us at 16384 x 2048, now 46, 0.85 of the measured copy rate; forward with
// 8-bit output at 16384 x 4096 86, now 75, 0.93). A row's sums
// go through shuffles and one shared-memory exchange. A block of 128, 64 or 32
// channels is 16, 8 or 4 neighbouring lanes, so its maximum needs shuffles
// only. w, and the backward's dw, of a thread's channels stay in registers; the
// CTAs' partial sums of dw are added in a second launch (reduce.cu).
// y is rounded once from fp32; y8 from the unrounded y.
#include "ssm_common.cuh"

namespace gla {
namespace {

using ssm::Raw8;
using ssm::copies_commit;
using ssm::copies_wait;
using ssm::copy_async;
using ssm::param8;
using ssm::raw_load;
using ssm::raw_unpack;
using ssm::raw_zero;
using ssm::store8;

constexpr float kTop = 448.f;   // the largest e4m3 value
constexpr int kMost = 512;      // threads of a CTA, two vectors a thread: D <= 8192

__device__ __forceinline__ float max_nan(float a, float b) {   // a NaN wins
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}
__device__ __forceinline__ float lanes_max(float v, int lanes) {
    for (int off = lanes / 2; off > 0; off >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
}

// Eight values over `inv` as e4m3, stored.
template <typename T> __device__ __forceinline__ void store_e4m3(unsigned char *dst, const float (&v)[8], float inv, bool whole) {
    uint32_t *o = reinterpret_cast<uint32_t *>(dst);
    const uint32_t a = e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
    const uint32_t b = e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
    if (sizeof(T) == 2) {
        *reinterpret_cast<uint2 *>(o) = make_uint2(a, b);
    } else {
        o[0] = a;
        if (whole) o[1] = b;
    }
}
__device__ __forceinline__ float scale_of(float top) { return top == 0.f ? 1.f : max_nan(top / kTop, 1.17549435e-38f); }

// Rows in the forward's ring, and its threads on an SM (16384 x 4096 with 8-bit output, rows 2, 3, 4 at 768
// threads: 75, 78, 81 us; at 1,024: 77, 87, 85).
constexpr int kFwdRows = 2, kFwdThreads = 768;

// Rows blockIdx.x, + gridDim.x, ...
template <typename T, int VPT> __global__ void __launch_bounds__(kMost) rmsnorm_fwd_kernel(const NormParams p) {
    extern __shared__ __align__(16) uint4 ring[];       // kFwdRows rows of x and res; a thread copies and reads its own
    __shared__ float s_sum[2][32], s_max[2][32];
    constexpr int H = sizeof(T) / 2, kRow = 2 * VPT * H;   // 16-byte pieces of a thread and row
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, nw = blockDim.x / 32;
    const int groups = p.group ? (p.D + p.group - 1) / p.group : 1;
    auto issue = [&](long row, int stage) {
        uint4 *dst = ring + (size_t)stage * kRow * blockDim.x + tid;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (i * (int)blockDim.x + tid) * 8;
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const bool in = row < p.rows && c + 4 * h < p.D;
                const size_t at = in ? (size_t)row * p.D + c + 4 * h : 0;
                copy_async<16>(dst + (2 * i * H + h) * blockDim.x, static_cast<const T *>(p.x) + at, in);
                if (p.res) copy_async<16>(dst + ((2 * i + 1) * H + h) * blockDim.x, static_cast<const T *>(p.res) + at, in);
            }
        }
        copies_commit();
    };
    auto held = [&](int stage, int k) {
        Raw8<T> r;
#pragma unroll
        for (int h = 0; h < H; ++h) r.w[h] = ring[((size_t)stage * kRow + k * H + h) * blockDim.x + tid];
        return r;
    };
    long row = blockIdx.x;
#pragma unroll
    for (int k = 0; k < kFwdRows - 1; ++k) issue(row + (long)k * gridDim.x, k);
    float w[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (i * (int)blockDim.x + tid) * 8;
        param8(p.w && c < p.D ? p.w : nullptr, c, c + 8 <= p.D, w[i]);
        if (!p.w)
#pragma unroll
            for (int j = 0; j < 8; ++j) w[i][j] = 1.f;
    }
    int par = 0, stage = 0;
    for (; row < p.rows; row += gridDim.x, par ^= 1) {
        copies_wait<kFwdRows - 2>();
        float v[VPT][8], ss = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            raw_unpack(held(stage, 2 * i), v[i]);
            if (p.res) {
                float r[8];
                raw_unpack(held(stage, 2 * i + 1), r);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] += r[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
        }
        issue(row + (long)(kFwdRows - 1) * gridDim.x, stage == 0 ? kFwdRows - 1 : stage - 1);   // the row before's stage
        stage = stage == kFwdRows - 1 ? 0 : stage + 1;
        ss = warp_sum(ss);
        if (nw > 1) {                                   // two buffers in turn: one barrier a sum
            if (lane == 0) s_sum[par][warp] = ss;
            __syncthreads();
            ss = warp_sum(lane < nw ? s_sum[par][lane] : 0.f);
        }
        const float rinv = rsqrtf(ss / (float)p.D + p.eps);
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (i * (int)blockDim.x + tid) * 8;
            const bool on = c < p.D, whole = c + 8 <= p.D;
            const size_t at = (size_t)row * p.D + c;
            if (p.s_out && on) store8(static_cast<T *>(p.s_out) + at, v[i], whole);
            float m = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[i][j] = on ? v[i][j] * rinv * w[i][j] : 0.f;   // (a lane past the end: its zeros, also where rinv is NaN)
                m = max_nan(m, fabsf(v[i][j]));
            }
            if (p.y && on) store8(static_cast<T *>(p.y) + at, v[i], whole);
            if (p.y8 && p.group) {
                const float scale = scale_of(lanes_max(m, p.group / 8));
                if (on && lane % (p.group / 8) == 0) p.scale[(size_t)row * groups + c / p.group] = scale;
                if (on) store_e4m3<T>(p.y8 + at, v[i], 1.f / scale, whole);
            }
            top = max_nan(top, m);
        }
        if (!p.y8 || p.group) continue;
        top = lanes_max(top, 32);
        if (nw > 1) {
            if (lane == 0) s_max[par][warp] = top;
            __syncthreads();
            top = lanes_max(lane < nw ? s_max[par][lane] : 0.f, 32);
        }
        const float scale = scale_of(top), inv = 1.f / scale;
        if (tid == 0) p.scale[row] = scale;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (i * (int)blockDim.x + tid) * 8;
            if (c < p.D) store_e4m3<T>(p.y8 + (size_t)row * p.D + c, v[i], inv, c + 8 <= p.D);
        }
    }
}

// Rows in the backward's ring (2, 3, 4, 6 measured: 57, 51, 55, 58 us at 16384 x 2048); two where three
// would not fit (fp32, D > 4096: 98 KB a row).
template <typename T, int VPT> constexpr int ring_rows() { return sizeof(T) == 4 && VPT == 2 ? 2 : 3; }

// p.x: s; rows blockIdx.x, + gridDim.x, ...; partial dw of the CTA at p.part.
template <typename T, int VPT> __global__ void __launch_bounds__(kMost) rmsnorm_bwd_kernel(const NormParams p) {
    constexpr int kStages = ring_rows<T, VPT>();
    __shared__ float2 s_red[2][32];
    ssm::let_next_start();
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, nw = blockDim.x / 32;
    // the ring: kStages rows of s, dy, ds; a thread copies and reads its own vectors
    extern __shared__ __align__(16) uint4 ring[];
    constexpr int H = sizeof(T) / 2, kRow = 3 * VPT * H;   // 16-byte pieces of a thread and row
    auto issue = [&](long row, int stage) {
        uint4 *dst = ring + (size_t)stage * kRow * blockDim.x + tid;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (i * (int)blockDim.x + tid) * 8;
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const bool in = row < p.rows && c + 4 * h < p.D;   // (a piece holds 8 / H channels)
                const size_t at = in ? (size_t)row * p.D + c + 4 * h : 0;
                copy_async<16>(dst + ((3 * i) * H + h) * blockDim.x, static_cast<const T *>(p.x) + at, in);
                copy_async<16>(dst + ((3 * i + 1) * H + h) * blockDim.x, static_cast<const T *>(p.dy) + at, in);
                copy_async<16>(dst + ((3 * i + 2) * H + h) * blockDim.x,
                               static_cast<const T *>(p.ds ? p.ds : p.x) + at, in && p.ds);
            }
        }
    };
    auto held = [&](int stage, int k) {
        Raw8<T> r;
#pragma unroll
        for (int h = 0; h < H; ++h) r.w[h] = ring[((size_t)stage * kRow + k * H + h) * blockDim.x + tid];
        return r;
    };
    float w[VPT][8], dw[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (i * (int)blockDim.x + tid) * 8;
        param8(p.w && c < p.D ? p.w : nullptr, c, c + 8 <= p.D, w[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (!p.w) w[i][j] = 1.f;
            dw[i][j] = 0.f;
        }
    }
    int par = 0, stage = 0;
    long row = blockIdx.x;
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) {
        issue(row + (long)k * gridDim.x, k);
        copies_commit();
    }
    for (; row < p.rows; row += gridDim.x, par ^= 1) {
        copies_wait<kStages - 2>();
        Raw8<T> cx[VPT], cy[VPT], cs[VPT];
        float ss = 0.f, sg = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            cx[i] = held(stage, 3 * i);
            cy[i] = held(stage, 3 * i + 1);
            cs[i] = held(stage, 3 * i + 2);
            float x[8], g[8];
            raw_unpack(cx[i], x);
            raw_unpack(cy[i], g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                ss = fmaf(x[j], x[j], ss);
                sg = fmaf(g[j] * w[i][j], x[j], sg);
            }
        }
        issue(row + (long)(kStages - 1) * gridDim.x, stage == 0 ? kStages - 1 : stage - 1);   // the row before's stage
        copies_commit();
        stage = stage == kStages - 1 ? 0 : stage + 1;
        ss = warp_sum(ss);
        sg = warp_sum(sg);
        if (nw > 1) {                                // two buffers in turn: one barrier a row
            if (lane == 0) s_red[par][warp] = make_float2(ss, sg);
            __syncthreads();
            const float2 r = lane < nw ? s_red[par][lane] : make_float2(0.f, 0.f);
            ss = warp_sum(r.x);
            sg = warp_sum(r.y);
        }
        const float rinv = rsqrtf(ss / (float)p.D + p.eps);
        const float k = rinv * rinv * (sg / (float)p.D);   // xn mean(g xn) = x k
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (i * (int)blockDim.x + tid) * 8;
            float x[8], g[8], s[8];
            raw_unpack(cx[i], x);
            raw_unpack(cy[i], g);
            raw_unpack(cs[i], s);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                dw[i][j] = fmaf(g[j], x[j] * rinv, dw[i][j]);
                s[j] = fmaf(rinv, fmaf(-k, x[j], g[j] * w[i][j]), s[j]);
            }
            if (c < p.D) store8(static_cast<T *>(p.dx) + (size_t)row * p.D + c, s, c + 8 <= p.D);
        }
    }
    if (!p.part) return;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (i * (int)blockDim.x + tid) * 8;
        if (c < p.D) store8(p.part + (size_t)blockIdx.x * p.D + c, dw[i], c + 8 <= p.D);
    }
}

int round32(int v) { return (v + 31) / 32 * 32; }

// More than the default 48 KB (1 KB of them for the kernels' own arrays) has to be asked for.
template <typename K> cudaError_t allow_smem(K *kern, int bytes) {
    if (bytes <= 47 * 1024) return cudaSuccess;
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <typename T> cudaError_t fwd(const NormParams &p, cudaStream_t s, int *launches) {
    const int vecs = (p.D + 7) / 8;
    // Few rows: one vector a thread, the shortest chain. Many: two, so that a
    // row has half the warps to exchange with.
    const int vpt = vecs > kMost || (p.rows > 2L * device_sm_count() && vecs > 32) ? 2 : 1;
    const int th = round32((vecs + vpt - 1) / vpt);
    const long held = (long)(kFwdThreads / th > 16 ? 16 : kFwdThreads / th) * device_sm_count();
    const int bytes = kFwdRows * 2 * vpt * th * 8 * (int)sizeof(T);
    auto *kern = vpt == 1 ? rmsnorm_fwd_kernel<T, 1> : rmsnorm_fwd_kernel<T, 2>;
    cudaError_t e = allow_smem(kern, bytes);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)(p.rows < held ? p.rows : held), th, bytes, s>>>(p);
    if (launches) ++*launches;
    return cudaGetLastError();
}

// The backward's shape by D alone: one vector a thread up to 4,096 channels.
int bwd_vpt(int vecs) { return vecs > kMost ? 2 : 1; }
int bwd_threads(int vecs) { return round32((vecs + bwd_vpt(vecs) - 1) / bwd_vpt(vecs)); }

template <typename T> cudaError_t bwd(const NormParams &p, cudaStream_t s, int *launches) {
    const int vecs = (p.D + 7) / 8, vpt = bwd_vpt(vecs), th = bwd_threads(vecs);
    const unsigned grid = (unsigned)norm_bwd_grid(p.rows, p.D);
    const int bytes = (vpt == 1 ? ring_rows<T, 1>() : ring_rows<T, 2>()) * 3 * vpt * th * 8 * (int)sizeof(T);
    auto *kern = vpt == 1 ? rmsnorm_bwd_kernel<T, 1> : rmsnorm_bwd_kernel<T, 2>;
    cudaError_t e = allow_smem(kern, bytes);
    if (e != cudaSuccess) return e;
    kern<<<grid, th, bytes, s>>>(p);
    if (launches) ++*launches;
    e = cudaGetLastError();
    if (e != cudaSuccess || !p.part) return e;
    SumJobs sums;
    sums.add(p.part, grid, p.D, p.D, p.dw);
    return launch_sums(sums, s, launches);
}

}  // namespace

// CTAs of the backward: 768 threads an SM, each CTA walking its share of the rows.
long norm_bwd_grid(long rows, int D) {
    const int th = bwd_threads((D + 7) / 8);
    const long per_sm = 768 / th > 8 ? 8 : 768 / th;
    const long most = per_sm * device_sm_count();
    return rows < most ? rows : most;
}

cudaError_t launch_rmsnorm_fwd(const NormParams &p, bool bf16, cudaStream_t s, int *launches) {
    return bf16 ? fwd<__nv_bfloat16>(p, s, launches) : fwd<float>(p, s, launches);
}
cudaError_t launch_rmsnorm_bwd(const NormParams &p, bool bf16, cudaStream_t s, int *launches) {
    return bf16 ? bwd<__nv_bfloat16>(p, s, launches) : bwd<float>(p, s, launches);
}

}  // namespace gla
