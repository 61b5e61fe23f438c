// layernorm.cu -- the layer norm in front of a layer, with the residual's
// addition before it, and its gradients, per row of D channels:
//     s = x + res,   c = s - mean(s),   r = 1 / sqrt(mean(c^2) + eps)
//     y = c r w + b
// and, with xn = c r and g = dy w,
//     dx = ds + r (g - mean(g) - xn mean(g xn)),
//     dw = sum over rows of dy xn,   db = sum over rows of dy.
//
// Streams over HBM, 8 bytes an element either way (bf16). A CTA walks every
// G-th row, the rows ahead of it arriving by asynchronous copies (a thread
// copies and reads its own vectors of eight channels). The row stays in
// registers between its two sums: the mean first, then the squares of what is
// left, since mean(s^2) - mean(s)^2 loses what a mean far from 0 leaves. Each
// sum goes through shuffles and one shared-memory exchange. w, b, and the
// backward's dw and db, of a thread's channels stay in registers; the CTAs'
// partial sums are added in a second launch (reduce.cu), in a fixed order.
#include "ssm_common.cuh"

namespace gla {
namespace {

using ssm::Raw8;
using ssm::copies_commit;
using ssm::copies_wait;
using ssm::copy_async;
using ssm::param8;
using ssm::raw_unpack;
using ssm::store8;

constexpr int kMost = 512;      // threads of a CTA, two vectors a thread: D <= 8192

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}
// Sums over the CTA, each thread adding the warps' in order (a second tree of
// shuffles costs more); `s` is not written again before the CTA's next barrier
// but one.
__device__ __forceinline__ float2 block_sums(float a, float b, float4 *s) {   // (two warps' sums an element)
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, nw = blockDim.x / 32;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, off);
        b += __shfl_xor_sync(0xffffffffu, b, off);
    }
    if (nw == 1) return make_float2(a, b);
    if (lane == 0) reinterpret_cast<float2 *>(s)[warp] = make_float2(a, b);
    __syncthreads();
    a = b = 0.f;
    for (int i = 0; i < nw / 2; ++i) {
        const float4 u = s[i];
        a += u.x;
        b += u.y;
        a += u.z;
        b += u.w;
    }
    if (nw & 1) {
        a += s[nw / 2].x;
        b += s[nw / 2].y;
    }
    return make_float2(a, b);
}
__device__ __forceinline__ float block_sum(float a, float4 *s) {   // (four warps' sums an element)
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, nw = blockDim.x / 32;
    a = warp_sum(a);
    if (nw == 1) return a;
    if (lane == 0) reinterpret_cast<float *>(s)[warp] = a;
    __syncthreads();
    a = 0.f;
    for (int i = 0; i < nw / 4; ++i) {
        const float4 u = s[i];
        a += u.x;
        a += u.y;
        a += u.z;
        a += u.w;
    }
    for (int i = nw & ~3; i < nw; ++i) a += reinterpret_cast<const float *>(s)[i];
    return a;
}
// sum / D with inv = 1 / D: one correction, without which a constant row's mean is off by a step.
__device__ __forceinline__ float mean_of(float sum, float D, float inv) {
    const float q = sum * inv;
    return fmaf(fmaf(-q, D, sum), inv, q);
}

// kIn rows of one array each (x, res; s, dy, ds) in a ring of kStages; a thread copies and reads its own vectors.
template <typename T, int VPT, int kIn> struct Ring {
    static constexpr int H = sizeof(T) / 2, kRow = kIn * VPT * H;   // 16-byte pieces of a thread and row
    uint4 *at;
    __device__ __forceinline__ void issue(int stage, int k, int i, const void *src, long row, bool in, int D) const {
        const int c = (i * (int)blockDim.x + (int)threadIdx.x) * 8;
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const bool on = in && c + 4 * h < D;      // (a piece holds 8 / H channels)
            copy_async<16>(at + ((size_t)stage * kRow + (i * kIn + k) * H + h) * blockDim.x + threadIdx.x,
                           static_cast<const T *>(src) + (on ? (size_t)row * D + c + 4 * h : 0), on);
        }
    }
    __device__ __forceinline__ Raw8<T> held(int stage, int k, int i) const {
        Raw8<T> r;
#pragma unroll
        for (int h = 0; h < H; ++h) r.w[h] = at[((size_t)stage * kRow + (i * kIn + k) * H + h) * blockDim.x + threadIdx.x];
        return r;
    }
};

constexpr int kFwdRows = 2, kFwdThreads = 768;   // rows in the forward's ring, its threads on an SM

template <typename T, int VPT> __global__ void __launch_bounds__(kMost) layernorm_fwd_kernel(const LayerNormParams p) {
    extern __shared__ __align__(16) uint4 smem[];
    __shared__ float4 s_a[4], s_b[4];
    const Ring<T, VPT, 2> ring{smem};
    const int tid = threadIdx.x;
    auto issue = [&](long row, int stage) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            ring.issue(stage, 0, i, p.x, row, row < p.rows, p.D);
            if (p.res) ring.issue(stage, 1, i, p.res, row, row < p.rows, p.D);
        }
        copies_commit();
    };
    long row = blockIdx.x;
#pragma unroll
    for (int k = 0; k < kFwdRows - 1; ++k) issue(row + (long)k * gridDim.x, k);
    float w[VPT][8], b[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (i * (int)blockDim.x + tid) * 8;
        const bool on = c < p.D, whole = c + 8 <= p.D;
        param8(p.w && on ? p.w : nullptr, c, whole, w[i]);
        param8(p.b && on ? p.b : nullptr, c, whole, b[i]);
        if (!p.w)
#pragma unroll
            for (int j = 0; j < 8; ++j) w[i][j] = 1.f;
    }
    const float D = (float)p.D, inv = 1.f / D;
    int stage = 0;
    for (; row < p.rows; row += gridDim.x) {
        copies_wait<kFwdRows - 2>();
        float v[VPT][8], sum = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            raw_unpack(ring.held(stage, 0, i), v[i]);
            if (p.res) {
                float r[8];
                raw_unpack(ring.held(stage, 1, i), r);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] += r[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) sum += v[i][j];
        }
        issue(row + (long)(kFwdRows - 1) * gridDim.x, stage == 0 ? kFwdRows - 1 : stage - 1);   // the row before's stage
        stage = stage == kFwdRows - 1 ? 0 : stage + 1;
        const float mean = mean_of(block_sum(sum, s_a), D, inv);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (i * (int)blockDim.x + tid) * 8;
            if (p.s_out && c < p.D) store8(static_cast<T *>(p.s_out) + (size_t)row * p.D + c, v[i], c + 8 <= p.D);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[i][j] = c + j < p.D ? v[i][j] - mean : 0.f;
                ss = fmaf(v[i][j], v[i][j], ss);
            }
        }
        const float r = rsqrtf(block_sum(ss, s_b) * inv + p.eps);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (i * (int)blockDim.x + tid) * 8;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = fmaf(v[i][j] * r, w[i][j], b[i][j]);
            if (c < p.D) store8(static_cast<T *>(p.y) + (size_t)row * p.D + c, v[i], c + 8 <= p.D);
        }
    }
}

// Rows in the backward's ring; two where three would not fit (fp32, D > 4096: 98 KB a row).
template <typename T, int VPT> constexpr int ring_rows() { return sizeof(T) == 4 && VPT == 2 ? 2 : 3; }

// p.x: s; rows blockIdx.x, + gridDim.x, ...; partial dw and db of the CTA at p.part.
template <typename T, int VPT> __global__ void __launch_bounds__(kMost) layernorm_bwd_kernel(const LayerNormParams p) {
    constexpr int kStages = ring_rows<T, VPT>();
    extern __shared__ __align__(16) uint4 smem[];
    __shared__ float4 s_a[8], s_b[8];
    const Ring<T, VPT, 3> ring{smem};
    ssm::let_next_start();
    const int tid = threadIdx.x;
    auto issue = [&](long row, int stage) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            ring.issue(stage, 0, i, p.x, row, row < p.rows, p.D);
            ring.issue(stage, 1, i, p.dy, row, row < p.rows, p.D);
            ring.issue(stage, 2, i, p.ds ? p.ds : p.x, row, row < p.rows && p.ds, p.D);
        }
        copies_commit();
    };
    float w[VPT][8], dw[VPT][8], db[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (i * (int)blockDim.x + tid) * 8;
        param8(p.w && c < p.D ? p.w : nullptr, c, c + 8 <= p.D, w[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (!p.w) w[i][j] = 1.f;
            dw[i][j] = db[i][j] = 0.f;
        }
    }
    const float D = (float)p.D, inv = 1.f / D;
    int stage = 0;
    long row = blockIdx.x;
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) issue(row + (long)k * gridDim.x, k);
    for (; row < p.rows; row += gridDim.x) {
        copies_wait<kStages - 2>();
        float x[VPT][8];
        Raw8<T> cy[VPT], cs[VPT];
        float sx = 0.f, sg = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            cy[i] = ring.held(stage, 1, i);
            cs[i] = ring.held(stage, 2, i);
            float g[8];
            raw_unpack(ring.held(stage, 0, i), x[i]);
            raw_unpack(cy[i], g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                sx += x[i][j];
                sg = fmaf(g[j], w[i][j], sg);
            }
        }
        issue(row + (long)(kStages - 1) * gridDim.x, stage == 0 ? kStages - 1 : stage - 1);   // the row before's stage
        stage = stage == kStages - 1 ? 0 : stage + 1;
        const float2 first = block_sums(sx, sg, s_a);
        const float mean = mean_of(first.x, D, inv), mg = first.y * inv;
        float ss = 0.f, sc = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (i * (int)blockDim.x + tid) * 8;
            float g[8];
            raw_unpack(cy[i], g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[i][j] = c + j < p.D ? x[i][j] - mean : 0.f;
                ss = fmaf(x[i][j], x[i][j], ss);
                sc = fmaf(g[j] * w[i][j], x[i][j], sc);
            }
        }
        const float2 second = block_sums(ss, sc, s_b);
        const float r = rsqrtf(second.x * inv + p.eps);
        const float k = r * r * (second.y * inv);      // xn mean(g xn) = c k
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (i * (int)blockDim.x + tid) * 8;
            float g[8], s[8];
            raw_unpack(cy[i], g);
            raw_unpack(cs[i], s);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                dw[i][j] = fmaf(g[j], x[i][j] * r, dw[i][j]);
                db[i][j] += g[j];
                s[j] = fmaf(r, fmaf(-k, x[i][j], fmaf(g[j], w[i][j], -mg)), s[j]);
            }
            if (c < p.D) store8(static_cast<T *>(p.dx) + (size_t)row * p.D + c, s, c + 8 <= p.D);
        }
    }
    if (!p.part) return;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (i * (int)blockDim.x + tid) * 8;
        if (c >= p.D) continue;
        store8(p.part + (size_t)blockIdx.x * 2 * p.D + c, dw[i], c + 8 <= p.D);
        store8(p.part + (size_t)blockIdx.x * 2 * p.D + p.D + c, db[i], c + 8 <= p.D);
    }
}

int round32(int v) { return (v + 31) / 32 * 32; }

// More than the default 48 KB (1 KB of them for the kernels' own arrays) has to be asked for.
template <typename K> cudaError_t allow_smem(K *kern, int bytes) {
    if (bytes <= 47 * 1024) return cudaSuccess;
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <typename T> cudaError_t fwd(const LayerNormParams &p, cudaStream_t s, int *launches) {
    const int vecs = (p.D + 7) / 8;
    // Few rows: one vector a thread, the shortest chain. Many: two, so that a
    // row has half the warps to exchange with.
    const int vpt = vecs > kMost || (p.rows > 2L * device_sm_count() && vecs > 32) ? 2 : 1;
    const int th = round32((vecs + vpt - 1) / vpt);
    const long held = (long)(kFwdThreads / th > 16 ? 16 : kFwdThreads / th) * device_sm_count();
    const int bytes = kFwdRows * 2 * vpt * th * 8 * (int)sizeof(T);
    auto *kern = vpt == 1 ? layernorm_fwd_kernel<T, 1> : layernorm_fwd_kernel<T, 2>;
    cudaError_t e = allow_smem(kern, bytes);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)(p.rows < held ? p.rows : held), th, bytes, s>>>(p);
    if (launches) ++*launches;
    return cudaGetLastError();
}

// The backward's shape by D alone: one vector a thread up to 4,096 channels.
int bwd_vpt(int vecs) { return vecs > kMost ? 2 : 1; }
int bwd_threads(int vecs) { return round32((vecs + bwd_vpt(vecs) - 1) / bwd_vpt(vecs)); }

template <typename T> cudaError_t bwd(const LayerNormParams &p, cudaStream_t s, int *launches) {
    const int vecs = (p.D + 7) / 8, vpt = bwd_vpt(vecs), th = bwd_threads(vecs);
    const unsigned grid = (unsigned)layernorm_bwd_grid(p.rows, p.D);
    const int bytes = (vpt == 1 ? ring_rows<T, 1>() : ring_rows<T, 2>()) * 3 * vpt * th * 8 * (int)sizeof(T);
    auto *kern = vpt == 1 ? layernorm_bwd_kernel<T, 1> : layernorm_bwd_kernel<T, 2>;
    cudaError_t e = allow_smem(kern, bytes);
    if (e != cudaSuccess) return e;
    kern<<<grid, th, bytes, s>>>(p);
    if (launches) ++*launches;
    e = cudaGetLastError();
    if (e != cudaSuccess || !p.part) return e;
    SumJobs sums;
    sums.add(p.part, grid, p.D, 2L * p.D, p.dw);
    sums.add(p.part + p.D, grid, p.D, 2L * p.D, p.db);
    return launch_sums(sums, s, launches);
}

}  // namespace

// CTAs of the backward: 768 threads an SM, each CTA walking its share of the rows.
long layernorm_bwd_grid(long rows, int D) {
    const int th = bwd_threads((D + 7) / 8);
    const long per_sm = 768 / th > 8 ? 8 : 768 / th;
    const long most = per_sm * device_sm_count();
    return rows < most ? rows : most;
}

cudaError_t launch_layernorm_fwd(const LayerNormParams &p, bool bf16, cudaStream_t s, int *launches) {
    return bf16 ? fwd<__nv_bfloat16>(p, s, launches) : fwd<float>(p, s, launches);
}
cudaError_t launch_layernorm_bwd(const LayerNormParams &p, bool bf16, cudaStream_t s, int *launches) {
    return bf16 ? bwd<__nv_bfloat16>(p, s, launches) : bwd<float>(p, s, launches);
}

}  // namespace gla
