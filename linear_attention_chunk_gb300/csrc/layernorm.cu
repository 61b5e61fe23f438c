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
using ssm::add2;
using ssm::both;
using ssm::f2;
using ssm::f2_pack;
using ssm::f2_split;
using ssm::fma2;
using ssm::mul2;
using ssm::raw_unpack;

constexpr int kMost = 512, kBwdThreads = 512;   // threads of a CTA, two vectors each: D <= 8192; the backward's on an SM

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}
__device__ __forceinline__ float pair_sum(f2 v) {
    const float2 u = f2_split(v);
    return u.x + u.y;
}
// Sums over threads that share a row, each adding the warps' in order; `s` is
// not written again before their next barrier but one. Of two sums, lanes 0 .. 15 take
// on one after the first exchange, 16 .. 31 the other: six exchanges for ten.
__device__ __forceinline__ float2 block_sums(float a, float b, float4 *s) {   // (two warps' sums an element)
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, nw = blockDim.x / 32;
    const bool upper = lane & 16;
    float v = (upper ? b : a) + __shfl_xor_sync(0xffffffffu, upper ? a : b, 16);
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if (nw == 1) {
        const float w = __shfl_xor_sync(0xffffffffu, v, 16);
        return upper ? make_float2(w, v) : make_float2(v, w);
    }
    if ((lane & 15) == 0) reinterpret_cast<float *>(s)[2 * warp + (lane >> 4)] = v;
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

// A thread's vectors are of eight channels, i = 0, 1: at bf16 eight neighbours;
// at fp32 two groups of four, neighbours' groups side by side, so that every
// load and store of a warp is whole sectors (eight neighbours a thread, half
// of each sector a store: forward 47 us for 33 at 3,972 x 2,832 fp32 with the
// residual, gradients 57 for 42).
template <typename T> __device__ __forceinline__ int upper_half() { return sizeof(T) == 2 ? 4 : 4 * (int)blockDim.x; }   // from the lower half's channels
template <typename T> __device__ __forceinline__ int channel(int i) {
    return sizeof(T) == 2 ? (i * (int)blockDim.x + (int)threadIdx.x) * 8 : (i * 2 * (int)blockDim.x + (int)threadIdx.x) * 4;
}
// A vector's halves that exist: `on` the lower, `whole` the upper.
template <typename T> __device__ __forceinline__ void load_params(const float *p, int c, bool on, bool whole, float otherwise, f2 (&v)[4]) {
    const float4 none = make_float4(otherwise, otherwise, otherwise, otherwise);
    const float4 a = p && on ? __ldg(reinterpret_cast<const float4 *>(p + c)) : none;
    const float4 b = p && whole ? __ldg(reinterpret_cast<const float4 *>(p + c + upper_half<T>())) : none;
    v[0] = f2_pack(a.x, a.y);
    v[1] = f2_pack(a.z, a.w);
    v[2] = f2_pack(b.x, b.y);
    v[3] = f2_pack(b.z, b.w);
}
template <typename T> __device__ __forceinline__ void store_floats(float *p, const f2 (&v)[4], bool on, bool whole) {
    const float2 a = f2_split(v[0]), b = f2_split(v[1]), c = f2_split(v[2]), d = f2_split(v[3]);
    if (on) *reinterpret_cast<float4 *>(p) = make_float4(a.x, a.y, b.x, b.y);
    if (whole) *reinterpret_cast<float4 *>(p + upper_half<T>()) = make_float4(c.x, c.y, d.x, d.y);
}
template <typename T> __device__ __forceinline__ void store(T *p, const f2 (&v)[4], bool on, bool whole) {
    if constexpr (sizeof(T) == 2) {
        if (on) ssm::store8(p, v, whole);
    } else {
        store_floats<T>(p, v, on, whole);
    }
}

// Rows of kIn arrays in a ring of kStages; a thread copies and reads its own
// vectors. `at` advances by the copied rows' distance.
template <typename T, int VPT, int kIn> struct Ring {
    static constexpr int H = sizeof(T) / 2, kRow = kIn * VPT * H;   // 16-byte pieces of a thread and row
    uint4 *base;
    __device__ __forceinline__ uint4 *piece(int stage, int k, int i, int h) const {
        return base + (stage * kRow + (i * kIn + k) * H + h) * (int)blockDim.x + (int)threadIdx.x;
    }
    __device__ __forceinline__ void issue(int stage, int k, const T *row, bool in, int D) const {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const int c = channel<T>(i) + h * upper_half<T>();   // (a piece holds 8 / H channels)
                copy_async<16>(piece(stage, k, i, h), row + c, in && c < D);
            }
    }
    __device__ __forceinline__ Raw8<T> held(int stage, int k, int i) const {
        Raw8<T> r;
#pragma unroll
        for (int h = 0; h < H; ++h) r.w[h] = *piece(stage, k, i, h);
        return r;
    }
};
// A row's mean for the channels of a vector that exist, 0 for the others (which hold zeros), in halves.
__device__ __forceinline__ void minus_mean(f2 (&v)[4], float mean, bool on, bool whole) {
    const f2 lo = both(on ? -mean : 0.f), hi = both(whole ? -mean : 0.f);
    v[0] = add2(v[0], lo);
    v[1] = add2(v[1], lo);
    v[2] = add2(v[2], hi);
    v[3] = add2(v[3], hi);
}

// Threads of the forward on an SM, rows in its ring (16384 x 2048 with the residual, 2 rows at 640, 768, 896, 1,024
// threads: 57, 44.6, 52, 48.6 us; 3 rows at 768: 49.7). Rows of one vector a thread have fewer bytes in flight: three
// (87,890 x 256 bf16: 35.4 us with two rows, 31.9 with three, 33.4 with four).
constexpr int kFwdThreads = 768;
template <int VPT> constexpr int fwd_rows() { return VPT == 1 ? 3 : 2; }

// kCta: the most threads it is launched with.
template <typename T, int VPT, int kCta> __global__ void __launch_bounds__(kCta, kFwdThreads / kCta) layernorm_fwd_kernel(const LayerNormParams p) {
    extern __shared__ __align__(16) uint4 smem[];
    __shared__ float4 s_a[4], s_b[4];
    constexpr int kRows = fwd_rows<VPT>();
    const Ring<T, VPT, 2> ring{smem};
    const size_t hop = (size_t)gridDim.x * p.D;
    long next = blockIdx.x;                             // the row copied next, and where it lies
    const T *x = static_cast<const T *>(p.x) + (size_t)next * p.D, *res = static_cast<const T *>(p.res) + (p.res ? (size_t)next * p.D : 0);
    auto issue = [&](int stage) {
        const bool in = next < p.rows;
        ring.issue(stage, 0, x, in, p.D);
        if (p.res) ring.issue(stage, 1, res, in, p.D);
        copies_commit();
        next += gridDim.x;
        x += hop;
        res += p.res ? hop : 0;
    };
#pragma unroll
    for (int k = 0; k < kRows - 1; ++k) issue(k);
    f2 w[VPT][4], b[VPT][4];
    bool on[VPT], whole[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = channel<T>(i);
        on[i] = c < p.D;
        whole[i] = c + upper_half<T>() < p.D;
        load_params<T>(p.w, c, on[i], whole[i], p.w ? 0.f : 1.f, w[i]);
        load_params<T>(p.b, c, on[i], whole[i], 0.f, b[i]);
    }
    const float D = (float)p.D, inv = 1.f / D;
    int stage = 0;
    size_t at = (size_t)blockIdx.x * p.D;               // of this row
    for (long row = blockIdx.x; row < p.rows; row += gridDim.x, at += hop) {
        copies_wait<kRows - 2>();
        f2 v[VPT][4], sum = both(0.f);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            raw_unpack(ring.held(stage, 0, i), v[i]);
            if (p.res) {
                f2 r[4];
                raw_unpack(ring.held(stage, 1, i), r);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[i][j] = add2(v[i][j], r[j]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) sum = add2(sum, v[i][j]);
        }
        issue(stage == 0 ? kRows - 1 : stage - 1);   // into the row before's stage
        stage = stage == kRows - 1 ? 0 : stage + 1;
        const float mean = mean_of(block_sum(pair_sum(sum), s_a), D, inv);
        f2 ss = both(0.f);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (p.s_out) store<T>(static_cast<T *>(p.s_out) + at + channel<T>(i), v[i], on[i], whole[i]);
            minus_mean(v[i], mean, on[i], whole[i]);
#pragma unroll
            for (int j = 0; j < 4; ++j) ss = fma2(v[i][j], v[i][j], ss);
        }
        const f2 r = both(rsqrtf(block_sum(pair_sum(ss), s_b) * inv + p.eps));
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[i][j] = fma2(mul2(v[i][j], r), w[i][j], b[i][j]);
            store<T>(static_cast<T *>(p.y) + at + channel<T>(i), v[i], on[i], whole[i]);
        }
    }
}

// Rows in the backward's ring (2, 3, 5 at 16384 x 2048 bf16: 50.6, 48.5, 61.6 us on the device). Two at fp32 of two vectors a
// thread, at every D: three would not fit at 512 threads (98 KB a row). At 384 they would; not measured.
template <typename T, int VPT> constexpr int ring_rows() { return sizeof(T) == 4 && VPT == 2 ? 2 : 3; }

// p.x: s; rows blockIdx.x, + gridDim.x, ...; partial dw and db of the CTA at
// p.part. 16384 x 2048 bf16: 48.5 us on the device, 51 a call with other inputs
// each time; the second launch takes 6 of them. (Measured while it took 53:
// clusters of two CTAs that add their sums up first, 52; of four, 68, fewer of
// them fit.)
template <typename T, int VPT, int kCta> __global__ void __launch_bounds__(kCta, kBwdThreads / kCta) layernorm_bwd_kernel(const LayerNormParams p) {
    constexpr int kStages = ring_rows<T, VPT>();
    extern __shared__ __align__(16) uint4 smem[];
    __shared__ float4 s_a[8], s_b[8];
    const Ring<T, VPT, 3> ring{smem};
    ssm::let_next_start();
    const size_t hop = (size_t)gridDim.x * p.D;
    long next = blockIdx.x;                             // the row copied next, and where it lies
    size_t ahead = (size_t)next * p.D;
    auto issue = [&](int stage) {
        const bool in = next < p.rows;
        ring.issue(stage, 0, static_cast<const T *>(p.x) + ahead, in, p.D);
        ring.issue(stage, 1, static_cast<const T *>(p.dy) + ahead, in, p.D);
        ring.issue(stage, 2, static_cast<const T *>(p.ds ? p.ds : p.x) + ahead, in && p.ds, p.D);
        copies_commit();
        next += gridDim.x;
        ahead += hop;
    };
    f2 w[VPT][4], dw[VPT][4], db[VPT][4];
    bool on[VPT], whole[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = channel<T>(i);
        on[i] = c < p.D;
        whole[i] = c + upper_half<T>() < p.D;
        load_params<T>(p.w, c, on[i], whole[i], p.w ? 0.f : 1.f, w[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) dw[i][j] = db[i][j] = both(0.f);
    }
    const float D = (float)p.D, inv = 1.f / D;
    int stage = 0;
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) issue(k);
    size_t at = (size_t)blockIdx.x * p.D;               // of this row
    for (long row = blockIdx.x; row < p.rows; row += gridDim.x, at += hop) {
        copies_wait<kStages - 2>();
        f2 x[VPT][4], g[VPT][4], sx = both(0.f), sg = both(0.f);
        Raw8<T> cs[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            raw_unpack(ring.held(stage, 0, i), x[i]);
            raw_unpack(ring.held(stage, 1, i), g[i]);
            cs[i] = ring.held(stage, 2, i);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sx = add2(sx, x[i][j]);
                sg = fma2(g[i][j], w[i][j], sg);
            }
        }
        issue(stage == 0 ? kStages - 1 : stage - 1);    // into the row before's stage
        stage = stage == kStages - 1 ? 0 : stage + 1;
        const float2 sums = block_sums(pair_sum(sx), pair_sum(sg), s_a);
        const float mean = mean_of(sums.x, D, inv);
        f2 ss = both(0.f), sc = both(0.f);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            minus_mean(x[i], mean, on[i], whole[i]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                db[i][j] = add2(db[i][j], g[i][j]);
                ss = fma2(x[i][j], x[i][j], ss);
                sc = fma2(mul2(g[i][j], w[i][j]), x[i][j], sc);
            }
        }
        const float2 squares = block_sums(pair_sum(ss), pair_sum(sc), s_b);
        const float r = rsqrtf(squares.x * inv + p.eps);
        // dx = ds + r (g w - mean(g w)) - c k, with xn mean(g w xn) r = c k
        const f2 r2 = both(r), k2 = both(-r * (r * (r * (squares.y * inv)))), m2 = both(-sums.y * inv);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            f2 s[4];
            raw_unpack(cs[i], s);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                dw[i][j] = fma2(g[i][j], mul2(x[i][j], r2), dw[i][j]);
                s[j] = fma2(r2, fma2(g[i][j], w[i][j], m2), fma2(k2, x[i][j], s[j]));
            }
            store<T>(static_cast<T *>(p.dx) + at + channel<T>(i), s, on[i], whole[i]);
        }
    }
    if (!p.part) return;
    float *part = p.part + (size_t)blockIdx.x * 2 * p.D;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        store_floats<T>(part + channel<T>(i), dw[i], on[i], whole[i]);
        store_floats<T>(part + p.D + channel<T>(i), db[i], on[i], whole[i]);
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
    const long held = (long)(kFwdThreads / th) * device_sm_count();   // (a warp each: 24 CTAs an SM)
    const int bytes = (vpt == 1 ? fwd_rows<1>() : fwd_rows<2>()) * 2 * vpt * th * 8 * (int)sizeof(T);
    auto *kern = th <= 256   ? (vpt == 1 ? layernorm_fwd_kernel<T, 1, 256> : layernorm_fwd_kernel<T, 2, 256>)
                 : th <= 384 ? (vpt == 1 ? layernorm_fwd_kernel<T, 1, 384> : layernorm_fwd_kernel<T, 2, 384>)
                             : (vpt == 1 ? layernorm_fwd_kernel<T, 1, 512> : layernorm_fwd_kernel<T, 2, 512>);
    cudaError_t e = allow_smem(kern, bytes);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)(p.rows < held ? p.rows : held), th, bytes, s>>>(p);
    if (launches) ++*launches;
    return cudaGetLastError();
}

// The backward's shape, by D alone: two vectors a thread from 264 channels on (one, at 16384 x 2048: 57 us on the device for 48.5).
int bwd_vpt(int D) { return D > 256 ? 2 : 1; }
int bwd_threads(int D) { return round32(((D + 7) / 8 + bwd_vpt(D) - 1) / bwd_vpt(D)); }

template <typename T> cudaError_t bwd(const LayerNormParams &p, cudaStream_t s, int *launches) {
    const int vpt = bwd_vpt(p.D), th = bwd_threads(p.D);
    const unsigned grid = (unsigned)layernorm_bwd_grid(p.rows, p.D);
    const int bytes = (vpt == 1 ? ring_rows<T, 1>() : ring_rows<T, 2>()) * 3 * vpt * th * 8 * (int)sizeof(T);
    auto *kern = vpt == 1 ? layernorm_bwd_kernel<T, 1, 128> : th <= 128 ? layernorm_bwd_kernel<T, 2, 128>
               : th <= 256 ? layernorm_bwd_kernel<T, 2, 256> : layernorm_bwd_kernel<T, 2, 512>;
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

// CTAs of the backward, each walking its share of the rows.
long layernorm_bwd_grid(long rows, int D) {
    const int th = bwd_threads(D);
    const long most = (long)(kBwdThreads / th) * device_sm_count();   // (a warp each: 16 an SM)
    return rows < most ? rows : most;
}

cudaError_t launch_layernorm_fwd(const LayerNormParams &p, bool bf16, cudaStream_t s, int *launches) {
    return bf16 ? fwd<__nv_bfloat16>(p, s, launches) : fwd<float>(p, s, launches);
}
cudaError_t launch_layernorm_bwd(const LayerNormParams &p, bool bf16, cudaStream_t s, int *launches) {
    return bf16 ? bwd<__nv_bfloat16>(p, s, launches) : bwd<float>(p, s, launches);
}

}  // namespace gla
