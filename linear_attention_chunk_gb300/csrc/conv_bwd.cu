// conv_bwd.cu -- the gradients of the causal depthwise Conv1d (width 4) with
// SiLU, per channel, with a_t = sum_j w_j x_{t-3+j} + b and sg = sigmoid(a):
//     dp_t = dy_t sg_t (1 + a_t (1 - sg_t))
//     dx_t = sum_j w_j dp_{t+3-j},   dw_j = sum_t dp_t x_{t-3+j},   db = sum_t dp_t
// (dp past the sequence's end is 0; x before its first token is the window,
// a constant).
//
// A stream: 6 bytes an element at bf16 (x, dy in, dx out): 403 MB in 81 us
// at 8 x 2048 x 4096 with the sums, 0.74 of the measured copy rate, the rest
// instructions. A thread owns four channels over a tile of tokens and walks it
// forward with the last three x and dp in registers, so dx lags three tokens
// behind, and reads three tokens past the tile's end for it (the tile's own
// sums leave those out). The inputs come through a ring of asynchronous
// copies, twelve tokens ahead: each thread copies and reads its own, so
// nothing waits for another. dw and db stay in registers and leave once per
// tile as partial sums, added in a second launch (reduce.cu).
#include <type_traits>

#include "ssm_common.cuh"

namespace gla {
namespace {

using namespace ssm;

constexpr int kThreads = 128;   // 512 channels a CTA
constexpr int kStep = 4, kStages = 4;   // tokens of a stage, stages of the ring
constexpr int kMinBlocks = 4;   // measured at 8 x 2048 x 4096, bf16: 84 us (tiles of 128), at 5 (spills) 108; at fp32 three fit (64 KB each)
constexpr int kLeastTile = 16, kMostTile = 256, kMostRounds = 16, kStart = 16;   // see conv_bwd_tile
static_assert(kStep >= 3, "a tile's first step covers the three tokens that dx lags behind");

template <typename T> struct Raw4 {
    uint2 w[sizeof(T) / 2];
};
template <typename T> __device__ __forceinline__ Raw4<T> load4(const T *p) {
    Raw4<T> r;
    if constexpr (sizeof(T) == 2) {
        r.w[0] = __ldg(reinterpret_cast<const uint2 *>(p));
    } else {
        const uint4 u = __ldg(reinterpret_cast<const uint4 *>(p));
        r.w[0] = make_uint2(u.x, u.y);
        r.w[1] = make_uint2(u.z, u.w);
    }
    return r;
}
__device__ __forceinline__ void unpack4(const Raw4<__nv_bfloat16> &r, f2 (&v)[2]) {
    v[0] = f2_pack(__uint_as_float(r.w[0].x << 16), __uint_as_float(r.w[0].x & 0xffff0000u));
    v[1] = f2_pack(__uint_as_float(r.w[0].y << 16), __uint_as_float(r.w[0].y & 0xffff0000u));
}
__device__ __forceinline__ void unpack4(const Raw4<float> &r, f2 (&v)[2]) {
    v[0] = f2_pack(__uint_as_float(r.w[0].x), __uint_as_float(r.w[0].y));
    v[1] = f2_pack(__uint_as_float(r.w[1].x), __uint_as_float(r.w[1].y));
}
__device__ __forceinline__ void store4(__nv_bfloat16 *p, f2 a, f2 b) {
    const float2 u = f2_split(a), v = f2_split(b);
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16x2(u.x, u.y), pack_bf16x2(v.x, v.y));
}
__device__ __forceinline__ void store4(float *p, f2 a, f2 b) {
    const float2 u = f2_split(a), v = f2_split(b);
    *reinterpret_cast<float4 *>(p) = make_float4(u.x, u.y, v.x, v.y);
}

template <typename T> __global__ void __launch_bounds__(kThreads, kMinBlocks) conv_bwd_kernel(const ConvBwdParams p, int blocks, int tiles) {
    extern __shared__ __align__(16) unsigned char smem[];
    Raw4<T> (*ring)[kThreads] = reinterpret_cast<Raw4<T> (*)[kThreads]>(smem);   // [stage][token][x, dy][thread]
    const int c = ((int)(blockIdx.x % (unsigned)blocks) * kThreads + threadIdx.x) * 4;
    const long unit = blockIdx.x / (unsigned)blocks;
    let_next_start();
    if (c >= p.D) return;
    const long b = unit / tiles;
    const int t0 = (int)(unit % tiles) * p.tile, t1 = min(t0 + p.tile, p.T), last = min(t1 + 3, p.T);
    const size_t D = (size_t)p.D;
    const T *x = static_cast<const T *>(p.x) + (size_t)b * p.T * D + c;
    const T *dy = static_cast<const T *>(p.dy) + (size_t)b * p.T * D + c;

    f2 w[kTaps][2], bias[2] = {0, 0}, dw[kTaps][2], db[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const float4 u = __ldg(reinterpret_cast<const float4 *>(p.w) + c + 2 * e);
        const float4 v = __ldg(reinterpret_cast<const float4 *>(p.w) + c + 2 * e + 1);
        w[0][e] = f2_pack(u.x, v.x);
        w[1][e] = f2_pack(u.y, v.y);
        w[2][e] = f2_pack(u.z, v.z);
        w[3][e] = f2_pack(u.w, v.w);
        if (p.b) bias[e] = f2_pack(p.b[c + 2 * e], p.b[c + 2 * e + 1]);
#pragma unroll
        for (int j = 0; j < kTaps; ++j) dw[j][e] = 0;
    }
    f2 h[3][2], dp[3][2];           // x and dp of the three tokens before
#pragma unroll
    for (int j = 0; j < 3; ++j) {
        const int t = t0 - 3 + j;
        if (t >= 0) {
            unpack4(load4(x + (size_t)t * D), h[j]);
        } else if (p.win) {
            const float *r = p.win + ((size_t)b * kTaps + kTaps + t) * D + c;
            h[j][0] = f2_pack(r[0], r[1]);
            h[j][1] = f2_pack(r[2], r[3]);
        } else {
            h[j][0] = h[j][1] = 0;
        }
        dp[j][0] = dp[j][1] = 0;
    }
    const f2 one = both(1.f), neg = both(-kLog2e), minus = both(-1.f);
    constexpr int kBytes = 4 * (int)sizeof(T);
    const T *ix = x + (size_t)t0 * D, *iy = dy + (size_t)t0 * D;   // the next token to ask for
    auto issue = [&](int t, int stage) {
        const bool all = t + kStep <= last;
#pragma unroll
        for (int i = 0; i < kStep; ++i) {
            const bool in = all || t + i < last;
            copy_async<kBytes>(&ring[(stage * kStep + i) * 2][threadIdx.x], in ? ix : x, in);
            copy_async<kBytes>(&ring[(stage * kStep + i) * 2 + 1][threadIdx.x], in ? iy : dy, in);
            ix += D;
            iy += D;
        }
        copies_commit();
    };
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) issue(t0 + k * kStep, k);
    T *dx = static_cast<T *>(p.dx) + ((size_t)b * p.T + t0) * D + c;   // the token three behind
    // kStep tokens from t on; kInside: all of them the tile's own.
    auto step = [&](int t, int stage, auto inside) {
        constexpr bool kInside = decltype(inside)::value;
        Raw4<T> rx[kStep], ry[kStep];
#pragma unroll
        for (int i = 0; i < kStep; ++i) {
            rx[i] = ring[(stage * kStep + i) * 2][threadIdx.x];
            ry[i] = ring[(stage * kStep + i) * 2 + 1][threadIdx.x];
        }
        issue(t + (kStages - 1) * kStep, stage == 0 ? kStages - 1 : stage - 1);   // the stage read before this one
#pragma unroll
        for (int i = 0; i < kStep; ++i) {
            f2 xv[2], g[2], o[2];
            unpack4(rx[i], xv);
            unpack4(ry[i], g);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                f2 a = fma2(w[0][e], h[0][e], bias[e]);
                a = fma2(w[1][e], h[1][e], a);
                a = fma2(w[2][e], h[2][e], a);
                a = fma2(w[3][e], xv[e], a);
                const f2 sg = rcp_pair(add2(ex2_pair(mul2(a, neg)), one));
                // sg (1 + a (1 - sg)); where a overflows the exponential, sg = 0 and a (1 - sg) is finite
                f2 d = mul2(g[e], mul2(sg, fma2(a, fma2(sg, minus, one), one)));
                if (!kInside && t + i >= last) d = 0;   // behind the end: dy is 0, but 0 x NaN (a may overflow there) is not
                if (kInside || t + i < t1) {
                    dw[0][e] = fma2(d, h[0][e], dw[0][e]);
                    dw[1][e] = fma2(d, h[1][e], dw[1][e]);
                    dw[2][e] = fma2(d, h[2][e], dw[2][e]);
                    dw[3][e] = fma2(d, xv[e], dw[3][e]);
                    db[e] = add2(d, db[e]);
                }
                o[e] = mul2(w[0][e], d);
                o[e] = fma2(w[1][e], dp[2][e], o[e]);
                o[e] = fma2(w[2][e], dp[1][e], o[e]);
                o[e] = fma2(w[3][e], dp[0][e], o[e]);
                h[0][e] = h[1][e];
                h[1][e] = h[2][e];
                h[2][e] = xv[e];
                dp[0][e] = dp[1][e];
                dp[1][e] = dp[2][e];
                dp[2][e] = d;
            }
            if (i >= 3 || t != t0) {            // token t + i - 3 of the tile
                if (kInside || t + i - 3 < t1) store4(dx, o[0], o[1]);
                dx += D;
            }
        }
    };
    int t = t0, stage = 0;
    for (; t + kStep <= t1; t += kStep) {
        copies_wait<kStages - 2>();
        step(t, stage, std::true_type{});
        stage = stage == kStages - 1 ? 0 : stage + 1;
    }
    for (; t < t1 + 3; t += kStep) {
        copies_wait<kStages - 2>();
        step(t, stage, std::false_type{});
        stage = stage == kStages - 1 ? 0 : stage + 1;
    }
    // partials: [D, 4] of dw, then [D] of db
    float *part = p.part + (size_t)unit * 5 * D;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const float2 a = f2_split(dw[0][e]), bb = f2_split(dw[1][e]), cc = f2_split(dw[2][e]), d = f2_split(dw[3][e]);
        reinterpret_cast<float4 *>(part)[c + 2 * e] = make_float4(a.x, bb.x, cc.x, d.x);
        reinterpret_cast<float4 *>(part)[c + 2 * e + 1] = make_float4(a.y, bb.y, cc.y, d.y);
        *reinterpret_cast<float2 *>(part + 4 * D + c + 2 * e) = f2_split(db[e]);
    }
}

}  // namespace

// Tokens per tile: as many tiles as fill a whole number of rounds of the CTAs
// that the GPU holds, of the rounds up to kMostRounds the ones that cost least
// when a tile costs its tokens and kStart more (three tokens past its end, the
// first loads, its partial sums). 8 x 2048 x 4096: tiles of 228, 576 CTAs in
// one round; of 128, 1,024 CTAs in one and two thirds: 1 us more. The rule
// counts bf16's four CTAs an SM; at fp32 three fit, and a round is a round and a
// third: 8 x 2048 x 2048 86 us (0.69 of the copy rate), x 4096 156 (0.76).
int conv_bwd_tile(int B, int T, int D) {
    const long chains = (long)B * ((D + 4 * kThreads - 1) / (4 * kThreads)), held = (long)kMinBlocks * device_sm_count();
    long best = kMostTile, least = -1;
    for (long r = 1; r <= kMostRounds; ++r) {
        const long n = r * held / chains;      // tiles of a sequence
        if (n < 1) continue;
        long tile = (((long)T + n - 1) / n + kStep - 1) / kStep * kStep;
        if (tile < kLeastTile) tile = kLeastTile;
        if (tile > kMostTile) tile = kMostTile;
        const long ctas = chains * ((T + tile - 1) / tile), cost = (ctas + held - 1) / held * (tile + kStart);
        if (least < 0 || cost < least) {
            least = cost;
            best = tile;
        }
    }
    return (int)best;
}

cudaError_t launch_conv_bwd(const ConvBwdParams &p, bool bf16, cudaStream_t s, int *launches) {
    const int blocks = (p.D + 4 * kThreads - 1) / (4 * kThreads), tiles = (p.T + p.tile - 1) / p.tile;
    const long units = (long)p.B * tiles;
    if ((long double)units * blocks > 2147483647.0L) return cudaErrorInvalidValue;
    const int bytes = kStages * kStep * 2 * kThreads * 4 * (bf16 ? 2 : 4);   // 32 KB, 64 KB at fp32
    auto *kern = bf16 ? conv_bwd_kernel<__nv_bfloat16> : conv_bwd_kernel<float>;
    cudaError_t e = cudaSuccess;
    if (bytes > 48 * 1024) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)(units * blocks), kThreads, bytes, s>>>(p, blocks, tiles);
    if (launches) ++*launches;
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    SumJobs sums;
    sums.add(p.part, units, 4L * p.D, 5L * p.D, p.dw);
    sums.add(p.part + 4L * p.D, units, p.D, 5L * p.D, p.db);
    return launch_sums(sums, s, launches);
}

}  // namespace gla
