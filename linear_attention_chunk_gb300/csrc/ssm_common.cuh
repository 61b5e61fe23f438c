// ssm_common.cuh -- device helpers of the selective state-space kernels
// (ssm.cu, ssm_step.cu, ssm_bwd.cu), the Conv1d's gradients (conv_bwd.cu) and
// the norm (rmsnorm.cu): fp32 pairs, the step's softplus and the SiLU gate,
// asynchronous copies, and vectors of eight channels in either element type.
#pragma once

#include <cfloat>

#include "common.cuh"
#include "kernels.h"

namespace gla {
namespace ssm {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kTaps = 4;
constexpr int kVec = 8;   // channels a thread loads and stores at once

// Two fp32 numbers in a 64-bit register pair: the packed instructions do two
// multiply-adds an issue slot (at the same rate per lane as the scalar ones).
using f2 = uint64_t;

__device__ __forceinline__ f2 f2_pack(float lo, float hi) {
    f2 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ float2 f2_split(f2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float ex2(float x) {   // 2^x, relative error below 1.5e-7 (measured on [-4, 0])
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// A rate, held to the lowest finite number: 0 x -inf is NaN, and a step of 0
// (also of the tokens behind a sequence's end) keeps the state at any rate.
// rate_log2: the rate of 2^x, rate * log2(e), which for a finite rate may be -inf.
__device__ __forceinline__ float finite_rate(float a) { return a < -FLT_MAX ? -FLT_MAX : a; }   // (NaN stays NaN)
__device__ __forceinline__ float rate_log2(float a) { return finite_rate(a * kLog2e); }

__device__ __forceinline__ f2 ex2_pair(f2 x) {
    const float2 v = f2_split(x);
    return f2_pack(ex2(v.x), ex2(v.y));
}

__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f2 both(float v) { return f2_pack(v, v); }
__device__ __forceinline__ f2 rcp_pair(f2 x) {
    const float2 v = f2_split(x);
    return f2_pack(rcp(v.x), rcp(v.y));
}

// log(1 + e^v) = max(v, 0) + log1p(w), w = e^-|v| in (0, 1], by the series
// log1p(w) = 2 atanh(s) = 2 (s + s^3/3 + s^5/5 + ...), s = w / (2 + w) <= 1/3:
// seven terms leave 2 s^15 / 15 < 1e-8. Relative to the result, not to 1: a
// step of 1e-3 keeps fp32's precision, which log(1 + w) would lose.
__device__ __forceinline__ f2 softplus2(f2 v) {
    const float2 x = f2_split(v);
    const f2 w = f2_pack(ex2(-fabsf(x.x) * kLog2e), ex2(-fabsf(x.y) * kLog2e));
    const f2 s = mul2(w, rcp_pair(add2(w, both(2.f))));
    const f2 q = mul2(s, s);
    f2 r = fma2(both(1.f / 13.f), q, both(1.f / 11.f));
    r = fma2(r, q, both(1.f / 9.f));
    r = fma2(r, q, both(1.f / 7.f));
    r = fma2(r, q, both(1.f / 5.f));
    r = fma2(r, q, both(1.f / 3.f));
    r = fma2(mul2(r, q), s, s);
    return fma2(both(2.f), r, f2_pack(fmaxf(x.x, 0.f), fmaxf(x.y, 0.f)));
}
__device__ __forceinline__ float softplus(float v) {
    const float w = ex2(-fabsf(v) * kLog2e), s = w * rcp(2.f + w), q = s * s;
    float r = fmaf(1.f / 13.f, q, 1.f / 11.f);
    r = fmaf(r, q, 1.f / 9.f);
    r = fmaf(r, q, 1.f / 7.f);
    r = fmaf(r, q, 1.f / 5.f);
    r = fmaf(r, q, 1.f / 3.f);
    r = fmaf(r * q, s, s);
    return fmaf(2.f, r, fmaxf(v, 0.f));
}
__device__ __forceinline__ float sigmoid(float v) { return rcp(1.f + ex2(-v * kLog2e)); }
__device__ __forceinline__ float silu(float v) { return v * sigmoid(v); }
__device__ __forceinline__ f2 sigmoid2(f2 v) { return rcp_pair(add2(ex2_pair(mul2(v, both(-kLog2e))), both(1.f))); }
__device__ __forceinline__ f2 silu2(f2 v) { return mul2(v, sigmoid2(v)); }

// Asynchronous copies of 8 or 16 bytes into shared memory; `in` false writes
// zeros and reads nothing.
template <int kBytes> __device__ __forceinline__ void copy_async(void *dst, const void *src, bool in) {
    static_assert(kBytes == 8 || kBytes == 16, "one vector");
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst), n = in ? kBytes : 0;
    if constexpr (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(d), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft> __device__ __forceinline__ void copies_wait() {   // all but the last kLeft groups have arrived
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// A launch that follows another of the same call on the same stream and reads
// what that leaves: its CTAs may start as soon as all of the other's have
// (`let_next_start`) and SMs have room, and begin with `wait_for_previous`,
// which returns when the other launch is done and its writes are visible. It
// hides the gap between the two (sums of the norm's gradients: 49 -> 46 us a call).
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <typename... P, typename... A>
cudaError_t launch_behind(void (*kern)(P...), dim3 grid, int threads, int bytes, cudaStream_t s, const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = s;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Eight consecutive channels as they lie in memory.
template <typename T> struct Raw8 {
    uint4 w[sizeof(T) / 2];
};

template <typename T> __device__ __forceinline__ Raw8<T> raw_zero() {
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.w[i] = make_uint4(0, 0, 0, 0);
    return r;
}
// `whole`: all eight channels exist. D is a multiple of 8 at bf16; at fp32 it
// may be a multiple of 4 only, and the last vector of a row half there.
template <typename T> __device__ __forceinline__ Raw8<T> raw_load(const T *p, bool whole) {
    Raw8<T> r;
    r.w[0] = __ldg(reinterpret_cast<const uint4 *>(p));
    if constexpr (sizeof(T) == 4) r.w[1] = whole ? __ldg(reinterpret_cast<const uint4 *>(p) + 1) : make_uint4(0, 0, 0, 0);
    return r;
}
__device__ __forceinline__ void raw_unpack(const Raw8<__nv_bfloat16> &r, f2 (&v)[4]) {
    const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ void raw_unpack(const Raw8<float> &r, f2 (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        v[2 * i] = f2_pack(__uint_as_float(r.w[i].x), __uint_as_float(r.w[i].y));
        v[2 * i + 1] = f2_pack(__uint_as_float(r.w[i].z), __uint_as_float(r.w[i].w));
    }
}
// The same from an address with no more than its element's alignment.
__device__ __forceinline__ Raw8<__nv_bfloat16> raw_gather(const __nv_bfloat16 *p) {
    const unsigned short *u = reinterpret_cast<const unsigned short *>(p);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = (uint32_t)__ldg(u + 2 * i) | ((uint32_t)__ldg(u + 2 * i + 1) << 16);
    Raw8<__nv_bfloat16> r;
    r.w[0] = make_uint4(w[0], w[1], w[2], w[3]);
    return r;
}
__device__ __forceinline__ Raw8<float> raw_gather(const float *p) {
    const uint32_t *u = reinterpret_cast<const uint32_t *>(p);
    Raw8<float> r;
#pragma unroll
    for (int i = 0; i < 2; ++i) r.w[i] = make_uint4(__ldg(u + 4 * i), __ldg(u + 4 * i + 1), __ldg(u + 4 * i + 2), __ldg(u + 4 * i + 3));
    return r;
}
__device__ __forceinline__ void raw_unpack(const Raw8<__nv_bfloat16> &r, float (&v)[8]) {
    const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void raw_unpack(const Raw8<float> &r, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        v[4 * i] = __uint_as_float(r.w[i].x);
        v[4 * i + 1] = __uint_as_float(r.w[i].y);
        v[4 * i + 2] = __uint_as_float(r.w[i].z);
        v[4 * i + 3] = __uint_as_float(r.w[i].w);
    }
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&v)[8], bool) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                               pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void store8(float *p, const float (&v)[8], bool whole) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    if (whole) reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
template <typename T> __device__ __forceinline__ void store8(T *p, const f2 (&v)[4], bool whole) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 u = f2_split(v[i]);
        f[2 * i] = u.x;
        f[2 * i + 1] = u.y;
    }
    store8(p, f, whole);
}
// Eight fp32 parameters of consecutive channels (zeros without an array).
__device__ __forceinline__ void param8(const float *p, int c, bool whole, float (&v)[8]) {
    if (p) {
        const float4 a = __ldg(reinterpret_cast<const float4 *>(p + c));
        const float4 b = whole ? __ldg(reinterpret_cast<const float4 *>(p + c) + 1) : make_float4(0.f, 0.f, 0.f, 0.f);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
    }
}

__device__ __forceinline__ void param8(const float *p, int c, bool whole, f2 (&v)[4]) {
    float f[8];
    param8(p, c, whole, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f2_pack(f[2 * i], f[2 * i + 1]);
}

// The four lanes that share channels ("a quad") are eight apart: lane / 8 is
// the lane's place in it, lane % 8 its channels. Eight neighbouring lanes then
// read one 16-byte piece of B or C, which shared memory serves in two clocks a
// warp instead of four (measured; four neighbours reading four pieces: four).
// Four numbers, one per token, each spread over the four lanes of a quad:
// returns the sum of number (lane / 8), in three exchanges.
__device__ __forceinline__ float quad_transpose_sum(const float (&v)[4], int lane) {
    const bool hi = lane & 16, lo = lane & 8;
    float k0 = hi ? v[2] : v[0], k1 = hi ? v[3] : v[1];
    k0 += __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[2], 16);
    k1 += __shfl_xor_sync(0xffffffffu, hi ? v[1] : v[3], 16);
    const float k = lo ? k1 : k0;
    return k + __shfl_xor_sync(0xffffffffu, lo ? k0 : k1, 8);
}

}  // namespace ssm
}  // namespace gla
