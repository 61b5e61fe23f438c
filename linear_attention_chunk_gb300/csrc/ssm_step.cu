// ssm_step.cu -- one token per sequence of the selective state-space scan,
// with the causal Conv1d's window when asked: the serving step. Per (sequence,
// channel) it moves 128 bytes of state at N = 16 (64 in, 64 out), 28 of the
// window and 8 of activations: an HBM stream, bound by the bytes in flight.
//
// A quad of lanes owns a (sequence, channel): each lane a quarter of the
// states, in one contiguous access per warp, and one tap of the filter: lane
// q loads the input at t-3+q (window row q+1, or the new token) and stores
// it as window row q, so the shift costs no traffic of its own.
#include "ssm_common.cuh"

namespace gla {
namespace {

using namespace ssm;

constexpr int kThreads = 256;             // 64 channels per pass

__device__ __forceinline__ float quad_sum(float v) {   // over four neighbouring lanes
    v += __shfl_xor_sync(0xffffffffu, v, 1);
    return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

// kRows sequences per CTA column of 64 channels, all their loads up front.
template <typename T, int N, int kRows> __global__ void __launch_bounds__(kThreads) ssm_step_kernel(const SsmParams p, int tiles) {
    constexpr int SP = N / 4, P = SP / 2;
    const int lane = threadIdx.x % 32, q = lane % 4;
    const int ch = (int)(blockIdx.x % (unsigned)tiles) * (kThreads / 4) + threadIdx.x / 4;
    const int n0 = (int)(blockIdx.x / (unsigned)tiles) * kRows;
    const bool on = ch < p.D;
    const int c = on ? ch : 0;            // idle lanes mirror channel 0 and store nothing

    int slot[kRows];
    bool live[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const int n = n0 + r;
        live[r] = n < p.nseq;
        slot[r] = live[r] ? (p.slots ? p.slots[n] : n) : 0;
        if (live[r] && (slot[r] < 0 || slot[r] >= p.n_slots)) {
            if (q == 0) atomicOr(p.status, kDevBadState);
            live[r] = false;
        }
    }
    float2 hv[kRows][P];
    float xv[kRows], tap[kRows], dv[kRows], zv[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        if (!live[r]) continue;
        const size_t n = (size_t)(n0 + r);
        const float2 *h = reinterpret_cast<const float2 *>(p.h0 + ((size_t)slot[r] * p.D + c) * N + q * SP);
#pragma unroll
        for (int i = 0; i < P; ++i) hv[r][i] = h[i];
        xv[r] = Elem<T>::load(static_cast<const T *>(p.x) + n * p.ldx + c);
        dv[r] = Elem<T>::load(static_cast<const T *>(p.dt) + n * p.ldt + c);
        zv[r] = p.z ? Elem<T>::load(static_cast<const T *>(p.z) + n * p.ldz + c) : 0.f;
        tap[r] = xv[r];
        if (p.win && q < kTaps - 1) tap[r] = p.win[((size_t)slot[r] * kTaps + q + 1) * p.D + c];
    }
    __syncwarp();   // a lane's window store below follows its neighbour's load of the same row
    float2 a[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        a[i] = __ldg(reinterpret_cast<const float2 *>(p.A + (size_t)c * N + q * SP) + i);
        a[i].x *= kLog2e;
        a[i].y *= kLog2e;
    }
    const float bias = p.dt_bias ? p.dt_bias[c] : 0.f, skip = p.skip ? p.skip[c] : 0.f;
    const float cw = p.conv_w ? p.conv_w[(size_t)c * kTaps + q] : 0.f, cb = p.conv_b ? p.conv_b[c] : 0.f;

#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        if (!live[r]) continue;           // uniform over the CTA: the shuffles below are whole
        const size_t n = (size_t)(n0 + r);
        float u = xv[r];
        if (p.conv_w) u = silu(quad_sum(cw * tap[r]) + cb);
        float dl = dv[r] + bias;
        if (p.softplus) dl = softplus(dl);
        const float du = dl * u;
        const T *b = static_cast<const T *>(p.Bm) + n * p.ldb + q * SP;
        const T *cc = static_cast<const T *>(p.Cm) + n * p.ldc + q * SP;
        float y = 0.f;
        float2 *h = reinterpret_cast<float2 *>(p.hT + ((size_t)slot[r] * p.D + c) * N + q * SP);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            float2 v = hv[r][i];
            v.x = fmaf(ex2(dl * a[i].x), v.x, du * Elem<T>::load(b + 2 * i));
            v.y = fmaf(ex2(dl * a[i].y), v.y, du * Elem<T>::load(b + 2 * i + 1));
            y = fmaf(v.x, Elem<T>::load(cc + 2 * i), y);
            y = fmaf(v.y, Elem<T>::load(cc + 2 * i + 1), y);
            if (on) h[i] = v;
        }
        y = fmaf(skip, u, quad_sum(y));
        if (p.z) y *= silu(zv[r]);
        if (on && q == 0) Elem<T>::store(static_cast<T *>(p.y) + n * p.D + ch, y);
        if (on && p.win) p.win[((size_t)slot[r] * kTaps + q) * p.D + ch] = tap[r];
    }
}

template <typename T, int N> cudaError_t run(const SsmParams &p, cudaStream_t s, int *launches) {
    constexpr int kRows = 1;
    const int tiles = (p.D + kThreads / 4 - 1) / (kThreads / 4);
    const long blocks = (long)((p.nseq + kRows - 1) / kRows) * tiles;
    if (blocks > 2147483647L) return cudaErrorInvalidValue;
    ssm_step_kernel<T, N, kRows><<<(unsigned)blocks, kThreads, 0, s>>>(p, tiles);
    if (launches) ++*launches;
    return cudaGetLastError();
}

template <typename T> cudaError_t by_state(const SsmParams &p, cudaStream_t s, int *launches) {
    switch (p.N) {
    case 8: return run<T, 8>(p, s, launches);
    case 16: return run<T, 16>(p, s, launches);
    case 32: return run<T, 32>(p, s, launches);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_ssm_step(const SsmParams &p, bool bf16, cudaStream_t s, int *launches) {
    return bf16 ? by_state<__nv_bfloat16>(p, s, launches) : by_state<float>(p, s, launches);
}

}  // namespace gla
