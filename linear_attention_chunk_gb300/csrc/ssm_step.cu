// ssm_step.cu -- one token per sequence of the selective state-space scan,
// with the causal Conv1d's window when asked: the serving step. Per (sequence,
// channel) it moves 128 bytes of state at N = 16 (64 in, 64 out), 28 of the
// window and 8 of activations: an HBM stream, bound by the bytes in flight
// (860 MB at 1,280 sequences of 4,096 channels in 165 us: 5.2 TB/s, 0.77 of the
// measured copy rate; without the filter 141 us, 0.74). The other instances at
// that size, with and without the filter: N = 8 131 and 102 us (0.59, 0.54 of
// the copy rate), N = 32 553 and 281 (0.41, 0.73); fp32 N = 8 125 and 102 (0.67,
// 0.60), N = 16 235 and 143 (0.56, 0.78), N = 32 814 and 485 (0.28, 0.43). With
// the filter fp32 N = 16 and both of N = 32 spill at the 80 registers of six
// CTAs an SM, as does fp32 N = 32 without it.
//
// A warp owns eight channels of four sequences. Elementwise work is lane
// (channel, sequence)'s: the filter over the window and the new input, the
// window's shift, the step, and at the end the skip and the gate. The states
// are lane (channel, quarter)'s, a quarter of the channel's states of all four
// sequences: per sequence the quad takes the step and its input from the lane
// that has them, and the four sums over states return to those lanes in three
// exchanges. With every lane of a quad doing one sequence's elementwise work
// over again the kernel was bound by instructions (265 a warp and sequence).
#include "ssm_common.cuh"

namespace gla {
namespace {

using namespace ssm;

constexpr int kThreads = 128;   // 32 channels
constexpr int kSeqs = 4, kStages = 3;
// CTAs an SM, of all instances, measured at bf16, N = 16 with the filter: 3, 4, 5, 6, 7: 248, 221, 194, 164, 175 us at 1280 x 4096
constexpr int kMinBlocks = 6;

// Four numbers, each spread over four neighbouring lanes: the sum of number
// (lane % 4), in three exchanges.
__device__ __forceinline__ float sum_to_own(const float (&v)[4], int lane) {
    const bool hi = lane & 2, lo = lane & 1;
    float k0 = hi ? v[2] : v[0], k1 = hi ? v[3] : v[1];
    k0 += __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[2], 2);
    k1 += __shfl_xor_sync(0xffffffffu, hi ? v[1] : v[3], 2);
    return (lo ? k1 : k0) + __shfl_xor_sync(0xffffffffu, lo ? k0 : k1, 1);
}

// The lane's states: pieces of V (4, or 2 at N = 8) at n = i * 4 V + q * V, so
// that a quad's piece is contiguous and every 32-byte sector is used whole.
template <int N> struct Piece {
    static constexpr int V = N == 8 ? 2 : 4, P = N / (4 * V);
};
template <int V> __device__ __forceinline__ void read_states(const float *p, float (&v)[V]) {   // from shared memory
    if constexpr (V == 4) {
        const float4 u = *reinterpret_cast<const float4 *>(p);
        v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
    } else {
        const float2 u = *reinterpret_cast<const float2 *>(p);
        v[0] = u.x; v[1] = u.y;
    }
}
template <int V> __device__ __forceinline__ void store_states(float *p, const float (&v)[V]) {
    if constexpr (V == 4) __stcs(reinterpret_cast<float4 *>(p), make_float4(v[0], v[1], v[2], v[3]));
    else __stcs(reinterpret_cast<float2 *>(p), make_float2(v[0], v[1]));
}
// V neighbours of B or C as they lie in memory; `wide`: their address and row
// step allow one access.
template <typename T, int V> struct Narrow {
    static constexpr int W = V * (int)sizeof(T) / 4;
    uint32_t w[W];
    __device__ __forceinline__ void load(const T *p, bool wide) {
        if (wide) {
            if constexpr (W == 4) {
                const uint4 u = __ldg(reinterpret_cast<const uint4 *>(p));
                w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
            } else if constexpr (W == 2) {
                const uint2 u = __ldg(reinterpret_cast<const uint2 *>(p));
                w[0] = u.x; w[1] = u.y;
            } else {
                w[0] = __ldg(reinterpret_cast<const uint32_t *>(p));
            }
        } else if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < W; ++i) w[i] = __ldg(reinterpret_cast<const uint32_t *>(p) + i);
        } else {
            const unsigned short *u = reinterpret_cast<const unsigned short *>(p);
#pragma unroll
            for (int i = 0; i < W; ++i) w[i] = (uint32_t)__ldg(u + 2 * i) | ((uint32_t)__ldg(u + 2 * i + 1) << 16);
        }
    }
    __device__ __forceinline__ float get(int k) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[k]);
        else return __uint_as_float(k % 2 ? w[k / 2] & 0xffff0000u : w[k / 2] << 16);
    }
};

template <typename T, int N, bool kConv> __global__ void __launch_bounds__(kThreads, kMinBlocks) ssm_step_kernel(const SsmParams p, bool wide) {
    constexpr int V = Piece<N>::V, P = Piece<N>::P;
    const int lane = threadIdx.x % 32, q = lane % 4;
    const int ch = (int)blockIdx.x * (kThreads / 4) + threadIdx.x / 4;
    if (ch - lane / 4 >= p.D) return;     // a warp past the last channel
    const bool on = ch < p.D;
    const int c = on ? ch : 0;            // idle lanes mirror channel 0 and store nothing
    // per-thread bases and 32-bit steps: one wide multiply-add an address
    const int ldx = (int)p.ldx, ldt = (int)p.ldt, ldz = (int)p.ldz, ldb = (int)p.ldb, ldc = (int)p.ldc, D = p.D, DN = p.D * N;
    const T *xb = static_cast<const T *>(p.x) + c, *db = static_cast<const T *>(p.dt) + c, *zb = static_cast<const T *>(p.z) + c;
    const T *bb = static_cast<const T *>(p.Bm) + q * V, *cb = static_cast<const T *>(p.Cm) + q * V;
    T *yb = static_cast<T *>(p.y) + c;
    float *hb = p.hT + (size_t)c * N + q * V, *wb = p.win + c;
    Narrow<float, V> a[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        a[i].load(p.A + (size_t)c * N + i * 4 * V + q * V, true);
#pragma unroll
        for (int k = 0; k < V; ++k) a[i].w[k] = __float_as_uint(finite_rate(a[i].get(k)));
    }
    const float bias = p.dt_bias ? p.dt_bias[c] : 0.f, skip = p.skip ? p.skip[c] : 0.f;
    float4 tw = make_float4(0.f, 0.f, 0.f, 0.f);
    float tb = 0.f;
    if (kConv) {
        tw = __ldg(reinterpret_cast<const float4 *>(p.conv_w) + c);
        if (p.conv_b) tb = p.conv_b[c];
    }
    // The states come through a ring of asynchronous copies two groups of four
    // sequences ahead (a lane copies and reads its own); the small inputs one
    // group ahead in registers, the slots two.
    __shared__ __align__(16) float ring[kStages][kSeqs][P][kThreads][V];
    const int step = gridDim.y * kSeqs;
    auto slot_of = [&](int n0) {          // of this lane's sequence; -1: left out
        const int n = n0 + q;
        if (n >= p.nseq) return -1;
        const int slot = p.slots ? p.slots[n] : n;
        if (slot >= 0 && slot < p.n_slots) return slot;
        if (ch == 0) atomicOr(p.status, kDevBadState);
        return -1;
    };
    auto issue = [&](int slot, int stage) {
#pragma unroll
        for (int r = 0; r < kSeqs; ++r) {
            const int at = __shfl_sync(0xffffffffu, slot, r, 4);
            const float *src = hb + (long)max(at, 0) * DN;
#pragma unroll
            for (int i = 0; i < P; ++i) copy_async<V * 4>(&ring[stage][r][i][threadIdx.x][0], src + i * 4 * V, at >= 0);
        }
        copies_commit();
    };
    struct Small {
        float x, dl, z, past[kTaps - 1];
        Narrow<T, V> b[kSeqs][P], cc[kSeqs][P];
    };
    auto fetch = [&](int n0, int slot, Small &v) {
        v.x = v.dl = v.z = v.past[0] = v.past[1] = v.past[2] = 0.f;
        if (slot >= 0) {
            const int n = n0 + q;
            v.x = Elem<T>::load(xb + (long)n * ldx);
            v.dl = Elem<T>::load(db + (long)n * ldt);
            if (p.z) v.z = Elem<T>::load(zb + (long)n * ldz);
            if (kConv) {
                const float *row = wb + (long)slot * (kTaps * D);
#pragma unroll
                for (int j = 0; j < kTaps - 1; ++j) v.past[j] = row[(j + 1) * D];
            }
        }
#pragma unroll
        for (int r = 0; r < kSeqs; ++r) {
            const int nr = min(n0 + r, p.nseq - 1);   // past the end: repeated, and nothing stored
#pragma unroll
            for (int i = 0; i < P; ++i) {
                v.b[r][i].load(bb + (long)nr * ldb + i * 4 * V, wide);
                v.cc[r][i].load(cb + (long)nr * ldc + i * 4 * V, wide);
            }
        }
    };
    int n0 = blockIdx.y * kSeqs, stage = 0;
    int slot = slot_of(n0), slot1 = slot_of(n0 + step);
    issue(slot, 0);
    issue(slot1, 1);
    Small now;
    fetch(n0, slot, now);
#pragma unroll 1
    for (; n0 < p.nseq; n0 += step) {
        const int slot2 = slot_of(n0 + 2 * step);
        Small next;
        fetch(n0 + step, slot1, next);
        const bool live = slot >= 0;
        float u = now.x;
        if (kConv) u = silu(fmaf(tw.w, now.x, fmaf(tw.z, now.past[2], fmaf(tw.y, now.past[1], fmaf(tw.x, now.past[0], tb)))));
        float dl = now.dl + bias;
        if (p.softplus) dl = softplus(dl);
        const float du = dl * u, d2 = dl * kLog2e;
        if (kConv && on && live) {
            float *row = wb + (long)slot * (kTaps * D);
            row[0] = now.past[0];
            row[D] = now.past[1];
            row[2 * D] = now.past[2];
            row[3 * D] = now.x;
        }
        copies_wait<1>();
        float part[kSeqs] = {};
#pragma unroll
        for (int r = 0; r < kSeqs; ++r) {
            const float dr = __shfl_sync(0xffffffffu, d2, r, 4), ur = __shfl_sync(0xffffffffu, du, r, 4);
            const int at = __shfl_sync(0xffffffffu, slot, r, 4);
            float *dst = hb + (long)at * DN;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                float h[V];
                read_states<V>(&ring[stage][r][i][threadIdx.x][0], h);
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    h[k] = fmaf(ex2(dr * a[i].get(k)), h[k], ur * now.b[r][i].get(k));
                    part[r] = fmaf(h[k], now.cc[r][i].get(k), part[r]);
                }
                if (on && at >= 0) store_states<V>(dst + i * 4 * V, h);
            }
        }
        float y = fmaf(skip, u, sum_to_own(part, lane));
        if (p.z) y *= silu(now.z);
        if (on && live) Elem<T>::store(yb + (long)(n0 + q) * D, y);
        issue(slot2, stage == 0 ? kStages - 1 : stage - 1);   // the stage read in the pass before
        stage = stage == kStages - 1 ? 0 : stage + 1;
        slot = slot1;
        slot1 = slot2;
        now = next;
    }
    copies_wait<0>();
}

template <typename T, int N> cudaError_t run(const SsmParams &p, cudaStream_t s, int *launches) {
    constexpr size_t piece = Piece<N>::V * sizeof(T);
    const bool wide = ((reinterpret_cast<uintptr_t>(p.Bm) | reinterpret_cast<uintptr_t>(p.Cm) |
                        (uintptr_t)p.ldb * sizeof(T) | (uintptr_t)p.ldc * sizeof(T)) % piece) == 0;
    const int groups = (p.nseq + kSeqs - 1) / kSeqs, tiles = (p.D + kThreads / 4 - 1) / (kThreads / 4);
    // as many CTAs as the GPU holds at once, each walking every gridDim.y-th
    // group; at N = 32 the ring takes 48 KB, four fit an SM, and the grid is a
    // round and a half
    const int held = kMinBlocks * device_sm_count() / tiles, rows = held > 0 ? held : 1;
    const dim3 grid(tiles, groups < rows ? groups : rows);
    if (p.conv_w) ssm_step_kernel<T, N, true><<<grid, kThreads, 0, s>>>(p, wide);
    else ssm_step_kernel<T, N, false><<<grid, kThreads, 0, s>>>(p, wide);
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
