// tree_common.cuh -- what the kernels over trees of drafted tokens share: a
// sequence's tree, checked, and the walk from a node to the state.
#pragma once

#include "common.cuh"
#include "kernels.h"
#include "ssm_common.cuh"

namespace gla {
namespace tree {

constexpr int kNodes = 64;   // the most a tree may have

// What counts as a bad entry: a sequence's offsets lo, hi and slot, and the parent of node i of its tree.
__device__ __forceinline__ bool bad_entry(const TreeParams &p, int lo, int hi, int slot) {
    return lo < 0 || hi < lo || hi > p.total_T || hi - lo > kNodes || slot < 0 || slot >= p.n_slots;
}
__device__ __forceinline__ bool bad_parent(int parent, int i) { return parent < -1 || parent >= i; }
__device__ __forceinline__ bool bad_last(int last, int nodes) { return last < -1 || last >= nodes; }

struct Tree {
    int first, nodes;   // its first packed node; nodes -1: a bad entry, the sequence is skipped
    size_t slot;
};

// Sequence n's tree, its parents into `par`. All threads of the CTA call it;
// the parents are visible to them when it returns. Every parent lies before
// its node, so walks end.
__device__ __forceinline__ Tree open_tree(const TreeParams &p, int n, int *par) {
    const int a = p.cu[n], b = p.cu[n + 1], slot = p.slots ? p.slots[n] : n;
    int bad = bad_entry(p, a, b, slot);
    Tree t{a, bad ? 0 : b - a, (size_t)slot};
    for (int i = threadIdx.x; i < t.nodes; i += blockDim.x) {
        par[i] = p.parents[a + i];
        bad |= bad_parent(par[i], i);
    }
    if (__syncthreads_or(bad)) t.nodes = -1;
    return t;
}

// The decay of a run of nodes from their log-decays: the sum in a high and a
// low part (in one float, 64 of them would be off by up to 64 half steps of a
// sum of, say, -10, which is 8 units of 2^-24 each in the decay), so that the
// decay has little more than the exponential's own error: 4 units, with its
// last rounding 5. A decay of 0 ends a path; nothing is asked of it behind.
class Decay {
    float hi_ = 0.f, lo_ = 0.f;
    __device__ __forceinline__ float value() const {   // e^(hi + lo)
        const float w = expf(hi_);
        return w == 0.f ? 0.f : fmaf(w, lo_, w);       // (of -inf the low part is NaN)
    }

public:
    __device__ __forceinline__ float then(float log) {   // one more node
        const float s = hi_ + log, t = s - hi_;
        lo_ += (hi_ - (s - t)) + (log - t);
        hi_ = s;
        return value();
    }
    __device__ __forceinline__ float of(int n, float log) {   // n nodes of the same decay
        hi_ = (float)n * log;
        lo_ = fmaf((float)n, log, -hi_);
        return value();
    }
};

// From node i to the state: visit(j, w) for every node j on the path, i first,
// with w the decay of the nodes behind j; `far` gets that of all of them, the
// state's. Returns the visited nodes, one bit each. The walk ends where the
// decay is 0: what lies before it is cleared (far = 0). gate: the nodes' log
// decays, or NULL for the fixed one.
template <typename F>
__device__ __forceinline__ unsigned long long walk(int i, const int *par, const float *gate, float fixed, float &far, F visit) {
    unsigned long long seen = 0;
    Decay decay;
    float w = 1.f;
    int steps = 0;
    for (int j = i; j >= 0; j = par[j]) {
        visit(j, w);
        seen |= 1ull << j;
        w = gate ? decay.then(gate[j]) : decay.of(++steps, fixed);
        if (w == 0.f) break;
    }
    far = w;
    return seen;
}

// The windows of a commit, in pieces of 128 channels of a sequence, a warp each
// (four channels a lane): the last four inputs of the accepted path, before them
// what the window held.
__host__ __device__ __forceinline__ long window_pieces(const TreeParams &p) { return p.x ? p.nseq * ((p.D + 127L) / 128) : 0; }

template <typename T> __device__ __forceinline__ void commit_window(const TreeParams &p, long piece) {
    const int lane = threadIdx.x % 32, per = (int)((p.D + 127L) / 128), n = (int)(piece / per);
    const unsigned c = (unsigned)(piece % per) * 128 + lane * 4;   // (unsigned: the last lanes go past D, which may be next to 2^31)
    const int a = __ldg(p.cu + n), b = __ldg(p.cu + n + 1), slot = p.slots ? __ldg(p.slots + n) : n, last = __ldg(p.last + n);
    bool bad = bad_entry(p, a, b, slot) || bad_last(last, b - a);
    int par[2] = {-1, -1};   // of nodes lane and lane + 32
    if (!bad)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = lane + 32 * e;
            if (i < b - a) par[e] = __ldg(p.parents + a + i);
            bad |= bad_parent(par[e], i);   // (-1 behind the tree)
        }
    if (__any_sync(0xffffffffu, bad)) {
        if (lane == 0) atomicOr(p.status, kDevBadState);
        return;
    }
    if (last < 0) return;
    int at[ssm::kTaps], len = 0;   // the newest first
#pragma unroll
    for (int k = 0, j = last; k < ssm::kTaps; ++k) {
        at[k] = j;
        len += j >= 0;
        const int lo = __shfl_sync(0xffffffffu, par[0], j & 31), hi = __shfl_sync(0xffffffffu, par[1], j & 31);
        if (j >= 0) j = j < 32 ? lo : hi;
    }
    if (c >= (unsigned)p.D) return;
    float *win = p.win + (size_t)slot * ssm::kTaps * p.D + c;
    float4 row[ssm::kTaps];
#pragma unroll
    for (int r = 0; r < ssm::kTaps; ++r) {
        const int back = ssm::kTaps - 1 - r;
        if (back < len) {
            const T *x = static_cast<const T *>(p.x) + (size_t)(a + at[back]) * p.ldx + c;
            if constexpr (sizeof(T) == 2) {
                const uint2 v = *reinterpret_cast<const uint2 *>(x);
                const float2 u = unpack_bf16x2(v.x), w = unpack_bf16x2(v.y);
                row[r] = make_float4(u.x, u.y, w.x, w.y);
            } else {
                row[r] = *reinterpret_cast<const float4 *>(x);
            }
        } else {
            row[r] = *reinterpret_cast<const float4 *>(win + (size_t)(r + len) * p.D);
        }
    }
#pragma unroll
    for (int r = 0; r < ssm::kTaps; ++r) *reinterpret_cast<float4 *>(win + (size_t)r * p.D) = row[r];
}

}  // namespace tree
}  // namespace gla
