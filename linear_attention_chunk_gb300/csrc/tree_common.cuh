// tree_common.cuh -- what the kernels over trees of drafted tokens share: a
// sequence's tree, checked, and the walk from a node to the state.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace gla {
namespace tree {

constexpr int kNodes = 64;   // the most a tree may have

struct Tree {
    int first, nodes;   // its first packed node; nodes -1: a bad entry, the sequence is skipped
    size_t slot;
};

// Sequence n's tree, its parents into `par`. All threads of the CTA call it;
// the parents are visible to them when it returns. Every parent lies before
// its node, so walks end.
__device__ __forceinline__ Tree open_tree(const TreeParams &p, int n, int *par) {
    const int a = p.cu[n], b = p.cu[n + 1], slot = p.slots ? p.slots[n] : n;
    int bad = a < 0 || b < a || b > p.total_T || b - a > kNodes || slot < 0 || slot >= p.n_slots;
    Tree t{a, bad ? 0 : b - a, (size_t)slot};
    for (int i = threadIdx.x; i < t.nodes; i += blockDim.x) {
        par[i] = p.parents[a + i];
        bad |= par[i] < -1 || par[i] >= i;
    }
    if (__syncthreads_or(bad)) t.nodes = -1;
    return t;
}

// From node i to the state: visit(j, w) for every node j on the path, i first,
// with w the decay of the nodes behind j; `far` gets that of all of them, the
// state's. Returns the visited nodes, one bit each. The walk ends where the
// decay is 0: what lies before it is cleared (far = 0). gate: the nodes' log
// decays, or NULL for the fixed one, 2^l2.
// The logarithms are added along the path, so that a product of many decays
// has no more error than its sum's.
template <typename F>
__device__ __forceinline__ unsigned long long walk(int i, const int *par, const float *gate, float l2, float &far, F visit) {
    unsigned long long seen = 0;
    float sum = 0.f, w = 1.f;
    int steps = 0;
    for (int j = i; j >= 0; j = par[j]) {
        visit(j, w);
        seen |= 1ull << j;
        if (gate) {
            sum += gate[j];
            w = expf(sum);
        } else {
            w = decay_pow(l2, ++steps);
        }
        if (w == 0.f) break;
    }
    far = w;
    return seen;
}

}  // namespace tree
}  // namespace gla
