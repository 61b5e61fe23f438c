// tree_tc.cu -- the readout of drafted trees at bf16, dk = 96, dv = 192: with
// F_i the decay of the whole path of node i and W_ij that of its nodes behind j,
//     O = scale ( diag(F) Q S + (W o Q K^T) V ),
// W_ij = 0 off the path. Up to 64 nodes share one read of the page S (73,728
// bytes fp32): the pages, q, k, v and o cross HBM once, which is what the call
// cannot do without (56 us for 256 trees of up to 32 nodes, H = 16).
//
// S goes from HBM to the tensor cores by way of shared memory and registers
// alone: six TMA stages of 16 rows (128-byte swizzle), whose entries
// the consumer warps split into two bf16 halves (hi + lo, 16 of an entry's 24
// bits: off by 2^-17 of it) and multiply Q by both; P = W o Q K^T is split
// likewise. Drafted tokens so get what the decode step's fp32 arithmetic gives
// to a few 2^-17 before their one rounding to bf16, which is off by up to 2^-9:
// against 64 bits both are off by 1.7e-3 of the outputs' norm. Three parts each,
// all 24 bits, measured: outputs that differ from fp32's by 3.8e-5 of their norm
// for 9.6e-5 (roundings that fall the other way), the error against 64 bits the
// same, at 75 us on the device for 62.8 (256 trees of up to 32 nodes) and 78 for
// 56.8 (128 of 48 to 64, gated).
// Warp-level products take the halves from registers. tcgen05 has not been
// tried here: S^T's halves as its A operand would go from registers to tensor
// memory, not back to shared memory.
//
// One CTA an SM, no CTA-wide barrier, every hand-over by mbarrier:
//   warp 17      the trees, up to four units (sequence, head) ahead: offsets,
//                parents and decays, the paths as bit masks and running sums by
//                pointer doubling;
//   warp 16      TMA, a unit ahead: 16 rows of q, k or v a copy (a tree's last
//                copy may hold rows of the next one), half of S as it comes free;
//   warps 12-15  P of the unit ahead, 16 x 16 tiles below the diagonal;
//   warps 0-11   16 channels each: Q S step by step, the decay, P V, the rows out.
// 256 trees of up to 32 nodes, H = 16: 65 us a call, 0.86 of the measured copy
// rate; 128 of 48 to 64, gated: 59, 0.71, where the products' 3,600 clocks a
// unit and their latencies show. (Two CTAs of six consumer warps that did all of it in
// turn, P between CTA barriers: 112 and 101. Two groups of consumers a unit
// each, 32 channels a warp: 85 and 80. Three halves of S held, k in one buffer:
// 71 and 63 on the device where these take 62 and 56: the consumers set the pace.)
//
// Accumulator columns: of the two 8-column tiles of a warp, column n of tile t
// is channel 2 n + t. A thread's entries of S are then 8-byte loads (the
// swizzle keeps them free of bank conflicts), and the channels of a row that it
// ends with are four neighbours; four threads store a 32-byte sector.
#include "ptx.cuh"
#include "tmap.h"
#include "tree_common.cuh"

namespace gla {
namespace {

using namespace ptx;
using tree::kNodes;

constexpr int kDk = 96, kDv = 192, kSteps = kDk / 16;
constexpr int kConsumers = 12, kScorers = 4, kThreads = (kConsumers + kScorers + 2) * 32;
constexpr int kMetas = 4, kHalf = kSteps / 2;   // (the stages of S are waited for and released three at a time)
constexpr uint32_t kBox = 16 * 128, kStage = 6 * kBox;   // S: 16 rows x 32 channels; x 192
constexpr uint32_t kTileQ = 16 * kDk * 2, kTileV = 16 * kDv * 2, kNodeQ = kNodes / 16 * kTileQ, kNodeV = kNodes / 16 * kTileV;
constexpr uint32_t kPitchP = kNodes * 2 + 16;   // (16 more: no bank conflicts)
constexpr uint32_t kOffQ = kSteps * kStage, kOffK = kOffQ + 2 * kNodeQ, kOffV = kOffK + 2 * kNodeQ, kOffPh = kOffV + 2 * kNodeV,
                   kOffPl = kOffPh + 2 * kNodes * kPitchP, kOffMeta = kOffPl + 2 * kNodes * kPitchP;   // (a unit's and the next one's)
constexpr float kClear = -104.f;   // e^-104 is 0 in fp32
constexpr float kLog2e = 1.4426950408889634f;

// A unit's tree.
struct Meta {
    unsigned long long path[kNodes];   // the nodes on the path that no decay of 0 cuts off, the node itself included
    float2 sum[kNodes];                // their summed logs (fixed decay: their number), high and low part
    float far[kNodes];                 // the state's decay
    float factor;                      // W_ij = 2^(factor (sum_i - sum_j))
    int first, nodes, row;             // row: the first of its page in the pool, as rows of dv
    int odd;                           // not 0: a score is not finite (as a node's own is where its q is not)
};
enum { FULL_S = 0, EMPTY_S = FULL_S + 2, FULL_M = EMPTY_S + 2, FREE_M = FULL_M + kMetas, FULL_N = FREE_M + kMetas, FULL_P = FULL_N + 2, FREE = FULL_P + 2, BARS = FREE + 2 };
constexpr uint32_t kOffNext = kOffMeta + kMetas * sizeof(Meta), kOffBars = kOffNext + kNodes * 4, kOffAbort = kOffBars + BARS * 8,
                   kSmem = kOffAbort + 16 + 1024;   // (1,024: the base is rounded up for the swizzle)
struct Maps {
    CUtensorMap s, q, k, v;
};
static_assert(kSmem <= 227 * 1024, "shared memory of an SM");

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *m, uint32_t bar, int c0, int c1, int c2) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}
// Rows of q or k: tiles of 16 rows, of which each has three pieces of 32
// columns with the 64-byte swizzle. Address of row r's columns c .. c + 7.
__device__ __forceinline__ uint32_t at_q(uint32_t base, uint32_t r, uint32_t c) {
    return base + (r >> 4) * kTileQ + (c >> 5) * 1024 + sw64_offset(r & 15, (c & 31) >> 3);
}
__device__ __forceinline__ float2 lds2f(uint32_t at) {
    float2 v;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds1(uint32_t at) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}
// Two numbers as their bf16 halves: x = hi + lo up to 2^-17. hi is finite unless x is NaN: of an infinite x (and one that
// bf16 would round to it) it is the largest number, so that lo is what is left and not inf - inf.
__device__ __forceinline__ void split(float x0, float x1, uint32_t &hi, uint32_t &lo) {
    asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(x1), "f"(x0));
    lo = pack_bf16x2(x0 - __uint_as_float(hi << 16), x1 - __uint_as_float(hi & 0xffff0000u));
}
// Zero where an element is not finite.
__device__ __forceinline__ uint32_t finite2(uint32_t a) {
    if ((a & 0x7f80u) == 0x7f80u) a &= 0xffff0000u;
    if ((a & 0x7f800000u) == 0x7f800000u) a &= 0x0000ffffu;
    return a;
}
__device__ __forceinline__ float2 add_parts(float2 a, float2 b) {   // high and low parts, renormalised
    const float s = a.x + b.x, t = s - a.x, e = (a.x - (s - t)) + (b.x - t) + a.y + b.y;
    const float h = s + e;
    return make_float2(h, e - (h - s));
}

// The trees of the units, one warp. A unit's offsets are read two units ahead, its parents and decays one.
template <bool kGate>
__device__ __forceinline__ void planner(const TreeParams &p, unsigned char *sm, uint32_t base, const WaitCtl &ctl, uint32_t units) {
    const int lane = threadIdx.x % 32;
    auto bar = [&](int i) { return base + kOffBars + 8u * (uint32_t)i; };
    int *next = reinterpret_cast<int *>(sm + kOffNext);
    const uint32_t H = (uint32_t)p.H;
    struct Offsets {
        int lo, hi, slot;
    };
    struct Nodes {
        int first, count, slot;   // count -1: a bad offset or slot
        int par[2];               // of nodes lane and lane + 32
        float gate[2];
    };
    auto offsets = [&](uint32_t u) {
        Offsets r{0, 0, 0};
        if (u < units) {
            const uint32_t n = u / H;
            r.lo = __ldg(p.cu + n);
            r.hi = __ldg(p.cu + n + 1);
            r.slot = p.slots ? __ldg(p.slots + n) : (int)n;
        }
        return r;
    };
    auto nodes = [&](uint32_t u, const Offsets &r) {
        Nodes a;
        a.first = r.lo;
        a.slot = r.slot;
        a.count = tree::bad_entry(p, r.lo, r.hi, r.slot) ? -1 : r.hi - r.lo;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = lane + 32 * e;
            const bool in = u < units && i < a.count;
            a.par[e] = in ? __ldg(p.parents + a.first + i) : -1;
            a.gate[e] = kGate && in ? __ldg(p.g + (size_t)(a.first + i) * H + u % H) : 0.f;
        }
        return a;
    };
    Nodes ahead = nodes(blockIdx.x, offsets(blockIdx.x));
    Offsets further = offsets(blockIdx.x + gridDim.x);
    int it = 0;
    for (uint32_t u = blockIdx.x; u < units; u += gridDim.x, ++it) {
        Nodes now = ahead;
        ahead = nodes(u + gridDim.x, further);
        further = offsets(u + 2 * gridDim.x);
        const int h = (int)(u % H), s = it % kMetas;
        bool bad = now.count < 0;
#pragma unroll
        for (int e = 0; e < 2; ++e) bad |= tree::bad_parent(now.par[e], lane + 32 * e);   // (-1 behind the tree)
        if (__any_sync(0xffffffffu, bad)) {
            now.count = 0;
            if (lane == 0) atomicOr(p.status, kDevBadState);
        }
        const int M = now.count;
        if (it >= kMetas && !__all_sync(0xffffffffu, mbar_wait(bar(FREE_M + s), (uint32_t)(it / kMetas - 1) & 1u, ctl))) return;
        Meta *m = reinterpret_cast<Meta *>(sm + kOffMeta) + s;
        const float fixed = kGate ? 0.f : __ldg(p.log_lambda + h);
        const float factor = kGate ? kLog2e : log2_of_decay(fixed);
        // Pointer doubling: node x's path so far, and the node it goes on from (-1: the state, -2: cut off by a decay of 0).
        int ptr[2];
        unsigned long long path[2];
        float2 sum[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int x = lane + 32 * e;
            const bool clears = (kGate ? now.gate[e] : fixed) < kClear;
            ptr[e] = x >= M ? -1 : clears ? -2 : now.par[e];
            path[e] = x < M ? 1ull << x : 0;
            sum[e] = make_float2(clears ? 0.f : kGate ? now.gate[e] : 1.f, 0.f);
            m->path[x] = path[e];
            m->sum[x] = sum[e];
            next[x] = ptr[e];
        }
        __syncwarp();
        while (__any_sync(0xffffffffu, ptr[0] >= 0 || ptr[1] >= 0)) {
            unsigned long long up[2];
            float2 add[2];
            int on[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int x = ptr[e] < 0 ? 0 : ptr[e];
                up[e] = m->path[x];
                add[e] = m->sum[x];
                on[e] = next[x];
            }
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (ptr[e] >= 0) {
                    m->path[lane + 32 * e] = path[e] |= up[e];
                    m->sum[lane + 32 * e] = sum[e] = add_parts(sum[e], add[e]);
                    next[lane + 32 * e] = ptr[e] = on[e];
                }
            __syncwarp();
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) m->far[lane + 32 * e] = ptr[e] == -2 ? 0.f : exp2f((sum[e].x + sum[e].y) * factor);
        if (lane == 0) {
            m->factor = factor;
            m->first = now.first;
            m->nodes = M;
            m->odd = 0;
            m->row = (now.slot * p.H + h) * kDk;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(FULL_M + s));
    }
}

// The copies of the units, one warp.
__device__ __forceinline__ void producer(const Maps &maps, const TreeParams &p, unsigned char *sm, uint32_t base, const WaitCtl &ctl, uint32_t units) {
    const int lane = threadIdx.x % 32;
    auto bar = [&](int i) { return base + kOffBars + 8u * (uint32_t)i; };
    auto wait = [&](int b, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar(b), parity, ctl)); };
    int done = 0, it = 0, halves = 0;   // units with nodes, units, halves of S
    bool ok = true;
    for (uint32_t u = blockIdx.x; u < units; u += gridDim.x, ++it) {
        const int s = it & 1, t = it % kMetas, h = (int)(u % (uint32_t)p.H);
        if (!(ok = wait(FULL_M + t, (uint32_t)(it / kMetas) & 1u))) break;
        const Meta *m = reinterpret_cast<const Meta *>(sm + kOffMeta) + t;
        const int M = m->nodes, first = m->first, row = m->row, tiles = (M + 15) / 16;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(FREE_M + t));
        if (it >= 2 && !(ok = wait(FREE + s, (uint32_t)((it >> 1) - 1) & 1u))) break;
        if (lane == 0) {   // (of an empty tree nothing is copied, but the barriers go on)
            mbar_arrive_expect_tx(bar(FULL_N + s), (uint32_t)tiles * (2 * kTileQ + kTileV));
            for (int i = 0; i < tiles; ++i) {
                const uint32_t at = (uint32_t)s * kNodeQ + (uint32_t)i * kTileQ;
                tma_load_3d(base + kOffQ + at, &maps.q, bar(FULL_N + s), 0, first + i * 16, h * 3);
                tma_load_3d(base + kOffK + at, &maps.k, bar(FULL_N + s), 0, first + i * 16, h * 3);
                tma_load_3d(base + kOffV + (uint32_t)s * kNodeV + (uint32_t)i * kTileV, &maps.v, bar(FULL_N + s), 0, first + i * 16, h * 3);
            }
        }
        if (M == 0) continue;
        for (int half = 0; half < 2; ++half) {
            if (done > 0 && !(ok = wait(EMPTY_S + half, (uint32_t)(done - 1) & 1u))) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(bar(FULL_S + half), kHalf * kStage);
                for (int j = half * kHalf; j < (half + 1) * kHalf; ++j)
                    tma_load_3d(base + (uint32_t)j * kStage, &maps.s, bar(FULL_S + half), 0, row + j * 16, 0);
            }
            ++halves;
        }
        if (!ok) break;
        ++done;
    }
    if (!ok) {   // a wait gave up: the copies in flight land before the CTA ends
        for (int k = halves > 2 ? halves - 2 : 0; k < halves; ++k) mbar_wait_drain(bar(FULL_S + (k & 1)), (uint32_t)(k >> 1) & 1u, 1000000ull);
        for (int k = it > 1 ? it - 1 : 0; k <= it; ++k) mbar_wait_drain(bar(FULL_N + (k & 1)), (uint32_t)(k >> 1) & 1u, 1000000ull);
    }
}

// P of every unit, the tiles dealt out to the scorers' warps.
__device__ __forceinline__ void scorer(unsigned char *sm, uint32_t base, const WaitCtl &ctl, uint32_t units, int warp) {
    const int lane = threadIdx.x % 32, g = lane / 4, q4 = lane % 4;
    const uint32_t a_row = lane % 16, a_col = lane / 16 * 8;                            // ldmatrix: A fragments of 16 rows
    const uint32_t b_row = (lane & 7) + (lane >> 4) * 8, b_col = (lane >> 3 & 1) * 8;   // and B fragments of 16 columns
    auto bar = [&](int i) { return base + kOffBars + 8u * (uint32_t)i; };
    auto wait = [&](int b, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar(b), parity, ctl)); };
    int it = 0;
    for (uint32_t u = blockIdx.x; u < units; u += gridDim.x, ++it) {
        const int s = it & 1, meta = it % kMetas;
        const uint32_t par = (uint32_t)(it >> 1) & 1u;
        if (!wait(FULL_N + s, par)) return;   // (and with it the plan, which the copies' warp has waited for)
        Meta *m = reinterpret_cast<Meta *>(sm + kOffMeta) + meta;
        const int tiles = (m->nodes + 15) / 16;
        const float factor = m->factor;
        float zero = 0.f;   // NaN where a score is not finite
        const uint32_t bQ = base + kOffQ + (uint32_t)s * kNodeQ, bK = base + kOffK + (uint32_t)s * kNodeQ;
        const uint32_t sQ[2] = {at_q(bQ, a_row, a_col), at_q(bQ, a_row, 16 + a_col)}, sK[2] = {at_q(bK, b_row, b_col), at_q(bK, b_row, 16 + b_col)};
        for (int x = warp; x < tiles * (tiles + 1) / 2; x += kScorers) {
            const int ti = x < 1 ? 0 : x < 3 ? 1 : x < 6 ? 2 : 3, tj = x - ti * (ti + 1) / 2;
            float c[2][4] = {};
#pragma unroll
            for (int half = 0; half < kSteps; half += 3) {
                uint32_t a[3][4], b[3][4];
#pragma unroll
                for (int ks = 0; ks < 3; ++ks) {
                    const uint32_t piece = (uint32_t)((half + ks) >> 1) * 1024;
                    ldmatrix4(a[ks], sQ[(half + ks) & 1] + (uint32_t)ti * kTileQ + piece);
                    ldmatrix4(b[ks], sK[(half + ks) & 1] + (uint32_t)tj * kTileQ + piece);
                }
#pragma unroll
                for (int ks = 0; ks < 3; ++ks) {
                    mma16816(c[0], a[ks], b[ks][0], b[ks][1]);
                    mma16816(c[1], a[ks], b[ks][2], b[ks][3]);
                }
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int i = ti * 16 + g + 8 * r;
                const unsigned long long path = m->path[i];
                const float2 si = m->sum[i];
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const int j = tj * 16 + b * 8 + 2 * q4;
                    float v[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float2 sj = m->sum[j + e];
                        const float w = exp2f(((si.x - sj.x) + (si.y - sj.y)) * factor);
                        // (a fixed decay of 0: a node's own weight is 2^(-inf 0))
                        v[e] = !(path >> (j + e) & 1) || w == 0.f ? 0.f : (i == j + e ? 1.f : w) * c[b][2 * r + e];
                    }
                    zero = fmaf(v[1], 0.f, fmaf(v[0], 0.f, zero));
                    uint32_t hi, lo;
                    split(v[0], v[1], hi, lo);
                    const uint32_t at = (uint32_t)(s * kNodes + i) * kPitchP + (uint32_t)j * 2;
                    *reinterpret_cast<uint32_t *>(sm + kOffPh + at) = hi;
                    *reinterpret_cast<uint32_t *>(sm + kOffPl + at) = lo;
                }
            }
        }
        if (zero != 0.f) m->odd = 1;
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(bar(FULL_P + s));
            mbar_arrive(bar(FREE + s));
            mbar_arrive(bar(FREE_M + meta));
        }
    }
}

// A consumer warp's share of a unit of 1 .. 16 kTiles nodes: 16 channels of its rows. Code of its own for each
// number of tiles: without branches, and no longer than it needs to be (a unit runs through it once, so that
// instructions not met cost as much as some that are). False: a wait has given up.
struct Unit {
    unsigned char *sm;
    uint32_t base, x0, x1;   // this thread's entries of a stage
    const Meta *m;
    int s, done, warp;
    uint32_t par;
    size_t row;              // the first node's row of o and of this head
};
// This thread's outputs again (every eighth node from g on, channels 4 q4 .. 4 q4 + 3 of the warp's 16, `o` and `S` their
// columns in the outputs and the page), where a score on a node's path is not finite (its own is not where its q is not) or a v
// there (of a v, in its channel): term by term in fp32. The halves of S and P make NaN of such terms where fp32 makes an
// infinity (inf hi + inf lo is inf - inf where the halves' signs differ, and inf 0 where one is 0), and a v that is not finite
// was left out. Not inline, and its outer loops rolled up: it is rarely called, and its length stands in the readout's way
// (256 trees of up to 32 nodes, on the device: 64.0 us unrolled, 62.8 so). One infinite q among those adds 7 us, NaN in every q 100.
__device__ __noinline__ void term_by_term(const unsigned char *sm, const Meta *m, int s, const float *S, __nv_bfloat16 *o, size_t step, float scale) {
    const int q4 = threadIdx.x % 4, warp = threadIdx.x / 32;
#pragma unroll 1
    for (int x = threadIdx.x % 32 / 4; x < m->nodes; x += 8) {
        const unsigned char *q = sm + kOffQ + (uint32_t)s * kNodeQ;
        const auto pair = [&](int r) { return *reinterpret_cast<const uint32_t *>(q + at_q(0, (uint32_t)x, (uint32_t)r & ~7u) + (uint32_t)(r & 7) * 2); };
        uint32_t odd = 0;   // the channels to form again, one bit each
        bool nan = false;   // a score is: the products have then given NaN everywhere, which stands
        const uint32_t row = (uint32_t)(s * kNodes + x) * kPitchP;
        float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (unsigned long long path = m->path[x]; path; path &= path - 1) {
            const int j = __ffsll((long long)path) - 1;
            const float2 si = m->sum[x], sj = m->sum[j];
            if (j != x && exp2f(((si.x - sj.x) + (si.y - sj.y)) * m->factor) == 0.f) continue;   // (cleared on the way)
            const float w = __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(sm + kOffPh + row + (uint32_t)j * 2)) +
                            __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(sm + kOffPl + row + (uint32_t)j * 2));
            const uint32_t piece = kOffV + (uint32_t)s * kNodeV + (uint32_t)(j >> 4) * kTileV + (uint32_t)(warp / 4) * 2048 + (uint32_t)(j & 15) * 128;
            const uint32_t c16 = ((uint32_t)(warp & 3) * 2 + (uint32_t)(q4 >> 1)) ^ (uint32_t)(j & 7);
            const uint2 v = *reinterpret_cast<const uint2 *>(sm + piece + c16 * 16 + (uint32_t)(q4 & 1) * 8);
            const float2 a = unpack_bf16x2(v.x), b = unpack_bf16x2(v.y);
            const float u[4] = {a.x, a.y, b.x, b.y};
            odd |= isfinite(w) ? 0u : 15u;
            nan |= w != w;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                odd |= isfinite(u[c]) ? 0u : 1u << c;
                y[c] = fmaf(w, u[c], y[c]);
            }
        }
        if (!odd || nan) continue;
        const float far = m->far[x];
        bool open = false;   // a channel to form again that the path has not made NaN
#pragma unroll
        for (int c = 0; c < 4; ++c) open |= (odd >> c & 1) && y[c] == y[c];
        if (open && far != 0.f) {
            float z[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
            for (int r = 0; r < kDk; ++r) {
                const float u = __uint_as_float(r & 1 ? pair(r - 1) & 0xffff0000u : pair(r) << 16);
                const float4 a = __ldg(reinterpret_cast<const float4 *>(S + (size_t)r * kDv));
                z[0] = fmaf(u, a.x, z[0]);
                z[1] = fmaf(u, a.y, z[1]);
                z[2] = fmaf(u, a.z, z[2]);
                z[3] = fmaf(u, a.w, z[3]);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) y[c] = fmaf(far, z[c], y[c]);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (odd >> c & 1) o[(size_t)x * step + c] = __float2bfloat16_rn(scale * y[c]);
    }
}
template <int kTiles> __device__ __forceinline__ bool readout(const TreeParams &p, const Unit &unit, const WaitCtl &ctl) {
    const int lane = threadIdx.x % 32, g = lane / 4, q4 = lane % 4;   // a fragment's row (or column), its pair of columns (or rows)
    const uint32_t a_row = lane % 16, a_col = lane / 16 * 8, base = unit.base, x0 = unit.x0, x1 = unit.x1, par = unit.par;
    const int s = unit.s, done = unit.done, warp = unit.warp, M = unit.m->nodes;
    const Meta *m = unit.m;
    unsigned char *sm = unit.sm;
    auto bar = [&](int i) { return base + kOffBars + 8u * (uint32_t)i; };
    auto wait = [&](int b, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar(b), parity, ctl)); };
    // q's fragments of even and odd steps: all else of their addresses is constant
    const uint32_t sQ[2] = {at_q(base + kOffQ + (uint32_t)s * kNodeQ, a_row, a_col), at_q(base + kOffQ + (uint32_t)s * kNodeQ, a_row, 16 + a_col)};
    float acc[kTiles][2][4];
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[i][t][c] = 0.f;
    const auto entries = [&](int ks, float2 (&y)[4]) {
        const uint32_t st = (uint32_t)ks * kStage;
        y[0] = lds2f(x0 + st);
        y[1] = lds2f(x1 + st);
        y[2] = lds2f(x0 + st + 1024);
        y[3] = lds2f(x1 + st + 1024);
    };
    if (!wait(FULL_S, (uint32_t)done & 1u)) return false;
    float2 y[2][4];   // a step's and the next one's
    entries(0, y[0]);
#pragma unroll
    for (int ks = 0; ks < kSteps; ++ks) {
        if (ks == kHalf - 1 && !wait(FULL_S + 1, (uint32_t)done & 1u)) return false;
        if (ks < kSteps - 1) entries(ks + 1, y[(ks + 1) & 1]);
        const float2(&now)[4] = y[ks & 1];
        uint32_t hi[2][2], lo[2][2];
        split(now[0].x, now[1].x, hi[0][0], lo[0][0]);
        split(now[0].y, now[1].y, hi[1][0], lo[1][0]);
        split(now[2].x, now[3].x, hi[0][1], lo[0][1]);
        split(now[2].y, now[3].y, hi[1][1], lo[1][1]);
        if (ks % kHalf == kHalf - 1) {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(EMPTY_S + ks / kHalf));
        }
        uint32_t a[kTiles][4];
#pragma unroll
        for (int i = 0; i < kTiles; ++i)
            ldmatrix4(a[i], sQ[ks & 1] + (uint32_t)i * kTileQ + (uint32_t)(ks >> 1) * 1024);
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
            mma16816(acc[i][0], a[i], hi[0][0], hi[0][1]);
            mma16816(acc[i][1], a[i], hi[1][0], hi[1][1]);
        }
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
            mma16816(acc[i][0], a[i], lo[0][0], lo[0][1]);
            mma16816(acc[i][1], a[i], lo[1][0], lo[1][1]);
        }
    }
    // the state's decay: 0 clears it, whatever it holds
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
        const float f[2] = {m->far[i * 16 + g], m->far[i * 16 + g + 8]};
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[i][t][c] *= f[c >> 1];
        if (__any_sync(0xffffffffu, f[0] == 0.f || f[1] == 0.f)) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[i][t][c] = f[c >> 1] == 0.f ? 0.f : acc[i][t][c];
        }
    }
    // P V: 16 nodes j at a time
    if (!wait(FULL_P + s, par)) return false;
    // (of a tile of v, three pieces of 64 channels with the 128-byte swizzle; channels 2 g, 2 g + 1 of the warp's 16)
    const uint32_t bV = base + kOffV + (uint32_t)s * kNodeV + (uint32_t)(warp / 4) * 2048 + (uint32_t)(g & 3) * 4, cV = (uint32_t)(warp & 3) * 2 + (uint32_t)(g >> 2);
    const uint32_t sV[2] = {bV + (uint32_t)(2 * q4) * 128 + ((cV ^ (uint32_t)(2 * q4)) << 4), bV + (uint32_t)(2 * q4 + 1) * 128 + ((cV ^ (uint32_t)(2 * q4 + 1)) << 4)};
    const uint32_t sP = base + kOffPh + ((uint32_t)s * kNodes + a_row) * kPitchP + a_col * 2;
    bool dirty = false;
#pragma unroll
    for (int js = 0; js < kTiles; ++js) {
        uint32_t x[4], odd = 0;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int j = 2 * q4 + (r & 1) + (r >> 1) * 8;
            x[r] = lds1(sV[r & 1] + (uint32_t)js * kTileV + (uint32_t)(r >> 1) * 1024);
            if (js * 16 + j >= M) x[r] = 0;             // (rows of another tree)
            odd |= mul_bf16x2(x[r], 0) & 0x7fff7fffu;        // not 0: an element that is not finite
        }
        // One that is not finite would reach every node by way of 0 x inf: it is left out here, its paths' nodes come again below.
        if (__any_sync(0xffffffffu, odd != 0)) {
            dirty = true;
#pragma unroll
            for (int r = 0; r < 4; ++r) x[r] = finite2(x[r]);
        }
        uint32_t b[2][2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            b[0][r] = __byte_perm(x[2 * r], x[2 * r + 1], 0x5410);
            b[1][r] = __byte_perm(x[2 * r], x[2 * r + 1], 0x7632);
        }
#pragma unroll
        for (int part = 0; part < 2; ++part) {
            uint32_t a[kTiles][4];
#pragma unroll
            for (int i = js; i < kTiles; ++i)
                ldmatrix4(a[i], sP + (uint32_t)part * (kOffPl - kOffPh) + (uint32_t)i * 16 * kPitchP + (uint32_t)js * 32);
#pragma unroll
            for (int i = js; i < kTiles; ++i) {
                mma16816(acc[i][0], a[i], b[0][0], b[0][1]);
                mma16816(acc[i][1], a[i], b[1][0], b[1][1]);
            }
        }
    }
    const size_t step = (size_t)p.H * kDv;
    __nv_bfloat16 *const first = static_cast<__nv_bfloat16 *>(p.o) + unit.row * kDv + warp * 16 + 4 * q4, *o = first + (size_t)g * step;
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int r = 0; r < 2; ++r, o += 8 * step) {
            const int x = i * 16 + g + 8 * r;
            if (x >= M) continue;
            *reinterpret_cast<uint2 *>(o) =
                make_uint2(pack_bf16x2(p.scale * acc[i][0][2 * r], p.scale * acc[i][1][2 * r]),
                           pack_bf16x2(p.scale * acc[i][0][2 * r + 1], p.scale * acc[i][1][2 * r + 1]));
        }
    if (dirty || m->odd) term_by_term(sm, m, s, p.pool + (size_t)m->row * kDv + warp * 16 + 4 * q4, first, step, p.scale);
    return true;
}

template <bool kGate> __global__ void __launch_bounds__(kThreads, 1) tree_fwd_tc_kernel(const __grid_constant__ Maps maps, const TreeParams p) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t base = smem_u32(sm);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t units = (uint32_t)p.nseq * (uint32_t)p.H;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + kOffAbort);
    const WaitCtl ctl{abort_flag, p.status};
    auto bar = [&](int i) { return base + kOffBars + 8u * (uint32_t)i; };
    if (threadIdx.x == 0) {
        *abort_flag = 0;
        for (int i = 0; i < BARS; ++i)   // arrivals: one of a copy or the producer, or one a warp
            mbar_init(bar(i), i >= FREE ? kConsumers + kScorers : i >= FULL_P ? kScorers : i >= FREE_M && i < FULL_N ? kConsumers + kScorers + 1
                              : i >= EMPTY_S && i < FULL_M ? kConsumers : 1);
        fence_mbar_init();
        prefetch_tmap(&maps.s);
        prefetch_tmap(&maps.q);
        prefetch_tmap(&maps.k);
        prefetch_tmap(&maps.v);
    }
    __syncthreads();
    if (warp == kConsumers + kScorers + 1) {
        planner<kGate>(p, sm, base, ctl, units);
        return;
    }
    if (warp == kConsumers + kScorers) {
        producer(maps, p, sm, base, ctl, units);
        return;
    }
    if (warp >= kConsumers) {
        scorer(sm, base, ctl, units, warp - kConsumers);
        return;
    }
    const int g = lane / 4, q4 = lane % 4;   // a fragment's row (or column), its pair of columns (or rows)
    // This thread's entries of a stage: channels 2 g, 2 g + 1 of the warp's 16, rows 2 q4, 2 q4 + 1 and eight below those
    const uint32_t box = base + (uint32_t)(warp / 2) * kBox + (uint32_t)(g & 1) * 8, chunk = (uint32_t)(warp & 1) * 4 + (uint32_t)(g >> 1);
    const uint32_t x0 = box + (uint32_t)(2 * q4) * 128 + ((chunk ^ (uint32_t)(2 * q4)) << 4);
    const uint32_t x1 = box + (uint32_t)(2 * q4 + 1) * 128 + ((chunk ^ (uint32_t)(2 * q4 + 1)) << 4);
    auto wait = [&](int b, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar(b), parity, ctl)); };
    int done = 0, it = 0;
    for (uint32_t u = blockIdx.x; u < units; u += gridDim.x, ++it) {
        const int s = it & 1, meta = it % kMetas;
        const uint32_t par = (uint32_t)(it >> 1) & 1u;
        if (!wait(FULL_N + s, par)) return;   // (and with it the plan, which the copies' warp has waited for)
        const Meta *m = reinterpret_cast<const Meta *>(sm + kOffMeta) + meta;
        const int M = m->nodes;
        if (M > 0) {
            const Unit unit{sm, base, x0, x1, m, s, done, warp, par, (size_t)m->first * p.H + u % (uint32_t)p.H};
            if (!(M <= 16 ? readout<1>(p, unit, ctl) : M <= 32 ? readout<2>(p, unit, ctl) : M <= 48 ? readout<3>(p, unit, ctl) : readout<4>(p, unit, ctl))) return;
            ++done;
        }
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(bar(FREE + s));
            mbar_arrive(bar(FREE_M + meta));
        }
    }
}

// A map of three dimensions, each of them `dims` elements `strides` bytes apart (the first contiguous).
bool make_map(CUtensorMap *m, CUtensorMapDataType type, const void *at, cuuint64_t d0, cuuint64_t d1, cuuint64_t s1, cuuint64_t d2,
              cuuint64_t s2, cuuint32_t b0, cuuint32_t b1, cuuint32_t b2, CUtensorMapSwizzle swizzle) {
    const cuuint64_t dims[3] = {d0, d1, d2}, strides[2] = {s1, s2};
    const cuuint32_t box[3] = {b0, b1, b2}, es[3] = {1, 1, 1};
    return encode_tiled_fn()(m, type, 3, const_cast<void *>(at), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t launch_tree_fwd_tc(const TreeParams &p, cudaStream_t s, int *launches) {
    if (!encode_tiled_fn()) return cudaErrorNotSupported;
    Maps maps;
    const cuuint64_t T = (cuuint64_t)p.total_T, H = (cuuint64_t)p.H;
    const auto bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    if (!make_map(&maps.s, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, p.pool, 32, (p.n_slots > 0 ? (cuuint64_t)p.n_slots : 1) * H * kDk, kDv * 4, 6, 128, 32, 16, 6, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map(&maps.q, bf16, p.q, 32, T, (cuuint64_t)p.ldq * 2, 3 * H, 64, 32, 16, 3, CU_TENSOR_MAP_SWIZZLE_64B) ||
        !make_map(&maps.k, bf16, p.k, 32, T, (cuuint64_t)p.ldk * 2, 3 * H, 64, 32, 16, 3, CU_TENSOR_MAP_SWIZZLE_64B) ||
        !make_map(&maps.v, bf16, p.v, 64, T, (cuuint64_t)p.ldv * 2, 3 * H, 128, 64, 16, 3, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    auto *kern = p.g ? tree_fwd_tc_kernel<true> : tree_fwd_tc_kernel<false>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
    const long units = (long)p.nseq * p.H, most = device_sm_count();
    kern<<<(unsigned)(units < most ? units : most), kThreads, kSmem, s>>>(maps, p);
    if (launches) ++*launches;
    return cudaGetLastError();
}

}  // namespace gla
