// tree_commit.cu -- the accepted path of each drafted tree kept: with j_1 .. j_L
// the path from the state to the accepted node and W_j the decay of the nodes
// behind j,
//     S <- F S + sum_j (W_j k_j) v_j^T        (F the decay of the whole path)
// per sequence and head, and the Conv1d's windows likewise.
//
// A page (96 x 192 fp32) is read and written once: HBM-bound at 12 FMAs an
// entry for a path of a dozen tokens. Persistent, one CTA an SM, hand-overs by
// mbarrier:
//   warps 0-11   two groups of six, half a page (48 rows) each; a thread owns
//                four columns of twelve rows, in registers from load to store;
//   warps 12, 13 the groups' copies: half pages into a ring of two buffers a
//                group, and back, by bulk copies;
//   warps 14-17  the paths, every fourth unit each, ahead of the groups: the
//                walk, the decays, and the path's tokens as fp32 W_j k_j and v_j,
//                eight a piece. (One such warp, whose unit waits for two loads in
//                turn, held the rest up: 583 us.)
//   warps 18, 19 the windows, beside the pages' copies (in a launch of their
//                own before this one: 26 us more).
// 1,280 sequences (1,200 of them keep a path), H = 16, windows of 2,048
// channels: 455 us, 0.94 of the measured copy rate. (A CTA for each page, its
// path found while nothing was in flight: 853 us.)
// Sums in fp32, in the path's order from the accepted node to the state.
#include "ptx.cuh"
#include "tree_common.cuh"

namespace gla {
namespace {

using namespace ptx;
using tree::kNodes;

constexpr int kDk = 96, kDv = 192, kRows = kDk / 2, kGroup = 6, kCompute = 2 * kGroup;
constexpr int kMetas = 4, kWindows = 2, kThreads = (kCompute + 2 + kMetas + kWindows) * 32, kPiece = 8, kOwn = 12;   // kMetas: planners, each with a plan and a piece; kOwn: a thread's rows
constexpr uint32_t kHalf = kRows * kDv * 4, kTokens = kPiece * (kDk + kDv) * 4;
constexpr uint32_t kOffPiece = 4 * kHalf, kOffMeta = kOffPiece + kMetas * kTokens;

struct Meta {
    size_t page;      // its first entry in the pool
    float far;
    int len;          // tokens of the path that count; -1: the page stays
};
// S's buffers: two a group.
enum { FULL_S = 0, DONE_S = FULL_S + 4, FULL_M = DONE_S + 4, FREE_M = FULL_M + kMetas, FULL_T = FREE_M + kMetas, FREE_T = FULL_T + kMetas, BARS = FREE_T + kMetas };
constexpr uint32_t kOffBars = kOffMeta + kMetas * sizeof(Meta), kOffAbort = kOffBars + BARS * 8, kSmem = kOffAbort + 16 + 128;

// The walks of units s, s + kMetas, ... of the CTA, one warp. Offsets are read two of them ahead, parents and decays one.
template <typename T, bool kGate>
__device__ __forceinline__ void planner(const TreeParams &p, unsigned char *sm, uint32_t base, const WaitCtl &ctl, uint32_t units, int s) {
    const int lane = threadIdx.x % 32;
    const uint32_t H = (uint32_t)p.H;
    auto bar = [&](int i) { return base + kOffBars + 8u * (uint32_t)i; };
    auto wait = [&](int b, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar(b), parity, ctl)); };
    struct Offsets {
        int lo, hi, slot, last;
    };
    struct Nodes {
        int first, count, slot, last;   // count -1: a bad entry
        int par[2];                     // of nodes lane and lane + 32
        float gate[2];
    };
    auto offsets = [&](uint32_t u) {
        Offsets r{0, 0, 0, -1};
        if (u < units) {
            const uint32_t n = u / H;
            r.lo = __ldg(p.cu + n);
            r.hi = __ldg(p.cu + n + 1);
            r.slot = p.slots ? __ldg(p.slots + n) : (int)n;
            r.last = __ldg(p.last + n);
        }
        return r;
    };
    auto nodes = [&](uint32_t u, const Offsets &r) {
        Nodes a;
        a.first = r.lo;
        a.slot = r.slot;
        a.last = r.last;
        a.count = tree::bad_entry(p, r.lo, r.hi, r.slot) || tree::bad_last(r.last, r.hi - r.lo) ? -1 : r.hi - r.lo;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = lane + 32 * e;
            const bool in = u < units && i < a.count;
            a.par[e] = in ? __ldg(p.parents + a.first + i) : -1;
            a.gate[e] = kGate && in ? __ldg(p.g + (size_t)(a.first + i) * H + u % H) : 0.f;
        }
        return a;
    };
    const uint32_t start = blockIdx.x + (uint32_t)s * gridDim.x, step = kMetas * gridDim.x;
    Nodes ahead = nodes(start, offsets(start));
    Offsets further = offsets(start + step);
    uint32_t turn = 0, piece = 0;
    for (uint32_t u = start; u < units; u += step, ++turn) {
        const Nodes now = ahead;
        ahead = nodes(u + step, further);
        further = offsets(u + 2 * step);
        const int h = (int)(u % H);
        bool bad = now.count < 0;
#pragma unroll
        for (int e = 0; e < 2; ++e) bad |= tree::bad_parent(now.par[e], lane + 32 * e);   // (-1 behind the tree)
        bad = __any_sync(0xffffffffu, bad);
        if (bad && lane == 0) atomicOr(p.status, kDevBadState);
        // The walk: lane k keeps the path's tokens k and k + 32 and the decays behind them.
        int at[2] = {0, 0}, len = 0;
        float w[2] = {0.f, 0.f}, far = 1.f;
        if (!bad && now.last >= 0) {
            const float fixed = kGate ? 0.f : __ldg(p.log_lambda + h);
            tree::Decay decay;
            for (int j = now.last; j >= 0 && far != 0.f;) {   // a decay of 0 ends it: what lies before is cleared
                if ((len & 31) == lane) {
                    at[len >> 5] = j;
                    w[len >> 5] = far;
                }
                ++len;
                const int up = j < 32 ? __shfl_sync(0xffffffffu, now.par[0], j) : __shfl_sync(0xffffffffu, now.par[1], j - 32);
                if (kGate) far = decay.then(j < 32 ? __shfl_sync(0xffffffffu, now.gate[0], j) : __shfl_sync(0xffffffffu, now.gate[1], j - 32));
                else far = decay.of(len, fixed);
                j = up;
            }
        } else {
            len = -1;
        }
        if (turn > 0 && !wait(FREE_M + s, (turn - 1) & 1u)) return;
        if (lane == 0) {
            Meta *m = reinterpret_cast<Meta *>(sm + kOffMeta) + s;
            m->page = ((size_t)now.slot * p.H + h) * (kDk * kDv);
            m->far = far;
            m->len = len;
            mbar_arrive(bar(FULL_M + s));
        }
        for (int c = 0; c < len; c += kPiece, ++piece) {
            if (piece > 0 && !wait(FREE_T + s, (piece - 1) & 1u)) return;
            float *ks = reinterpret_cast<float *>(sm + kOffPiece + (uint32_t)s * kTokens), *vs = ks + kPiece * kDk;
            for (int b = 0; b < kPiece && c + b < len; b += 4) {   // four tokens' loads in flight
                float kv[4][9], wt[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int x = c + b + e < len ? c + b + e : 0;   // (a token twice rather than a branch)
                    const int j = __shfl_sync(0xffffffffu, x < 32 ? at[0] : at[1], x & 31);
                    wt[e] = __shfl_sync(0xffffffffu, x < 32 ? w[0] : w[1], x & 31);
                    const T *k = static_cast<const T *>(p.k) + (size_t)(now.first + j) * p.ldk + (size_t)h * kDk + lane;
                    const T *v = static_cast<const T *>(p.v) + (size_t)(now.first + j) * p.ldv + (size_t)h * kDv + lane;
#pragma unroll
                    for (int i = 0; i < 3; ++i) kv[e][i] = Elem<T>::load(k + 32 * i);
#pragma unroll
                    for (int i = 0; i < 6; ++i) kv[e][3 + i] = Elem<T>::load(v + 32 * i);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (c + b + e >= len) break;
#pragma unroll
                    for (int i = 0; i < 3; ++i) ks[(b + e) * kDk + lane + 32 * i] = wt[e] * kv[e][i];
#pragma unroll
                    for (int i = 0; i < 6; ++i) vs[(b + e) * kDv + lane + 32 * i] = kv[e][3 + i];
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(FULL_T + s));
        }
    }
}

// A group's copies, one thread: buffer s of unit i is stored when the group is done with it, then takes unit i + 2.
__device__ __forceinline__ void copies(const TreeParams &p, unsigned char *sm, uint32_t base, const WaitCtl &ctl, uint32_t units, int group) {
    auto bar = [&](int i) { return base + kOffBars + 8u * (uint32_t)i; };
    float *held[2] = {nullptr, nullptr};
    int done = 0, it = 0;
    bool ok = true;
    auto store = [&](int i) {   // the i-th unit's half page
        const int s = i & 1;
        ok = mbar_wait(bar(DONE_S + 2 * group + s), (uint32_t)(i >> 1) & 1u, ctl);
        if (!ok) return;
        bulk_store(held[s], base + (uint32_t)(2 * group + s) * kHalf, kHalf);
        tma_store_commit();
    };
    for (uint32_t u = blockIdx.x; u < units; u += gridDim.x, ++it) {
        const int t = it % kMetas, s = done & 1;
        if (!(ok = mbar_wait(bar(FULL_M + t), (uint32_t)(it / kMetas) & 1u, ctl))) break;
        const Meta m = reinterpret_cast<const Meta *>(sm + kOffMeta)[t];
        mbar_arrive(bar(FREE_M + t));
        if (m.len < 0) continue;
        if (done >= 2) {
            store(done - 2);
            if (!ok) break;
            tma_store_wait_read_all();
        }
        held[s] = p.pool + m.page + (size_t)group * kRows * kDv;
        mbar_arrive_expect_tx(bar(FULL_S + 2 * group + s), kHalf);
        bulk_load(base + (uint32_t)(2 * group + s) * kHalf, held[s], kHalf, bar(FULL_S + 2 * group + s));
        ++done;
    }
    for (int i = done > 2 ? done - 2 : 0; i < done && ok; ++i) store(i);
    if (!ok)   // a wait gave up: the copies in flight land before the CTA ends
        for (int i = done > 2 ? done - 2 : 0; i < done; ++i) mbar_wait_drain(bar(FULL_S + 2 * group + (i & 1)), (uint32_t)(i >> 1) & 1u, 1000000ull);
    tma_store_wait_all();
}

template <typename T, bool kGate> __global__ void __launch_bounds__(kThreads, 1) tree_commit_kernel(const TreeParams p) {
    extern __shared__ __align__(128) unsigned char smem_raw[];
    unsigned char *sm = smem_raw + ((128u - (smem_u32(smem_raw) & 127u)) & 127u);
    const uint32_t base = smem_u32(sm);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t units = (uint32_t)p.nseq * (uint32_t)p.H;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + kOffAbort);
    const WaitCtl ctl{abort_flag, p.status};
    auto bar = [&](int i) { return base + kOffBars + 8u * (uint32_t)i; };
    if (threadIdx.x == 0) {
        *abort_flag = 0;
        for (int i = 0; i < BARS; ++i)   // arrivals: one of a copy or the planner, or one a warp (of a plan, the copies' two as well)
            mbar_init(bar(i), i >= FREE_T ? kCompute : i >= FULL_T ? 1 : i >= FREE_M ? kCompute + 2 : i >= FULL_M ? 1 : i >= DONE_S ? kGroup : 1);
        fence_mbar_init();
    }
    __syncthreads();
    if (warp >= kCompute + 2 + kMetas) {
        const long pieces = tree::window_pieces(p);
        for (long i = (long)blockIdx.x * kWindows + warp - (kCompute + 2 + kMetas); i < pieces; i += (long)gridDim.x * kWindows) tree::commit_window<T>(p, i);
    } else if (warp >= kCompute + 2) {
        planner<T, kGate>(p, sm, base, ctl, units, warp - kCompute - 2);
    } else if (warp >= kCompute) {
        if (lane == 0) copies(p, sm, base, ctl, units, warp - kCompute);
    } else {
        const int group = warp / kGroup, t = threadIdx.x - group * kGroup * 32, col = t % (kDv / 4), r0 = t / (kDv / 4) * kOwn;
        auto wait = [&](int b, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar(b), parity, ctl)); };
        int done = 0, it = 0;
        uint32_t turns = 0;   // of each planner's pieces, the parity of those seen
        bool ok = true;
        for (uint32_t u = blockIdx.x; u < units && ok; u += gridDim.x, ++it) {
            const int ms = it % kMetas, s = done & 1;
            if (!wait(FULL_M + ms, (uint32_t)(it / kMetas) & 1u)) break;
            const Meta m = reinterpret_cast<const Meta *>(sm + kOffMeta)[ms];
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(FREE_M + ms));
            if (m.len < 0) continue;
            if (!wait(FULL_S + 2 * group + s, (uint32_t)(done >> 1) & 1u)) break;
            float4 *S = reinterpret_cast<float4 *>(sm + (uint32_t)(2 * group + s) * kHalf) + r0 * (kDv / 4) + col;
            float4 x[kOwn];
#pragma unroll
            for (int i = 0; i < kOwn; ++i) {
                const float4 y = S[i * (kDv / 4)];
                x[i] = m.far == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(m.far * y.x, m.far * y.y, m.far * y.z, m.far * y.w);
            }
            for (int c = 0; c < m.len; c += kPiece, turns ^= 1u << ms) {
                if (!(ok = wait(FULL_T + ms, turns >> ms & 1u))) break;
                const float *ks = reinterpret_cast<const float *>(sm + kOffPiece + (uint32_t)ms * kTokens), *vs = ks + kPiece * kDk;
                const int n = m.len - c < kPiece ? m.len - c : kPiece;
                for (int j = 0; j < n; ++j) {
                    const float4 v = *reinterpret_cast<const float4 *>(vs + j * kDv + 4 * col);
                    const float4 *k4 = reinterpret_cast<const float4 *>(ks + j * kDk + group * kRows + r0);
#pragma unroll
                    for (int i = 0; i < kOwn / 4; ++i) {
                        const float4 k = k4[i];
                        const float kk[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            x[4 * i + e].x = fmaf(kk[e], v.x, x[4 * i + e].x);
                            x[4 * i + e].y = fmaf(kk[e], v.y, x[4 * i + e].y);
                            x[4 * i + e].z = fmaf(kk[e], v.z, x[4 * i + e].z);
                            x[4 * i + e].w = fmaf(kk[e], v.w, x[4 * i + e].w);
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(FREE_T + ms));
            }
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < kOwn; ++i) S[i * (kDv / 4)] = x[i];
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(DONE_S + 2 * group + s));
            ++done;
        }
    }
}

template <typename T> cudaError_t pages(const TreeParams &p, cudaStream_t s, int *launches) {
    auto *kern = p.g ? tree_commit_kernel<T, true> : tree_commit_kernel<T, false>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
    const long units = (long)p.nseq * p.H, pieces = (tree::window_pieces(p) + kWindows - 1) / kWindows, most = device_sm_count();
    const long want = units > pieces ? units : pieces;
    const unsigned grid = (unsigned)(want < most ? want : most);
    kern<<<grid, kThreads, kSmem, s>>>(p);
    if (launches) ++*launches;
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_pages(const TreeParams &p, bool bf16, cudaStream_t s, int *launches) {
    return bf16 ? pages<__nv_bfloat16>(p, s, launches) : pages<float>(p, s, launches);
}

}  // namespace gla
