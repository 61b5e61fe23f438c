// pages.cu -- the pages of the serving loop's pools (states, conv windows):
// copied (a prompt continued several times), cleared (a new sequence's page
// holds zeros) and moved to the front (holes closed up), in the pools of
// several layers at once. Pure HBM streams: a page's bytes read and written.
//
// The pages are cut into chunks of 32 KB, taken in turn by resident CTAs; a
// thread's loads of a chunk are all in flight before its stores (a ring of
// bulk copies through shared memory, one thread an SM, measured the same: 140
// us for 0.87 GB moved, 0.92 of the measured copy rate). Chunk by chunk, the
// pairs of one chunk side by side: several copies of one page read it from L2
// after the first.
//
// Compaction: with L pages in use, those at or above L move into the free ones
// below it, in ascending order both. Ranks come from ballots. Of pools of up to
// 4,096 pages every copying CTA works out the moves for itself (a launch of its
// own before the copy, 256 pages in six layers: 146 us for 140); of larger
// ones one CTA lists them in the workspace and the copy reads the list and its
// length there.
#include "ssm_common.cuh"

namespace gla {
namespace {

constexpr int kThreads = 256, kUnroll = 8, kChunk = kThreads * kUnroll * 16;
constexpr int kPlan = 1024, kOwnPlan = 4096;   // the listing CTA's threads; the most pages of a pool whose moves each CTA works out

struct Cut {
    int first[kMaxPools + 1];   // chunks of a page before each pool's
};

template <typename V> __device__ __forceinline__ void move_chunk(const char *src, char *dst, long bytes) {
    const V *a = reinterpret_cast<const V *>(src);
    V *b = reinterpret_cast<V *>(dst);
    const int n = (int)(bytes / (long)sizeof(V));
    for (int i = threadIdx.x; i < n; i += kThreads * kUnroll) {
        V v[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (src && i + u * kThreads < n) v[u] = __ldcs(a + i + u * kThreads);
            else v[u] = V{};
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (i + u * kThreads < n) __stcs(b + i + u * kThreads, v[u]);
    }
}

// Exclusive sum of a flag over the CTA, in thread order; `all` gets the total.
template <int kCta> __device__ __forceinline__ int rank_of(bool flag, int &all, int *s) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const unsigned m = __ballot_sync(0xffffffffu, flag);
    if (lane == 0) s[warp] = __popc(m);
    __syncthreads();
    int before = 0;
    all = 0;
    for (int w = 0; w < kCta / 32; ++w) {
        if (w < warp) before += s[w];
        all += s[w];
    }
    __syncthreads();
    return before + __popc(m & ((1u << lane) - 1));
}

// The moves: sources, targets; returns how many. `live` gets the number of pages in use. Page numbers are unsigned
// here and in write_map: of up to 2^31 - 1 pages, the last step of a thread goes past an int.
template <int kCta> __device__ __forceinline__ int make_plan(const PageParams &p, int *srcs, int *dsts, int *s, int &live) {
    live = 0;
    const unsigned slots = (unsigned)p.n_slots;
    for (unsigned i = threadIdx.x; i < slots; i += kCta) live += p.live[i] != 0;
    live = __reduce_add_sync(0xffffffffu, live);
    if (threadIdx.x % 32 == 0) s[threadIdx.x / 32] = live;
    __syncthreads();
    live = 0;
    for (int w = 0; w < kCta / 32; ++w) live += s[w];
    __syncthreads();
    int holes = 0, far = 0;
    for (unsigned base = 0; base < slots; base += kCta) {
        const unsigned i = base + threadIdx.x;
        const bool in = i < slots, on = in && p.live[i] != 0;
        const bool hole = in && !on && i < (unsigned)live, moves = on && i >= (unsigned)live;
        int n;
        const int a = holes + rank_of<kCta>(hole, n, s);
        holes += n;
        const int b = far + rank_of<kCta>(moves, n, s);
        far += n;
        if (hole) dsts[a] = (int)i;
        if (moves) srcs[b] = (int)i;
    }
    __syncthreads();
    return holes;
}
// The pages' new numbers, and how many are in use.
__device__ __forceinline__ void write_map(const PageParams &p, const int *srcs, const int *dsts, int moves, int live) {
    for (unsigned i = threadIdx.x; i < (unsigned)p.n_slots; i += blockDim.x) p.map[i] = p.live[i] ? (int)i : -1;
    if (threadIdx.x == 0) *p.count = live;
    __syncthreads();
    for (int j = threadIdx.x; j < moves; j += blockDim.x) p.map[srcs[j]] = dsts[j];
}

// Where a copy's pairs come from: the caller, the listing launch, this CTA.
enum Pairs { kGiven, kListed, kOwn };

template <Pairs kFrom> __global__ void __launch_bounds__(kThreads) pages_kernel(const PageParams p, const Cut cut) {
    __shared__ int s_src[kFrom == kOwn ? kOwnPlan / 2 : 1], s_dst[kFrom == kOwn ? kOwnPlan / 2 : 1], s_rank[kThreads / 32];
    const int half = p.n_slots / 2 + 1;
    const int *srcs = p.src, *dsts = p.dst;
    int pairs = p.n;
    if constexpr (kFrom == kListed) {
        ssm::wait_for_previous();
        pairs = __ldcg(p.moves + 2L * half);
        srcs = p.moves;
        dsts = p.moves + half;
    } else if constexpr (kFrom == kOwn) {
        int live;
        pairs = make_plan<kThreads>(p, s_src, s_dst, s_rank, live);
        srcs = s_src;
        dsts = s_dst;
        if (blockIdx.x == 0) write_map(p, srcs, dsts, pairs, live);
    }
    const long items = (long)cut.first[p.n_pools] * pairs;
    for (long item = blockIdx.x; item < items; item += gridDim.x) {
        const int chunk = (int)(item / pairs), i = (int)(item % pairs);
        const int dst = kFrom == kListed ? __ldcg(dsts + i) : dsts[i], src = !srcs ? dst : kFrom == kListed ? __ldcg(srcs + i) : srcs[i];
        if (dst < 0 || dst >= p.n_slots || src < 0 || src >= p.n_slots) {
            if (threadIdx.x == 0) atomicOr(p.status, kDevBadState);
            continue;
        }
        if (srcs && src == dst) continue;
        int k = 0;
        while (chunk >= cut.first[k + 1]) ++k;
        const long at = (long)(chunk - cut.first[k]) * kChunk;
        const long bytes = p.bytes[k] - at < kChunk ? p.bytes[k] - at : kChunk;
        char *to = static_cast<char *>(p.pool[k]) + (size_t)dst * p.bytes[k] + at;
        const char *from = srcs ? static_cast<const char *>(p.pool[k]) + (size_t)src * p.bytes[k] + at : nullptr;
        if (p.bytes[k] % 16 == 0) move_chunk<int4>(from, to, bytes);
        else move_chunk<int>(from, to, bytes);
    }
}

__global__ void __launch_bounds__(kPlan) plan_kernel(const PageParams p) {
    __shared__ int s[kPlan / 32];
    ssm::let_next_start();
    const int half = p.n_slots / 2 + 1;
    int *srcs = p.moves, *dsts = p.moves + half, live;
    const int moves = make_plan<kPlan>(p, srcs, dsts, s, live);
    if (threadIdx.x == 0) p.moves[2L * half] = moves;
    write_map(p, srcs, dsts, moves, live);
}

int grid_of(long items) {
    const long most = 8L * device_sm_count();   // 2,048 threads an SM
    return (int)(items < most ? items : most);
}

Cut cut_of(const PageParams &p) {
    Cut c;
    c.first[0] = 0;
    for (int k = 0; k < p.n_pools; ++k) c.first[k + 1] = c.first[k] + (int)((p.bytes[k] + kChunk - 1) / kChunk);
    return c;
}

}  // namespace

cudaError_t launch_pages_move(const PageParams &p, cudaStream_t s, int *launches) {
    const Cut cut = cut_of(p);
    const long items = (long)cut.first[p.n_pools] * p.n;
    if (items == 0) return cudaSuccess;
    pages_kernel<kGiven><<<grid_of(items), kThreads, 0, s>>>(p, cut);
    if (launches) ++*launches;
    return cudaGetLastError();
}

bool pages_plan_listed(int n_slots) { return n_slots > kOwnPlan; }

cudaError_t launch_pages_compact(PageParams &p, cudaStream_t s, int *launches) {
    const Cut cut = cut_of(p);
    const long items = (long)cut.first[p.n_pools] * (p.n_slots / 2);
    if (!pages_plan_listed(p.n_slots)) {   // (at least one CTA, for the map)
        pages_kernel<kOwn><<<grid_of(items > 0 ? items : 1), kThreads, 0, s>>>(p, cut);
        if (launches) ++*launches;
        return cudaGetLastError();
    }
    plan_kernel<<<1, kPlan, 0, s>>>(p);
    cudaError_t e = cudaGetLastError();
    if (launches) ++*launches;
    if (e != cudaSuccess || items == 0) return e;
    e = ssm::launch_behind(pages_kernel<kListed>, dim3(grid_of(items)), kThreads, 0, s, p, cut);
    if (e == cudaSuccess && launches) ++*launches;
    return e;
}

}  // namespace gla
