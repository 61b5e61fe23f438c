// pages.cu -- the pages of the serving loop's pools (states, conv windows):
// copied (a prompt continued several times), cleared (a new sequence's page
// holds zeros) and moved to the front (holes closed up), in the pools of
// several layers at once. Pure HBM streams: a page's bytes read and written.
//
// The pages are cut into chunks of 32 KB, taken in turn by resident CTAs; a
// thread's loads of a chunk are all in flight before its stores. Chunk by
// chunk, the pairs of one chunk side by side: several copies of one page read
// it from L2 after the first.
//
// Compaction: with L pages in use, those at or above L move into the free ones
// below it, in ascending order both. One CTA ranks them by ballots and lists
// the moves; the copy reads the list and its length on the device.
#include "ssm_common.cuh"

namespace gla {
namespace {

constexpr int kThreads = 256, kUnroll = 8, kChunk = kThreads * kUnroll * 16;
constexpr int kPlan = 1024;

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

// kList: the pairs are the plan's, their number too.
template <bool kList> __global__ void __launch_bounds__(kThreads) pages_kernel(const PageParams p, const Cut cut) {
    if (kList) ssm::wait_for_previous();
    const int half = p.n_slots / 2 + 1;
    const int pairs = kList ? __ldcg(p.moves + 2 * half) : p.n;
    const int *srcs = kList ? p.moves : p.src, *dsts = kList ? p.moves + half : p.dst;
    const long items = (long)cut.first[p.n_pools] * pairs;
    for (long item = blockIdx.x; item < items; item += gridDim.x) {
        const int chunk = (int)(item / pairs), i = (int)(item % pairs);
        const int dst = kList ? __ldcg(dsts + i) : dsts[i], src = !srcs ? dst : kList ? __ldcg(srcs + i) : srcs[i];
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

// Exclusive sum of a flag over the CTA, in thread order; `all` gets the total.
__device__ __forceinline__ int rank_of(bool flag, int &all, int *s) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const unsigned m = __ballot_sync(0xffffffffu, flag);
    if (lane == 0) s[warp] = __popc(m);
    __syncthreads();
    int before = 0;
    all = 0;
    for (int w = 0; w < kPlan / 32; ++w) {
        if (w < warp) before += s[w];
        all += s[w];
    }
    __syncthreads();
    return before + __popc(m & ((1u << lane) - 1));
}

__global__ void __launch_bounds__(kPlan) plan_kernel(const PageParams p) {
    __shared__ int s[kPlan / 32];
    __shared__ int s_holes;
    ssm::let_next_start();
    const int half = p.n_slots / 2 + 1;
    int *srcs = p.moves, *dsts = p.moves + half;
    int live = 0;
    for (int i = threadIdx.x; i < p.n_slots; i += kPlan) live += p.live[i] != 0;
    live = __reduce_add_sync(0xffffffffu, live);
    if (threadIdx.x % 32 == 0) s[threadIdx.x / 32] = live;
    __syncthreads();
    live = 0;
    for (int w = 0; w < kPlan / 32; ++w) live += s[w];
    __syncthreads();
    int holes = 0, far = 0;
    for (int base = 0; base < p.n_slots; base += kPlan) {
        const int i = base + threadIdx.x;
        const bool in = i < p.n_slots, on = in && p.live[i] != 0;
        const bool hole = in && !on && i < live, moves = on && i >= live;
        int n;
        const int a = holes + rank_of(hole, n, s);
        holes += n;
        const int b = far + rank_of(moves, n, s);
        far += n;
        if (hole) dsts[a] = i;
        if (moves) srcs[b] = i;
        if (in) p.map[i] = on ? i : -1;
    }
    if (threadIdx.x == 0) {
        s_holes = holes;
        p.moves[2 * half] = holes;
        *p.count = live;
    }
    __syncthreads();     // the lists and the map are visible to this CTA
    for (int j = threadIdx.x; j < s_holes; j += kPlan) p.map[srcs[j]] = dsts[j];
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
    pages_kernel<false><<<grid_of(items), kThreads, 0, s>>>(p, cut);
    if (launches) ++*launches;
    return cudaGetLastError();
}

cudaError_t launch_pages_compact(PageParams &p, cudaStream_t s, int *launches) {
    const Cut cut = cut_of(p);
    plan_kernel<<<1, kPlan, 0, s>>>(p);
    cudaError_t e = cudaGetLastError();
    if (launches) ++*launches;
    const long items = (long)cut.first[p.n_pools] * (p.n_slots / 2);
    if (e != cudaSuccess || items == 0) return e;
    e = ssm::launch_behind(pages_kernel<true>, dim3(grid_of(items)), kThreads, 0, s, p, cut);
    if (e == cudaSuccess && launches) ++*launches;
    return e;
}

}  // namespace gla
