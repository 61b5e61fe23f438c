// tree.cu -- trees of drafted tokens over the state pool: the serving steps of
// speculative decoding, where a draft model proposes a tree of tokens for each
// sequence, the model scores all of them at once, and the path that is
// accepted is kept. Per sequence and head, for node i with parent p(i) (-1:
// the sequence's state page S itself):
//     S_i = exp(g_i) S_p(i) + k_i v_i^T,   S_-1 = S,   o_i = scale S_i^T q_i
// (g_i = log_lambda[h] for the fixed per-head decay). Unrolled along the path
// from the state to i, with D_i the decay of all its nodes and W_ij that of
// the nodes behind j, up to i:
//     o_i = scale ( D_i S^T q_i + sum_{j on the path} W_ij (q_i . k_j) v_j ),
// so no node's state is formed and the page is read once for all of them.
// A decay of 0 clears what lies before it, also where that is not finite.
// The commit forms S_last alone and stores it; the convolution in front of the
// mixer reads the last three inputs of each node's path, behind the root those
// of the sequence's window.
#include "ssm_common.cuh"
#include "tree_common.cuh"

namespace gla {
namespace {

using namespace tree;

constexpr int kThreads = 256;

// A row of q or k in shared memory: an odd number of 16-byte pieces, so that neighbours' rows start in different banks.
__host__ __device__ constexpr int padded(int v) { return ((v + 3) / 4 | 1) * 4; }

// A thread's sums over the state and the path: kBlock nodes at a time, two columns `lanes` apart.
struct Sums {
    const float *qs, *P, *far, *S, *v;
    const unsigned long long *path;
    float *o;
    int M, ldq, dk, dv, lanes;
    size_t ldv, ldo;
    float scale;
    bool second;   // the second column exists
};
template <int kBlock> __device__ __forceinline__ void sum_nodes(const Sums &a, int grp, int groups) {
    for (int nb = grp * kBlock; nb < a.M; nb += groups * kBlock) {
        float acc[kBlock][2] = {};
        for (int r = 0; r < a.dk; r += 4) {
            float s[4][2];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                s[u][0] = r + u < a.dk ? __ldg(a.S + (size_t)(r + u) * a.dv) : 0.f;
                s[u][1] = r + u < a.dk && a.second ? __ldg(a.S + (size_t)(r + u) * a.dv + a.lanes) : 0.f;
            }
#pragma unroll
            for (int i = 0; i < kBlock; ++i) {
                const float4 q = *reinterpret_cast<const float4 *>(a.qs + (nb + i) * a.ldq + r);
#pragma unroll
                for (int x = 0; x < 2; ++x) acc[i][x] = fmaf(q.x, s[0][x], fmaf(q.y, s[1][x], fmaf(q.z, s[2][x], fmaf(q.w, s[3][x], acc[i][x]))));
            }
        }
#pragma unroll
        for (int i = 0; i < kBlock; ++i) {
            if (nb + i >= a.M) break;
            const float far = a.far[nb + i];
            float y0 = far == 0.f ? 0.f : far * acc[i][0], y1 = far == 0.f ? 0.f : far * acc[i][1];
            for (unsigned long long m = a.path[nb + i]; m;) {   // four of the path's nodes at a time, their loads in flight together
                float w[4], v0[4], v1[4];
                bool in[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    in[u] = m != 0;
                    const int j = in[u] ? __ffsll((long long)m) - 1 : 0;
                    m &= m - 1;
                    w[u] = in[u] ? a.P[(nb + i) * kNodes + j] : 0.f;
                    v0[u] = in[u] ? __ldg(a.v + (size_t)j * a.ldv) : 0.f;
                    v1[u] = in[u] && a.second ? __ldg(a.v + (size_t)j * a.ldv + a.lanes) : 0.f;
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    y0 = fmaf(w[u], v0[u], y0);
                    y1 = fmaf(w[u], v1[u], y1);
                }
            }
            a.o[(size_t)(nb + i) * a.ldo] = a.scale * y0;
            if (a.second) a.o[(size_t)(nb + i) * a.ldo + a.lanes] = a.scale * y1;
        }
    }
}

// Any head sizes, fp32 (the validation mode): one CTA per (sequence, head), a
// thread two state columns of as few nodes at a time (16, 8, 4: a load of q
// serves both columns, one of S all nodes) as keep the threads in work. 60 trees
// of 29 to 59 nodes, H = 16: 76 us at heads of 49 x 69, 406 at 128 x 256; 256
// trees of 1 to 32 at 96 x 192 367 (one column a thread, the path's nodes one by
// one: 98, 577, 476). Shared memory holds two or three such CTAs an SM, whose
// loads it waits for.
__global__ void __launch_bounds__(kThreads, 3) tree_fwd_kernel(const TreeParams p) {
    extern __shared__ float4 smem4[];
    __shared__ int par[kNodes];
    __shared__ unsigned long long path[kNodes];
    __shared__ float far[kNodes], gate[kNodes];
    const int n = blockIdx.x / p.H, h = blockIdx.x % p.H, tid = threadIdx.x;
    const Tree t = open_tree(p, n, par);
    if (t.nodes <= 0) {
        if (t.nodes < 0 && tid == 0) atomicOr(p.status, kDevBadState);
        return;
    }
    const int M = t.nodes, dk = p.dk, dv = p.dv, ldq = padded(dk);
    float *qs = reinterpret_cast<float *>(smem4), *ks = qs + kNodes * ldq, *P = ks + kNodes * ldq;
    const float *q = static_cast<const float *>(p.q) + (size_t)t.first * p.ldq + (size_t)h * dk;
    const float *k = static_cast<const float *>(p.k) + (size_t)t.first * p.ldk + (size_t)h * dk;
    const float *v = static_cast<const float *>(p.v) + (size_t)t.first * p.ldv + (size_t)h * dv;
    for (int e = tid; e < M * ldq; e += kThreads) {
        const int i = e / ldq, c = e % ldq;
        qs[e] = c < dk ? q[(size_t)i * p.ldq + c] : 0.f;
        ks[e] = c < dk ? k[(size_t)i * p.ldk + c] : 0.f;
    }
    const float fixed = p.g ? 0.f : p.log_lambda[h];
    if (p.g && tid < M) gate[tid] = p.g[(size_t)(t.first + tid) * p.H + h];
    __syncthreads();
    if (tid < M) path[tid] = walk(tid, par, p.g ? gate : nullptr, fixed, far[tid], [&](int j, float w) { P[tid * kNodes + j] = w; });
    __syncthreads();
    for (int e = tid; e < M * M; e += kThreads) {
        const int i = e / M, j = e % M;
        if (!(path[i] >> j & 1)) continue;
        float dot = 0.f;
        for (int c = 0; c < dk; c += 4) {   // (zeros behind the last channel)
            const float4 a = *reinterpret_cast<const float4 *>(qs + i * ldq + c), b = *reinterpret_cast<const float4 *>(ks + j * ldq + c);
            dot = fmaf(a.w, b.w, fmaf(a.z, b.z, fmaf(a.y, b.y, fmaf(a.x, b.x, dot))));
        }
        P[i * kNodes + j] *= dot;
    }
    __syncthreads();
    const int lanes = (dv + 1) / 2, groups = kThreads / lanes, c = tid % lanes, grp = tid / lanes;
    if (grp >= groups) return;
    const Sums a{qs, P, far, p.pool + (t.slot * p.H + h) * ((size_t)dk * dv) + c, v + c, path,
                 static_cast<float *>(p.o) + ((size_t)t.first * p.H + h) * dv + c, M, ldq, dk, dv, lanes, (size_t)p.ldv, (size_t)p.H * dv,
                 p.scale, c + lanes < dv};
    if (M <= 4 * groups) sum_nodes<4>(a, grp, groups);
    else if (M <= 8 * groups) sum_nodes<8>(a, grp, groups);
    else sum_nodes<16>(a, grp, groups);
}

// ----------------------------------------------------------------- commit
constexpr int kCommit = 256;

// The windows' pieces from CTA `first` on, a warp each.
template <typename T> __device__ __forceinline__ void windows_of(const TreeParams &p, unsigned first) {
    const long piece = (long)(blockIdx.x - first) * (kCommit / 32) + threadIdx.x / 32;
    if (piece < window_pieces(p)) commit_window<T>(p, piece);
}
// No heads: the windows alone.
template <typename T> __global__ void __launch_bounds__(kCommit) windows_kernel(const TreeParams p) { windows_of<T>(p, 0); }

// Any head sizes, fp32 (the validation mode): one CTA per (sequence, head),
// behind them the windows'. Pages of 96 x 192, all of bf16's, go through tree_commit.cu.
__global__ void __launch_bounds__(kCommit) tree_commit_any_kernel(const TreeParams p) {
    extern __shared__ float4 smem4[];
    __shared__ int par[kNodes], way[kNodes], s_len;
    __shared__ float s_w[kNodes], gate[kNodes], s_far;
    float *kt = reinterpret_cast<float *>(smem4);          // [path node][dk], decayed
    const unsigned pages = (unsigned)p.nseq * (unsigned)p.H;
    if (blockIdx.x >= pages) {
        windows_of<float>(p, pages);
        return;
    }
    const int n = blockIdx.x / p.H, h = blockIdx.x % p.H, tid = threadIdx.x;
    const int last = p.last[n];
    const Tree t = open_tree(p, n, par);
    if (t.nodes < 0 || bad_last(last, t.nodes)) {
        if (tid == 0) atomicOr(p.status, kDevBadState);
        return;
    }
    if (last < 0) return;
    const int dk = p.dk, dv = p.dv;
    if (p.g && tid < t.nodes) gate[tid] = p.g[(size_t)(t.first + tid) * p.H + h];
    __syncthreads();
    if (tid == 0) {
        int len = 0;
        walk(last, par, p.g ? gate : nullptr, p.g ? 0.f : p.log_lambda[h], s_far, [&](int j, float w) {
            way[len] = j;
            s_w[len++] = w;
        });
        s_len = len;
    }
    __syncthreads();
    const int len = s_len;
    const float far = s_far;
    for (int e = tid; e < len * dk; e += kCommit) {
        const int j = e / dk, r = e % dk;
        kt[e] = s_w[j] * static_cast<const float *>(p.k)[(size_t)(t.first + way[j]) * p.ldk + (size_t)h * dk + r];
    }
    __syncthreads();
    float *S = p.pool + (t.slot * p.H + h) * ((size_t)dk * dv);
    const float *v = static_cast<const float *>(p.v) + (size_t)t.first * p.ldv + (size_t)h * dv;
    if (dv % 4 == 0) {   // four columns of four rows a thread at a time
        const int cols = dv / 4, c = tid % cols * 4, step = kCommit / cols;
        for (int r0 = tid / cols; r0 < dk && tid < step * cols; r0 += 4 * step) {
            float4 x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (r0 + i * step < dk) {
                    const float4 y = *reinterpret_cast<const float4 *>(S + (size_t)(r0 + i * step) * dv + c);
                    x[i] = far == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(far * y.x, far * y.y, far * y.z, far * y.w);
                }
            for (int j = 0; j < len; ++j) {
                const float *w = v + (size_t)way[j] * p.ldv + c;   // (4-byte aligned)
                const float4 u = make_float4(w[0], w[1], w[2], w[3]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float k = r0 + i * step < dk ? kt[j * dk + r0 + i * step] : 0.f;
                    x[i].x = fmaf(k, u.x, x[i].x);
                    x[i].y = fmaf(k, u.y, x[i].y);
                    x[i].z = fmaf(k, u.z, x[i].z);
                    x[i].w = fmaf(k, u.w, x[i].w);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (r0 + i * step < dk) *reinterpret_cast<float4 *>(S + (size_t)(r0 + i * step) * dv + c) = x[i];
        }
        return;
    }
    for (int e = tid; e < dk * dv; e += kCommit) {
        const int r = e / dv, c = e % dv;
        float x = far == 0.f ? 0.f : far * S[e];
        for (int j = 0; j < len; ++j) x = fmaf(kt[j * dk + r], v[(size_t)way[j] * p.ldv + c], x);
        S[e] = x;
    }
}

// ------------------------------------------------------------- convolution
// A CTA takes the channels of one block of one tree: its rows of x and the
// window's last three arrive in shared memory by asynchronous copies, all in
// flight at once, and each is read up to four times from there (as a node and
// as an ancestor): 43 us at 256 trees of 16 to 64 nodes, D = 4096, 0.62 of the
// copy rate; rows straight from global memory 93. A CTA's copies and its
// arithmetic take turns: the copies and the output alone take 29 us, the taps
// (unpacking, and a branch for each while they had one: 3 us more) 8, SiLU 4.
// Measured at the same 41 to 44: the next tree's rows under way while one is
// worked on, four channels a thread and 1.5 to twice the warps, blocks of half
// the channels, the window's part summed ahead.
// CTAs of the channels stay for several trees: the taps of a thread's channels,
// 128 strided bytes, cost as much as ten nodes' rows. Three times as many as
// fit at a time, so that trees of different sizes even out (1, 2, 3, 4, 6
// times, all at once: 43.1, 43.9, 40.1, 41.2, 42.2, 44 us on the device).
constexpr int kConv = 128;   // threads, eight channels each
template <typename T> constexpr int conv_lanes() { return sizeof(T) == 2 ? 32 : 16; }   // of a row: 256 channels at bf16, 128 at fp32

template <typename T> __global__ void __launch_bounds__(kConv) conv_tree_kernel(const TreeParams p, int per) {
    constexpr int kLanes = conv_lanes<T>(), kRows = kConv / kLanes, H = sizeof(T) / 2;
    extern __shared__ uint4 smem_conv[];                      // [nodes][pieces of 16 bytes][lanes]
    __shared__ __align__(16) float4 wins[3][2][kLanes];       // the window's rows 1 .. 3
    __shared__ int par[kNodes];
    __shared__ int4 up[kNodes];   // a node's last three ancestors: where their rows start in smem_conv, or -1 - r: r rows before the window's last; w: all are nodes
    const int lane = threadIdx.x % kLanes, first_row = threadIdx.x / kLanes;
    // a thread's channels: eight neighbours at bf16; two groups of four at fp32, so that a warp's stores are whole sectors
    // (128 trees of 16 to 64 nodes, D = 4096, fp32: 34.5 us; eight neighbours 47)
    // (unsigned: the lanes of the last block go past D, which may be next to 2^31)
    const unsigned first = blockIdx.x % per * (kLanes * 8), c = first + lane * (8 / H), half = H == 1 ? 4 : kLanes * 4, D = (unsigned)p.D;
    const bool on = c < D, whole = c + half < D;
    // the taps by way of shared memory: coalesced in, and out again a channel's 16 bytes after 144 bytes a lane
    for (unsigned i = threadIdx.x; i < kLanes * 8; i += kConv) {
        if (first + i < D) smem_conv[i + i / 8] = __ldg(reinterpret_cast<const uint4 *>(p.w) + first + i);
    }
    __syncthreads();
    ssm::f2 w[4][4], b[4];                                    // taps of channel pairs
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    const float4 b_lo = p.b && on ? __ldg(reinterpret_cast<const float4 *>(p.b + c)) : zero;
    const float4 b_hi = p.b && whole ? __ldg(reinterpret_cast<const float4 *>(p.b + c + half)) : zero;
    b[0] = ssm::f2_pack(b_lo.x, b_lo.y), b[1] = ssm::f2_pack(b_lo.z, b_lo.w);
    b[2] = ssm::f2_pack(b_hi.x, b_hi.y), b[3] = ssm::f2_pack(b_hi.z, b_hi.w);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const unsigned ch = c - first + 2 * j + (j < 2 ? 0 : half - 4);   // (an even one and the next: no multiple of 8 between)
        const bool in = first + ch < D;
        const float4 u = in ? reinterpret_cast<const float4 *>(smem_conv)[ch + ch / 8] : zero;
        const float4 v = in ? reinterpret_cast<const float4 *>(smem_conv)[ch + ch / 8 + 1] : zero;
        w[0][j] = ssm::f2_pack(u.x, v.x);
        w[1][j] = ssm::f2_pack(u.y, v.y);
        w[2][j] = ssm::f2_pack(u.z, v.z);
        w[3][j] = ssm::f2_pack(u.w, v.w);
    }
    const T *x = static_cast<const T *>(p.x) + (on ? c : 0);
    for (int n = blockIdx.x / per; n < p.nseq; n += (int)(gridDim.x / per)) {
        __syncthreads();                                      // the taps, or the tree before, have been read
        // what open_tree checks, before the copies that do not depend on the parents
        const int lo = p.cu[n], hi = p.cu[n + 1], slot = p.slots ? p.slots[n] : n;
        if (!bad_entry(p, lo, hi, slot)) {
            for (int i = first_row; i < hi - lo; i += kRows)
#pragma unroll
                for (int h = 0; h < H; ++h)
                    ssm::copy_async<16>(&smem_conv[(i * H + h) * kLanes + lane], x + (size_t)(lo + i) * p.ldx + h * half, h == 0 ? on : whole);
            for (int r = first_row; r < 6 && hi > lo; r += kRows) {
                const bool in = r % 2 == 0 ? on : whole;
                ssm::copy_async<16>(&wins[r / 2][r % 2][lane], in ? p.win + ((size_t)slot * ssm::kTaps + 1 + r / 2) * p.D + c + half * (r % 2) : p.win, in);
            }
        }
        ssm::copies_commit();
        const Tree t = open_tree(p, n, par);
        if (t.nodes < 0 && threadIdx.x == 0) atomicOr(p.status, kDevBadState);
        if ((int)threadIdx.x < t.nodes) {
            int a[4] = {(int)threadIdx.x};
#pragma unroll
            for (int k = 1; k < 4; ++k) a[k] = a[k - 1] >= 0 ? par[a[k - 1]] : a[k - 1] - 1;
#pragma unroll
            for (int k = 1; k < 4; ++k) a[k] *= a[k] >= 0 ? H * kLanes : 1;
            up[threadIdx.x] = make_int4(a[1], a[2], a[3], a[3] >= 0);
        }
        ssm::copies_wait<0>();
        __syncthreads();
        if (!on) continue;
        T *y = static_cast<T *>(p.y) + (size_t)(t.first + first_row) * p.D + c;
        for (int i = first_row; i < t.nodes; i += kRows, y += (size_t)kRows * p.D) {
            ssm::f2 acc[4] = {b[0], b[1], b[2], b[3]};
            const auto add = [&](const ssm::f2 (&u)[4], const ssm::f2 (&wt)[4]) {
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[j] = ssm::fma2(wt[j], u[j], acc[j]);
            };
            const auto row = [&](int at) {
                ssm::Raw8<T> raw;
#pragma unroll
                for (int h = 0; h < H; ++h) raw.w[h] = smem_conv[at + h * kLanes + lane];
                return raw;
            };
            const auto node = [&](const ssm::Raw8<T> &raw, const ssm::f2 (&wt)[4]) {
                ssm::f2 u[4];
                ssm::raw_unpack(raw, u);
                add(u, wt);
            };
            const int4 a = up[i];
            const ssm::Raw8<T> own = row(i * H * kLanes);
            if (a.w) {   // without a branch for each
                const ssm::Raw8<T> r1 = row(a.x), r2 = row(a.y), r3 = row(a.z);
                node(own, w[3]);
                node(r1, w[2]);
                node(r2, w[1]);
                node(r3, w[0]);
            } else {
                node(own, w[3]);
                const auto tap = [&](int at, const ssm::f2 (&wt)[4]) {
                    if (at >= 0) {
                        node(row(at), wt);
                        return;
                    }
                    const float4 e = wins[3 + at][0][lane], f = wins[3 + at][1][lane];
                    const ssm::f2 u[4] = {ssm::f2_pack(e.x, e.y), ssm::f2_pack(e.z, e.w), ssm::f2_pack(f.x, f.y), ssm::f2_pack(f.z, f.w)};
                    add(u, wt);
                };
                tap(a.x, w[2]);
                tap(a.y, w[1]);
                tap(a.z, w[0]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[j] = ssm::silu2(acc[j]);
            if constexpr (H == 1) {
                ssm::store8(y, acc, whole);
            } else {
                const float2 a0 = ssm::f2_split(acc[0]), a1 = ssm::f2_split(acc[1]), a2 = ssm::f2_split(acc[2]), a3 = ssm::f2_split(acc[3]);
                *reinterpret_cast<float4 *>(y) = make_float4(a0.x, a0.y, a1.x, a1.y);
                if (whole) *reinterpret_cast<float4 *>(y + half) = make_float4(a2.x, a2.y, a3.x, a3.y);
            }
        }
    }
}

cudaError_t fwd_any(const TreeParams &p, cudaStream_t s, int *launches) {
    const int bytes = (2 * kNodes * padded(p.dk) + kNodes * kNodes) * (int)sizeof(float);
    cudaError_t e = cudaFuncSetAttribute(tree_fwd_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    tree_fwd_kernel<<<(unsigned)((size_t)p.nseq * p.H), kThreads, bytes, s>>>(p);
    if (launches) ++*launches;
    return cudaGetLastError();
}

long window_blocks(const TreeParams &p) { return (window_pieces(p) + kCommit / 32 - 1) / (kCommit / 32); }

template <typename T> cudaError_t windows(const TreeParams &p, cudaStream_t s, int *launches) {
    windows_kernel<T><<<(unsigned)window_blocks(p), kCommit, 0, s>>>(p);
    if (launches) ++*launches;
    return cudaGetLastError();
}

cudaError_t commit_any(const TreeParams &p, cudaStream_t s, int *launches) {
    const int bytes = kNodes * p.dk * (int)sizeof(float);   // at most 32 KB
    const long blocks = (long)p.nseq * p.H + window_blocks(p);
    tree_commit_any_kernel<<<(unsigned)blocks, kCommit, bytes, s>>>(p);
    if (launches) ++*launches;
    return cudaGetLastError();
}

template <typename T> cudaError_t conv(const TreeParams &p, cudaStream_t s, int *launches) {
    constexpr int kLanes = conv_lanes<T>();
    const int per = (int)((p.D + 8L * kLanes - 1) / (8 * kLanes)), bytes = kNodes * kLanes * 8 * (int)sizeof(T);   // 32 KB
    const long held = 18L * device_sm_count() / per;   // thrice the six CTAs an SM that shared memory holds
    const long trees = held < 1 ? 1 : held < p.nseq ? held : p.nseq;
    conv_tree_kernel<T><<<(unsigned)(trees * per), kConv, bytes, s>>>(p, per);
    if (launches) ++*launches;
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_fwd(const TreeParams &p, bool bf16, cudaStream_t s, int *launches) {
    return bf16 ? launch_tree_fwd_tc(p, s, launches) : fwd_any(p, s, launches);
}
cudaError_t launch_tree_commit(const TreeParams &p, bool bf16, cudaStream_t s, int *launches) {
    if (p.H == 0) return bf16 ? windows<__nv_bfloat16>(p, s, launches) : windows<float>(p, s, launches);
    return p.dk == 96 && p.dv == 192 ? launch_tree_pages(p, bf16, s, launches) : commit_any(p, s, launches);
}
cudaError_t launch_conv_tree(const TreeParams &p, bool bf16, cudaStream_t s, int *launches) {
    return bf16 ? conv<__nv_bfloat16>(p, s, launches) : conv<float>(p, s, launches);
}

}  // namespace gla
