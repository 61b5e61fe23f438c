// tree_tc.cu -- the readout of drafted trees at bf16, dk = 96, dv = 192: with
// F_i the decay of the whole path of node i and W_ij that of its nodes behind j,
//     O = scale ( diag(F) Q S + (W o Q K^T) V ),
// W_ij = 0 off the path. Up to 64 nodes share one read of the page S (73,728
// bytes fp32), so the call is bound by HBM: the pages, q, k, v and o once.
//
// S goes from HBM to the tensor cores by way of shared memory and registers
// alone: a ring of TMA boxes (96 rows x 32 channels, 128-byte swizzle), one
// consumer warp a box, which splits each entry into two bf16 halves (hi + lo,
// 2^-17 of the entry: drafted tokens get the values that the decode step's fp32
// arithmetic gives, to a few 2^-17) and multiplies Q by both. A box has too few
// products a byte to wait for tcgen05's operand layouts in shared memory (the
// halves would have to be written there first); warp-level products on
// registers leave the tensor pipe far from its limit. P = W o Q K^T is split likewise.
//
// One producer warp per CTA runs ahead: offsets, parents and decays of the next
// unit, the paths as bit masks and running sums by pointer doubling, the rows of
// q, k and v by bulk copies. Two CTAs on an SM: one's product phases lie under
// the other's loads.
//
// Accumulator columns: of the four 8-column tiles of a box, column n of tile t
// is channel 4 n + t. A thread's entries of S are then 16-byte loads (the
// swizzle keeps them free of bank conflicts), and the channels of a row that it
// ends with are eight neighbours, stored as 16 bytes.
#include "ptx.cuh"
#include "tmap.h"
#include "tree_common.cuh"

namespace gla {
namespace {

using namespace ptx;
using tree::kNodes;

constexpr int kDk = 96, kDv = 192, kSlice = 32, kSlices = kDv / kSlice;   // consumer warps: one a slice of channels
constexpr int kThreads = (kSlices + 1) * 32, kStages = 3;
constexpr uint32_t kBox = kDk * kSlice * 4;
constexpr uint32_t kPitchQ = kDk * 2 + 16, kPitchV = kDv * 2 + 16, kPitchP = kNodes * 2 + 16;   // (16 more: no bank conflicts)
constexpr uint32_t kOffQ = kStages * kBox, kOffK = kOffQ + kNodes * kPitchQ, kOffV = kOffK + kNodes * kPitchQ,
                   kOffPh = kOffV + kNodes * kPitchV, kOffPl = kOffPh + kNodes * kPitchP, kOffMeta = kOffPl + kNodes * kPitchP;
constexpr float kClear = -104.f;   // e^-104 is 0 in fp32
constexpr float kLog2e = 1.4426950408889634f;

// A unit's tree, made by the producer.
struct Meta {
    unsigned long long path[kNodes];   // the nodes on the path that no decay of 0 cuts off, the node itself included
    float2 sum[kNodes];                // their summed logs (fixed decay: their number), high and low part
    float far[kNodes];                 // the state's decay
    float factor;                      // W_ij = 2^(factor (sum_i - sum_j))
    int first, nodes, pad;
};
// The boxes of a unit take the ring's stages in turn, but their barriers go by slice: a waiter sees every phase of its own.
enum { FULL_S = 0, EMPTY_S = FULL_S + kSlices, FULL_Q = EMPTY_S + kSlices, FULL_K, FULL_V, FREE_Q, FREE_K, FREE_V, FULL_M, FREE_M = FULL_M + 2, BARS = FREE_M + 2 };
constexpr uint32_t kOffNext = kOffMeta + 2 * sizeof(Meta), kOffBars = kOffNext + kNodes * 4, kOffAbort = kOffBars + BARS * 8,
                   kSmem = kOffAbort + 16 + 1024;   // (1,024: the base is rounded up for the swizzle)

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap *m, uint32_t bar, int c0, int c1) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1)
                 : "memory");
}
__device__ __forceinline__ float4 lds4(uint32_t at) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds2(uint32_t at) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
    return v;
}
// Two numbers as their bf16 halves: x = hi + lo up to 2^-17.
__device__ __forceinline__ void split(float x0, float x1, uint32_t &hi, uint32_t &lo) {
    hi = pack_bf16x2(x0, x1);
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

// What the producer reads of a unit ahead of time.
struct Ahead {
    int first, nodes, slot;   // nodes -1: a bad offset or slot
    int par[2];               // of nodes lane and lane + 32
    float gate[2];
};

template <bool kGate>
__device__ __forceinline__ void producer(const TreeParams &p, const CUtensorMap *tm, unsigned char *sm, uint32_t base, const WaitCtl &ctl, long units) {
    const int lane = threadIdx.x % 32;
    auto bar = [&](int i) { return base + kOffBars + 8u * (uint32_t)i; };
    int *next = reinterpret_cast<int *>(sm + kOffNext);
    auto offsets = [&](long u, Ahead &a) {
        if (u >= units) return;
        const int n = (int)(u / p.H);
        const int lo = __ldg(p.cu + n), hi = __ldg(p.cu + n + 1);
        a.slot = p.slots ? __ldg(p.slots + n) : n;
        a.first = lo;
        a.nodes = lo < 0 || hi < lo || hi > p.total_T || hi - lo > kNodes || a.slot < 0 || a.slot >= p.n_slots ? -1 : hi - lo;
    };
    auto nodes = [&](long u, Ahead &a) {
        if (u >= units) return;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = lane + 32 * e;
            a.par[e] = i < a.nodes ? __ldg(p.parents + a.first + i) : -1;
            if (kGate) a.gate[e] = i < a.nodes ? __ldg(p.g + (size_t)(a.first + i) * p.H + u % p.H) : 0.f;
        }
    };
    auto wait = [&](int b, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar(b), parity, ctl)); };
    Ahead a[2];   // this unit's and the next one's
    offsets(blockIdx.x, a[0]);
    nodes(blockIdx.x, a[0]);
    offsets((long)blockIdx.x + gridDim.x, a[1]);
    long boxes = 0, done = 0;
    bool ok = true;
    int it = 0;
    for (long u = blockIdx.x; u < units && ok; u += gridDim.x, ++it) {
        Ahead now = a[0];
        a[0] = a[1];
        nodes(u + gridDim.x, a[0]);
        offsets(u + 2L * gridDim.x, a[1]);
        const int h = (int)(u % p.H);
        bool bad = now.nodes < 0;
#pragma unroll
        for (int e = 0; e < 2; ++e) bad |= lane + 32 * e < now.nodes && (now.par[e] < -1 || now.par[e] >= lane + 32 * e);
        if (__any_sync(0xffffffffu, bad)) {
            now.nodes = 0;
            if (lane == 0) atomicOr(p.status, kDevBadState);
        }
        const int s = it & 1, M = now.nodes;
        if (it >= 2 && !(ok = wait(FREE_M + s, (uint32_t)((it >> 1) - 1) & 1u))) break;
        Meta *m = reinterpret_cast<Meta *>(sm + kOffMeta) + s;
        const float fixed = kGate ? 0.f : p.log_lambda[h];
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
            for (int e = 0; e < 2; ++e)
                if (ptr[e] >= 0) {
                    up[e] = m->path[ptr[e]];
                    add[e] = m->sum[ptr[e]];
                    on[e] = next[ptr[e]];
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
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(FULL_M + s));
        if (M == 0) continue;
        auto rows = [&](int full, uint32_t off, const void *src, long ld, uint32_t bytes, uint32_t pitch) {
            if (lane == 0) mbar_arrive_expect_tx(bar(full), (uint32_t)M * bytes);
            __syncwarp();
            for (int i = lane; i < M; i += 32)
                bulk_load(base + off + (uint32_t)i * pitch,
                          static_cast<const char *>(src) + (size_t)(now.first + i) * ld * 2 + (size_t)h * bytes, bytes, bar(full));
        };
        auto box = [&](int j) {   // box number `boxes`: into the stage of the box kStages before it
            const long last = boxes - kStages;
            if (last >= 0 && !(ok = wait(EMPTY_S + (int)(last % kSlices), (uint32_t)(last / kSlices) & 1u))) return;
            if (lane == 0) {
                mbar_arrive_expect_tx(bar(FULL_S + j), kBox);
                tma_load_2d(base + (uint32_t)(boxes % kStages) * kBox, tm, bar(FULL_S + j), j * kSlice, (now.slot * p.H + h) * kDk);
            }
            ++boxes;
        };
        const uint32_t par = (uint32_t)(done - 1) & 1u;
        for (int j = 0; j < kStages && ok; ++j) box(j);
        if (!ok || (done > 0 && !(ok = wait(FREE_Q, par)))) break;
        rows(FULL_Q, kOffQ, p.q, p.ldq, kDk * 2, kPitchQ);
        if (done > 0 && !(ok = wait(FREE_K, par))) break;
        rows(FULL_K, kOffK, p.k, p.ldk, kDk * 2, kPitchQ);
        for (int j = kStages; j < kSlices && ok; ++j) box(j);
        if (!ok || (done > 0 && !(ok = wait(FREE_V, par)))) break;
        rows(FULL_V, kOffV, p.v, p.ldv, kDv * 2, kPitchV);
        ++done;
    }
    if (!ok) {   // a wait gave up: the copies in flight land before the CTA ends
        for (long k = boxes > kStages ? boxes - kStages : 0; k < boxes; ++k)
            mbar_wait_drain(bar(FULL_S + (int)(k % kSlices)), (uint32_t)(k / kSlices) & 1u, 1000000ull);
        for (int b : {FULL_Q, FULL_K, FULL_V})
            for (long k = done > 0 ? done - 1 : 0; k <= done; ++k) mbar_wait_drain(bar(b), (uint32_t)k & 1u, 1000000ull);
    }
}

template <bool kGate> __global__ void __launch_bounds__(kThreads, 2) tree_fwd_tc_kernel(const __grid_constant__ CUtensorMap tm, const TreeParams p) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t base = smem_u32(sm);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const long units = (long)p.nseq * p.H;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + kOffAbort);
    const WaitCtl ctl{abort_flag, p.status};
    auto bar = [&](int i) { return base + kOffBars + 8u * (uint32_t)i; };
    if (threadIdx.x == 0) {
        *abort_flag = 0;
        for (int i = 0; i < BARS; ++i)   // one arrival (a copy's, the slice's warp, the producer), or one a consumer warp
            mbar_init(bar(i), (i >= FREE_Q && i <= FREE_V) || i >= FREE_M ? kSlices : 1);
        fence_mbar_init();
        prefetch_tmap(&tm);
    }
    __syncthreads();
    if (warp == kSlices) {
        producer<kGate>(p, &tm, sm, base, ctl, units);
        return;
    }
    const int g = lane / 4, q4 = lane % 4;   // a fragment's row (or column), its pair of columns (or rows)
    const uint32_t sQ = base + kOffQ, sK = base + kOffK, sV = base + kOffV, sPh = base + kOffPh, sPl = base + kOffPl;
    const uint32_t a_row = lane % 16, a_col = lane / 16 * 8;                        // ldmatrix: A fragments of 16 rows
    const uint32_t b_row = (lane & 7) + (lane >> 4) * 8, b_col = (lane >> 3 & 1) * 8;   // and B fragments of 16 columns
    // Never left before its end: the warps meet twice a unit, also when a wait has given up.
    bool ok = true;
    long done = 0;
    int it = 0;
    auto wait = [&](int b, uint32_t parity) { ok = ok && __all_sync(0xffffffffu, mbar_wait(bar(b), parity, ctl)); };
    for (long u = blockIdx.x; u < units; u += gridDim.x, ++it) {
        const Meta *m = reinterpret_cast<const Meta *>(sm + kOffMeta) + (it & 1);
        wait(FULL_M + (it & 1), (uint32_t)(it >> 1) & 1u);
        const int M = ok ? m->nodes : 0, tiles = (M + 15) / 16;
        const uint32_t par = (uint32_t)done & 1u;
        named_sync(1, kSlices * 32);   // every warp is done with the unit before's P
        if (M > 0) {
            // P, tile by tile below the diagonal, the tiles dealt out to the warps
            wait(FULL_Q, par);
            wait(FULL_K, par);
            const float factor = ok ? m->factor : 0.f;
#pragma unroll 1
            for (int x = warp; ok && x < tiles * (tiles + 1) / 2; x += kSlices) {
                const int ti = x < 1 ? 0 : x < 3 ? 1 : x < 6 ? 2 : 3, tj = x - ti * (ti + 1) / 2;
                float c[2][4] = {};
#pragma unroll
                for (int ks = 0; ks < kDk / 16; ++ks) {
                    uint32_t a[4], b[4];
                    ldmatrix4(a, sQ + (ti * 16 + a_row) * kPitchQ + (ks * 16 + a_col) * 2);
                    ldmatrix4(b, sK + (tj * 16 + b_row) * kPitchQ + (ks * 16 + b_col) * 2);
                    mma16816(c[0], a, b[0], b[1]);
                    mma16816(c[1], a, b[2], b[3]);
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
                        uint32_t hi, lo;
                        split(v[0], v[1], hi, lo);
                        const uint32_t at = (uint32_t)i * kPitchP + (uint32_t)j * 2;
                        *reinterpret_cast<uint32_t *>(sm + kOffPh + at) = hi;
                        *reinterpret_cast<uint32_t *>(sm + kOffPl + at) = lo;
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(FREE_K));
        }
        named_sync(1, kSlices * 32);
        if (M > 0) {
            float acc[4][4][4];
            // Q S: a step of 16 rows of S at a time
            wait(FULL_S + warp, par);
            const uint32_t sS = base + (uint32_t)((done * kSlices + warp) % kStages) * kBox;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int c = 0; c < 4; ++c) acc[i][t][c] = 0.f;
            if (ok) {
#pragma unroll 2
                for (int ks = 0; ks < kDk / 16; ++ks) {
                    const uint32_t r = (uint32_t)(ks * 16 + 2 * q4);
                    const uint32_t e = sS + r * 128 + (((uint32_t)g ^ (r & 7u)) << 4), f = sS + (r + 1) * 128 + (((uint32_t)g ^ ((r + 1) & 7u)) << 4);
                    const float4 x0 = lds4(e), x1 = lds4(f), x2 = lds4(e + 1024), x3 = lds4(f + 1024);
                    uint32_t hi[4][2], lo[4][2];
                    split(x0.x, x1.x, hi[0][0], lo[0][0]);
                    split(x0.y, x1.y, hi[1][0], lo[1][0]);
                    split(x0.z, x1.z, hi[2][0], lo[2][0]);
                    split(x0.w, x1.w, hi[3][0], lo[3][0]);
                    split(x2.x, x3.x, hi[0][1], lo[0][1]);
                    split(x2.y, x3.y, hi[1][1], lo[1][1]);
                    split(x2.z, x3.z, hi[2][1], lo[2][1]);
                    split(x2.w, x3.w, hi[3][1], lo[3][1]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (i >= tiles) break;
                        uint32_t a[4];
                        ldmatrix4(a, sQ + (i * 16 + a_row) * kPitchQ + (ks * 16 + a_col) * 2);
#pragma unroll
                        for (int t = 0; t < 4; ++t) mma16816(acc[i][t], a, hi[t][0], hi[t][1]);
#pragma unroll
                        for (int t = 0; t < 4; ++t) mma16816(acc[i][t], a, lo[t][0], lo[t][1]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(EMPTY_S + warp));
                mbar_arrive(bar(FREE_Q));
            }
            // the state's decay: 0 clears it, whatever it holds
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < tiles) {
                    const float f0 = m->far[i * 16 + g], f1 = m->far[i * 16 + g + 8];
#pragma unroll
                    for (int t = 0; t < 4; ++t)
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const float f = c < 2 ? f0 : f1;
                            acc[i][t][c] = f == 0.f ? 0.f : f * acc[i][t][c];
                        }
                }
            // P V: 16 nodes j at a time
            wait(FULL_V, par);
            bool dirty = false;
            if (ok) {
#pragma unroll
                for (int js = 0; js < 4; ++js) {
                    if (js >= tiles) break;
                    uint2 x[4];
                    uint32_t odd = 0;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int j = js * 16 + 2 * q4 + (r & 1) + (r >> 1) * 8;
                        x[r] = lds2(sV + (uint32_t)j * kPitchV + (uint32_t)(warp * kSlice * 2 + g * 8));
                        if (j >= M) x[r] = make_uint2(0, 0);   // (rows that no copy has written)
                        odd |= (mul_bf16x2(x[r].x, 0) | mul_bf16x2(x[r].y, 0)) & 0x7fff7fffu;   // not 0: an element that is not finite
                    }
                    // One that is not finite would reach every node by way of 0 x inf: it is left out here and added on its paths below.
                    if (__any_sync(0xffffffffu, odd != 0)) {
                        dirty = true;
#pragma unroll
                        for (int r = 0; r < 4; ++r) x[r] = make_uint2(finite2(x[r].x), finite2(x[r].y));
                    }
                    uint32_t b[4][2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        b[0][r] = __byte_perm(x[2 * r].x, x[2 * r + 1].x, 0x5410);
                        b[1][r] = __byte_perm(x[2 * r].x, x[2 * r + 1].x, 0x7632);
                        b[2][r] = __byte_perm(x[2 * r].y, x[2 * r + 1].y, 0x5410);
                        b[3][r] = __byte_perm(x[2 * r].y, x[2 * r + 1].y, 0x7632);
                    }
#pragma unroll
                    for (int i = js; i < 4; ++i) {
                        if (i >= tiles) break;
                        uint32_t h[4], l[4];
                        const uint32_t at = (i * 16 + a_row) * kPitchP + (js * 16 + a_col) * 2;
                        ldmatrix4(h, sPh + at);
                        ldmatrix4(l, sPl + at);
#pragma unroll
                        for (int t = 0; t < 4; ++t) mma16816(acc[i][t], h, b[t][0], b[t][1]);
#pragma unroll
                        for (int t = 0; t < 4; ++t) mma16816(acc[i][t], l, b[t][0], b[t][1]);
                    }
                }
            }
            __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(p.o) + ((size_t)m->first * p.H + u % p.H) * kDv + warp * kSlice + 8 * q4;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int x = i * 16 + g + 8 * r;
                    if (!ok || x >= M) continue;
                    if (dirty) {
                        for (unsigned long long path = m->path[x]; path; path &= path - 1) {
                            const int j = __ffsll((long long)path) - 1;
                            const uint32_t at = (uint32_t)x * kPitchP + (uint32_t)j * 2;
                            const float w = __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(sm + kOffPh + at)) +
                                            __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(sm + kOffPl + at));
                            const __nv_bfloat16 *v = reinterpret_cast<const __nv_bfloat16 *>(sm + kOffV + (uint32_t)j * kPitchV) + warp * kSlice + 8 * q4;
#pragma unroll
                            for (int t = 0; t < 4; ++t)
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    const float y = __bfloat162float(v[4 * e + t]);
                                    if (!isfinite(y) && w != 0.f) acc[i][t][2 * r + e] += w * y;
                                }
                        }
                    }
                    uint4 y;
                    y.x = pack_bf16x2(p.scale * acc[i][0][2 * r], p.scale * acc[i][1][2 * r]);
                    y.y = pack_bf16x2(p.scale * acc[i][2][2 * r], p.scale * acc[i][3][2 * r]);
                    y.z = pack_bf16x2(p.scale * acc[i][0][2 * r + 1], p.scale * acc[i][1][2 * r + 1]);
                    y.w = pack_bf16x2(p.scale * acc[i][2][2 * r + 1], p.scale * acc[i][3][2 * r + 1]);
                    *reinterpret_cast<uint4 *>(o + (size_t)x * p.H * kDv) = y;
                }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(FREE_V));
            ++done;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(FREE_M + (it & 1)));
    }
}

}  // namespace

bool tree_fwd_tc_fits(const TreeParams &p) {
    return p.dk == kDk && p.dv == kDv && p.n_slots > 0 && (long)p.n_slots * p.H * kDk <= 0x7fffffffL;   // TMA coordinates are ints
}

cudaError_t launch_tree_fwd_tc(const TreeParams &p, cudaStream_t s, int *launches) {
    const EncodeTiledFn enc = encode_tiled_fn();
    if (!enc) return cudaErrorNotSupported;
    CUtensorMap tm;
    const cuuint64_t dims[2] = {kDv, (cuuint64_t)p.n_slots * p.H * kDk}, strides[1] = {kDv * 4};
    const cuuint32_t box[2] = {kSlice, kDk}, es[2] = {1, 1};
    if (enc(&tm, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, p.pool, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    auto *kern = p.g ? tree_fwd_tc_kernel<true> : tree_fwd_tc_kernel<false>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
    const long units = (long)p.nseq * p.H, most = 2L * device_sm_count();
    kern<<<(unsigned)(units < most ? units : most), kThreads, kSmem, s>>>(tm, p);
    if (launches) ++*launches;
    return cudaGetLastError();
}

}  // namespace gla
