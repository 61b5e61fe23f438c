// ssm_bwd.cu -- gradients of the selective state-space scan (ssm.cu). With
// delta = softplus(dt + bias), a_t = exp(delta_t A), dy'_t = dy_t SiLU(z_t),
// per channel and state:
//     h_t = a_t h_{t-1} + delta_t B_t u_t             (recomputed)
//     G_t = C_t dy'_t + c_t,   c_{t-1} = a_t G_t      (from the last token back, c_{T-1} = dhT)
//     P_t = c_{t-1} h_{t-1}                           (dL / d(delta_t A))
// and the sums
//     over states n:   y0 = sum C h,  s1 = sum G B,  s2 = sum P A
//         dx = delta s1 + skip dy',   ddt = (s2 + u s1) sigmoid(dt + bias),
//         dz = dy (y0 + skip u) SiLU'(z)
//     over channels:   dC_t = sum dy' h_t,  dB_t = sum delta u G_t
//     over tokens:     dA = sum delta P,  dskip = sum dy' u,  ddt_bias = sum ddt;  dh0 = c_{-1}
//
// Two chains run against each other in time, so every state is needed once
// more after the forward sweep has passed it. A CTA of four warps owns 128
// channels (a quad of lanes four of them, each lane a quarter of their states;
// half as many at N = 32) of one segment of a sequence. A first launch sweeps
// the segment forward from zero and leaves the state entering every 16-token
// tile, and the sum of its steps so far, in the workspace; with the state h
// that enters the segment, tile_h + exp(A tile_sum) h is the state entering
// the tile. The main launch takes the tiles from the last to the first:
// forward through the tile, keeping the state before every fourth token in
// shared memory, then for each four tokens, last first, the four states again
// in registers (64 of them) with y0 and dC on the way, and back through them
// with G. States are thus recomputed, never stored per token (64 bytes a token
// and channel) nor divided back.
// Sums over states are exchanged inside a quad, four tokens at a time; sums
// over channels between the quads, eight numbers over eight quads, then added
// over the warps of the CTA through shared memory and over CTAs in a last
// launch, in a fixed order. The elementwise ends (loads, SiLU, softplus, the
// products above) are vectors of eight channels a thread, as in the forward.
//
// Few sequences are cut into segments as in the forward: the first launch then
// leaves each segment's state from zero and its c from zero too, with the same
// exponentials (c needs the running product of the decays), and a small launch
// carries both from segment to segment.
//
// Bound by instructions and, at two CTAs an SM, by their latency: 4 x 2048 x
// 2048, N = 16: 444 us, of which the main launch about 320 at 49 % of the issue
// slots (361 instructions a token and 32 channels), the first 105 (its
// multiply-adds alone 60), the sums 16. Each CTA folding the segments itself:
// 482; sweeping the segment again instead of keeping the first launch's states:
// 513. The states take 250 registers; three CTAs with spills took 640. Loading
// a tile's inputs without copying them ahead cost another 200 us. States paired
// over channels instead of over N, so that no step or input has to be copied
// into both halves of a pair: as many instructions, and more of shared memory.
#include "ssm_common.cuh"

namespace gla {
namespace {

using namespace ssm;

constexpr int kTile = 16;          // tokens per tile
constexpr int kWarps = 4, kFoldThreads = 128;
constexpr float kLn2 = 0.6931471805599453f;

template <int K> struct Lane;      // K channels' numbers as one shared-memory access
template <> struct Lane<2> {
    static __device__ __forceinline__ void get(const float *p, float (&v)[2]) {
        const float2 u = *reinterpret_cast<const float2 *>(p);
        v[0] = u.x; v[1] = u.y;
    }
    static __device__ __forceinline__ void put(float *p, const float (&v)[2]) {
        *reinterpret_cast<float2 *>(p) = make_float2(v[0], v[1]);
    }
};
template <> struct Lane<4> {
    static __device__ __forceinline__ void get(const float *p, float (&v)[4]) {
        const float4 u = *reinterpret_cast<const float4 *>(p);
        v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
    }
    static __device__ __forceinline__ void put(float *p, const float (&v)[4]) {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    }
};

// Eight numbers, each spread over the eight quads of a warp: the sum of
// number (lane % 8), in seven exchanges.
__device__ __forceinline__ float across_quads(const float (&v)[8], int lane) {
    float a[4], b[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool up = lane & 4;
        a[i] = (up ? v[i + 4] : v[i]) + __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + 4], 4);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const bool up = lane & 2;
        b[i] = (up ? a[i + 2] : a[i]) + __shfl_xor_sync(0xffffffffu, up ? a[i] : a[i + 2], 2);
    }
    const bool up = lane & 1;
    return (up ? b[1] : b[0]) + __shfl_xor_sync(0xffffffffu, up ? b[0] : b[1], 1);
}

// Shapes of one instance: N states, K channels a lane.
template <int N_> struct Shape {
    static constexpr int N = N_, SP = N / 4, P = SP / 2;
    static constexpr int K = N == 32 ? 2 : 4;         // 16 states a lane at most (8 at N = 8)
    static constexpr int CW = 8 * K, CH = CW * kWarps, VW = CH / 8, TH = 32 * kWarps;
    static constexpr int RS = CH + 8;                 // row step of the [token][channel] arrays
    static constexpr int VPT = kTile * VW / TH;       // vectors a thread loads per tile
    static constexpr int kRow = kTile * RS;           // floats of one such array
    // delta, delta u (then s1), dy' (then y0), s2; B, C; states; dB, dC of every warp
    static constexpr int kCkpt = 3 * K * P * 32 * 2 * kWarps;
    static constexpr int kPart = kWarps * 2 * kTile * N;
    static constexpr int kMain = 4 * kRow + 2 * kTile * N + kCkpt + kPart;
    static constexpr int kLocal = 3 * kRow + 2 * kTile * N;
};

// A thread's vectors of a tile: rows and channels.
template <class S> struct Where {
    int c, vt;
    bool on, whole;
    __device__ __forceinline__ Where(int c0, int D)
        : c(c0 + (int)(threadIdx.x % S::VW) * 8), vt((int)threadIdx.x / S::VW), on(c < D), whole(c + 8 <= D) {}
};

// A tile's inputs on their way: a thread's vectors of x, dt, dy and z and, of
// the first threads, one vector of eight of B or C, copied asynchronously a
// tile ahead into slots that only this thread reads. Two stages at bf16, so
// that the elementwise end still finds its tile there; one at fp32.
template <typename T, class S> struct Ring {
    static constexpr int H = sizeof(T) / 2, kStages = sizeof(T) == 2 ? 2 : 1;
    static constexpr int kPieces = (4 * S::VPT + 1) * H;            // 16-byte slots of a thread and stage
    static constexpr int kNarrow = kTile * S::N / 8;                // vectors of B (and of C)
    static constexpr int kFloats = kStages * kPieces * S::TH * 4;
    static_assert(2 * kNarrow <= S::TH, "one vector of B or C a thread");
    uint4 *slots;
    bool wide;                                                      // B and C allow 16-byte copies

    __device__ __forceinline__ Ring(const SsmBwdParams &p, float *smem) : slots(reinterpret_cast<uint4 *>(smem) + threadIdx.x) {
        wide = ((reinterpret_cast<uintptr_t>(p.Bm) | reinterpret_cast<uintptr_t>(p.Cm) | (uintptr_t)p.ldb * sizeof(T) |
                 (uintptr_t)p.ldc * sizeof(T)) % 16) == 0;
    }
    __device__ __forceinline__ void copy(int stage, int piece, const T *src, bool in, bool whole) const {
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const bool on = in && (h == 0 || whole);
            copy_async<16>(slots + (stage * kPieces + piece * H + h) * S::TH, reinterpret_cast<const uint4 *>(src) + (on ? h : 0), on);
        }
    }
    __device__ __forceinline__ Raw8<T> held(int stage, int piece) const {
        Raw8<T> r;
#pragma unroll
        for (int h = 0; h < H; ++h) r.w[h] = slots[(stage * kPieces + piece * H + h) * S::TH];
        return r;
    }
    // This thread's vector of B (e < kNarrow) or C, or NULL past the tile's end.
    __device__ __forceinline__ const T *narrow(const SsmBwdParams &p, long row0, int ntok, bool grad) const {
        const int e = threadIdx.x, m = e % kNarrow, t = m / (S::N / 8), n = m % (S::N / 8) * 8;
        if (e >= (grad ? 2 : 1) * kNarrow || t >= ntok) return nullptr;
        const size_t row = (size_t)(row0 + t);
        return e < kNarrow ? static_cast<const T *>(p.Bm) + row * p.ldb + n : static_cast<const T *>(p.Cm) + row * p.ldc + n;
    }
    template <bool kGrad> __device__ __forceinline__ void issue(const SsmBwdParams &p, const Where<S> &w, long row0, int ntok, int stage) const {
#pragma unroll
        for (int k = 0; k < S::VPT; ++k) {
            const int t = w.vt + k * (kTile / S::VPT);
            const bool in = w.on && t < ntok;
            const size_t row = in ? (size_t)(row0 + t) : 0;
            const int c = in ? w.c : 0;
            copy(stage, 4 * k, static_cast<const T *>(p.x) + row * p.ldx + c, in, w.whole);
            copy(stage, 4 * k + 1, static_cast<const T *>(p.dt) + row * p.ldt + c, in, w.whole);
            if (kGrad) {
                copy(stage, 4 * k + 2, static_cast<const T *>(p.dy) + row * p.ldg + c, in, w.whole);
                if (p.z) copy(stage, 4 * k + 3, static_cast<const T *>(p.z) + row * p.ldz + c, in, w.whole);
            }
        }
        if (wide) {
            const T *src = narrow(p, row0, ntok, kGrad);
            copy(stage, 4 * S::VPT, src ? src : static_cast<const T *>(p.Bm), src != nullptr, true);
        }
        copies_commit();
    }
    // The tile's delta, delta u and (kGrad) dy', B and C, into shared memory.
    // Steps past the end are 0: they leave both chains as they are.
    template <bool kGrad>
    __device__ __forceinline__ void take(const SsmBwdParams &p, const Where<S> &w, long row0, int ntok, int stage, float *sD, float *sU,
                                         float *sG, float *sB, const f2 (&bias)[4]) const {
#pragma unroll
        for (int k = 0; k < S::VPT; ++k) {
            const int t = w.vt + k * (kTile / S::VPT);
            const bool in = w.on && t < ntok;
            f2 x[4], d[4], g[4];
            raw_unpack(held(stage, 4 * k), x);
            raw_unpack(held(stage, 4 * k + 1), d);
            if (kGrad) {
                raw_unpack(held(stage, 4 * k + 2), g);
                if (p.z) {
                    f2 z[4];
                    raw_unpack(held(stage, 4 * k + 3), z);
#pragma unroll
                    for (int i = 0; i < 4; ++i) g[i] = mul2(g[i], silu2(z[i]));
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                d[i] = add2(d[i], bias[i]);
                if (p.softplus) d[i] = softplus2(d[i]);
                if (!in) d[i] = 0;
                x[i] = mul2(x[i], d[i]);
            }
            const int at = t * S::RS + (int)(threadIdx.x % S::VW) * 8;
            store8(sD + at, d, true);
            store8(sU + at, x, true);
            if (kGrad) store8(sG + at, g, true);
        }
        if (threadIdx.x < (kGrad ? 2 : 1) * kNarrow) {             // C follows B
            f2 v[4];
            if (wide) {
                raw_unpack(held(stage, 4 * S::VPT), v);
            } else {
                const T *src = narrow(p, row0, ntok, kGrad);
                raw_unpack(src ? raw_gather(src) : raw_zero<T>(), v);
            }
            store8(sB + threadIdx.x * 8, v, true);
        }
    }
};

template <class S> struct State {
    f2 v[S::K][S::P];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int k = 0; k < S::K; ++k)
#pragma unroll
            for (int i = 0; i < S::P; ++i) v[k][i] = 0;
    }
    __device__ __forceinline__ void load(const float *src) {                   // src: the first channel's, in [D, N]
#pragma unroll
        for (int k = 0; k < S::K; ++k)
#pragma unroll
            for (int i = 0; i < S::P; ++i) {
                const float2 u = reinterpret_cast<const float2 *>(src + k * S::N)[i];
                v[k][i] = f2_pack(u.x, u.y);
            }
    }
    __device__ __forceinline__ void load_rates(const float *src) {             // as load, of A
#pragma unroll
        for (int k = 0; k < S::K; ++k)
#pragma unroll
            for (int i = 0; i < S::P; ++i) {
                const float2 u = reinterpret_cast<const float2 *>(src + k * S::N)[i];
                v[k][i] = f2_pack(rate_log2(u.x), rate_log2(u.y));
            }
    }
    __device__ __forceinline__ void store(float *dst) const {
#pragma unroll
        for (int k = 0; k < S::K; ++k)
#pragma unroll
            for (int i = 0; i < S::P; ++i) reinterpret_cast<float2 *>(dst + k * S::N)[i] = f2_split(v[k][i]);
    }
};

// h <- exp(delta A) h + (delta u) B for one token of the lane's channels.
template <class S>
__device__ __forceinline__ void advance(State<S> &h, const State<S> &a2, const float *sD, const float *sU, const float *sB) {
    float d[S::K], u[S::K];
    Lane<S::K>::get(sD, d);
    Lane<S::K>::get(sU, u);
    const f2 *b = reinterpret_cast<const f2 *>(sB);
#pragma unroll
    for (int k = 0; k < S::K; ++k) {
        const f2 dd = f2_pack(d[k], d[k]), uu = f2_pack(u[k], u[k]);
#pragma unroll
        for (int i = 0; i < S::P; ++i) h.v[k][i] = fma2(ex2_pair(mul2(dd, a2.v[k][i])), h.v[k][i], mul2(uu, b[i]));
    }
}

// ------------------------------------------------------------ first launch
// Of every tile: the state entering it, from zero at the segment's start, and
// the sum of the steps since (tile_h, tile_sum). With kCut (several segments a
// sequence), of every segment: the state it ends in from zero (seg_h), the c
// that leaves its first token from zero (seg_g), and the sum of its steps.
template <typename T, class S, bool kCut>
__global__ void __launch_bounds__(S::TH, 3) ssm_bwd_local_kernel(const SsmBwdParams p, int tiles) {
    extern __shared__ __align__(16) float smem[];
    float *sD = smem, *sU = sD + S::kRow, *sG = sU + S::kRow, *sB = sG + S::kRow, *sC = sB + kTile * S::N;
    let_next_start();
    const int c0 = (int)(blockIdx.x % (unsigned)tiles) * S::CH;
    const long unit = blockIdx.x / (unsigned)tiles;
    const int b = (int)(unit / p.nseg), seg = (int)(unit % p.nseg);
    const long row0 = (long)b * p.T + (long)seg * p.L;
    const int ntok = (int)min(p.L, (long)p.T - (long)seg * p.L);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, q = lane / 8;
    const int lc = warp * S::CW + lane % 8 * S::K, ch = c0 + lc;
    const size_t cell = (size_t)ch * S::N + q * S::SP;
    const bool on = ch < p.D;
    const Where<S> w(c0, p.D);
    f2 bias[4];
    param8(w.on ? p.dt_bias : nullptr, w.c, w.whole, bias);

    State<S> a2, h, pr, c;
    a2.zero();
    if (on) a2.load_rates(p.A + cell);
    h.zero();
    c.zero();
#pragma unroll
    for (int k = 0; k < S::K; ++k)
#pragma unroll
        for (int i = 0; i < S::P; ++i) pr.v[k][i] = f2_pack(1.f, 1.f);
    float sum[S::K] = {};
    auto enter = [&](size_t tile) {
        if (!on) return;
        h.store(p.tile_h + tile * p.D * S::N + cell);
        if (q == 0) Lane<S::K>::put(p.tile_sum + tile * p.D + ch, sum);
    };
    const Ring<T, S> ring(p, smem + S::kLocal);
    const size_t first = (size_t)b * p.tiles + (size_t)seg * p.L / kTile;   // of the segment's tiles
    const int end = kCut ? ntok : ntok - kTile;                             // not cut: only what enters the last tile
    ring.template issue<kCut>(p, w, row0, ntok, 0);
    for (int t0 = 0; t0 < end; t0 += kTile) {
        copies_wait<0>();
        ring.template take<kCut>(p, w, row0 + t0, ntok - t0, 0, sD, sU, sG, sB, bias);
        if (t0 + kTile < end) ring.template issue<kCut>(p, w, row0 + t0 + kTile, ntok - t0 - kTile, 0);
        if (t0 > 0) enter(first + t0 / kTile);
        __syncthreads();
#pragma unroll 4
        for (int t = 0; t < kTile; ++t) {
            float d[S::K], u[S::K], g[S::K];
            Lane<S::K>::get(sD + t * S::RS + lc, d);
            Lane<S::K>::get(sU + t * S::RS + lc, u);
            if (kCut) Lane<S::K>::get(sG + t * S::RS + lc, g);
            const f2 *bb = reinterpret_cast<const f2 *>(sB + t * S::N + q * S::SP);
            const f2 *cc = reinterpret_cast<const f2 *>(sC + t * S::N + q * S::SP);
#pragma unroll
            for (int k = 0; k < S::K; ++k) {
                const f2 dd = f2_pack(d[k], d[k]), uu = f2_pack(u[k], u[k]), gg = kCut ? f2_pack(g[k], g[k]) : 0;
                sum[k] += d[k];
#pragma unroll
                for (int i = 0; i < S::P; ++i) {
                    const f2 a = ex2_pair(mul2(dd, a2.v[k][i]));
                    h.v[k][i] = fma2(a, h.v[k][i], mul2(uu, bb[i]));
                    if (kCut) {
                        pr.v[k][i] = mul2(pr.v[k][i], a);
                        c.v[k][i] = fma2(pr.v[k][i], mul2(gg, cc[i]), c.v[k][i]);
                    }
                }
            }
        }
        __syncthreads();
    }
    if (!kCut) enter(first + end / kTile + (end % kTile > 0));
    if (kCut && on) {
        h.store(p.seg_h + (size_t)unit * p.D * S::N + cell);
        c.store(p.seg_g + (size_t)unit * p.D * S::N + cell);
        if (q == 0)
#pragma unroll
            for (int k = 0; k < S::K; ++k) p.seg_sum[(size_t)unit * p.D + ch + k] = sum[k];
    }
}

// ------------------------------------------------- between them, when cut
// From what the segments do from zero, the state entering each of them (in
// seg_h's place; blockIdx.y 0) and the c entering it from behind (in seg_g's
// place; 1). Two states a thread; the loads of kAhead segments at once.
template <int N> __global__ void __launch_bounds__(kFoldThreads) ssm_bwd_fold_kernel(const SsmBwdParams p) {
    wait_for_previous();
    let_next_start();
    constexpr int kAhead = 16;
    const long pairs = (long)p.D * N / 2, i = (long)blockIdx.x * kFoldThreads + threadIdx.x;
    if (i >= p.B * pairs) return;
    const long b = i / pairs, e = i % pairs * 2;
    const size_t plane = (size_t)p.D * N;
    const bool back = blockIdx.y;
    const float *first = back ? p.dhT : p.h0;
    float *seg = (back ? p.seg_g : p.seg_h) + b * p.nseg * plane + e;
    const float *sums = p.seg_sum + b * p.nseg * p.D + e / N;
    const float2 a = *reinterpret_cast<const float2 *>(p.A + e);
    const float2 v0 = first ? *reinterpret_cast<const float2 *>(first + b * plane + e) : make_float2(0.f, 0.f);
    const f2 a2 = f2_pack(rate_log2(a.x), rate_log2(a.y));
    f2 v = f2_pack(v0.x, v0.y);
    for (int s = 0; s < p.nseg; s += kAhead) {
        float2 own[kAhead];
        float sum[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (s + k >= p.nseg) break;
            const long u = back ? p.nseg - 1 - s - k : s + k;
            own[k] = *reinterpret_cast<const float2 *>(seg + u * plane);
            sum[k] = sums[u * p.D];
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (s + k >= p.nseg) break;
            const long u = back ? p.nseg - 1 - s - k : s + k;
            *reinterpret_cast<float2 *>(seg + u * plane) = f2_split(v);
            v = fma2(ex2_pair(mul2(both(sum[k]), a2)), v, f2_pack(own[k].x, own[k].y));
        }
    }
}

// ------------------------------------------------------------ last launch
template <typename T, class S>
__global__ void __launch_bounds__(S::TH, 2) ssm_bwd_kernel(const SsmBwdParams p, int tiles) {
    extern __shared__ __align__(16) float smem[];
    float *sD = smem, *sU = sD + S::kRow, *sG = sU + S::kRow, *sS = sG + S::kRow, *sB = sS + S::kRow;
    float *sC = sB + kTile * S::N;
    f2 *sH = reinterpret_cast<f2 *>(sC + kTile * S::N);        // [warp][3][K * P][lane]
    float *sP = reinterpret_cast<float *>(sH) + S::kCkpt;      // [warp][B, C][token][N]
    wait_for_previous();
    let_next_start();
    const int blk = (int)(blockIdx.x % (unsigned)tiles), c0 = blk * S::CH;
    const long unit = blockIdx.x / (unsigned)tiles;
    const int b = (int)(unit / p.nseg), seg = (int)(unit % p.nseg);
    const long row0 = (long)b * p.T + (long)seg * p.L;
    const int ntok = (int)min(p.L, (long)p.T - (long)seg * p.L), ntile = (ntok + kTile - 1) / kTile;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, q = lane / 8;
    const int lc = warp * S::CW + lane % 8 * S::K, ch = c0 + lc;
    const size_t cell = (size_t)ch * S::N + q * S::SP, plane = (size_t)p.D * S::N;
    const bool on = ch < p.D;
    const Where<S> w(c0, p.D);
    f2 bias[4];
    param8(w.on ? p.dt_bias : nullptr, w.c, w.whole, bias);

    // the state entering the segment and the c entering it from behind
    const float *hin = p.nseg > 1 ? p.seg_h + (size_t)unit * plane : p.h0 ? p.h0 + (size_t)b * plane : nullptr;
    const float *cin = p.nseg > 1 ? p.seg_g + (size_t)unit * plane : p.dhT ? p.dhT + (size_t)b * plane : nullptr;
    State<S> a2, c;
    a2.zero();
    c.zero();
    if (on) {
        a2.load_rates(p.A + cell);
        if (cin) c.load(cin + cell);
    }

    const size_t first = (size_t)b * p.tiles + (size_t)seg * p.L / kTile;   // of the segment's tiles
    const Ring<T, S> ring(p, smem + S::kMain);
    f2 skip[4], dskip[4] = {}, dbias[4] = {};
    param8(w.on ? p.skip : nullptr, w.c, w.whole, skip);
    State<S> dA;
    dA.zero();
    f2 *ck = sH + (size_t)warp * 3 * S::K * S::P * 32 + lane;
    float *myP = sP + warp * 2 * kTile * S::N;
    auto keep = [&](int s, const State<S> &v) {
#pragma unroll
        for (int k = 0; k < S::K; ++k)
#pragma unroll
            for (int j = 0; j < S::P; ++j) ck[(s * S::K * S::P + k * S::P + j) * 32] = v.v[k][j];
    };
    auto kept_state = [&](int s, State<S> &v) {
#pragma unroll
        for (int k = 0; k < S::K; ++k)
#pragma unroll
            for (int j = 0; j < S::P; ++j) v.v[k][j] = ck[(s * S::K * S::P + k * S::P + j) * 32];
    };
    // The state entering a tile is exp(A tile_sum) h + tile_h, h the one
    // entering the segment. The three wait in the lane's own places, copied
    // there while the tile behind is finished.
    auto entering = [&](int i) {
        const bool in = on && i > 0;                    // tile 0: h itself
        const size_t tile = first + i;
        const bool h_on = on && hin;
        const float *src = in ? p.tile_h + tile * plane + cell : p.tile_h, *h = h_on ? hin + cell : p.tile_h;
        const float *sum = in ? p.tile_sum + tile * p.D + ch : p.tile_sum;
#pragma unroll
        for (int k = 0; k < S::K; k += 2) copy_async<8>(ck + k / 2 * 32, in ? sum + k : sum, in);   // in the first place
#pragma unroll
        for (int k = 0; k < S::K; ++k)
#pragma unroll
            for (int j = 0; j < S::P; ++j) {
                copy_async<8>(ck + (2 * S::K * S::P + k * S::P + j) * 32, in ? src + k * S::N + 2 * j : src, in);
                copy_async<8>(ck + (S::K * S::P + k * S::P + j) * 32, h_on ? h + k * S::N + 2 * j : h, h_on);
            }
        copies_commit();
    };
    entering(ntile - 1);
    int stage = 0;
    ring.template issue<true>(p, w, row0 + (long)(ntile - 1) * kTile, ntok - (ntile - 1) * kTile, stage);
    for (int i = ntile - 1; i >= 0; --i) {
        const long tr = row0 + (long)i * kTile;
        const int left = min(kTile, ntok - i * kTile);
        copies_wait<0>();
        ring.template take<true>(p, w, tr, left, stage, sD, sU, sG, sB, bias);
        const int kept = stage;
        if (Ring<T, S>::kStages == 2) stage ^= 1;
        if (i > 0) ring.template issue<true>(p, w, tr - kTile, kTile, stage);
        __syncthreads();
        // ---- forward through the tile's first twelve tokens
        State<S> hs[4];
        {
            State<S> in;
            kept_state(2, hs[0]);
            kept_state(1, in);
#pragma unroll
            for (int k = 0; k < S::K; ++k) {
                const float2 pair = f2_split(ck[k / 2 * 32]);
                const f2 sum = both(k % 2 ? pair.y : pair.x);
#pragma unroll
                for (int j = 0; j < S::P; ++j)
                    hs[0].v[k][j] = fma2(ex2_pair(mul2(sum, a2.v[k][j])), in.v[k][j], hs[0].v[k][j]);
            }
        }
#pragma unroll
        for (int s = 0; s < 3; ++s) {
            keep(s, hs[0]);
#pragma unroll
            for (int t = 4 * s; t < 4 * s + 4; ++t)
                advance<S>(hs[0], a2, sD + t * S::RS + lc, sU + t * S::RS + lc, sB + t * S::N + q * S::SP);
        }
        // ---- four tokens at a time, the last first
#pragma unroll 1
        for (int s = 3; s >= 0; --s) {
            if (s < 3) kept_state(s, hs[0]);
            if (s == 0 && i > 0) entering(i - 1);       // (the places have been read)
            const int t0 = 4 * s;
            float pk[S::K][4];                          // a sum over states, per channel and token
            float pn[8];                                // a sum over channels, per token and state
            // the states again, with y0 and dC
            State<S> cur = hs[0];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = t0 + j;
                if (j) hs[j] = cur;
                advance<S>(cur, a2, sD + t * S::RS + lc, sU + t * S::RS + lc, sB + t * S::N + q * S::SP);
                float g[S::K];
                Lane<S::K>::get(sG + t * S::RS + lc, g);
                const f2 *cc = reinterpret_cast<const f2 *>(sC + t * S::N + q * S::SP);
                f2 dc[S::P];
#pragma unroll
                for (int k = 0; k < S::K; ++k) {
                    const f2 gg = f2_pack(g[k], g[k]);
                    f2 y = 0;
#pragma unroll
                    for (int m = 0; m < S::P; ++m) {
                        y = m ? fma2(cur.v[k][m], cc[m], y) : mul2(cur.v[k][m], cc[m]);
                        dc[m] = k ? fma2(gg, cur.v[k][m], dc[m]) : mul2(gg, cur.v[k][m]);
                    }
                    const float2 ys = f2_split(y);
                    pk[k][j] = ys.x + ys.y;
                }
                constexpr int per = 8 / S::SP;          // tokens whose sums fill eight numbers
#pragma unroll
                for (int m = 0; m < S::P; ++m) {
                    const float2 v = f2_split(dc[m]);
                    pn[j % per * S::SP + 2 * m] = v.x;
                    pn[j % per * S::SP + 2 * m + 1] = v.y;
                }
                if (j % per == per - 1) {
                    const int idx = lane % 8;
                    myP[(kTile + t - per + 1 + idx / S::SP) * S::N + q * S::SP + idx % S::SP] = across_quads(pn, lane);
                }
            }
            float y0[S::K];
#pragma unroll
            for (int k = 0; k < S::K; ++k) y0[k] = quad_transpose_sum(pk[k], lane);
            // past the end the step is 0, but 0 x inf would not be: no state there
            if (t0 + 4 > left)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (t0 + j >= left) hs[j].zero();
            // back through them
            float pk2[S::K][4];
#pragma unroll
            for (int j = 3; j >= 0; --j) {
                const int t = t0 + j;
                float d[S::K], u[S::K], g[S::K];
                Lane<S::K>::get(sD + t * S::RS + lc, d);
                Lane<S::K>::get(sU + t * S::RS + lc, u);
                Lane<S::K>::get(sG + t * S::RS + lc, g);
                const f2 *bb = reinterpret_cast<const f2 *>(sB + t * S::N + q * S::SP);
                const f2 *cc = reinterpret_cast<const f2 *>(sC + t * S::N + q * S::SP);
                f2 db[S::P];
#pragma unroll
                for (int k = 0; k < S::K; ++k) {
                    const f2 dd = f2_pack(d[k], d[k]), uu = f2_pack(u[k], u[k]), gg = f2_pack(g[k], g[k]);
                    f2 s1 = 0, s2 = 0;
#pragma unroll
                    for (int m = 0; m < S::P; ++m) {
                        const f2 G = fma2(gg, cc[m], c.v[k][m]);
                        db[m] = k ? fma2(uu, G, db[m]) : mul2(uu, G);
                        s1 = m ? fma2(G, bb[m], s1) : mul2(G, bb[m]);
                        c.v[k][m] = mul2(ex2_pair(mul2(dd, a2.v[k][m])), G);
                        const f2 P = mul2(c.v[k][m], hs[j].v[k][m]);
                        dA.v[k][m] = fma2(dd, P, dA.v[k][m]);
                        s2 = m ? fma2(P, a2.v[k][m], s2) : mul2(P, a2.v[k][m]);
                    }
                    const float2 v1 = f2_split(s1), v2 = f2_split(s2);
                    pk[k][j] = v1.x + v1.y;
                    pk2[k][j] = v2.x + v2.y;
                }
                constexpr int per = 8 / S::SP;
#pragma unroll
                for (int m = 0; m < S::P; ++m) {
                    const float2 v = f2_split(db[m]);
                    pn[j % per * S::SP + 2 * m] = v.x;
                    pn[j % per * S::SP + 2 * m + 1] = v.y;
                }
                if (j % per == 0) {
                    const int idx = lane % 8;
                    myP[(t + idx / S::SP) * S::N + q * S::SP + idx % S::SP] = across_quads(pn, lane);
                }
            }
            // lane q of the quad finishes token t0 + q; every lane of the warp has read the four tokens by now
            float s1[S::K], s2[S::K];
#pragma unroll
            for (int k = 0; k < S::K; ++k) {
                s1[k] = quad_transpose_sum(pk[k], lane);
                s2[k] = quad_transpose_sum(pk2[k], lane);
            }
            __syncwarp();
            const int at = (t0 + q) * S::RS + lc;
            Lane<S::K>::put(sU + at, s1);
            Lane<S::K>::put(sG + at, y0);
            Lane<S::K>::put(sS + at, s2);
        }
        __syncthreads();

        // ---- the elementwise end
#pragma unroll 1
        for (int k = 0; k < S::VPT; ++k) {
            const int t = w.vt + k * (kTile / S::VPT);
            if (!w.on || t >= left) continue;
            const size_t row = (size_t)(tr + t);
            const int at = t * S::RS + tid % S::VW * 8;
            f2 x[4], d[4], g[4], z[4], o[4], s1[4], y0[4], s2[4];
            auto take = [&](const float *src, f2 (&v)[4]) {
                const ulonglong2 a = reinterpret_cast<const ulonglong2 *>(src)[0], b = reinterpret_cast<const ulonglong2 *>(src)[1];
                v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
            };
            auto again = [&](int piece, const void *base, long ld) {
                if (Ring<T, S>::kStages == 2) return ring.held(kept, 4 * k + piece);
                return raw_load(static_cast<const T *>(base) + row * ld + w.c, w.whole);
            };
            raw_unpack(again(0, p.x, p.ldx), x);
            raw_unpack(again(2, p.dy, p.ldg), g);
            if (p.z) {
                raw_unpack(again(3, p.z, p.ldz), z);
                take(sG + at, y0);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const f2 sg = sigmoid2(z[e]), y = fma2(skip[e], x[e], y0[e]), zs = mul2(z[e], sg);
                    // SiLU'(z) = sg + z sg (1 - sg)
                    o[e] = mul2(mul2(g[e], y), fma2(fma2(sg, both(-1.f), both(1.f)), zs, sg));
                    g[e] = mul2(g[e], zs);
                }
                store8(static_cast<T *>(p.dz) + row * p.D + w.c, o, w.whole);
            }
            take(sD + at, d);
            take(sU + at, s1);
            take(sS + at, s2);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                dskip[e] = fma2(g[e], x[e], dskip[e]);
                o[e] = fma2(d[e], s1[e], mul2(skip[e], g[e]));
            }
            store8(static_cast<T *>(p.dx) + row * p.D + w.c, o, w.whole);
            if (p.softplus) raw_unpack(again(1, p.dt, p.ldt), d);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                o[e] = fma2(s2[e], both(kLn2), mul2(s1[e], x[e]));
                if (p.softplus) o[e] = mul2(o[e], sigmoid2(add2(d[e], bias[e])));
                dbias[e] = add2(dbias[e], o[e]);
            }
            store8(static_cast<T *>(p.ddt) + row * p.D + w.c, o, w.whole);
        }
        // dB and dC of the tile, over the warps
        for (int e = tid; e < 2 * kTile * S::N; e += S::TH) {
            const int t = e / S::N % kTile;
            float v = 0.f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) v += sP[k * 2 * kTile * S::N + e];
            if (t < left) {
                float *dst = e < kTile * S::N ? p.part_b : p.part_c;
                dst[((size_t)blk * p.B * p.T + tr + t) * S::N + e % S::N] = v;
            }
        }
        __syncthreads();
    }

    if (on) {
        dA.store(p.part_a + (size_t)unit * plane + cell);
        if (p.dh0 && seg == 0) c.store(p.dh0 + (size_t)b * plane + cell);
    }
    // dskip and ddt_bias: over the threads that share the eight channels
    float *red = smem;                                  // [thread][16]
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 u = f2_split(dskip[e]), v = f2_split(dbias[e]);
        red[2 * e * S::TH + tid] = u.x;
        red[(2 * e + 1) * S::TH + tid] = u.y;
        red[(2 * e + 8) * S::TH + tid] = v.x;
        red[(2 * e + 9) * S::TH + tid] = v.y;
    }
    __syncthreads();
    for (int e = tid; e < 2 * S::CH; e += S::TH) {
        const int which = e / S::CH, lc2 = e % S::CH;
        float v = 0.f;
        for (int r = lc2 / 8; r < S::TH; r += S::VW) v += red[(which * 8 + lc2 % 8) * S::TH + r];
        if (c0 + lc2 < p.D) p.part_v[((size_t)unit * 2 + which) * p.D + c0 + lc2] = v;
    }
}

template <typename T, int N> cudaError_t run(const SsmBwdParams &p, cudaStream_t s, int *launches) {
    using S = Shape<N>;
    const int tiles = (p.D + S::CH - 1) / S::CH;
    const long units = (long)p.B * p.nseg;
    if ((long double)units * tiles > 2147483647.0L) return cudaErrorInvalidValue;
    cudaError_t e;
    if (p.T > kTile) {
        constexpr int bytes = (S::kLocal + Ring<T, S>::kFloats) * (int)sizeof(float);
        auto *kern = p.nseg > 1 ? ssm_bwd_local_kernel<T, S, true> : ssm_bwd_local_kernel<T, S, false>;
        if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) != cudaSuccess) return e;
        kern<<<(unsigned)(units * tiles), S::TH, bytes, s>>>(p, tiles);
        if (launches) ++*launches;
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    if (p.nseg > 1) {
        const dim3 grid((unsigned)(((long)p.B * p.D * N / 2 + kFoldThreads - 1) / kFoldThreads), 2);
        if ((e = launch_behind(ssm_bwd_fold_kernel<N>, grid, kFoldThreads, 0, s, p)) != cudaSuccess) return e;
        if (launches) ++*launches;
    }
    constexpr int bytes = (S::kMain + Ring<T, S>::kFloats) * (int)sizeof(float);
    if ((e = cudaFuncSetAttribute(ssm_bwd_kernel<T, S>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) != cudaSuccess) return e;
    const dim3 grid((unsigned)(units * tiles));
    if (p.T > kTile) {
        e = launch_behind(ssm_bwd_kernel<T, S>, grid, S::TH, bytes, s, p, tiles);
    } else {
        ssm_bwd_kernel<T, S><<<grid, S::TH, bytes, s>>>(p, tiles);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess) return e;
    if (launches) ++*launches;
    SumJobs sums;
    const bool bf16 = sizeof(T) == 2;
    const long cols = (long)p.B * p.T * N, plane = (long)p.D * N;
    sums.add(p.part_b, tiles, cols, cols, p.dB, bf16);
    sums.add(p.part_c, tiles, cols, cols, p.dC, bf16);
    sums.add(p.part_a, units, plane, plane, p.dA);
    sums.add(p.part_v, units, p.D, 2L * p.D, p.dskip);
    sums.add(p.part_v + p.D, units, p.D, 2L * p.D, p.ddt_bias);
    return launch_sums(sums, s, launches);
}

template <typename T> cudaError_t by_state(const SsmBwdParams &p, cudaStream_t s, int *launches) {
    switch (p.N) {
    case 8: return run<T, 8>(p, s, launches);
    case 16: return run<T, 16>(p, s, launches);
    case 32: return run<T, 32>(p, s, launches);
    }
    return cudaErrorInvalidValue;
}

size_t round16(size_t floats) { return (floats + 3) / 4 * 4; }

}  // namespace

constexpr int kRounds = 4, kMostSegments = 128;

// Channels a CTA of the backward owns.
static int bwd_channels(int N) { return N == 32 ? Shape<32>::CH : Shape<16>::CH; }

// Cuts the sequences and lays out the workspace; returns its floats.
size_t plan_ssm_bwd(SsmBwdParams &p, float *ws) {
    const long chains = (long)p.B * ((p.D + bwd_channels(p.N) - 1) / bwd_channels(p.N));
    // Four rounds of the two CTAs an SM holds: the cut costs little (the first
    // launch walks every token once, whatever the cut). 2, 3, 4, 6, 8 rounds at
    // 4 x 2048 x 2048: 495, 475, 455, 455, 461 us. At most 128 segments, a tile
    // each at least: 1 x 4096 x 128 in 64, 128, 256: 55, 41, 46 us; segments of
    // two tiles at least: 2 x 301 x 516 38 us instead of 32.
    long nseg = kRounds * 2L * device_sm_count() / chains;
    if (nseg < 1) nseg = 1;
    if (nseg > kMostSegments) nseg = kMostSegments;
    long L = (p.T + nseg - 1) / nseg;
    L = (L + kTile - 1) / kTile * kTile;
    p.L = L;
    p.nseg = (int)((p.T + L - 1) / L);
    p.tiles = (int)(((long)p.T + kTile - 1) / kTile);
    const size_t plane = (size_t)p.D * p.N, units = (size_t)p.B * p.nseg, blocks = (p.D + bwd_channels(p.N) - 1) / bwd_channels(p.N);
    size_t at = 0;
    auto take = [&](float *&dst, size_t floats) {
        dst = ws ? ws + at : nullptr;
        at += round16(floats);
    };
    take(p.seg_h, p.nseg > 1 ? units * plane : 0);
    take(p.seg_g, p.nseg > 1 ? units * plane : 0);
    take(p.seg_sum, p.nseg > 1 ? units * p.D : 0);
    take(p.tile_h, (size_t)p.B * p.tiles * plane);
    take(p.tile_sum, (size_t)p.B * p.tiles * p.D);
    take(p.part_a, units * plane);
    take(p.part_v, units * 2 * p.D);
    take(p.part_b, blocks * p.B * p.T * p.N);
    take(p.part_c, blocks * p.B * p.T * p.N);
    return at;
}

cudaError_t launch_ssm_bwd(const SsmBwdParams &p, bool bf16, cudaStream_t s, int *launches) {
    return bf16 ? by_state<__nv_bfloat16>(p, s, launches) : by_state<float>(p, s, launches);
}

}  // namespace gla
