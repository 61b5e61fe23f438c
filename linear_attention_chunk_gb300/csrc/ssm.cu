// ssm.cu -- the selective state-space scan over prompts and training
// sequences, with the causal depthwise Conv1d fused in front when asked.
//
// Per sequence, channel d and state n, with delta = softplus(dt + bias):
//     h_t = exp(delta_t A[d][n]) h_{t-1} + delta_t B_t[n] u_t[d]
//     y_t = (sum_n C_t[n] h_t + skip[d] u_t[d]) SiLU(z_t[d])
// The decay differs by channel and state, so a chunk has no matrix-product
// form (the decays do not factor into one weight per token pair): the work is
// one exponential and four fp32 operations per (token, channel, state).
//
// Layout: a warp owns sixteen channels of one sequence (or of one segment of
// it) and walks it alone, 16 tokens at a time; a CTA is only a group of such
// warps, with no barrier between them, so their phases overlap. A quad of
// lanes (eight apart) owns two channels, each lane N / 4 of their states, in
// registers as fp32 pairs for the whole run. Two channels a lane halve the
// loads of B and C: shared memory fills registers at 128 bytes a clock per SM,
// and one channel a lane was bound by that. Per tile, every lane loads eight
// channels of one token (16-byte accesses; the next tile's are in flight
// during the scan), forms the input u and the step delta, and leaves
// (delta, delta u) in the warp's shared memory; then the warp walks the tokens;
// then the lane that loaded a vector adds the skip, applies the gate and
// stores it. Each elementwise value is computed once, and the quad's sums over
// states are exchanged four tokens at a time.
//
// Sequences are cut into segments when they are too few to fill the GPU: one
// launch runs every segment but a sequence's last (the first from the initial
// state, the others from zero) and leaves its final state and the sum of its
// steps; in the second launch each segment folds the ones before it,
// h <- exp(A sum delta) h + h_local, and runs from there. No CTA waits on
// another.
//
// Where no SM gets more than eight warps (`roomy`), the registers are there to
// read a step's four tokens from shared memory while the four before are
// walked: 8 x 2048 x 2048 201 us instead of 221; with more warps the registers
// that this takes cost more (packed prompts, below: 666 us).
//
// Measured: 8 x 2048 x 2048 at N = 16, bf16 with the gate, 201 us (271 MB; the
// exponentials and multiply-adds alone about 80 us): 55 instructions a token
// and 16 channels, and seven warps an SM that issue every second clock. Packed
// prompts of 16,024 tokens x 4,096 with the filter 614 us in two launches.
// Slower for the first: one channel a lane with 1, 2 or 4 lanes a channel (238
// to 303 us), a ring of asynchronous copies (no change: it does not wait for
// DRAM), a helper warp for the elementwise work (227 to 268 us), the next
// tile's elementwise work beside the scan (213), two or three segments (268 to
// 306 us).
#include "ssm_common.cuh"

namespace gla {
namespace {

using namespace ssm;

constexpr int kTile = 16;   // tokens per tile: 2 x 16 vectors of eight channels, one a lane
constexpr int kChan = 16;   // channels of a warp
constexpr int kMostWarps = 4, kMinBlocks = 4, kRoomyBlocks = 2;   // of a CTA; CTAs an SM holds (roomy: two)

// Shared memory of a warp: (delta, delta u) of the tile, y, B, C; the filter
// and the inputs of this tile and the one before (as they lie in memory).
template <typename T, int N, bool kConv> constexpr int warp_floats() {
    return kTile * kChan * 3 + 2 * kTile * N + (kConv ? (kTaps + 1) * kChan + 2 * 32 * 2 * (int)sizeof(T) : 0);
}

// The unit's sequence, its segment and its tokens. False: nothing to do.
struct Unit {
    int seq, seg, slot;
    long first;    // row of the sequence's first token
    long len;      // tokens of the sequence
    long base;     // first segment slot of the sequence in the workspace
    int nseg;      // segments of the sequence
};

// Varlen: the segments of sequence n take the slots cu[n] / L + n, ... (as
// many as ceil(length / L)): slots of different sequences cannot meet, and
// no prefix sum is needed. Every thread returns the same answer.
__device__ __forceinline__ bool find_unit(const SsmParams &p, long u, int *s_found, Unit &un) {
    if (!p.cu_seqlens) {
        un.seq = (int)(u / p.nseg);
        un.seg = (int)(u % p.nseg);
        un.slot = un.seq;
        un.first = (long)un.seq * p.T;
        un.len = p.T;
        un.base = (long)un.seq * p.nseg;
        un.nseg = p.nseg;
        return true;
    }
    if (threadIdx.x == 0) *s_found = p.nseq;
    __syncthreads();
    for (int n = threadIdx.x; n < p.nseq; n += blockDim.x) {
        const long s = p.cu_seqlens[n], e = p.cu_seqlens[n + 1];
        const int slot = p.slots ? p.slots[n] : n;
        if (s < 0 || e < s || e > p.rows || slot < 0 || slot >= p.n_slots) {
            if (u == 0) atomicOr(p.status, kDevBadState);
            if (e < s) atomicMin(s_found, -1);          // segments of several sequences would share slots: none runs
            continue;
        }
        const long b = s / p.L + n;
        if (u >= b && u < b + (e - s + p.L - 1) / p.L) atomicMin(s_found, n);
    }
    __syncthreads();
    const int n = *s_found;
    if (n < 0 || n >= p.nseq) return false;
    un.seq = n;
    un.first = p.cu_seqlens[n];
    un.len = p.cu_seqlens[n + 1] - un.first;
    un.base = un.first / p.L + n;
    un.seg = (int)(u - un.base);
    un.nseg = (int)((un.len + p.L - 1) / p.L);
    un.slot = p.slots ? p.slots[n] : n;
    return true;
}

// The filter's input at a row before the unit's first token, eight channels:
// from x inside the sequence, from the window before its first token (rows
// oldest first, the last four inputs).
template <typename T>
__device__ __forceinline__ void before(const SsmParams &p, const Unit &un, long src, int c, bool whole, f2 (&v)[4]) {
    if (src >= un.first) {
        raw_unpack(raw_load(static_cast<const T *>(p.x) + (size_t)src * p.ldx + c, whole), v);
        return;
    }
    // plain loads: this launch rewrites the window later
    const float4 *r = reinterpret_cast<const float4 *>(p.win + ((size_t)un.slot * kTaps + (kTaps + src - un.first)) * p.D + c);
    const float4 a = r[0], b = whole ? r[1] : make_float4(0.f, 0.f, 0.f, 0.f);
    v[0] = f2_pack(a.x, a.y);
    v[1] = f2_pack(a.z, a.w);
    v[2] = f2_pack(b.x, b.y);
    v[3] = f2_pack(b.z, b.w);
}

__device__ __forceinline__ void four(const float *src, f2 (&v)[4]) {   // eight floats of shared memory
    const ulonglong2 a = reinterpret_cast<const ulonglong2 *>(src)[0], b = reinterpret_cast<const ulonglong2 *>(src)[1];
    v[0] = a.x;
    v[1] = a.y;
    v[2] = b.x;
    v[3] = b.y;
}

template <typename T, int N, bool kFull, bool kConv, bool kRoomy>
__global__ void __launch_bounds__(32 * kMostWarps, kRoomy ? kRoomyBlocks : kMinBlocks) ssm_scan_kernel(const SsmParams p, int tiles) {
    constexpr int SP = N / 4, P = SP / 2;
    extern __shared__ __align__(16) float smem[];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, q = lane / 8;
    float *mine = smem + warp * warp_floats<T, N, kConv>();
    float4 *sD = reinterpret_cast<float4 *>(mine);     // [kTile][8 channel pairs, swizzled]
    float *sY = mine + kTile * kChan * 2;              // [kTile][kChan]
    float *sB = sY + kTile * kChan;                    // [kTile][N]
    float *sC = sB + kTile * N;
    float *sW = sC + kTile * N;                        // [taps and bias][kChan]
    uint4 *sX = reinterpret_cast<uint4 *>(sW + (kTaps + 1) * kChan);   // [tile parity][piece][vector]
    __shared__ int s_found;

    const int c0 = ((int)(blockIdx.x % (unsigned)tiles) * (int)(blockDim.x / 32) + warp) * kChan;
    const long unit = blockIdx.x / (unsigned)tiles;
    Unit un;
    if (!find_unit(p, unit, &s_found, un)) return;
    const long seg0 = (long)un.seg * p.L;
    const long row0 = un.first + seg0;
    const int ntok = (int)min((long)p.L, un.len - seg0);
    const bool last = seg0 + p.L >= un.len;
    if (!kFull && last) return;

    if (c0 >= p.D) return;                             // a warp past the last channel
    // the vector this lane loads and stores: channels c .. c+7 of token vt of every tile
    const int vt = lane / 2, c = c0 + lane % 2 * kVec;
    const bool vec_on = c < p.D, whole = c + kVec <= p.D;
    // the two channels and the states this lane scans
    const int ch = c0 + lane % 8 * 2;
    const bool ch_on = ch < p.D;                       // D is even

    f2 a2[2][P], h[2][P];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < P; ++i) a2[k][i] = h[k][i] = 0;
    const size_t cell = (size_t)ch * N + q * SP;       // of this lane's states in a [D, N] array; the second channel's
    if (ch_on) {                                       // are N further
        // The state entering the unit. The last segment of a sequence has no
        // local pass, and its workspace slot keeps a copy of the initial state:
        // the second launch overwrites the pool, and reads the copy instead.
        const float *src = nullptr;
        if (un.seg == 0 && (!kFull || un.nseg == 1)) {
            src = p.h0 ? p.h0 + (size_t)un.slot * p.D * N + cell : nullptr;
        } else if (kFull) {
            src = p.seg_h + (size_t)(un.base + (un.seg == 0 ? un.nseg - 1 : 0)) * p.D * N + cell;
        }
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const float2 a = __ldg(reinterpret_cast<const float2 *>(p.A + cell + k * N) + i);
                a2[k][i] = f2_pack(rate_log2(a.x), rate_log2(a.y));
                if (src) {
                    const float2 v = reinterpret_cast<const float2 *>(src + k * N)[i];
                    h[k][i] = f2_pack(v.x, v.y);
                }
            }
        if (!kFull && un.seg == 0) {
            float *dst = p.seg_h + (size_t)(un.base + un.nseg - 1) * p.D * N + cell;
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int i = 0; i < P; ++i) reinterpret_cast<float2 *>(dst + k * N)[i] = f2_split(h[k][i]);
        }
        if (kFull) {                                   // the first segment's state is final; fold the others
#pragma unroll 2
            for (int s = 1; s < un.seg; ++s) {
                const size_t slot = (size_t)(un.base + s);
                const float2 sum = *reinterpret_cast<const float2 *>(p.seg_sum + slot * p.D + ch);
                const float *e = p.seg_h + slot * p.D * N + cell;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const f2 ss = k ? f2_pack(sum.y, sum.y) : f2_pack(sum.x, sum.x);
#pragma unroll
                    for (int i = 0; i < P; ++i) {
                        const float2 v = reinterpret_cast<const float2 *>(e + k * N)[i];
                        h[k][i] = fma2(ex2_pair(mul2(ss, a2[k][i])), h[k][i], f2_pack(v.x, v.y));
                    }
                }
            }
        }
    }

    if (kConv) {
        if (lane < kChan) {
            const bool in = c0 + lane < p.D;
            const float4 w = in ? __ldg(reinterpret_cast<const float4 *>(p.conv_w) + c0 + lane)
                                : make_float4(0.f, 0.f, 0.f, 0.f);
            sW[lane] = w.x;
            sW[kChan + lane] = w.y;
            sW[2 * kChan + lane] = w.z;
            sW[3 * kChan + lane] = w.w;
            sW[4 * kChan + lane] = p.conv_b && in ? p.conv_b[c0 + lane] : 0.f;
        }
        __syncwarp();
    }
    f2 bias[4], skip[4];
    param8(vec_on ? p.dt_bias : nullptr, c, whole, bias);
    if (kFull) param8(vec_on ? p.skip : nullptr, c, whole, skip);

    // One tile's inputs as they lie in memory; B and C as vectors of eight too.
    // A lane past the last channel repeats the warp's first vector, and nothing
    // of it is kept; tokens past the end are looked after in the last tile only.
    constexpr int H = sizeof(T) / 2;
    constexpr int BV = kTile * N / 8, BL = (BV + 31) / 32;   // vectors of B (and of C), and per lane
    const int cv = vec_on ? c : c0;
    const bool cw = vec_on ? whole : c0 + kVec <= p.D;
    const T *px = static_cast<const T *>(p.x) + (size_t)(row0 + vt) * p.ldx + cv;
    const T *pd = static_cast<const T *>(p.dt) + (size_t)(row0 + vt) * p.ldt + cv;
    const T *pz = kFull && p.z ? static_cast<const T *>(p.z) + (size_t)(row0 + vt) * p.ldz + cv : nullptr;
    const int bt = lane / (N / 8), bn = lane % (N / 8) * 8;  // token and first state of this lane's first vector
    const T *pb = static_cast<const T *>(p.Bm) + (size_t)(row0 + bt) * p.ldb + bn;
    const T *pc = static_cast<const T *>(p.Cm) + (size_t)(row0 + bt) * p.ldc + bn;
    const bool wide = ((reinterpret_cast<uintptr_t>(p.Bm) | reinterpret_cast<uintptr_t>(p.Cm) | (uintptr_t)p.ldb * sizeof(T) |
                        (uintptr_t)p.ldc * sizeof(T)) % 16) == 0;
    Raw8<T> rx, rd, rz = raw_zero<T>(), rb[BL], rc[BL];
    auto narrow = [&](const T *src) { return wide ? raw_load(src, true) : raw_gather(src); };
    auto fetch = [&](int left) {                             // the next tile, of which `left` tokens exist
        constexpr int step = 32 / (N / 8);                   // tokens from one of this lane's vectors to the next
        if (left >= kTile) {
            rx = raw_load(px, cw);
            rd = raw_load(pd, cw);
            if (pz) rz = raw_load(pz, cw);
#pragma unroll
            for (int i = 0; i < BL; ++i) {
                if (BV % 32 != 0 && lane >= BV) break;
                rb[i] = narrow(pb + (size_t)(i * step) * p.ldb);
                if (kFull) rc[i] = narrow(pc + (size_t)(i * step) * p.ldc);
            }
        } else {
            const bool in = vt < left;
            rx = in ? raw_load(px, cw) : raw_zero<T>();
            rd = in ? raw_load(pd, cw) : raw_zero<T>();
            if (pz) rz = in ? raw_load(pz, cw) : raw_zero<T>();
#pragma unroll
            for (int i = 0; i < BL; ++i) {
                const bool on = i * 32 + lane < BV && bt + i * step < left;
                rb[i] = on ? narrow(pb + (size_t)(i * step) * p.ldb) : raw_zero<T>();
                if (kFull) rc[i] = on ? narrow(pc + (size_t)(i * step) * p.ldc) : raw_zero<T>();
            }
        }
        px += (size_t)kTile * p.ldx;
        pd += (size_t)kTile * p.ldt;
        if (pz) pz += (size_t)kTile * p.ldz;
        pb += (size_t)kTile * p.ldb;
        pc += (size_t)kTile * p.ldc;
    };
    fetch(ntok);

    T *py = static_cast<T *>(p.y) + (size_t)(row0 + vt) * p.D + c;
    float dsum[2] = {0.f, 0.f};
    int par = 0;                                             // the tile's parity
    for (int left = ntok; left > 0; left -= kTile, par ^= 1) {
        // ---- inputs of the tile: u, delta; zero steps past the end leave the state as it is
        f2 u[4], dl[4];
        raw_unpack(rd, dl);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            dl[i] = add2(dl[i], bias[i]);
            if (p.softplus) dl[i] = softplus2(dl[i]);
        }
        if (left < kTile && vt >= left)
#pragma unroll
            for (int i = 0; i < 4; ++i) dl[i] = 0;
        raw_unpack(rx, u);
        if (kConv) {
            // the three rows before this lane's come from the lanes that loaded them, in this tile or the one before
#pragma unroll
            for (int i = 0; i < H; ++i) sX[(par * H + i) * 32 + lane] = rx.w[i];
            __syncwarp();
            const float *w = sW + lane % 2 * kVec;
            f2 acc[4];
            four(w + kTaps * kChan, acc);
#pragma unroll
            for (int j = 0; j < kTaps; ++j) {
                f2 v[4], wj[4];
                if (j == kTaps - 1) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = u[i];
                } else if (left == ntok && vt < 3 - j) {     // before the unit
                    before<T>(p, un, row0 + vt - 3 + j, cv, cw, v);
                } else {
                    const int from = lane - 2 * (3 - j);
                    Raw8<T> r;
#pragma unroll
                    for (int i = 0; i < H; ++i) r.w[i] = sX[((from < 0 ? par ^ 1 : par) * H + i) * 32 + (from & 31)];
                    raw_unpack(r, v);
                }
                four(w + j * kChan, wj);
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i] = fma2(wj[i], v[i], acc[i]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) u[i] = left < kTile && vt >= left ? 0 : silu2(acc[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {                  // four tokens' 128-byte rows over all the banks
            const float2 d = f2_split(dl[i]), du = f2_split(mul2(dl[i], u[i]));
            sD[vt * 8 + lane % 2 * 4 + (i ^ (vt & 3))] = make_float4(d.x, du.x, d.y, du.y);
        }
#pragma unroll
        for (int i = 0; i < BL; ++i) {
            const int e = i * 32 + lane;
            if (e < BV) {
                f2 v[4];
                raw_unpack(rb[i], v);
                store8(sB + e * 8, v, true);
                if (kFull) {
                    raw_unpack(rc[i], v);
                    store8(sC + e * 8, v, true);
                }
            }
        }
        const Raw8<T> zc = rz;
        __syncwarp();
        if (left > kTile) fetch(left - kTile);

        // ---- the scan: the tile's tokens
        float4 d4[2][4];                               // four tokens' delta and delta u, B, C
        f2 b4[2][4][P], c4[2][4][P];
        auto look = [&](int t, int at) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                d4[at][j] = sD[(t + j) * 8 + ((lane % 8) ^ ((t + j) & 3))];
                const f2 *b = reinterpret_cast<const f2 *>(sB + (t + j) * N + q * SP);
                const f2 *cc = reinterpret_cast<const f2 *>(sC + (t + j) * N + q * SP);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    b4[at][j][i] = b[i];
                    if (kFull) c4[at][j][i] = cc[i];
                }
            }
        };
        if (kRoomy) look(0, 0);
#pragma unroll
        for (int t = 0; t < kTile; t += 4) {
            const int at = kRoomy ? t / 4 % 2 : 0;
            if (!kRoomy) look(t, 0);
            if (kRoomy && t + 4 < kTile) look(t + 4, at ^ 1);
            // the decays and products of four tokens first, then the chain through them
            f2 e[4][2][P], x[4][2][P];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float4 d = d4[at][j];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const f2 dd = both(k ? d.z : d.x), du = both(k ? d.w : d.y);
#pragma unroll
                    for (int i = 0; i < P; ++i) {
                        e[j][k][i] = ex2_pair(mul2(dd, a2[k][i]));
                        x[j][k][i] = mul2(du, b4[at][j][i]);
                    }
                    if (!kFull) dsum[k] += k ? d.z : d.x;
                }
            }
            float part[2][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    f2 y = 0;
#pragma unroll
                    for (int i = 0; i < P; ++i) {
                        h[k][i] = fma2(e[j][k][i], h[k][i], x[j][k][i]);
                        if (kFull) y = i == 0 ? mul2(h[k][i], c4[at][j][i]) : fma2(h[k][i], c4[at][j][i], y);
                    }
                    if (kFull) {
                        const float2 ys = f2_split(y);
                        part[k][j] = ys.x + ys.y;
                    }
                }
            }
            if (kFull)
                *reinterpret_cast<float2 *>(sY + (t + q) * kChan + lane % 8 * 2) =
                    make_float2(quad_transpose_sum(part[0], lane), quad_transpose_sum(part[1], lane));
        }
        __syncwarp();

        // ---- skip, gate, store
        if (kFull) {
            f2 y[4], z[4];
            four(sY + vt * kChan + lane % 2 * kVec, y);
            raw_unpack(zc, z);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                y[i] = fma2(skip[i], u[i], y[i]);
                if (p.z) y[i] = mul2(y[i], silu2(z[i]));
            }
            if (vec_on && (left >= kTile || vt < left)) store8(py, y, whole);
            py += (size_t)kTile * p.D;
        }
    }

    // ---- the state after the unit
    if (ch_on) {
        float *dst = nullptr;
        if (!kFull) dst = p.seg_h + (size_t)(un.base + un.seg) * p.D * N + cell;
        else if (last && p.hT) dst = p.hT + (size_t)un.slot * p.D * N + cell;
        if (dst) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int i = 0; i < P; ++i) reinterpret_cast<float2 *>(dst + k * N)[i] = f2_split(h[k][i]);
        }
        if (!kFull && q == 0)
            *reinterpret_cast<float2 *>(p.seg_sum + (size_t)(un.base + un.seg) * p.D + ch) = make_float2(dsum[0], dsum[1]);
    }
    // ---- the window after the call: of these channels this warp alone reads
    // it (at the sequence's first tokens), and has done so before the last __syncwarp
    if (kFull && kConv && un.seg == 0 && lane < kChan) {
        const int cc = c0 + lane;
        if (cc < p.D) {
            float *w = p.win + (size_t)un.slot * kTaps * p.D + cc;
#pragma unroll
            for (int k = 0; k < kTaps; ++k) {
                const long src = un.len - kTaps + k;   // row k after the call; an old row has a larger index
                w[(size_t)k * p.D] = src >= 0 ? Elem<T>::load(static_cast<const T *>(p.x) +
                                                              (size_t)(un.first + src) * p.ldx + cc)
                                              : w[(size_t)(kTaps + src) * p.D];
            }
        }
    }
}

// Warps per CTA: four neighbours share cache lines of the activations and of
// B and C; fewer where that leaves the SMs with unequal numbers of warps.
int warps_per_block(long units, int D) {
    const int sms = device_sm_count(), groups = (D + kChan - 1) / kChan;
    int best = 1;
    double least = 1e30;
    for (int w = kMostWarps; w >= 1; w /= 2) {
        const long blocks = units * ((groups + w - 1) / w);
        const double load = (double)((blocks + sms - 1) / sms) * w;   // warps of the fullest SM
        if (load < least * 0.93) {
            least = load;
            best = w;
        }
    }
    return best;
}

template <typename T, int N, bool kFull, bool kConv>
cudaError_t launch(const SsmParams &p, long units, cudaStream_t s, int *launches) {
    const int w = warps_per_block(units, p.D), tiles = (p.D + kChan * w - 1) / (kChan * w);
    if ((long double)units * tiles > 2147483647.0L) return cudaErrorInvalidValue;
    const int bytes = w * warp_floats<T, N, kConv>() * (int)sizeof(float);
    const long per_sm = (units * tiles + device_sm_count() - 1) / device_sm_count() * w;   // warps of the fullest SM
    auto *kern = ssm_scan_kernel<T, N, kFull, kConv, false>;
    if constexpr (kFull)
        if (per_sm <= kRoomyBlocks * kMostWarps) kern = ssm_scan_kernel<T, N, kFull, kConv, true>;
    kern<<<(unsigned)(units * tiles), 32 * w, bytes, s>>>(p, tiles);
    if (launches) ++*launches;
    return cudaGetLastError();
}

template <typename T, int N, bool kConv> cudaError_t run(const SsmParams &p, cudaStream_t s, int *launches) {
    const long units = p.cu_seqlens ? p.rows / p.L + p.nseq : (long)p.nseq * p.nseg;
    if (p.seg_h) {
        const cudaError_t e = launch<T, N, false, kConv>(p, units, s, launches);
        if (e != cudaSuccess) return e;
    }
    return launch<T, N, true, kConv>(p, units, s, launches);
}

template <typename T, bool kConv> cudaError_t by_state(const SsmParams &p, cudaStream_t s, int *launches) {
    switch (p.N) {
    case 8: return run<T, 8, kConv>(p, s, launches);
    case 16: return run<T, 16, kConv>(p, s, launches);
    case 32: return run<T, 32, kConv>(p, s, launches);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_ssm_scan(const SsmParams &p, bool bf16, cudaStream_t s, int *launches) {
    if (p.conv_w)
        return bf16 ? by_state<__nv_bfloat16, true>(p, s, launches) : by_state<float, true>(p, s, launches);
    return bf16 ? by_state<__nv_bfloat16, false>(p, s, launches) : by_state<float, false>(p, s, launches);
}

// The segment length, a multiple of the tile. A token costs the first launch
// two thirds of what it costs the second (packed prompts of 16,024 tokens x
// 4,096 with the filter: 211 us for the 12,800 that it walks, then 401).
// Equal-length sequences are cut where there are fewer than twelve groups of
// eight channels (half a warp's) an SM, into twice as many pieces. Cut and
// whole, us, B x 2048 x 2048: B = 1: 59, 135; 2: 91, 137; 3: 145, 139; 4: 166,
// 143; 5: 201, 195; 6: 227, 199; 7: 268, 199; 8 is left whole: 201. So the rule
// cuts too far from three such sequences on.
// Packed prompts are always cut, into 512 tokens at most: the prompts above 615
// and 629 us, with 5,120 channels 756 and 645, 64 prompts of 512 tokens x 4,096
// 773 and 754, of 2,048 tokens 4,401 and 2,893. It gains where few long prompts
// would leave SMs idle and costs where there are chains enough.
// The last launch folds the segments one after another: 1 x 4096 x 128 31 us
// instead of 264, 1 x 65536 x 256 180 instead of 4,112.
SsmPlan plan_ssm(long nseq, long rows, int D, bool varlen) {
    const long warps = nseq * ((D + 7) / 8);
    const long want = (long)device_sm_count() * 12;
    const long mean = nseq > 0 ? (rows + nseq - 1) / nseq : 0;
    SsmPlan pl{rows > 0 ? rows : 1, 1};
    if (rows <= 0 || nseq <= 0) return pl;
    if (!varlen && warps >= want) return SsmPlan{mean, 1};
    long nseg = (2 * want + warps - 1) / warps;
    long L = (mean + nseg - 1) / nseg;
    L = (L + 63) / 64 * 64;
    if (varlen && L > 512) L = 512;
    if (!varlen && 2 * L >= mean) return SsmPlan{mean, 1};   // two segments cost as much as they save
    if (varlen && L >= rows) return SsmPlan{rows, nseq};
    pl.L = L;
    pl.slots = varlen ? rows / L + nseq : nseq * ((mean + L - 1) / L);
    return pl;
}

// Segment states and sums of steps, [slots, D, N] and [slots, D] fp32.
size_t ssm_workspace_bytes(const SsmPlan &plan, long nseq, int D, int N) {
    return plan.slots <= nseq ? 0 : (size_t)plan.slots * D * (N + 1) * sizeof(float);
}

}  // namespace gla
