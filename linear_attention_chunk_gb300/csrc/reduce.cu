// reduce.cu -- the second stage of the parameter gradients: sums over the rows
// of fp32 [rows, cols] arrays of partial results, one row per CTA (or group of
// CTAs) of the first stage. In a fixed order, so results do not change from
// call to call (atomics would). All of a call's sums are one launch.
//
// Up to 32 rows, a thread adds four columns down the rows (16-byte loads).
// More rows, a CTA owns 32 columns and its 16 warps take every sixteenth row
// (128 contiguous bytes each), added up by shuffles and through shared memory.
// Few columns and many rows, where such CTAs would leave most SMs idle and
// wait for several rounds of loads: 8 columns and 64 groups of eight lanes, so
// that 456 rows are one round of loads (norm gradients at 16384 x 2048: 51 ->
// 49 us; with 20,480 columns of 128 rows it cost 6 us).
#include "ssm_common.cuh"

namespace gla {
namespace {

constexpr int kThreads = 512, kFew = 32, kBatch = 8;

__device__ __forceinline__ void put(const SumJob &j, long c, float v) {
    if (j.bf16) static_cast<__nv_bfloat16 *>(j.out)[c] = __float2bfloat16_rn(v);
    else static_cast<float *>(j.out)[c] = v;
}

__global__ void __launch_bounds__(kThreads) sum_rows_kernel(const SumJobs jobs) {
    __shared__ float s[kThreads / 32][32];
    ssm::wait_for_previous();   // (and plain loads: the read-only path may run ahead of it)
    int k = 0;
    while (k + 1 < jobs.n && blockIdx.x >= jobs.j[k + 1].block) ++k;
    const SumJob &j = jobs.j[k];
    const long blk = (long)blockIdx.x - j.block;
    if (j.rows <= kFew) {
        const long c = (blk * kThreads + threadIdx.x) * 4;
        if (c >= j.cols) return;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (long r = 0; r < j.rows; r += kBatch) {       // loads together, also of the last rows
            float4 u[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                u[i] = r + i < j.rows ? __ldcg(reinterpret_cast<const float4 *>(j.part + (size_t)(r + i) * j.pitch + c))
                                      : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                v.x += u[i].x;
                v.y += u[i].y;
                v.z += u[i].z;
                v.w += u[i].w;
            }
        }
        put(j, c, v.x);
        put(j, c + 1, v.y);
        put(j, c + 2, v.z);
        put(j, c + 3, v.w);
        return;
    }
    constexpr int W = kThreads / 32;
    const int w = j.width, G = kThreads / w;   // columns, groups of lanes
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const long c = blk * w + lane % w;
    float acc[8] = {};
    if (c < j.cols) {
        const float *p = j.part + c;
        for (long r = threadIdx.x / w; r < j.rows; r += 8 * G)
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] += r + i * G < j.rows ? __ldcg(p + (size_t)(r + i * G) * j.pitch) : 0.f;
    }
    float v = ((acc[0] + acc[1]) + (acc[2] + acc[3])) + ((acc[4] + acc[5]) + (acc[6] + acc[7]));
    for (int off = 16; off >= w; off /= 2) v += __shfl_xor_sync(0xffffffffu, v, off);
    if (lane < w) s[warp][lane] = v;
    __syncthreads();
    if (threadIdx.x < w && c < j.cols) {
        v = 0.f;
#pragma unroll
        for (int i = 0; i < W; ++i) v += s[i][threadIdx.x];
        put(j, c, v);
    }
}

}  // namespace

void SumJobs::add(const float *part, long rows, long cols, long pitch, void *out, bool bf16) {
    if (!out || cols == 0) return;
    const int width = cols < 64L * device_sm_count() && rows > 256 ? 8 : 32;   // (two CTAs of 32 columns an SM; two rounds of loads)
    const long per = rows <= kFew ? 4L * kThreads : width;
    j[n] = SumJob{part, rows, cols, pitch, out, bf16, width, blocks};
    blocks += (unsigned)((cols + per - 1) / per);
    ++n;
}

cudaError_t launch_sums(const SumJobs &jobs, cudaStream_t s, int *launches) {
    if (jobs.n == 0) return cudaSuccess;
    const cudaError_t e = ssm::launch_behind(sum_rows_kernel, dim3(jobs.blocks), kThreads, 0, s, jobs);
    if (e == cudaSuccess && launches) ++*launches;
    return e;
}

}  // namespace gla
