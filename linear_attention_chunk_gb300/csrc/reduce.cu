// reduce.cu -- the second stage of the parameter gradients: the sum over rows
// of an fp32 [rows, cols] array of partial sums, one partial per CTA of the
// first stage. In a fixed order, so results do not change from call to call
// (atomics would). A CTA owns 32 columns; its 32 warps take every 32nd row
// (128 contiguous bytes each) and are added up through shared memory.
#include "kernels.h"

namespace gla {
namespace {

__global__ void __launch_bounds__(1024) sum_rows_kernel(const float *part, long rows, long cols, long pitch, float *out) {
    __shared__ float s[32][33];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const long c = (long)blockIdx.x * 32 + lane;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    if (c < cols) {
        const float *p = part + c;
        long r = warp;
        for (; r + 96 < rows; r += 128)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] += p[(size_t)(r + 32 * i) * pitch];
        for (; r < rows; r += 32) acc[0] += p[(size_t)r * pitch];
    }
    s[warp][lane] = (acc[0] + acc[1]) + (acc[2] + acc[3]);
    __syncthreads();
    float v = s[lane][warp];   // warp w finishes column w
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    const long oc = (long)blockIdx.x * 32 + warp;
    if (lane == 0 && oc < cols) out[oc] = v;
}

}  // namespace

cudaError_t launch_sum_rows(const float *part, long rows, long cols, long pitch, float *out, cudaStream_t s, int *launches) {
    if (cols == 0 || out == nullptr) return cudaSuccess;
    sum_rows_kernel<<<(unsigned)((cols + 31) / 32), 1024, 0, s>>>(part, rows, cols, pitch, out);
    if (launches) ++*launches;
    return cudaGetLastError();
}

}  // namespace gla
