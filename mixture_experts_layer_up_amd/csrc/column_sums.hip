// column_sums.hip -- sums over the rows of a small fp32 table: column sums that
// blocks kept apart are joined in a fixed order.  A block owns 64 columns, its 16
// waves every 16th row each, joined through LDS.  Bound by the latency of a wave's
// chain of loads: 256 rows of 6144 columns (6.3 MB).
#include "device_common.h"
#include "kernels_block.h"

namespace moe_lora {
namespace {

constexpr int kWaves = 16;

__global__ __launch_bounds__(kWaves * kWave) void column_sums_kernel(const float *in, int rows, int sums,
                                                                     int columns, float *out0, float *out1,
                                                                     float *out2)
{
    __shared__ float part[kWaves][kWave];
    const int lane = threadIdx.x & (kWave - 1), wave = wave_id(), q = blockIdx.y;
    const int c = blockIdx.x * kWave + lane;
    float s = 0.0f;
    if (c < columns) {
        const size_t row = (size_t)sums * columns;
        const float *p = in + (size_t)q * columns + c;
#pragma unroll 8
        for (int r = wave; r < rows; r += kWaves)
            s += p[r * row];
    }
    part[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && c < columns) {
#pragma unroll
        for (int w = 1; w < kWaves; ++w)
            s += part[w][lane];
        (q == 0 ? out0 : q == 1 ? out1 : out2)[c] = s;
    }
}

} // namespace

hipError_t launch_column_sums(const float *in, int rows, int sums, int columns, float *const *out,
                              hipStream_t s)
{
    hipLaunchKernelGGL(column_sums_kernel, dim3((columns + kWave - 1) / kWave, sums), dim3(kWaves * kWave), 0, s,
                       in, rows, sums, columns, out[0], sums > 1 ? out[1] : nullptr, sums > 2 ? out[2] : nullptr);
    return hipGetLastError();
}

} // namespace moe_lora
