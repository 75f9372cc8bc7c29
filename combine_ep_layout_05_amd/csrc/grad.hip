// grad.hip -- gradient of the combine (gfx950).
//
// out[t] = sum_k w[t,k] * y[row(t,k)], so for every pair with a row
//   grad_y[row(t,k), c] = bf16_rne(w[t,k] * grad_out[t, c])
//   grad_w[t,k]         = sum_c grad_out[t, c] * y[row(t,k), c]      (fp32)
// and grad_w = 0 for a masked pair; rows that no pair names stay as they are.
// (The gradient of the dispatch, a token's receive-row gradients summed with
// weight 1, is the reduce mode of combine.hip with K entries per token.)
//
// One workgroup per pair: its waves take 512-column steps in turn (16 bytes
// per lane and load), each lane sums its products in fp32, and the waves' sums
// are joined through LDS in wave order, so the result does not depend on
// timing.  The pairs of one token are neighbours on one XCD, so grad_out[t]
// comes from HBM once and K - 1 times from that XCD's L2 (in launch order:
// 6.8 -> 8.5 us at 128 x 7168 top-8, 191 -> 198 us at 4096 x 7168).
//
// It moves each byte once and runs at the rate of a copy: graphs of launches on
// MI355X, 16384 x 4096 top-8 with 10 % of entries masked 411 us (5.0 TB/s; a 2
// GiB copy 4.9), 4096 x 7168 191 us (5.2 TB/s), 128 x 7168 6.6 us.
#include "ep_device.h"
#include "ep_launch.h"
#include "ep_numerics.h"

namespace ep {
namespace {

constexpr int kMaxGradBlocks = 1 << 20;

__device__ __forceinline__ float wave_sum_f(float v)
{
#pragma unroll
    for (int m = 1; m < kWave; m <<= 1) v += __shfl_xor(v, m);
    return v;
}

// o = bf16(w * g) and the sum of g * y over 8 columns.
__device__ __forceinline__ float grad_step(uint4 g, uint4 y, float w, uint4& o)
{
    const float gl[8] = {bf16_lo(g.x), bf16_hi(g.x), bf16_lo(g.y), bf16_hi(g.y),
                         bf16_lo(g.z), bf16_hi(g.z), bf16_lo(g.w), bf16_hi(g.w)};
    const float yl[8] = {bf16_lo(y.x), bf16_hi(y.x), bf16_lo(y.y), bf16_hi(y.y),
                         bf16_lo(y.z), bf16_hi(y.z), bf16_lo(y.w), bf16_hi(y.w)};
    o.x = pack2_bf16(w * gl[0], w * gl[1]);
    o.y = pack2_bf16(w * gl[2], w * gl[3]);
    o.z = pack2_bf16(w * gl[4], w * gl[5]);
    o.w = pack2_bf16(w * gl[6], w * gl[7]);
    float d = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) d = __builtin_fmaf(gl[i], yl[i], d);
    return d;
}

// kStream: rows touched once are loaded and stored nontemporally (4096 x 7168:
// 205 us with cached stores, 202 with cached loads).
template <bool kStream, int kWaves>
__global__ __launch_bounds__(kWaves * kWave) void combine_backward_kernel(
    const uint16_t* __restrict__ grad_out, const uint16_t* __restrict__ y,
    const int32_t* __restrict__ row_of_pair, const float* __restrict__ topk_w, int n_pairs, int H,
    int K, uint16_t* __restrict__ grad_y, float* __restrict__ grad_w)
{
    __shared__ float part[kWaves];
    for (int64_t first = 0; first < n_pairs; first += gridDim.x) {
        const int in_grid = (int)min((int64_t)gridDim.x, n_pairs - first);
        if ((int)blockIdx.x >= in_grid) return;
        const int pair = (int)first + xcd_block(blockIdx.x, in_grid);
        const int t = pair / K;
        const int row = row_of_pair[pair];
        const float w = topk_w[pair];
        if (row < 0 || row >= n_pairs) {
            if (threadIdx.x == 0) grad_w[pair] = 0.0f;
            continue;
        }
        const uint16_t* const g = grad_out + (int64_t)t * H;
        const uint16_t* const yr = y + (int64_t)row * H;
        uint16_t* const o = grad_y + (int64_t)row * H;
        float acc = 0.0f;
        for (int64_t c = threadIdx.x * kColsPerLane; c < H; c += kWaves * kStepCols) {
            uint4 ov;
            acc += grad_step(load16<false>(g + c), load16<kStream>(yr + c), w, ov);
            store16<kStream>(o + c, ov);
        }
        acc = wave_sum_f(acc);
        if constexpr (kWaves == 1) {
            if (threadIdx.x == 0) grad_w[pair] = acc;
        } else {
            if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = acc;
            __syncthreads();
            if (threadIdx.x == 0) {
                float s = 0.0f;
#pragma unroll
                for (int i = 0; i < kWaves; ++i) s += part[i];
                grad_w[pair] = s;
            }
            __syncthreads();                              // part is used again
        }
    }
}

}  // namespace

hipError_t launch_combine_backward(const uint16_t* grad_out, const uint16_t* y,
                                   const int32_t* row_of_pair, const float* topk_w, int T, int H,
                                   int K, uint16_t* grad_y, float* grad_w, hipStream_t stream)
{
    const int n = T * K;
    const bool streaming = (int64_t)n * H * 2 >= kStreamMinBytes;
    // Waves per pair.  Few pairs: 8 (2, 4, 8 waves: 4 x 6144 top-8 3.4, 2.8, 2.5
    // us, 128 x 7168 7.2, 6.8, 6.6).  Many narrow ones: 1, as the waves of a
    // pair would mostly wait for each other (1, 2, 4, 8 waves: 5000 x 1032 top-6
    // 31.8, 35.9, 41.0, 65.4).  Otherwise 4; there the rate is the same within 2 %.
    const int waves = n <= 2048 ? 8 : (H <= 3 * kStepCols ? 1 : 4);
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)(n < kMaxGradBlocks ? n : kMaxGradBlocks)),
                           dim3(waves * kWave), 0, stream, grad_out, y, row_of_pair, topk_w, n, H,
                           K, grad_y, grad_w);
    };
    if (waves == 8) streaming ? go(combine_backward_kernel<true, 8>) : go(combine_backward_kernel<false, 8>);
    else if (waves == 4) streaming ? go(combine_backward_kernel<true, 4>) : go(combine_backward_kernel<false, 4>);
    else streaming ? go(combine_backward_kernel<true, 1>) : go(combine_backward_kernel<false, 1>);
    return hipGetLastError();
}

}  // namespace ep
