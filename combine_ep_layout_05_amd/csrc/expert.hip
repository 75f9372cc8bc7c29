// expert.hip -- the experts' products with 4-bit weights on the dispatched
// rows (gfx950).
//
// Row r of expert e (expert_offset[e] <= r < expert_offset[e+1]):
//   acc[r, n] = sum_b d[b] * s[e][n, b] * xs[r, b],
//   d[b]      = sum over the 128 columns c of block b of x[r, c] * e2m1[e][n, c]
// in fp32, blocks in ascending order (xs = 1 for bf16 rows).  One matrix
// instruction per block and 16 x 16 outputs computes d when the rows are fp8:
// it takes e4m3 and e2m1 operands as they are stored, and its 128 columns are
// one scale block, so the scales are applied to its result.  bf16 rows take
// four bf16 instructions per block on codes converted to bf16, which is exact.
//
// Operands: the weights are the A side (16 outputs n), the rows the B side
// (16 rows m), so lane l holds the results of row m = l % 16 for the four
// neighbouring outputs n = 4 * (l / 16) + 0..3 and stores them as 8 bytes.
// Codes: lane l takes the 32 columns q*32 .. +31 of the block, q = l / 16 (16
// bytes).  fp8 rows: the instruction pairs them with columns q*16 .. +15 and
// 64 + q*16 .. +15 in lane l (16 bytes each; read off the instruction with
// one-hot operands).  bf16 rows: the columns of the codes, 8 per instruction
// (16 bytes each).
#include "ep_device.h"
#include "ep_launch.h"
#include "ep_numerics.h"

namespace ep {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

constexpr int kTile = 16;
constexpr int kExpertWaves = 4;

// Row tile `idx` of the batch: its expert, first row and row count, from the
// expert offsets (clamped to the rows there are).  False past the last tile.
// Called by whole waves; the result is wave-uniform.
template <int kRows>
__device__ __forceinline__ bool find_tile(const int32_t* __restrict__ off, int E, int rows, int idx,
                                          int lane, int& expert, int& row0, int& count)
{
    const int per = (E + kWave - 1) / kWave;
    const int e0 = lane * per;
    int tiles = 0;
    for (int j = 0; j < per; ++j) {
        const int e = e0 + j;
        if (e >= E) break;
        const int a = min(max(off[e], 0), rows), b = min(max(off[e + 1], a), rows);
        tiles += (b - a + kRows - 1) / kRows;
    }
    const int incl = wave_inclusive_scan(tiles);
    const uint64_t past = __ballot(incl > idx);
    if (!past) return false;
    const int win = __builtin_ctzll(past);
    int left = idx - read_lane(incl - tiles, win);
    const int first = win * per;
    for (int j = 0; j < per; ++j) {
        const int e = first + j;
        if (e >= E) break;
        const int a = min(max(off[e], 0), rows), b = min(max(off[e + 1], a), rows);
        const int n = (b - a + kRows - 1) / kRows;
        if (left < n) {
            expert = e;
            row0 = a + left * kRows;
            count = min(kRows, b - row0);
            return true;
        }
        left -= n;
    }
    return false;
}

template <int kSel>
__device__ __forceinline__ uint32_t bf16_of_codes(uint32_t codes)
{
    const v2bf v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, 1.0f, kSel);
    return __builtin_bit_cast(uint32_t, v);
}

// 8 codes (one dword, low nibble first) as 8 bf16 values.
__device__ __forceinline__ v8bf bf16x8_of_codes(uint32_t codes)
{
    const v4i v = {(int)bf16_of_codes<0>(codes), (int)bf16_of_codes<1>(codes),
                   (int)bf16_of_codes<2>(codes), (int)bf16_of_codes<3>(codes)};
    return __builtin_bit_cast(v8bf, v);
}

// d of one block for 16 outputs x 16 rows.
__device__ __forceinline__ v4f block_product(v4i w, v8i x)
{
    const v8i a = {w[0], w[1], w[2], w[3], 0, 0, 0, 0};
    const v4f zero = {0.0f, 0.0f, 0.0f, 0.0f};
    // cbsz 4: A is e2m1; blgp 0: B is e4m3; e8m0 scales of 127: factors of 1
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, x, zero, 4, 0, 0, 0x7F7F7F7F, 0,
                                                            0x7F7F7F7F);
}

__device__ __forceinline__ v4f block_product(v4i w, const v4i (&x)[4])
{
    v4f d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf16x8_of_codes((uint32_t)w[i]),
                                                    __builtin_bit_cast(v8bf, x[i]), d, 0, 0, 0);
    return d;
}

__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.0f + expf(-g)) * u; }

// One wave per tile of 16 outputs x 16 rows (with kSilu: 16 gate rows and the
// 16 up rows that belong to them).
template <bool kFp8, bool kSilu>
__global__ __launch_bounds__(kExpertWaves * kWave) void expert_kernel(
    const uint8_t* __restrict__ x, const float* __restrict__ xs, int rows, int cols,
    const int32_t* __restrict__ off, int E, const uint8_t* __restrict__ w,
    const float* __restrict__ ws, int outs, uint16_t* __restrict__ out)
{
    const int lane = threadIdx.x % kWave, m = lane % kTile, q = lane / kTile;
    const int n0 = (blockIdx.x * kExpertWaves + wave_uniform(threadIdx.x / kWave)) * kTile;
    if (n0 >= outs) return;
    int expert, row0, count;
    if (!find_tile<kTile>(off, E, rows, blockIdx.y, lane, expert, row0, count)) return;
    const int blocks = cols / kScaleBlock;
    const int64_t wrows = kSilu ? 2 * (int64_t)outs : outs;
    // lanes past the last row or output read a valid one; what they compute is not stored
    const int64_t row = row0 + min(m, count - 1);
    const uint8_t* const xr = x + row * cols * (kFp8 ? 1 : 2) + q * (kFp8 ? 16 : 64);
    const float* const xsr = kFp8 ? xs + row * blocks : nullptr;
    const int n_load = min(n0 + m, outs - 1);
    const uint8_t* wr[2];
    const float* sr[2];
#pragma unroll
    for (int h = 0; h < (kSilu ? 2 : 1); ++h) {
        const int64_t base = expert * wrows + (int64_t)h * outs;
        wr[h] = w + (base + n_load) * (cols / 2) + q * 16;
        sr[h] = ws + (base + n0) * blocks;
    }
    int ns[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) ns[i] = (min(n0 + q * 4 + i, outs - 1) - n0) * blocks;
    v4f acc[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
    for (int b = 0; b < blocks; ++b) {
        v8i x8;
        v4i x16[4];
        float f = 1.0f;
        if constexpr (kFp8) {
            const v4i lo = *(const v4i*)(xr + b * 128), hi = *(const v4i*)(xr + b * 128 + 64);
            x8 = (v8i){lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            f = xsr[b];
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) x16[i] = *(const v4i*)(xr + b * 256 + i * 16);
        }
#pragma unroll
        for (int h = 0; h < (kSilu ? 2 : 1); ++h) {
            const v4i wc = *(const v4i*)(wr[h] + b * 64);
            v4f d;
            if constexpr (kFp8) d = block_product(wc, x8);
            else d = block_product(wc, x16);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[h][i] = __builtin_fmaf(d[i], sr[h][ns[i] + b] * f, acc[h][i]);
        }
    }
    const int n = n0 + q * 4;
    if (m < count && n < outs) {
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = kSilu ? silu_mul(acc[0][i], acc[1][i]) : acc[0][i];
        const uint2 o = make_uint2(pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3]));
        store8<false>(out + row * outs + n, o);
    }
}

}  // namespace

bool expert_launch_ok(int rows, int outs, int E)
{
    const int64_t tiles = (int64_t)rows / kTile + (rows < E ? rows : E);
    return tiles < 65536 && (int64_t)outs + kTile * kExpertWaves < ((int64_t)1 << 31);
}

hipError_t launch_expert(const void* x, const float* x_scales, bool fp8, int rows, int cols,
                         const int32_t* expert_offset, int E, const uint8_t* w,
                         const float* w_scales, int outs, bool silu, uint16_t* out,
                         hipStream_t stream)
{
    // at most one partly filled tile per expert that has rows
    const int tiles = rows / kTile + (rows < E ? rows : E);
    const dim3 grid((unsigned)((outs + kTile * kExpertWaves - 1) / (kTile * kExpertWaves)), (unsigned)tiles);
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(kExpertWaves * kWave), 0, stream, (const uint8_t*)x,
                           x_scales, rows, cols, expert_offset, E, w, w_scales, outs, out);
    };
    if (fp8) silu ? go(expert_kernel<true, true>) : go(expert_kernel<true, false>);
    else silu ? go(expert_kernel<false, true>) : go(expert_kernel<false, false>);
    return hipGetLastError();
}

}  // namespace ep
