// expert.hip -- the experts' products with 4-bit weights on the dispatched
// rows (gfx950).
//
// Row r of expert e (expert_offset[e] <= r < expert_offset[e+1]):
//   acc[r, n] = sum_b d[b] * s[e][n, b] * xs[r, b],
//   d[b]      = sum over the 128 columns c of block b of x[r, c] * e2m1[e][n, c]
// in fp32 (xs = 1 for bf16 rows).  Two matrix instructions per block and 16 x 16
// outputs compute d when the rows are fp8: they take e4m3 and e2m1 operands as
// they are stored, and their 128 columns are one scale block, so the scales are
// applied to the result.  bf16 rows take four bf16 instructions per block on
// codes converted to bf16, which is exact.
//
// Rounding: the fp8 instruction adds the 16 products of a lane's 16 bytes in
// fixed point, in steps of 2^-14 of the power of two below the largest one, and
// drops what lies below (read off the instruction; everything after that it
// adds in fp32, and the bf16 one keeps fp32 throughout).  Next to a row's 448,
// products below 1/8 would be lost, and sums in which large products cancel
// would be wrong by many times their value.  So the values below 2 and those
// from 2 on go through it apart.  e2m1 values are multiples of 2^-1 up to 6, and
// e4m3 values below 2 multiples of 2^-9: their products are multiples of 2^-10
// below 2^3.5, at most 2^13 steps; values from 2 on are multiples of 2^-2 up to
// 448, the products multiples of 2^-3 below 2^11.4, at most 2^14.4 steps of
// which the lowest is 2^-14 of 2^11.  Both sums of 16 are exact, and all the
// others are fp32.  One instruction on the whole values takes 1.59 ms where the
// two take 2.17 (4096 tokens x 7168, gate and up, see below); where the weights'
// bytes are the bound they cost nothing.  Sums across blocks, scales and SiLU
// are fp32; the result is rounded to bf16 once.
//
// Two kernels share the batches: expert_stream_kernel for few rows per expert,
// expert_tile_kernel for more (expert_large).  Both are bound by the bytes of
// the weights up to about 30 rows per expert: 128 tokens, 288 experts, top-8 on
// MI355X 695 us for gate and up (7168 columns, 2 x 2048 rows; 6.3 TB/s) and 365
// us for down (2048 columns, 7168 rows; 6.0 TB/s); one token, 8 experts, 6144
// columns, 2 x 2048 rows 21.5 us (5.0 TB/s).  At 128 rows per expert (4096 tokens,
// Zipf routing) gate and up take 2.17 ms with fp8 rows (0.89 PFLOP/s) and 2.23
// ms with bf16 (0.86 PFLOP/s; on another card 2.22 and 2.30): twice 32 and four times 16 cycles of the matrix
// unit per 16 x 16 outputs and block (1.5 ms in all at the rate a library product
// reaches), beside 8 vector instructions that scale and add the result and, fp8,
// 8 that part the rows.
//
// Operands: the weights are the A side (16 outputs n), the rows the B side
// (16 rows m), so lane l holds the results of row m = l % 16 for the four
// neighbouring outputs n = 4 * (l / 16) + 0..3 and stores them as 8 bytes.
// Codes: lane l takes the 32 columns q*32 .. +31 of the block, q = l / 16 (16
// bytes).  fp8 rows: the instruction pairs them with columns q*16 .. +15 and
// 64 + q*16 .. +15 in lane l (16 bytes each; read off the instruction with
// one-hot operands).  bf16 rows: the columns of the codes, 8 per instruction
// (16 bytes each).
#include <algorithm>

#include "ep_device.h"
#include "ep_launch.h"
#include "ep_numerics.h"
#include "expert_plan.h"

namespace ep {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

static_assert(kStreamWaves * kWave == kExpertThreads && kTileWaves * kWave == kExpertThreads, "one workgroup size");
static_assert(kExpertXcds == kXcds, "the plan has no device header");
constexpr int kMaxExpertCols = 1 << 23;      // 64 rows of bf16 within 31-bit offsets
constexpr int64_t kMaxBuffer = 0x7FFFFFFF;

// Row tile `idx` of the batch: its expert, first row and row count, from the
// expert offsets (clamped to the rows there are).  False past the last tile.
// Called by whole waves; the result is wave-uniform.  Lane i counts the tiles
// of E / 64 neighbouring experts (all offsets loaded before the first is used:
// one round trip); a DPP scan gives the tiles before it.
template <int kRows>
__device__ __forceinline__ bool find_tile(const int32_t* __restrict__ off, int E, int rows, int idx,
                                          int lane, int& expert, int& row0, int& count)
{
    constexpr int kMaxPer = kMaxExperts / kWave;
    const int per = (E + kWave - 1) / kWave;
    const int e0 = lane * per;
    int o[kMaxPer + 1];
#pragma unroll
    for (int j = 0; j <= kMaxPer; ++j)
        if (j <= per) o[j] = off[min(e0 + j, E)];
    int tiles = 0;
#pragma unroll
    for (int j = 0; j <= kMaxPer; ++j) {
        if (j > per) break;
        o[j] = min(max(o[j], j > 0 ? o[j - 1] : 0), rows);
        if (j > 0) tiles += (o[j] - o[j - 1] + kRows - 1) / kRows;
    }
    const int incl = wave_inclusive_scan(tiles);
    const uint64_t past = __ballot(incl > idx);
    if (!past) return false;
    const int win = __builtin_ctzll(past);
    int left = idx - (incl - tiles), at = 0, first = 0, end = 0;      // lane `win`'s are the answer
#pragma unroll
    for (int j = 0; j < kMaxPer; ++j) {
        if (j >= per) break;
        const int n = (o[j + 1] - o[j] + kRows - 1) / kRows;
        if (left >= 0 && left < n) { at = j; first = o[j] + left * kRows; end = o[j + 1]; }
        left -= n;
    }
    expert = win * per + read_lane(at, win);
    row0 = read_lane(first, win);
    count = min(kRows, read_lane(end, win) - row0);
    return true;
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

// Four e4m3 values of a row in two parts whose sum they are: those below 2
// (returned in x) and those from 2 on, NaN among them, which are the bytes with
// bit 6 set; the other part's byte is 0.  One selector (byte i of x where it is
// from 2 on, else of 0) serves both.
__device__ __forceinline__ uint32_t take_high(uint32_t& x)
{
    const uint32_t sel = ((x >> 4) & 0x04040404u) | 0x03020100u;
    const uint32_t high = __builtin_amdgcn_perm(x, 0u, sel);
    x = __builtin_amdgcn_perm(0u, x, sel);
    return high;
}

__device__ __forceinline__ v8i take_high(v8i& x)
{
    v8i high;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t v = (uint32_t)x[i];
        high[i] = (int)take_high(v);
        x[i] = (int)v;
    }
    return high;
}

// c + the products of one block for 16 outputs x 16 rows, of one part of the rows.
__device__ __forceinline__ v4f part_product(v4i w, v8i x, v4f c)
{
    const v8i a = {w[0], w[1], w[2], w[3], 0, 0, 0, 0};
    // cbsz 4: A is e2m1; blgp 0: B is e4m3; no block scales (the unscaled form)
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, x, c, 4, 0, 0, 0, 0, 0);
}

// d of one block for 16 outputs x 16 rows, bf16.
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

// Bounded loads: a uniform base and size, a 32-bit offset per lane and a
// uniform one; what lies past the size reads as 0.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* base, int64_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0,
                                             (int)(bytes < kMaxBuffer ? bytes : kMaxBuffer), 0x00020000);
}

template <bool kOnce = false>              // kOnce: nontemporal
__device__ __forceinline__ v4i load_b128(__amdgpu_buffer_rsrc_t r, int lane_offset, int offset)
{
    return __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(r, lane_offset, offset, kOnce ? 2 : 0));
}

// Few rows per expert: the weights are read once and bound the time, so the
// work is split for loads in flight.  A team of kSplit waves takes kRows rows of
// one expert and 64 weight rows (silu: 32 + 32), each wave with its own run of
// blocks; their sums are joined through LDS in wave order (kSplit 1: nothing to
// join, and no barrier).  A wave takes two blocks at a time, whose codes are
// whole cache lines (one at a time: 4.6 instead of 5.2 TB/s), and has the next
// two in flight.  The scales of its next 16 blocks are copied to its own part
// of LDS, transposed.  Nontemporal code loads drop a line between its two
// halves here (5.5 -> 4.7 TB/s), and a team that goes on to further weight rows
// gains nothing on more, shorter workgroups (4.9 -> 5.6 TB/s).
constexpr int kGroupTiles = kGroupRows / kTile;
constexpr int kWindow = 16;                       // blocks whose scales are in LDS
constexpr int kScalePitch = kGroupRows + kTile + 4;   // weight rows, then fp8 rows

//
// kRows 8, fp8 rows: the two parts of a row are two of the 16 rows of one matrix
// instruction (lanes m and m + 8), whose sums are joined at the end.  kRows 16:
// two instructions.
template <bool kFp8, bool kSilu, int kSplit, int kRows>
__global__ __launch_bounds__(kExpertThreads, kRows < kTile ? 4 : 3) void expert_stream_kernel(
    const uint8_t* __restrict__ x, const float* __restrict__ xs, int rows, int cols,
    const int32_t* __restrict__ off, int E, const uint8_t* __restrict__ w,
    const float* __restrict__ ws, int outs, uint16_t* __restrict__ out, int n_groups,
    int n_parts)
{
    constexpr int kTeams = kStreamWaves / kSplit;                   // groups at a time
    constexpr int kOuts = kSilu ? kGroupRows / 2 : kGroupRows;      // outputs per group
    constexpr int kHalf = kOuts / kTile;                            // operand tiles of results
    constexpr bool kPaired = kRows < kTile;
    static_assert(kRows == kTile || (kFp8 && kRows == kTile / 2), "a row, or the two parts of an fp8 row, per lane");
    __shared__ __attribute__((aligned(16))) float s_scale[kStreamWaves][kWindow * kScalePitch];
    __shared__ v4f s_part[kSplit > 1 ? kStreamWaves : 1][kGroupTiles][kWave];
    const int lane = threadIdx.x % kWave, m = lane % kTile, q = lane / kTile;
    const int wave = wave_uniform(threadIdx.x / kWave), team = wave / kSplit, part = wave % kSplit;
    int expert, row0, count;
    if (!find_tile<kRows>(off, E, rows, blockIdx.x / n_parts, lane, expert, row0, count)) return;
    const int blocks = cols / kScaleBlock;
    const int run = ((blocks + 1) / 2 + kSplit - 1) / kSplit * 2;   // blocks per wave, in pairs
    const int b0 = min(part * run, blocks), b1 = min(b0 + run, blocks);
    const int64_t wrow0 = expert * (kSilu ? 2 * (int64_t)outs : (int64_t)outs);
    const int64_t wrow_end = wrow0 + (kSilu ? 2 * (int64_t)outs : (int64_t)outs);
    constexpr int kParts = kSilu ? 2 : 1;                           // gate and up rows
    const int half_cols = cols / 2;
    // lanes past the last row read a valid one; what they compute is not stored
    constexpr int kRowBytes = kFp8 ? 1 : 2;
    const __amdgpu_buffer_rsrc_t xr = buffer(x + (int64_t)row0 * cols * kRowBytes, (int64_t)count * cols * kRowBytes);
    const __amdgpu_buffer_rsrc_t xsr = buffer(kFp8 ? xs + (int64_t)row0 * blocks : nullptr, kFp8 ? (int64_t)count * blocks * 4 : 0);
    const int xo = min(m % kRows, count - 1) * cols * kRowBytes + q * (kFp8 ? 16 : 64);
    const int wo = m * half_cols + q * 16;

    // first weight row of part h of group g
    auto weight_row = [&](int g, int h) { return wrow0 + (int64_t)h * outs + (int64_t)g * kOuts; };
    // the codes of two neighbouring blocks: 128 bytes of every row
    struct Codes { v4i w[2][kGroupTiles]; };
    auto load = [&](Codes& s, int g, int b) {
#pragma unroll
        for (int h = 0; h < kParts; ++h) {
            const int64_t r = weight_row(g, h);
            const __amdgpu_buffer_rsrc_t wr = buffer(w + r * half_cols, (wrow_end - r) * half_cols);
#pragma unroll
            for (int j = 0; j < kHalf; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    s.w[i][h * kHalf + j] = load_b128(wr, wo, j * kTile * half_cols + min(b + i, blocks - 1) * 64);
        }
    };
    constexpr int kXRegs = kFp8 ? 2 : 4;
    auto load_x = [&](v4i (&v)[kXRegs], int b) {
#pragma unroll
        for (int i = 0; i < kXRegs; ++i)
            v[i] = load_b128(xr, xo, b * (kFp8 ? 128 : 256) + i * (kFp8 ? 64 : 16));
    };
    float* const sc = s_scale[wave];
    // Scales of blocks b .. b + 15: 16 rows per load, 4 blocks per lane.  No use
    // is made of a load that is partly past its buffer: a lane's 4 blocks end
    // at the row's last one at most (rows of fewer than 4 blocks: one per lane).
    auto stage_scales = [&](int g, int b) {
        const bool wide = blocks >= 4;
        const int bl = wide ? min(b + (lane % 4) * 4, blocks - 4) : min(b + lane % 4, blocks - 1);
        const int so = ((lane / 4) * blocks + bl) * 4;
        v4f v[kGroupTiles + 1];
        auto get = [&](__amdgpu_buffer_rsrc_t r, int offset) {
            if (wide) return __builtin_bit_cast(v4f, load_b128(r, so, offset));
            const v4i one = {(int)__builtin_amdgcn_raw_buffer_load_b32(r, so, offset, 0), 0, 0, 0};
            return __builtin_bit_cast(v4f, one);
        };
#pragma unroll
        for (int h = 0; h < kParts; ++h) {
            const int64_t r = weight_row(g, h);
            const __amdgpu_buffer_rsrc_t sr = buffer(ws + r * blocks, (wrow_end - r) * blocks * 4);
#pragma unroll
            for (int j = 0; j < kHalf; ++j) v[h * kHalf + j] = get(sr, j * kTile * blocks * 4);
        }
        if constexpr (kFp8) v[kGroupTiles] = get(xsr, 0);
        wave_lds_sync();
        const int at = bl - b;                             // negative: blocks before the window
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (at + i < 0 || (i > 0 && !wide)) continue;
#pragma unroll
            for (int j = 0; j < kGroupTiles + (kFp8 ? 1 : 0); ++j)
                sc[(at + i) * kScalePitch + j * kTile + lane / 4] = v[j][i];
        }
        wave_lds_sync();
    };

    const int g = (blockIdx.x % n_parts) * kTeams + team;
    v4f acc[kGroupTiles];
#pragma unroll
    for (int j = 0; j < kGroupTiles; ++j) acc[j] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
    if (g < n_groups && b0 < b1) {
        Codes cur, next;
        load(cur, g, b0);
        for (int b = b0; b < b1; b += 2) {
            const int at = (b - b0) % kWindow;
            if (at == 0) stage_scales(g, b);
            v4i xv[2][kXRegs];
            load_x(xv[0], b);
            load_x(xv[1], min(b + 1, blocks - 1));
            if (b + 2 < b1) load(next, g, b + 2);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if (b + u >= b1) break;
                const float* const sb = sc + (at + u) * kScalePitch;
                const float f = kFp8 ? sb[kGroupRows + m % kRows] : 1.0f;
                v8i high{}, low{};
                if constexpr (kFp8) {
                    low = (v8i){xv[u][0][0], xv[u][0][1], xv[u][0][2], xv[u][0][3],
                                xv[u][1][0], xv[u][1][1], xv[u][1][2], xv[u][1][3]};
                    high = take_high(low);
                    if (kPaired && m >= kRows) high = low;
                }
#pragma unroll
                for (int j = 0; j < kGroupTiles; ++j) {
                    const v4f sw = *(const v4f*)(sb + j * kTile + q * 4);
                    v4f d;
                    if constexpr (kFp8) {
                        d = part_product(cur.w[u][j], high, (v4f){0.0f, 0.0f, 0.0f, 0.0f});
                        if (!kPaired) d = part_product(cur.w[u][j], low, d);
                    } else {
                        d = block_product(cur.w[u][j], xv[u]);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[j][i] = __builtin_fmaf(d[i], sw[i] * f, acc[j][i]);
                }
            }
            cur = next;
        }
    }
    if constexpr (kPaired) {                          // the low parts' sums are 8 lanes on
#pragma unroll
        for (int j = 0; j < kGroupTiles; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float mine = acc[j][i];
                acc[j][i] = mine + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
                    0, __builtin_bit_cast(int, mine), 0x128, 0xF, 0xF, false));        // row_ror 8
            }
    }
    // operand tile j of lane ln: row ln % 16, outputs (ln / 16) * 4 .. + 3 of the tile
    auto store = [&](int j, int ln, v4f v, v4f u) {
        const int r = ln % kTile, n = g * kOuts + j * kTile + (ln / kTile) * 4;
        if (r >= count || n >= outs) return;
        if constexpr (kSilu)
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = silu_mul(v[i], u[i]);
        store8<false>(out + (int64_t)(row0 + r) * outs + n,
                      make_uint2(pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3])));
    };
    if constexpr (kSplit == 1) {
        if (g < n_groups)
#pragma unroll
            for (int j = 0; j < kHalf; ++j) store(j, lane, acc[j], kSilu ? acc[j + kHalf] : acc[j]);
    } else {
#pragma unroll
        for (int j = 0; j < kGroupTiles; ++j) s_part[wave][j][lane] = acc[j];
        lds_barrier();
        // the team's waves take its result tiles in turn
        for (int j = part; j < kHalf; j += kSplit) {
            v4f v = {0.0f, 0.0f, 0.0f, 0.0f}, u = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 2
            for (int i = 0; i < kSplit; ++i) {
                v += s_part[team * kSplit + i][j][lane];
                if constexpr (kSilu) u += s_part[team * kSplit + i][j + kHalf][lane];
            }
            if (g < n_groups) store(j, lane, v, u);
        }
    }
}

// Large batches: a workgroup of 4 waves computes up to 64 rows x 256 weight
// rows, 64 of them per wave.  Two blocks are a stage; the next stage is loaded
// while one is computed.  The rows go straight to LDS for all four waves.  The
// codes go through the registers of the wave that needs them to its own part
// of LDS: a load covers 128 bytes, a cache line, of each of 8 rows, where the
// operand has 64 bytes of 16 (loaded like that every line is asked for twice,
// and the address unit, 16 rows an instruction, bounds the kernel).  Scales are
// loaded for 4 blocks at a time (16 bytes of one row per lane) and kept in LDS
// transposed.
//
// The 16-byte pieces of a row in LDS are permuted (piece ^ row) so that 8
// lanes reading one piece of 8 neighbouring rows meet 8 different banks.
//
// Also measured, 4096 tokens x 7168, gate and up, fp8, with one matrix instruction
// per block (whole rows, 1.54 ms): 128-row tiles in one
// workgroup of 8 waves a CU 1.69 ms (nothing overlaps its prologue, and the
// waves wait together); codes straight to registers in operand order 1.84 ms;
// codes two stages ahead 1.67 ms; whole tiles of all experts before the rests
// 1.80 ms (long and memory-bound tiles then no longer overlap).
constexpr int kRowTiles = kTileRows / kTile;
constexpr int kColTiles = kWaveCols / kTile;
constexpr int kStageBlocks = 2;
constexpr int kCodeLoads = kWaveCols * kStageBlocks * 64 / 1024;                       // per wave
constexpr int kScaleBlocks = 4;                  // blocks per load of scales

template <bool kFp8> struct TileShared {
    // rows: fp8 a stage of 2 blocks (256 bytes of a row), bf16 of one (also 256)
    static constexpr int kRowBytes = 256;
    static constexpr int kXBlocks = kFp8 ? 2 : 1;
    static constexpr int kXLoads = kTileRows * kRowBytes / 1024 / kTileWaves;          // per wave
    uint8_t x[2][kTileRows * kRowBytes];
    uint8_t w[kTileWaves][kWaveCols * kStageBlocks * 64];
    float ws[kTileWaves][kScaleBlocks][kWaveCols];
    float xs[kFp8 ? 2 : 1][kScaleBlocks][kFp8 ? kTileRows : 4];
};

// 16 bytes per lane straight to LDS, lane after lane.  All of a kernel's LDS is
// one object: between separate ones the compiler tracks which of these loads
// might touch what is read, and waits for all in flight before every read.
__device__ __forceinline__ void load_lds16(__amdgpu_buffer_rsrc_t r, void* lds, int lane_offset, int offset)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16,
                                             lane_offset, offset, 0, 0);
}

// Waits until at most kOutstanding of this wave's loads are in flight (they
// complete in order) and its LDS accesses are done, and meets the workgroup:
// then every wave's older loads are in LDS and what was read before may be
// overwritten.  (The empty asm statements keep the compiler from moving
// accesses across; a fence would wait for every load in flight into LDS.)
template <int kOutstanding>
__device__ __forceinline__ void stage_barrier()
{
    static_assert(kOutstanding >= 0 && kOutstanding < 16, "one field of the encoding is used");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(kOutstanding | 0x70);   // gfx9 encoding: vmcnt, lgkmcnt 0, expcnt not waited for
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

template <bool kFp8, bool kSilu>
__global__ __launch_bounds__(kExpertThreads, 2) void expert_tile_kernel(
    const uint8_t* __restrict__ x, const float* __restrict__ xs, int rows, int cols,
    const int32_t* __restrict__ off, int E, const uint8_t* __restrict__ w,
    const float* __restrict__ ws, int outs, uint16_t* __restrict__ out, int n_groups)
{
    using S = TileShared<kFp8>;
    __shared__ __attribute__((aligned(16))) S lds;   // one object: see load_lds16
    const int lane = threadIdx.x % kWave, m = lane % kTile, q = lane / kTile;
    const int wave = wave_uniform(threadIdx.x / kWave);
    // 4 row tiles at a time on one XCD, column group by column group: tiles of
    // one expert share its codes in that XCD's L2, column groups the rows
    const int slot = blockIdx.x / kXcds, chunk = slot / (kChunkTiles * n_groups);
    const int in_chunk = slot % (kChunkTiles * n_groups), group = in_chunk / kChunkTiles;
    const int tile = (chunk * kXcds + blockIdx.x % kXcds) * kChunkTiles + in_chunk % kChunkTiles;
    constexpr int kParts = kSilu ? 2 : 1;                      // gate and up rows
    constexpr int kOuts = kWaveCols / kParts;                  // outputs per wave
    constexpr int kHalf = kOuts / kTile;                       // operand tiles of a part
    const int n0 = (group * kTileWaves + wave) * kOuts;
    int expert, row0, count;
    if (!find_tile<kTileRows>(off, E, rows, tile, lane, expert, row0, count)) return;
    const int blocks = cols / kScaleBlock, half_cols = cols / 2;
    const int64_t wrows = (int64_t)outs * kParts;
    // the expert's only tile: nobody else wants its codes in the L2, and loaded
    // nontemporally they come faster (512 tokens, 256 experts 434 -> 383 us; where
    // tiles share them slower, 1.64 -> 1.81 ms at 4096 tokens; both with one matrix
    // instruction per block)
    const bool alone = off[expert + 1] - off[expert] <= kTileRows;

    // (past the last output: other rows or 0, not stored)
    const int64_t n_base = min(n0, outs);
    __amdgpu_buffer_rsrc_t wr[kParts];
#pragma unroll
    for (int h = 0; h < kParts; ++h) {
        const int64_t r = n_base + (int64_t)h * outs;
        wr[h] = buffer(w + (expert * wrows + r) * half_cols, (wrows - r) * half_cols);
    }
    const __amdgpu_buffer_rsrc_t sr = buffer(ws + (expert * wrows + n_base) * blocks,
                                             (wrows - n_base) * blocks * 4);
    const int wo = (lane / 8) * half_cols + (lane % 8) * 16;
    // rows past the last are past the buffer: not fetched (read as another row
    // they would ask for lines already on their way); what they give is not stored
    constexpr int kElem = kFp8 ? 1 : 2;
    const __amdgpu_buffer_rsrc_t xr = buffer(x + (int64_t)row0 * cols * kElem, (int64_t)count * cols * kElem);
    const __amdgpu_buffer_rsrc_t xsr = buffer(kFp8 ? xs + (int64_t)row0 * blocks : nullptr,
                                              kFp8 ? (int64_t)count * blocks * 4 : 0);
    // load p of a wave is load p * 4 + wave of the stage: few rows are shared
    // out; lane i piece i % 16 of row i / 16 of the load
    int xo[S::kXLoads];
#pragma unroll
    for (int p = 0; p < S::kXLoads; ++p) {
        const int r = (p * kTileWaves + wave) * 4 + q;
        xo[p] = r * cols * kElem + ((m ^ (r % kTile)) * 16);
    }
    // (past the last block: the next row or 0, not used)
    auto load_x = [&](int buf, int b) {
#pragma unroll
        for (int p = 0; p < S::kXLoads; ++p)
            if ((p * kTileWaves + wave) * 4 < count)
                load_lds16(xr, lds.x[buf] + (p * kTileWaves + wave) * 1024, xo[p], b * kScaleBlock * kElem);
    };
    // codes of blocks b and b + 1: lane i piece i % 8 of row i / 8 of the load
    v4i cv[kCodeLoads];
    auto load_codes = [&](int b) {
        constexpr int kPer = kCodeLoads / kParts;
        if (alone) {
#pragma unroll
            for (int p = 0; p < kCodeLoads; ++p)
                cv[p] = load_b128<true>(wr[p / kPer], wo, (p % kPer) * 8 * half_cols + b * 64);
        } else {
#pragma unroll
            for (int p = 0; p < kCodeLoads; ++p)
                cv[p] = load_b128(wr[p / kPer], wo, (p % kPer) * 8 * half_cols + b * 64);
        }
    };
    auto store_codes = [&]() {
#pragma unroll
        for (int p = 0; p < kCodeLoads; ++p)
            *(v4i*)(lds.w[wave] + p * 1024 + (lane / 8) * 128 + ((lane % 8) ^ (lane / 8)) * 16) = cv[p];
    };
    // Scales of blocks b .. b + 3: lane i that of weight row i of the wave (silu:
    // lanes 32 .. 63 the up rows), lanes 0 .. 15 those of 16 of the fp8 rows.  The
    // 4 blocks end at the row's last one at most: no load is partly past its
    // buffer.
    const int so = (kSilu ? lane % kOuts + lane / kOuts * outs : lane) * blocks * 4;
    const int xso = min(wave * kTile + m, count - 1) * blocks * 4;
    struct Scales { float w[kScaleBlocks], x[kScaleBlocks]; };
    auto load_scales = [&](int b) {
        Scales v;
        if (blocks >= kScaleBlocks) {
            const int bl = min(b, blocks - kScaleBlocks);
            const v4f a = __builtin_bit_cast(v4f, load_b128(sr, so, bl * 4));
            const v4f c = kFp8 ? __builtin_bit_cast(v4f, load_b128(xsr, xso, bl * 4)) : a;
            v.w[0] = a[0]; v.w[1] = a[1]; v.w[2] = a[2]; v.w[3] = a[3];
            v.x[0] = c[0]; v.x[1] = c[1]; v.x[2] = c[2]; v.x[3] = c[3];
        } else {
#pragma unroll
            for (int i = 0; i < kScaleBlocks; ++i) {
                const int o = min(i, blocks - 1) * 4;
                v.w[i] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(sr, so, o, 0));
                v.x[i] = kFp8 ? __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(xsr, xso, o, 0)) : 0.0f;
            }
        }
        return v;
    };
    auto store_scales = [&](const Scales& v, int b, int buf) {
        const int skip = blocks >= kScaleBlocks ? b - min(b, blocks - kScaleBlocks) : 0;
#pragma unroll
        for (int i = 0; i < kScaleBlocks; ++i) {
            if (i < skip) continue;
            lds.ws[wave][i - skip][lane] = v.w[i];
            if constexpr (kFp8) if (lane < kTile) lds.xs[buf][i - skip][wave * kTile + lane] = v.x[i];
        }
    };

    // fp8 rows: the kBlocks blocks of a stage, block i of the scales the first,
    // kLive groups of 16 rows.  One sequence of (block, group) steps: the products
    // of a step's low values start while those of the step before are scaled and
    // added, those of its high values while the next step's rows are parted (in
    // another order, or left to the compiler, 1-2 % slower), and the operands of
    // the second block are read while the first is computed (every wave reads at
    // the start of a stage and none in between otherwise).
    auto compute_fp8 = [&](auto kLive, auto kBlocks, auto& acc, const uint8_t* sx, int buf, int i) {
        constexpr int kN = decltype(kLive)::value, kU = decltype(kBlocks)::value;
        constexpr int kSlots = kN <= 2 ? 2 * kN : kN;        // few groups: both blocks' rows at once
        v4i wc[kU][kColTiles];
        v4f sw[kColTiles], d[kColTiles];         // of the block whose products are added
        float f[kN];
        v8i xv[kSlots];
        auto get_w = [&](int u) {
#pragma unroll
            for (int j = 0; j < kColTiles; ++j)
                wc[u][j] = *(const v4i*)(lds.w[wave] + (j * kTile + m) * 128 + ((u * 4 + q) ^ (m % 8)) * 16);
        };
        auto get_scales = [&](int u) {
#pragma unroll
            for (int t = 0; t < kN; ++t) f[t] = lds.xs[buf][i + u][t * kTile + m];
#pragma unroll
            for (int j = 0; j < kColTiles; ++j) sw[j] = *(const v4f*)&lds.ws[wave][i + u][j * kTile + q * 4];
        };
        auto get_x = [&](int u, int t) {
            const uint8_t* const row = sx + (t * kTile + m) * S::kRowBytes;
            const v4i lo = *(const v4i*)(row + ((u * 8 + q) ^ m) * 16);
            const v4i hi = *(const v4i*)(row + ((u * 8 + 4 + q) ^ m) * 16);
            xv[(u * kN + t) % kSlots] = (v8i){lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        };
        auto add = [&](int t, int j) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                acc[t][j][k] = __builtin_fmaf(d[j][k], sw[j][k] * f[t], acc[t][j][k]);
        };
        get_w(0);
#pragma unroll
        for (int t = 0; t < kN; ++t) get_x(0, t);
        get_scales(0);
        v8i high = take_high(xv[0]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int step = 0; step < kU * kN; ++step) {
            const int u = step / kN, t = step % kN;
            v8i& low = xv[step % kSlots];
            v8i& next = xv[(step + 1) % kSlots];
#pragma unroll
            for (int j = 0; j < kColTiles; ++j) {
                if (step > 0) add((step - 1) % kN, j);
                d[j] = part_product(wc[u][j], low, (v4f){0.0f, 0.0f, 0.0f, 0.0f});
                __builtin_amdgcn_sched_barrier(0);
            }
            v8i next_high{};
#pragma unroll
            for (int j = 0; j < kColTiles; ++j) {
                if (kN > 1 && step + 1 < kU * kN)
#pragma unroll
                    for (int i = 2 * j; i < 2 * j + 2; ++i) {
                        uint32_t v = (uint32_t)next[i];
                        next_high[i] = (int)take_high(v);
                        next[i] = (int)v;
                    }
                d[j] = part_product(wc[u][j], high, d[j]);
                __builtin_amdgcn_sched_barrier(0);
            }
            if (u + 1 < kU) {                                // the next block's operands
                if (t == 0) get_w(u + 1);
                if (kSlots == kN) get_x(u + 1, t);
                else if (t == 0)
#pragma unroll
                    for (int r = 0; r < kN; ++r) get_x(u + 1, r);
            }
            if (u > 0 && t == 0) get_scales(u);              // (the block before is added by now)
            if (kN == 1 && step + 1 < kU) next_high = take_high(next);
            high = next_high;
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int j = 0; j < kColTiles; ++j) add(kN - 1, j);
    };
    // bf16 rows: block u of a stage, block i of the scales, kLive groups of 16 rows.
    auto compute_bf16 = [&](auto kLive, auto& acc, const uint8_t* sx, int u, int buf, int i) {
        constexpr int kN = decltype(kLive)::value;
        auto x_at = [&](int t, int piece) {
            return *(const v4i*)(sx + (t * kTile + m) * S::kRowBytes + (piece ^ m) * 16);
        };
        v4i wc[kColTiles];
#pragma unroll
        for (int j = 0; j < kColTiles; ++j)
            wc[j] = *(const v4i*)(lds.w[wave] + (j * kTile + m) * 128 + ((u * 4 + q) ^ (m % 8)) * 16);
        v8bf xv[kN][4];
#pragma unroll
        for (int t = 0; t < kN; ++t)
#pragma unroll
            for (int k = 0; k < 4; ++k) xv[t][k] = __builtin_bit_cast(v8bf, x_at(t, q * 4 + k));
#pragma unroll
        for (int j = 0; j < kColTiles; ++j) {
            const v4f sw = *(const v4f*)&lds.ws[wave][i][j * kTile + q * 4];
            v8bf wb[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) wb[k] = bf16x8_of_codes((uint32_t)wc[j][k]);
            v4f d[kN];
#pragma unroll
            for (int t = 0; t < kN; ++t) d[t] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int t = 0; t < kN; ++t)
                    d[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[k], xv[t][k], d[t], 0, 0, 0);
#pragma unroll
            for (int t = 0; t < kN; ++t)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    acc[t][j][k] = __builtin_fmaf(d[t][k], sw[k], acc[t][j][k]);
        }
    };
    // The whole product of kLive groups of 16 rows: a variant each, so that the
    // sums stay in their registers.
    auto run = [&](auto kLive) {
        constexpr int kN = decltype(kLive)::value;
        v4f acc[kN][kColTiles];
#pragma unroll
        for (int t = 0; t < kN; ++t)
#pragma unroll
            for (int j = 0; j < kColTiles; ++j) acc[t][j] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
        Scales scales = load_scales(0);
        load_x(0, 0);
        load_codes(0);
        for (int b0 = 0; b0 < blocks; b0 += kScaleBlocks) {
            const int buf = kFp8 ? (b0 / kScaleBlocks) % 2 : 0;
            store_scales(scales, b0, buf);
#pragma unroll
            for (int i = 0; i < kScaleBlocks; i += kStageBlocks) {
                const int b = b0 + i;
                if (b + (kFp8 ? 1 : 0) >= blocks) break;     // (fp8: a last single block follows the loop)
                const bool more = b + kStageBlocks < blocks;
                store_codes();
                stage_barrier<0>();
                if (i == 0 && b0 + kScaleBlocks < blocks) scales = load_scales(b0 + kScaleBlocks);
                if constexpr (kFp8) {
                    const int cur = i / kStageBlocks;
                    if (more) { load_x(1 - cur, b + kStageBlocks); load_codes(b + kStageBlocks); }
                    compute_fp8(kLive, std::integral_constant<int, 2>(), acc, lds.x[cur], buf, i);
                } else {
                    if (b + 1 < blocks) load_x(1, b + 1);
                    asm volatile("" ::: "memory");       // in this order: the barrier below counts
                    __builtin_amdgcn_sched_barrier(0);
                    if (more) load_codes(b + kStageBlocks);
                    __builtin_amdgcn_sched_barrier(0);
                    compute_bf16(kLive, acc, lds.x[0], 0, buf, i);
                    if (b + 1 < blocks) {
                        // the rows of block b + 1; the codes after them may still be in flight
                        if (more) stage_barrier<kCodeLoads>(); else stage_barrier<0>();
                        if (more) load_x(0, b + kStageBlocks);
                        compute_bf16(kLive, acc, lds.x[1], 1, buf, i + 1);
                    }
                }
            }
        }
        if (kFp8 && blocks % 2 != 0) {
            const int b = blocks - 1;
            store_codes();
            stage_barrier<0>();
            compute_fp8(kLive, std::integral_constant<int, 1>(), acc, lds.x[(b / kStageBlocks) % 2],
                        (b / kScaleBlocks) % 2, b % kScaleBlocks);
        }
#pragma unroll
        for (int t = 0; t < kN; ++t) {
            const int r = t * kTile + m;
            if (r >= count) continue;
            uint16_t* const orow = out + (int64_t)(row0 + r) * outs;
#pragma unroll
            for (int j = 0; j < kHalf; ++j) {
                const int n = n0 + j * kTile + q * 4;
                if (n >= outs) continue;
                float v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    v[k] = kSilu ? silu_mul(acc[t][j][k], acc[t][(j + kHalf) % kColTiles][k]) : acc[t][j][k];
                store8<false>(orow + n, make_uint2(pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3])));
            }
        }
    };
    const int live = (count + kTile - 1) / kTile;
    if (live == 1) run(std::integral_constant<int, 1>());
    else if (live == 2) run(std::integral_constant<int, 2>());
    else if (live == 3) run(std::integral_constant<int, 3>());
    else run(std::integral_constant<int, kRowTiles>());
}

}  // namespace

bool expert_launch_ok(bool fp8, bool silu, int rows, int cols, int outs, int E)
{
    // offsets within a tile are 32-bit; a grid dimension holds fewer than 2^32 threads
    if (cols > kMaxExpertCols || outs > (1 << 29)) return false;
    if (silu && (int64_t)outs * cols >= ((int64_t)1 << 35)) return false;
    return expert_plan(fp8, silu, rows, cols, outs, E).workgroups * kExpertThreads < ((int64_t)1 << 32);
}

hipError_t launch_expert(const void* x, const float* x_scales, bool fp8, int rows, int cols,
                         const int32_t* expert_offset, int E, const uint8_t* w,
                         const float* w_scales, int outs, bool silu, uint16_t* out,
                         hipStream_t stream)
{
    const ExpertPlan p = expert_plan(fp8, silu, rows, cols, outs, E);
    auto go = [&](auto kernel, auto... more) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)p.workgroups), dim3(kExpertThreads), 0, stream,
                           (const uint8_t*)x, x_scales, rows, cols, expert_offset, E, w, w_scales,
                           outs, out, p.groups, more...);
    };
    if (p.tiles) {
        if (fp8) silu ? go(expert_tile_kernel<true, true>) : go(expert_tile_kernel<true, false>);
        else silu ? go(expert_tile_kernel<false, true>) : go(expert_tile_kernel<false, false>);
        return hipGetLastError();
    }
    auto pick = [&](auto split) {
        constexpr int kS = decltype(split)::value, kHalf = kTile / 2;
        const int parts = p.parts;
        if (fp8 && p.rows == kHalf)
            silu ? go(expert_stream_kernel<true, true, kS, kHalf>, parts) : go(expert_stream_kernel<true, false, kS, kHalf>, parts);
        else if (fp8)
            silu ? go(expert_stream_kernel<true, true, kS, kTile>, parts) : go(expert_stream_kernel<true, false, kS, kTile>, parts);
        else
            silu ? go(expert_stream_kernel<false, true, kS, kTile>, parts) : go(expert_stream_kernel<false, false, kS, kTile>, parts);
    };
    if (p.split == 1) pick(std::integral_constant<int, 1>());
    else pick(std::integral_constant<int, kStreamWaves>());
    return hipGetLastError();
}

}  // namespace ep
