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
#include <algorithm>

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

// d of one block for 16 outputs x 16 rows.
__device__ __forceinline__ v4f block_product(v4i w, v8i x)
{
    const v8i a = {w[0], w[1], w[2], w[3], 0, 0, 0, 0};
    const v4f zero = {0.0f, 0.0f, 0.0f, 0.0f};
    // cbsz 4: A is e2m1; blgp 0: B is e4m3; no block scales (the unscaled form)
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, x, zero, 4, 0, 0, 0, 0, 0);
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

// Bounded loads: a uniform base and size, a 32-bit offset per lane and a
// uniform one; what lies past the size reads as 0.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* base, int64_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0,
                                             (int)(bytes < kMaxBuffer ? bytes : kMaxBuffer), 0x00020000);
}

__device__ __forceinline__ v4i load_b128(__amdgpu_buffer_rsrc_t r, int lane_offset, int offset)
{
    return __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(r, lane_offset, offset, 0));
}

// Few rows per expert: the weights are read once and bound the time, so the
// work is split for loads in flight.  A workgroup of 8 waves takes 16 rows of
// one expert and a share of the weight rows, 64 (silu: 32 + 32) at a time: a
// group.  kSplit waves share a group, each with its own run of blocks; their
// sums are joined through LDS in wave order (kSplit 1: nothing to join, and no
// barrier).  A wave always has the codes and rows of its next block in flight,
// across groups too.  The scales of its next 16 blocks are copied to a wave's
// own part of LDS, transposed.
constexpr int kStreamWaves = 4;
constexpr int kStreamManyGroups = 4096, kStreamLongCols = 4096;
constexpr int kGroupRows = 64;                    // weight rows per group: 4 operand tiles
constexpr int kGroupTiles = kGroupRows / kTile;
constexpr int kWindow = 16;                       // blocks whose scales are in LDS
constexpr int kScalePitch = kGroupRows + kTile + 4;   // weight rows, then fp8 rows

template <bool kFp8, bool kSilu, int kSplit>
__global__ __launch_bounds__(kStreamWaves * kWave, kFp8 ? 4 : 3) void expert_stream_kernel(
    const uint8_t* __restrict__ x, const float* __restrict__ xs, int rows, int cols,
    const int32_t* __restrict__ off, int E, const uint8_t* __restrict__ w,
    const float* __restrict__ ws, int outs, uint16_t* __restrict__ out, int n_groups,
    int n_parts)
{
    constexpr int kTeams = kStreamWaves / kSplit;                   // groups at a time
    constexpr int kOuts = kSilu ? kGroupRows / 2 : kGroupRows;      // outputs per group
    constexpr int kHalf = kOuts / kTile;                            // operand tiles of results
    __shared__ __attribute__((aligned(16))) float s_scale[kStreamWaves][kWindow * kScalePitch];
    __shared__ v4f s_part[kSplit > 1 ? kStreamWaves : 1][kGroupTiles][kWave];
    const int lane = threadIdx.x % kWave, m = lane % kTile, q = lane / kTile;
    const int wave = wave_uniform(threadIdx.x / kWave), team = wave / kSplit, part = wave % kSplit;
    int expert, row0, count;
    if (!find_tile<kTile>(off, E, rows, blockIdx.x / n_parts, lane, expert, row0, count)) return;
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
    const int xo = min(m, count - 1) * cols * kRowBytes + q * (kFp8 ? 16 : 64);
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
                const float f = kFp8 ? sb[kGroupRows + m] : 1.0f;
#pragma unroll
                for (int j = 0; j < kGroupTiles; ++j) {
                    const v4f sw = *(const v4f*)(sb + j * kTile + q * 4);
                    v4f d;
                    if constexpr (kFp8) {
                        const v8i x8 = {xv[u][0][0], xv[u][0][1], xv[u][0][2], xv[u][0][3],
                                        xv[u][1][0], xv[u][1][1], xv[u][1][2], xv[u][1][3]};
                        d = block_product(cur.w[u][j], x8);
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

// Large batches: a workgroup computes up to 64 rows x 256 weight rows, 64 of
// them per wave.  Codes and rows go from memory straight to LDS, a ring of
// stages of one block each, kStages - 1 of them in flight; every wave loads its
// own codes and a quarter of the rows, waits for its own loads of the oldest
// stage and meets the others at one barrier per block.  Scales are loaded for
// 4 blocks at a time (16 bytes of one row per lane: block by block they would
// be one 4-byte piece of 64 lines) and kept in LDS transposed.
//
// A load of 16 bytes per lane covers whole rows of the block (codes: 16 rows x
// 64 bytes; fp8 rows: 8 x 128; bf16: 4 x 256), and the 16-byte pieces of a row
// are permuted (piece ^ row bits) so that 8 lanes reading one piece of 8
// neighbouring rows meet 8 different banks.
constexpr int kWaveCols = 64;                    // weight rows per wave: 4 operand tiles
constexpr int kColTiles = kWaveCols / kTile;
constexpr int kTileRows = 64;                    // rows per workgroup
constexpr int kRowTiles = kTileRows / kTile;

template <bool kFp8> struct TileStage {
    static constexpr int kRowBytes = kScaleBlock * (kFp8 ? 1 : 2);
    static constexpr int kRowsPerLoad = 1024 / kRowBytes;
    static constexpr int kXLoads = kTileRows / kRowsPerLoad / kExpertWaves;      // per wave
    static constexpr int kLoads = kXLoads + kColTiles;                           // per wave and stage
    static constexpr int kStages = kFp8 ? 3 : 2;
    uint8_t w[kExpertWaves][kWaveCols * kScaleBlock / 2];
    uint8_t x[kTileRows * kRowBytes];
};
constexpr int kScaleBlocks = 4;                  // blocks per load of scales

// One object: between separate ones the compiler tracks which loads into LDS
// might touch what is read, and waits for all in flight before every read.
template <bool kFp8> struct TileShared {
    TileStage<kFp8> ring[TileStage<kFp8>::kStages];
    float ws[kExpertWaves][kScaleBlocks][kWaveCols];
    float xs[kFp8 ? 2 : 1][kScaleBlocks][kTileRows];
};

__device__ __forceinline__ void load_lds16(__amdgpu_buffer_rsrc_t r, void* lds, int lane_offset, int offset)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16,
                                             lane_offset, offset, 0, 0);
}

// Waits until at most kOutstanding of this wave's loads are in flight (they
// complete in order) and its LDS reads are done, and meets the workgroup: then
// the older loads of every wave are in LDS and what was read before may be
// overwritten.  A workgroup fence in place of the empty asm statements, which
// only keep the compiler from moving accesses across, would wait for every
// load in flight into LDS.
template <int kOutstanding>
__device__ __forceinline__ void stage_barrier()
{
    static_assert(kOutstanding >= 0 && kOutstanding < 64, "vmcnt holds 6 bits");
    asm volatile("" ::: "memory");
    // gfx9 encoding: vmcnt in bits 3:0 and 15:14, expcnt in 6:4 (not waited for), lgkmcnt 0 in 11:8
    __builtin_amdgcn_s_waitcnt((kOutstanding & 15) | ((kOutstanding >> 4) << 14) | 0x70);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

template <bool kFp8, bool kSilu>
__global__ __launch_bounds__(kExpertWaves * kWave, 2) void expert_tile_kernel(
    const uint8_t* __restrict__ x, const float* __restrict__ xs, int rows, int cols,
    const int32_t* __restrict__ off, int E, const uint8_t* __restrict__ w,
    const float* __restrict__ ws, int outs, uint16_t* __restrict__ out, int n_groups)
{
    using S = TileStage<kFp8>;
    __shared__ __attribute__((aligned(16))) TileShared<kFp8> lds;
    const int lane = threadIdx.x % kWave, m = lane % kTile, q = lane / kTile;
    const int wave = wave_uniform(threadIdx.x / kWave);
    // the column groups of one row tile on one XCD (they share its rows)
    const int slot = blockIdx.x / kXcds;
    const int tile = (slot / n_groups) * kXcds + blockIdx.x % kXcds;
    constexpr int kParts = kSilu ? 2 : 1;                      // gate and up rows
    constexpr int kOuts = kWaveCols / kParts;                  // outputs per wave
    constexpr int kHalf = kOuts / kTile;                       // operand tiles of a part
    const int n0 = ((slot % n_groups) * kExpertWaves + wave) * kOuts;
    int expert, row0, count;
    if (!find_tile<kTileRows>(off, E, rows, tile, lane, expert, row0, count)) return;
    const int live = (count + kTile - 1) / kTile;
    const int blocks = cols / kScaleBlock, half_cols = cols / 2;
    const int64_t wrows = (int64_t)outs * kParts;

    // codes: load j is operand tile j, lane i piece i % 4 of row i / 4 (past the
    // last output: other rows or 0, not stored)
    __amdgpu_buffer_rsrc_t wr[kParts];
    const int64_t n_base = min(n0, outs);
#pragma unroll
    for (int h = 0; h < kParts; ++h) {
        const int64_t r = n_base + (int64_t)h * outs;
        wr[h] = buffer(w + (expert * wrows + r) * half_cols, (wrows - r) * half_cols);
    }
    const __amdgpu_buffer_rsrc_t sr = buffer(ws + (expert * wrows + n_base) * blocks,
                                             (wrows - n_base) * blocks * 4);
    const int wo = (lane / 4) * half_cols + ((lane % 4) ^ ((lane / 8) % 4)) * 16;
    // rows past the last are read as the last one; what they give is not stored
    const __amdgpu_buffer_rsrc_t xr = buffer(x + (int64_t)row0 * cols * (S::kRowBytes / kScaleBlock),
                                             (int64_t)count * cols * (S::kRowBytes / kScaleBlock));
    const __amdgpu_buffer_rsrc_t xsr = buffer(kFp8 ? xs + (int64_t)row0 * blocks : nullptr,
                                              kFp8 ? (int64_t)count * blocks * 4 : 0);
    int xo[S::kXLoads];
#pragma unroll
    for (int p = 0; p < S::kXLoads; ++p) {
        constexpr int kPieces = S::kRowBytes / 16;
        const int r = (wave * S::kXLoads + p) * S::kRowsPerLoad + lane / kPieces;
        const int piece = (lane % kPieces) ^ (r % kPieces);
        xo[p] = min(r, count - 1) * cols * (S::kRowBytes / kScaleBlock) + piece * 16;
    }
    auto load = [&](S& s, int b) {
        b = min(b, blocks - 1);                  // past the end: loads that nobody reads
#pragma unroll
        for (int p = 0; p < S::kXLoads; ++p)
            load_lds16(xr, s.x + (wave * S::kXLoads + p) * 1024, xo[p], b * S::kRowBytes);
#pragma unroll
        for (int h = 0; h < kParts; ++h)
#pragma unroll
            for (int j = 0; j < kHalf; ++j)
                load_lds16(wr[h], s.w[wave] + (h * kHalf + j) * 1024, wo, j * kTile * half_cols + b * 64);
    };
    // Scales of blocks b .. b + 3: lane i that of weight row i of the wave (silu:
    // lanes 32 .. 63 the up rows), lanes 0 .. 15 those of 16 of the fp8 rows.  The
    // 4 blocks end at the row's last one at most: no load is partly past its
    // buffer.
    const int so = (kSilu ? lane % kOuts + lane / kOuts * outs : lane) * blocks * 4;
    const int xso = min(wave * kTile + m, count - 1) * blocks * 4;
    v4f wsv, xsv;
    auto load_scales = [&](int b) {
        if (blocks >= kScaleBlocks) {
            const int bl = min(b, blocks - kScaleBlocks);
            wsv = __builtin_bit_cast(v4f, load_b128(sr, so, bl * 4));
            if constexpr (kFp8) xsv = __builtin_bit_cast(v4f, load_b128(xsr, xso, bl * 4));
        } else {
            v4i a, c;
#pragma unroll
            for (int i = 0; i < kScaleBlocks; ++i) {
                a[i] = __builtin_amdgcn_raw_buffer_load_b32(sr, so, min(i, blocks - 1) * 4, 0);
                c[i] = kFp8 ? __builtin_amdgcn_raw_buffer_load_b32(xsr, xso, min(i, blocks - 1) * 4, 0) : 0;
            }
            wsv = __builtin_bit_cast(v4f, a);
            xsv = __builtin_bit_cast(v4f, c);
        }
    };
    auto store_scales = [&](int b, int buf) {
        const int skip = blocks >= kScaleBlocks ? b - min(b, blocks - kScaleBlocks) : 0;
#pragma unroll
        for (int i = 0; i < kScaleBlocks; ++i) {
            if (i < skip) continue;
            lds.ws[wave][i - skip][lane] = wsv[i];
            if constexpr (kFp8) if (lane < kTile) lds.xs[buf][i - skip][wave * kTile + lane] = xsv[i];
        }
    };
    v4f acc[kRowTiles][kColTiles];
#pragma unroll
    for (int t = 0; t < kRowTiles; ++t)
#pragma unroll
        for (int j = 0; j < kColTiles; ++j) acc[t][j] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};

    auto compute = [&](const S& s, int buf, int i_block) {
        v4i wc[kColTiles];
        v4f sw[kColTiles];
#pragma unroll
        for (int j = 0; j < kColTiles; ++j) {
            wc[j] = *(const v4i*)(s.w[wave] + j * 1024 + m * 64 + (q ^ ((m / 2) % 4)) * 16);
            sw[j] = *(const v4f*)&lds.ws[wave][i_block][j * kTile + q * 4];
        }
        if constexpr (kFp8) {
#pragma unroll
            for (int t = 0; t < kRowTiles; ++t) {
                if (t >= live) break;
                const uint8_t* const xrow = s.x + (t * kTile + m) * 128;
                const v4i lo = *(const v4i*)(xrow + (q ^ (m % 8)) * 16);
                const v4i hi = *(const v4i*)(xrow + ((4 + q) ^ (m % 8)) * 16);
                const v8i xb = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
                const float f = lds.xs[buf][i_block][t * kTile + m];
                v4f d[kColTiles];
#pragma unroll
                for (int j = 0; j < kColTiles; ++j) d[j] = block_product(wc[j], xb);
#pragma unroll
                for (int j = 0; j < kColTiles; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc[t][j][i] = __builtin_fmaf(d[j][i], sw[j][i] * f, acc[t][j][i]);
            }
        } else {
            v8bf wb[kColTiles][4];
#pragma unroll
            for (int j = 0; j < kColTiles; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) wb[j][i] = bf16x8_of_codes((uint32_t)wc[j][i]);
#pragma unroll
            for (int t = 0; t < kRowTiles; ++t) {
                if (t >= live) break;
                v8bf xb[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    xb[i] = *(const v8bf*)(s.x + (t * kTile + m) * 256 + ((q * 4 + i) ^ m) * 16);
#pragma unroll
                for (int j = 0; j < kColTiles; ++j) {
                    v4f d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[j][i], xb[i], d, 0, 0, 0);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc[t][j][i] = __builtin_fmaf(d[i], sw[j][i], acc[t][j][i]);
                }
            }
        }
    };

    constexpr int kAhead = S::kStages - 1;
    load_scales(0);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load(lds.ring[i], i);
    int at = 0;
    for (int b0 = 0; b0 < blocks; b0 += kScaleBlocks) {
        const int buf = kFp8 ? (b0 / kScaleBlocks) % 2 : 0;
        store_scales(b0, buf);
#pragma unroll
        for (int i = 0; i < kScaleBlocks; ++i) {
            if (b0 + i >= blocks) break;
            stage_barrier<(kAhead - 1) * S::kLoads>();
            if (i == 0 && b0 + kScaleBlocks < blocks) load_scales(b0 + kScaleBlocks);
            load(lds.ring[at == 0 ? kAhead : at - 1], b0 + i + kAhead);      // the stage read last
            compute(lds.ring[at], buf, i);
            at = at + 1 == S::kStages ? 0 : at + 1;
        }
    }
    stage_barrier<0>();                          // nothing in flight into LDS when the wave ends
#pragma unroll
    for (int t = 0; t < kRowTiles; ++t) {
        const int r = t * kTile + m;
        if (r >= count) continue;
        uint16_t* const orow = out + (int64_t)(row0 + r) * outs;
#pragma unroll
        for (int j = 0; j < kHalf; ++j) {
            const int n = n0 + j * kTile + q * 4;
            if (n >= outs) continue;
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = kSilu ? silu_mul(acc[t][j][i], acc[t][(j + kHalf) % kColTiles][i]) : acc[t][j][i];
            store8<false>(orow + n, make_uint2(pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3])));
        }
    }
}

}  // namespace

namespace {

// Row tiles of the given height a batch can have: at most one partly filled
// tile per expert that has rows.
int64_t max_tiles(int rows, int E, int height)
{
    return (int64_t)rows / height + (rows < E ? rows : E);
}

// Few rows per expert: the kernel that streams the weights; more: the tiles.
bool expert_large(int rows, int E) { return rows > 8 * (int64_t)E; }

int64_t tile_blocks(bool silu, int rows, int outs, int E)
{
    const int per = kExpertWaves * (silu ? kWaveCols / 2 : kWaveCols);
    const int64_t groups = ((int64_t)outs + per - 1) / per;
    return (max_tiles(rows, E, kTileRows) + kXcds - 1) / kXcds * kXcds * groups;
}

int stream_groups(bool silu, int outs)
{
    const int per = silu ? kGroupRows / 2 : kGroupRows;
    return (int)(((int64_t)outs + per - 1) / per);
}

// Waves that share a group in the streaming kernel.
int stream_split(bool silu, int rows, int cols, int outs, int E)
{
    const bool many = max_tiles(rows, E, kTile) * stream_groups(silu, outs) >= kStreamManyGroups;
    return many && cols < kStreamLongCols ? 1 : kStreamWaves;
}

int64_t stream_blocks(bool silu, int rows, int cols, int outs, int E)
{
    const int teams = kStreamWaves / stream_split(silu, rows, cols, outs, E);
    return max_tiles(rows, E, kTile) * ((stream_groups(silu, outs) + teams - 1) / teams);
}

}  // namespace

bool expert_launch_ok(bool silu, int rows, int cols, int outs, int E)
{
    // offsets within a tile are 32-bit; a grid dimension holds fewer than 2^32 threads
    if (cols > kMaxExpertCols || outs > (1 << 29)) return false;
    static_assert(kExpertWaves == kStreamWaves, "both kernels launch the same workgroups");
    if (silu && (int64_t)outs * cols >= ((int64_t)1 << 36)) return false;
    const int64_t blocks = expert_large(rows, E) ? tile_blocks(silu, rows, outs, E)
                                                 : stream_blocks(silu, rows, cols, outs, E);
    return blocks * kExpertWaves * kWave < ((int64_t)1 << 32);
}

hipError_t launch_expert(const void* x, const float* x_scales, bool fp8, int rows, int cols,
                         const int32_t* expert_offset, int E, const uint8_t* w,
                         const float* w_scales, int outs, bool silu, uint16_t* out,
                         hipStream_t stream)
{
    const dim3 block(kExpertWaves * kWave);
    if (expert_large(rows, E)) {
        const int per = kExpertWaves * (silu ? kWaveCols / 2 : kWaveCols);
        const int groups = (outs + per - 1) / per;
        const dim3 grid((unsigned)tile_blocks(silu, rows, outs, E));
        auto go = [&](auto kernel) {
            hipLaunchKernelGGL(kernel, grid, block, 0, stream, (const uint8_t*)x, x_scales, rows,
                               cols, expert_offset, E, w, w_scales, outs, out, groups);
        };
        if (fp8) silu ? go(expert_tile_kernel<true, true>) : go(expert_tile_kernel<true, false>);
        else silu ? go(expert_tile_kernel<false, true>) : go(expert_tile_kernel<false, false>);
        return hipGetLastError();
    }
    const int split = stream_split(silu, rows, cols, outs, E);
    const int groups = stream_groups(silu, outs), teams = kStreamWaves / split;
    const dim3 grid((unsigned)stream_blocks(silu, rows, cols, outs, E));
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, block, 0, stream, (const uint8_t*)x, x_scales, rows, cols,
                           expert_offset, E, w, w_scales, outs, out, groups, (groups + teams - 1) / teams);
    };
    auto pick = [&](auto sp) {
        constexpr int kS = decltype(sp)::value;
        if (fp8) silu ? go(expert_stream_kernel<true, true, kS>) : go(expert_stream_kernel<true, false, kS>);
        else silu ? go(expert_stream_kernel<false, true, kS>) : go(expert_stream_kernel<false, false, kS>);
    };
    if (split == 1) pick(std::integral_constant<int, 1>());
    else pick(std::integral_constant<int, kStreamWaves>());
    return hipGetLastError();
}

}  // namespace ep
