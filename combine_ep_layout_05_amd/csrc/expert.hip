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
constexpr int kMaxExpertCols = 1 << 24;      // 64 rows of bf16 within 32-bit offsets

// Row tile `idx` of the batch: its expert, first row and row count, from the
// expert offsets (clamped to the rows there are).  False past the last tile.
// Called by whole waves; the result is wave-uniform.  64 experts a round, one
// per lane: tiles before each by a DPP scan, the expert that holds `idx` by a
// ballot.
template <int kRows>
__device__ __forceinline__ bool find_tile(const int32_t* __restrict__ off, int E, int rows, int idx,
                                          int lane, int& expert, int& row0, int& count)
{
    int left = idx;
    for (int e0 = 0; e0 < E; e0 += kWave) {
        const int e = min(e0 + lane, E - 1);
        int a = off[e], b = off[e + 1];
        a = min(max(a, 0), rows);
        b = min(max(b, a), rows);
        const int tiles = e0 + lane < E ? (b - a + kRows - 1) / kRows : 0;
        const int incl = wave_inclusive_scan(tiles);
        const uint64_t past = __ballot(incl > left);
        if (past) {
            const int win = __builtin_ctzll(past);
            left -= read_lane(incl - tiles, win);
            expert = e0 + win;
            row0 = read_lane(a, win) + left * kRows;
            count = min(kRows, read_lane(b, win) - row0);
            return true;
        }
        left -= read_lane(incl, kWave - 1);
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

// Few rows per expert: the weights are read once and bound the time, so the
// work is split for loads in flight.  A workgroup of 8 waves takes 16 rows of
// one expert and a share of the weight rows, 64 (silu: 32 + 32) at a time; its
// waves split the columns, wave i taking blocks i, i + 8, ..., and always have
// the next block's codes and rows in flight, across the groups of 64 too.  The
// waves' sums are joined through LDS in wave order.  The scales of a group are
// one contiguous piece of memory; they are copied to LDS transposed, a window
// of at most 64 blocks at a time.
constexpr int kStreamWaves = 8;
constexpr int kGroupRows = 64;                    // weight rows per group: 4 operand tiles
constexpr int kGroupTiles = kGroupRows / kTile;
constexpr int kWindow = 64;                       // blocks whose scales are in LDS
constexpr int kScaleRows = kGroupRows + kTile;    // weight rows, then fp8 rows
constexpr int kScalePitch = kScaleRows + 4;

template <bool kFp8, bool kSilu>
__global__ __launch_bounds__(kStreamWaves * kWave, 4) void expert_stream_kernel(
    const uint8_t* __restrict__ x, const float* __restrict__ xs, int rows, int cols,
    const int32_t* __restrict__ off, int E, const uint8_t* __restrict__ w,
    const float* __restrict__ ws, int outs, uint16_t* __restrict__ out, int n_groups, int n_split)
{
    __shared__ __attribute__((aligned(16))) float s_scale[2][kWindow * kScalePitch];
    __shared__ v4f s_part[kStreamWaves][kGroupTiles][kWave];
    const int lane = threadIdx.x % kWave, m = lane % kTile, q = lane / kTile;
    const int wave = wave_uniform(threadIdx.x / kWave);
    constexpr int kOuts = kSilu ? kGroupRows / 2 : kGroupRows;      // outputs per group
    int expert, row0, count;
    if (!find_tile<kTile>(off, E, rows, blockIdx.x / n_split, lane, expert, row0, count)) return;
    const int g0 = blockIdx.x % n_split;
    const int blocks = cols / kScaleBlock;
    const int windows = (blocks + kWindow - 1) / kWindow;
    const int64_t wrow0 = expert * (kSilu ? 2 * (int64_t)outs : (int64_t)outs);
    // lanes past the last row or output read a valid one; what they compute is not stored
    const uint8_t* const xb = x + (int64_t)row0 * cols * (kFp8 ? 1 : 2);
    const uint32_t xo = (uint32_t)min(m, count - 1) * cols * (kFp8 ? 1 : 2) + q * (kFp8 ? 16 : 64);

    constexpr int kXRegs = kFp8 ? 2 : 4;
    struct Step { v4i w[kGroupTiles]; v4i x[kXRegs]; };
    // weight row j * 16 + m of group g (silu: tiles 0, 1 gate, 2, 3 up)
    auto weight_row = [&](int g, int r) {
        const int h = kSilu ? r / kOuts : 0;
        return wrow0 + (int64_t)h * outs + min(g * kOuts + (kSilu ? r % kOuts : r), outs - 1);
    };
    auto load = [&](Step& s, int g, int b) {
#pragma unroll
        for (int j = 0; j < kGroupTiles; ++j)
            s.w[j] = *(const v4i*)(w + weight_row(g, j * kTile + m) * (cols / 2) + b * 64 + q * 16);
#pragma unroll
        for (int i = 0; i < kXRegs; ++i)
            s.x[i] = *(const v4i*)(xb + xo + b * (kFp8 ? 128 : 256) + i * (kFp8 ? 64 : 16));
    };
    // the scales of 10 rows per wave, lane = block of the window
    constexpr int kMine = kFp8 ? kScaleRows / kStreamWaves : kGroupRows / kStreamWaves;
    float sc[kMine];
    auto load_scales = [&](int g, int win) {
        const int b = win * kWindow + lane;
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int r = i * kStreamWaves + wave;
            const float* p = r < kGroupRows ? ws + weight_row(g, r) * blocks
                                            : xs + (int64_t)(row0 + min(r - kGroupRows, count - 1)) * blocks;
            sc[i] = b < blocks ? p[b] : 0.0f;
        }
    };
    auto store_scales = [&](int buf) {
#pragma unroll
        for (int i = 0; i < kMine; ++i) s_scale[buf][lane * kScalePitch + i * kStreamWaves + wave] = sc[i];
    };

    if (g0 >= n_groups) return;
    Step cur, next;
    load_scales(g0, 0);
    if (wave < blocks) load(cur, g0, wave);
    store_scales(0);
    __syncthreads();
    int buf = 0;
    for (int g = g0; g < n_groups; g += n_split) {
        v4f acc[kGroupTiles];
#pragma unroll
        for (int j = 0; j < kGroupTiles; ++j) acc[j] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
        for (int win = 0; win < windows; ++win) {
            const bool last = win + 1 == windows;
            const int g_next = last ? g + n_split : g;
            const bool more = g_next < n_groups;
            if (more) load_scales(g_next, last ? 0 : win + 1);
            const int end = min(blocks, (win + 1) * kWindow);
            for (int b = win * kWindow + wave; b < end; b += kStreamWaves) {
                // the block after this one, in this window, the next or the next group
                const int bn = b + kStreamWaves;
                if (bn < blocks) load(next, g, bn);
                else if (g + n_split < n_groups) load(next, g + n_split, wave);
                const float* const sb = s_scale[buf] + (b - win * kWindow) * kScalePitch;
                const float f = kFp8 ? sb[kGroupRows + m] : 1.0f;
#pragma unroll
                for (int j = 0; j < kGroupTiles; ++j) {
                    const v4f sw = *(const v4f*)(sb + j * kTile + q * 4);
                    v4f d;
                    if constexpr (kFp8) {
                        const v8i xv = {cur.x[0][0], cur.x[0][1], cur.x[0][2], cur.x[0][3],
                                        cur.x[1][0], cur.x[1][1], cur.x[1][2], cur.x[1][3]};
                        d = block_product(cur.w[j], xv);
                    } else {
                        d = block_product(cur.w[j], cur.x);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[j][i] = __builtin_fmaf(d[i], sw[i] * f, acc[j][i]);
                }
                cur = next;
            }
            buf ^= 1;
            if (more) store_scales(buf);
            if (last)
#pragma unroll
                for (int j = 0; j < kGroupTiles; ++j) s_part[wave][j][lane] = acc[j];
            lds_barrier();
        }
        // two neighbouring outputs per thread: lane's quarter `half` of operand tile j
        const int idx = threadIdx.x / 2, half = threadIdx.x % 2;
        const int j = idx / kWave, ln = idx % kWave;
        if (j < kOuts / kTile) {
            float v[2] = {0.0f, 0.0f}, u[2] = {0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < kStreamWaves; ++i) {
                const float* const p = (const float*)&s_part[i][j][ln] + half * 2;
                v[0] += p[0];
                v[1] += p[1];
                if constexpr (kSilu) {
                    const float* const pu = (const float*)&s_part[i][j + kOuts / kTile][ln] + half * 2;
                    u[0] += pu[0];
                    u[1] += pu[1];
                }
            }
            const int r = ln % kTile, n = g * kOuts + j * kTile + (ln / kTile) * 4 + half * 2;
            if (r < count && n < outs) {
                if constexpr (kSilu) { v[0] = silu_mul(v[0], u[0]); v[1] = silu_mul(v[1], u[1]); }
                *(uint32_t*)(out + (int64_t)(row0 + r) * outs + n) = pack2_bf16(v[0], v[1]);
            }
        }
        lds_barrier();
    }
}

// Large batches: a workgroup computes up to kTileRows rows x 4 * kWaveCols
// weight rows.  Every wave has its own weight rows, loaded straight into
// registers (no other wave needs them), and all the rows: those go through
// LDS, one 128-column block at a time, double buffered, loaded one block
// ahead.  Row groups of 16 past the last row are skipped.
constexpr int kWaveCols = 64;                    // weight rows per wave: 4 operand tiles
constexpr int kColTiles = kWaveCols / kTile;

template <bool kFp8> struct TileShape {
    static constexpr int kRows = 64;                         // rows per workgroup
    static constexpr int kRowTiles = kRows / kTile;
    static constexpr int kBlockBytes = kScaleBlock * (kFp8 ? 1 : 2);
    static constexpr int kPieces = kRows * kBlockBytes / 1024 / kExpertWaves;   // 1 KB loads per wave
};

template <bool kFp8, bool kSilu>
__global__ __launch_bounds__(kExpertWaves * kWave, 2) void expert_tile_kernel(
    const uint8_t* __restrict__ x, const float* __restrict__ xs, int rows, int cols,
    const int32_t* __restrict__ off, int E, const uint8_t* __restrict__ w,
    const float* __restrict__ ws, int outs, uint16_t* __restrict__ out, int n_groups)
{
    using S = TileShape<kFp8>;
    __shared__ __attribute__((aligned(16))) uint8_t s_x[2][S::kRows * S::kBlockBytes];
    __shared__ float s_xs[2][kFp8 ? S::kRows : 1];
    __shared__ __attribute__((aligned(16))) float s_ws[2][kExpertWaves][kWaveCols];
    const int lane = threadIdx.x % kWave, m = lane % kTile, q = lane / kTile;
    const int wave = wave_uniform(threadIdx.x / kWave);
    // the column groups of one row tile on one XCD (they share its rows)
    const int slot = blockIdx.x / kXcds;
    const int tile = (slot / n_groups) * kXcds + blockIdx.x % kXcds;
    constexpr int kOuts = kSilu ? kWaveCols / 2 : kWaveCols;   // outputs per wave
    const int n0 = ((slot % n_groups) * kExpertWaves + wave) * kOuts;
    int expert, row0, count;
    if (!find_tile<S::kRows>(off, E, rows, tile, lane, expert, row0, count)) return;
    const int live = (count + kTile - 1) / kTile;
    const int blocks = cols / kScaleBlock;
    const int64_t wrows = kSilu ? 2 * (int64_t)outs : outs;

    // operand tile j: weight rows n0 + 16 j (silu: two of the gate, then the two of the up rows)
    // (a uniform base and a 32-bit offset per lane, which stays below 16 rows)
    const uint8_t* wp[kColTiles];
    int wo[kColTiles];
#pragma unroll
    for (int j = 0; j < kColTiles; ++j) {
        const int h = kSilu ? j / 2 : 0, t = kSilu ? j % 2 : j;
        const int n = min(n0 + t * kTile, outs - 1);
        wp[j] = w + (expert * wrows + (int64_t)h * outs + n) * (cols / 2);
        wo[j] = min(m, outs - 1 - n) * (cols / 2) + q * 16;
    }
    // lane i of a wave stages the scale of weight row (i / 16, i % 16) of its tiles
    const float* wsp;
    {
        const int h = kSilu ? q / 2 : 0, t = kSilu ? q % 2 : q;
        wsp = ws + (expert * wrows + (int64_t)h * outs + min(n0 + t * kTile + m, outs - 1)) * blocks;
    }
    // a wave stages row tile `wave`; fp8: piece p is half p of its operand, in
    // operand order; bf16: rows 4 p .. 4 p + 3, 16-byte pieces of row r at r ^ piece
    const uint8_t* const xp = x + (int64_t)row0 * cols * (kFp8 ? 1 : 2);
    int xo[S::kPieces];
    int xdst[S::kPieces];
    const bool xlive = wave < live;
#pragma unroll
    for (int p = 0; p < S::kPieces; ++p) {
        if constexpr (kFp8) {
            xo[p] = min(wave * kTile + m, count - 1) * cols + p * 64 + q * 16;
            xdst[p] = (wave * 2 + p) * 1024 + lane * 16;
        } else {
            const int r = wave * kTile + p * 4 + q;
            xo[p] = min(r, count - 1) * cols * 2 + m * 16;
            xdst[p] = r * 256 + ((m ^ (r % kTile)) * 16);
        }
    }
    const int xs_row = threadIdx.x;                 // fp8: thread i stages the scale of row i
    const float* const xsp = kFp8 ? xs + (int64_t)(row0 + min(xs_row, count - 1)) * blocks : nullptr;

    v4i xr[S::kPieces], wr[kColTiles];
    float xsr = 0.0f, wsr;
    auto load = [&](int b) {
#pragma unroll
        for (int p = 0; p < S::kPieces; ++p)
            if (xlive) xr[p] = *(const v4i*)(xp + (int64_t)b * S::kBlockBytes + (uint32_t)xo[p]);
        if constexpr (kFp8) if (xs_row < S::kRows) xsr = xsp[b];
        wsr = wsp[b];
    };
    auto load_w = [&](int b) {
#pragma unroll
        for (int j = 0; j < kColTiles; ++j) wr[j] = *(const v4i*)(wp[j] + (int64_t)b * 64 + (uint32_t)wo[j]);
    };
    v4f acc[S::kRowTiles][kColTiles];
#pragma unroll
    for (int t = 0; t < S::kRowTiles; ++t)
#pragma unroll
        for (int j = 0; j < kColTiles; ++j) acc[t][j] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};

    load(0);
    load_w(0);
    for (int b = 0; b < blocks; ++b) {
        const int buf = b & 1;
#pragma unroll
        for (int p = 0; p < S::kPieces; ++p)
            if (xlive) *(v4i*)(s_x[buf] + xdst[p]) = xr[p];
        if constexpr (kFp8) if (xs_row < S::kRows) s_xs[buf][xs_row] = xsr;
        s_ws[buf][wave][lane] = wsr;
        lds_barrier();
        v4i wc[kColTiles];
#pragma unroll
        for (int j = 0; j < kColTiles; ++j) wc[j] = wr[j];
        if (b + 1 < blocks) { load(b + 1); load_w(b + 1); }
        v4f sw[kColTiles];
#pragma unroll
        for (int j = 0; j < kColTiles; ++j) sw[j] = *(const v4f*)&s_ws[buf][wave][j * kTile + q * 4];
        if constexpr (kFp8) {
#pragma unroll
            for (int t = 0; t < S::kRowTiles; ++t) {
                if (t >= live) break;
                const v4i lo = *(const v4i*)(s_x[buf] + t * 2048 + lane * 16);
                const v4i hi = *(const v4i*)(s_x[buf] + t * 2048 + 1024 + lane * 16);
                const v8i xb = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
                const float f = s_xs[buf][t * kTile + m];
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
                for (int s = 0; s < 4; ++s) wb[j][s] = bf16x8_of_codes((uint32_t)wc[j][s]);
#pragma unroll
            for (int t = 0; t < S::kRowTiles; ++t) {
                if (t >= live) break;
                v8bf xb[4];
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    xb[s] = *(const v8bf*)(s_x[buf] + (t * kTile + m) * 256 + (((q * 4 + s) ^ m) * 16));
#pragma unroll
                for (int j = 0; j < kColTiles; ++j) {
                    v4f d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[j][s], xb[s], d, 0, 0, 0);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc[t][j][i] = __builtin_fmaf(d[i], sw[j][i], acc[t][j][i]);
                }
            }
        }
    }
#pragma unroll
    for (int t = 0; t < S::kRowTiles; ++t) {
        const int r = t * kTile + m;
        if (r >= count) continue;
        uint16_t* const orow = out + (int64_t)(row0 + r) * outs;
#pragma unroll
        for (int j = 0; j < (kSilu ? kColTiles / 2 : kColTiles); ++j) {
            const int n = n0 + j * kTile + q * 4;
            if (n >= outs) continue;
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = kSilu ? silu_mul(acc[t][j][i], acc[t][j + kColTiles / 2][i]) : acc[t][j][i];
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

constexpr int64_t kStreamBlocks = 4096;

// Few rows per expert: the kernel that streams the weights; more: the tiles.
bool expert_large(int rows, int E) { return rows > 8 * (int64_t)E; }

int64_t tile_blocks(bool fp8, bool silu, int rows, int outs, int E)
{
    const int per = kExpertWaves * (silu ? kWaveCols / 2 : kWaveCols);
    const int64_t groups = ((int64_t)outs + per - 1) / per;
    const int64_t tiles = max_tiles(rows, E, fp8 ? TileShape<true>::kRows : TileShape<false>::kRows);
    return (tiles + kXcds - 1) / kXcds * kXcds * groups;
}

}  // namespace

bool expert_launch_ok(bool fp8, bool silu, int rows, int cols, int outs, int E)
{
    // offsets within a tile are 32-bit; a grid dimension holds fewer than 2^32 threads
    if (cols > kMaxExpertCols || outs > (1 << 29)) return false;
    if (!expert_large(rows, E)) return true;       // at most kStreamBlocks + max_tiles workgroups
    return tile_blocks(fp8, silu, rows, outs, E) * kExpertWaves * kWave < ((int64_t)1 << 32);
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
        const dim3 grid((unsigned)tile_blocks(fp8, silu, rows, outs, E));
        auto go = [&](auto kernel) {
            hipLaunchKernelGGL(kernel, grid, block, 0, stream, (const uint8_t*)x, x_scales, rows,
                               cols, expert_offset, E, w, w_scales, outs, out, groups);
        };
        if (fp8) silu ? go(expert_tile_kernel<true, true>) : go(expert_tile_kernel<true, false>);
        else silu ? go(expert_tile_kernel<false, true>) : go(expert_tile_kernel<false, false>);
        return hipGetLastError();
    }
    const int per = silu ? kGroupRows / 2 : kGroupRows;
    const int groups = (outs + per - 1) / per;
    const int64_t tiles = max_tiles(rows, E, kTile);
    // about kStreamBlocks workgroups: several rounds of the 512 that run at once
    const int split = (int)std::min<int64_t>(groups, (kStreamBlocks + tiles - 1) / tiles);
    const dim3 grid((unsigned)(tiles * split));
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(kStreamWaves * kWave), 0, stream, (const uint8_t*)x,
                           x_scales, rows, cols, expert_offset, E, w, w_scales, outs, out, groups,
                           split);
    };
    if (fp8) silu ? go(expert_stream_kernel<true, true>) : go(expert_stream_kernel<true, false>);
    else silu ? go(expert_stream_kernel<false, true>) : go(expert_stream_kernel<false, false>);
    return hipGetLastError();
}

}  // namespace ep
