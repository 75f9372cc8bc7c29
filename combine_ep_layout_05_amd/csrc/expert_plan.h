// expert_plan.h -- which kernel of expert.hip a batch of expert products runs,
// in how many workgroups (plain C++: nothing here needs a GPU).
#pragma once

#include <stdint.h>

namespace ep {

constexpr int kTile = 16;                         // rows and outputs of one matrix instruction
constexpr int kExpertThreads = 256;

// expert_stream_kernel
constexpr int kStreamWaves = 4;
constexpr int kGroupRows = 64;                    // weight rows per group: 4 operand tiles
constexpr int kStreamManyGroups = 2048, kStreamLongCols = 4096;

// expert_tile_kernel
constexpr int kTileWaves = 4;
constexpr int kTileRows = 64;                     // rows per workgroup
constexpr int kWaveCols = 64;                     // weight rows per wave: 4 operand tiles
constexpr int kExpertXcds = 8;
// Row tiles that run together on an XCD and share codes and rows in its L2 (1,
// 2, 4, 8: 1.74, 1.66, 1.62, 1.74 ms at 4096 tokens x 7168, gate and up, with one
// matrix instruction per block).
constexpr int kChunkTiles = 4;

struct ExpertPlan {
    bool tiles;             // expert_tile_kernel, else expert_stream_kernel
    int rows;               // rows of one expert per workgroup (tiles) or team (streaming)
    int split;              // streaming: waves of a team
    int groups;             // groups of weight rows
    int parts;              // streaming: workgroups a row tile's groups are spread over
    int64_t workgroups;
};

// Row tiles of the given height a batch can have: at most one partly filled
// tile per expert that has rows.
inline int64_t expert_row_tiles(int rows, int E, int height)
{
    return (int64_t)rows / height + (rows < E ? rows : E);
}

inline int expert_groups(int outs, int per) { return (int)(((int64_t)outs + per - 1) / per); }

// Which kernel a batch runs, by its rows per expert (the routing is on the
// device, so by their average).  Measured on MI355X, streaming / tiles, gate
// and up products of 4096 columns:
//   32 experts x 2 x 2048 weight rows (512 workgroups of tiles), fp8 rows: 39 /
//   46 us at 1 row per expert, 52 / 47 at 2, 59 / 50 at 8, 119 / 65 at 32; bf16:
//   40 / 47, 54 / 48, 69 / 50, 149 / 67;
//   8 experts (128 workgroups, half the CUs), fp8: 17 / 38 at 8, 33 / 58 at 32,
//   56 / 70 at 64; bf16: 41 / 58 at 32, 71 / 71 at 64.
inline bool expert_large(int rows, int groups, int E)
{
    const bool fill = (int64_t)E * groups >= 512;
    return rows >= (fill ? 2 : 64) * (int64_t)E;
}

// Rows per team of the streaming kernel: 16, or 8 where fp8 rows are few and the
// two parts of all of them fit one matrix instruction, which leaves registers
// for a fourth wave per SIMD.  4096 columns x 2 x 2048, 8 / 16: 29.3 / 32.4 us
// with 24 experts of 1 row, 29.0 / 31.5 with 16 of 2, 277 / 281 with 288 of 1,
// otherwise the same up to 2 rows; with 8 experts 19.7 / 16.3 at 4 rows, 23.5 /
// 16.6 at 8, 56 / 33 at 32 (each team reads the codes again).
inline int stream_rows(bool fp8, int rows, int E)
{
    return fp8 && rows < 3 * (int64_t)E ? kTile / 2 : kTile;
}

// Waves that share a group in the streaming kernel: all four when the columns
// are many or there are few groups, else one.  Measured (1 / 4 waves): 288 rows
// on 288 experts, 2048 columns x 7168 bf16 259 / 306 us, 4096 columns x 2 x 2048
// fp8 292 / 277, 7168 columns 527 / 487; 32 rows on 32 experts, 2048 x 6144 (3264
// groups) 45 / 48; 16 rows on 16 experts, 2048 x 2048 (544 groups) 15 / 10; one
// token, 8 experts, 6144 columns 32 / 21.
inline int stream_split(int64_t row_tiles, int groups, int cols)
{
    return row_tiles * groups >= kStreamManyGroups && cols < kStreamLongCols ? 1 : kStreamWaves;
}

inline ExpertPlan expert_plan(bool fp8, bool silu, int rows, int cols, int outs, int E)
{
    ExpertPlan p{};
    const int parts = silu ? 2 : 1;                             // gate and up rows
    p.groups = expert_groups(outs, kTileWaves * kWaveCols / parts);
    p.tiles = expert_large(rows, p.groups, E);
    if (p.tiles) {
        constexpr int kRound = kExpertXcds * kChunkTiles;
        p.rows = kTileRows;
        p.workgroups = (expert_row_tiles(rows, E, p.rows) + kRound - 1) / kRound * kRound * p.groups;
        return p;
    }
    p.groups = expert_groups(outs, kGroupRows / parts);
    p.rows = stream_rows(fp8, rows, E);
    const int64_t tiles = expert_row_tiles(rows, E, p.rows);
    p.split = stream_split(tiles, p.groups, cols);
    p.parts = expert_groups(p.groups, kStreamWaves / p.split);
    p.workgroups = tiles * p.parts;
    return p;
}

}  // namespace ep
