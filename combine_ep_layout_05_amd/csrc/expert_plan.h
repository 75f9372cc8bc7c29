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
// device, so by their average).  The streaming kernel asks for an expert's codes
// again for every 16 rows, the tile kernel for every 64, but a workgroup of
// tiles takes its time however few there are: the fewer workgroups (experts x
// groups of weight rows), the more rows it takes to pay.  Measured on MI355X, gate
// and up products of 4096 columns, 2 x 2048 weight rows (16 groups), streaming /
// tiles, us:
//   experts  fp8 rows, by rows per expert               bf16 rows
//    1       64: 11.5 / 63, 512: 51 / 67                64: 12 / 62, 512: 65 / 68
//    4       64: 34 / 67, 128: 56 / 67, 256: 101 / 71   64: 42 / 68, 128: 70 / 67
//    8       32: 33 / 58, 64: 56 / 70                   32: 42 / 58, 64: 71 / 71
//   16       16: 43 / 51, 32: 64 / 60, 64: 105 / 73     16: 52 / 53, 32: 80 / 61
//   24       4: 44 / 46, 8: 46 / 46, 32: 92 / 63        4: 46 / 47, 8: 54 / 47
//   31       1: 37 / 45, 2: 48 / 46, 32: 117 / 64       2: 50 / 48, 32: 145 / 67
//   32       1: 39 / 46, 2: 52 / 47, 32: 119 / 65       1: 40 / 47, 2: 54 / 48
// Short columns: 18 experts, 1024 x 7168 (28 groups), 8: 17 / 24, 32: 35 / 37, 64:
// 58 / 44; 64 experts, 1024 x 2 x 256 (2 groups), 16: 10 / 12, 32: 15 / 15, 64: 23
// / 17.  Of 212 such points the rule takes the slower kernel by more than 14 % at
// 3: bf16 rows on 18 experts, 7168 x 2 x 1024, 32 rows (34 %), and 8 experts, 4096
// x 2 x 512, 256 rows (fp8 25, bf16 58 %).
inline bool expert_large(int rows, int cols, int groups, int E)
{
    const int64_t w = (int64_t)E * groups;
    if (w >= 512) return rows >= 2 * (int64_t)E;
    if (cols < 2048) return rows >= 32 * (int64_t)E;
    return rows * w >= E * (2 * w + 24 * (512 - w));      // 2 + 24 (512 / w - 1) rows per expert
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
    p.tiles = expert_large(rows, cols, p.groups, E);
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
