// How a launch of gemm_pair_kernel divides its work: token tiles, CTAs, shared tiles.
#pragma once

#include <cstdint>

#include "gemm_pair.cuh"

namespace w4a16 {

inline int64_t round256(int64_t b) { return (b + 255) / 256 * 256; }

// Launch of the tensor-core kernels (host copy of what the kernel derives its work from).
struct PairPlan {
    int bt;            // tokens of a CTA's tile
    int ctas;          // 1, or 2 for a pair
    int blocks;        // reduction blocks of 64 per tile
    int tiles_m;
    int64_t tiles;
    int split;         // 1: the tiles' units are divided evenly over the CTAs (pairs)
    int grid;          // CTAs (pairs) launched
    int64_t flag_bytes, bytes;   // workspace: ready flags, then parts
};

// Arguments of a launch that follow from its plan.
inline void pair_plan_args(const PairPlan& p, PairArgs* a) {
    a->bt = p.bt;
    a->acc_cols = 32;
    while (a->acc_cols < p.bt * p.ctas) a->acc_cols *= 2;
    a->blocks = p.blocks;
    a->tiles_m = p.tiles_m;
    a->tiles = (int)p.tiles;
    a->split = p.split;
}

// `rows` output rows (features or input channels) in tiles of `rows_per_cta` per CTA.
//
// Token tile: up to 96 tokens are one tile of a CTA each; more are divided evenly into tiles
// of at most 256 for a pair, in steps of 16.
//
// Split: whole tiles in waves leave CTAs idle in the last one.  Dividing all units evenly
// ends that, and costs each CTA writing a part, the tiles' first owners reading those of the
// others one after another, and the sharing of operands in L2 between CTAs that work side by
// side.  Pairs draw the power limit either way, so their waves are left whole from three
// quarters full on (M = 2048, 64 and 344 tiles on 74 pairs: 292 and 274 us whole, 306 and
// 284 us split; 16 tiles: 285 us whole, 101 us split), single CTAs' from nine tenths.  Below
// that the time is estimated for 1, 2, 3, ... sharers of each tile and for all CTAs, and the
// least is taken: a block takes about 0.55 us per 256 tokens and at least 0.5 us, 0.35 us for a
// single CTA (dequantization), a CTA writes or reads a part at about 80 GB/s, and 2 us go to
// the flags (M = 61, K = 11008, N = 4096: 31 us shared, 67 us whole).  It ranks the choices; as a
// time it is low, by the start, the last epilogue and the join's waits (gated, M = 61, N = 11008,
// K = 4096: 17.5 us for 29).
inline PairPlan pair_plan(int64_t M, int64_t rows, int rows_per_cta, int64_t blocks, int unit_blocks, int sm_count) {
    PairPlan p{};
    p.ctas = M > kPairMaxSingle ? 2 : 1;
    const int64_t widest = p.ctas == 2 ? 256 : kPairMaxSingle;
    const int64_t tiles_m = (M + widest - 1) / widest;
    const int64_t tokens = tiles_m > 0 ? ((M + tiles_m - 1) / tiles_m + 15) / 16 * 16 : 16;
    p.bt = (int)(tokens / p.ctas);
    p.tiles_m = (int)tiles_m;
    p.tiles = tiles_m * ((rows + rows_per_cta * p.ctas - 1) / (rows_per_cta * p.ctas));
    p.blocks = (int)blocks;
    const int64_t units = (blocks + unit_blocks - 1) / unit_blocks;
    const int64_t slots = sm_count / p.ctas;
    p.grid = (int)(p.tiles < slots ? p.tiles : slots);
    const int64_t waves = (p.tiles + slots - 1) / slots;
    if (p.ctas == 2 ? 4 * p.tiles < 3 * waves * slots : 10 * p.tiles < 9 * waves * slots) {
        const int64_t part = pair_part_floats((int)tokens) * 4;
        const double part_us = (double)part / 80e3;
        const double least_us = p.ctas == 2 ? 0.5 : 0.35;
        const double block_us = tokens * 0.55 / 256 > least_us ? tokens * 0.55 / 256 : least_us;
        int64_t most = p.tiles * units / 2;            // two units at least for each
        if (most > slots) most = slots;
        int64_t sharers = 0;
        double least = (double)(waves * blocks) * block_us;
        for (int64_t n = 2; waves == 1 && n * p.tiles <= most; ++n) {
            const double us = (double)((units + n - 1) / n * unit_blocks) * block_us + 2.0 + (double)n * part_us;
            if (us < least) least = us, sharers = n * p.tiles;
        }
        if (most >= p.grid) {
            const int64_t reads = (most + p.tiles - 1) / p.tiles;
            const double us = (double)(p.tiles * blocks) * block_us / (double)most + 2.0 + (double)(1 + reads) * part_us;
            if (us < least) least = us, sharers = most;
        }
        if (sharers > 0) {
            p.split = 1;
            p.grid = (int)sharers;
            p.flag_bytes = round256(sharers * p.ctas * kPairMaxWarps * 8);
            p.bytes = p.flag_bytes + sharers * p.ctas * part;
        }
    }
    return p;
}

}  // namespace w4a16
