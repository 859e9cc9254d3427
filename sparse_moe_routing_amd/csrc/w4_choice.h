// w4_choice.h - which kernel a product with 4-bit weights takes and how it is cut, from its sizes. Host code
// without a device call, so that a test can ask it.
#pragma once

#include <math.h>

namespace moe {

struct W4Sizes {
    int n_rows, E, M, K, group;
    bool grouped;  // rows are the experts' (their counts are on the device)
    bool x_f32, scale_f32, zero, y_f32, swiglu;
};

constexpr int kW4StreamChannels = 32;  // weight channels of a stream wave
constexpr int kW4StreamColumns = 256;  // columns of its slabs
constexpr int kW4StreamBlocks = 8;     // one-wave blocks launched per CU
constexpr int kW4Split = 8;            // waves that split K where there are few units

// The most rows of a block, a multiple of 64: what the registers hold. general: with zero points or fp32 scales.
constexpr int w4_block_rows(bool x_f32, bool general) { return x_f32 ? 128 : general ? 192 : 256; }

// About how many row tiles of `per` rows there will be. The host does not have the experts' counts, so even routing
// is taken. Waves of few rows: `more` of a tile more per expert.
inline double w4_likely_tiles(const W4Sizes &p, int per, double more) {
    if (!p.grouped) return (p.n_rows + per - 1) / per;
    const double experts = p.E < p.n_rows ? p.E : p.n_rows, each = p.n_rows / experts / per;
    return experts * (each + more > 1.0 ? each + more : 1.0);
}
// Blocks: a whole tile of one expert is many units' time, and whether its count passes a multiple of `per` decides
// it. The counts of an even routing scatter by their root: an expert has a tile k + 1 as often as its count
// passes k per. (256 rows an expert, 2048 x 1024 with SwiGLU: nearly all have two tiles of 192 rows, half have two of 256: 531
// and 478 us. With 0.35 of a tile more in place of this 192 rows were chosen.)
inline double w4_block_tiles(const W4Sizes &p, int per) {
    if (!p.grouped) return (p.n_rows + per - 1) / per;
    const double mean = (double)p.n_rows / p.E, scatter = sqrt(mean);
    if (scatter > per) return p.E * (mean / per + 0.5);  // any rest is as likely as any other
    const double sure = floor((mean - 6.0 * scatter) / per);
    double tiles = sure > 0 ? sure + 1.0 : 1.0 - exp(-mean);
    for (int k = sure > 0 ? (int)sure + 1 : 1; k * per < mean + 6.0 * scatter; ++k)
        tiles += 0.5 * erfc((k * per + 0.5 - mean) / (1.41421356 * scatter));
    return p.E * tiles;
}

// Which kernel, and how it is cut, from estimates of all in us, with constants measured on MI355X (dense 4096
// x 4096, groups of 128, one scale; here for 4-, 8- and 16-row waves of bf16 rows). A wave takes 1.1, 1.4 and 1.7 for
// a slab of its stream alone on its CU; a CU takes a wave's slab every 0.21, 0.24 and 0.34. Eight waves
// that split K take 5 and 1.7 to 2.7 for each slab of their eighth, one such block to a CU. A block's slab
// of 64 columns costs 0.9 and 0.4 per 16-row subtile of a wave, its unit 1.5, its start 5. HBM gives 6 TB/s.
// Measured where the choice turns (us; 4-, 8-, 16-row waves, blocks of 64, 128, 192, 256 rows), dense 4096 x 4096: 32 rows
// 27, 16, 12 (all split), 62, 62, 62, 62; 64 rows: 30, 28, 21 (split), 75, 75, 76, 76; 256 rows: 99, 69, 51, 77, 99, 123, 147;
// 512 rows: 191, 128, 91, 77, 100, 123, 149; 2048 rows blocks of 160, 107, 126, 150; 4096 rows 299, 199, 243, 154. 256 experts
// of 2048 x 1024 with SwiGLU, even routing, 1 row an expert: 40, 47, 54, 104; 6 rows: 90, 74, 76, 145; 16 rows: 185,
// 136, 123, 146; 32 rows: 350, 231, 192, 164; 64 rows blocks of 241, 212, 210, 212; 256 rows 707, 528, 528, 478.
struct W4Choice {
    int r, split, tile_rows;  // 4 r rows of a stream wave, split K or not; or r = 0: rows of a block
};
inline W4Choice w4_choose(const W4Sizes &p, int cus) {
    const bool wide = p.x_f32;
    const int Mo = p.swiglu ? p.M / 2 : p.M;
    const double experts = p.grouped ? (p.E < p.n_rows ? p.E : p.n_rows) : 1;
    const double weights = experts * p.M * p.K * (0.5 + (p.scale_f32 ? 4.0 : 2.0) / p.group);
    const double memory = (weights + (double)p.n_rows * (p.K * (wide ? 4.0 : 2.0) + Mo * (p.y_f32 ? 4.0 : 2.0))) / 6e6;
    auto most = [](double a, double b) { return a > b ? a : b; };
    W4Choice c{0, 0, 64};
    double best = 0;
    auto take = [&](double us, const W4Choice &d) {
        if (best == 0 || us < best) best = us, c = d;
    };
    const int cols = p.swiglu ? kW4StreamChannels / 2 : kW4StreamChannels, S = (Mo + cols - 1) / cols, nslab = (p.K + kW4StreamColumns - 1) / kW4StreamColumns;
    static const double kAlone[2][3] = {{1.13, 1.4, 1.7}, {1.9, 2.3, 0.0}}, kEach[2][3] = {{0.21, 0.24, 0.34}, {0.39, 0.45, 0.0}};
    for (int k = 0; k < (wide ? 2 : 3); ++k) {
        const double units = w4_likely_tiles(p, 4 << k, 0.6) * S, alone = kAlone[wide][k], busy = kEach[wide][k] * units / cus;
        take(most(nslab * cbrt(alone * alone * alone + busy * busy * busy), memory) + 2.0, {1 << k, 0, 0});
        const double share = (nslab + kW4Split - 1) / kW4Split;
        if (nslab > 1) take(most(ceil(units / cus) * (5.0 + share * (wide ? 1.5 + 1.0 * k : 1.7 + 0.5 * k)), memory) + 2.0, {1 << k, 1, 0});
    }
    const int bcols = p.swiglu ? 128 : 256, SB = (Mo + bcols - 1) / bcols;
    for (int rows = 64; rows <= w4_block_rows(wide, p.zero || p.scale_f32); rows += 64) {
        const double n = rows / 64, slab = wide ? 0.95 + 0.9 * n : 0.9 + 0.4 * n;
        const double unit = (p.K + 63) / 64 * slab + 1.5;
        take(most(ceil(floor(w4_block_tiles(p, rows) + 0.5) * SB / cus) * unit, memory) + 5.0, {0, 0, rows});
    }
    return c;
}

}  // namespace moe
