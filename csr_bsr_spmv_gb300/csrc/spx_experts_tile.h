// spx_experts_tile.h -- which tile an experts' product runs on: plain host
// arithmetic, no CUDA.
#pragma once

#include <algorithm>
#include <cstdint>

namespace spx_exp {

constexpr int kDepth = 64;      // reduction length of a stage: one 128-byte swizzle row of 16-bit values
constexpr int kRawDepth = 128;  // kCodes: reduction length of a raw stage, one 128-byte row

enum Kind : int { kProduct, kGradient, kCodes, kGateBack };  // kCodes: 8-bit factors widened on the way; kGateBack: the gate's gradient behind the sums

struct Tile {
    int tn = 0;         // output rows
    int cg = 1;         // CTAs of a tile: 1, or a pair
    int split = 1;      // CTAs that share a tile's reduction
    int split_red = 0;  // length of a share, a multiple of a stage's
};

// The tile (tn rows of 128 or, for a pair, 256 columns) and the CTAs that
// share a tile's reduction, by the least modelled time.  NL: output columns;
// rows: S in all over E experts or, for gradients, NC a gradient; NR: the
// reduction's length (gradients: an expert's rows).  Cycles of a 64-deep
// stage, measured on products of 512 to 16384 rows: small tiles are bound by
// what issuing a stage takes, single CTAs with large ones by the L2 reads of
// their factors, pairs come near the tensor rate.  A tile's stores (12 cycles a
// row) run beside the next tile's MMAs; rounds of tiles count whole.  Sharing a
// reduction costs about 1500 cycles a CTA for the exchange.  512 rows x 4096 x
// 4096: 128-row tiles 19 us, 256-row pairs 25, 64-row tiles 30; 16 rows: one
// CTA a tile 16.5 us, two 13.0, four 11.6, eight 16.1.  The gate's gradient
// takes 70 cycles a row for its stores, which a few tiles do not hide.
inline Tile choose_tile(Kind kind, int E, int S, int NL, int NC, int NR, int sms) {
    const bool wgrad = kind == kGradient, fused = kind == kCodes;
    struct Shape {
        int tn, cg, stage;
    };
    constexpr Shape shapes[] = {{256, 2, 615}, {256, 1, 725}, {128, 2, 435}, {128, 1, 460}, {64, 1, 390}, {32, 1, 350}};
    constexpr Shape codes[] = {{128, 1, 1165}, {64, 1, 985}, {32, 1, 900}};  // measured
    const Shape *from = fused ? codes : shapes, *to = fused ? codes + 3 : shapes + 6;
    const double mean = static_cast<double>(S) / E, used = std::min(E, S);
    double best = 0;
    Shape pick = *from;
    Tile t;
    for (; from != to; ++from) {
        const Shape sh = *from;
        if (wgrad && sh.tn < 128) continue;                    // boxes of 64 columns, two lanes a stage
        if (sh.cg == 2 && NL <= 128) continue;
        const int most = wgrad ? NC : S;
        if (sh.tn > (wgrad ? 128 : 64) && sh.tn / 2 >= most) continue;  // a smaller one holds as much
        const double lanes = (NL + 128 * sh.cg - 1) / (128 * sh.cg);
        // row tiles: an expert's last one is half full on average, unless one holds all its rows
        const double rows = wgrad    ? static_cast<double>(E) * ((NC + sh.tn - 1) / sh.tn)
                            : E == 1 ? (S + sh.tn - 1) / sh.tn
                                     : used * (2 * mean > sh.tn ? mean / sh.tn + 0.5 : 1.0);
        const double tiles = rows * lanes, slots = sms / sh.cg;
        const double stages = wgrad ? mean / kDepth + 0.5 : (NR + kDepth - 1) / kDepth;
        for (int split = 1; split <= 8; split *= 2) {
            if (split > 1 && (wgrad || sh.cg > 1 || sh.tn > 128 || tiles * split > slots)) break;
            const double rounds = tiles * split <= slots ? 1 : tiles / slots < 4 ? static_cast<int>(tiles / slots + 0.99) : tiles / slots;
            double cycles = rounds * (std::max(stages / split * sh.stage, 12.0 * sh.tn) + 600) + (split > 1 ? 1500 * split : 0);
            if (kind == kGateBack) {
                const double sums = stages / split * sh.stage, store = 70.0 * sh.tn / split;
                cycles = rounds * (std::max(sums, store) + 600) + std::min(sums, store) + (split > 1 ? 1500 * split : 0);
            }
            if (best == 0 || cycles < best) best = cycles, pick = sh, t.split = split;
        }
    }
    t.tn = pick.tn;
    t.cg = pick.cg;
    const int unit = fused ? kRawDepth : kDepth;
    t.split_red = ((NR + unit - 1) / unit + t.split - 1) / t.split * unit;
    return t;
}

}  // namespace spx_exp
