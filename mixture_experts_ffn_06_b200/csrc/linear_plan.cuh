// linear_plan.cuh -- which form of the int8 product runs, with its tile, ring and grid:
// host arithmetic alone, from the sizes and the device's SMs.
#pragma once
#include <algorithm>
#include <cstddef>
#include <cstdint>

#include "tmem_share.cuh"

namespace moe {
namespace {

constexpr int kABytes = 128 * 128;  // 128 weight rows x 128 bytes of K
constexpr int kMaxStages = 12;
constexpr int kSmemMax = 227 * 1024;
constexpr int kLinStatic = 4352;  // static shared memory of the tcgen05 forms, at most

inline int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// The tile of the many-token form: the one with the least estimated time, from what
// was measured on B200 for c token columns (c = 64 to 512) in ns.  A k-block takes an
// SM of a pair max(200 + 0.27 c, 90 + 0.86 c) (217 at 64, 255 at 192, 310 at 256) and a
// single CTA max(245 + 0.2 c, 135 + 0.86 c) (258, 300, 355), which loads all of a
// token tile where each CTA of a pair loads half; a pair takes 900 more to start.  A
// tile's epilogue takes about 1000 + 7 c beside the next tile's MMAs, while two
// accumulators fit (c <= 256), and 1500 + 10 c after its own.  T = 512, K = 4096,
// N = 14336: pairs of 256 columns 26.7 us,
// singles 29.9, pairs of 2 x 256 30.4; T = 512, K = 2816, 2 x 2112 gated: singles of 128
// 10.7, pairs 10.9, pairs of 256 13.9.
struct LinTiles {
  int cg, tn, nsub, TT;
  double ns;
};

inline LinTiles plan_tiles(int64_t T, int mt128, int KB, int sms) {
  LinTiles best{1, 0, 0, 0, 0.0};
  for (int cg = 1; cg <= 2; ++cg)
    for (int nsub = 1; nsub <= 2; ++nsub) {
      const int tt0 = ceil_div(T, 256 * nsub);
      for (int tt = tt0; tt <= tt0 + 4; ++tt) {
        const int tn = 16 * cg * ceil_div(ceil_div(T, (int64_t)tt * nsub), 16 * cg);
        const int TT = ceil_div(T, (int64_t)tn * nsub);
        const int64_t rounds = (ceil_div(mt128, cg) * (int64_t)TT + sms / cg - 1) / (sms / cg);
        const double c = (double)tn * nsub;
        const double body = KB * (cg == 1 ? std::max(245.0 + 0.2 * c, 135.0 + 0.86 * c)
                                          : std::max(200.0 + 0.27 * c, 90.0 + 0.86 * c));
        const double epi = nsub == 1 ? 1000.0 + 7.0 * c : 1500.0 + 10.0 * c;
        const double ns = (cg == 2 ? 900.0 : 0.0) +
                          (nsub == 1 ? (rounds - 1) * std::max(body, epi) + body + epi
                                     : rounds * (body + epi));
        if (best.tn == 0 || ns < best.ns) best = LinTiles{cg, tn, nsub, TT, ns};
      }
    }
  return best;
}

struct LinPlan {
  int few;     // warps of a small block (mma.sync); 0: the tcgen05 forms
  int blocks;  // small blocks, or clusters (CTAs where they are single); 0: too many tiles
  int cg, split, ew;
  int tn, nsub, nbuf, stages, panel, KB;
  uint32_t MT, TT, cols;
  size_t smem;  // dynamic; with TMEM at least tmem_smem_least
};

// T tokens, NO output channels, K; at_once(s): clusters of s CTAs that run at once, a
// CTA to an SM.
template <typename F>
LinPlan plan_linear(int64_t T, int NO, int K, bool gated, int sms, F at_once) {
  LinPlan p{};
  const int rows = gated ? 64 : 128;  // output channels of 128 weight rows
  // The small blocks, each of which walks all of K: while K is short, with sixteen warps
  // where at most two blocks come to an SM, which keeps enough loads in flight, else with
  // eight while the blocks are few, or read weights in two places (gated).  In us with
  // sixteen, with eight and on the tcgen05 forms, T = 1: gated 2816 x 4224 4.1, 6.1, 6.1;
  // 4096 x 4096 5.8, 7.4, 6.9; 2048 x 8192 6.5, 5.6, 6.7; 3584 x 10000 12.4, 8.6, 10.1;
  // 4096 x 14336 16.7, 15.7, 13.7; gated 4096 x 14336 15.4, 12.1, 13.8; 8192 x 1024 7.2, 12.2,
  // 5.9.  A second tile of tokens pays for small weights alone, since every block reads all
  // tokens (T = 16, sixteen and tcgen05: gated 2816 x 4224 5.8 and 6.1, 2112 x 2816 4.2
  // and 5.3, 4096 x 14336 20.1 and 12.9).
  // Gated, the last round decides: eight blocks of eight warps are on an SM at once, and three
  // tiles of the tcgen05 form.  With eight warps and on tcgen05, T = 1, gated 4096 x N:
  // N = 18944 (a whole round of blocks) 14.8 and 17.1, 19456 18.5 and 16.1, 21504 19.1 and
  // 17.7, 23040 19.6 and 19.6, 28672 21.5 and 22.8, 37888 (two rounds) 26.8 and 28.5, 40960
  // 30.8 and 29.7, 45056 32.1 and 32.4, 57344 (a little over three rounds and one) 41.9 and
  // 47.6; 2048 x 19456 10.6 and 9.8, x 28672 12.5 and 13.1; 1024 x 19456 6.8 and 6.8.  For longer
  // K tcgen05, but for a short last round of its own: 5120 x 51200 43.8 and 43.9, x 65536 55.3
  // and 60.7; 8192 x 28672 43.0 and 41.4, x 56832 76.3 and 72.7, x 57344 83.3 and 89.4, x 65536
  // 86.0 and 92.1, x 75776 101 and 97.6; 16384 x 57344 157 and 171.
  const int blocks = ceil_div(NO, gated ? 8 : 16);
  const int mt128 = ceil_div(NO, rows);
  const int block_rest = blocks % (8 * sms), tile_rest = mt128 % (3 * sms);
  const bool short_blocks = K >= 2048 && block_rest > 0 && 2 * block_rest <= 3 * sms;
  const bool short_tiles = mt128 > 3 * sms && tile_rest > 0 && 2 * tile_rest <= sms;
  if (K <= 4096 && blocks <= 2 * sms && T <= 16)
    p.few = 16;
  else if (T <= 8 && (gated ? short_tiles || (K <= 4096 && !short_blocks)
                            : K <= 4096 && blocks <= 5 * sms))
    p.few = 8;
  p.blocks = blocks;
  if (p.few) return p;
  p.cg = 1;
  p.KB = ceil_div(K, 128);
  // Tiles of 128 weight rows and up to 128 tokens, K split as far as the clusters all
  // run at once, a CTA to an SM (on B200 15 clusters of eight, 33 of four, 74 of two:
  // not all SMs are in full clusters).  K = 8192, T = 64, in us with 1, 2, 4 and 8 CTAs:
  // 14 tiles 19.1, 12.3, 8.5, 7.4; 16 tiles 19.1, 12.2, 8.6, 13.8; 36 tiles 19.3, 12.6,
  // 18.0, 17.0; 80 tiles 20.2, 18.6, 29.8.  Handing the sums over costs as much as 5 k-blocks
  // and one more for every 18 columns (4 tiles, T = 128, split and not: K = 1024 5.5
  // and 4.6, K = 2048 5.7 and 6.4, K = 8192 7.2 and 16.7).
  const int TT = ceil_div(T, 128), tn = 16 * ceil_div(ceil_div(T, TT), 16);
  const int64_t small = (int64_t)mt128 * TT;
  int split = 1;
  if (small <= sms / 2) {
    split = small <= at_once(8) ? 8 : small <= at_once(4) ? 4 : 2;
    while (split > p.KB) split /= 2;
    if (p.KB * (split - 1.0) / split <= 5.0 + tn / 18.0) split = 1;
  }
  // Unsplit tiles with several CTAs to an SM where there are more of them than SMs
  // (T = 64, K = 2816: 150 tiles 12.4 us, on persistent CTAs 16.6; 300 tiles 22.1 and 24.3),
  // and for the fewest tokens, whose short epilogue needs no sixteen warps (T = 17,
  // K = 2816, 100 tiles: 9.4 and 10.2; T = 64: 10.1 and 9.9; T = 128: 12.0 and 10.4).
  if (split > 1 || (T <= 128 && (mt128 > sms || T <= 32))) {
    p.nsub = 1;
    p.tn = tn;
    p.nbuf = 1;
    p.TT = ceil_div(T, tn);
    p.panel = 1;
    p.MT = mt128;
    p.cols = p.tn <= 32 ? 32 : p.tn <= 64 ? 64 : 128;
    // without a split, all CTAs resident at once where two or three fit an SM
    const int res = split > 1 ? 1 : std::min(3, ceil_div(mt128, sms));
    const int stage = kABytes + tn * 128;
    p.stages = std::min({kMaxStages, (kSmemMax / res - 4 * 1024) / stage, ceil_div(p.KB, split)});
    p.split = split;
    p.ew = split == 1 ? 4 : 8;
    p.blocks = (int)p.MT * p.TT;
    // one 512-byte row of partial sums per column, read in groups of up to 32
    const size_t part = split > 1 ? (size_t)ceil_div(tn, 32) * 32 * 512 : 0;
    p.smem = std::max({1024 + (size_t)p.stages * stage, 1024 + part, tmem_smem_least(p.cols)});
    return p;
  }
  const LinTiles pl = plan_tiles(T, mt128, p.KB, sms);
  p.cg = pl.cg;
  p.split = 1;
  p.ew = 16;
  p.tn = pl.tn;
  p.nsub = pl.nsub;
  p.nbuf = pl.nsub == 1 ? 2 : 1;
  p.TT = pl.TT;
  p.panel = 16;
  p.MT = ceil_div(mt128, pl.cg);
  p.cols = 512;
  const int stage = kABytes + p.tn / pl.cg * 128 * p.nsub;
  p.stages = std::min(kMaxStages, (kSmemMax - 6 * 1024) / stage);
  p.smem = std::max(1024 + (size_t)p.stages * stage, tmem_smem_least(p.cols));
  const int64_t tiles = (int64_t)p.MT * p.TT;
  p.blocks = tiles < (int64_t(1) << 31) ? (int)std::min<int64_t>(sms / p.cg, tiles) : 0;
  return p;
}

}  // namespace
}  // namespace moe
