// How the weight gradient's work is dealt to CTA pairs. Plain C++ where the host
// compiler reads it; the kernels walk the same lists.
#pragma once

#include <algorithm>
#include <cstddef>

#ifdef __CUDACC__
#define GRPO_HD __host__ __device__ __forceinline__
#else
#define GRPO_HD inline
#endif

namespace grpo {

constexpr int kTileM = 256;    // outputs of a pair's tile, 128 per CTA
constexpr int kTileN = 256;    // inputs of a pair's tile
constexpr int kTok = 64;       // tokens of a stage
constexpr int kGroupM = 8;     // tiles are walked 8 row tiles at a time, where not said otherwise
constexpr int kRefPairs = 76;  // GB300's SM pairs

GRPO_HD int least(int a, int b) { return a < b ? a : b; }

// The work of a launch, in stages of kTok tokens. Tiles are dealt whole, one to
// a pair and round, except the last round's `cut` tiles when they fill it
// badly: their stages are dealt evenly, `per_pair` in a row to each pair, and
// a second kernel adds the pieces of a tile in the order of its tokens.
struct WgradPlan {
  int n_m, n_n, kt;
  int whole;     // tiles dealt whole
  int cut;       // tiles dealt in pieces
  int per_pair;  // stages of a pair's part of them
  int group = kGroupM;  // row tiles that are walked together
};

struct WgradItem {
  int tile, kb, ke;
  int slot;  // partial tile to write, -1: the tile itself
};

// 32 bits hold every count: fewer than kRefPairs tiles are cut, of at most 2^24
// stages each.
struct WgradWork {
  int i = 0, pos = -1, end = 0;
  GRPO_HD bool next(const WgradPlan& p, int pair, int pairs, WgradItem& it) {
    if (pos < 0) {
      it.tile = pair + i++ * pairs;
      if (it.tile < p.whole) {
        it.kb = 0;
        it.ke = p.kt;
        it.slot = -1;
        return true;
      }
      const int all = p.cut * p.kt;
      pos = least(pair * p.per_pair, all);
      end = least(pos + p.per_pair, all);
      i = 0;
    }
    if (pos >= end) return false;
    const int t = static_cast<int>(static_cast<unsigned>(pos) / static_cast<unsigned>(p.kt));
    it.tile = p.whole + t;
    it.kb = pos - t * p.kt;
    it.ke = least(p.kt, it.kb + (end - pos));
    it.slot = it.ke - it.kb == p.kt ? -1 : 2 * pair + i;
    ++i;
    pos += it.ke - it.kb;
    return true;
  }
};

// The pairs that hold pieces of cut tile t, first to last (> first: a part is
// shorter than a tile), and the partial tile of pair q's piece: its second one
// begins with the tile; its first one does not, or is the first of its part.
GRPO_HD int first_piece(const WgradPlan& p, int t) { return t * p.kt / p.per_pair; }
GRPO_HD int last_piece(const WgradPlan& p, int t) { return (t * p.kt + p.kt - 1) / p.per_pair; }
GRPO_HD int piece_slot(const WgradPlan& p, int t, int q) {
  return 2 * q + (q * p.per_pair < t * p.kt ? 1 : 0);
}

// Row and column of a tile: column by column within `group` row tiles, so that
// the tiles of a round share both operands in L2.
GRPO_HD void tile_place(const WgradPlan& p, int tile, int& m, int& n) {
  const int per_group = p.group * p.n_n;
  const int g = tile / per_group, r = tile - g * per_group;
  const int rows = least(p.group, p.n_m - g * p.group);
  n = r / rows;
  m = g * p.group + (r - n * rows);
}

// Inputs of a tile: 256, or 128 where no more are left.
GRPO_HD int tile_cols(int in, int n) {
  return in - n * kTileN <= kTileN / 2 ? kTileN / 2 : kTileN;
}

// The plan for `pairs` SM pairs, at most kRefPairs. Its pieces fit the workspace,
// which is sized without a device, for kRefPairs: no tile is cut on fewer pairs
// where none would be on those.
inline WgradPlan make_plan(long long n, int out, int in, int pairs) {
  WgradPlan p;
  p.n_m = (out + kTileM - 1) / kTileM;
  p.n_n = (in + kTileN - 1) / kTileN;
  p.kt = static_cast<int>((n + kTok - 1) / kTok);
  const int tiles = p.n_m * p.n_n;
  p.cut = tiles % pairs;
  // Cut the last round's tiles when that saves at least kMinSaved stages of
  // its length, in pieces of at least kMinPiece.
  constexpr int kMinSaved = 24, kMinPiece = 8;
  p.per_pair = 0;
  if (p.cut > 0) {
    const long long stages = static_cast<long long>(p.cut) * p.kt;
    p.per_pair = static_cast<int>(std::max<long long>(kMinPiece, (stages + pairs - 1) / pairs));
    if (p.kt - p.per_pair < kMinSaved) p.cut = 0;
  }
  if (p.cut > 0 && pairs < kRefPairs && make_plan(n, out, in, kRefPairs).cut == 0) p.cut = 0;
  if (p.cut == 0) p.per_pair = 0;
  p.whole = tiles - p.cut;
  return p;
}

// CTA pairs of the launch. Whole tiles are dealt to `pairs` of them: fewer only
// when one round holds all.
inline int launch_pairs(const WgradPlan& p, int pairs) {
  if (p.whole > pairs) return pairs;
  const long long stages = static_cast<long long>(p.cut) * p.kt;
  const int cut =
      p.per_pair > 0 ? static_cast<int>((stages + p.per_pair - 1) / p.per_pair) : 0;
  return std::max(p.whole, cut);
}

// Partial tiles that the workspace holds.
inline size_t partial_tiles(long long n, int out, int in) {
  return make_plan(n, out, in, kRefPairs).cut > 0 ? 2 * kRefPairs : 0;
}

}  // namespace grpo
