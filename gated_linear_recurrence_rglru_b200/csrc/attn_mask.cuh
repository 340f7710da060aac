// Which keys a query sees, and the steps a tile of keys or queries needs
// (include/rglru_attn.h): key j is visible to position p when j <= p and
// (window == 0 or j > p - window or j < sinks).
#pragma once

#include "attn_kernels.h"

namespace rglru {

__host__ __device__ __forceinline__ bool attn_visible(int j, int pos, int window, int sinks) {
  return j <= pos && (window == 0 || j > pos - window || j < sinks);
}

// A query at `pos` that sees one key: its softmax is constant, so its scores get
// no gradient, and none is formed (rounding would leave a few units of one).
__host__ __device__ __forceinline__ bool attn_lone(int pos, int window, int sinks) {
  return pos == 0 || (window == 1 && sinks == 0);
}

// Tokens of batch row b: queries and keys (they differ only without lens).
struct RowLens {
  int nq, nk;
};

__device__ __forceinline__ RowLens row_lens(const AttnArgs &p, int b) {
  RowLens r = {p.T, p.S};
  if (p.lens != nullptr) {
    int n = __ldg(p.lens + b);
    n = n < 0 ? 0 : n > p.T ? p.T : n;
    r.nq = n;
    r.nk = n;
  }
  return r;
}

// Key tiles that queries at positions lo..hi see any key of: tiles
// [0, sink_end) and [win, end), sink_end <= win, in walking order i = 0..n-1.
struct KeyTiles {
  int sink_end, win, n;
  __host__ __device__ int tile(int i) const { return i < sink_end ? i : win + (i - sink_end); }
};

__host__ __device__ __forceinline__ KeyTiles key_tiles(int lo, int hi, int nk, int window,
                                                       int sinks, int tile) {
  KeyTiles k = {0, 0, 0};
  const int last = hi < nk - 1 ? hi : nk - 1;           // last visible key
  if (last < 0) return k;
  const int end = last / tile + 1;
  int first = 0;
  if (window > 0 && lo - window + 1 > 0) first = lo - window + 1;
  k.win = first / tile < end ? first / tile : end;
  if (k.win > 0) {
    const long long s = (static_cast<long long>(sinks) + tile - 1) / tile;
    k.sink_end = static_cast<int>(s < k.win ? s : k.win);
  }
  k.n = k.sink_end + (end - k.win);
  return k;
}

// Queries that see any key of the tile k0 .. k0 + tile - 1: [lo, hi), none when
// lo >= hi. off = S - T.
struct QueryRange {
  int lo, hi;
};

__host__ __device__ __forceinline__ QueryRange query_range(int k0, int tile, int nq, int nk,
                                                           int off, int window, int sinks) {
  QueryRange r = {0, 0};
  if (k0 >= nk) return r;
  r.lo = k0 - off > 0 ? k0 - off : 0;
  r.hi = nq;
  if (window > 0 && k0 >= sinks) {
    const int last = (k0 + tile < nk ? k0 + tile : nk) - 1;
    const long long e = static_cast<long long>(last) + window - off;
    if (e < r.hi) r.hi = static_cast<int>(e > 0 ? e : 0);
  }
  return r;
}

// Block -> place among the pieces of one (batch row, key head).
struct PieceAt {
  int tile, piece;
};

__host__ __device__ __forceinline__ PieceAt piece_at(const PiecePlan &pl, int x) {
  const int ns = pl.n_sink_tiles * pl.sink_pieces;
  if (x < ns) return {x / pl.sink_pieces, x % pl.sink_pieces};
  x -= ns;
  return {pl.n_sink_tiles + x / pl.pieces, x % pl.pieces};
}

__host__ __device__ __forceinline__ int first_slot(const PiecePlan &pl, int tile) {
  return tile < pl.n_sink_tiles
             ? tile * pl.sink_pieces
             : pl.n_sink_tiles * pl.sink_pieces + (tile - pl.n_sink_tiles) * pl.pieces;
}

// Steps of a tile: query tiles [q0, q0 + nq) of each of G heads.
struct Steps {
  int q0, nq, n;
};

__host__ __device__ __forceinline__ Steps steps_of(const QueryRange &r, int step, int G) {
  Steps s = {0, 0, 0};
  if (r.lo >= r.hi) return s;
  s.q0 = r.lo / step;
  s.nq = (r.hi + step - 1) / step - s.q0;
  s.n = s.nq * G;
  return s;
}

// Steps [first, last) of one piece of a tile of n steps, pieces of even length.
struct Piece {
  int first, last;
};

__host__ __device__ __forceinline__ Piece piece_of(const PiecePlan &pl, int n, int piece) {
  const int pieces = n > pl.len ? (n + pl.len - 1) / pl.len : 1;
  const int len = (n + pieces - 1) / pieces;
  const long long first = static_cast<long long>(piece) * len;
  if (first >= n) return {n, n};
  return {static_cast<int>(first), static_cast<int>(first) + (len < n - first ? len : static_cast<int>(n - first))};
}

}  // namespace rglru
