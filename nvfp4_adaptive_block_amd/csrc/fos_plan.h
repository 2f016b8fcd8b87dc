// fos_plan.h: how a product is cut into workgroups, from its sizes alone. Host
// code without the HIP headers, so that a test can compile it and ask which
// kernel a size takes.
#pragma once

#include <stdint.h>

namespace fos {

// The most tiles of `rows` rows that M rows in G groups and a tail can need:
// each non-empty group may end inside a tile.
inline int64_t max_tiles(int64_t M, int64_t G, int64_t rows) {
  const int64_t parts = G + 1 < M ? G + 1 : M;
  return (M + parts * (rows - 1)) / rows;
}

// How a product is cut, from its sizes alone (G = 0: dense).
struct Plan {
  bool stream;      // the stream kernel; else the tile kernel
  int bm;           // rows of a tile
  int splits;       // parts of K
  int64_t m_tiles;  // an upper bound for groups
};

// Column tiles of a stream workgroup: as many as leave the chip nearly full,
// since each reads the activations once (64 x 14336 x 4096: four 21 us, two 25).
inline int stream_columns(int64_t m_tiles, int64_t N) {
  const int64_t n16 = (N + 15) / 16;
  return n16 / 4 * m_tiles >= 224 ? 4 : n16 / 2 * m_tiles >= 224 ? 2 : 1;
}

// Eight waves; sixteen with half the steps in flight where a workgroup has one
// column tile and the chain of a wave's steps is what takes the time.
constexpr int stream_waves(int mt, int nt) { return mt == 1 && nt == 1 ? 16 : 8; }
// 128-deep steps of the weight that a wave has in flight. (More than 32 rows of
// activations leave the registers for one.)
constexpr int stream_depth(int mt, int nt) { return mt >= 3 ? 1 : stream_waves(mt, nt) == 16 ? 2 : 4 / nt; }

// A launch has fewer than 2^32 threads. (The join of parts of K comes nowhere
// near: parts are for at most 768 tiles.)
inline bool fits(const Plan& p, int64_t N) {
  const int nt = p.stream ? stream_columns(p.m_tiles, N) : 16;
  const int64_t threads = p.stream ? 64 * stream_waves(p.bm / 16, nt) : 256;
  return p.m_tiles * p.splits <= UINT32_MAX / threads / ((N + 16 * nt - 1) / (16 * nt));
}

// Estimated microseconds, fitted to what the kernels take on 256 CUs (fp16, N =
// 640 ... 14336, K = 2048 ... 14336); they only have to rank the choices.
//
// Stream kernel, 64 rows: one workgroup per CU at a time; its waves take K / 1024
// steps each. 64 x 4096 x 4096: 11 us (tile kernel at best 19), 256 x 4096 x
// 4096: 21 (25), 1024 x 4096 x 4096: 83 (50).
inline double stream_us(int64_t m_tiles, int64_t N, int64_t K) {
  const int columns = stream_columns(m_tiles, N);
  const int64_t wgs = m_tiles * ((N + 16 * columns - 1) / (16 * columns));
  const double step = columns == 1 ? 1.75 : columns == 2 ? 2.4 : 4.3;
  return 4.0 + (double)((wgs + 255) / 256) * ((double)K / 1024.0) * step;
}

// Tile kernel: a 128-deep step takes 2.15 us with one workgroup of 128 rows on a
// CU and 3.6 with two (64 rows: 1.4 and 2.25); parts of K cost a second launch
// and their sums' way through memory. 2048 x 4096 x 4096: 128 rows 79 us, 64 rows
// 76; 256 x 4096 x 4096 in 64-row tiles: one part 49 us, four 25; 128 x 4096 x
// 14336: one part 154 us, eight 32.
inline double tile_us(double tiles, int64_t M, int64_t N, int64_t K, int bm, int splits) {
  const int n = (int)((tiles * splits + 255.0) / 256.0);
  const double step = bm == 64 ? (n == 1 ? 1.4 : 1.125 * n) : (n == 1 ? 2.15 : 1.8 * n);
  const double steps = (double)((K + 127) / 128) / splits;
  const double join = splits > 1 ? 3.0 + (double)splits * (double)M * (double)N * 8.0 / 8e6 : 0.0;
  return (bm == 64 ? 5.0 : 9.0) + step * steps + join;
}

inline Plan plan(int64_t M, int64_t N, int64_t K, int64_t G) {
  const int64_t rows = G ? (M + G - 1) / G : M;  // rows that share a weight
  auto tiles = [&](int bm) { return G ? max_tiles(M, G, bm) : (M + bm - 1) / bm; };
  const int bm = rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 48 ? 48 : 64;
  Plan best{true, bm, 1, tiles(bm)};
  // few rows: the weights' way from memory is what counts (64 experts of
  // 2048 x 7168: 32 rows each 248 us, 292 with tiles; 64 rows 429 and 353). Both
  // sides were measured with 64 experts only. With fewer, tiles leave the chip
  // idle: 8 experts of 2048 x 7168 take 87 us at 64 bf16 rows each and 77 at 128
  // E4M3 rows, where the weights alone would take 13.
  if (rows <= (G ? 40 : 64)) return best;
  const int64_t n_tiles = (N + 255) / 256;
  double least = G || !fits(best, N) ? 1e30 : stream_us(best.m_tiles, N, K);
  for (int b = 64; b <= 128; b *= 2) {
    // a group ends inside a tile, on average at its middle
    const double t = (G ? (double)M / b + 0.5 * (double)G : (double)tiles(b)) * (double)n_tiles;
    for (int s = 1; s <= (G ? 1 : 8); s++) {
      if (s > 1 && (K / 128 < 2 * s || t * s > 768.0)) break;
      const double us = tile_us(t, M, N, K, b, s);
      if (us < least) {
        least = us;
        best = Plan{false, b, s, tiles(b)};
      }
    }
  }
  return best;
}

}  // namespace fos
