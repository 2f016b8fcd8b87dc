// fos_rows.h: rows that come in groups by cumulative end offsets, and the order of
// a wave's own LDS accesses. Shared by the products (fos_linear.hip) and the
// key/value cache (fos_kv.hip, fos_kv_attention.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fos_ops.h"

namespace fos {

// Offsets and lengths out of their range, reported by the first workgroup of a launch. (One condition:
// with the one of y apart, the attention's kernels spill and take 2 to 45 % longer.)
__device__ __forceinline__ void check_kv(const KvCache& c, const int32_t* offs, int T, int32_t* status) {
  if (!status || blockIdx.x != 0 || blockIdx.y != 0) return;
  for (int b = threadIdx.x; b < c.B; b += blockDim.x) {
    const int e = offs[b], p = b ? offs[b - 1] : 0, n = c.lens[b];
    if (e < p || e > T) atomicOr(status, kStatusBadOffs);
    if (n < 0 || n > c.W * c.P) atomicOr(status, kStatusBadCache);
  }
}

// Between LDS accesses of one wave that different lanes make to the same place.
// The hardware runs a wave's LDS operations in order; the compiler, which sees
// one lane at a time, moves no memory access past this, and it is no instruction.
// (A pair of wavefront fences in place of the asm made the forms of 16-bit
// activations spill: 64 x 14336 x 4096 bf16 60 us, 21 with this.)
__device__ __forceinline__ void wave_lds_order() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_wave_barrier();
}

// A tile of a group's rows: the rows [start, end) that the group has, and the
// tile's number among the group's. g < 0: no such tile; g == G: the tail past the
// last group.
struct GroupTile {
  int start, end, g, tile;
  int value;  // the group's, where find_group_tile is given one per group
};

// What a workgroup works on: rows [m0, end) of x with weight g; g < 0: no
// such tile; g == G: the tail past the last group, which is written as zero.
struct RowTile {
  int64_t m0, end;
  int g;
};

// Inclusive sum over the wave's lanes in lane order, by shifts within rows of
// 16 lanes and two broadcasts of a row's last lane.
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_add(int v) {
  return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ int wave_scan(int v) {
  v = dpp_add<0x111, 0xF>(v);  // row_shr:1
  v = dpp_add<0x112, 0xF>(v);
  v = dpp_add<0x114, 0xF>(v);
  v = dpp_add<0x118, 0xF>(v);
  v = dpp_add<0x142, 0xA>(v);  // row_bcast:15, into rows 1 and 3
  return dpp_add<0x143, 0xC>(v);  // row_bcast:31, into rows 2 and 3
}

// Tile `t` of the rows cut into groups and each group into tiles of `rows`
// rows, in group order, the tail last. The wave holds 64 groups' offsets at a
// time, one per lane, and finds the tile by a running sum of the groups' tile
// counts. Offsets are clamped to [previous, M], so a bad one sends no access out
// of bounds. Each row of a group stands for `per` rows of its tiles. M per is at
// most 2^31 - 1 less a tile, so row and tile counts fit an int.
__device__ __forceinline__ GroupTile find_group_tile(const int32_t* offs, int G, int M, int rows, int t, int per,
                                                     const int32_t* values = nullptr) {
  const int lane = threadIdx.x & 63;
  int prev = 0, tiles = 0;  // of the groups before this batch
  for (int base = 0; base <= G; base += 64) {
    const int g = base + lane;
    const bool have = g <= G;
    int end = g < G ? offs[g] : M;
    const int value = values && g < G ? values[g] : 0;
    int start = g == 0 ? 0 : g <= G ? offs[g - 1] : M;
    if (__ballot(have && (start < prev || end < start || end > M))) {
      // offsets that break the contract: running maximum of the clamped ends
      end = end > M ? M : end < prev ? prev : end;
      for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(end, d, 64);
        if (lane >= d && o > end) end = o;
      }
      start = __shfl_up(end, 1, 64);
      if (lane == 0) start = prev;
    }
    const int n = have ? (int)((uint32_t)((end - start) * per + rows - 1) / (uint32_t)rows) : 0;
    const int sum = wave_scan(n);
    const unsigned long long hit = __ballot(tiles + sum > t);
    if (hit) {
      const int l = __ffsll(hit) - 1;
      const int first = tiles + __builtin_amdgcn_readlane(sum - n, l);
      GroupTile r;
      r.start = __builtin_amdgcn_readlane(start, l);
      r.end = __builtin_amdgcn_readlane(end, l);
      r.g = base + l;
      r.tile = t - first;
      r.value = __builtin_amdgcn_readlane(value, l);
      return r;
    }
    tiles += __builtin_amdgcn_readlane(sum, 63);
    prev = __builtin_amdgcn_readlane(end, 63);
  }
  return GroupTile{0, 0, -1, 0, 0};
}

// Tile `t` of the rows of many groups, where each row of a group stands for `per` rows of its tiles of
// 2^ROWS. Group g's tiles start at number (offs[g-1] per >> ROWS) + g: no two groups share a number, every
// tile has one, some numbers have no tile (g < 0), and a number's group is found by search, 64 groups a
// round. There are (M per >> ROWS) + G + 1 numbers. Offsets are clamped, as above; M per is below 2^31.
template <int ROWS>
__device__ __forceinline__ GroupTile search_group_tile(const int32_t* offs, int G, int M, int t, int per, const int32_t* values) {
  const int lane = threadIdx.x & 63;
  GroupTile r{0, M, G, 0, 0};
  int lo = 0, hi = G;  // the group is one of [lo, hi]
  for (;;) {
    const int step = (hi - lo + 63) / 64, g = lo + step * (lane + 1) - 1;
    const bool have = g < G;
    const int start = have && g ? min(max(offs[g - 1], 0), M) : 0, end = have ? min(max(offs[g], 0), M) : M;
    const int value = have ? values[g] : 0;
    const unsigned long long behind = __ballot(g >= hi || (end * per >> ROWS) + g + 1 > t);
    const int l = behind ? __ffsll(behind) - 1 : 64;
    if (step == 1 && lo + l < G && l < 64) {
      r.g = lo + l;
      r.start = __builtin_amdgcn_readlane(start, l);
      r.end = __builtin_amdgcn_readlane(end, l);
      r.value = __builtin_amdgcn_readlane(value, l);
      break;
    }
    lo = min(hi, lo + step * l);
    if (behind) hi = min(hi, lo + step - 1);
    if (lo < hi) continue;
    r.g = lo;
    if (lo > 0) r.start = min(max(offs[lo - 1], 0), M);
    if (lo < G) r.end = min(max(offs[lo], 0), M), r.value = values[lo];
    break;
  }
  r.tile = t - ((r.start * per >> ROWS) + r.g);
  if (r.tile < 0 || ((int64_t)r.tile << ROWS) >= (int64_t)(r.end - r.start) * per) r.g = -1;
  return r;
}

// The first of n ascending ends that lies behind t, n if none does, by a wave: 64 places a round.
__device__ __forceinline__ int first_end_behind(const int32_t* ends, int n, int t) {
  const int lane = threadIdx.x & 63;
  int lo = 0, hi = n;
  while (lo < hi) {
    const int step = (hi - lo + 63) / 64, i = lo + step * (lane + 1) - 1;
    const unsigned long long behind = __ballot(i >= hi || ends[i] > t);
    lo = min(hi, lo + step * (behind ? __ffsll(behind) - 1 : 64));
    if (behind) hi = min(hi, lo + step - 1);
  }
  return lo;
}

__device__ inline RowTile find_tile(const int32_t* offs, int G, int M, int rows, int t) {
  const GroupTile r = find_group_tile(offs, G, M, rows, t, 1);
  return RowTile{(int64_t)r.start + (int64_t)r.tile * rows, r.end, r.g};
}

}  // namespace fos
