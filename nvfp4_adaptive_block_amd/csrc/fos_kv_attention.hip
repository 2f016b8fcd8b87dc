// fos_kv_attention.hip: attention over an NVFP4 key/value cache, and the sums of
// its weights per cached key.
//
//   z_rj = scale log2(e) q_r . k_j,  o_r = sum_j 2^(z_rj - m) v_j / sum_j 2^(z_rj - m)
//
// A cached value is c b S with an E2M1 code c, an E4M3 block scale b and the row's
// float32 S_dec. c b has at most 6 significant bits and lies in [2^-10, 2688], so it
// is exact in fp16, which is what the matrix instructions take on both sides:
//  - q in fp16 as it is; in bf16 times a power of two that brings the row's (or the tile's) largest
//    value to [2^15, 2^16), where fp16 still has all 8 bits. They are exact down to 2^-32 of
//    the row's largest, and what is smaller is off by 2^-40 of it (where a tile's rows share a
//    power of two, by 2^-40 of the tile's largest, which is 2^-32 of any row's).
//  - S_dec of a key multiplies the sum, in binary32: with the scale's mantissa first, then with
//    its power of two and what undoes q's, which are exact, so that nothing between leaves
//    binary32's range where the score does not.
//  - S_dec of a value row multiplies the softmax's weight: p_rj = 2^(z_rj - m) S_j is
//    rounded to fp16, and m runs along with the largest z_rj + log2 S_j, kAbove below it,
//    so the largest p of a query lies between 2^8 and 2^15 whatever the rows' sizes are. What is
//    2^-22 of it or more is rounded by at most 2^-11 of its own size, an eighth of what bf16
//    rounds; what is smaller by at most 2^-33 of the largest. (Where no S is 2^-82, p shrinks with
//    them, kLeast being what m goes down to: whole to S of 2^-104, gone at 2^-115.) m only has to be
//    near its maximum: log2 S is taken from the exponent bits, and m follows when it is left behind
//    by more than kLag.
// Sums, m and the softmax's denominator are binary32.
//
// Scores are computed as K Q^T: the matrix instruction leaves a query per lane and
// four neighbouring keys in a lane's registers, which is what the second product
// takes as its right operand (V^T P^T) if the order of the keys along the
// contraction is the same on both sides; no lane exchanges a weight with another.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fos_device.h"
#include "fos_ops.h"
#include "fos_rows.h"

namespace fos {
namespace {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef unsigned short us2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef short s4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) s4* LdsS4;
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr float kLowest = -kFltMax;  // m before any key
constexpr float kLag = 6.0f;
constexpr float kAbove = 8.0f;       // so that p is below 2^(kAbove + kLag + 1), and fp16 ends at 2^16
constexpr float kLeast = -90.0f;     // log2_of rows without a size: 2^96 a key sums up to 2^127
constexpr float kLn2 = 0.69314718055994531f;
constexpr int kMaxParts = 256;

union Frag {
  uint32_t u[4];
  h8 h;
};

__device__ __forceinline__ uint32_t bits(h2 v) { return __builtin_bit_cast(uint32_t, v); }

__device__ __forceinline__ f32x4 mfma16(const Frag& a, const Frag& b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a.h, b.h, c, 0, 0, 0);
}

// Over the four lanes that have the same column (lane % 16).
__device__ __forceinline__ float col_max(float v) {
  auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __builtin_fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
  p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __builtin_fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
}
__device__ __forceinline__ float col_sum(float v) {
  auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}

// Exponent of S (its floor's log2) less kAbove, for the running maximum; kLeast for 0, and for an
// infinity or a NaN, whose exponent is one more than any and so wraps to none.
__device__ __forceinline__ float log2_of(float S) {
  return __builtin_fmaxf((float)(((__float_as_uint(S) << 1) + 0x01000000u) >> 24) - (128.0f + kAbove), kLeast);
}

// Two weights in fp16. For fp16 results what the rounding leaves out is kept too, and
// multiplied in a second product: alone it would cost as much precision as the result's
// own rounding (at most 2^-11 each; measured 2.1e-4 of a result's norm with it, 2.7e-4
// to 3.3e-4 without). A bf16 result's rounding is eight times as large, errors grow by 1 % of
// it (1.61e-3 for 1.60e-3), and the second product would take 28 % of a prompt's time (8192 new
// tokens, 32 heads of 128: 907 us for 709) and 3 to 8 % of a decode step's: left out.
template <int DT>
__device__ __forceinline__ uint32_t round_pair(float a, float b, uint32_t& rest) {
  const f32x2 two = {a, b};
  const h2 near = __builtin_convertvector(two, h2);
  if constexpr (DT == kFP16) {
    const f32x2 left = {a - (float)near.x, b - (float)near.y};
    rest = bits(__builtin_convertvector(left, h2));
  }
  return bits(near);
}

// Eight codes of a dword times a block scale.
__device__ __forceinline__ void decode8(uint32_t codes, h2 s, uint32_t* out) {
  out[0] = bits(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 0) * s);
  out[1] = bits(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 1) * s);
  out[2] = bits(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 2) * s);
  out[3] = bits(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 3) * s);
}

// E4M3 NaN among four block scales: 0x80 in the byte of each; and all bits of such bytes.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t scales) {
  return ((scales & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}
__device__ __forceinline__ uint32_t whole_bytes(uint32_t tops) { return (tops << 1) - (tops >> 7); }

// A quarter of a row of D = 32 NC values: 8 NC neighbouring values, NC dwords of
// codes, and the scales of the blocks that they lie in.
template <int NC> struct Quarter {
  static constexpr int kScales = NC == 1 ? 1 : NC == 3 ? 2 : NC / 2;
  uint32_t codes[NC];
  uint32_t scales;  // kScales bytes

  // the first block of quarter g
  static __device__ __forceinline__ int block(int g) { return (g * NC) >> 1; }
  // the row's blocks, a bit each, that nan_bytes() names in this lane's quarter and in those of
  // the three lanes that have the rest of the row
  static __device__ __forceinline__ uint32_t blocks_of(int g, uint32_t tops) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kScales; i++) m |= ((tops >> (8 * i + 7)) & 1u) << (block(g) + i);
    m |= __shfl_xor(m, 1, 64);
    return m | __shfl_xor(m, 2, 64);
  }

  __device__ __forceinline__ void load_scales(const uint8_t* row, int g) {
    const uint8_t* p = row + block(g);
    scales = 0;
    if constexpr (NC == 4) {
      scales = *reinterpret_cast<const uint16_t*>(p);
    } else if constexpr (NC == 8) {
      scales = *reinterpret_cast<const uint32_t*>(p);
    } else {
#pragma unroll
      for (int i = 0; i < kScales; i++) scales |= (uint32_t)p[i] << (8 * i);
    }
  }
  __device__ __forceinline__ void load_codes(const uint8_t* p) {
    if constexpr (NC % 4 == 0) {
#pragma unroll
      for (int i = 0; i < NC; i += 4) {
        const u32x4 v = reinterpret_cast<const u32x4*>(p)[i / 4];
        codes[i] = v.x, codes[i + 1] = v.y, codes[i + 2] = v.z, codes[i + 3] = v.w;
      }
    } else if constexpr (NC % 2 == 0) {
#pragma unroll
      for (int i = 0; i < NC; i += 2) {
        const u32x2 v = reinterpret_cast<const u32x2*>(p)[i / 2];
        codes[i] = v.x, codes[i + 1] = v.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NC; i++) codes[i] = reinterpret_cast<const uint32_t*>(p)[i];
    }
  }
  __device__ __forceinline__ void store_codes(uint8_t* p) const {
    if constexpr (NC % 4 == 0) {
#pragma unroll
      for (int i = 0; i < NC; i += 4)
        reinterpret_cast<u32x4*>(p)[i / 4] = u32x4{codes[i], codes[i + 1], codes[i + 2], codes[i + 3]};
    } else if constexpr (NC % 2 == 0) {
#pragma unroll
      for (int i = 0; i < NC; i += 2) reinterpret_cast<u32x2*>(p)[i / 2] = u32x2{codes[i], codes[i + 1]};
    } else {
#pragma unroll
      for (int i = 0; i < NC; i++) reinterpret_cast<uint32_t*>(p)[i] = codes[i];
    }
  }
  // fp16 values; f[c] holds values 8c .. 8c + 7 of the quarter g. NUMBERS: a scale that is a NaN
  // becomes a number, and `most` collects the scales' bits, above an infinity's after a NaN (or a
  // negative scale).
  template <bool NUMBERS = false>
  __device__ __forceinline__ void decode(int g, Frag* f, us2* most = nullptr) const {
    h2 s[(kScales + 1) / 2 * 2];
#pragma unroll
    for (int i = 0; i < kScales; i += 2) {
      h2 p = i < 2 ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)scales, 1.0f, false)
                   : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)scales, 1.0f, true);
      if constexpr (NUMBERS) {
        *most = __builtin_elementwise_max(*most, __builtin_bit_cast(us2, p));
        p = __builtin_elementwise_min(p, h2{(_Float16)448.0f, (_Float16)448.0f});
      }
      s[i] = __builtin_shufflevector(p, p, 0, 0);
      s[i + 1] = __builtin_shufflevector(p, p, 1, 1);
    }
#pragma unroll
    for (int c = 0; c < NC; c++) {
      h2 m = s[0];
      if constexpr (NC % 2 == 0) {
        m = s[c / 2];
      } else if constexpr (NC == 3) {
        // an odd quarter starts in the middle of a block
        const int at = ((g * NC + c) >> 1) - block(g);
        m = at ? s[1] : s[0];
      }
      decode8(codes[c], m, f[c].u);
    }
  }
};

// The pages of one sequence and head.
struct Pages {
  const int32_t* table;
  int64_t pages;
  int H, h, P;
  FastDiv by_page;
  // The page of the 16 rows from `pos` on (a multiple of 16, so they are in one); -1 at
  // or past len. Wave-uniform, as are the next two.
  __device__ __forceinline__ int page(int pos, int len) const {
    typedef __attribute__((address_space(4))) const int32_t* Const;
    const int at = ((Const)(const void*)table)[pos < len ? by_page.div(pos) : 0];
    return pos < len ? at : -1;
  }
  // The first of these rows. Where there is no such key (no page, or one that is not the
  // cache's) there = false and the row is the cache's first: without a branch, at which
  // the compiler would wait for all loads.
  __device__ __forceinline__ int64_t row(int page, int pos, bool& there) const {
    there = page >= 0 && page < pages;
    return there ? ((int64_t)page * H + h) * P + (pos - by_page.div(pos) * P) : 0;
  }
};

// What a wave loads of 32 keys, ahead of their use. Codes and the value rows' scales come
// with four lanes to a row, so that the wave's 64 pieces are neighbours in memory, the
// keys' scales as the matrix instruction wants them, and S_dec one to a lane: of the keys
// to the lower half, of the values to the upper.
template <int NC> struct Step {
  Quarter<NC> k[2], v[2];
  float sdec;
  bool there[2];  // wave-uniform: a half's keys, but for those past the end

  __device__ __forceinline__ void load(const KvCache& c, const Pages& pg, const int (&page)[2], int first) {
    const int lane = threadIdx.x & 63, g = lane >> 4;
    int64_t row[2];
#pragma unroll
    for (int u = 0; u < 2; u++) {
      row[u] = pg.row(page[u], first + 16 * u, there[u]);
      k[u].load_codes(c.k.codes + row[u] * (16 * NC) + lane * (4 * NC));
      k[u].load_scales(c.k.scales + row[u] * (2 * NC) + (lane & 15) * (2 * NC), g);
      v[u].load_codes(c.v.codes + row[u] * (16 * NC) + lane * (4 * NC));
      v[u].load_scales(c.v.scales + row[u] * (2 * NC) + (lane >> 2) * (2 * NC), lane & 3);
    }
    sdec = ((lane & 32) ? c.v.sdec : c.k.sdec)[((lane & 16) ? row[1] : row[0]) + (lane & 15)];
  }
};

// 16 x 4 pieces of a wave's LDS, a row's four pieces turned by its quad, so that the
// lanes that an access serves together reach different banks.
__device__ __forceinline__ int piece(int key, int part) { return key * 4 + (part ^ ((4 - (key >> 2)) & 3)); }

// max over the lanes that share a row of q: the four of a column, or its two halves.
template <bool QUARTERS>
__device__ __forceinline__ float row_max(float v) {
  if constexpr (QUARTERS) return col_max(v);
  const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __builtin_fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
}

// One row of q as N fragments of eight values, `step` values apart from `at` on, or zeros
// (at is a row of q in any case).
template <int N>
__device__ __forceinline__ void read_q(const void* q, int64_t at, int step, bool have, Frag* f) {
  const uint16_t* p = (const uint16_t*)q + at;
#pragma unroll
  for (int c = 0; c < N; c++) {
    const u32x4 v = *reinterpret_cast<const u32x4*>(p + c * step);
    f[c].u[0] = have ? v.x : 0, f[c].u[1] = have ? v.y : 0, f[c].u[2] = have ? v.z : 0, f[c].u[3] = have ? v.w : 0;
  }
}

// Biased exponent of a bf16 row's largest finite value.
template <int N, bool QUARTERS>
__device__ __forceinline__ int q_exponent(const Frag* f) {
  uint32_t top = 0;  // of the finite values' bits
#pragma unroll
  for (int c = 0; c < N; c++)
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const uint32_t lo = f[c].u[i] & 0x7FFFu, hi = (f[c].u[i] >> 16) & 0x7FFFu;
      top = max(top, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
    }
  return (int)(__float_as_uint(row_max<QUARTERS>(__uint_as_float(top << 16))) >> 23);
}

// bf16 to fp16, times the power of two that brings exponent e to 2^15; returns what undoes it.
template <int N>
__device__ __forceinline__ float scale_q(Frag* f, int e) {
  int up = 142 - e;
  up = up > 126 ? 126 : up;
  const float by = __uint_as_float((uint32_t)(127 + up) << 23);
#pragma unroll
  for (int c = 0; c < N; c++)
#pragma unroll
    for (int i = 0; i < 4; i++) f[c].u[i] = pack_f16(bf16_lo(f[c].u[i]) * by, bf16_hi(f[c].u[i]) * by);
  return __uint_as_float((uint32_t)(127 - up) << 23);
}

template <int DT, int N, bool QUARTERS>
__device__ __forceinline__ float load_q(const void* q, int64_t at, int step, bool have, Frag* f) {
  read_q<N>(q, at, step, have, f);
  if constexpr (DT == kFP16) return 1.0f;
  return scale_q<N>(f, q_exponent<N, QUARTERS>(f));
}

// Rows of a tile: r counts the sequence's new tokens and, within one, the query
// heads of the cache's head.
struct Row {
  int64_t token;  // of the packed tensor
  int head;       // of all query heads
  int place;      // among the sequence's new tokens
  bool have;
};
__device__ __forceinline__ Row row_of(const KvAttendArgs& a, const GroupTile& gt, int h, int r) {
  Row o;
  o.place = a.by_group.div(r);
  o.head = h * a.G + (r - o.place * a.G);
  o.have = o.place < gt.end - gt.start;
  o.token = (int64_t)gt.start + (o.have ? o.place : 0);
  return o;
}

// A length, cut to what the table holds.
__device__ __forceinline__ int length_of(const KvCache& c, int n) {
  const int cap = c.W * c.P;
  return n < 0 ? 0 : n > cap ? cap : n;
}

// A workgroup's work, from its number: heads of the cache run fastest, so that eight of
// them are on an XCD each, then the parts of the keys, so that a tile that there is not
// leaves no XCD without work.
struct Place {
  int h, part, tile;
};
__device__ __forceinline__ Place place_of(const KvAttendArgs& a) {
  const uint32_t r = blockIdx.x / (uint32_t)a.c.H;
  return Place{(int)(blockIdx.x - r * a.c.H), (int)(r % (uint32_t)a.splits), (int)(r / (uint32_t)a.splits)};
}

// The rows of a tile of 2^ROWS: by the tile's number among those that there are, a pass over all
// sequences, or from 257 on by search, whose numbers have gaps (a token each on 128 keys, 8 heads of
// 128, passes and searches: 256 sequences 29 and 30 us, 1024 124 and 87, 16384 11961 and 1437; 17
// sequences of three tokens, 2999 keys, 12 heads of 64: 20.2 and 20.9).
template <int ROWS>
__device__ __forceinline__ GroupTile find_rows(const KvAttendArgs& a, int tile) {
  return a.c.B <= 256 ? find_group_tile(a.offs, a.c.B, a.T, 1 << ROWS, tile, a.G, a.c.lens)
                      : search_group_tile<ROWS>(a.offs, a.c.B, a.T, tile, a.G, a.c.lens);
}

// ---------------------------------------------------------------- few rows
//
// A workgroup has 16 rows and a part of their keys; its four waves (twelve for a short
// cache that is left whole) take the part's steps of 32 keys in turn, each on its own, and
// join in LDS at the end. Keys come from memory once, a step ahead, to registers; codes of
// keys turn through the wave's own LDS from the loads' order to the matrix instruction's,
// value rows are decoded into it and read back transposed.
//
// A key and its value of D are 9 D / 8 + 8 bytes, from 4 to 16 rows use them, so memory is the
// bound where there is work enough: 64 sequences of 2500 to 8192 tokens, 8 heads of 128, 416 MB
// in 90 to 93 us and a join of 5, 4.3 TB/s. One sequence of 131072 tokens on 4 heads, 80 MB, takes 24 us
// (3.3 TB/s): each of 1024 workgroups has eight steps, and its start and end weigh. Two steps ahead
// lost (17 x 12 heads of 64: 21.5 us for 19.4), and so did branches around the loads. Three waves
// to a SIMD where registers allow it (D up to 128).

template <int NC, int WAVES> struct StreamLds {
  // A value row in fp16. Where it is a multiple of the banks' 256 bytes its pieces of 16
  // are turned by its number, so that the lanes that an access serves together reach
  // different banks; else it is a step of the banks apart from the next.
  static constexpr bool kTurned = NC % 4 == 0;
  static constexpr int kRow = kTurned ? 64 * NC : 64 * NC + 32;
  static __device__ __forceinline__ int value(int row, int piece16) {
    return row * kRow + 16 * (kTurned ? piece16 ^ (5 * (row & 3)) ^ ((row >> 1) & 2) : piece16);
  }
  static constexpr int kKeys = 512 * NC;              // codes of 32 keys
  static constexpr int kSizes = kKeys + 32 * kRow;    // S_dec of 32 keys and of their values
  static constexpr int kWave = kSizes + 256;
  static constexpr int kJoinRow = 32 * NC + 4;        // floats
  static constexpr int kJoin = WAVES * 16 * kJoinRow * 4 + WAVES * 16 * 8;
  static constexpr int kAll = WAVES * kWave > kJoin ? WAVES * kWave : kJoin;
};

template <int DT>
__device__ __forceinline__ void store_out(void* out, int64_t i, const float* v) {  // 8 values
  u32x4 w;
#pragma unroll
  for (int k = 0; k < 4; k++)
    w[k] = DT == kBF16 ? pack_bf16(v[2 * k], v[2 * k + 1]) : pack_f16(v[2 * k], v[2 * k + 1]);
  *reinterpret_cast<u32x4*>((uint16_t*)out + i) = w;
}

template <int DT, int NC, int WAVES>
__global__ __launch_bounds__(64 * WAVES, WAVES > 4 ? 1 : NC <= 4 ? 3 : 2) void k_kv_stream(KvAttendArgs a) {
  typedef StreamLds<NC, WAVES> L;
  __shared__ __attribute__((aligned(16))) uint8_t lds[L::kAll];
  constexpr int D = 32 * NC, DT16 = 2 * NC;  // tiles of 16 values
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, col = lane & 15;
  check_kv(a.c, a.offs, a.T, a.status);
  const Place at_ = place_of(a);
  const int h = at_.h, tile = at_.tile, part = at_.part;
  const GroupTile gt = find_rows<4>(a, tile);
  if (gt.g < 0) return;
  const int n = gt.end - gt.start;
  const int len = length_of(a.c, gt.value);  // of the tail 0
  const Row row = row_of(a, gt, h, gt.tile * 16 + col);
  // keys that this lane's row sees, and what all and any rows of the tile see
  int limit = len, least = len, most = len;
  if (a.causal) {
    const int last = a.by_group.div(gt.tile * 16 + 15);
    limit = max(0, min(len, len - n + row.place + 1));
    least = max(0, min(len, len - n + a.by_group.div(gt.tile * 16) + 1));
    most = max(0, min(len, len - n + last + 1));
  }
  if (!row.have) limit = 0;
  const int steps = (most + 31) / 32;
  const int each = max(WAVES, (steps + a.splits - 1) / a.splits);
  const int from = part * each, to = min(steps, from + each);

  Frag q[NC];
  const float undo = load_q<DT, NC, true>(a.q, row.token * a.stride + (int64_t)row.head * D + g * 8 * NC, 8, row.have, q);
  const float qf = a.scale_pow * undo;
  f32x4 o[DT16];
#pragma unroll
  for (int t = 0; t < DT16; t++) o[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  float m = kLowest, l = 0.0f;
  int nan_blocks = 0;  // of o, a bit each, that a NaN belongs in
  uint8_t* keys = lds + wave * L::kWave;
  uint8_t* vals = keys + L::kKeys;
  float* sizes = reinterpret_cast<float*>(keys + L::kSizes);
  const Pages pg{a.c.table + (int64_t)(gt.g < a.c.B ? gt.g : 0) * a.c.W, a.c.pages, a.c.H, h, a.c.P, a.c.by_page};

  const float size_by = lane < 32 ? a.scale_mant : 1.0f;  // the keys' S_dec have the scale's mantissa
  // pages a step ahead of the loads, loads a step ahead of their use; past the last step
  // the cache's first rows, unused
  Step<NC> next;
  int page[2];
  int s = from + __builtin_amdgcn_readfirstlane(wave);
  auto find = [&](int first) {
#pragma unroll
    for (int u = 0; u < 2; u++) page[u] = pg.page(first + 16 * u, len);
  };
  find(32 * s);
  if (s < to) {
    next.load(a.c, pg, page, 32 * s);
    find(32 * (s + WAVES));
  }
  while (s < to) {
    Step<NC> st = next;
    const int first = 32 * s;
    s += WAVES;
    next.load(a.c, pg, page, 32 * s);
    find(32 * (s + WAVES));

    const bool missing = first + 32 > len || !st.there[0] || !st.there[1];
    const bool edge = first + 32 > least || missing;  // not all rows see all of these keys
    wave_lds_order();
#pragma unroll
    for (int u = 0; u < 2; u++) st.k[u].store_codes(keys + u * 256 * NC + 4 * NC * piece(lane >> 2, lane & 3));
    sizes[lane] = st.sdec * size_by;
    wave_lds_order();
    f32x4 sc[2];
#pragma unroll
    for (int u = 0; u < 2; u++) {
      Quarter<NC> t;
      t.load_codes(keys + u * 256 * NC + 4 * NC * piece(col, g));
      t.scales = st.k[u].scales;
      Frag kf[NC];
      t.decode(g, kf);
      sc[u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int c = 0; c < NC; c++) sc[u] = mfma16(kf[c], q[c], sc[u]);
    }
    // Value rows to fp16, zero where there is no key: a stale scale may be a NaN. A NaN in a row
    // that is there reaches the queries that see it by itself, and here no others: 0 times it is
    // a NaN too.
    if (edge) {
#pragma unroll
      for (int u = 0; u < 2; u++) {
        uint32_t& scales = st.v[u].scales;
        if (!st.there[u] || first + 16 * u + (lane >> 2) >= len) scales = 0;
        const uint32_t nans = nan_bytes(scales);
        if (!__any(nans != 0)) continue;
        scales &= ~whole_bytes(nans);
        const int rows = (int)Quarter<NC>::blocks_of(lane & 3, nans);
#pragma unroll 1
        for (int r = 0; r < 16; r++) {
          const int of_row = __builtin_amdgcn_readlane(rows, 4 * r);
          nan_blocks |= first + 16 * u + r < limit ? of_row : 0;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < 2; u++) {
      Frag vf[NC];
      st.v[u].decode(lane & 3, vf);
#pragma unroll
      for (int c = 0; c < NC; c++)
        *reinterpret_cast<u32x4*>(vals + L::value(16 * u + (lane >> 2), (lane & 3) * NC + c)) =
            u32x4{vf[c].u[0], vf[c].u[1], vf[c].u[2], vf[c].u[3]};
    }
    // scores to weights
    float z[8], top = kLowest;
    f32x4 vs[2];
#pragma unroll
    for (int u = 0; u < 2; u++) {
      const f32x4 ks = *reinterpret_cast<const f32x4*>(sizes + 16 * u + 4 * g);
      vs[u] = *reinterpret_cast<const f32x4*>(sizes + 32 + 16 * u + 4 * g);
#pragma unroll
      for (int i = 0; i < 4; i++) z[4 * u + i] = sc[u][i] * (ks[i] * qf);
    }
    if (edge) {
#pragma unroll
      for (int u = 0; u < 2; u++)
#pragma unroll
        for (int i = 0; i < 4; i++)
          if (!st.there[u] || first + 16 * u + 4 * g + i >= limit) {
            z[4 * u + i] = -__builtin_huge_valf();
            vs[u][i] = 0.0f;  // which may be a stale NaN
          }
    }
#pragma unroll
    for (int u = 0; u < 2; u++)
#pragma unroll
      for (int i = 0; i < 4; i++) top = __builtin_fmaxf(top, z[4 * u + i] + log2_of(vs[u][i]));
    top = col_max(top);
    if (__any(top > m + kLag)) {
      const float now = __builtin_fmaxf(m, top);
      const float f = __builtin_amdgcn_exp2f(m - now);
      m = now;
      l *= f;
#pragma unroll
      for (int t = 0; t < DT16; t++) o[t] *= f;
    }
    Frag p, rest;
    float w[8], sum = 0.0f;  // of the step's weights first: small ones are not lost beside l one by one
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const float e = __builtin_amdgcn_exp2f(z[i] - m);
      sum += e;
      w[i] = e * vs[i / 4][i % 4];
    }
    l += sum;
#pragma unroll
    for (int i = 0; i < 4; i++) p.u[i] = round_pair<DT>(w[2 * i], w[2 * i + 1], rest.u[i]);
    wave_lds_order();
#pragma unroll
    for (int t = 0; t < DT16; t++) {
      Frag v;
#pragma unroll
      for (int u = 0; u < 2; u++) {
        const uint8_t* at = vals + L::value(16 * u + 4 * g + (col >> 2), 2 * t + ((col >> 1) & 1)) + 8 * (col & 1);
        const u32x2 y = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsS4)at));
        v.u[2 * u] = y.x;
        v.u[2 * u + 1] = y.y;
      }
      o[t] = mfma16(v, p, o[t]);
      if constexpr (DT == kFP16) o[t] = mfma16(v, rest, o[t]);
    }
  }

  if (__any(nan_blocks != 0)) {
#pragma unroll
    for (int t = 0; t < DT16; t++)
      if ((nan_blocks >> t) & 1) o[t] += __builtin_nanf("");
  }
  // join the waves
  l = col_sum(l);
  __syncthreads();
  float* join = reinterpret_cast<float*>(lds);
  float2* ml = reinterpret_cast<float2*>(lds + WAVES * 16 * L::kJoinRow * 4);
  if (g == 0) ml[wave * 16 + col] = float2{m, l};
#pragma unroll
  for (int t = 0; t < DT16; t++)
    *reinterpret_cast<f32x4*>(join + (wave * 16 + col) * L::kJoinRow + 16 * t + 4 * g) = o[t];
  __syncthreads();
  constexpr int kEach = 4 * WAVES;  // threads to a row
  const int r = threadIdx.x / kEach, piece0 = threadIdx.x % kEach;
  const Row to_row = row_of(a, gt, h, gt.tile * 16 + r);
  if (!to_row.have) return;
  float M = kLowest, sum = 0.0f, f[WAVES];
#pragma unroll
  for (int w = 0; w < WAVES; w++) M = __builtin_fmaxf(M, ml[w * 16 + r].x);
#pragma unroll
  for (int w = 0; w < WAVES; w++) {
    f[w] = __builtin_amdgcn_exp2f(ml[w * 16 + r].x - M);
    sum += f[w] * ml[w * 16 + r].y;
  }
  const int64_t at = to_row.token * ((int64_t)a.c.H * a.G) + to_row.head;
  const bool whole = a.splits == 1;
  const float by = whole ? (sum == 0.0f ? 0.0f : 1.0f / sum) : 1.0f;
  for (int d = piece0 * 8; d < D; d += 8 * kEach) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; w++) {
      const f32x4* p = reinterpret_cast<const f32x4*>(join + (w * 16 + r) * L::kJoinRow + d);
#pragma unroll
      for (int i = 0; i < 8; i++) v[i] += f[w] * p[i / 4][i % 4];
    }
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] *= by;
    if (whole) {
      store_out<DT>(a.out, at * D + d, v);
    } else {
      float* po = (float*)a.work + (at * a.splits + part) * D + d;
      *reinterpret_cast<f32x4*>(po) = f32x4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4*>(po + 4) = f32x4{v[4], v[5], v[6], v[7]};
    }
  }
  if (piece0 == 0) {
    if (whole) {
      if (a.lse) a.lse[at] = sum == 0.0f ? -__builtin_huge_valf() : (M + __log2f(sum)) * kLn2;
    } else {
      float2* pm = reinterpret_cast<float2*>((float*)a.work + (int64_t)a.T * a.c.H * a.G * a.splits * D);
      pm[at * a.splits + part] = float2{M, sum};
    }
  }
}

// ---------------------------------------------------------------- many rows
//
// A workgroup has 128 rows, 32 of them to a wave, and walks over their keys 64 at a
// time. A wave decodes 16 of the 64 keys' rows to fp16 into LDS, one step ahead of their
// use and with the codes of the step after that on their way, and all four waves read
// them: keys as rows, values transposed.
//
// 4 D operations for each row and key are the bound, but the vector units' part (decode, scale,
// maximum, exponential, conversion) nearly fills the time beside them: 8192 new tokens, 32 query
// heads of 128, 0.555 TFLOP in 690 to 735 us from card to card, 755 to 805 TFLOP/s; matrix units
// busy 35 % of the cycles, vector units 56 %. Decode goes beside the first product and exponentials beside the
// second, which the scheduler is told. Two workgroups to a CU for D 96 and 128 (three of 32 keys:
// 730 us for 695 then; bounded to three with spills: 947). Not kept: the next step's first product beside this
// one's softmax (816 us), a wave's priority raised in its products (738 for 722 then), raw codes
// two steps ahead. D 256 fills 256 registers and spills 59, one workgroup to a CU: 540 TFLOP/s.

template <int NC> struct TileLds {
  static constexpr int kKeys = 64;
  // A key's row, in bytes: sixteen neighbouring rows' pieces of 16 bytes are in different
  // banks. A value's: where it is a multiple of the banks' 256 bytes, its pieces of 16 are
  // turned by 5 (row % 4), so that both four rows' pieces of 64 bytes (the transposed
  // reads) and sixteen lanes' pieces of 16 (the writes) are.
  static constexpr bool kTurned = NC % 4 == 0;
  static constexpr int kK = 64 * NC + 16, kV = kTurned || 64 * NC % 128 ? 64 * NC : 64 * NC + 64;
  static constexpr int kSide = kKeys * (kK + kV);
  static constexpr int kOut = 32 * (64 * NC + 16);  // a wave's rows of the result
  static constexpr int kAll = 2 * kSide > 4 * kOut ? 2 * kSide : 4 * kOut;
  static __device__ __forceinline__ int value(int row, int piece16) {
    return row * kV + 16 * (kTurned ? piece16 ^ (5 * (row & 3)) : piece16);
  }
};

// Sixteen rows of either side, by one wave.
template <int NC> struct TileStep {
  Quarter<NC> k, v;
  float sdec;  // lanes 0-15 (of each half): of the keys, 16-31: of the values
  bool there;  // wave-uniform
  __device__ __forceinline__ void load(const KvCache& c, const Pages& pg, int page, int first) {
    const int lane = threadIdx.x & 63;
    const int64_t row = pg.row(page, first, there);
    k.load_codes(c.k.codes + row * (16 * NC) + lane * (4 * NC));
    k.load_scales(c.k.scales + row * (2 * NC) + (lane >> 2) * (2 * NC), lane & 3);
    v.load_codes(c.v.codes + row * (16 * NC) + lane * (4 * NC));
    v.load_scales(c.v.scales + row * (2 * NC) + (lane >> 2) * (2 * NC), lane & 3);
    sdec = ((lane & 16) ? c.v.sdec : c.k.sdec)[row + (lane & 15)];
  }
};

// The order that the scheduler is asked for: `n` times a matrix instruction, `valu` others
// and `reads` of LDS.
#define FOS_INTERLEAVE(n, valu, reads)                      \
  _Pragma("unroll") for (int i_ = 0; i_ < (n); i_++) {      \
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);      \
    __builtin_amdgcn_sched_group_barrier(0x002, valu, 0);   \
    __builtin_amdgcn_sched_group_barrier(0x100, reads, 0);  \
  }

template <int DT, int NC>
__global__ __launch_bounds__(256, NC <= 2 ? 3 : NC <= 4 ? 2 : 1) void k_kv_tile(KvAttendArgs a) {
  typedef TileLds<NC> L;
  constexpr int D = 32 * NC;
  __shared__ __attribute__((aligned(16))) uint8_t lds[L::kAll];
  // Per step: S_dec of keys times the scale, of values, its log2, each of 64 keys; which
  // sixteens are not there; and places that the other lanes write to.
  constexpr int kValues = L::kKeys, kLog2 = 2 * L::kKeys, kGone = 3 * L::kKeys, kNowhere = 3 * L::kKeys + 4;
  __shared__ __attribute__((aligned(16))) float sizes[2][3 * L::kKeys + 8];
  __shared__ __attribute__((aligned(16))) float ones[L::kKeys];
  __shared__ int ends[8];  // largest and least exponent of a wave's rows of q
  __shared__ int found[4];  // whether a wave's value rows had a NaN
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = lane >> 5, col = lane & 31;
  check_kv(a.c, a.offs, a.T, a.status);
  // the last tiles of a sequence see the most keys: they start first
  const Place at_ = place_of(a);
  const int h = at_.h, tile = (int)gridDim.x / (a.c.H * a.splits) - 1 - at_.tile, part = at_.part;
  const GroupTile gt = find_rows<7>(a, tile);
  if (gt.g < 0) return;
  const int n = gt.end - gt.start;
  const int len = length_of(a.c, gt.value);  // of the tail 0
  const int r0 = gt.tile * 128 + wave * 32;
  const Row row = row_of(a, gt, h, r0 + col);
  // keys that this lane's row sees; that all and any rows of the wave, and any of the workgroup, see
  int limit = len, least = len, most = len, all = len;
  if (a.causal) {
    limit = max(0, min(len, len - n + row.place + 1));
    least = max(0, min(len, len - n + a.by_group.div(r0) + 1));
    most = max(0, min(len, len - n + a.by_group.div(r0 + 31) + 1));
    all = max(0, min(len, len - n + a.by_group.div(gt.tile * 128 + 127) + 1));
  }
  if (!row.have) limit = 0;
  const int steps = (all + L::kKeys - 1) / L::kKeys;
  const int each = max(4, (steps + a.splits - 1) / a.splits);
  const int from = part * each, to = min(steps, from + each);

  Frag q[2 * NC];
  read_q<2 * NC>(a.q, row.token * a.stride + (int64_t)row.head * D + 8 * half, 16, row.have, q);
  if (threadIdx.x < L::kKeys) ones[threadIdx.x] = 1.0f;
  // bf16 rows of about one size have one power of two, which then goes with the keys' sizes: a
  // multiplication less for each score (8192 new tokens, 32 heads of 128: 713 us for 806, of 64 451
  // for 526). The smallest row's values are then good to 2^-32 of its largest, and sizes grow no larger.
  bool common = true;
  float undo = 1.0f, undo_all = 1.0f;
  if constexpr (DT == kBF16) {
    int e = q_exponent<2 * NC, false>(q);
    int hi = e, lo = e ? e : 255;
    for (int d = 1; d < 32; d <<= 1) {
      hi = max(hi, __shfl_xor(hi, d, 64));
      lo = min(lo, __shfl_xor(lo, d, 64));
    }
    if (lane == 0) ends[wave] = hi, ends[4 + wave] = lo;
    __syncthreads();
    hi = max(max(ends[0], ends[1]), max(ends[2], ends[3]));
    lo = min(min(ends[4], ends[5]), min(ends[6], ends[7]));
    common = __builtin_amdgcn_readfirstlane(hi - lo <= 8 && hi <= 141 && hi >= 77);
    undo = scale_q<2 * NC>(q, common ? hi : e);
  }
  undo *= a.scale_pow;
  if (common) undo_all = undo, undo = 1.0f;
  f32x16 o[NC];
#pragma unroll
  for (int t = 0; t < NC; t++)
#pragma unroll
    for (int i = 0; i < 16; i++) o[t][i] = 0.0f;
  float m = kLowest, l = 0.0f;
  const Pages pg{a.c.table + (int64_t)(gt.g < a.c.B ? gt.g : 0) * a.c.W, a.c.pages, a.c.H, h, a.c.P, a.c.by_page};

  TileStep<NC> st;
  // of this wave's value rows: the scales' bits, and the lanes whose S_dec was no number or infinite
  us2 scale_bits = {0, 0};
  unsigned long long odd_sizes = 0;
  int page = 0;  // of this wave's rows of the step that is loaded next
  const int my_key = 16 * wave + (lane >> 2), my_size = 16 * wave + (lane & 15);
  const int to_size = lane < 16 ? my_size : lane < 32 ? kValues + my_size : kNowhere;
  const int to_log2 = lane >= 16 && lane < 32 ? kLog2 + my_size : kNowhere + 1;
  const int to_gone = lane == 0 ? kGone + wave : kNowhere + 2;
  // the keys' scale goes with their S_dec, so that what is left for a query is its power of two
  const float size_by = lane < 16 ? a.scale_mant : 1.0f, size_undo = lane < 16 ? undo_all : 1.0f;
  // This wave's rows of a step, decoded, to the step's side of the LDS, without a branch, so that
  // it can run beside matrix instructions. Zeros where there is no key: a stale scale may be a NaN.
  // One in a value row that is there must reach the queries that see it and no others, but 0 times
  // it is a NaN too: it becomes a number here, and is seen to after the last step. (8192 new tokens,
  // 32 heads: 698 us for 692 without this at D 128, 2038 for 2026 at D 256; by a branch in the loop
  // for steps with masked keys 699 and 2560.)
  auto put = [&](int step) {
    const int side = step & 1, first = step * L::kKeys;
    if (!st.there || first + my_key >= len) st.k.scales = st.v.scales = 0;
    Frag f[NC];
    uint8_t* base = lds + side * L::kSide;
    st.k.decode(lane & 3, f);
#pragma unroll
    for (int c = 0; c < NC; c++)
      *reinterpret_cast<u32x4*>(base + my_key * L::kK + 16 * ((lane & 3) * NC + c)) =
          u32x4{f[c].u[0], f[c].u[1], f[c].u[2], f[c].u[3]};
    st.v.template decode<true>(lane & 3, f, &scale_bits);
#pragma unroll
    for (int c = 0; c < NC; c++)
      *reinterpret_cast<u32x4*>(base + L::kKeys * L::kK + L::value(my_key, (lane & 3) * NC + c)) =
          u32x4{f[c].u[0], f[c].u[1], f[c].u[2], f[c].u[3]};
    float S = !st.there || first + my_size >= len ? 0.0f : st.sdec;
    const bool odd = (lane & 16) && !(__builtin_fabsf(S) < __builtin_huge_valf());
    odd_sizes |= __ballot(odd);
    S = odd ? 0.0f : S;
    sizes[side][to_size] = S * size_by * size_undo;
    sizes[side][to_log2] = log2_of(S);
    sizes[side][to_gone] = st.there ? 0.0f : 1.0f;
  };
  auto load = [&](int step) {  // past the last step: the cache's first rows, which put() makes zeros
    const int first = step * L::kKeys + 16 * wave;
    st.load(a.c, pg, page, first);
    page = pg.page(first + L::kKeys, len);
  };

  if (from < to) {
    page = pg.page(from * L::kKeys + 16 * wave, len);
    load(from);
    put(from);
    load(from + 1);
  }
  __syncthreads();
  for (int s = from; s < to; s++) {
    const int side = s & 1, first = s * L::kKeys;
    const float* size = sizes[side];
    if (first < most) {
      const uint8_t* kp = lds + side * L::kSide + col * L::kK + 16 * half;
      f32x16 x[2];
      Frag kf[2][2 * NC];
      const f32x4 absent = *reinterpret_cast<const f32x4*>(size + kGone);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int kb = 0; kb < 2; kb++)
#pragma unroll
        for (int c = 0; c < 2 * NC; c++) {
          const u32x4 t = *reinterpret_cast<const u32x4*>(kp + 32 * kb * L::kK + 32 * c);
          kf[kb][c].u[0] = t.x, kf[kb][c].u[1] = t.y, kf[kb][c].u[2] = t.z, kf[kb][c].u[3] = t.w;
        }
#pragma unroll
      for (int kb = 0; kb < 2; kb++) {
#pragma unroll
        for (int i = 0; i < 16; i++) x[kb][i] = 0.0f;
#pragma unroll
        for (int c = 0; c < 2 * NC; c++)
          x[kb] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf[kb][c].h, q[c].h, x[kb], 0, 0, 0);
      }
      put(s + 1);
      __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
      FOS_INTERLEAVE(4 * NC - 4, 5, 1)
      FOS_INTERLEAVE(4, 5, 0)
      __builtin_amdgcn_sched_barrier(0);
      load(s + 2);
      // a lane's sixteen keys of 32: 8b + 4 half + 0..3. What they are multiplied by below: the
      // keys' sizes, or where a key is not seen or rows differ much, ones, after the sizes here
      const bool edge = first + L::kKeys > least || __builtin_amdgcn_readfirstlane(__float_as_int(absent[0] + absent[1] + absent[2] + absent[3]));
      const float* by = size;
      if (edge || !common) {
        by = ones;
#pragma unroll
        for (int kb = 0; kb < 2; kb++)
#pragma unroll
          for (int b = 0; b < 4; b++) {
            const f32x4 ks = *reinterpret_cast<const f32x4*>(size + 32 * kb + 8 * b + 4 * half);
            const int j = 32 * kb + 8 * b;
            const int past = absent[j >> 4] != 0.0f ? 0 : limit - first - j - 4 * half;  // keys from here on are not seen
#pragma unroll
            for (int i = 0; i < 4; i++)
              x[kb][4 * b + i] = i < past ? x[kb][4 * b + i] * (ks[i] * undo) : -__builtin_huge_valf();
          }
      }
      auto size_of = [&](int kb, int b) { return *reinterpret_cast<const f32x4*>(by + 32 * kb + 8 * b + 4 * half); };
      float top = kLowest;
#pragma unroll
      for (int kb = 0; kb < 2; kb++)
#pragma unroll
        for (int b = 0; b < 4; b++) {
          const f32x4 lv = *reinterpret_cast<const f32x4*>(size + kLog2 + 32 * kb + 8 * b + 4 * half), ks = size_of(kb, b);
#pragma unroll
          for (int i = 0; i < 4; i++) top = __builtin_fmaxf(top, __builtin_fmaf(x[kb][4 * b + i], ks[i], lv[i]));
        }
      top = row_max<false>(top);
      if (__any(top > m + kLag)) {
        const float now = __builtin_fmaxf(m, top);
        const float f = __builtin_amdgcn_exp2f(m - now);
        m = now;
        l *= f;
#pragma unroll
        for (int t = 0; t < NC; t++)
#pragma unroll
          for (int i = 0; i < 16; i++) o[t][i] *= f;
      }
      // a sixteen of lanes reads four keys' rows, 16 values of each: which four, which half of 32 values
      const int i16 = lane & 15;
      const uint8_t* vp = lds + side * L::kSide + L::kKeys * L::kK + 8 * (i16 & 1);
      Frag vf[4][NC], p[4], rest[4];
      auto read_values = [&](int c) {
#pragma unroll
        for (int t = 0; t < NC; t++)
#pragma unroll
          for (int u = 0; u < 2; u++) {
            const int key = 16 * c + 8 * u + 4 * half + (i16 >> 2), at = 4 * t + 2 * ((lane >> 4) & 1) + ((i16 >> 1) & 1);
            const u32x2 y = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsS4)(vp + L::value(key, at))));
            vf[c][t].u[2 * u] = y.x;
            vf[c][t].u[2 * u + 1] = y.y;
          }
      };
      float sum = 0.0f;  // of the step's weights first: small ones are not lost beside l one by one
      auto weigh = [&](int kb) {
#pragma unroll
        for (int b = 0; b < 4; b++) {
          const f32x4 vs = *reinterpret_cast<const f32x4*>(size + kValues + 32 * kb + 8 * b + 4 * half), ks = size_of(kb, b);
          float w[4];
#pragma unroll
          for (int i = 0; i < 4; i++) {
            const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(x[kb][4 * b + i], ks[i], -m));
            sum += e;
            w[i] = e * vs[i];
          }
#pragma unroll
          for (int i = 0; i < 2; i++)
            p[2 * kb + (b >> 1)].u[2 * (b & 1) + i] =
                round_pair<DT>(w[2 * i], w[2 * i + 1], rest[2 * kb + (b >> 1)].u[2 * (b & 1) + i]);
        }
      };
      auto add = [&](int c) {
#pragma unroll
        for (int t = 0; t < NC; t++) {
          o[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf[c][t].h, p[c].h, o[t], 0, 0, 0);
          if constexpr (DT == kFP16) o[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf[c][t].h, rest[c].h, o[t], 0, 0, 0);
        }
      };
      read_values(0);
      __builtin_amdgcn_sched_barrier(0);
      weigh(0);
      read_values(1);
      __builtin_amdgcn_sched_barrier(0);
      add(0);
      add(1);
      weigh(1);
      l += sum;
      read_values(2);
      FOS_INTERLEAVE(2 * NC, 72 / (2 * NC), 2)
      __builtin_amdgcn_sched_barrier(0);
      read_values(3);
      add(2);
      add(3);
    } else {
      put(s + 1);
      load(s + 2);
    }
    __syncthreads();
  }

  // NaN where a row sees one: the value rows' scales and sizes once more, by every wave
  const int any = odd_sizes || __any(max(scale_bits.x, scale_bits.y) > 0x7C00);
  if (lane == 0) found[wave] = any;
  __syncthreads();
  if (found[0] | found[1] | found[2] | found[3]) {
    int blocks = 0;  // of the row's result, a bit each
#pragma unroll 1
    for (int first = from * L::kKeys; first < min(to * L::kKeys, most); first += 16) {
      bool there;
      const int64_t at = pg.row(pg.page(first, len), first, there);
      if (!there) continue;
      Quarter<NC> v;
      v.load_scales(a.c.v.scales + (at + (lane >> 2)) * (2 * NC), lane & 3);
      uint32_t tops = nan_bytes(v.scales);
      if (!(__builtin_fabsf(a.c.v.sdec[at + (lane >> 2)]) < __builtin_huge_valf())) tops = 0x80808080u;
      const int of_lane = (int)Quarter<NC>::blocks_of(lane & 3, tops);
#pragma unroll 1
      for (int r = 0; r < 16; r++) {
        const int of_row = __builtin_amdgcn_readlane(of_lane, 4 * r);
        blocks |= first + r < limit ? of_row : 0;
      }
    }
#pragma unroll
    for (int t = 0; t < NC; t++)
#pragma unroll
      for (int i = 0; i < 16; i++)
        if ((blocks >> (2 * t + (i >> 3))) & 1) o[t][i] += __builtin_nanf("");
  }
  const auto both = __builtin_amdgcn_permlane32_swap(__float_as_uint(l), __float_as_uint(l), false, false);
  l = __uint_as_float(both[0]) + __uint_as_float(both[1]);
  const int64_t at = row.token * ((int64_t)a.c.H * a.G) + row.head;
  if (a.splits > 1) {
    if (!row.have) return;
    float* po = (float*)a.work + (at * a.splits + part) * D + 4 * half;
#pragma unroll
    for (int t = 0; t < NC; t++)
#pragma unroll
      for (int b = 0; b < 4; b++)
        *reinterpret_cast<f32x4*>(po + 32 * t + 8 * b) = f32x4{o[t][4 * b], o[t][4 * b + 1], o[t][4 * b + 2], o[t][4 * b + 3]};
    if (half == 0) {
      float2* pm = reinterpret_cast<float2*>((float*)a.work + (int64_t)a.T * a.c.H * a.G * a.splits * D);
      pm[at * a.splits + part] = float2{m, l};
    }
    return;
  }
  // the result's rows turn through the wave's own LDS to whole pieces of 16 bytes
  const float by = l == 0.0f ? 0.0f : 1.0f / l;
  constexpr int kRow = 64 * NC + 16;
  uint8_t* turned = lds + wave * L::kOut;
#pragma unroll
  for (int t = 0; t < NC; t++)
#pragma unroll
    for (int b = 0; b < 4; b++) {
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; i++) v[i] = o[t][4 * b + i] * by;
      const u32x2 w = DT == kBF16 ? u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])}
                                  : u32x2{pack_f16(v[0], v[1]), pack_f16(v[2], v[3])};
      *reinterpret_cast<u32x2*>(turned + col * kRow + 64 * t + 16 * b + 8 * half) = w;
    }
  wave_lds_order();
#pragma unroll
  for (int i = 0; i < 2 * NC; i++) {
    const int e = i * 64 + lane, r = e / (4 * NC), piece16 = e % (4 * NC);
    const Row to_row = row_of(a, gt, h, r0 + r);
    if (to_row.have)
      *reinterpret_cast<u32x4*>((uint16_t*)a.out + (to_row.token * ((int64_t)a.c.H * a.G) + to_row.head) * D + 8 * piece16) =
          *reinterpret_cast<const u32x4*>(turned + r * kRow + 16 * piece16);
  }
  if (half == 0 && row.have && a.lse) a.lse[at] = l == 0.0f ? -__builtin_huge_valf() : (m + __log2f(l)) * kLn2;
}

// Joins the parts of a row. A wave has a row where there are at most 64 parts, else a
// workgroup of sixteen waves, each with every sixteenth part. Bound by its launch and the
// parts' bytes, which the caches hold.
template <int DT, int NC, int WAVES>
__global__ __launch_bounds__(WAVES == 1 ? 256 : 64 * WAVES) void k_kv_join(KvAttendArgs a) {
  constexpr int D = 32 * NC, kEach = (D + 63) / 64, kParts = WAVES == 1 ? 64 : kMaxParts;
  __shared__ float share[WAVES == 1 ? 4 * kParts : kParts];
  __shared__ float sums[WAVES][kEach * 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t rows = (int64_t)a.T * a.c.H * a.G;
  const int64_t at = WAVES == 1 ? (int64_t)blockIdx.x * 4 + wave : blockIdx.x;
  if (at >= rows) return;
  const float* po = (const float*)a.work + at * a.splits * D;
  const float2* pm = reinterpret_cast<const float2*>((const float*)a.work + rows * a.splits * D) + at * a.splits;
  float2 ml[kParts / 64];
  float M = kLowest;
#pragma unroll
  for (int i = 0; i < kParts / 64; i++) {
    ml[i] = float2{kLowest, 0.0f};
    if (lane + 64 * i < a.splits) ml[i] = pm[lane + 64 * i];
    M = __builtin_fmaxf(M, ml[i].x);
  }
  for (int d = 1; d < 64; d <<= 1) M = __builtin_fmaxf(M, __shfl_xor(M, d, 64));
  float sum = 0.0f;
  float* f = WAVES == 1 ? share + wave * kParts : share;
#pragma unroll
  for (int i = 0; i < kParts / 64; i++) {
    const float e = __builtin_amdgcn_exp2f(ml[i].x - M);
    if (WAVES == 1 || wave == 0) f[lane + 64 * i] = e;
    sum += e * ml[i].y;
  }
  if constexpr (WAVES > 1)
    __syncthreads();
  else
    wave_lds_order();
  for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d, 64);
  const float by = sum == 0.0f ? 0.0f : 1.0f / sum;
  float v[kEach];
#pragma unroll
  for (int i = 0; i < kEach; i++) v[i] = 0.0f;
  // a part without a key holds zeros
#pragma unroll 8
  for (int s = WAVES == 1 ? 0 : wave; s < a.splits; s += WAVES) {
#pragma unroll
    for (int i = 0; i < kEach; i++)
      if (D % 64 == 0 || lane + 64 * i < D) v[i] += f[s] * po[(int64_t)s * D + lane + 64 * i];
  }
  if constexpr (WAVES > 1) {
#pragma unroll
    for (int i = 0; i < kEach; i++) sums[wave][lane + 64 * i] = v[i];
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int i = 0; i < kEach; i++) {
      v[i] = 0.0f;
#pragma unroll
      for (int w = 0; w < WAVES; w++) v[i] += sums[w][lane + 64 * i];
    }
  }
#pragma unroll
  for (int i = 0; i < kEach; i++)
    if (D % 64 == 0 || lane + 64 * i < D) {
      const uint32_t two = DT == kBF16 ? pack_bf16(v[i] * by, 0.0f) : pack_f16(v[i] * by, 0.0f);
      ((uint16_t*)a.out)[at * D + lane + 64 * i] = (uint16_t)two;
    }
  if (lane == 0 && a.lse) a.lse[at] = sum == 0.0f ? -__builtin_huge_valf() : (M + __log2f(sum)) * kLn2;
}

// ---------------------------------------------------------------- weights
//
// A workgroup stages 256 rows of q (or 32, where sequences have no more) in LDS, in fp16,
// and passes over its keys, 32 to a wave at a time, decoded to registers. Here the keys are
// the columns of the matrix instruction's result, so that a lane has one key and sums its
// weights over the rows in its own registers. A key belongs to one wave, so the sums are
// added to what is there without atomics, in an order that is always the same.
//
// Keys alone are read, 9 D / 16 + 4 bytes each, and 4 bytes of sums read and written. 16 sequences
// of up to 4096 tokens on 8 heads of 128, a token each, 28 MB: 12.5 us, the chain of a workgroup's
// start and three or four steps. 64 new tokens of 32 query heads over 32768 keys, 17.4 GFLOP: 34 us,
// bound by the exponentials of 256 rows for each key beside the products (128 rows staged: 44 us
// for 40 then).

// Half a row: 16 NC neighbouring values, in NC blocks.
template <int NC> struct Half {
  struct __attribute__((packed, aligned(NC == 8 ? 8 : NC == 4 ? 4 : NC % 2 ? 1 : 2))) Scales {
    uint8_t v[NC];
  };
  Scales scales;
  __device__ __forceinline__ void decode(const Quarter<NC>* codes, Frag* f) const {
    uint32_t w[(NC + 3) / 4] = {};
#pragma unroll
    for (int i = 0; i < NC; i++) w[i / 4] |= (uint32_t)scales.v[i] << (8 * (i % 4));
#pragma unroll
    for (int i = 0; i < NC; i += 2) {
      const h2 p = i & 2 ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w[i / 4], 1.0f, true)
                         : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w[i / 4], 1.0f, false);
      const h2 lo = __builtin_shufflevector(p, p, 0, 0), hi = __builtin_shufflevector(p, p, 1, 1);
#pragma unroll
      for (int j = 0; j < 4; j++)
        if (2 * i + j < 2 * NC) {
          const int c = 2 * i + j;  // fragments 2i, 2i + 1 are block i, the next two block i + 1
          decode8(codes[c / NC].codes[c % NC], j < 2 ? lo : hi, f[c].u);
        }
    }
  }
};

template <int NC> struct KeyStep {
  Quarter<NC> k[2];  // codes alone, as loaded: four lanes to a row
  Half<NC> half;     // scales, and S_dec, of the lane's own key
  float sdec;
  bool there[2];     // wave-uniform
  __device__ __forceinline__ void load(const KvCache& c, const Pages& pg, const int (&page)[2], int first) {
    const int lane = threadIdx.x & 63;
    int64_t row[2];
#pragma unroll
    for (int u = 0; u < 2; u++) {
      row[u] = pg.row(page[u], first + 16 * u, there[u]);
      k[u].load_codes(c.k.codes + row[u] * (16 * NC) + lane * (4 * NC));
    }
    const int64_t mine = ((lane & 16) ? row[1] : row[0]) + (lane & 15);
    half.scales = *reinterpret_cast<const typename Half<NC>::Scales*>(c.k.scales + mine * (2 * NC) + (lane >> 5) * NC);
    sdec = c.k.sdec[mine];
  }
};

template <int DT, int NC, int kRows>
__global__ __launch_bounds__(256, kRows == 32 && NC <= 4 ? 4 : 2) void k_kv_weights(KvAttendArgs a) {
  constexpr int D = 32 * NC, kRow = 64 * NC + 16;
  __shared__ __attribute__((aligned(16))) uint8_t qs[kRows * kRow];
  __shared__ __attribute__((aligned(16))) uint8_t turn[4 * 512 * NC];
  __shared__ __attribute__((aligned(16))) float factor[kRows], ref[kRows];
  __shared__ __attribute__((aligned(16))) int limits[kRows];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = lane >> 5, col = lane & 31;
  check_kv(a.c, a.offs, a.T, a.status);
  const int h = blockIdx.x % a.c.H, b = blockIdx.x / a.c.H;
  GroupTile gt;
  gt.g = b;
  gt.tile = 0;
  gt.start = b ? a.offs[b - 1] : 0;
  gt.end = a.offs[b];
  gt.start = gt.start < 0 ? 0 : gt.start > a.T ? a.T : gt.start;
  gt.end = gt.end < gt.start ? gt.start : gt.end > a.T ? a.T : gt.end;
  const int n = gt.end - gt.start, len = length_of(a.c, a.c.lens[b]), rows = n * a.G;
  const Pages pg{a.c.table + (int64_t)b * a.c.W, a.c.pages, a.c.H, h, a.c.P, a.c.by_page};
  float* acc = a.acc + ((int64_t)b * a.c.H + h) * ((int64_t)a.c.W * a.c.P);
  uint8_t* mine = turn + wave * 512 * NC;
  if ((int64_t)blockIdx.y * 128 >= len) return;
  for (int g0 = 0; g0 < rows; g0 += kRows) {
    // keys that all of these rows see, and that any does
    const int least = a.causal ? min(len, len - n + a.by_group.div(g0) + 1) : len;
    const int most = a.causal ? min(len, len - n + a.by_group.div(min(g0 + kRows, rows) - 1) + 1) : len;
    if ((int64_t)blockIdx.y * 128 >= most) continue;
    // pages a step ahead of the loads, loads a step ahead of their use
    KeyStep<NC> next;
    const int stride = (int)gridDim.y * 128;
    int first = (int)(blockIdx.y * 4 + wave) * 32, page[2];
    auto after = [&](int pos) { return pos <= INT32_MAX - stride - 63 ? pos + stride : INT32_MAX - 63; };
    auto find = [&](int pos) {
#pragma unroll
      for (int u = 0; u < 2; u++) page[u] = pg.page(pos + 16 * u, len);
    };
    find(first);
    next.load(a.c, pg, page, first);
    find(after(first));
    __syncthreads();
#pragma unroll
    for (int r0 = 32 * wave; r0 < kRows; r0 += 128) {
      if (g0 + r0 >= rows) break;
      const Row row = row_of(a, gt, h, g0 + r0 + col);
      Frag q[2 * NC];
      const float undo = load_q<DT, 2 * NC, false>(
          a.q, row.token * a.stride + (int64_t)row.head * D + half * 16 * NC, 8, row.have, q);
      uint8_t* to = qs + (r0 + col) * kRow + half * 32 * NC;
#pragma unroll
      for (int c = 0; c < 2 * NC; c++)
        *reinterpret_cast<u32x4*>(to + 16 * c) = u32x4{q[c].u[0], q[c].u[1], q[c].u[2], q[c].u[3]};
      if (half == 0) {
        float lse = row.have ? a.lse[row.token * ((int64_t)a.c.H * a.G) + row.head] : 0.0f;
        // a row that sees nothing has no weights: 2^-infinity
        if (!row.have || lse == -__builtin_huge_valf()) lse = __builtin_huge_valf();
        factor[r0 + col] = a.scale_pow * undo;
        ref[r0 + col] = lse * 1.44269504088896341f;
        limits[r0 + col] = a.causal ? min(len, len - n + row.place + 1) : len;
      }
    }
    __syncthreads();
    for (; first < most; first += stride) {
      const KeyStep<NC> st = next;
      next.load(a.c, pg, page, after(first));
      find(after(after(first)));
      Frag kf[2 * NC];
      wave_lds_order();
#pragma unroll
      for (int u = 0; u < 2; u++) st.k[u].store_codes(mine + u * 256 * NC + 4 * NC * piece(lane >> 2, lane & 3));
      wave_lds_order();
      Quarter<NC> codes[2];
#pragma unroll
      for (int i = 0; i < 2; i++)
        codes[i].load_codes(mine + (col >> 4) * 256 * NC + 4 * NC * piece(col & 15, 2 * half + i));
      st.half.decode(codes, kf);
      const float key = st.sdec * a.scale_mant;
      float sum = 0.0f;
      auto product = [&](int rt) {
        f32x16 x;
#pragma unroll
        for (int i = 0; i < 16; i++) x[i] = 0.0f;
        const uint8_t* qp = qs + (rt + col) * kRow + half * 32 * NC;
#pragma unroll
        for (int c = 0; c < 2 * NC; c++) {
          Frag f;
          const u32x4 t = *reinterpret_cast<const u32x4*>(qp + 16 * c);
          f.u[0] = t.x, f.u[1] = t.y, f.u[2] = t.z, f.u[3] = t.w;
          x = __builtin_amdgcn_mfma_f32_32x32x16_f16(f.h, kf[c].h, x, 0, 0, 0);
        }
        return x;
      };
      // the weights of rows r .. r + 3, of which a lane has its key's
      auto weigh = [&](const f32x16& x, int i, int r, bool partly) {
        const f32x4 f = *reinterpret_cast<const f32x4*>(factor + r), z = *reinterpret_cast<const f32x4*>(ref + r);
        float e[4];
#pragma unroll
        for (int j = 0; j < 4; j++) e[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[4 * i + j], key * f[j], -z[j]));
        if (partly) {
          const int4 lim = *reinterpret_cast<const int4*>(limits + r);
          const int l4[4] = {lim.x, lim.y, lim.z, lim.w};
#pragma unroll
          for (int j = 0; j < 4; j++) e[j] = first + col < l4[j] ? e[j] : 0.0f;
        }
        sum += (e[0] + e[1]) + (e[2] + e[3]);
      };
      if (kRows > 32 && first + 32 <= least) {
        // rows that all see all keys: the next tile's matrix instructions beside this one's exponentials
        f32x16 x = product(0);
#pragma unroll 1
        for (int rt = 0; rt < kRows && g0 + rt < rows; rt += 32) {
          __builtin_amdgcn_sched_barrier(0);
          const f32x16 next = product(rt + 32 < kRows ? rt + 32 : rt);
#pragma unroll
          for (int i = 0; i < 4; i++) weigh(x, i, rt + 8 * i + 4 * half, false);
          __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
          FOS_INTERLEAVE(2 * NC, 64 / (2 * NC), 2)
          __builtin_amdgcn_sched_barrier(0);
          x = next;
        }
      } else {
#pragma unroll 1
        for (int rt = 0; rt < kRows && g0 + rt < rows; rt += 32) {
          const f32x16 x = product(rt);
          const bool partly = a.causal && first + 32 > len - n + a.by_group.div(g0 + rt) + 1;
#pragma unroll
          for (int i = 0; i < 4; i++) {
            if (g0 + rt + 8 * i >= rows) break;
            weigh(x, i, rt + 8 * i + 4 * half, partly);
          }
        }
      }
      const auto both = __builtin_amdgcn_permlane32_swap(__float_as_uint(sum), __float_as_uint(sum), false, false);
      sum = __uint_as_float(both[0]) + __uint_as_float(both[1]);
      const bool there = (lane & 16) ? st.there[1] : st.there[0];
      if (half == 0 && there && first + col < len) acc[first + col] += sum;
    }
  }
}

// Tiles of `rows` rows, of the mean sequence.
int64_t kv_tiles(int64_t T, int B, int H, int G, int64_t rows) {
  const int64_t per = (T * G / B + rows - 1) / rows;
  return (per < 1 ? 1 : per) * B * H;
}

// The tile kernel from 49 rows to a sequence on, unless the other's smallest parts are so few
// that the chip runs them at once. Few rows and tiles, us, heads of 128 unless said: 8 heads of
// 8192 keys, 32 rows 17.1 and 18.1, 48 19.9 and 18.6, 96 24.5 and 21.1; 4 sequences of that 32
// rows 26.4 and 35.8, 64 38.8 and 39.6, 96 54 and 42; 16 of 2048 keys, 32 rows 35.3 and 36.5, 64
// 44 and 39.8; 8 heads of 64 with 2048 keys, 256 rows 13.8 and 14.5; 8 heads of 1024 keys, 256
// rows 15.5 and 18.3.
bool kv_tiled(int64_t T, int B, int H, int G, int64_t max_len) {
  return T * G > (int64_t)48 * B && kv_tiles(T, B, H, G, 16) * ((max_len + 127) / 128) > 2048;
}

// Waves that one workgroup's LDS holds, of a whole cache (kv_wide).
template <int NC>
constexpr int kWideWaves = NC <= 4 ? 12 : NC == 6 ? 8 : 4;

template <int DT, int NC>
hipError_t attend(const KvAttendArgs& a, hipStream_t s) {
  const int64_t rows = (int64_t)a.T * a.G;
  const int per = kv_tiled(a.T, a.c.B, a.c.H, a.G, a.max_len) ? 128 : 16;
  const int64_t tiles = rows / per + a.c.B + 1;  // no fewer than the sequences' tiles and the tail's
  const dim3 grid((unsigned)(tiles * a.c.H * a.splits));
  if (per == 128)
    k_kv_tile<DT, NC><<<grid, 256, 0, s>>>(a);
  else if (a.wide)
    k_kv_stream<DT, NC, kWideWaves<NC>><<<grid, 64 * kWideWaves<NC>, 0, s>>>(a);
  else
    k_kv_stream<DT, NC, 4><<<grid, 256, 0, s>>>(a);
  // one wave to a row and sixteen, us of attention: 32 parts, 32 rows 8.9 and 9.6; 64 parts, 8 rows
  // 10.8 and 10.0, 128 rows 12.3 and 13.2; 9 parts, 4096 rows 35.2 and 49.6
  if (a.splits > 64 || (a.splits > 32 && rows * a.c.H < 64))
    k_kv_join<DT, NC, 16><<<dim3((unsigned)(rows * a.c.H)), 1024, 0, s>>>(a);
  else if (a.splits > 1)
    k_kv_join<DT, NC, 1><<<dim3((unsigned)((rows * a.c.H + 3) / 4)), 256, 0, s>>>(a);
  return hipGetLastError();
}

template <int DT, int NC>
hipError_t weights(const KvAttendArgs& a, hipStream_t s) {
  // 32 rows in LDS and four workgroups to a CU, or 256 and two, us: 8 heads of 8192 keys, 32 rows
  // 5.8 and 6.3, 64 9.3 and 7.9; 16 sequences of 2048 keys, 32 rows 9.6 and 11.6, 128 28.6 and 21.4.
  // Workgroups: as many as run at once (64 heads of 4096 keys, a token each: 256 workgroups 11.4 us,
  // 512 to 1280 8.8, 2048 11.1; 8 heads of 32768 keys, 256 rows: 256 43, 512 33.5, 1024 40).
  const bool few = (int64_t)a.T * a.G <= (int64_t)32 * a.c.B;
  const int64_t heads = (int64_t)a.c.B * a.c.H, most = (a.max_len + 127) / 128;
  int64_t chunks = (few ? 1280 : 512) / heads;
  chunks = chunks > most ? most : chunks;
  chunks = chunks < 1 ? 1 : chunks;
  const dim3 grid((unsigned)heads, (unsigned)chunks);
  if (few)
    k_kv_weights<DT, NC, 32><<<grid, 256, 0, s>>>(a);
  else
    k_kv_weights<DT, NC, 256><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

template <int DT>
hipError_t run(bool attention, const KvAttendArgs& a, hipStream_t s) {
  switch (a.c.D / 32) {
    case 1: return attention ? attend<DT, 1>(a, s) : weights<DT, 1>(a, s);
    case 2: return attention ? attend<DT, 2>(a, s) : weights<DT, 2>(a, s);
    case 3: return attention ? attend<DT, 3>(a, s) : weights<DT, 3>(a, s);
    case 4: return attention ? attend<DT, 4>(a, s) : weights<DT, 4>(a, s);
    case 6: return attention ? attend<DT, 6>(a, s) : weights<DT, 6>(a, s);
    case 8: return attention ? attend<DT, 8>(a, s) : weights<DT, 8>(a, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace

// A short cache is left whole, by twelve waves to a workgroup (eight for D 192: what LDS holds),
// with one launch and no workspace, where there are no more tiles than CUs. Whole and in parts, us,
// a token to a sequence on 4 query heads to each of the cache's: calls one after another, and
// captured in a graph in brackets. One sequence, 8 heads of 128: 256 keys 14.9 (8.3) and 19.4 (8.5),
// 1024 15.2 (12.9) and 19.8 (8.4), 1536 16.5 (16.6) and 19.2 (8.8), 2048 19.4 (19.8) and 20.1 (8.8):
// a call gains up to 2048 keys, a captured step loses from 512 on, and 1024 is between. 1000 keys:
// 64 tiles 15.2 (13.0) and 19.7 (10.2), 120 15.2 (13.0) and 19.7 (14.2), 256 15.1 (15.6) and 24.9
// (25.3), 264 25.7 (26.3) and 26.6 (27.1); heads of 64, 256 tiles 14.5 (10.7) and 18.9 (16.4), 264
// 18.1 (18.3) and 19.4 (17.9); of 192, 256 tiles 19.1 (19.5) and 36.4 (37.3).
bool kv_wide(int64_t T, int B, int H, int G, int D, int64_t max_len) {
  return !kv_tiled(T, B, H, G, max_len) && D <= 192 && max_len <= 1024 && kv_tiles(T, B, H, G, 16) <= 256;
}

// Parts of the keys. Few rows: where the tiles alone fill the chip's 256 CUs, workgroups enough
// to even out lengths (64 sequences of 2500 to 8192 tokens on 8 heads: 1024 workgroups 103 us,
// 2304 96); else about as many as run at once (131072 keys for one token on 4 heads: 512 to
// 2304 25 to 27 us, 384 30; 17 sequences of up to 2999 tokens, 12 heads of 64: 512 22.8, 1024
// 19.4, 1536 21.2). A part has four steps at least, one to a wave (1001 keys: 8.2 us; of two
// 9.4, of eight 9.7).
// Tiles: 512 workgroups, two to a CU, of eight steps or more, but no fewer than 256 where that
// leaves four (8 heads of 8192 keys, 96 rows, parts of 512 keys 25.5 us, 256 21.1; 256 rows,
// 512 workgroups of 256 keys 33.4, 256 of 512 29.5).
int kv_splits(int64_t T, int B, int H, int G, int D, int64_t max_len) {
  if (kv_wide(T, B, H, G, D, max_len)) return 1;
  auto parts = [=](int64_t tiles, int64_t groups, int64_t least) {
    const int64_t s = groups / tiles, most = (max_len + least - 1) / least;
    return (int)(s > most ? most : s);
  };
  int s;
  if (kv_tiled(T, B, H, G, max_len)) {
    const int64_t tiles = kv_tiles(T, B, H, G, 128);
    const int x = parts(tiles, 512, 512), y = parts(tiles, 256, 256);
    s = x > y ? x : y;
  } else {
    const int64_t tiles = kv_tiles(T, B, H, G, 16);
    s = parts(tiles, tiles >= 256 ? 2304 : 1024, 128);
  }
  return s < 1 ? 1 : s > kMaxParts ? kMaxParts : s;
}

int64_t kv_attend_workspace(int64_t T, int H, int G, int D, int splits) {
  return splits > 1 ? T * H * G * splits * (D + 2) * 4 : 0;
}

hipError_t launch_kv_attention(int dt, const KvAttendArgs& a, hipStream_t s) {
  return dt == kBF16 ? run<kBF16>(true, a, s) : run<kFP16>(true, a, s);
}

hipError_t launch_kv_weights(int dt, const KvAttendArgs& a, hipStream_t s) {
  return dt == kBF16 ? run<kBF16>(false, a, s) : run<kFP16>(false, a, s);
}

}  // namespace fos
