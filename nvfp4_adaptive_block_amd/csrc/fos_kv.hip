// fos_kv.hip: the NVFP4 key/value cache's writers: the append, which quantizes the
// rows of new tokens into the sequences' pages, and the eviction, which keeps the
// rows of the largest accumulated attention weight and closes the gaps.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fos_device.h"
#include "fos_ops.h"
#include "fos_rows.h"

namespace fos {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __amdgpu_buffer_rsrc_t Rsrc;

// Of a call without tokens, which has nothing else to do.
__global__ __launch_bounds__(256) void k_kv_check(KvCache c, const int32_t* offs, int32_t* status) {
  check_kv(c, offs, 0, status);
}

// ---------------------------------------------------------------- append
//
// One lane has one block of 16 values, and the D/16 blocks of a row are
// neighbouring lanes (2, 4, 8 or 16 of them, some idle where D/16 is no power of
// two), so the row's amax crosses lanes by shifts and everything else stays in the
// lane. Per row S_enc = 6B/amax and S_dec = 1/S_enc; per block both candidates are
// encoded, decoded and compared as fos_quantize does, with the candidate's
// multiplier by a division of its own: a table of all scales, which the quantizer
// keeps per tensor, would be rebuilt for every row.
//
// A row of D values is read once (and given back on request, past the caches, which
// nothing reads soon) and leaves 9 D / 16 + 4 bytes. A few tokens are bound by the launch
// and a chain of loads (offsets, row, length, page: 3.7 us for a token of 8 heads of
// 128); many by memory, with the arithmetic close behind: six prompts, 37900 tokens of 8 heads of
// 128 with the values given back, 357 MB in 65 us in a graph (72 call by call). Blocks without a NaN take a shorter
// conversion (98 us for all without it); several turns per workgroup lost (103 to 115).

template <int DT>
__device__ __forceinline__ void load_block(const void* p, int64_t i, float* x) {
  if constexpr (DT == kFP32) {
    const u32x4* s = reinterpret_cast<const u32x4*>((const float*)p + i);
    u32x4 v[4];
#pragma unroll
    for (int j = 0; j < 4; j++) v[j] = s[j];
#pragma unroll
    for (int j = 0; j < 16; j++) x[j] = __uint_as_float(v[j / 4][j % 4]);
  } else {
    const u32x4* s = reinterpret_cast<const u32x4*>((const uint16_t*)p + i);
    const u32x4 v[2] = {s[0], s[1]};
#pragma unroll
    for (int j = 0; j < 8; j++) {
      const uint32_t w = v[j / 4][j % 4];
      x[2 * j] = DT == kBF16 ? bf16_lo(w) : f16_lo(w);
      x[2 * j + 1] = DT == kBF16 ? bf16_hi(w) : f16_hi(w);
    }
  }
}

template <int DT>
__device__ __forceinline__ void store_block(void* p, int64_t i, const float* y) {
  if constexpr (DT == kFP32) {
    u32x4* s = reinterpret_cast<u32x4*>((float*)p + i);
#pragma unroll
    for (int j = 0; j < 4; j++)
      __builtin_nontemporal_store(u32x4{__float_as_uint(y[4 * j]), __float_as_uint(y[4 * j + 1]),
                                        __float_as_uint(y[4 * j + 2]), __float_as_uint(y[4 * j + 3])}, s + j);
  } else {
    u32x4* s = reinterpret_cast<u32x4*>((uint16_t*)p + i);
#pragma unroll
    for (int j = 0; j < 2; j++) {
      u32x4 v;
#pragma unroll
      for (int k = 0; k < 4; k++)
        v[k] = DT == kBF16 ? pack_bf16(y[8 * j + 2 * k], y[8 * j + 2 * k + 1])
                           : pack_f16(y[8 * j + 2 * k], y[8 * j + 2 * k + 1]);
      __builtin_nontemporal_store(v, s + j);
    }
  }
}

// max |x| without the NaN elements: by the magnitudes' bits where there may be some.
template <bool NANS>
__device__ __forceinline__ float amax16(const float* x) {
  if constexpr (NANS) {
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 16; i++) {
      const uint32_t m = __float_as_uint(x[i]) & 0x7FFFFFFFu;
      a = max(a, m <= 0x7F800000u ? m : 0u);
    }
    return __uint_as_float(a);
  } else {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; i++) a = __builtin_fmaxf(a, __builtin_fabsf(x[i]));
    return a;
  }
}
__device__ __forceinline__ bool any_nan16(const float* x) {
  float m = x[0];
#pragma unroll
  for (int i = 1; i < 16; i++) m = __builtin_elementwise_maximum(m, x[i]);
  return m != m;
}

struct Encoded {
  uint32_t c0, c1, scale;
  float D;  // RN(scale S_dec)
};

// q: the block's amax over the candidate's top value.
template <bool NANS>
__device__ __forceinline__ Encoded encode(const float* x, float q, float S_enc, float S_dec) {
  Encoded o;
  o.scale = e4m3_code(q * S_enc);
  const float sigma = e4m3_value(o.scale);
  const float E = sigma == 0.0f ? 0.0f : __builtin_fminf(S_enc / sigma, kFltMax);
  float v[16];
#pragma unroll
  for (int i = 0; i < 16; i++) v[i] = NANS && x[i] != x[i] ? 6.0f : x[i] * E;
  o.c0 = e2m1_pack8(v);
  o.c1 = e2m1_pack8(v + 8);
  o.D = sigma * S_dec;
  return o;
}

__device__ __forceinline__ void decode(const Encoded& o, float* y) {
  e2m1_unpack8(o.c0, y);
  e2m1_unpack8(o.c1, y + 8);
#pragma unroll
  for (int i = 0; i < 16; i++) y[i] = y[i] * o.D;
}

template <int METRIC, int PREC, int ORDER>
__device__ __forceinline__ float error16(const float* x, const float* y) {
  float u[16];
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    float e0, e1;
    if constexpr (PREC == kErrFP16) {
      sub_f16x2(x[i], x[i + 1], y[i], y[i + 1], e0, e1);
    } else {
      e0 = x[i] - y[i];
      e1 = x[i + 1] - y[i + 1];
    }
    u[i] = METRIC == kMAE ? __builtin_fabsf(e0) : e0 * e0;
    u[i + 1] = METRIC == kMAE ? __builtin_fabsf(e1) : e1 * e1;
  }
  return ORDER == kOrderSeq ? seq16(u) : tree16(u);
}

// The better of the two candidates for a block whose amax is a; a tie keeps map-to-6, and
// so does a block with a NaN, whose errors compare false.
template <int RECIPE, int METRIC, int PREC, int ORDER, bool NANS>
__device__ __forceinline__ Encoded quantize16(const float* x, float a, float S_enc, float S_dec) {
  const Encoded k6 = encode<NANS>(x, div6(a), S_enc, S_dec);
  if constexpr (RECIPE == kNVFP4) return k6;
  const Encoded k4 = encode<NANS>(x, a * 0.25f, S_enc, S_dec);
  float y[16];
  decode(k6, y);
  const float e6 = error16<METRIC, PREC, ORDER>(x, y);
  decode(k4, y);
  return error16<METRIC, PREC, ORDER>(x, y) < e6 ? k4 : k6;
}

template <int DT, int RECIPE, int METRIC, int PREC, int ORDER>
__global__ __launch_bounds__(256) void k_kv_append(KvAppendArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, side = blockIdx.y;
  const int blocks = a.c.D / 16;
  const int sh = blocks <= 2 ? 1 : blocks <= 4 ? 2 : blocks <= 8 ? 3 : 4;  // log2 of the lanes per row
  const int64_t first = ((int64_t)blockIdx.x * 4 + wave) * (64 >> sh);
  const int64_t rows = (int64_t)a.T * a.c.H;
  check_kv(a.c, a.offs, a.T, a.status);
  if (first >= rows) return;
  // the sequence of the wave's first token: the first whose end lies behind it
  const int t0 = a.by_head.div((int)first);
  int b = first_end_behind(a.offs, a.c.B, t0);
  const int64_t r = first + (lane >> sh);
  const int j = lane & ((1 << sh) - 1);
  const bool have = r < rows && j < blocks;
  const int t = a.by_head.div((int)(r < rows ? r : rows - 1)), h = (int)(r < rows ? r : rows - 1) - t * a.c.H;
  // a later token's, by steps that double and then halve again
  if (b < a.c.B && a.offs[b] <= t) {
    int step = 1;
    while (b + step < a.c.B && a.offs[b + step] <= t) b += step, step *= 2;
    for (; step > 0; step >>= 1)
      if (b + step < a.c.B && a.offs[b + step] <= t) b += step;
    b++;
  }
  const bool tail = b >= a.c.B;

  float x[16];
#pragma unroll
  for (int i = 0; i < 16; i++) x[i] = 0.0f;
  if (have && !tail) load_block<DT>(a.x[side], t * a.stride[side] + (int64_t)h * a.c.D + 16 * j, x);
  const bool nans = __any(any_nan16(x));
  const float top = nans ? amax16<true>(x) : amax16<false>(x);
  float A = top;
  for (int d = 1; d < 1 << sh; d <<= 1) A = __builtin_fmaxf(A, __shfl_xor(A, d, 64));
  const float S_enc = global_encode_scale(A, a.six_b);
  // a row of zeros has no size of its own: S_dec 0 keeps it from setting one
  const float S_dec = A == 0.0f ? 0.0f : 1.0f / S_enc;
  const Encoded o = nans ? quantize16<RECIPE, METRIC, PREC, ORDER, true>(x, top, S_enc, S_dec)
                         : quantize16<RECIPE, METRIC, PREC, ORDER, false>(x, top, S_enc, S_dec);
  if (have && a.y[side]) {
    float y[16];
    decode(o, y);
    if (tail) {
#pragma unroll
      for (int i = 0; i < 16; i++) y[i] = 0.0f;
    }
    store_block<DT>(a.y[side], r * a.c.D + 16 * j, y);
  }
  if (!have || tail) return;
  // so many before the end of the sequence's new rows, and of its cache
  const int len = min(a.c.lens[b], a.c.W * a.c.P);
  const int64_t pos = (int64_t)len - min(a.offs[b], a.T) + t;
  const bool inside = pos >= 0 && pos < len;
  int64_t page = -1;
  int slot = 0;
  if (inside) {
    const int w = a.c.by_page.div((int)pos);
    slot = (int)pos - w * a.c.P;
    page = a.c.table[(int64_t)b * a.c.W + w];
  }
  if (page < 0 || page >= a.c.pages) {
    if (a.status && j == 0) atomicOr(a.status, kStatusBadCache);
    return;
  }
  const KvRows& to = side ? a.c.v : a.c.k;
  const int64_t row = (page * a.c.H + h) * a.c.P + slot;
  *reinterpret_cast<u32x2*>(to.codes + row * (a.c.D / 2) + 8 * j) = u32x2{o.c0, o.c1};
  to.scales[row * blocks + j] = (uint8_t)o.scale;
  if (j == 0) to.sdec[row] = S_dec;
}

template <int DT, int RECIPE, int METRIC, int PREC>
void append(const KvAppendArgs& a, dim3 grid, hipStream_t s) {
  if (a.order == kOrderSeq)
    k_kv_append<DT, RECIPE, METRIC, PREC, kOrderSeq><<<grid, 256, 0, s>>>(a);
  else
    k_kv_append<DT, RECIPE, METRIC, PREC, kOrderTree><<<grid, 256, 0, s>>>(a);
}

template <int DT>
void append(const KvAppendArgs& a, dim3 grid, hipStream_t s) {
  if (a.recipe == kNVFP4) return append<DT, kNVFP4, kMSE, kErrExact>(a, grid, s);
  if (a.metric == kMAE)
    return a.prec == kErrFP16 ? append<DT, k4over6, kMAE, kErrFP16>(a, grid, s)
                              : append<DT, k4over6, kMAE, kErrExact>(a, grid, s);
  return a.prec == kErrFP16 ? append<DT, k4over6, kMSE, kErrFP16>(a, grid, s)
                            : append<DT, k4over6, kMSE, kErrExact>(a, grid, s);
}

// ---------------------------------------------------------------- evict
//
// One workgroup has one head of one sequence. The weights' order is that of their
// bits (made monotonic), so the smallest kept weight is found digit by digit from
// the top, 11, 11 and 10 bits at a time, by histograms in LDS. Kept rows behind the
// place where the middle of the shorter cache ends take the places before it that
// are given up, in order; neither side of such a move is the other side of another,
// so they run in any order. The last rows then move down together, a chunk at a
// time, each read before it is written.
//
// What has to move is little (256 heads of 1088 rows cut to 1024: 16 MB, 3 us of a copy), so
// the time is the chain in a workgroup: find its row's weights, three digits of four
// barriers each, the moves' list, and two rounds of loads before stores (14.4 us; the digits
// 3.4 of them, the list 1, moves and last rows 4.6).

constexpr int kThreads = 1024, kWaves = kThreads / 64;

// Weights in order as unsigned numbers: NaN lowest, zeros alike; 0 is no weight.
__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t u = __float_as_uint(v == 0.0f ? 0.0f : v);
  return v != v ? 1u : (u >> 31) ? ~u : u | 0x80000000u;
}

// Row of the cache at a position of sequence b.
struct Rows {
  const int32_t* table;
  int64_t H;
  int h, P;
  FastDiv by_page;
  __device__ __forceinline__ int64_t at(int pos) const {
    const int w = by_page.div(pos);
    return ((int64_t)table[w] * H + h) * P + (pos - w * P);
  }
};

// What a row is moved as: 2 NC pieces of 16 bytes of codes; the scales of either side in
// pieces of four bytes (two, where NC is odd), either S_dec and its weight, a lane each. A
// lane has the same piece of every row that its team moves, so a row is two loads and two
// stores.
template <int NC> struct Mover {
  static constexpr int kSmall = NC % 2 ? 2 : 4, kScales = 2 * NC / kSmall;  // bytes, pieces a side
  static constexpr int kItems = 2 * NC + 2 * kScales + 3;
  union Piece {
    u32x4 codes;
    uint32_t small;
  };
  uint8_t* base;   // of the first row's piece
  int64_t step;    // from one row to the next
  int item;

  __device__ __forceinline__ Mover(const KvCache& c, float* acc, int i) {
    item = i;
    const KvRows& s = (i < 2 * NC ? i < NC : i < 2 * NC + 2 * kScales ? i < 2 * NC + kScales : i == kItems - 3) ? c.k : c.v;
    if (i < 2 * NC) {
      base = s.codes + 16 * (i < NC ? i : i - NC);
      step = 16 * NC;
    } else if (i < 2 * NC + 2 * kScales) {
      base = s.scales + kSmall * ((i - 2 * NC) % kScales);
      step = 2 * NC;
    } else {
      base = i == kItems - 1 ? (uint8_t*)acc : (uint8_t*)s.sdec;
      step = 4;
    }
  }
  // `pos`: the row's place, by which the weights go
  __device__ __forceinline__ uint8_t* at(int64_t row, int pos) const {
    return base + (item == kItems - 1 ? pos : row) * step;
  }
  __device__ __forceinline__ Piece read(int64_t row, int pos) const {
    Piece p;
    const uint8_t* q = at(row, pos);
    if (item < 2 * NC)
      p.codes = *reinterpret_cast<const u32x4*>(q);
    else if (kSmall == 2 && item < 2 * NC + 2 * kScales)
      p.small = *reinterpret_cast<const uint16_t*>(q);
    else if (item < kItems)
      p.small = *reinterpret_cast<const uint32_t*>(q);
    return p;
  }
  __device__ __forceinline__ void write(int64_t row, int pos, const Piece& p) const {
    uint8_t* q = at(row, pos);
    if (item < 2 * NC)
      *reinterpret_cast<u32x4*>(q) = p.codes;
    else if (kSmall == 2 && item < 2 * NC + 2 * kScales)
      *reinterpret_cast<uint16_t*>(q) = (uint16_t)p.small;
    else if (item < kItems)
      *reinterpret_cast<uint32_t*>(q) = p.small;
  }
};

// The digit at `shift` of the wanted weight: counts are from the largest down.
// Leaves how many of the digit's own are wanted in `want`, and how many there are.
// `share` has a word for each wave, as many again that this leaves alone, and four for
// the result: waves that have read it go on while others still have to.
struct Digit {
  uint32_t digit;
  int want, of;
};
template <int BINS>
__device__ Digit find_digit(const int* hist, int* share, int want) {
  // thread t has the bins BINS - 1 - 2t and the one below
  const int t = threadIdx.x, lane = t & 63;
  int c0 = 0, c1 = 0;
  if (2 * t < BINS) {
    c0 = hist[BINS - 1 - 2 * t];
    c1 = hist[BINS - 2 - 2 * t];
  }
  const int sum = wave_scan(c0 + c1);
  if (lane == 63) share[t >> 6] = sum;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < (t >> 6); w++) before += share[w];
  const int above = before + sum - c0 - c1;  // weights in the bins above this thread's
  int* out = share + 2 * kWaves;
  if (2 * t < BINS && above < want && above + c0 + c1 >= want) {
    const bool first = above + c0 >= want;
    out[0] = BINS - 1 - 2 * t - (first ? 0 : 1);
    out[1] = want - above - (first ? 0 : c0);
    out[2] = first ? c0 : c1;
  }
  __syncthreads();
  return Digit{(uint32_t)out[0], out[1], out[2]};
}

// One head of one sequence, and what there is to do.
struct Cut {
  int b, h, n;
  bool whole;  // stays as it is
  float* acc;
  int2* moves;
  Rows rows;
};
// n is cut to the table; a sequence with a page that is none stays. Uniform over the
// workgroup; `bad` is a word of its LDS.
__device__ Cut find_cut(const KvEvictArgs& a, int bh, int* bad) {
  Cut c;
  c.b = bh / a.c.H;
  c.h = bh - c.b * a.c.H;
  const int cap = a.c.W * a.c.P, len = a.c.lens[c.b];
  c.n = len < 0 ? 0 : len > cap ? cap : len;
  const int32_t* table = a.c.table + (int64_t)c.b * a.c.W;
  c.acc = a.acc + (int64_t)bh * cap;
  c.moves = a.moves + (int64_t)bh * (a.budget - a.recent);
  c.rows = Rows{table, a.c.H, c.h, a.c.P, a.c.by_page};
  if (threadIdx.x == 0) *bad = 0;
  __syncthreads();
  if (c.n > a.budget) {
    for (int w = threadIdx.x; w <= a.c.by_page.div(c.n - 1); w += blockDim.x)
      if (table[w] < 0 || table[w] >= a.c.pages) *bad = 1;
  }
  __syncthreads();
  c.whole = c.n <= a.budget || *bad;
  if (threadIdx.x == 0 && c.h == 0) {
    a.new_lens[c.b] = c.whole ? c.n : a.budget;
    if (a.status && (len != c.n || *bad)) atomicOr(a.status, kStatusBadCache);
  }
  return c;
}

// The moves of the middle, in order; returns their number. A lane holds BATCH weights at a
// time. One CU has all of a head's, and is bound by the instructions for each (32768 weights:
// read 3 us, the three digits 4, 2 and 2, counted 2, written 3): lanes past the end hold the
// lowest order, which is counted but never wanted, instead of being masked (54 to 52 us for
// 32 heads of up to 32768 rows cut to 4096).
template <int BATCH>
__device__ int find_moves(const KvEvictArgs& a, const Cut& cut, int* hist, int* share) {
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int keep = a.budget - a.recent, lo = a.sinks, hi = cut.n - a.recent;  // the middle: [lo, hi)
  if (keep <= lo) return 0;
  const float* acc = cut.acc;
  // each wave has a stretch of the middle, in order, BATCH x 64 weights at a time; a
  // stretch of one batch is read once and stays in registers
  const int each = ((hi - lo + kWaves * 64 - 1) / (kWaves * 64)) * 64;
  const int from = min(hi, lo + wave * each), to = min(hi, from + each);
  const bool held = each <= 64 * BATCH;
  uint32_t o[BATCH];
  auto read = [&](int i) {
    const Rsrc r = __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(acc + i), (short)0, 4 * min(to - i, 64 * BATCH), 0x00020000);
    uint32_t v[BATCH];
#pragma unroll
    for (int k = 0; k < BATCH; k++) v[k] = __builtin_amdgcn_raw_buffer_load_b32(r, 4 * (64 * k + lane), 0, 0);
#pragma unroll
    for (int k = 0; k < BATCH; k++) o[k] = i + 64 * k + lane < to ? order_of(__uint_as_float(v[k])) : 0u;
  };
  if (held && from < to) read(from);
  // f(the first of 64 places, the order of this lane's weight) along the wave's stretch
  auto stretch = [&](auto f) {
    for (int i = from; i < to; i += 64 * BATCH) {
      if (!held) read(i);
#pragma unroll
      for (int k = 0; k < BATCH; k++) {
        if (i + 64 * k >= to) break;
        f(i + 64 * k, o[k]);
      }
    }
  };
  // the smallest kept weight, and how many of its equals are kept
  uint32_t found = 0, mask = 0;
  Digit d{0, keep - lo, 0};
#pragma unroll 1
  for (int pass = 0; pass < 3; pass++) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t low = pass == 2 ? 1023u : 2047u;
    hist[t] = 0;
    hist[t + 1024] = 0;
    __syncthreads();
    stretch([&](int, uint32_t w) {
      if ((w & mask) == found) atomicAdd(&hist[(w >> shift) & low], 1);
    });
    __syncthreads();
    d = find_digit<2048>(hist, share, d.want);
    found |= d.digit << shift;
    mask |= low << shift;
  }
  // equals of the smallest kept weight before this wave's, where only some are kept
  const bool some = d.want < d.of;
  int equals = 0;
  if (some) {
    int c = 0;
    stretch([&](int, uint32_t w) { c += __popcll(__ballot(w == found)); });
    if (lane == 0) share[wave] = c;
    __syncthreads();
    for (int w = 0; w < wave; w++) equals += share[w];
    __syncthreads();
  }
  // the places below `keep` that are given up, and the kept ones from there on: counted, then written
  auto below = [](unsigned long long m) {
    return (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0u));
  };
  const int ends = min(keep, to);
  int n_free = 0, n_moved = 0, eq = equals;
  // whether a place below `keep` is given up, and whether one behind is kept
  auto look = [&](int i, uint32_t w, bool& is_free, bool& is_moved) {
    bool kept = w >= found;
    if (some) {
      const unsigned long long same = __ballot(w == found);
      if (w == found && eq + below(same) >= d.want) kept = false;
      eq += __popcll(same);
    }
    const bool in = i + lane < ends;
    is_free = in && !kept;
    is_moved = kept && !in;
  };
  stretch([&](int i, uint32_t w) {
    bool is_free, is_moved;
    look(i, w, is_free, is_moved);
    n_free += __popcll(__ballot(is_free));
    n_moved += __popcll(__ballot(is_moved));
  });
  if (lane == 0) {
    share[wave] = n_free;
    share[kWaves + wave] = n_moved;
  }
  __syncthreads();
  int holes = 0;
  n_free = n_moved = 0;
  eq = equals;
  for (int w = 0; w < kWaves; w++) {
    if (w < wave) {
      n_free += share[w];
      n_moved += share[kWaves + w];
    }
    holes += share[w];
  }
  int2* out = cut.moves;
  stretch([&](int i, uint32_t w) {
    bool is_free, is_moved;
    look(i, w, is_free, is_moved);
    const unsigned long long f = __ballot(is_free), m = __ballot(is_moved);
    if (is_free) out[n_free + below(f)].y = i + lane;
    if (is_moved) out[n_moved + below(m)].x = i + lane;
    n_free += __popcll(f);
    n_moved += __popcll(m);
  });
  return holes;
}

// Rows are moved by teams of 16 lanes (32, where a row has more pieces), several at a time.
template <int NC>
struct Teams {
  typedef Mover<NC> M;
  static constexpr int kLanes = M::kItems <= 16 ? 16 : 32, kRows = 8;
  static_assert(M::kItems <= 32);
  typedef typename M::Piece Held[kRows];

  // Moves first, first + step, ... below `holes`.
  static __device__ __forceinline__ void move(const KvEvictArgs& a, const Cut& cut, int holes, int first, int step) {
    const M piece(a.c, cut.acc, threadIdx.x % kLanes);
    for (int i0 = first; i0 < holes; i0 += kRows * step) {
      int2 mv[kRows];
      Held p;
#pragma unroll
      for (int r = 0; r < kRows; r++)
        if (i0 + r * step < holes) mv[r] = cut.moves[i0 + r * step];
#pragma unroll
      for (int r = 0; r < kRows; r++)
        if (i0 + r * step < holes) {
          p[r] = piece.read(cut.rows.at(mv[r].x), mv[r].x);
        }
#pragma unroll
      for (int r = 0; r < kRows; r++)
        if (i0 + r * step < holes) {
          piece.write(cut.rows.at(mv[r].y), mv[r].y, p[r]);
        }
    }
  }

  // The last rows, `gap` down, by one workgroup of THREADS or by `parts` of them. A chunk's rows
  // are all read before any is written, and what a chunk writes lies below what later ones read;
  // where the rows' places and those they come from have none in common, chunks are
  // independent and each part has its own, else the first part has all. The weights behind
  // the cut are cleared, those of a chunk's rows by the part that has it.
  template <int THREADS>
  static __device__ __forceinline__ void shift(const KvEvictArgs& a, const Cut& cut, int part, int parts) {
    constexpr int kTeams = THREADS / kLanes;
    const M piece(a.c, cut.acc, threadIdx.x % kLanes);
    const int team = threadIdx.x / kLanes, keep = a.budget - a.recent, gap = cut.n - a.budget;
    const bool apart = gap >= a.recent;
    if (!apart) {
      if (part > 0) return;
      parts = 1;
    }
    for (int i = a.budget + part * THREADS + threadIdx.x; i < cut.n - a.recent; i += parts * THREADS) cut.acc[i] = 0.0f;
    for (int i0 = part * kRows * kTeams; i0 < a.recent; i0 += parts * kRows * kTeams) {
      Held p;
#pragma unroll
      for (int r = 0; r < kRows; r++) {
        const int i = i0 + r * kTeams + team;
        if (i < a.recent) {
          p[r] = piece.read(cut.rows.at(keep + i + gap), keep + i + gap);
        }
      }
      __syncthreads();
#pragma unroll
      for (int r = 0; r < kRows; r++) {
        const int i = i0 + r * kTeams + team;
        if (i < a.recent) {
          piece.write(cut.rows.at(keep + i), keep + i, p[r]);
          if (apart && threadIdx.x % kLanes == M::kItems - 1) cut.acc[keep + i + gap] = 0.0f;
        }
      }
    }
    if (apart) return;
    __syncthreads();
    for (int i = max(a.budget, cut.n - a.recent) + threadIdx.x; i < cut.n; i += THREADS) cut.acc[i] = 0.0f;
  }
};

// All of it in one launch, or (ALL = false) the search for the moves alone, whose number
// goes to counts (-1 for a sequence that stays as it is).
template <int NC, bool ALL>
__global__ __launch_bounds__(kThreads) void k_kv_evict(KvEvictArgs a) {
  __shared__ int hist[2048];
  __shared__ int share[2 * kWaves + 4];
  __shared__ int bad;
  const Cut cut = find_cut(a, blockIdx.x, &bad);
  if (cut.whole) {
    if (!ALL && threadIdx.x == 0) a.counts[blockIdx.x] = -1;
    return;
  }
  // (32 in both: 128 heads of 1088 tokens 36 us instead of 17, for the code's size and spills;
  // 8 in both: 32 heads of 32768 tokens 40 us instead of 29)
  const int holes = find_moves<ALL ? 8 : 32>(a, cut, hist, share);
  if constexpr (ALL) {
    __syncthreads();
    Teams<NC>::move(a, cut, holes, threadIdx.x / Teams<NC>::kLanes, kThreads / Teams<NC>::kLanes);
    __syncthreads();
    Teams<NC>::template shift<kThreads>(a, cut, 0, 1);
  } else if (threadIdx.x == 0) {
    a.counts[blockIdx.x] = holes;
  }
}

// The second and third launch: what the first has found.
__device__ __forceinline__ Cut found_cut(const KvEvictArgs& a, int bh) {
  Cut c;
  c.b = bh / a.c.H;
  c.h = bh - c.b * a.c.H;
  c.whole = false;
  const int cap = a.c.W * a.c.P, len = a.c.lens[c.b];
  c.n = len > cap ? cap : len;
  c.acc = a.acc + (int64_t)bh * cap;
  c.moves = a.moves + (int64_t)bh * (a.budget - a.recent);
  c.rows = Rows{a.c.table + (int64_t)c.b * a.c.W, a.c.H, c.h, a.c.P, a.c.by_page};
  return c;
}

template <int NC>
__global__ __launch_bounds__(256) void k_kv_move(KvEvictArgs a) {
  const int holes = a.counts[blockIdx.x];
  constexpr int kTeams = 256 / Teams<NC>::kLanes;
  if ((int)blockIdx.y * kTeams >= holes) return;
  Teams<NC>::move(a, found_cut(a, blockIdx.x), holes, blockIdx.y * kTeams + threadIdx.x / Teams<NC>::kLanes, gridDim.y * kTeams);
}

template <int NC>
__global__ __launch_bounds__(256) void k_kv_shift(KvEvictArgs a) {
  if (a.counts[blockIdx.x] < 0) return;
  Teams<NC>::template shift<256>(a, found_cut(a, blockIdx.x), blockIdx.y, gridDim.y);
}

// Three launches where there may be many moves and one workgroup to a head leaves the chip
// idle or reads its weights often (it holds 8192 of them, 32768 with the search alone).
// One launch and three, heads of 128, us: 8 heads, 1024 kept of 2304 rows 19.5 and 22.7,
// 1536 of 8192 31.1 and 28.5, 4096 of 8192 39.7 and 27.2; 128 heads, 2048 of 8192 44.7 and
// 46.6, 2048 of 32768 102 and 88. Few moves of a long sequence would gain too (8 heads,
// 1024 of 32768: 59 and 44), but the host knows the table's width, not the lengths, and
// short sequences under a wide table would lose (640 rows: 13.1 and 21.8).
template <int NC>
void evict(const KvEvictArgs& a, hipStream_t s) {
  const unsigned heads = (unsigned)(a.c.B * a.c.H);
  const int keep = a.budget - a.recent;
  const int64_t cap = (int64_t)a.c.W * a.c.P;
  if (min((int64_t)keep - a.sinks, cap - a.budget) <= 1024 || (heads >= 128 && cap <= 16384)) {
    k_kv_evict<NC, true><<<heads, kThreads, 0, s>>>(a);
    return;
  }
  const int each = 256 / Teams<NC>::kLanes * Teams<NC>::kRows;
  k_kv_evict<NC, false><<<heads, kThreads, 0, s>>>(a);
  k_kv_move<NC><<<dim3(heads, (unsigned)min((keep + each - 1) / each, 64)), 256, 0, s>>>(a);
  k_kv_shift<NC><<<dim3(heads, 4), 256, 0, s>>>(a);
}

}  // namespace

hipError_t launch_kv_check(const KvCache& c, const int32_t* offs, int32_t* status, hipStream_t s) {
  if (!status) return hipSuccess;
  k_kv_check<<<1, 256, 0, s>>>(c, offs, status);
  return hipGetLastError();
}

hipError_t launch_kv_append(int dt, const KvAppendArgs& a, hipStream_t s) {
  const int blocks = a.c.D / 16;
  const int sh = blocks <= 2 ? 1 : blocks <= 4 ? 2 : blocks <= 8 ? 3 : 4;
  const int64_t rows = (int64_t)a.T * a.c.H, per = 4 * (64 >> sh);
  const dim3 grid((unsigned)((rows + per - 1) / per), 2);
  if (dt == kBF16) append<kBF16>(a, grid, s);
  else if (dt == kFP16) append<kFP16>(a, grid, s);
  else append<kFP32>(a, grid, s);
  return hipGetLastError();
}

hipError_t launch_kv_evict(const KvEvictArgs& a, hipStream_t s) {
  switch (a.c.D / 32) {
    case 1: evict<1>(a, s); break;
    case 2: evict<2>(a, s); break;
    case 3: evict<3>(a, s); break;
    case 4: evict<4>(a, s); break;
    case 6: evict<6>(a, s); break;
    case 8: evict<8>(a, s); break;
  }
  return hipGetLastError();
}

}  // namespace fos
