// fos_linear.hip: products of activations with NVFP4 weights, with bias,
// activation and residual in the epilogue, dense and by groups of rows.
//
//   y[m, n] = act(Sx[m] * Sw[n] * sum_k x[m, k] * c[n, k] * b[n, k/16] + bias[n]) + res[m, n]
//
// c is an E2M1 value (2 significant bits), b an E4M3 scale (4), so c * b has
// at most 6 significant bits and lies between 2^-10 and 2688 (or is 0): it is
// exact in fp16 and in bf16. The weight is therefore decoded, without a
// rounding, to the 16-bit type that the matrix instruction takes beside the
// activations (bf16 for bf16 activations, fp16 otherwise; E4M3 and NVFP4
// activations are exact in fp16 too). Products of two 16-bit values are exact
// in binary32 and sums are held in binary32; the float32 scales of rows and
// columns are applied once, to the sum.
//
// The matrix instruction 16x16x32 takes, from lane l, eight values along k of
// row l % 16 of each operand, and any assignment of k to (lane, element) will
// do as long as both operands use the same. Here lane l owns the 16-value
// blocks 2g and 2g + 1 (g = l / 16) of a 128-deep step: one 16-byte load of
// codes, one 2-byte load of scales, four instructions. The weight is the first
// operand, so a lane's four sums are four neighbouring columns of one row of y.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fos_device.h"
#include "fos_ops.h"

namespace fos {
namespace {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef __bf16 b2 __attribute__((ext_vector_type(2)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// Eight 16-bit values along k of one row.
union Frag {
  uint32_t u[4];
  h8 h;
  b8 b;
};

// Loads of rows whose start is only as aligned as K % 16 == 0 makes it.
struct __attribute__((packed, aligned(8))) Bytes16 {
  uint32_t v[4];
};
struct __attribute__((packed, aligned(1))) Bytes2 {
  uint16_t v;
};

__device__ __forceinline__ uint32_t bits(h2 v) { return __builtin_bit_cast(uint32_t, v); }

// Eight codes of a dword times one block scale, as fp16 / bf16 pairs.
template <bool BF16>
__device__ __forceinline__ void decode8(uint32_t codes, float s, h2 s16, uint32_t* out) {
  if constexpr (BF16) {
#define FOS_PAIR(i)                                                              \
  {                                                                              \
    const f32x2 p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, i);    \
    const f32x2 q = {p.x * s, p.y * s};                                          \
    out[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(q, b2));       \
  }
    FOS_PAIR(0) FOS_PAIR(1) FOS_PAIR(2) FOS_PAIR(3)
#undef FOS_PAIR
  } else {
    out[0] = bits(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 0) * s16);
    out[1] = bits(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 1) * s16);
    out[2] = bits(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 2) * s16);
    out[3] = bits(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 3) * s16);
  }
}

// Two neighbouring blocks (16 bytes of codes, two scale bytes) to four fragments.
template <bool BF16>
__device__ __forceinline__ void decode_blocks(const uint32_t* codes, uint32_t scales, Frag* f) {
  const f32x2 s = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((int)scales, 1.0f, false);
  const h2 s16 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)scales, 1.0f, false);
  const h2 lo = __builtin_shufflevector(s16, s16, 0, 0), hi = __builtin_shufflevector(s16, s16, 1, 1);
  decode8<BF16>(codes[0], s.x, lo, f[0].u);
  decode8<BF16>(codes[1], s.x, lo, f[1].u);
  decode8<BF16>(codes[2], s.y, hi, f[2].u);
  decode8<BF16>(codes[3], s.y, hi, f[3].u);
}

// NVFP4 blocks b and b + 1 of a row with KB blocks; those past its end are zero.
template <bool BF16>
__device__ __forceinline__ void load_nvfp4(const uint8_t* codes, const uint8_t* scales, int64_t b, int64_t KB,
                                           Frag* f) {
  uint32_t c[4] = {0, 0, 0, 0}, s = 0;
  if (b + 1 < KB) {
    const Bytes16 t = *reinterpret_cast<const Bytes16*>(codes + 8 * b);
    for (int i = 0; i < 4; i++) c[i] = t.v[i];
    s = reinterpret_cast<const Bytes2*>(scales + b)->v;
  } else if (b < KB) {
    const uint2 t = *reinterpret_cast<const uint2*>(codes + 8 * b);
    c[0] = t.x;
    c[1] = t.y;
    s = scales[b];
  }
  decode_blocks<BF16>(c, s, f);
}

// 32 activations of one row from block b on, as four fragments.
template <int XT>
__device__ __forceinline__ void load_x(const LinearArgs& a, int64_t m, int64_t b, int64_t KB, Frag* f) {
  if constexpr (XT == kXNVFP4) {
    load_nvfp4<false>((const uint8_t*)a.x + m * (a.K / 2), a.xs + m * KB, b, KB, f);
  } else if constexpr (XT == kXE4M3) {
    const uint4* p = reinterpret_cast<const uint4*>((const uint8_t*)a.x + m * a.K + 16 * b);
#pragma unroll
    for (int i = 0; i < 2; i++) {
      uint4 t = {0, 0, 0, 0};
      if (b + i < KB) t = p[i];
      const uint32_t v[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
      for (int j = 0; j < 4; j++) {
        f[2 * i + j / 2].u[2 * (j & 1)] = bits(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)v[j], 1.0f, false));
        f[2 * i + j / 2].u[2 * (j & 1) + 1] = bits(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)v[j], 1.0f, true));
      }
    }
  } else {
    const uint4* p = reinterpret_cast<const uint4*>((const uint16_t*)a.x + m * a.K + 16 * b);
#pragma unroll
    for (int i = 0; i < 4; i++) {
      uint4 t = {0, 0, 0, 0};
      if (b + i / 2 < KB) t = p[i];
      f[i].u[0] = t.x;
      f[i].u[1] = t.y;
      f[i].u[2] = t.z;
      f[i].u[3] = t.w;
    }
  }
}

template <bool BF16>
__device__ __forceinline__ f32x4 mfma(const Frag& w, const Frag& x, f32x4 c) {
  if constexpr (BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.b, x.b, c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(w.h, x.h, c, 0, 0, 0);
}

// ---------------------------------------------------------------- groups

// What a workgroup works on: rows [m0, end) of x with weight g; g < 0: no
// such tile; g == G: the tail past the last group, which is written as zero.
struct RowTile {
  int64_t m0, end;
  int g;
};

// Tile `t` of the rows cut into groups and each group into tiles of `rows`
// rows, in group order, the tail last. The wave holds 64 groups' offsets at a
// time, one per lane, and finds the tile by a running sum of the groups' tile
// counts. Offsets are clamped to [previous, M], so a bad one sends no access
// out of bounds.
__device__ RowTile find_tile(const int32_t* offs, int G, int64_t M, int64_t rows, int64_t t) {
  const int lane = threadIdx.x & 63;
  int64_t prev = 0, tiles = 0;  // of the groups before this batch
  for (int base = 0; base <= G; base += 64) {
    const int g = base + lane;
    const bool have = g <= G;
    // running maximum of the ends, clamped
    int64_t run = g < G ? (int64_t)offs[g] : g == G ? M : 0;
    if (run > M) run = M;
    if (run < prev) run = prev;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t o = __shfl_up(run, d, 64);
      if (lane >= d && o > run) run = o;
    }
    int64_t start = __shfl_up(run, 1, 64);
    if (lane == 0) start = prev;
    const int64_t n = have ? (run - start + rows - 1) / rows : 0;
    int64_t sum = n;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t o = __shfl_up(sum, d, 64);
      if (lane >= d) sum += o;
    }
    const unsigned long long hit = __ballot(tiles + sum > t);
    if (hit) {
      const int l = __ffsll(hit) - 1;
      const int64_t first = tiles + __shfl(sum - n, l, 64);
      RowTile r;
      r.m0 = __shfl(start, l, 64) + (t - first) * rows;
      r.end = __shfl(run, l, 64);
      r.g = base + l;
      return r;
    }
    tiles += __shfl(sum, 63, 64);
    prev = __shfl(run, 63, 64);
  }
  return RowTile{0, 0, -1};
}

// The first wave of a launch reports offsets that break the contract.
__device__ void check_offs(const LinearArgs& a) {
  bool bad = false;
  for (int g = threadIdx.x & 63; g < a.G; g += 64) {
    const int32_t e = a.offs[g], p = g ? a.offs[g - 1] : 0;
    bad |= e < p || e > a.M;
  }
  if (bad) atomicOr(a.status, kStatusBadOffs);
}

// ---------------------------------------------------------------- epilogue

__device__ __forceinline__ float to_f32(const void* p, int dt, int64_t i) {
  if (dt == kFP32) return ((const float*)p)[i];
  const uint16_t v = ((const uint16_t*)p)[i];
  return dt == kBF16 ? __uint_as_float((uint32_t)v << 16) : (float)__builtin_bit_cast(_Float16, v);
}

__device__ __forceinline__ float activate(int act, float v) {
  switch (act) {
    case kActRelu: return v > 0.0f ? v : v != v ? v : 0.0f;
    case kActGelu: return 0.5f * v * erfcf(v * -0.70710678118654752f);
    case kActGeluTanh: {
      // 0.5 (1 + tanh u) = 1 / (1 + exp(-2u))
      const float u = 0.79788456080286536f * __builtin_fmaf(0.044715f * v * v, v, v);
      return v / (1.0f + expf(-2.0f * u));
    }
    case kActSilu: return v / (1.0f + expf(-v));
    default: return v;
  }
}

// Finish columns n .. n + 3 of row m from their sums and store them. The sum
// is rounded to the output type once, after the residual.
__device__ __forceinline__ void finish4(const LinearArgs& a, int g, int64_t m, int64_t n, f32x4 acc) {
  const float sx = a.x_gran == kScaleNone ? 1.0f : a.x_scale[a.x_gran == kScaleRow ? m : a.x_gran == kScaleGroup ? g : 0];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int64_t c = n + i;
    if (c >= a.N) break;
    const float sw = a.w_scale[a.w_gran == kScaleRow ? (int64_t)g * a.N + c : a.w_gran == kScaleGroup ? g : 0];
    float v = acc[i] * (sx * sw);
    if (a.bias) v += to_f32(a.bias, a.bias_dt, (int64_t)g * a.N + c);
    v = activate(a.act, v);
    const int64_t at = m * a.N + c;
    if (a.res) v += to_f32(a.res, a.out_dt, at);
    if (a.out_dt == kFP32)
      ((float*)a.y)[at] = v;
    else
      ((uint16_t*)a.y)[at] = (uint16_t)(a.out_dt == kBF16 ? pack_bf16(v, 0.0f) : pack_f16(v, 0.0f));
  }
}

__device__ __forceinline__ void zero4(const LinearArgs& a, int64_t m, int64_t n) {
  for (int i = 0; i < 4 && n + i < a.N; i++) {
    if (a.out_dt == kFP32)
      ((float*)a.y)[m * a.N + n + i] = 0.0f;
    else
      ((uint16_t*)a.y)[m * a.N + n + i] = 0;
  }
}

// ---------------------------------------------------------------- kernels

// One workgroup: 16 columns of y and 16 * MT rows. Its waves take the 128-deep
// steps of k in turn and their sums are joined through LDS in wave order.
template <int XT, int MT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_linear_stream(LinearArgs a, int n_tiles) {
  constexpr bool BF16 = XT == kBF16;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = blockIdx.x / n_tiles;
  const int64_t n0 = 16 * (int64_t)(blockIdx.x % n_tiles);
  RowTile rt{t * 16 * MT, a.M, 0};
  if (a.offs) {
    if (a.status && blockIdx.x == 0 && wave == 0) check_offs(a);
    rt = find_tile(a.offs, a.G, a.M, 16 * MT, t);
    if (rt.g < 0) return;
  }
  const int col = lane & 15, g4 = lane >> 4;
  const bool tail = a.offs && rt.g == a.G;
  const int64_t KB = a.K / 16;
  f32x4 acc[MT] = {};
  if (!tail) {
    const int64_t n = n0 + col < a.N ? n0 + col : a.N - 1;
    const int64_t row = (int64_t)rt.g * a.N + n;
    const uint8_t* wc = a.w + row * (a.K / 2);
    const uint8_t* wsc = a.ws + row * KB;
    for (int64_t b = 8 * wave; b < KB; b += 8 * WAVES) {
      Frag w[4];
      load_nvfp4<BF16>(wc, wsc, b + 2 * g4, KB, w);
#pragma unroll
      for (int i = 0; i < MT; i++) {
        int64_t m = rt.m0 + 16 * i + col;
        if (m >= rt.end) m = rt.end - 1;
        Frag x[4];
        load_x<XT>(a, m, b + 2 * g4, KB, x);
#pragma unroll
        for (int j = 0; j < 4; j++) acc[i] = mfma<BF16>(w[j], x[j], acc[i]);
      }
    }
  }
  __shared__ f32x4 part[WAVES][MT][64];
#pragma unroll
  for (int i = 0; i < MT; i++) part[wave][i][lane] = acc[i];
  __syncthreads();
  for (int i = wave; i < MT; i += WAVES) {
    f32x4 s = part[0][i][lane];
    for (int v = 1; v < WAVES; v++) s += part[v][i][lane];
    const int64_t m = rt.m0 + 16 * i + col, n = n0 + 4 * g4;
    if (m < rt.end && n < a.N) {
      if (tail)
        zero4(a, m, n);
      else
        finish4(a, rt.g, m, n, s);
    }
  }
}

constexpr int64_t kMaxGrid = INT32_MAX;

// The most tiles of `rows` rows that M rows in G groups and a tail can need:
// each non-empty group may end inside a tile.
int64_t max_tiles(int64_t M, int64_t G, int64_t rows) {
  const int64_t parts = G + 1 < M ? G + 1 : M;
  return (M + parts * (rows - 1)) / rows;
}

template <int XT>
hipError_t launch_type(const LinearArgs& a, hipStream_t s) {
  constexpr int WAVES = 8;
  const int64_t nt = (a.N + 15) / 16;
  const int64_t mt = a.offs ? max_tiles(a.M, a.G, 16) : (a.M + 15) / 16;
  if (mt > kMaxGrid / nt) return hipErrorInvalidConfiguration;
  k_linear_stream<XT, 1, WAVES><<<dim3((unsigned)(mt * nt)), dim3(64 * WAVES), 0, s>>>(a, (int)nt);
  return hipGetLastError();
}

}  // namespace

int64_t linear_workspace(int64_t, int64_t, int64_t, int) { return 0; }

hipError_t launch_linear(const LinearArgs& a, hipStream_t s) {
  switch (a.x_type) {
    case kBF16: return launch_type<kBF16>(a, s);
    case kFP16: return launch_type<kFP16>(a, s);
    case kXE4M3: return launch_type<kXE4M3>(a, s);
    default: return launch_type<kXNVFP4>(a, s);
  }
}

}  // namespace fos
