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
// blocks 2g and 2g + 1 (g = l / 16) of a 128-deep step: 16 bytes of codes, two
// scale bytes, four instructions. The weight is the first operand, so a lane's
// four sums are four neighbouring columns of one row of y.
//
// What bounds it: few rows, the weights' way from memory (64 experts of 2048 x
// 7168 at decode: 297 MB in 73 us, 4.1 TB/s where a copy reaches 5.0); many
// rows, the matrix units at the clock that the power limit leaves (8192 x 4096 x
// 14336: 1.2 to 1.3 PFLOP/s; a loop of matrix instructions alone reaches 1.88,
// the library's 16-bit product 1.45 to 1.53 without the decode).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fos_device.h"
#include "fos_ops.h"
#include "fos_plan.h"

namespace fos {
namespace {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef __bf16 b2 __attribute__((ext_vector_type(2)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
// the same at the alignment that a tensor's rows give
typedef f32x4 f32x4_a4 __attribute__((aligned(4)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef u32x4 u32x4_a8 __attribute__((aligned(8)));
typedef u32x2 u32x2_a2 __attribute__((aligned(2)));
typedef u32x2 u32x2_a1 __attribute__((aligned(1)));
typedef uint16_t u16_a1 __attribute__((aligned(1)));

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
// of bounds. M is at most 2^30, so row and tile counts fit an int.
__device__ RowTile find_tile(const int32_t* offs, int G, int M, int rows, int t) {
  const int lane = threadIdx.x & 63;
  int prev = 0, tiles = 0;  // of the groups before this batch
  for (int base = 0; base <= G; base += 64) {
    const int g = base + lane;
    const bool have = g <= G;
    int end = g < G ? offs[g] : M;
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
    const int n = have ? (int)((uint32_t)(end - start + rows - 1) / (uint32_t)rows) : 0;
    const int sum = wave_scan(n);
    const unsigned long long hit = __ballot(tiles + sum > t);
    if (hit) {
      const int l = __ffsll(hit) - 1;
      const int first = tiles + __builtin_amdgcn_readlane(sum - n, l);
      RowTile r;
      r.m0 = (int64_t)__builtin_amdgcn_readlane(start, l) + (int64_t)(t - first) * rows;
      r.end = __builtin_amdgcn_readlane(end, l);
      r.g = base + l;
      return r;
    }
    tiles += __builtin_amdgcn_readlane(sum, 63);
    prev = __builtin_amdgcn_readlane(end, 63);
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

__global__ __launch_bounds__(64) void k_check_offs(LinearArgs a) { check_offs(a); }

// ---------------------------------------------------------------- epilogue

// exp(v) by the base-2 instruction: off by about 1.5 |v| half steps.
__device__ __forceinline__ float exp_fast(float v) { return __builtin_amdgcn_exp2f(v * 1.44269504088896341f); }

// Activations of the epilogue, by the reciprocal and exponential instructions,
// which are good to a step of binary32. Their relative errors grow with the
// exponential's argument: 1.3 v^2 half steps and ten more for gelu, which is
// below a 16-bit output's rounding wherever that is not 0 (the library's erfc
// takes several times the instructions).
//
// erfc(z) exp(z^2) / 2 is t p(t) with t = 1 / (1 + 0.4 z) and p of degree 8, fitted
// to the smallest largest relative error over all z >= 0: 1.3e-7. No difference
// of two numbers near 1 is taken, so small results keep their bits.
__device__ __forceinline__ float gelu(float v) {
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.4f * 0.70710678118654752f, __builtin_fabsf(v), 1.0f));
  float p = __builtin_fmaf(t, 0.025128307f, -0.09144085f);
  p = __builtin_fmaf(t, p, 0.08452848f);
  p = __builtin_fmaf(t, p, -0.0027932455f);
  p = __builtin_fmaf(t, p, 0.07071148f);
  p = __builtin_fmaf(t, p, 0.0842719f);
  p = __builtin_fmaf(t, p, 0.10392126f);
  p = __builtin_fmaf(t, p, 0.112834804f);
  p = __builtin_fmaf(t, p, 0.11283793f);
  const float half_erfc = t * p * exp_fast(-0.5f * v * v);  // of |v| / sqrt 2
  return v * (v < 0.0f ? half_erfc : 1.0f - half_erfc);
}
__device__ __forceinline__ float gelu_tanh(float v) {
  // (1 + tanh u) / 2 = 1 / (1 + exp(-2u))
  const float u = 0.79788456080286536f * __builtin_fmaf(0.044715f * v * v, v, v);
  return v * __builtin_amdgcn_rcpf(1.0f + exp_fast(-2.0f * u));
}

// One branch for all values, whose chains of instructions then run side by side
// (8192 x 4096 x 4096 bf16 with gelu: a branch per value took 3 % longer).
template <int R>
__device__ __forceinline__ void activate(int act, f32x4 (&v)[R]) {
  auto each = [&](auto f) {
#pragma unroll
    for (int k = 0; k < R; k++)
#pragma unroll
      for (int i = 0; i < 4; i++) v[k][i] = f(v[k][i]);
  };
  switch (act) {
    case kActRelu: return each([](float x) { return x > 0.0f ? x : x != x ? x : 0.0f; });
    case kActGelu: return each(gelu);
    case kActGeluTanh: return each(gelu_tanh);
    case kActSilu: return each([](float x) { return x * __builtin_amdgcn_rcpf(1.0f + exp_fast(-x)); });
    default: return;
  }
}

// Four neighbouring values of a tensor, `have` of which exist, as they are in
// memory: what widens them waits for them, so that comes with their use. Rows of
// any length: the accesses need no more than the elements' own alignment.
__device__ __forceinline__ u32x4 load4(const void* p, int dt, int64_t i, int have) {
  u32x4 v = {0, 0, 0, 0};
  if (dt == kFP32) {
    if (have == 4) return *reinterpret_cast<const u32x4_a4*>((const float*)p + i);
#pragma unroll
    for (int j = 0; j < 3; j++)
      if (j < have) v[j] = ((const uint32_t*)p)[i + j];
  } else if (have == 4) {
    const u32x2 t = *reinterpret_cast<const u32x2_a2*>((const uint16_t*)p + i);
    v.x = t.x, v.y = t.y;
  } else {
#pragma unroll
    for (int j = 0; j < 3; j++)
      if (j < have) v[j / 2] |= (uint32_t)((const uint16_t*)p)[i + j] << (16 * (j & 1));
  }
  return v;
}
__device__ __forceinline__ f32x4 widen4(u32x4 v, int dt) {
  if (dt == kFP32) return __builtin_bit_cast(f32x4, v);
  return dt == kBF16 ? f32x4{bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y)}
                     : f32x4{f16_lo(v.x), f16_hi(v.x), f16_lo(v.y), f16_hi(v.y)};
}

// Columns n .. n + 3 and how many of them exist.
struct Quad {
  int64_t n;
  int have;
  __device__ __forceinline__ Quad(const LinearArgs& a, int64_t col) {
    n = col;
    have = col >= a.N ? 0 : a.N - col < 4 ? (int)(a.N - col) : 4;
  }
};

// What the epilogue needs of four columns of weight g, and of a row: loaded
// apart from their use, so that the loads of several run together.
struct ColumnTail {
  f32x4 scale;
  u32x4 bias;
  __device__ __forceinline__ void load(const LinearArgs& a, int g, const Quad& q) {
    scale = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    bias = u32x4{0, 0, 0, 0};
    if (q.have == 0) return;
    const int64_t at = (int64_t)g * a.N + q.n;
    if (a.w_gran == kScaleRow)
      scale = __builtin_bit_cast(f32x4, load4(a.w_scale, kFP32, at, q.have));
    else
      scale = f32x4{1.0f, 1.0f, 1.0f, 1.0f} * a.w_scale[a.w_gran == kScaleGroup ? g : 0];
    if (a.bias) bias = load4(a.bias, a.bias_dt, at, q.have);
  }
};
// R rows m, m + step ...; those past `last` take the last one's. SX: whether x
// may have a scale.
template <bool SX, int R>
struct RowTails {
  float scale[R];
  u32x4 res[R];
  __device__ __forceinline__ void load(const LinearArgs& a, int g, int m, int step, int last, const Quad& q) {
    auto each = [&](auto f) {
#pragma unroll
      for (int k = 0; k < R; k++) f(k, (int64_t)min(m + k * step, last));
    };
    each([&](int k, int64_t) { scale[k] = 1.0f, res[k] = u32x4{0, 0, 0, 0}; });
    if (SX && a.x_gran == kScaleRow) {
      each([&](int k, int64_t r) { scale[k] = a.x_scale[r]; });
    } else if (SX && a.x_gran != kScaleNone) {
      const float s = a.x_scale[a.x_gran == kScaleGroup ? g : 0];
      each([&](int k, int64_t) { scale[k] = s; });
    }
    if (!a.res) return;
    if (q.have < 4)
      each([&](int k, int64_t r) { res[k] = load4(a.res, a.out_dt, r * a.N + q.n, q.have); });
    else if (a.out_dt == kFP32)
      each([&](int k, int64_t r) { res[k] = load4(a.res, kFP32, r * a.N + q.n, 4); });
    else
      each([&](int k, int64_t r) { res[k] = load4(a.res, kBF16, r * a.N + q.n, 4); });
  }
};

// Finish four columns of rows m, m + step ... up to `last` from their sums and
// store them. The sum is rounded to the output type once, after the residual.
template <bool SX, int R>
__device__ __forceinline__ void finish(const LinearArgs& a, int m, int step, int last, const Quad& q,
                                       const ColumnTail& ct, const RowTails<SX, R>& rt, f32x4 (&v)[R]) {
  auto each = [&](auto f) {
#pragma unroll
    for (int k = 0; k < R; k++) f(k);
  };
  if (!SX || a.x_gran == kScaleNone) {
    each([&](int k) { v[k] *= ct.scale; });
  } else {
    // The product of two scales may leave binary32's range though the result does
    // not. A sum of decoded values is 0 or between 2^-20 and 2^45: it takes both
    // mantissas, then the exponents at once. (The columns' parts are taken anew for
    // each row: kept, they spill. 64 experts of 240 rows: 576 us, 570 with the
    // scales' product in binary32.)
    each([&](int k) {
      const int e = __builtin_amdgcn_frexp_expf(rt.scale[k]);
      const float m = __builtin_amdgcn_frexp_mantf(rt.scale[k]);
#pragma unroll
      for (int i = 0; i < 4; i++) {
        float c = ct.scale[i];
        asm volatile("" : "+v"(c));
        v[k][i] = __builtin_ldexpf(v[k][i] * (m * __builtin_amdgcn_frexp_mantf(c)), e + __builtin_amdgcn_frexp_expf(c));
      }
    });
  }
  if (a.bias) {
    const f32x4 bias = widen4(ct.bias, a.bias_dt);
    each([&](int k) { v[k] += bias; });
  }
  activate(a.act, v);
  if (a.out_dt == kFP32) {
    if (a.res) each([&](int k) { v[k] += widen4(rt.res[k], kFP32); });
    each([&](int k) {
      if (m + k * step > last) return;
      float* y = (float*)a.y + (int64_t)(m + k * step) * a.N + q.n;
      if (q.have == 4) {
        *reinterpret_cast<f32x4_a4*>(y) = v[k];
      } else {
#pragma unroll
        for (int i = 0; i < 3; i++)
          if (i < q.have) y[i] = v[k][i];
      }
    });
    return;
  }
  u32x2 w[R];
  if (a.out_dt == kBF16) {
    if (a.res) each([&](int k) { v[k] += widen4(rt.res[k], kBF16); });
    each([&](int k) { w[k] = u32x2{pack_bf16(v[k][0], v[k][1]), pack_bf16(v[k][2], v[k][3])}; });
  } else {
    if (a.res) each([&](int k) { v[k] += widen4(rt.res[k], kFP16); });
    each([&](int k) { w[k] = u32x2{pack_f16(v[k][0], v[k][1]), pack_f16(v[k][2], v[k][3])}; });
  }
  each([&](int k) {
    if (m + k * step > last) return;
    uint16_t* y = (uint16_t*)a.y + (int64_t)(m + k * step) * a.N + q.n;
    if (q.have == 4) {
      *reinterpret_cast<u32x2_a2*>(y) = w[k];
    } else {
#pragma unroll
      for (int i = 0; i < 3; i++)
        if (i < q.have) y[i] = (uint16_t)(w[k][i / 2] >> (16 * (i & 1)));
    }
  });
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

// Loads of the kernels' loops: a uniform address in scalar registers plus a
// 32-bit lane offset (K is at most 2^22, so 256 rows are within reach). Left to
// itself the compiler carries a 64-bit address per lane and load through the
// loop: 24 registers that spill. The alignments are those that K % 16 == 0 gives.
#define FOS_GLOBAL __attribute__((address_space(1)))
typedef const FOS_GLOBAL uint8_t* GlobalBytes;

__device__ __forceinline__ uint32_t lane_offset(uint32_t v) {  // stays 32 bits wide in the loop
  asm volatile("" : "+v"(v));
  return v;
}
__device__ __forceinline__ GlobalBytes scalar(const uint8_t* p) {
  GlobalBytes g = (GlobalBytes)p;
  asm volatile("" : "+s"(g));
  return g;
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

// Where the LDS tiles keep a row's 16-byte chunks. LDS serves a 16-byte read of
// 16 lanes at a time, but not of 16 neighbours: lanes 0-3 and 12-15 go with
// 20-27, and 4-11 with 16-19 and 28-31 (the same in the upper half). With lane l
// reading row l % 16 that is every row once, half of them one group of 16 lanes
// further on, at another chunk. Chunk c of row r stands at c ^ swizzle(r), where
// the two halves of the rows get different values of the bit that the chunk
// numbers of the two groups do not differ in; then all 16 places differ. (Plain
// c ^ r met every place twice: 41% of the tile kernel's LDS cycles.)
// BITS: log2 of the chunks in a row; with fewer than 16 the rows that share the
// 256 bytes count too.
template <int BITS>
__device__ __forceinline__ int swizzle(int r) {
  const int v = (r & 15) >> (4 - BITS);
  return v ^ ((v & (1 << (BITS - 2))) << 1);
}

// A 128-deep step of 16 rows of activations on its way through one wave: loaded
// with neighbouring lanes in the same row (16 lanes to a row of 16-bit values, 8
// of E4M3, 4 of NVFP4 codes), put into the wave's own piece of LDS as it is, and
// read back as the matrix instruction wants it, lane l the 32 values of its
// blocks 2g and 2g + 1 of row l % 16. Chunks of 16 bytes are swizzled so that the 16 rows that
// are read together lie in 16 different places of the 256 bytes that LDS serves
// at a time.
template <int XT>
struct XTile {
  static constexpr int kLanes = XT == kXE4M3 ? 8 : XT == kXNVFP4 ? 4 : 16;  // per row
  static constexpr int kLoads = kLanes / 4;                                  // of 64 / kLanes rows
  static constexpr int kBytes = 16 * 16 * kLanes;
  u32x4 v[kLoads];
  u32x2 s;

  static __device__ __forceinline__ int slot(int row, int chunk) {
    return row * 16 * kLanes + ((chunk ^ swizzle<kLanes == 16 ? 4 : kLanes == 8 ? 3 : 2>(row)) << 4);
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kLoads; i++) v[i] = u32x4{0, 0, 0, 0};
    s = u32x2{0, 0};
  }
  // Lane offsets of the first load and of the scales, from row 0.
  static __device__ __forceinline__ uint32_t offset(int64_t KB) {
    const int lane = threadIdx.x & 63;
    return (uint32_t)(lane / kLanes) * (uint32_t)(KB * 2 * kLanes) + 16 * (lane % kLanes);
  }
  static __device__ __forceinline__ uint32_t scale_offset(int64_t KB) { return (threadIdx.x & 15) * (uint32_t)KB; }
  // p: row 0 of the tile at the step; q: its scales; rows: how many exist. Rows
  // that do not keep what clear() put there.
  __device__ __forceinline__ void load(const uint8_t* p, const uint8_t* q, uint32_t off, uint32_t soff, int64_t KB, int rows) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < kLoads; i++) {
      const GlobalBytes g = scalar(p + i * (64 / kLanes) * (KB * 2 * kLanes));
      if (i * (64 / kLanes) + lane / kLanes < rows) v[i] = *(const FOS_GLOBAL u32x4_a8*)(g + lane_offset(off));
    }
    if constexpr (XT == kXNVFP4) {
      const GlobalBytes g = scalar(q);
      if ((lane & 15) < rows) s = *(const FOS_GLOBAL u32x2_a1*)(g + lane_offset(soff));
    }
  }
  __device__ __forceinline__ void put(uint8_t* lds) const {
    const int lane = threadIdx.x & 63;
    wave_lds_order();
#pragma unroll
    for (int i = 0; i < kLoads; i++)
      *reinterpret_cast<u32x4*>(lds + slot(i * (64 / kLanes) + lane / kLanes, lane % kLanes)) = v[i];
    wave_lds_order();
  }
  // (scales: this lane's two bytes, from row_scales of s)
  static __device__ __forceinline__ void get(const uint8_t* lds, uint32_t scales, Frag* f) {
    const int lane = threadIdx.x & 63, col = lane & 15, g4 = lane >> 4;
    u32x4 t[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; i++) t[i] = *reinterpret_cast<const u32x4*>(lds + slot(col, kLoads * g4 + i));
    if constexpr (XT == kXNVFP4) {
      const uint32_t c[4] = {t[0][0], t[0][1], t[0][2], t[0][3]};
      decode_blocks<false>(c, scales, f);
    } else if constexpr (XT == kXE4M3) {
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const int w = (int)t[j / 4][j % 4];
        f[j / 2].u[2 * (j & 1)] = bits(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false));
        f[j / 2].u[2 * (j & 1) + 1] = bits(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) f[i].u[j] = t[i][j];
    }
  }
};

// Scale bytes 2 g and 2 g + 1 of row l % 16, where lane `from + row` holds the
// eight bytes of a row.
__device__ __forceinline__ uint32_t row_scales(u32x2 s, int from) {
  const int lane = threadIdx.x & 63, g4 = lane >> 4;
  const uint32_t lo = __builtin_amdgcn_ds_bpermute(4 * (from + (lane & 15)), s[0]);
  const uint32_t hi = __builtin_amdgcn_ds_bpermute(4 * (from + (lane & 15)), s[1]);
  return (g4 < 2 ? lo : hi) >> (16 * (g4 & 1));
}

// The stream kernel, for few rows per weight: one workgroup takes 16 NT columns
// of y and 16 MT rows, and its waves take the 128-deep steps of k in turn, so
// that the weight is read once by as many waves as the chip has. A wave keeps
// DEPTH steps of the weight's loads in flight. Like the activations, the weights
// are loaded four lanes to a row and turned through the wave's own LDS: a load
// costs a cycle for every row that four consecutive lanes touch (16 x 4096 x
// 14336: 21 us with a row per lane, 14 so). The waves' sums are joined through
// LDS in wave order. 1 x 4096 x 14336 bf16: 10.2 us, 3.2 TB/s; 64 x 14336 x 4096:
// 21 us.
template <int XT, int MT, int NT, int WAVES>
__global__ __launch_bounds__(64 * WAVES, MT == 1 ? 4 : 2) void k_linear_stream(LinearArgs a, int n_tiles) {
  constexpr bool BF16 = XT == kBF16, SX = XT == kXE4M3 || XT == kXNVFP4;
  constexpr int DEPTH = stream_depth(MT, NT);
  static_assert(WAVES == stream_waves(MT, NT));
  constexpr int kWaveBytes = NT * 1024 + XTile<XT>::kBytes;
  constexpr int kPartBytes = (NT > 1 ? 2 : 1) * WAVES * MT * 1024;
  __shared__ __align__(16) uint8_t lds[kPartBytes > WAVES * kWaveBytes ? kPartBytes : WAVES * kWaveBytes];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = blockIdx.x / (uint32_t)n_tiles;
  const int64_t n0 = 16 * NT * (int64_t)(blockIdx.x % (uint32_t)n_tiles);
  RowTile rt{t * 16 * MT, a.M, 0};
  if (a.offs) {
    if (a.status && blockIdx.x == 0 && wave == 0) check_offs(a);
    rt = find_tile(a.offs, a.G, (int)a.M, 16 * MT, (int)t);
    if (rt.g < 0) return;
  }
  const int col = lane & 15, g4 = lane >> 4;
  if (a.offs && rt.g == a.G) {
    for (int i = wave; i < MT * NT; i += WAVES) {
      const int64_t m = rt.m0 + 16 * (i % MT) + col, n = n0 + 16 * (i / MT) + 4 * g4;
      if (m < rt.end) zero4(a, m, n);
    }
    return;
  }
  const int64_t KB = a.K / 16;
  const int whole = (int)(KB / 8);  // 128-deep steps; a part of one may follow
  f32x4 acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; i++)
#pragma unroll
    for (int j = 0; j < MT; j++) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  // columns past the end read the last row of the weight
  const int wrows = a.N - n0 < 16 * NT ? (int)(a.N - n0) : 16 * NT;
  const int64_t w0 = (int64_t)rt.g * a.N + n0;
  const uint8_t *wc = a.w + w0 * (a.K / 2), *wsc = a.ws + w0 * KB;
  uint32_t woff[NT];
#pragma unroll
  for (int i = 0; i < NT; i++) {
    const int r = 16 * i + (lane >> 2);
    woff[i] = (uint32_t)(r < wrows ? r : wrows - 1) * (uint32_t)(a.K / 2) + 16 * (lane & 3);
  }
  const uint32_t wsoff = (uint32_t)(lane < wrows ? lane : wrows - 1) * (uint32_t)KB;
  const int xrows = rt.end - rt.m0 < 16 * MT ? (int)(rt.end - rt.m0) : 16 * MT;
  const uint8_t* xc = (const uint8_t*)a.x + rt.m0 * KB * (2 * XTile<XT>::kLanes);
  const uint8_t* xsc = XT == kXNVFP4 ? a.xs + rt.m0 * KB : nullptr;
  const uint32_t xoff = XTile<XT>::offset(KB), xsoff = XTile<XT>::scale_offset(KB);

  // The tiles of y that this wave will finish (row tile turn(i) of column tile
  // i, where that is below MT: one in eight), and what that takes.
  constexpr int MP = MT == 3 ? 4 : MT;  // a divisor of the waves
  auto turn = [&](int i) { return (wave + WAVES - (i * MP) % WAVES) % WAVES; };
  constexpr int TURNS = (NT * MP + WAVES - 1) / WAVES;
  ColumnTail columns[TURNS];
  RowTails<SX, 1> row[TURNS];
  bool live[TURNS] = {};
#pragma unroll
  for (int i = 0; i < NT; i++) {
    if (const int j = turn(i); j < MT) {
      const int k = i * MP / WAVES;
      const Quad q(a, n0 + 16 * i + 4 * g4);
      const int m = (int)rt.m0 + 16 * j + col;
      live[k] = m < rt.end && q.have;
      if (live[k]) {
        columns[k].load(a, rt.g, q);
        row[k].load(a, rt.g, m, 0, m, q);
      }
    }
  }

  u32x4 codes[DEPTH][NT];
  u32x2 scales[DEPTH];
  XTile<XT> x[MT];  // the activations come from L2: one step ahead is enough
#pragma unroll
  for (int j = 0; j < MT; j++) x[j].clear();
  auto load_w = [&](int d, int64_t step) {
    const GlobalBytes p = scalar(wc + step * 64), q = scalar(wsc + step * 8);
#pragma unroll
    for (int i = 0; i < NT; i++) codes[d][i] = *(const FOS_GLOBAL u32x4_a8*)(p + lane_offset(woff[i]));
    if (NT == 4 || lane < 16 * NT) scales[d] = *(const FOS_GLOBAL u32x2_a1*)(q + lane_offset(wsoff));
  };
  auto load_rows = [&](int j, int64_t step) {
    x[j].load(xc + 16 * j * KB * (2 * XTile<XT>::kLanes) + step * (16 * XTile<XT>::kLanes),
              XT == kXNVFP4 ? xsc + 16 * j * KB + step * 8 : nullptr, xoff, xsoff, KB, xrows - 16 * j);
  };
  uint8_t* wl = lds + wave * kWaveBytes;
  uint8_t* xl = wl + NT * 1024;
  // One step from the registers of stage d, which are loaded again for the step
  // that they serve next as soon as their contents are in LDS.
  auto multiply = [&](int d, int step) {
    const int after = step + DEPTH * WAVES, after_x = step + WAVES;
    uint32_t ws[NT];
    wave_lds_order();
#pragma unroll
    for (int i = 0; i < NT; i++) {
      *reinterpret_cast<u32x4*>(wl + i * 1024 + XTile<kXNVFP4>::slot(lane >> 2, lane & 3)) = codes[d][i];
      ws[i] = row_scales(scales[d], 16 * i);
    }
    wave_lds_order();
    if (after < whole) load_w(d, after);
    auto take_w = [&](int i, Frag* w) {
      const u32x4 t = *reinterpret_cast<const u32x4*>(wl + i * 1024 + XTile<kXNVFP4>::slot(col, g4));
      const uint32_t c[4] = {t[0], t[1], t[2], t[3]};
      decode_blocks<BF16>(c, ws[i], w);
    };
    auto take_x = [&](int j, Frag* f) {
      x[j].put(xl);
      const uint32_t sc = XT == kXNVFP4 ? row_scales(x[j].s, 0) : 0;
      if (after_x < whole) load_rows(j, after_x);
      XTile<XT>::get(xl, sc, f);
    };
    if constexpr (MT == 1) {  // hold the activations, not the weights
      Frag f[4];
      take_x(0, f);
#pragma unroll
      for (int i = 0; i < NT; i++) {
        Frag w[4];
        take_w(i, w);
#pragma unroll
        for (int k = 0; k < 4; k++) acc[i][0] = mfma<BF16>(w[k], f[k], acc[i][0]);
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
      Frag w[NT][4];
#pragma unroll
      for (int i = 0; i < NT; i++) take_w(i, w[i]);
#pragma unroll
      for (int j = 0; j < MT; j++) {
        Frag f[4];
        take_x(j, f);
#pragma unroll
        for (int k = 0; k < 4; k++)
#pragma unroll
          for (int i = 0; i < NT; i++) acc[i][j] = mfma<BF16>(w[i][k], f[k], acc[i][j]);
      }
    }
  };
#pragma unroll
  for (int d = 0; d < DEPTH; d++)
    if (wave + d * WAVES < whole) load_w(d, wave + d * WAVES);
  if (wave < whole) {
#pragma unroll
    for (int j = 0; j < MT; j++) load_rows(j, wave);
  }
  for (int step = wave; step < whole; step += WAVES * DEPTH) {
#pragma unroll
    for (int d = 0; d < DEPTH; d++)
      if (step + d * WAVES < whole) multiply(d, step + d * WAVES);
  }
  if (KB % 8 && wave == whole % WAVES) {  // the part of a step that is left
    const int64_t b = (int64_t)whole * 8 + 2 * g4;
    Frag f[MT][4];
#pragma unroll
    for (int j = 0; j < MT; j++) load_x<XT>(a, rt.m0 + (16 * j + col < xrows ? 16 * j + col : 0), b, KB, f[j]);
#pragma unroll
    for (int i = 0; i < NT; i++) {
      const int64_t row = w0 + (16 * i + col < wrows ? 16 * i + col : wrows - 1);
      Frag w[4];
      load_nvfp4<BF16>(a.w + row * (a.K / 2), a.ws + row * KB, b, KB, w);
#pragma unroll
      for (int k = 0; k < 4; k++)
#pragma unroll
        for (int j = 0; j < MT; j++) acc[i][j] = mfma<BF16>(w[k], f[j][k], acc[i][j]);
    }
  }
  // one column tile at a time, in two halves of the LDS in turn (the place in y
  // is computed again: it has no registers in the loop)
  const int at = (int)lane_offset((uint32_t)lane);
  f32x4(*part)[WAVES][MT][64] = reinterpret_cast<f32x4(*)[WAVES][MT][64]>(lds);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NT; i++) {
#pragma unroll
    for (int j = 0; j < MT; j++) part[i & 1][wave][j][lane] = acc[i][j];
    __syncthreads();
    if (const int j = turn(i); j < MT) {
      const int k = i * MP / WAVES;  // the wave's first or second tile
      f32x4 s[1] = {part[i & 1][0][j][lane]};
#pragma unroll
      for (int v = 1; v < WAVES; v++) s[0] += part[i & 1][v][j][lane];
      const int m = (int)rt.m0 + 16 * j + (at & 15);
      if (live[k]) finish(a, m, 0, m, Quad(a, n0 + 16 * i + 4 * (at >> 4)), columns[k], row[k], s);
    }
  }
}

// The tile kernel: one workgroup of four waves takes BM rows and 256 columns,
// each wave all BM rows and 64 columns. A 128-deep step of the activations is
// staged in LDS as 16-bit values, twice (the next step's loads run while this
// one is multiplied); the weights never pass through LDS: a wave decodes its own
// 64 rows of them in registers, so each is decoded once per workgroup and the
// LDS carries half of what two staged operands would (per step and wave 32 KiB
// read for 128 matrix instructions of 16 cycles: half of the LDS's rate).
//
// LDS: row r of the tile is 16 chunks of 16 bytes (8 values), swizzled as above.
template <int XT, int BM>
struct XStage {
  static constexpr bool kDirect = XT == kBF16 || XT == kFP16;
  static constexpr int kBlocks = BM * 8 / 256;  // 16-value blocks per thread and step
  const uint8_t* base;   // first row of the tile
  const uint8_t* sbase;  // NVFP4: its scales
  uint32_t off[kDirect ? BM / 16 : kBlocks / 2];
  uint32_t soff[XT == kXNVFP4 ? kBlocks / 2 : 1];
  uint32_t regs[kBlocks / 2][XT == kXE4M3 ? 8 : XT == kXNVFP4 ? 4 : 16];
  uint32_t sreg[kBlocks / 2];

  // Byte offsets of what this thread loads in every step, from the tile's
  // first row; rows past the end read the last one (their sums are dropped).
  __device__ __forceinline__ void init(const LinearArgs& a, int64_t m0, int rows) {
    const int64_t KB = a.K / 16;
    if constexpr (kDirect) {
      base = (const uint8_t*)a.x + m0 * a.K * 2;
      const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
      for (int i = 0; i < BM / 16; i++) {
        const int r = (wave * (BM / 16) + i) * 4 + (lane >> 4);
        const int c = (lane & 15) ^ swizzle<4>(r);
        off[i] = (uint32_t)(r < rows ? r : rows - 1) * (uint32_t)(a.K * 2) + 16 * c;
      }
    } else {
      base = (const uint8_t*)a.x + m0 * (XT == kXE4M3 ? a.K : a.K / 2);
      sbase = XT == kXNVFP4 ? a.xs + m0 * KB : nullptr;
#pragma unroll
      for (int i = 0; i < kBlocks / 2; i++) {
        const int r = i * 64 + (threadIdx.x >> 2), p = threadIdx.x & 3;  // blocks 2p, 2p + 1 of row r
        const uint32_t row = r < rows ? r : rows - 1;
        off[i] = row * (uint32_t)(XT == kXE4M3 ? a.K : a.K / 2) + p * (XT == kXE4M3 ? 32 : 16);
        if constexpr (XT == kXNVFP4) soff[i] = row * (uint32_t)KB + 2 * p;
      }
    }
  }

  // Start the loads of the whole step that begins at block b: into LDS for
  // 16-bit activations, into registers for those that are decoded first.
  __device__ __forceinline__ void load(int64_t b, uint8_t* lds) {
    if constexpr (kDirect) {
      const GlobalBytes p = scalar(base + b * 32);
      const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
      for (int i = 0; i < BM / 16; i++)
        __builtin_amdgcn_global_load_lds((const FOS_GLOBAL void*)(p + lane_offset(off[i])),
                                         (__attribute__((address_space(3))) void*)(lds + (wave * (BM / 16) + i) * 1024),
                                         16, 0, 0);
    } else if constexpr (XT == kXE4M3) {
      const GlobalBytes p = scalar(base + b * 16);
#pragma unroll
      for (int i = 0; i < kBlocks / 2; i++)
#pragma unroll
        for (int j = 0; j < 2; j++) {
          const u32x4 t = *(const FOS_GLOBAL u32x4*)(p + lane_offset(off[i]) + 16 * j);
#pragma unroll
          for (int k = 0; k < 4; k++) regs[i][4 * j + k] = t[k];
        }
    } else {
      const GlobalBytes p = scalar(base + b * 8), q = scalar(sbase + b);
#pragma unroll
      for (int i = 0; i < kBlocks / 2; i++) {
        const u32x4 t = *(const FOS_GLOBAL u32x4_a8*)(p + lane_offset(off[i]));
#pragma unroll
        for (int j = 0; j < 4; j++) regs[i][j] = t[j];
        sreg[i] = *(const FOS_GLOBAL u16_a1*)(q + lane_offset(soff[i]));
      }
    }
  }

  // Decode what load() brought to registers and store it to LDS.
  __device__ __forceinline__ void store(uint8_t* lds) {
    if constexpr (!kDirect) {
#pragma unroll
      for (int i = 0; i < kBlocks / 2; i++) {
        Frag f[4];
        if constexpr (XT == kXE4M3) {
#pragma unroll
          for (int j = 0; j < 8; j++) {
            f[j / 2].u[2 * (j & 1)] = bits(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)regs[i][j], 1.0f, false));
            f[j / 2].u[2 * (j & 1) + 1] = bits(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)regs[i][j], 1.0f, true));
          }
        } else {
          decode_blocks<false>(regs[i], sreg[i], f);
        }
        put(lds, i * 64 + (threadIdx.x >> 2), 4 * (threadIdx.x & 3), f);
      }
    }
  }

  // Chunks c .. c + 3 of row r.
  static __device__ __forceinline__ void put(uint8_t* lds, int r, int c, const Frag* f) {
#pragma unroll
    for (int j = 0; j < 4; j++)
      *reinterpret_cast<h8*>(lds + r * 256 + (((c + j) ^ swizzle<4>(r)) << 4)) = f[j].h;
  }

  // The last step when K ends inside it: blocks past the end are zero.
  __device__ __forceinline__ void load_last(const LinearArgs& a, int64_t m0, int rows, int64_t b, uint8_t* lds) {
#pragma unroll 1
    for (int i = 0; i < BM / 64; i++) {
      const int r = i * 64 + (threadIdx.x >> 2), p = threadIdx.x & 3;
      Frag f[4];
      load_x<XT>(a, m0 + (r < rows ? r : rows - 1), b + 2 * p, a.K / 16, f);
      put(lds, r, 4 * p, f);
    }
  }
};

// The order of a launch's tiles. Consecutive workgroups go to the 8 XCDs in
// turn, so each XCD gets a contiguous range of the tiles; along it, 8 row tiles
// are taken per column tile, so that the workgroups that run on an XCD at a
// time share their rows of both operands in its L2.
__device__ __forceinline__ void tile_of(uint32_t m_tiles, uint32_t n_tiles, uint32_t id, int64_t& tm, int64_t& tn) {
  const uint32_t total = m_tiles * n_tiles;  // a grid: below 2^31
  const uint32_t x = id % 8, base = total / 8, more = total % 8;
  const uint32_t t = x * base + (x < more ? x : more) + id / 8;
  const uint32_t band = t / (8 * n_tiles), in = t % (8 * n_tiles);
  const uint32_t high = m_tiles - band * 8 < 8 ? m_tiles - band * 8 : 8;
  tm = band * 8 + in % high;
  tn = in / high;
}

// Every load of this wave has arrived, the direct ones to LDS among them: the
// compiler does not wait for those by itself. (vmcnt = 0, the other counters at
// their maximum.)
__device__ __forceinline__ void wait_loads() {
  __builtin_amdgcn_s_waitcnt(0x0F70);
  asm volatile("" ::: "memory");
}

// (three workgroups of 64 rows fit a CU without spills for fp16 only)
template <int XT, int BM>
__global__ __launch_bounds__(256, BM == 64 && XT == kFP16 ? 3 : 2)
void k_linear_tile(LinearArgs a, uint32_t m_tiles, uint32_t n_tiles, int splits) {
  constexpr bool BF16 = XT == kBF16, SX = XT == kXE4M3 || XT == kXNVFP4;
  constexpr int MT = BM / 16;
  __shared__ __align__(16) uint8_t lds[2][BM * 256];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, g4 = lane >> 4;
  int64_t tm, tn;
  tile_of(m_tiles, n_tiles, blockIdx.x % (m_tiles * n_tiles), tm, tn);
  RowTile rt{tm * BM, a.M, 0};
  if (a.offs) {
    if (a.status && blockIdx.x == 0 && wave == 0) check_offs(a);
    rt = find_tile(a.offs, a.G, (int)a.M, BM, (int)tm);
    if (rt.g < 0) return;
  }
  const int rows = rt.end - rt.m0 < BM ? (int)(rt.end - rt.m0) : BM;
  const int64_t n0 = tn * 256 + wave * 64;
  if (a.offs && rt.g == a.G) {
    for (int r = col; r < rows; r += 16)
      for (int i = 0; i < 4; i++) zero4(a, rt.m0 + r, n0 + 16 * i + 4 * g4);
    return;
  }
  const int64_t KB = a.K / 16;
  // 128-deep steps of this workgroup's part of K; the last part may end inside one
  const int part = (int)(blockIdx.x / (m_tiles * n_tiles)), all = (int)(KB / 8), per = (all + splits - 1) / splits;
  const int first = per * part < all ? per * part : all;
  const int whole = part == splits - 1 ? all : first + per < all ? first + per : all;
  const bool remainder = KB % 8 && part == splits - 1;

  // weight rows: uniform base, 32-bit lane offsets; columns past the end read
  // the last row
  const int64_t w0 = (int64_t)rt.g * a.N + (n0 < a.N ? n0 : a.N - 1);
  const uint8_t* wc = a.w + w0 * (a.K / 2);
  const uint8_t* wsc = a.ws + w0 * KB;
  const int wrows = n0 < a.N ? (a.N - n0 < 64 ? (int)(a.N - n0) : 64) : 1;

  // A load instruction costs a cycle for every 64 bytes or row that four
  // consecutive lanes touch, and the matrix instruction wants consecutive lanes
  // in different rows. So four neighbouring lanes load the 64 bytes of a row,
  // and one lane the 8 scale bytes of each of the wave's 64 rows, and the lanes
  // swap them when the step begins: 24 exchanges against 1500 cycles of loads.
  uint32_t woff[4], wsoff;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int r = 16 * i + (lane >> 2);
    woff[i] = (uint32_t)(r < wrows ? r : wrows - 1) * (uint32_t)(a.K / 2) + 16 * (lane & 3);
  }
  wsoff = (uint32_t)(lane < wrows ? lane : wrows - 1) * (uint32_t)KB;
  u32x4 w_load[4];
  u32x2 s_load;
  uint32_t codes[4][4], scales[4];
  auto load_w = [&](int step) {
    const GlobalBytes p = scalar(wc + (int64_t)step * 64), q = scalar(wsc + (int64_t)step * 8);
#pragma unroll
    for (int i = 0; i < 4; i++) w_load[i] = *(const FOS_GLOBAL u32x4_a8*)(p + lane_offset(woff[i]));
    s_load = *(const FOS_GLOBAL u32x2_a1*)(q + lane_offset(wsoff));
  };
  auto take_w = [&] {
#pragma unroll
    for (int i = 0; i < 4; i++) {
#pragma unroll
      for (int j = 0; j < 4; j++) codes[i][j] = __builtin_amdgcn_ds_bpermute(16 * col + 4 * g4, w_load[i][j]);
      // bytes 2 g and 2 g + 1 of the row's eight
      const uint32_t lo = __builtin_amdgcn_ds_bpermute(64 * i + 4 * col, s_load[0]);
      const uint32_t hi = __builtin_amdgcn_ds_bpermute(64 * i + 4 * col, s_load[1]);
      scales[i] = (g4 < 2 ? lo : hi) >> (16 * (g4 & 1));
    }
  };

  f32x4 acc[4][MT];
#pragma unroll
  for (int i = 0; i < 4; i++)
#pragma unroll
    for (int j = 0; j < MT; j++) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  uint32_t roff[4];  // fragment c = 2 h + j of this lane: LDS byte offset in rows 0 .. 15
#pragma unroll
  for (int c = 0; c < 4; c++) roff[c] = col * 256 + (((4 * g4 + c) ^ swizzle<4>(col)) << 4);

  // Multiply the staged step by the weights in registers. (Leaving out the row
  // tiles past a group's end made the loop slower by more than it saved: 64
  // experts of 240 rows 593 us, 584 without.)
  auto multiply = [&](const uint8_t* cur) {
#pragma unroll
    for (int h = 0; h < 2; h++) {
      Frag x[2][2];
#pragma unroll
      for (int j = 0; j < 2; j++) x[0][j].h = *reinterpret_cast<const h8*>(cur + roff[2 * h + j]);
      Frag w[4][2];
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const f32x2 s = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((int)scales[i], 1.0f, false);
        const h2 s16 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)scales[i], 1.0f, false);
        const h2 sh = h ? __builtin_shufflevector(s16, s16, 1, 1) : __builtin_shufflevector(s16, s16, 0, 0);
        decode8<BF16>(codes[i][2 * h], h ? s.y : s.x, sh, w[i][0].u);
        decode8<BF16>(codes[i][2 * h + 1], h ? s.y : s.x, sh, w[i][1].u);
      }
      // the other workgroup's wave on this SIMD decodes meanwhile
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int m = 0; m < MT; m++) {
        if (m + 1 < MT) {
#pragma unroll
          for (int j = 0; j < 2; j++)
            x[(m + 1) & 1][j].h = *reinterpret_cast<const h8*>(cur + roff[2 * h + j] + (m + 1) * 4096);
        }
#pragma unroll
        for (int j = 0; j < 2; j++)
#pragma unroll
          for (int i = 0; i < 4; i++) acc[i][m] = mfma<BF16>(w[i][j], x[m & 1][j], acc[i][m]);
        __builtin_amdgcn_sched_barrier(0);
      }
      __builtin_amdgcn_s_setprio(0);
    }
  };

  XStage<XT, BM> xs;
  xs.init(a, rt.m0, rows);
  if (whole > first) {
    xs.load((int64_t)first * 8, lds[first & 1]);
    load_w(first);
    xs.store(lds[first & 1]);
  }
  for (int step = first; step < whole; step++) {
    // This step's tile is in LDS and its weights are in registers, and no wave
    // reads the other tile any more. All of the next step's loads start here
    // and have this step's time. (The last step loads itself again: a load that
    // may not happen would make the compiler wait where the paths meet.)
    wait_loads();
    __syncthreads();
    take_w();
    uint8_t* next = lds[(step & 1) ^ 1];
    const int after = step + 1 < whole ? step + 1 : step;
    load_w(after);
    xs.load((int64_t)after * 8, next);
    multiply(lds[step & 1]);
    xs.store(next);
  }
  wait_loads();
  __syncthreads();
  if (remainder) {  // the part of a step that is left: zeros past the end
    uint8_t* last = lds[whole & 1];
    xs.load_last(a, rt.m0, rows, (int64_t)whole * 8, last);
    const int64_t b = (int64_t)whole * 8 + 2 * g4;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int64_t r = 16 * i + col < wrows ? 16 * i + col : wrows - 1;
      scales[i] = 0;
#pragma unroll
      for (int h = 0; h < 2; h++) {
        uint2 t = {0, 0};
        if (b + h < KB) {
          t = *reinterpret_cast<const uint2*>(wc + r * (a.K / 2) + 8 * (b + h));
          scales[i] |= (uint32_t)wsc[r * KB + b + h] << (8 * h);
        }
        codes[i][2 * h] = t.x, codes[i][2 * h + 1] = t.y;
      }
    }
    __syncthreads();
    multiply(last);
  }
  // Each wave turns its sums by way of its quarter of the LDS, half of the rows
  // at a time, so that 16 lanes store 64 neighbouring columns of a row. A batch
  // is R steps of four rows, as many as the registers hold (four for the third
  // workgroup of a CU); what it takes from memory is loaded one batch ahead, and
  // its rows go through each stage of the epilogue together. (1003 x 5003 x 2064
  // with silu and a binary32 residual: 43 us, 55 with each row's stages apart.)
  constexpr int R = BM == 64 && XT == kFP16 ? 4 : 8;
  const Quad q(a, n0 + 4 * col);
  ColumnTail columns;
  RowTails<SX, R> next;
  const int last = (int)rt.m0 + rows - 1;
  const bool finishes = splits == 1 && q.have;
  if (finishes) {
    columns.load(a, rt.g, q);
    next.load(a, rt.g, (int)rt.m0 + g4, 4, last, q);
  }
  __syncthreads();
  uint8_t* mine = &lds[0][0] + wave * (BM * 128);
#pragma unroll
  for (int half = 0; half < 2; half++) {
    wave_lds_order();
#pragma unroll
    for (int m = 0; m < MT / 2; m++)
#pragma unroll
      for (int i = 0; i < 4; i++)
        *reinterpret_cast<f32x4*>(mine + (16 * m + col) * 256 + (((4 * i + g4) ^ swizzle<4>(col)) << 4)) =
            acc[i][half * (MT / 2) + m];
    wave_lds_order();
#pragma unroll 1
    for (int it = 0; it < BM / 8 / R; it++) {
      const int b = half * (BM / 8 / R) + it;
      const int m = (int)rt.m0 + 4 * R * b + g4;
      const RowTails<SX, R> row = next;
      if (finishes && b + 1 < BM / 4 / R) next.load(a, rt.g, m + 4 * R, 4, last, q);
      f32x4 v[R];
#pragma unroll
      for (int k = 0; k < R; k++) {
        const int lr = 4 * R * it + 4 * k + g4;
        v[k] = *reinterpret_cast<const f32x4*>(mine + lr * 256 + ((col ^ swizzle<4>(lr)) << 4));
      }
      if (finishes) {
        finish(a, m, 4, last, q, columns, row, v);
      } else if (q.have) {  // rows of the workspace are padded to a multiple of 4 columns
#pragma unroll
        for (int k = 0; k < R; k++)
          if (m + 4 * k <= last)
            *reinterpret_cast<f32x4*>((float*)a.work + (part * a.M + m + 4 * k) * ((a.N + 3) / 4 * 4) + q.n) = v[k];
      }
    }
  }
}

// Joins the parts of K in order and finishes: four columns per thread.
__global__ __launch_bounds__(256) void k_linear_join(LinearArgs a, int splits) {
  const uint32_t quads = (uint32_t)((a.N + 3) / 4), blocks = (quads + 255) / 256;  // workgroups per row
  const int64_t m = blockIdx.x / blocks, total = a.M * quads;
  const uint32_t c = blockIdx.x % blocks * 256 + threadIdx.x;
  if (c >= quads) return;
  const Quad q(a, (int64_t)c * 4);
  ColumnTail columns;
  RowTails<true, 1> row;
  columns.load(a, 0, q);
  row.load(a, 0, (int)m, 0, (int)m, q);
  const f32x4* p = (const f32x4*)a.work + m * quads + c;
  f32x4 v[1] = {p[0]};
#pragma unroll 4
  for (int s = 1; s < splits; s++) v[0] += p[s * total];
  finish(a, (int)m, 0, (int)m, q, columns, row, v);
}

template <int XT, int MT, int NT>
hipError_t launch_stream_n(const LinearArgs& a, int64_t m_tiles, hipStream_t s) {
  const int64_t n_tiles = (a.N + 16 * NT - 1) / (16 * NT);
  constexpr int WAVES = stream_waves(MT, NT);
  k_linear_stream<XT, MT, NT, WAVES><<<dim3((unsigned)(m_tiles * n_tiles)), dim3(64 * WAVES), 0, s>>>(a, (int)n_tiles);
  return hipGetLastError();
}

template <int XT, int MT>
hipError_t launch_stream(const LinearArgs& a, int64_t m_tiles, hipStream_t s) {
  switch (stream_columns(m_tiles, a.N)) {
    case 4: return launch_stream_n<XT, MT, 4>(a, m_tiles, s);
    case 2: return launch_stream_n<XT, MT, 2>(a, m_tiles, s);
    default: return launch_stream_n<XT, MT, 1>(a, m_tiles, s);
  }
}

template <int XT>
hipError_t launch_type(const LinearArgs& a, hipStream_t s) {
  const Plan p = plan(a.M, a.N, a.K, a.offs ? a.G : 0);
  if (p.stream) {
    if (p.bm == 16) return launch_stream<XT, 1>(a, p.m_tiles, s);
    if (p.bm == 32) return launch_stream<XT, 2>(a, p.m_tiles, s);
    if (p.bm == 48) return launch_stream<XT, 3>(a, p.m_tiles, s);
    return launch_stream<XT, 4>(a, p.m_tiles, s);
  }
  const int64_t n_tiles = (a.N + 255) / 256;
  const dim3 grid((unsigned)(p.m_tiles * n_tiles * p.splits));
  if (p.bm == 64)
    k_linear_tile<XT, 64><<<grid, dim3(256), 0, s>>>(a, (uint32_t)p.m_tiles, (uint32_t)n_tiles, p.splits);
  else
    k_linear_tile<XT, 128><<<grid, dim3(256), 0, s>>>(a, (uint32_t)p.m_tiles, (uint32_t)n_tiles, p.splits);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  const int64_t blocks = a.M * (((a.N + 3) / 4 + 255) / 256);
  k_linear_join<<<dim3((unsigned)blocks), dim3(256), 0, s>>>(a, p.splits);
  return hipGetLastError();
}

}  // namespace

int64_t linear_workspace(int64_t M, int64_t N, int64_t K, int G) {
  const Plan p = plan(M, N, K, G);
  return p.splits == 1 ? 0 : p.splits * M * ((N + 3) / 4 * 4) * 4;
}

bool linear_fits(int64_t M, int64_t N, int64_t K, int G) { return fits(plan(M, N, K, G), N); }

hipError_t launch_linear(const LinearArgs& a, hipStream_t s) {
  if (a.M == 0 || a.N == 0) {  // nothing to write; offsets are reported all the same
    if (!a.offs || !a.status) return hipSuccess;
    k_check_offs<<<dim3(1), dim3(64), 0, s>>>(a);
    return hipGetLastError();
  }
  switch (a.x_type) {
    case kBF16: return launch_type<kBF16>(a, s);
    case kFP16: return launch_type<kFP16>(a, s);
    case kXE4M3: return launch_type<kXE4M3>(a, s);
    default: return launch_type<kXNVFP4>(a, s);
  }
}

}  // namespace fos
