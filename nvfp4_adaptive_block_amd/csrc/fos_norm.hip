// fos_norm.hip: root-mean-square norm of a residual sum with an 8-bit output.
//
//   h = x + res;  y = weight * h / sqrt(mean(h^2) + eps)
//   s = max|y| / 448 (1 when every y is 0), q = E4M3(y / s)
//
// The norm takes h before its rounding to the stored type. Squares are summed
// in binary64: that costs two instructions per element beside several bytes of
// traffic, and no h that binary32 holds overflows or vanishes in it. Everything
// else is binary32. A row with a NaN or an infinity in h has s = NaN, every
// code NaN (0x7F) and y = NaN; so has a row whose y overflows (s and codes).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fos_device.h"
#include "fos_ops.h"

namespace fos {
namespace {

template <int DT>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if constexpr (DT == kFP32) return ((const float*)p)[i];
  const uint16_t v = ((const uint16_t*)p)[i];
  if constexpr (DT == kBF16) return __uint_as_float((uint32_t)v << 16);
  return (float)__builtin_bit_cast(_Float16, v);
}

template <int DT>
__device__ __forceinline__ void store1(void* p, int64_t i, float v) {
  if constexpr (DT == kFP32)
    ((float*)p)[i] = v;
  else
    ((uint16_t*)p)[i] = (uint16_t)(DT == kBF16 ? pack_bf16(v, 0.0f) : pack_f16(v, 0.0f));
}

__device__ __forceinline__ float load_weight(const NormArgs& a, int64_t i) {
  return a.weight_dt == kFP32 ? load1<kFP32>(a.weight, i)
                              : a.weight_dt == kBF16 ? load1<kBF16>(a.weight, i) : load1<kFP16>(a.weight, i);
}

// 1 / sqrt(mean + eps) from a row's sum of squares, as r times a power of two;
// NaN if the sum is not finite. The power is 1 but where the reciprocal nears the
// ends of binary32's range (eps 0 and a row of subnormals; a row of the largest
// values): h takes it before r then, and neither is lost.
struct InverseRms {
  float r, up;
  bool far;  // the same in all lanes; up is 1 where it is not set
  __device__ __forceinline__ InverseRms(double sum, int64_t K, float eps) {
    const double w = sum < __builtin_huge_val() ? 1.0 / sqrt(sum / (double)K + (double)eps) : __builtin_nan("");
    r = (float)w;
    up = 1.0f;
    far = __builtin_amdgcn_readfirstlane(!(r >= 0x1p-100f && r <= 0x1p100f));
    if (far) {
      up = w > 1.0 ? 0x1p64f : 0x1p-64f;
      r = (float)(w * (w > 1.0 ? 0x1p-64 : 0x1p64));
    }
  }
};

// The row's scale from max|y|: NaN unless the maximum is finite.
__device__ __forceinline__ float row_scale(float top) {
  if (!(top < __builtin_huge_valf())) return __builtin_nanf("");
  return top > 0.0f ? __builtin_fmaxf(top / 448.0f, 0x1p-126f) : 1.0f;
}

// The row's divider: v / s in E4M3's range (v's magnitude is at most 448 s up to
// rounding), rounded to binary32 once, then to E4M3. v times 1 / s, whose two
// roundings put values beside the middle of two codes on its other side, is
// corrected by the remainder v - t s, which one fused multiply-add gives exactly
// (8192 x 4096: IEEE divisions took 53 us, this and no correction 48). Below
// 2^-90 the remainder may be subnormal, and such rows divide. (Where s is NaN,
// so is the row, and its codes are set apart from this.)
struct Divider {
  float s, inv;
  bool tiny;  // the same in all lanes
  __device__ __forceinline__ Divider(float scale) : s(scale), inv(1.0f / scale) {
    tiny = (uint32_t)__builtin_amdgcn_readfirstlane((int)__float_as_uint(s)) < __float_as_uint(0x1p-90f);
  }
  template <int N>
  __device__ __forceinline__ void operator()(const float* v, float* t) const {
    if (tiny) {
#pragma unroll
      for (int j = 0; j < N; j++) t[j] = v[j] / s;
    } else {
#pragma unroll
      for (int j = 0; j < N; j++) {
        const float t0 = v[j] * inv;
        t[j] = __builtin_fmaf(-__builtin_fmaf(t0, s, -v[j]), inv, t0);  // (-0 stays -0)
      }
    }
#pragma unroll
    for (int j = 0; j < N; j++) t[j] = __builtin_amdgcn_fmed3f(t[j], -448.0f, 448.0f);
  }
};

// max that keeps a NaN of either side
__device__ __forceinline__ float max_nan(float a, float b) { return (a != a) ? a : (b != b) ? b : a > b ? a : b; }

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v = max_nan(v, __shfl_xor(v, d, 64));
  return v;
}

// Rows that no register form takes (K below 8 or above 32768): one workgroup
// per row, one element per lane and step; x and res are read three times (from
// the caches after the first). 4096 x 40000 bf16 with a residual: 992 us, 1.2 TB/s:
// such rows are taken, not taken fast.
template <int DT>
__global__ __launch_bounds__(1024) void k_norm(NormArgs a) {
  const int64_t row = blockIdx.x, base = row * a.K;
  __shared__ double sums[16];
  __shared__ float tops[16];
  const int wave = threadIdx.x >> 6;
  const int threads = blockDim.x, waves = threads / 64;
  double ss = 0.0;
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < a.K; i += threads) {
    float h = load1<DT>(a.x, base + i);
    if (a.res) h += load1<DT>(a.res, base + i);
    ss += (double)h * (double)h;
  }
  ss = wave_sum(ss);
  if ((threadIdx.x & 63) == 0) sums[wave] = ss;
  __syncthreads();
  ss = sums[0];
  for (int i = 1; i < waves; i++) ss += sums[i];
  const InverseRms inv(ss, a.K, a.eps);
  float top = 0.0f;
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < a.K; i += threads) {
    float h = load1<DT>(a.x, base + i);
    if (a.res) h += load1<DT>(a.res, base + i);
    top = max_nan(top, __builtin_fabsf(load_weight(a, i) * (h * inv.up * inv.r)));
  }
  top = wave_max(top);
  if ((threadIdx.x & 63) == 0) tops[wave] = top;
  __syncthreads();
  top = tops[0];
  for (int i = 1; i < waves; i++) top = max_nan(top, tops[i]);
  const float s = row_scale(top);
  const Divider divide(s);
  if (threadIdx.x == 0) a.scale[row] = s;
  for (int64_t i = threadIdx.x; i < a.K; i += threads) {
    float h = load1<DT>(a.x, base + i);
    if (a.res) h += load1<DT>(a.res, base + i);
    const float y = load_weight(a, i) * (h * inv.up * inv.r);
    float t;
    divide.operator()<1>(&y, &t);
    a.q[base + i] = s != s ? 0x7F : (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(t, 0.0f, 0, false);
    if (a.h) store1<DT>(a.h, base + i, h);
    if (a.y) store1<DT>(a.y, base + i, y);
  }
}

// Eight values of a row from element i on (i + 8 <= the row's end), at any
// alignment: one or two 16-byte accesses.
struct __attribute__((packed, aligned(2))) Chunk16 {
  uint32_t v[4];
};
struct __attribute__((packed, aligned(4))) Chunk32 {
  float v[4];
};
struct __attribute__((packed, aligned(1))) Chunk8 {
  uint32_t v[2];
};

template <int DT>
__device__ __forceinline__ void load8(const void* p, int64_t i, float* v) {
  if constexpr (DT == kFP32) {
#pragma unroll
    for (int j = 0; j < 2; j++) {
      const Chunk32 t = *reinterpret_cast<const Chunk32*>((const float*)p + i + 4 * j);
#pragma unroll
      for (int k = 0; k < 4; k++) v[4 * j + k] = t.v[k];
    }
  } else {
    const Chunk16 t = *reinterpret_cast<const Chunk16*>((const uint16_t*)p + i);
#pragma unroll
    for (int k = 0; k < 4; k++) {
      v[2 * k] = DT == kBF16 ? bf16_lo(t.v[k]) : f16_lo(t.v[k]);
      v[2 * k + 1] = DT == kBF16 ? bf16_hi(t.v[k]) : f16_hi(t.v[k]);
    }
  }
}

template <int DT>
__device__ __forceinline__ void store8(void* p, int64_t i, const float* v) {
  if constexpr (DT == kFP32) {
#pragma unroll
    for (int j = 0; j < 2; j++) {
      Chunk32 t;
#pragma unroll
      for (int k = 0; k < 4; k++) t.v[k] = v[4 * j + k];
      *reinterpret_cast<Chunk32*>((float*)p + i + 4 * j) = t;
    }
  } else {
    Chunk16 t;
#pragma unroll
    for (int k = 0; k < 4; k++)
      t.v[k] = DT == kBF16 ? pack_bf16(v[2 * k], v[2 * k + 1]) : pack_f16(v[2 * k], v[2 * k + 1]);
    *reinterpret_cast<Chunk16*>((uint16_t*)p + i) = t;
  }
}

// Rows held in registers: x, res and weight are read once. PACK: a workgroup of
// four waves takes four rows of at most 64 chunks of 8 elements and needs no
// barrier. Otherwise a workgroup takes one row, C chunks per lane, with as many
// waves as that needs. K is at least 8.
//
// The K % 8 elements that may follow the last whole chunk are a chunk of one
// lane that reads the row's last 8 elements, drops those that another lane has,
// and writes its own one by one: reads need no branch, and rows of odd width,
// whose accesses straddle the 16-byte grid, run at the same instructions (a
// chunk grid aligned in memory, with two such edges per row, measured slower).
// Chunk c goes to thread c % threads, so that a wave's accesses are contiguous.
template <int DT, int WT, bool PACK, int C, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_norm_rows(NormArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row = PACK ? (int64_t)blockIdx.x * WAVES + wave : blockIdx.x;
  if (PACK && row >= a.M) return;
  const int t = PACK ? lane : threadIdx.x;
  constexpr int threads = PACK ? 64 : 64 * WAVES;
  const int K = (int)a.K;
  const int64_t base = row * a.K;
  float h[C][8], w[C][8];
  double ss = 0.0;
#pragma unroll
  for (int c = 0; c < C; c++) {
    const int e = 8 * (t + c * threads), at = e + 8 <= K ? e : K - 8;
    load8<DT>(a.x, base + at, h[c]);
    load8<WT>(a.weight, at, w[c]);
    if (a.res) {
      float r[8];
      load8<DT>(a.res, base + at, r);
#pragma unroll
      for (int j = 0; j < 8; j++) h[c][j] += r[j];
    }
    if (at != e) {
#pragma unroll
      for (int j = 0; j < 8; j++)
        if (at + j < e) h[c][j] = w[c][j] = 0.0f;
    }
  }
#pragma unroll
  for (int c = 0; c < C; c++) {
    const int e = 8 * (t + c * threads);
#pragma unroll
    for (int j = 0; j < 8; j++) ss += (double)h[c][j] * (double)h[c][j];
    if (a.h) {
      if (e + 8 <= K) {
        store8<DT>(a.h, base + e, h[c]);
      } else if (e < K) {
#pragma unroll
        for (int j = 1; j < 8; j++)
          if (K - 8 + j >= e) store1<DT>(a.h, base + K - 8 + j, h[c][j]);
      }
    }
  }
  ss = wave_sum(ss);
  if constexpr (!PACK) {
    __shared__ double sums[WAVES];
    if (lane == 0) sums[wave] = ss;
    __syncthreads();
    ss = sums[0];
    for (int i = 1; i < WAVES; i++) ss += sums[i];
  }
  const InverseRms inv(ss, a.K, a.eps);
  if (inv.far) {
#pragma unroll
    for (int c = 0; c < C; c++)
#pragma unroll
      for (int j = 0; j < 8; j++) h[c][j] *= inv.up;
  }
  float top = 0.0f;
#pragma unroll
  for (int c = 0; c < C; c++)
#pragma unroll
    for (int j = 0; j < 8; j++) {
      h[c][j] = w[c][j] * (h[c][j] * inv.r);
      // padding has h = w = 0 and adds nothing (it is NaN exactly where the row is)
      top = max_nan(top, __builtin_fabsf(h[c][j]));
    }
  top = wave_max(top);
  if constexpr (!PACK) {
    __shared__ float tops[WAVES];
    if (lane == 0) tops[wave] = top;
    __syncthreads();
    top = tops[0];
    for (int i = 1; i < WAVES; i++) top = max_nan(top, tops[i]);
  }
  const float s = row_scale(top);
  const Divider divide(s);
  if (t == 0) a.scale[row] = s;
#pragma unroll
  for (int c = 0; c < C; c++) {
    const int e = 8 * (t + c * threads);
    uint32_t q[2];
    float v[8];
    divide.operator()<8>(h[c], v);
#pragma unroll
    for (int k = 0; k < 2; k++) {
      int p = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * k], v[4 * k + 1], 0, false);
      q[k] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * k + 2], v[4 * k + 3], p, true);
      if (s != s) q[k] = 0x7F7F7F7Fu;
    }
    if (e + 8 <= K) {
      *reinterpret_cast<Chunk8*>(a.q + base + e) = Chunk8{{q[0], q[1]}};
      if (a.y) store8<DT>(a.y, base + e, h[c]);
    } else if (e < K) {
#pragma unroll
      for (int j = 1; j < 8; j++)
        if (K - 8 + j >= e) {
          a.q[base + K - 8 + j] = (uint8_t)(q[j / 4] >> (8 * (j % 4)));
          if (a.y) store1<DT>(a.y, base + K - 8 + j, h[c][j]);
        }
    }
  }
}

template <int DT, int WT, int C, int WAVES>
hipError_t rows(const NormArgs& a, hipStream_t s) {
  k_norm_rows<DT, WT, false, C, WAVES><<<dim3((unsigned)a.M), dim3(64 * WAVES), 0, s>>>(a);
  return hipGetLastError();
}

// The waves of a row: powers of two, so that the four SIMDs share them evenly
// (seven waves of four chunks took 116 us where sixteen of two take 89, 4096 x
// 14336 bf16), and the fewest registers that leaves (8192 x 4096: two chunks in
// four waves 51 us, one in eight 59; 4096 x 8192: two in eight 49, four in four
// 56). Bound by HBM: 8192 x 4096 bf16 with a residual moves 235 MB in 48 us when
// launches follow each other, 4.9 TB/s where a copy reaches 5.1 and an addition of
// tensors of this size 5.5. (Alone it takes 42 us: the end of its writes leaves
// the caches after it.)
template <int DT, int WT>
hipError_t by_width(const NormArgs& a, hipStream_t s) {
  const int64_t chunks = (a.K + 7) / 8;
  if (a.K >= 8 && chunks <= 64) {
    k_norm_rows<DT, WT, true, 1, 4><<<dim3((unsigned)((a.M + 3) / 4)), dim3(256), 0, s>>>(a);
    return hipGetLastError();
  }
  if (a.K >= 8) {
    if (chunks <= 128) return rows<DT, WT, 1, 2>(a, s);
    if (chunks <= 256) return rows<DT, WT, 1, 4>(a, s);
    if (chunks <= 512) return rows<DT, WT, 2, 4>(a, s);
    if (chunks <= 768) return rows<DT, WT, 3, 4>(a, s);
    if (chunks <= 1024) return rows<DT, WT, 2, 8>(a, s);
    if (chunks <= 1536) return rows<DT, WT, 3, 8>(a, s);
    if (chunks <= 2048) return rows<DT, WT, 2, 16>(a, s);
    if (chunks <= 4096) return rows<DT, WT, 4, 16>(a, s);
  }
  k_norm<DT><<<dim3((unsigned)a.M), dim3(a.K < 8 ? 64 : 1024), 0, s>>>(a);
  return hipGetLastError();
}

template <int DT>
hipError_t by_weight(const NormArgs& a, hipStream_t s) {
  switch (a.weight_dt) {
    case kBF16: return by_width<DT, kBF16>(a, s);
    case kFP16: return by_width<DT, kFP16>(a, s);
    default: return by_width<DT, kFP32>(a, s);
  }
}

}  // namespace

// A launch has fewer than 2^32 threads, up to 1024 of them for a row, so that
// calls of more rows are several launches.
hipError_t launch_norm(int dt, const NormArgs& a, hipStream_t s) {
  constexpr int64_t kRows = int64_t(1) << 21;
  const int64_t size = dt == kFP32 ? 4 : 2;
  for (int64_t row = 0; row < a.M; row += kRows) {
    NormArgs part = a;
    part.M = a.M - row < kRows ? a.M - row : kRows;
    part.x = (const uint8_t*)a.x + row * a.K * size;
    if (a.res) part.res = (const uint8_t*)a.res + row * a.K * size;
    part.q = a.q + row * a.K;
    part.scale = a.scale + row;
    if (a.h) part.h = (uint8_t*)a.h + row * a.K * size;
    if (a.y) part.y = (uint8_t*)a.y + row * a.K * size;
    const hipError_t e = dt == kBF16 ? by_weight<kBF16>(part, s)
                         : dt == kFP16 ? by_weight<kFP16>(part, s) : by_weight<kFP32>(part, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace fos
