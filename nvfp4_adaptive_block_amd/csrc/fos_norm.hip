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

// 1 / sqrt(mean + eps) from the sum of squares, NaN if the sum is not finite.
__device__ __forceinline__ float inv_rms(double sum, int64_t K, float eps) {
  const double r = 1.0 / sqrt(sum / (double)K + (double)eps);
  return sum < __builtin_huge_val() ? (float)r : __builtin_nanf("");
}

// The row's scale from max|y|: NaN unless the maximum is finite.
__device__ __forceinline__ float row_scale(float top) {
  if (!(top < __builtin_huge_valf())) return __builtin_nanf("");
  return top > 0.0f ? __builtin_fmaxf(top / 448.0f, 0x1p-126f) : 1.0f;
}

// E4M3 code of v / s, v's magnitude at most 448 s up to rounding.
__device__ __forceinline__ float to_e4m3_range(float v, float inv) {
  const float t = v * inv;
  return t != t ? t : __builtin_fminf(__builtin_fmaxf(t, -448.0f), 448.0f);
}

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

// One workgroup per row, one element per lane and step; x and res are read
// three times (from the caches after the first).
template <int DT>
__global__ __launch_bounds__(256) void k_norm(NormArgs a) {
  const int64_t row = blockIdx.x, base = row * a.K;
  __shared__ double sums[4];
  __shared__ float tops[4];
  const int wave = threadIdx.x >> 6;
  double ss = 0.0;
  for (int64_t i = threadIdx.x; i < a.K; i += 256) {
    float h = load1<DT>(a.x, base + i);
    if (a.res) h += load1<DT>(a.res, base + i);
    ss += (double)h * (double)h;
  }
  ss = wave_sum(ss);
  if ((threadIdx.x & 63) == 0) sums[wave] = ss;
  __syncthreads();
  ss = (sums[0] + sums[1]) + (sums[2] + sums[3]);
  const float r = inv_rms(ss, a.K, a.eps);
  float top = 0.0f;
  for (int64_t i = threadIdx.x; i < a.K; i += 256) {
    float h = load1<DT>(a.x, base + i);
    if (a.res) h += load1<DT>(a.res, base + i);
    const float y = load_weight(a, i) * (h * r);
    top = max_nan(top, __builtin_fabsf(y));
  }
  top = wave_max(top);
  if ((threadIdx.x & 63) == 0) tops[wave] = top;
  __syncthreads();
  top = max_nan(max_nan(tops[0], tops[1]), max_nan(tops[2], tops[3]));
  const float s = row_scale(top), inv = 1.0f / s;
  if (threadIdx.x == 0) a.scale[row] = s;
  for (int64_t i = threadIdx.x; i < a.K; i += 256) {
    float h = load1<DT>(a.x, base + i);
    if (a.res) h += load1<DT>(a.res, base + i);
    const float y = load_weight(a, i) * (h * r);
    const float t = to_e4m3_range(y, inv);
    a.q[base + i] = t != t ? 0x7F : (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(t, 0.0f, 0, false);
    if (a.h) store1<DT>(a.h, base + i, h);
    if (a.y) store1<DT>(a.y, base + i, y);
  }
}

template <int DT>
hipError_t launch_type(const NormArgs& a, hipStream_t s) {
  k_norm<DT><<<dim3((unsigned)a.M), dim3(256), 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm(int dt, const NormArgs& a, hipStream_t s) {
  switch (dt) {
    case kBF16: return launch_type<kBF16>(a, s);
    case kFP16: return launch_type<kFP16>(a, s);
    default: return launch_type<kFP32>(a, s);
  }
}

}  // namespace fos
