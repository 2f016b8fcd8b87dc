// fos_route.hip: the load-balance loss of a router, per-expert counts and the
// group offsets that the grouped calls take, and the loss's gradient.
//
//   p_t = softmax(logits_t) for each live token (mask 1); n live tokens
//   c_e = live assignments to expert e, C = sum c
//   slope_e = coef * E * c_e / (max(C, 1) * max(n, 1))
//   loss = sum_e slope_e * sum_t p_te
//   d loss / d logits_te = p_te * (slope_e - sum_j slope_j p_tj)
//
// A live row without a finite or +infinite logit (all -infinity) has p = 0: it
// counts as a token and neither adds to the loss nor gets a gradient. Masked
// rows are not read. Counts are integers; column sums of p are binary32 within
// a wave's rows and binary64 from there on, joined in a fixed order, so that
// results do not depend on the order of execution.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fos_device.h"
#include "fos_ops.h"

namespace fos {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

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

__device__ __forceinline__ float max_nan(float a, float b) { return (a != a) ? a : (b != b) ? b : a > b ? a : b; }

// softmax of row t in lane-strided columns: p[i] is column lane + 64 i.
template <int DT, int EPL>
__device__ __forceinline__ void softmax_row(const void* logits, int64_t t, int E, float* p) {
  const int lane = threadIdx.x & 63;
  float top = -__builtin_huge_valf();
#pragma unroll
  for (int i = 0; i < EPL; i++) {
    const int e = lane + 64 * i;
    p[i] = e < E ? load1<DT>(logits, t * E + e) : -__builtin_huge_valf();
    top = max_nan(top, p[i]);
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) top = max_nan(top, __shfl_xor(top, d, 64));
  const bool none = top == -__builtin_huge_valf();
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < EPL; i++) {
    p[i] = none ? 0.0f : expf(p[i] - top);
    sum += p[i];
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d, 64);
  const float inv = none ? 0.0f : 1.0f / sum;
#pragma unroll
  for (int i = 0; i < EPL; i++) p[i] *= inv;
}

// Each workgroup takes a contiguous range of rows and leaves E column sums, E
// counts and its number of live rows in the workspace.
template <int DT, int EPL>
__global__ __launch_bounds__(kThreads) void k_balance(BalanceArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t per = (a.T + gridDim.x - 1) / gridDim.x;
  const int64_t t0 = per * blockIdx.x, t1 = t0 + per < a.T ? t0 + per : a.T;
  extern __shared__ float lds[];
  float* sums = lds;                              // [kWaves][E]
  int32_t* hist = (int32_t*)(lds + kWaves * a.E);  // [E]
  __shared__ int32_t live_rows;
  for (int e = threadIdx.x; e < a.E; e += kThreads) hist[e] = 0;
  if (threadIdx.x == 0) live_rows = 0;
  __syncthreads();
  float acc[EPL] = {};
  int32_t live = 0;
  for (int64_t t = t0 + wave; t < t1; t += kWaves) {
    if (a.mask && !a.mask[t]) continue;
    live++;
    float p[EPL];
    softmax_row<DT, EPL>(a.logits, t, a.E, p);
#pragma unroll
    for (int i = 0; i < EPL; i++) acc[i] += p[i];
  }
  if (lane == 0) atomicAdd(&live_rows, live);
#pragma unroll
  for (int i = 0; i < EPL; i++)
    if (lane + 64 * i < a.E) sums[wave * a.E + lane + 64 * i] = acc[i];
  bool bad = false;
  for (int64_t j = t0 * a.k + threadIdx.x; j < t1 * a.k; j += kThreads) {
    if (a.mask && !a.mask[j / a.k]) continue;
    const int64_t e = a.idx64 ? ((const int64_t*)a.idx)[j] : (int64_t)((const int32_t*)a.idx)[j];
    if (e >= 0 && e < a.E)
      atomicAdd(&hist[e], 1);
    else
      bad |= e != -1;
  }
  if (bad && a.status) atomicOr(a.status, kStatusBadIndex);
  __syncthreads();
  double* psum = (double*)a.work;                                   // [blocks][E]
  int32_t* pcount = (int32_t*)(psum + (int64_t)gridDim.x * a.E);    // [blocks][E]
  int32_t* plive = pcount + (int64_t)gridDim.x * a.E;               // [blocks]
  for (int e = threadIdx.x; e < a.E; e += kThreads) {
    double s = 0.0;
    for (int w = 0; w < kWaves; w++) s += (double)sums[w * a.E + e];
    psum[(int64_t)blockIdx.x * a.E + e] = s;
    pcount[(int64_t)blockIdx.x * a.E + e] = hist[e];
  }
  if (threadIdx.x == 0) plive[blockIdx.x] = live_rows;
}

// One workgroup joins the partial rows.
__global__ __launch_bounds__(1024) void k_balance_finish(BalanceArgs a, int blocks) {
  const double* psum = (const double*)a.work;
  const int32_t* pcount = (const int32_t*)(psum + (int64_t)blocks * a.E);
  const int32_t* plive = pcount + (int64_t)blocks * a.E;
  __shared__ double col[1024];
  __shared__ int32_t cnt[1024];
  __shared__ int64_t total;
  __shared__ int32_t live;
  if (threadIdx.x == 0) {
    total = 0;
    live = 0;
  }
  __syncthreads();
  const int e = threadIdx.x;
  double s = 0.0;
  int32_t c = 0;
  if (e < a.E)
    for (int b = 0; b < blocks; b++) {
      s += psum[(int64_t)b * a.E + e];
      c += pcount[(int64_t)b * a.E + e];
    }
  int32_t n = 0;
  for (int b = threadIdx.x; b < blocks; b += 1024) n += plive[b];
  atomicAdd(&live, n);
  atomicAdd((unsigned long long*)&total, (unsigned long long)c);
  __syncthreads();
  const double C = total > 1 ? (double)total : 1.0, N = live > 1 ? (double)live : 1.0;
  const double slope = (double)a.coef * a.E * c / (C * N);
  if (e < a.E) {
    a.counts[e] = c;
    a.slope[e] = (float)slope;
  }
  col[e] = e < a.E ? slope * s : 0.0;
  cnt[e] = e < a.E ? (c + a.align - 1) / a.align * a.align : 0;
  __syncthreads();
  for (int d = 512; d >= 1; d >>= 1) {
    if (e < d) col[e] += col[e + d];
    __syncthreads();
  }
  for (int d = 1; d < 1024; d <<= 1) {
    const int32_t v = e >= d ? cnt[e - d] : 0;
    __syncthreads();
    cnt[e] += v;
    __syncthreads();
  }
  if (e == 0) *a.loss = (float)col[0];
  if (a.offs && e < a.E) a.offs[e] = cnt[e];
}

template <int DT, int EPL>
__global__ __launch_bounds__(kThreads) void k_balance_backward(BalanceArgs a) {
  const int lane = threadIdx.x & 63;
  const float g = *a.dloss;
  float slope[EPL];
#pragma unroll
  for (int i = 0; i < EPL; i++) slope[i] = lane + 64 * i < a.E ? a.slope[lane + 64 * i] : 0.0f;
  for (int64_t t = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6); t < a.T; t += (int64_t)gridDim.x * kWaves) {
    float p[EPL];
    float dot = 0.0f;
    const bool live = !a.mask || a.mask[t];
    if (live) {
      softmax_row<DT, EPL>(a.logits, t, a.E, p);
#pragma unroll
      for (int i = 0; i < EPL; i++) dot += p[i] * slope[i];
#pragma unroll
      for (int d = 32; d >= 1; d >>= 1) dot += __shfl_xor(dot, d, 64);
    }
#pragma unroll
    for (int i = 0; i < EPL; i++)
      if (lane + 64 * i < a.E)
        store1<DT>(a.dlogits, t * a.E + lane + 64 * i, live ? g * (p[i] * (slope[i] - dot)) : 0.0f);
  }
}

template <int DT, int EPL>
hipError_t run(const BalanceArgs& a, bool backward, hipStream_t s) {
  if (backward) {
    const int64_t g = (a.T + kWaves - 1) / kWaves;
    k_balance_backward<DT, EPL><<<dim3((unsigned)(g < 2048 ? g : 2048)), dim3(kThreads), 0, s>>>(a);
    return hipGetLastError();
  }
  const int blocks = balance_blocks(a.T, a.E);
  k_balance<DT, EPL><<<dim3(blocks), dim3(kThreads), (kWaves + 1) * a.E * 4, s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_balance_finish<<<dim3(1), dim3(1024), 0, s>>>(a, blocks);
  return hipGetLastError();
}

template <int DT>
hipError_t by_width(const BalanceArgs& a, bool backward, hipStream_t s) {
  if (a.E <= 64) return run<DT, 1>(a, backward, s);
  if (a.E <= 128) return run<DT, 2>(a, backward, s);
  if (a.E <= 256) return run<DT, 4>(a, backward, s);
  if (a.E <= 512) return run<DT, 8>(a, backward, s);
  return run<DT, 16>(a, backward, s);
}

hipError_t by_type(int dt, const BalanceArgs& a, bool backward, hipStream_t s) {
  switch (dt) {
    case kBF16: return by_width<kBF16>(a, backward, s);
    case kFP16: return by_width<kFP16>(a, backward, s);
    default: return by_width<kFP32>(a, backward, s);
  }
}

}  // namespace

int balance_blocks(int64_t T, int) {
  const int64_t b = (T + 31) / 32;
  return b < 1 ? 1 : b > 256 ? 256 : (int)b;
}

int64_t balance_workspace(int64_t T, int E) {
  const int64_t b = balance_blocks(T, E);
  return b * E * 12 + b * 4;
}

hipError_t launch_balance(int dt, const BalanceArgs& a, hipStream_t s) { return by_type(dt, a, false, s); }
hipError_t launch_balance_backward(int dt, const BalanceArgs& a, hipStream_t s) { return by_type(dt, a, true, s); }

}  // namespace fos
