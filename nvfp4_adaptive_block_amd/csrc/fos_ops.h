// fos_ops.h: launch interface between the C ABI (fos_api.hip) and the kernels
// of the operators around the quantizer: the NVFP4 product (fos_linear.hip),
// the RMS norm with an 8-bit output (fos_norm.hip), the balance loss
// (fos_route.hip) and the key/value cache (fos_kv.hip, fos_kv_attention.hip).
// Internal to the library.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fos_kernels.h"

namespace fos {

// numbering matches include/fos.h
enum { kXE4M3 = 3, kXNVFP4 = 4 };  // activation types after kBF16, kFP16
enum { kScaleNone = -1, kScaleTensor = 0, kScaleRow = 1, kScaleGroup = 2 };
enum { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };
enum { kStatusBadIndex = 8, kStatusBadCache = 16 };

struct LinearArgs {
  const void* x;          // [M, K] (NVFP4: [M, K/2])
  const uint8_t* xs;      // NVFP4: [M, K/16]
  const float* x_scale;   // nullable
  int x_type, x_gran;
  const uint8_t* w;       // [G, N, K/2]
  const uint8_t* ws;      // [G, N, K/16]
  const float* w_scale;
  int w_gran;
  const void* bias;       // nullable, [G, N]
  int bias_dt;
  const void* res;        // nullable, [M, N] of out_dt
  void* y;                // [M, N]
  int out_dt, act;
  int64_t M, N, K;
  const int32_t* offs;    // grouped: [G] cumulative end rows; dense: null
  int G;
  int32_t* status;        // nullable
  void* work;             // linear_workspace() bytes
};

// Bytes of workspace of a launch (G = 0: dense).
int64_t linear_workspace(int64_t M, int64_t N, int64_t K, int G);
// Whether a grid holds the tiles of a product with M, N > 0.
bool linear_fits(int64_t M, int64_t N, int64_t K, int G);
hipError_t launch_linear(const LinearArgs& a, hipStream_t s);

struct NormArgs {
  const void* x;
  const void* res;       // nullable
  const void* weight;
  int weight_dt;
  int64_t M, K;
  float eps;
  uint8_t* q;
  float* scale;
  void* h;               // nullable: x + res
  void* y;               // nullable: the normalised row before its 8-bit rounding
};

hipError_t launch_norm(int dt, const NormArgs& a, hipStream_t s);

struct BalanceArgs {
  const void* logits;
  const void* idx;
  bool idx64;
  const uint8_t* mask;   // nullable
  int64_t T;
  int E, k, align;
  float coef;
  float* loss;
  int32_t* counts;
  int32_t* offs;         // nullable
  float* slope;
  void* work;
  int32_t* status;       // nullable
  // backward
  const float* dloss;
  void* dlogits;
};

// Workgroups of a forward launch (each leaves one partial row in the
// workspace) and the workspace's bytes.
int balance_blocks(int64_t T, int E);
int64_t balance_workspace(int64_t T, int E);
hipError_t launch_balance(int dt, const BalanceArgs& a, hipStream_t s);
hipError_t launch_balance_backward(int dt, const BalanceArgs& a, hipStream_t s);

// ---------------------------------------------------------------- key/value cache

// n / d for 0 <= n < 2^31 by one multiplication: with 2^s >= d, m is
// 2^(31+s) / d rounded up, less than 2^32, and n times its excess stays below 2^(31+s).
struct FastDiv {
  uint32_t m, d;
  int s;
#ifdef __HIPCC__
  __host__ __device__
#endif
  int div(int n) const { return (int)(((uint64_t)(uint32_t)n * m) >> (31 + s)); }
};
inline FastDiv fast_div(uint32_t d) {
  int s = 0;
  while ((1u << s) < d) s++;
  return FastDiv{(uint32_t)(((uint64_t(1) << (31 + s)) + d - 1) / d), d, s};
}

// Rows of one side (keys or values): row (page H + head) P + slot has D values.
struct KvRows {
  uint8_t* codes;   // [rows, D/2]
  uint8_t* scales;  // [rows, D/16]
  float* sdec;      // [rows]
};

struct KvCache {
  KvRows k, v;
  const int32_t* table;  // [B, W]
  const int32_t* lens;   // [B]
  int64_t pages;
  int B, W, H, P, D;
  FastDiv by_page;       // / P
};

// Reports offsets and lengths out of their range to the nullable status, for a call without tokens.
hipError_t launch_kv_check(const KvCache& c, const int32_t* offs, int32_t* status, hipStream_t s);

struct KvAppendArgs {
  KvCache c;
  const void* x[2];      // k, v: rows of H D values
  int64_t stride[2];     // elements from one token to the next
  void* y[2];            // nullable: [T, H, D], the values that the cache then holds
  const int32_t* offs;
  int T;
  FastDiv by_head;       // / H
  int recipe, metric, prec, order;
  float six_b;
  int32_t* status;       // nullable
};
hipError_t launch_kv_append(int dt, const KvAppendArgs& a, hipStream_t s);

struct KvAttendArgs {
  KvCache c;             // weights: v unused
  const void* q;         // [T, H G, D]
  int64_t stride;        // elements from one token to the next
  const int32_t* offs;
  int T, G;
  FastDiv by_group;      // / G
  float scale_mant, scale_pow;  // scale log2(e) as m 2^k: m of 0 or 1 <= |m| < 4, and 2^k
  bool causal;
  void* out;             // [T, H G, D]
  float* lse;            // [T, H G]; nullable for attention, an input for weights
  float* acc;            // weights: [B, H, W P]
  int splits;            // parts of the keys per tile of rows
  bool wide;
  int64_t max_len;
  void* work;
  int32_t* status;       // nullable
};
// Parts that the keys are cut into, from sizes that the host knows.
int kv_splits(int64_t T, int B, int H, int G, int D, int64_t max_len);
// Whether a short cache is left whole, by more waves to a workgroup.
bool kv_wide(int64_t T, int B, int H, int G, int D, int64_t max_len);
int64_t kv_attend_workspace(int64_t T, int H, int G, int D, int splits);
hipError_t launch_kv_attention(int dt, const KvAttendArgs& a, hipStream_t s);
hipError_t launch_kv_weights(int dt, const KvAttendArgs& a, hipStream_t s);

struct KvEvictArgs {
  KvCache c;
  float* acc;            // [B, H, W P]
  int budget, sinks, recent;
  int32_t* new_lens;     // [B]
  int2* moves;           // [B, H, budget - recent] (from, to)
  int* counts;           // [B, H]
  int32_t* status;       // nullable
};
hipError_t launch_kv_evict(const KvEvictArgs& a, hipStream_t s);

}  // namespace fos
