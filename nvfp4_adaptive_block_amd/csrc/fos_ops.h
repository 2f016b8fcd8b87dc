// fos_ops.h: launch interface between the C ABI (fos_api.hip) and the kernels
// of the operators around the quantizer: the NVFP4 product (fos_linear.hip),
// the RMS norm with an 8-bit output (fos_norm.hip) and the balance loss
// (fos_route.hip). Internal to the library.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fos_kernels.h"

namespace fos {

// numbering matches include/fos.h
enum { kXE4M3 = 3, kXNVFP4 = 4 };  // activation types after kBF16, kFP16
enum { kScaleNone = -1, kScaleTensor = 0, kScaleRow = 1, kScaleGroup = 2 };
enum { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };
enum { kStatusBadIndex = 8 };

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

}  // namespace fos
