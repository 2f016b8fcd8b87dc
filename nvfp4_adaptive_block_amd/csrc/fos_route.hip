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
// rows are not read. Counts are integers; column sums of p are binary32 over at
// most 256 rows (64 of each of four lanes) and binary64 from there on, but that a
// workgroup's sum is rounded to binary32 once on its way to the join; the order is
// fixed, so that results do not depend on that of execution.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fos_device.h"
#include "fos_ops.h"

namespace fos {
namespace {

constexpr int kThreads = 512;  // forward
constexpr int kWaves = kThreads / 64;
constexpr int kRows = 64;  // that a lane adds up in binary32
constexpr int kMaxExperts = 1024;

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

// Four values from element i on, at the elements' own alignment.
struct __attribute__((packed, aligned(2))) Quad16 {
  uint32_t v[2];
};
struct __attribute__((packed, aligned(4))) Quad32 {
  float v[4];
};

template <int DT>
__device__ __forceinline__ void load4(const void* p, int64_t i, float* v) {
  if constexpr (DT == kFP32) {
    const Quad32 t = *reinterpret_cast<const Quad32*>((const float*)p + i);
#pragma unroll
    for (int j = 0; j < 4; j++) v[j] = t.v[j];
  } else {
    const Quad16 t = *reinterpret_cast<const Quad16*>((const uint16_t*)p + i);
#pragma unroll
    for (int j = 0; j < 2; j++) {
      v[2 * j] = DT == kBF16 ? bf16_lo(t.v[j]) : f16_lo(t.v[j]);
      v[2 * j + 1] = DT == kBF16 ? bf16_hi(t.v[j]) : f16_hi(t.v[j]);
    }
  }
}

template <int DT>
__device__ __forceinline__ void store4(void* p, int64_t i, const float* v) {
  if constexpr (DT == kFP32) {
    *reinterpret_cast<Quad32*>((float*)p + i) = Quad32{{v[0], v[1], v[2], v[3]}};
  } else {
    Quad16 t;
#pragma unroll
    for (int j = 0; j < 2; j++)
      t.v[j] = DT == kBF16 ? pack_bf16(v[2 * j], v[2 * j + 1]) : pack_f16(v[2 * j], v[2 * j + 1]);
    *reinterpret_cast<Quad16*>((uint16_t*)p + i) = t;
  }
}

// Reductions over the 16 lanes of a row, by rotations within a DPP row: each
// level adds the same pair in either lane, so all lanes get the same bits.
constexpr int kRor = 0x120;
__device__ __forceinline__ float sum16(float v) {
  v += dpp<kRor + 8>(v);
  v += dpp<kRor + 4>(v);
  v += dpp<kRor + 2>(v);
  v += dpp<kRor + 1>(v);
  return v;
}
__device__ __forceinline__ float max16(float v) {  // a NaN is dropped
  v = __builtin_fmaxf(v, dpp<kRor + 8>(v));
  v = __builtin_fmaxf(v, dpp<kRor + 4>(v));
  v = __builtin_fmaxf(v, dpp<kRor + 2>(v));
  v = __builtin_fmaxf(v, dpp<kRor + 1>(v));
  return v;
}

// A row of logits takes 16 lanes, so that a wave works on four and a row's
// reductions are four register rotations each. Lane l owns, in piece i, the
// four columns from 64 i + 4 l on. The lane in which E ends reads the row's
// last four instead and drops those that its neighbour has; every slot's column
// is at(i) + j, and it is the lane's own where mine() says so. (E below 4: every
// lane reads by element.) FULL: E is 64 P and every slot is its lane's own, which
// the compiler then knows: the comparisons are a fifth of the instructions, and
// these kernels are near the vector units' limit.
template <int P, bool FULL>
struct Columns {
  int E, first;
  __device__ __forceinline__ Columns(int e) : E(FULL ? 64 * P : e), first(4 * (threadIdx.x & 15)) {}
  __device__ __forceinline__ int begin(int i) const { return 64 * i + first; }
  __device__ __forceinline__ int at(int i) const {
    const int b = begin(i);
    return FULL || E < 4 ? b : b + 4 <= E ? b : E - 4;
  }
  __device__ __forceinline__ bool mine(int i, int j) const {
    return FULL || (at(i) + j >= begin(i) && at(i) + j < E);
  }
};

template <int DT, int P, bool FULL>
__device__ __forceinline__ void load_row(const void* logits, int64_t t, const Columns<P, FULL>& c, float (*v)[4]) {
#pragma unroll
  for (int i = 0; i < P; i++) {
    if (c.E < 4) {
#pragma unroll
      for (int j = 0; j < 4; j++) v[i][j] = c.mine(i, j) ? load1<DT>(logits, t * c.E + c.at(i) + j) : 0.0f;
    } else {
      load4<DT>(logits, t * c.E + c.at(i), v[i]);
    }
  }
}

// v becomes its softmax; slots that are not the lane's own and rows that are
// not live become 0. exp is the base-2 instruction: relative error about
// 1.5 |v - max| half steps. A NaN goes through exp into the sum and the whole row.
template <int P, bool FULL>
__device__ __forceinline__ void softmax(const Columns<P, FULL>& c, bool live, float (*v)[4]) {
  const float low = -__builtin_huge_valf();
  float top = low;
#pragma unroll
  for (int i = 0; i < P; i++)
#pragma unroll
    for (int j = 0; j < 4; j++) {
      v[i][j] = live && c.mine(i, j) ? v[i][j] : low;
      top = __builtin_fmaxf(top, v[i][j]);
    }
  top = max16(top);
  const float shift = top == low ? 0.0f : top;  // every logit -inf: each exp is 0
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < P; i++)
#pragma unroll
    for (int j = 0; j < 4; j++) {
      v[i][j] = __builtin_amdgcn_exp2f((v[i][j] - shift) * 1.44269504088896341f);
      sum += v[i][j];
    }
  sum = sum16(sum);
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
  for (int i = 0; i < P; i++)
#pragma unroll
    for (int j = 0; j < 4; j++) v[i][j] *= inv;
}

// The workspace: per workgroup E column sums and E counts, live rows, then the
// joined columns and the counter of the second launch.
struct Work {
  float* sums;
  int32_t* counts;
  int32_t* live;
  double* col;
  int32_t* cnt;
  int32_t* done;
  __host__ __device__ static int64_t bytes(int64_t blocks, int64_t E) {
    return (blocks * E * 8 + blocks * 4 + 7) / 8 * 8 + E * 12 + 4;
  }
  __device__ Work(void* p, int64_t blocks, int64_t E) {
    sums = (float*)p;
    counts = (int32_t*)(sums + blocks * E);
    live = counts + blocks * E;
    col = (double*)((uint8_t*)p + (blocks * E * 8 + blocks * 4 + 7) / 8 * 8);
    cnt = (int32_t*)(col + E);
    done = cnt + E;
  }
};

// The results from each expert's column sum and count (LDS, E of each), by all
// threads of a workgroup; thread t takes `per` neighbouring experts.
__device__ void finish(const BalanceArgs& a, const double* col, const int32_t* cnt, int32_t live) {
  __shared__ int32_t wave_cnt[16], wave_pad[16];
  __shared__ double wave_loss[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x / 64;
  const int per = (a.E + blockDim.x - 1) / blockDim.x;
  const int e0 = threadIdx.x * per, e1 = e0 + per < a.E ? e0 + per : a.E;
  // the host has checked that no padded count or sum of them exceeds int32
  const uint32_t align = a.align;
  auto padded = [&](int e) { return (int32_t)(((uint32_t)cnt[e] + align - 1) / align * align); };
  int32_t c = 0, pad = 0;
  for (int e = e0; e < e1; e++) {
    c += cnt[e];
    pad += padded(e);
  }
  int32_t sum = c, run = pad;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    sum += __shfl_xor(sum, d, 64);
    const int32_t o = __shfl_up(run, d, 64);
    if (lane >= d) run += o;
  }
  if (lane == 63) {
    wave_cnt[wave] = sum;
    wave_pad[wave] = run;
  }
  __syncthreads();
  int32_t all = 0, before = run - pad;
  for (int w = 0; w < waves; w++) {
    all += wave_cnt[w];
    if (w < wave) before += wave_pad[w];
  }
  const double scale = (double)a.coef * a.E / ((double)(all > 1 ? all : 1) * (double)(live > 1 ? live : 1));
  double loss = 0.0;
  for (int e = e0; e < e1; e++) {
    const double slope = scale * cnt[e];
    loss += slope * col[e];
    before += per == 1 ? pad : padded(e);
    a.counts[e] = cnt[e];
    a.slope[e] = (float)slope;
    if (a.offs) a.offs[e] = before;
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) loss += __shfl_xor(loss, d, 64);
  if (lane == 0) wave_loss[wave] = loss;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < waves; w++) loss += wave_loss[w];
    *a.loss = (float)loss;
  }
}

// Each workgroup takes a contiguous range of rows, its waves four at a time
// (the next four are loaded while these are worked on), and leaves E column
// sums, E counts and its number of live rows in the workspace; a workgroup that
// is alone finishes.
template <int DT, int P, bool FULL>
__global__ __launch_bounds__(kThreads) void k_balance(BalanceArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t per = (a.T + gridDim.x - 1) / gridDim.x;
  const int64_t t0 = per * blockIdx.x < a.T ? per * blockIdx.x : a.T, t1 = t0 + per < a.T ? t0 + per : a.T;
  __shared__ int32_t hist[64 * P];
  __shared__ double sums[kWaves][64 * P];
  __shared__ int32_t live_rows;
  for (int e = threadIdx.x; e < a.E; e += kThreads) hist[e] = 0;
  if (threadIdx.x == 0) live_rows = 0;
  __syncthreads();
  const Columns<P, FULL> c(a.E);
  float next[P][4];
  int32_t live = 0;
  int64_t t = t0 + wave * 4 + (lane >> 4);
  bool have = t < t1 && (!a.mask || a.mask[t]);
  if (have) load_row<DT, P, FULL>(a.logits, t, c, next);
  int64_t base = t0 + wave * 4;
  bool more = false;
  do {
    float acc[P][4] = {};
    for (int n = 0; n < kRows && base < t1; n++, base += 4 * kWaves) {
      float v[P][4];
#pragma unroll
      for (int i = 0; i < P; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) v[i][j] = next[i][j];
      const bool now = have;
      t += 4 * kWaves;
      have = t < t1 && (!a.mask || a.mask[t]);
      if (have) load_row<DT, P, FULL>(a.logits, t, c, next);
      softmax(c, now, v);
      live += now;
#pragma unroll
      for (int i = 0; i < P; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) acc[i][j] += v[i][j];
    }
    // the wave's four rows of lanes; the first 16 lanes own the columns
    auto add_up = [&](auto add) {
#pragma unroll
      for (int i = 0; i < P; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) {
          acc[i][j] += __shfl_xor(acc[i][j], 16, 64);
          acc[i][j] += __shfl_xor(acc[i][j], 32, 64);
          if (lane < 16 && c.mine(i, j)) add(sums[wave][c.at(i) + j], (double)acc[i][j]);
        }
    };
    if (more)
      add_up([](double& to, double d) { to += d; });
    else
      add_up([](double& to, double d) { to = d; });
    more = true;
  } while (base < t1);
  // assignments: a thread takes a row's k indices
  bool bad = false;
  for (int64_t r = t0 + threadIdx.x; r < t1; r += kThreads) {
    if (a.mask && !a.mask[r]) continue;
    for (int j = 0; j < a.k; j++) {
      const int64_t at = r * a.k + j;
      const int64_t e = a.idx64 ? ((const int64_t*)a.idx)[at] : (int64_t)((const int32_t*)a.idx)[at];
      if (e >= 0 && e < a.E)
        atomicAdd(&hist[e], 1);
      else
        bad |= e != -1;
    }
  }
  if (bad && a.status) atomicOr(a.status, kStatusBadIndex);
  if ((lane & 15) == 0 && live) atomicAdd(&live_rows, live);
  __syncthreads();
  if (gridDim.x == 1) {
    __shared__ double col[64 * P];
    for (int e = threadIdx.x; e < a.E; e += kThreads) {
      double s = 0.0;
      for (int w = 0; w < kWaves; w++) s += sums[w][e];
      col[e] = s;
    }
    __syncthreads();
    finish(a, col, hist, live_rows);
    return;
  }
  const Work w(a.work, gridDim.x, a.E);
  for (int e = threadIdx.x; e < a.E; e += kThreads) {
    double s = sums[0][e];
    for (int v = 1; v < kWaves; v++) s += sums[v][e];
    w.sums[(int64_t)blockIdx.x * a.E + e] = (float)s;
    w.counts[(int64_t)blockIdx.x * a.E + e] = hist[e];
  }
  if (threadIdx.x == 0) {
    w.live[blockIdx.x] = live_rows;
    if (blockIdx.x == 0) *w.done = 0;
  }
}

// Joins the workgroups' rows: each workgroup takes 32 columns, and the one that
// ends last (a counter that the first launch cleared) finishes. Bound by
// latency: a chain of five trips to memory, 9 us whatever T is. (One workgroup
// without the trips: 4096 x 256 15.0 us in all for 15.5, 4096 x 1000 35 for 31.)
__global__ __launch_bounds__(1024) void k_balance_join(BalanceArgs a, int blocks) {
  const Work w(a.work, blocks, a.E);
  const int c = threadIdx.x & 31, part = threadIdx.x >> 5, e = blockIdx.x * 32 + c;
  __shared__ double part_sum[16][32];
  __shared__ int32_t part_cnt[16][32];
  __shared__ double col[kMaxExperts];
  __shared__ int32_t cnt[kMaxExperts];
  __shared__ int32_t live, last;
  double s = 0.0;
  int32_t n = 0, rows = 0;
  for (int b = threadIdx.x; b < blocks; b += 1024) rows += w.live[b];
  if (e < a.E) {
#pragma unroll 8
    for (int b = part; b < blocks; b += 32) {
      s += (double)w.sums[(int64_t)b * a.E + e];
      n += w.counts[(int64_t)b * a.E + e];
    }
  }
  s += __shfl_xor(s, 32, 64);
  n += __shfl_xor(n, 32, 64);
  if (!(part & 1)) {
    part_sum[part >> 1][c] = s;
    part_cnt[part >> 1][c] = n;
  }
  if (threadIdx.x == 0) live = 0;
  __syncthreads();
  if (part == 0 && e < a.E) {
#pragma unroll
    for (int p = 1; p < 16; p++) {
      s += part_sum[p][c];
      n += part_cnt[p][c];
    }
    w.col[e] = s;
    w.cnt[e] = n;
  }
  // the workgroup's columns are released by one thread after the barrier, and
  // acquired by the one that counts last
  __syncthreads();
  if (threadIdx.x == 0)
    last = __hip_atomic_fetch_add(w.done, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == (int)gridDim.x - 1;
  __syncthreads();
  if (!last) return;
  for (int i = threadIdx.x; i < a.E; i += 1024) {
    col[i] = w.col[i];
    cnt[i] = w.cnt[i];
  }
  if (rows) atomicAdd(&live, rows);
  __syncthreads();
  finish(a, col, cnt, live);
}

template <int DT, int P, bool FULL>
__global__ __launch_bounds__(256) void k_balance_backward(BalanceArgs a) {
  const int lane = threadIdx.x & 63;
  const float g = *a.dloss;
  const Columns<P, FULL> c(a.E);
  float slope[P][4];
#pragma unroll
  for (int i = 0; i < P; i++)
#pragma unroll
    for (int j = 0; j < 4; j++) slope[i][j] = c.mine(i, j) ? a.slope[c.at(i) + j] : 0.0f;
  for (int64_t base = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * 4; base < a.T; base += (int64_t)gridDim.x * 16) {
    const int64_t t = base + (lane >> 4);
    if (t >= a.T) break;
    const bool live = !a.mask || a.mask[t];
    float v[P][4], dot = 0.0f;
    if (live) load_row<DT, P, FULL>(a.logits, t, c, v);
    softmax(c, live, v);
#pragma unroll
    for (int i = 0; i < P; i++)
#pragma unroll
      for (int j = 0; j < 4; j++) dot += v[i][j] * slope[i][j];
    dot = sum16(dot);
#pragma unroll
    for (int i = 0; i < P; i++) {
#pragma unroll
      for (int j = 0; j < 4; j++) v[i][j] = live ? g * (v[i][j] * (slope[i][j] - dot)) : 0.0f;
      if (c.E >= 4 && c.at(i) == c.begin(i)) {
        store4<DT>(a.dlogits, t * a.E + c.at(i), v[i]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; j++)
          if (c.mine(i, j)) store1<DT>(a.dlogits, t * a.E + c.at(i) + j, v[i][j]);
      }
    }
  }
}

template <int DT, int P, bool FULL>
hipError_t run(const BalanceArgs& a, bool backward, hipStream_t s) {
  if (backward) {
    const int64_t g = (a.T + 15) / 16;
    k_balance_backward<DT, P, FULL><<<dim3((unsigned)(g < 2048 ? g : 2048)), dim3(256), 0, s>>>(a);
    return hipGetLastError();
  }
  const int blocks = balance_blocks(a.T, a.E);
  k_balance<DT, P, FULL><<<dim3(blocks), dim3(kThreads), 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || blocks == 1) return e;
  k_balance_join<<<dim3((a.E + 31) / 32), dim3(1024), 0, s>>>(a, blocks);
  return hipGetLastError();
}

template <int DT, int P>
hipError_t by_fill(const BalanceArgs& a, bool backward, hipStream_t s) {
  return a.E == 64 * P ? run<DT, P, true>(a, backward, s) : run<DT, P, false>(a, backward, s);
}

template <int DT>
hipError_t by_width(const BalanceArgs& a, bool backward, hipStream_t s) {
  if (a.E <= 64) return by_fill<DT, 1>(a, backward, s);
  if (a.E <= 128) return by_fill<DT, 2>(a, backward, s);
  if (a.E <= 256) return by_fill<DT, 4>(a, backward, s);
  if (a.E <= 512) return by_fill<DT, 8>(a, backward, s);
  return by_fill<DT, 16>(a, backward, s);
}

hipError_t by_type(int dt, const BalanceArgs& a, bool backward, hipStream_t s) {
  switch (dt) {
    case kBF16: return by_width<kBF16>(a, backward, s);
    case kFP16: return by_width<kFP16>(a, backward, s);
    default: return by_width<kFP32>(a, backward, s);
  }
}

}  // namespace

// Up to 256 rows one workgroup does it all (128 x 64: 7 us, 10 with a second
// launch; 512 x 256: 19 and 13); then 64 rows each, up to two workgroups per CU.
// 65536 x 256 bf16, top 8: the forward pass reads 36 MB in 13 us and joins in 9
// (latency), the backward pass moves 67 MB in 13 us, 5.2 TB/s, the rate of a copy.
int balance_blocks(int64_t T, int) {
  const int64_t b = T <= 256 ? 1 : (T + 63) / 64;
  return b < 1 ? 1 : b > 512 ? 512 : (int)b;
}

int64_t balance_workspace(int64_t T, int E) { return Work::bytes(balance_blocks(T, E), E); }

hipError_t launch_balance(int dt, const BalanceArgs& a, hipStream_t s) { return by_type(dt, a, false, s); }
hipError_t launch_balance_backward(int dt, const BalanceArgs& a, hipStream_t s) { return by_type(dt, a, true, s); }

}  // namespace fos
