// balance.cu -- the router's balance loss, the tokens per expert and the
// gradient with respect to the logits (moe_balance_loss).
//
//   p_t = softmax(logits_t + bias),  c_e = live choices of expert e,  T live tokens
//   loss = f sum_t sum_e p_te c_e,   f = coef E / (k T^2)
//   dloss / dlogits_te = grad f p_te (c_e - sum_j p_tj c_j)
//
// (f sum_t sum_e p_te c_e is coef E sum_e (c_e / (k T)) (sum_t p_te / T): the
// share of the choices times the mean probability, summed over the experts.)
//
// The counts come from the ids alone, so with them in hand one pass over the
// logits gives both the loss and the gradient, and no per-expert sum of
// probabilities is ever formed: a row needs its maximum, its sum of
// exponentials and its dot product with the counts, one number.  Instead of c
// the kernels use c - c0, c0 the mean count rounded to a whole number: the
// gradient does not change (the p of a row add up to 1), but its difference no
// longer cancels two numbers of the size of c, and the loss is
// f (T' c0 + sum_t d_t) with small d_t (T' the rows that have a softmax).
//
// Sums: a row's in fp32 across a warp; rows, warps and CTAs in fp64, in a
// fixed order (no atomics on floats), so every call gives the same bits.
//
// What bounds it: HBM -- the logits once, and the gradient once: 65,536 tokens of
// 384 experts in fp32 with the gradient in 44 us, 4.6 TB/s (by a profiler the row
// kernel takes 34 us of it and the counting before it 8, most of that in the open);
// without the gradient 27 us, in bf16 with it 35.  Few tokens are bound by latency,
// so up to 512 tokens one cluster does all of it in one launch: 5.5 us at 64
// tokens, 7.9 at 512 (5.9 and 8.9 with the gradient), where the memset and two
// kernels of more tokens take 10.3 us from 513 to 2,048.  (385 to 512 experts
// spill 40 to 48 bytes a thread at the 64 registers of two CTAs on an SM.)
#include <cooperative_groups.h>

#include <cuda_fp16.h>

#include <type_traits>

#include "moe_device.cuh"
#include "moe_host.h"

namespace moe {

namespace cg = cooperative_groups;

struct BalanceArgs {
  const void* logits;
  long long stride;       // elements between rows
  const float* bias;      // [E] or nullptr
  const int32_t* ids;     // [tokens, k]
  const uint8_t* mask;    // [tokens] or nullptr
  int tokens, E, k;
  float coef;
  float* loss;
  int32_t* counts;        // [E + 1]: choices of each expert, live tokens
  void* dlogits;          // or nullptr
  long long dstride;
  const float* grad_loss; // one float or nullptr (1)
  double* row_sums;       // [grid of the row kernel]
  unsigned* ticket;       // zeroed by the counting kernel
};

constexpr int kBalThreads = 512;
constexpr int kBalWarps = kBalThreads / 32;
constexpr int kBalMaxCtas = 1024;       // row CTAs
constexpr int kBalCluster = 8;          // CTAs of the one-launch kernel

// Count this CTA's share (part b of n) of the choices of live tokens into
// s_cnt[0..E) and the live tokens into s_cnt[E]; s_cnt is zero on entry.
__device__ __forceinline__ void balance_count(const BalanceArgs& a, int32_t* s_cnt, int b, int n) {
  // (at most 2^24 tokens of 32 choices: 32 bits hold every index)
  const unsigned total = (unsigned)a.tokens * a.k;
  for (unsigned i = b * blockDim.x + threadIdx.x; i < total; i += n * blockDim.x) {
    const int e = __ldg(a.ids + i);
    const bool live = !a.mask || __ldg(a.mask + i / (unsigned)a.k);
    if (live && (unsigned)e < (unsigned)a.E) atomicAdd(s_cnt + e, 1);
  }
  if (!a.mask) {
    if (b == 0 && threadIdx.x == 0) s_cnt[a.E] = a.tokens;
    return;
  }
  int live = 0;
  for (int t = b * blockDim.x + threadIdx.x; t < a.tokens; t += n * blockDim.x) live += __ldg(a.mask + t) != 0;
  live = __reduce_add_sync(0xffffffffu, live);
  if ((threadIdx.x & 31) == 0 && live) atomicAdd(s_cnt + a.E, live);
}

__global__ void __launch_bounds__(kBalThreads) balance_count_kernel(const __grid_constant__ BalanceArgs a) {
  extern __shared__ int32_t s_cnt[];
  cudaTriggerProgrammaticLaunchCompletion();
  for (int e = threadIdx.x; e <= a.E; e += kBalThreads) s_cnt[e] = 0;
  __syncthreads();
  balance_count(a, s_cnt, blockIdx.x, gridDim.x);
  __syncthreads();
  // (whole numbers: the order of the additions does not matter)
  for (int e = threadIdx.x; e <= a.E; e += kBalThreads)
    if (s_cnt[e]) atomicAdd(a.counts + e, s_cnt[e]);
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0u;
}

template <typename T>
__device__ __forceinline__ float4 load4(const T* p) {
  if constexpr (sizeof(T) == 4) {
    return __ldcs(reinterpret_cast<const float4*>(p));
  } else {
    const uint2 v = __ldcs(reinterpret_cast<const uint2*>(p));
    float4 r;
    if constexpr (std::is_same_v<T, __half>) {
      const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&v.x));
      const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&v.y));
      r = make_float4(lo.x, lo.y, hi.x, hi.y);
    } else {
      bf16x2_to_f32(v.x, r.x, r.y);
      bf16x2_to_f32(v.y, r.z, r.w);
    }
    return r;
  }
}
template <typename T>
__device__ __forceinline__ void store4(T* p, float4 v) {
  if constexpr (sizeof(T) == 4) {
    __stcs(reinterpret_cast<float4*>(p), v);
  } else if constexpr (std::is_same_v<T, __half>) {
    const __half2 lo = __floats2half2_rn(v.x, v.y), hi = __floats2half2_rn(v.z, v.w);
    __stcs(reinterpret_cast<uint2*>(p),
           make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi)));
  } else {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
    __stcs(reinterpret_cast<uint2*>(p),
           make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi)));
  }
}

// 2^x, flushing results below 2^-126 (two steps off at most)
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// A warp's rows r0, r0 + step, ...: lane l holds the 4 CH experts
// 4 (l + 32 i) + {0..3}.  Returns the lane-uniform sum over the rows of
// sum_e p_e c_e (c as given: counts minus c0) and adds the rows that have a
// softmax to n_rows; with dlogits writes fg p (c - that sum).  `load` is
// called before the counts are needed, so the first row is in flight while
// they are being added up.
template <typename T, int CH>
struct BalanceRows {
  float z[CH][4];
  const BalanceArgs& a;
  int lane, r;
  bool live;
  __device__ BalanceRows(const BalanceArgs& args, int row0) : a(args), lane(threadIdx.x & 31), r(row0), live(false) {
    load();
  }
  __device__ __forceinline__ void load() {
    live = r < a.tokens && (!a.mask || __ldg(a.mask + r));
    if (!live) return;
    const T* p = static_cast<const T*>(a.logits) + (size_t)r * a.stride;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int e = 4 * (lane + 32 * i);
      float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (e < a.E) v = load4(p + e);
      z[i][0] = v.x;
      z[i][1] = v.y;
      z[i][2] = v.z;
      z[i][3] = v.w;
    }
  }
  __device__ double run(int step, const float* s_c, float fg, int& n_rows) {
    float c[CH][4];
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = 4 * (lane + 32 * i) + j;
        c[i][j] = e < a.E ? s_c[e] : 0.f;
      }
    constexpr float kLog2e = 1.4426950408889634f;
    double total = 0.0;
    n_rows = 0;
    while (r < a.tokens) {
      float ex[CH][4];
      const bool now = live;
      const int row = r;
      float m = -INFINITY;
      if (now) {
        if (a.bias) {
#pragma unroll
          for (int i = 0; i < CH; ++i) {
            const int e = 4 * (lane + 32 * i);
            if (e < a.E) {
              const float* b = a.bias + e;
#pragma unroll
              for (int j = 0; j < 4; ++j) z[i][j] += __ldg(b + j);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < CH; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            ex[i][j] = z[i][j];
            m = fmaxf(m, ex[i][j]);
          }
      }
      r += step;
      load();  // the next row, under this one's arithmetic
      T* d = a.dlogits ? static_cast<T*>(a.dlogits) + (size_t)row * a.dstride : nullptr;
      if (!now) {
        if (d) {
#pragma unroll
          for (int i = 0; i < CH; ++i) {
            const int e = 4 * (lane + 32 * i);
            if (e < a.E) store4(d + e, make_float4(0.f, 0.f, 0.f, 0.f));
          }
        }
        continue;
      }
      m = warp_max(m);
      // (fmaxf drops NaN, so a row of NaN and -inf alone has none either: its
      // sums are NaN, and so are the loss and the row's gradient)
      const bool some = m != -INFINITY;
      float sum = 0.f, dot = 0.f;
      auto take = [&](float& v, float arg, float cc) {
        v = exp2_fast(arg);
        sum += v;
        dot = fmaf(v, cc, dot);
      };
      if (fabsf(m) < 0x1p+20f) {
        // one rounding more of m log2(e), the same for the whole row: below 2^-4,
        // so no exponential leaves its range, and it drops out
        const float ml = m * kLog2e;
#pragma unroll
        for (int i = 0; i < CH; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) take(ex[i][j], fmaf(ex[i][j], kLog2e, -ml), c[i][j]);
      } else {
        // the difference before the product with log2(e): at 2^31 the rounding
        // above would be 128 (a row of 2^128 or of 0: NaN), and the type's lowest
        // value times log2(e) -inf
        const float top = some ? m : 0.f;
#pragma unroll
        for (int i = 0; i < CH; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) take(ex[i][j], (ex[i][j] - top) * kLog2e, c[i][j]);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        dot += __shfl_xor_sync(0xffffffffu, dot, o);
      }
      const float inv = some ? 1.f / sum : 0.f;  // a row of -inf only has no softmax
      dot *= inv;
      total += (double)dot;
      n_rows += some;
      if (d) {
        const float g = fg * inv, gdot = g * dot;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          const int e = 4 * (lane + 32 * i);
          if (e < a.E)
            store4(d + e, make_float4(ex[i][0] * fmaf(c[i][0], g, -gdot), ex[i][1] * fmaf(c[i][1], g, -gdot),
                                      ex[i][2] * fmaf(c[i][2], g, -gdot), ex[i][3] * fmaf(c[i][3], g, -gdot)));
        }
      }
    }
    return total;
  }
};

// f = coef E / (k T^2), 0 without live tokens.
__device__ __forceinline__ double balance_factor(const BalanceArgs& a, int live) {
  return live > 0 ? (double)a.coef * a.E / ((double)a.k * live * live) : 0.0;
}
// The whole number that stands for the mean count.
__device__ __forceinline__ int balance_centre(const BalanceArgs& a, int live) {
  return (int)((long long)live * a.k / a.E);
}

// The row kernel's shared memory: centred counts, the warps' sums.
struct BalanceShared {
  double sum[kBalWarps];
  int rows[kBalWarps];
  int live, last;
};

template <typename T, int CH>
__global__ void __launch_bounds__(kBalThreads, CH <= 4 ? 2 : 1)
    balance_rows_kernel(const __grid_constant__ BalanceArgs a) {
  extern __shared__ __align__(16) uint8_t bal_smem[];
  __shared__ BalanceShared sh;
  float* s_c = reinterpret_cast<float*>(bal_smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  BalanceRows<T, CH> rows(a, blockIdx.x * kBalWarps + warp);
  cudaGridDependencySynchronize();
  for (int e = tid; e <= a.E; e += kBalThreads) {
    const int v = __ldcg(a.counts + e);
    if (e == a.E) sh.live = v;
    reinterpret_cast<int*>(s_c)[e] = v;
  }
  __syncthreads();
  const int live = sh.live, c0 = balance_centre(a, live);
  for (int e = tid; e < a.E; e += kBalThreads) s_c[e] = (float)(reinterpret_cast<int*>(s_c)[e] - c0);
  __syncthreads();
  const double f = balance_factor(a, live);
  const float fg = (float)(f * (a.grad_loss ? (double)__ldg(a.grad_loss) : 1.0));
  int n_rows;
  const double s = rows.run(gridDim.x * kBalWarps, s_c, fg, n_rows);
  if (lane == 0) {
    sh.sum[warp] = s;
    sh.rows[warp] = n_rows;
  }
  __syncthreads();
  if (tid == 0) {
    double v = 0.0;
    for (int w = 0; w < kBalWarps; ++w) v += sh.sum[w] + (double)sh.rows[w] * c0;
    __stcg(a.row_sums + blockIdx.x, v);
    __threadfence();
    sh.last = atomicAdd(a.ticket, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!sh.last || warp != 0) return;
  __threadfence();
  double v = 0.0;
  for (int b = lane; b < (int)gridDim.x; b += 32) v += __ldcg(a.row_sums + b);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (lane == 0) *a.loss = (float)(f * v);
}

// Few tokens: everything in one launch of one cluster, the counts added
// through distributed shared memory.
template <typename T, int CH>
__global__ void __launch_bounds__(kBalThreads, 1) balance_small_kernel(const __grid_constant__ BalanceArgs a) {
  extern __shared__ __align__(16) uint8_t bal_smem[];
  __shared__ BalanceShared sh;
  __shared__ double s_sum;
  int32_t* s_cnt = reinterpret_cast<int32_t*>(bal_smem);           // [E + 1] this CTA's counts
  float* s_c = reinterpret_cast<float*>(bal_smem) + a.E + 4;       // [E] centred counts
  cg::cluster_group cluster = cg::this_cluster();
  const int S = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  BalanceRows<T, CH> rows(a, rank * kBalWarps + warp);
  for (int e = tid; e <= a.E; e += kBalThreads) s_cnt[e] = 0;
  __syncthreads();
  balance_count(a, s_cnt, rank, S);
  cluster.sync();
  int live = 0;
  for (int r = 0; r < S; ++r) live += cluster.map_shared_rank(s_cnt, r)[a.E];
  const int c0 = balance_centre(a, live);
  for (int e = tid; e < a.E; e += kBalThreads) {
    int v = 0;
    for (int r = 0; r < S; ++r) v += cluster.map_shared_rank(s_cnt, r)[e];
    s_c[e] = (float)(v - c0);
    if (rank == 0) a.counts[e] = v;
  }
  if (rank == 0 && tid == 0) a.counts[a.E] = live;
  __syncthreads();
  const double f = balance_factor(a, live);
  const float fg = (float)(f * (a.grad_loss ? (double)__ldg(a.grad_loss) : 1.0));
  int n_rows;
  const double s = rows.run(S * kBalWarps, s_c, fg, n_rows);
  if (lane == 0) {
    sh.sum[warp] = s;
    sh.rows[warp] = n_rows;
  }
  __syncthreads();
  if (tid == 0) {
    double v = 0.0;
    for (int w = 0; w < kBalWarps; ++w) v += sh.sum[w] + (double)sh.rows[w] * c0;
    s_sum = v;
  }
  cluster.sync();
  if (rank == 0 && tid == 0) {
    double v = 0.0;
    for (int r = 0; r < S; ++r) v += *cluster.map_shared_rank(&s_sum, r);
    *a.loss = (float)(f * v);
  }
  cluster.sync();  // no CTA leaves while another reads its sums
}

namespace {

bool balance_shape_ok(int tokens, int E, int k) {
  return tokens >= 0 && tokens <= MOE_BALANCE_MAX_TOKENS && E >= 8 && E <= kMaxExperts && E % 8 == 0 && k >= 1 &&
         k <= kMaxTopK && k <= E;
}

template <typename T, int CH>
int launch_balance(BalanceArgs a, int num_sms, cudaStream_t st) {
  cudaError_t e;
  static_assert(kBalCluster * kBalWarps * 4 == MOE_BALANCE_ONE_LAUNCH, "tokens of the one-launch kernel");
  if (a.tokens <= MOE_BALANCE_ONE_LAUNCH) {
    int s = 1;
    while (s < kBalCluster && s * kBalWarps < a.tokens) s *= 2;
    e = host_launch(balance_small_kernel<T, CH>, dim3((unsigned)s), kBalThreads, (size_t)(2 * a.E + 4) * 4, st, s, false, a);
    return e == cudaSuccess ? MOE_OK : host_fail_cuda(e);
  }
  if ((e = cudaMemsetAsync(a.counts, 0, (size_t)(a.E + 1) * 4, st)) != cudaSuccess) return host_fail_cuda(e);
  // counting: four choices to a thread, up to one CTA to an SM
  const long long ids = (long long)a.tokens * a.k;
  const long long want = (ids + kBalThreads * 4 - 1) / (kBalThreads * 4);
  const int n_count = (int)(want < num_sms ? want : num_sms);
  e = host_launch(balance_count_kernel, dim3((unsigned)n_count), kBalThreads, (size_t)(a.E + 1) * 4, st, 1, false, a);
  if (e != cudaSuccess) return host_fail_cuda(e);
  int grid = (a.tokens + kBalWarps - 1) / kBalWarps;
  const int cap = num_sms * (CH <= 4 ? 2 : 1);
  grid = grid < cap ? grid : cap;
  grid = grid < kBalMaxCtas ? grid : kBalMaxCtas;
  e = host_launch(balance_rows_kernel<T, CH>, dim3((unsigned)grid), kBalThreads, (size_t)(a.E + 1) * 4, st, 1, true, a);
  return e == cudaSuccess ? MOE_OK : host_fail_cuda(e);
}

template <typename T>
int pick_balance(const BalanceArgs& a, int num_sms, cudaStream_t st) {
  const int ch = (a.E + 127) / 128;
  if (ch <= 1) return launch_balance<T, 1>(a, num_sms, st);
  if (ch <= 2) return launch_balance<T, 2>(a, num_sms, st);
  if (ch <= 3) return launch_balance<T, 3>(a, num_sms, st);
  if (ch <= 4) return launch_balance<T, 4>(a, num_sms, st);
  return launch_balance<T, 8>(a, num_sms, st);
}

}  // namespace
}  // namespace moe

extern "C" {

uint64_t moe_balance_workspace_bytes(int32_t n_experts) {
  if (n_experts < 8 || n_experts > moe::kMaxExperts || n_experts % 8) return 0;
  return (uint64_t)moe::kBalMaxCtas * 8 + 256;
}

int moe_balance_loss(const void* logits, const float* router_bias, const int32_t* topk_ids, const uint8_t* token_mask,
                     float* loss, int32_t* counts, void* dlogits, const float* grad_loss, int32_t tokens,
                     int32_t n_experts, int32_t top_k, int64_t logits_stride, int64_t dlogits_stride, float coef,
                     int32_t dtype, void* workspace, void* stream) {
  using namespace moe;
  if (!balance_shape_ok(tokens, n_experts, top_k)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_FP16 && dtype != MOE_DTYPE_FP32) return MOE_ERR_INVALID_ARG;
  if (!loss || !counts || (!workspace && tokens > MOE_BALANCE_ONE_LAUNCH) || (tokens > 0 && (!logits || !topk_ids))) return MOE_ERR_INVALID_ARG;
  const uintptr_t vec = dtype == MOE_DTYPE_FP32 ? 16 : 8;  // four logits at a time
  if (!host_aligned(logits, vec) || !host_aligned(dlogits, vec) || !host_aligned(topk_ids, 4) || !host_aligned(loss, 4) ||
      !host_aligned(counts, 4) || !host_aligned(router_bias, 4) || !host_aligned(grad_loss, 4) ||
      !host_aligned(workspace, 16))
    return MOE_ERR_INVALID_ARG;
  if (tokens > 1 && (logits_stride < n_experts || logits_stride % 4)) return MOE_ERR_INVALID_ARG;
  if (tokens > 1 && dlogits && (dlogits_stride < n_experts || dlogits_stride % 4)) return MOE_ERR_INVALID_ARG;
  int dev, sms;
  const int rc = host_current_device(&dev, &sms);
  if (rc != MOE_OK) return rc;
  BalanceArgs a{};
  a.logits = logits;
  a.stride = logits_stride;
  a.bias = router_bias;
  a.ids = topk_ids;
  a.mask = token_mask;
  a.tokens = tokens;
  a.E = n_experts;
  a.k = top_k;
  a.coef = coef;
  a.loss = loss;
  a.counts = counts;
  a.dlogits = dlogits;
  a.dstride = dlogits_stride;
  a.grad_loss = grad_loss;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.row_sums = reinterpret_cast<double*>(ws);
  a.ticket = reinterpret_cast<unsigned*>(ws + (size_t)kBalMaxCtas * 8);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (dtype) {
    case MOE_DTYPE_FP32: return pick_balance<float>(a, sms, st);
    case MOE_DTYPE_FP16: return pick_balance<__half>(a, sms, st);
    default: return pick_balance<__nv_bfloat16>(a, sms, st);
  }
}

}  // extern "C"
