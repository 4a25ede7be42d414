// w4_linear.cu -- the dense layer on 4-bit weights (moe_w4_linear) and the
// one-time layout of a matrix (moe_w4_pack).
#include <cooperative_groups.h>

#include <atomic>
#include <type_traits>

#include "moe_host.h"
#include "w4_core.cuh"
#include "w4_tc.cuh"

// Status word of the tensor-memory kernel's bounded waits (moe_w4_linear_status):
// set when a wait gives up, otherwise untouched, so calls may share it.
static __device__ int g_w4_linear_status;

namespace moe {

namespace cg = cooperative_groups;

struct W4LinearArgs {
  const void* x;
  const uint8_t* w;
  const void* bias;  // or nullptr
  void* out;
  int batch, n_out, n_panels;
  W4Geom geom;
  long long x_stride, out_stride;  // elements between tokens
  int wait_limit, hold;            // of the tensor-memory kernel (hold: see w4_tc_stage)
};

// One CTA: 64 outputs x NT * 8 tokens x its share of K; the 8 warps split
// that share, and the CTAs of a cluster split K between them, so a matrix with
// few outputs still fills the GPU.  The partial sums are added in a fixed
// order: warps first, then the cluster's CTAs through distributed shared
// memory.  Nothing is kept in global memory between calls.
//
// Measured (device time, weights from HBM): 4,096 x 7,168 at one token 5.7 us (2.6
// TB/s), 7,168 x 2,048 at 8 tokens with zero points 5.1 us, 256 x 256 2.4 us -- the
// latency of a launch, one trip to HBM and the cluster's exchange bounds them; a
// call from Python costs the host 7 us.  16,384 x 7,168: 13.2 us at one token (4.6
// TB/s), 14.1 at 8.  At 16 tokens 23.6 us, 2.6 TB/s, and no pipe is full (tensor 40
// %, ALU 28 %): two token tiles take 128 registers and spill 4 to 136 bytes, so
// there are 3.4 warps to a scheduler (256 CTAs in 296 places), each of which issues
// every 9 cycles, waiting for loads of x and weights a third of that and mostly for
// its own dependent MMAs otherwise.
template <typename T, int NT, int GROUP, bool ZP>
__global__ void __launch_bounds__(kW4Threads, W4Cfg<NT, GROUP, ZP, kW4Warps>::kMinCtas)
    w4_linear_kernel(const __grid_constant__ W4LinearArgs a) {
  using C = W4Cfg<NT, GROUP, ZP, kW4Warps>;
  extern __shared__ __align__(1024) uint8_t w4_smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint8_t* ring = w4_smem + (size_t)warp * C::kDepth * C::kSlot;
  float* cta_sums = reinterpret_cast<float*>(w4_smem);  // over the ring, once it is empty

  cg::cluster_group cluster = cg::this_cluster();
  const int S = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int row_blk = blockIdx.x / S;
  const int n_tok = a.batch;

  const int q = rank * kW4Warps + warp, Q = S * kW4Warps;
  const int steps = w4_steps(a.geom);
  const int s0 = steps * q / Q, s1 = steps * (q + 1) / Q;

  W4Stream st;
  st.valid = 0;
  const int p0 = row_blk * kW4Panels;
#pragma unroll
  for (int m = 0; m < kW4Panels; ++m) {
    st.off[m] = p0 + m < a.n_panels ? m * a.geom.panel_bytes : 0u;
    st.valid |= p0 + m < a.n_panels ? 1u << m : 0u;
  }
  w4_stream_start<C>(st, a.w + (size_t)p0 * a.geom.panel_bytes, a.geom, s0, s1, lane);
  const T* xp[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int t = n * 8 + (lane >> 2);
    xp[n] = static_cast<const T*>(a.x) + (t < n_tok ? t : 0) * a.x_stride + s0 * (2 * kW4Tile) + 8 * (lane & 3);
  }

  const uint32_t ring_addr = smem_addr(ring);
  // launched while the kernel before it runs; nothing is read before that has
  // ended (the weights neither: it may be the one that lays them out)
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
  uint32_t p_slot = 0, slot = 0;
  auto produce = [&]() {
    if (st.left > 0) w4_stream_step<C, true>(st, ring_addr + p_slot, lane);
    cp_async_commit();
    p_slot = p_slot + C::kSlot == C::kDepth * C::kSlot ? 0 : p_slot + C::kSlot;
  };
  // the next step is in; every lane is done with the slot that is refilled
  auto advance = [&]() {
    cp_async_wait<C::kDepth - 2>();
    __syncwarp();
    produce();
  };
#pragma unroll
  for (int d = 0; d < C::kDepth - 1; ++d) produce();
  float acc[kW4Panels][NT][4] = {};
  W4X<T, C> xr;
  if (s0 < s1) w4_first_x<T, C>(xp, 2 * s0 + 1 < a.geom.tiles, xr);
  w4_run<T, C>(s0, s1, a.geom.tiles, ring, slot, xp, xr, lane, acc, advance);
  float* base = reinterpret_cast<float*>(w4_smem + C::kRing);
  constexpr int kStride = C::kSums / 4;
  w4_store_sums<T, C>(base + warp * kStride, lane, acc);
  cp_async_wait<0>();
  const float* sums[kW4Warps];
#pragma unroll
  for (int w = 0; w < kW4Warps; ++w) sums[w] = base + w * kStride;
  __syncthreads();

  const int row0 = row_blk * kW4Rows;
  auto store = [&](int tok, int row, float v) {
    const int n = row0 + row;
    if (n >= a.n_out) return;
    if (a.bias) v += W4Type<T>::to_f32(static_cast<const T*>(a.bias)[n]);
    static_cast<T*>(a.out)[tok * a.out_stride + n] = W4Type<T>::from_f32(v);
  };
  for (int i = tid; i < n_tok * kW4Rows; i += kW4Threads) {
    const int tok = i / kW4Rows, row = i % kW4Rows;
    const float v = w4_add_splits<C>(sums, tok * kW4SumPitch + row);
    if (S == 1)
      store(tok, row, v);
    else
      cta_sums[i] = v;
  }
  if (S == 1) return;
  cluster.sync();  // then every CTA of the cluster adds a share of them
  for (int i = rank * kW4Threads + tid; i < n_tok * kW4Rows; i += S * kW4Threads) {
    float v = 0.f;
    for (int r = 0; r < S; ++r) v += cluster.map_shared_rank(cta_sums, r)[i];
    store(i / kW4Rows, i % kW4Rows, v);
  }
  cluster.sync();  // no CTA leaves while another reads its sums
}

// More than 16 tokens: 256 outputs x up to 64 tokens on tcgen05 (w4_tc.cuh); the
// CTAs of a cluster split K as above.  16,384 x 7,168 at 64 tokens: 27 us.  (With
// the sums read by four warps, and each thread waiting for one remote value after
// another, 31 us.)  4,096 x 7,168 at 32 tokens: 14.8 us.  The other kernel is faster
// at every size up to 16 tokens (4.1 against 6.3 us for 256 x 1,024, 10.1 against
// 14.1 for 4,096 x 7,168, 23.4 against 23.5 for 16,384 x 7,168), and two of its
// calls of 16 tokens are slower than one of 32 here: 8.1 against 6.6, 20 against
// 14.8, 47 against 24.5.
template <typename T>
struct W4LinearItems {
  const W4LinearArgs& a;
  W4TcItem item;
  bool given;
  __device__ bool next(W4TcItem& it) {
    if (given) return false;
    given = true;
    it = item;
    return true;
  }
  __device__ const W4Geom& geom() const { return a.geom; }
  __device__ const T* rows() const { return static_cast<const T*>(a.x); }
  __device__ uint32_t row(const W4TcItem&, int t) const { return (uint32_t)t; }
  __device__ long long offset(uint32_t row) const { return row * a.x_stride; }
};

template <typename T>
__device__ __forceinline__ uint32_t pack2(T lo, T hi) {
  static_assert(sizeof(T) == 2, "16 bits");
  return (uint32_t)*reinterpret_cast<const uint16_t*>(&lo) | (uint32_t)*reinterpret_cast<const uint16_t*>(&hi) << 16;
}

template <typename T, int GROUP, bool ZP>
__global__ void __launch_bounds__(kW4TcThreads, 1) w4_linear_tc_kernel(const __grid_constant__ W4LinearArgs a) {
  extern __shared__ __align__(1024) uint8_t w4_smem[];
  __shared__ W4TcBars bars;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  cg::cluster_group cluster = cg::this_cluster();
  const int S = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int row0 = (int)(blockIdx.x / S) * kTcRows;

  // K in pairs of tiles between the CTAs: each has some (launch_linear_tc)
  const int pairs = w4_steps(a.geom);
  W4LinearItems<T> items{a, {}, false};
  items.item.tile0 = 2 * (pairs * rank / S);
  items.item.tile1 = min(a.geom.tiles, 2 * (pairs * (rank + 1) / S));
  items.item.n_tok = a.batch;
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const int p = row0 / 16 + 8 * m;
    items.item.n_panels[m] = max(0, min(8, a.n_panels - p));
    items.item.panel[m] = a.w + (size_t)(p < a.n_panels ? p : 0) * a.geom.panel_bytes;
  }
  // the rows' sums [token][row], over the B operands: the last MMAs have read them
  float* exch = reinterpret_cast<float*>(w4_smem + kTcB);
  static_assert(kTcSlots * kTcBSlot >= kTcTokens * kTcRows * 4, "rows' sums");

  // (tensor memory is held before the next kernel may come: one that takes tensor
  // memory first and then waits for this grid would never end)
  w4_tc_begin(bars, a.wait_limit);
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
  int* status = &g_w4_linear_status;
  // with one item the finishers have nothing to do until its end: they stage too
  if (warp < kTcUnpackers)
    w4_tc_unpack<T, GROUP, ZP>(w4_smem, bars, items, warp, status);
  else if (warp == kTcMmaWarp)
    w4_tc_mma<T>(w4_smem, bars, items, status);
  else if (warp - kTcUnpackers - (warp > kTcMmaWarp) < kTcSlots)
    w4_tc_stage<T, kTcSlots>(w4_smem, bars, items, warp - kTcUnpackers - (warp > kTcMmaWarp), status,
                             a.hold != 0 && blockIdx.x == 0);

  // then every warp takes 16 tokens of its quarter of both accumulators' rows
  static_assert(kW4TcThreads == 32 * 4 * (kTcTokens / 16), "a warp's quarter and tokens");
  const int c = 16 * (warp >> 2);
  if (c < a.batch && tc_wait(&bars.d_full[0], 0u, status, bars.ctl)) {
    tc_fence_after();
    constexpr float unit = W4Dequant<T, ZP>::kUnit;
    const uint32_t d = bars.tmem + ((uint32_t)(32 * (warp & 3)) << 16) + c;
    float* to = exch + c * kTcRows + 32 * (warp & 3) + lane;
    float lo[16], hi[16];
    tc5_load16(d, lo);
    tc5_load16(d + kTcTokens, hi);
#pragma unroll
    for (int n = 0; n < 16; ++n) {
      if (c + n < a.batch) {
        to[n * kTcRows] = unit * lo[n];
        to[n * kTcRows + 128] = unit * hi[n];
      }
    }
  }
  w4_tc_end(bars);

  // a thread: four rows of every (8 S)-th token, the CTAs' sums added in their order
  const int row = tid % (kTcRows / 4) * 4, n = row0 + row;
  const int step = S * (kW4TcThreads / (kTcRows / 4));
  float bias[4] = {};
  if (a.bias) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < a.n_out) bias[i] = W4Type<T>::to_f32(static_cast<const T*>(a.bias)[n + i]);
  }
  // one 8-byte store where the four exist and their address allows it
  const bool whole = n + 4 <= a.n_out && ((reinterpret_cast<uintptr_t>(a.out) | (uintptr_t)(a.out_stride * 2)) & 7) == 0;
  cluster.sync();
  auto add = [&](auto splits) {
    constexpr int N = decltype(splits)::value;  // S
    constexpr int kBatch = 8 / N;               // tokens whose 8 loads from the CTAs are in flight together
    const float* from[N];
#pragma unroll
    for (int r = 0; r < N; ++r) from[r] = cluster.map_shared_rank(exch, r) + row;
    for (int tok0 = (rank * kW4TcThreads + tid) / (kTcRows / 4); tok0 < a.batch; tok0 += kBatch * step) {
      float4 p[kBatch][N];
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
#pragma unroll
        for (int r = 0; r < N; ++r)
          if (tok0 + u * step < a.batch) p[u][r] = *reinterpret_cast<const float4*>(from[r] + (tok0 + u * step) * kTcRows);
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int tok = tok0 + u * step;
        if (tok < a.batch) {
          float v[4] = {};
#pragma unroll
          for (int r = 0; r < N; ++r) {
            v[0] += p[u][r].x;
            v[1] += p[u][r].y;
            v[2] += p[u][r].z;
            v[3] += p[u][r].w;
          }
          T* out = static_cast<T*>(a.out) + tok * a.out_stride + n;
          T o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = W4Type<T>::from_f32(v[i] + bias[i]);
          if (whole) {
            *reinterpret_cast<uint2*>(out) = make_uint2(pack2(o[0], o[1]), pack2(o[2], o[3]));
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (n + i < a.n_out) out[i] = o[i];
          }
        }
      }
    }
  };
  switch (S) {
    case 1: add(std::integral_constant<int, 1>()); break;
    case 2: add(std::integral_constant<int, 2>()); break;
    case 4: add(std::integral_constant<int, 4>()); break;
    default: add(std::integral_constant<int, 8>()); break;
  }
  cluster.sync();  // no CTA leaves while another reads its sums
}

// Plain codes to the packed layout: a thread builds one 32-bit word, another
// range of threads the group entries.  Outputs behind the last one get codes,
// scales and zero points of 0.
template <typename T>
__global__ void __launch_bounds__(256) w4_pack_kernel(const uint8_t* codes, const T* scales, const uint8_t* zeros,
                                                      uint8_t* packed, int n_out, int k, int group) {
  const int tiles = k / kW4Tile, groups = k / group;
  const bool zp = zeros != nullptr;
  const size_t panel_bytes = w4_panel_bytes(k, group, zp);
  const int p = blockIdx.y;
  uint8_t* out = packed + (size_t)p * panel_bytes;
  const int words = tiles * 128;
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < words + groups * 16; i += gridDim.x * blockDim.x) {
    if (i < words) {
      const int tile = i >> 7, lane = (i >> 2) & 31, s = i & 3;
      const int g = lane >> 2, t = lane & 3;
      const int in = tile * kW4Tile + 32 * (s >> 1) + 8 * t + 4 * (s & 1);
      uint32_t w = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = p * 16 + g + 8 * (j & 1);
        const uint32_t b = n < n_out ? codes[(size_t)n * (k / 2) + in / 2 + (j >> 1)] : 0u;
        w |= (b & 15u) << (4 * j) | (b >> 4) << (16 + 4 * j);
      }
      reinterpret_cast<uint32_t*>(out)[i] = w;
    } else {
      const int r = i - words, grp = r >> 4, g = (r >> 1) & 7, hi = r & 1;
      const int n = p * 16 + g + 8 * hi;
      T* ent = reinterpret_cast<T*>(out + (size_t)tiles * kW4TileBytes) + (size_t)grp * (zp ? 32 : 16) + g * (zp ? 4 : 2);
      ent[hi] = n < n_out ? scales[(size_t)n * groups + grp] : W4Type<T>::from_f32(0.f);
      if (zp) ent[2 + hi] = W4Type<T>::from_f32(n < n_out ? (float)(zeros[(size_t)n * groups + grp] & 15) : 0.f);
    }
  }
}

namespace {
std::atomic<int> g_w4_wait_limit{kTcWaitLimit};  // of moe_w4_linear
std::atomic<int> g_w4_hold{0};                   // launches left that hold a step back
}  // namespace

int host_w4_hold() {
  int n = g_w4_hold.load(std::memory_order_relaxed);
  while (n > 0 && !g_w4_hold.compare_exchange_weak(n, n - 1, std::memory_order_relaxed)) {
  }
  return n > 0;
}

namespace {

bool w4_shape_ok(int n_out, int k, int group) {
  if (n_out < 1 || n_out > MOE_W4_MAX_OUT || k < kW4Tile || k > MOE_W4_MAX_IN || k % kW4Tile) return false;
  return (group == 32 || group == 64 || group == 128) && k % group == 0;
}

bool dtype_ok(int dtype) { return dtype == MOE_DTYPE_BF16 || dtype == MOE_DTYPE_FP16; }

// Whether a row of out shares bytes with a row of x (rows of 16-bit elements
// whose bounding ranges may interleave, as columns of one buffer do).
bool rows_meet(const void* x, long long x_stride, int k, const void* out, long long out_stride, int n, int batch) {
  const auto span = [&](const void* p, long long stride, int row) {
    return reinterpret_cast<uintptr_t>(p) + (uintptr_t)(row * stride) * 2;
  };
  const int last = batch - 1;
  if (span(x, x_stride, last) + 2 * (uintptr_t)k <= reinterpret_cast<uintptr_t>(out) ||
      span(out, out_stride, last) + 2 * (uintptr_t)n <= reinterpret_cast<uintptr_t>(x))
    return false;
  for (int i = 0; i < batch; ++i)
    for (int j = 0; j < batch; ++j) {
      const uintptr_t a = span(x, x_stride, i), b = span(out, out_stride, j);
      if (a < b + 2 * (uintptr_t)n && b < a + 2 * (uintptr_t)k) return true;
    }
  return false;
}

// Cluster size (CTAs that split K): as many as fill two CTAs on every SM, as
// long as every warp keeps a step of its own.
int cluster_for(int row_blocks, int steps, int slots) {
  int s = 1;
  while (s < 8 && 2 * s * row_blocks <= slots && steps >= 2 * s * kW4Warps) s *= 2;
  return s;
}

template <typename T, int NT, int GROUP, bool ZP>
int launch_linear(const W4LinearArgs& a, int dev, int num_sms, cudaStream_t st) {
  using C = W4Cfg<NT, GROUP, ZP, kW4Warps>;
  static std::atomic<uint64_t> raised{0};
  const auto kern = w4_linear_kernel<T, NT, GROUP, ZP>;  // (NT token tiles: 8 (NT - 1) < batch <= 8 NT)
  const int rc = host_raise_smem(kern, C::kSmem, dev, raised);
  if (rc != MOE_OK) return rc;
  const int row_blocks = (a.n_panels + kW4Panels - 1) / kW4Panels;
  const int s = cluster_for(row_blocks, w4_steps(a.geom), C::kMinCtas * num_sms);
  const cudaError_t e = host_launch(kern, dim3((unsigned)(row_blocks * s)), kW4Threads, C::kSmem, st, s, true, a);
  return e == cudaSuccess ? MOE_OK : host_fail_cuda(e);
}

template <typename T, int GROUP, bool ZP>
int launch_linear_tc(W4LinearArgs a, int dev, int num_sms, cudaStream_t st) {
  a.wait_limit = g_w4_wait_limit.load(std::memory_order_relaxed);
  a.hold = host_w4_hold();
  static std::atomic<uint64_t> raised{0};
  const auto kern = w4_linear_tc_kernel<T, GROUP, ZP>;
  const int rc = host_raise_smem(kern, kTcSmem, dev, raised);
  if (rc != MOE_OK) return rc;
  const int row_blocks = (a.n_panels * 16 + kTcRows - 1) / kTcRows;
  // as many CTAs for K as fit one to an SM, with a step each at least; 8 for no
  // more than 8 clusters: not every GPC has room for two clusters of 8 whole SMs,
  // and 16 of them took two waves (K 7,168, 4,096 outputs, 32 tokens: 21 us in
  // clusters of 8, 14.7 in clusters of 4; 1,024 outputs, 17 tokens: 10.3 and 13.4)
  const int most = row_blocks <= 8 ? 8 : 4;
  int s = 1;
  while (s < most && 2 * s * row_blocks <= num_sms && a.geom.tiles >= 4 * s) s *= 2;
  const cudaError_t e =
      host_launch(kern, dim3((unsigned)(row_blocks * s)), kW4TcThreads, kTcSmem, st, s, true, a);
  return e == cudaSuccess ? MOE_OK : host_fail_cuda(e);
}

template <typename T, int GROUP, bool ZP>
int pick_nt(const W4LinearArgs& a, int dev, int num_sms, cudaStream_t st) {
  if (a.batch <= 8) return launch_linear<T, 1, GROUP, ZP>(a, dev, num_sms, st);
  if (a.batch <= 16) return launch_linear<T, 2, GROUP, ZP>(a, dev, num_sms, st);
  return launch_linear_tc<T, GROUP, ZP>(a, dev, num_sms, st);
}

template <typename T>
int pick_linear(const W4LinearArgs& a, int group, bool zeros, int dev, int num_sms, cudaStream_t st) {
  switch (group) {
    case 32: return zeros ? pick_nt<T, 32, true>(a, dev, num_sms, st) : pick_nt<T, 32, false>(a, dev, num_sms, st);
    case 64: return zeros ? pick_nt<T, 64, true>(a, dev, num_sms, st) : pick_nt<T, 64, false>(a, dev, num_sms, st);
    default: return zeros ? pick_nt<T, 128, true>(a, dev, num_sms, st) : pick_nt<T, 128, false>(a, dev, num_sms, st);
  }
}

}  // namespace
}  // namespace moe

extern "C" {

uint64_t moe_w4_packed_bytes(int32_t out_features, int32_t in_features, int32_t group, int32_t has_zeros) {
  if (!moe::w4_shape_ok(out_features, in_features, group)) return 0;
  return moe::w4_matrix_bytes(out_features, in_features, group, has_zeros != 0);
}

int moe_w4_pack(const void* codes, const void* scales, const void* zeros, void* packed, int32_t out_features,
                int32_t in_features, int32_t group, int32_t dtype, void* stream) {
  using namespace moe;
  if (!w4_shape_ok(out_features, in_features, group)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!dtype_ok(dtype) || !codes || !scales || !packed) return MOE_ERR_INVALID_ARG;
  if (!host_aligned(scales, 2) || !host_aligned(packed, 16)) return MOE_ERR_INVALID_ARG;
  int dev, sms;
  const int rc = host_current_device(&dev, &sms);
  if (rc != MOE_OK) return rc;
  const int items = in_features / kW4Tile * 128 + in_features / group * 16;
  const dim3 grid((unsigned)((items + 255) / 256), (unsigned)((out_features + 15) / 16));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      dtype == MOE_DTYPE_BF16
          ? host_launch(w4_pack_kernel<__nv_bfloat16>, grid, 256, 0, st, 1, false, static_cast<const uint8_t*>(codes),
                        static_cast<const __nv_bfloat16*>(scales), static_cast<const uint8_t*>(zeros),
                        static_cast<uint8_t*>(packed), (int)out_features, (int)in_features, (int)group)
          : host_launch(w4_pack_kernel<__half>, grid, 256, 0, st, 1, false, static_cast<const uint8_t*>(codes),
                        static_cast<const __half*>(scales), static_cast<const uint8_t*>(zeros),
                        static_cast<uint8_t*>(packed), (int)out_features, (int)in_features, (int)group);
  return e == cudaSuccess ? MOE_OK : host_fail_cuda(e);
}

int moe_w4_linear(const void* x, const void* packed, const void* bias, void* out, int32_t batch, int32_t in_features,
                  int32_t out_features, int32_t group, int32_t has_zeros, int64_t x_stride, int64_t out_stride,
                  int32_t dtype, void* stream) {
  using namespace moe;
  if (!w4_shape_ok(out_features, in_features, group) || batch < 0 || batch > MOE_W4_MAX_BATCH)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!dtype_ok(dtype)) return MOE_ERR_INVALID_ARG;
  if (batch == 0) return MOE_OK;
  if (!x || !packed || !out) return MOE_ERR_INVALID_ARG;
  if (!host_aligned(x, 16) || !host_aligned(packed, 16) || !host_aligned(out, 2) || !host_aligned(bias, 2))
    return MOE_ERR_INVALID_ARG;
  if (batch > 1 && (x_stride % 8 || x_stride < 0 || out_stride < out_features)) return MOE_ERR_INVALID_ARG;
  if (rows_meet(x, x_stride, in_features, out, out_stride, out_features, batch)) return MOE_ERR_INVALID_ARG;
  int dev, sms;
  const int rc = host_current_device(&dev, &sms);
  if (rc != MOE_OK) return rc;
  W4LinearArgs a{};
  a.x = x;
  a.w = static_cast<const uint8_t*>(packed);
  a.bias = bias;
  a.out = out;
  a.batch = batch;
  a.n_out = out_features;
  a.n_panels = (out_features + 15) / 16;
  a.geom.tiles = in_features / kW4Tile;
  a.geom.panel_bytes = (uint32_t)w4_panel_bytes(in_features, group, has_zeros != 0);
  a.geom.entry_off = (uint32_t)(a.geom.tiles * kW4TileBytes);
  a.x_stride = x_stride;
  a.out_stride = out_stride;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return dtype == MOE_DTYPE_BF16 ? pick_linear<__nv_bfloat16>(a, group, has_zeros != 0, dev, sms, st)
                                 : pick_linear<__half>(a, group, has_zeros != 0, dev, sms, st);
}

int moe_w4_linear_set_wait_limit(uint32_t probes) {
  using namespace moe;
  g_w4_wait_limit.store(probes == 0 || probes > (uint32_t)kTcWaitLimit ? kTcWaitLimit : (int)probes,
                        std::memory_order_relaxed);
  return MOE_OK;
}

int moe_w4_test_hold(int32_t launches) {
  if (launches < 0) return MOE_ERR_INVALID_ARG;
  moe::g_w4_hold.store(launches, std::memory_order_relaxed);
  return MOE_OK;
}

int moe_w4_linear_status(void* stream) {
  using namespace moe;
  int dev, sms;
  const int rc = host_current_device(&dev, &sms);
  if (rc != MOE_OK) return rc;
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  int st = 0;
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&st, g_w4_linear_status, sizeof st);
  if (e != cudaSuccess) return host_fail_cuda(e);
  if (st == kStatusOk) return MOE_OK;
  static_assert(kStatusOk == 0, "cleared to zero");
  void* word = nullptr;
  if ((e = cudaGetSymbolAddress(&word, g_w4_linear_status)) != cudaSuccess ||
      (e = cudaMemsetAsync(word, 0, sizeof st, static_cast<cudaStream_t>(stream))) != cudaSuccess ||
      (e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream))) != cudaSuccess)
    return host_fail_cuda(e);
  return MOE_ERR_DEVICE_TIMEOUT;
}

}  // extern "C"
