// w4_experts.cuh -- the block's experts on 4-bit weights: up projection and
// SwiGLU, down projection, and the weighted combine with the residual
// (moe_decode_forward_w4).  The router and its plan are the block's own.
//
//   a[slot, c] = bf16(silu(x_t . W13[:, c]) * (x_t . W13[:, I + c]))
//   y[slot, n] = w_slot * sum_c a[slot, c] W2[c, n]
//   out[t, n]  = bf16(x[t, n] + y[t k + 0, n] + ... + y[t k + k - 1, n] + y_shared[t, n])
//
// Experts of up to 8 tokens (an mma.sync token tile): a persistent kernel for
// each projection, one template.  A CTA takes items (128 weight rows of one
// expert), the shared expert's first: those need nothing from the router, so
// with programmatic dependent launch they stream while it runs, and the wait for
// its plan comes with the first routed item.  A warp's weight ring runs ahead
// over item borders.  An item's sums are added over the CTA's warps in a fixed
// order, and every (token, expert) product keeps its own fp32 row until the
// combine adds the rows in the order of the token's choices: no atomics, the same
// bits every time.  (The rows cost 4 H bytes per choice against an expert's
// 1.5 H I: a 1,000th at I = 2048.)
//
// Experts of more tokens, and the shared expert of a batch above 8: the tcgen05
// kernel of the same two projections (w4_tc.cuh, items of 256 weight rows), beside
// which the first kind runs.  With mma.sync up to 16 tokens (two token tiles, 128
// registers and 220 to 450 bytes of spills) the full-size block took 626 us
// instead of 519 at 16 tokens, the block of 16 experts 181 instead of 138.  (The
// rule is measured with experts of 7,168 x 2,048 only.  What it costs a batch of 9
// is three launches and the shared expert no longer under the router: 339 us where
// 8 tokens take 270 for the full-size block, 31 against 22 for a block of 256 x
// 128, whose work is a tenth of a microsecond.)
//
// What bounds it.  The full-size block: HBM at 8 tokens (64 experts, zero points:
// 276 us, 5.2 TB/s), the router's 15 us and the latency of short kernels at one
// token (60 us); at 16, 32 and 64 tokens 500, 813 and 1,267 us for 391, 667 and
// 1,005 of bytes.  16 experts at 64 tokens: 179 us, of which the router takes 34,
// the up projection 85 and the down projection 55: steps of w4_tc.cuh, and a last
// wave of items that fills the GPU in part (272 items of the up projection on 148
// SMs, 476 of the down projection).  Registers: 128 with 8 to 104 bytes of spills
// in w4_expert_kernel, 116 to 121 without in the tcgen05 kernel.
#pragma once

#include "moe_device.cuh"
#include "w4_core.cuh"
#include "w4_tc.cuh"

namespace moe {

// One phase of an expert kernel: the shared expert's items, then the routed.
struct W4Phase {
  W4Geom geom;
  int blocks;              // blocks of 64 weight rows of a unit (UP: 32 gate rows and their 32 up rows)
  int items;               // of a unit: ceil(blocks / row groups of a CTA)
  uint32_t items_inv;      // ceil(2^32 / items) (0 for 1): i / items by one multiplication, exact for i * items < 2^32
  uint32_t up_off;         // UP: bytes from a gate panel to its up panel
  const __nv_bfloat16* x;  // activations [rows, x_cols]
  int x_cols;
  void* out;               // UP: bf16 [rows, out_cols]; DOWN: float [rows, out_cols]
  int out_cols;
};

// The units a kernel takes: the plan's, or a list of some of them.
struct W4Units {
  const int *n, *expert, *begin, *count;
};

struct W4ExpertArgs {
  W4Phase ph[2];  // 0: shared expert, 1: routed experts
  const uint8_t* shared_w;
  int n_su;       // units of the shared expert, 0 without one or where another kernel has it
  int batch, top_k;
  W4Units units;
  const int* assign_slot;
  const float* assign_w;
  // Where both kernels of a projection run, w4_expert_tc_kernel comes first: it
  // waits for what is before it and lets this kernel start beside it, which waits
  // for it in the end (so that who waits for this one has waited for both).
  int beside;
  int* status;    // w4_expert_tc_kernel: status word and limit of its waits
  int wait_limit;
  int hold;       // testing: see w4_tc_stage
};

// An item's unit: loaded one item before the lane's tokens are, which are
// loaded one item before they are used -- no load of the plan is waited for
// where it is issued.
struct W4Unit {
  int count;  // tokens, 0: no such item
  int begin;  // shared: first token; routed: first assignment of the plan
};

constexpr int kW4LightTokens = 8;  // of an expert, at most, that stays with w4_expert_kernel
constexpr int kW4ExpertSplit = 4;  // warps that split K; the CTA's other factor of 2 stands in the rows

template <int GROUP, bool ZP, bool DOWN>
__global__ void __launch_bounds__(kW4Threads, W4Cfg<1, GROUP, ZP, kW4ExpertSplit>::kMinCtas)
    w4_expert_kernel(const __grid_constant__ W4ExpertArgs a, const __grid_constant__ ExpertTable tab) {
  using C = W4Cfg<1, GROUP, ZP, kW4ExpertSplit>;
  using T = __nv_bfloat16;
  extern __shared__ __align__(1024) uint8_t w4_smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ks = warp % C::KS, rg = warp / C::KS;  // share of K, row group
  uint8_t* ring = w4_smem + (size_t)warp * C::kDepth * C::kSlot;
  const uint32_t ring_addr = smem_addr(ring);
  float* sums = reinterpret_cast<float*>(w4_smem + C::kRing);  // the warps' sums of an item

  __shared__ int s_row[2][kW4LightTokens];   // output rows of an item's tokens (by item parity)
  __shared__ float s_wt[2][kW4LightTokens];  // DOWN: their routing weights

  const int shared_items = a.n_su * a.ph[0].items;
  const int step = gridDim.x;
  int n_items = shared_items;  // all items, once the plan has been read
  bool have_plan = false;
  auto read_plan = [&]() {
    if (have_plan) return;
    if (!a.beside) cudaGridDependencySynchronize();
    n_items = shared_items + __ldcg(a.units.n) * a.ph[1].items;
    have_plan = true;
  };
  // the next grid may be put in place as this one's CTAs leave; it waits for
  // this grid's completion before it reads anything of it
  cudaTriggerProgrammaticLaunchCompletion();

  // phase, unit and block of an item
  auto place = [&](int item, int& ph, int& u, int& blk) {
    ph = item >= shared_items;
    const uint32_t i = item - (ph ? shared_items : 0), inv = a.ph[ph].items_inv;
    u = inv ? __umulhi(i, inv) : i;
    blk = (i - u * a.ph[ph].items) * C::RW;
  };
  // this warp's steps of K in a phase
  auto steps_of = [&](int ph, int& s0, int& s1) {
    const int n = w4_steps(a.ph[ph].geom);
    s0 = n * ks / C::KS;
    s1 = n * (ks + 1) / C::KS;
  };

  // ---- the weight stream: runs up to kDepth - 1 steps ahead of the products,
  // over the borders of items; once the plan is there, the expert of the item
  // after the stream's present one is on its way early
  int p_item = blockIdx.x, p_expert = 0;
  uint32_t p_slot = 0;
  bool p_known = false;
  auto p_fetch = [&]() {  // the expert of item p_item
    p_known = true;
    if (p_item < shared_items || p_item >= n_items) return;
    int ph, u, blk;
    place(p_item, ph, u, blk);
    p_expert = __ldcg(a.units.expert + u);
  };
  W4Stream st;
  st.valid = 0xfu;
  auto p_locate = [&]() {  // start the stream of item p_item (its expert fetched); false: no more
    for (;;) {
      if (p_item >= shared_items) read_plan();
      if (p_item >= n_items) return false;
      int ph, u, b, s0, s1;
      place(p_item, ph, u, b);
      b += rg;
      steps_of(ph, s0, s1);
      const W4Phase& P = a.ph[ph];
      if (!p_known) p_fetch();
      const uint8_t* w = ph ? reinterpret_cast<const uint8_t*>(tab.p[p_expert]) : a.shared_w;
      p_item += step;
      p_known = false;
      if (s0 >= s1 || b >= P.blocks) continue;  // nothing for this warp
#pragma unroll
      for (int m = 0; m < kW4Panels; ++m)
        st.off[m] = DOWN ? m * P.geom.panel_bytes : (m & 1) * P.geom.panel_bytes + (m >> 1) * P.up_off;
      w4_stream_start<C>(st, w + (size_t)b * (DOWN ? kW4Panels : 2) * P.geom.panel_bytes, P.geom, s0, s1, lane);
      return true;
    }
  };
  bool p_more = p_locate();
  uint32_t slot = 0;
  auto produce = [&]() {
    if (p_more) {
      w4_stream_step<C, false>(st, ring_addr + p_slot, lane);
      if (have_plan && !p_known) p_fetch();
      if (st.left <= 0) p_more = p_locate();
    }
    cp_async_commit();
    p_slot = p_slot + C::kSlot == C::kDepth * C::kSlot ? 0 : p_slot + C::kSlot;
  };
  // the next step is in; every lane is done with the slot that is refilled
  auto advance = [&]() {
    cp_async_wait<C::kDepth - 2>();
    __syncwarp();
    produce();
  };
#pragma unroll 1
  for (int d = 0; d < C::kDepth - 1; ++d) produce();

  // ---- the products
  auto unit_of = [&](int item, W4Unit& un) {
    if (item >= shared_items) read_plan();
    un.count = un.begin = 0;
    if (item >= n_items) return;
    int ph, u, blk;
    place(item, ph, u, blk);
    if (ph) {
      un.begin = __ldcg(a.units.begin + u);
      un.count = __ldcg(a.units.count + u);
    } else {
      un.begin = 0;
      un.count = a.batch;
    }
  };
  // the lane's token: row of the activations (routed: the assignment's slot), the
  // first token's for one that does not exist
  auto slot_of = [&](const W4Unit& un, bool routed, int& slot) {
    if (un.count == 0) return;
    const int t = lane >> 2, i = un.begin + (t < un.count ? t : 0);
    slot = routed ? __ldcg(a.assign_slot + i) : i;
  };
  auto row_of = [&](int slot, int ph, int s0, const T* (&xp)[1]) {
    const int row = ph && !DOWN ? (int)((unsigned)slot / (unsigned)a.top_k) : slot;
    xp[0] = a.ph[ph].x + (size_t)row * a.ph[ph].x_cols + s0 * (2 * kW4Tile) + 8 * (lane & 3);
  };

  if constexpr (DOWN) read_plan();  // the activations are complete
  W4Unit un, next;
  int next_slot = 0;
  unit_of(blockIdx.x, un);
  unit_of(blockIdx.x + step, next);
  W4X<T, C> xr;
  const T* xp[1];
  int parity = 0;
  if (un.count > 0) {
    const int ph = (int)blockIdx.x >= shared_items;
    int s0, s1;
    steps_of(ph, s0, s1);
    slot_of(un, ph, next_slot);
    row_of(next_slot, ph, s0, xp);
    if (s0 < s1) w4_first_x<T, C>(xp, 2 * s0 + 1 < a.ph[ph].geom.tiles, xr);
  }
  for (int item = blockIdx.x;; item += step) {
    if (item >= shared_items) read_plan();
    if (item >= n_items) break;
    int ph, u, b0;  // b0: the item's first block
    place(item, ph, u, b0);
    const W4Phase& P = a.ph[ph];
    int s0, s1;
    steps_of(ph, s0, s1);
    if (b0 + rg >= P.blocks) s1 = s0;  // no rows for this warp
    const int next_ph = item + step >= shared_items;
    slot_of(next, next_ph, next_slot);
    W4Unit after;
    unit_of(item + 2 * step, after);
    if (warp == 0 && lane < un.count) {
      s_row[parity][lane] = ph ? __ldcg(a.assign_slot + un.begin + lane) : un.begin + lane;
      if constexpr (DOWN) s_wt[parity][lane] = ph ? __ldcg(a.assign_w + un.begin + lane) : 1.f;
    }
    float acc[kW4Panels][1][4] = {};
    w4_run<T, C>(s0, s1, P.geom.tiles, ring, slot, xp, xr, lane, acc, advance);
    if (next.count > 0) {  // the next item's first activations, under this one's epilogue
      int n0, n1;
      steps_of(next_ph, n0, n1);
      row_of(next_slot, next_ph, n0, xp);
      if (n0 < n1) w4_first_x<T, C>(xp, 2 * n0 + 1 < a.ph[next_ph].geom.tiles, xr);
    }
    __syncthreads();  // the last item's sums have been read
    w4_store_sums<T, C>(sums + warp * (C::kSums / 4), lane, acc);
    __syncthreads();

    // thread: a row (of 128) of every second token; UP: a column (of 64) of every fourth
    constexpr int kOut = DOWN ? C::kRows : C::kRows / 2;
    const int col = tid % kOut, group = DOWN ? col / kW4Rows : col / 32, row = DOWN ? col % kW4Rows : col % 32;
    const float* of[C::KS];
#pragma unroll
    for (int w = 0; w < C::KS; ++w) of[w] = sums + (group * C::KS + w) * (C::kSums / 4);
    const int out_col = b0 * (kOut / C::RW) + col;
    if (out_col < P.out_cols) {
      for (int tok = tid / kOut; tok < un.count; tok += kW4Threads / kOut) {
        const size_t at = (size_t)s_row[parity][tok] * P.out_cols + out_col;
        const float v = w4_add_splits<C>(of, tok * kW4SumPitch + row);
        if constexpr (DOWN) {
          static_cast<float*>(P.out)[at] = s_wt[parity][tok] * v;
        } else {  // 32 gate rows, then their 32 up rows
          const float up = w4_add_splits<C>(of, tok * kW4SumPitch + row + 32);
          static_cast<T*>(P.out)[at] = __float2bfloat16_rn(silu_f32(v) * up);
        }
      }
    }
    un = next;
    next = after;
    parity ^= 1;
  }
  if (a.beside) cudaGridDependencySynchronize();
}

// ------------------------------------------------ experts of many tokens (tcgen05)
// Above 8 tokens of a batch, experts that have more than 8 of them, and the
// shared expert, go to w4_expert_tc_kernel with all their tokens at once; a
// one-CTA kernel splits the plan's units (an expert's consecutive ones are joined).
struct W4Split {
  int n_light, n_heavy, pad_[2];
  int light[3][kMaxUnits];  // expert, begin, count
  int heavy[3][kMaxExperts];
};

__global__ void __launch_bounds__(1024) w4_split_kernel(const Plan* plan, W4Split* out) {
  __shared__ int s_warp[2][33];
  cudaGridDependencySynchronize();
  cudaTriggerProgrammaticLaunchCompletion();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = plan->n_active;
  int base[2] = {0, 0};  // light, heavy so far
  for (int u0 = 0; u0 < n; u0 += 1024) {
    const int u = u0 + tid;
    int expert = -1, count = 0, kind = -1;
    if (u < n) {
      expert = plan->unit_expert[u];
      if (u == 0 || plan->unit_expert[u - 1] != expert) {
        for (int v = u; v < n && plan->unit_expert[v] == expert; ++v) count += plan->unit_count[v];
        kind = count > kW4LightTokens;
      }
    }
    unsigned m[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      m[k] = __ballot_sync(0xffffffffu, kind == k);
      if (lane == 0) s_warp[k][warp] = __popc(m[k]);
    }
    __syncthreads();
    if (warp < 2) {  // exclusive scan of the warps' numbers
      const int v = s_warp[warp][lane];
      int inc = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += t;
      }
      s_warp[warp][lane] = inc - v;
      if (lane == 31) s_warp[warp][32] = inc;
    }
    __syncthreads();
    if (kind >= 0) {
      const int at = base[kind] + s_warp[kind][warp] + __popc(m[kind] & ((1u << lane) - 1u));
      int* e = kind ? &out->heavy[0][at] : &out->light[0][at];
      const int pitch = kind ? kMaxExperts : kMaxUnits;
      e[0] = expert;
      e[pitch] = plan->unit_begin[u];
      e[2 * pitch] = count;
    }
    base[0] += s_warp[0][32];
    base[1] += s_warp[1][32];
    __syncthreads();
  }
  if (tid == 0) {
    out->n_light = base[0];
    out->n_heavy = base[1];
  }
}

// A CTA's items, 256 weight rows each: UP: 128 gate rows and their 128 up rows.
template <bool DOWN>
struct W4ExpertItems {
  const W4ExpertArgs& a;
  const ExpertTable& tab;
  int idx, step, shared, total;  // the next item, ..., items of the shared expert, all items
  int ph, blk, begin;            // the present one
  __device__ bool next(W4TcItem& it) {
    if (idx >= total) return false;
    ph = idx >= shared;
    const uint32_t i = idx - (ph ? shared : 0);
    const W4Phase& P = a.ph[ph];
    const int u = P.items_inv ? __umulhi(i, P.items_inv) : i;
    blk = i - u * P.items;
    idx += step;
    const uint8_t* w;
    if (ph) {
      w = reinterpret_cast<const uint8_t*>(tab.p[__ldcg(a.units.expert + u)]);
      begin = __ldcg(a.units.begin + u);
      it.n_tok = __ldcg(a.units.count + u);
    } else {
      w = a.shared_w;
      begin = 0;
      it.n_tok = a.batch;
    }
    const int panels = P.out_cols / 16;  // of one projection
    if constexpr (DOWN) {
      it.panel[0] = w + (size_t)(16 * blk) * P.geom.panel_bytes;
      it.panel[1] = it.panel[0] + (size_t)8 * P.geom.panel_bytes;
      it.n_panels[0] = min(8, panels - 16 * blk);
      it.n_panels[1] = max(0, min(8, panels - 16 * blk - 8));
      if (it.n_panels[1] == 0) it.panel[1] = it.panel[0];
    } else {
      it.panel[0] = w + (size_t)(8 * blk) * P.geom.panel_bytes;
      it.panel[1] = it.panel[0] + P.up_off;
      it.n_panels[0] = it.n_panels[1] = min(8, panels - 8 * blk);
    }
    it.tile0 = 0;
    it.tile1 = P.geom.tiles;
    return true;
  }
  __device__ const W4Geom& geom() const { return a.ph[ph].geom; }
  __device__ int slot(int t) const { return ph ? __ldcg(a.assign_slot + begin + t) : t; }
  __device__ const __nv_bfloat16* rows() const { return a.ph[ph].x; }
  __device__ uint32_t row(const W4TcItem&, int t) const {
    const uint32_t s = (uint32_t)slot(t);
    return ph && !DOWN ? s / (uint32_t)a.top_k : s;
  }
  __device__ long long offset(uint32_t row) const { return (long long)row * a.ph[ph].x_cols; }
};

template <int GROUP, bool ZP, bool DOWN>
__global__ void __launch_bounds__(kW4TcThreads, 1)
    w4_expert_tc_kernel(const __grid_constant__ W4ExpertArgs a, const __grid_constant__ ExpertTable tab) {
  using T = __nv_bfloat16;
  extern __shared__ __align__(1024) uint8_t w4_smem[];
  __shared__ W4TcBars bars;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  w4_tc_begin(bars, a.wait_limit);
  cudaGridDependencySynchronize();
  cudaTriggerProgrammaticLaunchCompletion();
  const int shared = a.n_su * a.ph[0].items;
  W4ExpertItems<DOWN> items{a, tab, (int)blockIdx.x, (int)gridDim.x, shared,
                            shared + __ldcg(a.units.n) * a.ph[1].items, 0, 0, 0};
  if (warp < kTcUnpackers) {
    w4_tc_unpack<T, GROUP, ZP>(w4_smem, bars, items, warp, a.status);
  } else if (warp < kTcMmaWarp) {
    const int f = warp - kTcUnpackers;
    // output rows (and routing weights) of tokens lane and lane + 32
    int slot[kTcTokens / 32];
    float wt[kTcTokens / 32];
    const auto ready = [&](const W4ExpertItems<DOWN>& now, const W4TcItem& it) {
#pragma unroll
      for (int h = 0; h < kTcTokens / 32; ++h) {
        const int t = 32 * h + lane;
        slot[h] = t < it.n_tok ? now.slot(t) : 0;
        if constexpr (DOWN) wt[h] = t < it.n_tok && now.ph ? __ldcg(a.assign_w + now.begin + t) : 1.f;
      }
    };
    w4_tc_finish(bars, items, f, a.status, ready,
                 [&](const W4ExpertItems<DOWN>& now, const W4TcItem& it, int c, const float (&lo)[16], const float (&hi)[16]) {
                   constexpr float unit = W4Dequant<T, ZP>::kUnit;
                   const W4Phase& P = a.ph[now.ph];
                   const int col = now.blk * (DOWN ? kTcRows : kTcRows / 2) + 32 * f + lane;
#pragma unroll
                   for (int n = 0; n < 16; ++n) {
                     if (c + n < it.n_tok) {
                       const int from = (c + n) & 31;
                       const size_t row = (size_t)__shfl_sync(0xffffffffu, c < 32 ? slot[0] : slot[1], from) * P.out_cols;
                       if constexpr (DOWN) {
                         const float w = unit * __shfl_sync(0xffffffffu, c < 32 ? wt[0] : wt[1], from);
                         float* y = static_cast<float*>(P.out) + row;
                         if (col < P.out_cols) y[col] = w * lo[n];
                         if (col + 128 < P.out_cols) y[col + 128] = w * hi[n];
                       } else if (col < P.out_cols) {
                         static_cast<T*>(P.out)[row + col] = __float2bfloat16_rn(silu_f32(unit * lo[n]) * (unit * hi[n]));
                       }
                     }
                   }
                 });
  } else if (warp == kTcMmaWarp) {
    w4_tc_mma<T>(w4_smem, bars, items, a.status);
  } else {
    w4_tc_stage<T, kTcStagers>(w4_smem, bars, items, warp - kTcMmaWarp - 1, a.status,
                               a.hold != 0 && blockIdx.x == 0);
  }
  w4_tc_end(bars);
}

// out[t, c] = bf16_rne(x[t, c] + sum_j y[t k + j, c] + y_shared[t, c]); PARTIAL:
// the fp32 sum without x.  Four columns per thread.
template <bool PARTIAL>
__global__ void __launch_bounds__(256) w4_combine_kernel(const __nv_bfloat16* x, const float* y, const float* y_s,
                                                         void* out, int batch, int hidden, int top_k) {
  cudaGridDependencySynchronize();
  cudaTriggerProgrammaticLaunchCompletion();
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  const int per_row = hidden / 4;
  if (i >= batch * per_row) return;
  const int t = i / per_row, c = (i - t * per_row) * 4;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  const float* p = y + (size_t)t * top_k * hidden + c;
#pragma unroll 8
  for (int j = 0; j < top_k; ++j) {
    const float4 v = __ldcg(reinterpret_cast<const float4*>(p + (size_t)j * hidden));
    s.x += v.x;
    s.y += v.y;
    s.z += v.z;
    s.w += v.w;
  }
  if (y_s) {
    const float4 v = __ldcg(reinterpret_cast<const float4*>(y_s + (size_t)t * hidden + c));
    s.x += v.x;
    s.y += v.y;
    s.z += v.z;
    s.w += v.w;
  }
  const size_t at = (size_t)t * hidden + c;
  if constexpr (PARTIAL) {
    *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = s;
  } else {
    const uint2 xv = *reinterpret_cast<const uint2*>(x + at);
    float x0, x1, x2, x3;
    bf16x2_to_f32(xv.x, x0, x1);
    bf16x2_to_f32(xv.y, x2, x3);
    const __nv_bfloat162 lo = __floats2bfloat162_rn(x0 + s.x, x1 + s.y), hi = __floats2bfloat162_rn(x2 + s.z, x3 + s.w);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out) + at) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  }
}

}  // namespace moe
