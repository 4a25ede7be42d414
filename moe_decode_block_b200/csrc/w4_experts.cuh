// w4_experts.cuh -- the block's experts on 4-bit weights: up projection and
// SwiGLU, down projection, and the weighted combine with the residual
// (moe_decode_forward_w4).  The router and its plan are the block's own.
//
//   a[slot, c] = bf16(silu(x_t . W13[:, c]) * (x_t . W13[:, I + c]))
//   y[slot, n] = w_slot * sum_c a[slot, c] W2[c, n]
//   out[t, n]  = bf16(x[t, n] + y[t k + 0, n] + ... + y[t k + k - 1, n] + y_shared[t, n])
//
// Two persistent kernels of one template: a CTA takes items (128 weight rows of
// one unit -- an expert and up to 32 of its tokens), the shared expert's first:
// those need nothing from the router, so with programmatic dependent launch
// they stream while it runs, and the wait for its plan comes with the first
// routed item.  A warp's weight ring runs ahead over item borders.  An item's
// sums are added over the CTA's warps in a fixed order, and every (token,
// expert) product keeps its own fp32 row until the combine adds the rows in
// the order of the token's choices: no atomics, the same bits every time.
// (The rows cost 4 H bytes per choice against an expert's 1.5 H I: a 1,000th
// at I = 2048.)
#pragma once

#include "moe_device.cuh"
#include "w4_core.cuh"

namespace moe {

// One phase of an expert kernel: the shared expert's items, then the routed.
struct W4Phase {
  W4Geom geom;
  int blocks;              // blocks of 64 weight rows of a unit (UP: 32 gate rows and their 32 up rows)
  int items;               // of a unit: ceil(blocks / row groups of a CTA)
  uint32_t up_off;         // UP: bytes from a gate panel to its up panel
  const __nv_bfloat16* x;  // activations [rows, x_cols]
  int x_cols;
  void* out;               // UP: bf16 [rows, out_cols]; DOWN: float [rows, out_cols]
  int out_cols;
};

struct W4ExpertArgs {
  W4Phase ph[2];  // 0: shared expert, 1: routed experts
  const uint8_t* shared_w;
  int n_su;       // units of the shared expert: ceil(batch / 32), 0 without one
  int batch, top_k;
  const Plan* plan;
};

// A unit's tokens as seen by one lane.
template <int NT>
struct W4Unit {
  int count;    // tokens of the unit
  int begin;    // shared: first token; routed: first assignment of the plan
  int row[NT];  // activation row of the lane's token in each tile, -1: none
};

constexpr int kW4ExpertSplit = 4;  // warps that split K; the CTA's other factor of 2 stands in the rows

template <int NT, int GROUP, bool ZP, bool DOWN>
__global__ void __launch_bounds__(kW4Threads, W4Cfg<NT, GROUP, ZP, kW4ExpertSplit>::kMinCtas)
    w4_expert_kernel(const __grid_constant__ W4ExpertArgs a, const __grid_constant__ ExpertTable tab) {
  using C = W4Cfg<NT, GROUP, ZP, kW4ExpertSplit>;
  using T = __nv_bfloat16;
  extern __shared__ __align__(1024) uint8_t w4_smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ks = warp % C::KS, rg = warp / C::KS;
  uint8_t* ring = w4_smem + (size_t)warp * C::kDepth * C::kSlot;
  const uint32_t ring_addr = smem_addr(ring);
  float* red = reinterpret_cast<float*>(w4_smem + (size_t)kW4Warps * C::kDepth * C::kSlot);

  const int shared_items = a.n_su * a.ph[0].items;
  const int step = gridDim.x;
  int n_items = shared_items;  // all items, once the plan has been read
  bool have_plan = false;
  auto read_plan = [&]() {
    if (have_plan) return;
    cudaGridDependencySynchronize();
    n_items = shared_items + __ldcg(&a.plan->n_active) * a.ph[1].items;
    have_plan = true;
  };
  // the next grid may be put in place as this one's CTAs leave; it waits for
  // this grid's completion before it reads anything of it
  cudaTriggerProgrammaticLaunchCompletion();

  // this warp's steps of K in a phase
  auto steps_of = [&](int ph, int& s0, int& s1) {
    const int n = w4_steps(a.ph[ph].geom);
    s0 = n * ks / C::KS;
    s1 = n * (ks + 1) / C::KS;
  };

  // ---- the weight stream: runs up to kDepth - 1 steps ahead of the products,
  // over the borders of items
  int p_item = blockIdx.x, p_slot = 0;
  W4Stream st;
  st.valid = 0xfu;
  auto p_locate = [&]() {  // the stream's place for item p_item; false: no more
    for (;; p_item += step) {
      if (p_item >= shared_items) read_plan();
      if (p_item >= n_items) return false;
      const int ph = p_item >= shared_items;
      const W4Phase& P = a.ph[ph];
      const int i = p_item - (ph ? shared_items : 0);
      const int u = i / P.items, b = (i - u * P.items) * C::RW + rg;
      int s0, s1;
      steps_of(ph, s0, s1);
      if (s0 >= s1 || b >= P.blocks) continue;  // nothing for this warp
      const uint8_t* w = ph ? reinterpret_cast<const uint8_t*>(tab.p[__ldcg(&a.plan->unit_expert[u])]) : a.shared_w;
#pragma unroll
      for (int m = 0; m < kW4Panels; ++m)
        st.off[m] = DOWN ? m * P.geom.panel_bytes : (m & 1) * P.geom.panel_bytes + (m >> 1) * P.up_off;
      w4_stream_start<C>(st, w + (size_t)b * (DOWN ? kW4Panels : 2) * P.geom.panel_bytes, P.geom, s0, s1, lane);
      return true;
    }
  };
  bool p_more = p_locate();
  auto produce = [&]() {
    if (p_more) {
      w4_stream_step<C, false>(st, ring_addr + p_slot, lane);
      if (st.left <= 0) {
        p_item += step;
        p_more = p_locate();
      }
    }
    cp_async_commit();
    p_slot = p_slot + C::kSlot == C::kDepth * C::kSlot ? 0 : p_slot + C::kSlot;
  };
#pragma unroll 1
  for (int d = 0; d < C::kDepth - 1; ++d) produce();

  // ---- the products
  auto unit_of = [&](int item, W4Unit<NT>& un) {
    if (item >= shared_items) read_plan();
    un.count = 0;
    if (item >= n_items) return;
    const int ph = item >= shared_items;
    const int i = item - (ph ? shared_items : 0);
    const int u = i / a.ph[ph].items;
    un.begin = ph ? __ldcg(&a.plan->unit_begin[u]) : u * kMaxUnitTokens;
    un.count = ph ? __ldcg(&a.plan->unit_count[u]) : min(kMaxUnitTokens, a.batch - un.begin);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int t = n * 8 + (lane >> 2);
      un.row[n] = -1;
      if (t < un.count) {
        const int slot = ph ? __ldcg(&a.plan->assign_slot[un.begin + t]) : un.begin + t;
        un.row[n] = (ph && !DOWN) ? slot / a.top_k : slot;
      }
    }
  };
  auto rows_of = [&](const W4Unit<NT>& un, int ph, const T* (&xp)[NT]) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
      xp[n] = un.count > 0 && un.row[n] >= 0
                  ? a.ph[ph].x + (size_t)un.row[n] * a.ph[ph].x_cols + 8 * (lane & 3)
                  : nullptr;
  };

  if constexpr (DOWN) read_plan();  // the activations are complete
  W4Unit<NT> next;
  unit_of(blockIdx.x, next);
  uint4 xa[NT][2], xb[NT][2];
  int slot = 0;
  {
    const int ph = (int)blockIdx.x >= shared_items;
    int s0, s1;
    steps_of(ph, s0, s1);
    const T* xp[NT];
    rows_of(next, ph, xp);
    w4_load_x<T, NT>(xp, 2 * s0, s0 < s1, xa);
  }
  for (int item = blockIdx.x;; item += step) {
    if (item >= shared_items) read_plan();
    if (item >= n_items) break;
    const int ph = item >= shared_items;
    const W4Phase& P = a.ph[ph];
    const W4Unit<NT> un = next;
    const int n_tok_tiles = (un.count + 7) >> 3;
    const int i = item - (ph ? shared_items : 0);
    const int b0 = i % P.items * C::RW;  // the item's first block
    int s0, s1;
    steps_of(ph, s0, s1);
    if (b0 + rg >= P.blocks) s1 = s0;  // no rows for this warp
    const T* xp[NT];
    rows_of(un, ph, xp);
    unit_of(item + step, next);
    float acc[kW4Panels][NT][4] = {};
    float part[C::kKeep ? kW4Panels : 1][NT][4];
    for (int s = s0; s < s1; ++s) {
      w4_load_x<T, NT>(xp, 2 * s + 1, 2 * s + 1 < P.geom.tiles, xb);
      cp_async_wait<C::kDepth - 2>();
    __syncwarp();  // every lane's pieces are in; every lane is done with the slot refilled next
      produce();
      w4_tile<T, C, 0>(ring + slot, xa, n_tok_tiles, lane, part, acc);
      w4_load_x<T, NT>(xp, 2 * s + 2, s + 1 < s1, xa);
      w4_tile<T, C, 1>(ring + slot, xb, n_tok_tiles, lane, part, acc);
      slot = slot + C::kSlot == C::kDepth * C::kSlot ? 0 : slot + C::kSlot;
    }
    if (next.count > 0) {  // the next item's first activations, under this one's epilogue
      const int nph = item + step >= shared_items;
      int n0, n1;
      steps_of(nph, n0, n1);
      const T* np[NT];
      rows_of(next, nph, np);
      w4_load_x<T, NT>(np, 2 * n0, n0 < n1, xa);
    }
    __syncthreads();  // the last item's sums have been read
    w4_store_partials<C>(red, ks, rg, lane, n_tok_tiles, acc);
    __syncthreads();

    if constexpr (DOWN) {
      float* y = static_cast<float*>(P.out) + b0 * kW4Rows;
      const int rows = min(C::kRows, P.out_cols - b0 * kW4Rows);
      for (int e = tid; e < un.count * C::kRows; e += kW4Threads) {
        const int tok = e / C::kRows, row = e % C::kRows;
        if (row >= rows) continue;
        const float wt = ph ? __ldcg(&a.plan->assign_w[un.begin + tok]) : 1.f;
        const int r = ph ? __ldcg(&a.plan->assign_slot[un.begin + tok]) : un.begin + tok;
        y[(size_t)r * P.out_cols + row] = wt * w4_sum_partials<C>(red, tok, row);
      }
    } else {
      // row group r: 32 gate rows, then their 32 up rows
      T* o = static_cast<T*>(P.out) + b0 * (kW4Rows / 2);
      const int cols = min(C::kRows / 2, P.out_cols - b0 * (kW4Rows / 2));
      for (int e = tid; e < un.count * (C::kRows / 2); e += kW4Threads) {
        const int tok = e / (C::kRows / 2), col = e % (C::kRows / 2);
        if (col >= cols) continue;
        const int r = ph ? __ldcg(&a.plan->assign_slot[un.begin + tok]) : un.begin + tok;
        const int row = (col / 32) * kW4Rows + col % 32;
        const float gate = w4_sum_partials<C>(red, tok, row);
        const float up = w4_sum_partials<C>(red, tok, row + 32);
        o[(size_t)r * P.out_cols + col] = __float2bfloat16_rn(silu_f32(gate) * up);
      }
    }
  }
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
