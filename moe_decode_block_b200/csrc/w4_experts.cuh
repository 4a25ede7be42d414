// w4_experts.cuh -- the block's experts on 4-bit weights: up projection and
// SwiGLU, down projection, and the weighted combine with the residual
// (moe_decode_forward_w4).  The router and its plan are the block's own.
//
//   a[slot, c] = bf16(silu(x_t . W13[:, c]) * (x_t . W13[:, I + c]))
//   y[slot, n] = w_slot * sum_c a[slot, c] W2[c, n]
//   out[t, n]  = bf16(x[t, n] + y[t k + 0, n] + ... + y[t k + k - 1, n] + y_shared[t, n])
//
// Two persistent kernels of one template: a CTA takes items (64 weight rows of
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
  int blocks;              // items of a unit: its weight rows / 64 (UP: pairs of 32 gate and 32 up rows)
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

template <int NT, bool HALF, bool ZP, bool DOWN>
__global__ void __launch_bounds__(kW4Threads, W4Cfg<NT, HALF, ZP>::kMinCtas)
    w4_expert_kernel(const __grid_constant__ W4ExpertArgs a, const __grid_constant__ ExpertTable tab) {
  using C = W4Cfg<NT, HALF, ZP>;
  using T = __nv_bfloat16;
  extern __shared__ __align__(1024) uint8_t w4_smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint8_t* ring = w4_smem + (size_t)warp * C::kDepth * C::kSlot;
  const uint32_t ring_addr = smem_addr(ring);
  float* red = reinterpret_cast<float*>(w4_smem + (size_t)kW4Warps * C::kDepth * C::kSlot);

  const int shared_items = a.n_su * a.ph[0].blocks;
  const int step = gridDim.x;
  int n_items = shared_items;  // all items, once the plan has been read
  bool have_plan = false;
  auto read_plan = [&]() {
    if (have_plan) return;
    cudaGridDependencySynchronize();
    n_items = shared_items + __ldcg(&a.plan->n_active) * a.ph[1].blocks;
    have_plan = true;
  };
  // the next grid may be put in place as this one's CTAs leave; it waits for
  // this grid's completion before it reads anything of it
  cudaTriggerProgrammaticLaunchCompletion();
  if constexpr (DOWN) {
    // the activations come from the grid before; weights may stream already
  }

  auto tiles_of = [&](int ph, int& t0, int& t1) {
    const int n = a.ph[ph].geom.tiles;
    t0 = n * warp / kW4Warps;
    t1 = n * (warp + 1) / kW4Warps;
  };

  // ---- the weight stream: runs up to kDepth - 1 tiles ahead of the products
  int p_item = blockIdx.x, p_tile = 0, p_end = 0, p_slot = 0, p_ph = 0;
  const uint8_t* panel[kW4Panels];
  auto p_locate = [&]() {  // panels and tile range of item p_item; false: no more
    for (;;) {
      if (p_item >= shared_items) read_plan();
      if (p_item >= n_items) return false;
      p_ph = p_item >= shared_items;
      tiles_of(p_ph, p_tile, p_end);
      if (p_tile < p_end) break;
      p_item += step;  // this warp has no tile of such items
    }
    const W4Phase& ph = a.ph[p_ph];
    const int i = p_item - (p_ph ? shared_items : 0);
    const int u = i / ph.blocks, b = i - u * ph.blocks;
    const uint8_t* w =
        p_ph ? reinterpret_cast<const uint8_t*>(tab.p[__ldcg(&a.plan->unit_expert[u])]) : a.shared_w;
#pragma unroll
    for (int m = 0; m < kW4Panels; ++m) {
      if constexpr (DOWN)
        panel[m] = w + (size_t)(b * kW4Panels + m) * ph.geom.panel_bytes;
      else
        panel[m] = w + (size_t)(b * 2 + (m & 1)) * ph.geom.panel_bytes + (m >> 1) * (size_t)ph.up_off;
    }
    return true;
  };
  bool p_more = p_locate();
  auto produce = [&]() {
    if (p_more) {
      w4_issue<C>(ring_addr + p_slot * C::kSlot, panel, 0xfu, a.ph[p_ph].geom, p_tile, lane);
      if (++p_tile == p_end) {
        p_item += step;
        p_more = p_locate();
      }
    }
    cp_async_commit();
    p_slot = p_slot + 1 == C::kDepth ? 0 : p_slot + 1;
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
    const int u = i / a.ph[ph].blocks;
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
  uint4 xr[NT][2], xn[NT][2];
  int slot = 0;
  {
    const int ph = (int)blockIdx.x >= shared_items;
    int t0, t1;
    tiles_of(ph, t0, t1);
    const T* xp[NT];
    rows_of(next, ph, xp);
    if (t0 < t1) w4_load_x<T, NT>(xp, t0, xn);
  }
  for (int item = blockIdx.x;; item += step) {
    if (item >= shared_items) read_plan();
    if (item >= n_items) break;
    const int ph = item >= shared_items;
    const W4Unit<NT> un = next;
    const int n_tok_tiles = (un.count + 7) >> 3;
    int t0, t1;
    tiles_of(ph, t0, t1);
    const T* xp[NT];
    rows_of(un, ph, xp);
    unit_of(item + step, next);
    float acc[kW4Panels][NT][4] = {};
    for (int t = t0; t < t1; ++t) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        xr[n][0] = xn[n][0];
        xr[n][1] = xn[n][1];
      }
      if (t + 1 < t1) w4_load_x<T, NT>(xp, t + 1, xn);
      cp_async_wait<C::kDepth - 2>();
      produce();
      w4_tile<T, NT, HALF, ZP>(ring + slot * C::kSlot, xr, n_tok_tiles, lane, acc);
      slot = slot + 1 == C::kDepth ? 0 : slot + 1;
    }
    if (next.count > 0) {  // the next item's first activations, under this one's epilogue
      const int nph = item + step >= shared_items;
      int n0, n1;
      tiles_of(nph, n0, n1);
      const T* np[NT];
      rows_of(next, nph, np);
      if (n0 < n1) w4_load_x<T, NT>(np, n0, xn);
    }
    __syncthreads();  // the last item's sums have been read
    w4_store_partials<NT>(red, warp, lane, n_tok_tiles, acc);
    __syncthreads();

    const int i = item - (ph ? shared_items : 0);
    const int b = i % a.ph[ph].blocks;
    const int cols = a.ph[ph].out_cols;
    if constexpr (DOWN) {
      float* y = static_cast<float*>(a.ph[ph].out) + b * kW4Rows;
      for (int e = tid; e < un.count * kW4Rows; e += kW4Threads) {
        const int tok = e / kW4Rows, row = e % kW4Rows;
        const float wt = ph ? __ldcg(&a.plan->assign_w[un.begin + tok]) : 1.f;
        const int r = ph ? __ldcg(&a.plan->assign_slot[un.begin + tok]) : un.begin + tok;
        y[(size_t)r * cols + row] = wt * w4_sum_partials<NT>(red, tok, row);
      }
    } else {
      T* o = static_cast<T*>(a.ph[ph].out) + b * (kW4Rows / 2);
      for (int e = tid; e < un.count * (kW4Rows / 2); e += kW4Threads) {
        const int tok = e / (kW4Rows / 2), row = e % (kW4Rows / 2);
        const int r = ph ? __ldcg(&a.plan->assign_slot[un.begin + tok]) : un.begin + tok;
        const float gate = w4_sum_partials<NT>(red, tok, row);
        const float up = w4_sum_partials<NT>(red, tok, row + kW4Rows / 2);
        o[(size_t)r * cols + row] = __float2bfloat16_rn(silu_f32(gate) * up);
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
