// w4_core.cuh -- products of a few tokens with a 4-bit weight matrix, the part
// shared by the dense layer (w4_linear.cu) and the block's experts
// (w4_experts.cuh).
//
//   y[b, n] = sum_k x[b, k] * s[n, k / G] * (q[n, k] - z[n, k / G])
//
// q in 0..15, z = 8 without zero points, G = 32, 64 or 128 inputs to a group.
//
// Mathematics.  Within a 64-input tile (32 inputs for G = 32) the scale is one
// number per output, so the tile's sum over (q - z) * x is taken by mma.sync
// with fp32 accumulators -- q - z is a small whole number, exact in bf16 and
// fp16, and so is its product's operand x -- and the fp32 result is multiplied
// by the scale once: no weight is ever rounded.
//
// Layout (moe_w4_pack).  A matrix is stored as panels of 16 outputs; a panel is
// its K / 64 tiles of 512 bytes, then its group entries.  A tile is in
// mma-fragment order: lane (g, t) of a warp finds its 32 codes in one 16-byte
// word group, so a warp's load of a tile is one contiguous 512-byte access and a
// panel is one contiguous stream.  Word s of a lane holds step s of the tile:
// bits 4j / 16 + 4j are output g + 8 (j & 1), inputs
// 32 (s >> 1) + 8 t + 4 (s & 1) + 2 (j >> 1) and the next -- the order that
// turns into the four A registers of m16n8k16 with one mask and one exact
// subtraction each, while the lane's B registers are 16 contiguous bytes of x.
//
// What bounds it.  Up to 16 tokens: HBM for large matrices, then the ALU work of
// turning codes into operands (about 11 instructions per 8 codes in bf16, 9 in
// fp16).  Weights come through a ring of asynchronous 16-byte copies; every lane
// copies exactly the bytes it will read, so the ring needs no barrier between
// threads, only the lane's own wait.  A CTA's warps split the inputs (K), so
// x is read once per CTA and each warp's accumulators cover 4 panels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_device.cuh"

namespace moe {

constexpr int kW4Tile = 64;        // inputs of a tile
constexpr int kW4TileBytes = 512;  // 16 outputs x 64 inputs
constexpr int kW4Warps = 8;        // warps of a CTA: they split the tiles of K
constexpr int kW4Threads = 32 * kW4Warps;
constexpr int kW4Panels = 4;       // panels (of 16 outputs) of a warp's accumulators
constexpr int kW4Rows = 16 * kW4Panels;
constexpr int kW4RedPitch = kW4Rows + 4;  // floats; 2 * pitch = 8 mod 32: conflict-free fragment stores

// Bytes of one group entry of a panel: 16 scales, with zero points 16 of those too.
__host__ __device__ constexpr int w4_entry_bytes(bool zeros) { return zeros ? 64 : 32; }
__host__ __device__ inline size_t w4_panel_bytes(int k, int group, bool zeros) {
  return (size_t)(k / kW4Tile) * kW4TileBytes + (size_t)(k / group) * w4_entry_bytes(zeros);
}
__host__ __device__ inline size_t w4_matrix_bytes(int n, int k, int group, bool zeros) {
  return (size_t)((n + 15) / 16) * w4_panel_bytes(k, group, zeros);
}

// Compile-time shape of one instance.  NT: token tiles of 8; HALF: groups of
// 32 inputs (two to a tile); ZP: zero points.
template <int NT, bool HALF, bool ZP>
struct W4Cfg {
  static constexpr int kLaneEntry = ZP ? 8 : 4;               // a lane's bytes of an entry: outputs g and g + 8
  static constexpr int kEntries = HALF ? 2 : 1;               // entries of a tile
  static constexpr int kSlot = kW4Panels * (kW4TileBytes + kEntries * 32 * kLaneEntry);  // a warp's ring slot
  static constexpr int kRed = kW4Warps * NT * 8 * kW4RedPitch * 4;
  // two CTAs on an SM up to 16 tokens, one above (more accumulators)
  static constexpr int kMinCtas = NT <= 2 ? 2 : 1;
  static constexpr int kBudget = (kMinCtas == 2 ? 113 : 226) * 1024 - 1024;
  static constexpr int kFit = (kBudget - kRed) / (kW4Warps * kSlot);
  static constexpr int kDepth = kFit > 6 ? 6 : kFit;
  static constexpr int kSmem = kW4Warps * kDepth * kSlot + kRed;
  static_assert(kDepth >= 2, "ring depth");
};

// Geometry of a packed matrix, the same for every expert of a launch.
struct W4Geom {
  int tiles;             // K / 64
  uint32_t panel_bytes;
  uint32_t entry_off;    // of a panel's entries: tiles * 512
  int group_shift;       // log2(G / 64) for G >= 64: tile >> shift is the group
};

template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? BYTES : 0;  // the rest of the slot's bytes are zero-filled
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t mask, uint32_t bits) {
  uint32_t r;  // (a & mask) | bits in one instruction
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(a), "r"(mask), "r"(bits));
  return r;
}

// Per type: codes to A operands, the zero-point constants, scales, the mma.
template <typename T>
struct W4Type;

template <>
struct W4Type<__nv_bfloat16> {
  // 0x4300 | v is 128 + v; subtracting 128 + z is exact.
  static __device__ __forceinline__ uint32_t splat(float v) {
    const __nv_bfloat162 h = __float2bfloat162_rn(v);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r =
        __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  static __device__ __forceinline__ uint32_t add(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r =
        __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  // what is subtracted from the words of outputs g and g + 8
  static __device__ __forceinline__ void zero_consts(uint32_t zp, uint32_t& zg, uint32_t& zg8) {
    const uint32_t base = splat(128.f);
    zg = add(base, __byte_perm(zp, zp, 0x1010));
    zg8 = add(base, __byte_perm(zp, zp, 0x3232));
  }
  static __device__ __forceinline__ void dequant(uint32_t w, uint32_t zg, uint32_t zg8, uint32_t (&a)[4]) {
    a[0] = sub(and_or(w, 0x000f000fu, 0x43004300u), zg);
    a[1] = sub(and_or(w >> 4, 0x000f000fu, 0x43004300u), zg8);
    a[2] = sub(and_or(w >> 8, 0x000f000fu, 0x43004300u), zg);
    a[3] = sub(and_or(w >> 12, 0x000f000fu, 0x43004300u), zg8);
  }
  static __device__ __forceinline__ void scales(uint32_t s, float& s0, float& s1) { bf16x2_to_f32(s, s0, s1); }
  static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
  static __device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }
};

template <>
struct W4Type<__half> {
  static __device__ __forceinline__ uint32_t splat(float v) {
    const __half2 h = __float2half2_rn(v);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b) {
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  static __device__ __forceinline__ uint32_t fma(uint32_t a, uint32_t b, uint32_t c) {
    const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b),
                              *reinterpret_cast<const __half2*>(&c));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  // 0x6400 | v is 1024 + v and 0x6400 | 16 v is 1024 + 16 v: outputs g take
  // (1024 + v) - (1024 + z), outputs g + 8 (1024 + 16 v) / 16 - (64 + z), both
  // exact and the second without a shift.
  static __device__ __forceinline__ void zero_consts(uint32_t zp, uint32_t& zg, uint32_t& zg8) {
    zg = sub(__byte_perm(zp, zp, 0x1010), splat(-1024.f));
    zg8 = sub(splat(-64.f), __byte_perm(zp, zp, 0x3232));
  }
  static __device__ __forceinline__ void dequant(uint32_t w, uint32_t zg, uint32_t zg8, uint32_t (&a)[4]) {
    const uint32_t w8 = w >> 8, sixteenth = 0x2c002c00u;
    a[0] = sub(and_or(w, 0x000f000fu, 0x64006400u), zg);
    a[1] = fma(and_or(w, 0x00f000f0u, 0x64006400u), sixteenth, zg8);
    a[2] = sub(and_or(w8, 0x000f000fu, 0x64006400u), zg);
    a[3] = fma(and_or(w8, 0x00f000f0u, 0x64006400u), sixteenth, zg8);
  }
  static __device__ __forceinline__ void scales(uint32_t s, float& s0, float& s1) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&s));
    s0 = f.x;
    s1 = f.y;
  }
  static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
  static __device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half from_f32(float v) { return __float2half_rn(v); }
};

// The warp's ring: copies of one tile of its 4 panels.  `panel[m]` are the
// panels' addresses; a panel that does not exist (valid[m] false) is zero.
template <typename C>
__device__ __forceinline__ void w4_issue(uint32_t slot, const uint8_t* const (&panel)[kW4Panels], uint32_t valid,
                                         const W4Geom& g, int tile, int lane) {
#pragma unroll
  for (int m = 0; m < kW4Panels; ++m)
    cp_async<16>(slot + m * kW4TileBytes + lane * 16, panel[m] + (size_t)tile * kW4TileBytes + lane * 16,
                 (valid >> m) & 1u);
  const int e0 = C::kEntries == 2 ? 2 * tile : tile >> g.group_shift;
  const uint32_t dst = slot + kW4Panels * kW4TileBytes + lane * C::kLaneEntry;
#pragma unroll
  for (int m = 0; m < kW4Panels; ++m)
#pragma unroll
    for (int e = 0; e < C::kEntries; ++e)
      cp_async<C::kLaneEntry>(
          dst + (m * C::kEntries + e) * 32 * C::kLaneEntry,
          panel[m] + g.entry_off + (size_t)(e0 + e) * (8 * C::kLaneEntry) + (lane >> 2) * C::kLaneEntry,
          (valid >> m) & 1u);
}

// One tile of the warp's 4 panels times the lane's x (2 x 16 bytes per token
// tile) into acc.  n_tok_tiles <= NT is the same for the whole warp.
template <typename T, int NT, bool HALF, bool ZP>
__device__ __forceinline__ void w4_tile(const uint8_t* slot, const uint4 (&xr)[NT][2], int n_tok_tiles, int lane,
                                        float (&acc)[kW4Panels][NT][4]) {
  using C = W4Cfg<NT, HALF, ZP>;
  using W = W4Type<T>;
#pragma unroll
  for (int m = 0; m < kW4Panels; ++m) {
    const uint4 wv = *reinterpret_cast<const uint4*>(slot + m * kW4TileBytes + lane * 16);
    const uint32_t words[4] = {wv.x, wv.y, wv.z, wv.w};
    const uint8_t* ent = slot + kW4Panels * kW4TileBytes + m * C::kEntries * 32 * C::kLaneEntry + lane * C::kLaneEntry;
    float part[NT][4];
#pragma unroll
    for (int e = 0; e < C::kEntries; ++e) {
      uint32_t sc, zg, zg8;
      if constexpr (ZP) {
        const uint2 sz = *reinterpret_cast<const uint2*>(ent + e * 32 * C::kLaneEntry);
        sc = sz.x;
        W::zero_consts(sz.y, zg, zg8);
      } else {
        sc = *reinterpret_cast<const uint32_t*>(ent + e * 32 * C::kLaneEntry);
        W::zero_consts(W::splat(8.f), zg, zg8);  // folds to constants
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) part[n][0] = part[n][1] = part[n][2] = part[n][3] = 0.f;
#pragma unroll
      for (int i = 0; i < 4 / C::kEntries; ++i) {
        const int s = e * (4 / C::kEntries) + i;
        uint32_t a[4];
        W::dequant(words[s], zg, zg8, a);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (n == 0 || n < n_tok_tiles) {
            const uint4 xv = xr[n][s >> 1];
            W::mma(part[n], a, (s & 1) ? xv.z : xv.x, (s & 1) ? xv.w : xv.y);
          }
        }
      }
      float s0, s1;
      W::scales(sc, s0, s1);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (n == 0 || n < n_tok_tiles) {
          acc[m][n][0] = fmaf(s0, part[n][0], acc[m][n][0]);
          acc[m][n][1] = fmaf(s0, part[n][1], acc[m][n][1]);
          acc[m][n][2] = fmaf(s1, part[n][2], acc[m][n][2]);
          acc[m][n][3] = fmaf(s1, part[n][3], acc[m][n][3]);
        }
      }
    }
  }
}

// The lane's x of one tile: 16 bytes at inputs 32 h + 8 t of each of its
// tokens; xp[n] == nullptr (no such token) reads as zero.
template <typename T, int NT>
__device__ __forceinline__ void w4_load_x(const T* const (&xp)[NT], int tile, uint4 (&xr)[NT][2]) {
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    xr[n][0] = xr[n][1] = make_uint4(0, 0, 0, 0);
    if (xp[n]) {
      const T* p = xp[n] + (size_t)tile * kW4Tile;
      xr[n][0] = *reinterpret_cast<const uint4*>(p);
      xr[n][1] = *reinterpret_cast<const uint4*>(p + 32);
    }
  }
}

// Accumulators to the CTA's reduction buffer, red[warp][token][row].
template <int NT>
__device__ __forceinline__ void w4_store_partials(float* red, int warp, int lane, int n_tok_tiles,
                                                  const float (&acc)[kW4Panels][NT][4]) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    if (n == 0 || n < n_tok_tiles) {
      float* p = red + ((size_t)warp * NT * 8 + n * 8 + 2 * t) * kW4RedPitch + g;
#pragma unroll
      for (int m = 0; m < kW4Panels; ++m) {
        p[m * 16] = acc[m][n][0];
        p[m * 16 + kW4RedPitch] = acc[m][n][1];
        p[m * 16 + 8] = acc[m][n][2];
        p[m * 16 + 8 + kW4RedPitch] = acc[m][n][3];
      }
    }
  }
}

// Sum of the warps' partials of (token, row), in warp order.
template <int NT>
__device__ __forceinline__ float w4_sum_partials(const float* red, int token, int row) {
  float v = 0.f;
#pragma unroll
  for (int w = 0; w < kW4Warps; ++w) v += red[((size_t)w * NT * 8 + token) * kW4RedPitch + row];
  return v;
}

}  // namespace moe
