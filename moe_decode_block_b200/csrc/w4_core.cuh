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
// What bounds it.  Up to 16 tokens: HBM for large matrices, and close behind it
// the instructions that turn codes into operands (11 per 8 codes in bf16, 9 in
// fp16; at 46 weights a clock and SM, the rate of HBM, that is two thirds of
// the ALU pipe).  So everything else is kept off the issue slots: a step of a
// warp is a pair of tiles (128 inputs) of 4 panels, addresses advance by
// constants, x is read as whole 16-byte B fragments straight from L1 / L2.
// Weights come through a warp's own ring of asynchronous 16-byte copies: no
// barrier between warps, and no wait that another thread would have to end.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_device.cuh"

namespace moe {

constexpr int kW4Tile = 64;        // inputs of a tile
constexpr int kW4TileBytes = 512;  // 16 outputs x 64 inputs
constexpr int kW4Warps = 8;        // warps of a CTA
constexpr int kW4Threads = 32 * kW4Warps;
constexpr int kW4Panels = 4;       // panels (of 16 outputs) of a warp's accumulators
constexpr int kW4Rows = 16 * kW4Panels;

// Bytes of one group entry of a panel: 16 scales, with zero points 16 of those too.
__host__ __device__ constexpr int w4_entry_bytes(bool zeros) { return zeros ? 64 : 32; }
__host__ __device__ inline size_t w4_panel_bytes(int k, int group, bool zeros) {
  return (size_t)(k / kW4Tile) * kW4TileBytes + (size_t)(k / group) * w4_entry_bytes(zeros);
}
__host__ __device__ inline size_t w4_matrix_bytes(int n, int k, int group, bool zeros) {
  return (size_t)((n + 15) / 16) * w4_panel_bytes(k, group, zeros);
}

// Compile-time shape of one instance.  NT: token tiles of 8; GROUP: inputs of a
// group; ZP: zero points; KS: warps that split K (the other 8 / KS stand side
// by side in the outputs).
template <int NT_, int GROUP, bool ZP_, int KS_>
struct W4Cfg {
  static constexpr int NT = NT_, KS = KS_;
  static constexpr bool ZP = ZP_;
  static constexpr int RW = kW4Warps / KS;              // row groups of 64 outputs
  static constexpr int kRows = RW * kW4Rows;            // outputs of a CTA
  static constexpr int kPitch = kRows + 4;              // 2 * pitch = 8 mod 32: conflict-free fragment stores
  static constexpr int kLaneEntry = ZP ? 8 : 4;         // a lane's bytes of an entry: outputs g and g + 8
  static constexpr int kEntries = 2 * kW4Tile / GROUP;  // entries of a step (a pair of tiles)
  static constexpr int kEntryBytes = 8 * kLaneEntry;    // of one entry: 16 outputs
  static constexpr int kChunks = kEntries * kEntryBytes / 16;  // 16-byte pieces of a panel's entries of a step
  // groups of 128 keep their sums over both tiles of a step before the scale;
  // with more token tiles those sums would cost too many registers
  static constexpr bool kKeep = kEntries == 1 && NT == 1;
  static constexpr int kCodes = 2 * kW4Panels * kW4TileBytes;
  static constexpr int kSlot = kCodes + kW4Panels * kEntries * kEntryBytes;  // a warp's ring slot
  static constexpr int kRed = KS * NT * 8 * kPitch * 4;
  // two CTAs on an SM up to 16 tokens where two rings of two steps fit, one
  // above (more accumulators)
  static constexpr int fit(int kb) { return (kb * 1024 - 1024 - kRed) / (kW4Warps * kSlot); }
  static constexpr int kMinCtas = NT <= 2 && fit(113) >= 2 ? 2 : 1;
  static constexpr int kFit = fit(kMinCtas == 2 ? 113 : 226);
  static constexpr int kDepth = kFit > 4 ? 4 : kFit;
  static constexpr int kSmem = kW4Warps * kDepth * kSlot + kRed;
  static_assert(kDepth >= 2, "ring depth");
};

// Geometry of a packed matrix, the same for every expert of a launch.
struct W4Geom {
  int tiles;             // K / 64
  uint32_t panel_bytes;
  uint32_t entry_off;    // of a panel's entries: tiles * 512
};

// Steps (pairs of tiles) of K; the last may hold one tile only.
__host__ __device__ inline int w4_steps(const W4Geom& g) { return (g.tiles + 1) / 2; }

// 16 bytes, or zeros where the source does not exist (valid false).
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
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
  // c += a b; FIRST: c = a b
  template <bool FIRST>
  static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    const float z0 = FIRST ? 0.f : c[0], z1 = FIRST ? 0.f : c[1], z2 = FIRST ? 0.f : c[2], z3 = FIRST ? 0.f : c[3];
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(z0), "f"(z1), "f"(z2), "f"(z3));
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
  template <bool FIRST>
  static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    const float z0 = FIRST ? 0.f : c[0], z1 = FIRST ? 0.f : c[1], z2 = FIRST ? 0.f : c[2], z3 = FIRST ? 0.f : c[3];
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(z0), "f"(z1), "f"(z2), "f"(z3));
  }
  static __device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half from_f32(float v) { return __float2half_rn(v); }
};

// The lane's place in the weight stream: its 16 bytes of the first panel's next
// tile, its 16-byte piece of the step's entries (all panels' pieces are dealt to
// the lanes in turn), and the offsets of the other panels from the first.
struct W4Stream {
  const uint8_t *code, *entry;
  uint32_t off[kW4Panels];  // off[0] = 0
  uint32_t entry2;          // from `entry` to the lane's second piece (64 pieces: groups of 32 with zero points)
  int left;                 // tiles still to be copied
  uint32_t valid;           // bit m: panel m exists (otherwise it reads as zero)
};

template <typename C>
__device__ __forceinline__ void w4_stream_start(W4Stream& st, const uint8_t* panel0, const W4Geom& g, int step0,
                                                int step1, int lane) {
  st.code = panel0 + (size_t)step0 * (2 * kW4TileBytes) + lane * 16;
  const int m = lane / C::kChunks % kW4Panels;
  uint32_t off = 0;  // (selects: no indexed access to the registers)
#pragma unroll
  for (int i = 1; i < kW4Panels; ++i) off = m == i ? st.off[i] : off;
  st.entry = panel0 + off + g.entry_off + (size_t)step0 * (C::kEntries * C::kEntryBytes) + lane % C::kChunks * 16;
  if constexpr (C::kChunks * kW4Panels > 32) st.entry2 = (m == 0 ? st.off[2] : st.off[3]) - off;
  st.left = min(g.tiles, 2 * step1) - 2 * step0;
}

// Copy the next step (a pair of tiles of 4 panels) into `slot`.  CHECK: panels
// may be missing.
template <typename C, bool CHECK>
__device__ __forceinline__ void w4_stream_step(W4Stream& st, uint32_t slot, int lane) {
  const bool second = st.left > 1;
  const uint32_t dst = slot + lane * 16;
#pragma unroll
  for (int m = 0; m < kW4Panels; ++m) {
    const bool v = !CHECK || ((st.valid >> m) & 1u);
    const uint8_t* p = st.code + st.off[m];
    cp_async_16(dst + 2 * m * kW4TileBytes, p, v);
    cp_async_16(dst + (2 * m + 1) * kW4TileBytes, second ? p + kW4TileBytes : p, v && second);
  }
  // (groups of 128 come with K in whole pairs; the other groups' entries of a
  // missing tile, the second half of a panel's pieces, are not read)
  constexpr int kPieces = C::kChunks * kW4Panels;
  const bool in = C::kEntries == 1 || second || lane % C::kChunks < C::kChunks / 2;
  const int m = lane / C::kChunks;
  if (kPieces >= 32 || lane < kPieces) {
    cp_async_16(dst + C::kCodes, in ? st.entry : st.code, in && (!CHECK || ((st.valid >> m) & 1u)));
    if constexpr (kPieces > 32)
      cp_async_16(dst + C::kCodes + 512, in ? st.entry + st.entry2 : st.code,
                   in && (!CHECK || ((st.valid >> (m + 2)) & 1u)));
  }
  st.code += 2 * kW4TileBytes;
  st.entry += C::kEntries * C::kEntryBytes;
  st.left -= 2;
}

// Tile `half` of the step in `slot` times the lane's x (2 x 16 bytes per token
// tile) into acc.  With kKeep the sums stay in `part` from the first half to the
// second.  n_tok_tiles <= NT is the same for the whole warp.
template <typename T, typename C, int HALF>
__device__ __forceinline__ void w4_tile(const uint8_t* slot, const uint4 (&xr)[C::NT][2], int n_tok_tiles, int lane,
                                        float (&part)[C::kKeep ? kW4Panels : 1][C::NT][4],
                                        float (&acc)[kW4Panels][C::NT][4]) {
  using W = W4Type<T>;
  constexpr int NT = C::NT;
  constexpr int kPer = C::kEntries == 4 ? 2 : 4;  // mma steps of a group inside this tile
#pragma unroll
  for (int m = 0; m < kW4Panels; ++m) {
    const uint4 wv = *reinterpret_cast<const uint4*>(slot + (2 * m + HALF) * kW4TileBytes + lane * 16);
    const uint32_t words[4] = {wv.x, wv.y, wv.z, wv.w};
    float(&pt)[NT][4] = part[C::kKeep ? m : 0];
#pragma unroll
    for (int e = 0; e < 4 / kPer; ++e) {
      constexpr int kHalfEntries = C::kEntries / 2;  // entries of a tile, 0 for groups of 128
      const int ei = C::kEntries == 1 ? 0 : HALF * kHalfEntries + e;
      const uint8_t* ent = slot + C::kCodes + (m * C::kEntries + ei) * C::kEntryBytes + (lane >> 2) * C::kLaneEntry;
      uint32_t sc, zg, zg8;
      if constexpr (C::ZP) {
        const uint2 sz = *reinterpret_cast<const uint2*>(ent);
        sc = sz.x;
        W::zero_consts(sz.y, zg, zg8);
      } else {
        sc = *reinterpret_cast<const uint32_t*>(ent);
        W::zero_consts(W::splat(8.f), zg, zg8);  // folds to constants
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int s = e * kPer + i;
        uint32_t a[4];
        W::dequant(words[s], zg, zg8, a);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (n == 0 || n < n_tok_tiles) {
            const uint4 xv = xr[n][s >> 1];
            const uint32_t b0 = (s & 1) ? xv.z : xv.x, b1 = (s & 1) ? xv.w : xv.y;
            if (i == 0 && (!C::kKeep || HALF == 0))
              W::template mma<true>(pt[n], a, b0, b1);
            else
              W::template mma<false>(pt[n], a, b0, b1);
          }
        }
      }
      if (!C::kKeep || HALF == 1) {
        float s0, s1;
        W::scales(sc, s0, s1);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (n == 0 || n < n_tok_tiles) {
            acc[m][n][0] = fmaf(s0, pt[n][0], acc[m][n][0]);
            acc[m][n][1] = fmaf(s0, pt[n][1], acc[m][n][1]);
            acc[m][n][2] = fmaf(s1, pt[n][2], acc[m][n][2]);
            acc[m][n][3] = fmaf(s1, pt[n][3], acc[m][n][3]);
          }
        }
      }
    }
  }
}

// The lane's x of one tile: 16 bytes at inputs 32 h + 8 t of each of its
// tokens; x reads as zero for tokens (xp[n] == nullptr) and tiles that are not.
template <typename T, int NT>
__device__ __forceinline__ void w4_load_x(const T* const (&xp)[NT], int tile, bool exists, uint4 (&xr)[NT][2]) {
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    xr[n][0] = xr[n][1] = make_uint4(0, 0, 0, 0);
    if (exists && xp[n]) {
      const T* p = xp[n] + (size_t)tile * kW4Tile;
      xr[n][0] = *reinterpret_cast<const uint4*>(p);
      xr[n][1] = *reinterpret_cast<const uint4*>(p + 32);
    }
  }
}

// Accumulators to the CTA's reduction buffer, red[K split][token][row].
template <typename C>
__device__ __forceinline__ void w4_store_partials(float* red, int ks, int rg, int lane, int n_tok_tiles,
                                                  const float (&acc)[kW4Panels][C::NT][4]) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int n = 0; n < C::NT; ++n) {
    if (n == 0 || n < n_tok_tiles) {
      float* p = red + ((size_t)ks * C::NT * 8 + n * 8 + 2 * t) * C::kPitch + rg * kW4Rows + g;
#pragma unroll
      for (int m = 0; m < kW4Panels; ++m) {
        p[m * 16] = acc[m][n][0];
        p[m * 16 + C::kPitch] = acc[m][n][1];
        p[m * 16 + 8] = acc[m][n][2];
        p[m * 16 + 8 + C::kPitch] = acc[m][n][3];
      }
    }
  }
}

// Sum of the K splits' partials of (token, row), in their order.
template <typename C>
__device__ __forceinline__ float w4_sum_partials(const float* red, int token, int row) {
  float v = 0.f;
#pragma unroll
  for (int w = 0; w < C::KS; ++w) v += red[((size_t)w * C::NT * 8 + token) * C::kPitch + row];
  return v;
}

}  // namespace moe
