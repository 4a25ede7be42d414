// w4_core.cuh -- products of a few tokens with a 4-bit weight matrix, the part
// shared by the dense layer (w4_linear.cu) and the block's experts
// (w4_experts.cuh).
//
//   y[b, n] = sum_k x[b, k] * s[n, k / G] * (q[n, k] - z[n, k / G])
//
// q in 0..15, z = 8 without zero points, G = 32, 64 or 128 inputs to a group.
//
// Mathematics.  Within a group the scale and the zero point are one number per
// output, so the group's sum of q x is taken by mma.sync with fp32 accumulators,
// the sum of x beside it, and s (sum q x - z sum x) added in fp32: no weight is
// ever rounded.  The codes go to the tensor core as they are: a 16-bit float
// with nothing but a code in its lowest bits is q times the type's smallest
// subnormal, and in bits 4..7 it is 16 q times that -- also where bit 7 is
// bf16's lowest exponent bit, since the first binade of normal numbers continues
// the subnormals' steps.  mma.sync takes subnormal operands exactly (measured).
// So an operand register costs one mask, and every second one no shift.  The
// powers of two come off in the end; bf16 activations are multiplied by 2^64 on
// their way in (exact) so that their products with 2^-133 stay normal fp32
// numbers: |x| is held from 2^-57 to 2^63, and the scaled sums, in units of 2^-69,
// to within 2^-80 an addition.  An infinite activation gives NaN
// (infinity minus infinity), as do sums beyond fp32.
//
// Layout (moe_w4_pack).  A matrix is stored as panels of 16 outputs; a panel is
// its K / 64 tiles of 512 bytes, then its group entries.  A tile is in
// mma-fragment order: lane (g, t) of a warp finds its 32 codes in one 16-byte
// word group, so a warp's load of a tile is one contiguous 512-byte access and a
// panel is one contiguous stream.  Word s of a lane holds step s of the tile:
// bits 4j / 16 + 4j are output g + 8 (j & 1), inputs
// 32 (s >> 1) + 8 t + 4 (s & 1) + 2 (j >> 1) and the next -- the order that
// turns into the four A registers of m16n8k16 by masks, while the lane's B
// registers are 16 contiguous bytes of x.
//
// What bounds it.  With one token tile HBM comes first -- 16,384 x 7,168 at one
// token in 13.2 us, 4.6 TB/s -- and not far behind it the ALU pipe: 5 of its
// instructions for 8 codes, two cycles each, are 40 of the 88 cycles that a
// scheduler has for 1,024 weights at HBM's rate (46 weights a clock and SM; in the
// experts of a full-size block of 8 tokens it is busy 54 % of the time, HBM 63 %,
// the tensor pipe 37 %, and a warp's longest wait is for its own dependent
// instructions).  With two token tiles neither is: see w4_linear_kernel.  (Subtracting the zero point from every operand, with its
// shifts, took 28 ALU and 16 more instructions for 1,024 codes instead of 20,
// and held the kernel to 40 weights a clock.)  So everything else is kept off
// the issue slots: a step of a warp is a pair of tiles (128 inputs) of 4 panels,
// addresses advance by constants, x is read as whole 16-byte B fragments
// straight from L1 / L2.  Weights come through a warp's own ring of asynchronous
// 16-byte copies: no barrier between warps, and no wait that another thread
// would have to end.
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
constexpr int kW4SumPitch = kW4Rows + 4;  // 2 * pitch = 8 mod 32: conflict-free fragment stores

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
  static_assert(NT_ == 1 || NT_ == 2, "token tiles");
  static constexpr int NT = NT_, KS = KS_;
  static constexpr bool ZP = ZP_;
  static constexpr int RW = kW4Warps / KS;              // row groups of 64 outputs
  static constexpr int kRows = RW * kW4Rows;            // outputs of a CTA
  static constexpr int kLaneEntry = ZP ? 8 : 4;         // a lane's bytes of an entry: outputs g and g + 8
  static constexpr int kEntries = 2 * kW4Tile / GROUP;  // entries of a step (a pair of tiles)
  static constexpr int kEntryBytes = 8 * kLaneEntry;    // of one entry: 16 outputs
  static constexpr int kChunks = kEntries * kEntryBytes / 16;  // 16-byte pieces of a panel's entries of a step
  static constexpr int kPieces = kChunks * kW4Panels;          // of 4 panels': up to two for each lane
  static constexpr int kCodes = 2 * kW4Panels * kW4TileBytes;
  static constexpr int kSlot = kCodes + kPieces * 16;       // a warp's ring slot: a step of 4 panels
  // A warp's sums of an item, [token][row], beside the ring.  (In the ring slot
  // just emptied they would leave room for a third step, but hold up the refill
  // until the CTA has added them: 303 against 285 us for a full-size block of 8
  // tokens.)
  static constexpr int kSums = NT * 8 * kW4SumPitch * 4;
  // two CTAs on an SM where two rings of two steps fit
  static constexpr int fit(int kb) { return (kb * 1024 - 2048 - kW4Warps * kSums) / (kW4Warps * kSlot); }
  static constexpr int kMinCtas = fit(114) >= 2 ? 2 : 1;
  static constexpr int kFit = fit(kMinCtas == 2 ? 114 : 227);
  static constexpr int kDepth = kFit > 4 ? 4 : kFit;
  static constexpr int kRing = kW4Warps * kDepth * kSlot;
  static constexpr int kSmem = kRing + kW4Warps * kSums;
  static_assert(kDepth >= 2 && kPieces <= 64, "ring");
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
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A word's codes as the A operands of one mma step: outputs g (bits 0..3 of the
// 16-bit halves) and g + 8 (bits 4..7).
__device__ __forceinline__ void w4_operands(uint32_t w, uint32_t (&a)[4]) {
  const uint32_t w8 = w >> 8;
  a[0] = w & 0x000f000fu;
  a[1] = w & 0x00f000f0u;
  a[2] = w8 & 0x000f000fu;
  a[3] = w8 & 0x00f000f0u;
}

// Per type: the mma, scales, and the powers of two.
template <typename T>
struct W4Type;

template <>
struct W4Type<__nv_bfloat16> {
  static constexpr float kUnit = 0x1p+69f;  // 2^133 (a code's unit) / 2^64 (of x)
  static __device__ __forceinline__ uint32_t scale_x(uint32_t v) {
    const uint32_t k = 0x5f805f80u;  // 2^64
    const __nv_bfloat162 r =
        __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&v), *reinterpret_cast<const __nv_bfloat162*>(&k));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  static __device__ __forceinline__ void pair_f32(uint32_t s, float& s0, float& s1) { bf16x2_to_f32(s, s0, s1); }
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
  static constexpr float kUnit = 0x1p+24f;
  static __device__ __forceinline__ uint32_t scale_x(uint32_t v) { return v; }
  static __device__ __forceinline__ void pair_f32(uint32_t s, float& s0, float& s1) {
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

// At steps [step0, step1) of K.
template <typename C>
__device__ __forceinline__ void w4_stream_start(W4Stream& st, const uint8_t* panel0, const W4Geom& g, int step0,
                                                int step1, int lane) {
  st.code = panel0 + (size_t)step0 * (2 * kW4TileBytes) + lane * 16;
  const int m = lane / C::kChunks % kW4Panels;
  uint32_t off = 0;  // (selects: no indexed access to the registers)
#pragma unroll
  for (int i = 1; i < kW4Panels; ++i) off = m == i ? st.off[i] : off;
  st.entry = panel0 + off + g.entry_off + (size_t)step0 * (C::kEntries * C::kEntryBytes) + lane % C::kChunks * 16;
  if constexpr (C::kPieces > 32) st.entry2 = (m == 0 ? st.off[2] : st.off[3]) - off;
  st.left = min(g.tiles, 2 * step1) - 2 * step0;
}

// Copy the next step (a pair of tiles of 4 panels) into `slot`.  CHECK: panels
// may be missing.
template <typename C, bool CHECK>
__device__ __forceinline__ void w4_stream_step(W4Stream& st, uint32_t slot, int lane) {
  const uint32_t dst = slot + lane * 16;
  if (!CHECK && st.left > 1) {
#pragma unroll
    for (int m = 0; m < kW4Panels; ++m) {
      const uint8_t* p = st.code + st.off[m];
      cp_async_16(dst + 2 * m * kW4TileBytes, p);
      cp_async_16(dst + (2 * m + 1) * kW4TileBytes, p + kW4TileBytes);
    }
    if (C::kPieces >= 32 || lane < C::kPieces) {
      cp_async_16(dst + C::kCodes, st.entry);
      if constexpr (C::kPieces > 32) cp_async_16(dst + C::kCodes + 512, st.entry + st.entry2);
    }
  } else {
    // a missing panel is zero (its outputs are not stored), a missing tile is
    // not copied (and not multiplied); groups of 128 come with K in whole
    // pairs, the other groups' entries of a missing tile -- the second half of
    // a panel's pieces -- do not exist
    const bool second = st.left > 1;
#pragma unroll
    for (int m = 0; m < kW4Panels; ++m) {
      const bool v = !CHECK || ((st.valid >> m) & 1u);
      const uint8_t* p = st.code + st.off[m];
      cp_async_16(dst + 2 * m * kW4TileBytes, p, v);
      if (second) cp_async_16(dst + (2 * m + 1) * kW4TileBytes, p + kW4TileBytes, v);
    }
    const bool in = C::kEntries == 1 || second || lane % C::kChunks < C::kChunks / 2;
    const int m = lane / C::kChunks;
    if (C::kPieces >= 32 || lane < C::kPieces) {
      cp_async_16(dst + C::kCodes, in ? st.entry : st.code, in && (!CHECK || ((st.valid >> m) & 1u)));
      if constexpr (C::kPieces > 32) {
        const bool v = in && (!CHECK || ((st.valid >> (m + 2)) & 1u));
        cp_async_16(dst + C::kCodes + 512, v ? st.entry + st.entry2 : st.code, v);  // (entry2 is of panels that exist)
      }
    }
  }
  st.code += 2 * kW4TileBytes;
  st.entry += C::kEntries * C::kEntryBytes;
  st.left -= 2;
}

// FIRST .. FIRST + COUNT of a step's two tiles (in `slot`) times the lane's x (2
// x 16 bytes per tile and token tile) into acc, in units of 1 / kUnit (outputs g
// + 8: 16 / kUnit).  A group's sum is scaled once; groups of 128 are cut between
// the tiles where these are taken one by one.
template <typename T, typename C, int FIRST, int COUNT>
__device__ __forceinline__ void w4_tiles(const uint8_t* slot, const uint4 (&xv)[COUNT][C::NT][2], int lane,
                                         float (&acc)[kW4Panels][C::NT][4]) {
  using W = W4Type<T>;
  constexpr int N = C::NT;
  constexpr int kGroups = C::kEntries * COUNT / 2 > 0 ? C::kEntries * COUNT / 2 : 1;
  constexpr int kPer = 4 * COUNT / kGroups;  // mma steps of a group
  // B operands, and the groups' z0 sum x: z0 = 8, or 1 where zero points come
  // with the entries
  uint32_t xr[4 * COUNT][N][2];
  float sum[kGroups][N][2];
  const uint32_t one = C::ZP ? 0x00010001u : 0x00080008u, ones[4] = {one, one, one, one};
#pragma unroll
  for (int n = 0; n < N; ++n) {
#pragma unroll
    for (int s = 0; s < 4 * COUNT; ++s) {
      const uint4 v = xv[s / 4][n][(s >> 1) & 1];
      xr[s][n][0] = W::scale_x((s & 1) ? v.z : v.x);
      xr[s][n][1] = W::scale_x((s & 1) ? v.w : v.y);
    }
#pragma unroll
    for (int e = 0; e < kGroups; ++e) {
      float c[4];
      W::template mma<true>(c, ones, xr[e * kPer][n][0], xr[e * kPer][n][1]);
#pragma unroll
      for (int i = 1; i < kPer; ++i) W::template mma<false>(c, ones, xr[e * kPer + i][n][0], xr[e * kPer + i][n][1]);
      sum[e][n][0] = c[0];
      sum[e][n][1] = c[1];
    }
  }
#pragma unroll
  for (int m = 0; m < kW4Panels; ++m) {
    uint32_t words[4 * COUNT];
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
      const uint4 wv = *reinterpret_cast<const uint4*>(slot + (2 * m + FIRST + i) * kW4TileBytes + lane * 16);
      words[4 * i] = wv.x;
      words[4 * i + 1] = wv.y;
      words[4 * i + 2] = wv.z;
      words[4 * i + 3] = wv.w;
    }
#pragma unroll
    for (int e = 0; e < kGroups; ++e) {
      const uint8_t* entry = slot + C::kCodes + (lane >> 2) * C::kLaneEntry +
                             (m * C::kEntries + (C::kEntries == 1 ? 0 : FIRST * C::kEntries / 2 + e)) * C::kEntryBytes;
      float s0, s1, z0 = 1.f, z1 = 16.f;  // of outputs g and g + 8
      if constexpr (C::ZP) {
        const uint2 sz = *reinterpret_cast<const uint2*>(entry);
        W::pair_f32(sz.x, s0, s1);
        W::pair_f32(sz.y, z0, z1);
        z1 *= 16.f;
      } else {
        W::pair_f32(*reinterpret_cast<const uint32_t*>(entry), s0, s1);
      }
      float part[N][4];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int s = e * kPer + i;
        uint32_t a[4];
        w4_operands(words[s], a);
#pragma unroll
        for (int n = 0; n < N; ++n) {
          if (i == 0)
            W::template mma<true>(part[n], a, xr[s][n][0], xr[s][n][1]);
          else
            W::template mma<false>(part[n], a, xr[s][n][0], xr[s][n][1]);
        }
      }
#pragma unroll
      for (int n = 0; n < N; ++n) {
        acc[m][n][0] = fmaf(s0, fmaf(-z0, sum[e][n][0], part[n][0]), acc[m][n][0]);
        acc[m][n][1] = fmaf(s0, fmaf(-z0, sum[e][n][1], part[n][1]), acc[m][n][1]);
        acc[m][n][2] = fmaf(s1, fmaf(-z1, sum[e][n][0], part[n][2]), acc[m][n][2]);
        acc[m][n][3] = fmaf(s1, fmaf(-z1, sum[e][n][1], part[n][3]), acc[m][n][3]);
      }
    }
  }
}

// The lane's x of tile `half` of a step: 16 bytes at inputs 32 h + 8 t of each
// of its tokens; xp[n] is at the step's first input.  (A token that does not
// exist has the address of one that does: its column of the products is never
// stored, and no column sees another.)
template <typename T, int NT>
__device__ __forceinline__ void w4_load_x(const T* const (&xp)[NT], int half, uint4 (&xr)[NT][2]) {
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    xr[n][0] = *reinterpret_cast<const uint4*>(xp[n] + half * kW4Tile);
    xr[n][1] = *reinterpret_cast<const uint4*>(xp[n] + half * kW4Tile + 32);
  }
}

// A warp's share [s0, s1) of the steps of K for one item.  x of its first tile
// is in x.v[0] (loaded before, when there is a step).  `advance` returns once the
// next step is in its ring slot and refills the slot before; `slot` follows the
// ring.  One token tile takes both tiles of a step together and has x of the
// next step on its way meanwhile; more token tiles have registers for one tile
// ahead only.
template <typename T, typename C>
struct W4X {
  uint4 v[C::NT == 1 ? 4 : 2][1][C::NT][2];  // NT == 1: two steps of two tiles; else two tiles
};
template <typename T, typename C>
__device__ __forceinline__ void w4_first_x(const T* const (&xp)[C::NT], bool second, W4X<T, C>& x) {
  w4_load_x<T>(xp, 0, x.v[0][0]);
  if constexpr (C::NT == 1)
    if (second) w4_load_x<T>(xp, 1, x.v[1][0]);
}
template <typename T, typename C, typename Advance>
__device__ __forceinline__ void w4_run(int s0, int s1, int tiles, const uint8_t* ring, uint32_t& slot,
                                       const T* (&xp)[C::NT], W4X<T, C>& x, int lane,
                                       float (&acc)[kW4Panels][C::NT][4], Advance& advance) {
  auto consumed = [&]() { slot = slot + C::kSlot == C::kDepth * C::kSlot ? 0 : slot + C::kSlot; };
  auto next_x = [&]() {
#pragma unroll
    for (int n = 0; n < C::NT; ++n) xp[n] += 2 * kW4Tile;
  };
  if constexpr (C::NT == 1) {
    auto one = [&](int s, uint4 (&c0)[1][1][2], uint4 (&c1)[1][1][2], uint4 (&n0)[1][1][2], uint4 (&n1)[1][1][2]) {
      next_x();
      if (s + 1 < s1) {
        w4_load_x<T>(xp, 0, n0[0]);
        if (2 * s + 3 < tiles) w4_load_x<T>(xp, 1, n1[0]);
      }
      advance();
      if (2 * s + 1 < tiles) {
        const uint4 c[2][1][2] = {{{c0[0][0][0], c0[0][0][1]}}, {{c1[0][0][0], c1[0][0][1]}}};
        w4_tiles<T, C, 0, 2>(ring + slot, c, lane, acc);
      } else {
        w4_tiles<T, C, 0, 1>(ring + slot, c0, lane, acc);
      }
      consumed();
    };
    for (int s = s0; s < s1; s += 2) {
      one(s, x.v[0], x.v[1], x.v[2], x.v[3]);
      if (s + 1 >= s1) break;
      one(s + 1, x.v[2], x.v[3], x.v[0], x.v[1]);
    }
  } else {
    for (int s = s0; s < s1; ++s) {
      const bool second = 2 * s + 1 < tiles;
      if (second) w4_load_x<T>(xp, 1, x.v[1][0]);
      advance();
      w4_tiles<T, C, 0, 1>(ring + slot, x.v[0], lane, acc);
      next_x();
      if (s + 1 < s1) w4_load_x<T>(xp, 0, x.v[0][0]);
      if (second) w4_tiles<T, C, 1, 1>(ring + slot, x.v[1], lane, acc);
      consumed();
    }
  }
}

// Accumulators, brought back to units of 1, to the warp's sums [token][row].
template <typename T, typename C>
__device__ __forceinline__ void w4_store_sums(float* sums, int lane,
                                              const float (&acc)[kW4Panels][C::NT][4]) {
  const int g = lane >> 2, t = lane & 3;
  constexpr float u0 = W4Type<T>::kUnit, u1 = W4Type<T>::kUnit / 16.f;
#pragma unroll
  for (int n = 0; n < C::NT; ++n) {
    float* p = sums + (n * 8 + 2 * t) * kW4SumPitch + g;
#pragma unroll
    for (int m = 0; m < kW4Panels; ++m) {
      p[m * 16] = u0 * acc[m][n][0];
      p[m * 16 + kW4SumPitch] = u0 * acc[m][n][1];
      p[m * 16 + 8] = u1 * acc[m][n][2];
      p[m * 16 + 8 + kW4SumPitch] = u1 * acc[m][n][3];
    }
  }
}

// Sum over the K splits, in their order, of element `at` of their warps' sums.
template <typename C>
__device__ __forceinline__ float w4_add_splits(const float* const (&sums)[C::KS], int at) {
  float v = 0.f;
#pragma unroll
  for (int w = 0; w < C::KS; ++w) v += sums[w][at];
  return v;
}

}  // namespace moe
