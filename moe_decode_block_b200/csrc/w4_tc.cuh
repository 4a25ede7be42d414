// w4_tc.cuh -- products of many tokens (up to 64) with a 4-bit weight matrix on
// the 5th-generation tensor cores: the dense layer above 16 tokens, the block's
// experts above 8.
//
// mma.sync takes a token tile of 8 per instruction and does 1,024 products a
// clock and SM whatever it is given (measured: 976), so at 64 tokens it stops at
// 16 weights a clock and SM where HBM delivers 46.  tcgen05.mma takes all tokens
// at once: 128 weight rows x up to 64 tokens x 16 inputs in 45 to 52 clocks
// (measured, the same for 16, 32 and 64 tokens; the weights in tensor memory), 40
// to 45 weights a clock.  The dense layer changes over above 16 tokens, the block's
// experts above 8; both sides are measured at w4_linear_tc_kernel and in
// w4_experts.cuh.
//
// Mathematics.  Here a weight s (q - z) is rounded once to the activations' type
// (half a step: up to 2^-8 of it in bf16, 2^-11 in fp16; it has to fit the type)
// and the products are summed in fp32 over all of K in tensor memory.  The
// exact form of w4_core.cuh -- a group's sum read back and scaled in fp32 -- was
// built too: reading 64 sums a row back every 128 inputs, beside the MMAs' own
// traffic to tensor memory, took 1,700 clocks a step where the MMAs take 860, 52
// us for a layer of 16,384 x 7,168 at 64 tokens where the rounded form then took
// 38.  The rounding adds 6e-4 to the 1.7e-3 that rounding the result to bf16 costs.
//
// A code becomes an operand by a mask and, in bf16 (where it is a subnormal, as in
// w4_core.cuh) without zero points, one fused multiply-add, q (s 2^100) - 8 s 2^-33,
// whose one rounding is the weight's (times 2^-33, taken off in the end; s below
// 2^27).  Zero points and fp16 take two instructions: q - z, exact, then the product
// with the scale.  In bf16 that is (q - z) times a power of two, which the scale
// takes off (s below 2^122); in fp16 the code stands in the lowest bits of 1024 and
// the scale is as it came, so any that the weights allow will do.  (From subnormal
// codes fp16 needed s 2^9, which ended at 128.  To hold larger scales in bf16 too,
// by the two instructions or by a vote of the warp on a step's scales, cost the
// layer above 1.2 to 2 us of 27, for scales that no model has.)
//
// Layout of the work.  A CTA has 256 weight rows (two accumulators of 128) and up
// to 64 tokens, and takes K in steps of 128 inputs.  Its 16 warps:
//   8 unpackers   each streams two panels through its own ring of asynchronous
//                 copies and stores their operands to tensor memory with the
//                 16x256b shape, whose fragment order is the packed layout's;
//   4 finishers   read an item's sums out of tensor memory (a thread is a row of
//                 both accumulators) while the next item is multiplied;
//   1 MMA warp    one thread issues a step's tcgen05.mma and commits;
//   3 stagers     each every third step: the tokens' activations to shared memory
//                 as the B operand (K-major cores of 8 tokens x 8 inputs; 8-byte
//                 pieces move so that the inputs' order is the A operand's).
// The dense layer's CTA has one item: its finishers stage too (six warps), and in
// the end all 16 warps read the sums.  Tensor memory: two sets of sums (128
// columns each) and two buffers of operands.  (One set and three buffers: 211
// against 200 us for a block of 16 experts at 64 tokens.)
//
// What bounds it.  A step takes 1,130 clocks (0.6 us) at 17 to 64 tokens, of which
// its 16 MMAs, each reading 128 rows of operands from tensor memory, are 720 to
// 830; HBM gives 3.5 TB/s meanwhile.  Before, the load and store pipe was in the
// way: a load of 16 bytes from each of 8 tokens x 4 touches 8 lines where 4 tokens
// x 8 touch 4 (35 against 37 us for the layer above, 178 against 200 for the
// block), and asynchronous 8-byte copies, straight to their places, twice as many
// (48 us).  Around its 28 steps the layer above spends 9 us at 64 tokens: the
// launch, first loads from HBM, and the exchange of the halves of K.
//
// Every wait is bounded: a wait that runs out sets the status word and the CTA's
// abort flag, and the CTA leaves after its own copies and MMAs in flight have
// ended.
#pragma once

#include <type_traits>

#include "moe_device.cuh"
#include "tcgen05.cuh"
#include "w4_core.cuh"

namespace moe {

constexpr int kTcUnpackers = 8, kTcFinishers = 4, kTcStagers = 3;
constexpr int kTcMmaWarp = kTcUnpackers + kTcFinishers;
constexpr int kW4TcThreads = 32 * (kTcMmaWarp + 1 + kTcStagers);
constexpr int kTcRows = 256;     // weight rows of a CTA
constexpr int kTcTokens = 64;
constexpr int kTcStep = 128;     // inputs of a step
constexpr int kTcRingTiles = 8;  // of an unpacker's ring: 2 panels x 512 bytes each
constexpr int kTcRingBytes = kTcRingTiles * 2 * kW4TileBytes;
constexpr int kTcSlots = 6;                           // of the B operands
// Bytes between cores along K: 128, and a gap that puts the two cores which half a
// warp writes (4 tokens x 4 pieces) on different banks.
constexpr int kTcCore = 192;
constexpr int kTcBGroup = kTcStep / 8 * kTcCore;      // of 8 tokens
constexpr int kTcBSlot = kTcTokens / 8 * kTcBGroup;   // bytes
constexpr int kTcB = kTcUnpackers * kTcRingBytes;   // offset of the B operands
constexpr int kTcSmem = kTcB + kTcSlots * kTcBSlot;
constexpr uint32_t kTcOperandCol = 256;             // first tensor-memory column of the A operands
constexpr uint32_t kTcBufs = 2;                     // operand buffers

struct W4TcBars {
  uint64_t a_full[kTcBufs], a_empty[kTcBufs], d_full[2], d_empty[2], b_full[kTcSlots], b_empty[kTcSlots], drained;
  uint32_t tmem;
  int ctl[2];  // abort flag, wait limit
};

// What one CTA multiplies: 16 panels, tiles [tile0, tile1) of K (tile0 even), n_tok tokens.
struct W4TcItem {
  const uint8_t* panel[2];  // first panel of each 128 rows
  int n_panels[2];          // panels that exist of each 8
  int tile0, tile1, n_tok;
  __device__ __forceinline__ int steps() const { return (tile1 - tile0 + 1) / 2; }
};

// 1 in one lane of the warp
__device__ __forceinline__ uint32_t tc5_elect() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}
// D[tmem] (+)= A[tmem] x B[smem]: kind::f16, one CTA; by the lane whose `lead` is
// set, with the whole warp in step, so that the operands stay in uniform registers
__device__ __forceinline__ void tc5_mma(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate,
                                        uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void tc5_commit(uint64_t* bar, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_addr(bar)),
      "r"(lead)
      : "memory");
}
// Four fragments of 8 columns each (output g: columns 2 t, 2 t + 1, then g + 8's)
// of 16 lanes.
__device__ __forceinline__ void tc5_store_operands(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// 16 columns of this warp's 32 lanes (a thread is a lane); the wait that defines
// them comes with the load.
__device__ __forceinline__ void tc5_load16(uint32_t addr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
// fp32 sums, A and B of one 16-bit type, both K-major, M = 128
template <typename T>
__device__ __forceinline__ uint32_t tc5_idesc(int n) {
  const uint32_t type = std::is_same_v<T, __nv_bfloat16> ? 1u : 0u;
  return (1u << 4) | (type << 7) | (type << 10) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}
// Wait of a whole warp for the phase of `bar` with the given parity.  A phase
// that has passed already costs one probe and one vote (40 clocks; the loop
// below with its checks took 90 to 500, and three of them a step were half of the
// MMA warp's time).  A probe of the loop may suspend the warp for 20 us.  After
// ctl[1] of them, or once the CTA's abort flag ctl[0] is up, the wait gives up
// (status word, abort flag) and returns false.
static __device__ __noinline__ bool tc_wait_long(uint32_t bar, uint32_t parity, int* status, volatile int* ctl) {
  bool ok = false;
  for (int i = 0; i < ctl[1]; ++i) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity), "r"(20000u)
        : "memory");
    ok = __all_sync(0xffffffffu, done != 0);
    if (ok || __any_sync(0xffffffffu, ctl[0] != 0)) break;
  }
  if (!ok) {
    atomicCAS(status, kStatusOk, kStatusTimeout);
    ctl[0] = 1;
  }
  return ok;
}
__device__ __forceinline__ bool tc_wait(uint64_t* bar, uint32_t parity, int* status, volatile int* ctl) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return tc_wait_long(smem_addr(bar), parity, status, ctl);
}
// Probes of a wait by default, and at most: 2/3 s.
constexpr int kTcWaitLimit = 1 << 15;

__device__ __forceinline__ int tc_columns(int n_tok) { return (n_tok + 15) / 16 * 16; }

// Codes to weights: a word's four operand registers, two of outputs g, then two of
// outputs g + 8, whose codes stand four bits higher.
template <typename T, bool ZP>
struct W4Dequant;
template <bool ZP>
struct W4Dequant<__nv_bfloat16, ZP> {
  using V = __nv_bfloat162;
  static constexpr float kUnit = ZP ? 1.f : 0x1p+33f;  // what the sums are multiplied by in the end
  V mul[2], add[2], sc[2];
  static __device__ __forceinline__ V pair(float lo, float hi) { return __floats2bfloat162_rn(lo, hi); }
  static __device__ __forceinline__ V word(uint32_t w) { return *reinterpret_cast<const V*>(&w); }
  static __device__ __forceinline__ V low(V v) { return __low2bfloat162(v); }
  static __device__ __forceinline__ V high(V v) { return __high2bfloat162(v); }
  // an entry: scales of outputs g and g + 8, and their zero points
  __device__ __forceinline__ void set(uint32_t s, uint32_t z) {
    if constexpr (ZP) {
      // 2^-133 q 2^127 - z 2^-6 (outputs g + 8: 2^-2), times s 2^6 (2^2)
      const V k = __hmul2(word(s), pair(0x1p+6f, 0x1p+2f)), c = __hmul2(word(z), pair(-0x1p-6f, -0x1p-2f));
      mul[0] = mul[1] = pair(0x1p+127f, 0x1p+127f);
      add[0] = low(c);
      add[1] = high(c);
      sc[0] = low(k);
      sc[1] = high(k);
    } else {
      const V k = __hmul2(word(s), pair(0x1p+100f, 0x1p+96f)), c = __hmul2(word(s), pair(-0x1p-30f, -0x1p-30f));
      mul[0] = low(k);
      mul[1] = high(k);
      add[0] = low(c);
      add[1] = high(c);
    }
  }
  __device__ __forceinline__ void operator()(uint32_t w, uint32_t* r) const {
    uint32_t o[4];
    w4_operands(w, o);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int hi = i >> 1;
      V t = __hfma2(word(o[2 * (i & 1) + hi]), mul[hi], add[hi]);
      if constexpr (ZP) t = __hmul2(t, sc[hi]);
      r[i] = *reinterpret_cast<const uint32_t*>(&t);
    }
  }
};
template <bool ZP>
struct W4Dequant<__half, ZP> {
  using V = __half2;
  static constexpr float kUnit = 1.f;
  V add[2], sc[2];
  static __device__ __forceinline__ V pair(float lo, float hi) { return __floats2half2_rn(lo, hi); }
  static __device__ __forceinline__ V word(uint32_t w) { return *reinterpret_cast<const V*>(&w); }
  __device__ __forceinline__ void set(uint32_t s, uint32_t z) {
    // (1024 + q) - (1024 + z); outputs g + 8: (1024 + 16 q) / 16 - (64 + z)
    const V c = __hneg2(__hadd2(ZP ? word(z) : pair(8.f, 8.f), pair(1024.f, 64.f)));
    add[0] = __low2half2(c);
    add[1] = __high2half2(c);
    sc[0] = __low2half2(word(s));
    sc[1] = __high2half2(word(s));
  }
  // `base`: two of 1024, in a register of its own so that mask and bits are one
  // instruction (as two they cost the layer 3.5 us of 29)
  static __device__ __forceinline__ V code(uint32_t w, uint32_t mask, uint32_t base) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xf8;" : "=r"(r) : "r"(base), "r"(w), "r"(mask));  // base | (w & mask)
    return word(r);
  }
  __device__ __forceinline__ void operator()(uint32_t w, uint32_t* r) const {
    uint32_t base = 0x64006400u;
    asm("" : "+r"(base));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int hi = i >> 1;
      const V v = code(i & 1 ? w >> 8 : w, hi ? 0x00f000f0u : 0x000f000fu, base);
      const V t = __hmul2(__hfma2(v, hi ? pair(0x1p-4f, 0x1p-4f) : pair(1.f, 1.f), add[hi]), sc[hi]);
      r[i] = *reinterpret_cast<const uint32_t*>(&t);
    }
  }
};

// Before the roles: barriers and tensor memory.  All threads.
__device__ __forceinline__ void w4_tc_begin(W4TcBars& bars, int limit) {
  const int tid = threadIdx.x;
  if (tid == 0) {
    for (int i = 0; i < (int)kTcBufs; ++i) {
      mbar_init(&bars.a_full[i], kTcUnpackers);
      mbar_init(&bars.a_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.d_full[i], 1);
      mbar_init(&bars.d_empty[i], kTcFinishers);
    }
    for (int i = 0; i < kTcSlots; ++i) {
      mbar_init(&bars.b_full[i], 1);
      mbar_init(&bars.b_empty[i], 1);
    }
    mbar_init(&bars.drained, 1);
    bars.ctl[0] = 0;
    bars.ctl[1] = limit;
    mbar_fence_init();
  }
  if (tid >> 5 == kTcMmaWarp) {
    tmem_alloc(&bars.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
}
// After them.
__device__ __forceinline__ void w4_tc_end(W4TcBars& bars) {
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x >> 5 == kTcMmaWarp) tmem_dealloc(bars.tmem, 512);
}

// The MMA warp.  `items` gives the CTA's items in order: next(item) is false
// after the last.  (Issued from a branch of one thread, whose operands have to be
// moved to uniform registers one by one, a step's 16 took 1,030 clocks to issue.)
template <typename T, typename Items>
__device__ __forceinline__ void w4_tc_mma(const uint8_t* smem, W4TcBars& bars, Items items, int* status) {
  const uint32_t lead = tc5_elect();
  const uint32_t tmem = __shfl_sync(0xffffffffu, bars.tmem, 0);
  // K-major: cores of 8 tokens x 16 bytes, kTcCore apart along K, groups of 8 tokens
  // kTcBGroup apart
  const uint64_t b_first = smem_desc(smem_addr(smem + kTcB), kTcCore, kTcBGroup, kLayoutNone);
  uint32_t buf = 0, buf_phase = 0, slot = 0, slot_phase = 0, item = 0;
  bool ok = true;
  W4TcItem it;
  for (; ok && items.next(it); ++item) {
    const uint32_t idesc = tc5_idesc<T>(tc_columns(it.n_tok));
    const uint32_t d = tmem + 128u * (item & 1u);
    if (!(ok = tc_wait(&bars.d_empty[item & 1u], ((item >> 1) & 1u) ^ 1u, status, bars.ctl))) break;
    for (int tile = it.tile0; tile < it.tile1; tile += 2) {
      ok = tc_wait(&bars.b_full[slot], slot_phase, status, bars.ctl) &&
           tc_wait(&bars.a_full[buf], buf_phase, status, bars.ctl);
      if (!ok) break;
      tc_fence_after();
      const uint64_t b0 = b_first + (uint64_t)(slot * (uint32_t)(kTcBSlot >> 4));
      const uint32_t a = tmem + kTcOperandCol + buf * 128u;
      const uint32_t more = tile > it.tile0;
#pragma unroll
      for (uint32_t k = 0; k < kW4Tile / 16; ++k) {
        tc5_mma(d, a + 8u * k, b0 + (uint32_t)(kTcCore / 8) * k, idesc, k > 0 ? 1u : more, lead);
        tc5_mma(d + 64u, a + 64u + 8u * k, b0 + (uint32_t)(kTcCore / 8) * k, idesc, k > 0 ? 1u : more, lead);
      }
      if (tile + 1 < it.tile1) {  // (the last step may be one tile)
#pragma unroll
        for (uint32_t k = kW4Tile / 16; k < kTcStep / 16; ++k) {
          tc5_mma(d, a + 8u * k, b0 + (uint32_t)(kTcCore / 8) * k, idesc, 1u, lead);
          tc5_mma(d + 64u, a + 64u + 8u * k, b0 + (uint32_t)(kTcCore / 8) * k, idesc, 1u, lead);
        }
      }
      tc5_commit(&bars.a_empty[buf], lead);
      tc5_commit(&bars.b_empty[slot], lead);
      if (++buf == kTcBufs) {
        buf = 0;
        buf_phase ^= 1u;
      }
      if (++slot == kTcSlots) {
        slot = 0;
        slot_phase ^= 1u;
      }
    }
    tc5_commit(&bars.d_full[item & 1u], lead);
  }
  // every MMA has ended before tensor memory goes back
  tc5_commit(&bars.drained, lead);
  if (lead) mbar_wait_bounded(&bars.drained, 0u, status);
  __syncwarp();
}

// A stager warp (0 .. STAGERS - 1): the B operands of every STAGERS-th step.  `items.row(item,
// token)` numbers a token's activation row, `items.rows() + items.offset(row)` is it.
// `hold` (testing): the first step is never handed over, so the waits for it run out.
template <typename T, int STAGERS, typename Items>
__device__ __forceinline__ void w4_tc_stage(uint8_t* smem, W4TcBars& bars, Items items, int stager, int* status,
                                            bool hold) {
  // (a stager that was one step behind another's next use of its slot would take
  // the phase before for the one it waits for)
  static_assert(STAGERS <= kTcSlots, "a stager's step before step i + 2 kTcSlots has waited for step i's MMAs");
  const int lane = threadIdx.x & 31;
  constexpr int kQuads = kTcTokens / 4;
  constexpr int kBatch = kQuads / 2;  // fours of tokens whose loads are in flight together
  // lane: token (lane / 4) % 4 of a four, 16 bytes (8 inputs) h, t of a tile's 8;
  // their 8-byte halves q go to cores 2 (2 h + q) + t / 2
  const int tok = (lane >> 2) & 3, h = lane >> 4, t = lane & 3;
  uint8_t* to = smem + kTcB + tok * 16 + (4 * h + (t >> 1)) * kTcCore + (t & 1) * 8;
  uint32_t ci = 0;  // step of the item's first
  W4TcItem it;
  while (items.next(it)) {
    const int quads = tc_columns(it.n_tok) / 4, steps = it.steps();
    // rows of tokens 4 j + tok (the first token for those that do not exist)
    uint32_t mine[kTcTokens / 32], row[kQuads];
#pragma unroll
    for (int k = 0; k < kTcTokens / 32; ++k) mine[k] = items.row(it, 32 * k + lane < it.n_tok ? 32 * k + lane : 0);
#pragma unroll
    for (int j = 0; j < kQuads; ++j) row[j] = __shfl_sync(0xffffffffu, mine[j / 8], (4 * j + tok) & 31);
    for (int s = (int)((stager + STAGERS - ci % STAGERS) % STAGERS); s < steps; s += STAGERS) {
      const uint32_t i = ci + (uint32_t)s, at = i % kTcSlots;
      const int tile = it.tile0 + 2 * s;
      const bool both = tile + 1 < it.tile1;
      const T* first = items.rows() + (size_t)tile * kW4Tile + 32 * h + 8 * t;
      uint4 v[kBatch][2];
      auto load = [&](int j0) {
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          if (j0 + j < quads) {
            const T* p = first + items.offset(row[j0 + j]);
            v[j][0] = *reinterpret_cast<const uint4*>(p);
            if (both) v[j][1] = *reinterpret_cast<const uint4*>(p + kW4Tile);
          }
        }
      };
      load(0);
      if (!tc_wait(&bars.b_empty[at], ((i / kTcSlots) & 1u) ^ 1u, status, bars.ctl)) return;
      uint8_t* dst = to + at * kTcBSlot;
#pragma unroll
      for (int j0 = 0; j0 < kQuads; j0 += kBatch) {
        if (j0 >= quads) break;
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
#pragma unroll
          for (int tl = 0; tl < 2; ++tl)
            if (j0 + j < quads && (tl == 0 || both)) {
              uint8_t* o = dst + ((j0 + j) >> 1) * kTcBGroup + ((j0 + j) & 1) * 64 + tl * (8 * kTcCore);
              *reinterpret_cast<uint2*>(o) = make_uint2(v[j][tl].x, v[j][tl].y);
              *reinterpret_cast<uint2*>(o + 2 * kTcCore) = make_uint2(v[j][tl].z, v[j][tl].w);
            }
        if (j0 + kBatch < kQuads && j0 + kBatch < quads) load(j0 + kBatch);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0 && !(hold && i == 0)) mbar_arrive(&bars.b_full[at]);
    }
    ci += (uint32_t)steps;
  }
}

// An unpacker warp (0..7): the A operands of two panels.
template <typename T, int GROUP, bool ZP, typename Items>
__device__ __forceinline__ void w4_tc_unpack(uint8_t* smem, W4TcBars& bars, Items items, int unpacker, int* status) {
  const int lane = threadIdx.x & 31;
  const int quarter = unpacker & 3, mt = unpacker >> 2;
  const uint32_t a0 = bars.tmem + ((uint32_t)(32 * quarter) << 16) + kTcOperandCol + mt * 64u;
  uint8_t* ring = smem + unpacker * kTcRingBytes + lane * 16;
  const uint32_t ring_addr = smem_addr(ring);
  constexpr int kLaneEntry = ZP ? 8 : 4, kEntryBytes = 8 * kLaneEntry;
  constexpr int kEntries = kTcStep / GROUP;  // entries of a step
  // this warp's first panel of an item, and the offset of its second (a panel
  // that does not exist takes another: its rows are not stored)
  auto panels = [&](const W4TcItem& it, const W4Geom& g, const uint8_t*& p, uint32_t& second) {
    const int have = it.n_panels[mt] - 2 * quarter;
    p = it.panel[mt] + (have > 0 ? (size_t)(2 * quarter) * g.panel_bytes : 0);
    second = have > 1 ? g.panel_bytes : 0u;
  };

  // ---- the weight stream, over the borders of items
  Items ahead = items;
  const uint8_t* code = nullptr;
  uint32_t code2 = 0;
  int left = 0;
  uint32_t p_slot = 0, slot = 0;
  bool more = true;
  auto produce = [&]() {
    if (left == 0 && more) {
      W4TcItem it;
      do {
        more = ahead.next(it);
      } while (more && it.tile0 >= it.tile1);
      if (more) {
        panels(it, ahead.geom(), code, code2);
        code += (size_t)it.tile0 * kW4TileBytes + lane * 16;
        left = it.tile1 - it.tile0;
      }
    }
    if (more) {
      cp_async_16(ring_addr + p_slot, code);
      cp_async_16(ring_addr + p_slot + kW4TileBytes, code + code2);
      code += kW4TileBytes;
      --left;
    }
    cp_async_commit();
    p_slot = (p_slot + 2 * kW4TileBytes) % kTcRingBytes;
  };
#pragma unroll 1
  for (int d = 0; d < kTcRingTiles - 1; ++d) produce();

  uint32_t buf = 0, buf_phase = 0;
  bool ok = true;
  W4TcItem it;
  while (ok && items.next(it)) {
    const W4Geom& g = items.geom();
    const uint8_t* entry;
    uint32_t entry2;
    panels(it, g, entry, entry2);
    entry += g.entry_off + (size_t)(it.tile0 * kW4Tile / GROUP) * kEntryBytes + (lane >> 2) * kLaneEntry;
    // the lane's scales (and zero points) of a step, asked for one step before
    uint32_t e_next[2][kEntries][2];
    auto ask = [&](int tile) {
#pragma unroll
      for (int e = 0; e < kEntries; ++e) {
        if (tile * kW4Tile + e * GROUP < it.tile1 * kW4Tile) {
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const uint32_t* src = reinterpret_cast<const uint32_t*>(entry + p * entry2 + e * kEntryBytes);
            e_next[p][e][0] = src[0];
            if constexpr (ZP) e_next[p][e][1] = src[1];
          }
        }
      }
      entry += kEntries * kEntryBytes;
    };
    ask(it.tile0);
    for (int tile = it.tile0; tile < it.tile1; tile += 2) {
      W4Dequant<T, ZP> dq[2][kEntries];
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int e = 0; e < kEntries; ++e) dq[p][e].set(e_next[p][e][0], e_next[p][e][1]);
      ask(tile + 2);
      // the MMAs of two steps ago have read this buffer
      if (!(ok = tc_wait(&bars.a_empty[buf], buf_phase ^ 1u, status, bars.ctl))) break;
      tc_fence_after();
      const uint32_t a = a0 + buf * 128u;
#pragma unroll
      for (int ti = 0; ti < 2; ++ti) {
        if (ti == 1 && tile + 1 >= it.tile1) break;
        cp_async_wait<kTcRingTiles - 2>();
        produce();
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const uint4 w4 = *reinterpret_cast<const uint4*>(ring + slot + p * kW4TileBytes);
          const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
          uint32_t r[16];
#pragma unroll
          for (int i = 0; i < 4; ++i) dq[p][(ti * kW4Tile + 16 * i) / GROUP](w[i], r + 4 * i);
          tc5_store_operands(a + ((uint32_t)(16 * p) << 16) + 32u * ti, r);
        }
        slot = (slot + 2 * kW4TileBytes) % kTcRingBytes;
      }
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.a_full[buf]);
      if (++buf == kTcBufs) {
        buf = 0;
        buf_phase ^= 1u;
      }
    }
  }
  cp_async_wait<0>();
}

// A finisher warp (0..3).  `take(items, item, c, lo, hi)` gets the sums of tokens c ..
// c + 15 of the lane's rows 32 finisher + lane of both accumulators; called for
// every 16 tokens that there are.  `ready(items, item)` comes before, while the
// item is being multiplied.
template <typename Items, typename Ready, typename Take>
__device__ __forceinline__ void w4_tc_finish(W4TcBars& bars, Items items, int finisher, int* status, Ready ready,
                                             Take take) {
  const uint32_t lanes = (uint32_t)(32 * finisher) << 16;
  uint32_t item = 0;
  W4TcItem it;
  for (; items.next(it); ++item) {
    ready(items, it);
    if (!tc_wait(&bars.d_full[item & 1u], (item >> 1) & 1u, status, bars.ctl)) return;
    tc_fence_after();
    const uint32_t d = bars.tmem + lanes + 128u * (item & 1u);
    for (int c = 0; c < it.n_tok; c += 16) {
      float lo[16], hi[16];
      tc5_load16(d + c, lo);
      tc5_load16(d + 64u + c, hi);
      take(items, it, c, lo, hi);
    }
    tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&bars.d_empty[item & 1u]);
  }
}

}  // namespace moe
