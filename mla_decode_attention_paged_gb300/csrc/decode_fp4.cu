// decode_fp4.cu -- split-KV MLA decode attention over FP4 caches, on the FP8 tensor
// cores, for groups of 16 or 32 query rows (heads, or heads x tokens of
// multi-token decode and prefill; 16 rows are a group, more go in groups of 32
// of which the last may be half empty).
//
// What it computes ("The Weight Absorption Trick"; "Seven Ways LLMs Handle
// Attention", section 5; "Flash-Decoding and FlashInfer"; "The Architecture of
// Memory", "Leveraging Tensor Cores and Asynchronous Prefetching": caches of 2
// to 4 bits on the tensor cores): for one head group of one sequence and one
// contiguous range of its tokens, with q_full[h] = [W^UK_h^T q_nope_h | q_pe_h]
// (576 wide) and the cached rows c_t = [latent | RoPE key] (576 wide),
//     s[t][h] = scale * q_full[h] . c_t
//     o_lat[h] = sum_t softmax(s[., h])_t * c_t[0:512]
// and emits o_lat (normalised within the range) with the range's lse.
//
// Why FP8 operands.  A row of 320 bytes is 3.6 times shorter than a bf16 row, so
// what bounds a 16-head decode is no longer HBM alone: an SM's share of it, 22
// bytes a cycle, is a row every 14 cycles, and a row expanded to 16 bits costs
// shared memory (128 bytes a cycle) 1,152 bytes written and 2,176 read by the two
// products, 26 cycles.  E2M1 times a power of two is an E5M2 value (see
// decode_common.cuh), so the row is expanded to 576 bytes and costs half of that,
// and exactly.  The other operands are fp32 values split into FP8 terms that
// stand side by side in the MMA's N extent (16 heads fill an eighth of it: the
// MMA's time is its A operand's way through shared memory):
//   Q: two E4M3 terms, q = 2^-k (hi + lo / 16): off by at most 2^-9 of a fp16 value,
//      half of what bf16 is, and not at all of a bf16 value, as long as it is above
//      2^-12 of the largest of the 8 or 16 heads that share k; below, by at most 2^-8
//      of the value or 2^-21 of that largest
//   P: three E5M2 terms, hi + mid + lo = the weight's fp16 value, exactly down to
//      2^-16 of the running maximum and to 2^-26 of it below: as many bits as the
//      1-byte caches' weights
// Products as in decode_tc.cu, with the 128 tokens of a tile as M:
//     S^T [128 tok x 2 HC] = C_tile [128 x 576] * [Q_hi | Q_lo]^T          (K-major)
//     O^T [512 x 3 HC] += C_tile^T [512 x 128] * [P_hi | P_mid | P_lo]^T   (MN-major)
//
// Warp roles (640 threads):
//   warps 0-7    softmax, in two groups that share the heads: a thread to a token row
//                of S^T; Q of each segment; epilogue
//   warps 8-15   expansion: rows from global memory into registers, a tile (32 rows:
//                half a tile) ahead, then through byte permutations into one of two
//                operand slots
//   warp 16      tensor memory and QK issuer;  warp 17  PV issuer
//   warp 18      pages of the tiles to come, and their rows' way into L2
//   warp 19      no work
// Measured, 32 sequences of 32,768 tokens (1,048,576 rows of 320 bytes): 102 us at 16
// heads (3.3 TB/s), 133 us at 32 (2.5 TB/s, 549 TFLOP/s), 461 us for 128 x 8,192
// tokens at 128 heads (634 TFLOP/s).  At 16 rows the L1 and shared-memory data pipe
// bounds it: 3,330 wavefronts a tile (1,900 of loads and stores, 1,424 of the
// products' operands) in about 3,600 cycles, of the 1,900 about 990 for the rows'
// loads, the expanded rows and the weights, the others not looked into one by one;
// at 32 rows the chain expansion, QK, softmax, PV through two slots, about 4,700
// cycles a tile for 3,980 wavefronts.
// Every wait is bounded: on timeout the CTA records MLA_ERR_DEVICE_TIMEOUT,
// drains, frees its tensor memory and returns.  (The wait of setmaxnreg is not: the
// launch refuses a build that could not end it.)
#include <atomic>
#include <cuda_fp16.h>

#include "blackwell_ptx.cuh"
#include "decode_common.cuh"
#include "params.cuh"

namespace mla {
namespace {

using namespace ptx;
using namespace dc;

constexpr int kSlots = 2;
constexpr int kAhead = 4;                                 // tiles between the page lookup and the expansion
constexpr int kRing = 8;                                  // tiles of looked-up pages kept
constexpr uint32_t kLatBox = kTile * 128;                 // [128 tokens x 128 latent columns] E5M2, SW128: one O^T chunk
constexpr uint32_t kRopeBox = 4 * kLatBox;                // offset of [128 tokens x 64 RoPE columns] E5M2, SW64
constexpr uint32_t kSlotBytes = kRopeBox + kTile * kRope;  // 72 KB
constexpr uint32_t kWaitLimitNs = 2000000000u;            // 2 s
constexpr float kRescaleThreshold = 5.f;                  // log2 units
constexpr float kWeightBits = 10.f;                       // a weight is 2^10 at the running maximum, 2^15 at most

template <int HC>
struct Fp4Cfg {
  static constexpr int kHeads = HC / 2, kSoftWarps = 8;     // two softmax groups
  // expansion: four lanes to a cached row, the rows of a half tile to the eight
  // warps; 16 query rows: both halves at once, 32: one after the other
  static constexpr int kExpWarps = 8, kHalves = HC == 16 ? 2 : 1;
  static constexpr int kThreads = 32 * (kSoftWarps + kExpWarps + 4);
  // registers of a thread at the launch, and of each role (setmaxnreg)
  static constexpr bool kSplitRegs = HC == 32;
  static constexpr int kRegs = 96;
  static constexpr int kSoftRegs = 128, kExpRegs = 72, kIssueRegs = 80;
  static_assert(!kSplitRegs || 32 * (kSoftWarps * kSoftRegs + kExpWarps * kExpRegs + 4 * kIssueRegs) <= kThreads * kRegs,
                "setmaxnreg shares out what the block was launched with");
  static constexpr int kNQ = 2 * HC, kNP = 3 * HC;          // N of the products
  static constexpr uint32_t kQBox = kNQ * 128;              // [2 HC rows x 128 columns] E4M3, SW128
  static constexpr uint32_t kQBytes = 4 * kQBox + kNQ * 64;  // + [2 HC rows x 64 RoPE columns], SW64
  static constexpr uint32_t kPBytes = kTile * kNP;          // P^T core matrices: 16 rows x 8 tokens, 128 bytes each
  static constexpr uint32_t kOffQ = kSlots * kSlotBytes;
  static constexpr uint32_t kOffP = kOffQ + kQBytes;
  static constexpr uint32_t kOffLut = kOffP + 2 * kPBytes;  // magnitudes by scale byte
  static constexpr uint32_t kOffMisc = kOffLut + 256 * 8;
  static constexpr uint32_t kMiscBytes = 1024 + 17 * HC * 4;
  static constexpr uint32_t kSmem = kOffMisc + kMiscBytes + 1024;  // +1024: base alignment slack
  static constexpr uint32_t kColS = 0;                       // + buf * 2 HC
  static constexpr uint32_t kColO = 128, kColOStep = HC == 16 ? 64 : 96, kTmemCols = 512;
  static_assert(kSmem <= 232448, "dynamic shared memory of one CTA");
  static_assert(kColO + 3 * kColOStep + kNP <= kTmemCols && 2 * kNQ <= int(kColO), "tensor memory");
};

struct Fp4Barriers {
  // RoPE and latent boxes 0 and 1 expanded, boxes 2 and 3; PV has read boxes 0 and 1, 2 and 3
  uint64_t full[kSlots][2], empty[kSlots][2];
  uint64_t q_full, s_full[2], s_free[2], p_full[2], pv_done[2], o_full, o_free, drain[2];
  uint64_t ring_full[kRing];
  uint32_t tmem_base;
  int abort;
  int expanding;               // the tile that the expansion is at
  int valid[kRing];            // rows of a tile, 0 behind the last
  const uint8_t* page[kRing][kTile / 16];  // first row of each of its pages
};
static_assert(sizeof(Fp4Barriers) <= 1024, "barriers and page ring");

__device__ __forceinline__ void fail(Fp4Barriers* B, int* status) {
  B->abort = 1;
  set_status(status, MLA_ERR_DEVICE_TIMEOUT);
}

// OR over the 128 threads of a softmax group (named barrier 1 + group).
__device__ __forceinline__ bool group_any(int group, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %2, 0;\n\t"
      "bar.red.or.pred q, %1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(group + 1), "r"(uint32_t(pred))
      : "memory");
  return r != 0;
}

// Reduces 8 or 16 values per lane over a warp, each lane keeping half of them a
// round; every lane gets that of value lane / (32 / N).
template <int N, bool kMax>
__device__ __forceinline__ float warp_reduce(float (&v)[N], int lane) {
  if constexpr (N == 16) {
    return warp_transpose_reduce<16, kMax>(v, lane);
  } else {
    static_assert(N == 8, "8 or 16 values per lane");
#pragma unroll
    for (int w = 4, o = 16; w >= 1; w >>= 1, o >>= 1) {
      const bool upper = lane & o;
#pragma unroll
      for (int i = 0; i < w; ++i) {
        const float keep = upper ? v[i + w] : v[i], send = upper ? v[i] : v[i + w];
        const float got = __shfl_xor_sync(0xffffffffu, send, o);
        v[i] = kMax ? fmaxf(keep, got) : keep + got;
      }
    }
#pragma unroll
    for (int o = 2; o > 0; o >>= 1) {
      const float got = __shfl_xor_sync(0xffffffffu, v[0], o);
      v[0] = kMax ? fmaxf(v[0], got) : v[0] + got;
    }
    return v[0];
  }
}
// N (8 or 16) tensor memory columns.
template <int N>
__device__ __forceinline__ void tmem_load(uint32_t a, float (&v)[N]) {
  if constexpr (N == 16) tmem_ld16(a, v);
  else tmem_ld8(a, v);
}

// The same of three places `step` columns apart, with one wait.
template <int N>
__device__ __forceinline__ void tmem_load3(uint32_t a, uint32_t step, float (&v)[3][N]) {
  static_assert(N == 8 || N == 16, "8 or 16 columns");
  uint32_t r[3][N];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    uint32_t* x = r[i];
    if constexpr (N == 16)
      asm volatile(
          "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
          : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7]),
            "=r"(x[8]), "=r"(x[9]), "=r"(x[10]), "=r"(x[11]), "=r"(x[12]), "=r"(x[13]), "=r"(x[14]), "=r"(x[15])
          : "r"(a + i * step));
    else
      asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                   : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7])
                   : "r"(a + i * step));
  }
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < 3; ++i)
#pragma unroll
    for (int n = 0; n < N; ++n) {
      asm volatile("" : "+r"(r[i][n]));  // valid from the wait on
      v[i][n] = __uint_as_float(r[i][n]);
    }
}

// Instruction descriptor, kind::f8f6f4, fp32 accumulator (bits 4-5 = 1): A is
// E5M2 (bits 7-9 = 1), B E5M2 or E4M3 (bits 10-12 = 1 or 0), the rest as for f16.
constexpr uint32_t idesc_f8(int M, int N, bool mn_major, bool b_e5m2) {
  return (1u << 4) | (1u << 7) | (uint32_t(b_e5m2) << 10) | (uint32_t(mn_major) << 15) | (uint32_t(mn_major) << 16) |
         (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
template <int N>
__device__ __forceinline__ void tmem_store(uint32_t a, const float (&v)[N]) {
  if constexpr (N == 16) {
    tmem_st16(a, v);
  } else {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(a),
                 "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
                 "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
                 "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
                 : "memory");
  }
}
// Two fp16 values to E4M3.
__device__ __forceinline__ uint32_t e4m3x2_of_f16x2(uint32_t x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// The larger magnitudes; a NaN gives way to the other value.
__device__ __forceinline__ uint32_t max_abs_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b & 0x7fff7fffu));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Two fp16 values as they are, infinities as NaN (x + 0 x).
__device__ __forceinline__ uint32_t nan_of_inf_f16x2(uint32_t x) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %1;" : "=r"(r) : "r"(x), "r"(0u));
  return r;
}
// A warpgroup's registers per thread from here on.
template <bool kSplit, int N, int kFrom>
__device__ __forceinline__ void set_max_regs() {
  if constexpr (kSplit && N > kFrom) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
  if constexpr (kSplit && N < kFrom) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// A bounded wait.  Where registers are shared out it is inline, since a function
// call has registers of its own, and short, since the roles' loops share the
// instruction caches; else it calls (16 rows, when the batch above took 106 us by
// calls: 111 inline, 121 with a longer loop inline).
template <bool kInline>
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, const volatile int* abort) {
  if constexpr (!kInline) return mbar_wait(bar, parity, abort, kWaitLimitNs);
  if (mbar_try_wait(bar, parity)) return true;
  uint32_t t0, t1;  // nanoseconds; the low word wraps after 4.3 s
  asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t0));
#pragma unroll 1
  do {
    if (mbar_try_wait(bar, parity)) return true;
    asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t1));
  } while (!*abort && t1 - t0 < kWaitLimitNs);
  return false;
}
// Read-once data.
__device__ __forceinline__ uint4 ld_stream(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
// 32 codes (16 bytes of a row) to 32 E5M2 bytes.
__device__ __forceinline__ void expand_block(uint4 v, uint2 table, uint4& lo, uint4& hi) {
  e2m1_to_e5m2(v.x, table, lo.x, lo.y);
  e2m1_to_e5m2(v.y, table, lo.z, lo.w);
  e2m1_to_e5m2(v.z, table, hi.x, hi.y);
  e2m1_to_e5m2(v.w, table, hi.z, hi.w);
}

// A CTA's walker at its first tile, as TileWalkerT::init leaves it: a warp divides for
// several lanes at once and searches 32 ways, and all warps run one copy of this
// code (with a copy in each role and serial divisions the first tile's scores came
// 0.6 us later; one decode of 93 tokens 14.3 -> 12.3 us with what load_q does).
__device__ __forceinline__ void walk_start(TileWalkerT<true>& w, const DecodeParams& p, int cp, int Cp, int lane) {
  const int* ts = p.tile_start;
  const long long S = p.status[1], W = ts[p.batch];  // effective split count and tiles, from the plan
  w.tile_start = ts;
  w.seg_base = p.seg_base;
  w.len = p.len;
  w.W = W;
  w.S = S;
  const long long part = (cp + (lane & 1)) * S / Cp;  // first partition of this CTA, of the next
  const long long pa = __shfl_sync(0xffffffffu, part, 0), pb = __shfl_sync(0xffffffffu, part, 1);
  const long long unit = part_start(lane == 1 ? pa + 1 : lane == 2 ? pb : pa, W, S);
  w.p = pa;
  w.u = w.p_start = __shfl_sync(0xffffffffu, unit, 0);
  w.p_next = __shfl_sync(0xffffffffu, unit, 1);
  w.u_end = __shfl_sync(0xffffffffu, unit, 2);
  w.s_b = w.e_b = 0;
  w.b = w.len_b = w.seg_b = 0;
  if (w.u >= w.u_end) return;
  // the sequences that end at or before unit u: below(i) = tile_start[i + 1] <= u is
  // true for those and for no other; each round looks at the last of 32 ranges
  int lo = 0, hi = p.batch;
  while (lo < hi) {
    const int step = (hi - lo + 31) >> 5, i = lo + step * (lane + 1) - 1;
    const bool below = i < hi && ts[i + 1] <= w.u;
    lo += step * __popc(__ballot_sync(0xffffffffu, below));
    hi = min(hi, lo + step - 1);
  }
  w.b = lo;
  w.enter_sequence_body();
}

// kCausal: multi-token decode (q_len > 1, so groups of 32 rows) masks each row's
// later positions on a sequence's last tiles.
template <int HC, bool kCausal>
__global__ void __launch_bounds__(Fp4Cfg<HC>::kThreads, 1) decode_fp4_kernel(DecodeParams p) {
  using C = Fp4Cfg<HC>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Fp4Barriers* B = reinterpret_cast<Fp4Barriers*>(smem + C::kOffMisc);
  // [2][HC][4] maxima, [HC][4] sums, [HC] 1 / l, [2 groups][2][4] largest values of
  // Q, [HC] running maxima less kWeightBits, [HC] factors of a rescale
  float* red = reinterpret_cast<float*>(smem + C::kOffMisc + 1024);
  const uint32_t sbase = smem_u32(smem);
  const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x) >> 5, 0), lane = threadIdx.x & 31;
  constexpr int kQkWarp = C::kSoftWarps + C::kExpWarps, kPvWarp = kQkWarp + 1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      // the test hook: one arrival more than the first box gets
      for (int c = 0; c < 2; ++c) mbar_init(&B->full[i][c], C::kExpWarps + (p.inject_wait_timeout && i + c == 0 ? 1 : 0));
      for (int c = 0; c < 2; ++c) mbar_init(&B->empty[i][c], 1);
    }
    for (int i = 0; i < kRing; ++i) mbar_init(&B->ring_full[i], 1);
    mbar_init(&B->q_full, 32 * C::kSoftWarps);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B->s_full[i], 1);
      mbar_init(&B->s_free[i], 32 * C::kSoftWarps);
      mbar_init(&B->p_full[i], 32 * C::kSoftWarps);
      mbar_init(&B->pv_done[i], 1);
      mbar_init(&B->drain[i], 1);
    }
    mbar_init(&B->o_full, 1);
    mbar_init(&B->o_free, 32 * C::kSoftWarps);
    B->abort = 0;
    B->expanding = 1 - kAhead;  // two tiles first, the others' way into L2 once the first is here
    fence_mbar_init();
  }
  if (warp == kQkWarp) {
    tmem_alloc(&B->tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  if (threadIdx.x < 256) reinterpret_cast<uint2*>(smem + C::kOffLut)[threadIdx.x] = e2m1_table(threadIdx.x);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = B->tmem_base;
  griddep_wait();  // the plan and Q come from the kernel before
  griddep_launch_dependents();

  const int G = p.num_groups, g = blockIdx.x % G, cp = blockIdx.x / G, Cp = gridDim.x / G;
  TileWalkerT<true> start;
  walk_start(start, p, cp, Cp, lane);
  const volatile int* abort_flag = &B->abort;

  if (warp >= C::kSoftWarps && warp < kQkWarp) {
    // ------------------------------------------------------------ expansion
    set_max_regs<C::kSplitRegs, C::kExpRegs, C::kRegs>();
    // A warp has 8 rows of a half tile, all of one page; thread (r, j) takes block
    // 4c + j of its row, c = 0 .. 3, and piece j of the row's tail (RoPE blocks 16
    // and 17, scales 0 - 15, scales 16 and 17): four lanes read 64 bytes of a row,
    // and their stores and those of the next row's lanes go to distinct banks.  A
    // piece's registers are loaded again, for the next rows, as soon as it has
    // been expanded.
    constexpr int R = C::kHalves;
    const int w8 = 8 * (warp - C::kSoftWarps), j = lane & 3, r = w8 + (lane >> 2);
    const int lane2 = (lane & ~3) + 2, lane3 = lane2 + 1;
    // the block's two 16-byte pieces in its row of a latent and of the RoPE box
    const uint32_t at0 = r * 128 + (((2 * j) ^ (r & 7)) << 4), at1 = at0 ^ 16;
    const uint32_t rope0 = kRopeBox + r * 64 + (((2 * j) ^ ((r >> 1) & 3)) << 4), rope1 = rope0 ^ 16;
    const uint2* lut = reinterpret_cast<const uint2*>(smem + C::kOffLut);
    const uint32_t byte_j = 0x4440 + j, byte_r = 0x4440 + (j & 1);  // bytes j and j % 2 of a word
    const int page_log2 = __ffs(p.page_size) - 1;
    const uint8_t* row[R];
    // this thread's rows of half tile `half` (and the other) of the tile in ring entry e
    auto look = [&](int e, int half) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int at = w8 + 64 * (half + i);
        row[i] = B->page[e][at >> page_log2] + (((at & (p.page_size - 1)) + (lane >> 2)) * kFp4RowBytes + 16 * j);
      }
    };
    // scale bytes of 0 (values of 0) where there is no row
    bool ok = __all_sync(0xffffffffu, wait_for<C::kSplitRegs>(&B->ring_full[0], 0, abort_flag));
    int v0 = ok ? B->valid[0] : 0, v1 = 0;
    uint4 v[R][5];
    look(0, 0);
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int c = 0; c < 5; ++c) v[i][c] = r + 64 * i < v0 ? ld_stream(row[i] + 64 * c) : make_uint4(0, 0, 0, 0);
    for (uint32_t it = 0; v0 > 0; ++it) {
      const uint32_t k = R == 2 ? it : it >> 1, half = R == 2 ? 0 : it & 1, slot = k % kSlots;
      const bool begins = R == 2 || half == 0, ends = R == 2 || half == 1;
      uint8_t* base = smem + slot * kSlotBytes;
      int left;  // of the next rows: this thread's row r + 64 i is there if it is below
      if (ends) {
        const int e = (k + 1) % kRing;
        ok = __all_sync(0xffffffffu, wait_for<C::kSplitRegs>(&B->ring_full[e], ((k + 1) / kRing) & 1, abort_flag));
        if (!ok) break;
        left = v1 = B->valid[e];
        look(e, 0);
      } else {
        look(k % kRing, 1);
        left = v0 - 64;
      }
      // the blocks' scale bytes, and whether any is outside 2^-13 .. 2^13
      uint32_t sc[R][5];
      bool far = false;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const uint32_t tail[5] = {
            __shfl_sync(0xffffffffu, v[i][4].x, lane2), __shfl_sync(0xffffffffu, v[i][4].y, lane2),
            __shfl_sync(0xffffffffu, v[i][4].z, lane2), __shfl_sync(0xffffffffu, v[i][4].w, lane2),
            __shfl_sync(0xffffffffu, v[i][4].x, lane3)};
#pragma unroll
        for (int c = 0; c < 5; ++c) {
          sc[i][c] = __byte_perm(tail[c], 0, c < 4 ? byte_j : byte_r);
          far |= sc[i][c] - (127 - 13) > 26;
        }
      }
      if (begins && threadIdx.x == 32 * C::kSoftWarps) *reinterpret_cast<volatile int*>(&B->expanding) = int(k);
      // the tails first: their registers are the first that the next rows need
#pragma unroll
      for (int cc = 0; cc < 5; ++cc) {
        const int c = cc == 0 ? 4 : cc - 1;
        if ((c == 4 || c == 2) && begins) {
          ok = __all_sync(0xffffffffu, wait_for<C::kSplitRegs>(&B->empty[slot][c & 2 ? 1 : 0], ((k / kSlots) & 1) ^ 1, abort_flag));
          if (!ok) break;
        }
        if (c < 4 || j < 2) {
#pragma unroll
          for (int i = 0; i < R; ++i) {
            // the magnitudes' E5M2 bytes: within that range a scale adds to the
            // exponents, four to each byte and step (0 stays 0)
            uint2 tab = make_uint2(sc[i][c] * 0x04040400u + (0x3e3c3800u - 127u * 0x04040400u),
                                   sc[i][c] * 0x04040404u + (0x46444240u - 127u * 0x04040404u));
            if (far) tab = lut[sc[i][c]];
            uint4 lo, hi;
            expand_block(v[i][c], tab, lo, hi);
            uint8_t* dst = base + (c < 4 ? c * kLatBox + 64 * 128 * (half + i) : 64 * 64 * (half + i));
            *reinterpret_cast<uint4*>(dst + (c < 4 ? at0 : rope0)) = lo;
            *reinterpret_cast<uint4*>(dst + (c < 4 ? at1 : rope1)) = hi;
          }
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
          if (r + 64 * i < left) v[i][c] = ld_stream(row[i] + 64 * c);
          else if (c == 4) v[i][c] = make_uint4(0, 0, 0, 0);
        }
        if ((c == 1 || c == 3) && ends) {
          // no proxy fence here: it would wait for the loads in flight.  The QK
          // issuer, which acquires these writes, fences for them.
          __syncwarp();
          if (lane == 0) mbar_arrive(&B->full[slot][c >> 1]);
        }
      }
      if (!ok) break;
      if (ends) v0 = v1;
    }
    if (!ok) fail(B, p.status);
  } else if (warp >= kQkWarp) {
    set_max_regs<C::kSplitRegs, C::kIssueRegs, C::kRegs>();
    // Whole warps wait and compute addresses, one lane issues: with everything
    // uniform a product costs a few instructions (with a single lane in the
    // role, 190 cycles each).
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, wait_for<C::kSplitRegs>(bar, parity, abort_flag)) != 0;
    };
    if (warp == kQkWarp) {
      // ------------------------------------------------------------ QK issuer
      TileWalkerT<true> walk = start;
      constexpr uint32_t id_qk = idesc_f8(128, C::kNQ, false, false);
      constexpr uint64_t kDescK = smem_desc(0, 16, 1024, kSwizzle128B);   // K-major SW128 (8-row groups of 1 KB)
      constexpr uint64_t kDescRope = smem_desc(0, 16, 512, kSwizzle64B);  // K-major SW64 (8-row groups of 512 B)
      const uint64_t q = desc_addr(sbase + C::kOffQ);  // (no sum of addresses here leaves the descriptors' 14-bit field)
      uint32_t k = 0, seg = 0;
      TileInfo t;
      bool ok = true;
      while (walk.next(t)) {
        const uint32_t slot = k % kSlots, buf = k & 1;
        // every softmax thread has read tile k - 2's scores
        if (k >= 2 && !(ok = wait(&B->s_free[buf], ((k - 2) >> 1) & 1))) break;
        if (t.first && !(ok = wait(&B->q_full, seg++ & 1))) break;
        const uint32_t d = tmem + C::kColS + buf * C::kNQ;
        const uint64_t a = desc_addr(sbase + slot * kSlotBytes);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (!(ok = wait(&B->full[slot][half], (k / kSlots) & 1))) break;
          fence_proxy_async_smem();  // the expansion's writes, for this warp's and the PV issuer's products
          tc_fence_after();
          if (elect_one()) {
            if (half == 0) {
#pragma unroll
              for (int kk = 0; kk < 2; ++kk)
                mma_f8(d, kDescRope + a + (kRopeBox + 32 * kk) / 16, kDescRope + q + (4 * C::kQBox + 32 * kk) / 16, id_qk, kk);
            }
#pragma unroll
            for (int kk = 8 * half; kk < 8 * half + 8; ++kk) {
              const uint32_t box = kk >> 2, col = 32 * (kk & 3);
              mma_f8(d, kDescK + a + (box * kLatBox + col) / 16, kDescK + q + (box * C::kQBox + col) / 16, id_qk, 1);
            }
            if (half == 1) mma_commit(&B->s_full[buf]);
          }
          __syncwarp();
        }
        if (!ok) break;
        ++k;
      }
      if (!ok) fail(B, p.status);
      if (elect_one()) {  // every product this lane issued completes before teardown
        mma_commit(&B->drain[0]);
        mbar_wait_until(&B->drain[0], 0, global_timer_ns() + kWaitLimitNs / 4);
      }
      __syncwarp();
    } else if (warp == kPvWarp) {
      // ------------------------------------------------------------ PV issuer
      TileWalkerT<true> walk = start;
      constexpr uint32_t id_pv = idesc_f8(128, C::kNP, true, true);
      constexpr uint64_t kDescMN = smem_desc(0, kLatBox, 1024, kSwizzle128B);  // MN-major SW128: 128 columns, 8-token groups
      constexpr uint64_t kDescP = smem_desc(0, 128, 2048, kSwizzleNone);       // P^T core matrices
      uint32_t k = 0, seg = 0;
      TileInfo t;
      bool ok = true;
      while (walk.next(t)) {
        const uint32_t slot = k % kSlots, buf = k & 1;
        if (!(ok = wait(&B->p_full[buf], (k >> 1) & 1))) break;
        if (t.first && seg > 0 && !(ok = wait(&B->o_free, (seg - 1) & 1))) break;
        tc_fence_after();
        const int nk = (t.valid + 31) >> 5;
        const uint64_t a = kDescMN + desc_addr(sbase + slot * kSlotBytes);
        const uint64_t b = kDescP + desc_addr(sbase + C::kOffP + buf * C::kPBytes);
        const uint32_t later = !t.first;
        if (elect_one()) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t d = tmem + C::kColO + c * C::kColOStep;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              if (kk < nk) mma_f8(d, a + (c * kLatBox + 4096 * kk) / 16, b + 512 * kk / 16, id_pv, kk > 0 ? 1u : later);
            if (c & 1) mma_commit(&B->empty[slot][c >> 1]);
          }
          mma_commit(&B->pv_done[buf]);
          if (t.last) mma_commit(&B->o_full);
        }
        __syncwarp();
        if (t.last) ++seg;
        ++k;
      }
      if (!ok) fail(B, p.status);
      if (elect_one()) {
        mma_commit(&B->drain[1]);
        mbar_wait_until(&B->drain[1], 0, global_timer_ns() + kWaitLimitNs / 4);
      }
      __syncwarp();
    } else if (warp == kPvWarp + 1) {
      // ------------------------------------------------------------ page lookup
      // Where the rows of tile k + kAhead are when the expansion is at tile k (it
      // reads the ring a tile ahead), and those rows' way into L2.
      TileWalkerT<true> walk = start;
      const volatile int* at = &B->expanding;
      const int page_log2 = __ffs(p.page_size) - 1;
      TileInfo t;
      bool more = true, ok = true;
      for (int k = 0; more; ++k) {
        const uint64_t t0 = global_timer_ns();
        while (*at + kAhead < k && (ok = !*abort_flag && global_timer_ns() - t0 < kWaitLimitNs)) __nanosleep(64);
        if (!__all_sync(0xffffffffu, ok)) {
          fail(B, p.status);
          break;
        }
        more = walk.next(t);
        const int e = k % kRing, first = lane << page_log2;
        if (more && first < t.valid) {
          int page = __ldg(p.block_table + size_t(t.b) * p.max_pages + ((t.tile * kTile) >> page_log2) + lane);
          if (uint32_t(page) >= uint32_t(p.num_pages)) {
            set_status(p.status, MLA_ERR_DEVICE_BOUNDS);
            page = 0;
          }
          const uint8_t* rows = static_cast<const uint8_t*>(p.cache) + (size_t(page) << page_log2) * kFp4RowBytes;
          B->page[e][lane] = rows;
          if (k > 0) prefetch_l2(rows, min(p.page_size, t.valid - first) * kFp4RowBytes);
        }
        if (lane == 0) B->valid[e] = more ? t.valid : 0;
        __syncwarp();
        if (lane == 0) mbar_arrive(&B->ring_full[e]);
      }
    }
  } else {
    // ------------------------------------------------------------ Q, softmax, epilogue
    // Group c (four warps) has heads NH c .. NH (c + 1) - 1 of the head group; thread
    // st of it the token row st of S^T (its TMEM lane).
    set_max_regs<C::kSplitRegs, C::kSoftRegs, C::kRegs>();
    constexpr int NH = C::kHeads;
    const int c = warp >> 2, q4 = warp & 3, st = threadIdx.x & 127;
    const uint32_t lane_off = uint32_t(q4 * 32) << 16;
    // the last group of 32 may be half empty: rows of zeros that write nothing
    const bool live = HC == 16 || g * HC + NH * c < p.heads;
    uint32_t* qtop = reinterpret_cast<uint32_t*>(red + 13 * HC + 8 * c);  // [2 segments' parity][4] largest magnitude by warp
    TileWalkerT<true> walk = start;
    // Q of a segment's sequence as two E4M3 terms: eight threads per head, each
    // every eighth chunk of eight values.  Every QK MMA of the previous segment
    // has completed: this thread saw the s_full of its last tile.
    float qs = 0.f, qs_next = 0.f;  // what a sum of Q's terms is multiplied by, this segment and the next
    auto load_q = [&](int b, uint32_t seg) {
      constexpr int T = 128 / NH, N = (72 + T - 1) / T;  // threads per head, chunks of eight values each
      const int hl = st / T, i0 = st % T, row_hi = NH * c + hl, row_lo = HC + row_hi;
      const uint4* src = reinterpret_cast<const uint4*>(p.q_full + (size_t(b) * p.heads + g * HC + row_hi) * kRow);
      uint4 u[N];
      uint32_t top2 = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        u[i] = live && i0 + T * i < 72 ? src[i0 + T * i] : make_uint4(0, 0, 0, 0);
        // E4M3 has no infinity: one in a query makes its head NaN, not the largest finite
        // value, and has no part in the scale
        u[i] = make_uint4(nan_of_inf_f16x2(u[i].x), nan_of_inf_f16x2(u[i].y), nan_of_inf_f16x2(u[i].z), nan_of_inf_f16x2(u[i].w));
        top2 = max_abs_f16x2(max_abs_f16x2(max_abs_f16x2(max_abs_f16x2(top2, u[i].x), u[i].y), u[i].z), u[i].w);
      }
      uint32_t top = max(top2 & 0xffff, top2 >> 16);  // of magnitudes, in fp16 bits
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      if (lane == 0) qtop[4 * (seg & 1) + q4] = top;
      group_any(c, false);
      const uint4 top4 = *reinterpret_cast<const uint4*>(qtop + 4 * (seg & 1));
      top = max(max(top4.x, top4.y), max(top4.z, top4.w));
      // up to a power of two in [128, 256): by 2^(7 - floor(log2 top)), at most 2^30
      // (fp16 values: 2^-24 .. 2^15), in two steps that fp16 holds; what becomes
      // subnormal is below 2^-21 of the largest value
      const float ftop = __half2float(__ushort_as_half(uint16_t(top)));
      const int shift = top > 0 ? min(30, 7 + 127 - int(__float_as_uint(ftop) >> 23)) : 0, shift0 = min(shift, 15);
      const uint32_t up0 = uint32_t(15 + shift0) * 0x04000400u, up1 = uint32_t(15 + shift - shift0) * 0x04000400u;
      qs_next = __uint_as_float(uint32_t(127 - shift) << 23) * p.scale_log2;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int chunk = i0 + T * i;
        if (chunk >= 72) break;
        const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
        uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint32_t f = mul_f16x2(mul_f16x2(w[x], up0), up1);
          const uint32_t a = e4m3x2_of_f16x2(f);
          const uint32_t rest = sub_f16x2(f, e4m3x2_to_half2(a));  // exact, as is 16 times it
          hi[x >> 1] |= a << (16 * (x & 1));
          lo[x >> 1] |= e4m3x2_of_f16x2(mul_f16x2(rest, 0x4c004c00u)) << (16 * (x & 1));
        }
        // 16 chunks to a box, two to a 16-byte piece
        const int piece = (chunk & 15) >> 1;
        uint8_t* box = smem + C::kOffQ + (chunk >> 4) * C::kQBox + 8 * (chunk & 1);
#pragma unroll
        for (int term = 0; term < 2; ++term) {
          const int row = term ? row_lo : row_hi;
          uint8_t* dst = chunk < 64 ? box + row * 128 + ((piece ^ (row & 7)) << 4) : box + row * 64 + ((piece ^ ((row >> 1) & 3)) << 4);
          *reinterpret_cast<uint2*>(dst) = term ? make_uint2(lo[0], lo[1]) : make_uint2(hi[0], hi[1]);
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(&B->q_full);
    };
    float* m_run = red + 15 * HC + NH * c;  // kept once for the group's threads
    float* alpha = red + 16 * HC + NH * c;
    // 8 heads: a copy of m_run in registers (loads of one address by all lanes cost
    // shared memory four wavefronts each); 16: none to spare
    constexpr bool kCopies = NH == 8;
    float l_run[NH], mr[kCopies ? NH : 4] = {};
    // m_run of heads 4 h4 .. 4 h4 + 3
    auto m_four = [&](int h4) -> float4 {
      if constexpr (kCopies) return make_float4(mr[4 * h4], mr[4 * h4 + 1], mr[4 * h4 + 2], mr[4 * h4 + 3]);
      else return reinterpret_cast<const float4*>(m_run)[h4];
    };
    uint32_t k = 0, seg = 0;
    TileInfo t, tn;
    bool have = walk.next(t);
    int len_b = walk.len_b;
    if (have) load_q(t.b, 0);
    while (have) {
      const uint32_t buf = k & 1;
      const bool valid = st < t.valid;
      bool ok = wait_for<C::kSplitRegs>(&B->s_full[buf], (k >> 1) & 1, abort_flag);
      if (k >= 2) ok = ok && wait_for<C::kSplitRegs>(&B->pv_done[buf], ((k - 2) >> 1) & 1, abort_flag);
      tc_fence_after();
      if (t.first) qs = qs_next;
      // The weights' exponents y: the scores in log2 units less m_run.
      float y[NH];
      bool nan_row = false;  // a hidden row gave a NaN score
      auto sums = [&](float (&s)[NH]) {  // q . c, times 2^k
        float lo[NH];
        tmem_load<NH>(tmem + lane_off + C::kColS + buf * C::kNQ + NH * c, s);
        tmem_load<NH>(tmem + lane_off + C::kColS + buf * C::kNQ + HC + NH * c, lo);
#pragma unroll
        for (int h = 0; h < NH; ++h) s[h] = fmaf(lo[h], 0.0625f, s[h]);
      };
      auto mask = [&](float (&s)[NH]) {
        if (!valid) {
#pragma unroll
          for (int h = 0; h < NH; ++h) s[h] = -INFINITY;
        }
        if (kCausal && causal_tile(p, t, len_b)) {
          const int pos = t.tile * kTile + st - (len_b - p.q_len);  // against the query token's number
#pragma unroll
          for (int h = 0; h < NH; ++h)
            if (pos > (g * HC + NH * c + h) / p.heads_w) {
              nan_row |= s[h] != s[h];
              s[h] = -INFINITY;
            }
        }
      };
      // Running max: as in decode_tc.cu it only has to bound the scores, here to
      // within 2^5, so that the weights keep E5M2's range down.
      bool over = false;
      if (!t.first) {
        sums(y);
#pragma unroll
        for (int h4 = 0; h4 < NH / 4; ++h4) {
          const float4 m = m_four(h4);
          y[4 * h4] = fmaf(y[4 * h4], qs, -m.x);
          y[4 * h4 + 1] = fmaf(y[4 * h4 + 1], qs, -m.y);
          y[4 * h4 + 2] = fmaf(y[4 * h4 + 2], qs, -m.z);
          y[4 * h4 + 3] = fmaf(y[4 * h4 + 3], qs, -m.w);
        }
        mask(y);
#pragma unroll
        for (int h = 0; h < NH; ++h) over |= y[h] > kWeightBits + kRescaleThreshold;
      }
      bool rescale = false;
      if (t.first || group_any(c, over || !ok)) {
        // exactly: the scores themselves, once more
        sums(y);
#pragma unroll
        for (int h = 0; h < NH; ++h) y[h] *= qs;
        mask(y);
        float* rm = red + buf * 4 * HC + 4 * NH * c;
        {
          float tmp[NH];
#pragma unroll
          for (int h = 0; h < NH; ++h) tmp[h] = y[h];
          const float wm = warp_reduce<NH, true>(tmp, lane);
          if (lane % (32 / NH) == 0) rm[lane / (32 / NH) * 4 + q4] = wm;
        }
        if (group_any(c, !ok)) break;
        if (st < NH) {  // thread h: head h's maximum over the tile
          const float4 m4 = reinterpret_cast<const float4*>(rm)[st];
          const float mt = fmaxf(fmaxf(m4.x, m4.y), fmaxf(m4.z, m4.w)), old = m_run[st];
          float a = 1.f;
          if (t.first) {
            m_run[st] = fmaxf(mt, kEmptyRowMax) - kWeightBits;  // a row masked in the whole tile stays empty
          } else if (mt > old + (kWeightBits + kRescaleThreshold)) {
            a = exp2f(old - (mt - kWeightBits));
            m_run[st] = mt - kWeightBits;
            rescale = true;
          }
          alpha[st] = a;
        }
        rescale = group_any(c, rescale);
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          const float m = m_run[h];
          if (kCopies) mr[h % (kCopies ? NH : 4)] = m;
          y[h] -= m;
          l_run[h] = t.first ? 0.f : l_run[h] * alpha[h];
        }
      }
      tc_fence_before();
      mbar_arrive(&B->s_free[buf]);
      if (rescale) {
        // QK of this tile may have been issued before PV of the previous one:
        // wait for that PV first
        const bool ok3 = wait_for<C::kSplitRegs>(&B->pv_done[(k - 1) & 1], ((k - 1) >> 1) & 1, abort_flag);
        tc_fence_after();
        if (group_any(c, !ok3)) break;
#pragma unroll 1
        for (int i = 0; i < 12; ++i) {  // chunk i / 3, term i % 3
          float v[NH];
          const uint32_t a = tmem + lane_off + C::kColO + (i / 3) * C::kColOStep + (i % 3) * HC + NH * c;
          tmem_load<NH>(a, v);
#pragma unroll
          for (int h = 0; h < NH; ++h) v[h] *= alpha[h];
          tmem_store<NH>(a, v);
        }
        tmem_st_wait();
      }
      // weights -> P^T, three E5M2 terms of the fp16 value: the high byte rounded
      // to nearest, the same of what is left, and the rest (at most three bits)
      {
        uint32_t w[NH / 2];
#pragma unroll
        for (int h4 = 0; h4 < NH / 4; ++h4) {
          const float e0 = ex2_ftz(y[4 * h4]), e1 = ex2_ftz(y[4 * h4 + 1]);
          const float e2 = ex2_ftz(y[4 * h4 + 2]), e3 = ex2_ftz(y[4 * h4 + 3]);
          l_run[4 * h4] += e0;
          l_run[4 * h4 + 1] += e1;
          l_run[4 * h4 + 2] += e2;
          l_run[4 * h4 + 3] += e3;
          w[2 * h4] = pack_f16x2(e0, e1);
          w[2 * h4 + 1] = pack_f16x2(e2, e3);
        }
        // head n of a term is byte n % 16 of its row in core matrix n / 16
        uint8_t* pt = smem + C::kOffP + buf * C::kPBytes + (NH * c / 16) * 2048 + NH * c % 16 + (st >> 3) * 128 + (st & 7) * 16;
#pragma unroll
        for (int term = 0; term < 3; ++term) {
          uint32_t o[NH / 4];
#pragma unroll
          for (int i = 0; i < NH / 4; ++i) {
            uint32_t h[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint32_t& x2 = w[2 * i + e];
              h[e] = term < 2 ? (x2 + 0x00800080u) & 0xff00ff00u : x2;
              if (term < 2) x2 = sub_f16x2(x2, h[e]);
            }
            o[i] = __byte_perm(h[0], h[1], 0x7531);
          }
          uint8_t* dst = pt + term * (HC / 16) * 2048;
          if constexpr (NH == 16) *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
          else *reinterpret_cast<uint2*>(dst) = make_uint2(o[0], o[1]);
        }
      }
      if (kCausal && nan_row) {
        // A NaN in a hidden row would pass its weight of 0 in PV.  Rows that see it
        // have a NaN weight and sum already, so its pieces become zeros (QK of the
        // tile has read them, PV waits for this thread).  A NaN query gets here too
        // and changes nothing.
        const uint32_t slot = k % kSlots;
        uint8_t* row = smem + slot * kSlotBytes + st * 128;
        // acquires the expansion's writes (these phases have completed)
        for (int half = 0; half < 2; ++half) mbar_try_wait(&B->full[slot][half], (k / kSlots) & 1);
#pragma unroll 1
        for (int i = 0; i < 32; ++i) {  // a piece is half a block: all NaN or none
          uint4* piece = reinterpret_cast<uint4*>(row + (i >> 3) * kLatBox + 16 * (i & 7));
          if ((piece->x & 0x7f) == 0x7f) *piece = make_uint4(0, 0, 0, 0);
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive(&B->p_full[buf]);
      const bool have_next = walk.next(tn);
      if (t.last) {
        if (have_next) load_q(tn.b, seg + 1);
        const bool ok2 = wait_for<C::kSplitRegs>(&B->o_full, seg & 1, abort_flag);
        tc_fence_after();
        float* rl = red + 8 * HC + 4 * NH * c;  // [NH][4] sums
        {
          float tmp[NH];
#pragma unroll
          for (int h = 0; h < NH; ++h) tmp[h] = l_run[h];
          const float ls = warp_reduce<NH, false>(tmp, lane);
          if (lane % (32 / NH) == 0) rl[lane / (32 / NH) * 4 + q4] = ls;
        }
        if (group_any(c, !ok2)) break;
        float* rinv = red + 12 * HC + NH * c;
        float l = 0.f, il = 0.f;
        if (st < NH) {  // thread h divides for head h
          const float4 l4 = reinterpret_cast<const float4*>(rl)[st];
          l = (l4.x + l4.y) + (l4.z + l4.w);
          il = l > 0.f ? 1.f / l : l;  // 0: a row with no visible token; NaN stays
          rinv[st] = il;
        }
        group_any(c, false);
        const int row0 = g * HC + NH * c;
        float* dst = p.partial_o + (size_t(t.seg) * p.heads + row0) * kLatent + st;
#pragma unroll 1
        for (int ch = 0; ch < 4; ++ch) {
          float v[3][NH];
          tmem_load3<NH>(tmem + lane_off + C::kColO + ch * C::kColOStep + NH * c, HC, v);
#pragma unroll
          for (int h = 0; h < NH; ++h)
            if (live) dst[h * kLatent + ch * 128] = ((v[0][h] + v[1][h]) + v[2][h]) * rinv[h];
        }
        tc_fence_before();
        mbar_arrive(&B->o_free);
        if (st < NH && live) {  // thread h writes head h's lse
          p.partial_lse[size_t(t.seg) * p.heads + row0 + st] = l > 0.f ? (m_run[st] + log2f(l)) * kLn2 : lse_of_no_sum(l);
        }
        ++seg;
      }
      t = tn;
      len_b = walk.len_b;
      have = have_next;
      ++k;
    }
  }
  // ---------------------------------------------------------------- teardown
  __syncthreads();
  tc_fence_after();
  if (warp == kQkWarp) tmem_dealloc(tmem, C::kTmemCols);
}

// Registers of a thread as a block's launch gives them out.
constexpr int launch_registers(int regs) { return (regs + 7) / 8 * 8; }
static_assert(launch_registers(88) == 88 && launch_registers(89) == 96 && launch_registers(96) == 96, "by eights");

template <int HC, bool kCausal>
cudaError_t launch_fp4(const DecodeParams& p, int grid, cudaStream_t stream) {
  using C = Fp4Cfg<HC>;
  auto* kernel = decode_fp4_kernel<HC, kCausal>;
  static std::atomic<bool> attr[128];  // per device: attributes set (zero-initialised)
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 128 || !attr[dev]) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(C::kSmem));
    if (e != cudaSuccess) return e;
    if (C::kSplitRegs) {
      // setmaxnreg.inc waits, with no limit, for registers that the block was
      // launched with: a build of fewer than the roles share out is not launched
      cudaFuncAttributes a;
      e = cudaFuncGetAttributes(&a, kernel);
      if (e != cudaSuccess) return e;
      if (launch_registers(a.numRegs) != C::kRegs) return cudaErrorLaunchOutOfResources;
    }
    if (dev >= 0 && dev < 128) attr[dev] = true;
  }
  return launch_pdl(kernel, dim3(grid), dim3(C::kThreads), C::kSmem, stream, 1, p);
}

}  // namespace

cudaError_t launch_decode_fp4(const DecodeParams& p, int hc, int grid, cudaStream_t stream) {
  // 16 rows are the 16 heads of one token: no causal form
  if (hc == 16) return launch_fp4<16, false>(p, grid, stream);
  return p.q_len > 1 ? launch_fp4<32, true>(p, grid, stream) : launch_fp4<32, false>(p, grid, stream);
}

}  // namespace mla
