// expand.cu -- latents to per-head keys and values, the un-absorbed form:
// K_t = W^UK c_t and V_t = W^UV c_t ("Beyond the Attention Bottleneck",
// "Down-Projection and Up-Projection Mechanics").
//
// Two products of the same latents, [n x 512] x [512 x H*128] each, 262,144
// multiply-adds per row and head: the tensor cores bound it from some hundred
// rows on, and with only 512 latent dims to a product the operands' way from
// L2 is next.  So a pair of CTAs (one MMA over both SMs, M = 256 rows, N = 256
// columns = two heads) keeps one operand's [256 x 512] in shared memory, 128 KB
// in each CTA, and streams the other in 16 KB boxes of 128 rows x 64 latent dims
// to each CTA: 256 FLOP to a byte.  It walks a contiguous range of the (resident
// block, streamed block) list.  The smaller operand is streamed, as it is read
// once per resident block and should stay in L2: weights (4 MB at 16 heads)
// where there are more rows than weight rows (256 to a head), else latents.
// 34,816 rows at 16 heads: 110 us with the weights streamed, 120 with the
// latents; 5,003 rows at 128 heads: 137 and 128 us.  Accumulators (256 columns)
// alternate between the two halves of tensor memory, so that rounding and
// storing a tile overlaps the next tile's MMAs; each thread stores its row in
// whole 32-byte sectors.  What bounds both sizes now is products and outputs
// together: without the stores they take 72 and 82 us (1.9 and 2.0 PFLOP/s),
// without the streamed copies 92 and 106, and filling as many bytes takes 74 and
// 84 us.
//
// Warps: 0 TMA producer, 1 tensor memory and (in the leading CTA) MMA issue,
// 2-5 epilogue.  Every wait is bounded: on timeout the CTA records
// MLA_ERR_DEVICE_TIMEOUT and the pair ends together: once neither CTA issues any
// more, their MMAs and copies in flight are waited for on their own barriers
// (half a second at most), then tensor memory is freed.
#include <atomic>

#include "blackwell_ptx.cuh"
#include "decode_common.cuh"
#include "params.cuh"

namespace mla {
namespace {

using namespace ptx;

constexpr int kExpThreads = 192;
constexpr int kStages = 6;
constexpr int kKBlocks = kLatent / 64;
constexpr uint32_t kBox = 128 * 128;                  // [128 rows x 64 columns] bf16, SW128: 16 KB
constexpr uint32_t kOffRing = kKBlocks * kBox;        // after the resident operand
constexpr uint32_t kOffMisc = kOffRing + kStages * kBox;
constexpr uint32_t kSmem = kOffMisc + 256 + 1024;
constexpr uint64_t kWaitNs = 2000000000ull;           // 2 s
constexpr uint64_t kDrainNs = 500000000ull;           // 0.5 s
static_assert(kSmem <= 232448, "dynamic shared memory of one CTA");

struct ExpandBarriers {
  uint64_t full[kStages];        // leading CTA: both CTAs' streamed boxes landed
  uint64_t empty[kStages];       // each CTA: read by their MMAs
  uint64_t res_full, res_empty;  // resident operand landed (leading CTA) / read by its last MMA (each CTA)
  uint64_t acc_full[2];       // each CTA: accumulator complete
  uint64_t acc_empty[2];      // leading CTA: read by both CTAs' epilogues
  uint64_t drain;
  uint32_t tmem_base;
  int abort;                     // this CTA gave up
  int pair_abort;                // a CTA of the pair did
  uint32_t boxes[2], blocks[2];  // leading CTA: streamed boxes and resident blocks that each producer issued copies of
};
static_assert(sizeof(ExpandBarriers) <= 256, "shared memory behind the ring");

__device__ __forceinline__ void fail(ExpandBarriers* B, int* status) {
  B->abort = 1;
  set_status(status, MLA_ERR_DEVICE_TIMEOUT);
}

// ----- two-CTA forms ------------------------------------------------------------
__device__ __forceinline__ void tmem_alloc2(uint32_t* dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tmem_relinquish2() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc2(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// D (+)= A B over both CTAs of the pair: each CTA's shared memory holds its 128
// rows of A and its half of B's rows, its tensor memory its 128 rows of D.
__device__ __forceinline__ void mma2_bf16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives on the barrier at this offset in both CTAs when this thread's MMAs are complete.
__device__ __forceinline__ void mma2_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(uint16_t(3))
      : "memory");
}
// Box at (x, y) into this CTA's shared memory, its bytes counted on a barrier
// of either CTA of the pair (cluster address).
__device__ __forceinline__ void tma2_load_2d(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void store_cluster(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
// kRowsResident: latents resident, weights streamed; else the other way round.
template <bool kRowsResident>
__global__ void __launch_bounds__(kExpThreads, 1)
    expand_kernel(const __grid_constant__ CUtensorMap map_c, const __grid_constant__ CUtensorMap map_uk,
                  const __grid_constant__ CUtensorMap map_uv, ExpandParams p) {
  extern __shared__ uint8_t smem_raw[];
  // the same offset in both CTAs: barriers are addressed across the pair
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  ExpandBarriers* B = reinterpret_cast<ExpandBarriers*>(smem + kOffMisc);
  const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int rank = int(cluster_ctarank());
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&B->full[i], 1);
      mbar_init(&B->empty[i], 1);
    }
    mbar_init(&B->res_full, 1);
    mbar_init(&B->res_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B->acc_full[i], 1);
      mbar_init(&B->acc_empty[i], 8);  // one lane of each epilogue warp of both CTAs
    }
    mbar_init(&B->drain, 1);
    B->abort = B->pair_abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc2(&B->tmem_base, 512);
    tmem_relinquish2();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = B->tmem_base, sbase = smem_u32(smem);
  griddep_wait();
  griddep_launch_dependents();
  const volatile int* abort_flag = &B->abort;
  // units (resident block, streamed block), the resident ones outermost; column
  // blocks are W^UK's, then W^UV's
  const int blocks = p.heads, tiles = (p.n_rows + 255) / 256, inner = kRowsResident ? blocks : tiles;
  const int P = gridDim.x / 2, pair = blockIdx.x / 2;
  const long long total = (long long)tiles * blocks;
  const int u0 = int(total * pair / P), u1 = int(total * (pair + 1) / P);
  const uint32_t row_box = kRowsResident ? 0 : kOffRing, col_box = kRowsResident ? kOffRing : 0;

  if (warp == 0 && lane == 0) {
    // ------------------------------------------------------------ TMA producer
    bool ok = true;
    uint32_t k = 0, nr = 0;
    const uint32_t res_full = mapa_shared(smem_u32(&B->res_full), 0);
    // box i (64 latent dims) of this CTA's half of row tile / column block x
    auto load = [&](bool rows, int x, int i, uint8_t* dst, uint32_t bar) {
      const bool is_v = !rows && x >= blocks / 2;
      tma2_load_2d(dst, rows ? &map_c : is_v ? &map_uv : &map_uk, 64 * i, (is_v ? x - blocks / 2 : x) * 256 + 128 * rank,
                   bar);
    };
    int resident = -1;
    for (int u = u0; u < u1 && ok; ++u) {
      if (u / inner != resident) {
        if (nr > 0 && !(ok = mbar_wait(&B->res_empty, (nr - 1) & 1, abort_flag, kWaitNs))) break;
        ++nr;
        resident = u / inner;
        if (rank == 0) mbar_arrive_expect_tx(&B->res_full, 2 * kKBlocks * kBox);
        for (int i = 0; i < kKBlocks; ++i) load(kRowsResident, resident, i, smem + i * kBox, res_full);
      }
      for (int i = 0; i < kKBlocks; ++i, ++k) {
        const uint32_t s = k % kStages;
        if (k >= kStages && !(ok = mbar_wait(&B->empty[s], ((k / kStages) - 1) & 1, abort_flag, kWaitNs))) break;
        if (rank == 0) mbar_arrive_expect_tx(&B->full[s], 2 * kBox + (p.inject_wait_timeout && k == 0 ? 16 : 0));
        load(!kRowsResident, u % inner, i, smem + kOffRing + s * kBox, mapa_shared(smem_u32(&B->full[s]), 0));
      }
    }
    if (!ok) fail(B, p.status);
    store_cluster(mapa_shared(smem_u32(&B->boxes[rank]), 0), k);
    store_cluster(mapa_shared(smem_u32(&B->blocks[rank]), 0), nr);
  } else if (warp == 1 && rank == 0) {
    // ------------------------------------------------------------ MMA issue
    constexpr uint32_t idesc = idesc_bf16_f32(256, 256, false, false);
    constexpr uint64_t kDesc = smem_desc(0, 16, 1024, kSwizzle128B);
    const uint64_t a0 = kDesc | desc_addr(sbase + row_box), b0 = kDesc | desc_addr(sbase + col_box);
    const bool leader = elect_one();
    bool ok = true;  // of all lanes: they leave together
    uint32_t k = 0, nr = 0, t = 0;
    int resident = -1;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return ok = __all_sync(0xffffffffu, mbar_wait_cluster(bar, parity, abort_flag, kWaitNs));
    };
    for (int u = u0; u < u1 && ok; ++u, ++t) {
      if (u / inner != resident) {
        if (!wait(&B->res_full, nr & 1)) break;
        ++nr;
        resident = u / inner;
      }
      const uint32_t d = tmem + 256 * (t & 1);
      if (t >= 2 && !wait(&B->acc_empty[t & 1], ((t >> 1) - 1) & 1)) break;
      for (int i = 0; i < kKBlocks; ++i, ++k) {
        const uint32_t s = k % kStages;
        if (!wait(&B->full[s], (k / kStages) & 1)) break;
        tc_fence_after();
        if (leader) {
          const uint64_t a = a0 + (kRowsResident ? i : s) * (kBox >> 4), b = b0 + (kRowsResident ? s : i) * (kBox >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) mma2_bf16(d, a + 2 * kk, b + 2 * kk, idesc, kk > 0 ? 1 : i);
          mma2_commit(&B->empty[s]);
        }
        __syncwarp();
      }
      if (ok && leader) {
        mma2_commit(&B->acc_full[t & 1]);
        if (u + 1 == u1 || (u + 1) / inner != resident) mma2_commit(&B->res_empty);
      }
      __syncwarp();
    }
    if (leader) {
      if (!ok) fail(B, p.status);
      mma2_commit(&B->drain);  // every MMA issued completes before teardown
    }
    __syncwarp();
  } else if (warp >= 2) {
    // ------------------------------------------------------------ epilogue
    // Tensor memory lane = row of this CTA's 128; a thread stores its row's 512
    // contiguous bytes (two heads) as whole 32-byte sectors.
    const int q4 = warp & 3, r = 32 * q4 + lane;
    uint32_t t = 0;
    for (int u = u0; u < u1; ++u, ++t) {
      const int cb = kRowsResident ? u % inner : u / inner;
      const int row = (kRowsResident ? u / inner : u % inner) * 256 + 128 * rank + r;
      const bool is_v = cb >= blocks / 2;
      const int head = (is_v ? cb - blocks / 2 : cb) * 2;
      __nv_bfloat16* dst = (is_v ? p.v : p.k_nope) + (size_t(row) * p.heads + head) * 128;
      const bool ok = mbar_wait_cluster(&B->acc_full[t & 1], (t >> 1) & 1, abort_flag, kWaitNs);
      if (!__all_sync(0xffffffffu, ok)) {
        fail(B, p.status);
        break;
      }
      tc_fence_after();
      const uint32_t acc = tmem + (uint32_t(32 * q4) << 16) + 256 * (t & 1);
#pragma unroll 1
      for (int c = 0; c < 256; c += 64) {
        uint32_t v[2][32];
        tmem_ld32_async(acc + c, v[0]);
        tmem_ld32_async(acc + c + 32, v[1]);
        tmem_ld_wait();
        tie(v[0]);
        tie(v[1]);
        if (c == 192) {  // the accumulator is read
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_cluster(mapa_shared(smem_u32(&B->acc_empty[t & 1]), 0));
        }
        if (row < p.n_rows) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const uint32_t* x = &v[i >> 1][16 * (i & 1) + 2 * e];
              const __nv_bfloat162 y = __floats2bfloat162_rn(__uint_as_float(x[0]), __uint_as_float(x[1]));
              w[e] = *reinterpret_cast<const uint32_t*>(&y);
            }
            st_global_32(dst + c + 16 * i, make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7]));
          }
        }
      }
    }
  }
  // ---------------------------------------------------------------- teardown
  __syncthreads();
  if (warp == 1) {  // both CTAs: the commits arrive in both
    if (!mbar_wait(&B->drain, 0, abort_flag, kWaitNs)) fail(B, p.status);
    __syncwarp();
    if (lane < 2 && B->abort) store_cluster(mapa_shared(smem_u32(&B->pair_abort), lane), 1);
    __syncwarp();
  }
  tc_fence_before();
  cluster_sync();  // the peer issues no more copies, MMAs and arrivals into this CTA; without an abort all are done
  tc_fence_after();
  if (B->pair_abort) {
    if (threadIdx.x == 0) {
      const uint64_t end = global_timer_ns() + kDrainNs;
      mbar_wait_until(&B->drain, 0, end);
      if (rank == 0) {  // the last phase of each barrier that either CTA's copies count on; not to be met where only one issued them
        for (uint32_t s = 0; s < kStages; ++s) {
          const uint32_t k = max(B->boxes[0], B->boxes[1]), phases = (k + kStages - 1 - s) / kStages;
          if (phases > 0) mbar_wait_until(&B->full[s], (phases - 1) & 1, end);
        }
        const uint32_t blocks = max(B->blocks[0], B->blocks[1]);
        if (blocks > 0) mbar_wait_until(&B->res_full, (blocks - 1) & 1, end);
      }
    }
    __syncwarp();
    cluster_sync();
  }
  if (warp == 1) tmem_dealloc2(tmem, 512);
}

}  // namespace

cudaError_t launch_expand(const ExpandParams& p, cudaStream_t stream) {
  CUtensorMap mc, muk, muv;
  const uint64_t cols = uint64_t(p.heads) * 128;
  if (!dc::make_map_2d(&mc, p.c_kv, 2, kLatent, p.n_rows, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !dc::make_map_2d(&muk, p.W_UK, 2, kLatent, cols, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !dc::make_map_2d(&muv, p.W_UV, 2, kLatent, cols, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  static std::atomic<bool> attr[128];  // per device: attributes set (zero-initialised)
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 128 || !attr[dev]) {
    for (auto* k : {expand_kernel<false>, expand_kernel<true>}) {
      const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmem));
      if (e != cudaSuccess) return e;
    }
    if (dev >= 0 && dev < 128) attr[dev] = true;
  }
  const long long units = (long long)((p.n_rows + 255) / 256) * p.heads, pairs = p.sm_count / 2;
  // columns: 256 to a head (k_nope and v)
  auto* kernel = p.n_rows > 256ll * p.heads ? expand_kernel<true> : expand_kernel<false>;
  return launch_pdl(kernel, dim3(unsigned(2 * (units < pairs ? units : pairs))), dim3(kExpThreads), kSmem, stream,
                    2, mc, muk, muv, p);
}

}  // namespace mla
