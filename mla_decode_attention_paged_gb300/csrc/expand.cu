// expand.cu -- latents to per-head keys and values, the un-absorbed form:
// K_t = W^UK c_t and V_t = W^UV c_t ("Beyond the Attention Bottleneck",
// "Down-Projection and Up-Projection Mechanics").
//
// Two products of the same latents, [n x 512] x [512 x H*128] each: a CTA
// computes 128 rows x one head of one of them, [128 x 512] x [512 x 128], on
// the tensor cores (both operands K-major, TMA into 128-byte-swizzled shared
// memory in blocks of 64 latent dims, fp32 accumulation in tensor memory) and
// rounds once to bf16.
#include <atomic>

#include "blackwell_ptx.cuh"
#include "decode_common.cuh"
#include "params.cuh"

namespace mla {
namespace {

using namespace ptx;

constexpr int kExpThreads = 128;
constexpr int kExpStages = 4;
constexpr uint32_t kExpBox = 128 * 128;               // [128 rows x 64 latent dims] bf16, SW128
constexpr uint32_t kExpStage = 2 * kExpBox;           // rows, weights
constexpr uint32_t kExpOffMisc = kExpStages * kExpStage;
constexpr uint32_t kExpSmem = kExpOffMisc + 256 + 1024;
constexpr uint64_t kExpWaitNs = 2000000000ull;
constexpr int kKBlocks = kLatent / 64;

struct ExpandBarriers {
  uint64_t full[kExpStages], empty[kExpStages], done;
  uint32_t tmem_base;
  int abort;
};

__global__ void __launch_bounds__(kExpThreads) expand_kernel(const __grid_constant__ CUtensorMap map_c,
                                                             const __grid_constant__ CUtensorMap map_uk,
                                                             const __grid_constant__ CUtensorMap map_uv,
                                                             ExpandParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  ExpandBarriers* B = reinterpret_cast<ExpandBarriers*>(smem + kExpOffMisc);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kExpStages; ++i) {
      mbar_init(&B->full[i], 1);
      mbar_init(&B->empty[i], 1);
    }
    mbar_init(&B->done, 1);
    B->abort = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&B->tmem_base, 128);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = B->tmem_base, sbase = smem_u32(smem);
  griddep_wait();
  griddep_launch_dependents();
  const int unit = blockIdx.x % (2 * p.heads), m0 = (blockIdx.x / (2 * p.heads)) * 128;
  const int head = unit % p.heads;
  const bool is_v = unit >= p.heads;
  bool ok = true;
  if (tid == 0) {
    const CUtensorMap* map_w = is_v ? &map_uv : &map_uk;
    auto load = [&](int kb) {
      const int s = kb % kExpStages;
      mbar_arrive_expect_tx(&B->full[s], kExpStage);
      tma_load_2d(smem + s * kExpStage, &map_c, 64 * kb, m0, &B->full[s]);
      tma_load_2d(smem + s * kExpStage + kExpBox, map_w, 64 * kb, head * 128, &B->full[s]);
    };
    constexpr uint32_t idesc = idesc_bf16_f32(128, 128, false, false);
    constexpr uint64_t kDesc = smem_desc(0, 16, 1024, kSwizzle128B);
    for (int kb = 0; kb < kExpStages; ++kb) load(kb);
    for (int kb = 0; kb < kKBlocks && ok; ++kb) {
      const int s = kb % kExpStages;
      ok = mbar_wait(&B->full[s], (kb / kExpStages) & 1, &B->abort, kExpWaitNs);
      if (!ok) break;
      tc_fence_after();
      const uint32_t a = sbase + s * kExpStage;
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        mma_bf16(tmem, kDesc | desc_addr(a + 32 * kk), kDesc | desc_addr(a + kExpBox + 32 * kk), idesc, kb + kk > 0);
      mma_commit(&B->empty[s]);
      if (kb + kExpStages < kKBlocks) {
        ok = mbar_wait(&B->empty[s], (kb / kExpStages) & 1, &B->abort, kExpWaitNs);
        if (ok) load(kb + kExpStages);
      }
    }
    if (!ok) B->abort = 1;
    mma_commit(&B->done);
  }
  __syncwarp();
  ok = mbar_wait(&B->done, 0, &B->abort, kExpWaitNs) && ok;
  tc_fence_after();
  __syncthreads();
  if (!B->abort) {
    const int r = m0 + 32 * warp + lane;
    uint4* dst = reinterpret_cast<uint4*>((is_v ? p.v : p.k_nope) + (size_t(r) * p.heads + head) * 128);
#pragma unroll 1
    for (int c = 0; c < 128; c += 32) {
      uint32_t v[32];
      tmem_ld32(tmem + (uint32_t(32 * warp) << 16) + c, v);
      if (r < p.n_rows) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 b =
                __floats2bfloat162_rn(__uint_as_float(v[8 * i + 2 * j]), __uint_as_float(v[8 * i + 2 * j + 1]));
            o[j] = *reinterpret_cast<const uint32_t*>(&b);
          }
          dst[c / 8 + i] = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
    }
  } else if (tid == 0) {
    set_status(p.status, MLA_ERR_DEVICE_TIMEOUT);
    const uint64_t t0 = global_timer_ns();  // copies already issued land before the shared memory is released
    while (global_timer_ns() - t0 < 20000) {
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 128);
}

}  // namespace

cudaError_t launch_expand(const ExpandParams& p, cudaStream_t stream) {
  CUtensorMap mc, mk, mv;
  if (!dc::make_map_2d(&mc, p.c_kv, 2, kLatent, p.n_rows, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !dc::make_map_2d(&mk, p.W_UK, 2, kLatent, uint64_t(p.heads) * 128, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !dc::make_map_2d(&mv, p.W_UV, 2, kLatent, uint64_t(p.heads) * 128, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  static std::atomic<bool> attr[128];  // per device: attributes set (zero-initialised)
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 128 || !attr[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(expand_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kExpSmem));
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 128) attr[dev] = true;
  }
  const unsigned grid = unsigned((p.n_rows + 127) / 128) * 2u * unsigned(p.heads);
  return launch_pdl(expand_kernel, dim3(grid), dim3(kExpThreads), kExpSmem, stream, 1, mc, mk, mv, p);
}

}  // namespace mla
