// cache_read.cu -- read cached rows back out of their pages: the rows of a
// packed batch, dequantised to bf16.
//
// Row r of the packed output belongs to the sequence b with cu_rows[b] <= r <
// cu_rows[b + 1] and is the cached row at position starts[b] + r - cu_rows[b].
// bf16 caches: a copy; INT8: scale * (code - zero point); FP8: scale *
// e4m3(code), each in fp32 with one rounding to bf16 ("KV Cache Optimization",
// section 3).  These are the latents that W^UK and W^UV expand to keys and
// values, so the outputs have the append's input layout: latents [n, 512] and
// rotated RoPE keys [n, 64].
//
// Bound by memory: 1,152 / 584 / 580 bytes read and 1,152 written per row.  A
// CTA resolves its rows first (one thread per row: binary search in cu_rows,
// then the page-table entry), then all threads move 16-byte source pieces with
// every load of the CTA issued before its first store.  A 1-byte piece becomes
// 32 bytes, stored at once: as two 16-byte stores, each half of its sectors,
// 129,000 INT8 rows took 40.6 us, as whole sectors 33.4 us (5.9 TB/s, 88% of
// the measured copy peak); 194,000 FP8 rows 66 and 53 us (6.4 TB/s, 94%).  32
// rows to a CTA; 16 took 36.5 us on the INT8 rows.
#include "blackwell_ptx.cuh"
#include "decode_common.cuh"
#include "params.cuh"

namespace mla {
namespace {

constexpr int kReadThreads = 288;  // a multiple of the 36 (1-byte) or 72 (bf16) source pieces of a row

// bf16 pair of two dequantised values, `lo` in the low half.
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// 16 codes -> 16 bf16 values.  (code - zero point) is exact in fp32, the
// product rounds once to fp32 and once to bf16.
template <int kCode>
__device__ __forceinline__ void dequant_codes(uint4 v, float scale, float zp, uint4& lo, uint4& hi) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float f[4];
    if constexpr (kCode == kCodeInt8) {
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = __fsub_rn(float(int8_t(w[i] >> (8 * j))), zp);
    } else {
      const float2 a = dc::unpack_f16x2(dc::e4m3x2_to_half2(w[i])), b = dc::unpack_f16x2(dc::e4m3x2_to_half2(w[i] >> 16));
      f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
    }
    o[2 * i] = pack_bf16x2(__fmul_rn(f[0], scale), __fmul_rn(f[1], scale));
    o[2 * i + 1] = pack_bf16x2(__fmul_rn(f[2], scale), __fmul_rn(f[3], scale));
  }
  lo = make_uint4(o[0], o[1], o[2], o[3]);
  hi = make_uint4(o[4], o[5], o[6], o[7]);
}

template <int kCode, int kRows>
__global__ void __launch_bounds__(kReadThreads) cache_read_kernel(CacheReadParams p) {
  constexpr bool kByte = kCode != kCodeBf16;
  constexpr int kPieces = kByte ? 36 : 72;             // 16-byte source pieces of a row
  constexpr int kPerPass = kReadThreads / kPieces;     // rows of one pass
  constexpr int kPasses = kRows / kPerPass;
  static_assert(kRows % kPerPass == 0, "whole passes");
  __shared__ long long src_row[kRows];                 // cache row, or -1: not written
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int tid = threadIdx.x;
  const long long r0 = (long long)blockIdx.x * kRows;
  if (tid < kRows) {
    const long long r = r0 + tid;
    long long row = -1;
    if (r < p.n_rows) {
      // b = (number of entries <= r) - 1
      int lo = 0, hi = p.num_seqs + 1;
      while (lo < hi) {
        const int mid = lo + ((hi - lo) >> 1);
        if (p.cu_rows[mid] <= r) lo = mid + 1; else hi = mid;
      }
      const int b = lo - 1;
      if (b >= 0 && b < p.num_seqs) {  // rows before the first and behind the last sequence stay as they are
        const int first = p.cu_rows[b];
        const long long pos = (long long)(p.starts ? p.starts[b] : 0) + r - first;
        bool ok = pos >= 0 && pos / p.page_size < p.max_pages && first >= 0;
        if (ok) {
          const int page = p.block_table[size_t(b) * p.max_pages + pos / p.page_size];
          ok = page >= 0 && page < p.num_pages;
          row = (long long)page * p.page_size + pos % p.page_size;
        }
        if (!ok) {
          row = -1;
          set_status(p.status, MLA_ERR_DEVICE_BOUNDS);
        }
      }
    }
    src_row[tid] = row;
  }
  // the whole of cu_rows, by the first CTA: non-decreasing and within n_rows
  if (blockIdx.x == 0) {
    bool bad = false;
    for (int i = tid; i < p.num_seqs; i += kReadThreads) bad |= p.cu_rows[i] > p.cu_rows[i + 1];
    if (tid == 0) bad |= p.cu_rows[0] < 0 || p.cu_rows[p.num_seqs] > p.n_rows;
    if (bad) set_status(p.status, MLA_ERR_DEVICE_BOUNDS);
  }
  __syncthreads();
  const int q = tid % kPieces, rr = tid / kPieces;
  uint4 v[kPasses];
  float scale[kByte ? kPasses : 1], zp[kByte ? kPasses : 1];
#pragma unroll
  for (int u = 0; u < kPasses; ++u) {
    const long long row = src_row[rr + u * kPerPass];
    if (row >= 0) {
      v[u] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.cache) + row * (kPieces * 16)) + q);
      if constexpr (kCode == kCodeInt8) {
        const float2 sz = __ldg(reinterpret_cast<const float2*>(p.scale_zero) + row);
        scale[u] = sz.x;
        zp[u] = sz.y;
      }
      if constexpr (kCode == kCodeE4m3) scale[u] = __ldg(p.scale_zero + row);
    }
  }
#pragma unroll
  for (int u = 0; u < kPasses; ++u) {
    const int rl = rr + u * kPerPass;
    if (src_row[rl] < 0) continue;
    const size_t r = size_t(r0) + rl;
    if constexpr (kByte) {
      uint4 lo, hi;
      dequant_codes<kCode>(v[u], scale[u], kCode == kCodeInt8 ? zp[u] : 0.f, lo, hi);
      uint4* dst = q < 32 ? reinterpret_cast<uint4*>(p.c_kv + r * kLatent) + 2 * q
                          : reinterpret_cast<uint4*>(p.k_pe + r * kRope) + 2 * (q - 32);
      ptx::st_global_32(dst, lo, hi);
    } else {
      uint4* dst = q < 64 ? reinterpret_cast<uint4*>(p.c_kv + r * kLatent) + q
                          : reinterpret_cast<uint4*>(p.k_pe + r * kRope) + (q - 64);
      *dst = v[u];
    }
  }
}

template <int kCode>
cudaError_t launch_read(const CacheReadParams& p, cudaStream_t stream) {
  // few rows: eight to a CTA, so that they spread over the SMs
  if (p.n_rows <= 8 * 512)
    return launch_pdl(cache_read_kernel<kCode, 8>, dim3((unsigned(p.n_rows) + 7) / 8), dim3(kReadThreads), 0, stream, 1, p);
  return launch_pdl(cache_read_kernel<kCode, 32>, dim3((unsigned(p.n_rows) + 31) / 32), dim3(kReadThreads), 0, stream, 1, p);
}

}  // namespace

cudaError_t launch_cache_read(const CacheReadParams& p, int code, cudaStream_t stream) {
  return code == kCodeInt8   ? launch_read<kCodeInt8>(p, stream)
         : code == kCodeE4m3 ? launch_read<kCodeE4m3>(p, stream)
                             : launch_read<kCodeBf16>(p, stream);
}

}  // namespace mla
