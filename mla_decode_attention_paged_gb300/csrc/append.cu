// append.cu -- write new tokens into the paged latent cache.
//
// "The Architecture of Memory", decode phase: the new token's key/value state
// is appended to the cache; in MLA that state is one 576-wide row, the latent
// c_t plus the decoupled RoPE key ("Beyond the Attention Bottleneck", "The RoPE
// Compatibility Problem": only the positional key carries RoPE, rotated here
// once at its position).  Pages are found through the page table
// ("PagedAttention: Virtual Memory for LLMs").  1-byte caches quantise the
// row per token ("KV Cache Optimization", section 3; "The Architecture of
// Memory", KIVI section): INT8 with an asymmetric min/max scale and zero
// point, FP8 (E4M3) with one scale that maps the row's largest magnitude to
// 448, the format's largest finite value, and FP4 (E2M1) with a power-of-two
// scale for every 32 values, inside the row.
#include "blackwell_ptx.cuh"
#include "params.cuh"

namespace mla {

// Two fp32 values to E4M3 codes (round to nearest even, saturating to
// +-448), first value in the low byte.
__device__ __forceinline__ uint32_t e4m3x2_rn_sat(float first, float second) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(second), "f"(first));
  return r;
}

// ----- FP4 rows ------------------------------------------------------------------
// A code is a quarter of its block's largest value away from the next, so a
// rotated value that lands on the other side of its bf16 rounding can change by
// that much.  The rotation of FP4 rows is therefore exact to about 2^-32: the
// angle as a 64-bit fraction of a turn (pos times the frequency, modulo 2^64:
// two integer multiply-adds, where fp64 takes 64 times the issue slots of fp32
// on this part), sine and cosine as sums of two fp32 values, and one rounding
// to bf16.  Against the fp64 rotation about one value in 10^6 differs (fp32
// sine and cosine: one in 10^4).

// The product a * b as a rounded value and its rounding error.
__device__ __forceinline__ float mul_err(float a, float b, float& err) {
  const float p = __fmul_rn(a, b);
  err = __fmaf_rn(a, b, -p);
  return p;
}
// hi + lo = a + b, for |a| >= |b| or a = 0.
__device__ __forceinline__ float add_err(float a, float b, float& err) {
  const float s = __fadd_rn(a, b);
  err = __fadd_rn(b, -__fadd_rn(s, -a));
  return s;
}

// Sine and cosine of `phase` / 2^64 turns, each as hi + lo.  The phase goes to
// the nearest quarter turn; the remainder x, |x| <= pi / 4, through the Taylor
// series with the leading terms in two floats (the fp32 terms behind them are
// below 0.006 of the result).
__device__ __forceinline__ void sincos_turns(uint64_t phase, float& sh, float& sl, float& ch, float& cl) {
  const uint32_t quarter = uint32_t((phase + (1ull << 61)) >> 62);  // 0 .. 4, modulo 4 below
  const int64_t r = int64_t(phase - (uint64_t(quarter) << 62));     // in [-2^61, 2^61)
  const float a = float(int32_t(r >> 38)), b = float(int32_t((r >> 14) & 0xffffff));
  // x = a 2 pi 2^-26 + b 2 pi 2^-50, the first constant as two floats
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  constexpr float kC1 = float(kTwoPi / (1 << 26)), kC1l = float(kTwoPi / (1 << 26) - double(kC1));
  constexpr float kC2 = float(kTwoPi / (1 << 26) / (1 << 24));
  float xl, e;
  const float p = mul_err(a, kC1, e);
  const float xh = add_err(p, __fmaf_rn(b, kC2, __fmaf_rn(a, kC1l, e)), xl);
  // z = x^2, w = x^3, q = x^4
  float zl, wl, ql;
  const float zh = mul_err(xh, xh, zl);
  zl = __fmaf_rn(2.f * xh, xl, zl);
  const float wh = mul_err(zh, xh, wl);
  wl = __fmaf_rn(zh, xl, __fmaf_rn(zl, xh, wl));
  const float qh = mul_err(zh, zh, ql);
  ql = __fmaf_rn(2.f * zh, zl, ql);
  // sin x = x + x^3 (-1/6 + z/120 - z^2/5040 + z^3/362880 - z^4/39916800)
  constexpr float k6 = float(-1.0 / 6), k6l = float(-1.0 / 6 - double(k6));
  const float ts = zh * __fmaf_rn(zh, __fmaf_rn(zh, __fmaf_rn(zh, -1.f / 39916800.f, 1.f / 362880.f), -1.f / 5040.f),
                                  1.f / 120.f);
  float fl, pl;
  const float fs = add_err(k6, ts, fl);
  fl = __fadd_rn(fl, k6l);
  const float ps = mul_err(wh, fs, pl);
  pl = __fmaf_rn(wh, fl, __fmaf_rn(wl, fs, pl));
  float s_lo;
  const float s_hi = add_err(xh, ps, s_lo);
  s_lo = __fadd_rn(s_lo, __fadd_rn(pl, xl));
  // cos x = 1 - z/2 + x^4 (1/24 - z/720 + z^2/40320 - z^3/3628800 + z^4/479001600)
  constexpr float k24 = float(1.0 / 24), k24l = float(1.0 / 24 - double(k24));
  const float tc = zh * __fmaf_rn(zh, __fmaf_rn(zh, __fmaf_rn(zh, 1.f / 479001600.f, -1.f / 3628800.f), 1.f / 40320.f),
                                  -1.f / 720.f);
  const float fc = add_err(k24, tc, fl);
  fl = __fadd_rn(fl, k24l);
  const float pc = mul_err(qh, fc, pl);
  pl = __fmaf_rn(qh, fl, __fmaf_rn(ql, fc, pl));
  float h_lo, c_lo;
  const float h_hi = add_err(1.f, -0.5f * zh, h_lo);
  const float c_hi = add_err(h_hi, pc, c_lo);
  c_lo = __fadd_rn(c_lo, __fadd_rn(pl, __fmaf_rn(-0.5f, zl, h_lo)));
  const bool swap = quarter & 1, neg_s = quarter & 2, neg_c = (quarter + 1) & 2;
  sh = swap ? c_hi : s_hi;
  sl = swap ? c_lo : s_lo;
  ch = swap ? s_hi : c_hi;
  cl = swap ? s_lo : c_lo;
  if (neg_s) { sh = -sh; sl = -sl; }
  if (neg_c) { ch = -ch; cl = -cl; }
}

// x a + y b rounded once to bf16, for bf16 x and y and two-float a and b.
__device__ __forceinline__ __nv_bfloat16 dot2_bf16(float x, float ah, float al, float y, float bh, float bl) {
  float ep, eq;
  const float p = mul_err(x, ah, ep), q = mul_err(y, bh, eq);
  // the sum of p and q and its error, whichever is larger
  const float s = __fadd_rn(p, q), t = __fadd_rn(s, -p);
  const float es = __fadd_rn(__fadd_rn(p, -__fadd_rn(s, -t)), __fadd_rn(q, -t));
  const float low = __fadd_rn(es, __fadd_rn(__fmaf_rn(x, al, ep), __fmaf_rn(y, bl, eq)));
  const float v = __fadd_rn(s, low), rest = __fadd_rn(low, -__fadd_rn(v, -s));
  // where the fp32 sum sits on the border between two bf16 values, its own rounding error decides
  uint32_t bits = __float_as_uint(v);
  if ((bits & 0xffff) == 0x8000 && rest != 0.f) bits += (rest > 0.f) == (v > 0.f) ? 1 : -1;
  return __float2bfloat16_rn(__uint_as_float(bits));
}

// The larger of two packed pairs of 16-bit magnitudes, each half by itself.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }

// The scale byte of a block whose largest magnitude has these bf16 bits: the
// smallest power of two s with largest <= 6 s = 1.5 * 2^2 s, at least 2^-127;
// 255 (NaN) where the block holds an infinity or a NaN.
__device__ __forceinline__ uint32_t fp4_scale_byte(uint32_t top) {
  if (top >= 0x7f80) return 255;
  const int b = int(top >> 7) - 2 + ((top & 0x7f) > 0x40);
  return b > 0 ? b : 0;
}
// 1 / scale (0 for 255: every code of such a block is 0).
__device__ __forceinline__ float fp4_inv_scale(uint32_t byte) {
  return byte == 255 ? 0.f : __uint_as_float((254 - byte) << 23);
}
// Eight fp32 values to E2M1 codes (nearest, ties to even), value i in bits 4i .. 4i + 3.
__device__ __forceinline__ uint32_t e2m1x8_rn_sat(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}
// A code word from eight bf16 values (four pairs) and 1 / scale: magnitudes in
// the low three bits of nibble i, the signs of values 0 .. 3 in bits 7, 15, 23
// and 31, those of values 4 .. 7 in bits 3, 11, 19 and 27 -- so that a byte
// permutation with the word's own nibbles as selectors expands four codes at
// once, and one mask more gives them their signs.
__device__ __forceinline__ uint32_t fp4_word(const uint32_t (&x)[4], float inv) {
  float v[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float((x[j] & 0x7fff) << 16) * inv;
    v[2 * j + 1] = __uint_as_float(x[j] & 0x7fff0000) * inv;
  }
  const uint32_t lo = __byte_perm(x[0], x[1], 0x7531) & 0x80808080u, hi = __byte_perm(x[2], x[3], 0x7531) & 0x80808080u;
  return e2m1x8_rn_sat(v) | lo | (hi >> 4);
}

// Quantises and stores one row: lane l has latents [16l, 16l + 16) and the
// rotated pair l of the RoPE key.
__device__ __forceinline__ void store_fp4_row(uint8_t* dst, const uint4& c0, const uint4& c1, uint32_t pair, int lane) {
  const uint32_t x0[4] = {c0.x, c0.y, c0.z, c0.w}, x1[4] = {c1.x, c1.y, c1.z, c1.w};
  uint32_t top2 = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) top2 = max_u16x2(top2, max_u16x2(x0[j] & 0x7fff7fffu, x1[j] & 0x7fff7fffu));
  uint32_t top = max(top2 & 0xffff, top2 >> 16);
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));  // the block's other half
  const uint32_t scale = fp4_scale_byte(top);
  const float inv = fp4_inv_scale(scale);
  uint32_t w0 = fp4_word(x0, inv), w1 = fp4_word(x1, inv);
  if (scale == 255) w0 = w1 = 0;
  reinterpret_cast<uint2*>(dst)[lane] = make_uint2(w0, w1);
  // RoPE key: blocks 16 (lanes 0-15) and 17 (lanes 16-31); four lanes share a word
  uint32_t rtop = max(pair & 0x7fff, (pair >> 16) & 0x7fff);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) rtop = max(rtop, __shfl_xor_sync(0xffffffffu, rtop, o));
  const uint32_t rscale = fp4_scale_byte(rtop);
  const int g = lane & 3;
  // the lane's pair is values 2g and 2g + 1 of the word
  const uint32_t xr[4] = {g == 0 ? pair : 0, g == 1 ? pair : 0, g == 2 ? pair : 0, g == 3 ? pair : 0};
  uint32_t wr = rscale == 255 ? 0 : fp4_word(xr, fp4_inv_scale(rscale));
  wr |= __shfl_xor_sync(0xffffffffu, wr, 1);
  wr |= __shfl_xor_sync(0xffffffffu, wr, 2);
  if (g == 0) reinterpret_cast<uint32_t*>(dst + 256)[lane >> 2] = wr;
  // the scale bytes: lanes 8q, 8q + 2, 8q + 4 and 8q + 6 have those of word q
  uint32_t sw = scale << (8 * ((lane >> 1) & 3));
  sw |= __shfl_xor_sync(0xffffffffu, sw, 2);
  sw |= __shfl_xor_sync(0xffffffffu, sw, 4);
  const uint32_t s1 = __shfl_sync(0xffffffffu, sw, 8), s2 = __shfl_sync(0xffffffffu, sw, 16),
                 s3 = __shfl_sync(0xffffffffu, sw, 24), r17 = __shfl_sync(0xffffffffu, rscale, 16);
  const uint32_t r16 = __shfl_sync(0xffffffffu, rscale, 0);
  if (lane == 0) reinterpret_cast<uint4*>(dst + kFp4Scales)[0] = make_uint4(sw, s1, s2, s3);
  if (lane == 1) reinterpret_cast<uint4*>(dst + kFp4Scales)[1] = make_uint4(r16 | (r17 << 8), 0, 0, 0);
}

// One warp per token.  Lane l owns latent values [16l, 16l + 16) and RoPE pair l.
template <int kCode>
__global__ void __launch_bounds__(256) append_kernel(AppendParams p) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int i = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (i >= p.n_tokens) return;
  const int b = p.chunk > 0 ? i / p.chunk : p.seq_ids[i];
  // 64-bit: a length near the int32 limits must not wrap into a valid position
  const long long pos64 = p.chunk > 0 ? (long long)p.seq_lens[b] - p.chunk + i % p.chunk : p.positions[i];
  bool ok = b >= 0 && b < p.num_seqs && pos64 >= 0 && pos64 / p.page_size < p.max_pages;
  const int pos = int(pos64);  // in [0, max_pages * P) once ok
  int page = -1;
  if (ok) {
    page = p.block_table[size_t(b) * p.max_pages + pos / p.page_size];
    ok = page >= 0 && page < p.num_pages;
  }
  if (!ok) {
    if (lane == 0) set_status(p.status, MLA_ERR_DEVICE_BOUNDS);
    return;
  }
  const size_t row = size_t(page) * p.page_size + pos % p.page_size;

  // latent part: 16 bf16 per lane, two 16-byte loads
  const uint4* src = reinterpret_cast<const uint4*>(p.c_kv + size_t(i) * kLatent) + 2 * lane;
  uint4 c0 = src[0], c1 = src[1];

  // RoPE pair `lane`: angle = pos * theta^(-2 lane / 64) in fp64 (up to
  // ~2^31 rad), reduced modulo 2 pi in fp64 to [-pi, pi]; sine, cosine and
  // the rotation then in fp32 ahead of the one rounding to bf16.  A full
  // fp64 sincos per lane kept the few SMs an append runs on busy for
  // microseconds (the fp64 units are a small fraction of this part's), and
  // the reduced fp32 result stays far inside the bf16 rounding.
  const __nv_bfloat162 kp = reinterpret_cast<const __nv_bfloat162*>(p.k_pe + size_t(i) * kRope)[lane];
  __nv_bfloat162 kr = kp;
  if constexpr (kCode == kCodeE2m1) {
    if (p.rope_theta > 0.0) {
      float sh, sl, ch, cl;
      sincos_turns(uint64_t(pos) * p.turn[lane], sh, sl, ch, cl);
      const float x0 = __low2float(kp), x1 = __high2float(kp);
      kr.x = dot2_bf16(x0, ch, cl, -x1, sh, sl);
      kr.y = dot2_bf16(x0, sh, sl, x1, ch, cl);
    }
    store_fp4_row(static_cast<uint8_t*>(p.cache) + row * kFp4RowBytes, c0, c1, *reinterpret_cast<const uint32_t*>(&kr),
                  lane);
    return;
  }
  if (p.rope_theta > 0.0) {
    constexpr double kTwoPi = 6.283185307179586476925286766559, kInvTwoPi = 0.15915494309189533576888376337251;
    const double ang = __dmul_rn(double(pos), p.inv_freq[lane]);
    const double turns = rint(__dmul_rn(ang, kInvTwoPi));
    const float red = float(__fma_rn(-turns, kTwoPi, ang));
    float sn, cs;
    sincosf(red, &sn, &cs);
    const float x0 = __low2float(kp), x1 = __high2float(kp);
    kr = __floats2bfloat162_rn(fmaf(x0, cs, -x1 * sn), fmaf(x0, sn, x1 * cs));
  }

  if constexpr (kCode == kCodeBf16) {
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.cache) + row * kRow;
    reinterpret_cast<uint4*>(dst)[2 * lane] = c0;
    reinterpret_cast<uint4*>(dst)[2 * lane + 1] = c1;
    reinterpret_cast<__nv_bfloat162*>(dst + kLatent)[lane] = kr;
  } else {
    // the row's 576 bf16 values, as exact fp32
    float v[18];
    const __nv_bfloat162* c0h = reinterpret_cast<const __nv_bfloat162*>(&c0);
    const __nv_bfloat162* c1h = reinterpret_cast<const __nv_bfloat162*>(&c1);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __low2float(c0h[j]);
      v[2 * j + 1] = __high2float(c0h[j]);
      v[8 + 2 * j] = __low2float(c1h[j]);
      v[8 + 2 * j + 1] = __high2float(c1h[j]);
    }
    v[16] = __low2float(kr);
    v[17] = __high2float(kr);
    if constexpr (kCode == kCodeE4m3) {
      float a = 0.f;
#pragma unroll
      for (int j = 0; j < 18; ++j) a = fmaxf(a, fabsf(v[j]));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
      // IEEE fp32, round to nearest even, in the documented order
      float s = __fdiv_rn(a, 448.f);
      if (s == 0.f) s = 1.f;
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = e4m3x2_rn_sat(__fdiv_rn(v[4 * j], s), __fdiv_rn(v[4 * j + 1], s)) |
               (e4m3x2_rn_sat(__fdiv_rn(v[4 * j + 2], s), __fdiv_rn(v[4 * j + 3], s)) << 16);
      uint8_t* dst = static_cast<uint8_t*>(p.cache) + row * kRow;
      reinterpret_cast<uint4*>(dst)[lane] = make_uint4(w[0], w[1], w[2], w[3]);
      reinterpret_cast<uint16_t*>(dst + kLatent)[lane] =
          uint16_t(e4m3x2_rn_sat(__fdiv_rn(v[16], s), __fdiv_rn(v[17], s)));
      if (lane == 0) p.scale_zero[row] = s;
      return;
    }
    float lo = 0.f, hi = 0.f;  // the range always includes 0
#pragma unroll
    for (int j = 0; j < 18; ++j) {
      lo = fminf(lo, v[j]);
      hi = fmaxf(hi, v[j]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    // IEEE fp32, round to nearest even, no contraction, in the documented order
    float s = __fdiv_rn(__fsub_rn(hi, lo), 255.f);
    if (s == 0.f) s = 1.f;
    float zp = rintf(__fsub_rn(-128.f, __fdiv_rn(lo, s)));
    zp = fminf(fmaxf(zp, -128.f), 127.f);
    int8_t q[18];
#pragma unroll
    for (int j = 0; j < 18; ++j) {
      float c = __fadd_rn(rintf(__fdiv_rn(v[j], s)), zp);
      c = fminf(fmaxf(c, -128.f), 127.f);
      q[j] = int8_t(int(c));
    }
    int8_t* dst = static_cast<int8_t*>(p.cache) + row * kRow;
    uint4 packed;
    int8_t* pk = reinterpret_cast<int8_t*>(&packed);
#pragma unroll
    for (int j = 0; j < 16; ++j) pk[j] = q[j];
    reinterpret_cast<uint4*>(dst)[lane] = packed;
    char2 tail;
    tail.x = q[16];
    tail.y = q[17];
    reinterpret_cast<char2*>(dst + kLatent)[lane] = tail;
    if (lane == 0) {
      p.scale_zero[row * 2] = s;
      p.scale_zero[row * 2 + 1] = zp;
    }
  }
}

cudaError_t launch_append(const AppendParams& p, int code, cudaStream_t stream) {
  if (p.n_tokens == 0) return cudaSuccess;
  // a decode step appends one token per sequence: one warp per block spreads
  // the fp64 RoPE over as many SMs as there are tokens
  const int warps = p.n_tokens < 2048 ? 1 : 8;
  const int grid = (p.n_tokens + warps - 1) / warps;
  if (code == kCodeInt8) return launch_pdl(append_kernel<kCodeInt8>, dim3(grid), dim3(warps * 32), 0, stream, 1, p);
  if (code == kCodeE4m3) return launch_pdl(append_kernel<kCodeE4m3>, dim3(grid), dim3(warps * 32), 0, stream, 1, p);
  if (code == kCodeE2m1) return launch_pdl(append_kernel<kCodeE2m1>, dim3(grid), dim3(warps * 32), 0, stream, 1, p);
  return launch_pdl(append_kernel<kCodeBf16>, dim3(grid), dim3(warps * 32), 0, stream, 1, p);
}

}  // namespace mla
