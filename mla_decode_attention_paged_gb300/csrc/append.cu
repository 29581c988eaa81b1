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
// that much.  The rotation of FP4 rows is therefore exact to about 2^-35 before it is
// rounded, to fp32 and then to bf16: the angle as a 64-bit fraction of a turn (pos
// times the frequency, modulo 2^64: two integer multiply-adds, where fp64 takes 64
// times the issue slots of fp32 on this part), sine and cosine from a table of 256
// angles, each a sum of two floats, and the angle that is left.  The frequency is the
// fp64 one, held to about 2^-64 turns, so that the angle is off by as many times the
// position: 2^-35 radians at 2^26, 2^-31 at 2^30.  None of 8 million blocks had
// another code than the fp64 rotation so rounded (with fp32 sine and cosine, one
// value in 10^4).
struct alignas(16) SinCos {
  float sh, sl, ch, cl;  // sine and cosine as hi + lo
};
struct TurnTable {
  SinCos at[256];
};
// Sines and cosines of i / 256 turns, by their Taylor series in double around the nearest quarter.
constexpr TurnTable make_turn_table() {
  TurnTable t = {};
  for (int i = 0; i < 256; ++i) {
    const int quarter = (i + 32) / 64;
    const double x = (i - 64 * quarter) * (6.283185307179586476925286766559 / 256);
    double s = 0, c = 0, term = 1;
    for (int n = 0; n < 24; ++n) {  // term = x^n / n!
      if (n % 2 == 0) c += n % 4 == 0 ? term : -term;
      else s += n % 4 == 1 ? term : -term;
      term = term * x / (n + 1);
    }
    const double sine = quarter % 4 == 0 ? s : quarter % 4 == 1 ? c : quarter % 4 == 2 ? -s : -c;
    const double cosine = quarter % 4 == 0 ? c : quarter % 4 == 1 ? -s : quarter % 4 == 2 ? -c : s;
    t.at[i].sh = float(sine);
    t.at[i].sl = float(sine - double(float(sine)));
    t.at[i].ch = float(cosine);
    t.at[i].cl = float(cosine - double(float(cosine)));
  }
  return t;
}
__device__ const TurnTable kTurns = make_turn_table();

// The product a * b as a rounded value and its rounding error.
__device__ __forceinline__ float mul_err(float a, float b, float& err) {
  const float p = __fmul_rn(a, b);
  err = __fmaf_rn(a, b, -p);
  return p;
}

// The sum of a and b as a rounded value and its rounding error, whichever is larger.
__device__ __forceinline__ float add_err(float a, float b, float& err) {
  const float s = __fadd_rn(a, b), t = __fadd_rn(s, -a);
  err = __fadd_rn(__fadd_rn(a, -__fadd_rn(s, -t)), __fadd_rn(b, -t));
  return s;
}

// Sine and cosine of `phase` / 2^64 turns, each as hi + lo with lo up to 2^-13: with
// the nearest of the table's angles a, and b = what is left, at most 1 / 512 turn,
// sin(a + b) = sin a + cos a sin b + sin a (cos b - 1), and so on.  b is a sum of two
// floats and cos a sin b keeps its rounding error, so that what is rounded is below
// 2^-13, by 2^-38.
__device__ __forceinline__ SinCos sincos_turns(uint64_t phase, const SinCos* table) {
  const uint64_t near = phase + (1ull << 55);
  const SinCos a = table[near >> 56];
  constexpr double kUnit = 6.283185307179586476925286766559 / (1ll << 32);  // 2^-32 turns
  constexpr float kHi = float(kUnit), kLo = float(kUnit - double(kHi)), kLow = float(kUnit / (1ll << 32));
  const float n = float(int(uint32_t(near >> 32) & 0xffffff) - 0x800000);  // exact
  float b1;
  const float b = mul_err(n, kHi, b1), b2 = b * b;
  b1 += __fmaf_rn(n, kLo, float(uint32_t(near)) * kLow);
  const float sb = __fmaf_rn(b * b2, -1.f / 6.f, b1), cb = b2 * __fmaf_rn(b2, 1.f / 24.f, -0.5f);  // sin b - b, cos b - 1
  SinCos r;
  float e, f;
  const float u = mul_err(a.ch, b, e), v = mul_err(-a.sh, b, f);
  e = __fmaf_rn(a.cl, b, e) + a.sl;
  f = __fmaf_rn(-a.sl, b, f) + a.cl;
  float g, h;
  r.sh = add_err(a.sh, u, g);
  r.ch = add_err(a.ch, v, h);
  r.sl = __fmaf_rn(a.sh, cb, __fmaf_rn(a.ch, sb, e + g));
  r.cl = __fmaf_rn(a.ch, cb, __fmaf_rn(-a.sh, sb, f + h));
  return r;
}

// x a + y b rounded to fp32 and that to bf16, for bf16 x and y and two-float a and b.
__device__ __forceinline__ __nv_bfloat16 dot2_bf16(float x, float ah, float al, float y, float bh, float bl) {
  float ep, eq, es;
  const float p = mul_err(x, ah, ep), q = mul_err(y, bh, eq), s = add_err(p, q, es);
  const float low = __fadd_rn(es, __fadd_rn(__fmaf_rn(x, al, ep), __fmaf_rn(y, bl, eq)));
  return __float2bfloat16_rn(__fadd_rn(s, low));
}

// The larger magnitudes of two packed pairs of bf16 values, NaN where either is.
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 m = __hmax2_nan(__habs2(*reinterpret_cast<const __nv_bfloat162*>(&a)),
                                       __habs2(*reinterpret_cast<const __nv_bfloat162*>(&b)));
  return *reinterpret_cast<const uint32_t*>(&m);
}

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
// Two fp32 values to E2M1 codes, the first in the low four bits (the rest undefined).
__device__ __forceinline__ uint32_t e2m1x2_rn_sat(float first, float second) {
  uint32_t r;
  asm("{\n\t.reg .b8 a;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "mov.b32 %0, {a, a, a, a};\n\t}"
      : "=r"(r)
      : "f"(first), "f"(second));
  return r;
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
    v[2 * j] = __uint_as_float(x[j] << 16) * inv;
    v[2 * j + 1] = __uint_as_float(x[j] & 0xffff0000u) * inv;
  }
  const uint32_t lo = __byte_perm(x[0], x[1], 0x7531) & 0x80808080u, hi = __byte_perm(x[2], x[3], 0x7531) & 0x80808080u;
  return (e2m1x8_rn_sat(v) & 0x77777777u) | lo | (hi >> 4);
}

// Quantises and stores one row: lane l has latents [16l, 16l + 16) and the
// rotated pair l of the RoPE key.
__device__ __forceinline__ void store_fp4_row(uint8_t* dst, const uint4& c0, const uint4& c1, uint32_t pair, int lane) {
  const uint32_t x0[4] = {c0.x, c0.y, c0.z, c0.w}, x1[4] = {c1.x, c1.y, c1.z, c1.w};
  uint32_t top2 = max_abs_bf16x2(x0[0], x1[0]);
#pragma unroll
  for (int j = 1; j < 4; ++j) top2 = max_abs_bf16x2(top2, max_abs_bf16x2(x0[j], x1[j]));
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
  // the lane's pair is values 2g and 2g + 1 of the word: byte g, and the signs'
  // bits 16g + 7 and 16g + 15 (g < 2) or 16g - 29 and 16g - 21
  const float rinv = fp4_inv_scale(rscale);
  uint32_t wr = 0;
  if (rscale != 255)
    wr = ((e2m1x2_rn_sat(__uint_as_float(pair << 16) * rinv, __uint_as_float(pair & 0xffff0000u) * rinv) & 0x77) << (8 * g)) |
         (((pair >> 15 & 1) | (pair >> 31 << 8)) << (g < 2 ? 16 * g + 7 : 16 * g - 29));
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

// Position of token i and its cache row; false (and reported) if its sequence,
// position or page-table entry is out of range.
__device__ __forceinline__ bool locate(const AppendParams& p, int i, bool report, int& pos, size_t& row) {
  const int b = p.chunk > 0 ? i / p.chunk : p.seq_ids[i];
  // 64-bit: a length near the int32 limits must not wrap into a valid position
  const long long pos64 = p.chunk > 0 ? (long long)p.seq_lens[b] - p.chunk + i % p.chunk : p.positions[i];
  const int page_log2 = __ffs(p.page_size) - 1;
  bool ok = b >= 0 && b < p.num_seqs && pos64 >= 0 && pos64 < ((long long)p.max_pages << page_log2);
  pos = int(pos64);  // in [0, max_pages * P) once ok
  int page = -1;
  if (ok) {
    page = p.block_table[size_t(b) * p.max_pages + (pos >> page_log2)];
    ok = page >= 0 && page < p.num_pages;
  }
  if (!ok && report) set_status(p.status, MLA_ERR_DEVICE_BOUNDS);
  row = (size_t(page) << page_log2) + (pos & (p.page_size - 1));
  return ok;
}

// FP4: a warp takes a run of tokens (one where there are few), whose places its lanes
// look up side by side, the next one's values on their way while it works on one.
// Lane l owns latent values [16l, 16l + 16) and RoPE pair l.  Bound by instructions
// (rotation, quantisation, packing; about 350 a token) rather than memory (1,472 bytes
// a token): 34,817 tokens 15.6 us, 3.3 TB/s (17.3 where each token was looked up in
// its turn, by a warp of four of them).
template <bool kRuns>
__global__ void __launch_bounds__(256) append_fp4_kernel(AppendParams p) {
  __shared__ SinCos shared_turns[kRuns ? 256 : 1];
  const SinCos* turns = kTurns.at;
  if constexpr (kRuns) {  // 256 threads; gathers of 16 bytes are cheaper in shared memory
    shared_turns[threadIdx.x] = kTurns.at[threadIdx.x];
    turns = shared_turns;
    __syncthreads();
  }
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31, run = kRuns ? p.run : 1;
  const long long first = (long long)(blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)) * run;
  if (first >= p.n_tokens) return;
  const int i0 = int(first), n = min(run, p.n_tokens - i0);
  const uint64_t turn = p.turn[lane];
  uint4 c0, c1;
  __nv_bfloat162 kp;
  auto load = [&](int i) {
    const uint4* src = reinterpret_cast<const uint4*>(p.c_kv + size_t(i) * kLatent) + 2 * lane;
    c0 = src[0];
    c1 = src[1];
    kp = reinterpret_cast<const __nv_bfloat162*>(p.k_pe + size_t(i) * kRope)[lane];
  };
  load(i0);
  int pos = 0;  // lane t finds where token t goes
  size_t row = 0;
  const bool there = lane < n && locate(p, i0 + lane, true, pos, row);
  const uint32_t places = __ballot_sync(0xffffffffu, there);
#pragma unroll 1
  for (int t = 0; t < n; ++t) {
    const uint4 x0 = c0, x1 = c1;
    const __nv_bfloat162 k = kp;
    if (t + 1 < n) load(i0 + t + 1);
    if (!(places >> t & 1)) continue;
    __nv_bfloat162 kr = k;
    if (p.rotate) {
      const SinCos r = sincos_turns(uint64_t(__shfl_sync(0xffffffffu, pos, t)) * turn, turns);
      const float a = __low2float(k), b = __high2float(k);
      kr.x = dot2_bf16(a, r.ch, r.cl, -b, r.sh, r.sl);
      kr.y = dot2_bf16(a, r.sh, r.sl, b, r.ch, r.cl);
    }
    const size_t to = __shfl_sync(0xffffffffu, row, t);
    store_fp4_row(static_cast<uint8_t*>(p.cache) + to * kFp4RowBytes, x0, x1, *reinterpret_cast<const uint32_t*>(&kr),
                  lane);
  }
}

// One warp per token.  Lane l owns latent values [16l, 16l + 16) and RoPE pair l.
template <int kCode>
__global__ void __launch_bounds__(256) append_kernel(AppendParams p) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int i = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (i >= p.n_tokens) return;
  // latent part: 16 bf16 per lane, two 16-byte loads; RoPE pair `lane`.  They do
  // not wait for the page lookup.
  const uint4* src = reinterpret_cast<const uint4*>(p.c_kv + size_t(i) * kLatent) + 2 * lane;
  uint4 c0 = src[0], c1 = src[1];
  const __nv_bfloat162 kp = reinterpret_cast<const __nv_bfloat162*>(p.k_pe + size_t(i) * kRope)[lane];

  int pos;
  size_t row;
  if (!locate(p, i, lane == 0, pos, row)) return;

  // RoPE pair `lane`: angle = pos * theta^(-2 lane / 64) in fp64 (up to
  // ~2^31 rad), reduced modulo 2 pi in fp64 to [-pi, pi]; sine, cosine and
  // the rotation then in fp32 ahead of the one rounding to bf16.  A full
  // fp64 sincos per lane kept the few SMs an append runs on busy for
  // microseconds (the fp64 units are a small fraction of this part's), and
  // the reduced fp32 result stays far inside the bf16 rounding.
  __nv_bfloat162 kr = kp;
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
  if (code == kCodeE2m1) {
    // A token to a warp, or a run of them.  One / runs, us: 1,024 tokens 2.8 / 3.4, 2,048
    // 3.1 / 3.4, 3,500 3.8 / 4.1, 4,096 4.1 / 4.2, 5,000 5.8 / 4.8, 6,080 5.9 / 4.9, 8,192
    // 6.1 / 6.8, 12,160 7.6 / 7.0, 14,000 8.3 / 9.0, 18,240 10.2 / 9.2, 34,817 17.0 / 15.7.
    // Runs take steps, one for each token more to a warp (6,081, 12,161, ...), and up to
    // 18% more than one token a warp right behind such a step.
    if (p.n_tokens <= 4096) return launch_pdl(append_fp4_kernel<false>, dim3(grid), dim3(warps * 32), 0, stream, 1, p);
    const int tokens = 8 * p.run;  // of a block
    return launch_pdl(append_fp4_kernel<true>, dim3((p.n_tokens - 1) / tokens + 1), dim3(256), 0, stream, 1, p);
  }
  return launch_pdl(append_kernel<kCodeBf16>, dim3(grid), dim3(warps * 32), 0, stream, 1, p);
}

}  // namespace mla
