// prompt_attention.cu -- causal attention over packed prompts in the
// un-absorbed form: per-head keys [k_nope | k_pe] and values, grouped heads,
// sequences of different lengths.
//
// For query row i of sequence b (cu_q[b] <= i < cu_q[b + 1], Lq and Lk its
// query and key counts, t = i - cu_q[b]) and head h, with kv head g = h / (H /
// H_kv), over the keys j < t + 1 + Lk - Lq:
//     s_j = scale * (q_nope[i][h] . k_nope[j][g] + q_pe[i][h] . k_pe[j])
//     out[i][h] = sum_j softmax(s)_j v[j][g],   lse[i][h] = ln sum_j exp(s_j)
// ("Beyond the Attention Bottleneck", "Down-Projection and Up-Projection
// Mechanics" and "The RoPE Compatibility Problem"; "The Architecture of
// Memory", "The Prefill Phase": a prompt's tokens are processed together.)
// 320 multiply-adds per (query, key, head), against the 1,088 of the absorbed
// form: the tensor cores bound it.
//
// One CTA per SM takes units of work from the plan's list: a block of up to 256
// query rows of one sequence and one head, as two tiles of 128 rows (the MMA's
// M).  Heads that share a key/value head are packed into the rows, row = token *
// F + head, F the largest power of two that divides the group (at most 128): a
// block then spans 256 / F tokens, so less of its diagonal tiles is masked and
// few tokens fill it, and the copy of a query tile is one box of F heads.  Keys come in tiles of 128.  Per key tile and query tile,
//     S [128 x 128] = Q [128 x 192] K^T   12 MMAs, both operands in shared memory
//     O [128 x 128] += P [128 x 128] V     8 MMAs, P (bf16) in tensor memory over S
// of 65 cycles each, so a key tile takes the pipe 2,600 cycles; one query tile's
// softmax (about 1,250 cycles) runs while the pipe works on the other tile.
// Tensor memory: S x2, O x2, all 512 columns.  Shared memory: Q of both tiles
// (96 KB) and a ring of eight 16 KB boxes [128 keys x 64 columns] (three to a
// key tile, two to a value tile): 1.6 key tiles, which is all that fits.
//
// Softmax: one thread per query row, online in fp32 and base 2.  The running
// maximum only has to bound the scores within 8 (log2 units); a tile that
// breaks the bound raises it and rescales O and the sum.  P is rounded to bf16
// for the MMA, whose operands have one type (at most 2^-8 relative per weight,
// averaged over the keys: 0.0017 off the formula as a 2-norm over 93 and 16,384
// tokens alike, 0.0016 and 0.0017 with fp32 weights, most of it the output's own
// rounding); the sum takes the unrounded fp32 weights.
//
// Measured (16,384 tokens, 16 heads: 1.37 TFLOP): 864 us, 1,590 TFLOP/s, 84% of
// the measured bf16 peak (from 1,582 us).  What each step gave: one MMA warp per
// query tile instead of one for both 1.58 -> 1.08 ms; turns, one barrier per
// tile's boxes and PV from the first 96 weights on 0.98; MMA issue as
// straight-line code 0.90; key and value copies from two warps 0.86.  Short units
// leave the pipe idle while the next unit's first keys land and its first softmax
// runs: 24 ragged prompts of 1 to 2,048 tokens run at 128 us (970 TFLOP/s), 14%
// of it the masked halves of the diagonal tiles.
// Few rows behind long contexts (26 behind 32,768 and 20,011 keys) take 97 us,
// 4.5 TB/s: one query tile at work, and a key tile's chain QK, softmax, PV takes
// 2,930 cycles where its copies take 2,800.
//
// Warps: 0-3 softmax and epilogue of query tile 0, 4-7 of tile 1, 8 units and
// key copies, 9 (which also owns tensor memory) and 10 query copies and MMA
// issue for tiles 0 and 1, 11 value copies.  Every wait is bounded: on timeout
// the CTA records MLA_ERR_DEVICE_TIMEOUT, waits for its products and copies in
// flight on their own barriers (half a second at most), frees its tensor memory
// and returns.
#include <atomic>

#include "blackwell_ptx.cuh"
#include "decode_common.cuh"
#include "params.cuh"

namespace mla {
namespace {

using namespace ptx;
using namespace dc;

constexpr int kKeys = 128;                         // keys of a tile
constexpr uint32_t kBox = 128 * 128;               // [128 rows x 64 columns] bf16, SW128: 16 KB
constexpr uint32_t kQTile = 3 * kBox;              // q_nope columns 0-63, 64-127, q_pe
constexpr int kRing = 8;                           // boxes of the key / value ring
constexpr uint32_t kOffRing = 2 * kQTile;
constexpr uint32_t kOffMisc = kOffRing + kRing * kBox;
constexpr uint32_t kSmem = kOffMisc + 2048 + 1024;  // + barriers, alignment slack
constexpr int kPromptThreads = 384;
constexpr uint32_t kColS = 0, kColO = 256;         // tensor memory columns: S x2, O x2
constexpr uint64_t kWaitNs = 2000000000ull;        // 2 s
constexpr uint64_t kDrainNs = 500000000ull;        // 0.5 s
constexpr float kRescale = 8.f;                    // log2 units
constexpr int kPlanThreads = 1024, kFewPlan = 128;
constexpr int kPlanSeqs = 1024;                    // sequences whose offsets the plan holds in shared memory
constexpr float kMergeTiles = 5.f;                 // the merge, in key tiles' time
constexpr int kMinSplit = 10;                      // key tiles of a block that is never split
constexpr int kDirectTiles = 18;                   // key tiles of a call that one round of units runs without a plan
constexpr int kBuckets = kPlanThreads;             // cost classes of the plan's counting sort
static_assert(kSmem <= 232448, "dynamic shared memory of one CTA");

// ----- plan ----------------------------------------------------------------------
// One CTA: checks cu_q and cu_k, cuts every sequence into blocks of 256 query
// rows, splits the keys of long blocks where there are too few blocks to fill
// the SMs, and lists the items: sequences by falling number of key tiles (a
// counting sort), the blocks of a sequence from its last (the longest) to its
// first.  The CTAs take the units (item, head) in that order, so the blocks of
// a sequence, which share keys and values, run at about the same time and read
// them from L2 (a list sorted by block length alone read the keys and values of
// many equal prompts from memory once per block), and short units come last
// (heads before blocks left the last head's longest blocks for the end: 1,000
// instead of 893 us for 16,384 tokens at 16 heads).  A sequence whose offsets
// decrease or pass the end, and every one after it, is skipped and reported;
// this also bounds the list.
//
// Split: candidate k cuts the longest block into k + 1 pieces and every block
// into pieces of at most that length.  Its estimate, in key tiles: the longest
// piece where every unit (item, head) has its own CTA, else the mean load and a
// share of the longest piece for the uneven end, plus three tiles for a unit's
// start and end and five for the merge, a kernel of its own.  The pieces of a
// block depend on the lengths and the SM count alone, and are merged in order,
// so results repeat bit for bit.  A plan is all latency, and was 2.5 us more with a
// warp to each candidate, shuffles for the sums, and sorts and scans for the
// list: here a candidate is a lane, the sums are atomics in shared memory and a
// block counts the pieces ahead of it.
__device__ __forceinline__ int key_tiles(int vis_last) { return vis_last > 0 ? (vis_last + kKeys - 1) / kKeys : 0; }
__device__ __forceinline__ int pieces_of(int tiles, int longest) { return tiles > longest ? (tiles + longest - 1) / longest : 1; }

__device__ __forceinline__ bool bad_offsets(const PromptParams& p, int q0, int q1, int k0, int k1) {
  return q0 < 0 || q1 < q0 || q1 > p.n_q || k0 < 0 || k1 < k0 || k1 > p.n_k;
}
__device__ __forceinline__ int blocks_of(const PromptParams& p, int tokens) {
  return ((tokens << p.pack) + kPromptRows - 1) / kPromptRows;
}
// The whole item of block i of the sequence with query rows [q0, q1) and key rows [k0, k1).
__device__ __forceinline__ PromptItem make_item(const PromptParams& p, int q0, int q1, int k0, int k1, int i) {
  const int r0 = i * kPromptRows, t0 = r0 >> p.pack;
  PromptItem it;
  it.q_row0 = q0 + t0;
  it.rows = min(kPromptRows, ((q1 - q0) << p.pack) - r0);
  it.k_row0 = k0;
  it.vis0 = (k1 - k0) - (q1 - q0) + t0 + 1;
  it.kv_begin = 0;
  it.kv_end = max(0, it.vis0 + ((it.rows - 1) >> p.pack));
  it.pieces = 1;
  it.piece = 0;
  it.partial = 0;
  it.head = it.pad[0] = it.pad[1] = 0;
  return it;
}

// kThreads = kFewPlan: the call has at most that many blocks, no more units than
// two rounds, and may split keys (fewer warps to meet at barriers: with the
// merge's grid cut to its rows, 34.3 -> 33.4 us for 256 rows behind 8,192 keys).
template <int kThreads>
__global__ void __launch_bounds__(kThreads) prompt_plan_kernel(PromptParams p) {
  constexpr bool kFew = kThreads == kFewPlan;
  __shared__ int scan_tmp[32];
  __shared__ int hist[kFew ? 1 : kBuckets];
  __shared__ int carry, first_bad, longest, total_tiles, piece_tiles;
  __shared__ int few_tiles[kPromptMaxSplit], few_rows[kPromptMaxSplit], few_key[kPromptMaxSplit], few_pieces[kPromptMaxSplit];
  __shared__ int cand_pieces[32], cand_rows[32];  // sums over the blocks, of each candidate
  __shared__ unsigned long long taken;  // split blocks, their rows << 10, their partial rows << 32
  // offsets and block starts, here where they fit: the loops below read them over and over
  __shared__ int offsets[4][kPlanSeqs + 1];
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool fits = p.num_seqs <= kPlanSeqs;
  const int *cu_q = p.cu_q, *cu_k = p.cu_k;
  int *block_start = p.block_start, *seq_first = p.seq_first;
  if (fits) {
    for (int b = tid; b <= p.num_seqs; b += kThreads) {
      offsets[0][b] = p.cu_q[b];
      offsets[1][b] = p.cu_k[b];
    }
    cu_q = offsets[0];
    cu_k = offsets[1];
    block_start = offsets[2];
    seq_first = offsets[3];
  }
  if (tid == 0) {
    carry = 0;
    longest = total_tiles = 0;
    taken = 0;
    first_bad = p.num_seqs;
    p.status[0] = MLA_OK;
    p.status[2] = 0;  // units taken
    p.status[3] = 0;  // split blocks
  }
  if (!kFew) hist[tid] = 0;
  if (tid < 32) cand_pieces[tid] = cand_rows[tid] = 0;
  __syncthreads();
  for (int b = tid; b < p.num_seqs; b += kThreads) {
    const int q0 = cu_q[b], q1 = cu_q[b + 1], k0 = cu_k[b], k1 = cu_k[b + 1];
    if (bad_offsets(p, q0, q1, k0, k1)) atomicMin(&first_bad, b);
  }
  __syncthreads();
  const int good = first_bad;
  if (tid == 0 && good < p.num_seqs) set_status(p.status, MLA_ERR_DEVICE_BOUNDS);
  for (int base = 0; base < good; base += kThreads) {
    const int b = base + tid;
    const int blocks = b < good ? blocks_of(p, cu_q[b + 1] - cu_q[b]) : 0;
    int total;
    const int ex = block_exclusive_scan(blocks, scan_tmp, &total);
    if (b < good) block_start[b] = carry + ex;
    __syncthreads();
    if (tid == 0) carry += total;
    __syncthreads();
  }
  const int n = carry;  // block_start is read below by other threads: the barriers above order it
  auto blocks_in = [&](int b) { return blocks_of(p, cu_q[b + 1] - cu_q[b]); };
  auto sequence_of = [&](int i) {
    int lo = 0, hi = good - 1;  // last sequence whose first block is <= i
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (block_start[mid] <= i) lo = mid; else hi = mid - 1;
    }
    return lo;
  };
  auto block_item = [&](int i, int b) {
    return make_item(p, cu_q[b], cu_q[b + 1], cu_k[b], cu_k[b + 1], i - block_start[b]);
  };
  // short blocks are never split: a piece would be little more than its start and
  // merge.  Nor are more units than two rounds, where equal lengths fill the SMs
  // (24 single tokens behind 5,000 keys each at 16 heads: 204 us), at the cost
  // of unequal ones: one behind 100,000 keys beside 19 behind 1,000 takes 1,200 us,
  // beside nine, where it is split, 264.
  const int G = p.sm_count;
  if (kFew || (p.may_split && (long long)n * p.heads_v <= 2 * G && n <= kPromptMaxSplit)) {
    PromptItem it;
    int t = 0, key = 0;
    if (tid < n) {
      const int b = sequence_of(tid);
      it = block_item(tid, b);
      t = key_tiles(it.kv_end);
      key = key_tiles(cu_k[b + 1] - cu_k[b]);
      few_tiles[tid] = t;
      few_rows[tid] = it.rows;
      few_key[tid] = key;
      atomicMax(&longest, t);
      atomicAdd(&total_tiles, t);
    }
    __syncthreads();
    const bool split = longest > kMinSplit;
    const int T = (longest + lane) / (lane + 1);  // lane: candidate
    if (split) {
      for (int i = warp; i < n; i += kThreads / 32) {
        const int ti = few_tiles[i], c = pieces_of(ti, T);
        atomicAdd(&cand_pieces[lane], c);
        if (c > 1) atomicAdd(&cand_rows[lane], c * few_rows[i]);
      }
    }
    __syncthreads();
    if (warp == 0) {
      const int pieces = cand_pieces[lane];
      const float units = float(pieces) * p.heads_v, load = float(total_tiles) * p.heads_v + 3.f * units;
      float low = fmaxf(T + 3.f, load * __frcp_rn(float(G)) + (units > G ? 0.35f * T : 0.f));
      if (lane > 0) low = 1.1f * (low + kMergeTiles);  // only where it clearly pays
      if (units > 2 * G || pieces > n + kPromptExtraItems || (long long)cand_rows[lane] * p.heads_v > p.partial_rows)
        low = lane > 0 ? 1e30f : 1e29f;
      int best = lane;  // the lowest estimate, of equal ones the first
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const float e2 = __shfl_xor_sync(0xffffffffu, low, o);
        const int b2 = __shfl_xor_sync(0xffffffffu, best, o);
        if (e2 < low || (e2 == low && b2 < best)) {
          low = e2;
          best = b2;
        }
      }
      if (lane == best) {
        piece_tiles = split && best > 0 ? T : 0x7fffffff;
        p.status[1] = split && best > 0 ? pieces : n;
      }
    }
    __syncthreads();
    const int c = pieces_of(t, piece_tiles);
    if (tid < n) few_pieces[tid] = c;
    __syncthreads();
    if (tid < n) {
      int at = 0;  // pieces of the blocks listed before: of longer sequences, and the later ones of its own
      for (int j = 0; j < n; ++j)
        if (few_key[j] > key || (few_key[j] == key && j > tid)) at += few_pieces[j];
      const int keys = it.kv_end;
      it.pieces = c;
      if (c > 1) {
        const unsigned long long old =
            atomicAdd(&taken, 1ull | (unsigned long long)it.rows << 10 | (unsigned long long)(c * it.rows * p.heads_v) << 32);
        it.partial = int(old >> 32);
        p.splits[int(old & 1023)] = {it.q_row0, it.rows, c, it.partial, int(uint32_t(old) >> 10)};
      }
      for (int q = 0; q < c; ++q) {
        it.piece = q;
        it.kv_begin = q * t / c * kKeys;
        it.kv_end = min(keys, (q + 1) * t / c * kKeys);
        p.items[at + q] = it;
      }
    }
    __syncthreads();
    if (tid == 0) {
      p.status[3] = int(taken & 1023);
      p.status[4] = int(uint32_t(taken) >> 10);
    }
    return;
  }
  if constexpr (!kFew) {
    auto bucket_of = [&](int b) { return kBuckets - 1 - min(kBuckets - 1, key_tiles(cu_k[b + 1] - cu_k[b])); };
    for (int b = tid; b < good; b += kThreads) {
      const int c = blocks_in(b);
      if (c > 0) atomicAdd(&hist[bucket_of(b)], c);
    }
    __syncthreads();
    int total;
    const int ex = block_exclusive_scan(hist[tid], scan_tmp, &total);
    hist[tid] = ex;
    if (tid == 0) p.status[1] = total;
    __syncthreads();
    // the order of equally long sequences is arbitrary: it decides which CTA runs an item, not its result
    for (int b = tid; b < good; b += kThreads) {
      const int c = blocks_in(b);
      if (c > 0) seq_first[b] = atomicAdd(&hist[bucket_of(b)], c);
    }
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
      const int b = sequence_of(i);
      p.items[seq_first[b] + blocks_in(b) - 1 - (i - block_start[b])] = block_item(i, b);
    }
  }
}

// ----- attention -------------------------------------------------------------------
constexpr int kItemRing = 4, kDirectSeqs = 32;
struct PromptBarriers {
  uint64_t q_full[2], q_empty[2];  // query tile loaded / read by its last QK
  uint64_t k_full[2], v_full[2];   // boxes of even / odd key tiles landed
  uint64_t k_empty[2], v_empty[2]; // boxes of even / odd key tiles read by both MMA threads
  uint64_t s_full[2];              // scores of a tile complete
  uint64_t p_full[2], p_rest[2];   // P of the first 96 keys written (and O rescaled where needed); of the last 32
  uint64_t o_full[2], o_free[2];   // output complete / read
  uint64_t turn[2];                // the MMA threads' turns
  uint64_t drain[2];
  uint64_t item_full[kItemRing], item_empty[kItemRing];
  PromptItem items[kItemRing];     // the CTA's units, read ahead by the producer (rows = 0: no more)
  // without a plan: the sequences' offsets (q0, q1, k0, k1) and the blocks up to and with each
  int4 seqs[kDirectSeqs];
  int seq_end[kDirectSeqs];
  uint32_t tmem_base;
  int abort;
  uint32_t k_tiles, v_tiles, q_tiles[2];  // key, value and query tiles that copies were issued of
};
static_assert(sizeof(PromptBarriers) <= 2048, "shared memory behind the ring");

__device__ __forceinline__ void fail(PromptBarriers* B, int* status) {
  B->abort = 1;
  set_status(status, MLA_ERR_DEVICE_TIMEOUT);
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

// Two fp32 operations at once on a register pair.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  return uint64_t(__float_as_uint(a)) | (uint64_t(__float_as_uint(b)) << 32);
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  return make_float2(__uint_as_float(uint32_t(v)), __uint_as_float(uint32_t(v >> 32)));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ float row_max(const uint32_t (&s)[4][32]) {  // four chains
  float mx[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    mx[c] = fmaxf(__uint_as_float(s[c][0]), __uint_as_float(s[c][1]));
#pragma unroll
    for (int i = 2; i < 32; i += 2)
      mx[c] = fmaxf(fmaxf(mx[c], __uint_as_float(s[c][i])), __uint_as_float(s[c][i + 1]));
  }
  return fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), -INFINITY);  // NaN scores do not count
}

__device__ __forceinline__ PromptItem load_item(const PromptItem* src) {  // 16-byte loads, global or shared
  const int4* v = reinterpret_cast<const int4*>(src);
  const int4 a = v[0], b = v[1], c = v[2];
  return {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x, c.y, {c.z, c.w}};
}

// 1 / l; 0 for a row without keys (l = 0); NaN stays NaN.
__device__ __forceinline__ float inverse_sum(float l) { return l > 0.f ? __frcp_rn(l) : (l == 0.f ? 0.f : l); }

// Eight outputs, scaled and rounded to bf16.
__device__ __forceinline__ uint4 pack_out(const uint32_t* o, float inv) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
    w[e] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap* map, int x, int y, int z) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(z)
               : "memory");
}

// Key tiles of query tile t (0, 1) of an item.
__device__ __forceinline__ int tiles_of(const PromptItem& it, int t, int pack) {
  if (it.rows <= 128 * t) return 0;
  const int last = (min(it.rows, 128 * (t + 1)) - 1) >> pack;
  return key_tiles(min(it.kv_end, it.vis0 + last) - it.kv_begin);
}

// kDirect: few sequences, blocks and keys; the CTAs list the work themselves.
template <bool kDirect>
__global__ void __launch_bounds__(kPromptThreads, 1)
    prompt_attention_kernel(const __grid_constant__ CUtensorMap map_qn, const __grid_constant__ CUtensorMap map_qp,
                            const __grid_constant__ CUtensorMap map_kn, const __grid_constant__ CUtensorMap map_kp,
                            const __grid_constant__ CUtensorMap map_v, PromptParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  PromptBarriers* B = reinterpret_cast<PromptBarriers*>(smem + kOffMisc);
  const uint32_t sbase = smem_u32(smem);
  const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kItemRing; ++i) {
      mbar_init(&B->item_full[i], 1);
      mbar_init(&B->item_empty[i], 11);  // 8 softmax warps, 2 MMA warps, the value producer
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&B->q_full[t], 1);
      mbar_init(&B->q_empty[t], 1);
      mbar_init(&B->k_full[t], 1);
      mbar_init(&B->v_full[t], 1);
      mbar_init(&B->k_empty[t], 2);  // both MMA warps
      mbar_init(&B->v_empty[t], 2);
      mbar_init(&B->s_full[t], 1);
      mbar_init(&B->turn[t], 1);
      mbar_init(&B->drain[t], 1);
      mbar_init(&B->p_rest[t], 4);
      mbar_init(&B->p_full[t], 4);  // one lane of each of the tile's softmax warps
      mbar_init(&B->o_full[t], 1);
      mbar_init(&B->o_free[t], 4);
    }
    B->abort = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(&B->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = B->tmem_base;
  griddep_wait();  // the plan's list
  griddep_launch_dependents();
  const volatile int* abort_flag = &B->abort;
  const int H = p.heads_v, group = (p.heads / p.kv_heads) >> p.pack;  // (packed) heads, and those of a kv head
  // waits for the CTA's n-th unit; false: a wait failed
  auto item_ready = [&](int n) {
    return mbar_wait(&B->item_full[n % kItemRing], (n / kItemRing) & 1, abort_flag, kWaitNs);
  };

  int direct_items = 0;
  if (kDirect && warp == 8) {
    // No plan: this warp lists the sequences, at most 32, in shared memory.
    const bool in = lane < p.num_seqs;
    const int q0 = in ? p.cu_q[lane] : 0, q1 = in ? p.cu_q[lane + 1] : 0;
    const int k0 = in ? p.cu_k[lane] : 0, k1 = in ? p.cu_k[lane + 1] : 0;
    const unsigned bad = __ballot_sync(0xffffffffu, in && bad_offsets(p, q0, q1, k0, k1));
    const int good = bad ? __ffs(bad) - 1 : p.num_seqs;  // sequences from the first bad one on are skipped
    if (blockIdx.x == 0 && lane == 0) *p.status = bad ? MLA_ERR_DEVICE_BOUNDS : MLA_OK;
    int end = lane < good ? blocks_of(p, q1 - q0) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += x;
    }
    B->seqs[lane] = make_int4(q0, q1, k0, k1);
    B->seq_end[lane] = end;
    direct_items = __shfl_sync(0xffffffffu, end, 31);
    __syncwarp();
  }
  if (warp == 8 && lane == 0) {
    // ------------------------------------------------------------ units, key copies
    // Box i (0-2: K, 3-4: V) of key tile j sits at ring position (5 j + i) % 8,
    // last used by box (5 j + i - 8): K_{j-2} for i = 0, V_{j-2} for i = 1, 2,
    // K_{j-1} for i = 3, 4.  j counts the CTA's key tiles over all its items.
    // A thread issues in order and its waits hold back what follows, so the
    // values have their own (warp 11): 0.90 -> 0.86 ms for 16,384 tokens.
    // Units are published two ahead of their loads' end: the MMA warps fetch
    // their next query tile as soon as the last QK of a unit is done.
    bool ok = true;
    uint32_t j = 0;
    // Unit u is item u / H for head u % H.  Each CTA's first is its own number,
    // the others come from a counter: which CTA runs a unit does not change it.
    const int units = (kDirect ? direct_items : p.status[1]) * H;
    // The counter's answer and the item it leads to are each waited for a key
    // tile later: this thread issues in order, and a wait here holds back the
    // copies.
    PromptItem it, next, after;
    int dealt = blockIdx.x;
    auto take = [&]() { return kDirect ? dealt += gridDim.x : int(gridDim.x) + atomicAdd(&p.status[2], 1); };
    auto fetch = [&](int u) {
      PromptItem x;
      x.rows = 0;
      if (u < units) {
        const int i = u / H;
        if (kDirect) {
          int b = 0;  // the first sequence whose blocks end past i
          while (B->seq_end[b] <= i) ++b;
          const int4 q = B->seqs[b];
          x = make_item(p, q.x, q.y, q.z, q.w, b > 0 ? i - B->seq_end[b - 1] : i);
        } else {
          x = load_item(p.items + i);
        }
        x.head = u % H;
      }
      return x;
    };
    auto publish = [&](int n, const PromptItem& x) {
      const int slot = n % kItemRing;
      if (n >= kItemRing && !mbar_wait(&B->item_empty[slot], ((n / kItemRing) - 1) & 1, abort_flag, kWaitNs)) return false;
      B->items[slot] = x;
      mbar_arrive(&B->item_full[slot]);
      return true;
    };
    if (kDirect) {
      it = fetch(blockIdx.x);
    } else {
      it = load_item(p.items + blockIdx.x / H);  // in the list's bounds, if maybe not written: beside the count's load
      it.head = blockIdx.x % H;
      if (int(blockIdx.x) >= units) it.rows = 0;
    }
    ok = publish(0, it);
    int u_after = it.rows > 0 ? take() : units;
    next = fetch(u_after);  // the counter stops at most two past the units for each CTA
    for (int n = 0; ok && it.rows > 0; ++n, it = next, next = after) {
      if (!(ok = publish(n + 1, next))) break;
      u_after = take();
      bool fetched = false;
      if (next.rows > 0) {  // the next unit's queries on their way to L2
        for (int t = 0; 128 * t < next.rows; ++t) {
          tma_prefetch_3d(&map_qn, 0, next.head << p.pack, next.q_row0 + (128 * t >> p.pack));
          tma_prefetch_3d(&map_qn, 64, next.head << p.pack, next.q_row0 + (128 * t >> p.pack));
          tma_prefetch_3d(&map_qp, 0, next.head << p.pack, next.q_row0 + (128 * t >> p.pack));
        }
      }
      const int g = it.head / group;
      const int nt = max(tiles_of(it, 0, p.pack), tiles_of(it, 1, p.pack));
      for (int kt = 0; kt < nt && ok; ++kt, ++j) {
        const int key = it.k_row0 + it.kv_begin + kt * kKeys;
        uint64_t* bar = &B->k_full[j & 1];
        if (j >= 2 && !(ok = mbar_wait(&B->k_empty[j & 1], ((j - 2) >> 1) & 1, abort_flag, kWaitNs))) break;
        mbar_arrive_expect_tx(bar, 3 * kBox + (p.inject_wait_timeout && j == 0 ? 16 : 0));
        tma_load_3d(smem + kOffRing + (5 * j % kRing) * kBox, &map_kn, 0, g, key, bar);
        if (j >= 2 && !(ok = mbar_wait(&B->v_empty[j & 1], ((j - 2) >> 1) & 1, abort_flag, kWaitNs))) {
          ++j;  // one of its boxes is on its way
          break;
        }
        tma_load_3d(smem + kOffRing + ((5 * j + 1) % kRing) * kBox, &map_kn, 64, g, key, bar);
        tma_load_2d(smem + kOffRing + ((5 * j + 2) % kRing) * kBox, &map_kp, 0, key, bar);
        if (!fetched) {
          after = fetch(u_after);
          fetched = true;
        }
      }
      if (!fetched) after = fetch(u_after);
    }
    B->k_tiles = j;
    if (!ok) fail(B, p.status);
  } else if ((warp == 9 || warp == 10) && elect_one()) {
    // ------------------------------------------------------------ MMA issue
    // One warp per query tile t, each with its own chain: QK of the first key
    // tile, then PV of a key tile and QK of the next.  MMAs of one thread run
    // in order, so the QK may overwrite the scores whose P the PV before it
    // reads.
    //
    // The warps take turns, a product pair (PV, next QK) at a time: left to
    // themselves their MMAs interleave and both query tiles come to wait for
    // their softmax at the same time.  The pipe takes only a few MMAs ahead, so
    // whatever a turn does between two MMAs shows: the MMAs are straight-line
    // code, and only warp 9 waits for boxes (the other's turn follows on the same
    // boxes).  The next turn starts when this one's
    // MMAs and commits are issued: four MMAs before that, some of them run behind
    // the next turn's and the tiles' softmaxes come to run at the same time (128
    // heads over 8: 689 us, now 669); once the MMAs are complete, the pipe idles
    // (686).  Both warps pass every key tile, whether their query tile sees it or
    // not.
    //
    // One lane does all of it: a barrier tells a phase's end only until the next
    // phase ends, so a lane that only waited could come too late to see it.  All
    // lanes, meeting before the products of each turn, took 911 us for 16,384
    // tokens where one takes 865.
    const int t = warp - 9;
    constexpr uint32_t id_qk = idesc_bf16_f32(128, 128, false, false);
    constexpr uint32_t id_pv = idesc_bf16_f32(128, 128, false, true), id_pv64 = idesc_bf16_f32(128, 64, false, true);
    constexpr uint64_t kDescK = smem_desc(0, 16, 1024, kSwizzle128B);    // K-major
    constexpr uint64_t kDescMN = smem_desc(0, kBox, 1024, kSwizzle128B); // MN-major, 64-column blocks a box apart
    const uint32_t ds = tmem + kColS + 128 * t, dO = tmem + kColO + 128 * t;
    const uint64_t q_desc = kDescK | desc_addr(sbase + t * kQTile), ring_k = kDescK | desc_addr(sbase + kOffRing),
                   ring_v = kDescMN | desc_addr(sbase + kOffRing);
    bool ok = true;
    uint32_t j = 0, nload = 0, nq = 0, np = 0, no = 0, nturn = 0;
    // turn k of tile 1 follows turn k of tile 0, which follows turn k - 1 of tile 1
    auto take_turn = [&]() {
      const bool w = mbar_wait(&B->turn[t], (nturn & 1) ^ (t ^ 1), abort_flag, kWaitNs);
      ++nturn;
      tc_fence_after();
      return w;
    };
    auto pass_turn = [&]() { mbar_arrive(&B->turn[t ^ 1]); };
    // QK of key tile jj, `sees`: this query tile sees it, `last`: none after it.  Ends the turn.
    auto qk = [&](uint32_t jj, bool sees, bool last) -> bool {
      const uint64_t b0 = ring_k + ((5 * jj) % kRing) * (kBox >> 4), b1 = ring_k + ((5 * jj + 1) % kRing) * (kBox >> 4),
                     b2 = ring_k + ((5 * jj + 2) % kRing) * (kBox >> 4);
      if (t == 0) {
        if (!mbar_wait(&B->k_full[jj & 1], (jj >> 1) & 1, abort_flag, kWaitNs)) return false;
        tc_fence_after();
      }
      if (sees) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) mma_bf16(ds, q_desc + 2 * kk, b0 + 2 * kk, id_qk, kk > 0);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) mma_bf16(ds, q_desc + (kBox >> 4) + 2 * kk, b1 + 2 * kk, id_qk, 1);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) mma_bf16(ds, q_desc + 2 * (kBox >> 4) + 2 * kk, b2 + 2 * kk, id_qk, 1);
        mma_commit(&B->s_full[t]);
        mma_commit(&B->k_empty[jj & 1]);
        pass_turn();
        if (last) mma_commit(&B->q_empty[t]);
      } else {
        pass_turn();
        mbar_arrive(&B->k_empty[jj & 1]);
      }
      return true;
    };
    // this warp's query tile of unit n, once the last QK before it has read the buffer
    auto load_q = [&](int n) -> bool {
      if (!item_ready(n)) return false;
      const PromptItem it = load_item(&B->items[n % kItemRing]);
      if (tiles_of(it, t, p.pack) == 0) return true;
      if (nload > 0 && !mbar_wait(&B->q_empty[t], (nload - 1) & 1, abort_flag, kWaitNs)) return false;
      ++nload;
      uint8_t* q = smem + t * kQTile;
      const int row = it.q_row0 + (128 * t >> p.pack), head = it.head << p.pack;
      mbar_arrive_expect_tx(&B->q_full[t], kQTile);
      tma_load_3d(q, &map_qn, 0, head, row, &B->q_full[t]);
      tma_load_3d(q + kBox, &map_qn, 64, head, row, &B->q_full[t]);
      tma_load_3d(q + 2 * kBox, &map_qp, 0, head, row, &B->q_full[t]);
      return true;
    };
    ok = load_q(0);
    for (int n = 0;; ++n) {
      if (!(ok = ok && item_ready(n))) break;
      const PromptItem it = load_item(&B->items[n % kItemRing]);
      mbar_arrive(&B->item_empty[n % kItemRing]);
      if (it.rows == 0) break;
      const int mine = tiles_of(it, t, p.pack);
      const int nt = max(mine, tiles_of(it, t ^ 1, p.pack));
      const int keys = it.kv_end - it.kv_begin;
      if (mine == 0) ok = load_q(n + 1);
      if (nt == 0 || !ok) continue;
      if (mine > 0) {
        ok = mbar_wait(&B->q_full[t], nq & 1, abort_flag, kWaitNs);
        ++nq;
      }
      if (!(ok = ok && take_turn())) continue;
      ok = qk(j, mine > 0, mine == 1);
      for (int kt = 0; kt < nt && ok; ++kt, ++j) {
        const uint32_t s0 = (5 * j + 3) % kRing;
        const uint64_t v0 = ring_v + s0 * (kBox >> 4);
        ok = t == 1 || mbar_wait(&B->v_full[j & 1], (j >> 1) & 1, abort_flag, kWaitNs);
        const int valid = keys - kt * kKeys;
        if (t == 0 && ok && valid < kKeys && (valid & 15)) {
          // PV reads whole 16-key steps; the rows of the last tile past its
          // last key meet zero weights but must be finite: they are cleared
          // (for the other warp too, whose turn comes later)
          uint8_t* box[2] = {smem + kOffRing + s0 * kBox, smem + kOffRing + ((s0 + 1) % kRing) * kBox};
          for (int row = valid; row < ((valid + 15) & ~15); ++row) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              *reinterpret_cast<uint4*>(box[i >> 3] + row * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        if (ok && kt == mine - 1) ok = load_q(n + 1);  // while the last weights are computed
        if (ok && kt < mine) {
          if (kt == 0 && no > 0) ok = mbar_wait(&B->o_free[t], (no - 1) & 1, abort_flag, kWaitNs);
          ok = ok && mbar_wait(&B->p_full[t], np & 1, abort_flag, kWaitNs);
        }
        if (!(ok = ok && take_turn())) break;
        if (kt < mine) {
          const bool whole = valid >= kKeys && s0 != kRing - 1;
          if (whole) {
#pragma unroll
            for (int kk = 0; kk < 6; ++kk) mma_f16_tmem_a(dO, ds + 8 * kk, v0 + 128 * kk, id_pv, kk > 0 ? 1 : kt);
          }
          if (!(ok = mbar_wait(&B->p_rest[t], np & 1, abort_flag, kWaitNs))) break;
          ++np;
          tc_fence_after();
          if (whole) {
#pragma unroll
            for (int kk = 6; kk < 8; ++kk) mma_f16_tmem_a(dO, ds + 8 * kk, v0 + 128 * kk, id_pv, 1);
          } else {
            const int steps = (min(valid, kKeys) + 15) >> 4;
            if (s0 != kRing - 1) {
              for (int kk = 0; kk < steps; ++kk) mma_f16_tmem_a(dO, ds + 8 * kk, v0 + 128 * kk, id_pv, kt | kk);
            } else {  // the second box wrapped to the ring's start: a product for each
#pragma unroll
              for (int kk = 0; kk < 8; ++kk) {
                if (kk >= steps) break;
                mma_f16_tmem_a(dO, ds + 8 * kk, v0 + 128 * kk, id_pv64, kk > 0 ? 1 : kt);
                mma_f16_tmem_a(dO + 64, ds + 8 * kk, ring_v + 128 * kk, id_pv64, kk > 0 ? 1 : kt);
              }
            }
          }
          mma_commit(&B->v_empty[j & 1]);
          if (kt == mine - 1) mma_commit(&B->o_full[t]);
          if (kt == mine - 1) ++no;
        } else {
          mbar_arrive(&B->v_empty[j & 1]);
        }
        if (kt + 1 < nt) ok = qk(j + 1, kt + 1 < mine, kt + 2 == mine);
        else pass_turn();
      }
    }
    B->q_tiles[t] = nload;
    if (!ok) fail(B, p.status);
    mma_commit(&B->drain[t]);  // every MMA issued completes before teardown
    if (!mbar_wait(&B->drain[t], 0, abort_flag, kWaitNs)) fail(B, p.status);
  } else if (warp == 11 && lane == 0) {
    // ------------------------------------------------------------ value copies
    bool ok = true;
    uint32_t j = 0;
    for (int n = 0; ok; ++n) {
      if (!(ok = item_ready(n))) break;
      const PromptItem it = load_item(&B->items[n % kItemRing]);
      mbar_arrive(&B->item_empty[n % kItemRing]);
      if (it.rows == 0) break;
      const int g = it.head / group;
      const int nt = max(tiles_of(it, 0, p.pack), tiles_of(it, 1, p.pack));
      for (int kt = 0; kt < nt && ok; ++kt, ++j) {
        const int key = it.k_row0 + it.kv_begin + kt * kKeys;
        uint64_t* bar = &B->v_full[j & 1];
        if (j >= 1 && !(ok = mbar_wait(&B->k_empty[(j - 1) & 1], ((j - 1) >> 1) & 1, abort_flag, kWaitNs))) break;
        mbar_arrive_expect_tx(bar, 2 * kBox);
        tma_load_3d(smem + kOffRing + ((5 * j + 3) % kRing) * kBox, &map_v, 0, g, key, bar);
        tma_load_3d(smem + kOffRing + ((5 * j + 4) % kRing) * kBox, &map_v, 64, g, key, bar);
      }
    }
    B->v_tiles = j;
    if (!ok) fail(B, p.status);
  } else if (warp < 8) {
    // ------------------------------------------------------------ softmax, epilogue
    const int t = warp >> 2, r = 32 * (warp & 3) + lane;  // query tile, row = tensor memory lane
    const uint32_t lane_off = uint32_t(32 * (warp & 3)) << 16;
    const uint32_t ts = tmem + lane_off + kColS + 128 * t, to = tmem + lane_off + kColO + 128 * t;
    bool ok = true;
    uint32_t ns = 0, no = 0;
    for (int n = 0; ok; ++n) {
      ok = item_ready(n);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      int nt, vis, vis_first, keys;
      {
        const PromptItem it = load_item(&B->items[n % kItemRing]);
        if (it.rows == 0) break;
        nt = tiles_of(it, t, p.pack);
        vis = it.vis0 + ((128 * t + r) >> p.pack) - it.kv_begin;  // keys of this item's range that the row sees
        vis_first = it.vis0 + (128 * t >> p.pack) - it.kv_begin;
        keys = it.kv_end - it.kv_begin;
      }
      float m = -INFINITY, l = 0.f;
      for (int kt = 0; kt < nt; ++kt) {
        ok = mbar_wait(&B->s_full[t], ns & 1, abort_flag, kWaitNs);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        ++ns;
        tc_fence_after();
        uint32_t s[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32_async(ts + 32 * c, s[c]);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < 4; ++c) tie(s[c]);
        if (kKeys * (kt + 1) > min(vis_first, keys)) {  // some row does not see some key of this tile
          const int lim = min(vis, keys) - kKeys * kt;
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (32 * c + i >= lim) s[c][i] = 0xff800000u;  // -inf
        }
        const float mt = row_max(s);
        float alpha = 1.f;
        bool up = false;
        if (kt == 0) {
          m = mt;
        } else if ((mt - m) * p.scale_log2 > kRescale) {
          alpha = ex2_ftz((m - mt) * p.scale_log2);
          m = mt;
          up = true;
        }
        if (__any_sync(0xffffffffu, up)) {
          // s_full of this tile follows the PV of the tile before: O is complete up to there
          l *= alpha;
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            float o[16];
            tmem_ld16(to + 16 * c, o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] *= alpha;
            tmem_st16(to + 16 * c, o);
          }
        }
        // The MMA thread starts on the first 96 keys while the last 32 are computed.
        const float shift = m == -INFINITY ? 0.f : m * p.scale_log2;  // a row without keys: all weights 0
        const uint64_t scale2 = pack2(p.scale_log2, p.scale_log2), shift2 = pack2(-shift, -shift);
        uint64_t sum[2] = {0, 0};
        auto weights = [&](int c) {
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 x = unpack2(
                fma2(pack2(__uint_as_float(s[c][2 * i]), __uint_as_float(s[c][2 * i + 1])), scale2, shift2));
            const float a = ex2_ftz(x.x), b = ex2_ftz(x.y);
            sum[i & 1] = add2(sum[i & 1], pack2(a, b));
            const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
            w[i] = *reinterpret_cast<const uint32_t*>(&v);
          }
          tmem_st16u(ts + 16 * c, w);
        };
#pragma unroll
        for (int c = 0; c < 3; ++c) weights(c);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&B->p_full[t]);
        weights(3);
        const float2 total = unpack2(add2(sum[0], sum[1]));
        l += total.x + total.y;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&B->p_rest[t]);
      }
      if (!ok) break;
      const PromptItem it = load_item(&B->items[n % kItemRing]);  // not held in registers through the key loop
      __syncwarp();
      if (lane == 0) mbar_arrive(&B->item_empty[n % kItemRing]);
      const int h = it.head, row = 128 * t + r;  // row of the item
      const bool live = row < it.rows;
      const size_t orow = size_t(it.q_row0 + (row >> p.pack)) * p.heads + (h << p.pack) + (row & ((1 << p.pack) - 1));
      if (nt > 0) {
        ok = mbar_wait(&B->o_full[t], no & 1, abort_flag, kWaitNs);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        ++no;
        tc_fence_after();
      }
      if (it.pieces == 1) {
        uint4* dst = reinterpret_cast<uint4*>(p.out + orow * kVDim);
        if (nt > 0) {
          const float inv = inverse_sum(l);
#pragma unroll
          for (int c = 0; c < 4; c += 2) {
            uint32_t o[2][32];
            tmem_ld32_async(to + 32 * c, o[0]);
            tmem_ld32_async(to + 32 * c + 32, o[1]);
            tmem_ld_wait();
            tie(o[0]);
            tie(o[1]);
            if (c == 2) {  // the output is read: the next unit's products may overwrite it
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&B->o_free[t]);
            }
            if (live && l != 0.f) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                st_global_32(dst + 4 * c + 2 * i, pack_out(&o[i >> 1][16 * (i & 1)], inv),
                             pack_out(&o[i >> 1][16 * (i & 1) + 8], inv));
            }
          }
        }
        // A row without keys: its products are 0 times values that other rows
        // see, NaN where those are not finite, so they are not stored.
        if (live && l == 0.f) {
#pragma unroll
          for (int i = 0; i < 16; ++i) dst[i] = make_uint4(0, 0, 0, 0);
        }
        if (live && p.lse_out) p.lse_out[orow] = l == 0.f ? -INFINITY : m * p.scale + logf(l);
      } else {
        // A piece of a split block: its unnormalised output, reference maximum
        // and sum go to the workspace, for the merge.
        const size_t prow = size_t(it.partial) + (size_t(h) * it.pieces + it.piece) * it.rows + row;
        float* dst = p.partial_o + prow * kVDim;
        if (nt > 0) {
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t o[32];
            tmem_ld32(to + 32 * c, o);
            if (live) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                st_global_32(dst + 32 * c + 8 * i, make_uint4(o[8 * i], o[8 * i + 1], o[8 * i + 2], o[8 * i + 3]),
                             make_uint4(o[8 * i + 4], o[8 * i + 5], o[8 * i + 6], o[8 * i + 7]));
            }
          }
        }
        if (live) p.partial_ml[prow] = make_float2(m, l);
      }
      if (nt > 0 && it.pieces > 1) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&B->o_free[t]);
      }
    }
    if (!ok) fail(B, p.status);
  }
  __syncwarp();
  // ---------------------------------------------------------------- teardown
  __syncthreads();
  if (B->abort) {  // products complete, and copies land, before tensor and shared memory are released
    if (threadIdx.x == 0) {
      const uint64_t end = global_timer_ns() + kDrainNs;
      // The last phase of a barrier; the phases before are complete, or it would not have begun.
      auto last = [&](uint64_t* bar, uint32_t phases) {
        if (phases > 0) mbar_wait_until(bar, (phases - 1) & 1, end);
      };
      for (uint32_t i = 0; i < 2; ++i) {
        last(&B->drain[i], 1);
        last(&B->q_full[i], B->q_tiles[i]);
        last(&B->k_full[i], (B->k_tiles + 1 - i) / 2);
        last(&B->v_full[i], (B->v_tiles + 1 - i) / 2);
      }
    }
    __syncthreads();
  }
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

// 3-D map over a [rows, heads, width] bf16 tensor: boxes of 64 columns x `box_heads` heads x as many rows as make 128.
bool make_map_heads(CUtensorMap* m, const void* base, uint64_t width, uint64_t heads, uint64_t rows, uint32_t box_heads) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {width, heads, rows};
  cuuint64_t strides[2] = {width * 2, width * heads * 2};
  cuuint32_t box[3] = {64, box_heads, 128 / box_heads};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ----- merge -----------------------------------------------------------------------
// One warp per (row of a split block, head): out = sum_i w_i O_i / sum_i w_i l_i
// with w_i = 2^((m_i - max m) scale_log2) over the block's pieces, lane i holding
// piece i's m and l, every lane four of the 128 columns.  Pieces without keys for
// the row (l = 0) carry weight 0 and no output.  A merge by the CTA that brought
// the last piece, a row to a thread, took 60 us and more of blocks of 256 rows
// (256 rows behind 8,192 keys at 16 heads: 128 us in all).
constexpr int kMergeThreads = 256;
__global__ void __launch_bounds__(kMergeThreads) prompt_merge_kernel(PromptParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int splits = p.status[3];
  if (splits == 0) return;
  const int rows = p.status[4], lane = threadIdx.x & 31, warps = gridDim.x * (kMergeThreads / 32);
  for (int task = blockIdx.x * (kMergeThreads / 32) + (threadIdx.x >> 5); task < rows * p.heads_v; task += warps) {
    const int h = task / rows, r = task % rows;
    int lo = 0, hi = splits - 1;  // last split block that starts at or before row r
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (p.splits[mid].row_start <= r) lo = mid; else hi = mid - 1;
    }
    const PromptSplit sp = p.splits[lo];
    const int row = r - sp.row_start;
    const size_t prow0 = size_t(sp.partial) + size_t(h) * sp.pieces * sp.rows + row;
    const float2 ml = lane < sp.pieces ? p.partial_ml[prow0 + size_t(lane) * sp.rows] : make_float2(-INFINITY, 0.f);
    float top = ml.y != 0.f ? ml.x : -INFINITY;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float base = top == -INFINITY ? 0.f : top;
    const float w = ml.y != 0.f ? ex2_ftz((ml.x - base) * p.scale_log2) : 0.f;
    float l = ml.y != 0.f ? w * ml.y : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    const unsigned has = __ballot_sync(0xffffffffu, ml.y != 0.f);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = 0; i < sp.pieces; ++i) {
      const float wi = __shfl_sync(0xffffffffu, w, i);
      if (!(has >> i & 1)) continue;
      const float4 x = reinterpret_cast<const float4*>(p.partial_o + (prow0 + size_t(i) * sp.rows) * kVDim)[lane];
      acc.x = fmaf(x.x, wi, acc.x);
      acc.y = fmaf(x.y, wi, acc.y);
      acc.z = fmaf(x.z, wi, acc.z);
      acc.w = fmaf(x.w, wi, acc.w);
    }
    const float inv = inverse_sum(l);
    const size_t orow =
        size_t(sp.q_row0 + (row >> p.pack)) * p.heads + (h << p.pack) + (row & ((1 << p.pack) - 1));
    const __nv_bfloat162 a = __floats2bfloat162_rn(acc.x * inv, acc.y * inv), b = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
    reinterpret_cast<uint2*>(p.out + orow * kVDim)[lane] =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    if (lane == 0 && p.lse_out) p.lse_out[orow] = l == 0.f ? -INFINITY : base * p.scale + logf(l);
  }
}

}  // namespace

cudaError_t launch_prompt_attention(PromptParams p, cudaStream_t stream) {
  CUtensorMap qn, qp, kn, kp, v;
  if (!make_map_heads(&qn, p.q_nope, kNope, p.heads, p.n_q, 1u << p.pack) ||
      !make_map_heads(&qp, p.q_pe, kRope, p.heads, p.n_q, 1u << p.pack))
    return cudaErrorInvalidValue;
  if (p.n_k > 0) {
    if (!make_map_heads(&kn, p.k_nope, kNope, p.kv_heads, p.n_k, 1) ||
        !make_map_heads(&v, p.v, kVDim, p.kv_heads, p.n_k, 1) ||
        !make_map_2d(&kp, p.k_pe, 2, kRope, p.n_k, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  } else {
    kn = kp = v = qn;  // no keys: no key tile is ever loaded
  }
  static std::atomic<bool> attr[128];  // per device: attributes set (zero-initialised)
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 128 || !attr[dev]) {
    for (auto* k : {prompt_attention_kernel<false>, prompt_attention_kernel<true>}) {
      const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmem));
      if (e != cudaSuccess) return e;
    }
    if (dev >= 0 && dev < 128) attr[dev] = true;
  }
  const long long blocks = ((long long)p.n_q << p.pack) / kPromptRows + p.num_seqs;  // at most
  const long long most = blocks * kPromptMaxPieces * p.heads_v;                      // units
  const unsigned grid = unsigned(most < p.sm_count ? most : p.sm_count);
  // No plan where it would cost more than it can save: two rounds of units at
  // most with no block long enough to split, or one round that fills more than
  // two thirds of the SMs (half a unit more to each SM would be a second round)
  // over few keys.  93 tokens at 16 heads: 11 us without, 12.7 with one; 2,048
  // tokens: 34 and 39 us.  The bound on the keys (the rows of nine blocks, so that
  // one prompt without a history stays below it) is there because the lengths
  // are on the device, and one sequence may hold most keys.  Eight single tokens
  // at 16 heads, contexts equal and all but one of 16 keys: 2,304 keys take 11
  // and 33 us without a plan, 16 and 21 with one; 8,192 keys 19 and 101, 24 and 30.
  const long long whole = blocks * p.heads_v;
  if (p.num_seqs <= kDirectSeqs &&
      ((whole <= 2 * p.sm_count && p.n_k <= kMinSplit * kKeys) ||
       (whole <= p.sm_count && 3 * whole > 2 * p.sm_count && p.n_k <= kDirectTiles * kKeys)))
    return launch_pdl(prompt_attention_kernel<true>, dim3(grid), dim3(kPromptThreads), kSmem, stream, 1, qn, qp, kn, kp,
                      v, p);
  // Splitting keys is for calls whose query rows make two rounds at most, and
  // with keys to split (rows that cu_q leaves out count, too: the lengths are on
  // the device); only they launch the merge.
  p.may_split = (((long long)p.n_q << p.pack) / kPromptRows) * p.heads_v <= 2 * p.sm_count && p.n_k > kMinSplit * kKeys;
  const bool few = p.may_split && whole <= 2 * p.sm_count && blocks <= kFewPlan;
  cudaError_t e = few ? launch_pdl(prompt_plan_kernel<kFewPlan>, dim3(1), dim3(kFewPlan), 0, stream, 1, p)
                      : launch_pdl(prompt_plan_kernel<kPlanThreads>, dim3(1), dim3(kPlanThreads), 0, stream, 1, p);
  if (e != cudaSuccess) return e;
  e = launch_pdl(prompt_attention_kernel<false>, dim3(grid), dim3(kPromptThreads), kSmem, stream, 1, qn, qp, kn, kp, v, p);
  if (e != cudaSuccess || !p.may_split) return e;
  const long long merges = ((long long)p.n_q * p.heads + kMergeThreads / 32 - 1) / (kMergeThreads / 32);  // at most
  return launch_pdl(prompt_merge_kernel, dim3(unsigned(merges < 8 * p.sm_count ? merges : 8 * p.sm_count)),
                    dim3(kMergeThreads), 0, stream, 1, p);
}

}  // namespace mla
