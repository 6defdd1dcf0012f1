// Attention of new tokens over the paged INT4 KV cache (include/q4_attn.h).
//
//   o = sum_t softmax_t(scale * q . k_t) v_t,  k_t = ks_t * kc_t, v_t = vs_t * vc_t
//
// with codes c in [-8, 7] and one float16 scale s per token and group of channels. The
// scales never touch the codes: a K scale multiplies the group's dot product, a V scale
// the token's softmax weight, so the matrix instructions run on exact float16 integers.
//
// Rows. The query heads that share a KV head read the same keys, so a sequence's rows
// for one KV head are its new tokens times those heads: row m is token m / share, head
// m % share. A wavefront owns QT tiles of 16 rows and walks the keys 32 at a time in
// one pass, with the running maximum, the sum and the unnormalised output of each row
// in registers (float32).
//
// Operands (v_mfma_f32_16x16x32_f16; lane = col + 16 c).
//   S^T[key][row]  = K[key][channel] Q^T: A is a K tile as it lies in the cache, B the
//     queries. A lane ends up with keys 4c .. 4c + 3 of two 16-key tiles for row col.
//   O^T[channel][row] += V^T[channel][key] P^T[key][row]: B wants 8 keys per lane, and
//     any order of keys serves as long as A uses the same one. Taking the lane's own
//     eight (4c + i of tile 0, then of tile 1) makes the scores the operand without a
//     shuffle; the cache keeps V in that order.
//
// Maximum. All that has to hold is that the weights neither overflow nor vanish, so the
// held maximum m is raised (a reduction over the row's four lanes, a rescaling of l and O)
// only when some score exceeds it by more than kSlack binades: after a row's first few
// steps almost never.
//
// Split. In the first two kernels the four wavefronts of a workgroup have the same rows and
// take every fourth step of its keys, joined in LDS; the keys of all sequences and heads are
// cut into equal shares, one for each workgroup that fits on the chip (below), and a second
// kernel joins the partial results (O, m + E, l in float32) of what was cut, in order. In
// the third each wavefront has rows of its own, and only the jobs of the last, partly
// filled round of the chip are cut.
//
// What bounds it. Few rows: vector work between the loads (16.6 instructions a product: conversion,
// scales, softmax) and the join's launch: 48 rows over 8K contexts of 8 heads at 128 channels, 276 MB,
// in 63 to 66 us, 4.2 to 4.4 TB/s, where a plain read of as many bytes takes 40 us. Many rows:
// the matrix products and, beside them on the same issue ports, the vector work of the softmax and the
// conversion: four 509-token chunks in contexts of up to 8190 tokens, 64 heads over 8, 430 GFLOP, in 512
// to 541 us, 16 of them in 1420 us: 800 to 870 TFLOP/s (an 8192^3 library product in float16: 1148).
// Calls that mix long chunks with single tokens: one form serves the whole call (pick_attn), and in 128-row
// workgroups a single token's context is walked by one workgroup a KV head.
//
// Range of the weights. P = p * vs is rounded to float16 before the product (half a
// step, 2^-11 of each weight; its errors are independent and average over the keys).
// p lies in [0, 1] relative to the row's maximum, but vs can be anything a float16
// can be, and small products would fall among the subnormals. The exponent is
// therefore taken relative to m + E, E the exponent of the largest V scale so far minus
// kHeadroom: P stays in [0, 2^(kHeadroom + kSlack)], 26 binades of full precision below its
// maximum. (Infinite scales do not count: their rows are not finite, others' unharmed.)
// The sum l carries the same factor, so it cancels in o = O / l.
#include <algorithm>

#include "q4_paged.h"

namespace q4 {
namespace {

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

constexpr int kStep = 2 * kTokTile;  // keys per step (MFMA K of the second product)
constexpr float kHeadroom = 12.0f;
constexpr float kSlack = 3.0f;  // binades a score may exceed the held maximum by
constexpr float kLowest = -3.4028234663852886e38f;

__device__ __forceinline__ float4_t mfma(half8_t a, half8_t b, float4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }
__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

// Larger halves of two pairs of unsigned 16-bit numbers.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  typedef uint16_t us2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(us2, a), __builtin_bit_cast(us2, b)));
}

// Eight codes of the K operand, exact: a score then rounds relative to its own terms. (Codes that keep
// an offset, taken off again through the accumulator's start value, are three instructions
// shorter: 63.8 us against 65.7 for 48 rows over 8K contexts. But the accumulator then rounds relative to
// the offset times the sum of q, and scores small next to that moved the output by up to 7
// times its other errors. The start values' registers were worth as much: 43.4 -> 41.6 us for eight
// sequences of 5 rows.)
__device__ __forceinline__ half8_t k_operand(uint32_t w, const DequantRegs& k) {
  const half2_t lo_bias = {(_Float16)-1032.0f, (_Float16)-1032.0f};
  const half2_t hi_bias = {(_Float16)-72.0f, (_Float16)-72.0f};
  return dequant8r(w, k, lo_bias, hi_bias);
}

// Eight codes of the V operand: four tokens of each of two tiles. HI picks the channel
// in the high nibble.
template <bool HI>
__device__ __forceinline__ half8_t v_operand(uint32_t w0, uint32_t w1, const DequantRegs& k) {
  const half2_t lo_bias = {(_Float16)-1032.0f, (_Float16)-1032.0f};
  const half2_t hi_bias = {(_Float16)-72.0f, (_Float16)-72.0f};
  const half2_t sixteenth = {(_Float16)0.0625f, (_Float16)0.0625f};
  auto pair = [&](uint32_t w) __attribute__((always_inline)) {
    return HI ? __builtin_elementwise_fma(as_half2((w & k.hi) | k.magic), sixteenth, hi_bias)
              : as_half2((w & k.lo) | k.magic) + lo_bias;
  };
  const half2_t p0 = pair(w0), p1 = pair(w0 >> 8), p2 = pair(w1), p3 = pair(w1 >> 8);
  const half4_t a = __builtin_shufflevector(p0, p1, 0, 1, 2, 3);
  const half4_t b = __builtin_shufflevector(p2, p3, 0, 1, 2, 3);
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Raw codes and scales of one 16-key tile, as a lane holds them.
template <int D, int GC>
struct Tile {
  uint32_t k[D / 32], v[D / 32];
  uint2 ks[GC], vs[GC];
};

// ONCE: read by this workgroup alone, so not to be kept (nontemporal).
template <int D, bool ONCE = false>
__device__ __forceinline__ void load_codes(uint32_t (&w)[D / 32], const uint32_t* base, int lane) {
  auto get = [](auto* p) __attribute__((always_inline)) {
    if constexpr (ONCE) return __builtin_nontemporal_load(p);
    return *p;
  };
  if constexpr (D == 64) {
    const auto r = get(reinterpret_cast<const u32x2_t*>(base + 2 * lane));
    w[0] = r[0], w[1] = r[1];
  } else {
#pragma unroll
    for (int i = 0; i < D / 128; ++i) {
      const auto r = get(reinterpret_cast<const u32x4_t*>(base + (i * kWave + lane) * 4));
      w[4 * i] = r[0], w[4 * i + 1] = r[1], w[4 * i + 2] = r[2], w[4 * i + 3] = r[3];
    }
  }
}

// `tile` of the cache (D * 8 bytes of codes, GC * 16 scales, for K and for V).
template <int D, int GC, bool ONCE>
__device__ __forceinline__ void load_tile(Tile<D, GC>& t, const PagedArgs& c, int64_t tile, int lane) {
  load_codes<D, ONCE>(t.k, static_cast<const uint32_t*>(c.k_codes) + tile * (2 * D), lane);
  load_codes<D, ONCE>(t.v, static_cast<const uint32_t*>(c.v_codes) + tile * (2 * D), lane);
  const uint16_t* ks = static_cast<const uint16_t*>(c.k_scales) + tile * (GC * kTokTile) + 4 * (lane >> 4);
  const uint16_t* vs = static_cast<const uint16_t*>(c.v_scales) + tile * (GC * kTokTile) + 4 * (lane >> 4);
#pragma unroll
  for (int g = 0; g < GC; ++g) {
    t.ks[g] = *reinterpret_cast<const uint2*>(ks + g * kTokTile);
    t.vs[g] = *reinterpret_cast<const uint2*>(vs + g * kTokTile);
  }
}

// Read-only int32 arrays at uniform indexes go through the scalar cache: a vector load
// would have to be waited for behind the tile loads issued before it (they return in
// order), which would leave none in flight.
typedef const __attribute__((address_space(4))) int32_t* ScalarInts;
__device__ __forceinline__ ScalarInts scalar_ints(const int32_t* p) { return (ScalarInts)(uintptr_t)p; }

// What a workgroup works on.
struct Job {
  int first, rows, len, nq;  // the sequence's first row of q, rows = nq * share, length
  int seq, head, share;
};

__device__ __forceinline__ bool make_job(const AttnArgs& a, int seq, int head, Job* w) {
  // kept inside what the arguments promise
  w->seq = seq;
  w->head = head;
  w->share = __builtin_amdgcn_readfirstlane(a.q_heads / a.cache.kv_heads);
  const ScalarInts offsets = scalar_ints(a.q_offsets);
  w->first = min(max(offsets[seq], 0), a.tokens);
  w->nq = min(min(max(offsets[seq + 1], w->first), a.tokens) - w->first, a.max_q);
  w->len = min(max(scalar_ints(a.kv_lens)[seq], 0), a.max_kv);
  w->rows = w->nq * w->share;
  return w->rows > 0;
}

// Keys that rows r0 .. r0 + n - 1 see: [first (a multiple of kStep), last).
struct Span {
  int pos_lo, pos_hi, window, first, last;
};

__device__ __forceinline__ Span span_of(const AttnArgs& a, const Job& w, int r0, int n) {
  Span s;
  s.pos_lo = w.len - w.nq + __builtin_amdgcn_readfirstlane(r0 / w.share);
  s.pos_hi = w.len - w.nq + __builtin_amdgcn_readfirstlane((min(r0 + n, w.rows) - 1) / w.share);
  s.last = s.pos_hi + 1;
  s.window = a.window > 0 ? a.window : s.last + 1;
  s.first = max(0, s.pos_lo - s.window + 1) / kStep * kStep;
  return s;
}

// Walks 16-key tiles of a sequence's pages without a division per step (all scalar).
struct Walk {
  int tile, block, in_page;  // tile of the sequence, its page table entry, tile of the page
};

// Float16 row from sums: zeros where the row saw no key (sum 0). A part of a row that saw keys at scores of
// -infinity only carries a sum below 0, at the lowest base: any other key outweighs it, and where
// there is none the row is NaN, as its softmax is.
__device__ __forceinline__ uint2 to_row(float4_t o, float sum) {
  const float inv = sum > 0.0f ? 1.0f / sum : sum == 0.0f ? 0.0f : __builtin_nanf("");
  half4_t h;
#pragma unroll
  for (int e = 0; e < 4; ++e) h[e] = (_Float16)(o[e] * inv);
  return __builtin_bit_cast(uint2, h);
}

// Address of channel ch of row `row` of a job in the output.
template <int D>
__device__ __forceinline__ uint2* out_at(const AttnArgs& a, const Job& w, int row, int ch) {
  const int i = row / w.share, hs = row - i * w.share;
  const int64_t r = (int64_t)(w.first + i) * a.q_heads + w.head * w.share + hs;
  return reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + r * D + ch);
}

// ---------------------------------------------------------------------------------
// Work shares. Where the wavefronts of a workgroup split the keys, a job (RG rows of a sequence
// and KV head) is cut into units of 128 keys, all jobs' units form one line (sequence,
// row tile, head, keys), and each of the resident workgroups takes an equal share of it: the
// chip is full to the end whatever the lengths are, which only the device knows. A share
// may begin and end inside a job; those two pieces are partial results (slot 0: the piece
// does not begin its job, slot 1: it begins it and is cut), the jobs between are whole.
constexpr int kUnit = 128;
constexpr int kMinUnits = 4;  // units a share has at least: fewer workgroups for little work

struct SeqWork {
  int units, tiles, key0;  // units of a job, row tiles, first key (a multiple of kStep)
};

__device__ __forceinline__ SeqWork seq_work(const AttnArgs& a, int nq, int len, int rows, int rg) {
  SeqWork s;
  const int window = a.window > 0 ? a.window : len + 1;
  s.key0 = max(0, len - nq - window + 1) / kStep * kStep;
  s.units = max(1, (max(len - s.key0, 0) + kUnit - 1) / kUnit);
  s.tiles = (rows + rg - 1) / rg;
  return s;
}

// Units of the sequences `base + lane`.
__device__ __forceinline__ int64_t lane_work(const AttnArgs& a, int seq, int rg) {
  if (seq >= a.seqs) return 0;
  const int first = min(max(a.q_offsets[seq], 0), a.tokens);
  const int nq = min(min(max(a.q_offsets[seq + 1], first), a.tokens) - first, a.max_q);
  const int len = min(max(a.kv_lens[seq], 0), a.max_kv);
  const SeqWork s = seq_work(a, nq, len, nq * (a.q_heads / a.cache.kv_heads), rg);
  return (int64_t)s.tiles * a.cache.kv_heads * s.units;
}

// Values that are the same in every lane but were computed on the vector unit (divisions, lane
// operations), moved to scalar registers: addresses and branches made of them then stay scalar.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform64(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32));
  return (int64_t)((uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ int64_t total_work(const AttnArgs& a, int rg, int lane) {
  long long sum = 0;
  for (int base = 0; base < a.seqs; base += kWave) sum += lane_work(a, base + lane, rg);
#pragma unroll
  for (int m = 1; m < kWave; m <<= 1) sum += __shfl_xor(sum, m, 64);
  return uniform64(sum);
}

// The sequence that holds unit `unit` (below the total), and the units before it.
__device__ __forceinline__ int find_seq(const AttnArgs& a, int rg, int lane, int64_t unit, int64_t* before) {
  long long acc = 0;
  for (int base = 0; base < a.seqs; base += kWave) {
    const long long own = lane_work(a, base + lane, rg);
    long long incl = own;
#pragma unroll
    for (int m = 1; m < kWave; m <<= 1) {
      const long long up = __shfl_up(incl, m, 64);
      if (lane >= m) incl += up;
    }
    const uint64_t past = __ballot(acc + incl > unit);
    if (past) {
      const int at = __builtin_ctzll(past);
      *before = uniform64(acc + __shfl(incl - own, at, 64));
      return base + at;
    }
    acc += __shfl(incl, kWave - 1, 64);
  }
  *before = acc;  // not reached
  return a.seqs - 1;
}

__device__ __forceinline__ int64_t shares_of(const AttnArgs& a, int64_t total) {
  const int64_t want = total / kMinUnits;
  return uniform64(want < 1 ? 1 : want < a.shares ? want : a.shares);
}

// One piece of work: rows r0 .. of a job, keys [key0, key1) of it (key1 < 0: to the end);
// slot < 0: the whole job.
struct Piece {
  Job w;
  int r0, key0, key1, slot;
};

// `p` with every field in scalar registers.
__device__ __forceinline__ Piece uniform_piece(const Piece& p) {
  return Piece{Job{uniform(p.w.first), uniform(p.w.rows), uniform(p.w.len), uniform(p.w.nq), uniform(p.w.seq),
                   uniform(p.w.head), uniform(p.w.share)},
               uniform(p.r0), uniform(p.key0), uniform(p.key1), uniform(p.slot)};
}

struct Shares {
  int64_t at, end, total, count;
  int64_t before, seq_end;  // units before the current sequence and before the next
  int64_t cut_end;          // end of the job this share begins and does not end (0: none)
  Job w;
  SeqWork s;
  bool whole;  // no shares: one job a workgroup

  __device__ __forceinline__ void enter(const AttnArgs& a, int rg, int seq) {
    make_job(a, seq, 0, &w);
    s = seq_work(a, w.nq, w.len, w.rows, rg);
    seq_end = before + (int64_t)s.tiles * a.cache.kv_heads * s.units;
  }

  __device__ __forceinline__ bool begin(const AttnArgs& a, int rg, int lane) {
    whole = a.shares == 0;
    if (whole) {
      at = blockIdx.x;
      return true;
    }
    long long own = 0, incl = 0;
    if (a.seqs <= kWave) {  // one pass finds the total and the place
      own = incl = lane_work(a, lane, rg);
#pragma unroll
      for (int m = 1; m < kWave; m <<= 1) {
        const long long up = __shfl_up(incl, m, 64);
        if (lane >= m) incl += up;
      }
      total = uniform64(__shfl(incl, kWave - 1, 64));
    } else {
      total = total_work(a, rg, lane);
    }
    count = shares_of(a, total);
    cut_end = 0;
    if ((int64_t)blockIdx.x >= count) return false;
    at = uniform64((int64_t)blockIdx.x * total / count);
    end = uniform64(((int64_t)blockIdx.x + 1) * total / count);
    if (at >= end) return false;
    int seq;
    if (a.seqs <= kWave) {
      seq = __builtin_ctzll(__ballot(incl > at));
      before = uniform64(__shfl(incl - own, seq, 64));
    } else {
      seq = find_seq(a, rg, lane, at, &before);
    }
    enter(a, rg, uniform(seq));
    return true;
  }

  __device__ __forceinline__ bool next(const AttnArgs& a, int rg, int lane, int tiles, Piece* p) {
    if (whole) {
      if (at < 0) return false;
      const unsigned j = (unsigned)at, heads = (unsigned)a.cache.kv_heads;
      at = -1;
      const int group = uniform((int)(j / heads));
      const int seq = uniform((int)((unsigned)group / (unsigned)tiles));
      if (!make_job(a, seq, (int)j - group * (int)heads, &p->w)) return false;
      p->r0 = (group - seq * tiles) * rg;
      p->key0 = 0;
      p->key1 = -1;
      p->slot = -1;
      return p->r0 < p->w.rows;
    }
    if (at >= end) return false;
    if (at >= seq_end) {
      const int seq = find_seq(a, rg, lane, at, &before);
      enter(a, rg, uniform(seq));
    }
    const int64_t off = at - before;
    const int64_t job = uniform64(off / s.units);
    const int k0 = (int)(off - job * s.units);
    const int k1 = (int)(s.units - k0 < end - at ? s.units : k0 + (end - at));
    const int tile = uniform((int)(job / a.cache.kv_heads));
    p->w = w;
    p->w.head = (int)(job - (int64_t)tile * a.cache.kv_heads);
    p->r0 = tile * rg;
    p->key0 = s.key0 + k0 * kUnit;
    p->key1 = k1 == s.units ? -1 : s.key0 + k1 * kUnit;
    p->slot = k0 == 0 && k1 == s.units ? -1 : k0 > 0 ? 0 : 1;
    if (p->slot == 1) cut_end = at + s.units;
    at += k1 - k0;
    return true;
  }

  // For the join: the job that this share begins and does not end, and its pieces.
  __device__ __forceinline__ void finish(const AttnArgs& a, const Piece& last) const {
    if (whole || threadIdx.x != 0) return;
    const int n = cut_end > 0 ? (int)((cut_end * count - 1) / total) - (int)blockIdx.x + 1 : 0;
    int4* to = reinterpret_cast<int4*>(a.cuts) + 2 * blockIdx.x;
    to[0] = make_int4(n, last.w.first, last.w.rows, last.w.head);
    to[1] = make_int4(last.r0, 0, 0, 0);
  }
};

// Channels ch .. ch + 3 of a piece's row r0 + local: the output, or the piece's slot.
template <int D, int RG>
__device__ __forceinline__ void store_piece(const AttnArgs& a, const Piece& p, int local, int ch, float4_t o, float sum,
                                            float base) {
  if (p.slot < 0) {
    if (p.r0 + local < p.w.rows) *out_at<D>(a, p.w, p.r0 + local, ch) = to_row(o, sum);
    return;
  }
  const int64_t at = ((int64_t)blockIdx.x * 2 + p.slot) * RG + local;
  *reinterpret_cast<float4_t*>(a.part_o + at * D + ch) = o;
  if (ch == 0) *reinterpret_cast<float2*>(a.part_ml + 2 * at) = make_float2(base, sum);
}

template <int D, int GC>
struct Attn {
  static constexpr int KB = D / 32;    // 32-channel blocks
  static constexpr int BPG = KB / GC;  // of them per scale group
  // Steps of 32 keys a wavefront has in registers (one computed, the other in flight; three and
  // four stages were 3 us slower at 48 x 8K keys), and wavefronts per SIMD the registers are
  // budgeted for (three with two stages spill at 128 channels: 68 -> 86 us). What is spilled with these
  // budgets: 2 registers at 64 channels in two groups, 7 at 256 in eight.
  static constexpr int kStages = 2;
  static constexpr int kWavesSimd = D == 64 ? 3 : D == 128 ? 2 : 1;

  struct Step {
    Tile<D, GC> t[2];
    bool there[2];
  };
};

// At most 16 rows: all four wavefronts have the same ones and split the keys.
//
// ONCE: no other row tile reads these keys, so their codes are loaded past the caches' normal
// order. Caches larger than the last-level cache gain (48 rows over 8K contexts of 8 heads 69.5
// -> 64.2 us, 128 rows 152.8 -> 142.6), 100 MB read again and again lose (35.4 -> 37.6), which a
// model of many layers never does; three tiles over the same keys lose too (78 -> 83 us at 256
// channels) and load normally.
template <int D, int GC, bool ONCE>
__global__ __launch_bounds__(256, (Attn<D, GC>::kWavesSimd)) void attn16_kernel(AttnArgs a, int tiles) {
  using C = Attn<D, GC>;
  using Step = typename C::Step;
  constexpr int KB = C::KB, BPG = C::BPG;
  __shared__ float4_t buf[4][2 * KB][kWave];
  __shared__ float2 ml[4][16];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, c4 = lane >> 4;
  const float scale = a.scale * 1.4426950408889634f;
  const DequantRegs dq = DequantRegs::make();
  const int tpp = a.cache.page_size / kTokTile;
  constexpr int kStride = 8;  // tiles from one step of a wavefront to the next
  const int stride_block = kStride / tpp, stride_rem = kStride - stride_block * tpp;
  Shares shares;
  Piece pc{};
  bool more = uniform(shares.begin(a, 16, lane));
  for (bool again = false; more; again = true) {
    Piece next_piece;
    if (!uniform(shares.next(a, 16, lane, tiles, &next_piece))) break;
    pc = uniform_piece(next_piece);
    if (again) __syncthreads();  // buf of the piece before has been read
    const Job& w = pc.w;

    const int row = pc.r0 + col;
    half8_t q[KB];
    int pos;  // position of the lane's row: its own last visible key; -1: no row
    {
      const int i = min(row, w.rows - 1) / w.share, hs = min(row, w.rows - 1) - i * w.share;
      pos = row < w.rows ? w.len - w.nq + i : -1;
      const uint16_t* src = static_cast<const uint16_t*>(a.q) + (int64_t)(w.first + i) * a.q_stride +
                            (int64_t)(w.head * w.share + hs) * D + 8 * c4;
#pragma unroll
      for (int b = 0; b < KB; ++b) q[b] = as_half8(*reinterpret_cast<const uint4*>(src + 32 * b));
    }
    // base: m + E. A score more than `limit` above it makes m rise; a row that has seen no key
    // yet has base 0 and limit -infinity, and its first key sets m.
    float base = 0.0f, limit = -__builtin_inff(), l = 0.0f;
    bool low = false;  // keys seen at -infinity while no score was above it
    float4_t acc[2 * KB];
#pragma unroll
    for (int b = 0; b < 2 * KB; ++b) acc[b] = float4_t{0.f, 0.f, 0.f, 0.f};

    const Span sp = span_of(a, w, pc.r0, 16);
    const int t_first = max(pc.key0, sp.first);
    const int t_last = pc.key1 < 0 ? sp.last : min(sp.last, pc.key1);
    const ScalarInts table = scalar_ints(a.block_table + (int64_t)w.seq * a.max_blocks);
    float exp_v = -64.0f;  // E (wave-uniform)
    uint32_t cap_v = 0;    // largest V scale that E covers, as float16 bits

    const int last_tile = max(t_last - 1, 0) / kTokTile;
    Walk next;
    next.tile = t_first / kTokTile + 2 * wave;
    next.block = next.tile / tpp;
    next.in_page = next.tile - next.block * tpp;
    int page[2];   // page numbers of `next`'s two tiles
    int in_page2;  // and where the second lies in its page
    auto fetch_pages = [&]() __attribute__((always_inline)) {
      const bool wraps = next.in_page + 1 == tpp;
      in_page2 = wraps ? 0 : next.in_page + 1;
      const int b2 = next.block + (wraps ? 1 : 0);
      // entries behind the last key's are not read
      page[0] = next.tile <= last_tile && next.block < a.max_blocks ? table[next.block] : -1;
      page[1] = next.tile + 1 <= last_tile && b2 < a.max_blocks ? table[b2] : -1;
    };
    // Loads of the step at `next`, which then moves on. A tile behind the last key or of a
    // page outside the cache is read from page 0 and masked.
    auto load = [&](Step& s) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        s.there[j] = (unsigned)page[j] < (unsigned)a.cache.pages;
        const int64_t tile =
            ((int64_t)(s.there[j] ? page[j] : 0) * a.cache.kv_heads + w.head) * tpp + (j ? in_page2 : next.in_page);
        load_tile<D, GC, ONCE>(s.t[j], a.cache, tile, lane);
      }
      next.tile += kStride;
      next.block += stride_block;
      next.in_page += stride_rem;
      if (next.in_page >= tpp) {
        next.in_page -= tpp;
        ++next.block;
      }
      fetch_pages();
    };

    auto compute = [&](Step& st, int t0) __attribute__((always_inline)) {
      const bool edge = t0 + kStep > sp.pos_lo + 1 || t0 <= sp.pos_hi - sp.window || t0 + kStep > t_last ||
                        !st.there[0] || !st.there[1];
      auto key_of = [&](int e) __attribute__((always_inline)) { return t0 + 16 * (e >> 2) + 4 * c4 + (e & 3); };
      // scores, base 2, relative to m + E
      float s[8];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int g = 0; g < GC; ++g) {
          float4_t part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int b = g * BPG; b < (g + 1) * BPG; ++b) part = mfma(k_operand(st.t[j].k[b], dq), q[b], part);
          const half4_t kh = __builtin_bit_cast(half4_t, st.t[j].ks[g]);
#pragma unroll
          for (int i = 0; i < 4; ++i)  // one v_fma_mix
            s[4 * j + i] = __builtin_fmaf(part[i], (float)kh[i], g == 0 ? 0.0f : s[4 * j + i]);
        }
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] = __builtin_fmaf(s[e], scale, -base);
      uint32_t hidden = 0;  // keys of the lane that its row does not see
      if (edge) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int key = key_of(e);
          if (!st.there[e >> 2] || key >= t_last || key > pos || key <= pos - sp.window) {
            s[e] = -__builtin_inff();
            hidden |= 1u << e;
          }
        }
        // what no row sees may hold anything: 0 * NaN must not arise
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int g = 0; g < GC; ++g) {
            half4_t vh = __builtin_bit_cast(half4_t, st.t[j].vs[g]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int key = key_of(4 * j + i);
              vh[i] = st.there[j] && key < t_last && key > sp.pos_lo - sp.window ? vh[i] : (_Float16)0.0f;
            }
            st.t[j].vs[g] = __builtin_bit_cast(uint2, vh);
          }
      }
      // E, where a V scale exceeds what it covers
      uint32_t vmax = 0;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int g = 0; g < GC; ++g) vmax = max_u16x2(vmax, max_u16x2(st.t[j].vs[g].x, st.t[j].vs[g].y));
      vmax = max(vmax & 0xFFFFu, vmax >> 16);
      if (__any(vmax > cap_v)) {
        // the largest finite one, up to the end of its binade
        vmax = cap_v;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int g = 0; g < GC; ++g)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t bits = ((i < 2 ? st.t[j].vs[g].x : st.t[j].vs[g].y) >> (16 * (i & 1))) & 0xFFFFu;
              vmax = max(vmax, bits < 0x7C00u ? bits : 0u);
            }
#pragma unroll
        for (int i = 1; i < 64; i <<= 1) vmax = max(vmax, (uint32_t)__shfl_xor((int)vmax, i, 64));
        cap_v = vmax | 0x3FFu;
        const float up = (float)(int)(cap_v >> 10) - 14.0f - kHeadroom - exp_v, alpha = exp2_fast(-up);
        exp_v += up;
        if (limit > -__builtin_inff()) {
          base += up;
          limit = kSlack - exp_v;
          l *= alpha;
#pragma unroll
          for (int c = 0; c < 2 * KB; ++c) acc[c] *= alpha;
#pragma unroll
          for (int e = 0; e < 8; ++e) s[e] -= up;
        }
      }
      // a score far above its row's held maximum?
      float mx = fmaxf(max3(max3(s[0], s[1], s[2]), s[3], s[4]), max3(s[5], s[6], s[7]));
      if (__any(mx >= limit)) {
        mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
        mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
        if (mx > -__builtin_inff()) {
          const bool first = limit == -__builtin_inff();
          const float up = first ? mx + exp_v : fmaxf(mx + exp_v, 0.0f);
          const float alpha = first ? 1.0f : exp2_fast(-up);
          base += up;
          limit = kSlack - exp_v;
          l *= alpha;
#pragma unroll
          for (int c = 0; c < 2 * KB; ++c) acc[c] *= alpha;
#pragma unroll
          for (int e = 0; e < 8; ++e) s[e] -= up;
        } else if (limit == -__builtin_inff()) {
          low |= hidden != 0xFFu;
        }
      }
      // weights, to float16 with the V scale in them
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s[e] = exp2_fast(s[e]);
        l += s[e];
      }
      half8_t p[GC];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int g = 0; g < GC; ++g) {
          const half4_t vh = __builtin_bit_cast(half4_t, st.t[j].vs[g]);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            p[g][4 * j + i] = (_Float16)__builtin_fmaf(s[4 * j + i], (float)vh[i], 0.0f);  // one v_fma_mix
        }
      if (edge) {
        // a key that one row sees and another does not may have an infinite scale
#pragma unroll
        for (int g = 0; g < GC; ++g)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (hidden >> e & 1u) p[g][e] = (_Float16)0.0f;
      }
#pragma unroll
      for (int b = 0; b < KB; ++b) {
        acc[2 * b] = mfma(v_operand<false>(st.t[0].v[b], st.t[1].v[b], dq), p[b / BPG], acc[2 * b]);
        acc[2 * b + 1] = mfma(v_operand<true>(st.t[0].v[b], st.t[1].v[b], dq), p[b / BPG], acc[2 * b + 1]);
      }
    };

    // kStages - 1 steps in flight while one is computed
    const int t_own = t_first + kStep * wave;
    if (t_own < t_last) {
      Step ring[C::kStages];
      fetch_pages();
#pragma unroll
      for (int i = 0; i + 1 < C::kStages; ++i) load(ring[i]);
      for (int t0 = t_own; t0 < t_last;) {
#pragma unroll
        for (int i = 0; i < C::kStages; ++i) {
          load(ring[(i + C::kStages - 1) % C::kStages]);
          if (t0 < t_last) compute(ring[i], t0);
          t0 += kStride * kTokTile;
        }
      }
    }
    if (low && limit == -__builtin_inff()) l -= 1.0f;
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);
    if (limit == -__builtin_inff()) base = kLowest;

    // the four wavefronts' parts of the same rows, added in order
#pragma unroll
    for (int c = 0; c < 2 * KB; ++c) buf[wave][c][lane] = acc[c];
    if (c4 == 0) ml[wave][col] = make_float2(base, l);
    __syncthreads();
    float top = ml[0][col].x, sum = 0.0f, f[4];
#pragma unroll
    for (int v = 1; v < 4; ++v) top = fmaxf(top, ml[v][col].x);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      f[v] = exp2_fast(ml[v][col].x - top);
      sum = __builtin_fmaf(ml[v][col].y, f[v], sum);
    }
    for (int c = wave; c < 2 * KB; c += 4) {
      float4_t o = buf[0][c][lane] * f[0];
#pragma unroll
      for (int v = 1; v < 4; ++v) o += buf[v][c][lane] * f[v];
      store_piece<D, 16>(a, pc, col, 16 * c + 4 * c4, o, sum, top);
    }
  }
  shares.finish(a, pc);
}

// ---------------------------------------------------------------------------------
// More than 16 rows: tiles of 32 rows on v_mfma_f32_32x32x16_f16. At equal rate it holds the
// issue port half as often as the 16x16 form, and next to the softmax's vector work
// that counts: 131072 products beside 32 vector instructions took 195 cycles with it, 230 to
// 257 without (two wavefronts on a SIMD).
//
// The cache's tiles serve this shape too. K: lane (key, c), key < 32, c < 2, takes what lanes
// key % 16 + 16 c and + 32 of the key's tile own: channels 8c .. 8c + 7 of the even and the odd
// 16-channel steps. The scores come out with keys 8 (i / 4) + 4c + i % 4 in register i, so one
// tile's 16 keys are eight registers of both lane halves, and a V operand of 16 keys is the
// dwords of cache lanes r + 16 c and r + 32 + 16 c; channels 0..15 of a block are their low
// nibbles, 16..31 the high ones: lanes 16..31 read the same dwords with other masks.
//
// The four wavefronts of a workgroup share 32 rows and split the keys. V is loaded at the start
// of its step and K of the next one behind the scores, so about half a step covers each: the
// registers left (K, V, 64 of output, 64 of q at 128 channels) hold no whole second step. All
// instances have the registers of two wavefronts a SIMD: none is spilled at 64 channels (28 and 69
// with three wavefronts: 37.6 and 58.9 us, now 34.6 and 39.2, for eight sequences of 5 rows over 8K keys,
// 64 heads over 8, groups of 64 and 32), 2 at 128 channels in one group (42 us), 41 in two (49 us). With 256
// channels, or four scale groups, it spills far more and is not built (256 channels in groups of 64: 330 us,
// 74 with 16-row tiles).
typedef float float16_t __attribute__((ext_vector_type(16)));

__device__ __forceinline__ float16_t mfma32(half8_t a, half8_t b, float16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

// Four V codes of a dword for this lane's channel: low or high nibbles by mask and magic.
struct VRegs {
  uint32_t mask, magic;
  half2_t bias;
};
__device__ __forceinline__ half4_t v_codes4(uint32_t w, const VRegs& k) {
  const half2_t a = as_half2((w & k.mask) | k.magic) + k.bias;
  const half2_t b = as_half2(((w >> 8) & k.mask) | k.magic) + k.bias;
  return __builtin_shufflevector(a, b, 0, 1, 2, 3);
}

template <int D, int GC>
__global__ __launch_bounds__(256, 2) void attn32_kernel(AttnArgs a, int tiles) {
  constexpr int KB = D / 32, BPG = KB / GC;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 31, c = lane >> 5, r16 = lane & 15;
  __shared__ float4_t buf[4][4][kWave];
  __shared__ float2 ml[4][32];
  const float scale = a.scale * 1.4426950408889634f;
  const DequantRegs dq = DequantRegs::make();
  VRegs vr;
  vr.mask = lane & 16 ? 0x00F000F0u : 0x000F000Fu;   // 64 + n, or 1024 + n
  vr.magic = lane & 16 ? 0x54005400u : 0x64006400u;
  vr.bias = as_half2(lane & 16 ? 0xD480D480u : 0xE408E408u);  // -72, -1032
  const int tpp = a.cache.page_size / kTokTile;
  constexpr int kStride = 8;  // tiles from one step of a wavefront to the next
  const int stride_block = kStride / tpp, stride_rem = kStride - stride_block * tpp;
  Shares shares;
  Piece pc{};
  bool more = uniform(shares.begin(a, 32, lane));
  for (bool again = false; more; again = true) {
    Piece next_piece;
    if (!uniform(shares.next(a, 32, lane, tiles, &next_piece))) break;
    pc = uniform_piece(next_piece);
    if (again) __syncthreads();  // buf of the piece before has been read
    const Job& w = pc.w;
    const int r0 = pc.r0;

    const int row = r0 + col;
    half8_t q[2 * KB];
    int pos;  // position of the lane's row: its own last visible key; -1: no row
    {
      const int i = min(row, w.rows - 1) / w.share, hs = min(row, w.rows - 1) - i * w.share;
      pos = row < w.rows ? w.len - w.nq + i : -1;
      const uint16_t* src = static_cast<const uint16_t*>(a.q) + (int64_t)(w.first + i) * a.q_stride +
                            (int64_t)(w.head * w.share + hs) * D + 8 * c;
#pragma unroll
      for (int b = 0; b < 2 * KB; ++b) q[b] = as_half8(*reinterpret_cast<const uint4*>(src + 16 * b));
    }
    // base: m + E. A score more than `limit` above it makes m rise; a row that has seen no key
    // yet has base 0 and limit -infinity, and its first key sets m.
    float base = 0.0f, limit = -__builtin_inff(), l = 0.0f;
    bool low = false;  // keys seen at -infinity while no score was above it
    float16_t acc[KB];
#pragma unroll
    for (int b = 0; b < KB; ++b) acc[b] = float16_t{};

    const Span sp = span_of(a, w, r0, 32);
    const int t_own = max(pc.key0, sp.first) + kStep * wave;
    const int t_last = pc.key1 < 0 ? sp.last : min(sp.last, pc.key1);
    float exp_v = -64.0f;  // E (wave-uniform)
    uint32_t cap_v = 0;    // largest V scale that E covers, as float16 bits

    const ScalarInts table = scalar_ints(a.block_table + (int64_t)w.seq * a.max_blocks);
    const int last_tile = max(t_last - 1, 0) / kTokTile;
    Walk next;
    next.tile = t_own / kTokTile;
    next.block = next.tile / tpp;
    next.in_page = next.tile - next.block * tpp;
    // tiles of the step whose K is loaded, and whether their pages lie in the cache
    int64_t tile[2], tile_n[2];
    bool there[2], there_n[2];
    auto walk = [&]() __attribute__((always_inline)) {
      const bool wraps = next.in_page + 1 == tpp;
      const int in2 = wraps ? 0 : next.in_page + 1, b2 = next.block + (wraps ? 1 : 0);
      const int p0 = next.tile <= last_tile && next.block < a.max_blocks ? table[next.block] : -1;
      const int p1 = next.tile + 1 <= last_tile && b2 < a.max_blocks ? table[b2] : -1;
      there_n[0] = (unsigned)p0 < (unsigned)a.cache.pages;
      there_n[1] = (unsigned)p1 < (unsigned)a.cache.pages;
      // a tile behind the last key or of a page outside the cache is read from page 0 and masked
      tile_n[0] = ((int64_t)(there_n[0] ? p0 : 0) * a.cache.kv_heads + w.head) * tpp + next.in_page;
      tile_n[1] = ((int64_t)(there_n[1] ? p1 : 0) * a.cache.kv_heads + w.head) * tpp + in2;
      next.tile += kStride;
      next.block += stride_block;
      next.in_page += stride_rem;
      if (next.in_page >= tpp) {
        next.in_page -= tpp;
        ++next.block;
      }
    };
    uint32_t kw[2][KB];  // K codes: even and odd 16-channel steps
    uint2 ks[2][GC][2];  // scales of keys 8u + 4c .. + 3 of tile j: [j][g][u]
    auto load_k = [&]() __attribute__((always_inline)) {
      const int64_t mine = lane & 16 ? tile_n[1] : tile_n[0];
      const uint32_t* p = static_cast<const uint32_t*>(a.cache.k_codes) + mine * (2 * D);
      load_codes<D>(kw[0], p, r16 + 16 * c);
      load_codes<D>(kw[1], p, r16 + 16 * c + 32);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint16_t* sc = static_cast<const uint16_t*>(a.cache.k_scales) + tile_n[j] * (GC * kTokTile) + 4 * c;
#pragma unroll
        for (int g = 0; g < GC; ++g)
#pragma unroll
          for (int u = 0; u < 2; ++u) ks[j][g][u] = *reinterpret_cast<const uint2*>(sc + g * kTokTile + 8 * u);
        tile[j] = tile_n[j];
        there[j] = there_n[j];
      }
    };

    auto step = [&](int t0) __attribute__((always_inline)) {
      // V of this step: needed only after the softmax
      uint32_t vw[2][2][KB];  // [tile][cache lanes r + 16 c, + 32]
      uint2 vs[2][GC][2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t* p = static_cast<const uint32_t*>(a.cache.v_codes) + tile[j] * (2 * D);
        load_codes<D>(vw[j][0], p, r16 + 16 * c);
        load_codes<D>(vw[j][1], p, r16 + 16 * c + 32);
        const uint16_t* sc = static_cast<const uint16_t*>(a.cache.v_scales) + tile[j] * (GC * kTokTile) + 4 * c;
#pragma unroll
        for (int g = 0; g < GC; ++g)
#pragma unroll
          for (int u = 0; u < 2; ++u) vs[j][g][u] = *reinterpret_cast<const uint2*>(sc + g * kTokTile + 8 * u);
      }
      const bool there0 = there[0], there1 = there[1];
      const bool edge =
          t0 + kStep > sp.pos_lo + 1 || t0 <= sp.pos_hi - sp.window || t0 + kStep > t_last || !there0 || !there1;
      auto key_of = [&](int i) __attribute__((always_inline)) { return t0 + 8 * (i >> 2) + 4 * c + (i & 3); };

      // scores, base 2, relative to m + E
      float s[16];
#pragma unroll
      for (int g = 0; g < GC; ++g) {
        float16_t part = {};
#pragma unroll
        for (int b = g * BPG; b < (g + 1) * BPG; ++b)
#pragma unroll
          for (int u = 0; u < 2; ++u) part = mfma32(k_operand(kw[u][b], dq), q[2 * b + u], part);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const half4_t kh = __builtin_bit_cast(half4_t, ks[i >> 3][g][(i >> 2) & 1]);
          s[i] = __builtin_fmaf(part[i], (float)kh[i & 3], g == 0 ? 0.0f : s[i]);  // one v_fma_mix
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = __builtin_fmaf(s[i], scale, -base);
      // the next step's K while the rest of this one runs
      load_k();
      walk();

      uint32_t hidden = 0;  // keys of the lane that its row does not see
      if (edge) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int key = key_of(i);
          if (!(i < 8 ? there0 : there1) || key >= t_last || key > pos || key <= pos - sp.window) {
            s[i] = -__builtin_inff();
            hidden |= 1u << i;
          }
        }
        // what no row sees may hold anything: 0 * NaN must not arise
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int g = 0; g < GC; ++g)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              half4_t vh = __builtin_bit_cast(half4_t, vs[j][g][u]);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int key = key_of(8 * j + 4 * u + i);
                vh[i] = (j ? there1 : there0) && key < t_last && key > sp.pos_lo - sp.window ? vh[i] : (_Float16)0.0f;
              }
              vs[j][g][u] = __builtin_bit_cast(uint2, vh);
            }
      }
      // E, where a V scale exceeds what it covers
      uint32_t vmax = 0;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int g = 0; g < GC; ++g)
#pragma unroll
          for (int u = 0; u < 2; ++u) vmax = max_u16x2(vmax, max_u16x2(vs[j][g][u].x, vs[j][g][u].y));
      vmax = max(vmax & 0xFFFFu, vmax >> 16);
      if (__any(vmax > cap_v)) {
        // the largest finite one, up to the end of its binade
        vmax = cap_v;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int g = 0; g < GC; ++g)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint2 r = vs[j][g][i >> 2];
              const uint32_t bits = ((i & 2 ? r.y : r.x) >> (16 * (i & 1))) & 0xFFFFu;
              vmax = max(vmax, bits < 0x7C00u ? bits : 0u);
            }
#pragma unroll
        for (int i = 1; i < 64; i <<= 1) vmax = max(vmax, (uint32_t)__shfl_xor((int)vmax, i, 64));
        cap_v = vmax | 0x3FFu;
        const float up = (float)(int)(cap_v >> 10) - 14.0f - kHeadroom - exp_v, alpha = exp2_fast(-up);
        exp_v += up;
        if (limit > -__builtin_inff()) {
          base += up;
          limit = kSlack - exp_v;
          l *= alpha;
#pragma unroll
          for (int b = 0; b < KB; ++b) acc[b] *= alpha;
#pragma unroll
          for (int i = 0; i < 16; ++i) s[i] -= up;
        }
      }
      // one score far above its row's held maximum?
      float mx = max3(s[0], s[1], s[2]);
#pragma unroll
      for (int i = 3; i < 15; i += 2) mx = max3(mx, s[i], s[i + 1]);
      mx = fmaxf(mx, s[15]);
      if (__any(mx >= limit)) {
        mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
        if (mx > -__builtin_inff()) {
          const bool first = limit == -__builtin_inff();
          const float up = first ? mx + exp_v : fmaxf(mx + exp_v, 0.0f);
          const float alpha = first ? 1.0f : exp2_fast(-up);
          base += up;
          limit = kSlack - exp_v;
          l *= alpha;
#pragma unroll
          for (int b = 0; b < KB; ++b) acc[b] *= alpha;
#pragma unroll
          for (int i = 0; i < 16; ++i) s[i] -= up;
        } else if (limit == -__builtin_inff()) {
          low |= hidden != 0xFFFFu;
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[i] = exp2_fast(s[i]);
        l += s[i];
      }
      // weights, to float16 with the V scale in them, and O += V P, a tile's 16 keys at a time
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        half8_t p[GC];
#pragma unroll
        for (int g = 0; g < GC; ++g)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const half4_t vh = __builtin_bit_cast(half4_t, vs[j][g][i >> 2]);
            p[g][i] = (_Float16)__builtin_fmaf(s[8 * j + i], (float)vh[i & 3], 0.0f);  // one v_fma_mix
          }
        if (edge) {
          // a key that one row sees and another does not may have an infinite scale
#pragma unroll
          for (int g = 0; g < GC; ++g)
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (hidden >> (8 * j + i) & 1u) p[g][i] = (_Float16)0.0f;
        }
#pragma unroll
        for (int b = 0; b < KB; ++b) {
          const half4_t v0 = v_codes4(vw[j][0][b], vr), v1 = v_codes4(vw[j][1][b], vr);
          acc[b] = mfma32(__builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7), p[b / BPG], acc[b]);
        }
      }
    };

    if (t_own < t_last) {
      walk();
      load_k();
      walk();
      for (int t0 = t_own; t0 < t_last; t0 += kStride * kTokTile) step(t0);
    }
    if (low && limit == -__builtin_inff()) l -= 1.0f;
    l += __shfl_xor(l, 32, 64);
    if (limit == -__builtin_inff()) base = kLowest;

    // the four wavefronts' parts of the same rows, added in order
    if (c == 0) ml[wave][col] = make_float2(base, l);
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      if (b > 0) __syncthreads();
#pragma unroll
      for (int u = 0; u < 4; ++u)
        buf[wave][u][lane] = float4_t{acc[b][4 * u], acc[b][4 * u + 1], acc[b][4 * u + 2], acc[b][4 * u + 3]};
      __syncthreads();
      float top = ml[0][col].x, sum = 0.0f;
#pragma unroll
      for (int v = 1; v < 4; ++v) top = fmaxf(top, ml[v][col].x);
      float4_t o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const float f = exp2_fast(ml[v][col].x - top);
        sum = __builtin_fmaf(ml[v][col].y, f, sum);
        o += buf[v][wave][lane] * f;
      }
      store_piece<D, 32>(a, pc, col, 32 * b + 8 * wave + 4 * c, o, sum, top);
    }
  }
  shares.finish(a, pc);
}

// ---------------------------------------------------------------------------------
// Many rows: 128 a workgroup, 32 a wavefront, all reading the same keys. Two of the
// wavefronts convert the K codes of the next 64 keys to float16 operands in LDS, two the V
// codes, with their scales as floats (K's with the softmax scale in them; both zeroed where
// no row sees the key), so that a wavefront's vector work is the softmax and a quarter of
// the conversion, and its registers (no raw codes) leave room for three wavefronts on a
// SIMD, which cover each other's barriers: one buffer and two barriers per 64 keys. With two
// wavefronts (a second buffer, one barrier) the barriers cost what the sharing saves.
template <int D, int GC>
struct Shared {
  static constexpr int KB = D / 32;
  static constexpr int kKeys = 64;
  half8_t k[2][2 * KB][kWave];  // [32-key pair][16-channel step]
  half8_t v[2][2][KB][kWave];   // [pair][tile][32-channel block]
  float ks[GC][kKeys], vs[GC][kKeys];
  int there[4];  // whether a tile's page lies in the cache
  int vmax[2];   // largest finite V scale of a pair (float16 bits)
  int pad[2];
};

// Row tile, head and sequence of a job. Row tile fastest (last rows, the longest spans, first),
// then head, sequence; with `swizzle` the eight XCDs, which take workgroups in turn, each keep
// whole heads (their L2 then holds the keys all of a head's tiles read: a 4001-token prompt
// 390 -> 311 us).
__device__ __forceinline__ int rows_job(const AttnArgs& a, unsigned job, int tiles, int swizzle, Job* w) {
  unsigned group = job / (unsigned)tiles, at = job % (unsigned)tiles;
  if (swizzle) {
    const unsigned x = job % 8, y = job / 8;
    group = x + 8 * (y / (unsigned)tiles);
    at = y % (unsigned)tiles;
  }
  const int tile = tiles - 1 - uniform((int)at), heads = a.cache.kv_heads;
  const int seq = uniform((int)(group / (unsigned)heads));
  const bool any = make_job(a, seq, uniform((int)group) - seq * heads, w);
  return any && 128 * tile < w->rows ? tile : -1;
}

//
// Workgroups that fill the chip a whole number of times (a.whole of them) take a job each. The
// a.tail jobs behind would leave most of it idle for as long as one job takes; CUT cuts the keys
// of each into pieces, which a second kernel joins (four 509-token chunks, 1024 jobs on 768
// places: 626 -> 512 us; 1.5 us slower where nothing is cut, hence two instances). At 128 channels in two
// groups three wavefronts a SIMD spill 7 to 10 registers and are faster all the same (four chunks of 384
// tokens over 8K: 455 us, 474 with two); 256 channels in eight groups spill 26 to 31.
template <int D, int GC, bool CUT>
__global__ __launch_bounds__(256, (D == 256 ? 1 : D == 128 && (GC == 2 || (CUT && GC == 1)) ? 3 : 2))
void attn_rows_kernel(AttnArgs a, int tiles, int swizzle) {
  using S = Shared<D, GC>;
  constexpr int KB = S::KB, BPG = KB / GC, kKeys = S::kKeys;
  extern __shared__ __align__(16) unsigned char smem[];
  S& lds = *reinterpret_cast<S*>(smem);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 31, c = lane >> 5;
  constexpr int kGroup = 128;
  const bool cut = CUT && blockIdx.x >= (unsigned)a.whole;  // one piece of a job's keys
  const unsigned behind = cut ? blockIdx.x - a.whole : 0;
  const int piece = cut ? uniform((int)(behind / (unsigned)a.tail)) : 0;
  Job w;
  const int tile_q = rows_job(a, blockIdx.x - (unsigned)(piece * a.tail), tiles, swizzle, &w);
  if (tile_q < 0) return;  // the whole workgroup; a wavefront without rows still converts
  const int g0 = tile_q * kGroup, r0 = g0 + 32 * wave;
  const bool idle = r0 >= w.rows;

  const int row = r0 + col;
  half8_t q[2 * KB];
  int pos;  // position of the lane's row: its own last visible key; -1: no row
  {
    const int i = min(row, w.rows - 1) / w.share, hs = min(row, w.rows - 1) - i * w.share;
    pos = row < w.rows ? w.len - w.nq + i : -1;
    const uint16_t* src = static_cast<const uint16_t*>(a.q) + (int64_t)(w.first + i) * a.q_stride +
                          (int64_t)(w.head * w.share + hs) * D + 8 * c;
#pragma unroll
    for (int b = 0; b < 2 * KB; ++b) q[b] = as_half8(*reinterpret_cast<const uint4*>(src + 16 * b));
  }
  // base: m + E. A score more than `limit` above it makes m rise; a row that has seen no key
  // yet has base 0 and limit -infinity, and its first key sets m.
  float base = 0.0f, limit = -__builtin_inff(), l = 0.0f;
  bool low = false;  // keys seen at -infinity while no score was above it
  float16_t acc[KB];
#pragma unroll
  for (int b = 0; b < KB; ++b) acc[b] = float16_t{};

  const Span all = span_of(a, w, g0, kGroup);                   // the workgroup's keys
  const Span own = span_of(a, w, min(r0, w.rows - 1), 32);      // those of this wavefront's rows
  int t_first = all.first, t_last = all.last;
  if (cut) {
    const int blocks = (max(t_last - t_first, 0) + kKeys - 1) / kKeys;
    const int b0 = uniform((int)((int64_t)blocks * piece / a.pieces));
    const int b1 = uniform((int)((int64_t)blocks * (piece + 1) / a.pieces));
    t_last = min(t_last, t_first + kKeys * b1);
    t_first += kKeys * b0;
  }
  const float scale = a.scale * 1.4426950408889634f;
  float exp_v = -64.0f;  // E (wave-uniform)
  int cap_v = 0;         // largest V scale that E covers, as float16 bits

  // --- producer: one pair of tiles of K (wavefronts 0, 1) or of V (2, 3) every 64 keys
  const DequantRegs dq = DequantRegs::make();
  const bool is_v = wave >= 2;
  const int pair = wave & 1;
  const uint32_t* codes = static_cast<const uint32_t*>(is_v ? a.cache.v_codes : a.cache.k_codes);
  const uint16_t* scales = static_cast<const uint16_t*>(is_v ? a.cache.v_scales : a.cache.k_scales);
  const ScalarInts table = scalar_ints(a.block_table + (int64_t)w.seq * a.max_blocks);
  const int tpp = a.cache.page_size / kTokTile;
  const int stride_block = 4 / tpp, stride_rem = 4 - stride_block * tpp;
  const int last_tile = max(t_last - 1, 0) / kTokTile;
  Walk next;
  next.tile = t_first / kTokTile + 2 * pair;
  next.block = next.tile / tpp;
  next.in_page = next.tile - next.block * tpp;
  uint32_t raw[2][KB];  // codes of the 64 keys after those in LDS
  uint16_t raw_s[GC];   // scale of key lane % 32
  bool raw_there[2];
  int raw_t0 = t_first;
  int page[2], in_page2;
  int top_v = 0;  // largest V scale this wavefront has converted
  auto fetch_pages = [&]() __attribute__((always_inline)) {
    const bool wraps = next.in_page + 1 == tpp;
    in_page2 = wraps ? 0 : next.in_page + 1;
    const int b2 = next.block + (wraps ? 1 : 0);
    page[0] = next.tile <= last_tile && next.block < a.max_blocks ? table[next.block] : -1;
    page[1] = next.tile + 1 <= last_tile && b2 < a.max_blocks ? table[b2] : -1;
  };
  auto load = [&]() __attribute__((always_inline)) {
    int64_t tile[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      // a tile behind the last key or of a page outside the cache is read from page 0 and hidden
      raw_there[j] = (unsigned)page[j] < (unsigned)a.cache.pages;
      tile[j] = ((int64_t)(raw_there[j] ? page[j] : 0) * a.cache.kv_heads + w.head) * tpp + (j ? in_page2 : next.in_page);
      load_codes<D>(raw[j], codes + tile[j] * (2 * D), lane);
    }
    const uint16_t* sc = scales + ((lane & 16) ? tile[1] : tile[0]) * (GC * kTokTile) + (lane & 15);
#pragma unroll
    for (int g = 0; g < GC; ++g) raw_s[g] = sc[g * kTokTile];
    next.tile += 4;
    next.block += stride_block;
    next.in_page += stride_rem;
    if (next.in_page >= tpp) {
      next.in_page -= tpp;
      ++next.block;
    }
    fetch_pages();
  };
  auto convert = [&]() __attribute__((always_inline)) {
    const int r16 = lane & 15, c4 = lane >> 4;
    if (is_v) {
      // four tokens of channels r and 16 + r: half of an operand of lanes r, 16 + r (+ 32)
      VRegs lo{0x000F000Fu, 0x64006400u, as_half2(0xE408E408u)}, hi{0x00F000F0u, 0x54005400u, as_half2(0xD480D480u)};
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int b = 0; b < KB; ++b) {
          half4_t* to = reinterpret_cast<half4_t*>(&lds.v[pair][j][b][r16 + 32 * (c4 & 1)]) + (c4 >> 1);
          to[0] = v_codes4(raw[j][b], lo);
          to[2 * 16] = v_codes4(raw[j][b], hi);
        }
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int b = 0; b < KB; ++b)
          lds.k[pair][2 * b + (c4 >> 1)][r16 + 16 * j + 32 * (c4 & 1)] = k_operand(raw[j][b], dq);
    }
    // what no row sees may hold anything: 0 * NaN must not arise
    const int key = raw_t0 + 32 * pair + (lane & 31);
    const bool seen = ((lane & 16) ? raw_there[1] : raw_there[0]) && key < t_last && key > all.pos_lo - all.window;
    int top = 0;
#pragma unroll
    for (int g = 0; g < GC; ++g) {
      const uint32_t bits = seen ? raw_s[g] : 0u;
      const float f = (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
      if (lane < 32) (is_v ? lds.vs : lds.ks)[g][32 * pair + lane] = is_v ? f : f * scale;
      top = max(top, bits < 0x7C00u ? (int)bits : 0);
    }
    if (is_v) {
      if (__any(top > top_v)) {
#pragma unroll
        for (int i = 1; i < 32; i <<= 1) top = max(top, __shfl_xor(top, i, 64));
        top_v = max(top_v, __builtin_amdgcn_readfirstlane(top));
      }
      if (lane == 0) lds.vmax[pair] = top_v;
    } else if (lane < 2) {
      lds.there[2 * pair + lane] = lane ? raw_there[1] : raw_there[0];
    }
    raw_t0 += kKeys;
  };

  auto compute = [&](int t0) __attribute__((always_inline)) {
    const int vmax = __builtin_amdgcn_readfirstlane(max(lds.vmax[0], lds.vmax[1]));
    if (vmax > cap_v) {
      cap_v = vmax | 0x3FF;  // up to the end of its binade
      const float up = (float)(cap_v >> 10) - 14.0f - kHeadroom - exp_v, alpha = exp2_fast(-up);
      exp_v += up;
      if (limit > -__builtin_inff()) {
        base += up;
        limit = kSlack - exp_v;
        l *= alpha;
#pragma unroll
        for (int b = 0; b < KB; ++b) acc[b] *= alpha;
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int th = t0 + kStep * h;
      if (th > own.pos_hi || th + kStep <= own.first) continue;  // none of these rows sees any (uniform)
      const bool there0 = __builtin_amdgcn_readfirstlane(lds.there[2 * h]);
      const bool there1 = __builtin_amdgcn_readfirstlane(lds.there[2 * h + 1]);
      const bool edge =
          th + kStep > own.pos_lo + 1 || th <= own.pos_hi - own.window || th + kStep > t_last || !there0 || !there1;

      // scores, base 2, relative to m + E
      float s[16];
#pragma unroll
      for (int g = 0; g < GC; ++g) {
        float16_t part = {};
#pragma unroll
        for (int b = 2 * g * BPG; b < 2 * (g + 1) * BPG; ++b) part = mfma32(lds.k[h][b][lane], q[b], part);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float4_t ks = *reinterpret_cast<const float4_t*>(&lds.ks[g][32 * h + 8 * u + 4 * c]);
#pragma unroll
          for (int i = 0; i < 4; ++i) s[4 * u + i] = __builtin_fmaf(part[4 * u + i], ks[i], g == 0 ? -base : s[4 * u + i]);
        }
      }
      uint32_t hidden = 0;  // keys of the lane that its row does not see
      if (edge) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int key = th + 8 * (i >> 2) + 4 * c + (i & 3);
          if (!(i < 8 ? there0 : there1) || key >= t_last || key > pos || key <= pos - own.window) {
            s[i] = -__builtin_inff();
            hidden |= 1u << i;
          }
        }
      }
      // one far above its row's held maximum?
      float mx = max3(s[0], s[1], s[2]);
#pragma unroll
      for (int i = 3; i < 15; i += 2) mx = max3(mx, s[i], s[i + 1]);
      mx = fmaxf(mx, s[15]);
      if (__any(mx >= limit)) {
        mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
        if (mx > -__builtin_inff()) {
          const bool first = limit == -__builtin_inff();
          const float up = first ? mx + exp_v : fmaxf(mx + exp_v, 0.0f);
          const float alpha = first ? 1.0f : exp2_fast(-up);
          base += up;
          limit = kSlack - exp_v;
          l *= alpha;
#pragma unroll
          for (int b = 0; b < KB; ++b) acc[b] *= alpha;
#pragma unroll
          for (int i = 0; i < 16; ++i) s[i] -= up;
        } else if (limit == -__builtin_inff()) {
          low |= hidden != 0xFFFFu;
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[i] = exp2_fast(s[i]);
        l += s[i];
      }
      // weights, to float16 with the V scale in them, and O += V P, a tile's 16 keys at a time
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        half8_t p[GC];
#pragma unroll
        for (int g = 0; g < GC; ++g)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const float4_t vs = *reinterpret_cast<const float4_t*>(&lds.vs[g][32 * h + 16 * j + 8 * u + 4 * c]);
#pragma unroll
            for (int i = 0; i < 4; ++i) p[g][4 * u + i] = (_Float16)(s[8 * j + 4 * u + i] * vs[i]);
          }
        if (edge) {
          // a key that one row sees and another does not may have an infinite scale
#pragma unroll
          for (int g = 0; g < GC; ++g)
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (hidden >> (8 * j + i) & 1u) p[g][i] = (_Float16)0.0f;
        }
#pragma unroll
        for (int b = 0; b < KB; ++b) acc[b] = mfma32(lds.v[h][j][b][lane], p[b / BPG], acc[b]);
      }
    }
  };

  if (t_first < t_last) {
    fetch_pages();
    load();
    convert();
    load();
    lds_barrier();
    for (int t0 = t_first;;) {
      if (!idle) compute(t0);
      if ((t0 += kKeys) >= t_last) break;
      lds_barrier();  // all have read these keys
      convert();
      load();
      lds_barrier();
    }
  }
  if (low && limit == -__builtin_inff()) l -= 1.0f;
  l += __shfl_xor(l, 32, 64);
  if (row >= w.rows) return;
  if (cut) {
    const int64_t slot = (int64_t)behind * kGroup + 32 * wave + col;
#pragma unroll
    for (int b = 0; b < KB; ++b)
#pragma unroll
      for (int u = 0; u < 4; ++u)
        *reinterpret_cast<float4_t*>(a.part_o + slot * D + 32 * b + 8 * u + 4 * c) =
            float4_t{acc[b][4 * u], acc[b][4 * u + 1], acc[b][4 * u + 2], acc[b][4 * u + 3]};
    if (c == 0)
      *reinterpret_cast<float2*>(a.part_ml + 2 * slot) = make_float2(limit == -__builtin_inff() ? kLowest : base, l);
    return;
  }
#pragma unroll
  for (int b = 0; b < KB; ++b)
#pragma unroll
    for (int u = 0; u < 4; ++u)
      *out_at<D>(a, w, row, 32 * b + 8 * u + 4 * c) =
          to_row(float4_t{acc[b][4 * u], acc[b][4 * u + 1], acc[b][4 * u + 2], acc[b][4 * u + 3]}, l);
}

// Row `row` of a job from n partial results, the i-th in place at(i): a wavefront, D / 4 lanes
// of four channels each, the 256 / D groups taking every such piece, added in order.
template <int D, typename At>
__device__ __forceinline__ void join_row(const AttnArgs& a, const Job& w, int row, int n, At at) {
  constexpr int LPR = D / 4, G = kWave / LPR;
  const int lane = threadIdx.x & 63;
  const int g = lane / LPR, ch = 4 * (lane % LPR);
  const float2* ml = reinterpret_cast<const float2*>(a.part_ml);
  float top = kLowest, sum = 0.0f;
  float4_t o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int i = g; i < n; i += G) top = fmaxf(top, ml[at(i)].x);
#pragma unroll
  for (int m = LPR; m < kWave; m <<= 1) top = fmaxf(top, __shfl_xor(top, m, 64));
#pragma unroll 4
  for (int i = g; i < n; i += G) {
    const float2 v = ml[at(i)];
    const float f = exp2_fast(v.x - top);
    sum = __builtin_fmaf(v.y, f, sum);
    o += *reinterpret_cast<const float4_t*>(a.part_o + at(i) * D + ch) * f;
  }
#pragma unroll
  for (int m = LPR; m < kWave; m <<= 1) {
    sum += __shfl_xor(sum, m, 64);
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] += __shfl_xor(o[e], m, 64);
  }
  if (g == 0) *out_at<D>(a, w, row, ch) = to_row(o, sum);
}

// The job that share blockIdx.x / (rg / 4) begins and does not end.
template <int D>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a, int rg) {
  const int per = rg / 4;
  const int share = (int)(blockIdx.x / (unsigned)per);
  const int local = (int)(blockIdx.x - (unsigned)(share * per)) * 4 + uniform(threadIdx.x >> 6);
  const int4* cut = reinterpret_cast<const int4*>(a.cuts) + 2 * share;
  const int4 c0 = cut[0];
  const int n = c0.x;  // pieces: this share's slot 1, the next ones' slot 0
  const int row = cut[1].x + local;
  if (n == 0 || row >= c0.z) return;
  Job w{};
  w.first = c0.y;
  w.head = c0.w;
  w.share = a.q_heads / a.cache.kv_heads;
  join_row<D>(a, w, row, n, [&](int i) __attribute__((always_inline)) {
    return ((int64_t)(share + i) * 2 + (i == 0)) * rg + local;
  });
}

// The cut jobs of attn_rows_kernel, a wavefront per row.
template <int D>
__global__ __launch_bounds__(256) void attn_join_rows_kernel(AttnArgs a, int tiles, int swizzle) {
  const int job = (int)(blockIdx.x / 32), local = (int)(blockIdx.x % 32) * 4 + uniform(threadIdx.x >> 6);
  Job w;
  const int tile = rows_job(a, (unsigned)(a.whole + job), tiles, swizzle, &w);
  if (tile < 0 || 128 * tile + local >= w.rows) return;
  join_row<D>(a, w, 128 * tile + local, a.pieces,
              [&](int i) __attribute__((always_inline)) { return ((int64_t)i * a.tail + job) * 128 + local; });
}

template <int D, int GC>
hipError_t launch_t(const AttnArgs& a, hipStream_t stream) {
  const int64_t rows = (int64_t)a.max_q * (a.q_heads / a.cache.kv_heads);
  const int tiles = (int)((rows + a.rows_group - 1) / a.rows_group);
  const int64_t groups = (int64_t)a.cache.kv_heads * a.seqs;
  const dim3 grid((unsigned)(a.shares > 0 ? a.shares : tiles * groups));
  if (a.rows_group == 128) {
    const int swizzle = groups % 8 == 0 && tiles > 1;
    if (a.tail > 0) {
      hipLaunchKernelGGL((attn_rows_kernel<D, GC, true>), dim3((unsigned)(a.whole + a.tail * a.pieces)), dim3(256),
                         sizeof(Shared<D, GC>), stream, a, tiles, swizzle);
      hipLaunchKernelGGL(attn_join_rows_kernel<D>, dim3((unsigned)(a.tail * 32)), dim3(256), 0, stream, a, tiles,
                         swizzle);
    } else {
      hipLaunchKernelGGL((attn_rows_kernel<D, GC, false>), grid, dim3(256), sizeof(Shared<D, GC>), stream, a, tiles,
                         swizzle);
    }
  } else if (tiles == 1 && a.rows_group == 16) {
    hipLaunchKernelGGL((attn16_kernel<D, GC, true>), grid, dim3(256), 0, stream, a, tiles);
  } else if constexpr (has_attn32(D, GC)) {
    hipLaunchKernelGGL((attn32_kernel<D, GC>), grid, dim3(256), 0, stream, a, tiles);
  } else {
    hipLaunchKernelGGL((attn16_kernel<D, GC, false>), grid, dim3(256), 0, stream, a, tiles);
  }
  if (a.shares > 0)
    hipLaunchKernelGGL(attn_join_kernel<D>, dim3((unsigned)(a.shares * (a.rows_group / 4))), dim3(256), 0, stream, a,
                       a.rows_group);
  return hipGetLastError();
}

template <int D, int GC>
int resident_t(int rows_group) {
  if (rows_group == 128)
    return resident_per_cu(reinterpret_cast<const void*>(&attn_rows_kernel<D, GC, true>), 256, sizeof(Shared<D, GC>)) *
           device_cu_count_cached();
  if constexpr (has_attn32(D, GC)) {
    if (rows_group == 32) return resident_grid(reinterpret_cast<const void*>(&attn32_kernel<D, GC>), 256);
  }
  return resident_grid(reinterpret_cast<const void*>(&attn16_kernel<D, GC, true>), 256);
}

}  // namespace

// CALL(head_dim, scale groups a head) for the cache's sizes.
#define Q4_ATTN_DISPATCH(head_dim, group, CALL)                                       \
  switch ((head_dim) * 8 + (head_dim) / (group)) {                                    \
    case 64 * 8 + 1: return CALL(64, 1);                                              \
    case 64 * 8 + 2: return CALL(64, 2);                                              \
    case 128 * 8 + 1: return CALL(128, 1);                                            \
    case 128 * 8 + 2: return CALL(128, 2);                                            \
    case 128 * 8 + 4: return CALL(128, 4);                                            \
    case 256 * 8 + 2: return CALL(256, 2);                                            \
    case 256 * 8 + 4: return CALL(256, 4);                                            \
    default: return CALL(256, 8);                                                     \
  }

int attention_resident(int head_dim, int group, int rows_group) {
#define Q4_CALL(D, GC) resident_t<D, GC>(rows_group)
  Q4_ATTN_DISPATCH(head_dim, group, Q4_CALL)
#undef Q4_CALL
}

hipError_t launch_attention(const AttnArgs& a, hipStream_t stream) {
#define Q4_CALL(D, GC) launch_t<D, GC>(a, stream)
  Q4_ATTN_DISPATCH(a.cache.head_dim, a.cache.group, Q4_CALL)
#undef Q4_CALL
}

}  // namespace q4
