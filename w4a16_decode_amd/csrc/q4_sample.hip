// The next tokens from rows of logits (include/q4_serve.h).
//
// Weights are whole numbers: w_i = rint(2^shift exp((l_i - m) / T)) in 64 bits, a row's sum below
// 2^63. Their sums are exact, so any split of a row over threads and workgroups and any order of
// additions (atomics among them) give the same cuts and the same token.
//
// Cuts. The sums of a row's weights (top-p) or tokens (top-k) by the weight's logarithm, 1024 bins,
// say which bin a cut falls into; only the tokens of that bin are listed and ranked. Ranks go by
// key = (descending logit, ascending index) in 64 bits, without ties: digit by digit from the
// first one that differs, sums over the tokens that share the digits found so far by their next
// one. With top-k and top-p both, top-p's total is that of the tokens top-k left, so the list
// holds all tokens down to top-k's bin, and so it does for a top-k of up to 128 alone: where nothing but 128
// listed tokens can be left, the draw is made among them and no logit is read again (one row with top-k: 18.9 ->
// 17.9 us).
//
// A workgroup a row, in one launch, holds up to 32768 logits in registers. Longer rows, or few ones
// (q4_serve_api.cpp has the rule), are split into chunks of 4096 logits, a workgroup each, in four
// launches, each a pass over what the one before left (the last three read the logits from the caches):
//   tops    the chunks' largest logits;
//   bins    the sums by bin. Left out without top-k and top-p;
//   sums    per chunk the sum of the weights before the cut's bin, and the list;
//   choose  a workgroup a row: the cut inside the bin, the chunk that the draw falls into, and
//           the token in it.
//
// What bounds it: with few rows the chain of four launches (15 us of one greedy row in a graph, of 128256
// logits; 18 with top-k, 23 to 25 with top-p alone, whose bin holds more tokens than are ranked at once). 64 rows
// of 128256 float32 logits (33 MB, 7 us at a large copy's rate) take 5.7 + 12.4 + 13.0 + 12.1 us: logits and bins are
// waited for at the start of each pass, a weight's float64 arithmetic and its sum are 35 vector instructions a
// logit, the bins' sums meet in the caches (without that 8.9 for 12.4), and the last launch runs on 64 CUs. 256
// whole rows of 32000 take 14 us. One workgroup a row and digits over all tokens, no bins: one row 499 us, 64 rows 679.
#include "q4_device.h"
#include "q4_internal.h"

namespace q4 {
namespace {

typedef unsigned long long u64;

constexpr int kChunk = kSampleChunk, kThreads = 256, kRun = kChunk / kThreads;
constexpr int kChoose = 512;   // threads of the last launch
constexpr int kWhole = 1024;   // threads of the launch that takes whole rows
constexpr int kList = 4096;    // listed tokens that a workgroup holds in registers
constexpr int kBins = kSampleBins, kDigits = 256, kRounds = 8;

// ---- across the wavefront -----------------------------------------------------------
// Sums and maxima through DPP: rows of 16 lanes by shifts of 1, 2, 4, 8, then lane 15 of a row and
// lane 31 passed on (about 8 cycles a step; through the LDS crossbar it is over 60).
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp(uint32_t old, uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)old, (int)v, CTRL, ROWS, 0xF, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ u64 plus_dpp(u64 v) {
  return v + ((u64)dpp<CTRL, ROWS>(0, (uint32_t)(v >> 32)) << 32 | dpp<CTRL, ROWS>(0, (uint32_t)v));
}
__device__ __forceinline__ u64 wave_scan(u64 v) {  // inclusive
  v = plus_dpp<0x111, 0xF>(v);
  v = plus_dpp<0x112, 0xF>(v);
  v = plus_dpp<0x114, 0xF>(v);
  v = plus_dpp<0x118, 0xF>(v);
  v = plus_dpp<0x142, 0xA>(v);
  return plus_dpp<0x143, 0xC>(v);
}
__device__ __forceinline__ u64 lane_of(u64 v, int lane) {
  return (u64)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32 |
         (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ float max_dpp(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v);
  return fmaxf(v, __builtin_bit_cast(float, dpp<CTRL, ROWS>(b, b)));
}
__device__ __forceinline__ float wave_max(float v) {  // in every lane
  v = max_dpp<0x111, 0xF>(v);
  v = max_dpp<0x112, 0xF>(v);
  v = max_dpp<0x114, 0xF>(v);
  v = max_dpp<0x118, 0xF>(v);
  v = max_dpp<0x142, 0xA>(v);
  v = max_dpp<0x143, 0xC>(v);
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}
__device__ __forceinline__ uint32_t wave_or(uint32_t v) {  // in lane 63
  v |= dpp<0x111, 0xF>(0, v);
  v |= dpp<0x112, 0xF>(0, v);
  v |= dpp<0x114, 0xF>(0, v);
  v |= dpp<0x118, 0xF>(0, v);
  v |= dpp<0x142, 0xA>(0, v);
  return v | dpp<0x143, 0xC>(0, v);
}

// ---- across the workgroup: each call has its own LDS, so one barrier is enough ------------
template <int N>
struct Scan {
  u64 wave[N / kWave];
};
// Sum of the values of the threads before this one; *total: of all.
template <int N>
__device__ __forceinline__ u64 block_scan(u64 v, Scan<N>& s, u64* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const u64 incl = wave_scan(v);
  if (lane == kWave - 1) s.wave[wave] = incl;
  __syncthreads();
  u64 before = incl - v, all = 0;
#pragma unroll
  for (int w = 0; w < N / kWave; ++w) {
    const u64 x = s.wave[w];
    if (w < wave) before += x;
    all += x;
  }
  *total = all;
  return before;
}

// ---- logits ------------------------------------------------------------------------
__device__ __forceinline__ float clean(float v) {  // no NaN, one zero
  return v == v ? v + 0.0f : -__builtin_inff();
}
__device__ __forceinline__ float bf16(uint32_t bits) { return __builtin_bit_cast(float, bits << 16); }

template <int DT>
__device__ __forceinline__ float load_one(const void* p, int64_t i) {
  if constexpr (DT == 0) return clean((float)static_cast<const _Float16*>(p)[i]);
  if constexpr (DT == 1) return clean(bf16(static_cast<const uint16_t*>(p)[i]));
  return clean(static_cast<const float*>(p)[i]);
}

// Logits i .. i + N - 1 (rows may start at any element: the loads promise no more); -infinity behind the end.
template <int DT, int N>
__device__ __forceinline__ void load_run(const void* p, int i, int vocab, float (&v)[N]) {
  if (i + N <= vocab) {
    constexpr int kPiece = DT == 2 || N == 4 ? 4 : 8;
#pragma unroll
    for (int j = 0; j < N; j += kPiece) {
      if constexpr (DT == 2) {
        float4_t x;
        __builtin_memcpy(&x, static_cast<const float*>(p) + i + j, 16);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[j + e] = clean(x[e]);
      } else {
        uint16_t x[kPiece];
        __builtin_memcpy(x, static_cast<const uint16_t*>(p) + i + j, 2 * kPiece);
#pragma unroll
        for (int e = 0; e < kPiece; ++e) v[j + e] = clean(DT == 1 ? bf16(x[e]) : (float)__builtin_bit_cast(_Float16, x[e]));
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = i + e < vocab ? load_one<DT>(p, i + e) : -__builtin_inff();
  }
}

__device__ __forceinline__ const void* row_of(const SampleArgs& a, int row, int dt) {
  return static_cast<const char*>(a.logits) + (int64_t)row * a.stride * (dt == 2 ? 4 : 2);
}

// Smaller for the earlier rank.
__device__ __forceinline__ u64 rank_key(float v, int i) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  return (u64)~(u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u)) << 32 | (uint32_t)i;
}

// ---- weights ------------------------------------------------------------------------
// A row's settings. Greedy (temperature <= 0): only the largest logits have weight, and the draw is 0.
struct Row {
  double top;    // largest logit
  double slope;  // log2(e) / temperature; greedy: so steep that nothing below the largest has weight
  double shift;
  float half_top, bin_slope;  // half the largest logit, bins a half step of the logit
  int index_bits;            // of a key
  int k;  // 0: no top-k
  bool infinite;  // the largest logit is: those count as 0, all others as -infinity
  bool cut_p, greedy;
  double p;
  u64 w_min;  // smallest weight that min-p leaves
  __device__ __forceinline__ bool cuts() const { return k > 0 || cut_p; }
};

__device__ __forceinline__ Row row_settings(const SampleArgs& a, int row, float top) {
  Row r;
  r.infinite = top == __builtin_inff();
  r.top = r.infinite ? 0.0 : (double)top;
  const float t = a.temperature ? a.temperature[row] : 1.0f;
  r.greedy = !(t > 0.0f);
  r.slope = r.greedy ? 1e300 : 1.4426950408889634 / (double)t;
  r.shift = (double)a.shift;
  r.half_top = (float)r.top * 0.5f;
  r.bin_slope = (float)__builtin_fmin(r.slope * (2 * kBins) / (a.shift + 2), 1e38);
  r.index_bits = 32 - __builtin_clz((unsigned)(a.vocab - 1) | 1u);
  r.k = a.top_k ? a.top_k[row] : 0;
  if (r.greedy || r.k < 0 || r.k >= a.vocab) r.k = 0;
  r.p = a.top_p ? (double)a.top_p[row] : 1.0;
  r.cut_p = !r.greedy && r.p < 1.0;
  const double pm = a.min_p ? (double)a.min_p[row] : 0.0;
  r.w_min = pm > 0.0 ? (u64)ceil(ldexp(pm < 1.0 ? pm : 1.0, a.shift)) : 0;
  return r;
}

// A logit as the row counts it.
__device__ __forceinline__ float settle(const Row& r, float v) {
  return !r.infinite ? v : v == __builtin_inff() ? 0.0f : -__builtin_inff();
}
template <int N>
__device__ __forceinline__ void settle_all(const Row& r, float (&v)[N]) {
  if (!r.infinite) return;
#pragma unroll
  for (int e = 0; e < N; ++e) v[e] = settle(r, v[e]);
}

// log2 of the weight. (NaN where -infinity meets a slope of 0: it has no weight either.)
__device__ __forceinline__ double exponent(const Row& r, float v) {
  return __builtin_fma((double)v - r.top, r.slope, r.shift);
}

// rint(2^z), z <= 50, 0 for no weight: with k = rint(256 z), 2^(k / 256) from the table and
// 2^(z - k / 256) by its series to the fourth power, whose next term is below 2^-54; the whole is
// within 2^-50 of itself before the rounding.
__device__ __forceinline__ u64 weight_of(double z, const double* table) {
  constexpr double kMagic = 26388279066624.0;  // 1.5 * 2^44: the sum's last bit is 1/256
  z = __builtin_fmax(z, -2.0);
  const double m = z + kMagic;
  const int k = (int)(uint32_t)__builtin_bit_cast(u64, m);
  const double x = (z - (m - kMagic)) * 0.6931471805599453;
  double s = __builtin_fma(x, 1.0 / 24, 1.0 / 6);
  s = __builtin_fma(x, s, 0.5);
  s = __builtin_fma(x, s, 1.0);
  s = __builtin_fma(x, s, 1.0);
  const double w = ldexp(table[k & 255] * s, k >> 8);
  // + 2^52: rounded to a whole number, which is in the low bits
  return __builtin_bit_cast(u64, w + 4503599627370496.0) & 0xFFFFFFFFFFFFFull;
}
template <int N>
__device__ __forceinline__ void fill_table(double* table) {
  if (N == 256 || threadIdx.x < 256) table[threadIdx.x] = exp2((double)threadIdx.x / 256);
}
// The weight's binades below the largest one's, shift + 2 of them in kBins bins. In float32, as all that is asked
// of it is that it grows with the rank; tokens of the last bin have no weight. The difference is taken of halves:
// finite logits may lie up to twice float32's largest number apart and still have weight, at a temperature as large.
// (-infinity goes to the last bin also where an infinite temperature makes its product a NaN.)
constexpr int kNoBin = kBins - 1;
__device__ __forceinline__ int bin_of(const Row& r, float v) {
  return (int)fminf(__builtin_fmaf(v, -0.5f, r.half_top) * r.bin_slope, (float)kNoBin);
}

// ---- cuts -----------------------------------------------------------------------------
// Bins that a row's cuts need a closer look at: first .. last are listed, those before stay whole, and what
// comes before `first` in the sum that the cut goes by.
struct Cut {
  int first, last;
  u64 before;
  u64 target;  // the cut goes after the token with which the sum reaches it; 0: nothing is cut
};

__device__ __forceinline__ u64 part_of(double p, u64 total) {
  const double part = ceil(p * (double)total);
  const u64 t = part >= 1.0 ? (u64)part : 1;
  return t < total ? t : total;
}

constexpr int kFew = 128;  // listed tokens that are ranked by counting
// own: this thread's bins, the threadIdx.x-th kBins / N.
template <int N>
__device__ __forceinline__ Cut find_cut(const Row& r, const u64 (&own)[kBins / N], Scan<N>& s, u64* found) {
  if (!r.cuts()) return Cut{kBins, -1, 0, 0};
  constexpr int kPer = kBins / N;
  u64 sum = 0, total;
#pragma unroll
  for (int i = 0; i < kPer; ++i) sum += own[i];
  u64 before = block_scan<N>(sum, s, &total);
  const bool all = r.k > 0 && (u64)r.k >= total;  // top-k leaves every token that has weight
  const u64 target = r.k > 0 ? (all ? total : (u64)r.k) : part_of(r.p, total);
  if (target > before && target <= before + sum) {
    int i = 0;
#pragma unroll
    for (; i < kPer - 1; ++i) {
      if (target <= before + own[i]) break;
      before += own[i];
    }
    found[0] = threadIdx.x * kPer + i;
    found[1] = before;
  }
  __syncthreads();
  const int at = (int)found[0];
  if (r.k > 0 && (r.cut_p || r.k <= kFew)) return Cut{0, at, 0, all ? 0 : target};
  return all ? Cut{kBins, -1, 0, 0} : Cut{at, at, found[1], target};
}

struct Digits {
  u64 sums[kRounds][kDigits];
  uint32_t counts[kRounds][kDigits];
  u64 key;
  uint32_t ones, zeros;  // bits that some key has set, and clear
};

// Smallest key up to which the listed tokens with keys <= last add up to `target` or more
// (1 <= target <= their total). each(f): f(key, weight) for this thread's; ONES: a token counts 1.
template <int N, bool ONES, typename Each>
__device__ __forceinline__ u64 select_key(const Row& r, u64 last, u64 target, Digits& s, Each each) {
  const int lane = threadIdx.x & 63;
  __syncthreads();  // an earlier cut has been read
  for (int i = threadIdx.x; i < kRounds * kDigits; i += N) {
    (&s.sums[0][0])[i] = 0;
    (&s.counts[0][0])[i] = 0;
  }
  if (threadIdx.x == 0) s.ones = s.zeros = 0;
  __syncthreads();
  // the first bit that differs
  uint32_t ones = 0, zeros = 0;
  each([&](u64 key, u64) __attribute__((always_inline)) {
    if (key > last) return;
    ones |= (uint32_t)(key >> 32);
    zeros |= ~(uint32_t)(key >> 32);
  });
  ones = wave_or(ones), zeros = wave_or(zeros);
  if (lane == kWave - 1 && (ones | zeros)) {
    atomicOr(&s.ones, ones);
    atomicOr(&s.zeros, zeros);
  }
  __syncthreads();
  ones = s.ones;
  const uint32_t differ = ones & s.zeros;
  int bit = differ ? 64 - __builtin_clz(differ) : r.index_bits;  // digits from this bit down
  u64 prefix = bit < 64 ? ((u64)ones << 32) >> bit << bit : 0, before = 0;
  for (int round = 0; bit > 0; ++round) {
    // a digit does not reach from the logit into the index
    const int floor = bit > 32 ? 32 : 0, width = min(bit - floor, 8), at = bit - width;
    each([&](u64 key, u64 w) __attribute__((always_inline)) {
      if (key > last || (bit < 64 && (key ^ prefix) >> bit != 0)) return;
      const int d = (int)(key >> at) & ((1 << width) - 1);
      if (!ONES) atomicAdd(&s.sums[round][d], w);
      atomicAdd(&s.counts[round][d], 1u);
    });
    __syncthreads();
    // every wavefront for itself: four digits a lane
    u64 own[4], sum = 0;
    uint32_t count[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      count[i] = s.counts[round][4 * lane + i];
      sum += own[i] = ONES ? (u64)count[i] : s.sums[round][4 * lane + i];
    }
    u64 upto = before + wave_scan(sum) - sum;
    const bool here = target > upto && target <= upto + sum;
    int digit = 4 * lane;
    uint32_t n = count[0];
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (here && digit == 4 * lane + i && target > upto + own[i]) upto += own[i], ++digit, n = count[i + 1];
    const int l = __builtin_ctzll(__ballot(here));
    prefix |= (u64)(uint32_t)__builtin_amdgcn_readlane(digit, l) << at;
    before = lane_of(upto, l);
    if (at == 0) break;
    bit = at;
    if (at >= 32) {  // down to the next bit in which any two logits differ, or to the index
      const uint32_t below = differ & ((1u << (at - 32)) - 1);
      bit = below ? 64 - __builtin_clz(below) : r.index_bits;
      const uint32_t same = ((1u << (at - 32)) - 1) & ~(below ? (1u << (bit - 32)) - 1 : 0);
      prefix |= (u64)(ones & same) << 32;
    }
    if (__builtin_amdgcn_readlane((int)n, l) == 1) {  // the token itself
      each([&](u64 key, u64) __attribute__((always_inline)) {
        if (key <= last && (key ^ prefix) >> at == 0) s.key = key;
      });
      __syncthreads();
      return s.key;
    }
  }
  return prefix;
}

__device__ __forceinline__ u64 draw_of(const SampleArgs& a, const Row& r, int row, u64 total) {
  const double u = r.greedy ? 0.0 : (double)a.uniforms[row];
  const double at = u > 0.0 ? floor(u * (double)total) : 0.0;
  const u64 draw = at < 9.2e18 ? (u64)at : total;
  return draw < total ? draw : total - 1;
}

// The chosen token's share of the tokens that the cuts left, whose weights sum to `total`.
__device__ __forceinline__ float share_of(const SampleArgs& a, const Row& r, float v, u64 total) {
  return r.greedy ? 1.0f : (float)(exp2(exponent(r, v) - r.shift) / ldexp((double)total, -a.shift));
}

// Few listed tokens: every one counts those ranked up to it and adds their weights, N / kFew threads a
// token, which answers both cuts at once.
struct Few {
  u64 keys[kFew], weights[kFew];
  u64 upto[kFew];    // weights up to the token
  uint32_t rank[kFew];
  u64 total, key_k, key_p;
  u64 drawn[kFew], all;  // weights that stayed: up to the token's index, of all
};
template <int N>
__device__ __forceinline__ u64 cut_few(const Row& r, const Cut& cut, int count, u64 key, u64 w, Few& s) {
  const int i = (int)threadIdx.x % kFew;
  if (threadIdx.x < kFew) {
    const bool any = (int)threadIdx.x < count;
    s.keys[i] = any ? key : ~0ull, s.weights[i] = any ? w : 0;
    s.upto[i] = 0, s.rank[i] = 0;
  }
  if (threadIdx.x == 0) s.key_k = s.key_p = ~0ull;
  __syncthreads();
  constexpr int kShare = kFew / (N / kFew);
  const int j0 = (int)threadIdx.x / kFew * kShare;
  const u64 mine = s.keys[i];
  if (j0 < count) {
    u64 upto = 0;
    uint32_t rank = 0;
#pragma unroll 4
    for (int j = j0; j < j0 + kShare; ++j) {
      const bool before = s.keys[j] <= mine;
      upto += before ? s.weights[j] : 0;
      rank += before;
    }
    atomicAdd(&s.upto[i], upto);
    atomicAdd(&s.rank[i], rank);
  }
  __syncthreads();
  const bool any = (int)threadIdx.x < count;
  const u64 upto = any ? s.upto[i] : 0;
  const uint32_t rank = any ? s.rank[i] : 0;
  const u64 leave = r.k > 0 && cut.target > 0 ? cut.target - cut.before : (u64)count;  // by rank
  u64 last = ~0ull;
  if (r.k > 0) {
    if (any && rank == leave) s.key_k = mine, s.total = upto;
    __syncthreads();
    last = s.key_k;
  }
  if (r.cut_p) {
    const u64 target = r.k > 0 ? part_of(r.p, s.total) : cut.target - cut.before;
    if (any && upto >= target && upto - w < target) s.key_p = mine;
    __syncthreads();
    last = s.key_p < last ? s.key_p : last;
  }
  return last;
}

// The token that the draw falls into where the cuts leave listed tokens only, `last` from cut_few: each adds up
// the weights that stayed of those up to its index.
template <int N>
__device__ __forceinline__ void draw_few(const SampleArgs& a, const Row& r, int row, int count, u64 key, u64 w, float v,
                                         u64 last, Few& s) {
  const int i = (int)threadIdx.x % kFew;
  const bool any = (int)threadIdx.x < count;
  if (!any || key > last || w < r.w_min) w = 0;
  if (threadIdx.x < kFew) s.weights[i] = w, s.drawn[i] = 0;
  if (threadIdx.x == 0) s.all = 0;
  __syncthreads();
  constexpr int kShare = kFew / (N / kFew);
  const int j0 = (int)threadIdx.x / kFew * kShare;
  if (j0 < count) {
    const uint32_t mine = (uint32_t)s.keys[i];
    u64 upto = 0, all = 0;
#pragma unroll 4
    for (int j = j0; j < j0 + kShare; ++j) {
      const u64 x = s.weights[j];
      upto += (uint32_t)s.keys[j] <= mine ? x : 0;
      all += x;
    }
    atomicAdd(&s.drawn[i], upto);
    if (i == 0) atomicAdd(&s.all, all);
  }
  __syncthreads();
  const u64 total = s.all, draw = draw_of(a, r, row, total);
  if (any && draw < s.drawn[i] && draw >= s.drawn[i] - w) {
    a.tokens[row] = (int)(uint32_t)key;
    if (a.probs) a.probs[row] = share_of(a, r, v, total);
  }
}

// Key of the last token that top-k and top-p leave of the listed ones. kept(key, w): each that min-p leaves too.
template <int N, typename Each, typename Kept>
__device__ __forceinline__ u64 cut_list(const Row& r, const Cut& cut, Digits& s, Scan<N>& scan, Each each, Kept kept) {
  u64 last = ~0ull;
  if (r.k > 0 && cut.target > 0) last = select_key<N, true>(r, last, cut.target - cut.before, s, each);
  if (r.cut_p) {
    u64 target = cut.target - cut.before;
    if (r.k > 0) {
      u64 sum = 0, total;
      each([&](u64 key, u64 w) __attribute__((always_inline)) { sum += key <= last ? w : 0; });
      block_scan<N>(sum, scan, &total);
      target = part_of(r.p, total);
    }
    last = select_key<N, false>(r, last, target, s, each);
  }
  each([&](u64 key, u64 w) __attribute__((always_inline)) {
    if (key <= last && w >= r.w_min) kept(key, w);
  });
  return last;
}

// The same with the listed tokens token_at(0) .. token_at(count - 1): in registers, or where they are too
// many read again each time.
template <int N, typename TokenAt, typename Kept>
__device__ __forceinline__ u64 cut_tokens(const Row& r, const Cut& cut, int count, const double* table, Digits& s,
                                          Few& few, Scan<N>& scan, TokenAt token_at, Kept kept) {
  constexpr int kHeld = kList / N;
  auto look = [&](int n, u64* key, u64* w) __attribute__((always_inline)) {
    float v;
    const int token = token_at(n, &v);
    *key = rank_key(v, token);
    *w = weight_of(exponent(r, v), table);
  };
  if (count <= N) {
    u64 key = 0, w = 0;
    const bool any = (int)threadIdx.x < count;
    if (any) look(threadIdx.x, &key, &w);
    if (count <= kFew) {
      const u64 last = cut_few<N>(r, cut, count, key, w, few);
      if (any && key <= last && w >= r.w_min) kept(key, w);
      return last;
    }
    return cut_list<N>(r, cut, s, scan, [&](auto f) __attribute__((always_inline)) { if (any) f(key, w); }, kept);
  }
  if (count <= kList) {
    u64 keys[kHeld], weights[kHeld];
    float v[kHeld];
    int token[kHeld];
#pragma unroll
    for (int i = 0; i < kHeld; ++i)  // all loads, then what is computed of them
      if (i * N < count) token[i] = token_at(min(i * N + (int)threadIdx.x, count - 1), &v[i]);
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (i * N < count) keys[i] = rank_key(v[i], token[i]), weights[i] = weight_of(exponent(r, v[i]), table);
    return cut_list<N>(r, cut, s, scan, [&](auto f) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < kHeld; ++i)
        if (i * N < count && i * N + (int)threadIdx.x < count) f(keys[i], weights[i]);
    }, kept);
  }
  return cut_list<N>(r, cut, s, scan, [&](auto f) __attribute__((always_inline)) {
    for (int n = threadIdx.x; n < count; n += N) {
      u64 key, w;
      look(n, &key, &w);
      f(key, w);
    }
  }, kept);
}

// Weight of a token that the cuts left, else 0.
__device__ __forceinline__ u64 kept_weight(const Row& r, const Cut& cut, u64 last, float v, int i, const double* table) {
  if (cut.last >= 0) {
    const int bin = bin_of(r, v);
    if (bin > cut.last || (bin >= cut.first && rank_key(v, i) > last)) return 0;
  }
  const u64 w = weight_of(exponent(r, v), table);
  return w >= r.w_min ? w : 0;
}

// The token of this thread's run v, i0 .., that the draw falls into, `upto` being the sum before the run.
template <int N, typename Weight>
__device__ __forceinline__ void write_token(const SampleArgs& a, const Row& r, int row, int i0, const float (&v)[N],
                                            Weight weight, u64 upto, u64 draw, u64 total) {
  int i = 0;
  float x = v[0];
#pragma unroll
  for (int j = 0; j < N - 1; ++j) {
    upto += weight(j);
    if (draw >= upto) i = j + 1, x = v[j + 1];
  }
  a.tokens[row] = i0 + i;
  if (a.probs) a.probs[row] = share_of(a, r, x, total);
}

__device__ __forceinline__ void write_none(const SampleArgs& a, int row) {
  if (threadIdx.x != 0) return;
  a.tokens[row] = -1;
  if (a.probs) a.probs[row] = 0.0f;
}

// What is computed of v behind this is computed anew: keeping a whole run's exponents or weights from one
// pass to the next would take more registers than there are.
template <int N>
__device__ __forceinline__ void again(float (&v)[N]) {
#pragma unroll
  for (int e = 0; e < N; ++e) asm volatile("" : "+v"(v[e]));
}

// Between every four of a run's tokens: the scheduler else overlaps so many that registers spill.
__device__ __forceinline__ void apart(int e) {
  if (e % 4 == 3) __builtin_amdgcn_sched_barrier(0);
}

// ---- whole rows ------------------------------------------------------------------------
struct WholeLds {
  Scan<kWhole> scan[4];
  float wave[kWhole / kWave];
  double table[256];
  u64 bins[kBins];
  uint32_t counts[kBins];
  u64 found[2];
  Digits digits;
  Few few;
  int listed;
  uint2 list[kList];  // token and logit
};

template <int DT, int E>
__global__ __launch_bounds__(kWhole) void whole_kernel(SampleArgs a) {
  __shared__ WholeLds s;
  const int row = blockIdx.x;
  const void* p = row_of(a, row, DT);
  const int i0 = (int)threadIdx.x * E;
  float v[E];
  load_run<DT>(p, i0, a.vocab, v);
  fill_table<kWhole>(s.table);
  s.bins[threadIdx.x] = 0;
  s.counts[threadIdx.x] = 0;
  if (threadIdx.x == 0) s.listed = 0;
  float top = v[0];
#pragma unroll
  for (int e = 1; e < E; ++e) top = fmaxf(top, v[e]);
  top = wave_max(top);
  if ((threadIdx.x & 63) == 0) s.wave[threadIdx.x >> 6] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWhole / kWave; ++w) top = fmaxf(top, s.wave[w]);
  if (top == -__builtin_inff()) return write_none(a, row);
  const Row r = row_settings(a, row, top);
  settle_all(r, v);
  Cut cut{kBins, -1, 0, 0};
  u64 last = ~0ull;
  if (r.cuts()) {
    if (r.k > 0) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int bin = bin_of(r, v[e]);
        if (bin < kNoBin) atomicAdd(&s.counts[bin], 1u);
      }
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int bin = bin_of(r, v[e]);
        if (bin < kNoBin) atomicAdd(&s.bins[bin], weight_of(exponent(r, v[e]), s.table));
        apart(e);
      }
    }
    __syncthreads();
    const u64 own[1] = {r.k > 0 ? (u64)s.counts[threadIdx.x] : s.bins[threadIdx.x]};
    cut = find_cut<kWhole>(r, own, s.scan[0], s.found);
    if (cut.last >= 0) {
      again(v);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int bin = bin_of(r, v[e]);
        if (bin >= cut.first && bin <= cut.last) {
          const int at = atomicAdd(&s.listed, 1);
          if (at < kList) s.list[at] = make_uint2(i0 + e, __builtin_bit_cast(uint32_t, v[e]));
        }
      }
      __syncthreads();
      const int count = s.listed;
      if (count <= kList) {
        last = cut_tokens<kWhole>(r, cut, count, s.table, s.digits, s.few, s.scan[1],
                                  [&](int n, float* x) __attribute__((always_inline)) {
                                    const uint2 l = s.list[n];
                                    *x = __builtin_bit_cast(float, l.y);
                                    return (int)l.x;
                                  },
                                  [](u64, u64) {});
      } else {  // too many to list: all logits again, from the caches
        last = cut_list<kWhole>(r, cut, s.digits, s.scan[1], [&](auto f) __attribute__((always_inline)) {
          for (int i = threadIdx.x; i < a.vocab; i += kWhole) {
            const float x = settle(r, load_one<DT>(p, i));
            const int bin = bin_of(r, x);
            if (bin >= cut.first && bin <= cut.last) f(rank_key(x, i), weight_of(exponent(r, x), s.table));
          }
        }, [](u64, u64) {});
      }
    }
  }
  again(v);
  constexpr int kParts = E / 4;
  u64 part[kParts], sum = 0, total;  // every four tokens' weights
#pragma unroll
  for (int j = 0; j < kParts; ++j) {
    part[j] = 0;
#pragma unroll
    for (int e = 4 * j; e < 4 * j + 4; ++e) part[j] += kept_weight(r, cut, last, v[e], i0 + e, s.table);
    sum += part[j];
    __builtin_amdgcn_sched_barrier(0);
  }
  u64 upto = block_scan<kWhole>(sum, s.scan[2], &total);
  const u64 draw = draw_of(a, r, row, total);
  if (draw >= upto && draw < upto + sum) {
    int at = 0;
    float x[4] = {v[0], v[1], v[2], v[3]};
    bool past = true;
#pragma unroll
    for (int j = 0; j + 1 < kParts; ++j) {
      past = past && draw >= upto + part[j];
      if (past) {
        upto += part[j];
        at = 4 * j + 4;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = v[4 * j + 4 + e];
      }
    }
    again(x);
    write_token(a, r, row, i0 + at, x, [&](int e) __attribute__((always_inline)) {
      return kept_weight(r, cut, last, x[e], i0 + at + e, s.table);
    }, upto, draw, total);
  }
}

// ---- rows in chunks ----------------------------------------------------------------------
// Largest logit of a row from its chunks', every wavefront for itself.
__device__ __forceinline__ float row_top(const SampleArgs& a, int row) {
  float v = -__builtin_inff();
#pragma unroll
  for (int j = 0; j < kSampleMaxChunks / kWave; ++j) {
    const int c = j * kWave + (int)(threadIdx.x & 63);
    if (c < a.chunks) v = fmaxf(v, a.tops[(int64_t)row * a.chunks + c]);
  }
  return wave_max(v);
}

template <int DT>
__global__ __launch_bounds__(kThreads) void tops_kernel(SampleArgs a) {
  __shared__ float wave[kThreads / kWave];
  const int row = (int)(blockIdx.x / (unsigned)a.chunks), chunk = (int)(blockIdx.x - (unsigned)row * a.chunks);
  float v[kRun];
  load_run<DT>(row_of(a, row, DT), chunk * kChunk + (int)threadIdx.x * kRun, a.vocab, v);
  // the row's bins, for the next launch
  if (a.bins)
    for (int b = chunk * kThreads + (int)threadIdx.x; b < kBins; b += a.chunks * kThreads)
      a.bins[(int64_t)row * kBins + b] = 0;
  float top = v[0];
#pragma unroll
  for (int e = 1; e < kRun; ++e) top = fmaxf(top, v[e]);
  top = wave_max(top);
  if ((threadIdx.x & 63) == 0) wave[threadIdx.x >> 6] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / kWave; ++w) top = fmaxf(top, wave[w]);
  if (threadIdx.x == 0) a.tops[blockIdx.x] = top;
}

template <int DT>
__global__ __launch_bounds__(kThreads) void bins_kernel(SampleArgs a) {
  __shared__ double table[256];
  __shared__ u64 bins[kBins];
  const int row = (int)(blockIdx.x / (unsigned)a.chunks), chunk = (int)(blockIdx.x - (unsigned)row * a.chunks);
  float v[kRun];
  load_run<DT>(row_of(a, row, DT), chunk * kChunk + (int)threadIdx.x * kRun, a.vocab, v);
  const Row r = row_settings(a, row, row_top(a, row));
  if (!r.cuts()) return;
  settle_all(r, v);
  fill_table<kThreads>(table);
#pragma unroll
  for (int b = 0; b < kBins / kThreads; ++b) bins[b * kThreads + threadIdx.x] = 0;
  __syncthreads();
  uint32_t* counts = reinterpret_cast<uint32_t*>(bins);
  if (r.k > 0) {
#pragma unroll
    for (int e = 0; e < kRun; ++e) {
      const int bin = bin_of(r, v[e]);
      if (bin < kNoBin) atomicAdd(&counts[bin], 1u);
    }
  } else {
#pragma unroll
    for (int e = 0; e < kRun; ++e) {
      const int bin = bin_of(r, v[e]);
      if (bin < kNoBin) atomicAdd(&bins[bin], weight_of(exponent(r, v[e]), table));
    }
  }
  __syncthreads();
#pragma unroll
  for (int b = 0; b < kBins / kThreads; ++b) {
    const int i = b * kThreads + threadIdx.x;
    const u64 n = r.k > 0 ? (u64)counts[i] : bins[i];
    if (n > 0) atomicAdd(a.bins + (int64_t)row * kBins + b * kThreads + threadIdx.x, n);
  }
}

template <int DT>
__global__ __launch_bounds__(kThreads) void sums_kernel(SampleArgs a) {
  __shared__ double table[256];
  __shared__ Scan<kThreads> scan[2];
  __shared__ u64 found[2];
  __shared__ int listed;
  const int row = (int)(blockIdx.x / (unsigned)a.chunks), chunk = (int)(blockIdx.x - (unsigned)row * a.chunks);
  float v[kRun];
  load_run<DT>(row_of(a, row, DT), chunk * kChunk + (int)threadIdx.x * kRun, a.vocab, v);
  u64 own[kBins / kThreads] = {};
  if (a.bins) {
    const ulonglong2* from = reinterpret_cast<const ulonglong2*>(a.bins + (int64_t)row * kBins) + 2 * threadIdx.x;
    const ulonglong2 lo = from[0], hi = from[1];
    static_assert(kBins / kThreads == 4, "two loads of two");
    own[0] = lo.x, own[1] = lo.y, own[2] = hi.x, own[3] = hi.y;
  }
  fill_table<kThreads>(table);
  if (threadIdx.x == 0) listed = 0;
  const Row r = row_settings(a, row, row_top(a, row));
  settle_all(r, v);
  const Cut cut = find_cut<kThreads>(r, own, scan[0], found);
  __syncthreads();
  u64 sum = 0;
#pragma unroll
  for (int e = 0; e < kRun; ++e) {
    int bin = -1;
    if (cut.last >= 0) {
      bin = bin_of(r, v[e]);
      if (bin > cut.last) continue;
    }
    if (bin < cut.first) {
      const u64 w = weight_of(exponent(r, v[e]), table);
      sum += w >= r.w_min ? w : 0;
    } else {
      a.list[(int64_t)blockIdx.x * kChunk + atomicAdd(&listed, 1)] =
          make_uint2(chunk * kChunk + (int)threadIdx.x * kRun + e, __builtin_bit_cast(uint32_t, v[e]));
    }
  }
  u64 total;
  block_scan<kThreads>(sum, scan[1], &total);  // (and `listed` is whole)
  if (threadIdx.x == 0) {
    a.sums[blockIdx.x] = total;
    a.counts[blockIdx.x] = listed;
    if (chunk == 0) {
      a.cuts[row] = make_int4(cut.first, cut.last, 0, 0);
      a.cut_sums[2 * row] = cut.before;
      a.cut_sums[2 * row + 1] = cut.target;
    }
  }
}

struct ChooseLds {
  Scan<kChoose> scan[4];
  double table[256];
  u64 chunk_sums[kSampleMaxChunks];
  int starts[kSampleMaxChunks + 1];
  u64 found[2];
  Digits digits;
  Few few;
};

template <int DT>
__global__ __launch_bounds__(kChoose) void choose_kernel(SampleArgs a) {
  static_assert(kSampleMaxChunks <= kChoose, "a thread a chunk");
  __shared__ ChooseLds s;
  const int row = blockIdx.x;
  const void* p = row_of(a, row, DT);
  const int64_t first_chunk = (int64_t)row * a.chunks;
  const bool mine = (int)threadIdx.x < a.chunks;
  const int own_listed = mine ? a.counts[first_chunk + threadIdx.x] : 0;
  const u64 own_sum = mine ? a.sums[first_chunk + threadIdx.x] : 0;
  const int4 bins = a.cuts[row];
  const Cut cut{bins.x, bins.y, a.cut_sums[2 * row], a.cut_sums[2 * row + 1]};
  fill_table<kChoose>(s.table);
  const Row r = row_settings(a, row, row_top(a, row));
  if (r.top == -__builtin_inf()) return write_none(a, row);
  // places of the chunks' tokens in one list
  u64 listed;
  const u64 start = block_scan<kChoose>((u64)own_listed, s.scan[0], &listed);
  if (mine) {
    s.starts[threadIdx.x] = (int)start;
    s.chunk_sums[threadIdx.x] = own_sum;
  }
  __syncthreads();
  u64 last = ~0ull;  // key of the last token that top-k and top-p leave
  auto token_at = [&](int n, float* x) __attribute__((always_inline)) {
    int lo = 0, hi = a.chunks;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s.starts[mid] <= n) lo = mid; else hi = mid;
    }
    const uint2 l = a.list[(first_chunk + lo) * kChunk + (n - s.starts[lo])];
    *x = __builtin_bit_cast(float, l.y);
    return (int)l.x;
  };
  if (cut.first == 0 && listed <= kFew) {  // nothing but listed tokens, and few of them
    u64 key = 0, w = 0;
    float v = 0.0f;
    if (threadIdx.x < listed) {
      const int token = token_at(threadIdx.x, &v);
      key = rank_key(v, token);
      w = weight_of(exponent(r, v), s.table);
    }
    last = cut_few<kChoose>(r, cut, (int)listed, key, w, s.few);
    return draw_few<kChoose>(a, r, row, (int)listed, key, w, v, last, s.few);
  }
  if (listed > 0) {
    last = cut_tokens<kChoose>(
        r, cut, (int)listed, s.table, s.digits, s.few, s.scan[1], token_at,
        [&](u64 key, u64 w) __attribute__((always_inline)) { atomicAdd(&s.chunk_sums[(uint32_t)key / kChunk], w); });
    __syncthreads();
  }
  // the chunk that the draw falls into, and the token
  u64 total, all;
  const u64 own = mine ? s.chunk_sums[threadIdx.x] : 0;
  const u64 before = block_scan<kChoose>(own, s.scan[2], &total);
  u64 draw = draw_of(a, r, row, total);
  if (draw >= before && draw < before + own) {
    s.found[0] = threadIdx.x;
    s.found[1] = draw - before;
  }
  __syncthreads();
  const int chunk = (int)s.found[0];
  draw = s.found[1];
  constexpr int kPer = kChunk / kChoose;
  const int i0 = chunk * kChunk + (int)threadIdx.x * kPer;
  float v[kPer];
  load_run<DT>(p, i0, a.vocab, v);
  settle_all(r, v);
  u64 w[kPer], sum = 0;
#pragma unroll
  for (int e = 0; e < kPer; ++e) sum += w[e] = kept_weight(r, cut, last, v[e], i0 + e, s.table);
  const u64 upto = block_scan<kChoose>(sum, s.scan[3], &all);
  if (draw >= upto && draw < upto + sum)
    write_token(a, r, row, i0, v, [&](int e) __attribute__((always_inline)) { return w[e]; }, upto, draw, total);
}

template <int DT>
hipError_t launch_t(const SampleArgs& a, hipStream_t stream) {
  const dim3 rows((unsigned)a.rows);
  if (a.chunks == 0) {
    if (a.vocab <= 4 * kWhole)
      hipLaunchKernelGGL((whole_kernel<DT, 4>), rows, dim3(kWhole), 0, stream, a);
    else if (a.vocab <= 16 * kWhole)
      hipLaunchKernelGGL((whole_kernel<DT, 16>), rows, dim3(kWhole), 0, stream, a);
    else
      hipLaunchKernelGGL((whole_kernel<DT, 32>), rows, dim3(kWhole), 0, stream, a);
    return hipGetLastError();
  }
  const dim3 grid((unsigned)(a.rows * (int64_t)a.chunks)), block(kThreads);
  hipLaunchKernelGGL((tops_kernel<DT>), grid, block, 0, stream, a);
  if (a.bins) hipLaunchKernelGGL((bins_kernel<DT>), grid, block, 0, stream, a);
  hipLaunchKernelGGL((sums_kernel<DT>), grid, block, 0, stream, a);
  hipLaunchKernelGGL((choose_kernel<DT>), rows, dim3(kChoose), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_sample(const SampleArgs& a, hipStream_t stream) {
  return a.dtype == 0 ? launch_t<0>(a, stream) : a.dtype == 1 ? launch_t<1>(a, stream) : launch_t<2>(a, stream);
}

}  // namespace q4
