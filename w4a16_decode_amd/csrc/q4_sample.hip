// The next tokens from rows of logits (include/q4_serve.h).
//
// Weights are whole numbers: w_i = rint(2^shift exp((l_i - m) / T)) in 64 bits, a row's sum below
// 2^63. Their sums are exact, so any split of a row over workgroups and any order of additions
// (atomics among them) give the same cuts and the same token.
//
// A row is split into chunks of 4096 logits, a workgroup each. Four launches, each a pass over
// what the one before left (the last three read the logits from the caches):
//   tops    the chunks' largest logits;
//   bins    the row's weights (top-p) or tokens (top-k) by the weight's logarithm, 1024 bins: the
//           bin that a cut falls into follows from their sums alone. Left out without cuts;
//   sums    per chunk the sum of the weights before that bin, and a list of the tokens in it;
//   choose  a workgroup a row: the cut inside the bin, the chunk that the draw falls into, and
//           the token in it.
// Cuts inside a bin go by rank, key = (descending logit, ascending index) in 64 bits, without
// ties: digit by digit from the first one that differs, sums over the tokens that share the digits
// found so far by their next one. With top-k and top-p both, top-p's total is that of
// the tokens top-k left, so the list holds all tokens down to top-k's bin.
#include "q4_device.h"
#include "q4_internal.h"

namespace q4 {
namespace {

typedef unsigned long long u64;

constexpr int kChunk = kSampleChunk, kThreads = 256, kGroups = kChunk / kThreads / 4;
constexpr int kChoose = 512;                  // threads of the last launch
constexpr int kHeld = 8;                      // listed tokens one of its threads holds
constexpr int kBins = kSampleBins, kDigits = 256;

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

// Logits i .. i + 3 (rows may start at any element: the loads promise no more); -infinity behind the end.
template <int DT>
__device__ __forceinline__ void load_four(const void* p, int i, int vocab, float (&v)[4]) {
  if (i + 4 <= vocab) {
    if constexpr (DT == 2) {
      float4_t x;
      __builtin_memcpy(&x, static_cast<const float*>(p) + i, 16);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = clean(x[e]);
    } else {
      uint16_t x[4];
      __builtin_memcpy(x, static_cast<const uint16_t*>(p) + i, 8);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = clean(DT == 1 ? bf16(x[e]) : (float)__builtin_bit_cast(_Float16, x[e]));
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = i + e < vocab ? load_one<DT>(p, i + e) : -__builtin_inff();
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

// A row's settings. Greedy (temperature <= 0): only the largest logits have weight, and the draw is 0.
struct Row {
  float top;     // largest logit
  double slope;  // log2(e) / temperature
  double shift;
  float bin_scale;
  int k;  // 0: no top-k
  bool cut_p, greedy;
  double p;
  u64 w_min;  // smallest weight that min-p leaves
};

__device__ __forceinline__ Row row_settings(const SampleArgs& a, int row, float top) {
  Row r;
  r.top = top;
  const float t = a.temperature ? a.temperature[row] : 1.0f;
  r.greedy = !(t > 0.0f);
  r.slope = r.greedy ? __builtin_inf() : 1.4426950408889634 / (double)t;
  r.shift = (double)a.shift;
  r.bin_scale = (float)kBins / (float)(a.shift + 2);
  r.k = a.top_k ? a.top_k[row] : 0;
  if (r.greedy || r.k < 0 || r.k >= a.vocab) r.k = 0;
  r.p = a.top_p ? (double)a.top_p[row] : 1.0;
  r.cut_p = !r.greedy && r.p < 1.0;
  const double pm = a.min_p ? (double)a.min_p[row] : 0.0;
  r.w_min = pm > 0.0 ? (u64)ceil(ldexp(pm < 1.0 ? pm : 1.0, a.shift)) : 1;
  return r;
}

// log2 of the weight; below -1 (or NaN, where an infinity met a zero): no weight.
__device__ __forceinline__ double exponent(const Row& r, float v) {
  return v == r.top ? r.shift : __builtin_fma((double)v - (double)r.top, r.slope, r.shift);
}

// rint(2^z), -1 <= z <= 50: with k = rint(256 z), 2^(k / 256) from the table and 2^(z - k / 256) by its
// series to the fourth power, whose next term is below 2^-54; the whole is within 2^-50 of
// itself before the rounding.
__device__ __forceinline__ u64 weight_of(double z, const double* table) {
  if (!(z >= -1.0)) return 0;
  constexpr double kMagic = 26388279066624.0;  // 1.5 * 2^44: the sum's last bit is 1/256
  const double m = z + kMagic;
  const int k = (int)(uint32_t)__builtin_bit_cast(u64, m);
  const double x = (z - (m - kMagic)) * 0.6931471805599453;
  double s = __builtin_fma(x, 1.0 / 24, 1.0 / 6);
  s = __builtin_fma(x, s, 0.5);
  s = __builtin_fma(x, s, 1.0);
  s = __builtin_fma(x, s, 1.0);
  const double w = ldexp(table[k & 255] * s, k >> 8);
  return __builtin_bit_cast(u64, w + 4503599627370496.0) & 0xFFFFFFFFFFFFFull;  // + 2^52: rounded to a whole number
}
__device__ __forceinline__ int bin_of(const Row& r, double z) {  // of a token with weight
  return min(kBins - 1, (int)((float)(r.shift - z) * r.bin_scale));
}

template <int N>
struct Scan {
  u64 wave[N / kWave];
};

// Sum of the values of the threads before this one; *total: of all.
template <int N>
__device__ __forceinline__ u64 block_scan(u64 v, Scan<N>& s, u64* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  u64 incl = v;
#pragma unroll
  for (int m = 1; m < kWave; m <<= 1) {
    const u64 up = __shfl_up(incl, m, 64);
    if (lane >= m) incl += up;
  }
  if (lane == kWave - 1) s.wave[wave] = incl;
  __syncthreads();
  u64 before = incl - v, all = 0;
#pragma unroll
  for (int w = 0; w < N / kWave; ++w) {
    const u64 x = s.wave[w];
    if (w < wave) before += x;
    all += x;
  }
  __syncthreads();  // s may be written again
  *total = all;
  return before;
}

template <int N>
__device__ __forceinline__ float block_max(float v, float* wave) {
#pragma unroll
  for (int m = 1; m < kWave; m <<= 1) v = fmaxf(v, __shfl_xor(v, m, 64));
  if ((threadIdx.x & 63) == 0) wave[threadIdx.x >> 6] = v;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < N / kWave; ++w) v = fmaxf(v, wave[w]);
  return v;
}

// Largest logit of a row from its chunks'.
template <int N>
__device__ __forceinline__ float row_top(const SampleArgs& a, int row, float* wave) {
  float v = -__builtin_inff();
  for (int c = threadIdx.x; c < a.chunks; c += N) v = fmaxf(v, a.tops[(int64_t)row * a.chunks + c]);
  return block_max<N>(v, wave);
}

template <int DT>
__global__ __launch_bounds__(kThreads) void tops_kernel(SampleArgs a) {
  __shared__ float wave[kThreads / kWave];
  const int row = (int)(blockIdx.x / (unsigned)a.chunks), chunk = (int)(blockIdx.x - (unsigned)row * a.chunks);
  const void* p = row_of(a, row, DT);
  float top = -__builtin_inff();
#pragma unroll
  for (int j = 0; j < kGroups; ++j) {
    float v[4];
    load_four<DT>(p, chunk * kChunk + (j * kThreads + (int)threadIdx.x) * 4, a.vocab, v);
    top = fmaxf(fmaxf(fmaxf(top, v[0]), fmaxf(v[1], v[2])), v[3]);
  }
  top = block_max<kThreads>(top, wave);
  if (threadIdx.x == 0) a.tops[blockIdx.x] = top;
  // the row's bins, for the next launch
  if (a.bins)
    for (int b = chunk * kThreads + (int)threadIdx.x; b < kBins; b += a.chunks * kThreads)
      a.bins[(int64_t)row * kBins + b] = 0;
}

template <int DT>
__global__ __launch_bounds__(kThreads) void bins_kernel(SampleArgs a) {
  __shared__ float wave[kThreads / kWave];
  __shared__ double table[256];
  __shared__ u64 bins[kBins];
  const int row = (int)(blockIdx.x / (unsigned)a.chunks), chunk = (int)(blockIdx.x - (unsigned)row * a.chunks);
  const void* p = row_of(a, row, DT);
  float v[kGroups][4];
#pragma unroll
  for (int j = 0; j < kGroups; ++j)
    load_four<DT>(p, chunk * kChunk + (j * kThreads + (int)threadIdx.x) * 4, a.vocab, v[j]);
  table[threadIdx.x] = exp2((double)threadIdx.x / 256);
  for (int b = threadIdx.x; b < kBins; b += kThreads) bins[b] = 0;
  const Row r = row_settings(a, row, row_top<kThreads>(a, row, wave));  // (a barrier)
  if (r.k == 0 && !r.cut_p) return;
#pragma unroll
  for (int j = 0; j < kGroups; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const double z = exponent(r, v[j][e]);
      const u64 w = weight_of(z, table);
      if (w > 0) atomicAdd(&bins[bin_of(r, z)], r.k > 0 ? 1 : w);
    }
  __syncthreads();
  for (int b = threadIdx.x; b < kBins; b += kThreads)
    if (bins[b] > 0) atomicAdd(a.bins + (int64_t)row * kBins + b, bins[b]);
}

// Bins that a row's cuts need a closer look at: first .. last are listed, those before stay whole, and what
// comes before `first` in the sum that the cut goes by.
struct Cut {
  int first, last;
  u64 before;
  u64 target;  // the cut goes after the token with which the sum reaches it; 0: nothing is cut
};

template <int N>
__device__ __forceinline__ Cut find_cut(const SampleArgs& a, const Row& r, int row, Scan<N>& s, u64* found) {
  if (r.k == 0 && !r.cut_p) return Cut{kBins, -1, 0, 0};
  constexpr int kPer = kBins / N;
  u64 own[kPer], sum = 0, total;
#pragma unroll
  for (int i = 0; i < kPer; ++i) sum += own[i] = a.bins[(int64_t)row * kBins + threadIdx.x * kPer + i];
  u64 before = block_scan<N>(sum, s, &total);
  u64 target = (u64)r.k;
  if (r.k == 0) {
    const double part = ceil(r.p * (double)total);
    target = part >= 1.0 ? (u64)part : 1;
  }
  const bool all = r.k > 0 && target >= total;  // top-k leaves every token that has weight
  target = target < total ? target : total;
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
  if (r.k > 0 && r.cut_p) return Cut{0, at, 0, all ? 0 : target};
  return all ? Cut{kBins, -1, 0, 0} : Cut{at, at, found[1], target};
}

template <int DT>
__global__ __launch_bounds__(kThreads) void sums_kernel(SampleArgs a) {
  __shared__ float wave[kThreads / kWave];
  __shared__ double table[256];
  __shared__ Scan<kThreads> scan;
  __shared__ u64 found[2];
  __shared__ int listed;
  const int row = (int)(blockIdx.x / (unsigned)a.chunks), chunk = (int)(blockIdx.x - (unsigned)row * a.chunks);
  const void* p = row_of(a, row, DT);
  float v[kGroups][4];
#pragma unroll
  for (int j = 0; j < kGroups; ++j)
    load_four<DT>(p, chunk * kChunk + (j * kThreads + (int)threadIdx.x) * 4, a.vocab, v[j]);
  table[threadIdx.x] = exp2((double)threadIdx.x / 256);
  if (threadIdx.x == 0) listed = 0;
  const Row r = row_settings(a, row, row_top<kThreads>(a, row, wave));  // (a barrier)
  const Cut cut = find_cut<kThreads>(a, r, row, scan, found);
  u64 sum = 0;
#pragma unroll
  for (int j = 0; j < kGroups; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const double z = exponent(r, v[j][e]);
      const u64 w = weight_of(z, table);
      if (w == 0) continue;
      const int bin = cut.last < 0 ? 0 : bin_of(r, z);
      if (bin < cut.first)
        sum += w >= r.w_min ? w : 0;
      else if (bin <= cut.last)
        a.list[(int64_t)blockIdx.x * kChunk + atomicAdd(&listed, 1)] =
            (uint16_t)((j * kThreads + (int)threadIdx.x) * 4 + e);
    }
  u64 total;
  block_scan<kThreads>(sum, scan, &total);
  if (threadIdx.x == 0) {
    a.sums[blockIdx.x] = total;
    a.counts[blockIdx.x] = listed;
    if (chunk == 0) a.cuts[row] = make_int4(cut.first, cut.last, 0, 0);
    if (chunk == 0) {
      a.cut_sums[2 * row] = cut.before;
      a.cut_sums[2 * row + 1] = cut.target;
    }
  }
}

struct Chosen {
  Scan<kChoose> scan;
  double table[256];
  float wave[kChoose / kWave];
  u64 sums[kDigits];
  uint32_t counts[kDigits];
  u64 chunk_sums[kSampleMaxChunks];
  int starts[kSampleMaxChunks + 1];
  u64 found[4];
  u64 bits[2];
};

// Smallest key up to which the listed tokens with keys <= last add up to `target` or more
// (1 <= target <= their total). each(f): f(key, weight) for this thread's; ONES: a token counts 1.
template <bool ONES, typename Each>
__device__ __forceinline__ u64 select_key(u64 last, u64 target, Chosen& s, Each each) {
  __syncthreads();  // bits and found of an earlier cut have been read
  // the digits that differ
  if (threadIdx.x == 0) s.bits[0] = ~0ull, s.bits[1] = 0;
  __syncthreads();
  u64 low = ~0ull, high = 0;
  each([&](u64 key, u64) __attribute__((always_inline)) {
    if (key > last) return;
    low = key < low ? key : low;
    high = key > high ? key : high;
  });
#pragma unroll
  for (int m = 1; m < kWave; m <<= 1) {
    const u64 l = __shfl_xor(low, m, 64), h = __shfl_xor(high, m, 64);
    low = l < low ? l : low;
    high = h > high ? h : high;
  }
  if ((threadIdx.x & 63) == 0) {
    atomicMin(&s.bits[0], low);
    atomicMax(&s.bits[1], high);
  }
  __syncthreads();
  low = s.bits[0], high = s.bits[1];
  if (low == high) return low;
  int bit = 64 - __builtin_clzll(low ^ high);  // digits from this bit down
  u64 prefix = bit < 64 ? low >> bit << bit : 0, before = 0;
  while (bit > 0) {
    const int width = bit < 8 ? bit : 8, at = bit - width;
    if (threadIdx.x < kDigits) s.sums[threadIdx.x] = 0, s.counts[threadIdx.x] = 0;
    __syncthreads();
    each([&](u64 key, u64 w) __attribute__((always_inline)) {
      if (key > last || (bit < 64 && (key ^ prefix) >> bit != 0)) return;
      const int d = (int)(key >> at) & ((1 << width) - 1);
      if (!ONES) atomicAdd(&s.sums[d], w);
      atomicAdd(&s.counts[d], 1u);
    });
    __syncthreads();
    u64 total;
    const u64 own = threadIdx.x < kDigits ? ONES ? (u64)s.counts[threadIdx.x] : s.sums[threadIdx.x] : 0;
    const u64 sum = before + block_scan<kChoose>(own, s.scan, &total);
    if (target > sum && target <= sum + own) {
      s.found[0] = threadIdx.x;
      s.found[1] = sum;
      s.found[2] = s.counts[threadIdx.x];
    }
    __syncthreads();
    prefix |= s.found[0] << at;
    before = s.found[1];
    bit = at;
    const bool one = s.found[2] == 1;
    __syncthreads();
    if (one && bit > 0) {  // the token itself
      each([&](u64 key, u64) __attribute__((always_inline)) {
        if (key <= last && (key ^ prefix) >> bit == 0) s.found[3] = key;
      });
      __syncthreads();
      return s.found[3];
    }
  }
  return prefix;
}

template <int DT>
__global__ __launch_bounds__(kChoose) void choose_kernel(SampleArgs a) {
  __shared__ Chosen s;
  const int row = blockIdx.x;
  const void* p = row_of(a, row, DT);
  const int64_t first_chunk = (int64_t)row * a.chunks;
  const int4 cut_bins = a.cuts[row];
  const u64 cut_before = a.cut_sums[2 * row], cut_target = a.cut_sums[2 * row + 1];
  if (threadIdx.x < 256) s.table[threadIdx.x] = exp2((double)threadIdx.x / 256);
  const Row r = row_settings(a, row, row_top<kChoose>(a, row, s.wave));
  if (r.top == -__builtin_inff()) {
    if (threadIdx.x == 0) {
      a.tokens[row] = -1;
      if (a.probs) a.probs[row] = 0.0f;
    }
    return;
  }
  // places of the chunks' tokens in one list
  static_assert(kSampleMaxChunks <= kChoose, "a thread a chunk");
  const bool mine = (int)threadIdx.x < a.chunks;
  u64 listed;
  const u64 start = block_scan<kChoose>(mine ? (u64)a.counts[first_chunk + threadIdx.x] : 0, s.scan, &listed);
  if (mine) {
    s.starts[threadIdx.x] = (int)start;
    s.chunk_sums[threadIdx.x] = a.sums[first_chunk + threadIdx.x];
  }
  if (threadIdx.x == 0) s.starts[a.chunks] = (int)listed;
  __syncthreads();
  const int count = (int)listed;

  u64 last = ~0ull;  // key of the last token that top-k and top-p leave
  if (count > 0) {
    auto token_at = [&](int i) __attribute__((always_inline)) {
      int lo = 0, hi = a.chunks;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s.starts[mid] <= i) lo = mid; else hi = mid;
      }
      return lo * kChunk + (int)a.list[(first_chunk + lo) * kChunk + (i - s.starts[lo])];
    };
    auto cut = [&](auto each) __attribute__((always_inline)) {
      if (r.k > 0 && cut_target > 0) last = select_key<true>(last, cut_target - cut_before, s, each);
      if (r.cut_p) {
        u64 target = cut_target - cut_before;
        if (r.k > 0) {
          u64 sum = 0, total;
          each([&](u64 key, u64 w) __attribute__((always_inline)) { sum += key <= last ? w : 0; });
          block_scan<kChoose>(sum, s.scan, &total);
          const double part = ceil(r.p * (double)total);
          target = part >= 1.0 ? (u64)part : 1;
          target = target < total ? target : total;
        }
        last = select_key<false>(last, target, s, each);
      }
      each([&](u64 key, u64 w) __attribute__((always_inline)) {
        if (key <= last && w >= r.w_min) atomicAdd(&s.chunk_sums[(uint32_t)key / kChunk], w);
      });
    };
    if (count <= kChoose * kHeld) {
      u64 keys[kHeld], weights[kHeld];
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        keys[i] = ~0ull, weights[i] = 0;
        const int n = i * kChoose + (int)threadIdx.x;
        if (n < count) {
          const int token = token_at(n);
          const float v = load_one<DT>(p, token);
          keys[i] = rank_key(v, token);
          weights[i] = weight_of(exponent(r, v), s.table);
        }
      }
      cut([&](auto f) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
          if (i * kChoose + (int)threadIdx.x < count) f(keys[i], weights[i]);
      });
    } else {
      cut([&](auto f) __attribute__((always_inline)) {
        for (int n = threadIdx.x; n < count; n += kChoose) {
          const int token = token_at(n);
          const float v = load_one<DT>(p, token);
          f(rank_key(v, token), weight_of(exponent(r, v), s.table));
        }
      });
    }
    __syncthreads();
  }

  // the chunk that the draw falls into, and the token
  u64 total;
  const u64 own = mine ? s.chunk_sums[threadIdx.x] : 0;
  const u64 before = block_scan<kChoose>(own, s.scan, &total);
  const double u = r.greedy ? 0.0 : (double)a.uniforms[row];
  const double at = u > 0.0 ? floor(u * (double)total) : 0.0;
  u64 draw = at < 9.2e18 ? (u64)at : total;
  draw = draw < total ? draw : total - 1;
  if (draw >= before && draw < before + own) {
    s.found[0] = threadIdx.x;
    s.found[1] = draw - before;
  }
  __syncthreads();
  const int chunk = (int)s.found[0];
  draw = s.found[1];
  constexpr int kPer = kChunk / kChoose;
  const int i0 = chunk * kChunk + (int)threadIdx.x * kPer;
  u64 w[kPer], sum = 0, all;
#pragma unroll
  for (int j = 0; j < kPer; j += 4) {
    float v[4];
    load_four<DT>(p, i0 + j, a.vocab, v);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const double z = exponent(r, v[e]);
      u64 x = weight_of(z, s.table);
      if (x < r.w_min) x = 0;
      if (x > 0 && cut_bins.y >= 0) {
        const int bin = bin_of(r, z);
        if (bin > cut_bins.y || (bin >= cut_bins.x && rank_key(v[e], i0 + j + e) > last)) x = 0;
      }
      w[j + e] = x;
      sum += x;
    }
  }
  u64 upto = block_scan<kChoose>(sum, s.scan, &all);
  if (draw >= upto && draw < upto + sum) {
    int i = 0;
#pragma unroll
    for (; i < kPer - 1; ++i) {
      upto += w[i];
      if (draw < upto) break;
    }
    a.tokens[row] = i0 + i;
    if (a.probs)
      a.probs[row] = r.greedy ? 1.0f
                              : (float)(exp2(exponent(r, load_one<DT>(p, i0 + i)) - r.shift) /
                                        ldexp((double)total, -a.shift));
  }
}

template <int DT>
hipError_t launch_t(const SampleArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)(a.rows * (int64_t)a.chunks)), block(kThreads);
  hipLaunchKernelGGL((tops_kernel<DT>), grid, block, 0, stream, a);
  if (a.bins) hipLaunchKernelGGL((bins_kernel<DT>), grid, block, 0, stream, a);
  hipLaunchKernelGGL((sums_kernel<DT>), grid, block, 0, stream, a);
  hipLaunchKernelGGL((choose_kernel<DT>), dim3((unsigned)a.rows), dim3(kChoose), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_sample(const SampleArgs& a, hipStream_t stream) {
  return a.dtype == 0 ? launch_t<0>(a, stream) : a.dtype == 1 ? launch_t<1>(a, stream) : launch_t<2>(a, stream);
}

}  // namespace q4
