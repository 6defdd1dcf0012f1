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
// Range of the weights. P = p * vs is rounded to float16 before the product (half a
// step, 2^-11 of each weight; its errors are independent and average over the keys).
// p lies in [0, 1] relative to the row's maximum, but vs can be anything a float16
// can be, and small products would fall among the subnormals. The exponent is
// therefore taken relative to m + E, E the exponent of the largest V scale so far minus
// kHeadroom: P stays in [0, 2^kHeadroom], 26 binades of full precision below its
// maximum. (Infinite scales do not count: their rows are not finite, others' unharmed.) The sum l carries the same factor, so it cancels in o = O / l.
#include <algorithm>

#include "q4_paged.h"

namespace q4 {
namespace {

constexpr int kStep = 2 * kTokTile;  // keys per step (MFMA K of the second product)
constexpr float kHeadroom = 12.0f;
constexpr float kLowest = -3.4028234663852886e38f;

__device__ __forceinline__ float4_t mfma(half8_t a, half8_t b, float4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }

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

template <int D>
__device__ __forceinline__ void load_codes(uint32_t (&w)[D / 32], const uint32_t* base, int lane) {
  if constexpr (D == 64) {
    const uint2 r = *reinterpret_cast<const uint2*>(base + 2 * lane);
    w[0] = r.x, w[1] = r.y;
  } else {
#pragma unroll
    for (int i = 0; i < D / 128; ++i) {
      const uint4 r = *reinterpret_cast<const uint4*>(base + (i * kWave + lane) * 4);
      w[4 * i] = r.x, w[4 * i + 1] = r.y, w[4 * i + 2] = r.z, w[4 * i + 3] = r.w;
    }
  }
}

// `tile` of the cache (D * 8 bytes of codes, GC * 16 scales, for K and for V).
template <int D, int GC>
__device__ __forceinline__ void load_tile(Tile<D, GC>& t, const PagedArgs& c, int64_t tile, int lane) {
  load_codes<D>(t.k, static_cast<const uint32_t*>(c.k_codes) + tile * (2 * D), lane);
  load_codes<D>(t.v, static_cast<const uint32_t*>(c.v_codes) + tile * (2 * D), lane);
  const uint16_t* ks = static_cast<const uint16_t*>(c.k_scales) + tile * (GC * kTokTile) + 4 * (lane >> 4);
  const uint16_t* vs = static_cast<const uint16_t*>(c.v_scales) + tile * (GC * kTokTile) + 4 * (lane >> 4);
#pragma unroll
  for (int g = 0; g < GC; ++g) {
    t.ks[g] = *reinterpret_cast<const uint2*>(ks + g * kTokTile);
    t.vs[g] = *reinterpret_cast<const uint2*>(vs + g * kTokTile);
  }
}

// Rows of one wavefront: sequence n's rows r0 .. r0 + 16 QT - 1 for KV head h.
template <int D, int GC, int QT>
struct Rows {
  static constexpr int KB = D / 32;       // 32-channel blocks
  static constexpr int BPG = KB / GC;     // of them per scale group
  half8_t q[QT][KB];
  int pos[QT];      // position of the lane's row (its own last visible key); -1: no row
  float m[QT];      // running maximum of the scores (times log2 e)
  float base[QT];   // m + E: what exponents are relative to
  float l[QT];      // the lane's share of the sum
  float4_t acc[QT][2 * KB];
};

template <int D, int GC, int QT>
__global__ __launch_bounds__(256) void attn_kernel(AttnArgs a, unsigned tiles) {
  using R = Rows<D, GC, QT>;
  constexpr int KB = R::KB, BPG = R::BPG;
  const int lane = threadIdx.x & 63;
  const int col = lane & 15, c4 = lane >> 4;
  const int head = (int)(blockIdx.x / tiles % a.cache.kv_heads), seq = (int)(blockIdx.x / tiles / a.cache.kv_heads);
  const int share = a.q_heads / a.cache.kv_heads;

  // the sequence's rows and length, kept inside what the arguments promise
  const int first = min(max(a.q_offsets[seq], 0), a.tokens);
  const int nq = min(min(max(a.q_offsets[seq + 1], first), a.tokens) - first, a.max_q);
  const int len = min(max(a.kv_lens[seq], 0), a.max_kv);
  const int rows = nq * share;
  const int r0 = (int)(blockIdx.x % tiles * 4 + threadIdx.x / kWave) * 16 * QT;
  if (r0 >= rows) return;

  R r;
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    const int m = r0 + 16 * t + col;
    const bool real = m < rows;
    const int i = min(m, rows - 1) / share, hs = min(m, rows - 1) - i * share;
    r.pos[t] = real ? len - nq + i : -1;
    const uint16_t* src = static_cast<const uint16_t*>(a.q) + (int64_t)(first + i) * a.q_stride +
                          (int64_t)(head * share + hs) * D + 8 * c4;
#pragma unroll
    for (int b = 0; b < KB; ++b) r.q[t][b] = as_half8(*reinterpret_cast<const uint4*>(src + 32 * b));
    r.m[t] = r.base[t] = kLowest;
    r.l[t] = 0.0f;
#pragma unroll
    for (int b = 0; b < 2 * KB; ++b) r.acc[t][b] = float4_t{0.f, 0.f, 0.f, 0.f};
  }

  // keys any of the rows sees: [t_first, t_last)
  const int pos_lo = len - nq + r0 / share;
  const int pos_hi = len - nq + (min(r0 + 16 * QT, rows) - 1) / share;
  const int t_last = pos_hi + 1;
  const int window = a.window > 0 ? a.window : t_last + 1;
  const int t_first = max(0, pos_lo - window + 1) / kStep * kStep;
  const int page_size = a.cache.page_size, tpp = page_size / kTokTile;
  const int32_t* table = a.block_table + (int64_t)seq * a.max_blocks;
  const float scale = a.scale * 1.4426950408889634f;
  const DequantRegs dq = DequantRegs::make();
  float exp_v = -64.0f;  // E (wave-uniform)
  uint32_t cap_v = 0;    // largest V scale that E covers, as float16 bits

  for (int t0 = t_first; t0 < t_last; t0 += kStep) {
    Tile<D, GC> tile[2];
    bool there[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      // a tile behind the last key, or of a page outside the cache, is read from a
      // valid place and masked
      const int key = min(t0 + 16 * j, (t_last - 1) / kTokTile * kTokTile);
      const int block = key / page_size;
      const int page = block < a.max_blocks ? table[block] : -1;
      there[j] = page >= 0 && page < a.cache.pages && t0 + 16 * j < t_last;
      const int64_t at = ((int64_t)(there[j] ? page : 0) * a.cache.kv_heads + head) * tpp + (key - block * page_size) / kTokTile;
      load_tile<D, GC>(tile[j], a.cache, at, lane);
    }
    const bool edge = t0 + kStep > pos_lo + 1 || t0 <= pos_hi - window || !there[0] || !there[1];

    // scores, base 2
    float ks[2][GC][4], vs[2][GC][4];
    uint32_t vmax = 0;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int g = 0; g < GC; ++g) {
        const half4_t kh = __builtin_bit_cast(half4_t, tile[j].ks[g]), vh = __builtin_bit_cast(half4_t, tile[j].vs[g]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // an infinite scale makes its key's score NaN (0 codes times infinity), not +-inf
          ks[j][g][i] = __builtin_fmaf((float)kh[i], scale, (float)kh[i] * 0.0f);
          const int key = t0 + 16 * j + 4 * c4 + i;
          const bool seen = !edge || (there[j] && key < t_last && key > pos_lo - window);
          // what no row sees may hold anything: 0 * NaN must not arise
          vs[j][g][i] = seen ? (float)vh[i] : 0.0f;
          const uint32_t bits = __builtin_bit_cast(uint16_t, vh[i]);
          vmax = max(vmax, seen && bits < 0x7C00u ? bits : 0u);
        }
      }
    if (__any(vmax > cap_v)) {
#pragma unroll
      for (int s = 1; s < 64; s <<= 1) vmax = max(vmax, (uint32_t)__shfl_xor((int)vmax, s, 64));
      cap_v = vmax | 0x3FFu;  // up to the end of its binade
      exp_v = (float)(int)(cap_v >> 10) - 14.0f - kHeadroom;
    }

    float s[QT][2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      half8_t ka[KB];
      const half2_t lo_bias = {(_Float16)-1032.0f, (_Float16)-1032.0f};
      const half2_t hi_bias = {(_Float16)-72.0f, (_Float16)-72.0f};
#pragma unroll
      for (int b = 0; b < KB; ++b) ka[b] = dequant8r(tile[j].k[b], dq, lo_bias, hi_bias);
#pragma unroll
      for (int t = 0; t < QT; ++t) {
#pragma unroll
        for (int g = 0; g < GC; ++g) {
          float4_t part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int b = 0; b < BPG; ++b) part = mfma(ka[g * BPG + b], r.q[t][g * BPG + b], part);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            s[t][j][i] = g == 0 ? part[i] * ks[j][g][i] : __builtin_fmaf(part[i], ks[j][g][i], s[t][j][i]);
        }
      }
    }
    if (edge) {
#pragma unroll
      for (int t = 0; t < QT; ++t)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = t0 + 16 * j + 4 * c4 + i;
            if (!there[j] || key > r.pos[t] || key <= r.pos[t] - window) s[t][j][i] = -__builtin_inff();
          }
    }

    // softmax step, weights to float16
    half8_t p[QT][GC];
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      float mx = r.m[t];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) mx = fmaxf(mx, s[t][j][i]);
      mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
      mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
      const float base = mx + exp_v;
      const float alpha = exp2_fast(r.base[t] - base);
      r.m[t] = mx;
      r.base[t] = base;
      r.l[t] *= alpha;
#pragma unroll
      for (int b = 0; b < 2 * KB; ++b) r.acc[t][b] *= alpha;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float e = exp2_fast(s[t][j][i] - base);
          r.l[t] += e;
#pragma unroll
          for (int g = 0; g < GC; ++g)  // a key that this row does not see may have an infinite scale
            p[t][g][4 * j + i] = (_Float16)(edge && s[t][j][i] == -__builtin_inff() ? 0.0f : e * vs[j][g][i]);
        }
    }

#pragma unroll
    for (int b = 0; b < KB; ++b) {
      const half8_t lo = v_operand<false>(tile[0].v[b], tile[1].v[b], dq);
      const half8_t hi = v_operand<true>(tile[0].v[b], tile[1].v[b], dq);
#pragma unroll
      for (int t = 0; t < QT; ++t) {
        r.acc[t][2 * b] = mfma(lo, p[t][b / BPG], r.acc[t][2 * b]);
        r.acc[t][2 * b + 1] = mfma(hi, p[t][b / BPG], r.acc[t][2 * b + 1]);
      }
    }
  }

#pragma unroll
  for (int t = 0; t < QT; ++t) {
    float l = r.l[t];
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const int m = r0 + 16 * t + col;
    if (m >= rows) continue;
    const int i = m / share, hs = m - i * share;
    uint16_t* dst = static_cast<uint16_t*>(a.out) + ((int64_t)(first + i) * a.q_heads + head * share + hs) * D + 4 * c4;
#pragma unroll
    for (int b = 0; b < 2 * KB; ++b) {
      half4_t h;
#pragma unroll
      for (int e = 0; e < 4; ++e) h[e] = (_Float16)(r.acc[t][b][e] * inv);
      *reinterpret_cast<uint2*>(dst + 16 * b) = __builtin_bit_cast(uint2, h);
    }
  }
}

template <int D, int GC>
hipError_t launch_t(const AttnArgs& a, hipStream_t stream) {
  const int64_t rows = (int64_t)a.max_q * (a.q_heads / a.cache.kv_heads);
  const unsigned tiles = (unsigned)((rows + 63) / 64);
  hipLaunchKernelGGL((attn_kernel<D, GC, 1>), dim3(tiles * a.cache.kv_heads * a.seqs), dim3(256), 0, stream, a, tiles);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attention(const AttnArgs& a, hipStream_t stream) {
  const int gc = a.cache.head_dim / a.cache.group;
  switch (a.cache.head_dim) {
    case 64: return gc == 1 ? launch_t<64, 1>(a, stream) : launch_t<64, 2>(a, stream);
    case 128:
      return gc == 1 ? launch_t<128, 1>(a, stream) : gc == 2 ? launch_t<128, 2>(a, stream) : launch_t<128, 4>(a, stream);
    default:
      return gc == 2 ? launch_t<256, 2>(a, stream) : gc == 4 ? launch_t<256, 4>(a, stream) : launch_t<256, 8>(a, stream);
  }
}

}  // namespace q4
