// RMS norm and rotation of the q and k heads, and the append of k and v into the
// paged INT4 cache (include/q4_attn.h), in one pass over the projection's rows.
//
// One wavefront owns a token; a lane holds 8 channels of a head (one 16-byte load),
// so D / 8 lanes make a head and a wavefront takes RPW = 512 / D heads at a time. The
// token's cosines and sines depend on the lane's channels only: they are loaded once
// and stay in registers for all of the token's heads. The mean square is a butterfly
// over the head's lanes; a rotation partner that sits rot_dim / 2 channels away is
// another lane's chunk (four dword shuffles), one that is adjacent is the lane's own.
// A wavefront takes its token's k heads, then v's, then q's: each loop holds only what its own
// arithmetic needs (one loop for all three kept k's float64 values live in q's: 88 us below).
// For q the norm's weights are folded into the cosines and sines and four loads are in flight.
//
// Bound: every head is read once and written once. 8191 tokens of 64 + 8 heads of 128, both
// normed: 302 MB in 63 to 65 us, 4.7 TB/s, the rate of a large copy. The append is bound by its
// arithmetic and by V's scattered bytes (16 tokens share a dword's neighbours): 4097 tokens
// of 32 + 8 + 8 heads, k in float64, 23.5 us, 3.8 TB/s; few tokens by the launch: 3.4 us. An append alone
// moves half that rate (393280 tokens of 8 heads in 850 us, 2.04 GB): V's bytes, and no load ahead.
//
// Rounding: q takes x * (w c) and y * (w s) in float32, a handful of roundings of 2^-24 before the
// one to float16. k, whose value next decides a 4-bit code, is float64 arithmetic on exact products x * w,
// rounded to float32 and that to float16 (k_row): off by half a float16 step and 2^-24 at most.
#include <algorithm>

#include "q4_paged.h"
#include "q4_rtn.h"

namespace q4 {
namespace {

// 1 / sqrt(v): v_rsq_f64 (about 26 bits) and one Newton step; 0 for infinity (where the step
// would make infinity * 0).
__device__ __forceinline__ double inv_sqrt(double v) {
  const double y = __builtin_amdgcn_rsq(v);
  return v < __builtin_inf() ? __builtin_fma(0.5 * y, __builtin_fma(-v * y, y, 1.0), y) : y;
}

// v plus the value of another lane of the same 16, picked by a DPP control (no LDS).
template <int CTRL>
__device__ __forceinline__ float add_dpp(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}
template <int CTRL>
__device__ __forceinline__ double add_dpp(double v) {
  const int lo = __builtin_amdgcn_update_dpp(0, __double2loint(v), CTRL, 0xF, 0xF, true);
  const int hi = __builtin_amdgcn_update_dpp(0, __double2hiint(v), CTRL, 0xF, 0xF, true);
  return v + __hiloint2double(hi, lo);
}

// Sum over a head's LPH lanes: neighbours, pairs, then mirrored halves of 8 and 16 lanes
// (whose quads, resp. eights, are equal by then).
template <int LPH, typename T>
__device__ __forceinline__ T head_sum(T v) {
  v = add_dpp<0xB1>(v);   // quad_perm [1, 0, 3, 2]
  v = add_dpp<0x4E>(v);   // quad_perm [2, 3, 0, 1]
  v = add_dpp<0x141>(v);  // row_half_mirror
  if (LPH >= 16) v = add_dpp<0x140>(v);  // row_mirror
  if (LPH >= 32) v += __shfl_xor(v, 16, 64);
  return v;
}

// Rotation factors of a lane's 8 channels: out[e] = h[e] * c[e] + partner[e] * s[e],
// s carrying the sign. `turn` is false for channels behind rot_dim (c = 1, s = 0).
constexpr int kAhead = 4;

struct Turn {
  float c[8], s[8];
  int partner;  // lane of the partner's chunk (half-split pairs)
  bool turn;
};

template <int D>
__device__ __forceinline__ void load_turn(const RopeArgs& a, int64_t token, int lane, Turn& t) {
  constexpr int LPH = D / 8;
  const int ch = 8 * (lane & (LPH - 1));
  t.turn = ch < a.rot;
  if (!t.turn) return;
  const int64_t pos = min(max((int64_t)a.positions[token], (int64_t)0), a.table_positions - 1);
  const float* row = a.table + pos * a.rot;
  if (a.interleaved) {
    const float4_t* p = reinterpret_cast<const float4_t*>(row + ch);
    const float4_t lo = p[0], hi = p[1];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float4_t v = e < 4 ? lo : hi;
      t.c[e] = v[(e & 2)];
      t.s[e] = (e & 1) ? v[(e & 2) + 1] : -v[(e & 2) + 1];
    }
    return;
  }
  const bool first = ch < a.rot / 2;
  t.partner = lane + (first ? a.rot / 16 : -(a.rot / 16));
  const float4_t* p = reinterpret_cast<const float4_t*>(row + 2 * (first ? ch : ch - a.rot / 2));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4_t v = p[i];
    t.c[2 * i] = v[0];
    t.c[2 * i + 1] = v[2];
    t.s[2 * i] = first ? -v[1] : v[1];
    t.s[2 * i + 1] = first ? -v[3] : v[3];
  }
}

// A norm's weights for a lane's channels and for its rotation partner's (zeros where there is no
// partner: an infinite weight must not meet its sine of 0).
struct Weights {
  half8_t own, other;
};

// The two halves of every dword swapped: adjacent channels.
__device__ __forceinline__ uint4 swap_pairs(uint4 r) {
  return make_uint4(r.x >> 16 | r.x << 16, r.y >> 16 | r.y << 16, r.z >> 16 | r.z << 16, r.w >> 16 | r.w << 16);
}

__device__ __forceinline__ uint4 masked(uint4 r, bool keep) {
  const uint32_t m = keep ? 0xFFFFFFFFu : 0u;
  return make_uint4(r.x & m, r.y & m, r.z & m, r.w & m);
}

template <int D>
__device__ __forceinline__ Weights load_weights(const void* w, int lane, const Turn& t, bool interleaved) {
  constexpr int LPH = D / 8;
  const uint4* p = static_cast<const uint4*>(w);
  const uint4 own = p[lane & (LPH - 1)];
  const uint4 other = interleaved ? swap_pairs(own) : p[t.partner & (LPH - 1)];
  return Weights{as_half8(own), as_half8(masked(other, t.turn))};
}

// The rotation partners of a lane's 8 channels; zeros where there is no rotation (the
// lane's own values would bring infinities into a product with sine 0).
__device__ __forceinline__ half8_t partners(half8_t x, const Turn& t, bool interleaved) {
  uint4 r = __builtin_bit_cast(uint4, x);
  if (interleaved) {
    r = swap_pairs(r);
  } else {
    r = make_uint4(__shfl(r.x, t.partner, 64), __shfl(r.y, t.partner, 64), __shfl(r.z, t.partner, 64),
                   __shfl(r.w, t.partner, 64));
  }
  return as_half8(masked(r, t.turn));
}

// q: norm and rotation in float32, with the weights already in c and s:
// (x (w c) + y (w' s)) / rms. About 55 instructions for 8 channels a lane.
template <int D>
__device__ __forceinline__ half8_t q_row(half8_t x, half8_t y, bool norm, float eps, const Turn& t, bool rotate) {
  float r = 1.0f;
  if (norm) {
    float sum = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const half2_t v = {x[e], x[e + 1]};
      sum = __builtin_amdgcn_fdot2(v, v, sum, false);
    }
    r = __builtin_amdgcn_rsqf(head_sum<D / 8>(sum) * (1.0f / D) + eps);  // within one ulp
  }
  half8_t out;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float v = (float)x[e] * t.c[e];
    if (rotate) v = __builtin_fmaf((float)y[e], t.s[e], v);  // else y is x, and infinity * 0 a NaN
    out[e] = (_Float16)(v * r);
  }
  return out;
}

// k: the same in float64, rounded to float32 and that to float16, as torch converts float64: a
// torch program that keeps its own float64 k gets these bits. (Off by half a float16 step and 2^-24
// of the value at most; rounding once instead, as numpy does, differs on ties of the second
// rounding, one value in 16000, and through them in one code of 10 million.)
template <int D>
__device__ __forceinline__ half8_t k_row(half8_t x, half8_t y, bool norm, const Weights& w, float eps, const Turn& t,
                                         bool rotate) {
  double r = 1.0;
  if (norm) {
    double sum = 0.0;
#pragma unroll
    for (int e = 0; e < 8; ++e) sum += (double)((float)x[e] * (float)x[e]);  // 22 bits: exact in float32
    r = inv_sqrt(head_sum<D / 8>(sum) * (1.0 / D) + (double)eps);
  }
  half8_t out;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    double v = (double)(norm ? (float)x[e] * (float)w.own[e] : (float)x[e]);  // exact too
    if (rotate) {
      const double o = (double)(norm ? (float)y[e] * (float)w.other[e] : (float)y[e]);
      v = v * (double)t.c[e] + o * (double)t.s[e];
    }
    if (norm) v *= r;
    float f = (float)v;
    asm("" : "+v"(f));  // the compiler would join the two conversions into one, in integer steps
    out[e] = (_Float16)f;
  }
  return out;
}

// INT4 codes of a lane's 8 values (one nibble each, element 0 lowest, two's complement
// q) and the float16 scale of its group of GL lanes: the KV cache's rule (q4_kv.hip). The
// group's largest magnitude is taken over float16 bit patterns, which order as the
// values do with infinity and NaN on top; such a group gets a NaN scale.
__device__ __forceinline__ uint32_t quantize8(half8_t h, int GL, _Float16* scale) {
  typedef uint16_t us2 __attribute__((ext_vector_type(2)));
  const uint4 bits = __builtin_bit_cast(uint4, h);
  auto mag = [](uint32_t w) { return __builtin_bit_cast(us2, w & 0x7FFF7FFFu); };
  us2 a2 = __builtin_elementwise_max(__builtin_elementwise_max(mag(bits.x), mag(bits.y)),
                                     __builtin_elementwise_max(mag(bits.z), mag(bits.w)));
  int a = max((int)a2.x, (int)a2.y);
  for (int m = 1; m < GL; m <<= 1) a = max(a, __shfl_xor(a, m, 64));
  const float amax = (float)__builtin_bit_cast(_Float16, (uint16_t)a);
  const _Float16 s16 =
      a < 0x7C00 ? (_Float16)(fmaxf(amax, 1e-12f) * (1.0f / 7.0f)) : __builtin_bit_cast(_Float16, (uint16_t)0x7E00);
  const float rcp = rtn_recip((float)s16);
  uint32_t word = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int q = (int)fminf(fmaxf(rtn_quot((float)h[e], rcp), -8.0f), 7.0f);
    word |= (uint32_t)(q & 0xF) << (4 * e);
  }
  *scale = s16;
  return word;
}

// Codes and scale of a lane's 8 channels of a token (row tt of its tile) into the cache.
template <int D, bool IS_V>
__device__ __forceinline__ void store_codes(const PagedArgs& c, half8_t x, uint32_t slot, bool stored, int head,
                                            int chunk) {
  constexpr int LPH = D / 8;
  _Float16 scale;
  const int GL = c.group / 8;
  const uint32_t word = quantize8(x, GL, &scale);
  const uint32_t partner = IS_V ? __shfl_xor(word, 2, 64) : 0u;  // channels + 16
  if (!stored) return;
  const int64_t tile = slot_tile(slot, c.page_size, c.kv_heads, head);
  const int tt = (int)(slot % (uint32_t)kTokTile);  // page_size is a multiple of the tile
  if (chunk % GL == 0) {
    uint16_t* sc = static_cast<uint16_t*>(IS_V ? c.v_scales : c.k_scales);
    sc[(tile * (LPH / GL) + chunk / GL) * kTokTile + tt] = __builtin_bit_cast(uint16_t, scale);
  }
  const uint32_t off = word ^ 0x88888888u;  // q + 8
  if (!IS_V) {
    uint32_t dw = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) dw |= ((off >> (4 * e)) & 0xFu) << (4 * nibble_of(e));
    static_cast<uint32_t*>(c.k_codes)[tile * (2 * D) + tile_dword<D>(chunk / 4, tt + 16 * (chunk & 3))] = dw;
  } else {
    // a byte holds channels 32m + r and 32m + 16 + r: the lanes of the two halves
    // write four of their eight bytes each
    const uint32_t po = partner ^ 0x88888888u;
    const int hi = (chunk >> 1) & 1;
    const uint32_t lo_word = hi ? po : off, hi_word = hi ? off : po;
    uint8_t* vc = static_cast<uint8_t*>(c.v_codes) + tile * (8 * D) + v_byte(tt & 3);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = 4 * hi + i;
      const int r = 8 * (chunk & 1) + e;
      vc[tile_dword<D>(chunk / 4, r + 16 * (tt >> 2)) * 4] =
          (uint8_t)(((lo_word >> (4 * e)) & 0xFu) | (((hi_word >> (4 * e)) & 0xFu) << 4));
    }
  }
}

// Heads of a token in units of RPW heads: k's, then (append) v's, then q's.
template <int D, bool APPEND>
__global__ __launch_bounds__(256, 6) void rope_kernel(RopeArgs a, int segs, int units_per_seg) {
  constexpr int LPH = D / 8;
  constexpr int RPW = kWave / LPH;
  const int lane = threadIdx.x & 63;
  const int64_t wave = (int64_t)blockIdx.x * (blockDim.x / kWave) + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t token = wave / segs;
  if (token >= a.tokens) return;
  const int nk = (a.kv_heads + RPW - 1) / RPW, nq = (a.q_heads + RPW - 1) / RPW;
  const int v0 = nk, q0 = APPEND ? 2 * nk : nk;  // first units of v and q
  const int u0 = (int)(wave - token * segs) * units_per_seg;
  const int u1 = min(u0 + units_per_seg, q0 + nq);
  const int sub = lane / LPH, chunk = lane & (LPH - 1);
  const bool rotate = a.rot > 0;
  auto fetch = [&](const void* p, int64_t stride, int head, int heads) __attribute__((always_inline)) {
    return head < heads ? *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + token * stride + head * D + 8 * chunk)
                        : make_uint4(0u, 0u, 0u, 0u);
  };
  auto store = [&](void* p, int64_t stride, int head, int heads, half8_t x) __attribute__((always_inline)) {
    if (head < heads)
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + token * stride + head * D + 8 * chunk) =
          __builtin_bit_cast(uint4, x);
  };
  Turn t;
  t.turn = false;
  t.partner = lane;
#pragma unroll
  for (int e = 0; e < 8; ++e) t.c[e] = 1.0f, t.s[e] = 0.0f;
  if (rotate) load_turn<D>(a, token, lane, t);
  uint32_t slot = 0;
  bool stored = false;
  if (APPEND) {
    slot = (uint32_t)a.slots[token];
    stored = (int64_t)slot < a.cache.pages * a.cache.page_size;
  }

  if (u0 < nk) {
    Weights w{};
    if (a.k_weight) w = load_weights<D>(a.k_weight, lane, t, a.interleaved);
    for (int u = u0; u < min(u1, nk); ++u) {
      const int head = u * RPW + sub;
      const half8_t x = as_half8(fetch(a.k, a.k_stride, head, a.kv_heads));
      half8_t y = x;
      if (rotate) y = partners(x, t, a.interleaved);
      const half8_t k = k_row<D>(x, y, a.k_weight != nullptr, w, a.eps, t, rotate);
      if (APPEND) store_codes<D, false>(a.cache, k, slot, stored && head < a.kv_heads, head, chunk);
      else store(a.k_out, a.k_out_stride, head, a.kv_heads, k);
    }
  }
  if (APPEND) {
    for (int u = max(u0, v0); u < min(u1, q0); ++u) {
      const int head = (u - v0) * RPW + sub;
      const half8_t x = as_half8(fetch(a.v, a.v_stride, head, a.kv_heads));
      store_codes<D, true>(a.cache, x, slot, stored && head < a.kv_heads, head, chunk);
    }
  }
  if (u1 <= q0) return;
  if (a.q_weight) {
    const Weights w = load_weights<D>(a.q_weight, lane, t, a.interleaved);
#pragma unroll
    for (int e = 0; e < 8; ++e) t.c[e] *= (float)w.own[e], t.s[e] *= (float)w.other[e];
  }
  // the next kAhead units' loads are in flight while kAhead are computed
  const int first = max(u0, q0) - q0, last = u1 - q0;
  uint4 raw[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) raw[i] = fetch(a.q, a.q_stride, (first + i) * RPW + sub, a.q_heads);
  for (int u = first; u < last; u += kAhead) {
    uint4 next[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) next[i] = fetch(a.q, a.q_stride, (u + kAhead + i) * RPW + sub, a.q_heads);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (u + i >= last) break;
      const half8_t x = as_half8(raw[i]);
      half8_t y = x;
      if (rotate) y = partners(x, t, a.interleaved);
      store(a.q_out, a.q_out_stride, (u + i) * RPW + sub, a.q_heads, q_row<D>(x, y, a.q_weight != nullptr, a.eps, t, rotate));
      raw[i] = next[i];
    }
  }
}

template <int D>
__global__ __launch_bounds__(256) void paged_dequant_kernel(PagedArgs c, const int32_t* __restrict__ slots,
                                                            int64_t tokens, uint16_t* __restrict__ k_out,
                                                            uint16_t* __restrict__ v_out) {
  constexpr int LPH = D / 8;
  const int64_t chunks = tokens * c.kv_heads * LPH;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < chunks; i += (int64_t)gridDim.x * blockDim.x) {
    const int chunk = (int)(i % LPH);
    const int64_t th = i / LPH;
    const int64_t token = th / c.kv_heads;
    const int head = (int)(th - token * c.kv_heads);
    const uint32_t slot = (uint32_t)slots[token];
    half8_t k, v;
#pragma unroll
    for (int e = 0; e < 8; ++e) k[e] = v[e] = (_Float16)0.0f;
    if ((int64_t)slot < c.pages * c.page_size) {
      const int64_t tile = slot_tile(slot, c.page_size, c.kv_heads, head);
      const int tt = (int)(slot % (uint32_t)kTokTile);
      const int64_t si = (tile * (D / c.group) + 8 * chunk / c.group) * kTokTile + tt;
      const float ks = (float)__builtin_bit_cast(_Float16, static_cast<const uint16_t*>(c.k_scales)[si]);
      const float vs = (float)__builtin_bit_cast(_Float16, static_cast<const uint16_t*>(c.v_scales)[si]);
      const uint32_t kw =
          static_cast<const uint32_t*>(c.k_codes)[tile * (2 * D) + tile_dword<D>(chunk / 4, tt + 16 * (chunk & 3))];
      const uint8_t* vc = static_cast<const uint8_t*>(c.v_codes) + tile * (8 * D) + v_byte(tt & 3);
      const int sh = 4 * ((chunk >> 1) & 1);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        k[e] = (_Float16)((float)((int)((kw >> (4 * nibble_of(e))) & 0xFu) - 8) * ks);
        const int r = 8 * (chunk & 1) + e;
        const uint32_t b = vc[tile_dword<D>(chunk / 4, r + 16 * (tt >> 2)) * 4];
        v[e] = (_Float16)((float)((int)((b >> sh) & 0xFu) - 8) * vs);
      }
    }
    *reinterpret_cast<uint4*>(k_out + i * 8) = __builtin_bit_cast(uint4, k);
    *reinterpret_cast<uint4*>(v_out + i * 8) = __builtin_bit_cast(uint4, v);
  }
}

// cos and sin of position * theta^(-2 i / rot), all in float64, rounded once to float32.
__global__ __launch_bounds__(256) void rope_table_kernel(int64_t positions, int rot, double theta,
                                                         float* __restrict__ table) {
  const int half = rot / 2;
  const int64_t n = positions * half;
  for (int64_t j = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; j < n; j += (int64_t)gridDim.x * blockDim.x) {
    const int64_t pos = j / half;
    const int i = (int)(j - pos * half);
    const double angle = (double)pos * pow(theta, -2.0 * i / rot);
    double s, c;
    sincos(angle, &s, &c);
    table[2 * j] = (float)c;
    table[2 * j + 1] = (float)s;
  }
}

template <int D, bool APPEND>
void launch_rope_t(const RopeArgs& a, hipStream_t stream) {
  constexpr int RPW = 512 / D;
  const int nq = (a.q_heads + RPW - 1) / RPW, nk = (a.kv_heads + RPW - 1) / RPW;
  const int units = nq + nk * (APPEND ? 2 : 1);
  // one wavefront per token reads its cosines once; few tokens are spread over more
  // wavefronts, down to one unit of heads each
  const int64_t want = std::max<int64_t>(1, (int64_t)device_cu_count_cached() * 16 / a.tokens);
  const int per = (int)((units + std::min<int64_t>(want, units) - 1) / std::min<int64_t>(want, units));
  const int segs = (units + per - 1) / per;
  const int64_t blocks = (a.tokens * segs + 3) / 4;
  hipLaunchKernelGGL((rope_kernel<D, APPEND>), dim3((unsigned)blocks), dim3(256), 0, stream, a, segs, per);
}

int grid_of(int64_t work) { return (int)std::min<int64_t>(std::max<int64_t>((work + 255) / 256, 1), 65536); }

}  // namespace

hipError_t launch_rope(const RopeArgs& a, hipStream_t stream) {
  switch (a.head_dim) {
    case 64: a.append ? launch_rope_t<64, true>(a, stream) : launch_rope_t<64, false>(a, stream); break;
    case 128: a.append ? launch_rope_t<128, true>(a, stream) : launch_rope_t<128, false>(a, stream); break;
    default: a.append ? launch_rope_t<256, true>(a, stream) : launch_rope_t<256, false>(a, stream); break;
  }
  return hipGetLastError();
}

hipError_t launch_paged_dequant(const PagedArgs& c, const int32_t* slots, int64_t tokens, void* k_out, void* v_out,
                                hipStream_t stream) {
  const dim3 grid(grid_of(tokens * c.kv_heads * (c.head_dim / 8)));
  uint16_t* ko = static_cast<uint16_t*>(k_out);
  uint16_t* vo = static_cast<uint16_t*>(v_out);
  switch (c.head_dim) {
    case 64: hipLaunchKernelGGL(paged_dequant_kernel<64>, grid, dim3(256), 0, stream, c, slots, tokens, ko, vo); break;
    case 128: hipLaunchKernelGGL(paged_dequant_kernel<128>, grid, dim3(256), 0, stream, c, slots, tokens, ko, vo); break;
    default: hipLaunchKernelGGL(paged_dequant_kernel<256>, grid, dim3(256), 0, stream, c, slots, tokens, ko, vo); break;
  }
  return hipGetLastError();
}

hipError_t launch_rope_table(int64_t positions, int rot, double theta, float* table, hipStream_t stream) {
  hipLaunchKernelGGL(rope_table_kernel, dim3(grid_of(positions * (rot / 2))), dim3(256), 0, stream, positions, rot,
                     theta, table);
  return hipGetLastError();
}

}  // namespace q4
