// RMS norm and rotation of the q and k heads, and the append of k and v into the
// paged INT4 cache (include/q4_attn.h), in one pass over the projection's rows.
//
// One wavefront owns a token; a lane holds 8 channels of a head (one 16-byte load),
// so D / 8 lanes make a head and a wavefront takes RPW = 512 / D heads at a time. The
// token's cosines and sines depend on the lane's channels only: they are loaded once
// and stay in registers for all of the token's heads. The mean square is a butterfly
// over the head's lanes; a rotation partner that sits rot_dim / 2 channels away is
// another lane's chunk (four dword shuffles), one that is adjacent is the lane's own.
// Every head is read once and written once: the pass is bound by those bytes.
//
// Rounding: x * w is exact in float32 (11 + 11 significant bits). q continues in
// float32; k, whose value next decides a 4-bit code, in float64, so that a code
// differs from the exact one only where the value lies within ~1e-15 of a border.
#include <algorithm>

#include "q4_paged.h"
#include "q4_rtn.h"

namespace q4 {
namespace {

struct Row8 {
  half8_t x;
  bool real;
};

// Float16 of a float64, rounded once.
__device__ __forceinline__ _Float16 to_half(double v) { return (_Float16)v; }
__device__ __forceinline__ _Float16 to_half(float v) { return (_Float16)v; }

__device__ __forceinline__ float inv_sqrt(float v) { return 1.0f / sqrtf(v); }
__device__ __forceinline__ double inv_sqrt(double v) { return 1.0 / sqrt(v); }

// Rotation factors of a lane's 8 channels: out[e] = h[e] * c[e] + partner[e] * s[e],
// s carrying the sign. `turn` is false for channels behind rot_dim.
struct Turn {
  float c[8], s[8];
  int partner;  // lane of the partner's chunk (half-split pairs)
  bool turn;
};

template <int D>
__device__ __forceinline__ Turn load_turn(const RopeArgs& a, int64_t token, int lane) {
  constexpr int LPH = D / 8;
  Turn t;
  const int ch = 8 * (lane & (LPH - 1));
  t.turn = ch < a.rot;
  t.partner = lane;
  if (!t.turn) return t;
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
    return t;
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
  return t;
}

// Norm and rotation of one head row chunk, arithmetic in T.
template <int D, typename T>
__device__ __forceinline__ half8_t norm_rope(half8_t x, const uint16_t* weight, float eps, const Turn& t,
                                             bool interleaved, bool rotate, int lane) {
  constexpr int LPH = D / 8;
  float h[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) h[e] = (float)x[e];
  T r = (T)1;
  if (weight) {
    T sum = (T)0;
#pragma unroll
    for (int e = 0; e < 8; ++e) sum += (T)(h[e] * h[e]);
#pragma unroll
    for (int m = 1; m < LPH; m <<= 1) sum += __shfl_xor(sum, m, 64);
    r = inv_sqrt(sum / (T)D + (T)eps);
    const half8_t w = as_half8(*reinterpret_cast<const uint4*>(weight + 8 * (lane & (LPH - 1))));
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] *= (float)w[e];
  }
  float other[8];
  if (rotate) {
    if (interleaved) {
#pragma unroll
      for (int e = 0; e < 8; ++e) other[e] = h[e ^ 1];
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) other[e] = __shfl(h[e], t.partner, 64);
    }
  }
  half8_t out;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    T v = (T)h[e];
    if (rotate && t.turn) v = v * (T)t.c[e] + (T)other[e] * (T)t.s[e];
    out[e] = weight ? to_half(v * r) : to_half(v);
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

// Heads of a token in units of RPW heads: q's, then k's, then (append) v's.
template <int D, bool APPEND>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs a, int segs, int units_per_seg) {
  constexpr int LPH = D / 8;
  constexpr int RPW = kWave / LPH;
  const int lane = threadIdx.x & 63;
  const int64_t wave = (int64_t)blockIdx.x * (blockDim.x / kWave) + threadIdx.x / kWave;
  const int64_t token = wave / segs;
  if (token >= a.tokens) return;
  const int nq = (a.q_heads + RPW - 1) / RPW, nk = (a.kv_heads + RPW - 1) / RPW;
  const int units = nq + nk + (APPEND ? nk : 0);
  const int u0 = (int)(wave - token * segs) * units_per_seg;
  const int u1 = min(u0 + units_per_seg, units);
  const int sub = lane / LPH, chunk = lane & (LPH - 1);
  const bool rotate = a.rot > 0;
  Turn t;
  t.turn = false;
  if (rotate) t = load_turn<D>(a, token, lane);
  uint32_t slot = 0xFFFFFFFFu;
  if (APPEND) slot = (uint32_t)a.slots[token];
  const bool stored = APPEND && (int64_t)slot < a.cache.pages * a.cache.page_size;
  for (int u = u0; u < u1; ++u) {
    // kind 0: q, 1: k, 2: v (uniform)
    const int kind = u < nq ? 0 : u < nq + nk ? 1 : 2;
    const int head = (kind == 0 ? u : kind == 1 ? u - nq : u - nq - nk) * RPW + sub;
    const bool real = head < (kind == 0 ? a.q_heads : a.kv_heads);
    const uint16_t* src = kind == 0 ? static_cast<const uint16_t*>(a.q) + token * a.q_stride
                          : kind == 1 ? static_cast<const uint16_t*>(a.k) + token * a.k_stride
                                      : static_cast<const uint16_t*>(a.v) + token * a.v_stride;
    uint4 raw = make_uint4(0u, 0u, 0u, 0u);
    if (real) raw = *reinterpret_cast<const uint4*>(src + head * D + 8 * chunk);
    half8_t x = as_half8(raw);
    if (kind == 0) {
      x = norm_rope<D, float>(x, static_cast<const uint16_t*>(a.q_weight), a.eps, t, a.interleaved, rotate, lane);
      if (real)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.q_out) + token * a.q_out_stride + head * D + 8 * chunk) =
            __builtin_bit_cast(uint4, x);
      continue;
    }
    if (kind == 1) {
      x = norm_rope<D, double>(x, static_cast<const uint16_t*>(a.k_weight), a.eps, t, a.interleaved, rotate, lane);
      if (!APPEND) {
        if (real)
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.k_out) + token * a.k_out_stride + head * D + 8 * chunk) =
              __builtin_bit_cast(uint4, x);
        continue;
      }
    }
    if (!APPEND) continue;
    _Float16 scale;
    const int GL = a.cache.group / 8;
    const uint32_t word = quantize8(x, GL, &scale);
    const uint32_t partner = __shfl_xor(word, 2, 64);  // channels + 16 (V bytes)
    if (!stored || !real) continue;
    const int64_t tile = slot_tile(slot, a.cache.page_size, a.cache.kv_heads, head);
    const int tt = (int)(slot % (uint32_t)kTokTile);  // page_size is a multiple of the tile
    if (chunk % GL == 0) {
      uint16_t* sc = static_cast<uint16_t*>(kind == 1 ? a.cache.k_scales : a.cache.v_scales);
      sc[(tile * (LPH / GL) + chunk / GL) * kTokTile + tt] = __builtin_bit_cast(uint16_t, scale);
    }
    const uint32_t off = word ^ 0x88888888u;  // q + 8
    if (kind == 1) {
      uint32_t dw = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) dw |= ((off >> (4 * e)) & 0xFu) << (4 * nibble_of(e));
      static_cast<uint32_t*>(a.cache.k_codes)[tile * (2 * D) + tile_dword<D>(chunk / 4, tt + 16 * (chunk & 3))] = dw;
    } else {
      // a byte holds channels 32m + r and 32m + 16 + r: the lanes of the two halves
      // write four of their eight bytes each
      const uint32_t po = partner ^ 0x88888888u;
      const int hi = (chunk >> 1) & 1;
      const uint32_t lo_word = hi ? po : off, hi_word = hi ? off : po;
      uint8_t* vc = static_cast<uint8_t*>(a.cache.v_codes) + tile * (8 * D);
      const int byte = v_byte(tt & 3);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = 4 * hi + i;
        const int r = 8 * (chunk & 1) + e;
        vc[tile_dword<D>(chunk / 4, r + 16 * (tt >> 2)) * 4 + byte] =
            (uint8_t)(((lo_word >> (4 * e)) & 0xFu) | (((hi_word >> (4 * e)) & 0xFu) << 4));
      }
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
