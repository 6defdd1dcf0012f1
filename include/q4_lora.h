/*
 * q4_lora.h -- C ABI of libq4, the W4A16 product with low-rank adapters of many requests
 * at once, for AMD Instinct MI355X (gfx950). Same library, status codes and conventions
 * as q4.h (device pointers owned by the caller, enqueue-only on `stream`, host-side
 * validation before any HIP call, q4_last_error() for details).
 *
 * One frozen INT4 matrix serves every request (q4.h); each request may bring an adapter of
 * rank r, two thin float16 matrices A [rank][in] and B [out][rank], kept in 16 bits
 * ("Post-training quantization: GPTQ, AWQ and rotation", arganzheng.life, section 二.3:
 * weight-only quantization keeps 16-bit activations):
 *   y[b] = x[b] W_hat^T + scaling[a] * B_a (A_a x[b]),  a = ids[b].
 */
#ifndef Q4_LORA_H
#define Q4_LORA_H

#include "q4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of device workspace q4_gemm_lora needs for this shape (0 on invalid arguments). */
size_t q4_workspace_bytes_lora(int64_t B, int64_t out, int64_t in, int32_t group, int32_t rank);

/* q4_gemm (zeros NULL: symmetric codes) or q4_gemm_asym plus each row's adapter:
 *   lora_a: float16 [adapters][rank][in], 16-byte aligned;
 *   lora_b: float16 [adapters][out][rank], 16-byte aligned;
 *   scaling: float32 [adapters] (alpha / rank, say); ids: int32 [B], the adapter of each
 *   row; one outside [0, adapters), -1 say, is a row without an adapter, whose result
 *   is q4_gemm's. Rows may come in any order.
 * The weights are q4_gemm's and q4_gemm_asym's; act-order and INT8 weights have no form
 * with adapters.
 * rank is a multiple of 8 in [8, 128]. A_a x[b] is summed and kept in float32, the
 * adapter's part added to the product's float32 sum and the whole rounded once to
 * float16. Deterministic: sums are taken in a fixed order. adapters = 0 is the plain
 * product. `workspace` (16-byte aligned) must hold q4_workspace_bytes_lora() bytes, taken
 * on the device that the call runs on; contents as q4_gemm's. y must not overlap x. B is bounded
 * by the launch:
 * ceil(B / 16) * max(16 * ceil(in / 1024), ceil(out / 256)) < 2^24 (Q4_ERR_SHAPE). */
q4_status q4_gemm_lora(const void* x, int64_t B, const void* packed, const void* scales, const void* zeros,
                       int64_t out, int64_t in, int32_t group, const void* lora_a, const void* lora_b,
                       const float* scaling, int64_t adapters, int32_t rank, const int32_t* ids, void* y,
                       void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* Q4_LORA_H */
