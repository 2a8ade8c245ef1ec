// ddl_kv8.h -- what the 8-bit paged KV cache's translation units share: the
// checks of a pool descriptor and the code types' conversions.
#pragma once
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include "ddl_device.cuh"
#include "ddl_internal.h"

namespace ddl {

constexpr int KV8_BLOCK = DDL_KV8_BLOCK;  // tokens that share a scale
static_assert(KV8_BLOCK == 16, "the kernels take a block of 16 tokens as one MMA's key dimension");

// Pool rules of ddl.h (host).
inline int check_kv8(const ddl_kv8* kv, int32_t H_kv, int32_t hd) {
  if (!kv || !kv->k || !kv->v || !kv->k_scale || !kv->v_scale) return DDL_ERR_ARG;
  if (hd != 64 && hd != 128) return DDL_ERR_SHAPE;
  if (H_kv < 1 || H_kv > DDL_KV8_MAX_HEADS) return DDL_ERR_SHAPE;
  if (kv->pages < 1) return DDL_ERR_ARG;
  if (kv->type != DDL_KV8_E4M3 && kv->type != DDL_KV8_INT8) return DDL_ERR_UNSUPPORTED;
  if (kv->page_size < 16 || kv->page_size > (1 << 20) || (kv->page_size & (kv->page_size - 1))) return DDL_ERR_ARG;
  if (kv->pages > 0x7fffffffLL / kv->page_size) return DDL_ERR_UNSUPPORTED;  // slots are int32
  if (kv->pages > 0x7fffffffLL / (H_kv * (int64_t)(kv->page_size / KV8_BLOCK))) return DDL_ERR_UNSUPPORTED;  // and blocks
  if (!aligned16(kv->k) || !aligned16(kv->v) || !aligned16(kv->k_scale) || !aligned16(kv->v_scale))
    return DDL_ERR_ALIGN;
  return DDL_OK;
}

inline int check_attn_opts(const ddl_attn_opts* o) {
  if (!o) return DDL_ERR_ARG;
  if (!(fabsf(o->scale) < INFINITY) || !(o->softcap >= 0.f && o->softcap < INFINITY) || o->window < 0)
    return DDL_ERR_ARG;
  return ((uintptr_t)o->slopes & 3u) ? DDL_ERR_ALIGN : DDL_OK;
}

inline int log2_of(int32_t pow2) {
  int s = 0;
  while ((1 << s) < pow2) ++s;
  return s;
}

inline int dtype_bytes(int32_t t) { return t == DDL_T_F32 ? 4 : (t == DDL_T_BF16 || t == DDL_T_F16) ? 2 : 0; }

// Two e4m3 codes (bytes 0 and 1 of w, or 2 and 3) as fp16: exact.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint16_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(w));
  return r;
}
// Four e4m3 codes as two fp16 pairs.
__device__ __forceinline__ void e4m3x4_f16x2(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
// 2^x with results below 2^-126 flushed to zero.
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two fp32 values as e4m3 codes, round to nearest even, saturating at 448
// (NaN stays NaN); `lo` in the low byte.
__device__ __forceinline__ uint32_t f32x2_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// fp32 as an 8-bit integer code in [-127, 127], round to nearest even; NaN 0.
__device__ __forceinline__ uint32_t f32_int8(float v) {
  const float c = fminf(fmaxf(v, -127.f), 127.f);  // (NaN becomes -127 here)
  return v == v ? (uint32_t)(uint8_t)(int8_t)__float2int_rn(c) : 0u;
}

}  // namespace ddl
