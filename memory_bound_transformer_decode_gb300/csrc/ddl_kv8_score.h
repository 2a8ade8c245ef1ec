// ddl_kv8_score.h -- what the two kernels of the cache scores (warp MMAs for a few tiles of
// queries, tcgen05 for many) share.
#pragma once
#include "ddl_kv8_attn.h"

namespace ddl {

struct ScoreArgs {
  AttArgs a;
  float* score;    // [R][H_kv][stride]
  int64_t stride;
  float decay;
  int32_t wb;      // warp kernel: blocks of 16 tokens a warp takes; tcgen05: tiles of 128 tokens a CTA takes
  int32_t tiles;   // warp kernel: query tiles in shared memory; tcgen05: queries there at a time (a multiple of 16)
  uint64_t wait_ns;
};

// What the queries of a tile need apart from their fragments.
struct Column {
  float cf;       // factor of the MMA's sum (times the block's scale): log2 units, or softcap's argument
  float lse2;     // log2 e times lse; +inf for a query without keys
  float slope;    // log2 units a token
  int hi, lo;     // last and first token it sees; hi < 0: it adds nothing (masks are looked at then, whatever its scores)
};

// Query qi of request rq for K/V head h.
template <bool EX>
__device__ __forceinline__ Column column_of(const AttArgs& A, const Req& rq, int h, int qi, float qf) {
  Column c;
  const bool has = qi < rq.n * A.GH;
  const int row = has ? group_row(A, qi) : 0;
  const int64_t p = (int64_t)rq.p0 + row, lo = A.window > 0 ? p - A.window + 1 : 0;
  const float lse = has ? A.lse[(int64_t)(rq.row0 + row) * A.Hq + h * A.GH + qi - row * A.GH] : -INFINITY;
  c.hi = has && lse != -INFINITY ? (int)p : -1;
  c.lo = lo > 0 ? (int)lo : 0;
  c.slope = EX && A.slopes && has ? A.slopes[h * A.GH + qi - row * A.GH] * LOG2E : 0.f;
  c.cf = qf * A.scale;
  if (EX && A.softcap > 0.f) c.cf = __fdiv_rn(c.cf, A.softcap);
  else c.cf *= LOG2E;
  c.lse2 = lse == -INFINITY ? INFINITY : lse * LOG2E;
  return c;
}

// tanh of N numbers: below 0.3 its series up to x^9 (the next term is 2^-24 of it), which is
// relative to x at any cap; else, where a lane of the warp has a larger one, tanhf.
template <int N>
__device__ __forceinline__ void tanh_of(float (&x)[N]) {
  bool large = false;  // (or NaN)
#pragma unroll
  for (int j = 0; j < N; ++j) large |= !(fabsf(x[j]) < 0.3f);
  if (__any_sync(FULL, large)) {
#pragma unroll
    for (int j = 0; j < N; ++j) x[j] = tanhf(x[j]);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float y = x[j] * x[j];
      x[j] = fmaf(x[j] * y, fmaf(y, fmaf(y, fmaf(y, 62.f / 2835.f, -17.f / 315.f), 2.f / 15.f), -1.f / 3.f), x[j]);
    }
  }
}

// Launch of the tcgen05 kernel (s.wb, s.tiles are its own to choose).
int kv8_score_tc_launch(const ScoreArgs& s, int type, int dtype, bool ex, int sms, void* stream);
constexpr int SCORE_TC_TILES = 16;  // tiles of 128 tokens a CTA takes at most

}  // namespace ddl
