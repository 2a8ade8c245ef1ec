// ddl_kv8_evict.cu -- cutting requests of the 8-bit paged cache to their
// heaviest tokens (ddl_kv8_evict): which tokens of each K/V head stay, and their
// move to new pages.
//
// Two kernels.  The first chooses, one CTA per request and head: the m-th largest
// score among the tokens that may go, by radix select on order-preserving keys
// (digits of 11, 11 and 10 bits, histograms in shared memory), then the kept
// tokens in order: each warp counts those of its run of tokens, and with the sums
// of the warps before it writes their indices and scores.  The second moves the
// codes, a warp per block of 16 kept tokens and head: 16 rows of K and of V in
// registers, their largest value, the block's new power-of-two scale, and the
// codes in it.  Rows whose scale already is the new one keep their codes.
#include <cuda_bf16.h>

#include "ddl_kv8.h"

namespace ddl {
namespace {

struct EvictArgs {
  uint8_t* code[2];   // k, v
  float* scale[2];
  const float* score;  // [R][H][stride]
  float* score_out;
  const int32_t *kv_len, *keep_len, *table, *new_table;
  int32_t* kept;      // [R][H][max_keep]
  int32_t* bad;
  int64_t stride, pages;
  int32_t R, H, hd, pshift, per, new_per, max_len, max_keep, sinks, recent;
};

// What becomes of a request: `len` tokens, of which `keep` stay (-1: all, in place).
struct Cut {
  int32_t len, keep, sinks, recent;
  bool bad;
};
__device__ __forceinline__ Cut load_cut(const EvictArgs& A, int r) {
  Cut c;
  int32_t len = A.kv_len[r], keep = A.keep_len[r];
  const int64_t cap = (int64_t)A.per << A.pshift, most = A.max_len < cap ? A.max_len : cap;
  c.bad = len < 0 || len > most;
  len = len < 0 ? 0 : len > most ? (int32_t)most : len;
  c.len = len;
  c.keep = -1;
  c.sinks = c.recent = 0;
  if (keep < 0 || keep >= len) return c;
  const int64_t room = (int64_t)A.new_per << A.pshift, top = A.max_keep < room ? A.max_keep : room;
  if (keep > top) {
    c.bad = true;
    keep = (int32_t)top;
  }
  c.keep = keep;
  c.recent = A.recent < keep ? A.recent : keep;
  c.sinks = A.sinks < keep - c.recent ? A.sinks : keep - c.recent;
  return c;
}

// Order-preserving key of a score: NaN lowest, both zeros equal.
__device__ __forceinline__ uint32_t score_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return x == x ? (b & 0x80000000u ? ~b : b | 0x80000000u) : 0u;
}

constexpr int SEL_BINS = 2048;

template <int NT, bool SM>
__global__ void __launch_bounds__(NT) kv8_select_kernel(const __grid_constant__ EvictArgs A) {
  extern __shared__ uint32_t sel_keys[];  // SM: the tokens' keys
  __shared__ uint32_t hist[SEL_BINS];
  __shared__ uint32_t wsum[2][NT / 32];
  __shared__ uint32_t sh_digit, sh_need;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.x, r = blockIdx.y;
  pdl_trigger();
  pdl_wait();
  const Cut c = load_cut(A, r);
  if (c.bad && A.bad && h == 0 && tid == 0) atomicOr(A.bad, 1);
  const float* const score = A.score + ((int64_t)r * A.H + h) * A.stride;
  float* const out = A.score_out + ((int64_t)r * A.H + h) * A.stride;
  if (c.keep < 0) {
    for (int i = tid; i < c.len; i += NT) out[i] = score[i];
    return;
  }
  const int lo = c.sinks, hi = c.len - c.recent;  // the tokens that may go: [lo, hi)
  auto key = [&](int i) -> uint32_t { return SM ? sel_keys[i] : score_key(score[i]); };
  if (SM) {
    for (int i = tid; i < c.len; i += NT) sel_keys[i] = score_key(score[i]);
  }
  // the m-th largest key, and how many tokens of that key stay
  uint32_t need = (uint32_t)(c.keep - c.sinks - c.recent), thr = 0xffffffffu;
  if (need > 0) {
    uint32_t prefix = 0, mask = 0;
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
      for (int i = tid; i < SEL_BINS; i += NT) hist[i] = 0;
      __syncthreads();
      for (int i = lo + tid; i < hi; i += NT) {
        const uint32_t k = key(i);
        if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1)], 1u);
      }
      __syncthreads();
      // bins from the top: thread i takes bins SEL_BINS - 1 - i * PER ...
      constexpr int PER = SEL_BINS / NT;
      uint32_t n[PER], sum = 0;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        n[j] = hist[SEL_BINS - 1 - (tid * PER + j)];
        sum += n[j];
      }
      uint32_t inc = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(FULL, inc, o);
        if (lane >= o) inc += y;
      }
      if (lane == 31) wsum[0][warp] = inc;
      __syncthreads();
      for (int w = 0; w < warp; ++w) inc += wsum[0][w];
      uint32_t before = inc - sum;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        if (before < need && before + n[j] >= need) {
          sh_digit = (uint32_t)(SEL_BINS - 1 - (tid * PER + j));
          sh_need = need - before;
        }
        before += n[j];
      }
      __syncthreads();
      prefix |= sh_digit << shift;
      mask |= ((1u << bits) - 1) << shift;
      need = sh_need;
    }
    thr = prefix;
  }
  __syncthreads();  // (the keys, where nothing was chosen)
  // the kept tokens in order: run of tokens [w0, w1) per warp
  const int w0 = (int)((int64_t)c.len * warp / (NT / 32)), w1 = (int)((int64_t)c.len * (warp + 1) / (NT / 32));
  auto sure = [&](int i, uint32_t k) { return i < lo || i >= hi || k > thr; };
  uint32_t ns = 0, nt = 0;
  for (int i = w0 + lane; i < w1; i += 32) {
    const uint32_t k = key(i);
    const bool s = sure(i, k);
    ns += s;
    nt += !s && k == thr;
  }
  ns = __reduce_add_sync(FULL, ns);
  nt = __reduce_add_sync(FULL, nt);
  if (lane == 0) {
    wsum[0][warp] = ns;
    wsum[1][warp] = nt;
  }
  __syncthreads();
  uint32_t at = 0, ties = 0;  // kept for sure, and tokens of the threshold's key, before this warp's
  for (int w = 0; w < warp; ++w) {
    at += wsum[0][w];
    ties += wsum[1][w];
  }
  int32_t* const kept = A.kept + ((int64_t)r * A.H + h) * A.max_keep;
  const uint32_t below = (1u << lane) - 1;
  for (int i0 = w0; i0 < w1; i0 += 32) {
    const int i = i0 + lane;
    const bool in = i < w1;
    const uint32_t k = in ? key(i) : 0u;
    const bool s = in && sure(i, k), e = in && !s && k == thr;
    const uint32_t ms = __ballot_sync(FULL, s), me = __ballot_sync(FULL, e);
    const uint32_t tie = ties + __popc(me & below);
    const bool take = s || (e && tie < need);
    if (take) {
      const uint32_t to = at + __popc(ms & below) + (tie < need ? tie : need);
      kept[to] = i;
      out[to] = score[i];
    }
    at += __popc(ms);
    ties += __popc(me);
  }
}

// 16 rows of HD codes in a warp's registers: 16 bytes a lane, NI loads; row of load j:
// j * RPL + lane / LPR.
template <int HD>
struct Rows {
  static constexpr int LPR = HD / 16, RPL = 32 / LPR, NI = 16 / RPL;
};

template <int CT, int HD>
__device__ __forceinline__ void move_block(const EvictArgs& A, int kv, int64_t src_row, float src_scale, int64_t dst_row) {
  using G = Rows<HD>;
  const int lane = threadIdx.x & 31, sub = lane % G::LPR;
  const uint8_t* const base = A.code[kv];
  uint4 x[G::NI];
  float f[G::NI];
#pragma unroll
  for (int j = 0; j < G::NI; ++j) {
    const int64_t row = __shfl_sync(FULL, src_row, j * G::RPL + lane / G::LPR);
    f[j] = __shfl_sync(FULL, src_scale, j * G::RPL + lane / G::LPR);
    x[j] = row >= 0 ? *reinterpret_cast<const uint4*>(base + row * HD + sub * 16) : make_uint4(0u, 0u, 0u, 0u);
  }
  // the largest value: per row the largest |code| (exact in fp16; NaN does not count) times its scale
  float top = 0.f;
#pragma unroll
  for (int j = 0; j < G::NI; ++j) {
    const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
    __half2 m = __float2half2_rn(0.f);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t a, b;
      codes_f16<CT>(w[q], a, b);
      m = __hmax2(m, __habs2(*reinterpret_cast<const __half2*>(&a)));
      m = __hmax2(m, __habs2(*reinterpret_cast<const __half2*>(&b)));
    }
    top = fmaxf(top, fmaxf(__low2float(m), __high2float(m)) * f[j]);
  }
  const float amax = __uint_as_float(__reduce_max_sync(FULL, __float_as_uint(top)));
  const bool broken = __any_sync(FULL, !(src_scale >= 0.f && src_scale < INFINITY));
  const float now = broken ? __uint_as_float(0x7fffffffu) : pow2_scale<CT>(amax);
  const Divider by(now);
#pragma unroll
  for (int j = 0; j < G::NI; ++j) {
    const int64_t row = __shfl_sync(FULL, src_row, j * G::RPL + lane / G::LPR);
    uint4 y = x[j];
    if (row >= 0 && f[j] != now) {
      uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t a, b;
        codes_f16<CT>(w[q], a, b);
        const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&a));
        const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&b));
        const float v[4] = {by(lo.x * f[j]), by(lo.y * f[j]), by(hi.x * f[j]), by(hi.y * f[j])};
        w[q] = CT == DDL_KV8_E4M3 ? f32x2_e4m3x2(v[0], v[1]) | (f32x2_e4m3x2(v[2], v[3]) << 16)
                                  : f32_int8(v[0]) | (f32_int8(v[1]) << 8) | (f32_int8(v[2]) << 16) | (f32_int8(v[3]) << 24);
      }
      y = make_uint4(w[0], w[1], w[2], w[3]);
    }
    *reinterpret_cast<uint4*>(A.code[kv] + (dst_row + j * G::RPL + lane / G::LPR) * HD + sub * 16) = y;
  }
  if (lane == 0) A.scale[kv][dst_row >> 4] = now;
}

template <int CT, int HD>
__global__ void __launch_bounds__(256) kv8_move_kernel(const __grid_constant__ EvictArgs A) {
  const int lane = threadIdx.x & 31, b = blockIdx.x * 8 + (threadIdx.x >> 5), h = blockIdx.y, r = blockIdx.z;
  pdl_trigger();
  pdl_wait();
  const Cut c = load_cut(A, r);
  if (c.keep < 0 || b * 16 >= c.keep) return;
  const int64_t mask = (1ll << A.pshift) - 1;
  const int32_t page = A.new_table[(int64_t)r * A.new_per + ((b * 16) >> A.pshift)];
  const bool to = page >= 0 && page < A.pages;
  int64_t row = -1;
  float scale[2] = {0.f, 0.f};
  bool lost = !to;
  if (lane < 16 && b * 16 + lane < c.keep) {
    const int32_t i = A.kept[((int64_t)r * A.H + h) * A.max_keep + b * 16 + lane];
    const int32_t from = A.table[(int64_t)r * A.per + (i >> A.pshift)];
    if (from >= 0 && from < A.pages) {
      row = (((int64_t)from * A.H + h) << A.pshift) + (i & mask);
      scale[0] = A.scale[0][row >> 4];
      scale[1] = A.scale[1][row >> 4];
    } else {
      lost = true;
    }
  }
  if (lost && A.bad) atomicOr(A.bad, 1);
  if (!to) return;
  const int64_t dst = (((int64_t)page * A.H + h) << A.pshift) + ((b * 16) & mask);
  move_block<CT, HD>(A, 0, row, scale[0], dst);
  move_block<CT, HD>(A, 1, row, scale[1], dst);
}

constexpr int SEL_SMEM_KEYS = 50 * 1024;  // keys that fit shared memory (200 KB)

}  // namespace
}  // namespace ddl

using namespace ddl;

extern "C" int ddl_kv8_evict(const ddl_kv8* kv, int32_t H_kv, int32_t head_dim, int32_t R, int32_t max_len,
                             const float* score, int64_t score_stride, const int32_t* kv_len, const int32_t* keep_len,
                             int32_t sinks, int32_t recent, const int32_t* page_table, int32_t pages_per_seq,
                             const int32_t* new_table, int32_t new_pages_per_seq, int32_t max_keep, int32_t* kept,
                             float* score_out, int32_t* bad_out, void* stream) {
  int st = check_kv8(kv, H_kv, head_dim);
  if (st) return st;
  if (R < 1 || max_len < 1 || max_keep < 1 || pages_per_seq < 1 || new_pages_per_seq < 1 || sinks < 0 || recent < 0)
    return DDL_ERR_ARG;
  if (R > DDL_KV8_MAX_REQS) return DDL_ERR_UNSUPPORTED;
  if (!score || !kv_len || !keep_len || !page_table || !new_table || !kept || !score_out) return DDL_ERR_ARG;
  if (score_out == score || page_table == new_table || score_stride < max_len || max_keep > max_len) return DDL_ERR_ARG;
  if ((int64_t)pages_per_seq * kv->page_size > 0x7fffffffLL || (int64_t)new_pages_per_seq * kv->page_size > 0x7fffffffLL)
    return DDL_ERR_UNSUPPORTED;
  for (const void* p : {(const void*)score, (const void*)kv_len, (const void*)keep_len, (const void*)page_table,
                        (const void*)new_table, (const void*)kept, (const void*)score_out, (const void*)bad_out})
    if ((uintptr_t)p & 3u) return DDL_ERR_ALIGN;
  EvictArgs a;
  a.code[0] = kv->k;
  a.code[1] = kv->v;
  a.scale[0] = kv->k_scale;
  a.scale[1] = kv->v_scale;
  a.score = score;
  a.score_out = score_out;
  a.kv_len = kv_len;
  a.keep_len = keep_len;
  a.table = page_table;
  a.new_table = new_table;
  a.kept = kept;
  a.bad = bad_out;
  a.stride = score_stride;
  a.pages = kv->pages;
  a.R = R;
  a.H = H_kv;
  a.hd = head_dim;
  a.pshift = log2_of(kv->page_size);
  a.per = pages_per_seq;
  a.new_per = new_pages_per_seq;
  a.max_len = max_len;
  a.max_keep = max_keep;
  a.sinks = sinks;
  a.recent = recent;
  void* args[] = {&a};
  const bool sm = max_len <= SEL_SMEM_KEYS;
  const void* fn = sm ? (const void*)kv8_select_kernel<512, true> : (const void*)kv8_select_kernel<512, false>;
  const size_t smem = sm ? (size_t)max_len * 4 : 0;
  if (smem > 32 * 1024 &&
      (st = cuda_status(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, SEL_SMEM_KEYS * 4))))
    return st;
  if ((st = cuda_status(launch_pdl(fn, dim3((unsigned)H_kv, (unsigned)R), dim3(512), args, smem, (cudaStream_t)stream))))
    return st;
  fn = kv->type == DDL_KV8_E4M3
           ? head_dim == 128 ? (const void*)kv8_move_kernel<DDL_KV8_E4M3, 128> : (const void*)kv8_move_kernel<DDL_KV8_E4M3, 64>
           : head_dim == 128 ? (const void*)kv8_move_kernel<DDL_KV8_INT8, 128> : (const void*)kv8_move_kernel<DDL_KV8_INT8, 64>;
  const unsigned ctas = (unsigned)(((int64_t)max_keep + 127) / 128);
  return cuda_status(launch_pdl(fn, dim3(ctas, (unsigned)H_kv, (unsigned)R), dim3(256), args, 0, (cudaStream_t)stream));
}
