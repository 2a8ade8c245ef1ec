// ddl_kv8_evict.cu -- cutting requests of the 8-bit paged cache to their
// heaviest tokens (ddl_kv8_evict): which tokens of each K/V head stay, and their
// move to new pages.
//
// Two kernels.  The first chooses: a cluster of 1 to 8 CTAs takes a request and head, each CTA a run of tokens whose
// scores it keeps in shared memory.  The m-th largest by radix select on order-preserving keys, digits of 10 bits of its
// distance from the largest (so that neither digits nor histogram bins go to what all keys share), the histograms added
// up in distributed shared memory; it ends early where all of a digit stay.  Then the kept tokens in order: each warp
// counts those of its run, and with the sums of the warps before it writes their indices and scores.
// The second moves the codes, a warp per block of 16 kept tokens and head: 16 rows of K and of V in registers, their
// largest value, the block's new power-of-two scale, and the codes in it.  Between powers of two that is a product in
// fp16, exact but for the one rounding of the code; rows whose scale already is the new one keep their codes.
//
// What bounds it: few requests, the chain of barriers and dependent loads (1 of 32769 tokens to 8193, 8 heads: 23 us, with
// cold caches 30); many, the move behind the choice (32 of up to 8192 to 2048, 8 heads: 65 us, choice 19 and move 44 at 50 %
// of the DRAM rate; its bytes would take 33): a warp moves one block after four dependent loads (lengths, indices, pages,
// scale and codes), and with a third of the warps that an SM holds too few bytes are on their way.
#include <cuda_bf16.h>

#include <type_traits>

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

constexpr int SEL_BITS = 10, SEL_BINS = 1 << SEL_BITS, SEL_THREADS = 512, SEL_WARPS = SEL_THREADS / 32;
constexpr int SEL_PASSES = (32 + SEL_BITS - 1) / SEL_BITS;

// SM: the scores fit shared memory.  (If not, loops count without sign: their last step may end past 2^31.)
template <bool SM>
__global__ void __launch_bounds__(SEL_THREADS) kv8_select_kernel(const __grid_constant__ EvictArgs A, const int C) {
  extern __shared__ float sel_scores[];  // SM: the scores of the CTA's tokens
  __shared__ uint32_t hist[SEL_PASSES][SEL_BINS], sums[SEL_PASSES][SEL_BINS / 2];  // sums: of the cluster, SEL_BINS / C of them
  __shared__ uint32_t wsum[2][SEL_WARPS];
  __shared__ uint32_t cta_top, cta_low, cta_sure, cta_ties, sh_digit, sh_need, sh_inside;
  using Id = std::conditional_t<SM, int, uint32_t>;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x % C, h = blockIdx.x / C, r = blockIdx.y;
  for (int i = tid; i < SEL_PASSES * SEL_BINS; i += SEL_THREADS) hist[0][i] = 0;
  pdl_trigger();
  pdl_wait();
  const Cut c = load_cut(A, r);
  if (c.bad && A.bad && blockIdx.x == 0 && tid == 0) atomicOr(A.bad, 1);
  const float* const score = A.score + ((int64_t)r * A.H + h) * A.stride;
  float* const out = A.score_out + ((int64_t)r * A.H + h) * A.stride;
  // the CTA's tokens
  const int n0 = (int)((int64_t)c.len * rank / C), n1 = (int)((int64_t)c.len * (rank + 1) / C);
  if (c.keep < 0) {  // (the same for the whole cluster)
    for (Id i = n0 + tid; i < (Id)n1; i += SEL_THREADS) out[i] = score[i];
    return;
  }
  const int lo = c.sinks, hi = c.len - c.recent;  // the tokens that may go: [lo, hi)
  const int m0 = max(n0, lo), m1 = min(n1, hi);
  auto score_of = [&](int i) -> float { return SM ? sel_scores[i - n0] : score[i]; };
  auto key = [&](int i) -> uint32_t { return score_key(score_of(i)); };
  // the range of the keys
  uint32_t top = 0u, low = ~0u;
  constexpr int U = 8;  // loads on their way
  for (Id i = n0 + tid; i < (Id)n1; i += U * SEL_THREADS) {
    float s[U];
#pragma unroll
    for (int j = 0; j < U; ++j) s[j] = i + j * SEL_THREADS < (Id)n1 ? score[i + j * SEL_THREADS] : 0.f;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const Id x = i + j * SEL_THREADS;
      if (SM && x < (Id)n1) sel_scores[x - n0] = s[j];
      if (x >= (Id)m0 && x < (Id)m1) {
        const uint32_t k = score_key(s[j]);
        top = max(top, k);
        low = min(low, k);
      }
    }
  }
  top = __reduce_max_sync(FULL, top);
  low = __reduce_min_sync(FULL, low);
  if (lane == 0) {
    wsum[0][warp] = top;
    wsum[1][warp] = low;
  }
  __syncthreads();
  if (warp == 0) {
    top = __reduce_max_sync(FULL, lane < SEL_WARPS ? wsum[0][lane] : 0u);
    low = __reduce_min_sync(FULL, lane < SEL_WARPS ? wsum[1][lane] : ~0u);
    if (lane == 0) {
      cta_top = top;
      cta_low = low;
    }
  }
  cluster_sync();
  top = __reduce_max_sync(FULL, lane < C ? ldu_cluster(&cta_top, lane) : 0u);
  low = __reduce_min_sync(FULL, lane < C ? ldu_cluster(&cta_low, lane) : ~0u);
  // the distance `at` from the largest key, but for its last `bits` bits, at which `need` tokens are reached: those
  // nearer stay, and of those at it `need` (all: every one)
  uint32_t need = (uint32_t)(c.keep - c.sinks - c.recent), at = 0;
  int bits = top > low ? 32 - __clz(top - low) : 0;
  bool all = false;
  for (int pass = 0; need > 0 && !all && bits > 0; ++pass) {
    const int shift = bits > SEL_BITS ? bits - SEL_BITS : 0;
    uint32_t* const bins = hist[pass];
    for (Id i = m0 + tid; i < (Id)m1; i += SEL_THREADS) {
      const uint32_t x = top - key(i);
      if (pass == 0 || (x ^ at) >> bits == 0) atomicAdd(&bins[(x >> shift) & (SEL_BINS - 1)], 1u);
    }
    // (in two steps: 16 CTAs that read all 16 histograms took 10 us a digit)
    constexpr int PER = SEL_BINS / SEL_THREADS;
    uint32_t n[PER], sum = 0;
    if (C > 1) {
      const int per = SEL_BINS / C;
      cluster_sync();
      for (int i = tid; i < per; i += SEL_THREADS) {
        uint32_t s = 0;
#pragma unroll 8
        for (int k = 0; k < C; ++k) s += ldu_cluster(&bins[rank * per + i], k);
        sums[pass][i] = s;
      }
      cluster_sync();
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const int i = tid + j * SEL_THREADS, k = i / per;  // (neighbouring lanes, neighbouring words)
        bins[i] = ldu_cluster(&sums[pass][i - k * per], k);
      }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      n[j] = bins[tid * PER + j];
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
    uint32_t before = inc - sum + __reduce_add_sync(FULL, lane < warp ? wsum[0][lane] : 0u);
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      if (before < need && before + n[j] >= need) {
        sh_digit = (uint32_t)(tid * PER + j);
        sh_need = need - before;
        sh_inside = n[j];
      }
      before += n[j];
    }
    __syncthreads();
    at |= sh_digit << shift;
    need = sh_need;
    all = need == sh_inside;
    bits = shift;
  }
  // keys above k_stay stay, those from k_tie up to it are the ties (64 bits: none may be above, or all)
  int64_t k_stay = (int64_t)top - (int64_t)(at >> bits << bits), k_tie = k_stay - ((int64_t)1 << bits) + 1;
  if (all) k_stay = k_tie - 1;
  if (c.keep == c.sinks + c.recent) k_stay = k_tie = 1ll << 32;
  // 2: stays, 1: a tie, 0: goes
  const uint32_t stay_from = (uint32_t)(k_stay + 1 < 0 ? 0 : k_stay + 1 > 0xffffffffll ? 0xffffffffll : k_stay + 1);
  const uint32_t tie_from = (uint32_t)(k_tie < 0 ? 0 : k_tie > 0xffffffffll ? 0xffffffffll : k_tie);
  auto state = [&](int i) -> int {  // (no key is 0xffffffff)
    if (i < lo || i >= hi) return 2;
    const uint32_t k = key(i);
    return k >= stay_from ? 2 : k >= tie_from ? 1 : 0;
  };
  // the kept tokens in order: run of tokens [w0, w1) per warp
  const int w0 = n0 + (int)((int64_t)(n1 - n0) * warp / SEL_WARPS), w1 = n0 + (int)((int64_t)(n1 - n0) * (warp + 1) / SEL_WARPS);
  uint32_t ns = 0, nt = 0;
  if (SM) __syncthreads();  // (the keys, where no digit was needed)
  // 32 tokens a step: which stay and which are ties; lane l keeps step l's for the second time (of 32 steps)
  uint32_t my_stay = 0, my_tie = 0;
  int k = 0;
  for (Id i0 = w0; i0 < (Id)w1; i0 += 32, ++k) {
    const int s = i0 + lane < (Id)w1 ? state(i0 + lane) : 0;
    const uint32_t ms = __ballot_sync(FULL, s == 2), me = __ballot_sync(FULL, s == 1);
    if (k == lane) {
      my_stay = ms;
      my_tie = me;
    }
    ns += __popc(ms);
    nt += __popc(me);
  }
  __syncthreads();  // (wsum's last readers)
  if (lane == 0) {
    wsum[0][warp] = ns;
    wsum[1][warp] = nt;
  }
  __syncthreads();
  uint32_t to = __reduce_add_sync(FULL, lane < warp ? wsum[0][lane] : 0u);
  uint32_t ties = __reduce_add_sync(FULL, lane < warp ? wsum[1][lane] : 0u);
  if (C > 1) {
    if (tid == SEL_THREADS - 32) {  // (the last warp's first lane)
      cta_sure = to + ns;
      cta_ties = ties + nt;
    }
    cluster_sync();
    to += __reduce_add_sync(FULL, lane < rank ? ldu_cluster(&cta_sure, lane) : 0u);
    ties += __reduce_add_sync(FULL, lane < rank ? ldu_cluster(&cta_ties, lane) : 0u);
    cluster_sync();  // (nobody's shared memory goes while another reads it)
  }
  int32_t* const kept = A.kept + ((int64_t)r * A.H + h) * A.max_keep;
  const uint32_t below = (1u << lane) - 1;
  k = 0;
  for (Id i0 = w0; i0 < (Id)w1; i0 += 32, ++k) {
    const Id i = i0 + lane;
    uint32_t ms = __shfl_sync(FULL, my_stay, k & 31), me = __shfl_sync(FULL, my_tie, k & 31);
    if (k >= 32) {
      const int s = i < (Id)w1 ? state(i) : 0;
      ms = __ballot_sync(FULL, s == 2);
      me = __ballot_sync(FULL, s == 1);
    }
    const uint32_t tie = ties + __popc(me & below);
    if ((ms >> lane & 1) || ((me >> lane & 1) && tie < need)) {
      const uint32_t x = to + __popc(ms & below) + (tie < need ? tie : need);
      kept[x] = (int32_t)i;
      out[x] = score_of(i);
    }
    to += __popc(ms);
    ties += __popc(me);
  }
}

// 16 rows of HD codes in a warp's registers: 16 bytes a lane, NI loads; row of load j:
// j * RPL + lane / LPR.
template <int HD>
struct Rows {
  static constexpr int LPR = HD / 16, RPL = 32 / LPR, NI = 16 / RPL;
};

// A row's codes in a warp's registers, and the block that they become.
template <int CT, int HD>
struct Block {
  using G = Rows<HD>;
  uint4 x[G::NI];
  // rows' places (of lane's row; -1: zeros)
  __device__ __forceinline__ void load(const uint8_t* base, int64_t row) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < G::NI; ++j) {
      const int64_t from = __shfl_sync(FULL, row, j * G::RPL + lane / G::LPR);
      x[j] = from >= 0 ? *reinterpret_cast<const uint4*>(base + from * HD + lane % G::LPR * 16) : make_uint4(0u, 0u, 0u, 0u);
    }
  }
  // scale: of lane's row (0 for none); returns the block's new one and leaves its codes in x
  __device__ __forceinline__ float rescale(float scale) {
    const int lane = threadIdx.x & 31;
    // the largest value: per row the largest |code| (exact in fp16; NaN does not count) times its scale; and 2^-16 of it, for
    // products past fp32
    float top = 0.f, far = 0.f;
#pragma unroll
    for (int j = 0; j < G::NI; ++j) {
      const float f = __shfl_sync(FULL, scale, j * G::RPL + lane / G::LPR);
      const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
      __half2 m = __float2half2_rn(0.f);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t a, b;
        codes_f16<CT>(w[q], a, b);
        m = __hmax2(m, __habs2(*reinterpret_cast<const __half2*>(&a)));
        m = __hmax2(m, __habs2(*reinterpret_cast<const __half2*>(&b)));
      }
      const float most = fmaxf(__low2float(m), __high2float(m));
      top = fmaxf(top, most * f);
      far = fmaxf(far, most * (f * 0x1p-16f));
    }
    const float amax = __uint_as_float(__reduce_max_sync(FULL, __float_as_uint(top)));
    const uint32_t bits = __float_as_uint(scale + 0.f);  // (a scale of -0 is zero)
    const bool broken = __any_sync(FULL, !(scale >= 0.f && scale < INFINITY));
    // (the largest power of two is 2^127, of which the largest value may be more than the largest code)
    const float now = broken ? __uint_as_float(0x7fffffffu)
                             : amax < INFINITY ? pow2_scale<CT>(amax)
                                               : fminf(pow2_scale<CT>(__uint_as_float(__reduce_max_sync(FULL, __float_as_uint(far)))) * 0x1p16f, 0x1p127f);
    // all scales powers of two, none more than 2^15 above the new one (nor subnormal): factors in fp16
    const bool pow2 = (bits & 0x7fffffu) == 0 && (bits == 0 || bits >= 0x00800000u) &&
                      (int)(bits >> 23) - (int)(__float_as_uint(now) >> 23) <= 15;
    if (!broken && now > 0.f && __all_sync(FULL, pow2)) {
      // a code times 2^k (k <= 15): exact in fp16, or so small that the code is 0 whichever way it is rounded
      const int k = (int)(bits >> 23) - (int)(__float_as_uint(now) >> 23);
      const uint32_t mine = bits == 0 || k < -24 ? 0u : k < -14 ? 1u << (k + 24) : (uint32_t)(k + 15) << 10;
#pragma unroll
      for (int j = 0; j < G::NI; ++j) {
        const uint32_t f = __shfl_sync(FULL, mine | (mine << 16), j * G::RPL + lane / G::LPR);
        if (f == 0x3c003c00u) continue;  // 1
        const __half2 f2 = *reinterpret_cast<const __half2*>(&f);
        uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t a, b;
          codes_f16<CT>(w[q], a, b);
          if (CT == DDL_KV8_E4M3) {
            const __half2 u = __hmul2(*reinterpret_cast<const __half2*>(&a), f2), v = __hmul2(*reinterpret_cast<const __half2*>(&b), f2);
            w[q] = f16x2_e4m3x2(*reinterpret_cast<const uint32_t*>(&u)) | (f16x2_e4m3x2(*reinterpret_cast<const uint32_t*>(&v)) << 16);
          } else {  // 1536 + c 2^k, rounded to whole numbers by the addition: the code in the low byte
            const __half2 big = __half2(__ushort_as_half(0x6600), __ushort_as_half(0x6600));
            const __half2 u = __hfma2(*reinterpret_cast<const __half2*>(&a), f2, big), v = __hfma2(*reinterpret_cast<const __half2*>(&b), f2, big);
            w[q] = __byte_perm(*reinterpret_cast<const uint32_t*>(&u), *reinterpret_cast<const uint32_t*>(&v), 0x6420);
          }
        }
        x[j] = make_uint4(w[0], w[1], w[2], w[3]);
      }
      return now;
    }
    const bool large = now > 0x1p110f;  // (products past fp32: both sides 2^-16 of themselves)
    const float unit = large ? now * 0x1p-16f : now, mine = large ? scale * 0x1p-16f : scale;
    const Divider by(unit);
#pragma unroll
    for (int j = 0; j < G::NI; ++j) {
      const float f = __shfl_sync(FULL, mine, j * G::RPL + lane / G::LPR);
      if (f == unit) continue;
      uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t a, b;
        codes_f16<CT>(w[q], a, b);
        const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&a));
        const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&b));
        const float v[4] = {by(lo.x * f), by(lo.y * f), by(hi.x * f), by(hi.y * f)};
        w[q] = CT == DDL_KV8_E4M3 ? f32x2_e4m3x2(v[0], v[1]) | (f32x2_e4m3x2(v[2], v[3]) << 16)
                                  : f32_int8(v[0]) | (f32_int8(v[1]) << 8) | (f32_int8(v[2]) << 16) | (f32_int8(v[3]) << 24);
      }
      x[j] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return now;
  }
  __device__ __forceinline__ void store(uint8_t* base, float* scales, int64_t row, float scale) const {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < G::NI; ++j)
      *reinterpret_cast<uint4*>(base + (row + j * G::RPL + lane / G::LPR) * HD + lane % G::LPR * 16) = x[j];
    if (lane == 0) scales[row >> 4] = scale;
  }
};

template <int CT, int HD>
__global__ void __launch_bounds__(256, 3) kv8_move_kernel(const __grid_constant__ EvictArgs A) {
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
  Block<CT, HD> k, v;  // (both on their way before either is looked at)
  k.load(A.code[0], row);
  v.load(A.code[1], row);
  const float ks = k.rescale(scale[0]);
  k.store(A.code[0], A.scale[0], dst, ks);
  const float vs = v.rescale(scale[1]);
  v.store(A.code[1], A.scale[1], dst, vs);
}

constexpr int SEL_SMEM_KEYS = 48 * 1024;  // scores that fit shared memory beside the histograms (192 KB)

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
  int sms = 0;
  if ((st = device_sms(sms))) return st;
  // CTAs a request and head: as many as run at once, with 2048 tokens each at least (a barrier of 16 CTAs costs 1 us: 1
  // request of 32769 tokens, 8 heads, in clusters of 1 / 4 / 8 / 16 47 / 30 / 24 / 27 us)
  int clusters = 1;
  while (clusters < 8 && (int64_t)R * H_kv * clusters <= sms && max_len / (2 * clusters) >= 2048) clusters *= 2;
  const int64_t keys = ((int64_t)max_len + clusters - 1) / clusters;  // of a CTA
  const bool sm = keys <= SEL_SMEM_KEYS;
  const void* fn = sm ? (const void*)kv8_select_kernel<true> : (const void*)kv8_select_kernel<false>;
  const size_t smem = sm ? (size_t)keys * 4 : 0;
  if (smem > 16 * 1024 &&
      (st = cuda_status(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, SEL_SMEM_KEYS * 4))))
    return st;
  void* sargs[] = {&a, &clusters};
  if ((st = cuda_status(launch_pdl_cluster(fn, dim3((unsigned)(H_kv * clusters), (unsigned)R), dim3(SEL_THREADS), sargs, smem,
                                           clusters, (cudaStream_t)stream))))
    return st;
  fn = kv->type == DDL_KV8_E4M3
           ? head_dim == 128 ? (const void*)kv8_move_kernel<DDL_KV8_E4M3, 128> : (const void*)kv8_move_kernel<DDL_KV8_E4M3, 64>
           : head_dim == 128 ? (const void*)kv8_move_kernel<DDL_KV8_INT8, 128> : (const void*)kv8_move_kernel<DDL_KV8_INT8, 64>;
  const unsigned ctas = (unsigned)(((int64_t)max_keep + 127) / 128);
  void* args[] = {&a};
  return cuda_status(launch_pdl(fn, dim3(ctas, (unsigned)H_kv, (unsigned)R), dim3(256), args, 0, (cudaStream_t)stream));
}
