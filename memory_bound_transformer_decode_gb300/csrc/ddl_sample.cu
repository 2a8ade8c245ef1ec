// ddl_sample.cu -- the next token of each row of logits, with the row's own
// temperature, top-k, top-p and min-p (ddl_sample).
//
//     w_v = exp((l_v - l_max) / T);  the kept tokens are the first ones in the order
//     (logit descending, id ascending) that pass all filters;  the token drawn is the
//     first kept id, in ascending order, whose running sum of weights exceeds u times
//     the kept tokens' sum.
//
// Every filter keeps a head of one order, so what the filters decide is one element,
// the last that stays; no sort is needed, and the draw in id order needs sums only.
//
// Weights are integers in units of 2^-43, and so are their sums: neither the order of
// additions nor the split over CTAs changes a bit.  An fp32 exponential would be
// wrong by 2^-23 of a weight, and a draw over V tokens meets a border within d of
// its number about V d of the time; so w comes from a table of 2^(i/64) and a cubic for
// the remaining factor of less than 2^(1/128), argument, table and product in two
// floats each: 2^-33 of w before it is rounded to the unit.  Adding 6 and 1.5 2^-20
// rounds the two parts to multiples of 2^-21 and 2^-43, which then lie in the low bits:
// integers without a conversion.  (Double precision: 152 SMs do 2 operations a clock
// each; 64 rows of 152064 would take 160 us.)
//
// A cluster of 1 to 16 CTAs takes a row; a warp a contiguous run of ids.
//  1. The maximum (greedy rows end here), and each lane's own.
//  1b. top-k of fewer elements than half the lanes: the k-th largest of the lanes' maxima
//     is a bound of the k-th logit, and nearly it where ids and logits are unrelated.  A
//     histogram of the maxima gives it, the elements above it go to the list, and 4 does
//     the rest.  (If they are too many: 2.)
//  2. Rows with top-k or top-p: a histogram of log2 w in 2048 bins of 1/47.6 octave:
//     how many elements, and the sum of their places inside the bin, which bounds the
//     bin's sum of weights to 2^-13.  Where the k-th element and the end of the top-p
//     head may lie is then known to a bin or two.
//  3. Weights: sums per warp of what certainly stays; the elements of the open bins go
//     to a list.
//  4. The list decides both borders (radix select by number, then by sum of weights,
//     ties by id), in one CTA.  Lists that overflow (all logits alike, or top-p so near
//     1 that its border lies among very many small weights) are replaced by the row
//     itself: the same selection by the whole cluster, a pass over the row a digit.
//  5. The warps' sums, in id order, give the run that holds the draw, which its CTA
//     looks through again.
//
// What bounds it: one row, the chain of passes and cluster barriers (152064 fp32, greedy 5.2 us, unfiltered 13,
// top-k 50 16, top-p 0.9 27); many, instructions: some 50 for each weight that counts, shared-memory atomics of the
// histogram (256 rows of 128256 bf16: 15.7, 82, 38, 167 us; reading them once from HBM would take 9.7).  Top-p near 1,
// logits N(0, 2) and 32 high ones, T 1, at 0.9 / 0.99 / 0.995 / 0.999 / 0.9999: one row 27 / 32 / 36 / 90 / 93 us, 64 of
// 152064 68 / 80 / 112 / 218 / 226, the 256 167 / 184 / 371 / 796 / 839: from 0.995 or 0.999 on lists overflow.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ddl_device.cuh"
#include "ddl_internal.h"

namespace ddl {
namespace {

constexpr int SM_THREADS = 512, SM_WARPS = SM_THREADS / 32;
constexpr int SM_MAX_CLUSTER = 16;
constexpr int SM_BINS = 2048;
constexpr float SM_PER_OCTAVE = 47.6f;       // 2048 bins over 43 octaves
constexpr float SM_OCTAVES = 43.f;           // weights below 2^-43 are 0; 2^20 of them up to 1 + 2^-30 fit 64 bits
constexpr int SM_FRAC = 1024;                // places inside a bin
constexpr int SM_LIST = 4096;                // elements of a CTA's list, and of the row's
constexpr uint32_t SM_ALL_IDS = 0xfffffu;
static_assert(DDL_SAMPLE_MAX_VOCAB <= 1 << 20, "sums of weights, ids in 20 bits of a list entry");

// 2^(i/64) as two floats: by repeated square roots of 2 (Newton), multiplied up, in double.
struct ExpTable {
  float hi[64], lo[64];
};
constexpr ExpTable make_exp_table() {
  double root[6] = {};
  double x = 2.0;
  for (int k = 0; k < 6; ++k) {  // root[k] = 2^(1 / 2^(k + 1))
    double y = x;
    for (int n = 0; n < 60; ++n) y = 0.5 * (y + x / y);
    root[k] = y;
    x = y;
  }
  ExpTable t = {};
  for (int i = 0; i < 64; ++i) {
    double p = 1.0;
    for (int k = 0; k < 6; ++k)
      if (i & (32 >> k)) p *= root[k];
    t.hi[i] = (float)p;
    t.lo[i] = i ? (float)(p - (double)(float)p) : 0x1p-60f;  // (never zero: its exponent is changed by addition)
  }
  return t;
}
__device__ const ExpTable g_exp_table = make_exp_table();

constexpr float LOG2E_HI = 1.44269502162933349609375f, LOG2E_LO = 1.92596299e-8f;  // log2 e

struct SampleArgs {
  const void* logits;
  int64_t stride;
  const float *temperature, *top_p, *min_p, *u;
  const int32_t* top_k;
  int32_t* token;
  float* logp;
  int32_t V, cluster;
};

struct Entry {
  uint32_t key, id;
};

// The shared memory of a CTA that others of its cluster read, and its own.
struct SampleSmem {
  ExpTable table;
  union {
    struct {
      uint32_t count[SM_BINS], place[SM_BINS];    // histogram of the CTA's elements
      uint32_t rcount[SM_BINS], rplace[SM_BINS];  // 2048 / C bins of the cluster's
    };
    Entry all[SM_LIST];  // the row's list, when the histogram is done with
  };
  unsigned long long warp_sum[SM_WARPS];      // per warp: weights that certainly stay
  unsigned long long sums[2];                 // weights before the open bins, and before the k-th element's
  unsigned long long chunk[SM_MAX_CLUSTER * SM_WARPS];
  uint32_t num[256], mass_lo[256], mass_hi[256];  // a digit's elements and their weights
  uint32_t range[2];
  unsigned long long red64[SM_WARPS];
  float redf[SM_WARPS];
  uint32_t redu[SM_WARPS];
  float top;
  uint32_t top_id;
  double log_m;
  uint32_t list_n;
  struct {
    uint32_t key, id;          // the last element that stays
    unsigned long long total;  // the kept tokens' sum
    unsigned long long rest;   // the draw, from the run's first element
    int32_t run;               // cluster-wide warp that holds it
  } end;
  int32_t sel_i[4];
  unsigned long long sel_u[2];
  Entry list[SM_LIST];
};

__device__ __forceinline__ void ldu4_cluster(uint32_t a, uint32_t (&v)[4]) {
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ unsigned long long ldl_cluster(uint32_t a) {
  unsigned long long v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
  return v;
}

// Order-preserving key of a logit (both zeros alike); NaN and -inf are no candidates.
__device__ __forceinline__ uint32_t logit_key(float l) {
  const uint32_t b = __float_as_uint(l + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// The weights of a row.
struct Weigher {
  float top, ch, cl;  // log2 e / T in two floats
  bool inf;           // the row's largest logit is +inf: such logits count as 0, all others as none
  const ExpTable* table;
  template <int N>
  __device__ __forceinline__ void fix(float (&l)[N]) const {
    if (inf) {
#pragma unroll
      for (int i = 0; i < N; ++i) l[i] = l[i] == INFINITY ? 0.f : -INFINITY;
    }
  }
  // log2 of the weight, rounded: not increasing with falling logits.  Not above -43 (or NaN): no weight.
  __device__ __forceinline__ float log2w(float l) const { return (l - top) * ch; }
  static __device__ __forceinline__ bool has(float p) { return p > -SM_OCTAVES; }
  // The weight, as 2^22 hi + lo units of 2^-43; p = log2w(l) (not above -43: of no meaning).
  __device__ __forceinline__ void parts(float l, float p, uint32_t& hi, int32_t& low) const {
    // l - top = d + e exactly, log2 of the weight p + lo
    const float d = l - top, b = d - l, e = (l - (d - b)) + (-top - b);
    const float lo = fmaf(d, ch, -p) + fmaf(d, cl, e * ch);
    const float m = fmaf(p, 64.f, 0x1.8p23f);  // (rounds 64 p to an integer k in the low bits)
    const uint32_t k = __float_as_uint(m);
    const float r = fmaf(0x1.8p23f - m, 0x1p-6f, p);  // p = k / 64 + r, exactly
    const uint32_t n = k >> 6 << 23;                  // whole octaves, as an exponent
    const float th = __uint_as_float(__float_as_uint(table->hi[k & 63]) + n);
    const float tl = __uint_as_float(__float_as_uint(table->lo[k & 63]) + n);
    // 2^(r + lo) = 1 + z + t, z a float
    constexpr float LN2F = 0.693147180559945f;
    const float z = r * LN2F;
    const float zl = fmaf(lo, LN2F, fmaf(r, LN2F, -z));
    const float t = fmaf(z * z, fmaf(z, 0.16666667f, 0.5f), fmaf(zl, z, zl));
    // (th + tl) (1 + z + t) = wh + wl
    const float x = th * z, wh = th + x;
    const float wl = (x - (wh - th)) + (fmaf(th, z, -x) + fmaf(th, t, fmaf(tl, z, tl)));
    const float ah = (wh + wl) + 6.f, al = ((wh - (ah - 6.f)) + wl) + 0x1.8p-20f;
    hi = __float_as_uint(ah) - 0x40c00000u;
    low = (int32_t)(__float_as_uint(al) - 0x35c00000u);
  }
  static __device__ __forceinline__ unsigned long long units(uint32_t h, int32_t s) {
    return ((unsigned long long)h << 22) + (long long)s;
  }
  __device__ __forceinline__ unsigned long long weight(float l) const {
    const float p = log2w(l);
    uint32_t h;
    int32_t s;
    parts(l, p, h, s);
    return has(p) ? units(h, s) : 0ull;
  }
  // log2 w = p to bins, from the top: the nearest integer to 47.6 |p|, as the low bits of a float
  static __device__ __forceinline__ float bin_bits(float p) { return fmaf(p, -SM_PER_OCTAVE, 0x1p23f); }
  static __device__ __forceinline__ int bin_of(float p) { return (int)(__float_as_uint(bin_bits(p)) - 0x4b000000u); }
};

// The elements of a warp's run: f(id of the first, logits) for 16 bytes a lane, in ascending
// order within a lane; the row's ends and unaligned rows element by element (-inf outside).
template <int DT>
struct Row {
  static constexpr int VEC = DT == DDL_T_F32 ? 4 : 8;
  const uint8_t* base;  // of the row's first element, rounded down to 16 bytes
  int off;              // elements before it there
  int V, nvec;
  __device__ __forceinline__ Row(const SampleArgs& A, int b) {
    constexpr int SZ = DT == DDL_T_F32 ? 4 : 2;
    const uint8_t* p = reinterpret_cast<const uint8_t*>(A.logits) + (int64_t)b * A.stride * SZ;
    off = (int)((uintptr_t)p & 15) / SZ;
    base = p - off * SZ;
    V = A.V;
    nvec = (int)(((int64_t)V + off + VEC - 1) / VEC);
  }
  __device__ __forceinline__ int run_begin(int run, int runs) const { return (int)((int64_t)nvec * run / runs); }
  __device__ __forceinline__ float one(int64_t q) const {
    if (DT == DDL_T_F32) return reinterpret_cast<const float*>(base)[q];
    const uint16_t x = reinterpret_cast<const uint16_t*>(base)[q];
    if (DT == DDL_T_BF16) return bf16_bits_to_f32(x);
    return __half2float(__ushort_as_half(x));
  }
  static __device__ __forceinline__ void unpack(const uint4& x, float (&l)[VEC]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      if (DT == DDL_T_F32) l[i] = __uint_as_float(w[i & 3]);
      else if (DT == DDL_T_BF16) l[i] = i & 1 ? bf16hi_f32(w[i / 2]) : bf16lo_f32(w[i / 2]);
      else {
        const __half2 h2 = *reinterpret_cast<const __half2*>(&w[i / 2]);
        l[i] = i & 1 ? __high2float(h2) : __low2float(h2);
      }
    }
  }
  __device__ __forceinline__ uint4 load(int v) const { return *reinterpret_cast<const uint4*>(base + (int64_t)v * 16); }
  // The logits of vector v, -inf from v1 on and outside the row.
  __device__ __forceinline__ void values(int v, int v1, float (&l)[VEC]) const {
    if (v < v1 && v * VEC >= off && (int64_t)(v + 1) * VEC <= (int64_t)V + off) {
      unpack(load(v), l);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const int64_t q = (int64_t)v * VEC + i;
        l[i] = v < v1 && q >= off && q < (int64_t)V + off ? one(q) : -INFINITY;
      }
    }
  }
  // All lanes of the warp take part in every f, and in g, which comes after U of them at most.
  template <class F>
  __device__ __forceinline__ void each(int v0, int v1, F&& f) const {
    each(v0, v1, f, []() {});
  }
  // U: loads on their way.
  template <int U = 4, class F, class G>
  __device__ __forceinline__ void each(int v0, int v1, F&& f, G&& g) const {
    const int lane = threadIdx.x & 31, w0 = off > 0 ? 1 : 0, w1 = min(v1, (V + off) / VEC);  // whole: [w0, w1)
    for (int v = v0; v < v1; v += 32 * U) {
      if (v >= w0 && v + 32 * U <= w1) {
        uint4 x[U];
#pragma unroll
        for (int j = 0; j < U; ++j) x[j] = load(v + 32 * j + lane);
#pragma unroll
        for (int j = 0; j < U; ++j) {
          float l[VEC];
          unpack(x[j], l);
          f((v + 32 * j + lane) * VEC - off, l);
        }
        g();
      } else {
#pragma unroll 1
        for (int j = v; j < min(v + 32 * U, v1); j += 32) {
          float l[VEC];
          values(j + lane, v1, l);
          f((j + lane) * VEC - off, l);
        }
        g();
      }
    }
  }
};

__device__ __forceinline__ unsigned long long warp_add(unsigned long long x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(FULL, x, o);
  return x;
}
// Sum of a word of every CTA of the cluster (all lanes of a warp call it; C <= 32).
__device__ __forceinline__ uint32_t cluster_add(const uint32_t* p, int C) {
  const int lane = threadIdx.x & 31;
  return __reduce_add_sync(FULL, lane < C ? ldu_cluster(cluster_addr(smem_addr(p), lane)) : 0u);
}
// Exclusive sum over the CTA of a value per thread; `all` gets the sum of all.
template <class T>
__device__ __forceinline__ T block_before(T x, T* ws, T& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(FULL, inc, o);
    if (lane >= o) inc += y;
  }
  __syncthreads();
  if (lane == 31) ws[warp] = inc;
  __syncthreads();
  T before = 0;
  all = 0;
#pragma unroll
  for (int w = 0; w < SM_WARPS; ++w) {
    if (w < warp) before += ws[w];
    all += ws[w];
  }
  return before + inc - x;
}

// Sum of 64 bits in shared memory by two 32-bit additions (lo's old value tells its carry).
__device__ __forceinline__ void add64(uint32_t* lo, uint32_t* hi, unsigned long long x) {
  const uint32_t l = (uint32_t)x, was = atomicAdd(lo, l), h = (uint32_t)(x >> 32) + (was + l < was ? 1u : 0u);
  if (h) atomicAdd(hi, h);
}

// Where the elements of a selection come from: a list in this CTA's shared memory, or the
// whole cluster's runs of the row (which of them: in()).
template <int DT, bool LIST>
struct Source {
  SampleSmem& S;
  int n;
  const Row<DT>& row;
  const Weigher& W;
  int v0, v1, C;
  __device__ __forceinline__ void sync() const {
    if (LIST) __syncthreads();
    else cluster_sync();
  }
  __device__ __forceinline__ uint32_t all(uint32_t* p) const {  // a word's sum over the CTAs
    if (LIST) return *p;
    uint32_t s = 0;
    for (int c = 0; c < C; ++c) s += ldu_cluster(cluster_addr(smem_addr(p), c));
    return s;
  }
  // f(key, id) for every element
  template <class F>
  __device__ __forceinline__ void each(F&& f) const {
    if (LIST) {
      for (int i = threadIdx.x; i < n; i += SM_THREADS) f(S.all[i].key, S.all[i].id & SM_ALL_IDS);
    } else {
      row.each(v0, v1, [&](int id, float(&l)[Row<DT>::VEC]) {
        W.fix(l);
#pragma unroll
        for (int i = 0; i < Row<DT>::VEC; ++i)
          if (W.has(W.log2w(l[i]))) f(logit_key(l[i]), (uint32_t)(id + i));
      });
    }
  }
  // One digit of 256: the first, in ascending order, at which the running number of the elements (BY_MASS: of
  // their weights) reaches `want`; what lies before it is taken off `want`, the number of elements in it is left in
  // `inside`.  classify: an element's digit, or -1.
  template <bool BY_MASS, class F>
  __device__ __forceinline__ int digit(F&& classify, unsigned long long& want, uint32_t& inside) const {
    const int tid = threadIdx.x, lane = tid & 31;
    if (tid < 256) S.num[tid] = S.mass_lo[tid] = S.mass_hi[tid] = 0;
    __syncthreads();
    each([&](uint32_t key, uint32_t id) {
      const int d = classify(key, id);
      if (d < 0) return;
      atomicAdd(&S.num[d], 1u);
      if (BY_MASS) add64(&S.mass_lo[d], &S.mass_hi[d], W.weight(key_logit(key)));
    });
    sync();
    if (tid < 32) {  // eight digits a lane
      uint32_t num[8];
      unsigned long long mine[8], sum = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        num[j] = all(&S.num[lane * 8 + j]);
        mine[j] = num[j];
        if (BY_MASS) {
          if (LIST) {
            mine[j] = S.mass_lo[lane * 8 + j] + ((unsigned long long)S.mass_hi[lane * 8 + j] << 32);
          } else {
            mine[j] = 0;
            for (int c = 0; c < C; ++c)
              mine[j] += ldu_cluster(cluster_addr(smem_addr(&S.mass_lo[lane * 8 + j]), c)) +
                         ((unsigned long long)ldu_cluster(cluster_addr(smem_addr(&S.mass_hi[lane * 8 + j]), c)) << 32);
          }
        }
        sum += mine[j];
      }
      unsigned long long inc = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(FULL, inc, o);
        if (lane >= o) inc += y;
      }
      const unsigned long long total = __shfl_sync(FULL, inc, 31);
      if (want > total) want = total;  // (never, by the bounds of the bins)
      unsigned long long before = inc - sum;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (before < want && before + mine[j] >= want) {
          S.sel_i[0] = lane * 8 + j;
          S.sel_i[1] = (int)num[j];
          S.sel_u[0] = want - before;
        }
        before += mine[j];
      }
    }
    sync();  // (the cluster's numbers are read before they are cleared)
    const int d = S.sel_i[0];
    inside = (uint32_t)S.sel_i[1];
    want = S.sel_u[0];
    return d;
  }
  // The last element that stays of those `in` accepts: the `want`-th (BY_MASS: the first at which
  // the running sum of weights reaches `want`), in the order (key descending, id ascending); id
  // SM_ALL_IDS where all accepted ones of its key stay.
  template <bool BY_MASS, class F>
  __device__ __forceinline__ Entry select(F&& in, unsigned long long want) const {
    // the range of keys: what its numbers share needs no digit
    uint32_t top = 0u, low = ~0u;
    each([&](uint32_t key, uint32_t id) {
      if (in(key, id)) {
        top = max(top, key);
        low = min(low, key);
      }
    });
    top = __reduce_max_sync(FULL, top);
    low = __reduce_min_sync(FULL, low);
    __syncthreads();  // (earlier readers of these words)
    if (threadIdx.x == 0) {
      S.range[0] = 0u;
      S.range[1] = ~0u;
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) {
      atomicMax(&S.range[0], top);
      atomicMin(&S.range[1], low);
    }
    sync();
    top = S.range[0];
    low = S.range[1];
    if (!LIST) {
      for (int c = 0; c < C; ++c) {
        top = max(top, ldu_cluster(cluster_addr(smem_addr(&S.range[0]), c)));
        low = min(low, ldu_cluster(cluster_addr(smem_addr(&S.range[1]), c)));
      }
    }
    sync();
    // digits of top - key, ascending
    Entry e = {top, SM_ALL_IDS};
    uint32_t inside = 0, at = 0;  // top - key of the element sought, its digits so far
    int bits = top > low ? 32 - __clz(top - low) : 0;
    bool first = true;
    while (bits > 0) {
      const int shift = bits > 8 ? bits - 8 : 0;
      at |= (uint32_t)digit<BY_MASS>(
                [&](uint32_t key, uint32_t id) {
                  const uint32_t x = top - key;
                  return in(key, id) && (first || (x ^ at) >> bits == 0) ? (int)((x >> shift) & 255u) : -1;
                },
                want, inside)
            << shift;
      bits = shift;
      first = false;
      if (inside == 1 && bits > 0) break;  // one element left: its key is in range below
    }
    if (bits > 0) {  // the element's own key
      if (threadIdx.x == 0) S.range[1] = ~0u;
      sync();
      each([&](uint32_t key, uint32_t id) {
        const uint32_t x = top - key;
        if (in(key, id) && (x ^ at) >> bits == 0) S.range[1] = x;
      });
      sync();
      at = S.range[1];
      if (!LIST)
        for (int c = 0; c < C; ++c) at = min(at, ldu_cluster(cluster_addr(smem_addr(&S.range[1]), c)));
      sync();
      e.key = top - at;
      return e;  // (no other has its key)
    }
    e.key = top - at;
    if (first) {  // all keys are one
      uint32_t n = 0;
      each([&](uint32_t key, uint32_t id) { n += in(key, id); });
      n = __reduce_add_sync(FULL, n);
      if (threadIdx.x == 0) S.range[0] = 0u;
      __syncthreads();
      if ((threadIdx.x & 31) == 0) atomicAdd(&S.range[0], n);
      sync();
      inside = all(&S.range[0]);
      sync();
    }
    if (BY_MASS) {  // elements of one key weigh the same
      const unsigned long long w = W.weight(key_logit(e.key));
      want = w ? (want + w - 1) / w : 1;
    }
    if (want >= inside) return e;  // all of its key stay
    e.id = 0;
    for (int shift = 16; shift >= 0; shift -= 8) {
      const uint32_t hi = shift == 16 ? 0u : ~0u << (shift + 8);
      e.id |= (uint32_t)digit<false>(
                  [&](uint32_t key, uint32_t id) {
                    return in(key, id) && key == e.key && ((id ^ e.id) & hi) == 0 ? (int)((id >> shift) & 255u) : -1;
                  },
                  want, inside)
              << shift;
    }
    return e;
  }
  // Sum of the weights of the elements that `in` accepts.
  template <class F>
  __device__ __forceinline__ unsigned long long sum(F&& in) const {
    unsigned long long s = 0, whole;
    each([&](uint32_t key, uint32_t id) {
      if (in(key, id)) s += W.weight(key_logit(key));
    });
    block_before(s, S.red64, whole);
    if (!LIST) {
      if (threadIdx.x == 0) S.sel_u[1] = whole;
      cluster_sync();
      whole = 0;
      for (int c = 0; c < C; ++c) whole += ldl_cluster(cluster_addr(smem_addr(&S.sel_u[1]), c));
      cluster_sync();
    }
    return whole;
  }
};

// floor(x s) and ceil(x s) of a number x in [0, 1) with 64 fraction bits.
__device__ __forceinline__ unsigned long long frac64(float x) { return (unsigned long long)((double)x * 18446744073709551616.0); }
__device__ __forceinline__ unsigned long long ceil_mul(unsigned long long x, unsigned long long s) {
  return __umul64hi(x, s) + (x * s ? 1ull : 0ull);
}

// No element stays behind this one in the order (key descending, id ascending).
__device__ __forceinline__ bool stays(uint32_t key, uint32_t id, const Entry& last) {
  return key > last.key || (key == last.key && id <= last.id);
}

// f(logit, whether it is one) for the marked ones of a lane's logits, one after the other; `most`: of any lane of the warp.
template <int N, class F>
__device__ __forceinline__ void marked(uint32_t mark, uint32_t most, const float (&l)[N], const F& f) {
  for (; most > 0; --most) {
    const int at = __ffs(mark) - 1;
    mark &= mark - 1;
    float x = l[0];
#pragma unroll
    for (int i = 1; i < N; ++i) x = at == i ? l[i] : x;
    f(x, at >= 0);
  }
}

struct Open {     // what the histogram says of the row's borders
  int k_bin;      // bin of the k-th element (SM_BINS: none)
  uint32_t k_in;  // its place among the bin's elements, from 1
  int p_lo, p_hi; // bins in which the top-p head may end (p_lo > p_hi: no top-p)
};

template <int DT>
__global__ void __launch_bounds__(SM_THREADS, 2) sample_kernel(const __grid_constant__ SampleArgs A) {
  extern __shared__ __align__(16) uint8_t sample_smem[];
  SampleSmem& S = *reinterpret_cast<SampleSmem*>(sample_smem);
  constexpr int VEC = Row<DT>::VEC;
  constexpr int U = 16 / VEC;  // loads on their way where registers are short (256 rows of 128256 bf16, top-p 0.9: 167 us, with 4 187)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = A.cluster, b = blockIdx.x / C, rank = blockIdx.x % C, runs = C * SM_WARPS;
  if (tid < 64) {
    S.table.hi[tid] = g_exp_table.hi[tid];
    S.table.lo[tid] = g_exp_table.lo[tid];
  }
  for (int i = tid; i < SM_BINS; i += SM_THREADS) S.count[i] = S.place[i] = S.rcount[i] = S.rplace[i] = 0;
  pdl_trigger();
  pdl_wait();
  const Row<DT> row(A, b);
  const int v0 = row.run_begin(rank * SM_WARPS + warp, runs), v1 = row.run_begin(rank * SM_WARPS + warp + 1, runs);
  const float T = A.temperature ? A.temperature[b] : 1.f;
  const int32_t K = A.top_k ? A.top_k[b] : 0;
  const float P = A.top_p ? A.top_p[b] : 1.f, M = A.min_p ? A.min_p[b] : 0.f;
  const bool greedy = !(T >= 0x1p-60f) || M > 1.f;  // (no weight reaches a min-p above 1: the first candidate alone)
  const bool by_k = K > 0 && K < A.V, by_p = P < 1.f, by_m = M > 0.f && M < 1.f && T < INFINITY;
  // 1. the maximum, and its lowest id
  float top = -INFINITY;
  int top_id = 0x7fffffff;
  row.each(v0, v1, [&](int id, float(&l)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (l[i] > top) {
        top = l[i];
        top_id = id + i;
      }
  });
  auto better = [&](float l, int i) {
    if (l > top || (l == top && i < top_id)) {
      top = l;
      top_id = i;
    }
  };
  auto warp_best = [&]() {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const float l = __shfl_xor_sync(FULL, top, o);
      better(l, __shfl_xor_sync(FULL, top_id, o));
    }
  };
  const float mine_top = top;
  warp_best();
  if (lane == 0) {
    S.redf[warp] = top;
    S.redu[warp] = (uint32_t)top_id;
  }
  if (tid == 32 && by_m) S.log_m = (double)T * log((double)M);
  __syncthreads();
  if (warp == 0) {
    top = lane < SM_WARPS ? S.redf[lane] : -INFINITY;
    top_id = lane < SM_WARPS ? (int)S.redu[lane] : 0x7fffffff;
    warp_best();
    if (lane == 0) {
      S.top = top;
      S.top_id = (uint32_t)top_id;
      S.list_n = 0;
    }
  }
  cluster_sync();
  top = lane < C ? ld_cluster(cluster_addr(smem_addr(&S.top), lane)) : -INFINITY;
  top_id = lane < C ? (int)ldu_cluster(cluster_addr(smem_addr(&S.top_id), lane)) : 0x7fffffff;
  warp_best();
  if (greedy || top == -INFINITY) {
    if (rank == 0 && tid == 0) {
      const bool none = top == -INFINITY;
      A.token[b] = none ? -1 : top_id;
      if (A.logp) A.logp[b] = none ? -INFINITY : 0.f;
    }
    cluster_sync();  // (nobody's shared memory goes while another reads it)
    return;
  }
  Weigher W;
  W.inf = top == INFINITY;
  W.top = W.inf ? 0.f : top;
  W.ch = LOG2E_HI / T;  // log2 e / T: quotient and, from its exact remainder, the rest
  W.cl = T < INFINITY ? (fmaf(-W.ch, T, LOG2E_HI) + LOG2E_LO) / T : 0.f;
  W.table = &S.table;
  // min-p as a bound on the logit: the smallest fp32 number at or above top + T ln(min_p)
  // (an infinite T makes all weights 1)
  const float least = by_m ? __double2float_ru((double)W.top + S.log_m) : M == 1.f && T < INFINITY ? W.top : -INFINITY;

  // 1b. the bound by the lanes' maxima, in bins of 8; all elements from there up to the list.  For a k of up to half the
  // lanes (and half the list): among so many maxima the k-th largest is near the row's k-th, and there are enough of them.  It and the
  // histogram's way, 256 rows of 128256 bf16 (lanes 512), k 50 / 256: 38 and 83 us / 48 and 87; 64 of 152064 fp32
  // (2048), k 50 / 1000: 25 and 44 / 36 and 48; one row (8192), k 50 / 2000: 16 and 21 / 22.0 and 22.4.
  Open o = {SM_BINS, 0u, SM_BINS, -1};
  uint32_t listed = 0;
  bool heads = by_k && K <= min(C * SM_THREADS / 2, SM_LIST / 2);  // the list holds all elements of the top-k head
  if (heads) {
    float own[1] = {mine_top};
    W.fix(own);
    const float p = W.log2w(own[0]);
    if (tid < 256) S.num[tid] = 0;
    __syncthreads();
    if (W.has(p)) atomicAdd(&S.num[W.bin_of(p) >> 3], 1u);
    cluster_sync();
    uint32_t n = 0;
    if (tid < 256) {
#pragma unroll 8
      for (int c = 0; c < C; ++c) n += ldu_cluster(cluster_addr(smem_addr(&S.num[tid]), c));
    }
    uint32_t all;
    const uint32_t before = block_before(n, S.redu, all);
    if (before < (uint32_t)K && before + n >= (uint32_t)K) S.sel_i[0] = tid * 8 + 7;
    __syncthreads();
    heads = all >= (uint32_t)K;
    if (heads) {
      const int from = S.sel_i[0];
      row.each(v0, v1, [&](int id, float(&l)[VEC]) {
        W.fix(l);
        float top = l[0];
#pragma unroll
        for (int i = 1; i < VEC; ++i) top = fmaxf(top, l[i]);
        const float p = W.log2w(top);
        if (!W.has(p) || W.bin_of(p) > from) return;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float q = W.log2w(l[i]);
          if (W.has(q) && W.bin_of(q) <= from) {
            const uint32_t to = atomicAdd(&S.list_n, 1u);
            if (to < SM_LIST) S.list[to] = {logit_key(l[i]), (uint32_t)(id + i) | ((uint32_t)(rank * SM_WARPS + warp) << 20)};
          }
        }
      });
      if (tid < SM_WARPS) S.warp_sum[tid] = 0;
      cluster_sync();
      listed = cluster_add(&S.list_n, C);
      heads = listed <= SM_LIST;
      if (!heads) {
        cluster_sync();  // (all have read list_n)
        if (tid == 0) S.list_n = 0;
      }
    }
  }

  // 2. the histogram
  if (!heads && (by_k || by_p)) {
    row.each(v0, v1, [&](int, float(&l)[VEC]) {
      W.fix(l);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float p = W.log2w(l[i]), m = W.bin_bits(p);
        const uint32_t at = __float_as_uint(m) - 0x4b000000u;
        if (W.has(p)) atomicAdd(&S.count[at], 1u);
        // the place, -1/2 .. 1/2 of the bin, in units of 1/1024 from its upper end
        const float f = fmaf(p, -SM_PER_OCTAVE, 0x1p23f - m);
        if (by_p && W.has(p))
          atomicAdd(&S.place[at], __float_as_uint(fmaf(f, (float)SM_FRAC, 0x1p23f + SM_FRAC / 2)) - 0x4b000000u);
      }
    });
    cluster_sync();
    // bins [rank per, (rank + 1) per) of the cluster's CTAs: each of `split` parts of the threads adds up as many of them
    const int per = SM_BINS / C, split = max(SM_THREADS / per, 1), step = C / split;
    for (int i = tid & (per - 1), c0 = tid / per * step; i < per; i += SM_THREADS) {
      uint32_t n = 0, q = 0;
#pragma unroll 4
      for (int c = c0; c < c0 + step; ++c) {
        n += ldu_cluster(cluster_addr(smem_addr(&S.count[rank * per + i]), c));
        if (by_p) q += ldu_cluster(cluster_addr(smem_addr(&S.place[rank * per + i]), c));
      }
      atomicAdd(&S.rcount[i], n);
      if (by_p) atomicAdd(&S.rplace[i], q);
    }
    cluster_sync();
    // every CTA: the bins' numbers and bounds of their sums of weights; thread i has bins 4 i .. 4 i + 3
    constexpr int PER = SM_BINS / SM_THREADS;
    static_assert(PER == 4, "16 bytes a thread, of one CTA's bins");
    uint32_t n[PER], place[PER] = {}, sum = 0, all_n;
    {
      const int c = tid * PER / per, at = tid * PER - c * per;
      ldu4_cluster(cluster_addr(smem_addr(&S.rcount[at]), c), n);
      if (by_p) ldu4_cluster(cluster_addr(smem_addr(&S.rplace[at]), c), place);
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) sum += n[j];
    if (tid == 0) {
      S.sel_i[0] = S.sel_i[2] = S.sel_i[3] = SM_BINS;
      S.sel_i[1] = 0;
    }
    uint32_t before = block_before(sum, S.redu, all_n);
    if (by_k && (uint32_t)K < all_n) {
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        if (before < (uint32_t)K && before + n[j] >= (uint32_t)K) {
          S.sel_i[0] = tid * PER + j;
          S.sel_i[1] = K - (int)before;
        }
        before += n[j];
      }
    }
    __syncthreads();
    o.k_bin = S.sel_i[0];
    o.k_in = (uint32_t)S.sel_i[1];
    if (by_p) {
      // A bin's sum is n 2^-(i - 1/2 + mean place) / 47.6, up to the rounding of the places (1 / 2048 of a bin each:
      // 7e-6 of the sum), the curvature inside a bin ((ln 2 / 47.6)^2 / 8 = 2.7e-5) and log2 w's own rounding
      // (2^-19: 2e-6): within 1e-4.  Of the k-th element's bin, the last one, k_in elements of any place.
      float w[PER], sw = 0.f, all_w;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const int i = tid * PER + j;
        const float cnt = (float)n[j], at = (float)i - 0.5f;
        w[j] = i < o.k_bin && n[j]
                   ? cnt * exp2f(-(at + __fdividef((float)place[j], cnt * SM_FRAC)) * (1.f / SM_PER_OCTAVE)) : 0.f;
        sw += w[j];
      }
      float bw = block_before(sw, S.redf, all_w);
      const float k_top = o.k_bin < SM_BINS ? (float)o.k_in * exp2f(((float)o.k_bin - 0.5f) * (-1.f / SM_PER_OCTAVE)) : 0.f;
      const float k_low = k_top * exp2f(-1.f / SM_PER_OCTAVE);
      // sums of 2048 fp32 numbers: some 40 additions in a row, 2^-24 each: within 1e-5.  Taken with room: 3e-4 for the
      // bins' sums on both sides of the total, 1e-4 for the running sum.
      const float want_lo = P * (all_w + k_low) * 0.9997f, want_hi = P * (all_w + k_top) * 1.0003f;
      int first_lo = SM_BINS, first_hi = SM_BINS;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const int i = tid * PER + j;
        bw += w[j];
        if (w[j] > 0.f && bw * 1.0001f >= want_lo) first_lo = min(first_lo, i);
        if (w[j] > 0.f && bw * 0.9999f >= want_hi) first_hi = min(first_hi, i);
      }
      first_lo = __reduce_min_sync(FULL, first_lo);
      first_hi = __reduce_min_sync(FULL, first_hi);
      if (lane == 0) {
        atomicMin(&S.sel_i[2], first_lo);
        atomicMin(&S.sel_i[3], first_hi);
      }
      __syncthreads();
      o.p_hi = min(min(S.sel_i[3], o.k_bin), SM_BINS - 1);
      o.p_lo = min(S.sel_i[2], o.p_hi);
    }
    __syncthreads();
  }
  // Bins before `sure` stay (as far as top-k and top-p go).  Where min-p's bound lies in one of them it comes first,
  // and what the open bins would decide does not matter; else it hides none of them.
  const int sure = by_p ? o.p_lo : o.k_bin;
  bool open = heads || o.k_bin < SM_BINS || by_p;
  if (open && !heads && least > -INFINITY && W.has(W.log2w(least)) && W.bin_of(W.log2w(least)) < sure) open = false;

  // 3. exact sums of what certainly stays, the list of the open bins
  unsigned long long above = 0, to_k = 0;  // before the open bins; before the k-th element's bin, open ones among them
  uint32_t hs = 0, hs2 = 0;                // of a few elements: high and low parts
  int32_t ls = 0, ls2 = 0;
  if (heads) {
    // (nothing to add up)
  } else if (!open) {
    auto take = [&](float l, bool on) {
      const float p = W.log2w(l);
      uint32_t hi;
      int32_t low;
      W.parts(l, p, hi, low);
      if (on && W.has(p)) {
        hs += hi;
        ls += low;
      }
    };
    auto add_up = [&]() {
      above += W.units(hs, ls);
      hs = 0;
      ls = 0;
    };
    // min-p: the weights of what stays, one after the other, where no lane of the warp has more of them than half its elements
    // (256 rows of 128256 bf16, 0.05: 43 us, all weights 81; 1e-9: 91, 85)
    if (least == -INFINITY) {
      row.template each<U>(
          v0, v1,
          [&](int, float(&l)[VEC]) {
            W.fix(l);
#pragma unroll
            for (int i = 0; i < VEC; ++i) take(l[i], true);
          },
          add_up);
    } else {
      row.template each<U>(
          v0, v1,
          [&](int, float(&l)[VEC]) {
            W.fix(l);
            uint32_t mark = 0;
#pragma unroll
            for (int i = 0; i < VEC; ++i)
              if (l[i] >= least) mark |= 1u << i;
            const uint32_t most = __reduce_max_sync(FULL, (uint32_t)__popc(mark));
            if (most > VEC / 2) {
#pragma unroll
              for (int i = 0; i < VEC; ++i) take(l[i], (mark >> i & 1) != 0);
            } else {
              marked(mark, most, l, take);
            }
          },
          add_up);
    }
  } else {
    // bins as the floats that bin_bits gives
    const float p_lo = 0x1p23f + (float)sure, p_hi = 0x1p23f + (float)(by_p ? o.p_hi : o.k_bin), k_bin = 0x1p23f + (float)o.k_bin;
    auto bin = [&](float p) { return W.has(p) ? W.bin_bits(p) : INFINITY; };
    auto is_open = [&](float m) { return (m >= p_lo && m <= p_hi) || m == k_bin; };
    auto take = [&](float l, float p, float m) {
      uint32_t hi;
      int32_t low;
      W.parts(l, p, hi, low);
      if (m < p_lo) {
        hs += hi;
        ls += low;
      }
      if (m < k_bin) {
        hs2 += hi;
        ls2 += low;
      }
    };
    auto list = [&](uint32_t in, int id, const float(&l)[VEC]) {  // elements of the open bins
      if (!in) return;
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (in >> i & 1) {
          const uint32_t to = atomicAdd(&S.list_n, 1u);
          if (to < SM_LIST) S.list[to] = {logit_key(l[i]), (uint32_t)(id + i) | ((uint32_t)(rank * SM_WARPS + warp) << 20)};
        }
    };
    auto add_up = [&]() {
      above += W.units(hs, ls);
      to_k += W.units(hs2, ls2);
      hs = hs2 = 0;
      ls = ls2 = 0;
    };
    // all weights; of top-k that leaves few elements, only theirs (256 rows of 128256 bf16, theirs and all weights: top-k
    // 5000 108 and 135 us, 16032 128 and 139, 19008 132 and 140, 30000 146 and 144, 100000 184 and 144)
    if (o.k_bin == SM_BINS || K > A.V / 8) {
      row.template each<U>(
          v0, v1,
          [&](int id, float(&l)[VEC]) {
            W.fix(l);
            uint32_t in = 0;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
              const float p = W.log2w(l[i]), m = bin(p);
              take(l[i], p, m);
              if (is_open(m)) in |= 1u << i;
            }
            list(in, id, l);
          },
          add_up);
    } else {
      row.template each<U>(
          v0, v1,
          [&](int id, float(&l)[VEC]) {
            W.fix(l);
            uint32_t in = 0, mark = 0;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
              const float m = bin(W.log2w(l[i]));
              if (m < k_bin) mark |= 1u << i;
              if (is_open(m)) in |= 1u << i;
            }
            marked(mark, __reduce_max_sync(FULL, (uint32_t)__popc(mark)), l, [&](float x, bool on) {
              const float p = W.log2w(x);
              take(x, p, on ? W.bin_bits(p) : INFINITY);
            });
            list(in, id, l);
          },
          add_up);
    }
  }
  if (!heads) {
    above = warp_add(above);
    to_k = warp_add(to_k);
    if (lane == 0) {
      S.warp_sum[warp] = above;
      S.red64[warp] = to_k;
    }
    __syncthreads();
    if (warp < 2) {
      const unsigned long long s = warp_add(lane < SM_WARPS ? (warp ? S.red64[lane] : S.warp_sum[lane]) : 0ull);
      if (lane == 0) S.sums[warp] = s;
    }
    cluster_sync();
  }
  // 4. the borders
  Entry last = {0u, SM_ALL_IDS};  // all stay
  bool fits = true;
  if (open) {
    if (!heads) {
      // (all three on their way before the first is waited for)
      const uint32_t n = lane < C ? ldu_cluster(cluster_addr(smem_addr(&S.list_n), lane)) : 0u;
      above = lane < C ? ldl_cluster(cluster_addr(smem_addr(&S.sums[0]), lane)) : 0ull;
      to_k = lane < C ? ldl_cluster(cluster_addr(smem_addr(&S.sums[1]), lane)) : 0ull;
      listed = __reduce_add_sync(FULL, n);
      above = warp_add(above);
      to_k = warp_add(to_k);
      fits = listed <= SM_LIST;
    }
    auto bin_of_key = [&](uint32_t key) { return W.bin_of(W.log2w(key_logit(key))); };
    auto borders = [&](auto src) {
      if (heads || o.k_bin < SM_BINS)
        last = src.template select<false>([&](uint32_t key, uint32_t) { return heads || bin_of_key(key) == o.k_bin; },
                                          heads ? (uint32_t)K : o.k_in);
      if (by_p) {
        const Entry kth = last;
        auto inside = [&](uint32_t key, uint32_t id) {
          const int i = bin_of_key(key);
          return (heads || i == o.k_bin || (i >= o.p_lo && i <= o.p_hi)) && stays(key, id, kth);
        };
        unsigned long long total = to_k;
        if (heads || o.k_bin < SM_BINS)
          total += src.sum([&](uint32_t key, uint32_t id) { return (heads || bin_of_key(key) == o.k_bin) && stays(key, id, kth); });
        const unsigned long long want = P > 0.f ? ceil_mul(frac64(P), total) : 0ull;
        // (bins from p_lo on hold the first element whose running sum reaches `want`, by the bounds)
        const unsigned long long more = want > above ? want - above : 1ull;
        last = src.template select<true>(
            [&](uint32_t key, uint32_t id) { return (heads || bin_of_key(key) <= o.p_hi) && inside(key, id); }, more);
        if (last.key == kth.key) last.id = min(last.id, kth.id);
      }
    };
    if (fits) {
      if (rank == 0) {  // (the others wait below)
        // warp c copies CTA c's list
        const uint32_t mine = lane < C ? ldu_cluster(cluster_addr(smem_addr(&S.list_n), lane)) : 0u;
        const uint32_t from = __reduce_add_sync(FULL, lane < warp ? mine : 0u), m = __shfl_sync(FULL, mine, warp);
        if (warp < C) {
          const uint32_t src = cluster_addr(smem_addr(&S.list[0]), warp);
          for (uint32_t i = lane; i < m; i += 32) {
            const unsigned long long e = ldl_cluster(src + i * 8);
            S.all[from + i] = {(uint32_t)e, (uint32_t)(e >> 32)};
          }
        }
        __syncthreads();
        borders(Source<DT, true>{S, (int)listed, row, W, v0, v1, C});
      }
    } else {
      borders(Source<DT, false>{S, 0, row, W, v0, v1, C});
      // the runs' sums, with the borders known
      unsigned long long sum = 0;
      row.each(v0, v1, [&](int id, float(&l)[VEC]) {
        W.fix(l);
#pragma unroll
        for (int i = 0; i < VEC; ++i)
          if (l[i] >= least && stays(logit_key(l[i]), (uint32_t)(id + i), last)) sum += W.weight(l[i]);
      });
      sum = warp_add(sum);
      if (lane == 0) S.warp_sum[warp] = sum;
      cluster_sync();
    }
  }
  // 5. the run that holds the draw
  if (rank == 0) {
    if (tid < runs) S.chunk[tid] = ldl_cluster(cluster_addr(smem_addr(&S.warp_sum[tid % SM_WARPS]), tid / SM_WARPS));
    if (open && fits) {
      __syncthreads();
      for (int i = tid; i < (int)listed; i += SM_THREADS) {
        const Entry e = S.all[i];
        const float l = key_logit(e.key);
        if (l >= least && stays(e.key, e.id & SM_ALL_IDS, last)) atomicAdd(&S.chunk[e.id >> 20], W.weight(l));
      }
      __syncthreads();
    }
    const unsigned long long mine = tid < runs ? S.chunk[tid] : 0ull;
    unsigned long long total;
    const unsigned long long before = block_before(mine, S.red64, total);
    float u = A.u[b];
    u = u > 0.f ? (u < 1.f ? u : 0x1.fffffep-1f) : 0.f;
    const unsigned long long draw = __umul64hi(frac64(u), total);  // floor(u total) < total
    if (mine && before <= draw && before + mine > draw) {
      S.end.key = last.key;
      S.end.id = last.id;
      S.end.total = total;
      S.end.rest = draw - before;
      S.end.run = tid;
    }
  }
  cluster_sync();
  last.key = ldu_cluster(cluster_addr(smem_addr(&S.end.key), 0));
  last.id = ldu_cluster(cluster_addr(smem_addr(&S.end.id), 0));
  const unsigned long long total = ldl_cluster(cluster_addr(smem_addr(&S.end.total), 0));
  unsigned long long rest = ldl_cluster(cluster_addr(smem_addr(&S.end.rest), 0));
  const int run = (int)ldu_cluster(cluster_addr(smem_addr(&S.end.run), 0));
  cluster_sync();  // (nobody's shared memory goes while another reads it)
  if (run / SM_WARPS != rank) return;
  // the run's elements, a part a thread
  auto weight_if = [&](int id, float l) -> unsigned long long {
    return l >= least && stays(logit_key(l), (uint32_t)id, last) ? W.weight(l) : 0ull;
  };
  const int r0 = row.run_begin(run, runs), nv = row.run_begin(run + 1, runs) - r0;
  const int p0 = r0 + (int)((int64_t)nv * tid / SM_THREADS), p1 = r0 + (int)((int64_t)nv * (tid + 1) / SM_THREADS);
  unsigned long long s = 0, all;
  for (int v = p0; v < p1; ++v) {
    float l[VEC];
    row.values(v, p1, l);
    W.fix(l);
#pragma unroll
    for (int i = 0; i < VEC; ++i) s += weight_if(v * VEC + i - row.off, l[i]);
  }
  if (tid == 0) S.sel_i[0] = S.sel_i[1] = 0;
  const unsigned long long at = block_before(s, S.red64, all);
  if (s && at <= rest && at + s > rest) {  // (one thread)
    S.sel_i[0] = p0;
    S.sel_i[1] = p1;
    S.sel_u[0] = rest - at;
  }
  __syncthreads();
  // its part, an element a lane (one thread alone took 16 elements' weights one after the other)
  if (warp > 0) return;
  rest = S.sel_u[0];
  const int64_t q0 = (int64_t)S.sel_i[0] * VEC, q1 = (int64_t)S.sel_i[1] * VEC;
  for (int64_t q = q0; q < q1; q += 32) {
    const int64_t x = q + lane;
    float l[1] = {x < q1 && x >= row.off && x < (int64_t)row.V + row.off ? row.one(x) : -INFINITY};
    W.fix(l);
    const unsigned long long w = weight_if((int)(x - row.off), l[0]);
    unsigned long long inc = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long y = __shfl_up_sync(FULL, inc, o);
      if (lane >= o) inc += y;
    }
    if (inc > rest && inc - w <= rest) {
      A.token[b] = (int)(x - row.off);
      // (no cancellation: both terms are <= 0)
      if (A.logp) A.logp[b] = (l[0] - W.top) / T - logf(__ull2float_rn(total) * 0x1p-43f);
    }
    inc = __shfl_sync(FULL, inc, 31);
    if (inc > rest) return;
    rest -= inc;
  }
}

const size_t SAMPLE_SMEM = sizeof(SampleSmem);

// Clusters of `c` CTAs that the current device runs at once (asked for once a device).
int rows_at_once(const void* fn, int dtype, int c, int& rows) {
  static std::atomic<int> known[64][3][5];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_status(e);
  if (dev < 0 || dev >= 64) return DDL_ERR_UNSUPPORTED;
  std::atomic<int>& k = known[dev][dtype][log2_of(c)];
  rows = k.load(std::memory_order_relaxed);
  if (rows) return DDL_OK;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)c);
  cfg.blockDim = dim3(SM_THREADS);
  cfg.dynamicSmemBytes = SAMPLE_SMEM;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)c;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if ((e = cudaOccupancyMaxActiveClusters(&rows, fn, &cfg)) != cudaSuccess) return cuda_status(e);
  k.store(rows, std::memory_order_relaxed);
  return DDL_OK;
}

}  // namespace
}  // namespace ddl

using namespace ddl;

extern "C" int ddl_sample(const void* logits, ddl_dtype dtype, int64_t stride, int32_t B, int32_t V,
                          const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                          const float* u, int32_t* token_out, float* logp_out, void* stream) {
  if (!logits || !u || !token_out) return DDL_ERR_ARG;
  if (B < 1 || V < 1 || stride < V) return DDL_ERR_ARG;
  if (dtype != DDL_T_F32 && dtype != DDL_T_BF16 && dtype != DDL_T_F16) return DDL_ERR_UNSUPPORTED;
  if (V > DDL_SAMPLE_MAX_VOCAB || B > DDL_SAMPLE_MAX_ROWS) return DDL_ERR_UNSUPPORTED;
  if ((uintptr_t)logits & (dtype == DDL_T_F32 ? 3u : 1u)) return DDL_ERR_ALIGN;
  for (const void* p : {(const void*)temperature, (const void*)top_k, (const void*)top_p, (const void*)min_p,
                        (const void*)u, (const void*)token_out, (const void*)logp_out})
    if ((uintptr_t)p & 3u) return DDL_ERR_ALIGN;
  int st;
  SampleArgs a = {logits, stride, temperature, top_p, min_p, u, top_k, token_out, logp_out, V, 1};
  const void* fn = dtype == DDL_T_F32    ? (const void*)sample_kernel<DDL_T_F32>
                   : dtype == DDL_T_BF16 ? (const void*)sample_kernel<DDL_T_BF16>
                                         : (const void*)sample_kernel<DDL_T_F16>;
  if ((st = cuda_status(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SAMPLE_SMEM)))) return st;
  if ((st = cuda_status(cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)))) return st;
  // CTAs a row: as many as let all rows run at once (of 16: 14 rows, of 8: 36, of 4: 74; 17 rows of 50257 in clusters
  // of 16, in two waves, 34.5 us with top-k 50, of 8 18.7; 256 of 128256 bf16 by two CTAs each 57, by one 40), each with
  // 2048 elements at least
  for (int c = 2; c <= SM_MAX_CLUSTER && V / c >= 2048; c *= 2) {
    int rows = 0;
    if ((st = rows_at_once(fn, dtype, c, rows))) return st;
    if (rows < B) break;
    a.cluster = c;
  }
  void* args[] = {&a};
  return cuda_status(launch_pdl_cluster(fn, dim3((unsigned)(B * a.cluster)), dim3(SM_THREADS), args, SAMPLE_SMEM, a.cluster,
                                        (cudaStream_t)stream));
}
