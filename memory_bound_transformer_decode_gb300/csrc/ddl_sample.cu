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
// Weights are integers, rn(w 2^42), and so are their sums: neither the order of
// additions nor the split over CTAs changes a bit.  An fp32 exponential would be
// wrong by 2^-23 of a weight, and a draw over V tokens meets a border within d of
// its number about V d of the time; so w comes from a table of 2^(i/256) with 2^42
// as its unit and a cubic in fp32 for the remaining factor of less than 2^(1/512), its
// argument in two floats: 2^-33 of w.  (Double precision: 152 SMs do 2 operations
// a clock each; 64 rows of 152064 would take 160 us.)
//
// A cluster of 1 to 16 CTAs takes a row; a warp a contiguous run of ids.
//  1. The maximum (greedy rows end here).
//  2. Rows with top-k or top-p: a histogram of log2 w in 2048 bins of 1/47.6 octave:
//     how many elements, and the sum of their places inside the bin, which bounds the
//     bin's sum of weights to 2^-12.  Where the k-th element and the end of the top-p
//     head may lie is then known to a bin or two.
//  3. Weights, exact: sums per warp of what certainly stays; the elements of the open
//     bins go to a list.
//  4. The list decides both borders (radix select by number, then by sum of weights,
//     ties by id), in one CTA.  Lists that overflow (all logits alike, say) are
//     replaced by the row itself: the same selection by the whole cluster.
//  5. The warps' sums, in id order, give the run that holds the draw, which its CTA
//     looks through again.
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
constexpr float SM_OCTAVES = 43.f;           // weights below 2^-43 are 0
constexpr int SM_UNIT = 42;                  // weights are multiples of 2^-42; 2^20 of them fit 62 bits
constexpr int SM_FRAC = 1024;                // places inside a bin
constexpr int SM_LIST = 4096;                // elements of a CTA's list, and of the row's
static_assert(DDL_SAMPLE_MAX_VOCAB <= 1 << 20, "sums of weights, ids in 20 bits of a list entry");

// 2^(i/256) in units of 2^-42: by repeated square roots of 2 (Newton), multiplied up, in double.
struct ExpTable {
  unsigned long long v[256];
};
constexpr ExpTable make_exp_table() {
  double root[8] = {};
  double x = 2.0;
  for (int k = 0; k < 8; ++k) {  // root[k] = 2^(1 / 2^(k + 1))
    double y = x;
    for (int n = 0; n < 60; ++n) y = 0.5 * (y + x / y);
    root[k] = y;
    x = y;
  }
  ExpTable t = {};
  for (int i = 0; i < 256; ++i) {
    double p = 1.0;
    for (int k = 0; k < 8; ++k)
      if (i & (128 >> k)) p *= root[k];
    t.v[i] = (unsigned long long)(p * 4398046511104.0 + 0.5);
  }
  return t;
}
__device__ const ExpTable g_exp_table = make_exp_table();

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
  unsigned long long table[256];
  union {
    struct {
      uint32_t count[SM_BINS], place[SM_BINS];    // histogram of the CTA's elements
      uint32_t rcount[SM_BINS], rplace[SM_BINS];  // 2048 / C bins of the cluster's
    };
    Entry all[SM_LIST];  // the row's list, when the histogram is done with
  };
  unsigned long long warp_sum[SM_WARPS];      // per warp: weights that certainly stay
  unsigned long long sums[2];                 // weights above the open bins, and between them and the k-th element's
  unsigned long long chunk[SM_MAX_CLUSTER * SM_WARPS];
  unsigned long long mass[256];
  uint32_t num[256];
  unsigned long long red64[SM_WARPS];
  float redf[SM_WARPS], redg[SM_WARPS];
  uint32_t redu[SM_WARPS];
  float top;
  int32_t top_id;
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

__device__ __forceinline__ uint32_t ldu_cluster(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
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
  const unsigned long long* table;
  // log2 of the weight, rounded: not increasing with falling logits.  NaN for what is no candidate.
  __device__ __forceinline__ float log2w(float l) const { return l == top ? 0.f : (l - top) * ch; }
  // the weight in units of 2^-42; p = log2w(l) > -43
  __device__ __forceinline__ unsigned long long weight(float l, float p) const {
    if (l == top) return 1ull << SM_UNIT;
    // l - top = d + e exactly
    const float d = l - top, b = d - l, e = (l - (d - b)) + (-top - b);
    const float lo = fmaf(d, ch, -p) + fmaf(d, cl, e * ch);
    const float k = rintf(p * 256.f);
    const float r = fmaf(-k, 0x1p-8f, p) + lo;  // p = k / 256 + r
    const int ki = (int)k;
    const unsigned long long t = table[ki & 255];
    const float z = r * 0.693147180559945f;
    const float q = z * fmaf(z, fmaf(z, 0.16666667f, 0.5f), 1.f);  // 2^r - 1
    const float tq = __uint2float_rn((uint32_t)(t >> 11)) * q;      // of t in units of 2^-31, in [2^31, 2^32)
    const long long w = (long long)t + ((long long)__float2int_rn(tq * 0x1p7f) << 4);
    const int s = -(ki >> 8);
    return ((unsigned long long)w + ((1ull << s) >> 1)) >> s;
  }
};

// The elements of a warp's run: f(id, logit) for ids in ascending order within a lane,
// 16 bytes a lane and load; the row's ends and unaligned rows element by element.
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
  __device__ __forceinline__ bool whole(int v) const { return v * VEC >= off && (int64_t)(v + 1) * VEC <= (int64_t)V + off; }
  __device__ __forceinline__ uint4 load(int v, int end) const {
    if (v < end && whole(v)) return *reinterpret_cast<const uint4*>(base + (int64_t)v * 16);
    return make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void values(int v, const uint4& x, float (&l)[VEC]) const {
    if (whole(v)) {
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
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const int64_t q = (int64_t)v * VEC + i;
        l[i] = q >= off && q < (int64_t)V + off ? one(q) : -INFINITY;
      }
    }
  }
  template <class F>
  __device__ __forceinline__ void each(int v0, int v1, F&& f) const {
    constexpr int U = 4;  // loads on their way
    const int lane = threadIdx.x & 31;
    for (int v = v0 + lane; v < v1; v += 32 * U) {
      uint4 x[U];
#pragma unroll
      for (int j = 0; j < U; ++j) x[j] = load(v + 32 * j, v1);
#pragma unroll
      for (int j = 0; j < U; ++j) {
        if (v + 32 * j >= v1) break;
        float l[VEC];
        values(v + 32 * j, x[j], l);
#pragma unroll
        for (int i = 0; i < VEC; ++i) f((v + 32 * j) * VEC + i - off, l[i]);
      }
    }
  }
};

__device__ __forceinline__ unsigned long long warp_add(unsigned long long x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(FULL, x, o);
  return x;
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

// Where the elements of a selection come from: a list in this CTA's shared memory, or the
// whole cluster's runs of the row (which of them: in()).
template <int DT, bool LIST>
struct Source {
  SampleSmem& S;
  const Entry* list;
  int n;
  const Row<DT>& row;
  const Weigher& W;
  int v0, v1, C;
  // f(key, id) for every element
  template <class F>
  __device__ __forceinline__ void each(F&& f) const {
    if (LIST) {
      for (int i = threadIdx.x; i < n; i += SM_THREADS) f(list[i].key, list[i].id & 0xfffffu);
    } else {
      row.each(v0, v1, [&](int id, float l) {
        if (W.log2w(l) > -SM_OCTAVES) f(logit_key(l), (uint32_t)id);
      });
    }
  }
  // The counts and sums of digit threadIdx.x, of all CTAs.
  __device__ __forceinline__ void gather(uint32_t& num, unsigned long long& mass) const {
    const int i = threadIdx.x;
    num = 0;
    mass = 0;
    if (LIST) {
      __syncthreads();
      if (i < 256) {
        num = S.num[i];
        mass = S.mass[i];
      }
    } else {
      cluster_sync();
      if (i < 256)
        for (int c = 0; c < C; ++c) {
          num += ldu_cluster(cluster_addr(smem_addr(&S.num[i]), c));
          mass += ldl_cluster(cluster_addr(smem_addr(&S.mass[i]), c));
        }
      cluster_sync();  // (before they are cleared)
    }
  }
  // The digit, from the top, in which the running number (BY_MASS: sum of weights) reaches `want`; what
  // lies before it is taken off `want`, the number of elements in it is left in `inside`.
  template <bool BY_MASS, bool DOWN, class F>
  __device__ __forceinline__ uint32_t digit(F&& classify, unsigned long long& want, uint32_t& inside) const {
    __syncthreads();
    for (int i = threadIdx.x; i < 256; i += SM_THREADS) {
      S.num[i] = 0;
      S.mass[i] = 0;
    }
    __syncthreads();
    each([&](uint32_t key, uint32_t id) {
      const int d = classify(key, id);
      if (d < 0) return;
      atomicAdd(&S.num[d], 1u);
      if (BY_MASS) {
        const float l = key_logit(key);
        atomicAdd(&S.mass[d], W.weight(l, W.log2w(l)));
      }
    });
    uint32_t num;
    unsigned long long mass;
    gather(num, mass);
    // place x of the order holds digit 255 - x (DOWN) or x: back through shared memory
    __syncthreads();
    if (threadIdx.x < 256) {
      S.num[threadIdx.x] = num;
      S.mass[threadIdx.x] = mass;
    }
    __syncthreads();
    const int x = DOWN ? 255 - threadIdx.x : threadIdx.x;
    num = threadIdx.x < 256 ? S.num[x] : 0u;
    unsigned long long mine = threadIdx.x < 256 ? (BY_MASS ? S.mass[x] : (unsigned long long)num) : 0ull, all;
    const unsigned long long before = block_before(mine, S.red64, all);
    if (want > all) want = all;  // (never, by the bounds of the bins)
    if (threadIdx.x == 0) {
      S.sel_i[0] = S.sel_i[1] = 0;
      S.sel_u[0] = 1;
    }
    __syncthreads();
    if (threadIdx.x < 256 && num && before < want && before + mine >= want) {
      S.sel_i[0] = x;
      S.sel_i[1] = (int)num;
      S.sel_u[0] = want - before;
    }
    __syncthreads();
    const int d = S.sel_i[0];
    inside = (uint32_t)S.sel_i[1];
    want = S.sel_u[0];
    return (uint32_t)d;
  }
  // The last element that stays of those `in` accepts: the `want`-th (BY_MASS: the first at which
  // the running sum of weights reaches `want`), in the order (key descending, id ascending).
  template <bool BY_MASS, class F>
  __device__ __forceinline__ Entry select(F&& in, unsigned long long want) const {
    Entry e = {0u, 0u};
    uint32_t inside = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
      const uint32_t hi = shift == 24 ? 0u : ~0u << (shift + 8);
      e.key |= digit<BY_MASS, true>(
                   [&](uint32_t key, uint32_t id) {
                     return in(key, id) && ((key ^ e.key) & hi) == 0 ? (int)((key >> shift) & 255u) : -1;
                   },
                   want, inside)
               << shift;
    }
    if (BY_MASS) {  // elements of one key weigh the same
      const float l = key_logit(e.key);
      const unsigned long long w = W.weight(l, W.log2w(l));
      want = w ? (want + w - 1) / w : 1;
      want = want < inside ? want : inside;
    }
    for (int shift = 16; shift >= 0; shift -= 8) {
      const uint32_t hi = shift == 16 ? 0u : ~0u << (shift + 8);
      e.id |= digit<false, false>(
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
    unsigned long long s = 0, all;
    each([&](uint32_t key, uint32_t id) {
      if (in(key, id)) {
        const float l = key_logit(key);
        s += W.weight(l, W.log2w(l));
      }
    });
    block_before(s, S.red64, all);
    if (!LIST) {
      if (threadIdx.x == 0) S.sel_u[1] = all;
      cluster_sync();
      all = 0;
      for (int c = 0; c < C; ++c) all += ldl_cluster(cluster_addr(smem_addr(&S.sel_u[1]), c));
      cluster_sync();
    }
    return all;
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

struct Open {     // what the histogram says of the row's borders
  int k_bin;      // bin of the k-th element (SM_BINS: none)
  uint32_t k_in;  // its place among the bin's elements, from 1
  int p_lo, p_hi; // bins in which the top-p head may end (p_lo > p_hi: no top-p)
};

template <int DT>
__global__ void __launch_bounds__(SM_THREADS, 2) sample_kernel(const __grid_constant__ SampleArgs A) {
  extern __shared__ __align__(16) uint8_t sample_smem[];
  SampleSmem& S = *reinterpret_cast<SampleSmem*>(sample_smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = A.cluster, b = blockIdx.x / C, rank = blockIdx.x % C, runs = C * SM_WARPS;
  for (int i = tid; i < 256; i += SM_THREADS) S.table[i] = g_exp_table.v[i];
  pdl_trigger();
  pdl_wait();
  const Row<DT> row(A, b);
  const int v0 = row.run_begin(rank * SM_WARPS + warp, runs), v1 = row.run_begin(rank * SM_WARPS + warp + 1, runs);
  const float T = A.temperature ? A.temperature[b] : 1.f;
  const bool greedy = !(T >= 0x1p-60f);
  // 1. the maximum, and its lowest id
  float top = -INFINITY;
  int top_id = 0x7fffffff;
  row.each(v0, v1, [&](int id, float l) {
    if (l > top) {
      top = l;
      top_id = id;
    }
  });
  auto better = [](float l, int i, float& m, int& mi) {
    if (l > m || (l == m && i < mi)) {
      m = l;
      mi = i;
    }
  };
#pragma unroll
  for (int o = 16; o; o >>= 1) better(__shfl_xor_sync(FULL, top, o), __shfl_xor_sync(FULL, top_id, o), top, top_id);
  if (lane == 0) {
    S.redf[warp] = top;
    S.redu[warp] = (uint32_t)top_id;
  }
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < SM_WARPS; ++w) better(S.redf[w], (int)S.redu[w], top, top_id);
    S.top = top;
    S.top_id = top_id;
    S.list_n = 0;
  }
  for (int i = tid; i < SM_BINS; i += SM_THREADS) S.count[i] = S.place[i] = 0;
  cluster_sync();
  top = -INFINITY;
  top_id = 0x7fffffff;
  for (int c = 0; c < C; ++c)
    better(ld_cluster(cluster_addr(smem_addr(&S.top), c)), (int)ldu_cluster(cluster_addr(smem_addr(&S.top_id), c)), top, top_id);
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
  {
    const double c = 1.4426950408889634 / (double)T;
    W.top = top;
    W.ch = (float)c;
    W.cl = (float)(c - (double)W.ch);
    W.table = S.table;
  }
  const int32_t K = A.top_k ? A.top_k[b] : 0;
  const float P = A.top_p ? A.top_p[b] : 1.f, M = A.min_p ? A.min_p[b] : 0.f;
  const bool by_k = K > 0 && K < A.V, by_p = P < 1.f;
  // min-p as a bound on the logit (T below infinity: the weights of all are 1 otherwise)
  double least = -INFINITY;
  if (M > 0.f) least = M >= 1.f ? (double)top : (double)T < INFINITY ? (double)top + (double)T * log((double)M) : -INFINITY;
  // log2 w to bins, from the top
  auto bin_of = [&](float p) { return min((int)(-p * SM_PER_OCTAVE), SM_BINS - 1); };

  // 2. the histogram
  Open o = {SM_BINS, 0u, SM_BINS, -1};
  if (by_k || by_p) {
    row.each(v0, v1, [&](int, float l) {
      const float p = W.log2w(l);
      if (p > -SM_OCTAVES) {
        const float x = -p * SM_PER_OCTAVE;
        const int i = min((int)x, SM_BINS - 1);
        atomicAdd(&S.count[i], 1u);
        if (by_p) atomicAdd(&S.place[i], (uint32_t)((x - (float)i) * SM_FRAC));
      }
    });
    cluster_sync();
    const int per = SM_BINS / C;
    for (int i = tid; i < per; i += SM_THREADS) {
      uint32_t n = 0, q = 0;
      for (int c = 0; c < C; ++c) {
        n += ldu_cluster(cluster_addr(smem_addr(&S.count[rank * per + i]), c));
        if (by_p) q += ldu_cluster(cluster_addr(smem_addr(&S.place[rank * per + i]), c));
      }
      S.rcount[i] = n;
      S.rplace[i] = q;
    }
    cluster_sync();
    // every CTA: the bins' numbers and bounds of their sums of weights; thread i has bins 4 i .. 4 i + 3
    constexpr int PER = SM_BINS / SM_THREADS;
    uint32_t n[PER], sum = 0, all_n;
    float lo[PER], hi[PER], slo = 0.f, shi = 0.f, all_lo, all_hi;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int i = tid * PER + j, c = i / per, at = i - c * per;
      n[j] = ldu_cluster(cluster_addr(smem_addr(&S.rcount[at]), c));
      lo[j] = by_p ? (float)ldu_cluster(cluster_addr(smem_addr(&S.rplace[at]), c)) : 0.f;
      sum += n[j];
    }
    uint32_t before = block_before(sum, S.redu, all_n);
    if (tid == 0) {
      S.sel_i[0] = SM_BINS;
      S.sel_i[1] = 0;
      S.sel_i[2] = SM_BINS;
      S.sel_i[3] = SM_BINS;
    }
    __syncthreads();
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
      // A bin's sum: n 2^-(i + mean place) / 47.6, the mean place between the sum of the rounded-down places
      // and 1 / 1024 more, the curvature inside a bin at most (ln 2 / 47.6)^2 / 8 = 2.7e-5 more, and the places'
      // own rounding (log2 w up to 43 in fp32: 2^-12 of a bin).  Of the k-th element's bin, k_in elements of any place.
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const int i = tid * PER + j;
        const float cnt = (float)n[j];
        if (i > o.k_bin || n[j] == 0) {
          lo[j] = hi[j] = 0.f;
        } else if (i == o.k_bin) {
          lo[j] = (float)o.k_in * exp2f(-(float)(i + 1) / SM_PER_OCTAVE) * 0.9999f;
          hi[j] = (float)o.k_in * exp2f(-(float)i / SM_PER_OCTAVE) * 1.0001f;
        } else {
          const float mean = lo[j] / (cnt * SM_FRAC);
          const float w = cnt * exp2f(-((float)i + mean) / SM_PER_OCTAVE);
          lo[j] = w * 0.9999f;  // (1 / 1024 of a bin: 1.4e-5)
          hi[j] = w * 1.0001f;
          if (i == SM_BINS - 1) lo[j] = 0.f;
        }
        slo += lo[j];
        shi += hi[j];
      }
      float blo = block_before(slo, S.redf, all_lo), bhi = block_before(shi, S.redg, all_hi);
      // sums of 2048 fp32 numbers: within 1e-4 (2^-24 each addition)
      const float want_lo = P * all_lo * 0.9998f, want_hi = P * all_hi * 1.0002f;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const int i = tid * PER + j;
        blo += lo[j];
        bhi += hi[j];
        if (n[j] && i <= o.k_bin && bhi >= want_lo) atomicMin(&S.sel_i[2], i);
        if (n[j] && i <= o.k_bin && blo >= want_hi) atomicMin(&S.sel_i[3], i);
      }
      __syncthreads();
      o.p_lo = min(S.sel_i[2], SM_BINS - 1);
      o.p_hi = min(min(S.sel_i[3], o.k_bin), SM_BINS - 1);
      if (o.p_lo > o.p_hi) o.p_lo = o.p_hi;
    }
    __syncthreads();
  }

  // 3. exact sums of what certainly stays, the list of the open bins
  // (bins above p_lo, without top-p above k_bin: stay; between p_hi and k_bin: count for top-p's total only)
  const int sure = by_p ? o.p_lo : o.k_bin;
  unsigned long long above = 0, chosen = 0, between = 0;
  row.each(v0, v1, [&](int id, float l) {
    const float p = W.log2w(l);
    if (!(p > -SM_OCTAVES)) return;
    const int i = bin_of(p);
    if (i > o.k_bin) return;
    if (i == o.k_bin || (i >= o.p_lo && i <= o.p_hi)) {
      const uint32_t at = atomicAdd(&S.list_n, 1u);
      if (at < SM_LIST) S.list[at] = {logit_key(l), (uint32_t)id | ((uint32_t)(rank * SM_WARPS + warp) << 20)};
      return;
    }
    const unsigned long long w = W.weight(l, p);
    if (i < sure) {
      above += w;
      if ((double)l >= least) chosen += w;
    } else {
      between += w;
    }
  });
  above = warp_add(above);
  chosen = warp_add(chosen);
  between = warp_add(between);
  if (lane == 0) {
    S.warp_sum[warp] = chosen;
    S.red64[warp] = above;
    S.mass[warp] = between;
  }
  __syncthreads();
  if (tid < 2) {
    unsigned long long s = 0;
    for (int w = 0; w < SM_WARPS; ++w) s += tid ? S.mass[w] : S.red64[w];
    S.sums[tid] = s;
  }
  cluster_sync();
  // 4. the borders
  uint32_t listed = 0;
  for (int c = 0; c < C; ++c) listed += ldu_cluster(cluster_addr(smem_addr(&S.list_n), c));
  above = between = 0;
  for (int c = 0; c < C; ++c) {
    above += ldl_cluster(cluster_addr(smem_addr(&S.sums[0]), c));
    between += ldl_cluster(cluster_addr(smem_addr(&S.sums[1]), c));
  }
  Entry last = {0u, 0xffffffffu};  // all stay
  const bool open = o.k_bin < SM_BINS || by_p, fits = listed <= SM_LIST;
  auto bin_of_key = [&](uint32_t key) { return bin_of(W.log2w(key_logit(key))); };
  auto borders = [&](auto src) {
    if (o.k_bin < SM_BINS)
      last = src.template select<false>([&](uint32_t key, uint32_t) { return bin_of_key(key) == o.k_bin; }, o.k_in);
    if (by_p) {
      const Entry kth = last;
      auto inside = [&](uint32_t key, uint32_t id) {
        const int i = bin_of_key(key);
        return (i == o.k_bin || (i >= o.p_lo && i <= o.p_hi)) && stays(key, id, kth);
      };
      const unsigned long long total = above + between + src.sum(inside);
      const unsigned long long want = P > 0.f ? ceil_mul(frac64(P), total) : 0ull;
      // (bins from p_lo on hold the first element whose running sum reaches `want`, by the bounds)
      unsigned long long more = want > above ? want - above : 1ull;
      last = src.template select<true>(
          [&](uint32_t key, uint32_t id) { return bin_of_key(key) <= o.p_hi && inside(key, id); }, more);
    }
  };
  if (open && fits) {
    if (rank == 0) {  // (the others wait below)
      int n = 0;
      for (int c = 0; c < C; ++c) {
        const int m = (int)ldu_cluster(cluster_addr(smem_addr(&S.list_n), c));
        const uint32_t from = cluster_addr(smem_addr(&S.list[0]), c);
        for (int i = tid; i < m; i += SM_THREADS) {
          const unsigned long long e = ldl_cluster(from + i * 8);
          S.all[n + i] = {(uint32_t)e, (uint32_t)(e >> 32)};
        }
        n += m;
      }
      __syncthreads();
      borders(Source<DT, true>{S, S.all, n, row, W, v0, v1, C});
      listed = n;
    }
  } else if (open) {
    borders(Source<DT, false>{S, nullptr, 0, row, W, v0, v1, C});
    // the runs' sums, with the borders known
    unsigned long long s = 0;
    row.each(v0, v1, [&](int id, float l) {
      const float p = W.log2w(l);
      if (p > -SM_OCTAVES && stays(logit_key(l), (uint32_t)id, last) && (double)l >= least) s += W.weight(l, p);
    });
    s = warp_add(s);
    if (lane == 0) S.warp_sum[warp] = s;
    cluster_sync();
  }
  // 5. the run that holds the draw
  if (rank == 0) {
    for (int i = tid; i < runs; i += SM_THREADS)
      S.chunk[i] = ldl_cluster(cluster_addr(smem_addr(&S.warp_sum[i % SM_WARPS]), i / SM_WARPS));
    __syncthreads();
    if (open && fits) {
      for (int i = tid; i < (int)listed; i += SM_THREADS) {
        const Entry e = S.all[i];
        const float l = key_logit(e.key);
        if (stays(e.key, e.id & 0xfffffu, last) && (double)l >= least) atomicAdd(&S.chunk[e.id >> 20], W.weight(l, W.log2w(l)));
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
  {
    last.key = ldu_cluster(cluster_addr(smem_addr(&S.end.key), 0));
    last.id = ldu_cluster(cluster_addr(smem_addr(&S.end.id), 0));
    const unsigned long long total = ldl_cluster(cluster_addr(smem_addr(&S.end.total), 0));
    unsigned long long rest = ldl_cluster(cluster_addr(smem_addr(&S.end.rest), 0));
    const int run = (int)ldu_cluster(cluster_addr(smem_addr(&S.end.run), 0));
    cluster_sync();  // (nobody's shared memory goes while another reads it)
    if (run / SM_WARPS != rank) return;
    // the run's elements, a part a warp
    auto weight_if = [&](int id, float l) -> unsigned long long {
      const float p = W.log2w(l);
      return p > -SM_OCTAVES && stays(logit_key(l), (uint32_t)id, last) && (double)l >= least ? W.weight(l, p) : 0ull;
    };
    const int r0 = row.run_begin(run, runs), r1 = row.run_begin(run + 1, runs);
    const int p0 = r0 + (int)((int64_t)(r1 - r0) * warp / SM_WARPS), p1 = r0 + (int)((int64_t)(r1 - r0) * (warp + 1) / SM_WARPS);
    unsigned long long s = 0;
    row.each(p0, p1, [&](int id, float l) { s += weight_if(id, l); });
    s = warp_add(s);
    if (lane == 0) S.red64[warp] = s;
    __syncthreads();
    unsigned long long before = 0;
    for (int w = 0; w < warp; ++w) before += S.red64[w];
    if (!(before <= rest && before + s > rest)) return;
    rest -= before;
    constexpr int VEC = Row<DT>::VEC;
    for (int v = p0; v < p1; v += 32) {
      unsigned long long w[VEC], sum = 0;
      float l[VEC];
      const bool has = v + lane < p1;
      if (has) row.values(v + lane, row.load(v + lane, p1), l);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        w[i] = has ? weight_if((v + lane) * VEC + i - row.off, l[i]) : 0ull;
        sum += w[i];
      }
      unsigned long long inc = sum;
#pragma unroll
      for (int k = 1; k < 32; k <<= 1) {
        const unsigned long long y = __shfl_up_sync(FULL, inc, k);
        if (lane >= k) inc += y;
      }
      unsigned long long at = inc - sum;
      if (sum && at <= rest && inc > rest) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          if (w[i] && at <= rest && at + w[i] > rest) {
            A.token[b] = (v + lane) * VEC + i - row.off;
            if (A.logp) {
              const double x = l[i] == top ? 0.0 : ((double)l[i] - (double)top) / (double)T;
              A.logp[b] = (float)(x - log((double)total * 0x1p-42));
            }
          }
          at += w[i];
        }
      }
      const unsigned long long whole = __shfl_sync(FULL, inc, 31);
      if (whole > rest) break;
      rest -= whole;
    }
  }
}

const size_t SAMPLE_SMEM = sizeof(SampleSmem);

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
  int sms = 0, st;
  if ((st = device_sms(sms))) return st;
  SampleArgs a = {logits, stride, temperature, top_p, min_p, u, top_k, token_out, logp_out, V, 1};
  // CTAs a row: as many as the machine holds at once (two an SM), each with 2048 elements at least
  while (a.cluster < SM_MAX_CLUSTER && (int64_t)B * a.cluster * 2 <= 2 * sms && V / (a.cluster * 2) >= 2048) a.cluster *= 2;
  const void* fn = dtype == DDL_T_F32    ? (const void*)sample_kernel<DDL_T_F32>
                   : dtype == DDL_T_BF16 ? (const void*)sample_kernel<DDL_T_BF16>
                                         : (const void*)sample_kernel<DDL_T_F16>;
  if ((st = cuda_status(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SAMPLE_SMEM)))) return st;
  if (a.cluster > 8 && (st = cuda_status(cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1))))
    return st;
  void* args[] = {&a};
  return cuda_status(launch_pdl_cluster(fn, dim3((unsigned)(B * a.cluster)), dim3(SM_THREADS), args, SAMPLE_SMEM, a.cluster,
                                        (cudaStream_t)stream));
}
