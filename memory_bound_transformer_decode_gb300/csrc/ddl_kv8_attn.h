// ddl_kv8_attn.h -- what the two attention kernels over the 8-bit cache (warp
// MMAs, tcgen05) and the kernel that joins their records share: arguments,
// requests, the split into shares, elements of rows.
#pragma once
#include <cuda.h>

#include "ddl_kv8.h"

namespace ddl {

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

struct AttArgs {
  const uint8_t *k, *v;
  const float *ks, *vs;
  const int32_t *q_off, *kv_len, *table;
  const void* q;
  void* out;
  float* lse;
  int32_t* bad;
  float *rec_o, *rec_ml;  // records [share + unit][query of the unit][hd], [..][2]
  int64_t* prefix;        // [R + 1] blocks of all units before each request
  const float* slopes;
  int64_t pages, q_stride, out_stride;
  float scale, softcap;
  int32_t window;
  int32_t R, T, Hq, Hkv, GH, gmul, hd, pshift, per, max_rows, max_len;
  int32_t cluster;  // > 0: a cluster of so many CTAs a unit; 0: shares
  int32_t ctas;     // CTAs: of the clusters, or shares at most
  int32_t unit_cost, min_share;
  int32_t hp;       // K/V heads of a CTA (a power of two, nq hp <= 8; 1 but for whole units of the warp kernel)
  int32_t nq, nqc;  // query tiles of 8 a unit has (a power of two <= 8), units over a request's query tiles
};

// Shares.  Beginning and ending a unit (Q, the join of the warps, the record)
// costs a CTA about as much as unit_cost of its blocks, so a unit of nb blocks
// weighs unit_cost + nb, its block j standing at unit_cost + j; the weights of
// all units, end to end, are cut (range_lo, owner_of) into equal parts of at
// least min_share.
__device__ __forceinline__ int64_t share_count(const AttArgs& A, int64_t W) {
  const int64_t most = W < (1ll << 31) ? ((uint32_t)W + A.min_share - 1) / (uint32_t)A.min_share
                                       : (W + A.min_share - 1) / A.min_share;
  return most < 1 ? 1 : most < A.ctas ? most : A.ctas;
}
__device__ __forceinline__ void share_bounds(int64_t W, int64_t n, int64_t& x, int64_t& end) {
  if (W < (1 << 22)) {  // (32-bit divisions: n <= 1024)
    x = (uint32_t)W * blockIdx.x / (uint32_t)n;
    end = (uint32_t)W * (blockIdx.x + 1) / (uint32_t)n;
  } else {
    x = range_lo(W, n, blockIdx.x);
    end = range_lo(W, n, blockIdx.x + 1);
  }
}

// A request's rows and keys as the kernels compute them (clamped to what the
// launch and the tables allow).
struct Req {
  int32_t row0, n, len;  // first row of q, rows, tokens
  int32_t p0;            // position of its first row (negative: it has no keys)
  int32_t b0, b1;        // blocks of 16 tokens that any of its rows sees: [b0, b1)
  bool bad;
};
__device__ __forceinline__ Req load_req(const AttArgs& A, int r) {
  Req q;
  int64_t row0 = r, n = 1;
  if (A.q_off) {
    row0 = A.q_off[r];
    n = (int64_t)A.q_off[r + 1] - row0;
  }
  int64_t len = A.kv_len[r];
  const int64_t cap = (int64_t)A.per << A.pshift;
  q.bad = false;
  // rows outside [0, T) are left out, the others keep their positions: `skip`
  // rows before the first one that is computed, `n` from there to the newest
  int64_t skip = 0, take = n;
  if (row0 < 0 || n < 0 || row0 + n > A.T) {
    q.bad = true;
    skip = row0 < 0 ? -row0 : 0;
    take = (row0 + n < A.T ? row0 + n : A.T) - (row0 + skip);
    if (take <= 0) skip = n = take = 0;
    row0 = take > 0 ? row0 + skip : 0;
    n -= skip;
  }
  if (len < 0 || len > A.max_len || len > cap) {
    q.bad = true;
    len = len < 0 ? 0 : len;
    len = len > A.max_len ? A.max_len : len;
    len = len > cap ? cap : len;
  }
  q.row0 = (int32_t)row0;
  q.len = (int32_t)len;
  const int64_t p0 = len - n;  // (n < 2^32 where rows lie outside)
  q.p0 = (int32_t)(p0 < -(1 << 30) ? -(1 << 30) : p0);  // (so far from any key as its first 64 rows)
  int64_t lo = A.window > 0 ? len - n - A.window + 1 : 0;
  lo = lo < 0 ? 0 : lo;
  if (take > A.max_rows) {
    q.bad = true;
    take = A.max_rows;  // its first rows
  }
  n = take;
  q.n = (int32_t)n;
  q.b0 = (int32_t)(lo >> 4);
  q.b1 = n > 0 ? (int32_t)((len + 15) >> 4) : q.b0;
  if (q.b1 < q.b0) q.b1 = q.b0;
  return q;
}

// Units of request q: K/V heads times groups of query tiles.
__device__ __forceinline__ int unit_groups(const AttArgs& A, const Req& q) {
  return (q.n * A.GH + 8 * A.nq - 1) / (8 * A.nq);
}

// A scale that is not finite, or negative for V: NaN for the rows that see one of
// the block's tokens, through their scores, and nothing for the others (V's, as a
// weight's factor or in the units of O, would reach every row of the tile).
__device__ __forceinline__ void check_scales(float& ks, float& vs) {
  if (fabsf(ks) < INFINITY && vs >= 0.f && vs < INFINITY) return;
  vs = 0.f;
  ks = __uint_as_float(0x7fffffffu);
}
// The weights' reference.  A key contributes p_j vs_j code_j, p_j = e^{s_j - ..}.
// What a weight loses when it is rounded to the MMA's type is measured by the
// largest product p_j vs_j of the *query*, so that neither a block that other
// queries of the tile see nor a seen one of small weight costs it bits:
//  - O and the products are in units of vref, the power of two at or below the
//    largest V scale met in a block that some query sees (a unit only);
//  - per query the running reference is R = max_j (s_j + log2(vs_j / vref)) over
//    the keys it sees (base 2), p_j = 2^(s_j - R): the largest product is about 1,
//    and p_j itself above 1 where its block's scale lies below vref;
//  - p_j stays below 2^P_TOP and the logarithm is taken as -P_SPAN at least, so
//    that the sum of p_j is finite: blocks whose scale is down to 2^-P_SPAN of vref
//    keep all bits, smaller ones lose them gradually.
constexpr float P_SPAN = 90.f, P_TOP = 95.f;
constexpr float VREF_MIN = 0x1p-126f;          // (its inverse is finite)
// Power of two at or below a scale, at least VREF_MIN.
__device__ __forceinline__ float pow2_floor(float vs) {
  const uint32_t e = __float_as_uint(vs) & 0x7f800000u;
  return e < 0x00800000u ? VREF_MIN : __uint_as_float(e);
}
// 1 / x of a power of two in [2^-126, 2^127], log2 of the quotient of two.
__device__ __forceinline__ float pow2_inv(float x) {
  const uint32_t e = __float_as_uint(x);
  return e == 0x7f000000u ? 0x1p-127f : __uint_as_float(0x7f000000u - e);
}
__device__ __forceinline__ float pow2_log_ratio(float a, float b) {
  return (float)((int)(__float_as_uint(a) >> 23) - (int)(__float_as_uint(b) >> 23));
}
// log2 of a block's scale over vref.
__device__ __forceinline__ float scale_log(float vs_over_ref) { return fmaxf(__log2f(vs_over_ref), -P_SPAN); }

// Byte mask of the e4m3 NaN codes (low 7 bits all set) of four codes.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  const uint32_t top = ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
  return (top >> 7) * 255u;
}

// Row of a request that its query qi (row * group + head of the group) belongs to: qi / GH, qi < 512.
__device__ __forceinline__ int group_row(const AttArgs& A, int qi) { return (int)((uint32_t)qi * (uint32_t)A.gmul >> 16); }
// First token that the request's query qi sees (a window may reach back past any 32-bit number).
__device__ __forceinline__ int64_t first_seen(const AttArgs& A, const Req& q, int qi) {
  return A.window > 0 ? (int64_t)q.p0 + group_row(A, qi) - A.window + 1 : 0;
}
// Weight of request q's units.
__device__ __forceinline__ int64_t req_weight(const AttArgs& A, const Req& q) {
  const int nb = q.b1 - q.b0;
  return nb > 0 ? (int64_t)(nb + A.unit_cost) * A.Hkv * unit_groups(A, q) : 0;
}

// Weights before each request into pre[0 .. R] (every CTA adds them up: R <=
// 4096 lengths from L2); returns their sum.  CTA 0 leaves them for the join
// and reports bad requests.  wsum: a word per warp.
template <int NT>
__device__ __forceinline__ int64_t unit_prefix(const AttArgs& A, int64_t* pre, int64_t* wsum) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int64_t base = 0;
  for (int r0 = 0; r0 < A.R; r0 += NT) {
    const int r = r0 + tid;
    int64_t w = 0;
    if (r < A.R) {
      const Req rq = load_req(A, r);
      w = req_weight(A, rq);
      if (blockIdx.x == 0 && rq.bad && A.bad) atomicOr(A.bad, 1);
    }
    int64_t inc = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(FULL, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    int64_t before = base, all = 0;
#pragma unroll
    for (int v = 0; v < NT / 32; ++v) {
      if (v < warp) before += wsum[v];
      all += wsum[v];
    }
    if (r < A.R) pre[r] = before + inc - w;
    base += all;
    __syncthreads();
  }
  if (tid == 0) pre[A.R] = base;
  __syncthreads();
  if (blockIdx.x == 0)
    for (int r = tid; r <= A.R; r += NT) A.prefix[r] = pre[r];
  return base;
}

// The unit of request q (weights from p0 on) at weight x and the run of its
// blocks up to `end`: unit, first block, count; moves x past it.  False if the
// run has no blocks.
__device__ __forceinline__ bool share_segment(const AttArgs& A, const Req& q, int64_t p0, int64_t& x, int64_t end,
                                              int& unit, int& first, int& count) {
  const int nb = q.b1 - q.b0, w = nb + A.unit_cost;
  const int64_t in = x - p0;
  unit = in < (1ll << 31) ? (int)((uint32_t)in / (uint32_t)w) : (int)(in / w);
  const int at = (int)(in - (int64_t)unit * w);
  const int to = end - x < w - at ? at + (int)(end - x) : w;
  const int b0 = at > A.unit_cost ? at - A.unit_cost : 0, b1 = to > A.unit_cost ? to - A.unit_cost : 0;
  first = q.b0 + b0;
  count = b1 - b0;
  x += to - at;
  return count > 0;
}

// Four neighbouring elements (8- or 16-byte aligned).
template <int DT>
__device__ __forceinline__ float4 load_elem4(const void* p, int64_t i) {
  if (DT == DDL_T_F32) return *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + i);
  const uint2 u = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(p) + i);
  if (DT == DDL_T_BF16) return make_float4(bf16lo_f32(u.x), bf16hi_f32(u.x), bf16lo_f32(u.y), bf16hi_f32(u.y));
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
  return make_float4(a.x, a.y, b.x, b.y);
}
template <int DT>
__device__ __forceinline__ void store_elem4(void* p, int64_t i, float4 v) {
  if (DT == DDL_T_F32) {
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + i) = v;
  } else {
    uint2 u;
    if (DT == DDL_T_BF16) u = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    else u = make_uint2(pack_f16x2(v.x, v.y), pack_f16x2(v.z, v.w));
    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p) + i) = u;
  }
}

template <int DT>
__device__ __forceinline__ void store_elem(void* p, int64_t i, float v) {
  if (DT == DDL_T_F32) reinterpret_cast<float*>(p)[i] = v;
  else if (DT == DDL_T_BF16) reinterpret_cast<uint16_t*>(p)[i] = f32_to_bf16_bits(v);
  else reinterpret_cast<__half*>(p)[i] = __float2half_rn(v);
}

// ------------------------------------------------------------------ clusters
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, int rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  return a;
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// A CTA of a cluster and its run of the unit's blocks.
struct ClusterPart {
  int unit, rank;  // unit: ((request * H_kv) + head) * nqc + group of tiles
  __device__ __forceinline__ explicit ClusterPart(const AttArgs& A) {
    unit = blockIdx.x / A.cluster;
    rank = blockIdx.x - unit * A.cluster;
  }
  __device__ __forceinline__ void blocks(const AttArgs& A, const Req& q, int& c0, int& c1) const {
    const int64_t nb = q.b1 - q.b0;
    c0 = q.b0 + (int)(nb * rank / A.cluster);
    c1 = q.b0 + (int)(nb * (rank + 1) / A.cluster);
  }
};

// Joins the records that the unit's CTAs hold in shared memory (query x: O at
// rec + (x / 8) tile_stride + (x % 8) HD floats, (max, sum) at ml + 8 x bytes):
// CTA `rank` takes every cluster-th query, a thread one head dimension, the
// CTAs' values in rank order.  All threads of the cluster call it.
template <int DT, int HD>
__device__ __forceinline__ void cluster_join(const AttArgs& A, const ClusterPart& part, uint32_t rec,
                                             uint32_t tile_stride, uint32_t ml, int threads) {
  cluster_sync();
  int u = part.unit;
  const int qc = u % A.nqc;
  u /= A.nqc;
  const int h = u % A.Hkv, r = u / A.Hkv, nq8 = A.nq * 8, S = A.cluster;
  const Req rq = load_req(A, r);
  const int d = threadIdx.x % HD, step = S * (threads / HD);
  if ((int)threadIdx.x < threads)
    for (int x = part.rank + S * (threadIdx.x / HD); x < nq8; x += step) {
      const int qi = qc * nq8 + x;
      if (qi >= rq.n * A.GH) break;
      const uint32_t ro = rec + (x >> 3) * tile_stride + ((x & 7) * HD + d) * 4, rm = ml + x * 8;
      float m = -INFINITY, l = 0.f, acc = 0.f;
      for (int k0 = 0; k0 < S; k0 += 8) {
        float mk[8], lk[8], ok[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const bool in = k0 + k < S;
          const uint32_t am = cluster_addr(rm, in ? k0 + k : 0), ao = cluster_addr(ro, in ? k0 + k : 0);
          mk[k] = in ? ld_cluster(am) : -INFINITY;
          lk[k] = in ? ld_cluster(am + 4) : 0.f;
          ok[k] = in ? ld_cluster(ao) : 0.f;
        }
        float nm = m;
#pragma unroll
        for (int k = 0; k < 8; ++k) nm = fmaxf(nm, mk[k]);
        const float ref = nm == -INFINITY ? 0.f : nm, f0 = exp2_fast(m - ref);
        l *= f0;
        acc *= f0;
        m = nm;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float f = exp2_fast(mk[k] - ref);
          l = fmaf(f, lk[k], l);
          acc = fmaf(f, ok[k], acc);
        }
      }
      const int row = group_row(A, qi), head = h * A.GH + qi - row * A.GH;
      const float inv = l != 0.f ? 1.f / l : 0.f;  // (NaN stays NaN)
      store_elem<DT>(A.out, (int64_t)(rq.row0 + row) * A.out_stride + (int64_t)head * HD + d, acc * inv);
      if (d == 0 && A.lse) A.lse[(int64_t)(rq.row0 + row) * A.Hq + head] = (m + log2f(l)) * LN2;
    }
  cluster_sync();  // (nobody's shared memory goes while another reads it)
}

// A dependent launch of a grid of clusters.
inline cudaError_t launch_pdl_cluster(const void* fn, dim3 grid, dim3 block, void** args, size_t smem, int cluster,
                                      cudaStream_t s) {
  if (cluster <= 1) return launch_pdl(fn, grid, block, args, smem, s);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelExC(&cfg, fn, args);
}

// The tcgen05 kernel (e4m3, head_dim 128): rows of the pool's view < 2^31.
int kv8_tc_launch(const AttArgs& a, int dtype, int64_t rows, void* stream);
// Its CTAs an SM, by their shared memory; `reqs` requests' weights beside it (shares), 0: none.
int kv8_tc_ctas(int nq, bool f32, int reqs);

}  // namespace ddl
