// ddl_kv8_score.cu -- the attention weight that each token of the 8-bit paged
// cache has drawn (ddl_kv8_score).
//
// With the log-sum-exp that the attention of the same rows returned, a key's
// weight needs no other key: w_ij = exp(s_ij - lse_i), so
//     score_j = decay score_j + sum over rows i and heads of the K/V head of w_ij
// is one pass over K alone, without a join: each token's sum belongs to one
// warp, in a fixed order of rows and heads, and no atomics are needed.
//
// A warp takes 16 tokens (one scale block) x 8 queries at a time, as the
// attention's warp kernel does: S^T = K Q^T on m16n8k16 MMAs with the tokens as
// M, the head dimensions in an order that lets lane (g, t) load 16 neighbouring
// bytes of rows g and g + 8; e4m3 and int8 codes are exact in fp16, Q is scaled
// by a power of two per query and split into fp16 high part and (fp32 rows)
// remainder.  A token's weights lie in the four lanes of its row: two shuffles
// after the last query.
//
// What bounds it: K's bytes for many requests (64 of up to 8192 tokens, 64/8 heads: 53 us, 78 % of the copy rate, issue
// slots at 52 %); one request, launch and the chain lengths - page - codes (1 of 32769 int8, fp32 rows: 11 us of which
// the bytes are 5).
#include <cuda_bf16.h>

#include "ddl_kv8_score.h"

namespace ddl {
namespace {

constexpr int SC_MAX_BLOCKS = 12;  // blocks of 16 tokens a warp takes at most (a lane each)

// Weights exp(score - lse) of tokens key, key + 8 (c 0, 1 and 2, 3) for two queries: c are the MMA's sums.
// All lanes of the warp call it.
template <bool EX>
__device__ __forceinline__ void weights(const AttArgs& A, float (&c)[4], const Column& x, const Column& y, float ks,
                                        int key, bool edge) {
  const float fx = ks * x.cf, fy = ks * y.cf;
  if (!EX) {
    c[0] = exp2_fast(fmaf(c[0], fx, -x.lse2));
    c[1] = exp2_fast(fmaf(c[1], fy, -y.lse2));
    c[2] = exp2_fast(fmaf(c[2], fx, -x.lse2));
    c[3] = exp2_fast(fmaf(c[3], fy, -y.lse2));
  } else {
    c[0] *= fx;
    c[1] *= fy;
    c[2] *= fx;
    c[3] *= fy;
    if (A.softcap > 0.f) {
      tanh_of(c);
      const float cap = A.softcap * LOG2E;
#pragma unroll
      for (int j = 0; j < 4; ++j) c[j] *= cap;
    }
    c[0] = exp2_fast(fmaf(-x.slope, (float)(x.hi - key), c[0]) - x.lse2);
    c[1] = exp2_fast(fmaf(-y.slope, (float)(y.hi - key), c[1]) - y.lse2);
    c[2] = exp2_fast(fmaf(-x.slope, (float)(x.hi - key - 8), c[2]) - x.lse2);
    c[3] = exp2_fast(fmaf(-y.slope, (float)(y.hi - key - 8), c[3]) - y.lse2);
  }
  if (edge) {
    c[0] = key <= x.hi && key >= x.lo ? c[0] : 0.f;
    c[1] = key <= y.hi && key >= y.lo ? c[1] : 0.f;
    c[2] = key + 8 <= x.hi && key + 8 >= x.lo ? c[2] : 0.f;
    c[3] = key + 8 <= y.hi && key + 8 >= y.lo ? c[3] : 0.f;
  }
}

// The CTA's part of the tokens of request r for K/V head h: blocks c0 .. c0 + W wb, block
// c0 + warp + W i being this warp's i-th.
template <int W>
struct Part {
  Req rq;
  int r, h, c0, nb, first, mine;  // first block that changes, blocks of this warp
  int32_t place;                  // lane i: of this warp's block i among all heads' blocks of the pool (-1: nobody sees it)
  float scale;
  float* out;
  // False: nothing to do for the CTA.
  __device__ __forceinline__ bool load(const ScoreArgs& S) {
    const AttArgs& A = S.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    r = blockIdx.z;
    h = blockIdx.y;
    rq = load_req(A, r);
    if (rq.bad && A.bad && blockIdx.x == 0 && h == 0 && threadIdx.x == 0) atomicOr(A.bad, 1);
    if (rq.n <= 0) return false;
    nb = (rq.len + 15) >> 4;
    c0 = blockIdx.x * W * S.wb;
    first = S.decay == 1.f ? rq.b0 : 0;  // blocks before rq.b0 only decay
    if (c0 >= nb || c0 + W * S.wb <= first) return false;
    mine = c0 + warp < nb ? min(S.wb, (nb - c0 - warp + W - 1) / W) : 0;
    place = -1;
    scale = 0.f;
    if (lane < mine) {
      const int b = block(lane), bshift = A.pshift - 4;
      if (b >= rq.b0 && b < rq.b1) {
        const int32_t page = A.table[(int64_t)r * A.per + (b >> bshift)];
        if (page >= 0 && page < A.pages) {
          place = (int32_t)((((int64_t)page * A.Hkv + h) << bshift) + (b & ((1 << bshift) - 1)));
          scale = A.ks[place];  // (looked at where it is used, when the codes are on their way)
        } else if (A.bad) {
          atomicOr(A.bad, 1);
        }
      }
    }
    out = S.score + ((int64_t)r * A.Hkv + h) * S.stride;
    return true;
  }
  __device__ __forceinline__ int block(int i) const { return c0 + (int)(threadIdx.x >> 5) + W * i; }
  // the score that token `key` brings along
  __device__ __forceinline__ float old(const ScoreArgs& S, int key) const {
    return key < rq.p0 && key < rq.len && S.decay != 0.f ? out[key] : 0.f;
  }
  __device__ __forceinline__ void put(const ScoreArgs& S, int key, float was, float sum) const {
    if (key < rq.len) out[key] = fmaf(S.decay, was, sum);
  }
};

// A block's K codes in a lane: 16 bytes of rows g and g + 8 for each 64 of a row.
template <int HD>
struct KBlock {
  static constexpr int NV = HD / 64;
  uint4 v[2][NV];
  template <int CT>
  __device__ __forceinline__ void frag(int s, uint32_t (&a)[4]) const {
    const uint4 x = v[0][s / 4], y = v[1][s / 4];
    const uint32_t wx = (s & 3) == 0 ? x.x : (s & 3) == 1 ? x.y : (s & 3) == 2 ? x.z : x.w;
    const uint32_t wy = (s & 3) == 0 ? y.x : (s & 3) == 1 ? y.y : (s & 3) == 2 ? y.z : y.w;
    codes_f16<CT>(wx, a[0], a[2]);
    codes_f16<CT>(wy, a[1], a[3]);
  }
  static __device__ __forceinline__ const uint8_t* piece(const uint8_t* k, int32_t blk, int j) {
    const int lane = threadIdx.x & 31;
    return k + (int64_t)blk * (16 * HD) + ((lane >> 2) + (j / NV) * 8) * HD + (lane & 3) * 16 + (j % NV) * 64;
  }
};

// Fragments of the query of this lane's column g of tile `tile`, and its power of two.
template <int DT, int HD>
struct QTile {
  static constexpr int KS = HD / 16;
  static constexpr bool HL = DT == DDL_T_F32;
  uint32_t hi[KS][2], lo[HL ? KS : 1][2];
  float qf;
  __device__ __forceinline__ void load(const AttArgs& A, const Req& rq, int h, int tile, int lane) {
    const int qi = tile * 8 + (lane >> 2), t = lane & 3;
    const bool has = qi < rq.n * A.GH;
    const int row = has ? group_row(A, qi) : 0;
    const int64_t at = (int64_t)(rq.row0 + row) * A.q_stride + (int64_t)(h * A.GH + (has ? qi : 0) - row * A.GH) * HD + t * 16;
    float4 f[KS];
    float mx = 0.f;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      f[s] = has ? load_elem4<DT>(A.q, at + 64 * (s >> 2) + 4 * (s & 3)) : make_float4(0.f, 0.f, 0.f, 0.f);
      mx = fmaxf(mx, fmaxf(fmaxf(fabsf(f[s].x), fabsf(f[s].y)), fmaxf(fabsf(f[s].z), fabsf(f[s].w))));
    }
    mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 2));
    int e = (int)((__float_as_uint(mx) >> 23) & 255u) - 127 - 12;  // the largest lands in [2^12, 2^13)
    e = e < -100 ? -100 : e > 115 ? 115 : e;
    const float down = __uint_as_float((uint32_t)(127 - e) << 23);
    qf = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const float4 v = make_float4(f[s].x * down, f[s].y * down, f[s].z * down, f[s].w * down);
      hi[s][0] = pack_f16x2(v.x, v.y);
      hi[s][1] = pack_f16x2(v.z, v.w);
      if (HL) {
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&hi[s][0]));
        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi[s][1]));
        lo[HL ? s : 0][0] = pack_f16x2(v.x - a.x, v.y - a.y);
        lo[HL ? s : 0][1] = pack_f16x2(v.z - b.x, v.w - b.y);
      }
    }
  }
};

__device__ __forceinline__ void reduce_rows(float& s0, float& s1) {  // over the four lanes of a row
  s0 += __shfl_xor_sync(FULL, s0, 1);
  s1 += __shfl_xor_sync(FULL, s1, 1);
  s0 += __shfl_xor_sync(FULL, s0, 2);
  s1 += __shfl_xor_sync(FULL, s1, 2);
}

// Fragments and columns of several tiles in shared memory.
template <int DT, int HD>
struct TileSmem {
  static constexpr int KS = HD / 16, PARTS = DT == DDL_T_F32 ? 2 : 1;
  uint2* frags;  // [tile][part][k-step][lane]
  Column* cols;  // [tile][8]
  __device__ __forceinline__ TileSmem(uint8_t* p, int tiles)
      : frags(reinterpret_cast<uint2*>(p)), cols(reinterpret_cast<Column*>(p + (size_t)tiles * PARTS * KS * 32 * 8)) {}
  // tiles t0 .. t0 + nt - 1, a warp each
  template <bool EX>
  __device__ __forceinline__ void load(const AttArgs& A, const Req& rq, int h, int t0, int nt, int warps) const {
    const int lane = threadIdx.x & 31;
    for (int x = threadIdx.x >> 5; x < nt; x += warps) {
      QTile<DT, HD> q;
      q.load(A, rq, h, t0 + x, lane);
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        frags[((x * PARTS) * KS + s) * 32 + lane] = make_uint2(q.hi[s][0], q.hi[s][1]);
        if (PARTS == 2)
          frags[((x * PARTS + 1) * KS + s) * 32 + lane] =
              make_uint2(q.lo[PARTS == 2 ? s : 0][0], q.lo[PARTS == 2 ? s : 0][1]);
      }
      if ((lane & 3) == 0) cols[x * 8 + (lane >> 2)] = column_of<EX>(A, rq, h, (t0 + x) * 8 + (lane >> 2), q.qf);
    }
  }
};

// Requests of a few tiles of queries (8 rows x heads each).  Each warp's codes go through a ring of its own in
// shared memory: a lane copies its own pieces (cp.async) and reads them back, without a barrier.  ONE: a single
// tile, whose fragments stay in registers (remainders of fp32 rows in shared memory); else they lie in
// shared memory, behind the ring.
template <int HD>
struct Ring {
  static constexpr int STAGES = 4, STAGE = 16 * HD, BYTES = 8 * STAGES * STAGE;  // of 8 warps
};

template <int CT, int DT, int HD, bool EX, bool ONE>
__global__ void __launch_bounds__(256, 3) kv8_score_few_kernel(const __grid_constant__ ScoreArgs S) {
  constexpr int W = 8, KS = HD / 16, NV = HD / 64, PARTS = DT == DDL_T_F32 ? 2 : 1;
  constexpr bool HL = DT == DDL_T_F32;
  using Rg = Ring<HD>;
  extern __shared__ __align__(16) uint8_t sc_smem[];
  const AttArgs& A = S.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  pdl_trigger();
  pdl_wait();
  Part<W> part;
  if (!part.load(S)) return;
  const Req& rq = part.rq;
  const int nq = rq.n * A.GH;
  const uint32_t ring = smem_addr(sc_smem) + warp * Rg::STAGES * Rg::STAGE + lane * 16;
  auto fetch = [&](int i) {
    const int32_t blk = i < SC_MAX_BLOCKS ? __shfl_sync(FULL, part.place, i) : -1;
    if (blk >= 0) {  // (none past the last)
      const uint32_t dst = ring + (i % Rg::STAGES) * Rg::STAGE;
#pragma unroll
      for (int j = 0; j < 2 * NV; ++j) cp_async16(dst + j * 512, KBlock<HD>::piece(A.k, blk, j));
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < Rg::STAGES - 1; ++i) fetch(i);
  // the token of this lane (t 0: g, t 1: g + 8) of block i, and its old score two blocks ahead
  auto key_of = [&](int i) { return part.block(i) * 16 + g + (t == 1 ? 8 : 0); };
  auto old_of = [&](int i) { return t < 2 && i < part.mine ? part.old(S, key_of(i)) : 0.f; };
  float was = old_of(0), next = old_of(1);
  const TileSmem<DT, HD> tile(sc_smem + Rg::BYTES, S.tiles);
  uint2* const lo = tile.frags + warp * KS * 32;  // ONE: the warp's own
  QTile<DT, HD> q;
  Column col[2];
  if (ONE) {
    q.load(A, rq, part.h, 0, lane);
    if (HL) {
#pragma unroll
      for (int s = 0; s < KS; ++s) lo[s * 32 + lane] = make_uint2(q.lo[HL ? s : 0][0], q.lo[HL ? s : 0][1]);
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) col[c] = column_of<EX>(A, rq, part.h, 2 * t + c, __shfl_sync(FULL, q.qf, 4 * (2 * t + c)));
  } else {
    tile.template load<EX>(A, rq, part.h, 0, (nq + 7) >> 3, W);
    __syncthreads();
  }
#pragma unroll 1
  for (int i = 0; i < part.mine; ++i) {
    fetch(i + Rg::STAGES - 1);
    const float ahead = old_of(i + 2);
    const int32_t at = __shfl_sync(FULL, part.place, i);
    float ks = __shfl_sync(FULL, part.scale, i);
    if (!(fabsf(ks) < INFINITY)) ks = __uint_as_float(0x7fffffffu);
    const int key0 = part.block(i) * 16;
    float s0 = 0.f, s1 = 0.f;
    cp_async_wait<Rg::STAGES - 1>();
    if (at >= 0) {
      KBlock<HD> k;
      const uint32_t src = ring + (i % Rg::STAGES) * Rg::STAGE;
#pragma unroll
      for (int j = 0; j < 2 * NV; ++j) k.v[j / NV][j % NV] = lds128(src + j * 512);
      uint32_t a[KS][4];
#pragma unroll
      for (int s = 0; s < KS; ++s) k.template frag<CT>(s, a[s]);
#pragma unroll 1
      for (int x = 0; x < (ONE ? 1 : (nq + 7) >> 3); ++x) {
        const int q0 = x * 8, q1 = min(q0 + 7, nq - 1);
        if (!ONE && (key0 > rq.p0 + group_row(A, q1) || key0 + 15 < first_seen(A, rq, q0))) continue;  // nobody sees it
        float c[4] = {0.f, 0.f, 0.f, 0.f}, c2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const uint2 b = ONE ? make_uint2(q.hi[s][0], q.hi[s][1]) : tile.frags[(x * PARTS * KS + s) * 32 + lane];
          mma_f16((s & 1) ? c2 : c, a[s][0], a[s][1], a[s][2], a[s][3], b.x, b.y);
          if (HL) {
            const uint2 b2 = ONE ? lo[s * 32 + lane] : tile.frags[((x * PARTS + 1) * KS + s) * 32 + lane];
            mma_f16((s & 1) ? c2 : c, a[s][0], a[s][1], a[s][2], a[s][3], b2.x, b2.y);
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) c[j] += c2[j];
        // blocks that every query sees, in full tiles, need no masks
        const Column &cx = ONE ? col[0] : tile.cols[q0 + 2 * t], &cy = ONE ? col[1] : tile.cols[q0 + 2 * t + 1];
        const bool edge = q0 + 7 >= nq || key0 + 15 > rq.p0 + group_row(A, q0) || key0 < first_seen(A, rq, q1) ||
                          (cx.hi | cy.hi) < 0;
        weights<EX>(A, c, cx, cy, ks, key0 + g, edge);
        s0 += c[0] + c[1];
        s1 += c[2] + c[3];
      }
      reduce_rows(s0, s1);
    }
    if (t < 2 && part.block(i) >= part.first) part.put(S, key_of(i), was, t ? s1 : s0);
    was = next;
    next = ahead;
  }
}

// Tiles of the ring kernel at most, which passes over the queries' fragments once a block; more go to the tcgen05 kernel, whose
// time grows little with them.  Ring and tcgen05, 1 request of 8192 with 64/8 heads, 16 of up to 2048 and 64 of up to 4096 with
// 32/4: bf16, 4 tiles 8.7 and 11.7 us, 8.0 and 19.5, 35 and 74; 8: 10.4 and 12.3, 12.8 and 19.9, 59 and 74; 12: 13.8 and 13.0,
// 18.2 and 25.4, 74 and 77; 16: 16.9 and 13.6, 21.5 and 20.4, 87 and 76.  fp32, 4: 9.0 and 11.9, 11.2 and 19.3, 49 and 77;
// 8: 13.7 and 12.8, 16.9 and 19.8, 77 and 78; 12: 29 and 13.7, 28 and 25.7, 137 and 83 (one CTA an SM).
constexpr int FEW_16 = 8, FEW_F32 = 4;

enum { ONE_TILE, FEW_TILES, MANY_TILES };
template <int CT, int DT, int HD>
const void* score_fn(bool ex, int kind) {
  if (kind == ONE_TILE)
    return ex ? (const void*)kv8_score_few_kernel<CT, DT, HD, true, true> : (const void*)kv8_score_few_kernel<CT, DT, HD, false, true>;
  return ex ? (const void*)kv8_score_few_kernel<CT, DT, HD, true, false> : (const void*)kv8_score_few_kernel<CT, DT, HD, false, false>;
}
template <int CT>
const void* score_fn(int dt, int hd, bool ex, int kind) {
  if (hd == 128)
    return dt == DDL_T_F32    ? score_fn<CT, DDL_T_F32, 128>(ex, kind)
           : dt == DDL_T_BF16 ? score_fn<CT, DDL_T_BF16, 128>(ex, kind)
                              : score_fn<CT, DDL_T_F16, 128>(ex, kind);
  return dt == DDL_T_F32    ? score_fn<CT, DDL_T_F32, 64>(ex, kind)
         : dt == DDL_T_BF16 ? score_fn<CT, DDL_T_BF16, 64>(ex, kind)
                            : score_fn<CT, DDL_T_F16, 64>(ex, kind);
}
// Bytes of a tile's fragments and columns.
int tile_bytes(bool f32, int hd) { return (f32 ? 2 : 1) * hd / 16 * 32 * 8 + 8 * (int)sizeof(Column); }

}  // namespace
}  // namespace ddl

using namespace ddl;

extern "C" int ddl_kv8_score(const ddl_kv8* kv, int32_t H_q, int32_t H_kv, int32_t head_dim, ddl_dtype dtype,
                             const ddl_attn_opts* opts, int32_t R, int32_t T, int32_t max_rows, int32_t max_len,
                             const int32_t* q_off, const int32_t* kv_len, const int32_t* page_table,
                             int32_t pages_per_seq, const void* q, int64_t q_stride, const float* lse, float decay,
                             float* score, int64_t score_stride, int32_t* bad_out, void* stream) {
  int st = check_kv8(kv, H_kv, head_dim);
  if (st) return st;
  if (H_q < H_kv || H_q % H_kv || H_q / H_kv > DDL_MAX_GROUP_HEADS) return DDL_ERR_SHAPE;
  if (R < 1 || T < 1 || max_rows < 1 || max_len < 1 || pages_per_seq < 1) return DDL_ERR_ARG;
  if (R > DDL_KV8_MAX_REQS || max_rows > DDL_KV8_MAX_ROWS) return DDL_ERR_UNSUPPORTED;
  if (!opts || !kv_len || !page_table || !q || !lse || !score) return DDL_ERR_ARG;
  if (!dtype_bytes(dtype)) return DDL_ERR_UNSUPPORTED;
  if (!q_off && (max_rows != 1 || T < R)) return DDL_ERR_ARG;
  if ((int64_t)pages_per_seq * kv->page_size > 0x7fffffffLL) return DDL_ERR_UNSUPPORTED;
  if ((st = check_attn_opts(opts))) return st;
  if (!(decay >= 0.f && decay <= 1.f) || score_stride < max_len) return DDL_ERR_ARG;
  if (q_stride < (int64_t)H_q * head_dim || q_stride % 8) return DDL_ERR_ARG;
  if (!aligned16(q)) return DDL_ERR_ALIGN;
  for (const void* p : {(const void*)q_off, (const void*)kv_len, (const void*)page_table, (const void*)lse,
                        (const void*)score, (const void*)bad_out})
    if ((uintptr_t)p & 3u) return DDL_ERR_ALIGN;
  int sms = 0;
  if ((st = device_sms(sms))) return st;
  ScoreArgs s;
  memset(&s, 0, sizeof s);
  AttArgs& a = s.a;
  a.k = kv->k;
  a.ks = kv->k_scale;
  a.q_off = q_off;
  a.kv_len = kv_len;
  a.table = page_table;
  a.q = q;
  a.lse = const_cast<float*>(lse);  // (only read)
  a.bad = bad_out;
  a.slopes = opts->slopes;
  a.pages = kv->pages;
  a.q_stride = q_stride;
  a.scale = opts->scale;
  a.softcap = fminf(opts->softcap, 0x1p100f);  // (a score over more than that would be subnormal)
  a.window = opts->window >= max_len ? 0 : opts->window;  // (a window as long as the bound hides nothing)
  a.R = R;
  a.T = T;
  a.Hq = H_q;
  a.Hkv = H_kv;
  a.GH = H_q / H_kv;
  a.gmul = (65536 + a.GH - 1) / a.GH;
  a.hd = head_dim;
  a.pshift = log2_of(kv->page_size);
  a.per = pages_per_seq;
  a.max_rows = max_rows;
  a.max_len = max_len;
  s.score = score;
  s.stride = score_stride;
  s.decay = decay;
  const int tiles = (max_rows * a.GH + 7) / 8, per = tile_bytes(dtype == DDL_T_F32, head_dim);
  const bool f32 = dtype == DDL_T_F32, ex = opts->softcap > 0.f || opts->slopes;
  const int kind = tiles == 1 ? ONE_TILE : tiles <= (f32 ? FEW_F32 : FEW_16) ? FEW_TILES : MANY_TILES;
  const int64_t blocks = ((int64_t)max_len + 15) / 16, units = (int64_t)R * H_kv;
  if (kind == MANY_TILES) {
    s.wait_ns = wait_limit_ns();
    return kv8_score_tc_launch(s, kv->type, dtype, ex, sms, stream);
  }
  // A CTA begins with a chain of dependent loads (lengths, page, scale, codes) and its queries: as many blocks a warp as
  // leave one wave of CTAs (ragged lengths come to about 5/8 of the bound), but no more than 12, so that long
  // requests spread.  Blocks a warp 2 / 4 / 8 / 12 / 16: 64 requests of up to 8192, 64/8 heads 86 / 64 / 55 / 53 / 55 us, 16 of up
  // to 4096 13.8 / 11.8 / 10.1 / 13.0 / 15.1, 1 of 8192 5.4 / 5.8 / 6.7 / 8.5 / 9.7.
  constexpr int warps = 8;
  s.tiles = tiles;
  const size_t ring = (size_t)(head_dim == 128 ? Ring<128>::BYTES : Ring<64>::BYTES);
  const size_t smem = ring + (kind == FEW_TILES ? (size_t)tiles * per : f32 ? (size_t)8 * head_dim / 16 * 32 * 8 : 0);
  const int64_t ctas = sms * (smem > 74 * 1024 ? 2 : 3) * (R > 1 ? 8 : 5) / 5;
  const int64_t each = ctas / units > 1 ? ctas / units : 1, wb = (blocks + warps * each - 1) / (warps * each);
  s.wb = (int32_t)(wb < SC_MAX_BLOCKS ? wb : SC_MAX_BLOCKS);
  const int64_t chunks = (blocks + warps * s.wb - 1) / (warps * s.wb);
  const void* fn = kv->type == DDL_KV8_E4M3 ? score_fn<DDL_KV8_E4M3>(dtype, head_dim, ex, kind)
                                            : score_fn<DDL_KV8_INT8>(dtype, head_dim, ex, kind);
  // (the function's limit, which calls of other threads set too: the most that any call of it takes)
  const size_t most = kind == FEW_TILES ? ring + (size_t)(f32 ? FEW_F32 : FEW_16) * per : smem;
  if ((st = cuda_status(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most)))) return st;
  void* args[] = {&s};
  return cuda_status(launch_pdl(fn, dim3((unsigned)chunks, (unsigned)H_kv, (unsigned)R), dim3((unsigned)warps * 32), args,
                                smem, (cudaStream_t)stream));
}
