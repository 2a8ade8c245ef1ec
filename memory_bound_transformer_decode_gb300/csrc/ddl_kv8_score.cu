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
#include <cuda_bf16.h>

#include "ddl_kv8_attn.h"

namespace ddl {
namespace {

constexpr int SC_WARPS = 8;

struct ScoreArgs {
  AttArgs a;
  float* score;    // [R][H_kv][stride]
  int64_t stride;
  float decay;
  int32_t wb;      // blocks of 16 tokens a warp takes (<= 32)
};

// What the queries of a tile need apart from their fragments.
struct Column {
  float cf;       // factor of the MMA's sum (times the block's scale): log2 units, or softcap's argument
  float lse2;     // log2 e times lse; +inf for a query without keys
  float slope;    // log2 units a token
  int hi, lo;     // last and first token it sees
};

// Query qi of request rq for K/V head h.
template <bool EX>
__device__ __forceinline__ Column column_of(const AttArgs& A, const Req& rq, int h, int qi, float qf, float lse) {
  Column c;
  const bool has = qi < rq.n * A.GH;
  const int row = has ? group_row(A, qi) : 0;
  const int64_t p = (int64_t)rq.p0 + row, lo = A.window > 0 ? p - A.window + 1 : 0;
  c.hi = has ? (int)p : -1;
  c.lo = lo > 0 ? (int)lo : 0;
  c.slope = EX && A.slopes && has ? A.slopes[h * A.GH + qi - row * A.GH] * LOG2E : 0.f;
  c.cf = qf * A.scale;
  if (EX && A.softcap > 0.f) c.cf = __fdiv_rn(c.cf, A.softcap);
  else c.cf *= LOG2E;
  c.lse2 = lse == -INFINITY ? INFINITY : lse * LOG2E;
  return c;
}

// exp of a score (MMA sum `s`, block scale `ks`) less its query's lse.
template <bool EX>
__device__ __forceinline__ float weight_of(const AttArgs& A, const Column& c, float s, float ks, int key) {
  if (!EX) return exp2_fast(fmaf(s, ks * c.cf, -c.lse2));
  const float x = s * (ks * c.cf);
  const float y = A.softcap > 0.f ? A.softcap * LOG2E * tanhf(x) : x;
  return exp2_fast(fmaf(-c.slope, (float)(c.hi - key), y) - c.lse2);
}

// 16 bytes of row g (and g + 8) of a block, one load per 64 bytes of the row.
template <int HD>
struct KBlock {
  static constexpr int NV = HD / 64;
  uint4 v[2][NV];
  __device__ __forceinline__ void load(const uint8_t* k, int32_t blk, int lane) {
    const uint8_t* p = k + (int64_t)blk * (16 * HD) + (lane >> 2) * HD + (lane & 3) * 16;
#pragma unroll
    for (int j = 0; j < 2 * NV; ++j)
      v[j / NV][j % NV] = *reinterpret_cast<const uint4*>(p + (j / NV) * 8 * HD + (j % NV) * 64);
  }
  template <int CT>
  __device__ __forceinline__ void frag(int s, uint32_t (&a)[4]) const {
    const uint4 x = v[0][s / 4], y = v[1][s / 4];
    const uint32_t wx = (s & 3) == 0 ? x.x : (s & 3) == 1 ? x.y : (s & 3) == 2 ? x.z : x.w;
    const uint32_t wy = (s & 3) == 0 ? y.x : (s & 3) == 1 ? y.y : (s & 3) == 2 ? y.z : y.w;
    codes_f16<CT>(wx, a[0], a[2]);
    codes_f16<CT>(wy, a[1], a[3]);
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

// Shared memory of the kernel for several tiles: their fragments (and remainders) and columns.
template <int DT, int HD>
struct TileSmem {
  static constexpr int KS = HD / 16, PARTS = DT == DDL_T_F32 ? 2 : 1;
  static constexpr int PER = PARTS * KS * 32 * 8 + 8 * (int)sizeof(Column);  // bytes a tile
};
constexpr int TILE_SMEM = 142 * 1024;  // 64 tiles of 16-bit rows of 128

// One CTA: 8 wb blocks of a request's tokens for one K/V head.
//   ONE: the request has one tile of queries (8 rows x heads), whose fragments stay in
//   registers; else the tiles' fragments go through shared memory, smem_tiles at a time.
template <int CT, int DT, int HD, bool EX, bool ONE>
__global__ void __launch_bounds__(SC_WARPS * 32, ONE ? 3 : 1) kv8_score_kernel(const __grid_constant__ ScoreArgs S,
                                                                               int smem_tiles) {
  extern __shared__ __align__(16) uint8_t sc_smem[];
  __shared__ float sums[ONE ? 1 : SC_WARPS * 32 * 16];
  const AttArgs& A = S.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int r = blockIdx.z, h = blockIdx.y;
  constexpr int KS = HD / 16;
  pdl_trigger();
  pdl_wait();
  const Req rq = load_req(A, r);
  if (rq.bad && A.bad && blockIdx.x == 0 && h == 0 && threadIdx.x == 0) atomicOr(A.bad, 1);
  if (rq.n <= 0) return;
  const int nb = (rq.len + 15) >> 4, c0 = blockIdx.x * SC_WARPS * S.wb;
  const int first = S.decay == 1.f ? rq.b0 : 0;  // blocks before rq.b0 only decay
  if (c0 >= nb || c0 + SC_WARPS * S.wb <= first) return;
  // block i of this warp: c0 + warp + 8 i; lane l holds the place and scale of block l
  auto block_of = [&](int i) { return c0 + warp + SC_WARPS * i; };
  const int mine = c0 + warp < nb ? min(S.wb, (nb - c0 - warp + SC_WARPS - 1) / SC_WARPS) : 0;
  int32_t place = -1;
  float scale = 0.f;
  if (lane < mine) {
    const int b = block_of(lane), bshift = A.pshift - 4;
    if (b >= rq.b0 && b < rq.b1) {
      const int32_t page = A.table[(int64_t)r * A.per + (b >> bshift)];
      if (page >= 0 && page < A.pages) {
        place = (int32_t)((((int64_t)page * A.Hkv + h) << bshift) + (b & ((1 << bshift) - 1)));
        scale = A.ks[place];
        if (!(fabsf(scale) < INFINITY)) scale = __uint_as_float(0x7fffffffu);
      } else if (A.bad) {
        atomicOr(A.bad, 1);
      }
    }
  }
  float* const out = S.score + ((int64_t)r * A.Hkv + h) * S.stride;
  // score of token `key` from the sum of its weights
  auto put = [&](int key, float sum) {
    if (key >= rq.len) return;
    const float old = key < rq.p0 && S.decay != 0.f ? out[key] : 0.f;
    out[key] = fmaf(S.decay, old, sum);
  };
  // weights of one block for one tile: tokens g and g + 8
  auto tile_sum = [&](const float (&c)[4], const Column& x, const Column& y, float ks, int key0, bool edge, float& s0,
                      float& s1) {
    float w[4];
    w[0] = weight_of<EX>(A, x, c[0], ks, key0 + g);
    w[1] = weight_of<EX>(A, y, c[1], ks, key0 + g);
    w[2] = weight_of<EX>(A, x, c[2], ks, key0 + g + 8);
    w[3] = weight_of<EX>(A, y, c[3], ks, key0 + g + 8);
    if (edge) {
      w[0] = key0 + g <= x.hi && key0 + g >= x.lo ? w[0] : 0.f;
      w[1] = key0 + g <= y.hi && key0 + g >= y.lo ? w[1] : 0.f;
      w[2] = key0 + g + 8 <= x.hi && key0 + g + 8 >= x.lo ? w[2] : 0.f;
      w[3] = key0 + g + 8 <= y.hi && key0 + g + 8 >= y.lo ? w[3] : 0.f;
    }
    s0 += w[0] + w[1];
    s1 += w[2] + w[3];
  };
  const int nq = rq.n * A.GH, tiles = (nq + 7) >> 3;
  if (ONE) {
    QTile<DT, HD> q;
    q.load(A, rq, h, 0, lane);
    Column col[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int qi = 2 * t + c, row = qi < nq ? group_row(A, qi) : 0;
      const float lse = qi < nq ? A.lse[(int64_t)(rq.row0 + row) * A.Hq + h * A.GH + qi - row * A.GH] : 0.f;
      col[c] = column_of<EX>(A, rq, h, qi, __shfl_sync(FULL, q.qf, 4 * qi), lse);
    }
    // tokens that every query sees: blocks inside need no masks
    const int all_hi = nq == 8 ? rq.p0 : -1;
    const int64_t lo64 = first_seen(A, rq, nq - 1);
    KBlock<HD> k, n;
    int32_t blk = __shfl_sync(FULL, place, 0);
    if (blk >= 0) n.load(A.k, blk, lane);
    for (int i = 0; i < mine; ++i) {
      const int32_t at = blk;
      k = n;
      blk = i + 1 < 32 ? __shfl_sync(FULL, place, (i + 1) & 31) : -1;
      if (blk >= 0) n.load(A.k, blk, lane);
      const int key0 = block_of(i) * 16;
      const float ks = __shfl_sync(FULL, scale, i);
      float s0 = 0.f, s1 = 0.f;
      if (at >= 0) {
        float c[4] = {0.f, 0.f, 0.f, 0.f}, c2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          uint32_t a[4];
          k.template frag<CT>(s, a);
          mma_f16((s & 1) ? c2 : c, a[0], a[1], a[2], a[3], q.hi[s][0], q.hi[s][1]);
          if (QTile<DT, HD>::HL)
            mma_f16((s & 1) ? c2 : c, a[0], a[1], a[2], a[3], q.lo[QTile<DT, HD>::HL ? s : 0][0],
                    q.lo[QTile<DT, HD>::HL ? s : 0][1]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) c[j] += c2[j];
        const bool edge = key0 + 15 > all_hi || key0 < lo64;
        tile_sum(c, col[0], col[1], ks, key0, edge, s0, s1);
        s0 += __shfl_xor_sync(FULL, s0, 1);
        s1 += __shfl_xor_sync(FULL, s1, 1);
        s0 += __shfl_xor_sync(FULL, s0, 2);
        s1 += __shfl_xor_sync(FULL, s1, 2);
      }
      if (block_of(i) < first) continue;
      if (t == 0) put(key0 + g, s0);
      if (t == 1) put(key0 + g + 8, s1);
    }
  } else {
    constexpr int PARTS = TileSmem<DT, HD>::PARTS;
    uint2* const frags = reinterpret_cast<uint2*>(sc_smem);  // [tile][part][k-step][lane]
    Column* const cols = reinterpret_cast<Column*>(sc_smem + (size_t)smem_tiles * PARTS * KS * 32 * 8);
    for (int i = threadIdx.x; i < SC_WARPS * S.wb * 16; i += SC_WARPS * 32) sums[ONE ? 0 : i] = 0.f;
    for (int t0 = 0; t0 < tiles; t0 += smem_tiles) {
      const int nt = min(smem_tiles, tiles - t0);
      __syncthreads();
      for (int x = warp; x < nt; x += SC_WARPS) {
        QTile<DT, HD> q;
        q.load(A, rq, h, t0 + x, lane);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          frags[((x * PARTS) * KS + s) * 32 + lane] = make_uint2(q.hi[s][0], q.hi[s][1]);
          if (PARTS == 2)
            frags[((x * PARTS + 1) * KS + s) * 32 + lane] =
                make_uint2(q.lo[PARTS == 2 ? s : 0][0], q.lo[PARTS == 2 ? s : 0][1]);
        }
        if (t == 0) {
          const int qi = (t0 + x) * 8 + g, row = qi < nq ? group_row(A, qi) : 0;
          const float lse = qi < nq ? A.lse[(int64_t)(rq.row0 + row) * A.Hq + h * A.GH + qi - row * A.GH] : 0.f;
          cols[x * 8 + g] = column_of<EX>(A, rq, h, qi, q.qf, lse);
        }
      }
      __syncthreads();
      for (int i = 0; i < mine; ++i) {
        const int32_t at = __shfl_sync(FULL, place, i);
        if (at < 0) continue;
        const int key0 = block_of(i) * 16;
        const float ks = __shfl_sync(FULL, scale, i);
        KBlock<HD> k;
        k.load(A.k, at, lane);
        uint32_t a[KS][4];
#pragma unroll
        for (int s = 0; s < KS; ++s) k.template frag<CT>(s, a[s]);
        float s0 = 0.f, s1 = 0.f;
        for (int x = 0; x < nt; ++x) {
          const int q0 = (t0 + x) * 8, q1 = min(q0 + 7, nq - 1);
          const int last = rq.p0 + group_row(A, q1);
          const int64_t from = first_seen(A, rq, q0);
          if (key0 > last || key0 + 15 < from) continue;  // no query of the tile sees the block
          float c[4] = {0.f, 0.f, 0.f, 0.f}, c2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int s = 0; s < KS; ++s) {
            const uint2 b = frags[((x * PARTS) * KS + s) * 32 + lane];
            mma_f16((s & 1) ? c2 : c, a[s][0], a[s][1], a[s][2], a[s][3], b.x, b.y);
            if (PARTS == 2) {
              const uint2 b2 = frags[((x * PARTS + 1) * KS + s) * 32 + lane];
              mma_f16((s & 1) ? c2 : c, a[s][0], a[s][1], a[s][2], a[s][3], b2.x, b2.y);
            }
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) c[j] += c2[j];
          const bool edge = q0 + 7 >= nq || key0 + 15 > rq.p0 + group_row(A, q0) || key0 < first_seen(A, rq, q1);
          tile_sum(c, cols[x * 8 + 2 * t], cols[x * 8 + 2 * t + 1], ks, key0, edge, s0, s1);
        }
        s0 += __shfl_xor_sync(FULL, s0, 1);
        s1 += __shfl_xor_sync(FULL, s1, 1);
        s0 += __shfl_xor_sync(FULL, s0, 2);
        s1 += __shfl_xor_sync(FULL, s1, 2);
        float* const mysum = sums + (ONE ? 0 : (warp + SC_WARPS * i) * 16);
        if (t == 0) mysum[g] += s0;
        if (t == 1) mysum[g + 8] += s1;
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < SC_WARPS * S.wb * 16; i += SC_WARPS * 32)
      if (c0 + (i >> 4) >= first) put(c0 * 16 + i, sums[ONE ? 0 : i]);
  }
}

template <int CT, int DT, int HD>
const void* score_fn(bool ex, bool one) {
  if (one) return ex ? (const void*)kv8_score_kernel<CT, DT, HD, true, true> : (const void*)kv8_score_kernel<CT, DT, HD, false, true>;
  return ex ? (const void*)kv8_score_kernel<CT, DT, HD, true, false> : (const void*)kv8_score_kernel<CT, DT, HD, false, false>;
}
template <int CT>
const void* score_fn(int dt, int hd, bool ex, bool one) {
  if (hd == 128)
    return dt == DDL_T_F32    ? score_fn<CT, DDL_T_F32, 128>(ex, one)
           : dt == DDL_T_BF16 ? score_fn<CT, DDL_T_BF16, 128>(ex, one)
                              : score_fn<CT, DDL_T_F16, 128>(ex, one);
  return dt == DDL_T_F32    ? score_fn<CT, DDL_T_F32, 64>(ex, one)
         : dt == DDL_T_BF16 ? score_fn<CT, DDL_T_BF16, 64>(ex, one)
                            : score_fn<CT, DDL_T_F16, 64>(ex, one);
}

template <int HD>
int tile_bytes(int dt, int need, int& tiles) {
  const bool f32 = dt == DDL_T_F32;
  const int per = f32 ? TileSmem<DDL_T_F32, HD>::PER : TileSmem<DDL_T_BF16, HD>::PER;
  tiles = need < TILE_SMEM / per ? need : TILE_SMEM / per;
  return tiles * per;
}

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
  const int tiles = (max_rows * a.GH + 7) / 8;
  const bool one = tiles == 1, ex = opts->softcap > 0.f || opts->slopes;
  // Blocks a warp takes: as many as leave the machine a few CTAs an SM, since each CTA
  // begins with a chain of dependent loads (lengths, page, scale, codes) and its queries.
  const int64_t blocks = ((int64_t)max_len + 15) / 16;
  s.wb = 1;
  while (s.wb < 32 && (int64_t)R * H_kv * ((blocks + 2 * SC_WARPS * s.wb - 1) / (2 * SC_WARPS * s.wb)) >= 8 * sms) s.wb *= 2;
  const int64_t chunks = (blocks + SC_WARPS * s.wb - 1) / (SC_WARPS * s.wb);
  if (chunks > 0x7fffffffLL) return DDL_ERR_UNSUPPORTED;
  int smem_tiles = 0, smem = 0;
  if (!one) smem = head_dim == 128 ? tile_bytes<128>(dtype, tiles, smem_tiles) : tile_bytes<64>(dtype, tiles, smem_tiles);
  const void* fn = kv->type == DDL_KV8_E4M3 ? score_fn<DDL_KV8_E4M3>(dtype, head_dim, ex, one)
                                            : score_fn<DDL_KV8_INT8>(dtype, head_dim, ex, one);
  if (smem > 32 * 1024 &&
      (st = cuda_status(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, TILE_SMEM))))
    return st;
  void* args[] = {&s, &smem_tiles};
  return cuda_status(launch_pdl(fn, dim3((unsigned)chunks, (unsigned)H_kv, (unsigned)R), dim3(SC_WARPS * 32), args,
                                (size_t)smem, (cudaStream_t)stream));
}
