// ddl_kv8_attn.cu -- attention over the 8-bit paged KV cache.
//
// For a query row q at position p and the keys j it sees,
//     s_j = scale q . k_j  (capped, biased),  out = sum_j e^{s_j} v_j / sum_j e^{s_j},
// with k_j = ks code_j and one scale ks for 16 tokens.  One pass over the
// codes with a running maximum m and sum l per query (base 2: s log2 e).
//
// A warp takes 16 tokens (one scale block) x 8 queries at a time, the queries
// being the heads of one K/V head's group times the request's rows:
//  - S^T = K Q^T on m16n8k16 MMAs with the 16 tokens as M.  The order of the
//    head dimensions inside the contraction is free as long as K and Q agree,
//    so lane (g, t) takes bytes 16t .. 16t + 15 of each 64 of token rows g and
//    g + 8: 16 bytes a load, each 4 of which become the lane's part of one
//    k-step of A.
//  - O^T += V^T P^T with the head dimensions as M.  Lane (g, t) takes the
//    hd/8 neighbouring bytes at hd/8 g of tokens 2t, 2t+1, 2t+8, 2t+9; byte
//    permutes pair the tokens and conversion gives A.  P^T comes from the S^T
//    accumulators by movmatrix.
// So no lane needs another's codes: each copies its own pieces (cp.async) into
// its own places of a ring of three blocks per warp and reads them back without
// a barrier or a bank conflict, both streams in whole 64- and 128-byte rows.
// (Held in registers a block ahead instead, the loads covered less than one
// memory latency per block.)  e4m3 and int8 codes are exact in fp16.  Q is scaled by a
// power of two per query and split into fp16 high part and (fp32 rows only)
// remainder: bf16 and fp16 values fit the high part (down to 2^-26 of the
// row's largest).  P (with V's scale, relative to the query's largest such
// product: ddl_kv8_attn.h) is likewise one fp16 (16-bit outputs: its 2^-11 is no
// more than their own rounding) or two (2^-22; 2^-36 of the largest product).
// Scores, their reference, l and O are fp32.
//
// Work.  A *unit* is the blocks of one request for one K/V head and up to 8
// tiles of 8 queries; a CTA of 8 warps gives each tile 8 / tiles warps, which
// take the unit's blocks in turn and join their results in shared memory.
// Few units or short axes take a cluster of 1 to 16 CTAs a unit and one launch:
// the CTAs' records (max, sum, O in fp32) are joined in their shared memory, in
// rank order; many short units one CTA for up to 8 K/V heads of a request, its
// warps divided among them.  Else the blocks of all units, laid end to end (request, head,
// tiles), are cut into equal contiguous shares, one per CTA, two CTAs per SM:
// ragged lengths and any number of requests fill the machine evenly, and a CTA
// pays for the start and the end of a unit only two or three times.  A unit that
// lies in one share is written at once; the others leave a record per share,
// joined in share order by a second kernel.  att_plan estimates which costs less.
#include <cuda_bf16.h>

#include <mutex>

#include "ddl_kv8_attn.h"

namespace ddl {
namespace {

constexpr int ATT_WARPS = 8;
// P's fp16 values carry 2^11: with the reference allowed to lag by
// 2^M_LAG they stay below 2^16, and what rounds off below fp16's smallest
// subnormal is 2^-36 of the largest product.
constexpr float P_SCALE = 2048.f;
constexpr float M_LAG = 4.f;

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// Copy of 16 bytes through L1, which the warps of a CTA that hold other queries
// of the same blocks find there.
__device__ __forceinline__ void cp_async16_l1(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Bytes lo16 / hi16 of w (two codes) as fp16 pairs.
template <int CT>
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (CT == DDL_KV8_E4M3) {
    e4m3x4_f16x2(w, lo, hi);
  } else {  // 1024 + (c + 128) - 1152 = c, exact in fp16
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
  }
}

template <int CT, int DT, int HD, bool EX>
struct Att {
  static constexpr int KS = HD / 16;  // k-steps of the score MMAs
  static constexpr int NV = HD / 64;  // 16-byte loads of a K row per lane
  static constexpr int MT = HD / 16;  // M tiles of the output MMAs
  static constexpr bool HL = DT == DDL_T_F32;
  static constexpr int OROW = HD + 4;
  // A warp's ring of blocks: each lane's own pieces of K and V, 16 (V of hd 64: 8)
  // bytes at a time, so that a lane reads back only what it copied itself.
  static constexpr int STAGES = 3;
  static constexpr int KB = 2 * NV * 512, VB = HD == 128 ? 2048 : 1024, STAGE = KB + VB;
  struct Warp {
    union {
      alignas(16) uint8_t ring[STAGES][STAGE];
      float o[8][OROW];  // the warp's record, when its blocks are done
      struct {
        float o_[8][OROW];
        float rec[8][HD];  // the record of tile `warp` of the CTA, for the CTAs of its cluster
      } rest;
    };
  };
  struct Smem {
    Warp w[ATT_WARPS];
    union {  // (so that two CTAs of fp32 rows fit an SM)
      alignas(16) uint2 ql[HL ? ATT_WARPS : 1][HL ? KS * 32 : 1];  // the remainders of Q (fp32 rows)
      float2 rml[ATT_WARPS * 8];  // the record's (max, sum), when the blocks are done
    };
    float ml[ATT_WARPS][8][2];
  };
  static __device__ __forceinline__ void segment(const AttArgs& A, Smem& S, int r, const Req& rq, int h, int qc,
                                                 int c0, int c1, bool direct, int64_t rec);
};

// Blocks [c0, c1) of the unit (request r, K/V heads h .. h + A.hp - 1, query tiles qc); the
// result goes to the output (direct: they are all of the unit's blocks) or to
// record `rec`.
template <int CT, int DT, int HD, bool EX>
__device__ __forceinline__ void Att<CT, DT, HD, EX>::segment(const AttArgs& A, Smem& S, int r, const Req& rq, int h,
                                                             int qc, int c0, int c1, bool direct, int64_t rec) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int nqueries = rq.n * A.GH;
  const int nqs = __ffs(A.nq) - 1, ts = nqs + __ffs(A.hp) - 1, tiles = 1 << ts;  // (powers of two)
  const int groups = ATT_WARPS >> ts;  // warps that share a tile's blocks
  const int wt = warp & (tiles - 1), tile = qc * A.nq + (wt & (A.nq - 1)), hw = h + (wt >> nqs), kg = warp >> ts;
  const bool live = tile * 8 < nqueries;

  const int nb = live && c1 > c0 + kg ? (c1 - c0 - kg + groups - 1) / groups : 0;  // this warp's blocks
  // The query of this lane's column g of Q^T's fragments, on its way while the blocks are looked up.
  const int my_q = tile * 8 + g, my_row = my_q < nqueries ? group_row(A, my_q) : 0;
  float4 f[KS];
  {
    const int64_t at = (int64_t)(rq.row0 + my_row) * A.q_stride +
                       (int64_t)(hw * A.GH + my_q - my_row * A.GH) * HD + t * 16;
#pragma unroll
    for (int s = 0; s < KS; ++s)
      f[s] = my_q < nqueries ? load_elem4<DT>(A.q, at + 64 * (s >> 2) + 4 * (s & 3)) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  // block i of this warp: c0 + kg + i * groups; lane l holds the place and the
  // scales of blocks 32 w + l, of this batch of 32 and the next
  const int bshift = A.pshift - 4, bmask = (1 << bshift) - 1;
  auto block_row = [&](int i) -> int32_t {  // the block's index among all heads' blocks of the pool, -1: none
    if (i < nb) {
      const int b = c0 + kg + i * groups;
      const int32_t page = A.table[(int64_t)r * A.per + (b >> bshift)];
      if (page >= 0 && page < A.pages) return (int32_t)((((int64_t)page * A.Hkv + hw) << bshift) + (b & bmask));
      if (A.bad) atomicOr(A.bad, 1);
    }
    return -1;
  };
  auto block_scales = [&](int i, int32_t blk, float& ks, float& vs) {
    ks = vs = 0.f;
    if (blk < 0) return;
    ks = A.ks[blk];
    vs = A.vs[blk];
    check_scales(ks, vs);
    // V scales of blocks that no query of the tile sees do not count
    const int key = (c0 + kg + i * groups) * 16, last = min(tile * 8 + 7, nqueries - 1);
    if (key > rq.p0 + group_row(A, last) || key + 15 < first_seen(A, rq, tile * 8)) vs = 0.f;
  };
  int32_t blk_l = block_row(lane), blk_n = -1;
  float ks_l, vs_l, ks_n = 0.f, vs_n = 0.f;
  block_scales(lane, blk_l, ks_l, vs_l);
  // block i on its way into the ring; its place is lane i % 32's of this batch of 32 or the next
  const uint32_t ring = smem_addr(&S.w[warp].ring[0][0]) + lane * 16;
  const bool shared_codes = A.nq > 1;  // (4 requests of up to 16 rows, 4096 int8 tokens: 65 us through L1, 70 past it)
  const uint8_t *const k_lane = A.k + g * HD + t * 16, *const v_lane = A.v + 2 * t * HD + g * (HD / 8);
  uint32_t slot_in = 0, slot_out = 0;  // ring places of the next block to fetch and to use
  auto fetch = [&](int i, int32_t blks) {
    const int32_t blk = __shfl_sync(FULL, blks, i & 31);
    const uint32_t dst = ring + slot_in;
    slot_in = slot_in == (STAGES - 1) * STAGE ? 0u : slot_in + STAGE;
    if (blk >= 0) {  // (none past the last)
      const int64_t f = (int64_t)blk * (16 * HD);
      const uint8_t *pk = k_lane + f, *pv = v_lane + f;
#pragma unroll
      for (int j = 0; j < 2 * NV; ++j) {  // K: bytes 16 t of each 64 of rows g, g + 8
        const uint8_t* p = pk + (j / NV) * 8 * HD + (j % NV) * 64;
        if (shared_codes) cp_async16_l1(dst + j * 512, p);
        else cp_async16(dst + j * 512, p);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {  // V: bytes hd/8 g of tokens 2t, 2t+1, 2t+8, 2t+9
        const uint8_t* p = pv + ((j & 1) + (j >> 1) * 8) * HD;
        if (HD == 64) cp_async8(dst + KB + j * 256 - lane * 8, p);
        else if (shared_codes) cp_async16_l1(dst + KB + j * 512, p);
        else cp_async16(dst + KB + j * 512, p);
      }
    }
    cp_async_commit();
  };
  __syncwarp();
#pragma unroll
  for (int i = 0; i < STAGES; ++i) fetch(i, blk_l);
  // Q's fragments (column g), columns 2t, 2t + 1 of the scores
  // (the remainders of fp32 rows wait in shared memory)
  uint32_t qh[KS][2];
  uint2* const ql = &S.ql[HL ? warp : 0][HL ? lane : 0];
  float qf = 0.f;  // 2^e of query g
  {
    float mx = 0.f;
#pragma unroll
    for (int s = 0; s < KS; ++s)
      mx = fmaxf(mx, fmaxf(fmaxf(fabsf(f[s].x), fabsf(f[s].y)), fmaxf(fabsf(f[s].z), fabsf(f[s].w))));
    mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 2));
    int e = (int)((__float_as_uint(mx) >> 23) & 255u) - 127 - 12;  // the largest lands in [2^12, 2^13)
    e = e < -100 ? -100 : e > 115 ? 115 : e;
    const float down = __uint_as_float((uint32_t)(127 - e) << 23);
    qf = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const float4 v = make_float4(f[s].x * down, f[s].y * down, f[s].z * down, f[s].w * down);
      qh[s][0] = pack_f16x2(v.x, v.y);
      qh[s][1] = pack_f16x2(v.z, v.w);
      if (HL) {
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&qh[s][0]));
        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&qh[s][1]));
        ql[s * 32] = make_uint2(pack_f16x2(v.x - a.x, v.y - a.y), pack_f16x2(v.z - b.x, v.w - b.y));
      }
    }
  }
  // per score column: factor, the last and first key it sees, slope
  float cf[2], slope[2];
  int hi[2], lo[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int qi = tile * 8 + 2 * t + c;
    const bool has = qi < nqueries;
    const int row = has ? group_row(A, qi) : 0;
    const int p = rq.p0 + row;
    hi[c] = has ? p : -1;
    lo[c] = A.window > 0 ? p - A.window + 1 : 0;
    const float q2 = __shfl_sync(FULL, qf, 4 * (2 * t + c));
    cf[c] = q2 * A.scale;
    slope[c] = EX && A.slopes && has ? A.slopes[hw * A.GH + qi - row * A.GH] * LOG2E : 0.f;
    if (!EX) cf[c] *= LOG2E;
    else if (A.softcap > 0.f) cf[c] = __fdiv_rn(cf[c], A.softcap);
    else cf[c] *= LOG2E;
  }
  // keys that every column of the tile sees: blocks inside need no masks
  int all_hi = min(hi[0], hi[1]), all_lo = max(lo[0], lo[1]), any_hi = max(hi[0], hi[1]);
  {
    const bool h0 = tile * 8 + 2 * t < nqueries, h1 = tile * 8 + 2 * t + 1 < nqueries;
    all_hi = h0 ? (h1 ? all_hi : hi[0]) : 0x7fffffff;
    all_lo = h0 ? (h1 ? all_lo : lo[0]) : 0;
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      all_hi = min(all_hi, __shfl_xor_sync(FULL, all_hi, o));
      all_lo = max(all_lo, __shfl_xor_sync(FULL, all_lo, o));
      any_hi = max(any_hi, __shfl_xor_sync(FULL, any_hi, o));
    }
  }

  float o[MT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m) o[m][0] = o[m][1] = o[m][2] = o[m][3] = 0.f;
  float mrun[2] = {-INFINITY, -INFINITY}, lrun[2] = {0.f, 0.f};  // reference R, sum
  float vref = 0.f, vinv = 0.f;  // unit of O and its inverse

#pragma unroll 1
  for (int i = 0; i < nb; ++i) {
    const int l = i & 31;
    if (l == 4) blk_n = block_row((i & ~31) + 32 + lane);  // the next batch, long before it is used
    if (l == 16) block_scales((i & ~31) + 32 + lane, blk_n, ks_n, vs_n);
    const bool none = __shfl_sync(FULL, blk_l, l) < 0;
    const int key0 = (c0 + kg + i * groups) * 16;
    const float ks = __shfl_sync(FULL, ks_l, l), vs = __shfl_sync(FULL, vs_l, l);

    cp_async_wait<STAGES - 1>();
    const uint32_t src = ring + slot_out;
    slot_out = slot_out == (STAGES - 1) * STAGE ? 0u : slot_out + STAGE;
    uint4 kb[2][NV];
#pragma unroll
    for (int j = 0; j < 2 * NV; ++j) kb[j / NV][j % NV] = lds128(src + j * 512);
    // scores of tokens g (c 0, 1) and g + 8 (c 2, 3) for queries 2t, 2t + 1
    float c[4] = {0.f, 0.f, 0.f, 0.f}, c2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const uint4 x = kb[0][s / 4], y = kb[1][s / 4];
      const uint32_t wx = (s & 3) == 0 ? x.x : (s & 3) == 1 ? x.y : (s & 3) == 2 ? x.z : x.w;
      const uint32_t wy = (s & 3) == 0 ? y.x : (s & 3) == 1 ? y.y : (s & 3) == 2 ? y.z : y.w;
      uint32_t a0, a1, a2, a3;
      codes_f16<CT>(wx, a0, a2);
      codes_f16<CT>(wy, a1, a3);
      mma_f16((s & 1) ? c2 : c, a0, a1, a2, a3, qh[s][0], qh[s][1]);
      if (HL) {
        const uint2 q2 = ql[s * 32];
        mma_f16((s & 1) ? c2 : c, a0, a1, a2, a3, q2.x, q2.y);
      }
    }
    uint4 vb[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (HD == 128) {
        vb[j] = lds128(src + KB + j * 512);
      } else {
        const uint2 x = lds64(src + KB + j * 256 - lane * 8);
        vb[j] = make_uint4(x.x, x.y, 0u, 0u);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int col = j & 1;
      float s = (c[j] + c2[j]) * (ks * cf[col]);
      if (EX) {
        // (relative to the score at any cap, as 1 - 2 / (e^{2x} + 1) is not: a cap of 1e6 must not change a score of 3)
        if (A.softcap > 0.f) s = A.softcap * LOG2E * tanhf(s);
        s -= slope[col] * (float)(hi[col] - (key0 + g + (j >> 1) * 8));
      }
      c[j] = s;
    }
    const bool edge = none || key0 + 15 > all_hi || key0 < all_lo;
    if (edge) {  // some column does not see some token, or the block is missing
      uint32_t dead = 0;  // this lane's V tokens that nobody sees
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = key0 + 2 * t + (j & 1) + (j >> 1) * 8;
        if (none || key > any_hi) dead |= 1u << j;
      }
      uint32_t nan = 0;  // ... that hold a NaN code
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t w[4] = {vb[j].x, vb[j].y, HD == 128 ? vb[j].z : 0u, HD == 128 ? vb[j].w : 0u};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if ((dead >> j) & 1u) w[u] = 0u;
          if (CT == DDL_KV8_E4M3) {
            const uint32_t m = nan_bytes(w[u]);
            if (m) nan |= 1u << (2 * t + (j & 1) + (j >> 1) * 8);
            w[u] &= ~m;
          }
        }
        vb[j].x = w[0];
        vb[j].y = w[1];
        if (HD == 128) {
          vb[j].z = w[2];
          vb[j].w = w[3];
        }
      }
      // a NaN in V reaches exactly the queries that see its token, through their scores
      if (CT == DDL_KV8_E4M3) nan = __reduce_or_sync(FULL, nan);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int off = g + (j >> 1) * 8, key = key0 + off, col = j & 1;
        if (none || key > hi[col] || key < lo[col]) c[j] = -INFINITY;
        else if ((nan >> off) & 1u) c[j] = __uint_as_float(0x7fffffffu);
      }
    }
    if (vs >= 2.f * vref && vs > 0.f) {  // O moves to the unit of this block's scale, and with it the reference
      const float nref = pow2_floor(vs);
      if (vref > 0.f) {
        const float down = pow2_log_ratio(nref, vref), f = vref * pow2_inv(nref);
        float a[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float top = lrun[q];  // (a weight is at most its lane's sum)
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(FULL, top, x));
          const float nr = mrun[q] + fmaxf(-down, __log2f(top) - P_SPAN);
          a[q] = mrun[q] == -INFINITY ? 1.f : exp2_fast(mrun[q] - nr);
          mrun[q] = nr;
          lrun[q] *= a[q];
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int x = 0; x < 4; ++x) o[m][x] *= a[x & 1] * f;
      }
      vref = nref;
      vinv = pow2_inv(nref);
    }
    // the reference: raised only when some product passes it by M_LAG (or a weight by P_TOP)
    const float vn = vs * vinv, lv = scale_log(vn), thr = fminf(M_LAG - lv, P_TOP);
    const float t0 = fmaxf(c[0], c[2]), t1 = fmaxf(c[1], c[3]);
    if (__any_sync(FULL, t0 > mrun[0] + thr || t1 > mrun[1] + thr)) {
      float n0 = t0, n1 = t1;
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) {
        n0 = fmaxf(n0, __shfl_xor_sync(FULL, n0, x));
        n1 = fmaxf(n1, __shfl_xor_sync(FULL, n1, x));
      }
      n0 = fmaxf(mrun[0], n0 + lv);
      n1 = fmaxf(mrun[1], n1 + lv);
      const float a0 = mrun[0] == -INFINITY ? 0.f : exp2_fast(mrun[0] - n0);
      const float a1 = mrun[1] == -INFINITY ? 0.f : exp2_fast(mrun[1] - n1);
      mrun[0] = n0;
      mrun[1] = n1;
      lrun[0] *= a0;
      lrun[1] *= a1;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        o[m][0] *= a0;
        o[m][1] *= a1;
        o[m][2] *= a0;
        o[m][3] *= a1;
      }
    }
    const float wv = vn * P_SCALE;
    const float m0 = mrun[0] == -INFINITY ? 0.f : mrun[0], m1 = mrun[1] == -INFINITY ? 0.f : mrun[1];
    const float p0 = exp2_fast(c[0] - m0), p1 = exp2_fast(c[1] - m1), p2 = exp2_fast(c[2] - m0), p3 = exp2_fast(c[3] - m1);
    lrun[0] += p0 + p2;
    lrun[1] += p1 + p3;
    const float w0 = p0 * wv, w1 = p1 * wv, w2 = p2 * wv, w3 = p3 * wv;
    const uint32_t u0 = pack_f16x2(w0, w1), u1 = pack_f16x2(w2, w3);
    const uint32_t ph0 = movmatrix_trans(u0), ph1 = movmatrix_trans(u1);
    uint32_t pl0 = 0, pl1 = 0;
    if (HL) {
      const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&u0));
      const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&u1));
      pl0 = movmatrix_trans(pack_f16x2(w0 - a.x, w1 - a.y));
      pl1 = movmatrix_trans(pack_f16x2(w2 - b.x, w3 - b.y));
    }
#pragma unroll
    for (int w = 0; w < HD / 32; ++w) {  // four head dimensions of the lane: two M tiles
      const uint32_t x0 = w == 0 ? vb[0].x : w == 1 ? vb[0].y : w == 2 ? vb[0].z : vb[0].w;
      const uint32_t x1 = w == 0 ? vb[1].x : w == 1 ? vb[1].y : w == 2 ? vb[1].z : vb[1].w;
      const uint32_t x2 = w == 0 ? vb[2].x : w == 1 ? vb[2].y : w == 2 ? vb[2].z : vb[2].w;
      const uint32_t x3 = w == 0 ? vb[3].x : w == 1 ? vb[3].y : w == 2 ? vb[3].z : vb[3].w;
      uint32_t a[4], b[4];  // tiles 2 w and 2 w + 1
      codes_f16<CT>(__byte_perm(x0, x1, 0x5140), a[0], a[1]);
      codes_f16<CT>(__byte_perm(x2, x3, 0x5140), a[2], a[3]);
      codes_f16<CT>(__byte_perm(x0, x1, 0x7362), b[0], b[1]);
      codes_f16<CT>(__byte_perm(x2, x3, 0x7362), b[2], b[3]);
      mma_f16(o[2 * w], a[0], a[1], a[2], a[3], ph0, ph1);
      mma_f16(o[2 * w + 1], b[0], b[1], b[2], b[3], ph0, ph1);
      if (HL) {
        mma_f16(o[2 * w], a[0], a[1], a[2], a[3], pl0, pl1);
        mma_f16(o[2 * w + 1], b[0], b[1], b[2], b[3], pl0, pl1);
      }
    }
    // (the block's pieces are in registers: its place in the ring is free)
    fetch(i + STAGES, l + STAGES < 32 ? blk_l : blk_n);
    if (l == 31) {  // on to the next batch
      blk_l = blk_n;
      ks_l = ks_n;
      vs_l = vs_n;
    }
  }
  cp_async_wait<0>();

  // the warp's record: lane (g, t) holds head dimensions hd/8 g + ... of queries 2t, 2t + 1
#pragma unroll
  for (int x = 4; x < 32; x <<= 1) {
    lrun[0] += __shfl_xor_sync(FULL, lrun[0], x);
    lrun[1] += __shfl_xor_sync(FULL, lrun[1], x);
  }
  __syncwarp();
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    float* row = &S.w[warp].o[2 * t + c][g * (HD / 8)];
#pragma unroll
    for (int m = 0; m < MT; m += 2)
      *reinterpret_cast<float4*>(row + 2 * m) =
          make_float4(o[m][c] * (1.f / P_SCALE) * vref, o[m][2 + c] * (1.f / P_SCALE) * vref,
                      o[m + 1][c] * (1.f / P_SCALE) * vref, o[m + 1][2 + c] * (1.f / P_SCALE) * vref);
    if (g == 0) {
      S.ml[warp][2 * t + c][0] = mrun[c];
      S.ml[warp][2 * t + c][1] = lrun[c];
    }
  }
  __syncthreads();
  // the tile's warps joined (in warp order): thread = (tile, query, 4 head dimensions)
  constexpr int DQ = HD / 4;
  for (int x = threadIdx.x; x < tiles * 8 * DQ; x += ATT_WARPS * 32) {
    const int d = x % DQ, qq = (x / DQ) & 7, tl = x / (8 * DQ);
    const int qi = (qc * A.nq + (tl & (A.nq - 1))) * 8 + qq;
    if (qi >= nqueries) continue;
    float m = -INFINITY;
    for (int w = 0; w < groups; ++w) m = fmaxf(m, S.ml[tl + w * tiles][qq][0]);
    const float mref = m == -INFINITY ? 0.f : m;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
    for (int w = 0; w < groups; ++w) {
      const int wp = tl + w * tiles;
      const float f = exp2_fast(S.ml[wp][qq][0] - mref);
      const float4 v = *reinterpret_cast<const float4*>(&S.w[wp].o[qq][4 * d]);
      l = fmaf(f, S.ml[wp][qq][1], l);
      acc.x = fmaf(f, v.x, acc.x);
      acc.y = fmaf(f, v.y, acc.y);
      acc.z = fmaf(f, v.z, acc.z);
      acc.w = fmaf(f, v.w, acc.w);
    }
    const int row = group_row(A, qi), head = (h + (tl >> nqs)) * A.GH + qi - row * A.GH;
    const int64_t rh = (int64_t)(rq.row0 + row) * A.Hq + head;
    if (A.cluster > 1) {
      *reinterpret_cast<float4*>(&S.w[tl].rest.rec[qq][4 * d]) = acc;
      if (d == 0) S.rml[tl * 8 + qq] = make_float2(m, l);
    } else if (direct) {
      const float inv = l != 0.f ? 1.f / l : 0.f;  // (NaN stays NaN)
      store_elem4<DT>(A.out, (int64_t)(rq.row0 + row) * A.out_stride + (int64_t)head * HD + 4 * d,
                      make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
      if (d == 0 && A.lse) A.lse[(int64_t)(rq.row0 + row) * A.Hq + head] = (m + log2f(l)) * LN2;
    } else {
      const int64_t at = rec * (A.nq * 8) + tl * 8 + qq;
      *reinterpret_cast<float4*>(A.rec_o + at * HD + 4 * d) = acc;
      if (d == 0) *reinterpret_cast<float2*>(A.rec_ml + at * 2) = make_float2(m, l);
    }
  }
}

template <int CT, int DT, int HD, bool EX>
__global__ void __launch_bounds__(ATT_WARPS * 32, 2) kv8_attention_kernel(const __grid_constant__ AttArgs A) {
  using K = Att<CT, DT, HD, EX>;
  extern __shared__ __align__(16) uint8_t att_smem[];
  typename K::Smem& S = *reinterpret_cast<typename K::Smem*>(att_smem);
  int64_t* const pre = reinterpret_cast<int64_t*>(att_smem + ((sizeof(typename K::Smem) + 15) & ~size_t(15)));  // [R + 1], shares only
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  if (A.cluster) {
    const ClusterPart part(A);
    int u = part.unit;
    const int qc = u % A.nqc;
    u /= A.nqc;
    const int hg = A.Hkv >> (__ffs(A.hp) - 1), r = u / hg, h = (u - r * hg) * A.hp;
    const Req rq = load_req(A, r);
    if (rq.bad && A.bad && tid == 0) atomicOr(A.bad, 1);
    if (qc >= unit_groups(A, rq)) return;  // (all CTAs of the cluster)
    int c0, c1;
    part.blocks(A, rq, c0, c1);
    K::segment(A, S, r, rq, h, qc, c0, c1, A.cluster == 1, 0);
    if (A.cluster > 1) {
      __syncthreads();
      cluster_join<DT, HD>(A, part, smem_addr(&S.w[0].rest.rec[0][0]), sizeof(S.w[0]), smem_addr(&S.rml[0]),
                           ATT_WARPS * 32);
    }
    return;
  }
  __shared__ int64_t wsum[ATT_WARPS];
  const int64_t W = unit_prefix<ATT_WARPS * 32>(A, pre, wsum);
  const int64_t n = share_count(A, W);
  if ((int64_t)blockIdx.x >= n || W == 0) return;
  int64_t x, end;
  share_bounds(W, n, x, end);
  int r = 0;
  for (int hi = A.R; hi - r > 1;) {  // the last r with pre[r] <= x
    const int mid = (r + hi) >> 1;
    if (pre[mid] <= x) r = mid;
    else hi = mid;
  }
  while (x < end) {
    while (pre[r + 1] <= x) ++r;
    const Req rq = load_req(A, r);
    int unit, c0, cnt;
    if (!share_segment(A, rq, pre[r], x, end, unit, c0, cnt)) continue;
    const int per_head = unit_groups(A, rq), h = per_head == 1 ? unit : unit / per_head;
    K::segment(A, S, r, rq, h, unit - h * per_head, c0, c0 + cnt, cnt == rq.b1 - rq.b0,
               blockIdx.x + (int64_t)r * A.Hkv * A.nqc + unit);
    __syncthreads();  // the next segment writes the shared records
  }
}

// Joins the records of a query, in share order.  They stand 4 KB and more
// apart and are a unit's shares, two or three in a full batch and tens when one
// request is spread over the machine: the time is that of one round trip to L2
// if their loads go out together.  So PAR warps take a query, warp w of them
// every PAR-th record, four at a time, each lane hd / 32 head dimensions: 8 where
// a unit has 8 shares and more, else 1 (the whole call, 1 request of 32768 tokens
// 24.2 us against 30.7; 64 of up to 8192 105.8 against 96.9).
template <int DT, int HD, int PAR>
__global__ void __launch_bounds__(256) kv8_join_kernel(const __grid_constant__ AttArgs A) {
  constexpr int E = HD / 32;
  __shared__ float so[8][HD];
  __shared__ float2 sml[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, par = warp % PAR;
  const int nq8 = A.nq * 8;
  uint32_t id = blockIdx.x * (8 / PAR) + warp / PAR;  // (request, head, group of tiles, query)
  const uint32_t per_req = (uint32_t)A.Hkv * A.nqc * nq8;  // (a multiple of 8: a CTA's queries are of one request)
  const int r = (int)(id / per_req);
  id -= (uint32_t)r * per_req;
  const int x = (int)(id % nq8), u = (int)(id / nq8), h = u / A.nqc, qc = u - h * A.nqc;
  pdl_trigger();
  // The lengths too are read after the wait: this grid starts while the attention
  // runs, and only its own wait makes what came before visible to it.  (Read ahead of
  // it they saved 1 request of 32768 tokens 0.4 us of 24.7.)
  pdl_wait();
  const Req rq = load_req(A, r);
  const int64_t W = A.prefix[A.R], p0 = A.prefix[r];
  const int per_head = unit_groups(A, rq), nb = rq.b1 - rq.b0;
  const int qi = qc * nq8 + x, unit = h * per_head + qc;
  if (qc >= per_head || qi >= rq.n * A.GH) return;
  float m = -INFINITY, l = 0.f, acc[E];
#pragma unroll
  for (int k = 0; k < E; ++k) acc[k] = 0.f;
  if (nb > 0) {
    const int64_t n = share_count(A, W), lo = p0 + (int64_t)unit * (nb + A.unit_cost) + A.unit_cost;
    int i0, i1;
    if (W < (1 << 22)) {
      i0 = (int)owner32((uint32_t)W, (uint32_t)n, (uint32_t)lo);
      i1 = (int)owner32((uint32_t)W, (uint32_t)n, (uint32_t)(lo + nb - 1));
    } else {
      i0 = (int)owner_of(W, n, lo);
      i1 = (int)owner_of(W, n, lo + nb - 1);
    }
    if (i0 == i1) return;  // written at once
    const int64_t rec0 = ((int64_t)r * A.Hkv * A.nqc + unit) * nq8 + x;
    for (int i = i0 + par; i <= i1; i += 4 * PAR) {
      float2 ml[4];
      float v[4][E];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int j = i + k * PAR;
        const int64_t at = rec0 + (int64_t)j * nq8;
        ml[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int e = 0; e < E; ++e) v[k][e] = 0.f;
        if (j <= i1) {
          ml[k] = __ldcg(reinterpret_cast<const float2*>(A.rec_ml) + at);
          if (E == 4) {
            const float4 f = __ldcg(reinterpret_cast<const float4*>(A.rec_o + at * HD) + lane);
            v[k][0] = f.x; v[k][1] = f.y; v[k][E - 2] = f.z; v[k][E - 1] = f.w;
          } else {
            const float2 f = __ldcg(reinterpret_cast<const float2*>(A.rec_o + at * HD) + lane);
            v[k][0] = f.x; v[k][1] = f.y;
          }
        }
      }
      float nm = m;
#pragma unroll
      for (int k = 0; k < 4; ++k) nm = fmaxf(nm, ml[k].x);
      const float ref = nm == -INFINITY ? 0.f : nm, f0 = exp2_fast(m - ref);
      l *= f0;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] *= f0;
      m = nm;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float f = exp2_fast(ml[k].x - ref);
        l = fmaf(f, ml[k].y, l);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(f, v[k][e], acc[e]);
      }
    }
  }
  if (PAR > 1) {  // (all warps of the CTA are here: they share the query)
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][lane * E + e] = acc[e];
    if (lane == 0) sml[warp] = make_float2(m, l);
    __syncthreads();
    if (warp > 0) return;
    m = -INFINITY;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = fmaxf(m, sml[k].x);
    const float ref = m == -INFINITY ? 0.f : m;
    l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float f = exp2_fast(sml[k].x - ref);
      l = fmaf(f, sml[k].y, l);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(f, so[k][lane * E + e], acc[e]);
    }
  }
  const int row = group_row(A, qi), head = h * A.GH + qi - row * A.GH;
  const float inv = l != 0.f ? 1.f / l : 0.f;
  const int64_t at = (int64_t)(rq.row0 + row) * A.out_stride + (int64_t)head * HD + lane * E;
  if (E == 4) {
    store_elem4<DT>(A.out, at, make_float4(acc[0] * inv, acc[1] * inv, acc[E - 2] * inv, acc[E - 1] * inv));
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) store_elem<DT>(A.out, at + e, acc[e] * inv);
  }
  if (lane == 0 && A.lse) A.lse[(int64_t)(rq.row0 + row) * A.Hq + head] = (m + log2f(l)) * LN2;
}

// ------------------------------------------------------------------ host
int g_att_sms[64];
std::mutex g_att_mu;

int att_sms(int& sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_status(e);
  if (dev < 0 || dev >= 64) return DDL_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lk(g_att_mu);
  if (!g_att_sms[dev]) {
    int n = 0;
    if ((e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return cuda_status(e);
    g_att_sms[dev] = n;
  }
  sms = g_att_sms[dev];
  return DDL_OK;
}

// Clusters: CTAs of a unit at most (16 is past the portable 8, and two fit a
// GPC's SMs side by side), blocks a CTA takes at least.
constexpr int MAX_CLUSTER = 16, MIN_PART = 16;
// fp32 rows of 128: two CTAs fit an SM while the weights before so many requests fit beside the rings (64 requests of
// up to 2049 in shares: 72 us, one CTA an SM; whole units of two heads a CTA: 55).
constexpr int F32_TWO_CTAS_R = 55;
static_assert(2 * (sizeof(Att<DDL_KV8_INT8, DDL_T_F32, 128, false>::Smem) + (F32_TWO_CTAS_R + 1) * 8 + ATT_WARPS * 8 + 1024) <=
                  228 * 1024,
              "two CTAs an SM");

struct AttPlan {
  int32_t nq, nqc, hp, cluster, ctas, deep;  // deep: a unit may have many shares
  int32_t unit_cost, min_share;          // of a CTA's share, in blocks
  int64_t rec_ml, prefix, total;         // workspace offsets
  int64_t cost;                          // estimate, in 0.1 us
};

int check_sizes(int32_t H_q, int32_t H_kv, int32_t hd, int32_t R, int32_t T, int32_t max_rows, int32_t max_len) {
  if (hd != 64 && hd != 128) return DDL_ERR_SHAPE;
  if (H_kv < 1 || H_kv > DDL_KV8_MAX_HEADS || H_q < H_kv || H_q % H_kv || H_q / H_kv > DDL_MAX_GROUP_HEADS)
    return DDL_ERR_SHAPE;
  if (R < 1 || T < 1 || max_rows < 1 || max_len < 1) return DDL_ERR_ARG;
  if (R > DDL_KV8_MAX_REQS || max_rows > DDL_KV8_MAX_ROWS) return DDL_ERR_UNSUPPORTED;
  return DDL_OK;
}

int att_plan(bool tc, bool f32, int32_t H_q, int32_t H_kv, int32_t hd, int32_t R, int32_t max_rows, int32_t max_len,
             int32_t window, bool clusters, AttPlan& p) {
  int sms = 0;
  const int st = att_sms(sms);
  if (st) return st;
  const int tiles = (max_rows * (H_q / H_kv) + 7) / 8;
  p.nq = 1;
  while (p.nq < (tc ? 4 : ATT_WARPS) && p.nq < tiles) p.nq *= 2;
  p.nqc = (tiles + p.nq - 1) / p.nq;
  int64_t keys = max_len;
  if (window > 0 && (int64_t)window + max_rows + 15 < keys) keys = (int64_t)window + max_rows + 15;
  const int64_t blocks = (keys + 15) / 16, units = (int64_t)R * H_kv * p.nqc;
  int64_t slots = (tc ? kv8_tc_ctas(p.nq, f32, 0) : 2) * sms;  // CTAs that run at once (their shared memory)
  p.rec_ml = p.prefix = 0;
  p.total = 256;
  p.deep = 0;
  p.unit_cost = p.min_share = 1;
  // What it will take, in 0.1 us, by what the two kernels measured (head_dim
  // 128, one GB300): a call 4 us (tcgen05 7) apart from its blocks; 8 blocks in a
  // row of a CTA, for each of its query tiles, 0.9 us while the ring's first fill
  // lasts and 2.8 after it (1.4 where tiles share the codes; fp32 rows 1.5 and 4, in shares 1.0 and 3.1, at least 1.6), on tcgen05 1.0 us for one tile,
  // 1.6 for two, 2.1 for four; a further wave of CTAs 2 us (5); a cluster's join
  // 1.3 us; shares 6 to 8 us for the sums of the lengths, the records' way through
  // memory and the second launch, and every unit a CTA begins 3.5 us (5).
  // E.g. (bf16 rows, 64/8 heads, calls in a graph) 1 request of 600 int8 tokens:
  // clusters 7.4 us, shares 12.3 (e4m3 on tcgen05 in clusters 9.2); of 8193: 14.7,
  // 16.6 (12.5); 64 requests of up to 2049: shares 48 (38).  40 drawn sizes of e4m3
  // codes and head_dim 128: 0.4 % above the better kernel in the geometric mean,
  // 20 % at worst (26 requests of 6 rows on 119 tokens: 9.2 us against 7.7).  The same
  // costs choose the split for head_dim 64.
  const int64_t fixed = tc ? 70 : 40, again = fixed - 20;
  auto in_a_row = [&](int64_t b, int64_t filling, int64_t after) -> int64_t {
    if (tc) return (b + 7) / 8 * (p.nq == 1 ? 10 : p.nq == 2 ? 16 : 21);
    const int64_t groups = ATT_WARPS / p.nq, n = (b + groups - 1) / groups, first = n < 3 ? n : 3;
    const int64_t each = after / p.nq, least = f32 ? 16 : 14;
    return filling * first + (each < least ? least : each) * (n - first);
  };
  // A cluster per unit, of as many CTAs as fill the machine once; it pays for
  // every request what the longest costs.
  p.cluster = 1;
  while (p.cluster < MAX_CLUSTER && units * 2 * p.cluster <= slots && p.cluster * MIN_PART < blocks) p.cluster *= 2;
  p.hp = 1;
  if (p.cluster > 1 || tc) {
    const int64_t waves = (units * p.cluster + slots - 1) / slots;
    p.cost = waves * (again + in_a_row((blocks + p.cluster - 1) / p.cluster, f32 ? 15 : 9, f32 ? 40 : 28)) + 20 + (p.cluster > 1 ? 13 : 0);
  } else {
    // Many units: the CTA's warps are shared by hp K/V heads, whichever hp costs least: a wave of CTAs 3.5 us and
    // its rounds of 8 blocks 0.9 us where it is one CTA an SM, else 1.6 (fp32 rows a tenth more).  E.g. 64
    // requests of up to 512 int8 tokens, 32/8 heads: hp 1 / 2 / 4 / 8 21.1 / 18.0 / 19.4 / 32.6 us; 1000 of up to 128
    // 148 / 102 / 78 / 68.
    for (int hp = 1; hp == 1 || (hp * p.nq <= ATT_WARPS && H_kv % hp == 0); hp *= 2) {
      const int64_t ctas = units / hp, waves = (ctas + slots - 1) / slots;
      const int64_t rounds = (blocks * p.nq * hp + ATT_WARPS - 1) / ATT_WARPS, two = ctas > sms;
      const int64_t cost = waves * (35 + 2 * hp + (two ? 16 : 9) * rounds) * (f32 ? 11 : 10) / 10 + 20;
      if (hp > 1 && cost >= p.cost) continue;
      p.cost = cost;
      p.hp = hp;
    }
  }
  // (shares: ragged lengths up to the bound come to about 5/8 of it)
  if (tc) slots = kv8_tc_ctas(p.nq, f32, R) * sms;
  const int64_t least = tc ? 8 : 16;
  int64_t share = (units * blocks * (R > 1 ? 5 : 8) / 8 + slots - 1) / slots;
  share = share < least ? least : share;
  int64_t shares = units * (tc ? again : 35) / slots + in_a_row(share, f32 ? 10 : 9, f32 ? 31 : 28);
  if (!tc && f32 && hd == 128 && R > F32_TWO_CTAS_R) shares = shares * 5 / 2;
  shares += fixed + (tc ? 60 : 80);
  if (p.cost <= shares || clusters) {
    p.ctas = (int32_t)(units / p.hp * p.cluster);
    return DDL_OK;
  }
  p.cost = shares;
  // Measured at 64 requests of up to 8192 tokens, 64/8 heads (tcgen05: cost 16 / 24 / 40 110 / 106 / 99 us; warp MMAs
  // on 16 requests of 28/4 heads: cost 16 / 24 / 40 18 / 20 / 23 us).
  p.cluster = 0;
  p.hp = 1;
  p.unit_cost = tc ? 48 : 16;
  p.min_share = p.unit_cost + (int32_t)least;
  const int64_t all = ((int64_t)max_len + 15) / 16;
  const int64_t most = (units * (all + p.unit_cost) + p.min_share - 1) / p.min_share;
  p.ctas = (int32_t)(most < slots ? most : slots);
  if (p.ctas > 1024) return DDL_ERR_UNSUPPORTED;  // (the kernels' 32-bit share arithmetic)
  p.deep = units * 8 <= p.ctas;
  const int64_t queries = (units + p.ctas) * p.nq * 8;  // of all records
  p.rec_ml = align256(queries * hd * 4);
  p.prefix = align256(p.rec_ml + queries * 2 * 4);
  p.total = align256(p.prefix + (int64_t)(R + 1) * 8);
  return DDL_OK;
}

template <int CT, int DT, int HD>
const void* att_fn(bool ex) {
  return ex ? (const void*)kv8_attention_kernel<CT, DT, HD, true> : (const void*)kv8_attention_kernel<CT, DT, HD, false>;
}
template <int CT, int DT>
const void* att_fn(int hd, bool ex) {
  return hd == 128 ? att_fn<CT, DT, 128>(ex) : att_fn<CT, DT, 64>(ex);
}
template <int CT>
const void* att_fn(int dt, int hd, bool ex) {
  return dt == DDL_T_F32 ? att_fn<CT, DDL_T_F32>(hd, ex) : dt == DDL_T_BF16 ? att_fn<CT, DDL_T_BF16>(hd, ex)
                                                                           : att_fn<CT, DDL_T_F16>(hd, ex);
}
// Shared memory ahead of the prefix (the code types' kernels have the same).
size_t att_smem_bytes(int dt, int hd) {
  const bool f32 = dt == DDL_T_F32;
  const size_t n = hd == 128 ? (f32 ? sizeof(Att<DDL_KV8_INT8, DDL_T_F32, 128, false>::Smem)
                                    : sizeof(Att<DDL_KV8_INT8, DDL_T_BF16, 128, false>::Smem))
                             : (f32 ? sizeof(Att<DDL_KV8_INT8, DDL_T_F32, 64, false>::Smem)
                                    : sizeof(Att<DDL_KV8_INT8, DDL_T_BF16, 64, false>::Smem));
  return (n + 15) & ~size_t(15);
}
template <int DT>
const void* join_fn(int hd, bool deep) {
  if (hd == 128) return deep ? (const void*)kv8_join_kernel<DT, 128, 8> : (const void*)kv8_join_kernel<DT, 128, 1>;
  return deep ? (const void*)kv8_join_kernel<DT, 64, 8> : (const void*)kv8_join_kernel<DT, 64, 1>;
}

}  // namespace
}  // namespace ddl

using namespace ddl;

extern "C" size_t ddl_kv8_attention_workspace_bytes(int32_t H_q, int32_t H_kv, int32_t head_dim, int32_t R, int32_t T,
                                                    int32_t max_rows, int32_t max_len) {
  if (check_sizes(H_q, H_kv, head_dim, R, T, max_rows, max_len)) return 0;
  int64_t most = 0;  // of either kernel and any row type, without a window: as much as any call of these sizes takes
  for (int k = 0; k < 4; ++k) {
    AttPlan p;
    if (att_plan(k & 1, k >> 1, H_q, H_kv, head_dim, R, max_rows, max_len, 0, false, p)) return 0;
    if (p.total > most) most = p.total;
  }
  return (size_t)most;
}

extern "C" int ddl_kv8_attention(const ddl_kv8* kv, int32_t H_q, int32_t H_kv, int32_t head_dim, ddl_dtype dtype,
                                 const ddl_attn_opts* opts, int32_t R, int32_t T, int32_t max_rows, int32_t max_len,
                                 const int32_t* q_off, const int32_t* kv_len, const int32_t* page_table,
                                 int32_t pages_per_seq, const void* q, int64_t q_stride, void* out,
                                 int64_t out_stride, float* lse, int32_t* bad_out, void* workspace, size_t ws_bytes,
                                 void* stream) {
  int st = check_kv8(kv, H_kv, head_dim);
  if (st) return st;
  if ((st = check_sizes(H_q, H_kv, head_dim, R, T, max_rows, max_len))) return st;
  if (!opts || !kv_len || !page_table || !q || !out) return DDL_ERR_ARG;
  if (!workspace) return DDL_ERR_WORKSPACE;
  if (!dtype_bytes(dtype)) return DDL_ERR_UNSUPPORTED;
  if (pages_per_seq < 1 || out == q) return DDL_ERR_ARG;
  if (!q_off && (max_rows != 1 || T < R)) return DDL_ERR_ARG;
  if ((int64_t)pages_per_seq * kv->page_size > 0x7fffffffLL) return DDL_ERR_UNSUPPORTED;
  if ((st = check_attn_opts(opts))) return st;
  const int64_t w = (int64_t)H_q * head_dim;
  if (q_stride < w || out_stride < w || q_stride % 8 || out_stride % 8) return DDL_ERR_ARG;
  if (!aligned16(q) || !aligned16(out) || !aligned16(workspace)) return DDL_ERR_ALIGN;
  for (const void* p : {(const void*)q_off, (const void*)kv_len, (const void*)page_table, (const void*)lse,
                        (const void*)bad_out})
    if ((uintptr_t)p & 3u) return DDL_ERR_ALIGN;
  const int32_t window = opts->window >= max_len ? 0 : opts->window;  // (a window as long as the bound hides nothing)
  // The plan; with a window, shares only where the call without one has room for them.
  auto plan_of = [&](bool tcgen05, AttPlan& p) -> int {
    const int rc = att_plan(tcgen05, dtype == DDL_T_F32, H_q, H_kv, head_dim, R, max_rows, max_len, 0, false, p);
    if (rc || window == 0) return rc;
    return att_plan(tcgen05, dtype == DDL_T_F32, H_q, H_kv, head_dim, R, max_rows, max_len, window, p.cluster > 0, p);
  };
  AttPlan pl;
  if ((st = plan_of(false, pl))) return st;
  const int64_t pool_rows = kv->pages * kv->page_size * H_kv;
  bool tc = kv->type == DDL_KV8_E4M3 && head_dim == 128 && pool_rows < (1ll << 31);
  if (tc) {
    AttPlan p;
    if ((st = plan_of(true, p))) return st;
    tc = p.cost < pl.cost;
    if (tc) pl = p;
  }
  if (ws_bytes < (size_t)pl.total) return DDL_ERR_WORKSPACE;
  AttArgs a;
  a.k = kv->k;
  a.v = kv->v;
  a.ks = kv->k_scale;
  a.vs = kv->v_scale;
  a.q_off = q_off;
  a.kv_len = kv_len;
  a.table = page_table;
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.bad = bad_out;
  a.rec_o = (float*)workspace;
  a.rec_ml = (float*)((uint8_t*)workspace + pl.rec_ml);
  a.prefix = (int64_t*)((uint8_t*)workspace + pl.prefix);
  a.slopes = opts->slopes;
  a.pages = kv->pages;
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.scale = opts->scale;
  a.softcap = fminf(opts->softcap, 0x1p100f);  // (a score over more than that would be subnormal)
  a.window = window;
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
  a.cluster = pl.cluster;
  a.ctas = pl.ctas;
  a.unit_cost = pl.unit_cost;
  a.min_share = pl.min_share;
  a.nq = pl.nq;
  a.nqc = pl.nqc;
  a.hp = pl.hp;
  const bool ex = opts->softcap > 0.f || opts->slopes;
  const void* fn = nullptr;
  void* args[] = {&a};
  if (tc) {
    st = kv8_tc_launch(a, dtype, pool_rows, stream);
  } else {
    fn = kv->type == DDL_KV8_E4M3 ? att_fn<DDL_KV8_E4M3>(dtype, head_dim, ex) : att_fn<DDL_KV8_INT8>(dtype, head_dim, ex);
    const size_t smem = att_smem_bytes(dtype, head_dim) + (pl.cluster ? 0 : (size_t)(R + 1) * 8);
    if ((st = cuda_status(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024)))) return st;
    if (pl.cluster > 8 && (st = cuda_status(cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1))))
      return st;
    st = cuda_status(launch_pdl_cluster(fn, dim3((unsigned)pl.ctas), dim3(ATT_WARPS * 32), args, smem, pl.cluster,
                                        (cudaStream_t)stream));
  }
  if (st || pl.cluster) return st;
  fn = dtype == DDL_T_F32    ? join_fn<DDL_T_F32>(head_dim, pl.deep)
       : dtype == DDL_T_BF16 ? join_fn<DDL_T_BF16>(head_dim, pl.deep)
                             : join_fn<DDL_T_F16>(head_dim, pl.deep);
  const int64_t queries = (int64_t)R * H_kv * pl.nqc * pl.nq * 8;
  return cuda_status(launch_pdl(fn, dim3((unsigned)(pl.deep ? queries : queries / 8)), dim3(256), args, 0,
                                (cudaStream_t)stream));
}
