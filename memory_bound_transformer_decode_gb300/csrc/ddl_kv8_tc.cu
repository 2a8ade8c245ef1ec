// ddl_kv8_tc.cu -- attention over the 8-bit paged cache on the 5th-generation
// tensor cores: e4m3 codes, head_dim 128 (ddl_kv8_attn.cu has the mathematics,
// the units and shares, and the kernel for int8 codes and head_dim 64).
//
// The codes are never converted: K and V tiles of 128 tokens go by TMA from
// the pages into shared memory and are the A operands of kind::f8f6f4 MMAs,
//     S^T [128 tokens x N] = K [tokens x hd] Q^T,
//     O^T [128 head dims x N] += V^T [hd x tokens] P^T,
// with V read as an M-major operand, so that nothing is transposed either.
// The warp-MMA kernel spends most of its issue slots on turning codes into
// fp16 fragments (about 370 instructions a warp per 16 tokens and 8 queries,
// bound by them and not by HBM); here 128 tokens and 8 queries cost four warps
// about 200 each.
//
// Q and P, which are not 8-bit, are split into 8-bit limbs.  The B operand has 16
// columns per 8 queries: group A holds limbs 1 .. L (one MMA pass each, summed
// in the accumulator), group B the next L, scaled by 16^L so that the type's
// narrow range does not cut them off, in the same passes.
//  - Q: e4m3, each limb the rounding of what the ones before leave, 4
//    significant bits; L = 2 for 16-bit rows (2^-16 of a value, 2^-26 of the
//    row's largest), 3 for fp32 rows (2^-24).
//  - P of 16-bit rows: fp16 (2^-11, no more than the output's own rounding; 2^-30 of
//    the query's largest product of weight and V scale) in four e5m2 limbs of 3 bits, exactly.  (As e4m3, whose
//    conversions both ways the limbs then need: 64 rows on 8192 tokens 64.6 us,
//    so 63.4, and 61.6 with two scores an instruction; 65.3 since the
//    weights' reference follows the V scales.)
//  - P of fp32 rows: an fp16 in four e5m2 limbs, groups A and B, and what it
//    leaves, times 2^12 and again in fp16, in those of two more groups, C and D: 2^-22
//    of a weight, 2^-39 of the largest.  (Six e4m3 limbs ended at 2^-27 of the largest:
//    the weights of a long tail that lie below it were in the sum but not in O.)  Each
//    MMA rounds its accumulator off, by up to 2^-23 of it; with the largest limbs in an
//    accumulator of their own that is 8 times a tile, not 16.
//
// A segment's tiles are taken from the newest token to the oldest: a distance
// bias then raises the running maximum once and not with every tile (4 rows of
// 16 requests, ALiBi: all 8 tiles of a share raised it, 1 does).
//
// Roles: one or two warpgroups softmax (thread = token of the tile, then head
// dimension of the output; 8 or 16 queries each), a warp copies, a warp issues
// MMAs.  Bounds: HBM for one tile of 8
// queries, softmax issue slots for many.
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include "ddl_kv8_attn.h"

namespace ddl {
namespace {

constexpr int TOK = 128, TBLK = TOK / KV8_BLOCK;  // tokens and blocks of a tile
constexpr uint32_t KBYTES = TOK * 128;

// P carries 2^5 (fp32 rows 2^11, within e5m2's 2^15); with the reference
// lagging by less than 2^3 what the limbs of 16-bit rows leave, times 2^8, stays
// within fp16.  (Raising it stops the softmax warps three times for the
// exchange of the maxima and rescales O in tensor memory: with a lag of 2^1
// every third tile of 16 queries did.)
constexpr float T_LAG = 3.f;
template <int L>  // (Q's passes: 2 or, for fp32 rows, 3)
constexpr float TP_SCALE = L == 2 ? 32.f : 2048.f;

// How long a CTA that leaves waits for its copies and MMAs in flight.  They end
// by themselves, and until then they write shared and tensor memory that the next
// CTA may get; so the caller's limit, which may be short, does not hold here.
constexpr uint64_t DRAIN_NS = 10000000000ull;

struct TcAtt {
  AttArgs A;
  uint64_t wait_ns;
  int32_t rows;  // of the pool's view: a box that begins there reads zeros
  alignas(64) CUtensorMap kmap, vmap;
};

template <int NT, int L>
struct Geo {
  static constexpr int STAGES = NT == 1 ? 3 : 2;
  static constexpr int NQ = 8 * NT;             // queries
  static constexpr int QW = NT == 1 ? 8 : 16;   // of a softmax thread
  static constexpr int WG = NQ / QW;            // softmax warpgroups
  static constexpr int THREADS = 128 * WG + 64;
  static constexpr int N = 16 * NT;             // B columns
  static constexpr int LP = 2, PG = L == 2 ? 2 : 4;  // passes of P (L: of Q) and its groups of limbs
  static constexpr int ON = 8 * PG * NT;             // columns of O
  static constexpr uint32_t OPB = NT * 2048u;        // bytes of one pass's Q operand
  static constexpr uint32_t OPP = ON * 128u;         // and P operand
  static constexpr uint32_t Q_OFF = STAGES * 2 * KBYTES, P_OFF = Q_OFF + L * OPB, SH_OFF = P_OFF + LP * OPP;
  static constexpr uint32_t COLS = NT == 1 ? 64 : NT == 2 ? 128 : 256;  // S twice, O: 48 NT or 64 NT columns
};

struct Meta {  // of a stage's tile
  float ks[TBLK], vs[TBLK];
  float vmax;
  uint32_t ok;  // bit b: block b is there
};

template <int NT, int L>
struct Shared {
  Meta meta[Geo<NT, L>::STAGES];
  alignas(16) float cf[8 * NT], nslope[8 * NT], hif[8 * NT], m[8 * NT], al[8 * NT];  // nslope: negated; m: reference R
  alignas(16) float nref[8 * NT], shift[8 * NT];  // -m, 0 for -inf; what a raise moves scores by
  float over[8 * NT];  // a bound on (largest score - m)
  uint32_t fresh[2];  // per warpgroup: some query that may still meet a key has met none
  int32_t hi[8 * NT], lo[8 * NT];
  int64_t place[8 * NT];
  float2 ml[8 * NT];
  float wred[4][8 * NT], wtop[4 * NT];
  uint32_t nan[2][4];
  uint64_t fullk[3], fullv[3], empty[3], sfull[2], pfull, pvdone, qfull, fin;
  int64_t wsum[12];
  uint32_t tslot;
  int abort;
};

// Operand descriptor: layout 0 no swizzle, 2 the 128-byte swizzle.
__device__ __forceinline__ uint64_t sdesc(uint32_t addr, uint32_t lbo, uint32_t sbo, uint32_t layout) {
  return umma_sdesc(addr, lbo, sbo) | ((uint64_t)layout << 61);
}
// kind::f8f6f4 (e4m3 A; e4m3 or e5m2 B, by the descriptor), fp32 accumulators.
__device__ __forceinline__ void umma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
// Barriers of one softmax warpgroup (1 + wg) and of all of them (3, `n` threads),
// and the same with an OR of a predicate.
__device__ __forceinline__ void ssync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }
__device__ __forceinline__ bool ssync_or(int id, int n, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\tbar.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(n), "r"((uint32_t)x)
      : "memory");
  return r != 0;
}
// Largest of the warp's values (a NaN counts as the largest).
__device__ __forceinline__ float warp_fmax(float x) {
  const int b = __float_as_int(x), k = b ^ ((b >> 31) & 0x7fffffff);  // ordered as the values
  const int t = __reduce_max_sync(FULL, k);
  return __int_as_float(t ^ ((t >> 31) & 0x7fffffff));
}

// Sums over the warp of N values per lane: lane q ends with value q's in v[0].
// Every step halves the values a lane carries (N + log2(32 / N) shuffles).
template <int N>
__device__ __forceinline__ void warp_sums(float (&v)[N]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = N / 2; n > 0; n >>= 1) {
    const bool up = lane & n;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float give = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
      v[i] = keep + __shfl_xor_sync(FULL, give, n);
    }
  }
#pragma unroll
  for (int o = N; o < 32; o <<= 1) v[0] += __shfl_xor_sync(FULL, v[0], o);
}

// Two fp32 values in a register pair and the instructions that take both.
struct F2 {
  uint64_t u;
  __device__ __forceinline__ F2() {}
  __device__ __forceinline__ F2(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(u) : "f"(a), "f"(b)); }
  __device__ __forceinline__ explicit F2(float a) : F2(a, a) {}
  __device__ __forceinline__ void get(float& a, float& b) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(u)); }
};
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.u) : "l"(a.u), "l"(b.u), "l"(c.u));
  return d;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.u) : "l"(a.u), "l"(b.u));
  return d;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.u) : "l"(a.u), "l"(b.u));
  return d;
}

__device__ __forceinline__ float2 ld2(const float* p) { return *reinterpret_cast<const float2*>(p); }

// Eight values as e4m3 codes (byte i = value i), and what they leave.
__device__ __forceinline__ uint2 limb8(float (&v)[8], bool rest) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t a = f32x2_e4m3x2(v[4 * i], v[4 * i + 1]), b = f32x2_e4m3x2(v[4 * i + 2], v[4 * i + 3]);
    w[i] = __byte_perm(a, b, 0x5410);
    if (rest) {
      uint32_t lo, hi;
      e4m3x4_f16x2(w[i], lo, hi);
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&lo));
      const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&hi));
      v[4 * i] -= x.x;
      v[4 * i + 1] -= x.y;
      v[4 * i + 2] -= y.x;
      v[4 * i + 3] -= y.y;
    }
  }
  return make_uint2(w[0], w[1]);
}

// fp16 values (pairs) as e5m2 limbs.  e5m2 is the top byte of fp16, so that a
// limb is a byte permute and what it leaves one exact subtraction: each limb the
// next 3 significant bits, cut off.
__device__ __forceinline__ uint32_t h2_bits(__half2 x) { return *reinterpret_cast<const uint32_t*>(&x); }
__device__ __forceinline__ __half2 h2_of(uint32_t x) { return *reinterpret_cast<const __half2*>(&x); }
__device__ __forceinline__ uint2 limb8h(const uint32_t (&h)[4]) {
  return make_uint2(__byte_perm(h[0], h[1], 0x7531), __byte_perm(h[2], h[3], 0x7531));
}
__device__ __forceinline__ void drop_limb(uint32_t (&h)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = h2_bits(__hsub2(h2_of(h[i]), h2_of(h[i] & 0xff00ff00u)));
}

// A CTA's segments: runs of blocks of one unit.
struct Segs {
  int64_t x, end;
  int r;
  // the current segment
  Req rq;
  int h, qc, c0, c1;
  bool direct;
  int64_t rec;
  __device__ __forceinline__ bool next(const AttArgs& A, const int64_t* pre) {
    if (x >= end) return false;
    if (A.cluster) {
      const ClusterPart part(A);
      int u = part.unit;
      qc = u % A.nqc;
      u /= A.nqc;
      h = u % A.Hkv;
      r = u / A.Hkv;
      rq = load_req(A, r);
      x = end;
      if (qc >= unit_groups(A, rq)) return false;
      part.blocks(A, rq, c0, c1);
      direct = A.cluster == 1;
      rec = 0;
      return true;
    }
    for (;;) {
      while (pre[r + 1] <= x) ++r;
      rq = load_req(A, r);
      int unit, cnt;
      if (!share_segment(A, rq, pre[r], x, end, unit, c0, cnt)) {
        if (x >= end) return false;
        continue;
      }
      const int per_head = unit_groups(A, rq);
      h = per_head == 1 ? unit : unit / per_head;
      qc = unit - h * per_head;
      c1 = c0 + cnt;
      direct = cnt == rq.b1 - rq.b0;
      rec = blockIdx.x + (int64_t)r * A.Hkv * A.nqc + unit;
      return true;
    }
  }
};

// EX: 0 plain scores, 1 a distance bias, 2 a cap (and a bias).
template <int DT, int EX, int NT>
__global__ void __launch_bounds__(Geo<NT, DT == DDL_T_F32 ? 3 : 2>::THREADS, 2) kv8_tc_kernel(const __grid_constant__ TcAtt P) {
  constexpr int L = DT == DDL_T_F32 ? 3 : 2;
  constexpr float BSCALE = DT == DDL_T_F32 ? 4096.f : 256.f;  // 16^L (of Q and of P)
  using G = Geo<NT, L>;
  constexpr int NQ = G::NQ, QW = G::QW, WG = G::WG, NS = 128 * WG, LP = G::LP, PG = G::PG;  // NS: softmax threads
  constexpr int CW = 4 * WG, MW = 4 * WG + 1;                         // the copying and the MMA warp
  extern __shared__ __align__(1024) uint8_t smem[];
  Shared<NT, L>& S = *reinterpret_cast<Shared<NT, L>*>(smem + G::SH_OFF);
  int64_t* const pre = reinterpret_cast<int64_t*>(smem + G::SH_OFF + ((sizeof(Shared<NT, L>) + 15) & ~size_t(15)));
  const AttArgs& A = P.A;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sb = smem_addr(smem);
  const uint32_t fullk = smem_addr(S.fullk), fullv = smem_addr(S.fullv), empty = smem_addr(S.empty);
  const uint32_t sfull = smem_addr(S.sfull), pfull = smem_addr(&S.pfull), pvdone = smem_addr(&S.pvdone);
  const uint32_t qfull = smem_addr(&S.qfull);
  if (tid == 0) {
    for (int i = 0; i < G::STAGES; ++i) {
      mbar_init(fullk + 8 * i, 1);
      mbar_init(fullv + 8 * i, 1);
      mbar_init(empty + 8 * i, 1);
    }
    mbar_init(sfull, 1);
    mbar_init(sfull + 8, 1);
    mbar_init(pfull, 4 * WG);
    mbar_init(pvdone, 1);
    mbar_init(qfull, 4 * WG);
    mbar_init(smem_addr(&S.fin), 1);
    S.abort = 0;
  }
  mbar_init_fence();
  if (warp == MW) tmem_alloc(smem_addr(&S.tslot), G::COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = S.tslot, tO = tm + 2 * G::N;
  pdl_wait();
  pdl_trigger();
  Segs first;
  first.x = 0;
  first.end = 1;
  first.r = 0;
  if (!A.cluster) {
    const int64_t W = unit_prefix<G::THREADS>(A, pre, S.wsum);
    const int64_t n = share_count(A, W);
    if ((int64_t)blockIdx.x >= n || W == 0) {
      first.end = 0;
    } else {
      share_bounds(W, n, first.x, first.end);
      for (int hi = A.R; hi - first.r > 1;) {  // the last r with pre[r] <= x
        const int mid = (first.r + hi) >> 1;
        if (pre[mid] <= first.x) first.r = mid;
        else hi = mid;
      }
    }
  } else if (tid == 0 && A.bad) {
    if (load_req(A, blockIdx.x / A.cluster / A.nqc / A.Hkv).bad) atomicOr(A.bad, 1);
  }
  auto fail = [&]() {
    if (lane == 0 && A.bad) atomicOr(A.bad, 2);
    *reinterpret_cast<volatile int*>(&S.abort) = 1;
  };
  auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
    uint64_t t0 = 0;
    for (uint32_t it = 1;; ++it) {
      if (__all_sync(FULL, mbar_try_wait(bar, parity))) return true;
      if ((it & 1023u) == 0) {
        const uint64_t now = __shfl_sync(FULL, globaltimer(), 0);
        if (t0 == 0) t0 = now;
        if (now - t0 > P.wait_ns || __any_sync(FULL, *reinterpret_cast<volatile int*>(&S.abort))) {
          fail();
          return false;
        }
      }
    }
  };

  if (warp == CW) {  // -------------------------------------------------- copies
    // Codes that one unit alone reads leave L2 first (64 requests of up to 8192 tokens 96.9 us, else 100.8), others not
    // (64 rows of 16 requests 286 us, else 295).
    const uint64_t policy = A.nqc == 1 ? policy_evict_first() : policy_evict_normal();
    const int bshift = A.pshift - 4, bmask = (1 << bshift) - 1;
    uint32_t tc = 0;
    bool ok = true;
    Segs s = first;
    while (ok && s.next(A, pre)) {
      const int nblk = s.c1 - s.c0;
      auto page_of = [&](int i) -> int32_t {  // page of the segment's block i from the newest, -1: none
        if (i >= nblk) return -1;
        const int32_t page = A.table[(int64_t)s.r * A.per + ((s.c1 - 1 - i) >> bshift)];
        if (page >= 0 && page < A.pages) return page;
        if (A.bad) atomicOr(A.bad, 1);
        return -1;
      };
      // tokens that some query of the unit sees: V scales of blocks without any do not count
      const int qa = s.qc * NQ, qb = (s.rq.n * A.GH < qa + NQ ? s.rq.n * A.GH : qa + NQ) - 1;
      const int last_key = s.rq.p0 + group_row(A, qb);
      const int64_t first_key = first_seen(A, s.rq, qa);
      int32_t page = page_of(lane), page_n = -1;
      for (int g0 = 0; ok && g0 < nblk; g0 += 32) {  // lane l: block g0 + l
        const int sub = (s.c1 - 1 - g0 - lane) & bmask;
        const int64_t head = (int64_t)page * A.Hkv + s.h;
        float ks = 0.f, vs = 0.f;
        if (page >= 0) {
          ks = A.ks[(head << bshift) + sub];
          vs = A.vs[(head << bshift) + sub];
          check_scales(ks, vs);
          const int key = (s.c1 - 1 - g0 - lane) * 16;
          if (key > last_key || key + 15 < first_key) vs = 0.f;
        }
        const int32_t row = page >= 0 ? (int32_t)((head << A.pshift) + (sub << 4)) : P.rows;  // (none: zeros)
        page_n = page_of(g0 + 32 + lane);
        float vmax = vs;  // of the lane's tile
#pragma unroll
        for (int o = 1; o < TBLK; o <<= 1) vmax = fmaxf(vmax, __shfl_xor_sync(FULL, vmax, o));
        const uint32_t there = __ballot_sync(FULL, page >= 0);
        for (int t = 0; t < 4 && g0 + t * TBLK < nblk; ++t, ++tc) {
          const uint32_t st = tc % G::STAGES, k = tc / G::STAGES;
          if (k > 0 && !wait(empty + 8 * st, (k - 1) & 1)) {
            ok = false;
            break;
          }
          const uint32_t okm = (there >> (t * TBLK)) & 0xffu;
          const bool mine = (lane / TBLK) == t;
          if (mine) {
            S.meta[st].ks[lane % TBLK] = ks;
            S.meta[st].vs[lane % TBLK] = vs;
            if (lane % TBLK == 0) {
              S.meta[st].vmax = vmax;
              S.meta[st].ok = okm;
            }
          }
          __syncwarp();
          if (lane == 0) {
            mbar_arrive_expect_tx(fullk + 8 * st, KBYTES);
            mbar_arrive_expect_tx(fullv + 8 * st, KBYTES);
          }
          __syncwarp();
          if (mine) {
            const uint32_t dst = sb + st * 2 * KBYTES + (lane % TBLK) * 2048u;
            tensor2d_g2s(dst, &P.kmap, 0, row, fullk + 8 * st, policy);
            tensor2d_g2s(dst + KBYTES, &P.vmap, 0, row, fullv + 8 * st, policy);
          }
        }
        page = page_n;
      }
    }
    // copies in flight land before the CTA leaves (bounded)
    if (lane == 0)
      for (uint32_t j = tc > G::STAGES ? tc - G::STAGES : 0; j < tc; ++j) {
        if (!mbar_wait_thread(fullk + 8 * (j % G::STAGES), (j / G::STAGES) & 1, DRAIN_NS)) break;
        if (!mbar_wait_thread(fullv + 8 * (j % G::STAGES), (j / G::STAGES) & 1, DRAIN_NS)) break;
      }
  } else if (warp == MW) {  // ------------------------------------------ MMA issue
    constexpr uint32_t IDESC_S = (1u << 4) | ((uint32_t)(G::N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
    // P e5m2; A and B M/N-major
    constexpr uint32_t IDESC_O = (1u << 4) | ((uint32_t)(G::ON >> 3) << 17) | ((uint32_t)(128 >> 4) << 24) | (1u << 10) |
                                 (1u << 15) | (1u << 16);
    const uint64_t kd = sdesc(sb, 16, 1024, 2), vd = sdesc(sb + KBYTES, 16384, 1024, 2);
    const uint64_t qd = sdesc(sb + G::Q_OFF, 16, 1024, 2), pd = sdesc(sb + G::P_OFF, 128, 2048, 0);
    uint32_t tc = 0, sg = 0;
    bool ok = true;
    Segs s = first;
    auto scores = [&](uint32_t i) -> bool {  // S of tile i
      const uint32_t st = i % G::STAGES;
      if (!wait(fullk + 8 * st, (i / G::STAGES) & 1)) return false;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t a = kd + (uint64_t)(st * (2 * KBYTES >> 4));
        const uint32_t d = tm + (i & 1) * G::N;
#pragma unroll
        for (int p = 0; p < L; ++p)
#pragma unroll
          for (int k = 0; k < 4; ++k)  // 32 head dimensions each
            umma_f8(d, a + 2 * k, qd + (uint64_t)(p * (G::OPB >> 4)) + 2 * k, IDESC_S, p + k > 0 ? 1u : 0u);
        umma_commit(sfull + 8 * (i & 1));
      }
      __syncwarp();
      return true;
    };
    while (ok && s.next(A, pre)) {
      const int nt = (s.c1 - s.c0 + TBLK - 1) / TBLK;
      if (!(ok = wait(qfull, sg & 1))) break;
      ++sg;
      if (nt > 0) ok = scores(tc);
      for (int i = 0; ok && i < nt; ++i, ++tc) {
        if (i + 1 < nt && !(ok = scores(tc + 1))) break;
        const uint32_t st = tc % G::STAGES;
        if (!(ok = wait(fullv + 8 * st, (tc / G::STAGES) & 1))) break;
        if (!(ok = wait(pfull, tc & 1))) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t a = vd + (uint64_t)(st * (2 * KBYTES >> 4));
#pragma unroll
          for (int p = 0; p < LP; ++p)
#pragma unroll
            for (int k = 0; k < 4; ++k)  // 32 tokens each
              umma_f8(tO, a + k * (4096 >> 4), pd + (uint64_t)(p * (G::OPP >> 4)) + k * (512 >> 4), IDESC_O,
                      i + p + k > 0 ? 1u : 0u);
          umma_commit(empty + 8 * st);
          umma_commit(pvdone);
        }
        __syncwarp();
      }
    }
    // every MMA issued has completed before tensor memory is released
    if (elect_one()) umma_commit(smem_addr(&S.fin));
    __syncwarp();
    mbar_wait_thread(smem_addr(&S.fin), 0, DRAIN_NS);
    __syncwarp();
  } else {  // ------------------------------------------------------------ softmax
    const int wg = warp >> 2, tok = tid & 127, x0 = wg * QW;  // queries x0 .. x0 + QW - 1 of the unit
    uint32_t tc = 0;
    bool ok = true;
    Segs s = first;
    const uint32_t tlane = (uint32_t)(32 * (warp & 3)) << 16, tSq = tm + tlane + 2 * x0, tOq = tO + tlane + PG * x0;
    // A wait that gives up makes its warp go on without waiting, so that none is
    // left at a barrier; the results of that segment and of the CTA's later ones
    // become NaN, also in the records that the join adds up.
    while (s.next(A, pre)) {
      const int nqueries = s.rq.n * A.GH, q0 = s.qc * NQ;
      const int nblk = s.c1 - s.c0, nt = (nblk + TBLK - 1) / TBLK;
      ssync(3, NS);  // the previous segment's readers of the shared values are done
      // Q's limbs: 16 lanes a query, 8 head dimensions each; the loads of all rounds go out together
      constexpr int ROUNDS = NQ / (8 * WG);
      float4 qv[ROUNDS][2];
#pragma unroll
      for (int u = 0; u < ROUNDS; ++u) {
        const int qi = q0 + warp * 2 + (lane >> 4) + u * 8 * WG;
        qv[u][0] = qv[u][1] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (qi < nqueries) {
          const int row = group_row(A, qi), head = s.h * A.GH + qi - row * A.GH;
          const int64_t at = (int64_t)(s.rq.row0 + row) * A.q_stride + (int64_t)head * 128 + (lane & 15) * 8;
          qv[u][0] = load_elem4<DT>(A.q, at);
          qv[u][1] = load_elem4<DT>(A.q, at + 4);
        }
      }
#pragma unroll
      for (int u = 0; u < ROUNDS; ++u) {
        const int x = warp * 2 + (lane >> 4) + u * 8 * WG, qi = q0 + x, c = lane & 15;
        const bool has = qi < nqueries;
        const int row = has ? group_row(A, qi) : 0, head = s.h * A.GH + (has ? qi - row * A.GH : 0);
        float v[8] = {qv[u][0].x, qv[u][0].y, qv[u][0].z, qv[u][0].w, qv[u][1].x, qv[u][1].y, qv[u][1].z, qv[u][1].w};
        float mx = 0.f;
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          mx = fmaxf(mx, fabsf(v[i]));
          bad = bad || !(fabsf(v[i]) < INFINITY);
        }
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, o));
        int e = (int)((__float_as_uint(mx) >> 23) & 255u) - 127 - 7;  // the largest lands in [2^7, 2^8)
        e = e < -100 ? -100 : e > 120 ? 120 : e;
        const float down = __uint_as_float((uint32_t)(127 - e) << 23), up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= down;
        if (bad) v[0] = __uint_as_float(0x7fffffffu);  // (an infinity would saturate)
        const int n = (x >> 3) * 16 + (x & 7);
#pragma unroll
        for (int p = 0; p < 2 * L; ++p) {
          const uint2 w = limb8(v, true);
          if (p == L - 1) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= BSCALE;
          }
          const int nn = n + (p >= L ? 8 : 0);
          *reinterpret_cast<uint2*>(smem + G::Q_OFF + (p % L) * G::OPB + nn * 128 + (((c >> 1) ^ (nn & 7)) << 4) +
                                    (c & 1) * 8) = w;
        }
        if (c == 0) {
          const int p = s.rq.p0 + row;
          float cf = up * A.scale;
          if (EX == 2) cf = __fdiv_rn(cf, A.softcap);
          else cf *= LOG2E;
          S.cf[x] = cf;
          if (EX) {
            S.nslope[x] = A.slopes && has ? -A.slopes[head] * LOG2E : 0.f;
            S.hif[x] = (float)(p - s.c1 * 16);
          }
          S.hi[x] = has ? p : -1;
          S.lo[x] = A.window > 0 ? p - A.window + 1 : 0;
          S.m[x] = -INFINITY;
          S.nref[x] = 0.f;
          S.over[x] = -INFINITY;
        }
      }
      fence_proxy_async_smem();
      ssync(3, NS);
      if (lane == 0) mbar_arrive(qfull);
      const int last = (nqueries < q0 + NQ ? nqueries : q0 + NQ) - 1;
      const int all_hi = s.rq.p0 + group_row(A, q0), any_hi = s.rq.p0 + group_row(A, last);
      const int all_lo = A.window > 0 ? any_hi - A.window + 1 : 0;

      F2 l[QW / 2];
#pragma unroll
      for (int q = 0; q < QW / 2; ++q) l[q] = F2(0.f);
      float vref = 0.f, vinv = 0.f;  // unit of O and its inverse
      float tops = -INFINITY;        // largest score less its reference since that was last raised
      for (int i = 0; i < nt; ++i, ++tc) {
        const uint32_t st = tc % G::STAGES;
        ok = ok && wait(fullk + 8 * st, (tc / G::STAGES) & 1);  // (the tile's scales)
        const Meta& M = S.meta[st];
        const int blk = tok >> 4;
        const float ks = M.ks[blk], vs = M.vs[blk], vmax = M.vmax;
        const uint32_t okm = M.ok;
        const int newest = s.c1 - 1 - i * TBLK;  // block; the tile's others lie before it
        const int key = (newest - blk) * 16 + (tok & 15);
        const float back_of = (float)(s.c1 * 16 - key);
        ok = ok && wait(sfull + 8 * (tc & 1), (tc >> 1) & 1);
        tc_fence_after();
        float sc[QW];  // score less the running maximum's stand-in
        {
          uint32_t v[QW / 8][16];
#pragma unroll
          for (int j = 0; j < QW / 8; ++j) tmem_ld_32x32b_x16(tSq + (tc & 1) * G::N + 16 * j, v[j]);
          tmem_ld_wait();
          const F2 ks2(ks), far2(back_of), down2(1.f / BSCALE);
#pragma unroll
          for (int q = 0; q < QW; q += 2) {
            const uint32_t* w = &v[q / 8][q & 7];
            const float2 cf = ld2(&S.cf[x0 + q]), nr = ld2(&S.nref[x0 + q]);
            const F2 f = mul2(ks2, F2(cf.x, cf.y));
            F2 x = fma2(F2(__uint_as_float(w[8]), __uint_as_float(w[9])), down2, F2(__uint_as_float(w[0]), __uint_as_float(w[1])));
            if (EX == 0) {
              x = fma2(x, f, F2(nr.x, nr.y));
            } else {
              const float2 ns = ld2(&S.nslope[x0 + q]), hf = ld2(&S.hif[x0 + q]);
              x = mul2(x, f);
              if (EX == 2) {
                float a, b;
                x.get(a, b);
                x = mul2(F2(A.softcap * LOG2E), F2(tanhf(a), tanhf(b)));
              }
              x = fma2(F2(ns.x, ns.y), add2(F2(hf.x, hf.y), far2), x);  // (distances: exact to 2^24)
              x = add2(x, F2(nr.x, nr.y));
            }
            x.get(sc[q], sc[q + 1]);
          }
        }
        const bool there = (okm >> blk) & 1u;
        const int oldest = newest - TBLK + 1 > s.c0 ? newest - TBLK + 1 : s.c0;
        if (newest * 16 + 15 > all_hi || oldest * 16 < all_lo) {  // some query does not see some token
          // V rows that no query sees must not hold NaN codes, and a NaN code of
          // one that some see reaches exactly those, through their scores
          const bool dead = !there || key > any_hi;
          if (wg == 0) {
            ok = ok && wait(fullv + 8 * st, (tc / G::STAGES) & 1);
            uint4* row = reinterpret_cast<uint4*>(smem + st * 2 * KBYTES + KBYTES + tok * 128);
            bool nan = false;
#pragma unroll 2
            for (int c = 0; c < 8; ++c) {
              uint4 w = dead ? make_uint4(0u, 0u, 0u, 0u) : row[c];
              const uint32_t a = nan_bytes(w.x), b = nan_bytes(w.y), d = nan_bytes(w.z), e = nan_bytes(w.w);
              nan = nan || (a | b | d | e);
              w = make_uint4(w.x & ~a, w.y & ~b, w.z & ~d, w.w & ~e);
              if (dead || (a | b | d | e)) row[c] = w;
            }
            const uint32_t nans = __ballot_sync(FULL, nan);
            if (lane == 0) S.nan[tc & 1][warp] = nans;
          }
          ssync(3, NS);
          const bool nan = (S.nan[tc & 1][warp & 3] >> lane) & 1u;
#pragma unroll
          for (int q = 0; q < QW; ++q) {
            if (dead || key > S.hi[x0 + q] || key < S.lo[x0 + q]) sc[q] = -INFINITY;
            else if (nan) sc[q] = __uint_as_float(0x7fffffffu);
          }
        } else if (!there) {  // past the segment's blocks, or a page that is none: zeros in K and V
#pragma unroll
          for (int q = 0; q < QW; ++q) sc[q] = -INFINITY;
        }
        const bool unit_up = vmax > 0.f && vmax >= 2.f * vref;
        float lv = scale_log(vs * vinv);
        bool over = unit_up || i == 0 || S.fresh[wg];
        float top = sc[0];
#pragma unroll
        for (int q = 1; q < QW; ++q) top = fmaxf(top, sc[q]);
        over = over || top > fminf(T_LAG - lv, P_TOP);
        bool waited = tc == 0;
        if (ssync_or(1 + wg, 128, over)) {  // raise the reference (and V's unit): O and l in the new units
          const float nref = unit_up ? pow2_floor(vmax) : vref, fv = unit_up ? vref * pow2_inv(nref) : 1.f;
          const float down = unit_up && vref > 0.f ? pow2_log_ratio(nref, vref) : 0.f;
          if (unit_up) {
            vref = nref;
            vinv = pow2_inv(nref);
            lv = scale_log(vs * vinv);
          }
#pragma unroll
          for (int q = 0; q < QW; ++q) {
            const float x = warp_fmax(sc[q] + lv);
            if (lane == 0) S.wred[warp & 3][x0 + q] = x;
          }
          tops = warp_fmax(tops);
          if (lane == 0) S.wtop[warp] = tops;
          ssync(1 + wg, 128);
          if (tok < QW) {
            const int x = x0 + tok;
            const float old = S.m[x], ref = -S.nref[x];
            const float up = fmaxf(fmaxf(S.wred[0][x], S.wred[1][x]), fmaxf(S.wred[2][x], S.wred[3][x]));
            const float* const wt = &S.wtop[4 * wg];
            const float most = fmaxf(S.over[x], fmaxf(fmaxf(wt[0], wt[1]), fmaxf(wt[2], wt[3])));
            const float kept = old + fmaxf(-down, most - P_SPAN);  // (a new unit makes all products so far smaller)
            const float nm = fmaxf(down > 0.f ? kept : old, ref + up), now = nm == -INFINITY ? 0.f : nm;
            S.over[x] = old == -INFINITY ? -INFINITY : most + (old - nm);
            S.al[x] = old == -INFINITY ? 0.f : exp2_fast(old - nm);
            S.m[x] = nm;
            S.nref[x] = -now;
            S.shift[x] = ref - now;
            const bool none = nm == -INFINITY && S.hi[x] >= s.c0 * 16;
            const uint32_t any = __ballot_sync((1u << QW) - 1u, none);
            if (tok == 0) S.fresh[wg] = any;
          }
          if (!waited) ok = ok && wait(pvdone, (tc - 1) & 1);
          waited = true;
          ssync(1 + wg, 128);
          top = -INFINITY;
          tops = -INFINITY;
#pragma unroll
          for (int q = 0; q < QW; ++q) {
            sc[q] += S.shift[x0 + q];
            top = fmaxf(top, sc[q]);
          }
#pragma unroll
          for (int q = 0; q < QW; q += 2) l[q / 2] = mul2(l[q / 2], F2(S.al[x0 + q], S.al[x0 + q + 1]));
          if (i > 0) {
            tc_fence_after();
#pragma unroll
            for (int j = 0; j < QW * PG / 16; ++j) {  // 16 columns: two groups of 8 queries
              uint32_t v[16];
              tmem_ld_32x32b_x16(tOq + 16 * j, v);
              tmem_ld_wait();
#pragma unroll
              for (int q = 0; q < 16; ++q)
                v[q] = __float_as_uint(__uint_as_float(v[q]) * (S.al[x0 + 8 * (j / (PG / 2)) + (q & 7)] * fv));
              tmem_st_32x32b_x16(tOq + 16 * j, v);
            }
            tmem_st_wait();
          }
        }
        tops = fmaxf(tops, top);
        // the tile's weights, and their limbs as the PV operand (whose place is
        // free once the previous tile's PV MMAs are done)
        const F2 wv2(vs * vinv * TP_SCALE<L>);
        uint4 pk[QW / 8][LP][PG / 2];
#pragma unroll
        for (int j = 0; j < QW / 8; ++j) {
          float w[8];
#pragma unroll
          for (int q = 0; q < 8; q += 2) {
            const F2 p(exp2_fast(sc[8 * j + q]), exp2_fast(sc[8 * j + q + 1]));
            l[4 * j + q / 2] = add2(l[4 * j + q / 2], p);
            mul2(p, wv2).get(w[q], w[q + 1]);
          }
          uint2 limb[PG][LP];
          uint32_t h[4];  // fp16 (2^-11), 11 bits, as four limbs: exactly
#pragma unroll
          for (int q = 0; q < 4; ++q) h[q] = pack_f16x2(w[2 * q], w[2 * q + 1]);
          if (L == 2) {
            limb[0][0] = limb8h(h);
            drop_limb(h);
            limb[0][1] = limb8h(h);
            drop_limb(h);
#pragma unroll
            for (int q = 0; q < 4; ++q) h[q] = h2_bits(__hmul2(h2_of(h[q]), h2_of(0x5c005c00u)));  // times 256
            limb[1][0] = limb8h(h);
            drop_limb(h);
            limb[1][1] = limb8h(h);
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) {  // what the fp16 leaves
              const float2 f = __half22float2(h2_of(h[q]));
              w[2 * q] -= f.x;
              w[2 * q + 1] -= f.y;
            }
#pragma unroll
            for (int p = 0; p < 4; ++p) {
              limb[p / 2][p & 1] = limb8h(h);
              drop_limb(h);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {  // (and its last limb below e5m2's smallest step)
              const float2 f = __half22float2(h2_of(h[q]));
              h[q] = pack_f16x2((w[2 * q] + f.x) * BSCALE, (w[2 * q + 1] + f.y) * BSCALE);
            }
#pragma unroll
            for (int p = 0; p < 4; ++p) {
              limb[(2 + p / 2) % PG][p & 1] = limb8h(h);
              if (p < 3) drop_limb(h);
            }
          }
#pragma unroll
          for (int p = 0; p < LP; ++p)
#pragma unroll
            for (int g = 0; g < PG; g += 2)
              pk[j][p][g / 2] = make_uint4(limb[g][p].x, limb[g][p].y, limb[g + 1][p].x, limb[g + 1][p].y);
        }
        if (!waited) ok = ok && wait(pvdone, (tc - 1) & 1);
#pragma unroll
        for (int j = 0; j < QW / 8; ++j)
#pragma unroll
          for (int p = 0; p < LP; ++p)
#pragma unroll
            for (int g = 0; g < PG / 2; ++g)
              *reinterpret_cast<uint4*>(smem + G::P_OFF + p * G::OPP + ((x0 / 8 + j) * (PG / 2) + g) * 2048 + tok * 16) =
                  pk[j][p][g];
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(pfull);
      }
      // the result: thread = head dimension
      float ls[QW];
#pragma unroll
      for (int q = 0; q < QW; q += 2) l[q / 2].get(ls[q], ls[q + 1]);
      warp_sums(ls);  // lane q (and q + QW): the warp's sum of query q
      if (lane < QW) S.wred[warp & 3][x0 + lane] = ls[0];
      if (nt > 0) ok = ok && wait(pvdone, (tc - 1) & 1);
      tc_fence_after();
      ok = !ssync_or(3, NS, !ok);
      if (tok < QW) {  // thread q: the query's place, factor and statistics
        const int x = x0 + tok, qi = q0 + x;
        const float valid = ok ? 1.f : __uint_as_float(0x7fffffffu);
        const float lq = ((S.wred[0][x] + S.wred[1][x]) + (S.wred[2][x] + S.wred[3][x])) * valid, m = S.m[x];
        float f = 1.f / TP_SCALE<L> * valid;
        int64_t place = -1;
        if (qi < nqueries) {
          const int row = group_row(A, qi), head = s.h * A.GH + qi - row * A.GH;
          if (s.direct) {
            place = (int64_t)(s.rq.row0 + row) * A.out_stride + (int64_t)head * 128;
            f = lq != 0.f ? f / lq : 0.f;  // (NaN stays NaN)
            if (A.lse) A.lse[(int64_t)(s.rq.row0 + row) * A.Hq + head] = (m + log2f(lq)) * LN2;
          } else if (!A.cluster) {
            place = (s.rec * NQ + x) * 128;
            *reinterpret_cast<float2*>(A.rec_ml + (s.rec * NQ + x) * 2) = make_float2(m, lq);
          }
        }
        S.al[x] = f;
        S.place[x] = place;
        S.ml[x] = make_float2(m, lq);
      }
      ssync(1 + wg, 128);
#pragma unroll
      for (int j = 0; j < QW / 8; ++j) {
        float sum[8];
        if (nt > 0) {
          uint32_t v[PG / 2][16];
#pragma unroll
          for (int g = 0; g < PG / 2; ++g) tmem_ld_32x32b_x16(tOq + 8 * PG * j + 16 * g, v[g]);
          tmem_ld_wait();
          auto at = [&](int g, int q) { return __uint_as_float(v[g / 2][8 * (g & 1) + q]); };
#pragma unroll
          for (int q = 0; q < 8; ++q)
            sum[q] = PG == 2 ? fmaf(at(1, q), 1.f / BSCALE, at(0, q))
                             : fmaf(at(2 % PG, q) + at(3 % PG, q), 1.f / BSCALE, at(0, q) + at(1, q));
        } else {
#pragma unroll
          for (int q = 0; q < 8; ++q) sum[q] = 0.f;
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int x = x0 + 8 * j + q;
          const int64_t place = S.place[x];
          const float o = sum[q] * S.al[x] * vref;
          if (A.cluster > 1) {  // (the ring of K and V is done with: its copies have landed and been used)
            reinterpret_cast<float*>(smem)[x * 128 + tok] = o;
            continue;
          }
          if (place < 0) continue;
          if (s.direct) store_elem<DT>(A.out, place + tok, o);
          else A.rec_o[place + tok] = o;
        }
      }
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (A.cluster > 1) {
    const ClusterPart part(A);
    if (part.unit % A.nqc < unit_groups(A, load_req(A, part.unit / A.nqc / A.Hkv)))  // (the same for all its CTAs)
      cluster_join<DT, 128>(A, part, sb, 8 * 128 * 4, smem_addr(S.ml), NS);
  }
  if (warp == MW) {
    tc_fence_after();
    tmem_dealloc(tm, G::COLS);
  }
}

template <int DT, int EX>
const void* tc_fn(int nt) {
  return nt == 1 ? (const void*)kv8_tc_kernel<DT, EX, 1> : nt == 2 ? (const void*)kv8_tc_kernel<DT, EX, 2>
                                                                   : (const void*)kv8_tc_kernel<DT, EX, 4>;
}
template <int DT>
const void* tc_fn(int ex, int nt) {
  return ex == 2 ? tc_fn<DT, 2>(nt) : ex == 1 ? tc_fn<DT, 1>(nt) : tc_fn<DT, 0>(nt);
}
template <int NT>
size_t tc_smem(bool f32) {
  return f32 ? Geo<NT, 3>::SH_OFF + sizeof(Shared<NT, 3>) : Geo<NT, 2>::SH_OFF + sizeof(Shared<NT, 2>);
}

size_t tc_smem(int nq, bool f32, int reqs) {
  return (nq == 1 ? tc_smem<1>(f32) : nq == 2 ? tc_smem<2>(f32) : tc_smem<4>(f32)) + 16 +
         (reqs ? (size_t)(reqs + 1) * 8 : 0);
}

int encode_map(CUtensorMap* m, const uint8_t* base, int64_t rows) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return DDL_ERR_CUDA;
  const cuuint64_t dims[2] = {128, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {128};
  const cuuint32_t box[2] = {128, KV8_BLOCK};
  const cuuint32_t es[2] = {1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(base), dims, strides, box, es,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? DDL_OK : DDL_ERR_CUDA;
}

}  // namespace

int kv8_tc_ctas(int nq, bool f32, int reqs) {
  return 2 * (tc_smem(nq, f32, reqs) + 1024) <= 228 * 1024 ? 2 : 1;
}

// rows: of the pool's [pages * H_kv * page_size][128] view, < 2^31.
int kv8_tc_launch(const AttArgs& a, int dtype, int64_t rows, void* stream) {
  TcAtt p;
  p.A = a;
  p.wait_ns = wait_limit_ns();
  p.rows = (int32_t)rows;
  int st;
  if ((st = encode_map(&p.kmap, a.k, rows)) || (st = encode_map(&p.vmap, a.v, rows))) return st;
  const int threads = a.nq == 1 ? Geo<1, 2>::THREADS : a.nq == 2 ? Geo<2, 2>::THREADS : Geo<4, 2>::THREADS;
  const int ex = a.softcap > 0.f ? 2 : a.slopes ? 1 : 0;
  const void* fn = dtype == DDL_T_F32    ? tc_fn<DDL_T_F32>(ex, a.nq)
                   : dtype == DDL_T_BF16 ? tc_fn<DDL_T_BF16>(ex, a.nq)
                                         : tc_fn<DDL_T_F16>(ex, a.nq);
  const bool f32 = dtype == DDL_T_F32;
  const size_t smem = tc_smem(a.nq, f32, a.cluster ? 0 : a.R);
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
  if (e != cudaSuccess) return cuda_status(e);
  if (a.cluster > 8 && (e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess)
    return cuda_status(e);
  void* args[] = {&p};
  return cuda_status(launch_pdl_cluster(fn, dim3((unsigned)a.ctas), dim3((unsigned)threads), args, smem, a.cluster,
                                        (cudaStream_t)stream));
}

}  // namespace ddl
