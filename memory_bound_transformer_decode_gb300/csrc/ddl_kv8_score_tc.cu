// ddl_kv8_score_tc.cu -- the cache scores of requests with many queries (prompt chunks, drafted
// rows) on the tcgen05 tensor cores.
//
// S = K Q^T with 128 tokens as M and up to 256 queries as N, fp16 operands and fp32 accumulators in
// tensor memory: a thread then has one token and adds up the weights of its queries without shuffles.
// Codes (e4m3 and int8 alike) are exact in fp16; Q is scaled by a power of two per query and split as
// in the warp kernel, the remainders of fp32 rows as a second set of MMAs.
//
// Four threads share a token, one of each warpgroup, with every fourth 16 of its queries.  Their sums meet in shared
// memory (`part`), where the first warpgroup adds them up in a fixed order after the CTA's next barrier, the first one of
// the next tile; two tiles' sums lie there, so that the next tile's are left beside those still being read, and the
// barrier of the tile after that orders the ones that take their place.
//
// A CTA of four warpgroups takes one K/V head of a request, all its queries in shared memory (512 16-bit or 256
// fp32 ones of 128 at a time), and tiles of 128 tokens one after the other.  Two accumulators of 256 columns: the
// MMAs of the next 256 queries run while the warpgroups, each with every fourth 16 columns, go over the last ones;
// K tiles are converted a tile ahead, their codes and pages loaded two and three ahead.  N is as wide as it goes, since A
// and B both come from shared memory (128 bytes a clock: 128 x 128 is even with the MMA's own time).  64 rows of 64/8
// heads on 8192 tokens: warpgroups with tiles and accumulators of their own, two of 2 x 128 columns 31.7 us (two warps a
// scheduler: issue slots at 31 %), four of 128 21.8 (all wait at once), four of 2 x 64 24.8.
//
// What bounds it: exponentials (and tanh) of tokens x queries: 64 rows of 28/4 heads of two requests of up to 8192, capped
// scores, 28 us, issue slots at 59 %, tensor pipe at 10 %; without cap 20; fp32 rows (the layer stack's), half as many
// queries at a time, 35 and 28.
#include <cuda_bf16.h>

#include "ddl_kv8_score.h"

namespace ddl {
namespace {

constexpr int TOK = 128, QC = 256;     // tokens of a tile, queries of a chunk
constexpr int WGS = 4, THREADS = 128 * WGS;
constexpr int TMEM = 2 * QC;           // columns
constexpr uint64_t DRAIN_NS = 10000000000ull;

// D (+)= A B from shared memory, kind::f16.
__device__ __forceinline__ void umma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// Waits for the tensor-memory loads on their way; what v holds is used behind it.
__device__ __forceinline__ void landed(uint32_t (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
               :
               : "memory");
}
// Operands in shared memory: panels of 64 elements, a row of a panel 128 bytes whose 16-byte pieces are exchanged by
// the row's low bits (the 128-byte swizzle of the MMA's descriptor): a row's pieces, written by neighbouring lanes as they
// read them, and a column of 8 rows both fall on different banks.
__device__ __forceinline__ uint32_t piece_at(int rows, int row, int k8) {  // k8: piece of 8 elements
  return (uint32_t)(k8 >> 3) * rows * 128 + row * 128 + (((k8 & 7) ^ (row & 7)) << 4);
}
__device__ __forceinline__ uint64_t panel_desc(uint32_t addr) { return umma_sdesc(addr, 16, 1024) | (2ull << 61); }

// Dynamic shared memory: Q (and its remainders), two K tiles, the columns, the warpgroups' sums of two tiles.
struct Layout {
  uint32_t qlo, k, cn, slope, range, part, total;
  __host__ __device__ Layout(bool f32, int hd, int nq) {
    const uint32_t q = (uint32_t)nq * hd * 2;
    qlo = q;
    k = f32 ? 2 * q : q;  // (multiples of 1024: nq is one of 16)
    cn = k + 2u * TOK * hd * 2;
    slope = cn + (uint32_t)nq * 8;
    range = slope + (uint32_t)nq * 4;
    part = range + (uint32_t)nq * 8;
    total = part + 2u * WGS * TOK * 4;
  }
};

template <int DT, int HD, bool EX>
__global__ void __launch_bounds__(THREADS, 1) kv8_score_tc_kernel(const __grid_constant__ ScoreArgs S, const int type) {
  constexpr bool HL = DT == DDL_T_F32;
  constexpr int KL = HD / 16, RPL = 32 / KL, NG = 8 / RPL;  // lanes a token's codes take; tokens a load; loads (a warp: 8 tokens)
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[2];
  __shared__ uint32_t tslot;
  __shared__ int silent;  // some query adds nothing (its log-sum-exp is -inf)
  const AttArgs& A = S.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, wg = warp >> 2, tok = tid & 127;
  const Layout M(HL, HD, S.tiles);
  pdl_wait();
  const int r = blockIdx.z, h = blockIdx.y;
  const Req rq = load_req(A, r);
  if (rq.bad && A.bad && blockIdx.x == 0 && h == 0 && tid == 0) atomicOr(A.bad, 1);
  const int nq = rq.n * A.GH;
  float* const out = S.score + ((int64_t)r * A.Hkv + h) * S.stride;
  // tiles [t0, t1) change, [s0, s1) of them hold tokens that some row sees
  const int ntile = (int)(((int64_t)rq.len + TOK - 1) / TOK);  // (lengths up to 2^31 - 16: a tile's last token fits 32 bits)
  const int t0 = max((int)(blockIdx.x * S.wb), S.decay == 1.f ? rq.b0 >> 3 : 0), t1 = min((int)((blockIdx.x + 1) * S.wb), ntile);
  const int s0 = max(t0, rq.b0 >> 3), s1 = min(t1, (rq.b1 + 7) >> 3);
  if (rq.n <= 0 || t0 >= t1) return;  // (the same for the whole CTA)
  if (tid == 0) silent = 0;
  if (tid < 2) mbar_init(smem_addr(&bars[tid]), 1);
  mbar_init_fence();
  if (warp == 0) tmem_alloc(smem_addr(&tslot), TMEM);
  pdl_trigger();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t acc = tslot, bar = smem_addr(&bars[0]);
  uint32_t flying = 0, phase = 0;  // bit a: MMAs into accumulator a are on their way; the parity of their commit
  {
    // the score that a token brings along
    auto old_of = [&](int key) { return key < rq.p0 && key < rq.len && S.decay != 0.f ? out[key] : 0.f; };
    if (wg == 0)  // tiles that nobody sees only decay
      for (int t = t0; t < t1; ++t) {
        const int key = t * TOK + tok;
        if ((t < s0 || t >= s1) && key < rq.len) out[key] = S.decay * old_of(key);
      }
    // This thread's token of a tile: its scale.  The codes of 8 tokens a warp: KL neighbouring lanes a token, so that
    // a load meets whole rows (16 bytes of each of 8 rows a quarter of a warp took four times as long).  All of a
    // tile's loads are on their way before any is used, its pages (of the warp's 8 tokens' block, of the thread's own) a
    // tile ahead.
    const int wtok = warp * 8;  // first token whose codes this warp converts
    uint4 raw[NG];
    float ks = 0.f, was = 0.f;
    bool live = false;
    auto load_page = [&](int t, int x) -> int32_t {  // of token x of tile t
      const int b = (int)(((uint32_t)t * TOK + x) >> 4);  // (t may be one past the last)
      return t < s1 && b >= rq.b0 && b < rq.b1 ? A.table[(int64_t)r * A.per + (b >> (A.pshift - 4))] : -2;
    };
    auto row_of = [&](int32_t page, int t, int x) -> int64_t {
      return page >= 0 && page < A.pages ? (((int64_t)page * A.Hkv + h) << A.pshift) + ((t * TOK + x) & ((1 << A.pshift) - 1)) : -1;
    };
    int32_t page = load_page(s0, tok), wpage = load_page(s0, wtok);
    auto load_codes = [&](int t, bool again) {  // (of tile t, with its pages; then the pages of the next)
      const int64_t row = row_of(page, t, tok), from = row_of(wpage, t, wtok);
      live = row >= 0;
      if (!live && page != -2 && A.bad) atomicOr(A.bad, 1);
      ks = live ? A.ks[row >> 4] : 0.f;
      // (again: the next queries, onto what the first left)
      const int key = t * TOK + tok;
      was = wg > 0 ? 0.f : !again ? old_of(key) : key < rq.len ? out[key] : 0.f;
#pragma unroll
      for (int g = 0; g < NG; ++g)
        raw[g] = from >= 0 ? *reinterpret_cast<const uint4*>(A.k + (from + RPL * g + lane / KL) * HD + (lane % KL) * 16)
                           : make_uint4(0u, 0u, 0u, 0u);
      page = load_page(t + 1, tok);
      wpage = load_page(t + 1, wtok);
    };
    const uint32_t kbuf = smem_addr(smem + M.k);
    auto store_codes = [&](int t) {
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const uint32_t w[4] = {raw[g].x, raw[g].y, raw[g].z, raw[g].w};
        uint32_t f[8];
        if (type == DDL_KV8_E4M3) {
#pragma unroll
          for (int q = 0; q < 4; ++q) codes_f16<DDL_KV8_E4M3>(w[q], f[2 * q], f[2 * q + 1]);
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q) codes_f16<DDL_KV8_INT8>(w[q], f[2 * q], f[2 * q + 1]);
        }
        const int x = wtok + RPL * g + lane / KL, k8 = 2 * (lane % KL);
        const uint32_t to = kbuf + (uint32_t)(t & 1) * TOK * HD * 2;
        sts128(to + piece_at(TOK, x, k8), make_uint4(f[0], f[1], f[2], f[3]));
        sts128(to + piece_at(TOK, x, k8 + 1), make_uint4(f[4], f[5], f[6], f[7]));
      }
    };
    bool ok = true;  // no wait of the CTA gave up
    float2* const cn = reinterpret_cast<float2*>(smem + M.cn);
    float* const slope = reinterpret_cast<float*>(smem + M.slope);
    int2* const range = reinterpret_cast<int2*>(smem + M.range);
    float* const part = reinterpret_cast<float*>(smem + M.part);  // [tile & 1][warpgroup][token]
    for (int g0 = 0; s0 < s1 && g0 < nq; g0 += S.tiles) {
      const int n = min(S.tiles, nq - g0), npad = (n + 15) & ~15, nch = (npad + QC - 1) / QC;
      if (g0 > 0) {
        __syncthreads();  // (the last queries' MMAs are done, their scores written)
        page = load_page(s0, tok);
        wpage = load_page(s0, wtok);
      }
      const float unit = EX && A.softcap > 0.f ? __fdiv_rn(A.scale, A.softcap) : A.scale * LOG2E;
      // Q: a warp takes 4 queries, 8 lanes each, a lane the pieces of 8 elements c and c + 8; all rounds' loads on their
      // way (512 16-bit or 256 fp32 queries of 128)
      constexpr int PC = HD / 64, PW = HL ? 2 : 1, U = HL ? 4 : 8;  // pieces a lane, 16-byte words a piece, rounds
      constexpr int STEP = 4 * 4 * WGS;                             // queries of a round
      const int qr = lane >> 3, qp = lane & 7;
      for (int x0 = warp * 4; x0 == warp * 4 || x0 < npad; x0 += STEP * U) {  // (every warp comes once)
        uint4 in[U][PC][PW];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int qi = g0 + min(x0 + STEP * u + qr, n - 1), row = group_row(A, qi);  // (past the last: not used)
          const uint8_t* const from = reinterpret_cast<const uint8_t*>(A.q) +
              ((int64_t)(rq.row0 + row) * A.q_stride + (int64_t)(h * A.GH + qi - row * A.GH) * HD) * (HL ? 4 : 2);
#pragma unroll
          for (int p = 0; p < PC; ++p)
#pragma unroll
            for (int w = 0; w < PW; ++w) in[u][p][w] = *reinterpret_cast<const uint4*>(from + ((qp + 8 * p) * PW + w) * 16);
        }
        if (x0 == warp * 4) {  // (beside the first round's loads)
          if (tid < npad) {
            const Column c = column_of<EX>(A, rq, h, tid < n ? g0 + tid : nq, 1.f);  // (nq: none)
            cn[tid].y = tid < n ? c.lse2 : INFINITY;
            if (EX) slope[tid] = c.slope;
            range[tid] = make_int2(c.hi, c.lo);
            if (tid < n && c.hi < 0) silent = 1;
          }
          load_codes(s0, g0 > 0);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int x = x0 + STEP * u + qr;
          auto element = [&](int p, int e) -> float {
            const uint4 a = in[u][p][HL ? e >> 2 : 0];
            const int i = HL ? e & 3 : e >> 1;
            const uint32_t w = i == 0 ? a.x : i == 1 ? a.y : i == 2 ? a.z : a.w;
            if (HL) return __uint_as_float(w);
            if (DT == DDL_T_BF16) return e & 1 ? bf16hi_f32(w) : bf16lo_f32(w);
            const __half2 h2 = *reinterpret_cast<const __half2*>(&w);
            return e & 1 ? __high2float(h2) : __low2float(h2);
          };
          float mx = 0.f;
#pragma unroll
          for (int p = 0; p < PC; ++p)
#pragma unroll
            for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(element(p, e)));
          mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 2));
          mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 4));
          int e2 = (int)((__float_as_uint(mx) >> 23) & 255u) - 127 - 12;  // the largest lands in [2^12, 2^13)
          e2 = e2 < -100 ? -100 : e2 > 115 ? 115 : e2;
          const float down = x < n ? __uint_as_float((uint32_t)(127 - e2) << 23) : 0.f;
          if (x < npad) {
#pragma unroll
            for (int p = 0; p < PC; ++p) {
              uint32_t hi[4], lo[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float a = x < n ? element(p, 2 * e) * down : 0.f, b = x < n ? element(p, 2 * e + 1) * down : 0.f;
                hi[e] = pack_f16x2(a, b);
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi[e]));
                lo[e] = pack_f16x2(a - f.x, b - f.y);
              }
              const uint32_t to = smem_addr(smem) + piece_at(S.tiles, x, qp + 8 * p);
              sts128(to, make_uint4(hi[0], hi[1], hi[2], hi[3]));
              if (HL) sts128(to + M.qlo, make_uint4(lo[0], lo[1], lo[2], lo[3]));
            }
            if (qp == 0) cn[x].x = x < n ? __uint_as_float((uint32_t)(127 + e2) << 23) * unit : 0.f;
          }
        }
      }
      // the MMAs of chunk c of tile t into accumulator a
      auto issue = [&](int t, int c, uint32_t a) {
        const uint32_t idesc = umma_idesc_f16(TOK, min(QC, npad - c * QC));
        if (warp == 0) {
          tc_fence_after();
          if (elect_one()) {
            const uint64_t k0 = panel_desc(kbuf) + ((uint32_t)(t & 1) * TOK * HD * 2 >> 4);
            const uint64_t b = panel_desc(smem_addr(smem)) + (uint64_t)(c * QC * 128 >> 4);
            const uint32_t bp = (uint32_t)S.tiles * 128 >> 4;  // from panel to panel of Q
#pragma unroll
            for (int k = 0; k < HD / 16; ++k)
              umma_f16_ss(acc + a * QC, k0 + (k >> 2) * (TOK * 128 >> 4) + 2 * (k & 3), b + (k >> 2) * bp + 2 * (k & 3), idesc,
                          k ? 1u : 0u);
            if (HL) {
              const uint64_t b2 = b + (M.qlo >> 4);
#pragma unroll
              for (int k = 0; k < HD / 16; ++k)
                umma_f16_ss(acc + a * QC, k0 + (k >> 2) * (TOK * 128 >> 4) + 2 * (k & 3), b2 + (k >> 2) * bp + 2 * (k & 3), idesc, 1u);
            }
            umma_commit(bar + 8 * a);
          }
          __syncwarp();
        }
        flying |= 1u << a;
      };
      auto put = [&](int t, float base) {  // the sums of tile t (a barrier after they were left)
        const int key = t * TOK + tok;
        const float* const p = part + (t & 1) * WGS * TOK + tok;
        const float s = (p[0] + p[TOK]) + (p[2 * TOK] + p[3 * TOK]);
        if (key < rq.len) out[key] = base + s;
      };
      store_codes(s0);
      float f = ks, base = was;
      bool has = live;
      fence_proxy_async_smem();
      __syncthreads();
      const bool masks = silent != 0;
      if (ok) issue(s0, 0, 0);
      if (s0 + 1 < s1) load_codes(s0 + 1, g0 > 0);
      uint32_t a = 0;
      float last = 0.f;  // (warpgroup 0) what the last tile's token brought along
      bool late = false;
      for (int t = s0; t < s1; ++t) {
        f = fabsf(f) < INFINITY ? f : __uint_as_float(0x7fffffffu);
        base = g0 == 0 ? S.decay * base : base;
        const int key0 = t * TOK, key = key0 + tok;
        float nf = 0.f, nbase = 0.f;
        bool nhas = false;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        for (int c = 0; c < nch; ++c, a ^= 1) {
          // what comes next: its K, and its MMAs into the accumulator that all have read
          const bool more = c + 1 < nch, next = !more && t + 1 < s1;
          if (next) {
            store_codes(t + 1);
            nf = ks;
            nbase = was;
            nhas = live;
            fence_proxy_async_smem();
          }
          tc_fence_before();
          ok = !__syncthreads_or(late) && ok;
          if (c == 0 && t > s0 && wg == 0) put(t - 1, last);
          if (ok && more) issue(t, c + 1, a ^ 1);
          if (ok && next) issue(t + 1, 0, a ^ 1);
          if (next && t + 2 < s1) load_codes(t + 2, g0 > 0);
          if (!ok) continue;
          {  // (bounded)
            uint64_t since = 0;
            for (uint32_t it = 1; !__all_sync(FULL, mbar_try_wait(bar + 8 * a, phase >> a & 1)); ++it)
              if ((it & 1023u) == 0) {
                const uint64_t now = __shfl_sync(FULL, globaltimer(), 0);
                if (since == 0) since = now;
                else if (now - since > S.wait_ns) {
                  late = true;
                  break;
                }
              }
          }
          if (late) continue;
          flying &= ~(1u << a);
          phase ^= 1u << a;
          tc_fence_after();
          const uint32_t d = acc + a * QC + ((uint32_t)(warp & 3) << 21);
          const int q0 = g0 + c * QC, nc = min(QC, npad - c * QC), q1 = min(q0 + nc, nq) - 1;
          // tokens that every query of the chunk sees need no masks
          const bool edge = masks || key0 + TOK - 1 > rq.p0 + group_row(A, q0) || key0 < first_seen(A, rq, q1);
          const float2* const cc = cn + c * QC;
#pragma unroll 1
          for (int x = 16 * wg; x < nc; x += 16 * WGS) {
            uint32_t v[16];
            tmem_ld_32x32b_x16(d + x, v);
            float2 q[16];  // (two a load)
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              const float4 two = *reinterpret_cast<const float4*>(cc + x + j);
              q[j] = make_float2(two.x, two.y);
              q[j + 1] = make_float2(two.z, two.w);
            }
            landed(v);
            float w[16];
            if (!EX) {
#pragma unroll
              for (int j = 0; j < 16; ++j) w[j] = exp2_fast(fmaf(__uint_as_float(v[j]) * f, q[j].x, -q[j].y));
            } else {
#pragma unroll
              for (int j = 0; j < 16; ++j) w[j] = (__uint_as_float(v[j]) * f) * q[j].x;
              float cap = 1.f;
              if (A.softcap > 0.f) {
                tanh_of(w);
                cap = A.softcap * LOG2E;
              }
              if (A.slopes) {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                  q[j].y = fmaf(slope[c * QC + x + j], (float)(range[c * QC + x + j].x - key), q[j].y);
              }
#pragma unroll
              for (int j = 0; j < 16; ++j) w[j] = exp2_fast(fmaf(w[j], cap, -q[j].y));
            }
            if (edge) {
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const int2 a = range[c * QC + x + j];
                w[j] = key <= a.x && key >= a.y ? w[j] : 0.f;
              }
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) sum[j & 3] += w[j];
          }
        }
        part[((t & 1) * WGS + wg) * TOK + tok] =
            late || !ok ? __uint_as_float(0x7fffffffu) : has ? (sum[0] + sum[1]) + (sum[2] + sum[3]) : 0.f;
        last = base;
        f = nf;
        base = nbase;
        has = nhas;
      }
      tc_fence_before();
      ok = !__syncthreads_or(late) && ok;
      if (wg == 0) put(s1 - 1, last);
    }
    if (!ok && A.bad && tid == 0) atomicOr(A.bad, 2);
    // MMAs in flight end before their memory goes to another
    for (int x = 0; x < 2; ++x)
      if (flying >> x & 1) mbar_wait_thread(bar + 8 * x, phase >> x & 1, DRAIN_NS);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tslot, TMEM);
  }
}

template <int DT>
const void* tc_fn(int hd, bool ex) {
  if (hd == 128) return ex ? (const void*)kv8_score_tc_kernel<DT, 128, true> : (const void*)kv8_score_tc_kernel<DT, 128, false>;
  return ex ? (const void*)kv8_score_tc_kernel<DT, 64, true> : (const void*)kv8_score_tc_kernel<DT, 64, false>;
}

}  // namespace

int kv8_score_tc_launch(const ScoreArgs& s, int type, int dtype, bool ex, int sms, void* stream) {
  ScoreArgs a = s;
  const bool f32 = dtype == DDL_T_F32;
  const int hd = a.a.hd, nq = (a.a.max_rows * a.a.GH + 15) & ~15;
  // queries at a time: what 128 KB hold (with remainders of fp32 rows), a column a thread
  int most = 128 * 1024 / (hd * 2 * (f32 ? 2 : 1));
  most = most < THREADS ? most : THREADS;
  a.tiles = nq < most ? nq : most;
  // tiles a CTA takes: about one wave of CTAs, each of which begins with all queries (several requests, whose lengths are
  // taken to come to 5/8 of the bound: 8/5 waves of it; with other lengths the grain is another, the results are not).
  // Four waves, of 128 bf16 queries a head: 2 requests of up to 8192, 4 heads 21.9 us for 12.7, 16 of 2048 20.3 for 16.8,
  // 16 of 8192, 2 heads 25.9 for 23.8, but 2 of 32768 27.6 for 28.5; of 512, 4 heads: 33.0 for 21.4, 31.2 for 32.1.
  const int64_t tiles = ((int64_t)a.a.max_len + TOK - 1) / TOK, units = (int64_t)a.a.R * a.a.Hkv;
  int64_t ctas = (int64_t)sms * (a.a.R == 1 ? 5 : 8) / 5 / units;
  ctas = ctas < 1 ? 1 : ctas;
  a.wb = (int32_t)((tiles + ctas - 1) / ctas);
  if (a.wb > SCORE_TC_TILES) a.wb = SCORE_TC_TILES;
  const int64_t chunks = (tiles + a.wb - 1) / a.wb;
  const void* fn = dtype == DDL_T_F32    ? tc_fn<DDL_T_F32>(hd, ex)
                   : dtype == DDL_T_BF16 ? tc_fn<DDL_T_BF16>(hd, ex)
                                         : tc_fn<DDL_T_F16>(hd, ex);
  const size_t smem = Layout(f32, hd, a.tiles).total;
  // (the function's limit, which calls of other threads set too: the most that any call of it takes)
  const int st = cuda_status(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Layout(f32, hd, most).total));
  if (st) return st;
  void* args[] = {&a, &type};
  return cuda_status(launch_pdl(fn, dim3((unsigned)chunks, (unsigned)a.a.Hkv, (unsigned)a.a.R), dim3(THREADS), args, smem,
                                (cudaStream_t)stream));
}

}  // namespace ddl
