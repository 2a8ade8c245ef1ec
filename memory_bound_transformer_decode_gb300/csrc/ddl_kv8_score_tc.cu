// ddl_kv8_score_tc.cu -- the cache scores of requests with many queries (prompt chunks, drafted
// rows) on the tcgen05 tensor cores.
//
// S = K Q^T with 128 tokens as M and up to 128 queries as N, fp16 operands and fp32 accumulators in
// tensor memory: a thread then has one token and walks over its queries' scores, so that the sum of
// weights needs no other thread.  Codes (e4m3 and int8 alike) are exact in fp16; Q is scaled by a power
// of two per query and split as in the warp kernel, the remainders of fp32 rows as a second set of MMAs.
//
// A CTA takes one K/V head of a request, all its queries in shared memory (512 16-bit or 256 fp32 ones of 128
// at a time), and two independent warpgroups of 128 threads, each with tiles of 128 tokens of its own: while
// one waits for its MMAs or converts codes, the other takes exponentials.  Each has two accumulators of 128
// columns: the MMAs of the next 128 queries run while it goes over the last ones.
//
// Bound by the exponentials (one MUFU operation a pair: 16 a clock and SM) and the issue of some six instructions
// a pair.
#include <cuda_bf16.h>

#include "ddl_kv8_score.h"

namespace ddl {
namespace {

constexpr int TOK = 128, QC = 128;     // tokens of a tile, queries of a chunk
constexpr int TMEM = 512;              // columns: 2 warpgroups x 2 accumulators x QC
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
__device__ __forceinline__ void wg_sync(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool wg_or(int id, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\tbar.red.or.pred q, %1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"((uint32_t)x)
      : "memory");
  return r != 0;
}

// Operands in shared memory: cores of 8 rows x 16 bytes, those of a row's HD elements side by side.
template <int HD>
struct Core {
  static constexpr uint32_t LBO = 128, SBO = HD / 8 * 128;
  static __device__ __forceinline__ uint32_t at(int row, int k) {
    return (uint32_t)(row >> 3) * SBO + (uint32_t)(k >> 3) * LBO + (row & 7) * 16 + (k & 7) * 2;
  }
};

// Dynamic shared memory: Q (and its remainders), each warpgroup's K tile, the columns, the sums.
struct Layout {
  uint32_t qlo, k, cn, slope, range, part, total;
  __host__ __device__ Layout(bool f32, int hd, int nq, int tiles) {
    const uint32_t q = (uint32_t)nq * hd * 2;
    qlo = q;
    k = f32 ? 2 * q : q;
    cn = k + 2u * TOK * hd * 2;
    slope = cn + (uint32_t)nq * 8;
    range = slope + (uint32_t)nq * 4;
    part = range + (uint32_t)nq * 8;
    total = part + 2u * tiles * TOK * 4;
  }
};

template <int CT, int DT, int HD, bool EX>
__global__ void __launch_bounds__(256, 1) kv8_score_tc_kernel(const __grid_constant__ ScoreArgs S) {
  constexpr bool HL = DT == DDL_T_F32;
  constexpr int NV = HD / 16;  // 16-byte pieces of a token's codes
  using C = Core<HD>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[2][2];
  __shared__ uint32_t tslot;
  const AttArgs& A = S.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, wg = warp >> 2, tok = tid & 127;
  const Layout M(HL, HD, S.tiles, S.wb);
  if (tid == 0) {
    for (int i = 0; i < 4; ++i) mbar_init(smem_addr(&bars[i >> 1][i & 1]), 1);
  }
  mbar_init_fence();
  if (warp == 0) tmem_alloc(smem_addr(&tslot), TMEM);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = tslot;
  pdl_wait();
  pdl_trigger();
  const int r = blockIdx.z, h = blockIdx.y;
  const Req rq = load_req(A, r);
  if (rq.bad && A.bad && blockIdx.x == 0 && h == 0 && tid == 0) atomicOr(A.bad, 1);
  const int ntile = (rq.len + TOK - 1) / TOK, c0 = blockIdx.x * 2 * S.wb;
  const int first = S.decay == 1.f ? rq.b0 >> 3 : 0;  // tiles before it do not change
  const int nq = rq.n * A.GH;
  float* const out = S.score + ((int64_t)r * A.Hkv + h) * S.stride;
  float* const part = reinterpret_cast<float*>(smem + M.part) + (size_t)wg * S.wb * TOK + tok;  // [tile][token]
  if (rq.n > 0 && c0 < ntile && c0 + 2 * S.wb > first) {  // (the same for the whole CTA)
    const int mine = c0 + wg < ntile ? min(S.wb, (ntile - c0 - wg + 1) / 2) : 0;  // tiles c0 + wg + 2 i
    auto key_of = [&](int i) { return (c0 + wg + 2 * i) * TOK + tok; };
    auto seen = [&](int i) {  // does any row see a token of the tile?
      const int b = (c0 + wg + 2 * i) * (TOK / 16);
      return i < mine && b < rq.b1 && b + TOK / 16 > rq.b0;
    };
    // the scores that the tokens bring along
#pragma unroll
    for (int i = 0; i < SCORE_TC_TILES; ++i) {
      if (i >= mine) break;
      const int key = key_of(i);
      part[i * TOK] = key < rq.p0 && key < rq.len && S.decay != 0.f ? S.decay * out[key] : 0.f;
    }
    // this thread's token of a tile: its codes and scale
    uint4 raw[NV];
    float ks = 0.f;
    bool live = false;
    auto load_codes = [&](int i) {
      const int key = key_of(i), b = key >> 4, bshift = A.pshift - 4;
      live = false;
      ks = 0.f;
      if (b >= rq.b0 && b < rq.b1) {
        const int32_t page = A.table[(int64_t)r * A.per + (b >> bshift)];
        live = page >= 0 && page < A.pages;
        if (!live && A.bad) atomicOr(A.bad, 1);
        if (live) {
          const int64_t row = (((int64_t)page * A.Hkv + h) << A.pshift) + (key & ((1 << A.pshift) - 1));
          ks = A.ks[row >> 4];
          if (!(fabsf(ks) < INFINITY)) ks = __uint_as_float(0x7fffffffu);
#pragma unroll
          for (int j = 0; j < NV; ++j) raw[j] = *reinterpret_cast<const uint4*>(A.k + row * HD + j * 16);
        }
      }
      if (!live) {
#pragma unroll
        for (int j = 0; j < NV; ++j) raw[j] = make_uint4(0u, 0u, 0u, 0u);
      }
    };
    const uint32_t kbuf = smem_addr(smem + M.k) + (uint32_t)wg * TOK * HD * 2;
    auto store_codes = [&]() {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
        uint32_t f[8];
#pragma unroll
        for (int q = 0; q < 4; ++q) codes_f16<CT>(w[q], f[2 * q], f[2 * q + 1]);
        sts128(kbuf + C::at(tok, 16 * j), make_uint4(f[0], f[1], f[2], f[3]));
        sts128(kbuf + C::at(tok, 16 * j + 8), make_uint4(f[4], f[5], f[6], f[7]));
      }
    };
    const uint32_t bar0 = smem_addr(&bars[wg][0]);
    uint32_t flying = 0, phase = 0;  // bit a: MMAs into accumulator a are on their way; the parity of their commit
    bool ok = true;
    float2* const cn = reinterpret_cast<float2*>(smem + M.cn);
    float* const slope = reinterpret_cast<float*>(smem + M.slope);
    int2* const range = reinterpret_cast<int2*>(smem + M.range);
    for (int g0 = 0; g0 < nq; g0 += S.tiles) {
      const int n = min(S.tiles, nq - g0), npad = (n + 15) & ~15, nch = (npad + QC - 1) / QC;
      __syncthreads();  // (the last queries' MMAs are done: both warpgroups have waited for them)
      if (g0 == 0 && seen(0)) load_codes(0);
      for (int x = tid; x < npad; x += 256) {
        const Column c = column_of<EX>(A, rq, h, x < n ? g0 + x : nq, 1.f);  // (nq: none)
        cn[x].y = x < n ? c.lse2 : INFINITY;
        if (EX) slope[x] = c.slope;
        range[x] = make_int2(c.hi, c.lo);
      }
      const float unit = EX && A.softcap > 0.f ? __fdiv_rn(A.scale, A.softcap) : A.scale * LOG2E;
      // Q: a warp takes 8 queries, lane (query, c) the pieces of 8 elements c, c + 4, ..: stores without bank
      // conflicts; four rounds' loads on their way
      constexpr int PC = HD / 32, PW = HL ? 2 : 1;  // pieces a lane, 16-byte words a piece
      const int qr = lane & 7, qp = lane >> 3;
      constexpr int U = 4;
      for (int x0 = warp * 8; x0 < npad; x0 += 64 * U) {
        uint4 in[U][PC][PW];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int qi = g0 + min(x0 + 64 * u + qr, n - 1), row = group_row(A, qi);  // (past the last: not used)
          const uint8_t* const from = reinterpret_cast<const uint8_t*>(A.q) +
              ((int64_t)(rq.row0 + row) * A.q_stride + (int64_t)(h * A.GH + qi - row * A.GH) * HD) * (HL ? 4 : 2);
#pragma unroll
          for (int p = 0; p < PC; ++p)
#pragma unroll
            for (int w = 0; w < PW; ++w) in[u][p][w] = *reinterpret_cast<const uint4*>(from + ((qp + 4 * p) * PW + w) * 16);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int x = x0 + 64 * u + qr;
          float v[PC][8], mx = 0.f;
#pragma unroll
          for (int p = 0; p < PC; ++p) {
            const uint32_t w[8] = {in[u][p][0].x, in[u][p][0].y, in[u][p][0].z, in[u][p][0].w,
                                   in[u][p][PW - 1].x, in[u][p][PW - 1].y, in[u][p][PW - 1].z, in[u][p][PW - 1].w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              if (HL) v[p][e] = __uint_as_float(w[e]);
              else if (DT == DDL_T_BF16) v[p][e] = e & 1 ? bf16hi_f32(w[e / 2]) : bf16lo_f32(w[e / 2]);
              else {
                const __half2 h2 = *reinterpret_cast<const __half2*>(&w[e / 2]);
                v[p][e] = e & 1 ? __high2float(h2) : __low2float(h2);
              }
              if (x >= n) v[p][e] = 0.f;
              if (DT != DDL_T_F16) mx = fmaxf(mx, fabsf(v[p][e]));
            }
          }
          mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 16));
          int e2 = (int)((__float_as_uint(mx) >> 23) & 255u) - 127 - 12;  // the largest lands in [2^12, 2^13)
          e2 = e2 < -100 ? -100 : e2 > 115 ? 115 : e2;
          if (DT == DDL_T_F16) e2 = 0;  // (as they are)
          const float down = __uint_as_float((uint32_t)(127 - e2) << 23);
          if (x < npad) {
#pragma unroll
            for (int p = 0; p < PC; ++p) {
              uint32_t hi[4], lo[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float a = v[p][2 * e] * down, b = v[p][2 * e + 1] * down;
                hi[e] = pack_f16x2(a, b);
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi[e]));
                lo[e] = pack_f16x2(a - f.x, b - f.y);
              }
              const uint32_t to = smem_addr(smem) + C::at(x, 8 * (qp + 4 * p));
              sts128(to, make_uint4(hi[0], hi[1], hi[2], hi[3]));
              if (HL) sts128(to + M.qlo, make_uint4(lo[0], lo[1], lo[2], lo[3]));
            }
            if (qp == 0) cn[x].x = x < n ? __uint_as_float((uint32_t)(127 + e2) << 23) * unit : 0.f;
          }
        }
      }
      fence_proxy_async_smem();
      __syncthreads();
      // the MMAs of chunk c into accumulator c & 1
      const uint64_t adesc = umma_sdesc(kbuf, C::LBO, C::SBO), bdesc = umma_sdesc(smem_addr(smem), C::LBO, C::SBO);
      auto issue = [&](int c) {
        const uint32_t d = tm + wg * 2 * QC + (c & 1) * QC;
        const uint32_t idesc = umma_idesc_f16(TOK, min(QC, npad - c * QC));
        if ((warp & 3) == 0) {
          tc_fence_after();
          if (elect_one()) {
            const uint64_t b = bdesc + (uint64_t)(c * (QC / 8) * C::SBO >> 4);
#pragma unroll
            for (int k = 0; k < HD / 16; ++k) umma_f16_ss(d, adesc + 16 * k, b + 16 * k, idesc, k ? 1u : 0u);
            if (HL) {
              const uint64_t b2 = b + (M.qlo >> 4);
#pragma unroll
              for (int k = 0; k < HD / 16; ++k) umma_f16_ss(d, adesc + 16 * k, b2 + 16 * k, idesc, 1u);
            }
            umma_commit(bar0 + 8 * (c & 1));
          }
          __syncwarp();
        }
        flying |= 1u << (c & 1);
      };
      for (int i = 0; ok && i < mine; ++i) {
        if (!seen(i)) {
          if (seen(i + 1)) load_codes(i + 1);
          continue;
        }
        store_codes();
        const float f = ks;
        const bool has = live;
        fence_proxy_async_smem();
        tc_fence_before();
        wg_sync(1 + wg);  // codes there; the accumulators have been read
        issue(0);
        if (seen(i + 1)) load_codes(i + 1);
        else if (g0 + S.tiles < nq && seen(0)) load_codes(0);  // (the next queries begin there, or behind unseen tiles)
        const int key0 = (c0 + wg + 2 * i) * TOK, key = key0 + tok;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        for (int c = 0; c < nch; ++c) {
          if (c + 1 < nch) issue(c + 1);
          bool late = false;
          {  // (bounded)
            uint64_t t0 = 0;
            for (uint32_t it = 1; !__all_sync(FULL, mbar_try_wait(bar0 + 8 * (c & 1), phase >> (c & 1) & 1)); ++it)
              if ((it & 1023u) == 0) {
                const uint64_t now = __shfl_sync(FULL, globaltimer(), 0);
                if (t0 == 0) t0 = now;
                else if (now - t0 > S.wait_ns) {
                  late = true;
                  break;
                }
              }
          }
          ok = !wg_or(1 + wg, late);
          if (!ok) break;
          flying &= ~(1u << (c & 1));
          phase ^= 1u << (c & 1);
          tc_fence_after();
          const uint32_t d = tm + ((uint32_t)(warp & 3) << 21) + wg * 2 * QC + (c & 1) * QC;
          const int q0 = g0 + c * QC, nc = min(QC, npad - c * QC), q1 = min(q0 + nc, nq) - 1;
          // tokens that every query of the chunk sees need no masks
          const bool edge = key0 + TOK - 1 > rq.p0 + group_row(A, q0) || key0 < first_seen(A, rq, q1);
          const float2* const cc = cn + c * QC;
          auto add = [&](const uint32_t (&v)[16], int x) {  // queries x .. x + 15 of the chunk
            float w[16];
            float2 q[16];  // (two a load)
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              const float4 two = *reinterpret_cast<const float4*>(cc + x + j);
              q[j] = make_float2(two.x, two.y);
              q[j + 1] = make_float2(two.z, two.w);
            }
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
          };
          // 16 columns' loads on their way while the last 16 are gone over
          uint32_t u[16], v[16];
          tmem_ld_32x32b_x16(d, u);
          for (int x = 0; x < nc; x += 32) {
            landed(u);
            if (x + 16 < nc) tmem_ld_32x32b_x16(d + x + 16, v);
            add(u, x);
            if (x + 16 >= nc) break;
            landed(v);
            if (x + 32 < nc) tmem_ld_32x32b_x16(d + x + 32, u);
            add(v, x + 16);
          }
          tc_fence_before();
          wg_sync(1 + wg);  // the accumulator has been read
        }
        const float all = (sum[0] + sum[1]) + (sum[2] + sum[3]);
        if (has) part[i * TOK] += all;
      }
    }
    if (!ok) {  // a wait gave up: what this warpgroup has not finished is NaN
      if (A.bad && tok == 0) atomicOr(A.bad, 2);
      for (int i = 0; i < mine; ++i)
        if (seen(i)) part[i * TOK] = __uint_as_float(0x7fffffffu);
    }
    for (int i = 0; i < mine; ++i) {
      const int key = key_of(i);
      if (key < rq.len && c0 + wg + 2 * i >= first) out[key] = part[i * TOK];
    }
    // MMAs in flight end before their memory goes to another
    for (int a = 0; a < 2; ++a)
      if (flying >> a & 1) mbar_wait_thread(bar0 + 8 * a, phase >> a & 1, DRAIN_NS);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tm, TMEM);
  }
}

template <int CT, int DT>
const void* tc_fn(int hd, bool ex) {
  if (hd == 128) return ex ? (const void*)kv8_score_tc_kernel<CT, DT, 128, true> : (const void*)kv8_score_tc_kernel<CT, DT, 128, false>;
  return ex ? (const void*)kv8_score_tc_kernel<CT, DT, 64, true> : (const void*)kv8_score_tc_kernel<CT, DT, 64, false>;
}
template <int CT>
const void* tc_fn(int dt, int hd, bool ex) {
  return dt == DDL_T_F32 ? tc_fn<CT, DDL_T_F32>(hd, ex) : dt == DDL_T_BF16 ? tc_fn<CT, DDL_T_BF16>(hd, ex) : tc_fn<CT, DDL_T_F16>(hd, ex);
}

}  // namespace

size_t kv8_score_tc_smem(bool f32, int hd, int queries, int tiles) { return Layout(f32, hd, queries, tiles).total; }

int kv8_score_tc_launch(const ScoreArgs& s, int type, int dtype, bool ex, unsigned chunks, void* stream) {
  ScoreArgs a = s;
  const void* fn = type == DDL_KV8_E4M3 ? tc_fn<DDL_KV8_E4M3>(dtype, a.a.hd, ex) : tc_fn<DDL_KV8_INT8>(dtype, a.a.hd, ex);
  const size_t smem = kv8_score_tc_smem(dtype == DDL_T_F32, a.a.hd, a.tiles, a.wb);
  const int st = cuda_status(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
  if (st) return st;
  void* args[] = {&a};
  return cuda_status(launch_pdl(fn, dim3(chunks, (unsigned)a.a.Hkv, (unsigned)a.a.R), dim3(256), args, smem, (cudaStream_t)stream));
}

}  // namespace ddl
