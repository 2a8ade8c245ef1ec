// ddl_kv8.cu -- placing and storing the rows of a serving step in the 8-bit
// paged KV cache: ddl_page_plan (page tables and slot maps from lengths) and
// ddl_kv8_append (quantizing store).
#include <cuda_bf16.h>

#include "ddl_kv8.h"

namespace ddl {
namespace {

// ------------------------------------------------------------------ plan
// need_r = ceil((old + add) / P) - ceil(old / P); a request is admitted by the
// running sums of need and add over the requests whose lengths fit, and the
// admitted ones get the exclusive running sums as their first free page and
// first row.  Every CTA forms both sums itself (R <= 4096 lengths from L2),
// so that one launch without any hand-over between CTAs does it all; then the
// CTAs share out the step's rows and new pages, each of which finds its
// request by binary search in the sums in shared memory.
//
// Bound by its round trips (launch, lengths, sums, table, store): 64 requests
// 3.1 us on one GB300, 1000 with 65536 rows 5.5 (writing those takes 0.1 of HBM).
// CTAs of 128 threads up to 512 requests, else 512: 64 requests 3.1 against 4.4
// us, 300 3.8 against 4.7, 1000 (of a row each) 5.7 against 5.5.
struct PlanArgs {
  const int32_t *old_len, *add_len, *free_pages;
  int32_t *table, *row_off, *kv_len, *row_pos, *slot, *used, *status;
  int32_t R, pshift, n_free, per, T;
};

constexpr int PLAN_ITEMS = 8;  // requests a thread takes: 512 threads x 8 = DDL_KV8_MAX_REQS

// Inclusive sums over the block of (a, b); `total` gets the block's sums.
template <int NT>
__device__ __forceinline__ void block_sums(int64_t& a, int64_t& b, int64_t (*ws)[2], int64_t& ta, int64_t& tb) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(FULL, a, o), y = __shfl_up_sync(FULL, b, o);
    if (lane >= o) {
      a += x;
      b += y;
    }
  }
  if (lane == 31) {
    ws[warp][0] = a;
    ws[warp][1] = b;
  }
  __syncthreads();
  int64_t pa = 0, pb = 0;
  ta = tb = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    if (w == warp) {
      pa = ta;
      pb = tb;
    }
    ta += ws[w][0];
    tb += ws[w][1];
  }
  a += pa;
  b += pb;
  __syncthreads();
}

// Largest r < R with off[r] <= i (off is not decreasing, off[0] = 0): the
// last of equal entries, i.e. the request that owns item i.
__device__ __forceinline__ int owner_at(const int32_t* off, int R, int32_t i) {
  int lo = 0, hi = R;  // off[lo] <= i < off[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

template <int NT>
__global__ void __launch_bounds__(NT) page_plan_kernel(const __grid_constant__ PlanArgs A) {
  extern __shared__ int32_t plan_smem[];
  __shared__ int64_t ws[NT / 32][2];
  int32_t* roff = plan_smem;             // [R + 1] first row
  int32_t* poff = plan_smem + A.R + 1;   // [R + 1] first new page
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x;
  const int64_t P = 1ll << A.pshift, cap = (int64_t)A.per << A.pshift;
  const int items = (A.R + NT - 1) / NT;  // <= PLAN_ITEMS
  const int r0 = tid * items;
  int32_t old[PLAN_ITEMS], add[PLAN_ITEMS];
  uint32_t fits = 0, okay = 0;
  int64_t need[PLAN_ITEMS], sp = 0, sr = 0, tp, tr;
#pragma unroll
  for (int k = 0; k < PLAN_ITEMS; ++k) {
    need[k] = 0;
    old[k] = add[k] = 0;
    if (k < items && r0 + k < A.R) {
      old[k] = A.old_len[r0 + k];
      add[k] = A.add_len[r0 + k];
      const int64_t t = (int64_t)old[k] + add[k];
      if (old[k] >= 0 && add[k] >= 0 && t <= cap) {
        fits |= 1u << k;
        need[k] = ((t + P - 1) >> A.pshift) - (((int64_t)old[k] + P - 1) >> A.pshift);
        sp += need[k];
        sr += add[k];
      }
    }
  }
  int64_t ip = sp, ir = sr;
  block_sums<NT>(ip, ir, ws, tp, tr);
  ip -= sp;
  ir -= sr;
  sp = sr = 0;
  uint32_t no_page = 0;
#pragma unroll
  for (int k = 0; k < PLAN_ITEMS; ++k) {
    if (!((fits >> k) & 1u)) continue;
    ip += need[k];
    ir += add[k];
    if (need[k] > 0 && ip > A.n_free) {
      no_page |= 1u << k;
    } else if (!(add[k] > 0 && ir > A.T)) {
      okay |= 1u << k;
      sp += need[k];
      sr += add[k];
    }
  }
  ip = sp;
  ir = sr;
  block_sums<NT>(ip, ir, ws, tp, tr);
  ip -= sp;
  ir -= sr;
#pragma unroll
  for (int k = 0; k < PLAN_ITEMS; ++k) {
    if (k >= items || r0 + k >= A.R) continue;
    const int r = r0 + k;
    const bool ok = (okay >> k) & 1u, fit = (fits >> k) & 1u;
    roff[r] = (int32_t)ir;
    poff[r] = (int32_t)ip;
    if (blockIdx.x == 0) {
      A.row_off[r] = (int32_t)ir;
      A.status[r] = ok ? 0 : !fit ? 1 : ((no_page >> k) & 1u) ? 2 : 3;
      int64_t n = ok ? (int64_t)old[k] + add[k] : old[k];
      n = n < 0 ? 0 : n > cap ? cap : n;
      A.kv_len[r] = (int32_t)n;
    }
    if (ok) {
      ir += add[k];
      ip += need[k];
    }
  }
  if (tid == 0) {
    roff[A.R] = (int32_t)tr;
    poff[A.R] = (int32_t)tp;
    if (blockIdx.x == 0) {
      A.row_off[A.R] = (int32_t)tr;
      A.used[0] = (int32_t)tp;
    }
  }
  __syncthreads();
  const int64_t step = (int64_t)gridDim.x * NT, first = (int64_t)blockIdx.x * NT + tid;
  // the step's rows; the page of a row among its request's new ones comes
  // from the free list, not from the table another CTA is writing
  for (int64_t i64 = first; i64 < A.T; i64 += step) {
    const int32_t i = (int32_t)i64;
    int32_t pos = -1, sl = -1;
    if (i < tr) {
      const int r = owner_at(roff, A.R, i);
      const int32_t o = A.old_len[r];
      pos = o + (i - roff[r]);
      const int32_t j = pos >> A.pshift, held = (int32_t)(((int64_t)o + P - 1) >> A.pshift);
      const int32_t page = j < held ? A.table[(int64_t)r * A.per + j] : A.free_pages[poff[r] + j - held];
      sl = (int32_t)(((uint32_t)page << A.pshift) | ((uint32_t)pos & (uint32_t)(P - 1)));
    }
    A.row_pos[i] = pos;
    A.slot[i] = sl;
  }
  for (int64_t i64 = first; i64 < tp; i64 += step) {
    const int32_t i = (int32_t)i64;
    const int r = owner_at(poff, A.R, i);
    const int32_t held = (int32_t)(((int64_t)A.old_len[r] + P - 1) >> A.pshift);
    A.table[(int64_t)r * A.per + held + (i - poff[r])] = A.free_pages[i];
  }
}

// ------------------------------------------------------------------ append
struct AppendArgs {
  uint8_t* code[2];    // k, v
  float* scale[2];
  const void* x[2];
  int64_t stride[2];
  const int32_t* slot;
  int32_t* bad;
  int64_t slots;       // pages * page_size
  int32_t T, H, pshift, span, ppc, vec, small;  // vec: the map is 16-byte aligned; small: T <= 256 (and span 1)
};

// (No load here is of the non-coherent kind: under dependent launches the kernel
// is already resident while its predecessor writes.)
// Four (hd 128) or two (hd 64) neighbouring elements of a row, as they are
// stored (a 16-bit row takes half the registers until it is used), and as fp32.
template <int DT, int W>
struct Raw {
  static constexpr int N = DT == DDL_T_F32 ? W : W / 2;
  uint32_t w[N];
  __device__ __forceinline__ void load(const void* base, int64_t at) {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(reinterpret_cast<const uint8_t*>(base) +
                                                          at * (DT == DDL_T_F32 ? 4 : 2));
    if (N == 4) {
      const uint4 u = *reinterpret_cast<const uint4*>(p);
      w[0] = u.x; w[N > 1 ? 1 : 0] = u.y; w[N > 2 ? 2 : 0] = u.z; w[N - 1] = u.w;
    } else if (N == 2) {
      const uint2 u = *reinterpret_cast<const uint2*>(p);
      w[0] = u.x; w[N - 1] = u.y;
    } else {
      w[0] = *p;
    }
  }
  __device__ __forceinline__ void floats(float (&v)[W]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (DT == DDL_T_F32) {
        v[i] = __uint_as_float(w[i]);
      } else if (DT == DDL_T_BF16) {
        v[(2 * i) % W] = bf16lo_f32(w[i]);
        v[(2 * i + 1) % W] = bf16hi_f32(w[i]);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        v[(2 * i) % W] = f.x;
        v[(2 * i + 1) % W] = f.y;
      }
    }
  }
};

template <int CT, int W>
__device__ __forceinline__ uint32_t encode(const float (&v)[W]) {
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < W; i += 2)
    r |= (CT == DDL_KV8_E4M3 ? f32x2_e4m3x2(v[i], v[i + 1]) : f32_int8(v[i]) | (f32_int8(v[i + 1]) << 8)) << (8 * i);
  return r;
}
template <int W>
__device__ __forceinline__ void store_codes(uint8_t* p, uint32_t c) {
  if (W == 4) *reinterpret_cast<uint32_t*>(p) = c;
  else *reinterpret_cast<uint16_t*>(p) = (uint16_t)c;
}

// The smallest power of two s >= 2^-126 with amax / s <= the largest code
// (448 = 1.75 * 2^8 or 127 = 1.984375 * 2^6): from amax = m * 2^e its exponent
// is e - 8 (e - 6), one more where m is above 1.75 (1.984375).  A power of two
// makes x / s exact, so a code is x rounded once, and moves e4m3 codes to a
// larger scale without rounding them again (unless they become subnormal).
template <int CT>
__device__ __forceinline__ float pow2_scale(float amax) {
  if (!(amax > 0.f)) return 0.f;
  const uint32_t b = __float_as_uint(amax), frac = b & 0x7fffffu;
  int e = (int)(b >> 23) - (CT == DDL_KV8_E4M3 ? 8 : 6) + (frac > (CT == DDL_KV8_E4M3 ? 0x600000u : 0x7e0000u) ? 1 : 0);
  e = e < 1 ? 1 : e;
  return __uint_as_float((uint32_t)e << 23);
}

// x / s: a product with 1 / s where s is a power of two whose inverse is
// normal (both exact), else a division.
struct Divider {
  float s, inv;
  bool pow2;
  __device__ __forceinline__ explicit Divider(float scale) : s(scale) {
    const uint32_t b = __float_as_uint(scale), e = b >> 23;
    pow2 = (b & 0x7fffffu) == 0u && e >= 1u && e <= 253u;
    inv = __uint_as_float((254u - (e < 254u ? e : 253u)) << 23);
  }
  __device__ __forceinline__ float operator()(float x) const { return pow2 ? x * inv : s > 0.f ? __fdiv_rn(x, s) : x; }
};

// One warp stores the rows of one 16-token block of one head of K or of V:
// each lane W neighbouring elements of every row.  A block's rows are normally
// one run of neighbours in the slot map; the warp that owns the run's first
// row takes it.  The rows stay in registers between the maximum and the codes,
// so each is read once; the earlier tokens' codes are touched only when the
// scale grows.  A CTA takes a window of `span` rows for up to 8 (head, K or V)
// pairs.  Decode steps are bound by their dependent round trips (slot; rows and
// old scale; store) and want every block in a warp of its own; in prompts 15 of
// 16 rows begin no run, and warps without one cost their launch.  So 1 row up to
// 256 rows, then 2, 4 and, where one row a request is impossible, 16.  One GB300,
// 8 K/V heads, bf16, spans 1 / 2 / 4 / 8 / 16: 257 requests of a row 7.9 / 7.4 /
// 11.2 / 18.7 / 35 us, 1024 20.2 / 19.2 / 22.2 / 24.9 / 39.9; prompts of 600 rows
// in all 7.9 / 7.4 / 7.0 / 6.5 / 9.6, of 2000 11.3 / 9.5 / 8.8 / 9.6 / 10.0, of
// 8165 44.8 / 34.2 / 28.9 / 25.8 / 24.6.
//
// Rows of one block that are apart in the slot map (a page given to two
// requests) must not race: every CTA looks through the whole map for the
// blocks that begin in its window.  A run whose block occurs earlier is left
// to that occurrence's warp, which stores all runs of the block in map order.
// The look is T / 1024 loads of 16 bytes a thread from L2, while the first run's
// rows are on their way; it is the reason for the limit on T.
struct RunSeen {
  int first, count;  // lowest row and number of rows of the block in the whole map
};

template <int CT, int DT, int HD>
struct Run {
  static constexpr int W = HD / 32;
  static constexpr int ROWS = 16;  // rows in registers
  int i, block, n, low;            // first row, block, rows, lowest token of the block among them
  int32_t mine;                    // slot of row i + lane
  float was;                       // the block's scale (0 when low is its first token)
  float* sp;
  uint8_t* rows;                   // the block's codes, this lane's columns
  const void* x;
  int64_t stride, col;
  Raw<DT, W> v[ROWS];

  // The run of neighbouring rows in `block` that begins at row i: its rows and
  // the block's scale on their way into registers.
  __device__ __forceinline__ void load(const AppendArgs& A, int kv, int h, int first, int blk) {
    const int lane = threadIdx.x & 31;
    i = first;
    block = blk;
    x = A.x[kv];
    stride = A.stride[kv];
    col = (int64_t)h * HD + lane * W;
    v[0].load(x, (int64_t)i * stride + col);
    mine = i + lane < A.T ? A.slot[i + lane] : -1;
    const uint32_t in = __ballot_sync(FULL, mine >= 0 && (mine >> 4) == block);
    n = in == FULL ? 32 : __ffs(~in) - 1;
#pragma unroll
    for (int b = 1; b < ROWS; ++b)
      if (b < n) v[b].load(x, (int64_t)(i + b) * stride + col);
    const int64_t page = block >> (A.pshift - 4);
    const int sub = block & ((1 << (A.pshift - 4)) - 1);
    const int64_t row = ((page * A.H + h) << A.pshift) + ((int64_t)sub << 4);  // of the pool's [rows][hd] view
    sp = A.scale[kv] + (row >> 4);
    rows = A.code[kv] + row * HD + lane * W;
    was = *sp;
    low = __reduce_min_sync(FULL, lane < n ? (mine & 15) : 15);
    if (n == 32) {  // (only with repeated slots)
      for (int e = i + 32; e < A.T; ++e) {
        const int32_t s = A.slot[e];
        if (s < 0 || (s >> 4) != block) break;
        ++n;
        low = min(low, (int)(s & 15));
      }
    }
    if (low == 0) was = 0.f;
  }

  __device__ __forceinline__ void put(const Divider& by, int32_t s, const Raw<DT, W>& r) {
    float c[W];
    r.floats(c);
#pragma unroll
    for (int w = 0; w < W; ++w) c[w] = by(c[w]);
    store_codes<W>(rows + (s & 15) * HD, encode<CT, W>(c));
  }

  __device__ __forceinline__ void store(const AppendArgs& A) {
    const int lane = threadIdx.x & 31;
    uint32_t top = 0;  // largest finite magnitude, as bits (ordered as the values)
    auto add = [&](const Raw<DT, W>& r) {
      float f[W];
      r.floats(f);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const uint32_t a = __float_as_uint(f[w]) & 0x7fffffffu;
        top = a < 0x7f800000u ? max(top, a) : top;
      }
    };
#pragma unroll
    for (int b = 0; b < ROWS; ++b)
      if (b < n) add(v[b]);
    Raw<DT, W> t;
    for (int b = ROWS; b < n; ++b) {  // (only with repeated slots)
      t.load(x, (int64_t)(i + b) * stride + col);
      add(t);
    }
    const float fresh = pow2_scale<CT>(__uint_as_float(__reduce_max_sync(FULL, top)));
    const float now = was > fresh ? was : fresh;
    if (low > 0 && now != was) {  // the block's earlier tokens move to the larger scale
      const float ratio = was > 0.f ? __fdiv_rn(was, now) : 0.f;
      for (int o = 0; o < low; ++o) {
        float c[W];
        const uint32_t w = W == 4 ? *reinterpret_cast<const uint32_t*>(rows + o * HD)
                                  : *reinterpret_cast<const uint16_t*>(rows + o * HD);
#pragma unroll
        for (int q = 0; q < W; q += 2) {
          const uint16_t two = (uint16_t)(w >> (8 * q));
          if (CT == DDL_KV8_E4M3) {
            const uint32_t hh = e4m3x2_f16x2(two);
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hh));
            c[q] = f.x * ratio;
            c[q + 1] = f.y * ratio;
          } else {
            c[q] = (float)(int8_t)(two & 255) * ratio;
            c[q + 1] = (float)(int8_t)(two >> 8) * ratio;
          }
        }
        store_codes<W>(rows + o * HD, encode<CT, W>(c));
      }
    }
    const Divider by(now);
#pragma unroll
    for (int b = 0; b < ROWS; ++b)
      if (b < n) put(by, __shfl_sync(FULL, mine, b), v[b]);
    for (int b = ROWS; b < n; ++b) {
      t.load(x, (int64_t)(i + b) * stride + col);
      put(by, A.slot[i + b], t);
    }
    if (lane == 0 && (low == 0 || now != was)) *sp = now;
    __syncwarp();
  }
};

constexpr int APPEND_SPAN = 16;  // rows of a window at most

// Where in the whole map do the blocks of the runs that begin at the CTA's rows
// occur?  (block: lane l's, of the window's row l; mine: the warp speaks for it.)
__device__ __forceinline__ void look_up(const AppendArgs& A, int32_t block, bool mine, int win, int2* begun,
                                        RunSeen* seen, int& count) {
  const int tid = threadIdx.x;
  if (tid == 0) count = 0;
  __syncthreads();
  if (mine && block >= 0) {
    const int k = atomicAdd(&count, 1), at = win * A.span + (tid & 31);
    begun[k] = make_int2(block, at);
    seen[at] = {0x7fffffff, 0};
  }
  __syncthreads();
  // where else in the map do these blocks occur?
  auto look = [&](int e, int32_t s, int2 b) {
    if (s >= 0 && (s >> 4) == b.x) {
      atomicMin(&seen[b.y].first, e);
      atomicAdd(&seen[b.y].count, 1);
    }
  };
  const int nb = count;
  if (A.vec) {  // 16 bytes a load, four loads on their way together
    const int n4 = (A.T + 3) >> 2;
    for (int e = tid; e < n4; e += 4 * 256) {
      int4 s[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int f = e + 256 * u, left = A.T - 4 * f;  // (the last one may be cut)
        s[u] = make_int4(-1, -1, -1, -1);
        if (left >= 4) {
          s[u] = *(reinterpret_cast<const int4*>(A.slot) + f);
        } else if (left > 0) {
          s[u].x = A.slot[4 * f];
          if (left > 1) s[u].y = A.slot[4 * f + 1];
          if (left > 2) s[u].z = A.slot[4 * f + 2];
        }
      }
      for (int k = 0; k < nb; ++k) {
        const int2 b = begun[k];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int at = 4 * (e + 256 * u);
          look(at, s[u].x, b);
          look(at + 1, s[u].y, b);
          look(at + 2, s[u].z, b);
          look(at + 3, s[u].w, b);
        }
      }
    }
  } else {
    for (int e = tid; e < A.T; e += 256) {
      const int32_t s = A.slot[e];
      for (int k = 0; k < nb; ++k) look(e, s, begun[k]);
    }
  }
  __syncthreads();
}

template <int CT, int DT, int HD>
__global__ void __launch_bounds__(256, DT == DDL_T_F32 && HD == 128 ? 2 : 3) kv8_append_kernel(const __grid_constant__ AppendArgs A) {
  __shared__ RunSeen seen[8 * APPEND_SPAN];
  __shared__ int2 begun[8 * APPEND_SPAN];  // runs that begin at the CTA's rows: block, row
  __shared__ int count;
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // warps: A.ppc pairs of each of 8 / ppc windows
  const int win = warp / A.ppc, nwin = 8 / A.ppc, pair = blockIdx.y * A.ppc + warp % A.ppc;
  const int c0 = blockIdx.x * nwin * A.span;
  const bool mine = win < nwin && pair < 2 * A.H && c0 + win * A.span < A.T;
  // the warp's own window: which runs begin there, and the first one's rows
  int32_t block = -1;  // lane l: of the run that begins at the window's row l
  if (mine && lane < A.span && c0 + win * A.span + lane < A.T) {
    const int e = c0 + win * A.span + lane;
    const int32_t s = A.slot[e], sb = e > 0 ? A.slot[e - 1] : -1;
    const bool outside = s >= A.slots;
    if (outside && A.bad && pair == 0) atomicOr(A.bad, 1);
    if (s >= 0 && !outside && (sb < 0 || (sb >> 4) != (s >> 4))) block = s >> 4;
  }
  uint32_t starts = __ballot_sync(FULL, block >= 0);
  const int h = pair >> 1, kv = pair & 1;
  Run<CT, DT, HD> run;
  if (starts) {
    const int k = __ffs(starts) - 1;
    run.load(A, kv, h, c0 + win * A.span + k, __shfl_sync(FULL, block, k));
  }
  int first1 = 0x7fffffff, total1 = 0;
  if (A.small) {  // each warp looks for itself, without a barrier
    const int blk = __shfl_sync(FULL, block, 0);
    int32_t s[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) s[u] = lane + 32 * u < A.T ? A.slot[lane + 32 * u] : -1;
#pragma unroll
    for (int u = 7; u >= 0; --u) {
      const uint32_t m = __ballot_sync(FULL, s[u] >= 0 && (s[u] >> 4) == blk);
      if (m) first1 = 32 * u + __ffs(m) - 1;
      total1 += __popc(m);
    }
  } else {
    if (!__syncthreads_or(starts != 0)) return;
    look_up(A, block, mine && warp % A.ppc == 0, win, begun, seen, count);
  }
  bool loaded = true;
  for (; starts; starts &= starts - 1, loaded = false) {
    const int k = __ffs(starts) - 1, at = win * A.span + k, blk = __shfl_sync(FULL, block, k);
    int i = c0 + at, left = A.small ? total1 : seen[at].count;
    if ((A.small ? first1 : seen[at].first) != i) continue;  // an earlier run's warp takes this one
    for (;;) {  // the block's runs, in map order
      if (!loaded) run.load(A, kv, h, i, blk);
      loaded = false;
      run.store(A);
      left -= run.n;
      if (left <= 0) break;
      for (i += run.n; i < A.T; i += 32) {
        const int32_t s = i + lane < A.T ? A.slot[i + lane] : -1;
        const uint32_t m = __ballot_sync(FULL, s >= 0 && (s >> 4) == blk);
        if (m) {
          i += __ffs(m) - 1;
          break;
        }
      }
      if (i >= A.T) break;
    }
  }
}

template <int CT, int DT>
const void* append_fn(int hd) {
  return hd == 128 ? (const void*)kv8_append_kernel<CT, DT, 128> : (const void*)kv8_append_kernel<CT, DT, 64>;
}

bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

}  // namespace
}  // namespace ddl

using namespace ddl;

extern "C" int ddl_page_plan(const int32_t* old_len, const int32_t* add_len, int32_t R, int32_t page_size,
                             const int32_t* free_pages, int32_t n_free, int32_t* page_table, int32_t pages_per_seq,
                             int32_t* row_off, int32_t* kv_len, int32_t* row_pos, int32_t* slot, int32_t T,
                             int32_t* used, int32_t* status, void* stream) {
  if (!old_len || !add_len || !page_table || !row_off || !kv_len || !used || !status) return DDL_ERR_ARG;
  if (R < 1 || n_free < 0 || T < 0 || pages_per_seq < 1) return DDL_ERR_ARG;
  if ((n_free > 0 && !free_pages) || (T > 0 && (!row_pos || !slot))) return DDL_ERR_ARG;
  if (kv_len == old_len || kv_len == add_len) return DDL_ERR_ARG;
  if (page_size < 16 || page_size > (1 << 20) || (page_size & (page_size - 1))) return DDL_ERR_ARG;
  if (R > DDL_KV8_MAX_REQS || (int64_t)pages_per_seq * page_size > 0x7fffffffLL) return DDL_ERR_UNSUPPORTED;
  for (const void* p : {(const void*)old_len, (const void*)add_len, (const void*)free_pages, (const void*)page_table,
                        (const void*)row_off, (const void*)kv_len, (const void*)row_pos, (const void*)slot,
                        (const void*)used, (const void*)status})
    if (!aligned4(p)) return DDL_ERR_ALIGN;
  PlanArgs a = {old_len, add_len, free_pages, page_table, row_off, kv_len, row_pos, slot, used, status,
                R, log2_of(page_size), n_free, pages_per_seq, T};
  const int nt = R <= 512 ? 128 : 512;
  int64_t ctas = ((int64_t)T + nt - 1) / nt;  // (a new page has a row, so there are at most T of them)
  const int most = 152 * (512 / nt);
  ctas = ctas < 1 ? 1 : ctas > most ? most : ctas;
  void* args[] = {&a};
  const size_t smem = (size_t)(2 * (R + 1)) * 4;
  const void* fn = nt == 128 ? (const void*)page_plan_kernel<128> : (const void*)page_plan_kernel<512>;
  return cuda_status(launch_pdl(fn, dim3((unsigned)ctas), dim3(nt), args, smem, (cudaStream_t)stream));
}

extern "C" int ddl_kv8_append(const ddl_kv8* kv, int32_t H_kv, int32_t head_dim, ddl_dtype dtype, const void* k_new,
                              int64_t k_stride, const void* v_new, int64_t v_stride, const int32_t* slot, int32_t T,
                              int32_t* bad_out, void* stream) {
  int st = check_kv8(kv, H_kv, head_dim);
  if (st) return st;
  if (!k_new || !v_new || !slot || T < 1) return DDL_ERR_ARG;
  if (!dtype_bytes(dtype)) return DDL_ERR_UNSUPPORTED;
  const int64_t w = (int64_t)H_kv * head_dim;
  if (k_stride < w || v_stride < w || k_stride % 8 || v_stride % 8) return DDL_ERR_ARG;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned4(slot) || !aligned4(bad_out)) return DDL_ERR_ALIGN;
  AppendArgs a;
  a.code[0] = kv->k;
  a.code[1] = kv->v;
  a.scale[0] = kv->k_scale;
  a.scale[1] = kv->v_scale;
  a.x[0] = k_new;
  a.x[1] = v_new;
  a.stride[0] = k_stride;
  a.stride[1] = v_stride;
  a.slot = slot;
  a.bad = bad_out;
  a.slots = kv->pages * kv->page_size;
  a.T = T;
  a.H = H_kv;
  a.pshift = log2_of(kv->page_size);
  a.span = T <= 256 ? 1 : T <= 512 ? 2 : T <= 4096 ? 4 : APPEND_SPAN;
  a.vec = aligned16(slot);
  a.small = T <= 256;
  a.ppc = 2 * H_kv < 8 ? 2 * H_kv : 8;
  if (T > DDL_KV8_MAX_APPEND) return DDL_ERR_UNSUPPORTED;
  const int rows = 8 / a.ppc * a.span;  // of a CTA
  const dim3 grid((unsigned)((T + rows - 1) / rows), (unsigned)((2 * H_kv + a.ppc - 1) / a.ppc));
  const void* fn = nullptr;
#define DDL_APPEND(CTV)                                                     \
  fn = dtype == DDL_T_F32 ? append_fn<CTV, DDL_T_F32>(head_dim)             \
       : dtype == DDL_T_BF16 ? append_fn<CTV, DDL_T_BF16>(head_dim)         \
                             : append_fn<CTV, DDL_T_F16>(head_dim)
  if (kv->type == DDL_KV8_E4M3) DDL_APPEND(DDL_KV8_E4M3);
  else DDL_APPEND(DDL_KV8_INT8);
#undef DDL_APPEND
  void* args[] = {&a};
  return cuda_status(launch_pdl(fn, grid, dim3(256), args, 0, (cudaStream_t)stream));
}
