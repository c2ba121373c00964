// Appending packed new tokens to the paged cache with the rotary position
// rotation applied on the way: keys are rotated as they are written into their
// pages, values copied, the queries rotated in the same launch, and the key
// summaries of the pages that grow recomputed from the stored (rotated,
// rounded) keys, so that the page router, the sparse step and the dense
// attention all see one cache.
//
// Rotation of one head row x at position p with c = table[p, k], s =
// table[p, r/2 + k] (k < r/2): (x_i, x_j) -> (x_i c - x_j s, x_j c + x_i s) with
// (i, j) = (k, k + r/2), or (2k, 2k + 1) when interleaved; features past r are
// copied.  Every product and sum is one float32 rounding (no contraction), the
// result one rounding to bf16: the stored bits are those of the plain formula.
//
// Two kinds of CTA share the launch.  A page CTA owns some kv heads of a touched
// page (as many as its stage holds when there are pages enough to fill the GPU,
// so that their loads share one chain of look-ups; one otherwise): it reads the
// page's old keys and rotates and writes the new ones in 16-byte pieces (both
// halves of a rotated pair in one thread), leaves them in shared memory as well,
// and then sums each column in float64 from there (one column per thread: few
// registers, so enough CTAs are resident to keep the loads in flight; 8254 tokens
// with the sums kept per thread while loading 109 us, with one column per thread
// 65, with several heads per CTA 45, with two heads in flight 41, all as graph
// replays; 208 MB, so 5.1 TB/s, and 4.8 in the 43 us of a call among others).  One
// thread per sequence reports its new length and bad offsets.  A query CTA rotates the heads of a few tokens, one warp per token: a
// lane keeps its unit of the head, so it reads its cosines and sines once for all
// heads.  Page slots and tokens find their sequence by a 32-way search of the
// offsets: slot s belongs to the last b with floor(cu[b]/P) + 2b <= s (n tokens
// touch at most floor(n/P) + 2 pages), so the grid needs only the packed total.
// Memory-bound: every byte is moved once.
//
// Sources: "Universal Attention Engine — Declarative Sparse Attention for
// Production", "Architecture" (a PagedAttention-compatible cache) and
// "Content-Dependent Dynamic Routing" (the router scores mean(k_blocks)); the
// rotation is RoFormer's (Su et al., 2021).
#include "common.cuh"
#include "exact.cuh"
#include "internal.h"

namespace sa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxD = 256;
constexpr int kQTokens = 8;      // tokens per query CTA (one per warp)
constexpr int kStage = 16384;    // 16-bit elements of keys staged at a time

// Last b in [0, B) with key(b) <= x (key ascending, key(0) <= x); whole warp.
template <typename F>
SA_DEV int last_le(int B, int64_t x, F&& key) {
  const int lane = threadIdx.x & 31;
  int lo = 0, len = B;
  while (len > 1) {
    const int step = (len + 31) / 32;
    const int off = lane * step;
    const bool le = off < len && key(lo + off) <= x;
    const uint32_t m = __ballot_sync(0xffffffffu, le);
    const int idx = m ? 31 - __clz(m) : 0;
    lo += idx * step;
    len = min(step, len - idx * step);
  }
  return lo;
}

SA_DEV float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
SA_DEV float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

struct Pieces {   // one unit: 8 columns, or 8 + their 8 partners
  uint4 a, b;
};

// The cosines and sines of a unit's pairs: 8 of each (halves), or 4 (adjacent).
struct Trig {
  float4 c[2], s[2];
};
SA_DEV void rotate_halves(Pieces& u, const Trig& t) {
  uint32_t* pa = reinterpret_cast<uint32_t*>(&u.a);
  uint32_t* pb = reinterpret_cast<uint32_t*>(&u.b);
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const float cc[4] = {t.c[q].x, t.c[q].y, t.c[q].z, t.c[q].w};
    const float ss[4] = {t.s[q].x, t.s[q].y, t.s[q].z, t.s[q].w};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t wa = pa[2 * q + i], wb = pb[2 * q + i];
      const float a0 = bf_lo(wa), a1 = bf_hi(wa), b0 = bf_lo(wb), b1 = bf_hi(wb);
      const float c0 = cc[2 * i], c1 = cc[2 * i + 1], s0 = ss[2 * i], s1 = ss[2 * i + 1];
      pa[2 * q + i] = pack_bf16(__fsub_rn(__fmul_rn(a0, c0), __fmul_rn(b0, s0)),
                                __fsub_rn(__fmul_rn(a1, c1), __fmul_rn(b1, s1)));
      pb[2 * q + i] = pack_bf16(__fadd_rn(__fmul_rn(b0, c0), __fmul_rn(a0, s0)),
                                __fadd_rn(__fmul_rn(b1, c1), __fmul_rn(a1, s1)));
    }
  }
}
SA_DEV void rotate_pairs(uint4& x, const Trig& t) {
  const float cc[4] = {t.c[0].x, t.c[0].y, t.c[0].z, t.c[0].w};
  const float ss[4] = {t.s[0].x, t.s[0].y, t.s[0].z, t.s[0].w};
  uint32_t* p = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = bf_lo(p[i]), b = bf_hi(p[i]);
    p[i] = pack_bf16(__fsub_rn(__fmul_rn(a, cc[i]), __fmul_rn(b, ss[i])),
                     __fadd_rn(__fmul_rn(b, cc[i]), __fmul_rn(a, ss[i])));
  }
}

// Column of unit u's first piece, and of its second (-1: none).  Halves: units
// [0, r/16) pair columns 8u and 8u + r/2, the rest copy one piece.
SA_DEV int2 unit_cols(int u, int r, bool inter) {
  if (inter) return make_int2(8 * u, -1);
  const int np = r / 16;
  return u < np ? make_int2(8 * u, 8 * u + r / 2) : make_int2(r + 8 * (u - np), -1);
}
SA_DEV Pieces load_unit(const uint16_t* row, int2 c) {
  Pieces p;
  p.a = *reinterpret_cast<const uint4*>(row + c.x);
  p.b = c.y >= 0 ? *reinterpret_cast<const uint4*>(row + c.y) : make_uint4(0, 0, 0, 0);
  return p;
}
SA_DEV void store_unit(uint16_t* row, int2 c, const Pieces& p) {
  *reinterpret_cast<uint4*>(row + c.x) = p.a;
  if (c.y >= 0) *reinterpret_cast<uint4*>(row + c.y) = p.b;
}
// The trigonometry of the unit at columns c of a table row (none: unused).
SA_DEV Trig load_trig(const float* __restrict__ cs, int2 c, int r, bool inter) {
  Trig t = {};
  if (c.y >= 0) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      t.c[q] = __ldg(reinterpret_cast<const float4*>(cs + c.x + 4 * q));
      t.s[q] = __ldg(reinterpret_cast<const float4*>(cs + r / 2 + c.x + 4 * q));
    }
  } else if (inter && c.x < r) {
    t.c[0] = __ldg(reinterpret_cast<const float4*>(cs + c.x / 2));
    t.s[0] = __ldg(reinterpret_cast<const float4*>(cs + r / 2 + c.x / 2));
  }
  return t;
}
SA_DEV void rotate_unit(Pieces& p, int2 c, const Trig& t, int r, bool inter) {
  if (c.y >= 0)
    rotate_halves(p, t);
  else if (inter && c.x < r)
    rotate_pairs(p.a, t);
}

__global__ void __launch_bounds__(kThreads, 4) rope_append_kernel(const RopeAppendArgs a) {
  pdl_wait_and_release();
  const int tid = threadIdx.x, lane = tid & 31;
  const int D = a.D, r = a.rot;
  const bool inter = a.interleaved != 0;
  const int upr = inter ? D / 8 : r / 16 + (D - r) / 8;   // units per row
  if (blockIdx.x >= a.page_ctas) {
    // ================= queries: one token per warp
    const int t = (blockIdx.x - a.page_ctas) * kQTokens + (tid >> 5);
    if (t >= a.total) return;
    const int b = last_le(a.B, t, [&](int i) { return (int64_t)a.cu[i]; });
    const int t0 = a.cu[b], t1 = a.cu[b + 1], L = a.seq_lens[b];
    const int64_t i = (int64_t)t - t0;
    // no sequence's token, or one of a sequence that is skipped (offsets, length)
    if (t0 < 0 || i < 0 || t >= t1 || t1 > a.total || L < 0 ||
        L > (int64_t)a.max_pages * a.P)
      return;
    const int64_t pos = L + i;
    if (pos >= a.n_pos) {
      if (lane == 0) set_dev_error(a.err, SA_DEVERR_PAGE_RANGE);
      return;
    }
    const int hpl = 32 / upr, u = lane % upr;   // heads per pass of the warp, this lane's unit
    int h = lane / upr;
    if (h >= hpl) return;
    const int2 c = unit_cols(u, r, inter);
    const Trig t_cs = load_trig(a.table + pos * r, c, r, inter);
    const uint16_t* src = a.q + t * a.q0;
    uint16_t* dst = a.q_out + (int64_t)t * a.Hq * D;
    constexpr int kU = 2;   // heads in flight
    for (; h + (kU - 1) * hpl < a.Hq; h += kU * hpl) {
      Pieces p[kU];
#pragma unroll
      for (int k = 0; k < kU; ++k) p[k] = load_unit(src + (h + k * hpl) * a.q1, c);
#pragma unroll
      for (int k = 0; k < kU; ++k) {
        rotate_unit(p[k], c, t_cs, r, inter);
        store_unit(dst + (h + k * hpl) * D, c, p[k]);
      }
    }
    for (; h < a.Hq; h += hpl) {
      Pieces p = load_unit(src + h * a.q1, c);
      rotate_unit(p, c, t_cs, r, inter);
      store_unit(dst + h * D, c, p);
    }
    return;
  }
  const int64_t cap = (int64_t)a.max_pages * a.P;
  // ================= every sequence's length, and what is wrong with it: one thread per
  // sequence, whether or not its page slots can be found, in the last page CTAs (their
  // slots are the likeliest to be nobody's)
  if (a.page_ctas - 1 - blockIdx.x <= (a.B - 1) / kThreads) {
    const int b = (a.page_ctas - 1 - blockIdx.x) * kThreads + tid;
    if (b < a.B) {
      const int t0 = a.cu[b], t1 = a.cu[b + 1], L = a.seq_lens[b];
      const bool bad_cu = t0 < 0 || t1 < t0 || t1 > a.total, bad_len = L < 0 || L > cap;
      const int n = bad_cu || bad_len ? 0 : t1 - t0;
      if (a.out_seq_lens) a.out_seq_lens[b] = L + n;
      if (bad_cu) set_dev_error(a.err, SA_DEVERR_COUNT);
      const int64_t end = (int64_t)L + n;
      if (bad_len || (n > 0 && (end > cap || end > a.n_pos)))
        set_dev_error(a.err, SA_DEVERR_PAGE_RANGE);
    }
  }
  // ================= one touched page of one kv head
  __shared__ __align__(16) uint16_t key_s[kStage];   // a block of rows of keys
  __shared__ double sum_s[kThreads];                 // [row group][column]
  __shared__ uint16_t exp_s[kThreads];               // largest << 8 | smallest exponent field
  const int hgroups = (a.Hkv + a.page_heads - 1) / a.page_heads;
  const int h0 = (blockIdx.x % hgroups) * a.page_heads, s = blockIdx.x / hgroups;
  const int hn = min(a.page_heads, a.Hkv - h0);
  const int P = a.P;
  const int b = last_le(a.B, s, [&](int i) { return (int64_t)(a.cu[i] / P) + 2 * i; });
  const int t0 = a.cu[b], t1 = a.cu[b + 1], L = a.seq_lens[b];
  const int j = s - (t0 / P + 2 * b);
  if (t0 < 0 || t1 < t0 || t1 > a.total || L < 0 || L > cap) return;   // (flagged above)
  const int n = t1 - t0;
  int64_t end = (int64_t)L + n;
  if (end > cap || end > a.n_pos) end = cap < a.n_pos ? cap : a.n_pos;   // the rest is dropped
  const int64_t p = L / P + j, p0 = p * P;
  if (j < 0 || end <= L || p0 >= end) return;
  const int ph = page_at(a.pt, b, (int)p);
  if (ph < 0 || ph >= a.P_pool) {
    if (tid == 0) set_dev_error(a.err, SA_DEVERR_POOL_RANGE);
    return;
  }
  const int n_old = (int)(L > p0 ? L - p0 : 0);
  const int nval = (int)((end < p0 + P ? end : p0 + P) - p0);
  const int64_t tok0 = t0 + p0 - L;               // token of row 0 (rows >= n_old are new)
  uint16_t* kpage = a.k_cache + ph * a.ks0 + h0 * a.ks1;
  uint16_t* vpage = a.v_cache + ph * a.vs0 + h0 * a.vs1;
  // A thread takes one piece of a row (x of `per`) for every ng-th head: threads
  // that the pieces leave over take other heads.
  auto spread = [&](int per, auto&& body) {
    const int ng = per >= kThreads ? 1 : min(hn, kThreads / per);
    const int xg = ng > 1 ? tid / per : 0;
    if (xg >= ng) return;
    for (int x = tid - xg * per; x < per; x += ng > 1 ? per : kThreads) body(x, xg, ng);
  };
  constexpr int kU = 2;   // heads in flight
  // ---- values: copied
  const int cpr = D / 8;
  if (nval > n_old)
    spread((nval - n_old) * cpr, [&](int x, int xg, int ng) {
      const int row = n_old + x / cpr, c = (x % cpr) * 8;
      const uint16_t* src = a.v + (tok0 + row) * a.v0 + h0 * a.v1 + c;
      uint16_t* dst = vpage + row * a.vs2 + c;
      for (int h = xg; h < hn; h += kU * ng) {
        uint4 v[kU];
#pragma unroll
        for (int k = 0; k < kU; ++k)
          if (h + k * ng < hn) v[k] = *reinterpret_cast<const uint4*>(src + (h + k * ng) * a.v1);
#pragma unroll
        for (int k = 0; k < kU; ++k)
          if (h + k * ng < hn) *reinterpret_cast<uint4*>(dst + (h + k * ng) * a.vs1) = v[k];
      }
    });
  // ---- keys, a block of rows at a time: the new ones rotated and stored, all of
  // them staged; then one thread per column (and row group) sums
  const int block = max(1, kStage / (hn * D));     // rows per block: the page's, when hn > 1
  const int groups = max(1, kThreads / (hn * D));  // row groups
  const int d = tid % D, sg = tid / D;             // D <= 256
  double sum = 0.0;
  int emax = 0, emin = 255;
  auto add = [&](uint32_t bits) {
    if ((bits & 0x7fffu) == 0) return;
    const int e = max(1, (int)((bits >> 7) & 0xffu));
    emax = max(emax, e);
    emin = min(emin, e);
    sum += static_cast<double>(bf16_bits_to_float(bits));
  };
  const int lg = 32 - __clz(nval);   // >= ceil(log2 nval) + 1
  // the mean of column dd of head h0 + h from its float64 sum: |x| < 2^(hi - 126)
  // and a multiple of 2^(lo - 134), so the sum is exact in any order while that
  // span and the carries fit 53 bits
  auto mean = [&](double t, int hi, int lo, int h, int dd) {
    if (hi > 0 && hi - lo + 8 + lg > 53) {
      ExactAcc e;
      e.clear();
      for (int row = 0; row < nval; ++row) {   // this CTA's own stores: visible after the barriers
        uint32_t m;
        int ex;
        bool neg;
        bf16_fields(*(volatile uint16_t*)(kpage + h * a.ks1 + row * a.ks2 + dd), m, ex, neg);
        e.add(m, ex, neg);
      }
      t = e.round_to_double();
    }
    a.sig[((int64_t)ph * a.Hkv + h0 + h) * D + dd] =
        f64_to_bf16_rne(t / static_cast<double>(nval));
  };
  for (int r0 = a.sig ? 0 : n_old; r0 < nval; r0 += block) {
    const int nr = min(nval - r0, block);
    spread(nr * upr, [&](int x, int xg, int ng) {
      const int row = r0 + x / upr;
      const int2 c = unit_cols(x % upr, r, inter);
      uint16_t* cached = kpage + row * a.ks2;
      if (row < n_old) {
        for (int h = xg; h < hn; h += ng)
          store_unit(key_s + (h * nr + row - r0) * D, c, load_unit(cached + h * a.ks1, c));
        return;
      }
      const Trig t = load_trig(a.table + (p0 + row) * r, c, r, inter);
      const uint16_t* src = a.k + (tok0 + row) * a.k0 + h0 * a.k1;
      for (int h = xg; h < hn; h += kU * ng) {
        Pieces y[kU];
#pragma unroll
        for (int k = 0; k < kU; ++k)
          if (h + k * ng < hn) y[k] = load_unit(src + (h + k * ng) * a.k1, c);
#pragma unroll
        for (int k = 0; k < kU; ++k) {
          const int hk = h + k * ng;
          if (hk >= hn) continue;
          rotate_unit(y[k], c, t, r, inter);
          store_unit(cached + hk * a.ks1, c, y[k]);
          if (a.k_out) store_unit(a.k_out + ((tok0 + row) * a.Hkv + h0 + hk) * D, c, y[k]);
          if (a.sig) store_unit(key_s + (hk * nr + row - r0) * D, c, y[k]);
        }
      }
    });
    if (!a.sig) continue;
    __syncthreads();
    if (hn > 1) {   // the whole page is staged
      for (int x = tid; x < hn * D; x += kThreads) {
        const int h = x / D, dd = x - h * D;
        sum = 0.0;
        emax = 0, emin = 255;
        for (int row = 0; row < nval; ++row) add(key_s[(h * nval + row) * D + dd]);
        mean(sum, emax, emin, h, dd);
      }
      return;
    }
    if (sg < groups)
      for (int row = sg; row < nr; row += groups) add(key_s[row * D + d]);
    __syncthreads();
  }
  if (!a.sig) return;
  if (sg < groups) {
    sum_s[tid] = sum;
    exp_s[tid] = static_cast<uint16_t>(emax << 8 | emin);
  }
  __syncthreads();
  if (tid >= D) return;
  double t = 0.0;
  int hi = 0, lo = 255;
  for (int q = 0; q < groups; ++q) {
    t += sum_s[q * D + tid];
    hi = max(hi, exp_s[q * D + tid] >> 8);
    lo = min(lo, exp_s[q * D + tid] & 0xff);
  }
  mean(t, hi, lo, 0, tid);
}

}  // namespace

cudaError_t launch_rope_append(RopeAppendArgs a, cudaStream_t stream) {
  if (a.B == 0) return cudaSuccess;
  static_assert(kMaxD / 8 <= 32 && kMaxD <= kThreads, "a row's units fit a warp, its columns a CTA");
  // page CTAs first: their chains (search, table, page, sums) are the longest
  const int64_t pages = (int64_t)a.total / a.P + 2 * (int64_t)a.B;
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const int stage_heads = kStage / (a.P * a.D) < 1 ? 1 : kStage / (a.P * a.D);
  a.page_heads = pages * a.Hkv > 6 * sms ? (stage_heads < a.Hkv ? stage_heads : a.Hkv) : 1;
  const int64_t page_ctas = pages * ((a.Hkv + a.page_heads - 1) / a.page_heads);
  const int64_t q_ctas = a.q ? (a.total + kQTokens - 1) / kQTokens : 0;
  if (page_ctas + q_ctas > 0x7fffffff) return cudaErrorInvalidValue;
  a.page_ctas = (int)page_ctas;
  return launch_pdl(rope_append_kernel, dim3((unsigned)(page_ctas + q_ctas)), dim3(kThreads), 0,
                    stream, a);
}

}  // namespace sa
