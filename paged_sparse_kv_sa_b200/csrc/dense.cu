// Dense causal attention of packed query tokens on the 5th-generation tensor
// cores: new tokens over a whole paged cache (single decode tokens, drafts,
// prompt chunks, mixed in one batch), or whole packed prompts.
//
// Query row (token t, head h) of sequence b sits at position L_b - n_b + t and
// sees the keys j at or before it (and, with a window, j > position - window):
//   S = scale q.k_j,  O = sum_j softmax(S)_j v_j,  lse = log sum_j exp(S_j).
// The rows of one (sequence, kv head) are (token, group head) pairs, token
// major, so a K/V tile is read once for all heads of its group.  An item is two
// tiles of these rows (each the whole tokens that fit 128 rows); its work is the
// 128-key tiles any of its rows sees.
//
// Work split.  Every CTA (one per SM) takes an equal share of all items' tiles,
// laid end to end (sequence, kv head, row tile), wherever the share's ends cut
// an item: long contexts of single tokens, ragged batches and causal triangles
// all spread evenly.  Every CTA finds its share from the offsets and lengths
// alone (no plan kernel, no counters).  A cut item's parts go to the workspace
// (at most one part that starts an item and one that continues an item per CTA)
// and a second small kernel merges them; whole items are written at once.
//
// One CTA, two 128-row tiles A and B:
//   warps 0-3 / 4-7   softmax of tile A / B, one row per thread: S from TMEM,
//                 mask (only tiles some row does not see whole), lazily re-based
//                 base-2 softmax (the running max moves only by more than 2^8,
//                 so the O rescale through TMEM is rare), P as bf16 over the
//                 S columns in two 64-key halves, epilogue;
//   warp 8        issues tcgen05.mma: S_w = Q_w K^T (M 128, N 128), O_w += P_w V
//                 with P from TMEM, in the order PV_A(i), QK_A(i+1), PV_B(i),
//                 QK_B(i+1): one tile's MMAs run under the other's softmax;
//   warps 9, 11   K, V tiles by TMA through the page map into a ring each (a
//                 missing page loads zeros from an out-of-range coordinate);
//   warp 10       the next item's queries by TMA as soon as their buffer frees (the
//                 box is the group's heads of as many tokens as fit 128 rows), or,
//                 of at most 16 rows, by its own loads, the rest of the tile zero;
//   warp 11       also plans the CTA's share first, and zeroes the value rows past
//                 a sequence's end and behind the window.
// An item of at most 128 rows gives both tiles the same rows and every other
// key tile each ("halves"); the two running softmaxes merge in the epilogue,
// both accumulators being in the same TMEM lanes.
//
// P is one bf16 rounding of each probability (relative 2^-8 at most, the same
// step as the bf16 output's own rounding); the row sums, and so the LSE, are of
// the unrounded float32 probabilities.
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "tc05.cuh"

namespace sa {
namespace {

constexpr int kSoftWarps = 8, kMmaWarp = 8, kLoadWarp = 9, kQWarp = 10, kPlanWarp = 11;
constexpr int kThreads = 384;
constexpr int kKeys = 128;        // keys per tile
constexpr int kM = 128;           // rows per tile
constexpr int kMaxSegs = 32;      // segments planned at a time
constexpr int kItemUnits = 2;     // an item's fixed cost, in tiles (8192-token prompt: 518, 490, 495 us for 1, 2, 3)
constexpr int kMinUnits = 2;      // smallest share worth a CTA (one token over 2048 keys: 13.9, 14.8, 16.2 us for 2, 4, 6)
constexpr float kLazy = 8.f;
constexpr int kBadRing = 8;
constexpr int kFewRows = 16;      // items of so few query rows have them copied by a warp
constexpr int kStageRow = 80;     // bytes: 64 + 16 against bank conflicts
static_assert(kDenseMaxBatch * 4 <= kSoftWarps * 32 * kStageRow, "the units fit the stage");

template <int D>
struct Cfg {
  static constexpr int kChunks = D / 64;
  static constexpr int kQBytes = kM * D * 2;
  static constexpr int kTileBytes = kKeys * D * 2;
  static constexpr int kStages = D == 64 ? 4 : 2;
  // A tile's missing boxes are noted before its stage is waited for, when the tensor
  // core is known to have read the keys of tile c - 1 - kStages; the softmax of that
  // tile, and of the one before (the other half's), may still have to look theirs up.
  static_assert(kBadRing >= kStages + 3, "tiles whose missing boxes are still looked up");
  static constexpr int kDyn = 2 * kQBytes + 2 * kStages * kTileBytes + 1024;
  static constexpr uint32_t kIdQK = tc::idesc_bf16_f32(kM, kKeys, false, false);
  static constexpr uint32_t kIdPV = tc::idesc_bf16_f32(kM, D, false, true);
};

// ---------------------------------------------------------------- geometry
struct Seq {
  int q0, n, k0, L;   // first query token, query tokens, first packed key, keys
};
// Offsets and lengths of sequence b, held inside the packed totals and the map
// (err: also report what was out of range).
SA_DEV Seq seq_of(const DenseArgs& a, int b, int32_t* err) {
  Seq s;
  const int q0 = a.cu_q[b], q1 = a.cu_q[b + 1];
  s.q0 = min(max(q0, 0), a.total_q);
  s.n = min(max(q1, s.q0), a.total_q) - s.q0;
  if (err && (q0 < 0 || q1 < q0 || q1 > a.total_q)) set_dev_error(err, SA_DEVERR_COUNT);
  if (a.cu_k) {
    const int k0 = a.cu_k[b], k1 = a.cu_k[b + 1];
    s.k0 = min(max(k0, 0), a.total_k);
    s.L = min(max(k1, s.k0), a.total_k) - s.k0;
    if (err && (k0 < 0 || k1 < k0 || k1 > a.total_k)) set_dev_error(err, SA_DEVERR_COUNT);
  } else {
    const int L = a.seq_lens[b];
    s.k0 = 0;
    s.L = min(max(L, 0), a.max_pages * a.P);
    if (err && L != s.L) set_dev_error(err, SA_DEVERR_PAGE_RANGE);
  }
  return s;
}
// Key tiles [x, y) that some row of item qt (toks tokens) sees (empty: x == y == 0).
SA_DEV int2 tiles_of(const Seq& s, int toks, int window, int qt) {
  const int t_first = qt * toks, t_last = min(s.n, t_first + toks) - 1;
  const int hi = min(s.L, s.L - s.n + t_last + 1);
  const int lo = window ? max(0, s.L - s.n + t_first - window + 1) : 0;
  if (hi <= lo) return make_int2(0, 0);
  return make_int2(lo / kKeys, (hi + kKeys - 1) / kKeys);
}
SA_DEV int item_units(const Seq& s, int toks, int window, int qt) {
  const int2 t = tiles_of(s, toks, window, qt);
  return kItemUnits + t.y - t.x;
}

// First key that some token of a sequence of n tokens and L keys sees: those before it
// may be anyone's.
SA_DEV int first_key(int L, int n, int window) {
  return window ? max(0, L - n - window + 1) : 0;
}

// A run of one item's tiles, as every role needs it.
struct Seg {
  int q0, n, k0, L;    // its sequence
  int b, kvh, r0, nr;  // rows [r0, r0 + nr) of the (sequence, kv head)
  int j0, j1;          // key tiles of this run
  int part;            // -1: the whole item, else the workspace part
  int pad;
};

// ---------------------------------------------------------------- waits
// Wait for phase `parity`, at most kPolls polls (each suspends the thread for up
// to microseconds: a second or so in all; no copy or product takes near as long).
// false: gave up.  The result is meant to be kept and looked at once a tile, not
// branched on here: a vote or a branch at every wait made the tensor core's
// issuing warp, and with it every tile, slower (8192-token prompt 535 -> 516 us,
// packed short prompts 244 -> 213 us without), and so did raising the CTA's flag
// from here (packed prompts 187 -> 198 us).
#ifdef SA_DENSE_POLLS   // a build whose waits run out early: a test of the way out
#define SA_DENSE_TRY "test_wait"
constexpr uint32_t kPolls = SA_DENSE_POLLS;
#else
#define SA_DENSE_TRY "try_wait"
constexpr uint32_t kPolls = 1u << 17;
#endif
SA_DEV bool wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .u32 n;\n mov.u32 n, 0;\n"
      "W:\n mbarrier." SA_DENSE_TRY ".parity.shared::cta.b64 p, [%1], %2;\n"
      " @p bra D;\n add.u32 n, n, 1;\n setp.lt.u32 q, n, %3;\n @q bra W;\n"
      "D:\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "n"(kPolls)
      : "memory");
  return ok != 0;
}
// Whether no lane of the warp has given up; a warp that has raises the CTA's flag:
// the loaders then ask for nothing more, and the others' waits run out.
SA_DEV bool all_well(bool ok, volatile int* abort_flag) {
  if (__all_sync(0xffffffffu, ok)) return true;
  *abort_flag = 1;
  return false;
}
// Phase `parity` of `bar`, at most 2^16 polls, whatever the CTA's flag says: the copies
// and products in flight of a CTA that has given up.
SA_DEV void drain(uint64_t* bar, uint32_t parity) {
  for (uint32_t n = 0; n < 1u << 16 && !mbar_try_wait(bar, parity); ++n) {}
}
// All threads of the CTA, from whichever role's code they are in.
SA_DEV void cta_sync() { asm volatile("bar.sync 15, %0;" ::"n"(kThreads) : "memory"); }
// Registers per thread after the roles part: the launch's 384 x 168 divided as
// 256 x 192 for the softmax warps (a row of scores is 128 registers) + 128 x 120.
SA_DEV void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 192;"); }
SA_DEV void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 120;"); }
// A value every lane holds alike, as the compiler can see.
template <typename T>
SA_DEV T uni(T x) { return __shfl_sync(0xffffffffu, x, 0); }
SA_DEV void pair_sync(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }

// Largest of three, or of two (NaN if one is).
SA_DEV float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
SA_DEV float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// Largest of x[i0 .. i0 + 63], four chains.
SA_DEV float max64(const float (&x)[128], int i0) {
  float m[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = max3_nan(x[i0 + i], x[i0 + 4 + i], x[i0 + 8 + i]);
#pragma unroll
  for (int c = 12; c < 60; c += 8)
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = max3_nan(m[i], x[i0 + c + i], x[i0 + c + 4 + i]);
  m[0] = max3_nan(m[0], x[i0 + 60], x[i0 + 61]);
  m[1] = max3_nan(m[1], x[i0 + 62], x[i0 + 63]);
  return max3_nan(m[0], m[1], max_nan(m[2], m[3]));
}

// Where lane's box of key tile j comes from: a tile is kKeys / box boxes (lane mod
// their number) by D / 64 column chunks (lane / their number).
struct Box {
  int page, row;
  uint32_t bad;   // boxes on pages that are not in the pool (all lanes)
};
SA_DEV Box box_of(const DenseArgs& a, const Seg& s, int j, int lane) {
  const int nb = kKeys / a.box;
  const int key = j * kKeys + (lane & (nb - 1)) * a.box;
  Box x = {0, s.k0 + key, 0};
  bool bad = false;
  if (!a.cu_k) {
    x.page = a.P_pool;   // out of range: zeros
    x.row = 0;
    if (key < s.L && key + a.box > first_key(s.L, s.n, a.window)) {
      const int ph = page_at(a.pt, s.b, key / a.P);
      bad = ph < 0 || ph >= a.P_pool;
      if (!bad) x.page = ph, x.row = key % a.P;
    }
  }
  x.bad = __ballot_sync(0xffffffffu, bad) & ((1u << nb) - 1u);
  return x;
}
// Load the c-th tile of a ring, once its stage is free; the whole warp.
template <int D>
SA_DEV bool load_tile(const Box& x, int kvh, uint32_t c, uint8_t* ring, const CUtensorMap* map,
                      uint64_t* full, uint64_t* empty, int box, volatile int* abort_flag) {
  using C = Cfg<D>;
  const int lane = threadIdx.x & 31, nb = kKeys / box, st = c % C::kStages;
  if (c >= (uint32_t)C::kStages &&
      !all_well(wait(&empty[st], ((c / C::kStages) - 1) & 1) && !*abort_flag, abort_flag))
    return false;
  if (lane == 0) mbar_arrive_expect_tx(&full[st], C::kTileBytes);
  __syncwarp();
  const int g = lane & (nb - 1), ch = lane / nb;
  if (ch < C::kChunks)
    tma_load_4d(ring + st * C::kTileBytes + ch * (kKeys * 128) + g * box * 128, map, &full[st],
                ch * 64, x.row, kvh, x.page);
  return true;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    dense_kernel(const __grid_constant__ DenseArgs a, const __grid_constant__ CUtensorMap qmap,
                 const __grid_constant__ CUtensorMap kmap,
                 const __grid_constant__ CUtensorMap vmap) {
  using C = Cfg<D>;
  // the merge kernel may be set up under this one's tail: it waits for the end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x, n_ctas = gridDim.x;
  const int G = a.Hq / a.Hkv;
  const int toks = 2 * a.tile_toks, tile_rows = a.tile_toks * G;   // tokens of an item, rows of a tile

  extern __shared__ uint8_t dyn_smem[];
  uint8_t* smem = dyn_smem + ((1024 - (smem_u32(dyn_smem) & 1023)) & 1023);
  uint8_t* q_s = smem;
  uint8_t* k_s = smem + 2 * C::kQBytes;
  uint8_t* v_s = k_s + C::kStages * C::kTileBytes;
  __shared__ uint64_t k_full[C::kStages], k_empty[C::kStages];
  __shared__ uint64_t v_full[C::kStages], v_empty[C::kStages], v_part[C::kStages];
  __shared__ uint64_t s_full[2], p_full[2][2], o_done[2], q_full, q_empty, all_done;
  __shared__ uint32_t tmem_base_s;
  __shared__ int abort_s, n_segs_s, last_s;
  __shared__ Seg seg_s[kMaxSegs];
  // per softmax warp: 32 rows x 64 bytes of output on their way to global memory
  // (first, until the first segments are planned, the units of every sequence)
  __shared__ __align__(16) uint8_t stage_s[kSoftWarps][32 * kStageRow];
  uint32_t* units_s = reinterpret_cast<uint32_t*>(stage_s);
  __shared__ uint32_t bad_s[kBadRing];
  __shared__ float2 ml_s[2][kM];
  volatile int* abort_flag = &abort_s;

  // ---- set-up; the units of every sequence (one kv head's) into shared memory
  if (warp == kMmaWarp) tc::tmem_alloc(&tmem_base_s, 512);
  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
      mbar_init(&v_part[s], 1);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(&s_full[w], 1);
      mbar_init(&p_full[w][0], 4);
      mbar_init(&p_full[w][1], 4);
      mbar_init(&o_done[w], 1);
    }
    mbar_init(&q_full, 1);
    mbar_init(&q_empty, 1);
    mbar_init(&all_done, 1);
    abort_s = 0;
    fence_mbar_init();
    a.part_head[cta * 8] = 0;   // no part of this CTA starts an item, so far
  }
  if (warp == kLoadWarp && lane == 0) {
    prefetch_tmap(&qmap);
    prefetch_tmap(&kmap);
    prefetch_tmap(&vmap);
  }
  for (int b = warp; b < a.B; b += kThreads / 32) {
    const Seq s = seq_of(a, b, cta == 0 && lane == 0 ? a.err : nullptr);
    const int nqt = (s.n + toks - 1) / toks;
    uint32_t u = 0;
    for (int qt = lane; qt < nqt; qt += 32) u += item_units(s, toks, a.window, qt);
    u = __reduce_add_sync(0xffffffffu, u);
    if (lane == 0) units_s[b] = u;
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = tmem_base_s;

  uint32_t kc = 0;                  // key tiles so far
  uint32_t cw0 = 0, cw1 = 0;        // S / P hand-overs so far, per tile (softmax: its own, cw0)
  uint32_t oc0 = 0, oc1 = 0;        // accumulators finished so far: this tile's, the other's
  uint32_t qc = 0;                  // query loads so far
  bool ok = true;

  // ---- roles: each runs through the planned segments, a batch at a time
  if (warp < kSoftWarps) {
    // ================= softmax and epilogue
    regs_up();
    for (int x = tid; x < C::kQBytes / 16; x += kSoftWarps * 32)   // tile A's queries: zero
      reinterpret_cast<uint4*>(q_s)[x] = make_uint4(0, 0, 0, 0);
    tc::fence_proxy_async();
    for (bool last = false; !last;) {
      cta_sync();
      const int n_segs = n_segs_s;
      last = last_s;
      const int w = warp >> 2, quarter = warp & 3;
      const int row = quarter * 32 + lane;
      const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
      const uint32_t s_col = tmem + lanes + 128 * w;
      const uint32_t o_col = tmem + lanes + 256 + D * w;
      const float sl = a.scale_log2;
      const int boxes_log2 = 31 - __clz(a.box);
      for (int i = 0; i < n_segs; ++i) {
        const Seg s = seg_s[i];
        const int nt = s.j1 - s.j0;
        const bool halves = s.nr <= tile_rows;
        const int n_w = halves ? (w ? nt / 2 : (nt + 1) / 2) : nt;
        const int n_other = halves ? (w ? (nt + 1) / 2 : nt / 2) : nt;
        const int rr = (halves ? 0 : w * tile_rows) + row;
        const bool row_ok = row < tile_rows && rr < s.nr;
        const bool warp_ok = __any_sync(0xffffffffu, row_ok);
        const int rg = s.r0 + rr;
        const int t = row_ok ? rg / G : 0;
        const int head = s.kvh * G + (row_ok ? rg - t * G : 0);
        // visible keys [vis_lo, vis_hi)
        const int qpos = s.L - s.n + t;
        const int vis_hi = min(s.L, qpos + 1);
        const int vis_lo = a.window ? qpos - a.window + 1 : 0;
        float m_ref = -INFINITY, l = 0.f;
        for (int it = 0; it < n_w; ++it, ++cw0) {
          const int ti = halves ? 2 * it + w : it;
          const int k0 = (s.j0 + ti) * kKeys;
          if (!all_well(ok, abort_flag)) break;
          ok = wait(&s_full[w], cw0 & 1);
          if (!warp_ok) {   // no rows here: whatever P holds reaches no row that is kept
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&p_full[w][0]);
              mbar_arrive(&p_full[w][1]);
            }
            continue;
          }
          tc::fence_after_sync();
          const int lo = vis_lo - k0, hi = vis_hi - k0;
          const uint32_t bad = bad_s[(kc + ti) % kBadRing];
          const bool masked =
              __any_sync(0xffffffffu, bad || (row_ok && (lo > 0 || hi < kKeys)));
          float x[128], m_new = m_ref;
          for (bool moved = false;;) {
            auto hide = [&] {
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                uint32_t vis = hi >= 32 * c + 32 ? 0xffffffffu
                                                 : hi > 32 * c ? (1u << (hi - 32 * c)) - 1u : 0u;
                if (lo > 32 * c)
                  vis &= lo >= 32 * c + 32 ? 0u : ~((1u << (lo - 32 * c)) - 1u);
                if (bad) {
#pragma unroll
                  for (int h = 0; h < 2; ++h)
                    if ((bad >> ((32 * c + 16 * h) >> boxes_log2)) & 1u)
                      vis &= ~(0xffffu << (16 * h));
                }
#pragma unroll
                for (int k = 0; k < 32; ++k)
                  if (!((vis >> k) & 1u)) x[32 * c + k] = -INFINITY;
              }
            };
#pragma unroll
            for (int c = 0; c < 4; ++c)
              tc::ld32(s_col + 32 * c, *reinterpret_cast<float(*)[32]>(&x[32 * c]));
            tc::wait_ld();
            if (masked) hide();
            if (moved) break;
            // (a NaN score makes the row's maximum, and so the row, NaN)
            const float mx = max_nan(max64(x, 0), max64(x, 64)) * sl;
            // (only rows that are kept: the others hold whatever their queries' memory does)
            const bool move = row_ok && !(mx <= m_ref + kLazy);
            if (!__any_sync(0xffffffffu, move)) break;
            const float alpha = move ? exp2f(m_ref - mx) : 1.f;
            m_new = move ? mx : m_ref;
            l *= alpha;
            if (it == 0) break;
            // this row's PV of the previous tile is complete; the scores are
            // read again afterwards, so that they hold no registers meanwhile
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              float o[32];
              tc::ld32(o_col + c * 32, o);
              tc::wait_ld();
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] *= alpha;
              tc::st32(o_col + c * 32, o);
            }
            moved = true;
          }
          const float nb = m_new == -INFINITY ? 0.f : -m_new;
          m_ref = m_new;
          unsigned long long ls[4] = {0ull, 0ull, 0ull, 0ull};
          const unsigned long long sl2 = f2_pack(sl, sl), nb2 = f2_pack(nb, nb);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t p[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const int e = 32 * c + 2 * k;
              const float2 z = f2_unpack(f2_fma(f2_pack(x[e], x[e + 1]), sl2, nb2));
              const float p0 = ex2_approx(z.x), p1 = ex2_approx(z.y);
              ls[k & 3] = f2_add(ls[k & 3], f2_pack(p0, p1));
              p[k] = pack_bf16(p0, p1);
            }
            tc::st16(s_col + 16 * c, p);
            if (c & 1) {   // 64 keys
              tc::wait_st();
              tc::fence_before_sync();
              __syncwarp();
              if (lane == 0) mbar_arrive(&p_full[w][c >> 1]);
            }
          }
          const float2 l0 = f2_unpack(f2_add(ls[0], ls[1])), l1 = f2_unpack(f2_add(ls[2], ls[3]));
          l += (l0.x + l0.y) + (l1.x + l1.y);
        }
        // ---- epilogue
        if (n_w > 0) {
          ok = ok && wait(&o_done[w], oc0 & 1);
          ++oc0;
        }
        float wa = 1.f, wb = 0.f, m_all = m_ref, l_all = l;
        const int id = 1 + quarter;
        if (halves) {   // the other half's running max and sum, and its accumulator
          if (n_other > 0) {
            ok = ok && wait(&o_done[1 - w], oc1 & 1);
            ++oc1;
          }
          ml_s[w][row] = make_float2(m_ref, l);
          pair_sync(id);
          const float2 other = ml_s[1 - w][row];
          m_all = fmaxf(m_ref, other.x);
          wa = m_ref == -INFINITY ? 0.f : exp2f(m_ref - m_all);
          wb = other.x == -INFINITY ? 0.f : exp2f(other.x - m_all);
          l_all = l * wa + other.y * wb;
        } else {
          if (nt > 0) ++oc1;
        }
        ok = all_well(ok, abort_flag);
        tc::fence_after_sync();
        const bool empty = !ok || l_all == 0.f;
        const float inv = empty ? 0.f : 1.f / l_all;
        wa *= inv;
        wb *= inv;
        const bool use_a = n_w > 0, use_b = halves && n_other > 0;
        const uint32_t b_col = tmem + lanes + 256 + D * (1 - w);
        const int orow = (s.q0 + t) * a.Hq + head;
        if (warp_ok) {
          // The rows leave through shared memory, 64 bytes of each at a time, so
          // that a store covers whole sectors.  Lane 4 r + p of a store holds
          // piece p of rows r, 8 + r, 16 + r, 24 + r.
          uint8_t* stage = stage_s[warp];
          const int mine = !row_ok ? -1 : s.part < 0 ? orow : s.part * a.rows_cap + rr;
          int dst_row[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            dst_row[k] = __shfl_sync(0xffffffffu, mine, 8 * k + (lane >> 2));
          uint8_t* dst = s.part < 0 ? reinterpret_cast<uint8_t*>(a.o)
                                    : reinterpret_cast<uint8_t*>(a.part_o);
          const int64_t row_bytes = s.part < 0 ? D * 2 : D * 4;
          auto flush = [&](int byte0) {
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint4 v = *reinterpret_cast<const uint4*>(
                  stage + (8 * k + (lane >> 2)) * kStageRow + (lane & 3) * 16);
              if (dst_row[k] >= 0)
                *reinterpret_cast<uint4*>(dst + dst_row[k] * row_bytes + byte0 + (lane & 3) * 16) =
                    v;
            }
            __syncwarp();
          };
          uint4* own = reinterpret_cast<uint4*>(stage + lane * kStageRow);
          // 32 columns (o, final) of every row, columns 32 c ..
          auto put = [&](const float* o, int c) {
            if (s.part < 0) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                own[k] = make_uint4(pack_bf16(o[8 * k], o[8 * k + 1]),
                                    pack_bf16(o[8 * k + 2], o[8 * k + 3]),
                                    pack_bf16(o[8 * k + 4], o[8 * k + 5]),
                                    pack_bf16(o[8 * k + 6], o[8 * k + 7]));
              flush(c * 64);
            } else {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  own[k] = make_uint4(__float_as_uint(o[16 * h + 4 * k]),
                                      __float_as_uint(o[16 * h + 4 * k + 1]),
                                      __float_as_uint(o[16 * h + 4 * k + 2]),
                                      __float_as_uint(o[16 * h + 4 * k + 3]));
                flush(c * 128 + h * 64);
              }
            }
          };
          // 32 columns at a time, in a loop that stays small (a whole row's worth of
          // straight-line code ran into instruction fetches: 196 us for the packed
          // prompts, 186 us so); halves: each of the two threads of a row writes half
          const int c0 = halves ? w * (D / 64) : 0, c1 = halves ? c0 + D / 64 : D / 32;
#pragma unroll 1
          for (int c = c0; c < c1; ++c) {
            float o[32];
            tc::ld32(o_col + c * 32, o);
            tc::wait_ld();
            // (an accumulator that was never written may hold anything)
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = empty || !use_a ? 0.f : o[k] * wa;
            if (use_b) {
              float ob[32];
              tc::ld32(b_col + c * 32, ob);
              tc::wait_ld();
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = empty ? 0.f : fmaf(ob[k], wb, o[k]);
            }
            put(o, c);
          }
          if (row_ok && !(halves && w)) {
            const float lse2 = empty ? -INFINITY : m_all + log2f(l_all);
            if (s.part >= 0)
              a.part_lse[(int64_t)s.part * a.rows_cap + rr] = lse2;
            else if (a.lse)
              a.lse[orow] = lse2 * kLn2;
          }
        }
        tc::fence_before_sync();
        if (halves) pair_sync(id);   // both accumulators read: the next item may write them
        kc += nt;
      }
      cta_sync();
    }
  } else {
    regs_down();
    if (warp == kLoadWarp) {
      // ================= K tiles
      for (bool last = false; !last;) {
        cta_sync();
        const int n_segs = n_segs_s;
        last = last_s;
        for (int i = 0; i < n_segs && ok; ++i) {
          const Seg s = seg_s[i];
          for (int j = s.j0; j < s.j1; ++j, ++kc) {
            const Box x = box_of(a, s, j, lane);
            if (lane == 0) {
              bad_s[kc % kBadRing] = x.bad;
              if (x.bad) set_dev_error(a.err, SA_DEVERR_POOL_RANGE);
            }
            ok = load_tile<D>(x, s.kvh, kc, k_s, &kmap, k_full, k_empty, a.box, abort_flag);
            if (!ok) break;   // kc: the tiles asked for
          }
        }
        cta_sync();
      }
    } else if (warp == kQWarp) {
      // ================= queries
      int q_rows = 0;   // rows of tile A's queries that may not be zero
      for (bool last = false; !last;) {
        cta_sync();
        const int n_segs = n_segs_s;
        last = last_s;
        for (int i = 0; i < n_segs && ok; ++i) {
          const Seg& s = seg_s[i];
          if (s.j0 == s.j1) continue;
          ok = all_well((qc == 0 || wait(&q_empty, (qc - 1) & 1)) && !*abort_flag, abort_flag);
          if (!ok) break;
          if (s.nr <= kFewRows) {
            // Few rows: copied by the warp, the tile's other rows zero.  (Boxes would
            // bring other tokens' rows along: products nobody needs, at a power that
            // lowers the clock -- 16 x 32K-key decode under load 424 us with, 410 us
            // without them.)
            constexpr int kPieces = D / 8;
            auto at = [&](int row, int pc) {
              return q_s + (pc >> 3) * (kM * 128) + row * 128 + (((pc & 7) ^ (row & 7)) << 4);
            };
            const uint16_t* src = a.q + (s.q0 + s.r0 / G) * a.q0 + (int64_t)s.kvh * G * a.q1;
            for (int x0 = lane; x0 < s.nr * kPieces; x0 += 32 * 4) {
              uint4 v[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int row = (x0 + 32 * k) / kPieces, pc = (x0 + 32 * k) % kPieces, t = row / G;
                if (row < s.nr)
                  v[k] = *reinterpret_cast<const uint4*>(src + t * a.q0 + (row - t * G) * a.q1 +
                                                         pc * 8);
              }
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int row = (x0 + 32 * k) / kPieces, pc = (x0 + 32 * k) % kPieces;
                if (row < s.nr) *reinterpret_cast<uint4*>(at(row, pc)) = v[k];
              }
            }
            for (int x = s.nr * kPieces + lane; x < q_rows * kPieces; x += 32)
              *reinterpret_cast<uint4*>(at(x / kPieces, x % kPieces)) = make_uint4(0, 0, 0, 0);
            q_rows = s.nr;
            tc::fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_full);
            ++qc;
            continue;
          }
          q_rows = kM;
          // one box per tile and 64-column chunk; rows of other sequences' tokens
          // that a box holds are never kept, tokens past the tensor load as zeros
          const int tiles = s.nr > tile_rows ? 2 : 1;
          if (lane == 0) mbar_arrive_expect_tx(&q_full, tiles * C::kChunks * tile_rows * 128);
          __syncwarp();
          if (lane < tiles * C::kChunks) {
            const int w = lane / C::kChunks, ch = lane % C::kChunks;
            tma_load_4d(q_s + w * C::kQBytes + ch * (kM * 128), &qmap, &q_full, ch * 64,
                        s.kvh * G, s.q0 + s.r0 / G + w * a.tile_toks, 0);
          }
          ++qc;
        }
        cta_sync();
      }
    } else if (warp == kMmaWarp) {
      // ================= MMA issue: warp-uniform code, one elected lane issues
      const std::integral_constant<int, 0> A{};
      const std::integral_constant<int, 1> B{};
      const uint32_t q_desc = uni(tc::desc_lo(smem_u32(q_s), 16));
      const uint32_t k_desc = uni(tc::desc_lo(smem_u32(k_s), 16));
      const uint32_t v_desc = uni(tc::desc_lo(smem_u32(v_s), kKeys * 128));
      const uint32_t tmem_u = uni(tmem);
      // One run of an item's tiles.  halves: each row tile has every other key tile.
      auto run = [&](int j0, int nt, int hi, auto hv) {
        constexpr bool halves = decltype(hv)::value != 0;
        const int n_a = halves ? (nt + 1) / 2 : nt, n_b = halves ? nt / 2 : nt;
        int qk_left = n_a + n_b;
        // S_w = Q_w K^T of the tile of iteration it
        auto qk = [&](int it, auto wc) {
          constexpr int w = decltype(wc)::value;
          const uint32_t c = kc + (halves ? 2 * it + w : it);
          const int st = c % C::kStages;
          if (halves || w == 0) {
            ok = wait(&k_full[st], (c / C::kStages) & 1) && ok;
            tc::fence_after_sync();
          }
          if (tc::elect_one()) {
            const uint32_t qd = q_desc + ((halves ? 0 : w) * C::kQBytes >> 4);
            const uint32_t kd = k_desc + st * (C::kTileBytes >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t o = ((kk >> 2) * (kM * 128) + (kk & 3) * 32) >> 4;
              tc::mma_bf16_lo(tmem_u + 128 * w, qd + o, kd + o, C::kIdQK, kk > 0 ? 1u : 0u);
            }
            tc::commit(&s_full[w]);
            // (what may still be on its way frees no stage)
            if (ok && (halves || w == 1)) tc::commit(&k_empty[st]);
            if (ok && qk_left == 1) tc::commit(&q_empty);
          }
          __syncwarp();
          --qk_left;
        };
        // O_w += P_w V of the tile of iteration it
        auto pv = [&](int it, auto wc) {
          constexpr int w = decltype(wc)::value;
          const int ti = halves ? 2 * it + w : it;
          const uint32_t c = kc + ti;
          const int st = c % C::kStages, j = j0 + ti;
          // 16-key steps some row of the item sees
          const int steps = min(8, (hi - j * kKeys + 15) / 16);
          const uint32_t vd = v_desc + st * (C::kTileBytes >> 4);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            ok = wait(&p_full[w][h], (w ? cw1 : cw0) & 1) && ok;
            if (h == 0 && (halves || w == 0)) ok = wait(&v_full[st], (c / C::kStages) & 1) && ok;
            tc::fence_after_sync();
            if (tc::elect_one()) {
#pragma unroll
              for (int kk = 4 * h; kk < 4 * h + 4; ++kk)
                if (kk < steps)
                  tc::mma_bf16_ts_lo(tmem_u + 256 + D * w, tmem_u + 128 * w + 8 * kk,
                                     vd + kk * (2048 >> 4), C::kIdPV,
                                     (it > 0 || kk > 0) ? 1u : 0u);
              if (h == 1) {
                if (ok && (halves || w == 1)) tc::commit(&v_empty[st]);
                if (it + 1 == (w ? n_b : n_a)) tc::commit(&o_done[w]);
              }
            }
            __syncwarp();
          }
          w ? ++cw1 : ++cw0;
        };
        ok = wait(&q_full, qc & 1) && ok;
        tc::fence_after_sync();
        qk(0, A);
        if (n_b > 0) qk(0, B);
        for (int it = 0; it < n_a && all_well(ok, abort_flag); ++it) {
          pv(it, A);
          if (it + 1 < n_a) qk(it + 1, A);
          if (it >= n_b) continue;
          pv(it, B);
          if (it + 1 < n_b) qk(it + 1, B);
        }
      };
      for (bool last = false; !last;) {
        cta_sync();
        const int n_segs = n_segs_s;
        last = last_s;
        for (int i = 0; i < n_segs && all_well(ok, abort_flag); ++i) {
          const Seg& s = seg_s[i];
          const int j0 = uni(s.j0), nt = uni(s.j1) - j0, nr = uni(s.nr);
          if (nt == 0) continue;
          const int hi = uni(min(s.L, s.L - s.n + (s.r0 + nr - 1) / G + 1));
          if (nr <= tile_rows)
            run(j0, nt, hi, B);
          else
            run(j0, nt, hi, A);
          kc += nt;
          ++qc;
        }
        all_well(ok, abort_flag);
        cta_sync();
      }
    } else if (warp == kPlanWarp) {
      // ================= planner, V tiles
      // ---- this CTA's share [w_pos, w_hi) of all units, and the item it starts in.
      // Shares of w_share or w_share + 1 units, the first w_extra of them the longer.
      // The units of sequences that share no tokens are fewer than 2^31 (checked on
      // the host); offsets that turn back (and are flagged) can give more, and then
      // nothing is planned.
      // The sum in 64 bits, the lanes' high and low parts added apart (each lane holds
      // at most 128 sequences of fewer than 2^31).
      int64_t w_sum = 0;
      for (int b = lane; b < a.B; b += 32) w_sum += units_s[b];
      w_sum = (static_cast<int64_t>(__reduce_add_sync(0xffffffffu, static_cast<uint32_t>(w_sum >> 16)))
               << 16) +
              __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(w_sum & 0xffff));
      const bool countable = w_sum <= 0x7fffffff / a.Hkv;
      const int w_total = countable ? static_cast<int>(w_sum) * a.Hkv : 0;
      const int n_eff = min(n_ctas, max(1, w_total / kMinUnits));
      const int w_share = w_total / n_eff, w_extra = w_total - w_share * n_eff;
      int w_pos = w_share * cta + min(cta, w_extra);
      const int w_hi = cta < n_eff ? w_pos + w_share + (cta < w_extra) : w_pos;
      int cb = 0, ckvh = 0, cqt = 0, c_off = 0;   // c_off: units of the item before w_pos
      auto scan = [&](int x) {   // inclusive, over the lanes
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        return x;
      };
      if (w_pos < w_hi) {
        int off = w_pos;
        for (int b0 = 0; b0 < a.B; b0 += 32) {   // the sequence, 32 at a time
          const int b = b0 + lane;
          const int own = b < a.B ? units_s[b] * a.Hkv : 0, incl = scan(own);
          const uint32_t m = __ballot_sync(0xffffffffu, incl > off);
          if (m) {
            const int src = __ffs(m) - 1;
            cb = b0 + src;
            off -= __shfl_sync(0xffffffffu, incl - own, src);
            break;
          }
          off -= __shfl_sync(0xffffffffu, incl, 31);
        }
        const int per_head = units_s[cb];
        ckvh = off / per_head;
        off -= ckvh * per_head;
        const Seq s = seq_of(a, cb, nullptr);
        const int nqt = (s.n + toks - 1) / toks;
        for (int q0 = 0; q0 < nqt; q0 += 32) {   // the row tile, 32 at a time
          const int qt = q0 + lane;
          const int own = qt < nqt ? item_units(s, toks, a.window, qt) : 0, incl = scan(own);
          const uint32_t m = __ballot_sync(0xffffffffu, incl > off);
          if (m) {
            const int src = __ffs(m) - 1;
            cqt = q0 + src;
            c_off = off - __shfl_sync(0xffffffffu, incl - own, src);
            break;
          }
          off -= __shfl_sync(0xffffffffu, incl, 31);
        }
      }
      uint32_t parts = 0;           // bit st: phase of v_part[st]
      uint64_t* part = nullptr;     // the one whose copy was given up on
      bool last = false;
      do {
        // the next segments
        if (lane == 0) {
          int ns = 0;
          while (w_pos < w_hi && ns < kMaxSegs && cb < a.B) {
            const Seq s = seq_of(a, cb, nullptr);
            const int nqt = (s.n + toks - 1) / toks;
            while (w_pos < w_hi && ns < kMaxSegs && ckvh < a.Hkv && nqt > 0) {
              const int2 t = tiles_of(s, toks, a.window, cqt);
              const int nt = t.y - t.x, units = kItemUnits + nt;
              const int ua = c_off, ub = min(units, c_off + (w_hi - w_pos));
              // units past the item's fixed cost are its tiles
              const int ta = max(0, ua - kItemUnits), tb = max(0, ub - kItemUnits);
              if (tb > ta || nt == 0) {
                Seg& g = seg_s[ns++];
                g.q0 = s.q0, g.n = s.n, g.k0 = s.k0, g.L = s.L;
                g.b = cb, g.kvh = ckvh;
                g.r0 = cqt * toks * G;
                g.nr = min(toks, s.n - cqt * toks) * G;
                g.j0 = t.x + ta, g.j1 = t.x + tb;
                g.part = -1;
                if (ta > 0 || tb < nt) {
                  g.part = 2 * cta + (ta == 0);
                  if (ta == 0) {   // the parts that follow are the next CTAs' first ones
                    const int e = w_pos - ua + units - 1;         // the item's last unit
                    const int cut = (w_share + 1) * w_extra;      // the longer shares' end
                    const int last =
                        e < cut ? e / (w_share + 1) : w_extra + (e - cut) / w_share;
                    int32_t* h = a.part_head + cta * 8;
                    h[0] = g.nr, h[1] = last - cta + 1;
                    h[2] = s.q0, h[3] = g.r0, h[4] = ckvh;
                  }
                }
              }
              w_pos += ub - ua;
              c_off = 0;
              if (ub == units && ++cqt == nqt) cqt = 0, ++ckvh;
            }
            if (ckvh == a.Hkv || nqt == 0) ckvh = 0, cqt = 0, ++cb;
          }
          n_segs_s = ns;
          last_s = w_pos >= w_hi || cb >= a.B;
        }
        __syncwarp();
        cta_sync();
        last = last_s;
        const int n_segs = n_segs_s;
        for (int i = 0; i < n_segs && ok; ++i) {   // V tiles
          const Seg s = seg_s[i];
          const int hi = min(s.L, s.L - s.n + (s.r0 + s.nr - 1) / G + 1);
          const int low = first_key(s.L, s.n, a.window);
          for (int j = s.j0; j < s.j1; ++j, ++kc) {
            // Value rows past the sequence's end, or behind the window of its first token,
            // may hold anything (0 * NaN).  A tile with such rows (only an item's last, up
            // to the 16-key step that is multiplied, or its first) arrives on a barrier of
            // its own, and on the ring's once they are zeroed: the issuing warp, whose
            // every instruction counts, knows nothing of it (two compares a tile there:
            // 8192-token prompt 513 -> 542 us).
            const int st = kc % C::kStages, below = max(0, low - j * kKeys);
            const int z0 = s.L - j * kKeys, nz = 16 * min(8, (hi - j * kKeys + 15) / 16) - z0;
            const bool whole = nz <= 0 && below == 0;
            ok = load_tile<D>(box_of(a, s, j, lane), s.kvh, kc, v_s, &vmap, whole ? v_full : v_part,
                              v_empty, a.box, abort_flag);
            if (!ok) break;
            if (whole) continue;
            ok = all_well(wait(&v_part[st], (parts >> st) & 1), abort_flag);
            if (!ok) {
              part = &v_part[st];
              break;
            }
            parts ^= 1u << st;
            auto zero = [&](int row, int n) {
              uint8_t* vt = v_s + st * C::kTileBytes + row * 128;
              for (int x = lane; x < n * 8; x += 32)
#pragma unroll
                for (int ch = 0; ch < C::kChunks; ++ch)
                  *reinterpret_cast<uint4*>(vt + ch * (kKeys * 128) + x * 16) =
                      make_uint4(0, 0, 0, 0);
            };
            zero(0, below);
            zero(z0, nz);
            tc::fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&v_full[st]);
          }
        }
        cta_sync();
      } while (!last);
      if (part) drain(part, (parts >> (part - v_part)) & 1);
    }
  }
  // (every role has passed its last barrier: no wait is left that could raise the flag)
  if (abort_s) {
    // leave only when no copy and no product of this CTA is in flight any more
    if (warp == kLoadWarp || warp == kPlanWarp) {
      uint64_t* full = warp == kLoadWarp ? k_full : v_full;
      for (uint32_t c = kc > (uint32_t)C::kStages ? kc - C::kStages : 0; c < kc; ++c)
        drain(&full[c % C::kStages], (c / C::kStages) & 1);
    } else if (warp == kQWarp) {
      if (qc > 0) drain(&q_full, (qc - 1) & 1);
    } else if (warp == kMmaWarp) {
      if (tc::elect_one()) tc::commit(&all_done);
      __syncwarp();
      drain(&all_done, 0);
    }
    if (tid == 0) set_dev_error(a.err, SA_DEVERR_TIMEOUT);
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

// Merge of the cut items: block x takes the item that starts in CTA x's share.
// A warp does R rows at a time, four columns per lane; part 0 is CTA x's starting
// part, the others the continuing parts of the CTAs after it.  Most cut items have
// two parts: both parts' loads of all rows are in flight together.
template <int D, int R>
__global__ void __launch_bounds__(512) dense_merge_kernel(const __grid_constant__ DenseArgs a) {
  pdl_wait_and_release();
  const int32_t* h = a.part_head + blockIdx.x * 8;
  const int4 h0 = *reinterpret_cast<const int4*>(h);
  const int nr = h0.x, np = h0.y, q0 = h0.z, row0 = h0.w, kvh = h[4];
  const int lane = threadIdx.x & 31;
  const int rr = (blockIdx.y * (blockDim.x >> 5) + (threadIdx.x >> 5)) * R;
  if (rr >= nr) return;
  const int G = a.Hq / a.Hkv, x = blockIdx.x;
  // row rr + r of part p (rows past the last: the last); fewer than 2^31 rows in all
  auto part_row = [&](int p, int r) {
    return (p == 0 ? 2 * x + 1 : 2 * (x + p)) * a.rows_cap + min(rr + r, nr - 1);
  };
  auto load = [&](int row) {
    return lane < D / 4 ? *reinterpret_cast<const float4*>(a.part_o + (int64_t)row * D + lane * 4)
                        : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  auto finish = [&](int r, float4 v, float m, float tot) {   // v: sum of 2^(lse - m) o
    if (rr + r >= nr) return;
    const float inv = m == -INFINITY ? 0.f : 1.f / tot;
    const int rg = row0 + rr + r, t = rg / G;
    const int orow = (q0 + t) * a.Hq + kvh * G + (rg - t * G);
    if (lane < D / 4)
      *reinterpret_cast<uint2*>(a.o + (int64_t)orow * D + lane * 4) = make_uint2(
          pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv));
    if (lane == 0 && a.lse) a.lse[orow] = m == -INFINITY ? m : (m + log2f(tot)) * kLn2;
  };
  if (np == 2) {
    float l0[R], l1[R];
    float4 o0[R], o1[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      l0[r] = a.part_lse[part_row(0, r)];
      l1[r] = a.part_lse[part_row(1, r)];
      o0[r] = load(part_row(0, r));
      o1[r] = load(part_row(1, r));
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float m = max_nan(l0[r], l1[r]);
      const float w0 = m == -INFINITY ? 0.f : exp2f(l0[r] - m);
      const float w1 = m == -INFINITY ? 0.f : exp2f(l1[r] - m);
      finish(r,
             make_float4(fmaf(w0, o0[r].x, w1 * o1[r].x), fmaf(w0, o0[r].y, w1 * o1[r].y),
                         fmaf(w0, o0[r].z, w1 * o1[r].z), fmaf(w0, o0[r].w, w1 * o1[r].w)),
             m, w0 + w1);
    }
    return;
  }
#pragma unroll 1
  for (int r = 0; r < R; ++r) {
    float m = -INFINITY, tot = 0.f;
    for (int p = lane; p < np; p += 32) m = max_nan(m, a.part_lse[part_row(p, r)]);
    for (int o = 16; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p0 = 0; p0 < np; p0 += 32) {
      const int p = p0 + lane;
      const float w = p < np && m != -INFINITY ? exp2f(a.part_lse[part_row(p, r)] - m) : 0.f;
      tot += w;
      const int cnt = min(32, np - p0);
#pragma unroll 4
      for (int i = 0; i < cnt; ++i) {
        const float wi = __shfl_sync(0xffffffffu, w, i);
        const float4 v = load(part_row(p0 + i, r));
        acc.x = fmaf(wi, v.x, acc.x);
        acc.y = fmaf(wi, v.y, acc.y);
        acc.z = fmaf(wi, v.z, acc.z);
        acc.w = fmaf(wi, v.w, acc.w);
      }
    }
    for (int o = 16; o; o >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, o);
    finish(r, acc, m, tot);
  }
}

template <int D>
cudaError_t launch_d(const DenseArgs& a, const CUtensorMap& qmap, const CUtensorMap& kmap,
                     const CUtensorMap& vmap, cudaStream_t stream) {
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  e = allow_max_dyn_smem(reinterpret_cast<const void*>(dense_kernel<D>));
  if (e != cudaSuccess) return e;
  const int ctas = sms < kDenseMaxCtas ? sms : kDenseMaxCtas;
  dense_kernel<D><<<ctas, kThreads, Cfg<D>::kDyn, stream>>>(a, qmap, kmap, vmap);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // the merge is launched under the first kernel's tail (it waits for its end); a
  // warp does one row where rows are few, two where they are many (four, in blocks
  // of 32 warps: 16 x 32K-key decode 358 us, so 354, each in a burst of replays)
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = stream;
  if (a.rows_cap <= 64) {
    cfg.gridDim = dim3(ctas, (a.rows_cap + 15) / 16);
    cfg.blockDim = dim3(32 * (a.rows_cap < 16 ? a.rows_cap : 16));
    return cudaLaunchKernelEx(&cfg, dense_merge_kernel<D, 1>, a);
  }
  cfg.gridDim = dim3(ctas, (a.rows_cap + 31) / 32);
  cfg.blockDim = dim3(512);
  return cudaLaunchKernelEx(&cfg, dense_merge_kernel<D, 2>, a);
}

int rows_cap_of(int total_q, int Hq, int Hkv) {
  const int G = Hq / Hkv, item = 2 * dense_tile_toks(G);
  return (total_q < item ? total_q : item) * G;
}
size_t r16(size_t x) { return (x + 15) / 16 * 16; }

}  // namespace

int dense_tile_toks(int G) { return kM / G; }
size_t dense_workspace_bytes(int total_q, int Hq, int Hkv, int D) {
  const size_t rows = 2 * (size_t)kDenseMaxCtas * rows_cap_of(total_q, Hq, Hkv);
  return kDenseMaxCtas * 32 + r16(rows * 4) + rows * D * 4;
}
void dense_workspace(DenseArgs* a, void* ws) {
  a->rows_cap = rows_cap_of(a->total_q, a->Hq, a->Hkv);
  const size_t rows = 2 * (size_t)kDenseMaxCtas * a->rows_cap;
  uint8_t* p = static_cast<uint8_t*>(ws);
  a->part_head = reinterpret_cast<int32_t*>(p);
  a->part_lse = reinterpret_cast<float*>(p + kDenseMaxCtas * 32);
  a->part_o = reinterpret_cast<float*>(p + kDenseMaxCtas * 32 + r16(rows * 4));
}

cudaError_t launch_dense(const DenseArgs& a, const CUtensorMap& qmap, const CUtensorMap& kmap,
                         const CUtensorMap& vmap, cudaStream_t stream) {
  switch (a.D) {
    case 64: return launch_d<64>(a, qmap, kmap, vmap, stream);
    case 128: return launch_d<128>(a, qmap, kmap, vmap, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace sa
