// head_sm100.cuh -- losses of the output head on logits that are never
// stored: z = x W^T / tau for N token rows x [N][C] and V vocabulary rows
// W [V][C] (bf16, fp32 accumulate).
//
// Forward. Row n needs lse_n = log sum_v exp z[n][v] and z at the few ids its
// loss names (the target, or a teacher's list). The logits are formed one
// 256 x 256 tile at a time in tensor memory (256 x 128 where that fills more
// pairs of CTAs); the epilogue keeps, per row and half a tile, the running
// maximum and sum of exponentials (fp32, base 2) and the named logits, 8 bytes
// per 128 (64) logits instead of the logits.
//
// Backward. With p = exp(z - lse) the gradient of the logits is
//     dz[n][v] = (dloss_n + dlse_n) / tau * p[n][v] - dloss_n / tau * q[n][v],
// q the row's target distribution (non-zero at the named ids only), and
//     dx = dz W,   dW = dz^T x.
// The vocabulary is taken in pieces: the logits of a piece are formed again,
// dz of the piece is rounded to bf16 (the tensor cores' operand type; at most
// half a step, 2^-8 relative, which the sums of both products average) into a
// buffer that the two products of the piece read. dx is summed over the pieces
// in fp32, dW of a piece is final. In a row of dx one entry of dz, the target's,
// outweighs the others: where few ids are named, what their rounding takes is
// kept and added to dx in fp32, times their rows of W.
// Where the sums are short or more bits are asked for, dz is carried in two bf16
// terms, hi + lo (2^-16 relative): lo goes to a buffer of its own, whose K blocks
// follow hi's in the same accumulator. With an fp32 dW always; and where at most
// one row tile is kept, since an element of dW then comes from few entries,
// whose roundings do not average: they took the error of a bf16 dW to twice its
// output's own rounding (2 rows, 631 ids: 3.8e-3 of dW for 1.7e-3). dx takes
// lo too where it has no fp32 remainders of named columns. 100 rows of width
// 768 against 24576 ids take 61 us so, 55 with one term.
// A bf16 dW of more rows takes lo where a row names its foremost id (the target,
// or a teacher's largest share): that entry outweighs its row, and when every
// row's dloss is the same, as in a mean, all of them round alike and the error
// is one factor, up to 2^-8, on their part of dW. The row pass sorts the kept
// rows by the vocabulary tile of that id, so blocks of 64 rows meet the tiles
// they name along a staircase: at most (rows / 64 + tiles) blocks of lo exist,
// of rows / 64 x tiles, and they are all that is stored and multiplied. 8192
// rows of width 768: 0.96 ms before, 0.98 with lo, the sort and the gather of x;
// all of lo (an fp32 dW) takes 36 % more.
//
// Rows whose target is absent (or whose upstream gradients are both zero) are
// left out: the kept rows are compacted first, so the products cost what the
// kept rows cost, and what a left-out row holds (NaN included) reaches
// nothing. Their number lives on the device; every kernel reads it there.
//
// One kernel, head_gemm_kernel, runs all products of a call in one launch:
// clusters of two CTAs, each pair taking 256 x 256 output tiles (units) one
// after the other from a common counter. The backward's units are ordered
//     dz(0) dz(1) | dW(0) dx(0) dz(2) | dW(1) dx(1) dz(3) | ...
// (dx before dW where its units are the longer ones)
// with dz in three buffers, so what a unit waits for (its piece's dz, the
// readers of the buffer it overwrites, the previous piece's sums in dx) was
// handed out a whole group of units earlier. Waits are on counters in global
// memory and point only to units handed out before, so they end whatever the
// number of CTAs that run at a time.
//
// What bounds it: the tensor cores, and under a steady load the power limit.
// At 8192 rows, width 2048, 32063 ids the forward's products fill 95 % of the
// tensor cores' cycles (0.77 ms, 1395 TFLOP/s with the clock down to 1.37 GHz),
// and the backward takes 2.67 to 2.74 ms (1180 to 1210 TFLOP/s at 1.25-1.3 GHz);
// at width 768, where a logits tile is 12 stages long and its epilogue nearly as
// long, they fill 91 % and 79 % (0.303 and 1.11 ms). The same products by cuBLAS
// on the same box, logits stored: 0.84 and 2.46 to 2.50 ms, 0.37 and 1.05 ms.
#pragma once

#include <limits.h>

#include "common.cuh"
#include "sm100.cuh"

namespace head100 {

using namespace sm100;

constexpr int kTile = 256;            // output tile of a CTA pair (rows and columns)
constexpr int kKB = 64;               // K values per ring stage
constexpr int kStages = 5;  // 6 measured no faster; the room goes to the staging
constexpr int kOperandBytes = 128 * kKB * 2;  // 128 rows (or columns) of a stage
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// Named ids per row up to which the forward also takes their logits, and the
// backward their part of dx, in plain fp32. More of them average the errors
// that this is about, and their rows of W would cost more than the products
// hide.
constexpr int kFewNamed = 4;
constexpr int kPairs = 74;            // CTA pairs of a full persistent grid (148 SMs)

constexpr int kEpiWarps = 8;
constexpr int kThreads = 96 + 32 * kEpiWarps;  // TMA, MMA, epilogue, hand-out or dot-product warps
constexpr int kDzBuffers = 3;
constexpr int kTickets = 4;  // units known ahead, a ring in shared memory
// A pair takes its next unit when the loads of the last one end in kAhead
// stages (numbers taken earlier would keep long units from idle pairs at the
// end: 11 % of the backward at C = 768); units shorter than that run ahead.
constexpr int kAhead = 10;
constexpr int kSmRing = 0;
constexpr int kSmStage = kStages * kStageBytes;          // 2 x 4 KB per epilogue warp
constexpr int kSmBars = kSmStage + kEpiWarps * 8192;
constexpr int bFull = 0, bEmpty = kStages, bAccFull = 2 * kStages, bAccEmpty = 2 * kStages + 2,
              bTkFull = 2 * kStages + 4, bTkEmpty = bTkFull + kTickets, bWant = bTkEmpty + kTickets,
              bTkRead = bWant + 1;
constexpr int kNumBars = (bTkRead + kTickets + 1) / 2 * 2;  // what follows is 16-byte aligned
constexpr int kSmTickets = kSmBars + kNumBars * 8;       // kTickets x 32 bytes
constexpr int kSmMisc = kSmTickets + kTickets * 32;
constexpr int kSmAlloc = kSmMisc + 16;
static_assert(kSmAlloc <= 232448, "shared memory of one CTA");
static_assert(kSmTickets % 16 == 0 && kSmStage % 1024 == 0, "alignment");

enum Kind : int { LSE = 0, DZ = 1, DX = 2, DW = 3, END = 4 };

struct Maps {
  // operand loads: _k with K contiguous (boxes of 64 K x 128 rows; W's of 64
  // rows for narrow logits tiles), _mn with
  // the row index contiguous (boxes of 64 rows x 64 K, two of them in one box
  // when the extent is a multiple of 64)
  CUtensorMap x_k, xc_k, w_k, x_mn, xc_mn, w_mn, dz_k[kDzBuffers], dz_mn[kDzBuffers];
  CUtensorMap lo_k[kDzBuffers], lo_mn[kDzBuffers];
  // output boxes of 32 rows x 128 bytes
  CUtensorMap dz_out[kDzBuffers], lo_out[kDzBuffers], dx_out, dw_out;
};

// What a kept row brings to its logits' epilogue, by kept row: lse in base 2,
// the factors of p and of q in dz, and its target (one named id) or its row.
struct __align__(16) RowPar {
  float lse2, ca, cb;
  int id;
};

struct Params {
  const uint4 *x, *w;
  int N, V, C;
  int K;                 // named ids per row (1: the target)
  int piece, pieces;     // vocabulary rows per piece (all of V in the forward)
  int lw;                // columns of a logits tile: 256, or 128 where those are few
  int c_blocks;          // C % 64 == 0: _mn maps of x and W take both 64-wide blocks in one box
  int dw_f32;
  int lo_rows;           // 64-row blocks per vocabulary tile in lo's buffers
  const int* key;        // by kept row: the id of its foremost entry, or null
  const int* tile_start; // rows go by key: the first of each vocabulary tile; or null
  float inv_tau;
  // null in a forward of one row tile, which takes all rows as they are
  const int* n_kept;     // rows kept (device)
  const int* row_of;     // kept row -> row
  const RowPar* par;     // by kept row
  const int* ids;        // [N][K]: the targets, or a teacher's ids, ascending
  const float* share;    // [N][K] q, or null (1 at the target)
  const uint16_t* first; // [N][first_pitch] entries with an id below b lw / 2 (with share)
  int first_pitch;
  float2* part;          // LSE: [2 logits tiles][row_pitch] maximum (base 2), sum
  float* named;          // LSE: [kept row][K] z at the row's ids
  float* exact;          // the same from plain fp32 sums, for few ids per row, or null
  int row_pitch;
  // what rounding dz to bf16 takes from the row's named columns, by kept row,
  // where they are few, or from its foremost one (rest_k of them a row): dx gets
  // it back times their rows of W (or null)
  float* rest;
  int rest_k;
  const float* acc;      // fp32 sums of dx, slot_rows(kept) rows per split
  __nv_bfloat16* dx;
  // zero at launch: [0] the next unit; then counters, in epilogue warps: per
  // piece readers of dz and finished dx, per 256 vocabulary columns finished dz
  unsigned* ctl;
};
constexpr int kCtlPieces = 4;  // first per-piece counter in ctl
__host__ __device__ inline int ctl_words(int V, int pieces) {
  return kCtlPieces + 2 * pieces + (V + kTile - 1) / kTile;
}

// dx has few tiles when few rows are kept: its K axis (the vocabulary) is
// then split over units, each with an accumulator of its own that a closing
// pass adds in order (no atomics on values: results repeat). At most one unit
// per CTA pair, at least eight K blocks each.
__host__ __device__ inline void split_dx(int tiles, int kb_total, int& splits, int& kb_per) {
  splits = 1;
  if (tiles > 0 && tiles < kPairs) {
    splits = kPairs / tiles;
    const int most = kb_total / 8 > 1 ? kb_total / 8 : 1;
    splits = splits < most ? splits : most;
  }
  kb_per = (kb_total + splits - 1) / splits;
  if (kb_per < 1) kb_per = 1;
  splits = (kb_total + kb_per - 1) / kb_per;
  if (splits < 1) splits = 1;
}

// Rows of one dx accumulator (a multiple of the tile).
__host__ __device__ inline int slot_rows(int kept) { return (kept + kTile - 1) / kTile * kTile; }

// The units of a call, for `kept` rows.
struct Sched {
  int pieces, piece, V, lw;
  int tm, tc;          // tiles of kept rows, of C
  int kb_c, kb_n;      // K blocks of the logits, of dW
  int splits, kb_per;  // of dx over a whole piece
  // terms of dz that dW and dx take: 1, or 2, whose K blocks follow the first's
  int dw_terms, dx_terms;
  const int* tile_start;  // null where rows are in order
  int lo_step;            // 64-row blocks of lo between one vocabulary tile and the next
  bool dx_first;       // the longer units of a group go first
  __host__ __device__ int cols(int p) const { return p + 1 < pieces ? piece : V - p * piece; }
  __host__ __device__ int tv(int p) const { return (cols(p) + kTile - 1) / kTile; }
  __host__ __device__ int kb_v(int p) const { return (cols(p) + kKB - 1) / kKB; }
  // a shorter last piece keeps the parts' length: it adds into accumulators
  // that the first piece has written
  __host__ __device__ int splits_of(int p) const { return (kb_v(p) + kb_per - 1) / kb_per; }
  __host__ __device__ int tl(int p) const { return (cols(p) + lw - 1) >> (lw == kTile ? 8 : 7); }
  __host__ __device__ int dz(int p) const { return tm * tl(p); }
  __host__ __device__ int dw(int p) const { return tv(p) * tc; }
  __host__ __device__ int dx(int p) const { return tm * tc * splits_of(p); }
};
__host__ __device__ inline Sched make_sched(const Params& p, int kept) {
  Sched s;
  s.pieces = p.pieces;
  s.piece = p.piece;
  s.V = p.V;
  s.lw = p.lw;
  s.tm = (kept + kTile - 1) / kTile;
  s.tc = (p.C + kTile - 1) / kTile;
  s.kb_c = (p.C + kKB - 1) / kKB;
  s.kb_n = (kept + kKB - 1) / kKB;
  split_dx(s.tm * s.tc, s.kb_v(0), s.splits, s.kb_per);
  s.dw_terms = p.dw_f32 || kept <= kTile ? 2 : 1;
  s.dx_terms = p.K <= kFewNamed ? 1 : s.dw_terms;
  s.tile_start = s.dw_terms == 1 ? p.tile_start : nullptr;
  s.lo_step = s.tile_start ? 1 : p.lo_rows;
  // split dx units are one per pair and the last to have their dz: they end a
  // group (100 rows, first: 54 us)
  s.dx_first = s.splits == 1 && s.kb_per * s.dx_terms > s.kb_n * s.dw_terms;
  return s;
}

struct __align__(16) Unit {
  int kind, p, tm, tn, split, kb0, nkb, pad;
};

// Tile r of tiles_m x tiles_n: bands of `high` row tiles, columns within a
// band, rows fastest. Bands of 8 let the 74 pairs work on about 8 x 9 tiles at a
// time, whose operands (17 x 256 rows of K) come from L2; the logits take bands
// of 32, whose rows of x stay in L2 while W passes once per band. Width 2048:
// forward 0.742 ms (0.800 in bands of 8), backward 2.54 ms (2.67 all in 32).
constexpr int kBand = 8, kLogitsBand = 32;
__device__ __forceinline__ void band_tile(int r, int tiles_m, int tiles_n, int high, int& tm,
                                          int& tn) {
  const int band = r / (high * tiles_n);
  r -= band * high * tiles_n;
  const int h = min(high, tiles_m - band * high);
  tn = r / h;
  tm = band * high + r - tn * h;
}

// Unit u in the order above; kind END past the last one.
template <bool kBwd>
__device__ __forceinline__ Unit find_unit(const Sched& s, int u) {
  Unit o = {};
  o.kind = END;
  auto logits = [&](int kind, int p) {
    o.kind = kind;
    o.p = p;
    o.nkb = s.kb_c;
    band_tile(u, s.tm, s.tl(p), kLogitsBand, o.tm, o.tn);
  };
  if constexpr (!kBwd) {
    if (u < s.dz(0)) logits(LSE, 0);
  } else {
    for (int p = 0; p < min(2, s.pieces); ++p) {
      if (u < s.dz(p)) {
        logits(DZ, p);
        return o;
      }
      u -= s.dz(p);
    }
    // groups of whole pieces have one size
    const int group = s.dw(0) + s.dx(0) + s.dz(0);
    int p = s.pieces > 3 ? min(u / group, s.pieces - 3) : 0;
    u -= p * group;
    for (; p < s.pieces; ++p) {
      for (int k = 0; k < 2; ++k) {
        if ((k == 0) == s.dx_first) {
          if (u < s.dx(p)) {
            o.kind = DX;
            o.p = p;
            const int tiles = s.tm * s.tc;
            o.split = u / tiles;
            band_tile(u - o.split * tiles, s.tm, s.tc, kBand, o.tm, o.tn);
            o.kb0 = o.split * s.kb_per;
            o.nkb = (min(s.kb_v(p), o.kb0 + s.kb_per) - o.kb0) * s.dx_terms;
            return o;
          }
          u -= s.dx(p);
        } else {
          if (u < s.dw(p)) {
            o.kind = DW;
            o.p = p;
            o.nkb = s.kb_n * s.dw_terms;
            band_tile(u, s.tv(p), s.tc, kBand, o.tm, o.tn);
            if (s.tile_start) {  // lo of the rows that name this tile
              const int* at = s.tile_start + p * (s.piece / kTile) + o.tm;
              const int r0 = at[0], r1 = at[1];
              if (r0 < r1) {
                o.kb0 = r0 / kKB;
                o.nkb += (r1 + kKB - 1) / kKB - o.kb0;
              }
            }
            return o;
          }
          u -= s.dw(p);
        }
      }
      if (p + 2 < s.pieces) {
        if (u < s.dz(p + 2)) {
          logits(DZ, p + 2);
          return o;
        }
        u -= s.dz(p + 2);
      }
    }
  }
  return o;
}

// ---- instructions this kernel adds to sm100.cuh's ----
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(src), "r"(c0), "r"(c1)
      : "memory");
}
__device__ __forceinline__ void tma_reduce_add_2d(const CUtensorMap* map, uint32_t src, int c0,
                                                  int c1) {
  asm volatile(
      "cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(src), "r"(c0), "r"(c1)
      : "memory");
}
__device__ __forceinline__ void st_shared_v4(uint32_t a, uint32_t x, uint32_t y, uint32_t z,
                                             uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}
__device__ __forceinline__ float ld_shared_f32(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_shared_v4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ void st_shared_f32(uint32_t a, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}
// Into the shared memory of either CTA of the pair (an address of map_rank).
__device__ __forceinline__ void st_cluster_v4(uint32_t a, int x, int y, int z, int w) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z),
               "r"(w)
               : "memory");
}
// Arrive for reads of tensor memory that tcgen05.wait::ld and
// tcgen05.fence::before_thread_sync have closed: nothing else hangs on it.
__device__ __forceinline__ void mbar_arrive_tmem(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}
// mma_ss_pair by the lanes with `issue` set, without a branch.
__device__ __forceinline__ void mma_pair_if(uint32_t issue, uint32_t d_tmem, uint64_t a_desc,
                                            uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(issue)
      : "memory");
}
__device__ __forceinline__ void fence_proxy_async() {
  asm volatile("fence.proxy.async;" ::: "memory");
}
__device__ __forceinline__ unsigned ld_acquire(const unsigned* p) {
  unsigned v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void red_release(unsigned* p, unsigned v) {
  asm volatile("red.release.gpu.global.add.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// A warp's bounded wait, one answer for all of its lanes.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag));
}
__device__ __forceinline__ bool warp_wait_cl(uint32_t bar, uint32_t parity,
                                             volatile int* abort_flag) {
  return __all_sync(0xffffffffu, mbar_wait_cl(bar, parity, abort_flag));
}

__device__ __forceinline__ void red_relaxed(unsigned* p, unsigned v) {
  asm volatile("red.relaxed.gpu.global.add.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// Bounded wait for a counter of ctl, then for loads by TMA of what was written
// before it was raised.
__device__ __forceinline__ bool wait_count(const unsigned* c, unsigned want,
                                           volatile int* abort_flag) {
  if (ld_acquire(c) < want) {
    const long long t0 = clock64();
    while (ld_acquire(c) < want) {
      if (*abort_flag) return false;
      if (clock64() - t0 > kWaitLimitCycles) {
        *abort_flag = 1;
        report_status(ATTN_ETIMEOUT);
        return false;
      }
      __nanosleep(100);
    }
  }
  fence_proxy_async();
  return true;
}

__device__ __forceinline__ bool warp_count(const unsigned* c, unsigned want,
                                           volatile int* abort_flag) {
  return __all_sync(0xffffffffu, wait_count(c, want, abort_flag));
}

// Bounded wait for dz of the vocabulary tiles t0 to t1, a lane per tile; also
// looks at those behind (up to `end`): `to` is one past the last of the tiles
// from t0 on that were there without a gap. A tile's counter gets one from every
// epilogue warp of its logits tiles, two of these per row tile where they are
// narrow (one where the vocabulary ends in the tile's first half).
__device__ __forceinline__ bool wait_tiles(const unsigned* done, int t0, int t1, int end,
                                           const Sched& sc, int lane, int& to,
                                           volatile int* abort_flag) {
  const long long start = clock64();
  bool ok = true;
  to = t0;
  while (to <= t1) {
    const int t = to + lane;
    const int left = sc.V - t * kTile;
    const unsigned want = 2u * kEpiWarps * sc.tm * (left > sc.lw && sc.lw < kTile ? 2 : 1);
    const bool there = t < end && ld_acquire(done + t) >= want;
    const unsigned gap = ~__ballot_sync(0xffffffffu, there);
    to += gap ? __ffs(gap) - 1 : 32;
    if (to <= t1 && (gap & 1u)) {
      ok = *abort_flag == 0;
      if (ok && clock64() - start > kWaitLimitCycles) {
        *abort_flag = 1;
        report_status(ATTN_ETIMEOUT);
        ok = false;
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      __nanosleep(100);
    }
  }
  __syncwarp();
  fence_proxy_async();
  return ok;
}

// 128 rows (K contiguous: row0.., K from k0) or 128 columns (row index
// contiguous: from row0, 64 K rows from k0) of an operand into dst.
__device__ __forceinline__ void load_operand(const CUtensorMap* m, bool mn, bool one_box, int row0,
                                             int k0, uint32_t dst, uint32_t bar) {
  if (!mn) {
    tma_load_2d_pair(dst, m, bar, k0, row0);
  } else if (one_box) {
    tma_load_3d_pair(dst, m, bar, 0, k0, row0 >> 6);
  } else {
    tma_load_2d_pair(dst, m, bar, row0, k0);
    tma_load_2d_pair(dst + kOperandBytes / 2, m, bar, row0 + 64, k0);
  }
}

// s += g times four bf16 values.
__device__ __forceinline__ void add_scaled4(float4& s, float g, uint2 v) {
  s.x = fmaf(g, __uint_as_float(v.x << 16), s.x);
  s.y = fmaf(g, __uint_as_float(v.x & 0xffff0000u), s.y);
  s.z = fmaf(g, __uint_as_float(v.y << 16), s.z);
  s.w = fmaf(g, __uint_as_float(v.y & 0xffff0000u), s.w);
}

// A teacher's list of one row, from the entry that the current 128 columns
// begin with: the ids of the next entries (INT_MAX past the last one of these
// columns), with their shares in the backward. kDeep of them are on their way:
// a row with many entries in a tile takes them one after the other.
template <bool kShares>
struct Named {
  static constexpr int kDeep = 4;
  const int* ids;
  const float* shares;
  int pos, end, id[kDeep];
  float share[kDeep];
  __device__ __forceinline__ void load(int d, int at) {
    id[d] = at < end ? ids[at] : INT_MAX;
    if constexpr (kShares) share[d] = at < end ? shares[at] : 0.f;
  }
  __device__ __forceinline__ void none() {
    pos = end = 0;
#pragma unroll
    for (int d = 0; d < kDeep; ++d) id[d] = INT_MAX;
  }
  __device__ __forceinline__ void list(const int* row_ids, const float* row_shares, int from,
                                       int to) {
    ids = row_ids;
    shares = row_shares;
    pos = from;
    end = to;
#pragma unroll
    for (int d = 0; d < kDeep; ++d) load(d, from + d);
  }
  __device__ __forceinline__ void advance() {
    ++pos;
#pragma unroll
    for (int d = 0; d + 1 < kDeep; ++d) {
      id[d] = id[d + 1];
      share[d] = share[d + 1];
    }
    load(kDeep - 1, pos + kDeep - 1);
  }
};

// kBwd: the backward's units, else the forward's. kLw: columns of a logits
// tile. Kernels of their own, so that none carries another's epilogues (a width
// known at run time cost short tiles up to 11 %).
template <bool kBwd, int kLw>
__global__ void __launch_bounds__(kThreads, 1)
    head_gemm_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t sb0 = smem_u32(smem_raw);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem_raw + kSmMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem_raw + kSmMisc + 4);
  auto bar = [&](int i) -> uint32_t { return sb0 + kSmBars + 8u * i; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  if (sb0 & 1023u) {  // uniform across the cluster: nothing has been issued yet
    if (threadIdx.x == 0) report_status(ATTN_ECUDA_LAYOUT);
    return;
  }
  // set up before waiting for the row pass: nothing here touches global memory
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar(bFull + s), 1);
      mbar_init(bar(bEmpty + s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(bar(bAccFull + a), 1);
      mbar_init(bar(bAccEmpty + a), 2 * kEpiWarps);  // the epilogue warps of both CTAs
    }
    for (int t = 0; t < kTickets; ++t) {
      mbar_init(bar(bTkFull + t), 1);
      // readers: CTA 0's epilogue, TMA and MMA warps, and for those of CTA 1,
      // which arrive on its bTkRead, one that passes it on
      mbar_init(bar(bTkEmpty + t), kEpiWarps + 3);
      mbar_init(bar(bTkRead + t), kEpiWarps + 1);
    }
    mbar_init(bar(bWant), 1);
    *abort_flag = 0;
    prefetch_tensor_map(&maps.x_k);
    prefetch_tensor_map(&maps.w_k);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(sb0 + kSmMisc, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers ready before cross-CTA signals
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait_and_trigger();
  const int kept = !kBwd && !p.n_kept ? p.N : *p.n_kept;

  // Unit n of this pair (every reader of the ring calls it once per n). The
  // forward's units are all alike and wait for nothing: they are dealt in turn,
  // without a counter to clear (taking numbers measured up to 1 % slower).
  const Sched sc = make_sched(p, kept);
  auto next_unit = [&](int n, Unit& un) -> bool {
    if constexpr (!kBwd) {
      un = find_unit<kBwd>(sc, (int)(blockIdx.x >> 1) + n * (int)(gridDim.x >> 1));
      return un.kind != END;
    }
    const int t = n % kTickets;
    if (!warp_wait_cl(bar(bTkFull + t), (n / kTickets) & 1, abort_flag)) return false;
    const int4* src = reinterpret_cast<const int4*>(smem_raw + kSmTickets + t * 32);
    const int4 a = src[0], b = src[1];
    un.kind = a.x;
    un.p = a.y;
    un.tm = a.z;
    un.tn = a.w;
    un.split = b.x;
    un.kb0 = b.y;
    un.nkb = b.z;
    const bool more = __any_sync(0xffffffffu, un.kind != END);  // every lane has its values
    if (lane == 0) mbar_arrive(bar((rank == 0 ? bTkEmpty : bTkRead) + t));
    __syncwarp();
    return more;
  };
  unsigned* const dz_used = p.ctl + kCtlPieces;
  unsigned* const dx_done = dz_used + p.pieces;
  unsigned* const dz_done = dx_done + p.pieces;  // by vocabulary tile

  // The TMA and MMA warps run their loops converged, one elected lane issuing:
  // the operands of the issue then live in uniform registers. Issued from a
  // branch of one thread, a tcgen05.mma cost 130 cycles whatever its size;
  // so, 64 cycles at N = 128 and 128 at N = 256, the tensor core's own time.
  if (warp == 0) {
    // ---------------- TMA ----------------
    const bool el = elect_one();
    const bool all = kept == p.N && !sc.tile_start;  // x is read in place
    int s = 0;
    uint32_t phase = 1;  // a fresh barrier's previous phase counts as complete
    int used_ok = -1, dx_ok = -1;  // pieces whose counters are known to be full
    int dz_from = 0, dz_to = 0;    // vocabulary tiles whose dz is known to be there
    bool ok = true;
    Unit un;
    for (int n = 0; ok && next_unit(n, un); ++n) {
      const CUtensorMap *ma, *mb;
      bool a_mn = false, b_mn = true, b_one = p.c_blocks != 0;
      const int v0 = un.p * p.piece, buf = un.p % kDzBuffers;
      int bk = 0, brow = un.tn * kTile + rank * 128, bytes = 2 * kStageBytes;
      int nhi = un.nkb;  // blocks of hi; those of lo follow
      const int arow = un.tm * kTile + rank * 128;
      if (!kBwd || un.kind == DZ) {
        ma = all ? &maps.x_k : &maps.xc_k;
        mb = &maps.w_k;
        b_mn = false;
        brow = v0 + un.tn * kLw + rank * (kLw / 2);
        bytes = 2 * (kOperandBytes + kKB * kLw);  // lw / 2 rows of 128 bytes
        const int q = un.p - kDzBuffers;  // the piece whose dz this one overwrites
        if (q > used_ok) {
          if (!warp_count(dz_used + q, 2u * (sc.dw(q) + sc.dx(q)), abort_flag)) break;
          used_ok = q;
        }
      } else {
        if (un.kind == DX) {
          ma = &maps.dz_k[buf];
          mb = &maps.w_mn;
          bk = v0;
          nhi /= sc.dx_terms;
        } else {
          ma = &maps.dz_mn[buf];
          nhi = sc.kb_n;
          mb = all ? &maps.x_mn : &maps.xc_mn;
          a_mn = true;
        }
        // dz of its vocabulary tiles: of one (dW), or of its K range
        const int t0 = v0 / kTile + (un.kind == DW ? un.tm : un.kb0 / 4);
        const int t1 = v0 / kTile + (un.kind == DW ? un.tm : (un.kb0 + nhi - 1) / 4);
        if (t0 < dz_from || t1 >= dz_to) {
          ok = wait_tiles(dz_done, t0, t1, v0 / kTile + sc.tv(un.p), sc, lane, dz_to, abort_flag);
          dz_from = t0;
          if (!ok) break;
        }
        if (un.kind == DX && un.p - 1 > dx_ok) {
          if (!warp_count(dx_done + un.p - 1, 2u * kEpiWarps * sc.dx(un.p - 1), abort_flag)) break;
          dx_ok = un.p - 1;
        }
      }
      for (int kb = 0; kb < un.nkb; ++kb) {
        if (!warp_wait(bar(bEmpty + s), phase, abort_flag)) {
          ok = false;
          break;
        }
        if (el) {
          if (kBwd && rank == 0 && kb == un.nkb - 1 - kAhead) mbar_arrive(bar(bWant));
          // CTA 0's barrier counts the bytes of both CTAs' boxes
          if (rank == 0) mbar_arrive_expect_tx(bar(bFull + s), bytes);
          const uint32_t full = map_rank(bar(bFull + s), 0);
          const uint32_t dst = sb0 + kSmRing + s * kStageBytes;
          if (!kBwd || kb < nhi) {
            const int k0 = ((a_mn ? 0 : un.kb0) + kb) * kKB;
            load_operand(ma, a_mn, true, arow, k0, dst, full);
            load_operand(mb, b_mn, b_one, brow, bk + k0, dst + kOperandBytes, full);
          } else {
            // block k of the rows (dW) or of the piece's columns (dx) again,
            // against lo: by vocabulary tile, then by 64 rows, [64][256]
            const int k = un.kb0 + kb - nhi;
            if (a_mn) load_operand(&maps.lo_mn[buf], true, true, rank * 128,
                                   (un.tm * sc.lo_step + k) * 64, dst, full);
            else load_operand(&maps.lo_k[buf], false, true, (k >> 2) * sc.lo_step * 64 + arow,
                              (k & 3) * kKB, dst, full);
            load_operand(mb, b_mn, b_one, brow, bk + k * kKB, dst + kOperandBytes, full);
          }
        }
        __syncwarp();
        if (++s == kStages) {
          s = 0;
          phase ^= 1;
        }
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA (CTA 0 issues for the pair) ----------------
    if (rank == 0) {
      const uint32_t el = elect_one() ? 1u : 0u;
      const uint64_t k_desc = smem_desc_sw128(sb0 + kSmRing, 16, 1024);
      const uint64_t mn_desc = smem_desc_sw128(sb0 + kSmRing, 8192, 1024);
      int s = 0;
      uint32_t phase = 0;
      bool ok = true;
      Unit un;
      ok = next_unit(0, un);
      for (int n = 0; ok; ++n) {
        const bool a_mn = kBwd && un.kind == DW, b_mn = kBwd && un.kind >= DX;
        const uint32_t idesc = b_mn ? idesc_f16(kTile, kTile, true, true, a_mn, b_mn)
                                    : idesc_f16(kTile, kLw, true, true, false, false);
        // descriptors count in 16 bytes: 16 K values are 32 bytes along a row
        // of K, or 16 rows of 128 bytes
        const uint64_t a0 = a_mn ? mn_desc : k_desc;
        const uint64_t b0 = (b_mn ? mn_desc : k_desc) + (kOperandBytes >> 4);
        const uint32_t a_step = a_mn ? 128 : 2, b_step = b_mn ? 128 : 2;
        const int a = n & 1;
        if (n >= 2 && !warp_wait_cl(bar(bAccEmpty + a), ((n >> 1) - 1) & 1, abort_flag)) break;
        tc_fence_after();
        const uint32_t acc = tmem + a * kTile;
        uint32_t on = 0;
        for (int kb = 0; kb < un.nkb; ++kb) {
          if (!warp_wait_cl(bar(bFull + s), phase, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t da = a0 + (uint32_t)(s * (kStageBytes >> 4));
          const uint64_t db = b0 + (uint32_t)(s * (kStageBytes >> 4));
#pragma unroll
          for (int kk = 0; kk < kKB / 16; ++kk) {
            mma_pair_if(el, acc, da + kk * a_step, db + kk * b_step, idesc, on);
            on = 1;
          }
          if (el) commit_pair(bar(bEmpty + s));
          __syncwarp();
          if (++s == kStages) {
            s = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        if (el) commit_pair(bar(bAccFull + a));
        __syncwarp();
        ok = next_unit(n + 1, un);
      }
    } else if (kBwd) {
      // CTA 1's tickets are written by CTA 0, so their reads have to be released
      // at cluster scope. That waits for all that a warp has in flight (2 to 5 %
      // of the backward when the readers do it, 2800 cycles per unit in a warp
      // that issues products): this idle warp does it for them.
      for (int n = 0;; ++n) {
        const int t = n % kTickets;
        if (!warp_wait_cl(bar(bTkFull + t), (n / kTickets) & 1, abort_flag)) break;
        const int kind = *reinterpret_cast<const int*>(smem_raw + kSmTickets + t * 32);
        if (__any_sync(0xffffffffu, kind == END)) break;
        if (!warp_wait(bar(bTkRead + t), (n / kTickets) & 1, abort_flag)) break;
        if (lane == 0) mbar_arrive_remote(map_rank(bar(bTkEmpty + t), 0));
        __syncwarp();
      }
    }
  } else if (kBwd && warp == 2 + kEpiWarps) {
    // ---------------- hand-out of units to both CTAs ----------------
    // A warp of its own: taking a number and finding its unit are long chains
    // that would hold up the loads.
    int wants = 0;
    for (int n = 0; rank == 0; ++n) {
      const int t = n % kTickets;
      if (!warp_wait_cl(bar(bTkEmpty + t), ((n / kTickets) & 1) ^ 1, abort_flag)) break;
      unsigned u = 0;
      if (lane == 0) u = atomicAdd(p.ctl, 1u);
      const Unit un = find_unit<kBwd>(sc, (int)__shfl_sync(0xffffffffu, u, 0));
      if (lane < 2) {
        const uint32_t dst = map_rank(sb0 + kSmTickets + t * 32, lane);
        st_cluster_v4(dst, un.kind, un.p, un.tm, un.tn);
        st_cluster_v4(dst + 16, un.split, un.kb0, un.nkb, 0);
        mbar_arrive_remote(map_rank(bar(bTkFull + t), lane));
      }
      __syncwarp();
      if (un.kind == END) break;
      if (un.nkb > kAhead && !warp_wait(bar(bWant), wants++ & 1, abort_flag)) break;
    }
  } else if (warp == 2 + kEpiWarps) {
    // ---------------- the named logits ----------------
    // With few named ids per row their logits are also taken as dot products in
    // plain fp32, four at a time, eight lanes each, beside the products: the
    // loss is a difference of logits, and the tensor core's sums, cut instead
    // of rounded, would leave 1e-6 to 3e-6 of it.
    if (p.exact) {
      const int c8 = p.C / 8, sub = lane & 7;
      const long items = (long)kept * p.K, step = (long)gridDim.x * 4;
      auto find = [&](long i, int& row, int& id) {
        row = 0;
        id = -1;
        if (i >= items) return;
        const int m = (int)(i / p.K);
        row = p.n_kept ? p.row_of[m] : m;
        id = p.ids[(size_t)row * p.K + (int)(i - (long)m * p.K)];
      };
      long i = (long)blockIdx.x * 4 + (lane >> 3);
      int row, id, next_row, next_id;
      find(i, row, id);
      for (; __any_sync(0xffffffffu, i < items); i += step, row = next_row, id = next_id) {
        find(i + step, next_row, next_id);  // on its way during this one
        float s0 = 0.f, s1 = 0.f;
        if ((unsigned)id < (unsigned)p.V) {
          const uint4* xr = p.x + (size_t)row * c8;
          const uint4* wr = p.w + (size_t)id * c8;
#pragma unroll 8
          for (int q = sub; q < c8; q += 8) {
            const uint4 a = xr[q], b = wr[q];
            const uint32_t av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              s0 = fmaf(__uint_as_float(av[e] << 16), __uint_as_float(bv[e] << 16), s0);
              s1 = fmaf(__uint_as_float(av[e] & 0xffff0000u), __uint_as_float(bv[e] & 0xffff0000u),
                        s1);
            }
          }
        }
        s0 += s1;
        for (int o = 1; o < 8; o <<= 1) s0 += __shfl_xor_sync(0xffffffffu, s0, o);
        if (sub == 0 && i < items) p.exact[i] = s0 * p.inv_tau;
      }
    }
  } else {
    // ---------------- epilogue: thread = TMEM lane = output row ----------------
    // warp w reads lanes 32 (w % 4).. of one half of the columns: two warps per
    // lane quarter
    const int sub = warp & 3, half = (warp - 2) >> 2;
    const uint32_t tl = tmem + ((uint32_t)(sub * 32) << 16);
    constexpr int lhalf = kLw / 2, lchunks = kLw / 64;  // of a logits tile
    uint32_t stage = sb0 + kSmStage + (warp - 2) * 8192;  // of the two buffers, the next one
    const int sw = lane & 7;
    const float c2 = p.inv_tau * kLog2e;
    // the counter that this warp's stores of its last unit will raise (lane 0)
    unsigned* owed = nullptr;
    // staging is free again, and the stores are complete: raise what they owe
    auto settle = [&]() {
      if (lane == 0) {
        bulk_wait_group0();
        if (owed) {
          fence_proxy_async();
#ifdef ATTN_DEBUG_HOOKS
          if (!(g_attn_withhold == 2 && owed == dz_done) && !(g_attn_withhold == 3 && owed == dx_done))
#endif
          red_release(owed, 1u);
          owed = nullptr;
        }
      }
      __syncwarp();
    };
    auto reuse_stage = [&]() {  // the next buffer is free again
      if (lane == 0) bulk_wait_group_read1();
      __syncwarp();
    };
    Unit un;
    // what the unit's row needs, fetched while the unit before is worked on
    RowPar rp = {0.f, 0.f, 0.f, 0};
    int n_from = 0, n_to = 0;
    int key = -1, key2 = -1;  // foremost ids of this row and of one in the other half of its 64
    auto fetch_row = [&](const Unit& w) {
      const int m = w.tm * kTile + rank * 128 + sub * 32 + lane;
      if (kBwd && p.key && w.kind == DZ) {
        key = m < kept ? p.key[m] : -1;
        key2 = (m ^ 32) < kept ? p.key[m ^ 32] : -1;
      }
      if (!kBwd && !p.n_kept) rp.id = m < kept && !p.share ? p.ids[m] : m;
      else if (w.kind <= DZ && m < kept) rp = p.par[m];
    };
    auto fetch_named = [&](const Unit& w) {
      n_from = n_to = 0;
      const int m = w.tm * kTile + rank * 128 + sub * 32 + lane;
      if (p.share && w.kind <= DZ && m < kept) {
        const uint16_t* f = p.first + (size_t)rp.id * p.first_pitch +
                            (w.p * p.piece + w.tn * kLw) / lhalf + half;
        n_from = f[0];
        n_to = f[1];
      }
    };
    bool more = next_unit(0, un);
    if (more) {
      fetch_row(un);
      fetch_named(un);
    }
    for (int n = 0; more; ++n) {
      const int a = n & 1;
      const int row0 = un.tm * kTile + rank * 128 + sub * 32;  // of this warp
      const int m = row0 + lane;
      const bool logits = !kBwd || un.kind == DZ;
      // this warp's columns: within the piece, or of C
      const int col0 = logits ? un.tn * kLw + half * lhalf : un.tn * kTile + half * 128;
      const int v0 = un.p * p.piece, vn = min(p.piece, p.V - v0), vend = v0 + vn;
      Named<kBwd> nm;
      nm.none();
      if (p.share && n_from < n_to)
        nm.list(p.ids + (size_t)rp.id * p.K, p.share + (size_t)rp.id * p.K, n_from, n_to);
      const float lse2 = rp.lse2, ca = rp.ca, cb = rp.cb;
      // lo of this unit: all of it, or where a row of the 64 names the unit's tile
      const int vtile = (v0 + un.tn * kLw) / kTile, row_key = key;
      const bool unit_lo =
          kBwd && (sc.dw_terms == 2 ||
                   (sc.tile_start && __any_sync(0xffffffffu, key >= 0 && key / kTile == vtile ||
                                                                 key2 >= 0 && key2 / kTile == vtile)));
      // without a list: within these columns or not
      const int target = m < kept ? rp.id - (v0 + col0) : -1;
      const uint32_t full = bar(bAccFull + a), par = (n >> 1) & 1;
      // others may wait for what this warp owes: it never blocks owing
      if (!__all_sync(0xffffffffu, mbar_test(full, par))) settle();
      if (!warp_wait(full, par, abort_flag)) break;
      tc_fence_after();
      // the next unit, so that its rows' values arrive during this one
      Unit nu;
      more = next_unit(n + 1, nu);
      if (more) fetch_row(nu);
      __syncwarp();  // tcgen05.ld and its wait take a converged warp, here and below
      auto release = [&]() {
        // every column of this accumulator that this warp uses has been read
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_tmem(map_rank(bar(bAccEmpty + a), 0));
        __syncwarp();
      };
      const uint32_t src = tl + a * kTile + half * (logits ? lhalf : 128);
      if constexpr (!kBwd) {
        float mx = -INFINITY, sum = 0.f;
        uint32_t v[2][32];
        tmem_ld32(src, v[0]);
#pragma unroll
        for (int c = 0; c < lchunks; ++c) {
          tmem_wait_ld();
          if (c + 1 < lchunks) tmem_ld32(src + 32 * (c + 1), v[(c + 1) & 1]);
          else release();
          const uint32_t* t = v[c & 1];
          const int cc = v0 + col0 + 32 * c;
          // a teacher's ids among these 32 columns: each lane looks its row's up
          // in its own 128 bytes of the staging (swizzled in 16-byte groups)
          if (__any_sync(0xffffffffu, nm.id[0] < cc + 32)) {
            const uint32_t mine = stage + lane * 128;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              st_shared_v4(mine + ((e ^ sw) << 4), t[4 * e], t[4 * e + 1], t[4 * e + 2], t[4 * e + 3]);
            while (nm.id[0] < cc + 32) {
              const int e = nm.id[0] - cc;
              p.named[(size_t)m * p.K + nm.pos] =
                  ld_shared_f32(mine + (((e >> 2) ^ sw) << 4) + (e & 3) * 4) * p.inv_tau;
              nm.advance();
            }
            __syncwarp();
          }
          if (!p.share && __any_sync(0xffffffffu, (unsigned)(target - 32 * c) < 32u)) {
            float z = 0.f;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (target == 32 * c + e) z = __uint_as_float(t[e]);
            if ((unsigned)(target - 32 * c) < 32u) p.named[m] = z * p.inv_tau;
          }
          float f[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(t[e]);
          if (cc + 32 > vend) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (cc + e >= vend) f[e] = -INFINITY;
          }
          float cm = max3f(f[0], f[1], f[2]);
#pragma unroll
          for (int e = 3; e < 31; e += 2) cm = max3f(cm, f[e], f[e + 1]);
          cm = fmaxf(cm, f[31]) * c2;
          const float nx = fmaxf(mx, cm);
          if (nx > -INFINITY) {
            float2 s0 = make_float2(0.f, 0.f), s1 = s0;
            const float2 k2 = make_float2(c2, c2), n2 = make_float2(-nx, -nx);
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float2 x0 = __ffma2_rn(make_float2(f[e], f[e + 1]), k2, n2);
              const float2 x1 = __ffma2_rn(make_float2(f[e + 2], f[e + 3]), k2, n2);
              s0 = __fadd2_rn(s0, make_float2(ex2(x0.x), ex2(x0.y)));
              s1 = __fadd2_rn(s1, make_float2(ex2(x1.x), ex2(x1.y)));
            }
            sum = sum * ex2(mx - nx) + ((s0.x + s0.y) + (s1.x + s1.y));
            mx = nx;
          } else {
            // only -inf or NaN so far: NaN has to stay
#pragma unroll
            for (int e = 0; e < 32; ++e) sum += f[e] == -INFINITY ? 0.f : f[e];
          }
          __syncwarp();
        }
        if (m < kept) p.part[(size_t)(2 * un.tn + half) * p.row_pitch + m] = make_float2(mx, sum);
      } else if (un.kind == DZ) {
        const int buf = un.p % kDzBuffers;
        // lo goes out beside hi, through the other staging buffer
        const bool lo = unit_lo;
        uint32_t even[16];  // lo of the even 32 columns, until the odd ones join
        uint32_t v[2][32];
        tmem_ld32(src, v[0]);
        const float2 k2 = make_float2(c2, c2), l2 = make_float2(-lse2, -lse2),
                     a2 = make_float2(ca, ca);
#pragma unroll
        for (int c = 0; c < lchunks; ++c) {
          tmem_wait_ld();
          if (c + 1 < lchunks) tmem_ld32(src + 32 * (c + 1), v[(c + 1) & 1]);
          else release();
          const uint32_t* tv = v[c & 1];
          const int cc = v0 + col0 + 32 * c;
          float t[32];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 x =
                __ffma2_rn(make_float2(__uint_as_float(tv[e]), __uint_as_float(tv[e + 1])), k2, l2);
            const float2 y = __fmul2_rn(make_float2(ex2(x.x), ex2(x.y)), a2);
            t[e] = y.x;
            t[e + 1] = y.y;
          }
          if (p.share) {
            // a teacher's shares, in a staging buffer that no store reads
            if (__any_sync(0xffffffffu, nm.id[0] < cc + 32)) {
              if (lane == 0) bulk_wait_group_read0();
              __syncwarp();
              const uint32_t mine = (stage ^ 4096) + lane * 128;
#pragma unroll
              for (int e = 0; e < 8; ++e)
                st_shared_v4(mine + ((e ^ sw) << 4), __float_as_uint(t[4 * e]),
                             __float_as_uint(t[4 * e + 1]), __float_as_uint(t[4 * e + 2]),
                             __float_as_uint(t[4 * e + 3]));
              while (nm.id[0] < cc + 32) {
                const int e = nm.id[0] - cc;
                const uint32_t at = mine + (((e >> 2) ^ sw) << 4) + (e & 3) * 4;
                const float d = fmaf(-cb, nm.share[0], ld_shared_f32(at));
                st_shared_f32(at, d);
                if (p.rest) {  // of an id named again, the last one's counts
                  const float r = d - __bfloat162float(__float2bfloat16_rn(d));
                  if (p.rest_k == p.K) p.rest[(size_t)m * p.K + nm.pos] = nm.id[1] == nm.id[0] ? 0.f : r;
                  else if (nm.id[0] == row_key) p.rest[m] = r;
                }
                nm.advance();
              }
#pragma unroll
              for (int e = 0; e < 32; ++e)
                t[e] = ld_shared_f32(mine + (((e >> 2) ^ sw) << 4) + (e & 3) * 4);
              __syncwarp();
            }
          } else if (__any_sync(0xffffffffu, (unsigned)(target - 32 * c) < 32u)) {
            float d = 0.f;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (target == 32 * c + e) d = t[e] -= cb;
            if ((unsigned)(target - 32 * c) < 32u)
              p.rest[m] = d - __bfloat162float(__float2bfloat16_rn(d));
          }
          // rows that are not kept and columns past the vocabulary are zeros:
          // they are K values of the products that read this buffer
          const int left = m < kept ? vend - cc : 0;
          if (left < 32) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (e >= left) t[e] = 0.f;
          }
          if (c == 0 && __shfl_sync(0xffffffffu, owed != nullptr, 0)) settle();
          if ((c & 1) == 0) reuse_stage();
          const uint32_t my_row = stage + lane * 128;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            st_shared_v4(my_row + ((((c & 1) * 4 + e) ^ sw) << 4), pack_bf16(t[8 * e], t[8 * e + 1]),
                         pack_bf16(t[8 * e + 2], t[8 * e + 3]), pack_bf16(t[8 * e + 4], t[8 * e + 5]),
                         pack_bf16(t[8 * e + 6], t[8 * e + 7]));
          if (lo) {
            auto left2 = [&](int e) {  // of columns 2 e and 2 e + 1
              return pack_bf16(t[2 * e] - __bfloat162float(__float2bfloat16_rn(t[2 * e])),
                               t[2 * e + 1] - __bfloat162float(__float2bfloat16_rn(t[2 * e + 1])));
            };
            if ((c & 1) == 0) {
#pragma unroll
              for (int e = 0; e < 16; ++e) even[e] = left2(e);
            } else {
              if (lane == 0) bulk_wait_group_read0();
              __syncwarp();
              const uint32_t lo_row = (stage ^ 4096) + lane * 128;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                st_shared_v4(lo_row + ((e ^ sw) << 4), even[4 * e], even[4 * e + 1],
                             even[4 * e + 2], even[4 * e + 3]);
                st_shared_v4(lo_row + (((4 + e) ^ sw) << 4), left2(4 * e), left2(4 * e + 1),
                             left2(4 * e + 2), left2(4 * e + 3));
              }
            }
          }
          if (c & 1) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              const int at = col0 + 32 * (c - 1);
              tma_store_2d(&maps.dz_out[buf], stage, at, row0);
              bulk_commit_group();
              if (lo) {
                tma_store_2d(&maps.lo_out[buf], stage ^ 4096, at & (kTile - 1),
                             (at / kTile) * sc.lo_step * 64 + row0);
                bulk_commit_group();
              }
            }
            // the next buffer is the one whose store came first
            if (!lo) stage ^= 4096;
          }
          __syncwarp();
        }
        if (lane == 0) owed = dz_done + (v0 + un.tn * kLw) / kTile;
      } else {
        // dz of this unit has been read (by the products that this warp waited
        // for): its buffer may be overwritten, if a later piece does
        if (warp == 2 && lane == 0 && un.p + kDzBuffers < p.pieces) red_relaxed(dz_used + un.p, 1u);
        const bool is_dx = un.kind == DX;
        const bool last = un.p + 1 == p.pieces;  // of the vocabulary
        int splits = 1, kb_per;
        if (is_dx)
          split_dx(((kept + kTile - 1) / kTile) * ((p.C + kTile - 1) / kTile),
                   (min(p.piece, p.V) + kKB - 1) / kKB, splits, kb_per);
        const bool f32 = is_dx || p.dw_f32;
        const CUtensorMap* mo = is_dx ? &maps.dx_out : &maps.dw_out;
        const int slot = slot_rows(kept);
        const int out_row = is_dx ? un.split * slot + row0 : v0 + row0;
        const int out_rows = is_dx ? kept : vn;  // rows of the job that exist
        if (__shfl_sync(0xffffffffu, owed != nullptr, 0)) settle();
        if (is_dx && last && splits == 1) {
          // the sum ends here: the earlier pieces', this one's, and what the
          // rounding of dz took go straight to dx, by way of the staging, so
          // that eight lanes read and write a row (a row per lane took 20 us
          // at the end of the call, this 10)
          const int row = m < kept ? p.row_of[m] : 0;
          float rest[kFewNamed];
          int id[kFewNamed];
          const int n_rest = p.rest && sc.dx_terms == 1 ? p.rest_k : 0;
#pragma unroll
          for (int k = 0; k < kFewNamed; ++k) {
            rest[k] = 0.f;
            id[k] = 0;
            if (n_rest > k && m < kept) {
              const int named = p.rest_k == p.K ? p.ids[(size_t)row * p.K + k] : p.key[m];
              if ((unsigned)named < (unsigned)p.V) {
                id[k] = named;
                rest[k] = __ldcg(p.rest + (size_t)m * p.rest_k + k);
              }
            }
          }
          const int quad = lane & 7;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            const int cq = col0 + 32 * c + 4 * quad;
            float4 sum[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int r = 4 * i + (lane >> 3);
              sum[i] = make_float4(0.f, 0.f, 0.f, 0.f);
              if (un.p > 0 && row0 + r < kept && cq < p.C)
                sum[i] = __ldcg(reinterpret_cast<const float4*>(p.acc + (size_t)(row0 + r) * p.C + cq));
            }
#pragma unroll
            for (int k = 0; k < kFewNamed; ++k) {
              if (k >= n_rest) break;
              uint2 wv[8];  // rows of W (row 0 where there is nothing to add): all on their way
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const int col = __shfl_sync(0xffffffffu, id[k], 4 * i + (lane >> 3));
                wv[i] = *reinterpret_cast<const uint2*>(
                    reinterpret_cast<const __nv_bfloat16*>(p.w) + (size_t)col * p.C + min(cq, p.C - 4));
              }
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float g = __shfl_sync(0xffffffffu, rest[k], 4 * i + (lane >> 3));
                if (g != 0.f) add_scaled4(sum[i], g, wv[i]);
              }
            }
            __syncwarp();
            uint32_t v[32];
            tmem_ld32(src + 32 * c, v);
            tmem_wait_ld();
            if (c == 3) release();
            reuse_stage();
#pragma unroll
            for (int e = 0; e < 8; ++e)
              st_shared_v4(stage + lane * 128 + ((e ^ sw) << 4), v[4 * e], v[4 * e + 1],
                           v[4 * e + 2], v[4 * e + 3]);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int r = 4 * i + (lane >> 3);
              const int to = __shfl_sync(0xffffffffu, row, r);
              const float4 f = ld_shared_v4(stage + r * 128 + ((quad ^ (r & 7)) << 4));
              if (row0 + r < kept && cq < p.C)
                *reinterpret_cast<uint2*>(p.dx + (size_t)to * p.C + cq) =
                    make_uint2(pack_bf16(sum[i].x + f.x, sum[i].y + f.y),
                               pack_bf16(sum[i].z + f.z, sum[i].w + f.w));
            }
            __syncwarp();
          }
          if (more) fetch_named(nu);
          un = nu;
          continue;
        }
        uint32_t vv[2][32];
        tmem_ld32(src, vv[0]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int cs = col0 + 32 * c;
          __syncwarp();
          tmem_wait_ld();
          if (c < 3) tmem_ld32(src + 32 * (c + 1), vv[(c + 1) & 1]);
          else release();
          uint32_t* v = vv[c & 1];
          if (un.nkb == 0) {  // no rows kept: nothing was multiplied
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = 0u;
          }
          if (cs >= p.C || row0 >= out_rows) continue;  // uniform in the warp
          if (f32 || (c & 1) == 0) reuse_stage();
          const uint32_t my_row = stage + lane * 128;
          if (f32) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              st_shared_v4(my_row + ((e ^ sw) << 4), v[4 * e], v[4 * e + 1], v[4 * e + 2],
                           v[4 * e + 3]);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float f[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(v[8 * e + i]);
              st_shared_v4(my_row + ((((c & 1) * 4 + e) ^ sw) << 4), pack_bf16(f[0], f[1]),
                           pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
            }
          }
          if (f32 || (c & 1) || cs + 32 >= p.C) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              const int at = f32 ? cs : col0 + 32 * (c & ~1);
              if (is_dx && un.p > 0) tma_reduce_add_2d(mo, stage, at, out_row);
              else tma_store_2d(mo, stage, at, out_row);
              bulk_commit_group();
            }
            stage ^= 4096;
          }
        }
        if (is_dx && !last && lane == 0) owed = dx_done + un.p;
      }
      if (more) fetch_named(nu);
      un = nu;
    }
    settle();  // stores complete before the CTA ends
  }

  // Where a wait has run out, loads and products of either CTA may be on their way
  // into this one's memory still. They take microseconds: 400,000 cycles (0.2 ms)
  // pass before it is given back.
  __syncwarp();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) {
    const long long t0 = clock64();
    while (clock64() - t0 < 400000) __nanosleep(1000);
  }
  tc_fence_before();
  __syncwarp();
  __syncthreads();
  cluster_sync_all();  // no CTA leaves (or frees TMEM) while the other may still signal it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

}  // namespace head100
