// head_sm100.cuh -- losses of the output head on logits that are never
// stored: z = x W^T / tau for N token rows x [N][C] and V vocabulary rows
// W [V][C] (bf16, fp32 accumulate).
//
// Forward. Row n needs lse_n = log sum_v exp z[n][v] and z at the few ids its
// loss names (the target, or a teacher's list). The logits are formed one
// 256 x 256 tile at a time in tensor memory; the epilogue keeps, per row and
// 128 columns, the running maximum and sum of exponentials (fp32, base 2) and
// the named logits, 8 bytes per 128 logits instead of the logits.
//
// Backward. With p = exp(z - lse) the gradient of the logits is
//     dz[n][v] = (dloss_n + dlse_n) / tau * p[n][v] - dloss_n / tau * q[n][v],
// q the row's target distribution (non-zero at the named ids only), and
//     dx = dz W,   dW = dz^T x.
// The vocabulary is taken in pieces: the logits of a piece are formed again,
// dz of the piece is rounded to bf16 (the tensor cores' operand type, half a
// step of 2^-9 relative) into a buffer that the two products of the piece
// read. dx is summed over the pieces in fp32, dW of a piece is final.
//
// Rows whose target is absent (or whose upstream gradients are both zero) are
// left out: the kept rows are compacted first, so the products cost what the
// kept rows cost, and what a left-out row holds (NaN included) reaches
// nothing. Their number lives on the device; every kernel reads it there.
//
// One kernel runs all products, head_gemm_kernel: clusters of two CTAs, each
// pair walking a strided list of 256 x 256 output tiles (units) of up to
// three products that do not depend on one another; one launch of the
// backward runs dx and dW of a piece and the logits of the next one.
#pragma once

#include <limits.h>

#include "common.cuh"
#include "sm100.cuh"

namespace head100 {

using namespace sm100;

constexpr int kTile = 256;            // output tile of a CTA pair (rows and columns)
constexpr int kKB = 64;               // K values per ring stage
constexpr int kStages = 6;
constexpr int kOperandBytes = 128 * kKB * 2;  // 128 rows (or columns) of a stage
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kPairs = 74;            // CTA pairs of a full persistent grid (148 SMs)

constexpr int kEpiWarps = 8;
constexpr int kThreads = 96 + 32 * kEpiWarps;  // TMA, MMA, epilogue warps, target warp
constexpr int kSmRing = 0;
constexpr int kSmStage = kStages * kStageBytes;          // 4 KB per epilogue warp
constexpr int kSmBars = kSmStage + kEpiWarps * 4096;
constexpr int bFull = 0, bEmpty = kStages, bAccFull = 2 * kStages, bAccEmpty = 2 * kStages + 2;
constexpr int kNumBars = 2 * kStages + 4;
constexpr int kSmMisc = kSmBars + kNumBars * 8;
constexpr int kSmJobs = kSmMisc + 16;
constexpr int kSmAlloc = kSmJobs + 256;
static_assert(kSmAlloc <= 232448, "shared memory of one CTA");

enum Kind : int { JOB_LSE = 0, JOB_DZ = 1, JOB_DX = 2, JOB_DW = 3 };

// One product. Vocabulary rows [v0, v0 + vn), dz in buffer `buf`.
struct Job {
  int kind, v0, vn, buf;
  int add;  // JOB_DX: add to the accumulator (else store)
};

constexpr int kMaxJobs = 3;

struct Maps {
  // operand loads: _k with K contiguous (boxes of 64 K x 128 rows), _mn with
  // the row index contiguous (boxes of 64 rows x 64 K, two of them in one box
  // when the extent is a multiple of 64)
  CUtensorMap x_k, xc_k, w_k, x_mn, xc_mn, w_mn, dz_k[2], dz_mn[2];
  // output boxes of 32 rows x 128 bytes
  CUtensorMap dz_out[2], dx_out, dw_out;
};

struct Params {
  const uint4 *x, *w;
  int N, V, C;
  int K;                 // named ids per row (1: the target)
  int n_jobs;
  Job job[kMaxJobs];
  int kb_first;          // K blocks of dx over a whole piece
  int c_blocks;          // C % 64 == 0: _mn maps of x and W take both 64-wide blocks in one box
  int dw_f32;
  float inv_tau;
  const int* n_kept;     // rows kept (device)
  const int* row_of;     // kept row -> row
  const int* ids;        // [N][K] ascending; a negative or >= V id matches nothing
  const float* share;    // [N][K] q, or null (1 at the target)
  const float* lse;      // [N] (JOB_DZ)
  const float* dloss;    // [N]
  const float* dlse;     // [N] or null
  float2* part;          // JOB_LSE: [2 tiles_n][row_pitch] maximum (base 2), sum
  float* named;          // JOB_LSE: [kept row][K] z at the row's ids
  int row_pitch;
};

// Tiles and K blocks of a job for `kept` rows.
struct Dims {
  int tiles_m, tiles_n, splits, kb_total, kb_per, units;
};

// dx has few tiles when few rows are kept: its K axis (the vocabulary) is
// then split over units, each with an accumulator of its own that the closing
// pass adds in order (no atomics, so results repeat). Two units per CTA pair,
// at least eight K blocks each.
__host__ __device__ inline void split_dx(int tiles, int kb_total, int& splits, int& kb_per) {
  splits = 1;
  if (tiles > 0 && tiles < kPairs) {
    splits = (2 * kPairs + tiles - 1) / tiles;
    const int most = kb_total / 8 > 1 ? kb_total / 8 : 1;
    splits = splits < most ? splits : most;
  }
  kb_per = (kb_total + splits - 1) / splits;
  if (kb_per < 1) kb_per = 1;
  splits = (kb_total + kb_per - 1) / kb_per;
  if (splits < 1) splits = 1;
}

// kb_first: K blocks of a whole piece. A shorter last piece keeps the parts'
// length, so it adds into accumulators that the first piece has written.
__host__ __device__ inline Dims job_dims(const Job& j, int kept, int C, int kb_first) {
  Dims d;
  const int rows = (kept + kTile - 1) / kTile, cols = (C + kTile - 1) / kTile,
            voc = (j.vn + kTile - 1) / kTile;
  d.splits = 1;
  if (j.kind == JOB_LSE || j.kind == JOB_DZ) {
    d.tiles_m = rows;
    d.tiles_n = voc;
    d.kb_total = (C + kKB - 1) / kKB;
  } else if (j.kind == JOB_DX) {
    d.tiles_m = rows;
    d.tiles_n = cols;
    d.kb_total = (j.vn + kKB - 1) / kKB;
  } else {
    d.tiles_m = voc;
    d.tiles_n = cols;
    d.kb_total = (kept + kKB - 1) / kKB;
  }
  d.kb_per = d.kb_total;
  if (j.kind == JOB_DX) {
    split_dx(d.tiles_m * d.tiles_n, kb_first, d.splits, d.kb_per);
    d.splits = (d.kb_total + d.kb_per - 1) / d.kb_per;
  }
  d.units = d.tiles_m * d.tiles_n * d.splits;
  return d;
}

// Rows of one dx accumulator (a multiple of the tile).
__host__ __device__ inline int slot_rows(int kept) { return (kept + kTile - 1) / kTile * kTile; }

struct Unit {
  int job, tm, tn, split, kb0, nkb;
};

// Unit u of the launch. Within a job units go through bands of kBand row
// tiles, columns within a band, rows fastest: the 74 pairs then work on about
// 8 x 9 tiles at a time, whose operands (17 x 256 rows of K) come from L2.
constexpr int kBand = 8;
__device__ __forceinline__ bool find_unit(int u, int n_jobs, const Dims* dims, Unit& o) {
  for (int j = 0; j < n_jobs; ++j) {
    const Dims& d = dims[j];
    if (u >= d.units) {
      u -= d.units;
      continue;
    }
    const int tiles = d.tiles_m * d.tiles_n;
    o.job = j;
    o.split = u / tiles;
    int r = u - o.split * tiles;
    const int band = r / (kBand * d.tiles_n);
    r -= band * kBand * d.tiles_n;
    const int h = min(kBand, d.tiles_m - band * kBand);
    o.tn = r / h;
    o.tm = band * kBand + r - o.tn * h;
    o.kb0 = o.split * d.kb_per;
    o.nkb = min(d.kb_total, o.kb0 + d.kb_per) - o.kb0;
    return true;
  }
  return false;
}

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

// The row's named ids from column col on: position of the first one and its
// column (INT_MAX when there is none).
struct Named {
  const int* ids;
  int K, pos, next;
  __device__ __forceinline__ void start(const int* row_ids, int k, int col) {
    ids = row_ids;
    K = k;
    int lo = 0, hi = k;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (ids[mid] < col) lo = mid + 1;
      else hi = mid;
    }
    pos = lo;
    next = lo < k ? ids[lo] : INT_MAX;
  }
  __device__ __forceinline__ void none() {
    K = pos = 0;
    next = INT_MAX;
  }
  __device__ __forceinline__ void advance() {
    ++pos;
    next = pos < K ? ids[pos] : INT_MAX;
  }
};

__global__ void __launch_bounds__(kThreads, 1)
    head_gemm_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t sb0 = smem_u32(smem_raw);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem_raw + kSmMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem_raw + kSmMisc + 4);
  Dims* dims = reinterpret_cast<Dims*>(smem_raw + kSmJobs);
  auto bar = [&](int i) -> uint32_t { return sb0 + kSmBars + 8u * i; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  pdl_wait_and_trigger();
  if (sb0 & 1023u) {  // uniform across the cluster: nothing has been issued yet
    if (threadIdx.x == 0) report_status(ATTN_ECUDA_LAYOUT);
    return;
  }
  const int kept = *p.n_kept;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar(bFull + s), 1);
      mbar_init(bar(bEmpty + s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(bar(bAccFull + a), 1);
      mbar_init(bar(bAccEmpty + a), 2 * kEpiWarps);  // the epilogue warps of both CTAs
    }
    *abort_flag = 0;
    for (int j = 0; j < p.n_jobs; ++j) dims[j] = job_dims(p.job[j], kept, p.C, p.kb_first);
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
  const int u0 = (int)blockIdx.x >> 1, ustep = (int)gridDim.x >> 1;

  // The TMA and MMA warps run their loops converged, one elected lane issuing:
  // the operands of the issue then live in uniform registers. Issued from a
  // branch of one thread, a tcgen05.mma cost 130 cycles whatever its size;
  // so, 64 cycles at N = 128 and 128 at N = 256, the tensor core's own time.
  if (warp == 0) {
    // ---------------- TMA ----------------
    const bool el = elect_one();
    const bool all = kept == p.N;  // every row kept: x is read in place
    int s = 0;
    uint32_t phase = 1;  // a fresh barrier's previous phase counts as complete
    bool ok = true;
    Unit un;
    for (int u = u0; ok && find_unit(u, p.n_jobs, dims, un); u += ustep) {
      const Job& j = p.job[un.job];
      const CUtensorMap *ma, *mb;
      bool a_mn = false, b_mn = true, b_one = p.c_blocks != 0;
      int bk = 0, brow = un.tn * kTile + rank * 128;
      if (j.kind <= JOB_DZ) {
        ma = all ? &maps.x_k : &maps.xc_k;
        mb = &maps.w_k;
        b_mn = false;
        brow += j.v0;
      } else if (j.kind == JOB_DX) {
        ma = &maps.dz_k[j.buf];
        mb = &maps.w_mn;
        bk = j.v0;
      } else {
        ma = &maps.dz_mn[j.buf];
        mb = all ? &maps.x_mn : &maps.xc_mn;
        a_mn = true;
      }
      const int arow = un.tm * kTile + rank * 128;
      for (int kb = 0; kb < un.nkb; ++kb) {
        if (!mbar_wait(bar(bEmpty + s), phase, abort_flag)) {
          ok = false;
          break;
        }
        if (el) {
          // CTA 0's barrier counts the bytes of both CTAs' boxes
          if (rank == 0) mbar_arrive_expect_tx(bar(bFull + s), 2 * kStageBytes);
          const uint32_t full = map_rank(bar(bFull + s), 0);
          const uint32_t dst = sb0 + kSmRing + s * kStageBytes;
          const int k0 = (un.kb0 + kb) * kKB;
          load_operand(ma, a_mn, true, arow, k0, dst, full);
          load_operand(mb, b_mn, b_one, brow, bk + k0, dst + kOperandBytes, full);
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
      int s = 0, n = 0;
      uint32_t phase = 0;
      bool ok = true;
      Unit un;
      for (int u = u0; ok && find_unit(u, p.n_jobs, dims, un); u += ustep, ++n) {
        const int kind = p.job[un.job].kind;
        const bool a_mn = kind == JOB_DW, b_mn = kind >= JOB_DX;
        const uint32_t idesc = idesc_f16(kTile, kTile, true, true, a_mn, b_mn);
        // descriptors count in 16 bytes: 16 K values are 32 bytes along a row
        // of K, or 16 rows of 128 bytes
        const uint64_t a0 = a_mn ? mn_desc : k_desc;
        const uint64_t b0 = (b_mn ? mn_desc : k_desc) + (kOperandBytes >> 4);
        const uint32_t a_step = a_mn ? 128 : 2, b_step = b_mn ? 128 : 2;
        const int a = n & 1;
        if (n >= 2 && !mbar_wait_cl(bar(bAccEmpty + a), ((n >> 1) - 1) & 1, abort_flag)) break;
        tc_fence_after();
        const uint32_t acc = tmem + a * kTile;
        uint32_t on = 0;
        for (int kb = 0; kb < un.nkb; ++kb) {
          if (!mbar_wait_cl(bar(bFull + s), phase, abort_flag)) {
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
        if (ok && el) commit_pair(bar(bAccFull + a));
        __syncwarp();
      }
    }
  } else if (warp == 2 + kEpiWarps) {
    // ---------------- the target's logit ----------------
    // A single named id per row is a dot product of its own, in plain fp32: the
    // loss is the difference lse - z, and the tensor core's sums, cut instead
    // of rounded, would leave about 1e-6 of it. Runs beside the products.
    if (p.n_jobs == 1 && p.job[0].kind == JOB_LSE && !p.share) {
      const int c8 = p.C / 8;
      for (int m = blockIdx.x; m < kept; m += gridDim.x) {
        const int row = p.row_of[m];
        const uint4* xr = p.x + (size_t)row * c8;
        const uint4* wr = p.w + (size_t)p.ids[row] * c8;
        float s0 = 0.f, s1 = 0.f;
#pragma unroll 4
        for (int i = lane; i < c8; i += 32) {
          const uint4 a = xr[i], b = wr[i];
          const uint32_t av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s0 = fmaf(__uint_as_float(av[e] << 16), __uint_as_float(bv[e] << 16), s0);
            s1 = fmaf(__uint_as_float(av[e] & 0xffff0000u), __uint_as_float(bv[e] & 0xffff0000u), s1);
          }
        }
        s0 = warp_sum(s0 + s1);
        if (lane == 0) p.named[m] = s0 * p.inv_tau;
      }
    }
  } else {
    // ---------------- epilogue: thread = TMEM lane = output row ----------------
    // warp w reads lanes 32 (w % 4).. of columns 128 half..: two warps per lane quarter
    const int sub = warp & 3, half = (warp - 2) >> 2;
    const uint32_t tl = tmem + ((uint32_t)(sub * 32) << 16) + half * 128;
    const uint32_t stage = sb0 + kSmStage + (warp - 2) * 4096;
    const uint32_t my_row = stage + lane * 128;
    const int sw = lane & 7;
    const float c2 = p.inv_tau * kLog2e;
    int n = 0;
    Unit un;
    for (int u = u0; find_unit(u, p.n_jobs, dims, un); u += ustep, ++n) {
      const Job& j = p.job[un.job];
      const int a = n & 1;
      const int row0 = un.tm * kTile + rank * 128 + sub * 32;  // of this warp
      const int m = row0 + lane;
      const int col0 = un.tn * kTile + half * 128;  // within the job's columns
      // what the row needs is fetched while the main loop still runs
      Named nm;
      nm.none();
      float lse2 = 0.f, ca = 0.f, cb = 0.f;
      const float* share = nullptr;
      if (j.kind <= JOB_DZ && m < kept) {
        const int row = p.row_of[m];
        // the forward's single target has a warp of its own
        if (j.kind == JOB_DZ || p.share) nm.start(p.ids + (size_t)row * p.K, p.K, j.v0 + col0);
        if (j.kind == JOB_DZ) {
          lse2 = p.lse[row] * kLog2e;
          const float g = p.dloss[row];
          ca = (g + (p.dlse ? p.dlse[row] : 0.f)) * p.inv_tau;
          cb = g * p.inv_tau;
          if (p.share) share = p.share + (size_t)row * p.K;
        }
      }
      if (!mbar_wait(bar(bAccFull + a), (n >> 1) & 1, abort_flag)) break;
      tc_fence_after();
      auto release = [&]() {
        // every column of this accumulator that this warp uses has been read
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(map_rank(bar(bAccEmpty + a), 0));
      };
      const int vend = j.v0 + j.vn;  // columns of the logits stop here
      if (j.kind == JOB_LSE) {
        float mx = -INFINITY, sum = 0.f;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t v[32];
          tmem_ld32(tl + a * kTile + 32 * c, v);
          tmem_wait_ld();
          if (c == 3) release();
          const int cc = j.v0 + col0 + 32 * c;
          // named logits of this chunk, one column at a time for the warp
          while (true) {
            const int hit = __reduce_min_sync(0xffffffffu, nm.next);
            if (hit >= cc + 32) break;
            float z = 0.f;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (hit == cc + e) z = __uint_as_float(v[e]);
            while (nm.next == hit) {
              p.named[(size_t)m * p.K + nm.pos] = z * p.inv_tau;
              nm.advance();
            }
          }
          float t[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) t[e] = __uint_as_float(v[e]) * c2;
          if (cc + 32 > vend) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (cc + e >= vend) t[e] = -INFINITY;
          }
          float cm = t[0];
#pragma unroll
          for (int e = 1; e < 31; e += 2) cm = max3f(cm, t[e], t[e + 1]);
          cm = fmaxf(cm, t[31]);
          const float nx = fmaxf(mx, cm);
          if (nx > -INFINITY) {
            float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              s0 += ex2(t[e] - nx);
              s1 += ex2(t[e + 1] - nx);
              s2 += ex2(t[e + 2] - nx);
              s3 += ex2(t[e + 3] - nx);
            }
            sum = sum * ex2(mx - nx) + ((s0 + s1) + (s2 + s3));
            mx = nx;
          } else {
            // only -inf or NaN so far: NaN has to stay
#pragma unroll
            for (int e = 0; e < 32; ++e) sum += t[e] == -INFINITY ? 0.f : t[e];
          }
        }
        if (m < kept) p.part[(size_t)(2 * un.tn + half) * p.row_pitch + m] = make_float2(mx, sum);
      } else if (j.kind == JOB_DZ) {
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t v[32];
          tmem_ld32(tl + a * kTile + 32 * c, v);
          tmem_wait_ld();
          if (c == 3) release();
          const int cc = j.v0 + col0 + 32 * c;
          float t[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) t[e] = ca * ex2(fmaf(__uint_as_float(v[e]), c2, -lse2));
          while (true) {
            const int hit = __reduce_min_sync(0xffffffffu, nm.next);
            if (hit >= cc + 32) break;
            float q = 0.f;
            while (nm.next == hit) {
              q += share ? share[nm.pos] : 1.f;
              nm.advance();
            }
            q *= cb;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (hit == cc + e) t[e] -= q;
          }
          // rows that are not kept and columns past the vocabulary are zeros:
          // they are K values of the products that read this buffer
          const int left = m < kept ? vend - cc : 0;
          if (left < 32) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (e >= left) t[e] = 0.f;
          }
          if ((c & 1) == 0) {
            if (lane == 0) bulk_wait_group_read0();  // the staging buffer is free again
            __syncwarp();
          }
#pragma unroll
          for (int e = 0; e < 4; ++e)
            st_shared_v4(my_row + ((((c & 1) * 4 + e) ^ sw) << 4), pack_bf16(t[8 * e], t[8 * e + 1]),
                         pack_bf16(t[8 * e + 2], t[8 * e + 3]), pack_bf16(t[8 * e + 4], t[8 * e + 5]),
                         pack_bf16(t[8 * e + 6], t[8 * e + 7]));
          if (c & 1) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&maps.dz_out[j.buf], stage, col0 + 32 * (c - 1), row0);
              bulk_commit_group();
            }
          }
        }
      } else {
        const bool f32 = j.kind == JOB_DX || p.dw_f32;
        const CUtensorMap* mo = j.kind == JOB_DX ? &maps.dx_out : &maps.dw_out;
        const int out_row = j.kind == JOB_DX ? un.split * slot_rows(kept) + row0 : j.v0 + row0;
        const int out_rows = j.kind == JOB_DX ? kept : j.vn;  // rows of the job that exist
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t v[32];
          tmem_ld32(tl + a * kTile + 32 * c, v);
          tmem_wait_ld();
          if (c == 3) release();
          if (un.nkb == 0) {  // no rows kept: nothing was multiplied
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = 0u;
          }
          if (col0 + 32 * c >= p.C || row0 >= out_rows) continue;  // uniform in the warp
          if (f32 || (c & 1) == 0) {
            if (lane == 0) bulk_wait_group_read0();
            __syncwarp();
          }
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
          const bool last = col0 + 32 * (c + 1) >= p.C;
          if (f32 || (c & 1) || last) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              const int cs = col0 + 32 * (f32 ? c : (c & ~1));
              if (j.kind == JOB_DX && j.add) tma_reduce_add_2d(mo, stage, cs, out_row);
              else tma_store_2d(mo, stage, cs, out_row);
              bulk_commit_group();
            }
          }
        }
      }
    }
    if (lane == 0) bulk_wait_group0();  // stores complete before the CTA ends
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // no CTA leaves (or frees TMEM) while the other may still signal it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

}  // namespace head100
