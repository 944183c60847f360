// head_api.cuh -- host side of the output head's losses (included at the end
// of attn_api.cu, whose helpers it uses): checks, workspace plan, operand maps
// and the entry points attn_head_* of include/attn.h.
#pragma once

#include <float.h>

#include <algorithm>

#include "head_rows.cuh"

namespace {

// Vocabulary rows per piece of the backward: the dz buffer of a piece (three
// are in use) takes up to 96 MiB, or 2048 columns when the rows are many
// (shorter pieces would add into dx more often than their products are worth).
// 8192 rows of width 2048: 2.61 ms with 64 MiB, 2.55 with 96, 2.56 with 160.
// With an fp32 dW a column takes both terms of dz, and the fewest columns are
// half as many.
constexpr size_t kDzBytes = (size_t)96 << 20;
constexpr long kDzMinCols = 2048;

struct HeadPlan {
  int rows_pad = 0, piece = 0, pieces = 0, lw = 0, parts = 0;
  size_t n_kept = 0, ctl = 0, row_of = 0, pos = 0, par = 0, xc = 0, ids = 0, share = 0, entropy = 0, flags = 0, first = 0;
  size_t part = 0, named = 0, exact = 0;  // forward
  size_t dz[head100::kDzBuffers] = {}, lo[head100::kDzBuffers] = {}, acc = 0, rest = 0;  // backward
  size_t foremost = 0, key = 0, tile_start = 0;
  int rest_k = 0, tiles = 0;
  bool keyed = false, sorted = false;
  long acc_rows = 0, lo_blocks = 0;  // of 64 rows x 256 columns, in each of lo's buffers
  int lo_rows = 0;
  int n_ctl = 0, first_pitch = 0;
  size_t total = 0;
};

bool head_sizes_ok(int N, int V, int C, int K) {
  if (N <= 0 || V <= 0 || C <= 0 || K < 0 || K > head100::kMaxNamed) return false;
  if (C % 8 != 0 || C > (1 << 20) || N > (1 << 26) || V > (1 << 26)) return false;
  const long tiles_n = N / 256 + 1, tiles_v = V / 256 + 1, tiles_c = C / 256 + 1;
  // the units of a call are numbered in 32 bits: dz, dW, and dx per piece
  return tiles_n * tiles_v < (1L << 28) && tiles_v * tiles_c < (1L << 28) &&
         tiles_n * tiles_c * (2 * (V / kDzMinCols) + 1) < (1L << 28);
}

// K = 0: a single target per row (attn_head_ce), else teacher entries per row.
HeadPlan head_plan(int N, int V, int C, int K, bool bwd, bool dw_f32) {
  using namespace head100;
  HeadPlan p;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = round_up(off + bytes);
    return at;
  };
  p.rows_pad = (N + kTile - 1) / kTile * kTile;
  long cols = ((long)V + kTile - 1) / kTile * kTile;
  // The rows' foremost ids matter where a bf16 dW may have more than one row tile
  // kept; the rows are then sorted by them, while the tiles have room in the
  // row pass's shared memory.
  p.keyed = bwd && !dw_f32 && N > kTile;
  p.tiles = (V + kTile - 1) / kTile;
  p.sorted = p.keyed && p.tiles <= kMaxSortTiles;
  // rows of lo in whole: with a bf16 dW where one row tile is kept at most, and
  // otherwise a staircase of blocks (64 rows x a tile), one row block or one
  // tile further each
  const size_t stairs = p.sorted ? (size_t)p.rows_pad / 64 * 64 * kTile * 2 : 0;
  const long lo_pad = !bwd ? 0 : dw_f32 ? p.rows_pad : kTile;
  p.lo_rows = (int)(lo_pad / 64);
  if (bwd)
    cols = std::min(cols, std::max((long)((kDzBytes - std::min(kDzBytes, stairs)) /
                                           ((size_t)(p.rows_pad + lo_pad) * 2)) / kTile * kTile,
                                   dw_f32 ? kDzMinCols / 2 : kDzMinCols));
  p.pieces = (int)((V + cols - 1) / cols);
  p.piece = (int)(((V + p.pieces - 1) / p.pieces + kTile - 1) / kTile * kTile);
  p.pieces = (V + p.piece - 1) / p.piece;
  // Narrow logits tiles, half as long, where they still find a pair each (one
  // row tile against 5306 ids, width 888: 42 units of 3600 cycles for 21 of
  // 7200). Beyond, W bounds the time, and its boxes of 64 rows move slower: 33
  // rows against 24576 ids took 34 us narrow, 26 wide.
  const long narrow = (long)(p.rows_pad / kTile) * ((std::min(p.piece, V) + 127) / 128);
  p.lw = narrow <= kPairs ? 128 : 256;
  p.n_ctl = ctl_words(V, p.pieces);
  p.n_kept = take(4);
  p.ctl = take((size_t)p.n_ctl * 4);
  p.par = take((size_t)p.rows_pad * sizeof(RowPar));
  p.row_of = take((size_t)p.rows_pad * 4);
  p.pos = take((size_t)N * 4);
  p.xc = take((size_t)p.rows_pad * C * 2);
  if (K > 0) {
    p.ids = take((size_t)N * K * 4);
    p.share = take((size_t)N * K * 4);
    p.flags = take((size_t)N * 4);
    p.first_pitch = 2 * ((V + p.lw - 1) / p.lw) + 1;
    p.first = take((size_t)N * p.first_pitch * 2);
    if (!bwd) p.entropy = take((size_t)N * 4);
  }
  if (!bwd) {
    p.parts = 2 * ((V + p.lw - 1) / p.lw);
    p.part = take((size_t)p.parts * p.rows_pad * sizeof(float2));
    p.named = take((size_t)N * std::max(K, 1) * 4);
    if (K <= kFewNamed) p.exact = take((size_t)N * std::max(K, 1) * 4);
    p.total = off;
    return p;
  }
  p.lo_blocks = (long)p.lo_rows * (p.piece / kTile);
  if (p.sorted) p.lo_blocks = std::max(p.lo_blocks, (long)p.rows_pad / 64 + p.piece / kTile);
  for (int b = 0; b < std::min(p.pieces, kDzBuffers); ++b) {
    p.dz[b] = take((size_t)p.rows_pad * p.piece * 2);
    p.lo[b] = take((size_t)p.lo_blocks * 64 * kTile * 2);
  }
  // the accumulators of dx: the most rows that any number of kept rows takes
  const int tn = (C + kTile - 1) / kTile, kb = (std::min(p.piece, V) + kKB - 1) / kKB;
  long rows = p.rows_pad;
  for (int tm = 1; tm * kTile <= p.rows_pad && tm * tn < kPairs; ++tm) {
    int splits, per;
    split_dx(tm * tn, kb, splits, per);
    rows = std::max(rows, (long)tm * kTile * splits);
  }
  p.acc_rows = rows;
  p.acc = take((size_t)rows * C * 4);
  p.rest_k = K <= kFewNamed ? std::max(K, 1) : p.keyed ? 1 : 0;
  if (p.rest_k) p.rest = take((size_t)N * p.rest_k * 4);
  if (p.keyed) {
    if (K > 0) p.foremost = take((size_t)N * 4);
    p.key = take((size_t)p.rows_pad * 4);
  }
  if (p.sorted) p.tile_start = take((size_t)(p.tiles + 1) * 4);
  p.total = off;
  return p;
}

// The bytes that a call of either type of dW finds enough.
size_t head_bytes(int N, int V, int C, int K, bool bwd) {
  const size_t bytes = head_plan(N, V, C, K, bwd, false).total;
  return bwd ? std::max(bytes, head_plan(N, V, C, K, bwd, true).total) : bytes;
}

// A matrix [rows][cols] (row pitch `pitch` elements) in boxes of 128 bytes x
// box_rows rows, 128-byte swizzle; past the edges reads give zeros, writes are
// dropped.
bool head_map(CUtensorMap* m, const void* base, bool f32, long rows, long cols, long pitch,
              int box_rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const int es = f32 ? 4 : 2;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)pitch * es};
  cuuint32_t box[2] = {(cuuint32_t)(128 / es), (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
             const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same matrix in 64-column blocks, two of them (64 rows each) per box:
// [cols / 64][rows][64]. One box of 128 rows of 128 bytes moves 83 bytes per
// cycle and SM, boxes of 64 rows 66. cols % 64 == 0.
bool head_block_map(CUtensorMap* m, const void* base, long rows, long cols) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {64, (cuuint64_t)rows, (cuuint64_t)(cols / 64)};
  cuuint64_t strides[2] = {(cuuint64_t)cols * 2, 128};
  cuuint32_t box[3] = {64, (cuuint32_t)head100::kKB, 2};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Everything the entry points share: arguments as the caller gave them.
struct HeadCall {
  const void *x, *w;
  const int32_t* target;         // attn_head_ce*
  const int32_t* t_idx;          // attn_head_distill*
  const void* t_logit;
  float tau;
  int t_dtype;
  float *loss, *lse_out;         // forward
  const float *lse, *dloss, *dlse;  // backward
  void *dx, *dw;
  int dw_dtype;
  int N, V, C, K;
  bool bwd;
};

int head_check(const HeadCall& c, void* ws, size_t ws_bytes) {
  if (!c.x || !c.w) return ATTN_EINVAL;
  if (c.K == 0 ? !c.target : (!c.t_idx || !c.t_logit)) return ATTN_EINVAL;
  if (c.bwd ? (!c.lse || !c.dloss || !c.dx || !c.dw) : (!c.loss || !c.lse_out)) return ATTN_EINVAL;
  if (c.N <= 0 || c.V <= 0 || c.C <= 0) return ATTN_EINVAL;
  // normal: below, 1 / tau in base 2 overflows
  if (!(c.tau >= FLT_MIN) || !isfinite(c.tau)) return ATTN_EINVAL;
  if (c.t_dtype != ATTN_BF16 && c.t_dtype != ATTN_F32) return ATTN_EINVAL;
  if (c.dw_dtype != ATTN_BF16 && c.dw_dtype != ATTN_F32) return ATTN_EINVAL;
  if (!head_sizes_ok(c.N, c.V, c.C, c.K)) return ATTN_EUNSUPPORTED;
  if (!aligned(c.x, 16) || !aligned(c.w, 16) || !aligned(c.target, 4) || !aligned(c.t_idx, 4) ||
      !aligned(c.t_logit, c.t_dtype == ATTN_F32 ? 4 : 2) || !aligned(c.loss, 4) ||
      !aligned(c.lse_out, 4) || !aligned(c.lse, 4) || !aligned(c.dloss, 4) ||
      !aligned(c.dlse, 4) || !aligned(c.dx, 16) || !aligned(c.dw, 16))
    return ATTN_EALIGN;
  if (!ws || ws_bytes < head_bytes(c.N, c.V, c.C, c.K, c.bwd)) return ATTN_EWORKSPACE;
  if (!aligned(ws, 16)) return ATTN_EALIGN;
  return ATTN_OK;
}

template <bool kBwd, int kLw>
int head_gemm(const head100::Maps& maps, const head100::Params& p, cudaStream_t st) {
  using namespace head100;
  static bool smem_done[64];
  if (!ensure_smem(head_gemm_kernel<kBwd, kLw>, kSmAlloc, smem_done)) return ATTN_ECUDA;
  // pairs beyond the units that any number of kept rows gives would be idle
  const Sched s = make_sched(p, p.N);
  long units = kBwd ? kPairs : s.dz(0);
  // the fp32 logits of few named ids want warps, four of them each (two a pair)
  if (!kBwd && p.exact) units = std::max(units, ((long)p.N * p.K + 7) / 8);
  const unsigned pairs = (unsigned)std::min<long>(units, kPairs);
  ATTN_LAUNCH(KK_HEAD_GEMM, st, pdl_cluster_launch(head_gemm_kernel<kBwd, kLw>, dim3(2 * pairs), kThreads,
                                                   kSmAlloc, st, 2u, maps, p));
  return launch_status();
}

int head_run(const HeadCall& c, void* workspace, size_t ws_bytes, void* stream) {
  using namespace head100;
  if (int rc = head_check(c, workspace, ws_bytes)) return rc;
  const HeadPlan hp = head_plan(c.N, c.V, c.C, c.K, c.bwd, c.bwd && c.dw_dtype == ATTN_F32);
  cudaStream_t st = (cudaStream_t)stream;
  char* ws = (char*)workspace;
  const int N = c.N, V = c.V, C = c.C, K = c.K;
  const float inv_tau = 1.f / c.tau;
  int* ids = K ? (int*)(ws + hp.ids) : nullptr;
  float* share = K ? (float*)(ws + hp.share) : nullptr;
  float* entropy = K && !c.bwd ? (float*)(ws + hp.entropy) : nullptr;
  int* flags = K ? (int*)(ws + hp.flags) : nullptr;
  int* foremost = K && hp.keyed ? (int*)(ws + hp.foremost) : nullptr;
  int *row_of = (int*)(ws + hp.row_of), *pos = (int*)(ws + hp.pos),
      *n_kept = (int*)(ws + hp.n_kept);
  void* xc = ws + hp.xc;

  if (K) {
    const unsigned blocks = (unsigned)std::min<long>((N + kTeacherWarps - 1L) / kTeacherWarps, 148L * 16);
    const size_t smem = (size_t)kTeacherWarps * ((K + 3) / 4) * 32;
    uint16_t* first = (uint16_t*)(ws + hp.first);
    if (c.t_dtype == ATTN_F32)
      ATTN_LAUNCH(KK_HEAD_ROWS, st, pdl_launch(head_teacher_kernel<float>, blocks, 32 * kTeacherWarps, smem, st,
                                               c.t_idx, (const float*)c.t_logit, inv_tau, c.dloss, c.dlse,
                                               ids, share, first, hp.first_pitch, hp.lw / 2, entropy, foremost, flags, N, V, K));
    else
      ATTN_LAUNCH(KK_HEAD_ROWS, st, pdl_launch(head_teacher_kernel<__nv_bfloat16>, blocks, 32 * kTeacherWarps, smem, st,
                                               c.t_idx, (const __nv_bfloat16*)c.t_logit, inv_tau, c.dloss, c.dlse,
                                               ids, share, first, hp.first_pitch, hp.lw / 2, entropy, foremost, flags, N, V, K));
  }
  // A forward of one row tile costs the same for any number of kept rows, and
  // its rows do not meet: it goes without the row pass (4 of 27 us at one row).
  const bool whole = !c.bwd && N <= kTile;
  RowsArgs ra = {};
  ra.target = K ? nullptr : c.target;
  ra.foremost = K ? foremost : c.target;
  ra.key = hp.keyed ? (int*)(ws + hp.key) : nullptr;
  ra.tile_start = hp.sorted ? (int*)(ws + hp.tile_start) : nullptr;
  ra.tiles = hp.tiles;
  ra.flags = flags;
  ra.lse = c.lse;
  ra.dloss = c.dloss;
  ra.dlse = c.dlse;
  ra.x = (const uint4*)c.x;
  ra.xc = (uint4*)xc;
  ra.dx = (uint4*)c.dx;
  ra.row_of = row_of;
  ra.pos = pos;
  ra.n_kept = n_kept;
  ra.par = (RowPar*)(ws + hp.par);
  ra.ctl = (unsigned*)(ws + hp.ctl);
  ra.n_ctl = hp.n_ctl;
  ra.N = N;
  ra.V = V;
  ra.c8 = C / 8;
  ra.inv_tau = inv_tau;
  const int row_blocks = (int)std::min<long>((N + 15L) / 16, 148L);
  ra.rows_per_block = (N + row_blocks - 1) / row_blocks;
  if (!whole)
    ATTN_LAUNCH(KK_HEAD_ROWS, st, pdl_launch(head_rows_kernel, (unsigned)row_blocks, kRowThreads,
                                         hp.sorted ? (size_t)hp.tiles * 8 : 0, st, ra));
  if (launch_status()) return ATTN_ECUDA;

  Maps maps = {};
  Params p = {};
  p.x = (const uint4*)c.x;
  p.w = (const uint4*)c.w;
  p.N = N;
  p.V = V;
  p.C = C;
  p.K = std::max(K, 1);
  p.inv_tau = inv_tau;
  p.n_kept = whole ? nullptr : n_kept;
  p.row_of = row_of;
  p.par = ra.par;
  p.ctl = ra.ctl;
  p.piece = hp.piece;
  p.pieces = hp.pieces;
  p.lw = hp.lw;
  p.ids = K ? ids : c.target;
  p.share = share;
  p.first = K ? (const uint16_t*)(ws + hp.first) : nullptr;
  p.first_pitch = hp.first_pitch;
  p.row_pitch = hp.rows_pad;
  if (!head_map(&maps.x_k, c.x, false, N, C, C, 128) ||
      !head_map(&maps.xc_k, xc, false, hp.rows_pad, C, C, 128) ||
      !head_map(&maps.w_k, c.w, false, V, C, C, hp.lw / 2))
    return ATTN_ECUDA;

  if (!c.bwd) {
    p.part = (float2*)(ws + hp.part);
    p.named = (float*)(ws + hp.named);
    p.exact = K <= kFewNamed ? (float*)(ws + hp.exact) : nullptr;
    if (int rc = hp.lw == 128 ? head_gemm<false, 128>(maps, p, st) : head_gemm<false, 256>(maps, p, st))
      return rc;
    ATTN_LAUNCH(KK_HEAD_ROWS, st, pdl_launch(head_loss_kernel, (unsigned)((N + kLossThreads / 8 - 1) / (kLossThreads / 8)),
                                             kLossThreads, 0, st, p.part, p.named, p.exact, p.ids, share, entropy,
                                             whole ? nullptr : pos, c.target, flags, c.loss, c.lse_out, N,
                                             V, p.K, hp.parts, hp.rows_pad));
    return launch_status();
  }

  p.acc = (const float*)(ws + hp.acc);
  p.rest = hp.rest_k ? (float*)(ws + hp.rest) : nullptr;
  p.rest_k = hp.rest_k;
  p.dx = (__nv_bfloat16*)c.dx;
  p.dw_f32 = c.dw_dtype == ATTN_F32;
  p.lo_rows = hp.lo_rows;
  p.key = ra.key;
  p.tile_start = ra.tile_start;
  p.c_blocks = C % 64 == 0;
  bool ok = head_map(&maps.dx_out, p.acc, true, hp.acc_rows, C, C, 32) &&
            head_map(&maps.dw_out, c.dw, p.dw_f32 != 0, V, C, C, 32);
  if (p.c_blocks)
    ok = ok && head_block_map(&maps.x_mn, c.x, N, C) &&
         head_block_map(&maps.xc_mn, xc, hp.rows_pad, C) && head_block_map(&maps.w_mn, c.w, V, C);
  else
    ok = ok && head_map(&maps.x_mn, c.x, false, N, C, C, kKB) &&
         head_map(&maps.xc_mn, xc, false, hp.rows_pad, C, C, kKB) &&
         head_map(&maps.w_mn, c.w, false, V, C, C, kKB);
  for (int b = 0; b < std::min(hp.pieces, kDzBuffers); ++b) {
    const void* dz = ws + hp.dz[b];
    ok = ok && head_map(&maps.dz_k[b], dz, false, hp.rows_pad, hp.piece, hp.piece, 128) &&
         head_block_map(&maps.dz_mn[b], dz, hp.rows_pad, hp.piece) &&
         head_map(&maps.dz_out[b], dz, false, hp.rows_pad, hp.piece, hp.piece, 32);
    const void* lo = ws + hp.lo[b];
    ok = ok && head_map(&maps.lo_k[b], lo, false, hp.lo_blocks * 64, kTile, kTile, 128) &&
         head_block_map(&maps.lo_mn[b], lo, hp.lo_blocks * 64, kTile) &&
         head_map(&maps.lo_out[b], lo, false, hp.lo_blocks * 64, kTile, kTile, 32);
  }
  if (!ok) return ATTN_ECUDA;
  if (int rc = hp.lw == 128 ? head_gemm<true, 128>(maps, p, st) : head_gemm<true, 256>(maps, p, st))
    return rc;
  const long n8 = (long)N * (C / 8);
  ATTN_LAUNCH(KK_HEAD_ROWS, st, pdl_launch(head_dx_kernel, (unsigned)std::min<long>((n8 + 255) / 256, 148L * 8),
                                           256, 0, st, p.acc, row_of, n_kept, p.rest, p.ids,
                                           K > kFewNamed ? p.key : nullptr, p.w, (uint4*)c.dx,
                                           V, C, p.K, (std::min(hp.piece, V) + kKB - 1) / kKB));
  return launch_status();
}

}  // namespace

extern "C" {

size_t attn_head_workspace_bytes(int N, int V, int C, int K, int is_bwd) {
  if (!head_sizes_ok(N, V, C, K)) return 0;
  return head_bytes(N, V, C, K, is_bwd != 0);
}

int attn_head_ce(const void* x, const void* w, const int32_t* target, float* loss, float* lse,
                 int N, int V, int C, void* workspace, size_t ws_bytes, void* stream) {
  HeadCall c = {};
  c.x = x;
  c.w = w;
  c.target = target;
  c.tau = 1.f;
  c.loss = loss;
  c.lse_out = lse;
  c.N = N;
  c.V = V;
  c.C = C;
  return head_run(c, workspace, ws_bytes, stream);
}

int attn_head_ce_bwd(const void* x, const void* w, const int32_t* target, const float* lse,
                     const float* dloss, const float* dlse, void* dx, void* dw, int N, int V,
                     int C, int dw_dtype, void* workspace, size_t ws_bytes, void* stream) {
  HeadCall c = {};
  c.x = x;
  c.w = w;
  c.target = target;
  c.tau = 1.f;
  c.lse = lse;
  c.dloss = dloss;
  c.dlse = dlse;
  c.dx = dx;
  c.dw = dw;
  c.dw_dtype = dw_dtype;
  c.N = N;
  c.V = V;
  c.C = C;
  c.bwd = true;
  return head_run(c, workspace, ws_bytes, stream);
}

int attn_head_distill(const void* x, const void* w, const int32_t* t_idx, const void* t_logit,
                      float temperature, float* loss, float* lse, int N, int V, int C, int K,
                      int t_dtype, void* workspace, size_t ws_bytes, void* stream) {
  if (K <= 0) return ATTN_EINVAL;
  HeadCall c = {};
  c.x = x;
  c.w = w;
  c.t_idx = t_idx;
  c.t_logit = t_logit;
  c.tau = temperature;
  c.t_dtype = t_dtype;
  c.loss = loss;
  c.lse_out = lse;
  c.N = N;
  c.V = V;
  c.C = C;
  c.K = K;
  return head_run(c, workspace, ws_bytes, stream);
}

int attn_head_distill_bwd(const void* x, const void* w, const int32_t* t_idx, const void* t_logit,
                          float temperature, const float* lse, const float* dloss,
                          const float* dlse, void* dx, void* dw, int N, int V, int C, int K,
                          int t_dtype, int dw_dtype, void* workspace, size_t ws_bytes,
                          void* stream) {
  if (K <= 0) return ATTN_EINVAL;
  HeadCall c = {};
  c.x = x;
  c.w = w;
  c.t_idx = t_idx;
  c.t_logit = t_logit;
  c.tau = temperature;
  c.t_dtype = t_dtype;
  c.lse = lse;
  c.dloss = dloss;
  c.dlse = dlse;
  c.dx = dx;
  c.dw = dw;
  c.dw_dtype = dw_dtype;
  c.N = N;
  c.V = V;
  c.C = C;
  c.K = K;
  c.bwd = true;
  return head_run(c, workspace, ws_bytes, stream);
}

}  // extern "C"
