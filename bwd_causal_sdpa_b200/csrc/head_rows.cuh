// head_rows.cuh -- the row-wise passes around the output head's products:
// which rows count, the teacher's lists, and the closing sums.
#pragma once

#include <limits.h>

#include "common.cuh"
#include "head_sm100.cuh"

namespace head100 {

constexpr int kTeacherWarps = 4;
constexpr int kMaxNamed = 1024;  // teacher entries per row

// A row whose upstream gradients are both zero has none to pass on.
__device__ __forceinline__ bool has_weight(const float* dloss, const float* dlse, int r) {
  return !dloss || dloss[r] != 0.f || (dlse && dlse[r] != 0.f);
}

// Compacts the kept rows: row_of (kept row -> row), pos (row -> kept row or
// -1), their number, what each brings to the epilogues (par), and, unless all
// are kept in order, their x rows in xc, followed by zero rows up to a multiple
// of the tile (K values of dz^T x). Every block counts the rows before
// its own from the flags themselves (read from L2, several at a time), so
// there is one launch and no pass between. Also clears ctl, and dx of the rows
// left out.
// Order is kept, or, with tile_start and more than one row tile kept, rows go by
// the vocabulary tile of their foremost id (a counting sort, stable): the rows
// that name a tile then are few 64-row blocks, tile_start[t] to tile_start[t + 1].
// flags: [N] non-zero where the row counts; or null: target in [0, V) and an
// upstream gradient that is not zero. A target >= V is reported.
constexpr int kMaxSortTiles = 4096;  // 8 bytes of shared memory each
struct RowsArgs {
  const int *target, *flags;
  const float *lse, *dloss, *dlse;  // null in the forward (dlse: or when absent)
  const uint4* x;
  uint4 *xc, *dx;  // dx: null in the forward
  int *row_of, *pos, *n_kept;
  RowPar* par;
  const int* foremost;  // by row: the target, or the id of the teacher's largest share
  int *key, *tile_start;  // foremost by kept row, and [tiles + 1]; or null
  int tiles;
  unsigned* ctl;
  int n_ctl;
  int N, V, c8, rows_per_block;
  float inv_tau;
};
constexpr int kRowThreads = 512;
__global__ void __launch_bounds__(kRowThreads) head_rows_kernel(const RowsArgs a) {
  pdl_wait_and_trigger();
  constexpr int kWarps = kRowThreads / 32;
  __shared__ int s_sum[2][kWarps];
  __shared__ int s_warp[kWarps];
  __shared__ int s_tile[kRowThreads];
  extern __shared__ int s_count[];  // by tile: kept rows from this block on, then those before
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r0 = blockIdx.x * a.rows_per_block, r1 = min(a.N, r0 + a.rows_per_block);
  for (int i = blockIdx.x * kRowThreads + tid; i < a.n_ctl; i += gridDim.x * kRowThreads)
    a.ctl[i] = 0;
  const int* __restrict__ foremost = a.foremost;
  const int* __restrict__ flags = a.flags;
  const int* __restrict__ target = a.target;
  const float* __restrict__ dloss = a.dloss;
  const float* __restrict__ dlse = a.dlse;
  auto counts = [&](int r) -> int {
    if (flags) return flags[r] != 0;
    int k = (unsigned)target[r] < (unsigned)a.V;
    if (dloss) {
      const float g = dloss[r], h = dlse ? dlse[r] : 0.f;
      k &= (g != 0.f) | (h != 0.f);
    }
    return k;
  };
  if (a.tile_start) {
    for (int t = tid; t < 2 * a.tiles; t += kRowThreads) s_count[t] = 0;
    __syncthreads();
  }
  int before = 0, total = 0;
  for (int b = tid; b < a.N; b += 8 * kRowThreads) {
    int k[8], f[8];  // eight rows' loads before anything is counted
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int r = b + j * kRowThreads;
      k[j] = r < a.N ? counts(r) : 0;
      f[j] = a.tile_start && r < a.N ? foremost[r] : 0;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const bool earlier = b + j * kRowThreads < r0;
      total += k[j];
      before += earlier ? k[j] : 0;
      if (a.tile_start && k[j]) atomicAdd(&s_count[(earlier ? a.tiles : 0) + f[j] / kTile], 1);
    }
  }
  for (int o = 16; o > 0; o >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, o);
    total += __shfl_xor_sync(0xffffffffu, total, o);
  }
  if (lane == 0) {
    s_sum[0][warp] = before;
    s_sum[1][warp] = total;
  }
  __syncthreads();
  before = total = 0;
  for (int w = 0; w < kWarps; ++w) {
    before += s_sum[0][w];
    total += s_sum[1][w];
  }
  if (blockIdx.x == 0 && tid == 0) *a.n_kept = total;
  const bool sorted = a.tile_start && total > kTile;
  if (sorted) {
    // where each tile's rows start, and this block's among them: a few tiles a thread
    const int each = (a.tiles + kRowThreads - 1) / kRowThreads;
    const int t0 = min(a.tiles, tid * each), t1 = min(a.tiles, t0 + each);
    int sum = 0;
    for (int t = t0; t < t1; ++t) sum += s_count[t] + s_count[a.tiles + t];
    int upto = sum;
    for (int o = 1; o < 32; o <<= 1) {
      const int below = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += below;
    }
    if (lane == 31) s_warp[warp] = upto;
    __syncthreads();
    for (int w = 0; w < warp; ++w) upto += s_warp[w];
    int start = upto - sum;
    for (int t = t0; t < t1; ++t) {
      const int own = s_count[t], earlier = s_count[a.tiles + t];
      if (blockIdx.x == 0) a.tile_start[t] = start;
      s_count[t] = start + earlier;
      start += own + earlier;
    }
    if (blockIdx.x == 0 && tid == 0) a.tile_start[a.tiles] = total;
    __syncthreads();
  }
  for (int b = r0; b < r1; b += kRowThreads) {
    const int r = b + tid;
    const bool in = r < r1;
    const bool k = in && counts(r);
    if (in && a.target && a.target[r] >= a.V) report_status(ATTN_EDEVICE_INPUT);
    int at = 0;
    if (sorted) {
      const int t = k ? foremost[r] / kTile : -1;
      s_tile[tid] = t;
      __syncthreads();
      if (k) {
        at = s_count[t];
        for (int i = 0; i < tid; ++i) at += s_tile[i] == t ? 1 : 0;
      }
      __syncthreads();
      if (k) atomicAdd(&s_count[t], 1);
    } else {
      const unsigned votes = __ballot_sync(0xffffffffu, k);
      if (lane == 0) s_warp[warp] = __popc(votes);
      __syncthreads();
      int all = 0;
      at = before;
      for (int w = 0; w < kWarps; ++w) {
        at += w < warp ? s_warp[w] : 0;
        all += s_warp[w];
      }
      at += __popc(votes & ((1u << lane) - 1u));
      before += all;
    }
    if (in) a.pos[r] = k ? at : -1;
    if (k) {
      a.row_of[at] = r;
      RowPar rp = {0.f, 0.f, 0.f, a.target ? a.target[r] : r};
      if (a.dloss) {
        const float g = a.dloss[r];
        rp.lse2 = a.lse[r] * kLog2e;
        rp.ca = (g + (a.dlse ? a.dlse[r] : 0.f)) * a.inv_tau;
        rp.cb = g * a.inv_tau;
      }
      a.par[at] = rp;
      if (a.key) a.key[at] = foremost[r];
    }
    __syncthreads();
  }
  if (total == a.N && !sorted) return;  // the products read x in place
  // a warp copies four rows at a time (their pos entries were written by this block)
  const uint4* __restrict__ x = a.x;
  uint4* __restrict__ xc = a.xc;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int r = r0 + warp; r < r1; r += 4 * kWarps) {
    int at[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) at[j] = r + j * kWarps < r1 ? a.pos[r + j * kWarps] : -2;
#pragma unroll 2
    for (int i = lane; i < a.c8; i += 32) {
      uint4 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[j] = at[j] >= 0 ? x[(size_t)(r + j * kWarps) * a.c8 + i] : zero;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (at[j] >= 0) xc[(size_t)at[j] * a.c8 + i] = v[j];
        else if (at[j] == -1 && a.dx) a.dx[(size_t)(r + j * kWarps) * a.c8 + i] = zero;
      }
    }
  }
  const int pad = slot_rows(total);
  for (int r = total + blockIdx.x * kWarps + warp; r < pad; r += gridDim.x * kWarps)
    for (int i = lane; i < a.c8; i += 32) xc[(size_t)r * a.c8 + i] = zero;
}

// The teacher's list of one row per warp: q = softmax of t / tau over the
// entries present (0 <= id < V), ids sorted ascending with their q (absent
// ones last, id INT_MAX, q 0), how many of them lie below each multiple of
// first_cols columns, sum q log q, the id of the largest share (the lowest such
// id), and whether the row counts (some entry above -inf, and
// an upstream gradient that is not zero). The sort is by rank (K comparisons
// per entry): stable, so equal ids keep their order. The maximum is taken off
// before the division by tau: entries at the type's lowest value then differ
// by exactly 0.
template <typename TT>
__global__ void __launch_bounds__(32 * kTeacherWarps)
    head_teacher_kernel(const int* __restrict__ t_idx, const TT* __restrict__ t_logit,
                        float inv_tau, const float* __restrict__ dloss,
                        const float* __restrict__ dlse, int* __restrict__ ids,
                        float* __restrict__ share, uint16_t* __restrict__ first, int first_pitch, int first_cols,
                        float* __restrict__ entropy, int* __restrict__ foremost,
                        int* __restrict__ flags, int N, int V, int K) {
  pdl_wait_and_trigger();
  extern __shared__ __align__(16) int smem_teacher[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int K4 = (K + 3) / 4;
  int* key = smem_teacher + warp * 8 * K4;  // 16-byte aligned
  int* sorted = key + 4 * K4;
  for (int r = blockIdx.x * kTeacherWarps + warp; r < N; r += gridDim.x * kTeacherWarps) {
    const int* in = t_idx + (size_t)r * K;
    const TT* tl = t_logit + (size_t)r * K;
    float top = -INFINITY;
    bool bad = false, nan = false;
    for (int k = lane; k < K; k += 32) {
      const int id = in[k];
      const bool here = (unsigned)id < (unsigned)V;
      bad |= id >= V;
      key[k] = here ? id : INT_MAX;
      if (here) {
        const float t = to_f32(tl[k]);
        nan |= isnan(t);
        top = fmaxf(top, t);
      }
    }
    if (lane < 4 * K4 - K) key[K + lane] = INT_MAX;
    if (bad) report_status(ATTN_EDEVICE_INPUT);
    top = warp_max(top);
    nan = __any_sync(0xffffffffu, nan);
    __syncwarp();
    const bool some = top > -INFINITY || nan;
    float sum = 0.f;
    for (int k = lane; k < K; k += 32)
      if (key[k] != INT_MAX) sum += expf((to_f32(tl[k]) - top) * inv_tau);
    sum = warp_sum(sum);
    const float log_sum = logf(sum);
    float ent = 0.f;
    for (int k = lane; k < K; k += 32) {
      const int mine = key[k];
      float q = 0.f;
      if (some && mine != INT_MAX) {
        const float d = (to_f32(tl[k]) - top) * inv_tau;
        q = expf(d) / sum;
        if (q != 0.f) ent += q * (d - log_sum);  // NaN stays
      }
      int rank = 0;
#pragma unroll 4
      for (int i = 0; i < K4; ++i) {
        const int4 o = reinterpret_cast<const int4*>(key)[i];
        const int other[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          rank += (other[e] < mine || (other[e] == mine && 4 * i + e < k)) ? 1 : 0;
      }
      sorted[rank] = mine;
      ids[(size_t)r * K + rank] = mine;
      share[(size_t)r * K + rank] = q;
    }
    ent = warp_sum(ent);
    __syncwarp();
    for (int b = lane; b < first_pitch; b += 32) {
      int lo = 0, hi = K;
      const long col = (long)first_cols * b;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (sorted[mid] < col) lo = mid + 1;
        else hi = mid;
      }
      first[(size_t)r * first_pitch + b] = (uint16_t)lo;
    }
    if (foremost) {
      int id = INT_MAX;
      for (int k = lane; k < K; k += 32)
        if (key[k] < id && (nan || to_f32(tl[k]) == top)) id = key[k];
      id = __reduce_min_sync(0xffffffffu, id);
      if (lane == 0) foremost[r] = id;
    }
    if (lane == 0) {
      flags[r] = some && has_weight(dloss, dlse, r) ? 1 : 0;
      if (entropy) entropy[r] = ent;
    }
    __syncwarp();
  }
}

// lse and loss of every row from the parts of its logits: four rows per warp
// (the 32 bytes that their parts share), eight lanes per row. loss =
// sum_k q_k (log q_k + lse - z_k), for a single target lse - z. Without pos no
// row was left out before: flags or target say which rows count.
constexpr int kLossThreads = 128;
__global__ void __launch_bounds__(kLossThreads)
    head_loss_kernel(const float2* __restrict__ part, const float* __restrict__ named,
                     const float* __restrict__ exact, const int* __restrict__ ids,
                     const float* __restrict__ share, const float* __restrict__ entropy,
                     const int* __restrict__ pos, const int* __restrict__ target,
                     const int* __restrict__ flags, float* __restrict__ loss,
                     float* __restrict__ lse, int N, int V, int K, int parts, int row_pitch) {
  pdl_wait_and_trigger();
  const int lane = threadIdx.x & 31, slice = lane >> 2;
  const int r = (blockIdx.x * (kLossThreads / 32) + (threadIdx.x >> 5)) * 4 + (lane & 3);
  int at = -1;
  if (r < N) {
    if (pos) {
      at = pos[r];
    } else if (flags) {
      at = flags[r] ? r : -1;
    } else {
      at = (unsigned)target[r] < (unsigned)V ? r : -1;
      if (target[r] >= V) report_status(ATTN_EDEVICE_INPUT);
    }
  }
  float m = -INFINITY, s = 0.f;
  auto join = [&](float om, float os) {
    const float nm = fmaxf(m, om);
    s = nm > -INFINITY ? s * exp2f(m - nm) + os * exp2f(om - nm) : s + os;
    m = nm;
  };
  if (at >= 0) {
    const float2* mine = part + at;
    for (int j = slice; j < parts; j += 8 * 8) {
      float2 t[8];  // eight loads in flight
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int q = j + 8 * i;
        t[i] = q < parts ? mine[(size_t)q * row_pitch] : make_float2(-INFINITY, 0.f);
      }
      float top = t[0].x;
#pragma unroll
      for (int i = 1; i < 8; ++i) top = fmaxf(top, t[i].x);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        sum += top > -INFINITY ? t[i].y * exp2f(t[i].x - top) : t[i].y;
      join(top, sum);
    }
  }
  // the lanes of a row join in pairs; every lane ends with the same bits
  for (int o = 4; o < 32; o <<= 1) {
    const float om = __shfl_xor_sync(0xffffffffu, m, o), os = __shfl_xor_sync(0xffffffffu, s, o);
    const float nm = fmaxf(m, om);
    s = nm > -INFINITY
            ? __fadd_rn(__fmul_rn(s, exp2f(m - nm)), __fmul_rn(os, exp2f(om - nm)))
            : s + os;
    m = nm;
  }
  float l = (m + log2f(s)) * kLn2;
  float d = 0.f;
  const size_t own = (size_t)(at >= 0 ? at : 0) * K;
  const float* z = named;
  if (exact) {
    // lse takes the named logits' more exact values too: each moves it by its
    // share of the softmax times the difference (an id named twice, once)
    z = exact;
    if (at >= 0)
      for (int k = slice; k < K; k += 8) {
        const int id = ids[(size_t)r * K + k];
        const bool again = k > 0 && ids[(size_t)r * K + k - 1] == id;
        const float diff = exact[own + k] - named[own + k];
        // (both may be infinite)
        if ((unsigned)id < (unsigned)V && !again && isfinite(diff) && diff != 0.f)
          d += expf(named[own + k] - l) * diff;
      }
    for (int o = 4; o < 32; o <<= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    l += d;
    d = 0.f;
  }
  if (at >= 0)
    for (int k = slice; k < K; k += 8) {
      const float q = share ? share[(size_t)r * K + k] : 1.f;
      if (q != 0.f) d += q * (l - z[own + k]);
    }
  for (int o = 4; o < 32; o <<= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
  if (slice == 0 && r < N) {
    lse[r] = at >= 0 ? l : 0.f;
    loss[r] = at >= 0 ? (share ? entropy[r] + d : d) : 0.f;
  }
}

// dx of the kept rows where its vocabulary axis was split: the accumulators
// added in order, then what the rounding of dz took from the named columns (key
// instead of ids: from the foremost one), and rounded once. Eight columns per thread. Without a split
// the last piece's epilogue has written dx, and this pass ends at once.
__global__ void __launch_bounds__(256)
    head_dx_kernel(const float* __restrict__ acc, const int* __restrict__ row_of,
                   const int* __restrict__ n_kept, const float* __restrict__ rest,
                   const int* __restrict__ ids, const int* __restrict__ key,
                   const uint4* __restrict__ w, uint4* __restrict__ dx, int V, int C, int K,
                   int kb_total) {
  pdl_wait_and_trigger();
  const int kept = *n_kept;
  int splits, kb_per;
  split_dx(((kept + kTile - 1) / kTile) * ((C + kTile - 1) / kTile), kb_total, splits, kb_per);
  if (splits == 1) return;
  if (key) {
    K = 1;
    if (kept <= kTile) rest = nullptr;  // both terms of dz were multiplied
  }
  const size_t slot = (size_t)slot_rows(kept) * C;
  const int c8 = C / 8;
  const long n = (long)kept * c8;
  for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long)gridDim.x * 256) {
    const int m = (int)(i / c8), c = (int)(i - (long)m * c8) * 8;
    const float* src = acc + (size_t)m * C + c;
    const int row = row_of[m];
    float g[kFewNamed];
    uint4 wv[kFewNamed];
#pragma unroll
    for (int k = 0; k < kFewNamed; ++k) {
      g[k] = 0.f;
      wv[k] = make_uint4(0, 0, 0, 0);
      if (rest && k < K) {
        const int id = key ? key[m] : ids[(size_t)row * K + k];
        if ((unsigned)id < (unsigned)V) {
          g[k] = rest[(size_t)m * K + k];
          wv[k] = w[(size_t)id * c8 + c / 8];
        }
      }
    }
    float4 lo = make_float4(0.f, 0.f, 0.f, 0.f), hi = lo;
#pragma unroll 8
    for (int s = 0; s < splits; ++s, src += slot) {
      const float4 a = *reinterpret_cast<const float4*>(src);
      const float4 b = *reinterpret_cast<const float4*>(src + 4);
      lo.x += a.x; lo.y += a.y; lo.z += a.z; lo.w += a.w;
      hi.x += b.x; hi.y += b.y; hi.z += b.z; hi.w += b.w;
    }
#pragma unroll
    for (int k = 0; k < kFewNamed; ++k)
      if (g[k] != 0.f) {
        add_scaled4(lo, g[k], make_uint2(wv[k].x, wv[k].y));
        add_scaled4(hi, g[k], make_uint2(wv[k].z, wv[k].w));
      }
    dx[(size_t)row * c8 + c / 8] =
        make_uint4(pack_bf16(lo.x, lo.y), pack_bf16(lo.z, lo.w), pack_bf16(hi.x, hi.y),
                   pack_bf16(hi.z, hi.w));
  }
}

}  // namespace head100
