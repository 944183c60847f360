// head_rows.cuh -- the row-wise passes around the output head's products:
// which rows count, the teacher's lists, and the closing sums.
#pragma once

#include <limits.h>

#include "common.cuh"
#include "head_sm100.cuh"

namespace head100 {

constexpr int kRowThreads = 256;
constexpr int kTeacherWarps = 4;
constexpr int kMaxNamed = 1024;  // teacher entries per row

// A row whose upstream gradients are both zero has none to pass on.
__device__ __forceinline__ bool has_weight(const float* dloss, const float* dlse, int r) {
  return !dloss || dloss[r] != 0.f || (dlse && dlse[r] != 0.f);
}

// Compacts the kept rows: row_of (kept row -> row), pos (row -> kept row or
// -1), their number, and, unless all are kept, their x rows in xc, followed by
// zero rows up to a multiple of the tile (K values of dz^T x). Order is kept.
// Every block counts the rows before its own from the flags themselves (4
// bytes per row, read from L2), so there is one launch and no pass between.
// flags: [N] non-zero where the row counts; or null: target in [0, V) and an
// upstream gradient that is not zero. A target >= V is reported.
__global__ void __launch_bounds__(kRowThreads)
    head_rows_kernel(const int* __restrict__ target, const int* __restrict__ flags,
                     const float* __restrict__ dloss, const float* __restrict__ dlse,
                     const uint4* __restrict__ x, uint4* __restrict__ xc, int* __restrict__ row_of,
                     int* __restrict__ pos, int* __restrict__ n_kept, int N, int V, int c8,
                     int rows_per_block) {
  pdl_wait_and_trigger();
  __shared__ int s_sum[2][kRowThreads / 32];
  __shared__ int s_warp[kRowThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r0 = blockIdx.x * rows_per_block, r1 = min(N, r0 + rows_per_block);
  auto counts = [&](int r) -> bool {
    if (flags) return flags[r] != 0;
    return (unsigned)target[r] < (unsigned)V && has_weight(dloss, dlse, r);
  };
  int before = 0, total = 0;
  for (int r = tid; r < N; r += kRowThreads) {
    const int k = counts(r) ? 1 : 0;
    total += k;
    before += r < r0 ? k : 0;
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
  for (int w = 0; w < kRowThreads / 32; ++w) {
    before += s_sum[0][w];
    total += s_sum[1][w];
  }
  if (blockIdx.x == 0 && tid == 0) *n_kept = total;
  for (int b = r0; b < r1; b += kRowThreads) {
    const int r = b + tid;
    const bool in = r < r1;
    const bool k = in && counts(r);
    if (in && target && target[r] >= V) report_status(ATTN_EDEVICE_INPUT);
    const unsigned votes = __ballot_sync(0xffffffffu, k);
    if (lane == 0) s_warp[warp] = __popc(votes);
    __syncthreads();
    int at = before, all = 0;
    for (int w = 0; w < kRowThreads / 32; ++w) {
      at += w < warp ? s_warp[w] : 0;
      all += s_warp[w];
    }
    at += __popc(votes & ((1u << lane) - 1u));
    if (in) pos[r] = k ? at : -1;
    if (k) row_of[at] = r;
    before += all;
    __syncthreads();
  }
  if (total == N) return;  // the products read x in place
  // a warp copies a row at a time (its pos entries were written by this block)
  for (int r = r0 + warp; r < r1; r += kRowThreads / 32) {
    const int at = pos[r];
    if (at < 0) continue;
    for (int i = lane; i < c8; i += 32) xc[(size_t)at * c8 + i] = x[(size_t)r * c8 + i];
  }
  const int pad = slot_rows(total);
  for (int r = total + blockIdx.x * (kRowThreads / 32) + warp; r < pad;
       r += gridDim.x * (kRowThreads / 32))
    for (int i = lane; i < c8; i += 32) xc[(size_t)r * c8 + i] = make_uint4(0, 0, 0, 0);
}

// The teacher's list of one row per warp: q = softmax of t / tau over the
// entries present (0 <= id < V), ids sorted ascending with their q (absent
// ones last, id INT_MAX, q 0), sum q log q, and whether the row counts (some
// entry above -inf, and an upstream gradient that is not zero). The sort is by
// rank (K comparisons per entry): stable, so equal ids keep their order. The
// maximum is taken off before the division by tau: entries at the type's
// lowest value then differ by exactly 0.
template <typename TT>
__global__ void __launch_bounds__(32 * kTeacherWarps)
    head_teacher_kernel(const int* __restrict__ t_idx, const TT* __restrict__ t_logit,
                        float inv_tau, const float* __restrict__ dloss,
                        const float* __restrict__ dlse, int* __restrict__ ids,
                        float* __restrict__ share, float* __restrict__ entropy,
                        int* __restrict__ flags, int N, int V, int K) {
  pdl_wait_and_trigger();
  extern __shared__ int smem_teacher[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* key = smem_teacher + warp * K;
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
      for (int i = 0; i < K; ++i) {
        const int other = key[i];
        rank += (other < mine || (other == mine && i < k)) ? 1 : 0;
      }
      ids[(size_t)r * K + rank] = mine;
      share[(size_t)r * K + rank] = q;
    }
    ent = warp_sum(ent);
    if (lane == 0) {
      flags[r] = some && has_weight(dloss, dlse, r) ? 1 : 0;
      if (entropy) entropy[r] = ent;
    }
    __syncwarp();
  }
}

// lse and loss of every row from the parts of its logits: 32 rows per block,
// eight threads per row. loss = sum_k q_k (log q_k + lse - z_k), for a single
// target lse - z.
constexpr int kLossRows = 32, kLossSlices = 8;
__global__ void __launch_bounds__(kLossRows* kLossSlices)
    head_loss_kernel(const float2* __restrict__ part, const float* __restrict__ named,
                     const float* __restrict__ share, const float* __restrict__ entropy,
                     const int* __restrict__ pos, float* __restrict__ loss,
                     float* __restrict__ lse, int N, int K, int parts, int row_pitch) {
  pdl_wait_and_trigger();
  __shared__ float s_m[kLossSlices][kLossRows], s_s[kLossSlices][kLossRows];
  const int tx = threadIdx.x % kLossRows, ty = threadIdx.x / kLossRows;
  const int r = blockIdx.x * kLossRows + tx;
  const int at = r < N ? pos[r] : -1;
  float m = -INFINITY, s = 0.f;
  auto join = [&](float om, float os) {
    const float nm = fmaxf(m, om);
    s = nm > -INFINITY ? s * exp2f(m - nm) + os * exp2f(om - nm) : s + os;
    m = nm;
  };
  if (at >= 0)
    for (int j = ty; j < parts; j += kLossSlices) {
      const float2 t = part[(size_t)j * row_pitch + at];
      join(t.x, t.y);
    }
  s_m[ty][tx] = m;
  s_s[ty][tx] = s;
  __syncthreads();
  for (int j = 0; j < kLossSlices; ++j)
    if (j != ty) join(s_m[j][tx], s_s[j][tx]);
  // every slice now has the row's total (equal up to the order of the sum);
  // slice 0's is the row's lse
  __syncthreads();
  if (ty == 0) s_m[0][tx] = (m + log2f(s)) * kLn2;
  __syncthreads();
  const float l = s_m[0][tx];
  float d = 0.f;
  if (at >= 0)
    for (int k = ty; k < K; k += kLossSlices) {
      const float q = share ? share[(size_t)r * K + k] : 1.f;
      if (q != 0.f) d += q * (l - named[(size_t)at * K + k]);
    }
  s_s[ty][tx] = d;
  __syncthreads();
  if (ty == 0 && r < N) {
    d = 0.f;
    for (int j = 0; j < kLossSlices; ++j) d += s_s[j][tx];
    lse[r] = at >= 0 ? l : 0.f;
    loss[r] = at >= 0 ? (share ? entropy[r] + d : d) : 0.f;
  }
}

// dx of every row: its accumulators added in order and rounded once; zeros
// for a row that was left out. Eight columns per thread.
__global__ void __launch_bounds__(256)
    head_dx_kernel(const float* __restrict__ acc, const int* __restrict__ pos,
                   const int* __restrict__ n_kept, uint4* __restrict__ dx, int N, int C,
                   int kb_total) {
  pdl_wait_and_trigger();
  const int kept = *n_kept;
  int splits, kb_per;
  split_dx(((kept + kTile - 1) / kTile) * ((C + kTile - 1) / kTile), kb_total, splits, kb_per);
  const size_t slot = (size_t)slot_rows(kept) * C;
  const int c8 = C / 8;
  const long n = (long)N * c8;
  for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long)gridDim.x * 256) {
    const int r = (int)(i / c8), c = (int)(i - (long)r * c8) * 8;
    const int at = pos[r];
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (at >= 0) {
      const float* src = acc + (size_t)at * C + c;
      for (int s = 0; s < splits; ++s, src += slot) {
        const float4 a = *reinterpret_cast<const float4*>(src);
        const float4 b = *reinterpret_cast<const float4*>(src + 4);
        v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
        v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
      }
    }
    dx[i] = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                       pack_bf16(v[6], v[7]));
  }
}

}  // namespace head100
