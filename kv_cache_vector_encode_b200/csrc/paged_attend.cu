// Host side of tq_paged_attend, and the kernels before and after the decode steps' main kernel (paged_rows.cuh):
// queries into the rotated domain, partial results together and back.
//
//   out = Pi^T sum_t w_t n_t c_v[idx_t] (+ alpha S^T sum_t w_t n_t gamma_t (2 z_t - 1)),
//   w = softmax of x_t = scale n_t <Pi q, c_k[idx_t]>, capped, biased and masked.
// Nothing is dequantised to memory: the queries are rotated once (prep kernel), scores and value sums are
// formed in the rotated domain from the codes, and Pi^T / S^T are applied once per query row (combine). The
// three kernels are launched as dependents, each setting up while the one before it ends. Sequences with many
// query rows take the chunk kernels instead (paged_chunk.cu).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "paged_attend.h"
#include "sm100.cuh"

namespace tq {
namespace {

// ---- queries into the rotated domain --------------------------------------------------------------------
// q' = Pi q of an item's rows, as 16-bit integers relative to the row's largest coordinate (an error of 2^-16 of
// it), split into signed 8-bit limbs. Pi goes through shared memory (padded rows), so that its loads are wide and all
// in flight at once; thread = (coordinate, part of the sum).
constexpr int kPrepThreads = 512;
template <int D> constexpr size_t prep_smem() { return (size_t)D * (D + 4) * 4; }

template <int D, int RB>
__global__ void __launch_bounds__(kPrepThreads) prep_kernel(const __grid_constant__ PagedAttendParams p) {
  constexpr int PARTS = kPrepThreads / D, J = D / PARTS, PER = RB * D / kPrepThreads > 0 ? RB * D / kPrepThreads : 1;
  extern __shared__ __align__(16) float mat[];                   // [D][D + 4]
  __shared__ __align__(16) float q[RB][D];
  __shared__ float part[PARTS][RB][D];
  __shared__ float red[RB][D / 32];
  __shared__ int isum[RB][D / 32];
  grid_dep_launch();
  constexpr int PI = D * D / 4 / kPrepThreads;                   // the longest way first
  float4 pi[PI];
#pragma unroll
  for (int k = 0; k < PI; ++k) pi[k] = __ldg((const float4*)p.Pi + threadIdx.x + k * kPrepThreads);
  const int item = blockIdx.x, unit = item / p.row_blocks, rb = item - unit * p.row_blocks;
  const int b = unit / p.Hkv, hkv = unit - b * p.Hkv;
  if (threadIdx.x == 0) p.parts[item] = make_int2(0, 0);
  const PagedSeq s = paged_seq(p, b);
  const int row0 = rb * RB, rows = s.qn * p.g;
  if (row0 >= rows || rows > p.chunk_rows) return;
#pragma unroll
  for (int k = 0; k < PI; ++k) {
    const int e = threadIdx.x + k * kPrepThreads;
    *(float4*)&mat[(e / (D / 4)) * (D + 4) + (e % (D / 4)) * 4] = pi[k];
  }
  for (int e = threadIdx.x; e < RB * D; e += kPrepThreads) {
    const int row = row0 + e / D, j = row / p.g;
    q[e / D][e % D] = row < rows ? __uint_as_float((uint32_t)p.q[(int64_t)(s.q0 + j) * p.q_stride +
                                                                (int64_t)(hkv * p.g + row - j * p.g) * D + e % D] << 16) : 0.f;
  }
  __syncthreads();
  {
    const int i = threadIdx.x % D, pt = threadIdx.x / D;
    float acc[RB] = {};
#pragma unroll
    for (int j = 0; j < J; j += 4) {
      const float4 m = *(const float4*)&mat[i * (D + 4) + pt * J + j];
#pragma unroll
      for (int u = 0; u < RB; ++u) {
        const float4 v = *(const float4*)&q[u][pt * J + j];
        acc[u] = fmaf(m.x, v.x, fmaf(m.y, v.y, fmaf(m.z, v.z, fmaf(m.w, v.w, acc[u]))));
      }
    }
#pragma unroll
    for (int u = 0; u < RB; ++u) part[pt][u][i] = acc[u];
  }
  __syncthreads();
  float y[PER];
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int e = threadIdx.x + k * kPrepThreads, u = e / D, i = e % D;
    if (e >= RB * D) break;                                      // whole warps
    y[k] = 0.f;
#pragma unroll
    for (int t = 0; t < PARTS; ++t) y[k] += part[t][u][i];
    // NaN stays: what is not finite makes the whole row NaN below
    float m = fabsf(y[k]);
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const float v = __shfl_xor_sync(0xffffffffu, m, o);
      m = v > m || v != v ? v : m;
    }
    if ((i & 31) == 0) red[u][i >> 5] = m;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int e = threadIdx.x + k * kPrepThreads, u = e / D, i = e % D;
    if (e >= RB * D) break;
    float m = red[u][0];
#pragma unroll
    for (int w = 1; w < D / 32; ++w) m = red[u][w] > m || red[u][w] != red[u][w] ? red[u][w] : m;
    const bool fine = m < INFINITY;
    // the largest coordinate becomes 32512 = 127 * 256, the largest that two signed limbs hold either way; a row below
    // 2^-100 throughout is taken as zero
    const float per = fine && m > 7.8886091e-31f ? 32512.f / m : 0.f;
    const int v = fine ? __float2int_rn(y[k] * per) : 0;
    const int hi = (v + 128) >> 8, lo = v - (hi << 8);
    const int at = D == 128 ? (i >> 5) * 32 + ((i & 3) * 2 + ((i >> 4) & 1)) * 4 + ((i >> 2) & 3)
                            : (i >> 4) * 16 + (i & 3) * 4 + ((i >> 2) & 3);
    int8_t* dst = p.qr + ((int64_t)item * RB + u) * 2 * D + at;
    dst[0] = (int8_t)hi;
    dst[D] = (int8_t)lo;
    const int t = __reduce_add_sync(0xffffffffu, v);
    if ((i & 31) == 0) isum[u][i >> 5] = t;
  }
  __syncthreads();
  if (threadIdx.x < RB) {
    const int u = threadIdx.x;
    float m = red[u][0];
    int t = isum[u][0];
#pragma unroll
    for (int w = 1; w < D / 32; ++w) {
      m = red[u][w] > m || red[u][w] != red[u][w] ? red[u][w] : m;
      t += isum[u][w];
    }
    p.qs[(int64_t)item * RB + u] = make_float2(m < INFINITY ? m * (1.f / 32512.f) : __int_as_float(0x7FC00000), __int_as_float(t >> 1));
  }
}

// ---- partial results together, back to the original domain ---------------------------------------------
// o' = sum of an item's parts, then Pi^T o'_c + alpha S^T o'_z: warp = a run of matrix rows, lane = D / 32 columns. What a
// step waits for is latency, so the matrices are fetched before the partial results are there, and those all at once.
constexpr int kCombThreads = 256, kCombParts = 64;   // threads; parts of a pass where there are many
template <int D, bool ALG2, int RB>
__global__ void __launch_bounds__(kCombThreads) combine_kernel(const __grid_constant__ PagedAttendParams p) {
  constexpr int PD = ALG2 ? 2 * D : D, V = D / 32, W = kCombThreads / 32, J = D / W, PER = RB * PD / kCombThreads, FEW = PER <= 4 ? 8 : 4;   // outputs of a thread; parts fetched at once
  static_assert(PER >= 1 && RB <= W, "one output of a row at least per thread, one warp per row");
  __shared__ float so[RB][PD];
  __shared__ __align__(16) float red[W][RB][D];
  __shared__ float share[RB][kCombParts];                        // weights of a run of parts
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int item = blockIdx.x, unit = item / p.row_blocks, rb = item - unit * p.row_blocks;
  const int b = unit / p.Hkv, hkv = unit - b * p.Hkv;
  const PagedSeq s = paged_seq(p, b);
  const int row0 = rb * RB, rows = s.qn * p.g;
  if (row0 >= rows || rows > p.chunk_rows) {
    grid_dep_wait();
    return;
  }
  using Vec = typename std::conditional<V == 4, float4, float2>::type;
  Vec m[J], ms[ALG2 ? J : 1];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    m[j] = __ldg((const Vec*)(p.Pi + (size_t)(warp * J + j) * D) + lane);
    if (ALG2) ms[j] = __ldg((const Vec*)(p.S + (size_t)(warp * J + j) * D) + lane);
  }
  grid_dep_wait();
  const int2 parts = p.parts[item];
  const bool mine = warp < RB && row0 + warp < rows;             // warp u: the shares of row u's parts, lane = part
  const float2* ml = p.ml + (int64_t)parts.x * RB + warp;
  const float* po = p.po + (int64_t)parts.x * (RB * PD) + threadIdx.x;
  float top = -INFINITY, l = 0.f, o[PER] = {};
  if (parts.y <= FEW) {                                     // all at once
    const float2 x = mine && lane < parts.y ? ml[lane * RB] : make_float2(-INFINITY, 0.f);
    float v[FEW][PER];
#pragma unroll
    for (int k = 0; k < FEW; ++k)
#pragma unroll
      for (int e = 0; e < PER; ++e)
        v[k][e] = k < parts.y && row0 + (int)(threadIdx.x + e * kCombThreads) / PD < rows ? po[(int64_t)k * (RB * PD) + e * kCombThreads] : 0.f;
    if (warp < RB) {
      top = x.x;
#pragma unroll
      for (int i = 16; i; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
      const float f = ex2_approx(x.x - (top == -INFINITY ? 0.f : top));
      l = f * x.y;
#pragma unroll
      for (int i = 16; i; i >>= 1) l += __shfl_xor_sync(0xffffffffu, l, i);
      if (lane < FEW) share[warp][lane] = lane < parts.y ? f * (l == 0.f ? 0.f : 1.f / l) : 0.f;   // NaN stays NaN
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < FEW; ++k)
#pragma unroll
      for (int e = 0; e < PER; ++e)
        if (k < parts.y) o[e] = fmaf(share[(threadIdx.x + e * kCombThreads) / PD][k], v[k][e], o[e]);
  } else {
    if (mine) {
      for (int k = lane; k < parts.y; k += 32) top = fmaxf(top, ml[k * RB].x);
#pragma unroll
      for (int i = 16; i; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
      if (top == -INFINITY) top = 0.f;
      for (int k = lane; k < parts.y; k += 32) l = fmaf(ex2_approx(ml[k * RB].x - top), ml[k * RB].y, l);
#pragma unroll
      for (int i = 16; i; i >>= 1) l += __shfl_xor_sync(0xffffffffu, l, i);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int k0 = 0; k0 < parts.y; k0 += kCombParts) {
      const int n = min(kCombParts, parts.y - k0);
      if (warp < RB)
        for (int k = lane; k < n; k += 32) share[warp][k] = mine ? ex2_approx(ml[(k0 + k) * RB].x - top) * inv : 0.f;
      __syncthreads();
#pragma unroll 8
      for (int k = 0; k < n; ++k) {
#pragma unroll
        for (int e = 0; e < PER; ++e) {
          const int u = (threadIdx.x + e * kCombThreads) / PD;
          if (row0 + u < rows) o[e] = fmaf(share[u][k], po[(int64_t)(k0 + k) * (RB * PD) + e * kCombThreads], o[e]);
        }
      }
      __syncthreads();
    }
  }
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    const int at = threadIdx.x + e * kCombThreads, u = at / PD, i = at % PD;
    so[u][i] = (ALG2 && i >= D ? p.alpha : 1.f) * o[e];
  }
  __syncthreads();
  float acc[RB][V] = {};
  auto rows_times = [&](const Vec* mat, int at) {
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int u = 0; u < RB; ++u) {
        const float o = so[u][at + warp * J + j];
#pragma unroll
        for (int v = 0; v < V; ++v) acc[u][v] = fmaf(reinterpret_cast<const float*>(&mat[j])[v], o, acc[u][v]);
      }
  };
  rows_times(m, 0);
  if (ALG2) rows_times(ms, D);
#pragma unroll
  for (int u = 0; u < RB; ++u)
#pragma unroll
    for (int v = 0; v < V; ++v) red[warp][u][lane * V + v] = acc[u][v];
  __syncthreads();
  for (int e = threadIdx.x; e < RB * D; e += kCombThreads) {
    const int u = e / D, i = e % D, row = row0 + u;
    if (row >= rows) break;
    float o = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) o += red[w][u][i];
    const int j = row / p.g;
    p.out[((int64_t)(s.q0 + j) * p.Hq + hkv * p.g + row - j * p.g) * D + i] = __bfloat16_as_ushort(__float2bfloat16_rn(o));
  }
}

// ---- host -----------------------------------------------------------------------------------------------

struct Plan {
  int row_blocks, rows_per_item, ctas, chunk_rows;
  size_t qr, qs, parts, ml, po, total;
  PagedChunkPlan chunk;
};

Plan plan(const tq_paged_kv* kv, int B, int Hq, int64_t total_q, int max_q, int64_t max_kv, int window) {   // B and max_q > 0
  Plan P{};
  const int g = Hq / kv->Hkv;
  P.chunk_rows = paged_chunk_rows(B * kv->Hkv);
  const bool chunks = (int64_t)max_q * g > P.chunk_rows;
  const int rows = chunks ? P.chunk_rows : max_q * g;
  P.rows_per_item = rows <= 4 ? 4 : 8;                           // one or two column blocks
  P.row_blocks = (rows + P.rows_per_item - 1) / P.rows_per_item;
  P.ctas = 2 * sm_count();                                       // as many as run at a time
  auto al = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t items = (size_t)B * kv->Hkv * P.row_blocks, slots = items + P.ctas, pd = (size_t)kv->d * (kv->v_alg == 2 ? 2 : 1);
  size_t off = 0;
  P.qr = off; off += al(items * P.rows_per_item * kv->d * 2);
  P.qs = off; off += al(items * P.rows_per_item * 8);
  P.parts = off; off += al(items * 8);
  P.ml = off; off += al(slots * P.rows_per_item * 8);
  P.po = off; off += al(slots * P.rows_per_item * pd * 4);
  P.chunk = chunks ? paged_chunk_plan(kv, B, Hq, total_q, max_q, max_kv, window) : PagedChunkPlan{};
  P.chunk.base = off;
  P.total = off + P.chunk.bytes;
  return P;
}

void level_table(const uint16_t* half, int bits, uint32_t (&tab)[4]) {
  for (int i = 0; i < 4; ++i) tab[i] = 0;
  const int n = bits == 4 ? 8 : 1 << bits;
  for (int i = 0; i < n; ++i) {
    const uint16_t h = half[bits == 4 ? 8 + i : i];   // 16 levels: the magnitudes
    tab[i >> 2] |= (uint32_t)(h & 255) << (8 * (i & 3));
    tab[2 + (i >> 2)] |= (uint32_t)(h >> 8) << (8 * (i & 3));
  }
}

// The keys' levels as 16-bit integers c U, in the same form (two's complement: the low bytes count as unsigned, the
// high ones as signed). Of 16 levels the magnitudes, as X of c U = X + 1/2. Returns U.
float limb_table(const float* c, int bits, uint32_t (&tab)[4]) {
  const int L = 1 << bits;
  const float unit = 32000.0f / c[L - 1];
  for (int i = 0; i < 4; ++i) tab[i] = 0;
  const int n = bits == 4 ? 8 : L;
  for (int i = 0; i < n; ++i) {
    const double v = (double)c[bits == 4 ? 8 + i : i] * unit;
    const uint32_t x = (uint32_t)(int32_t)std::lrint(bits == 4 ? v - 0.5 : v);
    tab[i >> 2] |= (x & 255u) << (8 * (i & 3));
    tab[2 + (i >> 2)] |= ((x >> 8) & 255u) << (8 * (i & 3));
  }
  return unit;
}

template <int D, int RB>
tq_status launch_steps(const PagedAttendParams& p, const tq_paged_kv* kv, int items, int ctas, cudaStream_t st) {
  const bool alg2 = kv->v_alg == 2;
  auto prep = prep_kernel<D, RB>;
  cudaError_t e = cudaFuncSetAttribute(prep, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)prep_smem<D>());
  if (e != cudaSuccess) return cuda_fail(e, "tq_paged_attend: shared memory attribute");
  prep<<<items, kPrepThreads, prep_smem<D>(), st>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return cuda_fail(e, "tq_paged_attend: launch");
  const tq_status s = D == 128 ? paged_rows_launch_128(p, kv->k_bits, kv->v_bits, alg2, ctas, st)
                               : paged_rows_launch_64(p, kv->k_bits, kv->v_bits, alg2, ctas, st);
  if (s != TQ_OK) return s;
  e = launch_dependent(alg2 ? combine_kernel<D, true, RB> : combine_kernel<D, false, RB>, dim3(items), kCombThreads, 0, st, p);
  return e == cudaSuccess ? TQ_OK : cuda_fail(e, "tq_paged_attend: launch");
}

tq_status check_sizes(const std::string& f, const tq_paged_kv* kv, int32_t B, int32_t Hq, int64_t total_q,
                      int32_t max_q, int64_t max_kv) {
  if (!paged_ready(kv)) return fail(TQ_ERR_INVALID_ARG, f + ": kv was not filled by tq_paged_kv_init");
  if (B < 0 || total_q < 0 || max_q < 0 || max_kv < 0 || Hq < 1) return fail(TQ_ERR_INVALID_ARG, f + ": negative size");
  if (Hq % kv->Hkv || Hq / kv->Hkv > 128) return fail(TQ_ERR_UNSUPPORTED, f + ": Hq must be a multiple of Hkv, at most 128 times it");
  if (B > 65535 || (int64_t)B * kv->Hkv > 65535) return fail(TQ_ERR_UNSUPPORTED, f + ": B Hkv must be at most 65535");
  if (max_kv > ((int64_t)1 << 31) - 1024) return fail(TQ_ERR_UNSUPPORTED, f + ": max_kv_len too large");
  if (total_q > ((int64_t)1 << 31) - 1024 || total_q * Hq > ((int64_t)1 << 33))
    return fail(TQ_ERR_UNSUPPORTED, f + ": too many query rows for one call");
  if ((int64_t)max_q * (Hq / kv->Hkv) > 65535LL * 256)
    return fail(TQ_ERR_UNSUPPORTED, f + ": max_q_len too large for one call");
  return TQ_OK;
}

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" TQ_API size_t tq_paged_attend_workspace_bytes(const tq_paged_kv* kv, int32_t B, int32_t Hq, int64_t total_q,
                                                         int32_t max_q_len, int64_t max_kv_len) {
  if (check_sizes("tq_paged_attend_workspace_bytes", kv, B, Hq, total_q, max_q_len, max_kv_len) != TQ_OK) return 0;
  if (B == 0 || total_q == 0 || max_q_len == 0) return 0;
  return plan(kv, B, Hq, total_q, max_q_len, max_kv_len, 0).total;
}

extern "C" TQ_API tq_status tq_paged_attend(const tq_paged_kv* kv, int32_t B, int32_t Hq, int64_t total_q,
                                            int32_t max_q_len, int64_t max_kv_len, const void* q, int64_t q_token_stride,
                                            int32_t q_dtype, const int32_t* q_start, const int32_t* kv_len,
                                            const int32_t* page_table, int32_t max_pages, float scale, float softcap,
                                            int32_t window, const int32_t* prefix_len, const float* slopes,
                                            const void* rot, void* out, void* ws, size_t ws_bytes, void* stream) {
  clear_error();
  const std::string f = "tq_paged_attend";
  tq_status s = check_sizes(f, kv, B, Hq, total_q, max_q_len, max_kv_len);
  if (s != TQ_OK) return s;
  const bool work = B > 0 && total_q > 0 && max_q_len > 0;
  if (work && (!q || !q_start || !kv_len || (!page_table && max_pages > 0) || !rot || !out)) return fail(TQ_ERR_INVALID_ARG, f + ": NULL pointer");
  if (q_dtype != TQ_BF16) return fail(TQ_ERR_UNSUPPORTED, f + ": q must be TQ_BF16");
  if (max_pages < 0 || window < 0) return fail(TQ_ERR_INVALID_ARG, f + ": negative max_pages or window");
  if (!(softcap == 0.0f || softcap >= 1e-30f) || std::isinf(softcap))
    return fail(TQ_ERR_INVALID_ARG, f + ": softcap must be finite, and 0 (none) or at least 1e-30");
  if (std::isinf(scale)) return fail(TQ_ERR_INVALID_ARG, f + ": scale must be finite");
  if (q_token_stride < (int64_t)Hq * kv->d) return fail(TQ_ERR_INVALID_ARG, f + ": q_token_stride < Hq d");
  if (!aligned16(q) || !aligned16(out) || !aligned16(rot) || !aligned16(ws) || q_token_stride % 8)
    return fail(TQ_ERR_INVALID_ARG, f + ": pointers and query rows must be 16-byte aligned");
  if (((uintptr_t)q_start | (uintptr_t)kv_len | (uintptr_t)page_table | (uintptr_t)prefix_len | (uintptr_t)slopes) & 3)
    return fail(TQ_ERR_INVALID_ARG, f + ": int32 / fp32 arrays must be 4-byte aligned");
  if (!work) return TQ_OK;
  const int g = Hq / kv->Hkv;
  const Plan P = plan(kv, B, Hq, total_q, max_q_len, max_kv_len, prefix_len ? 0 : window);
  if (!ws || ws_bytes < tq_paged_attend_workspace_bytes(kv, B, Hq, total_q, max_q_len, max_kv_len))
    return fail(TQ_ERR_WORKSPACE, f + ": workspace too small");
  if (!(scale > 0.0f)) scale = (float)(1.0 / std::sqrt((double)kv->d));
  PagedAttendParams p{};
  p.k_codes = kv->k_codes;
  p.k_norms = kv->k_norms;
  p.v_codes = kv->v_codes;
  p.v_signs = kv->v_signs;
  p.v_norms = kv->v_norms;
  p.v_gammas = kv->v_gammas;
  p.num_pages = kv->num_pages;
  p.total_q = total_q;
  p.max_kv = max_kv_len;
  p.q_stride = q_token_stride;
  p.page_shift = __builtin_ctz((unsigned)kv->page_size);
  p.Hkv = kv->Hkv;
  p.Hq = Hq;
  p.g = g;
  p.B = B;
  p.max_pages = max_pages;
  p.max_q = max_q_len;
  p.window = window;
  p.q_start = q_start;
  p.kv_len = kv_len;
  p.table = page_table;
  p.prefix = prefix_len;
  p.slopes = slopes;
  p.q = (const uint16_t*)q;
  p.out = (uint16_t*)out;
  p.scale_log2 = scale * kLog2e;
  p.key_fac = p.scale_log2 * 256.0f / limb_table(kv->ck, kv->k_bits, p.klimb);
  if (softcap >= 1.2676506e30f) softcap = 0.0f;   // 2^100: it would change no score below 2^88 by as much as a rounding
  p.cap_log2 = softcap * kLog2e;
  p.cap2x = softcap > 0.0f ? 2.0f / softcap : 0.0f;   // x arrives times log2(e), as exp2 wants it
  p.v_inv_unit = 1.0f / kv->v_unit;
  p.alpha = (float)(std::sqrt(std::acos(-1.0) / 2.0) / kv->d);
  p.k_inv_unit = 1.0f / kv->k_unit;
  p.sign_unit = p.alpha * kv->v_unit;
  level_table(kv->k_half, kv->k_bits, p.ktab);
  level_table(kv->v_half, kv->v_bits, p.vtab);
  const RotLayout RL = rot_layout(kv->d);
  const uint8_t* base = (const uint8_t*)rot;
  p.Pi = (const float*)(base + RL.pi32);
  p.S = (const float*)(base + RL.s32);
  const size_t img[6] = {RL.pi_hi, RL.pi_lo, RL.pit_hi, RL.pit_lo, RL.st_hi, RL.st_lo};
  for (int i = 0; i < 6; ++i) p.img[i] = base + img[i];
  uint8_t* w = (uint8_t*)ws;
  p.qr = (int8_t*)(w + P.qr);
  p.qs = (float2*)(w + P.qs);
  p.parts = (int2*)(w + P.parts);
  p.ml = (float2*)(w + P.ml);
  p.po = (float*)(w + P.po);
  p.row_blocks = P.row_blocks;
  p.rows_per_item = P.rows_per_item;
  p.chunk_rows = P.chunk_rows;
  p.err = device_error_word();
  if (!p.err) return fail(TQ_ERR_CUDA, f + ": no device error word (is a CUDA device present?)");
  cudaStream_t st = (cudaStream_t)stream;
  if (P.chunk.slots) {
    s = paged_chunk_launch(p, kv, P.chunk, w + P.chunk.base, st);
    if (s != TQ_OK) return s;
  }
  const int items = B * kv->Hkv * P.row_blocks;
  if (kv->d == 128)
    return P.rows_per_item == 4 ? launch_steps<128, 4>(p, kv, items, P.ctas, st) : launch_steps<128, 8>(p, kv, items, P.ctas, st);
  return P.rows_per_item == 4 ? launch_steps<64, 4>(p, kv, items, P.ctas, st) : launch_steps<64, 8>(p, kv, items, P.ctas, st);
}
