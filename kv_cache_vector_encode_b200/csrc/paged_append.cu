// Append of new keys and values to the paged packed cache (tq_paged_append).
//
// Per vector: the key is turned to its position (rope.cu's formula, unrounded), then
//   n = |x|, y = Pi x / n, idx_i = #{k : t_k < y_i}                      (Algorithm 1)
//   r = x / n - Pi^T c[idx], gamma = |r|, z_i = [(S r)_i >= 0]             (Algorithm 2, values)
// and the record goes to the token's slot.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <string>

#include "sm100.cuh"
#include "tq_internal.h"

namespace tq {
namespace {

struct AppendParams {
  int64_t tokens, n_pos, slots_total, k_stride, v_stride;
  int Hkv, page_shift, half, pairs, f32;
  const void* k;
  const void* v;
  const int64_t* slots;
  const int32_t* positions;
  const float2* table;
  const float* Pi;
  const float* S;
  uint32_t* k_codes;
  uint16_t* k_norms;
  uint32_t* v_codes;
  uint32_t* v_signs;
  uint16_t* v_norms;
  uint16_t* v_gammas;
  int kb, vb;
  float ck[16], tk[16], cv[16], tv[16];
  uint32_t* err;
};

// A token's slot and position, checked; slot < 0 where nothing is to be written.
__device__ __forceinline__ int64_t append_slot(const AppendParams& p, int64_t t, int32_t& pos) {
  const int64_t slot = p.slots[t];
  pos = p.half ? p.positions[t] : 0;
  if (slot < 0) return -1;
  if (slot >= p.slots_total || (p.half && (pos < 0 || pos >= p.n_pos))) {
    atomicCAS(p.err, 0u, (uint32_t)kDevBadInput);
    return -1;
  }
  return slot;
}

// Few tokens: everything in fp64 on the SIMT cores, one thread per coordinate and VPB vectors per block.
// Three dependent passes over a d x d matrix (one for keys); with a few vectors per SM their latency is
// the time, whatever the arithmetic.
constexpr int kVpb = 4;

template <int D>
__device__ __forceinline__ void block_sum(double (&v)[kVpb], double (*red)[D / 32]) {
#pragma unroll
  for (int u = 0; u < kVpb; ++u) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v[u] += __shfl_xor_sync(0xffffffffu, v[u], o);
    if ((threadIdx.x & 31) == 0) red[u][threadIdx.x >> 5] = v[u];
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kVpb; ++u) {
    v[u] = 0.0;
#pragma unroll
    for (int w = 0; w < D / 32; ++w) v[u] += red[u][w];
  }
  __syncthreads();
}

template <int D>
__global__ void __launch_bounds__(D) append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int G = D / 32;
  __shared__ double sv[kVpb][D];
  __shared__ double red[kVpb][G];
  const bool value = blockIdx.y == 1;
  const bool alg2 = value && p.v_signs;
  const int i = threadIdx.x, g = i >> 5, lane = i & 31;
  const int64_t v0 = (int64_t)blockIdx.x * kVpb, nv = p.tokens * p.Hkv;
  int64_t rec[kVpb];
  double x[kVpb], n[kVpb];
#pragma unroll
  for (int u = 0; u < kVpb; ++u) {
    rec[u] = -1;
    x[u] = 0.0;
    if (v0 + u >= nv) continue;
    const int64_t t = (v0 + u) / p.Hkv;
    const int h = (int)((v0 + u) - t * p.Hkv);
    int32_t pos;
    const int64_t slot = append_slot(p, t, pos);
    if (slot < 0) continue;
    rec[u] = (((slot >> p.page_shift) * p.Hkv + h) << p.page_shift) + (slot & ((1 << p.page_shift) - 1));
    const int64_t at = t * (value ? p.v_stride : p.k_stride) + (int64_t)h * D;
    const void* src = value ? p.v : p.k;
    auto elem = [&](int e) -> double {
      return p.f32 ? (double)((const float*)src)[at + e] : (double)__uint_as_float((uint32_t)((const uint16_t*)src)[at + e] << 16);
    };
    x[u] = elem(i);
    if (!value && i < 2 * p.half) {
      const int pair = p.pairs ? i >> 1 : (i < p.half ? i : i - p.half);
      const bool second = p.pairs ? i & 1 : i >= p.half;
      const float2 cs = p.table[(int64_t)pos * p.half + pair];
      const double o = elem(p.pairs ? i ^ 1 : (second ? i - p.half : i + p.half));
      x[u] = second ? x[u] * cs.x + o * cs.y : x[u] * cs.x - o * cs.y;
    }
  }
#pragma unroll
  for (int u = 0; u < kVpb; ++u) n[u] = x[u] * x[u];
  block_sum<D>(n, red);
  bool ok[kVpb];
#pragma unroll
  for (int u = 0; u < kVpb; ++u) {
    n[u] = sqrt(n[u]);
    ok[u] = n[u] > 0.0 && n[u] <= 1.7976931348623157e308;
    x[u] = ok[u] ? x[u] / n[u] : 0.0;
    sv[u][i] = x[u];
  }
  __syncthreads();
  // acc[u] = sum_j M[i][j] sv[u][j]
  auto rows_product = [&](const float* M, double (&acc)[kVpb]) {
    const float4* row = (const float4*)(M + (size_t)i * D);
#pragma unroll 4
    for (int j = 0; j < D / 4; ++j) {
      const float4 m = __ldg(row + j);
#pragma unroll
      for (int u = 0; u < kVpb; ++u) {
        acc[u] = fma((double)m.x, sv[u][4 * j], acc[u]);
        acc[u] = fma((double)m.y, sv[u][4 * j + 1], acc[u]);
        acc[u] = fma((double)m.z, sv[u][4 * j + 2], acc[u]);
        acc[u] = fma((double)m.w, sv[u][4 * j + 3], acc[u]);
      }
    }
  };
  double y[kVpb] = {};
  rows_product(p.Pi, y);
  __syncthreads();
  const int bits = value ? p.vb : p.kb, L = 1 << bits;
  const float* tab = value ? p.tv : p.tk;
  uint32_t* codes = value ? p.v_codes : p.k_codes;
  uint16_t* norms = value ? p.v_norms : p.k_norms;
#pragma unroll
  for (int u = 0; u < kVpb; ++u) {
    int idx = 0;
    for (int k = 0; k < L - 1; ++k) idx += (double)tab[k] < y[u] ? 1 : 0;
    for (int b = 0; b < bits; ++b) {
      const uint32_t w = __ballot_sync(0xffffffffu, (idx >> b) & 1);
      if (lane == 0 && rec[u] >= 0) codes[(rec[u] * G + g) * bits + b] = w;
    }
    if (i == 0 && rec[u] >= 0) norms[rec[u]] = __half_as_ushort(__double2half(n[u]));
    if (alg2) sv[u][i] = (double)p.cv[idx];
  }
  if (!alg2) return;
  __syncthreads();
  double a[kVpb] = {};
#pragma unroll 4
  for (int j = 0; j < D; ++j) {
    const double m = (double)__ldg(p.Pi + (size_t)j * D + i);
#pragma unroll
    for (int u = 0; u < kVpb; ++u) a[u] = fma(m, sv[u][j], a[u]);
  }
  __syncthreads();
  double ga[kVpb];
#pragma unroll
  for (int u = 0; u < kVpb; ++u) {
    const double r = ok[u] ? x[u] - a[u] : 0.0;
    sv[u][i] = r;
    ga[u] = r * r;
  }
  block_sum<D>(ga, red);
  double s[kVpb] = {};
  rows_product(p.S, s);
#pragma unroll
  for (int u = 0; u < kVpb; ++u) {
    const uint32_t w = __ballot_sync(0xffffffffu, s[u] >= 0.0);
    if (rec[u] < 0) continue;
    if (lane == 0) p.v_signs[rec[u] * G + g] = w;
    if (i == 0) p.v_gammas[rec[u]] = __half_as_ushort(__double2half(sqrt(ga[u])));
  }
}

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" TQ_API tq_status tq_paged_append(const tq_paged_kv* kv, int64_t tokens, const void* k_new,
                                            int64_t k_token_stride, const void* v_new, int64_t v_token_stride,
                                            int32_t x_dtype, const int64_t* slots, const int32_t* positions,
                                            const float* table, int64_t n_pos, int32_t rot_dim, int32_t layout,
                                            const void* rot, void* stream) {
  clear_error();
  const std::string f = "tq_paged_append";
  if (!paged_ready(kv)) return fail(TQ_ERR_INVALID_ARG, f + ": kv was not filled by tq_paged_kv_init");
  if (tokens < 0 || n_pos < 0) return fail(TQ_ERR_INVALID_ARG, f + ": negative size");
  if (x_dtype != TQ_F32 && x_dtype != TQ_BF16) return fail(TQ_ERR_UNSUPPORTED, f + ": x_dtype must be TQ_F32 or TQ_BF16");
  if (rot_dim < 0 || rot_dim > kv->d || rot_dim % 2) return fail(TQ_ERR_UNSUPPORTED, f + ": rot_dim must be even, 0..d");
  if (layout != TQ_ROPE_HALF && layout != TQ_ROPE_PAIRS) return fail(TQ_ERR_INVALID_ARG, f + ": unknown layout");
  if (tokens > 0 && (!k_new || !v_new || !slots || !rot || (rot_dim && (!positions || !table))))
    return fail(TQ_ERR_INVALID_ARG, f + ": NULL pointer");
  const int64_t row = (int64_t)kv->Hkv * kv->d, unit = x_dtype == TQ_F32 ? 4 : 8;
  if (k_token_stride < row || v_token_stride < row) return fail(TQ_ERR_INVALID_ARG, f + ": token stride < Hkv d");
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(rot) || k_token_stride % unit || v_token_stride % unit)
    return fail(TQ_ERR_INVALID_ARG, f + ": rows of k_new and v_new must be 16-byte aligned");
  if ((uintptr_t)slots % 8 || (uintptr_t)positions % 4 || (uintptr_t)table % 8)
    return fail(TQ_ERR_INVALID_ARG, f + ": slots and table must be 8-byte aligned, positions 4-byte");
  if (tokens > ((int64_t)1 << 31) / kv->Hkv - 1024) return fail(TQ_ERR_UNSUPPORTED, f + ": tokens Hkv >= 2^31");
  if (tokens == 0) return TQ_OK;
  const RotLayout RL = rot_layout(kv->d);
  AppendParams p{};
  p.tokens = tokens;
  p.n_pos = n_pos;
  p.page_shift = __builtin_ctz((unsigned)kv->page_size);
  p.slots_total = kv->num_pages << p.page_shift;
  p.k_stride = k_token_stride;
  p.v_stride = v_token_stride;
  p.Hkv = kv->Hkv;
  p.half = rot_dim / 2;
  p.pairs = layout == TQ_ROPE_PAIRS;
  p.f32 = x_dtype == TQ_F32;
  p.k = k_new;
  p.v = v_new;
  p.slots = slots;
  p.positions = positions;
  p.table = (const float2*)table;
  p.Pi = (const float*)((const uint8_t*)rot + RL.pi32);
  p.S = (const float*)((const uint8_t*)rot + RL.s32);
  p.k_codes = kv->k_codes;
  p.k_norms = kv->k_norms;
  p.v_codes = kv->v_codes;
  p.v_signs = kv->v_signs;
  p.v_norms = kv->v_norms;
  p.v_gammas = kv->v_gammas;
  p.kb = kv->k_bits;
  p.vb = kv->v_bits;
  for (int k = 0; k < 16; ++k) {
    p.ck[k] = kv->ck[k];
    p.tk[k] = kv->tk[k];
    p.cv[k] = kv->cv[k];
    p.tv[k] = kv->tv[k];
  }
  p.err = device_error_word();
  if (!p.err) return fail(TQ_ERR_CUDA, f + ": no device error word (is a CUDA device present?)");
  const dim3 grid((unsigned)((tokens * kv->Hkv + kVpb - 1) / kVpb), 2);
  if (kv->d == 128)
    append_kernel<128><<<grid, 128, 0, (cudaStream_t)stream>>>(p);
  else
    append_kernel<64><<<grid, 64, 0, (cudaStream_t)stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? TQ_OK : cuda_fail(e, "tq_paged_append: launch");
}
