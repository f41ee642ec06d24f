// Rotary positions (tq_rope_table, tq_rope).
//
// Pair i of a head at position p turns by p f_i: (a, b) -> (a c - b s, b c + a s) with (c, s) from a
// table [positions][rot/2][2] made once in fp64. The operator moves every element once in and once
// out and does three flops for each, so HBM bounds it; the table row of a token is shared by its heads.
//
// A unit of work is a run of pairs of one token, kept with its (c, s) in registers while it goes over
// several heads: the row is then read once per unit instead of once per head. With few tokens the
// heads are spread over more units (down to one head each), so that the loads of a decode step are
// all in flight at once.
//
// Measured, the kernel alone (40 calls in a captured graph): 8192 tokens x 40 heads x 128 in bf16 31.8 us (5.4 TB/s, 0.82 of
// the copy rate), 4099 x 32 x 64 in fp32 with 48 coordinates turned in pairs 17.4 us (3.9 TB/s), 64 tokens x 40 heads
// 2.4 us. A call among others, the host's time included, takes 34.4, 19.9 and 7.8.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "sm100.cuh"
#include "tq_internal.h"

namespace tq {
namespace {

struct TableParams {
  int64_t n_pos;
  int half, scaling;
  double base, factor, low, high, original, magnitude;
  float2* table;
};

__global__ void table_kernel(TableParams p) {
  const int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (e >= p.n_pos * p.half) return;
  const int64_t pos = e / p.half;
  const int i = (int)(e - pos * p.half);
  double f = pow(p.base, -(double)i / p.half);
  if (p.scaling == TQ_ROPE_LINEAR) f /= p.factor;
  if (p.scaling == TQ_ROPE_BLEND) {
    const double turns = p.original * f / (2.0 * M_PI);
    const double keep = fmin(1.0, fmax(0.0, (turns - p.low) / (p.high - p.low)));
    f = keep * f + (1.0 - keep) * (f / p.factor);
  }
  double s, c;
  sincos((double)pos * f, &s, &c);
  p.table[e] = make_float2((float)(c * p.magnitude), (float)(s * p.magnitude));
}

template <typename T> struct Elem;
template <> struct Elem<float> {
  static __device__ float get(float v) { return v; }
  static __device__ float put(float v) { return v; }
};
template <> struct Elem<__half> {
  static __device__ float get(__half v) { return __half2float(v); }
  static __device__ __half put(float v) { return __float2half_rn(v); }
};
template <> struct Elem<__nv_bfloat16> {
  static __device__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};

template <typename T, int N> struct alignas(sizeof(T) * N) Pack { T v[N]; };

struct RopeParams {
  int64_t tokens, units;             // units: tokens * splits * runs
  int heads, half, rest0, splits, runs, turn_runs;
  float sign;
  const void* x;
  void* out;
  int64_t xt, xh, ot, oh, n_pos;
  const int32_t* positions;
  const float2* table;
  uint32_t* err;
};

// NV elements per access (16 bytes, or one); a run is NV pairs in the half layout, NV / 2 (at least one) in
// the pair layout. Runs from turn_runs on are the untouched rest of the head (none when in place).
template <typename T, int NV, bool HALF>
__global__ void __launch_bounds__(256) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int NP = HALF ? NV : (NV > 1 ? NV / 2 : 1);      // pairs per run
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= p.units) return;
  const int run = (int)(id % p.runs);
  const int64_t rem = id / p.runs;
  const int split = (int)(rem % p.splits);
  const int64_t t = rem / p.splits;
  const int32_t pos = p.positions[t];
  if (pos < 0) return;
  if (pos >= p.n_pos) {
    report_bad_input(p.err);
    return;
  }
  const T* x = (const T*)p.x + t * p.xt;
  T* out = (T*)p.out + t * p.ot;
  if (run >= p.turn_runs) {
    using V = Pack<T, NV>;
    const int at = p.rest0 + (run - p.turn_runs) * NV;
    for (int h = split; h < p.heads; h += p.splits) *(V*)(out + h * p.oh + at) = *(const V*)(x + h * p.xh + at);
    return;
  }
  float c[NP], s[NP];
  const float2* row = p.table + (int64_t)pos * p.half + run * NP;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const float2 cs = __ldg(row + i);
    c[i] = cs.x;
    s[i] = cs.y * p.sign;
  }
  if constexpr (HALF) {
    using V = Pack<T, NV>;
    const int at = run * NV;
#pragma unroll 4
    for (int h = split; h < p.heads; h += p.splits) {
      V a = *(const V*)(x + h * p.xh + at), b = *(const V*)(x + h * p.xh + p.half + at);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const float u = Elem<T>::get(a.v[i]), w = Elem<T>::get(b.v[i]);
        a.v[i] = Elem<T>::put(u * c[i] - w * s[i]);
        b.v[i] = Elem<T>::put(w * c[i] + u * s[i]);
      }
      *(V*)(out + h * p.oh + at) = a;
      *(V*)(out + h * p.oh + p.half + at) = b;
    }
  } else {
    // NV = 1: the two elements of the pair one by one (a pair need not be aligned to its size)
    using V = Pack<T, NV>;
    constexpr int NA = 2 * NP / NV;                        // accesses per run
    const int at = run * 2 * NP;
#pragma unroll 4
    for (int h = split; h < p.heads; h += p.splits) {
      T v[2 * NP];
#pragma unroll
      for (int a = 0; a < NA; ++a) *(V*)(v + a * NV) = *(const V*)(x + h * p.xh + at + a * NV);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const float u = Elem<T>::get(v[2 * i]), w = Elem<T>::get(v[2 * i + 1]);
        v[2 * i] = Elem<T>::put(u * c[i] - w * s[i]);
        v[2 * i + 1] = Elem<T>::put(w * c[i] + u * s[i]);
      }
#pragma unroll
      for (int a = 0; a < NA; ++a) *(V*)(out + h * p.oh + at + a * NV) = *(const V*)(v + a * NV);
    }
  }
}

template <typename T>
tq_status launch_rope(RopeParams& p, int d, bool half_layout, bool in_place, cudaStream_t st) {
  constexpr int NV = 16 / sizeof(T);
  const int rot = 2 * p.half;
  bool vec = aligned16(p.x) && aligned16(p.out) && p.xt % NV == 0 && p.xh % NV == 0 && p.ot % NV == 0 && p.oh % NV == 0 &&
             d % NV == 0 && rot % NV == 0 && (!half_layout || p.half % NV == 0);
  const int nv = vec ? NV : 1;
  const int np = half_layout ? nv : (nv > 1 ? nv / 2 : 1);
  p.turn_runs = p.half / np;
  p.rest0 = rot;
  p.runs = p.turn_runs + (in_place ? 0 : (d - rot) / nv);
  // as many units as eight blocks of 256 per SM hold, not more: each reads its part of the table once. The fp32 pair
  // kernel (32 registers) runs so many at a time; the others run five (16-bit half layout, 48 registers) or six (40), so
  // that there a prompt's blocks take a second, shorter wave (8192 tokens x 40 heads in bf16: 1024 blocks in 740 places)
  const int64_t want = (int64_t)sm_count() * 8 * 256, fit = want / (p.tokens * p.runs);
  const int splits = (int)(fit < 1 ? 1 : fit < p.heads ? fit : p.heads);
  const int each = (p.heads + splits - 1) / splits;              // heads of a unit
  p.splits = (p.heads + each - 1) / each;
  p.units = p.tokens * p.splits * p.runs;
  const int64_t grid = (p.units + 255) / 256;
  if (grid > 2147483647LL) return fail(TQ_ERR_UNSUPPORTED, "tq_rope: too many elements for one call");
  if (vec && half_layout)
    rope_kernel<T, NV, true><<<(unsigned)grid, 256, 0, st>>>(p);
  else if (vec)
    rope_kernel<T, NV, false><<<(unsigned)grid, 256, 0, st>>>(p);
  else if (half_layout)
    rope_kernel<T, 1, true><<<(unsigned)grid, 256, 0, st>>>(p);
  else
    rope_kernel<T, 1, false><<<(unsigned)grid, 256, 0, st>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? TQ_OK : cuda_fail(e, "tq_rope: launch");
}

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" TQ_API tq_status tq_rope_table(int64_t n_pos, int32_t rot_dim, double base, int32_t scaling, double factor,
                                          double low_turns, double high_turns, double original_len, double magnitude,
                                          float* table, void* stream) {
  clear_error();
  const std::string f = "tq_rope_table";
  if (n_pos < 0 || (n_pos > 0 && !table)) return fail(TQ_ERR_INVALID_ARG, f + ": n_pos < 0 or table NULL");
  if (rot_dim < 2 || rot_dim > 512 || rot_dim % 2) return fail(TQ_ERR_UNSUPPORTED, f + ": rot_dim must be even, 2..512");
  if (!(base > 0.0) || !std::isfinite(base) || !std::isfinite(magnitude))
    return fail(TQ_ERR_INVALID_ARG, f + ": base must be > 0, magnitude finite");
  if (scaling != TQ_ROPE_PLAIN && scaling != TQ_ROPE_LINEAR && scaling != TQ_ROPE_BLEND)
    return fail(TQ_ERR_INVALID_ARG, f + ": unknown scaling");
  if (scaling != TQ_ROPE_PLAIN && (!(factor > 0.0) || !std::isfinite(factor)))
    return fail(TQ_ERR_INVALID_ARG, f + ": factor must be > 0");
  if (scaling == TQ_ROPE_BLEND && (!(low_turns >= 0.0) || !(high_turns > low_turns) || !std::isfinite(high_turns) ||
                                   !(original_len > 0.0) || !std::isfinite(original_len)))
    return fail(TQ_ERR_INVALID_ARG, f + ": need 0 <= low_turns < high_turns and original_len > 0");
  if (n_pos > ((int64_t)1 << 31) - 1) return fail(TQ_ERR_UNSUPPORTED, f + ": n_pos >= 2^31");
  if ((uintptr_t)table % 8) return fail(TQ_ERR_INVALID_ARG, f + ": table must be 8-byte aligned");
  if (n_pos == 0) return TQ_OK;
  const int half = rot_dim / 2;
  TableParams p{n_pos, half, scaling, base, factor, low_turns, high_turns, original_len, magnitude, (float2*)table};
  const int64_t grid = (n_pos * half + 255) / 256;
  if (grid > 2147483647LL) return fail(TQ_ERR_UNSUPPORTED, f + ": table too large for one call");
  table_kernel<<<(unsigned)grid, 256, 0, (cudaStream_t)stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? TQ_OK : cuda_fail(e, "tq_rope_table: launch");
}

extern "C" TQ_API tq_status tq_rope(int64_t tokens, int32_t heads, int32_t d, int32_t rot_dim, int32_t layout,
                                    int32_t inverse, const void* x, int64_t x_token_stride, int64_t x_head_stride,
                                    int32_t dtype, const int32_t* positions, const float* table, int64_t n_pos,
                                    void* out, int64_t out_token_stride, int64_t out_head_stride, void* stream) {
  clear_error();
  const std::string f = "tq_rope";
  if (tokens < 0 || heads < 1 || n_pos < 0) return fail(TQ_ERR_INVALID_ARG, f + ": negative size");
  if (tokens > 0 && (!x || !out || !positions || (!table && n_pos > 0))) return fail(TQ_ERR_INVALID_ARG, f + ": NULL pointer");
  if (d < 2 || d > 4096) return fail(TQ_ERR_UNSUPPORTED, f + ": d must be in 2..4096");
  if (rot_dim < 2 || rot_dim > 512 || rot_dim > d || rot_dim % 2)
    return fail(TQ_ERR_UNSUPPORTED, f + ": rot_dim must be even, 2..min(d, 512)");
  if (layout != TQ_ROPE_HALF && layout != TQ_ROPE_PAIRS) return fail(TQ_ERR_INVALID_ARG, f + ": unknown layout");
  if (dtype != TQ_F32 && dtype != TQ_BF16 && dtype != TQ_F16) return fail(TQ_ERR_UNSUPPORTED, f + ": dtype");
  const uintptr_t es = dtype == TQ_F32 ? 4 : 2;
  if ((uintptr_t)x % es || (uintptr_t)out % es || (uintptr_t)positions % 4 || (uintptr_t)table % 8)
    return fail(TQ_ERR_INVALID_ARG, f + ": pointers must be aligned to their elements (table to 8 bytes)");
  if (x_token_stride < 0 || x_head_stride < 0) return fail(TQ_ERR_INVALID_ARG, f + ": negative stride");
  // every output element has one writer: heads must not overlap within a token, nor tokens each other. The stride of an
  // axis of length one has no meaning
  auto apart = [](int64_t inner, int64_t n, int64_t outer, int64_t len) {
    return inner >= len && outer >= (__int128)inner * (n - 1) + len;
  };
  const int64_t ot = tokens > 1 ? out_token_stride : INT64_MAX, oh = heads > 1 ? out_head_stride : INT64_MAX;
  if (out_head_stride < 0 || out_token_stride < 0 ||
      !(ot < oh ? apart(ot, tokens, oh, d) : (oh == INT64_MAX || apart(oh, heads, ot, d))))
    return fail(TQ_ERR_INVALID_ARG, f + ": output strides must keep heads and tokens apart");
  if (x == out && ((tokens > 1 && x_token_stride != out_token_stride) || (heads > 1 && x_head_stride != out_head_stride)))
    return fail(TQ_ERR_INVALID_ARG, f + ": in place needs the same strides");
  if (tokens == 0) return TQ_OK;
  if (tokens > ((int64_t)1 << 31) - 1 || heads > (1 << 20)) return fail(TQ_ERR_UNSUPPORTED, f + ": tokens or heads too many");
  RopeParams p{};
  p.tokens = tokens;
  p.heads = heads;
  p.half = rot_dim / 2;
  p.sign = inverse ? -1.0f : 1.0f;
  p.x = x;
  p.out = out;
  p.xt = x_token_stride;
  p.xh = x_head_stride;
  p.ot = out_token_stride;
  p.oh = out_head_stride;
  p.n_pos = n_pos;
  p.positions = positions;
  p.table = (const float2*)table;
  p.err = device_error_word();
  if (!p.err) return fail(TQ_ERR_CUDA, f + ": no device error word (is a CUDA device present?)");
  cudaStream_t st = (cudaStream_t)stream;
  const bool half_layout = layout == TQ_ROPE_HALF, in_place = x == out;
  switch (dtype) {
    case TQ_F32: return launch_rope<float>(p, d, half_layout, in_place, st);
    case TQ_BF16: return launch_rope<__nv_bfloat16>(p, d, half_layout, in_place, st);
    default: return launch_rope<__half>(p, d, half_layout, in_place, st);
  }
}
