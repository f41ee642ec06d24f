// Shared by the kernels of tq_paged_attend: the call's parameters and what a query row may see.
#pragma once
#include <cstdint>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "sm100.cuh"

#include "tq_internal.h"

namespace tq {

constexpr float kLog2e = 1.4426950408889634f;

struct PagedAttendParams {
  const uint32_t* k_codes;
  const uint16_t* k_norms;
  const uint32_t* v_codes;
  const uint32_t* v_signs;
  const uint16_t* v_norms;
  const uint16_t* v_gammas;
  int64_t num_pages, total_q, max_kv, q_stride;
  int page_shift, Hkv, Hq, g, B, max_pages, max_q, window;
  const int32_t* q_start;
  const int32_t* kv_len;
  const int32_t* table;
  const int32_t* prefix;
  const float* slopes;
  const uint16_t* q;           // bf16
  uint16_t* out;               // bf16
  float scale_log2;            // scale log2(e)
  float key_fac;               // scale_log2 times what a unit of the integer scores (over 256) is worth
  float cap2x, cap_log2;       // 2 / cap, cap log2(e) (cap = 0: none)
  float v_inv_unit, alpha;
  float k_inv_unit, sign_unit; // chunk kernels: sign_unit = alpha times the values' unit
  // level tables for byte permutes (low bytes of levels 0-3, 4-7, high bytes): fp16, and 16-bit integers
  uint32_t ktab[4], vtab[4], klimb[4];
  const float* Pi;
  const float* S;
  const uint8_t* img[6];       // Pi_hi, Pi_lo, PiT_hi, PiT_lo, ST_hi, ST_lo shared-memory images
  // decode steps: item (b Hkv + hkv) * row_blocks + rb holds rows_per_item query rows; see paged_rows.cuh
  int row_blocks, rows_per_item;
  int8_t* qr;                  // rotated queries [item][row][high, low limb][d], in the look-up's order
  float2* qs;                  // (value of a unit, half the sum of the integers) [item][row]
  int2* parts;                 // (first slot, number) of an item's partial results
  float2* ml;                  // partial (reference, sum) [slot][row]
  float* po;                   // partial outputs [slot][row][parts d]
  int chunk_rows;              // a sequence with more query rows per KV head takes the chunk kernels
  uint32_t* err;
};

// One sequence of the call, its lengths checked against the limits the launch was sized for. Past the limits (an error
// that is reported) no token is seen, but the queries stand where the length says.
struct PagedSeq {
  int q0, qn;                  // first query row, number of queries
  int first, end;              // position of query 0 (filled slots less queries); slots that may be read
};

// The chunk kernels (paged_chunk.cu): their share of the workspace, and the launch.
// Query rows per KV head up to which a sequence is a decode step. Eight rows of a step cost 8.4 ns per 128 tokens of a
// KV head, whatever the batch. A chunk costs 34 ns for opening as many tokens and the time of their scores: 1.9 us,
// on as many SMs as there are (sequence, KV head) units, at least 13 ns. Measured (step against chunk, us; d = 128, K 3 bits,
// V 2 by Algorithm 2, 32 heads over 8): 16 sequences of 4096 tokens 173 / 226 at 32 rows, 245 / 226 at 48, 454 / 227 at
// 96; 4 of 16384: 255 / 364 at 64, 371 / 366 at 96; one of 8192: 107 / 150 at 128 rows, 182 / 179 at 256. The costs are
// those of this format. Others meet nearer or further: at 48 rows of 16 sequences 203 / 166 (d = 64, K 4, V 4),
// 228 / 208 (K 2, V 2), 336 / 235 (K 4, V 4 by Algorithm 2, the largest loss measured).
inline int paged_chunk_rows(int units) {
  const int rows = 8 * (int)((34.0f + 1900.0f / (float)units) / 8.4f);
  return rows < 48 ? 48 : rows > 256 ? 256 : rows;
}
struct PagedChunkPlan {
  int slots;                   // sequences that may have so many rows (0: none)
  int group;                   // (sequence, KV head) units opened at a time
  int tiles;                   // 128-token tiles of a unit, at most
  int row_blocks;
  size_t list, images, heads, base, bytes;
};
PagedChunkPlan paged_chunk_plan(const tq_paged_kv* kv, int B, int Hq, int64_t total_q, int max_q, int64_t max_kv, int window);
tq_status paged_chunk_launch(const PagedAttendParams& p, const tq_paged_kv* kv, const PagedChunkPlan& P, uint8_t* ws,
                             cudaStream_t st);

// The main kernel of decode steps, on `ctas` CTAs.
tq_status paged_rows_launch_64(const PagedAttendParams& p, int kb, int vb, bool alg2, int ctas, cudaStream_t st);
tq_status paged_rows_launch_128(const PagedAttendParams& p, int kb, int vb, bool alg2, int ctas, cudaStream_t st);

#ifdef __CUDACC__
// Launch of a kernel that waits for the one before it itself (griddepcontrol).
inline cudaError_t launch_dependent(void (*kern)(PagedAttendParams), dim3 grid, int threads, size_t smem, cudaStream_t st,
                                    const PagedAttendParams& p) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

__device__ __forceinline__ PagedSeq paged_seq_checked(const PagedAttendParams& p, int b, bool& bad) {
  PagedSeq s;
  s.q0 = p.q_start[b];
  int q1 = p.q_start[b + 1];
  const int kv = p.kv_len[b], most = (int)min(p.max_kv, (int64_t)p.max_pages << p.page_shift);
  bad = false;
  if (s.q0 < 0 || q1 < s.q0 || q1 > p.total_q || q1 - s.q0 > p.max_q) {
    bad = true;
    s.q0 = q1 = 0;
  }
  if (kv < 0 || kv > most) bad = true;
  s.qn = q1 - s.q0;
  s.first = max(kv, 0) - s.qn;
  s.end = max(0, min(kv, most));
  return s;
}
__device__ __forceinline__ PagedSeq paged_seq_quiet(const PagedAttendParams& p, int b) {
  bool bad;
  return paged_seq_checked(p, b, bad);
}
__device__ __forceinline__ PagedSeq paged_seq(const PagedAttendParams& p, int b) {
  bool bad;
  const PagedSeq s = paged_seq_checked(p, b, bad);
  if (bad && threadIdx.x == 0) report_bad_input(p.err);
  return s;
}

// Tokens of a sequence that every query sees (a negative prefix is none).
__device__ __forceinline__ int64_t paged_prefix(const PagedAttendParams& p, const PagedSeq& s, int b) {
  return p.prefix ? max(0, min(p.prefix[b], s.end)) : 0;
}

// Tokens [lo, hi) that the queries at positions [p0, p1] of a sequence may see between them.
__device__ __forceinline__ void paged_range(const PagedAttendParams& p, const PagedSeq& s, int64_t p0, int64_t p1,
                                            int64_t prefix, int64_t& lo, int64_t& hi) {
  hi = min((int64_t)s.end, max(p1 + 1, prefix));
  lo = p.window > 0 && prefix <= 0 ? max((int64_t)0, p0 - p.window + 1) : 0;
  if (hi < lo) hi = lo;
}

// Index nibbles of coordinates s + 4 n (n = 0..7) of a 32-coordinate group, s known at compile time: a shift and
// a masked merge per plane. For 16 levels w holds the magnitudes' planes.
template <int BITS>
__device__ __forceinline__ uint32_t nibbles(const uint32_t* w, int s) {
  uint32_t x = 0;
#pragma unroll
  for (int b = 0; b < (BITS == 4 ? 3 : BITS); ++b)
    x |= (s >= b ? w[b] >> (s - b) : w[b] << (b - s)) & (0x11111111u << b);
  return x;
}
// Of 16 levels: the index planes into those of the magnitudes, and the bits where the level is negative.
template <int BITS>
__device__ __forceinline__ uint32_t magnitudes(uint32_t (&w)[BITS]) {
  if constexpr (BITS == 4) {
    const uint32_t f = ~w[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) w[i] ^= f;
    return f;
  } else {
    return 0u;
  }
}
// Four levels from the low four nibbles of `sel`: (0, 1) and (2, 3) as fp16 pairs.
template <int BITS>
__device__ __forceinline__ void look_up(uint32_t sel, uint32_t neg, const uint32_t (&tab)[4], uint32_t& p0, uint32_t& p1) {
  uint32_t lb, hb;
  if constexpr (BITS <= 2) {
    lb = __byte_perm(tab[0], 0u, sel);
    hb = __byte_perm(tab[2], 0u, sel);
  } else {
    lb = __byte_perm(tab[0], tab[1], sel);
    hb = __byte_perm(tab[2], tab[3], sel);
  }
  if constexpr (BITS == 4) hb ^= __byte_perm(0x8000u, 0u, neg);
  p0 = __byte_perm(lb, hb, 0x5140u);
  p1 = __byte_perm(lb, hb, 0x7362u);
}

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// cap tanh(x / cap) in log2 units, from x2 = 2 log2(e) x / cap: tanh(u) = 1 - 2 / (e^(2u) + 1). Its error is
// absolute, about 2^-23 of the cap, which is what a softmax needs of its scores as long as the cap is not far above
// them (kCapFar: 2^-14 there). e^(2u) may overflow: the quotient is then 0. NaN stays.
__device__ __forceinline__ float capped(float x2, float cap_log2) {
  return cap_log2 - __fdividef(2.0f * cap_log2, ex2_approx(x2) + 1.0f);
}
// The same for larger caps: u + u^3 q(u^2) where |u| <= 1, whose error is relative to u (q fitted to the least largest error
// of tanh, 3.2e-7).
constexpr float kCapFar = 512.f * kLog2e;
__device__ __forceinline__ float capped_far(float x2, float cap_log2) {
  const float u = x2 * 0.34657359f, w = u * u;                   // ln 2 / 2
  const float q = fmaf(fmaf(fmaf(fmaf(-0.00298308f, w, 0.01653281f), w, -0.05142535f), w, 0.13275615f), w, -0.33328670f);
  return fabsf(u) <= 1.f ? cap_log2 * fmaf(q * w, u, u) : capped(x2, cap_log2);
}
// Out of line, and all of a lane's scores at once, for loops that have no registers to spare for it.
static __device__ __noinline__ float4 capped_far4(float4 x2, float cap_log2) {
  return make_float4(capped_far(x2.x, cap_log2), capped_far(x2.y, cap_log2), capped_far(x2.z, cap_log2), capped_far(x2.w, cap_log2));
}
#endif

}  // namespace tq
