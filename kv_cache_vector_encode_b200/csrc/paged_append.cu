// Append of new keys and values to the paged packed cache (tq_paged_append).
//
// Per vector: the key is turned to its position (rope.cu's formula, unrounded), then
//   n = |x|, u = x / n, y = Pi u, idx_i = #{k : t_k < y_i}               (Algorithm 1)
//   r = u - Pi^T c[idx], gamma = |r|, z_i = [(S r)_i >= 0]                (Algorithm 2, values)
// and the record goes to the token's slot.
//
// Up to three dependent d x d products per vector, 128 vectors at a time on the tensor cores. fp16 operands are split,
// a = a_hi + 2^-12 a_lo, and three of the four partial products kept (what is left out is 2^-22 of the operands'
// lengths), which with fp32 accumulation gives y and r to about 2^-19 at worst. That decides all but a few
// coordinates as fp64 would. The others are known, since they lie within a band around a boundary that is wider
// than the error, and are decided again by the whole warp with fp64 sums: about one in 10^4.
//
// Measured: 8192 tokens of 8 heads of 128 (K 3 bits, V 3 bits by Algorithm 2) 111 us, where all in fp64 on the SIMT cores
// took 1279; 64 tokens 16.1 us (the kernel alone). A tile of values takes 24 thousand cycles, of keys 12 thousand: phases that wait for
// one another (2000 to 3000 each for the three products, 5000 for the indices), tensor pipe 12 %, issue 32 %.
//
// Layout: a CTA takes tiles of 128 vectors (keys or values of consecutive heads and tokens), thread = (vector, group of
// 32 coordinates), so that a thread packs a group's code words by itself. Products have the vectors as M (TMEM
// lane = vector). Pi and S are resident in shared memory as K-major images of their rows; Pi^T c takes the same
// image of Pi as an operand with the other major order, so that no transposed copy is needed.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "quant_device.cuh"
#include "sm100.cuh"
#include "tq_internal.h"

namespace tq {
namespace {

struct AppendParams {
  int64_t tokens, n_pos, slots_total, k_stride, v_stride;
  int Hkv, page_shift, half, pairs, f32;
  int tiles;                   // tiles of 128 vectors, of the values and again of the keys
  const void* k;
  const void* v;
  const int64_t* slots;
  const int32_t* positions;
  const float2* table;
  const float* Pi;
  const float* S;
  const float* T;              // S Pi^T
  const float* s_len;          // length of the longest row of S
  const uint8_t* img[4];       // shared-memory images of the rows of Pi and S: high and low parts of each
  uint32_t* k_codes;
  uint16_t* k_norms;
  uint32_t* v_codes;
  uint32_t* v_signs;
  uint16_t* v_norms;
  uint16_t* v_gammas;
  int kb, vb;
  float tk[16], cv[16], tv[16];
  uint32_t* err;
};

constexpr int kVec = 128;              // vectors of a tile
// |error of y| stays below 3.1e-6: 3 2^-22 for the splits, 16 2^-23 should every step of the fp32 accumulation lose a whole
// unit (the sums stay below 1), and 2^-21.3 of y for the length: sums of eight squares of turned coordinates (3 2^-24)
// and their sum, halved by the root
constexpr float kBandY = 3.8146973e-6f;   // 2^-18
// the length itself is rounded to fp16 only where 2^-20 of it makes no difference
constexpr float kBandN = 9.5367432e-7f;   // 2^-20
// A sign is decided again where |s| < band, s = (S r)_i. As vectors over the coordinates, with |u| = 1, |c| <= 1 + gamma:
//   Pi^T c   for the splits 2^-22 sqrt(D) |c| twice (Pi's low part rounded, low times low left out: elementwise 2^-22 of
//            Pi, whose Frobenius norm is sqrt(D)) and 2^-22 |c| (c's low part rounded: Pi keeps its length). The accumulation
//            is taken to lose up to two units of the largest of a step's sums and products, 2^-22 of it. Sums of the first k
//            steps have length |c_1..k| <= |c|, products of a step |c_step|: 2^-22 (sqrt(2) K + sqrt(K)) |c| over K = D / 16
//            steps. And 2^-22 |c| where the parts meet in fp32
//   u        2^-21.3 for the length
//   S r      (3 + K) 2^-22 |S_i| gamma for the product itself, everything above times |S_i|
// so band = max |S_i| ((1 + gamma) kBandC + gamma kBandP + 2^-21), 1.8e-4 at D = 128, |S_i| = 13, gamma = 0.35.
template <int D> struct SignBand {
  static constexpr float kSteps = D / 16, kRoot = D == 128 ? 11.313708f : 8.f, kStepRoot = D == 128 ? 2.8284271f : 2.f, kUnit = 2.3841858e-7f;
  static constexpr float kBandC = (2.f * kRoot + 1.4142136f * kSteps + kStepRoot + 2.f) * kUnit, kBandP = (3.f + kSteps) * kUnit;
  static __device__ __forceinline__ float of(float s_len, float gamma) {
    return s_len * fmaf(gamma, kBandC + kBandP, kBandC + 2.f * kUnit);
  }
};
constexpr float kResScale = 8192.f;    // 2^13: |r| < 4 keeps fp16 in range

template <int D>
struct AppendLayout {
  static constexpr uint32_t G = D / 32, kImg = kVec * D * 2, kMat = 128u * D * 2;
  static constexpr uint32_t kPiHi = 0, kSHi = 2 * kMat, kOpHi = 4 * kMat, kOpLo = kOpHi + kImg,
                            kPart = kOpLo + kImg, kTop = kPart + G * kVec * 4, kCode = kTop + G * kVec * 4,
                            kLevel = kCode + kVec * G * 16, kBar = kLevel + 64, kTotal = kBar + 64 + 1024;
};

template <int D>
struct AppendTile {
  const AppendParams& p;
  int v0;                              // first vector
  bool value;
  __device__ __forceinline__ double raw(int64_t base, int e) const {
    return p.f32 ? (double)((const float*)(value ? p.v : p.k))[base + e]
                 : (double)__uint_as_float((uint32_t)((const uint16_t*)(value ? p.v : p.k))[base + e] << 16);
  }
  // element e of vector v of the tile (turned), as fp64: for the coordinates that are decided again
  __device__ __forceinline__ double elem(int v, int e) const {
    const int t = (v0 + v) / p.Hkv;
    const int64_t base = t * (value ? p.v_stride : p.k_stride) + ((v0 + v) - t * p.Hkv) * D;
    const double x = raw(base, e);
    if (value || e >= 2 * p.half) return x;
    const int pair = p.pairs ? e >> 1 : (e < p.half ? e : e - p.half);
    const bool second = p.pairs ? e & 1 : e >= p.half;
    const float2 cs = p.table[(int64_t)p.positions[t] * p.half + pair];
    const double o = raw(base, p.pairs ? e ^ 1 : (second ? e - p.half : e + p.half));
    return second ? x * cs.x + o * cs.y : x * cs.x - o * cs.y;
  }
};

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// fp16 parts of eight values into the operand images.
__device__ __forceinline__ void split8(const float (&x)[8], uint8_t* hi, uint8_t* lo) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 a = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
    const float2 b = __half22float2(a);
    h[i] = h2_bits(a);
    l[i] = h2_bits(__floats2half2_rn((x[2 * i] - b.x) * kSplitScale, (x[2 * i + 1] - b.y) * kSplitScale));
  }
  *(uint4*)hi = make_uint4(h[0], h[1], h[2], h[3]);
  *(uint4*)lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// Code words of a thread's 32 coordinates from the two accumulators (columns at, at + 128), y = (a + 2^-12 b) inv, and
// the mask of those within the band of a boundary. The boundaries are symmetric: with m = #{positive ones below |y|}
// the index is H + m above zero and H - 1 - m below, so plane i is bit i of m, flipped where y is negative. A bit is
// the sign of a difference, shifted into its word; the smallest difference tells whether any coordinate is near.
template <int BITS>
__device__ __forceinline__ uint32_t code_words(uint32_t at, float inv, const float (&P)[8], uint32_t (&words)[4]) {
  constexpr int M = (1 << (BITS - 1)) - 1;                       // positive boundaries
  uint32_t neg = 0, w[3] = {0, 0, 0}, near = 0;
#pragma unroll
  for (int c = 16; c >= 0; c -= 16) {
    uint32_t a[16], b[16];
    tmem_ld16(at + c, a);
    tmem_ld16(at + 128 + c, b);
    tmem_ld_wait();
    uint32_t mask = 0;
    float nearest = INFINITY;
#pragma unroll
    for (int k = 15; k >= 0; --k) {
      const float y = fmaf(__uint_as_float(b[k]), kSplitScaleInv, __uint_as_float(a[k])) * inv, m = fabsf(y);
      neg = __funnelshift_l(__float_as_uint(y), neg, 1);
      float d[M > 0 ? M : 1], least = m;                         // negative where the boundary is below |y|
#pragma unroll
      for (int i = 0; i < M; ++i) {
        d[i] = P[i] - m;
        least = fminf(least, fabsf(d[i]));
      }
      nearest = fminf(nearest, least);
      a[k] = __float_as_uint(least);
      if (BITS == 2) w[0] = __funnelshift_l(__float_as_uint(d[0]), w[0], 1);
      if (BITS == 3) {
        w[1] = __funnelshift_l(__float_as_uint(d[1 % (M + 1)]), w[1], 1);
        w[0] = __funnelshift_l(__float_as_uint(d[1 % (M + 1)] < 0.f ? d[2 % (M + 1)] : d[0]), w[0], 1);
      }
      if (BITS == 4) {
        const bool m2 = d[3 % (M + 1)] < 0.f;
        const float d1 = m2 ? d[5 % (M + 1)] : d[1 % (M + 1)];
        const bool m1 = d1 < 0.f;
        const float lo = m1 ? d[2 % (M + 1)] : d[0], hi = m1 ? d[6 % (M + 1)] : d[4 % (M + 1)];
        w[2] = __funnelshift_l(__float_as_uint(d[3 % (M + 1)]), w[2], 1);
        w[1] = __funnelshift_l(__float_as_uint(d1), w[1], 1);
        w[0] = __funnelshift_l(__float_as_uint(m2 ? hi : lo), w[0], 1);
      }
    }
    if (nearest < kBandY) {
#pragma unroll
      for (int k = 0; k < 16; ++k) mask |= (uint32_t)(__uint_as_float(a[k]) < kBandY) << k;
    }
    near |= mask << c;
  }
#pragma unroll
  for (int i = 0; i < BITS - 1; ++i) words[i] = w[i] ^ neg;
  words[BITS - 1] = ~neg;
  return near;
}

// What a thread fetches of an item: its vector's slot and position and its 32 coordinates, as they come (nothing waits
// for them until the item's turn).
struct AppendFetch {
  int64_t slot;                // negative: nothing to write
  int pos, h;                  // position, head
  uint4 raw[8];
};

template <int D, bool F32>
__global__ void __launch_bounds__(4 * D, 1) append_kernel(const __grid_constant__ AppendParams p) {
  using L = AppendLayout<D>;
  constexpr int G = D / 32, NR = F32 ? 8 : 4;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  float* part = (float*)(smem + L::kPart);                       // [G][128] partial sums of squares
  uint32_t* top = (uint32_t*)(smem + L::kTop);                   // [G][128] largest magnitudes (as integers)
  uint32_t* codes = (uint32_t*)(smem + L::kCode);                // [128][G][4] code words
  uint32_t* level = (uint32_t*)(smem + L::kLevel);               // [8] fp16 parts of 2^12 c: high, low
  uint64_t* bar = (uint64_t*)(smem + L::kBar);                   // matrices loaded, products done
  uint32_t* tmem_slot = (uint32_t*)(bar + 2);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int v = (warp & 3) * 32 + lane, g = warp >> 2;           // this thread's vector and group
  const bool with_s = p.v_signs && (int)blockIdx.x < p.tiles;    // some item of this CTA needs S
  if (tid == 0) {
    mbar_init(&bar[0], 1);
    mbar_init(&bar[1], 1);
    *abort_flag = 0;
    fence_mbar_init();
    mbar_arrive_expect_tx(&bar[0], (with_s ? 4 : 2) * L::kMat);  // at d = 64 the images' first column block
    for (int i = 0; i < (with_s ? 4 : 2); ++i) bulk_g2s(smem + i * L::kMat, p.img[i], L::kMat, &bar[0]);
  }
  if (tid < 8) {
    const float c = p.cv[tid] * kSplitScale;
    const __half h = __float2half_rn(c);
    level[tid] = (uint32_t)__half_as_ushort(h) | (uint32_t)__half_as_ushort(__float2half_rn((c - __half2float(h)) * kSplitScale)) << 16;
  }
  auto fetch = [&](int item, AppendFetch& f) {
    f.slot = -1;
    f.pos = f.h = 0;
#pragma unroll
    for (int k = 0; k < NR; ++k) f.raw[k] = make_uint4(0, 0, 0, 0);
    if (item >= 2 * p.tiles) return;
    const bool value = item < p.tiles;
    const int n = (value ? item : item - p.tiles) * kVec + v, t = n / p.Hkv;   // below 2^31: checked by the host
    if (t >= p.tokens) return;
    const int h = n - t * p.Hkv;
    const int64_t base = t * (value ? p.v_stride : p.k_stride) + (int64_t)h * D + g * 32;
    const uint4* src = (const uint4*)((const uint8_t*)(value ? p.v : p.k) + base * (F32 ? 4 : 2));
    f.h = h;
    f.slot = p.slots[t];
    if (p.half) f.pos = p.positions[t];
#pragma unroll
    for (int k = 0; k < NR; ++k) f.raw[k] = __ldg(src + k);
  };
  AppendFetch in;
  fetch(blockIdx.x, in);
  if (warp == 0) {
    tmem_alloc(tmem_slot, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tacc = *tmem_slot, mine = tacc + ((uint32_t)((warp & 3) * 32) << 16) + g * 32;
  bool loaded = false;
  uint32_t phase = 0;
  // one product of the operand with a resident matrix (B = its rows, or its columns), into both accumulators
  auto product = [&](uint32_t mat, bool columns) -> bool {
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0 && elect_one_sync()) {
      const uint32_t mh = smem_u32(smem + mat), ml = mh + L::kMat, xh = smem_u32(smem + L::kOpHi), xl = xh + L::kImg;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const uint32_t at = (ks >> 2) * 16384u + (ks & 3) * 32u;
        const uint64_t dh = desc_kmajor_sw128(xh + at), dl = desc_kmajor_sw128(xl + at);
        if (columns) {
          // B[n][k] = M[k][n]: 16 rows (2048 bytes) of the image per step; 64 columns per block, blocks 16 KB apart
          const uint32_t idesc = idesc_f16_f32(128, D) | (1u << 16);
          const uint64_t bh = desc_smem(mh + ks * 2048u, 16384, 1024, 2), bl = desc_smem(ml + ks * 2048u, 16384, 1024, 2);
          mma_f16_ss(tacc, dh, bh, idesc, ks > 0);
          mma_f16_ss(tacc + 128, dh, bl, idesc, ks > 0);
          mma_f16_ss(tacc + 128, dl, bh, idesc, 1);
        } else {
          const uint32_t idesc = idesc_f16_f32(128, D);
          const uint64_t bh = desc_kmajor_sw128(mh + at), bl = desc_kmajor_sw128(ml + at);
          mma_f16_ss(tacc, dh, bh, idesc, ks > 0);
          mma_f16_ss(tacc + 128, dh, bl, idesc, ks > 0);
          mma_f16_ss(tacc + 128, dl, bh, idesc, 1);
        }
      }
      mma_commit(&bar[1]);
    }
    __syncwarp();
    const bool ok = __syncthreads_and(mbar_wait(&bar[1], phase, p.err, kDevTimeoutMma, abort_flag));
    phase ^= 1;
    tc_fence_after();
    return ok;
  };

#pragma unroll 1
  for (int item = blockIdx.x; item < 2 * p.tiles; item += gridDim.x) {
    const bool value = item < p.tiles, alg2 = value && p.v_signs;
    const AppendTile<D> tile{p, (value ? item : item - p.tiles) * kVec, value};
    int64_t rec = -1;                                            // record number
    if (in.slot >= p.slots_total || (in.slot >= 0 && p.half && (in.pos < 0 || in.pos >= p.n_pos)))
      report_bad_input(p.err);
    else if (in.slot >= 0)
      rec = (((in.slot >> p.page_shift) * p.Hkv + in.h) << p.page_shift) + (in.slot & ((1 << p.page_shift) - 1));
    float x[32];
    uint32_t most = 0;                                           // bits of the largest magnitude
#pragma unroll
    for (int k = 0; k < NR; ++k) {
      const uint32_t q[4] = {in.raw[k].x, in.raw[k].y, in.raw[k].z, in.raw[k].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (F32) {
          x[4 * k + i] = __uint_as_float(q[i]);
        } else {
          x[8 * k + 2 * i] = __uint_as_float(q[i] << 16);
          x[8 * k + 2 * i + 1] = __uint_as_float(q[i] & 0xFFFF0000u);
        }
      }
    }
    // ---- turn, with the partners through shared memory ---------------------------------------------------------
    if (!value && p.half) {                                      // uniform over the block
      const int rot = 2 * p.half, e0 = g * 32;
      const float2* row = p.table + (int64_t)(rec < 0 ? 0 : in.pos) * p.half;
      const bool turn = rec >= 0 && e0 < rot;
#pragma unroll
      for (int k = 0; k < 32; ++k) most |= x[k] != 0.f ? 1u : 0u;
      const bool wide = ((uintptr_t)p.table & 15) == 0;          // rows of the table then are, for the cases that ask
      if (p.pairs && rot % 32 == 0 && wide) {                    // both halves of a pair are here
        if (turn) {
          const float4* cs = (const float4*)(row + e0 / 2);      // half is a multiple of 16: rows are 16-byte aligned
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float4 w = __ldg(cs + k);
            const float a0 = x[4 * k], b0 = x[4 * k + 1], a1 = x[4 * k + 2], b1 = x[4 * k + 3];
            x[4 * k] = fmaf(a0, w.x, -(b0 * w.y));
            x[4 * k + 1] = fmaf(b0, w.x, a0 * w.y);
            x[4 * k + 2] = fmaf(a1, w.z, -(b1 * w.w));
            x[4 * k + 3] = fmaf(b1, w.z, a1 * w.w);
          }
        }
      } else {
        float* raw = (float*)(smem + L::kOpHi);                  // [coordinate][vector]
#pragma unroll
        for (int k = 0; k < 32; ++k) raw[(e0 + k) * kVec + v] = x[k];
        __syncthreads();
        if (!p.pairs && p.half % 32 == 0 && wide) {                      // a group is all first or all second halves
          if (turn) {
            const bool second = e0 >= p.half;
            const int other = second ? e0 - p.half : e0 + p.half;
            const float4* cs = (const float4*)(row + (second ? e0 - p.half : e0));
            const float sign = second ? 1.f : -1.f;
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float4 w = __ldg(cs + k);
              x[2 * k] = fmaf(x[2 * k], w.x, raw[(other + 2 * k) * kVec + v] * (sign * w.y));
              x[2 * k + 1] = fmaf(x[2 * k + 1], w.z, raw[(other + 2 * k + 1) * kVec + v] * (sign * w.w));
            }
          }
        } else if (turn) {
#pragma unroll
          for (int c = 0; c < 32; c += 16) {                     // loads of sixteen coordinates at a time
            float2 cs[16];
            float o[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const int e = e0 + c + k, at = e < rot ? e : 0;
              const bool second = p.pairs ? at & 1 : at >= p.half;
              cs[k] = __ldg(row + (p.pairs ? at >> 1 : (second ? at - p.half : at)));
              o[k] = raw[(p.pairs ? at ^ 1 : (second ? at - p.half : at + p.half)) * kVec + v] * (second ? cs[k].y : -cs[k].y);
            }
#pragma unroll
            for (int k = 0; k < 16; ++k)
              if (e0 + c + k < rot) x[c + k] = fmaf(x[c + k], cs[k].x, o[k]);
          }
        }
      }
    }
#pragma unroll
    for (int k = 0; k < 32; ++k) most = max(most, __float_as_uint(x[k]) & 0x7FFFFFFFu);
    top[g * kVec + v] = most;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < G; ++k) most = max(most, top[k * kVec + v]);
    // ---- y = Pi x: x times a power of two that brings its largest coordinate into [2^13, 2^14) -------------------
    const bool ok = rec >= 0 && most > 0 && most < 0x7F800000u;  // a row that is zero or not finite: u = 0
    // keys outside what fp32 turns well: above 5e37 (products may overflow) or below 1e-30 (they may be subnormal)
    const bool far = rec >= 0 && !value && p.half && most > 0 && (most < 0x0DA24260u || most > 0x7E167699u);
    float f1 = 0.f, f2 = 0.f;
    int E = 0;
    if (ok) {
      frexpf(__uint_as_float(most), &E);
      pow2_pair(14 - E, f1, f2);
    }
    float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        w[k] = x[8 * c + k] = ok ? x[8 * c + k] * f1 * f2 : 0.f;
        s4[c] = fmaf(w[k], w[k], s4[c]);
      }
      const uint32_t off = sw128_offset(v, (g * 32 + c * 8) * 2, kVec);
      split8(w, smem + L::kOpHi + off, smem + L::kOpLo + off);
    }
    part[g * kVec + v] = (s4[0] + s4[1]) + (s4[2] + s4[3]);
    if (!loaded) {
      if (!__syncthreads_and(mbar_wait(&bar[0], 0, p.err, kDevTimeoutLoad, abort_flag))) break;
      loaded = true;
    }
    if (!product(L::kPiHi, false)) break;
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < G; ++k) ss += part[k * kVec + v];
    const float len = sqrtf(ss);                                 // |x| 2^(14 - E)
    const float inv = ok ? 1.f / len : 0.f;
    fetch(item + gridDim.x, in);                                 // the next item's, while this one goes on
    // ---- indices --------------------------------------------------------------------------------------------
    const int bits = value ? p.vb : p.kb;
    uint32_t words[4] = {0, 0, 0, 0}, near;
    {
      float P[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int at = (1 << (bits - 1)) + k;                    // boundary 2^(bits-1) is the first positive one
        P[k] = at < (1 << bits) - 1 ? (value ? p.tv[at] : p.tk[at]) : INFINITY;
      }
      near = bits == 1   ? code_words<1>(mine, inv, P, words)
             : bits == 2 ? code_words<2>(mine, inv, P, words)
             : bits == 3 ? code_words<3>(mine, inv, P, words)
                         : code_words<4>(mine, inv, P, words);
    }
    near = far ? ~0u : ok ? near : 0u;
    if (!ok) {                                                   // y is exactly zero: index 2^(bits-1) - 1
#pragma unroll
      for (int b = 0; b < 4; ++b) words[b] = b < bits - 1 ? ~0u : 0u;
    }
    // coordinates to be decided again, by the whole warp
    const float* tab = value ? p.tv : p.tk;
    for (uint32_t who; (who = __ballot_sync(0xffffffffu, near != 0)) != 0;) {
      const int src = __ffs(who) - 1, vv = (warp & 3) * 32 + src;
      const int k = __ffs(__shfl_sync(0xffffffffu, near, src)) - 1, i = g * 32 + k;
      double d = 0.0, n = 0.0;
#pragma unroll
      for (int j = lane; j < D; j += 32) {
        const double e = tile.elem(vv, j);
        d = fma((double)__ldg(p.Pi + (size_t)i * D + j), e, d);
        n = fma(e, e, n);
      }
      n = sqrt(warp_sum(n));
      d = warp_sum(d);
      const double y = n > 0.0 && n <= 1.7976931348623157e308 ? d / n : 0.0;
      int idx = 0;
      for (int b = 0; b < (1 << bits) - 1; ++b) idx += (double)tab[b] < y ? 1 : 0;
      if (lane == src) {
        near &= near - 1;
#pragma unroll
        for (int b = 0; b < 4; ++b)
          if (b < bits) words[b] = (words[b] & ~(1u << k)) | (uint32_t)((idx >> b) & 1) << k;
      }
    }
    if (rec >= 0) {
      uint32_t* dst = (value ? p.v_codes : p.k_codes) + (rec * G + g) * bits;
      for (int b = 0; b < bits; ++b) dst[b] = words[b];
    }
    if (g == 0) {                                                // the length: whole warps
      float f1n, f2n;
      pow2_pair(E - 14, f1n, f2n);
      const float n = most < 0x7F800000u ? len * f1n * f2n : __uint_as_float(most);
      __half hn = __float2half_rn(n);
      bool again = rec >= 0 && (far || most >= 0x7F800000u ||
                                (ok && __half_as_ushort(__float2half_rn(n * (1.f - kBandN))) != __half_as_ushort(__float2half_rn(n * (1.f + kBandN)))));
      for (uint32_t who; (who = __ballot_sync(0xffffffffu, again)) != 0;) {
        const int src = __ffs(who) - 1, vv = (warp & 3) * 32 + src;
        double m = 0.0;
#pragma unroll
        for (int j = lane; j < D; j += 32) {
          const double e = tile.elem(vv, j);
          m = fma(e, e, m);
        }
        m = sqrt(warp_sum(m));
        if (lane == src) {
          again = false;
          hn = __double2half(m);
        }
      }
      if (rec >= 0) (value ? p.v_norms : p.k_norms)[rec] = __half_as_ushort(hn);
    }
    if (!alg2) {
      tc_fence_before();
      __syncthreads();                                           // the operands' and parts' space is free
      continue;
    }
    // ---- Pi^T c[idx] -----------------------------------------------------------------------------------------
#pragma unroll
    for (int b = 0; b < 4; ++b) codes[(v * G + g) * 4 + b] = words[b];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int at = 8 * c + k;
        const int idx = ((words[0] >> at) & 1) | ((words[1] >> at) & 1) << 1 | ((words[2] >> at) & 1) << 2;
        w[k] = level[idx];
      }
      const uint32_t off = sw128_offset(v, (g * 32 + c * 8) * 2, kVec);
      *(uint4*)(smem + L::kOpHi + off) = make_uint4(__byte_perm(w[0], w[1], 0x5410u), __byte_perm(w[2], w[3], 0x5410u),
                                                    __byte_perm(w[4], w[5], 0x5410u), __byte_perm(w[6], w[7], 0x5410u));
      *(uint4*)(smem + L::kOpLo + off) = make_uint4(__byte_perm(w[0], w[1], 0x7632u), __byte_perm(w[2], w[3], 0x7632u),
                                                    __byte_perm(w[4], w[5], 0x7632u), __byte_perm(w[6], w[7], 0x7632u));
    }
    if (!product(L::kPiHi, true)) break;
    // ---- r = u - Pi^T c, gamma ---------------------------------------------------------------------------------
    float gs = 0.f;
#pragma unroll
    for (int c = 0; c < 32; c += 16) {
      uint32_t a[16], b[16];
      tmem_ld16(mine + c, a);
      tmem_ld16(mine + 128 + c, b);
      tmem_ld_wait();
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const float e = fmaf(__uint_as_float(b[k]), kSplitScaleInv, __uint_as_float(a[k])) * kSplitScaleInv;
        x[c + k] = ok ? fmaf(x[c + k], inv, -e) : 0.f;
        gs = fmaf(x[c + k], x[c + k], gs);
      }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = x[8 * c + k] * kResScale;
      const uint32_t off = sw128_offset(v, (g * 32 + c * 8) * 2, kVec);
      split8(w, smem + L::kOpHi + off, smem + L::kOpLo + off);
    }
    part[g * kVec + v] = gs;
    const float s_len = __ldg(p.s_len);                          // before the wait
    if (!product(L::kSHi, false)) break;
    // ---- signs -------------------------------------------------------------------------------------------------
    gs = 0.f;
#pragma unroll
    for (int k = 0; k < G; ++k) gs += part[k * kVec + v];
    const float gamma = sqrtf(gs), band = SignBand<D>::of(s_len, gamma) * kResScale;
    uint32_t sign = 0;
    near = 0;
#pragma unroll
    for (int c = 0; c < 32; c += 16) {
      uint32_t a[16], b[16];
      tmem_ld16(mine + c, a);
      tmem_ld16(mine + 128 + c, b);
      tmem_ld_wait();
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const float s = fmaf(__uint_as_float(b[k]), kSplitScaleInv, __uint_as_float(a[k]));
        sign |= (uint32_t)(s >= 0.f) << (c + k);
        near |= (uint32_t)(fabsf(s) < band) << (c + k);
      }
    }
    if (!ok) near = 0;                                           // r is exactly zero
    for (uint32_t who; (who = __ballot_sync(0xffffffffu, near != 0)) != 0;) {
      const int src = __ffs(who) - 1, vv = (warp & 3) * 32 + src;
      const int k = __ffs(__shfl_sync(0xffffffffu, near, src)) - 1, i = g * 32 + k;
      // (S r)_i = S_i u - T_i c in fp64. T is rounded to fp32: off by 2^-24 |T_i| |c| at most
      auto level_of = [&](int q) {
        const uint32_t* w = codes + (vv * G + (q >> 5)) * 4;
        const int at = q & 31;
        return (double)p.cv[((w[0] >> at) & 1) | ((w[1] >> at) & 1) << 1 | ((w[2] >> at) & 1) << 2];
      };
      double su = 0.0, tc = 0.0, tt = 0.0, cc = 0.0, nn = 0.0;
#pragma unroll
      for (int j = lane; j < D; j += 32) {
        const double tij = (double)__ldg(p.T + (size_t)i * D + j), cj = level_of(j), e = tile.elem(vv, j);
        su = fma((double)__ldg(p.S + (size_t)i * D + j), e, su);
        nn = fma(e, e, nn);
        tc = fma(tij, cj, tc);
        tt = fma(tij, tij, tt);
        cc = fma(cj, cj, cc);
      }
      nn = sqrt(warp_sum(nn));
      double s = warp_sum(su) / nn - warp_sum(tc);
      tt = warp_sum(tt);
      cc = warp_sum(cc);
      if (fabs(s) <= 6e-8 * sqrt(tt * cc) + 1e-12) {             // still undecided: r itself, lane = coordinates
        double a[G] = {};
#pragma unroll 4
        for (int q = 0; q < D; ++q) {
          const double c = level_of(q);
#pragma unroll
          for (int j = 0; j < G; ++j) a[j] = fma((double)__ldg(p.Pi + (size_t)q * D + 32 * j + lane), c, a[j]);
        }
        s = 0.0;
#pragma unroll
        for (int j = 0; j < G; ++j)
          s = fma((double)__ldg(p.S + (size_t)i * D + 32 * j + lane), tile.elem(vv, 32 * j + lane) / nn - a[j], s);
        s = warp_sum(s);
      }
      if (lane == src) {
        near &= near - 1;
        sign = (sign & ~(1u << k)) | (uint32_t)(s >= 0.0) << k;
      }
    }
    if (rec >= 0) {
      p.v_signs[rec * G + g] = sign;
      if (g == 0) p.v_gammas[rec] = __half_as_ushort(__float2half_rn(gamma));
    }
    tc_fence_before();
    __syncthreads();
  }
  if (tid == 0 && !loaded) mbar_wait(&bar[0], 0, p.err, kDevTimeoutLoad, abort_flag);   // no copy outlives the block
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tacc, 256);
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
  if (tokens > 0 && (!k_new || !v_new || !slots || !rot || (rot_dim && (!positions || (!table && n_pos > 0)))))
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
  p.T = (const float*)((const uint8_t*)rot + RL.t32);
  p.s_len = (const float*)((const uint8_t*)rot + kRotSLen);
  const size_t img[4] = {RL.pi_hi, RL.pi_lo, RL.s_hi, RL.s_lo};
  for (int i = 0; i < 4; ++i) p.img[i] = (const uint8_t*)rot + img[i];
  p.k_codes = kv->k_codes;
  p.k_norms = kv->k_norms;
  p.v_codes = kv->v_codes;
  p.v_signs = kv->v_signs;
  p.v_norms = kv->v_norms;
  p.v_gammas = kv->v_gammas;
  p.kb = kv->k_bits;
  p.vb = kv->v_bits;
  for (int k = 0; k < 16; ++k) {
    p.tk[k] = kv->tk[k];
    p.cv[k] = kv->cv[k];
    p.tv[k] = kv->tv[k];
  }
  p.err = device_error_word();
  if (!p.err) return fail(TQ_ERR_CUDA, f + ": no device error word (is a CUDA device present?)");
  const int tiles = (int)((tokens * kv->Hkv + kVec - 1) / kVec);
  p.tiles = tiles;
  const unsigned grid = (unsigned)std::min(2 * tiles, sm_count());
  auto go = [&](auto kern, int smem, int threads) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return cuda_fail(e, "tq_paged_append: shared memory attribute");
    kern<<<grid, threads, smem, (cudaStream_t)stream>>>(p);
    e = cudaGetLastError();
    return e == cudaSuccess ? TQ_OK : cuda_fail(e, "tq_paged_append: launch");
  };
  if (kv->d == 128)
    return p.f32 ? go(append_kernel<128, true>, AppendLayout<128>::kTotal, 512) : go(append_kernel<128, false>, AppendLayout<128>::kTotal, 512);
  return p.f32 ? go(append_kernel<64, true>, AppendLayout<64>::kTotal, 256) : go(append_kernel<64, false>, AppendLayout<64>::kTotal, 256);
}
