// Attention of few query rows per KV head over the paged packed cache (decode steps of tq_paged_attend), and
// the host side of the call.
//
//   out = Pi^T sum_t w_t n_t c_v[idx_t] (+ alpha S^T sum_t w_t n_t gamma_t (2 z_t - 1)),
//   w = softmax of x_t = scale n_t <Pi q, c_k[idx_t]>, capped, biased and masked.
// Nothing is dequantised to memory: the queries are rotated once (prep kernel), scores and value sums are
// formed in the rotated domain from the codes, and Pi^T / S^T are applied once per query row (combine).
//
// What bounds it: a cached token of one KV head is 86 bytes at 3 + 2 bits and d = 128, so at the card's
// copy rate an SM has about 470 cycles for 128 tokens, in which 3 x 16384 coordinates have to be unpacked
// for the tensor cores. Unpacking is therefore the cost to keep down, and the reason for warp-level
// products (mma.sync) instead of tcgen05 here: their operands are registers, so that an unpacked
// coordinate is used where it was made. With tcgen05 the value planes would go through shared memory
// (32 KB written and read per plane and 128 tokens: about 1000 cycles), for products that are only eight
// columns wide.
//
// Layout. A CTA takes one (sequence, KV head, block of eight query rows, split of the visible tokens); its
// eight warps take 16-token blocks in turn, each with a softmax state of its own. Lane = 4 r + c.
//   scores  S[16 tokens x 8 rows] = K Q^T, A = keys: lane (r, c) unpacks a quarter of the coordinates of
//           tokens r and r + 8; the K order inside a quarter is the order in which the byte-permute
//           look-up yields them, and the query fragments are loaded in that order.
//   values  O^T[d x 8 rows] += V^T P^T, A = values: lane (r, c) supplies tokens 2c, 2c+1, 2c+8, 2c+9 for
//           the output coordinates of its r. One-bit planes (the signs, and one-bit codes) are used
//           without being unpacked: the words of two tokens are merged by a byte permute, and masking
//           one bit of each half leaves an fp16 value z 2^e, where e depends on the bit's place alone and is
//           taken out of the output row at the end (a bit in the sign place is XORed into 1.0 instead).
//           So four instructions make eight matrix elements. sum w (2z - 1) = 2 sum w z - sum w.
//   P       from the score layout to the operand's by an 8 x 8 transpose (movmatrix).
// The softmax reference of a row moves only when a score passes it by more than 8 (log2 domain), so that
// the accumulators are rarely rescaled; weights stay below 2^8. The value norms enter the weights, relative
// to the largest norm met so far (a power of two, kept with the reference), so that fp16 holds them.
//
// The packed records come by cp.async into a ring of 16-token stages per warp (no CTA-wide barrier in
// the loop).
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

constexpr int kRows = 8;          // query rows per CTA
constexpr int kWarps = 8;
constexpr int kStages = 4;
constexpr float kLazy = 8.0f;     // how far (log2) a score may pass the reference before it moves
constexpr float kRoom = 64.0f;    // weights are below 2^8 and enter fp16 times this (times a residual norm, below 2)

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int D, int KB, int VB, bool ALG2>
struct Stage {   // 32-bit words of a 16-token stage
  static constexpr int G = D / 32;
  static constexpr int kKey = 0, kVal = kKey + 16 * G * KB, kSign = kVal + 16 * G * VB,
                       kKn = kSign + (ALG2 ? 16 * G : 0), kVn = kKn + 8, kVg = kVn + 8, kWords = kVg + (ALG2 ? 8 : 0);
  static constexpr int kChunks = kWords / 4, kIter = (kChunks + 31) / 32;
  static constexpr int kParts = ALG2 ? 2 : 1;
  static constexpr size_t ring() { return (size_t)kWarps * kStages * kWords * 4; }
  static constexpr size_t merge() { return (size_t)kWarps * kRows * (kParts * D + 4) * 4; }
  static constexpr size_t smem() { return ring() > merge() ? ring() : merge(); }
};

template <int D, int KB, int VB, bool ALG2>
__global__ void __launch_bounds__(32 * kWarps, 2) rows_kernel(const __grid_constant__ PagedAttendParams p) {
  using L = Stage<D, KB, VB, ALG2>;
  constexpr int G = D / 32, KS = D / 16, MB = D / 16;
  extern __shared__ __align__(16) uint32_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  const int b = blockIdx.z / p.Hkv, hkv = blockIdx.z % p.Hkv;
  const PagedSeq sq = paged_seq(p, b);
  const int rows = sq.qn * p.g, row0 = blockIdx.y * kRows;
  if (row0 >= rows || rows > p.chunk_rows) return;
  const int64_t first = sq.kv - sq.qn;                           // position of query 0
  const int64_t prefix = p.prefix ? min((int64_t)p.prefix[b], sq.kv) : 0;
  const int jlo = row0 / p.g, jhi = min(rows - 1, row0 + kRows - 1) / p.g;
  int64_t lo, hi;
  paged_range(p, sq, first + jlo, first + jhi, prefix, lo, hi);
  const int64_t t0 = (lo & ~15LL) + (int64_t)blockIdx.x * p.span;
  const int64_t t1 = min(hi, t0 + p.span);
  const int nblk = t1 > t0 ? (int)((t1 - t0 + 15) >> 4) : 0;

  const int64_t slot0 = (int64_t)blockIdx.z * p.row_slots;       // this unit's rows in the workspace
  // this lane's two query rows (2c, 2c + 1 of the block)
  int64_t pos[2];
  float fac[2], slope[2], ref[2], sum[2], wsum[2] = {0.f, 0.f}, zsum[2] = {0.f, 0.f};
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int row = row0 + 2 * c + u;
    const bool on = row < rows;
    const int j = on ? row / p.g : 0, h = hkv * p.g + (on ? row - j * p.g : 0);
    pos[u] = on ? first + j : -1;
    fac[u] = on ? p.scale_log2 * p.qs[slot0 + row] : 0.f;
    slope[u] = on && p.slopes ? p.slopes[h] * kLog2e : 0.f;
    ref[u] = -INFINITY;
    sum[u] = 0.f;
    if (!on) pos[u] = INT64_MIN / 2;
  }
  float elim[2] = {0.f, 0.f};                                    // power of two >= every value norm seen
  // query fragments: row r of the block, coordinates of quarter c in look-up order
  uint32_t qf[KS][2];
  {
    const int row = row0 + r;
    const bool on = row < rows;
    const __half* q = p.qr + (slot0 + (on ? row : 0)) * D + c * (D / 4);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const int at = D == 128 ? (ks >> 1) + 16 * (ks & 1) : ks;
      const uint32_t x0 = __half_as_ushort(q[at]), x1 = __half_as_ushort(q[at + 4]);
      const uint32_t x2 = __half_as_ushort(q[at + 8]), x3 = __half_as_ushort(q[at + 12]);
      qf[ks][0] = on ? x0 | (x1 << 16) : 0u;
      qf[ks][1] = on ? x2 | (x3 << 16) : 0u;
    }
  }
  float oc[MB][4], oz[ALG2 ? MB : 1][4];
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      oc[m][i] = 0.f;
      if (ALG2) oz[m][i] = 0.f;
    }

  // ---- the ring: where this lane's 16-byte chunks of a stage come from --------------------------------
  uint32_t* ring = smem + warp * (kStages * L::kWords);
  const uint32_t ring_u32 = smem_u32(ring);
  const uint8_t* src[L::kIter];
  uint32_t unit[L::kIter];                                      // bytes of 16 tokens of its array
#pragma unroll
  for (int i = 0; i < L::kIter; ++i) {
    const int w = 4 * (lane + 32 * i);
    const void* base = p.k_codes;
    int at = w, len = L::kVal;
    if (w >= L::kVal) base = p.v_codes, at = w - L::kVal, len = L::kSign - L::kVal;
    if (ALG2 && w >= L::kSign) base = p.v_signs, at = w - L::kSign, len = 16 * G;
    if (w >= L::kKn) base = p.k_norms, at = w - L::kKn, len = 8;
    if (w >= L::kVn) base = p.v_norms, at = w - L::kVn, len = 8;
    if (ALG2 && w >= L::kVg) base = p.v_gammas, at = w - L::kVg, len = 8;
    src[i] = (const uint8_t*)base + 4 * at;
    unit[i] = 4 * len;
  }
  const int32_t* table = p.table + (int64_t)b * p.max_pages;
  const int units_per_page = 1 << (p.page_shift - 4);
  auto page_of = [&](int blk) { return blk < nblk ? table[(t0 + 16 * blk) >> p.page_shift] : 0; };
  uint32_t absent = 0;                                           // stages whose page number is out of range
  auto issue = [&](int blk, int page) {
    if (blk < nblk) {
      const int s = (blk / kWarps) % kStages;
      const bool good = page >= 0 && page < p.num_pages;
      if (!good && lane == 0) atomicCAS(p.err, 0u, (uint32_t)kDevBadInput);
      absent = good ? absent & ~(1u << s) : absent | (1u << s);
      const int64_t u16 = good ? ((int64_t)page * p.Hkv + hkv) * units_per_page + (((t0 >> 4) + blk) & (units_per_page - 1)) : 0;
      const uint32_t dst = ring_u32 + (s * L::kWords + 4 * lane) * 4;
#pragma unroll
      for (int i = 0; i < L::kIter; ++i)
        if (i + 1 < L::kIter || lane + 32 * i < L::kChunks)
          cp_async16(dst + 512 * i, src[i] + u16 * unit[i], good ? 16u : 0u);
    }
    cp_commit();
  };
  int page_next = page_of(warp);
  for (int k = 0; k < kStages - 1; ++k) {
    const int page = page_next;
    page_next = page_of(warp + (k + 1) * kWarps);
    issue(warp + k * kWarps, page);
  }

  uint32_t ktab[4], vtab[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) ktab[i] = p.ktab[i], vtab[i] = p.vtab[i];
  const uint32_t m0 = 0x00010001u << r, m1 = 0x01000100u << r, x1 = r == 7 ? 0x3C003C00u : 0u;
  const int64_t vis_lo = p.window > 0 ? first + jhi - p.window + 1 : 0;   // from here on every row's window is open

  for (int blk = warp; blk < nblk; blk += kWarps) {
    {
      const int page = page_next;
      page_next = page_of(blk + kStages * kWarps);
      cp_wait<kStages - 2>();
      __syncwarp();
      // the stage read in the previous turn is free: all lanes are past it
      issue(blk + (kStages - 1) * kWarps, page);
    }
    const int s = (blk / kWarps) % kStages;
    const uint32_t* st = ring + s * L::kWords;
    const int64_t t = t0 + 16 * blk;

    // ---- scores ----------------------------------------------------------------------------------
    float sc[2][4] = {};
    {
      uint32_t wa[KB], wb[KB];
      const int grp = D == 128 ? c : c >> 1;
#pragma unroll
      for (int b2 = 0; b2 < KB; ++b2) {
        wa[b2] = st[L::kKey + (r * G + grp) * KB + b2];
        wb[b2] = st[L::kKey + ((r + 8) * G + grp) * KB + b2];
      }
#pragma unroll
      for (int s4 = 0; s4 < 4; ++s4) {
        uint32_t na, nb;
        uint32_t xa, xb;
        if constexpr (D == 128) {
          xa = pick<KB>(wa, s4, na);
          xb = pick<KB>(wb, s4, nb);
        } else {
          xa = pick<KB>(wa, s4 + 16 * (c & 1), na);
          xb = pick<KB>(wb, s4 + 16 * (c & 1), nb);
        }
#pragma unroll
        for (int half = 0; half < (D == 128 ? 2 : 1); ++half) {
          uint32_t a0, a1, a2, a3;
          look_up<KB>(half ? xa >> 16 : xa, half ? na >> 16 : na, ktab, a0, a2);
          look_up<KB>(half ? xb >> 16 : xb, half ? nb >> 16 : nb, ktab, a1, a3);
          const int ks = D == 128 ? 2 * s4 + half : s4;
          mma_16816(sc[ks & 1], a0, a1, a2, a3, qf[ks][0], qf[ks][1]);
        }
      }
    }
    // ---- softmax weights: tokens r, r + 8 of rows 2c, 2c + 1 -----------------------------------------
    const uint16_t* kn = (const uint16_t*)(st + L::kKn);
    const uint16_t* vn = (const uint16_t*)(st + L::kVn);
    float x[2][2];                                               // [token][row]
    const int64_t ta = t + r;
    const bool whole = t + 16 <= t1 && !((absent >> s) & 1) &&
                       ((t + 15 <= first + jlo && t >= vis_lo) || t + 16 <= prefix);
    bool in[2] = {true, true};                                   // token within the range at all
    float nk[2], nv[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      in[k] = whole || (ta + 8 * k < t1 && !((absent >> s) & 1));
      nk[k] = in[k] ? __half2float(__ushort_as_half(kn[r + 8 * k])) : 0.f;
      nv[k] = in[k] ? __half2float(__ushort_as_half(vn[r + 8 * k])) : 0.f;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float v = (sc[0][2 * k + u] + sc[1][2 * k + u]) * (nk[k] * fac[u]);
        if (p.cap_log2 > 0.f) v = capped(v * p.cap2x, p.cap_log2);
        if (p.slopes) v += slope[u] * (float)(ta + 8 * k - pos[u]);
        if (!whole) {
          const int64_t tt = ta + 8 * k;
          const bool see = in[k] && pos[u] > INT64_MIN / 4 &&
                           ((tt <= pos[u] && (p.window == 0 || tt > pos[u] - p.window)) || tt < prefix);
          v = see ? v : -INFINITY;
        }
        x[k][u] = v;
      }
    }
    // largest score and largest finite value norm that a row sees
    float top[2], topn[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      top[u] = fmaxf(x[0][u], x[1][u]);
      topn[u] = fmaxf(x[0][u] > -INFINITY && nv[0] < INFINITY ? nv[0] : 0.f,
                      x[1][u] > -INFINITY && nv[1] < INFINITY ? nv[1] : 0.f);
    }
    if (__any_sync(0xffffffffu, top[0] > ref[0] + kLazy || top[1] > ref[1] + kLazy || topn[0] > elim[0] || topn[1] > elim[1])) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          top[u] = fmaxf(top[u], __shfl_xor_sync(0xffffffffu, top[u], o));
          topn[u] = fmaxf(topn[u], __shfl_xor_sync(0xffffffffu, topn[u], o));
        }
      float f[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float nr = fmaxf(ref[u], top[u]);
        const float fs = nr == ref[u] ? 1.f : ex2_approx(ref[u] - nr);   // 0 from the empty state
        ref[u] = nr;
        sum[u] *= fs;
        f[u] = fs;
        if (topn[u] > elim[u]) {
          // the norm limit: the next power of two (the exponent field of the largest norm, plus one)
          const float el = __int_as_float((__float_as_int(topn[u]) & 0x7F800000) + 0x00800000);
          f[u] *= elim[u] / el;
          elim[u] = el;
        }
        wsum[u] *= f[u];
        zsum[u] *= f[u];
      }
#pragma unroll
      for (int q = 0; q < MB; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          oc[q][i] *= f[i & 1];
          if (ALG2) oz[q][i] *= f[i & 1];
        }
    }
    const float einv[2] = {elim[0] > 0.f ? kRoom / elim[0] : 0.f, elim[1] > 0.f ? kRoom / elim[1] : 0.f};
    uint32_t pc[2], pz[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float w[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float e = ex2_approx(x[k][u] - (ref[u] == -INFINITY ? 0.f : ref[u]));
        sum[u] += e;
        w[u] = x[k][u] == -INFINITY ? 0.f : e * (nv[k] * einv[u]);   // an unseen token's norm may be anything
        if (VB == 1) wsum[u] += w[u];
      }
      pc[k] = transpose8x8(half2_of(w[0], w[1]));
      if constexpr (ALG2) {
        const uint16_t* vg = (const uint16_t*)(st + L::kVg);
        const float ga = in[k] ? __half2float(__ushort_as_half(vg[r + 8 * k])) : 0.f;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          w[u] = x[k][u] == -INFINITY ? 0.f : w[u] * ga;
          zsum[u] += w[u];
        }
        pz[k] = transpose8x8(half2_of(w[0], w[1]));
      }
    }
    // ---- values ----------------------------------------------------------------------------------
    const int tk[4] = {2 * c, 2 * c + 1, 2 * c + 8, 2 * c + 9};
    auto plane = [&](const uint32_t* words, int stride, float (&o)[MB][4], uint32_t b0, uint32_t b1) {
#pragma unroll
      for (int g = 0; g < G; ++g) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = words[tk[k] * stride + g];
        const uint32_t l01 = __byte_perm(w[0], w[1], 0x5410u), h01 = __byte_perm(w[0], w[1], 0x7632u);
        const uint32_t l23 = __byte_perm(w[2], w[3], 0x5410u), h23 = __byte_perm(w[2], w[3], 0x7632u);
        mma_16816(o[2 * g], l01 & m0, (l01 & m1) ^ x1, l23 & m0, (l23 & m1) ^ x1, b0, b1);
        mma_16816(o[2 * g + 1], h01 & m0, (h01 & m1) ^ x1, h23 & m0, (h23 & m1) ^ x1, b0, b1);
      }
    };
    if constexpr (VB == 1) {
      plane(st + L::kVal, G, oc, pc[0], pc[1]);
    } else {
#pragma unroll
      for (int g = 0; g < G; ++g) {
        uint32_t e[4][2];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t w[VB], neg;
#pragma unroll
          for (int b2 = 0; b2 < VB; ++b2) w[b2] = st[L::kVal + (tk[k] * G + g) * VB + b2];
          const uint32_t sel = pick<VB>(w, (r & 3) + 16 * (r >> 2), neg);
          look_up<VB>(sel, neg, vtab, e[k][0], e[k][1]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
          mma_16816(oc[2 * g + h], __byte_perm(e[0][h], e[1][h], 0x5410u), __byte_perm(e[0][h], e[1][h], 0x7632u),
                    __byte_perm(e[2][h], e[3][h], 0x5410u), __byte_perm(e[2][h], e[3][h], 0x7632u), pc[0], pc[1]);
      }
    }
    if constexpr (ALG2) plane(st + L::kSign, G, oz, pz[0], pz[1]);
  }

  // ---- merge the warps' states ---------------------------------------------------------------------
  cp_wait<0>();
  __syncthreads();                                               // the ring is free
  constexpr int PD = L::kParts * D, RS = PD + 4;
  float* mg = (float*)smem;                                      // [warp][row][parts D, ref, sum]
#pragma unroll
  for (int u = 0; u < 2; ++u) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      sum[u] += __shfl_xor_sync(0xffffffffu, sum[u], o);
      wsum[u] += __shfl_xor_sync(0xffffffffu, wsum[u], o);
      zsum[u] += __shfl_xor_sync(0xffffffffu, zsum[u], o);
    }
    float* dst = mg + (warp * kRows + 2 * c + u) * RS;
    if (r == 0) {
      dst[PD] = ref[u];
      dst[PD + 1] = sum[u];
    }
    // a one-bit plane: bit place i of a 16-bit half is the fp16 value 2^-24 2^i (i < 10), 2^-14, 2^-13,
    // 2^-11, 2^-7, 2 (i = 10 .. 14), or the sign of 1 (i = 15)
    auto bit_value = [](int i) {
      return i < 10 ? __int_as_float((127 - 24 + i) << 23) : __int_as_float((127 + (1 << (i - 10)) - 15) << 23);
    };
    auto put = [&](float (&o)[MB][4], int at, bool one_bit, float total, float unit) {
#pragma unroll
      for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float v = o[m][2 * h + u];
          int dim;
          if (one_bit) {
            const int i = r + 8 * h;
            dim = 16 * m + i;
            v = i == 15 ? -v : 2.f * v / bit_value(i) - total;
          } else {
            dim = 32 * (m >> 1) + (r & 3) + 16 * (r >> 2) + 4 * (2 * (m & 1) + h);
          }
          dst[at + dim] = v * (elim[u] * unit);
        }
    };
    put(oc, 0, VB == 1, wsum[u], p.v_inv_unit / kRoom);
    if constexpr (ALG2) put(oz, D, true, zsum[u], 1.f / kRoom);
  }
  __syncthreads();
  const int live = min(kRows, rows - row0);
  for (int e = threadIdx.x; e < live * PD; e += 32 * kWarps) {
    const int row = e / PD, i = e - row * PD;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, mg[(w * kRows + row) * RS + PD]);
    const float base = top == -INFINITY ? 0.f : top;
    float o = 0.f, l = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float* m = mg + (w * kRows + row) * RS;
      const float f = ex2_approx(m[PD] - base);
      o += f * m[i];
      l += f * m[PD + 1];
    }
    const int64_t at = (slot0 + row0 + row) * p.nsplit + blockIdx.x;
    p.po[at * PD + i] = o;
    if (i == 0) p.ml[at] = make_float2(top, l);
  }
}

// ---- queries into the rotated domain --------------------------------------------------------------------
// q' = Pi q of a row block (thread = coordinate), stored as fp16 times a power of two that brings
// the largest coordinate of the row into [2^11, 2^12): the rounding (2^-12 relative) is the only loss.
constexpr int kPrepRows = kRows;
template <int D>
__global__ void __launch_bounds__(D) prep_kernel(const __grid_constant__ PagedAttendParams p) {
  __shared__ float4 sq[kPrepRows][D / 4];
  __shared__ float red[kPrepRows][D / 32];
  const int i = threadIdx.x;
  const int b = blockIdx.y / p.Hkv, hkv = blockIdx.y % p.Hkv;
  const PagedSeq sq_ = paged_seq(p, b);
  const int row0 = blockIdx.x * kPrepRows, rows = sq_.qn * p.g;
  if (row0 >= rows || rows > p.chunk_rows) return;
#pragma unroll
  for (int u = 0; u < kPrepRows; ++u) {
    const int row = min(row0 + u, rows - 1), j = row / p.g;
    ((float*)sq[u])[i] = __uint_as_float(
        (uint32_t)p.q[(int64_t)(sq_.q0 + j) * p.q_stride + (int64_t)(hkv * p.g + row - j * p.g) * D + i] << 16);
  }
  __syncthreads();
  float acc[kPrepRows] = {};
  const float4* pi = (const float4*)(p.Pi + (size_t)i * D);
#pragma unroll 8
  for (int j = 0; j < D / 4; ++j) {
    const float4 m = __ldg(pi + j);
#pragma unroll
    for (int u = 0; u < kPrepRows; ++u) {
      const float4 x = sq[u][j];
      acc[u] = fmaf(m.x, x.x, fmaf(m.y, x.y, fmaf(m.z, x.z, fmaf(m.w, x.w, acc[u]))));
    }
  }
#pragma unroll
  for (int u = 0; u < kPrepRows; ++u) {
    float m = fabsf(acc[u]);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((i & 31) == 0) red[u][i >> 5] = m;
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kPrepRows; ++u) {
    if (row0 + u >= rows) break;
    const int64_t at = (int64_t)blockIdx.y * p.row_slots + row0 + u;
    float m = red[u][0];
#pragma unroll
    for (int w = 1; w < D / 32; ++w) m = fmaxf(m, red[u][w]);
    // exponent field of the largest coordinate, kept where both 2^e and 2^-e are normal numbers
    const int e = min(max((__float_as_int(m) >> 23) & 255, 20), 230);
    const float up = __int_as_float((254 + 11 - e) << 23), down = __int_as_float((e - 11) << 23);
    p.qr[at * D + i] = __float2half_rn(acc[u] * up);
    if (i == 0) p.qs[at] = down;
  }
}

// ---- splits together, back to the original domain ------------------------------------------------------
// Four rows per block (thread = coordinate): o' = sum of the splits' outputs, then Pi^T o'_c + alpha S^T o'_z.
constexpr int kCombRows = 4;
template <int D, bool ALG2>
__global__ void __launch_bounds__(D) combine_kernel(const __grid_constant__ PagedAttendParams p) {
  constexpr int PD = ALG2 ? 2 * D : D;
  __shared__ float so[kCombRows][PD];
  const int i = threadIdx.x;
  const int b = blockIdx.y / p.Hkv, hkv = blockIdx.y % p.Hkv;
  const PagedSeq sq = paged_seq(p, b);
  const int row0 = blockIdx.x * kCombRows, rows = sq.qn * p.g;
  if (row0 >= rows || rows > p.chunk_rows) return;
  int64_t at[kCombRows];
#pragma unroll
  for (int u = 0; u < kCombRows; ++u) {
    const int row = min(row0 + u, rows - 1), j = row / p.g;
    at[u] = (int64_t)(sq.q0 + j) * p.Hq + hkv * p.g + row - j * p.g;
  }
#pragma unroll
  for (int u = 0; u < kCombRows; ++u) {
    const int64_t slot = ((int64_t)blockIdx.y * p.row_slots + min(row0 + u, rows - 1)) * p.nsplit;
    const float2* ml = p.ml + slot;
    const float* po = p.po + slot * PD;
    float c = 0.f, z = 0.f, l = 0.f, top = -INFINITY;
    for (int s = 0; s < p.nsplit; ++s) top = fmaxf(top, ml[s].x);
    if (top == -INFINITY) top = 0.f;
    for (int s = 0; s < p.nsplit; ++s) {
      const float f = ex2_approx(ml[s].x - top);
      l = fmaf(f, ml[s].y, l);
      c = fmaf(f, po[s * PD + i], c);
      if (ALG2) z = fmaf(f, po[s * PD + D + i], z);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;   // NaN stays NaN
    so[u][i] = c * inv;
    if (ALG2) so[u][D + i] = p.alpha * z * inv;
  }
  __syncthreads();
  float acc[kCombRows] = {};
#pragma unroll 8
  for (int j = 0; j < D; ++j) {
    const float m = __ldg(p.Pi + (size_t)j * D + i);
    const float s = ALG2 ? __ldg(p.S + (size_t)j * D + i) : 0.f;
#pragma unroll
    for (int u = 0; u < kCombRows; ++u) {
      acc[u] = fmaf(m, so[u][j], acc[u]);
      if (ALG2) acc[u] = fmaf(s, so[u][D + j], acc[u]);
    }
  }
#pragma unroll
  for (int u = 0; u < kCombRows; ++u)
    if (row0 + u < rows) p.out[at[u] * D + i] = __bfloat16_as_ushort(__float2bfloat16_rn(acc[u]));
}

// ---- host -----------------------------------------------------------------------------------------------

struct Plan {
  int row_blocks, nsplit, span;
  size_t qr, qs, ml, po, total;
  PagedChunkPlan chunk;
};

Plan plan(const tq_paged_kv* kv, int B, int Hq, int64_t total_q, int max_q, int64_t max_kv, int window) {   // B and max_q > 0
  Plan P{};
  const int g = Hq / kv->Hkv;
  const bool chunks = (int64_t)max_q * g > kChunkRows;
  P.row_blocks = chunks ? (kChunkRows + kRows - 1) / kRows : (max_q * g + kRows - 1) / kRows;
  // about four CTAs per resident slot (two per SM) where the tokens allow it, at least 256 tokens each
  const int64_t units = (int64_t)B * kv->Hkv * P.row_blocks;
  const int64_t most = std::max<int64_t>(1, (max_kv + 255) / 256);
  P.nsplit = (int)std::min<int64_t>({most, std::max<int64_t>(1, 148 * 8 / units), 128});
  // with a window (and no prefix) a row block sees the window and its own queries' span
  int64_t seen = max_kv;
  if (window > 0) seen = std::min<int64_t>(seen, (int64_t)window + (kRows + g - 1) / g + 1);
  int64_t span = (seen + 15 + P.nsplit - 1) / P.nsplit;
  P.span = (int)((span + 15) / 16 * 16);
  auto al = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t rows = (size_t)B * kv->Hkv * P.row_blocks * kRows, pd = (size_t)kv->d * (kv->v_alg == 2 ? 2 : 1);
  size_t off = 0;
  P.qr = off; off += al(rows * kv->d * 2);
  P.qs = off; off += al(rows * 4);
  P.ml = off; off += al(rows * P.nsplit * 8);
  P.po = off; off += al(rows * P.nsplit * pd * 4);
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

template <int D, int KB, int VB, bool ALG2>
tq_status launch_rows(const PagedAttendParams& p, dim3 grid, cudaStream_t st) {
  auto kern = rows_kernel<D, KB, VB, ALG2>;
  const size_t smem = Stage<D, KB, VB, ALG2>::smem();
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return cuda_fail(e, "tq_paged_attend: shared memory attribute");
  kern<<<grid, 32 * kWarps, smem, st>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return cuda_fail(e, "tq_paged_attend: launch");
  return TQ_OK;
}
template <int D, int KB>
tq_status launch_values(const PagedAttendParams& p, int vb, bool alg2, dim3 grid, cudaStream_t st) {
  if (alg2) switch (vb) {
      case 1: return launch_rows<D, KB, 1, true>(p, grid, st);
      case 2: return launch_rows<D, KB, 2, true>(p, grid, st);
      default: return launch_rows<D, KB, 3, true>(p, grid, st);
    }
  switch (vb) {
    case 1: return launch_rows<D, KB, 1, false>(p, grid, st);
    case 2: return launch_rows<D, KB, 2, false>(p, grid, st);
    case 3: return launch_rows<D, KB, 3, false>(p, grid, st);
    default: return launch_rows<D, KB, 4, false>(p, grid, st);
  }
}
template <int D>
tq_status launch_keys(const PagedAttendParams& p, int kb, int vb, bool alg2, dim3 grid, cudaStream_t st) {
  switch (kb) {
    case 1: return launch_values<D, 1>(p, vb, alg2, grid, st);
    case 2: return launch_values<D, 2>(p, vb, alg2, grid, st);
    case 3: return launch_values<D, 3>(p, vb, alg2, grid, st);
    default: return launch_values<D, 4>(p, vb, alg2, grid, st);
  }
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
  if (work && (!q || !q_start || !kv_len || !page_table || !rot || !out)) return fail(TQ_ERR_INVALID_ARG, f + ": NULL pointer");
  if (q_dtype != TQ_BF16) return fail(TQ_ERR_UNSUPPORTED, f + ": q must be TQ_BF16");
  if (max_pages < 0 || window < 0) return fail(TQ_ERR_INVALID_ARG, f + ": negative max_pages or window");
  if (!(softcap >= 0.0f) || std::isinf(softcap)) return fail(TQ_ERR_INVALID_ARG, f + ": softcap must be finite and >= 0");
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
  p.scale_log2 = scale * kLog2e / kv->k_unit;
  p.cap_log2 = softcap * kLog2e;
  p.cap2x = softcap > 0.0f ? 2.0f / softcap : 0.0f;   // x arrives times log2(e), as exp2 wants it
  p.v_inv_unit = 1.0f / kv->v_unit;
  p.alpha = (float)(std::sqrt(std::acos(-1.0) / 2.0) / kv->d);
  p.k_unit = kv->k_unit;
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
  p.qr = (__half*)(w + P.qr);
  p.qs = (float*)(w + P.qs);
  p.ml = (float2*)(w + P.ml);
  p.po = (float*)(w + P.po);
  p.nsplit = P.nsplit;
  p.span = P.span;
  p.chunk_rows = kChunkRows;
  p.row_slots = P.row_blocks * kRows;
  p.err = device_error_word();
  if (!p.err) return fail(TQ_ERR_CUDA, f + ": no device error word (is a CUDA device present?)");
  cudaStream_t st = (cudaStream_t)stream;
  const bool alg2 = kv->v_alg == 2;
  const dim3 grid(P.nsplit, P.row_blocks, B * kv->Hkv), pg(P.row_blocks, B * kv->Hkv),
      cg(P.row_blocks * (kRows / kCombRows), B * kv->Hkv);
  cudaError_t e;
  if (P.chunk.slots) {
    s = paged_chunk_launch(p, kv, P.chunk, w + P.chunk.base, st);
    if (s != TQ_OK) return s;
  }
  if (kv->d == 128) {
    prep_kernel<128><<<pg, 128, 0, st>>>(p);
    if ((s = launch_keys<128>(p, kv->k_bits, kv->v_bits, alg2, grid, st)) != TQ_OK) return s;
    if (alg2) combine_kernel<128, true><<<cg, 128, 0, st>>>(p);
    else combine_kernel<128, false><<<cg, 128, 0, st>>>(p);
  } else {
    prep_kernel<64><<<pg, 64, 0, st>>>(p);
    if ((s = launch_keys<64>(p, kv->k_bits, kv->v_bits, alg2, grid, st)) != TQ_OK) return s;
    if (alg2) combine_kernel<64, true><<<cg, 64, 0, st>>>(p);
    else combine_kernel<64, false><<<cg, 64, 0, st>>>(p);
  }
  if ((e = cudaGetLastError()) != cudaSuccess) return cuda_fail(e, "tq_paged_attend: launch");
  return TQ_OK;
}
