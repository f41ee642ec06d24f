// Attention of few query rows per KV head over the paged packed cache: the main kernel of a decode step
// (instantiated per head size in paged_rows_64.cu and paged_rows_128.cu).
//
// What bounds it: a cached token of one KV head is 86 bytes at 3 + 2 bits and d = 128, so at the card's copy
// rate an SM quarter has 235 cycles for 16 tokens, in which 3 x 2048 coordinates have to reach the tensor
// cores. The integer pipe takes two cycles per warp instruction (measured: lop3, prmt and shifts all 2.0), so
// the time is the number of instructions that unpacking takes, and the formats below are chosen for few:
//   keys    as 8-bit limbs: four index nibbles select four bytes of a level table, so a byte-permute makes four
//           matrix elements (the high or the low byte of the 16-bit levels; m16n8k32, 8 cycles, twice the
//           rate of fp16). The queries are 16-bit integers in two limbs, next to each other as columns: four
//           rows make the eight columns of a product. Sums are exact; 16 bits are 2^-16 of the largest
//           level and of the largest query coordinate.
//   values  one-bit planes (the signs, and one-bit codes) are used without being unpacked at d = 128: a
//           transposing matrix load brings the 16-bit halves of two tokens into one register, and masking
//           one bit of each half leaves the fp16 value z 2^e, where e depends on the bit's place alone and is
//           taken out of the output row at the end (a bit in the sign place is XORed into 1.0 instead):
//           one instruction makes two elements. sum w (2 z - 1) = 2 sum w z - sum w.
//           Wider codes are looked up as fp16 levels.
// mma.sync instead of tcgen05, because its operands are registers: an unpacked coordinate is used where it was
// made, while tcgen05 would take the value planes through shared memory (32 KB written and read per plane and
// 128 tokens: about 1000 cycles) for products that are eight columns wide.
//
// Work. The 16-token blocks of all (sequence, KV head, row block) items in a row are cut into equal ranges, one per
// CTA (two CTAs per SM): ragged batches cost no waiting, and a CTA's start and end are paid once per range, not
// once per split of every sequence. A CTA's part of an item is a partial result in slot (CTA + item), which no
// other part can share; the first part of an item records (first slot, parts) for the combine kernel.
// Short batches are latency: a part costs some 4 us before and after its blocks, whose time is 0.6 us for eight (one per
// warp). Where it lengthens a range by less than that, items are therefore cut into parts of their own, none of which
// shares a CTA (4 sequences of 1000 tokens: 20.5 -> 16.4 us).
// Inside a part the eight warps take the blocks in turn, each with a softmax state and a cp.async ring of its own
// (no barrier in the loop). Lane = 4 r + c holds tokens r and r + 8 for the rows c and c + 4.
// The softmax reference of a row moves only when a score passes it by more than 8 (log2 domain), so that the
// accumulators are rarely rescaled; weights stay below 2^8. The value norms enter the weights, relative to the
// largest norm seen so far (a power of two, kept with the reference), so that fp16 holds them.
//
// Measured: one step of 16 sequences of up to 32768 tokens (32 query heads over 8, K 3 bits, V 2) 154 us with prep and
// combine, 1.8 TB/s of packed records; 420 warp instructions per 16 tokens, integer pipe 57 %, tensor pipe 25 %. Two
// CTAs of eight warps per SM: three at 80 registers gain nothing (177 against 172 us).
#pragma once
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "paged_attend.h"
#include "sm100.cuh"

namespace tq {

constexpr int kRowWarps = 8;
constexpr int kRowStages = 4;
constexpr int kRowSlack = 48;     // blocks by which a range may grow to hold a part of one item alone
constexpr float kRowLazy = 8.0f;  // how far (log2) a score may pass the reference before it moves
constexpr float kRowRoom = 64.0f; // weights are below 2^8 and enter fp16 times this (times a residual norm, below 2)

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_u8s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the same with zero for the sum so far
__device__ __forceinline__ void mma_s8_first(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(0));
}
__device__ __forceinline__ void mma_u8s8_first(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(0));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ void load_trans2(uint32_t addr, uint32_t& x, uint32_t& y) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];" : "=r"(x), "=r"(y) : "r"(addr));
}
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int D, int KB, int VB, bool ALG2, int NB>
struct RowStage {   // 32-bit words of a 16-token stage
  static constexpr int G = D / 32;
  static constexpr int kKey = 0, kVal = kKey + 16 * G * KB, kSign = kVal + 16 * G * VB,
                       kKn = kSign + (ALG2 ? 16 * G : 0), kVn = kKn + 8, kVg = kVn + 8, kWords = kVg + (ALG2 ? 8 : 0);
  static constexpr int kChunks = kWords / 4, kIter = (kChunks + 31) / 32;
  static constexpr int kParts = ALG2 ? 2 : 1;
  static constexpr int kRows = 4 * NB;
  static constexpr size_t ring() { return (size_t)kRowWarps * kRowStages * kWords * 4; }
  static constexpr size_t merge() { return (size_t)kRowWarps * kRows * (kParts * D + 4) * 4; }
  static constexpr size_t smem() { return ring() > merge() ? ring() : merge(); }
};

// Quotient of non-negative numbers that seldom need their 64 bits.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// 16-token blocks of row block rb of a sequence (none for the chunk kernels' sequences).
__device__ __forceinline__ int row_blocks_of(const PagedAttendParams& p, const PagedSeq& s, int64_t prefix, int rb, int64_t& lo,
                                             int64_t& hi) {
  const int rows = s.qn * p.g, row0 = rb * p.rows_per_item;
  lo = hi = 0;
  if (row0 >= rows || rows > p.chunk_rows) return 0;
  const int64_t first = s.first;
  const int j0 = row0 == 0 ? 0 : row0 / p.g, j1 = row0 + p.rows_per_item >= rows ? s.qn - 1 : (row0 + p.rows_per_item - 1) / p.g;
  paged_range(p, s, first + j0, first + j1, prefix, lo, hi);
  if (hi <= lo) return 0;      // before lo moves to the start of its block
  lo &= ~15LL;
  return (int)((hi - lo + 15) >> 4);
}

// Where a CTA starts. Its range counts blocks of all items, or (unit > 0) parts of all items, of `unit` blocks at most.
struct RowStart {
  int64_t pos, end, total;      // this CTA's range; blocks or parts of all items
  int64_t base;                 // first block or part of sequence b
  int b, ctas, unit;            // sequence that the range starts in; CTAs that take part
};
__device__ __forceinline__ int row_parts(int blocks, int unit) { return unit > 0 ? (blocks + unit - 1) / unit : blocks; }

template <int D, int KB, int VB, bool ALG2, int NB>
__global__ void __launch_bounds__(32 * kRowWarps, 2) rows_kernel(const __grid_constant__ PagedAttendParams p) {
  using L = RowStage<D, KB, VB, ALG2, NB>;
  constexpr int G = D / 32, MB = D / 16, RB = L::kRows, PD = L::kParts * D, RS = PD + 4, NT = 32 * kRowWarps;
  extern __shared__ __align__(16) uint32_t smem[];
  __shared__ RowStart start;
  __shared__ int64_t sums[kRowWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;

  // ---- this CTA's range: every CTA adds up the batch's blocks, each thread a run of sequences -------------------
  {
    auto count = [&](int b, int unit) {
      const PagedSeq s = paged_seq_quiet(p, b);
      const int64_t prefix = paged_prefix(p, s, b);
      int64_t lo, hi, n = 0;
      for (int rb = 0; rb < p.row_blocks; ++rb) n += row_parts(row_blocks_of(p, s, prefix, rb, lo, hi), unit);
      return n * p.Hkv;
    };
    const int per = (p.B + NT - 1) / NT, b0 = min(p.B, (int)threadIdx.x * per), b1 = min(p.B, b0 + per);
    int64_t mine, before, total;
    auto add_up = [&](int unit) {
      mine = 0;
      for (int b = b0; b < b1; ++b) mine += count(b, unit);
      before = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += v;
      }
      if (lane == 31) sums[warp] = before;
      __syncthreads();
      total = 0;
      before -= mine;
      for (int w = 0; w < kRowWarps; ++w) {
        if (w < warp) before += sums[w];
        total += sums[w];
      }
    };
    add_up(0);
    // at least a block per warp: fewer CTAs where there is less
    int ctas = (int)min((int64_t)gridDim.x, (total + kRowWarps - 1) / kRowWarps), unit = 0;
    const int64_t items = (int64_t)p.B * p.Hkv * p.row_blocks;
    if (items < (int64_t)gridDim.x) {                            // parts of `whole` blocks fit, whatever the items' lengths
      const int64_t whole = max((int64_t)kRowWarps, quotient(total + gridDim.x - items - 1, gridDim.x - items));
      if (whole <= quotient(total, gridDim.x) + kRowSlack) {
        __syncthreads();                                         // the sums have been read
        unit = (int)whole;
        add_up(unit);
        ctas = (int)total;
      }
    }
    if ((int)blockIdx.x >= ctas) {                               // uniform
      grid_dep_wait();                                           // the next kernel may rely on the one before this
      return;
    }
    const int64_t pos = unit ? blockIdx.x : quotient(blockIdx.x * total, ctas);
    const int64_t end = unit ? blockIdx.x + 1 : quotient((blockIdx.x + 1) * total, ctas);
    if (pos >= before && pos < before + mine) {
      int b = b0;
      int64_t base = before;
      for (; b + 1 < b1; ++b) {
        const int64_t n = count(b, unit);
        if (pos < base + n) break;
        base += n;
      }
      start = RowStart{pos, end, total, base, b, ctas, unit};
    }
    __syncthreads();
  }
  grid_dep_launch();
  bool waited = false;

  uint32_t ktab[4], vtab[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) ktab[i] = p.klimb[i], vtab[i] = p.vtab[i];
  uint32_t* ring = smem + warp * (kRowStages * L::kWords);
  const uint32_t ring_u32 = smem_u32(ring);
  const int units_per_page = 1 << (p.page_shift - 4);

  int64_t pos = start.pos, base = start.base;
  for (int b = start.b; pos < start.end && b < p.B; ++b) {
    const PagedSeq sq = paged_seq(p, b);
    const int64_t first = sq.first;
    const int64_t prefix = paged_prefix(p, sq, b);
    const int rows = sq.qn * p.g;
    // items in the order of their numbers, so that (CTA + item) grows with every part
    int hkv = 0;
    {                                                            // KV heads that lie before the range at once
      int64_t lo, hi, head = 0;
      for (int rb = 0; rb < p.row_blocks; ++rb) head += row_parts(row_blocks_of(p, sq, prefix, rb, lo, hi), start.unit);
      if (head == 0) continue;
      hkv = (int)min((int64_t)p.Hkv, quotient(pos - base, head));
      base += hkv * head;
    }
    for (; hkv < p.Hkv && pos < start.end; ++hkv) {
      int np;
      for (int rb = 0; rb < p.row_blocks && pos < start.end; ++rb, base += np) {
        int64_t lo, hi;
        const int nb = row_blocks_of(p, sq, prefix, rb, lo, hi);
        np = row_parts(nb, start.unit);
        if (pos >= base + np) continue;                          // done by CTAs before, or empty
        const int row0 = rb * RB;
        const int jlo = row0 == 0 ? 0 : row0 / p.g, jhi = row0 + RB >= rows ? sq.qn - 1 : (row0 + RB - 1) / p.g;
        // ---- one part: blocks [pos, stop) of item (b, hkv, rb) ------------------------------------------------
        const int64_t stop = min(base + np, start.end);
        const int blk_lo = start.unit ? (int)quotient((pos - base) * nb, np) : (int)(pos - base);
        const int blk_hi = start.unit ? (int)quotient((stop - base) * nb, np) : (int)(stop - base);
        const int t0 = (int)lo + 16 * blk_lo, t1 = (int)min(hi, lo + 16 * (int64_t)blk_hi);
        const int nblk = blk_hi - blk_lo;
        const int item = (b * p.Hkv + hkv) * p.row_blocks + rb;
        const bool opens = pos == base;                          // the item's first part
        pos = stop;

        // outputs: columns c and c + 4 of a product. With four rows the sign plane's go where the rows c + 4 would be
        constexpr bool SHARE = ALG2 && NB == 1;
        float oc[MB][4], oz[ALG2 && !SHARE ? MB : 1][4];
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            oc[m][i] = 0.f;
            if (ALG2 && !SHARE) oz[m][i] = 0.f;
          }

        // ---- the ring: where this lane's 16-byte chunks of a stage come from ----------------------------------
        const uint8_t* src[L::kIter];
        uint32_t unit[L::kIter];                                 // bytes of 16 tokens of its array
#pragma unroll
        for (int i = 0; i < L::kIter; ++i) {
          const int w = 4 * (lane + 32 * i);
          const void* array = p.k_codes;
          int at = w, len = L::kVal;
          if (w >= L::kVal) array = p.v_codes, at = w - L::kVal, len = L::kSign - L::kVal;
          if (ALG2 && w >= L::kSign) array = p.v_signs, at = w - L::kSign, len = 16 * G;
          if (w >= L::kKn) array = p.k_norms, at = w - L::kKn, len = 8;
          if (w >= L::kVn) array = p.v_norms, at = w - L::kVn, len = 8;
          if (ALG2 && w >= L::kVg) array = p.v_gammas, at = w - L::kVg, len = 8;
          src[i] = (const uint8_t*)array + 4 * at;
          unit[i] = 4 * len;
        }
        const int32_t* table = p.table + (int64_t)b * p.max_pages;
        const int blk0 = t0 >> 4;                                // block number in the sequence
        auto page_of = [&](int blk) { return blk < nblk ? table[(blk0 + blk) >> (p.page_shift - 4)] : 0; };
        uint32_t absent = 0;                                     // stages whose page number is out of range
        auto issue = [&](int blk, int page, int s) {
          if (blk < nblk) {
            uint32_t bytes = 16;
            if ((uint32_t)page >= (uint32_t)p.num_pages) {
              if (lane == 0) report_bad_input(p.err);
              absent |= 1u << s;
              page = 0;
              bytes = 0;
            }
            const uint32_t u16 = ((uint32_t)page * p.Hkv + hkv) * units_per_page + ((blk0 + blk) & (units_per_page - 1));
            const uint32_t dst = ring_u32 + (s * L::kWords + 4 * lane) * 4;
#pragma unroll
            for (int i = 0; i < L::kIter; ++i)
              if (i + 1 < L::kIter || lane + 32 * i < L::kChunks)
                cp_async16(dst + 512 * i, src[i] + (uint64_t)u16 * unit[i], bytes);
          }
          cp_commit();
        };
        int page_next = page_of(warp);
#pragma unroll 1
        for (int k = 0; k < kRowStages - 1; ++k) {
          const int page = page_next;
          page_next = page_of(warp + (k + 1) * kRowWarps);
          issue(warp + k * kRowWarps, page, k);
        }
        if (!waited) {
          grid_dep_wait();                                       // the queries come from the kernel before
          waited = true;
        }
        if (opens && threadIdx.x == 0) {
          // up to the CTA of the item's last block
          const int n = start.unit ? np : (int)(((base + np) * start.ctas - 1) / start.total) - (int)blockIdx.x + 1;
          p.parts[item] = make_int2(blockIdx.x + item, n);
        }
        // this lane's query rows (c and c + 4 of the block)
        int qpos[NB];
        // ref is the reference (from: the same, 0 in the empty state), elim a power of two >= every value norm seen
        // and room what its inverse times kRowRoom is
        float fac[NB], slope[NB], ref[NB], from[NB], sum[NB], wsum[NB], zsum[NB], elim[NB], room[NB];
        int qsum[NB];
#pragma unroll
        for (int u = 0; u < NB; ++u) {
          const int row = row0 + c + 4 * u;
          const bool on = row < rows;
          const int j = on ? row / p.g : 0, h = hkv * p.g + (on ? row - j * p.g : 0);
          const int64_t at = (int64_t)item * RB + c + 4 * u;
          qpos[u] = on ? (int)first + j : -1;
          fac[u] = on ? p.key_fac * p.qs[at].x : 0.f;
          qsum[u] = on && KB == 4 ? __float_as_int(p.qs[at].y) : 0;
          slope[u] = on && p.slopes ? p.slopes[h] * kLog2e : 0.f;
          ref[u] = -INFINITY;
          sum[u] = wsum[u] = zsum[u] = 0.f;
          from[u] = elim[u] = 0.f;
          room[u] = 1.f;
        }
        // query limbs: column 2 h + limb of block u is head row h + 4 u
        uint32_t qf[NB][D / 16];
#pragma unroll
        for (int u = 0; u < NB; ++u) {
          const int row = (r >> 1) + 4 * u;
          const bool on = row0 + row < rows;
          const uint4* src = (const uint4*)(p.qr + (((int64_t)item * RB + (on ? row : 0)) * 2 + (r & 1)) * D + c * (D / 4));
#pragma unroll
          for (int i = 0; i < D / 64; ++i) {
            const uint4 v = on ? src[i] : make_uint4(0, 0, 0, 0);
            qf[u][4 * i] = v.x, qf[u][4 * i + 1] = v.y, qf[u][4 * i + 2] = v.z, qf[u][4 * i + 3] = v.w;
          }
        }
        // tokens [open_lo, open_hi) are seen by every row (and those before the prefix)
        const int open_lo = p.window > 0 ? (int)first + jhi - p.window + 1 : 0, open_hi = min((int)first + jlo + 1, t1);
        const int pre = (int)prefix, open_pre = min(pre, t1);

#pragma unroll 1
        for (int blk = warp, s = 0; blk < nblk; blk += kRowWarps, s = (s + 1) % kRowStages) {
          {
            const int page = page_next;
            page_next = page_of(blk + kRowStages * kRowWarps);
            cp_wait<kRowStages - 2>();
            __syncwarp();
            // the stage read in the previous turn is free: all lanes are past it
            issue(blk + (kRowStages - 1) * kRowWarps, page, (s + kRowStages - 1) % kRowStages);
          }
          const uint32_t* st = ring + s * L::kWords;
          const uint32_t st_u32 = ring_u32 + s * (L::kWords * 4);
          const int t = t0 + 16 * blk;

          // ---- scores: high and low bytes of the levels against the query limbs ---------------------------------
          int ah[NB][4], al[NB][4];
          {
            uint32_t wa[KB], wb[KB];
            const int grp = D == 128 ? c : c >> 1;
#pragma unroll
            for (int i = 0; i < KB; ++i) {
              wa[i] = st[L::kKey + (r * G + grp) * KB + i];
              wb[i] = st[L::kKey + ((r + 8) * G + grp) * KB + i];
              if (D == 64 && (c & 1)) wa[i] >>= 16, wb[i] >>= 16;
            }
            const uint32_t fa = magnitudes<KB>(wa), fb = magnitudes<KB>(wb);
            // four levels' bytes from the low four nibbles of sel
            auto bytes = [&](uint32_t sel, uint32_t flip, uint32_t& hi8, uint32_t& lo8) {
              hi8 = __byte_perm(ktab[2], ktab[3], sel);
              lo8 = __byte_perm(ktab[0], ktab[1], sel);
              if constexpr (KB == 4) {                           // -(X + 1/2) = ~X + 1/2
                const uint32_t m = __byte_perm(0xFF00u, 0u, flip);
                hi8 ^= m;
                lo8 ^= m;
              }
            };
            uint32_t h[4], l[4];
#pragma unroll
            for (int s4 = 0; s4 < 4; ++s4) {
              const uint32_t xa = nibbles<KB>(wa, s4), xb = nibbles<KB>(wb, s4);
              const uint32_t na = KB == 4 ? (fa >> s4) & 0x11111111u : 0u, nb2 = KB == 4 ? (fb >> s4) & 0x11111111u : 0u;
              const int lo2 = D == 128 ? 0 : 2 * (s4 & 1);       // at d = 64 two turns make a product
              bytes(xa, na, h[lo2], l[lo2]);
              bytes(xb, nb2, h[lo2 + 1], l[lo2 + 1]);
              if (D == 128) {
                bytes(xa >> 16, na >> 16, h[2], l[2]);
                bytes(xb >> 16, nb2 >> 16, h[3], l[3]);
              }
              if (D == 128 || (s4 & 1)) {
                const int ks = D == 128 ? s4 : s4 >> 1;
#pragma unroll
                for (int u = 0; u < NB; ++u) {
                  if (ks == 0) {
                    mma_s8_first(ah[u], h[0], h[1], h[2], h[3], qf[u][0], qf[u][1]);
                    mma_u8s8_first(al[u], l[0], l[1], l[2], l[3], qf[u][0], qf[u][1]);
                  } else {
                    mma_s8(ah[u], h[0], h[1], h[2], h[3], qf[u][2 * ks], qf[u][2 * ks + 1]);
                    mma_u8s8(al[u], l[0], l[1], l[2], l[3], qf[u][2 * ks], qf[u][2 * ks + 1]);
                  }
                }
              }
            }
          }
          // ---- softmax weights: tokens r, r + 8 of rows c, c + 4 ------------------------------------------------
          const uint16_t* kn = (const uint16_t*)(st + L::kKn);
          const uint16_t* vn = (const uint16_t*)(st + L::kVn);
          float x[2][NB], n[2][NB], ga[2][NB];                   // [token][row]: score, value norm, residual norm
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float nk = __half2float(__ushort_as_half(kn[r + 8 * k]));
            // a key norm that is not finite makes the token's value NaN: its score alone might be taken to the cap, or to
            // minus infinity and a weight of 0
            const float nv = fmaf(nk, 0.f, __half2float(__ushort_as_half(vn[r + 8 * k])));
            const float ng = ALG2 ? __half2float(__ushort_as_half(((const uint16_t*)(st + L::kVg))[r + 8 * k])) : 0.f;
#pragma unroll
            for (int u = 0; u < NB; ++u) {
              int sc = (ah[u][2 * k] << 8) + ah[u][2 * k + 1] + al[u][2 * k];
              sc += KB == 4 ? (al[u][2 * k + 1] + qsum[u]) >> 8 : al[u][2 * k + 1] >> 8;
              float v = (float)sc * (nk * fac[u]);
              if (p.cap_log2 > 0.f) {
                v *= p.cap2x;
                if (p.cap_log2 <= kCapFar) v = capped(v, p.cap_log2);
              }
              x[k][u] = v;
              n[k][u] = nv;
              ga[k][u] = ng;
            }
          }
          if (p.cap_log2 > kCapFar) {
            const float4 y = capped_far4(make_float4(x[0][0], x[0][NB - 1], x[1][0], x[1][NB - 1]), p.cap_log2);
            x[0][NB - 1] = y.y, x[1][NB - 1] = y.w;
            if (NB > 1) x[0][0] = y.x, x[1][0] = y.z;
          }
          if (p.slopes) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int u = 0; u < NB; ++u) x[k][u] = fmaf(slope[u], (float)(t + r + 8 * k - qpos[u]), x[k][u]);
          }
          if (absent != 0 || !((t >= open_lo && t + 16 <= open_hi) || t + 16 <= open_pre)) {
            const bool gone = (absent >> s) & 1;
            absent &= ~(1u << s);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int tt = t + r + 8 * k;
#pragma unroll
              for (int u = 0; u < NB; ++u)
                if (gone || tt >= t1 || !((tt <= qpos[u] && (p.window == 0 || tt > qpos[u] - p.window)) || tt < pre)) {
                  x[k][u] = -INFINITY;                           // not seen; its norms may be anything
                  n[k][u] = ga[k][u] = 0.f;
                }
            }
          }
          // largest score and largest value norm that a row sees (a norm that is not finite has no say)
          float top[NB], topn[NB];
          bool move = false;
#pragma unroll
          for (int u = 0; u < NB; ++u) {
            top[u] = fmaxf(x[0][u], x[1][u]);
            topn[u] = fmaxf(n[0][u], n[1][u]);
            move |= top[u] > ref[u] + kRowLazy || topn[u] > elim[u];
          }
          if (__any_sync(0xffffffffu, move)) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1)
#pragma unroll
              for (int u = 0; u < NB; ++u) {
                top[u] = fmaxf(top[u], __shfl_xor_sync(0xffffffffu, top[u], o));
                topn[u] = fmaxf(topn[u], __shfl_xor_sync(0xffffffffu, topn[u], o));
              }
            float f[NB];
#pragma unroll
            for (int u = 0; u < NB; ++u) {
              const float nr = fmaxf(ref[u], top[u]);
              const float fs = nr == ref[u] ? 1.f : ex2_approx(ref[u] - nr);   // 0 from the empty state
              ref[u] = nr;
              sum[u] *= fs;
              f[u] = fs;
              from[u] = nr == -INFINITY ? 0.f : nr;
              if (topn[u] > elim[u]) {
                // the norm limit: the next power of two (the exponent field of the largest norm, plus one)
                const float el = __int_as_float((__float_as_int(fminf(topn[u], 65504.f)) & 0x7F800000) + 0x00800000);
                f[u] *= elim[u] / el;
                elim[u] = el;
                room[u] = kRowRoom / el;
              }
              wsum[u] *= f[u];
              zsum[u] *= f[u];
            }
#pragma unroll
            for (int q = 0; q < MB; ++q)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if ((i & 1) < NB || SHARE) {
                  oc[q][i] *= f[i & 1 & (NB - 1)];
                  if (ALG2 && !SHARE) oz[q][i] *= f[i & 1 & (NB - 1)];
                }
          }
          uint32_t pc[2], pz[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float w[2] = {0.f, 0.f};
#pragma unroll
            for (int u = 0; u < NB; ++u) {
              const float e = ex2_approx(x[k][u] - from[u]);
              sum[u] += e;
              w[u] = e * (n[k][u] * room[u]);
              if (VB == 1) wsum[u] += w[u];
            }
            pc[k] = transpose8x8(half2_of(w[0], w[1]));
            if constexpr (ALG2) {
#pragma unroll
              for (int u = 0; u < NB; ++u) {
                w[u] *= ga[k][u];
                zsum[u] += w[u];
              }
              pz[k] = transpose8x8(SHARE ? half2_of(0.f, w[0]) : half2_of(w[0], w[1]));
            }
          }
          // ---- values ----------------------------------------------------------------------------------
          const int tk[4] = {2 * c, 2 * c + 1, 2 * c + 8, 2 * c + 9};
          auto plane = [&](int at, float (&o)[MB][4], uint32_t b0, uint32_t b1) {
            if constexpr (D == 128) {
              // lane r gets half r (coordinates 16 r ..) of tokens 2c, 2c + 1 and 2c + 8, 2c + 9
              uint32_t y0, y1;
              load_trans2(st_u32 + 4 * at + (lane & 15) * 16, y0, y1);
#pragma unroll
              for (int m = 0; m < 8; ++m) {
                const uint32_t lo1 = 0x00010001u << m, hi1 = 0x01000100u << m, one = m == 7 ? 0x3C003C00u : 0u;
                mma_f16(o[m], y0 & lo1, (y0 & hi1) ^ one, y1 & lo1, (y1 & hi1) ^ one, b0, b1);
              }
            } else {
              const uint32_t m0 = 0x00010001u << r, m1 = 0x01000100u << r, x1 = r == 7 ? 0x3C003C00u : 0u;
#pragma unroll
              for (int g = 0; g < G; ++g) {
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) w[k] = st[at + tk[k] * G + g];
                const uint32_t l01 = __byte_perm(w[0], w[1], 0x5410u), h01 = __byte_perm(w[0], w[1], 0x7632u);
                const uint32_t l23 = __byte_perm(w[2], w[3], 0x5410u), h23 = __byte_perm(w[2], w[3], 0x7632u);
                mma_f16(o[2 * g], l01 & m0, (l01 & m1) ^ x1, l23 & m0, (l23 & m1) ^ x1, b0, b1);
                mma_f16(o[2 * g + 1], h01 & m0, (h01 & m1) ^ x1, h23 & m0, (h23 & m1) ^ x1, b0, b1);
              }
            }
          };
          if constexpr (VB == 1) {
            plane(L::kVal, oc, pc[0], pc[1]);
          } else {
            // lane r: 16 coordinates of group r / 2 (d = 128), or 8 of group r / 4, of each of its four tokens
            const int grp = D == 128 ? r >> 1 : r >> 2, shift = D == 128 ? 2 * (r & 1) : r & 3;
            uint32_t w[4][VB], flip[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
#pragma unroll
              for (int i = 0; i < VB; ++i) w[k][i] = st[L::kVal + (tk[k] * G + grp) * VB + i] >> shift;
              flip[k] = magnitudes<VB>(w[k]);
            }
#pragma unroll
            for (int s4 = 0; s4 < D / 64; ++s4) {
              uint32_t x[4], neg[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                x[k] = nibbles<VB>(w[k], s4);
                neg[k] = VB == 4 ? (flip[k] >> s4) & 0x11111111u : 0u;
              }
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                uint32_t t[4][2];                                // [token][pair]: levels of coordinates 4 q + 2 pair, + 1
#pragma unroll
                for (int k = 0; k < 4; ++k) look_up<VB>(x[k] >> (16 * q), neg[k] >> (16 * q), vtab, t[k][0], t[k][1]);
#pragma unroll
                for (int h = 0; h < 2; ++h)
                  mma_f16(oc[4 * s4 + 2 * q + h], __byte_perm(t[0][h], t[1][h], 0x5410u), __byte_perm(t[0][h], t[1][h], 0x7632u),
                          __byte_perm(t[2][h], t[3][h], 0x5410u), __byte_perm(t[2][h], t[3][h], 0x7632u), pc[0], pc[1]);
              }
            }
          }
          if constexpr (SHARE) plane(L::kSign, oc, pz[0], pz[1]);
          else if constexpr (ALG2) plane(L::kSign, oz, pz[0], pz[1]);
        }

        // ---- merge the warps' states --------------------------------------------------------------------------
        cp_wait<0>();
        __syncthreads();                                         // the ring is free
        float* mg = (float*)smem;                                // [warp][row][parts D, ref, sum]
#pragma unroll
        for (int u = 0; u < NB; ++u) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            sum[u] += __shfl_xor_sync(0xffffffffu, sum[u], o);
            wsum[u] += __shfl_xor_sync(0xffffffffu, wsum[u], o);
            zsum[u] += __shfl_xor_sync(0xffffffffu, zsum[u], o);
          }
          float* dst = mg + (warp * RB + c + 4 * u) * RS;
          if (r == 0) {
            dst[PD] = ref[u];
            dst[PD + 1] = sum[u];
          }
          // a one-bit plane: bit place i of a 16-bit half is the fp16 value 2^-24 2^i (i < 10), 2^-14, 2^-13,
          // 2^-11, 2^-7, 2 (i = 10 .. 14), or the sign of 1 (i = 15); the inverse of that value
          auto inv_bit = [](int i) {
            return i < 10 ? __int_as_float((127 + 24 - i) << 23) : __int_as_float((127 + 15 - (1 << (i - 10))) << 23);
          };
          auto put = [&](float (&o)[MB][4], int odd, int at, bool one_bit, float total, float unit) {
            unit *= elim[u];
#pragma unroll
            for (int m = 0; m < MB; ++m)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float v = o[m][2 * h + odd];
                if (one_bit) {
                  const int i = D == 128 ? m + 8 * h : r + 8 * h;
                  dst[at + (D == 128 ? 16 * r : 16 * m) + i] = (i == 15 ? -v : fmaf(2.f * v, inv_bit(i), -total)) * unit;
                } else {
                  const int e = 2 * m + h;                       // as the look-up yields them
                  dst[at + (D == 128 ? 32 * (r >> 1) + 2 * (r & 1) + (e >> 3) + 4 * (e & 7) : 32 * (r >> 2) + (r & 3) + 4 * e)] = v * unit;
                }
              }
          };
          put(oc, u, 0, VB == 1, wsum[u], p.v_inv_unit / kRowRoom);
          if constexpr (SHARE) put(oc, 1, D, true, zsum[u], 1.f / kRowRoom);
          else if constexpr (ALG2) put(oz, u, D, true, zsum[u], 1.f / kRowRoom);
        }
        __syncthreads();
        const int live = min(RB, rows - row0);
        const int64_t slot = (int64_t)blockIdx.x + item;
        for (int e = threadIdx.x; e < live * PD; e += NT) {
          const int row = e / PD, i = e - row * PD;
          float best = -INFINITY;
#pragma unroll
          for (int w = 0; w < kRowWarps; ++w) best = fmaxf(best, mg[(w * RB + row) * RS + PD]);
          const float base_ref = best == -INFINITY ? 0.f : best;
          float o = 0.f, l = 0.f;
#pragma unroll
          for (int w = 0; w < kRowWarps; ++w) {
            const float* m = mg + (w * RB + row) * RS;
            const float f = ex2_approx(m[PD] - base_ref);
            o += f * m[i];
            l += f * m[PD + 1];
          }
          p.po[(slot * RB + row) * PD + i] = o;
          if (i == 0) p.ml[slot * RB + row] = make_float2(best, l);
        }
        __syncthreads();                                         // before the ring fills again
      }
    }
  }
}

template <int D, int KB, int VB, bool ALG2>
tq_status launch_rows(const PagedAttendParams& p, int ctas, cudaStream_t st) {
  auto go = [&](auto kern, size_t smem) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return cuda_fail(e, "tq_paged_attend: shared memory attribute");
    if ((e = launch_dependent(kern, dim3(ctas), 32 * kRowWarps, smem, st, p)) != cudaSuccess)
      return cuda_fail(e, "tq_paged_attend: launch");
    return TQ_OK;
  };
  return p.rows_per_item == 4 ? go(rows_kernel<D, KB, VB, ALG2, 1>, RowStage<D, KB, VB, ALG2, 1>::smem())
                              : go(rows_kernel<D, KB, VB, ALG2, 2>, RowStage<D, KB, VB, ALG2, 2>::smem());
}
template <int D, int KB>
tq_status launch_row_values(const PagedAttendParams& p, int vb, bool alg2, int ctas, cudaStream_t st) {
  if (alg2) switch (vb) {
      case 1: return launch_rows<D, KB, 1, true>(p, ctas, st);
      case 2: return launch_rows<D, KB, 2, true>(p, ctas, st);
      default: return launch_rows<D, KB, 3, true>(p, ctas, st);
    }
  switch (vb) {
    case 1: return launch_rows<D, KB, 1, false>(p, ctas, st);
    case 2: return launch_rows<D, KB, 2, false>(p, ctas, st);
    case 3: return launch_rows<D, KB, 3, false>(p, ctas, st);
    default: return launch_rows<D, KB, 4, false>(p, ctas, st);
  }
}
template <int D>
tq_status launch_row_keys(const PagedAttendParams& p, int kb, int vb, bool alg2, int ctas, cudaStream_t st) {
  switch (kb) {
    case 1: return launch_row_values<D, 1>(p, vb, alg2, ctas, st);
    case 2: return launch_row_values<D, 2>(p, vb, alg2, ctas, st);
    case 3: return launch_row_values<D, 3>(p, vb, alg2, ctas, st);
    default: return launch_row_values<D, 4>(p, vb, alg2, ctas, st);
  }
}

}  // namespace tq
