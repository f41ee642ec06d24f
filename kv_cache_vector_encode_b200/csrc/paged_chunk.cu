// Attention of chunks (many query rows per KV head) over the paged packed cache: tq_paged_attend's path for
// sequences with more query rows per KV head than a decode step takes (paged_chunk_rows).
//
// Two kernels per group of (sequence, KV head) units:
//   open   decodes each 128-token tile once, K = n Pi^T c[idx] and V = n (Pi^T c[idx] + alpha gamma S^T (2 z - 1)),
//          by tensor-core products with the prepared Pi^T and S^T images, into fp16 tiles that are already the
//          shared-memory operands of the second kernel (K as [token][coordinate], V as [coordinate][token], both
//          K-major with the 128-byte swizzle);
//   chunk  out = softmax(scale q K^T, capped, biased, masked) V: tcgen05 products, 256 query rows per CTA.
// A chunk of 2048 queries reads every tile 32 times (four heads per KV head), so that unpacking inside the
// attention would cost more than the products; opened once, a tile is 64 KB that stay in L2 between its uses, and
// values of Algorithm 2 take one product instead of two. Query rows need no rotation, outputs neither.
//
// fp16 holds a tile because each tile has a power of two of its own for keys and for values (its largest norm):
// the keys' goes into the score factor. The values' exponent e is added to the scores of the softmax
// numerators, P = 2^(x + e - M) with the running reference M over x + e, and taken out of the denominators
// (2^-e sum P): no extra work per element, and P is rounded relative to what a row adds up.
// Norms down to about 2^-21 of a tile's largest keep the full precision of fp16; below, the last bits of values go.
//
// A record with a norm or residual norm that is not finite makes the rows that see it NaN; the tile holds zeros in
// its place, so that no other row meets it.
//
// Measured: a chunk of 2048 queries over 8192 tokens (32 heads over 8, V by Algorithm 2) 306 us, 774 TFLOP/s, of which
// opening takes 25 (512 tiles); twice 2048 over 16384 tokens with a cap 1615 us, 640 TFLOP/s. A step of 256 rows x 128
// tokens takes about 3700 cycles, five sixths of which the tensor cores' operand traffic needs, at 1.4 GHz under load.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "paged_attend.h"
#include "sm100.cuh"
#include "tq_internal.h"

namespace tq {
namespace {

constexpr int kTile = 128;            // tokens of a tile
constexpr int kHalf = kTile / 2;      // tokens of a step of the attention
constexpr int kCtaRows = 256;         // query rows of a CTA: two groups of 128
// How far (log2) a score may pass the reference before it moves: weights then stay below 2^14, within fp16. What is 2^14
// below the largest weight of a row no longer counts to a precision of 2^-25 of it.
constexpr float kLazy = 14.0f;
constexpr int kBits = 12;             // operands: norms below 1 after the tile's exponent, times 2^kBits

// What the attention needs to know of a tile besides its operands.
struct TileHead {
  float k_unit;                       // score = factor * k_unit * <q, K>
  float v_exp;                        // e
  float v_unit;                       // 2^-e
  uint32_t flags;                     // 1: some token is absent, 2: some token is not finite
  uint32_t present[4];                // bit per token
  uint32_t strange[4];                // bit per token: present, norm not finite
  uint32_t pad[4];
};
static_assert(sizeof(TileHead) == 64, "tile head");

struct ChunkParams {
  const int32_t* list;                // [0] count, then the sequences that take this path
  uint8_t* images;                    // [group][tiles][K, V][256 D bytes]
  TileHead* heads;                    // [group][tiles]
  int unit0, units, tiles;            // first unit of the group, units of the group, tiles of a unit
};

// Sequences with more than chunk_rows rows per KV head, in order.
__global__ void __launch_bounds__(256) list_kernel(const __grid_constant__ PagedAttendParams p, int32_t* list, int most) {
  __shared__ int warp_sum[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int base = 0;
  for (int b0 = 0; b0 < p.B; b0 += 256) {
    const int b = b0 + threadIdx.x;
    bool on = false;
    if (b < p.B) {
      const int q0 = p.q_start[b], q1 = p.q_start[b + 1];
      on = q0 >= 0 && q1 >= q0 && q1 <= p.total_q && q1 - q0 <= p.max_q && (int64_t)(q1 - q0) * p.g > p.chunk_rows;
    }
    const uint32_t vote = __ballot_sync(0xffffffffu, on);
    if (lane == 0) warp_sum[warp] = __popc(vote);
    __syncthreads();
    int at = base, all = 0;
    for (int w = 0; w < 8; ++w) {
      at += w < warp ? warp_sum[w] : 0;
      all += warp_sum[w];
    }
    at += __popc(vote & ((1u << lane) - 1));
    if (on && at < most) list[1 + at] = b;
    base += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) list[0] = min(base, most);
}

// One unit of the launch: its sequence and what its queries may see between them.
struct Unit {
  int b, hkv;
  PagedSeq sq;
  int64_t first, prefix, lo, hi;      // position of query 0; visible tokens [lo, hi)
};
__device__ __forceinline__ bool find_unit(const PagedAttendParams& p, const ChunkParams& c, int u, Unit& x) {
  const int slot = (c.unit0 + u) / p.Hkv;
  if (slot >= c.list[0]) return false;
  x.hkv = (c.unit0 + u) - slot * p.Hkv;
  x.b = c.list[1 + slot];
  x.sq = paged_seq(p, x.b);
  x.first = x.sq.first;
  x.prefix = paged_prefix(p, x.sq, x.b);
  paged_range(p, x.sq, x.first, x.first + x.sq.qn - 1, x.prefix, x.lo, x.hi);
  return true;
}

// ---- open -----------------------------------------------------------------------------------------------
template <int D, bool ALG2>
struct OpenLayout {
  static constexpr uint32_t kImg = 128 * D * 2, kMat = 0, kSgn = kImg, kTiles = kSgn + (ALG2 ? kImg : 0),
                            kS = kTiles + 3 * kImg, kInfo = kS + (ALG2 ? kImg : 0), kBar = kInfo + 2 * 128 * 4,
                            kTotal = kBar + 64 + 1024;
};
constexpr int kOpenThreads = 512;
__device__ __forceinline__ void bulk_wait_read1() { asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory"); }
constexpr int kOpenUnits = 256;       // units whose ranges a CTA keeps (those beyond are worked out for every tile)
struct OpenUnit {
  int b, hkv, t0, tiles, lo, hi;      // t0: first token of the first of `tiles` tiles; visible tokens [lo, hi)
};
__device__ __forceinline__ OpenUnit open_unit(const PagedAttendParams& p, const ChunkParams& c, int u) {
  Unit x;
  if (!find_unit(p, c, u, x) || x.hi <= x.lo) return OpenUnit{0, 0, 0, 0, 0, 0};
  const int t0 = (int)x.lo & ~(kTile - 1);
  return OpenUnit{x.b, x.hkv, t0, ((int)x.hi - t0 + kTile - 1) / kTile, (int)x.lo, (int)x.hi};
}

template <int D, int KB, int VB, bool ALG2>
__global__ void __launch_bounds__(kOpenThreads, 1)
    open_kernel(const __grid_constant__ PagedAttendParams p, const __grid_constant__ ChunkParams c) {
  using L = OpenLayout<D, ALG2>;
  constexpr int G = D / 32;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  float* info = (float*)(smem + L::kInfo);                       // [key factor, value factor][128]
  uint64_t* bar = (uint64_t*)(smem + L::kBar);                   // matrices loaded; products of the keys, of the values done
  uint32_t* tmem_slot = (uint32_t*)(bar + 3);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < 3; ++i) mbar_init(&bar[i], 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tk = *tmem_slot, tv = tk + 128;
  if (tid == 0) {   // 128-row images; at d = 64 the first column block alone
    mbar_arrive_expect_tx(&bar[0], (ALG2 ? 2u : 1u) * L::kImg);
    bulk_g2s(smem + L::kMat, p.img[2], L::kImg, &bar[0]);
    if (ALG2) bulk_g2s(smem + L::kSgn, p.img[4], L::kImg, &bar[0]);
  }
  uint32_t ktab[4], vtab[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) ktab[i] = p.ktab[i], vtab[i] = p.vtab[i];

  // this thread's (token, 32-coordinate group) of a tile, and its records
  const int tok = tid / G, grp = tid % G;
  const bool unpacker = tid < kTile * G;
  uint32_t kw[KB], vw[VB], sw = 0;
  uint16_t kn = 0, vn = 0, vg = 0;
  bool present = false;
  // A tile's page numbers are fetched two tiles ahead and its records one ahead, so that no turn waits for both.
  __shared__ OpenUnit units[kOpenUnits];
  for (int u = tid; u < min(c.units, kOpenUnits); u += kOpenThreads) units[u] = open_unit(p, c, u);
  __syncthreads();
  const int items = c.units * c.tiles;
  int next = items, next_t = 0;                                  // the tile after the one in hand; this thread's token of it
  bool next_want = false;                                        // some query may see the token (others have no say in the exponents)
  int next_page = 0, next_hkv = 0;
  auto locate = [&](int item) {                                  // the first tile from `item` on (in steps of the grid)
    next_want = false;
    for (; item < items; item += gridDim.x) {
      const int u = item / c.tiles, k = item - u * c.tiles;
      const OpenUnit x = u < kOpenUnits ? units[u] : open_unit(p, c, u);
      if (k >= x.tiles) continue;
      next_t = x.t0 + k * kTile + tok;
      next_want = unpacker && next_t >= x.lo && next_t < x.hi;
      next_hkv = x.hkv;
      if (next_want) next_page = p.table[(int64_t)x.b * p.max_pages + (next_t >> p.page_shift)];
      break;
    }
    next = item;
  };
  auto take = [&]() {
    present = false;
    kn = vn = vg = 0;
    sw = 0;
#pragma unroll
    for (int i = 0; i < KB; ++i) kw[i] = 0;
#pragma unroll
    for (int i = 0; i < VB; ++i) vw[i] = 0;
    if (!next_want) return;
    if (next_page >= 0 && next_page < p.num_pages) {
      const int64_t rec = (((int64_t)next_page * p.Hkv + next_hkv) << p.page_shift) + (next_t & ((1 << p.page_shift) - 1));
      present = true;
#pragma unroll
      for (int i = 0; i < KB; ++i) kw[i] = __ldg(p.k_codes + (rec * G + grp) * KB + i);
#pragma unroll
      for (int i = 0; i < VB; ++i) vw[i] = __ldg(p.v_codes + (rec * G + grp) * VB + i);
      kn = __ldg(p.k_norms + rec);
      vn = __ldg(p.v_norms + rec);
      if (ALG2) {
        sw = __ldg(p.v_signs + rec * G + grp);
        vg = __ldg(p.v_gammas + rec);
      }
    } else {
      report_bad_input(p.err);
    }
  };

  locate(blockIdx.x);
  int item = next;
  if (item < items) {
    take();
    locate(item + gridDim.x);
  }
  uint32_t phase = 0, turn = 0;
  bool loaded = false;
#pragma unroll 1
  while (item < items) {
    // ---- norms: factors of the tokens, exponents of the tile -------------------------------------------
    const float fk = __half2float(__ushort_as_half(kn)), fv = __half2float(__ushort_as_half(vn));
    const float fg = ALG2 ? __half2float(__ushort_as_half(vg)) : 0.f;
    const bool fine = fabsf(fk) < INFINITY && fabsf(fv) < INFINITY && fabsf(fg) < INFINITY;
    const float reach = fabsf(fv) * fmaxf(1.f, fabsf(fg));
    __shared__ uint32_t words[2][4];
    __shared__ int top[2];                                       // largest exponent fields: keys, values
    {
      // exponent fields (of positive floats these order like the values); a token's G threads agree
      const int ek = __reduce_max_sync(0xffffffffu, fine ? (__float_as_int(fabsf(fk)) >> 23) : 0);
      const int ev = __reduce_max_sync(0xffffffffu, fine ? (__float_as_int(reach) >> 23) : 0);
      if (tid < 8) words[tid >> 2][tid & 3] = 0;
      if (tid < 2) top[tid] = 0;
      if (tid == 0) bulk_wait_read1();                           // of the last tile's copies only the values' may still run
      __syncthreads();
      if (lane == 0 && unpacker) {
        atomicMax(&top[0], ek);
        atomicMax(&top[1], ev);
      }
      if (unpacker && grp == 0) {
        if (present) atomicOr(&words[0][tok >> 5], 1u << (tok & 31));
        if (present && !fine) atomicOr(&words[1][tok >> 5], 1u << (tok & 31));
      }
    }
    __syncthreads();
    // norms times 2^-(e - 127 + 1) are below 1 (an empty tile: any exponent will do)
    const int ek = top[0] == 0 ? 0 : top[0] - 126, ev = top[1] == 0 ? 0 : top[1] - 126;
    auto pow2 = [](int e) { return __int_as_float((127 + e) << 23); };   // |e| up to 60 here
    if (unpacker && grp == 0) {
      const bool use = present && fine;
      info[tok] = use ? fk * pow2(kBits - ek) * p.k_inv_unit : 0.f;
      info[128 + tok] = use ? fv * pow2(kBits - ev) * p.v_inv_unit : 0.f;
    }
    if (tid >= kOpenThreads - 8) {                               // the head, by eight threads of the last warp
      TileHead* h = c.heads + item;
      const int k = tid - (kOpenThreads - 8);
      (k < 4 ? h->present : h->strange)[k & 3] = words[k >> 2][k & 3];
      if (k == 0) {
        const bool all = (words[0][0] & words[0][1] & words[0][2] & words[0][3]) == 0xffffffffu;
        const bool odd = (words[1][0] | words[1][1] | words[1][2] | words[1][3]) != 0;
        *(float4*)h = make_float4(pow2(ek - kBits), (float)ev, pow2(-ev), __uint_as_float((all ? 0u : 1u) | (odd ? 2u : 0u)));
      }
    }
    // keys and values take two of three tiles in turn, so that the copies out of one turn run on into the next
    const uint32_t key_at = L::kTiles + (2 * turn % 3) * L::kImg, val_at = L::kTiles + ((2 * turn + 1) % 3) * L::kImg;
    ++turn;
    // ---- unpack into operands: the keys, whose product then runs while the values follow -------------------
    if (unpacker) {
      const uint32_t kf = magnitudes<KB>(kw);
#pragma unroll
      for (int s4 = 0; s4 < 4; ++s4) {
        const uint32_t xk = nibbles<KB>(kw, s4), nk = KB == 4 ? (kf >> s4) & 0x11111111u : 0u;
        uint32_t a[4];
        look_up<KB>(xk, nk, ktab, a[0], a[1]);
        look_up<KB>(xk >> 16, nk >> 16, ktab, a[2], a[3]);
        *(uint4*)(smem + key_at + sw128_offset(tok, (grp * 32 + s4 * 8) * 2, 128)) = make_uint4(a[0], a[1], a[2], a[3]);
      }
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    if (!loaded) {
      if (!__syncthreads_and(mbar_wait(&bar[0], 0, p.err, kDevTimeoutLoad, abort_flag))) break;
      loaded = true;
    }
    tc_fence_after();
    const uint32_t m = smem_u32(smem + L::kMat), sg = smem_u32(smem + L::kSgn);
    if (warp == 0 && elect_one_sync()) {
      const uint32_t k = smem_u32(smem + key_at);
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const uint32_t at = (ks >> 2) * 16384u + (ks & 3) * 32u;
        mma_f16_ss(tk, desc_kmajor_sw128(k + at), desc_kmajor_sw128(m + at), idesc_f16_f32(128, D), ks > 0);
      }
      mma_commit(&bar[1]);
    }
    __syncwarp();
    if (unpacker) {
      const uint32_t vf = magnitudes<VB>(vw);
      uint32_t sg_lo = 0, sg_hi = 0;
      if (ALG2) {   // alpha gamma in units of the levels, with either sign, as byte tables (z = 0: negative)
        const uint32_t h = __half_as_ushort(__float2half_rn(present && fine ? p.sign_unit * fg : 0.f));
        sg_lo = (h & 255u) * 0x0101u;
        sg_hi = ((h >> 8) ^ 0x80u) | ((h >> 8) << 8);
      }
#pragma unroll
      for (int s4 = 0; s4 < 4; ++s4) {
        const uint32_t xv = nibbles<VB>(vw, s4), nv = VB == 4 ? (vf >> s4) & 0x11111111u : 0u;
        uint32_t b[4];
        look_up<VB>(xv, nv, vtab, b[0], b[1]);
        look_up<VB>(xv >> 16, nv >> 16, vtab, b[2], b[3]);
        const uint32_t off = sw128_offset(tok, (grp * 32 + s4 * 8) * 2, 128);
        *(uint4*)(smem + val_at + off) = make_uint4(b[0], b[1], b[2], b[3]);
        if (ALG2) {
          const uint32_t z = (sw >> s4) & 0x11111111u;
          uint32_t o[4];
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t lb = __byte_perm(sg_lo, 0u, z >> (16 * half)), hb = __byte_perm(sg_hi, 0u, z >> (16 * half));
            o[2 * half] = __byte_perm(lb, hb, 0x5140u);
            o[2 * half + 1] = __byte_perm(lb, hb, 0x7362u);
          }
          *(uint4*)(smem + L::kS + off) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
    }
    fence_proxy_async_smem();
    __syncthreads();
    if (warp == 0 && elect_one_sync()) {
      const uint32_t v = smem_u32(smem + val_at), s = smem_u32(smem + L::kS);
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const uint32_t at = (ks >> 2) * 16384u + (ks & 3) * 32u;
        mma_f16_ss(tv, desc_kmajor_sw128(m + at), desc_kmajor_sw128(v + at), idesc_f16_f32(128, 128), ks > 0);
        if (ALG2) mma_f16_ss(tv, desc_kmajor_sw128(sg + at), desc_kmajor_sw128(s + at), idesc_f16_f32(128, 128), 1);
      }
      mma_commit(&bar[2]);
    }
    __syncwarp();
    const int done = item;
    item = next;
    if (item < items) {
      take();
      locate(item + gridDim.x);
    }
    if (!__syncthreads_and(mbar_wait(&bar[1], phase, p.err, kDevTimeoutMma, abort_flag))) break;
    tc_fence_after();
    // ---- products into fp16 tiles, in place of the operands -----------------------------------------------
    const int quarter = warp & 3, part = warp >> 2;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    {
      constexpr int W = D / 4;                                   // columns of a warp
      const int row = quarter * 32 + lane;
      const float f = info[row];
#pragma unroll
      for (int c0 = 0; c0 < W; c0 += 16) {
        uint32_t r[16];
        tmem_ld16(tk + lane_base + part * W + c0, r);
        tmem_ld_wait();
        uint32_t h[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const __half2 x = __floats2half2_rn(__uint_as_float(r[2 * i]) * f, __uint_as_float(r[2 * i + 1]) * f);
          h[i] = *reinterpret_cast<const uint32_t*>(&x);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
          *(uint4*)(smem + key_at + sw128_offset(row, (part * W + c0 + 8 * i) * 2, 128)) =
              make_uint4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
      }
    }
    if (!__syncthreads_and(mbar_wait(&bar[2], phase, p.err, kDevTimeoutMma, abort_flag))) break;
    phase ^= 1;
    tc_fence_after();
    if (quarter * 32 < D) {
      const int row = quarter * 32 + lane;
#pragma unroll
      for (int c0 = 0; c0 < 32; c0 += 16) {
        uint32_t r[16];
        tmem_ld16(tv + lane_base + part * 32 + c0, r);
        tmem_ld_wait();
        uint32_t h[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 f = *(const float4*)&info[128 + part * 32 + c0 + 4 * i];
          const __half2 x = __floats2half2_rn(__uint_as_float(r[4 * i]) * f.x, __uint_as_float(r[4 * i + 1]) * f.y);
          const __half2 y = __floats2half2_rn(__uint_as_float(r[4 * i + 2]) * f.z, __uint_as_float(r[4 * i + 3]) * f.w);
          h[2 * i] = *reinterpret_cast<const uint32_t*>(&x);
          h[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&y);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
          *(uint4*)(smem + val_at + sw128_offset(row, (part * 32 + c0 + 8 * i) * 2, D)) =
              make_uint4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
      }
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0) {
      uint8_t* dst = c.images + (size_t)done * 2 * L::kImg;
      bulk_s2g(dst, smem + key_at, L::kImg);
      bulk_commit();
      bulk_s2g(dst + L::kImg, smem + val_at, L::kImg);
      bulk_commit();
    }
  }
  if (tid == 0) {
    if (!loaded) mbar_wait(&bar[0], 0, p.err, kDevTimeoutLoad, abort_flag);   // no copy outlives the block
    bulk_wait0();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(*tmem_slot, 256);
}

// ---- chunk ----------------------------------------------------------------------------------------------
// Warps 0-3 and 4-7: the softmax of query rows 0-127 and 128-255, thread = row; warp 8 copies tiles; warps 9 and 10
// issue the products, one for each group; warp 9 owns TMEM. TMEM per group: scores of two half tiles (64 columns each;
// the weights P take the place of the first 32 as fp16 pairs), output O (D columns).
// A group's step i is a half tile of 64 tokens: scores S(i), softmax, O += P(i) V(i). S(i + 2) follows PV(i) into the
// same columns, so that the next step's scores are there when a softmax ends, and the softmax warps never wait for
// a product that waits for them. (Whole tiles leave TMEM for one score buffer per group: the chain softmax, PV, next
// scores, softmax then takes 4200 cycles per 256 x 128 scores, of which the tensor cores work 2048. Half tiles
// take 3700: a 128 x 64 score product takes as long as a 128 x 128 one, its queries' way out of shared memory.)
template <int D>
struct ChunkLayout {
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr uint32_t kImg = 128 * D * 2, kQ = 0, kRing = 2 * kImg, kBar = kRing + kStages * kImg,
                            kTotal = kBar + 256 + 1024;
};
constexpr int kChunkThreads = 352;
constexpr int kChunkCols = 512;

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,"
      "%30,%31}, [%32];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]),
        "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]),
        "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// Products with descriptors in two words, of which only the low one (the address) changes: K-major operands with the
// 128-byte swizzle, as desc_kmajor_sw128 makes them.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_low(uint32_t smem_addr) { return (smem_addr >> 4) | (1u << 16); }
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint32_t a_low, uint32_t b_low, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_low), "r"(b_low), "r"(idesc), "r"(accumulate), "r"(kDescHigh)
      : "memory");
}
// A in TMEM: fp16 pairs of its K in a column.
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_low, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_low), "r"(idesc), "r"(accumulate), "r"(kDescHigh)
      : "memory");
}

// A wait that is expected to be short: polls before it settles down to the bounded wait.
__device__ __forceinline__ bool wait_soon(uint64_t* bar, uint32_t phase, uint32_t* err, uint32_t code, volatile uint32_t* abort) {
  bool ok = false;
#pragma unroll 1
  for (int i = 0; i < 64 && !ok; ++i) ok = mbar_try_wait(bar, phase);
  return __all_sync(0xffffffffu, ok || mbar_wait_slow(bar, phase, err, code, abort));
}

// S_FULL, P_FULL: [group][half]
enum CBars { Q_FULL = 0, KV_FULL = 2, KV_EMPTY = 10, S_FULL = 18, P_FULL = 22, PV_DONE = 26, O_FULL = 28, CNBARS = 30 };

// the n lowest bits of 32
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u); }

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// 2^x of two numbers below 2^7 without the special-function unit, which bounds the softmax (8 cycles per warp and
// exponential): x = i + r by rounding, 2^r on [-1/2, 1/2] by a cubic fitted to the least largest relative error (7.5e-5,
// a third of an fp16 rounding), i into the exponent. Below 2^-126 the result is 2^-126.
__device__ __forceinline__ float2 exp2_poly(float2 x) {
  x.x = fmaxf(x.x, -126.f);
  x.y = fmaxf(x.y, -126.f);
  const float2 t = add2(x, both(12582912.f));                    // 1.5 2^23: the integer in the low bits
  const float2 r = add2(x, mul2(add2(t, both(-12582912.f)), both(-1.f)));
  float2 y = fma2(both(0.05517167f), r, both(0.24261113f));
  y = fma2(y, r, both(0.69326099f));
  y = fma2(y, r, both(0.99992807f));
  return make_float2(__int_as_float(__float_as_int(y.x) + (__float_as_int(t.x) << 23)),
                     __int_as_float(__float_as_int(y.y) + (__float_as_int(t.y) << 23)));
}

// Which of 16 pairs take the polynomial: three of eight balance the two units.
__device__ __forceinline__ constexpr bool by_poly(int k) { return (k & 7) == 1 || (k & 7) == 4 || (k & 7) == 6; }

// tanh(u) = u + u^3 q(u^2) with q of degree 2 for |u| <= 0.6 (largest error of tanh 9e-7) and of degree 4 for
// |u| <= 1 (3.2e-7), fitted to the least largest error.
template <int N, int DEG>
__device__ __forceinline__ void tanh_poly(float (&s)[N], float fu) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float2 u = mul2(make_float2(s[i], s[i + 1]), both(fu)), w = mul2(u, u);
    float2 q;
    if (DEG == 2) {
      q = fma2(both(-0.04072624f), w, both(0.13050765f));
      q = fma2(q, w, both(-0.33314597f));
    } else {
      q = fma2(both(-0.00298308f), w, both(0.01653281f));
      q = fma2(q, w, both(-0.05142535f));
      q = fma2(q, w, both(0.13275615f));
      q = fma2(q, w, both(-0.33328670f));
    }
    const float2 x = fma2(mul2(q, w), u, u);
    s[i] = x.x, s[i + 1] = x.y;
  }
}

// Scores of a row's consecutive tokens, the first of them `ahead` of the query: what they times the factor returned are
// in the log2 domain, capped and biased. A cap costs two more special-function results per score than the
// softmax's one; where no score of the warp reaches the cap, a polynomial takes their place.
template <int N>
__device__ __forceinline__ float shape(const PagedAttendParams& p, float (&s)[N], float f, float slope, int ahead) {
  if (p.cap_log2 > 0.f) {
    const float fu = f * (0.5f * p.cap2x * 0.69314718f);         // u = score / cap, both in one domain
    float m4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < N; ++i) m4[i & 3] = fmaxf(m4[i & 3], fabsf(s[i]));
    const float most = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * fu;
    if (__all_sync(0xffffffffu, most <= 0.6f)) {
      tanh_poly<N, 2>(s, fu);
    } else if (__all_sync(0xffffffffu, most <= 1.f)) {
      tanh_poly<N, 4>(s, fu);
    } else if (p.cap_log2 > kCapFar) {                           // one row reaches the cap, others may be far below
#pragma unroll
      for (int i = 0; i < N; ++i) s[i] = capped_far(s[i] * f * p.cap2x, 1.f);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) s[i] = capped(s[i] * f * p.cap2x, 1.f);
    }
    f = p.cap_log2;
  }
  if (p.slopes) {
    const float near = slope * (float)ahead;
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = fmaf(s[i], f, fmaf(slope, (float)i, near));
    f = 1.f;
  }
  return f;
}

template <int D>
__global__ void __launch_bounds__(kChunkThreads, 1)
    chunk_kernel(const __grid_constant__ PagedAttendParams p, const __grid_constant__ ChunkParams c) {
  using L = ChunkLayout<D>;
  constexpr int NS = L::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint64_t* bar = (uint64_t*)(smem + L::kBar);
  uint32_t* tmem_slot = (uint32_t*)(bar + CNBARS);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  Unit x;
  if (!find_unit(p, c, blockIdx.x, x)) return;
  const int rows = x.sq.qn * p.g, row0 = (gridDim.y - 1 - blockIdx.y) * kCtaRows;
  if (row0 >= rows) return;
  int64_t lo, hi;
  paged_range(p, x.sq, x.first + row0 / p.g, x.first + (min(rows, row0 + kCtaRows) - 1) / p.g, x.prefix, lo, hi);
  const int64_t unit_t0 = x.lo & ~(int64_t)(kTile - 1);
  const int tile0 = (int)((lo - unit_t0) / kTile);
  const int n = hi > lo ? (int)((hi - unit_t0 + kTile - 1) / kTile) - tile0 : 0;
  const bool two = rows > row0 + 128;
  const size_t item0 = (size_t)blockIdx.x * c.tiles + tile0;

  if (tid == 0) {
    for (int u = 0; u < 2; ++u) {
      mbar_init(&bar[Q_FULL + u], 4);
      mbar_init(&bar[PV_DONE + u], 1);
      mbar_init(&bar[O_FULL + u], 1);
      for (int k = 0; k < 2; ++k) {
        mbar_init(&bar[S_FULL + 2 * u + k], 1);
        mbar_init(&bar[P_FULL + 2 * u + k], 4);
      }
    }
    for (int s = 0; s < NS; ++s) {
      mbar_init(&bar[KV_FULL + s], 1);
      mbar_init(&bar[KV_EMPTY + s], two ? 2 : 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, kChunkCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;

  if (warp == 8) {
    if (elect_one_sync()) {
      int k = 0;
      for (; k < 2 * n; ++k) {                                   // K and V of tile k / 2 in turn
        const int s = k % NS;
        if (!mbar_wait(&bar[KV_EMPTY + s], ((k / NS) & 1) ^ 1, p.err, kDevTimeoutSync, abort_flag)) break;
        mbar_arrive_expect_tx(&bar[KV_FULL + s], L::kImg);
        bulk_g2s(smem + L::kRing + s * L::kImg, c.images + (2 * item0 + k) * L::kImg, L::kImg, &bar[KV_FULL + s]);
      }
      if (*abort_flag)                                           // no copy outlives the block
        for (int i = max(0, k - NS); i < k; ++i) mbar_wait(&bar[KV_FULL + i % NS], (i / NS) & 1, nullptr, 0, nullptr);
    }
    __syncwarp();
  } else if (warp >= 9) {
    // ---- products of group u ---------------------------------------------------------------------------------
    const int u = warp - 9;
    const uint32_t ring = desc_low(smem_u32(smem + L::kRing)), q = desc_low(smem_u32(smem + L::kQ) + u * L::kImg);
    const uint32_t ts = tbase + 128 * u, to = tbase + 256 + D * u;
    const bool leader = elect_one_sync();
    auto wait = [&](int b, int ph, uint32_t code) { return wait_soon(&bar[b], ph & 1, p.err, code, abort_flag); };
    // scores of half tile i; the second half is the last use of the keys' stage
    auto scores = [&](int i) {
      const int half = i & 1, stage = (i & ~1) % NS;
      const uint32_t b = ring + stage * (L::kImg >> 4) + half * (8192 >> 4);
      if (leader) {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t at = ((ks >> 2) * 16384u + (ks & 3) * 32u) >> 4;
          mma_ss(ts + 64 * half, q + at, b + at, idesc_f16_f32(128, 64), ks > 0);
        }
        mma_commit(&bar[S_FULL + 2 * u + half]);
        if (half) mma_commit(&bar[KV_EMPTY + stage]);
      }
      __syncwarp();
    };
    if (n > 0 && (u == 0 || two)) {
      bool ok = wait(KV_FULL, 0, kDevTimeoutLoad) && wait(Q_FULL + u, 0, kDevTimeoutSync);
      tc_fence_after();
      if (ok) {
        scores(0);
        scores(1);
      }
#pragma unroll 1
      for (int i = 0; ok && i < 2 * n; ++i) {
        const int half = i & 1, kv = i | 1, kn = (i & ~1) + 2;   // stages: this tile's V, the next one's K
        const bool more = i + 2 < 2 * n;
        if (!half) ok = wait(KV_FULL + kv % NS, kv / NS, kDevTimeoutLoad) && (!more || wait(KV_FULL + kn % NS, kn / NS, kDevTimeoutLoad));
        ok = ok && wait(P_FULL + 2 * u + half, i >> 1, kDevTimeoutSync);
        if (!ok) break;
        tc_fence_after();
        const uint32_t b = ring + (kv % NS) * (L::kImg >> 4) + half * (D * 8);
        if (leader) {
#pragma unroll
          for (int ks = 0; ks < kTile / 32; ++ks)
            mma_ts(to, ts + 64 * half + 8 * ks, b + 2 * ks, idesc_f16_f32(128, D), i > 0 || ks > 0);
          mma_commit(&bar[PV_DONE + u]);
          if (i + 1 == 2 * n) mma_commit(&bar[O_FULL + u]);
          if (half) mma_commit(&bar[KV_EMPTY + kv % NS]);
        }
        __syncwarp();
        if (more) scores(i + 2);
      }
    }
  } else if (warp < 4 || two) {
    const int u = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tbase + lane_base + 128 * u, to = tbase + lane_base + 256 + D * u;
    const int row = row0 + 128 * u + r;
    const bool on = row < rows;
    const int jq = on ? row / p.g : 0, h = x.hkv * p.g + (on ? row - jq * p.g : 0);
    const int pos = (int)x.first + jq;
    // ---- this row's query: fp16 times a power of two (exact for what lies within 2^-26 of its largest) -----
    float fac;
    bool fine;
    {
      const uint4* src = (const uint4*)(p.q + (int64_t)(x.sq.q0 + jq) * p.q_stride + (int64_t)h * D);
      uint4 w[D / 8];
      uint32_t most = 0;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        w[i] = on ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
        const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) most = max(most, max(v[k] & 0x7FFFu, (v[k] >> 16) & 0x7FFFu));
      }
      fine = most < 0x7F80u;
      const int e = min(max((int)(most >> 7), 20), 230);
      const float up = __int_as_float((254 + 11 - e) << 23);
      fac = p.scale_log2 * __int_as_float((e - 11) << 23);
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const __half2 x2 = __floats2half2_rn(__uint_as_float(v[k] << 16) * up, __uint_as_float(v[k] & 0xFFFF0000u) * up);
          o[k] = *reinterpret_cast<const uint32_t*>(&x2);
        }
        *(uint4*)(smem + L::kQ + u * L::kImg + sw128_offset(r, i * 16, 128)) = make_uint4(o[0], o[1], o[2], o[3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[Q_FULL + u]);
    }
    const float slope = p.slopes ? p.slopes[h] * kLog2e : 0.f;
    const bool shaped = p.cap_log2 > 0.f || p.slopes != nullptr;
    float ref = -INFINITY, sum = 0.f;
    // the group's first and last position, for tiles that every row sees whole
    const int pmin = (int)x.first + (row0 + 128 * u) / p.g, pmax = (int)x.first + (min(rows, row0 + 128 * u + 128) - 1) / p.g;
    const int pre = (int)x.prefix;
    const TileHead* heads = c.heads + item0;
    int t0 = (int)unit_t0 + tile0 * kTile;                       // first token of the half tile
    bool ok = true;
    float4 hd = n > 0 ? *(const float4*)&heads[0] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int i = 0; i < 2 * n; ++i, t0 += kHalf) {
      const int half = i & 1;
      const TileHead* head = heads + (i >> 1);
      const float4 cur = hd;
      if (half && i + 1 < 2 * n) hd = *(const float4*)(head + 1);
      const uint32_t flags = __float_as_uint(cur.w);
      ok = wait_soon(&bar[S_FULL + 2 * u + half], (i >> 1) & 1, p.err, kDevTimeoutMma, abort_flag);
      if (!ok) break;
      tc_fence_after();
      float s[kHalf];
#pragma unroll
      for (int k = 0; k < kHalf; k += 32) tmem_ld32(ts + 64 * half + k, s + k);
      tmem_ld_wait();
      float f = fmaxf(fac * cur.x, 1.2e-38f);                    // not zero: it meets infinite scores
      const bool whole = flags == 0 && ((t0 + kHalf - 1 <= pmin && (p.window == 0 || t0 > pmax - p.window)) || t0 + kHalf <= pre);
      if (shaped) f = shape(p, s, f, slope, t0 - pos);
      if (!whole) {
#pragma unroll
        for (int w = 0; w < kHalf / 32; ++w) {
          // seen: present and ((t <= pos and t > pos - window) or t < prefix)
          const int at = t0 + 32 * w;
          uint32_t m = below(min(pos - at, 31) + 1);             // pos may be 2^31 - 1
          if (p.window > 0) m &= ~below(pos - p.window + 1 - at);
          m |= below(pre - at);
          m = on ? m & __ldg(&head->present[2 * half + w]) : 0u;
          if ((flags & 2u) && (m & __ldg(&head->strange[2 * half + w]))) sum = __int_as_float(0x7FC00000);
#pragma unroll
          for (int k = 0; k < 32; ++k) s[32 * w + k] = (m >> k) & 1 ? s[32 * w + k] : -INFINITY;
        }
      }
      float m8[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) m8[k] = fmaxf(s[k], s[k + 8]);
#pragma unroll
      for (int t = 16; t < kHalf; t += 16)
#pragma unroll
        for (int k = 0; k < 8; ++k) m8[k] = fmaxf(fmaxf(m8[k], s[t + k]), s[t + k + 8]);
      const float top = fmaf(fmaxf(fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3])), fmaxf(fmaxf(m8[4], m8[5]), fmaxf(m8[6], m8[7]))),
                             f, cur.y);
      if (__any_sync(0xffffffffu, top > ref + kLazy)) {
        const float nr = fmaxf(ref, top);
        const float g = nr == ref ? 1.f : ex2_approx(ref - nr);  // 0 from the empty state
        ref = nr;
        sum *= g;
        if (i > 0) {
          // step i - 1's product; that of step i - 2 is done, since the scores of step i came after it
          ok = wait_soon(&bar[PV_DONE + u], (i - 1) & 1, p.err, kDevTimeoutMma, abort_flag);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < D; k += 32) {
            float o[32];
            tmem_ld32(to + k, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= g;
            tmem_st16(to + k, reinterpret_cast<const uint32_t*>(o));
            tmem_st16(to + k + 16, reinterpret_cast<const uint32_t*>(o) + 16);
          }
        }
      }
      // weights, in fp16 into the place of the scores
      const float2 off = both(cur.y - (ref == -INFINITY ? 0.f : ref)), f2 = both(f);
      float2 l2[2] = {both(0.f), both(0.f)};
#pragma unroll
      for (int t = 0; t < kHalf; t += 32) {
        uint32_t w[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const float2 x = fma2(make_float2(s[t + 2 * k], s[t + 2 * k + 1]), f2, off);
          const float2 e = by_poly(k) ? exp2_poly(x) : make_float2(ex2_approx(x.x), ex2_approx(x.y));
          l2[k & 1] = add2(l2[k & 1], e);
          const __half2 h2 = __floats2half2_rn(e.x, e.y);
          w[k] = *reinterpret_cast<const uint32_t*>(&h2);
        }
        tmem_st16(ts + 64 * half + t / 2, w);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[P_FULL + 2 * u + half]);
      sum = fmaf((l2[0].x + l2[0].y) + (l2[1].x + l2[1].y), cur.z, sum);
    }
    // ---- out = O / sum ------------------------------------------------------------------------------------
    // (a barrier of its own: PV_DONE shows the parity of a phase, which may be that of the product before last)
    if (n > 0 && ok) ok = wait_soon(&bar[O_FULL + u], 0, p.err, kDevTimeoutMma, abort_flag);
    if (ok) {
      tc_fence_after();
      if (n > 0 && !(fine && fabsf(slope) < INFINITY)) sum = __int_as_float(0x7FC00000);   // the cap and the polynomial may have hidden it
      // a query before the first token sees nothing, whatever it holds (the polynomial's weights are not quite 0 there)
      if (pos < 0 && pre <= 0) sum = 0.f;
      const float inv = sum == 0.f ? 0.f : __int_as_float((127 - kBits) << 23) / sum;
      uint4* dst = (uint4*)(p.out + ((int64_t)(x.sq.q0 + jq) * p.Hq + h) * D);
#pragma unroll
      for (int i = 0; i < D; i += 16) {
        uint32_t o[16];
        if (n > 0) {
          tmem_ld16(to + i, o);
          tmem_ld_wait();
        }
        uint32_t w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float a = sum == 0.f ? 0.f : __uint_as_float(o[2 * k]) * inv, b = sum == 0.f ? 0.f : __uint_as_float(o[2 * k + 1]) * inv;
          const __nv_bfloat162 h2 = __floats2bfloat162_rn(a, b);
          w[k] = *reinterpret_cast<const uint32_t*>(&h2);
        }
        if (on) {
          dst[i / 8] = make_uint4(w[0], w[1], w[2], w[3]);
          dst[i / 8 + 1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tbase, kChunkCols);
}

// ---- host -----------------------------------------------------------------------------------------------

template <int D, int KB, int VB, bool ALG2>
tq_status launch_open(const PagedAttendParams& p, const ChunkParams& c, cudaStream_t st) {
  auto kern = open_kernel<D, KB, VB, ALG2>;
  constexpr int smem = OpenLayout<D, ALG2>::kTotal;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return cuda_fail(e, "tq_paged_attend: shared memory attribute");
  const int64_t items = (int64_t)c.units * c.tiles;
  kern<<<(unsigned)std::min<int64_t>(items, sm_count()), kOpenThreads, smem, st>>>(p, c);
  if ((e = cudaGetLastError()) != cudaSuccess) return cuda_fail(e, "tq_paged_attend: launch");
  return TQ_OK;
}
template <int D, int KB>
tq_status launch_open_values(const PagedAttendParams& p, const ChunkParams& c, int vb, bool alg2, cudaStream_t st) {
  if (alg2) switch (vb) {
      case 1: return launch_open<D, KB, 1, true>(p, c, st);
      case 2: return launch_open<D, KB, 2, true>(p, c, st);
      default: return launch_open<D, KB, 3, true>(p, c, st);
    }
  switch (vb) {
    case 1: return launch_open<D, KB, 1, false>(p, c, st);
    case 2: return launch_open<D, KB, 2, false>(p, c, st);
    case 3: return launch_open<D, KB, 3, false>(p, c, st);
    default: return launch_open<D, KB, 4, false>(p, c, st);
  }
}
template <int D>
tq_status launch_unit_group(const PagedAttendParams& p, const ChunkParams& c, const tq_paged_kv* kv, int row_blocks, cudaStream_t st) {
  const bool alg2 = kv->v_alg == 2;
  tq_status s;
  switch (kv->k_bits) {
    case 1: s = launch_open_values<D, 1>(p, c, kv->v_bits, alg2, st); break;
    case 2: s = launch_open_values<D, 2>(p, c, kv->v_bits, alg2, st); break;
    case 3: s = launch_open_values<D, 3>(p, c, kv->v_bits, alg2, st); break;
    default: s = launch_open_values<D, 4>(p, c, kv->v_bits, alg2, st);
  }
  if (s != TQ_OK) return s;
  auto kern = chunk_kernel<D>;
  constexpr int smem = ChunkLayout<D>::kTotal;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return cuda_fail(e, "tq_paged_attend: shared memory attribute");
  kern<<<dim3(c.units, row_blocks), kChunkThreads, smem, st>>>(p, c);
  if ((e = cudaGetLastError()) != cudaSuccess) return cuda_fail(e, "tq_paged_attend: launch");
  return TQ_OK;
}

size_t tile_bytes(int d) { return (size_t)2 * 128 * d * 2; }

}  // namespace

// Opened tiles take 2 x 256 d bytes each, so a call opens its units in groups of at most this many bytes of tiles
// (one unit at least).
constexpr int64_t kOpenBytes = (int64_t)1 << 30;

PagedChunkPlan paged_chunk_plan(const tq_paged_kv* kv, int B, int Hq, int64_t total_q, int max_q, int64_t max_kv, int window) {
  PagedChunkPlan P{};
  const int g = Hq / kv->Hkv;
  P.slots = (int)std::min<int64_t>(B, total_q * g / (paged_chunk_rows(B * kv->Hkv) + 1));
  if (max_kv == 0) max_kv = 1;
  const int64_t units = std::max<int64_t>((int64_t)P.slots * kv->Hkv, 1), all = (max_kv + kTile - 1) / kTile;
  const int64_t most = std::min<int64_t>(units, std::max<int64_t>(1, kOpenBytes / (all * (int64_t)tile_bytes(kv->d)))) * all;
  // with a window a unit's queries see its span and their own; the tiles are then shared among more units
  int64_t tiles = all;
  if (window > 0) tiles = std::min<int64_t>(all, ((int64_t)window + max_q + kTile - 1) / kTile + 1);
  P.tiles = (int)tiles;
  P.group = (int)std::min<int64_t>(units, most / tiles);
  P.row_blocks = (int)(((int64_t)max_q * g + kCtaRows - 1) / kCtaRows);
  auto al = [](size_t v) { return (v + 255) / 256 * 256; };
  size_t off = 0;
  P.list = off; off += al((size_t)(P.slots + 1) * 4);
  P.heads = off; off += al((size_t)most * sizeof(TileHead));
  P.images = off; off += al((size_t)most * tile_bytes(kv->d));
  P.bytes = off;
  return P;
}

tq_status paged_chunk_launch(const PagedAttendParams& p, const tq_paged_kv* kv, const PagedChunkPlan& P, uint8_t* ws,
                             cudaStream_t st) {
  ChunkParams c{};
  int32_t* list = (int32_t*)(ws + P.list);
  c.list = list;
  c.heads = (TileHead*)(ws + P.heads);
  c.images = ws + P.images;
  c.tiles = P.tiles;
  list_kernel<<<1, 256, 0, st>>>(p, list, P.slots);
  const int units = P.slots * kv->Hkv;
  for (c.unit0 = 0; c.unit0 < units; c.unit0 += P.group) {
    c.units = std::min(P.group, units - c.unit0);
    const tq_status s = kv->d == 128 ? launch_unit_group<128>(p, c, kv, P.row_blocks, st)
                                     : launch_unit_group<64>(p, c, kv, P.row_blocks, st);
    if (s != TQ_OK) return s;
  }
  return TQ_OK;
}

}  // namespace tq
