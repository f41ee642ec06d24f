// Handle of the paged packed cache (host): checks, and the fp16 levels of its codebooks.
//
// The attention multiplies with fp16 levels, but a codebook's levels are fp32. Any common factor can
// be taken out of them (it goes into the softmax scale, or the output), so it is chosen to make
// unit * level as close to an fp16 value as possible for all levels at once: among 512 factors of one
// octave the best one leaves a relative error of 0 (1 bit), 2^-16 to 2^-18 (2 bits), 2^-13 (3 bits) and
// 2^-12.4 to 2^-13 (4 bits) at d = 64 and 128, where a power of two leaves 2^-11.5 to 2^-14.
#include <cmath>
#include <cstring>
#include <string>

#include "tq_internal.h"

namespace tq {
namespace {

// nearest value with an 11-bit significand (an fp16 normal) by the splitting of Dekker / Veltkamp
float round11(float x) {
  volatile float t = x * 8193.0f;
  volatile float u = t - x;
  return t - u;
}

uint16_t half_bits(float x) {   // exact for fp16 normals
  uint32_t u;
  std::memcpy(&u, &x, 4);
  return (uint16_t)(((u >> 16) & 0x8000u) | ((((u >> 23) & 255u) - 112u) << 10) | ((u >> 13) & 0x3FFu));
}

float fit_levels(const float* c, int levels, uint16_t* half) {
  const int H = levels / 2;
  const float base = std::exp2(std::floor(std::log2(1.0f / c[levels - 1])) + 1.0f);   // largest level in [1, 2]
  float best = base, best_err = 1.0f;
  for (int k = 0; k < 512; ++k) {
    const float unit = base * (0.5f + k * (1.0f / 1024.0f));
    float err = 0.0f;
    for (int i = 0; i < H; ++i) {
      const float v = unit * c[H + i];
      err = std::fmax(err, std::fabs(round11(v) - v) / v);
    }
    if (err < best_err) {
      best_err = err;
      best = unit;
    }
  }
  if (H == 1) best = 1.0f / c[1];   // a single magnitude: 1
  for (int i = 0; i < levels; ++i) half[i] = half_bits(round11(best * c[i]));
  return best;
}

bool symmetric(const tq_codebook* cb) {
  const int L = cb->levels;
  for (int k = 0; k < L; ++k)
    if (cb->c[L - 1 - k] != -cb->c[k]) return false;
  for (int k = 0; k + 1 < L; ++k)
    if (cb->t[L - 2 - k] != -cb->t[k]) return false;
  for (int k = L / 2; k < L; ++k)
    if (!(cb->c[k] > 1e-3f && cb->c[k] <= 1.0f) || (k > L / 2 && !(cb->c[k] > cb->c[k - 1]))) return false;
  return true;
}

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" TQ_API tq_status tq_paged_kv_init(const tq_codebook* cb_k, const tq_codebook* cb_v, int32_t d, int32_t Hkv,
                                             int32_t page_size, int64_t num_pages, uint32_t* k_codes,
                                             uint16_t* k_norms, uint32_t* v_codes, uint32_t* v_signs,
                                             uint16_t* v_norms, uint16_t* v_gammas, tq_paged_kv* kv) {
  clear_error();
  const std::string f = "tq_paged_kv_init";
  if (!kv) return fail(TQ_ERR_INVALID_ARG, f + ": kv is NULL");
  std::memset(kv, 0, sizeof(*kv));
  if (!cb_k || !cb_v || !k_codes || !k_norms || !v_codes || !v_norms) return fail(TQ_ERR_INVALID_ARG, f + ": NULL pointer");
  if (!v_signs != !v_gammas) return fail(TQ_ERR_INVALID_ARG, f + ": v_signs and v_gammas go together");
  if (d != 64 && d != 128) return fail(TQ_ERR_UNSUPPORTED, f + ": d must be 64 or 128");
  if (Hkv < 1 || Hkv > 1024) return fail(TQ_ERR_UNSUPPORTED, f + ": Hkv must be in 1..1024");
  if (page_size < 16 || page_size > 1024 || (page_size & (page_size - 1)))
    return fail(TQ_ERR_UNSUPPORTED, f + ": page_size must be a power of two in 16..1024");
  if (num_pages < 1 || num_pages > 2147483647LL) return fail(TQ_ERR_INVALID_ARG, f + ": num_pages must be in 1..2^31 - 1");
  if (num_pages * Hkv > (((int64_t)1 << 32) - 1) / (page_size / 16))
    return fail(TQ_ERR_UNSUPPORTED, f + ": more than 2^36 token slots over all KV heads");
  for (const tq_codebook* cb : {cb_k, cb_v}) {
    if (cb->d != d || cb->bits < 1 || cb->bits > 4 || cb->levels != (1 << cb->bits))
      return fail(TQ_ERR_INVALID_ARG, f + ": codebook does not match d / has bad bits");
    if (!symmetric(cb)) return fail(TQ_ERR_INVALID_ARG, f + ": codebook is not symmetric");
  }
  if (v_signs && cb_v->bits > 3) return fail(TQ_ERR_UNSUPPORTED, f + ": Algorithm 2 values take a codebook of 1..3 bits");
  for (const void* p : {(void*)k_codes, (void*)k_norms, (void*)v_codes, (void*)v_signs, (void*)v_norms, (void*)v_gammas})
    if (!aligned16(p)) return fail(TQ_ERR_INVALID_ARG, f + ": pointers must be 16-byte aligned");
  kv->d = d;
  kv->Hkv = Hkv;
  kv->page_size = page_size;
  kv->v_alg = v_signs ? 2 : 1;
  kv->num_pages = num_pages;
  kv->k_codes = k_codes;
  kv->k_norms = k_norms;
  kv->v_codes = v_codes;
  kv->v_signs = v_signs;
  kv->v_norms = v_norms;
  kv->v_gammas = v_gammas;
  kv->k_bits = cb_k->bits;
  kv->v_bits = cb_v->bits;
  std::memcpy(kv->ck, cb_k->c, sizeof(kv->ck));
  std::memcpy(kv->tk, cb_k->t, sizeof(kv->tk));
  std::memcpy(kv->cv, cb_v->c, sizeof(kv->cv));
  std::memcpy(kv->tv, cb_v->t, sizeof(kv->tv));
  kv->k_unit = fit_levels(cb_k->c, cb_k->levels, kv->k_half);
  kv->v_unit = fit_levels(cb_v->c, cb_v->levels, kv->v_half);
  kv->ready = kPagedReady;
  return TQ_OK;
}
