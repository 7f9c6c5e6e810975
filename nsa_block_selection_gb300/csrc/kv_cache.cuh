// The paged cache of keys and values as the kernels see it, and the host checks
// that its entry points share.
//
// A cache is `pages` pages of `page_size` token rows for each of G heads. Token
// position p of sequence b has row p % page_size of page table[b, p / page_size];
// an entry outside [0, pages) (-1, say) is a page that the sequence does not
// have. 16 bits: rows of D entries, any strides over page, token and head.
// 4 bits: rows of D / 2 bytes (even entries in the low four bits) and a pair of
// bf16 (step, low) for every (page, head, token): an entry is low + step * code.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "nsa_sel_attn.h"
#include "rope.cuh"

namespace nsa {

// A step below this is stored as 0, and the row is its low alone: a step's
// reciprocal, and the logarithm that the attention folds it into p by, stay
// far from the ends of fp32.
constexpr float kLeastStep = 8.673617379884035e-19f;  // 2^-60

struct KvPages {
  uint8_t *k, *v;
  uint32_t *ks, *vs;             // 4 bits: (step, low) pairs [pages, G, page_size]
  int64_t kp, kt, kh, vp, vt, vh;  // strides in bytes over page, token and head
  const int32_t* table;
  int pages, shift, cols;  // page_size = 1 << shift
};

// The page of position `at` (>= 0) of sequence b, or -1.
__device__ __forceinline__ int page_of(const KvPages& c, int b, int64_t at) {
  const int64_t col = at >> c.shift;
  if (col >= c.cols) return -1;
  const int id = __ldg(c.table + static_cast<int64_t>(b) * c.cols + col);
  return id >= 0 && id < c.pages ? id : -1;
}

// Checks of a cache and its page table; fills `c`. D and G are checked by the caller.
inline int take_cache(const nsa_kv_cache* kv, const int32_t* table, int64_t cols, int64_t B,
                      int64_t G, int64_t D, bool written, KvPages* c) {
  if (!kv || !kv->k || !kv->v || !table) return NSA_ERR_NULL;
  if (kv->bits != 16 && kv->bits != 4) return NSA_ERR_DTYPE;
  const int64_t lim = int64_t(1) << 31;
  if (kv->pages <= 0 || kv->pages >= lim || cols <= 0 || cols >= lim) return NSA_ERR_SHAPE;
  if (kv->page_size < 16 || kv->page_size > 1024 || (kv->page_size & (kv->page_size - 1)) != 0)
    return NSA_ERR_PAGE_SIZE;
  if (cols * kv->page_size > int64_t(1) << 30) return NSA_ERR_SHAPE;
  if (B > 0 && cols > (int64_t(1) << 40) / B) return NSA_ERR_SHAPE;
  if (!aligned(kv->k, 16) || !aligned(kv->v, 16) || !aligned(table, 4)) return NSA_ERR_ALIGN;
  c->k = static_cast<uint8_t*>(kv->k);
  c->v = static_cast<uint8_t*>(kv->v);
  c->ks = c->vs = nullptr;
  c->table = table;
  c->pages = static_cast<int>(kv->pages);
  c->cols = static_cast<int>(cols);
  c->shift = 0;
  while ((int64_t(1) << c->shift) < kv->page_size) ++c->shift;
  if (kv->bits == 4) {
    if (!kv->k_scale || !kv->v_scale) return NSA_ERR_NULL;
    if (!aligned(kv->k_scale, 16) || !aligned(kv->v_scale, 16)) return NSA_ERR_ALIGN;
    c->ks = static_cast<uint32_t*>(kv->k_scale);
    c->vs = static_cast<uint32_t*>(kv->v_scale);
    c->kh = c->vh = D / 2;
    c->kt = c->vt = G * (D / 2);
    c->kp = c->vp = kv->page_size * c->kt;
    return NSA_OK;
  }
  const int64_t extent[3] = {kv->pages, kv->page_size, G};
  int64_t s[6];
  for (int i = 0; i < 6; ++i) {
    s[i] = (i < 3 ? kv->k_strides : kv->v_strides)[i % 3];
    if (s[i] < 0 || s[i] > (int64_t(1) << 36)) return NSA_ERR_SHAPE;
    if (s[i] % 8 != 0) return NSA_ERR_ALIGN;
    if (written && s[i] == 0 && extent[i % 3] > 1) return NSA_ERR_SHAPE;
  }
  c->kp = 2 * s[0], c->kt = 2 * s[1], c->kh = 2 * s[2];
  c->vp = 2 * s[3], c->vt = 2 * s[4], c->vh = 2 * s[5];
  return NSA_OK;
}

}  // namespace nsa
