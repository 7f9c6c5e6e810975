// What the kernels of the attention over pages share: the problem, what a row tile
// sees and has to read, and the CTAs' shares of it.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "kv_cache.cuh"
#include "nsa_sel_attn.h"

namespace nsa {

constexpr int kPaWarps = 4;
constexpr int kPaThreads = 32 * kPaWarps;
constexpr int kPaTile = 16;       // keys of a tile
constexpr int kPaSlotRows = 128;  // (head, key) rows of a 4-bit slot
constexpr int kPaItems = 512;     // row tiles of a batch that shares are formed of
constexpr int kPaSms = 152;
constexpr int kPaMostPerSm = 4;
// What an item costs beside its keys, in keys: its positions, pages and first
// copies one after the other, and the joining of the warps, some 4 us where 16
// keys take 0.3. (Shares by keys alone: a CTA with seven short items took 34 us
// where the others took 13.)
constexpr int kPaItemCost = 320;
// Keys of an item that is never cut, and where there is an item for every SM. (A token
// of 64 + 8 heads over 300 keys: whole 9.0 us, cut 10.8; over 500 10.9 and 10.3. 48
// sequences of 32 + 4 heads, 192 items: 1028 keys each whole 22 us, cut 26; 1500 each 28
// and 32, up to 1500 23 and 20, up to 3000 41 and 33.)
constexpr int kPaWhole = 512, kPaWholeMany = 2048;
// The same of paged_attn_tc_kernel, whose steps are faster. (512: a prompt of 4096
// tokens 179 us instead of 167, 2 x 65 tokens after 8900 others 30 instead of 32; 1024:
// 170 and 33.)
constexpr int kTcItemCost = 768;
// Keys of a share at least, that cost among them. (448: a token of 64 + 8 heads of 128
// over 1000 keys 14.3 us instead of 11.1, two over 3000 in 4 bits 18.4 instead of 13.6;
// 64: 10.6 and 15.8.)
constexpr int kPaLeast = 128;
// A row's reference is moved where an x exceeds the largest at its last move by more
// than kPaSlack. It lies kPaLift below that largest where p is rounded to fp16, so that
// p reaches 2^15 and what is small beside it keeps seven bits more (without, keys of
// 2^-26 of the largest were in the sum l and 0 in O); bf16 has the range anyway.
constexpr float kPaSlack = 8.0f, kPaLift = 7.0f;
template <bool F16>
constexpr float kPaBelow = F16 ? kPaLift : 0.0f;

// First key of a tile that is not there, past every position.
constexpr int kNoKey = 0x7ffffff0, kPaFar = 0x7fffffe0;

struct PagedProblem {
  KvPages c;
  const uint8_t* q;
  int64_t qb, qm, qh;  // element strides
  uint16_t* o;         // [B, M, H, D]
  float* lse;          // [B, H, M] or NULL
  const int32_t* pos;
  int64_t pos_b;
  // [2 ctas][rows of an item][D] (many rows: [2 ctas][D / 8][rows][8], as the rows are
  // a thread's each), then [2 ctas][rows of an item][2] (reference, sum)
  float* piece;
  int64_t* count;     // [items + 1]: running steps of the items, and a share's steps
  int B, M, H, G, hpg, rows, tiles, items;  // rows of a KV head, row tiles, B * tiles
  int left, sinks, ctas;
  int heads_item, groups;  // KV heads of an item, G / heads_item
  int step_shift;          // keys of a step: 16; 4 bits: 128 / heads_item
  int item_cost;           // kPaItemCost in steps
  int split;               // 4 bits: copies that a step's keys take (small pages)
  float sl2;
  bool cut, many;  // many rows: paged_attn_tc_kernel
};

// What a row tile of a sequence has to read: n steps of 1 << shift keys, of which
// the first `st` start at key 0 and the others `jump` steps further on.
struct PaSpan {
  int n, st, jump, shift;
  int lo_pos, hi_pos;  // smallest and largest position of its queries
  __device__ __forceinline__ int key(int t) const { return (t < st ? t : t + jump) << shift; }
};

// A query's position (padding as -1; one at the end of int32 as kPaFar: kNoKey is past
// them all).
__device__ __forceinline__ int pa_position(const PagedProblem& p, int b, int m) {
  return max(min(__ldg(p.pos + b * p.pos_b + m), kPaFar), -1);
}

// WARP: a whole warp calls it, a position a lane; else a thread by itself, several
// loads at once.
template <bool WARP>
__device__ __forceinline__ PaSpan pa_span(const PagedProblem& p, int b, int rt, int rows_tile) {
  const int r0 = rt * rows_tile, r1 = min(r0 + rows_tile, p.rows) - 1;
  PaSpan s{0, 0, 0, p.step_shift, 0x7fffffff, -1};
  const int m0 = r0 / p.hpg, m1 = r1 / p.hpg;
#pragma unroll 8
  for (int m = m0 + (WARP ? static_cast<int>(threadIdx.x) & 31 : 0); m <= m1; m += WARP ? 32 : 1) {
    const int at = pa_position(p, b, m);
    s.lo_pos = min(s.lo_pos, at < 0 ? 0x7fffffff : at);
    s.hi_pos = max(s.hi_pos, at);
  }
  if constexpr (WARP) {
    if (m1 > m0) {
      s.lo_pos = __reduce_min_sync(kFull, s.lo_pos);
      s.hi_pos = __reduce_max_sync(kFull, s.hi_pos);
    } else {
      s.lo_pos = __shfl_sync(kFull, s.lo_pos, 0);
      s.hi_pos = __shfl_sync(kFull, s.hi_pos, 0);
    }
  }
  if (s.hi_pos < 0) return s;
  const int last = min(s.hi_pos, (p.c.cols << p.c.shift) - 1) >> s.shift;  // (at most 2^30 tokens)
  const int first = (p.left < s.lo_pos ? s.lo_pos - p.left : 0) >> s.shift;
  s.st = min((p.sinks + (1 << s.shift) - 1) >> s.shift, last + 1);
  if (first <= s.st) {
    s.n = last + 1;
  } else if (first > last) {  // the window lies behind the table's end
    s.n = s.st;
  } else {
    s.jump = first - s.st;
    s.n = s.st + last - first + 1;
  }
  return s;
}

// What the queries of a row tile see of a key.
struct PaSight {
  int lo_pos, hi_pos, left, sinks;
  // no query sees it (its row may hold anything), but for keys in a gap between windows
  __device__ __forceinline__ bool nobody(int key) const {
    return key > hi_pos || (key < lo_pos - left && key >= sinks);
  }
  // every query sees the tile from n0 on
  __device__ __forceinline__ bool all(int n0) const {
    return n0 + kPaTile - 1 <= lo_pos && (n0 >= hi_pos - left || n0 + kPaTile <= sinks);
  }
  // no query sees a key of the tile
  __device__ __forceinline__ bool nothing(int n0) const {
    return n0 > hi_pos || (n0 + kPaTile - 1 < lo_pos - left && n0 >= sinks);
  }
  // Some key from the first window to the last query may be in no window. (A key up to
  // lo_pos is in lo_pos's; one after it in hi_pos's, where that reaches lo_pos.)
  __device__ __forceinline__ bool gaps() const { return hi_pos - lo_pos > left; }
  __device__ __forceinline__ bool hidden(int key, int pos) const {
    return key > pos || (key < pos - left && key >= sinks);
  }
};

// A CTA's share of the steps of all items, KV-head groups innermost.
struct PaShare {
  int64_t begin, end;  // steps
  int64_t at;          // the first step of the item that holds `begin`
  int item, group;
};

// `count` [items + 1] and `sums` (one of each warp) are shared memory; all threads of
// a CTA of kThreads.
template <int kThreads>
__device__ __forceinline__ PaShare pa_share(const PagedProblem& p, int rows_tile, int* count,
                                            int* sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // the running count of the items' steps, a run of items to a thread
  const int run = (p.items + kThreads - 1) / kThreads;
  const int i0 = min(static_cast<int>(threadIdx.x) * run, p.items), i1 = min(i0 + run, p.items);
  int mine = 0;
  for (int i = i0; i < i1; ++i) {
    count[i] = mine;
    const int n = pa_span<false>(p, i / p.tiles, i % p.tiles, rows_tile).n;
    mine += n > 0 ? n + p.item_cost : 0;
  }
  int scan = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kFull, scan, o);
    if (lane >= o) scan += v;
  }
  if (lane == 31) sums[warp] = scan;
  __syncthreads();
  int before = scan - mine;
  for (int w = 0; w < warp; ++w) before += sums[w];
  for (int i = i0; i < i1; ++i) count[i] += before;
  if (i0 < i1 && i1 == p.items) count[p.items] = before + mine;
  __syncthreads();
  const int64_t all = static_cast<int64_t>(count[p.items]) * p.groups;
  int64_t per = (all + p.ctas - 1) / p.ctas;
  per = max(per, static_cast<int64_t>(kPaLeast >> p.step_shift));
  PaShare s{min(all, static_cast<int64_t>(blockIdx.x) * per), 0, 0, 0, 0};
  s.end = min(all, s.begin + per);
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i <= p.items; i += kThreads) p.count[i] = count[i];
    if (threadIdx.x == 0) p.count[p.items + 1] = per;
  }
  if (s.begin < s.end) {  // the item that holds step `begin`
    int lo = 0, hi = p.items - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (static_cast<int64_t>(count[mid]) * p.groups <= s.begin) lo = mid;
      else hi = mid - 1;
    }
    s.item = lo;
    const int n = count[lo + 1] - count[lo];  // (its cost among them)
    const int64_t first = static_cast<int64_t>(count[lo]) * p.groups;
    s.group = static_cast<int>((s.begin - first) / n);
    s.at = first + static_cast<int64_t>(s.group) * n;
  }
  return s;
}

// Items without a step, dealt to the CTAs: zeros. `count`: as of pa_share.
template <int D>
__device__ __forceinline__ void pa_zeros(const PagedProblem& p, int rows_tile, const int* count) {
  for (int item = blockIdx.x; item < p.items; item += gridDim.x) {
    if (count[item + 1] != count[item]) continue;
    const int b = item / p.tiles, r0 = (item - b * p.tiles) * rows_tile;
    const int rows = min(rows_tile, p.rows - r0);
    const int64_t all = static_cast<int64_t>(rows) * p.G * (D / 8);
    for (int64_t i = threadIdx.x; i < all; i += blockDim.x) {
      const int x = static_cast<int>(i / (D / 8)), g = x / rows, rw = r0 + x - g * rows;
      const int mq = rw / p.hpg, h = g * p.hpg + rw - mq * p.hpg;
      reinterpret_cast<uint4*>(p.o + ((static_cast<int64_t>(b) * p.M + mq) * p.H + h) *
                                         D)[i % (D / 8)] = make_uint4(0, 0, 0, 0);
      if (i % (D / 8) == 0 && p.lse != nullptr)
        p.lse[(static_cast<int64_t>(b) * p.H + h) * p.M + mq] = -INFINITY;
    }
  }
}

// What a V row enters the exponent with: its step, or, for a row without one (all
// codes are 0, the row is its low), a number so far below low that the keys beside it
// lose nothing that O has, and so near that p' low / step stays in fp32. Such a row's
// p' is not multiplied with its codes (p low is its part of O). (With 1 for all of
// them p' of small rows beside a row of zeros fell among fp16's subnormals: 500 keys
// of std 0.002 and one of zeros with 0.96 of the weight, O 34 % off.)
__device__ __forceinline__ float pa_step(float step, float low) {
  return step == 0.f ? fmaxf(kLeastStep, fabsf(low) * 0x1p-40f) : step;
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2_approx(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float pa_lse(float ref, float sum) {
  return sum == 0.f ? -INFINITY : (ref + __log2f(sum)) * 0.69314718055994530942f;
}

// Rows of the tiles of paged_attn_tc_kernel: 128, or as many as whole queries have.
inline int tc_rows_of_tile(int64_t hpg) { return static_cast<int>(128 / hpg * hpg); }

// The tensor-core kernel for many rows (paged_attn_tc.cu); fills p.ctas.
int launch_paged_tc(PagedProblem& p, const nsa_kv_cache* kv, int64_t D, bool bf16,
                    cudaStream_t st);
int paged_tc_read_and_clear_status(unsigned int* value);

}  // namespace nsa
