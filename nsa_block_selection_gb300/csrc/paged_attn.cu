// Attention of new tokens over a paged cache of keys and values, 16-bit or
// 4-bit, for sm_103a.
//
// Query (b, m) at position p sees key j of its sequence iff j <= p, and
// j >= p - left or j < sinks (the first tokens, which stay visible behind a
// window), and the page of j is there. With x_j = scale log2(e) q.k_j:
//   O = sum_j 2^(x_j - r) v_j / l,  l = sum_j 2^(x_j - r),
//   LSE = ln 2 (r + log2 l),
// r a reference that follows the largest x (by steps of 8: p <= 2^8). One pass
// over the keys; x, p, sums and O are fp32, p is rounded to 16 bits for the
// product with V.
//
// Rows. A row tile is 8 or 16 of the M H/G (query, head) rows of a KV head, the
// N of the products: S^T (16 keys x rows) = K Q^T and O^T (D x rows) += V^T P^T
// (mma.sync m16n8k16). A decoding step has 8 rows or fewer, of which a 128-row
// tcgen05 tile would be 1/16 full; what bounds the call is the cache's bytes.
//
// Keys. A warp takes 16-key tiles, which lie in one page each, through a ring of
// its own of shared-memory slots that lane 0 fills with TMA copies; a CTA's four
// warps take its tiles in turn and are joined in shared memory at the end of an
// item (row tile and KV head). The tiles of all items are dealt to the CTAs in
// equal, contiguous shares, whatever the lengths of the sequences: positions
// are on the device, so every CTA forms the running count of the items' tiles
// for itself. An item that a share's border cuts leaves fp32 pieces, which
// paged_attn_join_kernel adds in a fixed order: equal calls give equal bits.
//
// 4 bits. k = low + step c gives q.k = step (q.c) + low sum(q): the codes
// themselves enter the product, as fp16 subnormals (c 2^-24, or 16 c 2^-24 for
// the upper four bits of a byte, which Q's entries are divided by 16 for): a
// mask, or a shift and a mask, makes two entries. Q's rows are scaled by a power
// of two into fp16's range. For V, 2^(x + log2 step - r) c is summed, so r
// follows x + log2(step), and p = that / step; sum p low is added at the end.

#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "common.cuh"
#include "kv_cache.cuh"
#include "nsa_sel_attn.h"
#include "ptx.cuh"
#include "status.cuh"

namespace nsa {
namespace {

constexpr int kPaWarps = 4;
constexpr int kPaThreads = 32 * kPaWarps;
constexpr int kPaTile = 16;       // keys of a tile
constexpr int kPaItems = 1024;    // row tiles of a batch that shares are formed of
constexpr int kPaSms = 152;
constexpr int kPaLeast = 8;       // tiles of a share at least
constexpr float kPaSlack = 8.0f;

template <int D, bool Q4, int NT>
struct PaCfg {
  static constexpr int kStages = Q4 ? 4 : 2;
  static constexpr int kPerSm = Q4 && (D == 64 || NT == 1) ? 4 : 3;  // CTAs
  static constexpr int kRowBytes = Q4 ? D / 2 : 2 * D;
  static constexpr int kKv = kPaTile * kRowBytes;          // one K or V tile
  static constexpr int kScales = Q4 ? 2 * kPaTile * 4 : 0;  // (step, low) of K, of V
  static constexpr int kBytes = 2 * kKv + kScales;         // copied for a tile
  static constexpr int kSlot = Q4 ? 2 * kKv : kBytes;
  static constexpr int kOffScale = kPaWarps * kStages * kSlot;
  static constexpr int kPad = D + 4;  // row stride of the joined O, in floats
  static constexpr int kJoin = kPaWarps * 8 * NT * kPad * 4;
  static constexpr int kRing = kOffScale + kPaWarps * kStages * kScales;
  static constexpr int kOffStat = kRing > kJoin ? kRing : kJoin;  // 2 floats a warp and row
  static constexpr int kOffBar = kOffStat + kPaWarps * 8 * NT * 8;
  static constexpr int kOffKey = kOffBar + kPaWarps * kStages * 8;
  static constexpr int kOffCount = kOffKey + kPaWarps * kStages * 4;
  static constexpr int kSmem = kOffCount + (kPaItems + 1) * 4 + 1024;
};

struct PagedProblem {
  KvPages c;
  const uint8_t* q;
  int64_t qb, qm, qh;  // element strides
  uint16_t* o;         // [B, M, H, D]
  float* lse;          // [B, H, M] or NULL
  const int32_t* pos;
  int64_t pos_b;
  float* piece;       // [2 gridDim.x][8 NT][D], then [..][8 NT][2] (reference, sum)
  int64_t* count;     // [items + 1]: running tiles of the items, and a share's tiles
  int B, M, H, G, hpg, rows, tiles, items;  // rows of a KV head, row tiles, B * tiles
  int left, sinks, ctas;
  float sl2;
  bool cut;
};

// What a row tile of a sequence has to read: n 16-key tiles, of which the first
// `st` start at key 0 and the others `jump` tiles further on.
struct PaSpan {
  int n, st, jump;
  int lo_pos, hi_pos;  // smallest and largest position of its queries
};

__device__ __forceinline__ PaSpan pa_span(const PagedProblem& p, int b, int rt, int rows_tile) {
  const int r0 = rt * rows_tile, r1 = min(r0 + rows_tile, p.rows) - 1;
  PaSpan s{0, 0, 0, 0x7fffffff, -1};
  const int m1 = r1 / p.hpg;
  for (int m = r0 / p.hpg; m <= m1; ++m) {
    const int at = __ldg(p.pos + b * p.pos_b + m);
    if (at < 0) continue;
    s.lo_pos = min(s.lo_pos, at);
    s.hi_pos = max(s.hi_pos, at);
  }
  if (s.hi_pos < 0) return s;
  const int last = min(s.hi_pos, (p.c.cols << p.c.shift) - 1) / kPaTile;  // (at most 2^30 tokens)
  const int first = (p.left < s.lo_pos ? s.lo_pos - p.left : 0) / kPaTile;
  s.st = min((p.sinks + kPaTile - 1) / kPaTile, last + 1);
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

template <bool BF16>
__device__ __forceinline__ float half_of(uint32_t v, int hi) {
  const uint32_t h = hi ? v >> 16 : v & 0xffffu;
  if constexpr (BF16) return __uint_as_float(h << 16);
  return __half2float(__ushort_as_half(static_cast<unsigned short>(h)));
}

// MMA row i of a 4-bit tile is key swap(i): with the lowest two bits swapped the
// loads of V by pairs of keys meet no bank twice.
__device__ __forceinline__ int swap01(int i) { return (i & ~3) | ((i & 1) << 1) | ((i >> 1) & 1); }

template <int D, bool BF16, bool Q4, int NT>
__global__ void __launch_bounds__(kPaThreads, PaCfg<D, Q4, NT>::kPerSm)
    paged_attn_kernel(const PagedProblem p, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV) {
  using C = PaCfg<D, Q4, NT>;
  constexpr int kRowsTile = 8 * NT;
  constexpr int KS = D / 16;  // k steps of S
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const gbase = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, c = lane & 3;
  int* const count = reinterpret_cast<int*>(gbase + C::kOffCount);
  int* const keys = reinterpret_cast<int*>(gbase + C::kOffKey) + warp * C::kStages;
  const uint32_t bars = base + C::kOffBar + warp * C::kStages * 8;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kPaWarps * C::kStages; ++i) mbar_init(base + C::kOffBar + 8 * i, 1);
    fence_mbar_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  // the share of this CTA: tiles [begin, end) of all items, KV heads innermost
  int64_t begin = 0, end = 0, per = 0;
  int item = 0, head = 0;  // (sequence, row tile), KV head
  int64_t at = 0;          // the item's first tile
  if (p.cut) {
    // the running count of the items' tiles, a run of items to a thread
    int* const sums = reinterpret_cast<int*>(gbase + C::kOffStat);
    const int run = (p.items + kPaThreads - 1) / kPaThreads;
    const int i0 = min(static_cast<int>(threadIdx.x) * run, p.items), i1 = min(i0 + run, p.items);
    int mine = 0;
    for (int i = i0; i < i1; ++i) {
      count[i] = mine;
      mine += pa_span(p, i / p.tiles, i % p.tiles, kRowsTile).n;
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
    const int64_t all = static_cast<int64_t>(count[p.items]) * p.G;
    per = (all + p.ctas - 1) / p.ctas;
    if (per < kPaLeast) per = kPaLeast;
    begin = min(all, static_cast<int64_t>(blockIdx.x) * per);
    end = min(all, begin + per);
    if (blockIdx.x == 0) {
      for (int i = threadIdx.x; i <= p.items; i += kPaThreads) p.count[i] = count[i];
      if (threadIdx.x == 0) p.count[p.items + 1] = per;
    }
    if (begin < end) {  // the item that holds tile `begin`
      int lo = 0, hi = p.items - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (static_cast<int64_t>(count[mid]) * p.G <= begin) lo = mid;
        else hi = mid - 1;
      }
      item = lo;
      const int n = count[item + 1] - count[item];
      head = static_cast<int>((begin - static_cast<int64_t>(count[item]) * p.G) / n);
      at = static_cast<int64_t>(count[item]) * p.G + static_cast<int64_t>(head) * n;
    }
  } else {
    item = blockIdx.x / p.G;
    head = blockIdx.x - item * p.G;
    __syncthreads();
  }
  const uint64_t policy = p.tiles > 1 ? l2_policy_evict_last() : l2_policy_evict_first();
  bool failed = false;
  uint32_t issued = 0, done = 0;  // tiles of this warp, over all items
  for (bool more = !p.cut || begin < end; more;) {
    const int b = item / p.tiles, rt = item - b * p.tiles;
    const PaSpan sp = pa_span(p, b, rt, kRowsTile);
    const int t0 = p.cut ? static_cast<int>(max(begin - at, static_cast<int64_t>(0))) : 0;
    const int t1 = p.cut ? static_cast<int>(min(end - at, static_cast<int64_t>(sp.n))) : sp.n;

    // ---- this warp's tiles t0 + warp, + kPaWarps, ...: pages of 32 at a time
    int ahead = t0 + warp, left_in = 0, page_id = -1;
    auto issue = [&]() -> bool {  // the next tile that has a page, into its slot
      for (;;) {
        if (ahead >= t1) return false;
        if (left_in == 0) {
          const int t = ahead + lane * kPaWarps;
          page_id = -1;
          if (t < t1) {
            const int64_t key = static_cast<int64_t>(t < sp.st ? t : t + sp.jump) * kPaTile;
            page_id = page_of(p.c, b, key);
          }
          left_in = 32;
        }
        const int page = __shfl_sync(kFull, page_id, 32 - left_in);
        const int t = ahead;
        ahead += kPaWarps;
        --left_in;
        if (page < 0) continue;
        const int key = (t < sp.st ? t : t + sp.jump) * kPaTile;
        if (lane == 0) {
          const int s = issued % C::kStages;
          const uint32_t bar = bars + 8 * s;
          const uint32_t dst = base + (warp * C::kStages + s) * C::kSlot;
          const int off = key & ((1 << p.c.shift) - 1);
          keys[s] = key;
          mbar_arrive_expect_tx(bar, C::kBytes);
          if constexpr (Q4) {
            tma_load_4d(dst, &tmK, bar, 0, head, off, page, policy);
            tma_load_4d(dst + C::kKv, &tmV, bar, 0, head, off, page, policy);
            const uint32_t sc = base + C::kOffScale + (warp * C::kStages + s) * C::kScales;
            const int64_t so = ((page * static_cast<int64_t>(p.G) + head) << p.c.shift) + off;
            bulk_load(sc, p.c.ks + so, kPaTile * 4, bar);
            bulk_load(sc + kPaTile * 4, p.c.vs + so, kPaTile * 4, bar);
          } else {
#pragma unroll
            for (int a = 0; a < D / 64; ++a) {
              tma_load_4d(dst + a * kBoxBytes, &tmK, bar, a * 64, head, off, page, policy);
              tma_load_4d(dst + C::kKv + a * kBoxBytes, &tmV, bar, a * 64, head, off, page, policy);
            }
          }
        }
        ++issued;
        return true;
      }
    };
    if (!failed) {
      for (int s = 0; s < C::kStages; ++s)
        if (!issue()) break;
    }

    // ---- the rows: Q as B operand, and the positions of this lane's columns
    uint32_t qf[NT][KS][2];
    int col_pos[NT][2];
    float ka[NT][2], kb[NT][2];  // 4 bits: x = step dot ka + low kb
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = rt * kRowsTile + nt * 8 + r;
      const int m = row / p.hpg;
      const bool in = row < p.rows;
      const uint32_t* src = reinterpret_cast<const uint32_t*>(
          p.q + 2 * (b * p.qb + m * p.qm + (head * p.hpg + row - m * p.hpg) * p.qh));
      if constexpr (!Q4) {
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          qf[nt][k][0] = in ? src[8 * k + c] : 0u;
          qf[nt][k][1] = in ? src[8 * k + 4 + c] : 0u;
        }
      } else {
        // this lane's D / 4 entries, from (D / 4) c on
        constexpr int W = D / 32;  // words of a row of codes that a lane holds
        uint4 v[W];
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) {
          v[j] = in ? reinterpret_cast<const uint4*>(src)[c * W + j] : make_uint4(0, 0, 0, 0);
          const uint32_t u[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            top = fmaxf(top, fmaxf(fabsf(half_of<BF16>(u[i], 0)), fabsf(half_of<BF16>(u[i], 1))));
        }
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
        // 2^e: the largest entry between 2^13 and 2^14 (a row that is not
        // finite, or zero, as it is)
        int e = 0;
        if (top > 0.f && top < INFINITY)
          e = min(13 - (static_cast<int>(__float_as_uint(top) >> 23) - 127), 100);
        const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) {
          const uint32_t u[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
          float f[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            f[i] = __half2float(__float2half_rn(half_of<BF16>(u[i >> 1], i & 1) * up));
            sum += f[i];
          }
          // entries (0, 4), (1, 5) / 16 and (2, 6), (3, 7) / 16: the order of
          // the codes under the masks
          constexpr float k16 = 1.f / 16.f;
          qf[nt][2 * j][0] = pack_half2(f[0], f[4]);
          qf[nt][2 * j][1] = pack_half2(f[1] * k16, f[5] * k16);
          qf[nt][2 * j + 1][0] = pack_half2(f[2], f[6]);
          qf[nt][2 * j + 1][1] = pack_half2(f[3] * k16, f[7] * k16);
        }
        sum += __shfl_xor_sync(kFull, sum, 1);
        sum += __shfl_xor_sync(kFull, sum, 2);
        const float back = p.sl2 * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float f = __shfl_sync(kFull, back, 4 * (2 * c + j));
          ka[nt][j] = f * 16777216.f;
          kb[nt][j] = f * __shfl_sync(kFull, sum, 4 * (2 * c + j));
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int rw = rt * kRowsTile + nt * 8 + 2 * c + j;
        col_pos[nt][j] = rw < p.rows ? __ldg(p.pos + b * p.pos_b + rw / p.hpg) : -1;
      }
    }
    float acc[NT][KS][4];
    float ref[NT][2], neg[NT][2], l[NT][2], base_v[NT][2];  // base_v: sum of p low
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < KS; ++i)
        acc[nt][i][0] = acc[nt][i][1] = acc[nt][i][2] = acc[nt][i][3] = 0.f;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        ref[nt][j] = -INFINITY;
        neg[nt][j] = l[nt][j] = base_v[nt][j] = 0.f;
      }
    }
    const int in_lo = sp.hi_pos - p.left;  // keys in [in_lo, lo_pos] are seen by every row

    while (!failed && done != issued) {
      const int s = done % C::kStages;
      if (!__all_sync(kFull, wait_phase(bars + 8 * s, (done / C::kStages) & 1, kWaitLimitNs))) {
        failed = true;
        break;
      }
      const int n0 = keys[s];
      const uint32_t slot = base + (warp * C::kStages + s) * C::kSlot;
      // this lane's two keys: rows r and r + 8 of S^T
      const int key0 = n0 + (Q4 ? swap01(r) : r);
      auto tile = [&](auto edge_c) {
        constexpr bool EDGE = decltype(edge_c)::value;
        [[maybe_unused]] uint32_t ksc[2], vsc[2];  // (step, low) of the two keys
        if constexpr (Q4) {
          const uint32_t* sc =
              reinterpret_cast<const uint32_t*>(gbase + C::kOffScale +
                                                (warp * C::kStages + s) * C::kScales) + (key0 - n0);
          ksc[0] = sc[0], ksc[1] = sc[8], vsc[0] = sc[kPaTile], vsc[1] = sc[kPaTile + 8];
        }
        if constexpr (EDGE) {
          // rows that no query sees may hold anything: V's (or the scales) as zeros
          auto nobody = [&](int key) {
            return key > sp.hi_pos || (key < sp.lo_pos - p.left && key >= p.sinks);
          };
          if constexpr (Q4) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
              if (nobody(key0 + 8 * j)) ksc[j] = vsc[j] = 0u;
          } else {
            for (int i = lane; i < kPaTile * (D / 8); i += 32) {
              const int row = i / (D / 8), ch = i % (D / 8);
              if (nobody(n0 + row))
                st_shared_zero16(slot + C::kKv + (ch >> 3) * kBoxBytes + row * 128 + (ch & 7) * 16);
            }
            fence_proxy_async_smem();  // (before the slot's next copy)
            __syncwarp();
          }
        }
        // S^T = K Q^T
        float sc4[NT][2][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) sc4[nt][0][i] = sc4[nt][1][i] = 0.f;
        if constexpr (!Q4) {
          const int krow = (lane & 7) + (lane & 8);
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            const int ch = 2 * k + (lane >> 4);
            uint32_t a0, a1, a2, a3;
            ldsm_x4(slot + (ch >> 3) * kBoxBytes + krow * 128 + (((ch & 7) ^ (krow & 7)) << 4), a0,
                    a1, a2, a3);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_16816_t<BF16>(sc4[nt][k & 1], a0, a1, a2, a3, qf[nt][k][0], qf[nt][k][1]);
          }
        } else {
          constexpr int W = D / 32;
          uint32_t w[2][W];
          const int row = key0 - n0;
          if constexpr (D == 128) {
            const uint32_t o = slot - base + row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
            const uint4 x = *reinterpret_cast<const uint4*>(gbase + o);
            const uint4 y = *reinterpret_cast<const uint4*>(gbase + o + 512);
            w[0][0] = x.x, w[0][1] = x.y, w[0][2] = x.z, w[0][3] = x.w;
            w[1][0] = y.x, w[1][1] = y.y, w[1][2] = y.z, w[1][3] = y.w;
          } else {
            const uint32_t o = slot - base + row * 32 + c * 8;
            const uint2 x = *reinterpret_cast<const uint2*>(gbase + o);
            const uint2 y = *reinterpret_cast<const uint2*>(gbase + o + 256);
            w[0][0] = x.x, w[0][1] = x.y, w[1][0] = y.x, w[1][1] = y.y;
          }
#pragma unroll
          for (int j = 0; j < W; ++j) {
            const uint32_t u = w[0][j], v = w[1][j], u8 = u >> 8, v8 = v >> 8;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_16816(sc4[nt][0], u & 0x000f000fu, v & 0x000f000fu, u & 0x00f000f0u,
                        v & 0x00f000f0u, qf[nt][2 * j][0], qf[nt][2 * j][1]);
              mma_16816(sc4[nt][1], u8 & 0x000f000fu, v8 & 0x000f000fu, u8 & 0x00f000f0u,
                        v8 & 0x00f000f0u, qf[nt][2 * j + 1][0], qf[nt][2 * j + 1][1]);
            }
          }
        }
        // x in the log2 domain; element i: key key0 + 8 (i / 2), column 2 c + i % 2
        float x[NT][4];
        [[maybe_unused]] float rstep[2], lstep[2], lowv[2];
        if constexpr (Q4) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float step = __uint_as_float(vsc[j] << 16);
            lowv[j] = __uint_as_float(vsc[j] & 0xffff0000u);
            const bool none = step == 0.f;  // all codes are 0: any step serves
            rstep[j] = none ? 1.f : __frcp_rn(step);
            lstep[j] = none ? 0.f : __log2f(step);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float dot = sc4[nt][0][i] + sc4[nt][1][i];
            if constexpr (Q4) {
              const float step = __uint_as_float(ksc[i >> 1] << 16);
              const float low = __uint_as_float(ksc[i >> 1] & 0xffff0000u);
              x[nt][i] = fmaf(step * ka[nt][i & 1], dot, fmaf(low, kb[nt][i & 1], lstep[i >> 1]));
            } else {
              x[nt][i] = dot * p.sl2;
            }
            if constexpr (EDGE) {
              const int key = key0 + 8 * (i >> 1), q = col_pos[nt][i & 1];
              if (key > q || (key < q - p.left && key >= p.sinks)) x[nt][i] = -INFINITY;
            }
          }
        }
        // the reference moves when an element exceeds it by more than the slack
        bool move = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            move = move || fmaxf(x[nt][j], x[nt][j + 2]) > ref[nt][j] + kPaSlack;
        if (__any_sync(kFull, move)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float mx = fmaxf(x[nt][j], x[nt][j + 2]);
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
              if (mx > ref[nt][j] + kPaSlack) {  // (alike in the lanes of a column)
                const float f = ex2(ref[nt][j] - mx);  // 0 while nothing was seen
                l[nt][j] *= f;
                base_v[nt][j] *= f;
#pragma unroll
                for (int i = 0; i < KS; ++i) {
                  acc[nt][i][j] *= f;
                  acc[nt][i][j + 2] *= f;
                }
                ref[nt][j] = mx;
                neg[nt][j] = -mx;
              }
            }
          }
        }
        uint32_t pf[NT][2];  // P^T as B operand
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float e[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            e[i] = ex2(x[nt][i] + neg[nt][i & 1]);
            if constexpr (Q4) {
              float pr = e[i] * rstep[i >> 1], lw = lowv[i >> 1];
              if constexpr (EDGE) {
                const int key = key0 + 8 * (i >> 1), q = col_pos[nt][i & 1];
                if (key > q || (key < q - p.left && key >= p.sinks)) pr = lw = 0.f;
              }
              l[nt][i & 1] += pr;
              base_v[nt][i & 1] = fmaf(pr, lw, base_v[nt][i & 1]);
            } else {
              l[nt][i & 1] += e[i];
            }
          }
          pf[nt][0] = movmatrix_t(pack2_t<BF16 && !Q4>(e[0], e[1]));
          pf[nt][1] = movmatrix_t(pack2_t<BF16 && !Q4>(e[2], e[3]));
        }
        // O^T += V^T P^T
        if constexpr (!Q4) {
          const int vrow = (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
          for (int i = 0; i < KS; ++i) {
            const int ch = 2 * i + ((lane >> 3) & 1);
            uint32_t a0, a1, a2, a3;
            ldsm_x4_t(slot + C::kKv + (ch >> 3) * kBoxBytes + vrow * 128 +
                          (((ch & 7) ^ (vrow & 7)) << 4),
                      a0, a1, a2, a3);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_16816_t<BF16>(acc[nt][i], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
          }
        } else {
          // keys 2 c, 2 c + 1, 2 c + 8, 2 c + 9 of S^T's rows; words W r .. of each
          constexpr int W = D / 64;
          uint32_t w[4][W];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int row = swap01(2 * c + (j & 1)) + 8 * (j >> 1);
            if constexpr (D == 128) {
              const uint32_t o = slot - base + C::kKv + row * 64 +
                                 (((r >> 1) ^ ((row >> 1) & 3)) << 4) + (r & 1) * 8;
              const uint2 v = *reinterpret_cast<const uint2*>(gbase + o);
              w[j][0] = v.x;
              w[j][W - 1] = v.y;
            } else {
              w[j][0] = *reinterpret_cast<const uint32_t*>(gbase + (slot - base) + C::kKv +
                                                           row * 32 + r * 4);
            }
          }
#pragma unroll
          for (int j = 0; j < W; ++j) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {  // entries 0..3, 4..7 of the word
              const uint32_t sel = half ? 0x7632u : 0x5410u;
              const uint32_t u = __byte_perm(w[0][j], w[1][j], sel);
              const uint32_t v = __byte_perm(w[2][j], w[3][j], sel);
              const uint32_t u8 = u >> 8, v8 = v >> 8;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma_16816(acc[nt][4 * j + 2 * half], u & 0x000f000fu, u & 0x00f000f0u,
                          v & 0x000f000fu, v & 0x00f000f0u, pf[nt][0], pf[nt][1]);
                mma_16816(acc[nt][4 * j + 2 * half + 1], u8 & 0x000f000fu, u8 & 0x00f000f0u,
                          v8 & 0x000f000fu, v8 & 0x00f000f0u, pf[nt][0], pf[nt][1]);
              }
            }
          }
        }
      };
      const int n1 = n0 + kPaTile - 1;
      if (n1 <= sp.lo_pos && (n0 >= in_lo || n1 < p.sinks))
        tile(std::false_type{});
      else
        tile(std::true_type{});
      __syncwarp();  // the slot has been read
      ++done;
      issue();
    }

    // ---- the four warps' results, joined in shared memory
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          l[nt][j] += __shfl_xor_sync(kFull, l[nt][j], o);
          base_v[nt][j] += __shfl_xor_sync(kFull, base_v[nt][j], o);
        }
    __syncthreads();  // every warp is done with the ring
    float* const joined = reinterpret_cast<float*>(gbase);
    float* const stat = reinterpret_cast<float*>(gbase + C::kOffStat);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int row = nt * 8 + 2 * c + j;
        float* const dst = joined + (warp * kRowsTile + row) * C::kPad;
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          if constexpr (Q4) {
            // words W r + i / 4 of a row, entries 2 (i % 4) and the one after,
            // which the mask left 16 times as large
            const int d = 8 * (D / 64 * r + (i >> 2)) + 2 * (i & 3);
            dst[d] = fmaf(acc[nt][i][j], 16777216.f, base_v[nt][j]);
            dst[d + 1] = fmaf(acc[nt][i][j + 2], 1048576.f, base_v[nt][j]);
          } else {
            dst[16 * i + r] = acc[nt][i][j];
            dst[16 * i + r + 8] = acc[nt][i][j + 2];
          }
        }
        if (r == 0) {
          stat[2 * (warp * kRowsTile + row)] = ref[nt][j];
          stat[2 * (warp * kRowsTile + row) + 1] = l[nt][j];
        }
      }
    __syncthreads();
    const bool whole = t0 == 0 && t1 == sp.n;
    // a piece of an item that begins in this share: slot 2 CTA + 1; that
    // goes on from an earlier one: 2 CTA
    const int64_t slot_id = 2 * static_cast<int64_t>(blockIdx.x) + (t0 == 0 ? 1 : 0);
    for (int i = threadIdx.x; i < kRowsTile * (D / 2); i += kPaThreads) {
      const int row = i / (D / 2), d = 2 * (i % (D / 2));
      const int rw = rt * kRowsTile + row;
      if (rw >= p.rows) continue;
      float m = -INFINITY, sum = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll
      for (int w = 0; w < kPaWarps; ++w) m = fmaxf(m, stat[2 * (w * kRowsTile + row)]);
#pragma unroll
      for (int w = 0; w < kPaWarps; ++w) {
        const float rw_ref = stat[2 * (w * kRowsTile + row)];
        // (a warp that saw nothing has a sum of 0, or NaN where scores are)
        const float f = rw_ref == m ? 1.f : ex2(rw_ref - m);
        const float2 v =
            *reinterpret_cast<const float2*>(joined + (w * kRowsTile + row) * C::kPad + d);
        sum = fmaf(f, stat[2 * (w * kRowsTile + row) + 1], sum);
        o0 = fmaf(f, v.x, o0);
        o1 = fmaf(f, v.y, o1);
      }
      if (whole) {
        const int mq = rw / p.hpg, h = head * p.hpg + rw - mq * p.hpg;
        if (__ldg(p.pos + b * p.pos_b + mq) < 0) sum = o0 = o1 = 0.f;  // padding
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        reinterpret_cast<uint32_t*>(
            p.o + ((static_cast<int64_t>(b) * p.M + mq) * p.H + h) * D)[d >> 1] =
            pack2_t<BF16>(o0 * inv, o1 * inv);
        if (d == 0 && p.lse != nullptr)
          p.lse[(static_cast<int64_t>(b) * p.H + h) * p.M + mq] =
              sum == 0.f ? -INFINITY : (m + __log2f(sum)) * 0.69314718055994530942f;
      } else {
        float* const dst = p.piece + (slot_id * kRowsTile + row) * D + d;
        *reinterpret_cast<float2*>(dst) = make_float2(o0, o1);
        if (d == 0) {
          float* const st =
              p.piece + (2 * static_cast<int64_t>(p.ctas) * D + 2 * slot_id) * kRowsTile + 2 * row;
          st[0] = m;
          st[1] = sum;
        }
      }
    }
    fence_proxy_async_smem();  // the ring's next copies come after these reads and writes
    __syncthreads();
    if (!p.cut) break;
    // the next item of the share
    at += sp.n;
    if (++head == p.G) {
      head = 0;
      do ++item;
      while (item < p.items && count[item + 1] == count[item]);
    }
    more = at < end;
  }
  if (failed) {
    // leave nothing in flight
    for (; done != issued; ++done)
      wait_phase(bars + 8 * (done % C::kStages), (done / C::kStages) & 1, kWaitLimitNs);
    if (lane == 0) report_timeout();
  }
}

// Items that shares have cut: their pieces joined in order; items without a
// tile: zeros. A CTA a row; a piece to each of kJoinSets sets of threads in turn.
constexpr int kJoinSets = 4;

template <int D, bool BF16>
__global__ void __launch_bounds__(kJoinSets * D / 2)
    paged_attn_join_kernel(const PagedProblem p, int rows_tile) {
  __shared__ float weight[4 * kPaSms + 2];
  __shared__ float2 part[kJoinSets][D / 2];
  const int item = blockIdx.x / p.G, head = blockIdx.x - item * p.G;
  const int row = blockIdx.y;
  const int b = item / p.tiles, rt = item - b * p.tiles;
  const int rw = rt * rows_tile + row;
  if (rw >= p.rows) return;
  const int64_t c0 = p.count[item], per = p.count[p.items + 1];
  const int64_t n = p.count[item + 1] - c0;
  const int64_t at = c0 * p.G + head * n;
  const int first = static_cast<int>(at / per), last = n > 0 ? static_cast<int>((at + n - 1) / per) : first;
  if (n > 0 && first == last) return;  // whole in one share
  const int d = threadIdx.x % (D / 2), set = threadIdx.x / (D / 2);
  const int pieces = n > 0 ? last - first + 1 : 0;
  const float* const stats = p.piece + 2 * static_cast<int64_t>(p.ctas) * rows_tile * D;
  auto slot = [&](int i) { return 2 * static_cast<int64_t>(first + i) + (i == 0 ? 1 : 0); };
  auto stat = [&](int i, int k) { return stats[(slot(i) * rows_tile + row) * 2 + k]; };
  // the largest reference, then every piece's weight (all threads alike)
  float m = -INFINITY;
  for (int i = threadIdx.x & 31; i < pieces; i += 32) m = fmaxf(m, stat(i, 0));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
  for (int i = threadIdx.x; i < pieces; i += kJoinSets * D / 2) {
    const float ref = stat(i, 0);
    weight[i] = ref == m ? 1.f : ex2(ref - m);
  }
  __syncthreads();
  float2 o = make_float2(0.f, 0.f);
  for (int i = set; i < pieces; i += kJoinSets) {
    const float2 v =
        reinterpret_cast<const float2*>(p.piece + (slot(i) * rows_tile + row) * D)[d];
    o.x = fmaf(weight[i], v.x, o.x);
    o.y = fmaf(weight[i], v.y, o.y);
  }
  part[set][d] = o;
  __syncthreads();
  if (set != 0) return;
  float sum = 0.f;
  for (int i = 0; i < pieces; ++i) sum = fmaf(weight[i], stat(i, 1), sum);
  o = make_float2(0.f, 0.f);
#pragma unroll
  for (int k = 0; k < kJoinSets; ++k) o.x += part[k][d].x, o.y += part[k][d].y;
  const int mq = rw / p.hpg, h = head * p.hpg + rw - mq * p.hpg;
  if (__ldg(p.pos + b * p.pos_b + mq) < 0) sum = o.x = o.y = 0.f;  // padding
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  reinterpret_cast<uint32_t*>(p.o + ((static_cast<int64_t>(b) * p.M + mq) * p.H + h) * D)[d] =
      pack2_t<BF16>(o.x * inv, o.y * inv);
  if (d == 0 && p.lse != nullptr)
    p.lse[(static_cast<int64_t>(b) * p.H + h) * p.M + mq] =
        sum == 0.f ? -INFINITY : (m + __log2f(sum)) * 0.69314718055994530942f;
}

// ---- host ---------------------------------------------------------------

// Row tiles: 8 rows where a KV head has no more, else 16.
int rows_of_tile(int64_t rows) { return rows <= 8 ? 8 : 16; }

bool encode_code_map(CUtensorMap* tm, const void* ptr, const KvPages& c, int64_t G, int64_t D) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t row = static_cast<cuuint64_t>(D / 2), page = cuuint64_t(1) << c.shift;
  const cuuint64_t dims[4] = {row, static_cast<cuuint64_t>(G), page,
                              static_cast<cuuint64_t>(c.pages)};
  const cuuint64_t strides[3] = {row, row * G, row * G * page};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(row), 1, kPaTile, 1};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return enc(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(ptr), dims, strides, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE,
             D == 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int check_paged(int64_t B, int64_t M, int64_t H, int64_t G, int64_t D, int dtype) {
  const int rc = check_rope(B, M, H, G, D, 0, 0, 0, 0.f, dtype, NSA_F32);
  if (rc != NSA_OK) return rc;
  if (H % G != 0) return NSA_ERR_GROUPS;
  if (M * (H / G) >= int64_t(1) << 30) return NSA_ERR_SHAPE;
  const int64_t rows = M * (H / G), tile = rows_of_tile(rows);
  if (B * ((rows + tile - 1) / tile) * G >= int64_t(1) << 31) return NSA_ERR_SHAPE;
  return NSA_OK;
}

template <int D, bool BF16, bool Q4, int NT>
int launch_paged(PagedProblem& p, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t st) {
  using C = PaCfg<D, Q4, NT>;
  static_assert(C::kSmem * C::kPerSm <= 232448, "CTAs of an SM");
  static_assert(C::kPerSm <= 4, "pieces in the workspace");
  auto kern = paged_attn_kernel<D, BF16, Q4, NT>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) !=
      cudaSuccess)
    return NSA_ERR_LAUNCH;
  p.ctas = C::kPerSm * kPaSms;
  const int64_t blocks = p.cut ? p.ctas : static_cast<int64_t>(p.items) * p.G;
  kern<<<static_cast<unsigned>(blocks), kPaThreads, C::kSmem, st>>>(p, tk, tv);
  if (cudaGetLastError() != cudaSuccess) return NSA_ERR_LAUNCH;
  if (p.cut) {
    paged_attn_join_kernel<D, BF16>
        <<<dim3(p.items * p.G, 8 * NT), kJoinSets * D / 2, 0, st>>>(p, 8 * NT);
    if (cudaGetLastError() != cudaSuccess) return NSA_ERR_LAUNCH;
  }
  return NSA_OK;
}

template <int D, bool BF16>
int launch_paged_d(PagedProblem& p, const nsa_kv_cache* kv, cudaStream_t st) {
  CUtensorMap tk, tv;
  if (kv->bits == 4) {
    if (!encode_code_map(&tk, p.c.k, p.c, p.G, D) || !encode_code_map(&tv, p.c.v, p.c, p.G, D))
      return NSA_ERR_LAUNCH;
  } else {
    constexpr CUtensorMapDataType dt =
        BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const int64_t page = int64_t(1) << p.c.shift;
    if (!encode_kv_map_strided(&tk, p.c.k, p.c.pages, page, p.G, D, kPaTile, dt, p.c.kp / 2,
                               p.c.kt / 2, p.c.kh / 2) ||
        !encode_kv_map_strided(&tv, p.c.v, p.c.pages, page, p.G, D, kPaTile, dt, p.c.vp / 2,
                               p.c.vt / 2, p.c.vh / 2))
      return NSA_ERR_LAUNCH;
  }
  if (rows_of_tile(p.rows) == 8)
    return kv->bits == 4 ? launch_paged<D, BF16, true, 1>(p, tk, tv, st)
                         : launch_paged<D, BF16, false, 1>(p, tk, tv, st);
  return kv->bits == 4 ? launch_paged<D, BF16, true, 2>(p, tk, tv, st)
                       : launch_paged<D, BF16, false, 2>(p, tk, tv, st);
}

}  // namespace

int paged_read_and_clear_status(unsigned int* value) { return read_and_clear_status(value); }

}  // namespace nsa

extern "C" int64_t nsa_paged_attn_workspace_bytes(int64_t B, int64_t M, int64_t H, int64_t G,
                                                  int64_t D) {
  using namespace nsa;
  const int rc = check_paged(B, M, H, G, D, NSA_F16);
  if (rc != NSA_OK) return rc;
  const int64_t rows = M * (H / G), tile = rows_of_tile(rows);
  const int64_t items = B * ((rows + tile - 1) / tile);
  if (items == 0 || items > kPaItems) return 0;
  // two pieces of every share, and the running counts
  return 2 * 4 * kPaSms * tile * (D + 2) * 4 + (kPaItems + 2) * 8;
}

extern "C" int nsa_paged_attn(const void* Q, const nsa_kv_cache* cache, const int32_t* page_table,
                              const int32_t* positions, void* O, float* LSE, int64_t B, int64_t M,
                              int64_t H, int64_t G, int64_t D, int64_t positions_stride,
                              int64_t table_cols, int64_t window_left, int64_t sinks, float scale,
                              int dtype, const int64_t* q_strides, void* workspace,
                              int64_t workspace_bytes, void* stream) {
  using namespace nsa;
  int rc = check_paged(B, M, H, G, D, dtype);
  if (rc != NSA_OK) return rc;
  if (positions_stride < 0 || sinks < 0) return NSA_ERR_SHAPE;
  int64_t s[3];
  if ((rc = take_strides(q_strides, 1, &H, B, M, D, s, 0)) != NSA_OK) return rc;
  if (B == 0 || M == 0) return NSA_OK;
  if (!Q || !O || !positions) return NSA_ERR_NULL;
  if (!aligned(Q, 16) || !aligned(O, 16) || !aligned(LSE, 4) || !aligned(positions, 4))
    return NSA_ERR_ALIGN;
  PagedProblem p{};
  if ((rc = take_cache(cache, page_table, table_cols, B, G, D, true, &p.c)) != NSA_OK) return rc;
  const int64_t need = nsa_paged_attn_workspace_bytes(B, M, H, G, D);
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return NSA_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return NSA_ERR_ALIGN;
  }
  // (the running count of tiles is 32 bits wide)
  p.q = static_cast<const uint8_t*>(Q);
  p.qb = s[0], p.qm = s[1], p.qh = s[2];
  p.o = static_cast<uint16_t*>(O);
  p.lse = LSE;
  p.pos = positions;
  p.pos_b = positions_stride;
  p.count = static_cast<int64_t*>(workspace);
  p.piece = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + (kPaItems + 2) * 8);
  p.B = static_cast<int>(B);
  p.M = static_cast<int>(M);
  p.H = static_cast<int>(H);
  p.G = static_cast<int>(G);
  p.hpg = static_cast<int>(H / G);
  p.rows = static_cast<int>(M * (H / G));
  const int tile = rows_of_tile(p.rows);
  p.tiles = (p.rows + tile - 1) / tile;
  p.items = static_cast<int>(B * p.tiles);
  p.cut = need > 0 && p.items * (table_cols * cache->page_size / kPaTile) < int64_t(1) << 31;
  // a window that reaches behind key 0 from any position; sinks as many as a table's tokens
  const int64_t far = 0x7fffffff, most = int64_t(1) << 30;
  p.left = static_cast<int>(window_left < 0 || window_left > far ? far : window_left);
  p.sinks = static_cast<int>(sinks > most ? most : sinks);
  const float sc = scale > 0.f ? scale : 1.0f / sqrtf(static_cast<float>(D));
  p.sl2 = sc * 1.4426950408889634f;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf = dtype == NSA_BF16;
  if (D == 64)
    return bf ? launch_paged_d<64, true>(p, cache, st) : launch_paged_d<64, false>(p, cache, st);
  return bf ? launch_paged_d<128, true>(p, cache, st) : launch_paged_d<128, false>(p, cache, st);
}
