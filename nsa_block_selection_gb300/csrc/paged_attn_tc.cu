// Attention over pages with many rows a KV head (a piece of a prompt, drafted
// tokens) on the 5th-generation tensor cores, for sm_103a. The mathematics and the
// items' shares are paged_attn.cu's; here a row tile is up to 128 (query, head) rows
// of a KV head, the M of the products, and a step 128 keys:
//   S (128 rows x 128 keys) = Q K^T,  O (128 rows x D) += P V,
// with S, P and O in tensor memory. Two groups of four softmax warps, a row a thread,
// take the steps in turn, each with a running maximum, a sum and an O of its own, which
// they join at the end of an item: one group's exponentials run beside the other's
// products, and a row tile needs no more rows for it. Warp 1 issues S_0, S_1, PV_0,
// S_2, PV_1, ... over all of the CTA's items; P lies over its S.
//
// 16 bits: warp 0 brings a step's K by TMA, warp 2 its V (with both in one warp the
// copies alone took a warp 1900 clocks a step, and K waited for V's stage), a copy a
// page, or a part of one, a lane; a page that the sequence does not have is asked for
// outside the map and arrives as zeros. V's rows that no query sees are zeroed by the
// softmax warps before P is handed over, so whatever they hold never meets a product.
//
// 4 bits: four loader warps load the codes a step ahead and write c - 8, exact in
// fp16, as the operands' rows; five numbers of a key (steps, the middles low + 8 step,
// log2 of V's step) go beside them, and a key that nobody sees gets -inf for x and
// zeros. Rows of V without a step become codes of 8 (pa_step). With k = mid + step (c - 8):
//   x = step ka (q'.(c - 8)) + mid kb + log2 step_v,  p' = 2^(x - r),
//   l += p' / step_v,  O = sum p' (c - 8) + sum p' mid_v / step_v,
// q' = 2^e q in fp16, written by the softmax warps, ka and kb the row's factors.
//
// What bounds it: a step takes some 1500 clocks (16 bits; the products 800 of the
// tensor cores' time, a group's softmax 2600 for every other step) and 3000 (4 bits:
// the shared-memory pipe, by the operands' rows that the loaders write and the five
// numbers of a key that every row reads; loaders of a warpgroup each for K and V gained
// nothing); an item's own cost is some 6000. Prompts of 32 + 4 heads of 128: 16,384
// tokens 1747 us (1260 TFLOP/s), 4096 tokens 167 us (4 bits 279); 3 x 200 tokens of 64
// + 8 heads after 8800 others 175 us (291). One group with two S and a P of its own,
// and one producer warp: 2160, 232 (371), 266 (384).
//
// Every mbarrier wait is bounded (1 s); a role that gives up sets the status word
// and leaves its loop, so every role reaches the teardown, which frees the tensor
// memory.

#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "common.cuh"
#include "kv_cache.cuh"
#include "nsa_sel_attn.h"
#include "paged_attn.cuh"
#include "ptx.cuh"
#include "tc.cuh"

namespace nsa {
namespace {

constexpr int kTcKeys = 128;
// Tensor memory of softmax group x: S (and over it P) at 128 x, O at 256 + 128 x.
constexpr uint32_t kTcTmem = 512, kColS = 0, kColO = 256;

enum TcBar : int {
  kQFull = 0,    // 2 Q buffers
  kQEmpty = 2,   // 2: every QK^T of the item that used Q buffer b has completed
  kKFull = 4,    // 2 K stages
  kKEmpty = 6,   // 2
  kVFull = 8,    // 2 V stages
  kVEmpty = 10,  // 2
  kSFull = 12,   // 2 S buffers
  kPFull = 14,   // 2 P buffers
  kPvDone = 16,  // 2
  kMerge = 18,   // both groups' sums of an item are there
  kOEmpty = 19,  // the softmax warps have read O of the item before
  // 4: a step's facts for the softmax (which pages are there, or the keys' numbers).
  // Four, as K of the step after the next may come before its softmax begins.
  kInfo = 20,
  kTcBars = 24
};

template <int D, bool Q4>
struct TcCfg {
  // warpgroups: (Q and K, MMA, V, .), two of softmax; 4 bits: and one of loaders
  static constexpr int kSoftWarp = 4, kLoadWarp = 12;
  static constexpr int kThreads = Q4 ? 512 : 384;
  [[maybe_unused]] static constexpr int kAtoms = D / 64;
  static constexpr int kAtomBytes = 128 * 128;
  static constexpr int kTile = 128 * D * 2;  // Q, K or V
  static constexpr int kOffK = 2 * kTile, kOffV = 4 * kTile;
  static constexpr int kOffInfo = 6 * kTile;  // 4 x (5 numbers of each key, or a mask)
  static constexpr int kInfoBytes = Q4 ? 5 * kTcKeys * 4 : 16;
  static constexpr int kOffStat = kOffInfo + 4 * kInfoBytes;  // a group's rows' 4 floats
  static constexpr int kOffBar = kOffStat + 2 * 128 * 16;
  static constexpr int kOffTmem = kOffBar + kTcBars * 8;
  static constexpr int kOffCount = kOffTmem + 8;
  static constexpr int kUsed = kOffCount + (kPaItems + 1) * 4 + 64 + 1024;
  // at least 116 KB, so that one CTA holds an SM (all 512 tensor-memory columns)
  static constexpr int kSmem = kUsed > 118784 ? kUsed : 118784;
  static_assert(kSmem <= 232448, "one CTA an SM");
};

// The items of a CTA, one after the other, the same for every role. A whole warp
// calls it: positions are read by its lanes.
struct TcWalk {
  PaShare sh;
  PaSpan sp;
  int b, rt, t0, t1;
  bool more;

  __device__ __forceinline__ void load(const PagedProblem& p, int rows_tile) {
    b = sh.item / p.tiles;
    rt = sh.item - b * p.tiles;
    sp = pa_span<true>(p, b, rt, rows_tile);
    t0 = 0;
    t1 = sp.n;
    if (p.cut) {
      const int64_t first = sh.at + p.item_cost, n = sp.n, zero = 0;
      t0 = static_cast<int>(min(max(sh.begin - first, zero), n));
      t1 = static_cast<int>(min(max(sh.end - first, zero), n));
    }
  }
  __device__ __forceinline__ void start(const PagedProblem& p, const PaShare& share,
                                        int rows_tile) {
    sh = share;
    if (!p.cut) {
      sh.item = blockIdx.x / p.groups;
      sh.group = blockIdx.x - sh.item * p.groups;
    }
    more = !p.cut || sh.begin < sh.end;
    if (more) load(p, rows_tile);
  }
  __device__ __forceinline__ void next(const PagedProblem& p, const int* count, int rows_tile) {
    if (!p.cut) {
      const int64_t x = static_cast<int64_t>(sh.item) * p.groups + sh.group + gridDim.x;
      more = x < static_cast<int64_t>(p.items) * p.groups;
      sh.item = static_cast<int>(x / p.groups);
      sh.group = static_cast<int>(x - static_cast<int64_t>(sh.item) * p.groups);
    } else {
      sh.at += sp.n + p.item_cost;
      if (++sh.group == p.groups) {
        sh.group = 0;
        do ++sh.item;
        while (sh.item < p.items && count[sh.item + 1] == count[sh.item]);
      }
      more = sh.at < sh.end;
    }
    if (more) load(p, rows_tile);
  }
};

// A matrix descriptor moved by `bytes` (shared memory ends below the address field's
// 2^18 bytes): an addition instead of the descriptor built again.
__device__ __forceinline__ uint64_t desc_at(uint64_t desc, uint32_t bytes) {
  const uint32_t lo = static_cast<uint32_t>(desc) + (bytes >> 4);
  return (desc & 0xffffffff00000000ull) | lo;
}

// Bit c set: column c of 32 lies in [lo, hi].
__device__ __forceinline__ uint32_t columns(int lo, int hi) {
  const uint32_t below = hi < 0 ? 0u : hi >= 31 ? ~0u : (2u << hi) - 1u;
  return lo <= 0 ? below : lo > 31 ? 0u : below & (~0u << lo);
}

// 32 bytes, in one store where the address allows it.
__device__ __forceinline__ void store32(void* dst, const uint4& a, const uint4& b) {
  if ((reinterpret_cast<uintptr_t>(dst) & 31) == 0) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(dst), "r"(a.x),
                 "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(dst)[0] = a;
    reinterpret_cast<uint4*>(dst)[1] = b;
  }
}
__device__ __forceinline__ uint4 words(const float* f) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                    __float_as_uint(f[3]));
}

// Two codes of the bits under 0x000f000f as fp16 c - 8.
__device__ __forceinline__ uint32_t less8(uint32_t two) {
  const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&two),
                            __halves2half2(__ushort_as_half(0x6408), __ushort_as_half(0x6408)));
  return *reinterpret_cast<const uint32_t*>(&h);
}
// The 8 codes of a word as a 16-byte chunk, in the order 0, 4, 1, 5, 2, 6, 3, 7.
__device__ __forceinline__ uint4 codes_chunk(uint32_t w) {
  constexpr uint32_t kMask = 0x000f000fu, k1024 = 0x64006400u;
  return make_uint4(less8((w & kMask) | k1024), less8((w >> 4 & kMask) | k1024),
                    less8((w >> 8 & kMask) | k1024), less8((w >> 12 & kMask) | k1024));
}
// Place of entry i of 8 in that order.
__device__ __forceinline__ constexpr int code_place(int i) { return i < 4 ? 2 * i : 2 * i - 7; }

template <int D, bool BF16, bool Q4>
__global__ void __launch_bounds__(TcCfg<D, Q4>::kThreads, 1)
    paged_attn_tc_kernel(const PagedProblem p, int rows_tile, const __grid_constant__ CUtensorMap tmQ,
                         const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV) {
  using C = TcCfg<D, Q4>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const gbase = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](int i) { return base + C::kOffBar + 8u * static_cast<uint32_t>(i); };
  int* const count = reinterpret_cast<int*>(gbase + C::kOffCount);
  int* const sums = count + kPaItems + 1;
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(kQFull + s), Q4 ? 256 : 1);
      mbar_init(bar(kQEmpty + s), 1);
      mbar_init(bar(kKFull + s), Q4 ? 128 : 1);
      mbar_init(bar(kKEmpty + s), 1);
      mbar_init(bar(kVFull + s), Q4 ? 128 : 1);
      mbar_init(bar(kVEmpty + s), 1);
      mbar_init(bar(kSFull + s), 1);
      mbar_init(bar(kPFull + s), 128);
      mbar_init(bar(kPvDone + s), 1);
    }
    mbar_init(bar(kMerge), 256);
    mbar_init(bar(kOEmpty), 256);
    for (int s = 0; s < 4; ++s) mbar_init(bar(kInfo + s), Q4 ? 128 : 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tc_alloc(base + C::kOffTmem, kTcTmem);
    tc_relinquish();
  }
  asm volatile("griddepcontrol.launch_dependents;\n");  // the join waits for this grid's end
  PaShare share{0, 0, 0, 0, 0};
  if (p.cut) {
    share = pa_share<C::kThreads>(p, rows_tile, count, sums);
    pa_zeros<D>(p, rows_tile, count);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(gbase + C::kOffTmem);
  bool failed = false;
  TcWalk it;
  it.start(p, share, rows_tile);
  int64_t gt = 0;  // steps of the items before
  int n = 0;       // items with steps before

  // ---- TMA producers (16 bits): one warp brings Q and K, one V ----
  auto producer = [&](auto value_c) {
    if constexpr (!Q4) {
      constexpr bool V = decltype(value_c)::value;
      constexpr int kFull_ = V ? kVFull : kKFull, kEmpty_ = V ? kVEmpty : kKEmpty;
      constexpr int kOff = V ? C::kOffV : C::kOffK;
      const CUtensorMap* const tm = V ? &tmV : &tmK;
      const uint64_t keep = p.tiles > 1 ? l2_policy_evict_normal() : l2_policy_evict_first();
      const int rows = min(kTcKeys, 1 << p.c.shift);  // keys of a copy
      const int split = kTcKeys / rows;
      // lane l < split * kAtoms issues atom l % kAtoms of copy l / kAtoms
      const int part = lane / C::kAtoms, atom = lane % C::kAtoms;
      const uint32_t dst = base + kOff + atom * C::kAtomBytes + part * rows * 128;
      auto wait_all = [&](int b, uint32_t parity) {
        return __all_sync(kFull, wait_phase(bar(b), parity, kWaitLimitNs));
      };
      for (; it.more && !failed; it.next(p, count, rows_tile)) {
        const int nt = it.t1 - it.t0;
        if (nt <= 0) continue;
        // the page of this lane's copy of step t
        auto look = [&](int t) {
          return t < it.t1 && part < split ? page_of(p.c, it.b, it.sp.key(t) + part * rows) : -1;
        };
        int page_next = look(it.t0);
        if constexpr (!V) {
          const int qb = n & 1;
          if (n >= 2 && !wait_all(kQEmpty + qb, ((n - 2) >> 1) & 1)) {
            failed = true;
            break;
          }
          if (lane == 0) mbar_arrive_expect_tx(bar(kQFull + qb), rows_tile * D * 2);
          __syncwarp();
          if (lane < C::kAtoms)
            tma_load_4d(base + qb * C::kTile + lane * C::kAtomBytes, &tmQ, bar(kQFull + qb),
                        lane * 64, it.sh.group * p.hpg, it.rt * (rows_tile / p.hpg), it.b,
                        l2_policy_evict_first());
        }
        for (int i = 0; i < nt; ++i) {
          const int64_t g = gt + i;
          const int s = static_cast<int>(g & 1);
          const int page = page_next;
          page_next = look(it.t0 + i + 1);
          const int off = it.sp.key(it.t0 + i) & ((1 << p.c.shift) - 1);
          if (g >= 2 && !wait_all(kEmpty_ + s, static_cast<uint32_t>(((g - 2) >> 1) & 1))) {
            failed = true;
            break;
          }
          const uint32_t there = __ballot_sync(kFull, page >= 0);
          if (lane == 0) {
            if constexpr (!V) {
              *reinterpret_cast<uint32_t*>(gbase + C::kOffInfo + (g & 3) * C::kInfoBytes) = there;
              mbar_arrive(bar(kInfo + static_cast<int>(g & 3)));
            }
            mbar_arrive_expect_tx(bar(kFull_ + s), C::kTile);
          }
          __syncwarp();
          if (part < split)
            tma_load_4d(dst + s * C::kTile, tm, bar(kFull_ + s), atom * 64, it.sh.group,
                        split > 1 ? 0 : off, page < 0 ? p.c.pages : page, keep);
        }
        gt += nt;
        ++n;
      }
      if (failed) {  // leave nothing in flight
        if (lane == 0)
          for (int s = 0; s < 2; ++s)
            for (int ph = 0; ph < 2; ++ph) wait_phase(bar(kFull_ + s), ph, kWaitLimitNs / 8);
        __syncwarp();
      }
    }
  };
  auto issuer = [&]() {
    // ---- MMA issuer: the steps of all items as one stream ----
    constexpr bool kBf = BF16 && !Q4;
    constexpr uint32_t idesc_s = umma_idesc_f16(128, kTcKeys, kBf, false);
    constexpr uint32_t idesc_o = umma_idesc_f16(128, D, kBf, true);
    const uint64_t k_major = umma_desc_sw128(base, 16);
    const uint64_t mn_major = umma_desc_sw128(base, C::kAtomBytes);
    // (the whole warp waits and one lane issues: under a branch an MMA costs more)
    const uint32_t on = elect_one();
    auto wait_all = [&](int b, uint32_t parity) {
      return __all_sync(kFull, wait_phase(bar(b), parity, kWaitLimitNs));
    };
    auto issue_s = [&](int64_t g, int qb) -> bool {
      const int s = static_cast<int>(g & 1);
      if (!wait_all(kKFull + s, static_cast<uint32_t>((g >> 1) & 1))) return false;
      tc_fence_after();
      const uint32_t d = tmem + kColS + static_cast<uint32_t>(s) * 128;
      const uint64_t q = desc_at(k_major, qb * C::kTile);
      const uint64_t k = desc_at(k_major, C::kOffK + s * C::kTile);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = (kk >> 2) * C::kAtomBytes + (kk & 3) * 32;
        tc_mma_if(on, d, desc_at(q, off), desc_at(k, off), idesc_s, kk > 0 ? 1u : 0u);
      }
      tc_commit_if(on, bar(kKEmpty + s));
      tc_commit_if(on, bar(kSFull + s));
      return true;
    };
    auto issue_pv = [&](int64_t g, bool first, int item) -> bool {
      const int s = static_cast<int>(g & 1);
      const uint32_t ph = static_cast<uint32_t>((g >> 1) & 1);
      if (!wait_all(kPFull + s, ph) || !wait_all(kVFull + s, ph)) return false;
      if (first && item >= 1 && !wait_all(kOEmpty, (item - 1) & 1)) return false;
      tc_fence_after();
      const uint64_t v = desc_at(mn_major, C::kOffV + s * C::kTile);
      const uint32_t pcol = tmem + kColS + static_cast<uint32_t>(s) * 128;
      const uint32_t ocol = tmem + kColO + static_cast<uint32_t>(s) * 128;
#pragma unroll
      for (int kk = 0; kk < kTcKeys / 16; ++kk)
        tc_mma_ts_if(on, ocol, pcol + 8 * kk, desc_at(v, kk * 2048), idesc_o,
                     (!first || kk > 0) ? 1u : 0u);
      tc_commit_if(on, bar(kVEmpty + s));
      tc_commit_if(on, bar(kPvDone + s));
      return true;
    };
    bool ok = true;
    int64_t pv = 0;  // the next step whose PV is to be issued
    // of the last two steps: whether they are their group's first of the item, and its number
    bool first[2] = {false, false};
    int item[2] = {0, 0};
    auto values_before = [&](int64_t g) {
      for (; ok && pv < g; ++pv) {
        const bool odd = pv & 1;
        ok = issue_pv(pv, odd ? first[1] : first[0], odd ? item[1] : item[0]);
      }
    };
    for (; it.more && ok; it.next(p, count, rows_tile)) {
      const int nt = it.t1 - it.t0;
      if (nt <= 0) continue;
      const int qb = n & 1;
      // (4 bits: Q comes from the softmax warps once they have the last item's O,
      // so its last PVs cannot wait for this item's first S)
      if (Q4) values_before(gt);
      ok = ok && wait_all(kQFull + qb, (n >> 1) & 1);
      for (int i = 0; i < nt && ok; ++i) {
        // S of step g takes the place of step g - 2's P: it is issued after the PV that
        // reads it, and the tensor pipe runs the MMAs in that order
        const int64_t g = gt + i;
        values_before(g - 1);
        ok = ok && issue_s(g, qb);
        if (ok && i == nt - 1) tc_commit_if(on, bar(kQEmpty + qb));
        if (g & 1) {
          first[1] = i < 2;
          item[1] = n;
        } else {
          first[0] = i < 2;
          item[0] = n;
        }
      }
      gt += nt;
      ++n;
    }
    values_before(gt);
    failed = !ok;
  };
  auto softmax = [&]() {
    // ---- softmax: thread <-> row of the item's tile; group 0 has the even steps ----
    constexpr int kUnroll = Q4 ? 1 : kTcKeys / 32;
    const int quarter = warp & 3, group = (warp - C::kSoftWarp) >> 2;
    const int row = quarter * 32 + lane;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    auto wait_all = [&](int b, uint32_t parity) {
      return __all_sync(kFull, wait_phase(bar(b), parity, kWaitLimitNs));
    };
    // the row's query and head in the item, looked up with it
    bool next_mine = false;
    int next_mq = 0, next_h = 0, next_pos = -1;
    auto place = [&]() {
      const int rw = it.rt * rows_tile + row;
      next_mine = it.more && row < rows_tile && rw < p.rows;
      next_mq = rw / p.hpg;
      next_h = it.sh.group * p.hpg + rw - next_mq * p.hpg;
      next_pos = next_mine ? pa_position(p, it.b, next_mq) : -1;
    };
    place();
    while (it.more) {
      const int nt = it.t1 - it.t0;
      if (nt <= 0 && p.cut) {  // (nothing of it in this share)
        it.next(p, count, rows_tile);
        place();
        continue;
      }
      const bool mine = next_mine;
      const int mq = next_mq, h = next_h, pos = next_pos;
      const PaSight see{it.sp.lo_pos, it.sp.hi_pos, p.left, p.sinks};
      // which of the 32 keys from `key` on a query at `pos` sees
      auto seen = [&](int pos, int key) {
        const int hi = max(pos - key, -1);
        return columns(hi - p.left, hi) | columns(0, min(hi, p.sinks - key - 1));
      };
      float ka = p.sl2, kb = 0.f;
      if constexpr (Q4) {
        if (nt > 0) {
          // Q's row: 2^e q in fp16 (the largest entry between 2^13 and 2^14)
          const int qb = n & 1;
          if (n >= 2 && !wait_all(kQEmpty + qb, ((n - 2) >> 1) & 1)) {
            failed = true;
            break;
          }
          const uint4* const src = reinterpret_cast<const uint4*>(
              p.q + 2 * (it.b * p.qb + mq * p.qm + h * p.qh));
          float top = 0.f;
          if (mine) {
#pragma unroll 4
            for (int i = 0; i < D / 8; ++i) {
              float f[8];
              unpack8<BF16>(src[i], f);
#pragma unroll
              for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(f[j]));
            }
          }
          int e = 0;
          if (top > 0.f && top < INFINITY)
            e = min(13 - (static_cast<int>(__float_as_uint(top) >> 23) - 127), 100);
          const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
          float sum = 0.f;
          uint8_t* const dst = gbase + qb * C::kTile + row * 128;
#pragma unroll 4
          for (int i = 0; i < D / 8; ++i) {
            float f[8];
            unpack8<BF16>(mine ? src[i] : make_uint4(0, 0, 0, 0), f);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              f[j] = __half2float(__float2half_rn(f[j] * up));
              sum += f[j];
            }
            if (i / (D / 16) == group)  // (half of the row each)
              *reinterpret_cast<uint4*>(dst + (i >> 3) * C::kAtomBytes + (((i & 7) ^ (row & 7)) << 4)) =
                  make_uint4(pack_half2(f[0], f[4]), pack_half2(f[1], f[5]), pack_half2(f[2], f[6]),
                           pack_half2(f[3], f[7]));
          }
          fence_proxy_async_smem();
          mbar_arrive(bar(kQFull + qb));
          ka = p.sl2 * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
          kb = ka * sum;
        }
      }
      float ref = -INFINITY, neg = 0.f, l = 0.f, mid_sum = 0.f;
      constexpr uint32_t kNoRow = 0xff800000u;  // -inf
      const int begin = (static_cast<int>(gt) ^ group) & 1;  // the group's first step
      const int sb = group;
      for (int i = begin; i < nt; i += 2) {
        const int64_t g = gt + i;
        if (!wait_all(kSFull + sb, static_cast<uint32_t>((g >> 1) & 1)) ||
            !wait_all(kInfo + static_cast<int>(g & 3), static_cast<uint32_t>((g >> 2) & 1))) {
          failed = true;
          break;
        }
        tc_fence_after();
        const int n0 = it.sp.key(it.t0 + i);
        const uint8_t* const info = gbase + C::kOffInfo + (g & 3) * C::kInfoBytes;
        const bool inside = n0 + kTcKeys - 1 <= see.lo_pos &&
                            (n0 >= see.hi_pos - see.left || n0 + kTcKeys <= see.sinks);
        // The largest x: S in 32 columns at a time, read again for the exponentials
        // (a row of 128 beside them does not fit the registers of two groups). Over
        // S come the x of 4 bits, and -inf where a key is not seen; 16 bits: whose
        // page is not there (4 bits: the key's numbers say so).
        bool masked = !inside;
        [[maybe_unused]] uint32_t have = ~0u;  // bit j: the page of keys 16 j .. of the step is there
        if constexpr (!Q4) {
          // (a bit for each of kAtoms copies of a page's keys)
          const uint32_t there = *reinterpret_cast<const uint32_t*>(info);
          const int shift = min(7, p.c.shift);
          if (there != (1u << ((kTcKeys >> shift) * C::kAtoms)) - 1u) {
            masked = true;
            have = 0u;
            for (int j = 0; j < kTcKeys / 16; ++j)
              have |= (there >> ((16 * j >> shift) * C::kAtoms) & 1u) << j;
          }
        }
        float m8[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) m8[j] = -INFINITY;
        const uint32_t s_addr = lane_addr + kColS + sb * kTcKeys;
        // (16 bits: the next columns come while these are worked on; 4 bits: no registers)
        constexpr int kAhead = Q4 ? 0 : 1;
        uint32_t xs[1 + kAhead][32];
        auto columns_of = [&](int c) { tc_ld32(s_addr + 32 * c, xs[c & kAhead]); };
        if (kAhead) columns_of(0);
#pragma unroll kUnroll
        for (int c = 0; c < kTcKeys / 32; ++c) {
          uint32_t(&x)[32] = xs[c & kAhead];
          if (!kAhead) columns_of(c);
          tc_wait_ld();
          if (kAhead && c + 1 < kTcKeys / 32) columns_of(c + 1);
          if constexpr (Q4) {
            const ulonglong2* const num = reinterpret_cast<const ulonglong2*>(info);
            const uint64_t ka2 = pair(ka, ka), kb2 = pair(kb, kb);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const ulonglong2 st = num[8 * c + j], md = num[32 + 8 * c + j], lg = num[64 + 8 * c + j];
              const uint64_t s0 = pair(__uint_as_float(x[4 * j]), __uint_as_float(x[4 * j + 1]));
              const uint64_t s1 = pair(__uint_as_float(x[4 * j + 2]), __uint_as_float(x[4 * j + 3]));
              const float2 x0 = unpair(fma2(mul2(st.x, ka2), s0, fma2(md.x, kb2, lg.x)));
              const float2 x1 = unpair(fma2(mul2(st.y, ka2), s1, fma2(md.y, kb2, lg.y)));
              x[4 * j] = __float_as_uint(x0.x), x[4 * j + 1] = __float_as_uint(x0.y);
              x[4 * j + 2] = __float_as_uint(x1.x), x[4 * j + 3] = __float_as_uint(x1.y);
            }
          }
          if (masked) {
            uint32_t bits = seen(pos, n0 + 32 * c);
            if constexpr (!Q4)
              bits &= (have >> (2 * c) & 1u ? 0xffffu : 0u) | (have >> (2 * c) & 2u ? ~0xffffu : 0u);
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!(bits >> j & 1u)) x[j] = kNoRow;
          }
#pragma unroll
          for (int j = 0; j < 32; ++j) m8[j & 7] = fmaxf(m8[j & 7], __uint_as_float(x[j]));
          if (Q4 || masked) tc_st32(s_addr + 32 * c, x);
        }
        if (Q4 || masked) tc_wait_st();
        if (!Q4 && masked) {
          // V rows that no query sees may hold anything (this thread's: key `row`)
          if (!wait_all(kVFull + sb, static_cast<uint32_t>((g >> 1) & 1))) {
            failed = true;
            break;
          }
          bool nobody = see.nobody(n0 + row);
          if (see.gaps()) {  // the tile's queries asked, 32 at a time, about the warp's 32 keys
            const int m0 = it.rt * (rows_tile / p.hpg);
            const int m1 = min(m0 + rows_tile / p.hpg, p.M);
            uint32_t some = 0u;
            for (int m = m0 + lane; m < m1; m += 32)
              some |= seen(pa_position(p, it.b, m), n0 + 32 * quarter);
            nobody = !(__reduce_or_sync(kFull, some) >> lane & 1u);
          }
          if (nobody) {
#pragma unroll
            for (int c = 0; c < D / 8; ++c)
              *reinterpret_cast<uint4*>(gbase + C::kOffV + sb * C::kTile + (c >> 3) * C::kAtomBytes +
                                        row * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();  // before P is handed over
        }
        float mx = fmaxf(fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3])),
                         fmaxf(fmaxf(m8[4], m8[5]), fmaxf(m8[6], m8[7])));
        if constexpr (!Q4) mx *= ka;
        constexpr float kBelow = kPaBelow<Q4 || !BF16>;
        const bool move = mx > ref + (kPaSlack + kBelow);
        mx -= kBelow;
        if (kAhead) columns_of(0);
        if (__any_sync(kFull, move)) {
          const float alpha = move ? ex2(ref - mx) : 1.f;
          if (i >= 2) {  // (the group's last PV is over: this S came after it)
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tc_ld32(lane_addr + kColO + sb * 128 + 32 * c, o);
              tc_wait_ld();
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
              tc_st32(lane_addr + kColO + sb * 128 + 32 * c, o);
            }
            tc_wait_st();
          }
          if (move) {
            l *= alpha;
            mid_sum *= alpha;
            ref = mx;
            neg = -mx;
          }
        }
        uint64_t l2[2] = {0, 0}, s2[2] = {0, 0};  // sums of pairs
        const uint64_t neg2 = pair(neg, neg), ka2 = pair(ka, ka);
        // 32 columns: exponentials, their sums and P
        auto exps = [&](const uint32_t* x, int q) {
          uint32_t pw[16];
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            uint64_t y[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              y[j] = pair(__uint_as_float(x[4 * c + 2 * j]), __uint_as_float(x[4 * c + 2 * j + 1]));
              const float2 v = unpair(Q4 ? add2(y[j], neg2) : fma2(y[j], ka2, neg2));
              const float e0 = ex2(v.x), e1 = ex2(v.y);
              y[j] = pair(e0, e1);
              pw[2 * c + j] = pack2_t<BF16 && !Q4>(e0, e1);
            }
            if constexpr (Q4) {
              const ulonglong2* const num = reinterpret_cast<const ulonglong2*>(info);
              const ulonglong2 rs = num[96 + 8 * q + c], rm = num[128 + 8 * q + c];
              l2[0] = fma2(y[0], rs.x, l2[0]);
              l2[1] = fma2(y[1], rs.y, l2[1]);
              s2[0] = fma2(y[0], rm.x, s2[0]);
              s2[1] = fma2(y[1], rm.y, s2[1]);
            } else {
              l2[0] = add2(l2[0], y[0]);
              l2[1] = add2(l2[1], y[1]);
            }
          }
          tc_st16(lane_addr + kColS + sb * kTcKeys + 16 * q, pw);  // (S of them is read)
        };
#pragma unroll kUnroll
        for (int q = 0; q < kTcKeys / 32; ++q) {
          if (!kAhead) columns_of(q);
          tc_wait_ld();
          if (kAhead && q + 1 < kTcKeys / 32) columns_of(q + 1);
          exps(xs[q & kAhead], q);
        }
        const float2 lsum = unpair(add2(l2[0], l2[1]));
        l += lsum.x + lsum.y;
        if constexpr (Q4) {
          const float2 ssum = unpair(add2(s2[0], s2[1]));
          mid_sum += ssum.x + ssum.y;
        }
        tc_wait_st();
        tc_fence_before();
        mbar_arrive(bar(kPFull + sb));
      }
      if (failed) break;
      // epilogue: the groups' sums joined, half of the row's columns each; O is
      // released to the next item's PVs. (The next item is looked up meanwhile.)
      const bool whole = it.t0 == 0 && it.t1 == it.sp.n;
      const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (it.t0 == 0 ? 1 : 0);
      const int64_t out_row = (static_cast<int64_t>(it.b) * p.M + mq) * p.H + h;
      const int64_t lse_at = (static_cast<int64_t>(it.b) * p.H + h) * p.M + mq;
      it.next(p, count, rows_tile);
      place();
      float top = -INFINITY, f_own = 0.f, f_other = 0.f;
      if (nt > 0) {
        const int64_t gl = gt + nt - 1;
        if (!wait_all(kPvDone + static_cast<int>(gl & 1), static_cast<uint32_t>((gl >> 1) & 1)) ||
            (nt > 1 && !wait_all(kPvDone + static_cast<int>((gl - 1) & 1),
                                 static_cast<uint32_t>(((gl - 1) >> 1) & 1)))) {
          failed = true;
          break;
        }
        float4* const stat = reinterpret_cast<float4*>(gbase + C::kOffStat);
        stat[128 * group + row] = make_float4(ref, l, mid_sum, 0.f);
        mbar_arrive(bar(kMerge));
        if (!wait_all(kMerge, n & 1)) {
          failed = true;
          break;
        }
        tc_fence_after();
        const float4 other = stat[128 * (group ^ 1) + row];
        top = fmaxf(ref, other.x);
        f_own = ref == top ? 1.f : ex2(ref - top);
        f_other = other.x == top ? 1.f : ex2(other.x - top);
        l = fmaf(other.y, f_other, l * f_own);
        mid_sum = fmaf(other.z, f_other, mid_sum * f_own);
      }
      const bool none = whole && (l == 0.f || pos < 0);
      const float inv = !whole ? 1.f : none ? 0.f : 1.f / l;
#pragma unroll kUnroll
      for (int c = 0; c < D / 64; ++c) {
        float o[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) o[j] = 0.f;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (nt <= 0 || (nt == 1 && x != static_cast<int>(gt & 1))) continue;  // (had no step)
          const float f = x == group ? f_own : f_other;
          uint32_t v[32];
          tc_ld32(lane_addr + kColO + 128 * x + group * (D / 2) + 32 * c, v);
          tc_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = fmaf(__uint_as_float(v[j]), f, o[j]);
        }
        if (mine) {
          const int64_t col = group * (D / 2) + 32 * c;
          uint16_t* const dst = p.o + out_row * D + col;
          float* const piece = p.piece + slot * rows_tile * D + (col * rows_tile + row * 8);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            float e[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              // (4 bits: columns are in the codes' order, and p mid_v is added)
              const float v = Q4 ? o[16 * q + (j & 8) + code_place(j & 7)] + mid_sum : o[16 * q + j];
              e[j] = none ? 0.f : v * inv;
            }
            if (whole) {
              const uint4 lo = pack8<BF16>(e), hi = pack8<BF16>(e + 8);
              store32(dst + 16 * q, lo, hi);
            } else {
#pragma unroll
              for (int j = 0; j < 16; j += 8)
                store32(piece + (16 * q + j) * rows_tile, words(e + j), words(e + j + 4));
            }
          }
        }
        __syncwarp();
      }
      if (nt > 0) {
        tc_fence_before();
        mbar_arrive(bar(kOEmpty));
      }
      if (mine && group == 0) {
        if (!whole)
          reinterpret_cast<float2*>(p.piece + 2 * static_cast<int64_t>(p.ctas) * rows_tile *
                                                  D)[slot * rows_tile + row] = make_float2(top, l);
        else if (p.lse != nullptr)
          p.lse[lse_at] = none ? -INFINITY : pa_lse(top, l);
      }
      gt += nt;
      if (nt > 0) ++n;
    }
  };
  // ---- loaders (4 bits): thread <-> key of the step ----
  auto loader = [&]() {
    if constexpr (Q4) {
      constexpr int kLanes = D / 32;         // lanes of a row of codes, 16 bytes each
      constexpr int kRowsAt = 32 / kLanes;   // rows that a warp loads at once
      constexpr int W = kLanes;              // 16-byte words of a lane
      const int key_in = threadIdx.x & 127;
      auto wait_all = [&](int b, uint32_t parity) {
        return __all_sync(kFull, wait_phase(bar(b), parity, kWaitLimitNs));
      };
      // Register j of a lane is of row kRowsAt j + lane / kLanes of the warp's 32: the
      // first half of them of keys 0 to 15, in one page, the others of 16 to 31.
      const int row0 = lane / kLanes, in_page = (1 << p.c.shift) - 1;
      // (D = 128: lanes of the second atom take their words in another order, or they
      // would meet the first atom's banks)
      const bool turned = D == 128 && (lane & 2) != 0;
      uint32_t place[4];  // of a word's chunk in the operands
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int ch = 4 * (lane % kLanes) + (turned ? q ^ 2 : q);
        place[q] = ((key_in & ~31) + row0) * 128 + (ch >> 3) * C::kAtomBytes +
                   (((ch & 7) ^ (row0 & 7)) << 4);
      }
      for (; it.more && !failed; it.next(p, count, rows_tile)) {
        const int nt = it.t1 - it.t0;
        if (nt <= 0) continue;
        const PaSight see{it.sp.lo_pos, it.sp.hi_pos, p.left, p.sinks};
        const int32_t* const table = p.c.table + static_cast<int64_t>(it.b) * p.c.cols;
        const int64_t in_row = row0 * p.c.kt + it.sh.group * p.c.kh + 16 * (lane % kLanes);
        // a step's page is looked up a step before its codes, and those a step
        // before they are stored (and nothing is done with it until then: a warp
        // waits where it first uses what it has loaded)
        int id_next = -1;
        bool there_next = false;
        uint4 k_next[W], v_next[W];
        uint32_t ks_next = 0, vs_next = 0;
        auto look = [&](int t) {
          id_next = -1;
          const int col = (it.sp.key(t) + key_in) >> p.c.shift;
          if (t < it.t1 && col < p.c.cols) id_next = __ldg(table + col);
        };
        auto fetch = [&](int t) {
          const int page = id_next < p.c.pages ? id_next : -1;
          const int key = it.sp.key(t) + key_in, off = key & in_page;
          there_next = page >= 0 && !see.nobody(key);
          // (rows that nobody sees come along: the codes are finite, whatever they are)
          const int64_t at = page * p.c.kp + (off & ~15) * p.c.kt;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int pg = __shfl_sync(kFull, page, 16 * half);
            const int64_t o = __shfl_sync(kFull, at, 16 * half) + in_row;
#pragma unroll
            for (int j = 0; j < W / 2; ++j) {
              uint4 &kw = k_next[half * (W / 2) + j], &vw = v_next[half * (W / 2) + j];
              kw = vw = make_uint4(0, 0, 0, 0);
              if (pg >= 0) {
                kw = __ldg(reinterpret_cast<const uint4*>(p.c.k + o + j * kRowsAt * p.c.kt));
                vw = __ldg(reinterpret_cast<const uint4*>(p.c.v + o + j * kRowsAt * p.c.kt));
              }
            }
          }
          if (there_next) {
            const int64_t so = ((page * static_cast<int64_t>(p.G) + it.sh.group) << p.c.shift) + off;
            ks_next = __ldg(p.c.ks + so);
            vs_next = __ldg(p.c.vs + so);
          }
          look(t + 1);
        };
        auto store = [&](uint8_t* tile, const uint4 (&w)[W]) {
#pragma unroll
          for (int j = 0; j < W; ++j) {
            const uint32_t u[4] = {turned ? w[j].z : w[j].x, turned ? w[j].w : w[j].y,
                                   turned ? w[j].x : w[j].z, turned ? w[j].y : w[j].w};
#pragma unroll
            for (int q = 0; q < 4; ++q)
              *reinterpret_cast<uint4*>(tile + place[q] + j * kRowsAt * 128) = codes_chunk(u[q]);
          }
          fence_proxy_async_smem();
        };
        look(it.t0);
        fetch(it.t0);
        for (int i = 0; i < nt; ++i) {
          const int64_t g = gt + i;
          const int s = static_cast<int>(g & 1);
          const uint32_t prev = static_cast<uint32_t>(((g - 2) >> 1) & 1);
          uint4 k[W], v[W];
#pragma unroll
          for (int j = 0; j < W; ++j) k[j] = k_next[j], v[j] = v_next[j];
          const bool have = there_next;
          const float kstep = __uint_as_float(ks_next << 16),
                      klow = __uint_as_float(ks_next & 0xffff0000u);
          const float vstep = __uint_as_float(vs_next << 16),
                      vlow = __uint_as_float(vs_next & 0xffff0000u);
          fetch(it.t0 + i + 1);
          if (g >= 2 && !wait_all(kKEmpty + s, prev)) {
            failed = true;
            break;
          }
          // the key's numbers: K's step and middle, log2 of V's step, its reciprocal
          // and the middle by that. (Their slot was last read by the softmax of
          // step g - 4, which is over: the S after its PV is.)
          const float some = pa_step(vstep, vlow);
          const float rs = rcp_approx(some), rm = fmaf(8.f, vstep, vlow) * rs;
          // a row that is not finite reaches the queries that see it by their x alone: the
          // others multiply its numbers by 0
          const bool fine = rs < INFINITY && fabsf(rm) < INFINITY;
          // rows without a step: codes of 8, whose c - 8 is 0
          const uint32_t flat = __ballot_sync(kFull, vstep == 0.f);
          if (flat != 0u) {
#pragma unroll
            for (int j = 0; j < W; ++j)
              if (flat >> (kRowsAt * j + row0) & 1u)
                v[j] = make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);
          }
          float* const num =
              reinterpret_cast<float*>(gbase + C::kOffInfo + (g & 3) * C::kInfoBytes) + key_in;
          num[0] = have ? kstep : 0.f;
          num[128] = have ? fmaf(8.f, kstep, klow) : 0.f;
          num[256] = !have ? -INFINITY : fine ? lg2_approx(some) : __uint_as_float(0x7fc00000u);
          num[384] = have && fine ? rs : 0.f;
          num[512] = have && fine ? rm : 0.f;
          mbar_arrive(bar(kInfo + static_cast<int>(g & 3)));
          store(gbase + C::kOffK + s * C::kTile, k);
          mbar_arrive(bar(kKFull + s));
          if (g >= 2 && !wait_all(kVEmpty + s, prev)) {
            failed = true;
            break;
          }
          store(gbase + C::kOffV + s * C::kTile, v);
          mbar_arrive(bar(kVFull + s));
        }
        gt += nt;
      }
    }
  };
  if constexpr (Q4) {
    // 512 threads of 128 registers; 88 + 2 x 144 + 136 = 4 x 128
    if (warp < C::kSoftWarp) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 88;\n" ::: "memory");
      if (warp == 1) issuer();
    } else if (warp < C::kLoadWarp) {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 144;\n" ::: "memory");
      softmax();
    } else {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 136;\n" ::: "memory");
      loader();
    }
  } else {
    if (warp == 0) producer(std::false_type{});
    else if (warp == 1) issuer();
    else if (warp == 2) producer(std::true_type{});
    else if (warp >= C::kSoftWarp) softmax();
  }

  if (failed && lane == 0) report_timeout();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tc_dealloc(tmem, kTcTmem);
  }
}

template <int D, bool BF16, bool Q4>
int launch(PagedProblem& p, cudaStream_t st) {
  using C = TcCfg<D, Q4>;
  constexpr CUtensorMapDataType dt =
      BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  CUtensorMap tq, tk, tv;
  memset(&tq, 0, sizeof(tq));  // (4 bits: none is used)
  memset(&tk, 0, sizeof(tk));
  memset(&tv, 0, sizeof(tv));
  const int rows = tc_rows_of_tile(p.hpg);
  if constexpr (!Q4) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return NSA_ERR_LAUNCH;
    // Q as (d, head, query, sequence): the heads of a KV head and whole queries in a box
    const int64_t sh = p.H > 1 ? p.qh : D, sm = p.M > 1 ? p.qm : p.H * sh,
                  sb = p.B > 1 ? p.qb : p.M * sm;
    const cuuint64_t dims[4] = {D, static_cast<cuuint64_t>(p.H), static_cast<cuuint64_t>(p.M),
                                static_cast<cuuint64_t>(p.B)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(2 * sh), static_cast<cuuint64_t>(2 * sm),
                                   static_cast<cuuint64_t>(2 * sb)};
    const cuuint32_t box[4] = {kBoxCols, static_cast<cuuint32_t>(p.hpg),
                               static_cast<cuuint32_t>(rows / p.hpg), 1};
    const cuuint32_t one[4] = {1, 1, 1, 1};
    if (enc(&tq, dt, 4, const_cast<uint8_t*>(p.q), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return NSA_ERR_LAUNCH;
    const int64_t page = int64_t(1) << p.c.shift;
    const int keys = page < kTcKeys ? static_cast<int>(page) : kTcKeys;
    if (!encode_kv_map_strided(&tk, p.c.k, p.c.pages, page, p.G, D, keys, dt, p.c.kp / 2,
                               p.c.kt / 2, p.c.kh / 2) ||
        !encode_kv_map_strided(&tv, p.c.v, p.c.pages, page, p.G, D, keys, dt, p.c.vp / 2,
                               p.c.vt / 2, p.c.vh / 2))
      return NSA_ERR_LAUNCH;
  }
  auto kern = paged_attn_tc_kernel<D, BF16, Q4>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) !=
      cudaSuccess)
    return NSA_ERR_LAUNCH;
  p.ctas = kPaSms;
  const int64_t all = static_cast<int64_t>(p.items) * p.groups;
  const int64_t blocks = p.cut || all > kPaSms ? kPaSms : all;
  kern<<<static_cast<unsigned>(blocks), C::kThreads, C::kSmem, st>>>(p, rows, tq, tk, tv);
  return cudaGetLastError() == cudaSuccess ? NSA_OK : NSA_ERR_LAUNCH;
}

}  // namespace

int launch_paged_tc(PagedProblem& p, const nsa_kv_cache* kv, int64_t D, bool bf16,
                    cudaStream_t st) {
  const bool q4 = kv->bits == 4;
  if (D == 64) {
    if (bf16) return q4 ? launch<64, true, true>(p, st) : launch<64, true, false>(p, st);
    return q4 ? launch<64, false, true>(p, st) : launch<64, false, false>(p, st);
  }
  if (bf16) return q4 ? launch<128, true, true>(p, st) : launch<128, true, false>(p, st);
  return q4 ? launch<128, false, true>(p, st) : launch<128, false, false>(p, st);
}

int paged_tc_read_and_clear_status(unsigned int* value) { return read_and_clear_status(value); }

}  // namespace nsa
