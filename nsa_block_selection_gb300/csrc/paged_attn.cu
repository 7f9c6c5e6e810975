// Attention of new tokens over a paged cache of keys and values, 16-bit or
// 4-bit, for sm_103a.
//
// Query (b, m) at position p sees key j of its sequence iff j <= p, and
// j >= p - left or j < sinks (the first tokens, which stay visible behind a
// window), and the page of j is there. With x_j = scale log2(e) q.k_j:
//   O = sum_j 2^(x_j - r) v_j / l,  l = sum_j 2^(x_j - r),
//   LSE = ln 2 (r + log2 l),
// r a reference that follows the largest x (by steps of 8, and 7 below it where p is
// rounded to fp16: p <= 2^8, 2^15). One pass over the keys; x, p, sums and O are fp32,
// p is rounded to 16 bits for the product with V, and what the rounding leaves is
// multiplied too (but for a bf16 O over 4 bits).
//
// Rows. A row tile is 8 or 16 of the M H/G (query, head) rows of a KV head, the
// N of the products: S^T (16 keys x rows) = K Q^T and O^T (D x rows) += V^T P^T
// (mma.sync m16n8k16). A decoding step has 8 rows or fewer, of which a 128-row
// tcgen05 tile would be 1/16 full; what bounds the call is the cache's bytes.
//
// Keys. A warp takes 16-key tiles, which lie in one page each; the four warps of
// a CTA take its tiles in turn and are joined in shared memory at the end of an
// item (a row tile and a KV head, or a few neighbouring KV heads). The tiles of
// all items are dealt to the CTAs in equal, contiguous shares, whatever the
// lengths of the sequences: positions are on the device, so every CTA forms the
// running count of the items' tiles for itself. An item that a share's border
// cuts leaves fp32 pieces, which paged_attn_join_kernel adds in a fixed order:
// equal calls give equal bits.
//
// 16 bits: tiles come by TMA through a ring of shared-memory slots of the warp's
// own, ldmatrix makes the operands.
//
// 4 bits: k = low + step c gives q.k = step (q.c) + low sum(q): the codes
// themselves enter the product, as fp16 subnormals (c 2^-24, or 16 c 2^-24 for
// the upper four bits of a byte, which Q's entries are divided by 16 for): a
// mask, or a shift and a mask, makes two entries. Q's rows are scaled by a power
// of two into fp16's range. For V, p' = 2^(x + log2 step - r) is the product's
// operand (r follows x + log2 step) and p = p' / step; with
// v = (low + 8 step) + step (c - 8) it sums p' (c - 8), and p (low + 8 step) is
// summed beside it. A slot of the CTA's one ring holds 128 rows, 32 for each warp,
// and the warps issue the copies in turn: neighbouring heads of a token lie in one
// 128-byte line, so a CTA takes two or four of them at once.
//
// Many rows (drafts, pieces of a prompt) go to paged_attn_tc_kernel.
//
// What bounds it. 16 bits: the cache's bytes, and what surrounds them: a token of 64 +
// 8 heads of 128 over 65,536 keys takes 44 to 48 us (5.6 to 6.1 TB/s of 268 MB), of
// which some 6 us are the first positions, pages and copies and the join; 48 windowed
// sequences of 32 + 4 heads (1028 keys each, 102 MB) 22 us in one kernel. 4 bits: the
// warps' instructions, some 300 for 16 keys of a KV head: 64 ragged sequences of up to
// 16,384 tokens of 64 + 8 heads (580 MB) 146 us, 4.0 TB/s, a warp issues in 53 % of
// the clocks at 12 warps an SM.

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
#include "status.cuh"

namespace nsa {
namespace {

template <int D, bool Q4, int NT>
struct PaCfg {
  // CTAs of an SM. 16 bits: 128 KB of copies in flight (a token over 65,536 keys 44
  // us; three CTAs 48); 4 bits: registers for two tiles at once
  static constexpr int kPerSm = !Q4 ? 2 : D == 64 ? 4 : NT == 1 ? 3 : 2;
  // 16 bits: a ring for each warp, 16 keys of K and V in a slot. 4 bits: one for
  // the CTA, 128 rows of K and V and their scales in a slot, 32 for each warp.
  static constexpr int kStages = Q4 ? 3 : 2;
  static constexpr int kRings = Q4 ? 1 : kPaWarps;
  static constexpr int kKv = Q4 ? kPaSlotRows * (D / 2) : kPaTile * 2 * D;  // K's (or V's) part
  static constexpr int kScales = Q4 ? kPaSlotRows * 4 : 0;
  static constexpr int kSlot = 2 * kKv + 2 * kScales;
  static constexpr int kRing = kRings * kStages * kSlot;
  static constexpr int kKeys = Q4 ? kPaSlotRows / kPaTile : 1;  // first keys kept for a slot
  static constexpr int kPad = D + 4;  // row stride of the joined O, in floats
  static constexpr int kJoin = kPaWarps * 8 * NT * kPad * 4;
  static constexpr int kOffStat = kRing > kJoin ? kRing : kJoin;  // 2 floats a warp and row
  static constexpr int kOffBar = kOffStat + kPaWarps * 8 * NT * 8;
  static constexpr int kOffKey = kOffBar + kRings * kStages * 16;  // (full, empty)
  static constexpr int kOffCount = kOffKey + kRings * kStages * kKeys * 4;
  static constexpr int kSmem = kOffCount + (kPaItems + 1) * 4 + 1024;
};

// The state of one warp's rows: column 2 c + j of n-tile nt belongs to lanes of
// c = lane % 4; rows of O^T to lane / 4.
template <int D, int NT>
struct PaRows {
  float acc[NT][D / 16][4];
  float ref[NT][2], neg[NT][2], l[NT][2];
  float base_v[NT][2];  // 4 bits: sum of p (low + 8 step)
  int pos[NT][2];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
        acc[nt][i][0] = acc[nt][i][1] = acc[nt][i][2] = acc[nt][i][3] = 0.f;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        ref[nt][j] = -INFINITY;
        neg[nt][j] = l[nt][j] = base_v[nt][j] = 0.f;
      }
    }
  }

  // Moves the references that an element of x exceeds by more than the slack (F16: p is
  // rounded to fp16).
  template <bool F16, int TILES>
  __device__ __forceinline__ void follow(const float (&x)[TILES][NT][4]) {
    constexpr float kOver = kPaSlack + kPaBelow<F16>;
    float top[NT][2];
    bool move = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        top[nt][j] = fmaxf(x[0][nt][j], x[0][nt][j + 2]);
#pragma unroll
        for (int u = 1; u < TILES; ++u)
          top[nt][j] = fmaxf(top[nt][j], fmaxf(x[u][nt][j], x[u][nt][j + 2]));
        move = move || top[nt][j] > ref[nt][j] + kOver;
      }
    if (!__any_sync(kFull, move)) return;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float mx = top[nt][j];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
        if (mx > ref[nt][j] + kOver) {  // (alike in the lanes of a column)
          mx -= kPaBelow<F16>;
          const float f = ex2(ref[nt][j] - mx);  // 0 while nothing was seen
          l[nt][j] *= f;
          base_v[nt][j] *= f;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            acc[nt][i][j] *= f;
            acc[nt][i][j + 2] *= f;
          }
          ref[nt][j] = mx;
          neg[nt][j] = -mx;
        }
      }
    }
  }
};

// What the 16-bit words of `two` leave of a and b, in the same type.
template <bool BF16>
__device__ __forceinline__ uint32_t pa_rest(uint32_t two, float a, float b) {
  float2 f;
  if constexpr (BF16)
    f = make_float2(__uint_as_float(two << 16), __uint_as_float(two & 0xffff0000u));
  else
    f = __half22float2(*reinterpret_cast<const __half2*>(&two));
  return pack2_t<BF16>(a - f.x, b - f.y);
}

// ---- 16 bits -----------------------------------------------------------

// One tile of the ring: S^T, the softmax step and O^T. EDGE: some query does not
// see some key of it.
template <int D, bool BF16, int NT, bool EDGE>
__device__ __forceinline__ void pa_tile16(PaRows<D, NT>& a, const uint32_t (&qf)[NT][D / 16][2],
                                          uint32_t slot, int n0, const PaSight& see, float sl2) {
  constexpr int KS = D / 16;
  const int lane = threadIdx.x & 31, r = lane >> 2;
  const uint32_t vt = slot + kPaTile * 2 * D;
  if constexpr (EDGE) {
    // V rows that no query sees may hold anything: they become zeros. (Each question is
    // asked of the columns' own positions: between windows there may be gaps. The four
    // lanes of a key pair hold all columns.)
    bool one = false, two = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        one = one || !see.hidden(n0 + r, a.pos[nt][j]);
        two = two || !see.hidden(n0 + r + 8, a.pos[nt][j]);
      }
    const uint32_t seen[2] = {__ballot_sync(kFull, one), __ballot_sync(kFull, two)};
    for (int i = lane; i < kPaTile * (D / 8); i += 32) {
      const int row = i / (D / 8), ch = i % (D / 8);
      if ((seen[row >> 3] >> (4 * (row & 7)) & 15u) == 0u)
        st_shared_zero16(vt + (ch >> 3) * kBoxBytes + row * 128 + (ch & 7) * 16);
    }
    fence_proxy_async_smem();  // (before the slot's next copy)
    __syncwarp();
  }
  float sc[NT][2][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) sc[nt][0][i] = sc[nt][1][i] = 0.f;
  const int krow = (lane & 7) + (lane & 8);
#pragma unroll
  for (int k = 0; k < KS; ++k) {
    const int ch = 2 * k + (lane >> 4);
    uint32_t a0, a1, a2, a3;
    ldsm_x4(slot + (ch >> 3) * kBoxBytes + krow * 128 + (((ch & 7) ^ (krow & 7)) << 4), a0, a1, a2,
            a3);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      mma_16816_t<BF16>(sc[nt][k & 1], a0, a1, a2, a3, qf[nt][k][0], qf[nt][k][1]);
  }
  // element i: key n0 + r + 8 (i / 2), column 2 c + i % 2
  float x[1][NT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[0][nt][i] = (sc[nt][0][i] + sc[nt][1][i]) * sl2;
      if (EDGE && see.hidden(n0 + r + 8 * (i >> 1), a.pos[nt][i & 1])) x[0][nt][i] = -INFINITY;
    }
  a.template follow<!BF16>(x);
  // P^T as B operand, and what its rounding leaves: the copies bound the call, so a
  // second product costs nothing, and O is off by its own rounding alone
  uint32_t pf[NT][2], pl[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float e[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      e[i] = ex2(x[0][nt][i] + a.neg[nt][i & 1]);
      a.l[nt][i & 1] += e[i];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t two = pack2_t<BF16>(e[2 * i], e[2 * i + 1]);
      pf[nt][i] = movmatrix_t(two);
      pl[nt][i] = movmatrix_t(pa_rest<BF16>(two, e[2 * i], e[2 * i + 1]));
    }
  }
  const int vrow = (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
  for (int i = 0; i < KS; ++i) {
    const int ch = 2 * i + ((lane >> 3) & 1);
    uint32_t a0, a1, a2, a3;
    ldsm_x4_t(vt + (ch >> 3) * kBoxBytes + vrow * 128 + (((ch & 7) ^ (vrow & 7)) << 4), a0, a1, a2,
              a3);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      mma_16816_t<BF16>(a.acc[nt][i], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
      mma_16816_t<BF16>(a.acc[nt][i], a0, a1, a2, a3, pl[nt][0], pl[nt][1]);
    }
  }
}

// ---- 4 bits ------------------------------------------------------------

// mma_16816, or the same from zero (without registers to be cleared first).
__device__ __forceinline__ void pa_mma_from(bool zero, float (&d)[4], uint32_t a0, uint32_t a1,
                                            uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if (zero)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%10,%10,%10};\n"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
  else
    mma_16816(d, a0, a1, a2, a3, b0, b1);
}

// Key of MMA row i of a tile. Any order serves; in this one the 16- and 8-byte
// loads of 128-byte swizzled rows meet no bank twice.
__device__ __forceinline__ int pa_row4(int i) { return (i & 14) ^ (i & 1 ? 5 : 0); }

// Where a lane's words of a tile lie in a slot: K's of rows r and r + 8 of S^T
// (the c-th quarter of a row), V's for its rows 2 c, 2 c + 1, 2 c + 8, 2 c + 9 (the
// r-th eighth of a row), and the scales of rows r and r + 8.
struct PaLanes {
  uint32_t k[2], v[4], scale;
};

// S^T of a tile as x in the log2 domain, with log2 of V's step; mid and rstep: V's
// low + 8 step and 1 / step of the lane's two keys.
template <int D, int NT, bool EDGE>
__device__ __forceinline__ void pa_scores4(const PaRows<D, NT>& a, const uint8_t* kt,
                                           const uint8_t* scales, const PaLanes& at, int n0,
                                           const uint32_t (&qf)[NT][D / 16][2],
                                           const float (&ka)[NT][2], const float (&kb)[NT][2],
                                           const PaSight& see, float (&x)[NT][4], float (&mid)[2],
                                           float (&rstep)[2]) {
  constexpr int W = D / 32;
  const int key = n0 + pa_row4((threadIdx.x & 31) >> 2);
  float sc[NT][2][4];
  uint32_t w[2][W];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if constexpr (D == 128) {
      const uint4 v = *reinterpret_cast<const uint4*>(kt + at.k[j]);
      w[j][0] = v.x, w[j][1] = v.y, w[j][W - 2] = v.z, w[j][W - 1] = v.w;
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(kt + at.k[j]);
      w[j][0] = v.x, w[j][1] = v.y;
    }
  }
  uint32_t ks[2], vs[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    ks[j] = *reinterpret_cast<const uint32_t*>(scales + at.scale + 32 * j);
    vs[j] = *reinterpret_cast<const uint32_t*>(scales + kPaSlotRows * 4 + at.scale + 32 * j);
    // keys that no query sees may hold anything
    if (EDGE && see.nobody(key + 8 * j)) ks[j] = vs[j] = 0u;
  }
#pragma unroll
  for (int j = 0; j < W; ++j) {
    const uint32_t u = w[0][j], v = w[1][j], u8 = u >> 8, v8 = v >> 8;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      pa_mma_from(j == 0, sc[nt][0], u & 0x000f000fu, v & 0x000f000fu, u & 0x00f000f0u,
                  v & 0x00f000f0u, qf[nt][2 * j][0], qf[nt][2 * j][1]);
      pa_mma_from(j == 0, sc[nt][1], u8 & 0x000f000fu, v8 & 0x000f000fu, u8 & 0x00f000f0u,
                  v8 & 0x00f000f0u, qf[nt][2 * j + 1][0], qf[nt][2 * j + 1][1]);
    }
  }
  float kstep[2], klow[2], lstep[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    kstep[j] = __uint_as_float(ks[j] << 16);
    klow[j] = __uint_as_float(ks[j] & 0xffff0000u);
    const float step = __uint_as_float(vs[j] << 16), low = __uint_as_float(vs[j] & 0xffff0000u);
    const float some = pa_step(step, low);
    mid[j] = fmaf(8.f, step, low);
    rstep[j] = rcp_approx(some);
    lstep[j] = lg2_approx(some);
    if (step == 0.f) rstep[j] = -rstep[j];
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[nt][i] = fmaf(kstep[i >> 1] * ka[nt][i & 1], sc[nt][0][i] + sc[nt][1][i],
                      fmaf(klow[i >> 1], kb[nt][i & 1], lstep[i >> 1]));
      if (EDGE && see.hidden(key + 8 * (i >> 1), a.pos[nt][i & 1])) x[nt][i] = -INFINITY;
    }
}

// p' of a tile, its sums, and O^T. The codes lose their mean in the product, by
// operands of -8 (-128 for the upper ones): sums of p' c, all of one sign, would
// grow with the keys, and what every addition to them loses with them, while
// their difference from 8 sum p' does not. (Flat attention over 8192 keys: 0.6 %
// of O instead of 0.17 with lower and upper codes in one sum.)
constexpr uint32_t kLess8 = 0x80088008u, kLess128 = 0x80808080u;

// REST: also the product with what the rounding of p' leaves, r (c - 8) = r c - 8 r, so
// that an fp16 O is off by little more than its own rounding (without: 1.4 times that;
// a bf16 one is anyway).
template <int D, int NT, bool EDGE, bool REST>
__device__ __forceinline__ void pa_values4(PaRows<D, NT>& a, const uint8_t* vt, const PaLanes& at,
                                           int n0, const PaSight& see, const float (&x)[NT][4],
                                           const float (&mid)[2], const float (&rstep)[2]) {
  constexpr int W = D / 64;
  const int key = n0 + pa_row4((threadIdx.x & 31) >> 2);
  uint32_t w[4][W];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (D == 128) {
      const uint2 v = *reinterpret_cast<const uint2*>(vt + at.v[j]);
      w[j][0] = v.x, w[j][W - 1] = v.y;
    } else {
      w[j][0] = *reinterpret_cast<const uint32_t*>(vt + at.v[j]);
    }
  }
  uint32_t pf[NT][2];
  [[maybe_unused]] uint32_t pl[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float e[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = ex2(x[nt][i] + a.neg[nt][i & 1]);
    uint32_t p0 = pack_half2(e[0], e[1]), p1 = pack_half2(e[2], e[3]);
    [[maybe_unused]] uint32_t r0 = 0u, r1 = 0u;
    if constexpr (REST) {
      r0 = pa_rest<false>(p0, e[0], e[1]);
      r1 = pa_rest<false>(p1, e[2], e[3]);
    }
    if (rstep[0] < 0.f) p0 = r0 = 0u;
    if (rstep[1] < 0.f) p1 = r1 = 0u;
    if constexpr (REST) {
      const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&r0));
      const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&r1));
      a.base_v[nt][0] = fmaf(f0.x + f1.x, -8.f, a.base_v[nt][0]);
      a.base_v[nt][1] = fmaf(f0.y + f1.y, -8.f, a.base_v[nt][1]);
      pl[nt][0] = movmatrix_t(r0);
      pl[nt][1] = movmatrix_t(r1);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float md = mid[i >> 1], pr = e[i] * fabsf(rstep[i >> 1]);
      if (EDGE && see.hidden(key + 8 * (i >> 1), a.pos[nt][i & 1])) md = pr = 0.f;
      a.l[nt][i & 1] += pr;
      a.base_v[nt][i & 1] = fmaf(pr, md, a.base_v[nt][i & 1]);
    }
    pf[nt][0] = movmatrix_t(p0);
    pf[nt][1] = movmatrix_t(p1);
  }
#pragma unroll
  for (int j = 0; j < W; ++j) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {  // entries 0..3, 4..7 of a word, two keys each
      const uint32_t sel = half ? 0x7632u : 0x5410u;
      const uint32_t u = __byte_perm(w[0][j], w[1][j], sel);
      const uint32_t v = __byte_perm(w[2][j], w[3][j], sel);
      const uint32_t u8 = u >> 8, v8 = v >> 8;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float(&lo)[4] = a.acc[nt][4 * j + 2 * half];
        float(&hi)[4] = a.acc[nt][4 * j + 2 * half + 1];
        mma_16816(lo, kLess8, kLess128, kLess8, kLess128, pf[nt][0], pf[nt][1]);
        mma_16816(lo, u & 0x000f000fu, u & 0x00f000f0u, v & 0x000f000fu, v & 0x00f000f0u, pf[nt][0],
                  pf[nt][1]);
        mma_16816(hi, kLess8, kLess128, kLess8, kLess128, pf[nt][0], pf[nt][1]);
        mma_16816(hi, u8 & 0x000f000fu, u8 & 0x00f000f0u, v8 & 0x000f000fu, v8 & 0x00f000f0u,
                  pf[nt][0], pf[nt][1]);
        if constexpr (REST) {
          mma_16816(lo, u & 0x000f000fu, u & 0x00f000f0u, v & 0x000f000fu, v & 0x00f000f0u,
                    pl[nt][0], pl[nt][1]);
          mma_16816(hi, u8 & 0x000f000fu, u8 & 0x00f000f0u, v8 & 0x000f000fu, v8 & 0x00f000f0u,
                    pl[nt][0], pl[nt][1]);
        }
      }
    }
  }
}

// A warp's 32 keys of a slot: two tiles, at once where the registers hold both (64
// sequences over 4 bits 146 us, one after the other 150).
template <int D, int NT, bool EDGE, bool REST>
__device__ __forceinline__ void pa_step4(PaRows<D, NT>& a, const uint8_t* slot,
                                         const uint8_t* scales, const PaLanes& at, int row_bytes,
                                         const int (&n0)[2], const uint32_t (&qf)[NT][D / 16][2],
                                         const float (&ka)[NT][2], const float (&kb)[NT][2],
                                         const PaSight& see) {
  constexpr int kTogether = D == 64 && NT == 2 ? 1 : 2;
#pragma unroll
  for (int u0 = 0; u0 < 2; u0 += kTogether) {
    float x[kTogether][NT][4], mid[kTogether][2], rstep[kTogether][2];
#pragma unroll
    for (int u = 0; u < kTogether; ++u)
      pa_scores4<D, NT, EDGE>(a, slot + (u0 + u) * kPaTile * row_bytes,
                              scales + (u0 + u) * kPaTile * 4, at, n0[u0 + u], qf, ka, kb, see, x[u],
                              mid[u], rstep[u]);
    a.template follow<true>(x);
#pragma unroll
    for (int u = 0; u < kTogether; ++u)
      pa_values4<D, NT, EDGE, REST>(
          a, slot + kPaSlotRows * (D / 2) + (u0 + u) * kPaTile * row_bytes, at, n0[u0 + u], see,
          x[u], mid[u], rstep[u]);
  }
}

// Q's rows of a row tile as B operands. 4 bits: scaled by 2^e into fp16, in the
// order of the codes under the masks; x = step dot ka + low kb.
template <int D, bool BF16, bool Q4, int NT>
__device__ __forceinline__ void pa_queries(const PagedProblem& p, int b, int rt, int head,
                                           uint32_t (&qf)[NT][D / 16][2], float (&ka)[NT][2],
                                           float (&kb)[NT][2]) {
  const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int row = rt * 8 * NT + nt * 8 + r;
    const int m = row / p.hpg;
    const bool in = row < p.rows;
    const uint32_t* src = reinterpret_cast<const uint32_t*>(
        p.q + 2 * (b * p.qb + m * p.qm + (head * p.hpg + row - m * p.hpg) * p.qh));
    if constexpr (!Q4) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        qf[nt][k][0] = in ? src[8 * k + c] : 0u;
        qf[nt][k][1] = in ? src[8 * k + 4 + c] : 0u;
      }
    } else {
      constexpr int W = D / 32;  // words of codes, and 8 entries of q each, of this lane
      uint4 v[W];
      float top = 0.f;
#pragma unroll
      for (int j = 0; j < W; ++j) {
        v[j] = in ? reinterpret_cast<const uint4*>(src)[c * W + j] : make_uint4(0, 0, 0, 0);
        float f[8];
        unpack8<BF16>(v[j], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(f[i]));
      }
      top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
      top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
      // the largest entry between 2^13 and 2^14 (a row that is not finite, or
      // zero, as it is)
      int e = 0;
      if (top > 0.f && top < INFINITY)
        e = min(13 - (static_cast<int>(__float_as_uint(top) >> 23) - 127), 100);
      const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < W; ++j) {
        float f[8];
        unpack8<BF16>(v[j], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          f[i] = __half2float(__float2half_rn(f[i] * up));
          sum += f[i];
        }
        // entries (0, 4), (1, 5) / 16 and (2, 6), (3, 7) / 16
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
  }
}

template <int D, bool BF16, bool Q4, int NT>
__global__ void __launch_bounds__(kPaThreads, PaCfg<D, Q4, NT>::kPerSm)
    paged_attn_kernel(const PagedProblem p, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV) {
  using C = PaCfg<D, Q4, NT>;
  constexpr int kRowsTile = 8 * NT;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const gbase = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, c = lane & 3;
  int* const count = reinterpret_cast<int*>(gbase + C::kOffCount);
  float* const stat = reinterpret_cast<float*>(gbase + C::kOffStat);
  const int ring = Q4 ? 0 : warp;
  int* const keys = reinterpret_cast<int*>(gbase + C::kOffKey) + ring * C::kStages * C::kKeys;
  const uint32_t bars = base + C::kOffBar + ring * C::kStages * 16;  // full, then empty
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kRings; ++i)
      for (int st = 0; st < C::kStages; ++st) {
        const uint32_t bar = base + C::kOffBar + (2 * i * C::kStages + st) * 8;
        mbar_init(bar, Q4 ? p.split : 1);
        if (Q4) mbar_init(bar + C::kStages * 8, kPaWarps);
      }
    fence_mbar_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  PaShare sh{0, 0, 0, 0, 0};
  asm volatile("griddepcontrol.launch_dependents;\n");  // the join waits for this grid's end
  if (p.cut) {
    sh = pa_share<kPaThreads>(p, kRowsTile, count, reinterpret_cast<int*>(stat));
    pa_zeros<D>(p, kRowsTile, count);
  } else {
    sh.item = blockIdx.x / p.groups;
    sh.group = blockIdx.x - sh.item * p.groups;
    __syncthreads();
  }
  // the warps of a head, this one's place among them, and its head of the item
  const int warps_head = kPaWarps / p.heads_item, warp_in = warp % warps_head;
  const int head_in = warp / warps_head;
  // (with several row tiles the keys are read again)
  const uint64_t policy = p.tiles > 1 ? l2_policy_evict_normal() : l2_policy_evict_first();
  [[maybe_unused]] PaLanes lanes{};
  [[maybe_unused]] int row_bytes = 0;
  if constexpr (Q4) {
    // a row holds a token's codes of the item's heads: 128 or 64 bytes, swizzled
    // by TMA, or 32
    row_bytes = p.heads_item * (D / 2);
    auto at = [&](int row, int byte) {
      const uint32_t o = row * row_bytes + head_in * (D / 2) + byte;
      const uint32_t swizzle = row_bytes == 128 ? 7u : row_bytes == 64 ? 3u : 0u;
      return (o ^ ((o >> 7 & swizzle) << 4)) + static_cast<uint32_t>(warp_in * 32 * row_bytes);
    };
#pragma unroll
    for (int j = 0; j < 2; ++j) lanes.k[j] = at(pa_row4(r) + 8 * j, c * (D / 8));
#pragma unroll
    for (int j = 0; j < 4; ++j)
      lanes.v[j] = at(pa_row4(2 * c + (j & 1)) + 8 * (j >> 1), r * (D / 16));
    lanes.scale = 4 * ((head_in << p.step_shift) + warp_in * 32 + pa_row4(r));
  }
  bool failed = false;
  uint32_t issued = 0, done = 0;  // slots of the ring, over all items
  [[maybe_unused]] uint32_t stage = 0, phase = 0;  // 4 bits: of the next slot to be read
  for (bool more = !p.cut || sh.begin < sh.end; more;) {
    const int b = sh.item / p.tiles, rt = sh.item - b * p.tiles;
    const int head = sh.group * p.heads_item + head_in;
    const PaSpan sp = pa_span<true>(p, b, rt, kRowsTile);
    // steps [t0, t1) of the item, after its cost
    int t0 = 0, t1 = sp.n;
    if (p.cut) {
      const int64_t first = sh.at + p.item_cost;
      t0 = static_cast<int>(min(max(sh.begin - first, static_cast<int64_t>(0)),
                                static_cast<int64_t>(sp.n)));
      t1 = static_cast<int>(min(max(sh.end - first, static_cast<int64_t>(0)),
                                static_cast<int64_t>(sp.n)));
    }
    const PaSight see{sp.lo_pos, sp.hi_pos, p.left, p.sinks};

    const int in_page = (1 << p.c.shift) - 1;
    PaRows<D, NT> a;
    a.clear();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int rw = rt * kRowsTile + nt * 8 + 2 * c + j;
        a.pos[nt][j] = rw < p.rows ? pa_position(p, b, rw / p.hpg) : -1;
      }
    uint32_t qf[NT][D / 16][2];
    float ka[NT][2], kb[NT][2];

    if constexpr (Q4) {
      // The warps issue the item's steps in turn: step t is warp t % 4's. Lane j
      // of a window of 32 holds where the j-th copy of this warp's steps lies
      // (`split` to a step), looked up one window ahead, and issues it.
      const int steps = t1 - t0;
      const int split_shift = __ffs(p.split) - 1;
      const int rows = 1 << (p.step_shift - split_shift);  // tokens of a copy
      int key_l = -1, page_l = -1, key_next = -1, page_next = -1;
      auto look = [&](int j) {
        const int t = (j >> split_shift) * kPaWarps + warp, part = j & (p.split - 1);
        page_next = -1;
        if (t < steps) {
          key_next = sp.key(t0 + t) + part * rows;
          page_next = page_of(p.c, b, key_next);
        }
      };
      auto issue = [&](int t) {  // (t % 4 = warp: this warp's turn)
        const uint32_t g = issued + t;  // of the ring
        const int s = g % C::kStages;
        const uint32_t bar = bars + 8 * s;
        // the step that had the slot has been read by all warps
        if (g >= C::kStages &&
            !__all_sync(kFull, wait_phase(bar + 8 * C::kStages, (g / C::kStages - 1) & 1,
                                          kWaitLimitNs))) {
          failed = true;
          return;
        }
        const int e = (t / kPaWarps << split_shift) & 31;
        if (e == 0) {
          key_l = key_next;
          page_l = page_next;
          look((t / kPaWarps << split_shift) + 32 + lane);
        }
        if (lane >= e && lane < e + p.split) {
          const int first = (lane - e) * rows;  // of the copy's rows, in the step
          // each tile's first key, and whether every query sees all of it (bit 0)
          for (int i = 0; i < rows; i += kPaTile)
            keys[s * C::kKeys + (first + i) / kPaTile] =
                page_l < 0 ? kNoKey : key_l + i + (see.all(key_l + i) ? 1 : 0);
          if (page_l < 0) {
            mbar_arrive(bar);  // a page that is not there
          } else {
            const int off = key_l & in_page, h0 = sh.group * p.heads_item;
            const uint32_t dst = base + s * C::kSlot;
            mbar_arrive_expect_tx(bar, 2 * p.heads_item * rows * (D / 2 + 4));
            tma_load_4d(dst + first * row_bytes, &tmK, bar, h0 * (D / 2), off, page_l, 0, policy);
            tma_load_4d(dst + C::kKv + first * row_bytes, &tmV, bar, h0 * (D / 2), off, page_l, 0,
                        policy);
            for (int h = 0; h < p.heads_item; ++h) {
              const int64_t so =
                  ((page_l * static_cast<int64_t>(p.G) + h0 + h) << p.c.shift) + off;
              const uint32_t sc = dst + 2 * C::kKv + 4 * ((h << p.step_shift) + first);
              bulk_load(sc, p.c.ks + so, rows * 4, bar);
              bulk_load(sc + C::kScales, p.c.vs + so, rows * 4, bar);
            }
          }
        }
        __syncwarp();
      };
      look(lane);
      for (int t = 0; t < C::kStages - 1 && t < steps && !failed; ++t)
        if (t % kPaWarps == warp) issue(t);
      pa_queries<D, BF16, true, NT>(p, b, rt, head, qf, ka, kb);
      for (int t = 0; t < steps && !failed; ++t) {
        if (!__all_sync(kFull, wait_phase(bars + 8 * stage, phase, kWaitLimitNs))) {
          failed = true;
          // leave nothing in flight: of this warp's copies, step t's or the next one's (step
          // t + 2 is issued when t has been read, and a turn is four steps)
          const int own = t % kPaWarps == warp ? t : t + 1;
          const uint32_t g = issued + own;
          if (own % kPaWarps == warp && own < steps)
            wait_phase(bars + 8 * (g % C::kStages), (g / C::kStages) & 1, kWaitLimitNs);
          break;
        }
        const int k0 = keys[stage * C::kKeys + 2 * warp_in];
        const int k1 = keys[stage * C::kKeys + 2 * warp_in + 1];
        const int n0[2] = {k0 & ~1, k1 & ~1};
        const uint8_t* const slot = gbase + stage * C::kSlot;
        const uint8_t* const scales = slot + 2 * C::kKv;
        if (k0 & k1 & 1)
          pa_step4<D, NT, false, !BF16>(a, slot, scales, lanes, row_bytes, n0, qf, ka, kb, see);
        else if (!see.nothing(n0[0]) || !see.nothing(n0[1]))
          pa_step4<D, NT, true, !BF16>(a, slot, scales, lanes, row_bytes, n0, qf, ka, kb, see);
        __syncwarp();  // the slot has been read
        if (lane == 0) mbar_arrive(bars + 8 * (C::kStages + stage));
        if (++stage == C::kStages) {
          stage = 0;
          phase ^= 1;
        }
        const int next = t + C::kStages - 1;
        if (next < steps && next % kPaWarps == warp) issue(next);
      }
      issued += steps;
    } else {
      // This warp's tiles are t0 + warp_in + warps_head k. Lane j of a window of
      // 32 holds the page of the j-th, looked up one window ahead.
      int tile_k = 0, page_l = -1, page_next = -1;
      auto look = [&](int k) {
        const int t = t0 + warp_in + warps_head * k;
        page_next = t < t1 ? page_of(p.c, b, sp.key(t)) : -1;
      };
      look(lane);
      auto issue = [&]() {  // the next tile that has a page, into its slot
        int key = -1, page = -1;
        for (int t; page < 0 && (t = t0 + warp_in + warps_head * tile_k) < t1; ++tile_k) {
          if ((tile_k & 31) == 0) {
            page_l = page_next;
            look(tile_k + 32 + lane);
          }
          page = __shfl_sync(kFull, page_l, tile_k & 31);
          key = sp.key(t);
        }
        if (page < 0) return;
        if (lane == 0) {
          const int s = issued % C::kStages, off = key & in_page;
          const uint32_t bar = bars + 8 * s;
          const uint32_t dst = base + (warp * C::kStages + s) * C::kSlot;
          keys[s] = key;
          mbar_arrive_expect_tx(bar, C::kSlot);
#pragma unroll
          for (int i = 0; i < D / 64; ++i) {
            tma_load_4d(dst + i * kBoxBytes, &tmK, bar, i * 64, head, off, page, policy);
            tma_load_4d(dst + C::kKv + i * kBoxBytes, &tmV, bar, i * 64, head, off, page, policy);
          }
        }
        ++issued;
      };
      if (!failed)
        for (int s = 0; s < C::kStages; ++s) issue();
      pa_queries<D, BF16, false, NT>(p, b, rt, head, qf, ka, kb);
      while (!failed && done != issued) {
        const int s = done % C::kStages;
        if (!__all_sync(kFull, wait_phase(bars + 8 * s, (done / C::kStages) & 1, kWaitLimitNs))) {
          failed = true;
          break;
        }
        const int n0 = keys[s];
        const uint32_t slot = base + (warp * C::kStages + s) * C::kSlot;
        if (see.all(n0))
          pa_tile16<D, BF16, NT, false>(a, qf, slot, n0, see, p.sl2);
        else
          pa_tile16<D, BF16, NT, true>(a, qf, slot, n0, see, p.sl2);
        __syncwarp();  // the slot has been read
        ++done;
        issue();
      }
    }

    if (t0 == t1 && p.cut) break;  // (the share ends within an item's cost)
    // ---- the warps' results, joined in shared memory
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          a.l[nt][j] += __shfl_xor_sync(kFull, a.l[nt][j], o);
          a.base_v[nt][j] += __shfl_xor_sync(kFull, a.base_v[nt][j], o);
        }
    // every warp is done with the ring; where one's wait gave up, all leave
    if (__syncthreads_or(failed)) {
      failed = true;
      break;
    }
    float* const joined = reinterpret_cast<float*>(gbase);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int row = nt * 8 + 2 * c + j;
        float* const dst = joined + (warp * kRowsTile + row) * C::kPad;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          if constexpr (Q4) {
            // byte i % 4 of word D / 64 r + i / 4 of a row: its lower code, and its
            // upper, 16 times as large
            const int d = 8 * (D / 64 * r + (i >> 2)) + 2 * (i & 3);
            dst[d] = fmaf(a.acc[nt][i][j], 16777216.f, a.base_v[nt][j]);
            dst[d + 1] = fmaf(a.acc[nt][i][j + 2], 1048576.f, a.base_v[nt][j]);
          } else {
            dst[16 * i + r] = a.acc[nt][i][j];
            dst[16 * i + r + 8] = a.acc[nt][i][j + 2];
          }
        }
        if (r == 0) {
          stat[2 * (warp * kRowsTile + row)] = a.ref[nt][j];
          stat[2 * (warp * kRowsTile + row) + 1] = a.l[nt][j];
        }
      }
    __syncthreads();
    const bool whole = t0 == 0 && t1 == sp.n;
    // a piece of an item that begins in this share: slot 2 CTA + 1; that
    // goes on from an earlier one: 2 CTA
    const int64_t slot_id = 2 * static_cast<int64_t>(blockIdx.x) + (t0 == 0 ? 1 : 0);
    const int piece_rows = p.heads_item * kRowsTile;
    for (int i = threadIdx.x; i < piece_rows * (D / 2); i += kPaThreads) {
      const int prow = i / (D / 2), d = 2 * (i % (D / 2));
      const int hd = prow / kRowsTile, row = prow % kRowsTile;  // head of the item, row
      const int rw = rt * kRowsTile + row;
      if (rw >= p.rows) continue;
      const int w0 = hd * warps_head, w1 = w0 + warps_head;
      float m = -INFINITY, sum = 0.f, o0 = 0.f, o1 = 0.f;
      for (int w = w0; w < w1; ++w) m = fmaxf(m, stat[2 * (w * kRowsTile + row)]);
      for (int w = w0; w < w1; ++w) {
        const float ref = stat[2 * (w * kRowsTile + row)];
        // (a warp that saw nothing has a sum of 0, or NaN where scores are)
        const float f = ref == m ? 1.f : ex2(ref - m);
        const float2 v =
            *reinterpret_cast<const float2*>(joined + (w * kRowsTile + row) * C::kPad + d);
        sum = fmaf(f, stat[2 * (w * kRowsTile + row) + 1], sum);
        o0 = fmaf(f, v.x, o0);
        o1 = fmaf(f, v.y, o1);
      }
      if (whole) {
        const int mq = rw / p.hpg;
        const int h = (sh.group * p.heads_item + hd) * p.hpg + rw - mq * p.hpg;
        if (__ldg(p.pos + b * p.pos_b + mq) < 0) sum = o0 = o1 = 0.f;  // padding
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        reinterpret_cast<uint32_t*>(
            p.o + ((static_cast<int64_t>(b) * p.M + mq) * p.H + h) * D)[d >> 1] =
            pack2_t<BF16>(o0 * inv, o1 * inv);
        if (d == 0 && p.lse != nullptr)
          p.lse[(static_cast<int64_t>(b) * p.H + h) * p.M + mq] = pa_lse(m, sum);
      } else {
        float* const dst = p.piece + (slot_id * piece_rows + prow) * D + d;
        *reinterpret_cast<float2*>(dst) = make_float2(o0, o1);
        if (d == 0) {
          float* const st =
              p.piece + (2 * static_cast<int64_t>(p.ctas) * D + 2 * slot_id) * piece_rows + 2 * prow;
          st[0] = m;
          st[1] = sum;
        }
      }
    }
    fence_proxy_async_smem();  // the ring's next copies come after this
    __syncthreads();
    if (!p.cut) break;
    // the next item of the share
    sh.at += sp.n + p.item_cost;
    if (++sh.group == p.groups) {
      sh.group = 0;
      do ++sh.item;
      while (sh.item < p.items && count[sh.item + 1] == count[sh.item]);
    }
    more = sh.at < sh.end;
  }
  if (failed) {
    if constexpr (!Q4) {  // leave nothing in flight
      for (; done != issued; ++done)
        wait_phase(bars + 8 * (done % C::kStages), (done / C::kStages) & 1, kWaitLimitNs);
    }
    if (lane == 0) report_timeout();
  }
}

// Items that shares have cut: their pieces joined in order. A CTA takes `rows_cta`
// rows of an item (blockIdx.x: the item, or, where there are more items than shares,
// the share that it begins in and does not end in: a prompt of 4096 tokens has 1024
// items, and their CTAs took 45 us), D / 4 threads a row; the pieces are dealt to the
// sets of threads that are left. A thread merges its pieces as it loads them,
// statistics and values at once, four in flight: the kernel is a chain of latencies
// (the counts, the pieces, the sets).
constexpr int kJoinThreads = 256;

struct PaPiece {
  float m = -INFINITY, sum = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);

  __device__ __forceinline__ void add(float2 s, float4 v) {
    const float top = fmaxf(m, s.x);
    const float f = m == top ? 1.f : ex2(m - top), g = s.x == top ? 1.f : ex2(s.x - top);
    m = top;
    sum = fmaf(sum, f, s.y * g);
    o.x = fmaf(o.x, f, v.x * g), o.y = fmaf(o.y, f, v.y * g);
    o.z = fmaf(o.z, f, v.z * g), o.w = fmaf(o.w, f, v.w * g);
  }
};

template <int D, bool BF16>
__global__ void __launch_bounds__(kJoinThreads)
    paged_attn_join_kernel(const PagedProblem p, int rows_tile, int rows_cta, bool by_share) {
  constexpr int kLanes = D / 4;  // threads of a row
  __shared__ float4 part[kJoinThreads];
  __shared__ float2 part_stat[kJoinThreads];
  __shared__ int holds;
  int item = blockIdx.x / p.groups, group = blockIdx.x - item * p.groups;
  // (launched while the kernel before is at its end; its results are there from here on)
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const int64_t per = p.count[p.items + 1];
  if (by_share) {  // the item that holds the first step of the next share
    const int64_t next = (static_cast<int64_t>(blockIdx.x) + 1) * per;
    if (threadIdx.x == 0) holds = -1;
    __syncthreads();
    for (int i = threadIdx.x; i < p.items; i += kJoinThreads)
      if (p.count[i] * p.groups <= next && next < p.count[i + 1] * p.groups) holds = i;
    __syncthreads();
    item = holds;
    if (item < 0) return;  // (the shares after this one are empty)
    const int64_t c0 = p.count[item];
    group = static_cast<int>((next - c0 * p.groups) / (p.count[item + 1] - c0));
  }
  const int piece_rows = p.heads_item * rows_tile;
  const int b = item / p.tiles, rt = item - b * p.tiles;
  const int sets = kJoinThreads / (kLanes * rows_cta);
  const int d = threadIdx.x % kLanes, lrow = threadIdx.x / kLanes % rows_cta;
  const int set = threadIdx.x / (kLanes * rows_cta);
  const int prow = blockIdx.y * rows_cta + lrow, hd = prow / rows_tile;
  const int rw = rt * rows_tile + prow - hd * rows_tile;
  const bool in = prow < piece_rows && rw < p.rows;
  const int mq = rw / p.hpg, h = (group * p.heads_item + hd) * p.hpg + rw - mq * p.hpg;
  const bool padding = in && __ldg(p.pos + b * p.pos_b + mq) < 0;
  const int64_t c0 = p.count[item], c1 = p.count[item + 1];
  const int64_t n = c1 - c0 - p.item_cost;  // (below 0: no step)
  const int64_t at = c0 * p.groups + group * (c1 - c0) + p.item_cost;
  const int first = static_cast<int>(at / per);
  const int last = n > 0 ? static_cast<int>((at + n - 1) / per) : first;
  if (first == last || (by_share && first != static_cast<int>(blockIdx.x))) return;
  const int pieces = last - first + 1;
  const float* const stats = p.piece + 2 * static_cast<int64_t>(p.ctas) * piece_rows * D;
  const int at_row = p.many ? ((d >> 1) * piece_rows + prow) * 8 + (d & 1) * 4 : prow * D + 4 * d;
  PaPiece a;
  if (in) {
    for (int i0 = set; i0 < pieces; i0 += 4 * sets) {
      float2 s[4];
      float4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = i0 + k * sets;
        s[k] = make_float2(-INFINITY, 0.f);
        v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < pieces) {
          const int64_t slot = 2 * static_cast<int64_t>(first + i) + (i == 0 ? 1 : 0);
          s[k] = *reinterpret_cast<const float2*>(stats + (slot * piece_rows + prow) * 2);
          v[k] = *reinterpret_cast<const float4*>(p.piece + slot * piece_rows * D + at_row);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) a.add(s[k], v[k]);
    }
  }
  part[threadIdx.x] = a.o;
  part_stat[threadIdx.x] = make_float2(a.m, a.sum);
  __syncthreads();
  if (set != 0 || !in) return;
  for (int k = 1; k < sets; ++k) {
    const int t = threadIdx.x + k * kLanes * rows_cta;
    a.add(part_stat[t], part[t]);
  }
  if (padding) a = PaPiece{};
  const float inv = a.sum == 0.f ? 0.f : 1.f / a.sum;
  reinterpret_cast<uint2*>(p.o + ((static_cast<int64_t>(b) * p.M + mq) * p.H + h) * D)[d] =
      make_uint2(pack2_t<BF16>(a.o.x * inv, a.o.y * inv), pack2_t<BF16>(a.o.z * inv, a.o.w * inv));
  if (d == 0 && p.lse != nullptr)
    p.lse[(static_cast<int64_t>(b) * p.H + h) * p.M + mq] = pa_lse(a.m, a.sum);
}

// ---- host ---------------------------------------------------------------

// Row tiles: 8 rows where a KV head has no more, else 16; from kTcRows rows on (4 bits:
// kTcRows4, as two tiles of 16 are faster there) whole queries of up to 128
// (paged_attn_tc_kernel). Measured, 8 rows a token, D = 128, tiles of 16 against
// paged_attn_tc_kernel: 16 sequences of up to 4000 tokens over 16 bits, 16 rows 36
// and 39 us, 24 rows 53 and 38; of up to 8000 over 4 bits, 24 rows 75 and 91, 32 rows
// 82 and 90, 40 rows 120 and 82.
constexpr int64_t kTcRows = 17, kTcRows4 = 33;
constexpr int64_t kPaCounts = ((kPaItems + 2) * 8 + 127) / 128 * 128;  // bytes of the counts
bool many_rows(int64_t rows, int64_t hpg, bool q4) {
  return rows >= (q4 ? kTcRows4 : kTcRows) && hpg <= 128;
}
int rows_of_tile(int64_t rows, int64_t hpg, bool q4) {
  return rows <= 8 ? 8 : many_rows(rows, hpg, q4) ? tc_rows_of_tile(hpg) : 16;
}

// KV heads of an item. The rows of a 4-bit cache are 64 or 32 bytes for each
// head of a token, but what comes from memory is 128: neighbouring heads are
// read by the warps of one CTA at the same time.
int heads_of_item(int64_t G, int64_t D, int64_t bits) {
  if (bits == 16) return 1;
  return D == 64 && G % 4 == 0 ? 4 : G % 2 == 0 ? 2 : 1;
}

// The codes of `heads` neighbouring KV heads, 128, 64 or 32 bytes, of `tokens`
// tokens; a token's heads lie side by side.
bool encode_code_map(CUtensorMap* tm, const void* ptr, const KvPages& c, int64_t G, int64_t D,
                     int heads, int tokens) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t row = static_cast<cuuint64_t>(G * (D / 2)), page = cuuint64_t(1) << c.shift;
  const cuuint32_t wide = static_cast<cuuint32_t>(heads * (D / 2));
  const cuuint64_t dims[4] = {row, page, static_cast<cuuint64_t>(c.pages), 1};
  const cuuint64_t strides[3] = {row, row * page, row * page * c.pages};
  const cuuint32_t box[4] = {wide, static_cast<cuuint32_t>(tokens), 1, 1};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return enc(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(ptr), dims, strides, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE,
             wide == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
             : wide == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                          : CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int check_paged(int64_t B, int64_t M, int64_t H, int64_t G, int64_t D, int dtype) {
  const int rc = check_rope(B, M, H, G, D, 0, 0, 0, 0.f, dtype, NSA_F32);
  if (rc != NSA_OK) return rc;
  if (H % G != 0) return NSA_ERR_GROUPS;
  if (M * (H / G) >= int64_t(1) << 30) return NSA_ERR_SHAPE;
  const int64_t rows = M * (H / G), tile = rows_of_tile(rows, H / G, true);
  if (B * ((rows + tile - 1) / tile) * G >= int64_t(1) << 31) return NSA_ERR_SHAPE;
  return NSA_OK;
}

// Bytes of a call over a cache of 4 or 16 bits; 0: no item is cut.
int64_t workspace_for(int64_t B, int64_t M, int64_t H, int64_t G, int64_t D, int64_t tokens,
                      int64_t window_left, int64_t sinks, bool q4) {
  const int64_t rows = M * (H / G), tile = rows_of_tile(rows, H / G, q4);
  const int64_t items = B * ((rows + tile - 1) / tile);
  if (items == 0 || items > kPaItems) return 0;
  if (tokens > int64_t(1) << 30) tokens = int64_t(1) << 30;
  // where every query sees few keys an item is short enough for one CTA, without a
  // second kernel
  if (M == 1 && window_left >= 0 && window_left < tokens && sinks < tokens &&
      window_left + 1 + sinks < tokens)
    tokens = window_left + 1 + sinks;
  // (and the running count of steps has 32 bits)
  if (tokens <= (items * G >= kPaSms ? kPaWholeMany : kPaWhole) ||
      items * (tokens / kPaTile + 32) >= int64_t(1) << 31)
    return 0;
  // two pieces of every share, and the running counts
  const int64_t ctas = many_rows(rows, H / G, q4) ? kPaSms : kPaMostPerSm * kPaSms;
  const int heads = many_rows(rows, H / G, q4) ? 1 : heads_of_item(G, D, q4 ? 4 : 16);
  return 2 * ctas * heads * tile * (D + 2) * 4 + kPaCounts;
}

// The pieces of items that shares have cut.
template <int D, bool BF16>
int launch_join(const PagedProblem& p, int rows_tile, cudaStream_t st) {
  if (!p.cut) return NSA_OK;
  // rows of a CTA: as many as leave a CTA for each SM, so that few items
  // have their many pieces added by many threads
  const int rows = p.heads_item * rows_tile;
  int rows_cta = 1024 / D;  // a thread for every four entries
  const int64_t all = static_cast<int64_t>(p.items) * p.groups;
  const bool by_share = all >= p.ctas;
  while (rows_cta > 1 && all * (rows / rows_cta) < kPaSms) rows_cta >>= 1;
  if (rows_cta > 8) rows_cta = 8;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(by_share ? p.ctas - 1 : all),
                     (rows + rows_cta - 1) / rows_cta);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, paged_attn_join_kernel<D, BF16>, PagedProblem(p), rows_tile,
                         rows_cta, by_share) != cudaSuccess)
    return NSA_ERR_LAUNCH;
  return NSA_OK;
}

template <int D, bool BF16, bool Q4, int NT>
int launch_paged(PagedProblem& p, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t st) {
  using C = PaCfg<D, Q4, NT>;
  static_assert((C::kSmem + 1024) * C::kPerSm <= 233472, "CTAs of an SM");
  static_assert(C::kPerSm <= kPaMostPerSm, "pieces in the workspace");
  auto kern = paged_attn_kernel<D, BF16, Q4, NT>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) !=
      cudaSuccess)
    return NSA_ERR_LAUNCH;
  p.ctas = C::kPerSm * kPaSms;
  const int64_t blocks = p.cut ? p.ctas : static_cast<int64_t>(p.items) * p.groups;
  kern<<<static_cast<unsigned>(blocks), kPaThreads, C::kSmem, st>>>(p, tk, tv);
  if (cudaGetLastError() != cudaSuccess) return NSA_ERR_LAUNCH;
  return launch_join<D, BF16>(p, 8 * NT, st);
}

template <int D, bool BF16>
int launch_paged_d(PagedProblem& p, const nsa_kv_cache* kv, cudaStream_t st) {
  if (p.many) {
    const int rc = launch_paged_tc(p, kv, D, BF16, st);
    return rc != NSA_OK ? rc : launch_join<D, BF16>(p, tc_rows_of_tile(p.hpg), st);
  }
  CUtensorMap tk, tv;
  if (kv->bits == 4) {
    const int wide = kPaSlotRows / p.heads_item, page = 1 << p.c.shift;
    const int tokens = wide < page ? wide : page;
    p.split = wide / tokens;
    if (!encode_code_map(&tk, p.c.k, p.c, p.G, D, p.heads_item, tokens) ||
        !encode_code_map(&tv, p.c.v, p.c, p.G, D, p.heads_item, tokens))
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
  if (p.rows <= 8)
    return kv->bits == 4 ? launch_paged<D, BF16, true, 1>(p, tk, tv, st)
                         : launch_paged<D, BF16, false, 1>(p, tk, tv, st);
  return kv->bits == 4 ? launch_paged<D, BF16, true, 2>(p, tk, tv, st)
                       : launch_paged<D, BF16, false, 2>(p, tk, tv, st);
}

}  // namespace

int paged_read_and_clear_status(unsigned int* value) {
  unsigned int tc = 0u;
  const int rc = read_and_clear_status(value);
  if (rc != NSA_OK) return rc;
  const int rt = paged_tc_read_and_clear_status(&tc);
  *value |= tc;
  return rt;
}

}  // namespace nsa

extern "C" int64_t nsa_paged_attn_workspace_bytes(int64_t B, int64_t M, int64_t H, int64_t G,
                                                  int64_t D, int64_t tokens, int64_t window_left,
                                                  int64_t sinks) {
  using namespace nsa;
  const int rc = check_paged(B, M, H, G, D, NSA_F16);
  if (rc != NSA_OK) return rc;
  if (tokens < 0 || sinks < 0) return NSA_ERR_SHAPE;
  const int64_t a = workspace_for(B, M, H, G, D, tokens, window_left, sinks, false);
  const int64_t b = workspace_for(B, M, H, G, D, tokens, window_left, sinks, true);
  return a > b ? a : b;
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
  if ((rc = take_strides(q_strides, 1, &H, B, M, D, s, 1)) != NSA_OK) return rc;
  if (B == 0 || M == 0) return NSA_OK;
  if (!Q || !O || !positions) return NSA_ERR_NULL;
  if (!aligned(Q, 16) || !aligned(O, 16) || !aligned(LSE, 4) || !aligned(positions, 4))
    return NSA_ERR_ALIGN;
  PagedProblem p{};
  if ((rc = take_cache(cache, page_table, table_cols, B, G, D, true, &p.c)) != NSA_OK) return rc;
  const int64_t need = workspace_for(B, M, H, G, D, table_cols * cache->page_size, window_left,
                                     sinks, cache->bits == 4);
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return NSA_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return NSA_ERR_ALIGN;
  }
  p.q = static_cast<const uint8_t*>(Q);
  p.qb = s[0], p.qm = s[1], p.qh = s[2];
  p.o = static_cast<uint16_t*>(O);
  p.lse = LSE;
  p.pos = positions;
  p.pos_b = positions_stride;
  p.count = static_cast<int64_t*>(workspace);
  p.piece = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kPaCounts);
  p.B = static_cast<int>(B);
  p.M = static_cast<int>(M);
  p.H = static_cast<int>(H);
  p.G = static_cast<int>(G);
  p.hpg = static_cast<int>(H / G);
  p.rows = static_cast<int>(M * (H / G));
  const bool many = p.many = many_rows(p.rows, p.hpg, cache->bits == 4);
  p.heads_item = many ? 1 : heads_of_item(G, D, cache->bits);
  p.groups = p.G / p.heads_item;
  p.step_shift =
      many ? 7 : cache->bits == 16 ? 4 : p.heads_item == 1 ? 7 : p.heads_item == 2 ? 6 : 5;
  p.item_cost = ((many ? kTcItemCost : kPaItemCost) + (1 << p.step_shift) - 1) >> p.step_shift;
  const int tile = rows_of_tile(p.rows, p.hpg, cache->bits == 4);
  p.tiles = (p.rows + tile - 1) / tile;
  p.items = static_cast<int>(B * p.tiles);
  p.cut = need > 0;
  // a window that reaches behind key 0 from any position; sinks as many as a table's tokens
  const int64_t far = 0x7fffffff, tokens = int64_t(1) << 30;
  p.left = static_cast<int>(window_left < 0 || window_left > far ? far : window_left);
  p.sinks = static_cast<int>(sinks > tokens ? tokens : sinks);
  const float sc = scale > 0.f ? scale : 1.0f / sqrtf(static_cast<float>(D));
  p.sl2 = sc * 1.4426950408889634f;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf = dtype == NSA_BF16;
  if (D == 64)
    return bf ? launch_paged_d<64, true>(p, cache, st) : launch_paged_d<64, false>(p, cache, st);
  return bf ? launch_paged_d<128, true>(p, cache, st) : launch_paged_d<128, false>(p, cache, st);
}
