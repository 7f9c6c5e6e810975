// Gradients of the GQA sliding-window (or dense) attention forward for
// sm_103a, on the 5th-generation tensor cores.
//
// Per visible (query i, key j) of a head, with the forward's LSE and O:
//   p = exp(scale q.k - LSE_i),  delta_i = dO_i . O_i,  dP = dO_i . v_j,
//   dS = p (dP - delta_i),
//   dQ_i = scale sum_j dS k_j,  dK_j = scale sum_i dS q_i,  dV_j = sum_i p dO_i
// (dK, dV over the query heads of the KV head too). Scores, p, dP, dS and all
// sums are fp32; p and dS are rounded to the inputs' type for the products
// they enter, gradients once when they are stored.
//
// Two kernels form p and dP each for itself: 7 products of 2 D operations a
// pair instead of the 5 that one pass needs, but no dQ row has to be added up
// in memory. A pass over key tiles adds 4 D bytes of fp32 a (query, key tile)
// to dQ, 64 KB for the 5 x 512 tensor-pipe clocks of a 128 x 128 tile at
// D = 128: 7 TB/s over 152 SMs, twice the 3.6 TB/s that fp32 reductions
// reach here, in an order that changes from run to run. Here every sum is
// made in tensor memory in a fixed order: equal calls give equal bits.
//
// Both kernels are persistent, one CTA to an SM (tensor memory holds one set
// of accumulators), their items dealt in rounds in snake order, and their
// steps of all items one stream: the operands of an item are staged while the
// one before runs, and its gradients leave while the next one runs. Every A
// operand stays in tensor memory, which leaves 64 B a clock of shared-memory
// reads for B: with A in shared memory the 64-column products would need 192
// of the 128 there are (measured: 33 clocks a product against 49).
//
//  0. swa_bwd_vmax_kernel (fp16 alone): the largest |v| of every key tile.
//  1. swa_bwd_dq_kernel: an item is 128 queries of a head (or, with few query
//     tiles, a part of their keys), a step 64 keys. Q and dO are the A operands
//     of S = Q K^T and dP = dO V^T; dS overwrites S and is the A operand of
//     dQ += dS K. S and dP have two buffers each, so the tensor pipe runs S and
//     dP of the next step and dQ of the previous one while eight warps form dS.
//     Four auxiliary warps form delta and move Q and dO in and dQ out. LSE
//     log2 e and delta of every query are left for the second kernel.
//  2. swa_bwd_dkv_kernel: an item is 128 keys of a KV head (or a part of its
//     steps), a step 64 queries of a head: S^T = K Q^T, dP^T = V dO^T,
//     dV += P^T dO, dK += dS^T Q. K and V are the A operands of the first two;
//     P overwrites S, dS dP. At D = 128 the accumulators leave one buffer for
//     each of S and dP, so a step is two groups of 32 queries: one's products
//     run during the other's exponentials; at D = 64 there are two buffers. Two
//     warps issue, (S, dV) and (dP, dK): the waits of one pass while the
//     other's products run.
//  3. swa_bwd_join_dq_kernel, swa_bwd_join_kernel: where tiles were cut, the sum
//     of their fp32 parts.
//
// What bounds it. D = 128: the tensor pipe, busy 68 % (dQ) and 69 % (dK, dV) of
// the clocks at 8192 tokens of 64 + 8 heads, window (512, 0), where the items
// have 10 (dQ) and 80 steps (40 where cut): 165 and 225 us, 6 us of joining,
// DRAM at 3.1 and 1.6 TB/s; a step's products take 1024 (dQ: 768) of its some
// 1530 (1160) clocks, and its barriers, of which one that is over still takes a
// warp 100 to 300 clocks, are most of the rest. 16,384 tokens, window (4096, 0):
// 1.51 and 2.13 ms, 1.8 PFLOP/s over the 7 products; back to back the clock
// falls to 1.6 to 1.9 GHz at the power limit. D = 64 (2 x 16 heads of
// 1500 x 2048: 48 and 70 us): neither the products (396 and 528 of a step's some
// 1000 and 1450 clocks) nor the exponentials (256); what is left is the chain of
// a step from S to its last barrier, and whole tiles in rounds, 96 steps for
// an SM where an even share is 81. Short calls: launches one after another and
// the latency of a few dependent steps (2 x 1000 tokens, 8 + 2 heads: 12, 19 and
// 6 us, with fp16 inputs 13, 22, 6 and 5 for the largest |v|).
//
// Every mbarrier wait is bounded (1 s); a role that gives up sets the status
// word, waits for its own copies, and every role reaches the teardown, which
// frees the tensor memory. The auxiliary warps, which time their waits each for
// itself, vote at their named barriers: one that gave up goes on to the next
// vote, after which all four leave.

#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "common.cuh"
#include "nsa_sel_attn.h"
#include "ptx.cuh"
#include "status.cuh"
#include "tc.cuh"

namespace nsa {
namespace {

constexpr int kBlk = 128;       // queries (dQ) or keys (dK, dV) of a CTA: the M of its products
constexpr int kStep = 64;       // keys (dQ) or queries (dK, dV) of a step
constexpr int kAtomStep = kStep * 128;  // bytes of 64 rows x 64 entries
constexpr int kAtomBlk = kBlk * 128;
constexpr uint32_t kTmemAll = 512;

// fp16 has no exponents below 2^-14 at full precision and none above 2^15. Over
// thousands of keys p is smaller than the one: with fp16 inputs it is carried as
// 2^12 p (at most 4096). dS, as large as dO and V make it, may pass either: it is
// carried as 2^e dS, with an e of its own for every row of dQ and of dK (an
// accumulator's row has one scale), the largest for which a bound of |dP - delta|
// stays below 2^15 (p <= 1; a factor of 2 is left for roundings). By
// Cauchy-Schwarz, |dP - delta| <= |dO_i| |v_j| + |delta_i|, with the largest |v|
// of the key tiles of a row of dQ, and the largest |dO| and |delta| of the query
// blocks of a row of dK. All are exact factors that the epilogues divide out.
// bf16 needs none of it.
template <bool BF16>
struct Shift {
  static constexpr float kP = BF16 ? 0.f : 12.f;
  static constexpr float kPInv = BF16 ? 1.f : 1.f / 4096.f;
};
constexpr int kTopExp = 40;  // of e, where the bound is small or 0

// e for a bound. (One that is not finite comes of a dO, O or V that is not,
// which the products carry into the gradients whatever e is.)
__device__ __forceinline__ int shift_for(float bound) {
  if (!(bound < INFINITY)) return 0;
  return min(kTopExp, 14 - (static_cast<int>(__float_as_uint(bound) >> 23) - 127));
}
__device__ __forceinline__ float pow2(int e) {  // |e| < 127
  return __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
}
// The bit of the largest |dO| that row i of 32 keeps: four rows that a lane reads
// together hold one of each byte.
__device__ __forceinline__ int top_bit(int i) { return (i & 3) * 8 + (i >> 2); }
// Non-negative numbers order as their bits; one that is not finite counts as 0
// (a row that hidden pairs alone use may hold anything).
__device__ __forceinline__ uint32_t finite_bits(float x) {
  return x < INFINITY ? __float_as_uint(x) : 0u;
}

struct SwaBwdProblem {
  const uint16_t *Q, *K, *V, *O, *dO;
  const float* LSE;
  void *dQ, *dK, *dV;
  float* nlse2;   // [B, H, Mp]: Shift::kP - LSE log2 e; -inf for rows without keys
  // [B, H, Mp]: -delta. fp16: the last bits of 32 rows' (which delta, good to some
  // 2^-20, can spare) are the largest |dO| of those rows, a float: top_bit().
  float* ndelta;
  // fp16: the largest |v| of every key tile, until dV is written, in the first
  // 4 bytes of the tile's first row of dV
  const float* vmax;
  int64_t vmax_b, vmax_t, vmax_g;  // its strides over (batch, key tile, KV head)
  float* part;    // [parts, 2 (dK, dV), kBlk, D], or NULL
  float* part_q;  // [parts, kBlk, D] of dQ, or NULL
  int B, M, N, H, Hkv, hpg, Mp, qtiles, ktiles, splits;
  int dq_whole, dq_splits, dq_items;  // the same for the query tiles of the dQ kernel
  int whole_tiles, dkv_items;  // key tiles that are not cut, and all items of the dK, dV kernel
  int left, right;  // clamped to [0, M] and [0, N]: unbounded in effect
  float sl2, scale;
  bool g32;  // gradients fp32 instead of the inputs' type
  bool wide;  // gradients (and parts) 32-byte aligned
};

// An auxiliary warp waits for a whole item of `steps` steps at a time, at its
// last item from the item's start on, which 1 s may not hold: 20 us more for
// each of them (they take under 1 us).
__device__ __forceinline__ uint64_t item_limit_ns(int steps) {
  return kWaitLimitNs + 20000ull * static_cast<uint64_t>(steps);
}

// A matrix descriptor moved by `bytes`: the address field takes the sum as
// it is (shared memory ends below its 2^18 bytes), and an addition leaves the
// issuing warp less to do per MMA than building the descriptor again.
__device__ __forceinline__ uint64_t desc_at(uint64_t desc, uint32_t bytes) {
  const uint32_t lo = static_cast<uint32_t>(desc) + (bytes >> 4);
  return (desc & 0xffffffff00000000ull) | lo;
}

// Two fp32 operations an instruction.
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  return pair(__float_as_uint(lo), __float_as_uint(hi));
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  uint32_t lo, hi;
  asm("mov.b64 {%0, %1}, %2;\n" : "=r"(lo), "=r"(hi) : "l"(v));
  return make_float2(__uint_as_float(lo), __uint_as_float(hi));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// 2^x of both halves.
__device__ __forceinline__ uint64_t ex2_2(uint64_t x) {
  const float2 v = unpair(x);
  return pair(ex2(v.x), ex2(v.y));
}

// Bit c set: column c of 32 lies in [lo, hi].
__device__ __forceinline__ uint32_t seen_bits(int lo, int hi) {
  const uint32_t below = hi < 0 ? 0u : hi >= 31 ? ~0u : (2u << hi) - 1u;
  return lo <= 0 ? below : lo > 31 ? 0u : below & (~0u << lo);
}

// Zeroes the 16-bit entries of 32 columns whose bit is clear, whatever they
// hold: four bits at a time are multiplied onto the sign bits of a word's
// bytes, and byte permutes that repeat those signs make the masks. (A compare
// and a select for every entry took 650 clocks a step longer.)
__device__ __forceinline__ void keep_seen(uint32_t (&w)[16], uint32_t bits) {
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    const uint32_t y = ((bits >> (4 * g)) & 0xfu) * 0x10204080u;
    uint32_t a, b;
    asm("prmt.b32 %0, %1, 0, 0x9988;\n" : "=r"(a) : "r"(y));
    asm("prmt.b32 %0, %1, 0, 0xbbaa;\n" : "=r"(b) : "r"(y));
    w[2 * g] &= a;
    w[2 * g + 1] &= b;
  }
}

// Warps of both kernels: two elementwise warpgroups, each with 32 of a step's
// 64 columns to a thread, an auxiliary warpgroup, the TMA warp, the MMA warps.
// (At D = 64 two pairs of warpgroups for the even and the odd steps took 66 us
// against 68 for dK/dV of 2 x 16 heads of 1500 x 2048, and 48 against 47 for dQ:
// not kept. At D = 128 the dQ kernel's forms spill 8 to 16 bytes a thread.)
constexpr int kAuxWarp = 8, kTmaWarp = 12, kMmaWarp = 13;

// The 16 columns kk of a step's P or dS as an A operand: each warpgroup writes
// its 16-bit columns over the first half of its 32-bit ones.
__device__ __forceinline__ uint32_t step_col(int kk) { return (kk >> 1) * 32 + (kk & 1) * 8; }

template <bool BF16>
__device__ __forceinline__ float lo16(uint32_t v) {
  if constexpr (BF16) return __uint_as_float(v << 16);
  return __half2float(__ushort_as_half(static_cast<unsigned short>(v & 0xffffu)));
}
template <bool BF16>
__device__ __forceinline__ float hi16(uint32_t v) {
  if constexpr (BF16) return __uint_as_float(v & 0xffff0000u);
  return __half2float(__ushort_as_half(static_cast<unsigned short>(v >> 16)));
}

// `words` words of a row; wide: 32-byte stores (whole sectors, half the
// instructions).
__device__ __forceinline__ void store_words(void* dst, const uint32_t* w, int words, bool wide) {
#pragma unroll
  for (int q = 0; q < words / 8; ++q) {
    uint32_t* const d = static_cast<uint32_t*>(dst) + 8 * q;
    const uint32_t* const x = w + 8 * q;
    if (wide) {
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(d), "r"(x[0]),
                   "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                   : "memory");
    } else {
      reinterpret_cast<uint4*>(d)[0] = make_uint4(x[0], x[1], x[2], x[3]);
      reinterpret_cast<uint4*>(d)[1] = make_uint4(x[4], x[5], x[6], x[7]);
    }
  }
}

template <bool BF16>
__device__ __forceinline__ void pack32(uint32_t* w, const uint32_t* r, float f) {
#pragma unroll
  for (int e = 0; e < 16; ++e)
    w[e] = pack2_t<BF16>(__uint_as_float(r[2 * e]) * f, __uint_as_float(r[2 * e + 1]) * f);
}

// 32 fp32 columns times `f`, stored from column `col` of a row of gradients.
template <bool BF16>
__device__ __forceinline__ void store_row32(void* base, int64_t row_off, int col, bool g32,
                                            const uint32_t* r, float f, bool wide) {
  if (g32) {
    uint32_t w[32];
#pragma unroll
    for (int e = 0; e < 32; ++e) w[e] = __float_as_uint(__uint_as_float(r[e]) * f);
    store_words(static_cast<float*>(base) + row_off + col, w, 32, wide);
  } else {
    uint32_t w[16];
    pack32<BF16>(w, r, f);
    store_words(static_cast<uint16_t*>(base) + row_off + col, w, 16, wide);
  }
}

// ---------------------------------------------------------------- fp16: |v|

// The largest |v| of every key tile of a KV head, which the dQ kernel bounds dS
// by: a CTA a tile, 16 rows a warp. One pass over V; left in dV's rows, which
// are not written before the dK, dV kernel, so that the call needs no more
// workspace than it does with bf16. What the powers of two cost, this launch
// and the products by them in the dK, dV kernel, replayed from a graph: 2 x 1000
// tokens of 8 + 2 heads 29 -> 33 us, 8192 of 64 + 8 (window 512) 404 -> 420,
// D = 64, 2 x 16 heads of 1500 x 2048, 114 -> 121. With a fixed 2^6, |dP - delta|
// of 1023 overflowed, which a dO of standard deviation 200 reaches.
template <int D>
__global__ void __launch_bounds__(256) swa_bwd_vmax_kernel(const SwaBwdProblem p, float* vmax) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;  // of a row; rows of a warp at a time
  __shared__ uint32_t sh[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int kt = static_cast<int>(blockIdx.x % static_cast<unsigned>(p.ktiles));
  const int bg = static_cast<int>(blockIdx.x / static_cast<unsigned>(p.ktiles));
  const int b = bg / p.Hkv, g = bg - b * p.Hkv;
  uint4 v[16 / kRows];
#pragma unroll
  for (int r = 0; r < 16 / kRows; ++r) {
    const int j = kt * kBlk + warp * 16 + r * kRows + lane / kLanes;
    v[r] = make_uint4(0, 0, 0, 0);
    if (j < p.N)
      v[r] = reinterpret_cast<const uint4*>(
          p.V + ((static_cast<int64_t>(b) * p.N + j) * p.Hkv + g) * D)[lane % kLanes];
  }
  uint32_t top = 0u;
#pragma unroll
  for (int r = 0; r < 16 / kRows; ++r) {
    const uint32_t vv[4] = {v[r].x, v[r].y, v[r].z, v[r].w};
    float sq = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      sq = fmaf(lo16<false>(vv[e]), lo16<false>(vv[e]), sq);
      sq = fmaf(hi16<false>(vv[e]), hi16<false>(vv[e]), sq);
    }
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) sq += __shfl_xor_sync(kFull, sq, o);
    top = max(top, finite_bits(sq));
  }
  top = __reduce_max_sync(kFull, top);
  if (lane == 0) sh[warp] = top;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 1; w < 8; ++w) top = max(top, sh[w]);
    vmax[b * p.vmax_b + kt * p.vmax_t + g * p.vmax_g] = sqrtf(__uint_as_float(top));
  }
}

// ---------------------------------------------------------------- dQ

template <int D>
struct DqCfg {
  static constexpr int kAtoms = D / 64;
  static constexpr int kTile = kStep * D * 2;      // one K or V tile
  static constexpr int kStages = D == 128 ? 4 : 6;
  static constexpr int kOffQ = kStages * 2 * kTile;      // the next item's O, then its Q; dO
  static constexpr int kOffDo = kOffQ + kBlk * D * 2;
  // 2 x (LSE in base 2 less the shift of dS, delta) of the rows; fp16: and the
  // factor of dQ
  static constexpr int kOffStat = kOffDo + kBlk * D * 2, kOffOut = kOffStat + 4 * kBlk * 4;
  static constexpr int kOffBar = kOffOut + 2 * kBlk * 4;
  static constexpr int kFull = 0, kEmpty = kStages, kOStaged = 2 * kStages, kQStaged = kOStaged + 1,
                       kQReady = kQStaged + 1, kDoReady = kQReady + 1, kSDone = kDoReady + 2,
                       kDpDone = kSDone + 1, kSFull = kDpDone + 1, kDsFull = kSFull + 2,
                       kDqDone = kDsFull + 2, kDqFree = kDqDone + 1, kNumBars = kDqFree + 1;
  static constexpr int kOffTmem = kOffBar + kNumBars * 8;
  static constexpr int kSmem = kOffTmem + 16 + 1024;
  static_assert(kSmem <= 232448 && kSmem > 118784, "one CTA per SM");
  // tensor-memory columns
  static constexpr uint32_t kColQ = 0, kColDo = D / 2, kColDq = D, kColS = 2 * D,
                            kColP = 2 * D + 2 * kStep;
  static_assert(2 * D + 4 * kStep <= 512, "tensor memory");
};

// One item of the dQ kernel: 128 queries of a head, and the key tiles of 64
// that their windows touch, or a part of those.
struct DqItem {
  int b, g, h, q0, q_last, t0, nt;
  int part;   // its place among the parts, or -1
  bool stat;  // leaves the rows' LSE and delta
};

// Items in the order (b, KV head, query tile, head): heads fastest, so that
// the CTAs of a moment share K and V in L2; later tiles, which see more keys
// under a causal window, first. CUT: the last ones are cut into parts. (In a
// kernel of its own: one for both took 427 us instead of 398 for the whole call
// at 8k, window (512, 0), where nothing is cut.)
template <bool CUT>
__device__ __forceinline__ DqItem dq_item(const SwaBwdProblem& p, uint32_t x) {
  DqItem it;
  uint32_t sp = 0;
  it.part = -1;
  if (CUT && x >= static_cast<uint32_t>(p.dq_whole)) {
    it.part = static_cast<int>(x) - p.dq_whole;
    x = p.dq_whole + static_cast<uint32_t>(it.part) / static_cast<uint32_t>(p.dq_splits);
    sp = static_cast<uint32_t>(it.part) % static_cast<uint32_t>(p.dq_splits);
  }
  const int hh = static_cast<int>(x % static_cast<uint32_t>(p.hpg));
  x /= static_cast<uint32_t>(p.hpg);
  const int qt = p.qtiles - 1 - static_cast<int>(x % static_cast<uint32_t>(p.qtiles));
  x /= static_cast<uint32_t>(p.qtiles);
  it.g = static_cast<int>(x % static_cast<uint32_t>(p.Hkv));
  it.b = static_cast<int>(x / static_cast<uint32_t>(p.Hkv));
  it.h = it.g * p.hpg + hh;
  it.q0 = qt * kBlk;
  it.q_last = min(it.q0 + kBlk, p.M) - 1;
  const int jlo = max(0, it.q0 - p.left), jhi = min(p.N - 1, it.q_last + p.right);
  it.t0 = jlo / kStep;
  const int all = jhi >= jlo ? jhi / kStep - it.t0 + 1 : 0;
  it.nt = all;
  it.stat = true;
  if (CUT && it.part >= 0) {
    const int first = static_cast<int>(static_cast<int64_t>(all) * sp / p.dq_splits);
    it.nt = static_cast<int>(static_cast<int64_t>(all) * (sp + 1) / p.dq_splits) - first;
    it.t0 += first;
    it.stat = first == 0 && (it.nt > 0 || (all == 0 && sp == 0));
  }
  return it;
}

template <int D, bool BF16, bool CUT>
__global__ void __launch_bounds__(32 * (kMmaWarp + 1), 1)
    swa_bwd_dq_kernel(const SwaBwdProblem p, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV,
                      const __grid_constant__ CUtensorMap tmQ,
                      const __grid_constant__ CUtensorMap tmO,
                      const __grid_constant__ CUtensorMap tmDo) {
  using C = DqCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const gbase = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](int i) { return base + C::kOffBar + 8u * static_cast<uint32_t>(i); };
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(bar(C::kFull + s), 1);
      mbar_init(bar(C::kEmpty + s), 1);
    }
    mbar_init(bar(C::kOStaged), 1);
    mbar_init(bar(C::kQStaged), 1);
    mbar_init(bar(C::kQReady), 4);
    // two, for even and odd items: an elementwise warp may ask for an item's
    // when the next item's dO is there already
    mbar_init(bar(C::kDoReady), 4);
    mbar_init(bar(C::kDoReady + 1), 4);
    mbar_init(bar(C::kSDone), 1);
    mbar_init(bar(C::kDpDone), 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(C::kSFull + s), 1);
      mbar_init(bar(C::kDsFull + s), 8);
    }
    mbar_init(bar(C::kDqDone), 1);
    mbar_init(bar(C::kDqFree), 4);
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tc_alloc(base + C::kOffTmem, kTmemAll);
    tc_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(gbase + C::kOffTmem);
  float* const stat = reinterpret_cast<float*>(gbase + C::kOffStat);
  bool failed = false;
  auto wait_all = [&](int i, uint32_t parity) {
    const bool r = __all_sync(kFull, wait_phase(bar(i), parity, kWaitLimitNs));
    tc_fence_after();
    return r;
  };
  // Items are dealt in rounds of gridDim.x, in snake order, as in the forward.
  // Below, n counts the items with keys, g0 their steps.
  const uint32_t items = static_cast<uint32_t>(p.dq_items);
  const uint32_t rounds = (items + gridDim.x - 1) / gridDim.x;
  auto item_of = [&](uint32_t k) {
    return k * gridDim.x + ((k & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
  };

  if (warp == kTmaWarp) {
    if (lane == 0) {
      // ---- TMA producer: K and V tiles of 64 keys ----
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
      const uint64_t keep = l2_policy_evict_last();
      int s = 0;
      uint32_t ph = 1;  // of the wait for an empty stage: the first round passes
      int in_flight = 0;
      for (uint32_t k = 0; k < rounds && !failed; ++k) {
        const uint32_t x = item_of(k);
        if (x >= items) continue;
        const DqItem it = dq_item<CUT>(p, x);
        for (int i = 0; i < it.nt; ++i) {
          if (!wait_phase(bar(C::kEmpty + s), ph, kWaitLimitNs)) {
            failed = true;
            break;
          }
          mbar_arrive_expect_tx(bar(C::kFull + s), 2 * C::kTile);
          const uint32_t dst = base + s * 2 * C::kTile;
          const int j0 = (it.t0 + i) * kStep;
          for (int a = 0; a < C::kAtoms; ++a) {
            tma_load_4d(dst + a * kAtomStep, &tmK, bar(C::kFull + s), a * 64, it.g, j0, it.b, keep);
            tma_load_4d(dst + C::kTile + a * kAtomStep, &tmV, bar(C::kFull + s), a * 64, it.g, j0,
                        it.b, keep);
          }
          if (in_flight < C::kStages) ++in_flight;
          if (++s == C::kStages) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      if (failed) {  // leave nothing in flight: the last loads of the stages before s
        for (int k = 0; k < in_flight; ++k) {
          s = s == 0 ? C::kStages - 1 : s - 1;
          if (s == C::kStages - 1) ph ^= 1;
          wait_phase(bar(C::kFull + s), ph ^ 1, kWaitLimitNs);
        }
      }
    }
  } else if (warp == kMmaWarp) {
    // ---- MMA issuer (the whole warp, one lane elected): S_g, dP_g, dQ_{g-1},
    // the steps of all items as one stream ----
    constexpr uint32_t id_s = umma_idesc_f16(kBlk, kStep, BF16, false);
    constexpr uint32_t id_q = umma_idesc_f16(kBlk, D, BF16, true);
    const uint32_t on = elect_one();
    int s = 0, s_prev = 0;
    uint32_t ph = 0, g = 0, n = 0;
    const uint64_t k_major = umma_desc_sw128(base, 16);
    const uint64_t mn_major = umma_desc_sw128(base, kAtomStep);
    bool start = false, last = false;  // dQ_{g-1} is its item's first, last
    uint32_t n_prev = 0;               // and its item
    auto issue_dq = [&](uint32_t gq) -> bool {
      // (an item's first dQ overwrites the item's before)
      if (start && n_prev > 0 && !wait_all(C::kDqFree, (n_prev - 1) & 1)) return false;
      if (!wait_all(C::kDsFull + (gq & 1), (gq >> 1) & 1)) return false;
      const uint32_t ds = tmem + C::kColS + (gq & 1) * kStep;
      const uint64_t kd = desc_at(mn_major, s_prev * 2 * C::kTile);
#pragma unroll
      for (int kk = 0; kk < kStep / 16; ++kk)
        tc_mma_ts_if(on, tmem + C::kColDq, ds + step_col(kk),
                     desc_at(kd, kk * 2048), id_q, (!start || kk > 0) ? 1u : 0u);
      tc_commit_if(on, bar(C::kEmpty + s_prev));
      if (last) tc_commit_if(on, bar(C::kDqDone));
      return true;
    };
    bool ok = true;
    for (uint32_t k = 0; k < rounds && ok; ++k) {
      const uint32_t x = item_of(k);
      if (x >= items) continue;
      const int nt = dq_item<CUT>(p, x).nt;
      for (int i = 0; i < nt && ok; ++i, ++g) {
        if (i == 0) ok = wait_all(C::kQReady, n & 1);
        ok = ok && wait_all(C::kFull + s, ph);
        if (!ok) break;
        const uint64_t kd = desc_at(k_major, s * 2 * C::kTile), vd = desc_at(kd, C::kTile);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          tc_mma_ts_if(on, tmem + C::kColS + (g & 1) * kStep, tmem + C::kColQ + 8 * kk,
                       desc_at(kd, (kk >> 2) * kAtomStep + (kk & 3) * 32), id_s, kk > 0 ? 1u : 0u);
        if (i == nt - 1) tc_commit_if(on, bar(C::kSDone));  // Q has been read
        if (i == 0) ok = wait_all(C::kDoReady + (n & 1), (n >> 1) & 1);
        if (!ok) break;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          tc_mma_ts_if(on, tmem + C::kColP + (g & 1) * kStep, tmem + C::kColDo + 8 * kk,
                       desc_at(vd, (kk >> 2) * kAtomStep + (kk & 3) * 32), id_s, kk > 0 ? 1u : 0u);
        tc_commit_if(on, bar(C::kSFull + (g & 1)));
        if (i == nt - 1) tc_commit_if(on, bar(C::kDpDone));
        if (g > 0) ok = issue_dq(g - 1);
        start = i == 0;
        last = i == nt - 1;
        n_prev = n;
        s_prev = s;
        if (++s == C::kStages) {
          s = 0;
          ph ^= 1;
        }
      }
      if (nt > 0) ++n;
    }
    if (ok && g > 0) ok = issue_dq(g - 1);
    if (!ok) {  // leave nothing in flight: one more phase of a barrier
      failed = true;
      tc_commit_if(on, bar(C::kSDone));
      wait_all(C::kSDone, 0);
      wait_all(C::kSDone, 1);
    }
  } else if (warp >= kAuxWarp) {
    // ---- auxiliary warpgroup, thread <-> query row: delta and LSE of the
    // next item, its Q and dO into tensor memory, and dQ of the last one out.
    // O and dO are staged while an item runs, delta is formed, Q follows in
    // O's place; Q moves once the item's last S, dO once its last dP is done. ----
    const int quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint8_t* const q_row = gbase + C::kOffQ + row * 128;
    const uint8_t* const do_row = gbase + C::kOffDo + row * 128;
    const bool leader = warp == kAuxWarp && lane == 0;
    const uint64_t once = l2_policy_evict_first();
    // 16-byte chunk c of a row of a staged tile
    auto chunk = [&](const uint8_t* r, int c) {
      return *reinterpret_cast<const uint4*>(r + (c >> 3) * kAtomBlk + (((c & 7) ^ (row & 7)) << 4));
    };
    auto load = [&](const CUtensorMap* tm, int off, int b, const DqItem& it) {
      for (int a = 0; a < C::kAtoms; ++a)
        for (int r = 0; r < 2; ++r)  // rows past M arrive as zeros
          tma_load_4d(base + off + a * kAtomBlk + r * kAtomStep, tm, bar(b), a * 64, it.h,
                      it.q0 + r * kStep, it.b, once);
    };
    auto load_o = [&](const DqItem& it) {  // one thread
      mbar_arrive_expect_tx(bar(C::kOStaged), 2 * kBlk * D * 2);
      load(&tmO, C::kOffQ, C::kOStaged, it);
      load(&tmDo, C::kOffDo, C::kOStaged, it);
    };
    float* const factor = reinterpret_cast<float*>(gbase + C::kOffOut) + row;
    uint32_t n = 0;
    auto out = [&](const DqItem& it, bool zero) {  // dQ rows of an item, the last one if not zero
      const int iq = it.q0 + row;
      const bool part = CUT && it.part >= 0, f32 = p.g32 || part;
      void* const dst = part ? p.part_q : p.dQ;
      const int64_t off = part ? (static_cast<int64_t>(it.part) * kBlk + row) * D
                               : ((static_cast<int64_t>(it.b) * p.M + iq) * p.H + it.h) * D;
      auto column = [&](int c, uint32_t (&r)[32]) {
        if (zero) {
#pragma unroll
          for (int e = 0; e < 32; ++e) r[e] = 0u;
          return;
        }
        tc_ld32(lane_addr + C::kColDq + 32 * c, r);
        tc_wait_ld();
        if (c == D / 32 - 1) {  // the next item may start its dQ
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::kDqFree));
        }
      };
      const float f_out = BF16 || zero ? p.scale : factor[((n - 1) & 1) * kBlk];
      uint32_t r[32];
      if (f32) {
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          column(c, r);
          if (iq < p.M) store_row32<BF16>(dst, off, 32 * c, true, r, f_out, p.wide);
        }
      } else {  // everything out of tensor memory first
        uint32_t w[D / 2];
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          column(c, r);
          pack32<BF16>(w + 16 * c, r, f_out);
        }
        if (iq < p.M) store_words(static_cast<uint16_t*>(dst) + off, w, D / 2, p.wide);
      }
    };
    DqItem last{};
    bool ok = true;  // no wait of this warp has given up
    auto wait_last = [&](int b) {  // for something of the last item
      const bool r =
          __all_sync(kFull, wait_phase(bar(b), (n - 1) & 1, item_limit_ns(last.nt)));
      tc_fence_after();
      return r;
    };
    auto next = [&](uint32_t from) {  // the next round with an item that has keys
      for (; from < rounds; ++from)
        if (item_of(from) < items && dq_item<CUT>(p, item_of(from)).nt > 0) break;
      return from;
    };
    uint32_t kn = next(0);
    if (kn < rounds && leader) load_o(dq_item<CUT>(p, item_of(kn)));
    for (uint32_t k = 0; k < rounds && !failed; ++k) {
      const uint32_t x = item_of(k);
      if (x >= items) continue;
      const DqItem it = dq_item<CUT>(p, x);
      const int iq = it.q0 + row;
      float l2 = INFINITY, dl = 0.f;
      uint32_t top = 0u;  // fp16: the largest |dO| of the warp's rows
      if (it.nt > 0) {
        // fp16: the largest |v| of the item's key tiles, read before what follows
        // and used after it
        const float* const vsrc = p.vmax + it.b * p.vmax_b + it.g * p.vmax_g;
        const int vlast = (it.t0 + it.nt - 1) / 2;
        int vt = it.t0 / 2 + lane;
        float vm = 0.f;
        if (!BF16 && vt <= vlast) vm = vsrc[vt * p.vmax_t];
        const float l = iq < p.M ? p.LSE[(static_cast<int64_t>(it.b) * p.H + it.h) * p.M + iq]
                                 : -INFINITY;
        ok = ok && wait_all(C::kOStaged, n & 1);
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const uint4 v = chunk(do_row, c), o = chunk(q_row, c);
          const uint32_t vv[4] = {v.x, v.y, v.z, v.w}, oo[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            acc[e] = fmaf(lo16<BF16>(vv[e]), lo16<BF16>(oo[e]), acc[e]);
            acc[e] = fmaf(hi16<BF16>(vv[e]), hi16<BF16>(oo[e]), acc[e]);
          }
        }
        if (!bar_vote(1, 128, ok)) {  // every row of O has been read
          failed = true;
          break;
        }
        if (leader) {
          mbar_arrive_expect_tx(bar(C::kQStaged), kBlk * D * 2);
          load(&tmQ, C::kOffQ, C::kQStaged, it);
        }
        if (l != -INFINITY) {  // else: a row without keys
          l2 = l * 1.4426950408889634f;
          dl = (acc[0] + acc[1]) + (acc[2] + acc[3]);
        }
        float e = 0.f;
        if constexpr (!BF16) {  // (while Q arrives)
          float sq[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
          for (int c = 0; c < D / 8; ++c) {
            const uint4 v = chunk(do_row, c);
            const uint32_t vv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              sq[i] = fmaf(lo16<BF16>(vv[i]), lo16<BF16>(vv[i]), sq[i]);
              sq[i] = fmaf(hi16<BF16>(vv[i]), hi16<BF16>(vv[i]), sq[i]);
            }
          }
          while ((vt += 32) <= vlast) vm = fmaxf(vm, vsrc[vt * p.vmax_t]);
          vm = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(vm)));
          const float norm = sqrtf((sq[0] + sq[1]) + (sq[2] + sq[3]));
          const int shift = shift_for(fmaf(norm, vm, fabsf(dl)));
          e = static_cast<float>(shift);
          factor[(n & 1) * kBlk] = p.scale * pow2(-shift);
          top = __reduce_max_sync(kFull, l2 != INFINITY ? finite_bits(norm) : 0u);
        }
        stat[(n & 1) * 2 * kBlk + row] = l2 - e;
        stat[(n & 1) * 2 * kBlk + kBlk + row] = dl;
      }
      if ((!CUT || it.stat) && iq < p.Mp) {  // (a tile without keys: no pair reads them)
        const int64_t at = (static_cast<int64_t>(it.b) * p.H + it.h) * p.Mp + iq;
        p.nlse2[at] = Shift<BF16>::kP - l2;
        p.ndelta[at] =
            BF16 ? -dl : __uint_as_float((__float_as_uint(-dl) & ~1u) | ((top >> top_bit(lane)) & 1u));
      }
      if (it.nt == 0) {
        out(it, true);
        continue;
      }
      // a staged row into tensor memory; the barrier tells the MMA warp
      auto move = [&](const uint8_t* src, uint32_t col, int done, int ready) -> bool {
        uint32_t r[D / 2];
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const uint4 v = chunk(src, c);
          r[4 * c] = v.x, r[4 * c + 1] = v.y, r[4 * c + 2] = v.z, r[4 * c + 3] = v.w;
        }
        if (n > 0 && !wait_last(done)) return false;
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
          tc_st32(lane_addr + col + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&r[32 * c]));
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(ready));
        return true;
      };
      ok = wait_all(C::kQStaged, n & 1) && move(q_row, C::kColQ, C::kSDone, C::kQReady) &&
           move(do_row, C::kColDo, C::kDpDone, C::kDoReady + static_cast<int>(n & 1));
      if (!bar_vote(1, 128, ok)) {  // all four warps have read the staged rows
        failed = true;
        break;
      }
      kn = next(k + 1);
      if (kn < rounds && leader) load_o(dq_item<CUT>(p, item_of(kn)));
      if (n > 0) {
        ok = wait_last(C::kDqDone);
        if (ok) out(last, false);
      }
      last = it;
      ++n;
    }
    if (!failed && n > 0) {
      ok = ok && wait_last(C::kDqDone);
      if (ok) out(last, false);
    }
    failed = !ok || failed;
    if (failed && leader) {  // a load may still be in flight
      wait_phase(bar(C::kOStaged), 0, kWaitLimitNs);
      wait_phase(bar(C::kOStaged), 1, kWaitLimitNs);
      wait_phase(bar(C::kQStaged), 0, kWaitLimitNs);
      wait_phase(bar(C::kQStaged), 1, kWaitLimitNs);
    }
  } else {
    // ---- elementwise: thread <-> (query row, half of a step's columns) ----
    const int wg = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint64_t sl2_2 = pair(p.sl2, p.sl2);
    uint32_t g0 = 0, n = 0;
    for (uint32_t k = 0; k < rounds && !failed; ++k) {
      const uint32_t x = item_of(k);
      if (x >= items) continue;
      const DqItem it = dq_item<CUT>(p, x);
      if (it.nt == 0) continue;
      if (!wait_all(C::kDoReady + (n & 1), (n >> 1) & 1)) {
        failed = true;
        break;
      }
      const float neg = -stat[(n & 1) * 2 * kBlk + row];
      const float dl = stat[(n & 1) * 2 * kBlk + kBlk + row];
      const uint64_t neg_2 = pair(neg, neg), ndl_2 = pair(-dl, -dl);
      const int iq = it.q0 + row;
      const int lo_i = max(0, iq - p.left), hi_i = min(p.N - 1, iq + p.right);
      const int in_lo = max(0, it.q_last - p.left), in_hi = min(p.N - 1, it.q0 + p.right);
      for (int i = 0; i < it.nt; ++i) {
        const uint32_t g = g0 + i;
        if (!wait_all(C::kSFull + (g & 1), (g >> 1) & 1)) {
          failed = true;
          break;
        }
        const uint32_t sa = lane_addr + C::kColS + (g & 1) * kStep + 32 * wg;
        const uint32_t da = lane_addr + C::kColP + (g & 1) * kStep + 32 * wg;
        const int jc = (it.t0 + i) * kStep + 32 * wg;
        const bool edge = jc - 32 * wg < in_lo || jc - 32 * wg + kStep - 1 > in_hi;  // CTA-wide
        const uint32_t seen = edge ? seen_bits(lo_i - jc, hi_i - jc) : 0u;
        uint32_t s[32], d[32], w[16];
        tc_ld32(sa, s);
        tc_ld32(da, d);
        tc_wait_ld();
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float2 f = unpair(mul2(ex2_2(fma2(pair(s[2 * c], s[2 * c + 1]), sl2_2, neg_2)),
                                       add2(pair(d[2 * c], d[2 * c + 1]), ndl_2)));
          w[c] = pack2_t<BF16>(f.x, f.y);
        }
        if (edge) keep_seen(w, seen);
        tc_st16(sa, w);
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::kDsFull + (g & 1)));
      }
      g0 += it.nt;
      ++n;
    }
  }

  if (failed) report_timeout();
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tc_dealloc(tmem, kTmemAll);
  }
}

// ---------------------------------------------------------------- dK, dV

template <int D>
struct DkvCfg {
  static constexpr int kAtoms = D / 64;
  static constexpr int kTile = kStep * D * 2;      // one Q or dO tile
  static constexpr int kStage = 2 * kTile + 2 * kStep * 4;  // and the nlse2, ndelta of its queries
  static constexpr int kStagePitch = (kStage + 1023) / 1024 * 1024;
  static constexpr int kStages = D == 128 ? 4 : 6;
  static constexpr int kBuf = D == 128 ? 1 : 2;  // buffers of S and of dP
  // Groups of a step: at D = 128, with one buffer, each warpgroup's 32 queries
  // are a group of their own, so that one's products run during the other's
  // exponentials (16k, window (4096, 0), before one warp's issue was split in
  // two: 2.41 ms against 2.65). At D = 64 the
  // products are half as long, there are two buffers, and the waits of twice
  // the groups cost more than they hide.
  static constexpr int kGroups = D == 128 ? 2 : 1;
  static constexpr int kCols = kStep / kGroups;
  static constexpr int kOffK = kStages * kStagePitch;  // the next item's K and V
  static constexpr int kOffV = kOffK + kBlk * D * 2;
  // fp16: 2 x 2^(e - 12) of the rows (P carries 2^12 already), the warps' largest
  // |dO| and |delta|
  static constexpr int kOffShift = kOffV + kBlk * D * 2, kOffTop = kOffShift + 2 * kBlk * 4;
  static constexpr int kOffBar = kOffTop + 2 * 4 * 4;
  static constexpr int kFull = 0, kEmpty = kStages, kStaged = 2 * kStages, kKReady = kStaged + 1,
                       kVReady = kKReady + 1, kSDone = kVReady + 1, kDpDone = kSDone + 1,
                       kDvDone = kDpDone + 1, kDkDone = kDvDone + 1, kDvFree = kDkDone + 1,
                       kDkFree = kDvFree + 1, kSFull = kDkFree + 1, kPFull = kSFull + 4,
                       kDpFull = kPFull + 4, kDsFull = kDpFull + 4, kShift = kDsFull + 4,
                       kNumBars = kShift + 2;
  static constexpr int kOffTmem = kOffBar + kNumBars * 8;
  static constexpr int kSmem = kOffTmem + 16 + 1024;
  static_assert(kSmem <= 232448 && kSmem > 118784, "one CTA per SM");
  static constexpr uint32_t kColK = 0, kColV = D / 2, kColDv = D, kColDk = 2 * D, kColS = 3 * D,
                            kColP = 3 * D + kBuf * kStep;
  static_assert(3 * D + 2 * kBuf * kStep <= 512, "tensor memory");
};

// One item of the dK, dV kernel: 128 keys of a KV head, and the steps of its
// query heads and query blocks of 64 that see them (numbered head after
// head), or a part of those steps.
struct DkvItem {
  int b, g, j0, u0, nq;   // u0, nq: first block of queries and their number, for each head
  int h, u, nt;           // first head and block of the item, and its steps
  int part;               // its place among the parts, or -1
};

// Tiles in order of falling work (as far as the window's sides tell), the
// (batch, KV head) pairs fastest: neighbouring tiles, which read the same
// queries, run at the same time. The last tiles are cut into parts.
__device__ __forceinline__ DkvItem dkv_item(const SwaBwdProblem& p, uint32_t x) {
  DkvItem it;
  uint32_t tile = x, sp = 0;
  it.part = -1;
  if (x >= static_cast<uint32_t>(p.whole_tiles)) {
    it.part = static_cast<int>(x) - p.whole_tiles;
    tile = p.whole_tiles + static_cast<uint32_t>(it.part) / static_cast<uint32_t>(p.splits);
    sp = static_cast<uint32_t>(it.part) % static_cast<uint32_t>(p.splits);
  }
  const uint32_t pairs = static_cast<uint32_t>(p.B * p.Hkv);
  const uint32_t bg = tile % pairs;
  int kt = static_cast<int>(tile / pairs);
  if (p.right > p.left) kt = p.ktiles - 1 - kt;
  it.g = static_cast<int>(bg % static_cast<uint32_t>(p.Hkv));
  it.b = static_cast<int>(bg / static_cast<uint32_t>(p.Hkv));
  it.j0 = kt * kBlk;
  const int j_last = min(it.j0 + kBlk, p.N) - 1;
  const int ilo = max(0, it.j0 - p.right), ihi = min(p.M - 1, j_last + p.left);
  it.u0 = ilo / kStep;
  it.nq = ihi >= ilo ? ihi / kStep - it.u0 + 1 : 0;
  const int all = it.nq * p.hpg;  // at most 2^31 (checked on the host)
  int first = 0;
  it.nt = all;
  if (it.part >= 0) {
    first = static_cast<int>(static_cast<int64_t>(all) * sp / p.splits);
    it.nt = static_cast<int>(static_cast<int64_t>(all) * (sp + 1) / p.splits) - first;
  }
  it.h = it.g * p.hpg + (it.nq > 0 ? first / it.nq : 0);
  it.u = it.nq > 0 ? first % it.nq : 0;
  return it;
}

template <int D, bool BF16>
__global__ void __launch_bounds__(32 * (kMmaWarp + 2), 1)
    swa_bwd_dkv_kernel(const SwaBwdProblem p, const __grid_constant__ CUtensorMap tmQ,
                       const __grid_constant__ CUtensorMap tmDo,
                       const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV) {
  using C = DkvCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const gbase = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](int i) { return base + C::kOffBar + 8u * static_cast<uint32_t>(i); };
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(bar(C::kFull + s), 1);
      mbar_init(bar(C::kEmpty + s), 2);
    }
    mbar_init(bar(C::kStaged), 1);
    mbar_init(bar(C::kKReady), 4);
    mbar_init(bar(C::kVReady), 4);
    mbar_init(bar(C::kSDone), 1);
    mbar_init(bar(C::kDpDone), 1);
    mbar_init(bar(C::kDvDone), 1);
    mbar_init(bar(C::kDkDone), 1);
    mbar_init(bar(C::kDvFree), 4);
    mbar_init(bar(C::kDkFree), 4);
    for (int s = 0; s < 4; ++s) {
      mbar_init(bar(C::kSFull + s), 1);
      mbar_init(bar(C::kPFull + s), 8 / C::kGroups);
      mbar_init(bar(C::kDpFull + s), 1);
      mbar_init(bar(C::kDsFull + s), 8 / C::kGroups);
    }
    // two, for even and odd items, as in the dQ kernel
    mbar_init(bar(C::kShift), 4);
    mbar_init(bar(C::kShift + 1), 4);
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tc_alloc(base + C::kOffTmem, kTmemAll);
    tc_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(gbase + C::kOffTmem);
  bool failed = false;
  auto wait_all = [&](int i, uint32_t parity) {
    const bool r = __all_sync(kFull, wait_phase(bar(i), parity, kWaitLimitNs));
    tc_fence_after();
    return r;
  };
  const uint32_t items = static_cast<uint32_t>(p.dkv_items);
  const uint32_t rounds = (items + gridDim.x - 1) / gridDim.x;
  auto item_of = [&](uint32_t k) {  // dealt in snake order, as in the dQ kernel
    return k * gridDim.x + ((k & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
  };
  auto next = [&](uint32_t from) {  // the next round with an item that has steps
    for (; from < rounds; ++from)
      if (item_of(from) < items && dkv_item(p, item_of(from)).nt > 0) break;
    return from;
  };

  if (warp == kTmaWarp) {
    if (lane == 0) {
      // ---- TMA producer: Q and dO of 64 queries, their nlse2 and ndelta ----
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmDo);
      const uint64_t keep = l2_policy_evict_last();
      int s = 0, in_flight = 0;
      uint32_t ph = 1;  // of the wait for an empty stage: the first round passes
      for (uint32_t k = next(0); k < rounds && !failed; k = next(k + 1)) {
        const DkvItem it = dkv_item(p, item_of(k));
        int h = it.h, u = it.u;
        for (int n = 0; n < it.nt; ++n) {
          if (!wait_phase(bar(C::kEmpty + s), ph, kWaitLimitNs)) {
            failed = true;
            break;
          }
          const uint32_t full = bar(C::kFull + s), dst = base + s * C::kStagePitch;
          const int i0 = (it.u0 + u) * kStep;
          mbar_arrive_expect_tx(full, C::kStage);
          for (int a = 0; a < C::kAtoms; ++a) {
            tma_load_4d(dst + a * kAtomStep, &tmQ, full, a * 64, h, i0, it.b, keep);
            tma_load_4d(dst + C::kTile + a * kAtomStep, &tmDo, full, a * 64, h, i0, it.b, keep);
          }
          const int64_t at = (static_cast<int64_t>(it.b) * p.H + h) * p.Mp + i0;
          bulk_load(dst + 2 * C::kTile, p.nlse2 + at, kStep * 4, full);
          bulk_load(dst + 2 * C::kTile + kStep * 4, p.ndelta + at, kStep * 4, full);
          if (++u == it.nq) {
            u = 0;
            ++h;
          }
          if (in_flight < C::kStages) ++in_flight;
          if (++s == C::kStages) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      if (failed) {  // leave nothing in flight: the last loads of the stages before s
        for (int k = 0; k < in_flight; ++k) {
          s = s == 0 ? C::kStages - 1 : s - 1;
          if (s == C::kStages - 1) ph ^= 1;
          wait_phase(bar(C::kFull + s), ph ^ 1, kWaitLimitNs);
        }
      }
    }
  } else if (warp >= kMmaWarp) {
    // ---- MMA issuers (a whole warp each, one lane elected). The first forms S
    // and dV, the second dP and dK: P overwrites its S and dS its dP, so the
    // two share no tensor memory, each accumulator is added to in one
    // order, and one warp's waits pass while the other's products run.
    // With two groups, group w of a step (queries 32 w .. 32 w + 31) belongs to
    // warpgroup w.
    // The steps of all items are one stream: S (dP) is formed kBuf steps ahead. ----
    constexpr uint32_t id_s = umma_idesc_f16(kBlk, C::kCols, BF16, false);
    constexpr uint32_t id_d = umma_idesc_f16(kBlk, D, BF16, true);
    const uint32_t on = elect_one();
    const bool is_v = warp == kMmaWarp;
    const uint32_t a_col = tmem + (is_v ? C::kColK : C::kColV);
    const uint32_t s_col = tmem + (is_v ? C::kColS : C::kColP);
    const uint32_t d_col = tmem + (is_v ? C::kColDv : C::kColDk);
    // in a stage: the tile that forms S (dP), and the one dV (dK) sums over
    const uint64_t k_major = umma_desc_sw128(base + (is_v ? 0 : C::kTile), 16);
    const uint64_t mn_major = umma_desc_sw128(base + (is_v ? C::kTile : 0), kAtomStep);
    const int s_bar = is_v ? C::kSFull : C::kDpFull, p_bar = is_v ? C::kPFull : C::kDsFull;
    const int a_ready = is_v ? C::kKReady : C::kVReady, a_done = is_v ? C::kSDone : C::kDpDone;
    const int d_done = is_v ? C::kDvDone : C::kDkDone, d_free = is_v ? C::kDvFree : C::kDkFree;
    auto slot = [&](uint32_t n, int w) {
      return s_col + (C::kBuf == 2 ? (n & 1) * kStep : 0) + w * C::kCols;
    };
    auto rows_of = [&](int stage, int w) { return stage * C::kStagePitch + w * (C::kCols * 128); };
    auto form = [&](uint32_t n, int w, int stage) {
      const uint64_t b0 = desc_at(k_major, rows_of(stage, w));
      const uint32_t d = slot(n, w);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        tc_mma_ts_if(on, d, a_col + 8 * kk, desc_at(b0, (kk >> 2) * kAtomStep + (kk & 3) * 32), id_s,
                     kk > 0 ? 1u : 0u);
      tc_commit_if(on, bar(s_bar + 2 * w + (n & 1)));
    };
    auto add = [&](uint32_t n, int w, int stage, bool start) {
      const uint64_t b0 = desc_at(mn_major, rows_of(stage, w));
      const uint32_t a = slot(n, w);
#pragma unroll
      for (int kk = 0; kk < C::kCols / 16; ++kk)
        tc_mma_ts_if(on, d_col, a + step_col(kk), desc_at(b0, kk * 2048), id_d,
                     (!start || kk > 0) ? 1u : 0u);
    };
    // n, st: the step that is added and its stage; sl, ph: stage and phase of
    // the step that is formed; na: the item's number
    uint32_t n = 0, na = 0, ph = 0;
    int st = 0, sl = 0;
    auto next_stage = [&]() {
      if (++sl == C::kStages) {
        sl = 0;
        ph ^= 1;
      }
    };
    // P (dS) of the first half of step n and, if `more`, the tiles of the step
    // that is formed: one question for both, as a wait that is over still
    // takes some 100 clocks
    auto wait_first = [&](bool more) -> bool {
      const int pb = p_bar + (n & 1), fb = more ? C::kFull + sl : pb;
      const uint32_t pp = (n >> 1) & 1, fp = more ? ph : pp;
      const bool x1 = mbar_try_wait(bar(pb), pp), x2 = mbar_try_wait(bar(fb), fp);
      if (__all_sync(kFull, x1 && x2)) {
        tc_fence_after();
        return true;
      }
      return wait_all(pb, pp) && wait_all(fb, fp);
    };
    auto added = [&]() {
      tc_commit_if(on, bar(C::kEmpty + st));
      if (++st == C::kStages) st = 0;
      ++n;
    };
    bool ok = true;
    uint32_t k = next(0);
    int nt = k < rounds ? dkv_item(p, item_of(k)).nt : 0;
    int ahead = 0;  // steps of the item that are formed already
    for (; nt > 0 && ok; ++na) {
      const uint32_t k2 = next(k + 1);
      const int nt2 = k2 < rounds ? dkv_item(p, item_of(k2)).nt : 0;
      if (ahead == 0) ok = wait_all(a_ready, na & 1);
      for (; ahead < C::kBuf && ahead < nt && ok; ++ahead) {
        ok = wait_all(C::kFull + sl, ph);
        if (!ok) break;
#pragma unroll
        for (int w = 0; w < C::kGroups; ++w) form(n + ahead, w, sl);
        if (ahead + 1 == nt) tc_commit_if(on, bar(a_done));
        next_stage();
      }
      int i = 0;
      for (; i + C::kBuf < nt && ok; ++i) {
        ok = wait_first(true);
        // (an item's first product overwrites the accumulator of the item before)
        if (i == 0 && na > 0) ok = ok && wait_all(d_free, (na - 1) & 1);
        if (!ok) break;
        const uint32_t m = n + C::kBuf;
        add(n, 0, st, i == 0);
        form(m, 0, sl);
        if constexpr (C::kGroups == 2) {
          ok = wait_all(p_bar + 2 + (n & 1), (n >> 1) & 1);
          if (!ok) break;
          add(n, 1, st, false);
          form(m, 1, sl);
        }
        if (i + C::kBuf + 1 == nt) tc_commit_if(on, bar(a_done));
        next_stage();
        added();
      }
      // the item's last steps; each is followed by a first step of the next
      // item, whose K (V) may have to wait for sums to be read out: nothing
      // of this step comes after it
      ahead = 0;
      for (; i < nt && ok; ++i) {
        ok = wait_first(false);
        if (i == 0 && na > 0) ok = ok && wait_all(d_free, (na - 1) & 1);
        if (!ok) break;
        add(n, 0, st, i == 0);
        if constexpr (C::kGroups == 2) {
          ok = wait_all(p_bar + 2 + (n & 1), (n >> 1) & 1);
          if (!ok) break;
          add(n, 1, st, false);
        }
        added();
        if (i + 1 == nt) tc_commit_if(on, bar(d_done));
        if (ahead < C::kBuf && ahead < nt2) {
          if (ahead == 0) ok = wait_all(a_ready, (na + 1) & 1);
          ok = ok && wait_all(C::kFull + sl, ph);
          if (!ok) break;
          const uint32_t m = n + (nt - 1 - i) + ahead;  // (n is the step after this one)
#pragma unroll
          for (int w = 0; w < C::kGroups; ++w) form(m, w, sl);
          if (ahead + 1 == nt2) tc_commit_if(on, bar(a_done));
          next_stage();
          ++ahead;
        }
      }
      k = k2;
      nt = nt2;
    }
    if (!ok) {  // leave nothing in flight: one more phase of a barrier
      failed = true;
      tc_commit_if(on, bar(a_done));
      wait_all(a_done, 0);
      wait_all(a_done, 1);
    }
  } else if (warp >= kAuxWarp) {
    // ---- auxiliary warpgroup, thread <-> key row: K and V of the next item
    // into tensor memory (K once the item's last S, V once its last dP is
    // done), dV and dK of the last one out ----
    const int quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const bool leader = warp == kAuxWarp && lane == 0;
    const uint64_t once = l2_policy_evict_first();
    auto load = [&](const DkvItem& it) {  // one thread
      mbar_arrive_expect_tx(bar(C::kStaged), 2 * kBlk * D * 2);
      for (int a = 0; a < C::kAtoms; ++a)
        for (int r = 0; r < 2; ++r) {  // rows past N arrive as zeros
          tma_load_4d(base + C::kOffK + a * kAtomBlk + r * kAtomStep, &tmK, bar(C::kStaged), a * 64,
                      it.g, it.j0 + r * kStep, it.b, once);
          tma_load_4d(base + C::kOffV + a * kAtomBlk + r * kAtomStep, &tmV, bar(C::kStaged), a * 64,
                      it.g, it.j0 + r * kStep, it.b, once);
        }
    };
    float f_out = p.scale, f_next = p.scale;  // of the last item's dK, of the next one's
    // one accumulator's rows out; is_v: dV
    auto out = [&](const DkvItem& it, bool is_v, bool zero) {
      const int j = it.j0 + row;
      const float f = is_v ? Shift<BF16>::kPInv : f_out;
      void* dst = is_v ? p.dV : p.dK;
      int64_t off = ((static_cast<int64_t>(it.b) * p.N + j) * p.Hkv + it.g) * D;
      bool f32 = p.g32;
      if (it.part >= 0) {
        dst = p.part;
        off = ((static_cast<int64_t>(it.part) * 2 + (is_v ? 1 : 0)) * kBlk + row) * D;
        f32 = true;
      }
      auto column = [&](int c, uint32_t (&r)[32]) {
        if (zero) {
#pragma unroll
          for (int e = 0; e < 32; ++e) r[e] = 0u;
          return;
        }
        tc_ld32(lane_addr + (is_v ? C::kColDv : C::kColDk) + 32 * c, r);
        tc_wait_ld();
        if (c == D / 32 - 1) {  // the next item may start
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(is_v ? C::kDvFree : C::kDkFree));
        }
      };
      uint32_t r[32];
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        column(c, r);
        if (j < p.N) store_row32<BF16>(dst, off, 32 * c, f32, r, f, p.wide);
      }
    };
    uint32_t n = 0;
    DkvItem last{};
    bool ok = true;  // no wait of this warp has given up
    auto wait_last = [&](int b) {  // for something of the last item
      const bool r =
          __all_sync(kFull, wait_phase(bar(b), (n - 1) & 1, item_limit_ns(last.nt)));
      tc_fence_after();
      return r;
    };
    auto out_last = [&]() -> bool {
      if (!wait_last(C::kDvDone)) return false;
      out(last, true, false);
      if (!wait_last(C::kDkDone)) return false;
      out(last, false, false);
      return true;
    };
    uint32_t kn = next(0);
    if (kn < rounds && leader) load(dkv_item(p, item_of(kn)));
    for (uint32_t k = 0; k < rounds && !failed; ++k) {
      const uint32_t x = item_of(k);
      if (x >= items) continue;
      const DkvItem it = dkv_item(p, x);
      if (it.nt == 0) {  // no query sees the keys
        out(it, true, true);
        out(it, false, true);
        continue;
      }
      // a staged row into tensor memory; the barrier tells the MMA warp
      auto move = [&](int off, uint32_t col, int done, int ready) -> bool {
        const uint8_t* const src = gbase + off + row * 128;
        uint32_t r[D / 2];
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const uint4 v = *reinterpret_cast<const uint4*>(src + (c >> 3) * kAtomBlk +
                                                          (((c & 7) ^ (row & 7)) << 4));
          r[4 * c] = v.x, r[4 * c + 1] = v.y, r[4 * c + 2] = v.z, r[4 * c + 3] = v.w;
        }
        if (n > 0 && !wait_last(done)) return false;
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
          tc_st32(lane_addr + col + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&r[32 * c]));
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(ready));
        return true;
      };
      ok = ok && wait_all(C::kStaged, n & 1);
      if constexpr (!BF16) {
        // the largest |dO| and |delta| of the item's steps, a step to 16 lanes, the
        // warps' loads four at a time
        uint32_t* const tops = reinterpret_cast<uint32_t*>(gbase + C::kOffTop);
        const int w = warp - kAuxWarp;
        uint32_t top = 0u, delta = 0u;
        for (int i = w; 2 * i < it.nt; i += 16) {
          uint4 x[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int step = 2 * (i + 4 * j) + (lane >> 4);
            const uint32_t at = static_cast<uint32_t>(it.u + step), nq = it.nq;
            x[j] = make_uint4(0, 0, 0, 0);
            if (step < it.nt)
              x[j] = *reinterpret_cast<const uint4*>(
                  p.ndelta + (static_cast<int64_t>(it.b) * p.H + it.h + at / nq) * p.Mp +
                  static_cast<int64_t>(it.u0 + at % nq) * kStep + 4 * (lane & 15));
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t xx[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
            uint32_t word = 0u;  // of the 8 lanes that hold the same 32 rows
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint32_t bits = __ballot_sync(kFull, (xx[c] & 1u) != 0u);
              word |= ((bits >> (lane & 24)) & 0xffu) << (8 * c);
              delta = max(delta, finite_bits(fabsf(__uint_as_float(xx[c]))));
            }
            top = max(top, word);
          }
        }
        top = __reduce_max_sync(kFull, top);
        delta = __reduce_max_sync(kFull, delta);
        if (lane == 0) {
          tops[w] = top;
          tops[4 + w] = delta;
        }
        if (!bar_vote(1, 128, ok)) {
          failed = true;
          break;
        }
        float sq[4] = {0.f, 0.f, 0.f, 0.f};
        const uint8_t* const v_row = gbase + C::kOffV + row * 128;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const uint4 v = *reinterpret_cast<const uint4*>(v_row + (c >> 3) * kAtomBlk +
                                                          (((c & 7) ^ (row & 7)) << 4));
          const uint32_t vv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            sq[e] = fmaf(lo16<BF16>(vv[e]), lo16<BF16>(vv[e]), sq[e]);
            sq[e] = fmaf(hi16<BF16>(vv[e]), hi16<BF16>(vv[e]), sq[e]);
          }
        }
        const uint32_t t = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
        const uint32_t d = max(max(tops[4], tops[5]), max(tops[6], tops[7]));
        const float norm = sqrtf((sq[0] + sq[1]) + (sq[2] + sq[3]));
        const int e = shift_for(fmaf(norm, __uint_as_float(t), __uint_as_float(d)));
        f_next = p.scale * pow2(-e);
        reinterpret_cast<float*>(gbase + C::kOffShift)[(n & 1) * kBlk + row] = pow2(e - 12);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::kShift + static_cast<int>(n & 1)));
      }
      ok = ok && move(C::kOffK, C::kColK, C::kSDone, C::kKReady) &&
           move(C::kOffV, C::kColV, C::kDpDone, C::kVReady);
      if (!bar_vote(1, 128, ok)) {  // all four warps have read the staged rows
        failed = true;
        break;
      }
      kn = next(k + 1);
      if (kn < rounds && leader) load(dkv_item(p, item_of(kn)));
      ok = n == 0 || out_last();
      last = it;
      f_out = f_next;
      ++n;
    }
    if (!failed && n > 0) ok = ok && out_last();
    failed = !ok || failed;
    if (failed && leader) {  // a load may still be in flight
      wait_phase(bar(C::kStaged), 0, kWaitLimitNs);
      wait_phase(bar(C::kStaged), 1, kWaitLimitNs);
    }
  } else {
    // ---- elementwise: thread <-> (key row, half of a step's queries) ----
    const int wg = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane;
    const int gb = C::kGroups == 2 ? 2 * wg : 0;  // its group's barriers
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint64_t sl2_2 = pair(p.sl2, p.sl2);
    uint32_t n = 0, ph = 0, na = 0;  // steps, phase of their stages, items
    int st = 0;
    for (uint32_t k = next(0); k < rounds && !failed; k = next(k + 1)) {
      const DkvItem it = dkv_item(p, item_of(k));
      const int j = it.j0 + row;
      const int lo_j = j - p.right, hi_j = min(j + p.left, p.M - 1);  // the queries that see key j
      uint64_t shift_2 = 0;
      if constexpr (!BF16) {
        if (!wait_all(C::kShift + static_cast<int>(na & 1), (na >> 1) & 1)) {
          failed = true;
          break;
        }
        const float f = reinterpret_cast<const float*>(gbase + C::kOffShift)[(na & 1) * kBlk + row];
        shift_2 = pair(f, f);
        ++na;
      }
      int u = it.u;
      for (int t = 0; t < it.nt; ++t, ++n) {
        const int i0 = (it.u0 + u) * kStep, ic = i0 + 32 * wg;
        const int stage = st;
        const uint32_t fp = ph, np = (n >> 1) & 1;
        if (++u == it.nq) u = 0;
        if (++st == C::kStages) {
          st = 0;
          ph ^= 1;
        }
        // S and the stage's nlse2 and ndelta (and, with two buffers, dP): one
        // question for all. A wait of its own for the stage took 330 of a step's
        // 1300 clocks, although it was over: barrier operations are slow
        // beside the operand traffic.
        const int sb = C::kSFull + gb + (n & 1), db = C::kDpFull + gb + (n & 1);
        const bool x0 = mbar_try_wait(bar(C::kFull + stage), fp), x1 = mbar_try_wait(bar(sb), np);
        const bool x2 = C::kBuf == 2 && mbar_try_wait(bar(db), np);
        const bool dp_there = C::kBuf == 2 && __all_sync(kFull, x2);
        if (__all_sync(kFull, x0 && x1)) {
          tc_fence_after();
        } else if (!wait_all(C::kFull + stage, fp) || !wait_all(sb, np)) {
          failed = true;
          break;
        }
        const uint32_t sa =
            lane_addr + C::kColS + (C::kBuf == 2 ? (n & 1) * kStep : 0) + 32 * wg;
        const uint32_t da = sa + C::kBuf * kStep;
        const ulonglong2* nl2 = reinterpret_cast<const ulonglong2*>(
            gbase + stage * C::kStagePitch + 2 * C::kTile + 32 * wg * 4);
        const ulonglong2* ndl = nl2 + kStep / 4;
        const bool edge =
            it.j0 < i0 + kStep - 1 - p.left || it.j0 + kBlk - 1 > i0 + p.right || i0 + kStep > p.M;
        const uint32_t seen = edge ? seen_bits(lo_j - ic, hi_j - ic) : 0u;
        auto store = [&](uint32_t at, const uint64_t (&v)[16]) {
          uint32_t w[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const float2 f = unpair(v[c]);
            w[c] = pack2_t<BF16>(f.x, f.y);
          }
          if (edge) keep_seen(w, seen);
          tc_st16(at, w);
        };
        auto arrive = [&](int b) {
          tc_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(b + gb + (n & 1)));
        };
        uint32_t s[32];
        uint64_t pr[16];  // P, then dS
        tc_ld32(sa, s);
        tc_wait_ld();
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const ulonglong2 l = nl2[c];  // Shift::kP - lse2 of 4 queries
          pr[2 * c] = ex2_2(fma2(pair(s[4 * c], s[4 * c + 1]), sl2_2, l.x));
          pr[2 * c + 1] = ex2_2(fma2(pair(s[4 * c + 2], s[4 * c + 3]), sl2_2, l.y));
        }
        store(sa, pr);
        arrive(C::kPFull);
        if (!dp_there && !wait_all(db, np)) {
          failed = true;
          break;
        }
        tc_ld32(da, s);
        tc_wait_ld();
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const ulonglong2 d = ndl[c];  // -delta of 4 queries
          const uint64_t x = pair(s[4 * c], s[4 * c + 1]), y = pair(s[4 * c + 2], s[4 * c + 3]);
          if constexpr (!BF16) {
            pr[2 * c] = mul2(pr[2 * c], shift_2);
            pr[2 * c + 1] = mul2(pr[2 * c + 1], shift_2);
          }
          pr[2 * c] = mul2(pr[2 * c], add2(x, d.x));
          pr[2 * c + 1] = mul2(pr[2 * c + 1], add2(y, d.y));
        }
        store(da, pr);
        arrive(C::kDsFull);
      }
    }
  }

  if (failed) report_timeout();
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tc_dealloc(tmem, kTmemAll);
  }
}

// Gradients of the tiles that were cut, their parts added in order; 8 entries a
// thread. The parts of a tile are `pitch` entries apart.
template <bool BF16>
__device__ __forceinline__ void join_parts(const float* part, int64_t pitch, int parts, void* dst,
                                           int64_t at, bool g32) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = 0.f;
#pragma unroll 4
  for (int s = 0; s < parts; ++s, part += pitch) {
    const float4* src = reinterpret_cast<const float4*>(part);
    const float4 a = src[0], c = src[1];
    f[0] += a.x, f[1] += a.y, f[2] += a.z, f[3] += a.w;
    f[4] += c.x, f[5] += c.y, f[6] += c.z, f[7] += c.w;
  }
  if (g32) {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(dst) + at);
    o[0] = make_float4(f[0], f[1], f[2], f[3]);
    o[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(dst) + at) =
        make_uint4(pack2_t<BF16>(f[0], f[1]), pack2_t<BF16>(f[2], f[3]), pack2_t<BF16>(f[4], f[5]),
                   pack2_t<BF16>(f[6], f[7]));
  }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(256) swa_bwd_join_kernel(const SwaBwdProblem p) {
  constexpr int kRowThreads = D / 8;
  const int e = threadIdx.x % kRowThreads * 8;
  const int row = static_cast<int>(blockIdx.y) * (256 / kRowThreads) + threadIdx.x / kRowThreads;
  const int which = blockIdx.z;  // 0 dK, 1 dV
  const DkvItem it = dkv_item(p, p.whole_tiles + blockIdx.x * static_cast<uint32_t>(p.splits));
  const int j = it.j0 + row;
  if (j >= p.N) return;
  join_parts<BF16>(p.part + ((static_cast<int64_t>(it.part) * 2 + which) * kBlk + row) * D + e,
                   2 * kBlk * D, p.splits, which == 0 ? p.dK : p.dV,
                   ((static_cast<int64_t>(it.b) * p.N + j) * p.Hkv + it.g) * D + e, p.g32);
}

template <int D, bool BF16>
__global__ void __launch_bounds__(256) swa_bwd_join_dq_kernel(const SwaBwdProblem p) {
  constexpr int kRowThreads = D / 8;
  const int e = threadIdx.x % kRowThreads * 8;
  const int row = static_cast<int>(blockIdx.y) * (256 / kRowThreads) + threadIdx.x / kRowThreads;
  const DqItem it = dq_item<true>(p, p.dq_whole + blockIdx.x * static_cast<uint32_t>(p.dq_splits));
  const int i = it.q0 + row;
  if (i >= p.M) return;
  join_parts<BF16>(p.part_q + (static_cast<int64_t>(it.part) * kBlk + row) * D + e, kBlk * D,
                   p.dq_splits, p.dQ,
                   ((static_cast<int64_t>(it.b) * p.M + i) * p.H + it.h) * D + e, p.g32);
}

// ---------------------------------------------------------------- host

constexpr int kSms = 152;
// In steps of the dK, dV kernel (0.7 us): what an item costs beside its steps, the
// fewest steps of a part, the join (on the host too) and a part's 128 KB
// through it.
constexpr int kItemSteps = 3, kMinSteps = 4, kJoinSteps = 8;
constexpr double kPartSteps = 0.05;
constexpr int kMaxSplits = 64;

int check_swa_bwd(int64_t B, int64_t M, int64_t N, int64_t H, int64_t H_kv, int64_t D) {
  if (B < 0 || M < 0 || N < 0 || H <= 0 || H_kv <= 0) return NSA_ERR_SHAPE;
  if (H % H_kv != 0) return NSA_ERR_GROUPS;
  if (D != 64 && D != 128) return NSA_ERR_HEAD_DIM;
  const int64_t lim = int64_t(1) << 29;
  if (M > lim || N > lim || H > 65536 || B > 65536) return NSA_ERR_SHAPE;
  const int64_t top = (int64_t(1) << 31) - 1 - (1 << 20);  // items, steps of a tile
  if (B * H * ((M + kStep - 1) / kStep + 1) > top || B * H * ((N + kBlk - 1) / kBlk) > top)
    return NSA_ERR_SHAPE;
  return NSA_OK;
}

// How the tiles of a kernel are cut: `whole` of them are items of their own,
// the others (the last) are cut into `splits` parts of their steps, so that the
// SMs do not wait for a last, mostly empty round. Uneven tiles (a causal window
// over the whole sequence) are left alone once they are more than the SMs:
// their last ones are short.
struct Cut {
  int64_t tiles, whole;
  int splits;
  int64_t items() const { return whole + (tiles - whole) * splits; }
  int64_t parts() const { return (tiles - whole) * splits; }
};

// `save`: the share of the kernel that cutting has to save.
Cut cut_tiles(int64_t tiles, int64_t steps, bool even, double save) {
  Cut k{tiles, tiles, 1};
  const int64_t rest = k.tiles % kSms;
  if (k.tiles == 0 || rest == 0 || (k.tiles > kSms && !even)) return k;
  // the rest's time in steps for each number of parts: rounds of parts, each
  // with kItemSteps steps' worth of its own
  const double item = steps + kItemSteps, full = static_cast<double>(k.tiles / kSms) * item;
  double best = (1 - save) * (full + item) - full;
  for (int s = 2; s <= kMaxSplits && steps / s >= kMinSteps; ++s) {
    const double t = static_cast<double>((rest * s + kSms - 1) / kSms) *
                         (static_cast<double>(steps) / s + kItemSteps) +
                     kJoinSteps + kPartSteps * rest * s;
    if (t < best) {
      best = t;
      k.whole = k.tiles - rest;
      k.splits = s;
    }
  }
  return k;
}

// Of the dK, dV kernel, whose key tiles' steps are those of all query heads, and
// of the dQ kernel, whose steps take some 7 % longer when it can be cut: 4 heads
// of 2048 x 2048 would save 11 % by the rule and lost 2 of 55 us, a head of
// 4096 x 4096, causal, gained 6 to 12 of 66, 8 of 128 x 32,768 went from 300 to 87.
Cut key_tiles(int64_t B, int64_t M, int64_t N, int64_t H, int64_t H_kv, int64_t left,
              int64_t right) {
  const int64_t rows = left + right + kBlk;  // queries that see a key tile
  return cut_tiles(B * H_kv * ((N + kBlk - 1) / kBlk),
                   ((rows < M ? rows : M) + kStep - 1) / kStep * (H / H_kv),
                   rows <= M || (left >= M && right >= N), 0.05);
}

Cut query_tiles(int64_t B, int64_t M, int64_t N, int64_t H, int64_t left, int64_t right) {
  const int64_t keys = left + right + kBlk;  // keys that a query tile sees
  return cut_tiles(B * H * ((M + kBlk - 1) / kBlk), ((keys < N ? keys : N) + kStep - 1) / kStep,
                   keys <= N || (left >= M && right >= N), 0.2);
}

struct WindowSides {
  int64_t left, right;
};

WindowSides clamp_window(int64_t M, int64_t N, int64_t left, int64_t right) {
  return {left < 0 || left > M ? M : left, right < 0 || right > N ? N : right};
}

template <int D, bool BF16>
int launch_swa_bwd(const SwaBwdProblem& p, cudaStream_t st) {
  constexpr CUtensorMapDataType dt =
      BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  CUtensorMap tk, tv, tq, td, to;
  if (!encode_kv_map(&tk, p.K, p.B, p.N, p.Hkv, D, kStep, dt) ||
      !encode_kv_map(&tv, p.V, p.B, p.N, p.Hkv, D, kStep, dt) ||
      !encode_kv_map(&tq, p.Q, p.B, p.M, p.H, D, kStep, dt) ||
      !encode_kv_map(&to, p.O, p.B, p.M, p.H, D, kStep, dt) ||
      !encode_kv_map(&td, p.dO, p.B, p.M, p.H, D, kStep, dt))
    return NSA_ERR_LAUNCH;
  auto dq = p.part_q != nullptr ? swa_bwd_dq_kernel<D, BF16, true> : swa_bwd_dq_kernel<D, BF16, false>;
  auto dkv = swa_bwd_dkv_kernel<D, BF16>;
  if (cudaFuncSetAttribute(dq, cudaFuncAttributeMaxDynamicSharedMemorySize, DqCfg<D>::kSmem) !=
          cudaSuccess ||
      cudaFuncSetAttribute(dkv, cudaFuncAttributeMaxDynamicSharedMemorySize, DkvCfg<D>::kSmem) !=
          cudaSuccess)
    return NSA_ERR_LAUNCH;
  if constexpr (!BF16) {
    swa_bwd_vmax_kernel<D><<<static_cast<unsigned>(p.B * p.Hkv * p.ktiles), 256, 0, st>>>(
        p, static_cast<float*>(p.dV));
    if (cudaGetLastError() != cudaSuccess) return NSA_ERR_LAUNCH;
  }
  const int64_t qi = p.dq_items, ki = p.dkv_items;
  // one CTA per SM, items dealt to them
  dq<<<static_cast<unsigned>(qi < kSms ? qi : kSms), 32 * (kMmaWarp + 1), DqCfg<D>::kSmem, st>>>(p, tk, tv,
                                                                                       tq, to, td);
  if (cudaGetLastError() != cudaSuccess) return NSA_ERR_LAUNCH;
  dkv<<<static_cast<unsigned>(ki < kSms ? ki : kSms), 32 * (kMmaWarp + 2), DkvCfg<D>::kSmem, st>>>(
      p, tq, td, tk, tv);
  if (cudaGetLastError() != cudaSuccess) return NSA_ERR_LAUNCH;
  if (p.part_q != nullptr) {
    const dim3 grid(static_cast<unsigned>(p.B * p.H * p.qtiles - p.dq_whole), kBlk * D / 8 / 256);
    swa_bwd_join_dq_kernel<D, BF16><<<grid, 256, 0, st>>>(p);
    if (cudaGetLastError() != cudaSuccess) return NSA_ERR_LAUNCH;
  }
  if (p.part != nullptr) {
    const dim3 grid(static_cast<unsigned>(p.B * p.Hkv * p.ktiles - p.whole_tiles), kBlk * D / 8 / 256,
                    2);
    swa_bwd_join_kernel<D, BF16><<<grid, 256, 0, st>>>(p);
    if (cudaGetLastError() != cudaSuccess) return NSA_ERR_LAUNCH;
  }
  return NSA_OK;
}

}  // namespace

int swa_bwd_read_and_clear_status(unsigned int* value) { return read_and_clear_status(value); }

}  // namespace nsa

extern "C" int64_t nsa_swa_bwd_workspace_bytes(int64_t B, int64_t M, int64_t N, int64_t H,
                                               int64_t H_kv, int64_t D, int64_t window_left,
                                               int64_t window_right) {
  using namespace nsa;
  const int rc = check_swa_bwd(B, M, N, H, H_kv, D);
  if (rc != NSA_OK) return rc;
  if (B == 0 || M == 0 || N == 0) return 0;
  const WindowSides w = clamp_window(M, N, window_left, window_right);
  const int64_t Mp = (M + kStep - 1) / kStep * kStep;
  return 2 * B * H * Mp * 4 +
         (key_tiles(B, M, N, H, H_kv, w.left, w.right).parts() * 2 +
          query_tiles(B, M, N, H, w.left, w.right).parts()) *
             kBlk * D * 4;
}

extern "C" int nsa_swa_bwd(const void* Q, const void* K, const void* V, const void* O,
                           const float* LSE, const void* dO, void* dQ, void* dK, void* dV,
                           int64_t B, int64_t M, int64_t N, int64_t H, int64_t H_kv, int64_t D,
                           int64_t window_left, int64_t window_right, float scale, int dtype,
                           int grad_dtype, void* workspace, int64_t workspace_bytes,
                           void* stream) {
  using namespace nsa;
  const int rc = check_swa_bwd(B, M, N, H, H_kv, D);
  if (rc != NSA_OK) return rc;
  if (dtype != NSA_F16 && dtype != NSA_BF16) return NSA_ERR_DTYPE;
  if (grad_dtype != NSA_F32 && grad_dtype != dtype) return NSA_ERR_DTYPE;
  auto mis = [](const void* ptr, uintptr_t a) {
    return ptr != nullptr && (reinterpret_cast<uintptr_t>(ptr) & (a - 1)) != 0;
  };
  const bool queries = B > 0 && M > 0, keys = B > 0 && N > 0;
  if (queries && (!Q || !O || !LSE || !dO || !dQ)) return NSA_ERR_NULL;
  if (keys && (!K || !V || !dK || !dV)) return NSA_ERR_NULL;
  if (mis(Q, 16) || mis(K, 16) || mis(V, 16) || mis(O, 16) || mis(dO, 16) || mis(dQ, 16) ||
      mis(dK, 16) || mis(dV, 16) || mis(LSE, 4))
    return NSA_ERR_ALIGN;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int64_t ge = grad_dtype == NSA_F32 ? 4 : 2;
  if (!queries || !keys) {  // nothing is visible: zero gradients
    if (queries && cudaMemsetAsync(dQ, 0, B * M * H * D * ge, st) != cudaSuccess)
      return NSA_ERR_LAUNCH;
    if (keys && (cudaMemsetAsync(dK, 0, B * N * H_kv * D * ge, st) != cudaSuccess ||
                 cudaMemsetAsync(dV, 0, B * N * H_kv * D * ge, st) != cudaSuccess))
      return NSA_ERR_LAUNCH;
    return NSA_OK;
  }
  if (!workspace || workspace_bytes < nsa_swa_bwd_workspace_bytes(B, M, N, H, H_kv, D, window_left,
                                                                  window_right))
    return NSA_ERR_WORKSPACE;
  if (mis(workspace, 16)) return NSA_ERR_ALIGN;
  const WindowSides w = clamp_window(M, N, window_left, window_right);
  SwaBwdProblem p{};
  p.Q = static_cast<const uint16_t*>(Q);
  p.K = static_cast<const uint16_t*>(K);
  p.V = static_cast<const uint16_t*>(V);
  p.O = static_cast<const uint16_t*>(O);
  p.dO = static_cast<const uint16_t*>(dO);
  p.LSE = LSE;
  p.dQ = dQ;
  p.dK = dK;
  p.dV = dV;
  p.B = static_cast<int>(B);
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.H = static_cast<int>(H);
  p.Hkv = static_cast<int>(H_kv);
  p.hpg = static_cast<int>(H / H_kv);
  p.Mp = static_cast<int>((M + kStep - 1) / kStep * kStep);
  p.qtiles = static_cast<int>((M + kBlk - 1) / kBlk);
  p.ktiles = static_cast<int>((N + kBlk - 1) / kBlk);
  const Cut keys_cut = key_tiles(B, M, N, H, H_kv, w.left, w.right);
  p.splits = keys_cut.splits;
  p.whole_tiles = static_cast<int>(keys_cut.whole);
  p.dkv_items = static_cast<int>(keys_cut.items());
  const Cut queries_cut = query_tiles(B, M, N, H, w.left, w.right);
  p.dq_splits = queries_cut.splits;
  p.dq_whole = static_cast<int>(queries_cut.whole);
  p.dq_items = static_cast<int>(queries_cut.items());
  p.left = static_cast<int>(w.left);
  p.right = static_cast<int>(w.right);
  p.scale = scale > 0.f ? scale : 1.0f / sqrtf(static_cast<float>(D));
  p.sl2 = p.scale * 1.4426950408889634f;
  p.g32 = grad_dtype == NSA_F32;
  p.wide = !mis(dQ, 32) && !mis(dK, 32) && !mis(dV, 32) && !mis(workspace, 32);
  p.vmax = static_cast<const float*>(dV);
  p.vmax_g = D * ge / 4;
  p.vmax_t = kBlk * H_kv * p.vmax_g;
  p.vmax_b = N * H_kv * p.vmax_g;
  const int64_t stat = B * H * p.Mp;
  p.nlse2 = static_cast<float*>(workspace);
  p.ndelta = p.nlse2 + stat;
  float* const parts = p.ndelta + stat;
  p.part = keys_cut.parts() > 0 ? parts : nullptr;
  p.part_q = queries_cut.parts() > 0 ? parts + keys_cut.parts() * 2 * kBlk * D : nullptr;
  const bool bf = dtype == NSA_BF16;
  if (D == 64) return bf ? launch_swa_bwd<64, true>(p, st) : launch_swa_bwd<64, false>(p, st);
  return bf ? launch_swa_bwd<128, true>(p, st) : launch_swa_bwd<128, false>(p, st);
}
