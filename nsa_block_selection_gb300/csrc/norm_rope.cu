// RMS norm of every query and key head and the position rotation in one pass
// over the projections' outputs, and its backward, for sm_103a.
//
// Per row x of D entries (one head of one token), with the head norm's weight
// w and the token's angles c_i, s_i (cos and sin tables, row = position):
//   r = rsqrt(mean(x^2) + eps),  n = x r w,
//   (a, b) -> (a c_i - b s_i, b c_i + a s_i)  for the R / 2 pairs (a, b) of
//   the first R entries (entries i and i + R/2, or 2i and 2i + 1),
// entries past R pass through. Backward, with g = the pairs of dy turned by
// the opposite angle and xhat = x r:
//   dw += g xhat,   dx = r (g w - xhat mean(g w xhat)).
// All of it is fp32, rounded once when a result is stored. In the forward every
// operation is rounded by itself, in this order, and a row's squares are added in a
// fixed one (row_squares): the same row comes out of any layout and kernel, and of
// elementary fp32 operations, so that the 4-bit codes a cache makes of it, which jump
// by a step where a last bit moves, can be formed again anywhere. (Fused turns and
// x (r w) moved 1 in 10,000 last bits.)
//
// The bytes bound both: each row is read once and written once. In the forward
// a row is held by D / 16 lanes, 16 entries each, as two 16-byte chunks that
// hold both entries of every pair: lane t takes chunks t and t + R/16 while
// t < R/16, and two consecutive chunks of the tail after that, so the rotation
// needs no exchange between lanes in either pairing and the only shuffles are
// the row sums' (2 at D = 64; 7 at 128, or 3 and loads from the cache where R < D).
// The backward does the same with D / 8 lanes of two 8-byte chunks. A warp has 4
// (D = 128) or 8 row slots in the forward and 2 or 4 in the backward; with many heads
// they walk the heads of one token, whose angles they share, with few they hold several
// tokens.
//
// Measured, bf16, 64 + 8 heads of D = 128: 65,536 tokens forward 360 us
// (6.7 TB/s, 99 % of a copy), 32,768 tokens backward 333 us (5.5 TB/s, 81 %:
// of the instruction slots 58 % are taken, and 24 warps an SM, what 80
// registers a thread allow, keep too few loads in flight for more). Short
// calls are bound by their launches: a token of 64 + 8 heads takes 2.6 us on
// the device, most of it the launch.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "common.cuh"
#include "nsa_sel_attn.h"
#include "ptx.cuh"
#include "rope.cuh"

namespace nsa {
namespace {

constexpr int kRopeThreads = 128;      // forward CTAs: 4 warps, each a unit of its own
constexpr int kRopeBwdThreads = 256;   // backward CTAs: 8 warps that share one dw partial
constexpr int kRopeBwdPerSm = 3;       // and how many of them an SM holds
constexpr int kRopeSms = 152;
constexpr int kFewPerSm = 7;  // CTAs of norm_rope_few_kernel that an SM holds
// The forward gives every row slot its own token up to this many groups of
// slots a token, or this many groups in all; beyond, a warp walks a token's
// heads with one set of angles. Both measured, 32,768 tokens of 48 + 8 heads at
// D = 64 (7 groups): 93 us against 94, of 24 + 4 at D = 128 (7): 96 and 97, of 24 + 8
// (8): 109 against 101, of 32 + 4 (9): 122 against 106; 2000 tokens of 32 + 4 at
// D = 128 (18,000 groups): 9.2 against 10.5, 1000 of 64 + 8 (18,000) 9.0 and 8.0, 4096
// of those (73,728) 33 against 31.
constexpr int kFewPerToken = 7;
constexpr int64_t kFewGroups = 128 * kRopeSms;
// What a unit of the backward that walks a token's heads costs, beside a
// group of slots that hold several tokens: its position and angles, and each
// group of the heads. Shares of the CTAs by these against shares by groups of
// slots alone: 32,768 tokens of 32 + 4 heads at D = 64 102 us against 143,
// of 64 + 8 at D = 128 338 against 351.
constexpr double kUnitCost = 0.5, kGroupCost = 0.6;

// One warp per unit: `per` rows of the H + G head rows of one token.
template <int D, bool BF16, bool FULL, int UN>
__global__ void __launch_bounds__(kRopeThreads, FULL ? 5 : 4)
    norm_rope_kernel(const RopeProblem p, int segs, int per, int64_t units) {
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kRopeThreads / 32) + (threadIdx.x >> 5);
  if (unit >= units) return;
  const uint32_t tok = static_cast<uint32_t>(unit) / static_cast<uint32_t>(segs);
  const int seg = static_cast<int>(static_cast<uint32_t>(unit) - tok * segs);
  const int b = static_cast<int>(tok / static_cast<uint32_t>(p.M));
  const int m = static_cast<int>(tok - static_cast<uint32_t>(b) * p.M);
  const int64_t at = token_position(p, b, m);
  const bool live = at >= 0;
  int c0, c1;
  const int t = (threadIdx.x & 31) % (D / 16), half = FULL ? D / 2 : p.half;
  row_chunks(t, half, c0, c1);
  const bool rot = t < (half >> 3);
  float c[8], s[8];
  if (live && rot) load_angles(p, at, half, c0, c1, c, s);
  const int r0 = seg * per, r1 = min(r0 + per, p.q.heads + p.k.heads);
  if (r0 < p.q.heads)
    norm_rope_rows<D, BF16, FULL, !FULL, UN>(p, p.q, b, m, r0, min(r1, p.q.heads), live, rot, c0, c1,
                                             c, s);
  if (r1 > p.q.heads)
    norm_rope_rows<D, BF16, FULL, !FULL, UN>(p, p.k, b, m, max(r0 - p.q.heads, 0), r1 - p.q.heads,
                                             live, rot, c0, c1, c, s);
}

// The forward where a token has few heads: a row slot of a warp keeps its head,
// and the head's weights, and walks the tokens, each with its own position and
// angles. (A warp per token leaves row slots empty and pays the latencies of
// position, angles and rows for each: 32,768 tokens of 1 + 1 heads at D = 64
// 51 us against 5.5, of 8 + 2 55 against 27. Two rows in flight a lane, for 16
// to 20 warps an SM, took a tenth more of the latter than 28 warps of one row;
// loading the next position early gave nothing.)
template <int D, bool BF16, bool FULL>
__global__ void __launch_bounds__(kRopeThreads, kFewPerSm)
    norm_rope_few_kernel(const RopeProblem p, const RowGroups rg) {
  constexpr int LPR = D / 16, RPW = 32 / LPR;
  const int lane = threadIdx.x & 31, sub = lane / LPR, tl = lane % LPR;
  // this warp's place among the groups of a token, and where its walk begins
  const uint32_t groups = static_cast<uint32_t>(rg.per_token);
  const uint32_t wid = blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
  const uint32_t walks = gridDim.x * (kRopeThreads / 32) / groups;
  const uint32_t first = wid / groups;
  if (first >= walks) return;
  // slots of a group that hold one token, and tokens of a group
  const int wide = rg.per_token > 1 ? RPW : 1 << rg.shift;
  const uint32_t sets = static_cast<uint32_t>(RPW / wide);
  const int head = static_cast<int>(wid - first * groups) * RPW + (sub & (wide - 1));
  const bool is_k = head >= p.q.heads, slot = head < p.q.heads + p.k.heads;
  const RopeRows& t = is_k ? p.k : p.q;
  const int64_t h = is_k ? head - p.q.heads : head;
  int c0, c1;
  const int half = FULL ? D / 2 : p.half;
  row_chunks(tl, half, c0, c1);
  const bool rot = tl < (half >> 3);
  float w[16];
  load_weights<BF16>(t.w, p.w32, c0, c1, w);
  const uint8_t* const x = t.x + 2 * h * t.xh;
  uint8_t* const y = t.y + 2 * h * t.yh;
  const uint64_t tokens = static_cast<uint64_t>(p.B) * p.M;
  // (all lanes of a warp go through the loop together: row_sum needs them)
  for (uint64_t begin = static_cast<uint64_t>(first) * sets; begin < tokens;
       begin += static_cast<uint64_t>(walks) * sets) {
    const uint64_t tok = begin + static_cast<uint32_t>(sub / wide);
    const bool in = slot && tok < tokens;
    bool live = false;
    int64_t yo = 0;
    float f[16], c[8], s[8];
    uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0;
    const uint8_t* src = x;
    if (in) {
      const int b = static_cast<int>(static_cast<uint32_t>(tok) / static_cast<uint32_t>(p.M));
      const int m = static_cast<int>(static_cast<uint32_t>(tok) - static_cast<uint32_t>(b) * p.M);
      const int64_t at = token_position(p, b, m);
      yo = 2 * (b * t.yb + m * t.ym);
      live = at >= 0;
      if (live) {  // (padding is not read)
        src += 2 * (b * t.xb + m * t.xm);
        v0 = reinterpret_cast<const uint4*>(src)[c0];
        v1 = reinterpret_cast<const uint4*>(src)[c1];
        if (rot) load_angles(p, at, half, c0, c1, c, s);
      }
    }
    const float sq = row_squares<D, BF16, FULL>(v0, v1, src, live);
    unpack8<BF16>(v0, f);
    unpack8<BF16>(v1, f + 8);
    if (live) {  // a padding token's rows are zero
      scale_row(f, rsqrtf(sq * (1.f / D) + p.eps), w);
      if (rot) turn(f, c, s, p.interleaved);
    }
    if (in) {
      uint4* dst = reinterpret_cast<uint4*>(y + yo);
      dst[c0] = pack8<BF16>(f);
      dst[c1] = pack8<BF16>(f + 8);
    }
  }
}

struct RopeBwdRows {
  const uint8_t* x;   // Q or K as the forward read it
  const uint8_t* dy;  // gradient of the forward's result, in the grad type
  uint8_t* dx;
  const void* w;
  int64_t xb, xm, xh, gb, gm, gh, db, dm, dh;
  int heads;
  int segs, per;      // a token's heads are cut into segs units of per heads
  int64_t units;
  bool few;           // the row slots of a warp hold several tokens instead
  RowGroups groups;
  int ctas;           // CTAs that work on this tensor
};

struct RopeBwdProblem {
  RopeProblem a;  // tables, positions, flags (its q and k are unused)
  RopeBwdRows q, k;
  float* part;    // [q.ctas + k.ctas, D] partial dw, or NULL
};

// The backward's lanes hold half as much of a row as the forward's, two
// chunks of 4 entries: with the sums of dw, the weights and two inputs to keep,
// 16 entries a lane left 16 warps an SM, too few loads in flight and too few
// row sums to overlap (32,768 tokens of 64 + 8 heads at D = 128: 373 us).
__device__ __forceinline__ void row_quads(int t, int half, int& c0, int& c1) {
  const int pc = half >> 2;  // chunks of a half
  if (t < pc) {
    c0 = t;
    c1 = t + pc;
  } else {
    c0 = 2 * t;
    c1 = 2 * t + 1;
  }
}

template <bool BF16>
__device__ __forceinline__ void unpack4(const uint2& v, float* f) {
  const float2 a = unpack2<BF16>(v.x), b = unpack2<BF16>(v.y);
  f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
}

__device__ __forceinline__ void load4(const float* p, float* f) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
}

// The token and head of a row slot in group q.
template <int RPW>
__device__ __forceinline__ void group_row(const RowGroups& g, uint32_t q, int sub, uint32_t& tok,
                                          int& head) {
  tok = q * (static_cast<uint32_t>(RPW) >> g.shift) + (static_cast<uint32_t>(sub) >> g.shift);
  head = sub & ((1 << g.shift) - 1);
}

// What a lane of the backward holds of one row, and what it does with it.
template <bool BF16, bool G32>
struct BwdRow {
  uint2 v[2];
  uint4 g[G32 ? 2 : 1];  // fp32: the two chunks; 16 bits: both in one

  __device__ __forceinline__ void zero() {
    v[0] = v[1] = make_uint2(0, 0);
#pragma unroll
    for (int i = 0; i < (G32 ? 2 : 1); ++i) g[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void load(const uint8_t* x, const uint8_t* dy, int c0, int c1) {
    const uint2* src = reinterpret_cast<const uint2*>(x);
    v[0] = src[c0];
    v[1] = src[c1];
    if constexpr (G32) {
      const uint4* gr = reinterpret_cast<const uint4*>(dy);
      g[0] = gr[c0];
      g[1] = gr[c1];
    } else {
      const uint2* gr = reinterpret_cast<const uint2*>(dy);
      const uint2 ga = gr[c0], gb = gr[c1];
      g[0] = make_uint4(ga.x, ga.y, gb.x, gb.y);
    }
  }
  // dx, stored at dst, and the row's share of dw (neither when the slot is
  // not in use)
  template <int D>
  __device__ __forceinline__ void work(const RopeProblem& p, bool rot, const float* c,
                                       const float* s, const float* w, float* dw, bool in,
                                       uint8_t* base, int64_t off, int c0, int c1) const {
    float f[8], y[8];
    unpack4<BF16>(v[0], f);
    unpack4<BF16>(v[1], f + 4);
    if constexpr (G32) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        y[4 * i] = __uint_as_float(g[i].x);
        y[4 * i + 1] = __uint_as_float(g[i].y);
        y[4 * i + 2] = __uint_as_float(g[i].z);
        y[4 * i + 3] = __uint_as_float(g[i].w);
      }
    } else {
      unpack4<BF16>(make_uint2(g[0].x, g[0].y), y);
      unpack4<BF16>(make_uint2(g[0].z, g[0].w), y + 4);
    }
    if (rot) {  // the opposite turn: (a, b) -> (a c + b s, b c - a s)
      if (p.interleaved) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float a = y[2 * j], e = y[2 * j + 1];
          y[2 * j] = a * c[j] + e * s[j];
          y[2 * j + 1] = e * c[j] - a * s[j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float a = y[j], e = y[j + 4];
          y[j] = a * c[j] + e * s[j];
          y[j + 4] = e * c[j] - a * s[j];
        }
      }
    }
    float sq = 0.f, gx = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      sq = fmaf(f[i], f[i], sq);
      gx = fmaf(y[i] * w[i], f[i], gx);
    }
    sq = row_sum<D / 8>(sq);
    gx = row_sum<D / 8>(gx);
    // slots without a row hold zeros (with eps = 0 their rs is infinite)
    if (in) {
      const float rs = rsqrtf(sq * (1.f / D) + p.eps);
      const float kx = gx * rs * rs * (1.f / D);  // mean(g w xhat) rs
      float d[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        dw[i] = fmaf(y[i], f[i] * rs, dw[i]);
        d[i] = rs * fmaf(-f[i], kx, y[i] * w[i]);
      }
      uint2* o = reinterpret_cast<uint2*>(base + off);
      o[c0] = make_uint2(pack2_t<BF16>(d[0], d[1]), pack2_t<BF16>(d[2], d[3]));
      o[c1] = make_uint2(pack2_t<BF16>(d[4], d[5]), pack2_t<BF16>(d[6], d[7]));
    }
  }
};

// The 4 angles of a lane's pairs.
__device__ __forceinline__ void load_angles4(const RopeProblem& p, int64_t at, int c0, int c1,
                                             float* c, float* s) {
  const float* ct = p.cos_t + at * p.half;
  const float* st = p.sin_t + at * p.half;
  if (p.interleaved) {  // pairs 0, 1 of the first chunk, 2, 3 of the second
    const float2 ca = *reinterpret_cast<const float2*>(ct + 2 * c0);
    const float2 cb = *reinterpret_cast<const float2*>(ct + 2 * c1);
    const float2 sa = *reinterpret_cast<const float2*>(st + 2 * c0);
    const float2 sb = *reinterpret_cast<const float2*>(st + 2 * c1);
    c[0] = ca.x, c[1] = ca.y, c[2] = cb.x, c[3] = cb.y;
    s[0] = sa.x, s[1] = sa.y, s[2] = sb.x, s[3] = sb.y;
  } else {
    load4(ct + 4 * c0, c);
    load4(st + 4 * c0, s);
  }
}

template <bool BF16>
__device__ __forceinline__ void load_weights8(const RopeProblem& p, const void* w, int c0, int c1,
                                              float* f) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = 1.f;
  if (w == nullptr) return;
  if (p.w32) {
    load4(static_cast<const float*>(w) + 4 * c0, f);
    load4(static_cast<const float*>(w) + 4 * c1, f + 4);
  } else {
    unpack4<BF16>(static_cast<const uint2*>(w)[c0], f);
    unpack4<BF16>(static_cast<const uint2*>(w)[c1], f + 4);
  }
}

// A CTA's partial dw from its lanes' sums: the row slots of a warp, then the
// warps, in a fixed order.
template <int D>
__device__ __forceinline__ void cta_dw(float* dw, int c0, int c1, float (*sh)[D], float* part) {
  constexpr int LPR = D / 8, kWarps = kRopeBwdThreads / 32;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1) dw[i] += __shfl_xor_sync(kFull, dw[i], o);
  }
  if ((threadIdx.x & 31) < LPR) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sh[threadIdx.x >> 5][4 * c0 + i] = dw[i];
      sh[threadIdx.x >> 5][4 * c1 + i] = dw[4 + i];
    }
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) v += sh[i][threadIdx.x];
    part[static_cast<int64_t>(blockIdx.x) * D + threadIdx.x] = v;
  }
}

// A warp's walk over the rows of one tensor, a token's heads at a time.
template <int D, bool BF16, bool G32, int UN>
__device__ __forceinline__ void bwd_tokens(const RopeProblem& p, const RopeBwdRows& t, int64_t first,
                                           int sub, int c0, int c1, bool rot, const float* w,
                                           float* dw) {
  constexpr int RPW = 32 / (D / 8);
  // (the step formed here: kept in registers across the loop it cost 1 %)
  for (int64_t u = first; u < t.units;
       u += static_cast<int64_t>(t.ctas) * (kRopeBwdThreads / 32)) {
    const uint32_t tok = static_cast<uint32_t>(u) / static_cast<uint32_t>(t.segs);
    const int seg = static_cast<int>(static_cast<uint32_t>(u) - tok * t.segs);
    const int b = static_cast<int>(tok / static_cast<uint32_t>(p.M));
    const int m = static_cast<int>(tok - static_cast<uint32_t>(b) * p.M);
    const int r0 = seg * t.per, r1 = min(r0 + t.per, t.heads);
    const int64_t at = token_position(p, b, m);
    uint8_t* const dx = t.dx + 2 * (b * t.db + m * t.dm);
    if (at < 0) {  // padding: a zero gradient
      for (int row = r0 + sub; row < r1; row += RPW) {
        uint2* dst = reinterpret_cast<uint2*>(dx + 2 * row * t.dh);
        dst[c0] = dst[c1] = make_uint2(0, 0);
      }
      continue;
    }
    float c[4], s[4];
    if (rot) load_angles4(p, at, c0, c1, c, s);
    const uint8_t* const x = t.x + 2 * (b * t.xb + m * t.xm);
    const uint8_t* const dy = t.dy + (G32 ? 4 : 2) * (b * t.gb + m * t.gm);
    for (int r = r0; r < r1; r += RPW * UN) {
      BwdRow<BF16, G32> d[UN];
#pragma unroll
      for (int k = 0; k < UN; ++k) {
        const int row = r + k * RPW + sub;
        d[k].zero();
        if (row < r1) d[k].load(x + 2 * row * t.xh, dy + (G32 ? 4 : 2) * row * t.gh, c0, c1);
      }
#pragma unroll
      for (int k = 0; k < UN; ++k) {
        const int row = r + k * RPW + sub;
        d[k].template work<D>(p, rot, c, s, w, dw, row < r1, dx, 2 * row * t.dh, c0, c1);
      }
    }
  }
}

// The same where a token has no more heads than a warp has row slots, UN
// neighbouring groups of slots at a time (32,768 tokens of 1 + 1 heads at
// D = 64: 50 us a token at a time, 21 here), with an fp32 gradient one. At 80
// registers all of the backward's forms spill a little: this one 48 to 64 bytes a
// thread with 16-bit gradients, 8 to 16 with fp32 ones, of which two groups at
// a time would spill 124 to 144.
template <int D, bool BF16, bool G32, int UN>
__device__ __forceinline__ void bwd_groups(const RopeProblem& p, const RopeBwdRows& t, int64_t first,
                                           int64_t stride, int sub, int c0, int c1, bool rot,
                                           const float* w, float* dw) {
  constexpr int RPW = 32 / (D / 8);
  const uint32_t tokens = static_cast<uint32_t>(p.B) * static_cast<uint32_t>(p.M);
  for (int64_t q = first * UN; q < t.groups.groups; q += stride * UN) {
    BwdRow<BF16, G32> d[UN];
    uint8_t* dst[UN];
    float c[UN][4], s[UN][4];
#pragma unroll
    for (int k = 0; k < UN; ++k) {
      uint32_t tok;
      int head;
      group_row<RPW>(t.groups, static_cast<uint32_t>(q) + k, sub, tok, head);
      d[k].zero();
      dst[k] = nullptr;
      if (q + k < t.groups.groups && tok < tokens && head < t.heads) {
        const int b = static_cast<int>(tok / static_cast<uint32_t>(p.M));
        const int m = static_cast<int>(tok - static_cast<uint32_t>(b) * p.M);
        const int64_t at = token_position(p, b, m), h = head;
        uint8_t* const o = t.dx + 2 * (b * t.db + m * t.dm + h * t.dh);
        if (at >= 0) {
          dst[k] = o;
          d[k].load(t.x + 2 * (b * t.xb + m * t.xm + h * t.xh),
                    t.dy + (G32 ? 4 : 2) * (b * t.gb + m * t.gm + h * t.gh), c0, c1);
          if (rot) load_angles4(p, at, c0, c1, c[k], s[k]);
        } else {  // padding: a zero gradient
          reinterpret_cast<uint2*>(o)[c0] = reinterpret_cast<uint2*>(o)[c1] = make_uint2(0, 0);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < UN; ++k)
      d[k].template work<D>(p, rot && dst[k] != nullptr, c[k], s[k], w, dw, dst[k] != nullptr, dst[k], 0,
                            c0, c1);
  }
}

// A CTA works on the rows of Q or of K (so that a lane carries one norm's
// sums) and leaves one partial dw. Warps walk the units.
template <int D, bool BF16, bool G32, bool FEW>
__global__ void __launch_bounds__(kRopeBwdThreads, kRopeBwdPerSm)
    norm_rope_bwd_kernel(const __grid_constant__ RopeBwdProblem pr) {
  const RopeProblem& p = pr.a;
  constexpr int LPR = D / 8, kWarps = kRopeBwdThreads / 32;
  __shared__ float sh[kWarps][D];
  const bool is_k = blockIdx.x >= static_cast<unsigned>(pr.q.ctas);
  const RopeBwdRows& t = is_k ? pr.k : pr.q;
  const int cta = static_cast<int>(blockIdx.x) - (is_k ? pr.q.ctas : 0);
  int c0, c1;
  const int lane = threadIdx.x & 31, tl = lane % LPR, sub = lane / LPR;
  row_quads(tl, p.half, c0, c1);
  const bool rot = tl < (p.half >> 2);
  float dw[8], w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[i] = 0.f;
  load_weights8<BF16>(p, t.w, c0, c1, w);
  const int64_t first = static_cast<int64_t>(cta) * kWarps + (threadIdx.x >> 5);
  if (FEW && t.few)
    bwd_groups<D, BF16, G32, G32 ? 1 : 2>(p, t, first, static_cast<int64_t>(t.ctas) * kWarps, sub, c0,
                                          c1, rot, w, dw);
  else
    bwd_tokens<D, BF16, G32, 2>(p, t, first, sub, c0, c1, rot, w, dw);
  if (pr.part != nullptr) cta_dw<D>(dw, c0, c1, sh, pr.part);
}

// dw from the CTAs' partials: a CTA sums 32 columns of dwq or dwk, 32 rows of
// partials side by side, in a fixed order.
template <int D>
__global__ void __launch_bounds__(1024)
    norm_rope_dw_kernel(const float* part, int q_ctas, int k_ctas, float* dwq, float* dwk) {
  __shared__ float sh[32][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const bool is_k = blockIdx.y == 1;
  const float* src = part + (is_k ? static_cast<int64_t>(q_ctas) * D : 0) + blockIdx.x * 32 + x;
  const int rows = is_k ? k_ctas : q_ctas;
  float v = 0.f;
  for (int r = y; r < rows; r += 32) v += src[static_cast<int64_t>(r) * D];
  sh[y][x] = v;
  __syncthreads();
  v = sh[x][y];  // the 32 sums of column y of this CTA
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  float* dst = is_k ? dwk : dwq;
  if (x == 0 && dst != nullptr) dst[blockIdx.x * 32 + y] = v;
}

// ---- host ---------------------------------------------------------------

// Most CTAs of the backward, each with one dw partial: what the SMs hold at
// once, for Q and K together; one of each at least.
constexpr int kRopeBwdCtas = kRopeBwdPerSm * kRopeSms;

int rope_bwd_most_ctas(int64_t B, int64_t M) {
  const int64_t tokens = B * M;
  return tokens == 0 ? 0 : kRopeBwdCtas;
}

// What a tensor's rows cost the backward, in groups of row slots, and whether
// the slots hold several tokens.
double rope_bwd_cost(RopeBwdRows& t, int64_t tokens, int slots) {
  t.few = t.heads <= slots;
  t.groups = plan_row_groups(t.heads, tokens, slots);
  if (t.few) return static_cast<double>(t.groups.groups);
  return static_cast<double>(tokens) * (kUnitCost + kGroupCost * ((t.heads + slots - 1) / slots));
}

// A token's heads in units of `per` (a multiple of a warp's rows): whole
// tokens when they alone give every warp of `ctas` one, else as few heads as
// it takes. Fewer CTAs where the units do not fill them.
void plan_rope_rows(RopeBwdRows& t, int64_t tokens, int rows_per_warp, int ctas) {
  if (t.few) {
    const int64_t need = (t.groups.groups + kRopeBwdThreads / 32 - 1) / (kRopeBwdThreads / 32);
    t.ctas = static_cast<int>(need < ctas ? need : ctas);
    return;
  }
  const int64_t warps = static_cast<int64_t>(ctas) * (kRopeBwdThreads / 32);
  const int64_t most = (t.heads + rows_per_warp - 1) / rows_per_warp;
  int64_t segs = (warps + tokens - 1) / tokens;
  if (segs > most) segs = most;
  const int64_t per = ((t.heads + segs - 1) / segs + rows_per_warp - 1) / rows_per_warp * rows_per_warp;
  t.per = static_cast<int>(per);
  t.segs = static_cast<int>((t.heads + per - 1) / per);
  t.units = tokens * t.segs;
  const int64_t need = (t.units + kRopeBwdThreads / 32 - 1) / (kRopeBwdThreads / 32);
  t.ctas = static_cast<int>(need < ctas ? need : ctas);
}

template <int D, bool BF16, bool FULL>
int launch_norm_rope_full(const RopeProblem& p, cudaStream_t st) {
  constexpr int RPW = 32 / (D / 16), UN = 4;
  const int rows = p.q.heads + p.k.heads;
  const int64_t tokens = static_cast<int64_t>(p.B) * p.M;
  const RowGroups g = plan_row_groups(rows, tokens, RPW);
  if (rows <= kFewPerToken * RPW || g.groups <= kFewGroups) {
    // a warp for every group of all tokens, or as many as the SMs hold, but one
    // for each group of a token
    constexpr int64_t kWarps = kRopeThreads / 32;
    int64_t warps = g.groups;
    if (warps > kFewPerSm * kRopeSms * kWarps) warps = kFewPerSm * kRopeSms * kWarps;
    if (warps < g.per_token) warps = g.per_token;
    norm_rope_few_kernel<D, BF16, FULL>
        <<<static_cast<unsigned>((warps + kWarps - 1) / kWarps), kRopeThreads, 0, st>>>(p, g);
    return cudaGetLastError() == cudaSuccess ? NSA_OK : NSA_ERR_LAUNCH;
  }
  // rows per warp: a whole token when the tokens alone give every SM 16
  // warps, else as few rows as it takes to get there
  const int64_t want = 16 * kRopeSms;
  int64_t segs = (want + tokens - 1) / tokens;
  const int64_t most = (rows + RPW - 1) / RPW;
  if (segs > most) segs = most;
  int64_t per = (rows + segs - 1) / segs;
  per = (per + RPW - 1) / RPW * RPW;
  segs = (rows + per - 1) / per;
  // (under 2^32, as the kernel takes them: there are fewer than 2^31 tokens, and
  // with more than one segment each no more than some 2 x 16 x 152 units)
  const int64_t units = tokens * segs;
  const int64_t blocks = (units + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  norm_rope_kernel<D, BF16, FULL, UN><<<static_cast<unsigned>(blocks), kRopeThreads, 0, st>>>(
      p, static_cast<int>(segs), static_cast<int>(per), units);
  return cudaGetLastError() == cudaSuccess ? NSA_OK : NSA_ERR_LAUNCH;
}

template <int D, bool BF16>
int launch_norm_rope(const RopeProblem& p, cudaStream_t st) {
  return 2 * p.half == D ? launch_norm_rope_full<D, BF16, true>(p, st)
                         : launch_norm_rope_full<D, BF16, false>(p, st);
}

template <int D, bool BF16, bool G32>
int launch_norm_rope_bwd(RopeBwdProblem& p, float* dwq, float* dwk, cudaStream_t st) {
  constexpr int RPW = 32 / (D / 8);
  const int64_t tokens = static_cast<int64_t>(p.a.B) * p.a.M;
  // the CTAs, by what the rows of Q and of K cost
  const double cq = rope_bwd_cost(p.q, tokens, RPW), ck = rope_bwd_cost(p.k, tokens, RPW);
  int k_ctas = static_cast<int>(kRopeBwdCtas * ck / (cq + ck) + 0.5);
  k_ctas = k_ctas < 1 ? 1 : k_ctas > kRopeBwdCtas - 1 ? kRopeBwdCtas - 1 : k_ctas;
  plan_rope_rows(p.q, tokens, RPW, kRopeBwdCtas - k_ctas);
  plan_rope_rows(p.k, tokens, RPW, k_ctas);
  const int ctas = p.q.ctas + p.k.ctas;
  if (p.q.few || p.k.few)
    norm_rope_bwd_kernel<D, BF16, G32, true><<<ctas, kRopeBwdThreads, 0, st>>>(p);
  else
    norm_rope_bwd_kernel<D, BF16, G32, false><<<ctas, kRopeBwdThreads, 0, st>>>(p);
  if (cudaGetLastError() != cudaSuccess) return NSA_ERR_LAUNCH;
  if (p.part != nullptr) {
    norm_rope_dw_kernel<D><<<dim3(D / 32, 2), 1024, 0, st>>>(p.part, p.q.ctas, p.k.ctas, dwq, dwk);
    if (cudaGetLastError() != cudaSuccess) return NSA_ERR_LAUNCH;
  }
  return NSA_OK;
}

}  // namespace
}  // namespace nsa

extern "C" int nsa_qk_norm_rope(const void* Q, const void* K, void* Qo, void* Ko, const void* wq,
                                const void* wk, const float* cos_table, const float* sin_table,
                                const int32_t* positions, int64_t B, int64_t M, int64_t H,
                                int64_t G, int64_t D, int64_t R, int64_t table_rows,
                                int64_t positions_stride, float eps, int interleaved, int dtype,
                                int weight_dtype, const int64_t* strides, void* stream) {
  using namespace nsa;
  int rc = check_rope(B, M, H, G, D, R, table_rows, positions_stride, eps, dtype, weight_dtype);
  if (rc != NSA_OK) return rc;
  const int64_t heads[4] = {H, G, H, G};
  int64_t s[12];
  if ((rc = take_strides(strides, 4, heads, B, M, D, s)) != NSA_OK) return rc;
  if (B == 0 || M == 0) return NSA_OK;
  if (!Q || !K || !Qo || !Ko) return NSA_ERR_NULL;
  if (!aligned(Q, 16) || !aligned(K, 16) || !aligned(Qo, 16) || !aligned(Ko, 16) ||
      !aligned(wq, 16) || !aligned(wk, 16))
    return NSA_ERR_ALIGN;
  if ((rc = check_tables(cos_table, sin_table, positions, M, R, table_rows)) != NSA_OK) return rc;
  RopeProblem p{};
  p.q = {static_cast<const uint8_t*>(Q), static_cast<uint8_t*>(Qo), wq, s[0], s[1], s[2], s[6], s[7],
         s[8], static_cast<int>(H)};
  p.k = {static_cast<const uint8_t*>(K), static_cast<uint8_t*>(Ko), wk, s[3], s[4], s[5], s[9],
         s[10], s[11], static_cast<int>(G)};
  p.cos_t = cos_table;
  p.sin_t = sin_table;
  p.pos = positions;
  p.pos_b = positions_stride;
  p.table_rows = table_rows;
  p.B = static_cast<int>(B);
  p.M = static_cast<int>(M);
  p.half = static_cast<int>(R / 2);
  p.interleaved = interleaved != 0;
  p.w32 = weight_dtype == NSA_F32;
  p.eps = eps;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf = dtype == NSA_BF16;
  if (D == 64) return bf ? launch_norm_rope<64, true>(p, st) : launch_norm_rope<64, false>(p, st);
  return bf ? launch_norm_rope<128, true>(p, st) : launch_norm_rope<128, false>(p, st);
}

extern "C" int64_t nsa_qk_norm_rope_bwd_workspace_bytes(int64_t B, int64_t M, int64_t D) {
  using namespace nsa;
  const int rc = check_rope(B, M, 1, 1, D, 0, 0, 0, 0.f, NSA_F16, NSA_F32);
  if (rc != NSA_OK) return rc;
  return static_cast<int64_t>(rope_bwd_most_ctas(B, M)) * D * 4;
}

extern "C" int nsa_qk_norm_rope_bwd(
    const void* Q, const void* K, const void* dQo, const void* dKo, void* dQ, void* dK, float* dwq,
    float* dwk, const void* wq, const void* wk, const float* cos_table, const float* sin_table,
    const int32_t* positions, int64_t B, int64_t M, int64_t H, int64_t G, int64_t D, int64_t R,
    int64_t table_rows, int64_t positions_stride, float eps, int interleaved, int dtype,
    int weight_dtype, int grad_dtype, const int64_t* strides, void* workspace,
    int64_t workspace_bytes, void* stream) {
  using namespace nsa;
  int rc = check_rope(B, M, H, G, D, R, table_rows, positions_stride, eps, dtype, weight_dtype);
  if (rc != NSA_OK) return rc;
  if (grad_dtype != NSA_F32 && grad_dtype != dtype) return NSA_ERR_DTYPE;
  const int64_t heads[6] = {H, G, H, G, H, G};
  int64_t s[18];
  if ((rc = take_strides(strides, 6, heads, B, M, D, s)) != NSA_OK) return rc;
  if (!aligned(dwq, 4) || !aligned(dwk, 4)) return NSA_ERR_ALIGN;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (B == 0 || M == 0) {  // no token: the weights' gradients are zero
    if (dwq && cudaMemsetAsync(dwq, 0, D * 4, st) != cudaSuccess) return NSA_ERR_LAUNCH;
    if (dwk && cudaMemsetAsync(dwk, 0, D * 4, st) != cudaSuccess) return NSA_ERR_LAUNCH;
    return NSA_OK;
  }
  if (!Q || !K || !dQo || !dKo || !dQ || !dK) return NSA_ERR_NULL;
  if (!aligned(Q, 16) || !aligned(K, 16) || !aligned(dQo, 16) || !aligned(dKo, 16) ||
      !aligned(dQ, 16) || !aligned(dK, 16) || !aligned(wq, 16) || !aligned(wk, 16))
    return NSA_ERR_ALIGN;
  if ((rc = check_tables(cos_table, sin_table, positions, M, R, table_rows)) != NSA_OK) return rc;
  const bool want_dw = dwq != nullptr || dwk != nullptr;
  if (want_dw) {
    if (!workspace || workspace_bytes < nsa_qk_norm_rope_bwd_workspace_bytes(B, M, D))
      return NSA_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return NSA_ERR_ALIGN;
  }
  RopeBwdProblem p{};
  p.a.cos_t = cos_table;
  p.a.sin_t = sin_table;
  p.a.pos = positions;
  p.a.pos_b = positions_stride;
  p.a.table_rows = table_rows;
  p.a.B = static_cast<int>(B);
  p.a.M = static_cast<int>(M);
  p.a.half = static_cast<int>(R / 2);
  p.a.interleaved = interleaved != 0;
  p.a.w32 = weight_dtype == NSA_F32;
  p.a.eps = eps;
  p.q = {static_cast<const uint8_t*>(Q), static_cast<const uint8_t*>(dQo), static_cast<uint8_t*>(dQ),
         wq, s[0], s[1], s[2], s[6], s[7], s[8], s[12], s[13], s[14],
         static_cast<int>(H)};
  p.k = {static_cast<const uint8_t*>(K), static_cast<const uint8_t*>(dKo), static_cast<uint8_t*>(dK),
         wk, s[3], s[4], s[5], s[9], s[10], s[11], s[15], s[16], s[17],
         static_cast<int>(G)};
  p.part = want_dw ? static_cast<float*>(workspace) : nullptr;
  const bool bf = dtype == NSA_BF16, g32 = grad_dtype == NSA_F32;
  if (D == 64) {
    if (bf)
      return g32 ? launch_norm_rope_bwd<64, true, true>(p, dwq, dwk, st)
                 : launch_norm_rope_bwd<64, true, false>(p, dwq, dwk, st);
    return g32 ? launch_norm_rope_bwd<64, false, true>(p, dwq, dwk, st)
               : launch_norm_rope_bwd<64, false, false>(p, dwq, dwk, st);
  }
  if (bf)
    return g32 ? launch_norm_rope_bwd<128, true, true>(p, dwq, dwk, st)
               : launch_norm_rope_bwd<128, true, false>(p, dwq, dwk, st);
  return g32 ? launch_norm_rope_bwd<128, false, true>(p, dwq, dwk, st)
             : launch_norm_rope_bwd<128, false, false>(p, dwq, dwk, st);
}
