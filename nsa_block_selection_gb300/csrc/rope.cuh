// Pieces of the norm-and-rotation kernels that also serve the cache's append:
// how lanes hold a head's row, its weights and angles, the turn, and the host
// checks of their arguments.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "common.cuh"
#include "nsa_sel_attn.h"
#include "ptx.cuh"

namespace nsa {
namespace {

// Kernels with FULL are for R = D: where a lane's chunks lie is known to the compiler.
struct RopeRows {
  const uint8_t* x;  // one of Q, K: element strides over (b, m, h)
  uint8_t* y;
  const void* w;
  int64_t xb, xm, xh, yb, ym, yh;
  int heads;
};

struct RopeProblem {
  RopeRows q, k;
  const float* cos_t;
  const float* sin_t;
  const int32_t* pos;
  int64_t pos_b, table_rows;
  int B, M, half;  // half = R / 2
  bool interleaved, w32;
  float eps;
};

// The two chunks of 8 entries that lane t of a row holds.
__device__ __forceinline__ void row_chunks(int t, int half, int& c0, int& c1) {
  const int pc = half >> 3;  // chunks of a half
  if (t < pc) {
    c0 = t;
    c1 = t + pc;
  } else {
    c0 = 2 * t;  // 2 pc + 2 (t - pc)
    c1 = 2 * t + 1;
  }
}

template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
  if constexpr (BF16) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  } else {
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
  }
}

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& v, float* f) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = unpack2<BF16>(u[i]);
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(pack2_t<BF16>(f[0], f[1]), pack2_t<BF16>(f[2], f[3]),
                    pack2_t<BF16>(f[4], f[5]), pack2_t<BF16>(f[6], f[7]));
}

__device__ __forceinline__ void load8(const float* p, float* f) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  const float4 b = *reinterpret_cast<const float4*>(p + 4);
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
  f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}

// The 16 weights of this lane's chunks (1 without a weight).
template <bool BF16>
__device__ __forceinline__ void load_weights(const void* w, bool w32, int c0, int c1, float* f) {
  if (w == nullptr) {
#pragma unroll
    for (int i = 0; i < 16; ++i) f[i] = 1.f;
  } else if (w32) {
    load8(static_cast<const float*>(w) + 8 * c0, f);
    load8(static_cast<const float*>(w) + 8 * c1, f + 8);
  } else {
    const uint4* p = static_cast<const uint4*>(w);
    unpack8<BF16>(p[c0], f);
    unpack8<BF16>(p[c1], f + 8);
  }
}

// The 8 angles of the lane's 8 pairs. Halves: pair j is entries j of the two
// chunks. Interleaved: pairs 0..3 are the entries (2j, 2j + 1) of the first
// chunk, 4..7 those of the second.
__device__ __forceinline__ void load_angles(const RopeProblem& p, int64_t at, int half, int c0,
                                            int c1, float* c, float* s) {
  const float* ct = p.cos_t + at * half;
  const float* st = p.sin_t + at * half;
  if (p.interleaved) {
    const float4 a = *reinterpret_cast<const float4*>(ct + 4 * c0);
    const float4 b = *reinterpret_cast<const float4*>(ct + 4 * c1);
    const float4 d = *reinterpret_cast<const float4*>(st + 4 * c0);
    const float4 e = *reinterpret_cast<const float4*>(st + 4 * c1);
    c[0] = a.x, c[1] = a.y, c[2] = a.z, c[3] = a.w, c[4] = b.x, c[5] = b.y, c[6] = b.z, c[7] = b.w;
    s[0] = d.x, s[1] = d.y, s[2] = d.z, s[3] = d.w, s[4] = e.x, s[5] = e.y, s[6] = e.z, s[7] = e.w;
  } else {
    load8(ct + 8 * c0, c);
    load8(st + 8 * c0, s);
  }
}

// Two fp32 operations an instruction.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// The turn of the lane's 8 pairs: (a, b) -> (a c - b s, b c + a s), every operation
// rounded by itself.
__device__ __forceinline__ void turn(float* f, const float* c, const float* s, bool interleaved) {
  if (interleaved) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float a = f[2 * j], b = f[2 * j + 1];
      f[2 * j] = __fsub_rn(__fmul_rn(a, c[j]), __fmul_rn(b, s[j]));
      f[2 * j + 1] = __fadd_rn(__fmul_rn(b, c[j]), __fmul_rn(a, s[j]));
    }
  } else {
    // (products two at a time, sums one: sums of pairs were fused with the products)
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const uint64_t a = pair(f[j], f[j + 1]), b = pair(f[j + 8], f[j + 9]);
      const uint64_t cc = pair(c[j], c[j + 1]), ss = pair(s[j], s[j + 1]);
      const float2 ac = unpair(mul2(a, cc)), bs = unpair(mul2(b, ss));
      const float2 bc = unpair(mul2(b, cc)), as = unpair(mul2(a, ss));
      f[j] = __fsub_rn(ac.x, bs.x), f[j + 1] = __fsub_rn(ac.y, bs.y);
      f[j + 8] = __fadd_rn(bc.x, as.x), f[j + 9] = __fadd_rn(bc.y, as.y);
    }
  }
}

// (f r) w, two at a time.
__device__ __forceinline__ void scale_row(float* f, float r, const float* w) {
  const uint64_t rr = pair(r, r);
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    const float2 x = unpair(mul2(mul2(pair(f[i], f[i + 1]), rr), pair(w[i], w[i + 1])));
    f[i] = x.x, f[i + 1] = x.y;
  }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// The sum of a row's squares (exact in fp32 one by one) in a fixed order that does
// not depend on how lanes hold the row: entries 32 apart first, one after the other,
// then neighbours, pairs, pairs of pairs and so on. Lane t of a row begins with the
// sums of N entries from 8 t (D = 64) or 8 (t % 4) + 4 (t / 4) on: where all of a row
// is turned (FULL) its chunks hold them, or (D = 128) its chunks and those of lane
// t ^ 4; else it loads them from x again (cached). `have`: the slot holds a row.
template <int D, bool BF16, bool FULL>
__device__ __forceinline__ float row_squares(const uint4& v0, const uint4& v1, const uint8_t* x,
                                             bool have) {
  constexpr int N = 512 / D, K = D / 32;
  const int t = (threadIdx.x & 31) % (D / 16);
  uint32_t w[K][N / 2];  // entry pairs, of each of the row's 32s
  if constexpr (D == 64) {
    uint4 a = v0, b = v1;
    if (!FULL && have) {
      a = reinterpret_cast<const uint4*>(x)[t];
      b = reinterpret_cast<const uint4*>(x)[t + 4];
    }
    w[0][0] = a.x, w[0][1] = a.y, w[0][2] = a.z, w[0][3] = a.w;
    w[1][0] = b.x, w[1][1] = b.y, w[1][2] = b.z, w[1][3] = b.w;
  } else if constexpr (FULL) {
    // (k = 0 and 1 may change places: they are added to one another first)
    const bool up = (t & 4) != 0;
    const uint32_t own[4] = {up ? v0.z : v0.x, up ? v0.w : v0.y, up ? v1.z : v1.x,
                             up ? v1.w : v1.y};
    const uint32_t give[4] = {up ? v0.x : v0.z, up ? v0.y : v0.w, up ? v1.x : v1.z,
                              up ? v1.y : v1.w};
    uint32_t got[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) got[i] = __shfl_xor_sync(kFull, give[i], 4);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      w[0][i] = own[i], w[1][i] = got[i];
      w[2][i] = up ? got[2 + i] : own[2 + i];
      w[3][i] = up ? own[2 + i] : got[2 + i];
    }
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const uint2 a = have ? reinterpret_cast<const uint2*>(x)[8 * k + 2 * (t & 3) + (t >> 2)]
                           : make_uint2(0, 0);
      w[k][0] = a.x, w[k][1] = a.y;
    }
  }
  uint64_t a[N / 2];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const float2 p = unpack2<BF16>(w[k][i]);
      const uint64_t z = pair(p.x, p.y);
      a[i] = k == 0 ? mul2(z, z) : fma2(z, z, a[i]);
    }
  float b[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const float2 p = unpair(a[i]);
    b[i] = __fadd_rn(p.x, p.y);
  }
#pragma unroll
  for (int n = N / 4; n > 0; n >>= 1)
#pragma unroll
    for (int i = 0; i < n; ++i) b[i] = __fadd_rn(b[2 * i], b[2 * i + 1]);
  if constexpr (D == 128) b[0] = __fadd_rn(b[0], __shfl_xor_sync(kFull, b[0], 4));
  b[0] = __fadd_rn(b[0], __shfl_xor_sync(kFull, b[0], 1));
  return __fadd_rn(b[0], __shfl_xor_sync(kFull, b[0], 2));
}

// A token's position, or -1 for padding (outside the table).
__device__ __forceinline__ int64_t token_position(const RopeProblem& p, int b, int m) {
  int64_t at = m;
  if (p.pos != nullptr) at = p.pos[b * p.pos_b + m];
  if (at < 0 || (p.half > 0 && at >= p.table_rows)) return -1;
  return at;
}

// Rows [r0, r1) of one token's heads, UN groups of rows in flight per warp. FIRST: the
// sums of them all before the first is stored, so that no row's loads wait for
// another's stores (65,536 tokens of 64 + 8 heads of 128: the append 404 us with and
// 412 without; the norm alone, whose registers it takes, 366 and 360).
template <int D, bool BF16, bool FULL, bool FIRST, int UN>
__device__ __forceinline__ void norm_rope_rows(const RopeProblem& p, const RopeRows& t, int b, int m,
                                               int r0, int r1, bool live, bool rot, int c0, int c1,
                                               const float* c, const float* s, bool norm = true) {
  constexpr int LPR = D / 16, RPW = 32 / LPR;
  const int sub = (threadIdx.x & 31) / LPR;
  const uint8_t* x = t.x + 2 * (b * t.xb + m * t.xm);
  uint8_t* y = t.y + 2 * (b * t.yb + m * t.ym);
  float w[16];
  if (live) load_weights<BF16>(t.w, p.w32, c0, c1, w);
  for (int r = r0; r < r1; r += RPW * UN) {
    uint4 v[UN][2];
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int row = r + u * RPW + sub;
      v[u][0] = v[u][1] = make_uint4(0, 0, 0, 0);
      if (live && row < r1) {
        const uint4* src = reinterpret_cast<const uint4*>(x + 2 * row * t.xh);
        v[u][0] = src[c0];
        v[u][1] = src[c1];
      }
    }
    float sq[UN];
    auto squares = [&](int u) {
      const int row = r + u * RPW + sub;
      sq[u] = row_squares<D, BF16, FULL>(v[u][0], v[u][1], x + 2 * row * t.xh, live && row < r1);
    };
    if (FIRST && norm) {
#pragma unroll
      for (int u = 0; u < UN; ++u) squares(u);
    }
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int row = r + u * RPW + sub;
      if (!FIRST && norm) squares(u);
      float f[16];
      unpack8<BF16>(v[u][0], f);
      unpack8<BF16>(v[u][1], f + 8);
      // (a padding token's rows are zero)
      if (norm && live) scale_row(f, rsqrtf(sq[u] * (1.f / D) + p.eps), w);
      if (live && rot) turn(f, c, s, p.interleaved);
      if (row < r1) {
        uint4* dst = reinterpret_cast<uint4*>(y + 2 * row * t.yh);
        dst[c0] = pack8<BF16>(f);
        dst[c1] = pack8<BF16>(f + 8);
      }
    }
  }
}

// How a warp's row slots map to (token, head) where a token has few heads: one
// token to a group of slots, or several, with the heads rounded up to a power
// of two; more heads than slots take several groups.
struct RowGroups {
  int per_token;  // groups of a token (1 where tokens share a group)
  int shift;      // log2 of the slots of a token, where tokens share a group
  int64_t groups;
};

// ---- host ---------------------------------------------------------------

inline bool aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

inline int check_rope(int64_t B, int64_t M, int64_t H, int64_t G, int64_t D, int64_t R,
                      int64_t table_rows, int64_t positions_stride, float eps, int dtype,
                      int weight_dtype) {
  if (B < 0 || M < 0 || H <= 0 || G <= 0) return NSA_ERR_SHAPE;
  if (D != 64 && D != 128) return NSA_ERR_HEAD_DIM;
  if (R < 0 || R > D || R % 16 != 0) return NSA_ERR_SHAPE;
  if (table_rows < 0 || table_rows > (int64_t(1) << 31) || positions_stride < 0)
    return NSA_ERR_SHAPE;
  if (!(eps >= 0.f) || std::isinf(eps)) return NSA_ERR_SHAPE;
  const int64_t lim = int64_t(1) << 30;
  if (B > lim || M > lim || H > 65536 || G > 65536) return NSA_ERR_SHAPE;
  if (B * M >= (int64_t(1) << 31)) return NSA_ERR_SHAPE;
  if (dtype != NSA_F16 && dtype != NSA_BF16) return NSA_ERR_DTYPE;
  if (weight_dtype != NSA_F32 && weight_dtype != dtype) return NSA_ERR_DTYPE;
  return NSA_OK;
}

// n groups of 3 element strides; NULL: contiguous rows of D. The last
// `written` groups are written: a stride of 0 would put several rows in one place.
inline int take_strides(const int64_t* strides, int n, const int64_t* heads, int64_t B, int64_t M,
                        int64_t D, int64_t* out, int written = 2) {
  for (int i = 0; i < n; ++i) {
    if (strides == nullptr) {
      out[3 * i] = M * heads[i] * D;
      out[3 * i + 1] = heads[i] * D;
      out[3 * i + 2] = D;
    } else {
      for (int j = 0; j < 3; ++j) {
        const int64_t s = strides[3 * i + j];
        if (s < 0 || s > (int64_t(1) << 40)) return NSA_ERR_SHAPE;
        if (s % 8 != 0) return NSA_ERR_ALIGN;
        const int64_t extent = j == 0 ? B : j == 1 ? M : heads[i];
        if (i >= n - written && s == 0 && extent > 1) return NSA_ERR_SHAPE;
        out[3 * i + j] = s;
      }
    }
  }
  return NSA_OK;
}

inline int check_tables(const float* cos_t, const float* sin_t, const int32_t* positions, int64_t M,
                        int64_t R, int64_t table_rows) {
  if (R > 0) {
    if (table_rows > 0 && (!cos_t || !sin_t)) return NSA_ERR_NULL;
    if (!aligned(cos_t, 16) || !aligned(sin_t, 16)) return NSA_ERR_ALIGN;
    if (positions == nullptr && M > table_rows) return NSA_ERR_SHAPE;
  }
  return aligned(positions, 4) ? NSA_OK : NSA_ERR_ALIGN;
}

inline RowGroups plan_row_groups(int heads, int64_t tokens, int slots) {
  RowGroups g{1, 0, 0};
  if (heads > slots) {
    g.per_token = (heads + slots - 1) / slots;
    g.groups = tokens * g.per_token;
  } else {
    while ((1 << g.shift) < heads) ++g.shift;
    const int64_t shared = slots >> g.shift;  // tokens of a group
    g.groups = (tokens + shared - 1) / shared;
  }
  return g;
}

}  // namespace
}  // namespace nsa
