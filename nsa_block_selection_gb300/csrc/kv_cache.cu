// Appending new tokens to a paged cache of keys and values, with the norm of the
// query and key heads and the position rotation applied on the way, and reading
// rows of the cache back, for sm_103a.
//
// Append, per token at position p: Q and K rows become
//   y = turn_p(x rsqrt(mean(x^2) + eps) w),
// fp32, rounded once to the 16-bit type, in norm_rope.cu's order of operations; Q is
// written as a tensor, K and V as rows of the token's page. A 4-bit row is made of the 16-bit
// one: low = bf16(min), step = bf16((max - low) / 15),
// code = clamp(rint((x - low) / step), 0, 15), all divisions IEEE, so that the
// codes are the same wherever they are formed.
// Read: rows of given positions back as K and V tensors, fma(code, step, low)
// rounded once where the cache has 4 bits.
//
// The bytes bound both: every row is read once and written once. A row is held
// by D / 16 lanes, 16 entries each (append), which hold both entries of every
// pair, so that the turn needs no exchange; or by D / 8 lanes, 16 bytes of the
// result each (read). 16,384 tokens of 64 + 8 heads of 128 are appended in 109 us
// (680 MB, 6.2 TB/s), 65,536 tokens of 8 heads read from 4 bits in 57 us (340 MB,
// 6.0 TB/s); one token is 2.3 us on the device.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "common.cuh"
#include "kv_cache.cuh"
#include "nsa_sel_attn.h"
#include "ptx.cuh"
#include "rope.cuh"

namespace nsa {
namespace {

constexpr int kKvThreads = 128;
// CTAs of kv_append_kernel. (16 bits with 4: 4 x 2000 tokens of 16 + 2 heads of 64 12.0
// us instead of 11.1; 4 bits with 5 22.0, with 4 24.4, with 6 21.0, but 48 single tokens
// 4.3 us instead of 4.0.)
constexpr int kAppendPerSm = 6, kAppendPerSm4 = 5;
// Beyond so many groups of row slots a token, and in all, a warp takes a token. (16,384
// tokens of 64 + 8 heads: 109 us, by kv_append_kernel 142.)
constexpr int kAppendFewPerToken = 8;
constexpr int64_t kAppendFewGroups = 128 * 152;
constexpr int kKvSms = 152;

struct AppendProblem {
  RopeProblem r;  // q: Q and its result; k: K (its y is unused)
  const uint8_t* v;
  int64_t vb, vm, vh;  // element strides
  KvPages c;
  bool norm;
};

template <int LPR>
__device__ __forceinline__ float row_min(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v = fminf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}

// The 8 codes of a chunk, entry i in bits 4 i.
__device__ __forceinline__ uint32_t codes8(const float* f, float low, float step, bool live) {
  uint32_t w = 0;
  if (live) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q = rintf(__fdiv_rn(f[i] - low, step));
      w |= static_cast<uint32_t>(fminf(fmaxf(q, 0.f), 15.f)) << (4 * i);
    }
  }
  return w;
}

// The 16-bit row f (packed in v0, v1) as a 4-bit row of the cache. All lanes of the
// warp; `write`: this one's row has a place.
template <int D, bool BF16>
__device__ __forceinline__ void store_codes(const uint4& v0, const uint4& v1, int c0, int c1, int tl,
                                            uint8_t* row, uint32_t* scale, bool write) {
  constexpr int LPR = D / 16;
  float f[16];
  unpack8<BF16>(v0, f);
  unpack8<BF16>(v1, f + 8);
  float lo = f[0], hi = f[0], bad = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    lo = fminf(lo, f[i]);
    hi = fmaxf(hi, f[i]);
    bad = fmaf(f[i], 0.f, bad);  // NaN where an entry is not finite
  }
  lo = row_min<LPR>(lo);
  hi = -row_min<LPR>(-hi);
  bad = row_sum<LPR>(bad);
  const float low = __bfloat162float(__float2bfloat16_rn(lo));
  float step = __bfloat162float(__float2bfloat16_rn(__fdiv_rn(hi - low, 15.f)));
  const bool some = step >= kLeastStep;
  if (!some) step = 0.f;
  // a row that is not finite, or too wide for fp32, reads as NaN
  if (!(bad == 0.f) || !(hi - low < INFINITY)) step = __uint_as_float(0x7fc00000u);
  const bool fine = some && step < INFINITY;
  if (write) {
    uint32_t* const dst = reinterpret_cast<uint32_t*>(row);
    dst[c0] = codes8(f, low, step, fine);
    dst[c1] = codes8(f + 8, low, step, fine);
    if (tl == 0) *scale = pack_bf162(step, low);
  }
}

// K's or V's rows [r0, r1) of one token, UN groups of rows in flight per warp.
template <int D, bool BF16, bool Q4, bool FULL, bool V, int UN>
__device__ __forceinline__ void append_rows(const AppendProblem& p, const uint8_t* x, int64_t xh,
                                            int r0, int r1, int page, int off, bool rot, int c0,
                                            int c1, const float* c, const float* s) {
  constexpr int LPR = D / 16, RPW = 32 / LPR;
  const int sub = (threadIdx.x & 31) / LPR, tl = (threadIdx.x & 31) % LPR;
  uint8_t* const y = V ? p.c.v + page * p.c.vp + off * p.c.vt : p.c.k + page * p.c.kp + off * p.c.kt;
  const int64_t yh = V ? p.c.vh : p.c.kh;
  float w[16];
  if (!V && p.norm) load_weights<BF16>(p.r.k.w, p.r.w32, c0, c1, w);
  for (int r = r0; r < r1; r += RPW * UN) {
    uint4 v[UN][2];
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int row = r + u * RPW + sub;
      v[u][0] = v[u][1] = make_uint4(0, 0, 0, 0);
      if (row < r1) {
        const uint4* src = reinterpret_cast<const uint4*>(x + 2 * row * xh);
        v[u][0] = src[c0];
        v[u][1] = src[c1];
      }
    }
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int row = r + u * RPW + sub;
      if constexpr (!V) {
        float f[16], sq = 0.f;
        if (p.norm) sq = row_squares<D, BF16, FULL>(v[u][0], v[u][1], x + 2 * row * xh, row < r1);
        unpack8<BF16>(v[u][0], f);
        unpack8<BF16>(v[u][1], f + 8);
        if (p.norm) scale_row(f, rsqrtf(sq * (1.f / D) + p.r.eps), w);
        if (rot) turn(f, c, s, p.r.interleaved);
        v[u][0] = pack8<BF16>(f);
        v[u][1] = pack8<BF16>(f + 8);
      }
      if constexpr (Q4) {
        const int64_t so = ((page * static_cast<int64_t>(p.r.k.heads) + row) << p.c.shift) + off;
        store_codes<D, BF16>(v[u][0], v[u][1], c0, c1, tl, y + row * yh, (V ? p.c.vs : p.c.ks) + so,
                             row < r1);
      } else if (row < r1) {
        uint4* const dst = reinterpret_cast<uint4*>(y + row * yh);
        dst[c0] = v[u][0];
        dst[c1] = v[u][1];
      }
    }
  }
}

// Many heads: one warp per unit of `per` rows of the H + 2 G of a token (Q's, K's,
// V's), which share its position, page and angles, as norm_rope_kernel.
template <int D, bool BF16, bool Q4, bool FULL, int UN>
__global__ void __launch_bounds__(kKvThreads, FULL ? 5 : 4)
    kv_append_token_kernel(const AppendProblem p, int segs, int per, int64_t units) {
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kKvThreads / 32) + (threadIdx.x >> 5);
  if (unit >= units) return;
  const uint32_t tok = static_cast<uint32_t>(unit) / static_cast<uint32_t>(segs);
  const int seg = static_cast<int>(static_cast<uint32_t>(unit) - tok * segs);
  const int b = static_cast<int>(tok / static_cast<uint32_t>(p.r.M));
  const int m = static_cast<int>(tok - static_cast<uint32_t>(b) * p.r.M);
  const int64_t at = token_position(p.r, b, m);
  const bool live = at >= 0;
  const int H = p.r.q.heads, G = p.r.k.heads;
  int c0, c1;
  const int t = (threadIdx.x & 31) % (D / 16), half = FULL ? D / 2 : p.r.half;
  row_chunks(t, half, c0, c1);
  const bool rot = t < (half >> 3);
  float c[8], s[8];
  if (live && rot) load_angles(p.r, at, half, c0, c1, c, s);
  const int r0 = seg * per, r1 = min(r0 + per, H + 2 * G);
  const int page = live && r1 > H ? page_of(p.c, b, at) : -1;
  const int off = static_cast<int>(at) & ((1 << p.c.shift) - 1);
  if (r0 < H)
    norm_rope_rows<D, BF16, FULL, true, UN>(p.r, p.r.q, b, m, r0, min(r1, H), live, rot, c0, c1, c, s,
                                            p.norm);
  if (page < 0) return;
  if (r1 > H && r0 < H + G)
    append_rows<D, BF16, Q4, FULL, false, 2>(p, p.r.k.x + 2 * (b * p.r.k.xb + m * p.r.k.xm),
                                             p.r.k.xh, max(r0 - H, 0), min(r1 - H, G), page, off,
                                             rot, c0, c1, c, s);
  if (r1 > H + G)
    append_rows<D, BF16, Q4, FULL, true, 2>(p, p.v + 2 * (b * p.vb + m * p.vm), p.vh,
                                            max(r0 - H - G, 0), r1 - H - G, page, off, false, c0, c1,
                                            c, s);
}

// Few heads, or few tokens: a row slot of a warp keeps its head (of Q, K or V) and the
// head's weights, and walks the tokens, as in norm_rope_few_kernel.
template <int D, bool BF16, bool Q4, bool FULL>
__global__ void __launch_bounds__(kKvThreads, Q4 ? kAppendPerSm4 : kAppendPerSm)
    kv_append_kernel(const AppendProblem p, const RowGroups rg) {
  constexpr int LPR = D / 16, RPW = 32 / LPR;
  const int lane = threadIdx.x & 31, sub = lane / LPR, tl = lane % LPR;
  const uint32_t groups = static_cast<uint32_t>(rg.per_token);
  const uint32_t wid = blockIdx.x * (kKvThreads / 32) + (threadIdx.x >> 5);
  const uint32_t walks = gridDim.x * (kKvThreads / 32) / groups;
  const uint32_t first = wid / groups;
  if (first >= walks) return;
  const int wide = rg.per_token > 1 ? RPW : 1 << rg.shift;
  const uint32_t sets = static_cast<uint32_t>(RPW / wide);
  const int head = static_cast<int>(wid - first * groups) * RPW + (sub & (wide - 1));
  const int H = p.r.q.heads, G = p.r.k.heads;
  const bool slot = head < H + 2 * G, is_q = head < H, is_v = head >= H + G;
  const int64_t h = is_q ? head : is_v ? head - H - G : head - H;
  int c0, c1;
  const int half = FULL ? D / 2 : p.r.half;
  row_chunks(tl, half, c0, c1);
  const bool rot = tl < (half >> 3) && !is_v;
  float w[16];
  load_weights<BF16>(is_v ? nullptr : is_q ? p.r.q.w : p.r.k.w, p.r.w32, c0, c1, w);
  const uint8_t* x;
  int64_t xb, xm;
  if (is_v) {
    x = p.v + 2 * h * p.vh, xb = p.vb, xm = p.vm;
  } else {
    const RopeRows& t = is_q ? p.r.q : p.r.k;
    x = t.x + 2 * h * t.xh, xb = t.xb, xm = t.xm;
  }
  uint8_t* const y =
      is_q ? p.r.q.y + 2 * h * p.r.q.yh : is_v ? p.c.v + h * p.c.vh : p.c.k + h * p.c.kh;
  const uint64_t tokens = static_cast<uint64_t>(p.r.B) * p.r.M;
  // (all lanes of a warp go through the loop together: the row sums need them)
  for (uint64_t begin = static_cast<uint64_t>(first) * sets; begin < tokens;
       begin += static_cast<uint64_t>(walks) * sets) {
    const uint64_t tok = begin + static_cast<uint32_t>(sub / wide);
    bool write = slot && tok < tokens, live = false;
    int64_t yo = 0, so = 0;
    float f[16], c[8], s[8];
    uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0;
    const uint8_t* src = x;
    if (write) {
      const int b = static_cast<int>(static_cast<uint32_t>(tok) / static_cast<uint32_t>(p.r.M));
      const int m = static_cast<int>(static_cast<uint32_t>(tok) - static_cast<uint32_t>(b) * p.r.M);
      const int64_t at = token_position(p.r, b, m);
      live = at >= 0;
      if (is_q) {
        yo = 2 * (b * p.r.q.yb + m * p.r.q.ym);
      } else {  // a token without a page is not stored
        const int page = live ? page_of(p.c, b, at) : -1;
        const int64_t row = at & ((1 << p.c.shift) - 1);
        live = write = page >= 0;
        yo = is_v ? page * p.c.vp + row * p.c.vt : page * p.c.kp + row * p.c.kt;
        so = ((page * static_cast<int64_t>(G) + h) << p.c.shift) + row;
      }
      if (live) {  // (padding is not read)
        src += 2 * (b * xb + m * xm);
        v0 = reinterpret_cast<const uint4*>(src)[c0];
        v1 = reinterpret_cast<const uint4*>(src)[c1];
        if (rot) load_angles(p.r, at, half, c0, c1, c, s);
      }
    }
    float sq = 0.f;
    if (p.norm) sq = row_squares<D, BF16, FULL>(v0, v1, src, live);
    if (!is_v) {
      unpack8<BF16>(v0, f);
      unpack8<BF16>(v1, f + 8);
      if (live && p.norm) scale_row(f, rsqrtf(sq * (1.f / D) + p.r.eps), w);
      if (live && rot) turn(f, c, s, p.r.interleaved);
      v0 = pack8<BF16>(f);
      v1 = pack8<BF16>(f + 8);
    }
    if constexpr (Q4) {
      // (a warp of query rows alone passes)
      if (__any_sync(kFull, write && !is_q))
        store_codes<D, BF16>(v0, v1, c0, c1, tl, y + yo, (is_v ? p.c.vs : p.c.ks) + so,
                             write && !is_q);
      write = write && is_q;
    }
    if (write) {
      uint4* const dst = reinterpret_cast<uint4*>(y + yo);
      dst[c0] = v0;
      dst[c1] = v1;
    }
  }
}

struct ReadProblem {
  KvPages c;
  const int32_t* pos;
  uint8_t *k, *v;  // [B, M, G, D]
  int64_t pos_b;
  int M, G;
  uint32_t tokens;
};

// 8 entries of a 4-bit row.
template <bool BF16>
__device__ __forceinline__ uint4 from_codes(uint32_t w, uint32_t scale) {
  const float step = __uint_as_float(scale << 16), low = __uint_as_float(scale & 0xffff0000u);
  float f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = fmaf(static_cast<float>((w >> (4 * i)) & 15u), step, low);
  return pack8<BF16>(f);
}

// A group of `lanes` lanes takes a token, whose position and page it looks up once,
// and then four chunks of 8 entries of K and of V a lane at a time. (A chunk a
// thread, each looking up its own, left too little in flight: 65,536 tokens of 8
// heads from 4 bits 77 us; four chunks of four tokens a thread 70.)
constexpr int kReadChunks = 4;

template <int D, bool BF16, bool Q4>
__global__ void __launch_bounds__(256) kv_read_kernel(const ReadProblem p, int lanes) {
  // (under 2^31 tokens, in 32-bit numbers of CTAs and 64-bit ones of threads)
  const uint32_t tok = static_cast<uint32_t>(
      (static_cast<uint64_t>(blockIdx.x) * 256u + threadIdx.x) / static_cast<uint32_t>(lanes));
  if (tok >= p.tokens) return;
  const int b = static_cast<int>(tok / static_cast<uint32_t>(p.M));
  const int m = static_cast<int>(tok - static_cast<uint32_t>(b) * p.M);
  const int at = __ldg(p.pos + b * p.pos_b + m);
  const int page = at >= 0 ? page_of(p.c, b, at) : -1;
  const int off = at & ((1 << p.c.shift) - 1);
  const uint8_t* const ks = p.c.k + page * p.c.kp + off * p.c.kt;
  const uint8_t* const vs = p.c.v + page * p.c.vp + off * p.c.vt;
  const int64_t so = ((page * static_cast<int64_t>(p.G)) << p.c.shift) + off;
  const int chunks = p.G * (D / 8);
  const int64_t out = static_cast<int64_t>(tok) * chunks;
  for (int i0 = static_cast<int>(threadIdx.x) & (lanes - 1); i0 < chunks; i0 += kReadChunks * lanes) {
    uint4 k[kReadChunks], v[kReadChunks];  // 4 bits: a word of codes and the scale
#pragma unroll
    for (int u = 0; u < kReadChunks; ++u) {
      const int i = i0 + u * lanes, g = i / (D / 8), t = i % (D / 8);
      k[u] = v[u] = make_uint4(0, 0, 0, 0);
      if (page >= 0 && i < chunks) {
        if constexpr (Q4) {
          k[u].x = reinterpret_cast<const uint32_t*>(ks + g * p.c.kh)[t];
          v[u].x = reinterpret_cast<const uint32_t*>(vs + g * p.c.vh)[t];
          const int64_t s = so + (static_cast<int64_t>(g) << p.c.shift);
          k[u].y = p.c.ks[s];
          v[u].y = p.c.vs[s];
        } else {
          k[u] = reinterpret_cast<const uint4*>(ks + g * p.c.kh)[t];
          v[u] = reinterpret_cast<const uint4*>(vs + g * p.c.vh)[t];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kReadChunks; ++u) {
      const int i = i0 + u * lanes;
      if (i < chunks) {
        // (no page: codes and scales of 0 are zeros)
        reinterpret_cast<uint4*>(p.k)[out + i] = Q4 ? from_codes<BF16>(k[u].x, k[u].y) : k[u];
        reinterpret_cast<uint4*>(p.v)[out + i] = Q4 ? from_codes<BF16>(v[u].x, v[u].y) : v[u];
      }
    }
  }
}

template <int D, bool BF16, bool Q4, bool FULL>
int launch_append_full(const AppendProblem& p, cudaStream_t st) {
  constexpr int RPW = 32 / (D / 16);
  constexpr int64_t kWarps = kKvThreads / 32;
  const int64_t tokens = static_cast<int64_t>(p.r.B) * p.r.M;
  const RowGroups g = plan_row_groups(p.r.q.heads + 2 * p.r.k.heads, tokens, RPW);
  const int rows = p.r.q.heads + 2 * p.r.k.heads;
  if (rows > kAppendFewPerToken * RPW && g.groups > kAppendFewGroups) {
    // as launch_norm_rope: a whole token a warp, or as few rows as give every SM 16 warps
    int64_t segs = (16 * kKvSms + tokens - 1) / tokens;
    const int64_t most = (rows + RPW - 1) / RPW;
    if (segs > most) segs = most;
    int64_t per = (rows + segs - 1) / segs;
    per = (per + RPW - 1) / RPW * RPW;
    segs = (rows + per - 1) / per;
    const int64_t units = tokens * segs;
    kv_append_token_kernel<D, BF16, Q4, FULL, 4>
        <<<static_cast<unsigned>((units + kWarps - 1) / kWarps), kKvThreads, 0, st>>>(
            p, static_cast<int>(segs), static_cast<int>(per), units);
    return cudaGetLastError() == cudaSuccess ? NSA_OK : NSA_ERR_LAUNCH;
  }
  int64_t warps = g.groups;
  constexpr int64_t kMost = (Q4 ? kAppendPerSm4 : kAppendPerSm) * kKvSms * kWarps;
  if (warps > kMost) warps = kMost;
  if (warps < g.per_token) warps = g.per_token;
  kv_append_kernel<D, BF16, Q4, FULL>
      <<<static_cast<unsigned>((warps + kWarps - 1) / kWarps), kKvThreads, 0, st>>>(p, g);
  return cudaGetLastError() == cudaSuccess ? NSA_OK : NSA_ERR_LAUNCH;
}

template <int D, bool BF16, bool Q4>
int launch_append(const AppendProblem& p, cudaStream_t st) {
  return 2 * p.r.half == D ? launch_append_full<D, BF16, Q4, true>(p, st)
                           : launch_append_full<D, BF16, Q4, false>(p, st);
}

template <int D, bool BF16>
int launch_read(const ReadProblem& p, bool q4, cudaStream_t st) {
  int lanes = 32;  // a token's chunks, or a warp
  while (lanes / 2 >= p.G * (D / 8)) lanes /= 2;
  const unsigned blocks =
      static_cast<unsigned>((static_cast<int64_t>(p.tokens) * lanes + 255) / 256);
  if (q4)
    kv_read_kernel<D, BF16, true><<<blocks, 256, 0, st>>>(p, lanes);
  else
    kv_read_kernel<D, BF16, false><<<blocks, 256, 0, st>>>(p, lanes);
  return cudaGetLastError() == cudaSuccess ? NSA_OK : NSA_ERR_LAUNCH;
}

}  // namespace
}  // namespace nsa

extern "C" int nsa_kv_append(const void* Q, const void* K, const void* V, void* Qo,
                             const nsa_kv_cache* cache, const int32_t* page_table, const void* wq,
                             const void* wk, const float* cos_table, const float* sin_table,
                             const int32_t* positions, int64_t B, int64_t M, int64_t H, int64_t G,
                             int64_t D, int64_t R, int64_t table_rows, int64_t positions_stride,
                             int64_t table_cols, float eps, int interleaved, int dtype,
                             int weight_dtype, const int64_t* strides, void* stream) {
  using namespace nsa;
  const bool norm = !(eps < 0.f);
  // (H = 0: keys and values alone)
  int rc = check_rope(B, M, H == 0 ? 1 : H, G, D, R, table_rows, positions_stride,
                      norm ? eps : 0.f, dtype, weight_dtype);
  if (rc != NSA_OK) return rc;
  const int64_t heads[4] = {G, G, H, H};  // K, V and Q are read, the last is written
  int64_t s[12] = {};
  // (without queries neither of the last two is looked at)
  if ((rc = take_strides(strides, H > 0 ? 4 : 2, heads, B, M, D, s, H > 0)) != NSA_OK) return rc;
  if (B == 0 || M == 0) return NSA_OK;
  if (!K || !V || (H > 0 && (!Q || !Qo))) return NSA_ERR_NULL;
  if (!norm && (wq || wk)) return NSA_ERR_SHAPE;
  if (!aligned(Q, 16) || !aligned(K, 16) || !aligned(V, 16) || !aligned(Qo, 16) ||
      !aligned(wq, 16) || !aligned(wk, 16))
    return NSA_ERR_ALIGN;
  if ((rc = check_tables(cos_table, sin_table, positions, M, R, table_rows)) != NSA_OK) return rc;
  AppendProblem p{};
  if ((rc = take_cache(cache, page_table, table_cols, B, G, D, true, &p.c)) != NSA_OK) return rc;
  p.r.k = {static_cast<const uint8_t*>(K), nullptr, wk, s[0], s[1], s[2], 0, 0, 0,
           static_cast<int>(G)};
  p.v = static_cast<const uint8_t*>(V);
  p.vb = s[3], p.vm = s[4], p.vh = s[5];
  p.r.q = {static_cast<const uint8_t*>(Q), static_cast<uint8_t*>(Qo), wq, s[6], s[7], s[8], s[9],
           s[10], s[11], static_cast<int>(H)};
  p.r.cos_t = cos_table;
  p.r.sin_t = sin_table;
  p.r.pos = positions;
  p.r.pos_b = positions_stride;
  p.r.table_rows = table_rows;
  p.r.B = static_cast<int>(B);
  p.r.M = static_cast<int>(M);
  p.r.half = static_cast<int>(R / 2);
  p.r.interleaved = interleaved != 0;
  p.r.w32 = weight_dtype == NSA_F32;
  p.r.eps = eps;
  p.norm = norm;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf = dtype == NSA_BF16, q4 = cache->bits == 4;
  if (D == 64) {
    if (bf) return q4 ? launch_append<64, true, true>(p, st) : launch_append<64, true, false>(p, st);
    return q4 ? launch_append<64, false, true>(p, st) : launch_append<64, false, false>(p, st);
  }
  if (bf) return q4 ? launch_append<128, true, true>(p, st) : launch_append<128, true, false>(p, st);
  return q4 ? launch_append<128, false, true>(p, st) : launch_append<128, false, false>(p, st);
}

extern "C" int nsa_kv_read(const nsa_kv_cache* cache, const int32_t* page_table,
                           const int32_t* positions, void* K, void* V, int64_t B, int64_t M,
                           int64_t G, int64_t D, int64_t positions_stride, int64_t table_cols,
                           int dtype, void* stream) {
  using namespace nsa;
  int rc = check_rope(B, M, 1, G, D, 0, 0, positions_stride, 0.f, dtype, NSA_F32);
  if (rc != NSA_OK) return rc;
  if (B * M * G > (int64_t(1) << 34)) return NSA_ERR_SHAPE;
  if (B == 0 || M == 0) return NSA_OK;
  if (!K || !V || !positions) return NSA_ERR_NULL;
  if (!aligned(K, 16) || !aligned(V, 16) || !aligned(positions, 4)) return NSA_ERR_ALIGN;
  ReadProblem p{};
  if ((rc = take_cache(cache, page_table, table_cols, B, G, D, false, &p.c)) != NSA_OK) return rc;
  p.pos = positions;
  p.pos_b = positions_stride;
  p.k = static_cast<uint8_t*>(K);
  p.v = static_cast<uint8_t*>(V);
  p.M = static_cast<int>(M);
  p.G = static_cast<int>(G);
  p.tokens = static_cast<uint32_t>(B * M);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf = dtype == NSA_BF16, q4 = cache->bits == 4;
  if (D == 64) return bf ? launch_read<64, true>(p, q4, st) : launch_read<64, false>(p, q4, st);
  return bf ? launch_read<128, true>(p, q4, st) : launch_read<128, false>(p, q4, st);
}
