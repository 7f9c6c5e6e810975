/*
 * nsa_sel_attn.h -- C ABI of the NSA selection-attention forward library
 * (libnsa_sel_attn.so, sm_103a).
 *
 * The operation is the one stated in "[wave] NSA: selection attention forward
 * kernel":
 *   section "Operation"    -- Q [B,M,H,D], K [B,N,G,D], V [B,N,G,D],
 *                             block_indices [B,M,G,T] in; O_slc [B,M,H,D],
 *                             LSE_slc [B,H,M] out; T = selected blocks/query;
 *   section "Algorithm"    -- for query m and each selected block t, the keys
 *                             [t*block_size, (t+1)*block_size) are gathered,
 *                             scored against q[m] (QK^T), causally masked and
 *                             softmaxed; V is accumulated with an online
 *                             softmax (running max + log-sum-exp); O and LSE
 *                             are stored;
 *   section "Requirements" -- the heads of a GQA group share block_indices;
 *                             online softmax across all T blocks; causal mask
 *                             inside gathered blocks; FP16 matmuls with FP32
 *                             accumulation; LSE returned for the backward
 *                             pass; block_size 64 and 32.
 *
 * Conventions where the pages are silent (the library's contract):
 *   - head h belongs to KV group h / (H/G) (contiguous heads per group);
 *   - key n is visible to query m iff n <= m and n < N;
 *   - scores are multiplied by `scale` (pass <= 0 for 1/sqrt(D));
 *   - block_indices entries < 0 or >= ceil(N/block_size) are padding and may
 *     sit anywhere in a row; a row must not list a block twice (a top-k
 *     output never does; a repeated block is counted twice);
 *   - a row with no visible key yields O = 0 and LSE = -inf;
 *   - LSE is the natural log of sum(exp(scale * q.k)) over visible keys.
 *
 * Every buffer is contiguous row-major in the layout given, owned by the
 * caller, and not retained after the call returns. Key/value rows that no
 * index selects are never read; rows after a query inside its own 16-key
 * tile may be read but never reach the output (whatever they hold).
 */
#ifndef NSA_SEL_ATTN_H
#define NSA_SEL_ATTN_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes. Values < 0 are errors; nothing was launched when an argument
 * check fails. */
typedef enum nsa_status {
  NSA_OK = 0,
  NSA_ERR_NULL = -1,        /* a required pointer is NULL                     */
  NSA_ERR_SHAPE = -2,       /* a size is negative or the sizes are too large */
  NSA_ERR_BLOCK_SIZE = -3,  /* block_size not in {32, 64}                     */
  NSA_ERR_HEAD_DIM = -4,    /* D not in {64, 128}                             */
  NSA_ERR_GROUPS = -5,      /* H % G != 0, or H/G > 8 and not a multiple of 8 */
  NSA_ERR_ALIGN = -6,       /* Q, K, V or O not 16-byte aligned, LSE or
                               block_indices not 4-byte aligned               */
  NSA_ERR_LAUNCH = -7,      /* the CUDA runtime refused the launch or a copy
                               (no device, no sm_103a image, bad stream ...) */
  NSA_ERR_TIMEOUT = -8,     /* a bounded device-side wait gave up (reported by
                               nsa_sync_status)                               */
  NSA_ERR_WORKSPACE = -9,   /* workspace NULL or smaller than required        */
  NSA_ERR_SCRATCH = -10,    /* problem needs more scratch than the fixed
                               buffer of nsa_sel_attn_bwd_noalloc (64 MiB)    */
  NSA_ERR_DTYPE = -11,      /* element type combination not supported by
                               nsa_sel_attn_fwd_ex                            */
  NSA_ERR_BOUNDS = -12,     /* (library built with NSA_DEBUG_BOUNDS only) a
                               kernel's own bounds check found a tile outside
                               the keys its row may read; reported by
                               nsa_sync_status                                */
  NSA_ERR_PAGE_SIZE = -13   /* a cache's page_size is no power of two from 16
                               to 1024                                        */
} nsa_status;

/* Element types of nsa_sel_attn_fwd_ex. */
typedef enum nsa_dtype {
  NSA_F16 = 0,   /* IEEE binary16                                  */
  NSA_BF16 = 1,  /* bfloat16 (the upper 16 bits of an IEEE binary32) */
  NSA_F32 = 2    /* IEEE binary32                                  */
} nsa_dtype;

/* Human-readable name of a status code (static string, never NULL). */
const char* nsa_status_string(int status);

/* Library version as 10000*major + 100*minor + patch. */
int nsa_version(void);

/*
 * nsa_sel_attn_fwd -- selection-attention forward on the GPU.
 *
 *   Q              device, IEEE fp16, [B, M, H, D]
 *   K, V           device, IEEE fp16, [B, N, G, D]
 *   block_indices  device, int32,     [B, M, G, T]; block ids, -1 = padding
 *   O              device, fp32,      [B, M, H, D]   (output)
 *   LSE            device, fp32,      [B, H, M]      (output, natural log)
 *   B, M, N, T     >= 0; an empty problem (B*M == 0) returns NSA_OK at once
 *   H, G, D        > 0, H % G == 0, D in {64, 128}; H/G (query heads per
 *                  KV group) is 1..8, or a multiple of 8 -- a warp serves up to
 *                  8 heads of a group: fewer are padded, more are split into
 *                  sub-groups of 8 that share the group's K/V and index row
 *   block_size     32 or 64
 *   scale          score multiplier; <= 0 selects 1/sqrt(D)
 *   stream         cudaStream_t to launch on (NULL = legacy default stream)
 *
 * Asynchronous: validates the arguments on the host, enqueues one kernel on
 * `stream` and returns without synchronising. K and V are fetched with TMA
 * through tensor maps encoded on the host for each call. It allocates
 * nothing, frees nothing and keeps no state between calls (the per-device
 * status word of nsa_sync_status aside); concurrent calls on different
 * streams are safe. Returns NSA_OK, or a negative nsa_status. Errors that
 * surface only when the kernel runs are reported by the next CUDA call that
 * synchronises with `stream`, as for any CUDA launch.
 */
int nsa_sel_attn_fwd(const void* Q, const void* K, const void* V,
                     const int32_t* block_indices, float* O, float* LSE,
                     int64_t B, int64_t M, int64_t N, int64_t H, int64_t G,
                     int64_t D, int64_t T, int block_size, float scale,
                     void* stream);

/*
 * nsa_sel_attn_fwd_ex -- nsa_sel_attn_fwd with a choice of element types.
 *
 *   qkv_dtype  NSA_F16 or NSA_BF16: the type of Q, K and V (all three alike)
 *   o_dtype    NSA_F32, or qkv_dtype: the type O is written in
 *
 * Every other argument, layout, check and property is that of
 * nsa_sel_attn_fwd; LSE stays fp32. nsa_sel_attn_fwd is this call with
 * (NSA_F16, NSA_F32). With bf16 inputs both products run as bf16 MMAs with
 * fp32 accumulation, so the probabilities are rounded to bf16 (8 significant
 * bits) before the PV product -- the bf16 reading of the "FP16 matmuls, FP32
 * accumulation" requirement ("[wave] NSA: selection attention forward
 * kernel", section "Requirements"). Scores, running max and row sums are
 * fp32 in every combination; a 16-bit O is the fp32 result rounded to
 * nearest even. Any other combination returns NSA_ERR_DTYPE before launch.
 */
int nsa_sel_attn_fwd_ex(const void* Q, const void* K, const void* V,
                        const int32_t* block_indices, void* O, float* LSE,
                        int64_t B, int64_t M, int64_t N, int64_t H, int64_t G,
                        int64_t D, int64_t T, int block_size, float scale,
                        int qkv_dtype, int o_dtype, void* stream);

/*
 * nsa_sel_attn_fwd_strided -- nsa_sel_attn_fwd_ex on strided tensors.
 *
 *   strides  host array of 12 element strides, or NULL for contiguous:
 *            [0..2]  Q over (b, m, h)     [3..5]  K over (b, n, g)
 *            [6..8]  V over (b, n, g)     [9..11] O over (b, m, h)
 *            The last dimension (d) of Q, K, V and O is contiguous; LSE and
 *            block_indices are contiguous as in nsa_sel_attn_fwd.
 *
 * Lets Q, K and V be views into one fused projection (for example
 * [B, M, H + 2G, D] with Q the first H heads) and O a slice of a larger
 * buffer, without copies. Every stride must be a multiple of 8 elements (so
 * every row starts 16-byte aligned; else NSA_ERR_ALIGN) and in
 * [0, 2^40] (else NSA_ERR_SHAPE); the strides must describe memory the
 * caller owns, and O must not overlap Q, K or V. Everything else is
 * nsa_sel_attn_fwd_ex.
 */
int nsa_sel_attn_fwd_strided(const void* Q, const void* K, const void* V,
                             const int32_t* block_indices, void* O, float* LSE,
                             int64_t B, int64_t M, int64_t N, int64_t H, int64_t G,
                             int64_t D, int64_t T, int block_size, float scale,
                             int qkv_dtype, int o_dtype, const int64_t* strides,
                             void* stream);

/*
 * nsa_sel_attn_fwd_shared_workspace_bytes -- device workspace of
 * nsa_sel_attn_fwd_shared: one 32-byte record per (b, g, tile of 16
 * queries), rounded up to 256 bytes. Negative nsa_status for invalid sizes
 * (B * G * ceil(M/16) must stay below 2^31). Pure host arithmetic.
 */
int64_t nsa_sel_attn_fwd_shared_workspace_bytes(int64_t B, int64_t M, int64_t G);

/*
 * nsa_sel_attn_fwd_shared -- the forward of nsa_sel_attn_fwd_ex (O fp32) in
 * two passes over the blocks that consecutive queries share.
 *
 *   qkv_dtype   NSA_F16 or NSA_BF16
 *   workspace   device memory of at least
 *               nsa_sel_attn_fwd_shared_workspace_bytes(B, M, G) bytes,
 *               16-byte aligned, owned by the caller (else NSA_ERR_WORKSPACE
 *               or NSA_ERR_ALIGN); on return it holds the per-tile records
 *
 * Index rows that keep the initial block and the most recent blocks of
 * every query (as nsa_topk_blocks with n_init, n_local > 0 writes them) give
 * the queries of a tile of 16 consecutive positions some blocks in common.
 * Per (b, g, tile) a list pass records up to 7
 * blocks that every query of the tile lists, whose first key the tile's
 * first query sees and whose keys all lie below M and N, in the order the
 * tile's first query lists them. A tile-shared pass gathers those blocks
 * once and computes, on the tcgen05 tensor cores, the softmax of all
 * 16 x 8 (query, head) rows over their keys (each row masked to the keys
 * at or before its query); it writes the normalised partial O and its LSE
 * into O and LSE. The gather kernel of
 * nsa_sel_attn_fwd then skips the recorded blocks and continues the online
 * softmax from that state, so its outputs cover every selected key once.
 * The result is the same operation as nsa_sel_attn_fwd_ex with the same
 * tolerance (the partial sums are added in another order; outputs are not
 * bit-identical to the one-pass call). Three kernels are enqueued on
 * `stream`; nothing is allocated or synchronised.
 *
 * The two-pass path serves block_size = 64, D = 128, H/G = 8, M >= 16,
 * N >= block_size and T >= 1; any other valid problem runs the one-pass
 * kernel (the workspace is then unused). With 32-key blocks the common
 * blocks are too small a share of a row's bytes for the extra passes to pay
 * (measured slower than one pass), so those problems take the one-pass
 * kernel too. Every other argument, layout, check and property is that
 * of nsa_sel_attn_fwd_ex, with one difference in what non-finite inputs
 * may do: NaN or Inf in K/V rows past every query (>= M), in blocks no
 * query lists, and in the keys of a tile's own block past the tile's last
 * query never reach an output (as for the one-pass call), but a non-finite
 * V row between two queries of the same 16-query tile reaches the earlier
 * query's output too (the tile's rows share one P.V product over those
 * keys).
 */
int nsa_sel_attn_fwd_shared(const void* Q, const void* K, const void* V,
                            const int32_t* block_indices, float* O, float* LSE, int64_t B,
                            int64_t M, int64_t N, int64_t H, int64_t G, int64_t D, int64_t T,
                            int block_size, float scale, int qkv_dtype, void* workspace,
                            int64_t workspace_bytes, void* stream);

/*
 * nsa_sel_attn_fwd_host_workspace_bytes -- device workspace that
 * nsa_sel_attn_fwd_host needs for these sizes and query chunk length
 * (chunk_m <= 0 selects the default). Returns the byte count, or a negative
 * nsa_status for invalid sizes. Pure host arithmetic; no CUDA call.
 */
int64_t nsa_sel_attn_fwd_host_workspace_bytes(int64_t B, int64_t M, int64_t N, int64_t H,
                                              int64_t G, int64_t D, int64_t T, int block_size,
                                              int64_t chunk_m);

/*
 * nsa_sel_attn_fwd_host -- the same forward with HOST buffers in and out.
 *
 *   Q, K, V, block_indices   host memory, layouts as in nsa_sel_attn_fwd
 *   O, LSE                   host memory, written
 *   workspace                device memory of at least
 *                            nsa_sel_attn_fwd_host_workspace_bytes(...) bytes,
 *                            256-byte aligned, owned by the caller
 *   chunk_m                  queries per pipeline chunk, rounded up to a
 *                            multiple of 64 (<= 0: default, about M/32)
 *   stream                   caller's stream: the call's work starts after
 *                            the work already queued on it, and it waits for
 *                            all of the call's work
 *
 * The queries are processed in chunks of chunk_m positions. For each chunk
 * the call enqueues, on an internal upload stream, the copies of its Q rows,
 * its index rows and the K/V rows it can see (keys below the chunk's end,
 * each copied once); the kernel (even chunks on `stream`, odd chunks on an
 * internal second compute stream); and on an internal download
 * stream, the copies of its O rows and LSE columns. Chunk buffers are double
 * buffered in the workspace, so uploads, kernels and downloads of adjacent
 * chunks overlap. Copies overlap only if the host buffers are page-locked
 * (pinned); with pageable memory they are correct but serial.
 *
 * Returns after enqueueing; `stream` is made to wait for every copy, so the
 * outputs are complete once `stream` is synchronised. Results are
 * bit-identical to nsa_sel_attn_fwd on the same inputs. It allocates no
 * memory (the internal streams and events are created and released by the
 * call). Errors: as nsa_sel_attn_fwd, plus NSA_ERR_WORKSPACE.
 */
int nsa_sel_attn_fwd_host(const void* Q, const void* K, const void* V,
                          const int32_t* block_indices, float* O, float* LSE, int64_t B,
                          int64_t M, int64_t N, int64_t H, int64_t G, int64_t D, int64_t T,
                          int block_size, float scale, void* workspace,
                          int64_t workspace_bytes, int64_t chunk_m, void* stream);

/*
 * nsa_sel_attn_fwd_host_ex -- nsa_sel_attn_fwd_host with the element types of
 * nsa_sel_attn_fwd_ex: Q, K, V in host memory as qkv_dtype (NSA_F16 or
 * NSA_BF16), O written as o_dtype (NSA_F32 or qkv_dtype); LSE fp32. Any
 * other combination returns NSA_ERR_DTYPE before anything is enqueued. The
 * workspace of nsa_sel_attn_fwd_host_workspace_bytes (sized for fp32 O)
 * suffices for every combination. Results are bit-identical to
 * nsa_sel_attn_fwd_ex on the same inputs; everything else is
 * nsa_sel_attn_fwd_host.
 */
int nsa_sel_attn_fwd_host_ex(const void* Q, const void* K, const void* V,
                             const int32_t* block_indices, void* O, float* LSE, int64_t B,
                             int64_t M, int64_t N, int64_t H, int64_t G, int64_t D, int64_t T,
                             int block_size, float scale, int qkv_dtype, int o_dtype,
                             void* workspace, int64_t workspace_bytes, int64_t chunk_m,
                             void* stream);

/*
 * nsa_sel_attn_bwd_workspace_bytes -- device workspace nsa_sel_attn_bwd
 * needs: an fp16 copy of dO, one 64-byte (LSE, delta) record per (b, m, g,
 * 8-head sub-group), the per-(b, g, block) query lists (at most B*M*G*T
 * entries) and their counts and offsets, and 8 bytes per (b, m, g) row
 * for the row's local entries. Negative nsa_status for invalid sizes
 * (B*M*G*T must stay below 2^31). Pure host arithmetic.
 */
int64_t nsa_sel_attn_bwd_workspace_bytes(int64_t B, int64_t M, int64_t N, int64_t H,
                                         int64_t G, int64_t D, int64_t T, int block_size);

/*
 * nsa_sel_attn_bwd -- gradients of nsa_sel_attn_fwd (the section
 * "Requirements" returns LSE for this pass).
 *
 *   Q, K, V, block_indices   as for the forward (device)
 *   O, LSE                   the forward's outputs (device, fp32)
 *   dO                       upstream gradient of O, fp32 [B, M, H, D]
 *   dQ                       fp32 [B, M, H, D]   (written)
 *   dK, dV                   fp32 [B, N, G, D]   (written; zeroed first)
 *   workspace                device memory of at least
 *                            nsa_sel_attn_bwd_workspace_bytes() bytes,
 *                            256-byte aligned
 *
 * With p = exp(scale q.k - LSE), dP = dO.v and delta = dO.O per row and head:
 * dS = p (dP - delta), dQ = scale sum dS k, dK += scale dS q, dV += p dO over
 * every visible (query, head, key). Stages on `stream`: per-row inputs
 * (delta, an fp16 copy of dO; with D = 64 also dQ, from a query-major
 * kernel); a transposed index listing, per (b, g, block), the queries that
 * selected it; a key-major kernel that loads each block once per chunk of
 * its list and adds its dK / dV partial sums. With D = 128, the entries
 * of each query's own block c and of block c - 1 go to a local-block
 * kernel instead (one CTA per block row of 32 or 64 queries: their dQ rows
 * summed on the tensor cores and stored once, dK / dV of the two blocks
 * summed over the block row), and the key-major kernel also forms dQ =
 * dS K for the other entries and adds it with fp32 reductions; dK / dV are
 * added with fp32 atomics (D = 64) or bulk fp32 reductions (D = 128). dK /
 * dV (and dQ when D = 128) sum in an order set by atomics (equal within
 * rounding from run to run). With D = 128 every key of a block some query
 * selects may enter the dQ of the queries that share its block row or its
 * chunk (with weight 0 where a query does not select or see it), so K
 * must be finite in every selected block, including keys after a query's
 * position. With D = 128 the index transpose runs on a second stream that
 * the call creates and releases, beside the per-row stage and the
 * local-block kernel; `stream` waits for it. Asynchronous, allocates no
 * device memory; errors as nsa_sel_attn_fwd plus NSA_ERR_WORKSPACE.
 * Pointers must be 16-byte aligned (LSE and block_indices 4-byte).
 */
int nsa_sel_attn_bwd(const void* Q, const void* K, const void* V,
                     const int32_t* block_indices, const float* O, const float* LSE,
                     const float* dO, float* dQ, float* dK, float* dV, int64_t B, int64_t M,
                     int64_t N, int64_t H, int64_t G, int64_t D, int64_t T, int block_size,
                     float scale, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * nsa_sel_attn_bwd_ex -- nsa_sel_attn_bwd with a choice of input type.
 *
 *   qkv_dtype  NSA_F16 or NSA_BF16: the type of Q, K and V (else
 *              NSA_ERR_DTYPE before anything is enqueued)
 *
 * With bf16 inputs every tensor-core product takes bf16 operands (the 16-bit
 * copy of dO, P and dS are rounded to bf16) with fp32 accumulation -- the
 * bf16 reading of "FP16 matmuls, FP32 accumulation" that nsa_sel_attn_fwd_ex
 * takes for the forward. O, LSE, dO and the gradients stay fp32. Everything
 * else, the workspace included, is nsa_sel_attn_bwd; nsa_sel_attn_bwd is
 * this call with NSA_F16.
 */
int nsa_sel_attn_bwd_ex(const void* Q, const void* K, const void* V,
                        const int32_t* block_indices, const float* O, const float* LSE,
                        const float* dO, float* dQ, float* dK, float* dV, int64_t B, int64_t M,
                        int64_t N, int64_t H, int64_t G, int64_t D, int64_t T, int block_size,
                        float scale, int qkv_dtype, void* workspace, int64_t workspace_bytes,
                        void* stream);

/*
 * nsa_sel_attn_bwd_noalloc -- nsa_sel_attn_bwd for callers that cannot
 * allocate device memory. The pages have no counterpart to this entry point.
 *
 * Some callers may not allocate at all: a plugin inside a host application
 * that owns every device allocation through its own pool and hands plugins
 * no allocator, or a service that reserves all of its memory at start-up and
 * forbids allocation while it serves. They still pass every input and
 * output; the scratch the backward needs (delta, the per-block query lists
 * and their offsets) comes from a fixed 64 MiB array inside the library,
 * which every GPU that loads the library holds until the process exits.
 *
 * Arguments, layouts and results are those of nsa_sel_attn_bwd without the
 * workspace. A problem whose scratch (nsa_sel_attn_bwd_workspace_bytes)
 * exceeds 64 MiB is rejected with NSA_ERR_SCRATCH before anything is
 * launched; a problem without queries (B == 0 or M == 0) needs no scratch
 * and only zeroes dK and dV. The call allocates and frees nothing and creates
 * no stream: all of its stages run in order on `stream`. Every
 * call looks up the array's device address in the current device's context
 * (cudaGetSymbolAddress: a host-side query, no allocation, no
 * synchronisation), so a context created anew after cudaDeviceReset gets
 * its own array. The first lookup on a device may load the library's
 * device code: make the first call on each device before any stream
 * capture. Every call uses the same array and finds the previous call's
 * contents in it; the parts that must start at zero are cleared on the
 * call's stream. Calls whose work overlaps on the GPU (on different
 * streams, or from different threads on one device) race on the array:
 * serialise them.
 */
int nsa_sel_attn_bwd_noalloc(const void* Q, const void* K, const void* V,
                             const int32_t* block_indices, const float* O, const float* LSE,
                             const float* dO, float* dQ, float* dK, float* dV, int64_t B,
                             int64_t M, int64_t N, int64_t H, int64_t G, int64_t D, int64_t T,
                             int block_size, float scale, void* stream);

/*
 * nsa_topk_blocks -- top-k block selection: block_indices from block scores.
 *
 * The selection-attention issue takes block_indices from a top-k selection
 * kernel ("[wave] NSA: selection attention forward kernel", section
 * "Depends on"); its section "Operation" fixes the output [B,M,G,T] and
 * section "Requirements" one row per GQA group. The pages do not say how
 * blocks are scored, so the scores are the input:
 *
 *   scores         device, fp32,  [B, M, G, ceil(N/block_size)]; the score
 *                  of key block t for query (b, m) and KV group g. Only
 *                  entries of free candidate blocks (below) are read.
 *   block_indices  device, int32, [B, M, G, T] (output)
 *   B, M, N, T     >= 0; G > 0; ceil(N/block_size) <= 4096
 *   block_size     >= 1 (keys per block, as in nsa_sel_attn_fwd)
 *   n_init,        >= 0 with n_init + n_local <= T: the first n_init and the
 *   n_local        last n_local candidate blocks of a row are always chosen
 *   stream         cudaStream_t to launch on
 *
 * Row (b, m, g): the candidates are the blocks t = 0..c holding a key
 * visible to query m, c = floor(min(m, N-1) / block_size) (none if N = 0).
 * With at most T candidates all are chosen. Otherwise the forced blocks are
 * chosen and the remaining T - n_init - n_local slots go to the other
 * candidates with the highest scores; equal scores choose the lower block
 * (-0.0 equals +0.0) and NaN ranks below every number. The row is written
 * in ascending block order and padded with -1, so it is a valid
 * block_indices row for nsa_sel_attn_fwd (distinct, causal).
 *
 * Asynchronous: one kernel on `stream`, no allocation, no synchronisation.
 * Returns NSA_ERR_SHAPE (bad sizes, n_init/n_local out of range, too many
 * blocks), NSA_ERR_BLOCK_SIZE, NSA_ERR_NULL, NSA_ERR_ALIGN (a pointer not
 * 4-byte aligned) before launch; an empty output returns NSA_OK at once.
 * A row copy that does not arrive within 1 s makes nsa_sync_status report
 * NSA_ERR_TIMEOUT; the outputs of that launch are then undefined.
 */
int nsa_topk_blocks(const float* scores, int32_t* block_indices, int64_t B, int64_t M,
                    int64_t N, int64_t G, int64_t T, int block_size, int n_init,
                    int n_local, void* stream);

/*
 * nsa_swa_fwd -- GQA sliding-window (or dense) attention forward, the
 * second workload on the pages ("[Kernel][MI350] Add 8 wave GQA
 * sliding-window attention kernel", sections "Summary" and "What it does").
 *
 *   Q              device, [B, M, H, D],    fp16 or bf16 (dtype)
 *   K, V           device, [B, N, H_kv, D], same type
 *   O              device, [B, M, H, D],    same type (output)
 *   LSE            device, fp32 [B, H, M] (output, natural log), or NULL
 *   H % H_kv == 0  query head h reads KV head h / (H / H_kv)
 *   D              64 or 128
 *   window_left,   query i attends to keys j with i - window_left <= j <=
 *   window_right   i + window_right and 0 <= j < N; a negative value leaves
 *                  that side unbounded: (-1, -1) is dense attention, (-1, 0)
 *                  causal, (L, 0) causal with L keys of history
 *   scale          score multiplier; <= 0 selects 1/sqrt(D)
 *   dtype          NSA_F16 or NSA_BF16
 *
 * Query i is aligned with key i. Both products run on the 5th-generation
 * tensor cores (tcgen05, fp32 accumulation in tensor memory). P is rounded
 * to the input type before the PV product, and O is the fp32 result rounded
 * once. A row with no visible key gets O = 0 and LSE = -inf. The call is
 * asynchronous and allocates nothing. Each CTA holds 512 tensor-memory
 * columns of its SM for its lifetime. Errors returned before launch:
 * NSA_ERR_SHAPE, NSA_ERR_GROUPS, NSA_ERR_HEAD_DIM, NSA_ERR_DTYPE,
 * NSA_ERR_NULL, NSA_ERR_ALIGN (Q, K, V, O not 16-byte aligned, LSE not
 * 4-byte aligned). A timed-out device wait is reported by nsa_sync_status.
 */
int nsa_swa_fwd(const void* Q, const void* K, const void* V, void* O, float* LSE,
                int64_t B, int64_t M, int64_t N, int64_t H, int64_t H_kv, int64_t D,
                int64_t window_left, int64_t window_right, float scale, int dtype,
                void* stream);

/*
 * nsa_swa_bwd_workspace_bytes -- device workspace of nsa_swa_bwd: LSE and
 * delta of every (batch, head, query), and, where tiles of keys or of queries
 * are cut because they do not fill the SMs, fp32 parts of dK and dV (128 KB
 * each at D = 128, some 152 to 304 of them as a rule) and of dQ (64 KB).
 * Negative nsa_status for invalid sizes. Pure host arithmetic.
 */
int64_t nsa_swa_bwd_workspace_bytes(int64_t B, int64_t M, int64_t N, int64_t H, int64_t H_kv,
                                    int64_t D, int64_t window_left, int64_t window_right);

/*
 * nsa_swa_bwd -- gradients of nsa_swa_fwd.
 *
 *   Q, K, V, window_left, window_right, scale, dtype   as for the forward
 *   O, LSE         the forward's outputs: O of type dtype, LSE fp32 [B, H, M]
 *   dO             upstream gradient of O, dtype, [B, M, H, D]
 *   dQ             [B, M, H, D]     (output, grad_dtype)
 *   dK, dV         [B, N, H_kv, D]  (output, grad_dtype)
 *   grad_dtype     NSA_F32, or dtype: the fp32 sums rounded once (nearest even)
 *   workspace      device memory of at least nsa_swa_bwd_workspace_bytes()
 *                  bytes for these arguments, 16-byte aligned (else
 *                  NSA_ERR_WORKSPACE, NSA_ERR_ALIGN)
 *
 * With p = exp(scale q.k - LSE), dP = dO.v and delta = dO.O per row and head:
 * dS = p (dP - delta), dQ = scale sum dS k, dK = scale sum dS q, dV = sum p dO
 * over the visible pairs (dK and dV over the query heads of the KV head too).
 * The products run on the 5th-generation tensor cores with fp32 sums in tensor
 * memory; p and dS are rounded to dtype before the products they enter. Every
 * sum has a fixed order: equal calls give equal bits. With fp16 inputs p is
 * carried times 2^12, and dS times a power of two that every row of dQ and of dK
 * takes from the norms of the dO and V rows that its tiles hold, so that dS
 * neither overflows nor loses bits, whatever the scale of dO.
 *
 * A query without keys (LSE = -inf) gets dQ = 0 and adds nothing to dK, dV; a
 * key that no query sees gets dK = dV = 0. p and dS of hidden pairs are exactly
 * 0 whatever Q, K, V and dO hold there, but they are multiplied by rows that
 * share a tile with visible ones: K must be finite in the 64-key tiles that
 * hold a key some query of a 128-query tile sees, Q and dO in the 64-query
 * tiles that hold a query which sees some key of a 128-key tile (as V must for
 * the forward, in 128-key tiles). M and N are at most 2^29. The outputs must
 * not overlap the inputs or one another.
 *
 * Asynchronous: two kernels on `stream` (three with fp16 inputs, and up to two
 * more where gradients are joined from parts), no allocation; calls that may overlap need workspaces of their own.
 * Errors before launch as nsa_swa_fwd, plus NSA_ERR_WORKSPACE. With no query,
 * or no key, the gradients are zeroed and no workspace is needed. A timed-out
 * device wait is reported by nsa_sync_status.
 */
int nsa_swa_bwd(const void* Q, const void* K, const void* V, const void* O, const float* LSE,
                const void* dO, void* dQ, void* dK, void* dV, int64_t B, int64_t M, int64_t N,
                int64_t H, int64_t H_kv, int64_t D, int64_t window_left, int64_t window_right,
                float scale, int dtype, int grad_dtype, void* workspace, int64_t workspace_bytes,
                void* stream);

/*
 * nsa_qk_norm_rope -- RMS norm of every query and key head and the position
 * rotation in one pass: what a layer does between its Q/K projections and
 * the attention entry points of this library.
 *
 *   Q, K           device, fp16 or bf16 (dtype), [B, M, H, D] and [B, M, G, D]
 *   Qo, Ko         device, same type and shapes (output); each may be its
 *                  input (same address and strides), else no overlap
 *   wq, wk         device, [D] norm weights, weight_dtype NSA_F32 or dtype;
 *                  NULL: no weight (ones)
 *   cos_table,     device, fp32, [table_rows, R/2]: cosine and sine of the
 *   sin_table      angle of pair i at a position (row); unused when R = 0
 *   positions      device, int32: token (b, m) is at
 *                  positions[b * positions_stride + m] (stride 0: one row for
 *                  the whole batch); NULL: token m is at position m
 *   H, G           > 0 (no relation between them is needed); D 64 or 128
 *   R              rotated entries per head, the first R: 0 (norm alone) to D,
 *                  a multiple of 16
 *   eps            >= 0, finite
 *   interleaved    0: pair i is entries (i, i + R/2); else (2i, 2i + 1)
 *   strides        host array of 12 element strides, (b, m, head) of Q, K, Qo
 *                  and Ko, or NULL for contiguous; each a multiple of 8 (else
 *                  NSA_ERR_ALIGN) in [0, 2^40], and not 0 for a written
 *                  tensor's dimension of more than one (else NSA_ERR_SHAPE).
 *                  D is contiguous. Q and K can so be slices of one projection.
 *
 * Per row x: n = x rsqrt(mean(x^2) + eps) w, then every pair (a, b) of n
 * becomes (a cos - b sin, b cos + a sin); all in fp32, each operation rounded
 * by itself ((x r) w; two products, then their sum), and once (nearest even) to
 * dtype. The sum of squares adds entries 32 apart first, in rising order, then
 * neighbours, pairs, pairs of pairs and so on. A token whose position is
 * negative, or >= table_rows when R > 0, is padding: its inputs are not read and
 * its output rows are zero. A non-finite entry reaches its own row only. With
 * positions NULL and R > 0 the table must hold M rows (else NSA_ERR_SHAPE).
 *
 * One kernel on `stream`; allocates nothing and keeps no state. Errors before
 * launch: NSA_ERR_SHAPE (sizes, R, eps, B*M >= 2^31), NSA_ERR_HEAD_DIM,
 * NSA_ERR_DTYPE, NSA_ERR_NULL, NSA_ERR_ALIGN (Q, K, Qo, Ko, weights, tables
 * 16-byte; positions 4-byte). An empty problem returns NSA_OK at once.
 */
int nsa_qk_norm_rope(const void* Q, const void* K, void* Qo, void* Ko, const void* wq,
                     const void* wk, const float* cos_table, const float* sin_table,
                     const int32_t* positions, int64_t B, int64_t M, int64_t H, int64_t G,
                     int64_t D, int64_t R, int64_t table_rows, int64_t positions_stride,
                     float eps, int interleaved, int dtype, int weight_dtype,
                     const int64_t* strides, void* stream);

/*
 * nsa_qk_norm_rope_bwd_workspace_bytes -- device workspace of
 * nsa_qk_norm_rope_bwd: a partial weight gradient of each of up to 456 CTAs.
 * Negative nsa_status for invalid sizes. Pure host arithmetic.
 */
int64_t nsa_qk_norm_rope_bwd_workspace_bytes(int64_t B, int64_t M, int64_t D);

/*
 * nsa_qk_norm_rope_bwd -- gradients of nsa_qk_norm_rope.
 *
 *   Q, K           the forward's inputs (the norms are formed again)
 *   dQo, dKo       gradients of its outputs, grad_dtype NSA_F32 (what
 *                  nsa_sel_attn_bwd writes) or dtype
 *   dQ, dK         device, dtype (output); each may be the input of its shape
 *                  (dQo, dKo of type dtype, or Q, K) with the same strides
 *   dwq, dwk       device, fp32 [D] (output), or NULL: not wanted
 *   strides        host array of 18 element strides, (b, m, head) of Q, K,
 *                  dQo, dKo, dQ, dK, or NULL; rules as for the forward
 *   workspace      device memory of at least
 *                  nsa_qk_norm_rope_bwd_workspace_bytes() bytes, 16-byte
 *                  aligned (else NSA_ERR_WORKSPACE, NSA_ERR_ALIGN); unused
 *                  when both dwq and dwk are NULL
 *
 * With g the pairs of a row of dQo (dKo) turned back and xhat = x
 * rsqrt(mean(x^2) + eps): dw = sum over rows of g xhat, dx = rsqrt(...) (g w -
 * xhat mean(g w xhat)); fp32, dx rounded once. Padding tokens (as in the
 * forward; their rows are not read) get a zero gradient and add nothing to
 * dw. The sums of dw have a fixed order: equal calls give equal bits. Two
 * kernels on `stream` (one when no dw is wanted); allocates nothing. With no
 * token, dwq and dwk are zeroed. Everything else is nsa_qk_norm_rope.
 */
int nsa_qk_norm_rope_bwd(const void* Q, const void* K, const void* dQo, const void* dKo, void* dQ,
                         void* dK, float* dwq, float* dwk, const void* wq, const void* wk,
                         const float* cos_table, const float* sin_table, const int32_t* positions,
                         int64_t B, int64_t M, int64_t H, int64_t G, int64_t D, int64_t R,
                         int64_t table_rows, int64_t positions_stride, float eps,
                         int interleaved, int dtype, int weight_dtype, int grad_dtype,
                         const int64_t* strides, void* workspace, int64_t workspace_bytes,
                         void* stream);

/*
 * A paged cache of keys and values (device memory of the caller's).
 *
 * `pages` pages hold page_size token rows for each of G KV heads of D entries.
 * A sequence has its tokens where its row of a page table says: position p of
 * sequence b is row p % page_size of page page_table[b * table_cols +
 * p / page_size]. An entry outside [0, pages) (-1, say) is a page that the
 * sequence does not have: one that it has not come to, or one given back
 * behind a window. Sequences may share pages that are only read.
 *
 *   k, v           bits 16: the 16-bit rows [pages, page_size, G, D], with
 *                  element strides k_strides, v_strides over (page, token,
 *                  head), D contiguous; multiples of 8 in [0, 2^36], and not 0
 *                  for a dimension of more than one.
 *                  bits 4: bytes [pages, page_size, G, D / 2], contiguous (the
 *                  strides are not used); byte i holds entry 2 i in its lower
 *                  and entry 2 i + 1 in its upper four bits
 *   k_scale,       bits 4: bf16 [pages, G, page_size, 2], contiguous: (step,
 *   v_scale        low) of a row, whose entries are low + step * code. A step
 *                  is 0 (all codes are 0), 2^-60 or more, or NaN.
 *                  bits 16: not used
 *   page_size      a power of two from 16 to 1024 (else NSA_ERR_PAGE_SIZE);
 *                  table_cols * page_size is at most 2^30
 *   bits           16 or 4 (else NSA_ERR_DTYPE)
 *
 * All pointers are 16-byte aligned. Every field is 8 bytes wide.
 */
typedef struct nsa_kv_cache {
  void* k;
  void* v;
  void* k_scale;
  void* v_scale;
  int64_t pages;
  int64_t page_size;
  int64_t k_strides[3];
  int64_t v_strides[3];
  int64_t bits;
} nsa_kv_cache;

/*
 * nsa_kv_append -- the RMS norm of every new query and key head and the
 * position rotation, as nsa_qk_norm_rope, with K and V written into the cache:
 * what a layer that answers does between its projections and nsa_paged_attn.
 *
 *   Q, Qo          device, dtype, [B, M, H, D]; Qo may be Q (same strides);
 *                  H = 0: neither is used
 *   K, V           device, dtype, [B, M, G, D]
 *   cache,         the cache, written, and int32 [B, table_cols]
 *   page_table
 *   wq, wk, cos_table, sin_table, positions, R, table_rows, positions_stride,
 *   interleaved, dtype, weight_dtype     as for nsa_qk_norm_rope
 *   eps            >= 0: the norm's; < 0: no norm (wq, wk NULL)
 *   strides        host array of 12 element strides, (b, m, head) of K, V, Q
 *                  and Qo, or NULL for contiguous; rules as for
 *                  nsa_qk_norm_rope. All can be slices of one projection.
 *
 * A 16-bit cache has the type of K and V. A 4-bit row is made of the row
 * rounded to that type: low = bf16(min), step = bf16((max - low) / 15), 0 where
 * that is below 2^-60, code = clamp(rint((x - low) / step), 0, 15); a row with
 * an entry that is not finite, or whose range passes fp32's, reads as NaN. Codes
 * jump where a last bit of the 16-bit row moves: they are those of that row, whose
 * bits the order of operations above decides.
 *
 * A token of negative position, or (R > 0) of one past the angle tables, is
 * padding: its Q row is zero and nothing is stored. A token in a page that the
 * sequence does not have is not stored; its Q row is formed. Two tokens of a
 * call must not have the same place. Rows of the cache that no token is stored
 * to are left as they are.
 *
 * One kernel on `stream`; allocates nothing and keeps no state. Errors before
 * launch as nsa_qk_norm_rope, plus the cache's.
 */
int nsa_kv_append(const void* Q, const void* K, const void* V, void* Qo,
                  const nsa_kv_cache* cache, const int32_t* page_table, const void* wq,
                  const void* wk, const float* cos_table, const float* sin_table,
                  const int32_t* positions, int64_t B, int64_t M, int64_t H, int64_t G, int64_t D,
                  int64_t R, int64_t table_rows, int64_t positions_stride, int64_t table_cols,
                  float eps, int interleaved, int dtype, int weight_dtype, const int64_t* strides,
                  void* stream);

/*
 * nsa_kv_read -- rows of the cache as K and V tensors, as nsa_sel_attn_fwd and
 * nsa_swa_fwd take them.
 *
 *   positions      as for nsa_kv_append: (b, m) reads the row of that position
 *   K, V           device, dtype, [B, M, G, D], contiguous (output); dtype is
 *                  the type of a 16-bit cache, either one for a 4-bit cache
 *                  (low + step * code, rounded once)
 *
 * A negative position, or one in a page that the sequence does not have, gives
 * rows of zeros. One kernel on `stream`. B M G is at most 2^34.
 */
int nsa_kv_read(const nsa_kv_cache* cache, const int32_t* page_table, const int32_t* positions,
                void* K, void* V, int64_t B, int64_t M, int64_t G, int64_t D,
                int64_t positions_stride, int64_t table_cols, int dtype, void* stream);

/*
 * nsa_paged_attn_workspace_bytes -- device workspace of nsa_paged_attn for a page
 * table of `tokens` = table_cols * page_size tokens, enough for 16 and 4 bits. 0
 * where no row tile of a KV head is cut along its keys: a query sees few (512, or
 * 2048 where there is a row tile for every SM), or the batch has more than 512 row
 * tiles; else up to 20 MB, whatever the lengths. Negative nsa_status for invalid
 * sizes. Pure host arithmetic.
 *
 * A row tile is 8 of the M H/G rows of a KV head where there are no more, else 16,
 * or, with 17 rows (4 bits: 33) or more and H/G up to 128, as many whole queries as
 * make up to 128 rows.
 */
int64_t nsa_paged_attn_workspace_bytes(int64_t B, int64_t M, int64_t H, int64_t G, int64_t D,
                                       int64_t tokens, int64_t window_left, int64_t sinks);

/*
 * nsa_paged_attn -- attention of new tokens over the cache: the decoding step
 * (M = 1), drafted tokens, or a piece of a prompt, after nsa_kv_append has
 * stored their own keys and values.
 *
 *   Q              device, dtype, [B, M, H, D]; q_strides: host array of 3
 *                  element strides (b, m, head), multiples of 8 and not 0 for a
 *                  dimension of more than one, or NULL
 *   positions      device, int32, not NULL: as for nsa_kv_append; negative:
 *                  padding; at most 2^31 - 32
 *   O              device, dtype, [B, M, H, D], contiguous (output)
 *   LSE            device, fp32, [B, H, M] (output), or NULL
 *   window_left,   query at position p sees key j of its sequence iff j <= p,
 *   sinks          and j >= p - window_left (negative: no bound) or j < sinks,
 *                  and the sequence has j's page
 *   scale          score multiplier; <= 0 selects 1/sqrt(D)
 *   workspace      device memory of nsa_paged_attn_workspace_bytes() bytes,
 *                  16-byte aligned (else NSA_ERR_WORKSPACE, NSA_ERR_ALIGN);
 *                  calls that may overlap need one each
 *
 * H is a multiple of G. p is rounded to 16 bits before the product with V (to
 * dtype, or fp16 over a 4-bit cache); in row tiles of 8 and 16 what that leaves is
 * multiplied too (over a 4-bit cache where O is fp16). Sums are fp32, O is rounded once. LSE is
 * the natural log of sum(exp(scale q.k)) over the visible keys. A query that
 * sees no key, or is padding, gets O = 0, LSE = -inf.
 * Keys and values that no query of the sequence sees may hold anything. A V row of a
 * 16-bit cache that some query of a row tile sees is multiplied by 0 for those that
 * do not, and has to be finite; one of a 4-bit cache that is not finite reaches only
 * the queries that see it.
 *
 * Over a 4-bit cache p carries V's step (a row without one counts as the larger of
 * 2^-60 and 2^-40 |low|): keys whose p is 2^-26 of the largest or more are all in
 * the sums while these lie within 2^100 of one another. Entries of Q stay below
 * 2^112.
 *
 * Every sum has an order that the sizes and positions alone decide: equal calls
 * give equal bits. Two kernels on `stream` (one where no workspace is needed), no
 * allocation. Errors before launch: as nsa_swa_fwd, the cache's and the
 * workspace's. A timed-out device wait is reported by nsa_sync_status.
 */
int nsa_paged_attn(const void* Q, const nsa_kv_cache* cache, const int32_t* page_table,
                   const int32_t* positions, void* O, float* LSE, int64_t B, int64_t M, int64_t H,
                   int64_t G, int64_t D, int64_t positions_stride, int64_t table_cols,
                   int64_t window_left, int64_t sinks, float scale, int dtype,
                   const int64_t* q_strides, void* workspace, int64_t workspace_bytes,
                   void* stream);

/*
 * nsa_sync_status -- wait for `stream`, then read and clear the device status
 * word of the current device.
 *
 * Every device-side wait of this library's kernels is bounded (1 s). A warp
 * whose wait gives up records it in a per-device status word, lets its own
 * copies in flight land, and returns without writing its outputs. This call
 * returns NSA_ERR_TIMEOUT if that happened in any launch since the last call,
 * NSA_ERR_LAUNCH if synchronising the stream reports a CUDA error, NSA_OK
 * otherwise. A library built with NSA_DEBUG_BOUNDS also checks, before every
 * K/V tile copy of the selection forward, that the tile starts on a 16-key
 * boundary, at or before the query's last visible key, inside a block of the
 * index range; a failed check is returned here as NSA_ERR_BOUNDS (ahead of a
 * timeout). It synchronises; it allocates nothing.
 */
int nsa_sync_status(void* stream);

/*
 * nsa_selftest_wait_timeout -- test hook for the bounded waits.
 *
 * Launches four warps on `stream`, one of which waits on a barrier nothing will
 * ever complete; after `limit_ns` (1e3 .. 2e9) it gives up, the others learn of
 * it and one of them sets the status word, so the next nsa_sync_status()
 * returns NSA_ERR_TIMEOUT. Touches no other memory. Returns NSA_ERR_SHAPE for a limit out of range.
 */
int nsa_selftest_wait_timeout(int64_t limit_ns, void* stream);

/*
 * nsa_probe_l2_gather -- measurement kernel: the gather of
 * nsa_sel_attn_fwd with nothing else, to measure the ceiling that gather
 * meets ("[wave] NSA: selection attention forward kernel", section "MI350
 * considerations": the irregular block gather is the most
 * performance-critical part of the kernel).
 *
 *   K, V            device, IEEE fp16, [N, G, D] (one batch), 16-byte aligned
 *   N               >= block_size; blocks 0 .. floor(N/block_size)-1 are drawn
 *   G, g            KV groups; the group read (0 <= g < G), or -1 for a
 *                   group drawn with every block (all groups interleaved)
 *   D               64 or 128
 *   block_size      32 or 64
 *   ctas            grid size (1 .. 2^31); size it as SMs x CTAs per SM
 *   warps_per_cta   1 .. 32
 *   slots_per_warp  1 .. 16 tiles each warp keeps in flight
 *   loads_per_warp  tiles each warp copies (>= 0)
 *   rows_per_box    key rows per TMA box and per tile: 16 (the forward's), 32
 *                   or 64, at most block_size
 *   seed            block draw seed
 *   cta_record      device int64 [ctas, 3] written with (SM id, start ns,
 *                   end ns) of every CTA (%globaltimer), or NULL
 *
 * Each warp copies loads_per_warp tiles of rows_per_box key rows x D (TMA
 * boxes of rows_per_box x 64, 128-byte swizzle, L2 evict_last: with 16 rows,
 * the forward's copies) into
 * shared memory, alternating K and V and walking the 16-key tiles of
 * randomly drawn blocks, keeping slots_per_warp copies in flight and doing
 * nothing with the data. The bytes moved, nsa_probe_l2_gather_bytes(), over
 * the kernel's time is the gather bandwidth this GPU delivers for that
 * access pattern and in-flight depth. Shared memory per CTA is
 * warps x slots x D/64 x rows_per_box x 128 B (+ 1 KB + barriers), within
 * 227 KB (else NSA_ERR_SHAPE). Asynchronous; allocates nothing. Errors:
 * NSA_ERR_NULL, NSA_ERR_ALIGN, NSA_ERR_HEAD_DIM, NSA_ERR_BLOCK_SIZE,
 * NSA_ERR_SHAPE, NSA_ERR_LAUNCH. A timed-out wait is reported by
 * nsa_sync_status.
 */
int nsa_probe_l2_gather(const void* K, const void* V, int64_t N, int64_t G, int64_t D,
                        int64_t g, int block_size, int64_t ctas, int warps_per_cta,
                        int slots_per_warp, int64_t loads_per_warp, int rows_per_box,
                        uint32_t seed, int64_t* cta_record, void* stream);

/* Bytes nsa_probe_l2_gather moves for these arguments (negative nsa_status
 * for invalid ones). Pure host arithmetic. */
int64_t nsa_probe_l2_gather_bytes(int64_t D, int64_t ctas, int warps_per_cta,
                                  int64_t loads_per_warp, int rows_per_box);

/*
 * nsa_probe_gather_rows -- measurement kernel: exactly the copies
 * nsa_sel_attn_fwd makes for these index rows, and nothing else.
 *
 *   K, V, block_indices, B, M, N, G, D, T, block_size
 *                   as for nsa_sel_attn_fwd (H plays no part: the copies are
 *                   per (b, m, g) row); same checks and errors
 *   ctas            grid size (1 .. 2^31 - 1)
 *   warps_per_cta   1 .. 32
 *   slots_per_warp  1 .. 16 copies each warp keeps in flight
 *   extra_smem_bytes  >= 0: unused shared memory added to each CTA, to
 *                   measure how the gather rate depends on the shared
 *                   memory a kernel reserves (total within 227 KB)
 *
 * Every warp takes the (b, g, m) rows w, w + W, w + 2W, ... (W warps in the
 * grid, m fastest) and walks each row as the forward does -- padding,
 * out-of-range ids and blocks after the query skipped, the 16-key tiles of
 * each selected block that start at or before the query -- copying the K
 * tile and then the V tile of every 16-key tile into shared memory (TMA
 * boxes of 16 x 64, 128-byte swizzle, L2 evict_last). It moves the bytes of
 * every whole 16-key tile the forward gathers, back to back across rows,
 * so the forward's gathered bytes over this kernel's time bound the
 * forward's gather rate from above for these rows. Shared memory and
 * asynchrony as nsa_probe_l2_gather; allocates nothing.
 */
int nsa_probe_gather_rows(const void* K, const void* V, const int32_t* block_indices, int64_t B,
                          int64_t M, int64_t N, int64_t G, int64_t D, int64_t T, int block_size,
                          int64_t ctas, int warps_per_cta, int slots_per_warp,
                          int64_t extra_smem_bytes, void* stream);

/*
 * nsa_probe_reduce_rows -- measurement kernel: the backward's dQ reductions
 * alone, to measure the rate they can reach on this GPU.
 *
 *   buf             device fp32, at least rows * stride floats, 16-byte
 *                   aligned; its contents are left unchanged (zeros are added)
 *   rows, stride    rows of 1024 floats (4 KB: 8 head rows of 128 dims, one
 *                   query and KV group of dQ), `stride` floats apart
 *                   (>= 1024, a multiple of 4); dQ of one KV group is
 *                   rows = B*M, stride = H*128
 *   ctas, warps_per_cta  grid (warps_per_cta 1 .. 32)
 *   iters_per_warp  rows each warp adds into
 *
 * Each warp adds one 4 KB row at a time into a row drawn at random, with
 * 16-byte fp32 reductions (red.global.add.v4.f32), as the key-major backward
 * kernel adds its dQ partial sums. Bytes reduced = ctas x warps x iters x
 * 4096. Asynchronous; allocates nothing. Errors: NSA_ERR_NULL,
 * NSA_ERR_ALIGN, NSA_ERR_SHAPE, NSA_ERR_LAUNCH.
 */
int nsa_probe_reduce_rows(float* buf, int64_t rows, int64_t stride, int64_t ctas,
                          int warps_per_cta, int64_t iters_per_warp, uint32_t seed,
                          void* stream);

#ifdef __cplusplus
}
#endif

#endif /* NSA_SEL_ATTN_H */
