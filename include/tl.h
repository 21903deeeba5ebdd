/*
 * tl.h - C ABI of the GB300 (sm_103a) tile-centric communication-overlapped GEMM library.
 *
 * The library computes, on ONE GPU, the four overlapped operators of the pages it is
 * built from, with the W tensor-parallel ranks emulated as W separate HBM buffers (and, further down,
 * the operators of a decoder's serving step: its plan, norms and rotation, cache append and gather, paged and
 * window attention, MoE for few tokens, log probabilities):
 *
 *   tl_ag_gemm      AllGather + GEMM:        C = [A_0; A_1; ...; A_{W-1}] . B
 *   tl_gemm_rs      GEMM + ReduceScatter:    out_o = rows_o( sum_p A_p . B_p )
 *   tl_mlp2         2-layer MLP chain:       out_o = rows_o( sum_r GELU(AG(X) . W1_r) . W2_r )
 *   tl_moe_combine  top-k MoE layer:         out_t = sum_j g_tj * (SiLU(x_t Wg_e) * (x_t Wu_e)) Wd_e
 *
 * "Communication" is the movement of shards between the ranks' buffers inside one HBM,
 * done by mover warps that publish per-chunk release flags; the persistent tcgen05 GEMM
 * waits on those flags (acquire) before its TMA loads, walking its tiles in a rank-swizzled
 * order that starts from the local shard.
 *
 * Sources (page titles; sections as printed on the pages):
 *   [TL] TileLink: Generating Efficient Compute-Communication Overlapping Kernels using
 *        Tile-Centric Primitives - §2.1 (tensor-parallel FFN), §3.1 (decoupled tile size /
 *        order / resource binding), §3.2 Table 3 (producer_tile_notify, consumer_tile_wait,
 *        peer_tile_notify/wait, tile_push_data, tile_pull_data), §4.1 (static and dynamic
 *        tile-centric mapping), §4.2 (release/acquire lowering), §6 (BlockChannel context).
 *   [TD] Triton-distributed: Programming Overlapping Kernels on Distributed AI Systems with
 *        the Triton Compiler - §2.1 (symmetric memory, signal exchange, async tasks),
 *        §3.2 Algorithm 2 (pull-mode AllGather), §3.3 Algorithm 3 (push-mode ReduceScatter),
 *        §3.7 (tile swizzle for AG+GEMM and GEMM+RS), §3.8 (signal reset, resource partition).
 *   [RA] Resource-aware Computation-Communication Overlap for multi-GPU ML Workloads -
 *        CTA-pipelining abstract (2-layer GEMM with CTA-level dependencies) and the MoE
 *        abstract (persistent expert producer, persistent combine consumer on a small
 *        dedicated SM partition, tile-level signalling).
 *
 * Conventions for every entry point
 *   - Matrices are row-major bf16 (IEEE bfloat16, passed as raw 16-bit storage), fp32 where
 *     stated.  Every device pointer must be 16-byte aligned.  Accumulation is fp32.
 *   - Ownership: the caller allocates every device buffer, including the workspace (size from
 *     the matching *_workspace_bytes function).  The library owns only the context (a small
 *     device status word).  No entry point allocates device memory.
 *   - A workspace must be zero-filled once before its first use (e.g. cudaMemset) and again
 *     after any call whose tl_ctx_check reported an error; between successful calls the
 *     library keeps it valid itself (its signals are epoch-valued, never reset).
 *   - Calls are asynchronous on `stream` and return once the work is enqueued.  Two calls that
 *     share a workspace must be ordered (same stream, or events).
 *   - Return values: TL_OK (0) or a negative TL_ERR_* code.  Argument errors are reported
 *     before anything is enqueued.  Device-side errors (a bounded wait that ran out) are read
 *     with tl_ctx_check after the stream has been synchronised.
 *   - Threading: a context is not thread-safe; use one per host thread.
 */
#ifndef TL_GB300_H
#define TL_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct CUstream_st; /* == cudaStream_t / CUstream */
typedef struct CUstream_st* tl_stream_t;

/* ---------------------------------------------------------------- status codes */
#define TL_OK 0
#define TL_ERR_INVALID (-1)     /* null / misaligned pointer, unsupported shape, bad config      */
#define TL_ERR_UNSUPPORTED (-2) /* device is not sm_103 / co-residency of the persistent grid fails */
#define TL_ERR_CUDA (-3)        /* a CUDA runtime or driver call failed                          */
#define TL_ERR_TIMEOUT (-4)     /* (tl_ctx_check) a bounded device wait on a signal ran out        */
#define TL_ERR_WORKSPACE (-5)   /* workspace smaller than *_workspace_bytes                     */
#define TL_ERR_INDEX (-6)       /* (tl_ctx_check) a slot, page or length read on the device was out of range */

/* ---------------------------------------------------------------- configuration
 * The BlockChannel-like launch context of [TL] §6: rank/world come per call; this struct
 * carries the decoupled design-space choices of [TL] §3.1 (communication tile size = mover
 * chunk, tile order = swizzle, resource binding = mover warps / combine partition) and the
 * bound on every device-side wait.
 */
typedef struct tl_config {
  int mover_warps;            /* warps per persistent CTA that move shards (1..4; default 4)          */
  int chunks_per_slab;        /* mover chunks, hence signals, per 128-row slab (1..32; default 32)     */
  int swizzle;                /* 0: identity tile order; 1: rank-swizzled ([TD] §3.7; default)          */
  int grid_ctas;              /* persistent CTAs; 0 = one per SM (default)                              */
  int combine_ctas;           /* MoE combine partition, CTAs = SMs ([RA]; default 8)                    */
  int debug_skip_chunk;       /* fault injection: this mover chunk is copied but never signalled (-1 off) */
  unsigned long long timeout_ns; /* bound of every device wait (default 2e9 ns)                       */
  int pair_ctas;              /* where shards / owner blocks are 256-row multiples, 256 x 256 tiles run
                                 on: 0 single CTAs; 1 CTA pairs (two SMs, tcgen05 cta_group::2) for
                                 every op; 2 (default) CTA pairs for tl_gemm_rs and tl_mlp2, whose
                                 heavier epilogues gain from the pair's double-buffered
                                 accumulators, single CTAs for tl_ag_gemm                           */
  int moe_renorm;             /* MoE gates: 0 (default) the softmax over all E logits taken at the
                                 chosen experts; 1 those values divided by their sum over the topk
                                 chosen experts (they then sum to 1 per token)                      */
  int rs_ring;                /* tl_gemm_rs reduction: 0 (default) the owner-slot chain; 1 a ring
                                 ([TL] §5, Figure 4 text), workspace from
                                 tl_gemm_rs_ring_workspace_bytes                                    */
  int ag_push;                /* tl_mlp2's AllGather, where every rank gathers: 0 (default) pull
                                 ([TD] §3.2 Algorithm 2, each rank reads every other shard); 1 push
                                 (Algorithm 1, each shard read once and written to the other ranks'
                                 copies).  tl_ag_gemm and tl_allgather gather into one rank, where
                                 both modes move the same bytes: they always pull              */
  int mover_kparts;           /* tl_ag_gemm's mover chunks along K ([TL] §3.1, the communication
                                 tile): 1 each chunk is whole rows of a 128-row slab; 2 or 4 each
                                 slab of the first two shards gathered is also cut into that many
                                 K parts (of at least 16 64-column k-blocks), copied part by
                                 part, and a tile waits for each part before its first k-block in
                                 it; 0 (default) 4.  tl_allgather and tl_mlp2 always copy whole
                                 rows (as measured on GB300, K parts only slow them)          */
  int ag_ll;                  /* tl_ag_gemm's gather protocol: 0 (default) pull with one signal
                                 per chunk; 1 low-latency push ([TD] §3.2 Algorithm 1 with the
                                 flag carried in every word): the remote shards' owners write
                                 8-byte words {bf16 x 2, call signal} into the workspace's LL
                                 slabs and each tile reads them straight into its operand
                                 buffer, with no separate signal or fence.  For small problems
                                 only (tl_ag_gemm_ll_capable); otherwise TL_ERR_UNSUPPORTED  */
  int mover_tma;              /* tl_allgather's copy engine: 0 (default) the SMs' load/store path
                                 (16-byte vectors, several CTAs of copy warps per SM); 1 the TMA
                                 unit of each SM (bulk copies through shared-memory stages, one
                                 issuing thread per SM): the pages' copy-engine mover ([TL]
                                 §7.2) in its GB300 form.  Same result and signals.          */
} tl_config;

typedef struct tl_ctx tl_ctx;

/* Fill *cfg with the defaults above.  Returns TL_OK, or TL_ERR_INVALID for cfg == NULL. */
int tl_config_default(tl_config* cfg);

/* Create a context on `device` (must be compute capability 10.3, i.e. sm_103).  cfg may be
 * NULL (defaults).  Allocates one small device status word.  On failure *out is NULL. */
int tl_ctx_create(tl_ctx** out, int device, const tl_config* cfg);

/* Destroy a context (NULL is ignored).  Synchronises the device first. */
void tl_ctx_destroy(tl_ctx* ctx);

/* Read and clear the device status word.  Call after synchronising the streams used with ctx.
 * Returns TL_OK, or TL_ERR_TIMEOUT if a bounded wait ran out (the results of that call are
 * undefined and its workspace must be zero-filled again), or TL_ERR_INDEX if a serving operator
 * met an index out of range (it left that entry out; its workspace stays valid), or TL_ERR_CUDA.
 * If both happened since the last check, in whatever order, it is TL_ERR_TIMEOUT. */
int tl_ctx_check(tl_ctx* ctx);

/* Human-readable text for a status code (static storage). */
const char* tl_strerror(int code);

/* Library version, major*10000 + minor*100 + patch. */
int tl_version(void);

/* Number of SMs / persistent CTAs the context launches with. */
int tl_ctx_num_ctas(const tl_ctx* ctx);

/* ---------------------------------------------------------------- trace buffer
 * A per-CTA timeline of the persistent kernels.  Every warp role records spans into a
 * caller-owned device buffer.  A span is a %globaltimer start, a duration in ns, and a kind
 * plus a tile or chunk index.  The pages name no such facility.  It shows where a fused kernel
 * waits: a mover chunk landing, a tile waiting on its signal, the MMA warp starved of data.
 *
 * tl_trace_bytes(ctas, spans_per_warp): bytes a buffer needs to hold `ctas` CTAs.
 * tl_ctx_set_trace(ctx, buf, bytes, spans_per_warp): every later persistent-kernel launch on
 *   ctx records into buf.  buf is device memory, 16-byte aligned and caller-owned; it must stay
 *   valid while such launches run.  buf NULL turns tracing off.  Each launch overwrites the
 *   previous trace.  CTAs beyond what `bytes` holds are not recorded.  Spans beyond
 *   spans_per_warp are dropped, but the per-warp count still counts them.
 *   Returns TL_ERR_INVALID for a null ctx, a misaligned buf, a size below
 *   tl_trace_bytes(1, spans_per_warp), or spans_per_warp < 1.
 * Layout (little-endian), written by the kernels:
 *   uint32 header[8]: magic 0x544c5452, version 1, grid of the last launch, warps per CTA (16),
 *                     spans per warp, CTAs held, 0, 0
 *   uint32 count[CTAs held][16]: spans each warp recorded (may exceed spans per warp)
 *   span[CTAs held][16][spans per warp], 16 bytes each: uint64 t0_ns, uint32 dur_ns,
 *                     uint32 tag = kind << 24 | index
 * Kinds:
 *   1 producer tile; 2 producer signal wait; 3 producer ring-stall total (t0 = tile start);
 *   4 MMA tile; 5 MMA starve total (t0 = tile start); 6 MMA accumulator wait;
 *   7 epilogue tile; 8 epilogue accumulator wait;
 *   9 mover chunk; 10 side-partition unit (from the start of its wait); 11 side-partition wait.
 * Waits shorter than 200 ns are not recorded.
 * Warp w of a GEMM CTA: 0 producer, 1 MMA, 2.. epilogue, then the movers.  In a side partition
 * (the MoE combine CTAs) warps 0 and 4 record.  Only the persistent kernels trace.  While on,
 * tracing costs a few timer reads per tile and k-block.
 */
size_t tl_trace_bytes(int ctas, int spans_per_warp);
int tl_ctx_set_trace(tl_ctx* ctx, void* buf, size_t bytes, int spans_per_warp);

/* ---------------------------------------------------------------- AllGather + GEMM
 * [TL] §2.1, [TD] §3.2 Algorithm 2 (pull mode) and §3.7 (AG+GEMM swizzle).
 *
 *   C[(W*m_per_rank) x n] = A . B,  A = [A_0; ...; A_{W-1}] (rank order), B [k x n].
 *
 * a_shards: host array of W device pointers, shard r is bf16 [m_per_rank x k] (rank r's
 *           "local buffer").  b: bf16 [k x n].  c: bf16 [(W*m_per_rank) x n] (output).
 * workspace: device buffer of tl_ag_gemm_workspace_bytes(); its first W*m_per_rank*k*2
 *           bytes are the gathered A (the symmetric buffer T of Algorithm 2, rank order), the
 *           rest holds the per-chunk ready signals.
 * The emulated self rank `rank` (0 <= rank < W) reads its own shard in place; the mover pulls
 * the remote shards (rank+1) mod W, (rank+2) mod W, ... into their slots of T in that order,
 * and the GEMM visits row blocks of shard rank first, then (rank+1) mod W, ... waiting on each
 * slab's signals before its first load.  The self rank's slot of T is not written (nothing
 * reads it; tl_allgather fills all W slots).  The result does not depend on `rank` or the
 * swizzle.
 * W = 1 has nothing to gather: the call is the plain GEMM on shard 0, read in place, and the
 * gathered region of the workspace is not written.
 * Shapes: 1 <= W <= 8; m_per_rank % 128 == 0; n % 8 == 0; k % 8 == 0 (n, k need not be
 * tile multiples: ragged edges are zero-filled by TMA on load and clipped on store).
 * Any zero dimension is a no-op returning TL_OK.
 * Low-latency gather (cfg.ag_ll = 1, W > 1): instead of the mover and its chunk signals, the
 * owners of the remote shards push them as LL words {bf16 x 2, low 32 bits of the call's
 * signal} into the workspace's LL slabs, after the signal words, and every 128 x 256 output
 * tile reads the words of its rows straight into its operand buffer, polling only those that
 * do not carry this call's signal yet.  The gathered region is not written.  The result is
 * the same operation; for m_per_rank % 256 != 0 it is bit-identical to the pull path (the
 * same 128-row MMAs in the same k order).  Only problems with W * m_per_rank * k <= 2^20
 * (their workspace has the LL slabs) and at most (the context's CTAs - 1) output tiles can
 * take it (tl_ag_gemm_ll_capable); others return TL_ERR_UNSUPPORTED with nothing enqueued.
 * The LL slabs need no zeroing between calls on one context.
 */
size_t tl_ag_gemm_workspace_bytes(int W, int m_per_rank, int n, int k);
int tl_ag_gemm(tl_ctx* ctx, int W, int rank, const void* const* a_shards, const void* b, void* c,
               void* workspace, size_t workspace_bytes, int m_per_rank, int n, int k, tl_stream_t stream);
/* 1 if tl_ag_gemm on ctx with cfg.ag_ll = 1 runs the low-latency gather for this shape, else 0
 * (also 0 for a NULL ctx or a negative size; W = 1 has nothing to gather: 0). */
int tl_ag_gemm_ll_capable(const tl_ctx* ctx, int W, int m_per_rank, int n, int k);

/* ---------------------------------------------------------------- AllGather alone
 * [TD] §3.2 Algorithm 2 (pull-mode one-sided AllGather) as its own kernel: the shard mover of
 * tl_ag_gemm (same chunk order and signals, whole-row chunks) without the GEMM, run by four
 * CTAs of 16 warps per SM, two resident at a time (alone, the copy has the whole GPU).  Fills
 * the gathered buffer at the start of `workspace` (sized by tl_ag_gemm_workspace_bytes(W,
 * m_per_rank, 8, k)) with all of
 * [A_0; ...; A_{W-1}], the self rank's shard last, and releases every chunk signal.  Shapes
 * and errors as tl_ag_gemm; W = 1 is a no-op.  This is the "communication alone" leg of the
 * overlap measurement.
 */
int tl_allgather(tl_ctx* ctx, int W, int rank, const void* const* a_shards, void* workspace, size_t workspace_bytes,
                 int m_per_rank, int k, tl_stream_t stream);

/* ---------------------------------------------------------------- GEMM + ReduceScatter
 * [TD] §3.3 Algorithm 3 (each producer pushes its partial into the owner's slot, the owner
 * accumulates), [TL] §5 / Figure 4 text (producer tiles notify; peer tiles chain the partial
 * sums from rank to rank) and [TD] §3.7 (start at the next rank's chunk, own chunk last).
 *
 *   out_o [(m/W) x n] = rows [o*m/W, (o+1)*m/W) of  sum_{p=0}^{W-1} A_p . B_p
 *
 * a: W device pointers, A_p bf16 [m x k_r];  b: W device pointers, B_p bf16 [k_r x n];
 * out: W device pointers, out_o bf16 [(m/W) x n].
 * Owner-slot chain (cfg.rs_ring = 0, default).  workspace: tl_gemm_rs_workspace_bytes(): an
 * fp32 [m x n] accumulation slot (owner o owns rows o*m/W..) plus one signal per 128-row block
 * and 256-column block of the output.  The output is walked in bands of 2048 rows x 4096
 * columns; inside a band the producers run p = 0..W-1, producer p starting at the rows of
 * owner (p+1) mod W when the band holds some (swizzle = 1).  Producer 0 stores its partial
 * tile into the slot, producer p > 0 waits for producer p-1's signal on that tile
 * (peer_tile_wait) and adds its partial with a TMA bulk reduction, and producer W-1 adds its
 * partial to the slot in registers and writes bf16 out_o.  The fp32 summation order is fixed
 * (p = 0, 1, ..., W-1): results are bit-identical across runs, swizzle modes and grid sizes.
 * Ring (cfg.rs_ring = 1).  workspace: tl_gemm_rs_ring_workspace_bytes(): W fp32 [m x n]
 * receive buffers (rank q's at q*m*n*4 bytes), then the signals.  The partial of an output
 * tile of owner o starts at rank o+1 and travels o+1 -> o+2 -> ... -> o (mod W): each rank
 * waits for its predecessor's signal on the tile (peer_tile_wait), adds the partial in its
 * receive buffer to its own, stores the sum into the next rank's receive buffer and signals
 * it (peer_tile_notify); the owner, last, writes bf16 out_o.  The fp32 order of owner o's
 * rows is P_{o+1} + P_{o+2} + ... + P_o: fixed, so results are bit-identical run to run.
 * Shapes: 1 <= W <= 8; m % (128*W) == 0; n % 8 == 0; k_r % 8 == 0.
 */
size_t tl_gemm_rs_workspace_bytes(int W, int m, int n, int k_r);
size_t tl_gemm_rs_ring_workspace_bytes(int W, int m, int n, int k_r);
int tl_gemm_rs(tl_ctx* ctx, int W, const void* const* a, const void* const* b, void* const* out,
               void* workspace, size_t workspace_bytes, int m, int n, int k_r, tl_stream_t stream);

/* ---------------------------------------------------------------- ReduceScatter alone
 * [TD] §3.3 Algorithm 3 (push-mode ReduceScatter) as its own kernel, without a GEMM: the
 * communication half of tl_gemm_rs, and its "communication alone" leg in an overlap
 * measurement.
 *
 *   out_o [(m/W) x n] = rows [o*m/W, (o+1)*m/W) of  P_0 + P_1 + ... + P_{W-1}
 *
 * partials: host array of W device pointers, P_p fp32 [m x n] row-major (rank p's partial);
 * out: W device pointers, out_o bf16 [(m/W) x n].  The sum is taken in fp32 in the order
 * p = 0, 1, ..., W-1 (the order of tl_gemm_rs's chain) and rounded to bf16 once, so the
 * result is bit-identical run to run.  No workspace.  Partials are read once.
 * Shapes: 1 <= W <= 8; m % W == 0; n % 4 == 0.  m == 0 or n == 0 is a no-op.
 */
int tl_reduce_scatter(tl_ctx* ctx, int W, const float* const* partials, void* const* out, int m, int n,
                      tl_stream_t stream);

/* ---------------------------------------------------------------- 2-layer MLP chain
 * [TL] §2.1 (AG + GEMM -> activation -> GEMM + RS), [RA] CTA-pipelining (the second GEMM's
 * CTAs start as soon as the first GEMM's CTAs that produce their inputs are done).
 *
 *   X = [X_0; ...; X_{W-1}]  (tokens x hidden),   H_r = GELU(X . W1_r)  (exact erf GELU),
 *   out_o = rows_o( sum_r H_r . W2_r ).
 *
 * x_shards: W pointers, X_r bf16 [(tokens/W) x hidden]; w1: W pointers, bf16 [hidden x f_r];
 * w2: W pointers, bf16 [f_r x hidden]; out: W pointers, bf16 [(tokens/W) x hidden].
 * workspace: tl_mlp2_workspace_bytes(): per-rank gathered X (W x tokens x hidden bf16; rank
 * r's own shard is read in place, its slot of r's copy is not written) at offset 0, then, each at the next 256-byte boundary, the intermediate H (W x tokens x f_r bf16,
 * H_r at rows r*tokens.., readable after the call), the fp32 reduction slot (tokens x hidden)
 * and the signals.
 * One persistent launch runs, per emulated rank r: the mover (gather X into rank r's copy, by
 * pull or, with cfg.ag_push, push), layer-1 tiles (wait for each K quarter of their gathered
 * rows, GELU epilogue, notify per H tile) and layer-2 tiles (wait on the H tiles covering their
 * K range, then the owner-slot GEMM+RS chain; cfg.rs_ring does not apply here).
 * Shapes: 1 <= W <= 8; tokens % (128*W) == 0; hidden % 8 == 0; f_r % 8 == 0.
 */
size_t tl_mlp2_workspace_bytes(int W, int tokens, int hidden, int f_r);
int tl_mlp2(tl_ctx* ctx, int W, const void* const* x_shards, const void* const* w1, const void* const* w2,
            void* const* out, void* workspace, size_t workspace_bytes, int tokens, int hidden, int f_r,
            tl_stream_t stream);

/* ---------------------------------------------------------------- MoE layer with combine partition
 * [TL] §4.1 (dynamic mapping tables filled by the routing), §7.2 (Gather + GroupGEMM, then
 * GroupGEMM + Scatter + TopK reduce), [RA] MoE abstract (persistent expert producer; a
 * persistent combine consumer on `combine_ctas` dedicated SMs that handles output tiles as
 * their ready signals arrive; the GEMM partition's CTAs join it after their last GEMM tile,
 * each y tile claimed once at run time).
 *
 * x: bf16 [T x H]; logits: fp32 [T x E]; w_gate, w_up: bf16 [E x H x F]; w_down: bf16 [E x F x H].
 * out: fp32 [T x H] (written, not accumulated into).
 * perm_out (optional, may be NULL): int32 [T*topk]: perm_out[pos] = t*topk + j, assignments
 *   ordered by (expert, t, j).  counts_out (optional): int32 [E] assignments per expert.
 * Routing: experts = the topk largest logits (ties to the lower expert index), gates = softmax
 * over all E logits taken at those experts; with cfg.moe_renorm = 1 the topk gates of a token
 * are divided by their sum (the pages define no router: both readings are offered).
 *   y_(t,j) = (SiLU(x_t . Wg_e) * (x_t . Wu_e)) . Wd_e   (h kept in bf16, y in bf16)
 *   out_t   = sum_j gate_(t,j) * y_(t,j)                  (fp32)
 * workspace: tl_moe_workspace_bytes().
 * Three launches: the routing (a warp per token), the permutation and tile tables (a CTA per
 * expert, while the remaining CTAs zero `out`), then one persistent launch of one CTA per SM
 * whose GEMM partition runs the gather and the grouped GEMMs while the combine partition adds
 * finished y tiles into `out`.  The second and third are dependent launches (programmatic
 * stream serialization): each starts while the one before it runs and waits for it before
 * reading its results.  TL_ERR_UNSUPPORTED if the device cannot hold the persistent grid at
 * once.
 * Shapes: T >= 1; 1 <= topk <= 8; topk <= E <= 256; H % 256 == 0; F % 128 == 0.
 */
size_t tl_moe_workspace_bytes(int T, int H, int E, int F, int topk);
/* The tile order of tl_moe_combine's persistent kernel, for host-side checks ([TL] §4.1: the
 * tile-to-work mapping is filled at run time; here the closed form behind it).  m_tiles is
 * the number of 128-row padded row tiles the routing produced (sum over experts of
 * ceil(count_e / 128)); 0 <= m_tiles <= the bound the workspace is sized for.
 * tl_moe_tile_order: for t = 0..count-1, the tile's kind (1 = gate/up, 2 = down), row tile
 *   and column block (128 columns of F for kind 1, 256 columns of H for kind 2).
 * tl_moe_combine_order: for v = 0..count-1, the row tile and column block of the v-th y tile
 *   the combine claims.
 * Both return the number of tiles, or TL_ERR_INVALID (bad shape, m_tiles out of range, or
 * arrays shorter than `cap`).  Arrays may all be NULL to query the count.  Host only. */
int tl_moe_tile_order(int T, int H, int E, int F, int topk, int m_tiles, int* kind, int* row_tile, int* col_block,
                      int cap);
int tl_moe_combine_order(int T, int H, int E, int F, int topk, int m_tiles, int* row_tile, int* col_block, int cap);
int tl_moe_combine(tl_ctx* ctx, const void* x, const float* logits, int topk, const void* w_gate,
                   const void* w_up, const void* w_down, float* out, int* perm_out, int* counts_out,
                   void* workspace, size_t workspace_bytes, int T, int H, int E, int F, tl_stream_t stream);

/* ---------------------------------------------------------------- AllGather KV + self-attention
 * [TL] §5 (AllGather KV + self-attention: the KV cache sequence split into W equal shards)
 * and §7.2 (sequence-parallel self-attention; Table 4 Attn-1/Attn-2: head dim 128); [TD] §3.7
 * (the local shard first).  Non-causal (the pages give no mask):
 *   out[h] = softmax(q[h] K[h]^T / sqrt(d)) V[h],  K = [K_0 | K_1 | ... | K_{W-1}] along the
 *   sequence (rank order), V likewise.
 * q: bf16 [heads x l_r x d] (this rank's queries).  k_shards, v_shards: host arrays of W device
 * pointers, shard r bf16 [heads x l_r x d].  out: bf16 [heads x l_r x d].
 * workspace: tl_ag_attention_workspace_bytes(): the gathered K and V, shard-major
 * [W x heads x l_r x d] (shard r at r, filled completely, the local shard last), one signal
 * per (shard, head, 128-key block), and room for the partial results of split items (below).
 * One persistent launch of CTA pairs (clusters of 2, one CTA per SM): mover warps pull the
 * remote shards' K/V blocks into the gathered buffers and release each block's signal; the
 * attention of each (head, 256-query tile) reads its own shard in place first and a remote
 * shard's blocks once all of them are signalled.  The pages run this gather on the copy
 * engine from a second stream; that makes the kernel wait on work outside its own launch,
 * which nothing guarantees to run alongside it, so the gather runs inside the kernel, as for
 * tl_ag_gemm.  When the (head, tile) items leave the last wave of pairs less than half full,
 * those last items are each split into two halves of their keys that run on two pairs; the
 * half that finishes second combines both (in a fixed order: the result does not depend on
 * which finished first).
 * Shapes: 1 <= W <= 8; d == 128; any l_r (a shard's last 256-key block and the last 256-query
 * tile may be partial).  heads == 0 or l_r == 0 is a no-op.
 */
size_t tl_ag_attention_workspace_bytes(int W, int heads, int l_r, int d);
int tl_ag_attention(tl_ctx* ctx, int W, int rank, const void* q, const void* const* k_shards,
                    const void* const* v_shards, void* out, void* workspace, size_t workspace_bytes,
                    int heads, int l_r, int d, tl_stream_t stream);

/* ---------------------------------------------------------------- AllGather + GEMM without allocation
 * The pages have no counterpart of this entry point.  It exists for callers that cannot
 * allocate device memory when they call in: code being recorded into a CUDA graph by stream
 * capture (cudaMalloc cannot be recorded), plug-ins whose host framework owns the allocator
 * and gives out no scratch, and real-time paths that forbid allocation after start-up.
 *
 * Same operation, arguments, shapes and result as tl_ag_gemm, minus the workspace: the
 * gathered operand and the chunk signals live in a fixed device array of
 * TL_AG_GEMM_STATIC_SCRATCH_BYTES inside the library, which every GPU that loads the library
 * keeps until the process exits.  A problem whose tl_ag_gemm_workspace_bytes() exceeds that
 * size is rejected with TL_ERR_WORKSPACE before anything is enqueued.  The entry point
 * allocates nothing (no cudaMalloc, cudaFree or allocating library call).  Its first call on a
 * device looks up the array's device address with that device current; make that first call
 * before any stream capture begins.  The address is kept for the life of the process: after
 * cudaDeviceReset on that device (or anything else that destroys its primary context) the
 * entry point must not be called on that device again.  Every argument check (those of
 * tl_ag_gemm, then the size check) runs before anything is enqueued.  All calls share the one
 * array (each call clears the signals and overwrites the gathered operand), so calls whose GPU
 * work overlaps in time race and give undefined results: order them on one stream or with
 * events.
 */
#define TL_AG_GEMM_STATIC_SCRATCH_BYTES (16u << 20)
int tl_ag_gemm_static_scratch(tl_ctx* ctx, int W, int rank, const void* const* a_shards, const void* b, void* c,
                              int m_per_rank, int n, int k, tl_stream_t stream);

/* ---------------------------------------------------------------- serving: types and the paged cache
 * The operators of a decoder's serving step: the plan of its tokens in the cache, the norms and the rotation of
 * queries and keys, the cache append and gather, the attention of one new token over the cache, the causal
 * attention of prompts, the MoE layer for a few tokens, and the log probabilities of the chosen ones.  The
 * pages have no counterpart of these entry points.  They are the single-GPU steps that
 * run between the overlapped operators when a model answers, on the same buffers and streams.
 *
 * Types: bf16 or fp16 activations; a cache holds the activations' type, or e4m3 (8-bit float, 4
 * exponent and 3 mantissa bits, no infinity) with one fp32 scale per kv head: the value that a
 * stored byte b stands for is scale * b; or 4 bits (e2m1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign, two values a
 * byte, the lower half first) with an e4m3 scale for every block of 16 values of a row beside the head's: the value
 * that a code c stands for is c * block scale * scale.
 * Rows: the innermost dimension (d) is contiguous; every other stride is the caller's, in
 * elements (of a 4-bit cache in bytes), a multiple of 16 bytes.  So a view of a fused projection's output, or a cache that is
 * token-major [pages][page_size][kv_heads][d] or head-major [pages][kv_heads][page_size][d], is
 * passed as it is.
 * Indices read on the device (slots, page numbers, lengths, tokens) are checked there: an entry out of
 * range is left out, nothing outside the buffers is read or written, and tl_ctx_check returns
 * TL_ERR_INDEX.  All of them can be captured into a graph and replayed.
 * Workspaces: the first TL_SERVE_COUNTER_BYTES hold counters that each call leaves at zero again.  So one
 * workspace, zero-filled once, serves calls of tl_paged_attention, tl_moe_tokens and tl_token_logprobs of any shapes, in
 * order; after another operator used it, those bytes have to be zero-filled again.
 */
#define TL_SERVE_COUNTER_BYTES 139264
#define TL_BF16 0
#define TL_FP16 1
#define TL_E4M3 2
#define TL_FP32 3
#define TL_E2M1 4

typedef struct tl_paged_cache {
  void* k;                /* the K rows of all pages                                            */
  void* v;                /* the V rows; the same strides as k                                  */
  const float* k_scale;   /* e4m3, e2m1: fp32 [kv_heads] (NULL: all 1); otherwise NULL           */
  const float* v_scale;
  long long page_stride;  /* elements (e2m1: bytes) from a page to the next                     */
  long long row_stride;   /* elements from a row (token) of a page to the next                  */
  long long head_stride;  /* elements from a kv head to the next                                */
  int dtype;              /* TL_BF16, TL_FP16, TL_E4M3 or TL_E2M1                                */
  int num_pages;
  int page_size;          /* rows in a page, any number >= 1                                    */
  int kv_heads;
  int d;                  /* head dim: 64 or 128                                                */
  /* only read where dtype is TL_E2M1: the e4m3 block scales, d / 16 bytes a row, with strides of their own
     (bytes, multiples of d / 16); both 16-byte aligned */
  void* k_blocks;
  void* v_blocks;
  long long block_page_stride;
  long long block_row_stride;
  long long block_head_stride;
} tl_paged_cache;

/* ---------------------------------------------------------------- plan of a step's tokens in the cache
 * Sequence b holds lengths[b] rows and gets counts[b] new ones (counts NULL: one each).  Its rows lie in pages
 * page_table[b][0 ..]; pages that it still needs are taken from free_pages, from entry *taken on, in the order of
 * the sequences.  The call writes
 *   page_table[b][i]  the new pages' entries (the others are left as they are),
 *   cu_q              int32 [batch + 1]: bounds of the packed new tokens (the first at 0),
 *   slots, positions  int32 [tokens]: of each packed new token its slot, page * page_size + row, as tl_kv_append takes it,
 *                     and its position in its sequence; from cu_q[batch] on (padding) -1 and 0,
 *   new_lengths       int32 [batch]: lengths with the new rows, as tl_paged_attention takes them,
 *   *taken_out        the entries of free_pages taken so far,
 *   cu_k              int32 [batch + 1] (may be NULL): bounds of the packed rows, old and new,
 *   kv_slots          int32 [kv_tokens] (may be NULL): the slot of every row, as tl_kv_gather takes it; -1 from cu_k[batch] on.
 * new_lengths may be lengths, and taken_out may be taken: a captured step then goes on by itself with each replay.
 * The other outputs must not overlap the inputs (page_table is both).
 * Reported (tl_ctx_check: TL_ERR_INDEX), with nothing written outside the buffers: a negative length or count, or more
 * rows than max_pages * page_size (the sequence counts as one without new tokens, of no rows if its length is
 * wrong); tokens beyond `tokens`, or pages beyond num_free (the sequence gets none of its new rows: its tokens have slot
 * -1, its length stays); rows beyond kv_tokens (their slots are left out); a page that is negative (slot -1); a
 * *taken outside 0..num_free (nothing can be taken).
 * Shapes: batch <= 4096; page_size >= 1; (max_pages + 1) * page_size < 2^31.  No workspace.
 */
int tl_cache_plan(tl_ctx* ctx, const int* lengths, const int* counts, int batch, int page_size, int* page_table,
                  int max_pages, const int* free_pages, int num_free, const int* taken, int* taken_out, int* new_lengths,
                  int* cu_q, int* cu_k, int* slots, int* positions, int tokens, int* kv_slots, int kv_tokens,
                  tl_stream_t stream);

/* ---------------------------------------------------------------- norms and rotation of queries and keys
 * Each row x of d values (one head of one token) of q and of k becomes, in one pass,
 *   y = x / sqrt(mean(x^2) + eps) * weight                              (no weight: y = x)
 *   (y_i, y_j) -> (y_i cos a - y_j sin a, y_i sin a + y_j cos a),        a = positions[token] * inv_freq[p]
 * for the pairs p = 0 .. rotary / 2 - 1 of its first `rotary` values: (i, j) = (p, p + rotary / 2), or with
 * interleaved = 1 (2p, 2p + 1).  The other values are not turned.
 * q, k and the outputs: dtype (TL_BF16 or TL_FP16) [tokens x heads (kv_heads) x d], strides as given; an output may be
 * its input (the same pointer and strides), and must not overlap it otherwise.  q_weight, k_weight: [d] of
 * weight_dtype (dtype or TL_FP32), or NULL: no norm.  positions: int32 [tokens], any value; inv_freq: fp32
 * [rotary / 2], finite (both may be NULL if rotary is 0).
 * Precision: all sums and products are fp32, rounded once; a row whose squares pass fp32's range becomes 0 (one
 * whose squares lie below it is scaled first, so eps may be 0).  Angles are held
 * as fractions of a turn in 64 bits, so that far positions lose nothing (off by 2^-31 turns where |inv_freq| <= 1);
 * sines and cosines are off by 2^-21 at most.
 * Shapes: d 64 or 128; rotary a multiple of 16, at most d; eps >= 0; heads + kv_heads <= 65536; tokens < 2^30.  tokens == 0 or no
 * heads is a no-op.  No workspace.
 */
int tl_norm_rope(tl_ctx* ctx, int dtype, const void* q, long long q_token_stride, long long q_head_stride, const void* k,
                 long long k_token_stride, long long k_head_stride, const void* q_weight, const void* k_weight,
                 int weight_dtype, float eps, const int* positions, const float* inv_freq, int rotary, int interleaved,
                 void* q_out, long long q_out_token_stride, long long q_out_head_stride, void* k_out,
                 long long k_out_token_stride, long long k_out_head_stride, int tokens, int heads, int kv_heads, int d,
                 tl_stream_t stream);

/* ---------------------------------------------------------------- append to a paged cache
 *   K[slot / page_size][slot % page_size][h] = k[t][h], V likewise, for slot = slots[t]
 *
 * k, v: dtype (TL_BF16 or TL_FP16) [tokens x kv_heads x d] with the strides given.  slots: int32
 * [tokens]; a negative slot skips its token (padding); one >= num_pages * page_size is left out
 * and reported.  Two tokens with the same slot: either may end up there, row by row (in a 4-bit cache block by block, and
 * a block's codes may be one's and its scale the other's).
 * A cache of the activations' type takes the rows as they are.  An e4m3 cache takes
 * k / k_scale[h], computed in fp32, rounded to nearest even and saturated at +-448 (infinities
 * too; NaN stays NaN).  A 4-bit cache takes, for each block of 16 values x and s = k_scale[h] (finite, > 0), the scale
 * b = e4m3(max |x| / (6 s)) and the codes e2m1(x / (b s)), each product and quotient in fp32, each conversion to nearest even and
 * saturating (infinities too); a block with b = 0 is all 0, a NaN makes its whole block NaN.
 * Shapes: d 64 or 128; num_pages * page_size < 2^31; tokens * kv_heads < 2^30.  tokens == 0 or kv_heads == 0 is a no-op.
 */
int tl_kv_append(tl_ctx* ctx, const tl_paged_cache* cache, int dtype, const void* k, const void* v,
                 long long k_token_stride, long long k_head_stride, long long v_token_stride,
                 long long v_head_stride, const int* slots, int tokens, tl_stream_t stream);

/* ---------------------------------------------------------------- rows of a paged cache, packed
 *   k[t][h] = K[slot / page_size][slot % page_size][h], v likewise, for slot = slots[t]
 *
 * The way back: the rows that a later turn's queries need beside the new ones (tl_window_attention takes packed rows; the
 * slots are tl_cache_plan's kv_slots).  k, v: dtype [tokens x kv_heads x d], strides as given; the values that the cache's
 * rows stand for, computed in fp32 and rounded once (a cache of dtype: as they are).  A negative slot leaves its
 * row of k and v as it is; one >= num_pages * page_size too, and is reported.
 * Shapes as tl_kv_append.
 */
int tl_kv_gather(tl_ctx* ctx, const tl_paged_cache* cache, int dtype, const int* slots, int tokens, void* k, void* v,
                 long long k_token_stride, long long k_head_stride, long long v_token_stride, long long v_head_stride,
                 tl_stream_t stream);

/* ---------------------------------------------------------------- attention of one new token
 * One query row per sequence over that sequence's rows of a paged cache.  n = lengths[b] counts
 * the rows in the cache, the new token's own among them (append it first).  Row j is visible if
 *   j < n  and  (window == 0  or  j >= n - window  or  j < sinks):
 * a sliding window of the last `window` tokens beside the first `sinks` ones.  Row j of sequence
 * b is row j % page_size of page page_table[b][j / page_size].
 *   out[b][h] = sum_j p_j V_j[h / G],  p = softmax_j(scale * q[b][h] . K_j[h / G]),  G = heads / kv_heads
 *   lse[b][h] = log sum_j exp(scale * q . K_j)         (fp32, natural log; lse may be NULL)
 * A sequence with nothing visible (n == 0), or only scores of -inf, has out = 0 and lse = -inf.  Rows that are not visible
 * are not read: whatever they hold has no effect.
 * q, out: dtype (TL_BF16 or TL_FP16) [batch x heads x d] with the strides given (out must not
 * overlap q).  cache: dtype, TL_E4M3 or TL_E2M1.  page_table: int32 [batch x max_pages], dense; only the entries
 * of visible rows are read.  lengths: int32 [batch]; a length over max_pages * page_size is cut to
 * that and reported, a page out of range is left out (its rows are not visible) and reported.
 * workspace: tl_paged_attention_workspace_bytes(): counters, and partial results of sequences split
 * over several CTAs.
 * Shapes: batch <= 4096; heads % kv_heads == 0; d 64 or 128; window, sinks >= 0; max_pages *
 * page_size < 2^31; scale > 0 and at most 2.358e38 (times log2(e) finite); batch * heads * (visible rows at most / 64 + 1) < 2^31.
 * A 4-bit cache's codes reach over less than 2^32 units of the largest power of two that divides their strides (rows side by
 * side, d 64: 128 GB), its block scales likewise.
 * batch == 0 or heads == 0 is a no-op.
 * Precision: scores, weights and all sums are fp32.  Where a weight meets V it is a sum of two terms of dtype, off by
 * half a step squared (over a 4-bit cache of fp16); with an e4m3 cache one fp16 term, and in tl_window_attention one
 * term of dtype, off by half a step.  fp16 terms are also off by up to 2^-32 of the largest weight.  The division by the weights' sum comes
 * last, and a weight may be 2^8 until then: sums of bf16 rows within 2^-8 / n of fp32's largest value can overflow.
 * The result does not depend on what else runs, and is bit-identical run to run on one device.
 */
size_t tl_paged_attention_workspace_bytes(int batch, int heads, int kv_heads, int d);
int tl_paged_attention(tl_ctx* ctx, const tl_paged_cache* cache, int dtype, const void* q, long long q_seq_stride,
                       long long q_head_stride, const int* page_table, int max_pages, const int* lengths, void* out,
                       long long out_seq_stride, long long out_head_stride, float* lse, int batch, int heads,
                       float scale, int window, int sinks, void* workspace, size_t workspace_bytes,
                       tl_stream_t stream);

/* ---------------------------------------------------------------- causal attention of prompts
 * A batch of sequences packed one after the other: sequence b has the query rows
 * [cu_q[b], cu_q[b+1]) and the key/value rows [cu_k[b], cu_k[b+1]).  Its last query stands at its
 * last key: query i of n_q stands at p = n_k - n_q + i (n_k > n_q continues a sequence whose first
 * keys were there already).  Key j is visible to it if
 *   j <= p  and  (window == 0  or  j > p - window  or  j < sinks).
 *   out[i][h] = softmax_j(scale * q[i][h] . k[j][h / G]) . v[j][h / G],  lse as tl_paged_attention.
 * A query with nothing visible (p < 0), or only scores of -inf, has out = 0 and lse = -inf.  A key that is not visible to a
 * query has no effect on it, whatever it holds (infinities and NaN too).
 * Infinities and NaN in v cost time: results that they make non-finite are computed twice, the second time more
 * slowly (about 20 times a whole call's time if every query sees one).  In k they cost none.
 * q, out: dtype [total_q x heads x d]; k, v: dtype [total_k x kv_heads x d], strides as given (out
 * must not overlap the inputs).  lse: fp32 [total_q x heads] or NULL.  cu_q, cu_k: int32 [batch + 1], not
 * decreasing, cu_q[0] >= 0, cu_q[batch] <= total_q, cu_k likewise (rows outside every sequence are
 * left alone); a bound out of order or range leaves that sequence out and is reported.
 * Shapes: batch <= 1024; heads % kv_heads == 0, heads / kv_heads <= 128; d 64 or 128; window, sinks >= 0;
 * scale as tl_paged_attention; total_q * heads < 2^31.
 * strides of q, k and v > 0 where the dimension has more than one entry.
 * total_q == 0, heads == 0 or batch == 0 is a no-op.  No workspace.
 */
int tl_window_attention(tl_ctx* ctx, int dtype, const void* q, long long q_token_stride, long long q_head_stride,
                        const void* k, long long k_token_stride, long long k_head_stride, const void* v,
                        long long v_token_stride, long long v_head_stride, const int* cu_q, const int* cu_k,
                        void* out, long long out_token_stride, long long out_head_stride, float* lse, int batch,
                        int total_q, int total_k, int heads, int kv_heads, int d, float scale, int window, int sinks,
                        tl_stream_t stream);

/* ---------------------------------------------------------------- MoE layer for a few tokens
 * The layer of tl_moe_combine (the same routing, weights and gates; cfg.moe_renorm applies) for the
 * few tokens of a decoding step, where reading the chosen experts' weights is all that takes time:
 *   y_(t,j) = (SiLU(x_t . Wg_e) * (x_t . Wu_e)) . Wd_e,   out_t = sum_j gate_(t,j) * y_(t,j)
 * Unlike there, h keeps fp32 precision between the two products, the sums over j are taken in fp32
 * in the order j = 0, 1, ... and each distinct expert's weights are read once for every 16 of its tokens (again
 * from L2 where the experts are small, from HBM where one alone is larger than L2); results are bit-identical
 * run to run.
 * x: bf16 [T x H]; logits: fp32 [T x E]; w_gate, w_up: bf16 [E x H x F]; w_down: bf16 [E x F x H];
 * out: fp32 [T x H].  experts_out (int32 [T x topk]) and gates_out (fp32 [T x topk]) are optional: the
 * chosen experts, best first, and their gates.  NaN logits count as the lowest (the gates are NaN).
 * workspace: tl_moe_tokens_workspace_bytes().  One cooperative launch of one CTA per SM:
 * TL_ERR_UNSUPPORTED if the device cannot hold it at once.
 * Shapes: 1 <= T <= 128; 1 <= topk <= 8; topk <= E <= 256; H % 8 == 0; F % 8 == 0; H, F <= 32768.
 */
size_t tl_moe_tokens_workspace_bytes(int T, int H, int E, int F, int topk);
int tl_moe_tokens(tl_ctx* ctx, const void* x, const float* logits, int topk, const void* w_gate, const void* w_up,
                  const void* w_down, float* out, int* experts_out, float* gates_out, void* workspace,
                  size_t workspace_bytes, int T, int H, int E, int F, tl_stream_t stream);

/* ---------------------------------------------------------------- log probabilities of chosen tokens
 * For each row x of logits, with p = softmax(scale * x):
 *   logprob[r] = ln p[targets[r]],  entropy[r] = - sum_i p_i ln p_i,  lse[r] = ln sum_i exp(scale * x_i),
 *   top_logprobs[r][0 .. top), top_ids[r][0 .. top): the most likely tokens' ln p and indices, best first
 * (equal logits: the lower index first; NaN counts as the lowest).
 * logits: dtype (TL_BF16, TL_FP16 or TL_FP32) [rows x vocab], starting at any element, a row row_stride elements after the
 * one before (any number).  targets: int32 [rows]; a negative target skips its row (padding): its outputs are left as they are; one
 * >= vocab too, and is reported.  targets may be NULL if logprob is: no row is skipped then.  logprob, entropy, lse: fp32
 * [rows], any may be NULL.  top_logprobs: fp32, top_ids: int32 [rows x top].
 * A logit of -inf (a masked token) has probability 0.  Where all of a row are -inf, its entropy is 0 and its
 * lse and all its log probabilities are -inf.  A NaN or +inf among a row's logits makes all its fp32 outputs NaN (ids not).
 * Precision: maxima, sums and logarithms are fp32; a result below fp32's range (scale times a mask's lowest value) is -inf.
 * Results are bit-identical run to run on one device.
 * workspace: tl_token_logprobs_workspace_bytes(): counters, and parts of rows split over several CTAs.
 * Shapes: 1 <= vocab <= 2^30; 0 <= top <= 32, top <= vocab; rows <= 2^24; scale as tl_paged_attention.  rows == 0 is a no-op.
 */
size_t tl_token_logprobs_workspace_bytes(int rows, int vocab, int top);
int tl_token_logprobs(tl_ctx* ctx, int dtype, const void* logits, long long row_stride, const int* targets, float* logprob,
                      float* entropy, float* lse, float* top_logprobs, int* top_ids, int top, float scale, int rows,
                      int vocab, void* workspace, size_t workspace_bytes, tl_stream_t stream);

/* ---------------------------------------------------------------- host-side tile maps (no GPU)
 * The static tile-centric mappings the kernels use ([TL] §4.1), evaluated on the host by the
 * same code the device runs, for inspection and testing.
 *
 * Tiles are 256 x 256 when every shard (AG) or owner block (RS) is a multiple of 256 rows,
 * else 128 x 256; row blocks are reported in units of 128 rows (the first 128-row block a
 * tile covers), column blocks in units of 256 columns.
 * tl_ag_tile_order: for the AllGather + GEMM tile sequence t = 0..count-1 writes the source
 *   rank, the row block inside that rank's shard and the column block.  Returns the number of
 *   tiles, or TL_ERR_INVALID.  Arrays may be NULL to query the count; otherwise they must hold
 *   `cap` entries.
 * tl_rs_tile_order: the same for GEMM + ReduceScatter (owner-slot chain): producer, owner, row
 *   block within the owner's rows, column block.
 * tl_rs_ring_tile_order: the same for the ring (cfg.rs_ring = 1), plus each tile's hop (its
 *   position 0..W-1 on the ring of its owner's partial).
 */
int tl_ag_tile_order(int W, int rank, int m_per_rank, int n, int swizzle, int* src_rank, int* m_block,
                     int* n_block, int cap);
int tl_rs_tile_order(int W, int m, int n, int swizzle, int* producer, int* owner, int* m_block, int* n_block,
                     int cap);
int tl_rs_ring_tile_order(int W, int m, int n, int* producer, int* owner, int* m_block, int* n_block, int* hop,
                          int cap);

#ifdef __cplusplus
}
#endif
#endif /* TL_GB300_H */
