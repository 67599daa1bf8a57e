/*
 * loglinear.h — C ABI of the log-linear Mamba-2 forward and decode step
 * (sm_103a, one GPU).
 *
 * What is computed.  For every batch b, head h and query position t
 * (0-indexed), with group g = h / heads_per_group:
 *
 *     o[b,t,h,:] = sum_{s <= t} lambda[b,t,h, l(t,s)] * M^S(t,s) * (q[b,t,g,:] . k[b,s,g,:]) * v[b,s,h,:]
 *
 *   M^S(t,s) = a[b,s+1,h] * ... * a[b,t,h]   (Mamba-2 scalar-decay, 1-semiseparable mask;
 *              state-space-duality article http://biyoush.com/article/202409/463109.htm,
 *              section 狀態空間對偶性)
 *   l(t,s)   = 0 if s == t, else the bit length of (t xor s): the level of the Fenwick-tree
 *              bucket of t that holds s; buckets have power-of-two sizes and are finer near t
 *              (log-linear attention write-up https://www.yoousoft.com/industry/3746.html,
 *              section 特殊结构：树划分; the mask M^H(t,s) = lambda_t^{l(t,s)} and its
 *              composition with M^S, section 对Mamba-2和门控的对数线性推广).
 *
 * The forward uses the chunkwise algorithm of the write-up (section 高效训练算法):
 * dense masked products inside aligned chunks and a hierarchical state pass
 * across chunks.  The result does not depend on the chunk length; it is an exact
 * re-association of the sum above.
 *
 * Conventions shared by all entry points.
 *  - Every tensor is row-major and contiguous, and is owned by the caller.  Device
 *    pointers must be 16-byte aligned (LL_ERR_ALIGN otherwise).
 *  - q, k, v, o share ll_shape.dtype (fp32 or bf16); a, lambda and the states are fp32.
 *  - All work is enqueued on the caller's CUDA stream (`stream`, a cudaStream_t, may be
 *    NULL for the legacy default stream).  The library allocates no device memory, frees
 *    nothing and does not synchronise, except where a function says so.
 *  - Arguments are validated on the host before any launch; a failed check returns its
 *    code and enqueues nothing.  A launch error returns LL_ERR_CUDA.  Errors detected on
 *    the device (a bounded wait that ran out) are recorded in a device status word and
 *    reported by loglinear_check_status().  No C++ exception crosses this boundary.
 */
#ifndef LOGLINEAR_H
#define LOGLINEAR_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  LL_OK = 0,
  LL_ERR_NULL = 1,          /* a required pointer is NULL */
  LL_ERR_SHAPE = 2,         /* sizes out of the supported range or inconsistent */
  LL_ERR_DTYPE = 3,         /* unsupported dtype */
  LL_ERR_ALIGN = 4,         /* a pointer is not 16-byte aligned */
  LL_ERR_WORKSPACE = 5,     /* workspace NULL or smaller than the query says */
  LL_ERR_CUDA = 6,          /* a CUDA runtime call or launch failed */
  LL_ERR_TIMEOUT = 7,       /* a bounded device-side wait ran out (see check_status) */
  LL_ERR_UNIMPLEMENTED = 8  /* valid request that this library does not implement */
} ll_status;

typedef enum { LL_F32 = 0, LL_BF16 = 1 } ll_dtype;

/*
 * Problem shape.
 *   batch            B >= 1
 *   T                sequence length, T >= 1 and T % chunk == 0 (forward); unused by decode
 *   heads            H >= 1, H % heads_per_group == 0
 *   heads_per_group  heads sharing one q/k group (MVA); G = H / heads_per_group groups
 *   d_k              16, 32, 64 or 128 (q/k width, the state's row count)
 *   d_v              16, 32 or 64 (v/o width, the state's column count)
 *   chunk            C in {16, 32, 64, 128}
 *   levels           L: lambda holds L weights per (b, t, h); forward needs
 *                    L >= bit_length(T-1) + 1 (every level a query below T can see);
 *                    decode uses L as the number of state slots too
 *   dtype            dtype of q, k, v and o
 */
typedef struct {
  int batch;
  int T;
  int heads;
  int heads_per_group;
  int d_k;
  int d_v;
  int chunk;
  int levels;
  ll_dtype dtype;
} ll_shape;

/* Bytes of device workspace loglinear_fwd needs for this shape (0 if the shape is
 * invalid).  The workspace holds per-chunk decays, chunk states and the Fenwick block
 * states of the inter-chunk pass (write-up section 高效训练算法). */
size_t loglinear_fwd_workspace_bytes(const ll_shape* shape);

/*
 * Forward over the whole sequence (write-up sections 高效训练算法 and
 * 对Mamba-2和门控的对数线性推广, Algorithm 1 / Fig. 3).
 *   q, k      (B, T, G, d_k)     dtype
 *   v         (B, T, H, d_v)     dtype
 *   a         (B, T, H)          fp32, each in (0, 1]; a <= 0 gives undefined results
 *   lambda    (B, T, H, L)       fp32
 *   o         (B, T, H, d_v)     dtype, written
 *   workspace device buffer of at least loglinear_fwd_workspace_bytes(shape) bytes,
 *             16-byte aligned; its contents on entry do not matter
 *   states_out        NULL, or (B, H, state_levels, d_k, d_v) fp32: the Fenwick bucket
 *                     states at position T, i.e. the memory a decode step at position T
 *                     starts from.  Level l holds sum over the level-l bucket of T of
 *                     M^S(T-1, s) k_s v_sᵀ.  Only the levels live at T (level l >= 1
 *                     with bit l-1 of T set) are written; the other slots hold
 *                     unspecified values, as the decode step allows.
 *   state_logscale_out NULL, or (B, H, state_levels) fp32, written as zeros (the decay
 *                     is folded into states_out).
 *   state_levels      slots in states_out; must be >= bit_length(T) + 1 when states_out
 *                     is given, ignored otherwise.
 * Which kernels run (loglinear_fwd_path reports it): bf16 with d_k = 128, d_v = 64 and
 * T % 64 == 0 takes the tensor-core path (tcgen05 products over 128-token tiles; when
 * T % 128 == 64 the last tile holds 64 tokens).  Every other accepted shape runs the fp32
 * CUDA-core path, which computes the same result several times more slowly.
 */
ll_status loglinear_fwd(const ll_shape* shape, const void* q, const void* k, const void* v,
                        const float* a, const float* lambda, void* o, void* workspace,
                        size_t workspace_bytes, float* states_out, float* state_logscale_out,
                        int state_levels, void* stream);

/*
 * One decode step at position `pos` for every (b, h) (write-up section 特殊结构：树划分:
 * O(log T) time and memory per decoded token).  shape->T is ignored;
 * shape->levels = L is the number of state slots and of lambda weights.
 *   q_t, k_t   (B, G, d_k)   dtype
 *   v_t        (B, H, d_v)   dtype
 *   a_t        (B, H)        fp32 in (0, 1]
 *   lambda_t   (B, H, L)     fp32
 *   o_t        (B, H, d_v)   dtype, written
 *   states     (B, H, L, d_k, d_v) fp32, read and updated in place
 *   state_logscale (B, H, L) fp32, read and updated in place
 * The bucket memory of level l is exp(state_logscale[l]) * states[l]; level l >= 1 is
 * live at position pos when bit l-1 of pos is set; slots of levels that are not live
 * hold unspecified values.  The step decays the live levels by a_t (in the log-scale),
 * forms o_t = lambda^0 (q.k) v + sum over live l of lambda^l q^T S^l, then merges the
 * token and the levels 1..m (m = trailing ones of pos) into level m+1 of pos+1.
 * Requires pos >= 0 and L >= bit_length(pos + 1) + 1.  A state exported by
 * loglinear_fwd at T continues with pos = T.
 */
ll_status loglinear_decode_step(const ll_shape* shape, long long pos, const void* q_t,
                                const void* k_t, const void* v_t, const float* a_t,
                                const float* lambda_t, void* o_t, float* states,
                                float* state_logscale, void* stream);

/*
 * End-to-end forward from HOST buffers: copies q, k, v, a, lambda (host, same layouts
 * as loglinear_fwd; pinned memory lets the copies run asynchronously) into
 * `device_arena`, runs loglinear_fwd and copies o back to the host buffer o_host.  The
 * batch is cut into up to 8 pieces of consecutive batch elements whose copies and
 * forwards overlap: inputs go in on a library stream, each piece's forward runs on
 * `stream`, outputs come back on a second library stream, and `stream` waits for the
 * last copy, so the call is complete once `stream` reaches that point.  The first call
 * on a device creates the two streams and their events (kept until exit).  The host
 * buffers must stay valid until then; the caller synchronises.  `device_arena` must hold
 * at least loglinear_fwd_host_arena_bytes(shape) bytes (16-byte aligned).
 * Calls from several host threads are safe: the library holds a per-device lock while a
 * call enqueues its work.  Their copies share the two library streams, so concurrent
 * calls' copies run one after another; each call needs its own arena and host buffers.
 */
size_t loglinear_fwd_host_arena_bytes(const ll_shape* shape);
ll_status loglinear_fwd_host(const ll_shape* shape, const void* q_host, const void* k_host,
                             const void* v_host, const float* a_host, const float* lambda_host,
                             void* o_host, void* device_arena, size_t arena_bytes, void* stream);

/*
 * Forward for callers that cannot allocate device memory.  The pages have no
 * counterpart to this entry point; it exists for code that is not allowed to call
 * cudaMalloc or any other allocator while it runs (for example a plugin whose host owns
 * every device allocation, or code sharing the context with an allocator it must not
 * disturb), and for callers that cannot size or keep a workspace between calls.
 *
 * Same arguments and results as loglinear_fwd, without the workspace: the library uses
 * a fixed device array of LOGLINEAR_STATIC_WORKSPACE_BYTES (32 MiB) that each GPU loading
 * the library holds until the process exits.  The call allocates nothing and frees
 * nothing.
 *   - Shapes whose loglinear_fwd_workspace_bytes() exceeds LOGLINEAR_STATIC_WORKSPACE_BYTES
 *     are rejected with LL_ERR_WORKSPACE before anything is enqueued (for example
 *     B*H = 16 heads of T = 2048 at d_k = 128, d_v = 64 fit; the pages workload does not).
 *   - The first call on each device looks up the array's device address (with that
 *     device current); make that first call before any stream capture begins.
 *   - Every call on a device shares the one array and leaves its contents behind;
 *     nothing in it needs to start at zero, since every call writes each word before
 *     reading it.  Calls whose work
 *     overlaps on the GPU (other streams, other threads) race on the array: serialise
 *     them, e.g. on one stream.
 */
#define LOGLINEAR_STATIC_WORKSPACE_BYTES (32u << 20)
ll_status loglinear_fwd_static_workspace(const ll_shape* shape, const void* q, const void* k,
                                         const void* v, const float* a, const float* lambda,
                                         void* o, float* states_out, float* state_logscale_out,
                                         int state_levels, void* stream);

/* ---- sequence segments -------------------------------------------------------------------
 * A forward can start at a position T0 > 0 from the bucket memories there, and those
 * memories can be built from the memories of whole earlier segments.  This is what a
 * sequence split over several devices needs (each holds one segment of 2^p tokens; one
 * all-gather of the segments' memories and summed log-decays lets every segment form the
 * buckets of its start), and what a prefill in pieces needs.  Sources: the per-bucket
 * memories of the write-up (section 特殊结构：树划分, Fig. 2) and the combination of the
 * memories of pieces level by level (section 高效训练算法, Algorithm 1).
 *
 * Bucket memories use the decode step's format: (B, H, levels, d_k, d_v) fp32 blocks with
 * (B, H, levels) fp32 log-scales; the memory of level l is exp(logscale[l]) * block[l];
 * level l >= 1 is live at a position p when bit l-1 of p is set, and the block holds
 * sum over the bucket of M^S(p-1, s) k_s v_sᵀ.  Slots of levels that are not live hold
 * unspecified values and are neither read nor written.
 */

/* Bytes of workspace loglinear_fwd_continue needs (0: invalid shape or start). */
size_t loglinear_fwd_continue_workspace_bytes(const ll_shape* shape, long long T0);

/*
 * Forward over the tokens at positions T0 .. T0+T-1 (T = shape->T), given the bucket
 * memories at T0.  q, k, v, a, lambda and o hold the segment's T tokens, laid out as for
 * loglinear_fwd; lambda's levels are absolute (level l of every bucket, near or far), so
 * shape->levels must be >= bit_length(T0 + T - 1) + 1.
 *   T0               >= 0 and a multiple of the smallest power of two >= T (then every
 *                    bucket of a position in the segment lies either inside the segment
 *                    or before T0, where it is a bucket of T0); else LL_ERR_SHAPE
 *   prefix_states    (B, H, prefix_levels, d_k, d_v) fp32, the memories at T0 (read);
 *   prefix_logscale  (B, H, prefix_levels) fp32; both may be NULL when T0 == 0
 *   prefix_levels    >= bit_length(T0) + 1, <= 64
 *   states_out       NULL, or (B, H, state_levels, d_k, d_v): the memories at T0 + T
 *                    (written with zero log-scales into state_logscale_out if given), the
 *                    live levels only; may be the same buffer as prefix_states (then with
 *                    state_levels == prefix_levels, and state_logscale_out may be
 *                    prefix_logscale): a decode or a further continuation goes on from it
 *   state_levels     >= bit_length(T0 + T) + 1 when states_out is given
 *   workspace        >= loglinear_fwd_continue_workspace_bytes(shape, T0) bytes
 * With T0 == 0 this is loglinear_fwd.  The shapes of loglinear_fwd run on the same paths
 * (tensor cores for bf16, d_k = 128, d_v = 64, T % 64 == 0; the CUDA cores otherwise).
 */
ll_status loglinear_fwd_continue(const ll_shape* shape, long long T0, const void* q, const void* k,
                                 const void* v, const float* a, const float* lambda,
                                 const float* prefix_states, const float* prefix_logscale,
                                 int prefix_levels, void* o, void* workspace, size_t workspace_bytes,
                                 float* states_out, float* state_logscale_out, int state_levels,
                                 void* stream);

/* Bytes of workspace loglinear_segment_total needs (0: invalid shape; shape->levels is
 * ignored). */
size_t loglinear_segment_total_workspace_bytes(const ll_shape* shape);

/*
 * The memory of a whole segment of T tokens and the decay it applies to everything
 * before it:
 *   total_state     (B, H, d_k, d_v) fp32: sum over s < T of M^S(T-1, s) k_s v_sᵀ
 *   total_logdecay  (B, H) fp32: sum over t < T of ln a_t
 * k, v, a as for loglinear_fwd (no q or lambda).  shape->levels is ignored.
 */
ll_status loglinear_segment_total(const ll_shape* shape, const void* k, const void* v, const float* a,
                                  void* workspace, size_t workspace_bytes, float* total_state,
                                  float* total_logdecay, void* stream);

/*
 * The bucket memories at T0 = n_segments * T (T = shape->T, a power of two: every bucket
 * of T0 is then made of whole segments) from the memories of the n_segments segments
 * before it, as loglinear_segment_total returns them:
 *   seg_states     (n_segments, B, H, d_k, d_v) fp32, segment 0 first
 *   seg_logdecay   (n_segments, B, H) fp32
 *   states_out     (B, H, state_levels, d_k, d_v): the levels live at T0 are written;
 *   state_logscale_out NULL or (B, H, state_levels): zeros at those levels
 *   state_levels   >= bit_length(T0) + 1, <= 64
 * n_segments <= 64.  Uses shape->batch, heads, d_k, d_v and T.  Nothing is enqueued for
 * n_segments == 0 (position 0 has no buckets).
 */
ll_status loglinear_prefix_states(const ll_shape* shape, int n_segments, const float* seg_states,
                                  const float* seg_logdecay, float* states_out,
                                  float* state_logscale_out, int state_levels, void* stream);

/* ---- log-linear Gated DeltaNet -----------------------------------------------------------
 * The write-up extends Gated DeltaNet the same way (section 对Mamba-2和门控的对数线性推广):
 * the model's own transition, the gated delta rule
 *   S_t = a_t S_{t-1} (I - beta_t k_t k_tᵀ) + beta_t v_t k_tᵀ,
 * is kept and its attention mask is combined with the hierarchical one.  The delta rule
 * equals S_t = a_t S_{t-1} + u_t k_tᵀ with u_t = beta_t (v_t - a_t S_{t-1} k_t), so the
 * output is the masked form over u:
 *   o_t = sum_{s<=t} lambda_t^{l(t,s)} M^S(t,s) (q_t . k_s) u_s.
 */

/* Bytes of device workspace loglinear_gdn_fwd needs (0: invalid shape). */
size_t loglinear_gdn_fwd_workspace_bytes(const ll_shape* shape);

/*
 * Log-linear Gated DeltaNet forward.  Arguments as for loglinear_fwd, plus
 *   beta  (B, T, H)  fp32, the delta-rule write strength (in [0, 1] for a stable rule)
 * Keys are used as given; the model normalises them (the delta rule is stable for
 * beta |k|^2 <= 2).  u is computed chunk by chunk in the delta rule's WY form: the
 * chunks' local solves run in parallel, then one CTA per (b, h) carries the state across
 * the chunks in order.  For bf16 with d_k = 128, d_v = 64 and T % 128 == 0 the chunks
 * are 128 tokens and the products run on the tensor cores (fp16 high and low parts,
 * fp32 accumulation); otherwise 32-token chunks run in fp32 on the CUDA cores.  u is
 * stored in the input dtype in the workspace, then the level-fused forward runs on
 * (q, k, u, a, lambda).  On the tensor-core path with batch >= 2 the last batch element's
 * state pass and forward run on a second, high-priority stream that the library creates
 * on a device's first such call, forked from and joined back into `stream` with events,
 * so that the other elements' forward starts as soon as their passes end; every launch
 * is still ordered after the work already on `stream`, and later work on `stream` waits
 * for all of it.  Concurrent calls on one device are serialised inside the library.
 */
ll_status loglinear_gdn_fwd(const ll_shape* shape, const void* q, const void* k, const void* v,
                            const float* a, const float* beta, const float* lambda, void* o,
                            void* workspace, size_t workspace_bytes, void* stream);

/* ---- backward -------------------------------------------------------------------------
 * The pages give no backward; this is the chain rule on the forward's masked form
 * o_t = sum_{s<=t} lambda_t^{l(t,s)} M^S(t,s) (q_t . k_s) v_s (write-up sections
 * 特殊结构：树划分 and 对Mamba-2和门控的对数线性推广), laid out by the same chunks and
 * Fenwick blocks as the forward (section 高效训练算法, Algorithm 1).
 */

/* Bytes of device workspace loglinear_bwd needs for this shape (0: invalid shape). */
size_t loglinear_bwd_workspace_bytes(const ll_shape* shape);

/*
 * Gradients of the scalar sum(dO * o) where o = loglinear_fwd(q, k, v, a, lambda), for
 * every shape loglinear_fwd accepts.  Inputs as for loglinear_fwd, plus
 *   dO       (B, T, H, d_v)  dtype
 * and the outputs, all written (no accumulation into them):
 *   dq, dk   (B, T, G, d_k)  dtype; the heads of a group add up
 *   dv       (B, T, H, d_v)  dtype
 *   dlog_a   (B, T, H)       fp32, the gradient with respect to log a, the form in which
 *                            a enters the forward; the gradient with respect to a is
 *                            dlog_a / a (badly conditioned for a near 0, hence not
 *                            returned); 0 at t = 0, whose decay multiplies nothing
 *   dlambda  (B, T, H, L)    fp32; levels with no bucket get 0
 *   workspace >= loglinear_bwd_workspace_bytes(shape) bytes, 16-byte aligned, contents on
 *            entry do not matter
 * For bf16 with d_k = 128, d_v = 64, T % 128 == 0 and chunk >= 64 the products run on the
 * tensor cores (fp16 operands with power-of-two scales, fp32 accumulation); other shapes
 * run fp32 on the CUDA cores.  The terms of the levels above a tile (or chunk) are summed
 * through each node's dual with fp32 atomics, so results can differ between calls by
 * rounding.
 */
ll_status loglinear_bwd(const ll_shape* shape, const void* q, const void* k, const void* v,
                        const float* a, const float* lambda, const void* dO, void* dq, void* dk,
                        void* dv, float* dlog_a, float* dlambda, void* workspace,
                        size_t workspace_bytes, void* stream);

/* ---- comparators ---------------------------------------------------------------------
 * Two other ways to compute on the tensor-core shape (bf16, d_k = 128, d_v = 64,
 * T % 128 == 0), kept to measure the level-fused forward against.  Any other shape
 * returns LL_ERR_UNIMPLEMENTED.  Same layouts, alignment and stream rules as
 * loglinear_fwd; outputs written, workspace contents on entry do not matter.
 */

/* Bytes of workspace loglinear_fwd_naive needs (0: invalid or unsupported shape). */
size_t loglinear_fwd_naive_workspace_bytes(const ll_shape* shape);

/*
 * The same output as loglinear_fwd, computed without level fusion: after the tile
 * states and the Fenwick tree, one output pass per level (the intra-tile levels 0..7,
 * then each inter-tile level), each re-reading its inputs and adding its level's term
 * to an fp32 sum in the workspace.  This mirrors the write-up's naive variant, which
 * re-runs an existing Mamba-2 computation once per level (section
 * 对Mamba-2和门控的对数线性推广, Fig. 4).
 */
ll_status loglinear_fwd_naive(const ll_shape* shape, const void* q, const void* k, const void* v,
                              const float* a, const float* lambda, void* o, void* workspace,
                              size_t workspace_bytes, void* stream);

/* Bytes of workspace ssd_fwd needs (0: invalid or unsupported shape). */
size_t ssd_fwd_workspace_bytes(const ll_shape* shape);

/*
 * The lambda-constant special case, i.e. Mamba-2's SSD (state-space-duality article,
 * section 狀態空間對偶性): o_t = sum over s <= t of M^S(t, s) (q_t . k_s) v_s.  It runs
 * the Mamba-2 structure: chunk states, a sequential state pass over tiles, then one
 * chunk output pass with a single prefix state per tile.  Same as loglinear_fwd with
 * lambda = 1 everywhere, up to rounding.  shape->levels is ignored.
 */
ll_status ssd_fwd(const ll_shape* shape, const void* q, const void* k, const void* v,
                  const float* a, void* o, void* workspace, size_t workspace_bytes, void* stream);

/* ---- linear attention with a decay per head ----------------------------------------------
 * Where the forward above takes a decay per token and weighs each bucket, these take one
 * constant decay per head and no weights: for every batch row b and head h, with group
 * g = h / heads_per_group and gamma = exp(log_a[h]),
 *     S_t = gamma S_{t-1} + k[b,t,g,:] v[b,t,h,:]ᵀ,     o[b,t,h,:] = S_tᵀ q[b,t,g,:],
 * S_{-1} = state_in or 0.  (The state-space-duality article, section 狀態空間對偶性, with
 * the decay held constant.)
 *
 * Shapes: ll_shape with any T >= 1 (2^30 at most); d_k and d_v multiples of 8 from 8 to 128;
 * batch * heads <= 2^20; chunk and levels are ignored.  q, k, v, o and their gradients have
 * shape->dtype; states (B, H, d_k, d_v), log_a (H) and their gradients are fp32.
 *
 * Precision, as errors relative in the 2-norm: fp32 calls (three tf32 products each) below
 * 2^-19, 3 to 5e-7 as a rule.  bf16 calls (on tcgen05): outputs and gradients 2.1e-3 of which
 * 1.7e-3 is their own rounding; final states and dstate_in, though fp32, below 2^-16, 4e-6 as
 * a rule, since each token's decayed v enters its product as two bf16 parts (16 bits).  A
 * decode step adds to the states in fp32.
 *
 * log_a is a constant of the model (no gradient is returned for it).  Values above 0 count
 * as 0 (no decay), values below -1000 as -1000 (gamma is 0 in fp32).
 *
 * lengths: NULL, or (B) int32 on the device: row b holds lengths[b] tokens, clamped to
 * [0, T].  What the tensors hold past them is not used, NaN included; the outputs there are
 * written as zeros, and final states are those after lengths[b] tokens (state_in itself for
 * length 0).  A NaN or infinity inside a row's length can reach every output of its
 * 128-token chunk, earlier tokens included (0 times infinity in a masked product).
 */

/* Bytes of device workspace lindecay_fwd needs (0: invalid shape; 16: none is used, NULL
 * will do), on whichever device, stream or part of its SMs the call is made. */
size_t lindecay_fwd_workspace_bytes(const ll_shape* shape);

/*
 * The whole sequence.
 *   q, k (B, T, G, d_k), v (B, T, H, d_v)   dtype
 *   log_a     (H) fp32
 *   lengths   NULL or (B) int32
 *   state_in  NULL or (B, H, d_k, d_v) fp32, the state before the first token
 *   o         (B, T, H, d_v) dtype, written; may be v, overlaps neither q nor k
 *   state_out NULL or (B, H, d_k, d_v) fp32, written; may be state_in
 *   workspace >= lindecay_fwd_workspace_bytes(shape) bytes; contents do not matter
 */
ll_status lindecay_fwd(const ll_shape* shape, const void* q, const void* k, const void* v, const float* log_a,
                       const int* lengths, const float* state_in, void* o, float* state_out, void* workspace,
                       size_t workspace_bytes, void* stream);

/* Bytes of device workspace lindecay_bwd needs (0: invalid shape; 16: none is used, NULL
 * will do), on whichever device, stream or part of its SMs the call is made. */
size_t lindecay_bwd_workspace_bytes(const ll_shape* shape);

/*
 * Gradients of sum(dO * o) + sum(dstate_out * state_out), (o, state_out) = lindecay_fwd.
 *   dO         (B, T, H, d_v) dtype; ignored past a row's length
 *   state_in   as for the forward (NULL: zero)
 *   dstate_out NULL (zero) or (B, H, d_k, d_v) fp32
 *   dq, dk     (B, T, G, d_k) dtype, dv (B, T, H, d_v) dtype, written; the heads of a group
 *              add up in fp32, in order (the result does not vary between calls)
 *   dstate_in  NULL or (B, H, d_k, d_v) fp32, written; neither state_in nor dstate_out
 * No output may overlap an input or another output.
 */
ll_status lindecay_bwd(const ll_shape* shape, const void* q, const void* k, const void* v, const float* log_a,
                       const int* lengths, const float* state_in, const void* dO, const float* dstate_out, void* dq,
                       void* dk, void* dv, float* dstate_in, void* workspace, size_t workspace_bytes, void* stream);

/*
 * One token for every (b, h): the recurrence itself.  shape->T is ignored.
 *   q_t, k_t (B, G, d_k), v_t (B, H, d_v) dtype; log_a (H) fp32; o_t (B, H, d_v) dtype, written
 *   states (B, H, d_k, d_v) fp32, read and updated in place; lindecay_fwd's state_out
 *   continues here.
 */
ll_status lindecay_decode_step(const ll_shape* shape, const void* q_t, const void* k_t, const void* v_t,
                               const float* log_a, void* o_t, float* states, void* stream);

/* ---- norms around a block ----------------------------------------------------------------
 * The norm after a block (of its output y, over groups of `group` values), its gate, the
 * residual add with a scale per channel, and the norm before the next block, in one pass:
 *     n  = y * rsqrt(mean over the group of y^2 + eps) * w_post
 *     x' = x + scale * act(gate) * n
 *     h  = x' * rsqrt(mean over the row of x'^2 + eps) * w_pre
 * x, gate, w_post, scale and the pair (w_pre, h) may be left out (NULL): without x, x' is
 * the gated norm alone (a norm per head before the output projection: group = d_v); without
 * y, h is the norm of x alone (in front of the first block).
 *   rows   >= 1, below 2^31
 *   dim    1 to 16384 values per row; a multiple of 8 runs faster
 *   group  divides dim into at most 4096 groups (dim: one norm per row); dim itself, or a
 *          power of two from 8 to 256, runs faster
 *   act    of the gate
 *   eps    0 to 1
 * Activations have `dtype`; weights and their gradients are fp32 (dim).  Sums are fp32.
 */
enum { BN_IDENTITY = 0, BN_SILU = 1, BN_SIGMOID = 2 };
typedef struct {
  long long rows;
  int dim;
  int group;
  int act;
  float eps;
  ll_dtype dtype;
} blocknorm_shape;

/*
 * Forward.  x, y, gate (rows, dim); x_new (rows, dim), written when y is given (NULL
 * otherwise); h NULL or (rows, dim), written.  x_new may be x, y or gate, h too (not the
 * same buffer as x_new).
 */
ll_status blocknorm_fwd(const blocknorm_shape* shape, const void* x, const void* y, const void* gate,
                        const float* w_post, const float* scale, const float* w_pre, void* x_new, void* h,
                        void* stream);

/* Bytes of device workspace blocknorm_bwd needs (0: invalid shape). */
size_t blocknorm_bwd_workspace_bytes(const blocknorm_shape* shape);

/*
 * Gradients of sum(dx_new * x') + sum(dh * h).
 *   dx_new   NULL (zero) or (rows, dim);  dh NULL, or (rows, dim) together with x_new, the
 *            forward's x' as stored (x itself without y)
 *   y, gate, w_post, scale, w_pre as for the forward
 *   dx       NULL, or (rows, dim): the gradient of x (and of x')
 *   dy       (rows, dim), with y;  dgate (rows, dim), with gate
 *   dw_post, dscale, dw_pre  NULL, or (dim) fp32, each with its weight; summed over the rows in a
 *            fixed order (the result does not vary between calls)
 *   workspace >= blocknorm_bwd_workspace_bytes(shape) bytes; contents do not matter
 * No output may overlap an input.
 */
ll_status blocknorm_bwd(const blocknorm_shape* shape, const void* dx_new, const void* dh, const void* x_new,
                        const void* y, const void* gate, const float* w_post, const float* scale,
                        const float* w_pre, void* dx, void* dy, void* dgate, float* dw_post, float* dscale,
                        float* dw_pre, void* workspace, size_t workspace_bytes, void* stream);

/* ---- gated recurrence ---------------------------------------------------------------------
 * One state per channel, with a decay from the data:
 *     s_t = sigmoid(r_t);  a_t = exp(-decay[c] s_t);  u_t = n(a_t) sigmoid(i_t) x_t
 *     h_t = a_t h_{t-1} + u_t
 * n(a) keeps the state's size whatever the decay: sqrt(1 - a^2) (GS_RMS: a unit variance stays
 * one), 1 - a (GS_LERP: a moving average) or 1 (GS_NONE).  Without i its sigmoid is 1.
 *   batch  1 to 2^20;  T 1 to 2^30;  dim 1 to 2^20 channels (sequences run faster
 *     with multiples of 8 in bf16 and of 4 in fp32, single tokens with even numbers)
 *   x, r, i, h and their gradients (B, T, dim) dtype;  decay (dim) fp32, finite; values below 0
 *   count as 0, and their gradient is 0;  states (B, dim) fp32
 * lengths: NULL, or (B) int32 on the device: row b holds lengths[b] tokens, clamped to [0, T].
 * What the tensors hold past them is not read; outputs there are written as zeros, and final
 * states are those after lengths[b] tokens (state_in itself for length 0).
 * r of -inf holds a state (a = 1, and n = 0 but for GS_NONE), inf decays it by exp(-decay).  GS_RMS:
 * where 1 - a^2 is below 2^-126, a decay of 0 among them, n and its slope count as 0.
 * The state and all arithmetic are fp32; h_t is rounded once, the state that goes on is not.
 * Results do not vary between calls of the same sizes; in another batch a row may be shared out
 * otherwise, and its states rounded otherwise.
 */
enum { GS_RMS = 0, GS_LERP = 1, GS_NONE = 2 };
typedef struct {
  int batch;
  int T;
  int dim;
  int mix;
  ll_dtype dtype;
} gatescan_shape;

/*
 * The whole sequence.  i, lengths, state_in, state_out may be NULL.  h may be x, r or i;
 * state_out may be state_in; otherwise no output may overlap an input or another output.
 */
ll_status gatescan_fwd(const gatescan_shape* shape, const void* x, const void* r, const void* i, const float* decay,
                       const int* lengths, const float* state_in, void* h, float* state_out, void* stream);

/* Bytes of device workspace gatescan_bwd needs for ddecay (0: invalid shape). */
size_t gatescan_bwd_workspace_bytes(const gatescan_shape* shape);

/*
 * Gradients of sum(dh * h) + sum(dstate_out * state_out), (h, state_out) = gatescan_fwd, from the
 * forward's h as stored.  state_in NULL: zero; dstate_out NULL: zero.
 *   dx, dr, di  (B, T, dim) dtype, written, zeros past a row's length; di with i
 *   ddecay      NULL or (dim) fp32, written, summed in a fixed order; asks for the workspace,
 *               whose contents do not matter
 *   dstate_in   NULL or (B, dim) fp32, written
 * No output may overlap an input or another output.
 */
ll_status gatescan_bwd(const gatescan_shape* shape, const void* dh, const void* x, const void* r, const void* i,
                       const float* decay, const void* h, const int* lengths, const float* state_in,
                       const float* dstate_out, void* dx, void* dr, void* di, float* ddecay, float* dstate_in,
                       void* workspace, size_t workspace_bytes, void* stream);

/*
 * One token of every row; shape->T is ignored.  x_t, r_t, i_t (NULL: none), h_t (B, dim) dtype;
 * states (B, dim) fp32, read and updated in place.  h_t may be x_t, r_t or i_t; nothing else may overlap.
 */
ll_status gatescan_decode_step(const gatescan_shape* shape, const void* x_t, const void* r_t, const void* i_t,
                               const float* decay, float* states, void* h_t, void* stream);

/* ---- norms and rotation of heads ----------------------------------------------------------
 * For every head of q and k, in one pass over both:
 *     y = scale * R(position) (norm(x) * w)
 * norm: x * rsqrt(mean of x^2 + eps) (HR_RMS), x * rsqrt(sum of x^2 + eps) (HR_L2) or x (HR_NONE);
 * w (dim) fp32, shared by the heads, or NULL.  R turns the first `rot` values by pairs: pair n by
 * position * inv_freq[n] radians, (x_n, x_{n + rot/2}) (HR_HALF) or (x_2n, x_2n+1)
 * (HR_INTERLEAVED); the rest of the head stays.  Angles are reduced modulo a turn to 2^-28 radians at
 * every position, and what is left, an eighth of a turn at most, is held in fp32 (2^-25 radians).
 *   rows     1 to 2^31 - 1 tokens;  q (rows, q_heads, dim), k (rows, k_heads, dim) dtype
 *   q_heads  1 to 65536;  k_heads 0 (k is NULL) to 65536
 *   dim      1 to 256;  rot even, 0 to dim (multiples of 8 of both run faster)
 *   positions (rows) int32, may be negative; NULL: row % T, a batch of sequences from 0
 *   inv_freq  (rot / 2) fp32, below 2^63 in size
 *   eps      0 to 1 (with 0, a head whose mean or sum of squares is below 2^-126 counts as that)
 */
enum { HR_HALF = 0, HR_INTERLEAVED = 1 };
enum { HR_NONE = 0, HR_RMS = 1, HR_L2 = 2 };
typedef struct {
  long long rows;
  int T;
  int q_heads;
  int k_heads;
  int dim;
  int rot;
  int layout;
  int norm;
  float eps;
  float scale_q;
  float scale_k;
  ll_dtype dtype;
} headrope_shape;

/* q_out and k_out are written; each may be its own input, and may overlap nothing else. */
ll_status headrope_fwd(const headrope_shape* shape, const void* q, const void* k, const float* w_q, const float* w_k,
                       const float* inv_freq, const int* positions, void* q_out, void* k_out, void* stream);

/* Bytes of device workspace headrope_bwd needs for dw_q or dw_k (0: invalid shape). */
size_t headrope_bwd_workspace_bytes(const headrope_shape* shape);

/*
 * Gradients of sum(dq_out * q_out) + sum(dk_out * k_out), from the forward's inputs.
 *   dq, dk      written; each may be its own dq_out or dk_out, and may overlap nothing else
 *   dw_q, dw_k  NULL, or (dim) fp32, each with its weight, written; summed in a fixed order
 *   workspace   with dw_q or dw_k; contents do not matter
 */
ll_status headrope_bwd(const headrope_shape* shape, const void* dq_out, const void* dk_out, const void* q, const void* k,
                       const float* w_q, const float* w_k, const float* inv_freq, const int* positions, void* dq,
                       void* dk, float* dw_q, float* dw_k, void* workspace, size_t workspace_bytes, void* stream);

/* ---- gated feed-forward block ---------------------------------------------------------------
 * m = act(x w_gate^T) * (x w_up^T): both projections, the activation and the product in one kernel.
 *   rows  1 to 2^24;  dim, ff  8 to 2^20, multiples of 8
 *   x (rows, dim), w_gate and w_up (ff, dim), m (rows, ff), gradients like what they are of: dtype
 *   act   of the gate: identity, silu, sigmoid or gelu (0.5 z (1 + erf(z / sqrt 2)))
 * bf16: products of bf16 values summed in fp32, everything after them in fp32, rounded once; the
 * backward rounds the gradients of gate and up to bf16 before its products, which take nothing wider.
 * fp32: forward products of fp32 values up to 8 rows; with more, rows of x and of the weights are two
 * fp16 parts of values scaled by their row's largest, three products each: a value is within 2^-23
 * of itself or 2^-39 of its row's largest, whichever is more, so that one 2^-30 of the largest has 9
 * bits.  Backward three bf16 parts (24 bits, whatever the row), six products.  An infinity (backward
 * also a value beyond bf16's range) can come out as NaN in its row or column.
 * Results do not vary between calls of the same sizes on the same kind of GPU.
 */
enum { FF_IDENTITY = 0, FF_SILU = 1, FF_SIGMOID = 2, FF_GELU = 3 };
typedef struct {
  long long rows;
  int dim;
  int ff;
  int act;
  ll_dtype dtype;
} ffgate_shape;

/* Bytes of device workspace ffgate_fwd needs (0: invalid shape; 16: none, NULL will do). */
size_t ffgate_fwd_workspace_bytes(const ffgate_shape* shape);

/* gate and up: NULL both, or (rows, ff) dtype, written: the projections, for ffgate_bwd.  No output
 * may overlap an input or another output.  Workspace contents do not matter. */
ll_status ffgate_fwd(const ffgate_shape* shape, const void* x, const void* w_gate, const void* w_up, void* m, void* gate,
                     void* up, void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of device workspace ffgate_bwd needs (0: invalid shape). */
size_t ffgate_bwd_workspace_bytes(const ffgate_shape* shape);

/*
 * Gradients of sum(dm * m), from the forward's gate and up.
 *   dx (rows, dim), dw_gate, dw_up (ff, dim)  written, each NULL where it is not asked for (one is)
 * No output may overlap an input or another output.  Workspace contents do not matter.
 */
ll_status ffgate_bwd(const ffgate_shape* shape, const void* dm, const void* x, const void* w_gate, const void* w_up,
                     const void* gate, const void* up, void* dx, void* dw_gate, void* dw_up, void* workspace,
                     size_t workspace_bytes, void* stream);

/* ---- diagnostics -------------------------------------------------------------------- */

/* Same as loglinear_fwd, and records CUDA events on `stream` around its kernels:
 * events[0] before the first kernel and events[i + 1] right after kernel i, for as many
 * as n_events allows (events are cudaEvent_t handles created by the caller).  The kernel
 * order is the one loglinear_fwd_kernel_names() lists. */
ll_status loglinear_fwd_profiled(const ll_shape* shape, const void* q, const void* k,
                                 const void* v, const float* a, const float* lambda, void* o,
                                 void* workspace, size_t workspace_bytes, float* states_out,
                                 float* state_logscale_out, int state_levels, void* stream,
                                 void** events, int n_events);

/* Comma-separated names of the kernels loglinear_fwd launches for this shape, in launch
 * order (with_export != 0: states_out is given).  Empty string for an invalid shape. */
const char* loglinear_fwd_kernel_names(const ll_shape* shape, int with_export);

/* Number of kernels this library has launched in this process so far (all devices). */
unsigned long long loglinear_launch_count(void);

/* Synchronises `stream`, then reads and clears the device status word of the current
 * device.  Returns LL_OK, LL_ERR_TIMEOUT when a bounded device-side wait ran out since
 * the last check (the launch returned early; its outputs are undefined), or
 * LL_ERR_CUDA when the synchronisation itself failed. */
ll_status loglinear_check_status(void* stream);

/* Self-test of the bounded-wait path: launches one block that waits on a barrier that
 * nothing completes, giving up after about `spins` polls, which records LL_ERR_TIMEOUT
 * in the status word.  Faults nothing; the context stays usable. */
ll_status loglinear_selftest_wait_timeout(long long spins, void* stream);

/* Static description of a status code. */
const char* loglinear_status_string(ll_status status);

/* Which kernels loglinear_fwd would launch for this shape: 0 = invalid shape,
 * 1 = generic CUDA-core path, 2 = tensor-core (tcgen05) path. */
int loglinear_fwd_path(const ll_shape* shape);

#ifdef __cplusplus
}
#endif

#endif /* LOGLINEAR_H */
