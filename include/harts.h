/*
 * harts.h - C ABI of the packed-tree KDA library (GB300, sm_103a).
 *
 * The library runs chunkwise gated-delta (KDA-style) linear attention, forward and
 * backward, once over a prefix-compressed rollout tree instead of once per
 * root-to-leaf trajectory, as HARTS describes it (arXiv 2608.28158; page
 * "HARTS ... 精读", sections 4.2-4.3; page "thelatestinai ... 2608.28158", Fig. 1(c),
 * Fig. 2 and Figure C.1 captions).
 *
 * Model of one layer.  Per trajectory and head, with per-channel log-decay g_t,
 *     S_t = (I - beta_t k_t k_t^T) diag(exp g_t) S_{t-1} + beta_t k_t v_t^T
 *     o_t = scale * S_t^T q_t
 * computed chunkwise with chunk length B (chunks anchored at trajectory position 0).
 *
 * Conventions for every call below:
 *  - Return 0 on success, or a negative HARTS_E* code; harts_last_error() then holds
 *    a message for the calling thread.  No C++ exception crosses the ABI.
 *  - "device pointer" = memory on the current CUDA device, allocated and owned by the
 *    caller.  The library never allocates device memory and never frees caller memory.
 *  - Work is enqueued on the given stream and returns without synchronising.  Faults
 *    found by the kernels (a bad plan, out-of-range decay) are recorded in the plan's
 *    device error word; harts_plan_device_error() reads it (it synchronises).  Calls
 *    without a plan record theirs in the word that they are given, or in the library's
 *    own, which harts_device_error() reads.
 *  - All tensors are contiguous, token-major: [rows, H, d].  Rows are compact tokens
 *    in the plan's layout (see harts_plan_arrays.seg_offset).
 *  - A plan is immutable once built; the forward and the backward pass reuse the same
 *    plan (activation recomputation re-runs the same rounds, replays and handoffs,
 *    section 4.3).  Distinct plans may be used from distinct threads.
 */
#ifndef HARTS_H
#define HARTS_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define HARTS_OK            0
#define HARTS_EINVAL       -1   /* malformed argument (tree, pointer, size) */
#define HARTS_EUNSUPPORTED -2   /* chunk/head dim/dtype combination without a kernel */
#define HARTS_EOVERFLOW    -3   /* a size or index does not fit the library's types */
#define HARTS_ESMALLBUF    -4   /* caller buffer smaller than required */
#define HARTS_ECUDA        -5   /* a CUDA runtime call failed */
#define HARTS_ETIMEOUT     -6   /* a bounded device wait ran out */
#define HARTS_EDEVICE      -7   /* a kernel recorded an error in the device error word */
#define HARTS_ENOPLAN      -8   /* plan not uploaded to the device */

typedef enum { HARTS_FP32 = 0, HARTS_BF16 = 1 } harts_dtype;

/* Kernel selection.  AUTO picks the tensor-core kernels where they exist
 * (bf16, dk = dv = 128, B = 64) and the exact fp32 CUDA-core kernels otherwise. */
typedef enum { HARTS_KERNEL_AUTO = 0, HARTS_KERNEL_SIMT = 1, HARTS_KERNEL_TC = 2 } harts_kernel;

typedef struct CUstream_st *harts_stream_t;   /* same type as cudaStream_t */
typedef struct harts_plan harts_plan;          /* opaque, host memory, library-owned */

/* ------------------------------------------------------------------------------ */
/* Planning (host only).                                                          */
/* ------------------------------------------------------------------------------ */

/*
 * harts_plan_calls - minimum-call plan over a segment forest (section 4.2).
 *
 * n_seg    number of segments (fork-free token paths), >= 1.
 * parent   host [n_seg]: parent[i] < i, or -1 for a root (forests allowed).
 * seg_len  host [n_seg]: tokens per segment, >= 1.
 * chunk    chunk length B >= 1 (the kernels support 16, 32, 64).
 * flags    0: the minimum-call plan below.  HARTS_PLAN_NODEWISE: the node-wise
 *          baseline the pages compare against (one call per tree level; section 5,
 *          Fig. 4 "Node-wise LA"): every segment is its own sequence, starting one
 *          round after its parent from the parent sequence's end state (a slot at
 *          that sequence's end), with its own chunk grid and no replay.
 *          HARTS_PLAN_NOREPLAY: the pages' no-replay comparison (section 5.3, Fig. 5):
 *          the continuations of the minimum-call plan, but every side branch starts
 *          one round after its producer from the producer's exact state at the fork
 *          position e_v (usually inside a chunk), with its own chunk grid and no
 *          replay; forward only (harts_kda_bwd returns HARTS_EUNSUPPORTED).
 *          Both bits, or any other bit: HARTS_EINVAL.
 * out      receives a new plan; free it with harts_plan_free.
 *
 * The plan holds: the rounds (one packed call each; their number is the minimum
 * under the packed chunkwise-call model, T_pre/T_in recurrence with a
 * max/second-max pass, linear time), the input sequences per round, the compact
 * layout, each side branch's resume anchor a(p) = B*floor(p/B) and replay rows
 * [a(p), p), and the boundary-state slots with their consumers.  Conventions that
 * make the plan unique: the continuation is the lowest-id child of maximal T_pre;
 * rounds are as early as possible; sequences are ordered by round, then by the id
 * of their first segment; slots by producer sequence, then position.
 * Errors: HARTS_EINVAL (bad parent order, zero length, chunk < 1),
 *         HARTS_EOVERFLOW (token counts beyond int32 rows).
 */
int harts_plan_calls(int32_t n_seg, const int32_t *parent, const int64_t *seg_len,
                     int32_t chunk, uint32_t flags, harts_plan **out);

#define HARTS_PLAN_NODEWISE 1u   /* harts_plan_calls flag: one sequence per segment */
#define HARTS_PLAN_NOREPLAY 2u   /* harts_plan_calls flag: exact-position handoffs, no replay */

typedef struct {
    int32_t n_seg, n_roots, n_leaves, chunk;
    int32_t n_rounds;        /* packed calls per pass */
    int32_t n_seq;           /* input sequences (= leaves) */
    int32_t n_states;        /* materialised boundary-state slots */
    int32_t n_cons;          /* sequences that start from a slot */
    int64_t C;               /* compact (non-replay) tokens */
    int64_t S;               /* expanded trajectory tokens */
    int64_t R;               /* replay tokens, sum of (|children|-1)*(e_v mod B) */
    int64_t n_chunks;        /* chunks over all sequences, replay rows included */
    int32_t max_seq_chunks;  /* longest sequence in chunks */
    int32_t n_fold_rows;     /* distinct compact rows that are replayed */
    uint32_t flags;          /* the harts_plan_calls flags the plan was built with */
} harts_plan_info;

int harts_plan_get_info(const harts_plan *plan, harts_plan_info *out);

/* Plan arrays, exported into caller-allocated host arrays sized from the info.
 * Any pointer may be NULL to skip that array. */
typedef struct {
    int64_t *seg_offset;     /* [n_seg]   compact row of the segment's first token     */
    int64_t *seg_pos;        /* [n_seg]   trajectory position s_v of that token         */
    int32_t *seg_seq;        /* [n_seg]   sequence that executes the segment            */
    int32_t *seg_ctop;       /* [n_seg]   direct-continuation child, -1 for a leaf      */
    int32_t *seg_tpre;       /* [n_seg]   T_pre(v)                                      */
    int32_t *seg_tin;        /* [n_seg]   T_in(v)                                       */
    int32_t *round_seq_ptr;  /* [n_rounds+1] sequences of round r: [ptr[r], ptr[r+1])   */
    int64_t *cu_seqlens;     /* [n_seq+1] own (non-replay) rows of sequence i           */
    int32_t *seq_round;      /* [n_seq]   1-based round                                  */
    int32_t *seq_first_seg;  /* [n_seq]                                                  */
    int64_t *seq_anchor;     /* [n_seq]   trajectory position of local position 0       */
    int32_t *seq_replay;     /* [n_seq]   replay rows rho < B before the own rows        */
    int32_t *seq_src;        /* [n_seq]   initial state: slot id >= 0, or -1-r = root r  */
    int64_t *replay_ptr;     /* [n_seq+1]                                               */
    int64_t *replay_idx;     /* [R]       compact rows replayed, in position order       */
    int32_t *seq_state_ptr;  /* [n_seq+1] slots produced by sequence i                   */
    int32_t *state_seq;      /* [n_states] producer sequence                             */
    int64_t *state_pos;      /* [n_states] local position (multiple of B) in producer    */
    int32_t *state_cons_ptr; /* [n_states+1]                                             */
    int32_t *state_cons;     /* [n_cons]   consumer sequences, ascending                 */
    int32_t *root_cons_ptr;  /* [n_roots+1]                                              */
    int32_t *root_cons;      /* [n_seq - n_cons] sequences starting from a root state    */
} harts_plan_arrays;

int harts_plan_export(const harts_plan *plan, harts_plan_arrays *dst);

/* Bytes of device memory the plan needs (int32 tables plus the device error word). */
size_t harts_plan_device_bytes(const harts_plan *plan);

/* Copy the plan tables into dev_buf (device pointer, >= harts_plan_device_bytes,
 * 256-byte aligned, caller-owned, kept alive while the plan is used) on `stream`.
 * Records dev_buf in the plan; clears the device error word. */
int harts_plan_upload(harts_plan *plan, void *dev_buf, size_t bytes, harts_stream_t stream);

/* Synchronise `stream`, read the device error word; 0 or HARTS_EDEVICE.  The word
 * is cleared after reading.  *code (nullable) receives the raw device code. */
int harts_plan_device_error(harts_plan *plan, harts_stream_t stream, int32_t *code);

void harts_plan_free(harts_plan *plan);

/* The same for the library's own error word on the current device, in which calls without a plan
 * and without a word of their own record a bounded wait that ran out (code 3: the outputs are
 * incomplete).  Calls on other streams report there too. */
int harts_device_error(harts_stream_t stream, int32_t *code);

/* Self-test of the device failure path (for tests of error reporting): one thread waits on
 * a barrier that nothing completes, gives up after max_cycles SM cycles (1 .. 1e8) and
 * records device code 3 (timeout) in the plan's error word (plan NULL: in the library's own),
 * the way every kernel of the library reports a wait that ran out; harts_plan_device_error
 * (harts_device_error) then returns HARTS_EDEVICE and the context stays usable.  Never traps.  Errors: HARTS_EINVAL, HARTS_ENOPLAN,
 * HARTS_ECUDA. */
int harts_selftest_timeout(harts_plan *plan, uint32_t max_cycles, harts_stream_t stream);

/* ------------------------------------------------------------------------------ */
/* Forward: one packed call per round (section 4.3, "KDA").                       */
/* ------------------------------------------------------------------------------ */

typedef struct {
    int32_t H, dk, dv;
    int32_t dtype;           /* harts_dtype of q, k, v, g, beta, o, chunk_states */
    int32_t kernel;          /* harts_kernel */
    float scale;             /* o = scale * S^T q */
    const void *q;           /* device [C,H,dk], 16-byte aligned (so are k, v, g, o,
                                chunk_states and the backward's d_o, dq, dk, dv, dg) */
    const void *k;           /* device [C,H,dk] */
    const void *v;           /* device [C,H,dv] */
    const void *g;           /* device [C,H,dk] natural-log per-channel decay (<= 0) */
    const void *beta;        /* device [C,H] */
    void *o;                 /* device [C,H,dv] output */
    float *states;           /* device [n_states,H,dk,dv] fp32 boundary-state slots;
                                may be NULL only if n_states == 0 */
    float *final_state;      /* device [n_seq,H,dk,dv] fp32, nullable */
    const float *h0;         /* device [n_roots,H,dk,dv] fp32 root initial state, nullable
                                (NULL = zero state) */
    void *chunk_states;      /* device, nullable: per (chunk, head) a record of dk*dv + B*B
                                elements in `dtype`: the state at the chunk start stored
                                transposed ([dv][dk]) followed by the chunk's
                                T = (I + diag(beta) A)^-1 ([B][B]); saved for the backward
                                pass; records ordered [chunk][head], chunks by sequence.
                                The tensor-core kernels store the state column-scaled as
                                their products use it, S^T diag(e^m) with m the chunk's
                                reference log-decay (half the chunk's total per-channel
                                log-decay, Gamma_L / 2); the exact-fp32 kernels
                                store S^T.  A backward call must therefore select the same
                                kernel family as the forward call that wrote the records. */
} harts_kda_fwd_args;

/* Bytes for chunk_states (n_chunks * H * (dk*dv + B*B) * sizeof(dtype)). */
size_t harts_kda_chunk_state_bytes(const harts_plan *plan, int32_t H, int32_t dk, int32_t dv,
                                   int32_t dtype);

/*
 * harts_kda_fwd - forward pass over all rounds, enqueued on `stream`.
 * Round r launches one kernel over its (sequence, head) pairs.  A sequence starts
 * from the zero state (root; or h0), or from a slot written by an earlier round,
 * runs its replay rows and own rows chunk by chunk, writes o for its own rows only,
 * stores requested boundary states into their slots and its final state.
 * Errors: HARTS_EINVAL (NULL or misaligned pointers), HARTS_EUNSUPPORTED (dk, dv not in {32,64,128}, dk != dv,
 * B not in {16,32,64}), HARTS_ENOPLAN, HARTS_EOVERFLOW (C * H above 2^31 - 1),
 * HARTS_ECUDA.
 */
int harts_kda_fwd(const harts_plan *plan, const harts_kda_fwd_args *args, harts_stream_t stream);

/* ------------------------------------------------------------------------------ */
/* Backward: rounds in reverse, gradients through the state handoffs.             */
/* ------------------------------------------------------------------------------ */

typedef struct {
    harts_kda_fwd_args fwd;  /* the forward arguments; fwd.o is not read; fwd.states and
                                fwd.chunk_states must hold what harts_kda_fwd wrote */
    const void *d_o;         /* device [C,H,dv] gradient of the loss w.r.t. o */
    const float *d_final;    /* device [n_seq,H,dk,dv] fp32, nullable (zero) */
    void *dq, *dk, *dv, *dg; /* device [C,H,dk] / [C,H,dv] outputs in `dtype` */
    void *dbeta;             /* device [C,H] output in `dtype` */
    float *dh0;              /* device [n_roots,H,dk,dv] fp32, nullable */
    void *workspace;         /* device, >= harts_kda_bwd_workspace_bytes, 256-B aligned */
    size_t workspace_bytes;
} harts_kda_bwd_args;

size_t harts_kda_bwd_workspace_bytes(const harts_plan *plan, int32_t H, int32_t dk, int32_t dv);

/*
 * harts_kda_bwd - backward pass, enqueued on `stream`.
 * Rounds run in reverse.  Per (sequence, head) a reverse chunk loop carries dS; at a
 * slot the sequence produced, the gradients w.r.t. that slot from all its consumers
 * (sequences of later rounds) are added in ascending consumer order; the gradient
 * w.r.t. the sequence's own initial state is stored for its producer (section 4.3:
 * the initial-state gradient flows back into the call that produced the boundary).
 * Replay rows get no dq; their dk, dv, dg, dbeta are added into the ancestor rows
 * in a fixed order after all rounds.  Deterministic: no floating-point atomics.
 * Errors: as harts_kda_fwd, plus HARTS_ESMALLBUF.
 */
int harts_kda_bwd(const harts_plan *plan, const harts_kda_bwd_args *args, harts_stream_t stream);

/*
 * The backward pass in its two phases; harts_kda_bwd is harts_kda_bwd_state followed by
 * harts_kda_bwd_grad with the same arguments (same workspace, same stream order).
 *  - state: rounds in reverse, one launch per round; carries dL/dS through every
 *    sequence and its handoffs; stores each sequence's initial-state gradient and (on
 *    the tensor-core path) the carried gradient at every chunk end in the workspace.
 *    On the exact fp32 path this phase also forms all input gradients.
 *  - grad:  on the tensor-core path one launch over every (chunk, head), forming dq, dk,
 *    dv, dg, dbeta from the saved chunk states; then the deterministic fold of replay-row
 *    gradients into ancestor rows and dh0.
 * Errors: as harts_kda_bwd.
 */
int harts_kda_bwd_state(const harts_plan *plan, const harts_kda_bwd_args *args, harts_stream_t stream);
int harts_kda_bwd_grad(const harts_plan *plan, const harts_kda_bwd_args *args, harts_stream_t stream);

/*
 * harts_kda_bwd_static - harts_kda_bwd without any caller-provided device memory.
 * (This entry point has no counterpart in the paper; it is a deployment convenience.)
 *
 * For callers that cannot give the library device memory of its own: plugins inside a
 * host framework that owns the device pool and offers no allocation hook, or step loops
 * that must not allocate.  The caller still passes every input and output; the scratch
 * (initial-state gradients, replay-row gradients, saved chunk-end state gradients) lives
 * in a file-scope device array of harts_kda_bwd_static_max_bytes() = 32 MiB that every
 * GPU loading the library holds until the process exits.
 *  - args->workspace and args->workspace_bytes are ignored.
 *  - The first call on a device (with that device current) looks up the array's device
 *    address; make that first call before any stream capture.  It allocates nothing and
 *    calls no allocating routine.
 *  - Every call on a device shares the one array and leaves its last contents there.
 *    Nothing in it needs to start at zero: each call writes every scratch entry before
 *    reading it.  Calls whose work overlaps on the GPU (two streams, or two host
 *    threads) race on the array; serialise them.
 * Errors: as harts_kda_bwd, plus HARTS_ESMALLBUF when the plan, heads and head size need
 * more scratch than the array holds (harts_kda_bwd_workspace_bytes tells the need).
 */
int harts_kda_bwd_static(const harts_plan *plan, const harts_kda_bwd_args *args, harts_stream_t stream);
size_t harts_kda_bwd_static_max_bytes(void);

/* ------------------------------------------------------------------------------ */
/* Causal short convolution over the compact layout.                              */
/* ------------------------------------------------------------------------------ */

/*
 * The convolution that precedes KDA in the layer (page "HARTS ... 精读", section 4.3,
 * KDA paragraph; summary page, section 4 "KDA execution"), run once per compact row:
 * the window over the previous w - 1 tokens reads the row's real ancestors on its own
 * trajectory (a temporary prefix of the parent's rows), never the neighbouring rows of
 * another packed sequence, and is zero before the trajectory start.  Depthwise:
 *   pre[r][c] = bias[c] + sum_{j<w} weight[c][w-1-j] * x[row j positions before r][c],
 *   y = pre (activation 0) or pre * sigmoid(pre) (activation 1).
 * The plan (uploaded) carries the ancestor context and the successor lists for any
 * w <= 8; any of the three plan modes works.  Deterministic (no atomics).
 */
typedef struct {
    int32_t channels;        /* ch: values per row (e.g. H * d), a multiple of 8 */
    int32_t width;           /* w: 1..8 */
    int32_t dtype;           /* harts_dtype of x, y, dy, dx */
    int32_t activation;      /* 0 none, 1 SiLU */
    const void *x;           /* device [C][ch], compact layout, 16-byte aligned */
    const float *weight;     /* device [ch][w] fp32; weight[c][w-1] multiplies the current row */
    const float *bias;       /* device [ch] fp32, or NULL */
    void *y;                 /* device [C][ch] output (forward only), 16-byte aligned */
} harts_conv_fwd_args;

/* Forward.  Errors: HARTS_EINVAL (NULL / misaligned pointer, channels not a positive
 * multiple of 8, activation), HARTS_EUNSUPPORTED (dtype, width outside 1..8),
 * HARTS_ENOPLAN, HARTS_ECUDA. */
int harts_conv_fwd(const harts_plan *plan, const harts_conv_fwd_args *args, harts_stream_t stream);

typedef struct {
    harts_conv_fwd_args fwd; /* y is not used */
    const void *dy;          /* device [C][ch] dL/dy per compact row (already summed over the
                                trajectories that share the row) */
    void *dx;                /* device [C][ch] output */
    float *dweight;          /* device [ch][w] output (overwritten) */
    float *dbias;            /* device [ch] output (overwritten), or NULL */
    void *workspace;         /* device, harts_conv_bwd_workspace_bytes, 16-byte aligned */
    size_t workspace_bytes;
} harts_conv_bwd_args;

/* Workspace of harts_conv_bwd: the per-256-row partial sums of dweight / dbias, fp32
 * [ceil(C/256)][ch][w+1].  0 for invalid arguments. */
size_t harts_conv_bwd_workspace_bytes(const harts_plan *plan, int32_t channels, int32_t width);

/* Backward: dx[r] sums weight * dL/dpre over the rows 0..w-1 positions after r on every
 * branch below it (gathered in a fixed order); dweight and dbias are reduced over rows in
 * a fixed order.  Errors as harts_conv_fwd, plus HARTS_ESMALLBUF (workspace). */
int harts_conv_bwd(const harts_plan *plan, const harts_conv_bwd_args *args, harts_stream_t stream);

/* ------------------------------------------------------------------------------ */
/* Gated linear recurrence over the compact layout.                               */
/* ------------------------------------------------------------------------------ */

/*
 * One state per channel, run once per compact row, from the row before it on its own trajectory
 * (its segment's, or its parent's last one; the root's initial state at a trajectory's start):
 *   a = e^g,  h[r] = a h[before r] + x[r]            (HARTS_SCAN_ADD)
 *             h[r] = a h[before r] + (1 - a) x[r]    (HARTS_SCAN_MIX)
 * g is the natural-log decay, as KDA's: g <= 0, -inf starts afresh.  A positive g is not looked for, and
 * its results are not defined.  States, and what the long products of decays are made of, are fp32.
 * All plan modes work; results do not depend on the rounds, and their bits do not depend on timing.
 * Decays are within two half steps of fp32, but for one case: in bf16's add form, where no trajectory of the
 * plan has more than 4,096 rows and no fp32 state (final_state, dh0) is asked for, they are the hardware's
 * exponential, 2^-22 off.  There, asking for a state or adding a long tree to the forest can change the last bit of
 * the other results.  A forest whose segments are roots of one row each is a decoding step: h0 holds the
 * states before, final_state those behind.
 * What is not finite reaches the rows behind it on its trajectories (backward: before it), and no others.
 */
#define HARTS_SCAN_ADD 0
#define HARTS_SCAN_MIX 1

typedef struct {
    int32_t channels;        /* D: values per row, a positive multiple of 8 */
    int32_t dtype;           /* harts_dtype of x, g, h, d_h, dx, dg */
    int32_t form;            /* HARTS_SCAN_ADD or HARTS_SCAN_MIX */
    const void *x;           /* device [C][D], compact layout, 16-byte aligned (so are the others) */
    const void *g;           /* device [C][D] */
    const float *h0;         /* device [n_roots][D] initial state of every root, or NULL (zero) */
    void *h;                 /* device [C][D]: written by the forward, read by the backward; not x or g */
    float *final_state;      /* device [n_seq][D] output: state after every sequence's last row, or NULL;
                                may be h0 in a decoding step (a plan of single rows) */
    void *workspace;         /* device, harts_scan_workspace_bytes, 16-byte aligned; calls that may run
                                at the same time have one each */
    size_t workspace_bytes;
} harts_scan_fwd_args;

/* Workspace of either direction: the tiles' maps and the states between them; 0 where no segment follows
 * another and none is longer than 128 rows (workspace may be NULL then), and for invalid arguments. */
size_t harts_scan_workspace_bytes(const harts_plan *plan, int32_t channels, int32_t dtype);

/* Forward.  Errors: HARTS_EINVAL (NULL / misaligned pointers, channels, form), HARTS_EUNSUPPORTED
 * (dtype), HARTS_ENOPLAN, HARTS_EOVERFLOW (more than 2^31 - 1 tiles), HARTS_ESMALLBUF (workspace),
 * HARTS_ECUDA.  A bounded wait that runs out records device code 3 in the plan's error word. */
int harts_scan_fwd(const harts_plan *plan, const harts_scan_fwd_args *args, harts_stream_t stream);

typedef struct {
    harts_scan_fwd_args fwd; /* h as the forward wrote it; final_state is not used */
    const void *d_h;         /* device [C][D] dL/dh per compact row, 16-byte aligned (so are the others) */
    const float *d_final;    /* device [n_seq][D] dL/dfinal_state, or NULL */
    void *dx;                /* device [C][D] output; dx and dg may be none of the inputs */
    void *dg;                /* device [C][D] output */
    float *dh0;              /* device [n_roots][D] output, or NULL; not h0, d_final only in a decoding step */
} harts_scan_bwd_args;

/* Backward: with lam[r] = d_h[r] + the sum of a[c] lam[c] over the rows c that follow r (+ d_final
 * at a sequence's end, where it has one),
 *   dx[r] = lam or (1 - a) lam,   dg[r] = lam a (h[before r], minus x[r] in the mix form),
 * and dh0 the sum of a lam over a root's first row.  Sums over branches run by ascending segment.
 * Errors as the forward. */
int harts_scan_bwd(const harts_plan *plan, const harts_scan_bwd_args *args, harts_stream_t stream);

/* ------------------------------------------------------------------------------ */
/* Compact-to-semantic log-probabilities.                                         */
/* ------------------------------------------------------------------------------ */

/*
 * Page "HARTS ... 精读", section 4.4 ("紧凑到语义的 log 概率"); summary page "Semantic
 * Preservation": a compact logit row is reduced over the vocabulary once (its
 * log-sum-exp), and every semantic position s -- a token occurrence of an original
 * trajectory -- reads its own target logit from the row its token maps to:
 *   logp[s] = logits[c(s)][target[s]] - lse[c(s)].
 * The backward (eq. 19) sums the independently formed gradients of a row's semantic
 * positions onto it: dlogits[c] = sum_{s -> c} dlogp[s] (onehot(target[s]) - softmax(row c)).
 * Work is O(C V) + O(S); no S x V array is formed.  Deterministic (no atomics).
 *
 * harts_plan_semantic_map fills, on the host: sem_row[S] (compact row of each semantic
 * position; trajectories in increasing leaf id, each from its root to its leaf), and the
 * positions grouped by row: row_ptr[C+1], row_sem[S] (ascending within a row).  Callers
 * with another semantic order may build these arrays themselves.
 */
int harts_plan_semantic_map(const harts_plan *plan, int32_t *sem_row, int32_t *row_ptr, int32_t *row_sem);

typedef struct {
    int64_t C;               /* compact rows */
    int32_t V;               /* vocabulary, a multiple of 8 */
    int32_t dtype;           /* harts_dtype of logits / dlogits */
    int64_t S;               /* semantic positions, < 2^31 */
    const void *logits;      /* device [C][V], 16-byte aligned */
    const int32_t *row_ptr;  /* device [C+1]: semantic positions of row c are row_sem[row_ptr[c] ..] */
    const int32_t *row_sem;  /* device [S] */
    const int32_t *target;   /* device [S] label of each semantic position, 0 <= target < V */
    float *lse;              /* device [C]: written by the forward, read by the backward */
    float *logp;             /* device [S]: written by the forward */
} harts_logprob_fwd_args;

/* Forward.  Errors: HARTS_EINVAL (NULL / misaligned pointers, V not a multiple of 8),
 * HARTS_EUNSUPPORTED (dtype), HARTS_EOVERFLOW (S), HARTS_ECUDA. */
int harts_logprob_fwd(const harts_logprob_fwd_args *args, harts_stream_t stream);

typedef struct {
    harts_logprob_fwd_args fwd;  /* lse as written by the forward; logp unused */
    const float *dlogp;          /* device [S] dL/dlogp */
    void *dlogits;               /* device [C][V] output (overwritten), 16-byte aligned */
} harts_logprob_bwd_args;

int harts_logprob_bwd(const harts_logprob_bwd_args *args, harts_stream_t stream);

/* ------------------------------------------------------------------------------ */
/* Branch attention over the compact layout (the softmax-attention layers).       */
/* ------------------------------------------------------------------------------ */

/*
 * Page "HARTS ... 精读", section 4.3 (MLA paragraph); summary page, section 4 ("MLA
 * execution"); figures page, Figure C.1(c).  Projections run once per compact row; each
 * sequence of the plan is a branch whose queries (its own rows) attend to the keys and
 * values of its ancestors and itself with bottom-right causal alignment: own query t sees
 * view entries 0 .. h + t, where h is the number of trajectory positions before the
 * sequence.  The view is gathered inside the kernel; outputs go to the unique compact
 * rows.  Per head: o = softmax(scale q k^T) v, lse = log sum_j exp(scale q k_j).
 * Equal to plain causal attention of every trajectory through a row.
 *
 * The plan's attention tables (each sequence's ancestor rows) are built when they add up
 * to at most 2^27 rows; for deeper plans the call fails with HARTS_EOVERFLOW.
 */
typedef struct {
    int32_t H;               /* heads */
    int32_t d;               /* head dimension of q, k and v: 128 */
    int32_t dtype;           /* harts_dtype of q, k, v, o: HARTS_BF16 */
    float scale;             /* softmax scale, positive and finite (typically 1/sqrt(d)) */
    const void *q, *k, *v;   /* device [C][H][d], compact layout, 16-byte aligned */
    void *o;                 /* device [C][H][d] output, 16-byte aligned */
    float *lse;              /* device [C][H] output (natural-log sum-exp of scaled scores), or NULL */
} harts_attn_fwd_args;

/* Forward.  Errors: HARTS_EINVAL (NULL / misaligned pointers, H < 1, scale not positive), HARTS_EUNSUPPORTED
 * (dtype other than bf16, d other than 128), HARTS_ENOPLAN, HARTS_EOVERFLOW (no attention
 * tables in the plan, too many blocks), HARTS_ECUDA.  A bounded wait that runs out records
 * device code 3 (timeout) in the plan's device error word (harts_plan_device_error). */
int harts_attn_fwd(const harts_plan *plan, const harts_attn_fwd_args *args, harts_stream_t stream);

/* Backward of harts_attn_fwd for L with dL/do = d_o: each compact query row counts once,
 * over its own view; keys and values collect every query that sees them, across branches.
 * With D = rowsum(d_o * o) and P recomputed from lse:
 *   dv_j = sum_t P_tj d_o_t,  dS_tj = scale P_tj (d_o_t . v_j - D_t),
 *   dq_t = sum_j dS_tj k_j,   dk_j = sum_t dS_tj q_t.
 * Sums run in a fixed order (no atomics): per query tile over its view's key tiles, per
 * key tile (128 own rows of a sequence) over the query tiles that see it, in ascending
 * (sequence, tile) order. */
typedef struct {
    harts_attn_fwd_args fwd; /* q, k, v; o and lse as written by the forward (lse required) */
    const void *d_o;         /* device [C][H][d] bf16 dL/do per compact row */
    void *dq, *dk, *dv;      /* device [C][H][d] bf16 outputs (overwritten), 16-byte aligned */
    void *workspace;         /* device, harts_attn_bwd_workspace_bytes, 16-byte aligned */
    size_t workspace_bytes;
} harts_attn_bwd_args;

/* Workspace of harts_attn_bwd: D, fp32 [C][H] (rounded up to 256 bytes); 0 for invalid
 * arguments. */
size_t harts_attn_bwd_workspace_bytes(const harts_plan *plan, int32_t H);

/* Errors as harts_attn_fwd, plus HARTS_EINVAL (NULL / misaligned lse, d_o, dq, dk, dv,
 * workspace) and HARTS_ESMALLBUF (workspace). */
int harts_attn_bwd(const harts_plan *plan, const harts_attn_bwd_args *args, harts_stream_t stream);

/* ------------------------------------------------------------------------------ */
/* Root-mean-square norm with the residual's addition.                            */
/* ------------------------------------------------------------------------------ */

/*
 * Per compact row (the rows of every layer's norm, and of the one before the vocabulary
 * projection):
 *   h = x + residual,  rstd = 1 / sqrt(mean_j h_j^2 + eps),  y_j = h_j rstd weight_j.
 * h is normalised in fp32 before it is rounded to `dtype` for the residual stream.  The
 * 8-bit output holds y as e4m3 values with one power-of-two scale (e8m0: 2^(byte - 127))
 * per 32 channels, the smallest that keeps the block within 448; a block that holds an
 * infinity gets scale 255 (NaN), a NaN stays one.  Scales are in row order; a block-scaled
 * product of the tensor cores wants them rearranged in its own.  Squares are summed in fp32: a
 * row whose sum overflows gets rstd 0, and zeros for its finite values.  h may be x or residual, and y may be x
 * (rows are read before they are written), but not both x.  The backward wants h: without a
 * residual and with y over x, give one.
 */
typedef struct {
    int64_t C;               /* rows, >= 0 */
    int32_t D;               /* channels, 1 .. 16384 */
    int32_t dtype;           /* harts_dtype of x, residual, h, y */
    float eps;               /* >= 0 */
    const void *x;           /* device [C][D], 16-byte aligned (so are residual, weight, h, y, y8) */
    const void *residual;    /* device [C][D], or NULL */
    const float *weight;     /* device [D] fp32 */
    void *h;                 /* device [C][D] output, x + residual; required with a residual,
                                NULL allowed without */
    void *y;                 /* device [C][D] output, or NULL */
    void *y8;                /* device [C][D] e4m3 output, or NULL; D a multiple of 32 */
    void *y8_scale;          /* device [C][D/32] e8m0 output, given exactly when y8 is */
    float *rstd;             /* device [C] output, or NULL */
} harts_rmsnorm_fwd_args;

/* Forward.  Errors: HARTS_EINVAL (NULL / misaligned pointers, no output, negative C, eps),
 * HARTS_EUNSUPPORTED (dtype, D above 16384, y8 with D not a multiple of 32), HARTS_ECUDA. */
int harts_rmsnorm_fwd(const harts_rmsnorm_fwd_args *args, harts_stream_t stream);

typedef struct {
    int64_t C;
    int32_t D;
    int32_t dtype;           /* harts_dtype of dy, h, dh, dx */
    const void *dy;          /* device [C][D] dL/dy, 16-byte aligned (so are h, dh, weight, dx) */
    const void *h;           /* device [C][D] as the forward wrote it (x where it had no residual) */
    const void *dh;          /* device [C][D] dL/dh along the residual stream, or NULL */
    const float *weight;     /* device [D] fp32 */
    const float *rstd;       /* device [C] from the forward */
    void *dx;                /* device [C][D] output: dL/dx = dL/dresidual; may be dy or dh */
    float *dweight;          /* device [D] output (overwritten; zero when C is 0) */
    int32_t *error;          /* device [1]: set to 3 if a bounded wait ran out; cleared by the caller.
                                NULL: the library's own word (harts_device_error) */
    void *workspace;         /* device, harts_rmsnorm_bwd_workspace_bytes, 16-byte aligned */
    size_t workspace_bytes;
} harts_rmsnorm_bwd_args;

/* Workspace of harts_rmsnorm_bwd: fp32 column sums; 0 for invalid arguments. */
size_t harts_rmsnorm_bwd_workspace_bytes(int64_t C, int32_t D, int32_t dtype);

/* Backward.  dweight is summed in a fixed order (no atomics).  Errors as the forward, plus
 * HARTS_ESMALLBUF (workspace). */
int harts_rmsnorm_bwd(const harts_rmsnorm_bwd_args *args, harts_stream_t stream);

/* ------------------------------------------------------------------------------ */
/* The norms around a block, with its gate and the residual's scaled addition.    */
/* ------------------------------------------------------------------------------ */

/*
 * Per row, between a block's output y and the next block's input n:
 *   u = y / sqrt(mean_j y_j^2 + eps) * post_weight        (u = y where post_weight is NULL)
 *   h = residual + scale * act(gate) * u                  (1 for a gate, 0 for a residual that is NULL)
 *   n = h / sqrt(mean_j h_j^2 + eps) * pre_weight         (none where pre_weight is NULL)
 * with at least one of the norms.  Without a residual and a second norm this is the gated norm of
 * an attention's or a recurrence's heads (C rows and heads, D a head's channels).  act is
 * HARTS_GATE_LINEAR (the gate itself), HARTS_GATE_SILU (z sigmoid(z)) or HARTS_GATE_SIGMOID.
 * Statistics are fp32; h is normalised before it is rounded to `dtype`.  A row whose sum of squares
 * overflows gets rstd 0.  h and n may each be y, gate or residual (rows are read before they are
 * written), but not one buffer.
 */
#define HARTS_GATE_LINEAR 0
#define HARTS_GATE_SILU 1
#define HARTS_GATE_SIGMOID 2

typedef struct {
    int64_t C;               /* rows, >= 0 */
    int32_t D;               /* channels, 1 .. 8192 */
    int32_t dtype;           /* harts_dtype of y, gate, residual, h, n */
    int32_t gate_act;        /* HARTS_GATE_*; 0 without a gate */
    float scale;             /* of the gated block, finite */
    float eps;               /* >= 0; not used by the backward */
    const void *y;           /* device [C][D], 16-byte aligned (so are all [C][D] and the weights) */
    const void *gate;        /* device [C][D], or NULL */
    const void *residual;    /* device [C][D], or NULL; not used by the backward */
    const float *post_weight;/* device [D] fp32, or NULL: no norm of y */
    const float *pre_weight; /* device [D] fp32, or NULL: no n */
    void *h;                 /* device [C][D]: written by the forward; the backward reads it with a pre_weight */
    void *n;                 /* device [C][D] output, given exactly when pre_weight is; not used by the backward */
    float *rstd_post;        /* device [C]: written by the forward (or NULL), read by the backward; with post_weight */
    float *rstd_pre;         /* device [C]: the same with pre_weight */
    int32_t *error;          /* device [1]: set to 3 if a bounded wait ran out; cleared by the caller.
                                NULL: the library's own word (harts_device_error) */
} harts_block_norm_args;

/* Forward.  Errors: HARTS_EINVAL (NULL / misaligned pointers, no norm, negative C, scale, eps,
 * gate_act), HARTS_EUNSUPPORTED (dtype, D above 8192), HARTS_ECUDA. */
int harts_block_norm_fwd(const harts_block_norm_args *args, harts_stream_t stream);

typedef struct {
    harts_block_norm_args fwd;  /* as for the forward, with what it wrote */
    const void *d_n;         /* device [C][D] dL/dn, given exactly when pre_weight is */
    const void *d_h;         /* device [C][D] dL/dh along the residual stream, or NULL (then d_n is there) */
    void *dy;                /* device [C][D] output; the outputs may each be an input, but not one buffer */
    void *dresidual;         /* device [C][D] output: the whole gradient of h, or NULL */
    void *dgate;             /* device [C][D] output, or NULL */
    float *dpost_weight;     /* device [D] output with post_weight (overwritten; zero when C is 0) */
    float *dpre_weight;      /* device [D] output with pre_weight */
    void *workspace;         /* device, harts_block_norm_bwd_workspace_bytes, 16-byte aligned */
    size_t workspace_bytes;
} harts_block_norm_bwd_args;

/* Workspace of the backward: fp32 column sums; 0 for invalid arguments. */
size_t harts_block_norm_bwd_workspace_bytes(int64_t C, int32_t D, int32_t dtype);

/* Backward.  The weights' gradients are summed in a fixed order (no atomics).  Errors as the
 * forward, plus HARTS_ESMALLBUF (workspace). */
int harts_block_norm_bwd(const harts_block_norm_bwd_args *args, harts_stream_t stream);

/* ------------------------------------------------------------------------------ */
/* The gradients' global norm, and clipping.                                      */
/* ------------------------------------------------------------------------------ */

/*
 * norm = sqrt(sum over all tensors of the squares of their values);
 * out_i = g_i * (norm > max_norm ? max_norm / norm : 1).
 * Squares are summed in fp32 over the 64 bytes that a thread loads at a time and in fp64 from
 * there on, in a fixed order (no atomics); squares that overflow fp32, or that it holds as zero or
 * with few bits where there are no larger ones, are summed again in fp64.  When the norm is not
 * finite the gradients are passed on unscaled, and the caller sees it in *norm.
 */
typedef struct {
    const void *g;           /* device [n] values, aligned to their type */
    void *out;               /* device [n] output of harts_grad_clip; g itself (with the same
                                dtype) scales in place; not read by harts_grad_norm */
    int64_t n;               /* values, >= 0 (0: pointers are not looked at) */
    int32_t dtype;           /* harts_dtype of g */
    int32_t out_dtype;       /* harts_dtype of out */
} harts_grad_tensor;

/* Workspace for `count` tensors: fp64 partial sums; 0 for invalid arguments. */
size_t harts_grad_workspace_bytes(int32_t count);

/* tensors: host array of `count` >= 0 descriptors, read before the call returns.
 * norm: device [1] fp32 output.  workspace: device, 16-byte aligned.
 * Errors: HARTS_EINVAL (NULL / misaligned pointers, negative sizes, max_norm negative or
 * NaN, in place with two dtypes), HARTS_EUNSUPPORTED (dtype), HARTS_EOVERFLOW (more than
 * 2^44 values), HARTS_ESMALLBUF (workspace), HARTS_ECUDA. */
int harts_grad_norm(const harts_grad_tensor *tensors, int32_t count, float *norm, void *workspace,
                    size_t workspace_bytes, harts_stream_t stream);
int harts_grad_clip(const harts_grad_tensor *tensors, int32_t count, float max_norm, float *norm, void *workspace,
                    size_t workspace_bytes, harts_stream_t stream);

/* ------------------------------------------------------------------------------ */
/* Matrix product with bias, activation and residual in its epilogue.             */
/* ------------------------------------------------------------------------------ */

/*
 * A projection of compact rows:
 *   z = x weight^T + bias,   y = act(z) + residual
 * act is HARTS_ACT_NONE, HARTS_ACT_SILU (z sigmoid(z)) or HARTS_ACT_GELU (z Phi(z), Phi the normal
 * distribution's; not its tanh approximation).  Sums, bias, activation and residual are fp32, rounded
 * once.  z may be kept in bf16 for the gradient; act is taken of the unrounded one.
 */
#define HARTS_ACT_NONE 0
#define HARTS_ACT_SILU 1
#define HARTS_ACT_GELU 2

typedef struct {
    int64_t C;               /* rows, >= 0 */
    int32_t K;               /* width of x, a multiple of 8 */
    int32_t N;               /* width of y, a multiple of 8 */
    int32_t dtype;           /* harts_dtype of all but bias and dbias: HARTS_BF16 */
    int32_t activation;      /* HARTS_ACT_* */
    const void *x;           /* device [C][K], 16-byte aligned (so are the others) */
    const void *weight;      /* device [N][K] */
    const float *bias;       /* device [N] fp32, or NULL; not used by the backward */
    const void *residual;    /* device [C][N], or NULL; not used by the backward (its gradient is d_y) */
    void *y;                 /* device [C][N] output; y or z may be residual; not used by the backward */
    void *z;                 /* device [C][N]: output of the forward, or NULL; read by the backward where there
                                is an activation */
    int32_t *error;          /* device [1]: set to 3 if a bounded wait ran out; cleared by the caller.
                                NULL: the library's own word (harts_device_error) */
    void *workspace;         /* device, harts_linear_{fwd,bwd}_workspace_bytes; 256-byte aligned for the backward */
    size_t workspace_bytes;
} harts_linear_args;

/* Workspace of the forward: fp32 pieces of the sums where there are few tiles; 0 where there are none (workspace
 * may be NULL then), and for invalid arguments. */
size_t harts_linear_fwd_workspace_bytes(int64_t C, int32_t K, int32_t N);

/* Forward.  Errors: HARTS_EINVAL (NULL / misaligned pointers, sizes, activation, y or z over x, weight, bias
 * or one another), HARTS_EUNSUPPORTED (dtype other than bf16, K or N not a multiple of 8), HARTS_EOVERFLOW (more
 * than 2^24 tiles), HARTS_ESMALLBUF (workspace), HARTS_ECUDA. */
int harts_linear_fwd(const harts_linear_args *args, harts_stream_t stream);

typedef struct {
    harts_linear_args fwd;   /* x, weight; z as the forward kept it */
    const void *d_y;         /* device [C][N] dL/dy, 16-byte aligned (so are the outputs) */
    void *dx;                /* device [C][K] bf16 output, or NULL; dx and dweight may be none of the inputs */
    void *dweight;           /* device [N][K] bf16 output, or NULL (overwritten; zero when C is 0) */
    float *dbias;            /* device [N] fp32 output, or NULL */
} harts_linear_bwd_args;

/* Workspace of the backward: dz in bf16 where there is an activation, column sums where dbias is wanted,
 * fp32 pieces of the sums where there are few tiles; 0 where there is none of it, and for invalid arguments. */
size_t harts_linear_bwd_workspace_bytes(int64_t C, int32_t K, int32_t N, int32_t activation, int32_t with_bias);

/* Backward: dz = d_y act'(z) (each entry formed in fp32; held in bf16 for the products, unrounded for
 * dbias), dx = dz weight, dweight = dz^T x, dbias = sum over rows of dz; all sums fp32 and in a fixed
 * order.  x, weight and dz must be finite for dx and dweight to be.  Errors as the forward. */
int harts_linear_bwd(const harts_linear_bwd_args *args, harts_stream_t stream);

/* ------------------------------------------------------------------------------ */
/* Log-probabilities from hidden rows and the vocabulary weight.                  */
/* ------------------------------------------------------------------------------ */

/*
 * harts_logprob_* with the vocabulary projection inside: the logits
 *   z[c][v] = scale * (x[c] . weight[v])
 * exist tile by tile only.  lse[c] = log sum_v e^z[c][v] and
 *   logp[s] = z[c(s)][target[s]] - lse[c(s)]
 * for the same semantic positions (row_ptr, row_sem, target).  A position whose target lies
 * outside 0 .. V-1 has no label: logp 0, and its dlogp is not used.
 *   dx[c] = scale sum_v dz[c][v] weight[v],   dweight[v] = scale sum_c dz[c][v] x[c],
 *   dz[c][v] = sum_{s -> c, target[s] = v} dlogp[s] - (sum_{s -> c} dlogp[s]) e^(z[c][v] - lse[c]).
 * The backward forms the logits again, one piece of the vocabulary at a time, and holds that
 * piece's dz in bf16 (each entry formed in fp32 and rounded once; up to 32 rows in two bf16
 * terms); all sums are fp32 and in a fixed order.  x and weight must be finite: dweight sums
 * over every row, also over rows without positions (whose dx is zero).  Where they are not, lse
 * is not either: a NaN in weight reaches every row's, one in x its own row's.
 */
typedef struct {
    int64_t C;               /* compact rows, >= 0 */
    int32_t V;               /* vocabulary, >= 1 (any) */
    int32_t D;               /* width of the hidden rows, a multiple of 8 */
    int32_t dtype;           /* harts_dtype of x, weight, dx, dweight: HARTS_BF16 */
    float scale;             /* of the logits (1 / temperature), finite */
    int64_t S;               /* semantic positions; C, V and S are 2^31 - 256 at most */
    const void *x;           /* device [C][D], 16-byte aligned */
    const void *weight;      /* device [V][D], 16-byte aligned */
    const int32_t *row_ptr;  /* device [C+1]: semantic positions of row c are row_sem[row_ptr[c] ..] */
    const int32_t *row_sem;  /* device [S] */
    const int32_t *target;   /* device [S] label of each semantic position */
    float *lse;              /* device [C]: written by the forward, read by the backward */
    float *logp;             /* device [S]: written by the forward */
    int32_t *error;          /* device [1]: set to 3 if a bounded wait ran out (the outputs are then
                                incomplete); cleared by the caller.  NULL: the library's own word
                                (harts_device_error) */
    void *workspace;         /* device, harts_linear_logprob_{fwd,bwd}_workspace_bytes; 16-byte aligned for
                                the forward, 256-byte for the backward */
    size_t workspace_bytes;
} harts_linear_logprob_fwd_args;

/* Workspace of the forward: a (max, sum) pair and the maximum's column per row and tile, and a copy of x where D is no
 * multiple of 64; 0 for invalid arguments. */
size_t harts_linear_logprob_fwd_workspace_bytes(int64_t C, int32_t V, int32_t D);

/* Forward.  Errors: HARTS_EINVAL (NULL / misaligned pointers, sizes, scale not finite),
 * HARTS_EUNSUPPORTED (dtype other than bf16, D not a multiple of 8), HARTS_EOVERFLOW (C, V or
 * S), HARTS_ESMALLBUF (workspace), HARTS_ECUDA. */
int harts_linear_logprob_fwd(const harts_linear_logprob_fwd_args *args, harts_stream_t stream);

typedef struct {
    harts_linear_logprob_fwd_args fwd;  /* lse as written by the forward; logp unused */
    const float *dlogp;      /* device [S] dL/dlogp */
    void *dx;                /* device [C][D] bf16 output (overwritten), 16-byte aligned */
    void *dweight;           /* device [V][D] bf16 output (overwritten), 16-byte aligned */
    int32_t piece;           /* vocabulary entries held at a time (rounded down to a multiple of
                                256, at least 256), or 0: as many as make dz 512 MiB */
} harts_linear_logprob_bwd_args;

/* Workspace of the backward for a given piece (0: the library's choice); 0 for invalid
 * arguments.  About 2 C piece bytes of dz, and fp32 sums of dx. */
size_t harts_linear_logprob_bwd_workspace_bytes(int64_t C, int32_t V, int32_t D, int64_t S, int32_t piece);

/* Errors as the forward. */
int harts_linear_logprob_bwd(const harts_linear_logprob_bwd_args *args, harts_stream_t stream);

/* Message for the last error on the calling thread ("" if none). */
const char *harts_last_error(void);

#ifdef __cplusplus
}
#endif
#endif /* HARTS_H */
