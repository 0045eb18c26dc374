/*
 * evs.h - replay-free speculative block verification for a hybrid short-FIR /
 * modal-IIR / causal-attention target, on one GB300 (sm_103a).
 *
 * Method: "EvSpark: Lossless Speculative Decoding for Hybrid DNA Foundation Models"
 * (summary page). Figure 1(c): the target verifies the old anchor plus gamma drafts in
 * one block forward and a correction becomes the next unconsumed anchor. Figure 1(d):
 * state returns to the accepted block index k - the readable KV prefix is shortened, the
 * last L-1 outer-FIR inputs are selected and IIR state s_k is kept - with no target
 * computation replayed. Interpretation, paragraph 1: one initial-state block forward plus
 * a common state-slicing protocol (Lemma 2 block-forward contract, Lemma 3 state
 * restoration, Theorem 1 sequence-level exactness). Acceptance: greedy argmax match, or
 * rejection sampling with min(1, p/q) and a correction from norm(max(0, p - q))
 * (ReaDy summary, section 3.1 and appendix D.2).
 *
 * Target model (the pages name only the three state classes; this is the reading the
 * library implements): h = E[x]; per layer xh = h / sqrt(mean(h^2) + 1e-6), then
 *   FIR-L : v = xh W_in, y_t = sum_{j<L} taps[:, j] * v_{t-j},            h += y W_out
 *   IIR-N : u = xh W_in, s_t = lam * s_{t-1} + b * u_t (N complex poles),
 *           y = Re sum_n c_n s_{t,n},                                       h += y W_out
 *   attn  : q, k, v = xh W_q, W_k, W_v; per head softmax(q K^T / sqrt(dh)) V over the
 *           readable cache plus the block keys up to the query's position,  h += o W_o
 * logits = (h / rms(h)) W_head; p = softmax(logits / temperature).
 *
 * Conventions
 *   - Every entry point is asynchronous on the handle's stream unless stated otherwise,
 *     and never synchronises the device. Pointers marked "device" must be device memory
 *     (or managed memory) valid until the enqueued work completes.
 *   - The caller owns every buffer: weights, the workspace and all inputs and outputs.
 *     The handle stores pointers into them and owns only its host-side struct.
 *   - Matrices are "out-major": row n is output channel n, its input weights
 *     contiguous (the transpose of the math convention y = x W).
 *   - dtype EVS_DTYPE_BF16 stores weights, activations fed to projections, and K/V in
 *     bfloat16; accumulation, the residual stream, FIR inputs and the complex IIR state
 *     are fp32. EVS_DTYPE_F32 keeps everything in fp32.
 *   - Block rows are ordered m = (b * n_cand + c) * (gamma + 1) + i, i = block position
 *     (0 = anchor, i >= 1 = draft i).
 *   - Errors found on the host are returned before anything is enqueued. Kernels never
 *     trap: a condition only the device can see (a KV capacity overflow, k outside
 *     [0, gamma], a token id out of range) skips or clamps the affected access and sets a
 *     bit readable through evs_device_flags.
 */
#ifndef EVS_H
#define EVS_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct evs_handle evs_handle;

typedef enum {
    EVS_OK = 0,
    EVS_ERR_INVALID_ARG = 1, /* null pointer, bad size, unsupported shape            */
    EVS_ERR_CAPACITY = 2,    /* KV rows would exceed t_max, or workspace too small   */
    EVS_ERR_STATE = 3,       /* call out of order (slice without a verify before it) */
    EVS_ERR_CUDA = 4         /* a CUDA runtime call or kernel launch failed          */
} evs_status;

enum { EVS_LAYER_FIR = 0, EVS_LAYER_IIR = 1, EVS_LAYER_ATTN = 2 };
enum { EVS_DTYPE_F32 = 0, EVS_DTYPE_BF16 = 1 };
enum { EVS_MODE_GREEDY = 0, EVS_MODE_SAMPLING = 1 };
/* How several candidate blocks per sequence are verified under sampling (greedy commits
 * the candidate with the most accepted drafts under both, which is exact there):
 *   EVS_CAND_RECURSIVE   lossless: rejection sampling applied recursively across the
 *                        candidates that share the accepted prefix (a token tree with equal
 *                        prefixes merged); the output follows the target distribution.
 *   EVS_CAND_MAX_ACCEPT  each candidate tested alone with its own uniforms, the one with
 *                        the most accepted drafts committed (lowest index on ties); not
 *                        distribution-preserving in general. */
enum { EVS_CAND_RECURSIVE = 0, EVS_CAND_MAX_ACCEPT = 1 };

/* Bits of the device flag word (evs_device_flags). */
enum {
    EVS_FLAG_KV_OVERFLOW = 1u,    /* a write past t_max was skipped                     */
    EVS_FLAG_BAD_K = 2u,          /* slice saw k outside [0, gamma] or a bad candidate  */
    EVS_FLAG_EMPTY_RESIDUAL = 4u, /* max(0, p - q) summed to 0 in fp32; p was used      */
    EVS_FLAG_BAD_TOKEN = 8u,      /* a token id outside [0, vocab) was clamped (or, among
                                     given tokens, has the log probability -inf)       */
    EVS_FLAG_TIMEOUT = 16u,       /* a kernel gave up a bounded wait; its output is void */
    EVS_FLAG_BAD_LEN = 32u,       /* a sequence length outside its range was clamped     */
    EVS_FLAG_EMPTY_ROW = 64u,     /* a row whose tokens are all ruled out: no draw (-1)  */
    EVS_FLAG_BAD_PARENT = 128u    /* a parent that is no earlier node was read as -1     */
};

#define EVS_MAX_LAYERS 64

typedef struct {
    int32_t d;                            /* model width (multiple of 64, <= 8192)      */
    int32_t vocab;                        /* vocabulary (256 * 2^j, 256 .. 4096)        */
    int32_t n_layers;                     /* 1 .. EVS_MAX_LAYERS                        */
    int32_t layer_kind[EVS_MAX_LAYERS];   /* EVS_LAYER_*                                */
    int32_t layer_param[EVS_MAX_LAYERS];  /* FIR taps L (2..16) | IIR poles N (1,2,4,8,16,32)
                                             | attention heads H (H * head_dim == d)    */
    int32_t head_dim;                     /* attention head width (16, 32, 64 or 128)   */
    int32_t gamma;                        /* drafts per block (1..31)                   */
    int32_t batch;                        /* sequences B (1..64)                        */
    int32_t n_cand;                       /* candidate blocks C per sequence            */
    int32_t t_max;                        /* KV capacity per sequence, tokens (<= 2^21) */
    int32_t prefill_chunk;                /* tokens per sequence per prefill pass       */
    int32_t dtype;                        /* EVS_DTYPE_*                                */
    int32_t mode;                         /* EVS_MODE_*                                 */
    float temperature;                    /* p = softmax(logits / temperature), > 0     */
    float near_tie_tau;                   /* relative threshold of the near-tie flags   */
    int32_t cand_rule;                    /* EVS_CAND_* (n_cand > 1, sampling)          */
} evs_config;

typedef struct {
    const void* w_in;        /* FIR, IIR: [d][d] out-major, dtype                        */
    const void* w_out;       /* FIR, IIR: [d][d] out-major, dtype                        */
    const float* fir_taps;   /* FIR: [d][L] fp32, taps[c][j] multiplies v_{t-j}[c]        */
    const float* iir_lambda; /* IIR: [d][N][2] fp32 (re, im) poles                         */
    const float* iir_b;      /* IIR: [d][N][2] fp32 input coefficients                     */
    const float* iir_c;      /* IIR: [d][N][2] fp32 readout coefficients                   */
    const void* w_qkv;       /* attn: [3d][d] out-major, dtype; rows q (0..d-1), k, v     */
    const void* w_o;         /* attn: [d][d] out-major, dtype                              */
} evs_layer_weights;

typedef struct {
    const void* embed;                    /* [vocab][d] dtype                            */
    const void* head;                     /* [vocab][d] out-major dtype                  */
    evs_layer_weights layer[EVS_MAX_LAYERS];
} evs_weights;

/* Caller-side view of the decode state, for import / export (checkpoint and resume;
 * the slicing contract of Figure 1(d) is exactly this state). Pointers are device
 * memory except kv_len. Arrays are indexed by layer index; entries of other kinds are
 * ignored. */
typedef struct {
    int32_t* kv_len;                        /* host [B] readable KV length per sequence */
    int32_t t_stride;                       /* rows per (sequence, head) in k and v      */
    void* k[EVS_MAX_LAYERS];                /* attn: [B][H][t_stride][dh] dtype          */
    void* v[EVS_MAX_LAYERS];                /* attn: [B][H][t_stride][dh] dtype          */
    float* fir_tail[EVS_MAX_LAYERS];        /* FIR: [B][L-1][d] fp32, oldest input first */
    float* iir_state[EVS_MAX_LAYERS];       /* IIR: [B][d][N][2] fp32                    */
} evs_state_view;

/* Internal buffers exposed read-only for tests and diagnostics (evs_debug_buffer). */
enum {
    EVS_BUF_LOGITS = 0,     /* [B*C*(gamma+1)][vocab] fp32, last verify                 */
    EVS_BUF_FIR_STAGE = 1,  /* layer: [B][C][L-1+gamma+1][d] fp32 = [tail || inputs v]    */
    EVS_BUF_IIR_U = 2,      /* layer: [B][C][gamma+1][d] fp32 scan inputs u_0..u_gamma    */
    EVS_BUF_K_CACHE = 3,    /* layer: [B][H][t_max][dh] dtype                             */
    EVS_BUF_V_CACHE = 4,    /* layer: [B][H][t_max][dh] dtype                             */
    EVS_BUF_K_SIDE = 5,     /* layer, n_cand > 1: [B][C][H][gamma+1][dh] dtype block keys  */
    EVS_BUF_V_SIDE = 6,     /* layer, n_cand > 1: [B][C][H][gamma+1][dh] dtype             */
    EVS_BUF_KV_LEN = 7,     /* [B] int32                                                  */
    EVS_BUF_FIR_TAIL = 8,   /* layer: [B][L-1][d] fp32                                    */
    EVS_BUF_IIR_STATE = 9,  /* layer: [B][d][N][2] fp32                                   */
    EVS_BUF_CAND_K = 10,    /* [B][C] int32 accepted drafts per candidate, last verify
                               (EVS_CAND_RECURSIVE sampling: drafts on the accepted path) */
    EVS_BUF_CAND_CORR = 11  /* [B][C] int32 correction per candidate, last verify
                               (EVS_CAND_RECURSIVE sampling: -1 but for the committed one) */
};

typedef struct {
    void* ptr;        /* device pointer into the workspace (do not write)              */
    size_t bytes;
} evs_buffer_info;

/* Bytes of device workspace that evs_create needs for this configuration (0 if the
 * configuration is invalid). Pure host function. */
size_t evs_workspace_bytes(const evs_config* cfg);

/* Validate the configuration, lay out state and scratch buffers inside the caller's
 * workspace (device, >= evs_workspace_bytes, 256-byte aligned) and build the handle.
 * Weights are device pointers in the layouts above and must outlive the handle.
 * stream is a cudaStream_t (NULL = legacy default stream). The state starts empty
 * (kv_len = 0, FIR tails and IIR states zero); the zeroing is enqueued on the stream.
 * Returns EVS_ERR_INVALID_ARG for a bad configuration or pointer, EVS_ERR_CAPACITY if
 * ws_bytes is too small, EVS_ERR_CUDA if a CUDA call fails. */
evs_status evs_create(const evs_config* cfg, const evs_weights* weights, void* workspace,
                      size_t ws_bytes, void* stream, evs_handle** out);

/* Free the host-side handle. Does not touch caller-owned memory. NULL is allowed. */
void evs_destroy(evs_handle* h);

/* Change the stream later calls enqueue on (a cudaStream_t). */
evs_status evs_set_stream(evs_handle* h, void* stream);

/* Return the state to empty (kv_len 0, zero FIR tails and IIR states). */
evs_status evs_reset(evs_handle* h);

/* Consume P prefix tokens per sequence from the current state, prefill_chunk tokens per
 * pass, committing every pass (no logits are produced). tokens: device int32 [B][P],
 * ids in [0, vocab). Prefill is excluded from the pages' token benchmarks (Perspective,
 * paragraph 1). EVS_ERR_CAPACITY if kv_len + P could exceed t_max. */
evs_status evs_prefill(evs_handle* h, const int32_t* tokens, int32_t P);

/* One block forward plus acceptance (Figure 1(c); Lemma 2).
 *   tokens   device int32 [B][C][gamma+1]: position 0 is the anchor, 1..gamma drafts.
 *   anchor   device int32 [B] or NULL: when given, replaces tokens[b][c][0] for every
 *            candidate (pass the previous round's correction to chain rounds).
 *   q_probs  device fp32 [B][C][gamma][vocab]: draft distributions (sampling mode; NULL
 *            in greedy mode).
 *   uniforms device fp32 [B][C][gamma+1] in [0, 1): u[j] tests draft j+1 by
 *            u * q(d) < p(d); u[gamma] draws the correction or bonus by inverse CDF over
 *            ascending ids (sampling mode; NULL in greedy mode).
 * Outputs (device, written by the enqueued kernels):
 *   accepted_len [B] int32: k, accepted drafts of the committed candidate (0..gamma).
 *   correction   [B] int32: next anchor (correction at the first rejection, or bonus).
 *   best_cand    [B] int32 or NULL: committed candidate (see EVS_CAND_*: the lowest
 *                candidate on the accepted path, or the most accepted drafts with the
 *                lowest index on ties); required when n_cand > 1.
 *   near_tie     [B] uint32 or NULL: 1 when a decision was within near_tie_tau of
 *                flipping (greedy top-2 logit gap < tau * rms(logits); |u q - p| < tau p;
 *                u * sum(r) within tau * sum(r) of an inverse-CDF boundary).
 * Writes the block's K/V rows, FIR inputs and IIR scan inputs u_0..u_gamma into the
 * workspace for evs_slice_state. State itself is not modified.
 * EVS_ERR_CAPACITY if kv_len + gamma + 1 could exceed t_max. */
evs_status evs_verify_block(evs_handle* h, const int32_t* tokens, const int32_t* anchor,
                            const float* q_probs, const float* uniforms,
                            int32_t* accepted_len, int32_t* correction, int32_t* best_cand,
                            uint32_t* near_tie);

/* State slicing at the accepted index (Figure 1(d); Lemma 3), in place, no replay of the
 * forward: kv_len += k + 1 (for n_cand > 1 the chosen candidate's k+1 block K/V rows are
 * first copied into the cache), FIR tail <- the last L-1 inputs up to block position k, IIR
 * state <- s_k (k+1 steps of the diagonal recurrence from the pre-round state over the kept
 * scan inputs, the same operations as the verify's scan). accepted_len and best_cand are
 * device int32 [B] (usually the outputs of the verify; best_cand may be NULL when
 * n_cand == 1). k stays on the device: nothing is read back. EVS_ERR_STATE if no verify was
 * enqueued since the last slice, prefill, decode step or import. */
evs_status evs_slice_state(evs_handle* h, const int32_t* accepted_len, const int32_t* best_cand);

/* Replay-based recovery, the ablation that slicing replaces (EvSpark summary,
 * Interpretation: slicing against a second target forward over the accepted prefix). After
 * evs_verify_block, k and the committed candidate are read back to the host (the stream is
 * synchronised), then a committed forward runs over that candidate's accepted tokens
 * [anchor, d_1..d_k] from the pre-round state, as a prefill does. The state it leaves equals
 * the one evs_slice_state leaves, up to rounding. One sequence only (batch == 1): the
 * accepted lengths of different sequences differ.
 *   tokens, anchor  as given to the verify (anchor may be NULL).
 *   accepted_len, best_cand  the verify's outputs (device; best_cand NULL when n_cand == 1).
 * EVS_ERR_STATE without a preceding verify; EVS_ERR_INVALID_ARG if batch > 1, a pointer is
 * missing, or k / the candidate read back is out of range. */
evs_status evs_replay_state(evs_handle* h, const int32_t* tokens, const int32_t* anchor,
                            const int32_t* accepted_len, const int32_t* best_cand);

/* One step of plain autoregressive decoding: the target's native token-by-token loop that
 * block verification is measured against (EvSpark summary, Interpretation: the
 * identity-drafter control is reported as a multiple of native throughput). Every
 * sequence consumes one token and its state advances in place (the K/V row is appended,
 * the FIR tail shifts, the IIR state takes one step), then the next token is drawn from
 * softmax(logits / temperature) of the new position: the argmax, lowest id on ties
 * (greedy mode), or the inverse CDF at u[b] over ascending ids (sampling mode). Uses the
 * verify's kernels with one row per sequence.
 *   tokens    device int32 [B]: the token each sequence consumes.
 *   uniforms  device fp32 [B] in [0, 1) (sampling mode; NULL in greedy mode).
 *   next      device int32 [B]: the drawn next token. It may alias tokens (the draw is
 *             written after every read of tokens, in stream order).
 *   near_tie  device uint32 [B] or NULL: 1 when the draw was within near_tie_tau of
 *             flipping (same tests as evs_verify_block).
 * The step's logits are left in EVS_BUF_LOGITS rows [0, B). EVS_ERR_INVALID_ARG for a
 * missing pointer, EVS_ERR_CAPACITY if kv_len + 1 could exceed t_max. */
evs_status evs_decode_step(evs_handle* h, const int32_t* tokens, const float* uniforms, int32_t* next,
                           uint32_t* near_tie);

/* Copy a caller state into the handle (import) or the handle's state out (export).
 * Enqueued copies; export writes kv_len to the host view after synchronising the
 * stream. Import rejects kv_len > t_max or > t_stride with EVS_ERR_CAPACITY. */
evs_status evs_import_state(evs_handle* h, const evs_state_view* view);
evs_status evs_export_state(evs_handle* h, const evs_state_view* view);

/* Read-only location of an internal buffer (see EVS_BUF_*); layer is a layer index
 * where the buffer is per layer. EVS_ERR_INVALID_ARG if the buffer does not exist. */
evs_status evs_debug_buffer(evs_handle* h, int32_t which, int32_t layer, evs_buffer_info* out);

/* Synchronise the stream and return the device flag word (EVS_FLAG_*); clear it when
 * clear != 0. */
evs_status evs_device_flags(evs_handle* h, uint32_t* flags, int32_t clear);

/* Kernel kinds for per-kind timing. */
enum {
    EVS_K_EMBED = 0, EVS_K_NORM = 1, EVS_K_GEMM = 2, EVS_K_FIR = 3, EVS_K_IIR = 4,
    EVS_K_KV_WRITE = 5, EVS_K_ATTN = 6, EVS_K_ATTN_COMBINE = 7, EVS_K_ACCEPT = 8,
    EVS_K_SLICE = 9, EVS_K_ADVANCE = 10, EVS_K_COUNT = 11
};

/* Per-kernel-kind timing with CUDA events (tracing for measurement; the pages describe no
 * tracing mechanism). While enabled, every launch is bracketed by two events recorded on
 * the handle's stream, so calls must not be captured into a CUDA graph. evs_profile_read
 * synchronises the stream and returns, for each kind < n, the launches and summed
 * milliseconds since the previous read, then clears the counters. */
evs_status evs_profile_enable(evs_handle* h, int32_t on);
evs_status evs_profile_read(evs_handle* h, int32_t* launches, float* ms, int32_t n);

/* Number of kernel launches the last public call enqueued (for accounting). */
int32_t evs_last_launch_count(evs_handle* h);

/* Diagnostics: Y[m][n] (+)= sum_k X[m][k] W[n][k] with the library's projection kernel
 * (the same launch path the block forward uses). X: device bf16 [x_rows][K] (x_rows >= M),
 * W: device bf16 out-major [N][K], Y: device fp32 [M][ldy]. Uses the handle's stream and
 * split-K scratch; needs a bf16 handle, M <= 512, N % 128 == 0, K % 64 == 0, K <= d and
 * N <= max(3d, vocab). EVS_ERR_INVALID_ARG otherwise. */
evs_status evs_debug_projection(evs_handle* h, const void* X, int32_t x_rows, const void* W, float* Y,
                                int32_t M, int32_t N, int32_t K, int32_t ldy, int32_t accumulate);

/* Projection for callers that cannot allocate device memory: no handle, no workspace,
 * no cudaMalloc / cudaFree or allocating library call. The pages have no counterpart of
 * this entry point; it exists for hosts that own all device memory and forbid allocation
 * while they execute (plugin-style engines), and for latency-critical loops where an
 * allocation would synchronise the device.
 * Computes Y[m][n] (+)= sum_k X[m][k] W[n][k] with the same tcgen05 kernel as
 * evs_debug_projection; split-K partial sums always go through the fixed array (never
 * through a thread-block cluster). X: device bf16 [x_rows][K] (x_rows >= M); W: device bf16
 * out-major [N][K]; Y: device fp32 [M][ldy]; stream: a cudaStream_t. Needs M <= 512,
 * N % 128 == 0, K % 64 == 0.
 * Scratch: one fixed array of 8 MiB of fp32 partial sums, 256 arrival counters and a flag
 * word, compiled into the library and held on every GPU that loads it until the process
 * exits. The K split is capped so that its partial sums (splits x M x N floats) fit 2^21
 * floats (a shape that fits no split runs unsplit), so the only size limit is N <= 32768
 * (one counter per 128-channel tile); wider N returns EVS_ERR_CAPACITY.
 * The first call on a device (of this function or evs_projection_noalloc_flags) looks up
 * the array's device address, sets the kernel's shared-memory limit for that device and
 * clears the flag word; make that first call before any stream capture. The set-up is
 * guarded, so host threads may make their first calls concurrently. A device reset
 * (cudaDeviceReset) invalidates it: reload the library after one.
 * Every call reuses the same array and finds the previous call's contents there; the
 * counters are cleared on the stream at each call. Calls that overlap on the GPU (issued
 * on different streams, or from several host threads) race on it: order them on one
 * stream. A kernel that gives up a bounded wait sets EVS_FLAG_TIMEOUT in the array's flag
 * word, and Y is then void; read the word with evs_projection_noalloc_flags.
 * EVS_ERR_INVALID_ARG for bad shapes or pointers, EVS_ERR_CUDA if a CUDA call fails. */
evs_status evs_projection_noalloc(const void* X, int32_t x_rows, const void* W, float* Y, int32_t M,
                                  int32_t N, int32_t K, int32_t ldy, int32_t accumulate, void* stream);

/* Device status of evs_projection_noalloc on the current device: synchronises stream, then
 * writes to *flags the EVS_FLAG_* bits (EVS_FLAG_TIMEOUT) that its calls have set since the
 * word was last cleared, and clears it when clear != 0 (enqueued on stream). Allocates
 * nothing. EVS_ERR_INVALID_ARG for a null flags pointer, EVS_ERR_CUDA if a CUDA call
 * fails. */
evs_status evs_projection_noalloc_flags(uint32_t* flags, int32_t clear, void* stream);

/* ---- Stand-alone operators ----------------------------------------------------------
 * No handle: every call says what it works on. The caller owns all memory; the work is
 * enqueued on stream (a cudaStream_t of the current device) and nothing is allocated or
 * synchronised, so calls may be captured into CUDA graphs. Strides are in elements, the last
 * dimension is contiguous, offsets are 64-bit. Sums, statistics and states are fp32 or wider.
 * flags, in every struct: device uint32 or NULL, an EVS_FLAG_* word that the kernels OR into
 * (never cleared by them). Bad arguments return EVS_ERR_INVALID_ARG before anything is
 * enqueued; an empty call (no rows, no sequences) returns EVS_OK and does nothing. */

/* The filtered draw. Per row r, with l the logits, T, k, p and m the row's parameters:
 *   w_i = exp((l_i - max l) / T), tokens ordered by (l descending, id ascending);
 *   keep the first k; of these the shortest prefix whose mass before a token is below p times
 *   their mass (at least one token); of these the tokens with w_i >= m * max w;
 *   token = the smallest id whose cumulative kept mass over ascending ids exceeds u * total.
 * The weights are summed in 64-bit fixed point (2^-45 of the largest; smaller ones are 0): the
 * same inputs give the same token whatever the launch, and equal logits go by their ids. NaN and
 * -inf logits are ruled out; where the largest logit is +inf, the +inf tokens share the mass. A row with every token
 * ruled out gives token -1, logprob -inf, zero probabilities and EVS_FLAG_EMPTY_ROW. */
typedef struct {
    int32_t rows, vocab;         /* vocab 1 .. 262144                                       */
    int32_t dtype;               /* EVS_DTYPE_* of the logits                               */
    int64_t ld;                  /* row stride of logits (>= vocab)                         */
    const void* logits;          /* device [rows][vocab]                                    */
    const float* temperature;    /* device [rows] or NULL (1); not above 0: the argmax      */
    const int32_t* top_k;        /* device [rows] or NULL; outside [1, vocab): off          */
    const float* top_p;          /* device [rows] or NULL; >= 1 or NaN: off, <= 0: one token */
    const float* min_p;          /* device [rows] or NULL; not above 0: off, above 1: as 1  */
    const float* uniforms;       /* device [rows], in [0, 1) (clamped)                      */
    int32_t* token;              /* device [rows]                                           */
    float* logprob;              /* device [rows] or NULL: log of the token's kept share    */
    float* probs;                /* device [rows][vocab] or NULL: the distribution drawn from */
    int64_t probs_ld;            /* row stride of probs                                     */
    uint32_t* flags;
} evs_sample_args;
evs_status evs_sample(const evs_sample_args* args, void* stream);

/* The native decode step (evs_decode_step) with the filtered draw over the step's logits in
 * place of the draw from softmax(logits / temperature); the configuration's mode and temperature
 * are not used. draw: temperature, top_k, top_p, min_p, uniforms, logprob, probs and probs_ld are
 * taken from it ([batch] rows); its other members are ignored. next: device int32 [B], may alias
 * tokens. EVS_FLAG_EMPTY_ROW goes to the handle's flag word. */
evs_status evs_decode_filtered(evs_handle* h, const int32_t* tokens, const evs_sample_args* draw, int32_t* next);

/* Attention for a batch that shares a prefix. Query (b, c, i) of head h reads, with the K/V head
 * g = h / (heads / kv_heads): the `prefix` shared rows (one copy for the whole batch), the own
 * rows [0, own_len[b] - own_skip) of its sequence (all its candidates share them), and the block
 * rows j <= i of its candidate. o = softmax(scale q k^T) v over them; lse = log of the sum of
 * exponentials. The block rows lie in k_block / v_block, or (both NULL, n_cand 1) in the own rows
 * behind the readable ones, row own_len[b] - own_skip + j.
 * Lengths outside [0, own_max] are clamped (EVS_FLAG_BAD_LEN); block rows past own_max are left
 * out (EVS_FLAG_KV_OVERFLOW). A query whose every score is -inf gives o = 0 and lse = -inf; one whose
 * kernel gave up a bounded wait gives NaN for both (EVS_FLAG_TIMEOUT). Rows that no query reads may hold
 * anything. K, V and o are dtype; q is q_dtype and enters every product as
 * dtype: fp32 queries of a bf16 cache are rounded to bf16. Statistics and accumulators are fp32; softmax
 * weights enter the products as bf16 on the tensor cores (dtype bf16, head_dim 64 or 128, rows on 16
 * bytes) and as fp32 elsewhere. */
typedef struct {
    int32_t batch, n_cand, block;        /* 1 .. 1024 sequences, <= 64 candidates, <= 128 positions */
    int32_t heads, kv_heads, head_dim;   /* heads a multiple of kv_heads; 16, 32, 64 or 128 */
    int32_t dtype, q_dtype;              /* EVS_DTYPE_*                                     */
    int32_t prefix, own_max;             /* shared rows; rows of one sequence's own K/V     */
    int32_t own_skip;                    /* subtracted from own_len (rows counted elsewhere) */
    float scale;                         /* 0: 1 / sqrt(head_dim)                           */
    const void* q;                       /* device, row (b * n_cand + c) * block + i: heads x head_dim */
    int64_t q_ld;
    const void *k_prefix, *v_prefix;     /* device [kv_heads][prefix][head_dim]             */
    int64_t prefix_row, prefix_head;     /* strides of both                                 */
    const void *k_own, *v_own;           /* device [batch][kv_heads][own_max][head_dim]     */
    int64_t own_row, own_head, own_seq;
    const int32_t* own_len;              /* device [batch]                                  */
    const void *k_block, *v_block;       /* device [batch * n_cand][kv_heads][block][head_dim] or NULL */
    int64_t block_row, block_head, block_cand;
    void* o;                             /* device, rows as q                               */
    int64_t o_ld;
    float* lse;                          /* device [batch * n_cand * block][heads] or NULL  */
    void* workspace;                     /* device, 256-byte aligned; not shared by calls that may overlap */
    size_t ws_bytes;
    uint32_t* flags;
} evs_shared_attn_args;
/* Bytes of workspace for these sizes (pointers may still be null; 0 if invalid). */
size_t evs_shared_attention_workspace(const evs_shared_attn_args* args);
evs_status evs_shared_attention(const evs_shared_attn_args* args, void* stream);

/* Short causal convolution of every channel, with bias and SiLU (the FIR mixer of a selective
 * layer): y_t[c] = act(bias[c] + sum_{j < taps} weight[c][j] x_{t-j}[c]), the inputs before the
 * first token taken from tail_in. Sequence b has lens[b] tokens (NULL: all have `tokens`; clamped
 * to [0, tokens]); rows of y past them are left as they were. tail_out gets the last taps - 1
 * inputs at that point, so state slicing at k is a call with lens k + 1 and y NULL. tail_out may
 * be tail_in; y must not overlap x. */
typedef struct {
    int32_t batch, tokens, width;
    int32_t taps;                /* 2 .. 16                                                 */
    int32_t dtype;               /* of x and y                                              */
    int32_t silu;                /* 1: act = v / (1 + exp(-v)), 0: none                     */
    const void* x;               /* device [batch][tokens][width], strides x_seq, x_ld      */
    int64_t x_ld, x_seq;
    void* y;                     /* likewise, or NULL when only the tail is wanted          */
    int64_t y_ld, y_seq;
    const float* weight;         /* device [width][taps]: weight[c][j] multiplies x_{t-j}   */
    const float* bias;           /* device [width] or NULL                                  */
    const float* tail_in;        /* device [batch][taps - 1][width], oldest first, or NULL (0) */
    float* tail_out;             /* likewise, or NULL                                       */
    const int32_t* lens;         /* device [batch] or NULL                                  */
    uint32_t* flags;
} evs_conv_args;
evs_status evs_causal_conv(const evs_conv_args* args, void* stream);

/* Selective scan (the modal IIR mixer's input-dependent sibling). Per channel c, state n:
 *   dl_t = softplus(dt_t + dt_bias)  (or dt_t + dt_bias where softplus is 0)
 *   s_t  = exp(dl_t A[c][n]) s_{t-1} + dl_t x_t B_t[n]
 *   y_t  = (sum_n C_t[n] s_t[n] + D[c] x_t) * z_t / (1 + exp(-z_t))
 * A is finite and normally negative. lens, y and the two states as in evs_causal_conv: state_out
 * is the state after lens[b] tokens and may be state_in; y must not overlap the inputs. States
 * and A start on 16 bytes. */
typedef struct {
    int32_t batch, tokens, width;
    int32_t states;              /* 4, 8, 16 or 32                                          */
    int32_t dtype;               /* of x, dt, z, B, C and y                                 */
    int32_t softplus;
    const void* x;               /* device [batch][tokens][width]                           */
    int64_t x_ld, x_seq;
    const void* dt;              /* device [batch][tokens][width]                           */
    int64_t dt_ld, dt_seq;
    const void* z;               /* device [batch][tokens][width] or NULL (no gate)         */
    int64_t z_ld, z_seq;
    const void* B;               /* device [batch][tokens][states]                          */
    int64_t b_ld, b_seq;
    const void* C;               /* device [batch][tokens][states]                          */
    int64_t c_ld, c_seq;
    void* y;                     /* device [batch][tokens][width], or NULL                  */
    int64_t y_ld, y_seq;
    const float* A;              /* device [width][states]                                  */
    const float* D;              /* device [width] or NULL (0)                              */
    const float* dt_bias;        /* device [width] or NULL (0)                              */
    const float* state_in;       /* device [batch][width][states] or NULL (0)               */
    float* state_out;            /* likewise, or NULL                                       */
    const int32_t* lens;         /* device [batch] or NULL                                  */
    uint32_t* flags;
    void* workspace;             /* device, 16-byte aligned, or NULL where none is needed; not shared
                                    by calls that may overlap                               */
    size_t ws_bytes;
} evs_scan_args;
/* Bytes of workspace for these sizes (0: none; prompts of few sequences are run in segments). */
size_t evs_selective_scan_workspace(int32_t batch, int32_t tokens, int32_t width, int32_t states);
evs_status evs_selective_scan(const evs_scan_args* args, void* stream);

/* Log probabilities of given tokens, the row's entropy and its largest tokens. Per row r, with T its
 * temperature: y_i = (l_i - max l) / T, Z = sum exp(y_i);
 *   logprob[r][j] = y_t - log Z for t = tokens[r][j],  entropy[r] = -sum p_i log p_i (natural logarithms),
 *   top_token[r][0 .. top) the largest logits' ids in the order (logit descending, id ascending), and
 *   top_logprob their log probabilities.
 * NaN and -inf logits are ruled out (-inf); where the largest logit is +inf, the +inf tokens share the
 * mass. A temperature that is not above zero puts all mass on the first largest token; one above 1e30 is
 * taken as 1e30. Places of top behind the last token that is not ruled out hold id -1 and -inf. A given id
 * outside [0, vocab) has -inf (EVS_FLAG_BAD_TOKEN); a row with every token ruled out has -inf, entropy 0,
 * ids -1 (EVS_FLAG_EMPTY_ROW). Sums are fp32 over a running maximum, and carry along what their additions
 * lose; the ids are exact. */
typedef struct {
    int32_t rows, vocab;         /* at most 2^24 each                                       */
    int32_t n_tokens, top;       /* given tokens a row; largest ones, at most 64 and vocab  */
    int32_t dtype;               /* EVS_DTYPE_* of the logits                               */
    int64_t ld;                  /* row stride of logits (>= vocab)                         */
    const void* logits;          /* device [rows][vocab]                                    */
    const float* temperature;    /* device [rows] or NULL (1)                               */
    const int32_t* tokens;       /* device [rows][n_tokens]                                 */
    float* logprob;              /* device [rows][n_tokens]                                 */
    float* entropy;              /* device [rows] or NULL                                   */
    float* top_logprob;          /* device [rows][top]                                      */
    int32_t* top_token;          /* device [rows][top]                                      */
    uint32_t* flags;
} evs_logprob_args;
evs_status evs_token_logprobs(const evs_logprob_args* args, void* stream);

/* Causal attention over whole prompts packed behind each other. Sequence b has rows starts[b] ..
 * starts[b + 1] - 1 of q, k, v and o; its query row i of head h reads its rows j <= i with the K/V head
 * g = h / (heads / kv_heads): o = softmax(scale q k^T) v, lse = log of the sum of exponentials. Rows of no
 * sequence (before starts[0], behind starts[batch]) may hold anything; o is left as it was there, or with
 * zero_rest is zero, and lse is -inf. Starts are made to ascend within [0, tokens] (EVS_FLAG_BAD_LEN where
 * they did not). A query whose every score is -inf gives o = 0 and lse = -inf; one whose kernel gave up a
 * bounded wait gives NaN for both (EVS_FLAG_TIMEOUT). Types, statistics and weights as in
 * evs_shared_attention. A value of V that is not finite shows in the rows that read it (0 times it, where their
 * weights of it are 0, may be NaN, even in a row whose every score is -inf), and in no other. How the keys are
 * dealt, and with it the last bits and the time, goes by tokens, batch and heads, as if all sequences were of one
 * length. bf16 with heads of 64 or 128 and q, k and v on 16 bytes (their strides, too) runs on the tensor cores,
 * everything else on CUDA cores. */
typedef struct {
    int32_t tokens, batch;               /* rows of the buffers, sequences (<= 1024)        */
    int32_t heads, kv_heads, head_dim;   /* heads a multiple of kv_heads; 16, 32, 64 or 128 */
    int32_t dtype;                       /* EVS_DTYPE_* of all                              */
    int32_t zero_rest;
    float scale;                         /* 1e-30 to 1e30; 0: 1 / sqrt(head_dim)            */
    const void* q;                       /* device [tokens][heads][head_dim]                */
    int64_t q_row, q_head;
    const void *k, *v;                   /* device [tokens][kv_heads][head_dim]             */
    int64_t kv_row, kv_head;             /* strides of both                                 */
    const int32_t* starts;               /* device [batch + 1]                              */
    void* o;                             /* device [tokens][heads][head_dim], heads contiguous */
    int64_t o_row;
    float* lse;                          /* device [tokens][heads] or NULL                  */
    void* workspace;                     /* device, 256-byte aligned, or NULL where none is needed; not shared by
                                            calls that may overlap                          */
    size_t ws_bytes;
    uint32_t* flags;
} evs_prompt_attn_args;
/* Bytes of workspace for these sizes (pointers may still be null; 0: none is needed, or invalid). */
size_t evs_prompt_attention_workspace(const evs_prompt_attn_args* args);
evs_status evs_prompt_attention(const evs_prompt_attn_args* args, void* stream);

/* Attention of a tree of drafted tokens over each sequence's cache. Node i of sequence b reads the cached
 * rows [0, cache_len[b]) and the nodes on its path to the root: itself, parent[b][i], that one's parent,
 * and so on to a parent of -1 (a node below the last cached token). A parent comes before its children;
 * one that does not is read as -1 (EVS_FLAG_BAD_PARENT). Sequence b has lens[b] nodes (NULL: all have
 * `nodes`; clamped to [0, nodes], EVS_FLAG_BAD_LEN); o of the rest is left as it was, or with zero_rest is
 * zero, and their lse is -inf. A tree of one node is a decode step, a chain a verify block.
 * The nodes' K/V lie in k_nodes / v_nodes, or (both NULL) in the cache behind the readable rows, row
 * cache_len[b] + j; rows past the capacity are left out (EVS_FLAG_KV_OVERFLOW). Lengths outside [0,
 * capacity] are clamped (EVS_FLAG_BAD_LEN). Rows that no query reads may hold anything, and a
 * node's V that is not finite shows in that node and those below it alone (as in evs_prompt_attention).
 * bf16 with heads of 64 or 128 and K and V on 16 bytes (their strides, too, none of them 0) runs on the tensor cores,
 * everything else on CUDA cores: one cache expanded over a batch, as well. Everything else as in
 * evs_shared_attention. */
typedef struct {
    int32_t batch, nodes;                /* 1 .. 1024 sequences, 1 .. 128 nodes             */
    int32_t heads, kv_heads, head_dim;   /* heads a multiple of kv_heads; 16, 32, 64 or 128 */
    int32_t dtype;                       /* EVS_DTYPE_* of all                              */
    int32_t capacity;                    /* rows of one sequence's cache                    */
    int32_t zero_rest;
    float scale;                         /* 1e-30 to 1e30; 0: 1 / sqrt(head_dim)            */
    const void* q;                       /* device, row b * nodes + i: heads x head_dim     */
    int64_t q_ld;
    const void *k_cache, *v_cache;       /* device [batch][kv_heads][capacity][head_dim]    */
    int64_t cache_row, cache_head, cache_seq;
    const int32_t* cache_len;            /* device [batch]                                  */
    const int32_t* parents;              /* device [batch][nodes], stride parents_seq (0: one tree for all) */
    int64_t parents_seq;
    const void *k_nodes, *v_nodes;       /* device [batch][kv_heads][nodes][head_dim] or NULL */
    int64_t node_row, node_head, node_seq;
    const int32_t* lens;                 /* device [batch] or NULL                          */
    void* o;                             /* device, rows as q                               */
    int64_t o_ld;
    float* lse;                          /* device [batch][nodes][heads] or NULL            */
    void* workspace;                     /* device, 256-byte aligned; not shared by calls that may overlap */
    size_t ws_bytes;
    uint32_t* flags;
} evs_tree_attn_args;
size_t evs_tree_attention_workspace(const evs_tree_attn_args* args);
evs_status evs_tree_attention(const evs_tree_attn_args* args, void* stream);

/* Static description of a status code. */
const char* evs_status_str(evs_status s);

#ifdef __cplusplus
}
#endif
#endif /* EVS_H */
