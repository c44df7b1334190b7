/*
 * dwpt_seq.h -- C ABI of the sequence-model operators of libdwpt_scan.so:
 * embedding lookup and its gradient by sorted tokens, the short causal
 * convolution, the selective state-space scan and the gated linear recurrence,
 * each with its gradient and (all but the embedding) its form for single
 * tokens; tokens sorted by expert and back, with gradients; sampling of tokens.
 *
 * The selective scan is the affine recurrence of SCAN_OP_AFFINE over real
 * maps, one per channel and state, made from the inputs on the way in and
 * contracted over the states on the way out; sequences packed one behind the
 * other are its segments.  The gradient of the lookup is a stable split of
 * the positions by token followed by the sum of every segment.
 *
 * Conventions (besides those of dwpt_scan.h: device pointers on the current
 * device, stream as void*, calls only enqueue, argument errors returned
 * before anything is launched):
 *   - Channels come last and are contiguous, at most 2^20; a `*_stride` counts
 *     elements from one row to the next, at most 2^31.  Rows and sequences
 *     number less than 2^31.  16-byte aligned pointers, strides and
 *     channel counts select the vector path, anything else a slower path with
 *     the same results, but for the convolution's dweight and dbias: the path
 *     decides which rows are added up first, so their last bits may differ.
 *   - Rows are flat.  With seq_offsets == NULL there are `seqs` sequences of
 *     rows / seqs rows each.  Otherwise seq_offsets holds seqs + 1 ascending
 *     int32 (device memory) and sequence s is rows [seq_offsets[s],
 *     seq_offsets[s+1]), possibly none; seqs may be 0.  Rows outside every
 *     sequence (before the first, behind the last) are neither read nor
 *     written.  Values that do not ascend or lie outside 0 .. rows give
 *     unspecified results, but no access outside the arrays.
 *   - SEQ_F32, SEQ_F16 and SEQ_BF16 arrays are converted to 32 bits on the
 *     way in; every sum, state and activation is held in 32 bits; results are
 *     rounded once, to nearest even.  Infinities and NaN reach what the
 *     formulas let them reach and nothing else; which of the two a state that
 *     is no longer finite reads as may depend on how its sequence is cut.
 *   - Workspace is the caller's: `workspace` must hold the bytes the matching
 *     *_workspace function returns for the same arguments (256-byte aligned;
 *     contents need not be kept or cleared).  Nothing is allocated and no
 *     state is kept, so the calls can be captured into a graph, and calls
 *     with different workspaces may overlap in time.
 *   - No floating-point atomics: results repeat bit for bit (on one path, see
 *     above).
 *   - Bounded waits: workgroups of the gated recurrence wait for one another.
 *     A wait that gives up (after some seconds; see seq_set_spin_limit) yields
 *     NaN from its row on, and seq_get_device_error reports it.
 *   - Outputs must not overlap inputs or one another (SCAN_ERR_INVALID),
 *     except where a state is updated in place.
 */
#ifndef DWPT_SEQ_H
#define DWPT_SEQ_H

#include "dwpt_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    SEQ_F32 = 0,
    SEQ_F16 = 1,
    SEQ_BF16 = 2
} seq_dtype_t;

typedef enum {
    SEQ_ACT_NONE = 0,
    SEQ_ACT_SILU = 1 /* u / (1 + exp(-u)) */
} seq_activation_t;

/*
 * Synchronises `stream`, then reads and clears the current device's word of the calls of this header:
 * SCAN_ERR_TIMEOUT if a wait gave up since the last check (the results of that call hold NaN then), else SCAN_OK.
 */
scan_status_t seq_get_device_error(void* stream);

/* Looks after which a wait gives up (process-wide, thread-safe; 0: at once).  Returns the old value; default 2^22. */
uint32_t seq_set_spin_limit(uint32_t polls);

/*
 * out[i] = scale * table[tokens[i]], i < n; a token outside 0 .. n_rows - 1
 * gives a row of zeros.  tokens: n int32 (token_bytes 4) or int64 (8);
 * table: n_rows x channels, out: n x channels (contiguous), both dtype.
 */
scan_status_t embedding_lookup(seq_dtype_t dtype, const void* tokens, int token_bytes, size_t n, const void* table,
                               int64_t table_stride, size_t n_rows, uint32_t channels, float scale, void* out,
                               void* stream);

/*
 * Gradient of embedding_lookup: dtable[v] = scale * the sum of dout[i] over
 * the positions i with tokens[i] == v, added up in an order that depends on
 * the tokens alone; zero for rows without a position.  accumulate != 0 adds to what dtable holds instead and leaves the
 * other rows untouched.  Tokens outside the table are left out.
 * dout: n x channels of dtype; dtable: n_rows x channels (contiguous) of
 * dtype or SEQ_F32.  n < 2^31, n_rows <= 2^24.
 */
scan_status_t embedding_grad(seq_dtype_t dtype, seq_dtype_t grad_dtype, const void* tokens, int token_bytes, size_t n,
                             const void* dout, int64_t dout_stride, size_t n_rows, uint32_t channels, float scale,
                             int accumulate, void* dtable, void* workspace, size_t workspace_bytes, void* stream);
size_t embedding_grad_workspace(size_t n, size_t n_rows, uint32_t channels);

/*
 * Depthwise causal convolution of `width` taps (2 .. 4) along every sequence:
 *   u[t] = bias + sum_k weight[.][k] * x[t - width + 1 + k],   y = act(u),
 * inputs before a sequence's first row coming from initial_state[s] (width-1
 * rows, oldest first; NULL: zeros).  final_state[s] (may be NULL) receives
 * the last width - 1 inputs of the sequence, those of initial_state included
 * where it has fewer rows.  weight (channels x width) and bias (channels, may
 * be NULL) are of weight_dtype, which is dtype or SEQ_F32; x, y and the
 * states of dtype, the states contiguous (seqs x (width - 1) x channels).
 */
typedef struct {
    int32_t dtype, weight_dtype, activation, width;
    uint64_t rows, seqs;
    const int32_t* seq_offsets;
    uint32_t channels, reserved;
    const void* x;
    int64_t x_stride;
    const void* weight;
    const void* bias;
    const void* initial_state;
    void* y;
    int64_t y_stride;
    void* final_state;
} causal_conv1d_args_t;
scan_status_t causal_conv1d(const causal_conv1d_args_t* args, void* stream);

/*
 * Gradients of causal_conv1d for dy (and dfinal_state, may be NULL: zeros).
 * dx (may not be NULL), dweight and dbias (float32; dbias NULL if there is no
 * bias), dinitial_state (dtype, NULL if not wanted).  `args` are the forward
 * call's; its y and final_state are not used.
 */
typedef struct {
    causal_conv1d_args_t args;
    const void* dy;
    int64_t dy_stride;
    const void* dfinal_state;
    void* dx;
    int64_t dx_stride;
    float* dweight;
    float* dbias;
    void* dinitial_state;
    void* workspace;
    uint64_t workspace_bytes;
} causal_conv1d_grad_args_t;
scan_status_t causal_conv1d_grad(const causal_conv1d_grad_args_t* args, void* stream);
size_t causal_conv1d_grad_workspace(const causal_conv1d_args_t* args);

/*
 * One token per row: y[i] from state[slots[i]] (width - 1 rows, oldest first)
 * and x[i]; the state is shifted by one row in place.  slots (int32 device
 * memory, NULL: slot i for row i) must not repeat a slot within a call (the
 * repeated slot's state and rows are then unspecified); rows whose slot lies
 * outside 0 .. n_slots - 1 are skipped: neither their output nor any state is
 * written.  state: n_slots x (width - 1) x channels, contiguous, of dtype.
 * rows <= 65535.
 */
typedef struct {
    int32_t dtype, weight_dtype, activation, width;
    uint64_t rows, n_slots;
    const int32_t* slots;
    uint32_t channels, reserved;
    const void* x;
    int64_t x_stride;
    const void* weight;
    const void* bias;
    void* state;
    void* y;
    int64_t y_stride;
} causal_conv1d_step_args_t;
scan_status_t causal_conv1d_step(const causal_conv1d_step_args_t* args, void* stream);

/*
 * Selective state-space scan.  For every channel d and state n of a sequence,
 * with group g = d / (channels / groups):
 *   dt[t] = delta[t][d] + delta_bias[d], through softplus if delta_softplus
 *   h[t]  = exp(dt[t] * A[d][n]) * h[t-1] + dt[t] * x[t][d] * B[t][g][n]
 *   y[t]  = (sum_n C[t][g][n] * h[t] + D[d] * x[t][d]) * silu(z[t][d])
 * h before the first row is initial_state[s] (NULL: zeros); final_state[s]
 * (may be NULL) receives h after the last row (initial_state where the
 * sequence is empty).  D, z and delta_bias may be NULL: no term, no factor,
 * no bias.  x, delta, z, B, C, y: dtype; B and C rows hold groups x states
 * values (contiguous).  A (channels x states), D, delta_bias and the states
 * (seqs x channels x states): float32, contiguous.  1 <= states <= 64; groups
 * divides channels.  saved (may be NULL) receives selective_scan_saved()
 * float32 values, the states that selective_scan_grad starts from.  y may be
 * NULL if only the states are wanted.
 */
typedef struct {
    int32_t dtype, delta_softplus;
    uint64_t rows, seqs;
    const int32_t* seq_offsets;
    uint32_t channels, states, groups, reserved;
    const void* x;
    int64_t x_stride;
    const void* delta;
    int64_t delta_stride;
    const float* A;
    const void* B;
    int64_t b_stride;
    const void* C;
    int64_t c_stride;
    const float* D;
    const void* z;
    int64_t z_stride;
    const float* delta_bias;
    const float* initial_state;
    void* y;
    int64_t y_stride;
    float* final_state;
    float* saved;
    void* workspace;
    uint64_t workspace_bytes;
} selective_scan_args_t;
scan_status_t selective_scan(const selective_scan_args_t* args, void* stream);
size_t selective_scan_workspace(const selective_scan_args_t* args);
size_t selective_scan_saved(const selective_scan_args_t* args);

/*
 * Gradients of selective_scan for dy (and dfinal_state, may be NULL: zeros).
 * `args` are the forward call's, with `saved` as it left it; y and
 * final_state are not used, workspace is this call's.  dx, ddelta, dz (NULL
 * exactly if z is), dB and dC of dtype; dA, dD (NULL exactly if D is),
 * ddelta_bias (NULL exactly if delta_bias is) and dinitial_state (may be
 * NULL) float32.  Gradients of shared values (A, D, delta_bias over rows, B
 * and C over a group's channels) are summed over all of their uses.
 */
typedef struct {
    selective_scan_args_t args;
    const void* dy;
    int64_t dy_stride;
    const float* dfinal_state;
    void* dx;
    int64_t dx_stride;
    void* ddelta;
    int64_t ddelta_stride;
    void* dz;
    int64_t dz_stride;
    void* dB;
    int64_t db_stride;
    void* dC;
    int64_t dc_stride;
    float* dA;
    float* dD;
    float* ddelta_bias;
    float* dinitial_state;
} selective_scan_grad_args_t;
scan_status_t selective_scan_grad(const selective_scan_grad_args_t* args, void* stream);
size_t selective_scan_grad_workspace(const selective_scan_grad_args_t* args);

/*
 * One token per row: one step of the recurrence from state[slots[i]]
 * (n_slots x channels x states float32, contiguous, updated in place).
 * slots as in causal_conv1d_step.
 */
typedef struct {
    int32_t dtype, delta_softplus;
    uint64_t rows, n_slots;
    const int32_t* slots;
    uint32_t channels, states, groups, reserved;
    const void* x;
    int64_t x_stride;
    const void* delta;
    int64_t delta_stride;
    const float* A;
    const void* B;
    int64_t b_stride;
    const void* C;
    int64_t c_stride;
    const float* D;
    const void* z;
    int64_t z_stride;
    const float* delta_bias;
    float* state;
    void* y;
    int64_t y_stride;
} selective_scan_step_args_t;
scan_status_t selective_scan_step(const selective_scan_step_args_t* args, void* stream);

/*
 * Gated linear recurrence.  For every channel d of a sequence:
 *   a[t] = exp(rate[d] * sigmoid(decay_gate[t][d]))
 *   h[t] = a[t] * h[t-1] + sqrt(1 - a[t]^2) * sigmoid(input_gate[t][d]) * x[t][d],   y[t] = h[t]
 * h before the first row is initial_state[s] (NULL: zeros); final_state[s] (may be NULL) receives h after the
 * last row (initial_state where the sequence is empty).  x, decay_gate, input_gate, y: dtype; rate (channels),
 * not above 0 (a above 1 gives NaN), and the states (seqs x channels): float32, contiguous.  saved (may be NULL)
 * receives gated_scan_saved() float32 values, the states that gated_scan_grad starts from.  y may be NULL if only
 * the states are wanted.
 */
typedef struct {
    int32_t dtype, reserved;
    uint64_t rows, seqs;
    const int32_t* seq_offsets;
    uint32_t channels, reserved2;
    const void* x;
    int64_t x_stride;
    const void* decay_gate;
    int64_t decay_stride;
    const void* input_gate;
    int64_t input_stride;
    const float* rate;
    const float* initial_state;
    void* y;
    int64_t y_stride;
    float* final_state;
    float* saved;
    void* workspace;
    uint64_t workspace_bytes;
} gated_scan_args_t;
scan_status_t gated_scan(const gated_scan_args_t* args, void* stream);
size_t gated_scan_workspace(const gated_scan_args_t* args);
size_t gated_scan_saved(const gated_scan_args_t* args);

/*
 * Gradients of gated_scan for dy (and dfinal_state, may be NULL: zeros).  `args` are the forward call's, with
 * `saved` as it left it; y and final_state are not used, workspace is this call's.  dx, ddecay_gate and
 * dinput_gate of dtype; drate (summed over all rows) and dinitial_state (may be NULL) float32.  Where
 * 1 - a^2 is 0 in 32 bits (no decay; a sigmoid below 2^-126 counts as 0), the derivative of its root is taken as 0.
 */
typedef struct {
    gated_scan_args_t args;
    const void* dy;
    int64_t dy_stride;
    const float* dfinal_state;
    void* dx;
    int64_t dx_stride;
    void* ddecay_gate;
    int64_t ddecay_stride;
    void* dinput_gate;
    int64_t dinput_stride;
    float* drate;
    float* dinitial_state;
} gated_scan_grad_args_t;
scan_status_t gated_scan_grad(const gated_scan_grad_args_t* args, void* stream);
size_t gated_scan_grad_workspace(const gated_scan_args_t* args);

/*
 * One token per row: one step of the recurrence from state[slots[i]] (n_slots x channels float32, contiguous,
 * updated in place).  slots as in causal_conv1d_step; rows < 2^31.
 */
typedef struct {
    int32_t dtype, reserved;
    uint64_t rows, n_slots;
    const int32_t* slots;
    uint32_t channels, reserved2;
    const void* x;
    int64_t x_stride;
    const void* decay_gate;
    int64_t decay_stride;
    const void* input_gate;
    int64_t input_stride;
    const float* rate;
    float* state;
    void* y;
    int64_t y_stride;
} gated_scan_step_args_t;
scan_status_t gated_scan_step(const gated_scan_step_args_t* args, void* stream);

/*
 * Tokens sorted by expert and back.  A token's choices are `choices` expert numbers; those outside
 * 0 .. n_experts - 1 go to no expert.
 *
 * expert_split: the stable split of n choices (token by token) by expert.  offsets (n_experts + 1): expert e has
 * rows [offsets[e], offsets[e+1]) of the experts' order, its choices in ascending order; places (n): the row of every
 * choice, -1 where it has no expert; source (n): the choice of every row, -1 from row offsets[n_experts] on.
 * n < 2^31, n_experts <= 1024.  Up to 4096 choices need no workspace (0 bytes; it may be NULL).
 */
scan_status_t expert_split(const int32_t* experts, size_t n, uint32_t n_experts, int32_t* offsets, int32_t* places,
                           int32_t* source, void* workspace, size_t workspace_bytes, void* stream);
size_t expert_split_workspace(size_t n, uint32_t n_experts);

/*
 * expert_dispatch: out[places[t][j]] = x[t] for every token t and choice j; places outside 0 .. rows - 1 are
 * skipped (here and below), a row that two choices lead to holds parts of either's.  Rows that no choice leads to are
 * left as they were, but set to zero from *used on (device memory, may be NULL: none) or, with clear != 0, everywhere (used is
 * not looked at then).  source (source_rows values, may be NULL) is the split's and saves writing: rows r with
 * places[source[r]] == r need not be cleared; it may hold anything.
 * x: tokens x channels, out: rows x channels; choices <= 256, tokens * choices < 2^31.  The gradient of x is
 * expert_combine without weights.
 */
typedef struct {
    int32_t dtype, clear;
    uint64_t tokens, rows;
    uint32_t choices, channels;
    const int32_t* places;
    const int32_t* used;
    const void* x;
    int64_t x_stride;
    void* out;
    int64_t out_stride;
    const int32_t* source;
    uint64_t source_rows;
} expert_dispatch_args_t;
scan_status_t expert_dispatch(const expert_dispatch_args_t* args, void* stream);

/*
 * expert_combine: out[t] = the sum over j of weights[t][j] * y[places[t][j]], in the order of j.  weights (tokens x
 * choices, contiguous, weight_dtype: dtype or SEQ_F32) may be NULL: ones.
 */
typedef struct {
    int32_t dtype, weight_dtype;
    uint64_t tokens, rows;
    uint32_t choices, channels;
    const int32_t* places;
    const void* weights;
    const void* y;
    int64_t y_stride;
    void* out;
    int64_t out_stride;
} expert_combine_args_t;
scan_status_t expert_combine(const expert_combine_args_t* args, void* stream);

/*
 * Gradients of expert_combine: dy[places[t][j]] = weights[t][j] * dout[t] (used, clear and source as in expert_dispatch), and
 * dweights[t][j] (tokens x choices float32; may be NULL, y may be NULL then) = the sum over the channels of dout[t] *
 * y[places[t][j]], 0 where there is no place.
 */
typedef struct {
    int32_t dtype, weight_dtype;
    uint64_t tokens, rows;
    uint32_t choices, channels;
    const int32_t* places;
    const int32_t* used;
    const void* weights;
    const void* dout;
    int64_t dout_stride;
    const void* y;
    int64_t y_stride;
    void* dy;
    int64_t dy_stride;
    float* dweights;
    const int32_t* source;
    uint64_t source_rows;
    int32_t clear, reserved;
} expert_combine_grad_args_t;
scan_status_t expert_combine_grad(const expert_combine_grad_args_t* args, void* stream);

/*
 * Sampling from given random numbers: tokens[r] for every row of logits (rows x n, n <= 2^19).  With settings
 * from the row's own temperature, top_k, top_p and min_p (device memory, rows values each) or, where that is NULL, the
 * call's:
 *   weights w[i] = exp((logits[r][i] - max) / temperature); minus infinity and NaN weigh nothing, and
 *   next to a plus infinity only those weigh
 *   tokens by falling logit, equal ones by ascending index, of which are kept
 *     the first top_k (<= 0: all); of these the first whose predecessors' weights add up to less than
 *     top_p times the weight of them all, and at least one; and those with w >= min_p (at most 1)
 *   tokens[r] = the first kept i, by ascending index, up to which the kept weights add up to more than
 *     uniform[r] times the kept weight (uniform outside [0, 1): the first or the last)
 * A temperature that is not above 0 takes the first largest logit.  A row without a finite or plus infinite
 * logit gives -1.  Weights (off by 2^-44 of themselves at most, 0 below 2^-1074) and their sums are held in 64 bits.
 * tokens: int32 (token_bytes 4) or int64 (8).
 */
typedef struct {
    int32_t dtype, token_bytes;
    uint64_t rows;
    uint32_t n, reserved;
    const void* logits;
    int64_t logits_stride;
    const float* uniform;
    const float* temperatures;
    const int32_t* top_ks;
    const float* top_ps;
    const float* min_ps;
    double temperature, top_p, min_p;
    int64_t top_k;
    void* tokens;
} sample_tokens_args_t;
scan_status_t sample_tokens(const sample_tokens_args_t* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DWPT_SEQ_H */
