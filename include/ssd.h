/*
 * ssd.h -- C ABI of the MI355X (gfx950) complex chunkwise SSD scan library.
 *
 * The operation is the complex-valued selective state-space scan of the
 * Mamba-3-Lite pages. For every batch row b and head h, independently:
 *
 *   Abar_t = exp(softplus(dt_t) * A_h)                       (discretisation)
 *   s_t    = Abar_t * s_{t-1} + B_t (outer) x_t              (state, N x D)
 *   y_t    = Re( sum_n C_t[n] * s_t[n, :] )                   (output, D)
 *
 * with no conjugation anywhere, s_{-1} the initial state (zero by default)
 * and final_state = s_{T-1}. Sources: "Extending -- SSM variants & Triton
 * kernels" (Path A Step 1: the naive scan and the discretisation; Step 3: the
 * chunkwise function returns the real part), "index.html" lab 03 (the
 * chunkwise decomposition: per-chunk log-decay running sums, the masked
 * decay matrix L, the intra-chunk term, per-chunk states and the passing of
 * states between chunks), and "Skills Reference" Skill 3 (chunk_size 32..256,
 * default 64).
 *
 * Gradients (ssd_chunk_backward) follow from the same recurrence by reverse-mode
 * differentiation.
 *
 * Conventions common to every call:
 *   * All tensor pointers are DEVICE pointers owned by the caller. The library
 *     allocates no memory and keeps no state between calls.
 *   * Layouts are dense row-major. Complex numbers are interleaved (re, im)
 *     pairs of float32, bit-identical to torch.complex64.
 *   * Argument checks run before anything is launched; a failed check returns
 *     a negative status and touches no memory. Work is launched on `stream`
 *     and is asynchronous; a launch failure returns SSD_ERR_HIP.
 *   * There is one code path: no fallback exists when a check fails.
 *   * Calls on different streams with different workspaces are independent.
 */
#ifndef SSD_H
#define SSD_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* A HIP stream, or NULL for the null stream. The same type as hipStream_t
 * (a pointer to struct ihipStream_t), declared here so that this header needs
 * no HIP header. */
typedef struct ihipStream_t *ssd_stream_t;

/* One complex64 value, laid out as torch.complex64. */
typedef struct {
    float re, im;
} ssd_c64;

enum {
    SSD_OK = 0,
    SSD_ERR_NULL = -1,        /* a required pointer is NULL */
    SSD_ERR_SHAPE = -2,       /* a size is negative, or N, D, chunk_size < 1 */
    SSD_ERR_ODD_N = -3,       /* N is odd: the state must pack into real pairs */
    SSD_ERR_BLOCK_DIMS = -4,  /* N, D or chunk_size above 256 */
    SSD_ERR_WORKSPACE = -5,   /* workspace missing or smaller than required */
    SSD_ERR_ALIGN = -6,       /* a pointer is not aligned as documented */
    SSD_ERR_HIP = -7,         /* the HIP runtime reported an error */
    SSD_ERR_UNSUPPORTED = -8, /* a valid size this build does not cover yet */
    SSD_ERR_ALIAS = -9        /* an output overlaps an input it must not */
};

/* Largest N, D and chunk_size accepted (the pages cap kernel blocks at 256). */
#define SSD_MAX_BLOCK 256

/*
 * ssd_discretise -- the discretisation step and the per-chunk cumulative
 * log-decay ("Extending", Path A Step 1 and Path B Step 2; index.html lab 03).
 *
 *   dt        (batch, T, H) float32, step logits.
 *   A         (H) complex64, one eigenvalue per head.
 *   A_bar     out, nullable: (batch, T, H) complex64, exp(softplus(dt) * A).
 *   log_decay_cumsum
 *             out, nullable: (batch, H, nc, chunk_size) complex64 with
 *             nc = ceil(T / chunk_size). Entry [b,h,c,l] is the sum of
 *             softplus(dt_t) * A_h over t = c*chunk_size .. c*chunk_size + l.
 *             Positions of a last partial chunk past T repeat the final sum.
 *   chunk_size 0 when log_decay_cumsum is NULL, else 1..256.
 * Alignment: 4 bytes for dt, 8 bytes for the complex arrays.
 * batch, T or H equal to 0 is a no-op.
 */
int ssd_discretise(const float *dt, const ssd_c64 *A, int64_t batch, int64_t T, int64_t H,
                   int64_t chunk_size, ssd_c64 *A_bar, ssd_c64 *log_decay_cumsum,
                   ssd_stream_t stream);

/*
 * ssd_chunk_forward_workspace_bytes -- device workspace that ssd_chunk_forward
 * needs for these sizes (0 when none is needed). The value depends only on
 * the arguments. Negative or invalid sizes return 0.
 */
size_t ssd_chunk_forward_workspace_bytes(int64_t batch, int64_t T, int64_t H, int64_t N,
                                         int64_t D, int64_t chunk_size);

/*
 * ssd_chunk_forward -- the chunkwise complex SSD scan forward
 * ("Extending", Path A Step 3: the chunkwise function; index.html lab 03).
 *
 *   x            (batch, T, H, D) complex64, token content.
 *   A            (H) complex64.
 *   B_t, C_t     (batch, T, H, N) complex64, input and output maps.
 *   dt           (batch, T, H) float32.
 *   chunk_size   1..256; a last chunk shorter than chunk_size is allowed
 *                (T need not be a multiple of it). It sets the span of the
 *                intra-chunk quadratic term, up to 64 tokens: a longer chunk is
 *                evaluated as 64-token sub-chunks with the state passed between
 *                them. The result does not depend on chunk_size beyond rounding.
 *   initial_state nullable: (batch, H, N, D) complex64 state s_{-1}; NULL
 *                means zero.
 *   y            out: (batch, T, H, D) float32, the real part of the output.
 *   final_state  out, nullable: (batch, H, N, D) complex64, s_{T-1}.
 *   workspace    device scratch of at least
 *                ssd_chunk_forward_workspace_bytes(...) bytes, 256-byte
 *                aligned; may be NULL when that size is 0. Its contents on
 *                entry are ignored. It is needed when there are fewer
 *                (batch, head) sequences than the GPU has compute units (the
 *                sequences are then cut into segments) and when N > 64 (the
 *                state is then split into 64-row slices whose partial outputs
 *                are added up).
 * Constraints: N even (SSD_ERR_ODD_N); N, D, chunk_size <= 256
 * (SSD_ERR_BLOCK_DIMS).
 * Alignment: x, A, B_t, C_t, initial_state, final_state 8 bytes (B_t and C_t
 * rows are read 16 bytes at a time, at any 8-byte alignment); dt and y 4 bytes.
 * batch or H equal to 0 is a no-op; T equal to 0 copies initial_state (or
 * zeros) into final_state.
 */
int ssd_chunk_forward(const ssd_c64 *x, const ssd_c64 *A, const ssd_c64 *B_t, const ssd_c64 *C_t,
                      const float *dt, int64_t batch, int64_t T, int64_t H, int64_t N, int64_t D,
                      int64_t chunk_size, const ssd_c64 *initial_state, float *y,
                      ssd_c64 *final_state, void *workspace, size_t workspace_bytes,
                      ssd_stream_t stream);

/* Size of the static device scratch of ssd_chunk_forward_noalloc (32 MiB per GPU). */
#define SSD_NOALLOC_SCRATCH_BYTES (32 * 1024 * 1024)

/*
 * ssd_chunk_forward_noalloc -- ssd_chunk_forward for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc): the same scan, with the same arguments minus
 * the workspace. The workspace lives in a static device array of
 * SSD_NOALLOC_SCRATCH_BYTES bytes, one per GPU, created when the library's code
 * object is loaded on that GPU and held until the process ends; this call and
 * the kernels it launches allocate nothing.
 *   Arguments, constraints, alignment and results: as ssd_chunk_forward.
 *   SSD_ERR_WORKSPACE when ssd_chunk_forward_workspace_bytes(...) for these
 *   sizes exceeds SSD_NOALLOC_SCRATCH_BYTES (checked before anything runs).
 * The scratch used is that of the current device; `stream` must belong to it.
 * Every call on one GPU shares that GPU's scratch: calls that may overlap in
 * time on one GPU (different streams, or host threads) race and must be
 * serialised by the caller. Its contents on entry are ignored.
 */
int ssd_chunk_forward_noalloc(const ssd_c64 *x, const ssd_c64 *A, const ssd_c64 *B_t,
                              const ssd_c64 *C_t, const float *dt, int64_t batch, int64_t T,
                              int64_t H, int64_t N, int64_t D, int64_t chunk_size,
                              const ssd_c64 *initial_state, float *y, ssd_c64 *final_state,
                              ssd_stream_t stream);

/*
 * ssd_chunk_forward_proj -- the same scan read straight from the in_proj output
 * ("Extending", Path A Step 2: Mamba3Block._forward_impl slices the projection
 * of each token into x (H*D), four H*N blocks and a trailing dt (H); the
 * in_proj width is H*(D + 4N + 1)). x is real here, and B_t, C_t are given by
 * their real and imaginary blocks.
 *
 *   proj         (batch, T, token_stride) float32; the row of token (b, t) is
 *                  [ x (H, D) | Re B_t (H, N) | Im B_t (H, N) |
 *                    Re C_t (H, N) | Im C_t (H, N) | dt (H) | unused ]
 *                (the order of the four N-blocks is this library's reading).
 *   token_stride floats between consecutive token rows, >= H*(D + 4N + 1),
 *                even. Floats past the last block are never read.
 *   A, chunk_size, initial_state, y, final_state, workspace: as for
 *                ssd_chunk_forward; the workspace size is
 *                ssd_chunk_forward_workspace_bytes(batch, T, H, N, D, chunk_size).
 * Result: identical in exact arithmetic to ssd_chunk_forward with
 * x = x_real + 0i, B_t = Re B + i Im B, C_t = Re C + i Im C.
 * Constraints: as ssd_chunk_forward; token_stride <= 2^22 (SSD_ERR_UNSUPPORTED).
 * Alignment: proj 8 bytes and H*D even (the N-blocks are read as float pairs),
 * else SSD_ERR_ALIGN.
 */
int ssd_chunk_forward_proj(const float *proj, int64_t token_stride, const ssd_c64 *A,
                           int64_t batch, int64_t T, int64_t H, int64_t N, int64_t D,
                           int64_t chunk_size, const ssd_c64 *initial_state, float *y,
                           ssd_c64 *final_state, void *workspace, size_t workspace_bytes,
                           ssd_stream_t stream);

/*
 * ssd_chunk_forward_proj_bf16 -- ssd_chunk_forward_proj with the in_proj rows
 * in bfloat16 ("AGENTS & System Architecture": the model trains in BF16
 * (section 1, subagent notes) while the recurrent state stays complex64
 * (section 3, numerical-stability rules)). proj holds bfloat16 bit patterns
 * (uint16); each element is
 * widened to float32 as it is loaded and every product, sum and the state
 * stay float32, so the result equals ssd_chunk_forward_proj on the widened
 * rows. Same arguments, constraints and workspace as ssd_chunk_forward_proj,
 * except the alignment: proj 4 bytes (and token_stride, H*D even).
 */
int ssd_chunk_forward_proj_bf16(const uint16_t *proj, int64_t token_stride, const ssd_c64 *A,
                                int64_t batch, int64_t T, int64_t H, int64_t N, int64_t D,
                                int64_t chunk_size, const ssd_c64 *initial_state, float *y,
                                ssd_c64 *final_state, void *workspace, size_t workspace_bytes,
                                ssd_stream_t stream);

/*
 * ssd_chunk_backward_workspace_bytes -- device workspace that
 * ssd_chunk_backward needs for these sizes (0 when T, batch or H is 0, or the
 * sizes are invalid). It holds the state entering and the adjoint leaving
 * every chunk, in 64 x 64 blocks: about 2 * batch * H * ceil(T / min(chunk_size,
 * 32)) * ceil(N/64) * ceil(D/64) * 32 KiB; with N or D above 64 also the
 * per-slice partial gradients (8 * batch * T * H * (ceil(N/64) D +
 * 2 ceil(D/64) N) + 4 * batch * T * H * ceil(N/64) ceil(D/64) bytes).
 */
size_t ssd_chunk_backward_workspace_bytes(int64_t batch, int64_t T, int64_t H, int64_t N,
                                          int64_t D, int64_t chunk_size);

/*
 * ssd_chunk_backward -- gradients of the chunkwise scan ("Extending", Path B
 * Step 3: the backward of a scan's autograd Function is seeded with the true
 * upstream gradients of y and final_state and returns a gradient for every
 * differentiated input).
 *
 * For the loss l = sum(grad_y * y) + sum(Re(conj(grad_final_state) * final_state))
 * of the forward call with the same inputs, each output receives dl/dRe(z) +
 * i dl/dIm(z) for a complex input z (the convention of torch's autograd for
 * complex tensors) and dl/dz for a real one:
 *   x, A, B_t, C_t, dt, initial_state, chunk_size
 *                  as for ssd_chunk_forward (initial_state nullable = zero).
 *   grad_y         (batch, T, H, D) float32, upstream gradient of y.
 *   grad_final_state nullable: (batch, H, N, D) complex64; NULL means zero.
 *   grad_x         out: (batch, T, H, D) complex64.
 *   grad_A         out: (H) complex64, summed over batch rows and time.
 *   grad_B_t, grad_C_t out: (batch, T, H, N) complex64.
 *   grad_dt        out: (batch, T, H) float32.
 *   grad_initial_state out, nullable: (batch, H, N, D) complex64.
 *   workspace      device scratch of at least
 *                  ssd_chunk_backward_workspace_bytes(...) bytes, 256-byte
 *                  aligned (required whenever T > 0). Contents on entry ignored.
 * The chunk evaluated at once is min(chunk_size, 32) tokens; the result does
 * not depend on chunk_size beyond rounding. With N or D above 64 the state is
 * evaluated in 64 x 64 blocks whose partial gradients are added in a fixed
 * order (deterministic).
 * Constraints: as ssd_chunk_forward (N even; N, D, chunk_size <= 256), and
 * batch * H * ceil(N/64) * ceil(D/64) * ceil(T / min(chunk_size, 32)) below 2^31
 * (the chunks are indexed with 32-bit integers; SSD_ERR_UNSUPPORTED otherwise, and
 * the workspace size is then 0).
 * Alignment: complex arrays 8 bytes; dt, grad_y, grad_dt 4 bytes.
 * batch or H equal to 0 is a no-op; T equal to 0 writes grad_final_state (or
 * zeros) to grad_initial_state and zeros to grad_A.
 */
int ssd_chunk_backward(const ssd_c64 *x, const ssd_c64 *A, const ssd_c64 *B_t, const ssd_c64 *C_t,
                       const float *dt, int64_t batch, int64_t T, int64_t H, int64_t N, int64_t D,
                       int64_t chunk_size, const ssd_c64 *initial_state, const float *grad_y,
                       const ssd_c64 *grad_final_state, ssd_c64 *grad_x, ssd_c64 *grad_A,
                       ssd_c64 *grad_B_t, ssd_c64 *grad_C_t, float *grad_dt,
                       ssd_c64 *grad_initial_state, void *workspace, size_t workspace_bytes,
                       ssd_stream_t stream);

/*
 * ssd_chunk_backward_proj -- ssd_chunk_backward for the scan read from in_proj
 * rows (ssd_chunk_forward_proj, float32 rows): the gradients are written as
 * gradient rows of the same layout.
 *   proj, token_stride, A, chunk_size, initial_state, grad_y, grad_final_state,
 *                as for ssd_chunk_forward_proj and ssd_chunk_backward.
 *   grad_proj    out: (batch, T, token_stride) float32; in each token row the x
 *                block receives dl/dx (x is real), the Re/Im B and C blocks the
 *                real and imaginary parts of the B_t and C_t gradients, the dt
 *                block dl/ddt. Floats past the blocks are not written.
 *   grad_A, grad_initial_state, workspace: as for ssd_chunk_backward (same
 *                workspace size).
 * Constraints: as ssd_chunk_backward.
 * Alignment: proj, grad_proj, grad_y 4 bytes; A and the states 8 bytes.
 */
int ssd_chunk_backward_proj(const float *proj, int64_t token_stride, const ssd_c64 *A,
                            int64_t batch, int64_t T, int64_t H, int64_t N, int64_t D,
                            int64_t chunk_size, const ssd_c64 *initial_state, const float *grad_y,
                            const ssd_c64 *grad_final_state, float *grad_proj, ssd_c64 *grad_A,
                            ssd_c64 *grad_initial_state, void *workspace, size_t workspace_bytes,
                            ssd_stream_t stream);

/*
 * ssd_chunk_backward_proj_bf16 -- ssd_chunk_backward_proj for bfloat16 rows (the
 * training precision of AGENTS & System Architecture: BF16 activations, the
 * recurrent state complex64): proj and grad_proj hold bfloat16 values as their
 * 16-bit patterns. Rows are widened to float32 as they are loaded; every
 * product, sum and stored state stays float32 (as in ssd_chunk_forward_proj_bf16),
 * and each gradient is rounded to bfloat16 (nearest, ties to even) as it is
 * stored. grad_y, grad_final_state, grad_A and grad_initial_state stay float32
 * / complex64.
 * Arguments, constraints and workspace: as ssd_chunk_backward_proj.
 * Alignment: proj, grad_proj 2 bytes; grad_y 4 bytes; A and the states 8 bytes.
 */
int ssd_chunk_backward_proj_bf16(const uint16_t *proj, int64_t token_stride, const ssd_c64 *A,
                                 int64_t batch, int64_t T, int64_t H, int64_t N, int64_t D,
                                 int64_t chunk_size, const ssd_c64 *initial_state,
                                 const float *grad_y, const ssd_c64 *grad_final_state,
                                 uint16_t *grad_proj, ssd_c64 *grad_A,
                                 ssd_c64 *grad_initial_state, void *workspace,
                                 size_t workspace_bytes, ssd_stream_t stream);

/*
 * ssd_head_mix -- the MIMO head mixer that follows the scan (index.html lab 02
 * "MIMO MIXER": fully connected across the SSM heads, 1024 -> 1024 as 16 heads
 * of 64 channels, identity at initialisation; "Knows cold" item 2 of the AGENTS
 * page; the in_proj -> scan -> MIMO -> out_proj order of "Extending", Path A;
 * the model's parameter count in the "Extending" guide's documentation rule,
 * which holds only with a dense 1024 x 1024 matrix per layer). Each token's
 * heads are flattened head-major, k = h * D + d (F = H * D), and mapped by one
 * dense real F x F matrix:
 *
 *   z[m, o] = sum_k W[o, k] * y[m, k]          (z = y W^T, no bias)
 *
 *   y        (tokens, H, D) float32: the scan output, tokens = batch * T.
 *   W        (F, F) float32, row-major: row o holds the weights of output o
 *            (the layout of a linear layer's weight); the block
 *            W[i*D:(i+1)*D, j*D:(j+1)*D] links head j to head i.
 *   z        out: (tokens, H, D) float32; must not overlap y or W
 *            (SSD_ERR_ALIAS).
 *   tokens   >= 0; with 0 nothing is launched and y, W, z may be NULL.
 *            H, D >= 1; D <= 256; H * D <= 16384.
 * Arithmetic: float32 products summed in float32 (fp32 MFMA).
 * Alignment: 4 bytes (16-byte aligned y and W with H * D % 4 == 0 take the
 * vector loads).
 * Status: SSD_ERR_SHAPE for sizes out of range, SSD_ERR_BLOCK_DIMS for D > 256,
 * SSD_ERR_UNSUPPORTED for H * D > 16384.
 */
int ssd_head_mix(const float *y, const float *W, int64_t tokens, int64_t H, int64_t D, float *z,
                 ssd_stream_t stream);

/* Workspace bytes that ssd_head_mix_backward needs (0 for invalid sizes, for
 * tokens == 0, and when the weight gradient is formed in one pass). It holds
 * partial weight gradients over token ranges: at most 256 * (H*D)^2 * 4 bytes,
 * 64 MiB at H * D = 1024 with 65,536 tokens. */
size_t ssd_head_mix_backward_workspace_bytes(int64_t tokens, int64_t H, int64_t D);

/*
 * ssd_head_mix_backward -- gradients of l = sum grad_z * z for ssd_head_mix,
 * by the chain rule on its definition:
 *
 *   grad_y[m, k] = sum_o grad_z[m, o] * W[o, k]      (grad_y = grad_z W)
 *   grad_W[o, k] = sum_m grad_z[m, o] * y[m, k]      (grad_W = grad_z^T y)
 *
 *   y, W, tokens, H, D  as for ssd_head_mix (y is the forward's input).
 *   grad_z    (tokens, H, D) float32.
 *   grad_y    out: (tokens, H, D) float32.
 *   grad_W    out: (F, F) float32, overwritten. The sum over tokens runs in a
 *             fixed order: repeated calls give identical bits. With tokens == 0
 *             it is set to zero and every other pointer may be NULL.
 *   workspace device memory of ssd_head_mix_backward_workspace_bytes bytes,
 *             256-byte aligned (NULL allowed when that is 0).
 * No output may overlap an input, each other or the workspace (SSD_ERR_ALIAS).
 * Alignment and status codes as ssd_head_mix; SSD_ERR_WORKSPACE when the
 * workspace is missing or too small.
 */
int ssd_head_mix_backward(const float *y, const float *W, const float *grad_z, int64_t tokens,
                          int64_t H, int64_t D, float *grad_y, float *grad_W, void *workspace,
                          size_t workspace_bytes, ssd_stream_t stream);

/* Element types of the operators below (any other value: SSD_ERR_SHAPE). */
enum {
    SSD_F32 = 0,
    SSD_BF16 = 1 /* bfloat16 values as their 16-bit patterns */
};

/* Tokens between two stored states of the gated scan. */
#define SSD_GATED_CHUNK 64

/*
 * ssd_gated_scan -- the gated linear recurrence: a real, per-channel recurrence
 * whose decay and input are gated by the tokens. For every batch row b and
 * channel c, with i = sigmoid(input_gate) and r = sigmoid(decay_gate),
 *
 *   l_t = -decay_scale * softplus(lam_c) * r_t       a_t = exp(l_t)
 *   h_t = a_t * h_{t-1} + sqrt(1 - a_t^2) * i_t * x_t
 *
 *   x, input_gate, decay_gate
 *                (batch, T, C) of `dtype`; a channel's neighbours lie side by
 *                side, consecutive tokens *_stride elements apart (>= C) and
 *                consecutive batch rows T * *_stride apart, so the three may be
 *                column ranges of one matrix of projected rows. Read only.
 *   lam          (C) float32. decay_scale: >= 0, at most 1e30.
 *   initial_state nullable: (batch, C) float32, h_{-1}; NULL means zero.
 *   lengths      nullable: (batch) int32 in device memory: the tokens of each
 *                row, clamped to 0 .. T. Tokens from there on are padding: what they
 *                hold does not matter, their h is 0, and the state stays as it is.
 *                (They are memory that may be read: a first token is, and then left out.)
 *   h            out: (batch, T, C) of `dtype`, dense.
 *   final_state  out, nullable: (batch, C) float32, the state after the row's last
 *                token. It may be initial_state itself (updated in place).
 *   chunk_states out, nullable: (batch, ceil(T / SSD_GATED_CHUNK), C) float32, the
 *                state before each chunk's first token, for the backward.
 *   workspace    ssd_gated_scan_workspace_bytes(...) bytes, 256-byte aligned (NULL
 *                allowed when that is 0); needed when batch and C alone give too
 *                few workgroups, the tokens are then cut into segments.
 * Gates, products and the state are float32; h is rounded once to `dtype`.
 * Where 1 - a^2 lies below 2^-126, the smallest normal float, its root and so the
 * input's share and the gradients through it may come out as 0 (they are below 2^-63 of
 * the input). An infinity or a NaN in a sequence makes what follows it in its channel
 * infinite or NaN.
 * T = 1 is the form for generation: one step on the state.
 * No output may overlap an input or another output (SSD_ERR_ALIAS), but for the
 * state in place. Alignment: the element size. batch equal to 0 is a no-op; T
 * equal to 0 copies the initial state (or zeros) into final_state.
 * SSD_ERR_UNSUPPORTED: T above 2^30, batch or C above 2^24, or more workgroups than one
 * launch takes, which begins at batch * ceil(C / 64) = 2^22 (for T up to 32 at 2^26). The
 * same for the backward, at 2^22 whatever T.
 */
size_t ssd_gated_scan_workspace_bytes(int64_t batch, int64_t T, int64_t C, int dtype);

int ssd_gated_scan(const void *x, int64_t x_stride, const void *input_gate,
                   int64_t input_gate_stride, const void *decay_gate, int64_t decay_gate_stride,
                   const float *lam, float decay_scale, int dtype, int64_t batch, int64_t T,
                   int64_t C, const float *initial_state, const int32_t *lengths, void *h,
                   float *final_state, float *chunk_states, void *workspace,
                   size_t workspace_bytes, ssd_stream_t stream);

/*
 * ssd_gated_scan_backward -- gradients of l = sum grad_h * h + sum
 * grad_final_state * final_state for ssd_gated_scan.
 *   x .. C, lengths as for the forward; chunk_states as it wrote them.
 *   grad_h       (batch, T, C) of `dtype`, dense; what the padding holds does not matter.
 *   grad_final_state nullable: (batch, C) float32.
 *   grad_x, grad_input_gate, grad_decay_gate
 *                out: (batch, T, C) of `dtype`, dense; 0 in the padding.
 *   grad_lam     out: (C) float32, summed over batch rows and tokens in a fixed
 *                order.
 *   grad_initial_state out, nullable: (batch, C) float32.
 *   workspace    ssd_gated_scan_backward_workspace_bytes(...) bytes.
 * The states between the stored ones are computed again in float32. No output
 * may overlap an input, another output or the workspace (SSD_ERR_ALIAS). batch or
 * T equal to 0 sets grad_lam to zero and copies grad_final_state (or zeros).
 */
size_t ssd_gated_scan_backward_workspace_bytes(int64_t batch, int64_t T, int64_t C, int dtype);

int ssd_gated_scan_backward(const void *x, int64_t x_stride, const void *input_gate,
                            int64_t input_gate_stride, const void *decay_gate,
                            int64_t decay_gate_stride, const float *lam, float decay_scale,
                            int dtype, int64_t batch, int64_t T, int64_t C,
                            const float *chunk_states, const int32_t *lengths, const void *grad_h,
                            const float *grad_final_state, void *grad_x, void *grad_input_gate,
                            void *grad_decay_gate, float *grad_lam, float *grad_initial_state,
                            void *workspace, size_t workspace_bytes, ssd_stream_t stream);

/*
 * ssd_rms_norm -- the root-mean-square norm with the residual's addition, its
 * result in `dtype`, in 8 bits, or both. Per row of F values:
 *
 *   s = x + residual        rstd = 1 / sqrt(sum s^2 / F + eps)
 *   y = s * rstd * weight   q = e4m3(y / scale), one scale per 128 neighbours
 *
 *   x            (rows, F) of `dtype`, rows x_stride elements apart (>= F).
 *   residual     nullable (s = x): as x, with its own stride.
 *   weight       (F) float32.
 *   y            out, nullable: (rows, F) of `dtype`, dense.
 *   residual_out out, nullable (only with residual): s, rounded to `dtype`, dense.
 *                It may be residual itself if that is dense.
 *   q, scale     out, nullable together: (rows, F) e4m3 bytes and
 *                (ceil(F / 128), rows) float32, as ssd_fp8_quantise makes them of y
 *                and as ssd_fp8_matmul reads them; q is taken of the float32 y.
 *                One of y and q has to be given.
 *   rstd         out, nullable: (rows) float32, for the backward.
 * Sums are float32 and taken of the unrounded s: a row's sum of squares has to stay below
 * 2^128, and without an epsilon a row whose mean square is below 2^-150 counts as zeros (its
 * rstd is infinite). F at most 16384 (SSD_ERR_UNSUPPORTED). eps >= 0. rows equal to 0 is a no-op. No other overlap of
 * outputs (SSD_ERR_ALIAS). Alignment: the element size.
 */
int ssd_rms_norm(const void *x, int64_t x_stride, const void *residual, int64_t residual_stride,
                 const float *weight, int dtype, int64_t rows, int64_t F, float eps, void *y,
                 void *residual_out, uint8_t *q, float *scale, float *rstd, ssd_stream_t stream);

/*
 * ssd_rms_norm_backward -- gradients of l = sum grad_y * y + sum grad_residual * s:
 *
 *   grad_x = grad_residual + rstd (w grad_y - s rstd^2 (sum w grad_y s) / F)
 *   grad_weight = sum over rows grad_y * s * rstd
 *
 *   s            (rows, F) of `dtype`: the forward's residual_out (its x, without a
 *                residual). rstd: as the forward wrote it.
 *   grad_y       (rows, F) of `dtype`; grad_residual nullable, the same: the gradient
 *                that reaches s through the residual stream.
 *   grad_x       out: (rows, F) of `dtype`, dense: the gradient of x and of residual.
 *   grad_weight  out: (F) float32, summed in a fixed order.
 *   workspace    ssd_rms_norm_backward_workspace_bytes(rows, F) bytes, 256-byte aligned.
 * rows equal to 0 sets grad_weight to zero. No output may overlap an input
 * (SSD_ERR_ALIAS).
 */
size_t ssd_rms_norm_backward_workspace_bytes(int64_t rows, int64_t F);

int ssd_rms_norm_backward(const void *s, int64_t s_stride, const float *weight, const float *rstd,
                          const void *grad_y, int64_t grad_y_stride, const void *grad_residual,
                          int64_t grad_residual_stride, int dtype, int64_t rows, int64_t F,
                          void *grad_x, float *grad_weight, void *workspace,
                          size_t workspace_bytes, ssd_stream_t stream);

/*
 * ssd_fp8_quantise -- 8-bit values (e4m3: 4 exponent and 3 mantissa bits, largest
 * 448) with a float32 scale per block of 128: scale = max(max |v| / 448, 2^-126)
 * over the block, q = v / scale rounded to nearest, ties to even. Let v be x
 * (rows, cols), or, with `transpose`, x turned (cols, rows); R and K its sizes.
 *
 *   x            (rows, cols) of `dtype`, rows x_stride elements apart.
 *   block_rows   1: blocks of 1 x 128 along v's rows; scale is (ceil(K / 128), R).
 *                128: blocks of 128 x 128; scale is (ceil(R / 128), ceil(K / 128)).
 *   q            out: (R, K) bytes, rows q_stride bytes apart (>= K); bytes between
 *                the rows are not written.
 * A block with an infinity or a NaN comes back as NaN (its scale is infinite or
 * NaN); other blocks are untouched by it. rows equal to 0 is a no-op.
 * SSD_ERR_UNSUPPORTED: rows or cols above 2^31, from 2^24 tiles of 128 x 128 on (plain with
 * block_rows 1: from 2^30 blocks on).
 * Alignment: the element size; 4 bytes for scale.
 */
int ssd_fp8_quantise(const void *x, int64_t x_stride, int dtype, int64_t rows, int64_t cols,
                     int64_t block_rows, int transpose, uint8_t *q, int64_t q_stride, float *scale,
                     ssd_stream_t stream);

/*
 * ssd_fp8_matmul -- the product of two such operands, in_proj's and out_proj's form:
 *
 *   out[m, n] = sum over blocks kb of 128 k of
 *                   a_scale[kb, m] * s_b * sum over k in kb of a[m, k] * b[n, k]
 *   with s_b = b_scale[n / 128, kb] (b_block_rows 128) or b_scale[kb, n] (1).
 *
 *   a            (M, K) e4m3 bytes, rows a_stride bytes apart (>= K); a_scale
 *                (ceil(K / 128), M): 1 x 128 blocks, as ssd_fp8_quantise and
 *                ssd_rms_norm make them.
 *   b            (N, K) e4m3 bytes, rows b_stride bytes apart; b_scale as
 *                ssd_fp8_quantise makes it with block_rows b_block_rows.
 *   out          (M, N) of out_dtype, rows out_stride elements apart (>= N); elements
 *                between the rows are not written.
 *   workspace    ssd_fp8_matmul_workspace_bytes(...) bytes, 256-byte aligned (NULL
 *                allowed when that is 0): partial sums where few outputs and a long K
 *                have the sum over k split (they are added in a fixed order), and the
 *                operands laid out anew where their rows do not start on 16 bytes or K is no
 *                multiple of 16.
 *                rows_on_16: whether they do, that is a, b, a_stride and b_stride are
 *                multiples of 16 and the strides below 2^24.
 * With y = x W^T: forward a = x, b = W (blocks of 128 x 128); grad_x takes a = grad_y and
 * b = W quantised with transpose; grad_W takes a = grad_y and b = x, both quantised with
 * transpose in blocks of 1 x 128.
 * Sums are float32, rounded once to out_dtype; for a bfloat16 result the sum inside a block
 * is the 8-bit matrix instruction's, which holds each eight neighbouring products to 2^-13
 * of the largest of them. M equal to 0 is a no-op; K equal to 0 writes zeros. M and N at most
 * 2^30 and K at most 2^24 - 16, at most 2^25 tiles of 128 x 128 results and fewer than 2^32
 * threads in one launch (SSD_ERR_UNSUPPORTED). No output may overlap an input (SSD_ERR_ALIAS).
 * The product of the two scales of a block has to be a float32 number.
 * Alignment: 4 bytes for the scales, the element size for out; rows of a and b that start
 * on 16 bytes, with K a multiple of 16, are read fastest.
 */
size_t ssd_fp8_matmul_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t b_block_rows,
                                      int out_dtype, int rows_on_16);

int ssd_fp8_matmul(const uint8_t *a, int64_t a_stride, const float *a_scale, const uint8_t *b,
                   int64_t b_stride, const float *b_scale, int64_t M, int64_t N, int64_t K,
                   int64_t b_block_rows, int out_dtype, void *out, int64_t out_stride,
                   void *workspace, size_t workspace_bytes, ssd_stream_t stream);

/* Tokens between two stored states of the gated delta rule. */
#define SSD_DELTA_CHUNK 64

/*
 * ssd_gated_delta -- the gated delta rule: a matrix state that decays by the token and is
 * corrected along the token's key. For every batch row b and value head h, with the key head
 * h / (Hv / Hk) and S (Dk, Dv),
 *
 *   S' = exp(g_t) S_{t-1}          u_t = beta_t (v_t - S'^T k_t)
 *   S_t = S' + k_t u_t^T           o_t = scale S_t^T q_t
 *
 *   q, k         (batch, T, Hk, Dk) of `dtype`; a token's heads and features lie side by side,
 *                consecutive tokens *_stride elements apart (>= Hk Dk) and consecutive
 *                batch rows T * *_stride, so that q, k and v may be column ranges of one
 *                matrix of projected rows. Read only.
 *   v            (batch, T, Hv, Dv) of `dtype`, v_stride >= Hv Dv. Hv is a multiple of Hk:
 *                neighbouring value heads share a key head.
 *   g, beta      (batch, T, Hv) float32, dense: the log of the decay (at most 0 for a
 *                state that fades; below -1000, also -infinity, it counts as -1000, and the state
 *                is forgotten) and the strength of the correction.
 *   scale        at most 1e30 in magnitude (usually Dk^-1/2).
 *   initial_state nullable: (batch, Hv, Dk, Dv) float32, S_{-1}; NULL means zero.
 *   lengths      nullable: (batch) int32 in device memory: the tokens of each row, clamped
 *                to 0 .. T. Tokens from there on are padding: what they hold does not matter, their
 *                o is 0, and the state stays as it is.
 *   o            out: (batch, T, Hv, Dv) of `dtype`, dense.
 *   final_state  out, nullable: (batch, Hv, Dk, Dv) float32, the state after the row's last
 *                token. It may be initial_state itself (updated in place).
 *   chunk_states out, nullable: (batch, ceil(T / SSD_DELTA_CHUNK), Hv, Dk, Dv) float32, the
 *                state before each chunk's first token, for the backward.
 *   workspace    ssd_gated_delta_workspace_bytes(...) bytes, 256-byte aligned (NULL allowed
 *                when that is 0).
 * The state, sums and products are float32 (operands as sums of up to three bfloat16 parts,
 * 24 bits); o is rounded once to `dtype`. The rule is a contraction where beta |k|^2 lies
 * in 0 .. 2: keys are meant to be scaled to a length of at most 1. Longer ones are
 * computed as they stand and may grow without bound, errors with them. An infinity, a NaN or a value
 * above 3.38e38 makes what it reaches NaN (or infinite): in v its column of the head,
 * in q the token's o of its heads, elsewhere what follows in its heads, and the tokens
 * before it in the same chunk.
 * T up to 8 is the form for generation: one or a few steps on the state.
 * No output may overlap an input or another output (SSD_ERR_ALIAS), but for the state in
 * place. Alignment: the element size. batch equal to 0 is a no-op; T equal to 0
 * copies the initial state (or zeros) into final_state.
 * SSD_ERR_BLOCK_DIMS: Dk above 128 or Dv above 256. SSD_ERR_UNSUPPORTED: T above 2^30,
 * batch above 2^24, heads above 2^16, a stride or Hv Dv above 2^23, a stride that makes an
 * operand longer than 2^40, or batch * Hv * max(ceil(T / 64), c) from 2^24 on, where c is 1 for
 * Dv up to 64 and 2 ceil(Dv / 128) beyond.
 */
size_t ssd_gated_delta_workspace_bytes(int64_t batch, int64_t T, int64_t Hk, int64_t Hv,
                                       int64_t Dk, int64_t Dv, int dtype);

int ssd_gated_delta(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                    const void *v, int64_t v_stride, const float *g, const float *beta,
                    float scale, int dtype, int64_t batch, int64_t T, int64_t Hk, int64_t Hv,
                    int64_t Dk, int64_t Dv, const float *initial_state, const int32_t *lengths,
                    void *o, float *final_state, float *chunk_states, void *workspace,
                    size_t workspace_bytes, ssd_stream_t stream);

/*
 * ssd_gated_delta_backward -- gradients of l = sum grad_o * o + sum grad_final_state *
 * final_state for ssd_gated_delta.
 *   q .. Dv, lengths as for the forward; chunk_states as it wrote them.
 *   grad_o       (batch, T, Hv, Dv) of `dtype`, dense; what the padding holds does not matter.
 *   grad_final_state nullable: (batch, Hv, Dk, Dv) float32.
 *   grad_q, grad_k out: (batch, T, Hk, Dk) of `dtype`, dense: the sums over the value heads
 *                that share the key head, in a fixed order; 0 in the padding.
 *   grad_v       out: (batch, T, Hv, Dv) of `dtype`, dense; 0 in the padding.
 *   grad_g, grad_beta out: (batch, T, Hv) float32; 0 in the padding.
 *   grad_initial_state out, nullable: (batch, Hv, Dk, Dv) float32.
 *   workspace    ssd_gated_delta_backward_workspace_bytes(...) bytes, 256-byte aligned.
 * What the chunks hold between the stored states is computed again in float32. No output
 * may overlap an input, another output or the workspace (SSD_ERR_ALIAS). batch or T
 * equal to 0 copies grad_final_state (or zeros) into grad_initial_state.
 */
size_t ssd_gated_delta_backward_workspace_bytes(int64_t batch, int64_t T, int64_t Hk, int64_t Hv,
                                                int64_t Dk, int64_t Dv, int dtype);

int ssd_gated_delta_backward(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                             const void *v, int64_t v_stride, const float *g, const float *beta,
                             float scale, int dtype, int64_t batch, int64_t T, int64_t Hk,
                             int64_t Hv, int64_t Dk, int64_t Dv, const float *chunk_states,
                             const int32_t *lengths, const void *grad_o,
                             const float *grad_final_state, void *grad_q, void *grad_k,
                             void *grad_v, float *grad_g, float *grad_beta,
                             float *grad_initial_state, void *workspace, size_t workspace_bytes,
                             ssd_stream_t stream);

/*
 * ssd_gated_norm -- the norm of a mixer's outputs by heads, fused with their gate, its result in
 * `dtype`, in 8 bits, or both. Per row of F values and head of D of them:
 *
 *   rstd = 1 / sqrt(sum x^2 / D + eps)     y = x * rstd * weight * silu(gate)
 *   q = e4m3(y / scale), one scale per 128 neighbours of the row
 *
 *   x, gate      (rows, F) of `dtype`, rows *_stride elements apart (>= F).
 *   weight       (D) float32, the same for every head. D divides F.
 *   y            out, nullable: (rows, F) of `dtype`, dense.
 *   q, scale     out, nullable together: (rows, F) e4m3 bytes and (ceil(F / 128), rows)
 *                float32, as ssd_fp8_matmul reads them; q is taken of the float32 y.
 *                One of y and q has to be given.
 *   rstd         out, nullable: (rows, F / D) float32, for the backward.
 * Sums are float32: a head's sum of squares has to stay below 2^128, and without an epsilon a
 * head whose mean square is below 2^-150 counts as zeros (its rstd is infinite). eps >= 0.
 * rows equal to 0 is a no-op. No output may overlap an input or another output
 * (SSD_ERR_ALIAS). Alignment: the element size. SSD_ERR_UNSUPPORTED: F above 16384, D below 8.
 */
int ssd_gated_norm(const void *x, int64_t x_stride, const void *gate, int64_t gate_stride,
                   const float *weight, int dtype, int64_t rows, int64_t F, int64_t D, float eps,
                   void *y, uint8_t *q, float *scale, float *rstd, ssd_stream_t stream);

/*
 * ssd_gated_norm_backward -- gradients of l = sum grad_y * y for ssd_gated_norm. With
 * n = x rstd, z = gate and b = grad_y silu(z) weight:
 *
 *   grad_x = rstd (b - n (sum b n) / D)        sums over the head
 *   grad_gate = grad_y n weight sigmoid(z) (1 + z (1 - sigmoid(z)))
 *   grad_weight = sum over rows and heads grad_y silu(z) n
 *
 *   rstd         as the forward wrote it.
 *   grad_y       (rows, F) of `dtype`, rows grad_y_stride elements apart.
 *   grad_x, grad_gate out: (rows, F) of `dtype`, dense.
 *   grad_weight  out: (D) float32, summed in a fixed order (in float32 over at most 256 rows, then in
 *                float64).
 *   workspace    ssd_gated_norm_backward_workspace_bytes(rows, F, D) bytes, 256-byte aligned.
 * rows equal to 0 sets grad_weight to zero. No output may overlap an input, another
 * output or the workspace (SSD_ERR_ALIAS).
 */
size_t ssd_gated_norm_backward_workspace_bytes(int64_t rows, int64_t F, int64_t D);

int ssd_gated_norm_backward(const void *x, int64_t x_stride, const void *gate,
                            int64_t gate_stride, const float *weight, const float *rstd,
                            const void *grad_y, int64_t grad_y_stride, int dtype, int64_t rows,
                            int64_t F, int64_t D, void *grad_x, void *grad_gate,
                            float *grad_weight, void *workspace, size_t workspace_bytes,
                            ssd_stream_t stream);

/*
 * ssd_block_norm -- the end of a block and the start of the next: the norm of the block's
 * output, its scaled addition to the residual stream, and the norm of that. Per row of F:
 *
 *   post_rstd = 1 / sqrt(sum x^2 / F + eps)   s = residual + residual_scale x post_rstd post_weight
 *   pre_rstd = 1 / sqrt(sum s^2 / F + eps)    y = s pre_rstd pre_weight
 *   q = e4m3(y / scale), one scale per 128 neighbours
 *
 *   x, residual  (rows, F) of `dtype`, rows *_stride elements apart (>= F).
 *   post_weight, pre_weight (F) float32. residual_scale: at most 1e30 in magnitude.
 *   y            out, nullable: (rows, F) of `dtype`, dense.
 *   residual_out out: s, rounded to `dtype`, (rows, F) dense. It may be residual itself if
 *                that is dense.
 *   q, scale     out, nullable together: as ssd_gated_norm. One of y and q has to be given.
 *   post_rstd, pre_rstd out, nullable: (rows) float32, for the backward.
 * Sums are float32 and taken of the unrounded s, with the limits of ssd_rms_norm. rows equal to
 * 0 is a no-op. No other overlap of outputs (SSD_ERR_ALIAS). Alignment: the element
 * size. SSD_ERR_UNSUPPORTED: F above 16384.
 */
int ssd_block_norm(const void *x, int64_t x_stride, const void *residual, int64_t residual_stride,
                   const float *post_weight, const float *pre_weight, float residual_scale,
                   int dtype, int64_t rows, int64_t F, float eps, void *y, void *residual_out,
                   uint8_t *q, float *scale, float *post_rstd, float *pre_rstd,
                   ssd_stream_t stream);

/*
 * ssd_block_norm_backward -- gradients of l = sum grad_y * y + sum grad_residual * s for
 * ssd_block_norm. With m = s pre_rstd and n = x post_rstd, means over the row:
 *
 *   grad_residual_in = grad_residual + pre_rstd (w grad_y - m mean(w grad_y m)), w = pre_weight
 *   a = residual_scale grad_residual_in
 *   grad_x = post_rstd (w a - n mean(w a n)), w = post_weight
 *   grad_post_weight = sum over rows a n      grad_pre_weight = sum over rows grad_y m
 *
 *   s            (rows, F) of `dtype`: the forward's residual_out.
 *   grad_y       (rows, F) of `dtype`; grad_residual nullable, the same: the gradient that
 *                reaches s through the residual stream.
 *   grad_x, grad_residual_in out: (rows, F) of `dtype`, dense.
 *   grad_post_weight, grad_pre_weight out: (F) float32, summed as grad_weight above.
 *   workspace    ssd_block_norm_backward_workspace_bytes(rows, F) bytes, 256-byte aligned.
 * rows equal to 0 sets the weights' gradients to zero. No output may overlap an input,
 * another output or the workspace (SSD_ERR_ALIAS).
 */
size_t ssd_block_norm_backward_workspace_bytes(int64_t rows, int64_t F);

int ssd_block_norm_backward(const void *x, int64_t x_stride, const void *s, int64_t s_stride,
                            const float *post_weight, const float *pre_weight,
                            const float *post_rstd, const float *pre_rstd, float residual_scale,
                            const void *grad_y, int64_t grad_y_stride, const void *grad_residual,
                            int64_t grad_residual_stride, int dtype, int64_t rows, int64_t F,
                            void *grad_x, void *grad_residual_in, float *grad_post_weight,
                            float *grad_pre_weight, void *workspace, size_t workspace_bytes,
                            ssd_stream_t stream);

/* Static text for a status code (never NULL). */
const char *ssd_status_string(int status);

/* Library version, major * 10000 + minor * 100 + patch. */
int ssd_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SSD_H */
