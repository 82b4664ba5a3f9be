/*
 * attn_gb300.h -- C ABI of the GB300 (sm_103a) scaled dot-product attention
 * forward library, libattn_gb300.so.
 *
 * The operation (per batch b, head h, query row i):
 *
 *   O[b,h,i,:] = sum_j softmax_j( scale * Q[b,h,i,:] . K[b,h,j,:] + mask(b,i,j) ) V[b,h,j,:]
 *
 * i.e. Eq. (1), Attention(Q,K,V) = softmax(Q K^T / sqrt(d_k)) V, of "Attention
 * Is All You Need" (rockcohen.cc/paper/t1-transformer, section 5.1; vlmlib.cn
 * paper summary, "scaled dot-product attention"), applied independently to
 * every head of multi-head attention (vlmlib.cn, "multi-head attention";
 * rockcohen.cc section 5.2). mask(b,i,j) is 0 for a legal connection and -inf for
 * an illegal one, added at the softmax input, so illegal keys get an exact zero
 * weight (rockcohen.cc sections 5.3 and 6.3). The three uses of attention
 * (rockcohen.cc section 5.3) are expressed through mask_mode and the shapes:
 *   encoder self-attention      ATTN_MASK_KEY_PADDING, n_q == n_k
 *   decoder masked self-attn.   ATTN_MASK_CAUSAL (optionally | KEY_PADDING), n_q == n_k
 *   encoder-decoder attention   ATTN_MASK_KEY_PADDING or NONE, n_q != n_k allowed
 *
 * Conventions shared by the entry points below:
 *   - Layouts are contiguous row-major [B, h, n, d] (the per-head layout that a
 *     split_heads reshape produces, csdn blog reimplementation):
 *       q   [B, h, n_q, d_k]    k [B, h, n_k, d_k]    v [B, h, n_k, d_v]
 *       out [B, h, n_q, d_v]    lse [B, h, n_q] (float32, optional)
 *   - Every pointer is a DEVICE pointer owned by the caller (the *_host entry points
 *     excepted). The library allocates no device memory; it neither keeps nor frees
 *     the pointers.
 *   - Calls are asynchronous on `stream` (a cudaStream_t passed as void*, NULL
 *     for the legacy default stream) and return before the GPU work finishes.
 *   - scale is used exactly as given; callers normally pass 1/sqrt(d_k) computed
 *     in double and rounded to float.
 *   - key_lens (int32 [B], device memory) gives each batch's number of valid keys
 *     (right padding); key j of batch b is illegal when j >= key_lens[b]. It is
 *     read only when mask_mode has ATTN_MASK_KEY_PADDING and may be NULL otherwise.
 *     Values are clamped to [0, n_k].
 *   - With ATTN_MASK_CAUSAL, key j is illegal for query i when j > i; it requires
 *     n_q == n_k.
 *   - lse[b,h,i] = ln sum_{j legal} exp(scale * q_i . k_j). A query row with no
 *     legal key (key length 0) gets out = 0 and lse = -inf. lse may be NULL.
 *   - Errors are returned as a status; nothing is printed and the process never
 *     exits. A status other than ATTN_OK means nothing was launched.
 */
#ifndef ATTN_GB300_H
#define ATTN_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  ATTN_OK = 0,
  ATTN_ERR_INVALID = -1,     /* null pointer, non-positive size, non-finite scale, bad mask,
                                causal with n_q != n_k, misaligned pointer, size overflow */
  ATTN_ERR_UNSUPPORTED = -2, /* shape this path does not implement (see each entry point) */
  ATTN_ERR_CUDA = -3,        /* a CUDA runtime/driver call failed (no GPU, launch error, ...) */
  ATTN_ERR_TIMEOUT = -4      /* a kernel gave up waiting on an internal barrier (reported by
                                attn_fault_status) */
} attn_status;

enum { ATTN_MASK_NONE = 0, ATTN_MASK_CAUSAL = 1, ATTN_MASK_KEY_PADDING = 2 };

/* attn_bwd flags */
enum { ATTN_BWD_DETERMINISTIC = 1 };

/*
 * attn_fwd -- bf16 inputs and output, fp32 accumulation (sm_103a tensor cores).
 *   q, k, v, out: bf16 (raw 16-bit) arrays, 16-byte aligned.
 *   lse: float32 or NULL.
 *   Supported: d_k == d_v in {64, 128}; any B, h, n_q, n_k >= 1 whose element
 *   counts fit in int32 per head-row index and whose byte strides fit TMA limits.
 *   Otherwise ATTN_ERR_UNSUPPORTED.
 * Numerics: QK^T and PV accumulate in fp32 on the tensor cores; the softmax is the
 * online (running max / running sum) form in fp32 with exp2 and the scale folded
 * in; the probabilities are rounded to bf16 before the PV product; the output is
 * divided by the row sum in fp32 and rounded to bf16 (nearest-even).
 */
int attn_fwd(const void* q, const void* k, const void* v, void* out, float* lse,
             int B, int h, int n_q, int n_k, int d_k, int d_v, float scale,
             int mask_mode, const int32_t* key_lens, void* stream);

/*
 * attn_weights -- the softmax weights of Eq. (1) themselves (rockcohen.cc "Attention Is
 * All You Need" section 5.1), the second value the pages' scaled_dot_product_attention
 * returns beside the output (csdn blog reimplementation, scaled_dot_product_attention):
 *   w[b, h, i, j] = exp(scale * q_i . k_j - lse_i) for every legal key j of row i
 *   (the mask of attn_fwd), and exactly 0 for the others and for every key of a row
 *   with no legal key (lse_i = -inf).
 * With lse the log-sum-exp that attn_fwd returned for the same q, k, scale, mask_mode
 * and key_lens, each row of legal weights sums to 1 up to that lse's rounding.
 *   q [B, h, n_q, d], k [B, h, n_k, d]: bf16 device arrays, 16-byte aligned.
 *   lse [B, h, n_q]: float32 device array (required).
 *   w [B, h, n_q, n_k]: float32 device array, 16-byte aligned, written in full;
 *           B*h*n_q*n_k floats, owned by the caller.
 *   mask_mode, key_lens, scale and stream as in attn_fwd.
 * Supported: d in {64, 128}; otherwise ATTN_ERR_UNSUPPORTED. The score q_i . k_j
 * accumulates in fp32 on the tensor cores; the exponential is exp2 of the scaled score
 * in log2 units. The matrix is B*h*n_q*n_k floats: this is for inspecting attention
 * (the forward never forms it), and its cost is that write.
 */
int attn_weights(const void* q, const void* k, const float* lse, float* w, int B, int h, int n_q, int n_k, int d,
                 float scale, int mask_mode, const int32_t* key_lens, void* stream);

/*
 * attn_fwd_host_workspace_size -- bytes of device workspace attn_fwd_host needs for
 * this shape and mask (four chunk slots of Q, K, V, out, lse plus the key lengths;
 * the mask enters through the chunk plan). Returns 0 for an invalid shape or mask
 * (d must be 64 or 128). Depends only on the arguments.
 */
size_t attn_fwd_host_workspace_size(int B, int h, int n_q, int n_k, int d, int mask_mode);

/*
 * attn_fwd_host -- attn_fwd for operands that live in HOST memory, the call an
 * application makes when its Q, K, V are not yet on the GPU. Same operation, masks,
 * numerics and results as attn_fwd (bit for bit: the same kernel runs on each chunk).
 *   q, k, v, key_lens: host memory, read by the call;   out, lse: host memory, written.
 *   Page-locked (pinned) host memory is strongly recommended: with pageable memory the
 *   copies are staged by the driver and do not overlap the kernels.
 *   workspace: device scratch of at least attn_fwd_host_workspace_size(B, h, n_q,
 *   n_k, d_k, mask_mode) bytes, 256-byte aligned, owned by the caller.
 * The flattened (b, h) head range is cut into chunks. Chunk c's host-to-device copy,
 * its attention kernel and its device-to-host copy run on the library's own streams
 * (one for each direction, one per slot for the kernels) through a four-slot ring in
 * the workspace, so transfers overlap computation and consecutive kernels overlap
 * each other. Every stream waits for what `stream` had queued before the call, and
 * `stream` waits for all of them. The call is asynchronous: the host buffers must
 * stay valid and unmodified (q, k, v, key_lens) or unread (out, lse) until `stream`
 * reaches this call's end, which includes every copy back; calls made
 * from several host threads are serialised per device. Errors as attn_fwd; a failure
 * after some chunks were queued returns ATTN_ERR_CUDA with those chunks in flight.
 */
int attn_fwd_host(const void* q, const void* k, const void* v, void* out, float* lse,
                  int B, int h, int n_q, int n_k, int d_k, int d_v, float scale,
                  int mask_mode, const int32_t* key_lens, void* workspace,
                  size_t workspace_bytes, void* stream);

/*
 * attn_fwd_local -- restricted (local-window) self-attention, bf16, on the same
 * tensor-core kernel as attn_fwd. The pages propose, for very long sequences,
 * letting each position attend only to positions within a neighbourhood r, which
 * lowers the cost from O(n^2 d) to O(r n d) (csdn blog section 4.3 and "future
 * work"; vlmlib.cn "limitations"). Here r = `window` is a radius: key j is legal
 * for query i only if |i - j| <= window, in addition to whatever mask_mode imposes
 * (ATTN_MASK_CAUSAL makes the window one-sided, i - window <= j <= i;
 * ATTN_MASK_KEY_PADDING as in attn_fwd). Self-attention only: q, k, v, out are
 * [B, h, n, d]. K/V tiles outside every row's window are never loaded.
 * window >= 0 (ATTN_ERR_INVALID otherwise); a window of n or more restricts nothing
 * (|i - j| < n always). Other rules as attn_fwd.
 */
int attn_fwd_local(const void* q, const void* k, const void* v, void* out, float* lse,
                   int B, int h, int n, int d_k, int d_v, float scale, int window,
                   int mask_mode, const int32_t* key_lens, void* stream);

/*
 * attn_fwd_f32 -- float32 inputs and output, float32 arithmetic throughout
 * (CUDA cores). Same semantics and conventions as attn_fwd; pointers 4-byte
 * aligned; 1 <= d_k, d_v <= 256, otherwise ATTN_ERR_UNSUPPORTED.
 */
int attn_fwd_f32(const float* q, const float* k, const float* v, float* out, float* lse,
                 int B, int h, int n_q, int n_k, int d_k, int d_v, float scale,
                 int mask_mode, const int32_t* key_lens, void* stream);

/*
 * attn_decode_workspace_size -- bytes of device workspace attn_decode needs for
 * this shape (the split-K partial results: fp32 partial outputs, running maxima
 * and sums). Returns 0 for an invalid shape. Depends only on the arguments.
 */
size_t attn_decode_workspace_size(int B, int h, int n_q, int n_max, int d);

/*
 * attn_decode -- one autoregressive decoding step against a key/value cache:
 * n_q new queries per (b, h) attend to the cached keys up to their own position.
 * Generation proceeds one position at a time under the causal mask of decoder
 * self-attention (attention-paper-guide section 05; rockcohen.cc sections 5.3,
 * 6.3); query i of batch b sits at position cache_lens[b] - n_q + i and key j is
 * legal iff j <= cache_lens[b] - n_q + i. The result equals the last n_q rows of
 * causal self-attention over the first cache_lens[b] positions.
 *   q       bf16 [B, h, n_q, d]         k_cache, v_cache  bf16 [B, h, n_max, d]
 *   out     bf16 [B, h, n_q, d]         lse  float [B, h, n_q] or NULL
 *   cache_lens  int32 [B], device, each in [0, n_max] (a value outside is clamped to
 *           that range before the query positions are placed). A query whose
 *           position is negative (cache_lens[b] < n_q) has no legal key: out = 0,
 *           lse = -inf.
 *   workspace   device scratch of at least attn_decode_workspace_size(...) bytes,
 *           16-byte aligned, owned by the caller; its contents on entry do not
 *           matter and on return are undefined. Two calls that run at the same time
 *           must not share a workspace.
 * Supported: 1 <= n_q <= 16, d in {64, 128}, B*h <= 65535. Pointers 16-byte
 * aligned. fp32 arithmetic throughout (scores, exp2, sums, P.V); the output is
 * rounded to bf16 once. Asynchronous on `stream`; two kernels are launched (one
 * warp per cache chunk for n_q = 1, one block per cache range for n_q > 1; then the
 * merge).
 */
int attn_decode(const void* q, const void* k_cache, const void* v_cache, void* out, float* lse,
                int B, int h, int n_q, int n_max, int d, float scale,
                const int32_t* cache_lens, void* workspace, size_t workspace_bytes, void* stream);

/*
 * attn_decode_noalloc -- attn_decode for callers that cannot allocate device memory.
 * (An addition of this library; the paper has no counterpart.)
 * Some callers have no way to obtain device scratch: plug-ins whose host framework
 * owns every device buffer and hands a kernel only its inputs and outputs,
 * latency-critical serving loops that must not enter the allocator (cudaMalloc and
 * cudaFree can synchronise the whole device), and programs that fix their device
 * memory at start-up. This entry point takes the same arguments as attn_decode minus
 * the workspace and allocates nothing: no cudaMalloc, cudaFree or allocating
 * library call. Its scratch is a static buffer of ATTN_DECODE_NOALLOC_MAX_BYTES
 * inside the library's device image, present on every GPU that loads the library
 * until the process exits.
 *   - The first call on a device looks up the buffer's device address (with that
 *     device current) and keeps it; make that first call before any stream capture.
 *     A cudaDeviceReset after that first call is not supported: the kept address
 *     belongs to the context the reset destroyed.
 *   - Every call on a device shares the one buffer, which keeps the last call's
 *     contents (the kernels write every slot before reading it, an abandoned range
 *     included, so nothing needs clearing). Calls whose GPU work overlaps -- on
 *     different streams, or from several host threads -- race on it: order them,
 *     e.g. on one stream.
 *   - A shape whose workspace (attn_decode_workspace_size) exceeds
 *     ATTN_DECODE_NOALLOC_MAX_BYTES returns ATTN_ERR_UNSUPPORTED and launches
 *     nothing; use attn_decode with a caller workspace for it.
 * Results are those of attn_decode on the same inputs.
 */
#define ATTN_DECODE_NOALLOC_MAX_BYTES (4u << 20)
int attn_decode_noalloc(const void* q, const void* k_cache, const void* v_cache, void* out, float* lse,
                        int B, int h, int n_q, int n_max, int d, float scale,
                        const int32_t* cache_lens, void* stream);

/*
 * attn_bwd_workspace_size -- bytes of device workspace attn_bwd needs for this shape,
 * head size d and flags: two fp32 per query row (-lse_i log2(e) and -D_i below),
 * padded to whole 128-row tiles, plus, for the fused schedule (d = 64 without
 * ATTN_BWD_DETERMINISTIC), an fp32 dQ accumulator of B*h*n_q*64 floats. Returns 0 for
 * an invalid shape, head size or flag.
 */
size_t attn_bwd_workspace_size(int B, int h, int n_q, int d, int flags);

/*
 * attn_bwd -- gradients of attn_fwd with respect to q, k and v, given the gradient
 * dout of the output. Training the model by gradient descent needs them
 * (attention-paper-guide section 05; vlmlib.cn "training"). With P the softmax
 * weights of Eq. (1) (rockcohen.cc section 5.1) recomputed from lse,
 * P[i,j] = exp(scale * q_i . k_j - lse_i) on legal pairs and 0 on illegal ones:
 *   dv_j = sum_i P[i,j] dout_i
 *   dP[i,j] = dout_i . v_j,  D_i = dout_i . out_i,  dS[i,j] = P[i,j] (dP[i,j] - D_i)
 *   dq_i = scale sum_j dS[i,j] k_j,      dk_j = scale sum_i dS[i,j] q_i
 *   q, k, v, out, dout: bf16 as in attn_fwd (out and lse are those attn_fwd returned
 *           for the same q, k, v, scale, mask_mode and key_lens; lse is required)
 *   dq [B, h, n_q, d], dk, dv [B, h, n_k, d]: bf16, written in full (a key that no
 *           query may see gets dk = dv = 0; a query with no legal key gets dq = 0)
 *   flags: 0, or ATTN_BWD_DETERMINISTIC (any other bit: ATTN_ERR_INVALID).
 *   workspace: device scratch of at least attn_bwd_workspace_size(B, h, n_q, d_k,
 *           flags) bytes, 16-byte aligned, owned by the caller, contents undefined on
 *           return; concurrent calls must not share it.
 * mask_mode and key_lens as in attn_fwd. Supported: d_k == d_v in {64, 128}.
 * Numerics: S and dP accumulate in fp32 on the tensor cores; P and dS are rounded to
 * bf16 before the three products that consume them, which accumulate in fp32; D_i
 * is accumulated in fp32 from the bf16 out and dout; results are rounded to bf16
 * once. Schedules:
 *   - fused (d = 64, flags = 0): each of the five products is computed once; the
 *     partial dQ of every 128-key tile is added into the fp32 workspace accumulator
 *     with TMA reduce-adds, whose order varies, so the last bits of dq can differ
 *     from run to run (dk and dv are deterministic). A memset and three kernels.
 *   - deterministic (d = 128, or ATTN_BWD_DETERMINISTIC): a dK/dV kernel and a dQ
 *     kernel that recomputes S and dP (seven products), no atomics: bit-identical
 *     results on every run. Three kernels.
 * All launches are on `stream`.
 */
int attn_bwd(const void* q, const void* k, const void* v, const void* out, const void* dout, const float* lse,
             void* dq, void* dk, void* dv, int B, int h, int n_q, int n_k, int d_k, int d_v, float scale,
             int mask_mode, const int32_t* key_lens, int flags, void* workspace, size_t workspace_bytes,
             void* stream);

/*
 * attn_bwd_local -- gradients of attn_fwd_local (restricted self-attention: key j is
 * legal for query i only if |i - j| <= window, together with mask_mode; vlmlib.cn
 * "restricted self-attention"), exactly as attn_bwd computes them for
 * attn_fwd: the same definitions, numerics, schedules, flags and workspace
 * (attn_bwd_workspace_size(B, h, n, d_k, flags)), with n_q = n_k = n and the window
 * entering P's mask. out and lse are those attn_fwd_local returned for the same
 * q, k, v, scale, window, mask_mode and key_lens. window < 0: ATTN_ERR_INVALID; a
 * window of n or more is the unrestricted mask (as in attn_fwd_local).
 * Key tiles no query of a query tile may see, and query tiles outside a key tile's
 * window, are skipped; every dq, dk, dv element is still written.
 */
int attn_bwd_local(const void* q, const void* k, const void* v, const void* out, const void* dout,
                   const float* lse, void* dq, void* dk, void* dv, int B, int h, int n, int d_k, int d_v,
                   float scale, int window, int mask_mode, const int32_t* key_lens, int flags, void* workspace,
                   size_t workspace_bytes, void* stream);

/*
 * attn_bwd_host_workspace_size -- bytes of device workspace attn_bwd_host needs for
 * this shape, head size, mask and flags (four chunk slots of the nine per-head tensors
 * and their gradient workspace, plus the key lengths). Returns 0 for an invalid shape,
 * head size, mask or flag. Depends only on the arguments.
 */
size_t attn_bwd_host_workspace_size(int B, int h, int n_q, int n_k, int d, int mask_mode, int flags);

/*
 * attn_bwd_host -- attn_bwd for operands that live in HOST memory (a training step
 * whose tensors are on the host). Same gradients, schedules, flags and numerics as
 * attn_bwd: the same kernels run on each chunk of heads (dk and dv bit-identical to
 * attn_bwd on the same data; dq as well with ATTN_BWD_DETERMINISTIC).
 *   q, k, v, out, dout, lse, key_lens: host memory, read;   dq, dk, dv: host memory,
 *   written. Page-locked (pinned) host memory is strongly recommended.
 *   workspace: device scratch of at least attn_bwd_host_workspace_size(B, h, n_q, n_k,
 *   d_k, mask_mode, flags) bytes, 256-byte aligned, owned by the caller.
 * The flattened (b, h) head range is cut into chunks whose host-to-device copies,
 * gradient kernels and device-to-host copies run on the library's own streams through
 * a four-slot ring in the workspace, as in attn_fwd_host. The call is asynchronous on
 * `stream` and ordered with it at both ends; the host buffers must stay valid (and the
 * inputs unmodified) until `stream` reaches the end of the call. Errors as attn_bwd.
 */
int attn_bwd_host(const void* q, const void* k, const void* v, const void* out, const void* dout, const float* lse,
                  void* dq, void* dk, void* dv, int B, int h, int n_q, int n_k, int d_k, int d_v, float scale,
                  int mask_mode, const int32_t* key_lens, int flags, void* workspace, size_t workspace_bytes,
                  void* stream);

/*
 * attn_linear -- one linear projection of the multi-head layer, bf16 in and out:
 *   y[M, N] = x[M, K] w[K, N] + bias[N]
 * The layer projects queries, keys and values with per-head matrices W_i^Q, W_i^K,
 * W_i^V and the concatenated heads with W^O (vlmlib.cn paper summary, "multi-head
 * attention"; the csdn blog's MultiHeadAttention uses nn.Linear layers with biases);
 * placing the h per-head matrices side by side makes each projection this product.
 *   x  [M, K], w [K, N] (the paper's x W orientation; an nn.Linear weight is the
 *      transpose), y [M, N]: row-major bf16, 16-byte aligned, caller-owned device memory
 *   bias [N] bf16, 16-byte aligned, or NULL for none.
 * Supported: N and K multiples of 8 (16-byte rows); otherwise ATTN_ERR_UNSUPPORTED.
 * Numerics: the products accumulate in fp32 on the sm_103a tensor cores (tcgen05,
 * operands staged by TMA); the bias is added in fp32 and the sum rounded to bf16
 * (nearest-even) once. One launch on `stream`; x and y must not overlap.
 */
int attn_linear(const void* x, const void* w, const void* bias, void* y, int M, int N, int K, void* stream);

/*
 * attn_mha_workspace_size -- bytes of device workspace attn_mha_fwd needs: the
 * projected Q', K', V' and the concatenated heads (bf16, each padded to 256 bytes).
 * Returns 0 for an invalid or unsupported shape.
 */
size_t attn_mha_workspace_size(int B, int n_q, int n_k, int d_model, int h, int d);

/*
 * attn_mha_fwd -- the multi-head attention layer (vlmlib.cn "multi-head attention":
 * MultiHead(Q,K,V) = Concat(head_1..head_h) W^O, head_i = Attention(Q W_i^Q, K W_i^K,
 * V W_i^V); the csdn blog's MultiHeadAttention with its linear projections, split_heads
 * and concatenation), bf16 in and out:
 *   Q' = x_q W^Q + b_Q, K' = x_kv W^K + b_K, V' = x_kv W^V + b_V     [B, n, h*d]
 *   A  = attn_fwd(Q', K', V') per head, heads concatenated          [B, n_q, h*d]
 *   out = A W^O + b_O                                                [B, n_q, d_model]
 *   x_q  [B, n_q, d_model], x_kv [B, n_k, d_model] (pass x_q twice for self-attention)
 *   w_q, w_k, w_v [d_model, h*d], w_o [h*d, d_model]: row-major, the paper's x W
 *           orientation (an nn.Linear weight is the transpose); head i uses columns
 *           i*d .. i*d + d - 1 of W^Q, W^K, W^V and rows i*d .. of W^O
 *   b_q, b_k, b_v [h*d], b_o [d_model]: bf16 or NULL for no bias
 *   out  [B, n_q, d_model] bf16
 *   mask_mode, key_lens, scale: as attn_fwd (scale is normally 1/sqrt(d)).
 *   workspace: device scratch of at least attn_mha_workspace_size(...) bytes, 16-byte
 *           aligned, owned by the caller, contents undefined on return; concurrent
 *           calls must not share it.
 * Supported: d_k == d_v in {64, 128}, d_model a multiple of 8; every pointer 16-byte
 * aligned. The four projections have the numerics of attn_linear (fp32 accumulation
 * on the tensor cores, bias added in fp32, one rounding to bf16); the three input
 * projections run as one launch of the projection kernel. The attention is the
 * attn_fwd kernel reading Q', K', V' and writing A in their [B, n, h*d] layout, so
 * splitting and concatenating the heads moves no data. Three launches on `stream`.
 */
int attn_mha_fwd(const void* x_q, const void* x_kv, const void* w_q, const void* b_q, const void* w_k,
                 const void* b_k, const void* w_v, const void* b_v, const void* w_o, const void* b_o, void* out,
                 int B, int n_q, int n_k, int d_model, int h, int d_k, int d_v, float scale, int mask_mode,
                 const int32_t* key_lens, void* workspace, size_t workspace_bytes, void* stream);

/* flags of attn_norm_rope, attn_norm_rope_bwd, attn_paged_append (both) and attn_paged_decode (the second) */
enum { ATTN_ROPE_INTERLEAVED = 1, ATTN_CACHE_E4M3 = 2 };

/*
 * attn_norm_rope -- what a decoder does to its projected queries and keys before the
 * attention, in one pass: the RMS norm of every head and the position rotation.
 * (An addition of this library; the paper adds position encodings to the embeddings.)
 * For each head row x of d columns, with w the norm's weight,
 *   y = x / sqrt(mean(x^2) + eps) * w          (no weights: y = x)
 *   o_a = y_a cos t_i - y_b sin t_i,  o_b = y_b cos t_i + y_a sin t_i   for the column pairs (a, b)
 * where t_i is angle i of the token's position: pairs (i, i + d_rot / 2), or with
 * ATTN_ROPE_INTERLEAVED (2 i, 2 i + 1), i < d_rot / 2; columns from d_rot on are not turned.
 *   q, k    bf16, token-major: head h of token x (of B * n) starts at q + x * q_stride + h * d
 *           (strides in elements, multiples of 8, at least heads * d): slices of one fused
 *           projection, for instance
 *   q_out [B, h_q, n, d], k_out [B, h_kv, n, d]: bf16, the layout attn_fwd reads (which has
 *           one h: for h_kv < h_q the caller repeats each key head for its h_q / h_kv query
 *           heads); they must not overlap q or k
 *   q_weight, k_weight [d]: bf16, or both NULL for no norm;   eps >= 0, finite
 *   cos_sin [n_pos, d_rot]: float32, row = position: d_rot / 2 cosines, then their sines
 *           (any scaling of the angles is in the table); not read when d_rot is 0
 *   positions [B, n]: int32, or NULL for 0 .. n - 1 in every sequence (then n <= n_pos).
 *           A token whose position is negative or, with d_rot > 0, not below n_pos, is
 *           padding: its outputs are zero.
 *   flags   0 or ATTN_ROPE_INTERLEAVED
 * Supported: d in {64, 128}, d_rot a multiple of 16 in [0, d]; heads * d < 2^31; data
 * pointers 16-byte aligned. fp32 arithmetic, one rounding to bf16. One launch on `stream`.
 */
int attn_norm_rope(const void* q, const void* k, int64_t q_stride, int64_t k_stride, const void* q_weight,
                   const void* k_weight, float eps, const float* cos_sin, int n_pos, int d_rot,
                   const int32_t* positions, void* q_out, void* k_out, int B, int n, int h_q, int h_kv, int d,
                   int flags, void* stream);

/*
 * attn_norm_rope_bwd_workspace_size -- bytes of device workspace attn_norm_rope_bwd needs
 * with a norm (each CTA's share of the weights' gradients). Returns 0 for an invalid shape.
 */
size_t attn_norm_rope_bwd_workspace_size(int B, int n, int h_q, int h_kv, int d);

/*
 * attn_norm_rope_bwd -- gradients of attn_norm_rope. With g the gradient of one output row,
 * gy that row turned back, r = 1 / sqrt(mean(x^2) + eps) and u = gy w:
 *   dx = r (u - x r^2 mean(u x)),   dw = sum over tokens and heads of gy x r   (no norm: dx = gy)
 *   q, k, q_stride .. positions, B .. flags: as in the forward call
 *   dq_out [B, h_q, n, d], dk_out [B, h_kv, n, d]: bf16, what attn_bwd returns
 *   dq, dk  bf16, token-major with strides dq_stride, dk_stride; written in full (columns
 *           between the heads' and the stride are left as they were); no overlap with inputs
 *   dq_weight, dk_weight [d]: float32, written; required with a norm, NULL without
 *   workspace: with a norm, device scratch of at least attn_norm_rope_bwd_workspace_size
 *           bytes, 16-byte aligned, owned by the caller, contents undefined on return;
 *           concurrent calls must not share it. Without a norm it may be NULL.
 * Padding tokens get dq = dk = 0 and add nothing to the weights' gradients. fp32
 * arithmetic; no atomics: the same bits on every run. Two launches with a norm, else one.
 */
int attn_norm_rope_bwd(const void* q, const void* k, int64_t q_stride, int64_t k_stride, const void* q_weight,
                       const void* k_weight, float eps, const float* cos_sin, int n_pos, int d_rot,
                       const int32_t* positions, const void* dq_out, const void* dk_out, void* dq, void* dk,
                       int64_t dq_stride, int64_t dk_stride, float* dq_weight, float* dk_weight, int B, int n,
                       int h_q, int h_kv, int d, int flags, void* workspace, size_t workspace_bytes, void* stream);

/*
 * attn_paged_append -- writes the keys and values of T new tokens into a paged cache, with
 * the norm and rotation of attn_norm_rope applied to the keys on the way, and (q not NULL)
 * normalises and rotates the tokens' queries: the step before attn_paged_decode, or a
 * packed batch of prompts of different lengths. (An addition of this library.)
 *   q [T, h_q, d], k, v [T, h_kv, d]: bf16, token-major with strides as in attn_norm_rope
 *   q_out [T, h_q, d]: bf16, contiguous; NULL exactly when q is (then q_weight is NULL too);
 *           it and the pages must not overlap q, k or v
 *   q_weight, k_weight, eps, cos_sin, n_pos, d_rot: as in attn_norm_rope (values are neither
 *           normalised nor turned)
 *   positions [T]: int32, the token's place in its sequence: its angle and its cache row
 *   seq_ids [T]: int32, the token's sequence, or NULL: token x belongs to sequence x (T <= n_seqs)
 *   page_table [n_seqs, max_pages]: int32; entry (s, p) is the page that holds positions
 *           p * page_size .. of sequence s
 *   k_pages, v_pages [n_pages, h_kv, page_size, d]: bf16, or with ATTN_CACHE_E4M3 8-bit
 *           floats (4 exponent, 3 mantissa bits) of value / k_scale[h] and value / v_scale[h],
 *           rounded to nearest, saturated at 448
 *   k_scale, v_scale [h_kv]: float32, positive; required with ATTN_CACHE_E4M3, else NULL
 * A token is skipped whole (nothing of it is written, q_out included) when its position is
 * negative, not below n_pos (d_rot > 0) or beyond max_pages pages, when its sequence id is
 * outside [0, n_seqs), or when its page table entry is outside [0, n_pages): a batch padded
 * to a fixed size marks its padding with position -1. Cache rows of no token stay as they
 * were. Two tokens with the same sequence and position leave either's values, column by
 * column. Supported: d in {64, 128}, d_rot a multiple of 16, heads * d < 2^31, any page size
 * (n_pages * h_kv * page_size < 2^31, max_pages * page_size <= 2^30). One launch on `stream`.
 */
int attn_paged_append(const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
                      int64_t v_stride, const void* q_weight, const void* k_weight, float eps, const float* cos_sin,
                      int n_pos, int d_rot, const int32_t* positions, const int32_t* seq_ids,
                      const int32_t* page_table, int n_seqs, int max_pages, void* q_out, void* k_pages,
                      void* v_pages, int n_pages, int page_size, const float* k_scale, const float* v_scale, int T,
                      int h_q, int h_kv, int d, int flags, void* stream);

/*
 * attn_paged_decode_workspace_size -- bytes of device workspace attn_paged_decode needs.
 * Independent of B and of the lengths (two partial results per resident warp). Returns 0
 * for an invalid or unsupported shape.
 */
size_t attn_paged_decode_workspace_size(int B, int n_q, int h_q, int h_kv, int d);

/*
 * attn_paged_decode -- attn_decode over a paged cache: the newest n_q tokens of each of B
 * sequences attend to the cached keys up to their own position. Query head h uses
 * key/value head h / (h_q / h_kv).
 *   q, out  bf16 [B, n_q, h_q, d] (token-major: what attn_paged_append returns for B * n_q
 *           tokens, and what the output projection reads)
 *   lse     float32 [B, n_q, h_q], or NULL
 *   k_pages, v_pages, page_table, max_pages, n_pages, page_size: the cache, as in
 *           attn_paged_append, one page table row per sequence
 *   cache_lens [B]: int32, tokens in the cache including the new ones, clamped to [0,
 *           max_pages * page_size]. Query i stands at position cache_lens[b] - n_q + i; one
 *           whose position is negative has no legal key: out = 0, lse = -inf.
 *   window  -1, or the radius of attn_fwd_local: key j is legal for position x only if
 *           x - window <= j <= x ...
 *   sinks   ... or j < sinks, j <= x: the first tokens that stay visible (>= 0; nothing
 *           without a window)
 *   k_scale, v_scale, flags: ATTN_CACHE_E4M3 and the scales as in attn_paged_append, or 0, NULL
 *   workspace: device scratch of at least attn_paged_decode_workspace_size(...) bytes,
 *           16-byte aligned, owned by the caller, contents undefined on return; concurrent
 *           calls must not share it.
 * A page table entry outside [0, n_pages) names no page: its keys count as illegal. Cache
 * rows behind the length are never used, whatever they hold; a key that one of the rows
 * may not see does not reach that row, infinities and NaN included.
 * Supported: 1 <= n_q <= 16, d in {64, 128}, h_q a multiple of h_kv (of at most 8192
 * h_kv), any page size (limits as in attn_paged_append), and with `keys` the most that a
 * sequence may see (max_pages * page_size, or window + n_q + sinks),
 * B * h_kv * ceil(n_q * h_q / h_kv / 8) * (ceil(keys / 16) + 2) < 2^30.
 * Numerics: the products accumulate in fp32 on the tensor cores, softmax statistics in fp32;
 * the weights enter the second product as two bf16 parts, within 2^-15 of each (8-bit
 * cache: as f16, within 2^-11, or 2^-40 of the largest), and the output is rounded once to
 * bf16. With an 8-bit cache the queries enter the first product as f16, scaled by a power of
 * two: exact but for entries below 2^-14 of the row's largest, which move by at most 2^-25
 * of it. One or two launches on `stream`.
 */
int attn_paged_decode(const void* q, const void* k_pages, const void* v_pages, void* out, float* lse,
                      const int32_t* page_table, const int32_t* cache_lens, int B, int n_q, int h_q, int h_kv, int d,
                      int n_pages, int page_size, int max_pages, float scale, int window, int sinks,
                      const float* k_scale, const float* v_scale, int flags, void* workspace, size_t workspace_bytes,
                      void* stream);

/*
 * attn_packed_fwd_workspace_size -- bytes of device workspace attn_packed_fwd needs: its work
 * list, and partial results whose size does not depend on T_q or n_seqs. Returns 0 for an
 * invalid or unsupported shape.
 */
size_t attn_packed_fwd_workspace_size(int T_q, int n_seqs, int h_q, int h_kv, int d);

/*
 * attn_packed_fwd -- attn_fwd for sequences of different lengths packed one after the other,
 * without padding between them, whose query heads share key/value heads. (An addition of this
 * library.) Query head h uses key/value head h / (h_q / h_kv).
 *   q, out  bf16 [T_q, h_q, d], k, v bf16 [T_k, h_kv, d]: element (x, h, c) at x * stride +
 *           h * head_stride + c. Strides are multiples of 8, and tokens or heads are the
 *           outer side (slices of one fused projection [T, (h_q + 2 h_kv) d], or what
 *           attn_norm_rope returns for B = 1); the stride of a single token or head is not
 *           read. out must not overlap the others.
 *   lse     float32 [T_q, h_q], contiguous, or NULL
 *   q_starts, k_starts [n_seqs + 1]: int32, not decreasing: sequence b's queries are rows
 *           q_starts[b] .. q_starts[b + 1] - 1, its keys rows k_starts[b] .. of k and v.
 *           k_starts NULL: the queries' rows. Rows of no sequence (before the first, behind the
 *           last) are not used, and left as they were in out and lse. Offsets outside the
 *           arrays are clamped to them; a sequence that ends before it starts is empty. (Offsets that
 *           decrease and so name rows more than once leave rows with any or no result.)
 *   mask_mode  ATTN_MASK_NONE or ATTN_MASK_CAUSAL. Query i of a sequence of n_q queries and n_k
 *           keys stands at position x = n_k - n_q + i (the last query at the last key); causal:
 *           key j is legal for j <= x only.
 *   window  -1, or the radius of attn_fwd_local: key j is legal for |x - j| <= window only
 *   workspace: device scratch of at least attn_packed_fwd_workspace_size(...) bytes, 256-byte
 *           aligned, owned by the caller, contents undefined on return; concurrent calls must
 *           not share it.
 * A query without a legal key gets out = 0, lse = -inf. What other sequences' rows and rows of
 * no sequence hold, infinities and NaN included, does not reach a sequence; within a sequence a
 * value row's infinities and NaN may reach every query whose 128-key tile holds it, masked or not.
 * Supported: d in {64, 128}, h_q a multiple of h_kv (of at most 128 h_kv), scale > 0, T_q and
 * T_k below 2^28, n_seqs h_kv and the numbers of 128-row tiles below 2^30 together.
 * Numerics as attn_fwd: fp32 accumulation on the tensor cores, weights rounded to bf16 for the
 * second product, one rounding of the output. One to three launches on `stream`; no atomics on
 * results: the same bits on every run.
 */
int attn_packed_fwd(const void* q, const void* k, const void* v, void* out, float* lse, int64_t q_stride,
                    int64_t q_head_stride, int64_t k_stride, int64_t k_head_stride, int64_t v_stride,
                    int64_t v_head_stride, int64_t out_stride, int64_t out_head_stride, const int32_t* q_starts,
                    const int32_t* k_starts, int n_seqs, int T_q, int T_k, int h_q, int h_kv, int d, float scale,
                    int mask_mode, int window, void* workspace, size_t workspace_bytes, void* stream);

/*
 * attn_packed_bwd_workspace_size -- bytes of device workspace attn_packed_bwd needs: its work
 * lists, two floats per query row, and partial results of fixed size. Returns 0 for an invalid
 * or unsupported shape.
 */
size_t attn_packed_bwd_workspace_size(int T_q, int T_k, int n_seqs, int h_q, int h_kv, int d);

/*
 * attn_packed_bwd -- gradients of attn_packed_fwd, with the definitions of attn_bwd; the
 * gradients of a key/value head are the sums over the query heads that share it.
 *   q, k, v, q_starts .. window: as in the forward call; out and lse are what it returned
 *   dout, dq  bf16 [T_q, h_q, d], dk, dv  bf16 [T_k, h_kv, d]
 *   strides  HOST array of 16: token stride and head stride of q, k, v, out, dout, dq, dk, dv, with
 *           the forward's rules. The gradients must not overlap one another or the inputs
 *           (slices of one array are fine).
 *   workspace: as in attn_packed_fwd, of at least attn_packed_bwd_workspace_size(...) bytes
 * Written for every row of every sequence: a key that no query may see gets dk = dv = 0, a query
 * with no legal key dq = 0. Rows of no sequence are not used and left as they were. What other
 * sequences' rows hold, infinities and NaN included, does not reach a sequence; within a sequence those of a row of q,
 * k or dout may reach the gradients of every row that meets its 128-row tile, masked or not.
 * Supported: as attn_packed_fwd. Numerics as attn_bwd: fp32 accumulation on the tensor cores, P and dS
 * rounded to bf16, results rounded to bf16 once; no atomics: the same bits on every run. Three or
 * four launches on `stream`.
 */
int attn_packed_bwd(const void* q, const void* k, const void* v, const void* out, const void* dout, const float* lse,
                    void* dq, void* dk, void* dv, const int64_t* strides, const int32_t* q_starts,
                    const int32_t* k_starts, int n_seqs, int T_q, int T_k, int h_q, int h_kv, int d, float scale,
                    int mask_mode, int window, void* workspace, size_t workspace_bytes, void* stream);

/*
 * attn_paged_chunk_workspace_size -- bytes of device workspace attn_paged_chunk needs, for
 * either cache type. Returns 0 for an invalid or unsupported shape.
 */
size_t attn_paged_chunk_workspace_size(int T, int n_seqs, int h_q, int h_kv, int d);

/*
 * attn_paged_chunk -- attn_paged_decode for any number of new tokens in every sequence, from none
 * to a whole prompt: the step after attn_paged_append for prompts, pieces of prompts, and
 * batches in which some sequences bring a piece and others one token. (An addition of this
 * library.)
 *   q, out  bf16 [T, h_q, d], contiguous: what attn_paged_append returns
 *   lse     float32 [T, h_q], or NULL
 *   q_starts [n_seqs + 1]: int32, as in attn_packed_fwd: sequence b's new tokens are rows
 *           q_starts[b] .. q_starts[b + 1] - 1, the newest last. Rows of no sequence are left as
 *           they were.
 *   k_pages, v_pages, page_table, n_pages, page_size, max_pages, k_scale, v_scale, flags: the
 *           cache, as in attn_paged_append, one page table row per sequence
 *   cache_lens [n_seqs]: int32, tokens in the cache including the new ones, clamped to [0,
 *           max_pages * page_size]. New token i of n stands at position cache_lens[b] - n + i; one
 *           whose position is negative has no legal key: out = 0, lse = -inf.
 *   window, sinks: as in attn_paged_decode
 *   workspace: as in attn_packed_fwd, of at least attn_paged_chunk_workspace_size(...) bytes
 * A page table entry outside [0, n_pages) names no page: its keys count as illegal. Cache rows
 * behind the length are never used, whatever they hold; nor are pages of which no new token may see a row (behind
 * its sequence's first tokens and before all windows), whatever their entries name: they may be given to others.
 * As in attn_packed_fwd, and unlike attn_paged_decode, infinities and NaN in a value row of the other pages may reach
 * every new token of its sequence whose 128-key tile holds it, masked or not.
 * Supported: d in {64, 128}, h_q a multiple of h_kv (of at most 128 h_kv), scale > 0, any page size
 * (limits as in attn_paged_append; copies are of gcd(page_size, 128) rows, so page sizes that are
 * multiples of 8 or more are the fast ones), T below 2^28. Numerics as attn_packed_fwd (over bf16 pages the weights are
 * rounded to bf16, where attn_paged_decode keeps two parts of each: where values cancel, a token's output can be off
 * by more than its own rounding), except with an 8-bit cache: its numbers enter the products exactly, as f16, and the operands beside them are f16
 * too, each row of q times a power of two (exact but for entries below 2^-28 of the row's largest, which
 * are rounded to 2^-39 of it) and the weights (rounded to 11 bits; those below 2^-32 of the row's largest
 * may vanish). One to three launches on `stream`.
 */
int attn_paged_chunk(const void* q, const void* k_pages, const void* v_pages, void* out, float* lse,
                     const int32_t* q_starts, const int32_t* page_table, const int32_t* cache_lens, int n_seqs, int T,
                     int h_q, int h_kv, int d, int n_pages, int page_size, int max_pages, float scale, int window,
                     int sinks, const float* k_scale, const float* v_scale, int flags, void* workspace,
                     size_t workspace_bytes, void* stream);

/*
 * attn_fault_status -- synchronises `stream`, then reports whether any kernel of
 * this library on the current device gave up waiting on one of its internal
 * barriers since the last clear (each such wait is bounded in time; a kernel that
 * gives up writes no further output and returns). Returns ATTN_OK,
 * ATTN_ERR_TIMEOUT, or ATTN_ERR_CUDA. If `clear` is non-zero the record is reset.
 * `fault_code` (may be NULL) receives the raw record: bit 0 producer, bit 1 MMA
 * issuer, bit 2 softmax, bit 3 epilogue (attn_fwd), bit 4 decode copy (attn_decode),
 * bit 5 gradient kernels (attn_bwd), bit 6 attn_fwd found its shared memory not
 * 1024-byte aligned (it then writes nothing), bit 7 projection kernel (attn_linear,
 * attn_mha_fwd), bit 8 attn_weights, bit 9 attn_packed_fwd and attn_paged_chunk,
 * bit 10 attn_packed_bwd.
 */
int attn_fault_status(void* stream, int clear, uint32_t* fault_code);

/* attn_status_string -- static, human-readable name of a status code. */
const char* attn_status_string(int status);

#ifdef __cplusplus
}
#endif
#endif /* ATTN_GB300_H */
