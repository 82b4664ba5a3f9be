// attn_api.cu -- the extern "C" entry points of libattn_gb300.so: argument
// validation, the tensor-map encoder lookup, and dispatch to the kernels. The
// semantics are documented in include/attn_gb300.h.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "attn_internal.h"

namespace {

attn::PFN_encodeTiled tensor_map_encoder() {
  static attn::PFN_encodeTiled fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult qres = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &qres) !=
            cudaSuccess ||
        qres != cudaDriverEntryPointSuccess)
      return static_cast<attn::PFN_encodeTiled>(nullptr);
    return reinterpret_cast<attn::PFN_encodeTiled>(f);
  }();
  return fn;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Checks shared by both entry points; returns ATTN_OK or an error status.
int check_common(const void* q, const void* k, const void* v, const void* out, const float* lse, int B, int h,
                 int n_q, int n_k, int d_k, int d_v, float scale, int mask_mode, const int32_t* key_lens) {
  if (!q || !k || !v || !out) return ATTN_ERR_INVALID;
  if (B <= 0 || h <= 0 || n_q <= 0 || n_k <= 0 || d_k <= 0 || d_v <= 0) return ATTN_ERR_INVALID;
  if (!std::isfinite(scale)) return ATTN_ERR_INVALID;
  if (mask_mode < 0 || mask_mode > (ATTN_MASK_CAUSAL | ATTN_MASK_KEY_PADDING)) return ATTN_ERR_INVALID;
  if ((mask_mode & ATTN_MASK_CAUSAL) && n_q != n_k) return ATTN_ERR_INVALID;
  if ((mask_mode & ATTN_MASK_KEY_PADDING) && (!key_lens || !aligned(key_lens, 4))) return ATTN_ERR_INVALID;
  if (lse && !aligned(lse, 4)) return ATTN_ERR_INVALID;
  const long long bh = (long long)B * h;
  if (bh > 0x7fffffffLL) return ATTN_ERR_INVALID;
  // every element index must fit in a signed 64-bit offset with room to spare
  const long long maxn = n_q > n_k ? n_q : n_k, maxd = d_k > d_v ? d_k : d_v;
  if (bh * maxn > (1LL << 40) / maxd) return ATTN_ERR_INVALID;
  return ATTN_OK;
}

// The kernels count a token's columns in 32 bits.
bool too_wide(int h, int d) { return (long long)h * d > 0x7fffffffLL; }

// Heads' rows laid out by token: `tokens` rows of h * d columns, `stride` elements apart.
bool bad_rows(const void* x, long long tokens, int64_t stride, int h, int d) {
  return !x || too_wide(h, d) || !aligned(x, 16) || stride < (long long)h * d || stride % 8 != 0 || stride > (1LL << 40) / tokens;
}

// The norm and rotation arguments that attn_norm_rope, its gradients and attn_paged_append
// share; d is checked by the caller.
int check_rope(const void* q_weight, const void* k_weight, float eps, const float* cos_sin, int n_pos, int d_rot,
               int d) {
  if ((q_weight && !aligned(q_weight, 16)) || (k_weight && !aligned(k_weight, 16))) return ATTN_ERR_INVALID;
  if (!std::isfinite(eps) || eps < 0.0f) return ATTN_ERR_INVALID;
  if (d_rot < 0 || d_rot > d) return ATTN_ERR_INVALID;
  if (d_rot > 0 && (!cos_sin || !aligned(cos_sin, 16) || n_pos <= 0)) return ATTN_ERR_INVALID;
  return d_rot % 16 == 0 ? ATTN_OK : ATTN_ERR_UNSUPPORTED;
}

// The checks of attn_norm_rope and its gradients on the forward's operands.
int check_norm_rope(const void* q, const void* k, int64_t q_stride, int64_t k_stride, const void* q_weight,
                    const void* k_weight, float eps, const float* cos_sin, int n_pos, int d_rot,
                    const int32_t* positions, int B, int n, int h_q, int h_kv, int d, int flags) {
  if (B <= 0 || n <= 0 || h_q <= 0 || h_kv <= 0 || d <= 0) return ATTN_ERR_INVALID;
  const long long tokens = (long long)B * n;
  if (tokens > 0x7fffff00LL || (long long)h_q + h_kv > (1LL << 40) / d / tokens) return ATTN_ERR_INVALID;
  if (bad_rows(q, tokens, q_stride, h_q, d) || bad_rows(k, tokens, k_stride, h_kv, d)) return ATTN_ERR_INVALID;
  if ((q_weight == nullptr) != (k_weight == nullptr)) return ATTN_ERR_INVALID;
  if (flags & ~ATTN_ROPE_INTERLEAVED) return ATTN_ERR_INVALID;
  if (positions && !aligned(positions, 4)) return ATTN_ERR_INVALID;
  if (!positions && d_rot > 0 && n > n_pos) return ATTN_ERR_INVALID;
  const int st = check_rope(q_weight, k_weight, eps, cos_sin, n_pos, d_rot, d);
  if (st != ATTN_OK) return st;
  return d == 64 || d == 128 ? ATTN_OK : ATTN_ERR_UNSUPPORTED;
}

// A paged cache's geometry: rows addressed by 31 bits, lengths by 30.
bool bad_cache(const void* k_pages, const void* v_pages, int n_pages, int page_size, int max_pages, int h_kv,
               const int32_t* page_table) {
  if (!k_pages || !v_pages || !aligned(k_pages, 16) || !aligned(v_pages, 16)) return true;
  if (!page_table || !aligned(page_table, 4)) return true;
  if (n_pages <= 0 || page_size <= 0 || max_pages <= 0 || h_kv <= 0) return true;
  if ((long long)n_pages * page_size > 0x7fffffffLL / h_kv) return true;
  return (long long)max_pages * page_size > (1LL << 30);
}

// One packed operand [tokens, heads, d] with strides between tokens and heads, either of them the
// outer one; the stride of a single token or head does not matter and is replaced.
bool bad_packed(const void* x, long long tokens, int heads, int d, int64_t& ts, int64_t& hs) {
  if (!x || !aligned(x, 16)) return true;
  if (heads == 1) hs = tokens == 1 || ts >= d ? d : ts;
  if (tokens == 1) ts = heads == 1 || hs >= d ? d : hs;
  if (ts < d || hs < d || ts % 8 != 0 || hs % 8 != 0 || ts > (1LL << 38) || hs > (1LL << 38)) return true;
  if (ts > (1LL << 40) / tokens || hs > (1LL << 40) / heads) return true;
  if (tokens == 1 || heads == 1) return false;
  return ts < (heads - 1) * hs + d && hs < (tokens - 1) * ts + d;  // neither token-major nor head-major: rows overlap
}

constexpr int kMaxPacked = 1 << 28;  // tokens of a packed array

// Sizes of a ragged batch: an error status, or ATTN_OK.
int check_ragged(int n_seqs, long long T_q, long long T_k, int h_q, int h_kv, int d) {
  if (n_seqs <= 0 || T_q <= 0 || T_k <= 0 || h_q <= 0 || h_kv <= 0 || d <= 0 || h_q % h_kv != 0) return ATTN_ERR_INVALID;
  if (T_q >= kMaxPacked || T_k >= kMaxPacked || n_seqs >= kMaxPacked) return ATTN_ERR_INVALID;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  const int group = h_q / h_kv;
  if (group > 128) return ATTN_ERR_UNSUPPORTED;
  // the work list is counted in 32 bits
  const long long tok = 128 / group;
  if ((T_q / tok + T_k / 128 + 2LL * n_seqs + 2) * h_kv > (1LL << 30)) return ATTN_ERR_UNSUPPORTED;
  if ((T_q > T_k ? T_q : T_k) > (1LL << 40) / d / h_q) return ATTN_ERR_INVALID;
  return ATTN_OK;
}

}  // namespace

extern "C" {

int attn_fwd(const void* q, const void* k, const void* v, void* out, float* lse, int B, int h, int n_q, int n_k,
             int d_k, int d_v, float scale, int mask_mode, const int32_t* key_lens, void* stream) {
  int st = check_common(q, k, v, out, lse, B, h, n_q, n_k, d_k, d_v, scale, mask_mode, key_lens);
  if (st != ATTN_OK) return st;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16)) return ATTN_ERR_INVALID;
  if (d_k != d_v || (d_k != 64 && d_k != 128)) return ATTN_ERR_UNSUPPORTED;
  attn::PFN_encodeTiled enc = tensor_map_encoder();
  if (!enc) return ATTN_ERR_CUDA;
  attn::TcArgs a{q, k, v, out, lse, B, h, n_q, n_k, d_k, scale, mask_mode, key_lens,
                 static_cast<cudaStream_t>(stream), -1};
  return attn::launch_attn_tc(a, enc);
}

int attn_weights(const void* q, const void* k, const float* lse, float* w, int B, int h, int n_q, int n_k, int d,
                 float scale, int mask_mode, const int32_t* key_lens, void* stream) {
  int st = check_common(q, k, k, w, lse, B, h, n_q, n_k, d, d, scale, mask_mode, key_lens);
  if (st != ATTN_OK) return st;
  if (!lse || !aligned(q, 16) || !aligned(k, 16) || !aligned(w, 16)) return ATTN_ERR_INVALID;
  // the weights tensor itself must stay addressable with 64-bit element offsets
  if ((long long)B * h * n_q > (1LL << 62) / n_k) return ATTN_ERR_INVALID;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  attn::PFN_encodeTiled enc = tensor_map_encoder();
  if (!enc) return ATTN_ERR_CUDA;
  attn::WeightsArgs a{q, k, lse, w, B, h, n_q, n_k, d, scale, mask_mode, key_lens, static_cast<cudaStream_t>(stream)};
  return attn::launch_attn_weights(a, enc);
}

size_t attn_fwd_host_workspace_size(int B, int h, int n_q, int n_k, int d, int mask_mode) {
  if (B <= 0 || h <= 0 || n_q <= 0 || n_k <= 0 || (d != 64 && d != 128)) return 0;
  if (mask_mode < 0 || mask_mode > (ATTN_MASK_CAUSAL | ATTN_MASK_KEY_PADDING)) return 0;
  const long long bh = (long long)B * h;
  if (bh > 0x7fffffffLL || bh * (n_q > n_k ? n_q : n_k) > (1LL << 40) / d) return 0;
  return attn::host_workspace_bytes(B, h, n_q, n_k, d, mask_mode);
}

int attn_fwd_host(const void* q, const void* k, const void* v, void* out, float* lse, int B, int h, int n_q,
                  int n_k, int d_k, int d_v, float scale, int mask_mode, const int32_t* key_lens, void* workspace,
                  size_t workspace_bytes, void* stream) {
  int st = check_common(q, k, v, out, lse, B, h, n_q, n_k, d_k, d_v, scale, mask_mode, key_lens);
  if (st != ATTN_OK) return st;
  if (!workspace || !aligned(workspace, 256)) return ATTN_ERR_INVALID;
  if (d_k != d_v || (d_k != 64 && d_k != 128)) return ATTN_ERR_UNSUPPORTED;
  if (workspace_bytes < attn::host_workspace_bytes(B, h, n_q, n_k, d_k, mask_mode)) return ATTN_ERR_INVALID;
  attn::PFN_encodeTiled enc = tensor_map_encoder();
  if (!enc) return ATTN_ERR_CUDA;
  attn::TcArgs a{q, k, v, out, lse, B, h, n_q, n_k, d_k, scale, mask_mode, key_lens,
                 static_cast<cudaStream_t>(stream), -1};
  return attn::launch_attn_host(a, enc, workspace);
}

int attn_fwd_local(const void* q, const void* k, const void* v, void* out, float* lse, int B, int h, int n,
                   int d_k, int d_v, float scale, int window, int mask_mode, const int32_t* key_lens,
                   void* stream) {
  int st = check_common(q, k, v, out, lse, B, h, n, n, d_k, d_v, scale, mask_mode, key_lens);
  if (st != ATTN_OK) return st;
  if (window < 0) return ATTN_ERR_INVALID;
  window = window < n ? window : n;  // |i - j| < n always: a wider window is the same mask
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16)) return ATTN_ERR_INVALID;
  if (d_k != d_v || (d_k != 64 && d_k != 128)) return ATTN_ERR_UNSUPPORTED;
  attn::PFN_encodeTiled enc = tensor_map_encoder();
  if (!enc) return ATTN_ERR_CUDA;
  attn::TcArgs a{q, k, v, out, lse, B, h, n, n, d_k, scale, mask_mode, key_lens,
                 static_cast<cudaStream_t>(stream), window};
  return attn::launch_attn_tc(a, enc);
}

int attn_fwd_f32(const float* q, const float* k, const float* v, float* out, float* lse, int B, int h, int n_q,
                 int n_k, int d_k, int d_v, float scale, int mask_mode, const int32_t* key_lens, void* stream) {
  int st = check_common(q, k, v, out, lse, B, h, n_q, n_k, d_k, d_v, scale, mask_mode, key_lens);
  if (st != ATTN_OK) return st;
  if (!aligned(q, 4) || !aligned(k, 4) || !aligned(v, 4) || !aligned(out, 4)) return ATTN_ERR_INVALID;
  if (d_k > 256 || d_v > 256) return ATTN_ERR_UNSUPPORTED;
  attn::F32Args a{q, k, v, out, lse, B, h, n_q, n_k, d_k, d_v, scale, mask_mode, key_lens,
                  static_cast<cudaStream_t>(stream)};
  return attn::launch_attn_f32(a);
}

size_t attn_decode_workspace_size(int B, int h, int n_q, int n_max, int d) {
  if (B <= 0 || h <= 0 || n_q < 1 || n_q > 16 || n_max <= 0 || (d != 64 && d != 128)) return 0;
  if ((long long)B * h > 65535) return 0;
  return attn::decode_workspace_bytes(B, h, n_q, n_max, d);
}

int attn_decode(const void* q, const void* k_cache, const void* v_cache, void* out, float* lse, int B, int h,
                int n_q, int n_max, int d, float scale, const int32_t* cache_lens, void* workspace,
                size_t workspace_bytes, void* stream) {
  if (!q || !k_cache || !v_cache || !out || !cache_lens || !workspace) return ATTN_ERR_INVALID;
  if (B <= 0 || h <= 0 || n_q <= 0 || n_max <= 0 || d <= 0) return ATTN_ERR_INVALID;
  if (!std::isfinite(scale)) return ATTN_ERR_INVALID;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
      !aligned(workspace, 16) || !aligned(cache_lens, 4) || (lse && !aligned(lse, 4)))
    return ATTN_ERR_INVALID;
  if (n_q > 16 || (d != 64 && d != 128) || (long long)B * h > 65535) return ATTN_ERR_UNSUPPORTED;
  if ((long long)B * h * n_max > (1LL << 40) / d) return ATTN_ERR_INVALID;
  if (workspace_bytes < attn::decode_workspace_bytes(B, h, n_q, n_max, d)) return ATTN_ERR_INVALID;
  attn::DecodeArgs a{q, k_cache, v_cache, out, lse, B, h, n_q, n_max, d, scale, cache_lens,
                     static_cast<cudaStream_t>(stream)};
  return attn::launch_attn_decode(a, workspace);
}

int attn_decode_noalloc(const void* q, const void* k_cache, const void* v_cache, void* out, float* lse, int B,
                        int h, int n_q, int n_max, int d, float scale, const int32_t* cache_lens, void* stream) {
  if (!q || !k_cache || !v_cache || !out || !cache_lens) return ATTN_ERR_INVALID;
  if (B <= 0 || h <= 0 || n_q <= 0 || n_max <= 0 || d <= 0) return ATTN_ERR_INVALID;
  if (!std::isfinite(scale)) return ATTN_ERR_INVALID;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
      !aligned(cache_lens, 4) || (lse && !aligned(lse, 4)))
    return ATTN_ERR_INVALID;
  if (n_q > 16 || (d != 64 && d != 128) || (long long)B * h > 65535) return ATTN_ERR_UNSUPPORTED;
  if ((long long)B * h * n_max > (1LL << 40) / d) return ATTN_ERR_INVALID;
  attn::DecodeArgs a{q, k_cache, v_cache, out, lse, B, h, n_q, n_max, d, scale, cache_lens,
                     static_cast<cudaStream_t>(stream)};
  return attn::launch_attn_decode_noalloc(a);
}

size_t attn_bwd_workspace_size(int B, int h, int n_q, int d, int flags) {
  if (B <= 0 || h <= 0 || n_q <= 0 || (long long)B * h > 0x7fffffffLL) return 0;
  if ((d != 64 && d != 128) || (flags & ~ATTN_BWD_DETERMINISTIC)) return 0;
  if ((long long)B * h * n_q > (1LL << 40) / 64) return 0;
  return attn::bwd_workspace_bytes(B, h, n_q, d, flags);
}

int attn_bwd(const void* q, const void* k, const void* v, const void* out, const void* dout, const float* lse,
             void* dq, void* dk, void* dv, int B, int h, int n_q, int n_k, int d_k, int d_v, float scale,
             int mask_mode, const int32_t* key_lens, int flags, void* workspace, size_t workspace_bytes,
             void* stream) {
  int st = check_common(q, k, v, out, lse, B, h, n_q, n_k, d_k, d_v, scale, mask_mode, key_lens);
  if (st != ATTN_OK) return st;
  if (!dout || !lse || !dq || !dk || !dv || !workspace) return ATTN_ERR_INVALID;
  if (flags & ~ATTN_BWD_DETERMINISTIC) return ATTN_ERR_INVALID;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(dout, 16) ||
      !aligned(dq, 16) || !aligned(dk, 16) || !aligned(dv, 16) || !aligned(workspace, 16))
    return ATTN_ERR_INVALID;
  if (d_k != d_v || (d_k != 64 && d_k != 128)) return ATTN_ERR_UNSUPPORTED;
  if (workspace_bytes < attn::bwd_workspace_bytes(B, h, n_q, d_k, flags)) return ATTN_ERR_INVALID;
  attn::PFN_encodeTiled enc = tensor_map_encoder();
  if (!enc) return ATTN_ERR_CUDA;
  attn::BwdArgs a{q, k, v, out, dout, lse, dq, dk, dv, B, h, n_q, n_k, d_k, scale, mask_mode, key_lens,
                  static_cast<cudaStream_t>(stream), flags};
  return attn::launch_attn_bwd(a, enc, workspace);
}

int attn_bwd_local(const void* q, const void* k, const void* v, const void* out, const void* dout,
                   const float* lse, void* dq, void* dk, void* dv, int B, int h, int n, int d_k, int d_v,
                   float scale, int window, int mask_mode, const int32_t* key_lens, int flags, void* workspace,
                   size_t workspace_bytes, void* stream) {
  int st = check_common(q, k, v, out, lse, B, h, n, n, d_k, d_v, scale, mask_mode, key_lens);
  if (st != ATTN_OK) return st;
  if (window < 0) return ATTN_ERR_INVALID;
  window = window < n ? window : n;  // |i - j| < n always: a wider window is the same mask
  if (!dout || !lse || !dq || !dk || !dv || !workspace) return ATTN_ERR_INVALID;
  if (flags & ~ATTN_BWD_DETERMINISTIC) return ATTN_ERR_INVALID;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(dout, 16) ||
      !aligned(dq, 16) || !aligned(dk, 16) || !aligned(dv, 16) || !aligned(workspace, 16))
    return ATTN_ERR_INVALID;
  if (d_k != d_v || (d_k != 64 && d_k != 128)) return ATTN_ERR_UNSUPPORTED;
  if (workspace_bytes < attn::bwd_workspace_bytes(B, h, n, d_k, flags)) return ATTN_ERR_INVALID;
  attn::PFN_encodeTiled enc = tensor_map_encoder();
  if (!enc) return ATTN_ERR_CUDA;
  attn::BwdArgs a{q, k, v, out, dout, lse, dq, dk, dv, B, h, n, n, d_k, scale, mask_mode, key_lens,
                  static_cast<cudaStream_t>(stream), flags, window};
  return attn::launch_attn_bwd(a, enc, workspace);
}

size_t attn_bwd_host_workspace_size(int B, int h, int n_q, int n_k, int d, int mask_mode, int flags) {
  if (B <= 0 || h <= 0 || n_q <= 0 || n_k <= 0 || (d != 64 && d != 128)) return 0;
  if (mask_mode < 0 || mask_mode > (ATTN_MASK_CAUSAL | ATTN_MASK_KEY_PADDING)) return 0;
  if (flags & ~ATTN_BWD_DETERMINISTIC) return 0;
  const long long bh = (long long)B * h;
  if (bh > 0x7fffffffLL || bh * (n_q > n_k ? n_q : n_k) > (1LL << 40) / d) return 0;
  return attn::bwd_host_workspace_bytes(B, h, n_q, n_k, d, mask_mode, flags);
}

int attn_bwd_host(const void* q, const void* k, const void* v, const void* out, const void* dout, const float* lse,
                  void* dq, void* dk, void* dv, int B, int h, int n_q, int n_k, int d_k, int d_v, float scale,
                  int mask_mode, const int32_t* key_lens, int flags, void* workspace, size_t workspace_bytes,
                  void* stream) {
  int st = check_common(q, k, v, out, lse, B, h, n_q, n_k, d_k, d_v, scale, mask_mode, key_lens);
  if (st != ATTN_OK) return st;
  if (!dout || !lse || !dq || !dk || !dv || !workspace || !aligned(workspace, 256)) return ATTN_ERR_INVALID;
  if (flags & ~ATTN_BWD_DETERMINISTIC) return ATTN_ERR_INVALID;
  if (d_k != d_v || (d_k != 64 && d_k != 128)) return ATTN_ERR_UNSUPPORTED;
  if (workspace_bytes < attn::bwd_host_workspace_bytes(B, h, n_q, n_k, d_k, mask_mode, flags)) return ATTN_ERR_INVALID;
  attn::PFN_encodeTiled enc = tensor_map_encoder();
  if (!enc) return ATTN_ERR_CUDA;
  attn::BwdArgs a{q, k, v, out, dout, lse, dq, dk, dv, B, h, n_q, n_k, d_k, scale, mask_mode, key_lens,
                  static_cast<cudaStream_t>(stream), flags};
  return attn::launch_attn_bwd_host(a, enc, workspace);
}

int attn_linear(const void* x, const void* w, const void* bias, void* y, int M, int N, int K, void* stream) {
  if (!x || !w || !y) return ATTN_ERR_INVALID;
  if (M <= 0 || N <= 0 || K <= 0) return ATTN_ERR_INVALID;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(y, 16) || (bias && !aligned(bias, 16))) return ATTN_ERR_INVALID;
  if (N % 8 != 0 || K % 8 != 0) return ATTN_ERR_UNSUPPORTED;
  if ((long long)M * (N > K ? N : K) > (1LL << 40) || (long long)K * N > (1LL << 40)) return ATTN_ERR_INVALID;
  attn::PFN_encodeTiled enc = tensor_map_encoder();
  if (!enc) return ATTN_ERR_CUDA;
  const attn::LinearJob job{x, w, bias, y, M, N, K};
  return attn::launch_linear(&job, 1, enc, static_cast<cudaStream_t>(stream));
}

size_t attn_mha_workspace_size(int B, int n_q, int n_k, int d_model, int h, int d) {
  if (B <= 0 || n_q <= 0 || n_k <= 0 || d_model <= 0 || h <= 0 || (d != 64 && d != 128)) return 0;
  if ((long long)B * (n_q > n_k ? n_q : n_k) * h * d > (1LL << 38)) return 0;
  if ((long long)B * (n_q > n_k ? n_q : n_k) > 0x7fffffffLL) return 0;
  return attn::mha_workspace_bytes(B, n_q, n_k, h, d);
}

int attn_mha_fwd(const void* x_q, const void* x_kv, const void* w_q, const void* b_q, const void* w_k,
                 const void* b_k, const void* w_v, const void* b_v, const void* w_o, const void* b_o, void* out,
                 int B, int n_q, int n_k, int d_model, int h, int d_k, int d_v, float scale, int mask_mode,
                 const int32_t* key_lens, void* workspace, size_t workspace_bytes, void* stream) {
  if (!x_q || !x_kv || !w_q || !w_k || !w_v || !w_o || !out || !workspace) return ATTN_ERR_INVALID;
  if (B <= 0 || n_q <= 0 || n_k <= 0 || d_model <= 0 || h <= 0 || d_k <= 0 || d_v <= 0) return ATTN_ERR_INVALID;
  if (!std::isfinite(scale)) return ATTN_ERR_INVALID;
  if (mask_mode < 0 || mask_mode > (ATTN_MASK_CAUSAL | ATTN_MASK_KEY_PADDING)) return ATTN_ERR_INVALID;
  if ((mask_mode & ATTN_MASK_CAUSAL) && n_q != n_k) return ATTN_ERR_INVALID;
  if ((mask_mode & ATTN_MASK_KEY_PADDING) && (!key_lens || !aligned(key_lens, 4))) return ATTN_ERR_INVALID;
  const void* ptrs16[] = {x_q, x_kv, w_q, w_k, w_v, w_o, out, workspace, b_q, b_k, b_v, b_o};
  for (const void* ptr : ptrs16)
    if (ptr && !aligned(ptr, 16)) return ATTN_ERR_INVALID;
  if (d_k != d_v || (d_k != 64 && d_k != 128) || d_model % 8 != 0) return ATTN_ERR_UNSUPPORTED;
  const size_t need = attn_mha_workspace_size(B, n_q, n_k, d_model, h, d_k);
  if (need == 0) return ATTN_ERR_INVALID;
  if (workspace_bytes < need) return ATTN_ERR_INVALID;
  attn::PFN_encodeTiled enc = tensor_map_encoder();
  if (!enc) return ATTN_ERR_CUDA;
  attn::MhaArgs a{x_q, x_kv, w_q, b_q, w_k, b_k, w_v, b_v, w_o, b_o, out, B, n_q, n_k, d_model, h, d_k, scale,
                  mask_mode, key_lens, static_cast<cudaStream_t>(stream)};
  return attn::launch_attn_mha(a, enc, workspace);
}

int attn_norm_rope(const void* q, const void* k, int64_t q_stride, int64_t k_stride, const void* q_weight,
                   const void* k_weight, float eps, const float* cos_sin, int n_pos, int d_rot,
                   const int32_t* positions, void* q_out, void* k_out, int B, int n, int h_q, int h_kv, int d,
                   int flags, void* stream) {
  const int st = check_norm_rope(q, k, q_stride, k_stride, q_weight, k_weight, eps, cos_sin, n_pos, d_rot, positions,
                                 B, n, h_q, h_kv, d, flags);
  if (st != ATTN_OK) return st;
  if (!q_out || !k_out || !aligned(q_out, 16) || !aligned(k_out, 16)) return ATTN_ERR_INVALID;
  attn::RopeArgs a{q, k, q_stride, k_stride, q_weight, k_weight, eps, cos_sin, n_pos, d_rot, positions, q_out, k_out,
                   B, n, h_q, h_kv, d, (flags & ATTN_ROPE_INTERLEAVED) != 0, static_cast<cudaStream_t>(stream)};
  return attn::launch_attn_norm_rope(a);
}

size_t attn_norm_rope_bwd_workspace_size(int B, int n, int h_q, int h_kv, int d) {
  if (B <= 0 || n <= 0 || h_q <= 0 || h_kv <= 0 || (d != 64 && d != 128)) return 0;
  const long long tokens = (long long)B * n;
  if (tokens > 0x7fffff00LL || (long long)h_q + h_kv > (1LL << 40) / d / tokens) return 0;
  if (too_wide(h_q, d) || too_wide(h_kv, d)) return 0;
  return attn::norm_rope_bwd_workspace_bytes(B, n, h_q, h_kv, d);
}

int attn_norm_rope_bwd(const void* q, const void* k, int64_t q_stride, int64_t k_stride, const void* q_weight,
                       const void* k_weight, float eps, const float* cos_sin, int n_pos, int d_rot,
                       const int32_t* positions, const void* dq_out, const void* dk_out, void* dq, void* dk,
                       int64_t dq_stride, int64_t dk_stride, float* dq_weight, float* dk_weight, int B, int n,
                       int h_q, int h_kv, int d, int flags, void* workspace, size_t workspace_bytes, void* stream) {
  const int st = check_norm_rope(q, k, q_stride, k_stride, q_weight, k_weight, eps, cos_sin, n_pos, d_rot, positions,
                                 B, n, h_q, h_kv, d, flags);
  if (st != ATTN_OK) return st;
  if (!dq_out || !dk_out || !aligned(dq_out, 16) || !aligned(dk_out, 16)) return ATTN_ERR_INVALID;
  const long long tokens = (long long)B * n;
  if (bad_rows(dq, tokens, dq_stride, h_q, d) || bad_rows(dk, tokens, dk_stride, h_kv, d)) return ATTN_ERR_INVALID;
  if (q_weight) {
    if (!dq_weight || !dk_weight || !aligned(dq_weight, 4) || !aligned(dk_weight, 4)) return ATTN_ERR_INVALID;
    if (!workspace || !aligned(workspace, 16)) return ATTN_ERR_INVALID;
    if (workspace_bytes < attn::norm_rope_bwd_workspace_bytes(B, n, h_q, h_kv, d)) return ATTN_ERR_INVALID;
  } else if (dq_weight || dk_weight) {
    return ATTN_ERR_INVALID;  // no norm: there is no such gradient
  }
  attn::RopeBwdArgs a{q, k, q_stride, k_stride, q_weight, k_weight, eps, cos_sin, n_pos, d_rot, positions, dq_out,
                      dk_out, dq, dk, dq_stride, dk_stride, dq_weight, dk_weight, B, n, h_q, h_kv, d,
                      (flags & ATTN_ROPE_INTERLEAVED) != 0, static_cast<cudaStream_t>(stream)};
  return attn::launch_attn_norm_rope_bwd(a, workspace);
}

int attn_paged_append(const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
                      int64_t v_stride, const void* q_weight, const void* k_weight, float eps, const float* cos_sin,
                      int n_pos, int d_rot, const int32_t* positions, const int32_t* seq_ids,
                      const int32_t* page_table, int n_seqs, int max_pages, void* q_out, void* k_pages,
                      void* v_pages, int n_pages, int page_size, const float* k_scale, const float* v_scale, int T,
                      int h_q, int h_kv, int d, int flags, void* stream) {
  if (T <= 0 || T > 0x7fffff00 || h_kv <= 0 || d <= 0 || n_seqs <= 0) return ATTN_ERR_INVALID;
  if (flags & ~(ATTN_ROPE_INTERLEAVED | ATTN_CACHE_E4M3)) return ATTN_ERR_INVALID;
  if ((long long)h_kv + (q && h_q > 0 ? h_q : 0) > (1LL << 40) / d / T) return ATTN_ERR_INVALID;
  if (bad_cache(k_pages, v_pages, n_pages, page_size, max_pages, h_kv, page_table)) return ATTN_ERR_INVALID;
  if (bad_rows(k, T, k_stride, h_kv, d) || bad_rows(v, T, v_stride, h_kv, d)) return ATTN_ERR_INVALID;
  if (q) {
    if (h_q <= 0 || bad_rows(q, T, q_stride, h_q, d) || !q_out || !aligned(q_out, 16)) return ATTN_ERR_INVALID;
    if ((q_weight == nullptr) != (k_weight == nullptr)) return ATTN_ERR_INVALID;
  } else if (q_out || q_weight) {
    return ATTN_ERR_INVALID;
  }
  if (!positions || !aligned(positions, 4) || (seq_ids && !aligned(seq_ids, 4))) return ATTN_ERR_INVALID;
  if (!seq_ids && T > n_seqs) return ATTN_ERR_INVALID;
  const bool e4m3 = (flags & ATTN_CACHE_E4M3) != 0;
  if ((k_scale != nullptr) != e4m3 || (v_scale != nullptr) != e4m3) return ATTN_ERR_INVALID;
  if (e4m3 && (!aligned(k_scale, 4) || !aligned(v_scale, 4))) return ATTN_ERR_INVALID;
  const int st = check_rope(q_weight, k_weight, eps, cos_sin, n_pos, d_rot, d);
  if (st != ATTN_OK) return st;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  attn::AppendArgs a{q, k, v, q_stride, k_stride, v_stride, q_weight, k_weight, eps, cos_sin, n_pos, d_rot,
                     positions, seq_ids, page_table, n_seqs, max_pages, q_out, k_pages, v_pages, n_pages, page_size,
                     k_scale, v_scale, T, h_q, h_kv, d, (flags & ATTN_ROPE_INTERLEAVED) != 0, e4m3,
                     static_cast<cudaStream_t>(stream)};
  return attn::launch_attn_paged_append(a);
}

size_t attn_paged_decode_workspace_size(int B, int n_q, int h_q, int h_kv, int d) {
  if (B <= 0 || n_q < 1 || n_q > 16 || h_q <= 0 || h_kv <= 0 || h_q % h_kv != 0) return 0;
  if (h_q / h_kv > 8192 || (d != 64 && d != 128)) return 0;
  return attn::paged_decode_workspace_bytes(n_q, h_q / h_kv, d);
}

int attn_paged_decode(const void* q, const void* k_pages, const void* v_pages, void* out, float* lse,
                      const int32_t* page_table, const int32_t* cache_lens, int B, int n_q, int h_q, int h_kv, int d,
                      int n_pages, int page_size, int max_pages, float scale, int window, int sinks,
                      const float* k_scale, const float* v_scale, int flags, void* workspace, size_t workspace_bytes,
                      void* stream) {
  if (!q || !out || !cache_lens || !workspace) return ATTN_ERR_INVALID;
  if (B <= 0 || n_q <= 0 || h_q <= 0 || h_kv <= 0 || d <= 0 || h_q % h_kv != 0) return ATTN_ERR_INVALID;
  if (!std::isfinite(scale) || window < -1 || sinks < 0 || (flags & ~ATTN_CACHE_E4M3)) return ATTN_ERR_INVALID;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 16) || !aligned(cache_lens, 4) ||
      (lse && !aligned(lse, 4)))
    return ATTN_ERR_INVALID;
  if (bad_cache(k_pages, v_pages, n_pages, page_size, max_pages, h_kv, page_table)) return ATTN_ERR_INVALID;
  const bool e4m3 = (flags & ATTN_CACHE_E4M3) != 0;
  if ((k_scale != nullptr) != e4m3 || (v_scale != nullptr) != e4m3) return ATTN_ERR_INVALID;
  if (e4m3 && (!aligned(k_scale, 4) || !aligned(v_scale, 4))) return ATTN_ERR_INVALID;
  if (n_q > 16 || (d != 64 && d != 128) || h_q / h_kv > 8192) return ATTN_ERR_UNSUPPORTED;
  if ((long long)B * n_q > (1LL << 40) / d / h_q) return ATTN_ERR_INVALID;
  if (workspace_bytes < attn::paged_decode_workspace_bytes(n_q, h_q / h_kv, d)) return ATTN_ERR_INVALID;
  attn::PagedArgs a{q, k_pages, v_pages, out, lse, page_table, cache_lens, B, n_q, h_q, h_kv, d, n_pages, page_size,
                    max_pages, scale, window, sinks, k_scale, v_scale, e4m3, static_cast<cudaStream_t>(stream)};
  return attn::launch_attn_paged_decode(a, workspace);
}

size_t attn_packed_fwd_workspace_size(int T_q, int n_seqs, int h_q, int h_kv, int d) {
  if (check_ragged(n_seqs, T_q, 1, h_q, h_kv, d) != ATTN_OK) return 0;
  return attn::packed_fwd_workspace_bytes(T_q, n_seqs, h_q, h_kv, d);
}

int attn_packed_fwd(const void* q, const void* k, const void* v, void* out, float* lse, int64_t q_stride,
                    int64_t q_head_stride, int64_t k_stride, int64_t k_head_stride, int64_t v_stride,
                    int64_t v_head_stride, int64_t out_stride, int64_t out_head_stride, const int32_t* q_starts,
                    const int32_t* k_starts, int n_seqs, int T_q, int T_k, int h_q, int h_kv, int d, float scale,
                    int mask_mode, int window, void* workspace, size_t workspace_bytes, void* stream) {
  if (!q_starts || !aligned(q_starts, 4) || (k_starts && !aligned(k_starts, 4))) return ATTN_ERR_INVALID;
  if (!std::isfinite(scale) || scale <= 0.0f || window < -1 || (mask_mode & ~ATTN_MASK_CAUSAL)) return ATTN_ERR_INVALID;
  if (!workspace || !aligned(workspace, 256) || (lse && !aligned(lse, 4))) return ATTN_ERR_INVALID;
  const int st = check_ragged(n_seqs, T_q, T_k, h_q, h_kv, d);
  if (st != ATTN_OK) return st;
  if (bad_packed(q, T_q, h_q, d, q_stride, q_head_stride) || bad_packed(k, T_k, h_kv, d, k_stride, k_head_stride) ||
      bad_packed(v, T_k, h_kv, d, v_stride, v_head_stride) || bad_packed(out, T_q, h_q, d, out_stride, out_head_stride))
    return ATTN_ERR_INVALID;
  if (workspace_bytes < attn::packed_fwd_workspace_bytes(T_q, n_seqs, h_q, h_kv, d)) return ATTN_ERR_INVALID;
  attn::PFN_encodeTiled enc = tensor_map_encoder();
  if (!enc) return ATTN_ERR_CUDA;
  // no two positions are further apart than two arrays are long
  const int w = window < (1 << 29) ? window : (1 << 29);
  attn::PackedArgs a{q, k, v, out, lse, q_stride, q_head_stride, k_stride, k_head_stride, v_stride, v_head_stride,
                     out_stride, out_head_stride, q_starts, k_starts, n_seqs, T_q, T_k, h_q, h_kv, d, scale,
                     (mask_mode & ATTN_MASK_CAUSAL) != 0, w, 0, static_cast<cudaStream_t>(stream)};
  return attn::launch_attn_packed(a, enc, workspace);
}

size_t attn_packed_bwd_workspace_size(int T_q, int T_k, int n_seqs, int h_q, int h_kv, int d) {
  if (check_ragged(n_seqs, T_q, T_k, h_q, h_kv, d) != ATTN_OK) return 0;
  return attn::packed_bwd_workspace_bytes(T_q, T_k, n_seqs, h_q, h_kv, d);
}

int attn_packed_bwd(const void* q, const void* k, const void* v, const void* out, const void* dout, const float* lse,
                    void* dq, void* dk, void* dv, const int64_t* strides, const int32_t* q_starts,
                    const int32_t* k_starts, int n_seqs, int T_q, int T_k, int h_q, int h_kv, int d, float scale,
                    int mask_mode, int window, void* workspace, size_t workspace_bytes, void* stream) {
  if (!strides || !q_starts || !aligned(q_starts, 4) || (k_starts && !aligned(k_starts, 4))) return ATTN_ERR_INVALID;
  if (!std::isfinite(scale) || scale <= 0.0f || window < -1 || (mask_mode & ~ATTN_MASK_CAUSAL)) return ATTN_ERR_INVALID;
  if (!workspace || !aligned(workspace, 256) || !lse || !aligned(lse, 4)) return ATTN_ERR_INVALID;
  const int st = check_ragged(n_seqs, T_q, T_k, h_q, h_kv, d);
  if (st != ATTN_OK) return st;
  const void* ptrs[8] = {q, k, v, out, dout, dq, dk, dv};
  int64_t ts[8], hs[8];
  for (int i = 0; i < 8; ++i) {
    const bool keys = i == 1 || i == 2 || i >= 6;
    ts[i] = strides[2 * i];
    hs[i] = strides[2 * i + 1];
    if (bad_packed(ptrs[i], keys ? T_k : T_q, keys ? h_kv : h_q, d, ts[i], hs[i])) return ATTN_ERR_INVALID;
  }
  if (workspace_bytes < attn::packed_bwd_workspace_bytes(T_q, T_k, n_seqs, h_q, h_kv, d)) return ATTN_ERR_INVALID;
  attn::PFN_encodeTiled enc = tensor_map_encoder();
  if (!enc) return ATTN_ERR_CUDA;
  const int w = window < (1 << 29) ? window : (1 << 29);  // as in attn_packed_fwd
  attn::PackedBwdArgs a{q, k, v, out, dout, lse, dq, dk, dv, ts[0], hs[0], ts[1], hs[1], ts[2], hs[2], ts[3], hs[3],
                        ts[4], hs[4], ts[5], hs[5], ts[6], hs[6], ts[7], hs[7], q_starts, k_starts, n_seqs, T_q, T_k,
                        h_q, h_kv, d, scale, (mask_mode & ATTN_MASK_CAUSAL) != 0, w, static_cast<cudaStream_t>(stream)};
  return attn::launch_attn_packed_bwd(a, enc, workspace);
}

size_t attn_paged_chunk_workspace_size(int T, int n_seqs, int h_q, int h_kv, int d) {
  if (check_ragged(n_seqs, T, 1, h_q, h_kv, d) != ATTN_OK) return 0;
  return attn::paged_chunk_workspace_bytes(T, n_seqs, h_q, h_kv, d);
}

int attn_paged_chunk(const void* q, const void* k_pages, const void* v_pages, void* out, float* lse,
                     const int32_t* q_starts, const int32_t* page_table, const int32_t* cache_lens, int n_seqs, int T,
                     int h_q, int h_kv, int d, int n_pages, int page_size, int max_pages, float scale, int window,
                     int sinks, const float* k_scale, const float* v_scale, int flags, void* workspace,
                     size_t workspace_bytes, void* stream) {
  if (!q || !out || !aligned(q, 16) || !aligned(out, 16) || (lse && !aligned(lse, 4))) return ATTN_ERR_INVALID;
  if (!q_starts || !cache_lens || !aligned(q_starts, 4) || !aligned(cache_lens, 4)) return ATTN_ERR_INVALID;
  if (!std::isfinite(scale) || scale <= 0.0f || window < -1 || sinks < 0 || (flags & ~ATTN_CACHE_E4M3))
    return ATTN_ERR_INVALID;
  if (!workspace || !aligned(workspace, 256)) return ATTN_ERR_INVALID;
  if (bad_cache(k_pages, v_pages, n_pages, page_size, max_pages, h_kv, page_table)) return ATTN_ERR_INVALID;
  const bool e4m3 = (flags & ATTN_CACHE_E4M3) != 0;
  if ((k_scale != nullptr) != e4m3 || (v_scale != nullptr) != e4m3) return ATTN_ERR_INVALID;
  if (e4m3 && (!aligned(k_scale, 4) || !aligned(v_scale, 4))) return ATTN_ERR_INVALID;
  const int st = check_ragged(n_seqs, T, 1, h_q, h_kv, d);
  if (st != ATTN_OK) return st;
  if (workspace_bytes < attn::paged_chunk_workspace_bytes(T, n_seqs, h_q, h_kv, d)) return ATTN_ERR_INVALID;
  attn::PFN_encodeTiled enc = tensor_map_encoder();
  if (!enc) return ATTN_ERR_CUDA;
  const int w = window < (1 << 30) ? window : (1 << 30);  // no sequence is longer
  const long long row = (long long)h_q * d;
  attn::PackedArgs a{q, k_pages, v_pages, out, lse, row, d, 0, 0, 0, 0, row, d, q_starts, nullptr, n_seqs, T, 0,
                     h_q, h_kv, d, scale, 1, w, sinks, static_cast<cudaStream_t>(stream),
                     page_table, cache_lens, n_pages, page_size, max_pages, k_scale, v_scale};
  return attn::launch_attn_packed(a, enc, workspace);
}

int attn_fault_status(void* stream, int clear, uint32_t* fault_code) {
  uint32_t w = 0, wb = 0, wl = 0, ww = 0, wp = 0, wg = 0;
  const int st = attn::read_fault_word(static_cast<cudaStream_t>(stream), clear, &w);
  if (st == ATTN_ERR_CUDA || attn::read_bwd_fault_word(clear, &wb) != ATTN_OK ||
      attn::read_linear_fault_word(clear, &wl) != ATTN_OK || attn::read_weights_fault_word(clear, &ww) != ATTN_OK ||
      attn::read_packed_fault_word(clear, &wp) != ATTN_OK || attn::read_packed_bwd_fault_word(clear, &wg) != ATTN_OK)
    return ATTN_ERR_CUDA;
  w |= wb | wl | ww | wp | wg;
  if (fault_code) *fault_code = w;
  return w ? ATTN_ERR_TIMEOUT : ATTN_OK;
}

// Internal test hook, deliberately not declared in attn_gb300.h: the next plain d = 64
// attn_fwd call made on this host thread runs the fault-injection instantiation of the
// forward kernel, whose waits give up after wait_ns and whose producer never copies
// the V tile of K/V tile skip_v_tile. That call then ends through the bounded-wait
// abort path and attn_fault_status reports ATTN_ERR_TIMEOUT. wait_ns is clamped to
// [1 us, 1 s].
void attn_internal_arm_wait_timeout(unsigned long long wait_ns, int skip_v_tile) {
  if (wait_ns < 1000ull) wait_ns = 1000ull;
  if (wait_ns > 1000000000ull) wait_ns = 1000000000ull;
  attn::arm_wait_timeout_injection(wait_ns, skip_v_tile < 0 ? 0 : skip_v_tile);
}

// As attn_internal_arm_wait_timeout, for the next attn_paged_chunk call made on this host thread: in every CTA the
// copying warps of V give up before their tile v_tile, with the copies before it in flight.
void attn_internal_arm_chunk_give_up(int v_tile) { attn::arm_chunk_give_up(v_tile < 0 ? 0 : v_tile); }

const char* attn_status_string(int status) {
  switch (status) {
    case ATTN_OK: return "ATTN_OK";
    case ATTN_ERR_INVALID: return "ATTN_ERR_INVALID: invalid argument";
    case ATTN_ERR_UNSUPPORTED: return "ATTN_ERR_UNSUPPORTED: shape not supported by this path";
    case ATTN_ERR_CUDA: return "ATTN_ERR_CUDA: CUDA call failed";
    case ATTN_ERR_TIMEOUT: return "ATTN_ERR_TIMEOUT: a kernel gave up waiting on an internal barrier";
    default: return "unknown attn status";
  }
}

}  // extern "C"
