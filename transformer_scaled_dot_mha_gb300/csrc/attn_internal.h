// attn_internal.h -- declarations shared by the host API and the kernels of
// libattn_gb300.so (not part of the public C ABI; see include/attn_gb300.h).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn_gb300.h"

namespace attn {

// cuTensorMapEncodeTiled, fetched from the driver at run time (no -lcuda link).
typedef CUresult (*PFN_encodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                    const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                    CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Validated arguments of one bf16 call.
struct TcArgs {
  const void* q;
  const void* k;
  const void* v;
  void* out;
  float* lse;
  int B, H, n_q, n_k, d;
  float scale;
  int mask_mode;
  const int32_t* key_lens;
  cudaStream_t stream;
  int window;  // local-window radius (>= 0), or -1 for none
  int heads_interleaved = 0;  // 1: q, k, v, out are [B, n, H*d] instead of [B, H, n, d]
};

// Validated arguments of one attn_weights call.
struct WeightsArgs {
  const void* q;
  const void* k;
  const float* lse;
  float* w;
  int B, H, n_q, n_k, d;
  float scale;
  int mask_mode;
  const int32_t* key_lens;
  cudaStream_t stream;
};

// Validated arguments of one fp32 call.
struct F32Args {
  const float* q;
  const float* k;
  const float* v;
  float* out;
  float* lse;
  int B, H, n_q, n_k, d_k, d_v;
  float scale;
  int mask_mode;
  const int32_t* key_lens;
  cudaStream_t stream;
};

// Validated arguments of one decode step.
struct DecodeArgs {
  const void* q;
  const void* k;
  const void* v;
  void* out;
  float* lse;
  int B, H, n_q, n_max, d;
  float scale;
  const int32_t* cache_lens;
  cudaStream_t stream;
};

// Validated arguments of one gradient call (d_k == d_v == d).
struct BwdArgs {
  const void* q;
  const void* k;
  const void* v;
  const void* out;
  const void* dout;
  const float* lse;
  void* dq;
  void* dk;
  void* dv;
  int B, H, n_q, n_k, d;
  float scale;
  int mask_mode;
  const int32_t* key_lens;
  cudaStream_t stream;
  int flags = 0;    // ATTN_BWD_DETERMINISTIC
  int window = -1;  // local-window radius (>= 0), or -1 for none
};

// Validated arguments of one multi-head layer call (d_k == d_v == d).
struct MhaArgs {
  const void* x_q;
  const void* x_kv;
  const void* w_q;
  const void* b_q;
  const void* w_k;
  const void* b_k;
  const void* w_v;
  const void* b_v;
  const void* w_o;
  const void* b_o;
  void* out;
  int B, n_q, n_k, d_model, H, d;
  float scale;
  int mask_mode;
  const int32_t* key_lens;
  cudaStream_t stream;
};

// One projection Y[M, N] = X[M, K] W[K, N] (+ bias[N]), bf16, row-major, validated.
struct LinearJob {
  const void* x;
  const void* w;
  const void* bias;  // nullptr: no bias
  void* y;
  int M, N, K;
};

// Validated arguments of one attn_norm_rope call. Strides: elements between tokens.
struct RopeArgs {
  const void* q;
  const void* k;
  long long q_stride, k_stride;
  const void* q_weight;  // nullptr: no norm
  const void* k_weight;
  float eps;
  const float* cos_sin;
  int n_pos, d_rot;
  const int32_t* positions;  // nullptr: 0 .. n - 1
  void* q_out;
  void* k_out;
  int B, n, h_q, h_kv, d;
  bool pairs;  // adjacent columns turn together
  cudaStream_t stream;
};

// Validated arguments of one attn_norm_rope_bwd call.
struct RopeBwdArgs {
  const void* q;
  const void* k;
  long long q_stride, k_stride;
  const void* q_weight;
  const void* k_weight;
  float eps;
  const float* cos_sin;
  int n_pos, d_rot;
  const int32_t* positions;
  const void* dq_out;
  const void* dk_out;
  void* dq;
  void* dk;
  long long dq_stride, dk_stride;
  float* dq_weight;
  float* dk_weight;
  int B, n, h_q, h_kv, d;
  bool pairs;
  cudaStream_t stream;
};

// Validated arguments of one attn_paged_append call.
struct AppendArgs {
  const void* q;  // nullptr: keys and values only
  const void* k;
  const void* v;
  long long q_stride, k_stride, v_stride;
  const void* q_weight;
  const void* k_weight;
  float eps;
  const float* cos_sin;
  int n_pos, d_rot;
  const int32_t* positions;
  const int32_t* seq_ids;  // nullptr: token t belongs to sequence t
  const int32_t* page_table;
  int n_seqs, max_pages;
  void* q_out;
  void* k_pages;
  void* v_pages;
  int n_pages, page_size;
  const float* k_scale;
  const float* v_scale;
  int T, h_q, h_kv, d;
  bool pairs, e4m3;
  cudaStream_t stream;
};

// Validated arguments of one attn_paged_decode call.
struct PagedArgs {
  const void* q;
  const void* k_pages;
  const void* v_pages;
  void* out;
  float* lse;
  const int32_t* page_table;
  const int32_t* cache_lens;
  int B, n_q, h_q, h_kv, d, n_pages, page_size, max_pages;
  float scale;
  int window, sinks;  // window -1: none
  const float* k_scale;
  const float* v_scale;
  bool e4m3;
  cudaStream_t stream;
};

// Validated arguments of one attn_packed_fwd or attn_paged_chunk call. Strides: elements between
// tokens (ts) and heads (hs).
struct PackedArgs {
  const void* q;
  const void* k;  // pages, with a page table
  const void* v;
  void* out;
  float* lse;
  long long q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, out_ts, out_hs;
  const int32_t* q_starts;
  const int32_t* k_starts;  // nullptr: as the queries'
  int B, T_q, T_k, h_q, h_kv, d;
  float scale;
  int causal, window, sinks;  // window -1: none
  cudaStream_t stream;
  // pages
  const int32_t* page_table = nullptr;
  const int32_t* cache_lens = nullptr;
  int n_pages = 0, page_size = 0, max_pages = 0;
  const float* k_scale = nullptr;  // 8-bit pages
  const float* v_scale = nullptr;
};

// Validated arguments of one attn_packed_bwd call.
struct PackedBwdArgs {
  const void* q;
  const void* k;
  const void* v;
  const void* out;
  const void* dout;
  const float* lse;
  void* dq;
  void* dk;
  void* dv;
  long long q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, out_ts, out_hs, dout_ts, dout_hs, dq_ts, dq_hs, dk_ts, dk_hs, dv_ts, dv_hs;
  const int32_t* q_starts;
  const int32_t* k_starts;  // nullptr: as the queries'
  int B, T_q, T_k, h_q, h_kv, d;
  float scale;
  int causal, window;  // window -1: none
  cudaStream_t stream;
};

int launch_attn_tc(const TcArgs& a, PFN_encodeTiled enc);   // attn_fwd_tc.cu
int launch_attn_f32(const F32Args& a);                       // attn_fwd_f32.cu
int read_fault_word(cudaStream_t stream, int clear, uint32_t* out);  // attn_fwd_tc.cu
void arm_wait_timeout_injection(uint64_t wait_ns, int skip_v_tile);  // attn_fwd_tc.cu (tests only)
void arm_chunk_give_up(int v_tile);                                  // attn_packed.cu (tests only)
int decode_splits(int B, int H, int n_q, int n_max, int d);               // attn_decode.cu
int decode_chunk_keys(int B, int H, int n_max, int d);                    // attn_decode.cu
size_t decode_workspace_bytes(int B, int H, int n_q, int n_max, int d);  // attn_decode.cu
int launch_attn_decode(const DecodeArgs& a, void* workspace);            // attn_decode.cu
int launch_attn_decode_noalloc(const DecodeArgs& a);                     // attn_decode.cu
int read_decode_fault_word(int clear, uint32_t* out);                   // attn_decode.cu
size_t bwd_workspace_bytes(int B, int H, int n_q, int d, int flags);     // attn_bwd.cu
int launch_attn_bwd(const BwdArgs& a, PFN_encodeTiled enc, void* workspace);  // attn_bwd.cu
bool bwd_fused(int d, int flags);                                        // attn_bwd.cu
size_t bwd_host_workspace_bytes(int B, int H, int n_q, int n_k, int d, int mask_mode, int flags);  // attn_bwd_host.cu
int launch_attn_bwd_host(const BwdArgs& a, PFN_encodeTiled enc, void* workspace);                 // attn_bwd_host.cu
int read_bwd_fault_word(int clear, uint32_t* out);                       // attn_bwd.cu
int launch_linear(const LinearJob* jobs, int n_jobs, PFN_encodeTiled enc, cudaStream_t stream);  // attn_linear.cu
int read_linear_fault_word(int clear, uint32_t* out);                    // attn_linear.cu
int launch_attn_weights(const WeightsArgs& a, PFN_encodeTiled enc);     // attn_weights.cu
int read_weights_fault_word(int clear, uint32_t* out);                   // attn_weights.cu
int launch_attn_norm_rope(const RopeArgs& a);                            // attn_rope.cu
size_t norm_rope_bwd_workspace_bytes(int B, int n, int h_q, int h_kv, int d);  // attn_rope.cu
int launch_attn_norm_rope_bwd(const RopeBwdArgs& a, void* workspace);    // attn_rope.cu
int launch_attn_paged_append(const AppendArgs& a);                       // attn_rope.cu
size_t paged_decode_workspace_bytes(int n_q, int group, int d);          // attn_paged.cu
int launch_attn_paged_decode(const PagedArgs& a, void* workspace);       // attn_paged.cu
size_t packed_fwd_workspace_bytes(int T_q, int B, int h_q, int h_kv, int d);   // attn_packed.cu
size_t paged_chunk_workspace_bytes(int T_q, int B, int h_q, int h_kv, int d);  // attn_packed.cu
int launch_attn_packed(const PackedArgs& a, PFN_encodeTiled enc, void* workspace);  // attn_packed.cu
int read_packed_fault_word(int clear, uint32_t* out);                    // attn_packed.cu
size_t packed_bwd_workspace_bytes(int T_q, int T_k, int B, int h_q, int h_kv, int d);      // attn_packed_bwd.cu
int launch_attn_packed_bwd(const PackedBwdArgs& a, PFN_encodeTiled enc, void* workspace);  // attn_packed_bwd.cu
int read_packed_bwd_fault_word(int clear, uint32_t* out);                // attn_packed_bwd.cu
size_t mha_workspace_bytes(int B, int n_q, int n_k, int H, int d);         // attn_mha.cu
int launch_attn_mha(const MhaArgs& a, PFN_encodeTiled enc, void* workspace);  // attn_mha.cu
// Host-operand pipelines (attn_host.cu, attn_bwd_host.cu): chunks of the flattened
// [B, h] head range, each covered by at most three (batches x heads) rectangles.
constexpr int kMaxHostChunks = 64;
int plan_chunks(long long bh, size_t in_bytes, size_t out_bytes, double kernel_us, long long* sizes);  // attn_host.cu
// The rectangle that starts at flattened head f of [f, f1): batch b, pb whole batches of
// H heads, or (pb = 1) ph heads of batch b up to the end of the batch or of the range.
inline void head_rect(long long f, long long f1, int H, int& b, int& pb, int& ph) {
  b = (int)(f / H);
  const int h = (int)(f % H);
  if (h != 0 || f1 - f < H) {
    pb = 1;
    ph = (int)((f1 - f < H - h) ? f1 - f : H - h);
  } else {
    pb = (int)((f1 - f) / H);
    ph = H;
  }
}
size_t host_workspace_bytes(int B, int H, int n_q, int n_k, int d, int mask_mode);  // attn_host.cu
int launch_attn_host(const TcArgs& a, PFN_encodeTiled enc, void* workspace);  // attn_host.cu

}  // namespace attn
