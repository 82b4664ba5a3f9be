// attn_rope.cu -- what lies between the Q/K projections and the attention: the RMS norm of
// every query and key head, the position rotation, and (for generation) the write of the
// new keys and values into a paged cache. Entry points attn_norm_rope, attn_norm_rope_bwd
// and attn_paged_append (include/attn_gb300.h has the definitions).
//
// One head row x of d columns:
//   r = 1 / sqrt(mean(x^2) + eps),  y = x r w                      (no norm: y = x)
//   for the column pairs (a, b) of angle i:  o_a = y_a c_i - y_b s_i,  o_b = y_b c_i + y_a s_i
// and backwards, with g the gradient of o:
//   gy_a = g_a c_i + g_b s_i,  gy_b = g_b c_i - g_a s_i            (rotation by the opposite angle)
//   dw = sum over rows of gy x r,   u = gy w,   dx = r (u - x r^2 mean(u x))
//
// About ten operations per element against four (six) bytes, so every kernel here is bound
// by HBM: each row is read once and written once, all arithmetic in registers in fp32, one
// rounding at the store.
//
// Layout of the work: a row is held by d / 16 lanes, two 16-byte chunks of 8 columns each.
// With pairs (i, i + d_rot / 2) the two chunks of a lane are partners (columns 8l.. and
// 8l + d_rot / 2 ..), with adjacent pairs a partner lies in the same chunk: no rotation ever
// crosses a lane, and the norm needs one sum over 4 or 8 lanes. The lane groups of a warp
// stand on consecutive tokens and walk over `heads_per_unit` heads of one kind (query, key
// or value), so that the angles and the norm weights stay in registers, kRows rows in
// flight; consecutive tokens of one head are adjacent in the outputs ([B, h, n, d], cache
// pages), consecutive heads of one token in the inputs.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn_internal.h"
#include "ptx_sm103.cuh"

namespace attn {
namespace {

constexpr int kSMs = 152;
constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 4;          // rows in flight per lane group, forward and append
// Gradients: resident CTAs, and bytes of copies in flight per warp. More of either leaves less
// L1 for the angles (16384 tokens x 40 heads of 128: 84.8 us; 12 KB per warp 96, 4 CTAs and
// 12 KB 92.6, 4 KB 88.2).
constexpr int kBwdCtasPerSM = 3;
constexpr int kBwdBytes = 6144;

enum Kind { kQuery = 0, kKey = 1, kValue = 2 };

// The cosines and sines of one token that a lane needs.
struct Angles {
  float c[8], s[8];
};

template <int D>
struct Lanes {
  static constexpr int PER_ROW = D / 16;           // lanes that share a row
  static constexpr int GROUPS = 32 / PER_ROW;      // rows side by side in a warp
  static constexpr int TOKENS = kWarps * GROUPS;   // tokens side by side in a CTA
};

// The two 8-column chunks of lane l, and which of them are rotated.
template <int D, bool PAIRS>
__device__ __forceinline__ void chunks_of(int l, int d_rot, int& c0, int& c1, bool& rot0, bool& rot1) {
  const int nr = d_rot / 8;  // rotated chunks, an even number
  if (PAIRS) {
    c0 = l;
    c1 = l + D / 16;
    rot0 = c0 < nr;
    rot1 = c1 < nr;
  } else {
    rot0 = rot1 = l < nr / 2;
    c0 = rot0 ? l : nr + 2 * (l - nr / 2);
    c1 = rot0 ? l + nr / 2 : c0 + 1;
  }
}

__device__ __forceinline__ void load4(float* dst, const float* src) {
  const float4 v = *reinterpret_cast<const float4*>(src);
  dst[0] = v.x, dst[1] = v.y, dst[2] = v.z, dst[3] = v.w;
}

// row: the token's d_rot / 2 cosines, then its sines.
template <bool PAIRS>
__device__ __forceinline__ void load_angles(Angles& a, const float* row, int d_rot, int c0, int c1, bool rot0,
                                            bool rot1) {
  const int m = d_rot / 2;
  if (PAIRS) {
    if (rot0) load4(a.c, row + 4 * c0), load4(a.s, row + m + 4 * c0);
    if (rot1) load4(a.c + 4, row + 4 * c1), load4(a.s + 4, row + m + 4 * c1);
  } else if (rot0) {
    load4(a.c, row + 8 * c0), load4(a.c + 4, row + 8 * c0 + 4);
    load4(a.s, row + m + 8 * c0), load4(a.s + 4, row + m + 8 * c0 + 4);
  }
}

// x[0..8): chunk c0, x[8..16): chunk c1. BACK: the opposite angle.
template <bool PAIRS, bool BACK>
__device__ __forceinline__ void rotate(float (&x)[16], const Angles& a, bool rot0, bool rot1) {
  if (PAIRS) {
#pragma unroll
    for (int q = 0; q < 2; ++q)
      if (q ? rot1 : rot0)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float c = a.c[4 * q + e], s = BACK ? -a.s[4 * q + e] : a.s[4 * q + e];
          const float u = x[8 * q + 2 * e], v = x[8 * q + 2 * e + 1];
          x[8 * q + 2 * e] = u * c - v * s;
          x[8 * q + 2 * e + 1] = v * c + u * s;
        }
  } else if (rot0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float c = a.c[e], s = BACK ? -a.s[e] : a.s[e];
      const float u = x[e], v = x[8 + e];
      x[e] = u * c - v * s;
      x[8 + e] = v * c + u * s;
    }
  }
}

__device__ __forceinline__ void widen(float* x, const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = __uint_as_float(w[e] << 16);
    x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 narrow(const float* x) {
  return make_uint4(ptx::pack_bf16x2(x[0], x[1]), ptx::pack_bf16x2(x[2], x[3]), ptx::pack_bf16x2(x[4], x[5]),
                    ptx::pack_bf16x2(x[6], x[7]));
}

// Eight values divided by the head's scale, in e4m3; beyond +-448 they saturate. The
// division is the IEEE one: a value next to a rounding border goes where x / scale goes.
__device__ __forceinline__ uint2 narrow_e4m3(const float* x, float scale) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    w[e] = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(x[2 * e], scale), __fdiv_rn(x[2 * e + 1], scale)),
                                    __NV_SATFINITE, __NV_E4M3);
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// Inputs are read once: past L1, so that they do not push out the angles. (No load here uses
// the read-only path: a kernel starts before the one that writes its inputs has ended, and
// such a load could be moved ahead of the wait for it.)
__device__ __forceinline__ uint4 load_once(const uint16_t* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

// Outputs are written once and not read here: first to leave L2 (16384 tokens x 40 heads of
// 128: 52.9 us, 55.0 with plain stores).
__device__ __forceinline__ void store_once(uint16_t* p, uint4 v) { __stcs(reinterpret_cast<uint4*>(p), v); }

template <int D>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = 1; o < Lanes<D>::PER_ROW; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

struct RopeParams {
  const uint16_t* x[3];      // query, key, value rows; token t of kind z starts at x[z] + t * stride[z]
  long long stride[3];
  const uint16_t* weight[2];  // norm weights, or null
  float eps;
  const float* cos_sin;
  int n_pos, d_rot;
  const int32_t* positions;  // null: position = index in the sequence
  uint16_t* out[2];          // query and key outputs (append: queries only)
  int n, tokens;             // tokens per sequence (norm_rope), all tokens
  int heads[3];
  int units[3], heads_per_unit;
  // append
  const int32_t* seq_ids;
  const int32_t* page_table;
  int n_seqs, max_pages, n_pages, page_size;
  void* pages[3];            // [1] keys, [2] values
  const float* scale[3];     // [1], [2]: e4m3 scale per head
};

// Which kind of row and which heads a unit index stands for.
__device__ __forceinline__ int unit_kind(const RopeParams& p, int unit, int& h0, int& h1) {
  int kind = kQuery;
  if (unit >= p.units[0]) unit -= p.units[0], kind = kKey;
  if (kind == kKey && unit >= p.units[1]) unit -= p.units[1], kind = kValue;
  h0 = unit * p.heads_per_unit;
  h1 = min(h0 + p.heads_per_unit, p.heads[kind]);
  return kind;
}

// PAGED: attn_paged_append; E4M3: its cache's type. Otherwise attn_norm_rope.
template <int D, bool PAIRS, bool PAGED, bool E4M3>
__global__ void __launch_bounds__(kThreads) attn_rope_kernel(const RopeParams p) {
  using L = Lanes<D>;
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int l = lane % L::PER_ROW;
  const int n_units = p.units[0] + p.units[1] + p.units[2];
  int h0, h1;
  const int kind = unit_kind(p, blockIdx.x % n_units, h0, h1);
  const long long t0 = (long long)(blockIdx.x / n_units) * L::TOKENS + warp * L::GROUPS;
  if (t0 >= p.tokens) return;  // whole warps: the sums below are over all 32 lanes
  const bool there = t0 + lane / L::PER_ROW < p.tokens;
  const int t = there ? (int)t0 + lane / L::PER_ROW : p.tokens - 1;
  const int b = PAGED ? 0 : t / p.n, i = PAGED ? t : t - b * p.n;

  // where the token stands; a position without a table row makes it a padding token
  const int pos = p.positions ? p.positions[t] : i;
  bool valid = there && pos >= 0 && (p.d_rot == 0 || pos < p.n_pos);
  long long page_row = 0;  // cache row of head 0
  if (PAGED) {
    const int seq = p.seq_ids ? p.seq_ids[t] : t;
    const int slot = max(pos, 0) / p.page_size;
    valid = valid && seq >= 0 && seq < p.n_seqs && slot < p.max_pages;
    const int page = valid ? p.page_table[(long long)seq * p.max_pages + slot] : -1;
    valid = valid && page >= 0 && page < p.n_pages;
    page_row = (long long)page * p.heads[kKey] * p.page_size + (pos - slot * p.page_size);
  }

  int c0, c1;
  bool rot0, rot1;
  chunks_of<D, PAIRS>(l, p.d_rot, c0, c1, rot0, rot1);
  const bool normed = kind != kValue && p.weight[kind & 1] != nullptr;
  uint4 w0{}, w1{};
  Angles a;
  if (kind == kValue) {
    rot0 = rot1 = false;
  } else {
    if (normed) {
      w0 = *reinterpret_cast<const uint4*>(p.weight[kind & 1] + 8 * c0);
      w1 = *reinterpret_cast<const uint4*>(p.weight[kind & 1] + 8 * c1);
    }
    if (valid) load_angles<PAIRS>(a, p.cos_sin + (long long)pos * p.d_rot, p.d_rot, c0, c1, rot0, rot1);
  }
  const uint16_t* src = p.x[kind] + t * p.stride[kind];

  for (int h = h0; h < h1; h += kRows) {
    uint4 v[kRows][2];
#pragma unroll
    for (int u = 0; u < kRows; ++u)
      if (h + u < h1 && valid) {
        v[u][0] = load_once(src + (h + u) * D + 8 * c0);
        v[u][1] = load_once(src + (h + u) * D + 8 * c1);
      } else {
        v[u][0] = v[u][1] = make_uint4(0, 0, 0, 0);
      }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      if (h + u >= h1) break;
      float x[16];
      widen(x, v[u][0]);
      widen(x + 8, v[u][1]);
      if (normed) {
        float ss = 0.0f;
#pragma unroll
        for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
        const float r = rsqrtf(row_sum<D>(ss) * (1.0f / D) + p.eps);
        float w[16];
        widen(w, w0);
        widen(w + 8, w1);
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = x[e] * r * w[e];
      }
      if (valid) rotate<PAIRS, false>(x, a, rot0, rot1);
      if (!PAGED) {
        if (there) {
          uint16_t* dst = p.out[kind & 1] + (((long long)b * p.heads[kind] + h + u) * p.n + i) * D;
          const uint4 zero = make_uint4(0, 0, 0, 0);  // a padding token
          store_once(dst + 8 * c0, valid ? narrow(x) : zero);
          store_once(dst + 8 * c1, valid ? narrow(x + 8) : zero);
        }
      } else if (valid) {
        if (kind == kQuery) {
          uint16_t* dst = p.out[0] + ((long long)t * p.heads[0] + h + u) * D;
          store_once(dst + 8 * c0, narrow(x));
          store_once(dst + 8 * c1, narrow(x + 8));
        } else {
          const long long at = (page_row + (long long)(h + u) * p.page_size) * D;
          if (E4M3) {
            const float scale = p.scale[kind][h + u];
            uint8_t* dst = static_cast<uint8_t*>(p.pages[kind]) + at;
            __stcs(reinterpret_cast<uint2*>(dst + 8 * c0), narrow_e4m3(x, scale));
            __stcs(reinterpret_cast<uint2*>(dst + 8 * c1), narrow_e4m3(x + 8, scale));
          } else {
            uint16_t* dst = static_cast<uint16_t*>(p.pages[kind]) + at;
            store_once(dst + 8 * c0, narrow(x));
            store_once(dst + 8 * c1, narrow(x + 8));
          }
        }
      }
    }
  }
}

struct RopeBwdParams {
  const uint16_t* x[2];
  const uint16_t* g[2];  // gradients of the outputs, [B, h, n, d]
  uint16_t* dx[2];
  long long stride[2], dstride[2];
  const uint16_t* weight[2];
  float eps;
  const float* cos_sin;
  int n_pos, d_rot;
  const int32_t* positions;
  int n, tokens;
  int heads[2];
  int ctas[2];      // the first ctas[0] CTAs take the queries, the others the keys
  int items[2];     // per warp
  float* partials;  // [ctas[0] + ctas[1]][d], sums of the weights' gradients
  float* dw[2];
};

__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "r"(addr)
               : "memory");
  return r;
}

// An item is one head of the tokens side by side in a warp (32 * 16 / d rows). The items of a
// kind, heads first, form one list cut into equal runs, a warp each; a warp keeps STAGES items'
// rows (x and g, whole rows by cp.async: its own ring, its own waits) in flight, so that HBM
// does not wait for the arithmetic, and its share of the weight's gradient in registers. The
// shares go to the workspace and are summed in a fixed order by attn_rope_dw_kernel: no
// atomics, the same bits on every run.
template <int D, bool PAIRS, bool NORM>
__global__ void __launch_bounds__(kThreads, kBwdCtasPerSM) attn_rope_bwd_kernel(const RopeBwdParams p) {
  using L = Lanes<D>;
  constexpr int PIECES = D / 8;              // 16-byte pieces of a row
  constexpr int COPIES = L::GROUPS * PIECES / 32;  // per operand and item
  constexpr int ITEM = (NORM ? 2 : 1) * 1024;      // bytes of an item: g, then x
  constexpr int STAGES = kBwdBytes / ITEM;
  static_assert(L::GROUPS * D * 2 == 1024, "an item's rows");
  __shared__ __align__(128) uint8_t ring_sh[kWarps][STAGES * ITEM];
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int l = lane % L::PER_ROW, side = lane / L::PER_ROW;
  const int kind = (int)blockIdx.x >= p.ctas[0];
  const int cta = blockIdx.x - (kind ? p.ctas[0] : 0);
  const int H = p.heads[kind];
  const long long total = ((long long)p.tokens + L::GROUPS - 1) / L::GROUPS * H;
  const long long begin = ((long long)cta * kWarps + warp) * p.items[kind];
  const int count = (int)max(0ll, min((long long)p.items[kind], total - begin));
  const uint32_t ring = ptx::smem_u32(ring_sh[warp]);
  int c0, c1;
  bool rot0, rot1;
  chunks_of<D, PAIRS>(l, p.d_rot, c0, c1, rot0, rot1);
  uint4 w0{}, w1{};
  if (NORM) {
    w0 = *reinterpret_cast<const uint4*>(p.weight[kind] + 8 * c0);
    w1 = *reinterpret_cast<const uint4*>(p.weight[kind] + 8 * c1);
  }
  float dw[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) dw[e] = 0.0f;

  // the requests' place in the list, and where their rows start: copy y takes piece
  // lane % PIECES of row y * 32 / PIECES + lane / PIECES
  int group_a = (int)(begin / H), h_a = (int)(begin - (long long)group_a * H);
  const uint16_t* g_src[COPIES];
  const uint16_t* x_src[COPIES];
  bool row_there[COPIES];
  auto rows_of = [&]() {
#pragma unroll
    for (int y = 0; y < COPIES; ++y) {
      const long long t = (long long)group_a * L::GROUPS + y * (32 / PIECES) + lane / PIECES;
      row_there[y] = t < p.tokens;
      const int tt = row_there[y] ? (int)t : 0, b = tt / p.n, i = tt - b * p.n;
      g_src[y] = p.g[kind] + ((long long)b * H * p.n + i) * D + 8 * (lane % PIECES);
      x_src[y] = p.x[kind] + tt * p.stride[kind] + 8 * (lane % PIECES);
    }
  };
  if (count > 0) rows_of();
  auto request = [&](int stage) {
    const uint32_t at = ring + stage * ITEM + 16 * lane;
#pragma unroll
    for (int y = 0; y < COPIES; ++y) {
      copy_async(at + 512 * y, g_src[y] + (long long)h_a * p.n * D, row_there[y]);
      if (NORM) copy_async(at + 1024 + 512 * y, x_src[y] + h_a * D, row_there[y]);
    }
    if (++h_a == H) {
      h_a = 0;
      ++group_a;
      rows_of();
    }
  };

  int group = group_a, h = h_a, stage = 0;
  bool fresh = true, there = false, valid = false;
  Angles a;
  uint16_t* dst = nullptr;
  // the steps below 0 fill the ring
  for (int i = -STAGES; i < count; ++i) {
    if (i >= 0) {
      if (fresh) {  // the next tokens
        const long long t_ = (long long)group * L::GROUPS + side;
        there = t_ < p.tokens;
        const int t = there ? (int)t_ : p.tokens - 1;
        const int pos = p.positions ? p.positions[t] : t % p.n;
        valid = there && pos >= 0 && (p.d_rot == 0 || pos < p.n_pos);
        if (valid) load_angles<PAIRS>(a, p.cos_sin + (long long)pos * p.d_rot, p.d_rot, c0, c1, rot0, rot1);
        dst = p.dx[kind] + t * p.dstride[kind];
        fresh = false;
      }
      asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
      __syncwarp();
      const uint32_t at = ring + stage * ITEM + side * (2 * D);
      float gy[16];
      widen(gy, lds128(at + 16 * c0));
      widen(gy + 8, lds128(at + 16 * c1));
      if (valid) rotate<PAIRS, true>(gy, a, rot0, rot1);
      if (NORM) {
        float x[16], w[16];
        widen(x, lds128(at + 1024 + 16 * c0));
        widen(x + 8, lds128(at + 1024 + 16 * c1));
        widen(w, w0);
        widen(w + 8, w1);
        float ss = 0.0f, dot = 0.0f;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          ss = fmaf(x[e], x[e], ss);
          dot = fmaf(gy[e] * w[e], x[e], dot);
        }
        ss = row_sum<D>(ss);
        dot = row_sum<D>(dot);
        const float r = rsqrtf(ss * (1.0f / D) + p.eps);
        const float back = r * r * dot * (1.0f / D);
        if (valid)
#pragma unroll
          for (int e = 0; e < 16; ++e) dw[e] = fmaf(gy[e], x[e] * r, dw[e]);
#pragma unroll
        for (int e = 0; e < 16; ++e) gy[e] = r * (gy[e] * w[e] - x[e] * back);
      }
      if (there) {  // a padding token's gradient is zero
        const uint4 zero = make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4*>(dst + h * D + 8 * c0) = valid ? narrow(gy) : zero;
        *reinterpret_cast<uint4*>(dst + h * D + 8 * c1) = valid ? narrow(gy + 8) : zero;
      }
      if (++h == H) {
        h = 0;
        ++group;
        fresh = true;
      }
      __syncwarp();  // the stage is read
    }
    if (i + STAGES < count) request(stage);
    asm volatile("cp.async.commit_group;" ::: "memory");
    stage = stage + 1 < STAGES ? stage + 1 : 0;
  }

  if (NORM) {
    float(*part)[D] = reinterpret_cast<float(*)[D]>(ring_sh);  // every copy has landed and been read
    __syncthreads();
#pragma unroll
    for (int o = L::PER_ROW; o < 32; o <<= 1)
#pragma unroll
      for (int e = 0; e < 16; ++e) dw[e] += __shfl_xor_sync(0xffffffffu, dw[e], o);
    if (lane < L::PER_ROW)
#pragma unroll
      for (int e = 0; e < 16; ++e) part[warp][(e < 8 ? 8 * c0 : 8 * c1) + (e & 7)] = dw[e];
    __syncthreads();
    for (int x = threadIdx.x; x < D; x += kThreads) {
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) sum += part[w][x];
      p.partials[(long long)blockIdx.x * D + x] = sum;
    }
  }
}

// Sums the CTAs' shares: block (column group of 32, kind), 32 columns x 32 shares at a time.
template <int D>
__global__ void __launch_bounds__(1024) attn_rope_dw_kernel(const RopeBwdParams p) {
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int kind = blockIdx.y, col = blockIdx.x * 32 + threadIdx.x;
  const int first = kind ? p.ctas[0] : 0, count = p.ctas[kind];
  float sum = 0.0f;
  constexpr int kEach = (kBwdCtasPerSM * kSMs + 31) / 32 + 1;  // shares per thread at most: all loads at once
  float x[kEach];
#pragma unroll
  for (int s = 0; s < kEach; ++s) {
    const int at = threadIdx.y + 32 * s;
    x[s] = at < count ? p.partials[(long long)(first + at) * D + col] : 0.0f;
  }
#pragma unroll
  for (int s = 0; s < kEach; ++s) sum += x[s];
  __shared__ float part[32][33];
  part[threadIdx.y][threadIdx.x] = sum;
  __syncthreads();
  if (threadIdx.y == 0) {
    float total = 0.0f;
#pragma unroll
    for (int s = 0; s < 32; ++s) total += part[s][threadIdx.x];
    p.dw[kind][col] = total;
  }
}

template <typename... KArgs, typename... Args>
int launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

// Heads a lane group walks over: as many, up to 8, as leave two CTAs per SM. More heads per
// group read the token's angles fewer times; fewer give short batches more CTAs. (8192 tokens x
// 16 heads of 64: 8.1 us, 8.8 from eight CTAs per SM, 12.2 from sixteen; 16384 x 40 heads of
// 128 with plain stores: 55.0 with up to 8 heads, 59.9 with 4, 59.6 with 32.)
int heads_per_unit(long long token_tiles, const int* heads, int kinds) {
  for (int hp = 8; hp > 1; hp /= 2) {
    long long units = 0;
    for (int z = 0; z < kinds; ++z) units += (heads[z] + hp - 1) / hp;
    if (token_tiles * units >= 2LL * kSMs) return hp;
  }
  return 1;
}

int tokens_per_tile(int d) { return d == 64 ? Lanes<64>::TOKENS : Lanes<128>::TOKENS; }

int launch_rope(RopeParams& p, int d, bool pairs, bool paged, bool e4m3, cudaStream_t stream) {
  const long long tiles = ((long long)p.tokens + tokens_per_tile(d) - 1) / tokens_per_tile(d);
  p.heads_per_unit = heads_per_unit(tiles, p.heads, 3);
  long long units = 0;
  for (int z = 0; z < 3; ++z) units += p.units[z] = (p.heads[z] + p.heads_per_unit - 1) / p.heads_per_unit;
  if (tiles * units > 0x7fffffffLL) return ATTN_ERR_INVALID;
  void (*kernel)(const RopeParams) = nullptr;
#define ATTN_PICK(D_, P_)                                            \
  if (d == D_ && pairs == P_)                                        \
    kernel = !paged ? attn_rope_kernel<D_, P_, false, false>         \
             : e4m3 ? attn_rope_kernel<D_, P_, true, true>           \
                    : attn_rope_kernel<D_, P_, true, false>;
  ATTN_PICK(64, false)
  ATTN_PICK(64, true)
  ATTN_PICK(128, false)
  ATTN_PICK(128, true)
#undef ATTN_PICK
  return launch_pdl(kernel, dim3((unsigned)(tiles * units)), dim3(kThreads), stream, p);
}

// CTAs of the gradient kernel: the device filled, shared out by the kinds' heads; and the
// items per warp. False where those are too many to count.
bool bwd_grid(long long tokens, int h_q, int h_kv, int d, int* ctas, int* items) {
  const int side = 512 / d;  // tokens of an item
  const int heads[2] = {h_q, h_kv};
  const long long most = (long long)kBwdCtasPerSM * kSMs, all = (long long)h_q + h_kv;
  long long shares[2];  // together no more CTAs than are resident
  shares[0] = (most * h_q + all / 2) / all;
  shares[0] = shares[0] < 1 ? 1 : shares[0] > most - 1 ? most - 1 : shares[0];
  shares[1] = most - shares[0];
  for (int z = 0; z < 2; ++z) {
    const long long total = (tokens + side - 1) / side * heads[z], share = shares[z];
    const long long need = (total + kWarps - 1) / kWarps;
    ctas[z] = (int)(need < share ? need : share);
    const long long per = (total + (long long)ctas[z] * kWarps - 1) / ((long long)ctas[z] * kWarps);
    if (per > 0x7fffff00LL) return false;
    items[z] = (int)per;
  }
  return true;
}

}  // namespace

int launch_attn_norm_rope(const RopeArgs& a) {
  RopeParams p = {};
  p.x[0] = static_cast<const uint16_t*>(a.q), p.x[1] = static_cast<const uint16_t*>(a.k);
  p.stride[0] = a.q_stride, p.stride[1] = a.k_stride;
  p.weight[0] = static_cast<const uint16_t*>(a.q_weight), p.weight[1] = static_cast<const uint16_t*>(a.k_weight);
  p.eps = a.eps;
  p.cos_sin = a.cos_sin, p.n_pos = a.n_pos, p.d_rot = a.d_rot, p.positions = a.positions;
  p.out[0] = static_cast<uint16_t*>(a.q_out), p.out[1] = static_cast<uint16_t*>(a.k_out);
  p.n = a.n, p.tokens = a.B * a.n;
  p.heads[0] = a.h_q, p.heads[1] = a.h_kv, p.heads[2] = 0;
  return launch_rope(p, a.d, a.pairs, false, false, a.stream);
}

int launch_attn_paged_append(const AppendArgs& a) {
  RopeParams p = {};
  p.x[0] = static_cast<const uint16_t*>(a.q), p.x[1] = static_cast<const uint16_t*>(a.k);
  p.x[2] = static_cast<const uint16_t*>(a.v);
  p.stride[0] = a.q_stride, p.stride[1] = a.k_stride, p.stride[2] = a.v_stride;
  p.weight[0] = static_cast<const uint16_t*>(a.q_weight), p.weight[1] = static_cast<const uint16_t*>(a.k_weight);
  p.eps = a.eps;
  p.cos_sin = a.cos_sin, p.n_pos = a.n_pos, p.d_rot = a.d_rot, p.positions = a.positions;
  p.out[0] = static_cast<uint16_t*>(a.q_out);
  p.n = a.T, p.tokens = a.T;
  p.heads[0] = a.q ? a.h_q : 0, p.heads[1] = a.h_kv, p.heads[2] = a.h_kv;
  p.seq_ids = a.seq_ids, p.page_table = a.page_table;
  p.n_seqs = a.n_seqs, p.max_pages = a.max_pages, p.n_pages = a.n_pages, p.page_size = a.page_size;
  p.pages[1] = a.k_pages, p.pages[2] = a.v_pages;
  p.scale[1] = a.k_scale, p.scale[2] = a.v_scale;
  return launch_rope(p, a.d, a.pairs, true, a.e4m3, a.stream);
}

size_t norm_rope_bwd_workspace_bytes(int B, int n, int h_q, int h_kv, int d) {
  int ctas[2], items[2];
  bwd_grid((long long)B * n, h_q, h_kv, d, ctas, items);
  return (size_t)(ctas[0] + ctas[1]) * d * sizeof(float);
}

int launch_attn_norm_rope_bwd(const RopeBwdArgs& a, void* workspace) {
  RopeBwdParams p = {};
  p.x[0] = static_cast<const uint16_t*>(a.q), p.x[1] = static_cast<const uint16_t*>(a.k);
  p.g[0] = static_cast<const uint16_t*>(a.dq_out), p.g[1] = static_cast<const uint16_t*>(a.dk_out);
  p.dx[0] = static_cast<uint16_t*>(a.dq), p.dx[1] = static_cast<uint16_t*>(a.dk);
  p.stride[0] = a.q_stride, p.stride[1] = a.k_stride;
  p.dstride[0] = a.dq_stride, p.dstride[1] = a.dk_stride;
  p.weight[0] = static_cast<const uint16_t*>(a.q_weight), p.weight[1] = static_cast<const uint16_t*>(a.k_weight);
  p.eps = a.eps;
  p.cos_sin = a.cos_sin, p.n_pos = a.n_pos, p.d_rot = a.d_rot, p.positions = a.positions;
  p.n = a.n, p.tokens = a.B * a.n;
  p.heads[0] = a.h_q, p.heads[1] = a.h_kv;
  if (!bwd_grid(p.tokens, a.h_q, a.h_kv, a.d, p.ctas, p.items)) return ATTN_ERR_INVALID;
  p.partials = static_cast<float*>(workspace);
  p.dw[0] = a.dq_weight, p.dw[1] = a.dk_weight;
  const bool norm = a.q_weight != nullptr;
  void (*kernel)(const RopeBwdParams) = nullptr;
#define ATTN_PICK(D_, P_)         \
  if (a.d == D_ && a.pairs == P_) \
    kernel = norm ? attn_rope_bwd_kernel<D_, P_, true> : attn_rope_bwd_kernel<D_, P_, false>;
  ATTN_PICK(64, false)
  ATTN_PICK(64, true)
  ATTN_PICK(128, false)
  ATTN_PICK(128, true)
#undef ATTN_PICK
  int st = launch_pdl(kernel, dim3((unsigned)(p.ctas[0] + p.ctas[1])), dim3(kThreads), a.stream, p);
  if (st != ATTN_OK || !norm) return st;
  return launch_pdl(a.d == 64 ? attn_rope_dw_kernel<64> : attn_rope_dw_kernel<128>, dim3(a.d / 32, 2), dim3(32, 32),
                    a.stream, p);
}

}  // namespace attn
