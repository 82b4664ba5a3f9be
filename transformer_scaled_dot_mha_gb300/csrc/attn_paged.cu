// attn_paged.cu -- attn_paged_decode: the newest n_q (1..16) tokens of every sequence attend
// over a paged key/value cache. Shared key/value heads (query head h uses key/value head
// h / group), an optional sliding window whose first `sinks` tokens stay visible, pages in
// bf16 or e4m3 (value = stored value * the head's scale).
//
// For row r (token i, query head) of a sequence of `len` tokens, pos = len - n_q + i:
//   legal keys: j <= pos and (no window, or j >= pos - window, or j < sinks)
//   out = sum_j p_j v_j / sum_j p_j,   p_j = 2^(s_j - m),  s_j = scale log2(e) q . k_j,  m = max_j s_j
//
// What bounds it: each visible K and V row is read once, 4 (8-bit: 2) bytes per column pair
// against 4 x group operations, so HBM. The arithmetic has only to stay out of the way,
// which CUDA cores cannot at group 8 (54 TFLOP/s at the full HBM rate): both products run
// on the warp-level matrix instruction m16n8k16, whose operands are registers. A tcgen05
// MMA would need 128 rows and its operands in shared memory; one key/value head offers 1 to
// 16 rows, and the cache would pass through shared memory for nothing.
//
// The products are formed transposed, S^T = K Q^T and O^T = V^T P^T, so that the keys (then
// the columns) are the 16 rows of an MMA and the query rows its 8 columns (NT column tiles
// for up to 8 NT rows):
//   * K fragments come straight from global memory: the order of the contracted columns is
//     free, so a lane takes 16-byte pieces of "its" key (row lane / 4) and Q is loaded in
//     the same order;
//   * S^T leaves a lane with (key lane / 4, rows 2 (lane % 4) and + 1); a register
//     transpose (movmatrix) turns the rounded P^T into the second product's operand;
//   * V fragments too come straight from global memory: a lane holds 16 bytes of columns
//     (all 8 or 16 of "its" columns) of each of four keys and pairs up the keys by byte
//     permutes; the order of the columns is free again.
// No shared memory, barrier or wait in the stream: K of the next tile is requested when the
// scores are done with this one's registers, V when the second product is.
//
// Work split: the tiles (KT keys) of all (sequence, key/value head) pairs form one list,
// cut into equal parts, one per resident CTA, by the lengths on the device -- ragged
// batches and capacities far above the lengths cost nothing. A CTA's four warps take a
// pair's tiles in turn and join their (m, l, O) through shared memory. A pair that lies
// within one CTA's part is finished there; of one that does not, every part leaves (m, l, O)
// in the workspace and attn_paged_merge_kernel joins them. When no sequence can be longer
// than a few tiles, each pair gets a CTA of its own and there is no second launch.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "attn_internal.h"
#include "ptx_sm103.cuh"

namespace attn {
namespace {

constexpr int kSMs = 152;
constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCtasPerSM = 4;
constexpr int kMinTiles = 2 * kWarps;      // tiles per CTA, at least: two per warp
constexpr int kWholeTiles = 8 * kWarps;    // up to here a pair is one CTA's
constexpr uint32_t kAll = 0xffffffffu;

// D columns, NT tiles of 8 query rows, FP8: e4m3 pages.
template <int D, int NT, bool FP8>
struct Cfg {
  static constexpr int KT = (D == 128 && !FP8) ? 16 : 32;  // keys per warp tile: 32 registers of K, 32 of V at most
  static constexpr int KB = KT / 16;                       // 16-key blocks
  static constexpr int KC = FP8 ? D / 64 : D / 32;         // 16-byte pieces of a key per lane
  static constexpr int VW = FP8 ? D / 32 : D / 16;         // 32-bit words of a value row per lane
  static constexpr int S = D / 16;                         // MMA steps over the columns; column tiles of O
  static constexpr int ROWS = 8 * NT;
  static constexpr int CTAS_PER_SM = NT == 1 ? (D == 64 ? 4 : 3) : (D == 64 ? 3 : 2);
  static constexpr int O_PITCH = D + 4;  // floats
};

struct PagedParams {
  const uint16_t* q;
  const void* k;
  const void* v;
  uint16_t* out;
  float* lse;
  const int32_t* page_table;
  const int32_t* cache_lens;
  const float* k_scale;
  const float* v_scale;
  float* ws_o;   // [2 * CTAs][ROWS][D]: slot 2 c for the pair CTA c's part begins in, 2 c + 1 for the one it ends in
  float* ws_ml;  // [2 * CTAs][ROWS][2]
  int B, n_q, h_q, h_kv, group, rows, m_tiles;  // rows = n_q * group
  int n_pages, page_size, page_shift, max_pages, max_len;  // page_shift < 0: not a power of two
  int window, sinks;
  int whole;  // one CTA per pair, no split
  float scale_log2;
};

// ---------------------------------------------------------------- instructions
template <bool FP8>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (FP8)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 8 x 8 transpose of 16-bit values, two per lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two e4m3 values (the low or high half of x) as f16: exact.
__device__ __forceinline__ uint32_t e4m3_f16x2(uint32_t x, bool high) {
  uint32_t r;
  const uint16_t h = (uint16_t)(high ? x >> 16 : x);
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(h));
  return r;
}
__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}
__device__ __forceinline__ uint2 load8(const void* p) {
  uint2 r;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
  return r;
}

// ---------------------------------------------------------------- ranges
// The visible keys of a sequence, numbered 0 .. count - 1: the first `head` are keys 0 ..
// head - 1 (sinks below the window), number x >= head is key x + skip.
struct Visible {
  int len, head, skip, count;
  __device__ int key(int x) const { return x < head ? x : x + skip; }
};

__device__ __forceinline__ Visible visible_of(const PagedParams& p, int b) {
  Visible v;
  v.len = min(max(__ldg(p.cache_lens + b), 0), p.max_len);
  // the first token that stands in the sequence sees furthest back
  const int pos0 = max(v.len - p.n_q, 0);
  const int low = p.window < 0 ? 0 : max(pos0 - p.window, 0);
  v.head = min(p.sinks, low);
  v.skip = low - v.head;
  v.count = v.len - v.skip;
  return v;
}

template <int KT>
__device__ __forceinline__ int tiles_of(const PagedParams& p, int b) {
  return (visible_of(p, b).count + KT - 1) / KT;
}

// Where the list of tiles stands. Sequence b holds pairs (head, row tile) one after the
// other, each of tiles_of(b) tiles.
struct Split {
  long long total;  // tiles of all pairs
  int ctas;         // parts: cta c has tiles [total c / ctas, total (c + 1) / ctas)
  __device__ long long first(long long c) const { return total * c / ctas; }
};

// Sums tiles_of over the sequences with the whole CTA: thread t takes `per` sequences in a
// row; sums[t] = tiles before them. All threads get the split.
template <int KT>
__device__ __forceinline__ Split make_split(const PagedParams& p, long long (&sums)[kThreads + 1], int max_ctas,
                                            int& per) {
  __shared__ long long warp_sum[kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  per = (p.B + kThreads - 1) / kThreads;
  long long mine = 0;
  for (int x = 0; x < per; ++x) {
    const long long b = (long long)tid * per + x;
    if (b < p.B) mine += tiles_of<KT>(p, (int)b);
  }
  long long x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(kAll, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  for (int w = 0; w < warp; ++w) x += warp_sum[w];
  sums[tid] = x - mine;
  if (tid == kThreads - 1) sums[kThreads] = x;
  __syncthreads();
  const long long pairs = (long long)p.h_kv * p.m_tiles;
  Split s;
  s.total = sums[kThreads] * pairs;
  s.ctas = (int)max(1ll, min((long long)max_ctas, s.total / kMinTiles));
  return s;
}

// The sequence that holds tile x (of the list without heads: x < sums[kThreads]), and the
// tiles before it.
template <int KT>
__device__ __forceinline__ int find_sequence(const PagedParams& p, const long long (&sums)[kThreads + 1], int per,
                                             long long x, long long& before) {
  int lo = 0, hi = kThreads - 1;  // the last t with sums[t] <= x
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (sums[mid] <= x)
      lo = mid;
    else
      hi = mid - 1;
  }
  before = sums[lo];
  int b = lo * per;
  for (int n = tiles_of<KT>(p, b); b + 1 < p.B && before + n <= x; n = tiles_of<KT>(p, b)) before += n, ++b;
  return b;
}

// ---------------------------------------------------------------- one pair's tiles
template <int D, int NT, bool FP8>
struct Shared {
  using C = Cfg<D, NT, FP8>;
  float o[kWarps][C::ROWS][C::O_PITCH];
  float m[kWarps][C::ROWS], l[kWarps][C::ROWS];
};

// Cache row of key number x, -1 where there is none.
__device__ __forceinline__ int cache_row(const PagedParams& p, const Visible& vis, const int32_t* pages, int head,
                                         int x) {
  if (x >= vis.count) return -1;
  const int j = vis.key(x);
  const int slot = p.page_shift >= 0 ? j >> p.page_shift : j / p.page_size;
  const int page = __ldg(pages + slot);
  if (page < 0 || page >= p.n_pages) return -1;  // names no page: its keys count as illegal
  return (page * p.h_kv + head) * p.page_size + (j - slot * p.page_size);
}

// Writes four columns of a finished row.
template <int D>
__device__ __forceinline__ void finish(const PagedParams& p, int b, int head, int row, int col, float4 o, float M,
                                       float L) {
  const int i = row / p.group;
  const long long at = ((long long)b * p.n_q + i) * p.h_q + head * p.group + (row - i * p.group);
  const bool none = M == -INFINITY && L == 0.0f;  // no legal key
  const float inv = none ? 0.0f : 1.0f / L;
  *reinterpret_cast<uint2*>(p.out + at * D + col) =
      make_uint2(ptx::pack_bf16x2(o.x * inv, o.y * inv), ptx::pack_bf16x2(o.z * inv, o.w * inv));
  if (p.lse && col == 0) p.lse[at] = none ? -INFINITY : (M + log2f(L)) * 0.69314718055994530942f;
}

// Tiles [t0, t1) of (sequence b, key/value head, row tile mt), joined over the CTA's warps.
// slot < 0: the pair is complete, write out and lse; else leave (m, l, O) in that slot.
template <int D, int NT, bool FP8>
__device__ __forceinline__ void attend(const PagedParams& p, Shared<D, NT, FP8>& sh, int b, int head, int mt, int t0,
                                       int t1, long long slot) {
  using C = Cfg<D, NT, FP8>;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const Visible vis = visible_of(p, b);
  const int32_t* pages = p.page_table + (long long)b * p.max_pages;
  const int rows = min(p.rows - mt * C::ROWS, C::ROWS);
  constexpr int kElem = FP8 ? 1 : 2;
  const uint8_t* kp = static_cast<const uint8_t*>(p.k) + 16 * t;
  const uint8_t* vp = static_cast<const uint8_t*>(p.v) + (FP8 ? D / 8 : 16) * g;

  // ---- K and V of a tile; rows_l: the lanes' cache rows
  uint4 kr[C::KB][2][C::KC];
  uint32_t vr[C::KB][4][C::VW];
  auto load_k = [&](int rows_l) {
#pragma unroll
    for (int kb = 0; kb < C::KB; ++kb)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int row = __shfl_sync(kAll, rows_l, kb * 16 + hf * 8 + g);
        const uint8_t* src = kp + (long long)row * (D * kElem);
#pragma unroll
        for (int c = 0; c < C::KC; ++c) kr[kb][hf][c] = row >= 0 ? load16(src + 64 * c) : make_uint4(0, 0, 0, 0);
      }
  };
  auto load_v = [&](int rows_l) {  // keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9 of each block
#pragma unroll
    for (int kb = 0; kb < C::KB; ++kb)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int row = __shfl_sync(kAll, rows_l, kb * 16 + (x >> 1) * 8 + 2 * t + (x & 1));
        const uint8_t* src = vp + (long long)row * (D * kElem);
        if (C::VW == 2) {
          const uint2 w = row >= 0 ? load8(src) : make_uint2(0, 0);
          vr[kb][x][0] = w.x, vr[kb][x][1] = w.y;
        } else {
#pragma unroll
          for (int c = 0; c < C::VW / 4; ++c) {
            const uint4 w = row >= 0 ? load16(src + 128 * c) : make_uint4(0, 0, 0, 0);
            vr[kb][x][4 * c] = w.x, vr[kb][x][4 * c + 1] = w.y, vr[kb][x][4 * c + 2] = w.z, vr[kb][x][4 * c + 3] = w.w;
          }
        }
      }
  };
  auto rows_of = [&](int tile) {
    return tile < t1 && lane < C::KT ? cache_row(p, vis, pages, head, tile * C::KT + lane) : -1;
  };

  int tile = t0 + warp;
  int row_now = rows_of(tile), row_next = rows_of(tile + kWarps);
  if (tile < t1) {
    load_k(row_now);
    load_v(row_now);
  }

  // ---- queries: B fragments in the order of the K pieces, zeros past the last row
  uint32_t qf[NT][C::S][2];
  float factor[NT][2];  // of rows 2 t, 2 t + 1: scores in log2 units = factor * accumulator
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = mt * C::ROWS + nt * 8 + g;
    const bool real = r < p.rows;
    const int i = real ? r / p.group : 0, hq = head * p.group + (real ? r - i * p.group : 0);
    const uint16_t* src = p.q + (((long long)b * p.n_q + i) * p.h_q + hq) * D;
    if (!FP8) {
#pragma unroll
      for (int c = 0; c < C::KC; ++c) {
        const uint4 w = real ? __ldg(reinterpret_cast<const uint4*>(src + 8 * (t + 4 * c))) : make_uint4(0, 0, 0, 0);
        qf[nt][2 * c][0] = w.x, qf[nt][2 * c][1] = w.y;
        qf[nt][2 * c + 1][0] = w.z, qf[nt][2 * c + 1][1] = w.w;
      }
      factor[nt][0] = factor[nt][1] = p.scale_log2;
    } else {
      // f16 operands (e4m3 is exact in f16): the row is scaled by the power of two that
      // brings its largest entry to [1, 2). A bf16 entry above 2^-14 of the largest stays
      // exact, a smaller one moves by at most 2^-25 of the largest.
      uint32_t raw[C::S][2];
      float top = 0.0f;
#pragma unroll
      for (int s = 0; s < C::S; ++s) {
        const uint2 w = real ? __ldg(reinterpret_cast<const uint2*>(src + 16 * (t + 4 * (s / 4)) + 4 * (s % 4)))
                             : make_uint2(0, 0);
        raw[s][0] = w.x, raw[s][1] = w.y;
#pragma unroll
        for (int e = 0; e < 2; ++e)
          top = fmaxf(top, fmaxf(fabsf(__uint_as_float(raw[s][e] << 16)),
                                 fabsf(__uint_as_float(raw[s][e] & 0xffff0000u))));
      }
      top = fmaxf(top, __shfl_xor_sync(kAll, top, 1));
      top = fmaxf(top, __shfl_xor_sync(kAll, top, 2));
      const int ex = min(max((int)(__float_as_uint(top) >> 23), 1), 253);  // 2^(ex - 127) <= top
      const float down = __uint_as_float((uint32_t)(254 - ex) << 23);       // 2^(127 - ex)
      const float up = __uint_as_float((uint32_t)ex << 23);
#pragma unroll
      for (int s = 0; s < C::S; ++s)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          qf[nt][s][e] = pack_f16x2(__uint_as_float(raw[s][e] << 16) * down,
                                    __uint_as_float(raw[s][e] & 0xffff0000u) * down);
      const float mine = p.scale_log2 * __ldg(p.k_scale + head) * up;
      factor[nt][0] = __shfl_sync(kAll, mine, 8 * t);
      factor[nt][1] = __shfl_sync(kAll, mine, 8 * t + 4);
    }
  }

  // ---- bounds of this lane's rows; `same`: every row sees every key of the range
  const bool same = p.n_q == 1;
  int last[NT][2], low[NT][2];
  int last_min = vis.len - 1, low_max = 0;
  if (!same) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = mt * C::ROWS + nt * 8 + 2 * t + e;
        last[nt][e] = vis.len - p.n_q + min(r / p.group, p.n_q - 1);
        low[nt][e] = p.window < 0 ? 0 : last[nt][e] - p.window;
      }
    last_min = vis.len - p.n_q;
    low_max = p.window < 0 ? 0 : vis.len - 1 - p.window;
  }
  auto legal = [&](int j, int nt, int e) { return j <= last[nt][e] && (j >= low[nt][e] || j < p.sinks); };

  float o[NT][C::S][4];
  float m_run[NT][2], l_run[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int s = 0; s < C::S; ++s)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[nt][s][e] = 0.0f;
    m_run[nt][0] = m_run[nt][1] = -INFINITY;
    l_run[nt][0] = l_run[nt][1] = 0.0f;
  }

  for (; tile < t1; tile += kWarps) {
    // ---- S^T = K Q^T
    float sc[C::KB][NT][4];
#pragma unroll
    for (int kb = 0; kb < C::KB; ++kb)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[kb][nt][e] = 0.0f;
#pragma unroll
    for (int kb = 0; kb < C::KB; ++kb)
#pragma unroll
      for (int c = 0; c < C::KC; ++c) {
        const uint32_t a0[4] = {kr[kb][0][c].x, kr[kb][0][c].y, kr[kb][0][c].z, kr[kb][0][c].w};
        const uint32_t a1[4] = {kr[kb][1][c].x, kr[kb][1][c].y, kr[kb][1][c].z, kr[kb][1][c].w};
        if (!FP8) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t a[4] = {a0[2 * x], a1[2 * x], a0[2 * x + 1], a1[2 * x + 1]};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma<FP8>(sc[kb][nt], a, qf[nt][2 * c + x][0], qf[nt][2 * c + x][1]);
          }
        } else {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint32_t a[4] = {e4m3_f16x2(a0[x], false), e4m3_f16x2(a1[x], false), e4m3_f16x2(a0[x], true),
                                   e4m3_f16x2(a1[x], true)};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma<FP8>(sc[kb][nt], a, qf[nt][4 * c + x][0], qf[nt][4 * c + x][1]);
          }
        }
      }
    const bool more = tile + kWarps < t1;
    const int row_cur = row_now;
    row_now = row_next;
    if (more) {
      load_k(row_now);
      row_next = rows_of(tile + 2 * kWarps);
    }

    // ---- masks: keys that are not there, and where rows differ, each row's own bounds
    const int x0 = tile * C::KT;
    const bool holes = __any_sync(kAll, lane < C::KT && row_cur < 0);
    const bool mixed =
        !same && (vis.key(x0 + C::KT - 1) > last_min || x0 < vis.head || x0 + vis.skip < low_max);
#pragma unroll
    for (int kb = 0; kb < C::KB; ++kb)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[kb][nt][e] *= factor[nt][e & 1];
    if (holes || mixed) {
#pragma unroll
      for (int kb = 0; kb < C::KB; ++kb)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const int x = kb * 16 + hf * 8 + g;
          const bool there = __shfl_sync(kAll, row_cur, x) >= 0;
          const int j = vis.key(x0 + x);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (!there || (mixed && !legal(j, nt, e))) sc[kb][nt][2 * hf + e] = -INFINITY;
        }
    }

    // ---- online softmax; l_run is this lane's share, summed at the end
    uint32_t pf[C::KB][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float alpha[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float mx = sc[0][nt][e];
#pragma unroll
        for (int kb = 0; kb < C::KB; ++kb) mx = fmaxf(mx, fmaxf(sc[kb][nt][e], sc[kb][nt][2 + e]));
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, x));
        const float m_new = fmaxf(m_run[nt][e], mx);
        const float m_use = m_new == -INFINITY ? 0.0f : m_new;  // nothing legal yet
        alpha[e] = ptx::ex2(m_run[nt][e] - m_use);
        m_run[nt][e] = m_new;
        float sum = 0.0f;
#pragma unroll
        for (int kb = 0; kb < C::KB; ++kb)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            sc[kb][nt][2 * hf + e] = ptx::ex2(sc[kb][nt][2 * hf + e] - m_use);
            sum += sc[kb][nt][2 * hf + e];
          }
        l_run[nt][e] = fmaf(l_run[nt][e], alpha[e], sum);
      }
      if (__any_sync(kAll, alpha[0] != 1.0f || alpha[1] != 1.0f)) {
#pragma unroll
        for (int s = 0; s < C::S; ++s)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nt][s][e] *= alpha[e & 1];
      }
      // P^T as the second product's operand, rounded to the cache's compute type (bf16, or
      // f16 for 8-bit pages): relative 2^-9 (2^-12) per weight, of either sign, below the
      // output's own rounding; the sum l keeps the unrounded weights
#pragma unroll
      for (int kb = 0; kb < C::KB; ++kb)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
          pf[kb][nt][hf] = transpose8(FP8 ? pack_f16x2(sc[kb][nt][2 * hf], sc[kb][nt][2 * hf + 1])
                                          : ptx::pack_bf16x2(sc[kb][nt][2 * hf], sc[kb][nt][2 * hf + 1]));
    }

    // ---- O^T += V^T P^T
    bool plain = true;
    if (mixed) {
      // a key that some rows may not see: its weight there is 0, and 0 * inf would still
      // be NaN, so a tile with infinities or NaN among its values goes key by key
      bool bad = false;
#pragma unroll
      for (int kb = 0; kb < C::KB; ++kb)
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
          for (int w = 0; w < C::VW; ++w) {
            const uint32_t y = vr[kb][x][w];
            if (FP8)
              bad |= __vcmpeq4(y & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0;  // NaN is the only special value
            else
              bad |= (y & 0x7f80u) == 0x7f80u || (y & 0x7f800000u) == 0x7f800000u;
          }
      plain = !__any_sync(kAll, bad);
    }
    if (plain) {
#pragma unroll
      for (int kb = 0; kb < C::KB; ++kb)
#pragma unroll
        for (int s = 0; s < C::S; ++s) {
          uint32_t a[4];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (!FP8) {
              a[2 * x] = __byte_perm(vr[kb][2 * x][s], vr[kb][2 * x + 1][s], 0x5410);
              a[2 * x + 1] = __byte_perm(vr[kb][2 * x][s], vr[kb][2 * x + 1][s], 0x7632);
            } else {
              const uint32_t y =
                  __byte_perm(vr[kb][2 * x][s / 2], vr[kb][2 * x + 1][s / 2], s % 2 ? 0x7362 : 0x5140);
              a[2 * x] = e4m3_f16x2(y, false);
              a[2 * x + 1] = e4m3_f16x2(y, true);
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma<FP8>(o[nt][s], a, pf[kb][nt][0], pf[kb][nt][1]);
        }
    } else {
#pragma unroll
      for (int kb = 0; kb < C::KB; ++kb)
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll 1
          for (int owner = 0; owner < 4; ++owner) {  // key (x >> 1) * 8 + 2 owner + (x & 1) of the block
            const int in8 = 2 * owner + (x & 1), key = kb * 16 + (x >> 1) * 8 + in8;
            const bool there = __shfl_sync(kAll, row_cur, key) >= 0;
            const int j = vis.key(x0 + key);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float w = __shfl_sync(kAll, sc[kb][nt][2 * (x >> 1) + e], in8 * 4 + t);
                const bool on = there && legal(j, nt, e);
#pragma unroll
                for (int s = 0; s < C::S; ++s) {
                  float v0, v1;
                  if (!FP8) {
                    const uint32_t y = __shfl_sync(kAll, vr[kb][x][s], (lane & ~3) | owner);
                    v0 = __uint_as_float(y << 16);
                    v1 = __uint_as_float(y & 0xffff0000u);
                  } else {
                    const uint32_t y =
                        e4m3_f16x2(__shfl_sync(kAll, vr[kb][x][s / 2], (lane & ~3) | owner), s % 2);
                    asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; cvt.f32.f16 %0, l; cvt.f32.f16 %1, h;}"
                        : "=f"(v0), "=f"(v1)
                        : "r"(y));
                  }
                  if (on) {
                    o[nt][s][e] = fmaf(w, v0, o[nt][s][e]);
                    o[nt][s][2 + e] = fmaf(w, v1, o[nt][s][2 + e]);
                  }
                }
              }
          }
    }
    if (more) load_v(row_now);
  }

  // ---- join the warps
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float l = l_run[nt][e];
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) l += __shfl_xor_sync(kAll, l, x);
      const int r = nt * 8 + 2 * t + e;
      if (g == 0) {
        sh.m[warp][r] = m_run[nt][e];
        sh.l[warp][r] = l;
      }
      if (r < rows)
#pragma unroll
        for (int s = 0; s < C::S; ++s) {
          const int col = FP8 ? (D / 8) * g + 2 * s : (s / 4) * 64 + 8 * g + 2 * (s % 4);
          *reinterpret_cast<float2*>(&sh.o[warp][r][col]) = make_float2(o[nt][s][e], o[nt][s][2 + e]);
        }
    }
  __syncthreads();
  const float v_scale = FP8 ? __ldg(p.v_scale + head) : 1.0f;
  for (int x = tid; x < rows * (D / 4); x += kThreads) {
    const int r = x / (D / 4), col = 4 * (x % (D / 4));
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sh.m[w][r]);
    const float base = M == -INFINITY ? 0.0f : M;
    float L = 0.0f;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = ptx::ex2(sh.m[w][r] - base);
      const float4 y = *reinterpret_cast<const float4*>(&sh.o[w][r][col]);
      L = fmaf(f, sh.l[w][r], L);
      acc.x = fmaf(f, y.x, acc.x), acc.y = fmaf(f, y.y, acc.y);
      acc.z = fmaf(f, y.z, acc.z), acc.w = fmaf(f, y.w, acc.w);
    }
    acc.x *= v_scale, acc.y *= v_scale, acc.z *= v_scale, acc.w *= v_scale;
    if (slot >= 0) {
      *reinterpret_cast<float4*>(p.ws_o + (slot * C::ROWS + r) * D + col) = acc;
      if (col == 0) {
        p.ws_ml[(slot * C::ROWS + r) * 2] = M;
        p.ws_ml[(slot * C::ROWS + r) * 2 + 1] = L;
      }
    } else {
      finish<D>(p, b, head, mt * C::ROWS + r, col, acc, M, L);
    }
  }
  __syncthreads();  // the next pair writes the same shared memory
}

template <int D, int NT, bool FP8>
__global__ void __launch_bounds__(kThreads, Cfg<D, NT, FP8>::CTAS_PER_SM) attn_paged_kernel(const PagedParams p) {
  using C = Cfg<D, NT, FP8>;
  __shared__ __align__(16) Shared<D, NT, FP8> sh;
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int pairs = p.h_kv * p.m_tiles;
  if (p.whole) {
    const int b = blockIdx.x / pairs, pair = blockIdx.x % pairs;
    attend<D, NT, FP8>(p, sh, b, pair / p.m_tiles, pair % p.m_tiles, 0, tiles_of<C::KT>(p, b), -1);
    return;
  }
  __shared__ long long sums[kThreads + 1];
  int per;
  const Split s = make_split<C::KT>(p, sums, gridDim.x, per);
  if ((int)blockIdx.x >= s.ctas) return;
  const long long begin = s.first(blockIdx.x), end = s.first(blockIdx.x + 1);
  if (begin >= end) return;
  long long before;
  int b = find_sequence<C::KT>(p, sums, per, begin / pairs, before);
  for (long long at = begin; at < end;) {
    int n = tiles_of<C::KT>(p, b);
    while (n == 0 || at >= (before + n) * pairs) {  // on to the sequence that holds tile `at`
      before += n;
      n = tiles_of<C::KT>(p, ++b);
    }
    const long long in = at - before * pairs;
    const int pair = (int)(in / n);
    const int t0 = (int)(in - (long long)pair * n);
    const int t1 = (int)min((long long)n, t0 + (end - at));
    const long long slot = t0 == 0 && t1 == n ? -1 : 2ll * blockIdx.x + (at != begin);
    attend<D, NT, FP8>(p, sh, b, pair / p.m_tiles, pair % p.m_tiles, t0, t1, slot);
    at += t1 - t0;
  }
}

// Joins the parts of a pair that several CTAs share, and writes the rows of pairs without a
// visible key. Block = pair.
template <int D, int NT, bool FP8>
__global__ void __launch_bounds__(kThreads) attn_paged_merge_kernel(const PagedParams p, int max_ctas) {
  using C = Cfg<D, NT, FP8>;
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  __shared__ long long sums[kThreads + 1];
  int per;
  const Split s = make_split<C::KT>(p, sums, max_ctas, per);
  const int pairs = p.h_kv * p.m_tiles;
  const int b = blockIdx.x / pairs, pair = blockIdx.x % pairs, head = pair / p.m_tiles, mt = pair % p.m_tiles;
  long long before = sums[b / per];
  for (int x = b / per * per; x < b; ++x) before += tiles_of<C::KT>(p, x);
  const int n = tiles_of<C::KT>(p, b);
  const long long begin = before * pairs + (long long)pair * n, end = begin + n;
  long long c0 = 0, c1 = -1;
  if (n > 0) {
    c0 = (begin * s.ctas) / s.total;  // the parts that hold tiles begin and end - 1
    while (s.first(c0 + 1) <= begin) ++c0;
    while (s.first(c0) > begin) --c0;
    c1 = ((end - 1) * s.ctas) / s.total;
    while (s.first(c1 + 1) <= end - 1) ++c1;
    while (s.first(c1) > end - 1) --c1;
    if (c0 == c1) return;  // finished by that CTA
  }
  const int rows = min(p.rows - mt * C::ROWS, C::ROWS);
  for (int x = threadIdx.x; x < rows * (D / 4); x += kThreads) {
    const int r = x / (D / 4), col = 4 * (x % (D / 4));
    // part c: slot 2 c if its tiles begin in this pair, else 2 c + 1 (only c0 can begin before it)
    auto ws_row = [&](long long c) { return (2 * c + (s.first(c) < begin)) * C::ROWS + r; };
    float M = -INFINITY;
    for (long long c = c0; c <= c1; ++c) M = fmaxf(M, p.ws_ml[ws_row(c) * 2]);
    const float base = M == -INFINITY ? 0.0f : M;
    float L = 0.0f;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (long long c = c0; c <= c1; ++c) {
      const long long w = ws_row(c);
      const float f = ptx::ex2(p.ws_ml[w * 2] - base);
      const float4 y = *reinterpret_cast<const float4*>(p.ws_o + w * D + col);
      L = fmaf(f, p.ws_ml[w * 2 + 1], L);
      acc.x = fmaf(f, y.x, acc.x), acc.y = fmaf(f, y.y, acc.y);
      acc.z = fmaf(f, y.z, acc.z), acc.w = fmaf(f, y.w, acc.w);
    }
    finish<D>(p, b, head, mt * C::ROWS + r, col, acc, M, L);
  }
}

template <typename... KArgs, typename... Args>
int launch_pdl(void (*kernel)(KArgs...), unsigned grid, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

template <int D, int NT, bool FP8>
int launch(const PagedArgs& a, float* ws) {
  using C = Cfg<D, NT, FP8>;
  PagedParams p;
  p.q = static_cast<const uint16_t*>(a.q);
  p.k = a.k_pages, p.v = a.v_pages;
  p.out = static_cast<uint16_t*>(a.out), p.lse = a.lse;
  p.page_table = a.page_table, p.cache_lens = a.cache_lens;
  p.k_scale = a.k_scale, p.v_scale = a.v_scale;
  p.B = a.B, p.n_q = a.n_q, p.h_q = a.h_q, p.h_kv = a.h_kv;
  p.group = a.h_q / a.h_kv, p.rows = a.n_q * p.group, p.m_tiles = (p.rows + C::ROWS - 1) / C::ROWS;
  p.n_pages = a.n_pages, p.page_size = a.page_size, p.max_pages = a.max_pages;
  p.page_shift = (a.page_size & (a.page_size - 1)) == 0 ? __builtin_ctz(a.page_size) : -1;
  p.max_len = a.max_pages * a.page_size;
  // no key is further back than max_len: wider windows and more sinks say the same
  p.window = a.window < p.max_len ? a.window : p.max_len;
  p.sinks = a.window < 0 ? 0 : a.sinks < p.max_len ? a.sinks : p.max_len;
  p.scale_log2 = (float)((double)a.scale * 1.4426950408889634074);
  const int ctas = C::CTAS_PER_SM * kSMs;
  p.ws_o = ws, p.ws_ml = ws + (size_t)2 * ctas * C::ROWS * D;
  // keys that any sequence may have in sight
  long long most = p.max_len;
  if (p.window >= 0 && (long long)p.window + a.n_q + p.sinks < most) most = (long long)p.window + a.n_q + p.sinks;
  const long long pairs = (long long)a.B * a.h_kv * p.m_tiles;
  if (pairs > 0x7fffffffLL) return ATTN_ERR_INVALID;
  p.whole = (most + C::KT - 1) / C::KT <= kWholeTiles;
  const int st = launch_pdl(attn_paged_kernel<D, NT, FP8>, p.whole ? (unsigned)pairs : (unsigned)ctas, a.stream, p);
  if (st != ATTN_OK || p.whole) return st;
  return launch_pdl(attn_paged_merge_kernel<D, NT, FP8>, (unsigned)pairs, a.stream, p, ctas);
}

template <int D, bool FP8>
int launch_rows(const PagedArgs& a, float* ws) {
  return a.n_q * (a.h_q / a.h_kv) <= 8 ? launch<D, 1, FP8>(a, ws) : launch<D, 2, FP8>(a, ws);
}

}  // namespace

// Two slots for every CTA that can be resident, whatever the lengths.
size_t paged_decode_workspace_bytes(int n_q, int group, int d) {
  const int rows = (long long)n_q * group <= 8 ? 8 : 16;
  return (size_t)2 * kMaxCtasPerSM * kSMs * rows * (d + 2) * sizeof(float);
}

int launch_attn_paged_decode(const PagedArgs& a, void* workspace) {
  float* ws = static_cast<float*>(workspace);
  if (a.d == 64) return a.e4m3 ? launch_rows<64, true>(a, ws) : launch_rows<64, false>(a, ws);
  return a.e4m3 ? launch_rows<128, true>(a, ws) : launch_rows<128, false>(a, ws);
}

}  // namespace attn
