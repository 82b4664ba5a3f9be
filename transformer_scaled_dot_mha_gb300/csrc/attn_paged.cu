// attn_paged.cu -- attn_paged_decode: the newest n_q (1..16) tokens of every sequence attend
// over a paged key/value cache. Shared key/value heads (query head h uses key/value head
// h / group), an optional sliding window whose first `sinks` tokens stay visible, pages in
// bf16 or e4m3 (value = stored value * the head's scale).
//
// For row r (token i, query head) of a sequence of `len` tokens, pos = len - n_q + i:
//   legal keys: j <= pos and (no window, or j >= pos - window, or j < sinks)
//   out = sum_j p_j v_j / sum_j p_j,   p_j = 2^(s_j - m),  s_j = scale log2(e) q . k_j,  m = max_j s_j
// (8-bit pages: all p_j times 2^15, see Cfg::SHIFT, which the quotient takes back).
//
// What bounds it, up to 16 rows (n_q x group) per key/value head: each visible K and V row is
// read once, 4 (8-bit: 2) bytes per column pair against 4 x rows operations, so HBM. The
// arithmetic has only to stay out of the way, which CUDA cores cannot at group 8 (54 TFLOP/s at
// the full HBM rate): both products run on the warp-level matrix instruction m16n8k16, whose
// operands are registers. A tcgen05 MMA would need 128 rows and its operands in shared
// memory; for 1 to 16 rows the cache would pass through shared memory for nothing.
// More rows (several tokens of a large group) are tiles of 16, each a pair of its own in the
// list below that reads the keys again: the matrix pipe and the reads from L2 bound those calls
// (16 x 64/8 heads of d 128, 4096-8192 keys, floor 60 us: 8 rows 72 us, 16 76, 32 120, 128 437;
// e4m3, 8 x 64/8 heads, 9001-65521 keys, floor 90 us: 104, 113, 207, 777).
//
// The products are formed transposed, S^T = K Q^T and O^T = V^T P^T, so that the keys (then
// the columns) are the 16 rows of an MMA and the query rows its 8 columns (NT column tiles
// for up to 8 NT rows):
//   * the order of the contracted columns is free: a lane takes 16-byte pieces of "its" key
//     (row lane / 4) of K as they lie, and Q is loaded in the same order;
//   * S^T leaves a lane with (key lane / 4, rows 2 (lane % 4) and + 1); a register
//     transpose (movmatrix) turns the rounded P^T into the second product's operand;
//   * of V a lane takes 16 bytes of columns (all 8 or 16 of "its" columns) of each of four
//     keys and pairs up the keys by byte permutes; the order of the columns is free again.
// Tiles come by asynchronous copies (cp.async) into a ring of shared memory of the warp's own,
// STAGES tiles in flight without registers to hold them, whole rows side by side in one
// instruction: a copy of 512 contiguous bytes streams at 6.6 TB/s where the fragments' own
// pattern (8 rows x 64 bytes) stayed at 5.0 (402 MB, 12 warps per SM). The 16-byte pieces of
// a row are swapped by its number so that the fragment reads meet no bank conflict. Waits
// are cp.async.wait_group, which ends by itself; no block barrier in the stream.
//
// Work split: the tiles (KT keys) of all (sequence, key/value head, row tile) pairs form one
// list, cut into equal parts by the lengths on the device, so that ragged batches leave no
// warp idle and what a capacity holds above the lengths is not read. There is a part for
// every warp that can be resident, and a warp is a CTA (two or three parts for each, to even out
// the warps' speeds, cost more in starts and joins: 71.2, 71.8, 75.4 us at 16 x 8 heads of d 128
// and 4096-8192 keys when that was tried, with the weights in one part). It
// streams its part from one pair into the next without a pause in its copies. A pair that
// lies within one warp's part is finished there; of one that does not, every part leaves
// (m, l, O) in the workspace, the warp that has its first tile leaves a note of the parts,
// and attn_paged_merge_kernel joins them. When no sequence can be longer than a few tiles,
// each pair gets a warp of its own and there is no second launch. The host chooses between the
// two and knows the capacity alone, not the lengths: short sequences under a wide page table
// are cut up and joined (200 x 8 heads of d 128, 10-300 keys: 33.1 us, 27.6 under a table of
// 300 keys).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "attn_internal.h"
#include "ptx_sm103.cuh"

namespace attn {
namespace {

constexpr int kSMs = 152;
constexpr int kMaxParts = 12 * kSMs;  // parts of the list of tiles at most, one per resident warp
constexpr int kMinTiles = 2;          // tiles per part, at least (8 heads, 500 keys: 7.3 us; 8.0 from three)
constexpr int kPairCost = 2;          // tiles that a pair's queries and results cost
constexpr int kWholeTiles = 4;        // up to here no pair is split (8 heads, 250 keys: 7.3 us; 9.0 up to eight)
constexpr int kMergeThreads = 1024;   // at most
constexpr uint32_t kAll = 0xffffffffu;

// D columns, NT tiles of 8 query rows, FP8: e4m3 pages.
template <int D, int NT, bool FP8>
struct Cfg {
  static constexpr int KT = (D == 128 && !FP8) ? 16 : 32;  // keys per warp tile
  static constexpr int KB = KT / 16;                       // 16-key blocks
  static constexpr int KC = FP8 ? D / 64 : D / 32;         // 16-byte pieces of a key per lane
  static constexpr int VW = FP8 ? D / 32 : D / 16;         // 32-bit words of a value row per lane
  static constexpr int ROW_BYTES = D * (FP8 ? 1 : 2);
  static constexpr int PIECES = ROW_BYTES / 16;            // of a row
  static constexpr int SIDE = 32 / PIECES;                 // rows that one copy instruction covers
  static constexpr int S = D / 16;                         // MMA steps over the columns; column tiles of O
  static constexpr int ROWS = 8 * NT;
  static constexpr int PARTS_P = FP8 ? 1 : 2;  // of a weight, in the second product
  // e4m3: the weights go through f16, which ends at 2^16 and has all its bits from 2^-14 up only.
  // As 2^15 p they keep them down to 2^-29 of the largest, and none above 2^-40 of it vanishes.
  // (An early token that takes nearly all the weight and has no value leaves an output made of
  // such weights.) O and l carry the factor; it leaves with their quotient, and in lse.
  static constexpr float SHIFT = FP8 ? 15.0f : 0.0f;
  static constexpr int TILE_BYTES = KT * ROW_BYTES;          // of K, and of V
  static constexpr int CTAS_PER_SM = D == 128 && NT == 2 ? 8 : 12;  // 255 or 168 registers
  static constexpr int PARTS = CTAS_PER_SM * kSMs;
  static constexpr int STAGES = 196608 / CTAS_PER_SM / (2 * TILE_BYTES);  // tiles in flight: 192 KB per SM
  static constexpr int SMEM_BYTES = STAGES * 2 * TILE_BYTES;
};

// A pair whose tiles several parts share: its first slot, and the slots 2 (first + 1), 2 (first
// + 2) .. 2 last of the parts behind it; last < 0: nothing to join.
struct Note {
  int pair, slot, first, last;
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
  float* ws_o;   // [2 * PARTS][ROWS][D]: slot 2 c for the pair that part c begins in, 2 c + 1 for the one it ends in
  float* ws_ml;  // [2 * PARTS][ROWS][2]
  Note* notes;   // [PARTS], of pair x where there are at most PARTS pairs, else of the pair that part x begins
  int B, n_q, h_q, h_kv, group, rows, m_tiles;  // rows = n_q * group
  int n_pages, page_size, max_pages, max_len;
  uint32_t page_inv, page_shift;  // x / page_size = mulhi(2 x, page_inv) >> page_shift for x < 2^30
  uint32_t group_inv;             // x / group = mulhi(x, group_inv) for x < 16 group, group <= 8192
  int window, sinks;
  int whole;  // one warp per pair, no split
  int notes_by_pair;
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
// The bits of bf16's leading part of a weight: of the next number below it, so that the rest of a
// weight above zero is above zero too (0 times an infinite value would be NaN).
__device__ __forceinline__ uint32_t leading(float w) { return max(__float_as_int(w) - 1, 0) & 0xffff0000; }
// 16 bytes to shared memory, zeros where `there` is false (then nothing is read).
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "r"(addr)
               : "memory");
  return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 r;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(addr) : "memory");
  return r;
}

// Whether a word of V holds an infinity or NaN (e4m3: NaN is the only special value).
template <bool FP8>
__device__ __forceinline__ bool special(uint32_t y) {
  if (FP8) return __vcmpeq4(y & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0;
  return (y & 0x7f80u) == 0x7f80u || (y & 0x7f800000u) == 0x7f800000u;
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
  v.len = min(max(p.cache_lens[b], 0), p.max_len);
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

// The list of tiles. Sequence b holds its pairs (head, row tile) one after the other, each of
// n = tiles_of(b) tiles. A pair costs kPairCost tiles more (its queries, its results): in the
// count that parts are cut from it has kPairCost units, if it has tiles at all, and then one
// per tile; part c is units [c * part, (c + 1) * part). (64 sequences of 3 to 8191 keys, windows
// of 1024: 21.7 us, 28.0 without.) All of it counts in 32 bits: the launch refuses a list
// that could be longer.
struct Scan {
  int b0;            // the first of the 32 sequences that the lanes stand for
  int n, units;      // tiles of the lane's, units up to and with it
  uint32_t some;     // which have tiles
  int tiles, before;  // tiles and units of the sequences below b0 (of one pair each)
};

template <int KT>
__device__ __forceinline__ int lane_tiles(const PagedParams& p, int b) {
  return b < p.B ? tiles_of<KT>(p, b) : 0;
}

__device__ __forceinline__ void scan(Scan& s, int n) {
  s.n = n;
  s.some = __ballot_sync(kAll, n > 0);
  s.units = n > 0 ? n + kPairCost : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kAll, s.units, o);
    if (threadIdx.x >= o) s.units += y;
  }
}

// The sequence, pair of it and tile at which unit x stands (the first tile, if x is among the
// pair's own units), searching on from s; returns the list's tiles before that one.
template <int KT>
__device__ __forceinline__ int locate(const PagedParams& p, Scan& s, int pairs, int x, int& b, int& pair, int& tile) {
  for (;;) {
    const uint32_t past = __ballot_sync(kAll, (s.before + s.units) * pairs > x);
    const int last = past ? __ffs(past) - 1 : 32;  // the sequence that holds x
    const int skipped = __popc(s.some & (uint32_t)((1ull << last) - 1));
    const int at = __shfl_sync(kAll, s.units, (last - 1) & 31), units = last > 0 ? at : 0;
    if (past) {
      const int n = __shfl_sync(kAll, s.n, last);
      const int in = x - (s.before + units) * pairs;
      b = s.b0 + last;
      pair = (uint32_t)in / (uint32_t)(n + kPairCost);
      tile = max(in - pair * (n + kPairCost) - kPairCost, 0);
      return (s.tiles + units - kPairCost * skipped) * pairs + pair * n + tile;
    }
    s.before += units;
    s.tiles += units - kPairCost * skipped;
    s.b0 += 32;
    scan(s, lane_tiles<KT>(p, s.b0 + threadIdx.x));
  }
}

// Part c: its first sequence, pair and tile, and how many tiles (0: the list ends before it, or
// it has a pair's units only).
template <int KT, int PARTS>
__device__ __forceinline__ int find_part(const PagedParams& p, int c, int& part, int& b, int& pair, int& tile) {
  const int pairs = p.h_kv * p.m_tiles, lane = threadIdx.x;
  const int n0 = lane_tiles<KT>(p, lane);  // the first 32 sequences, where the search begins
  int more = 0, more_some = 0;
#pragma unroll 4
  for (int x = 32 + lane; x < p.B; x += 32) {
    const int n = tiles_of<KT>(p, x);
    more += n;
    more_some += n > 0;
  }
  Scan s;
  s.b0 = s.tiles = s.before = 0;
  scan(s, n0);
  int units = __shfl_sync(kAll, s.units, 31), tiles = units - kPairCost * __popc(s.some);
  if (p.B > 32) {
    more = __reduce_add_sync(kAll, more);
    tiles += more;
    units += more + kPairCost * __reduce_add_sync(kAll, more_some);
  }
  units *= pairs;
  part = max(kMinTiles, (int)((uint32_t)(units + PARTS - 1) / PARTS));
  const int begin = c * part, end = begin + part;
  if (begin >= units) return 0;
  const int first = locate<KT>(p, s, pairs, begin, b, pair, tile);
  int b2, pair2, tile2;
  const int last = end < units ? locate<KT>(p, s, pairs, end, b2, pair2, tile2) : tiles * pairs;
  return last - first;
}

// A place in the list.
template <int KT>
struct Cursor {
  int b, head, mt, tile, n;  // tile of n of the pair (head, row tile mt)
  Visible vis;
  __device__ __forceinline__ void sequence(const PagedParams& p) {
    vis = visible_of(p, b);
    n = (vis.count + KT - 1) / KT;
  }
  __device__ __forceinline__ void step(const PagedParams& p) {
    if (++tile < n) return;
    tile = 0;
    if (++mt < p.m_tiles) return;
    mt = 0;
    if (++head < p.h_kv) return;
    head = 0;
    do {
      if (++b >= p.B) return;  // past the end of the list: not used
      sequence(p);
    } while (n == 0);
  }
};

// ---------------------------------------------------------------- one warp's part

// Looking up the cache row of the key that `lane` has of the cursor's tile, in two steps: the
// page's number travels while something else is done. page < 0: there is no such key.
struct Lookup {
  int page, rest;  // rest: of the row's number, behind the page's first
};

template <int KT>
__device__ __forceinline__ Lookup start_lookup(const PagedParams& p, const Cursor<KT>& c, int lane) {
  const int x = c.tile * KT + lane;
  if (lane >= KT || x >= c.vis.count) return Lookup{-1, 0};
  const int j = c.vis.key(x);
  const int slot = (int)(__umulhi(2u * j, p.page_inv) >> p.page_shift);
  return Lookup{p.page_table[(long long)c.b * p.max_pages + slot],
                (c.head - slot) * p.page_size + j};  // head rows of whole pages, then the key's place
}

__device__ __forceinline__ int finish_lookup(const PagedParams& p, const Lookup& l) {
  if (l.page < 0 || l.page >= p.n_pages) return -1;  // names no page: its keys count as illegal
  return l.page * p.h_kv * p.page_size + l.rest;
}

// The token that row `row` of a pair belongs to.
__device__ __forceinline__ int token_of(const PagedParams& p, int row) {
  return p.group == 1 ? row : (int)__umulhi(row, p.group_inv);
}

// Where row `row` of (sequence, head) stands in out and lse.
__device__ __forceinline__ long long out_row(const PagedParams& p, int b, int head, int row) {
  const int i = token_of(p, row);
  return ((long long)b * p.n_q + i) * p.h_q + head * p.group + (row - i * p.group);
}

// The rows of sequences without a visible key, shared out over the CTAs.
template <int D>
__device__ __forceinline__ void empty_rows(const PagedParams& p) {
  const int lane = threadIdx.x;
#pragma unroll 1
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    if (visible_of(p, b).count > 0) continue;
    const long long row0 = (long long)b * p.n_q * p.h_q;
    for (int r = 0; r < p.n_q * p.h_q; ++r) {
      if (lane < D / 8) *reinterpret_cast<uint4*>(p.out + (row0 + r) * D + 8 * lane) = make_uint4(0, 0, 0, 0);
      if (p.lse && lane == 0) p.lse[row0 + r] = -INFINITY;
    }
    if (!p.whole && p.notes_by_pair)
      for (int x = lane; x < p.h_kv * p.m_tiles; x += 32) p.notes[b * p.h_kv * p.m_tiles + x] = Note{0, 0, 0, -1};
  }
}

// ln of 2^m l, where l is 2^shift times the sum; __log2f is within 2^-22, relative (absolute near
// 1): below lse's own rounding.
__device__ __forceinline__ float log_sum(float m, float l, float shift) {
  return (m + (__log2f(l) - shift)) * 0.69314718055994530942f;
}

// The rows of one pair as a warp holds them: queries, bounds, running statistics.
template <int D, int NT, bool FP8>
struct Rows {
  using C = Cfg<D, NT, FP8>;
  uint32_t q[NT][C::S][2];      // B fragments in the order of the K pieces, zeros past the last row
  float factor[NT][2];          // of rows 2 t, 2 t + 1: scores in log2 units = factor * accumulator
  int last[NT][2], low[NT][2];  // of the same rows, where rows differ (n_q > 1): keys they may see
  float o[NT][C::S][4];
  float m[NT][2], l[NT][2];     // l: this lane's share

  __device__ __forceinline__ void begin(const PagedParams& p, const Cursor<C::KT>& c, int lane) {
    const int g = lane >> 2, t = lane & 3;
    const int head = c.head, row0 = c.mt * C::ROWS;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = row0 + nt * 8 + g;
      const bool real = r < p.rows;
      const uint16_t* src = p.q + out_row(p, c.b, head, real ? r : 0) * D;
      if (!FP8) {
#pragma unroll
        for (int x = 0; x < C::KC; ++x) {
          const uint4 w = real ? *reinterpret_cast<const uint4*>(src + 8 * (t + 4 * x)) : make_uint4(0, 0, 0, 0);
          q[nt][2 * x][0] = w.x, q[nt][2 * x][1] = w.y;
          q[nt][2 * x + 1][0] = w.z, q[nt][2 * x + 1][1] = w.w;
        }
        factor[nt][0] = factor[nt][1] = p.scale_log2;
      } else {
        // f16 operands (e4m3 is exact in f16): the row is scaled by the power of two that
        // brings its largest entry to [1, 2). A bf16 entry above 2^-14 of the largest stays
        // exact, a smaller one moves by at most 2^-25 of the largest.
        float top = 0.0f;
#pragma unroll
        for (int x = 0; x < C::S; ++x) {
          const uint2 w = real ? *reinterpret_cast<const uint2*>(src + 16 * (t + 4 * (x / 4)) + 4 * (x % 4))
                               : make_uint2(0, 0);
          q[nt][x][0] = w.x, q[nt][x][1] = w.y;
#pragma unroll
          for (int e = 0; e < 2; ++e)
            top = fmaxf(top, fmaxf(fabsf(__uint_as_float(q[nt][x][e] << 16)),
                                   fabsf(__uint_as_float(q[nt][x][e] & 0xffff0000u))));
        }
        top = fmaxf(top, __shfl_xor_sync(kAll, top, 1));
        top = fmaxf(top, __shfl_xor_sync(kAll, top, 2));
        const int ex = min(max((int)(__float_as_uint(top) >> 23), 1), 253);  // 2^(ex - 127) <= top
        const float down = __uint_as_float((uint32_t)(254 - ex) << 23);       // 2^(127 - ex)
        const float up = __uint_as_float((uint32_t)ex << 23);
#pragma unroll
        for (int x = 0; x < C::S; ++x)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            q[nt][x][e] = pack_f16x2(__uint_as_float(q[nt][x][e] << 16) * down,
                                     __uint_as_float(q[nt][x][e] & 0xffff0000u) * down);
        const float mine = p.scale_log2 * p.k_scale[head] * up;
        factor[nt][0] = __shfl_sync(kAll, mine, 8 * t);
        factor[nt][1] = __shfl_sync(kAll, mine, 8 * t + 4);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (p.n_q > 1) {
          last[nt][e] = c.vis.len - p.n_q + min(token_of(p, row0 + nt * 8 + 2 * t + e), p.n_q - 1);
          low[nt][e] = p.window < 0 ? 0 : last[nt][e] - p.window;
        }
        m[nt][e] = -INFINITY;
        l[nt][e] = 0.0f;
      }
#pragma unroll
      for (int x = 0; x < C::S; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][x][e] = 0.0f;
    }
  }

  __device__ __forceinline__ bool legal(const PagedParams& p, int j, int nt, int e) const {
    return j <= last[nt][e] && (j >= low[nt][e] || j < p.sinks);
  }

  // Writes the pair's rows: finished (slot < 0), or (m, l, O) into the slot. A lane has 8 (16)
  // adjacent columns of rows 2 t, 2 t + 1: whole sectors.
  __device__ __forceinline__ void end(const PagedParams& p, const Cursor<C::KT>& c, int lane, int slot) {
    const int g = lane >> 2, t = lane & 3;
    const int head = c.head, row0 = c.mt * C::ROWS;
    const float v_scale = FP8 ? p.v_scale[head] : 1.0f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[nt][e];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) sum += __shfl_xor_sync(kAll, sum, x);
        const int r = nt * 8 + 2 * t + e;
        if (row0 + r >= p.rows) continue;
        const bool none = m[nt][e] == -INFINITY && sum == 0.0f;  // no legal key
        const float f = slot >= 0 ? v_scale : none ? 0.0f : __fdividef(v_scale, sum);
        const long long at = slot >= 0 ? (long long)slot * C::ROWS + r : out_row(p, c.b, head, row0 + r);
#pragma unroll
        for (int x = 0; x < C::S; x += 4) {
          const int col = FP8 ? (D / 8) * g + 2 * x : 16 * x + 8 * g;
          float y[8];
#pragma unroll
          for (int z = 0; z < 4; ++z) y[2 * z] = o[nt][x + z][e] * f, y[2 * z + 1] = o[nt][x + z][2 + e] * f;
          if (slot >= 0) {
            float4* dst = reinterpret_cast<float4*>(p.ws_o + at * D + col);
            dst[0] = make_float4(y[0], y[1], y[2], y[3]);
            dst[1] = make_float4(y[4], y[5], y[6], y[7]);
          } else {
            *reinterpret_cast<uint4*>(p.out + at * D + col) =
                make_uint4(ptx::pack_bf16x2(y[0], y[1]), ptx::pack_bf16x2(y[2], y[3]), ptx::pack_bf16x2(y[4], y[5]),
                           ptx::pack_bf16x2(y[6], y[7]));
          }
        }
        if (g == 0) {
          if (slot >= 0)
            *reinterpret_cast<float2*>(p.ws_ml + at * 2) = make_float2(m[nt][e], sum);
          else if (p.lse)
            p.lse[at] = none ? -INFINITY : log_sum(m[nt][e], sum, C::SHIFT);
        }
      }
  }
};

// `count` tiles from `cur` on. A pair whose tiles are not all among them leaves its (m, l, O) in
// `slot` (the first one) or slot + 1 (the last); part: tiles of a part of the list.
template <int D, int NT, bool FP8>
__device__ __forceinline__ void stream(const PagedParams& p, uint8_t* smem, Cursor<Cfg<D, NT, FP8>::KT> cur,
                                       int count, int slot, int part) {
  using C = Cfg<D, NT, FP8>;
  const int lane = threadIdx.x;
  const int g = lane >> 2, t = lane & 3;

  // ---- the ring: stage x holds K at ring + 2 x TILE_BYTES, V behind it. Piece c of row r
  // stands at place c ^ 4 (r & 1) of the row in K, c ^ 2 (r / 2 & 3) in V (of rows of four
  // pieces: c, and c ^ 2 (r / 2 & 1)): eight lanes that read together, two keys of K or four
  // of V, meet different banks.
  const uint32_t ring = ptx::smem_u32(smem);
  const int piece = lane % C::PIECES, side = lane / C::PIECES;
  const uint8_t* kp = static_cast<const uint8_t*>(p.k) + 16 * piece;
  const uint8_t* vp = static_cast<const uint8_t*>(p.v) + 16 * piece;
  auto request = [&](int stage, int rows_l) {
    const uint32_t at = ring + stage * 2 * C::TILE_BYTES;
#pragma unroll
    for (int x = 0; x < C::KT / C::SIDE; ++x) {
      const int r = x * C::SIDE + side;
      const int row = __shfl_sync(kAll, rows_l, r);
      const long long off = (long long)max(row, 0) * C::ROW_BYTES;
      const int k_to = C::PIECES == 4 ? piece : piece ^ (r & 1) << 2;
      const int v_to = C::PIECES == 4 ? piece ^ (r & 2) : piece ^ (r & 6);
      copy_async(at + r * C::ROW_BYTES + 16 * k_to, kp + off, row >= 0);
      copy_async(at + C::TILE_BYTES + r * C::ROW_BYTES + 16 * v_to, vp + off, row >= 0);
    }
  };
  // where this lane reads: key g of K (pieces t + 4 c), keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9 of V
  const uint32_t k_lane = g * C::ROW_BYTES + 16 * t + (C::PIECES == 4 ? 0 : 64 * (g & 1));
  const uint32_t v_lane = C::TILE_BYTES + 2 * t * C::ROW_BYTES +
                          (C::PIECES == 4 ? 16 * ((g >> 1) ^ (2 * t & 2)) + 8 * (g & 1) : 16 * (g ^ 2 * t));
  uint32_t there[C::STAGES];  // which keys of the tiles in flight exist; [0]: of the current one
  Cursor<C::KT> ahead = cur;  // the next tile to look up
  int rows_ahead[C::STAGES];  // rows of the next tiles to request
  Lookup pending;             // and of the one behind them
  int looked = 0;
  auto look_up = [&]() {
    if (looked >= count) return Lookup{-1, 0};
    if (ahead.tile == 0 || looked == 0) {  // a new pair: its queries into L1, a line per lane
      constexpr int LINES = D / 64;
      const int r = ahead.mt * C::ROWS + lane / LINES;
      if (lane < C::ROWS * LINES && r < p.rows)
        asm volatile("prefetch.global.L1 [%0];" ::"l"(p.q + out_row(p, ahead.b, ahead.head, r) * D +
                                                      64 * (lane % LINES)));
    }
    const Lookup l = start_lookup(p, ahead, lane);
    ahead.step(p);
    ++looked;
    return l;
  };
  {
    Lookup first[C::STAGES];
#pragma unroll
    for (int x = 0; x < C::STAGES; ++x) first[x] = look_up();
    pending = look_up();
#pragma unroll
    for (int x = 0; x < C::STAGES; ++x) rows_ahead[x] = finish_lookup(p, first[x]);
  }
  Rows<D, NT, FP8> rows;
  bool fresh = true;          // cur's pair has not begun
  int first_tile = cur.tile;  // of this part, of cur's pair
  int later = 0;              // whether that pair is not the part's first
  int stage = 0;
  // Step i works on tile i and refills its stage; the steps below 0 only fill the ring. (One
  // copy of the code for both: it has to stay in the instruction caches.)
  for (int i = -C::STAGES; i < count; ++i) {
    if (i >= 0) {
      if (fresh) rows.begin(p, cur, lane);
      fresh = false;
      copy_wait<C::STAGES - 1>();
      __syncwarp();  // every lane's copies are there
      const uint32_t at = ring + stage * 2 * C::TILE_BYTES;
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
          const uint32_t k_at = at + kb * 16 * C::ROW_BYTES + (k_lane ^ (c & 1) * 64) + (c >> 1) * 128;
          const uint4 k0 = lds128(k_at), k1 = lds128(k_at + 8 * C::ROW_BYTES);
          const uint32_t a0[4] = {k0.x, k0.y, k0.z, k0.w}, a1[4] = {k1.x, k1.y, k1.z, k1.w};
          if (!FP8) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint32_t a[4] = {a0[2 * x], a1[2 * x], a0[2 * x + 1], a1[2 * x + 1]};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma<FP8>(sc[kb][nt], a, rows.q[nt][2 * c + x][0], rows.q[nt][2 * c + x][1]);
            }
          } else {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const uint32_t a[4] = {e4m3_f16x2(a0[x], false), e4m3_f16x2(a1[x], false), e4m3_f16x2(a0[x], true),
                                     e4m3_f16x2(a1[x], true)};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma<FP8>(sc[kb][nt], a, rows.q[nt][4 * c + x][0], rows.q[nt][4 * c + x][1]);
            }
          }
        }
      // ---- masks: keys that are not there, and where rows differ, each row's own bounds
      const Visible& vis = cur.vis;
      const int x0 = cur.tile * C::KT;
      const bool holes = there[0] != (uint32_t)((1ull << C::KT) - 1);
      const bool mixed = p.n_q > 1 && (vis.key(x0 + C::KT - 1) > vis.len - p.n_q || x0 < vis.head ||
                                       (p.window >= 0 && x0 + vis.skip < vis.len - 1 - p.window));
#pragma unroll
      for (int kb = 0; kb < C::KB; ++kb)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[kb][nt][e] *= rows.factor[nt][e & 1];
      if (holes || mixed) {
#pragma unroll
        for (int kb = 0; kb < C::KB; ++kb)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const int x = kb * 16 + hf * 8 + g;
            const bool is = there[0] >> x & 1;
            const int j = vis.key(x0 + x);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (!is || (mixed && !rows.legal(p, j, nt, e))) sc[kb][nt][2 * hf + e] = -INFINITY;
          }
      }

      // ---- online softmax; rows.l is this lane's share, summed at the end
      uint32_t pf[C::KB][NT][2][C::PARTS_P];  // [.][.][half of the keys][part]
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
          const float m_new = fmaxf(rows.m[nt][e], mx);
          const float m_use = m_new == -INFINITY ? 0.0f : m_new;  // nothing legal yet
          alpha[e] = ptx::ex2(rows.m[nt][e] - m_use);
          rows.m[nt][e] = m_new;
          float sum = 0.0f;
#pragma unroll
          for (int kb = 0; kb < C::KB; ++kb)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              // at most SHIFT, however large m: the difference is at most 0 before it is shifted
              const float x = sc[kb][nt][2 * hf + e] - m_use;
              sc[kb][nt][2 * hf + e] = ptx::ex2(FP8 ? x + C::SHIFT : x);
              sum += sc[kb][nt][2 * hf + e];
            }
          rows.l[nt][e] = fmaf(rows.l[nt][e], alpha[e], sum);
        }
        if (__any_sync(kAll, alpha[0] != 1.0f || alpha[1] != 1.0f)) {
#pragma unroll
          for (int s = 0; s < C::S; ++s)
#pragma unroll
            for (int e = 0; e < 4; ++e) rows.o[nt][s][e] *= alpha[e & 1];
        }
        // P^T as the second product's operand. bf16 pages: in two parts, the leading bits of a
        // weight and what they leave, so that at most 2^-15 of it is lost; one part alone loses
        // up to 2^-8 of every term, as much as the output's own rounding (16 x 8 heads of d 128
        // 68.9 us, 68.4 with one part; 64 sequences x 64 rows and windows of 1024, bound by the
        // MMAs, 53.4 and 48.3). 8-bit pages: one part in f16, which loses 2^-11 of a weight
        // (2^-40 of the largest), an eighth of the output's rounding; two would take 125.7 us
        // instead of 112.7 (8 x 8 heads of 16 rows, 9001-65521 keys).
#pragma unroll
        for (int kb = 0; kb < C::KB; ++kb)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const float p0 = sc[kb][nt][2 * hf], p1 = sc[kb][nt][2 * hf + 1];
            if (FP8) {
              pf[kb][nt][hf][0] = transpose8(pack_f16x2(p0, p1));
            } else {
              const uint32_t h0 = leading(p0), h1 = leading(p1);
              pf[kb][nt][hf][0] = transpose8(__byte_perm(h0, h1, 0x7632));
              pf[kb][nt][hf][C::PARTS_P - 1] =
                  transpose8(ptx::pack_bf16x2(p0 - __uint_as_float(h0), p1 - __uint_as_float(h1)));
            }
          }
      }

      // ---- O^T += V^T P^T
      uint32_t vr[C::KB][4][C::VW];
      bool bad = false;
#pragma unroll
      for (int kb = 0; kb < C::KB; ++kb)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint32_t v_at = at + v_lane + (kb * 16 + (x >> 1) * 8 + (x & 1)) * C::ROW_BYTES;
          if (C::VW == 2) {
            const uint2 w = lds64(v_at);
            vr[kb][x][0] = w.x, vr[kb][x][1] = w.y;
          } else {
#pragma unroll
            for (int c = 0; c < C::VW / 4; ++c) {
              const uint4 w = lds128(v_at + 128 * c);
              vr[kb][x][4 * c] = w.x, vr[kb][x][4 * c + 1] = w.y;
              vr[kb][x][4 * c + 2] = w.z, vr[kb][x][4 * c + 3] = w.w;
            }
          }
          if (mixed)
#pragma unroll
            for (int w = 0; w < C::VW; ++w) bad |= special<FP8>(vr[kb][x][w]);
        }
      // In a mixed tile some rows may not see a key: its weight there is 0, and 0 * inf would
      // still be NaN, so a mixed tile with infinities or NaN among its values goes key by key.
      const bool plain = !mixed || !__any_sync(kAll, bad);
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
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int x = 0; x < C::PARTS_P; ++x) mma<FP8>(rows.o[nt][s], a, pf[kb][nt][0][x], pf[kb][nt][1][x]);
          }
      } else {
        // the weights go where the tile's K was, [key][row]; a lane's columns of V are read anew
        float* w_sh = reinterpret_cast<float*>(smem + (at - ring));
#pragma unroll
        for (int kb = 0; kb < C::KB; ++kb)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w_sh[(kb * 16 + (e >> 1) * 8 + g) * C::ROWS + nt * 8 + 2 * t + (e & 1)] = sc[kb][nt][e];
        __syncwarp();
#pragma unroll 1
        for (int key = 0; key < C::KT; ++key) {
          if (!(there[0] >> key & 1)) continue;
          const int j = vis.key(x0 + key);
          const uint32_t v_row = at + C::TILE_BYTES + key * C::ROW_BYTES;
#pragma unroll
          for (int x = 0; x < C::S; ++x) {
            // the word with this lane's columns 2 x, 2 x + 1 (e4m3: two columns of a word)
            const int byte = FP8 ? (D / 8) * g + 4 * (x / 2) : 128 * (x / 4) + 16 * g + 4 * (x % 4);
            const int swap = C::PIECES == 4 ? key & 2 : key & 6;
            uint32_t y;
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(y) : "r"(v_row + (byte ^ 16 * swap)) : "memory");
            float v0, v1;
            if (!FP8) {
              v0 = __uint_as_float(y << 16);
              v1 = __uint_as_float(y & 0xffff0000u);
            } else {
              asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; cvt.f32.f16 %0, l; cvt.f32.f16 %1, h;}"
                  : "=f"(v0), "=f"(v1)
                  : "r"(e4m3_f16x2(y, x % 2)));
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (rows.legal(p, j, nt, e)) {
                  const float w = w_sh[key * C::ROWS + nt * 8 + 2 * t + e];
                  rows.o[nt][x][e] = fmaf(w, v0, rows.o[nt][x][e]);
                  rows.o[nt][x][2 + e] = fmaf(w, v1, rows.o[nt][x][2 + e]);
                }
          }
        }
      }
      if (cur.tile + 1 == cur.n || i + 1 == count) {
        const bool complete = cur.tile + 1 == cur.n && first_tile == 0;
        rows.end(p, cur, lane, complete ? -1 : slot + later);
        if (!p.whole && first_tile == 0 && lane == 0 && (p.notes_by_pair || !complete)) {
          const int c = slot / 2, left = cur.n - 1 - cur.tile, pair = (cur.b * p.h_kv + cur.head) * p.m_tiles + cur.mt;
          p.notes[p.notes_by_pair ? pair : c] =
              Note{pair, slot + later, c, complete ? -1 : c + (left + part - 1) / part};
        }
        fresh = true;
        first_tile = 0;
        later = 1;
      }
      if (i + 1 < count) cur.step(p);
      __syncwarp();  // the stage is read
    }
    // ask for the tile STAGES further on, and look up the rows of another
#pragma unroll
    for (int x = 0; x + 1 < C::STAGES; ++x) there[x] = there[x + 1];
    there[C::STAGES - 1] = __ballot_sync(kAll, rows_ahead[0] >= 0);
    if (i + C::STAGES < count) request(stage, rows_ahead[0]);
    copy_commit();
    stage = stage + 1 < C::STAGES ? stage + 1 : 0;
#pragma unroll
    for (int x = 0; x + 1 < C::STAGES; ++x) rows_ahead[x] = rows_ahead[x + 1];
    rows_ahead[C::STAGES - 1] = finish_lookup(p, pending);
    pending = look_up();
  }
}

template <int D, int NT, bool FP8>
__global__ void __launch_bounds__(32, Cfg<D, NT, FP8>::CTAS_PER_SM) attn_paged_kernel(const PagedParams p) {
  using C = Cfg<D, NT, FP8>;
  extern __shared__ __align__(16) uint8_t smem[];
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int pairs = p.h_kv * p.m_tiles, c = blockIdx.x;
  if (!p.whole && !p.notes_by_pair && threadIdx.x == 0) p.notes[c] = Note{0, 0, 0, -1};
  Cursor<C::KT> cur;
  int pair = 0, part = 0;  // pair: of the sequence
  int count = 0;
  cur.tile = 0;
  if (p.whole) {
    cur.b = c / pairs;
    cur.sequence(p);
    pair = c - cur.b * pairs;
    count = cur.n;
  } else {
    count = find_part<C::KT, C::PARTS>(p, c, part, cur.b, pair, cur.tile);
    if (count > 0) cur.sequence(p);
  }
  if (count > 0) {
    cur.head = p.m_tiles == 1 ? pair : pair / p.m_tiles, cur.mt = pair - cur.head * p.m_tiles;
    stream<D, NT, FP8>(p, smem, cur, count, 2 * c, part);
  }
  empty_rows<D>(p);
}

// Joins the parts of a pair that several warps share. Block (note, group of `group_rows`
// rows). A warp takes a slice of a row's parts, a lane four columns; the slices are joined
// through shared memory.
template <int D, int NT, bool FP8>
__global__ void __launch_bounds__(kMergeThreads) attn_paged_merge_kernel(const PagedParams p, int group_rows) {
  using C = Cfg<D, NT, FP8>;
  constexpr int LANES = D / 4;          // lanes of a row of O
  constexpr int SIDE = 32 / LANES;      // parts side by side in a warp
  __shared__ float sh_m[kMergeThreads / 32], sh_l[kMergeThreads / 32];
  __shared__ __align__(16) float sh_o[kMergeThreads / 32][D];
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const Note note = p.notes[blockIdx.x];
  if (note.last < 0) return;
  const int bh = note.pair / p.m_tiles, mt = note.pair - bh * p.m_tiles;
  const int b = bh / p.h_kv, head = bh - b * p.h_kv;
  const int parts = note.last - note.first + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows = min(p.rows - mt * C::ROWS, C::ROWS);
  const int slices = blockDim.x / 32 / group_rows;  // warps per row
  const int slice = warp % slices, r = blockIdx.y * group_rows + warp / slices;
  const int col = 4 * (lane % LANES), side = lane / LANES;
  float M = -INFINITY, L = 0.0f;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  // 32 parts of the slice at a time: lane x has the statistics of the x-th. The first columns
  // are asked for together with them.
  if (r < rows)
#pragma unroll 1
    for (int c0 = slice; c0 < parts; c0 += 32 * slices) {
      auto row_of = [&](int c) { return (c == 0 ? note.slot : 2 * (note.first + c)) * C::ROWS + r; };
      const int mine = c0 + lane * slices, here = min(32, (parts - c0 + slices - 1) / slices);
      float2 ml = make_float2(-INFINITY, 0.0f);
      if (mine < parts) ml = *reinterpret_cast<const float2*>(p.ws_ml + (long long)row_of(mine) * 2);
      constexpr int BATCH = 4;
      float4 v[BATCH];
      auto load = [&](int x) {
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
          const int y = x + u * SIDE + side;
          v[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (y < here)
            v[u] = *reinterpret_cast<const float4*>(p.ws_o + (long long)row_of(c0 + y * slices) * D + col);
        }
      };
      load(0);
      float top = ml.x;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
      const float m_new = fmaxf(M, top), use = m_new == -INFINITY ? 0.0f : m_new;
      const float old = ptx::ex2(M - use), f = ptx::ex2(ml.x - use);
      M = m_new;
      float l = f * ml.y;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(kAll, l, o);
      L = fmaf(L, old, l);
      acc.x *= old, acc.y *= old, acc.z *= old, acc.w *= old;
#pragma unroll 1
      for (int x = 0; x < here;) {
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
          const float w = __shfl_sync(kAll, f, (x + u * SIDE + side) & 31);
          if (x + u * SIDE + side < here) {
            acc.x = fmaf(w, v[u].x, acc.x), acc.y = fmaf(w, v[u].y, acc.y);
            acc.z = fmaf(w, v[u].z, acc.z), acc.w = fmaf(w, v[u].w, acc.w);
          }
        }
        x += BATCH * SIDE;
        if (x < here) load(x);
      }
    }
  if (SIDE == 2) {
    acc.x += __shfl_xor_sync(kAll, acc.x, 16), acc.y += __shfl_xor_sync(kAll, acc.y, 16);
    acc.z += __shfl_xor_sync(kAll, acc.z, 16), acc.w += __shfl_xor_sync(kAll, acc.w, 16);
  }
  if (slices > 1) {
    *reinterpret_cast<float4*>(&sh_o[warp][col]) = acc;
    if (lane == 0) sh_m[warp] = M, sh_l[warp] = L;
    __syncthreads();
    if (slice > 0) return;
    float top = M;
    for (int x = 1; x < slices; ++x) top = fmaxf(top, sh_m[warp + x]);
    const float use = top == -INFINITY ? 0.0f : top;
    const float f = ptx::ex2(M - use);
    L *= f;
    acc.x *= f, acc.y *= f, acc.z *= f, acc.w *= f;
#pragma unroll 1
    for (int x = 1; x < slices; ++x) {
      const float w = ptx::ex2(sh_m[warp + x] - use);
      const float4 v = *reinterpret_cast<const float4*>(&sh_o[warp + x][col]);
      L = fmaf(w, sh_l[warp + x], L);
      acc.x = fmaf(w, v.x, acc.x), acc.y = fmaf(w, v.y, acc.y);
      acc.z = fmaf(w, v.z, acc.z), acc.w = fmaf(w, v.w, acc.w);
    }
    M = top;
  }
  if (r >= rows || side > 0) return;
  const long long row = out_row(p, b, head, mt * C::ROWS + r);
  const bool none = M == -INFINITY && L == 0.0f;  // no legal key
  const float inv = none ? 0.0f : __fdividef(1.0f, L);
  *reinterpret_cast<uint2*>(p.out + row * D + col) =
      make_uint2(ptx::pack_bf16x2(acc.x * inv, acc.y * inv), ptx::pack_bf16x2(acc.z * inv, acc.w * inv));
  if (p.lse && col == 0) p.lse[row] = none ? -INFINITY : log_sum(M, L, C::SHIFT);
}

template <typename... KArgs, typename... Args>
int launch_pdl(void (*kernel)(KArgs...), dim3 grid, int block, int smem, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  // the same division of L1 for both kernels: an SM has to run empty to change it
  at[1].id = cudaLaunchAttributePreferredSharedMemoryCarveout;
  at[1].val.sharedMemCarveout = cudaSharedmemCarveoutMaxShared;
  cfg.attrs = at;
  cfg.numAttrs = 2;
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
  p.page_shift = 0;
  while ((1LL << p.page_shift) < a.page_size) ++p.page_shift;
  p.page_inv = (uint32_t)(((1ULL << (31 + p.page_shift)) + a.page_size - 1) / a.page_size);
  p.group_inv = (uint32_t)((0x100000000ULL + p.group - 1) / p.group);  // group 1 does without
  p.max_len = a.max_pages * a.page_size;
  // no key is further back than max_len: wider windows and more sinks say the same
  p.window = a.window < p.max_len ? a.window : p.max_len;
  p.sinks = a.window < 0 ? 0 : a.sinks < p.max_len ? a.sinks : p.max_len;
  p.scale_log2 = (float)((double)a.scale * 1.4426950408889634074);
  p.ws_o = ws, p.ws_ml = ws + (size_t)2 * C::PARTS * C::ROWS * D;
  p.notes = reinterpret_cast<Note*>(p.ws_ml + (size_t)2 * C::PARTS * C::ROWS * 2);
  // Tiles that any pair may have decide whether pairs are split. They are not where that is
  // few; nor up to 24 tiles with pairs for half the warps (200 x 8 heads of d 128, 10-300 keys:
  // 27.6 us, 33.1 split; but 256 x 8 heads of 64 with 1000 keys, 32 tiles: 102.6 and 92.0), nor,
  // from 1.5 pairs per warp on, up to 22 times as many tiles as pairs per warp: the longest
  // pair is then no long tail (1000 x 8 heads, 500-2000 keys: 373.8 us, 398.9 split).
  long long most = p.max_len;
  if (p.window >= 0 && (long long)p.window + a.n_q + p.sinks < most) most = (long long)p.window + a.n_q + p.sinks;
  const long long pairs = (long long)a.B * a.h_kv * p.m_tiles, tiles = (most + C::KT - 1) / C::KT;
  if (pairs > 0x7ffff000LL / (tiles + kPairCost)) return ATTN_ERR_UNSUPPORTED;  // tiles are counted in 32 bits
  p.whole = tiles <= kWholeTiles || (tiles <= 6 * kWholeTiles && 2 * pairs >= C::PARTS) ||
            (2 * pairs >= 3 * C::PARTS && tiles * C::PARTS <= 22 * pairs);
  static_assert(C::SMEM_BYTES <= 48 * 1024, "fits without raising the kernel's limit");
  p.notes_by_pair = pairs <= C::PARTS;
  const int st = launch_pdl(attn_paged_kernel<D, NT, FP8>, dim3(p.whole ? (unsigned)pairs : C::PARTS), 32,
                            C::SMEM_BYTES, a.stream, p);
  if (st != ATTN_OK || p.whole) return st;
  // Few pairs have many parts each: all warps of a block on one row's. Many pairs' blocks take
  // several rows (256 pairs of 16 rows: 21.7 us, 34.8 with a block for each row).
  const int rows = p.rows < C::ROWS ? p.rows : C::ROWS;
  const int group_rows = pairs * rows <= 8 * kSMs ? 1 : rows <= 4 ? 4 : 8;
  // More than 160 parts to a pair are worth blocks of 32 warps (8 heads of d 128: 32000 keys
  // 33.7 -> 30.5 us, 128000 91.6 -> 87.8); fewer are joined later by them (256 pairs of 7: 23.5
  // -> 27.5; 8 heads of 64, 8000 keys, 125 parts: 8.7 -> 9.9).
  const bool many = 160 * pairs < C::PARTS && tiles > 160 * kMinTiles && pairs * rows <= 2 * kSMs;
  const int threads = many ? kMergeThreads : 256;
  const dim3 grid(p.notes_by_pair ? (unsigned)pairs : C::PARTS, (unsigned)((rows + group_rows - 1) / group_rows));
  return launch_pdl(attn_paged_merge_kernel<D, NT, FP8>, grid, threads, 0, a.stream, p, group_rows);
}

template <int D, bool FP8>
int launch_rows(const PagedArgs& a, float* ws) {
  return a.n_q * (a.h_q / a.h_kv) <= 8 ? launch<D, 1, FP8>(a, ws) : launch<D, 2, FP8>(a, ws);
}

}  // namespace

// Two slots for every warp that can be resident, whatever the lengths.
size_t paged_decode_workspace_bytes(int n_q, int group, int d) {
  const int rows = (long long)n_q * group <= 8 ? 8 : 16;
  return (size_t)kMaxParts * (2 * rows * (d + 2) * sizeof(float) + sizeof(Note));
}

int launch_attn_paged_decode(const PagedArgs& a, void* workspace) {
  float* ws = static_cast<float*>(workspace);
  if (a.d == 64) return a.e4m3 ? launch_rows<64, true>(a, ws) : launch_rows<64, false>(a, ws);
  return a.e4m3 ? launch_rows<128, true>(a, ws) : launch_rows<128, false>(a, ws);
}

}  // namespace attn
