// attn_packed.cu -- attention over ragged batches on the sm_103a tensor cores: sequences of
// different lengths packed one after the other (attn_packed_fwd), and chunks of new tokens over
// a paged cache (attn_paged_chunk), query heads sharing key/value heads.
//
//   s_ij = scale q_i . k_j on legal pairs,  out_i = sum_j exp(s_ij - lse_i) v_j,
//   lse_i = ln sum_j exp(s_ij);  query i of a sequence stands at position n_k - n_q + i.
//
// The softmax is the online form of attn_fwd_tc.cu: a running reference maximum, raised only
// when a row's maximum grows by more than 2^8, and a running sum; O / l is exact whatever the
// reference.
//
// Rows. The g = h_q / h_kv query heads of one key/value head read the same keys, so a row tile
// is floor(128 / g) tokens times g heads (row = token * g + head): one TMA box of a
// four-dimensional view of q. A tile of keys is then read once for all g heads, and one new
// token of a sequence fills g rows, not one.
//
// Work. attn_plan.cuh lists the units (row tiles of a sequence for one key/value head) with the
// key tiles that each streams; the CTAs are persistent and their roles run through their units
// without meeting, so the copies and the products of the next unit start while the softmax warps
// still write the last one's rows. Units that are too long the plan cuts: a piece leaves its
// rows' unnormalised sums, reference maxima and row sums in the workspace, and attn_join_kernel
// adds the pieces up.
//
// Tiles. As in attn_fwd_tc.cu: at d = 64 a CTA has one row tile, two CTAs share an SM, and P has
// TMEM columns of its own, with an MMA issuer for each product; at d = 128, and with pages, whose copies cost
// more, a CTA has two row tiles, P written over S, with an issuer for each row tile (8 bits: one for both,
// as four more warps have other work). Keys come as 128-row tiles through a shared-memory ring:
//   dense   one TMA box per 64 columns;
//   pages   warps for K and warps for V copy a tile page by page (TMA, or cp.async for the smallest), page
//           numbers looked up ahead. Rows of no page (a bad entry, or behind the length) are zeros. Bad
//           entries' keys are masked by bits that go with the tile.
//   8 bits  the rows land in a raw tile, and four more warps turn it into the f16 tile that the
//           products read: exact, as f16 holds every e4m3 number (the scales are folded into the
//           exponent's factor and the last division). An MMA's operands are of one type, so Q
//           becomes f16 too, each row times a power of two, and P is f16.
// Dense values behind the sequence's end (the next sequence's rows) would meet
// P = 0 in the product, and 0 times infinity or NaN is NaN: a spare warp zeroes them in shared
// memory when the issuer of that product has seen the tile land and asks for it.
//
// Every wait is bounded, as in attn_fwd_tc.cu.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <utility>

#include "attn_internal.h"
#include "attn_plan.cuh"
#include "ptx_warp.cuh"

namespace attn {

__device__ unsigned int g_packed_fault_word;  // fault record, read by attn_fault_status

namespace {

constexpr int BM = 128, BN = 128;  // rows and keys per tile
constexpr int kMaxDevices = 64;
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr uint64_t kDrainLimitNs = 200000000ull;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr uint32_t FAULT_PACKED = 512;
constexpr int UNITS = 4;    // units whose entries a CTA holds at a time
constexpr int FLAGS = 8;    // tiles whose page bits are held: more than the roles are apart
constexpr int kMinShare = 2;   // tiles
constexpr int kTmaShift = 3;   // 2^3 rows of a page or more go by one TMA copy, fewer by cp.async
constexpr float kBias = 7.0f;  // P in f16 is 2^7 times the weight

enum { DENSE = 0, PAGED = 1, PAGED8 = 2 };

// As ptx::idesc_bf16_f32, for f16 operands (format 0).
__host__ __device__ constexpr uint32_t idesc_f16_f32(uint32_t M, uint32_t N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

template <int D, int KIND>
struct Cfg {
  static constexpr bool SINGLE = D == 64 && KIND == DENSE;
  static constexpr int Q_TILES = SINGLE ? 1 : 2;
  static constexpr int ROWS = Q_TILES * BM;
  static constexpr int CTAS_PER_SM = SINGLE ? 2 : 1;
  static constexpr int CHUNKS = D / 64;
  static constexpr int CHUNK_BYTES = BM * 128;
  static constexpr int TILE_BYTES = BM * D * 2;
  static constexpr int Q_BUFS = D == 64 && KIND != PAGED8 ? 2 : 1;  // 2: the next unit's Q is there when the last S is issued
  static constexpr int SLOTS = SINGLE ? 5 : D == 64 ? 8 : 4;        // K and V tiles in turn
  static constexpr int RAW_BYTES = KIND == PAGED8 ? BN * D : 0;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_KV = OFF_Q + Q_BUFS * Q_TILES * TILE_BYTES;
  static constexpr int OFF_RAW = OFF_KV + SLOTS * TILE_BYTES;  // [K, V]
  static constexpr int OFF_UNITS = OFF_RAW + 2 * RAW_BYTES;    // Entry [UNITS]
  static constexpr int OFF_FLAGS = OFF_UNITS + UNITS * 64;     // uint32 [FLAGS][8]: any, four words of key bits
  static constexpr int OFF_BAR = OFF_FLAGS + (KIND == DENSE ? 0 : FLAGS * 32);
  static constexpr int B_QFULL = 0;                  // [Q_BUFS]
  static constexpr int B_QEMPTY = B_QFULL + 2;       // [Q_BUFS]
  static constexpr int B_QREADY = B_QEMPTY + 2;      // PAGED8: Q in f16
  static constexpr int B_FULL = B_QREADY + 1;        // [SLOTS]
  static constexpr int B_EMPTY = B_FULL + SLOTS;     // [SLOTS]
  static constexpr int B_SFULL = B_EMPTY + SLOTS;    // [2] S_t computed
  static constexpr int B_SFREE = B_SFULL + 2;        // S loaded by the softmax (SINGLE)
  static constexpr int B_PFULL = B_SFREE + 1;        // [2] P_t stored
  static constexpr int B_ODONE = B_PFULL + 2;        // [2] PV_t completed
  static constexpr int B_TAILREQ = B_ODONE + 2;      // a tile with values behind the end has landed
  static constexpr int B_TAIL = B_TAILREQ + 1;       // [2] they are zeroed, by the place of the values (SINGLE: [0])
  static constexpr int B_RAWFULL = B_TAIL + 2;       // [K, V]
  static constexpr int B_RAWEMPTY = B_RAWFULL + 2;
  static constexpr int B_DRAIN = B_RAWEMPTY + 2;     // [2] the last MMAs and commits, one per issuer
  static constexpr int B_TURN = B_DRAIN + 2;         // [2] an issuer's turn
  static constexpr int B_UNITFULL = B_TURN + 2;      // [UNITS]
  static constexpr int B_UNITEMPTY = B_UNITFULL + UNITS;
  static constexpr int NUM_BARS = B_UNITEMPTY + UNITS;
  static constexpr int OFF_SLOT = OFF_BAR + NUM_BARS * 8;
  static constexpr int OFF_ABORT = OFF_SLOT + 4;
  static constexpr int SMEM_BYTES = OFF_ABORT + 4;
  static constexpr uint32_t TMEM_COLS = SINGLE ? 256 : 512;
  // warps: softmax (4 per row tile); units and copies; MMA issuer (SINGLE: of S); tail; SINGLE: PV issuer.
  // PAGED: four more copy pages. PAGED8: four more convert, the third and fourth control warp copy
  static constexpr int SOFTMAX_WARPS = 4 * Q_TILES;
  static constexpr int WARP_LOAD = SOFTMAX_WARPS, WARP_MMA = SOFTMAX_WARPS + 1, WARP_TAIL = SOFTMAX_WARPS + 2,
                       WARP_PV = SOFTMAX_WARPS + 3, WARP_MORE = SOFTMAX_WARPS + 4;
  static constexpr int ISSUERS = SINGLE || KIND == PAGED8 ? 1 : 2;  // of both products; SINGLE: one for each product
  static constexpr int THREADS = 32 * (SOFTMAX_WARPS + 4 + (KIND == DENSE ? 0 : 4));
  // readers of a unit's entry: softmax warps, MMA issuers, tail or copying warps, converting warps
  static constexpr int UNIT_READERS = SOFTMAX_WARPS + (SINGLE ? 2 : ISSUERS) + (KIND == DENSE ? 1 : KIND == PAGED ? 4 : 6);
  static constexpr bool SLEEPY = SINGLE || KIND != DENSE;  // control warps' waits suspend: fewer issue slots taken
  // May find its unit without a list: 5 sequences of 3 to 61 tokens, 8 heads of 64, 5.6 us on the device against 10.6.
  // Not with 8 bits, whose roles crowd the instruction cache: the code alone took the long chunk from 785 to 818 us.
  static constexpr bool LISTLESS = KIND != PAGED8;
  static constexpr int REGS_CONTROL = SINGLE ? 48 : KIND == DENSE ? 80 : KIND == PAGED ? 48 : 56;
  static constexpr int REGS_MORE = KIND == PAGED ? 48 : 40;
  static constexpr int REGS_SOFTMAX = 208;
  static constexpr int LAUNCH_REGS = (65536 / (THREADS * CTAS_PER_SM)) & ~7;
  static_assert(128 * REGS_CONTROL + (KIND == DENSE ? 0 : 128 * REGS_MORE) + 32 * SOFTMAX_WARPS * REGS_SOFTMAX <=
                    THREADS * LAUNCH_REGS,
                "register split");
  static constexpr uint32_t TMEM_P = SINGLE ? BN : 0;  // else P_t over S_t
  static constexpr uint32_t TMEM_O = SINGLE ? BN + BN / 2 : 2 * BN;
  static constexpr uint32_t IDESC_S = KIND == PAGED8 ? idesc_f16_f32(BM, BN, false) : ptx::idesc_bf16_f32(BM, BN, false);
  static constexpr uint32_t IDESC_PV = KIND == PAGED8 ? idesc_f16_f32(BM, D, true) : ptx::idesc_bf16_f32(BM, D, true);
  static_assert(TMEM_O + Q_TILES * D <= TMEM_COLS, "TMEM budget");
  static_assert(OFF_UNITS % 16 == 0 && OFF_BAR % 8 == 0, "alignment");
  static_assert(CTAS_PER_SM * (SMEM_BYTES + 1024) <= 228 * 1024, "shared memory budget");
};

// A place in the ring of key and value tiles and the parity of its phase.
template <int N>
struct RingPos {
  uint32_t s = 0, ph = 0;
  __device__ __forceinline__ void step(uint32_t by) {
    s += by;
    if (s >= N) {
      s -= N;
      ph ^= 1;
    }
  }
};

struct Params {
  plan::Args plan;   // read where there is no list
  int no_list;       // 1: CTA u's one unit is u, and it finds it itself
  plan::Header* head;
  const int2* range;
  const plan::Entry* list;
  uint16_t* out;
  float* lse;                // [T, h_q] or null
  long long out_ts, out_hs;  // elements between tokens, heads
  int h_q, group, tok;       // query heads per key/value head, tokens per row tile
  int causal, window, sinks;
  float scale_log2;
  float* part;  // partial results: per slot [ROWS][D] sums, [ROWS] maxima, [ROWS] row sums
  // pages
  const uint8_t* k_pages;
  const uint8_t* v_pages;
  const int32_t* page_table;
  int max_pages, n_pages, page_size, box_shift;  // boxes of 2^box_shift rows are in one page, in any tile
  int h_kv;
  const float* k_scale;
  const float* v_scale;
  int back;  // keys further before a unit's first token are not for it, unless they are first tokens
  int inject_v_tile;  // INJECT: the values' copying warps give up before this tile
};

__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag, bool sleepy = false) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = ptx::globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (sleepy ? ptx::mbar_try_wait_sleep(bar, parity, 1000u) : ptx::mbar_try_wait(bar, parity)) return true;
    if ((it & 63u) == 0) {
      if (*abort_flag) return false;
      if (ptx::globaltimer_ns() - t0 > kWaitLimitNs) {
        *abort_flag = 1;
        atomicOr(&g_packed_fault_word, FAULT_PACKED);
        return false;
      }
    }
  }
}

// Only while tearing down after an abort.
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = ptx::globaltimer_ns();
  while (!ptx::mbar_try_wait(bar, parity))
    if (ptx::globaltimer_ns() - t0 > kDrainLimitNs) return;
}

// Four-dimensional tiled copy global -> shared, as ptx::tma_load_3d.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* tmap, uint32_t bar, int x, int y, int z, int w,
                                            uint64_t cache_hint) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w), "l"(cache_hint)
      : "memory");
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// Two e4m3 numbers, in bits 7:0 and 15:8 of x, as two f16: exact, NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t x) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((unsigned short)x));
  return r;
}

// Two floats -> packed f16x2 (nearest even); `lo` lands in bits 15:0.
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A word with its lowest n bits set; none for n <= 0, all from 32 on.
__device__ __forceinline__ uint32_t bits_below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

// The key tile of list entry j.
__device__ __forceinline__ int tile_of(const plan::Entry& e, int j) {
  const int l = e.j0 + j;
  return l + (l >= e.n_first ? e.skip : 0);
}

// 16 bytes global -> shared, past L1; with n = 0 zeros, and src is not read.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
// Arrives on `bar` when this thread's copies so far have landed (an arrival that the barrier counts).
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// A copy warp's view of the pages: where the 128 rows of a key tile lie, and their copies into a tile (bf16:
// 128-byte swizzle, a slab per 64 columns; 8 bits: rows of d bytes). Rows come in boxes of
// gcd(page size, 128), which no page border cuts.
// Boxes of 8 rows and more (the swizzle's period) go by TMA, a lane issuing each, smaller and partly filled ones by
// cp.async. With 16 rows a page, TMA against cp.async: 509 tokens over 60001 keys of 8 bits, 64/8 heads of 128,
// 827 us against 1356; 16 prompts' pieces, 16/4 heads of 64, window 1023, 111 against 120. With 8 rows 892
// against 1367 and 113 against 121.
template <int D, int KIND>
struct PageRows {
  static constexpr int ROW = KIND == PAGED8 ? D : 2 * D;  // bytes
  static constexpr int LPR = ROW / 16, RPS = 32 / LPR;    // lanes per row, rows per step of the warp
  static constexpr int PITCH = KIND == PAGED8 ? ROW : 128;
  static constexpr int NONE = INT32_MIN;  // no key there
  const Params& p;
  const int lane, shift;  // a box has 2^shift rows
  const bool ahead;       // 32 boxes, a look-up, cover whole tiles: page numbers are asked for early
  int id = NONE, in = 0, next_id = NONE, next_in = 0;  // of this lane's box: page number, first row in it
  int base = -1;  // lane x: first row in the pool of box x; -1: zeros; -2: bad page (not used without `ahead`)

  __device__ __forceinline__ PageRows(const Params& p_, int lane_)
      : p(p_), lane(lane_), shift(p_.box_shift), ahead(p_.box_shift >= 2) {}
  __device__ __forceinline__ int boxes() const { return BN >> shift; }                     // per tile
  __device__ __forceinline__ int tiles() const { return 1 << (shift >= 2 ? shift - 2 : 0); }  // per look-up

  // The page of the n keys from `key` on (a box, or one row). NONE behind the length, and where all of them lie between
  // the first tokens and the windows of the unit's tokens: such a page may be another sequence's by now and hold
  // anything, and 0 times infinity is NaN.
  __device__ __forceinline__ void look(int key, int n, const plan::Entry& e, int& id_, int& in_) const {
    id_ = NONE;
    in_ = 0;
    if (key < e.str_len && (key + n > e.pos - p.back || key < p.sinks)) {
      const int page = key / p.page_size;
      in_ = key - page * p.page_size;
      id_ = max(p.page_table[(size_t)e.str_row * p.max_pages + page], -1);  // any bad one, but never NONE
    }
  }
  // Page numbers of list entries j .. j + tiles() - 1 of a unit, for take(); nothing waits for them here.
  __device__ __forceinline__ void ask(const plan::Entry& e, int j) {
    const int at = j + (lane >> (7 - shift));
    look(at < e.n ? tile_of(e, at) * BN + ((lane & (boxes() - 1)) << shift) : e.str_len, 1 << shift, e, next_id, next_in);
  }
  __device__ __forceinline__ void take() {
    id = next_id;
    in = next_in;
  }
  __device__ __forceinline__ int place(int id_, int in_, int hk) const {
    if (id_ == NONE) return -1;
    if (id_ < 0 || id_ >= p.n_pages) return -2;
    return (id_ * p.h_kv + hk) * p.page_size + in_;
  }
  // The boxes of list entry j.
  __device__ __forceinline__ void tile(int j, const plan::Entry& e) {
    if (!ahead) return;
    const int from = ((j & (tiles() - 1)) << (7 - shift)) + (lane & (boxes() - 1));
    base = place(__shfl_sync(0xffffffffu, id, from), __shfl_sync(0xffffffffu, in, from), e.hk);
  }
  // Without `ahead` (pages of one or two rows, or odd ones): row 32 k + lane of the tile.
  __device__ __forceinline__ int row_of(int k, int key0, const plan::Entry& e) const {
    int i, r;
    look(key0 + k * 32 + lane, 1, e, i, r);
    return place(i, r, e.hk);
  }
  // The bits of keys of bad pages go to fl[1 .. 4], and whether there are any to fl[0].
  __device__ __forceinline__ void mark(uint32_t* fl, int key0, const plan::Entry& e) const {
    bool bad = ahead && lane < boxes() && base == -2;
    if (!ahead)
      for (int k = 0; k < 4; ++k) bad |= row_of(k, key0, e) == -2;
    const bool any = __any_sync(0xffffffffu, bad);
    if (lane < 5) *(volatile uint32_t*)(fl + lane) = lane == 0 && any ? 1u : 0u;
    __syncwarp();
    if (any) {  // rare
      if (ahead) {
        if (bad)
          for (int key = lane << shift; key < (lane + 1) << shift; ++key) atomicOr(fl + 1 + (key >> 5), 1u << (key & 31));
      } else {
        for (int k = 0; k < 4; ++k)
          if (row_of(k, key0, e) == -2) atomicOr(fl + 1 + k, 1u << lane);
      }
    }
    __syncwarp();
  }
  static __device__ __forceinline__ uint32_t offset(int r, int c) {  // of row r's 16-byte unit c in the tile
    if constexpr (KIND == PAGED8) return r * ROW + c * 16;
    else return (c >> 3) * (BM * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
  }
  // n rows from row r of the tile on, of one box that starts at row `row` of the pool; n a multiple of 8, of which
  // `there` exist. Eight rows at a time: the swizzle repeats.
  __device__ __forceinline__ void copy_box(uint32_t dst, const uint8_t* pool, int r, int row, int n, int there) const {
    const int c = lane % LPR, r_lane = lane / LPR;
    const uint8_t* src = pool + (size_t)(max(row, 0) + r_lane) * ROW + c * 16;
    const uint32_t to = dst + r * PITCH;
#pragma unroll 2
    for (int st = 0; st < n; st += 8) {
#pragma unroll
      for (int y = 0; y < 8; y += RPS)
        copy16(to + st * PITCH + offset(y + r_lane, c), src + (st + y) * ROW, st + y + r_lane < there ? 16 : 0);
    }
  }
  // Rows [r0, r0 + rows) of the tile, 64 or 128 of them. Every lane arrives on `full` when its copies have
  // landed, and lane 0 once more, for the TMA copies' bytes.
  __device__ __forceinline__ void copy(uint32_t dst, const uint8_t* pool, const CUtensorMap* map, uint32_t full, int key0,
                                       const plan::Entry& e, int r0, int rows) const {
    const int len = e.str_len;
    if (p.box_shift >= kTmaShift) {
      // boxes whose rows are all there: by TMA, a lane each (here a box may be cut at r0)
      const int n = min(1 << shift, rows), r = r0 + lane * n;
      const bool mine = lane * n < rows;
      const int first = __shfl_sync(0xffffffffu, base, (r >> shift) & 31);
      const int row = first < 0 ? first : first + (r & ((1 << shift) - 1));
      const bool whole = mine && row >= 0 && key0 + r + n <= len;
      const uint32_t by_tma = __ballot_sync(0xffffffffu, whole);
      if (lane == 0) ptx::mbar_arrive_expect_tx(full, __popc(by_tma) * n * ROW);
      __syncwarp();
      if (whole) {
        for (int x = 0; x < (KIND == PAGED8 ? 1 : D / 64); ++x)
          ptx::tma_load_2d(dst + r * PITCH + x * (BM * 128), map, full, x * 64, row, ptx::policy_evict_last());
      }
      __syncwarp();
      for (uint32_t rest = __ballot_sync(0xffffffffu, mine && !whole); rest; rest &= rest - 1) {
        const int i = __ffs(rest) - 1, row_i = __shfl_sync(0xffffffffu, row, i);
        copy_box(dst, pool, r0 + i * n, row_i, n, row_i < 0 ? 0 : len - key0 - r0 - i * n);
      }
      copies_arrive(full);
      return;
    }
    const int c = lane % LPR, r_lane = lane / LPR;
    for (int k = r0 >> 5; k < (r0 + rows) >> 5; ++k) {  // small boxes, row by row
      const int rows32 = ahead ? base : row_of(k, key0, e);
      for (int st = 0; st < 32; st += RPS) {
        const int r = k * 32 + st + r_lane;
        int row = __shfl_sync(0xffffffffu, rows32, ahead ? r >> shift : r & 31);
        if (ahead && row >= 0) row += r & ((1 << shift) - 1);
        const bool there = row >= 0 && key0 + r < len;
        copy16(dst + offset(r, c), pool + (size_t)(there ? row : 0) * ROW + c * 16, there ? 16 : 0);
      }
    }
    copies_arrive(full);
    if (lane == 0) ptx::mbar_arrive(full);
  }
};

// INJECT is a test-only instantiation over pages: the copying warps of V give up before tile p.inject_v_tile, as if
// a wait had run out there, with whatever copies are in flight. INJECT = false compiles to the plain kernel.
template <int D, int KIND, bool INJECT>
__global__ void __launch_bounds__(Cfg<D, KIND>::THREADS, Cfg<D, KIND>::CTAS_PER_SM)
    attn_packed_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const Params p) {
  using C = Cfg<D, KIND>;
  constexpr bool SINGLE = C::SINGLE;
  constexpr bool RAW = KIND == PAGED8;
  using Pos = RingPos<C::SLOTS>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((ptx::smem_u32(smem) & 1023u) != 0) {
    if (threadIdx.x == 0) atomicOr(&g_packed_fault_word, FAULT_PACKED);
    return;
  }
  const uint32_t s_base = ptx::smem_u32(smem);
  auto s_q = [&](uint32_t b) -> uint32_t { return s_base + C::OFF_Q + b * (C::Q_TILES * C::TILE_BYTES); };
  auto s_kv = [&](uint32_t slot) -> uint32_t { return s_base + C::OFF_KV + slot * C::TILE_BYTES; };
  auto bar = [&](int i) -> uint32_t { return s_base + C::OFF_BAR + 8u * i; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_ABORT);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_SLOT);
  const plan::Entry* units = reinterpret_cast<const plan::Entry*>(smem + C::OFF_UNITS);
  volatile uint32_t* flags = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_FLAGS);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // uniform: see the issuing warps

  if (threadIdx.x == 0) {
    for (int b = 0; b < C::Q_BUFS; ++b) {
      ptx::mbar_init(bar(C::B_QFULL + b), 1);
      ptx::mbar_init(bar(C::B_QEMPTY + b), SINGLE ? 4 : C::ISSUERS);  // the softmax warps, or the last S
    }
    ptx::mbar_init(bar(C::B_QREADY), 2 * BM);
    for (int s = 0; s < C::SLOTS; ++s) {
      // converting warps; two copy warps' lanes and their lanes 0 again; or the copies' bytes
      ptx::mbar_init(bar(C::B_FULL + s), RAW ? 4 : KIND == PAGED ? 66 : 1);
      ptx::mbar_init(bar(C::B_EMPTY + s), C::ISSUERS);
    }
    for (int t = 0; t < 2; ++t) {
      // pages: the issuer arrives besides its commit, so that the page bits, written before the
      // copies, are ordered before the softmax reads them
      ptx::mbar_init(bar(C::B_SFULL + t), KIND == DENSE ? 1 : 2);
      ptx::mbar_init(bar(C::B_PFULL + t), BM);
      ptx::mbar_init(bar(C::B_ODONE + t), 1);
      ptx::mbar_init(bar(C::B_RAWFULL + t), 33);
      ptx::mbar_init(bar(C::B_RAWEMPTY + t), 4);
      ptx::mbar_init(bar(C::B_DRAIN + t), 1);
      ptx::mbar_init(bar(C::B_TURN + t), 1);
      ptx::mbar_init(bar(C::B_TAIL + t), 1);
    }
    ptx::mbar_init(bar(C::B_SFREE), BM);
    ptx::mbar_init(bar(C::B_TAILREQ), 1);
    for (int u = 0; u < UNITS; ++u) {
      ptx::mbar_init(bar(C::B_UNITFULL + u), 1);
      ptx::mbar_init(bar(C::B_UNITEMPTY + u), C::UNIT_READERS);
    }
    *abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == C::WARP_MMA) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), C::TMEM_COLS);
    ptx::tmem_relinquish();
  }
  if (warp == C::WARP_LOAD && lane == 0) {
    ptx::prefetch_tmap(&tm_q);
    ptx::prefetch_tmap(&tm_k);
    ptx::prefetch_tmap(&tm_v);
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  ptx::grid_dep_wait();  // the plan is written
  ptx::grid_dep_launch();

  // The copy warp passes the units' entries on through a ring of UNITS places; every other warp
  // runs through them in that order, each at its own pace. n < 0: no more units.
  auto unit_wait = [&](uint32_t un) -> bool { return wait_bar(bar(C::B_UNITFULL + un % UNITS), (un / UNITS) & 1, abort_flag, C::SLEEPY); };
  auto unit_done = [&](uint32_t un) { ptx::mbar_arrive(bar(C::B_UNITEMPTY + un % UNITS)); };
  // The issuing warps run their loops together, and one lane issues: with control flow and operands that are
  // the same for the warp, descriptors and addresses are computed in uniform registers, where the MMA
  // takes them from. (In a branch of one thread every operand is moved there first; an MMA then costs the
  // issuing warp some 90 cycles between the softmax warps' instructions.)
  auto uniform = [](uint32_t x) -> uint32_t { return __shfl_sync(0xffffffffu, x, 0); };
  auto wait_warp = [&](uint32_t b, uint32_t parity, bool sleepy = false) -> bool {
    return __all_sync(0xffffffffu, wait_bar(b, parity, abort_flag, sleepy));
  };
  const uint32_t issue = lane == 0;
  bool ok = true;

  // A copying warp's part of K (kv = 0) or V (1) of all units: rows [128 part / parts, + 128 / parts) of every
  // tile. The first of K's also leaves the bits of the keys whose pages are not there.
  auto page_copies = [&](int kv, int part, int parts) -> bool {
    bool good = true;
    PageRows<D, KIND> pages(p, lane);
    const uint8_t* pool = kv ? p.v_pages : p.k_pages;
    uint32_t n_kv = 0;
    Pos pos;
    pos.step(kv);
    bool asked = false;  // the unit's first look-up is done already
    for (uint32_t un = 0;; ++un) {
      good = __all_sync(0xffffffffu, unit_wait(un));
      if (!good) break;
      const plan::Entry& e = units[un % UNITS];
      const int n = e.n;
      if (n < 0) break;
      if (n > 0 && pages.ahead) {
        if (!asked) pages.ask(e, 0);
        pages.take();
      }
      asked = false;  // what was asked for a unit without keys is of no use to the one after it
      for (int j = 0; j < n; ++j, ++n_kv) {
        if (pages.ahead && (j & (pages.tiles() - 1)) == 0) {
          if (j + pages.tiles() < n) {
            pages.ask(e, j + pages.tiles());
          } else if (__all_sync(0xffffffffu, ptx::mbar_try_wait(bar(C::B_UNITFULL + (un + 1) % UNITS), ((un + 1) / UNITS) & 1))) {
            pages.ask(units[(un + 1) % UNITS], 0);  // the next unit is known already
            asked = true;
          }
        }
        const int key0 = tile_of(e, j) * BN;
        const uint32_t full = bar(RAW ? C::B_RAWFULL + kv : C::B_FULL + (int)pos.s);
        pages.tile(j, e);
        if (INJECT && kv == 1 && n_kv == (uint32_t)p.inject_v_tile) {
          *abort_flag = 1;
          if (lane == 0) atomicOr(&g_packed_fault_word, FAULT_PACKED);
          good = false;
          break;
        }
        good = __all_sync(0xffffffffu, wait_bar(bar(RAW ? C::B_RAWEMPTY + kv : C::B_EMPTY + (int)pos.s),
                                                (RAW ? n_kv & 1 : pos.ph) ^ 1, abort_flag, true));
        if (!good) break;
        if (kv == 0 && part == 0) pages.mark(const_cast<uint32_t*>(flags) + (n_kv % FLAGS) * 8, key0, e);
        pages.copy(RAW ? s_base + C::OFF_RAW + kv * C::RAW_BYTES : s_kv(pos.s), pool, kv ? &tm_v : &tm_k, full, key0, e,
                   part * (BN / parts), BN / parts);
        if (pages.ahead && ((j + 1) & (pages.tiles() - 1)) == 0 && j + 1 < n) pages.take();
        pos.step(2);
      }
      if (!good) break;
      __syncwarp();
      if (lane == 0) unit_done(un);
      __syncwarp();
    }
    copies_wait();
    if (!good && lane == 0) {
      // boxes in flight must land before this CTA's shared memory goes away: the phases that this warp armed last. (bf16:
      // one that the other half's warp has not armed as well does not end; the limit is then the boxes' time.)
      if (RAW) {
        if (n_kv > 0) drain_wait(bar(C::B_RAWFULL + kv), (n_kv - 1) & 1);
      } else {
#pragma unroll 1
        for (uint32_t x = n_kv < C::SLOTS / 2 ? 0 : n_kv - C::SLOTS / 2; x < n_kv; ++x)
          drain_wait(bar(C::B_FULL + kv + (int)(2 * x % C::SLOTS)), (2 * x / C::SLOTS) & 1);
      }
    }
    __syncwarp();
    return good;
  };

  if (warp < C::SOFTMAX_WARPS) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_SOFTMAX));
    // ================================================================ softmax
    const int t = warp >> 2;               // row tile
    const int r = (warp & 3) * 32 + lane;  // row of the tile = TMEM lane
    const int rt = r / p.group;            // its token
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lane_off + t * BN;
    const uint32_t t_p = tmem + lane_off + C::TMEM_P + t * BN;
    const uint32_t t_o = tmem + lane_off + C::TMEM_O + t * D;
    uint32_t cnt0 = 0;   // key tiles of this row tile so far
    uint32_t tiles = 0;  // key tiles of the units so far (pages: their bits' place)
    uint32_t n_q = 0;    // units with keys so far
    for (uint32_t un = 0;; ++un) {
      ok = __all_sync(0xffffffffu, unit_wait(un));
      if (!ok) break;
      // the entry is read from shared memory where it is used: the score tile and P leave no
      // registers to hold it
      const plan::Entry& e = units[un % UNITS];
      if (e.n < 0) break;
      const int lo = t ? e.lo1 : e.lo0, n_tiles = (t ? e.hi1 : e.hi0) - lo;
      float c = p.scale_log2;
      if constexpr (RAW) {
        c *= p.k_scale[e.hk];
        if (e.n > 0) {
          // this row of Q as f16, times the power of two that brings its largest entry to 2^14:
          // bf16's eight bits fit, and entries below 2^-28 of the largest are rounded to 2^-39 of it
          ok = __all_sync(0xffffffffu, wait_bar(bar(C::B_QFULL), n_q & 1, abort_flag));
          if (!ok) break;
          if (t * p.tok < e.own_n) {
            const uint32_t row = s_q(0) + t * C::TILE_BYTES + r * 128;
            float top = 0.0f;
#pragma unroll
            for (int u = 0; u < D / 8; ++u) {
              const uint4 w = ld_shared_v4(row + (u >> 3) * C::CHUNK_BYTES + (((u & 7) ^ (r & 7)) << 4));
              const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int i = 0; i < 4; ++i)
                top = ptx::max3(top, fabsf(__uint_as_float(in[i] << 16)), fabsf(__uint_as_float(in[i] & 0xffff0000u)));
            }
            // exponents of two normal numbers; zero, subnormal, infinite rows stay as they are
            const int field = (int)(__float_as_uint(top) >> 23);
            const int up = field == 0 || field >= 255 ? 0 : min(max(127 + 14 - field, -126), 126);
            const float mul = __uint_as_float((uint32_t)(127 + up) << 23);
            c *= __uint_as_float((uint32_t)(127 - up) << 23);
#pragma unroll
            for (int u = 0; u < D / 8; ++u) {
              const uint32_t at = row + (u >> 3) * C::CHUNK_BYTES + (((u & 7) ^ (r & 7)) << 4);
              const uint4 w = ld_shared_v4(at);
              const uint32_t in[4] = {w.x, w.y, w.z, w.w};
              uint32_t o[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                o[i] = pack_f16x2(__uint_as_float(in[i] << 16) * mul, __uint_as_float(in[i] & 0xffff0000u) * mul);
              ptx::st_shared_v4(at, o[0], o[1], o[2], o[3]);
            }
            ptx::fence_proxy_async_smem();
          }
          ptx::mbar_arrive(bar(C::B_QREADY));
        }
      }
      if (e.n > 0) ++n_q;
      // list entries [inner, outer) of this row tile are legal for all of its rows; the others need the mask
      int inner = 0, outer;
      {
        const int pos_lo = e.pos + t * p.tok, pos_hi = pos_lo + min(e.own_n - t * p.tok, p.tok) - 1;
        int end = e.str_len;
        if (p.causal) end = min(end, pos_lo + 1);
        if (p.window >= 0) {
          if (!p.causal) end = min(end, pos_lo + p.window + 1);
          inner = max(pos_hi - p.window + BN - 1, 0) / BN - e.skip;
          if (e.skip > 0) inner = max(inner, e.n_first);  // the first keys' tiles are masked
        }
        outer = max(end, 0) / BN - e.skip - e.j0 - lo;
        inner -= p.window >= 0 ? e.j0 + lo : 0;
      }
      float m_ref = -INFINITY;  // reference maximum, log2 units
      float l = 0.0f;           // sum of 2^(c s - m_ref + kBias)
      for (int j = 0; j < n_tiles; ++j) {
        const uint32_t cnt = cnt0 + j;
        ok = __all_sync(0xffffffffu, wait_bar(bar(C::B_SFULL + t), cnt & 1, abort_flag));
        if (!ok) break;
        ptx::tc_fence_after();
        uint32_t sr[4][32];
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) ptx::tmem_ld32(t_s + q4 * 32, sr[q4]);
        ptx::tmem_wait_ld();
        if constexpr (SINGLE) {  // S is in registers
          ptx::tc_fence_before();
          ptx::mbar_arrive_after(bar(C::B_SFREE), __uint_as_float(sr[3][31]));
        }
        bool masked = j < inner || j >= outer;
        volatile const uint32_t* fl = flags + ((tiles + lo + j) % FLAGS) * 8;
        if constexpr (KIND != DENSE) masked = masked || fl[0];  // keys of pages that are not there
        if (masked) {
          const int key0 = tile_of(e, lo + j) * BN;
          const int pos = e.pos + t * p.tok + rt;
          int lim = e.str_len - key0;  // columns [first, lim) are legal, and those below `sink`
          if (p.causal) lim = min(lim, pos + 1 - key0);
          int first = 0, sink = 0;
          if (p.window >= 0) {
            if (!p.causal) lim = min(lim, pos + p.window + 1 - key0);
            first = pos - p.window - key0;
            sink = p.sinks - key0;
          }
          // as bits, a word for 32 columns
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) {
            uint32_t legal = bits_below(lim - q4 * 32) & (~bits_below(first - q4 * 32) | bits_below(sink - q4 * 32));
            if constexpr (KIND != DENSE) legal &= fl[0] ? ~fl[1 + q4] : ~0u;
#pragma unroll
            for (int x = 0; x < 32; ++x)
              if (!((legal >> x) & 1u)) sr[q4][x] = __float_as_uint(-INFINITY);
          }
        }
        uint32_t pk[2][32];
        auto col = [&](int a, int x) { return __uint_as_float(sr[a >> 1][(a & 1) * 16 + x]); };
        // row maximum: eight independent chains of three-way maxima
        auto row_max = [&]() -> float {
          float mc[8];
#pragma unroll
          for (int a = 0; a < 8; ++a) {
            mc[a] = fmaxf(col(a, 0), col(a, 1));
#pragma unroll
            for (int x = 2; x < 16; x += 2) mc[a] = ptx::max3(mc[a], col(a, x), col(a, x + 1));
          }
          return ptx::max3(ptx::max3(mc[0], mc[1], mc[2]), ptx::max3(mc[3], mc[4], mc[5]), fmaxf(mc[6], mc[7])) * c;
        };
        // P, rounded for the tensor cores (the row sum takes it unrounded). bf16: each weight moves by at
        // most 2^-8 of itself, independently, less than the output's own rounding in the mean. f16, with
        // 8-bit pages: 2^-11, and P is 2^7 times the weight, so that 2^-32 of the largest still counts
        auto exps = [&](float m_now) -> float {
          const float m_use = ((m_now == -INFINITY) ? 0.0f : m_now) - (RAW ? kBias : 0.0f);
          const uint64_t c2 = ptx::f2_pack(c, c);
          const uint64_t negm2 = ptx::f2_pack(-m_use, -m_use);
          uint64_t part[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4)
#pragma unroll
            for (int x = 0; x < 32; x += 2) {
              const uint64_t sx = ptx::f2_pack(__uint_as_float(sr[q4][x]), __uint_as_float(sr[q4][x + 1]));
              float a0, a1;
              ptx::f2_unpack(ptx::f2_fma(sx, c2, negm2), a0, a1);
              const float p0 = ptx::ex2(a0), p1 = ptx::ex2(a1);
              part[q4] = ptx::f2_add(part[q4], ptx::f2_pack(p0, p1));
              pk[q4 >> 1][(q4 & 1) * 16 + (x >> 1)] = RAW ? pack_f16x2(p0, p1) : ptx::pack_bf16x2(p0, p1);
            }
          float l0, l1;
          ptx::f2_unpack(ptx::f2_add(ptx::f2_add(part[0], part[1]), ptx::f2_add(part[2], part[3])), l0, l1);
          return l0 + l1;
        };
        bool pv_done = j == 0;  // the PV before this tile is known to be complete
        // O, holding the PVs so far, to the reference that the rows which grew now have
        auto rescale = [&](float alpha) -> bool {
          if (!__all_sync(0xffffffffu, wait_bar(bar(C::B_ODONE + t), (cnt - 1) & 1, abort_flag))) return false;
          pv_done = true;
          ptx::tc_fence_after();
#pragma unroll
          for (int q4 = 0; q4 < D / 32; ++q4) {
            uint32_t o[32];
            ptx::tmem_ld32(t_o + q4 * 32, o);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * alpha);
            ptx::tmem_st32(t_o + q4 * 32, o);
          }
          return true;
        };
        if constexpr (SINGLE) {
          // after the first tile, exponentials against the current reference, before the tile's
          // maximum is known: a sum of at most 2^7 shows that no score exceeds the reference by
          // the threshold; only a larger one (or NaN, or a reference still at -inf) needs the maximum
          if (j == 0) {
            m_ref = row_max();
            l = exps(m_ref);
          } else {
            float l_tile = exps(m_ref);
            float m_tile = m_ref;
            bool grow = false;
            if (__any_sync(0xffffffffu, !(l_tile <= 128.0f) || m_ref == -INFINITY)) {
              m_tile = row_max();
              grow = m_tile > m_ref + kRescaleThreshold;
            }
            if (__any_sync(0xffffffffu, grow)) {
              float alpha = 1.0f;
              if (grow) {
                alpha = ptx::ex2(m_ref - m_tile);
                l *= alpha;
                m_ref = m_tile;
              }
              if (!(ok = rescale(alpha))) break;
              l_tile = exps(m_ref);
            }
            l += l_tile;
          }
        } else {
          const float m_tile = row_max();
          const bool grow = m_tile > m_ref + kRescaleThreshold;
          float alpha = 1.0f;
          if (grow) {
            alpha = ptx::ex2(m_ref - m_tile);  // 0 when m_ref is still -inf
            l *= alpha;
            m_ref = m_tile;
          }
          if (j > 0 && __any_sync(0xffffffffu, grow) && !(ok = rescale(alpha))) break;
          l += exps(m_ref);
        }
        if (SINGLE && !pv_done) {
          // P is still the A operand of the PV before until that completes
          ok = __all_sync(0xffffffffu, wait_bar(bar(C::B_ODONE + t), (cnt - 1) & 1, abort_flag));
          if (!ok) break;
          ptx::tc_fence_after();
        }
        ptx::tmem_st32(t_p, pk[0]);
        ptx::tmem_st32(t_p + 32, pk[1]);
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        ptx::mbar_arrive(bar(C::B_PFULL + t));
      }
      if (!ok) break;

      // ---------------------------------------------------------------- this unit's rows
      const bool row_valid = rt < min(e.own_n - t * p.tok, p.tok);
      if (n_tiles > 0) {
        ok = __all_sync(0xffffffffu, wait_bar(bar(C::B_ODONE + t), (cnt0 + n_tiles - 1) & 1, abort_flag));
        if (!ok) break;
        ptx::tc_fence_after();
      }
      cnt0 += n_tiles;
      tiles += e.n;
      if (e.slot >= 0) {
        // a piece: unnormalised sums, their reference, the row sum
        float* part = p.part + (size_t)e.slot * (C::ROWS * (D + 2)) + (size_t)(t * BM + r) * D;
        float* stat = p.part + (size_t)e.slot * (C::ROWS * (D + 2)) + (size_t)C::ROWS * D + t * BM + r;
#pragma unroll
        for (int q4 = 0; q4 < D / 32; ++q4) {
          uint32_t o[32];
          if (n_tiles > 0) {
            ptx::tmem_ld32(t_o + q4 * 32, o);
            ptx::tmem_wait_ld();
          } else {
#pragma unroll
            for (int x = 0; x < 32; ++x) o[x] = 0u;
          }
          if (row_valid) {
#pragma unroll
            for (int x = 0; x < 8; ++x)
              reinterpret_cast<uint4*>(part + q4 * 32)[x] = make_uint4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
          }
          __syncwarp();
        }
        if (row_valid) {
          stat[0] = m_ref - (RAW ? kBias : 0.0f);
          stat[C::ROWS] = l;
        }
      } else {
        const float v_mul = RAW ? p.v_scale[e.hk] : 1.0f;
        const float inv = l == 0.0f ? 0.0f : v_mul / l;  // no legal key: zeros
        const long long row = (long long)e.own_row + t * p.tok + rt;
        const int head_q = e.hk * p.group + r - rt * p.group;
        const long long at = row_valid ? row * p.out_ts + head_q * p.out_hs : -1;
        const uint32_t stage = s_q((n_q - 1) % C::Q_BUFS) + (warp & 3) * 4096;
#pragma unroll
        for (int c64 = 0; c64 < D / 64; ++c64) {
          uint32_t w[32];
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t o[32];
            if (n_tiles > 0) {
              ptx::tmem_ld32(t_o + c64 * 64 + half * 32, o);
              ptx::tmem_wait_ld();
            } else {
#pragma unroll
              for (int x = 0; x < 32; ++x) o[x] = 0u;
            }
#pragma unroll
            for (int x = 0; x < 16; ++x)
              w[half * 16 + x] = ptx::pack_bf16x2(__uint_as_float(o[2 * x]) * inv, __uint_as_float(o[2 * x + 1]) * inv);
          }
          if (SINGLE && e.n > 0) {
            // through the unit's Q, which no S reads any more (16-byte units swizzled by the row), so that eight
            // lanes store one row's 128 bytes: a lane's own row would be 16 bytes of 32 lines in every store
            // (64 x 256 tokens, 16 heads: 51.0 -> 43.7 us; at d = 128, through a place of its own, 1 to 8 % slower)
#pragma unroll
            for (int u = 0; u < 8; ++u)
              ptx::st_shared_v4(stage + lane * 128 + ((u ^ (lane & 7)) << 4), w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int from = i * 4 + (lane >> 3);
              const long long to = __shfl_sync(0xffffffffu, at, from);
              const uint4 v = ld_shared_v4(stage + from * 128 + (((lane & 7) ^ (from & 7)) << 4));
              if (to >= 0) *reinterpret_cast<uint4*>(p.out + to + c64 * 64 + (lane & 7) * 8) = v;
            }
          } else {
            if (row_valid) {
              uint4* dst = reinterpret_cast<uint4*>(p.out + at + c64 * 64);
#pragma unroll
              for (int x = 0; x < 8; ++x) dst[x] = make_uint4(w[4 * x], w[4 * x + 1], w[4 * x + 2], w[4 * x + 3]);
            }
            __syncwarp();
          }
        }
        if (row_valid && p.lse)
          p.lse[row * p.h_q + head_q] =
              l == 0.0f ? -INFINITY : (m_ref - (RAW ? kBias : 0.0f) + __log2f(l)) * 0.69314718055994530942f;
      }
      if (SINGLE && e.n > 0) ptx::fence_proxy_async_smem();  // Q's place: before the copies of another Q
      __syncwarp();
      if (lane == 0) {
        if (SINGLE && e.n > 0) ptx::mbar_arrive(bar(C::B_QEMPTY + (n_q - 1) % C::Q_BUFS));
        unit_done(un);
      }
    }
  } else if (KIND == PAGED && warp >= C::WARP_MORE) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_MORE));
    // ================================================================ pages: two warps for K, two for V
    ok = page_copies((warp - C::WARP_MORE) >> 1, (warp - C::WARP_MORE) & 1, 2);
  } else if (RAW && warp >= C::WARP_MORE) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_MORE));
    // ================================================================ 8 bits to f16
    // Sixteen numbers per thread and step: D / 16 lanes a row.
    const int id = threadIdx.x - 32 * C::WARP_MORE;
    constexpr int LPR = D / 16, STEP = 128 / LPR;  // lanes per row, rows per step
    const int unit = ((id % LPR) & 3) * 2;
    const bool swap = D == 128 && (id & 4) != 0;
    uint32_t n_raw = 0;
    Pos pos;
    for (uint32_t un = 0;; ++un) {
      ok = __all_sync(0xffffffffu, unit_wait(un));
      if (!ok) break;
      const plan::Entry& e = units[un % UNITS];
      const int n = e.n;
      if (n < 0) break;
      for (int j = 0; j < n && ok; ++j, ++n_raw) {
        for (int kv = 0; kv < 2; ++kv, pos.step(1)) {
          ok = __all_sync(0xffffffffu, wait_bar(bar(C::B_RAWFULL + kv), n_raw & 1, abort_flag, true) &&
                                           wait_bar(bar(C::B_EMPTY + pos.s), pos.ph ^ 1, abort_flag, true));
          if (!ok) break;
          const uint32_t src = s_base + C::OFF_RAW + kv * C::RAW_BYTES + (id / LPR) * D + (id % LPR) * 16;
          const uint32_t slab = s_kv(pos.s) + ((id % LPR) >> 2) * C::CHUNK_BYTES;
#pragma unroll 1
          for (int r0 = 0; r0 < BN; r0 += STEP) {
            const int r = r0 + id / LPR;
            const uint4 w = ld_shared_v4(src + r0 * D);
            const uint32_t lo[4] = {e4m3_pair(w.x), e4m3_pair(w.x >> 16), e4m3_pair(w.y), e4m3_pair(w.y >> 16)};
            const uint32_t hi[4] = {e4m3_pair(w.z), e4m3_pair(w.z >> 16), e4m3_pair(w.w), e4m3_pair(w.w >> 16)};
            // d = 128: a row's lanes store their two units in opposite orders in the two slabs, so that eight
            // lanes' units lie in eight different bank groups (at d = 64 their two rows' swizzles see to it)
            const uint32_t row = slab + r * 128, first = swap ? 1 : 0;
            ptx::st_shared_v4(row + (((unit + first) ^ (r & 7)) << 4), swap ? hi[0] : lo[0], swap ? hi[1] : lo[1],
                              swap ? hi[2] : lo[2], swap ? hi[3] : lo[3]);
            ptx::st_shared_v4(row + (((unit + 1 - first) ^ (r & 7)) << 4), swap ? lo[0] : hi[0], swap ? lo[1] : hi[1],
                              swap ? lo[2] : hi[2], swap ? lo[3] : hi[3]);
          }
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            ptx::mbar_arrive(bar(C::B_RAWEMPTY + kv));
            ptx::mbar_arrive(bar(C::B_FULL + pos.s));
          }
          __syncwarp();
        }
      }
      if (!ok) break;
      if (lane == 0) unit_done(un);
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_CONTROL));
    if (warp == C::WARP_LOAD) {
      // ================================================================ units and copies
      const uint64_t pol_q = ptx::policy_evict_first();
      const uint64_t pol_kv = ptx::policy_evict_last();
      plan::Header head = {};
      const bool no_list = C::LISTLESS && p.no_list;
      if (!no_list) head = *p.head;
      plan::Turn turn(head, p.range, p.h_kv);
      auto next_unit = [&]() -> int { return __shfl_sync(0xffffffffu, lane == 0 ? turn.next(p.head) : 0, 0); };
      auto word_of = [&](int u) -> int { return turn.word(p.list, u, lane & 15); };
      // lane x: word x of the entry; all -1: no more units
      int word = no_list ? plan::word_without_list(p.plan, blockIdx.x) : word_of(next_unit());
      uint32_t n_q = 0;   // units with keys so far
      Pos pos;
      for (uint32_t un = 0;; ++un) {
        ok = __all_sync(0xffffffffu, wait_bar(bar(C::B_UNITEMPTY + un % UNITS), ((un / UNITS) & 1) ^ 1, abort_flag, C::SLEEPY));
        if (!ok) break;
        if (lane < 16) reinterpret_cast<int*>(smem + C::OFF_UNITS)[(un % UNITS) * 16 + lane] = word;
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(C::B_UNITFULL + un % UNITS));
        const int n = __shfl_sync(0xffffffffu, word, 9);
        if (n < 0) break;
        word = no_list ? -1 : word_of(next_unit());
        const plan::Entry& e = units[un % UNITS];  // stays: this warp alone replaces it
        if (n > 0) {
          const uint32_t qb = n_q % C::Q_BUFS;
          ok = __all_sync(0xffffffffu, wait_bar(bar(C::B_QEMPTY + qb), ((n_q / C::Q_BUFS) & 1) ^ 1, abort_flag, C::SLEEPY));
          if (!ok) break;
          if (lane == 0) {
            const int n_qt = e.own_n > p.tok ? 2 : 1;
            ptx::mbar_arrive_expect_tx(bar(C::B_QFULL + qb), n_qt * p.tok * p.group * 128 * C::CHUNKS);
            for (int t = 0; t < n_qt; ++t)
              for (int c = 0; c < C::CHUNKS; ++c)
                tma_load_4d(s_q(qb) + t * C::TILE_BYTES + c * C::CHUNK_BYTES, &tm_q, bar(C::B_QFULL + qb), c * 64, 0,
                            e.own_row + t * p.tok, e.hk, pol_q);
          }
          ++n_q;
        }
        for (int j = 0; KIND == DENSE && j < n && ok; ++j) {
          const int key0 = tile_of(e, j) * BN;
          for (int kv = 0; kv < 2; ++kv) {
            ok = __all_sync(0xffffffffu, wait_bar(bar(C::B_EMPTY + pos.s), pos.ph ^ 1, abort_flag, SINGLE));
            if (!ok) break;
            if (lane == 0) {
              ptx::mbar_arrive_expect_tx(bar(C::B_FULL + pos.s), C::TILE_BYTES);
              for (int c = 0; c < C::CHUNKS; ++c)
                ptx::tma_load_3d(s_kv(pos.s) + c * C::CHUNK_BYTES, kv ? &tm_v : &tm_k, bar(C::B_FULL + pos.s), c * 64,
                                 e.str_row + key0, e.hk, pol_kv);
            }
            pos.step(1);
          }
        }
        if (!ok) break;
      }
      if (!ok && lane == 0) {
        // copies in flight must land before this CTA's shared memory goes away: every barrier's last
        // phase that was armed, told by its parity after the last use of the slot
        for (int b = 0; b < C::Q_BUFS; ++b)
          if (n_q > (uint32_t)b) drain_wait(bar(C::B_QFULL + b), ((n_q - 1 - b) / C::Q_BUFS) & 1);
        if (KIND == DENSE) {
          for (int s = 0; s < C::SLOTS; ++s) drain_wait(bar(C::B_FULL + s), s < (int)pos.s ? pos.ph : pos.ph ^ 1);
        }
      }
      __syncwarp();
    } else if (SINGLE && warp == C::WARP_MMA) {
      // ================================================================ S = Q K^T (one row tile)
      {
        const uint32_t t_mem = uniform(tmem);
        uint32_t n_q = 0, tiles = 0;
        Pos pos;
        for (uint32_t un = 0;; ++un) {
          if (!(ok = __all_sync(0xffffffffu, unit_wait(un)))) break;
          const int n = (int)uniform(units[un % UNITS].n);
          if (issue) unit_done(un);
          if (n < 0) break;
          if (n == 0) continue;
          const uint32_t qb = n_q % C::Q_BUFS, q_tile = s_q(qb);
          ok = wait_warp(bar(C::B_QFULL + qb), (n_q / C::Q_BUFS) & 1, true);
          ++n_q;
          for (int j = 0; j < n && ok; ++j, ++tiles) {
            // S loaded first: with an odd number of places this one's last phase was a V tile's, which only the
            // PV issuer waits for, and a wait for a phase is a wait for its parity. That S(j - 1) was loaded says
            // that P(j - 2) was stored, so PV(j - 3), which read that tile, is complete.
            ok = (tiles == 0 || wait_warp(bar(C::B_SFREE), (tiles - 1) & 1, true)) &&
                 wait_warp(bar(C::B_FULL + pos.s), pos.ph, true);
            if (!ok) break;
            ptx::tc_fence_after();
            const uint32_t k_tile = s_kv(pos.s);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t koff = (kk >> 2) * C::CHUNK_BYTES + (kk & 3) * 32;
              ptx::mma_ss_warp(t_mem, ptx::sdesc_sw128(q_tile + koff, 16, 1024), ptx::sdesc_sw128(k_tile + koff, 16, 1024),
                               C::IDESC_S, kk > 0 ? 1u : 0u, issue);
            }
            ptx::mma_commit_warp(bar(C::B_SFULL), issue);
            ptx::mma_commit_warp(bar(C::B_EMPTY + pos.s), issue);
            pos.step(2);
          }
          if (!ok) break;
        }
        // every MMA and every arrival of this warp's commits is done before the CTA's shared memory goes: the
        // last commits may come after those that the softmax has waited for
        ptx::mma_commit_warp(bar(C::B_DRAIN), issue);
        drain_wait(bar(C::B_DRAIN), 0);
      }
      __syncwarp();
    } else if (SINGLE && warp == C::WARP_PV) {
      // ================================================================ O += P V (one row tile)
      {
        const uint32_t t_mem = uniform(tmem);
        uint32_t tiles = 0, tails = 0;
        Pos pos;
        pos.step(1);
        for (uint32_t un = 0;; ++un) {
          if (!(ok = __all_sync(0xffffffffu, unit_wait(un)))) break;
          const plan::Entry& e = units[un % UNITS];
          const int n = (int)uniform(e.n), len = (int)uniform(e.str_len);
          if (n < 0) break;
          for (int j = 0; j < n && ok; ++j, ++tiles) {
            const bool tail = uniform((tile_of(e, j) + 1) * BN > len) != 0;
            ok = wait_warp(bar(C::B_FULL + pos.s), pos.ph, true);
            if (!ok) break;
            if (tail && issue) ptx::mbar_arrive(bar(C::B_TAILREQ));
            ok = wait_warp(bar(C::B_PFULL), tiles & 1, true) &&
                 (!tail || wait_warp(bar(C::B_TAIL), tails & 1, true));
            if (!ok) break;
            tails += tail;
            ptx::tc_fence_after();
            const uint32_t v_tile = s_kv(pos.s);
#pragma unroll
            for (int kk = 0; kk < BN / 16; ++kk)
              ptx::mma_ts_warp(t_mem + C::TMEM_O, t_mem + C::TMEM_P + kk * 8,
                          ptx::sdesc_sw128(v_tile + kk * 2048, C::CHUNK_BYTES, 1024), C::IDESC_PV,
                          (j > 0 || kk > 0) ? 1u : 0u, issue);
            ptx::mma_commit_warp(bar(C::B_ODONE), issue);
            ptx::mma_commit_warp(bar(C::B_EMPTY + pos.s), issue);
            pos.step(2);
          }
          if (!ok) break;
          __syncwarp();
          if (issue) unit_done(un);
        }
        ptx::mma_commit_warp(bar(C::B_DRAIN + 1), issue);
        drain_wait(bar(C::B_DRAIN + 1), 0);
      }
      __syncwarp();
    } else if (!SINGLE && (warp == C::WARP_MMA || (C::ISSUERS == 2 && warp == C::WARP_PV))) {
      // ================================================================ both products of one or two row tiles
      // P_t lies in S_t, so S_t(j) follows PV_t(j - 1), over all units as one stream: a unit's last PV waits for the
      // softmax while the next one's keys are on their way. Only where a unit starts does the PV come first, since S
      // needs the new Q. The issue of an MMA blocks while two or three wait to run, and a barrier or a commit takes
      // the issuer 80 to 150 cycles, so one warp cannot keep the tensor cores busy. An issuer per row tile waits for
      // its operands beforehand and the two take turns, in the order PV0 S0 PV1 S1 (8192 causal tokens, 32/8 heads
      // of 128: 838 us with one issuer, 738 with two; 925 without the turns, as then the two tiles' products
      // mix and both softmaxes wait at the same time).
      {
        constexpr int TILES = 2 / C::ISSUERS;  // row tiles of this warp, from t0 on
        const int t0 = TILES == 1 && warp == C::WARP_PV ? 1 : 0;
        const uint32_t t_mem = uniform(tmem);
        uint32_t n_q = 0, qb = 0, turns = 0, tails = 0;  // tails: a parity bit per place of values
        uint32_t cnt[TILES] = {};             // key tiles of the row tiles so far
        bool pend = false, pend_tail = false, pend_in[TILES] = {}, acc[TILES] = {};  // the PVs not yet issued
        Pos kpos, vpos;  // this tile's keys; the values of the PVs not yet issued
        vpos.step(1);
        // the values for the PVs still to come have landed
        auto values = [&]() -> bool {
          if (!wait_warp(bar(C::B_FULL + vpos.s), vpos.ph)) return false;
          if (KIND == PAGED) ptx::fence_proxy_async_smem();  // written by cp.async, read by the tensor cores
          if (!pend_tail) return true;
          if (issue && t0 == 0) ptx::mbar_arrive(bar(C::B_TAILREQ));
          const uint32_t place = vpos.s >> 1, parity = (tails >> place) & 1;
          tails ^= 1u << place;
          return wait_warp(bar(C::B_TAIL + (int)place), parity);
        };
        auto stored = [&](int x) -> bool { return !pend_in[x] || wait_warp(bar(C::B_PFULL + t0 + x), (cnt[x] - 1) & 1); };
        auto issue_pv = [&](int x) {
          const int t = t0 + x;
          const uint32_t v_tile = s_kv(vpos.s);
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk)
            ptx::mma_ts_warp(t_mem + C::TMEM_O + t * D, t_mem + t * BN + kk * 8,
                             ptx::sdesc_sw128(v_tile + kk * 2048, C::CHUNK_BYTES, 1024), C::IDESC_PV,
                             (acc[x] || kk > 0) ? 1u : 0u, issue);
        };
        auto values_done = [&]() {
          ptx::mma_commit_warp(bar(C::B_EMPTY + vpos.s), issue);
          vpos.step(2);
          pend = false;
        };
        for (uint32_t un = 0;; ++un) {
          if (pend) {
            ok = values();
#pragma unroll
            for (int x = 0; x < TILES; ++x) {
              ok = ok && stored(x);
              ptx::tc_fence_after();
              if (!ok) break;
              if (!pend_in[x]) continue;
              issue_pv(x);
              ptx::mma_commit_warp(bar(C::B_ODONE + t0 + x), issue);
            }
            if (!ok) break;
            values_done();
          }
          if (!(ok = __all_sync(0xffffffffu, unit_wait(un)))) break;
          const plan::Entry& e = units[un % UNITS];
          const int n = (int)uniform(e.n), len = (int)uniform(e.str_len);
          if (n < 0) break;
          int lo[TILES], hi[TILES];
#pragma unroll
          for (int x = 0; x < TILES; ++x) {
            lo[x] = (int)uniform(t0 + x ? e.lo1 : e.lo0);
            hi[x] = (int)uniform(t0 + x ? e.hi1 : e.hi0);
          }
          if (n > 0) {
            qb = n_q % C::Q_BUFS;
            ok = wait_warp(bar(RAW ? C::B_QREADY : C::B_QFULL + (int)qb), (n_q / C::Q_BUFS) & 1);
            ++n_q;
          }
          for (int j = 0; j < n && ok; ++j) {
            // also where no row of this warp's has a key in the tile: its arrivals below must not run ahead
            ok = !pend || values();
#pragma unroll
            for (int x = 0; x < TILES; ++x) {
              const int t = t0 + x;
              if (x == 0) {
                ok = ok && wait_warp(bar(C::B_FULL + kpos.s), kpos.ph);
                if (KIND == PAGED) ptx::fence_proxy_async_smem();
              }
              if (pend) ok = ok && stored(x);
              if (TILES == 1) ok = ok && (t0 == 0 ? turns == 0 || wait_warp(bar(C::B_TURN), (turns - 1) & 1)
                                                  : wait_warp(bar(C::B_TURN + 1), turns & 1));
              if (!ok) break;
              ptx::tc_fence_after();
              const bool before = pend && pend_in[x];
              if (before) issue_pv(x);
              pend_in[x] = j >= lo[x] && j < hi[x];
              acc[x] = j > lo[x];
              if (pend_in[x]) {
                const uint32_t q_tile = s_q(qb) + t * C::TILE_BYTES, k_tile = s_kv(kpos.s);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                  const uint32_t koff = (kk >> 2) * C::CHUNK_BYTES + (kk & 3) * 32;
                  ptx::mma_ss_warp(t_mem + t * BN, ptx::sdesc_sw128(q_tile + koff, 16, 1024),
                                   ptx::sdesc_sw128(k_tile + koff, 16, 1024), C::IDESC_S, kk > 0 ? 1u : 0u, issue);
                }
              }
              if (TILES == 1 && issue) ptx::mbar_arrive(bar(C::B_TURN + (t0 ^ 1)));
              if (pend_in[x]) {
                ptx::mma_commit_warp(bar(C::B_SFULL + t), issue);
                if (KIND != DENSE && issue) ptx::mbar_arrive(bar(C::B_SFULL + t));
                ++cnt[x];
              }
              if (before) ptx::mma_commit_warp(bar(C::B_ODONE + t), issue);
            }
            if (!ok) break;
            ++turns;
            ptx::mma_commit_warp(bar(C::B_EMPTY + kpos.s), issue);
            kpos.step(2);
            if (pend) values_done();
            pend = true;
            pend_tail = KIND == DENSE && uniform((tile_of(e, j) + 1) * BN > len) != 0;
          }
          if (!ok) break;
          if (n > 0) ptx::mma_commit_warp(bar(C::B_QEMPTY + qb), issue);
          __syncwarp();
          if (issue) unit_done(un);
        }
        // every MMA and every arrival of this warp's commits is done before the CTA's shared memory goes: the
        // last commits may come after those that the softmax has waited for
        ptx::mma_commit_warp(bar(C::B_DRAIN + t0), issue);
        drain_wait(bar(C::B_DRAIN + t0), 0);
      }
      __syncwarp();
    } else if (RAW && (warp == C::WARP_TAIL || warp == C::WARP_PV)) {
      // ================================================================ 8-bit pages: a warp for V, one for K
      ok = page_copies(warp == C::WARP_TAIL, 0, 1);
    } else if (KIND == DENSE && warp == C::WARP_TAIL) {
      // ================================================================ values behind the end: zero
      uint32_t tails = 0;
      Pos pos;
      pos.step(1);
      for (uint32_t un = 0;; ++un) {
        ok = __all_sync(0xffffffffu, unit_wait(un));
        if (!ok) break;
        const plan::Entry& e = units[un % UNITS];
        const int n = e.n, len = e.str_len;
        if (n < 0) break;
        for (int j = 0; j < n; ++j, pos.step(2)) {
          const int there = len - tile_of(e, j) * BN;
          if (there >= BN) continue;
          ok = __all_sync(0xffffffffu, wait_bar(bar(C::B_TAILREQ), tails++ & 1, abort_flag, true));
          if (!ok) break;
          for (int c = 0; c < C::CHUNKS; ++c)
            for (int x = there * 8 + lane; x < BN * 8; x += 32)
              ptx::st_shared_v4(s_kv(pos.s) + c * C::CHUNK_BYTES + x * 16, 0, 0, 0, 0);
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(bar(C::B_TAIL + (SINGLE ? 0 : (int)pos.s >> 1)));
          __syncwarp();
        }
        if (!ok) break;
        if (lane == 0) unit_done(un);
        __syncwarp();
      }
    }
  }

  // ---- teardown
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == C::WARP_MMA) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// Rows of the units that were cut: out = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i over the pieces, in
// their order. A block takes 32 rows of one unit, a warp four of them at once, D / 32 columns per
// lane: a row's loads do not wait for another's.
struct JoinParams {
  const plan::Header* head;
  const plan::Join* joins;
  const float* part;
  uint16_t* out;
  float* lse;
  long long out_ts, out_hs;
  int h_q, group, tok, rows;  // rows per slot
  const float* v_scale;
};

template <int D>
__global__ void __launch_bounds__(256) attn_join_kernel(const JoinParams p) {
  constexpr int W = D / 32, R = 4;
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  if ((int)blockIdx.x >= p.head->n_join) return;
  const plan::Join j = p.joins[blockIdx.x];
  const int lane = threadIdx.x & 31;
  const size_t slot_floats = (size_t)p.rows * (D + 2);
  int row[R], token[R];
  bool valid[R], some = false;
#pragma unroll
  for (int y = 0; y < R; ++y) {
    row[y] = (int)blockIdx.y * 32 + (threadIdx.x >> 5) * R + y;
    const int t = row[y] / BM, rt = row[y] % BM / p.group;
    token[y] = t * p.tok + rt;
    valid[y] = rt < p.tok && token[y] < j.own_n;
    some |= valid[y];
  }
  if (!some) return;
  auto slot = [&](int i) { return p.part + (size_t)(i == 0 ? j.slot : j.next + 2 * (i - 1)) * slot_floats; };
  float m[R], sum[R], o[R][W];
#pragma unroll
  for (int y = 0; y < R; ++y) {
    m[y] = -INFINITY;
    sum[y] = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) o[y][w] = 0.0f;
    if (!valid[y]) row[y] = row[0] - row[0] % R;  // a row whose statistics may be read; not used
  }
  for (int i = lane; i < j.pieces; i += 32) {
    const float* s = slot(i) + (size_t)p.rows * D;
#pragma unroll
    for (int y = 0; y < R; ++y)
      if (valid[y]) m[y] = fmaxf(m[y], s[row[y]]);
  }
#pragma unroll
  for (int y = 0; y < R; ++y)
#pragma unroll
    for (int off = 16; off; off >>= 1) m[y] = fmaxf(m[y], __shfl_xor_sync(0xffffffffu, m[y], off));
#pragma unroll 2
  for (int i = 0; i < j.pieces; ++i) {
    const float* s = slot(i);
#pragma unroll
    for (int y = 0; y < R; ++y) {
      if (!valid[y]) continue;
      const float mi = s[(size_t)p.rows * D + row[y]], li = s[(size_t)p.rows * (D + 1) + row[y]];
      float v[W];
      const float* at = s + (size_t)row[y] * D + lane * W;
      if constexpr (W == 4) {
        const float4 x = *reinterpret_cast<const float4*>(at);
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
      } else {
        const float2 x = *reinterpret_cast<const float2*>(at);
        v[0] = x.x, v[1] = x.y;
      }
      const float w = mi == -INFINITY ? 0.0f : exp2f(mi - m[y]);
      sum[y] += w * li;
#pragma unroll
      for (int z = 0; z < W; ++z) o[y][z] = w == 0.0f ? o[y][z] : o[y][z] + w * v[z];
    }
  }
#pragma unroll
  for (int y = 0; y < R; ++y) {
    if (!valid[y]) continue;
    const int head_q = j.hk * p.group + row[y] % BM % p.group;
    const long long at = (long long)j.own_row + token[y];
    const float inv = sum[y] == 0.0f ? 0.0f : (p.v_scale ? p.v_scale[j.hk] : 1.0f) / sum[y];
    uint32_t* to = reinterpret_cast<uint32_t*>(p.out + at * p.out_ts + head_q * p.out_hs) + lane * (W / 2);
#pragma unroll
    for (int z = 0; z < W; z += 2) to[z / 2] = ptx::pack_bf16x2(o[y][z] * inv, o[y][z + 1] * inv);
    if (lane == 0 && p.lse)
      p.lse[at * p.h_q + head_q] = sum[y] == 0.0f ? -INFINITY : (m[y] + log2f(sum[y])) * 0.69314718055994530942f;
  }
}

// q [T, heads, d] as (d, head of the group, token, key/value head): a row tile is one box.
CUresult encode_q(PFN_encodeTiled enc, CUtensorMap* map, const PackedArgs& a, int d, int group, int tok) {
  cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)group, (cuuint64_t)a.T_q, (cuuint64_t)a.h_kv};
  cuuint64_t strides[3] = {(cuuint64_t)a.q_hs * 2, (cuuint64_t)a.q_ts * 2, (cuuint64_t)a.q_hs * 2 * group};
  cuuint32_t box[4] = {64, (cuuint32_t)group, (cuuint32_t)tok, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(a.q), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

// k or v [T, heads, d] as (d, token, head): a key tile is one box per 64 columns.
CUresult encode_rows(PFN_encodeTiled enc, CUtensorMap* map, const void* base, int d, long long rows, int heads,
                     long long ts, long long hs) {
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)rows, (cuuint64_t)heads};
  cuuint64_t strides[2] = {(cuuint64_t)ts * 2, (cuuint64_t)hs * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)BN, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

// All pages' rows as (d, row): boxes of `rows` rows that no page border cuts.
CUresult encode_pages(PFN_encodeTiled enc, CUtensorMap* map, const void* base, int d, long long all, int rows, bool bytes) {
  cuuint64_t dims[2] = {(cuuint64_t)d, (cuuint64_t)all};
  cuuint64_t strides[1] = {(cuuint64_t)d * (bytes ? 1 : 2)};
  cuuint32_t box[2] = {(cuuint32_t)(bytes ? d : 64), (cuuint32_t)rows};
  cuuint32_t estr[2] = {1, 1};
  return enc(map, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base),
             dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             bytes ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

struct Geometry {
  int group, tok, own_tiles, ctas;
  long long items;
  size_t plan_bytes, part_bytes;
};

// Streaming multiprocessors of the GB300; a workspace's size may not depend on the current device.
constexpr int kSms = 152;

template <int D, int KIND>
Geometry geometry_of(int T_q, int B, int h_q, int h_kv) {
  using C = Cfg<D, KIND>;
  Geometry g;
  g.group = h_q / h_kv;
  g.tok = BM / g.group;
  g.own_tiles = C::Q_TILES;
  g.ctas = kSms * C::CTAS_PER_SM;
  g.items = T_q / (g.tok * g.own_tiles) + B;
  g.plan_bytes = plan::bytes(g.items, h_kv, B, g.ctas);
  g.part_bytes = (size_t)2 * g.ctas * C::ROWS * (D + 2) * sizeof(float);
  return g;
}

template <typename Kernel, typename... A>
bool launch(Kernel* kernel, dim3 grid, unsigned threads, size_t smem, cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess;
}

// The tile of the INJECT instantiation, for the next call over pages on the arming host thread; -1: not armed.
thread_local int t_inject_v_tile = -1;

template <int D, int KIND, bool INJECT = false>
int run(const PackedArgs& a, PFN_encodeTiled enc, void* workspace) {
  using C = Cfg<D, KIND>;
  const Geometry g = geometry_of<D, KIND>(a.T_q, a.B, a.h_q, a.h_kv);
  static std::atomic<bool> attr_done[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return ATTN_ERR_CUDA;
  if (!attr_done[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(attn_packed_kernel<D, KIND, INJECT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             C::SMEM_BYTES) != cudaSuccess)
      return ATTN_ERR_CUDA;
    attr_done[dev].store(true, std::memory_order_release);
  }
  CUtensorMap mq, mk, mv;
  int box_shift = 0;
  while (box_shift < 7 && a.page_size % (2 << box_shift) == 0) ++box_shift;
  if (encode_q(enc, &mq, a, D, g.group, g.tok) != CUDA_SUCCESS) return ATTN_ERR_UNSUPPORTED;
  if (KIND == DENSE) {
    if (encode_rows(enc, &mk, a.k, D, a.T_k, a.h_kv, a.k_ts, a.k_hs) != CUDA_SUCCESS ||
        encode_rows(enc, &mv, a.v, D, a.T_k, a.h_kv, a.v_ts, a.v_hs) != CUDA_SUCCESS)
      return ATTN_ERR_UNSUPPORTED;
  } else if (box_shift >= kTmaShift) {
    const int rows = std::min(1 << box_shift, KIND == PAGED ? BN / 2 : BN);  // at most a copy warp's part of a tile
    if (encode_pages(enc, &mk, a.k, D, (long long)a.n_pages * a.h_kv * a.page_size, rows, KIND == PAGED8) != CUDA_SUCCESS ||
        encode_pages(enc, &mv, a.v, D, (long long)a.n_pages * a.h_kv * a.page_size, rows, KIND == PAGED8) != CUDA_SUCCESS)
      return ATTN_ERR_UNSUPPORTED;
  } else {
    mk = mv = mq;  // not read
  }
  const long long reach = KIND == DENSE ? a.T_k : (long long)a.max_pages * a.page_size;
  // no sequence has more tiles than a CTA's least share, so none is longer than one: nothing to cut
  const bool may_cut = (reach + BN - 1) / BN > kMinShare;
  // and with a CTA for every unit there can be, each finds its own, without a list
  const bool no_list = C::LISTLESS && !may_cut && g.items * a.h_kv <= g.ctas;
  plan::Args pa = {};
  pa.q_starts = a.q_starts;
  pa.k_starts = a.k_starts;
  pa.cache_lens = a.cache_lens;
  pa.B = a.B;
  pa.T_q = a.T_q;
  pa.T_k = a.T_k;
  pa.max_keys = (int)reach;
  pa.own_keys = 0;
  pa.own_tiles = g.own_tiles;
  pa.tok = g.tok;
  pa.h_kv = a.h_kv;
  pa.causal = a.causal;
  pa.window = a.window;
  pa.sinks = a.sinks;
  pa.ctas = g.ctas;
  pa.min_share = kMinShare;
  pa.may_cut = may_cut;
  plan::place(pa, workspace, g.items);
  Params p = {};
  p.plan = pa;
  p.no_list = no_list;
  p.head = pa.head;
  p.range = pa.range;
  p.list = pa.list;
  p.out = static_cast<uint16_t*>(a.out);
  p.lse = a.lse;
  p.out_ts = a.out_ts;
  p.out_hs = a.out_hs;
  p.h_q = a.h_q;
  p.group = g.group;
  p.tok = g.tok;
  p.causal = a.causal;
  p.window = a.window;
  p.sinks = a.sinks;
  p.scale_log2 = (float)((double)a.scale * 1.4426950408889634074);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + g.plan_bytes);
  p.k_pages = static_cast<const uint8_t*>(a.k);
  p.v_pages = static_cast<const uint8_t*>(a.v);
  p.page_table = a.page_table;
  p.max_pages = a.max_pages;
  p.n_pages = a.n_pages;
  p.page_size = a.page_size;
  p.box_shift = box_shift;
  p.h_kv = a.h_kv;
  p.k_scale = a.k_scale;
  p.v_scale = a.v_scale;
  p.back = a.window >= 0 ? a.window : 1 << 30;  // no sequence is longer
  p.inject_v_tile = -1;
  if (INJECT) std::swap(p.inject_v_tile, t_inject_v_tile);
  const unsigned grid = no_list ? (unsigned)(g.items * a.h_kv) : (unsigned)g.ctas;
  if (!no_list && !launch(plan::attn_plan_kernel, 1, plan::THREADS, 0, a.stream, pa)) return ATTN_ERR_CUDA;
  if (!launch(attn_packed_kernel<D, KIND, INJECT>, grid, C::THREADS, C::SMEM_BYTES, a.stream, mq, mk, mv, p))
    return ATTN_ERR_CUDA;
  if (may_cut) {
    const JoinParams j = {pa.head, pa.joins, p.part, p.out,  p.lse,  p.out_ts,
                          p.out_hs, p.h_q,    p.group, p.tok, C::ROWS, KIND == PAGED8 ? p.v_scale : nullptr};
    if (!launch(attn_join_kernel<D>, dim3((unsigned)g.ctas, C::ROWS / 32), 256, 0, a.stream, j)) return ATTN_ERR_CUDA;
  }
  return cudaPeekAtLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

template <int KIND>
size_t workspace_of(int T_q, int B, int h_q, int h_kv, int d) {
  const Geometry g = d == 64 ? geometry_of<64, KIND>(T_q, B, h_q, h_kv) : geometry_of<128, KIND>(T_q, B, h_q, h_kv);
  return g.plan_bytes + g.part_bytes;
}

}  // namespace

size_t packed_fwd_workspace_bytes(int T_q, int B, int h_q, int h_kv, int d) {
  return workspace_of<DENSE>(T_q, B, h_q, h_kv, d);
}

size_t paged_chunk_workspace_bytes(int T_q, int B, int h_q, int h_kv, int d) {
  // either cache type
  return std::max(workspace_of<PAGED>(T_q, B, h_q, h_kv, d), workspace_of<PAGED8>(T_q, B, h_q, h_kv, d));
}

int launch_attn_packed(const PackedArgs& a, PFN_encodeTiled enc, void* workspace) {
  if (!a.page_table) return a.d == 64 ? run<64, DENSE>(a, enc, workspace) : run<128, DENSE>(a, enc, workspace);
  if (t_inject_v_tile >= 0) {
    if (!a.k_scale) return a.d == 64 ? run<64, PAGED, true>(a, enc, workspace) : run<128, PAGED, true>(a, enc, workspace);
    return a.d == 64 ? run<64, PAGED8, true>(a, enc, workspace) : run<128, PAGED8, true>(a, enc, workspace);
  }
  if (!a.k_scale) return a.d == 64 ? run<64, PAGED>(a, enc, workspace) : run<128, PAGED>(a, enc, workspace);
  return a.d == 64 ? run<64, PAGED8>(a, enc, workspace) : run<128, PAGED8>(a, enc, workspace);
}

void arm_chunk_give_up(int v_tile) { t_inject_v_tile = v_tile; }

int read_packed_fault_word(int clear, uint32_t* out) {
  uint32_t w = 0;
  if (cudaMemcpyFromSymbol(&w, g_packed_fault_word, sizeof w) != cudaSuccess) return ATTN_ERR_CUDA;
  if (clear) {
    const uint32_t zero = 0;
    if (cudaMemcpyToSymbol(g_packed_fault_word, &zero, sizeof zero) != cudaSuccess) return ATTN_ERR_CUDA;
  }
  *out = w;
  return ATTN_OK;
}

}  // namespace attn
