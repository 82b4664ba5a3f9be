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
// still write the last one's rows. When the units are few the plan cuts them: a piece leaves its
// rows' unnormalised sums, reference maxima and row sums in the workspace, and attn_join_kernel
// adds the pieces up.
//
// Tiles. As in attn_fwd_tc.cu: at d = 64 a CTA has one row tile, two CTAs share an SM, and P has
// TMEM columns of its own; at d = 128 a CTA has two row tiles, P written over S. Keys come as
// 128-row tiles through a shared-memory ring:
//   dense   one TMA box per 64 columns;
//   pages   a tile is 128 / r boxes of r rows, r = gcd(page size, 128), so that no box crosses a
//           page or a tile; a lane of the copy warp looks up the page of its boxes and issues
//           them. Rows of no page (a bad entry, or behind the length) are boxes outside the
//           tensor: zeros. Bad entries' keys are masked by bits that go with the tile.
//   8 bits  the boxes land in a raw tile, and four more warps turn it into the bf16 tile that the
//           products read: exact, as bf16 holds every e4m3 number (the scales are folded
//           into the exponent's factor and the last division). Two row tiles at either d, so that
//           a tile is converted once for 256 rows.
// Values behind the sequence's end (the next sequence's rows, a page's stale rows) would meet
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

#include "attn_internal.h"
#include "attn_plan.cuh"
#include "ptx_sm103.cuh"

namespace attn {

__device__ unsigned int g_packed_fault_word;  // fault record, read by attn_fault_status

namespace {

constexpr int BM = 128, BN = 128;  // rows and keys per tile
constexpr int kMaxDevices = 64;
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr uint64_t kDrainLimitNs = 200000000ull;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr uint32_t FAULT_PACKED = 512;
constexpr int FLAGS = 8;    // tiles whose page bits are held: more than the roles are apart
constexpr int kMinShare = 2;   // tiles
constexpr int kMaxDeal = 4;    // units per CTA from which on they are not cut

enum { DENSE = 0, PAGED = 1, PAGED8 = 2 };

template <int D, int KIND>
struct Cfg {
  static constexpr bool SINGLE = D == 64 && KIND != PAGED8;
  static constexpr int Q_TILES = SINGLE ? 1 : 2;
  static constexpr int ROWS = Q_TILES * BM;
  static constexpr int CTAS_PER_SM = SINGLE ? 2 : 1;
  static constexpr int CHUNKS = D / 64;
  static constexpr int CHUNK_BYTES = BM * 128;
  static constexpr int TILE_BYTES = BM * D * 2;
  static constexpr int STAGES = SINGLE ? 3 : 2;
  static constexpr int RAW_BYTES = KIND == PAGED8 ? BN * 128 : 0;  // 128-byte row pitch for single rows at d = 64
  static constexpr int BATCH = SINGLE ? 8 : 16;  // units whose entries a CTA holds at a time
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + Q_TILES * TILE_BYTES;
  static constexpr int OFF_V = OFF_K + STAGES * TILE_BYTES;
  static constexpr int OFF_RAW = OFF_V + STAGES * TILE_BYTES;  // [K, V]
  static constexpr int OFF_UNITS = OFF_RAW + 2 * RAW_BYTES;    // Entry [BATCH]
  static constexpr int OFF_FLAGS = OFF_UNITS + BATCH * 64;     // uint32 [FLAGS][8]: any, four words of key bits
  static constexpr int OFF_BAR = OFF_FLAGS + (KIND == DENSE ? 0 : FLAGS * 32);
  static constexpr int B_QFULL = 0;
  static constexpr int B_QEMPTY = 1;
  static constexpr int B_KFULL = 2;
  static constexpr int B_KEMPTY = B_KFULL + STAGES;
  static constexpr int B_VFULL = B_KEMPTY + STAGES;
  static constexpr int B_VEMPTY = B_VFULL + STAGES;
  static constexpr int B_SFULL = B_VEMPTY + STAGES;  // [2] S_t computed
  static constexpr int B_SFREE = B_SFULL + 2;        // S loaded by the softmax (SINGLE)
  static constexpr int B_PFULL = B_SFREE + 1;        // [2] P_t stored
  static constexpr int B_ODONE = B_PFULL + 2;        // [2] PV_t completed
  static constexpr int B_TAILREQ = B_ODONE + 2;      // a tile with values behind the end has landed
  static constexpr int B_TAIL = B_TAILREQ + 1;       // they are zeroed
  static constexpr int B_RAWFULL = B_TAIL + 1;       // [K, V]
  static constexpr int B_RAWEMPTY = B_RAWFULL + 2;
  static constexpr int B_DRAIN = B_RAWEMPTY + 2;     // [2] MMAs after an abort, one per issuer
  static constexpr int NUM_BARS = B_DRAIN + 2;
  static constexpr int OFF_SLOT = OFF_BAR + NUM_BARS * 8;
  static constexpr int OFF_ABORT = OFF_SLOT + 4;
  static constexpr int SMEM_BYTES = OFF_ABORT + 4;
  static constexpr uint32_t TMEM_COLS = SINGLE ? 256 : 512;
  // warps: softmax (4 per row tile); copies; MMA issuer (SINGLE: of S); tail; SINGLE: PV issuer;
  // PAGED8: four converting warps
  static constexpr int SOFTMAX_WARPS = 4 * Q_TILES;
  static constexpr int WARP_LOAD = SOFTMAX_WARPS, WARP_MMA = SOFTMAX_WARPS + 1, WARP_TAIL = SOFTMAX_WARPS + 2,
                       WARP_PV = SOFTMAX_WARPS + 3, WARP_CVT = SOFTMAX_WARPS + 4;
  static constexpr int THREADS = 32 * (SOFTMAX_WARPS + 4 + (KIND == PAGED8 ? 4 : 0));
  static constexpr int REGS_CONTROL = SINGLE || KIND == PAGED8 ? 40 : 72;
  static constexpr int REGS_CVT = 40;
  static constexpr int REGS_SOFTMAX = 216;
  static constexpr int LAUNCH_REGS = (65536 / (THREADS * CTAS_PER_SM)) & ~7;
  static_assert(128 * REGS_CONTROL + (KIND == PAGED8 ? 128 * REGS_CVT : 0) + 32 * SOFTMAX_WARPS * REGS_SOFTMAX <=
                    THREADS * LAUNCH_REGS,
                "register split");
  static constexpr uint32_t TMEM_P = SINGLE ? BN : 0;  // else P_t over S_t
  static constexpr uint32_t TMEM_O = SINGLE ? BN + BN / 2 : 2 * BN;
  static constexpr uint32_t IDESC_S = ptx::idesc_bf16_f32(BM, BN, false);
  static constexpr uint32_t IDESC_PV = ptx::idesc_bf16_f32(BM, D, true);
  static_assert(TMEM_O + Q_TILES * D <= TMEM_COLS, "TMEM budget");
  static_assert(OFF_UNITS % 16 == 0 && OFF_BAR % 8 == 0, "alignment");
  static_assert(CTAS_PER_SM * (SMEM_BYTES + 1024) <= 228 * 1024, "shared memory budget");
};

struct Params {
  const plan::Header* head;
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
  const int32_t* page_table;
  int max_pages, n_pages, page_size, box;  // box: rows per copy
  int h_kv;
  const float* k_scale;
  const float* v_scale;
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

// Two e4m3 numbers, in bits 15:8 and 31:24 of x (the other bits zero), as two bf16: the exponent and
// mantissa fields moved to their places read 2^-120 times the value, subnormal ones included, and
// the product with 2^120 is exact. 0x7f, NaN, would read 480: the caller looks for it.
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t x) {
  const uint32_t y = ((x >> 4) & 0x07f007f0u) | (x & 0x80008000u);
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(y), "r"(0x7b807b80u));  // 2^120
  return r;
}

// The key tile of list entry j.
__device__ __forceinline__ int tile_of(const plan::Entry& e, int j) {
  const int l = e.j0 + j;
  return l + (l >= e.n_first ? e.skip : 0);
}

template <int D, int KIND>
__global__ void __launch_bounds__(Cfg<D, KIND>::THREADS, Cfg<D, KIND>::CTAS_PER_SM)
    attn_packed_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const Params p) {
  using C = Cfg<D, KIND>;
  constexpr bool SINGLE = C::SINGLE;
  constexpr int STAGES = C::STAGES;
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((ptx::smem_u32(smem) & 1023u) != 0) {
    if (threadIdx.x == 0) atomicOr(&g_packed_fault_word, FAULT_PACKED);
    return;
  }
  const uint32_t s_base = ptx::smem_u32(smem);
  const uint32_t s_q = s_base + C::OFF_Q, s_k = s_base + C::OFF_K, s_v = s_base + C::OFF_V;
  auto bar = [&](int i) -> uint32_t { return s_base + C::OFF_BAR + 8u * i; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_ABORT);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_SLOT);
  const plan::Entry* units = reinterpret_cast<const plan::Entry*>(smem + C::OFF_UNITS);
  volatile uint32_t* flags = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_FLAGS);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    ptx::mbar_init(bar(C::B_QFULL), 1);
    ptx::mbar_init(bar(C::B_QEMPTY), 1);
    for (int s = 0; s < STAGES; ++s) {
      ptx::mbar_init(bar(C::B_KFULL + s), KIND == PAGED8 ? 4 : 1);  // converting warps, or the copies' bytes
      ptx::mbar_init(bar(C::B_KEMPTY + s), 1);
      ptx::mbar_init(bar(C::B_VFULL + s), KIND == PAGED8 ? 4 : 1);
      ptx::mbar_init(bar(C::B_VEMPTY + s), 1);
    }
    for (int t = 0; t < 2; ++t) {
      // pages: the issuer arrives besides its commit, so that the page bits, written before the
      // copies, are ordered before the softmax reads them
      ptx::mbar_init(bar(C::B_SFULL + t), KIND == DENSE ? 1 : 2);
      ptx::mbar_init(bar(C::B_PFULL + t), BM);
      ptx::mbar_init(bar(C::B_ODONE + t), 1);
      ptx::mbar_init(bar(C::B_RAWFULL + t), 1);
      ptx::mbar_init(bar(C::B_RAWEMPTY + t), 4);
      ptx::mbar_init(bar(C::B_DRAIN + t), 1);
    }
    ptx::mbar_init(bar(C::B_SFREE), BM);
    ptx::mbar_init(bar(C::B_TAILREQ), 1);
    ptx::mbar_init(bar(C::B_TAIL), 1);
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

  const plan::Header head = *p.head;
  const int2 range = p.range[blockIdx.x];

  // The entries of this CTA's next units, up to BATCH, into shared memory; their number. Every warp
  // calls it, from its role's own loop (the register split forbids one loop around the roles).
  auto next_batch = [&](int batch) -> int {
    __syncwarp();  // the barrier counts whole warps
    ptx::named_bar_sync(1, C::THREADS);  // every role is through with the batch before
    if (*abort_flag) return 0;
    int n_b = 0;
    while (n_b < C::BATCH && plan::unit_of(head, range, blockIdx.x, gridDim.x, batch * C::BATCH + n_b) >= 0) ++n_b;
    for (int x = threadIdx.x; x < n_b * 4; x += C::THREADS) {
      const int u = plan::unit_of(head, range, blockIdx.x, gridDim.x, batch * C::BATCH + (x >> 2));
      reinterpret_cast<int4*>(smem + C::OFF_UNITS)[x] = reinterpret_cast<const int4*>(p.list + u)[x & 3];
    }
    __syncwarp();
    ptx::named_bar_sync(1, C::THREADS);
    return n_b;
  };

  // Counters that run through all units, each kept by the roles that need it.
  uint32_t ring = 0;   // key tiles so far
  uint32_t tails = 0;  // tails zeroed so far: asked for and answered one at a time
  bool ok = true;

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
      uint32_t cnt0 = 0;  // key tiles of this row tile so far
      for (int batch = 0, n_b; (n_b = next_batch(batch)) > 0; ++batch) {
      for (int b = 0; b < n_b && ok; ++b) {
        // the entry is read from shared memory where it is used: the score tile and P leave no
        // registers to hold it
        const plan::Entry& e = units[b];
        const int lo = t ? e.lo1 : e.lo0, n_tiles = (t ? e.hi1 : e.hi0) - lo;
        const float c = KIND == PAGED8 ? p.scale_log2 * p.k_scale[e.hk] : p.scale_log2;
        float m_ref = -INFINITY;  // reference maximum, log2 units
        float l = 0.0f;           // sum of 2^(c s - m_ref)
        for (int j = 0; j < n_tiles; ++j) {
          const uint32_t cnt = cnt0 + j;
          ok = __all_sync(0xffffffffu, wait_bar(bar(C::B_SFULL + t), cnt & 1, abort_flag));
          if (!ok) break;
          ptx::tc_fence_after();
          uint32_t sr[4][32];
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) ptx::tmem_ld32(t_s + q4 * 32, sr[q4]);
          ptx::tmem_wait_ld();
          if constexpr (KIND != DENSE) {
            volatile const uint32_t* fl = flags + ((ring + lo + j) % FLAGS) * 8;
            if (fl[0]) {  // keys of pages that are not there
#pragma unroll
              for (int q4 = 0; q4 < 4; ++q4) {
                const uint32_t bad = fl[1 + q4];
#pragma unroll
                for (int x = 0; x < 32; ++x)
                  if ((bad >> x) & 1u) sr[q4][x] = __float_as_uint(-INFINITY);
              }
            }
          }
          if constexpr (SINGLE) {  // S is in registers, the page bits are read
            ptx::tc_fence_before();
            ptx::mbar_arrive_after(bar(C::B_SFREE), __uint_as_float(sr[3][31]));
          }
          const int key0 = tile_of(e, lo + j) * BN;
          const int pos_lo = e.pos + t * p.tok;
          const bool edge =
              key0 + BN > e.str_len || (p.causal && key0 + BN - 1 > pos_lo) ||
              (p.window >= 0 && (key0 < pos_lo + min(e.own_n - t * p.tok, p.tok) - 1 - p.window ||
                                 (!p.causal && key0 + BN - 1 > pos_lo + p.window)));
          if (edge) {
            const int pos = pos_lo + rt;
            int lim = e.str_len - key0;  // columns [first, lim) are legal, and those below `sink`
            if (p.causal) lim = min(lim, pos + 1 - key0);
            int first = 0, sink = 0;
            if (p.window >= 0) {
              if (!p.causal) lim = min(lim, pos + p.window + 1 - key0);
              first = pos - p.window - key0;
              sink = p.sinks - key0;
            }
            if (first <= 0) sink = BN;
#pragma unroll
            for (int q4 = 0; q4 < 4; ++q4)
#pragma unroll
              for (int x = 0; x < 32; ++x)
                if (q4 * 32 + x >= lim || (q4 * 32 + x < first && q4 * 32 + x >= sink))
                  sr[q4][x] = __float_as_uint(-INFINITY);
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
          // P, rounded to bf16 for the tensor cores (the row sum takes it unrounded): each weight moves
          // by at most 2^-9 of itself, independently, less than the output's own rounding in the mean
          auto exps = [&](float m_now) -> float {
            const float m_use = (m_now == -INFINITY) ? 0.0f : m_now;
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
                pk[q4 >> 1][(q4 & 1) * 16 + (x >> 1)] = ptx::pack_bf16x2(p0, p1);
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
        ring += e.n;
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
            stat[0] = m_ref;
            stat[C::ROWS] = l;
          }
          continue;
        }
        const float v_mul = KIND == PAGED8 ? p.v_scale[e.hk] : 1.0f;
        const float inv = l == 0.0f ? 0.0f : v_mul / l;  // no legal key: zeros
        const long long row = (long long)e.own_row + t * p.tok + rt;
        const int head_q = e.hk * p.group + r - rt * p.group;
        uint16_t* orow = p.out + (row_valid ? row * p.out_ts + head_q * p.out_hs : 0);
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
          uint32_t w[16];
#pragma unroll
          for (int x = 0; x < 16; ++x)
            w[x] = ptx::pack_bf16x2(__uint_as_float(o[2 * x]) * inv, __uint_as_float(o[2 * x + 1]) * inv);
          if (row_valid) {
            uint4* dst = reinterpret_cast<uint4*>(orow + q4 * 32);
#pragma unroll
            for (int x = 0; x < 4; ++x) dst[x] = make_uint4(w[4 * x], w[4 * x + 1], w[4 * x + 2], w[4 * x + 3]);
          }
          __syncwarp();
        }
        if (row_valid && p.lse)
          p.lse[row * p.h_q + head_q] =
              l == 0.0f ? -INFINITY : (m_ref + __log2f(l)) * 0.69314718055994530942f;
      }
      }
  } else if (KIND == PAGED8 && warp >= C::WARP_CVT) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_CVT));
      // ================================================================ 8 bits to bf16
      // Sixteen numbers per thread and step: D / 16 lanes a row. Rows behind the end become zero.
      const int id = threadIdx.x - 32 * C::WARP_CVT;
      constexpr int LPR = D / 16, STEP = 128 / LPR;  // lanes per row, rows per step
      const uint32_t raw_pitch = p.box == 1 ? 128u : (uint32_t)D;
      for (int batch = 0, n_b; (n_b = next_batch(batch)) > 0; ++batch) {
      for (int b = 0; b < n_b && ok; ++b) {
        const plan::Entry& e = units[b];
        const int n = e.n, len = e.str_len;
        for (int j = 0; j < n && ok; ++j, ++ring) {
          const int s = ring % STAGES;
          const int there = len - tile_of(e, j) * BN;
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            ok = __all_sync(0xffffffffu, wait_bar(bar(C::B_RAWFULL + kv), ring & 1, abort_flag, true) &&
                                             wait_bar(bar((kv ? C::B_VEMPTY : C::B_KEMPTY) + s), ((ring / STAGES) & 1) ^ 1,
                                                      abort_flag, true));
            if (!ok) break;
            const uint32_t src = s_base + C::OFF_RAW + kv * C::RAW_BYTES + (id / LPR) * raw_pitch + (id % LPR) * 16;
            const uint32_t tile = (kv ? s_v : s_k) + s * C::TILE_BYTES;
            const uint32_t slab = tile + ((id % LPR) >> 2) * C::CHUNK_BYTES;
            const int unit = ((id % LPR) & 3) * 2;
#pragma unroll 4
            for (int r0 = 0; r0 < BN; r0 += STEP) {
              const int r = r0 + id / LPR;
              const uint4 w = ld_shared_v4(src + r0 * raw_pitch);
              const uint32_t in[4] = {w.x, w.y, w.z, w.w};
              uint32_t o[8];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                o[2 * i] = e4m3_pair(__byte_perm(in[i], 0, 0x1404));
                o[2 * i + 1] = e4m3_pair(__byte_perm(in[i], 0, 0x3424));
                if ((((in[i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0) {  // a NaN among the four
#pragma unroll
                  for (int y = 0; y < 4; ++y)
                    if (((in[i] >> (8 * y)) & 0x7f) == 0x7f) o[2 * i + (y >> 1)] |= 0x7fffu << (16 * (y & 1));
                }
              }
              if (r >= there) {
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = 0;
              }
              const uint32_t row = slab + r * 128;
              ptx::st_shared_v4(row + ((unit ^ (r & 7)) << 4), o[0], o[1], o[2], o[3]);
              ptx::st_shared_v4(row + (((unit + 1) ^ (r & 7)) << 4), o[4], o[5], o[6], o[7]);
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              ptx::mbar_arrive(bar(C::B_RAWEMPTY + kv));
              ptx::mbar_arrive(bar((kv ? C::B_VFULL : C::B_KFULL) + s));
            }
          }
          if (!ok) break;
        }
      }
      }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_CONTROL));
    if (warp == C::WARP_LOAD) {
      // ================================================================ copies
      const uint64_t pol_q = ptx::policy_evict_first();
      const uint64_t pol_kv = ptx::policy_evict_last();
      uint32_t n_q = 0;  // units with keys so far
      for (int batch = 0, n_b; (n_b = next_batch(batch)) > 0; ++batch) {
      for (int b = 0; b < n_b && ok; ++b) {
        const plan::Entry& e = units[b];
        const int n = e.n;
        if (n == 0) continue;
        ok = __all_sync(0xffffffffu,
                        n_q == 0 || wait_bar(bar(C::B_QEMPTY), (n_q - 1) & 1, abort_flag, SINGLE));
        if (!ok) break;
        if (lane == 0) {
          const int n_qt = e.own_n > p.tok ? 2 : 1;
          const int bytes = p.tok * p.group * 128 * C::CHUNKS;
          ptx::mbar_arrive_expect_tx(bar(C::B_QFULL), n_qt * bytes);
          for (int t = 0; t < n_qt; ++t)
            for (int c = 0; c < C::CHUNKS; ++c)
              tma_load_4d(s_q + t * C::TILE_BYTES + c * C::CHUNK_BYTES, &tm_q, bar(C::B_QFULL), c * 64, 0,
                          e.own_row + t * p.tok, e.hk, pol_q);
        }
        ++n_q;
        for (int j = 0; j < n && ok; ++j) {
          const uint32_t x = ring;
          const int s = x % STAGES;
          const uint32_t ph = (x / STAGES) & 1;
          const int key0 = tile_of(e, j) * BN;
          if constexpr (KIND == DENSE) {
            ok = __all_sync(0xffffffffu, wait_bar(bar(C::B_KEMPTY + s), ph ^ 1, abort_flag, SINGLE));
            if (!ok) break;
            if (lane == 0) {
              ptx::mbar_arrive_expect_tx(bar(C::B_KFULL + s), C::TILE_BYTES);
              for (int c = 0; c < C::CHUNKS; ++c)
                ptx::tma_load_3d(s_k + s * C::TILE_BYTES + c * C::CHUNK_BYTES, &tm_k, bar(C::B_KFULL + s), c * 64,
                                 e.str_row + key0, e.hk, pol_kv);
            }
            ok = __all_sync(0xffffffffu, wait_bar(bar(C::B_VEMPTY + s), ph ^ 1, abort_flag, SINGLE));
            if (!ok) {
              // K of this tile is in flight, V is not
              if (lane == 0) drain_wait(bar(C::B_KFULL + s), ph);
              break;
            }
            if (lane == 0) {
              ptx::mbar_arrive_expect_tx(bar(C::B_VFULL + s), C::TILE_BYTES);
              for (int c = 0; c < C::CHUNKS; ++c)
                ptx::tma_load_3d(s_v + s * C::TILE_BYTES + c * C::CHUNK_BYTES, &tm_v, bar(C::B_VFULL + s), c * 64,
                                 e.str_row + key0, e.hk, pol_kv);
            }
          } else {
            // boxes of p.box rows, lane by lane; a row behind the length or of a page that is
            // not there comes from outside the tensor
            constexpr bool RAW = KIND == PAGED8;
            const int boxes = BN / p.box;
            const int32_t* pages = p.page_table + (size_t)e.str_row * p.max_pages;
            const uint32_t full_k = bar(RAW ? C::B_RAWFULL : C::B_KFULL + s), full_v = bar(RAW ? C::B_RAWFULL + 1 : C::B_VFULL + s);
            const uint32_t empty_k = bar(RAW ? C::B_RAWEMPTY : C::B_KEMPTY + s),
                           empty_v = bar(RAW ? C::B_RAWEMPTY + 1 : C::B_VEMPTY + s);
            const uint32_t eph = RAW ? (x & 1) ^ 1 : ph ^ 1, fph = RAW ? x & 1 : ph;
            const uint32_t bytes = RAW ? BN * D : C::TILE_BYTES;
            const uint32_t pitch = RAW ? max(p.box * D, 128) : p.box * 128;
            volatile uint32_t* fl = flags + (x % FLAGS) * 8;
            auto lookup = [&](int i, int& row, int& z) -> bool {  // false: a key there whose page is bad
              const int key = key0 + i * p.box;
              z = p.n_pages * p.h_kv;
              row = 0;
              if (key >= e.str_len) return true;
              const int page = key / p.page_size;
              const int id = pages[page];
              if (id < 0 || id >= p.n_pages) return false;
              row = key - page * p.page_size;
              z = id * p.h_kv + e.hk;
              return true;
            };
            int row0, z0;  // this lane's first box, the only one unless pages are cut finer than 4 rows
            const bool good = lane >= boxes || lookup(lane, row0, z0);
            ok = __all_sync(0xffffffffu, wait_bar(empty_k, eph, abort_flag, SINGLE));
            if (!ok) break;
            bool bad = !good;
            for (int i = lane + 32; i < boxes; i += 32) {
              int row, z;
              bad |= !lookup(i, row, z);
            }
            const bool any = __any_sync(0xffffffffu, bad);
            if (lane < 5) fl[lane] = lane == 0 ? (any ? 1u : 0u) : 0u;
            __syncwarp();
            if (any) {
              for (int i = lane; i < boxes; i += 32) {
                int row, z;
                if (lookup(i, row, z)) continue;
                for (int key = i * p.box; key < (i + 1) * p.box; ++key)
                  atomicOr(const_cast<uint32_t*>(fl) + 1 + (key >> 5), 1u << (key & 31));
              }
              __syncwarp();
            }
            if (lane == 0) ptx::mbar_arrive_expect_tx(full_k, bytes);
            __syncwarp();
            auto copy = [&](const CUtensorMap* map, uint32_t dst, uint32_t full) {
              for (int i = lane; i < boxes; i += 32) {
                int row = row0, z = z0;
                if (i != lane) lookup(i, row, z);
                else if (!good) {
                  row = 0;
                  z = p.n_pages * p.h_kv;
                }
                if constexpr (RAW) {
                  ptx::tma_load_3d(dst + i * pitch, map, full, 0, row, z, pol_kv);
                } else {
                  for (int c = 0; c < C::CHUNKS; ++c)
                    ptx::tma_load_3d(dst + c * C::CHUNK_BYTES + i * pitch, map, full, c * 64, row, z, pol_kv);
                }
              }
            };
            copy(&tm_k, RAW ? s_base + C::OFF_RAW : s_k + s * C::TILE_BYTES, full_k);
            ok = __all_sync(0xffffffffu, wait_bar(empty_v, eph, abort_flag, SINGLE));
            if (!ok) {
              if (lane == 0) drain_wait(full_k, fph);
              break;
            }
            if (lane == 0) ptx::mbar_arrive_expect_tx(full_v, bytes);
            __syncwarp();
            copy(&tm_v, RAW ? s_base + C::OFF_RAW + C::RAW_BYTES : s_v + s * C::TILE_BYTES, full_v);
          }
          ++ring;
        }
      }
      if (!ok && lane == 0) {
        // copies in flight must land before this CTA's shared memory goes away
        if (n_q > 0) drain_wait(bar(C::B_QFULL), (n_q - 1) & 1);
        for (uint32_t x = ring > STAGES ? ring - STAGES : 0; x < ring; ++x) {
          if (KIND == PAGED8) {
            drain_wait(bar(C::B_RAWFULL), x & 1);
            drain_wait(bar(C::B_RAWFULL + 1), x & 1);
          } else {
            drain_wait(bar(C::B_KFULL + x % STAGES), (x / STAGES) & 1);
            drain_wait(bar(C::B_VFULL + x % STAGES), (x / STAGES) & 1);
          }
        }
      }
      __syncwarp();
      }
    } else if (SINGLE && warp == C::WARP_MMA) {
      uint32_t n_q = 0;  // units with keys so far
      for (int batch = 0, n_b; (n_b = next_batch(batch)) > 0; ++batch) {
      // ================================================================ S = Q K^T (one row tile)
      if (lane == 0) {
        for (int b = 0; b < n_b && ok; ++b) {
          const int n = units[b].n;
          if (n == 0) continue;
          ok = wait_bar(bar(C::B_QFULL), n_q & 1, abort_flag, true);
          ++n_q;
          for (int j = 0; j < n && ok; ++j) {
            const int s = ring % STAGES;
            ok = wait_bar(bar(C::B_KFULL + s), (ring / STAGES) & 1, abort_flag, true) &&
                 (ring == 0 || wait_bar(bar(C::B_SFREE), (ring - 1) & 1, abort_flag, true));
            if (!ok) break;
            ptx::tc_fence_after();
            const uint32_t k_stage = s_k + s * C::TILE_BYTES;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t koff = (kk >> 2) * C::CHUNK_BYTES + (kk & 3) * 32;
              ptx::mma_ss(tmem, ptx::sdesc_sw128(s_q + koff, 16, 1024), ptx::sdesc_sw128(k_stage + koff, 16, 1024),
                          C::IDESC_S, kk > 0 ? 1u : 0u);
            }
            ptx::mma_commit(bar(C::B_SFULL));
            if (KIND != DENSE) ptx::mbar_arrive(bar(C::B_SFULL));
            ptx::mma_commit(bar(C::B_KEMPTY + s));
            ++ring;
          }
          if (ok) ptx::mma_commit(bar(C::B_QEMPTY));
        }
        if (!ok) {
          ptx::mma_commit(bar(C::B_DRAIN));
          drain_wait(bar(C::B_DRAIN), 0);
        }
      }
      __syncwarp();
      }
    } else if (SINGLE && warp == C::WARP_PV) {
      for (int batch = 0, n_b; (n_b = next_batch(batch)) > 0; ++batch) {
      // ================================================================ O += P V (one row tile)
      if (lane == 0) {
        for (int b = 0; b < n_b && ok; ++b) {
          const plan::Entry& e = units[b];
          const int n = e.n, len = e.str_len;
          for (int j = 0; j < n && ok; ++j) {
            const int s = ring % STAGES;
            const bool tail = (tile_of(e, j) + 1) * BN > len;
            ok = wait_bar(bar(C::B_VFULL + s), (ring / STAGES) & 1, abort_flag, true);
            if (!ok) break;
            if (tail) ptx::mbar_arrive(bar(C::B_TAILREQ));
            ok = wait_bar(bar(C::B_PFULL), ring & 1, abort_flag, true) &&
                 (!tail || wait_bar(bar(C::B_TAIL), tails & 1, abort_flag, true));
            if (!ok) break;
            tails += tail;
            ptx::tc_fence_after();
            const uint32_t v_stage = s_v + s * C::TILE_BYTES;
#pragma unroll
            for (int kk = 0; kk < BN / 16; ++kk)
              ptx::mma_ts(tmem + C::TMEM_O, tmem + C::TMEM_P + kk * 8,
                          ptx::sdesc_sw128(v_stage + kk * 2048, C::CHUNK_BYTES, 1024), C::IDESC_PV,
                          (j > 0 || kk > 0) ? 1u : 0u);
            ptx::mma_commit(bar(C::B_ODONE));
            ptx::mma_commit(bar(C::B_VEMPTY + s));
            ++ring;
          }
        }
        if (!ok) {
          ptx::mma_commit(bar(C::B_DRAIN + 1));
          drain_wait(bar(C::B_DRAIN + 1), 0);
        }
      }
      __syncwarp();
      }
    } else if (!SINGLE && warp == C::WARP_MMA) {
      uint32_t n_q = 0;             // units with keys so far
      uint32_t cnt0 = 0, cnt1 = 0;  // key tiles of row tile 0 and 1 so far
      bool pend = false, pend0 = false, pend1 = false, acc0 = false, acc1 = false, pend_tail = false;  // PVs not yet issued
      for (int batch = 0, n_b; (n_b = next_batch(batch)) > 0; ++batch) {
      // ================================================================ both products of two row tiles
      // P_t lies in S_t, so S_t(j) follows PV_t(j - 1). In order PV0(j - 1), S0(j), PV1(j - 1), S1(j),
      // over all units as one stream: a unit's last PV waits for the softmax while the next one's
      // keys are on their way. Only where a unit starts do both PVs come first, since S needs
      // the new Q.
      if (lane == 0) {
        auto issue_pv = [&](int t, uint32_t cnt, bool acc) -> bool {
          if (!wait_bar(bar(C::B_PFULL + t), (cnt - 1) & 1, abort_flag)) return false;
          ptx::tc_fence_after();
          const uint32_t v_stage = s_v + ((ring - 1) % STAGES) * C::TILE_BYTES;
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk)
            ptx::mma_ts(tmem + C::TMEM_O + t * D, tmem + t * BN + kk * 8,
                        ptx::sdesc_sw128(v_stage + kk * 2048, C::CHUNK_BYTES, 1024), C::IDESC_PV,
                        (acc || kk > 0) ? 1u : 0u);
          ptx::mma_commit(bar(C::B_ODONE + t));
          return true;
        };
        auto issue_s = [&](int t) {
          const uint32_t q_tile = s_q + t * C::TILE_BYTES, k_stage = s_k + (ring % STAGES) * C::TILE_BYTES;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t koff = (kk >> 2) * C::CHUNK_BYTES + (kk & 3) * 32;
            ptx::mma_ss(tmem + t * BN, ptx::sdesc_sw128(q_tile + koff, 16, 1024),
                        ptx::sdesc_sw128(k_stage + koff, 16, 1024), C::IDESC_S, kk > 0 ? 1u : 0u);
          }
          ptx::mma_commit(bar(C::B_SFULL + t));
          if (KIND != DENSE) ptx::mbar_arrive(bar(C::B_SFULL + t));
        };
        // the values of the ring use before this one, for the PVs still to come
        auto values = [&]() -> bool {
          const uint32_t s = (ring - 1) % STAGES;
          if (!wait_bar(bar(C::B_VFULL + s), ((ring - 1) / STAGES) & 1, abort_flag)) return false;
          if (!pend_tail) return true;
          ptx::mbar_arrive(bar(C::B_TAILREQ));
          pend_tail = false;
          return wait_bar(bar(C::B_TAIL), tails++ & 1, abort_flag);
        };
        auto flush = [&]() -> bool {
          if (!values()) return false;
          if (pend0 && !issue_pv(0, cnt0, acc0)) return false;
          if (pend1 && !issue_pv(1, cnt1, acc1)) return false;
          ptx::mma_commit(bar(C::B_VEMPTY + (ring - 1) % STAGES));
          pend = false;
          return true;
        };
        for (int b = 0; b < n_b && ok; ++b) {
          const plan::Entry& e = units[b];
          const int n = e.n, len = e.str_len;
          if (n == 0) continue;
          const int lo0 = e.lo0, hi0 = e.hi0, lo1 = e.lo1, hi1 = e.hi1;
          if (pend) ok = flush();
          ok = ok && wait_bar(bar(C::B_QFULL), n_q & 1, abort_flag);
          ++n_q;
          for (int j = 0; j < n && ok; ++j) {
            ok = wait_bar(bar(C::B_KFULL + ring % STAGES), (ring / STAGES) & 1, abort_flag) && (!pend || values());
            if (!ok) break;
            ptx::tc_fence_after();
            if (pend && pend0 && !(ok = issue_pv(0, cnt0, acc0))) break;
            const bool in0 = j >= lo0 && j < hi0, in1 = j >= lo1 && j < hi1;
            if (in0) {
              issue_s(0);
              ++cnt0;
            }
            if (pend && pend1 && !(ok = issue_pv(1, cnt1, acc1))) break;
            if (in1) {
              issue_s(1);
              ++cnt1;
            }
            ptx::mma_commit(bar(C::B_KEMPTY + ring % STAGES));
            if (pend) ptx::mma_commit(bar(C::B_VEMPTY + (ring - 1) % STAGES));
            pend = true;
            pend0 = in0;
            pend1 = in1;
            acc0 = j > lo0;
            acc1 = j > lo1;
            pend_tail = KIND != PAGED8 && (tile_of(e, j) + 1) * BN > len;
            ++ring;
          }
          if (ok) ptx::mma_commit(bar(C::B_QEMPTY));
        }
        if (ok && pend) ok = flush();
        if (!ok) {
          ptx::mma_commit(bar(C::B_DRAIN));
          drain_wait(bar(C::B_DRAIN), 0);
        }
      }
      __syncwarp();
      }
    } else if (KIND != PAGED8 && warp == C::WARP_TAIL) {
      for (int batch = 0, n_b; (n_b = next_batch(batch)) > 0; ++batch) {
      // ================================================================ values behind the end: zero
      for (int b = 0; b < n_b && ok; ++b) {
        const plan::Entry& e = units[b];
        const int n = e.n, len = e.str_len;
        for (int j = 0; j < n && ok; ++j, ++ring) {
          const int there = len - tile_of(e, j) * BN;
          if (there >= BN) continue;
          const int s = ring % STAGES;
          ok = __all_sync(0xffffffffu, wait_bar(bar(C::B_TAILREQ), tails++ & 1, abort_flag, true));
          if (!ok) break;
          for (int c = 0; c < C::CHUNKS; ++c)
            for (int x = there * 8 + lane; x < BN * 8; x += 32)
              ptx::st_shared_v4(s_v + s * C::TILE_BYTES + c * C::CHUNK_BYTES + x * 16, 0, 0, 0, 0);
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(bar(C::B_TAIL));
        }
      }
      }
    } else {  // no role
      for (int batch = 0; next_batch(batch) > 0; ++batch) {
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
// their order. A warp per row, D / 32 columns per lane.
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
  constexpr int W = D / 32;
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int n_join = p.head->n_join;
  const int lane = threadIdx.x & 31;
  const long long warps = (long long)gridDim.x * 8;
  const size_t slot_floats = (size_t)p.rows * (D + 2);
  for (long long x = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); x < (long long)n_join * p.rows; x += warps) {
    const plan::Join j = p.joins[x / p.rows];
    const int row = (int)(x % p.rows), t = row / BM, r = row % BM;
    const int rt = r / p.group, tok = t * p.tok + rt;
    if (rt >= p.tok || tok >= j.own_n) continue;
    auto slot = [&](int i) { return p.part + (size_t)(i == 0 ? j.slot : j.next + 2 * (i - 1)) * slot_floats; };
    float m = -INFINITY;
    for (int i = lane; i < j.pieces; i += 32) m = fmaxf(m, slot(i)[(size_t)p.rows * D + row]);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float sum = 0.0f, o[W] = {};
#pragma unroll 4
    for (int i = 0; i < j.pieces; ++i) {
      const float* s = slot(i);
      const float mi = s[(size_t)p.rows * D + row], li = s[(size_t)p.rows * (D + 1) + row];
      const float w = mi == -INFINITY ? 0.0f : exp2f(mi - m);
      sum += w * li;
      const float* v = s + (size_t)row * D + lane * W;
      if (w != 0.0f) {
#pragma unroll
        for (int y = 0; y < W; ++y) o[y] += w * v[y];
      }
    }
    const int head_q = j.hk * p.group + (r - rt * p.group);
    const long long at = (long long)j.own_row + tok;
    const float inv = sum == 0.0f ? 0.0f : (p.v_scale ? p.v_scale[j.hk] : 1.0f) / sum;
    uint32_t* to = reinterpret_cast<uint32_t*>(p.out + at * p.out_ts + head_q * p.out_hs) + lane * (W / 2);
#pragma unroll
    for (int y = 0; y < W; y += 2) to[y / 2] = ptx::pack_bf16x2(o[y] * inv, o[y + 1] * inv);
    if (lane == 0 && p.lse)
      p.lse[at * p.h_q + head_q] = sum == 0.0f ? -INFINITY : (m + log2f(sum)) * 0.69314718055994530942f;
  }
}

int gcd_128(int x) {
  int r = 1;
  while (r < 128 && x % (2 * r) == 0) r *= 2;
  return r;
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

// (d, row, z) with the given strides in elements.
CUresult encode_rows(PFN_encodeTiled enc, CUtensorMap* map, const void* base, int d, long long rows, long long z,
                     long long row_stride, long long z_stride, int box_rows, bool bytes) {
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)rows, (cuuint64_t)z};
  const int size = bytes ? 1 : 2;
  cuuint64_t strides[2] = {(cuuint64_t)row_stride * size, (cuuint64_t)z_stride * size};
  cuuint32_t box[3] = {(cuuint32_t)(bytes ? d : 64), (cuuint32_t)box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base),
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
bool launch(Kernel* kernel, unsigned grid, unsigned threads, size_t smem, cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
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

template <int D, int KIND>
int run(const PackedArgs& a, PFN_encodeTiled enc, void* workspace) {
  using C = Cfg<D, KIND>;
  const Geometry g = geometry_of<D, KIND>(a.T_q, a.B, a.h_q, a.h_kv);
  static std::atomic<bool> attr_done[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return ATTN_ERR_CUDA;
  if (!attr_done[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(attn_packed_kernel<D, KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES) !=
        cudaSuccess)
      return ATTN_ERR_CUDA;
    attr_done[dev].store(true, std::memory_order_release);
  }
  CUtensorMap mq, mk, mv;
  const int box = KIND == DENSE ? BN : gcd_128(a.page_size);
  if (encode_q(enc, &mq, a, D, g.group, g.tok) != CUDA_SUCCESS) return ATTN_ERR_UNSUPPORTED;
  for (int x = 0; x < 2; ++x) {
    const CUresult st =
        KIND == DENSE
            ? encode_rows(enc, x ? &mv : &mk, x ? a.v : a.k, D, a.T_k, a.h_kv, x ? a.v_ts : a.k_ts, x ? a.v_hs : a.k_hs,
                          BN, false)
            : encode_rows(enc, x ? &mv : &mk, x ? a.v : a.k, D, a.page_size, (long long)a.n_pages * a.h_kv, D,
                          (long long)D * a.page_size, box, KIND == PAGED8);
    if (st != CUDA_SUCCESS) return ATTN_ERR_UNSUPPORTED;
  }
  const long long reach = KIND == DENSE ? a.T_k : (long long)a.max_pages * a.page_size;
  // no sequence has more tiles than a CTA's least share, so none is longer than one: nothing to cut
  const bool may_cut = (reach + BN - 1) / BN > kMinShare;
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
  pa.max_deal = kMaxDeal;
  pa.may_cut = may_cut;
  plan::place(pa, workspace, g.items);
  Params p = {};
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
  p.page_table = a.page_table;
  p.max_pages = a.max_pages;
  p.n_pages = a.n_pages;
  p.page_size = a.page_size;
  p.box = box;
  p.h_kv = a.h_kv;
  p.k_scale = a.k_scale;
  p.v_scale = a.v_scale;
  if (!launch(plan::attn_plan_kernel, 1, plan::THREADS, 0, a.stream, pa)) return ATTN_ERR_CUDA;
  if (!launch(attn_packed_kernel<D, KIND>, (unsigned)g.ctas, C::THREADS, C::SMEM_BYTES, a.stream, mq, mk, mv, p))
    return ATTN_ERR_CUDA;
  if (may_cut) {
    const JoinParams j = {pa.head, pa.joins, p.part, p.out,  p.lse,  p.out_ts,
                          p.out_hs, p.h_q,    p.group, p.tok, C::ROWS, KIND == PAGED8 ? p.v_scale : nullptr};
    if (!launch(attn_join_kernel<D>, kSms * 4, 256, 0, a.stream, j)) return ATTN_ERR_CUDA;
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
  if (!a.k_scale) return a.d == 64 ? run<64, PAGED>(a, enc, workspace) : run<128, PAGED>(a, enc, workspace);
  return a.d == 64 ? run<64, PAGED8>(a, enc, workspace) : run<128, PAGED8>(a, enc, workspace);
}

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
