// attn_packed_bwd.cu -- gradients of attn_packed_fwd (dQ, dK, dV of packed sequences whose query
// heads share key/value heads) on the sm_103a tensor cores, bf16 in and out, fp32 accumulation.
//
//   P_ij = exp(scale q_i . k_j - lse_i) on legal pairs, else 0
//   dV = P^T dO,  dP = dO V^T,  dS = P (dP - D),  D_i = dO_i . O_i,  dQ = scale dS K,  dK = scale dS^T Q
// dK and dV of a key/value head are sums over its g = h_q / h_kv query heads.
//
// Rows are packed as in attn_packed.cu: a row tile is floor(128 / g) tokens times g heads, so the
// sums over the group are part of the products' own sums over rows, without atomics or copies.
//
// Two passes of one kernel: own rows stay in shared memory, the other side's tiles of 128 rows stream through a ring
// in halves, with an MMA issuer and a warpgroup for the elementwise part per half.
//   keys own   (dK, dV) S^T = K Q_i^T, dP^T = V dO_i^T, then dV += P^T dO_i, dK += dS^T Q_i
//   rows own   (dQ)     S = Q K_j^T,  dP = dO V_j^T,    then dQ += dS K_j
// Seven products where the formulas have five, and in return no sums whose order varies: the same
// bits on every run. Work is handed out by attn_plan.cuh, the CTAs are persistent, and units
// that the plan cut leave fp32 sums that attn_packed_sum_kernel adds up in their order.
//
// Streamed rows that belong to other sequences (behind a sequence's last row in its last tile)
// count nothing, whatever they hold: their P and dS are set to 0, and a spare warp zeroes them in
// shared memory before the products whose sums run over them (0 times infinity is NaN). A half of a
// streamed row tile is floor(64 / g) tokens, or, for g above 64, one token's first 64 heads or the others;
// rows of the ring that no copy writes are zeroed once.
//
// What bounds it: at d = 128 the issue of the products (S and dP of half a tile are MMAs of 64 columns, which
// shared memory feeds at 49 cycles each instead of 32: both operands are read from there), then the
// seven products against five; at d = 64 the chain product, elementwise part, product of each half, and
// for short sequences the units' starts and ends. 8192 causal tokens, 32/8 heads of 128: 1670 us, 823 TFLOP/s
// of the formulas' five products; 64 sentences of 21 to 500 tokens, 8 heads of 64: 125 us.
//
// Every wait is bounded, as in attn_bwd.cu.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "attn_internal.h"
#include "attn_plan.cuh"
#include "ptx_warp.cuh"

namespace attn {

__device__ unsigned int g_packed_bwd_fault_word;

namespace {

constexpr int T = 128;  // rows per tile
constexpr int H = 64;   // rows per half of a streamed tile
// warps 0-7 elementwise (a warpgroup per half of every streamed tile), 8 copies, 9 and 10 MMA
// issuers, 11 zeroes rows of other sequences
constexpr int EW_THREADS = 256, THREADS = 384;
constexpr int WARP_LOAD = 8, WARP_MMA = 9, WARP_TAIL = 11;
constexpr int kMaxDevices = 64;
constexpr int kSms = 152;
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr uint64_t kDrainLimitNs = 200000000ull;
constexpr uint32_t FAULT_PACKED_BWD = 1024;
constexpr int UNITS = 4;      // units whose entries a CTA holds at a time
constexpr int kMinShare = 2;  // tiles

template <int D>
struct BCfg {
  // The ring holds half tiles: at d = 128 whole ones leave room for two, and a tile's place is free only when
  // the sums over the tile before are done, just when its rows are needed (8192 causal tokens, 32/8 heads of 128:
  // 1935 us with two tiles, 1663 with four halves; a fifth changes nothing).
  static constexpr int SLOTS = D == 64 ? 6 : 4;
  static constexpr int A_BUFS = D == 64 ? 2 : 1;  // 2: the next unit's own tiles are there when the last S and dP are issued
  static constexpr int CHUNKS = D / 64;
  static constexpr int CHUNK_BYTES = T * 128;
  static constexpr int TILE_BYTES = T * D * 2;
  static constexpr int OFF_A0 = 0;                                      // [A_BUFS] K, or Q; and behind each
  static constexpr int OFF_A1 = OFF_A0 + TILE_BYTES;                    // V, or dO
  static constexpr int HCHUNK_BYTES = H * 128;
  static constexpr int HALF_BYTES = H * D * 2;
  static constexpr int OFF_R0 = OFF_A0 + A_BUFS * 2 * TILE_BYTES;       // ring: Q, or K; and behind each
  static constexpr int OFF_R1 = OFF_R0 + HALF_BYTES;                    // dO, or V
  static constexpr int OFF_VEC = OFF_R0 + SLOTS * 2 * HALF_BYTES;       // float [SLOTS][-lse log2(e)[H], -D[H]], or of the own rows
  // d = 64: rows on their way out, 32 per elementwise warp
  static constexpr int OFF_STAGE = OFF_VEC + SLOTS * 2 * H * 4;
  static constexpr int OFF_UNITS = OFF_STAGE + (D == 64 ? 8 * 4096 : 0);
  static constexpr int OFF_BAR = OFF_UNITS + UNITS * 64;
  static constexpr int B_AFULL = 0, B_AEMPTY = 2, B_FULL = 4, B_EMPTY = B_FULL + SLOTS, B_MMFULL = B_EMPTY + SLOTS;
  static constexpr int B_PFULL = B_MMFULL + 2, B_ACC = B_PFULL + 2, B_TAILREQ = B_ACC + 1, B_TAIL = B_TAILREQ + 2;
  static constexpr int B_DRAIN = B_TAIL + 2, B_TURN = B_DRAIN + 2, B_UNITFULL = B_TURN + 2, B_UNITEMPTY = B_UNITFULL + UNITS,
                       NUM_BARS = B_UNITEMPTY + UNITS;
  static constexpr int OFF_SLOT = OFF_BAR + NUM_BARS * 8;
  static constexpr int OFF_ABORT = OFF_SLOT + 4;
  static constexpr int SMEM_BYTES = OFF_ABORT + 4;
  // TMEM: of half h of the streamed tile, X_h (S^T or S) and Y_h (dP^T or dP), 64 columns each; bf16
  // pairs are written back over their first 32 columns; the accumulators from column 256
  __host__ __device__ static constexpr uint32_t tm_x(int h) { return 128u * h; }
  __host__ __device__ static constexpr uint32_t tm_y(int h) { return 128u * h + 64u; }
  static constexpr uint32_t IDESC_NN = ptx::idesc_bf16_f32(T, T / 2, false);
  static constexpr uint32_t IDESC_ACC = ptx::idesc_bf16_f32(T, D, true);
  static_assert(SLOTS * H >= A_BUFS * T, "tables");
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
};

struct BwdParams {
  plan::Header* head;
  const int2* range;
  const plan::Entry* list;
  const float* stats;  // [2][h_kv][T_q g]: -lse log2(e), then -D, by packed row
  long long rows;      // T_q g
  long long stat_size;  // h_kv T_q g
  uint16_t* g0;        // dK, or dQ
  uint16_t* g1;        // dV
  long long g0_ts, g0_hs, g1_ts, g1_hs;
  int group, tok, T_q, h_kv;  // tok: tokens per row tile
  // keys own: a half of a row tile is half_tok tokens times half_per rows; half 1 starts half_step tokens behind half 0
  int half_tok, half_per, half_step;
  int causal, window;
  float scale, scale_log2;
  float* part;  // [slots][T][accumulator columns]
};

__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = ptx::globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    if ((it & 63u) == 0) {
      if (*abort_flag) return false;
      if (ptx::globaltimer_ns() - t0 > kWaitLimitNs) {
        *abort_flag = 1;
        atomicOr(&g_packed_bwd_fault_word, FAULT_PACKED_BWD);
        return false;
      }
    }
  }
}

__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = ptx::globaltimer_ns();
  while (!ptx::mbar_try_wait(bar, parity))
    if (ptx::globaltimer_ns() - t0 > kDrainLimitNs) return;
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* tmap, uint32_t bar, int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}
__device__ __forceinline__ void tma_load_rows(uint32_t dst, const void* tmap, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void copy_word(uint32_t dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// Arrives on `bar` when this thread's copies so far have landed (an arrival that the barrier counts).
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// ------------------------------------------------------------------ plans and D_i = dO_i . O_i
// Blocks 0 and 1 write the two passes' work lists; the others' warps the table of -lse log2(e) and
// -D of every row of the packed array, D / 8 lanes per row, all loads of a warp's rows first. Rows of
// no sequence get whatever they hold: nothing reads them.
constexpr int DOT_STEPS = 4;
struct DotParams {
  const uint16_t* out;
  const uint16_t* dout;
  const float* lse;
  float* stats;
  long long out_ts, out_hs, dout_ts, dout_hs;
  long long n;  // T_q h_q
  long long T_q;
  int h_q, group;
};

template <int D>
__global__ void __launch_bounds__(plan::THREADS) attn_packed_bwd_prepare_kernel(const plan::Args keys, const plan::Args rows,
                                                                              const DotParams p) {
  ptx::grid_dep_launch();
  if (blockIdx.x < 2) {
    __shared__ plan::Scratch scratch;
    plan::write(blockIdx.x == 0 ? keys : rows, scratch);
    return;
  }
  ptx::grid_dep_wait();
  constexpr int LPR = D / 8, RPS = 32 / LPR;
  const int lane = threadIdx.x & 31, cg = lane % LPR;
  const long long first = ((long long)(blockIdx.x - 2) * (plan::THREADS / 32) + (threadIdx.x >> 5)) * (RPS * DOT_STEPS) + lane / LPR;
  uint4 o4[DOT_STEPS], g4[DOT_STEPS];
#pragma unroll
  for (int u = 0; u < DOT_STEPS; ++u) {
    const long long x = first + (long long)u * RPS;  // token * h_q + head
    o4[u] = g4[u] = make_uint4(0, 0, 0, 0);
    if (x < p.n) {
      const long long tok = x / p.h_q;
      const int head = (int)(x - tok * p.h_q);
      o4[u] = *(reinterpret_cast<const uint4*>(p.out + tok * p.out_ts + head * p.out_hs) + cg);
      g4[u] = *(reinterpret_cast<const uint4*>(p.dout + tok * p.dout_ts + head * p.dout_hs) + cg);
    }
  }
#pragma unroll
  for (int u = 0; u < DOT_STEPS; ++u) {
    const uint32_t a[4] = {o4[u].x, o4[u].y, o4[u].z, o4[u].w}, b[4] = {g4[u].x, g4[u].y, g4[u].z, g4[u].w};
    float acc = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      acc = fmaf(__uint_as_float(a[e] << 16), __uint_as_float(b[e] << 16), acc);
      acc = fmaf(__uint_as_float(a[e] & 0xffff0000u), __uint_as_float(b[e] & 0xffff0000u), acc);
    }
#pragma unroll
    for (int off = 1; off < LPR; off <<= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
    const long long x = first + (long long)u * RPS;
    if (cg == 0 && x < p.n) {
      const long long tok = x / p.h_q;
      const int head = (int)(x - tok * p.h_q), hk = head / p.group;
      float* dst = p.stats + ((long long)hk * p.T_q + tok) * p.group + (head - hk * p.group);
      dst[0] = -p.lse[x] * 1.4426950408889634f;
      dst[p.n] = -acc;
    }
  }
}

// ------------------------------------------------------------------ one pass
template <int D, bool DKDV>
__global__ void __launch_bounds__(THREADS, 1)
    attn_packed_bwd_kernel(const __grid_constant__ CUtensorMap tm_a0, const __grid_constant__ CUtensorMap tm_a1,
                           const __grid_constant__ CUtensorMap tm_r0, const __grid_constant__ CUtensorMap tm_r1,
                           const BwdParams p) {
  using C = BCfg<D>;
  constexpr int SLOTS = C::SLOTS;
  constexpr int ACC_COLS = DKDV ? 2 * D : D;  // of a piece
  auto acc_col = [](int which) -> uint32_t { return 256u + which * D; };
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t s_base = ptx::smem_u32(smem);
  if ((s_base & 1023u) != 0) {
    if (threadIdx.x == 0) atomicOr(&g_packed_bwd_fault_word, FAULT_PACKED_BWD);
    return;
  }
  auto bar = [&](int x) -> uint32_t { return s_base + C::OFF_BAR + 8u * x; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_ABORT);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_SLOT);
  const plan::Entry* units = reinterpret_cast<const plan::Entry*>(smem + C::OFF_UNITS);
  const float* vec = reinterpret_cast<const float*>(smem + C::OFF_VEC);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // uniform: see the issuing warps
  const int row_tile = p.tok * p.group;            // rows of a row tile (rows own)
  const int half_rows = p.half_tok * p.half_per;  // rows that a half's copies write (keys own)

  if (threadIdx.x == 0) {
    for (int b = 0; b < C::A_BUFS; ++b) {
      ptx::mbar_init(bar(C::B_AFULL + b), DKDV ? 1 : 33);  // bytes, and the copy warp's lanes for the table
      ptx::mbar_init(bar(C::B_AEMPTY + b), DKDV ? 2 : 2 + 8);  // issuers; elementwise warps, which read the table
    }
    for (int s = 0; s < SLOTS; ++s) {
      ptx::mbar_init(bar(C::B_FULL + s), DKDV ? 33 : 1);  // bytes, and the copy warp's lanes for the table
      ptx::mbar_init(bar(C::B_EMPTY + s), 1);
    }
    for (int h = 0; h < 2; ++h) {
      ptx::mbar_init(bar(C::B_MMFULL + h), 1);
      ptx::mbar_init(bar(C::B_PFULL + h), EW_THREADS / 2);
      ptx::mbar_init(bar(C::B_TAILREQ + h), 1);
      ptx::mbar_init(bar(C::B_TAIL + h), 1);
      ptx::mbar_init(bar(C::B_DRAIN + h), 1);
      ptx::mbar_init(bar(C::B_TURN + h), 1);
    }
    ptx::mbar_init(bar(C::B_ACC), 2);
    for (int u = 0; u < UNITS; ++u) {
      ptx::mbar_init(bar(C::B_UNITFULL + u), 1);
      ptx::mbar_init(bar(C::B_UNITEMPTY + u), 8 + 2 + 1);  // elementwise, issuing and tail warps
    }
    *abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (DKDV) {
    // rows of the ring, and of the table, that no copy writes
    for (int x = threadIdx.x; x < SLOTS * 2 * C::CHUNKS * (H - half_rows) * 8; x += THREADS) {
      const int slab = x / ((H - half_rows) * 8), at = x % ((H - half_rows) * 8);
      ptx::st_shared_v4(s_base + C::OFF_R0 + slab * C::HCHUNK_BYTES + half_rows * 128 + at * 16, 0, 0, 0, 0);
    }
    for (int x = threadIdx.x; x < SLOTS * 2 * H; x += THREADS) reinterpret_cast<float*>(smem + C::OFF_VEC)[x] = 0.0f;
    ptx::fence_proxy_async_smem();
  }
  if (warp == WARP_MMA) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), 512);
    ptx::tmem_relinquish();
  }
  if (warp == WARP_LOAD && lane == 0) {
    ptx::prefetch_tmap(&tm_a0);
    ptx::prefetch_tmap(&tm_a1);
    ptx::prefetch_tmap(&tm_r0);
    ptx::prefetch_tmap(&tm_r1);
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();

  // The copy warp passes the units' entries on through a ring of UNITS places; every other warp
  // runs through them in that order, each at its own pace. n < 0: no more units.
  auto unit_wait = [&](uint32_t un) -> bool { return wait_bar(bar(C::B_UNITFULL + un % UNITS), (un / UNITS) & 1, abort_flag); };
  auto unit_done = [&](uint32_t un) { ptx::mbar_arrive(bar(C::B_UNITEMPTY + un % UNITS)); };
  // Rows of half h of streamed tile j that belong to the sequence, when they are not all (else H or more).
  auto there = [&](const plan::Entry& e, int j, int h) -> int {
    const int tile = e.j0 + j + e.skip;
    const int left = max(e.str_len - tile * (DKDV ? p.tok : T) - h * (DKDV ? p.half_step : H), 0);
    return DKDV ? (left >= p.half_tok ? H : left * p.half_per) : left;
  };

  // All lanes of a warp together.
  auto wait_warp = [&](uint32_t b, uint32_t parity, volatile int* flag) -> bool {
    return __all_sync(0xffffffffu, wait_bar(b, parity, flag));
  };

  uint32_t ring = 0;  // streamed tiles so far (copies: half tiles)
  auto half_use = [](uint32_t tile, int h) -> uint32_t { return 2 * tile + h; };  // of the ring: place modulo SLOTS
  bool ok = true;

  if (warp == WARP_LOAD) {
    // ================================================================ copies
    uint32_t n_a = 0;  // units with tiles so far
    const plan::Header head = *p.head;
    plan::Turn turn(head, p.range, p.h_kv);
    auto next_unit = [&]() -> int { return __shfl_sync(0xffffffffu, lane == 0 ? turn.next(p.head) : 0, 0); };
    auto word_of = [&](int u) -> int { return turn.word(p.list, u, lane & 15); };
    int word = word_of(next_unit());  // lane x: word x of the entry; all -1: no more units
    {
      for (uint32_t un = 0;; ++un) {
        ok = __all_sync(0xffffffffu, wait_bar(bar(C::B_UNITEMPTY + un % UNITS), ((un / UNITS) & 1) ^ 1, abort_flag));
        if (!ok) break;
        if (lane < 16) reinterpret_cast<int*>(smem + C::OFF_UNITS)[(un % UNITS) * 16 + lane] = word;
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(C::B_UNITFULL + un % UNITS));
        const int n = __shfl_sync(0xffffffffu, word, 9);
        if (n < 0) break;
        word = word_of(next_unit());
        const plan::Entry& e = units[un % UNITS];  // stays: this warp alone replaces it
        if (n == 0) continue;
        const uint32_t ab = n_a % C::A_BUFS, a_full = bar(C::B_AFULL + ab);
        ok = __all_sync(0xffffffffu, wait_bar(bar(C::B_AEMPTY + ab), ((n_a / C::A_BUFS) & 1) ^ 1, abort_flag));
        if (!ok) break;
        if (lane == 0) {
          ptx::mbar_arrive_expect_tx(a_full, 2 * C::CHUNKS * (DKDV ? T : row_tile) * 128);
          for (int c = 0; c < C::CHUNKS; ++c) {
            const uint32_t a0 = s_base + C::OFF_A0 + ab * 2 * C::TILE_BYTES + c * C::CHUNK_BYTES, a1 = a0 + C::TILE_BYTES;
            if (DKDV) {
              tma_load_rows(a0, &tm_a0, a_full, c * 64, e.own_row, e.hk);
              tma_load_rows(a1, &tm_a1, a_full, c * 64, e.own_row, e.hk);
            } else {
              tma_load_4d(a0, &tm_a0, a_full, c * 64, 0, e.own_row, e.hk);
              tma_load_4d(a1, &tm_a1, a_full, c * 64, 0, e.own_row, e.hk);
            }
          }
        }
        if (!DKDV) {
          const int rows = min(row_tile, (p.T_q - e.own_row) * p.group);
          const float* src = p.stats + e.hk * p.rows + (long long)e.own_row * p.group;
          const uint32_t dst = s_base + C::OFF_VEC + ab * 2 * T * 4;
          for (int x = lane; x < rows; x += 32) {
            copy_word(dst + x * 4, src + x);
            copy_word(dst + (T + x) * 4, src + p.stat_size + x);
          }
          copies_arrive(a_full);
        }
        ++n_a;
        for (int jh = 0; jh < 2 * n; ++jh) {
          const int st = ring % SLOTS, h = jh & 1, tile = e.j0 + (jh >> 1) + e.skip;
          ok = __all_sync(0xffffffffu, wait_bar(bar(C::B_EMPTY + st), ((ring / SLOTS) & 1) ^ 1, abort_flag));
          if (!ok) break;
          const uint32_t full = bar(C::B_FULL + st);
          const int tok0 = e.str_row + tile * p.tok + h * p.half_step;          // keys own: first token of the half
          const int head0 = DKDV && p.half_step == 0 ? h * H : 0;               // and first head (more than H of them)
          if (lane == 0) {
            ptx::mbar_arrive_expect_tx(full, 2 * C::CHUNKS * (DKDV ? half_rows : H) * 128);
            for (int c = 0; c < C::CHUNKS; ++c) {
              const uint32_t r0 = s_base + C::OFF_R0 + st * 2 * C::HALF_BYTES + c * C::HCHUNK_BYTES, r1 = r0 + C::HALF_BYTES;
              if (DKDV) {
                tma_load_4d(r0, &tm_r0, full, c * 64, head0, tok0, e.hk);
                tma_load_4d(r1, &tm_r1, full, c * 64, head0, tok0, e.hk);
              } else {
                tma_load_rows(r0, &tm_r0, full, c * 64, e.str_row + tile * T + h * H, e.hk);
                tma_load_rows(r1, &tm_r1, full, c * 64, e.str_row + tile * T + h * H, e.hk);
              }
            }
          }
          if (DKDV) {
            const int rows = min(min(half_rows, p.group * p.half_tok - head0), (p.T_q - tok0) * p.group - head0);
            const float* src = p.stats + e.hk * p.rows + (long long)tok0 * p.group + head0;
            const uint32_t dst = s_base + C::OFF_VEC + st * 2 * H * 4;
            for (int x = lane; x < rows; x += 32) {
              copy_word(dst + x * 4, src + x);
              copy_word(dst + (H + x) * 4, src + p.stat_size + x);
            }
            copies_arrive(full);
          }
          ++ring;
        }
        if (!ok) break;
      }
      if (!ok && lane == 0) {
        for (int b = 0; b < C::A_BUFS; ++b)
          if (n_a > (uint32_t)b) drain_wait(bar(C::B_AFULL + b), ((n_a - 1 - b) / C::A_BUFS) & 1);
        for (uint32_t x = ring > SLOTS ? ring - SLOTS : 0; x < ring; ++x) drain_wait(bar(C::B_FULL + x % SLOTS), (x / SLOTS) & 1);
      }
    }
  } else if (warp == WARP_MMA || warp == WARP_MMA + 1) {
    // ================================================================ MMA issuers
    // A warp per half of the streamed tiles: the sums of the tile before, then S and dP; where a unit starts, the
    // sums come first, since S and dP need the new own tiles. They take turns, half 0 before half 1: one waits for
    // its operands while the other issues, and the sums' order is always the same.
    // The whole warp runs the loops, one lane issues: what goes into descriptors and addresses is uniform.
    auto uniform = [](uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); };
    const int hs = (int)uniform(warp - WARP_MMA);
    const uint32_t issue = lane == 0, acc = uniform(tmem);
    uint32_t n_a = 0, tails = 0, turns = 0;
    uint64_t d_own = 0;  // offset of this unit's own tiles, in descriptors
    bool pend = false, pend_tail = false, first = false;  // sums of the tile before not yet issued
    const uint64_t d_a0 = ptx::sdesc_sw128(s_base + C::OFF_A0, 16, 1024);
    const uint64_t d_a1 = ptx::sdesc_sw128(s_base + C::OFF_A1, 16, 1024);
    const uint64_t d_r0k = ptx::sdesc_sw128(s_base + C::OFF_R0, 16, 1024);
    const uint64_t d_r1k = ptx::sdesc_sw128(s_base + C::OFF_R1, 16, 1024);
    const uint64_t d_r0m = ptx::sdesc_sw128(s_base + C::OFF_R0, C::HCHUNK_BYTES, 1024);
    const uint64_t d_r1m = ptx::sdesc_sw128(s_base + C::OFF_R1, C::HCHUNK_BYTES, 1024);
    auto koff16 = [](int kk, int chunk) { return (uint64_t)(((kk >> 2) * chunk + (kk & 3) * 32) >> 4); };
    auto place = [&](uint32_t x) { return (int)uniform(half_use(x, hs) % SLOTS); };
    auto issue_sdp = [&](uint32_t x) {
      const uint64_t so = (uint64_t)((place(x) * 2 * C::HALF_BYTES) >> 4);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        ptx::mma_ss_warp(acc + C::tm_x(hs), d_a0 + d_own + koff16(kk, C::CHUNK_BYTES), d_r0k + so + koff16(kk, C::HCHUNK_BYTES), C::IDESC_NN, kk > 0 ? 1u : 0u, issue);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        ptx::mma_ss_warp(acc + C::tm_y(hs), d_a1 + d_own + koff16(kk, C::CHUNK_BYTES), d_r1k + so + koff16(kk, C::HCHUNK_BYTES), C::IDESC_NN, kk > 0 ? 1u : 0u, issue);
    };
    // the sums of this half of ring use x
    auto issue_acc = [&](uint32_t x) {
      const uint64_t so = (uint64_t)((place(x) * 2 * C::HALF_BYTES) >> 4);
      const uint32_t start = first && hs == 0 ? 0u : 1u;
      // one accumulator after the other: MMAs that change it in turn run slower
#pragma unroll
      for (int which = DKDV ? 1 : 0; which >= 0; --which)
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint64_t brow = (uint64_t)((kk * 2048) >> 4);
          const uint32_t a = acc + (which == 0 && DKDV ? C::tm_y(hs) : C::tm_x(hs)) + kk * 8;
          ptx::mma_ts_warp(acc + acc_col(which), a, (which ? d_r1m : d_r0m) + so + brow, C::IDESC_ACC, kk > 0 ? 1u : start, issue);
        }
    };
    // what the sums of ring use x read is there: this half's P and dS; and with a unit's first tile, for the issuer that
    // goes first and overwrites the accumulators, the other half's too, which says that the warps of both have
    // read them for the unit before. (Not for the second: the first may be a tile ahead by then, and a wait for a
    // phase is a wait for its parity.)
    auto stored = [&](uint32_t x) -> bool {
      if (pend_tail && !wait_warp(bar(C::B_TAIL + hs), tails++ & 1, abort_flag)) return false;
      const bool good = (!first || hs == 1 || wait_warp(bar(C::B_PFULL + 1), x & 1, abort_flag)) &&
                        wait_warp(bar(C::B_PFULL + hs), x & 1, abort_flag);
      ptx::tc_fence_after();
      return good;
    };
    auto my_turn = [&]() -> bool {
      const bool good = hs == 0 ? turns == 0 || wait_warp(bar(C::B_TURN), (turns - 1) & 1, abort_flag)
                                : wait_warp(bar(C::B_TURN + 1), turns & 1, abort_flag);
      ++turns;
      ptx::tc_fence_after();
      return good;
    };
    auto pass_on = [&]() {
      if (issue) ptx::mbar_arrive(bar(C::B_TURN + (hs ^ 1)));
    };
    for (uint32_t un = 0;; ++un) {
      if (pend) {
        // the unit's last tile; the accumulators are complete after it
        if (!(ok = stored(ring - 1) && my_turn())) break;
        issue_acc(ring - 1);
        pass_on();
        ptx::mma_commit_warp(bar(C::B_ACC), issue);
        ptx::mma_commit_warp(bar(C::B_EMPTY + place(ring - 1)), issue);
        pend = false;
      }
      if (!(ok = __all_sync(0xffffffffu, unit_wait(un)))) break;
      const plan::Entry& e = units[un % UNITS];
      const int n = (int)uniform(e.n);
      if (n < 0) break;
      const uint32_t ab = n_a % C::A_BUFS;
      if (n > 0) {
        if (!(ok = wait_warp(bar(C::B_AFULL + ab), (n_a / C::A_BUFS) & 1, abort_flag))) break;
        ++n_a;
        d_own = (uint64_t)((uniform(ab) * 2 * C::TILE_BYTES) >> 4);
      }
      for (int j = 0; j < n; ++j) {
        if (!(ok = (!pend || stored(ring - 1)) && wait_warp(bar(C::B_FULL + place(ring)), (half_use(ring, hs) / SLOTS) & 1, abort_flag) &&
                   my_turn()))
          break;
        if (pend) issue_acc(ring - 1);
        issue_sdp(ring);
        pass_on();
        ptx::mma_commit_warp(bar(C::B_MMFULL + hs), issue);
        if (pend) ptx::mma_commit_warp(bar(C::B_EMPTY + place(ring - 1)), issue);
        pend = true;
        first = j == 0;
        pend_tail = uniform(there(e, j, hs) < H) != 0;
        if (pend_tail && issue) ptx::mbar_arrive(bar(C::B_TAILREQ + hs));
        ++ring;
      }
      if (!ok) break;
      if (n > 0) ptx::mma_commit_warp(bar(C::B_AEMPTY + ab), issue);
      __syncwarp();
      if (issue) unit_done(un);
    }
    // every MMA and every arrival of this warp's commits is done before the CTA's shared memory goes
    ptx::mma_commit_warp(bar(C::B_DRAIN + hs), issue);
    drain_wait(bar(C::B_DRAIN + hs), 0);
    __syncwarp();
  } else if (warp == WARP_TAIL) {
    // ================================================================ rows of other sequences: zero
    uint32_t tails[2] = {};
    {
      for (uint32_t un = 0;; ++un) {
        ok = __all_sync(0xffffffffu, unit_wait(un));
        if (!ok) break;
        const plan::Entry& e = units[un % UNITS];
        const int n = e.n;
        if (n < 0) break;
        for (int j = 0; j < n && ok; ++j, ++ring) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int from = there(e, j, h);
            if (from >= H) continue;
            ok = __all_sync(0xffffffffu, wait_bar(bar(C::B_TAILREQ + h), tails[h]++ & 1, abort_flag));
            if (!ok) break;
            // what the sums read. Keys own: Q and dO; rows own: K
            for (int c = 0; c < (DKDV ? 2 : 1) * C::CHUNKS; ++c) {
              const uint32_t slab = s_base + C::OFF_R0 + (half_use(ring, h) % SLOTS) * 2 * C::HALF_BYTES + c * C::HCHUNK_BYTES;
              for (int x = from * 8 + lane; x < H * 8; x += 32) ptx::st_shared_v4(slab + x * 16, 0, 0, 0, 0);
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(C::B_TAIL + h));
            __syncwarp();
          }
        }
        if (!ok) break;
        if (lane == 0) unit_done(un);
        __syncwarp();
      }
    }
  } else {
    // ================================================================ elementwise (warps 0-7)
    // Thread = own row = TMEM lane; warpgroup g takes half g of every streamed tile.
    const int g = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_x = tmem + lane_off + C::tm_x(g), t_y = tmem + lane_off + C::tm_y(g);
    const uint64_t c2 = ptx::f2_pack(p.scale_log2, p.scale_log2);
    const int rt = r / p.group;  // rows own: this row's token
    uint32_t n_a = 0;
    {
      for (uint32_t un = 0;; ++un) {
        ok = __all_sync(0xffffffffu, unit_wait(un));
        if (!ok) break;
        const plan::Entry& e = units[un % UNITS];
        const int n = e.n;
        if (n < 0) break;
        const bool row_valid = DKDV ? r < e.own_n : rt < min(e.own_n, p.tok);
        // the streamed side's rows that this row pairs with: [my_lo, my_hi), query tokens or keys
        int my_lo = 0, my_hi = 0;
        uint64_t nl2 = 0ull, nd2 = 0ull;
        if (row_valid) {
          my_hi = e.str_len;
          if (DKDV) {
            const int at = e.pos + r - e.off;  // token at this key's position
            if (p.causal) my_lo = max(0, at);
            if (p.window >= 0) {
              if (!p.causal) my_lo = max(0, at - p.window);
              my_hi = min(my_hi, at + p.window + 1);
            }
          } else {
            const int at = e.pos + rt;
            if (p.causal) my_hi = min(my_hi, at + 1);
            if (p.window >= 0) {
              my_lo = max(0, at - p.window);
              if (!p.causal) my_hi = min(my_hi, at + p.window + 1);
            }
          }
        }
        if (!DKDV && n > 0) {
          const uint32_t ab = n_a % C::A_BUFS;
          ok = __all_sync(0xffffffffu, wait_bar(bar(C::B_AFULL + ab), (n_a / C::A_BUFS) & 1, abort_flag));
          if (!ok) break;
          const float nl = vec[ab * 2 * T + r], nd = vec[(ab * 2 + 1) * T + r];  // of rows that are no row: any
          nl2 = ptx::f2_pack(nl, nl);
          nd2 = ptx::f2_pack(nd, nd);
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(bar(C::B_AEMPTY + ab));
        }
        for (int j = 0; j < n; ++j, ++ring) {
          const int st = half_use(ring, g) % SLOTS;
          ok = __all_sync(0xffffffffu, wait_bar(bar(C::B_MMFULL + g), ring & 1, abort_flag));
          // the place's table: complete already, waited on for its order
          if (DKDV && ok) ok = __all_sync(0xffffffffu, wait_bar(bar(C::B_FULL + st), (half_use(ring, g) / SLOTS) & 1, abort_flag));
          if (!ok) break;
          ptx::tc_fence_after();
          // columns [lo, hi) of this half are legal; the others' P and dS are 0. Rows of a row tile
          // that no token fills are zeros in Q and dO and need no mask.
          int lo, hi;
          const int tile = e.j0 + j + e.skip;
          if (DKDV) {
            const int t0 = tile * p.tok + g * p.half_step;
            lo = min(max(my_lo - t0, 0), p.half_tok) * p.half_per;
            hi = my_hi - t0 >= p.half_tok ? H : max(my_hi - t0, 0) * p.half_per;
            if (p.half_step == 0 && g == 1) hi = min(hi, p.group - H);  // one token's other heads: the table ends with them
          } else {
            lo = my_lo - tile * T - g * 64;
            hi = my_hi - tile * T - g * 64;
          }
          const bool full = lo <= 0 && hi >= 64;
          const float* vnl = vec + st * 2 * H;
          const float* vnd = vnl + H;
#pragma unroll
          for (int ch = 0; ch < 2; ++ch) {
            uint32_t xs[32], ys[32];
            ptx::tmem_ld32(t_x + ch * 32, xs);
            ptx::tmem_ld32(t_y + ch * 32, ys);
            ptx::tmem_wait_ld();
            uint32_t pw[16], dw[16];
            float4 nl4, nd4;
#pragma unroll
            for (int x = 0; x < 32; x += 2) {
              const int cc = ch * 32 + x;
              uint64_t nl, nd;
              if (DKDV) {
                if ((x & 2) == 0) {
                  nl4 = *reinterpret_cast<const float4*>(vnl + cc);
                  nd4 = *reinterpret_cast<const float4*>(vnd + cc);
                }
                nl = (x & 2) ? ptx::f2_pack(nl4.z, nl4.w) : ptx::f2_pack(nl4.x, nl4.y);
                nd = (x & 2) ? ptx::f2_pack(nd4.z, nd4.w) : ptx::f2_pack(nd4.x, nd4.y);
              } else {
                nl = nl2;
                nd = nd2;
              }
              float a0, a1;
              ptx::f2_unpack(ptx::f2_fma(ptx::f2_pack(__uint_as_float(xs[x]), __uint_as_float(xs[x + 1])), c2, nl), a0, a1);
              float p0 = ptx::ex2(a0), p1 = ptx::ex2(a1);
              const uint64_t dp = ptx::f2_add(ptx::f2_pack(__uint_as_float(ys[x]), __uint_as_float(ys[x + 1])), nd);
              float d0, d1;
              ptx::f2_unpack(ptx::f2_mul(ptx::f2_pack(p0, p1), dp), d0, d1);
              if (!full) {  // both: what is masked may be infinite or NaN
                const bool in0 = cc >= lo && cc < hi, in1 = cc + 1 >= lo && cc + 1 < hi;
                p0 = in0 ? p0 : 0.0f;
                p1 = in1 ? p1 : 0.0f;
                d0 = in0 ? d0 : 0.0f;
                d1 = in1 ? d1 : 0.0f;
              }
              if (DKDV) pw[x >> 1] = ptx::pack_bf16x2(p0, p1);
              dw[x >> 1] = ptx::pack_bf16x2(d0, d1);
            }
            if (DKDV) ptx::tmem_st16(t_x + ch * 16, pw);
            ptx::tmem_st16((DKDV ? t_y : t_x) + ch * 16, dw);
          }
          ptx::tmem_wait_st();
          ptx::tc_fence_before();
          ptx::mbar_arrive(bar(C::B_PFULL + g));
        }
        if (!ok) break;

        // ---------------------------------------------------------------- this unit's gradients
        // keys own: warpgroup 0 writes dK, 1 dV; rows own: each half the columns of dQ
        if (n > 0) {
          ok = __all_sync(0xffffffffu, wait_bar(bar(C::B_ACC), n_a & 1, abort_flag));
          if (!ok) break;
          ++n_a;
          ptx::tc_fence_after();
        }
        constexpr int NCH = DKDV ? D / 32 : D / 64;
        const uint32_t col0 = DKDV ? acc_col(g) : acc_col(0) + g * (D / 2);
        float* part = e.slot < 0 ? nullptr : p.part + ((size_t)e.slot * T + r) * ACC_COLS + (DKDV ? g * D : g * (D / 2));
        uint16_t* to = nullptr;
        if (row_valid) {
          if (DKDV)
            to = (g ? p.g1 : p.g0) + (e.own_row + r) * (g ? p.g1_ts : p.g0_ts) + e.hk * (g ? p.g1_hs : p.g0_hs);
          else
            to = p.g0 + (e.own_row + rt) * p.g0_ts + (e.hk * p.group + r - rt * p.group) * p.g0_hs + g * (D / 2);
        }
        const float mul = DKDV && g == 1 ? 1.0f : p.scale;
        auto sums = [&](int q4, uint32_t (&o)[32]) {  // 32 columns of this row
          if (n == 0) {
#pragma unroll
            for (int x = 0; x < 32; ++x) o[x] = 0u;
            return;
          }
          ptx::tmem_ld32(tmem + lane_off + col0 + q4 * 32, o);
          ptx::tmem_wait_ld();
        };
        if (D == 64 && part == nullptr) {
          // through shared memory, so that neighbouring lanes store one row's 128 (dQ: this half's 64) bytes:
          // units of 16 bytes, swizzled by the row
          constexpr int U = NCH * 4;  // units per row
          const uint32_t stage = s_base + C::OFF_STAGE + warp * 4096;
#pragma unroll
          for (int q4 = 0; q4 < NCH; ++q4) {
            uint32_t o[32], w[16];
            sums(q4, o);
#pragma unroll
            for (int x = 0; x < 16; ++x)
              w[x] = ptx::pack_bf16x2(__uint_as_float(o[2 * x]) * mul, __uint_as_float(o[2 * x + 1]) * mul);
#pragma unroll
            for (int u = 0; u < 4; ++u)
              ptx::st_shared_v4(stage + lane * (U * 16) + (((q4 * 4 + u) ^ (lane & (U - 1))) << 4), w[4 * u], w[4 * u + 1],
                                w[4 * u + 2], w[4 * u + 3]);
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < U; ++i) {
            const int from = i * (32 / U) + lane / U, u = lane % U;
            uint16_t* dst = reinterpret_cast<uint16_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(to), from));
            uint4 v;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                         : "r"(stage + from * (U * 16) + ((u ^ (from & (U - 1))) << 4))
                         : "memory");
            if (dst != nullptr) *reinterpret_cast<uint4*>(dst + u * 8) = v;
          }
          __syncwarp();
        } else {
#pragma unroll
          for (int q4 = 0; q4 < NCH; ++q4) {
            uint32_t o[32];
            sums(q4, o);
            if (part != nullptr) {
              if (row_valid) {
#pragma unroll
                for (int x = 0; x < 8; ++x)
                  reinterpret_cast<uint4*>(part + q4 * 32)[x] = make_uint4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
              }
            } else if (row_valid) {
              uint32_t w[16];
#pragma unroll
              for (int x = 0; x < 16; ++x)
                w[x] = ptx::pack_bf16x2(__uint_as_float(o[2 * x]) * mul, __uint_as_float(o[2 * x + 1]) * mul);
              uint4* dst = reinterpret_cast<uint4*>(to + q4 * 32);
#pragma unroll
              for (int x = 0; x < 4; ++x) dst[x] = make_uint4(w[4 * x], w[4 * x + 1], w[4 * x + 2], w[4 * x + 3]);
            }
            __syncwarp();
          }
        }
        if (lane == 0) unit_done(un);
        __syncwarp();
      }
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == WARP_MMA) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ units that were cut
// The pieces' fp32 sums added up in their order, four columns per thread.
struct SumSide {
  const plan::Header* head;
  const plan::Join* joins;
  const float* part;
};
struct SumParams {
  SumSide keys, rows;
  uint16_t *dq, *dk, *dv;
  long long dq_ts, dq_hs, dk_ts, dk_hs, dv_ts, dv_hs;
  int group, tok;
  float scale;
};

template <int D>
__global__ void __launch_bounds__(256) attn_packed_sum_kernel(const SumParams p) {
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const SumSide& s = side ? p.rows : p.keys;
    const int cols = side ? D : 2 * D, per = T * cols / 4;
    const long long all = (long long)s.head->n_join * per;
    for (long long x = (long long)blockIdx.x * 256 + threadIdx.x; x < all; x += (long long)gridDim.x * 256) {
      const plan::Join j = s.joins[x / per];
      const int at = (int)(x % per), r = at / (cols / 4), c = at % (cols / 4) * 4;
      if (side ? r / p.group >= min(j.own_n, p.tok) : r >= j.own_n) continue;
      float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int i = 0; i < j.pieces; ++i) {
        const int slot = i == 0 ? j.slot : j.next + 2 * (i - 1);
        const float4 v = *reinterpret_cast<const float4*>(s.part + ((size_t)slot * T + r) * cols + c);
        sum.x += v.x;
        sum.y += v.y;
        sum.z += v.z;
        sum.w += v.w;
      }
      uint16_t* to;
      float mul = p.scale;
      if (side) {
        const int rt = r / p.group;
        to = p.dq + (j.own_row + rt) * p.dq_ts + (j.hk * p.group + r - rt * p.group) * p.dq_hs + c;
      } else if (c < D) {
        to = p.dk + (j.own_row + r) * p.dk_ts + j.hk * p.dk_hs + c;
      } else {
        to = p.dv + (j.own_row + r) * p.dv_ts + j.hk * p.dv_hs + c - D;
        mul = 1.0f;
      }
      *reinterpret_cast<uint2*>(to) = make_uint2(ptx::pack_bf16x2(sum.x * mul, sum.y * mul), ptx::pack_bf16x2(sum.z * mul, sum.w * mul));
    }
  }
}

// [tokens, heads, d] as (d, head of the group, token, key/value head), boxes of tok tokens times so many heads.
CUresult encode_group(PFN_encodeTiled enc, CUtensorMap* map, const void* base, int d, long long tokens, int h_kv, int group,
                      int heads, int tok, long long ts, long long hs) {
  cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)group, (cuuint64_t)tokens, (cuuint64_t)h_kv};
  cuuint64_t strides[3] = {(cuuint64_t)hs * 2, (cuuint64_t)ts * 2, (cuuint64_t)hs * 2 * group};
  cuuint32_t box[4] = {64, (cuuint32_t)heads, (cuuint32_t)tok, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

CUresult encode_keys(PFN_encodeTiled enc, CUtensorMap* map, const void* base, int d, long long tokens, int h_kv, long long ts,
                     long long hs, int rows) {
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)tokens, (cuuint64_t)h_kv};
  cuuint64_t strides[2] = {(cuuint64_t)ts * 2, (cuuint64_t)hs * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

struct Sizes {
  int group, tok;                         // rows own: tokens per row tile
  int half_tok, half_per, half_step;  // keys own: see BwdParams
  int str_tok;                        // tokens per streamed row tile
  long long key_items, row_items;
  size_t key_plan, row_plan, stats, key_part, row_part;
};

Sizes sizes_of(int T_q, int T_k, int B, int h_q, int h_kv, int d) {
  Sizes s;
  s.group = h_q / h_kv;
  s.tok = T / s.group;
  // each half of a streamed row tile is whole tokens; one token of more than H heads is cut between heads
  const bool cut = s.group > H;
  s.half_tok = cut ? 1 : H / s.group;
  s.half_per = cut ? H : s.group;
  s.half_step = cut ? 0 : s.half_tok;
  s.str_tok = cut ? 1 : 2 * s.half_tok;
  s.key_items = T_k / T + B;
  s.row_items = T_q / s.tok + B;
  s.key_plan = plan::bytes(s.key_items, h_kv, B, kSms);
  s.row_plan = plan::bytes(s.row_items, h_kv, B, kSms);
  s.stats = ((size_t)2 * T_q * h_q * sizeof(float) + 255) & ~size_t(255);
  s.key_part = (size_t)2 * kSms * T * 2 * d * sizeof(float);
  s.row_part = (size_t)2 * kSms * T * d * sizeof(float);
  return s;
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

template <int D>
int run(const PackedBwdArgs& a, PFN_encodeTiled enc, void* workspace) {
  using C = BCfg<D>;
  static std::atomic<bool> attr_done[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return ATTN_ERR_CUDA;
  if (!attr_done[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(attn_packed_bwd_kernel<D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES) !=
            cudaSuccess ||
        cudaFuncSetAttribute(attn_packed_bwd_kernel<D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES) !=
            cudaSuccess)
      return ATTN_ERR_CUDA;
    attr_done[dev].store(true, std::memory_order_release);
  }
  const Sizes s = sizes_of(a.T_q, a.T_k, a.B, a.h_q, a.h_kv, D);
  CUtensorMap own[4], str[4];  // q, dout, k, v as own tiles and as halves of streamed ones
  const int heads = std::min(s.group, H);
  if (encode_group(enc, &own[0], a.q, D, a.T_q, a.h_kv, s.group, s.group, s.tok, a.q_ts, a.q_hs) != CUDA_SUCCESS ||
      encode_group(enc, &own[1], a.dout, D, a.T_q, a.h_kv, s.group, s.group, s.tok, a.dout_ts, a.dout_hs) != CUDA_SUCCESS ||
      encode_keys(enc, &own[2], a.k, D, a.T_k, a.h_kv, a.k_ts, a.k_hs, T) != CUDA_SUCCESS ||
      encode_keys(enc, &own[3], a.v, D, a.T_k, a.h_kv, a.v_ts, a.v_hs, T) != CUDA_SUCCESS ||
      encode_group(enc, &str[0], a.q, D, a.T_q, a.h_kv, s.group, heads, s.half_tok, a.q_ts, a.q_hs) != CUDA_SUCCESS ||
      encode_group(enc, &str[1], a.dout, D, a.T_q, a.h_kv, s.group, heads, s.half_tok, a.dout_ts, a.dout_hs) != CUDA_SUCCESS ||
      encode_keys(enc, &str[2], a.k, D, a.T_k, a.h_kv, a.k_ts, a.k_hs, H) != CUDA_SUCCESS ||
      encode_keys(enc, &str[3], a.v, D, a.T_k, a.h_kv, a.v_ts, a.v_hs, H) != CUDA_SUCCESS)
    return ATTN_ERR_UNSUPPORTED;
  uint8_t* at = static_cast<uint8_t*>(workspace);
  plan::Args keys = {};
  keys.q_starts = a.q_starts;
  keys.k_starts = a.k_starts;
  keys.B = a.B;
  keys.T_q = a.T_q;
  keys.T_k = a.T_k;
  keys.own_tiles = 1;
  keys.tok = s.tok;
  keys.h_kv = a.h_kv;
  keys.causal = a.causal;
  keys.window = a.window;
  keys.ctas = kSms;
  keys.min_share = kMinShare;
  plan::Args rows = keys;
  keys.own_keys = 1;
  keys.tok = s.str_tok;
  keys.may_cut = (a.T_q + s.str_tok - 1) / s.str_tok > kMinShare;
  rows.may_cut = (a.T_k + T - 1) / T > kMinShare;
  plan::place(keys, at, s.key_items);
  at += s.key_plan;
  plan::place(rows, at, s.row_items);
  at += s.row_plan;
  float* stats = reinterpret_cast<float*>(at);
  at += s.stats;
  float* key_part = reinterpret_cast<float*>(at);
  at += s.key_part;
  float* row_part = reinterpret_cast<float*>(at);

  const DotParams dot = {static_cast<const uint16_t*>(a.out), static_cast<const uint16_t*>(a.dout), a.lse, stats, a.out_ts,
                         a.out_hs, a.dout_ts, a.dout_hs, (long long)a.T_q * a.h_q, a.T_q, a.h_q, s.group};
  const long long per = (plan::THREADS / 32) * (256 / D) * DOT_STEPS;  // rows per block
  const long long blocks = 2 + (dot.n + per - 1) / per;
  if (blocks > 0x7fffffffLL) return ATTN_ERR_UNSUPPORTED;
  if (!launch(attn_packed_bwd_prepare_kernel<D>, (unsigned)blocks, plan::THREADS, 0, a.stream, keys, rows, dot))
    return ATTN_ERR_CUDA;
  BwdParams p = {};
  p.head = keys.head;
  p.range = keys.range;
  p.list = keys.list;
  p.stats = stats;
  p.rows = (long long)a.T_q * s.group;
  p.stat_size = (long long)a.T_q * a.h_q;
  p.g0 = static_cast<uint16_t*>(a.dk);
  p.g1 = static_cast<uint16_t*>(a.dv);
  p.g0_ts = a.dk_ts;
  p.g0_hs = a.dk_hs;
  p.g1_ts = a.dv_ts;
  p.g1_hs = a.dv_hs;
  p.group = s.group;
  p.tok = s.str_tok;
  p.half_tok = s.half_tok;
  p.half_per = s.half_per;
  p.half_step = s.half_step;
  p.T_q = a.T_q;
  p.h_kv = a.h_kv;
  p.causal = a.causal;
  p.window = a.window;
  p.scale = a.scale;
  p.scale_log2 = (float)((double)a.scale * 1.4426950408889634074);
  p.part = key_part;
  if (!launch(attn_packed_bwd_kernel<D, true>, kSms, THREADS, C::SMEM_BYTES, a.stream, own[2], own[3], str[0], str[1], p)) return ATTN_ERR_CUDA;
  p.tok = s.tok;
  p.head = rows.head;
  p.range = rows.range;
  p.list = rows.list;
  p.g0 = static_cast<uint16_t*>(a.dq);
  p.g0_ts = a.dq_ts;
  p.g0_hs = a.dq_hs;
  p.g1 = nullptr;
  p.part = row_part;
  if (!launch(attn_packed_bwd_kernel<D, false>, kSms, THREADS, C::SMEM_BYTES, a.stream, own[0], own[1], str[2], str[3], p)) return ATTN_ERR_CUDA;
  if (keys.may_cut || rows.may_cut) {
    const SumParams sum = {{keys.head, keys.joins, key_part},
                           {rows.head, rows.joins, row_part},
                           static_cast<uint16_t*>(a.dq),
                           static_cast<uint16_t*>(a.dk),
                           static_cast<uint16_t*>(a.dv),
                           a.dq_ts,
                           a.dq_hs,
                           a.dk_ts,
                           a.dk_hs,
                           a.dv_ts,
                           a.dv_hs,
                           s.group,
                           s.tok,
                           a.scale};
    if (!launch(attn_packed_sum_kernel<D>, kSms * 4, 256, 0, a.stream, sum)) return ATTN_ERR_CUDA;
  }
  return cudaPeekAtLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace

size_t packed_bwd_workspace_bytes(int T_q, int T_k, int B, int h_q, int h_kv, int d) {
  const Sizes s = sizes_of(T_q, T_k, B, h_q, h_kv, d);
  return s.key_plan + s.row_plan + s.stats + s.key_part + s.row_part;
}

int launch_attn_packed_bwd(const PackedBwdArgs& a, PFN_encodeTiled enc, void* workspace) {
  return a.d == 64 ? run<64>(a, enc, workspace) : run<128>(a, enc, workspace);
}

int read_packed_bwd_fault_word(int clear, uint32_t* out) {
  uint32_t w = 0;
  if (cudaMemcpyFromSymbol(&w, g_packed_bwd_fault_word, sizeof w) != cudaSuccess) return ATTN_ERR_CUDA;
  if (clear) {
    const uint32_t zero = 0;
    if (cudaMemcpyToSymbol(g_packed_bwd_fault_word, &zero, sizeof zero) != cudaSuccess) return ATTN_ERR_CUDA;
  }
  *out = w;
  return ATTN_OK;
}

}  // namespace attn
