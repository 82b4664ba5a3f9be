// attn_plan.cuh -- the work list of attention over ragged batches.
//
// The lengths of packed sequences live in device memory, so the host cannot say which CTA
// does what. One CTA writes the list: an item is a block of own rows of one sequence (query
// tokens, or keys), a unit is an item for one key/value head, and a unit's cost is the number
// of tiles that it streams. Two ways to hand the units out:
//   whole    heaviest first, to the CTA that asks next; no unit is cut. Taken when there are many
//            units for every CTA. (Who computes a unit does not change its result.)
//   cut      the units' tiles one after the other, in equal shares of consecutive tiles, so a
//            CTA's first and last units may be pieces, whose partial results a second kernel
//            joins. Taken when one unit is far longer than a CTA's even share, or few are long.
// Everything about a unit is in its entry, so a CTA needs one load to know its work. Where a call cannot have more
// units than CTAs, nor any that would be cut, there is no list: each CTA finds its one unit itself.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

namespace attn {
namespace plan {

constexpr int TILE = 128;      // streamed keys per tile, own rows per tile
constexpr int THREADS = 1024;  // of the planning CTA
constexpr int SMEM_LENS = 512;  // sequences whose offsets are kept from the first reading
constexpr int SMEM_SEQS = 2047, SMEM_ITEMS = 2048;  // with more, these lists are in the workspace
constexpr int BINS = 640;
constexpr int FEW = 4, LONG_SHARE = 128;  // units per CTA, tiles: see where `cut` is decided

struct Entry {        // 64 bytes
  int own_row;        // first own row (token or key) in the packed array
  int own_n;          // own tokens or keys of the block
  int str_row;        // first row of the sequence's streamed side (paged: the sequence)
  int str_len;        // its rows (keys; or query tokens where keys are the own rows)
  int pos;            // queries own: position of the first own token; keys own: index of the first own key
  int off;            // keys minus queries of the sequence: position of its first query
  int n_first, skip;  // list entry j is tile j, from n_first on tile j + skip
  int j0, n;          // this unit's list entries [j0, j0 + n)
  int lo0, hi0;       // of these, those that own tile 0 needs, counted from j0
  int lo1, hi1;       // and own tile 1
  int slot;           // place of the partial result, or -1: the unit is whole
  int hk;             // key/value head
};
static_assert(sizeof(Entry) == 64, "read as four 16-byte words");

struct Join {  // 32 bytes: a unit that was cut
  int own_row, own_n, hk;
  int slot;      // of the first piece
  int next;      // of the second; the further ones two apart
  int pieces;
  int pad[2];
};

struct Header {
  int cut;      // 1: CTA a takes entries [range[a].x, range[a].y); 0: the next of n_units, as CTAs ask
  int n_units;  // whole: unit u is the list's entry u / h_kv, head u % h_kv
  int n_join;
  int next;     // units handed out so far, when they are whole
};

struct Args {
  const int32_t* q_starts;
  const int32_t* k_starts;    // null: as the queries'
  const int32_t* cache_lens;  // paged: keys per sequence (then k_starts is null)
  int B, T_q, T_k, max_keys;  // max_keys: paged, the page table's reach
  int own_keys;               // 1: own rows are keys (tiles of TILE), streamed rows query tokens
  int own_tiles;              // own tiles per unit: 1, or 2 (queries own)
  int tok;                    // query tokens per tile of rows
  int h_kv, causal, window, sinks;  // window -1: none
  int ctas;                   // CTAs of the kernel that works the list off
  int min_share;              // least tiles of a CTA's share when units are cut
  int may_cut;
  long long items;  // places for items; offsets that do not decrease have no more
  Header* head;
  int2* range;   // [ctas]
  Join* joins;   // [ctas]
  int* first;    // [B + 1]: items before each sequence
  long long* at;  // [items]: cost before each item
  int* rank;     // [items]: place among the items of like cost
  Entry* list;   // [items * h_kv + ctas]
};

// Bytes of the plan part of a workspace; items: an upper bound.
inline size_t bytes(long long items, int h_kv, int B, int ctas) {
  const size_t lists = ((size_t)items * h_kv + ctas) * sizeof(Entry) + (size_t)ctas * (sizeof(Join) + sizeof(int2));
  const size_t scratch = (size_t)items * (sizeof(long long) + sizeof(int)) + ((size_t)B + 1) * sizeof(int);
  return (sizeof(Header) + lists + scratch + 255) & ~size_t(255);
}

inline void place(Args& a, void* base, long long items) {
  uint8_t* p = static_cast<uint8_t*>(base);
  a.items = items;
  a.head = reinterpret_cast<Header*>(p);
  p += sizeof(Header);
  a.list = reinterpret_cast<Entry*>(p);
  p += ((size_t)items * a.h_kv + a.ctas) * sizeof(Entry);
  a.joins = reinterpret_cast<Join*>(p);
  p += (size_t)a.ctas * sizeof(Join);
  a.range = reinterpret_cast<int2*>(p);
  p += (size_t)a.ctas * sizeof(int2);
  a.at = reinterpret_cast<long long*>(p);
  p += (size_t)items * sizeof(long long);
  a.rank = reinterpret_cast<int*>(p);
  p += (size_t)items * sizeof(int);
  a.first = reinterpret_cast<int*>(p);
}

struct Seq {
  int q0, n_q, k0, n_k;  // n_k: keys
};

// Offsets that decrease or leave the array give empty or shortened sequences, never rows outside it.
__device__ __forceinline__ Seq sequence(const Args& a, int b) {
  Seq s;
  s.q0 = min(max(a.q_starts[b], 0), a.T_q);
  s.n_q = max(min(a.q_starts[b + 1], a.T_q) - s.q0, 0);
  if (a.cache_lens) {
    s.k0 = b;
    s.n_k = min(max(a.cache_lens[b], 0), a.max_keys);
  } else if (a.k_starts) {
    s.k0 = min(max(a.k_starts[b], 0), a.T_k);
    s.n_k = max(min(a.k_starts[b + 1], a.T_k) - s.k0, 0);
  } else {
    s.k0 = min(s.q0, a.T_k);
    s.n_k = min(s.n_q, a.T_k - s.k0);
  }
  return s;
}

__device__ __forceinline__ int blocks_of(const Args& a, const Seq& s) {
  const int rows = a.own_keys ? s.n_k : s.n_q, per = a.own_keys ? TILE : a.tok * a.own_tiles;
  return rows / per + (rows % per != 0);
}

// Keys [lo, hi) that some query at positions [p0, p1] may use, in tiles, and the tiles of the first
// keys before them; empty: hi <= lo.
__device__ __forceinline__ void key_tiles(const Args& a, int n_k, int p0, int p1, int& first, int& lo, int& hi) {
  int top = n_k, bottom = 0;
  if (a.causal) top = min(top, p1 + 1);
  if (a.window >= 0) {
    if (!a.causal) top = min(top, p1 + a.window + 1);
    bottom = max(0, p0 - a.window);
  }
  first = lo = hi = 0;
  if (top <= 0) return;
  bottom = min(bottom, top);
  lo = bottom / TILE;
  hi = (top + TILE - 1) / TILE;
  if (a.window >= 0) first = min((min(a.sinks, top) + TILE - 1) / TILE, lo);
}

// Block `own` of a sequence: everything but the head, the piece and its slot.
__device__ __forceinline__ Entry item(const Args& a, const Seq& s, int own) {
  Entry e;
  e.off = s.n_k - s.n_q;
  e.j0 = 0;
  e.slot = -1;
  e.hk = 0;
  e.lo1 = e.hi1 = 0;
  if (a.own_keys) {
    const int key = own * TILE, n = min(TILE, s.n_k - key);
    e.own_row = s.k0 + key;
    e.own_n = n;
    e.str_row = s.q0;
    e.str_len = s.n_q;
    e.pos = key;
    // query tokens [t0, t1) that may use one of the keys
    int t0 = a.causal ? key - e.off : 0, t1 = s.n_q;
    if (a.window >= 0) {
      if (!a.causal) t0 = key - a.window - e.off;
      t1 = min(t1, key + n + a.window - e.off);
    }
    t0 = max(t0, 0);
    const bool none = t1 <= t0;
    e.n_first = 0;
    e.skip = none ? 0 : t0 / a.tok;
    e.n = none ? 0 : (t1 + a.tok - 1) / a.tok - e.skip;
    e.lo0 = 0;
    e.hi0 = e.n;
    return e;
  }
  const int t0 = own * a.tok * a.own_tiles, n = min(a.tok * a.own_tiles, s.n_q - t0);
  e.own_row = s.q0 + t0;
  e.own_n = n;
  e.str_row = s.k0;
  e.str_len = s.n_k;
  e.pos = e.off + t0;
  int first, lo, hi;
  key_tiles(a, s.n_k, e.pos, e.pos + n - 1, first, lo, hi);
  e.n_first = first;
  e.skip = lo - first;
  e.n = first + hi - lo;
  e.lo0 = 0;
  e.hi0 = e.n;
  if (a.own_tiles == 2) {
    // each tile of rows: its own end of the list, and without first keys its own start
    const int n0 = min(n, a.tok);
    int f, l, h;
    key_tiles(a, s.n_k, e.pos, e.pos + n0 - 1, f, l, h);
    e.hi0 = h > l || f > 0 ? e.n - (hi - h) : 0;
    if (n > a.tok) {
      key_tiles(a, s.n_k, e.pos + a.tok, e.pos + n - 1, f, l, h);
      e.lo1 = f > 0 || first > 0 ? 0 : l - lo;
      e.hi1 = e.n;
    }
  }
  return e;
}

__device__ __forceinline__ void put(Entry* to, const Entry& e) {
  int4* d = reinterpret_cast<int4*>(to);
  d[0] = make_int4(e.own_row, e.own_n, e.str_row, e.str_len);
  d[1] = make_int4(e.pos, e.off, e.n_first, e.skip);
  d[2] = make_int4(e.j0, e.n, e.lo0, e.hi0);
  d[3] = make_int4(e.lo1, e.hi1, e.slot, e.hk);
}

// Sum of v over the threads before this one, and over all of them.
__device__ __forceinline__ long long scan(long long v, long long* warps, long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // `warps` may still be read from the call before
  if (lane == 31) warps[warp] = x;
  __syncthreads();
  long long w = lane < THREADS / 32 ? warps[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const long long before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  return x - v + (warp ? before : 0);
}

struct Scratch {  // shared memory
  long long warps[THREADS / 32];
  int first[SMEM_SEQS + 1];
  Seq seq[SMEM_LENS];
  long long at[SMEM_ITEMS];  // cost of the items before each
  int rank[SMEM_ITEMS];      // its place among the items of its bin
  int bin[BINS];
  int max, joins;
};

// Bins of the counting sort, heaviest first: exact costs below 256, sixteen bins per doubling above.
__device__ __forceinline__ int bin_of(int n) {
  if (n < 256) return BINS - 1 - n;
  const int e = 31 - __clz(n);  // 8 ..
  return max(BINS - 256 - ((e - 8) * 16 + ((n >> (e - 4)) & 15)) - 1, 0);
}

// Units [w0, w0 + cost) of the cut list; I: a type that holds the whole work.
template <typename I>
__device__ __forceinline__ void cut_unit(const Args& a, Scratch& sh, Entry e, int u, I w0, I cost, I share, I work) {
  const I w1 = w0 + cost;
  const int c0 = (int)(w0 / share), c1 = (int)((w1 - 1) / share);
  const int n = e.n, lo0 = e.lo0, hi0 = e.hi0, lo1 = e.lo1, hi1 = e.hi1;
  for (int c = c0; c <= c1; ++c) {
    // entry u + c: units and CTAs both only go up along the tiles, so it is this piece's alone
    const I r0 = (I)c * share, r1 = r0 + share;
    const int j0 = (int)((r0 > w0 ? r0 : w0) - w0), j1 = (int)((r1 < w1 ? r1 : w1) - w0);
    e.j0 = j0;
    e.n = n == 0 ? 0 : j1 - j0;
    auto clip = [&](int x) { return min(max(x - j0, 0), e.n); };
    e.lo0 = clip(lo0);
    e.hi0 = clip(hi0);
    e.lo1 = clip(lo1);
    e.hi1 = clip(hi1);
    e.slot = c0 == c1 ? -1 : (r0 >= w0 ? 2 * c : 2 * c + 1);
    put(a.list + u + c, e);
    if (r0 >= w0) a.range[c].x = u + c;                    // the CTA's share starts here
    if (r1 <= w1 || w1 == work) a.range[c].y = u + c + 1;  // and ends here
  }
  if (c0 == c1) return;
  Join& j = a.joins[atomicAdd(&sh.joins, 1)];
  j.own_row = e.own_row;
  j.own_n = e.own_n;
  j.hk = e.hk;
  j.slot = (I)c0 * share >= w0 ? 2 * c0 : 2 * c0 + 1;
  j.next = 2 * (c0 + 1);
  j.pieces = c1 - c0 + 1;
}

// Writes the list: one CTA of THREADS threads. A thread takes an item to count, a unit to write.
__device__ __forceinline__ void write(const Args& a, Scratch& sh) {
  const int t = threadIdx.x;
  if (t == 0) {
    sh.max = 0;
    sh.joins = 0;
  }
  for (int x = t; x < BINS; x += THREADS) sh.bin[x] = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // items before each sequence
  int* first = a.B <= SMEM_SEQS ? sh.first : a.first;
  long long items = 0;
  for (int b0 = 0; b0 < a.B; b0 += THREADS) {
    const int b = b0 + t;
    int mine = 0;
    if (b < a.B) {
      const Seq s = sequence(a, b);
      if (b < SMEM_LENS) sh.seq[b] = s;
      mine = blocks_of(a, s);
    }
    long long total;
    const long long at = scan(mine, sh.warps, total);
    if (b < a.B) first[b] = (int)min(items + at, 0x7fffffffLL);
    items += total;
  }
  __syncthreads();
  // offsets that decrease may name rows again and again: what has no place in the list is left out
  const int N = (int)min(items, a.items);
  long long* at = N <= SMEM_ITEMS ? sh.at : a.at;
  int* rank = N <= SMEM_ITEMS ? sh.rank : a.rank;
  auto find = [&](int i) -> Entry {  // item i: the last sequence that starts at or before it and has items
    int lo = 0, hi = a.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (first[mid] <= i) lo = mid;
      else hi = mid - 1;
    }
    return item(a, lo < SMEM_LENS ? sh.seq[lo] : sequence(a, lo), i - first[lo]);
  };
  // costs: the sum before every item, the largest, and how many there are of each
  long long sum = 0;
  Entry mine;  // item t
  for (int i0 = 0; i0 < N; i0 += THREADS) {
    const int i = i0 + t;
    int cost = 0;
    if (i < N) {
      const Entry e = find(i);
      if (i0 == 0) mine = e;
      cost = max(e.n, 1);
      rank[i] = atomicAdd(&sh.bin[bin_of(cost)], 1);
    }
    long long total;
    const long long before = scan(cost, sh.warps, total);
    if (i < N) at[i] = sum + before;
    sum += total;
    const int top = __reduce_max_sync(0xffffffffu, cost);
    if ((t & 31) == 0 && top > 0) atomicMax(&sh.max, top);
  }
  __syncthreads();
  const int top = sh.max;
  const long long units = (long long)N * a.h_kv, work = sum * a.h_kv;
  const long long share = max((work + a.ctas - 1) / a.ctas, (long long)a.min_share);
  // cut: one is far longer than an even share, or a few long ones would leave CTAs without work at the end. A piece
  // costs its CTA some ten tiles' time (its sums go through memory), so unevenness is often the better choice:
  // cut against whole, forward, 4096 positions, 16 heads of 128, causal (shares of 28 tiles) 111.5 and 72.7 us, 4 x 1024
  // unmasked (14) 62.5 and 42.3, but 8192 unmasked (216) 357.5 and 383, 509 tokens over 60510 keys of 8 bits (398; 128
  // units for 152 CTAs) 782 and 877; gradients, 4096 causal (56) 382 and 260, but 8192 causal, 32/8 heads (438), with
  // the pass that owns keys cut (512 units) 1632 and 1697.
  const bool cut = a.may_cut && (top > share + share / 2 || (share >= LONG_SHARE && units <= (long long)FEW * a.ctas));
  if (t == 0) {
    a.head->cut = cut;
    a.head->n_units = (int)units;
    a.head->next = a.ctas;
  }
  if (cut) {
    for (int i = t; i < a.ctas; i += THREADS) a.range[i] = make_int2(0, 0);
  } else {
    // places of the bins: a scan over BINS = THREADS counts
    long long all;
    const int count = t < BINS ? sh.bin[t] : 0;
    const long long before = scan(count, sh.warps, all);
    if (t < BINS) sh.bin[t] = (int)before;
  }
  __syncthreads();
  if (!cut) {
    for (int i = t; i < N; i += THREADS) {
      const Entry e = i == t ? mine : find(i);
      put(a.list + sh.bin[bin_of(max(e.n, 1))] + rank[i], e);
    }
    if (t == 0) a.head->n_join = 0;
    return;
  }
  const bool narrow = work < (1LL << 30);
  for (long long u0 = 0; u0 < units; u0 += THREADS) {
    const long long u = u0 + t;
    if (u >= units) break;
    // by head, then by item: a thread's first unit is the item that it has counted
    const int hk = (int)((unsigned)u / (unsigned)N), i = (int)((unsigned)u - (unsigned)hk * (unsigned)N);
    Entry e = u == t && t < N ? mine : find(i);
    const int cost = max(e.n, 1);
    e.hk = hk;
    const long long w0 = at[i] * a.h_kv + (long long)hk * cost;
    if (narrow) cut_unit<unsigned>(a, sh, e, i * a.h_kv + hk, (unsigned)w0, (unsigned)cost, (unsigned)share, (unsigned)work);
    else cut_unit<long long>(a, sh, e, i * a.h_kv + hk, w0, cost, share, work);
  }
  __syncthreads();
  if (t == 0) a.head->n_join = sh.joins;
}

static __global__ void __launch_bounds__(THREADS, 1) attn_plan_kernel(const Args a) {
  __shared__ Scratch scratch;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  write(a, scratch);
}

// Word `lane` (< 16) of unit u's entry, found without a list by a warp of its own; all are -1 for no unit.
__device__ __forceinline__ int word_without_list(const Args& a, int u) {
  const int lane = threadIdx.x & 31, i = u / a.h_kv;
  int before = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    Seq s = {};
    int n = 0;
    if (b0 + lane < a.B) {
      s = sequence(a, b0 + lane);
      n = blocks_of(a, s);
    }
    int upto = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    const int own = i - (before + upto - n);
    const uint32_t has = __ballot_sync(0xffffffffu, own >= 0 && own < n);
    if (has) {
      const Entry e = item(a, s, own);  // in one lane
      const int w[16] = {e.own_row, e.own_n, e.str_row, e.str_len, e.pos, e.off, e.n_first, e.skip,
                         e.j0,      e.n,     e.lo0,     e.hi0,     e.lo1, e.hi1, e.slot,    u - i * a.h_kv};
      int word = -1;
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        const int v = __shfl_sync(0xffffffffu, w[x], __ffs(has) - 1);
        if (lane == x) word = v;
      }
      return word;
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
  return -1;
}

// The copy warp's way through the list: the number of its CTA's next unit, or -1. Lane 0 asks.
struct Turn {
  int at, end;  // cut: the rest of this CTA's range
  bool cut;
  int h_kv;
  __device__ __forceinline__ Turn(const Header& h, const int2* range, int h_kv_) : cut(h.cut != 0), h_kv(h_kv_) {
    at = cut ? range[blockIdx.x].x : (int)blockIdx.x;
    end = cut ? range[blockIdx.x].y : h.n_units;
  }
  __device__ __forceinline__ int next(Header* head) {  // one past: the unit after the one returned is asked for
    const int u = at < end ? at : -1;
    if (cut) {
      ++at;
    } else if (u >= 0) {
      at = atomicAdd(&head->next, 1);
    }
    return u;
  }
  // Word x of unit u's entry, x < 16; all are -1 for no unit.
  __device__ __forceinline__ int word(const Entry* list, int u, int x) const {
    if (u < 0) return -1;
    const int i = cut ? u : u / h_kv;
    if (!cut && x == 15) return u - i * h_kv;
    return reinterpret_cast<const int*>(list + i)[x];
  }
};

}  // namespace plan
}  // namespace attn
