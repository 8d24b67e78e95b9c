// What the attention kernels on the NVFP4 cache share: the problem, the work
// schedule and the partial results of items that several blocks work on.
//
// An item is a tile of query rows of one sequence and kv head; a row is one
// (token, query head) pair, tokens outermost, so that all query heads of a kv
// head read its keys and values once.  An item's work is counted in units of
// keys (pages, or tiles of 128 keys).  All units of all items, in the order
// (sequence, kv head, row tile), are one line that is cut into equal ranges,
// one per block (or group of its warps): every block has the same work whatever the lengths are, and
// at most two items per block are left incomplete, one at each end of its
// range.  Those go to the workspace as (sum, maximum, unnormalised output)
// and are joined, in the order of the blocks, by a second kernel.
#pragma once

#include "kv4.cuh"

namespace moe {
namespace kv4 {

// P is held as p * 2^kShift in fp16, p the weight relative to the running
// maximum.  That maximum is moved only when a row's grows by more than
// 2^kSlack, so O is hardly ever rescaled; P reaches 2^15 at most, its normal
// numbers reach down to 2^(-14 - kShift), and what is lost below is at most
// 2^(-25 - kShift) per key.  The sums and O carry the factor too, so it cancels
// except in the log of the sum.
constexpr int kRowsSmall = 16, kRowsTile = 256;
constexpr float kSlack = 8.0f, kShift = 15.0f - kSlack;
constexpr float kLog2e = 1.4426950408889634f;

// 2^x by the hardware's approximation (2 ulp), 0 for -infinity
DEVINL float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
DEVINL uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
DEVINL uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Four bytes of E2M1 pairs -> four fp16 pairs (low nibble first).
DEVINL void e2m1x8(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
// 16 bytes to shared memory, without a memory clobber: loads of record bytes may
// move past stores to operand tiles.
DEVINL void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d));
}

// A query row's power of two and softmax scale, from its largest magnitude (as
// bf16 bits): |q| * up stays below 2^15, and scores in log2 units are sc times
// the products.  sc > 0: the sign of the scale goes into up, a zero scale
// into a zero row, so that the largest score is that of the largest product.
DEVINL void row_scale(float scale_gk, uint32_t top, float& up, float& sc) {
  const int e = min(14 + 127 - static_cast<int>(top >> 7), 120);
  up = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
  sc = scale_gk * kLog2e * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  if (sc < 0.0f) sc = -sc, up = -up;
  if (sc == 0.0f) sc = 1.0f, up = 0.0f;
}

// What a row's output is multiplied by, and its lse, from the sum and maximum of
// its weights.  A sum of 0 is a row that sees no key; one that is not a number
// (a query or a key is not) makes the row's answer none either.
DEVINL float row_factor(float gv, float l) { return l == 0.0f ? 0.0f : gv / l; }
DEVINL float row_lse(float m, float l) {
  return l == 0.0f ? -INFINITY : (m + log2f(l) - kShift) * (1.0f / kLog2e);
}

struct AttnParams {
  const uint16_t* q;  // bf16 [T][Hq][D], q_stride elements between tokens
  long long q_stride;
  const uint8_t* pool;
  const float *g_k, *g_v;
  const int32_t *q_offsets, *kv_lens, *table;
  uint16_t* out;
  float* lse;  // may be null
  int T, B, Hq, Hkv, G, num_pages, P, max_pages, causal, window;
  float scale;
  // schedule (workspace)
  int* starts;          // [B + 1] q_offsets as used: inside [0, T], never falling
  int* tile_base;       // [B + 1] row tiles before sequence b
  long long* unit_sum;  // [tiles + 1] units of one kv head before row tile f
  int blocks;           // ranges: blocks of the main kernel, or groups of its warps
  int min_units;        // least units of a block's range
  int plan_here;        // every block of the main kernel makes the schedule for itself
  int *part_item;  // [2 * blocks][8]: what a slot holds (PartItem)
  // partial results: slot 2 * block (the item begun by an earlier block) and 2 * block + 1
  float *part_o, *part_ml;  // [2 * blocks][ROWS][D], [2 * blocks][2][ROWS]
  unsigned int* err;
  unsigned long long timeout_ns;
};

struct Seq {
  int q0, n, len;  // first query row, queries, keys
};

// Lengths as the kernels use them: inside q and the table.
DEVINL Seq load_seq(const AttnParams& p, int b) {
  Seq s;
  s.q0 = p.starts[b];
  s.n = p.starts[b + 1] - s.q0;
  const long long cap = static_cast<long long>(p.max_pages) * p.P;
  s.len = static_cast<int>(max(0ll, min(static_cast<long long>(__ldg(p.kv_lens + b)), cap)));
  return s;
}

// Keys [lo, hi) that the query at index i of its sequence sees.
DEVINL void row_keys(const AttnParams& p, const Seq& s, int i, int& lo, int& hi) {
  const int place = s.len - s.n + i;
  hi = p.causal ? min(max(place + 1, 0), s.len) : s.len;
  lo = p.window > 0 ? max(place - p.window + 1, 0) : 0;
}

// Units [u0, u1) of a row tile (u1 > u0: a tile that sees nothing has one
// unit, whose block writes its zeros).
template <int ROWS>
DEVINL void tile_units(const AttnParams& p, const Seq& s, int tile, int unit, int& u0, int& u1) {
  const int first = tile * ROWS / p.G;
  const int last = min(s.n - 1, (tile * ROWS + ROWS - 1) / p.G);
  int lo, hi, x;
  row_keys(p, s, first, lo, x);
  row_keys(p, s, last, x, hi);
  u1 = max(1, (hi + unit - 1) / unit);
  u0 = min(lo / unit, u1 - 1);
}

// Largest i in [0, n) with at(i) <= x (at ascending, at(0) <= x), by a whole warp.
template <class At>
DEVINL int warp_find(int n, long long x, At at) {
  int lo = 0, hi = n;
  const int lane = threadIdx.x & 31;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + lane * step;
    const bool le = i < hi && at(i) <= x;
    const int k = __popc(__ballot_sync(0xFFFFFFFFu, le));
    lo += (k - 1) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// A place on the line of units.
struct Cursor {
  int b, h, tile;  // sequence, kv head, row tile inside the sequence
  Seq s;
  int u, u0, u1;   // unit, and the item's units
};

template <int ROWS>
DEVINL void cursor_item(const AttnParams& p, int unit, Cursor& c) {
  tile_units<ROWS>(p, c.s, c.tile, unit, c.u0, c.u1);
  c.u = c.u0;
}

// The cursor at place x (a whole warp calls it; the same in every lane).
template <int ROWS>
DEVINL Cursor cursor_at(const AttnParams& p, int unit, long long x) {
  Cursor c;
  // largest b whose first unit is at or before x: sequences without queries
  // take no room, so step over tile_base to the sequence that owns the tile
  c.b = warp_find(p.B, x, [&](int i) { return p.unit_sum[p.tile_base[i]] * p.Hkv; });
  const int t0 = p.tile_base[c.b], t1 = p.tile_base[c.b + 1];
  const long long base = p.unit_sum[t0], w = p.unit_sum[t1] - base;
  long long r = x - base * p.Hkv;
  c.h = static_cast<int>(r / w);
  r -= c.h * w;
  c.tile = warp_find(t1 - t0, base + r, [&](int i) { return p.unit_sum[t0 + i]; });
  c.s = load_seq(p, c.b);
  cursor_item<ROWS>(p, unit, c);
  c.u = c.u0 + static_cast<int>(base + r - p.unit_sum[t0 + c.tile]);
  return c;
}

// On to the next item.
template <int ROWS>
DEVINL void cursor_next(const AttnParams& p, int unit, Cursor& c) {
  const int tiles = (c.s.n * p.G + ROWS - 1) / ROWS;
  if (++c.tile == tiles) {
    c.tile = 0;
    if (++c.h == p.Hkv) {
      c.h = 0;
      do {
        ++c.b;
        c.s = load_seq(p, c.b);
      } while (c.s.n == 0 && c.b < p.B - 1);
    }
  }
  cursor_item<ROWS>(p, unit, c);
}

// What the roles of a block need of an item: one warp walks the line of units
// and publishes them, so that the divisions and searches are in the program
// once and the loops over keys stay in the instruction cache.
struct Item {
  int row0;    // first of its rows (token, head of the kv head) in the sequence
  int rows;    // rows that are there
  int q0, nq, len;  // first query row of the sequence, its queries, its keys
  int b, h;
  int u, n;    // first unit here, and how many (0: no more items)
  int slot;    // -1: the whole item is here; else where its partial result goes
};
constexpr int kItems = 8;
struct ItemRing {
  Item item[kItems];
  uint64_t full[kItems], empty[kItems];
};
DEVINL void item_ring_init(ItemRing& r, int readers) {
  for (int i = 0; i < kItems; ++i) {
    mbar_init(&r.full[i], 1);
    mbar_init(&r.empty[i], readers);
  }
}
template <int ROWS>
DEVINL Item make_item(const AttnParams& p, const Cursor& c, int n, int block) {
  Item t;
  t.row0 = c.tile * ROWS;
  t.rows = min(ROWS, c.s.n * p.G - t.row0);
  t.q0 = c.s.q0, t.nq = c.s.n, t.len = c.s.len;
  t.b = c.b, t.h = c.h, t.u = c.u, t.n = n;
  t.slot = c.u == c.u0 ? (n == c.u1 - c.u0 ? -1 : 2 * block + 1) : 2 * block;
  return t;
}
// Keys of row idx of an item's sequence.
DEVINL void item_keys(const AttnParams& p, const Item& t, int idx, int& lo, int& hi) {
  const Seq s{t.q0, t.nq, t.len};
  row_keys(p, s, idx / p.G, lo, hi);
}

// Bounded wait of a whole warp, every lane testing.  A test that fails has
// suspended the warp in hardware for kTestNs, unless the phase completed before
// that (measured: 3.9 to 4.0 us, with a block's other warps idle, busy or
// arriving on the same barrier; a suspend time given with the test changes
// nothing).  So the bound is a number of tests: reading a clock in each of some
// thirty waits makes a third of the program, which has to stay in the
// instruction cache.  LAZY: for warps that nothing waits for soon.
constexpr unsigned long long kTestNs = 4000;
template <bool LAZY = false>
DEVINL void wait_warp(uint64_t* bar, uint32_t parity, uint32_t polls, unsigned int* err, volatile int* abort) {
#pragma unroll 1
  for (uint32_t k = 0; !mbar_try_wait(bar, parity); ++k) {
    if (LAZY) __nanosleep(200);
    if (k >= polls) {
      atomicOr(err, kErrTimeout);
      *abort = 1;
    }
    if (*abort) break;
  }
  __syncwarp();
}
// For what the hardware has in hand when a block ends (copies, products): it
// completes by itself, and has to before shared and tensor memory go to the next
// block, so this is not the limit that callers set, which may be as short as they like.
constexpr unsigned long long kLandNs = 1000000000ull;
// Failing tests after which a wait gives up.
DEVINL uint32_t polls_of(unsigned long long timeout_ns) {
  return static_cast<uint32_t>(min(timeout_ns / kTestNs, 0xFFFFFF00ull));
}
// Whether the block has given up waiting: one answer for the whole warp, which
// reads it after what it waited for.  (Lanes that decided each by itself could
// part, and meet the next vote or warp-wide instruction apart.)
DEVINL bool given_up(volatile int* abort) { return __any_sync(0xFFFFFFFFu, *abort != 0); }
// One reader's (a warp's) place in an ItemRing.
struct ItemReader {
  int i = 0;
  DEVINL Item next(ItemRing& r, uint32_t polls, unsigned int* err, volatile int* abort) {
    const int k = i & (kItems - 1);
    wait_warp(&r.full[k], (i / kItems) & 1, polls, err, abort);
    Item t = r.item[k];
    if (given_up(abort)) t.n = 0;
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&r.empty[k]);
    ++i;
    return t;
  }
};
// The publishing warp's side (the item is the same in every lane).
struct ItemWriter {
  int i = 0;
  DEVINL void put(ItemRing& r, const Item& t, uint32_t polls, unsigned int* err, volatile int* abort) {
    const int k = i & (kItems - 1);
    if (i >= kItems) wait_warp<true>(&r.empty[k], (i / kItems - 1) & 1, polls, err, abort);
    if (given_up(abort)) return;  // some reader may not have read what lies there: all read the same items
    if ((threadIdx.x & 31) == 0) {
      r.item[k] = t;
      mbar_arrive(&r.full[k]);
    }
    __syncwarp();
    ++i;
  }
};

// What a slot of the partial results holds; rows == 0: nothing.  The first
// part of an item (an odd slot) also says which range holds its last part.
struct PartItem {
  int row0, rows, q0, h, last, pad[3];
};
static_assert(sizeof(PartItem) == 32, "eight words");

// One lane's slot of a ring that bulk copies fill.  Each lane feeds its slot at
// its own pace (one thread feeding all slots took about 900 cycles per copy, in
// waits and barrier round trips).  A ring has ONE consumer, a warp or a team
// that waits together: it takes the uses of a slot in order, so that a barrier's
// parity names the use it waits for.  (A consumer that could be ahead of another
// one's use of the same slot would pass on the phase before.)
struct Slot {
  uint8_t* to;             // null: the lane feeds none
  uint64_t *full, *empty;  // count 1; count: arrivals of the consumer
  int index, slots;        // in its ring
  uint32_t uses = 0;
  int at = 0;              // slot of the item's first copy
  // Copies k = 0 .. all-1 of the ring, `bytes` each: from byte offset_of(k) of
  // the record of page page_of(k) of the item's table row (past the item's
  // keys: nothing is copied).  A whole warp calls it.
  template <class PageOf, class OffsetOf>
  DEVINL void feed(const AttnParams& p, const Item& it, int all, int bytes, int rec, PageOf page_of,
                   OffsetOf offset_of, volatile int* abort) {
    const uint8_t* pool = p.pool + static_cast<long long>(it.h) * rec;
    const long long stride = static_cast<long long>(p.Hkv) * rec;
    const int32_t* table = p.table + static_cast<long long>(it.b) * p.max_pages;
    const int last = (it.len + p.P - 1) / p.P;
    int k = to != nullptr ? (index >= at ? index - at : index - at + slots) : all;
    int id = -2;  // page of copy k: -2 not looked up, -1 none
    uint64_t t0 = 0;
    while (__any_sync(0xFFFFFFFFu, k < all)) {
      bool moved = false;
      if (k < all) {
        if (id == -2) {
          const int pg = page_of(k);
          id = -1;
          if (pg < last) {
            id = __ldg(table + pg);
            if (id < 0 || id >= p.num_pages) {
              atomicOr(p.err, kErrBadIndex);
              id = 0;
            }
          }
        }
        // (A consumer that has given up hands its slots back unread, some of them
        // with copies on the way, so the flag is read after the slot came back.
        // The first use finds the phase before the barrier's first complete.  Both
        // reads in flight at once, a vote only where nothing moved: 176 and 950 us
        // on the decode and prefill cases, as without the flag; one after the
        // other 179 and 957, with a vote each time 179 and 976.)
        const bool back = mbar_test_wait(empty, (uses - 1) & 1);
        const int gone = *abort;
        if (back && gone == 0) {
          if (id < 0) {
            mbar_arrive(full);  // no key of this page
          } else {
            mbar_arrive_expect_tx(full, bytes);
            bulk_load(to, pool + id * stride + offset_of(k), bytes, full);
          }
          ++uses;
          k += slots;
          id = -2;
          moved = true;
        }
      }
      if (__any_sync(0xFFFFFFFFu, moved)) {
        t0 = 0;
      } else {
        const uint64_t now = globaltimer_ns();
        if (t0 == 0) t0 = now;
        if (now - t0 > p.timeout_ns) {
          atomicOr(p.err, kErrTimeout);
          *abort = 1;
        }
        if (given_up(abort)) return;
        __nanosleep(100);
      }
    }
    if (to != nullptr) at = (at + all) % slots;
  }
  // Until the lane's last copy has landed: whoever gave up, no block ends with
  // bytes on their way to its shared memory.
  DEVINL void land(const AttnParams& p) {
    if (uses > 0) mbar_wait_bounded(full, (uses - 1) & 1, kLandNs, p.err, nullptr, true);
  }
};

// Walks range `block` and hands its items to `use(item)`, the end mark (n == 0)
// last; writes down what the range's two slots hold, also where `use` gives up
// (false): the join that is queued behind goes by it.  A whole warp calls it.
template <int ROWS, class Use>
DEVINL void walk_range(const AttnParams& p, int unit, int block, long long x0, long long x1, long long range, Use use) {
  PartItem* notes = reinterpret_cast<PartItem*>(p.part_item) + 2 * block;
  const bool writes = (threadIdx.x & 31) == 0;
  bool noted[2] = {false, false};
  if (x0 < x1) {
    Cursor c = cursor_at<ROWS>(p, unit, x0);
    long long x = x0;
    while (true) {
      const int n = static_cast<int>(min(x1 - x, static_cast<long long>(c.u1 - c.u)));
      const Item t = make_item<ROWS>(p, c, n, block);
      if (t.slot >= 0) {
        const int side = t.slot & 1;
        noted[side] = true;
        if (writes) {
          PartItem q;
          q.row0 = t.row0, q.rows = t.rows, q.q0 = t.q0, q.h = t.h;
          q.last = static_cast<int>((x + (c.u1 - c.u) - 1) / range);
          notes[side] = q;
        }
      }
      if (!use(t)) break;  // given up: what was not noted is still marked below, the join reads it
      x += n;
      if (x >= x1) break;
      cursor_next<ROWS>(p, unit, c);
    }
  }
  if (writes) {
    if (!noted[0]) notes[0].rows = 0;
    if (!noted[1]) notes[1].rows = 0;
  }
  Item end{};
  use(end);
}

// The schedule (starts, tile_base, unit_sum) by a warp or a block of 1024
// threads, which shares the 32 words s_warp.
template <int ROWS, int THREADS>
DEVINL void plan(const AttnParams& p, int unit, long long* s_warp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tid = THREADS == 32 ? lane : threadIdx.x;
  auto sync = [] {
    if (THREADS == 32) __syncwarp();
    else __syncthreads();
  };
  auto scan = [&](long long v, long long& total) {
    long long incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += up;
    }
    if (THREADS == 32) {
      __syncwarp();
      total = __shfl_sync(0xFFFFFFFFu, incl, 31);
      return incl - v;
    }
    if (lane == 31) s_warp[warp] = incl;
    sync();
    if (warp == 0) {
      long long w = s_warp[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xFFFFFFFFu, w, o);
        if (lane >= o) w += up;
      }
      s_warp[lane] = w;
    }
    sync();
    const long long before = warp ? s_warp[warp - 1] : 0;
    total = s_warp[31];
    sync();
    return before + incl - v;
  };
  // running maximum of the offsets: whatever they hold, the rows of all
  // sequences are disjoint and inside q, so the tiles fit the workspace
  int before_all = 0;
  for (int base = 0; base <= p.B; base += THREADS) {
    const int b = base + tid;
    int v = b <= p.B ? min(max(p.q_offsets[b], 0), p.T) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xFFFFFFFFu, v, o);
      if (lane >= o) v = max(v, up);
    }
    if (THREADS > 32) {
      if (lane == 31) s_warp[warp] = v;
      sync();
      // lane w: what warp w reached
      int all = static_cast<int>(s_warp[lane]), mine = lane < warp ? all : 0;
      mine = __reduce_max_sync(0xFFFFFFFFu, mine);
      all = __reduce_max_sync(0xFFFFFFFFu, all);
      v = max(max(v, mine), before_all);
      before_all = max(before_all, all);
    } else {
      v = max(v, before_all);
      before_all = __shfl_sync(0xFFFFFFFFu, v, 31);
    }
    if (b <= p.B) p.starts[b] = v;
    sync();
  }
  long long tiles = 0;
  for (int base = 0; base < p.B; base += THREADS) {
    const int b = base + tid;
    long long n = 0, total;
    if (b < p.B) n = (static_cast<long long>(load_seq(p, b).n) * p.G + ROWS - 1) / ROWS;
    const long long at = scan(n, total);
    if (b < p.B) p.tile_base[b] = static_cast<int>(tiles + at);
    tiles += total;
  }
  if (tid == 0) p.tile_base[p.B] = static_cast<int>(tiles);
  sync();
  long long units = 0;
  for (long long base = 0; base < tiles; base += THREADS) {
    const long long f = base + tid;
    long long n = 0, total;
    if (f < tiles) {
      int lo = 0, hi = p.B;  // largest b with tile_base[b] <= f
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.tile_base[mid] <= f) lo = mid;
        else hi = mid;
      }
      const Seq s = load_seq(p, lo);
      int u0, u1;
      tile_units<ROWS>(p, s, static_cast<int>(f - p.tile_base[lo]), unit, u0, u1);
      n = u1 - u0;
    }
    const long long at = scan(n, total);
    if (f < tiles) p.unit_sum[f] = units + at;
    units += total;
  }
  if (tid == 0) p.unit_sum[tiles] = units;
}

DEVINL long long total_units(const AttnParams& p) { return p.unit_sum[p.tile_base[p.B]] * p.Hkv; }
DEVINL long long range_of(const AttnParams& p, long long total) {
  const long long r = (total + p.blocks - 1) / p.blocks;
  return r < p.min_units ? p.min_units : r;
}

// Main kernel over 256-row tiles and 128-key units (kv4_prefill.cu).
int attention_tiles(const AttnParams& p, int D, cudaStream_t s);
// Main kernel over 16-row tiles and 128-key units, heads of 128 (kv4_decode.cu);
// a warp of each block makes the schedule for up to kPlanHere sequences and tiles.
constexpr int kPlanHere = 31;
int attention_decode(const AttnParams& p, cudaStream_t s);

}  // namespace kv4
}  // namespace moe
