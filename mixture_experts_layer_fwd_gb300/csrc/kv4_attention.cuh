// What the attention kernels on the NVFP4 cache share: the problem, the work
// schedule and the partial results of items that several blocks work on.
//
// An item is a tile of query rows of one sequence and kv head; a row is one
// (token, query head) pair, tokens outermost, so that all query heads of a kv
// head read its keys and values once.  An item's work is counted in units of
// keys (pages, or tiles of 128 keys).  All units of all items, in the order
// (sequence, kv head, row tile), are one line that is cut into equal ranges,
// one per block: every block has the same work whatever the lengths are, and
// at most two items per block are left incomplete, one at each end of its
// range.  Those go to the workspace as (sum, maximum, unnormalised output)
// and are joined, in the order of the blocks, by a second kernel.
#pragma once

#include "kv4.cuh"

namespace moe {
namespace kv4 {

// P is held as p * 2^shift in fp16, p the weight relative to the running
// maximum: normal numbers reach down to 2^(-14-shift), and what is lost below
// is at most 2^(-25-shift) per key.  The largest value is 2^15: the 16-row
// kernel's maximum is exact, the 256-row kernel's lags by up to 2^8.  The sums
// and O carry the factor too, so it cancels except in the log of the sum.
constexpr int kRowsSmall = 16, kRowsTile = 256;
constexpr float kSlack = 8.0f;
__host__ __device__ constexpr float p_shift(int rows) { return rows == kRowsSmall ? 15.0f : 15.0f - kSlack; }

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
  int blocks;           // blocks of the main kernel
  int min_units;        // least units of a block's range
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

// Largest i in [0, n) with a[i] <= x (a ascending, a[0] <= x), by a whole warp.
template <class T>
DEVINL int warp_find(const T* a, int n, long long x, long long factor) {
  int lo = 0, hi = n;
  const int lane = threadIdx.x & 31;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + lane * step;
    const bool le = i < hi && a[i] * factor <= x;
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
  int lo = 0, hi = p.B;
  const int lane = threadIdx.x & 31;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + lane * step;
    const bool le = i < hi && p.unit_sum[p.tile_base[i]] * p.Hkv <= x;
    const int k = __popc(__ballot_sync(0xFFFFFFFFu, le));
    lo += (k - 1) * step;
    hi = min(hi, lo + step);
  }
  c.b = lo;
  const int t0 = p.tile_base[lo], t1 = p.tile_base[lo + 1];
  const long long base = p.unit_sum[t0], w = p.unit_sum[t1] - base;
  long long r = x - base * p.Hkv;
  c.h = static_cast<int>(r / w);
  r -= c.h * w;
  c.tile = warp_find(p.unit_sum + t0, t1 - t0, base + r, 1);
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

DEVINL long long total_units(const AttnParams& p) { return p.unit_sum[p.tile_base[p.B]] * p.Hkv; }
DEVINL long long range_of(const AttnParams& p, long long total) {
  const long long r = (total + p.blocks - 1) / p.blocks;
  return r < p.min_units ? p.min_units : r;
}

// Main kernel over 256-row tiles and 128-key units (kv4_prefill.cu).
int attention_tiles(const AttnParams& p, int D, cudaStream_t s);

}  // namespace kv4
}  // namespace moe
