// Eviction from the paged NVFP4 cache by accumulated attention weight: rows longer
// than `limit` keep `keep` tokens, the first `sinks`, the last `recent` and, of
// those between, the ones with the largest sums, the first of equal ones; in every
// layer and kv head for itself, in the order of the tokens.
//
// Bound: the bytes of the tokens that stay, read and written once (D * 9/8 each and
// kv head), and the sums, read once.  Three launches: a one-block plan (which rows,
// a free page in place of each page that another row maps too; of up to eight rows and
// 8192 pages every block of the next launch makes it for its row, a launch less); a block per (layer,
// row, kv head) that finds the keep-th largest sum by three passes of a radix
// select and lists the tokens that stay; a block per (layer, row, kv head, keys or
// values) that moves them.  Tokens only move towards the front, so that block moves
// them in place, 256 at a time: what one step writes, no later step reads.
//
// 32 conversations of 4096 tokens, 1500 of which stay, 32 layers, 4 heads of 128: 5 + 56 +
// 262 us with nothing in L2 (the move at 5.1 TB/s of both ways, 0.8 of DRAM's cycles), 261 to
// 304 us with the call after itself, by the GPU.  One conversation of 1300 tokens, 4 layers:
// 9 + 10 us, the call 27 (33 with a plan in front).
#include "kv4.cuh"

namespace moe {
namespace kv4 {
namespace {

constexpr int kPlan = 1024;
constexpr int kPer = 4;           // refs per thread and scan step of the plan
constexpr int kThreads = 256;
// Of a radix pass: 12, 10 and 10 bits.  The first has the sign, the exponent and three bits
// behind it: sums lie in few binades, and lanes that count in one bin wait for each other
// (11, 11 and 10 bits: 59 against 56 us).
constexpr int kBins = 4096, kLowBins = 1024;
constexpr int kCached = 16384;    // tokens whose sums are held in shared memory
constexpr int kTile = 256;        // tokens moved at a time
constexpr long long kListBytes = 256ll << 20;  // of the workspace, for lists of a group of layers: bounds it, two launches more

struct Params {
  const int32_t *table_in, *lens_in, *refs_in;
  int32_t *table, *lens, *refs, *dropped;
  uint8_t* pool;
  long long layer_stride;
  float* score;
  int S, M, N, P, D, Hkv, layers, cap, keep, limit, sinks, recent;
  // workspace
  int* fresh;      // [N] free pages, lowest first
  int* count;      // [1] how many of those that are wanted there are
  int* row_rank;   // [S] first of the row's fresh pages; -1: the row stays as it is
  int* row_more;   // [S] how many it takes
  int* row_len;    // [S] its tokens before
  int *src, *dst;  // [S][M] its pages before, and after
  int* list;       // [group of layers][S][Hkv][keep] tokens that stay
  unsigned int* err;
};

DEVINL bool page_ok(int p, int N) { return p >= 0 && p < N; }
// Page j of a row gets a copy of its own: another row maps it too, and not all of it stays where it is.
DEVINL bool shared(const Params& p, int page, int j) { return j >= p.sinks / p.P && page_ok(page, p.N) && p.refs_in[page] > 1; }

template <int THREADS>
DEVINL int block_scan(int v, int* s_warp, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  int w = lane < THREADS / 32 ? s_warp[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xFFFFFFFFu, w, o);
    if (lane >= o) w += up;
  }
  total = __shfl_sync(0xFFFFFFFFu, w, 31);
  const int before = __shfl_sync(0xFFFFFFFFu, w, max(warp - 1, 0));
  __syncthreads();
  return (warp ? before : 0) + incl - v;
}

// -------------------------------------------------------------------- plan
// in -> out where they are different arrays, by `step` threads.
DEVINL void carry(const Params& p, long long id, long long step) {
  if (p.table != p.table_in)
    for (long long i = id; i < static_cast<long long>(p.S) * p.M; i += step) p.table[i] = p.table_in[i];
  if (p.lens != p.lens_in)
    for (long long i = id; i < p.S; i += step) p.lens[i] = p.lens_in[i];
  if (p.refs != p.refs_in)
    for (long long i = id; i < p.N; i += step) p.refs[i] = p.refs_in[i];
}
DEVINL int len_of(const Params& p, int r) {
  return static_cast<int>(max(0ll, min(static_cast<long long>(p.lens_in[r]), static_cast<long long>(p.M) * p.P)));
}
// Pages that a row needs in place of shared ones (by a warp).
DEVINL int more_of(const Params& p, int r, int len) {
  const int lane = threadIdx.x & 31, used = (p.keep + p.P - 1) / p.P;
  int n = 0;
  if (len > p.limit)
    for (int j0 = 0; j0 < used; j0 += 32) {
      const int j = j0 + lane;
      n += __popc(__ballot_sync(0xFFFFFFFFu, j < used && shared(p, p.table_in[static_cast<long long>(r) * p.M + j], j)));
    }
  return n;
}
struct RowPlan {  // of Params' row_len, row_more, row_rank, count
  int len, more, rank, count;
};
// The row is short enough, or has not found its pages.
DEVINL bool stays(const RowPlan& x) { return x.rank < 0 || (x.more > 0 && x.rank + x.more > x.count); }

__global__ void __launch_bounds__(kPlan) evict_plan_kernel(const Params p) {
  __shared__ int s_warp[32];
  launch_dependents();
  if (blockIdx.x > 0)
    return carry(p, static_cast<long long>(blockIdx.x - 1) * kPlan + threadIdx.x, static_cast<long long>(gridDim.x - 1) * kPlan);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // a warp counts a row's shared pages
  for (int r = warp; r < p.S; r += kPlan / 32) {
    const int len = len_of(p, r), n = more_of(p, r, len);
    if (lane == 0) p.row_len[r] = len, p.row_more[r] = n;
  }
  __syncthreads();
  int need = 0;
  for (int base = 0; base < p.S; base += kPlan) {
    const int r = base + threadIdx.x;
    const int more = r < p.S ? p.row_more[r] : 0;
    int total;
    const int rank = block_scan<kPlan>(more, s_warp, total);
    if (r < p.S) p.row_rank[r] = p.row_len[r] > p.limit ? need + rank : -1;
    need += total;
  }
  need = min(need, p.N);
  int found = 0;
  for (int base = 0; base < p.N && found < need; base += kPlan * kPer) {
    const int p0 = base + threadIdx.x * kPer;
    int n = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) n += p0 + i < p.N && p.refs_in[p0 + i] <= 0;
    int total;
    int k = found + block_scan<kPlan>(n, s_warp, total);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (p0 + i < p.N && p.refs_in[p0 + i] <= 0 && k < need) p.fresh[k++] = p0 + i;
    found = min(need, found + total);
  }
  if (threadIdx.x == 0) p.count[0] = found;
}

// The same of a few rows and pages, by each block of the next kernel for its row; the block
// that writes the row's pages down (`pages`) also finds the free ones that it takes.
constexpr int kSmallRows = kThreads / 32, kSmallPages = 8192;
DEVINL RowPlan plan_small(const Params& p, int r, bool pages, int* s_warp) {
  __shared__ int s_len[kSmallRows], s_n[kSmallRows];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (warp < p.S) {
    const int len = len_of(p, warp), n = more_of(p, warp, len);
    if (lane == 0) s_len[warp] = len, s_n[warp] = n;
  }
  __syncthreads();
  int need = 0, before = 0;
  for (int k = 0; k < p.S; ++k) {
    if (k == r) before = need;
    need += s_n[k];
  }
  RowPlan x{s_len[r], s_n[r], -1, 0};
  if (x.len > p.limit) x.rank = before;
  need = min(need, p.N);
  for (int base = 0; base < p.N && x.count < need; base += kThreads) {
    const int page = base + threadIdx.x;
    const bool is_free = page < p.N && p.refs_in[page] <= 0;
    int total;
    const int k = x.count + block_scan<kThreads>(is_free, s_warp, total);
    if (pages && is_free && k >= before && k < before + x.more) p.fresh[k] = page;
    x.count = min(need, x.count + total);
  }
  __syncthreads();  // the pages have been written
  return x;
}
DEVINL RowPlan plan_of(const Params& p, int r) { return {p.row_len[r], p.row_more[r], p.row_rank[r], p.count[0]}; }

// ------------------------------------------------------------------ select
// Larger sums have larger keys; -0 is 0, and what is not a number comes before any.
DEVINL uint32_t key_of(float v) {
  if (v != v) return 0xFFFFFFFFu;
  const uint32_t b = __float_as_uint(v + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Block x: (layer of the group, row, kv head); then S blocks: a row's pages; in the small
// form, without a plan in front, then those that carry over.
__global__ void __launch_bounds__(kThreads) evict_select_kernel(const Params p, int layer0, int layers, bool small) {
  extern __shared__ uint32_t s_key[];
  __shared__ __align__(16) int s_hist[kBins];
  __shared__ int s_warp[32], s_more[2][kThreads / 32];
  __shared__ int s_bin, s_want;
  wait_for_previous();
  launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int heads = layers * p.S * p.Hkv;
  if (static_cast<int>(blockIdx.x) >= heads + p.S) {
    const int first = heads + p.S;
    return carry(p, static_cast<long long>(blockIdx.x - first) * kThreads + threadIdx.x,
                 static_cast<long long>(gridDim.x - first) * kThreads);
  }
  if (static_cast<int>(blockIdx.x) >= heads) {
    const int r = blockIdx.x - heads;
    const RowPlan x = small ? plan_small(p, r, true, s_warp) : plan_of(p, r);
    if (small && threadIdx.x == 0) {
      p.row_len[r] = x.len, p.row_more[r] = x.more, p.row_rank[r] = x.rank;
      if (r == 0) p.count[0] = x.count;
    }
    if (stays(x)) return;
    const int used = (p.keep + p.P - 1) / p.P;
    const long long at = static_cast<long long>(r) * p.M;
    if (warp != 0) return;
    for (int j0 = 0, k = x.rank; j0 < p.M; j0 += 32) {
      const int j = j0 + lane, page = j < p.M ? p.table_in[at + j] : -1;
      const bool own = j < used && shared(p, page, j);
      const uint32_t all = __ballot_sync(0xFFFFFFFFu, own);
      if (j < p.M) {
        p.src[at + j] = page;
        p.dst[at + j] = j >= used ? -1 : own ? p.fresh[k + __popc(all & ((1u << lane) - 1))] : page;
      }
      k += __popc(all);
    }
    return;
  }
  const int h = blockIdx.x % p.Hkv, r = blockIdx.x / p.Hkv % p.S, l = blockIdx.x / p.Hkv / p.S;
  const RowPlan x = small ? plan_small(p, r, false, s_warp) : plan_of(p, r);
  if (stays(x)) return;
  const int len = x.len, first = p.sinks, last = len - p.recent;  // the middle
  const float* score = p.score + ((static_cast<long long>(layer0 + l) * p.S + r) * p.Hkv + h) * p.cap;
  int* list = p.list + ((static_cast<long long>(l) * p.S + r) * p.Hkv + h) * p.keep;
  const int mid = last - first;
  const bool cached = mid <= kCached;
  int want = p.keep - p.sinks - p.recent;  // of the middle; fewer than it has
  // the ends stay as a whole
  for (int i = threadIdx.x; i < p.sinks; i += kThreads) list[i] = i;
  for (int i = threadIdx.x; i < p.recent; i += kThreads) list[p.keep - p.recent + i] = last + i;
  if (want == 0) return;
  // keys of the middle four at a time, behind the last one 0, which is below every key
  auto load4 = [&](int i) {
    uint4 k;
    k.x = i < mid ? key_of(__ldg(score + first + i)) : 0;
    k.y = i + 1 < mid ? key_of(__ldg(score + first + i + 1)) : 0;
    k.z = i + 2 < mid ? key_of(__ldg(score + first + i + 2)) : 0;
    k.w = i + 3 < mid ? key_of(__ldg(score + first + i + 3)) : 0;
    return k;
  };
  auto keys_at = [&](int i) { return cached ? *reinterpret_cast<const uint4*>(s_key + i) : load4(i); };
  constexpr int kTop = 20, kMiddle = 10;  // lowest bits of the first two passes' bins
  for (int i = threadIdx.x; i < kBins; i += kThreads) s_hist[i] = 0;
  if (cached) {  // eight loads in flight; the first pass's count on the way
    __syncthreads();
    for (int i0 = threadIdx.x; i0 < (mid + 3) / 4 * 4; i0 += 8 * kThreads) {
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = i0 + e * kThreads < mid ? __ldg(score + first + i0 + e * kThreads) : 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = i0 + e * kThreads;
        const uint32_t k = key_of(v[e]);
        if (i < mid) s_key[i] = k, atomicAdd(&s_hist[k >> kTop], 1);
        else if (i < (mid + 3) / 4 * 4) s_key[i] = 0;
      }
    }
  }
  uint32_t prefix = 0, mask = 0;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? kTop : pass == 1 ? kMiddle : 0;
    const int bins = pass == 0 ? kBins : kLowBins;
    if (pass > 0)
      for (int i = threadIdx.x; i < kLowBins; i += kThreads) s_hist[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x * 4; i < mid && (pass > 0 || !cached); i += kThreads * 4) {
      const uint4 k = keys_at(i);
      auto count = [&](uint32_t v, bool have) {
        if (have && (v & mask) == prefix) atomicAdd(&s_hist[v >> shift & (bins - 1)], 1);
      };
      count(k.x, true), count(k.y, i + 1 < mid), count(k.z, i + 2 < mid), count(k.w, i + 3 < mid);
    }
    __syncthreads();
    // the bin that the want-th largest falls into; thread i has sixteen, or four, bins from the top
    const int E = bins / kThreads;
    int n = 0;
    for (int e = 0; e < E; e += 4) {
      const int4 h = *reinterpret_cast<const int4*>(s_hist + bins - (threadIdx.x + 1) * E + e);
      n += h.x + h.y + h.z + h.w;
    }
    int total;
    int before = block_scan<kThreads>(n, s_warp, total);
    if (before < want && want <= before + n) {
      int bin = bins - 1 - threadIdx.x * E;
      while (before + s_hist[bin] < want) before += s_hist[bin--];
      s_bin = bin, s_want = want - before;
    }
    __syncthreads();
    want = s_want;
    prefix |= static_cast<uint32_t>(s_bin) << shift;
    mask |= static_cast<uint32_t>(bins - 1) << shift;
  }
  // Keys above the bound stay, and the first `want` of those equal to it (0 is no key).
  // A warp has a part of the middle, a lane four keys side by side.
  const uint32_t bound = prefix;
  const int part = ((mid + kThreads / 32 - 1) / (kThreads / 32) + 127) & ~127;
  const int i0 = warp * part, i1 = min(mid, i0 + part);
  int more = 0, eqs = 0;
  for (int i = i0 + lane * 4; i < i1; i += 128) {
    const uint4 k = keys_at(i);
    more += (k.x > bound) + (k.y > bound) + (k.z > bound) + (k.w > bound);
    eqs += (k.x == bound) + (k.y == bound) + (k.z == bound) + (k.w == bound);
  }
  more = __reduce_add_sync(0xFFFFFFFFu, more), eqs = __reduce_add_sync(0xFFFFFFFFu, eqs);
  if (lane == 0) s_more[0][warp] = more, s_more[1][warp] = eqs;
  __syncthreads();
  int eq_before = 0, at = p.sinks;
  for (int w = 0; w < warp; ++w) {
    at += s_more[0][w] + max(0, min(want - eq_before, s_more[1][w]));
    eq_before += s_more[1][w];
  }
  for (int base = i0; base < i1; base += 128) {
    const int i = base + lane * 4;
    const uint4 k = i < i1 ? keys_at(i) : make_uint4(0, 0, 0, 0);
    const uint32_t v[4] = {k.x, k.y, k.z, k.w};
    int gt = 0, eq = 0;  // bits
#pragma unroll
    for (int e = 0; e < 4; ++e) gt |= (v[e] > bound) << e, eq |= (v[e] == bound) << e;
    // keys above and equal in front of the lane's, in one scan
    int both = __popc(gt) | __popc(eq) << 16;
    const int mine = both;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xFFFFFFFFu, both, o);
      if (lane >= o) both += up;
    }
    const int all = __shfl_sync(0xFFFFFFFFu, both, 31), front = both - mine;
    int eq_at = eq_before + (front >> 16);
    int to = at + (front & 0xFFFF) + max(0, min(want, eq_at) - min(want, eq_before));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool equal = eq >> e & 1;
      if ((gt >> e & 1) || (equal && eq_at < want)) list[to++] = first + i + e;
      eq_at += equal;
    }
    at += (all & 0xFFFF) + max(0, min(want, eq_before + (all >> 16)) - min(want, eq_before));
    eq_before += all >> 16;
  }
}

// -------------------------------------------------------------------- move
// Block x: (layer of the group, row, kv head, keys or values); the last S blocks
// write the rows' new pages down.
template <int D>
__global__ void __launch_bounds__(kThreads) evict_move_kernel(const Params p, int layer0, int layers) {
  constexpr int U = D / 32;               // 16-byte units of a token's codes
  constexpr int R = kTile * U / kThreads; // units per thread and step
  constexpr int SB = D / 16;              // bytes of a token's scales
  wait_for_previous();
  const int items = layers * p.S * p.Hkv * 2;
  if (static_cast<int>(blockIdx.x) >= items) {
    const int r = blockIdx.x - items;
    const bool kept = stays(plan_of(p, r));
    if (threadIdx.x == 0) {
      if (p.row_rank[r] >= 0 && kept) atomicOr(p.err, kErrNoPages);
      if (p.dropped) p.dropped[r] = kept ? 0 : p.row_len[r] - p.keep;
      if (!kept) p.lens[r] = p.keep;
    }
    if (kept) return;
    const int used = (p.row_len[r] + p.P - 1) / p.P;
    for (int j = threadIdx.x; j < used; j += kThreads) {
      const int a = p.src[static_cast<long long>(r) * p.M + j], b = p.dst[static_cast<long long>(r) * p.M + j];
      if (a == b) continue;
      if (page_ok(a, p.N)) atomicSub(p.refs + a, 1);
      if (b >= 0) p.refs[b] = 1;
      p.table[static_cast<long long>(r) * p.M + j] = b;
    }
    return;
  }
  const int half = blockIdx.x & 1, x = blockIdx.x >> 1;
  const int h = x % p.Hkv, r = x / p.Hkv % p.S, l = x / p.Hkv / p.S;
  if (stays(plan_of(p, r))) return;
  const int* list = p.list + ((static_cast<long long>(l) * p.S + r) * p.Hkv + h) * p.keep;
  const int *src = p.src + static_cast<long long>(r) * p.M, *dst = p.dst + static_cast<long long>(r) * p.M;
  const int rec = record_bytes(p.P, D);
  uint8_t* codes = p.pool + (layer0 + l) * p.layer_stride + static_cast<long long>(h) * rec + half * (rec / 2);
  uint8_t* scales = codes + codes_bytes(p.P, D);
  float* score = half == 0 && p.score ? p.score + ((static_cast<long long>(layer0 + l) * p.S + r) * p.Hkv + h) * p.cap : nullptr;
  const long long page_bytes = static_cast<long long>(p.Hkv) * rec;
  const int shift = 31 - __clz(p.P), in_page = p.P - 1;
  // places of a step's tokens: page before and after in bytes, offset in the page; -1: stays where it is, or has no page
  __shared__ long long s_from[3][kTile], s_to[3][kTile];
  __shared__ int s_off[3][kTile];  // offsets before and after, 16 bits each
  auto plan = [&](int k) {
    const int d = k * kTile + threadIdx.x;
    if (d >= p.keep) return;
    const int t = list[d], pa = src[t >> shift], pb = dst[d >> shift];
    const bool ok = page_ok(pa, p.N) && page_ok(pb, p.N);
    if (!ok) atomicOr(p.err, kErrBadIndex);
    s_from[k % 3][threadIdx.x] = pa * page_bytes;
    s_to[k % 3][threadIdx.x] = ok && (pa != pb || t != d) ? pb * page_bytes : -1;
    s_off[k % 3][threadIdx.x] = (t & in_page) | (d & in_page) << 16;
  };
  struct Held {
    uint4 v[R];
    uint2 s;
    float sum;
  };
  auto load = [&](int k, Held& x) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int unit = threadIdx.x + i * kThreads, tok = unit / U, c = unit % U;
      if (k * kTile + tok < p.keep && s_to[k % 3][tok] >= 0)
        x.v[i] = *reinterpret_cast<const uint4*>(codes + s_from[k % 3][tok] + (s_off[k % 3][tok] & 0xFFFF) * (D / 2) + c * 16);
    }
    const int d = k * kTile + threadIdx.x;
    if (d >= p.keep) return;
    if (score) x.sum = score[list[d]];
    if (s_to[k % 3][threadIdx.x] >= 0) {
      const uint8_t* from = scales + s_from[k % 3][threadIdx.x] + (s_off[k % 3][threadIdx.x] & 0xFFFF) * SB;
      if (SB == 8) x.s = *reinterpret_cast<const uint2*>(from);
      else x.s.x = *reinterpret_cast<const uint32_t*>(from);
    }
  };
  auto store = [&](int k, const Held& x) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int unit = threadIdx.x + i * kThreads, tok = unit / U, c = unit % U;
      if (k * kTile + tok < p.keep && s_to[k % 3][tok] >= 0)
        *reinterpret_cast<uint4*>(codes + s_to[k % 3][tok] + (s_off[k % 3][tok] >> 16) * (D / 2) + c * 16) = x.v[i];
    }
    const int d = k * kTile + threadIdx.x;
    if (d >= p.keep) return;
    if (score) score[d] = x.sum;
    if (s_to[k % 3][threadIdx.x] >= 0) {
      uint8_t* to = scales + s_to[k % 3][threadIdx.x] + (s_off[k % 3][threadIdx.x] >> 16) * SB;
      if (SB == 8) *reinterpret_cast<uint2*>(to) = x.s;
      else *reinterpret_cast<uint32_t*>(to) = x.s.x;
    }
  };
  // a step's loads in flight while the one before is stored: those read tokens behind
  // all that these write.  The barrier in between: a step's loads, every thread's, come
  // before its stores.
  const int steps = (p.keep + kTile - 1) / kTile;
  Held now, next;
  plan(0);
  if (steps > 1) plan(1);
  __syncthreads();
  load(0, now);
  for (int k = 0; k < steps; ++k) {
    __syncthreads();
    if (k + 1 < steps) load(k + 1, next);
    if (k + 2 < steps) plan(k + 2);
    store(k, now);
    now = next;
  }
}

// Tokens of a list: `keep`, where any row has more than that (a page holds 128 at most).
long long listed(int keep, int M) { return std::min<long long>(keep, 128ll * M); }
int group_of(int layers, int S, int Hkv, int M, int keep) {
  const long long per = static_cast<long long>(S) * Hkv * listed(keep, M) * 4;
  return static_cast<int>(std::max<long long>(1, std::min<long long>(layers, kListBytes / std::max(per, 1ll))));
}

size_t carve(Params& p, void* ws, int layers, int S, int M, int N, int Hkv, int keep) {
  Carve c(ws, 0);
  p.count = c.take<int>(1);
  p.fresh = c.take<int>(N);
  p.row_rank = c.take<int>(S);
  p.row_more = c.take<int>(S);
  p.row_len = c.take<int>(S);
  p.src = c.take<int>(static_cast<size_t>(S) * M);
  p.dst = c.take<int>(static_cast<size_t>(S) * M);
  p.list = c.take<int>(static_cast<size_t>(group_of(layers, S, Hkv, M, keep)) * S * Hkv * listed(keep, M));
  return c.used;
}

bool sizes_ok(int layers, int S, int M, int N, int Hkv, int keep) {
  return layers >= 1 && S >= 0 && M >= 1 && N >= 1 && Hkv >= 1 && keep >= 1;
}
bool sizes_fit(int layers, int S, int M, int N, int P, int Hkv) {
  return S <= (1 << 20) && N <= (1 << 27) && static_cast<long long>(M) * P <= (1 << 30) &&
         static_cast<long long>(layers) * S * Hkv < (1 << 29);
}

}  // namespace
}  // namespace kv4
}  // namespace moe

using namespace moe;

extern "C" size_t moe_kv4_evict_workspace_size(int layers, int rows, int max_pages, int num_pages, int Hkv, int keep) {
  if (!kv4::sizes_ok(layers, rows, max_pages, num_pages, Hkv, keep) || rows > (1 << 20)) return 0;
  kv4::Params p;
  return kv4::carve(p, nullptr, layers, rows, max_pages, num_pages, Hkv, keep);
}

extern "C" int moe_kv4_evict(const int32_t* table_in, const int32_t* lens_in, const int32_t* refs_in, int rows,
                             int max_pages, int num_pages, int page_size, int32_t* table_out, int32_t* lens_out,
                             int32_t* refs_out, int32_t* dropped, uint8_t* pool, int layers, long long layer_stride,
                             int Hkv, int D, float* score, int cap, int keep, int limit, int sinks, int recent, void* ws,
                             size_t ws_bytes, void* stream) {
  using namespace kv4;
  if (!sizes_ok(layers, rows, max_pages, num_pages, Hkv, keep) || sinks < 0 || recent < 0 || limit < keep ||
      static_cast<long long>(sinks) + recent > keep)
    return MOE_ERR_INVALID_ARG;
  if (!page_size_ok(page_size) || !head_dim_ok(D) || !sizes_fit(layers, rows, max_pages, num_pages, page_size, Hkv))
    return MOE_ERR_UNSUPPORTED;
  if (!refs_in || !refs_out || !aligned(refs_in, 4) || !aligned(refs_out, 4)) return MOE_ERR_INVALID_ARG;
  if (!pool || !aligned(pool, 16) || layer_stride % 16 != 0 ||
      (layers > 1 && layer_stride < static_cast<long long>(num_pages) * Hkv * record_bytes(page_size, D)))
    return MOE_ERR_INVALID_ARG;
  if (rows > 0 && (!table_in || !lens_in || !table_out || !lens_out || !aligned(table_in, 4) || !aligned(lens_in, 4) ||
                   !aligned(table_out, 4) || !aligned(lens_out, 4) || !aligned(dropped, 4)))
    return MOE_ERR_INVALID_ARG;
  // the sums decide where the first and last tokens are not all that stays
  if (rows > 0 && !score && keep > sinks + recent) return MOE_ERR_INVALID_ARG;
  if (score && (!aligned(score, 4) || cap < max_pages * page_size)) return MOE_ERR_INVALID_ARG;
  Params p{table_in, lens_in, refs_in, table_out, lens_out, refs_out, dropped, pool, layer_stride, score,
           rows, max_pages, num_pages, page_size, D, Hkv, layers, cap, keep, limit, sinks, recent};
  if (!ws || !aligned(ws, 256)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < carve(p, ws, layers, rows, max_pages, num_pages, Hkv, keep)) return MOE_ERR_WORKSPACE;
  p.err = device_error_word();
  if (!p.err) return MOE_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool carries = p.table != p.table_in || p.lens != p.lens_in || p.refs != p.refs_in;
  const long long n = std::max<long long>(static_cast<long long>(rows) * max_pages, num_pages);
  const int wide = carries ? static_cast<int>(std::max<long long>(1, std::min<long long>(num_sms(), n / (4 * kPlan)))) : 0;
  const bool small = rows > 0 && rows <= kSmallRows && num_pages <= kSmallPages;
  if (!small) {
    evict_plan_kernel<<<1 + wide, kPlan, 0, s>>>(p);
    MOE_TRY(check_launch());
  }
  if (rows == 0) return MOE_OK;
  static std::atomic<bool> set[64];
  MOE_TRY(allow_smem(evict_select_kernel, kCached * 4, set));
  const int smem = std::min(kCached, max_pages * page_size) * 4;
  const int group = group_of(layers, rows, Hkv, max_pages, keep);
  for (int l0 = 0; l0 < layers; l0 += group) {
    const int m = std::min(group, layers - l0);
    const bool begin = l0 == 0, end = l0 + m >= layers;
    const dim3 choose(m * rows * Hkv + (begin ? rows + (small ? 4 * wide : 0) : 0));
    if (begin && small) {
      evict_select_kernel<<<choose, kThreads, smem, s>>>(p, l0, m, true);
      MOE_TRY(check_launch());
    } else {
      MOE_TRY(launch_after(evict_select_kernel, choose, kThreads, smem, s, p, l0, m, false));
    }
    const dim3 grid(m * rows * Hkv * 2 + (end ? rows : 0));
    if (D == 128) MOE_TRY(launch_after(evict_move_kernel<128>, grid, kThreads, 0, s, p, l0, m));
    else MOE_TRY(launch_after(evict_move_kernel<64>, grid, kThreads, 0, s, p, l0, m));
  }
  return MOE_OK;
}
