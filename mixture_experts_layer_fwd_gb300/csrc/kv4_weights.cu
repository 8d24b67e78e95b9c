// Attention weights of a step's queries, summed up for each key of the paged
// NVFP4 cache:
//   score[b][h][t] (+)= sum over queries i that see t and query heads a of h of
//                       exp(scale * q_{i,a} . k_t - lse_{i,a})
// with the lse that the step's attention gave.  A key that the step wrote itself
// has no older sum: its score is set, not added to.
//
// Bound: few queries the bytes of the keys, D * 9/16 each, read once per kv head;
// many the products and the exponentials.  A first launch brings the queries into the
// order that the products read (fp16, each row times a power of two) with what each row
// needs beside them.  Then, by the rows (query, head) of a sequence and kv head:
//   up to 16    every warp takes an equal range of the line of all (sequence, kv head,
//               32 keys), holds the rows' operands in registers and streams the keys
//               through a ring of asynchronous copies
//   up to 255   a block takes 32 to 128 keys, expands them into registers and walks the
//               rows that see one of them, staged 32 KB at a time
//   more        tcgen05, in a launch of its own (see there)
// A key's rows are added in a fixed order: the same result each time.
//
// 256 sequences of up to 8192 keys, one query of 64 heads on 4 of 128: 6.5 + 90 us on the
// GPU (0.59 of the copy bandwidth; half of the issue slots, half of them expanding codes).
// Five chunks of 600 queries, window 1024, 35 heads on 5 of 64: 9 + 40 us; 4096 queries
// on 12289 keys, 64 heads on 4 of 128: 28 + 640 us (1.1 PFLOP/s).
#include <climits>
#include <type_traits>

#include "nvfp4_mma.cuh"

namespace moe {
namespace kv4 {
namespace {

constexpr int kKeys = 32;         // of a warp's step
constexpr int kFewRows = 16;      // of a sequence and kv head: a warp holds them in registers
// These and more go to the tiles' kernel: 32 sequences of 8192 keys, heads of 128, 128 /
// 192 / 256 / 384 / 512 rows 178 / 217 / 194 / 218 / 231 us on the GPU there, 149 / 189 /
// 226 / 311 / 395 in registers; of up to 8192 keys 78 / 96 / 108 / 123 / 140 and 69 / 82 /
// 97 / 124 / 154; 16 of 4096 keys, heads of 64, 128 / 256 / 384 / 512 rows 44 / 49 / 56 / 60
// and 35 / 47 / 62 / 74.
constexpr int kTileRows = 256;
constexpr int kTileKeys = 128;    // of an item there
constexpr int kParts = 4;         // of an item, where they are few
constexpr int kPrepThreads = 256, kThreads = 256;
constexpr int kMaxRows = 1 << 14; // sequences

// What eight query rows need beside their values: weight = 2^(product * sc - lse2) on
// the keys [lo, hi).
struct Rows {
  float2 sc_lse2[8];
  int2 see[8];
};
// The same for the kernel that has the keys on the rows of its products: one after the
// other from where a sequence's and kv head's Rows would begin.
struct Columns {
  float sc[8], less_lse2[8];
};

struct Params {
  const uint16_t* q;
  long long q_stride;
  const uint8_t* pool;
  const float* g_k;
  const float* lse;
  const int32_t *q_offsets, *kv_lens, *table;
  float* score;
  int T, B, Hq, Hkv, G, num_pages, P, P_log2, max_pages, causal, window, cap;
  float scale;
  int tile_rows;        // rows of a sequence and kv head from which on the tiles' kernel has them
  unsigned long long timeout_ns;
  // workspace
  int* starts;          // [B + 1] q_offsets as used
  int* row_tiles;       // [B + 1] row tiles of one kv head before sequence b
  long long* few;       // [B + 1] steps of one kv head before sequence b: of 32 keys, of sequences with few rows
  long long* many;      // [3][B + 1] the same of those with more: of 32, 64 and 128 keys
  long long* big;       // [B + 1] of those that the tiles' kernel has: of 128 keys
  int* taken;           // [2] steps of many rows, of the tiles' kernel, that a block has taken
  int split;            // items of the tiles' kernel, fewer of which are split
  int* parts_done;      // [split] parts of an item that are summed up
  float* part;          // [split][kParts][kTileKeys]
  uint4* frag;          // [row tile of all][D / 32][32]; the tiles' kernel's: of each sequence and kv head
                        // [D / 64][row tile][8 rows of 128 bytes], swizzled
  Rows* rows;           // [row tile of all]
  unsigned int* err;
};

DEVINL int seq_len(const Params& p, int b) {
  const long long cap = static_cast<long long>(p.max_pages) * p.P;
  return static_cast<int>(max(0ll, min(static_cast<long long>(p.kv_lens[b]), cap)));
}
// First key that any of the n queries of a sequence sees.
DEVINL int first_key(const Params& p, int n, int len) {
  return p.window > 0 ? static_cast<int>(min(static_cast<long long>(len), max(0ll, static_cast<long long>(len) - n - p.window + 1))) : 0;
}
// Steps of `keys` keys of one kv head.
DEVINL int steps_of(const Params& p, int n, int len, int keys) {
  return n > 0 && len > 0 ? (len + keys - 1) / keys - first_key(p, n, len) / keys : 0;
}
DEVINL int kind_of(const Params& p, int n) {  // 0: few rows, 1: many, 2: the tiles' kernel
  return n <= kFewRows / p.G ? 0 : n * p.G < p.tile_rows ? 1 : 2;
}

// Running maxima (MAX) or sums over a warp.
template <bool MAX, class T>
DEVINL T warp_scan(T v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T up = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v = MAX ? max(v, up) : v + up;
  }
  return v;
}

// A warp brings one row tile into place; each of the `blocks` blocks makes the prefix sums
// for itself (s_sum: [B + 1] starts, [B + 1] row tiles), the first one writes them down.
template <int D>
DEVINL void prepare(const Params& p, int block, int blocks, int* s_sum) {
  constexpr int kWarps = kPrepThreads / 32;
  __shared__ int s_end[kWarps];
  constexpr int kSums = 6;  // row tiles; steps of few rows; of many, of 32, 64 and 128 keys; of the tiles' kernel
  __shared__ long long s_total[kSums][kWarps];
  int *s_start = s_sum, *s_tile = s_sum + p.B + 1;
  const bool writes = block == 0;
  // offsets inside the tokens, never falling
  int reached = min(max(p.q_offsets[0], 0), p.T);
  long long before[kSums] = {};
  if (threadIdx.x == 0) s_start[0] = reached, s_tile[0] = 0;
  auto sums_of = [&](int k) { return k == 1 ? p.few : k < 5 ? p.many + (k - 2) * (p.B + 1) : p.big; };
  if (writes && threadIdx.x > 0 && threadIdx.x < kSums) sums_of(threadIdx.x)[0] = 0;
  if (writes && threadIdx.x < 2) p.taken[threadIdx.x] = 0;
  if (writes)
    for (int i = threadIdx.x; i < p.split; i += kPrepThreads) p.parts_done[i] = 0;
  {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int base = 0; base < p.B; base += kPrepThreads) {
      const int b = base + threadIdx.x;
      const bool have = b < p.B;
      const int len = have && writes ? seq_len(p, b) : 0;
      int end = warp_scan<true>(have ? min(max(p.q_offsets[b + 1], 0), p.T) : 0);
      if (lane == 31) s_end[warp] = end;
      __syncthreads();
      int begin = reached;
      for (int w = 0; w < warp; ++w) begin = max(begin, s_end[w]);
      for (int w = 0; w < kWarps; ++w) reached = max(reached, s_end[w]);
      const int up = __shfl_up_sync(0xFFFFFFFFu, end, 1);
      end = max(end, begin);
      if (lane > 0) begin = max(begin, up);
      const int n = have ? end - begin : 0;
      const int kind = kind_of(p, n);
      long long v[kSums] = {(static_cast<long long>(n) * p.G + 7) / 8};
      v[0] = warp_scan<false>(v[0]);
      if (writes) {
#pragma unroll
        for (int k = 1; k < kSums; ++k)
          v[k] = warp_scan<false>(static_cast<long long>(
              kind == (k + 1) / 3 ? steps_of(p, n, len, k < 5 ? kKeys << max(k - 2, 0) : kTileKeys) : 0));
      }
      if (lane == 31)
#pragma unroll
        for (int k = 0; k < kSums; ++k) s_total[k][warp] = v[k];
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kSums; ++k) {
        if (k > 0 && !writes) break;
        long long at = before[k];
        for (int w = 0; w < kWarps; ++w) {
          at += w < warp ? s_total[k][w] : 0;
          before[k] += s_total[k][w];
        }
        v[k] += at;
      }
      if (have) {
        s_start[b + 1] = end, s_tile[b + 1] = static_cast<int>(v[0]);
        if (writes) {
#pragma unroll
          for (int k = 1; k < kSums; ++k) sums_of(k)[b + 1] = v[k];
        }
      }
    }
  }
  __syncthreads();
  if (writes)
    for (int i = threadIdx.x; i <= p.B; i += kPrepThreads) p.starts[i] = s_start[i], p.row_tiles[i] = s_tile[i];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c4 = lane & 3;
  const int total = s_tile[p.B];
  const long long all = static_cast<long long>(total) * p.Hkv;
  for (long long x = static_cast<long long>(block) * kWarps + warp; x < all; x += static_cast<long long>(blocks) * kWarps) {
    const int h = static_cast<int>(x % p.Hkv), f = static_cast<int>(x / p.Hkv);
    const int b = warp_find(p.B, f, [&](int i) { return static_cast<long long>(s_tile[i]); });
    const int n = s_start[b + 1] - s_start[b], len = seq_len(p, b);
    const int tiles = s_tile[b + 1] - s_tile[b], mine = f - s_tile[b];
    const int r = mine * 8 + g, tok = r / p.G;
    const bool have = r < n * p.G;
    uint4 v[D / 32];
    uint32_t top = 0;
    const long long token = s_start[b] + tok;
    const int head = h * p.G + r - tok * p.G;
    const float l = have ? p.lse[token * p.Hq + head] : -INFINITY;
    const bool gives = l != -INFINITY;  // a row without weight is one of zeros, whatever lies in it
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
      v[j] = make_uint4(0, 0, 0, 0);
      if (have) v[j] = __ldg(reinterpret_cast<const uint4*>(p.q + token * p.q_stride + head * D + c4 * (D / 4)) + j);
    }
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
      if (!gives) v[j] = make_uint4(0, 0, 0, 0);
      top = max(top, bf16x8_top(v[j]));
    }
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    const int e = f16_exponent(top);
    const long long to = static_cast<long long>(s_tile[b]) * p.Hkv + static_cast<long long>(h) * tiles + mine;
    const bool columns = kind_of(p, n) == 2;
    uint4* at = p.frag + to * D + lane;  // a row tile's D units
    int next = 32;
    if (columns) at = p.frag + (to - mine) * D + mine * 64 + 8 * g, next = 0;
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
      const int unit = c4 * (D / 32) + j;  // of 16 bytes
      at[columns ? (unit >> 3) * (tiles * 64) + ((unit & 7) ^ g) : j * next] = bf16x8_to_f16x8(v[j], power_of_two(e));
    }
    if (c4 == 0) {
      float2 w = make_float2(0.0f, INFINITY);
      int2 see = make_int2(0, 0);
      if (gives) {
        w.x = p.scale * __ldg(p.g_k + h) * kLog2e * power_of_two(-e);
        w.y = l * kLog2e;
      }
      if (have) {
        const int place = len - n + tok;
        see.x = p.window > 0 ? max(place - p.window + 1, 0) : 0;
        see.y = p.causal ? min(max(place + 1, 0), len) : len;
      }
      if (columns) {
        Columns& c = reinterpret_cast<Columns*>(p.rows + (to - mine))[mine];
        c.sc[g] = w.x, c.less_lse2[g] = -w.y;
      } else {
        p.rows[to].sc_lse2[g] = w;
        p.rows[to].see[g] = see;
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kPrepThreads) weights_prepare_kernel(const Params p) {
  extern __shared__ int s_sum[];
  launch_dependents();
  prepare<D>(p, blockIdx.x, gridDim.x, s_sum);
}

// Codes and scales of 16 keys, g and g + 8: a quarter of each.
template <int D>
struct Keys {
  uint32_t c[2][D / 32];
  uint32_t s[2];
};
// The record of kv head h in page `page` (one outside the pool: reported, and page 0's).
template <int D>
DEVINL const uint8_t* record_of(const Params& p, int page, int h) {
  const bool ok = page >= 0 && page < p.num_pages;
  if (!ok && (threadIdx.x & 31) == 0) atomicOr(p.err, kErrBadIndex);
  return p.pool + (static_cast<long long>(ok ? page : 0) * p.Hkv + h) * record_bytes(p.P, D);
}
template <int D>
DEVINL void load_keys(const Params& p, const uint8_t* rec, int off, Keys<D>& k) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c4 = lane & 3;
  const uint8_t* sf = rec + codes_bytes(p.P, D);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int key = off + g + 8 * i;
    if (D == 128) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(rec + key * (D / 2) + c4 * 16));
      k.c[i][0] = v.x, k.c[i][1] = v.y, k.c[i][D / 64] = v.z, k.c[i][D / 32 - 1] = v.w;
      k.s[i] = __ldg(reinterpret_cast<const uint16_t*>(sf + key * 8 + c4 * 2));
    } else {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(rec + key * (D / 2) + c4 * 8));
      k.c[i][0] = v.x, k.c[i][1] = v.y;
      k.s[i] = __ldg(sf + key * 4 + c4);
    }
  }
}
template <int D>
DEVINL Expanded expand_word(const Keys<D>& k, int j, uint32_t s0, uint32_t s1) {
  const uint32_t at = D == 128 && j >= 2 ? 0x3232u : 0x1010u;
  return expand(k.c[0][j], __byte_perm(s0, s0, at), k.c[1][j], __byte_perm(s1, s1, at));
}

// sum[i] += the weights of key t + 8 i (t the lane's) with the lane's two rows of an
// accumulator; w: their sc, lse2; see: their lo, hi where some row of the tile does not
// see all of the step's keys, else null.
DEVINL void add_weights(float (&sum)[2], const float (&acc)[4], const float4& w) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    sum[i] += ex2(fmaf(acc[2 * i], w.x, -w.y));
    sum[i] += ex2(fmaf(acc[2 * i + 1], w.z, -w.w));
  }
}
DEVINL void add_weights(float (&sum)[2], const float (&acc)[4], const float4& w, const int4& see, int t) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int k = t + 8 * i;
    if (k >= see.x && k < see.y) sum[i] += ex2(fmaf(acc[2 * i], w.x, -w.y));
    if (k >= see.z && k < see.w) sum[i] += ex2(fmaf(acc[2 * i + 1], w.z, -w.w));
  }
}
DEVINL float4 weights_at(const Rows& r, int c4) { return reinterpret_cast<const float4*>(r.sc_lse2)[c4]; }
DEVINL int4 see_at(const Rows& r, int c4) { return reinterpret_cast<const int4*>(r.see)[c4]; }
// Sums over the four lanes of a key; lane c gets that of s[c >> 1][c & 1].
DEVINL float quad_sums(const float (&s)[2][2]) {
  const int c4 = threadIdx.x & 3;
  const bool up = c4 & 2, odd = c4 & 1;
  const float a = (up ? s[1][0] : s[0][0]) + __shfl_xor_sync(0xFFFFFFFFu, up ? s[0][0] : s[1][0], 2);
  const float b = (up ? s[1][1] : s[0][1]) + __shfl_xor_sync(0xFFFFFFFFu, up ? s[0][1] : s[1][1], 2);
  return (odd ? b : a) + __shfl_xor_sync(0xFFFFFFFFu, odd ? a : b, 1);
}
// A warp's ring of steps in flight: each lane copies the codes that it reads itself, and
// the scales of one key.
constexpr int kSlots = 4;
template <int D>
struct Slot {
  uint4 codes[D / 32][32];     // [16 keys][key g or g + 8][lane], D = 64: two of the latter side by side
  uint8_t scales[kKeys][D / 16];
};
template <int D>
__host__ __device__ constexpr int ring_bytes() { return static_cast<int>(sizeof(Slot<D>)) * kSlots * (kThreads / 32); }
template <int D>
DEVINL void cp_async(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}

// A warp's equal range of the line of all (sequence, kv head, 32 keys) with few
// rows: their operands stay in registers while the keys stream past.
template <int D>
DEVINL void few_rows(const Params& p, Slot<D>* ring) {
  constexpr int W = D / 32;  // words of codes of a lane and key
  const int lane = threadIdx.x & 31, g = lane >> 2, c4 = lane & 3;
  const long long total = p.few[p.B] * p.Hkv, warps = static_cast<long long>(gridDim.x) * (kThreads / 32);
  const long long range = (total + warps - 1) / warps;
  const long long x0 = (static_cast<long long>(threadIdx.x >> 5) * gridDim.x + blockIdx.x) * range;
  const int count = static_cast<int>(min(total, x0 + range) - x0);
  if (count <= 0) return;
  struct Cursor {  // a place on the line
    int b, h, step, first, steps, older;  // older: keys that the step did not write
  };
  auto enter = [&](Cursor& c) {
    const int n = p.starts[c.b + 1] - p.starts[c.b], len = seq_len(p, c.b);
    c.first = first_key(p, n, len) / kKeys, c.steps = static_cast<int>(p.few[c.b + 1] - p.few[c.b]), c.older = len - n;
  };
  auto advance = [&](Cursor& c) {
    if (++c.step < c.steps) return;
    c.step = 0;
    if (++c.h < p.Hkv) return;
    c.h = 0;
    do {
      ++c.b;
      enter(c);
    } while (c.steps == 0);
  };
  auto page_of = [&](const Cursor& c) {
    return p.table[static_cast<long long>(c.b) * p.max_pages + ((c.first + c.step) * kKeys >> p.P_log2)];
  };
  Cursor in;  // of the step whose page is known: the next to be copied
  in.b = warp_find(p.B, x0, [&](int i) { return p.few[i] * p.Hkv; });
  enter(in);
  const long long r0 = x0 - p.few[in.b] * p.Hkv;
  in.h = static_cast<int>(r0 / in.steps), in.step = static_cast<int>(r0 - static_cast<long long>(in.h) * in.steps);
  Cursor at = in;  // of the step at hand, from the middle of a step on of the next
  int page = page_of(in), to_copy = count, slot_in = 0;
  // a lane's part of a step: its codes of four keys (D = 128; else 16 bytes of 16 keys, as
  // they lie, twice), one key's scales
  const int lane_codes = D == 128 ? g * 64 + c4 * 16 : lane * 16, lane_scales = lane * (D / 16);
  auto copy_next = [&] {
    if (to_copy > 0) {
      Slot<D>& s = ring[slot_in];
      const int off = (in.first + in.step) * kKeys & (p.P - 1);
      const uint8_t* rec = record_of<D>(p, page, in.h);
      const uint8_t* from = rec + (off * (D / 2) + lane_codes);
#pragma unroll
      for (int i = 0; i < W; ++i) cp_async<D>(&s.codes[i][lane], from + i * 512);
      from = rec + codes_bytes(p.P, D) + (off * (D / 16) + lane_scales);
      if (D == 128) asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(s.scales[lane])), "l"(from) : "memory");
      else asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(s.scales[lane])), "l"(from) : "memory");
      if (--to_copy > 0) advance(in), page = page_of(in);
      slot_in = slot_in + 1 == kSlots ? 0 : slot_in + 1;
    }
    cp_async_commit();
  };
#pragma unroll 1
  for (int i = 0; i < kSlots - 1; ++i) copy_next();
  // the older sum of the lane's key, loaded a step ahead; keys that the step wrote itself have none
  auto old_at = [&](const Cursor& c) {
    const int t = (c.first + c.step) * kKeys + g + 8 * c4;
    return t < c.older ? p.score[(static_cast<long long>(c.b) * p.Hkv + c.h) * p.cap + t] : 0.0f;
  };
  float next_old = old_at(at);
  int of_b = -1, of_h = -1, len = 0, all_lo = 0, all_hi = 0, slot = 0;
  bool two = false;
  uint4 q[2][W];
  float4 w[2];
  const Rows* rows = nullptr;
  float* score = nullptr;

  // the weights of a step's keys, by one tile of rows or two
  auto tile = [&](auto two_tiles, auto masked, const Slot<D>& s, int t0) {
    constexpr int F = decltype(two_tiles)::value ? 2 : 1;
    constexpr bool MASK = decltype(masked)::value;
    float acc[2][F][4], sum[2][2];
    Keys<D> keys[2];
    uint32_t s0[2], s1[2];
#pragma unroll
    for (int a = 0; a < 2; ++a) {
#pragma unroll
      for (int f = 0; f < F; ++f) acc[a][f][0] = acc[a][f][1] = acc[a][f][2] = acc[a][f][3] = 0.0f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int key = 16 * a + 8 * i + g;
        if (D == 128) {
          const uint4 v = s.codes[(2 * a + i) % W][lane];
          keys[a].c[i][0] = v.x, keys[a].c[i][1] = v.y, keys[a].c[i][D / 64] = v.z, keys[a].c[i][D / 32 - 1] = v.w;
          keys[a].s[i] = *reinterpret_cast<const uint16_t*>(&s.scales[key][2 * c4 % (D / 16)]);
        } else {
          const uint2 v = reinterpret_cast<const uint2*>(&s.codes[0][0])[key * 4 + c4];
          keys[a].c[i][0] = v.x, keys[a].c[i][1] = v.y;
          keys[a].s[i] = s.scales[key][c4];
        }
      }
      s0[a] = e4m3x2_to_f16x2(keys[a].s[0]), s1[a] = e4m3x2_to_f16x2(keys[a].s[1]);
    }
#pragma unroll
    for (int j = 0; j < W; ++j) {
      Expanded e[2];
#pragma unroll
      for (int a = 0; a < 2; ++a) e[a] = expand_word<D>(keys[a], j, s0[a], s1[a]);
#pragma unroll
      for (int f = 0; f < F; ++f)
#pragma unroll
        for (int a = 0; a < 2; ++a) mma_half<0>(acc[a][f], e[a], q[f][j]);
#pragma unroll
      for (int f = 0; f < F; ++f)
#pragma unroll
        for (int a = 0; a < 2; ++a) mma_half<1>(acc[a][f], e[a], q[f][j]);
    }
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      sum[a][0] = sum[a][1] = 0.0f;
#pragma unroll
      for (int f = 0; f < F; ++f) {
        if (MASK) add_weights(sum[a], acc[a][f], w[f], see_at(rows[f], c4), t0 + 16 * a + g);
        else add_weights(sum[a], acc[a][f], w[f]);
      }
    }
    return quad_sums(sum);
  };
#pragma unroll 1
  for (int x = 0; x < count; ++x) {
    if (at.b != of_b || at.h != of_h) {  // the rows of another sequence or head
      of_b = at.b, of_h = at.h;
      len = seq_len(p, of_b);
      const int tiles = p.row_tiles[of_b + 1] - p.row_tiles[of_b];
      const long long row0 = static_cast<long long>(p.row_tiles[of_b]) * p.Hkv + static_cast<long long>(of_h) * tiles;
      two = tiles > 1;
      rows = p.rows + row0;
      score = p.score + (static_cast<long long>(of_b) * p.Hkv + of_h) * p.cap;
      all_lo = 0, all_hi = 0x7FFFFFFF;
#pragma unroll
      for (int f = 0; f < 2; ++f) {
#pragma unroll
        for (int j = 0; j < W; ++j) q[f][j] = p.frag[((row0 + (two ? f : 0)) * W + j) * 32 + lane];
        const Rows& r = rows[two ? f : 0];
        const int4 see = see_at(r, c4);
        w[f] = weights_at(r, c4);
        all_lo = max(all_lo, max(see.x, see.z)), all_hi = min(all_hi, min(see.y, see.w));
      }
      all_lo = __reduce_max_sync(0xFFFFFFFFu, all_lo);
      all_hi = __reduce_min_sync(0xFFFFFFFFu, all_hi);
    }
    const int t0 = (at.first + at.step) * kKeys, t = t0 + g + 8 * c4;
    const float old = next_old;
    copy_next();
    if (x + 1 < count) advance(at), next_old = old_at(at);
    cp_async_wait_group<kSlots - 1>();
    __syncwarp();
    const Slot<D>& s = ring[slot];
    slot = slot + 1 == kSlots ? 0 : slot + 1;
    const bool mask = t0 < all_lo || t0 + kKeys > all_hi;
    float mine;
    constexpr std::true_type yes{};
    constexpr std::false_type no{};
    if (mask) mine = two ? tile(yes, yes, s, t0) : tile(no, yes, s, t0);
    else mine = two ? tile(yes, no, s, t0) : tile(no, no, s, t0);
    if (t < len) score[t] = old + mine;
    __syncwarp();  // the slot has been read
  }
  cp_async_wait_group<0>();
}

// Sequences with more rows: a block takes 32 keys << K of a kv head; of its eight warps
// 1 << K have 32 keys each, the others the same keys and other row tiles, which are
// staged for all.  K is as large (and the rows are staged as seldom) as leaves every
// block two such steps: 32 sequences of 8192 keys and 64 rows, K = 0 / 1 / 2: 342 / 192 /
// 122 us.
template <int D>
struct Stage {
  static constexpr int kChunk = 2048 / D;  // row tiles at a time: 32 KB
  uint4 frag[2][kChunk][D / 32][32];
  Rows rows[2][kChunk];
  float sum[kThreads];
  int next;  // the step that the block takes
};

template <int D>
DEVINL void many_rows(const Params& p, Stage<D>& sh) {
  constexpr int W = D / 32, kChunk = Stage<D>::kChunk;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c4 = lane & 3;
  int K = 2;
  while (K > 0 && p.many[K * (p.B + 1) + p.B] * p.Hkv < 2 * static_cast<int>(gridDim.x)) --K;
  const long long* many = p.many + K * (p.B + 1);
  const int kg = warp & ((1 << K) - 1), rg = warp >> K, rgs = 8 >> K, block_keys = kKeys << K;
  const long long total = many[p.B] * p.Hkv;
  // steps differ in rows: a block takes the next one when it is through with its last
  for (long long x = blockIdx.x, next; x < total; x = next) {
    const int b = warp_find(p.B, x, [&](int i) { return many[i] * p.Hkv; });
    const int n = p.starts[b + 1] - p.starts[b], len = seq_len(p, b), steps = static_cast<int>(many[b + 1] - many[b]);
    const long long r0 = x - many[b] * p.Hkv;
    const int h = static_cast<int>(r0 / steps), step = static_cast<int>(r0 - static_cast<long long>(h) * steps);
    const int first = first_key(p, n, len), k0 = (first / block_keys + step) * block_keys, t0 = k0 + kKeys * kg;
    // row tiles with a query that sees one of the block's keys
    const int base = len - n, end = min(k0 + block_keys, len);  // place of the first query
    int i0 = 0, i1 = n - 1;
    if (p.causal) i0 = max(0, k0 - base);
    if (p.window > 0) i1 = static_cast<int>(min(static_cast<long long>(i1), static_cast<long long>(end) - 1 + p.window - 1 - base));
    const int f0 = i0 * p.G / 8, f1 = i1 < i0 ? f0 : (i1 * p.G + p.G + 7) / 8;
    // of them, those whose rows all see all of the warp's keys
    int u0 = 0, u1 = n - 1;
    if (p.causal) u0 = max(0, t0 + kKeys - 1 - base);
    if (p.window > 0) u1 = static_cast<int>(min(static_cast<long long>(u1), static_cast<long long>(t0) + p.window - 1 - base));
    const bool some = u0 <= u1 && t0 + kKeys <= len;
    const int g0 = some ? (u0 * p.G + 7) / 8 : f1, g1 = some ? (u1 + 1) * p.G / 8 : f1;
    const int tiles = p.row_tiles[b + 1] - p.row_tiles[b];
    const long long row0 = static_cast<long long>(p.row_tiles[b]) * p.Hkv + static_cast<long long>(h) * tiles;
    auto stage = [&](int f, int to) {
      const int m = min(kChunk, f1 - f);
      const uint4* from = p.frag + (row0 + f) * (W * 32);
      uint4* frag = &sh.frag[to][0][0][0];
      for (int i = threadIdx.x; i < m * W * 32; i += kThreads) cp_async<D>(frag + i, from + i);
      constexpr int R = sizeof(Rows) / 16;
      static_assert(kChunk * R <= kThreads, "a copy per thread");
      if (static_cast<int>(threadIdx.x) < m * R)
        cp_async<D>(reinterpret_cast<uint4*>(sh.rows[to]) + threadIdx.x, reinterpret_cast<const uint4*>(p.rows + row0 + f) + threadIdx.x);
      cp_async_commit();
    };
    if (f0 < f1) stage(f0, 0);
    // keys in front of the first that any query sees may have no page any more
    const bool active = t0 < len && t0 + kKeys > first;
    Expanded e[2][W];
    if (active) {
      const uint8_t* rec = record_of<D>(p, p.table[static_cast<long long>(b) * p.max_pages + (t0 >> p.P_log2)], h);
      Keys<D> keys[2];
#pragma unroll
      for (int a = 0; a < 2; ++a) load_keys<D>(p, rec, (t0 & (p.P - 1)) + 16 * a, keys[a]);
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        const uint32_t s0 = e4m3x2_to_f16x2(keys[a].s[0]), s1 = e4m3x2_to_f16x2(keys[a].s[1]);
#pragma unroll
        for (int j = 0; j < W; ++j) e[a][j] = expand_word<D>(keys[a], j, s0, s1);
      }
    }
    float sum[2][2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
    for (int f = f0, to = 0; f < f1; f += kChunk, to ^= 1) {
      if (f + kChunk < f1) {
        stage(f + kChunk, to ^ 1);
        cp_async_wait_group<1>();
      } else {
        cp_async_wait_group<0>();
      }
      __syncthreads();
      if (active) {
        const int m = min(kChunk, f1 - f);
        // tiles [lo, hi) of the chunk without masks, two at a time; the others with them
        auto products = [&](int i, int step, auto two_tiles, float (&acc)[2][2][4]) {
          constexpr int F = decltype(two_tiles)::value ? 2 : 1;
#pragma unroll
          for (int f = 0; f < F; ++f)
#pragma unroll
            for (int a = 0; a < 2; ++a) acc[f][a][0] = acc[f][a][1] = acc[f][a][2] = acc[f][a][3] = 0.0f;
#pragma unroll
          for (int j = 0; j < W; ++j) {
            uint4 v[F];
#pragma unroll
            for (int f = 0; f < F; ++f) v[f] = sh.frag[to][i + f * step][j][lane];
#pragma unroll
            for (int f = 0; f < F; ++f)
#pragma unroll
              for (int a = 0; a < 2; ++a) mma_half<0>(acc[f][a], e[a][j], v[f]);
#pragma unroll
            for (int f = 0; f < F; ++f)
#pragma unroll
              for (int a = 0; a < 2; ++a) mma_half<1>(acc[f][a], e[a][j], v[f]);
          }
        };
        const int lo = max(0, g0 - f), hi = min(m, g1 - f);
        for (int i = rg; i < m; i += rgs) {
          float acc[2][2][4];
          if (i >= lo && i + rgs < hi) {
            products(i, rgs, std::true_type{}, acc);
            const float4 w0 = weights_at(sh.rows[to][i], c4), w1 = weights_at(sh.rows[to][i + rgs], c4);
#pragma unroll
            for (int a = 0; a < 2; ++a) add_weights(sum[a], acc[0][a], w0);
#pragma unroll
            for (int a = 0; a < 2; ++a) add_weights(sum[a], acc[1][a], w1);
            i += rgs;
          } else {
            products(i, 0, std::false_type{}, acc);
            const float4 w = weights_at(sh.rows[to][i], c4);
            const int4 see = see_at(sh.rows[to][i], c4);
#pragma unroll
            for (int a = 0; a < 2; ++a) add_weights(sum[a], acc[0][a], w, see, t0 + 16 * a + g);
          }
        }
      }
      __syncthreads();  // the chunk has been read
    }
    const float mine = quad_sums(sum);
    const int at = kKeys * kg + g + 8 * c4;
    if (rg > 0) sh.sum[rg * block_keys + at] = mine;
    if (threadIdx.x == 0) sh.next = atomicAdd(p.taken, 1);
    __syncthreads();
    next = static_cast<long long>(gridDim.x) + sh.next;
    if (rg == 0 && k0 + at < len) {
      float v = mine, *s = p.score + (static_cast<long long>(b) * p.Hkv + h) * p.cap + k0 + at;
      for (int r = 1; r < rgs; ++r) v += sh.sum[r * block_keys + at];
      // keys that the step wrote itself have no older sum
      *s = (k0 + at < len - n ? *s : 0.0f) + v;
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------ sequences of more rows
// tcgen05: S^T = K Q^T, 128 keys on M, 128 rows on N.  A thread has a key: its weights
// are summed up in a register, and which rows see it is a range of them.  The roles of
// a block, by warp:
//
//   0-3, 4-7  sums, each four of every other tile of rows, with two accumulators of 128
//             columns
//   8         bulk copies of tiles of rows and of what their columns need
//   9, 10     issue the matrix instructions for the first and the second four: what one
//             waits for is hidden under the other's (one for both 1150 against 878 us on the long chunk)
//   11        takes items (sequence, kv head, keys) and publishes them, one ahead
//   12-15     expand the next item's keys into the swizzle that the instructions read
//
// Which tile is whose goes by the count of tiles over all items, not by the place in an
// item: a slot of the rings of tiles and of columns then has the same reader for good, who
// waits for each of its uses.  (A reader that left one out could find the barrier in the
// phase before, which has the parity that it waits for, and read what has not come.)
//
// Bound: a tile of 128 x 128 scores takes its products 710 cycles and its four warps 990
// (the exponentials; two fours, so 500); items end and begin.  256 keys to an item,
// which halves the rows' way from L2, was slower (1169 against 878 us on the long chunk).
constexpr int kTileThreads = 512, kCopy = 8, kIssue = 9, kWalk = 11, kExpand = 12, kItemReaders = 8 + 3 + 4;
// What a tile's columns need is read until it is summed up, after its product: two of each four
// warps' accumulators later.
constexpr int kColumnSlots = 16;
template <int D>
struct TileCfg {
  static constexpr int SUB = 128 * 128;             // 64 values of 128 keys or rows
  static constexpr int TILE = 128 * D * 2;          // of keys or rows
  static constexpr int STAGES = D == 128 ? 4 : 8;   // tiles of rows in flight
  static_assert(STAGES % 2 == 0 && kColumnSlots % 2 == 0, "a slot has one reader");
  static constexpr int Q0 = 2 * TILE;               // behind two items' keys
  static constexpr int COLUMNS0 = Q0 + STAGES * TILE;
  static constexpr int COLUMNS = 16 * static_cast<int>(sizeof(Columns));
  static constexpr int BARS0 = COLUMNS0 + kColumnSlots * COLUMNS;
};
struct TileBars {
  uint64_t qfull[8], qempty[8], cfull[kColumnSlots], kfull[2], kempty[2], sfull[4], sempty[4], done;
  ItemRing items;
  float sum[2][128];
  uint32_t tmem;
  int abort, last;
};
// Parts that an item comes in at most: so many that there are six to a block or more, if
// each has kPartTiles tiles of rows.  Their sums join in the order of the rows.  (4096
// queries on 12289 keys, 384 items of up to 512 tiles: 823 us whole, 670 in three parts;
// 325 items of some 16 tiles 41 us whole, 43.5 in two.)
constexpr int kPartTiles = 16;
DEVINL int most_parts(const Params& p, long long items) {
  return items >= p.split ? 1 : min(kParts, static_cast<int>((p.split + items - 1) / max(items, 1ll)));
}

template <int D>
__global__ void __launch_bounds__(kTileThreads, 1) weights_tiles_kernel(const Params p) {
  using C = TileCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_tiles[];
  uint8_t* const smem = smem_tiles;
  const uint32_t sk = smem_u32(smem);
  TileBars& bars = *reinterpret_cast<TileBars*>(smem + C::BARS0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t polls = polls_of(p.timeout_ns);
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&bars.qfull[i], 1);
      mbar_init(&bars.qempty[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bars.sfull[i], 1);
      mbar_init(&bars.sempty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.kfull[i], 4);
      mbar_init(&bars.kempty[i], 2);
    }
    for (int i = 0; i < kColumnSlots; ++i) mbar_init(&bars.cfull[i], 1);
    mbar_init(&bars.done, 2);
    item_ring_init(bars.items, kItemReaders);
    bars.abort = 0;
    fence_mbar_init();
  }
  if (warp == kIssue) {
    tmem_alloc(&bars.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem;
  wait_for_previous();
  int* const abort = &bars.abort;

  if (warp < kCopy) {
    // ==================================================================== sums
    const int grp = warp >> 2, in = (warp & 3) * 32 + lane;
    const uint32_t ts = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + grp * 256;
    ItemReader items;
    uint32_t uses = 0;    // of the four warps' accumulators
    uint32_t stage0 = 0;  // tiles of rows of the items so far
    for (int i = 0;; ++i) {
      const Item it = items.next(bars.items, polls, p.err, abort);
      if (named_bar_red_or(1, 256, it.n == 0)) break;  // all eight together
      const int key = it.u + in, base = it.len - it.nq;
      float* score = p.score + (static_cast<long long>(it.b) * p.Hkv + it.h) * p.cap + key;
      bool mine = grp == 0 && key < it.len;
      const float old = mine && key < base ? *score : 0.0f;  // keys that the step wrote itself have no older sum
      // rows [lo, hi) see the key
      int lo = 0, hi = key < it.len ? it.nq * p.G : 0;
      if (p.causal && hi > 0) lo = max(0, key - base) * p.G;
      if (p.window > 0 && hi > 0)
        hi = static_cast<int>(max(0ll, min(static_cast<long long>(it.nq), static_cast<long long>(key) + p.window - base))) * p.G;
      uint64_t sum[2] = {0, 0};
      for (int f = static_cast<int>((stage0 + grp) & 1); f < it.n; f += 2, ++uses) {
        const int buf = 2 * grp + (uses & 1), r0 = (it.q0 + f) * 128;
        const uint32_t stage = stage0 + f, slot = stage % kColumnSlots;
        const Columns* c = reinterpret_cast<const Columns*>(smem + C::COLUMNS0 + slot * C::COLUMNS);
        wait_warp(&bars.cfull[slot], (stage / kColumnSlots) & 1, polls, p.err, abort);
        wait_warp(&bars.sfull[buf], uses >> 1 & 1, polls, p.err, abort);
        tc_fence_after();
        const uint32_t at = ts + (uses & 1) * 128;
        // sixteen columns at a time, the next ones' loads in flight; where some key is not
        // seen by all of the rows, each column with a test
        auto add_all = [&](auto masked) {
          constexpr bool MASK = decltype(masked)::value;
          const int from = lo - r0, to = hi - r0;
          uint32_t v[2][16];
          ulonglong2 sc[2][4], nl[2][4];
          auto load = [&](int q) {
            tmem_ld_32x32b_x16(at + 16 * q, v[q & 1]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              sc[q & 1][j] = *reinterpret_cast<const ulonglong2*>(&c[2 * q + j / 2].sc[4 * (j & 1)]);
              nl[q & 1][j] = *reinterpret_cast<const ulonglong2*>(&c[2 * q + j / 2].less_lse2[4 * (j & 1)]);
            }
          };
          load(0);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            tmem_ld_wait();
            if (q < 7) load(q + 1);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t* w = &v[q & 1][4 * j];
              float x[4];
              unpair(fma2(pair(__uint_as_float(w[0]), __uint_as_float(w[1])), sc[q & 1][j].x, nl[q & 1][j].x), x[0], x[1]);
              unpair(fma2(pair(__uint_as_float(w[2]), __uint_as_float(w[3])), sc[q & 1][j].y, nl[q & 1][j].y), x[2], x[3]);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                x[e] = ex2(x[e]);
                if (MASK && (16 * q + 4 * j + e < from || 16 * q + 4 * j + e >= to)) x[e] = 0.0f;
              }
              sum[0] = add2(sum[0], pair(x[0], x[1]));
              sum[1] = add2(sum[1], pair(x[2], x[3]));
            }
          }
        };
        if (__all_sync(0xFFFFFFFFu, lo <= r0 && hi >= r0 + 128)) add_all(std::false_type{});
        else if (__any_sync(0xFFFFFFFFu, lo < r0 + 128 && hi > r0)) add_all(std::true_type{});
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.sempty[buf]);
      }
      stage0 += it.n;
      float s0, s1;
      unpair(add2(sum[0], sum[1]), s0, s1);
      float all = s0 + s1;
      if (grp == 1) bars.sum[i & 1][in] = all;
      named_bar_sync(1, 256);
      if (grp == 0) {
        all += bars.sum[i & 1][in];
        const int parts = it.slot & 15;
        if (parts > 1) {  // the item's last part to be summed up adds them all
          const int item = it.slot >> 8;
          float* part = p.part + static_cast<long long>(item) * (kParts * kTileKeys) + in;
          __stcg(part + (it.slot >> 4 & 15) * kTileKeys, all);
          __threadfence();
          named_bar_sync(2, 128);
          if (in == 0) bars.last = atomicAdd(p.parts_done + item, 1) == parts - 1;
          named_bar_sync(2, 128);
          mine = mine && bars.last;
          __threadfence();
          all = 0.0f;
          if (mine)
            for (int k = 0; k < parts; ++k) all += __ldcg(part + k * kTileKeys);
        }
        if (mine) *score = old + all;
      }
    }
  } else if (warp == kCopy) {
    // ==================================================================== copies
    ItemReader items;
    uint32_t uses = 0, turn = 0;  // tiles of rows; parity of the stages' ring
    int st = 0;
    bool gone = false;
    while (!gone) {
      const Item it = items.next(bars.items, polls, p.err, abort);
      if (it.n == 0) break;
      const uint8_t* from = reinterpret_cast<const uint8_t*>(p.frag) + static_cast<long long>(it.row0) * (16 * D);
      const Columns* columns = reinterpret_cast<const Columns*>(p.rows + it.row0);
      for (int f = 0; f < it.n; ++f, ++uses) {
        if (uses >= C::STAGES) wait_warp(&bars.qempty[st], turn ^ 1, polls, p.err, abort);
        gone = given_up(abort);
        if (gone) break;
        const int t0 = (it.q0 + f) * 16, m = min(16, it.rows - t0);
        if (lane == 0) {
          const int slot = uses % kColumnSlots;
          mbar_arrive_expect_tx(&bars.qfull[st], m * 16 * D);
#pragma unroll
          for (int k = 0; k < D / 64; ++k)
            bulk_load(smem + C::Q0 + st * C::TILE + k * C::SUB, from + (static_cast<long long>(k) * it.rows + t0) * 1024, m * 1024,
                      &bars.qfull[st]);
          mbar_arrive_expect_tx(&bars.cfull[slot], m * static_cast<int>(sizeof(Columns)));
          bulk_load(smem + C::COLUMNS0 + slot * C::COLUMNS, columns + t0, m * static_cast<int>(sizeof(Columns)), &bars.cfull[slot]);
        }
        __syncwarp();
        if (++st == C::STAGES) st = 0, turn ^= 1;
      }
    }
    // no block ends with bytes on their way to its shared memory: the last uses of all slots
    // (an older tile's columns may be on their way still where the sums were given up)
    for (uint32_t u = uses > C::STAGES ? uses - C::STAGES : 0; u < uses; ++u)
      mbar_wait_warp(&bars.qfull[u % C::STAGES], (u / C::STAGES) & 1, kLandNs, p.err, nullptr);
    for (uint32_t u = uses > kColumnSlots ? uses - kColumnSlots : 0; u < uses; ++u)
      mbar_wait_warp(&bars.cfull[u % kColumnSlots], (u / kColumnSlots) & 1, kLandNs, p.err, nullptr);
  } else if (warp < kWalk) {
    // ======================================================= matrix instructions
    const int grp = warp - kIssue;
    const uint64_t dk = smem_desc_kmajor_sw128(sk), dq = smem_desc_kmajor_sw128(sk + C::Q0);
    ItemReader items;
    uint32_t turn = 0, uses = 0;
    int st = 0;  // its parity is that of the count of tiles
    bool gone = false;
    for (uint32_t i = 0; !gone; ++i) {
      const Item it = items.next(bars.items, polls, p.err, abort);
      if (it.n == 0) break;
      const int kb = i & 1;
      wait_warp(&bars.kfull[kb], i >> 1 & 1, polls, p.err, abort);
      for (int f = 0; f < it.n && !gone; ++f) {
        if ((st & 1) == grp) {
          const int buf = 2 * grp + (uses & 1);
          wait_warp(&bars.qfull[st], turn, polls, p.err, abort);
          if (uses >= 2) wait_warp(&bars.sempty[buf], ((uses >> 1) - 1) & 1, polls, p.err, abort);
          gone = given_up(abort);
          if (gone) break;
          tc_fence_after();
          const uint64_t a = dk + kb * (C::TILE >> 4), b = dq + st * (C::TILE >> 4);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint64_t o = (kk >> 2) * (C::SUB >> 4) + (kk & 3) * 2;
              umma_f16(tmem + buf * 128, a + o, b + o, idesc_f16_f32(128, 128), kk ? 1u : 0u);
            }
            umma_commit(&bars.sfull[buf]);
            umma_commit(&bars.qempty[st]);
          }
          __syncwarp();
          ++uses;
        }
        if (++st == C::STAGES) st = 0, turn ^= 1;
      }
      if (!gone) umma_commit_warp(&bars.kempty[kb]);
    }
    umma_commit_warp(&bars.done);
    mbar_wait_warp(&bars.done, 0, kLandNs, p.err, nullptr);
  } else if (warp == kWalk) {
    // ====================================================================== walk
    // all items' first parts, then the second ones: those are not there where an item has fewer
    const long long items = p.big[p.B] * p.Hkv;
    const int most = most_parts(p, items);
    const long long total = items * most;
    ItemWriter out;
    for (long long x = blockIdx.x;;) {
      Item t{};
      if (x < total) {
        const int mine = static_cast<int>(x / items);
        const long long item = x - mine * items;
        const int b = warp_find(p.B, item, [&](int i) { return p.big[i] * p.Hkv; });
        const int n = p.starts[b + 1] - p.starts[b], len = seq_len(p, b), steps = static_cast<int>(p.big[b + 1] - p.big[b]);
        const long long r0 = item - p.big[b] * p.Hkv;
        t.b = b, t.h = static_cast<int>(r0 / steps);
        t.u = (first_key(p, n, len) / kTileKeys + static_cast<int>(r0 - static_cast<long long>(t.h) * steps)) * kTileKeys;
        t.nq = n, t.len = len, t.rows = p.row_tiles[b + 1] - p.row_tiles[b];
        t.row0 = p.row_tiles[b] * p.Hkv + t.h * t.rows;
        // tiles of rows that see one of the keys: there is one, the steps begin with the first key that any sees
        const int base = len - n, end = min(t.u + kTileKeys, len);
        const int i0 = p.causal ? max(0, t.u - base) : 0;
        const int i1 = p.window > 0 ? static_cast<int>(min(n - 1ll, static_cast<long long>(end) + p.window - 2 - base)) : n - 1;
        t.q0 = i0 * p.G / 128;
        t.n = (i1 * p.G + p.G + 127) / 128 - t.q0;
        const int parts = max(1, min(most, t.n / kPartTiles)), each = (t.n + parts - 1) / parts;
        t.slot = parts > 1 ? static_cast<int>(item) << 8 | mine << 4 | (t.n + each - 1) / each : 1;
        t.q0 += mine * each, t.n = min(each, t.n - mine * each);
      }
      if (x >= total || t.n > 0) {
        out.put(bars.items, t, polls, p.err, abort);
        if (t.n == 0 || given_up(abort)) break;
        // the next one when all have begun with this one, so that the blocks end together
        wait_warp<true>(&bars.items.empty[(out.i - 1) & (kItems - 1)], ((out.i - 1) / kItems) & 1, polls, p.err, abort);
      }
      x = static_cast<long long>(gridDim.x) + __shfl_sync(0xFFFFFFFFu, lane == 0 ? atomicAdd(p.taken + 1, 1) : 0, 0);
    }
  } else if (warp >= kExpand) {
    // ==================================================================== expand
    constexpr int W = D / 32;  // words of codes of a lane and key
    const int c4 = lane & 3, in32 = 8 * (warp & 3) + (lane >> 2);
    const bool up = W == 4 && (c4 & 2);
    ItemReader items;
    for (uint32_t i = 0;; ++i) {
      const Item it = items.next(bars.items, polls, p.err, abort);
      if (it.n == 0) break;
      const int kb = i & 1, first = first_key(p, it.nq, it.len);
      const int32_t* table = p.table + static_cast<long long>(it.b) * p.max_pages;
      uint32_t cw[4][W], sb[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int t0 = it.u + 32 * k;
        sb[k] = 0;
#pragma unroll
        for (int q = 0; q < W; ++q) cw[k][q] = 0;
        // keys in front of the first that any query sees may have no page any more
        if (t0 >= it.len || t0 + 32 <= first) continue;
        const uint8_t* rec = record_of<D>(p, __ldg(table + (t0 >> p.P_log2)), it.h);
        const int off = (t0 + in32) & (p.P - 1);
        if (W == 4) {
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(rec + off * (D / 2) + 16 * c4));
          cw[k][0] = v.x, cw[k][1] = v.y, cw[k][2 % W] = v.z, cw[k][3 % W] = v.w;
          sb[k] = __ldg(reinterpret_cast<const uint16_t*>(rec + codes_bytes(p.P, D) + off * (D / 16) + 2 * c4));
        } else {
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(rec + off * (D / 2) + 8 * c4));
          cw[k][0] = v.x, cw[k][1] = v.y;
          sb[k] = __ldg(rec + codes_bytes(p.P, D) + off * (D / 16) + c4);
        }
      }
      if (i >= 2) wait_warp(&bars.kempty[kb], ((i >> 1) - 1) & 1, polls, p.err, abort);
      const uint32_t row = sk + kb * C::TILE + (W == 4 ? (c4 >> 1) * C::SUB : 0) + in32 * 128;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t f = e4m3x2_to_f16x2(sb[k]);
        // lanes 2, 3 of a key write their pieces in another order: no two of a phase on the same banks
        const uint32_t f0 = __byte_perm(f, f, up ? 0x3232 : 0x1010), f1 = __byte_perm(f, f, up ? 0x1010 : 0x3232);
#pragma unroll
        for (int q = 0; q < W; ++q) {
          uint32_t x[4];
          e2m1x8(up ? cw[k][(q ^ 2) % W] : cw[k][q], x);
          const int unit = W == 4 ? 4 * (c4 & 1) + (q ^ (c4 & 2)) : 2 * c4 + q;
          const uint32_t fq = W == 4 && q >= 2 ? f1 : f0;
          st_shared_v4(row + k * 32 * 128 + ((unit ^ (in32 & 7)) << 4), hmul2(x[0], fq), hmul2(x[1], fq), hmul2(x[2], fq),
                       hmul2(x[3], fq));
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.kfull[kb]);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kIssue) tmem_dealloc(tmem, 512);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2) weights_kernel(const Params p) {
  extern __shared__ __align__(16) uint8_t smem[];
  launch_dependents();
  wait_for_previous();
  few_rows<D>(p, reinterpret_cast<Slot<D>*>(smem) + (threadIdx.x >> 5) * kSlots);
  __syncthreads();
  many_rows<D>(p, *reinterpret_cast<Stage<D>*>(smem));
}

// The tiles' kernel is a launch more: where many rows are left beside a few for every
// sequence.  (Not with so many rows that a wait for an item's keys would run out.)
int tile_rows_of(int T, int B, int G) {
  const long long rows = static_cast<long long>(T) * G;
  return rows >= kTileRows + 64ll * B && rows <= (1 << 26) ? kTileRows : INT_MAX;
}

// No more rows than a warp holds in all: each block prepares them for itself, where the
// workspace would be in its shared memory, a launch less (one query on 700 keys with the
// call 17.4 against 19.4 us).
constexpr int kSmallSmem = 100 * 1024;
constexpr uintptr_t kCarved = 256;  // where the host has it carved from (from null there are no places)
template <int D>
__global__ void __launch_bounds__(kThreads, 2) weights_small_kernel(Params p, int sums_at) {
  extern __shared__ __align__(256) uint8_t smem_small[];
  static_assert(kThreads == kPrepThreads, "the same warps");
  uint8_t* const ws = smem_small + ring_bytes<D>();
  auto place = [&](auto*& x) { x = reinterpret_cast<std::remove_reference_t<decltype(x)>>(ws + (reinterpret_cast<uintptr_t>(x) - kCarved)); };
  place(p.starts), place(p.row_tiles), place(p.few), place(p.many), place(p.big), place(p.taken), place(p.rows), place(p.frag);
  prepare<D>(p, 0, 1, reinterpret_cast<int*>(ws + sums_at));
  __syncthreads();
  few_rows<D>(p, reinterpret_cast<Slot<D>*>(smem_small) + (threadIdx.x >> 5) * kSlots);
}

size_t carve(Params& p, void* ws, int T, int B, int G, int Hkv, int D) {
  Carve c(ws, 0);
  const long long tiles = ((static_cast<long long>(T) * G + 7) / 8 + B) * Hkv;
  p.starts = c.take<int>(B + 1);
  p.row_tiles = c.take<int>(B + 1);
  p.few = c.take<long long>(B + 1);
  p.taken = c.take<int>(2);
  p.many = c.take<long long>(3 * static_cast<size_t>(B + 1));
  p.big = c.take<long long>(B + 1);
  p.tile_rows = tile_rows_of(T, B, G);
  p.split = p.tile_rows == INT_MAX ? 0 : 6 * num_sms();
  p.parts_done = c.take<int>(p.split);
  p.part = c.take<float>(static_cast<size_t>(p.split) * kParts * kTileKeys);
  p.rows = c.take<Rows>(tiles);
  p.frag = c.take<uint4>(tiles * (D / 32) * 32);
  return c.used;
}

template <int D>
int launch(const Params& p, cudaStream_t s) {
  if (p.T * static_cast<long long>(p.G) <= kFewRows) {
    Params q = p;
    const size_t used = carve(q, reinterpret_cast<void*>(kCarved), p.T, p.B, p.G, p.Hkv, D), sums = 2 * (p.B + 1) * sizeof(int);
    const size_t bytes = ring_bytes<D>() + used + sums;
    if (bytes <= kSmallSmem) {
      static std::atomic<bool> small_set[64];
      MOE_TRY(allow_smem(weights_small_kernel<D>, kSmallSmem, small_set));
      weights_small_kernel<D><<<num_sms() * 2, kThreads, bytes, s>>>(q, static_cast<int>(used));
      return check_launch();
    }
  }
  static std::atomic<bool> set[64];
  const int smem = 2 * (p.B + 1) * static_cast<int>(sizeof(int));
  MOE_TRY(allow_smem(weights_prepare_kernel<D>, 2 * (kMaxRows + 1) * static_cast<int>(sizeof(int)), set));
  const long long tiles = ((static_cast<long long>(p.T) * p.G + 7) / 8 + p.B) * p.Hkv;
  const int per = kPrepThreads / 32;
  const int blocks = static_cast<int>(std::min<long long>((tiles + per - 1) / per, num_sms() * 4));
  weights_prepare_kernel<D><<<blocks, kPrepThreads, smem, s>>>(p);
  MOE_TRY(check_launch());
  static std::atomic<bool> main_set[64];
  constexpr int bytes = std::max(static_cast<int>(sizeof(Stage<D>)), ring_bytes<D>());
  MOE_TRY(allow_smem(weights_kernel<D>, bytes, main_set));
  MOE_TRY(launch_after(weights_kernel<D>, dim3(num_sms() * 2), kThreads, bytes, s, p));
  if (p.tile_rows == INT_MAX) return MOE_OK;
  static std::atomic<bool> tiles_set[64];
  constexpr int smem_tiles = TileCfg<D>::BARS0 + sizeof(TileBars);
  MOE_TRY(allow_smem(weights_tiles_kernel<D>, smem_tiles, tiles_set));
  return launch_after(weights_tiles_kernel<D>, dim3(num_sms()), kTileThreads, smem_tiles, s, p);
}

bool shapes_ok(int T, int B, int Hq, int Hkv, int D) {
  return T >= 0 && B >= 0 && Hkv >= 1 && Hq >= 1 && Hq % Hkv == 0 && head_dim_ok(D);
}

}  // namespace
}  // namespace kv4
}  // namespace moe

using namespace moe;

extern "C" size_t moe_kv4_weights_workspace_size(int T, int B, int Hq, int Hkv, int D) {
  if (!kv4::shapes_ok(T, B, Hq, Hkv, D) || T == 0 || B == 0) return 0;
  kv4::Params p;
  return kv4::carve(p, nullptr, T, B, Hq / Hkv, Hkv, D);
}

extern "C" int moe_kv4_weights(const uint16_t* q, long long q_stride, int T, int Hq, const uint8_t* pool, int num_pages,
                               int page_size, int Hkv, int D, const float* g_k, const float* lse,
                               const int32_t* q_offsets, const int32_t* kv_lens, const int32_t* table, int B,
                               int max_pages, float scale, int causal, int window, float* score, int cap, void* ws,
                               size_t ws_bytes, void* stream) {
  using namespace kv4;
  if (T < 0 || B < 0 || window < 0 || (window > 0 && !causal)) return MOE_ERR_INVALID_ARG;
  if (!shapes_ok(T, B, Hq, Hkv, D) || !page_size_ok(page_size)) return MOE_ERR_UNSUPPORTED;
  if (T == 0 || B == 0) return MOE_OK;
  if (max_pages < 1 || num_pages < 1 || cap < static_cast<long long>(max_pages) * page_size) return MOE_ERR_INVALID_ARG;
  // places and rows are held in 32 bits
  if (B > kMaxRows || static_cast<long long>(max_pages) * page_size > (1 << 30) || static_cast<long long>(T) * Hq >= (1 << 29))
    return MOE_ERR_UNSUPPORTED;
  if (!q || !pool || !g_k || !lse || !q_offsets || !kv_lens || !table || !score || !ws) return MOE_ERR_INVALID_ARG;
  if (!aligned(q, 16) || q_stride % 8 != 0 || (T > 1 && q_stride < static_cast<long long>(Hq) * D) || !aligned(pool, 16) ||
      !aligned(g_k, 4) || !aligned(lse, 4) || !aligned(q_offsets, 4) || !aligned(kv_lens, 4) || !aligned(table, 4) ||
      !aligned(score, 4) || !aligned(ws, 256))
    return MOE_ERR_INVALID_ARG;
  if (window >= max_pages * page_size) window = 0;  // reaches past the first key from anywhere
  Params p{q, q_stride, pool, g_k, lse, q_offsets, kv_lens, table, score, T, B, Hq, Hkv, Hq / Hkv, num_pages, page_size,
           page_size == 32 ? 5 : page_size == 64 ? 6 : 7, max_pages, causal != 0, window, cap, scale};
  if (ws_bytes < carve(p, ws, T, B, p.G, Hkv, D)) return MOE_ERR_WORKSPACE;
  p.err = device_error_word();
  if (!p.err) return MOE_ERR_CUDA;
  p.timeout_ns = wait_timeout_ns();
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return D == 128 ? launch<128>(p, s) : launch<64>(p, s);
}
