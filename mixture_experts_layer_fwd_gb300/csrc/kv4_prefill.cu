// Attention over the paged NVFP4 cache, 256 query rows at a time: two tiles A
// and B of 128 rows share every 128 keys (chunks of prompts, or a few tokens
// of many heads; an item of up to 128 rows uses tile A alone).
//
// Bound: the tensor cores, 4 * 128 * D multiply-adds per row and tile of keys,
// then the exponentials.  One block per SM; the roles, by warp:
//
//   0-7, 8-15 softmax of tile A / B, half a row per thread: S from tensor
//             memory, running maximum and sum, P (fp16) back over S's columns
//   16-19     expand the codes of K, 20-23 those of V, both as [key][d], fp16 in
//             the swizzle the matrix instructions read (V with d contiguous)
//   24        bulk copies of the halves (keys, values) of page records
//   25, 26    issue the matrix instructions of tile A / B
//   27        walks the block's items and publishes them to the others
//
// S = Q K^T comes from shared memory, O += P V takes P from tensor memory.  One
// tile's softmax runs under the other's products, and so does the time from a
// barrier to the first instruction after it (about 450 cycles: with one warp
// issuing for both tiles it came four times per tile of keys).  S and O fill tensor
// memory: 2 x 128 + 2 x D columns; P lies over its S, each half row over its own.
//
// The running maximum is moved only when a row's grows by more than 2^kSlack:
// until then O needs no rescaling, and P keeps fp16's relative precision.
// Numbers are as in the 16-row kernel: codes times block scales and Q times a
// power of two are exact in fp16, P is rounded to fp16, sums are fp32.
//
// 4096 queries on 12289 keys, 64 heads on 4 of 128: 0.96 ms, 1.43 PFLOP/s; the
// same with heads of 64 0.83 ms.  What bounds it is the chain scores, softmax,
// weights, next scores of a tile, since scores and weights share columns.  Half
// a row per thread 1.17 against 1.21 ms, one tester of a barrier for the eight
// warps of a tile 1.09 against 1.13, walking the items in a warp of its own
// (half the code) 1.39 against 2.12; with heads of 64 P has room beside S, but
// without turns the tiles fall into step: 1.02 against 0.88.
#include "kv4_attention.cuh"

namespace moe {
namespace kv4 {
namespace {

constexpr int kRows = kRowsTile;
constexpr int kKeys = 128;
constexpr int kThreads = 896;  // at 72 registers; shared out as 512 x 88, 256 x 56, 128 x 40
constexpr int kMaxSlots = 16;
constexpr int kSoftmax = 16, kExpandV = 20, kLoad = 24, kMma = 25, kWalk = 27;
constexpr int kReaders = 16 + 8 + 3;

template <int D>
struct Cfg {
  static constexpr int Q_BYTES = 128 * D * 2;     // one row tile
  static constexpr int K_BYTES = kKeys * D * 2;   // one tile of keys; V the same
  static constexpr int SUB_Q = 128 * 128;         // 64-wide sub-tile of Q, K or V
  static constexpr int BARS0 = 2 * Q_BYTES + 4 * K_BYTES;
  static constexpr int RING0 = BARS0 + 3328;
  static constexpr int RING = (D == 128 ? 227 : 160) * 1024 - RING0;
};

struct Bars {
  uint64_t full[2][kMaxSlots], empty[2][kMaxSlots];  // rings of key and of value halves
  uint64_t kfull[2], kempty[2], vfull[2], vempty[2];
  uint64_t qfull[2], sfull[2], pfull[2], ofull[2], turn[2], done;
  ItemRing items;
  float swap[2][2][128];  // between the two threads of a row: [tile][half][row]
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(Bars) <= 3328, "between the operand tiles and the ring");

// Half h of a query row to fp16 in the swizzled tile, read in one round trip;
// the two threads of a row exchange their largest magnitudes.  Returns the
// softmax scale of the row in log2 units (> 0).
template <int D>
DEVINL float load_q(const AttnParams& p, const Item& t, int idx, int r, int h, uint32_t tile, float* give,
                    const float* take, int pair_bar) {
  constexpr int N = D / 16;  // 16-byte pieces of half a row
  uint4 v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = make_uint4(0, 0, 0, 0);
  if (idx < t.nq * p.G) {
    const int tok = idx / p.G;
    const uint4* src = reinterpret_cast<const uint4*>(p.q + (t.q0 + tok) * p.q_stride + (t.h * p.G + idx - tok * p.G) * D) +
                       h * N;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __ldg(src + i);
  }
  const float gk = __ldg(p.g_k + t.h);
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
    for (int q = 0; q < 4; ++q) top = max(top, max(w[q] & 0x7FFFu, (w[q] >> 16) & 0x7FFFu));
  }
  *give = __uint_as_float(top);
  named_bar_sync(pair_bar, 64);
  top = max(top, __float_as_uint(*take));
  named_bar_sync(pair_bar, 64);  // both have read before either writes again
  float up, sc;
  row_scale(p.scale * gk, top, up, sc);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
    uint32_t x[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
      x[q] = pack_f16x2(__uint_as_float(w[q] << 16) * up, __uint_as_float(w[q] & 0xFFFF0000u) * up);
    const int c = h * N + i;  // piece of the row
    st_shared_v4(tile + (c >> 3) * Cfg<D>::SUB_Q + r * 128 + (((c & 7) ^ (r & 7)) << 4), x[0], x[1], x[2], x[3]);
  }
  return sc;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attn_tiles_kernel(const AttnParams p, int k_slots, int v_slots) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // 1024-byte aligned operand tiles: Q_A Q_B | K0 K1 | V0 V1 | barriers | ring of record halves
  const uint32_t base = smem_u32(smem_raw);
  const uint32_t sq = base, sk = base + 2 * C::Q_BYTES, sv = sk + 2 * C::K_BYTES;
  Bars& bars = *reinterpret_cast<Bars*>(smem_raw + C::BARS0);
  uint8_t* ring = smem_raw + C::RING0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int half = record_bytes(p.P, D) / 2, pages = kKeys / p.P;
  const uint32_t polls = polls_of(p.timeout_ns);
  const int slots[2] = {k_slots, v_slots};

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2 * kMaxSlots; ++i) {
      mbar_init(&bars.full[0][i], 1);
      mbar_init(&bars.empty[0][i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.kfull[i], 4);
      mbar_init(&bars.kempty[i], 2);
      mbar_init(&bars.vfull[i], 4);
      mbar_init(&bars.vempty[i], 2);
      mbar_init(&bars.qfull[i], 8);
      mbar_init(&bars.sfull[i], 1);
      mbar_init(&bars.pfull[i], 8);
      mbar_init(&bars.ofull[i], 1);
      mbar_init(&bars.turn[i], 1);
    }
    mbar_init(&bars.done, 2);
    item_ring_init(bars.items, kReaders);
    bars.abort = 0;
    fence_mbar_init();
  }
  if (warp == kMma) {
    tmem_alloc(&bars.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem;

  launch_dependents();
  wait_for_previous();
  const long long total = total_units(p), range = range_of(p, total);
  const long long x0 = blockIdx.x * range, x1 = min(total, x0 + range);
  int* const abort = &bars.abort;
  if (x0 >= x1 && threadIdx.x < 2) reinterpret_cast<PartItem*>(p.part_item)[2 * blockIdx.x + threadIdx.x].rows = 0;
  if (x0 < x1) {
    if (warp < kSoftmax) {
      // ================================================================ softmax
      asm volatile("setmaxnreg.inc.sync.aligned.u32 88;");
      const int g = warp >> 3, h = (warp >> 2) & 1;  // tile A or B; keys 64 h .. of S, columns h D/2 .. of O
      const int r = (warp & 3) * 32 + lane;          // row in the tile
      const int pair_bar = 1 + 4 * g + (warp & 3);   // of the two warps that share 32 rows
      const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const uint32_t ts = tmem + lanes + g * 128 + 64 * h, to = tmem + lanes + 256 + g * 128 + h * (D / 2);
      // One warp of the tile's eight tests a barrier, the others wait for it at a
      // hardware barrier (1.09 ms; all eight testing 1.13).
      const int tile_bar = 9 + g;
      const bool tests = (warp & 7) == 0;
      float* const give = &bars.swap[g][h][r];
      const float* const take = &bars.swap[g][h ^ 1][r];
      uint32_t cnt = 0;  // tiles of keys done
      ItemReader items;
      Item it, nx = items.next(bars.items, polls, p.err, abort);
      bool end = named_bar_red_or(tile_bar, 256, nx.n == 0);  // all eight leave together
      bool done_one = false;          // `it` holds an item whose output is still in tensor memory
      float sc = 0.0f, gv = 0.0f;
      float m = -INFINITY, nb = 0.0f;  // running maximum as used (log2 units); P's shift less it (0 for none)
      uint64_t l2 = 0ull;
      while (true) {
        // the next item's queries while the last products of this one run
        const bool mine = !end && nx.rows > g * 128;
        float sc_next = 0.0f;
        if (mine) {
          sc_next = load_q<D>(p, nx, nx.row0 + g * 128 + r, r, h, sq + g * C::Q_BYTES, give, take, pair_bar);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.qfull[g]);
        }
        if (done_one) {
          const int rr = g * 128 + r, idx = it.row0 + rr;
          float l, lb;
          unpair(l2, l, lb);
          l += lb;
          *give = l;
          if (tests) wait_warp(&bars.ofull[g], (cnt - 1) & 1, polls, p.err, abort);
          named_bar_sync(tile_bar, 256);
          tc_fence_after();
          l = h ? *take + l : l + *take;
          const int tok = idx / p.G;
          const long long row = static_cast<long long>(it.q0 + tok) * p.Hq + it.h * p.G + (idx - tok * p.G);
          const bool whole = it.slot < 0, have = rr < it.rows;
          const float inv = row_factor(gv, l);
#pragma unroll 1
          for (int q = 0; q < D / 64; ++q) {
            uint32_t o[32];
            tmem_ld_32x32b_x32(to + 32 * q, o);
            tmem_ld_wait();
            if (whole) {
              if (have) {
                uint4* dst = reinterpret_cast<uint4*>(p.out + row * D + h * (D / 2) + 32 * q);
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                  uint32_t w[4];
#pragma unroll
                  for (int k = 0; k < 4; ++k)
                    w[k] = pack_bf16x2(__uint_as_float(o[8 * v + 2 * k]) * inv, __uint_as_float(o[8 * v + 2 * k + 1]) * inv);
                  dst[v] = make_uint4(w[0], w[1], w[2], w[3]);
                }
              }
            } else {
              uint4* dst = reinterpret_cast<uint4*>(p.part_o + (static_cast<long long>(it.slot) * kRows + rr) * D +
                                                    h * (D / 2) + 32 * q);
#pragma unroll
              for (int v = 0; v < 8; ++v) dst[v] = make_uint4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
            }
          }
          if (h == 0) {
            if (!whole) {
              p.part_ml[static_cast<long long>(it.slot) * 2 * kRows + rr] = m;
              p.part_ml[(static_cast<long long>(it.slot) * 2 + 1) * kRows + rr] = l;
            } else if (p.lse && have) {
              p.lse[row] = row_lse(m, l);
            }
          }
          tc_fence_before();
        }
        if (end) break;
        it = nx;
        done_one = mine;
        if (mine) {
          sc = sc_next;
          gv = __ldg(p.g_v + it.h);
          int lo = 0, hi = it.len;  // a row that is not there masks nothing
          if (g * 128 + r < it.rows) item_keys(p, it, it.row0 + g * 128 + r, lo, hi);
          lo -= it.u * kKeys + 64 * h;  // in the thread's 64 keys of the first tile
          hi -= it.u * kKeys + 64 * h;
          m = -INFINITY, nb = 0.0f;
          l2 = 0ull;
          for (int i = 0; i < it.n; ++i, ++cnt, lo -= kKeys, hi -= kKeys) {
            if (tests) wait_warp(&bars.sfull[g], cnt & 1, polls, p.err, abort);
            named_bar_sync(tile_bar, 256);
            tc_fence_after();
            if (!__all_sync(0xFFFFFFFFu, lo <= 0 && hi >= 64)) {  // some row does not see all of these keys
#pragma unroll 1
              for (int q = 0; q < 2; ++q) {
                uint32_t v[32];
                tmem_ld_32x32b_x32(ts + 32 * q, v);
                tmem_ld_wait();
                // bit j: key 32 q + j is seen
                const int x = min(max(lo - 32 * q, 0), 32), y = min(max(hi - 32 * q, 0), 32);
                const uint32_t see = static_cast<uint32_t>(((1ull << y) - 1ull) & ~((1ull << x) - 1ull));
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  if (!(see & (1u << j))) v[j] = 0xFF800000u;  // -infinity
                tmem_st_32x32b_x32(ts + 32 * q, v);
              }
              tmem_st_wait();
            }
            uint32_t va[32], vb[32];
            tmem_ld_32x32b_x32(ts, va);
            tmem_ld_32x32b_x32(ts + 32, vb);
            tmem_ld_wait();
            float top = __uint_as_float(va[0]), alt = __uint_as_float(vb[0]);
#pragma unroll
            for (int j = 1; j < 31; j += 2) {
              top = fmaxf(fmaxf(top, __uint_as_float(va[j])), __uint_as_float(va[j + 1]));
              alt = fmaxf(fmaxf(alt, __uint_as_float(vb[j])), __uint_as_float(vb[j + 1]));
            }
            top = fmaxf(fmaxf(top, __uint_as_float(va[31])), fmaxf(alt, __uint_as_float(vb[31]))) * sc;
            // does any row of the pair's 32 need a new maximum? (also the rows' first keys)
            if (named_bar_red_or(pair_bar, 64, top > m + kSlack)) {
              *give = top;
              named_bar_sync(pair_bar, 64);
              top = fmaxf(top, *take);
              float f = 1.0f;
              if (top > m + kSlack) {
                f = m == -INFINITY ? 0.0f : ex2(m - top);
                m = top;
                nb = kShift - top;
              }
              l2 = fma2(l2, pair(f, f), 0ull);
              if (i > 0) {  // O holds something: bring it to the new maximum
                wait_warp(&bars.ofull[g], (cnt - 1) & 1, polls, p.err, abort);
                tc_fence_after();
#pragma unroll 1
                for (int q = 0; q < D / 16; ++q) {
                  uint32_t o[8];
                  tmem_ld_32x32b_x8(to + 8 * q, o);
                  tmem_ld_wait();
#pragma unroll
                  for (int j = 0; j < 8; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                  tmem_st_32x32b_x8(to + 8 * q, o);
                }
              }
            }
            const uint64_t sc2 = pair(sc, sc), nb2 = pair(nb, nb);
            auto weigh = [&](int q, const uint32_t* v) {  // P of 16 keys, over the thread's own columns
              uint32_t w[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                float x, y;
                unpair(fma2(pair(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])), sc2, nb2), x, y);
                x = ex2(x);
                y = ex2(y);
                l2 = add2(l2, pair(x, y));
                w[j] = pack_f16x2(x, y);
              }
              tmem_st_32x32b_x8(ts + 8 * q, w);
            };
            weigh(0, va);
            weigh(1, va + 16);
            weigh(2, vb);
            weigh(3, vb + 16);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.pfull[g]);
          }
        }
        nx = items.next(bars.items, polls, p.err, abort);
        end = named_bar_red_or(tile_bar, 256, nx.n == 0);
      }
    } else {
      if (warp < kLoad) {
        // ============================================================== expand
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        const bool is_v = warp >= kExpandV;
        const int w = warp & 3, c4 = lane & 3;
        const int team_bar = is_v ? 12 : 11;  // warp 0 tests barriers for the four
        const int logp = p.P == 32 ? 5 : p.P == 64 ? 6 : 7;
        const int n_slots = is_v ? v_slots : k_slots;
        const uint8_t* my_ring = ring + (is_v ? k_slots * half : 0);
        uint64_t *full = bars.full[is_v], *empty = bars.empty[is_v];
        int slot = 0;        // of the team's next half
        uint32_t round = 0;  // its parity
        // Byte offset of a key's half, the key counted in the tile.
        auto half_of = [&](int key) {
          int sl = slot + (key >> logp);
          if (sl >= n_slots) sl -= n_slots;
          return sl * half;
        };
        ItemReader items;
        uint32_t j = 0;
        while (true) {
          const Item it = items.next(bars.items, polls, p.err, abort);
          if (named_bar_red_or(team_bar, 128, it.n == 0)) break;  // all four together
          for (int i = 0; i < it.n; ++i, ++j) {
            const uint32_t st = j & 1, ph = (j >> 1) & 1;
            if (w == 0) {
              int sl = slot;
              uint32_t rd = round;
              for (int pg = 0; pg < pages; ++pg) {
                wait_warp(&full[sl], rd, polls, p.err, abort);
                if (++sl == n_slots) sl = 0, rd ^= 1;
              }
            }
            if (w == 0 && j >= 2) wait_warp(is_v ? &bars.vempty[st] : &bars.kempty[st], ph ^ 1, polls, p.err, abort);
            named_bar_sync(team_bar, 128);
            // lane = (key, quarter of its values); the warp's keys are 32k + 8w ..
            constexpr int W = D / 32;  // words of 8 codes per lane
            const bool hi = W == 4 && (c4 & 2);
            const int key0 = 8 * w + (lane >> 2);
            const int keys = it.len - (it.u + i) * kKeys;  // past them the bytes are not a key's
#pragma unroll 1
            for (int k2 = 0; k2 < 4; k2 += 2) {
              uint32_t cw[2][W], sb[2];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int in = (32 * (k2 + k) + key0) & (p.P - 1);
                const uint8_t* kc = my_ring + half_of(32 * (k2 + k));
                if (W == 4) {
                  const uint4 v = *reinterpret_cast<const uint4*>(kc + in * (D / 2) + 16 * c4);
                  cw[k][0] = v.x, cw[k][1] = v.y, cw[k][2 % W] = v.z, cw[k][3 % W] = v.w;
                  sb[k] = *reinterpret_cast<const uint16_t*>(kc + codes_bytes(p.P, D) + in * (D / 16) + 2 * c4);
                } else {
                  const uint2 v = *reinterpret_cast<const uint2*>(kc + in * (D / 2) + 8 * c4);
                  cw[k][0] = v.x, cw[k][1] = v.y;
                  sb[k] = kc[codes_bytes(p.P, D) + in * (D / 16) + c4];
                }
              }
              const uint32_t row =
                  (is_v ? sv : sk) + st * C::K_BYTES + (W == 4 ? (c4 >> 1) * C::SUB_Q : 0) + (32 * k2 + key0) * 128;
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const uint32_t f = e4m3x2_to_f16x2(32 * (k2 + k) + key0 < keys ? sb[k] : 0u);
                // lanes 2, 3 of a key write their chunks in another order: no two of a phase on the same banks
                const uint32_t f0 = __byte_perm(f, f, hi ? 0x3232 : 0x1010), f1 = __byte_perm(f, f, hi ? 0x1010 : 0x3232);
#pragma unroll
                for (int q = 0; q < W; ++q) {
                  uint32_t h[4];
                  e2m1x8(W == 4 && hi ? cw[k][(q ^ 2) % W] : cw[k][q], h);
                  const int chunk = W == 4 ? 4 * (c4 & 1) + (q ^ (c4 & 2)) : 2 * c4 + q;
                  const uint32_t fq = W == 4 && q >= 2 ? f1 : f0;
                  st_shared_v4(row + k * 32 * 128 + ((chunk ^ (key0 & 7)) << 4), hmul2(h[0], fq), hmul2(h[1], fq),
                               hmul2(h[2], fq), hmul2(h[3], fq));
                }
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(is_v ? &bars.vfull[st] : &bars.kfull[st]);
            for (int pg = 0; pg < pages; ++pg) {
              if (lane == 0) mbar_arrive(&empty[slot]);
              if (++slot == n_slots) slot = 0, round ^= 1;
            }
          }
        }
      } else {
       asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
       if (warp == kLoad) {
        // ================================================================ load
        // lanes 0 .. feed the keys' ring, 16 .. the values'
        const int v = lane >> 4, i = lane & 15;
        Slot slot;
        slot.index = i, slot.slots = slots[v];
        slot.to = i < slots[v] ? ring + ((v ? slots[0] : 0) + i) * half : nullptr;
        slot.full = &bars.full[v][i], slot.empty = &bars.empty[v][i];
        ItemReader items;
        while (true) {
          const Item it = items.next(bars.items, polls, p.err, abort);
          if (it.n == 0) break;
          slot.feed(
              p, it, pages * it.n, half, 2 * half, [&](int k) { return it.u * pages + k; },
              [&](int) { return v ? half : 0; }, abort);
          if (given_up(abort)) break;
        }
        slot.land(p);
      } else if (warp == kWalk) {
        // ================================================================ walk
        ItemWriter out;
        walk_range<kRows>(p, kKeys, blockIdx.x, x0, x1, range, [&](const Item& t) {
          out.put(bars.items, t, polls, p.err, abort);
          return !given_up(abort);
        });
      } else {
        // =================================================== matrix instructions
        // Warp kMma issues tile A's, kMma + 1 tile B's: what one waits for is
        // hidden under the other's.  Per tile of keys: all waits, then
        // O_g += P_g V(j - 1) and S_g = Q_g K(j)^T back to back.
        const int g = warp - kMma;
        const uint64_t dq = smem_desc_kmajor_sw128(sq + g * C::Q_BYTES);
        const uint64_t dk = smem_desc_kmajor_sw128(sk), dv = smem_desc_mnmajor_sw128(sv, C::SUB_Q);
        const uint32_t ts = tmem + g * 128, to = tmem + 256 + g * 128;
        uint32_t pq = 0, pp = 0;  // parities of qfull and pfull
        ItemReader items;
        Item nx = items.next(bars.items, polls, p.err, abort);
        int rem = nx.n;
        bool nx_first = true, cur = false, cur_mine = false, cur_first = false;
        for (uint32_t j = 0; rem > 0 || cur; ++j) {
          const uint32_t st = j & 1, so = st ^ 1;
          const bool more = rem > 0, mine = more && nx.rows > g * 128;
          if (more) wait_warp(&bars.kfull[st], (j >> 1) & 1, polls, p.err, abort);
          if (cur) wait_warp(&bars.vfull[so], ((j - 1) >> 1) & 1, polls, p.err, abort);
          // The tiles take turns, one's products queued while the other's S is in
          // the making: left to themselves they fall into step, and the tensor
          // cores idle while both are in their softmax.
          if (g == 1 || j > 0) wait_warp(&bars.turn[g], (j - (g == 0)) & 1, polls, p.err, abort);
          // O += P V, then S = Q K^T, which P lies over.  A rolled loop keeps what
          // S needs out of the way of P's product: 0.98 against 1.05 ms unrolled.  One
          // election for all of a product's instructions: 0.95 against 0.98.
#pragma unroll 1
          for (int step = 0; step < 2; ++step) {
            if (step == 0) {
              if (cur_mine) {
                wait_warp(&bars.pfull[g], pp, polls, p.err, abort);
                pp ^= 1;
                tc_fence_after();
                const uint64_t b = dv + so * (C::K_BYTES >> 4);
                if (elect_one()) {
#pragma unroll
                  for (int kk = 0; kk < kKeys / 16; ++kk)
                    umma_f16_ts(to, ts + (kk >> 2) * 64 + (kk & 3) * 8, b + kk * (16 * 128 >> 4),
                                idesc_f16_f32(128, D) | kMajorB, cur_first && kk == 0 ? 0u : 1u);
                  umma_commit(&bars.ofull[g]);
                  umma_commit(&bars.turn[g ^ 1]);
                  umma_commit(&bars.vempty[so]);
                }
              } else if (cur && lane == 0) {
                mbar_arrive(&bars.vempty[so]);
              }
            } else if (mine) {
              if (nx_first) {  // an item's first tile: its queries
                wait_warp(&bars.qfull[g], pq, polls, p.err, abort);
                pq ^= 1;
              }
              tc_fence_after();
              const uint64_t b = dk + st * (C::K_BYTES >> 4);
              if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                  const uint64_t o = (kk >> 2) * (C::SUB_Q >> 4) + (kk & 3) * 2;
                  umma_f16(ts, dq + o, b + o, idesc_f16_f32(128, kKeys), kk ? 1u : 0u);
                }
                umma_commit(&bars.sfull[g]);
                umma_commit(&bars.kempty[st]);
              }
            } else if (more && lane == 0) {
              mbar_arrive(&bars.kempty[st]);
            }
          }
          if (!cur_mine && lane == 0) mbar_arrive(&bars.turn[g ^ 1]);
          __syncwarp();
          cur = more, cur_mine = mine, cur_first = nx_first;
          nx_first = false;
          if (more && --rem == 0) {
            nx = items.next(bars.items, polls, p.err, abort);
            rem = nx.n;
            nx_first = true;
          }
        }
        umma_commit_warp(&bars.done);
        mbar_wait_warp(&bars.done, 0, kLandNs, p.err, nullptr);
       }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMma) tmem_dealloc(tmem, 512);
}

template <int D>
int launch(const AttnParams& p, cudaStream_t s) {
  using C = Cfg<D>;
  const int half = record_bytes(p.P, D) / 2;
  // a tile's halves at least, the rest shared out, keys first
  const int all = std::min(2 * kMaxSlots, C::RING / half);
  const int k_slots = (all + 1) / 2, v_slots = all / 2;
  const int smem = C::RING0 + all * half;
  static std::atomic<bool> set[64];
  MOE_TRY(allow_smem(attn_tiles_kernel<D>, C::RING0 + C::RING, set));
  return launch_after(attn_tiles_kernel<D>, dim3(p.blocks), kThreads, smem, s, p, k_slots, v_slots);
}

}  // namespace

int attention_tiles(const AttnParams& p, int D, cudaStream_t s) { return D == 128 ? launch<128>(p, s) : launch<64>(p, s); }

}  // namespace kv4
}  // namespace moe
