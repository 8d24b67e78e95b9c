// Attention over the paged NVFP4 cache for at most 16 query rows per sequence
// and kv head (a decode step), heads of 128, on the 5th-generation tensor cores
// with the KEYS on the matrix's M side:
//
//   S^T [128 keys][16 rows] = K Q^T        A = K from tensor memory, B = Q
//   O^T [128 d][16 rows]   += V^T P^T      A = V from shared memory, B = P
//
// so that 16 rows cost a 16-wide product and not a 128-wide one (measured: 49
// cycles for 16 keys of either product, 47 where the two alternate, 65 with the
// rows on the M side).
// V lies in shared memory key by key as it comes from the codes, rows (d)
// contiguous, so neither operand is transposed on the way; the order of d in K
// and Q is free, so a lane of an expanding warp takes 16 consecutive bytes.
//
// One block per SM; the roles, by warp:
//
//   0-7    softmax: two groups take turns with pairs of 128-key tiles.  P (fp16)
//          goes to shared memory, S is read twice so that 16 of its values per
//          thread are live.  Each group has maxima, sums and an O of its own.
//   8-15   expand the codes of K into tensor memory: two teams, every other tile
//   16-23  expand the codes of V into shared memory, the same
//   24-27  the items' ends: the next item's queries, the output of this one
//   28     bulk copies of the halves (keys, values) of page records
//   29, 30 issue the products of K and of V (what one waits for is hidden
//          under the other's)
//   31     walks the block's items and publishes them
//
// The maxima are moved only when a score exceeds one by 2^kSlack; only then do
// a group's 128 threads reduce over the keys, and O is rescaled.  Numbers are
// as in the 16-row kernel on mma instructions.
//
// Bound: three things come close to each other, of 0.57 us (1090 cycles) per tile.
// The cache's bytes, 18 KB, are 0.41 us of an SM's share of HBM.  The two
// products are 0.39 us: 16 instructions that hold the tensor pipe for 47 cycles
// each, whichever of the two they belong to and into however many accumulators
// (measured alone; the multiplication in one takes 8 of the 47, which is all
// that the pipe's counter shows, 10 %).  Expanding and the softmax take 70 % of
// the issue slots.  On top come the hand-over between roles and the instruction
// cache (eight programs of 75 KB together run side by side: loops unrolled
// further, or code at an item's end in the warps that everything waits for, cost
// more than they save): 256 sequences of up to 8192 keys, 64 heads on 4, 175 us
// (3.7 TB/s, 0.55 of a copy).
#include "kv4_attention.cuh"

namespace moe {
namespace kv4 {
namespace {

constexpr int D = 128;
constexpr int kRows = kRowsSmall;
constexpr int kKeys = 128;
constexpr int kThreads = 1024;
constexpr int kSlots = 16;                // of a ring at most
constexpr int kKStages = 4, kVStages = 3;
constexpr int kVSteps = 12;               // a multiple of V's stages and P's four buffers
constexpr int kK0 = 8, kV0 = 16, kEnds = 24, kLoad = 28, kMmaK = 29, kWalk = 31;
constexpr int kReaders = 8 + 8 + 8 + 4 + 3;
constexpr int kBarSoft = 1, kBarEnds = 3;  // a softmax group's (1, 2), the items' ends'

constexpr int V_BYTES = kKeys * D * 2;
constexpr int SUB_V = kKeys * 128;        // 64 of V's columns, one key after the other
constexpr int Q_BYTES = kRows * D * 2;    // 16 rows, two 64-wide sub-tiles
constexpr int SUB_Q = kRows * 128;
constexpr int P_BYTES = kRows * kKeys * 2;
constexpr int Q0 = kVStages * V_BYTES, P0 = Q0 + 2 * Q_BYTES, BARS0 = P0 + 4 * P_BYTES, RING0 = BARS0 + 12288;
constexpr int kSmem = 227 * 1024;
// tensor memory columns
constexpr int K_COLS = D / 2, S0 = kKStages * K_COLS, O0 = S0 + 4 * kRows, TMEM_COLS = 512;

struct Bars {
  uint64_t full[2][kSlots], empty[2][kSlots];  // rings of key and of value halves
  // of tile j: [j % kKStages] keys expanded and S's place free, their product
  // done; [j % kVSteps] values expanded and P there, their product done
  uint64_t kready[kKStages], kdone[kKStages], vready[kVSteps], vdone[kVSteps];
  // of an item, by its parity: queries there; sums there; O complete
  uint64_t qfull[2], sums[2], oready[2], end;
  ItemRing items;
  float sc[2][kRows];  // softmax scale of a row, by item parity
  int lo[2][kRows], hi[2][kRows];  // keys that a row sees
  long long row[2][kRows];         // and its place in the output
  float top[2][4][kRows];        // by softmax group: maxima of a warp's keys
  // by item parity and softmax group
  float4 l[2][2][4][32];         // sums of a warp's thread (four rows)
  float m[2][2][kRows];          // maxima
  float fac[2][kRows];           // what a group's O is multiplied by
  long long unit_sum[kPlanHere + 1];  // the schedule, where the block makes it
  int starts[kPlanHere + 1], tile_base[kPlanHere + 1];
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(Bars) <= RING0 - BARS0, "between the tiles and the ring");
static_assert(O0 + 4 * kRows <= TMEM_COLS, "tensor memory");

DEVINL void st_shared_v2(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b));
}
// 16 lanes of tensor memory by 16 columns as matrix fragments: register 4 c + 2 r + e
// of a thread is lane 8 r + (thread / 4), column 8 c + 2 (thread % 4) + e.
DEVINL void tmem_ld_16x256b_x2(uint32_t addr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(addr));
}
DEVINL void tmem_st_16x256b_x2(uint32_t addr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.16x256b.x2.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// The same with 32 columns.
DEVINL void tmem_st_16x256b_x4(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// Four 8 x 8 matrices of 16-bit values, transposed on the way; lane 8 i + k
// gives the address of row k of the i-th in shared memory.
DEVINL void stmatrix_x4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
               "r"(c), "r"(d)
               : "memory");
}

DEVINL int even(int n) { return (n + 1) & ~1; }

// HERE: the block makes the schedule (a form of its own: 20 KB of code that the
// others' loops would share the instruction cache with, 180 against 175 us).
template <bool HERE>
__global__ void __launch_bounds__(kThreads, 1) attn_decode_kernel(const AttnParams p, int k_slots, int v_slots) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  Bars& bars = *reinterpret_cast<Bars*>(smem + BARS0);
  uint8_t* ring = smem + RING0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int half = record_bytes(p.P, D) / 2, pages = kKeys / p.P;
  const uint32_t polls = polls_of(p.timeout_ns);
  int* const abort = &bars.abort;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2 * kSlots; ++i) {
      mbar_init(&bars.full[0][i], 1);
      mbar_init(&bars.empty[0][i], p.P / 32);
    }
    for (int i = 0; i < kKStages; ++i) {
      mbar_init(&bars.kready[i], 8);
      mbar_init(&bars.kdone[i], 1);
    }
    for (int i = 0; i < kVSteps; ++i) {
      mbar_init(&bars.vready[i], 8);
      mbar_init(&bars.vdone[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.qfull[i], 4);
      mbar_init(&bars.sums[i], 8);
      mbar_init(&bars.oready[i], 1);
    }
    mbar_init(&bars.end, 2);
    item_ring_init(bars.items, kReaders);
    bars.abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaK) {
    tmem_alloc(&bars.tmem, TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem;

  launch_dependents();
  wait_for_previous();
  AttnParams sched = p;
  if (HERE) {
    sched.starts = bars.starts, sched.tile_base = bars.tile_base, sched.unit_sum = bars.unit_sum;
    if (warp == kWalk) plan<kRows, 32>(sched, kKeys, nullptr);
    __syncthreads();
  }
  const long long total = total_units(sched), range = range_of(p, total);
  const long long x0 = blockIdx.x * range, x1 = min(total, x0 + range);
  if (x0 >= x1 && threadIdx.x < 2) reinterpret_cast<PartItem*>(p.part_item)[2 * blockIdx.x + threadIdx.x].rows = 0;
  if (x0 < x1) {
    if (warp < kK0) {
      // ================================================================ softmax
      asm volatile("setmaxnreg.inc.sync.aligned.u32 96;");
      // Two groups of four warps take turns with pairs of tiles; each has maxima,
      // sums and an O of its own, joined at the item's end.  S and O in
      // fragments: of each, a thread has keys (or d) 32 w + lane / 4 + 0, 8,
      // 16, 24 and rows col0 + 0, 1, 8, 9, which it numbers q.
      const int g = warp >> 2, w = warp & 3;
      const uint32_t lanes = static_cast<uint32_t>(w * 32) << 16;
      const uint32_t ts = tmem + lanes + S0 + 2 * g * kRows;
      const int key0 = w * 32 + (lane >> 2), col0 = 2 * (lane & 3);
      auto row_of = [&](int q) { return col0 + (q & 1) + 8 * (q >> 1); };
      // where the lane's row of P's transposed matrices goes
      const int ph = ((lane >> 4) << 3) + (lane & 7), pk = 4 * (w & 1) + ((lane >> 3) & 1);
      const uint32_t p_at = base + P0 + 2 * g * P_BYTES + (w >> 1) * SUB_Q + ph * 128 + ((pk ^ (ph & 7)) << 4);
      uint32_t j = 2 * g;   // the group's next pair of the block's tiles: j, j + 1
      int vs = 2 * g;       // j % kVSteps
      uint32_t vround = 0;  // j / kVSteps
      // the pair before: are its products of the values done?
      auto wait_before = [&]() {
        if (j > 2) {
          const bool wrap = vs < 3;
          wait_warp(&bars.vdone[wrap ? vs + kVSteps - 3 : vs - 3], (wrap ? vround - 1 : vround) & 1, polls, p.err, abort);
        }
      };
      if (lane == 0) {
        mbar_arrive(&bars.kready[2 * g]);
        mbar_arrive(&bars.kready[2 * g + 1]);
      }
      uint32_t j0 = 0;    // tiles of the items before
      uint32_t seq = 0;   // items begun
      ItemReader items;
      // of the thread's four rows: scale, maximum, kShift - maximum (0 before
      // there is one), what a score may be before the maximum moves, sum
      float sc[4], m[4], nb[4], most[4], l[4];
      while (true) {
        const Item it = items.next(bars.items, polls, p.err, abort);
        if (named_bar_red_or(kBarSoft + g, 128, it.n == 0)) break;
        const int par = seq & 1;
        wait_warp(&bars.qfull[par], (seq >> 1) & 1, polls, p.err, abort);
        ++seq;
        const uint32_t to = tmem + lanes + O0 + (2 * par + g) * kRows;
        const int last = (it.u + it.n) * kKeys;  // past it, an item with an odd number of tiles has a ghost
        const int all_lo = __reduce_max_sync(0xFFFFFFFFu, bars.lo[par][lane & 15]);
        const int all_hi = min(last, __reduce_min_sync(0xFFFFFFFFu, bars.hi[par][lane & 15]));
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          sc[q] = bars.sc[par][row_of(q)];
          m[q] = most[q] = -INFINITY;
          nb[q] = l[q] = 0.0f;
        }
#pragma unroll 1
        for (int i = j - j0; i < it.n; i += 4) {
          wait_warp(&bars.kdone[(j + 1) & (kKStages - 1)], (j / kKStages) & 1, polls, p.err, abort);  // and j's
          tc_fence_after();
          // S is read twice, once for the maxima and once for P, a tile at a time:
          // register 8 h + 4 c + 2 r + e is key key0 + 16 h + 8 r, row 2 c + e of the thread's
          auto q_of = [](int x) { return 2 * ((x >> 2) & 1) + (x & 1); };
          const int k0 = (it.u + i) * kKeys;
          const bool whole = k0 >= all_lo && k0 + 2 * kKeys <= all_hi;  // every row sees all of these keys
          uint32_t s[16];
          auto load = [&](int tile) {
            tmem_ld_16x256b_x2(ts + tile * kRows, s);
            tmem_ld_16x256b_x2(ts + tile * kRows + (16u << 16), s + 8);
            tmem_ld_wait();
            if (!whole) {
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const int first = k0 + tile * kKeys + key0;
                const int lo = bars.lo[par][row_of(q)] - first, hi = min(bars.hi[par][row_of(q)], last) - first;
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                  const int key = 16 * (x >> 3) + 8 * ((x >> 1) & 1);
                  if (q_of(x) == q && (key < lo || key >= hi)) s[x] = 0xFF800000u;  // -infinity
                }
              }
            }
          };
          float t[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) t[q] = -INFINITY;
#pragma unroll 1
          for (int tile = 0; tile < 2; ++tile) {
            load(tile);
#pragma unroll
            for (int x = 0; x < 16; ++x) t[q_of(x)] = fmaxf(t[q_of(x)], __uint_as_float(s[x]));
          }
          bool over = false;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            t[q] = fmaf(t[q], sc[q], nb[q]);  // sc > 0
            over = over || t[q] > most[q];
          }
          over = named_bar_red_or(kBarSoft + g, 128, over);
          wait_before();  // P's buffers are free, O at rest
          if (over) {
            // new maxima: over the warp's keys, then the warps'
#pragma unroll
            for (int q = 0; q < 4; ++q) {
#pragma unroll
              for (int o = 16; o > 2; o >>= 1) t[q] = fmaxf(t[q], __shfl_xor_sync(0xFFFFFFFFu, t[q], o));
              if (lane < 4) bars.top[g][w][row_of(q)] = t[q];
            }
            named_bar_sync(kBarSoft + g, 128);
            float fac[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int h = row_of(q);
              const float up = fmaxf(fmaxf(bars.top[g][0][h], bars.top[g][1][h]),
                                     fmaxf(bars.top[g][2][h], bars.top[g][3][h])) - nb[q];
              fac[q] = 1.0f;
              if (up > m[q]) {  // every row takes its own, once one has to
                fac[q] = m[q] == -INFINITY ? 0.0f : ex2(m[q] - up);
                m[q] = up;
                nb[q] = kShift - up;
                most[q] = kShift + kSlack;
              }
              l[q] *= fac[q];
            }
            if (i > 3) {  // O holds something: bring it to the new maxima
              tc_fence_after();
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                uint32_t o[8];
                tmem_ld_16x256b_x2(to + (h << 20), o);
                tmem_ld_wait();
#pragma unroll
                for (int x = 0; x < 8; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * fac[q_of(x)]);
                tmem_st_16x256b_x2(to + (h << 20), o);
              }
              tmem_st_wait();
              tc_fence_before();
            }
          }
#pragma unroll 1
          for (int tile = 0; tile < 2; ++tile) {
            load(tile);
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // matrix (8 keys, 8 rows): keys 8 r, rows 8 c
              float y[8];
#pragma unroll
              for (int x = 0; x < 8; ++x) {
                y[x] = ex2(fmaf(__uint_as_float(s[8 * h + x]), sc[q_of(x)], nb[q_of(x)]));
                l[q_of(x)] += y[x];
              }
              stmatrix_x4_trans((p_at ^ (h << 5)) + tile * P_BYTES, pack_f16x2(y[0], y[1]), pack_f16x2(y[2], y[3]),
                                pack_f16x2(y[4], y[5]), pack_f16x2(y[6], y[7]));
            }
          }
          tc_fence_before();
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&bars.kready[j & (kKStages - 1)]);  // S has been read
            mbar_arrive(&bars.kready[(j + 1) & (kKStages - 1)]);
            mbar_arrive(&bars.vready[vs]);
            mbar_arrive(&bars.vready[vs + 1]);
          }
          j += 4;
          if ((vs += 4) >= kVSteps) vs -= kVSteps, ++vround;
        }
        j0 += even(it.n);
        bars.l[par][g][w][lane] = make_float4(l[0], l[1], l[2], l[3]);
        if (w == 0 && lane < 4) {
#pragma unroll
          for (int q = 0; q < 4; ++q) bars.m[par][g][row_of(q)] = m[q];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.sums[par]);
      }
    } else if (warp >= kEnds && warp < kLoad) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
      // =============================================================== item ends
      // The next item's queries, then this one's output; whatever of an item is
      // here twice is free again when the item before has been written.
      const int w = warp & 3, tid = threadIdx.x & 127;
      const int r = tid >> 3, part = tid & 7;  // a row's thread: 16 of its values, an eighth of its sums
      uint32_t seq = 0;
      ItemReader items;
      Item nx = items.next(bars.items, polls, p.err, abort);
      bool end = named_bar_red_or(kBarEnds, 128, nx.n == 0);
      auto queries = [&](int par) {
        const int idx = nx.row0 + r, tok = idx / p.G;
        uint4 v[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
        int lo = 0, hi = nx.len;  // a row that is not there masks nothing
        if (r < nx.rows) {
          const uint4* src = reinterpret_cast<const uint4*>(p.q + (nx.q0 + tok) * p.q_stride +
                                                            (nx.h * p.G + idx - tok * p.G) * D) + 2 * part;
          v[0] = __ldg(src);
          v[1] = __ldg(src + 1);
          item_keys(p, nx, idx, lo, hi);
        }
        const float gk = __ldg(p.g_k + nx.h);
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
          for (int q = 0; q < 4; ++q) top = max(top, max(u[q] & 0x7FFFu, (u[q] >> 16) & 0x7FFFu));
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        float up, scale;
        row_scale(p.scale * gk, top, up, scale);
        // four values of d = 32 p + 4 c + .. go to place 16 c + 4 p of the order in which K lies
        const uint32_t qt = base + Q0 + par * Q_BYTES + (part & 1) * SUB_Q + r * 128 + ((part >> 1) & 1) * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 u = v[i >> 1];
          const uint32_t a[2] = {i & 1 ? u.z : u.x, i & 1 ? u.w : u.y};
          uint32_t x[2];
#pragma unroll
          for (int q = 0; q < 2; ++q)
            x[q] = pack_f16x2(__uint_as_float(a[q] << 16) * up, __uint_as_float(a[q] & 0xFFFF0000u) * up);
          st_shared_v2(qt + (((2 * i + (part >> 2)) ^ (r & 7)) << 4), x[0], x[1]);
        }
        if (part == 0) {
          bars.sc[par][r] = scale;
          bars.row[par][r] = static_cast<long long>(nx.q0 + tok) * p.Hq + nx.h * p.G + (idx - tok * p.G);
          bars.lo[par][r] = lo, bars.hi[par][r] = hi;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.qfull[par]);
      };
      if (!end) queries(0);
      while (!end) {
        const Item it = nx;
        const int par = seq & 1;
        const uint32_t phase = (seq >> 1) & 1;
        ++seq;
        nx = items.next(bars.items, polls, p.err, abort);
        end = named_bar_red_or(kBarEnds, 128, nx.n == 0);
        if (!end) queries(par ^ 1);
        const float gv = __ldg(p.g_v + it.h);
        wait_warp<true>(&bars.sums[par], phase, polls, p.err, abort);
        // the thread's share of row r: its sums lie with lanes 4 .. + (r & 7) / 2 of each warp
        const float m0 = bars.m[par][0][r], m1 = bars.m[par][1][r], mm = fmaxf(m0, m1);
        float f[2] = {m0 == -INFINITY ? 0.0f : ex2(m0 - mm), m1 == -INFINITY ? 0.0f : ex2(m1 - mm)};
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float x = 0.0f;
#pragma unroll
          for (int v = 0; v < 4; ++v)
            x += reinterpret_cast<const float*>(&bars.l[par][k][v][4 * part + ((r & 7) >> 1)])[(r & 1) + 2 * (r >> 3)];
          sum += f[k] * x;
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        if (part == 0) {
          if (it.slot >= 0) {
            p.part_ml[static_cast<long long>(it.slot) * 2 * kRows + r] = mm;
            p.part_ml[(static_cast<long long>(it.slot) * 2 + 1) * kRows + r] = sum;
          } else {
            const float inv = row_factor(gv, sum);
            f[0] *= inv, f[1] *= inv;
            if (p.lse && r < it.rows) p.lse[bars.row[par][r]] = row_lse(mm, sum);
          }
          bars.fac[0][r] = f[0], bars.fac[1][r] = f[1];
        }
        wait_warp<true>(&bars.oready[par], phase, polls, p.err, abort);
        named_bar_sync(kBarEnds, 128);
        tc_fence_after();
        float* po = p.part_o + static_cast<long long>(it.slot) * kRows * D + tid;
#pragma unroll 1
        for (int c = 0; c < kRows; c += 8) {  // a thread a column of the output
          uint32_t o[2][8];
          const uint32_t to = tmem + (static_cast<uint32_t>(w * 32) << 16) + O0 + 2 * par * kRows + c;
          tmem_ld_32x32b_x8(to, o[0]);
          tmem_ld_32x32b_x8(to + kRows, o[1]);
          tmem_ld_wait();
#pragma unroll
          for (int h = 0; h < 8; ++h) {
            const float a = bars.fac[0][c + h], b = bars.fac[1][c + h];
            // a group that had no tile left nothing in its O
            float v = a != 0.0f ? a * __uint_as_float(o[0][h]) : 0.0f;
            if (b != 0.0f) v += b * __uint_as_float(o[1][h]);
            if (c + h < it.rows) {
              if (it.slot < 0) p.out[bars.row[par][c + h] * D + tid] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
              else po[(c + h) * D] = v;
            }
          }
        }
        tc_fence_before();
        named_bar_sync(kBarEnds, 128);  // fac and the rows' places have been read
      }
    } else if (warp < kEnds) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
      // ================================================================ expand
      // Two teams of four warps for the keys, two for the values; a team takes
      // every other tile, a warp 32 keys of it (which lie in one page).
      const bool is_v = warp >= kV0;
      const int team = ((warp - kK0) >> 2) & 1, w = warp & 3;
      const int slots = is_v ? v_slots : k_slots;
      const uint8_t* my_ring = ring + (is_v ? k_slots * half : 0);
      uint64_t *full = bars.full[is_v], *empty = bars.empty[is_v];
      const int in = (32 * w) & (p.P - 1);  // first of the warp's keys in its page
      int slot = team * pages + 32 * w / p.P;
      uint32_t round = 0;                  // parity of the slot's use
      uint32_t j = team;                   // the team's next tile of the block's
      int vs = team;                       // j % kVSteps
      uint32_t vround = 0;                 // j / kVSteps
      uint32_t j0 = 0;                     // tiles of the items before
      ItemReader items;
      while (true) {
        const Item it = items.next(bars.items, polls, p.err, abort);
        if (it.n == 0) break;
#pragma unroll 1
        for (int i = j - j0; i < even(it.n); i += 2) {
          wait_warp(&full[slot], round, polls, p.err, abort);
          const uint8_t* rec = my_ring + slot * half + in * (D / 2);
          const uint8_t* scales = my_ring + slot * half + codes_bytes(p.P, D) + in * (D / 16);
          // (rolled loops: what the warps of a scheduler run has to stay in its instruction cache)
          if (!is_v) {
            // four threads per key, 32 values each: column 8 c + 2 p + e of
            // tensor memory holds values 32 p + 4 c + 2 e, + 1
            const int st = j & (kKStages - 1);
            if (j >= kKStages) wait_warp(&bars.kdone[st], (j / kKStages - 1) & 1, polls, p.err, abort);
            tc_fence_after();
            const uint32_t to = tmem + (static_cast<uint32_t>(32 * w) << 16) + st * K_COLS;
#pragma unroll 2
            for (int x = 0; x < 4; ++x) {  // 16 keys, 16 of the 32 values (a block)
              const int k = 16 * (x >> 1) + (lane >> 2), at = 2 * (lane & 3) + (x & 1);
              uint2 c[2];
              uint32_t sb[2], r[16];
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                c[y] = reinterpret_cast<const uint2*>(rec)[(k + 8 * y) * (D / 16) + at];
                sb[y] = scales[(k + 8 * y) * (D / 16) + at];
              }
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const uint32_t f = e4m3x2_to_f16x2(sb[y] * 0x101u);
                const uint32_t wd[2] = {c[y].x, c[y].y};
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                  uint32_t h[4];
                  e2m1x8(wd[q], h);
#pragma unroll
                  for (int z = 0; z < 4; ++z) r[4 * (2 * q + (z >> 1)) + 2 * y + (z & 1)] = hmul2(h[z], f);
                }
              }
              tmem_st_16x256b_x4(to + (static_cast<uint32_t>(16 * (x >> 1)) << 16) + 32 * (x & 1), r);
            }
            tmem_st_wait();
            tc_fence_before();
          } else {
            // a thread per key; pieces of 32 values in an order that spreads the lanes over the banks
            const bool there = i < it.n && (it.u + i) * kKeys + 32 * w + lane < it.len;  // else the bytes are not a key's
            // the tile that had the stage before
            const bool wrap = vs < kVStages;
            if (j >= kVStages)
              wait_warp(&bars.vdone[wrap ? vs + kVSteps - kVStages : vs - kVStages], (wrap ? vround - 1 : vround) & 1, polls, p.err, abort);
            const uint32_t line = base + vs % kVStages * V_BYTES + (32 * w + lane) * 128;
#pragma unroll 1
            for (int x = 0; x < 4; ++x) {
              const int pc = x ^ ((lane >> 1) & 3);
              const uint4 c = reinterpret_cast<const uint4*>(rec + lane * (D / 2))[pc];
              const uint32_t sb = reinterpret_cast<const uint16_t*>(scales + lane * (D / 16))[pc];
              const uint32_t at = line + (pc >> 1) * SUB_V + (((4 * (pc & 1)) ^ (lane & 7)) << 4);
              const uint32_t two = e4m3x2_to_f16x2(there ? sb : 0u);
              const uint32_t wd[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const uint32_t f = __byte_perm(two, two, q >> 1 ? 0x3232 : 0x1010);
                uint32_t h[4];
                e2m1x8(wd[q], h);
                st_shared_v4(at ^ (q << 4), hmul2(h[0], f), hmul2(h[1], f), hmul2(h[2], f), hmul2(h[3], f));
              }
            }
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&empty[slot]);
            mbar_arrive(is_v ? &bars.vready[vs] : &bars.kready[j & (kKStages - 1)]);
          }
          j += 2;
          if ((vs += 2) >= kVSteps) vs -= kVSteps, ++vround;
          if ((slot += 2 * pages) >= slots) slot -= slots, round ^= 1;
        }
        j0 += even(it.n);
      }
    } else {
     asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
     if (warp == kLoad) {
      // ================================================================== load
      const int v = lane >> 4, i = lane & 15;  // lanes 0 .. feed the keys' ring, 16 .. the values'
      const int slots = v ? v_slots : k_slots;
      Slot slot;
      slot.index = i, slot.slots = slots;
      slot.to = i < slots ? ring + ((v ? k_slots : 0) + i) * half : nullptr;
      slot.full = &bars.full[v][i], slot.empty = &bars.empty[v][i];
      ItemReader items;
      while (true) {
        const Item it = items.next(bars.items, polls, p.err, abort);
        if (it.n == 0) break;
        slot.feed(
            p, it, pages * even(it.n), half, 2 * half,
            [&](int k) { return k < pages * it.n ? it.u * pages + k : p.max_pages; },  // a ghost: no bytes
            [&](int) { return v ? half : 0; },
            abort);
        if (given_up(abort)) break;
      }
      slot.land(p);
    } else if (warp == kWalk) {
      ItemWriter out;
      walk_range<kRows>(sched, kKeys, blockIdx.x, x0, x1, range, [&](const Item& t) {
        out.put(bars.items, t, polls, p.err, abort);
        return !given_up(abort);
      });
    } else {
      // ================================================================ products
      const bool of_k = warp == kMmaK;
      uint32_t j = 0, seq = 0, vround = 0;
      int vs = 0;
      ItemReader items;
      while (true) {
        const Item it = items.next(bars.items, polls, p.err, abort);
        if (it.n == 0) break;
#pragma unroll 1
        for (int i = 0; i < even(it.n); ++i, ++j) {
          const int buf = j & 3;
          if (of_k) {  // S^T = K Q^T
            const int st = j & (kKStages - 1);
            if (i == 0) wait_warp(&bars.qfull[seq & 1], (seq >> 1) & 1, polls, p.err, abort);
            wait_warp(&bars.kready[st], (j / kKStages) & 1, polls, p.err, abort);
            tc_fence_after();
            const uint64_t b = smem_desc_kmajor_sw128(base + Q0 + (seq & 1) * Q_BYTES);
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
                umma_f16_ts(tmem + S0 + buf * kRows, tmem + st * K_COLS + 8 * kk,
                            b + (kk >> 2) * (SUB_Q >> 4) + (kk & 3) * 2, idesc_f16_f32(128, kRows), kk ? 1u : 0u);
              umma_commit(&bars.kdone[st]);
            }
          } else {  // O^T += V^T P^T
            wait_warp(&bars.vready[vs], vround & 1, polls, p.err, abort);
            tc_fence_after();
            const uint64_t a = smem_desc_mnmajor_sw128(base + vs % kVStages * V_BYTES, SUB_V);
            const uint64_t b = smem_desc_kmajor_sw128(base + P0 + buf * P_BYTES);
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < kKeys / 16; ++kk)
                umma_f16(tmem + O0 + (2 * (seq & 1) + (buf >> 1)) * kRows, a + kk * (16 * 128 >> 4), b + (kk >> 2) * (SUB_Q >> 4) + (kk & 3) * 2,
                         idesc_f16_f32(128, kRows) | kMajorA, (i & ~2) || kk ? 1u : 0u);
              umma_commit(&bars.vdone[vs]);
            }
            if (++vs == kVSteps) vs = 0, ++vround;
          }
          __syncwarp();
        }
        if (!of_k) umma_commit_warp(&bars.oready[seq & 1]);
        ++seq;
      }
      umma_commit_warp(&bars.end);
      mbar_wait_warp(&bars.end, 0, kLandNs, p.err, nullptr);
     }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaK) tmem_dealloc(tmem, TMEM_COLS);
}

template <bool HERE>
int launch(const AttnParams& p, int k_slots, int v_slots, int smem, cudaStream_t s) {
  static std::atomic<bool> set[64];
  MOE_TRY(allow_smem(attn_decode_kernel<HERE>, kSmem, set));
  // with a schedule kernel in front, this one may begin under it
  if (!HERE) return launch_after(attn_decode_kernel<HERE>, dim3(p.blocks), kThreads, smem, s, p, k_slots, v_slots);
  attn_decode_kernel<HERE><<<p.blocks, kThreads, smem, s>>>(p, k_slots, v_slots);
  return check_launch();
}

}  // namespace

int attention_decode(const AttnParams& p, cudaStream_t s) {
  const int half = record_bytes(p.P, D) / 2;
  // an even number of tiles in each ring, so that a slot is always the same
  // team's; the values' gets what the keys' leaves
  const int two = 2 * kKeys / p.P, all = (kSmem - RING0) / half;
  const int k_slots = std::min(kSlots, all / 2) / two * two, v_slots = std::min(kSlots, all - k_slots) / two * two;
  const int smem = RING0 + (k_slots + v_slots) * half;
  return p.plan_here ? launch<true>(p, k_slots, v_slots, smem, s) : launch<false>(p, k_slots, v_slots, smem, s);
}

}  // namespace kv4
}  // namespace moe
