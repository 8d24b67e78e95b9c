// Attention over the paged NVFP4 cache, 16 query rows at a time (one decode
// step's heads of a kv head) for heads of 64, and the schedule and joining
// kernels.
//
// Bound: the cache's bytes, 9/8 byte per key-value dimension pair, read once
// per kv head; next is expanding the codes (two conversions and two products
// per four values) and then the 16-row matrix instructions.  So the records
// stream into shared memory by bulk copies, one page and head each, several
// in flight per block, and every code is expanded straight into the operand
// registers of the matrix instructions, never back to shared memory:
//
//  - S = Q K^T: the order of the reduction index is free as long as Q and K
//    share it, so a lane takes D/4 consecutive values of one key.
//  - O = P V: the order of the output columns is free, so a lane takes D/8
//    consecutive values of four keys; nibbles of two keys are joined to one
//    byte before the conversion, which yields the pair the instruction wants.
//
// Codes times block scales are exact in fp16.  Q (bf16) is scaled per row by
// a power of two into fp16's range, exact for values within 2^-29 of the
// row's largest; P is rounded to fp16 (2^-12); all sums are fp32.  The
// global scales and Q's power of two go into the softmax scale and the output.
//
// 64 sequences of 8192 keys, 64 heads on 4 of 64: 67 us (2.3 TB/s); the matrix
// instructions and the conversions share issue slots (11.5 cycles per product
// with its two conversions and two multiplications, and scheduler).  Heads of
// 128 took 198 us this way where kv4_decode.cu takes 175; three groups of four
// warps 198, two 204, four with Q in shared memory 245.
#include "kv4_attention.cuh"

namespace moe {
namespace kv4 {
namespace {

constexpr int kRows = kRowsSmall;
constexpr int kWarps = 4;     // consumer warps of a group
constexpr int kGroups = 3;    // groups of a block, each with its own range of the work
constexpr int kThreads = 32 * kGroups * kWarps + 128;  // and a warpgroup with their producers
constexpr int kMaxSlots = 32;
constexpr int D = 64;         // of the 16-row kernel here; heads of 128 have kv4_decode.cu's
constexpr int kSmem = 226 * 1024;

// ------------------------------------------------------------------ schedule
// One block; of a warp where a warp has a lane for every sequence and tile (no
// block-wide steps), else of 1024 threads.
template <int ROWS, int THREADS>
__global__ void __launch_bounds__(THREADS) attn_plan_kernel(const AttnParams p, int unit) {
  __shared__ long long s_warp[32];
  launch_dependents();
  plan<ROWS, THREADS>(p, unit, s_warp);
}

// -------------------------------------------------------------------- joining
// Block (c, y): the item whose first part lies in range c.  Parts are added in
// a fixed order, so a call's result is the same each time.
DEVINL void write_row(const AttnParams& p, const PartItem& t, int r, float m, float l, int D, int lane,
                      const float* o, int V) {
  const int idx = t.row0 + r, tok = idx / p.G;
  const long long row = static_cast<long long>(t.q0 + tok) * p.Hq + t.h * p.G + (idx - tok * p.G);
  const float inv = row_factor(__ldg(p.g_v + t.h), l);
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + row * D) + lane * (V / 2);
#pragma unroll
  for (int v = 0; v < V / 2; ++v) dst[v] = pack_bf16x2(o[2 * v] * inv, o[2 * v + 1] * inv);
  if (p.lse && lane == 0) p.lse[row] = row_lse(m, l);
}

// Few rows.  With many parts (one context over the whole GPU has a hundred) a
// block per row, four warps share its parts, eight reads in flight each; with
// few (a decode batch: two) a warp per row.
template <int ROWS, int D>
__global__ void __launch_bounds__(128) attn_join_parts_kernel(const AttnParams p) {
  constexpr int V = D / 32;  // columns per lane
  __shared__ float s_o[4][D], s_l[4], s_m[4];
  wait_for_previous();
  const int c = blockIdx.x, r = blockIdx.y;
  const PartItem t = reinterpret_cast<const PartItem*>(p.part_item)[2 * c + 1];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float m = -INFINITY, l = 0.0f, o[V];
#pragma unroll
  for (int v = 0; v < V; ++v) o[v] = 0.0f;
  if (t.last - c < 4) {
    const int row = 4 * r + w;
    if (row >= t.rows) return;
    float pm[4], pl[4], x[4][V];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = min(c + j, t.last);
      const long long slot = 2ll * i + (i == c);
      pm[j] = c + j <= t.last ? p.part_ml[slot * 2 * ROWS + row] : -INFINITY;
      pl[j] = p.part_ml[(slot * 2 + 1) * ROWS + row];
      const float* po = p.part_o + (slot * ROWS + row) * D + lane * V;
#pragma unroll
      for (int v = 0; v < V; ++v) x[j][v] = po[v];
    }
    m = fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3]));
    const float ref = m == -INFINITY ? 0.0f : m;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float f = ex2(pm[j] - ref);
      l += f * pl[j];
#pragma unroll
      for (int v = 0; v < V; ++v) o[v] += f * x[j][v];
    }
    write_row(p, t, row, m, l, D, lane, o, V);
    return;
  }
  if (r >= t.rows) return;
  for (int base = c + w; base <= t.last; base += 128) {  // lane j: part base + 4 j
    const int mine = base + 4 * lane;
    const long long slot = 2ll * mine + (mine == c);
    float pm = -INFINITY, pl = 0.0f;
    if (mine <= t.last) {
      pm = p.part_ml[slot * 2 * ROWS + r];
      pl = p.part_ml[(slot * 2 + 1) * ROWS + r];
    }
    float top = pm;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
    const float mn = fmaxf(m, top);
    const float ref = mn == -INFINITY ? 0.0f : mn;
    const float old = ex2(m - ref), f = ex2(pm - ref);
    float sum = f * pl;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, x);
    l = l * old + sum;
    m = mn;
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] *= old;
    const int n = min(32, (t.last - base) / 4 + 1);
    for (int j0 = 0; j0 < n; j0 += 8) {
      float x[8][V];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = base + 4 * min(j0 + j, n - 1);
        const float* po = p.part_o + ((2ll * i + (i == c)) * ROWS + r) * D + lane * V;
#pragma unroll
        for (int v = 0; v < V; ++v) x[j][v] = po[v];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float fj = j0 + j < n ? __shfl_sync(0xFFFFFFFFu, f, j0 + j) : 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] += fj * x[j][v];
      }
    }
  }
  if (lane == 0) s_m[w] = m, s_l[w] = l;
#pragma unroll
  for (int v = 0; v < V; ++v) s_o[w][lane * V + v] = o[v];
  __syncthreads();
  if (w != 0) return;
  const float mx = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
  const float ref = mx == -INFINITY ? 0.0f : mx;
  l = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) o[v] = 0.0f;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const float f = ex2(s_m[x] - ref);
    l += f * s_l[x];
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] += f * s_o[x][lane * V + v];
  }
  write_row(p, t, r, mx, l, D, lane, o, V);
}

// Many rows with few parts: a warp takes four rows side by side.
template <int ROWS, int D>
__global__ void __launch_bounds__(128) attn_join_rows_kernel(const AttnParams p) {
  constexpr int V = D / 32, R = 4;
  wait_for_previous();
  const int c = blockIdx.x;
  const PartItem t = reinterpret_cast<const PartItem*>(p.part_item)[2 * c + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int r0 = (blockIdx.y * 4 + warp) * R; r0 < t.rows; r0 += gridDim.y * 4 * R) {
    float m[R], l[R], o[R][V];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      m[k] = -INFINITY, l[k] = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) o[k][v] = 0.0f;
    }
#pragma unroll 2
    for (int i = c; i <= t.last; ++i) {
      const long long slot = 2ll * i + (i == c);
      const float* ml = p.part_ml + slot * 2 * ROWS + r0;  // rows past t.rows: the item's own padding
      const float* po = p.part_o + (slot * ROWS + r0) * D + lane * V;
#pragma unroll
      for (int k = 0; k < R; ++k) {
        const float pm = ml[k], pl = ml[ROWS + k];
        float x[V];
#pragma unroll
        for (int v = 0; v < V; ++v) x[v] = po[k * D + v];
        const float mn = fmaxf(m[k], pm);
        const float ref = mn == -INFINITY ? 0.0f : mn;
        const float old = ex2(m[k] - ref), f = ex2(pm - ref);
        l[k] = l[k] * old + f * pl;
#pragma unroll
        for (int v = 0; v < V; ++v) o[k][v] = o[k][v] * old + f * x[v];
        m[k] = mn;
      }
    }
#pragma unroll
    for (int k = 0; k < R; ++k)
      if (r0 + k < t.rows) write_row(p, t, r0 + k, m[k], l[k], D, lane, o[k], V);
  }
}

// ------------------------------------------------------------------- main
DEVINL void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// One group's shared memory beside its ring: 4 consumer warps share it.
struct Group {
  uint64_t full[kMaxSlots], empty[kMaxSlots];  // warp w's ring: slots w * slots of a warp ..
  ItemRing items;
  float m[kWarps][kRows], l[kWarps][kRows];
  int abort;
  alignas(16) float o[kWarps][kRows][D / 2];  // half the columns at a time
};

__global__ void __launch_bounds__(kThreads, 1) attn_rows16_kernel(const AttnParams p, int slots) {
  constexpr int KS = D / 16;  // k steps of S
  constexpr int LD = D / 4;   // values of a key per lane (S), of a row of O per lane
  constexpr int NT = D / 8;   // column tiles of O
  extern __shared__ __align__(128) uint8_t smem[];
  const int rec = record_bytes(p.P, D), hb = rec / 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = warp < kGroups * kWarps ? warp / kWarps : warp - kGroups * kWarps;
  constexpr int head = (sizeof(Group) + 127) & ~127;
  uint8_t* mine = smem + min(grp, kGroups - 1) * (head + kWarps * slots * hb);
  Group& sh = *reinterpret_cast<Group*>(mine);
  uint8_t* ring = mine + head;

  if (warp < kGroups * kWarps && warp % kWarps == 0 && lane == 0) {
    for (int i = 0; i < kMaxSlots; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    item_ring_init(sh.items, kWarps);
    sh.abort = 0;
    fence_mbar_init();
  }
  __syncthreads();

  launch_dependents();
  wait_for_previous();
  const int block = blockIdx.x * kGroups + grp;  // the group's range
  const long long total = total_units(p), range = range_of(p, total);
  const long long x0 = block * range, x1 = min(total, x0 + range);
  int* const abort = &sh.abort;
  const uint32_t polls = polls_of(p.timeout_ns);

  if (warp >= kGroups * kWarps) {
    // -------- one warp per group walks its range and feeds the four warps' rings
    asm volatile("setmaxnreg.dec.sync.aligned.u32 32;");
    if (grp >= kGroups) return;
    ItemWriter out;
    const int w = lane / slots;  // whose ring; its units of an item are every fourth
    Slot slot;
    slot.index = lane % slots, slot.slots = slots;
    slot.to = w < kWarps ? ring + lane * hb : nullptr;
    slot.full = &sh.full[lane], slot.empty = &sh.empty[lane];
    uint32_t it = 0;  // units of the group so far
    walk_range<kRows>(p, p.P, block, x0, x1, range, [&](const Item& t) {
      out.put(sh.items, t, polls, p.err, abort);
      if (t.n > 0) {
        const int first = (w - static_cast<int>(it)) & (kWarps - 1);
        const int mine = first < t.n ? (t.n - first + kWarps - 1) / kWarps : 0;
        slot.feed(
            p, t, 2 * mine, hb, rec, [&](int k) { return t.u + first + kWarps * (k >> 1); },
            [&](int k) { return k & 1 ? hb : 0; }, abort);
        it += t.n;
      }
      return !given_up(abort);
    });
    slot.land(p);
    return;
  }

  // -------- consumers: warp w of the group takes the units w, w + 4, ...
  asm volatile("setmaxnreg.inc.sync.aligned.u32 160;");
  const int wg = warp % kWarps;
  const int g = lane >> 2, c4 = lane & 3;
  ItemReader items;
  uint32_t it = 0;   // units of the group so far
  int st = 0;        // slot of the warp's next half record, and its parity
  uint32_t par = 0;
  const uint8_t* my_ring = ring + wg * slots * hb;
  uint64_t *full = sh.full + wg * slots, *empty = sh.empty + wg * slots;
  while (true) {
    const Item t = items.next(sh.items, polls, p.err, abort);
    if (named_bar_red_or(1 + grp, 32 * kWarps, t.n == 0)) return;  // all four together
    const int n = t.n;
    // rows g and g + 8 of the tile
    uint32_t qa[KS][4];
    float sc[2];
    int lo[2], hi[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int idx = t.row0 + g + 8 * half;
      const bool have = g + 8 * half < t.rows;
      const int tok = idx / p.G;
      lo[half] = 0, hi[half] = t.len;  // a row that is not there masks nothing
      if (have) item_keys(p, t, idx, lo[half], hi[half]);
      uint32_t w[LD / 2];
#pragma unroll
      for (int i = 0; i < LD / 2; ++i) w[i] = 0;
      if (have) {
        const uint4* src = reinterpret_cast<const uint4*>(p.q + (t.q0 + tok) * p.q_stride +
                                                          (t.h * p.G + idx - tok * p.G) * D + c4 * LD);
#pragma unroll
        for (int i = 0; i < LD / 8; ++i) {
          const uint4 v = __ldg(src + i);
          w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
        }
      }
      uint32_t top = 0;  // largest magnitude as bits
#pragma unroll
      for (int i = 0; i < LD / 2; ++i) top = max(top, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
      top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
      top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
      float up;
      row_scale(p.scale * __ldg(p.g_k + t.h), top, up, sc[half]);
#pragma unroll
      for (int i = 0; i < LD / 2; ++i)
        qa[i >> 1][half + 2 * (i & 1)] =
            pack_f16x2(__uint_as_float(w[i] << 16) * up, __uint_as_float(w[i] & 0xFFFF0000u) * up);
    }
    float o[NT][4], m[2] = {-INFINITY, -INFINITY}, nb[2] = {0.0f, 0.0f};
    uint64_t l2[2] = {0ull, 0ull};
#pragma unroll
    for (int i = 0; i < NT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
    // keys that every row of the tile sees
    int all_lo = max(lo[0], lo[1]), all_hi = min(hi[0], hi[1]);
#pragma unroll
    for (int s = 4; s < 32; s <<= 1) {
      all_lo = max(all_lo, __shfl_xor_sync(0xFFFFFFFFu, all_lo, s));
      all_hi = min(all_hi, __shfl_xor_sync(0xFFFFFFFFu, all_hi, s));
    }

    for (int i = (wg - static_cast<int>(it)) & (kWarps - 1); i < n; i += kWarps) {
      // keys in slot st, values in the next one
      const int sv = st + 1 == slots ? 0 : st + 1;
      const uint32_t pv = par ^ static_cast<uint32_t>(sv == 0);
      const uint8_t* kc = my_ring + st * hb;
      const uint8_t* ks = kc + codes_bytes(p.P, D);
      const uint8_t* vc = my_ring + sv * hb;
      const uint8_t* vs = vc + codes_bytes(p.P, D);
      const int key0 = (t.u + i) * p.P;
      const int keys = min(p.P, t.len - key0);
      wait_warp<true>(&full[st], par, polls, p.err, abort);
      if (keys <= 0) {  // a unit without keys
        if (lane == 0) mbar_arrive(&empty[st]);
        wait_warp<true>(&full[sv], pv, polls, p.err, abort);
      }
#pragma unroll 1
      for (int t0 = 0; t0 < keys; t0 += 32) {
        float s[4][4];
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) {
          s[kt][0] = s[kt][1] = s[kt][2] = s[kt][3] = 0.0f;
          const int tok = t0 + 8 * kt + (g ^ ((g >> 1) & 1));
          const uint2 v = *reinterpret_cast<const uint2*>(kc + tok * (D / 2) + c4 * 8);
          const uint32_t w[LD / 8] = {v.x, v.y};
          const uint32_t two = e4m3x2_to_f16x2(ks[tok * (D / 16) + c4]);
          const uint32_t f = __byte_perm(two, two, 0x1010);
#pragma unroll
          for (int j = 0; j < LD / 8; ++j) {
            uint32_t h[4];
            e2m1x8(w[j], h);
#pragma unroll
            for (int q = 0; q < 4; ++q) h[q] = hmul2(h[q], f);
            mma_f16(s[kt], qa[2 * j], h[0], h[1]);
            mma_f16(s[kt], qa[2 * j + 1], h[2], h[3]);
          }
        }
        if (t0 + 32 >= keys) {  // the last of the unit's keys
          __syncwarp();
          if (lane == 0) mbar_arrive(&empty[st]);
        }
        const int k0 = key0 + t0;
        if (__any_sync(0xFFFFFFFFu, k0 < all_lo || k0 + 32 > all_hi)) {  // some row does not see all of these keys
#pragma unroll
          for (int kt = 0; kt < 4; ++kt)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int key = k0 + 8 * kt + ((2 * c4 + (q & 1)) ^ (c4 & 1));
              if (key < lo[q >> 1] || key >= hi[q >> 1]) s[kt][q] = -INFINITY;
            }
        }
        float top[2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int q = 2 * half;
          float a = fmaxf(fmaxf(s[0][q], s[0][q + 1]), s[1][q]);
          a = fmaxf(fmaxf(a, s[1][q + 1]), s[2][q]);
          a = fmaxf(fmaxf(a, s[2][q + 1]), s[3][q]);
          top[half] = fmaxf(a, s[3][q + 1]) * sc[half];
        }
        if (__any_sync(0xFFFFFFFFu, top[0] > m[0] + kSlack || top[1] > m[1] + kSlack)) {
          float f[2];
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            top[half] = fmaxf(top[half], __shfl_xor_sync(0xFFFFFFFFu, top[half], 1));
            top[half] = fmaxf(top[half], __shfl_xor_sync(0xFFFFFFFFu, top[half], 2));
            f[half] = 1.0f;
            if (top[half] > m[half] + kSlack) {
              f[half] = m[half] == -INFINITY ? 0.0f : ex2(m[half] - top[half]);
              m[half] = top[half];
              nb[half] = kShift - top[half];
            }
            l2[half] = fma2(l2[half], pair(f[half], f[half]), 0ull);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            o[nt][0] *= f[0], o[nt][1] *= f[0];
            o[nt][2] *= f[1], o[nt][3] *= f[1];
          }
        }
        uint32_t pa[2][4];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint64_t sc2 = pair(sc[half], sc[half]), nb2 = pair(nb[half], nb[half]);
#pragma unroll
          for (int kt = 0; kt < 4; ++kt) {
            float a, b;
            unpair(fma2(pair(s[kt][2 * half], s[kt][2 * half + 1]), sc2, nb2), a, b);
            a = ex2(a);
            b = ex2(b);
            l2[half] = add2(l2[half], pair(a, b));
            pa[kt >> 1][2 * (kt & 1) + half] = pack_f16x2(a, b);
          }
        }
        if (t0 == 0) {
          wait_warp<true>(&full[sv], pv, polls, p.err, abort);
          if (__any_sync(0xFFFFFFFFu, keys < p.P)) {
            // values of keys that were never written: zero scales in the slot,
            // which is the warp's until it hands it back
            uint8_t* z = const_cast<uint8_t*>(vs);
            for (int b = keys * (D / 16) + lane; b < p.P * (D / 16); b += 32) z[b] = 0;
            fence_proxy_async_smem();
            __syncwarp();
          }
        }
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
          uint32_t wa[2], wb[2], f[2];
#pragma unroll
          for (int pr = 0; pr < 2; ++pr) {
            const int ta = t0 + 16 * kb + 8 * pr + ((2 * c4) ^ (c4 & 1)), tb = ta ^ 1;
            const uint32_t sa = vs[ta * (D / 16) + (g >> 1)];
            const uint32_t sb = vs[tb * (D / 16) + (g >> 1)];
            f[pr] = e4m3x2_to_f16x2(sa | (sb << 8));
            wa[pr] = *reinterpret_cast<const uint32_t*>(vc + ta * (D / 2) + 4 * g);
            wb[pr] = *reinterpret_cast<const uint32_t*>(vc + tb * (D / 2) + 4 * g);
          }
#pragma unroll
          for (int odd = 0; odd < 2; ++odd) {
            uint32_t b[2][4];
#pragma unroll
            for (int pr = 0; pr < 2; ++pr) {
              e2m1x8(odd ? ((wa[pr] >> 4) & 0x0F0F0F0Fu) | (wb[pr] & 0xF0F0F0F0u)
                         : (wa[pr] & 0x0F0F0F0Fu) | ((wb[pr] << 4) & 0xF0F0F0F0u),
                     b[pr]);
#pragma unroll
              for (int q = 0; q < 4; ++q) b[pr][q] = hmul2(b[pr][q], f[pr]);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) mma_f16(o[2 * q + odd], pa[kb], b[0][q], b[1][q]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[sv]);
      st = sv, par = pv;
      if (++st == slots) st = 0, par ^= 1;
    }
    it += n;

    // -------- the four warps' results become one, half the columns at a time
    const bool whole = t.slot < 0;
    const int rows = t.rows;
    const long long slot = t.slot;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float l, lb;
      unpair(l2[half], l, lb);
      l += lb;
      l += __shfl_xor_sync(0xFFFFFFFFu, l, 1);
      l += __shfl_xor_sync(0xFFFFFFFFu, l, 2);
      if (c4 == 0) {
        sh.m[wg][g + 8 * half] = m[half];
        sh.l[wg][g + 8 * half] = l;
      }
    }
    // Lane's columns of a row are LD * c4 .. + LD; part k of two holds the
    // lane's columns [k * LD / 2, (k + 1) * LD / 2).  16-byte chunks are moved so
    // that the eight lanes of a store phase hit different banks.
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      if (part) named_bar_sync(1 + grp, 32 * kWarps);  // the first half has been read
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int r = g + 8 * half;
#pragma unroll
        for (int v = 0; v < LD / 8; ++v) {
          float4 f;
          float* fp = reinterpret_cast<float*>(&f);
#pragma unroll
          for (int q = 0; q < 4; ++q) fp[q] = o[4 * v + q][2 * half + part];  // LD / 2 = NT columns: tile 4v + q
          const int chunk = (LD / 8) * c4 + v;
          *reinterpret_cast<float4*>(&sh.o[wg][r][4 * (chunk ^ ((c4 + 4 * (r & 1)) & (D / 8 - 1)))]) = f;
        }
      }
      named_bar_sync(1 + grp, 32 * kWarps);
      constexpr int CH = D / 8;  // 16-byte chunks of half a row
      for (int k = wg * 32 + lane; k < rows * CH; k += 32 * kWarps) {
        const int r = k / CH, q = k % CH;
        const int col = (q / (LD / 8)) * LD + part * (LD / 2) + 4 * (q % (LD / 8));
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sh.m[w][r]);
        const float base = mm == -INFINITY ? 0.0f : mm;
        float ll = 0.0f;
        float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const int from = 4 * (q ^ ((q / (LD / 8) + 4 * (r & 1)) & (D / 8 - 1)));
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float f = ex2(sh.m[w][r] - base);
          const float4 v = *reinterpret_cast<const float4*>(&sh.o[w][r][from]);
          ll += f * sh.l[w][r];
          a.x += f * v.x, a.y += f * v.y, a.z += f * v.z, a.w += f * v.w;
        }
        if (whole) {
          const int idx = t.row0 + r, tok = idx / p.G;
          const long long row = static_cast<long long>(t.q0 + tok) * p.Hq + t.h * p.G + (idx - tok * p.G);
          const float inv = row_factor(__ldg(p.g_v + t.h), ll);
          *reinterpret_cast<uint2*>(p.out + row * D + col) =
              make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
          if (p.lse && q == 0 && part == 0) p.lse[row] = row_lse(mm, ll);
        } else {
          *reinterpret_cast<float4*>(p.part_o + (slot * kRows + r) * D + col) = a;
          if (q == 0 && part == 0) {
            p.part_ml[slot * 2 * kRows + r] = mm;
            p.part_ml[(slot * 2 + 1) * kRows + r] = ll;
          }
        }
      }
    }
  }
}

int launch_rows16(const AttnParams& p, cudaStream_t s) {
  const int half = record_bytes(p.P, D) / 2;
  const int head = static_cast<int>(round_up(sizeof(Group), 128));
  // half records per warp: two at least (a unit's keys and values)
  const int slots = std::min(kMaxSlots / kWarps, (kSmem / kGroups - head) / (kWarps * half));
  const int smem = kGroups * (head + kWarps * slots * half);
  static std::atomic<bool> set[64];
  MOE_TRY(allow_smem(attn_rows16_kernel, kSmem, set));
  return launch_after(attn_rows16_kernel, dim3(p.blocks / kGroups), kThreads, smem, s, p, slots);
}

// A wait of the kernels above on a barrier that nothing arrives on.
__global__ void attn_wait_selftest_kernel(unsigned int* err, unsigned long long timeout_ns, int lazy) {
  __shared__ uint64_t bar;
  __shared__ int abort;
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1);
    abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  if (lazy) wait_warp<true>(&bar, 0, polls_of(timeout_ns), err, &abort);
  else wait_warp(&bar, 0, polls_of(timeout_ns), err, &abort);
}

// Schedule, main kernel, joining.
template <int ROWS, int D>
int run(const AttnParams& p, int unit, cudaStream_t s) {
  if (!p.plan_here) {
    if (p.B < 32 && static_cast<long long>(p.T) * p.G / ROWS + p.B <= 32) attn_plan_kernel<ROWS, 32><<<1, 32, 0, s>>>(p, unit);
    else attn_plan_kernel<ROWS, 1024><<<1, 1024, 0, s>>>(p, unit);
    MOE_TRY(check_launch());
  }
  MOE_TRY(ROWS != kRows ? attention_tiles(p, D, s) : D == 128 ? attention_decode(p, s) : launch_rows16(p, s));
  if constexpr (ROWS == kRows) return launch_after(attn_join_parts_kernel<ROWS, D>, dim3(p.blocks, ROWS), 128, 0, s, p);
  else return launch_after(attn_join_rows_kernel<ROWS, D>, dim3(p.blocks, ROWS / 16), 128, 0, s, p);
}

constexpr int kTileRows = kRowsTile, kTileKeys = 128;

struct Layout {
  int rows, blocks;
  size_t bytes;
};

// Kernel variant, its blocks, and the workspace they need; fills p's pointers.
Layout layout(AttnParams& p, int D, void* ws) {
  Layout r;
  // Rows per sequence and kv head on average: the 16-row kernels expand the
  // cache's codes again for every 16 rows, the 256-row kernel once, at the price
  // of products 256 rows wide.  64 sequences of 8192 keys, 4 kv heads of 128: 85 /
  // 151 / 215 us for 16 / 32 / 48 rows on the one, 223 for 64 on the other, which
  // takes about as long for fewer (242 / 241 / 241 / 239 when it was measured for
  // 64 .. 16, and the one 282 for 64); heads of 64: 67 / 109 / 156, and 170 (203).
  // The rule takes the whole call's average, so a batch of single tokens beside a
  // chunk runs on one of the two: 255 single tokens and a chunk of 512, 4096 keys
  // each, 401 us, where two calls take 152 and 83.
  const bool tiles16 = static_cast<long long>(p.T) * p.G <= 48ll * p.B;
  r.rows = tiles16 ? kRows : kTileRows;
  r.blocks = tiles16 && D != 128 ? kGroups * num_sms() : num_sms();
  Carve c(ws, 0);
  const long long tiles = static_cast<long long>(p.T) * p.G / r.rows + p.B + 1;
  p.starts = c.take<int>(p.B + 1);
  p.tile_base = c.take<int>(p.B + 1);
  p.unit_sum = c.take<long long>(tiles + 1);
  p.part_item = c.take<int>(static_cast<size_t>(2) * r.blocks * 8);
  p.part_ml = c.take<float>(static_cast<size_t>(2) * r.blocks * 2 * r.rows);
  p.part_o = c.take<float>(static_cast<size_t>(2) * r.blocks * r.rows * D);
  p.blocks = r.blocks;
  p.min_units = tiles16 ? 1 : 2;
  // a launch less for few sequences: one query 22 against 28 us with the call's host time
  p.plan_here = tiles16 && D == 128 && p.B <= kPlanHere && static_cast<long long>(p.T) * p.G / r.rows + p.B <= kPlanHere;
  r.bytes = c.used;
  return r;
}

}  // namespace

int attention_wait_selftest(unsigned long long timeout_ns, int lazy, cudaStream_t s) {
  unsigned int* err = device_error_word();
  if (!err) return MOE_ERR_CUDA;
  attn_wait_selftest_kernel<<<1, 32, 0, s>>>(err, timeout_ns, lazy);
  return check_launch();
}

int attention(const AttnParams& p, int D, int rows, cudaStream_t s) {
  if (rows == kRows) return D == 128 ? run<kRows, 128>(p, kTileKeys, s) : run<kRows, 64>(p, p.P, s);
  return D == 128 ? run<kTileRows, 128>(p, kTileKeys, s) : run<kTileRows, 64>(p, kTileKeys, s);
}

}  // namespace kv4
}  // namespace moe

using namespace moe;

extern "C" int moe_selftest_attention_wait_timeout(unsigned long long timeout_ns, int lazy, void* stream) {
  return kv4::attention_wait_selftest(timeout_ns, lazy, static_cast<cudaStream_t>(stream));
}

extern "C" size_t moe_kv4_attention_workspace_size(int T, int B, int Hq, int Hkv, int D) {
  if (T < 1 || B < 1 || Hkv < 1 || Hq < Hkv || Hq % Hkv || !kv4::head_dim_ok(D)) return 0;
  kv4::AttnParams p{};
  p.T = T, p.B = B, p.Hq = Hq, p.Hkv = Hkv, p.G = Hq / Hkv;
  return kv4::layout(p, D, nullptr).bytes;
}

extern "C" int moe_kv4_attention(const uint16_t* q, long long q_stride, int T, int Hq, const uint8_t* pool,
                                 int num_pages, int page_size, int Hkv, int D, const float* g_k, const float* g_v,
                                 const int32_t* q_offsets, const int32_t* kv_lens, const int32_t* table, int B,
                                 int max_pages, float scale, int causal, int window, uint16_t* out, float* lse,
                                 void* ws, size_t ws_bytes, void* stream) {
  if (T < 0 || B < 0 || Hq < 1 || Hkv < 1 || window < 0 || (window > 0 && !causal)) return MOE_ERR_INVALID_ARG;
  if (!kv4::head_dim_ok(D) || !kv4::page_size_ok(page_size) || Hq % Hkv != 0 || Hq > 1024) return MOE_ERR_UNSUPPORTED;
  if (T > (1 << 24) || B > (1 << 20)) return MOE_ERR_UNSUPPORTED;
  if (T == 0 || B == 0) return MOE_OK;
  if (!q || !pool || !g_k || !g_v || !q_offsets || !kv_lens || !table || !out || !ws) return MOE_ERR_INVALID_ARG;
  if (num_pages < 1 || max_pages < 1) return MOE_ERR_INVALID_ARG;
  if (static_cast<long long>(max_pages) * page_size > (1ll << 30)) return MOE_ERR_UNSUPPORTED;
  if (!aligned(q, 16) || !aligned(pool, 16) || !aligned(out, 16) || !aligned(ws, 256) || !aligned(lse, 4) ||
      !aligned(g_k, 4) || !aligned(g_v, 4) || !aligned(q_offsets, 4) || !aligned(kv_lens, 4) || !aligned(table, 4))
    return MOE_ERR_INVALID_ARG;
  if (q_stride % 8 || q_stride < static_cast<long long>(Hq) * D) return MOE_ERR_INVALID_ARG;
  kv4::AttnParams p{};
  p.q = q, p.q_stride = q_stride, p.pool = pool, p.g_k = g_k, p.g_v = g_v;
  p.q_offsets = q_offsets, p.kv_lens = kv_lens, p.table = table, p.out = out, p.lse = lse;
  p.T = T, p.B = B, p.Hq = Hq, p.Hkv = Hkv, p.G = Hq / Hkv, p.num_pages = num_pages, p.P = page_size;
  p.max_pages = max_pages, p.causal = causal, p.scale = scale;
  // a window as long as the table is none; a longer one could overflow with a
  // query in front of the first key (2^24 of them at most)
  p.window = static_cast<int>(std::min(static_cast<long long>(window), static_cast<long long>(max_pages) * page_size));
  p.timeout_ns = wait_timeout_ns();
  p.err = device_error_word();
  if (!p.err) return MOE_ERR_CUDA;
  const kv4::Layout l = kv4::layout(p, D, ws);
  if (l.bytes > ws_bytes) return MOE_ERR_WORKSPACE;
  return kv4::attention(p, D, l.rows, static_cast<cudaStream_t>(stream));
}
