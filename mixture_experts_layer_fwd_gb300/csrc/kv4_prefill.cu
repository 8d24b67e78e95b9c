// Attention over the paged NVFP4 cache, 256 query rows at a time: two tiles A
// and B of 128 rows share every 128 keys (chunks of prompts, or a few tokens
// of many heads; an item of up to 128 rows uses tile A alone).
//
// Bound: the tensor cores, 4 * 128 * D multiply-adds per row and tile of keys,
// then the exponentials.  One block per SM; the roles, by warp:
//
//   0-3, 4-7  softmax of tile A / B, one row per thread: S from tensor memory,
//             running maximum and sum, P (fp16) back over S's columns
//   8-11      expand the codes: K as [key][d], V transposed to [d][key], both
//             fp16 in the 128-byte swizzle the matrix instructions read
//   12        bulk copies of the halves (keys, values) of page records
//   13        issues the matrix instructions, 14 waits for it (a wait in the
//             issuing warp would queue behind its instructions)
//
// S = Q K^T comes from shared memory, O += P V takes P from tensor memory.  The
// order of issue is P_A V, Q_A K', P_B V, Q_B K' (K' the next tile), so that
// one tile's softmax runs under the other's products.  S and O fill tensor
// memory: 2 x 128 + 2 x D columns; P lies in the first half of its S.
//
// The running maximum is moved only when a row's grows by more than 2^kSlack:
// until then O needs no rescaling, and P keeps fp16's relative precision.
// Numbers are as in the 16-row kernel: codes times block scales and Q times a
// power of two are exact in fp16, P is rounded to fp16, sums are fp32.
#include "kv4_attention.cuh"

namespace moe {
namespace kv4 {
namespace {

constexpr int kRows = kRowsTile;
constexpr int kKeys = 128;
constexpr int kThreads = 512;
constexpr int kMaxSlots = 16;
constexpr int kExpand0 = 8, kLoad = 12, kMma = 13, kWait = 14;

template <int D>
struct Cfg {
  static constexpr int Q_BYTES = 128 * D * 2;     // one row tile
  static constexpr int K_BYTES = kKeys * D * 2;   // one tile of keys; V the same
  static constexpr int SUB_Q = 128 * 128;         // 64-wide sub-tile of Q or K
  static constexpr int SUB_V = D * 128;           // 64-key sub-tile of V transposed
  static constexpr int RING = D == 128 ? 33 * 1024 : 48 * 1024;
  static constexpr int RING0 = 2 * Q_BYTES + 4 * K_BYTES;
};

struct Bars {
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  uint64_t kfull[2], kempty[2], vfull[2], vempty[2];
  uint64_t qfull[2], sfull[2], pfull[2], ofull[2], done;
  uint32_t tmem;
  int abort;
};

// D[tmem] (+)= A[smem] * B[smem]^T from a whole converged warp.
DEVINL void umma_f16_ss_warp(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
DEVINL void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// The block's tiles of keys, in order.
struct Tiles {
  Cursor c;
  long long left;  // tiles of this block's range from the current one on
  int n;           // tiles of the current item from the current one on
  bool two;        // the item has rows in tile B
  bool first;      // the current tile is the item's first here
  DEVINL void item(const AttnParams& p) {
    n = static_cast<int>(min(left, static_cast<long long>(c.u1 - c.u)));
    two = c.s.n * static_cast<long long>(p.G) - static_cast<long long>(c.tile) * kRows > 128;
    first = true;
  }
  DEVINL Tiles(const AttnParams& p, long long x0, long long x1) : c(cursor_at<kRows>(p, kKeys, x0)), left(x1 - x0) {
    item(p);
  }
  DEVINL void next(const AttnParams& p) {
    --left;
    if (left <= 0) return;
    if (--n == 0) {
      cursor_next<kRows>(p, kKeys, c);
      item(p);
    } else {
      ++c.u;
      first = false;
    }
  }
};

// One query row (thread's) to fp16 in the swizzled tile; returns the softmax
// scale of the row in log2 units (>= 0).
template <int D>
DEVINL float load_q(const AttnParams& p, const Cursor& c, int idx, int r, uint32_t tile) {
  const bool have = idx < c.s.n * p.G;
  const int tok = idx / p.G;
  const uint4* src = reinterpret_cast<const uint4*>(p.q + (c.s.q0 + tok) * p.q_stride + (c.h * p.G + idx % p.G) * D);
  uint32_t top = 0;
  if (have) {
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      const uint4 v = __ldg(src + i);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) top = max(top, max(w[q] & 0x7FFFu, (w[q] >> 16) & 0x7FFFu));
    }
  }
  float up, sc;
  row_scale(p.scale * __ldg(p.g_k + c.h), top, up, sc);
#pragma unroll
  for (int i = 0; i < D / 8; ++i) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (have) v = __ldg(src + i);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t h[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
      h[q] = pack_f16x2(__uint_as_float(w[q] << 16) * up, __uint_as_float(w[q] & 0xFFFF0000u) * up);
    st_shared_v4(tile + (i >> 3) * Cfg<D>::SUB_Q + r * 128 + (((i & 7) ^ (r & 7)) << 4), h[0], h[1], h[2], h[3]);
  }
  return sc;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attn_tiles_kernel(const AttnParams p, int slots) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Bars bars;
  // 1024-byte aligned operand tiles: Q_A Q_B | K0 K1 | V0 V1 | ring of record halves
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  const uint32_t sq = base, sk = base + 2 * C::Q_BYTES, sv = sk + 2 * C::K_BYTES, ring_s = base + C::RING0;
  uint8_t* ring = smem_raw + (ring_s - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int half = record_bytes(p.P, D) / 2, pages = kKeys / p.P;
  const unsigned long long tmo = p.timeout_ns;

  if (threadIdx.x == 0) {
    for (int i = 0; i < slots; ++i) {
      mbar_init(&bars.full[i], 1);
      mbar_init(&bars.empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.kfull[i], 4);
      mbar_init(&bars.kempty[i], 1);
      mbar_init(&bars.vfull[i], 4);
      mbar_init(&bars.vempty[i], 1);
      mbar_init(&bars.qfull[i], 4);
      mbar_init(&bars.sfull[i], 1);
      mbar_init(&bars.pfull[i], 4);
      mbar_init(&bars.ofull[i], 1);
    }
    mbar_init(&bars.done, 1);
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

  const long long total = total_units(p), range = range_of(p, total);
  const long long x0 = blockIdx.x * range, x1 = min(total, x0 + range);
  if (x0 < x1) {
    if (warp < 8) {
      // ================================================================ softmax
      asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
      const int g = warp >> 2;                       // tile A or B
      const int r = (warp & 3) * 32 + lane;          // row in the tile
      const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const uint32_t ts = tmem + lanes + g * 128, to = tmem + lanes + 256 + g * 128;
      const uint32_t tile_q = sq + g * C::Q_BYTES;
      uint32_t cnt = 0;  // tiles of keys done
      bool loaded = false;
      float sc = 0.0f;
      Cursor c = cursor_at<kRows>(p, kKeys, x0);
      long long left = x1 - x0;
      while (left > 0) {
        const int n = static_cast<int>(min(left, static_cast<long long>(c.u1 - c.u)));
        const int row0 = c.tile * kRows;
        const bool mine = g == 0 || c.s.n * p.G - row0 > 128;
        if (mine) {
          const int idx = row0 + g * 128 + r;
          if (!loaded) {
            sc = load_q<D>(p, c, idx, r, tile_q);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.qfull[g]);
          }
          loaded = false;
          int lo = 0, hi = c.s.len;  // a row that is not there masks nothing
          const bool have = idx < c.s.n * p.G;
          if (have) row_keys(p, c.s, idx / p.G, lo, hi);
          float m = -INFINITY, nb = 0.0f;  // running maximum as used (log2 units); P's shift less it (0 for none)
          uint64_t l2[2] = {0ull, 0ull};
          for (int i = 0; i < n; ++i, ++cnt) {
            mbar_wait_warp(&bars.sfull[g], cnt & 1, tmo, p.err, &bars.abort);
            tc_fence_after();
            uint32_t s[4][32];
#pragma unroll
            for (int q = 0; q < 4; ++q) tmem_ld_32x32b_x32(ts + 32 * q, s[q]);
            tmem_ld_wait();
            const int k0 = (c.u + i) * kKeys;
            if (!__all_sync(0xFFFFFFFFu, lo <= k0 && k0 + kKeys <= hi)) {
              const int a = lo - k0, b = hi - k0;
#pragma unroll
              for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  if (32 * q + j < a || 32 * q + j >= b) s[q][j] = 0xFF800000u;  // -infinity
            }
            float mx[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              mx[q] = __uint_as_float(s[q][0]);
#pragma unroll
              for (int j = 1; j < 31; j += 2)
                mx[q] = fmaxf(fmaxf(mx[q], __uint_as_float(s[q][j])), __uint_as_float(s[q][j + 1]));
              mx[q] = fmaxf(mx[q], __uint_as_float(s[q][31]));
            }
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;
            const bool grow = top > m + kSlack;  // also the row's first keys
            if (__any_sync(0xFFFFFFFFu, grow)) {
              float f = 1.0f;
              if (grow) {
                f = m == -INFINITY ? 0.0f : ex2(m - top);
                m = top;
                nb = kShift - top;
              }
              const uint64_t ff = pair(f, f);
#pragma unroll
              for (int q = 0; q < 2; ++q) l2[q] = fma2(l2[q], ff, 0ull);
              if (i > 0) {  // O holds something: bring it to the new maximum
                mbar_wait_warp(&bars.ofull[g], (cnt - 1) & 1, tmo, p.err, &bars.abort);
                tc_fence_after();
#pragma unroll 1
                for (int q = 0; q < D / 16; ++q) {
                  uint32_t o[16];
                  tmem_ld_32x32b_x16(to + 16 * q, o);
                  tmem_ld_wait();
#pragma unroll
                  for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                  tmem_st_32x32b_x16(to + 16 * q, o);
                }
              }
            }
            const uint64_t sc2 = pair(sc, sc), nb2 = pair(nb, nb);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t w[16];
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                float a, b;
                unpair(fma2(pair(__uint_as_float(s[q][2 * j]), __uint_as_float(s[q][2 * j + 1])), sc2, nb2), a, b);
                a = ex2(a);
                b = ex2(b);
                l2[j & 1] = add2(l2[j & 1], pair(a, b));
                w[j] = pack_f16x2(a, b);
              }
              tmem_st_32x32b_x16(ts + 16 * q, w);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.pfull[g]);
          }
          // the next item's queries while the last products run
          Cursor nx = c;
          if (left > n) cursor_next<kRows>(p, kKeys, nx);
          if (left > n && (g == 0 || nx.s.n * p.G - nx.tile * kRows > 128)) {
            sc = load_q<D>(p, nx, nx.tile * kRows + g * 128 + r, r, tile_q);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.qfull[g]);
            loaded = true;
          }
          mbar_wait_warp(&bars.ofull[g], (cnt - 1) & 1, tmo, p.err, &bars.abort);
          tc_fence_after();
          float l, la, lb;
          unpair(add2(l2[0], l2[1]), la, lb);
          l = la + lb;
          const bool whole = c.u == c.u0 && n == c.u1 - c.u0;
          if (whole) {
            const long long row = static_cast<long long>(c.s.q0 + idx / p.G) * p.Hq + c.h * p.G + idx % p.G;
            const float inv = l > 0.0f ? __ldg(p.g_v + c.h) / l : 0.0f;
#pragma unroll
            for (int q = 0; q < D / 32; ++q) {
              uint32_t o[32];
              tmem_ld_32x32b_x32(to + 32 * q, o);
              tmem_ld_wait();
              if (have) {
                uint4* dst = reinterpret_cast<uint4*>(p.out + row * D + 32 * q);
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                  uint32_t w[4];
#pragma unroll
                  for (int k = 0; k < 4; ++k)
                    w[k] = pack_bf16x2(__uint_as_float(o[8 * v + 2 * k]) * inv, __uint_as_float(o[8 * v + 2 * k + 1]) * inv);
                  dst[v] = make_uint4(w[0], w[1], w[2], w[3]);
                }
              }
            }
            if (p.lse && have) p.lse[row] = l > 0.0f ? (m + log2f(l) - kShift) * (1.0f / kLog2e) : -INFINITY;
          } else {
            const long long slot = 2ll * blockIdx.x + (c.u == c.u0 ? 1 : 0);
            const int rr = g * 128 + r;
#pragma unroll
            for (int q = 0; q < D / 32; ++q) {
              uint32_t o[32];
              tmem_ld_32x32b_x32(to + 32 * q, o);
              tmem_ld_wait();
              uint4* dst = reinterpret_cast<uint4*>(p.part_o + (slot * kRows + rr) * D + 32 * q);
#pragma unroll
              for (int v = 0; v < 8; ++v) dst[v] = make_uint4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
            }
            p.part_ml[slot * 2 * kRows + rr] = m;
            p.part_ml[(slot * 2 + 1) * kRows + rr] = l;
          }
          tc_fence_before();
        }
        left -= n;
        if (left > 0) cursor_next<kRows>(p, kKeys, c);
      }
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
      if (warp < kLoad) {
        // ============================================================== expand
        const int w = warp - kExpand0, c4 = lane & 3;
        const int tg = lane & 7, tgh = w & 1;  // V: group of 8 keys in a 64-key sub-tile
        const int blk = D == 128 ? (2 * (tg >> 1) + (lane >> 3) + 4 * (w >> 1)) & 7 : (2 * (tg >> 1) + (lane >> 3)) & 3;
        const int odd = tg & 1;
        Tiles t(p, x0, x1);
        uint32_t s = 0;  // halves taken from the ring
        for (uint32_t j = 0; t.left > 0; ++j, t.next(p)) {
          const uint32_t st = j & 1, ph = (j >> 1) & 1;
          // ---- K
          if (j >= 2) mbar_wait_warp(&bars.kempty[st], ph ^ 1, tmo, p.err, &bars.abort);
          const uint32_t kt = sk + st * C::K_BYTES;
          for (int pg = 0; pg < pages; ++pg, ++s) {
            const uint32_t slot = s % slots;
            mbar_wait_warp(&bars.full[slot], (s / slots) & 1, tmo, p.err, &bars.abort);
            const uint8_t* kc = ring + slot * half;
            const uint8_t* ks = kc + codes_bytes(p.P, D);
            for (int t0 = 8 * w; t0 < p.P; t0 += 32) {
              const int in = t0 + (lane >> 2), key = pg * p.P + in;
              constexpr int W = D / 32;  // words of 8 codes per lane
              uint32_t cw[W];
              uint32_t sb[2];
              if (W == 4) {
                const uint4 v = *reinterpret_cast<const uint4*>(kc + in * (D / 2) + 16 * c4);
                // lanes 2, 3 of a key write their chunks in another order: no two of a phase on the same banks
                const bool hi = c4 & 2;
                cw[0] = hi ? v.z : v.x, cw[1] = hi ? v.w : v.y, cw[2 % W] = hi ? v.x : v.z, cw[3 % W] = hi ? v.y : v.w;
                const uint32_t f = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(ks + in * (D / 16) + 2 * c4));
                sb[0] = __byte_perm(f, f, hi ? 0x3232 : 0x1010);
                sb[1] = __byte_perm(f, f, hi ? 0x1010 : 0x3232);
              } else {
                const uint2 v = *reinterpret_cast<const uint2*>(kc + in * (D / 2) + 8 * c4);
                cw[0] = v.x, cw[1] = v.y;
                const uint32_t f = e4m3x2_to_f16x2(ks[in * (D / 16) + c4]);
                sb[0] = sb[1] = __byte_perm(f, f, 0x1010);
              }
              const uint32_t row = kt + (W == 4 ? (c4 >> 1) * C::SUB_Q : 0) + key * 128;
#pragma unroll
              for (int i = 0; i < W; ++i) {
                uint32_t h[4];
                e2m1x8(cw[i], h);
                const int chunk = W == 4 ? 4 * (c4 & 1) + (i ^ (c4 & 2)) : 2 * c4 + i;
                const uint32_t f = sb[W == 4 ? i >> 1 : 0];
                st_shared_v4(row + ((chunk ^ (key & 7)) << 4), hmul2(h[0], f), hmul2(h[1], f), hmul2(h[2], f),
                             hmul2(h[3], f));
              }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.empty[slot]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.kfull[st]);
          // ---- V
          if (j >= 2) mbar_wait_warp(&bars.vempty[st], ph ^ 1, tmo, p.err, &bars.abort);
          for (int pg = 0; pg < pages; ++pg)
            mbar_wait_warp(&bars.full[(s + pg) % slots], ((s + pg) / slots) & 1, tmo, p.err, &bars.abort);
          if (D == 128 || w < 2) {
            const int first = tgh * 64 + tg * 8;  // the thread's 8 keys in the tile
            const uint8_t* vc = ring + ((s + first / p.P) % slots) * half + (first % p.P) * (D / 2) + 8 * blk;
            const uint8_t* vs = ring + ((s + first / p.P) % slots) * half + codes_bytes(p.P, D) +
                                (first % p.P) * (D / 16) + blk;
            const int keys = t.c.s.len - t.c.u * kKeys - first;  // of the 8 that were written
            uint2 cw[8];
            uint32_t sb[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {  // register i: key i ^ odd, so that neighbours read different banks
              cw[i] = *reinterpret_cast<const uint2*>(vc + (i ^ odd) * (D / 2));
              sb[i] = (i ^ odd) < keys ? vs[(i ^ odd) * (D / 16)] : 0u;
            }
            uint32_t f[4];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              const uint32_t a = odd ? sb[2 * m + 1] : sb[2 * m], b = odd ? sb[2 * m] : sb[2 * m + 1];
              f[m] = e4m3x2_to_f16x2(a | (b << 8));
            }
            const uint32_t vt = sv + st * C::K_BYTES + tgh * C::SUB_V + 16 * blk * 128;
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              uint32_t h[8][4];
#pragma unroll
              for (int m = 0; m < 4; ++m) {
                const uint32_t x = v ? cw[2 * m].y : cw[2 * m].x, y = v ? cw[2 * m + 1].y : cw[2 * m + 1].x;
                const uint32_t a = odd ? y : x, b = odd ? x : y;
                uint32_t even[4], odds[4];
                e2m1x8((a & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u), even);
                e2m1x8(((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u), odds);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  h[2 * q][m] = hmul2(even[q], f[m]);
                  h[2 * q + 1][m] = hmul2(odds[q], f[m]);
                }
              }
#pragma unroll
              for (int k = 0; k < 8; ++k)
                st_shared_v4(vt + (8 * v + k) * 128 + ((tg ^ k) << 4), h[k][0], h[k][1], h[k][2], h[k][3]);
            }
          }
          __syncwarp();
          if (lane == 0)
            for (int pg = 0; pg < pages; ++pg) mbar_arrive(&bars.empty[(s + pg) % slots]);
          s += pages;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.vfull[st]);
        }
      } else if (warp == kLoad) {
        // ================================================================ load
        Tiles t(p, x0, x1);
        uint32_t s = 0;
        for (; t.left > 0; t.next(p)) {
          int page = -1;
          const int at = t.c.u * pages + lane;
          if (lane < pages && static_cast<long long>(at) * p.P < t.c.s.len) {
            page = __ldg(p.table + static_cast<long long>(t.c.b) * p.max_pages + at);
            if (page < 0 || page >= p.num_pages) {
              atomicOr(p.err, kErrBadIndex);
              page = 0;
            }
          }
          for (int k = 0; k < 2 * pages; ++k, ++s) {
            const int pg = __shfl_sync(0xFFFFFFFFu, page, k % pages);
            const uint32_t slot = s % slots;
            if (lane == 0) {
              if (s >= static_cast<uint32_t>(slots))
                mbar_wait_bounded(&bars.empty[slot], (s / slots - 1) & 1, tmo, p.err, &bars.abort);
              if (pg < 0 || *static_cast<volatile int*>(&bars.abort)) {
                mbar_arrive(&bars.full[slot]);  // no key of this tile
              } else {
                mbar_arrive_expect_tx(&bars.full[slot], half);
                bulk_load(ring + slot * half,
                          p.pool + (static_cast<long long>(pg) * p.Hkv + t.c.h) * 2 * half + (k < pages ? 0 : half), half,
                          &bars.full[slot]);
              }
            }
            __syncwarp();
          }
        }
        // after a time-out elsewhere, stay until the copies in flight have landed
        if (*static_cast<volatile int*>(&bars.abort) && lane == 0)
          for (uint32_t k = s > static_cast<uint32_t>(slots) ? s - slots : 0; k < s; ++k)
            mbar_wait_bounded(&bars.full[k % slots], (k / slots) & 1, tmo, p.err, nullptr);
      } else if (warp == kMma || warp == kWait) {
        // ========================================== matrix instructions / waits
        // Both warps walk the same steps; the waiting warp lets the other one
        // through a named barrier when a step's operands are there.
        const bool issue = warp == kMma;
        const uint64_t dq[2] = {smem_desc_kmajor_sw128(sq), smem_desc_kmajor_sw128(sq + C::Q_BYTES)};
        const uint64_t dk = smem_desc_kmajor_sw128(sk), dv = smem_desc_kmajor_sw128(sv);
        uint32_t nq[2] = {0, 0}, np[2] = {0, 0};  // items' queries and P tiles taken, per row tile
        auto go = [&]() {
          named_bar_sync(1, 64);
          if (issue) tc_fence_after();
        };
        auto score = [&](int g, uint32_t j, bool first, bool last_use) {  // S_g = Q_g K(j)^T
          if (!issue) {
            if (first) mbar_wait_warp(&bars.qfull[g], nq[g] & 1, tmo, p.err, &bars.abort);
            if (g == 0) mbar_wait_warp(&bars.kfull[j & 1], (j >> 1) & 1, tmo, p.err, &bars.abort);
          }
          if (first) ++nq[g];
          go();
          if (issue) {
            const uint64_t b = dk + (j & 1) * (C::K_BYTES >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint64_t o = (kk >> 2) * (C::SUB_Q >> 4) + (kk & 3) * 2;
              umma_f16_ss_warp(tmem + g * 128, dq[g] + o, b + o, idesc_f16_f32(128, kKeys), kk ? 1u : 0u);
            }
            umma_commit_warp(&bars.sfull[g]);
            if (last_use) umma_commit_warp(&bars.kempty[j & 1]);
          }
        };
        auto value = [&](int g, uint32_t j, bool first, bool last_use) {  // O_g += P_g V(j)
          if (!issue) {
            if (g == 0) mbar_wait_warp(&bars.vfull[j & 1], (j >> 1) & 1, tmo, p.err, &bars.abort);
            mbar_wait_warp(&bars.pfull[g], np[g] & 1, tmo, p.err, &bars.abort);
          }
          ++np[g];
          go();
          if (issue) {
            const uint64_t b = dv + (j & 1) * (C::K_BYTES >> 4);
#pragma unroll
            for (int kk = 0; kk < kKeys / 16; ++kk)
              umma_f16_ts_warp(tmem + 256 + g * 128, tmem + g * 128 + 8 * kk, b + (kk >> 2) * (C::SUB_V >> 4) + (kk & 3) * 2,
                               idesc_f16_f32(128, D), first && kk == 0 ? 0u : 1u);
            umma_commit_warp(&bars.ofull[g]);
            if (last_use) umma_commit_warp(&bars.vempty[j & 1]);
          }
        };
        Tiles t(p, x0, x1);
        score(0, 0, true, !t.two);
        if (t.two) score(1, 0, true, true);
        for (uint32_t j = 0; t.left > 0; ++j) {
          const bool two = t.two, first = t.first;
          value(0, j, first, !two);
          t.next(p);
          if (t.left > 0) score(0, j + 1, t.first, !t.two);
          if (two) value(1, j, first, true);
          if (t.left > 0 && t.two) score(1, j + 1, t.first, true);
        }
        if (issue) {
          umma_commit_warp(&bars.done);
          mbar_wait_warp(&bars.done, 0, tmo, p.err, nullptr);
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
  const int slots = std::min(kMaxSlots, C::RING / half);
  const int smem = 1024 + C::RING0 + slots * half;
  static bool set[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MOE_ERR_CUDA;
  if (!set[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(attn_tiles_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               1024 + C::RING0 + C::RING);
    if (e != cudaSuccess) {
      set_cuda_error(e);
      return MOE_ERR_CUDA;
    }
    set[dev] = true;
  }
  attn_tiles_kernel<D><<<p.blocks, kThreads, smem, s>>>(p, slots);
  return check_launch();
}

}  // namespace

int attention_tiles(const AttnParams& p, int D, cudaStream_t s) { return D == 128 ? launch<128>(p, s) : launch<64>(p, s); }

}  // namespace kv4
}  // namespace moe
