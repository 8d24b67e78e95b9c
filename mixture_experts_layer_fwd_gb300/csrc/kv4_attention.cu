// Attention over the paged NVFP4 cache, 16 query rows at a time (one decode
// step's heads of a kv head), and the schedule and joining kernels.
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
#include "kv4_attention.cuh"

namespace moe {
namespace kv4 {
namespace {

constexpr int kRows = kRowsSmall;
constexpr int kWarps = 4;                      // consumer warps
constexpr int kThreads = 32 * (kWarps + 1);    // and a producer warp
constexpr int kMaxStages = 16;
constexpr float kLog2e = 1.4426950408889634f;

// ------------------------------------------------------------------ schedule
template <int ROWS>
__global__ void __launch_bounds__(1024) attn_plan_kernel(const AttnParams p, int unit) {
  __shared__ long long s_warp[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto scan = [&](long long v, long long& total) {
    long long incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += up;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    if (warp == 0) {
      long long w = s_warp[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xFFFFFFFFu, w, o);
        if (lane >= o) w += up;
      }
      s_warp[lane] = w;
    }
    __syncthreads();
    const long long before = warp ? s_warp[warp - 1] : 0;
    total = s_warp[31];
    __syncthreads();
    return before + incl - v;
  };
  // running maximum of the offsets: whatever they hold, the rows of all
  // sequences are disjoint and inside q, so the tiles fit the workspace
  int before_all = 0;
  for (int base = 0; base <= p.B; base += 1024) {
    const int b = base + threadIdx.x;
    int v = b <= p.B ? min(max(p.q_offsets[b], 0), p.T) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xFFFFFFFFu, v, o);
      if (lane >= o) v = max(v, up);
    }
    if (lane == 31) s_warp[warp] = v;
    __syncthreads();
    for (int w = 0; w < warp; ++w) v = max(v, static_cast<int>(s_warp[w]));
    v = max(v, before_all);
    if (b <= p.B) p.starts[b] = v;
    for (int w = 0; w < 32; ++w) before_all = max(before_all, static_cast<int>(s_warp[w]));
    __syncthreads();
  }
  long long tiles = 0;
  for (int base = 0; base < p.B; base += 1024) {
    const int b = base + threadIdx.x;
    long long n = 0, total;
    if (b < p.B) n = (static_cast<long long>(load_seq(p, b).n) * p.G + ROWS - 1) / ROWS;
    const long long at = scan(n, total);
    if (b < p.B) p.tile_base[b] = static_cast<int>(tiles + at);
    tiles += total;
  }
  if (threadIdx.x == 0) p.tile_base[p.B] = static_cast<int>(tiles);
  __syncthreads();
  long long units = 0;
  for (long long base = 0; base < tiles; base += 1024) {
    const long long f = base + threadIdx.x;
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
  if (threadIdx.x == 0) p.unit_sum[tiles] = units;
}

// -------------------------------------------------------------------- joining
// Block (c, y): the item that is cut first at the start of range c; the rows
// y, y + gridDim.y, ... of it, one warp each.
template <int ROWS, int D>
__global__ void __launch_bounds__(128) attn_join_kernel(const AttnParams p, int unit) {
  const long long total = total_units(p), range = range_of(p, total);
  const int c = blockIdx.x + 1;
  const long long cut = c * range;
  if (cut >= total) return;
  const Cursor cur = cursor_at<ROWS>(p, unit, cut);
  const long long start = cut - (cur.u - cur.u0);
  if (start == cut || start < cut - range) return;  // not cut here, or first cut at an earlier range
  const long long end = start + (cur.u1 - cur.u0);
  const int last = static_cast<int>((end - 1) / range);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows = min(ROWS, cur.s.n * p.G - cur.tile * ROWS);
  for (int r = blockIdx.y * 4 + warp; r < rows; r += gridDim.y * 4) {
    float m = -INFINITY;
    for (int i = c - 1; i <= last; ++i) m = fmaxf(m, p.part_ml[(2 * i + (i == c - 1)) * 2 * ROWS + r]);
    const float base = m == -INFINITY ? 0.0f : m;
    float l = 0.0f, o[D / 32];
#pragma unroll
    for (int v = 0; v < D / 32; ++v) o[v] = 0.0f;
    for (int i = c - 1; i <= last; ++i) {
      const int slot = 2 * i + (i == c - 1);
      const float f = exp2f(p.part_ml[slot * 2 * ROWS + r] - base);
      l += f * p.part_ml[(slot * 2 + 1) * ROWS + r];
      const float* po = p.part_o + (static_cast<long long>(slot) * ROWS + r) * D + lane * (D / 32);
#pragma unroll
      for (int v = 0; v < D / 32; ++v) o[v] += f * po[v];
    }
    const int idx = cur.tile * ROWS + r;
    const long long row = static_cast<long long>(cur.s.q0 + idx / p.G) * p.Hq + cur.h * p.G + idx % p.G;
    const float inv = l > 0.0f ? __ldg(p.g_v + cur.h) / l : 0.0f;
    uint32_t w[D / 64];
#pragma unroll
    for (int v = 0; v < D / 64; ++v) w[v] = pack_bf16x2(o[2 * v] * inv, o[2 * v + 1] * inv);
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + row * D) + lane * (D / 64);
#pragma unroll
    for (int v = 0; v < D / 64; ++v) dst[v] = w[v];
    if (p.lse && lane == 0) p.lse[row] = l > 0.0f ? (m + log2f(l) - p_shift(ROWS)) * (1.0f / kLog2e) : -INFINITY;
  }
}

// ------------------------------------------------------------------- main
DEVINL void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

template <int D>
struct Shared {
  uint64_t full[kMaxStages], empty[kMaxStages];
  float m[kWarps][kRows], l[kWarps][kRows];
  int abort;
  alignas(16) float o[kWarps][kRows][D];
};

template <int D>
__global__ void __launch_bounds__(kThreads) attn_rows16_kernel(const AttnParams p, int stages) {
  constexpr int KS = D / 16;  // k steps of S
  constexpr int LD = D / 4;   // values of a key per lane (S), of a row of O per lane
  constexpr int NT = D / 8;   // column tiles of O
  extern __shared__ __align__(128) uint8_t smem[];
  Shared<D>& sh = *reinterpret_cast<Shared<D>*>(smem);
  uint8_t* ring = smem + ((sizeof(Shared<D>) + 127) & ~size_t(127));
  const int rec = record_bytes(p.P, D);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    sh.abort = 0;
    fence_mbar_init();
  }
  __syncthreads();

  const long long total = total_units(p), range = range_of(p, total);
  const long long x0 = blockIdx.x * range, x1 = min(total, x0 + range);
  if (x0 >= x1) return;

  if (warp == kWarps) {
    // -------- producer: one page record per stage
    Cursor c = cursor_at<kRows>(p, p.P, x0);
    uint32_t it = 0;
    long long left = x1 - x0;
    while (left > 0) {
      const int n = static_cast<int>(min(left, static_cast<long long>(c.u1 - c.u)));
      const int32_t* row = p.table + static_cast<long long>(c.b) * p.max_pages + c.u;
      for (int base = 0; base < n; base += 32) {
        const int mine = base + lane;
        int page = -1;
        if (mine < n && (c.u + mine) * p.P < c.s.len) {
          page = __ldg(row + mine);
          if (page < 0 || page >= p.num_pages) {
            atomicOr(p.err, kErrBadIndex);
            page = 0;
          }
        }
        const int m = min(32, n - base);
        for (int i = 0; i < m; ++i, ++it) {
          const int pg = __shfl_sync(0xFFFFFFFFu, page, i);
          const int st = it % stages;
          if (lane == 0) {
            if (it >= static_cast<uint32_t>(stages))
              mbar_wait_bounded(&sh.empty[st], (it / stages - 1) & 1, p.timeout_ns, p.err, &sh.abort);
            if (pg < 0 || sh.abort) {
              mbar_arrive(&sh.full[st]);  // no key in this unit
            } else {
              mbar_arrive_expect_tx(&sh.full[st], rec);
              bulk_load(ring + static_cast<size_t>(st) * rec,
                        p.pool + (static_cast<long long>(pg) * p.Hkv + c.h) * rec, rec, &sh.full[st]);
            }
          }
          __syncwarp();
        }
      }
      left -= n;
      if (left > 0) cursor_next<kRows>(p, p.P, c);
    }
    // copies in flight are all waited for by the consumers, whose waits are
    // bounded too; after a time-out this warp stays until they have landed
    if (*static_cast<volatile int*>(&sh.abort) && lane == 0)
      for (uint32_t k = it > static_cast<uint32_t>(stages) ? it - stages : 0; k < it; ++k)
        mbar_wait_bounded(&sh.full[k % stages], (k / stages) & 1, p.timeout_ns, p.err, nullptr);
    return;
  }

  // -------- consumers: warp w takes the stages w, w + 4, ...
  const int g = lane >> 2, c4 = lane & 3;
  Cursor c = cursor_at<kRows>(p, p.P, x0);
  uint32_t it = 0;
  long long left = x1 - x0;
  while (left > 0) {
    const int n = static_cast<int>(min(left, static_cast<long long>(c.u1 - c.u)));
    // rows g and g + 8 of the tile
    uint32_t qa[KS][4];
    float sc[2];
    int lo[2], hi[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int idx = c.tile * kRows + g + 8 * half;
      const bool have = idx < c.s.n * p.G;
      const int tok = idx / p.G;
      lo[half] = 0, hi[half] = c.s.len;  // a row that is not there masks nothing
      if (have) row_keys(p, c.s, tok, lo[half], hi[half]);
      uint32_t w[LD / 2];
#pragma unroll
      for (int i = 0; i < LD / 2; ++i) w[i] = 0;
      if (have) {
        const uint4* src = reinterpret_cast<const uint4*>(p.q + (c.s.q0 + tok) * p.q_stride +
                                                          (c.h * p.G + idx % p.G) * D + c4 * LD);
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
      // 2^14 <= largest * 2^e < 2^15
      const int e = min(14 + 127 - static_cast<int>(top >> 7), 120);
      const float up = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
      sc[half] = p.scale * kLog2e * __ldg(p.g_k + c.h) * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
      for (int i = 0; i < LD / 2; ++i) {
        const uint32_t h = pack_f16x2(__uint_as_float(w[i] << 16) * up, __uint_as_float(w[i] & 0xFFFF0000u) * up);
        qa[i >> 1][half + 2 * (i & 1)] = h;
      }
    }
    float o[NT][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
    // keys that every row of the tile sees
    int all_lo = max(lo[0], lo[1]), all_hi = min(hi[0], hi[1]);
#pragma unroll
    for (int s = 4; s < 32; s <<= 1) {
      all_lo = max(all_lo, __shfl_xor_sync(0xFFFFFFFFu, all_lo, s));
      all_hi = min(all_hi, __shfl_xor_sync(0xFFFFFFFFu, all_hi, s));
    }

    for (int i = 0; i < n; ++i, ++it) {
      if ((it & (kWarps - 1)) != static_cast<uint32_t>(warp)) continue;
      const int st = it % stages;
      mbar_wait_warp(&sh.full[st], (it / stages) & 1, p.timeout_ns, p.err, &sh.abort);
      const uint8_t* kc = ring + static_cast<size_t>(st) * rec;
      const uint8_t* ks = kc + codes_bytes(p.P, D);
      const uint8_t* vc = kc + rec / 2;
      const uint8_t* vs = vc + codes_bytes(p.P, D);
      const int key0 = (c.u + i) * p.P;
      const int keys = min(p.P, c.s.len - key0);
      for (int t0 = 0; t0 < keys; t0 += 32) {
        float s[4][4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.0f;
          const int tok = t0 + 8 * t + (g ^ ((g >> 1) & 1));
          uint32_t w[LD / 8];
          if (LD == 32) {
            const uint4 v = *reinterpret_cast<const uint4*>(kc + tok * (D / 2) + c4 * 16);
            w[0] = v.x, w[1] = v.y, w[2 % (LD / 8)] = v.z, w[3 % (LD / 8)] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(kc + tok * (D / 2) + c4 * 8);
            w[0] = v.x, w[1] = v.y;
          }
          uint32_t sb[2];
          if (LD == 32) {
            const uint32_t f = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(ks + tok * (D / 16) + 2 * c4));
            sb[0] = __byte_perm(f, f, 0x1010);
            sb[1] = __byte_perm(f, f, 0x3232);
          } else {
            const uint32_t f = e4m3x2_to_f16x2(ks[tok * (D / 16) + c4]);
            sb[0] = sb[1] = __byte_perm(f, f, 0x1010);
          }
#pragma unroll
          for (int j = 0; j < LD / 8; ++j) {
            uint32_t h[4];
            e2m1x8(w[j], h);
            const uint32_t f = sb[j >> 1];
#pragma unroll
            for (int q = 0; q < 4; ++q) h[q] = hmul2(h[q], f);
            mma_f16(s[t], qa[2 * j], h[0], h[1]);
            mma_f16(s[t], qa[2 * j + 1], h[2], h[3]);
          }
        }
        const int k0 = key0 + t0;
        const bool open = k0 >= all_lo && k0 + 32 <= all_hi;  // no key of these is masked for any row
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int half = q >> 1;
            float x = s[t][q] * sc[half];
            if (!open) {
              const int key = k0 + 8 * t + ((2 * c4 + (q & 1)) ^ (c4 & 1));
              if (key < lo[half] || key >= hi[half]) x = -INFINITY;
            }
            s[t][q] = x;
            top[half] = fmaxf(top[half], x);
          }
        float corr[2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          top[half] = fmaxf(top[half], __shfl_xor_sync(0xFFFFFFFFu, top[half], 1));
          top[half] = fmaxf(top[half], __shfl_xor_sync(0xFFFFFFFFu, top[half], 2));
          const float mn = fmaxf(m[half], top[half]);
          const float base = mn == -INFINITY ? 0.0f : mn;
          corr[half] = ex2(m[half] - base);
          m[half] = mn;
          l[half] *= corr[half];
          top[half] = base - p_shift(kRows);
        }
        uint32_t pa[2][4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          float e[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            e[q] = ex2(s[t][q] - top[q >> 1]);
            l[q >> 1] += e[q];
          }
          pa[t >> 1][2 * (t & 1)] = pack_f16x2(e[0], e[1]);
          pa[t >> 1][2 * (t & 1) + 1] = pack_f16x2(e[2], e[3]);
        }
        if (__any_sync(0xFFFFFFFFu, corr[0] != 1.0f || corr[1] != 1.0f)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            o[nt][0] *= corr[0], o[nt][1] *= corr[0];
            o[nt][2] *= corr[1], o[nt][3] *= corr[1];
          }
        }
        const bool tail = t0 + 32 > keys;  // some of these keys were never written
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
          uint32_t b[2][NT];
#pragma unroll
          for (int pr = 0; pr < 2; ++pr) {
            const int ta = t0 + 16 * kb + 8 * pr + ((2 * c4) ^ (c4 & 1)), tb = ta ^ 1;
            uint32_t sa = vs[ta * (D / 16) + (D == 128 ? g : g >> 1)], sb = vs[tb * (D / 16) + (D == 128 ? g : g >> 1)];
            if (tail) {
              if (ta >= keys) sa = 0;
              if (tb >= keys) sb = 0;
            }
            const uint32_t f = e4m3x2_to_f16x2(sa | (sb << 8));
            constexpr int W = D / 64;  // words of a key per lane
            uint32_t wa[W], wb[W];
            if (W == 2) {
              const uint2 va = *reinterpret_cast<const uint2*>(vc + ta * (D / 2) + 8 * g);
              const uint2 vb = *reinterpret_cast<const uint2*>(vc + tb * (D / 2) + 8 * g);
              wa[0] = va.x, wa[W - 1] = va.y, wb[0] = vb.x, wb[W - 1] = vb.y;
            } else {
              wa[0] = *reinterpret_cast<const uint32_t*>(vc + ta * (D / 2) + 4 * g);
              wb[0] = *reinterpret_cast<const uint32_t*>(vc + tb * (D / 2) + 4 * g);
            }
#pragma unroll
            for (int j = 0; j < W; ++j) {
              uint32_t even[4], odd[4];
              e2m1x8((wa[j] & 0x0F0F0F0Fu) | ((wb[j] << 4) & 0xF0F0F0F0u), even);
              e2m1x8(((wa[j] >> 4) & 0x0F0F0F0Fu) | (wb[j] & 0xF0F0F0F0u), odd);
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                b[pr][8 * j + 2 * q] = hmul2(even[q], f);
                b[pr][8 * j + 2 * q + 1] = hmul2(odd[q], f);
              }
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_f16(o[nt], pa[kb], b[0][nt], b[1][nt]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.empty[st]);
    }

    // -------- the four warps' results become one
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      l[half] += __shfl_xor_sync(0xFFFFFFFFu, l[half], 1);
      l[half] += __shfl_xor_sync(0xFFFFFFFFu, l[half], 2);
      if (c4 == 0) {
        sh.m[warp][g + 8 * half] = m[half];
        sh.l[warp][g + 8 * half] = l[half];
      }
      // lane's LD consecutive columns, 16-byte chunks moved so that the eight
      // lanes of a store phase hit different banks
      const int r = g + 8 * half;
#pragma unroll
      for (int v = 0; v < LD / 4; ++v) {
        float4 f;
        float* fp = reinterpret_cast<float*>(&f);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int col = 4 * v + q;  // of the lane's LD: column tile col % NT, second column of the pair from NT on
          fp[q] = o[col % NT][2 * half + col / NT];
        }
        const int chunk = (LD / 4) * c4 + v;
        *reinterpret_cast<float4*>(&sh.o[warp][r][4 * (chunk ^ ((c4 + 4 * (r & 1)) & (D / 4 - 1)))]) = f;
      }
    }
    named_bar_sync(1, 32 * kWarps);
    const bool whole = c.u == c.u0 && n == c.u1 - c.u0;
    const int rows = min(kRows, c.s.n * p.G - c.tile * kRows);
    const long long slot = 2ll * blockIdx.x + (c.u == c.u0 ? 1 : 0);
    constexpr int CH = D / 4;  // 16-byte chunks of a row
    for (int k = threadIdx.x; k < rows * CH; k += 32 * kWarps) {
      const int r = k / CH, q = k % CH;
      float mm = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sh.m[w][r]);
      const float base = mm == -INFINITY ? 0.0f : mm;
      float ll = 0.0f;
      float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      const int at = 4 * (q ^ ((q / (LD / 4) + 4 * (r & 1)) & (D / 4 - 1)));
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = exp2f(sh.m[w][r] - base);
        const float4 v = *reinterpret_cast<const float4*>(&sh.o[w][r][at]);
        ll += f * sh.l[w][r];
        a.x += f * v.x, a.y += f * v.y, a.z += f * v.z, a.w += f * v.w;
      }
      if (whole) {
        const int idx = c.tile * kRows + r;
        const long long row = static_cast<long long>(c.s.q0 + idx / p.G) * p.Hq + c.h * p.G + idx % p.G;
        const float inv = ll > 0.0f ? __ldg(p.g_v + c.h) / ll : 0.0f;
        *reinterpret_cast<uint2*>(p.out + row * D + 4 * q) =
            make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
        if (p.lse && q == 0) p.lse[row] = ll > 0.0f ? (mm + log2f(ll) - p_shift(kRows)) * (1.0f / kLog2e) : -INFINITY;
      } else {
        *reinterpret_cast<float4*>(p.part_o + (slot * kRows + r) * D + 4 * q) = a;
        if (q == 0) {
          p.part_ml[slot * 2 * kRows + r] = mm;
          p.part_ml[(slot * 2 + 1) * kRows + r] = ll;
        }
      }
    }
    named_bar_sync(1, 32 * kWarps);
    left -= n;
    if (left > 0) cursor_next<kRows>(p, p.P, c);
  }
}

constexpr int kRingBytes = 72 * 1024;

template <int D>
int launch_rows16(const AttnParams& p, cudaStream_t s) {
  const int rec = record_bytes(p.P, D);
  const int stages = std::min(kMaxStages, std::max(4, kRingBytes / rec));
  const int smem = static_cast<int>(round_up(sizeof(Shared<D>), 128)) + stages * rec;
  static int set[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MOE_ERR_CUDA;
  if (set[dev] < smem) {
    const cudaError_t e = cudaFuncSetAttribute(attn_rows16_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) {
      set_cuda_error(e);
      return MOE_ERR_CUDA;
    }
    set[dev] = smem;
  }
  attn_rows16_kernel<D><<<p.blocks, kThreads, smem, s>>>(p, stages);
  return check_launch();
}

// Schedule, main kernel, joining.
template <int ROWS, int D>
int run(const AttnParams& p, int unit, cudaStream_t s) {
  attn_plan_kernel<ROWS><<<1, 1024, 0, s>>>(p, unit);
  MOE_TRY(check_launch());
  MOE_TRY(ROWS == kRows ? launch_rows16<D>(p, s) : attention_tiles(p, D, s));
  if (p.blocks > 1) {
    attn_join_kernel<ROWS, D><<<dim3(p.blocks - 1, ROWS == kRows ? 4 : 16), 128, 0, s>>>(p, unit);
    MOE_TRY(check_launch());
  }
  return MOE_OK;
}

constexpr int kTileRows = kRowsTile, kTileKeys = 128;

struct Layout {
  int rows, blocks;
  size_t bytes;
};

// Kernel variant, its blocks, and the workspace they need; fills p's pointers.
Layout layout(AttnParams& p, int D, void* ws) {
  Layout r;
  // Up to 32 rows per sequence and kv head on average: 16 rows at a time.
  const bool tiles16 = static_cast<long long>(p.T) * p.G <= 32ll * p.B;
  r.rows = tiles16 ? kRows : kTileRows;
  r.blocks = tiles16 ? 2 * num_sms() : num_sms();
  Carve c(ws, 0);
  const long long tiles = static_cast<long long>(p.T) * p.G / r.rows + p.B + 1;
  p.starts = c.take<int>(p.B + 1);
  p.tile_base = c.take<int>(p.B + 1);
  p.unit_sum = c.take<long long>(tiles + 1);
  p.part_ml = c.take<float>(static_cast<size_t>(2) * r.blocks * 2 * r.rows);
  p.part_o = c.take<float>(static_cast<size_t>(2) * r.blocks * r.rows * D);
  p.blocks = r.blocks;
  p.min_units = tiles16 ? 1 : 2;
  r.bytes = c.used;
  return r;
}

}  // namespace

int attention(const AttnParams& p, int D, int rows, cudaStream_t s) {
  if (rows == kRows) return D == 128 ? run<kRows, 128>(p, p.P, s) : run<kRows, 64>(p, p.P, s);
  return D == 128 ? run<kTileRows, 128>(p, kTileKeys, s) : run<kTileRows, 64>(p, kTileKeys, s);
}

}  // namespace kv4
}  // namespace moe

using namespace moe;

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
  p.max_pages = max_pages, p.causal = causal, p.window = window, p.scale = scale;
  p.timeout_ns = wait_timeout_ns();
  p.err = device_error_word();
  if (!p.err) return MOE_ERR_CUDA;
  const kv4::Layout l = kv4::layout(p, D, ws);
  if (l.bytes > ws_bytes) return MOE_ERR_WORKSPACE;
  return kv4::attention(p, D, l.rows, static_cast<cudaStream_t>(stream));
}
