// Per-head RMS norms of queries and keys, the position rotation, and the
// NVFP4 write of keys and values into the paged cache, in one pass.
//
//   y = x * r * w,  r = 1 / sqrt(mean(x^2) + eps)        (per head, D values)
//   (a, b) -> (a cos - b sin, b cos + a sin)             (rot/2 pairs of y)
//
// Every operation is one IEEE rounding and the sum of squares is a fixed
// binary tree over neighbours, so a token's results, down to the cache's
// bytes, do not depend on the batch it came in or on the launch shape, and
// equal the elementary formula's bit for bit.
//
// Bound: HBM for many tokens.  16384 tokens of 64 + 4 heads of 128: 129 us, 4.6
// TB/s (0.67 of a copy), with 59 % of the issue slots taken; plain fp32
// instructions 175 us, packed pairs with four inverse roots side by side 129;
// 64 registers 132 us, 48 157, the next loads in flight during a step 129.  One
// token: 6 us, latency.
#include "kv4.cuh"

namespace moe {
namespace {

using kv4::add2, kv4::fma2, kv4::pair, kv4::unpair;

constexpr int kThreads = 256;
constexpr int kUnroll = 4;  // head groups in flight per warp

struct NormParams {
  const uint16_t *q, *k, *v;
  long long q_stride, k_stride, v_stride;  // elements between tokens
  int T, Hq, Hkv;
  const uint16_t *wq, *wk;  // null: no norm
  float eps;
  const float* cos_sin;  // [max_pos][rot]: cosines, then sines
  int max_pos, rot;
  const int32_t* pos;
  uint16_t *q_out, *k_out;
  uint8_t* pool;
  int num_pages, P;
  const float *g_k, *g_v;
  const long long* slots;
  int chunks;  // warps per token
  uint64_t neg_zero2;  // a pair of -0
  unsigned int* err;
};

// a * b + (-0): the product rounded once, with its sign.  The zero comes from
// the kernel's parameters because the assembler turns a constant one back into
// a product and then contracts packed products with sums.
DEVINL uint64_t mul2(uint64_t a, uint64_t b, uint64_t neg_zero) { return fma2(a, b, neg_zero); }

// A lane's 8 consecutive values (D/8 lanes per head) as pairs (0,2) (1,3) (4,6)
// (5,7): the sum's neighbours and an interleaved rotation's partners face each
// other in the two halves of two pairs.
struct Eight {
  uint64_t v[4];
};
DEVINL Eight from_bf16(const uint4& u) {
  auto lo = [](uint32_t w) { return __uint_as_float(w << 16); };
  auto hi = [](uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); };
  return Eight{{pair(lo(u.x), lo(u.y)), pair(hi(u.x), hi(u.y)), pair(lo(u.z), lo(u.w)), pair(hi(u.z), hi(u.w))}};
}
DEVINL Eight from_float(const float (&x)[8]) {
  return Eight{{pair(x[0], x[2]), pair(x[1], x[3]), pair(x[4], x[6]), pair(x[5], x[7])}};
}
DEVINL void to_float(const Eight& e, float (&x)[8]) {
  unpair(e.v[0], x[0], x[2]);
  unpair(e.v[1], x[1], x[3]);
  unpair(e.v[2], x[4], x[6]);
  unpair(e.v[3], x[5], x[7]);
}
DEVINL uint4 to_bf16(const Eight& e) {
  float x[8];
  to_float(e, x);
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

// Sum of squares of a head, neighbours first.
template <int D>
DEVINL float head_sum(const Eight& e, uint64_t nz) {
  const uint64_t a = add2(mul2(e.v[0], e.v[0], nz), mul2(e.v[1], e.v[1], nz));  // (0+1, 2+3)
  const uint64_t b = add2(mul2(e.v[2], e.v[2], nz), mul2(e.v[3], e.v[3], nz));
  float a0, a1, b0, b1;
  unpair(a, a0, a1);
  unpair(b, b0, b1);
  float t = __fadd_rn(__fadd_rn(a0, a1), __fadd_rn(b0, b1));
#pragma unroll
  for (int o = 1; o < D / 8; o <<= 1) t = __fadd_rn(t, __shfl_xor_sync(0xFFFFFFFFu, t, o));
  return t;
}

// Keeps a NaN: the scale of its block is one too, so that a key that is not a
// number does not turn into one.
DEVINL float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The lane's 8 values (half a block of 16; lanes 2j and 2j+1 share it) as
// NVFP4 with global scale g: returns the 8 codes, `s` the block's scale byte.
DEVINL uint32_t quantise8(const float (&v)[8], float g, uint32_t& s) {
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = max_nan(amax, fabsf(v[i]));
  amax = max_nan(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
  s = e4m3_encode_satfinite(__fdiv_rn(amax, __fmul_rn(6.0f, g)));
  const float denom = __fmul_rn(e4m3_decode(s), g);
  const float r = denom != 0.0f ? __frcp_rn(denom) : 0.0f;
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = denom != 0.0f ? e2m1_quotient(v[i], denom, r) : copysignf(0.0f, v[i]);
  return e2m1x8_rn_satfinite(q);
}

// What a lane needs of its token and place.
template <int D, bool PAIRS>
struct Lane {
  int l, sub;     // lane in the head, head in the warp's step
  bool turns;     // its values are rotated
  int partner;    // lane with the other half of its pairs
  Eight c, s;     // signed: y = x * c + partner * s for either half
  uint8_t* page;  // the token's page in the cache, or null
  int off;
};

// Norm, rotation and output of `n` <= U groups of heads from h0 on.  The
// inverse roots of U groups are formed side by side, one in each of four
// neighbouring lanes: an IEEE root and reciprocal cost as much as the rest.
template <int D, bool PAIRS, int U>
DEVINL void heads_step(const NormParams& p, const Lane<D, PAIRS>& L, const uint16_t* src, int h0, int n, int heads,
                       bool norm, const Eight& w, uint16_t* dst, bool cache) {
  constexpr int HPW = 256 / D;
  const int lane = threadIdx.x & 31;
  const uint64_t nz = p.neg_zero2;
  uint4 raw[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = h0 + u * HPW + L.sub;
    raw[u] = make_uint4(0, 0, 0, 0);
    if (u < n && h < heads) raw[u] = __ldcs(reinterpret_cast<const uint4*>(src + h * D + 8 * L.l));
  }
  float r[U];
  if (norm) {
    float mine = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float t = head_sum<D>(from_bf16(raw[u]), nz);
      if (U == 1 || (lane & (U - 1)) == u) mine = t;
    }
    mine = __frcp_rn(__fsqrt_rn(__fadd_rn(__fmul_rn(mine, 1.0f / D), p.eps)));
#pragma unroll
    for (int u = 0; u < U; ++u) r[u] = U == 1 ? mine : __shfl_sync(0xFFFFFFFFu, mine, (lane & ~(U - 1)) | u);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (u >= n) break;
    const int h = h0 + u * HPW + L.sub;
    Eight x = from_bf16(raw[u]);
    if (norm) {
      const uint64_t rr = pair(r[u], r[u]);
#pragma unroll
      for (int i = 0; i < 4; ++i) x.v[i] = mul2(mul2(x.v[i], rr, nz), w.v[i], nz);
    }
    if (p.rot > 0) {
      Eight y;
      if (PAIRS) {
        y = Eight{{x.v[1], x.v[0], x.v[3], x.v[2]}};
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) y.v[i] = __shfl_sync(0xFFFFFFFFu, x.v[i], L.partner);
      }
      if (L.turns) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x.v[i] = add2(mul2(x.v[i], L.c.v[i], nz), mul2(y.v[i], L.s.v[i], nz));
      }
    }
    const bool have = h < heads;
    if (dst != nullptr && have) *reinterpret_cast<uint4*>(dst + h * D + 8 * L.l) = to_bf16(x);
    if (cache) {
      float f[8];
      to_float(x, f);
      uint32_t sf;
      const uint32_t codes = quantise8(f, __ldg(p.g_k + min(h, heads - 1)), sf);
      if (have && L.page != nullptr) {
        uint8_t* sec = L.page + static_cast<long long>(h) * kv4::record_bytes(p.P, D);
        *reinterpret_cast<uint32_t*>(sec + L.off * (D / 2) + 4 * L.l) = codes;
        if ((L.l & 1) == 0) sec[kv4::codes_bytes(p.P, D) + L.off * (D / 16) + L.l / 2] = static_cast<uint8_t>(sf);
      }
    }
  }
}

template <int D, bool PAIRS>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const NormParams p) {
  constexpr int LPH = D / 8;     // lanes per head
  constexpr int HPW = 32 / LPH;  // heads per warp step
  const int lane = threadIdx.x & 31;
  Lane<D, PAIRS> L;
  L.l = lane % LPH, L.sub = lane / LPH;
  const int l = L.l;
  const long long wid = (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
  const int t = static_cast<int>(wid / p.chunks), chunk = static_cast<int>(wid % p.chunks);
  if (t >= p.T) return;

  const int nq = (p.Hq + HPW - 1) / HPW, nk = (p.Hkv + HPW - 1) / HPW;
  const int groups = nq + nk + (p.pool != nullptr ? nk : 0);
  const int g0 = static_cast<int>(static_cast<long long>(groups) * chunk / p.chunks);
  const int g1 = static_cast<int>(static_cast<long long>(groups) * (chunk + 1) / p.chunks);

  float c[8], s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    c[i] = 1.0f;
    s[i] = 0.0f;
  }
  const int half = p.rot / 2, hl = half / 8;  // pairs, and lanes that hold the first half
  L.turns = 8 * l < p.rot;
  if (L.turns) {
    int at = __ldg(p.pos + t);
    if (at < 0 || at >= p.max_pos) {
      if (l == 0 && chunk == 0) atomicOr(p.err, kErrBadIndex);
      at = max(0, min(at, p.max_pos - 1));
    }
    const float* row = p.cos_sin + static_cast<long long>(at) * p.rot;
    if (PAIRS) {
      const float4 cc = __ldg(reinterpret_cast<const float4*>(row + 4 * l));
      const float4 ss = __ldg(reinterpret_cast<const float4*>(row + half + 4 * l));
      const float cv[4] = {cc.x, cc.y, cc.z, cc.w}, sv[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c[2 * i] = c[2 * i + 1] = cv[i];
        s[2 * i] = -sv[i];
        s[2 * i + 1] = sv[i];
      }
    } else {
      const int j = 8 * (l < hl ? l : l - hl);
      const float sign = l < hl ? -1.0f : 1.0f;
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const float4 cc = __ldg(reinterpret_cast<const float4*>(row + j) + v);
        const float4 ss = __ldg(reinterpret_cast<const float4*>(row + half + j) + v);
        c[4 * v] = cc.x, c[4 * v + 1] = cc.y, c[4 * v + 2] = cc.z, c[4 * v + 3] = cc.w;
        s[4 * v] = sign * ss.x, s[4 * v + 1] = sign * ss.y, s[4 * v + 2] = sign * ss.z, s[4 * v + 3] = sign * ss.w;
      }
    }
  }
  L.c = from_float(c), L.s = from_float(s);
  L.partner = L.sub * LPH + (!L.turns ? l : l < hl ? l + hl : l - hl);
  L.page = nullptr, L.off = 0;
  if (p.pool != nullptr && g1 > nq) {
    const long long slot = __ldg(p.slots + t);
    if (slot >= static_cast<long long>(p.num_pages) * p.P) {
      if (lane == 0) atomicOr(p.err, kErrBadIndex);
    } else if (slot >= 0) {
      L.page = p.pool + (slot / p.P) * p.Hkv * kv4::record_bytes(p.P, D);
      L.off = static_cast<int>(slot % p.P);
    }
  }

  const Eight one = Eight{{0, 0, 0, 0}};
  if (g0 < nq) {
    const Eight w = p.wq ? from_bf16(__ldg(reinterpret_cast<const uint4*>(p.wq + 8 * l))) : one;
    const uint16_t* src = p.q + t * p.q_stride;
    uint16_t* dst = p.q_out + static_cast<long long>(t) * p.Hq * D;
    for (int g = g0; g < min(g1, nq); g += kUnroll)
      heads_step<D, PAIRS, kUnroll>(p, L, src, g * HPW, min(g1, nq) - g, p.Hq, p.wq != nullptr, w, dst, false);
  }
  if (g1 > nq && g0 < nq + nk) {
    const Eight w = p.wk ? from_bf16(__ldg(reinterpret_cast<const uint4*>(p.wk + 8 * l))) : one;
    const uint16_t* src = p.k + t * p.k_stride;
    uint16_t* dst = p.k_out ? p.k_out + static_cast<long long>(t) * p.Hkv * D : nullptr;
    const int first = max(g0, nq) - nq, last = min(g1 - nq, nk);
    for (int g = first; g < last; g += 2)
      heads_step<D, PAIRS, 2>(p, L, src, g * HPW, last - g, p.Hkv, p.wk != nullptr, w, dst, p.pool != nullptr);
  }
  // values: two groups of heads at a time
  for (int g = max(g0 - nq - nk, 0); g < g1 - nq - nk; g += 2) {
    const uint16_t* src = p.v + t * p.v_stride;
    uint4 raw[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int h = (g + u) * HPW + L.sub;
      raw[u] = make_uint4(0, 0, 0, 0);
      if (g + u < g1 - nq - nk && h < p.Hkv) raw[u] = __ldcs(reinterpret_cast<const uint4*>(src + h * D + 8 * l));
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (g + u >= g1 - nq - nk) break;
      const int h = (g + u) * HPW + L.sub;
      float x[8];
      to_float(from_bf16(raw[u]), x);
      uint32_t sf;
      const uint32_t codes = quantise8(x, __ldg(p.g_v + min(h, p.Hkv - 1)), sf);
      if (h < p.Hkv && L.page != nullptr) {
        uint8_t* sec = L.page + static_cast<long long>(h) * kv4::record_bytes(p.P, D) + kv4::record_bytes(p.P, D) / 2;
        *reinterpret_cast<uint32_t*>(sec + L.off * (D / 2) + 4 * l) = codes;
        if ((l & 1) == 0) sec[kv4::codes_bytes(p.P, D) + L.off * (D / 16) + l / 2] = static_cast<uint8_t>(sf);
      }
    }
  }
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_qk_norm_rope(const uint16_t* q, long long q_stride, const uint16_t* k, long long k_stride,
                                const uint16_t* v, long long v_stride, int T, int Hq, int Hkv, int D,
                                const uint16_t* wq, const uint16_t* wk, float eps, const float* cos_sin, int max_pos,
                                int rot, int interleaved, const int32_t* pos, uint16_t* q_out, uint16_t* k_out,
                                uint8_t* pool, int num_pages, int page_size, const float* g_k, const float* g_v,
                                const long long* slots, void* stream) {
  if (T < 0 || Hq < 1 || Hkv < 1 || rot < 0 || max_pos < 0) return MOE_ERR_INVALID_ARG;
  if (!kv4::head_dim_ok(D) || Hq > 1024 || Hkv > 1024 || T >= (1 << 24)) return MOE_ERR_UNSUPPORTED;
  if (rot > D || rot % 16 != 0) return MOE_ERR_UNSUPPORTED;
  if (pool != nullptr && !kv4::page_size_ok(page_size)) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!q || !k || !q_out || (!k_out && !pool)) return MOE_ERR_INVALID_ARG;
  if (rot > 0 && (!cos_sin || !pos || max_pos < 1)) return MOE_ERR_INVALID_ARG;
  if (pool && (!v || !g_k || !g_v || !slots || num_pages < 1)) return MOE_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(wq, 16) || !aligned(wk, 16) ||
      !aligned(cos_sin, 16) || !aligned(q_out, 16) || !aligned(k_out, 16) || !aligned(pool, 16) || !aligned(pos, 4) ||
      !aligned(slots, 8) || !aligned(g_k, 4) || !aligned(g_v, 4))
    return MOE_ERR_INVALID_ARG;
  if (q_stride % 8 || k_stride % 8 || q_stride < static_cast<long long>(Hq) * D ||
      k_stride < static_cast<long long>(Hkv) * D || (pool && (v_stride % 8 || v_stride < static_cast<long long>(Hkv) * D)))
    return MOE_ERR_INVALID_ARG;
  NormParams p{q, k, v, q_stride, k_stride, v_stride, T, Hq, Hkv, wq, wk, eps, cos_sin, max_pos, rot, pos, q_out, k_out,
               pool, num_pages, page_size, g_k, g_v, slots, 1, 0x8000000080000000ull, device_error_word()};
  if (!p.err) return MOE_ERR_CUDA;
  const int hpw = 256 / D;
  const int groups = (Hq + hpw - 1) / hpw + (pool ? 2 : 1) * ((Hkv + hpw - 1) / hpw);
  // one warp per token where that fills the GPU, else a token's heads over several warps
  const int want = num_sms() * 32;
  p.chunks = std::max(1, std::min(groups, (want + T - 1) / T));
  const long long warps = static_cast<long long>(T) * p.chunks;
  const unsigned blocks = static_cast<unsigned>((warps * 32 + kThreads - 1) / kThreads);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (D == 128) {
    if (interleaved) qk_norm_rope_kernel<128, true><<<blocks, kThreads, 0, s>>>(p);
    else qk_norm_rope_kernel<128, false><<<blocks, kThreads, 0, s>>>(p);
  } else {
    if (interleaved) qk_norm_rope_kernel<64, true><<<blocks, kThreads, 0, s>>>(p);
    else qk_norm_rope_kernel<64, false><<<blocks, kThreads, 0, s>>>(p);
  }
  return check_launch();
}
