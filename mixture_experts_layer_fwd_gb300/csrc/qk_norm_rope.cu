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
#include "kv4.cuh"

namespace moe {
namespace {

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
  unsigned int* err;
};

// 8 values of one head per lane, D/8 lanes per head.
template <int D>
DEVINL float head_sum(const float (&x)[8]) {
  float s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = __fmul_rn(x[i], x[i]);
#pragma unroll
  for (int w = 4; w > 0; w >>= 1)
#pragma unroll
    for (int i = 0; i < w; ++i) s[i] = __fadd_rn(s[2 * i], s[2 * i + 1]);
  float t = s[0];
#pragma unroll
  for (int o = 1; o < D / 8; o <<= 1) t = __fadd_rn(t, __shfl_xor_sync(0xFFFFFFFFu, t, o));
  return t;
}

DEVINL void unpack8(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// The lane's 8 values (half a block of 16; lanes 2j and 2j+1 share it) as
// NVFP4 with global scale g: returns the 8 codes, `s` the block's scale byte.
DEVINL uint32_t quantise8(const float (&v)[8], float g, uint32_t& s) {
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
  amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
  s = e4m3_encode_satfinite(__fdiv_rn(amax, __fmul_rn(6.0f, g)));
  const float denom = __fmul_rn(e4m3_decode(s), g);
  const float r = denom != 0.0f ? __frcp_rn(denom) : 0.0f;
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = denom != 0.0f ? e2m1_quotient(v[i], denom, r) : copysignf(0.0f, v[i]);
  return e2m1x8_rn_satfinite(q);
}

template <int D, bool PAIRS>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const NormParams p) {
  constexpr int LPH = D / 8;     // lanes per head
  constexpr int HPW = 32 / LPH;  // heads per warp step
  const int lane = threadIdx.x & 31;
  const int l = lane % LPH, sub = lane / LPH;
  const long long wid = (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
  const int t = static_cast<int>(wid / p.chunks), chunk = static_cast<int>(wid % p.chunks);
  if (t >= p.T) return;

  const int nq = (p.Hq + HPW - 1) / HPW, nk = (p.Hkv + HPW - 1) / HPW;
  const int groups = nq + nk + (p.pool != nullptr ? nk : 0);
  const int g0 = static_cast<int>(static_cast<long long>(groups) * chunk / p.chunks);
  const int g1 = static_cast<int>(static_cast<long long>(groups) * (chunk + 1) / p.chunks);

  // this lane's rotation: signed so that y = x * c + partner * s for either half
  float c[8], s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    c[i] = 1.0f;
    s[i] = 0.0f;
  }
  const int half = p.rot / 2, hl = half / 8;  // pairs, and lanes that hold the first half
  const bool turns = 8 * l < p.rot;
  if (turns) {
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
  const int partner = sub * LPH + (!turns ? l : l < hl ? l + hl : l - hl);

  uint8_t* page = nullptr;
  int off = 0;
  if (p.pool != nullptr && g1 > nq) {
    const long long slot = __ldg(p.slots + t);
    if (slot >= static_cast<long long>(p.num_pages) * p.P) {
      if (lane == 0) atomicOr(p.err, kErrBadIndex);
    } else if (slot >= 0) {
      page = p.pool + (slot / p.P) * p.Hkv * kv4::record_bytes(p.P, D);
      off = static_cast<int>(slot % p.P);
    }
  }

  for (int g = g0; g < g1; g += kUnroll) {
    uint4 raw[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      raw[u] = make_uint4(0, 0, 0, 0);
      const int gu = g + u;
      if (gu >= g1) continue;
      const int kind = gu < nq ? 0 : gu < nq + nk ? 1 : 2;
      const int h = (gu - (kind == 0 ? 0 : kind == 1 ? nq : nq + nk)) * HPW + sub;
      const uint16_t* src = kind == 0 ? p.q + t * p.q_stride : kind == 1 ? p.k + t * p.k_stride : p.v + t * p.v_stride;
      if (h < (kind == 0 ? p.Hq : p.Hkv)) raw[u] = *reinterpret_cast<const uint4*>(src + h * D + 8 * l);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int gu = g + u;
      if (gu >= g1) break;
      const int kind = gu < nq ? 0 : gu < nq + nk ? 1 : 2;
      const int h = (gu - (kind == 0 ? 0 : kind == 1 ? nq : nq + nk)) * HPW + sub;
      const bool have = h < (kind == 0 ? p.Hq : p.Hkv);
      float x[8];
      unpack8(raw[u], x);
      if (kind < 2) {
        const uint16_t* w = kind == 0 ? p.wq : p.wk;
        if (w != nullptr) {
          const float r = __frcp_rn(__fsqrt_rn(__fadd_rn(__fmul_rn(head_sum<D>(x), 1.0f / D), p.eps)));
          float wf[8];
          unpack8(__ldg(reinterpret_cast<const uint4*>(w + 8 * l)), wf);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = __fmul_rn(__fmul_rn(x[i], r), wf[i]);
        }
        if (p.rot > 0) {
          float y[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = PAIRS ? x[i ^ 1] : __shfl_sync(0xFFFFFFFFu, x[i], partner);
          if (turns) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __fadd_rn(__fmul_rn(x[i], c[i]), __fmul_rn(y[i], s[i]));
          }
        }
        uint16_t* dst = kind == 0 ? p.q_out : p.k_out;
        if (dst != nullptr && have) {
          dst += (static_cast<long long>(t) * (kind == 0 ? p.Hq : p.Hkv) + h) * D + 8 * l;
          *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                      pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
        }
      }
      if (kind > 0 && p.pool != nullptr) {
        uint32_t sf;
        const float gs = __ldg((kind == 1 ? p.g_k : p.g_v) + min(h, p.Hkv - 1));
        const uint32_t codes = quantise8(x, gs, sf);
        if (have && page != nullptr) {
          uint8_t* sec = page + static_cast<long long>(h) * kv4::record_bytes(p.P, D) +
                         (kind == 2 ? kv4::record_bytes(p.P, D) / 2 : 0);
          *reinterpret_cast<uint32_t*>(sec + off * (D / 2) + 4 * l) = codes;
          if ((l & 1) == 0) sec[kv4::codes_bytes(p.P, D) + off * (D / 16) + l / 2] = static_cast<uint8_t>(sf);
        }
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
               pool, num_pages, page_size, g_k, g_v, slots, 1, device_error_word()};
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
