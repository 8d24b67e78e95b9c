// Verification of drafted tokens against the target's probabilities, from given
// random numbers, and the token behind the accepted ones.
//
// With p = softmax(logits / temperature) of a row and q the draft's probabilities,
// a drafted token x is accepted while u q(x) < p(x); behind the first refused one
// the next token is drawn from max(p - q, 0), behind none from p: the first index
// whose running sum passes u' times the whole.
//
// Which token that is must not depend on the order of sums.  So the weights
// 2^(log2(p) - log2(largest p)) are integers, multiples of 2^-40, formed by fp32
// pairs within 2^-26 of their value, and their sums are exact.  Bound: the logits,
// read once by the first launch, which makes fast fp32 sums of every row (within
// 2^-16 for 151936 words), enough to decide on a drafted token unless u q(x) is that near to p(x);
// the row in question is then summed in integers.  The second launch reads the one
// row per sequence that the next token comes from, and its draft probabilities;
// the last of a sequence's blocks finds the token.
//
// 64 sequences of up to seven drafts, 151936 words, bf16: 20 + 32 us on the GPU (the first
// launch 4.1 TB/s of the logits; the second 68 instructions per value, 0.38 of the issue
// slots, since it begins and ends with chains of dependent loads).  One sequence of four drafts: 4 + 14 us, the call with moe_kv_drop 43 - 46.
#include "kv4_attention.cuh"

namespace moe {
namespace {

using kv4::ex2;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kGroup = 8;                              // values of a lane at a time
constexpr int kLoads = 2;                              // groups of a lane in flight
constexpr int kChunk = kThreads * kGroup * kLoads;     // values of a row that a block of the first launch takes at a time
constexpr int kSub = 2 * 32 * kGroup;                  // whose sums the second launch writes down
static_assert(kSub == 2 * kThreads, "two values per thread");
// What the fast p(x) may be off at most, relative to it.  An exponent e: its three roundings,
// |e| 2^-22.9 of the weight; in the sum of up to 2^22 weights, the largest of them 1, 2^-18.8
// (17 |e| on average of the weight at most).  With 2^-22 per exponential, nine additions of
// a lane's chunk, the quotient and u q: kNear.  Each further step of a sum, a lane's next
// chunk or a join, rounds an exponential, a product and a sum: kNearStep.
constexpr float kNear = 0x1p-18f, kNearStep = 0x1.8p-22f, kNearExponent = 0x1p-22f;
constexpr int kBits = 40;                              // of a weight's fraction
constexpr float kLowest = -3.4028234663852886e38f;

struct Part {  // of a row: largest logit, its first index (greedy rows; else 0), sum of the weights relative to it
  float m, s;
  int idx, pad;
};
constexpr int kNone = 0x7FFFFFFF;  // index where no logit is a number
struct Sums {  // of kSub values: weights; weights and draft probabilities where p > q
  long long all, over, q;
};

struct Params {
  const void* logits;
  long long stride;
  const int32_t *tokens, *q_offsets;
  const float *u, *u_next, *probs;
  long long probs_stride;
  const float* temperature;
  int32_t *accepted, *token, *refused;
  int T, V, B;
  int chunks, chunk;    // blocks of a row in the first launch, values of each
  int subs, per_warp;
  float near;           // how far the fast p(x) may be off, its own exponent aside
  Part* parts;    // [T][chunks]
  Sums* sums;     // [B][subs]
  unsigned* done; // [B] blocks of the second launch that have written theirs
  unsigned int* err;
};

DEVINL int offset_at(const Params& p, int b) { return min(max(p.q_offsets[b], 0), p.T); }
// log2(e) / temperature as a pair, within 2^100 and 2^-100; 0: the largest logit has all weight.
struct Sharp {
  float hi, lo;
};
DEVINL Sharp sharpness(const Params& p, int b) {
  constexpr double kLog2e = 1.44269504088896340736;
  constexpr float L_hi = static_cast<float>(kLog2e), L_lo = static_cast<float>(kLog2e - static_cast<double>(L_hi));
  if (!p.temperature) return {L_hi, L_lo};
  const float t = p.temperature[b];
  if (!(t > 0.0f)) return {0.0f, 0.0f};
  const float c = L_hi / t;
  if (!(c > 0x1p-100f)) return {0x1p-100f, 0.0f};
  if (!(c < 0x1p100f)) return {0x1p100f, 0.0f};
  return {c, (fmaf(-c, t, L_hi) + L_lo) / t};
}
DEVINL bool greedy(const Params& p, int b) { return p.temperature && !(p.temperature[b] > 0.0f); }

// Elements in front of a row's first 16-byte boundary are counted from below 0:
// groups of eight then lie on such boundaries whatever the row's address.
template <class T>
DEVINL int lead_of(const T* row) { return static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T)); }

// Eight logits as they lie; what is not in [0, V) is -infinity.
template <class L>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint4 a;
};
template <>
struct Raw<float> {
  float4 a, b;
};
DEVINL Raw<__nv_bfloat16> load_raw(const __nv_bfloat16* row, int i, int V) {
  if (i >= 0 && i + kGroup <= V) return {*reinterpret_cast<const uint4*>(row + i)};
  uint32_t x[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int j = i + 2 * k;
    const uint32_t lo = j >= 0 && j < V ? __bfloat16_as_ushort(row[j]) : 0xFF80u;
    const uint32_t hi = j + 1 >= 0 && j + 1 < V ? __bfloat16_as_ushort(row[j + 1]) : 0xFF80u;
    x[k] = hi << 16 | lo;
  }
  return {make_uint4(x[0], x[1], x[2], x[3])};
}
DEVINL Raw<float> load_raw(const float* row, int i, int V) {
  if (i >= 0 && i + kGroup <= V)
    return {*reinterpret_cast<const float4*>(row + i), *reinterpret_cast<const float4*>(row + i + 4)};
  float x[kGroup];
#pragma unroll
  for (int k = 0; k < kGroup; ++k) x[k] = i + k >= 0 && i + k < V ? row[i + k] : -INFINITY;
  return {make_float4(x[0], x[1], x[2], x[3]), make_float4(x[4], x[5], x[6], x[7])};
}
DEVINL void expand(const Raw<__nv_bfloat16>& r, float (&v)[kGroup]) {
  const uint32_t x[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) v[2 * k] = __uint_as_float(x[k] << 16), v[2 * k + 1] = __uint_as_float(x[k] & 0xFFFF0000u);
}
DEVINL void expand(const Raw<float>& r, float (&v)[kGroup]) {
  v[0] = r.a.x, v[1] = r.a.y, v[2] = r.a.z, v[3] = r.a.w;
  v[4] = r.b.x, v[5] = r.b.y, v[6] = r.b.z, v[7] = r.b.w;
}
// not a number, or -infinity: -infinity, no weight (the lowest finite number has one, beside
// its equals); infinity: as the largest finite number
DEVINL float value_of(float v) { return fminf(fmaxf(v, -INFINITY), -kLowest); }
template <class L>
DEVINL void load_group(const L* row, int i, int V, float (&v)[kGroup]) {
  expand(load_raw(row, i, V), v);
#pragma unroll
  for (int e = 0; e < kGroup; ++e) v[e] = value_of(v[e]);
}
DEVINL float prob_of(float q) { return __saturatef(q); }  // not a number: 0
DEVINL void load_probs(const float* row, int i, int V, float (&q)[kGroup]) {
  if (i >= 0 && i + kGroup <= V && (reinterpret_cast<uintptr_t>(row + i) & 15) == 0) {
    const float4 a = *reinterpret_cast<const float4*>(row + i), b = *reinterpret_cast<const float4*>(row + i + 4);
    q[0] = prob_of(a.x), q[1] = prob_of(a.y), q[2] = prob_of(a.z), q[3] = prob_of(a.w);
    q[4] = prob_of(b.x), q[5] = prob_of(b.y), q[6] = prob_of(b.z), q[7] = prob_of(b.w);
  } else {
#pragma unroll
    for (int k = 0; k < kGroup; ++k) q[k] = i + k >= 0 && i + k < V ? prob_of(row[i + k]) : 0.0f;
  }
}

// ------------------------------------------------------------ fast sums of rows
DEVINL uint64_t twice(float v) { return kv4::pair(v, v); }
DEVINL uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
DEVINL void join(Part& a, const Part& b, float c) {
  if (b.m > a.m || (b.m == a.m && b.idx < a.idx)) a.idx = b.idx;
  const float m = fmaxf(a.m, b.m);
  a.s = a.s * ex2((a.m - m) * c) + b.s * ex2((b.m - m) * c);
  a.m = m;
}
DEVINL Part shuffle(const Part& a, int x) {
  return Part{__shfl_xor_sync(0xFFFFFFFFu, a.m, x), __shfl_xor_sync(0xFFFFFFFFu, a.s, x),
              __shfl_xor_sync(0xFFFFFFFFu, a.idx, x), 0};
}

// A lane's next values: their weights, or (TOP) the first index of the largest.
template <bool TOP, class L>
DEVINL void add_values(Part& a, const Raw<L> (&raw)[kLoads], int i0, float c) {
  float v[kLoads][kGroup], m = a.m;
#pragma unroll
  for (int k = 0; k < kLoads; ++k) {
    expand(raw[k], v[k]);
#pragma unroll
    for (int e = 0; e < kGroup; ++e) {
      if (TOP) v[k][e] = value_of(v[k][e]);  // (weights: where some sum is no number, see below)
      m = fmaxf(m, v[k][e]);
    }
  }
  if (TOP) {
    if (m > a.m || a.idx == kNone) {
#pragma unroll
      for (int k = kLoads - 1; k >= 0; --k)
#pragma unroll
        for (int e = kGroup - 1; e >= 0; --e)
          if (v[k][e] == m) a.idx = i0 + k * kThreads * kGroup + e;
    }
  } else {
    const uint64_t nm = twice(-m), cc = twice(c);
    uint64_t s = 0;
#pragma unroll
    for (int k = 0; k < kLoads; ++k)
#pragma unroll
      for (int e = 0; e < kGroup; e += 2) {
        float x0, x1;
        kv4::unpair(mul2(kv4::add2(kv4::pair(v[k][e], v[k][e + 1]), nm), cc), x0, x1);
        s = kv4::add2(s, kv4::pair(ex2(x0), ex2(x1)));
      }
    float s0, s1;
    kv4::unpair(s, s0, s1);
    a.s = a.s * ex2((a.m - m) * c) + (s0 + s1);
  }
  a.m = m;
}

template <class L>
__global__ void __launch_bounds__(kThreads, 5) verify_rows_kernel(const Params p) {
  __shared__ Part s_part[kWarps];
  kv4::launch_dependents();
  const int t = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const L* row = static_cast<const L*>(p.logits) + t * p.stride;
  Raw<L> next[kLoads];
  int i0 = blockIdx.x * p.chunk + threadIdx.x * kGroup - lead_of(row);
  const int begin = i0, end = min(p.V, (static_cast<int>(blockIdx.x) + 1) * p.chunk - lead_of(row));
#pragma unroll
  for (int k = 0; k < kLoads; ++k) next[k] = load_raw(row, i0 + k * kThreads * kGroup, p.V);
  if (t == 0 && blockIdx.x == 0)
    for (int b = threadIdx.x; b < p.B; b += kThreads) p.done[b] = 0;
  // the row's sequence: the last that begins at or before it
  int before = 0;
  for (int b0 = 0; b0 < p.B; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    before += __syncthreads_count(b < p.B && offset_at(p, b) <= t);
  }
  const int seq = max(before - 1, 0);
  const bool top = greedy(p, seq);
  const float c = sharpness(p, seq).hi;
  Part a{kLowest, 0.0f, kNone, 0};
  for (; i0 < end; i0 += kChunk) {
    Raw<L> now[kLoads];
#pragma unroll
    for (int k = 0; k < kLoads; ++k) now[k] = next[k];
    if (i0 + kChunk < end) {
#pragma unroll
      for (int k = 0; k < kLoads; ++k) next[k] = load_raw(row, i0 + kChunk + k * kThreads * kGroup, p.V);
    }
    if (top) add_values<true, L>(a, now, i0, c);
    else add_values<false, L>(a, now, i0, c);
  }
  if (a.s != a.s) {  // some logit is infinite or not a number: once more with what counts for it
    a.s = 0.0f, a.m = value_of(a.m);  // (kLowest or more)
    for (i0 = begin; i0 < end; i0 += kThreads * kGroup) {
      float v[kGroup];
      load_group(row, i0, p.V, v);
      for (int e = 0; e < kGroup; ++e) a.s += ex2((v[e] - a.m) * c);
    }
  }
  if (!top && a.s > 0.0f) a.idx = 0;  // the largest one's weight is 1
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) join(a, shuffle(a, x), c);
  if (lane == 0) s_part[warp] = a;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kWarps; ++w) join(a, s_part[w], c);
    p.parts[static_cast<long long>(t) * p.chunks + blockIdx.x] = a;
  }
}

// ---------------------------------------------------------------- exact weights
struct Exact {
  float m, c_hi, c_lo;  // largest logit, log2(e) / temperature as a pair
};
DEVINL uint64_t less2(uint64_t a, uint64_t b) { return kv4::fma2(b, twice(-1.0f), a); }  // a - b

// A number from 0 to 1 (and a rest below 2^-23) in multiples of 2^-40, as multiples of
// 2^-21 and of 2^-40 that are added up in 32 bits for up to 64 numbers.  Adding 6 or
// 1.5 * 2^-17 leaves the multiple in the low bits of the sum: no conversions, which
// take the time of four to sixteen additions.
struct Units {
  int hi, lo;
};
constexpr int kHi = kBits - 21;
constexpr int kOfHi = 0x40C00000, kOfLo = 0x37400000;  // the bits of 6 and 1.5 * 2^-17
DEVINL void units_of(uint64_t v, uint64_t rest, Units& u0, Units& u1) {
  const uint64_t m = kv4::add2(v, twice(6.0f));
  const uint64_t n = kv4::add2(kv4::add2(less2(v, kv4::add2(m, twice(-6.0f))), rest), twice(0x1.8p-17f));
  u0 = {static_cast<int>(m) - kOfHi, static_cast<int>(n) - kOfLo};
  u1 = {static_cast<int>(m >> 32) - kOfHi, static_cast<int>(n >> 32) - kOfLo};
}
DEVINL long long whole(const Units& u) { return (static_cast<long long>(u.hi) << kHi) + u.lo; }

// 2^((l - m) c) of two logits, off by 2^-26 of its value at most, and its multiple of
// 2^-40; 0 below 2^-42.  Pairs of fp32, without branches: the time of this is the
// launch's, and eight values' steps fill each other's gaps.
struct Weights {
  float w0, w1;
  Units u0, u1;
};
DEVINL Weights weights_of(float l0, float l1, const Exact& x) {
  using kv4::add2, kv4::fma2, kv4::pair;
  const uint64_t one = twice(1.0f), c = twice(x.c_hi);
  // l - m and its rounding error, times c
  const uint64_t l = pair(l0, l1), m = twice(x.m), d = less2(l, m), bv = less2(d, l);
  const uint64_t e = less2(less2(l, less2(d, bv)), add2(m, bv));
  const uint64_t na = mul2(d, twice(-x.c_hi));  // -a, a the product's first part
  const uint64_t a_lo = add2(fma2(d, c, na), fma2(d, twice(x.c_lo), mul2(e, c)));
  // a = n + f0, n the nearest whole number (in the low bits of `whole`); f = f0 + a_lo and its rest
  const uint64_t magic = twice(12582912.0f), whole_n = less2(magic, na);
  const uint64_t nf0 = add2(na, add2(whole_n, twice(-12582912.0f)));
  const uint64_t f = less2(a_lo, nf0), f_lo = less2(a_lo, add2(f, nf0));
  // 2^f = 1 + h + h^2/2 + ..., h = f ln 2, |h| <= 0.35, h_lo below 2^-25
  constexpr double kLn2 = 0.69314718055994530942;
  constexpr float L_hi = static_cast<float>(kLn2), L_lo = static_cast<float>(kLn2 - static_cast<double>(L_hi));
  const uint64_t h = mul2(f, twice(L_hi)), nh = mul2(f, twice(-L_hi));
  const uint64_t h_lo = add2(fma2(f, twice(L_hi), nh), fma2(f, twice(L_lo), mul2(f_lo, twice(L_hi))));
  uint64_t t = twice(1.0f / 362880.0f);
  t = fma2(t, h, twice(1.0f / 40320.0f));
  t = fma2(t, h, twice(1.0f / 5040.0f));
  t = fma2(t, h, twice(1.0f / 720.0f));
  t = fma2(t, h, twice(1.0f / 120.0f));
  t = fma2(t, h, twice(1.0f / 24.0f));
  t = fma2(t, h, twice(1.0f / 6.0f));
  t = fma2(t, h, twice(0.5f));
  // what is behind 1 + h; the sums' rounding errors (|h| > g) are exact
  const uint64_t g = fma2(mul2(h, h), t, fma2(h, h_lo, h_lo));
  const uint64_t v = add2(h, g), v_lo = less2(g, add2(v, nh));
  const uint64_t v1 = add2(one, v), rest = add2(less2(v, add2(v1, twice(-1.0f))), v_lo);
  const uint64_t pow = static_cast<uint64_t>((static_cast<uint32_t>(whole_n >> 32) << 23) + 0x3F800000u) << 32 |
                       ((static_cast<uint32_t>(whole_n) << 23) + 0x3F800000u);
  Weights w;
  const uint64_t value = mul2(v1, pow);
  units_of(value, mul2(rest, pow), w.u0, w.u1);
  kv4::unpair(value, w.w0, w.w1);
  float na0, na1;
  kv4::unpair(na, na0, na1);
  if (!(na0 < static_cast<float>(kBits + 2))) w.w0 = 0.0f, w.u0 = {0, 0};
  if (!(na1 < static_cast<float>(kBits + 2))) w.w1 = 0.0f, w.u1 = {0, 0};
  return w;
}
// a * b / 2^40, 0 <= a < 2^62, 0 <= b
DEVINL long long scaled(long long a, long long b) {
  return static_cast<long long>(__umul64hi(a, b) << (64 - kBits) | static_cast<unsigned long long>(a * b) >> kBits);
}
constexpr double kUnitInv = 1.0 / static_cast<double>(1ll << kBits);
DEVINL long long prob_units(float q) {  // q <= 1
  Units u, u1;
  units_of(twice(q), 0, u, u1);
  return whole(u);
}

DEVINL long long warp_sum(long long v) {
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, x);
  return v;
}

// Sum of a whole row's weights (a whole block calls it).
template <class L>
DEVINL long long row_sum(const L* row, int V, const Exact& x, long long* s_sum) {
  long long sum = 0;
  const int lead = lead_of(row);
  for (int i = threadIdx.x * kGroup - lead; i < V; i += kThreads * kGroup) {
    float v[kGroup];
    load_group(row, i, V, v);
#pragma unroll
    for (int e = 0; e < kGroup; e += 2) {
      const Weights w = weights_of(v[e], v[e + 1], x);
      sum += whole(w.u0) + whole(w.u1);
    }
  }
  sum = warp_sum(sum);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = sum;
  __syncthreads();
  sum = 0;
  for (int w = 0; w < kWarps; ++w) sum += s_sum[w];
  return sum;
}

// Running sums over a warp.
DEVINL long long scan(long long v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long up = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += up;
  }
  return v;
}
// Sum over the threads in front of this one, and over all (a whole block calls it).
// Not inlined, as little as possible is, behind the main loop: code that runs once
// comes from memory, some 200 cycles for eight instructions.
__device__ __noinline__ long long block_scan(long long v, long long* s_sum, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long incl = scan(v);
  __syncthreads();
  if (lane == 31) s_sum[warp] = incl;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll 1
  for (int w = 0; w < kWarps; ++w) {
    before = w == warp ? all : before;
    all += s_sum[w];
  }
  *total = all;
  return before + incl - v;
}
// The largest whole number at or below u * total (0 <= total < 2^62): a sum of whole
// numbers passes u * total if it passes that.
DEVINL long long part_of(float u, long long total) {
  if (!(u > 0.0f)) return 0;
  if (u >= 1.0f) return total;
  const uint32_t bits = __float_as_uint(u);
  const int e = max(static_cast<int>(bits >> 23), 1);
  const unsigned long long m = (bits & 0x7FFFFFu) | (bits >> 23 ? 0x800000u : 0u);  // u = m 2^(e - 150)
  const unsigned long long hi = __umul64hi(total, m), lo = static_cast<unsigned long long>(total) * m;
  const int down = 150 - e;  // 24 at least
  if (down >= 128) return 0;
  return static_cast<long long>(down >= 64 ? hi >> (down - 64) : hi << (64 - down) | lo >> down);
}

template <class L>
__global__ void __launch_bounds__(kThreads) verify_token_kernel(const Params p) {
  __shared__ Part s_row[kWarps];
  __shared__ int s_flag[kWarps];  // 0: refused, or behind the last; 1: accepted; 2: too near to tell
  __shared__ long long s_sum[kWarps];
  __shared__ unsigned s_last;
  __shared__ int s_pick, s_sub;
  __shared__ long long s_before;
  const int b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int first = offset_at(p, b), n = offset_at(p, b + 1) - first - 1;  // drafted tokens
  if (n < 0) {
    kv4::wait_for_previous();
    if (blockIdx.x == 0 && threadIdx.x == 0) p.accepted[b] = 0, p.refused[b] = 0, p.token[b] = -1;
    return;
  }
  const bool top = greedy(p, b);
  const Sharp sharp = sharpness(p, b);
  Exact x{0.0f, sharp.hi, sharp.lo};
  // the token behind row t, its logit, its q and its u
  struct Draft {
    int word;
    float l, q, u;
  };
  auto drafted = [&](int t) {
    Draft d{p.tokens[t + 1], -INFINITY, 0.0f, p.u[t + 1]};
    if (d.word >= 0 && d.word < p.V) {
      if (sizeof(L) == 2) d.l = __bfloat162float(static_cast<const __nv_bfloat16*>(p.logits)[t * p.stride + d.word]);
      else d.l = static_cast<const float*>(p.logits)[t * p.stride + d.word];
      d.l = value_of(d.l);
      d.q = p.probs ? prob_of(p.probs[t * p.probs_stride + d.word]) : 1.0f;
    }
    return d;
  };
  Draft mine{};  // of this warp's row, read while the first launch still runs
  if (lane == 0 && warp < n) mine = drafted(first + warp);
  kv4::wait_for_previous();

  // how many are accepted: a warp per row
  int stop = -1;
  Part at{};
  for (int i0 = 0; stop < 0; i0 += kWarps) {
    const int i = i0 + warp, t = first + i;
    if (i <= n) {
      Part a{kLowest, 0.0f, kNone, 0};
      for (int k = lane; k < p.chunks; k += 32) join(a, p.parts[static_cast<long long>(t) * p.chunks + k], x.c_hi);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) join(a, shuffle(a, o), x.c_hi);
      if (lane == 0) {
        int flag = 0;
        if (i < n) {
          const Draft d = i0 == 0 ? mine : drafted(t);
          if (d.word < 0 || d.word >= p.V) {
            if (blockIdx.x == 0) atomicOr(p.err, kErrBadIndex);
          } else {
            const float uq = d.u * d.q;
            if (top) {
              flag = d.word == a.idx && uq < 1.0f;
            } else if (d.l > kLowest || (d.l == kLowest && a.m == kLowest)) {  // (a mask, unless all are)
              // (far below 2^-100 p is still no 0)
              const float e = (d.l - a.m) * x.c_hi, pw = ex2(e) / a.s;
              if (uq == 0.0f) flag = 1;
              else if (e < -100.0f) flag = uq < 0x1p-80f ? 2 : 0;
              else flag = fabsf(uq - pw) <= (p.near + fabsf(e) * kNearExponent) * pw ? 2 : uq < pw;
            }
          }
        }
        s_row[warp] = a, s_flag[warp] = flag;
      }
    }
    __syncthreads();
    for (int k = 0; k < kWarps && i0 + k <= n && stop < 0; ++k) {
      int flag = s_flag[k];
      if (flag == 2) {
        const int row = first + i0 + k;
        const L* r = static_cast<const L*>(p.logits) + row * p.stride;
        x.m = s_row[k].m;
        const double z = static_cast<double>(row_sum(r, p.V, x, s_sum)) * kUnitInv;
        const Draft d = drafted(row);
        const double c = static_cast<double>(x.c_hi) + static_cast<double>(x.c_lo);
        flag = static_cast<double>(d.u) * static_cast<double>(d.q) * z <
               exp2((static_cast<double>(d.l) - static_cast<double>(x.m)) * c);
      }
      if (flag == 0) stop = i0 + k, at = s_row[k];
    }
    __syncthreads();
  }
  const int t = first + stop;
  const bool refused = stop < n;
  if (blockIdx.x == 0 && threadIdx.x == 0) p.accepted[b] = stop, p.refused[b] = n - stop;
  if (top || at.idx == kNone) {  // no logit that is a number: no token
    if (blockIdx.x == 0 && threadIdx.x == 0) {
      p.token[b] = at.idx == kNone ? -1 : at.idx;
      if (at.idx == kNone) atomicOr(p.err, kErrBadIndex);
    }
    return;
  }

  // the row's weights, kSub at a time
  x.m = at.m;
  const L* row = static_cast<const L*>(p.logits) + t * p.stride;
  const float* probs = refused && p.probs ? p.probs + t * p.probs_stride : nullptr;
  const int out = refused && !p.probs ? p.tokens[t + 1] : -1;  // a draft that was certain: its token has no weight left
  const int lead = lead_of(row);
  const float zq = static_cast<float>(at.s);
  // half of kSub values of a warp at a time, the next ones' loads in flight
  const int sub0 = (blockIdx.x * kWarps + warp) * p.per_warp, halves = 2 * max(0, min(p.per_warp, p.subs - sub0));
  const int base = sub0 * kSub + lane * kGroup - lead;
  constexpr int kStep = 32 * kGroup;
  Raw<L> next = load_raw(row, base, p.V);
  float next_q[kGroup];
  if (probs) load_probs(probs, base, p.V, next_q);
  Units all{0, 0}, over{0, 0}, sq{0, 0};
#pragma unroll 1
  for (int k = 0; k < halves; ++k) {
    const int i = base + k * kStep;
    float v[kGroup], q[kGroup];
    expand(next, v);
#pragma unroll
    for (int e = 0; e < kGroup; ++e) v[e] = value_of(v[e]), q[e] = probs ? next_q[e] : 0.0f;
    if (k + 1 < halves) {
      next = load_raw(row, i + kStep, p.V);
      if (probs) load_probs(probs, i + kStep, p.V, next_q);
    }
    float top_v = v[0];
#pragma unroll
    for (int e = 1; e < kGroup; ++e) top_v = fmaxf(top_v, v[e]);
    if (__any_sync(0xFFFFFFFFu, (top_v - x.m) * x.c_hi > -static_cast<float>(kBits + 3))) {
#pragma unroll
      for (int e = 0; e < kGroup; e += 2) {
        const Weights w = weights_of(v[e], v[e + 1], x);
        all.hi += w.u0.hi + w.u1.hi, all.lo += w.u0.lo + w.u1.lo;
        if (probs) {
          // p > q, by the fast sum: where that is wrong p - q is next to nothing
          Units q0, q1;
          units_of(kv4::pair(q[e], q[e + 1]), 0, q0, q1);
          if (w.w0 > q[e] * zq) over.hi += w.u0.hi, over.lo += w.u0.lo, sq.hi += q0.hi, sq.lo += q0.lo;
          if (w.w1 > q[e + 1] * zq) over.hi += w.u1.hi, over.lo += w.u1.lo, sq.hi += q1.hi, sq.lo += q1.lo;
        } else {
          if (i + e != out) over.hi += w.u0.hi, over.lo += w.u0.lo;
          if (i + e + 1 != out) over.hi += w.u1.hi, over.lo += w.u1.lo;
        }
      }
    }
    if (k & 1) {
      Sums s{warp_sum(whole(all)), warp_sum(whole(over)), 0};
      if (probs) s.q = warp_sum(whole(sq));
      if (lane == 0) p.sums[static_cast<long long>(b) * p.subs + sub0 + k / 2] = s;
      all = over = sq = {0, 0};
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    s_last = atomicAdd(p.done + b, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();

  // the last block: the whole, the kSub values that pass u' times it, the value
  const Sums* sums = p.sums + static_cast<long long>(b) * p.subs;
  const int per = (p.subs + kThreads - 1) / kThreads, k0 = min(p.subs, static_cast<int>(threadIdx.x) * per);
  const int k1 = min(p.subs, k0 + per);  // a thread's
  long long whole_row = 0, z;
  for (int k = k0; k < k1; ++k) whole_row += __ldcg(&sums[k].all);
  block_scan(whole_row, s_sum, &z);
  bool plain = false;  // nothing is left of p - q: by p
  auto sub_weight = [&](int k) -> long long {
    if (plain) return __ldcg(&sums[k].all);
    const long long over = __ldcg(&sums[k].over);
    return probs ? max(0ll, over - scaled(z, __ldcg(&sums[k].q))) : over;
  };
  long long total = 0, before = 0, own = 0;
#pragma unroll 1
  for (int pass = 0; pass < 2 && total == 0; ++pass) {
    plain = pass == 1;
    own = 0;
    for (int k = k0; k < k1; ++k) own += sub_weight(k);
    before = block_scan(own, s_sum, &total);
  }
  const long long limit = part_of(p.u_next[b], total);
  // the thread whose values pass the limit, or else the last that has any weight
  if (threadIdx.x == 0) s_pick = -1;
  __syncthreads();
  if (own > 0 && (before + own > limit ? before <= limit : before + own == total)) s_pick = threadIdx.x;
  __syncthreads();
  if (static_cast<int>(threadIdx.x) == s_pick) {
    int k = k0;
    for (long long w; k < k1 - 1 && before + (w = sub_weight(k)) <= limit; ++k) before += w;
    s_sub = k, s_before = before;
  }
  __syncthreads();
  if (s_pick < 0) {  // no weight at all
    if (threadIdx.x == 0) p.token[b] = 0;
    return;
  }
  // two of its values per thread
  const int i = s_sub * kSub + static_cast<int>(threadIdx.x) * 2 - lead;
  long long w[2], in_sub;
  float v[2], q[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const bool have = i + e >= 0 && i + e < p.V;
    v[e] = !have ? -INFINITY : value_of(sizeof(L) == 2 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(row)[i + e])
                                                     : reinterpret_cast<const float*>(row)[i + e]);
    q[e] = have && !plain && probs ? prob_of(probs[i + e]) : 0.0f;
  }
  const Weights both = weights_of(v[0], v[1], x);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    w[e] = whole(e ? both.u1 : both.u0);
    if (!plain && probs) w[e] = max(0ll, w[e] - scaled(z, prob_units(q[e])));
    if (!plain && i + e == out) w[e] = 0;
  }
  own = w[0] + w[1];
  before = s_before + block_scan(own, s_sum, &in_sub);
  // as above; where rounding has left nothing that passes the limit, the last with any weight
  if (threadIdx.x == 0) s_pick = -1;
  __syncthreads();
  if (own > 0 && (before + own > limit ? before <= limit : before + own == s_before + in_sub)) s_pick = threadIdx.x;
  __syncthreads();
  if (static_cast<int>(threadIdx.x) == max(s_pick, 0))
    p.token[b] = w[0] > 0 && (before + w[0] > limit || w[1] == 0) ? i : max(0, min(i + 1, p.V - 1));
}

int subs_of(int V) { return (V + 7 + kSub - 1) / kSub; }      // with a lead of 7
int chunks_of(int V) { return (V + 7 + kChunk - 1) / kChunk; }  // at most

size_t carve(Params& p, void* ws, int T, int V, int B) {
  Carve c(ws, 0);
  p.parts = c.take<Part>(static_cast<size_t>(T) * chunks_of(V));
  p.sums = c.take<Sums>(static_cast<size_t>(B) * subs_of(V));
  p.done = c.take<unsigned>(B);
  return c.used;
}

template <class L>
int launch(const Params& p, cudaStream_t s) {
  verify_rows_kernel<L><<<dim3(p.chunks, p.T), kThreads, 0, s>>>(p);
  MOE_TRY(check_launch());
  const int per_block = kWarps * p.per_warp;
  return kv4::launch_after(verify_token_kernel<L>, dim3((p.subs + per_block - 1) / per_block, p.B), kThreads, 0, s, p);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_verify_draft_workspace_size(int T, int V, int B) {
  if (T < 1 || V < 1 || B < 1 || V > (1 << 22) || T > 65535 || B > 65535) return 0;
  Params p;
  return carve(p, nullptr, T, V, B);
}

extern "C" int moe_verify_draft(const void* logits, int logits_f32, long long logits_stride, int T, int V,
                                const int32_t* tokens, const int32_t* q_offsets, int B, const float* u,
                                const float* u_next, const float* draft_probs, long long probs_stride,
                                const float* temperature, int32_t* accepted, int32_t* token, int32_t* refused, void* ws,
                                size_t ws_bytes, void* stream) {
  if (T < 0 || B < 0 || V < 1) return MOE_ERR_INVALID_ARG;
  if (V > (1 << 22) || T > 65535 || B > 65535) return MOE_ERR_UNSUPPORTED;
  if (B == 0) return MOE_OK;
  if (!q_offsets || !accepted || !token || !refused || !aligned(q_offsets, 4) || !aligned(accepted, 4) ||
      !aligned(token, 4) || !aligned(refused, 4))
    return MOE_ERR_INVALID_ARG;
  if (T == 0) {  // no sequence has a row
    Params p{};
    p.q_offsets = q_offsets, p.accepted = accepted, p.token = token, p.refused = refused, p.B = B, p.V = V;
    verify_token_kernel<float><<<dim3(1, B), kThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return check_launch();
  }
  if (!logits || !tokens || !u || !u_next || !aligned(logits, logits_f32 ? 4 : 2) || !aligned(tokens, 4) || !aligned(u, 4) ||
      !aligned(u_next, 4) || !aligned(draft_probs, 4) || !aligned(temperature, 4))
    return MOE_ERR_INVALID_ARG;
  if (T > 1 && (logits_stride < V || (draft_probs && probs_stride < V))) return MOE_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, 256)) return MOE_ERR_INVALID_ARG;
  Params p{logits, logits_stride, tokens, q_offsets, u, u_next, draft_probs, probs_stride, temperature, accepted, token,
           refused, T, V, B};
  p.subs = subs_of(V);
  if (ws_bytes < carve(p, ws, T, V, B)) return MOE_ERR_WORKSPACE;
  p.err = device_error_word();
  if (!p.err) return MOE_ERR_CUDA;
  // where rows are many a block takes several chunks of one, so that all run at once
  // (one / two / 38 blocks per row: 44 / 34 / 24 us for 5 rows, 74 / 65 / 73 for 276)
  const int most = chunks_of(V), split = std::max(1, std::min(most, num_sms() * 5 / T));
  p.chunk = (most + split - 1) / split * kChunk;
  p.chunks = (most * kChunk + p.chunk - 1) / p.chunk;
  // a lane's chunks, joins of a warp's lanes, of warps, of a row's chunks by a lane, of those lanes
  p.near = kNear + (p.chunk / kChunk + 5 + kWarps + (p.chunks + 31) / 32 + 5) * kNearStep;
  // a warp takes several parts of a row where there are more than a few rounds of them
  // (1 / 2 / 4 / 8: 24 / 28 / 32 / 42 us for one sequence, 69 / 67 / 71 / 95 for 64)
  p.per_warp = static_cast<int>(
      std::max<long long>(1, std::min<long long>(8, static_cast<long long>(B) * p.subs / (kWarps * num_sms() * 4))));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return logits_f32 ? launch<float>(p, s) : launch<__nv_bfloat16>(p, s);
}
