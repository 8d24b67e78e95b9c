// Matrix-vector products of a decoding step: up to 32 tokens times a matrix in
// NVFP4,
//   y[t][n] = g * sum_k x[t][k] e2m1(w[n][k]) e4m3(s[n][k/16])  (+ add[t][n]).
//
// Bound: the matrix's bytes, 9/16 per weight, read once; from about 16 tokens on the
// 16 x 8 x 16 matrix instructions (8.5 cycles each per quarter of an SM) and the operands'
// way from shared memory too.
//
// The tokens lie in shared memory as fp16 in the order of the operand registers; sixteen
// of them or fewer each block brings there itself, more a launch of their own prepares.
// A block's warps are RW row tiles of 32 matrix rows times KW parts of the reduction;
// where there are few rows, or the tokens are too many for one block's shared memory,
// the blocks of a cluster take parts of the reduction as well.  Row tiles are dealt out
// to the blocks one by one.  Parts are joined in shared memory, in a fixed order.
//
// A warp's step is 32 rows times 256 values, copied by tensor maps (128-byte rows of
// codes, swizzled, and 16 bytes of scales, by a lane of the warp into a ring of its own).
// Tokens that do not fit beside the rings come in chunks, one while another is used.
// Where K % 256 != 0 the scales have no tensor map, and where rows are few the tokens
// have no room beside the rings: steps of 128 values, straight into registers, two in
// flight.
//
// On the GPU alone (matrices in turn, none in L2): 1 token 1024 x 4096 6.0 us, 5 tokens
// 9216 x 4096 11.0 us, 16 tokens 4096 x 8192 16 us, 1 / 8 / 24 / 32 tokens 151936 x 4096
// 62 / 66 / 100 / 121 us (5.6 / 5.3 / 3.5 / 2.9 TB/s).  Registers instead of rings 78 /
// 82 / 132 / 134 us there, 7.1 against 6.7 us for 1 token 4096 x 4096.
#include <cmath>

#include "nvfp4_mma.cuh"

namespace moe {
namespace {

constexpr int kMaxTokens = 32;
constexpr int kRows = 32;                // matrix rows of a warp's tile
template <bool MAP>
struct Cfg {
  static constexpr int kWarps = 16, kThreads = 32 * kWarps;
  static constexpr int kStep = MAP ? 256 : 128;  // values of a row per step
  static constexpr int kUnits = kStep / 8;       // of a token: 16 bytes
};
constexpr int kSlots = 4;                // of a warp's ring, at most
constexpr int kSlotCodes = kRows * 128, kSlotScales = kRows * 16;
constexpr int kMaxCluster = 4;
constexpr int kRed = kRows + 4;          // of a warp's sums of a token: their lanes in different banks
constexpr int kSmem = 225 * 1024;

struct Params {
  const uint16_t* x;
  long long x_stride;
  const uint8_t *w, *sf;
  const float* g;
  const uint16_t* add;
  long long add_stride;
  void* out;
  int T, N, K, out_f32;
  int tiles, steps;  // of 32 rows; of a row
  int kw, ck;        // warps of a block, and blocks of a cluster, along the reduction
  int sets;          // blocks, or clusters of them, that have row tiles of their own
  int slab;          // steps of a block
  int chunk;         // steps whose tokens are in shared memory at a time (a multiple of kw)
  int slots;         // of each warp's ring
  // workspace
  int* exps;         // [T] each token's power of two
  uint4* units;      // [T][steps][units of a step] tokens in the order of the operand registers
  unsigned int* err;
  unsigned long long timeout_ns;
};
struct Maps {
  CUtensorMap codes, scales;
};

// Codes and scales of a lane's part of a step: rows g, g + 8, g + 16, g + 24.
struct Piece {
  uint4 c[4];
  uint32_t s[4];
};
DEVINL uint4 load_stream(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
DEVINL void load_piece(const Params& p, int row0, int step, Piece& d) {
  const int lane = threadIdx.x & 31;
  const int k = step * Cfg<false>::kStep + (lane & 3) * 32;  // K % 32 == 0: all of the lane's values are there, or none
  const int at = k < p.K ? k : 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = min(row0 + (lane >> 2) + 8 * i, p.N - 1);
    d.c[i] = load_stream(p.w + static_cast<long long>(row) * (p.K / 2) + at / 2);
    d.s[i] = __ldg(reinterpret_cast<const uint16_t*>(p.sf + static_cast<long long>(row) * (p.K / 16) + at / 16));
    if (k >= p.K) d.s[i] = 0;
  }
}

// A token's units lie step after step; in a step, unit v of lane quarter c (its v-th eight
// values) is at 4 v + c.  In shared memory a token's room is 4 units more than its steps',
// so that two tokens' quarters lie in different banks.
template <bool MAP>
__host__ __device__ constexpr int token_units(int steps) { return steps * Cfg<MAP>::kUnits + 4; }
template <bool MAP>
DEVINL int unit_at(int u) {  // of the values from 8 u on
  return MAP ? (u & ~31) + 4 * (u & 7) + (u >> 3 & 3) : (u & ~15) + 4 * (u & 3) + (u >> 2 & 3);
}

// A block per token.
constexpr int kPrepThreads = 512;
template <bool MAP>
__global__ void __launch_bounds__(kPrepThreads) linear_prepare_kernel(const Params p) {
  __shared__ uint32_t s_top;
  kv4::launch_dependents();
  const int t = blockIdx.x, units = p.steps * Cfg<MAP>::kUnits;
  const uint4* x = reinterpret_cast<const uint4*>(p.x + t * p.x_stride);
  if (threadIdx.x == 0) s_top = 0;
  __syncthreads();
  uint32_t top = 0;
  for (int u = threadIdx.x; u < p.K / 8; u += kPrepThreads) top = max(top, bf16x8_top(__ldg(x + u)));
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  if ((threadIdx.x & 31) == 0) atomicMax(&s_top, top);
  __syncthreads();
  const int e = f16_exponent(s_top);
  if (threadIdx.x == 0) p.exps[t] = e;
  uint4* to = p.units + static_cast<long long>(t) * units;
  for (int u = threadIdx.x; u < units; u += kPrepThreads) {
    const uint4 v = u < p.K / 8 ? __ldg(x + u) : make_uint4(0, 0, 0, 0);
    to[unit_at<MAP>(u)] = bf16x8_to_f16x8(v, power_of_two(e));
  }
}

// Few tokens: a block brings them into place itself, a launch less (with the call, 1 token
// 1024 x 4096 14 against 19 us, 16 tokens 4096 x 8192 18.6 against 19.8, although the GPU
// alone takes 1 us more there: every block reads all tokens).  They are read once: bf16
// as it lies goes to its place, and when the largest value of each token is known (of the
// values that the block has) a thread brings its own units to fp16 there.
constexpr int kInline = 16, kInlineK = 16384;
template <bool MAP>
DEVINL void stage(const Params& p, uint4* xs, int* s_exp, uint32_t* s_top, int k0, int n) {
  const int units = n * Cfg<MAP>::kUnits, total = units * p.T;
  constexpr int kLanes = Cfg<MAP>::kUnits;  // side by side that have the same token (a multiple of these is all there is)
  static_assert(kLanes == 16 || kLanes == 32, "half of a warp, or one");
  const int lane = threadIdx.x & 31;
  const uint32_t same = kLanes == 32 ? 0xFFFFFFFFu : 0xFFFFu << (lane & 16);
  constexpr int kBatch = 5;  // loads of a thread in flight
#pragma unroll 1
  for (int i0 = threadIdx.x; i0 < total; i0 += kBatch * Cfg<MAP>::kThreads) {
    uint4 v[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int i = i0 + b * Cfg<MAP>::kThreads, t = i / units, k = k0 * Cfg<MAP>::kStep + 8 * (i % units);
      v[b] = i < total && k < p.K ? __ldg(reinterpret_cast<const uint4*>(p.x + t * p.x_stride + k)) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int i = i0 + b * Cfg<MAP>::kThreads, t = i / units;
      if (i >= total) break;
      xs[t * token_units<MAP>(p.slab) + unit_at<MAP>(i % units)] = v[b];
      const uint32_t top = __reduce_max_sync(same, bf16x8_top(v[b]));
      if (lane % kLanes == 0) atomicMax(s_top + t, top);
    }
  }
  __syncthreads();
  if (static_cast<int>(threadIdx.x) < p.T) s_exp[threadIdx.x] = f16_exponent(s_top[threadIdx.x]);
#pragma unroll 1
  for (int i = threadIdx.x; i < total; i += Cfg<MAP>::kThreads) {
    const int t = i / units;
    uint4& unit = xs[t * token_units<MAP>(p.slab) + unit_at<MAP>(i % units)];
    unit = bf16x8_to_f16x8(unit, power_of_two(f16_exponent(s_top[t])));
  }
}

DEVINL void store_remote(uint32_t cluster_addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_addr), "f"(v) : "memory");
}

template <int NT, bool INLINE, bool MAP>
__global__ void __launch_bounds__(Cfg<MAP>::kThreads, 1) linear_kernel(const Params p, const __grid_constant__ Maps maps) {
  constexpr int kWarps = Cfg<MAP>::kWarps, kThreads = Cfg<MAP>::kThreads, kUnits = Cfg<MAP>::kUnits;
  constexpr auto token_units = moe::token_units<MAP>;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __shared__ uint64_t s_bar[kWarps][kSlots];
  __shared__ int s_abort;
  __shared__ int s_exp[kMaxTokens];
  __shared__ uint32_t s_top[kMaxTokens];
  __shared__ uint64_t s_full[2];
  __shared__ int s_copied[2];      // uses of a buffer of tokens
  __shared__ int s_first, s_left;  // MAP: first step of the next chunk of tokens, and how many there are (not in registers, which are few)
  const int rw = kWarps / p.kw, rows = rw * kRows, room = min(p.chunk, p.slab);
  // MAP: the rings; tokens; KW > 1: the warps' sums; clusters: the blocks' sums of this block's share, twice
  uint8_t* codes = smem_raw + (MAP ? -smem_u32(smem_raw) & 1023 : 0);  // swizzled: on 1024-byte boundaries
  uint8_t* scales = codes + (MAP ? kWarps * p.slots * kSlotCodes : 0);
  uint8_t* smem = scales + (MAP ? kWarps * p.slots * kSlotScales : 0);
  uint4* xs = reinterpret_cast<uint4*>(smem);
  const bool whole = INLINE || p.chunk >= p.slab;
  const int buffer = token_units(room) * (p.T + 1);  // of tokens; MAP: two where they come a chunk at a time
  float* s_red = reinterpret_cast<float*>(xs + (MAP && !whole ? 2 : 1) * buffer);
  float* s_part = s_red + (p.kw > 1 ? kWarps * kRed * p.T : 0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c4 = lane & 3;
  const int part = warp % p.kw, mine = warp / p.kw;
  const int rank = p.ck > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int k0 = rank * p.slab, steps = max(0, min(p.slab, p.steps - k0));  // the block's steps
  const int per = (p.slab + p.kw - 1) / p.kw;                                // of a warp and row tile
  // row tiles are dealt out one to every block in turn, so that few of them keep all SMs busy
  const int sets = gridDim.x / p.ck, set = blockIdx.x / p.ck, rounds = (p.tiles + rw * sets - 1) / (rw * sets);
  auto tile_of = [&](int round, int m) { return (round * rw + m) * sets + set; };
  const int my_rounds = rounds - (tile_of(rounds - 1, mine) >= p.tiles);  // in which the warp has a tile

  // the next step to load
  const int exist = steps > part ? (steps - part + p.kw - 1) / p.kw : 0;  // steps of a row tile that the warp has
  int load_round = exist > 0 ? 0 : my_rounds, load_s = 0;
  int left = exist * my_rounds;  // that the warp has not used yet
  auto load_next = [&](Piece& d) {
    if (load_round >= my_rounds) return;
    load_piece(p, tile_of(load_round, mine) * kRows, load_s * p.kw + part < steps ? k0 + load_s * p.kw + part : p.steps, d);
    if (++load_s == per) load_s = 0, ++load_round;
  };
  codes += warp * p.slots * kSlotCodes, scales += warp * p.slots * kSlotScales;
  auto copy_next = [&](int slot) {  // by a lane
    if (load_round >= my_rounds) return;
    const int row = tile_of(load_round, mine) * kRows, step = k0 + load_s * p.kw + part;
    mbar_arrive_expect_tx(&s_bar[warp][slot], kSlotCodes + kSlotScales);
    tma_load_2d(&maps.codes, &s_bar[warp][slot], codes + slot * kSlotCodes, step * 128, row);
    tma_load_2d(&maps.scales, &s_bar[warp][slot], scales + slot * kSlotScales, step * 16, row);
    if (++load_s == exist) load_s = 0, ++load_round;
  };
  Piece piece[2];  // two steps in flight, or (MAP) half a step at hand
  if (MAP) {
    if (lane == 0) {
      for (int i = 0; i < p.slots; ++i) mbar_init(&s_bar[warp][i], 1);
      fence_mbar_init();
      for (int i = 0; i < p.slots; ++i) copy_next(i);
    }
    if (threadIdx.x == 0) s_abort = 0;
  } else {
    load_next(piece[0]);
    load_next(piece[1]);
  }

  // a row of zeros in the place of the tokens that fill the last eight
  for (int i = threadIdx.x; i < token_units(room); i += kThreads) {
    xs[p.T * token_units(room) + i] = make_uint4(0, 0, 0, 0);
    if (MAP && !whole) xs[buffer + p.T * token_units(room) + i] = make_uint4(0, 0, 0, 0);
  }
  if (INLINE) {
    if (threadIdx.x < kInline) s_top[threadIdx.x] = 0;
    __syncthreads();
    stage<MAP>(p, xs, s_exp, s_top, k0, steps);
  } else {
    if (threadIdx.x == 0) {
      for (int i = 0; i < 2; ++i) mbar_init(&s_full[i], 1), s_copied[i] = 0;
      s_first = 0, s_left = (steps + p.chunk - 1) / p.chunk * rounds;
      fence_mbar_init();
    }
    kv4::wait_for_previous();
    if (static_cast<int>(threadIdx.x) < p.T) s_exp[threadIdx.x] = p.exps[threadIdx.x];
    __syncthreads();
  }
  uint32_t parity = 0;
  bool landed = true;
  // Steps [k0 + first, .. + n) of all tokens, by a warp that has seen what the buffer held
  // before land.  Whether or not they come in time (reported, the result is undefined) the
  // block goes on, so that its cluster does, but copies no more.
  auto copy_tokens = [&](int b, int first, int n) {
    if (lane == 0) {
      fence_proxy_async_smem();
      mbar_arrive_expect_tx(&s_full[b], n * kUnits * 16 * p.T);
      ++s_copied[b];
    }
    __syncwarp();
    if (lane < p.T)
      bulk_load(xs + b * buffer + lane * token_units(room), p.units + (static_cast<long long>(lane) * p.steps + k0 + first) * kUnits,
                n * kUnits * 16, &s_full[b]);
  };
  auto fetch = [&](int first, int n) {  // by the block, between barriers
    if (n <= 0) return;
    if (warp == 0 && landed) copy_tokens(0, first, n);
    if (landed) landed = mbar_wait_warp(&s_full[0], parity, p.timeout_ns, p.err, nullptr);
    parity ^= 1;
  };
  // MAP, a chunk of all tokens at a time, row tile after row tile, by the first warp: the
  // next one comes while one is used.  (Copied by the warp that is the last to be through
  // with the one before, without a barrier: 114 against 112 us for 24 tokens 151936 x 4096,
  // 145 against 137 for 32, one after the other.)
  auto fetch_chunk = [&](int b) {
    const int first = s_first, n = min(p.chunk, steps - first);
    if (s_left > 0 && landed) copy_tokens(b, first, n);
    __syncwarp();
    if (lane == 0) s_first = first + n < steps ? first + n : 0, --s_left;
    __syncwarp();
  };
  if (whole && !INLINE) fetch(0, steps);
  if (MAP && !whole && warp == 0) fetch_chunk(0), fetch_chunk(1);
  __syncthreads();
  if (p.ck > 1) cluster_sync_all();  // the cluster's blocks have all begun
  const float scale = __ldg(p.g);
  auto put = [&](int n, int t, float y) {
    y *= scale;
    if (p.add) y += __uint_as_float(static_cast<uint32_t>(p.add[t * p.add_stride + n]) << 16);
    const long long at = static_cast<long long>(t) * p.N + n;
    if (p.out_f32) static_cast<float*>(p.out)[at] = y;
    else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(y);
  };

  float acc[2][NT][4];
  const uint4* xt[NT];  // the lane's quarter of each token of its column
#pragma unroll
  for (int i = 0; i < NT; ++i) xt[i] = xs + min(8 * i + g, p.T) * token_units(room) + c4;
  // products of a lane's 32 values of four rows, the tokens' from unit `at` on
  auto multiply = [&](const Piece& d, int at) {
    uint32_t f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = e4m3x2_to_f16x2(d.s[i]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t half = j >= 2 ? 0x3232u : 0x1010u;
      Expanded e[2];
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        const uint4 &lo = d.c[2 * a], &hi = d.c[2 * a + 1];
        e[a] = expand(j == 0 ? lo.x : j == 1 ? lo.y : j == 2 ? lo.z : lo.w, __byte_perm(f[2 * a], f[2 * a], half),
                      j == 0 ? hi.x : j == 1 ? hi.y : j == 2 ? hi.z : hi.w, __byte_perm(f[2 * a + 1], f[2 * a + 1], half));
      }
      uint4 x[NT];
#pragma unroll
      for (int i = 0; i < NT; ++i) x[i] = xt[i][at + 4 * j];
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int a = 0; a < 2; ++a) mma_half<0>(acc[a][i], e[a], x[i]);
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int a = 0; a < 2; ++a) mma_half<1>(acc[a][i], e[a], x[i]);
    }
  };
  float back[NT][2];  // each token's power of two taken out again
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int t = 8 * i + 2 * c4 + q;
      back[i][q] = t < p.T ? power_of_two(-s_exp[t]) : 0.0f;
    }
  int flip = 0, slot = 0;
  uint32_t turn = 0;   // parity of the ring's slots
  bool come = true;    // every step so far
  bool odd = false;    // which piece is at hand
  int chunk = 0;       // MAP: the one at hand
  for (int round = 0; round < rounds; ++round, flip ^= 1) {
    const bool has_tile = round < my_rounds;
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[a][i][0] = acc[a][i][1] = acc[a][i][2] = acc[a][i][3] = 0.0f;
    if (MAP) {
#pragma unroll 1
      for (int s = 0, in_chunk = 0; s < exist; ++s) {
        if (!whole && in_chunk == 0 && landed) landed = mbar_wait_warp(&s_full[chunk & 1], chunk >> 1 & 1, p.timeout_ns, p.err, nullptr);
        if (come && has_tile) come = mbar_wait_warp(&s_bar[warp][slot], turn, p.timeout_ns, p.err, &s_abort);
        const int at = whole ? (s * p.kw + part) * kUnits : (chunk & 1) * buffer + in_chunk * kUnits;
        if (!whole && (++in_chunk == p.chunk || s + 1 == exist)) in_chunk = 0;
        if (has_tile && come) {
          const uint8_t *c = codes + slot * kSlotCodes + g * 128, *f = scales + slot * kSlotScales + g * 16 + c4 * 4;
          uint32_t sf[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) sf[i] = *reinterpret_cast<const uint32_t*>(f + 128 * i);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              piece[h].c[i] = *reinterpret_cast<const uint4*>(c + 1024 * i + ((2 * c4 + h) ^ g) * 16);
              piece[h].s[i] = h ? sf[i] >> 16 : sf[i] & 0xFFFFu;
            }
            multiply(piece[h], at + 16 * h);
          }
          __syncwarp();  // the slot has been read
          if (lane == 0) copy_next(slot);
          --left;
          if (++slot == p.slots) slot = 0, turn ^= 1;
        }
        if (!whole && in_chunk == 0) {  // every warp is through with the chunk (whether or not its steps came)
          __syncthreads();
          if (warp == 0) fetch_chunk(chunk & 1);
          ++chunk;
        }
      }
    } else {
      int first = 0;  // step that the staged tokens begin with
#pragma unroll 1
      for (int s = 0; s < per; ++s) {
        if (!whole && (s * p.kw) % p.chunk == 0) {
          first = s * p.kw;
          __syncthreads();
          fetch(first, min(p.chunk, steps - first));
          __syncthreads();
        }
        // (the code of a step twice: moving the next piece to its place took a fifth longer)
        const int at = (s * p.kw + part - first) * kUnits;
        const bool have = has_tile && s * p.kw + part < steps;
        if (odd) {
          if (have) multiply(piece[1], at);
          load_next(piece[1]);
        } else {
          if (have) multiply(piece[0], at);
          load_next(piece[0]);
        }
        odd = !odd;
      }
    }
    // sums of the warp's tile: rows 16 a + g (+ 8), tokens 8 i + 2 c4 (+ 1)
    const int n0 = tile_of(round, mine) * kRows;
    auto each = [&](auto use) {
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int r = 16 * a + g + 8 * (q >> 1), t = 8 * i + 2 * c4 + (q & 1);
            if (t < p.T) use(r, t, acc[a][i][q] * back[i][q & 1]);
          }
    };
    if (p.kw == 1 && p.ck == 1) {
      each([&](int r, int t, float y) {
        if (n0 + r < p.N) put(n0 + r, t, y);
      });
      continue;
    }
    const int values = rows * p.T, share = (values + p.ck - 1) / p.ck;
    auto hand_over = [&](int i, float y) {  // the block's sum of value i to the block that has its share
      const int to = i / share;
      store_remote(mapa_shared(smem_u32(s_part + (flip * p.ck + rank) * share + i - to * share), to), y);
    };
    if (p.kw > 1) {  // the KW warps of a row tile join their sums, without the others
      float* red = s_red + mine * p.kw * p.T * kRed;
      each([&](int r, int t, float y) { red[(part * p.T + t) * kRed + r] = y; });
      named_bar_sync(1 + mine, 32 * p.kw);
      for (int i = part * 32 + lane; i < kRows * p.T; i += 32 * p.kw) {
        const int t = i / kRows, r = i % kRows;
        float y = 0.0f;
        for (int q = 0; q < p.kw; ++q) y += red[(q * p.T + t) * kRed + r];
        if (p.ck > 1) hand_over(t * rows + mine * kRows + r, y);
        else if (n0 + r < p.N) put(n0 + r, t, y);
      }
      named_bar_sync(1 + mine, 32 * p.kw);
    } else {
      each([&](int r, int t, float y) { hand_over(t * rows + mine * kRows + r, y); });
    }
    if (p.ck > 1) {
      cluster_sync_all();  // every block's part of this one's share has come
      for (int i = threadIdx.x; i < share && rank * share + i < values; i += kThreads) {
        float y = 0.0f;
        for (int q = 0; q < p.ck; ++q) y += s_part[(flip * p.ck + q) * share + i];
        const int v = rank * share + i, t = v / rows, r = v - t * rows, n = tile_of(round, r / kRows) * kRows + r % kRows;
        if (n < p.N) put(n, t, y);
      }
    }
  }
  if (p.ck > 1) cluster_sync_all();  // no block leaves while another may still write to it
  // nor before its copies have landed
  if (!INLINE) {
    __syncthreads();  // no more copies
    if (!landed)
      for (int b = 0; b < 2; ++b)
        if (s_copied[b] > 0) mbar_wait_warp(&s_full[b], (s_copied[b] - 1) & 1, 1000000000ull, p.err, nullptr);
  }
  if (MAP && !come)
    for (int i = 0; i < min(p.slots, left); ++i) {
      mbar_wait_warp(&s_bar[warp][slot], turn, 1000000000ull, p.err, nullptr);
      if (++slot == p.slots) slot = 0, turn ^= 1;
    }
}

template <bool MAP>
size_t smem_of(const Params& p) {
  constexpr int kWarps = Cfg<MAP>::kWarps;
  const size_t rows = static_cast<size_t>(kWarps / p.kw) * kRows, values = rows * p.T;
  size_t n = static_cast<size_t>(token_units<MAP>(std::min(p.chunk, p.slab))) * 16 * (p.T + 1) * (MAP && p.chunk < p.slab ? 2 : 1);
  if (p.kw > 1) n += static_cast<size_t>(kWarps) * kRed * p.T * 4;
  if (p.ck > 1) n += 2 * p.ck * ((values + p.ck - 1) / p.ck) * 4;
  if (MAP) n += 1024 + static_cast<size_t>(kWarps) * p.slots * (kSlotCodes + kSlotScales);
  return n;
}

// (room for either kernel's steps)
size_t carve(Params& p, void* ws) {
  Carve c(ws, 0);
  p.exps = c.take<int>(p.T);
  p.units = c.take<uint4>(static_cast<size_t>(p.T) * ((p.K + 255) / 256) * 32);
  return c.used;
}
bool brought_inside(int T, int K) { return T <= kInline && K <= kInlineK; }

template <int NT, bool INLINE, bool MAP>
int launch(const Params& p, const Maps& maps, cudaStream_t s) {
  static std::atomic<bool> set[64];
  MOE_TRY(kv4::allow_smem(linear_kernel<NT, INLINE, MAP>, kSmem, set));
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(p.sets * p.ck), cfg.blockDim = dim3(Cfg<MAP>::kThreads);
  cfg.dynamicSmemBytes = smem_of<MAP>(p), cfg.stream = s;
  cudaLaunchAttribute a[2]{};
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  a[1].id = cudaLaunchAttributeClusterDimension;
  a[1].val.clusterDim.x = p.ck, a[1].val.clusterDim.y = a[1].val.clusterDim.z = 1;
  cfg.attrs = INLINE ? a + 1 : a, cfg.numAttrs = (INLINE ? 0 : 1) + (p.ck > 1 ? 1 : 0);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, linear_kernel<NT, INLINE, MAP>, p, maps);
  if (e != cudaSuccess) {
    set_cuda_error(e);
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

// Clusters of four blocks that run at once on the current device: fewer than a quarter
// of its SMs (one more would wait for another to end).
int clusters_of_four() {
  static std::atomic<int> known[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
  static std::atomic<bool> set[64];
  const auto kernel = linear_kernel<1, true, false>;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(4), cfg.blockDim = dim3(Cfg<false>::kThreads), cfg.dynamicSmemBytes = kSmem - 1024;
  cudaLaunchAttribute a{};
  a.id = cudaLaunchAttributeClusterDimension;
  a.val.clusterDim.x = 4, a.val.clusterDim.y = a.val.clusterDim.z = 1;
  cfg.attrs = &a, cfg.numAttrs = 1;
  if (kv4::allow_smem(kernel, kSmem, set) != MOE_OK || cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = num_sms() / 8;
  }
  n = std::max(1, n);
  if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

// How the reduction is split: the one with the least estimated time, counted in steps
// of a warp: rounds of row tiles, joining the warps' and the blocks' sums, the tokens'
// copies.  (Clusters of eight were slower than what they save at every size.)
// Returns that time in steps of 128 values, infinite where nothing fits.  (A step by
// tensor maps takes 0.75 to 0.95 of two of the others, from a million weights to 600.)
template <bool MAP>
double choose(Params& p) {
  p.steps = (p.K + Cfg<MAP>::kStep - 1) / Cfg<MAP>::kStep;
  constexpr int kWarps = Cfg<MAP>::kWarps;
  const bool inside = brought_inside(p.T, p.K);
  const int sms = num_sms(), clusters4 = clusters_of_four(), step_bytes = p.T * Cfg<MAP>::kStep * 2;
  double best = 0.0;
  Params found = p;
  found.kw = 0;
  for (int ck = 1; ck <= kMaxCluster; ck *= 2)
    for (int kw = 1; kw <= kWarps; kw *= 2) {
      Params q = p;
      q.kw = kw, q.ck = ck, q.slab = (p.steps + ck - 1) / ck;
      q.chunk = (q.slab + kw - 1) / kw * kw;
      q.slots = kSlots;
      if (MAP) {
        while (smem_of<MAP>(q) > kSmem - 1024 && q.slots > 2) --q.slots;
        // (in chunks only by blocks whose warps all take every step)
        if (!inside && kw == 1 && ck == 1)
          while (smem_of<MAP>(q) > kSmem - 1024 && q.chunk > 1) q.chunk = q.chunk > 8 ? q.chunk / 2 : q.chunk - 1;
      } else if (!inside) {
        while (smem_of<MAP>(q) > kSmem - 1024 && q.chunk > kw) q.chunk = std::max(kw, (q.chunk / 2 + kw - 1) / kw * kw);
      }
      if (smem_of<MAP>(q) > kSmem - 1024) continue;
      const int rw = kWarps / kw;
      q.sets = std::min(ck == 4 ? clusters4 : sms / ck, p.tiles);
      const int rounds = (p.tiles + rw * q.sets - 1) / (rw * q.sets);
      // a step takes less where fewer of the block's warps have one
      const int last = (p.tiles - (rounds - 1) * rw * q.sets + q.sets - 1) / q.sets * kw;
      const double turns = rounds - 1 + 0.4 + 0.6 * last / kWarps;
      const double stage = q.slab * step_bytes / 50000.0 / (Cfg<MAP>::kStep / 128);
      const double join = (kw > 1 ? 0.5 : 0.2) + (ck > 1 ? 1.5 : 0.0);
      const double cost = turns * ((q.slab + kw - 1) / kw) + rounds * join * (256 / Cfg<MAP>::kStep) + stage * (MAP || q.chunk >= q.slab ? 1.0 : rounds);
      if (found.kw == 0 || cost < best) best = cost, found = q;
    }
  p = found;
  return p.kw == 0 ? INFINITY : MAP ? best * 2 * 0.87 : best;
}

template <bool MAP>
int run(const Params& p, const Maps& maps, cudaStream_t s) {
  if (brought_inside(p.T, p.K)) return p.T <= 8 ? launch<1, true, MAP>(p, maps, s) : launch<2, true, MAP>(p, maps, s);
  linear_prepare_kernel<MAP><<<p.T, kPrepThreads, 0, s>>>(p);
  MOE_TRY(check_launch());
  switch ((p.T + 7) / 8) {
    case 1: return launch<1, false, MAP>(p, maps, s);
    case 2: return launch<2, false, MAP>(p, maps, s);
    case 3: return launch<3, false, MAP>(p, maps, s);
    default: return launch<4, false, MAP>(p, maps, s);
  }
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_linear_nvfp4_workspace_size(int T, int K) {
  if (T < 1 || T > kMaxTokens || K < 1 || K % 32 != 0 || K > (1 << 24) || brought_inside(T, K)) return 0;
  Params p{};
  p.T = T, p.K = K;
  return carve(p, nullptr);
}

extern "C" int moe_linear_nvfp4(const uint16_t* x, long long x_stride, int T, const uint8_t* w, const uint8_t* w_sf,
                                const float* w_g, int N, int K, const uint16_t* add, long long add_stride, void* out,
                                int out_f32, void* ws, size_t ws_bytes, void* stream) {
  if (T < 0 || N < 0 || K < 1) return MOE_ERR_INVALID_ARG;
  if (T > kMaxTokens || K % 32 != 0 || N > (1 << 27) || K > (1 << 24)) return MOE_ERR_UNSUPPORTED;
  if (T == 0 || N == 0) return MOE_OK;
  if (!x || !w || !w_sf || !w_g || !out) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || x_stride % 8 != 0 || (T > 1 && x_stride < K)) return MOE_ERR_INVALID_ARG;
  if (!aligned(w, 16) || !aligned(w_sf, 4) || !aligned(w_g, 4) || !aligned(out, out_f32 ? 4 : 2)) return MOE_ERR_INVALID_ARG;
  if (add && (!aligned(add, 2) || (T > 1 && add_stride < N))) return MOE_ERR_INVALID_ARG;
  Params p{x, x_stride, w, w_sf, w_g, add, add_stride, out, T, N, K, out_f32, (N + kRows - 1) / kRows};
  if (!brought_inside(T, K)) {
    if (!ws || !aligned(ws, 256)) return MOE_ERR_INVALID_ARG;
    if (ws_bytes < carve(p, ws)) return MOE_ERR_WORKSPACE;
  }
  p.timeout_ns = wait_timeout_ns();
  p.err = device_error_word();
  if (!p.err) return MOE_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  Maps maps{};
  Params q = p;
  const double plain = choose<false>(p);
  if (std::isinf(plain)) return MOE_ERR_UNSUPPORTED;
  if (K % Cfg<true>::kStep == 0 && aligned(w_sf, 16) && choose<true>(q) <= plain) {
    const uint64_t cd[2] = {static_cast<uint64_t>(K / 2), static_cast<uint64_t>(N)}, sd[2] = {static_cast<uint64_t>(K / 16), cd[1]};
    const uint32_t cb[2] = {128, kRows}, sb[2] = {16, kRows};
    MOE_TRY(encode_tmap_nd(&maps.codes, w, false, 2, cd, cd, cb, true));
    MOE_TRY(encode_tmap_nd(&maps.scales, w_sf, false, 2, sd, sd, sb, false));
    return run<true>(q, maps, s);
  }
  return run<false>(p, maps, s);
}
