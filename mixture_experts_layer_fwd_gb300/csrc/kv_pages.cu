// Pages of the paged key/value cache: allocation for new tokens, forks with
// copy-on-write of the partial page, release, compaction, plain copies.
//
// The state is three integer arrays on the device: refs[p], how many table
// rows map page p (0: free); table[row][j], the page of tokens j*P..j*P+P-1
// of a sequence (-1: none); lens[row].  There is no free list to keep in
// step: an allocation takes the lowest free ids, found by one scan over refs
// (4 bytes a page, L2-resident), so that the same state always gives the same
// result.  A call is a one-block plan (scans, ranks) and a wide kernel that
// applies it and copies pages.  The copies are the only large traffic: 2 bytes
// moved per byte of page, 16 bytes per thread and access, four in flight:
// compaction of 1.39 GB 231 us (6.0 TB/s, 0.89 of a copy), a fork of 302 MB 50 us
// (6.0 TB/s) with the plan in front.  The wide kernel is launched under the plan (a
// programmatic dependent launch; 3 us more without).  Placing new tokens takes 4 us
// on the GPU for one row, 5.4 for 256 on 40000 pages, 8.6 for 8 rows of 2048 tokens.
#include "kv4.cuh"

namespace moe {
namespace {

constexpr int kPlan = 1024;       // threads of a plan block
constexpr int kPer = 16;          // pages per thread and scan step
constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;
constexpr int kPart = kCopyThreads * kCopyUnroll * 16;  // bytes per block and copy step

struct State {
  const int32_t *table_in, *lens_in, *refs_in;
  int32_t *table, *lens, *refs;
  int S, M, N, P;
};

struct Pool {
  uint8_t* base;
  int layers;
  long long layer_stride, page_bytes;
};

// Workspace: counts, then lists of up to N pages and up to S rows.
struct Plan {
  int* count;   // [0] pages found / moves
  int* list_a;  // [N]
  int* list_b;  // [N]
  int* row_a;   // [rows]
  int* row_b;   // [rows]
  int* starts;  // extend: [rows + 1] q_offsets as used; fork: [rows] first pair that names a row
};

Plan carve(void* ws, int N, int rows, size_t* bytes) {
  Carve c(ws, 0);
  Plan p;
  p.count = c.take<int>(64);
  p.list_a = c.take<int>(N);
  p.list_b = c.take<int>(N);
  p.row_a = c.take<int>(rows);
  p.row_b = c.take<int>(rows);
  p.starts = c.take<int>(rows + 1);
  if (bytes) *bytes = c.used;
  return p;
}

// Exclusive prefix of v over the block's threads; total in `total`.
DEVINL int block_scan(int v, int* s_warp, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int w = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xFFFFFFFFu, w, o);
      if (lane >= o) w += up;
    }
    s_warp[lane] = w;
  }
  __syncthreads();
  const int before = warp ? s_warp[warp - 1] : 0;
  total = s_warp[31];
  __syncthreads();
  return before + incl - v;
}

// Bit i of the result: page p0 + i is in use.
DEVINL uint32_t live_bits(const int32_t* refs, int N, int p0) {
  uint32_t m = 0;
  if (p0 + kPer <= N) {
#pragma unroll
    for (int q = 0; q < kPer / 4; ++q) {
      const int4 r = *reinterpret_cast<const int4*>(refs + p0 + 4 * q);
      m |= (static_cast<uint32_t>(r.x > 0) | static_cast<uint32_t>(r.y > 0) << 1 | static_cast<uint32_t>(r.z > 0) << 2 |
            static_cast<uint32_t>(r.w > 0) << 3)
           << (4 * q);
    }
  } else {
    for (int i = 0; i < kPer && p0 + i < N; ++i) m |= static_cast<uint32_t>(refs[p0 + i] > 0) << i;
  }
  return m;
}
DEVINL uint32_t in_range_bits(int N, int p0) {
  const int n = max(0, min(kPer, N - p0));
  return (1u << n) - 1u;
}

// The first `need` free page ids into list; returns how many there are (all threads).
DEVINL int find_free(const int32_t* refs, int N, int need, int* list, int* s_warp) {
  int found = 0;
  for (int base = 0; base < N && found < need; base += kPlan * kPer) {
    const int p0 = base + threadIdx.x * kPer;
    uint32_t bits = p0 < N ? ~live_bits(refs, N, p0) & in_range_bits(N, p0) : 0u;
    int total;
    int k = found + block_scan(__popc(bits), s_warp, total);
    while (bits && k < need) {
      const int i = __ffs(bits) - 1;
      bits &= bits - 1;
      list[k++] = p0 + i;
    }
    found = min(need, found + total);
  }
  return found;
}

// in -> out where they are different arrays (blocks after the plan's).
DEVINL void carry_over(const State& s) {
  const long long id = static_cast<long long>(blockIdx.x - 1) * kPlan + threadIdx.x;
  const long long step = static_cast<long long>(gridDim.x - 1) * kPlan;
  if (s.table != s.table_in)
    for (long long i = id; i < static_cast<long long>(s.S) * s.M; i += step) s.table[i] = s.table_in[i];
  if (s.lens != s.lens_in)
    for (long long i = id; i < s.S; i += step) s.lens[i] = s.lens_in[i];
  if (s.refs != s.refs_in)
    for (long long i = id; i < s.N; i += step) s.refs[i] = s.refs_in[i];
}

DEVINL bool page_ok(int p, int N) { return p >= 0 && p < N; }  // or row

// Items (layer, list entry, part) of a page copy, spread over the blocks from `first` on.
DEVINL void copy_pages(const Pool& pool, const int* src, const int* dst, int n, int N, int first, unsigned int* err) {
  const int parts = static_cast<int>((pool.page_bytes + kPart - 1) / kPart);
  const long long items = static_cast<long long>(n) * pool.layers * parts;
  for (long long it = static_cast<long long>(blockIdx.x) - first; it < items; it += gridDim.x - first) {
    const int part = static_cast<int>(it % parts);
    const long long r = it / parts;
    const int e = static_cast<int>(r % n), layer = static_cast<int>(r / n);
    const int a = src[e], b = dst[e];
    if (!page_ok(a, N) || !page_ok(b, N)) {
      if (threadIdx.x == 0) atomicOr(err, kErrBadIndex);
      continue;
    }
    if (a == b) continue;
    uint8_t* l = pool.base + layer * pool.layer_stride;
    const uint4* from = reinterpret_cast<const uint4*>(l + a * pool.page_bytes);
    uint4* to = reinterpret_cast<uint4*>(l + b * pool.page_bytes);
    const int end = static_cast<int>(pool.page_bytes / 16);
    const int i0 = part * (kPart / 16) + threadIdx.x;
    uint4 v[kCopyUnroll];
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u)
      if (i0 + u * kCopyThreads < end) v[u] = __ldcs(from + i0 + u * kCopyThreads);
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u)
      if (i0 + u * kCopyThreads < end) __stcs(to + i0 + u * kCopyThreads, v[u]);
  }
}

// ------------------------------------------------------------------ extend
// The offsets are read as attention reads them: inside the tokens, a running
// maximum, so that whatever they hold each token has one row at most.
__global__ void __launch_bounds__(kPlan) extend_plan_kernel(State s, const int32_t* q_offsets, int T, Plan w,
                                                            unsigned int* err) {
  __shared__ int s_warp[32];
  kv4::launch_dependents();
  if (blockIdx.x > 0) return carry_over(s);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int need = 0, reached = min(max(q_offsets[0], 0), T);  // largest offset so far
  if (threadIdx.x == 0) w.starts[0] = reached;
  for (int base = 0; base < s.S; base += kPlan) {
    const int r = base + threadIdx.x;
    int end = r < s.S ? min(max(q_offsets[r + 1], 0), T) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xFFFFFFFFu, end, o);
      if (lane >= o) end = max(end, up);
    }
    if (lane == 31) s_warp[warp] = end;
    __syncthreads();
    const int of_warp = s_warp[lane];
    const int before = max(reached, __reduce_max_sync(0xFFFFFFFFu, lane < warp ? of_warp : 0));
    const int up = __shfl_up_sync(0xFFFFFFFFu, end, 1);
    const int n = max(before, end) - (lane > 0 ? max(before, up) : before);
    reached = max(reached, __reduce_max_sync(0xFFFFFFFFu, of_warp));
    __syncthreads();  // s_warp has been read
    int more = 0;
    if (r < s.S) {
      w.starts[r + 1] = max(before, end);
      const int len = max(0, s.lens_in[r]);
      const long long want = (static_cast<long long>(len) + n + s.P - 1) / s.P;
      if (n > 0 && want > s.M) {
        atomicOr(err, kErrBadIndex);
        more = -1;
      } else {
        more = n > 0 ? max(0, static_cast<int>(want) - (len + s.P - 1) / s.P) : 0;
      }
    }
    int total;
    const int rank = block_scan(max(more, 0), s_warp, total);
    if (r < s.S) {
      w.row_a[r] = more < 0 ? -1 : need + rank;
      w.row_b[r] = max(more, 0);
    }
    need += total;
  }
  const int found = find_free(s.refs_in, s.N, min(need, s.N), w.list_a, s_warp);
  if (threadIdx.x == 0) w.count[0] = found;
}

__global__ void extend_apply_kernel(State s, int T, Plan w, long long* slots, int32_t* pos, int32_t* kv_lens,
                                    unsigned int* err) {
  kv4::wait_for_previous();
  const int r = blockIdx.x;
  if (r == s.S) {  // tokens of no row: in front of the first one's and behind the last one's
    const int first = w.starts[0], last = w.starts[s.S];
    for (int t = threadIdx.x; t < first + T - last; t += blockDim.x) {
      const int at = t < first ? t : last + t - first;
      slots[at] = -1;
      pos[at] = 0;
    }
    return;
  }
  const int t0 = w.starts[r], t1 = w.starts[r + 1];
  const int rank = w.row_a[r], more = w.row_b[r];
  const int len = max(0, s.lens[r]);
  const bool ok = rank >= 0 && (more == 0 || rank + more <= w.count[0]);
  const int have = (len + s.P - 1) / s.P;
  int32_t* row = s.table + static_cast<long long>(r) * s.M;
  if (!ok && t1 > t0 && threadIdx.x == 0) atomicOr(err, rank >= 0 ? kErrNoPages : kErrBadIndex);
  if (ok)
    for (int j = threadIdx.x; j < more; j += blockDim.x) {
      const int p = w.list_a[rank + j];
      row[have + j] = p;
      s.refs[p] = 1;
    }
  __syncthreads();
  for (int t = t0 + threadIdx.x; t < t1; t += blockDim.x) {
    const int at = len + (t - t0);
    const int j = at / s.P;
    const int p = !ok ? -1 : j >= have ? w.list_a[rank + j - have] : row[j];
    slots[t] = page_ok(p, s.N) ? static_cast<long long>(p) * s.P + at % s.P : -1;
    pos[t] = at;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    if (ok && t1 > t0) s.lens[r] = len + (t1 - t0);
    if (kv_lens) kv_lens[r] = ok ? len + max(0, t1 - t0) : 0;
  }
}

// -------------------------------------------------------------------- fork
__global__ void __launch_bounds__(kPlan) fork_plan_kernel(State s, const int32_t* src, const int32_t* dst, int n, Plan w,
                                                          unsigned int* err) {
  __shared__ int s_warp[32];
  kv4::launch_dependents();
  if (blockIdx.x > 0) return carry_over(s);
  // A row may be named once: the first pair that does has it.  Few pairs look at
  // those in front of them (a lane at most 31), many find the first by row; all
  // by the loop took 82 ms for 65536 pairs.
  const bool few = n <= 32;
  if (!few) {
    for (int i = threadIdx.x; i < n; i += kPlan)
      if (page_ok(dst[i], s.S)) w.starts[dst[i]] = n;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kPlan)
      if (page_ok(dst[i], s.S)) atomicMin(w.starts + dst[i], i);
    __syncthreads();
  }
  int need = 0;
  for (int base = 0; base < n; base += kPlan) {
    const int i = base + threadIdx.x;
    int len = -1;
    if (i < n) {
      const int r = src[i], d = dst[i];
      bool ok = r >= 0 && r < s.S && d >= 0 && d < s.S;
      if (ok && s.lens_in[d] != 0) ok = false;
      if (few) {
        for (int j = 0; ok && j < i; ++j) ok = dst[j] != d;
      } else if (ok) {
        ok = __ldcg(w.starts + d) == i;
      }
      if (ok) len = static_cast<int>(max(0ll, min(static_cast<long long>(s.lens_in[r]), static_cast<long long>(s.M) * s.P)));
      else atomicOr(err, kErrBadIndex);
    }
    const bool partial = len > 0 && len % s.P != 0;
    int total;
    const int rank = need + block_scan(partial ? 1 : 0, s_warp, total);
    if (i < n) {
      w.row_a[i] = len;
      w.row_b[i] = partial ? rank : -1;
      if (partial && rank < s.N) {  // the page to copy
        const int p = s.table_in[static_cast<long long>(src[i]) * s.M + len / s.P];
        w.list_b[rank] = p;
      }
    }
    need += total;
  }
  const int found = find_free(s.refs_in, s.N, min(need, s.N), w.list_a, s_warp);
  if (threadIdx.x == 0) w.count[0] = found;
}

__global__ void __launch_bounds__(kCopyThreads) fork_apply_kernel(State s, const int32_t* src, const int32_t* dst, int n,
                                                                  Plan w, Pool pool, unsigned int* err) {
  kv4::wait_for_previous();
  if (blockIdx.x >= n) return copy_pages(pool, w.list_b, w.list_a, w.count[0], s.N, n, err);
  const int i = blockIdx.x;
  const int len = w.row_a[i];
  if (len < 0) return;
  const int rank = w.row_b[i], full = len / s.P;
  const bool got = rank >= 0 && rank < w.count[0];
  const int fresh = got ? w.list_a[rank] : -1;
  const int32_t* from = s.table_in + static_cast<long long>(src[i]) * s.M;
  int32_t* to = s.table + static_cast<long long>(dst[i]) * s.M;
  for (int j = threadIdx.x; j < s.M; j += blockDim.x) {
    int p = -1;
    if (j < full) {
      p = from[j];
      if (page_ok(p, s.N)) atomicAdd(s.refs + p, 1);
      else atomicOr(err, kErrBadIndex);
    } else if (j == full) {
      p = fresh;
    }
    to[j] = p;
  }
  if (threadIdx.x == 0) {
    if (got) s.refs[fresh] = 1;
    else if (rank >= 0) atomicOr(err, kErrNoPages);
    s.lens[dst[i]] = rank >= 0 && !got ? full * s.P : len;
  }
}

// -------------------------------------------------------------------- free
__global__ void __launch_bounds__(kPlan) carry_kernel(State s) {
  kv4::launch_dependents();
  carry_over(s);
}

__global__ void free_apply_kernel(State s, const int32_t* rows, int n, unsigned int* err) {
  __shared__ int s_dup;
  kv4::wait_for_previous();
  const int i = blockIdx.x, r = rows[i];
  if (r < 0 || r >= s.S) {
    if (threadIdx.x == 0) atomicOr(err, kErrBadIndex);
    return;
  }
  if (threadIdx.x == 0) s_dup = 0;
  __syncthreads();
  for (int j = threadIdx.x; j < i; j += blockDim.x)
    if (rows[j] == r) s_dup = 1;
  __syncthreads();
  if (s_dup) return;  // listed twice: freed once
  const int len = max(0, s.lens[r]);
  const int used = static_cast<int>(min(static_cast<long long>(s.M), (static_cast<long long>(len) + s.P - 1) / s.P));
  int32_t* row = s.table + static_cast<long long>(r) * s.M;
  for (int j = threadIdx.x; j < s.M; j += blockDim.x) {
    if (j < used) {
      const int p = row[j];
      if (page_ok(p, s.N)) atomicSub(s.refs + p, 1);
      else atomicOr(err, kErrBadIndex);
    }
    row[j] = -1;
  }
  __syncthreads();
  if (threadIdx.x == 0) s.lens[r] = 0;
}

// ----------------------------------------------------------------- compact
// Live pages from n_live on move, in order, to the free pages below it: the
// fewest moves, and no page is both read and written.
__global__ void __launch_bounds__(kPlan) compact_plan_kernel(State s, Plan w, int32_t* remap) {
  __shared__ int s_warp[32];
  kv4::launch_dependents();
  if (blockIdx.x > 0) {
    const int id = (blockIdx.x - 1) * kPlan + threadIdx.x, step = (gridDim.x - 1) * kPlan;
    for (int p = id; p < s.N; p += step) {
      const int r = s.refs_in[p];
      remap[p] = r > 0 ? p : -1;
      if (s.refs != s.refs_in) s.refs[p] = max(r, 0);
    }
    return;
  }
  int mine = 0, live;
  for (int base = 0; base < s.N; base += kPlan * kPer) {
    const int p0 = base + threadIdx.x * kPer;
    if (p0 < s.N) mine += __popc(live_bits(s.refs_in, s.N, p0));
  }
  block_scan(mine, s_warp, live);
  int holes = 0, movers = 0;
  for (int base = 0; base < s.N; base += kPlan * kPer) {
    const int p0 = base + threadIdx.x * kPer;
    const uint32_t in = p0 < s.N ? in_range_bits(s.N, p0) : 0u;
    const uint32_t bits = p0 < s.N ? live_bits(s.refs_in, s.N, p0) : 0u;
    const uint32_t low = in_range_bits(live, p0) & in;
    uint32_t hole = ~bits & low, high = bits & in & ~low;
    int th, tm;
    int kh = holes + block_scan(__popc(hole), s_warp, th);
    int km = movers + block_scan(__popc(high), s_warp, tm);
    for (; hole; hole &= hole - 1) w.list_a[kh++] = p0 + __ffs(hole) - 1;
    for (; high; high &= high - 1) w.list_b[km++] = p0 + __ffs(high) - 1;
    holes += th;
    movers += tm;
  }
  if (threadIdx.x == 0) {
    w.count[0] = movers;
    w.count[1] = live;
  }
}

__global__ void __launch_bounds__(kCopyThreads) compact_apply_kernel(State s, Plan w, Pool pool, int32_t* remap,
                                                                     int small, unsigned int* err) {
  kv4::wait_for_previous();
  const int moves = w.count[0], live = w.count[1];
  if (blockIdx.x >= small) return copy_pages(pool, w.list_b, w.list_a, moves, s.N, small, err);
  const long long id = static_cast<long long>(blockIdx.x) * kCopyThreads + threadIdx.x;
  const long long step = static_cast<long long>(small) * kCopyThreads;
  for (long long k = id; k < moves; k += step) {
    const int a = w.list_b[k], b = w.list_a[k];
    remap[a] = b;
    s.refs[b] = s.refs[a];
    s.refs[a] = 0;
  }
  for (long long i = id; i < static_cast<long long>(s.S) * s.M; i += step) {
    int p = s.table_in[i];
    if (p >= live) {
      int lo = 0, hi = moves;  // movers are sorted
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (w.list_b[mid] < p) lo = mid + 1;
        else hi = mid;
      }
      p = lo < moves && w.list_b[lo] == p ? w.list_a[lo] : -1;
    }
    s.table[i] = p < 0 ? -1 : p;
  }
}

__global__ void __launch_bounds__(kCopyThreads) copy_kernel(Pool pool, const int32_t* src, const int32_t* dst, int n,
                                                            int N, unsigned int* err) {
  copy_pages(pool, src, dst, n, N, 0, err);
}

int check_state(const State& s) {
  if (s.S < 0 || s.M < 1 || s.N < 1) return MOE_ERR_INVALID_ARG;
  if (!kv4::page_size_ok(s.P) || s.N > (1 << 27) || s.S > (1 << 20)) return MOE_ERR_UNSUPPORTED;
  // (with no rows too: a compaction reads refs all the same, 16 bytes at a time)
  if (!s.refs_in || !s.refs || !aligned(s.refs_in, 16) || !aligned(s.refs, 16)) return MOE_ERR_INVALID_ARG;
  if (s.S == 0) return MOE_OK;
  if (!s.table_in || !s.table) return MOE_ERR_INVALID_ARG;
  if (!aligned(s.table_in, 4) || !aligned(s.table, 4) || !aligned(s.lens_in, 4) || !aligned(s.lens, 4))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}
int check_pool(const Pool& p) {
  if (p.layers < 0 || p.page_bytes < 16) return MOE_ERR_INVALID_ARG;
  if (p.layers == 0) return MOE_OK;
  if (!aligned(p.base, 16) || !p.base || p.page_bytes % 16 || p.layer_stride % 16) return MOE_ERR_INVALID_ARG;
  if (p.page_bytes > (1 << 30)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}
int check_ws(const void* ws, size_t have, int N, int rows) {
  size_t need;
  carve(nullptr, N, rows, &need);
  if (!ws || !aligned(ws, 256)) return MOE_ERR_INVALID_ARG;
  return have < need ? MOE_ERR_WORKSPACE : MOE_OK;
}
// blocks that carry arrays over to the outputs beside the plan block
int carry_blocks(const State& s) {
  if (s.table == s.table_in && s.lens == s.lens_in && s.refs == s.refs_in) return 0;
  const long long n = std::max<long long>(static_cast<long long>(s.S) * s.M, s.N);
  return static_cast<int>(std::max<long long>(1, std::min<long long>(num_sms(), (n + 4 * kPlan - 1) / (4 * kPlan))));
}
// A table without rows: what there is to carry over.
int carry_refs(const State& s, void* stream) {
  if (s.refs == s.refs_in) return MOE_OK;
  carry_kernel<<<1 + carry_blocks(s), kPlan, 0, static_cast<cudaStream_t>(stream)>>>(s);
  return check_launch();
}
int copy_blocks(const Pool& p, long long most) {
  const long long items = most * p.layers * ((p.page_bytes + kPart - 1) / kPart);
  return static_cast<int>(std::min<long long>(items, num_sms() * 8));
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_kv_pages_workspace_size(int num_pages, int rows) {
  if (num_pages < 1 || rows < 0) return 0;
  size_t n;
  carve(nullptr, num_pages, rows, &n);
  return n;
}

extern "C" int moe_kv_extend(const int32_t* q_offsets, int T, const int32_t* table_in, const int32_t* lens_in,
                             const int32_t* refs_in, int rows, int max_pages, int num_pages, int page_size,
                             int32_t* table_out, int32_t* lens_out, int32_t* refs_out, long long* slots, int32_t* pos,
                             void* ws, size_t ws_bytes, void* stream) {
  return moe_kv_extend_ex(q_offsets, T, table_in, lens_in, refs_in, rows, max_pages, num_pages, page_size, table_out,
                          lens_out, refs_out, slots, pos, nullptr, ws, ws_bytes, stream);
}

extern "C" int moe_kv_extend_ex(const int32_t* q_offsets, int T, const int32_t* table_in, const int32_t* lens_in,
                                const int32_t* refs_in, int rows, int max_pages, int num_pages, int page_size,
                                int32_t* table_out, int32_t* lens_out, int32_t* refs_out, long long* slots, int32_t* pos,
                                int32_t* kv_lens, void* ws, size_t ws_bytes, void* stream) {
  State s{table_in, lens_in, refs_in, table_out, lens_out, refs_out, rows, max_pages, num_pages, page_size};
  if (T < 0) return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_state(s));
  if (rows == 0) return carry_refs(s, stream);
  if (!q_offsets || !lens_in || !lens_out || !aligned(q_offsets, 4)) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!slots || !pos || !aligned(slots, 8) || !aligned(pos, 4))) return MOE_ERR_INVALID_ARG;
  if (kv_lens && (kv_lens == lens_out || kv_lens == lens_in || !aligned(kv_lens, 4))) return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_ws(ws, ws_bytes, num_pages, rows));
  unsigned int* err = device_error_word();
  if (!err) return MOE_ERR_CUDA;
  Plan w = carve(ws, num_pages, rows, nullptr);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  extend_plan_kernel<<<1 + carry_blocks(s), kPlan, 0, st>>>(s, q_offsets, T, w, err);
  MOE_TRY(check_launch());
  return kv4::launch_after(extend_apply_kernel, dim3(rows + 1), 128, 0, st, s, T, w, slots, pos, kv_lens, err);
}

extern "C" int moe_kv_fork(const int32_t* src, const int32_t* dst, int n, const int32_t* table_in,
                           const int32_t* lens_in, const int32_t* refs_in, int rows, int max_pages, int num_pages,
                           int page_size, int32_t* table_out, int32_t* lens_out, int32_t* refs_out, uint8_t* pool,
                           int layers, long long layer_stride, long long page_bytes, void* ws, size_t ws_bytes,
                           void* stream) {
  State s{table_in, lens_in, refs_in, table_out, lens_out, refs_out, rows, max_pages, num_pages, page_size};
  Pool p{pool, layers, layer_stride, page_bytes};
  if (n < 0) return MOE_ERR_INVALID_ARG;
  if (n > 65536) return MOE_ERR_UNSUPPORTED;
  MOE_TRY(check_state(s));
  MOE_TRY(check_pool(p));
  if (rows == 0) return carry_refs(s, stream);
  if (!lens_in || !lens_out || (n > 0 && (!src || !dst || !aligned(src, 4) || !aligned(dst, 4))))
    return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_ws(ws, ws_bytes, num_pages, std::max(rows, n)));
  unsigned int* err = device_error_word();
  if (!err) return MOE_ERR_CUDA;
  Plan w = carve(ws, num_pages, std::max(rows, n), nullptr);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  fork_plan_kernel<<<1 + carry_blocks(s), kPlan, 0, st>>>(s, src, dst, n, w, err);
  MOE_TRY(check_launch());
  if (n == 0) return MOE_OK;
  return kv4::launch_after(fork_apply_kernel, dim3(n + copy_blocks(p, n)), kCopyThreads, 0, st, s, src, dst, n, w, p, err);
}

extern "C" int moe_kv_free(const int32_t* rows_to_free, int n, const int32_t* table_in, const int32_t* lens_in,
                           const int32_t* refs_in, int rows, int max_pages, int num_pages, int page_size,
                           int32_t* table_out, int32_t* lens_out, int32_t* refs_out, void* stream) {
  State s{table_in, lens_in, refs_in, table_out, lens_out, refs_out, rows, max_pages, num_pages, page_size};
  if (n < 0) return MOE_ERR_INVALID_ARG;
  if (n > 65536) return MOE_ERR_UNSUPPORTED;
  MOE_TRY(check_state(s));
  if (rows == 0) return carry_refs(s, stream);
  if (!lens_in || !lens_out || (n > 0 && (!rows_to_free || !aligned(rows_to_free, 4)))) return MOE_ERR_INVALID_ARG;
  unsigned int* err = device_error_word();
  if (!err) return MOE_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (const int b = carry_blocks(s)) {
    carry_kernel<<<1 + b, kPlan, 0, st>>>(s);
    MOE_TRY(check_launch());
  }
  if (n == 0) return MOE_OK;
  return kv4::launch_after(free_apply_kernel, dim3(n), 128, 0, st, s, rows_to_free, n, err);
}

extern "C" int moe_kv_compact(const int32_t* table_in, const int32_t* refs_in, int rows, int max_pages, int num_pages,
                              int32_t* table_out, int32_t* refs_out, int32_t* remap, uint8_t* pool, int layers,
                              long long layer_stride, long long page_bytes, void* ws, size_t ws_bytes, void* stream) {
  State s{table_in, nullptr, refs_in, table_out, nullptr, refs_out, rows, max_pages, num_pages, 64};
  Pool p{pool, layers, layer_stride, page_bytes};
  MOE_TRY(check_state(s));
  MOE_TRY(check_pool(p));
  if (!remap || !aligned(remap, 4)) return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_ws(ws, ws_bytes, num_pages, 0));
  unsigned int* err = device_error_word();
  if (!err) return MOE_ERR_CUDA;
  Plan w = carve(ws, num_pages, 0, nullptr);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int wide = std::max(1, std::min(num_sms(), (num_pages + 4 * kPlan - 1) / (4 * kPlan)));
  compact_plan_kernel<<<1 + wide, kPlan, 0, st>>>(s, w, remap);
  MOE_TRY(check_launch());
  const long long entries = std::max<long long>(static_cast<long long>(rows) * max_pages, num_pages / 2);
  const int small = static_cast<int>(
      std::max<long long>(1, std::min<long long>(num_sms(), (entries + 4 * kCopyThreads - 1) / (4 * kCopyThreads))));
  return kv4::launch_after(compact_apply_kernel, dim3(small + copy_blocks(p, num_pages / 2)), kCopyThreads, 0, st, s, w, p,
                           remap, small, err);
}

extern "C" int moe_kv_copy_pages(uint8_t* pool, int layers, long long layer_stride, long long page_bytes, int num_pages,
                                 const int32_t* src, const int32_t* dst, int n, void* stream) {
  Pool p{pool, layers, layer_stride, page_bytes};
  if (n < 0 || num_pages < 1) return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_pool(p));
  if (n == 0 || layers == 0) return MOE_OK;
  if (!src || !dst || !aligned(src, 4) || !aligned(dst, 4)) return MOE_ERR_INVALID_ARG;
  unsigned int* err = device_error_word();
  if (!err) return MOE_ERR_CUDA;
  copy_kernel<<<copy_blocks(p, n), kCopyThreads, 0, static_cast<cudaStream_t>(stream)>>>(p, src, dst, n, num_pages, err);
  return check_launch();
}
