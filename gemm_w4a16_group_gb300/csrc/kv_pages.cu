// The paged key/value cache around the drafted-token attention: writing new
// tokens' rows (append), the greedy walk down a draft tree (accept), moving
// the accepted rows together (compact), and the page table's upkeep (free,
// fork, reserve). Everything here moves bytes or counts pages, so HBM and, for
// the small calls, launch and load latency are the only bounds.
//
// Indices that only the device sees (page ids, lengths, starts, row numbers)
// are checked where they are used; a bad one sets kErrIndex and is skipped.
#include <cuda_fp8.h>

#include <algorithm>
#include <climits>

#include "w4a16_internal.h"

namespace w4a16 {
namespace {

__device__ __forceinline__ void flag_index(int *err) { atomicOr(err, kErrIndex); }

// Byte offset of position `pos` of table row `b` inside one head of one
// layer, or -1 when the position or its page id is out of range.
__device__ __forceinline__ long long row_offset(const KvSide &s, const KvRows &r, int page_shift, int pages, int b,
                                                long long pos) {
  const long long pi = pos >> page_shift;
  if (pos < 0 || pi >= r.max_pages) return -1;
  const int id = r.table[(long long)b * r.max_pages + pi];
  if ((unsigned)id >= (unsigned)pages) return -1;
  return (long long)id * s.page + (pos & ((1 << page_shift) - 1)) * s.row;
}

// The row that each lane's token belongs to: the last b with starts[b] <= token
// (rows without tokens are passed over); `rows` when the token is padding.
// `token` ascends by one from lane to lane. The warp looks for lane 0's row, 32
// starts at a time; most lanes' tokens are in the same one.
__device__ __forceinline__ int owner_of(const int32_t *starts, int rows, int token) {
  const int lane = threadIdx.x & 31, token0 = token - lane;
  int lo = 0, n = rows;  // lane 0's row, the first b with starts[b + 1] > token0, is one of lo .. lo + n
  while (n > 0) {
    const int step = (n + 31) / 32, probe = lo + min((lane + 1) * step, n);
    const uint32_t above = __ballot_sync(0xFFFFFFFFu, starts[probe] > token0);
    if (!above) {
      lo += n;
      break;
    }
    const int part = __ffs(above) - 1;
    lo += part * step;
    n = min(step, n - part * step) - 1;
  }
  if (lo >= rows || starts[lo + 1] > token) return lo;
  int hi = rows;
  for (++lo; lo < hi;) {
    const int mid = (lo + hi) >> 1;
    if (starts[mid + 1] > token) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// ---------------------------------------------------------------------------
// append: a thread has one 16-byte chunk of one head in four tokens, all in
// flight at once. Bound by HBM; in 8 bits nearly as much by the integer pipe,
// which unpacks and converts: 25,446 tokens of 8 heads of 128 to e4m3 (156 MB)
// 28.7 us, 5.4 TB/s (blocks of 256 threads 29.3 us, of 512 35.2; eight tokens a
// thread 28.5).
// ---------------------------------------------------------------------------
constexpr int kAppendThreads = 128;
constexpr int kAppendBatch = 4;  // tokens of a thread
constexpr int kAppendTokens = kAppendThreads / 8 * kAppendBatch;  // of a block at most (a token has 8 chunks or more)

struct AppendParams {
  const uint16_t *src[2];
  long long token_stride[2], head_stride[2];  // elements
  KvSide side[2];
  KvRows r;
  int kv_heads, dim_chunks_log2, page_shift, pages;
  int per_token, groups;  // chunks of a token; tokens side by side in a block
  int *err;
};

// Eight quotients x / s, correctly rounded, from r = 1 / s: x * r corrected
// once by its residual (P. Markstein, "IA-64 and Elementary Functions", ch. 8).
// The residual is formed as q * s - x and taken off: with x - q * s added, the
// quotient of a negative zero would lose its sign. r = 0 stands for a scale
// outside 2^-60 .. 2^60, where a residual could underflow; there, and where one
// of the eight quotients is 1,024 or more (its residual need not be finite),
// all eight take the division, which gives the same codes.
__device__ __forceinline__ float2 divisor_of(float s) {
  return make_float2(s, s > 8.6736174e-19f && s < 1.1529215e18f ? __fdiv_rn(1.f, s) : 0.f);
}
__device__ __forceinline__ uint2 to_e4m3(const uint4 &x, const float2 &d) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  const f32x2 minus_r2 = f32_pair(-d.y, -d.y), s2 = f32_pair(d.x, d.x);
  f32x2 minus[4], q2[4];  // -x, x * r
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t v = w[i] ^ 0x80008000u;
    minus[i] = f32_pair(bf16lo_to_f32(v), bf16hi_to_f32(v));
    q2[i] = mul2(minus[i], minus_r2);
    const float2 q = f32_halves(q2[i]);
    top = fmaxf(fmaxf(top, fabsf(q.x)), fabsf(q.y));
  }
  float2 q[4];
  if (d.y != 0.f && top < 1024.f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = f32_halves(fma2(fma2(q2[i], s2, minus[i]), minus_r2, q2[i]));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      q[i] = make_float2(__fdiv_rn(bf16lo_to_f32(w[i]), d.x), __fdiv_rn(bf16hi_to_f32(w[i]), d.x));
  }
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = __nv_cvt_float2_to_fp8x2(q[i], __NV_SATFINITE, __NV_E4M3);
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// A block moves some tokens' rows of one side (blockIdx.y), or of heads with
// more chunks than it has threads a part (blockIdx.z). Its data does not depend
// on where it goes, so the loads are in flight while some threads look up the
// places.
template <bool E4M3>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const __grid_constant__ AppendParams p) {
  __shared__ long long off[kAppendTokens];
  grid_dependency_wait();
  grid_launch_dependents();
  const bool values = blockIdx.y != 0;
  const KvSide &s = values ? p.side[1] : p.side[0];
  const long long token_stride = values ? p.token_stride[1] : p.token_stride[0];
  const int t0 = blockIdx.x * p.groups * kAppendBatch;
  const int nt = min(p.groups * kAppendBatch, p.r.tokens - t0);
  const int group = threadIdx.x / p.per_token, chunk = blockIdx.z * kAppendThreads + threadIdx.x - group * p.per_token;
  const int h = chunk >> p.dim_chunks_log2, c = chunk & ((1 << p.dim_chunks_log2) - 1);
  const int n = group < p.groups && chunk < p.per_token ? nt : 0;  // (the last threads may have no chunk)
  uint4 x[kAppendBatch];
  float scale = 0.f;
  if (n > 0) {
    const uint16_t *src = (values ? p.src[1] : p.src[0]) + (long long)(t0 + group) * token_stride +
                          h * (values ? p.head_stride[1] : p.head_stride[0]) + c * 8;
#pragma unroll
    for (int u = 0; u < kAppendBatch; ++u)
      if (group + u * p.groups < n) x[u] = *reinterpret_cast<const uint4 *>(src + u * p.groups * token_stride);
    if (E4M3) scale = s.scale[h];
  }
  if ((int)(threadIdx.x & ~31u) < nt) {
    const int t = t0 + threadIdx.x;
    const int b = owner_of(p.r.starts, p.r.rows, t);
    long long o = -1;
    if (b < p.r.rows && (int)threadIdx.x < nt) {
      const int first = p.r.starts[b], len = p.r.lengths[b];
      // (starts that descend or do not begin at 0 leave a token before its row's first)
      if (t >= first && len >= 0) o = row_offset(s, p.r, p.page_shift, p.pages, b, (long long)len + (t - first));
      if (o < 0) flag_index(p.err);
    }
    if ((int)threadIdx.x < nt) off[threadIdx.x] = o;
  }
  const float2 divisor = E4M3 ? divisor_of(scale) : make_float2(0.f, 0.f);
  __syncthreads();
  uint8_t *dst = s.base + h * s.head + c * (E4M3 ? 8 : 16);
#pragma unroll
  for (int u = 0; u < kAppendBatch; ++u) {
    const int t = group + u * p.groups;
    if (t >= n) break;
    const long long o = off[t];
    if (o < 0) continue;
    if (E4M3) *reinterpret_cast<uint2 *>(dst + o) = to_e4m3(x[u], divisor);
    else *reinterpret_cast<uint4 *>(dst + o) = x[u];
  }
}

// ---------------------------------------------------------------------------
// accept: one warp per row; lane l holds nodes l and l + 32, and each step of
// the walk is one vote over "is a fitting child of the node I stand on"
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(32) tree_accept_kernel(const int64_t *target, const int64_t *draft,
                                                         const int64_t *mask, const int32_t *starts, int rows,
                                                         int tokens, int max_tree, int32_t *path, int32_t *count,
                                                         int64_t *token, int *err) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int b = blockIdx.x, lane = threadIdx.x;
  const int s0 = starts[b], s1 = starts[b + 1];
  int n = s1 - s0;
  if (s0 < 0 || n < 0 || n > max_tree || s1 > tokens) {
    if (lane == 0) flag_index(err);
    n = 0;
  }
  int parent[2];
  bool fits[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int node = lane + 32 * i;
    parent[i] = -1;
    fits[i] = false;
    if (node < n) {
      const unsigned long long word = mask ? (unsigned long long)mask[s0 + node] : ~0ull;
      const unsigned long long above = word & ((1ull << node) - 1);
      parent[i] = above ? 63 - __clzll(above) : -1;
      fits[i] = parent[i] >= 0 && draft[s0 + node] == target[s0 + parent[i]];
    }
  }
  int cur = 0, got = n > 0 ? 1 : 0;
  int mine[2] = {lane == 0 && n > 0 ? 0 : -1, -1};
  while (n > 0) {  // a child's index is above its parent's: at most n steps
    const uint32_t lo = __ballot_sync(0xFFFFFFFFu, fits[0] && parent[0] == cur);
    const uint32_t hi = __ballot_sync(0xFFFFFFFFu, fits[1] && parent[1] == cur);
    if (!(lo | hi)) break;
    cur = lo ? __ffs(lo) - 1 : 31 + __ffs(hi);
    if (lane == got) mine[0] = cur;
    if (lane + 32 == got) mine[1] = cur;
    ++got;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (lane + 32 * i < max_tree) path[(long long)b * max_tree + lane + 32 * i] = mine[i];
  if (lane == 0) {
    count[b] = got;
    token[b] = got ? target[s0 + cur] : -1;
  }
}

// ---------------------------------------------------------------------------
// compact: one warp per (row, layer, side, head). Accepted nodes ascend, so
// path[i] >= i and no later move reads a row that an earlier one wrote; a
// batch of rows is read whole before any of it is written. Bound by latency:
// lengths, path, page ids and rows are loads that depend on one another (32
// trees of 32 nodes, 48 layers of 8 heads of 128, 25 MB, nothing in a cache:
// 11.8 us, the acceptance before it 4.2 us).
// ---------------------------------------------------------------------------
constexpr int kCompactWarps = 8;

struct CompactParams {
  KvSide side[2];
  KvRows r;
  const int32_t *path, *count;
  int32_t *lengths_out;
  int layers, kv_heads, page_shift, pages, max_tree, row_chunks_log2;
  int *err;
};

__global__ void __launch_bounds__(kCompactWarps * 32) kv_compact_kernel(const CompactParams p) {
  __shared__ long long src_off[kCompactWarps][kMaxTree], dst_off[kCompactWarps][kMaxTree];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int b = blockIdx.y;
  const int slab = blockIdx.x * kCompactWarps + w;  // (layer, side, head)
  const int slabs = p.layers * 2 * p.kv_heads;
  if (slab >= slabs) return;
  const int head = slab % p.kv_heads, side = slab / p.kv_heads % 2, layer = slab / (2 * p.kv_heads);
  const KvSide &s = p.side[side];
  const int len = p.r.lengths[b];
  int n = p.count[b];
  // the lane's two path entries, each checked against the one before it
  int at[2];
  bool bad = len < 0 || n < 0 || n > p.max_tree;
  if (bad) n = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int j = lane + 32 * i;
    at[i] = j < n ? p.path[(long long)b * p.max_tree + j] : j;
    const int before = j > 0 && j < n ? p.path[(long long)b * p.max_tree + j - 1] : -1;
    if (j < n && (at[i] < j || at[i] >= p.max_tree || (j > 0 && at[i] <= before))) bad = true;
  }
  bad = __any_sync(0xFFFFFFFFu, bad);
  if (!bad && slab == 0 && lane == 0) p.lengths_out[b] = len + n;
  if (bad) {
    if (slab == 0 && lane == 0) {
      p.lengths_out[b] = len;
      flag_index(p.err);
    }
    return;
  }
  // rows that move, and from where
  bool lost = false;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int j = lane + 32 * i;
    if (j < n) {
      const bool moves = at[i] != j;
      const long long f = moves ? row_offset(s, p.r, p.page_shift, p.pages, b, (long long)len + at[i]) : -1;
      const long long t = moves ? row_offset(s, p.r, p.page_shift, p.pages, b, (long long)len + j) : -1;
      if (moves && (f < 0 || t < 0)) lost = true;
      src_off[w][j] = f;
      dst_off[w][j] = f < 0 ? -1 : t;
    }
  }
  if (lost) flag_index(p.err);
  __syncwarp();
  uint8_t *base = s.base + (long long)layer * s.layer + (long long)head * s.head;
  const int chunks = n << p.row_chunks_log2;  // 16-byte chunks, row by row
  constexpr int U = 4;
  for (int c0 = 0; c0 < chunks; c0 += 32 * U) {
    uint4 x[U];
    long long to[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * 32 + lane;
      to[u] = -1;
      if (c < chunks) {
        const int j = c >> p.row_chunks_log2;
        const int o = (c & ((1 << p.row_chunks_log2) - 1)) * 16;
        if (dst_off[w][j] >= 0) {
          x[u] = *reinterpret_cast<const uint4 *>(base + src_off[w][j] + o);
          to[u] = dst_off[w][j] + o;
        }
      }
    }
    __syncwarp();
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (to[u] >= 0) *reinterpret_cast<uint4 *>(base + to[u]) = x[u];
    __syncwarp();
  }
}

// ---------------------------------------------------------------------------
// the page table: one CTA each, so that every decision is in one fixed order
// (freeing decides nothing: a warp per row). Bound by launch and dependent
// loads: 48 rows of 16 entries and 512 pages, freed 4 us, branched 8, given
// room 7.5, with nothing in a cache.
// ---------------------------------------------------------------------------
constexpr int kTableThreads = 1024;

// Inclusive sum over the block of one value per thread (all threads call it).
template <class T>
__device__ T block_scan(T v, T *warp_sums) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const T o = __shfl_up_sync(0xFFFFFFFFu, v, d);
    if (lane >= d) v += o;
  }
  if (lane == 31) warp_sums[w] = v;
  __syncthreads();
  if (w == 0) {
    T s = warp_sums[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const T o = __shfl_up_sync(0xFFFFFFFFu, s, d);
      if (lane >= d) s += o;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  if (w > 0) v += warp_sums[w - 1];
  __syncthreads();  // warp_sums may be written again
  return v;
}

// Hands the free pages (refs == 0), lowest id first, to take(k, page) for k =
// 0 .. need - 1. True if there are that many; nothing is taken otherwise.
template <class Take>
__device__ bool take_free_pages(int32_t *refs, int pages, int need, int *warp_sums, int *shared_total, Take take) {
  if (need == 0) return true;
  for (int pass = 0; pass < 2; ++pass) {
    int seen = 0;
    for (int p0 = 0; p0 < pages && seen < need; p0 += kTableThreads) {
      const int page = p0 + threadIdx.x;
      const bool free = page < pages && refs[page] == 0;
      const int upto = block_scan<int>(free ? 1 : 0, warp_sums);
      if (threadIdx.x == kTableThreads - 1) *shared_total = upto;
      if (pass == 1 && free && seen + upto - 1 < need) {
        refs[page] = 1;
        take(seen + upto - 1, page);
      }
      __syncthreads();
      seen += *shared_total;
      __syncthreads();
    }
    if (seen < need) return false;
  }
  return true;
}

// the row of item k among n rows with inclusive sums `ends` (ascending)
__device__ __forceinline__ int row_of_item(const int *ends, int n, int k) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (ends[mid] > k) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kTableThreads) kv_free_kernel(int32_t *table, int max_pages, int table_rows,
                                                                int32_t *lengths, int32_t *refs, int pages,
                                                                const int32_t *rows, int n, int *err) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int nw = gridDim.x * (blockDim.x >> 5);
  for (int j = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); j < n; j += nw) {
    const int b = rows[j];
    bool bad = (unsigned)b >= (unsigned)table_rows;
    for (int i = lane; i < j; i += 32) bad = bad || rows[i] == b;  // named twice: dropped once
    if (__any_sync(0xFFFFFFFFu, bad)) {
      if (lane == 0) flag_index(err);
      continue;
    }
    int32_t *row = table + (long long)b * max_pages;
    for (int c0 = 0; c0 < max_pages; c0 += 32) {
      const int c = c0 + lane;
      const int id = c < max_pages ? row[c] : -1;
      if (id >= 0) {
        row[c] = -1;
        if (id >= pages) {
          flag_index(err);
        } else if (atomicSub(&refs[id], 1) <= 0) {  // was free already: leave it so
          atomicAdd(&refs[id], 1);
          flag_index(err);
        }
      }
      if (!__any_sync(0xFFFFFFFFu, id >= 0)) break;  // entries in use come first
    }
    if (lane == 0) lengths[b] = 0;
  }
}

struct ForkParams {
  int32_t *table, *lengths, *refs;
  int max_pages, table_rows, pages, page_shift;
  const int32_t *src, *dst;
  int n;
  int32_t *ok;
  int *err;
};

// Plans a fork: checks every pair, counts the copies it needs, takes the free
// pages and writes the new rows. Rows are claimed by their lengths entry (0 ->
// -1 - j), which also finds a row named twice.
__global__ void __launch_bounds__(kTableThreads) kv_fork_kernel(const ForkParams p) {
  __shared__ int warp_sums[32];
  __shared__ int shared_total, any_bad, total_need;
  __shared__ int ends[kMaxRows];
  grid_dependency_wait();
  grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  if (tid == 0) any_bad = 0;
  __syncthreads();
  const int page_rows = 1 << p.page_shift;
  for (int j = tid; j < p.n; j += kTableThreads) {
    const int s = p.src[j], d = p.dst[j];
    const bool bad = (unsigned)s >= (unsigned)p.table_rows || (unsigned)d >= (unsigned)p.table_rows;
    if (bad || p.table[(long long)d * p.max_pages] >= 0 || atomicCAS(&p.lengths[d], 0, -1 - j) != 0) any_bad = 1;
  }
  __syncthreads();
  int base = 0;
  for (int j0 = 0; j0 < p.n; j0 += kTableThreads) {
    const int j = j0 + tid;
    int part = 0;
    if (j < p.n && (unsigned)p.src[j] < (unsigned)p.table_rows) {
      const int len = p.lengths[p.src[j]];  // below 0 too where the source is claimed as a branch
      if (len < 0 || (((long long)len + page_rows - 1) >> p.page_shift) > p.max_pages) any_bad = 1;
      part = (len & (page_rows - 1)) ? 1 : 0;
    }
    const int upto = block_scan<int>(part, warp_sums);
    if (j < p.n) ends[j] = base + upto;
    if (tid == kTableThreads - 1) shared_total = upto;
    __syncthreads();
    base += shared_total;
    __syncthreads();
  }
  if (tid == 0) total_need = base;
  __syncthreads();
  // a source's entries must be pages of the cache (one warp per pair)
  for (int j = w; j < p.n && !any_bad; j += kTableThreads / 32) {
    const int s = p.src[j];
    const int used = (p.lengths[s] + page_rows - 1) >> p.page_shift;
    bool bad = false;
    for (int c = lane; c < used; c += 32)
      if ((unsigned)p.table[(long long)s * p.max_pages + c] >= (unsigned)p.pages) bad = true;
    if (bad) any_bad = 1;
  }
  __syncthreads();
  bool done = false;
  if (!any_bad) {
    done = take_free_pages(p.refs, p.pages, total_need, warp_sums, &shared_total, [&](int k, int page) {
      const int j = row_of_item(ends, p.n, k);
      p.table[(long long)p.dst[j] * p.max_pages + (p.lengths[p.src[j]] >> p.page_shift)] = page;
    });
  }
  __syncthreads();
  for (int j = w; j < p.n; j += kTableThreads / 32) {
    const int s = p.src[j], d = p.dst[j];
    if (done) {
      const int full = p.lengths[s] >> p.page_shift;
      for (int c = lane; c < full; c += 32) {
        const int id = p.table[(long long)s * p.max_pages + c];
        p.table[(long long)d * p.max_pages + c] = id;
        atomicAdd(&p.refs[id], 1);
      }
      __syncwarp();
      if (lane == 0) p.lengths[d] = p.lengths[s];
    } else if (lane == 0 && (unsigned)d < (unsigned)p.table_rows && p.lengths[d] == -1 - j) {
      p.lengths[d] = 0;
    }
  }
  if (tid == 0) {
    p.ok[0] = done ? 1 : 0;
    if (any_bad) flag_index(p.err);
  }
}

// The part-filled last page of every pair: one warp per (pair, layer, side, head).
// Bound by HBM: 48 branches of 32 layers of 8 heads of 128, 403 MB read and
// written in 52 us, 7.7 TB/s (several branches of one source read it from L2).
constexpr int kCopyWarps = 8;
struct CopyParams {
  KvSide side[2];
  const int32_t *table, *lengths, *src, *dst, *ok;
  int max_pages, page_shift, layers, kv_heads, row_chunks_log2;
};

__global__ void __launch_bounds__(kCopyWarps * 32) kv_fork_copy_kernel(const CopyParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  if (*p.ok == 0) return;
  const int j = blockIdx.y, lane = threadIdx.x & 31;
  const int slab = blockIdx.x * kCopyWarps + (threadIdx.x >> 5);
  if (slab >= p.layers * 2 * p.kv_heads) return;
  const int len = p.lengths[p.src[j]];
  const int rest = len & ((1 << p.page_shift) - 1), full = len >> p.page_shift;
  if (rest == 0) return;
  const int head = slab % p.kv_heads, side = slab / p.kv_heads % 2, layer = slab / (2 * p.kv_heads);
  const KvSide &s = p.side[side];
  uint8_t *base = s.base + (long long)layer * s.layer + (long long)head * s.head;
  const uint8_t *from = base + (long long)p.table[(long long)p.src[j] * p.max_pages + full] * s.page;
  uint8_t *to = base + (long long)p.table[(long long)p.dst[j] * p.max_pages + full] * s.page;
  const int chunks = rest << p.row_chunks_log2;
  constexpr int U = 8;
  for (int c0 = lane; c0 < chunks; c0 += 32 * U) {
    uint4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + 32 * u;
      if (c < chunks)
        x[u] = *reinterpret_cast<const uint4 *>(from + (long long)(c >> p.row_chunks_log2) * s.row +
                                                (c & ((1 << p.row_chunks_log2) - 1)) * 16);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + 32 * u;
      if (c < chunks)
        *reinterpret_cast<uint4 *>(to + (long long)(c >> p.row_chunks_log2) * s.row +
                                   (c & ((1 << p.row_chunks_log2) - 1)) * 16) = x[u];
    }
  }
}

struct ReserveParams {
  int32_t *table, *refs;
  int max_pages, table_rows, pages, page_shift;
  const int32_t *rows, *want;
  int n;
  int32_t *ok;
  int *err;
};

__global__ void __launch_bounds__(kTableThreads) kv_reserve_kernel(const ReserveParams p) {
  __shared__ int warp_sums[32];
  __shared__ long long wide_sums[32];
  __shared__ long long wide_total;
  __shared__ int shared_total, any_bad;
  __shared__ int ends[kMaxRows], have[kMaxRows];
  grid_dependency_wait();
  grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  if (tid == 0) any_bad = 0;
  __syncthreads();
  // pages that each row holds: its entries in use come first (one warp per row)
  for (int j = w; j < p.n; j += kTableThreads / 32) {
    const int b = p.rows[j];
    bool bad = (unsigned)b >= (unsigned)p.table_rows;
    for (int i = lane; i < j; i += 32) bad = bad || p.rows[i] == b;
    const int need = p.want[j];
    if (need < 0 || (((long long)need + (1 << p.page_shift) - 1) >> p.page_shift) > p.max_pages) bad = true;
    bad = __any_sync(0xFFFFFFFFu, bad);
    int held = 0;
    if (!bad) {
      for (int c0 = 0; c0 < p.max_pages; c0 += 32) {
        const int c = c0 + lane;
        const uint32_t m =
            __ballot_sync(0xFFFFFFFFu, c < p.max_pages && p.table[(long long)b * p.max_pages + c] >= 0);
        held += __popc(m);
        if (m != 0xFFFFFFFFu) break;
      }
    } else if (lane == 0) {
      any_bad = 1;
    }
    if (lane == 0) have[j] = held;
  }
  __syncthreads();
  long long base = 0;  // 4,096 rows of up to 2^27 pages each pass 32 bits
  for (int j0 = 0; j0 < p.n; j0 += kTableThreads) {
    const int j = j0 + tid;
    int more = 0;
    if (j < p.n && !any_bad) more = max(0, ((p.want[j] - 1) >> p.page_shift) + 1 - have[j]);
    const long long upto = block_scan<long long>(more, wide_sums);
    if (j < p.n) ends[j] = (int)min(base + upto, (long long)INT_MAX);
    if (tid == kTableThreads - 1) wide_total = upto;
    __syncthreads();
    base += wide_total;
    __syncthreads();
  }
  bool done = false;
  if (!any_bad && base <= p.pages)
    done = take_free_pages(p.refs, p.pages, (int)base, warp_sums, &shared_total, [&](int k, int page) {
      const int j = row_of_item(ends, p.n, k);
      const int first = j ? ends[j - 1] : 0;
      p.table[(long long)p.rows[j] * p.max_pages + have[j] + (k - first)] = page;
    });
  if (tid == 0) {
    p.ok[0] = done ? 1 : 0;
    if (any_bad) flag_index(p.err);
  }
}

// ---------------------------------------------------------------------------
// launch
// ---------------------------------------------------------------------------
int log2_of(int v) {
  int s = 0;
  while ((1 << s) < v) ++s;
  return s;
}

// Every kernel here waits for the work before it (griddepcontrol.wait) before
// its first access, so it may always be launched while that work ends.
template <class... K, class... A>
cudaError_t launch(void (*kern)(K...), dim3 grid, int threads, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t lc = {};
  lc.gridDim = grid;
  lc.blockDim = dim3(threads, 1, 1);
  lc.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, kern, args...);
}

}  // namespace

cudaError_t launch_kv_append(const AppendCall &c) {
  AppendParams p;
  p.src[0] = c.k;
  p.src[1] = c.v;
  p.token_stride[0] = c.k_token;
  p.token_stride[1] = c.v_token;
  p.head_stride[0] = c.k_head;
  p.head_stride[1] = c.v_head;
  p.side[0] = c.cache.k;
  p.side[1] = c.cache.v;
  p.r = c.rows;
  p.kv_heads = c.cache.kv_heads;
  p.dim_chunks_log2 = log2_of(c.cache.dim / 8);
  p.page_shift = c.cache.page_shift;
  p.pages = c.cache.pages;
  p.err = c.err;
  p.per_token = c.cache.kv_heads * (c.cache.dim / 8);
  p.groups = std::max(1, kAppendThreads / p.per_token);
  const int tokens = p.groups * kAppendBatch, parts = (p.per_token + kAppendThreads - 1) / kAppendThreads;
  // whole warps (they look for rows together)
  const int threads = std::min(kAppendThreads, (p.groups * p.per_token + 31) / 32 * 32);
  const dim3 grid((c.rows.tokens + tokens - 1) / tokens, 2, parts);
  return launch(c.cache.e4m3 ? kv_append_kernel<true> : kv_append_kernel<false>, grid, threads, c.stream, p);
}

cudaError_t launch_tree_accept(const int64_t *target, const int64_t *draft, const int64_t *mask, const int32_t *starts,
                               int rows, int tokens, int max_tree, int32_t *path, int32_t *count, int64_t *token,
                               int *err, cudaStream_t stream) {
  return launch(tree_accept_kernel, dim3(rows), 32, stream, target, draft, mask, starts, rows, tokens, max_tree, path,
                count, token, err);
}

cudaError_t launch_kv_compact(const KvCache &cache, const KvRows &r, const int32_t *path, const int32_t *count,
                              int max_tree, int32_t *lengths_out, int *err, cudaStream_t stream) {
  CompactParams p;
  p.side[0] = cache.k;
  p.side[1] = cache.v;
  p.r = r;
  p.path = path;
  p.count = count;
  p.lengths_out = lengths_out;
  p.layers = cache.layers;
  p.kv_heads = cache.kv_heads;
  p.page_shift = cache.page_shift;
  p.pages = cache.pages;
  p.max_tree = max_tree;
  p.row_chunks_log2 = log2_of(cache.row_bytes() / 16);
  p.err = err;
  const int slabs = cache.layers * 2 * cache.kv_heads;
  return launch(kv_compact_kernel, dim3((slabs + kCompactWarps - 1) / kCompactWarps, r.rows), kCompactWarps * 32,
                stream, p);
}

cudaError_t launch_kv_free(const TableCall &t, const int32_t *rows, int n) {
  const int warps = 4;
  return launch(kv_free_kernel, dim3((n + warps - 1) / warps), warps * 32, t.stream, t.table, t.max_pages,
                t.table_rows, t.lengths, t.refs, t.pages, rows, n, t.err);
}

cudaError_t launch_kv_fork(const TableCall &t, const KvCache &cache, const int32_t *src, const int32_t *dst, int n,
                           int32_t *ok) {
  ForkParams p{t.table, t.lengths, t.refs, t.max_pages, t.table_rows, t.pages, cache.page_shift, src, dst, n, ok,
               t.err};
  cudaError_t e = launch(kv_fork_kernel, dim3(1), kTableThreads, t.stream, p);
  if (e != cudaSuccess) return e;
  CopyParams c;
  c.side[0] = cache.k;
  c.side[1] = cache.v;
  c.table = t.table;
  c.lengths = t.lengths;
  c.src = src;
  c.dst = dst;
  c.ok = ok;
  c.max_pages = t.max_pages;
  c.page_shift = cache.page_shift;
  c.layers = cache.layers;
  c.kv_heads = cache.kv_heads;
  c.row_chunks_log2 = log2_of(cache.row_bytes() / 16);
  const int slabs = cache.layers * 2 * cache.kv_heads;
  return launch(kv_fork_copy_kernel, dim3((slabs + kCopyWarps - 1) / kCopyWarps, n), kCopyWarps * 32, t.stream, c);
}

cudaError_t launch_kv_reserve(const TableCall &t, int page_shift, const int32_t *rows, const int32_t *want, int n,
                              int32_t *ok) {
  ReserveParams p{t.table, t.refs, t.max_pages, t.table_rows, t.pages, page_shift, rows, want, n, ok, t.err};
  return launch(kv_reserve_kernel, dim3(1), kTableThreads, t.stream, p);
}

}  // namespace w4a16
