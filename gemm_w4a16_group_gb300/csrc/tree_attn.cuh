// What the attention kernels over the paged cache share: the work list, the
// partial results and their workspace, and the rules for single keys.
//
// Work list. Row b of the page table with T new tokens and L cached ones has
// K = L + T keys; its T * G query rows of one kv head (G query heads each) are
// packed token by token into tiles of ROWS rows, so its items are
// (kv head, row tile), each of ceil(K / KT) key tiles. A key tile counts some
// units by its query rows (the tcgen05 kernel works on up to 256, and takes half
// as long again over more than 128 as over fewer), and an item counts LEAD key
// tiles more, for what beginning and ending an item costs. All items, in
// the order (b, head, row tile), form one list of units, and every CTA takes an
// equal, contiguous share of it (to whole key tiles), whatever the lengths are:
// long contexts are split over many CTAs, short ones share one. An item whose tiles
// lie in one share is finished there; otherwise each CTA leaves a partial
// result (running maximum, sum and unnormalised output per row) in the
// workspace, and a second kernel joins them in the order of the CTAs, so
// results do not depend on timing. A CTA leaves at most two partials: of the
// item it begins in the middle of (slot 0), and of the one it does not end
// (slot 1). The CTA that ends an item which others began leaves a record of it,
// at most one per CTA, and the joining kernel works through the records.
#pragma once

#include "w4a16_internal.h"

namespace w4a16 {

constexpr int kMaxCtas = 320;    // CTAs of an attention launch: shares of the work list
constexpr int kTcMaxCtas = 160;  // of the tcgen05 kernel
// the tcgen05 kernel (tree_attn_tc.cu): query rows of an item, keys of a tile
constexpr int tc_attn_rows(int dim, bool e4m3) { return dim == 256 || e4m3 ? 128 : 256; }
constexpr int tc_attn_keys(int dim) { return dim == 256 ? 64 : 128; }
// Tables of so few keys are worked on without splitting items, so nothing has
// to be joined, and no second launch is made (2.3 us of the host's time). On the
// device, whole against split: one row of 400 keys 13.1 and 14.3 us, 40 rows of
// 400 24.4 and 24.4, of 700 34.9 and 29.8; on the tcgen05 kernel 12 rows of 700
// keys 19.6 and 24.5 us, one of 1,000 with 40 nodes 30.0 and 24.0.
constexpr long long kWholeKeys = 512, kTcWholeKeys = 768;
constexpr float kLog2e = 1.4426950408889634f;

struct AttnParams {
  const uint16_t *q;
  long long q_token, q_head;
  KvCache c;
  KvRows r;
  const int64_t *mask;
  int heads, group, max_tree;
  bool whole;        // items are not split: one belongs to the share that holds its first unit
  float scale_log2;  // scale * log2(e): scores are kept in powers of two
  uint16_t *out;
  float *partials;       // [kMaxCtas][2] partials, see Partial
  int *joins;            // [kMaxCtas] query rows of the item that a CTA ended for others (0: none), then
                         // [kMaxCtas] of its first CTA, first token, first query row and kv head
  int *err;
};

// One partial: unnormalised outputs as [DIM / 4][ROWS] blocks of four elements
// of a row, so that threads that own neighbouring rows write neighbouring
// addresses, then maximum and sum of every row
template <int DIM, int ROWS>
struct Partial {
  static constexpr int kFloats = ROWS * (DIM + 2);
  float *base;
  __device__ Partial(float *all, long long cta, int slot) : base(all + (cta * 2 + slot) * kFloats) {}
  __device__ float *at(int r, int d) const { return base + ((d >> 2) * ROWS + r) * 4 + (d & 3); }
  __device__ float2 *ml(int r) const { return reinterpret_cast<float2 *>(base + ROWS * DIM) + r; }
};

// a / b of numbers that are not negative. A 64-bit division takes some hundred
// instructions, and nearly every work list fits 32 bits.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// One row of the table as the work list sees it
struct RowInfo {
  int start, n, len, keys;  // first token, new tokens, cached, len + n (no more than the table holds)
};

__device__ __forceinline__ void attn_flag(int *err) { atomicOr(err, kErrIndex); }

// n = 0 for a row without new tokens or with numbers that cannot be; `flag`: report those
__device__ __forceinline__ RowInfo row_info(const AttnParams &p, int b, bool flag) {
  RowInfo i;
  i.start = p.r.starts[b];
  const int end = p.r.starts[b + 1];
  i.len = p.r.lengths[b];
  i.n = end - i.start;
  if (i.start < 0 || end > p.r.tokens || i.n < 0 || i.n > p.max_tree || i.len < 0) {
    if (flag) attn_flag(p.err);
    i.n = 0;
  }
  const long long room = (long long)p.r.max_pages << p.c.page_shift;
  const long long keys = (long long)i.len + i.n;
  if (i.n > 0 && keys > room && flag) attn_flag(p.err);
  i.keys = (int)min(keys, min(room, (long long)INT32_MAX - 4096));
  return i;
}

// Query rows of an item, keys of a tile, query rows of a narrow item, key tiles that an item costs by itself
template <int ROWS_, int KT_, int NARROW_, int LEAD_>
struct Tiling {
  static constexpr int ROWS = ROWS_, KT = KT_, NARROW = NARROW_, LEAD = LEAD_;
  static constexpr int FULL_COST = ROWS > NARROW ? 3 : 1;  // units of a key tile of a full item
  static __device__ __forceinline__ int cost(int rows) { return ROWS > NARROW ? (rows > NARROW ? 3 : 2) : 1; }
  // key tiles in some of an item's units (fewer than 2^32: an item has under 2^31 keys)
  static __device__ __forceinline__ int tiles(long long units, int cost) {
    const uint32_t u = (uint32_t)units;
    return (int)(ROWS > NARROW ? (cost == 3 ? u / 3u : u >> 1) : u);
  }
};

template <int KT>
__device__ __forceinline__ int key_tiles(const RowInfo &i) {
  return (i.keys + KT - 1) / KT;
}
template <int ROWS>
__device__ __forceinline__ int row_tiles(const RowInfo &i, int group) {
  return (i.n * group + ROWS - 1) / ROWS;
}
// of one kv head; all of them count the same
template <class T>
__device__ __forceinline__ long long units_of(const RowInfo &i, const AttnParams &p) {
  if (i.n == 0) return 0;
  const int rows = i.n * p.group, full = (rows - 1) / T::ROWS;  // (the last item is full or less)
  return (long long)(key_tiles<T::KT>(i) + T::LEAD) * (full * T::FULL_COST + T::cost(rows - full * T::ROWS));
}

// A CTA's place in the work list: units [at, end) are its share, `unit` is the
// first one of the item it has come to
struct Cursor {
  long long at, end, unit;
  int b, head, rt;
};

struct PlanShared {
  long long sums[16];
  long long at, end, share, unit;
  int b, head, rt;
};

// The CTA's share, found by all NT threads: thread i sums the tiles of its
// own run of rows, a block scan places the runs, and the thread whose run holds
// the share's first tile walks it. The CTA's record is cleared. The caller
// synchronises before it reads `s`.
template <class T, int NT>
__device__ void plan_share(const AttnParams &p, PlanShared &s) {
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int per = (p.r.rows + NT - 1) / NT;
  const int b0 = min(tid * per, p.r.rows), b1 = min(b0 + per, p.r.rows);
  const bool flag = blockIdx.x == 0;  // one CTA reports rows that cannot be
  long long mine = 0, per_head = 0;
  RowInfo i;  // of the run's last row (nearly always its only one)
  for (int b = b0; b < b1; ++b) {
    i = row_info(p, b, flag);
    per_head = units_of<T>(i, p);
    mine += per_head * p.c.kv_heads;
  }
  long long upto = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xFFFFFFFFu, upto, d);
    if (lane >= d) upto += o;
  }
  if (lane == 31) s.sums[w] = upto;
  __syncthreads();
  long long before = 0, total = 0;
#pragma unroll
  for (int i = 0; i < (NT + 31) / 32; ++i) {
    const long long x = s.sums[i];
    if (i < w) before += x;
    total += x;
  }
  const long long first = before + upto - mine;
  // As many CTAs as get two key tiles of a narrow item each (a share then holds a whole one of any item), and no share
  // larger than it has to be. One token, or 16 nodes, over 2,048 keys: 13.7 and 16.0 us; with three 14.6 and 16.6, with
  // four 14.4 and 17.4.
  const long long ctas = max(1ll, min((long long)gridDim.x, quotient(total, 2 * T::cost(1))));
  const long long share = max(1ll, quotient(total + ctas - 1, ctas));
  const long long at = min(share * blockIdx.x, total), end = min(at + share, total);
  if (tid == 0) {
    s.at = at;
    s.end = end;
    s.share = share;
    p.joins[blockIdx.x] = 0;
  }
  if (at < end && first <= at && at < first + mine) {
    long long f = first;
    int b = b0;
    if (per > 1)
      for (;; ++b) {
        i = row_info(p, b, false);
        per_head = units_of<T>(i, p);
        if (at < f + per_head * p.c.kv_heads) break;
        f += per_head * p.c.kv_heads;
      }
    const long long o = at - f;
    const int head = (int)quotient(o, per_head);
    int rt = 0;
    long long unit = f + head * per_head;
    if (i.n * p.group > T::ROWS) {
      const long long per_tile = (long long)(key_tiles<T::KT>(i) + T::LEAD) * T::FULL_COST;  // a full item
      rt = (int)quotient(at - unit, per_tile);
      unit += rt * per_tile;
    }
    s.b = b;
    s.head = head;
    s.rt = rt;
    s.unit = unit;
  }
}

// The part of an item that a CTA works on: key tiles [kt0, kt1)
struct Segment {
  RowInfo i;
  int b, head, rt, rows, kt0, kt1, ktiles;
  long long first;  // unit of the item's first key tile
  int cost;         // units of a key tile
  __device__ bool whole() const { return kt0 == 0 && kt1 == ktiles; }
};

// Leaves the record of an item that this CTA ends and others began (one thread)
template <class T>
__device__ __forceinline__ void leave_record(const AttnParams &p, const Segment &s, long long share) {
  const int first_cta = (int)quotient(s.first + s.cost - 1, share);  // that has a part of the item
  reinterpret_cast<int4 *>(p.joins + kMaxCtas)[blockIdx.x] = make_int4(first_cta, s.i.start, s.rt * T::ROWS, s.head);
  p.joins[blockIdx.x] = s.rows;
}

// Next segment of the share (false: none is left)
template <class T>
__device__ __forceinline__ bool next_segment(const AttnParams &p, Cursor &c, Segment &s) {
  while (c.unit < c.end) {
    s.i = row_info(p, c.b, false);
    while (s.i.n == 0) s.i = row_info(p, ++c.b, false);  // rows without work; units are left, so one with work follows
    s.b = c.b;
    s.head = c.head;
    s.rt = c.rt;
    s.rows = min(T::ROWS, s.i.n * p.group - c.rt * T::ROWS);
    s.ktiles = key_tiles<T::KT>(s.i);
    const int cost = T::cost(s.rows);
    const bool mine = c.unit >= c.at;  // whole items: this share's (the list ends it at the first beyond)
    const long long first = c.unit + T::LEAD * cost, units = (long long)s.ktiles * cost;  // of the item's first tile
    // a key tile belongs to the share that holds its last unit
    s.kt0 = c.at > first ? T::tiles(c.at - first, cost) : 0;
    s.kt1 = c.end - first >= units ? s.ktiles : c.end > first ? T::tiles(c.end - first, cost) : 0;
    if (p.whole) {
      s.kt0 = 0;
      s.kt1 = mine ? s.ktiles : 0;
    }
    s.first = first;
    s.cost = cost;
    c.unit = first + units;
    if (++c.rt == row_tiles<T::ROWS>(s.i, p.group)) {
      c.rt = 0;
      if (++c.head == p.c.kv_heads) {
        c.head = 0;
        ++c.b;
      }
    }
    if (s.kt0 < s.kt1) return true;
  }
  return false;
}

cudaError_t launch_tree_tc(const AttnCall &c, const AttnParams &p);

template <class... K, class... A>
inline cudaError_t launch_dependent(void (*kern)(K...), unsigned grid, int threads, size_t smem, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(grid, 1, 1);
  lc.blockDim = dim3(threads, 1, 1);
  lc.dynamicSmemBytes = smem;
  lc.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, kern, args...);
}

// Tensor map of one side of a cache layer: (element, row, head, page), boxes of
// `box_rows` rows by `box_bytes` bytes, swizzled over the box's width if asked
bool encode_cache(CUtensorMap *m, const KvSide &s, const KvCache &c, int box_rows, int box_bytes, bool swizzled);

// 4-D tiled TMA load
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void *tmap, int c0, int c1, int c2, int c3, uint32_t bar,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar), "l"(policy)
      : "memory");
}

// four e4m3 codes as two f16x2 (codes 0 and 1, codes 2 and 3), exactly
__device__ __forceinline__ void e4m3x4_f16(uint32_t x, uint32_t &lo, uint32_t &hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(x));
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

}  // namespace w4a16
