// Sampled decoding after the output head: the probabilities of bf16 logits,
// and the walk down a draft tree by two distributions and given random numbers
// (the sampled form of the greedy tree_accept, kv_pages.cu).
//
// A row of the vocabulary belongs to one cluster of CTAs, each with a slice of
// it; they exchange a few words through distributed shared memory. Both
// kernels are bound by HBM where there are many rows, and by launch, loads that
// depend on one another and the cluster's barriers where there is one.
#include "w4a16_internal.h"

namespace w4a16 {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kMaxCluster = 16;
using u64 = unsigned long long;

// The halves of a cluster barrier: what a CTA does between them need not wait
// for the others.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// A row of `n` elements seen in quads: quad k holds elements 4k - shift .. +3,
// so that whole quads are aligned wherever the row begins. [lo, hi) are the
// quads of part `i` of 2^log2. Loads of whole quads carry no condition that a
// branch would come of, so that many are on their way at once.
struct Quads {
  int shift, lo, hi;
  int whole_lo, whole_hi;  // those of [lo, hi) that are whole; the others are the row's first and last one
  __device__ __forceinline__ Quads(int n, int shift, uint32_t i, int log2) : shift(shift) {
    const uint32_t all = ((uint32_t)(shift + n) + 3) / 4, each = (all + (1u << log2) - 1) >> log2;
    lo = (int)min(i * each, all);
    hi = (int)min(i * each + each, all);
    whole_lo = max(lo, shift ? 1 : 0);
    whole_hi = max(min(hi, (shift + n) / 4), whole_lo);
  }
  // quad u of the ones at the part's ends, or -1
  __device__ __forceinline__ int end(int u) const {
    if (u == 0) return lo < min(whole_lo, hi) ? lo : -1;
    return whole_hi < hi && hi - 1 >= whole_lo ? hi - 1 : -1;
  }
  __device__ __forceinline__ bool is_whole(int k) const { return k >= whole_lo && k < whole_hi; }
  // Where quads begin `off` elements after words of four: the end of the words, from whole_lo on, that hold some of the whole
  // quads; each has an element of the row. (Without a whole quad there is none: the word at whole_hi may be past the row.)
  __device__ __forceinline__ int words_end(int off) const { return whole_hi + (off && whole_lo < whole_hi ? 1 : 0); }
};

// ---------------------------------------------------------------------------
// probabilities: p_j = 2^((l_j - m) a) / sum_i 2^((l_i - m) a), a = log2(e) / T.
// One pass: a thread holds 64 logits in registers while its own powers' sum (each
// relative to the thread's maximum) and the cluster's agree on one maximum and
// sum, then makes the powers again. Slices that do not fit are read twice.
//
// 256 rows of 248,320 (127 MB read, 254 written): 75 us, 5.1 TB/s, where HBM would
// take 57; a CTA loads, waits for its cluster and stores in turn, four of them an
// SM, with 46 % of issue slots taken (greedy rows, which need no powers: 70). Before
// those had a path of their own it took 83, and in other shapes, as threads x quads
// x CTAs an SM: 128 x 16 x 8 91 us, 256 x 8 x 6 94, 512 x 16 x 2 91, 512 x 8 x 3 112,
// 1024 x 8 x 1 138; as clusters that go on to further rows with the next one's logits
// copied ahead to shared memory 102. One row: 3.8 us, where a launch with a cluster barrier
// is most of it.
// ---------------------------------------------------------------------------
constexpr int kProbThreads = 256;
constexpr int kProbQuads = 16;  // of a thread
constexpr uint32_t kNone = 0xFF80FF80u;  // two bf16 -inf: no probability

struct ProbParams {
  const uint16_t *logits;
  long long row;  // elements from one row of logits to the next
  const float *temperature, *floor;
  float *out;
  int vocab;
};

// Four logits of the row, two to a word, one by one; -inf past its ends.
__device__ __forceinline__ uint2 load_end(const uint16_t *row, const Quads &q, int k, int n) {
  const int j = 4 * k - q.shift;
  uint32_t x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = j + i >= 0 && j + i < n ? row[j + i] : kNone & 0xFFFFu;
  return make_uint2(x[0] | x[1] << 16, x[2] | x[3] << 16);
}
// -inf where a logit is below the floor
__device__ __forceinline__ void drop(uint2 &w, float floor) {
  uint32_t *v = &w.x;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (bf16lo_to_f32(v[i]) < floor) v[i] = (v[i] & 0xFFFF0000u) | (kNone & 0xFFFFu);
    if (bf16hi_to_f32(v[i]) < floor) v[i] = (v[i] & 0xFFFFu) | (kNone & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void store_end(float *row, const Quads &q, int k, int n, float2 a, float2 b) {
  const int j = 4 * k - q.shift;
  const float v[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (j + i >= 0 && j + i < n) row[j + i] = v[i];
}
// Quads begin on 16 bytes of `out`. Where the row's logits are `off` of them after 8 bytes, a quad is in two words: its
// own and the next.
__device__ __forceinline__ uint2 from_words(uint2 w, uint2 next, int off) {
  const uint32_t a = off & 2 ? w.y : w.x, b = off & 2 ? next.x : w.y, c = off & 2 ? next.y : next.x;
  return make_uint2(__funnelshift_r(a, b, 16 * (off & 1)), __funnelshift_r(b, c, 16 * (off & 1)));
}
__device__ __forceinline__ uint2 load_word(const uint16_t *row, const Quads &q, int k, int off) {
  return *reinterpret_cast<const uint2 *>(row + 4 * k - q.shift - off);
}
__device__ __forceinline__ void store_whole(float *row, const Quads &q, int k, float2 a, float2 b) {
  *reinterpret_cast<float4 *>(row + 4 * k - q.shift) = make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ uint2 load_quad(const uint16_t *row, const Quads &q, int k, int off, int n) {
  if (!q.is_whole(k)) return load_end(row, q, k, n);
  const uint2 w = load_word(row, q, k, off);
  return from_words(w, off ? load_word(row, q, k + 1, off) : w, off);
}
__device__ __forceinline__ void store_quad(float *row, const Quads &q, int k, int n, float2 a, float2 b) {
  if (q.is_whole(k)) store_whole(row, q, k, a, b);
  else store_end(row, q, k, n, a, b);
}

__device__ __forceinline__ float exp2_fast(float y) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(y));
  return r;
}
// 2^((l - m) a) of two logits
__device__ __forceinline__ float2 powers(uint32_t w, f32x2 minus_m, f32x2 a) {
  const float2 y = f32_halves(mul2(add2(f32_pair(bf16lo_to_f32(w), bf16hi_to_f32(w)), minus_m), a));
  return make_float2(exp2_fast(y.x), exp2_fast(y.y));
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {  // (of a NaN and a number the number)
  const __nv_bfloat162 r = __hmax2(*reinterpret_cast<__nv_bfloat162 *>(&a), *reinterpret_cast<__nv_bfloat162 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&r);
}

__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {  // (of a NaN and a number the NaN)
  const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<__nv_bfloat162 *>(&a), *reinterpret_cast<__nv_bfloat162 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&r);
}

// all ones in the halves of x that are the ones of `top` (0 and -0 are the same, and so are NaNs)
__device__ __forceinline__ uint32_t same2(uint32_t x, uint32_t top) {
  const __nv_bfloat162 a = *reinterpret_cast<__nv_bfloat162 *>(&x), b = *reinterpret_cast<__nv_bfloat162 *>(&top);
  return __heq2_mask(a, b) | (__hisnan(b.x) ? ~__heq2_mask(a, a) : 0u);
}

__device__ __forceinline__ u64 key_max(u64 a, u64 b) { return a > b ? a : b; }

// (maximum, sum of powers relative to it) over the first N lanes' parts; an empty part is (lowest, 0)
template <int N>
__device__ __forceinline__ void join(float &m, float &s, float a) {
  const float mine = m;
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
  s = mine == m ? s : s * exp2_fast((mine - m) * a);
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
}

template <bool ALIGNED>
__global__ void __launch_bounds__(kProbThreads, 4) probabilities_kernel(const ProbParams p) {
  constexpr int kWarps = kProbThreads / 32;
  // !ALIGNED: a word's other half comes from the lane above, and the last lane's quads are the next warp's
  constexpr int kStep = ALIGNED ? kProbThreads : kWarps * 31, kQuads = ALIGNED ? kProbQuads : kProbQuads + 1;
  static_assert(kStep * kQuads >= kProbThreads * kProbQuads, "as much in a CTA's registers, however rows begin");
  __shared__ u64 slots[kMaxCluster], warps[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t S = cluster_nctarank(), rank = cluster_ctarank();
  const long long r = cluster_id_x();
  cluster_arrive();  // (a slot is written once its CTA runs)
  grid_dependency_wait();
  grid_launch_dependents();

  const uint16_t *row = p.logits + r * p.row;
  float *out = p.out + r * p.vocab;
  const Quads q(p.vocab, (int)(reinterpret_cast<uintptr_t>(out) >> 2 & 3), rank, __ffs(S) - 1);
  const int off = ALIGNED ? 0 : (int)((reinterpret_cast<uintptr_t>(row) >> 1) - q.shift & 3);
  const float t = p.temperature ? p.temperature[r] : 1.f, floor = p.floor ? p.floor[r] : -INFINITY;
  const bool greedy = !(t > 0.f), ends = q.whole_lo > q.lo || q.whole_hi < q.hi;

  // a logit of -inf stays -inf through difference and product, whatever the temperature (below 2^-127 as there, where the factor
  // is still a number)
  const float lowest = -3.40282347e38f, a = greedy ? 1.f : fmaxf(__fdiv_rn(1.44269502f, fmaxf(t, 5.87747175e-39f)), 1e-44f);
  const f32x2 a2 = f32_pair(a, a);
  uint2 x[kQuads];
  float m = lowest, s = 0.f, mine = lowest;
  u64 best = 0;
  const int at0 = ALIGNED ? tid : warp * 31 + lane;
  const bool own = ALIGNED || lane < 31;
  for (int k0 = q.lo; k0 < q.hi; k0 += kStep * kQuads) {
#pragma unroll
    for (int u = 0; u < kQuads; ++u) {
      const int k = k0 + u * kStep + at0;
      x[u] = make_uint2(kNone, kNone);
      if (k >= q.whole_lo && k < q.words_end(off)) x[u] = load_word(row, q, k, off);
    }
    if (!ALIGNED) {
#pragma unroll
      for (int u = 0; u < kQuads; ++u) {
        const uint2 next = make_uint2(__shfl_down_sync(kFull, x[u].x, 1), __shfl_down_sync(kFull, x[u].y, 1));
        x[u] = own && q.is_whole(k0 + u * kStep + at0) ? from_words(x[u], next, off) : make_uint2(kNone, kNone);
      }
    }
    if (ends && own) {
#pragma unroll
      for (int u = 0; u < kQuads; ++u) {
        const int k = k0 + u * kStep + at0;
        if (k < q.hi && !q.is_whole(k)) x[u] = load_end(row, q, k, p.vocab);
      }
    }
    if (floor > -INFINITY) {
#pragma unroll
      for (int u = 0; u < kQuads; ++u) drop(x[u], floor);
    }
    if (greedy) {  // the thread's maximum, then the first element that is it (none: -inf)
      uint32_t top = kNone;
#pragma unroll
      for (int u = 0; u < kQuads; ++u) top = max2_nan(top, max2_nan(x[u].x, x[u].y));
      top = max2_nan(top, top >> 16 | top << 16);
      const uint32_t key = order_key16(top & 0xFFFFu);
      if (top != kNone && key > (uint32_t)(best >> 32)) {
        uint32_t at = 0, lo = 0, hi = 0;
#pragma unroll
        for (int u = kQuads - 1; u >= 0; --u) {
          const uint32_t l = same2(x[u].x, top), h = same2(x[u].y, top);
          if (l | h) {
            at = u;
            lo = l;
            hi = h;
          }
        }
        const uint32_t i = lo ? (lo & 0xFFFFu ? 0 : 1) : hi & 0xFFFFu ? 2 : 3;
        best = (u64)key << 32 | (0xFFFFFFFFu - (uint32_t)(4 * (k0 + (int)at * kStep + at0) - q.shift + (int)i));
      }
      continue;
    }
    uint32_t top = kNone;
#pragma unroll
    for (int u = 0; u < kQuads; ++u) top = max2(top, max2(x[u].x, x[u].y));
    mine = fmaxf(fmaxf(bf16lo_to_f32(top), bf16hi_to_f32(top)), lowest);
    const f32x2 minus = f32_pair(-mine, -mine);
    f32x2 sum = 0;
#pragma unroll
    for (int u = 0; u < kQuads; ++u) {
      const float2 v = powers(x[u].x, minus, a2), w = powers(x[u].y, minus, a2);
      sum = add2(sum, add2(f32_pair(v.x, v.y), f32_pair(w.x, w.y)));
    }
    const float2 both = f32_halves(sum);
    const float high = fmaxf(m, mine);  // (more than one chunk: joined with the ones before)
    s = (m == high ? s : s * exp2_fast((m - high) * a)) + (mine == high ? 1.f : exp2_fast((mine - high) * a)) * (both.x + both.y);
    m = high;
  }
  if (greedy) {  // the first maximum has it all
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = key_max(best, __shfl_xor_sync(kFull, best, o));
    if (lane == 0) warps[warp] = best;
    __syncthreads();
    if (warp == 0) {  // (every lane gets it: up to 16 write it to the cluster's CTAs)
      best = lane < kWarps ? warps[lane] : 0;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) best = key_max(best, __shfl_xor_sync(kFull, best, o));
    }
    cluster_wait();
    if (tid < (int)S) st_cluster_u64(mapa_shared(smem_u32(&slots[rank]), tid), best);
    cluster_arrive();
    for (int k = q.lo + tid; k < q.hi; k += kProbThreads) store_quad(out, q, k, p.vocab, make_float2(0.f, 0.f), make_float2(0.f, 0.f));
    cluster_wait();
    best = 0;
    for (uint32_t i = 0; i < S; ++i) best = key_max(best, slots[i]);
    const int first = best ? (int)(0xFFFFFFFFu - (uint32_t)best) : -4, mine = (first + q.shift) >> 2;
    if (first >= 0 && mine >= q.lo && mine < q.hi && (mine - q.lo) % kProbThreads == tid) out[first] = 1.f;  // (over its own 0)
    return;
  }
  join<32>(m, s, a);
  if (lane == 0) warps[warp] = f32_pair(m, s);
  __syncthreads();
  if (warp == 0) {
    const float2 v = lane < kWarps ? f32_halves(warps[lane]) : make_float2(lowest, 0.f);
    m = v.x;
    s = v.y;
    join<32>(m, s, a);
  }
  cluster_wait();
  if (tid < (int)S) st_cluster_u64(mapa_shared(smem_u32(&slots[rank]), tid), f32_pair(m, s));
  cluster_sync_all();
  const float2 slot = (lane & 15) < (int)S ? f32_halves(slots[lane & 15]) : make_float2(lowest, 0.f);
  m = slot.x;
  s = slot.y;
  join<kMaxCluster>(m, s, a);
  const float inv = s == 0.f ? 0.f : __fdiv_rn(1.f, s);
  // each thread's logits are still in registers, where the slice is one chunk and the sum is a number (else a dropped
  // logit's 0 has to be told from a kept one's)
  if (q.hi - q.lo <= kStep * kQuads && s == s) {
    const f32x2 f2 = f32_pair(inv, inv), minus = f32_pair(-m, -m);
#pragma unroll
    for (int u = 0; u < kQuads; ++u) {
      const int k = q.lo + u * kStep + at0;
      const float2 v = powers(x[u].x, minus, a2), w = powers(x[u].y, minus, a2);
      const float2 a0 = f32_halves(mul2(f32_pair(v.x, v.y), f2)), b0 = f32_halves(mul2(f32_pair(w.x, w.y), f2));
      if (own && q.is_whole(k)) store_whole(out, q, k, a0, b0);
      else if (ends && own && k < q.hi) store_end(out, q, k, p.vocab, a0, b0);
    }
    return;
  }
  const f32x2 minus = f32_pair(-m, -m);
  for (int k = q.lo + tid; k < q.hi; k += kProbThreads) {
    uint2 w = load_quad(row, q, k, off, p.vocab);
    drop(w, floor);
    float2 v[2] = {powers(w.x, minus, a2), powers(w.y, minus, a2)};
    v[0].x = bf16lo_to_f32(w.x) == -INFINITY ? 0.f : v[0].x * inv;
    v[0].y = bf16hi_to_f32(w.x) == -INFINITY ? 0.f : v[0].y * inv;
    v[1].x = bf16lo_to_f32(w.y) == -INFINITY ? 0.f : v[1].x * inv;
    v[1].y = bf16hi_to_f32(w.y) == -INFINITY ? 0.f : v[1].y * inv;
    store_quad(out, q, k, p.vocab, v[0], v[1]);
  }
}

// ---------------------------------------------------------------------------
// sampled acceptance. Children of a node come from the drafter's distribution q
// at it. After k of them were refused, what is left of the target's p is
//
//   r_k = max(p - c_k q, 0) / S_k,  S_k = sum max(p - c_k q, 0),
//   c_0 = 0, S_0 = 1,  c_{k+1} = c_k + S_k
//
// (max(r_k - q, 0), normalised, is r_{k+1}), so that a refusal costs one pass
// over two rows, and nothing is written back. Child x with random number u is
// accepted where u q(x) < r_k(x); with none left, the token is drawn from r_k
// by the root's number. Children that were picked, not drawn (no q), have q = 1
// at themselves: a refused one's probability is taken out.
//
// Sums are 64-bit integers of probabilities in units of 2^-46: they do not depend
// on the order, and the token drawn is the one that 64-bit floats give, also where
// the number falls next to one of 248,320 borders (they differ in less than one
// draw of a million; 32-bit sums, off by 1e-7, in one of a hundred).
//
// A pass is one row of p, or one of p and one of q, over a cluster; its sums are
// exchanged once, and every CTA then walks by itself to the next row to sum. 32
// trees of 8 nodes over 248,320 tokens: 31 us. 18 are the tree's own loads (the
// offsets, then the nodes, then their probabilities: 5 us) and the first pass of all
// rows; the rest is further passes of rows with refusals, one after the other on the
// few SMs that a cluster is on. One draw each for 64 tokens over 128,000: 8.9 us, 3.7
// TB/s.
// ---------------------------------------------------------------------------
constexpr int kFrac = 56;
constexpr u64 kOne = 1ull << kFrac;
// Sums stop at 64, in whatever order they are taken, so that none wraps: rows of probabilities are far from it, and a row that
// gets there has no token and is reported. So is a c of 128 (64 nodes whose rows sum to 2 keep below 126).
constexpr u64 kMost = 64 * kOne;
__device__ __forceinline__ u64 add_up(u64 a, u64 b) { return min(a + b, kMost); }  // (of at most 2^63 and kMost)
// The sum of up to 16 such sums. The upper bits' sum is at least 16 (so the sum kMost), or the sum has not wrapped. (With
// add_up, one step waiting for the other's comparison, a chain of 6 took 7.82 us, so 7.66, without a limit 7.48.)
struct Total {
  u64 sum = 0;
  uint32_t upper = 0;
  __device__ __forceinline__ void add(u64 x) {
    sum += x;
    upper += (uint32_t)(x >> 58);
  }
  __device__ __forceinline__ u64 value() const { return upper >= 16 ? kMost : min(sum, kMost); }
};

struct SampleParams {
  const float *p, *q;  // q null: children that were picked
  long long p_row, q_row;
  const int64_t *draft, *mask;
  const int32_t *starts;
  const float *u;
  int rows, tokens, vocab, max_tree;
  int32_t *path, *count;
  int64_t *token;
  int *err;
};

enum { kDone = 0, kSum = 1, kDraw = 2, kTooMuch = 3 };

// What a CTA does next
struct Order {
  u64 c;
  int what, row, gone;  // row: of p and q; gone: children taken out
  float u;
  int ids[kMaxTree];
};

// A node of the draft tree: its children, and what decides on itself
struct Node {
  u64 kids;
  double px, qx;
  float u;
  int id;
};
static_assert(sizeof(Node) == 32, "four words of 64 bits");

struct SampleSmem {
  Node nodes[kMaxTree];
  u64 fits;  // nodes that are accepted if they are asked first
  int n, first;  // tokens of the row, the first of them
  Order order;
  u64 sums[2][kMaxCluster], warps[16], fine[16];
  int path[kMaxTree], accepted;
};

__device__ __forceinline__ float sound(float p) { return fminf(fmaxf(p, 0.f), 1.f); }  // (NaN: 0)

// Two probabilities, rounded to the nearest multiple of 2^-46, in two whole
// numbers each: added to 1 the upper 23 bits of x are the mantissa's, what that
// leaves of x is exact, and added to 1.5 * 2^-23 it has its mantissa in units of
// 2^-46. Their sums are sums of bit patterns, two 32-bit additions for a pair.
// (Conversions to 64-bit integers run on the double precision pipe: 32 rows of
// two times 248,320 took 85 us, three quarters of it that pipe's; moving the
// mantissa to its place with 64-bit shifts took 49.)
constexpr uint32_t kUpper = 0x3F800000u, kLower = 0x34400000u;  // 1, 1.5 * 2^-23
struct Bits {
  uint32_t hi_a, hi_b, lo_a, lo_b;
};
__device__ __forceinline__ Bits bits_of(float a, float b) {
  const f32x2 x = f32_pair(a, b), one = f32_pair(1.f, 1.f), minus = f32_pair(-1.f, -1.f);
  const f32x2 small = f32_pair(__uint_as_float(kLower), __uint_as_float(kLower));
  const f32x2 t = add2(x, one), low = add2(fma2(add2(t, minus), minus, x), small);
  const float2 h = f32_halves(t), l = f32_halves(low);
  return {__float_as_uint(h.x), __float_as_uint(h.y), __float_as_uint(l.x), __float_as_uint(l.y)};
}
constexpr int kBitsQuads = 32;  // 128 differences of below 2^23 each
constexpr int kUnits = kFrac - 46;  // sums are in units of 2^-56, as what c q cuts off is
__device__ __forceinline__ u64 join_bits(uint32_t hi, uint32_t lo) {
  return ((u64)hi << 23) + (u64)(int64_t)(int32_t)lo << kUnits;
}
__device__ __forceinline__ u64 fixed(float p) {
  const Bits x = bits_of(sound(p), 0.f);
  return join_bits(x.hi_a - kUpper, x.lo_a - kLower);
}

// max(p - c q, 0) of two elements, in units of 2^-46 (off by 0.2 of them in the mean, by 1.2 at most), added to sums of
// bit patterns. c is the sum of two floats (48 bits). p and c q are split at multiples of 2^-23; what is below them is put
// together with what the product rounds off, and its carry taken to the upper part. (As 64-bit products of whole numbers:
// 32 trees of 8, 248,320 probabilities each, 39.7 us against 34.2.)
struct Factor {
  f32x2 high, minus_high, minus_low;
  __device__ __forceinline__ explicit Factor(u64 c) {
    const float h = __ull2float_rn(c), l = __ll2float_rn((long long)(c - __float2ull_rz(h)));
    const float unit = 1.f / (float)kOne;
    high = f32_pair(h * unit, h * unit);
    minus_high = f32_pair(-h * unit, -h * unit);
    minus_low = f32_pair(-l * unit, -l * unit);
  }
};
__device__ __forceinline__ void add_cut(float p0, float p1, float q0, float q1, const Factor &c, uint32_t &hi, uint32_t &lo) {
  const f32x2 one = f32_pair(1.f, 1.f), minus = f32_pair(-1.f, -1.f);
  const f32x2 near = f32_pair(1.5f, 1.5f), minus_near = f32_pair(-1.5f, -1.5f);
  const f32x2 small = f32_pair(__uint_as_float(kLower), __uint_as_float(kLower));
  const f32x2 p = f32_pair(sound(p0), sound(p1)), q = f32_pair(sound(q0), sound(q1));
  const f32x2 m = mul2(q, c.minus_high), e = fma2(q, c.high, m);  // -(c q), and what it lacks
  const f32x2 p_hi = add2(add2(p, one), minus), m_hi = add2(add2(m, minus), one);
  f32x2 h = add2(p_hi, m_hi), l = add2(fma2(p_hi, minus, p), fma2(m_hi, minus, m));
  l = fma2(q, c.minus_low, fma2(e, minus, l));
  const f32x2 carry = add2(add2(l, near), minus_near);
  h = add2(h, carry);
  l = fma2(carry, minus, l);
  const float2 hf = f32_halves(h), lf = f32_halves(l), hw = f32_halves(add2(h, one)), lw = f32_halves(add2(l, small));
  if (hf.x > -lf.x) {
    hi += __float_as_uint(hw.x) - kUpper;
    lo += __float_as_uint(lw.x) - kLower;
  }
  if (hf.y > -lf.y) {
    hi += __float_as_uint(hw.y) - kUpper;
    lo += __float_as_uint(lw.y) - kLower;
  }
}

// max(p - c q, 0), as every sum has it; `factor` is c's
__device__ __forceinline__ u64 weight(float p, float q, u64 c, const Factor &factor) {
  if (c == 0) return fixed(p);
  if (c == kOne) {
    const u64 a = fixed(p), b = fixed(q);
    return a > b ? a - b : 0;
  }
  uint32_t hi = 0, lo = 0;
  add_cut(p, 0.f, q, 0.f, factor, hi, lo);
  return join_bits(hi, lo);
}

// Four values of a row, one by one; 0 past its ends.
__device__ __forceinline__ void load_ends(const float *row, const Quads &q, int k, int n, float (&x)[4]) {
  const int j = 4 * k - q.shift;
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = j + i >= 0 && j + i < n ? row[j + i] : 0.f;
}

// The walk, as far as it gets without another sum over the vocabulary. One thread
// of every CTA walks: they have the same nodes and get the same sums, so they
// need not wait for anybody's orders.
struct Walk {
  u64 c, total;  // of the node that it stands on; total: the sum that `order` asked for
  u64 kids;
  int node, asked, gone;
  bool known;  // total belongs to c

  __device__ void stand(int i, const SampleSmem &sm) {
    node = i;
    kids = sm.nodes[i].kids;
    c = 0;
    asked = gone = 0;
    known = false;
  }
  __device__ void go(SampleSmem &sm, bool drawn) {
    Order &o = sm.order;
    o.row = sm.first + node;
    while (kids) {
      if (asked && !known) {
        o.what = kSum;
        o.c = c;
        o.gone = 0;
        return;
      }
      const int i = __ffsll((long long)kids) - 1;
      kids &= kids - 1;
      const Node &kid = sm.nodes[i];
      bool fits = sm.fits >> i & 1;
      if (asked) {
        double r = kid.px;
        if (drawn) r -= (double)c * 0x1p-56 * kid.qx;
        for (int g = 0; g < gone; ++g)
          if (o.ids[g] == kid.id) r = 0;
        fits = (double)kid.u * kid.qx * ((double)total * 0x1p-56) < r;
      }
      if (fits) {
        sm.path[sm.accepted++] = i;
        stand(i, sm);
        o.row = sm.first + node;
        continue;
      }
      if (drawn) {
        c += asked ? total : kOne;
        if (c >= 2 * kMost) {
          o.what = kTooMuch;
          return;
        }
        known = false;
      } else {
        bool twin = false;
        for (int g = 0; g < gone; ++g) twin |= o.ids[g] == kid.id;
        if (!twin) {
          o.ids[gone++] = kid.id;
          if (known) total -= min(total, fixed((float)kid.px));
        }
      }
      ++asked;
    }
    o.what = kDraw;
    o.c = c;
    o.gone = gone;
  }
  // the sum that was asked for
  __device__ void learn(u64 sum, const SampleSmem &sm) {
    total = sum;
    for (int g = 0; g < gone; ++g) {
      // (taken out one by one; px of a removed id is that of the child that was refused)
      for (int i = 0; i < kMaxTree; ++i)
        if (sm.nodes[node].kids >> i & 1 && sm.nodes[i].id == sm.order.ids[g]) {
          total -= min(total, fixed((float)sm.nodes[i].px));
          break;
        }
    }
    known = true;
  }
};

// SINGLE: no row has a child (max_tree 1), so that every CTA knows what to do by
// itself and the cluster need not be told.
template <bool ALIGNED, bool SINGLE, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, WARPS == 16 ? 1 : 4) tree_sample_kernel(const SampleParams p) {
  static_assert(WARPS <= 16 && (WARPS & (WARPS - 1)) == 0 && WARPS * 32 >= kMaxTree, "parts of a row, nodes of a tree");
  __shared__ SampleSmem sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t S = cluster_nctarank(), rank = cluster_ctarank();
  const int b = cluster_id_x();
  cluster_arrive();
  grid_dependency_wait();
  grid_launch_dependents();
  const bool drawn = p.q != nullptr;
  const int parts_log2 = __ffs(S * WARPS) - 1;
  Walk walk;
  if (SINGLE) {
    if (tid == 0) {
      const int s0 = p.starts[b], s1 = p.starts[b + 1];
      const bool sound = s0 >= 0 && s1 >= s0 && s1 - s0 <= 1 && s1 <= p.tokens;
      if (!sound && rank == 0) atomicOr(p.err, kErrIndex);
      sm.accepted = sound ? s1 - s0 : 0;
      sm.path[0] = 0;
      sm.order.row = sm.accepted ? s0 : -1;
      sm.order.u = sm.accepted ? p.u[s0] : 0.f;
    }
  } else {
    // the first CTA reads the tree, and the others get it from there (whatever may be written to its arrays meanwhile,
    // all walk the same way)
    if (rank == 0) {
      const int s0 = p.starts[b], s1 = p.starts[b + 1];
      const bool sound_row = s0 >= 0 && s1 >= s0 && s1 - s0 <= p.max_tree && s1 <= p.tokens;
      const int n = sound_row ? s1 - s0 : 0;
      if (!sound_row && tid == 0) atomicOr(p.err, kErrIndex);
      if (tid < kMaxTree) sm.nodes[tid].kids = 0;
      if (tid == 0) {
        sm.fits = 0;
        sm.n = n;
        sm.first = s0;
      }
      __syncthreads();
      if (tid < n) {
        const u64 word = p.mask ? (u64)p.mask[s0 + tid] : ~0ull;
        const u64 above = word & ((1ull << tid) - 1);
        const int parent = above ? 63 - __clzll((long long)above) : -1;
        const float u = p.u[s0 + tid];
        sm.nodes[tid].u = u;
        if (parent >= 0) {
          const int64_t id = p.draft[s0 + tid];
          if (id >= 0 && id < p.vocab) {
            const double px = sound(p.p[(s0 + parent) * p.p_row + id]);
            const double qx = drawn ? sound(p.q[(s0 + parent) * p.q_row + id]) : 1.0;
            sm.nodes[tid].id = (int)id;
            sm.nodes[tid].px = px;
            sm.nodes[tid].qx = qx;
            atomicOr(&sm.nodes[parent].kids, 1ull << tid);
            if ((double)u * qx < px) atomicOr(&sm.fits, 1ull << tid);
          } else {
            atomicOr(p.err, kErrIndex);
          }
        }
      }
      __syncthreads();
    }
    cluster_wait();
    if (rank == 0) {
      const uint32_t words = sm.n * 4 + 2;  // the nodes, and what stands behind them: fits, n and first
      for (uint32_t i = tid; i < words * (S - 1); i += WARPS * 32) {
        const uint32_t to = 1 + i / words, w = i % words, at = w < 2 ? kMaxTree * 4 + w : w - 2;
        st_cluster_u64(mapa_shared(smem_u32(&sm) + 8 * at, to), reinterpret_cast<const u64 *>(&sm)[at]);
      }
    }
    cluster_sync_all();
    if (tid == 0) {
      sm.accepted = 0;
      sm.order.what = kDone;
      if (sm.n > 0) {
        sm.path[sm.accepted++] = 0;
        sm.order.u = sm.nodes[0].u;
        walk.stand(0, sm);
        walk.go(sm, drawn);
      }
    }
  }
  int64_t none = -1;
  for (int pass = 0;; pass ^= 1) {
    __syncthreads();
    const int what = SINGLE ? (int)kDraw : sm.order.what, row = sm.order.row, gone = SINGLE ? 0 : sm.order.gone;
    const u64 c = SINGLE ? 0 : sm.order.c;
    const float u = sm.order.u;
    if (what == kDone) break;
    if (what == kTooMuch) {
      if (rank == 0 && tid == 0) atomicOr(p.err, kErrIndex);
      break;
    }

    // this warp's part of the row
    const float *pr = p.p + row * p.p_row, *qr = p.q + row * p.q_row;
    const int shift = ALIGNED ? (int)(reinterpret_cast<uintptr_t>(pr) >> 2 & 3) : 0;
    Quads mine(p.vocab, shift, rank * WARPS + warp, parts_log2);
    if (SINGLE && row < 0) mine.hi = mine.whole_lo = mine.whole_hi = mine.lo;  // (no token: nothing to sum, and every barrier as ever)
    const Factor factor(c);
    u64 sum = 0;
    // the row's first and last quad, where they are not whole (not ALIGNED: all of them)
    auto alone = [&](int k) {
      float x[4], y[4] = {0.f, 0.f, 0.f, 0.f};
      load_ends(pr, mine, k, p.vocab, x);
      if (c) load_ends(qr, mine, k, p.vocab, y);
#pragma unroll
      for (int i = 0; i < 4; ++i) sum = add_up(sum, weight(x[i], y[i], c, factor));
    };
    if (!ALIGNED) {
      for (int k = mine.lo + lane; k < mine.hi; k += 32) alone(k);
    } else {
      if (lane < 2 && mine.end(lane) >= 0) alone(mine.end(lane));
      const float4 *p4 = reinterpret_cast<const float4 *>(pr - shift), *q4 = reinterpret_cast<const float4 *>(qr - shift);
      for (int k0 = mine.whole_lo + lane; k0 < mine.whole_hi; k0 += 32 * kBitsQuads) {  // (so long the bits' sums hold)
        uint32_t hi = 0, lo = 0;
        const int k1 = min(k0 + 32 * kBitsQuads, mine.whole_hi);
        constexpr int U = 4;  // quads on their way (past the part: zeros, which add nothing)
        const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
        auto two_rows = [&](auto add) {
          for (int k = k0; k < k1; k += 32 * U) {
            float4 x[U], y[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
              x[i] = y[i] = zero;
              if (k + 32 * i < k1) {
                x[i] = p4[k + 32 * i];
                y[i] = q4[k + 32 * i];
              }
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
              add(x[i].x, x[i].y, y[i].x, y[i].y);
              add(x[i].z, x[i].w, y[i].z, y[i].w);
            }
          }
        };
        if (c == 0) {
          for (int k = k0; k < k1; k += 32 * U) {
            float4 x[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
              x[i] = zero;
              if (k + 32 * i < k1) x[i] = p4[k + 32 * i];
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
              const Bits d = bits_of(sound(x[i].x), sound(x[i].y)), e = bits_of(sound(x[i].z), sound(x[i].w));
              hi += d.hi_a + d.hi_b + (e.hi_a + e.hi_b) - 4 * kUpper;
              lo += d.lo_a + d.lo_b + (e.lo_a + e.lo_b) - 4 * kLower;
            }
          }
        } else if (c == kOne) {  // max(p, q) - q
          two_rows([&](float x0, float x1, float y0, float y1) {
            const Bits d = bits_of(fminf(fmaxf(fmaxf(x0, y0), 0.f), 1.f), sound(y0));
            const Bits e = bits_of(fminf(fmaxf(fmaxf(x1, y1), 0.f), 1.f), sound(y1));
            hi += d.hi_a - d.hi_b + (e.hi_a - e.hi_b);
            lo += d.lo_a - d.lo_b + (e.lo_a - e.lo_b);
          });
        } else {
          two_rows([&](float x0, float x1, float y0, float y1) { add_cut(x0, x1, y0, y1, factor, hi, lo); });
        }
        sum = add_up(join_bits(hi, lo), sum);
      }
    }
    const uint32_t upper = __reduce_add_sync(kFull, (uint32_t)(sum >> 57));  // (as Total's, of 32)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    sum = upper >= 32 ? kMost : min(sum, kMost);
    if (gone && sum < kMost) {  // (else they are not all of it)
      u64 less = 0;
      for (int g = lane; g < gone; g += 32) {
        const int id = sm.order.ids[g], k = (id + shift) >> 2;
        if (k >= mine.lo && k < mine.hi) less += fixed(pr[id]);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) less += __shfl_xor_sync(kFull, less, o);
      sum -= less;
    }
    if (lane == 0) sm.warps[warp] = sum;
    __syncthreads();
    if (SINGLE) cluster_wait();
    if (tid < (int)S) {
      Total all;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) all.add(sm.warps[w]);
      st_cluster_u64(mapa_shared(smem_u32(&sm.sums[pass][rank]), tid), all.value());
    }
    cluster_sync_all();  // (the next pass's sums go elsewhere, so nobody waits for these to be read)
    Total whole;
    u64 before = 0;
    for (uint32_t i = 0; i < S; ++i) {
      if (i == rank) before = whole.sum;
      whole.add(sm.sums[pass][i]);
    }
    const u64 total = whole.value();
    if (total == kMost) {
      if (rank == 0 && tid == 0) atomicOr(p.err, kErrIndex);
      break;
    }
    if (what == kSum) {
      if (tid == 0) {
        walk.learn(total, sm);
        walk.go(sm, drawn);
      }
      continue;
    }
    if (total == 0) {  // nothing is left: p itself; nothing there either: no token
      if (c == 0 && gone == 0) break;
      if (tid == 0) {
        sm.order.c = 0;
        sm.order.gone = 0;
      }
      continue;
    }
    none = 0;
    // the first element at which the running sum passes u * total
    const u64 goal = __umul64hi(total, __float2ull_rz(fminf(fmaxf(u, 0.f), 0.99999994f) * 18446744073709551616.f));
    if (goal < before || goal - before >= sm.sums[pass][rank]) break;
    // in this CTA's slice: which warp's part of it, and all warps look through that
    u64 run = before;
    int part = 0;
    while (part < WARPS - 1 && goal - run >= sm.warps[part]) run += sm.warps[part++];
    const Quads theirs(p.vocab, shift, rank * WARPS + part, parts_log2);
    const int each = (theirs.hi - theirs.lo + WARPS - 1) / WARPS;
    const int lo = theirs.lo + warp * each, hi = min(lo + each, theirs.hi);
    auto weights = [&](int k, u64 (&v)[4]) {
      float x[4], y[4] = {0.f, 0.f, 0.f, 0.f};
      load_ends(pr, theirs, k, p.vocab, x);
      if (c) load_ends(qr, theirs, k, p.vocab, y);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = weight(x[i], y[i], c, factor);
        for (int g = 0; g < gone; ++g)
          if (sm.order.ids[g] == 4 * k - shift + i) v[i] = 0;
      }
    };
    u64 v[4];
    sum = 0;
    for (int k = lo + lane; k < hi; k += 32) {
      weights(k, v);
      sum += v[0] + v[1] + v[2] + v[3];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    if (lane == 0) sm.fine[warp] = sum;
    __syncthreads();
    for (int w = 0; w < warp; ++w) run += sm.fine[w];
    if (goal < run || goal - run >= sum) break;
    for (int k0 = lo; k0 < hi; k0 += 32) {  // (a part of 2,048 elements: once)
      const int k = k0 + lane;
      if (k >= hi) v[0] = v[1] = v[2] = v[3] = 0;
      if (k < hi && each > 32) weights(k, v);  // (else they are still there)
      const u64 four = v[0] + v[1] + v[2] + v[3];
      u64 upto = four;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 t = __shfl_up_sync(kFull, upto, o);
        if (lane >= o) upto += t;
      }
      const uint32_t past = __ballot_sync(kFull, run + upto > goal);
      if (past) {
        if (lane == __ffs(past) - 1) {
          u64 at = run + upto - four;
          int i = 0;
          while (i < 3 && at + v[i] <= goal) at += v[i++];
          p.token[b] = 4 * k - shift + i;
        }
        break;
      }
      run += __shfl_sync(kFull, upto, 31);
    }
    break;
  }
  if (rank == 0) {
    if (tid < p.max_tree) p.path[(long long)b * p.max_tree + tid] = tid < sm.accepted ? sm.path[tid] : -1;
    if (tid == 0) {
      p.count[b] = sm.accepted;
      if (none) p.token[b] = -1;
    }
  }
}

// `rows` clusters of up to `want` CTAs (a power of two up to 16; 8 where
// clusters of 16 do not fit)
template <class P>
cudaError_t launch_rows(void (*kern)(P), PerDevice &fits16, int rows, int want, int threads, int device,
                        cudaStream_t stream, const P &params) {
  if (want == kMaxCluster) {
    int f = fits16.v[device].load(std::memory_order_relaxed);
    if (f == 0) {
      f = -1;
      if (cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess) {
        cudaLaunchConfig_t lc = {};
        lc.gridDim = dim3(kMaxCluster, 1, 1);
        lc.blockDim = dim3(threads, 1, 1);
        cudaLaunchAttribute a;
        a.id = cudaLaunchAttributeClusterDimension;
        a.val.clusterDim.x = kMaxCluster;
        a.val.clusterDim.y = 1;
        a.val.clusterDim.z = 1;
        lc.attrs = &a;
        lc.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, kern, &lc) == cudaSuccess && n >= 1) f = 1;
      }
      (void)cudaGetLastError();
      fits16.v[device].store(f, std::memory_order_relaxed);
    }
    if (f < 0) want = 8;
  }
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)(rows * want), 1, 1);
  lc.blockDim = dim3(threads, 1, 1);
  lc.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = want;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = 2;
  return cudaLaunchKernelEx(&lc, kern, params);
}

// CTAs of a row: the fewest (a power of two) that leave each `most` elements at
// most; with few rows more of them, up to `fit` in all, while each keeps `least`
// (probabilities of 24 rows of 32,001 with at least 4,096 5.9 us, 2,048 6.9, 8,192
// 6.4; trees of 16 picked nodes over as many with 1,024 or 512 11.7, 2,048 12.4,
// 4,096 13.0).
int ctas_of(int rows, int vocab, int most, int least, int fit) {
  int s = 1;
  while (s < kMaxCluster && vocab > (long long)most * s) s *= 2;
  while (s < kMaxCluster && 2LL * rows * s <= fit && vocab >= 2LL * least * s) s *= 2;
  return s;
}

}  // namespace

cudaError_t launch_probabilities(const uint16_t *logits, long long row, const float *temperature, const float *floor,
                                 int tokens, int vocab, float *out, int device, int sm_count, cudaStream_t stream) {
  static PerDevice fits[2];
  // quads of logits and of probabilities are aligned together (columns of a wider head, 256 x 248,319 of 248,320, are not:
  // 92 us against 77; moved one by one they took 159)
  const bool aligned = ((reinterpret_cast<uintptr_t>(logits) >> 1) - (reinterpret_cast<uintptr_t>(out) >> 2)) % 4 == 0 && (row - vocab) % 4 == 0;
  const ProbParams p{logits, row, temperature, floor, out, vocab};
  const int s = ctas_of(tokens, vocab, kProbThreads * kProbQuads * 4, 4096, sm_count * 4);
  return launch_rows(aligned ? probabilities_kernel<true> : probabilities_kernel<false>, fits[aligned], tokens, s,
                     kProbThreads, device, stream, p);
}

cudaError_t launch_tree_sample(const SampleCall &c) {
  static PerDevice fits[2][2][2];
  // quads of p and of q are aligned together (else, element by element, 8 trees of 8 over 128,000 take 26 us, not 13)
  const bool aligned = !c.q || (((reinterpret_cast<uintptr_t>(c.p) - reinterpret_cast<uintptr_t>(c.q)) / 4) % 4 == 0 && (c.q_row - c.p_row) % 4 == 0);
  const SampleParams p{c.p, c.q, c.p_row, c.q_row, c.draft, c.mask, c.starts, c.u, c.rows, c.tokens, c.vocab, c.max_tree,
                       c.path, c.count, c.token, c.err};
  // 16 warps a CTA while every CTA has an SM to itself (a chain of six 7.5 us against 9.9 with 8, sums without a limit), 8 where that makes more
  // of them (32 trees of eight 31 us against 34)
  const int s = ctas_of(c.rows, c.vocab, 32768, 1024, c.sm_count * 2);
  const bool few = (long long)c.rows * s * 2 <= c.sm_count * 2, one = c.max_tree == 1;
  void (*kern)(SampleParams);
  if (one) kern = few ? aligned ? tree_sample_kernel<true, true, 16> : tree_sample_kernel<false, true, 16>
                      : aligned ? tree_sample_kernel<true, true, 8> : tree_sample_kernel<false, true, 8>;
  else kern = few ? aligned ? tree_sample_kernel<true, false, 16> : tree_sample_kernel<false, false, 16>
                  : aligned ? tree_sample_kernel<true, false, 8> : tree_sample_kernel<false, false, 8>;
  return launch_rows(kern, fits[one][few][aligned], c.rows, few ? s : ctas_of(c.rows, c.vocab, 32768, 1024, c.sm_count * 4),
                     few ? 512 : 256, c.device, c.stream, p);
}

}  // namespace w4a16
