// Low-rank adapters of many requests beside a shared product:
//
//   out[t] = y[t] + scale_e (x[t] A_e^T) B_e^T,   e the adapter of token t's row
//
// Two launches. `shrink` makes t = x A^T, the sum over K split over CTAs;
// `expand` applies the scale and adds t B^T to y. Tokens are taken together by
// adapter, whichever rows they belong to, so that an adapter is read once for all
// tokens of a tile. Which tokens those are every CTA works out for itself from
// the rows' adapters: a count for each adapter, whose running sums number the
// tiles.
//
// 16 ranks against every element are 8 to 32 FLOP a byte, a twentieth of the
// machine's balance: the work is to move x, y and the adapters, and where tokens
// are few, to begin early (expand has its part of B and y on their way before
// shrink is done).
//
// - Few tokens: tiles of 16, products on mma.sync (m16n8k16), whose fragments
//   come straight from memory or a warp's own copies; the parts of the sums over K
//   go to the workspace as float32 and expand adds them up. The k order of a
//   fragment is free as long as both operands agree, so a lane's 16 bytes of
//   consecutive k serve two products as they come. One token of rank 16, 5,120
//   by 5,120: 5.2 us; 48 tokens of 12 adapters of rank 64, 5,120 by 34,816: 23.2
//   us, 3.0 TB/s.
// - Prompts: tiles of 128, products on tcgen05, sums in TMEM; a cluster adds up
//   the parts over K in distributed shared memory. 4,096 tokens of rank 16, 5,120
//   by 34,816: 121 us, 5.1 TB/s; six prompts of 2,000 and rank 64, 5,120 by 7,168:
//   75 us, 4.0 TB/s.
#include "w4a16_internal.h"

namespace w4a16 {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kColumns = kWarps * 32;  // of a unit of expand

struct LoraParams {
  const uint16_t *y, *x, *a, *b;
  int y_row, x_row;  // elements (32 bits: a token's offset is one wide multiplication)
  long long a_adapter, a_row, b_adapter, b_row;
  int out_row;
  const float *scale;
  const int32_t *adapter, *starts;
  int rows, tokens, adapters, rank, inner, outer, ksplit;
  uint16_t *out;
  float *parts;  // few tokens: x A^T in parts, [ksplit][tokens][RP]
  // prompts: x A^T in its bf16 parts, [tokens][parts][RP]; how many tiles there are (with an adapter, in all); the tiles
  uint16_t *low;
  int *head, *lists;
  int *err;
  bool in_place, alike;  // alike: rows of y and of out begin equally far after 16-byte boundaries
};

__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Exclusive sum over the block of one value per thread, and the total (all
// threads call it; `sums` is free again after the next barrier).
__device__ __forceinline__ int block_scan(int v, int *sums, int &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(kFull, inc, o);
    if (lane >= o) inc += t;
  }
  if (lane == 31) sums[warp] = inc;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w == warp) before = total;
    total += sums[w];
  }
  return before + inc - v;
}

// First token and number of tokens of row b; none, and `bad`, where the offsets cannot be.
__device__ __forceinline__ int row_tokens(const LoraParams &p, int b, int &first, bool &bad) {
  if (!p.starts) {
    first = b;
    return 1;
  }
  first = p.starts[b];
  const int end = p.starts[b + 1];
  if (first < 0 || end < first || end > p.tokens) {
    atomicOr(p.err, kErrIndex);
    bad = true;
    return 0;
  }
  return end - first;
}

// Row b's adapter; p.adapters where it has none.
__device__ __forceinline__ int row_adapter(const LoraParams &p, int b) {
  const int e = p.adapter[b];
  if ((unsigned)e < (unsigned)p.adapters) return e;
  if (e != -1) atomicOr(p.err, kErrIndex);
  return p.adapters;
}

// Offsets that descend: the tokens of row b that lie behind the ends of all rows before it, `end` the largest end before the
// block's rows: first one, how many, and the largest end so far. (All threads call it, in the rows' order.) Whatever the
// offsets, no token is counted twice so, and there are no more tiles than of ascending ones.
__device__ int4 tokens_behind(const LoraParams &p, int b, int end, int *sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int first = 0;
  bool known;
  int n = b < p.rows ? row_tokens(p, b, first, known) : 0;
  const int mine = n ? first + n : 0;
  int upto = mine;
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(kFull, upto, o);
    if (lane >= o) upto = max(upto, t);
  }
  __syncthreads();
  if (lane == 31) sums[warp] = upto;
  const int left = __shfl_up_sync(kFull, upto, 1);
  int before = lane ? max(end, left) : end;
  __syncthreads();
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before = max(before, sums[w]);
    end = max(end, sums[w]);
  }
  __syncthreads();
  if (n && first < before) {
    n = max(mine - before, 0);
    first = before;
  }
  return make_int4(first, n, end, 0);
}

// The adapters' counts of tokens, and the tokens of row threadIdx.x, where offsets descend; order[1] gets the largest end of
// the block's first rows. (Out of line, as the next: in line they cost registers, up to 2 us of 24.)
__device__ __noinline__ int2 count_again(const LoraParams &p, int *count, int *sums, int *order) {
  for (int e = threadIdx.x; e <= p.adapters; e += kThreads) count[e] = 0;
  int2 mine = make_int2(0, 0);
  int end = 0;
  for (int b0 = 0; b0 < p.rows; b0 += kThreads) {
    const int4 row = tokens_behind(p, b0 + threadIdx.x, end, sums);
    end = row.z;
    if (row.y) atomicAdd(&count[row_adapter(p, b0 + threadIdx.x)], row.y);
    if (b0 == 0) {
      mine = make_int2(row.x, row.y);
      if (threadIdx.x == 0) order[1] = end;
    }
  }
  __syncthreads();
  return mine;
}

// As Tiles::tokens, for the rows from kThreads on; `done` of the adapter's tokens are in rows before those
__device__ __noinline__ void tokens_of_more_rows(const LoraParams &p, int e, int lo, int hi, int *list, int done, int *sums,
                                                 const int *order) {
  const bool descend = order[0];
  int end = descend ? order[1] : 0;
  bool known;
  for (int b0 = kThreads; b0 < p.rows && done < hi; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    int s = 0, n = 0, total;
    if (descend) {
      const int4 row = tokens_behind(p, b, end, sums);
      s = row.x;
      n = row.y && row_adapter(p, b) == e ? row.y : 0;
      end = row.z;
    } else if (b < p.rows && row_adapter(p, b) == e) {
      n = row_tokens(p, b, s, known);
    }
    __syncthreads();
    const int at = done + block_scan(n, sums, total);
    for (int i = max(lo, at); i < min(hi, at + n); ++i) list[i - lo] = s + i - at;
    done += total;
  }
}

// The tiles of a call, T tokens of one adapter each: count[e] tokens of adapter
// e (the last bin: of none), tiles first[e] .. first[e + 1].
struct Tiles {
  int *count, *first, *sums;
  int *order;  // whether some row's offsets cannot be (the others may descend then), and the largest end of the block's first rows
  int bins;
  int mine, mine_at, mine_n;  // adapter, first token and number of tokens of row threadIdx.x (the block's first pass over the rows)

  static __host__ __device__ int ints(int adapters) { return 2 * adapters + 5 + kWarps; }
  __device__ Tiles(int *mem, int adapters)
      : count(mem), first(mem + adapters + 1), sums(mem + 2 * adapters + 3), order(mem + 2 * adapters + 3 + kWarps), bins(adapters + 1) {}

  template <int T>
  __device__ void make(const LoraParams &p) {
    mine = -1;
    mine_at = mine_n = 0;
    bool bad = false;
    if (threadIdx.x == 0) order[0] = 0;
    if ((int)threadIdx.x < p.rows) {
      mine = row_adapter(p, threadIdx.x);
      mine_n = row_tokens(p, threadIdx.x, mine_at, bad);
    }
    for (int e = threadIdx.x; e < bins; e += kThreads) count[e] = 0;
    __syncthreads();
    if (mine_n) atomicAdd(&count[mine], mine_n);
    for (int b = kThreads + threadIdx.x; b < p.rows; b += kThreads) {
      int s;
      const int n = row_tokens(p, b, s, bad);
      if (n) atomicAdd(&count[row_adapter(p, b)], n);
    }
    if (bad) order[0] = 1;
    __syncthreads();
    if (order[0]) {
      const int2 row = count_again(p, count, sums, order);
      mine_at = row.x;
      mine_n = row.y;
    }
    const int each = (bins + kThreads - 1) / kThreads, e0 = threadIdx.x * each, e1 = min(e0 + each, bins);
    int n = 0, total;
    for (int e = e0; e < e1; ++e) n += (count[e] + T - 1) / T;
    n = block_scan(n, sums, total);
    for (int e = e0; e < e1; ++e) {
      first[e] = n;
      n += (count[e] + T - 1) / T;
    }
    if (threadIdx.x == 0) first[bins] = total;
    __syncthreads();
  }

  // the adapter of tile w
  __device__ int of(int w) const {
    int lo = 0, hi = bins - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (first[mid] <= w) lo = mid;
      else hi = mid - 1;
    }
    return lo;
  }

  // Tokens lo .. hi of adapter e, in the rows' order, into list (all threads)
  __device__ void tokens(const LoraParams &p, int e, int lo, int hi, int *list) const {
    int total;
    const int n = mine == e ? mine_n : 0, at = block_scan(n, sums, total);
    for (int i = max(lo, at); i < min(hi, at + n); ++i) list[i - lo] = mine_at + i - at;
    if (total < hi && p.rows > kThreads) tokens_of_more_rows(p, e, lo, hi, list, total, sums, order);
    __syncthreads();
  }
};

// ---------------------------------------------------------------------------
// shrink: a unit is one tile and one part of K. A warp has all of the tile's
// tokens and up to 64 ranks, and every eighth (RP = 128: fourth) 32 of the
// part's k, straight from memory; the warps' sums meet in shared memory.
// ---------------------------------------------------------------------------
template <int RP>
struct ShrinkGeo {
  static constexpr int NB = (RP < 64 ? RP : 64) / 8;  // blocks of 8 ranks of a warp
  static constexpr int KW = RP > 64 ? kWarps / 2 : kWarps;  // warps that share K
  static constexpr int STRIDE = NB * 8 + 8;        // floats of a token's sums
  static constexpr int SUMS = kWarps * 16 * STRIDE * 4;
  static constexpr int OFF_LIST = SUMS, OFF_TILES = OFF_LIST + 16 * 4;
  static int smem(int adapters) { return OFF_TILES + Tiles::ints(adapters) * 4; }
};

template <int RP>
__global__ void __launch_bounds__(kThreads, 2) lora_shrink_kernel(const __grid_constant__ LoraParams p) {
  using G = ShrinkGeo<RP>;
  extern __shared__ __align__(16) uint8_t smem[];
  float *sums = reinterpret_cast<float *>(smem);
  int *list = reinterpret_cast<int *>(smem + G::OFF_LIST);
  Tiles tiles(reinterpret_cast<int *>(smem + G::OFF_TILES), p.adapters);
  grid_dependency_wait();
  grid_launch_dependents();  // (so all that came before is complete when expand begins)
  tiles.make<16>(p);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int kw = warp % G::KW, rank0 = warp / G::KW * 64;
  const int steps = (p.inner + 31) / 32;
  const long long units = (long long)tiles.first[p.adapters] * p.ksplit;
  for (long long unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int tile = (int)(unit / p.ksplit), part = (int)(unit % p.ksplit);
    const int e = tiles.of(tile), lo = (tile - tiles.first[e]) * 16, n = min(16, tiles.count[e] - lo);
    tiles.tokens(p, e, lo, lo + n, list);
    const uint16_t *xr[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) xr[h] = h * 8 + g < n ? p.x + (long long)list[h * 8 + g] * p.x_row : nullptr;
    const uint16_t *ar = p.a + e * p.a_adapter + (rank0 + g) * p.a_row;
    float acc[G::NB][4] = {};
    const int s1 = (int)((long long)steps * (part + 1) / p.ksplit);
#pragma unroll 2
    for (int s = (int)((long long)steps * part / p.ksplit) + kw; s < s1; s += G::KW) {
      const int k = s * 32 + t * 8;
      const bool in = k < p.inner;
      const uint4 zero = make_uint4(0, 0, 0, 0);
      uint4 xv[2], av[G::NB];
#pragma unroll
      for (int j = 0; j < G::NB; ++j)
        av[j] = in && rank0 + j * 8 + g < p.rank ? __ldg(reinterpret_cast<const uint4 *>(ar + j * 8 * p.a_row + k)) : zero;
#pragma unroll
      for (int h = 0; h < 2; ++h) xv[h] = in && xr[h] ? *reinterpret_cast<const uint4 *>(xr[h] + k) : zero;
#pragma unroll
      for (int j = 0; j < G::NB; ++j) {
        mma16(acc[j], xv[0].x, xv[1].x, xv[0].y, xv[1].y, av[j].x, av[j].y);
        mma16(acc[j], xv[0].z, xv[1].z, xv[0].w, xv[1].w, av[j].z, av[j].w);
      }
    }
#pragma unroll
    for (int j = 0; j < G::NB; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<float2 *>(sums + (warp * 16 + h * 8 + g) * G::STRIDE + j * 8 + 2 * t) =
            make_float2(acc[j][2 * h], acc[j][2 * h + 1]);
    __syncthreads();
    float *out = p.parts + (long long)part * p.tokens * RP;
    for (int i = threadIdx.x; i < n * RP / 4; i += kThreads) {
      const int row = i * 4 / RP, r = i * 4 % RP;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < G::KW; ++w) {
        const float4 u = *reinterpret_cast<const float4 *>(sums + ((r / 64 * G::KW + w) * 16 + row) * G::STRIDE + r % 64);
        v.x += u.x;
        v.y += u.y;
        v.z += u.z;
        v.w += u.w;
      }
      *reinterpret_cast<float4 *>(out + (long long)list[row] * RP + r) = v;
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// expand: a unit is one tile and 256 columns; a warp has 32 of them, for all of
// the tile's tokens. t goes into the product whole, as three bf16 parts (with two,
// 16 bits of mantissa, one output in a thousand is the neighbour of what float32
// gives, with three one in four thousand, by the order of sums; 48 tokens of 12
// adapters of rank 16 11.9 | 12.3 us, of 64 22.8 | 23.2, of 128 32.2 | 35.0). The rows
// of B that a product's eight columns stand for are chosen such that a lane ends up
// with eight consecutive columns of a token: y is read and written 16 bytes at a time.
// B is what there is to read: every warp copies its own columns to shared memory some
// units ahead, and begins before there is a t. Small slots hide more of the latency as
// many of them than as more CTAs, large ones the other way: rank 64 with three CTAs of
// two slots an SM 23.5 us, two of three 24.9 (and, with t in two parts, one of four 24.4
// where three of two took 21.1, B straight to registers 23.8, B brought to L2 by shrink
// 26.7).
// ---------------------------------------------------------------------------
template <int RP>
struct ExpandGeo {
  static constexpr int KS = RP < 32 ? 1 : RP / 32;  // 16-byte pieces of k of a lane
  static constexpr int ROW = RP < 32 ? RP * 2 : RP == 32 ? 64 : RP * 2 + 64;  // bytes of a token's t, without bank conflicts
  static constexpr int CPR = RP / 8;                // 16-byte pieces of a row of B
  static constexpr int SLOT = 32 * RP * 2, SLOTS = RP <= 16 ? 8 : RP == 32 ? 3 : 2;
  // CTAs per SM. Rank 64 with rows off 16 bytes does not fit a third of the registers (48 tokens of 12 adapters, 34,813 columns
  // with 3 25.8 us, 2 25.0; 69 of 6, 5,121 columns 16.1 | 14.9)
  static constexpr int ctas(bool even) { return RP <= 16 ? 2 : RP < 64 || (RP == 64 && even) ? 3 : RP == 64 ? 2 : 1; }
  static constexpr int PART = 16 * ROW, OFF_RING = 3 * PART, OFF_LIST = OFF_RING + kWarps * SLOTS * SLOT;
  static constexpr int OFF_TILES = OFF_LIST + 16 * 4;
  static int smem(int adapters) { return OFF_TILES + Tiles::ints(adapters) * 4; }
  // where piece c of row r is: every other row's halves change places, so that a fragment's rows meet different banks
  static __device__ __forceinline__ int place(int r, int c) { return r * RP * 2 + ((RP >= 64 ? c ^ ((r & 1) << 2) : c) << 4); }
};

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A lane's piece of k: 8 consecutive values (RP >= 32), 4 (16) or 2 (8).
template <int RP>
__device__ __forceinline__ uint4 piece(const uint8_t *at) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (RP >= 32) v = *reinterpret_cast<const uint4 *>(at);
  else if (RP == 16) *reinterpret_cast<uint2 *>(&v) = *reinterpret_cast<const uint2 *>(at);
  else v.x = *reinterpret_cast<const uint32_t *>(at);
  return v;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&b);
}
// The upper 16 bits of a value, as a bf16 value: cut, not rounded, and one step less where nothing would be left below. So
// what is left is not 0 and has the same sign, and an infinite weight times the parts of a value is infinite, not inf - inf or
// 0 inf (of values from 2^-95 on, whose last part is no smaller than 2^-126). Of infinity it is the largest bf16 value, and
// infinity is left.
__device__ __forceinline__ uint32_t upper_bits(float a) { return __float_as_uint(a) - (a != 0.f ? 1 : 0) & 0xFFFF0000u; }
// Two values as bf16 parts each: three, whose sum is the value, or two, off by 2^-16 of it at most
__device__ __forceinline__ void in_parts(float a, float b, uint32_t (&part)[3]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t x = upper_bits(a), y = upper_bits(b);
    part[i] = __byte_perm(x, y, 0x7632);
    a -= __uint_as_float(x);
    b -= __uint_as_float(y);
  }
  part[2] = pack_bf16(a, b);
}
__device__ __forceinline__ void in_parts(float a, float b, uint32_t (&part)[2]) {
  const uint32_t x = upper_bits(a), y = upper_bits(b);
  part[0] = __byte_perm(x, y, 0x7632);
  part[1] = pack_bf16(a - __uint_as_float(x), b - __uint_as_float(y));
}

// Eight columns of a row from column c on, `wide`: as one 16-byte access
__device__ __forceinline__ uint4 load8(const uint16_t *row, int c, int n, bool wide) {
  if (wide) return __ldcg(reinterpret_cast<const uint4 *>(row + c));
  uint32_t v[4] = {};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c + i < n) v[i / 2] |= (uint32_t)__ldcg(row + c + i) << (i % 2 * 16);
  return make_uint4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store8(uint16_t *row, int c, int n, bool wide, const uint4 &x) {
  if (wide) {
    *reinterpret_cast<uint4 *>(row + c) = x;
    return;
  }
  const uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c + i < n) row[c + i] = (uint16_t)(v[i / 2] >> (i % 2 * 16));
}

// Rows that do not begin on 16 bytes are moved in whole pieces too (one by one: 48 tokens of rank 64, 34,813 columns
// 22.9 us against 18.9, 512 of rank 16 113 against 41). Eight elements from the e-th of two pieces on:
__device__ __forceinline__ uint4 from_pieces(const uint4 &a, const uint4 &b, int e) {
  uint32_t w[7] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z};
  if (e & 4) {
    w[0] = w[2], w[1] = w[3], w[2] = w[4], w[3] = w[5], w[4] = w[6];
    w[5] = b.w;
  }
  if (e & 2) w[0] = w[1], w[1] = w[2], w[2] = w[3], w[3] = w[4], w[4] = w[5];
  const int bits = 16 * (e & 1);
  return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits), __funnelshift_r(w[2], w[3], bits),
                    __funnelshift_r(w[3], w[4], bits));
}
__device__ __forceinline__ uint4 load_across(const uint16_t *at) {
  const int e = (int)(reinterpret_cast<uintptr_t>(at) >> 1 & 7);
  const uint4 *from = reinterpret_cast<const uint4 *>(at - e);
  const uint4 a = __ldcg(from), b = __ldcg(from + (e ? 1 : 0));  // (both hold some of the eight)
  return from_pieces(a, b, e);
}
// Four lanes' 32 elements, eight each, to `at` on: whole pieces from two lanes each, what is before and behind them in
// halves of pieces, quarters and ones. All lanes call it, `there`: with something to store.
__device__ __forceinline__ void store_across(uint16_t *at, int t, uint4 v, bool there) {
  const uint4 next = make_uint4(__shfl_down_sync(kFull, v.x, 1), __shfl_down_sync(kFull, v.y, 1), __shfl_down_sync(kFull, v.z, 1),
                                __shfl_down_sync(kFull, v.w, 1));
  if (!there) return;
  const int e = (int)(0 - (reinterpret_cast<uintptr_t>(at) >> 1) & 7);  // elements before the first whole piece
  const uint4 w = from_pieces(v, next, e);
  if (t < 3 || e == 0) *reinterpret_cast<uint4 *>(at + e) = w;
  if (t == 0) {
    if (e & 1) {
      *at++ = (uint16_t)v.x;
      v = make_uint4(__funnelshift_r(v.x, v.y, 16), __funnelshift_r(v.y, v.z, 16), __funnelshift_r(v.z, v.w, 16), 0);
    }
    if (e & 2) {
      *reinterpret_cast<uint32_t *>(at) = v.x;
      at += 2;
      v.x = v.y;
      v.y = v.z;
    }
    if (e & 4) *reinterpret_cast<uint2 *>(at) = make_uint2(v.x, v.y);
  } else if (t == 3 && e) {
    at += e;
    const int n = 8 - e;
    uint32_t x = w.x, y = w.y;
    if (n & 4) {
      *reinterpret_cast<uint2 *>(at) = make_uint2(x, y);
      at += 4;
      x = w.z;
      y = w.w;
    }
    if (n & 2) {
      *reinterpret_cast<uint32_t *>(at) = x;
      at += 2;
      x = y;
    }
    if (n & 1) *at = (uint16_t)x;
  }
}

template <int RP, bool EVEN>
__global__ void __launch_bounds__(kThreads, ExpandGeo<RP>::ctas(EVEN)) lora_expand_kernel(const __grid_constant__ LoraParams p) {
  using G = ExpandGeo<RP>;
  extern __shared__ __align__(16) uint8_t smem[];
  int *list = reinterpret_cast<int *>(smem + G::OFF_LIST);
  Tiles tiles(reinterpret_cast<int *>(smem + G::OFF_TILES), p.adapters);
  // What shrink waited for before it let this launch begin is complete: rows,
  // adapters, y and B may be read; t only after the wait below.
  tiles.make<16>(p);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int chunks = (p.outer + kColumns - 1) / kColumns, all = tiles.first[p.in_place ? p.adapters : p.adapters + 1];
  // CTAs that share a tile's chunks, and tiles that are worked on at once: with
  // a tile of its own a CTA makes one t (48 tokens of 12 adapters and 34,816
  // columns: five or six chunks a CTA)
  const int sharing = max(1, (int)gridDim.x / max(all, 1)), at_once = (int)gridDim.x / sharing;
  const int share = (int)blockIdx.x % sharing;
  const int c_lo = (int)((long long)chunks * share / sharing), c_hi = (int)((long long)chunks * (share + 1) / sharing);
  int tile = (int)blockIdx.x / sharing;
  if (tile >= at_once || c_lo >= c_hi) tile = all;

  // the warp's columns of B, SLOTS - 1 units ahead; a lane copies one piece of every (32 / CPR)th row
  constexpr int kEach = 32 / G::CPR;
  const uint32_t ring = smem_u32(smem) + G::OFF_RING + warp * G::SLOTS * G::SLOT;
  const uint32_t lane_to = G::place(lane / G::CPR, lane % G::CPR);
  const uint16_t *lane_b = p.b + (warp * 32 + lane / G::CPR) * p.b_row + lane % G::CPR * 8;
  const bool lane_in = lane % G::CPR * 8 < p.rank, dense = p.rank == RP && p.b_row == RP;
  int next_tile = tile, next_chunk = c_lo, next_slot = 0;
  const uint16_t *next_b = nullptr;  // null: of no adapter
  auto fetch = [&]() {
    if (next_tile < all) {
      if (next_chunk == c_lo) {
        const int e = tiles.of(next_tile);
        next_b = e < p.adapters ? lane_b + e * p.b_adapter + (long long)c_lo * kColumns * p.b_row : nullptr;
      }
      if (next_b) {
        const uint32_t to = ring + next_slot * G::SLOT + lane_to;
        const int rows = p.outer - next_chunk * kColumns - warp * 32;  // from the warp's first row to the last
        if (dense && rows >= 32) {  // (addresses a constant apart)
#pragma unroll
          for (int i = 0; i < G::CPR; ++i) copy16(to + i * kEach * RP * 2, next_b + i * kEach * RP);
        } else {
#pragma unroll
          for (int i = 0; i < G::CPR; ++i) {
            const bool in = lane_in && i * kEach + lane / G::CPR < rows;
            copy16(to + i * kEach * RP * 2, in ? next_b + i * kEach * p.b_row : p.b, in);
          }
        }
        next_b += kColumns * p.b_row;
      }
      if (++next_chunk == c_hi) {
        next_chunk = c_lo;
        next_tile += at_once;
      }
      next_slot = next_slot + 1 == G::SLOTS ? 0 : next_slot + 1;
    }
    copy_commit();
  };
  static_assert(RP < 64 || kEach % 2 == 0, "a lane's rows are all even or all odd: their pieces have one place");
#pragma unroll
  for (int i = 0; i < G::SLOTS - 1; ++i) fetch();

  int slot = 0;
  bool waited = false;
  for (; tile < all; tile += at_once) {
    __syncthreads();  // (the tile before is done with)
    const int e = tiles.of(tile), lo = (tile - tiles.first[e]) * 16, n = min(16, tiles.count[e] - lo);
    tiles.tokens(p, e, lo, lo + n, list);
    const uint16_t *yr[2];
    uint16_t *to[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int token = h * 8 + g < n ? list[h * 8 + g] : 0;
      yr[h] = p.y + (long long)token * p.y_row;
      to[h] = p.out + (long long)token * p.out_row;
    }
    uint4 yv[2];
    auto fetch_y = [&](int chunk) {
      const int c = chunk * kColumns + warp * 32 + 8 * t;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (h * 8 + g < n) {
          if (!EVEN && c + 8 <= p.outer) yv[h] = load_across(yr[h] + c);
          else yv[h] = load8(yr[h], c, p.outer, EVEN && c + 8 <= p.outer);
        }
    };
    fetch_y(c_lo);
    if (!waited) {
      grid_dependency_wait();
      waited = true;
    }
    if (e < p.adapters) {
      const float scale = p.scale ? p.scale[e] : 1.f;
      for (int i = threadIdx.x; i < n * RP / 2; i += kThreads) {
        const int row = i * 2 / RP, r = i * 2 % RP;
        const float *from = p.parts + (long long)list[row] * RP + r;
        float2 v = make_float2(0.f, 0.f);
#pragma unroll 8
        for (int s = 0; s < p.ksplit; ++s) {
          const float2 u = __ldcg(reinterpret_cast<const float2 *>(from + (long long)s * p.tokens * RP));
          v.x += u.x;
          v.y += u.y;
        }
        v = r < p.rank ? make_float2(v.x * scale, v.y * scale) : make_float2(0.f, 0.f);  // (infinity times the padding's zeros is not a number)
        uint32_t part[3];
        in_parts(v.x, v.y, part);
#pragma unroll
        for (int k = 0; k < 3; ++k) *reinterpret_cast<uint32_t *>(smem + k * G::PART + row * G::ROW + r * 2) = part[k];
      }
      __syncthreads();
    }
    for (int chunk = c_lo; chunk < c_hi; ++chunk) {
      const int c = chunk * kColumns + warp * 32 + 8 * t;
      fetch();
      copy_wait<G::SLOTS - 1>();
      __syncwarp();
      if (e < p.adapters) {
        float acc[4][4] = {};
#pragma unroll
        for (int s = 0; s < G::KS; ++s) {
          uint4 bv[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int r = 8 * (g >> 1) + 2 * j + (g & 1);
            const uint8_t *from = smem + G::OFF_RING + (warp * G::SLOTS + slot) * G::SLOT;
            bv[j] = piece<RP>(from + (RP < 32 ? r * RP * 2 + t * (RP / 2) : G::place(r, s * 4 + t)));
          }
          const int at = g * G::ROW + (RP < 32 ? t * (RP / 2) : s * 64 + t * 16);
#pragma unroll
          for (int part = 0; part < 3; ++part) {
            const uint8_t *from = smem + part * G::PART + at;
            const uint4 a0 = piece<RP>(from), a1 = piece<RP>(from + 8 * G::ROW);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              mma16(acc[j], a0.x, a1.x, a0.y, a1.y, bv[j].x, bv[j].y);
              if (RP >= 32) mma16(acc[j], a0.z, a1.z, a0.w, a1.w, bv[j].z, bv[j].w);
            }
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t *v = &yv[h].x;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            v[j] = pack_bf16(bf16lo_to_f32(v[j]) + acc[j][2 * h], bf16hi_to_f32(v[j]) + acc[j][2 * h + 1]);
        }
      }
      if (!EVEN && chunk * kColumns + warp * 32 + 32 <= p.outer) {
#pragma unroll
        for (int h = 0; h < 2; ++h) store_across(to[h] + c, t, yv[h], h * 8 + g < n);
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (h * 8 + g < n) store8(to[h], c, p.outer, EVEN && c + 8 <= p.outer, yv[h]);
      }
      __syncwarp();  // (the slot is free)
      slot = slot + 1 == G::SLOTS ? 0 : slot + 1;
      if (chunk + 1 < c_hi) fetch_y(chunk + 1);
    }
  }
  copy_wait<0>();
  if (!waited) grid_dependency_wait();
  grid_launch_dependents();
}

// ---------------------------------------------------------------------------
// Prompts. shrink: a cluster of CTAs has up to 128 tokens of one adapter, each
// CTA a part of K, which it streams through shared memory 64 k at a time into
// tcgen05 products (128 tokens by RP ranks, sums in TMEM): the warps only copy.
// (With mma.sync, whose fragments come from shared memory, six prompts of rank 64
// took 33 us here.) The parts of the sums meet over distributed shared memory, and
// x A^T is written once, in its bf16 parts: three up to rank 32, two above, where the products of the third would show (4,096
// tokens, 34,816 columns, two | three parts: rank 16 117.2 | 118.1 us, 32 119.8 | 122.9, 64 126.8 | 136.1, 128 203 | 231; six
// prompts of rank 64 74 | 80).
// ---------------------------------------------------------------------------
__host__ __device__ constexpr int parts_of_rank(int padded) { return padded <= 32 ? 3 : 2; }
constexpr int kTile = 64;       // tokens of a list
constexpr int kListInts = 68;   // a tile's tokens, adapter and number of tokens

template <int RP>
struct PromptShrinkGeo {
  static constexpr int X = 128 * 128, STAGE = X + RP * 128;  // bytes: rows of 64 k, swizzled
  static constexpr int STAGES = RP <= 32 ? 5 : RP == 64 ? 4 : 3;
  static constexpr int COLS = RP < 32 ? 32 : RP;  // of TMEM
  static constexpr int PITCH = RP + 4;            // floats of a token's sums (they take the stages' place)
  static constexpr int OFF_LIST = STAGES * STAGE, OFF_BAR = OFF_LIST + 128 * 4, OFF_TILES = OFF_BAR + STAGES * 8 + 16;
  static_assert(128 * PITCH * 4 <= OFF_LIST && STAGE % 1024 == 0, "sums in the stages' place, stages on whole atoms");
  static int smem(int adapters) { return OFF_TILES + Tiles::ints(adapters) * 4 + 1024; }
};

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}

template <int RP>
__global__ void __launch_bounds__(kThreads, 2) lora_prompt_shrink_kernel(const __grid_constant__ LoraParams p) {
  using G = PromptShrinkGeo<RP>;
  extern __shared__ __align__(16) uint8_t raw[];
  uint8_t *smem = raw + (1024 - smem_u32(raw) % 1024) % 1024;  // (the swizzle goes by address)
  int *list = reinterpret_cast<int *>(smem + G::OFF_LIST);
  volatile int *abort = reinterpret_cast<volatile int *>(smem + G::OFF_BAR + G::STAGES * 8);
  const uint32_t base = smem_u32(smem), bar = base + G::OFF_BAR, slot = bar + G::STAGES * 8 + 4;
  Tiles tiles(reinterpret_cast<int *>(smem + G::OFF_TILES), p.adapters);
  const int parts = (int)cluster_nctarank(), part = (int)cluster_ctarank(), tile = (int)cluster_id_x();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dependency_wait();
  grid_launch_dependents();
  tiles.make<2 * kTile>(p);
  // No token is counted twice, so there are as many clusters (and lists) as tiles, and more
  const int all = tiles.first[p.adapters + 1];
  if (tile == 0 && part == 0 && threadIdx.x == 0) {
    p.head[0] = 2 * tiles.first[p.adapters];
    p.head[1] = 2 * all;
  }
  if (tile >= all) return;  // (all CTAs of the cluster do, here and below)
  const int e = tiles.of(tile), lo = (tile - tiles.first[e]) * 2 * kTile, n = min(2 * kTile, tiles.count[e] - lo);
  if (e == p.adapters && p.in_place) return;
  tiles.tokens(p, e, lo, lo + n, list);
  if (part == 0) {  // two lists, the second one perhaps empty
    int *to = p.lists + 2ll * tile * kListInts;
    for (int i = threadIdx.x; i < n; i += kThreads) to[i / kTile * kListInts + i % kTile] = list[i];
    if (threadIdx.x < 2) {
      to[threadIdx.x * kListInts + kTile] = e;
      to[threadIdx.x * kListInts + kTile + 1] = max(0, min(kTile, n - (int)threadIdx.x * kTile));
    }
  }
  if (e == p.adapters) return;

  __syncwarp();
  if (warp == 0) {
    tmem_alloc(slot, G::COLS);
    tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    *abort = 0;
    for (int i = 0; i < G::STAGES; ++i) mbar_init(bar + 8 * i, 1);
    fence_mbar_init();
  }
  const int steps = (p.inner + 63) / 64;
  const int s0 = (int)((long long)steps * part / parts), count = (int)((long long)steps * (part + 1) / parts) - s0;
  // a thread copies the same 16 bytes of k of every 32nd row
  const int c = threadIdx.x & 7, r0 = threadIdx.x >> 3;
  const uint16_t *xr[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) xr[i] = r0 + i * 32 < n ? p.x + (long long)list[r0 + i * 32] * p.x_row + c * 8 : nullptr;
  const uint16_t *ar = p.a + e * p.a_adapter + r0 * p.a_row + c * 8;
  const uint32_t to = base + r0 * 128 + ((c ^ (r0 & 7)) << 4);
  auto fetch = [&](int i) {
    if (i < count) {
      const uint32_t at = to + i % G::STAGES * G::STAGE;
      const int k = (s0 + i) * 64;
      const bool in = k + c * 8 < p.inner;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (xr[r]) copy16(at + r * 32 * 128, in ? xr[r] + k : p.x, in);
#pragma unroll
      for (int r = 0; r < (RP + 31) / 32; ++r)
        if (RP >= 32 || r0 < RP) {
          const bool there = in && r0 + r * 32 < p.rank;
          copy16(at + G::X + r * 32 * 128, there ? ar + r * 32 * p.a_row + k : p.a, there);
        }
    }
    copy_commit();
  };
#pragma unroll
  for (int i = 0; i < G::STAGES - 1; ++i) fetch(i);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = lds32(slot);
  __syncwarp();
  bool ok = true;
  auto wait = [&](int i) {
    if (ok && !mbar_wait<true>(bar + i % G::STAGES * 8, i / G::STAGES & 1, abort)) {
      ok = false;
      *abort = 1;
      atomicOr(p.err, kErrTimeout);
    }
  };
  for (int i = 0; i < count; ++i) {
    copy_wait<G::STAGES - 2>();
    fence_proxy_async_smem();
    __syncthreads();
    if (threadIdx.x == 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(128, RP);
      const uint64_t x = sw128_desc(base + i % G::STAGES * G::STAGE), a = sw128_desc(base + i % G::STAGES * G::STAGE + G::X);
#pragma unroll
      for (int k = 0; k < 4; ++k) tc_mma_f16(tmem, x + 2 * k, a + 2 * k, idesc, (uint32_t)(i | k));
      tc_commit(bar + i % G::STAGES * 8);
    }
    if (i) wait(i - 1);  // (its stage is the one that the next copies go to)
    fetch(i + G::STAGES - 1);
  }
  copy_wait<0>();
  if (count) {
    wait(count - 1);
    if (!ok) mbar_wait_drain(bar + (count - 1) % G::STAGES * 8, (count - 1) / G::STAGES & 1);
  }
  tc_fence_after();
  __syncthreads();  // (nobody writes sums before everybody's products are done)
  float *sums = reinterpret_cast<float *>(smem);
  {
    const int row = (warp & 3) * 32 + lane, c0 = warp < 4 ? 0 : RP / 2;
#pragma unroll
    for (int q = 0; q < (RP >= 32 ? RP / 32 : 1); ++q) {
      if (RP < 32 && warp >= 4) break;
      float v[16];
      tmem_ld16(tmem + ((uint32_t)((warp & 3) * 32) << 16) + c0 + q * 16, v);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (c0 + q * 16 + k * 4 < RP)
          *reinterpret_cast<float4 *>(sums + row * G::PITCH + c0 + q * 16 + k * 4) =
              count ? make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, G::COLS);
  cluster_sync_all();
  const float scale = p.scale ? p.scale[e] : 1.f;
  const int rows = 128 / parts;
  for (int i = threadIdx.x; i < rows * RP / 4; i += kThreads) {
    const int row = part * rows + i * 4 / RP, r = i * 4 % RP;
    if (row >= n) break;
    const uint32_t at = base + (row * G::PITCH + r) * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int q = 0; q < parts; ++q) {
      const float4 u = ld_cluster_f4(mapa_shared(at, q));
      v.x += u.x;
      v.y += u.y;
      v.z += u.z;
      v.w += u.w;
    }
    v = r < p.rank ? make_float4(v.x * scale, v.y * scale, v.z * scale, v.w * scale) : make_float4(0.f, 0.f, 0.f, 0.f);  // (as above)
    constexpr int P = parts_of_rank(RP);
    uint32_t a[P], b[P];
    in_parts(v.x, v.y, a);
    in_parts(v.z, v.w, b);
    uint16_t *out = p.low + (long long)list[row] * (P * RP) + r;
#pragma unroll
    for (int k = 0; k < P; ++k) *reinterpret_cast<uint2 *>(out + k * RP) = make_uint2(a[k], b[k]);
  }
  cluster_sync_all();  // (the others may still be reading this CTA's part)
}

// 16 lanes of TMEM by 16 or 32 columns: thread 4g + t has of lane g columns 8i + 2t
// and the next in v[4i], v[4i + 1], of lane g + 8 in v[4i + 2], v[4i + 3]
__device__ __forceinline__ void tmem_ld_16x256b(uint32_t taddr, uint32_t (&v)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "r"(taddr)
               : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_ld_16x256b(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// ---------------------------------------------------------------------------
// expand: a step is 128 tokens of one adapter and NC columns. x A^T of the
// tokens stays in shared memory (its parts side by side, so that one row of B
// serves all), B comes for each step, the product is tcgen05's, 128 by NC, in
// one of two TMEM buffers. y is copied to shared memory two steps ahead; the
// products are added there in place, and a step later the sums leave in whole
// rows. Bound by HBM, which does 6.0 - 6.2 TB/s of such rows read and written (64
// bytes of eight rows an instruction, as a fragment has them: 5.6); rank 16, 4,096
// tokens of 34,816 columns: 103 us from a cold cache, 5.5 TB/s. (With mma.sync and B in
// registers the warps had 460 - 560 instructions for 1,024 elements and ranks of 64 took
// 63 us where 16 took 36.)
//
// Rows need not begin on 16 bytes: element c of a row that begins s elements
// after such a boundary has place c + s, and places are moved eight at a time
// (SHIFT; those at the ends of a row one by one).
// ---------------------------------------------------------------------------
template <int RP>
struct PromptExpandGeo {
  static constexpr int THREADS = 512;
  static constexpr int NC = RP <= 64 ? 128 : 64;
  static constexpr int A_ROW = parts_of_rank(RP) * RP;  // k of a token's x A^T
  static constexpr int A_PANELS = (A_ROW + 63) / 64, A = A_PANELS * 128 * 128;  // of 64 k, rows of 128 bytes, swizzled
  static constexpr int B_PANELS = (RP + 63) / 64, B_PANEL = NC * 128, B = B_PANELS * B_PANEL;
  static constexpr int PITCH = NC * 2 + 16;  // bytes of a token's y: NC places and up to 7 more, without bank conflicts
  static constexpr int OUT = 128 * PITCH;
  static constexpr int OFF_B = A, OFF_OUT = OFF_B + 3 * B, OFF_LISTS = OFF_OUT + 4 * OUT;
  static constexpr int OFF_BAR = OFF_LISTS + 8 * 2 * kListInts * 4;
  static constexpr int SMEM = OFF_BAR + 32 + 1024;
  static constexpr int COLS = 2 * NC;         // of TMEM
  static constexpr int LANES = NC / 8;        // 16-byte pieces of a row
  static constexpr int ROWS = 32 / LANES;     // rows of a warp's copy
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

template <int RP, bool SHIFT>
__global__ void __launch_bounds__(512, 1) lora_prompt_expand_kernel(const __grid_constant__ LoraParams p) {
  using G = PromptExpandGeo<RP>;
  extern __shared__ __align__(16) uint8_t raw[];
  uint8_t *smem = raw + (1024 - smem_u32(raw) % 1024) % 1024;  // (the swizzle goes by address)
  const int *lists = reinterpret_cast<const int *>(smem + G::OFF_LISTS);
  volatile int *abort = reinterpret_cast<volatile int *>(smem + G::OFF_BAR + 16);
  const uint32_t base = smem_u32(smem), bar = base + G::OFF_BAR, slot = bar + 20;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dependency_wait();
  grid_launch_dependents();
  const int chunks = (p.outer + G::NC - 1) / G::NC, tiles = __ldcg(p.head + (p.in_place ? 0 : 1)) / 2;
  const long long steps = (long long)chunks * tiles, first = steps * blockIdx.x / gridDim.x;
  const int count = (int)(steps * (blockIdx.x + 1) / gridDim.x - first);
  if (count <= 0) return;
  if (warp == 0) {
    tmem_alloc(slot, G::COLS);
    tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    *abort = 0;
    mbar_init(bar, 1);
    mbar_init(bar + 8, 1);
    fence_mbar_init();
  }

  // Step i of this CTA's: a tile and a chunk of columns; the chunks of one tile come one after the other. A tile's two
  // lists are in a slot of a ring of 8.
  struct Step {
    int i, tile, chunk;
  };
  auto after = [&](const Step &s) { return s.chunk + 1 < chunks ? Step{s.i + 1, s.tile, s.chunk + 1} : Step{s.i + 1, s.tile + 1, 0}; };
  auto list_of = [&](int tile) { return lists + (tile & 7) * 2 * kListInts; };
  auto token_of = [&](int tile, int r) { return list_of(tile)[r + (r < kTile ? 0 : kListInts - kTile)]; };
  auto adapter_of = [&](int tile) { return list_of(tile)[kTile]; };
  auto tokens_of = [&](int tile) { return list_of(tile)[kTile + 1] + list_of(tile)[kListInts + kTile + 1]; };
  auto fetch_list = [&](int tile) {
    if (tile < tiles && threadIdx.x < 2 * kListInts / 4)
      copy16(base + G::OFF_LISTS + (tile & 7) * 2 * kListInts * 4 + threadIdx.x * 16,
             p.lists + 2ll * tile * kListInts + threadIdx.x * 4);
  };
  // how many elements after a 16-byte boundary a token's row of out begins
  const uint32_t out_at = (uint32_t)(reinterpret_cast<uintptr_t>(p.out) / 2);
  auto shift_of = [&](int token) { return SHIFT ? (int)(out_at + (uint32_t)token * (uint32_t)p.out_row & 7u) : 0; };

  auto fetch_a = [&](int tile) {  // x A^T of a tile
    const int n = tokens_of(tile);
#pragma unroll 4
    for (int id = threadIdx.x; id < 128 * G::A_ROW / 8; id += G::THREADS) {
      const int r = id / (G::A_ROW / 8), c = id % (G::A_ROW / 8);
      if (r < n)
        copy16(base + c / 8 * 128 * 128 + r * 128 + ((c % 8 ^ (r & 7)) << 4), p.low + (long long)token_of(tile, r) * G::A_ROW + c * 8);
    }
  };
  auto fetch_b = [&](const Step &s) {
    const int e = adapter_of(s.tile);
    if (e >= p.adapters) return;
    const uint16_t *b = p.b + e * p.b_adapter + (long long)s.chunk * G::NC * p.b_row;
    const int rows = p.outer - s.chunk * G::NC;
    const uint32_t to = base + G::OFF_B + s.i % 3 * G::B;
#pragma unroll
    for (int id = threadIdx.x; id < G::NC * RP / 8; id += G::THREADS) {
      const int r = id / (RP / 8), c = id % (RP / 8);
      if (r < rows) {
        const bool in = c * 8 < p.rank;
        copy16(to + c / 8 * G::B_PANEL + r * 128 + ((c % 8 ^ (r & 7)) << 4), in ? b + r * p.b_row + c * 8 : p.b, in);
      }
    }
  };
  // y's columns c .. c + 7 of a row, one by one, to shared memory
  auto slow = [&](const uint16_t *from, int c, int c0, int to) {
    uint16_t *v = reinterpret_cast<uint16_t *>(smem + to);
#pragma unroll 1
    for (int k = 0; k < 8; ++k)
      if (c + k >= c0 && c + k < p.outer) v[k] = __ldcg(from + k);
  };
  auto fetch_y = [&](const Step &s) {
    const int n = tokens_of(s.tile), c0 = s.chunk * G::NC, at = G::OFF_OUT + (s.i & 3) * G::OUT;
    const bool inner = c0 > 0 && c0 + G::NC + 8 <= p.outer && (!SHIFT || p.alike);  // whole pieces on all sides
    // piece l of row r (brought with what it holds of the columns beside, which is not used; where that is not y's, slowly)
    auto bring = [&](int r, int l) {
      if (r >= n) return;
      const int token = token_of(s.tile, r), c = c0 - shift_of(token) + 8 * l;
      const uint16_t *from = p.y + (long long)token * p.y_row + c;
      if (inner) {
        copy16(base + at + r * G::PITCH + l * 16, from);
      } else if (c < p.outer && c + 8 > c0) {
        if ((!SHIFT || p.alike) && (c >= 0 || token > 0) && (c + 8 <= p.outer || (SHIFT && token + 1 < p.tokens)))
          copy16(base + at + r * G::PITCH + l * 16, from);
        else slow(from, c, c0, at + r * G::PITCH + l * 16);
      }
    };
#pragma unroll
    for (int i = 0; i < 8 / G::ROWS; ++i) bring(warp * 8 + i * G::ROWS + lane / G::LANES, lane % G::LANES);
    if (SHIFT && lane < 8) bring(warp * 8 + lane, G::LANES);
  };
  auto store = [&](const Step &s) {
    const int n = tokens_of(s.tile), c0 = s.chunk * G::NC;
    const uint8_t *from = smem + G::OFF_OUT + (s.i & 3) * G::OUT;
#pragma unroll
    for (int i = 0; i < 8 / G::ROWS; ++i) {
      const int r = warp * 8 + i * G::ROWS + lane / G::LANES, l = lane % G::LANES;
      if (r >= n) continue;
      const int token = token_of(s.tile, r), sh = shift_of(token), left = p.outer - c0 + sh;  // places of the row from here on
      if (8 * l >= sh && 8 * l + 8 <= left)
        *reinterpret_cast<uint4 *>(p.out + (long long)token * p.out_row + (c0 - sh) + 8 * l) =
            *reinterpret_cast<const uint4 *>(from + r * G::PITCH + l * 16);
    }
    // the places before the first whole piece and past the chunk's, and of the row's last piece, one a thread
    const bool last = c0 + G::NC >= p.outer;
    if (SHIFT || (last && p.outer % 8)) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = warp * 8 + i * 4 + lane / 8, k = lane % 8;
        if (r >= n) continue;
        const int token = token_of(s.tile, r), sh = shift_of(token), left = p.outer - c0 + sh;
        uint16_t *row = p.out + (long long)token * p.out_row + (c0 - sh);
        const uint16_t *one = reinterpret_cast<const uint16_t *>(from + r * G::PITCH);
        if (SHIFT && sh) {
          const int place = k >= sh ? k : G::NC + k;
          if (place < left) row[place] = one[place];
        }
        if (left < G::NC && left % 8) {
          const int place = left / 8 * 8 + k;
          if (place < left && place >= (sh ? 8 : 0)) row[place] = one[place];
        }
      }
    }
  };

  Step now{0, (int)(first / chunks), (int)(first % chunks)}, before = now;
  Step next = after(now), ahead_y = now, ahead_b = now;  // ahead: the next ones to be fetched
  int listed = now.tile, held = now.tile;  // the next list to be fetched; the tile that A is of
#pragma unroll
  for (int i = 0; i < 4; ++i) fetch_list(listed++);
  copy_commit();
  copy_wait<0>();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = lds32(slot);
  __syncwarp();

  bool ok = true;
  int issued = 0;  // products so far: number m goes to TMEM buffer and barrier m % 2
  auto wait = [&](int m) {
    if (ok && !mbar_wait<true>(bar + 8 * (m & 1), m >> 1 & 1, abort)) {
      ok = false;
      *abort = 1;
      atomicOr(p.err, kErrTimeout);
    }
  };
  auto multiply = [&](const Step &s) {  // (what it needs is in shared memory, and fenced)
    if (adapter_of(s.tile) >= p.adapters) return;
    if (threadIdx.x == 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(128, G::NC);
      const uint32_t b = base + G::OFF_B + s.i % 3 * G::B, d = tmem + (issued & 1) * G::NC;
#pragma unroll
      for (int part = 0; part < parts_of_rank(RP); ++part)
#pragma unroll
        for (int k = 0; k < RP; k += 16) {
          const int ka = part * RP + k;
          tc_mma_f16(d, sw128_desc(base + ka / 64 * 128 * 128) + ka % 64 / 8, sw128_desc(b + k / 64 * G::B_PANEL) + k % 64 / 8, idesc,
                     (uint32_t)(ka != 0));
        }
      tc_commit(bar + 8 * (issued & 1));
    }
    ++issued;
  };
  auto fetch_y_next = [&]() {
    if (ahead_y.i < count) {
      fetch_y(ahead_y);
      const int tile = ahead_y.tile;
      ahead_y = after(ahead_y);
      if (ahead_y.tile != tile) fetch_list(listed++);  // (of the tile three on: B is a step ahead of y)
    }
  };
  auto fetch_b_next = [&]() {
    if (ahead_b.i < count) {
      fetch_b(ahead_b);
      ahead_b = after(ahead_b);
    }
  };
  fetch_a(now.tile);
  fetch_b_next();
  copy_commit();
  fetch_y_next();
  fetch_b_next();
  copy_commit();
  fetch_y_next();
  fetch_b_next();
  copy_commit();
  copy_wait<2>();
  fence_proxy_async_smem();
  __syncthreads();
  multiply(now);
  for (; now.i < count; before = now, now = next, next = after(next)) {
    copy_wait<1>();
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();  // this step's y and the next one's B are there, the sums of the step before, and its TMEM is read
    tc_fence_after();
    const int mine = issued - 1;
    const bool adapted = adapter_of(now.tile) < p.adapters;
    if (next.i < count && next.tile != held) {
      if (adapted) wait(mine);  // (A is still being read)
      held = next.tile;
      if (adapter_of(held) < p.adapters) fetch_a(held);
      copy_commit();
      copy_wait<0>();
      fence_proxy_async_smem();
      __syncthreads();
    }
    if (next.i < count) multiply(next);
    if (adapted) wait(mine);
    fetch_y_next();
    fetch_b_next();
    copy_commit();
    if (now.i) store(before);
    if (adapted) {
      tc_fence_after();
      constexpr int W = G::NC / 4;  // columns of a warp, which has 32 tokens
      const int r0 = (warp & 3) * 32, c = (warp >> 2) * W, n = tokens_of(now.tile);
      const uint32_t sums = tmem + ((uint32_t)r0 << 16) + (mine & 1) * G::NC + c;
      uint8_t *out = smem + G::OFF_OUT + (now.i & 3) * G::OUT;
      __syncwarp();
      if (!SHIFT) {  // a token a lane, eight columns at a time
        uint8_t *row = out + (r0 + lane) * G::PITCH + c * 2;
#pragma unroll
        for (int q = 0; q < W; q += 16) {
          float v[16];
          tmem_ld16(sums + q, v);
#pragma unroll
          for (int o = 0; o < 16; o += 8) {
            uint4 *at = reinterpret_cast<uint4 *>(row + (q + o) * 2);
            uint4 y = *at;
            y.x = pack_bf16(bf16lo_to_f32(y.x) + v[o], bf16hi_to_f32(y.x) + v[o + 1]);
            y.y = pack_bf16(bf16lo_to_f32(y.y) + v[o + 2], bf16hi_to_f32(y.y) + v[o + 3]);
            y.z = pack_bf16(bf16lo_to_f32(y.z) + v[o + 4], bf16hi_to_f32(y.z) + v[o + 5]);
            y.w = pack_bf16(bf16lo_to_f32(y.w) + v[o + 6], bf16hi_to_f32(y.w) + v[o + 7]);
            *at = y;
          }
        }
      } else {
        // two columns of eight tokens a lane (columns 8i + 2t, 8i + 2t + 1), one by one, so that the lanes' places,
        // wherever the tokens' rows begin, are in different banks
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int up = 0; up < 32; up += 16) {
          uint32_t v[W / 2];
          tmem_ld_16x256b(sums + ((uint32_t)up << 16), v);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int r = r0 + up + h * 8 + g, sh = r < n ? shift_of(token_of(now.tile, r)) : 0;
            uint16_t *y = reinterpret_cast<uint16_t *>(out + r * G::PITCH) + c + sh + 2 * t, x[W / 4];
#pragma unroll
            for (int i = 0; i < W / 8; ++i) {
              x[2 * i] = y[8 * i];
              x[2 * i + 1] = y[8 * i + 1];
            }
#pragma unroll
            for (int i = 0; i < W / 8; ++i) {
              const uint32_t w = pack_bf16(bf16lo_to_f32(x[2 * i]) + __uint_as_float(v[4 * i + 2 * h]),
                                           bf16lo_to_f32(x[2 * i + 1]) + __uint_as_float(v[4 * i + 2 * h + 1]));
              y[8 * i] = (uint16_t)w;
              y[8 * i + 1] = (uint16_t)(w >> 16);
            }
          }
        }
      }
    }
  }
  copy_wait<0>();
  tc_fence_before();
  __syncthreads();
  store(before);
  if (!ok && issued) mbar_wait_drain(bar + 8 * (issued - 1 & 1), issued - 1 >> 1 & 1);
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, G::COLS);
}

// ---------------------------------------------------------------------------
int padded_rank(int rank, bool few) { return rank <= 8 && few ? 8 : rank <= 16 ? 16 : rank <= 32 ? 32 : rank <= 64 ? 64 : 128; }

// Few tokens take the first pair of kernels, whose tiles of 16 read their adapter
// anew; the prompts' tiles of 128 are late to begin, and mostly empty where many
// adapters share few tokens. First | second pair, K 5,120, one adapter, three
// inputs in turn:
//   columns  tokens  rank 16     rank 64     rank 128
//    34,816     256  19.2 | 25.2 25.0 | 26.2  53 | 34 us
//    34,816     512  30.8 | 32.1 39.0 | 33.5  94 | 45
//    34,816     768  42.3 | 38.5 56.0 | 40.9 128 | 58
//     7,168   1,024  20.0 | 23.4 26.0 | 24.2
//     7,168   2,048  31.4 | 28.9 45.7 | 30.5
//     1,024   1,536  11.1 | 19.2 16.8 | 19.9  31 | 23
// and 1,024 rows of one token and 48 adapters, 34,816 columns 83 | 146 with rank 16,
// 120 | 163 with 64. So the first pair has y up to 2^24 elements and products up to
// 2^30 of tokens, ranks and K + columns (above rank 64, where an SM has one CTA of
// expand, K + 2 columns: 1,090 tokens, K 320, 7,232 columns 45 | 26, but 515 tokens, K
// 7,248, 2,854 columns 23 | 30). At three points of the table that is the slower side,
// by 4 to 9 %. It also has calls of fewer than 32 tokens for each adapter that the rows
// could have (as many as the store has, or as there are rows: which ones they have only
// the device knows, so a prompt that is given as a row for each token, beside a large
// store, takes it too).
constexpr int kAlwaysFew = 128, kMostFew = 2048;
bool few(const LoraCall &c, int groups) {
  if (c.tokens <= kAlwaysFew || c.tokens > kMostFew) return c.tokens <= kAlwaysFew;
  const long long t = c.tokens, columns = c.rank > 64 ? 2LL * c.outer : c.outer;
  return (t * c.outer <= 1 << 24 && t * c.rank * (c.inner + columns) <= 1 << 30) || t < 32LL * groups;
}
int groups_of(int adapters, int rows) { return adapters < rows ? adapters : rows; }

// Few tokens: parts of K. As many CTAs as fit at once (304: two on each of 152 SMs;
// not asked of the device, because the workspace's size follows from it), but at least
// two steps of 32 k for each warp (one token: 5.4 us, with one step 6.1, with four
// 6.1), and no more than 32 sums for expand to add up.
int parts_of(int tokens, int rank, int inner) {
  const int tiles = (tokens + 15) / 16, step = 2 * 32 * (rank > 64 ? kWarps / 2 : kWarps);
  const int want = 304 / tiles, most = (inner + step - 1) / step;
  return want < 1 ? 1 : want < most ? (want < 32 ? want : 32) : (most < 32 ? most : 32);
}

// Prompts: CTAs of a cluster, which share K: as many as bring 128 tokens each to
// a wave (two CTAs per SM), while each keeps 512 k. Up to four: 4,096 tokens 144 us
// with one, 128 with two, 121 with four or eight; six prompts of 2,000 92.7, 80.3,
// 74.5 (two and more). Three, or five to eight, where they fit: 6,000 tokens 57 us
// against 65 with three.
int cluster_of(int tokens, int inner, int sm_count) {
  int s = 1;
  while (s < 4 && (long long)((tokens + 127) / 128) * s * 2 <= 2 * sm_count && inner >= 1024 * s) s *= 2;
  return s;
}

// Prompts: x A^T, after the numbers of tiles
size_t low_bytes(int tokens, int rank) {
  const int padded = padded_rank(rank, false);
  return align_up((size_t)tokens * padded * parts_of_rank(padded) * sizeof(uint16_t), 256);
}

// Prompts: clusters at most, whatever the rows' adapters (no more groups than tokens); each has two lists
long long most_clusters(int tokens, int groups) { return tokens / (2 * kTile) + (long long)groups + 1; }

// `most`: what the kernel may need of shared memory, asked for on its first launch on a device (every time: 0.4 us)
template <class K>
cudaError_t launch(K kern, PerDevice &asked, int most, int device, unsigned grid, int cluster, int smem, cudaStream_t stream,
                   const LoraParams &p, int threads = kThreads) {
  if (smem > 48 * 1024 && !asked.v[device].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
    asked.v[device].store(1, std::memory_order_release);
  }
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(grid, 1, 1);
  lc.blockDim = dim3(threads, 1, 1);
  lc.dynamicSmemBytes = smem;
  lc.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&lc, kern, p);
}

template <int RP>
cudaError_t run_few(const LoraCall &c, const LoraParams &p, bool even) {
  const long long tiles = c.tokens / 16 + groups_of(c.adapters, c.rows) + 1;  // at most
  const long long shrink = tiles * p.ksplit, expand = tiles * ((c.outer + kColumns - 1) / kColumns);
  const long long cap = c.sm_count * 2;
  static PerDevice first, second[2];
  const cudaError_t e = launch(lora_shrink_kernel<RP>, first, ShrinkGeo<RP>::smem(kMaxAdapters), c.device, (unsigned)(shrink < cap ? shrink : cap), 1,
                               ShrinkGeo<RP>::smem(c.adapters), c.stream, p);
  if (e != cudaSuccess) return e;
  return launch(even ? lora_expand_kernel<RP, true> : lora_expand_kernel<RP, false>, second[even],
                ExpandGeo<RP>::smem(kMaxAdapters), c.device,
                (unsigned)(expand < c.sm_count * ExpandGeo<RP>::ctas(even) ? expand : c.sm_count * ExpandGeo<RP>::ctas(even)), 1, ExpandGeo<RP>::smem(c.adapters), c.stream, p);
}

template <int RP>
cudaError_t run_prompts(const LoraCall &c, const LoraParams &p, bool even) {
  const int cluster = cluster_of(c.tokens, c.inner, c.sm_count);
  const long long clusters = most_clusters(c.tokens, groups_of(groups_of(c.adapters, c.rows), c.tokens));
  static PerDevice first, second[2];
  const cudaError_t e = launch(lora_prompt_shrink_kernel<RP>, first, PromptShrinkGeo<RP>::smem(kMaxAdapters), c.device, (unsigned)(clusters * cluster), cluster,
                               PromptShrinkGeo<RP>::smem(c.adapters), c.stream, p);
  if (e != cudaSuccess) return e;
  return launch(even ? lora_prompt_expand_kernel<RP, false> : lora_prompt_expand_kernel<RP, true>, second[even],
                PromptExpandGeo<RP>::SMEM, c.device,
                (unsigned)c.sm_count, 1, PromptExpandGeo<RP>::SMEM, c.stream, p, PromptExpandGeo<RP>::THREADS);
}

template <int RP>
cudaError_t run(const LoraCall &c, const LoraParams &p, bool few, bool even) {
  if (few) return run_few<RP>(c, p, even);
  return run_prompts<(RP < 16 ? 16 : RP)>(c, p, even);
}

}  // namespace

// Of the pair that needs more, of those that a call of up to so many tokens may
// take: what is enough for many tokens is enough for few.
size_t lora_workspace_bytes(int tokens, int rank, int inner) {
  size_t sums = 0;
  for (int t = 16; t < 16 + tokens && t <= kMostFew; t += 16) {
    const size_t n = (size_t)parts_of(t, rank, inner) * (t < tokens ? t : tokens);
    if (n > sums) sums = n;
  }
  size_t bytes = align_up(sums * padded_rank(rank, true) * sizeof(float), 256);
  if (tokens > kAlwaysFew) {
    const size_t lists = (size_t)most_clusters(tokens, groups_of(kMaxAdapters, tokens)) * 2 * kListInts * sizeof(int);
    const size_t prompts = 256 + low_bytes(tokens, rank) + align_up(lists, 256);
    if (prompts > bytes) bytes = prompts;
  }
  return bytes;
}

cudaError_t launch_lora_add(const LoraCall &c) {
  LoraParams p{c.y, c.x, c.a, c.b, (int)c.y_row, (int)c.x_row, c.a_adapter, c.a_row, c.b_adapter, c.b_row, (int)c.out_row,
               c.scale, c.adapter, c.starts, c.rows, c.tokens, c.adapters, c.rank, c.inner, c.outer,
               1, c.out, nullptr, nullptr, nullptr, nullptr, c.err, c.out == c.y && c.out_row == c.y_row,
               (reinterpret_cast<uintptr_t>(c.out) - reinterpret_cast<uintptr_t>(c.y)) % 16 == 0 && (c.out_row - c.y_row) % 8 == 0 &&
                   (c.y_row >= c.outer || c.tokens == 1)};
  uint8_t *ws = static_cast<uint8_t *>(c.workspace);
  const bool is_few = few(c, groups_of(c.adapters, c.rows));
  if (is_few) {
    p.ksplit = parts_of(c.tokens, c.rank, c.inner);
    p.parts = reinterpret_cast<float *>(ws);
  } else {
    p.head = reinterpret_cast<int *>(ws);
    p.low = reinterpret_cast<uint16_t *>(ws + 256);
    p.lists = reinterpret_cast<int *>(ws + 256 + low_bytes(c.tokens, c.rank));
  }
  const uintptr_t bits = reinterpret_cast<uintptr_t>(c.y) | reinterpret_cast<uintptr_t>(c.out);
  const bool even = bits % 16 == 0 && c.y_row % 8 == 0 && c.out_row % 8 == 0;
  switch (padded_rank(c.rank, is_few)) {
    case 8: return run<8>(c, p, is_few, even);
    case 16: return run<16>(c, p, is_few, even);
    case 32: return run<32>(c, p, is_few, even);
    case 64: return run<64>(c, p, is_few, even);
    default: return run<128>(c, p, is_few, even);
  }
}

}  // namespace w4a16
