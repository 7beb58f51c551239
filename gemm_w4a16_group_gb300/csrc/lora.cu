// Low-rank adapters of many requests beside a shared product:
//
//   out[t] = y[t] + scale_e (x[t] A_e^T) B_e^T,   e the adapter of token t's row
//
// Two launches. `shrink` makes t = x A^T, the sum over K split over CTAs, whose
// float32 parts go to the workspace; `expand` adds them up, applies the scale,
// and adds t B^T to y. Tokens are taken together by adapter, up to 16 or 64 in a
// tile, whichever rows they belong to, so that an adapter is read once for all
// of its tokens (64: once for every 64). Which tokens those are every CTA works
// out for itself from the rows' adapters: a count for each adapter, whose running
// sums number the tiles.
//
// Products are mma.sync (m16n8k16): 16 ranks against every element are 8 to 32
// FLOP a byte, a twentieth of the machine's balance, and the work is to move x,
// y and the adapters. The k order of a fragment is free as long as both operands
// agree, so a lane's 16 bytes of consecutive k serve two products as they come.
#include "w4a16_internal.h"

namespace w4a16 {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kColumns = kWarps * 32;  // of a unit of expand

struct LoraParams {
  const uint16_t *y, *x, *a, *b;
  long long y_row, x_row, a_adapter, a_row, b_adapter, b_row, out_row;
  const float *scale;
  const int32_t *adapter, *starts;
  int rows, tokens, adapters, rank, inner, outer, ksplit;
  uint16_t *out;
  float *parts;  // [ksplit][tokens][RP]
  int *err;
  bool in_place;
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

// First token and number of tokens of row b; none where the offsets cannot be.
__device__ __forceinline__ int row_tokens(const LoraParams &p, int b, int &first) {
  if (!p.starts) {
    first = b;
    return 1;
  }
  first = p.starts[b];
  const int end = p.starts[b + 1];
  if (first < 0 || end < first || end > p.tokens) {
    atomicOr(p.err, kErrIndex);
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

// The tiles of a call, T tokens of one adapter each: count[e] tokens of adapter
// e (the last bin: of none), tiles first[e] .. first[e + 1].
struct Tiles {
  int *count, *first, *sums;
  int bins;

  static __host__ __device__ int ints(int adapters) { return 2 * adapters + 3 + kWarps; }
  __device__ Tiles(int *mem, int adapters)
      : count(mem), first(mem + adapters + 1), sums(mem + 2 * adapters + 3), bins(adapters + 1) {}

  template <int T>
  __device__ void make(const LoraParams &p) {
    for (int e = threadIdx.x; e < bins; e += kThreads) count[e] = 0;
    __syncthreads();
    for (int b = threadIdx.x; b < p.rows; b += kThreads) {
      int s;
      const int n = row_tokens(p, b, s);
      if (n) atomicAdd(&count[row_adapter(p, b)], n);
    }
    __syncthreads();
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
    int done = 0;
    for (int b0 = 0; b0 < p.rows && done < hi; b0 += kThreads) {
      const int b = b0 + threadIdx.x;
      int s = 0, n = 0, total;
      if (b < p.rows && row_adapter(p, b) == e) n = row_tokens(p, b, s);
      __syncthreads();
      const int at = done + block_scan(n, sums, total);
      for (int i = max(lo, at); i < min(hi, at + n); ++i) list[i - lo] = s + i - at;
      done += total;
    }
    __syncthreads();
  }
};

// ---------------------------------------------------------------------------
// shrink: a unit is one tile and one part of K. A warp has all of the tile's
// tokens and up to 64 ranks, and every eighth (RP = 128: fourth) 32 of the
// part's k, straight from memory; the warps' sums meet in shared memory.
// ---------------------------------------------------------------------------
template <int T, int RP>
struct ShrinkGeo {
  static constexpr int MB = T / 16;                // blocks of 16 tokens
  static constexpr int NB = (RP < 64 ? RP : 64) / 8;  // blocks of 8 ranks of a warp
  static constexpr int KW = RP > 64 ? kWarps / 2 : kWarps;  // warps that share K
  static constexpr int STRIDE = NB * 8 + 8;        // floats of a token's sums
  static constexpr int SUMS = kWarps * T * STRIDE * 4;
  static constexpr int OFF_LIST = SUMS, OFF_TILES = OFF_LIST + T * 4;
  static int smem(int adapters) { return OFF_TILES + Tiles::ints(adapters) * 4; }
};

template <int T, int RP>
__global__ void __launch_bounds__(kThreads, T == 16 ? 2 : 1) lora_shrink_kernel(const __grid_constant__ LoraParams p) {
  using G = ShrinkGeo<T, RP>;
  extern __shared__ __align__(16) uint8_t smem[];
  float *sums = reinterpret_cast<float *>(smem);
  int *list = reinterpret_cast<int *>(smem + G::OFF_LIST);
  Tiles tiles(reinterpret_cast<int *>(smem + G::OFF_TILES), p.adapters);
  grid_dependency_wait();
  grid_launch_dependents();  // (so all that came before is complete when expand begins)
  tiles.make<T>(p);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int kw = warp % G::KW, rank0 = warp / G::KW * 64;
  const int steps = (p.inner + 31) / 32;
  const long long units = (long long)tiles.first[p.adapters] * p.ksplit;
  for (long long unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int tile = (int)(unit / p.ksplit), part = (int)(unit % p.ksplit);
    const int e = tiles.of(tile), lo = (tile - tiles.first[e]) * T, n = min(T, tiles.count[e] - lo);
    tiles.tokens(p, e, lo, lo + n, list);
    const uint16_t *xr[G::MB][2];
#pragma unroll
    for (int m = 0; m < G::MB; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = m * 16 + h * 8 + g;
        xr[m][h] = i < n ? p.x + list[i] * p.x_row : nullptr;
      }
    const uint16_t *ar = p.a + e * p.a_adapter + (rank0 + g) * p.a_row;
    float acc[G::MB][G::NB][4] = {};
    const int s1 = (int)((long long)steps * (part + 1) / p.ksplit);
#pragma unroll 2
    for (int s = (int)((long long)steps * part / p.ksplit) + kw; s < s1; s += G::KW) {
      const int k = s * 32 + t * 8;
      const bool in = k < p.inner;
      const uint4 zero = make_uint4(0, 0, 0, 0);
      uint4 xv[G::MB][2], av[G::NB];
#pragma unroll
      for (int j = 0; j < G::NB; ++j)
        av[j] = in && rank0 + j * 8 + g < p.rank ? __ldg(reinterpret_cast<const uint4 *>(ar + j * 8 * p.a_row + k)) : zero;
#pragma unroll
      for (int m = 0; m < G::MB; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) xv[m][h] = in && xr[m][h] ? *reinterpret_cast<const uint4 *>(xr[m][h] + k) : zero;
#pragma unroll
      for (int m = 0; m < G::MB; ++m) {
        if (m * 16 >= n) break;
#pragma unroll
        for (int j = 0; j < G::NB; ++j) {
          mma16(acc[m][j], xv[m][0].x, xv[m][1].x, xv[m][0].y, xv[m][1].y, av[j].x, av[j].y);
          mma16(acc[m][j], xv[m][0].z, xv[m][1].z, xv[m][0].w, xv[m][1].w, av[j].z, av[j].w);
        }
      }
    }
#pragma unroll
    for (int m = 0; m < G::MB; ++m)
#pragma unroll
      for (int j = 0; j < G::NB; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<float2 *>(sums + (warp * T + m * 16 + h * 8 + g) * G::STRIDE + j * 8 + 2 * t) =
              make_float2(acc[m][j][2 * h], acc[m][j][2 * h + 1]);
    __syncthreads();
    float *out = p.parts + (long long)part * p.tokens * RP;
    for (int i = threadIdx.x; i < n * RP / 4; i += kThreads) {
      const int row = i * 4 / RP, r = i * 4 % RP;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < G::KW; ++w) {
        const float4 u = *reinterpret_cast<const float4 *>(sums + ((r / 64 * G::KW + w) * T + row) * G::STRIDE + r % 64);
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
// the tile's tokens. t goes into the product as two bf16 parts (16 bits of
// mantissa: rounded once it would add an error of the size of the output's own
// rounding). The rows of B that a product's eight columns stand for are chosen
// such that a lane ends up with eight consecutive columns of a token: y is read
// and written 16 bytes at a time.
// ---------------------------------------------------------------------------
template <int T, int RP>
struct ExpandGeo {
  static constexpr int MB = T / 16;
  static constexpr int KS = RP < 32 ? 1 : RP / 32;  // 16-byte pieces of k of a lane
  static constexpr int ROW = RP < 32 ? RP * 2 : RP == 32 ? 64 : RP * 2 + 64;  // bytes of a token's t, without bank conflicts
  static constexpr int OFF_LO = T * ROW, OFF_LIST = 2 * T * ROW, OFF_TILES = OFF_LIST + T * 4;
  static int smem(int adapters) { return OFF_TILES + Tiles::ints(adapters) * 4; }
};

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

// eight columns of a row from column c on, `wide`: as one 16-byte access
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

template <int T, int RP, bool EVEN>
__global__ void __launch_bounds__(kThreads, 2) lora_expand_kernel(const __grid_constant__ LoraParams p) {
  using G = ExpandGeo<T, RP>;
  extern __shared__ __align__(16) uint8_t smem[];
  int *list = reinterpret_cast<int *>(smem + G::OFF_LIST);
  Tiles tiles(reinterpret_cast<int *>(smem + G::OFF_TILES), p.adapters);
  // What shrink waited for before it let this launch begin is complete: rows,
  // adapters, y and B may be read; t only after the wait below.
  tiles.make<T>(p);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int chunks = (p.outer + kColumns - 1) / kColumns;
  const long long units = (long long)tiles.first[p.in_place ? p.adapters : p.adapters + 1] * chunks;
  const long long u0 = units * blockIdx.x / gridDim.x, u1 = units * (blockIdx.x + 1) / gridDim.x;
  int here = -1, e = 0, n = 0;
  bool waited = false;
  for (long long unit = u0; unit < u1; ++unit) {
    const int tile = (int)(unit / chunks), c0 = (int)(unit % chunks) * kColumns + warp * 32, c = c0 + 8 * t;
    const bool next = tile != here;
    if (next) {
      __syncthreads();  // (the tile before is done with)
      here = tile;
      e = tiles.of(tile);
      const int lo = (tile - tiles.first[e]) * T;
      n = min(T, tiles.count[e] - lo);
      tiles.tokens(p, e, lo, lo + n, list);
    }
    const bool adapted = e < p.adapters, wide = EVEN && c + 8 <= p.outer;
    uint4 bv[4][G::KS], yv[G::MB][2];
    if (adapted) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int col = c0 + 8 * (g >> 1) + 2 * j + (g & 1);
        const uint8_t *br = reinterpret_cast<const uint8_t *>(p.b + e * p.b_adapter + col * p.b_row);
#pragma unroll
        for (int s = 0; s < G::KS; ++s) {
          const int k = RP < 32 ? t * (RP / 4) : s * 32 + t * 8;
          bv[j][s] = col < p.outer && k < p.rank ? piece<RP>(br + k * 2) : make_uint4(0, 0, 0, 0);
        }
      }
    }
#pragma unroll
    for (int m = 0; m < G::MB; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = m * 16 + h * 8 + g;
        if (i < n) yv[m][h] = load8(p.y + list[i] * p.y_row, c, p.outer, wide);
      }
    if (!waited) {
      grid_dependency_wait();
      waited = true;
    }
    if (next && adapted) {
      const float scale = p.scale ? p.scale[e] : 1.f;
      for (int i = threadIdx.x; i < n * RP / 2; i += kThreads) {
        const int row = i * 2 / RP, r = i * 2 % RP;
        const float *from = p.parts + (long long)list[row] * RP + r;
        float2 v = make_float2(0.f, 0.f);
#pragma unroll 4
        for (int s = 0; s < p.ksplit; ++s) {
          const float2 u = __ldcg(reinterpret_cast<const float2 *>(from + (long long)s * p.tokens * RP));
          v.x += u.x;
          v.y += u.y;
        }
        v.x *= scale;
        v.y *= scale;
        const uint32_t hi = pack_bf16(v.x, v.y);
        const float hx = bf16lo_to_f32(hi), hy = bf16hi_to_f32(hi);
        // (what is left of an infinite value is not a number)
        const uint32_t low = pack_bf16(fabsf(hx) < INFINITY ? v.x - hx : 0.f, fabsf(hy) < INFINITY ? v.y - hy : 0.f);
        *reinterpret_cast<uint32_t *>(smem + row * G::ROW + r * 2) = hi;
        *reinterpret_cast<uint32_t *>(smem + G::OFF_LO + row * G::ROW + r * 2) = low;
      }
      __syncthreads();
    }
#pragma unroll
    for (int m = 0; m < G::MB; ++m) {
      if (m * 16 >= n) break;
      if (adapted) {
        float acc[4][4] = {};
#pragma unroll
        for (int s = 0; s < G::KS; ++s) {
          const int at = (m * 16 + g) * G::ROW + (RP < 32 ? t * (RP / 2) : s * 64 + t * 16);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint8_t *from = smem + (half ? G::OFF_LO : 0) + at;
            const uint4 a0 = piece<RP>(from), a1 = piece<RP>(from + 8 * G::ROW);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              mma16(acc[j], a0.x, a1.x, a0.y, a1.y, bv[j][s].x, bv[j][s].y);
              if (RP >= 32) mma16(acc[j], a0.z, a1.z, a0.w, a1.w, bv[j][s].z, bv[j][s].w);
            }
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t *v = &yv[m][h].x;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            v[j] = pack_bf16(bf16lo_to_f32(v[j]) + acc[j][2 * h], bf16hi_to_f32(v[j]) + acc[j][2 * h + 1]);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = m * 16 + h * 8 + g;
        if (i < n) store8(p.out + list[i] * p.out_row, c, p.outer, wide, yv[m][h]);
      }
    }
  }
  if (!waited) grid_dependency_wait();
  grid_launch_dependents();
}

// ---------------------------------------------------------------------------
int padded_rank(int rank) { return rank <= 8 ? 8 : rank <= 16 ? 16 : rank <= 32 ? 32 : rank <= 64 ? 64 : 128; }

// Tokens of a tile: 16 while a tile of 64 would mostly be empty
int tile_of(int tokens) { return tokens <= 512 ? 16 : 64; }

// Parts of K: as many CTAs as fit at once, but at least one step of 32 k for
// each warp, and no more than 32 sums for expand to add up.
int parts_of(int tokens, int rank, int inner) {
  const int tile = tile_of(tokens), tiles = (tokens + tile - 1) / tile, step = 32 * (rank > 64 ? kWarps / 2 : kWarps);
  const int want = (tile == 16 ? 304 : 152) / tiles, most = (inner + step - 1) / step;
  return want < 1 ? 1 : want < most ? (want < 32 ? want : 32) : (most < 32 ? most : 32);
}

template <class K>
cudaError_t launch(K kern, unsigned grid, int smem, cudaStream_t stream, const LoraParams &p) {
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(grid, 1, 1);
  lc.blockDim = dim3(kThreads, 1, 1);
  lc.dynamicSmemBytes = smem;
  lc.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, kern, p);
}

template <int T, int RP>
cudaError_t run(const LoraCall &c, const LoraParams &p, bool even) {
  const int groups = c.adapters < c.rows ? c.adapters : c.rows;
  const long long tiles = c.tokens / T + groups + 1;  // at most
  const long long shrink = tiles * p.ksplit, expand = tiles * ((c.outer + kColumns - 1) / kColumns);
  const long long cap = c.sm_count * 2;
  const cudaError_t e = launch(lora_shrink_kernel<T, RP>, (unsigned)(shrink < cap ? shrink : cap),
                               ShrinkGeo<T, RP>::smem(c.adapters), c.stream, p);
  if (e != cudaSuccess) return e;
  return launch(even ? lora_expand_kernel<T, RP, true> : lora_expand_kernel<T, RP, false>,
                (unsigned)(expand < cap ? expand : cap), ExpandGeo<T, RP>::smem(c.adapters), c.stream, p);
}

template <int T>
cudaError_t run_rank(const LoraCall &c, const LoraParams &p, bool even) {
  switch (padded_rank(c.rank)) {
    case 8: return run<T, 8>(c, p, even);
    case 16: return run<T, 16>(c, p, even);
    case 32: return run<T, 32>(c, p, even);
    case 64: return run<T, 64>(c, p, even);
    default: return run<T, 128>(c, p, even);
  }
}

}  // namespace

size_t lora_workspace_bytes(int tokens, int rank, int inner) {
  return align_up((size_t)parts_of(tokens, rank, inner) * tokens * padded_rank(rank) * sizeof(float), 256);
}

cudaError_t launch_lora_add(const LoraCall &c) {
  const LoraParams p{c.y, c.x, c.a, c.b, c.y_row, c.x_row, c.a_adapter, c.a_row, c.b_adapter, c.b_row, c.out_row,
                     c.scale, c.adapter, c.starts, c.rows, c.tokens, c.adapters, c.rank, c.inner, c.outer,
                     parts_of(c.tokens, c.rank, c.inner), c.out, c.workspace, c.err, c.out == c.y && c.out_row == c.y_row};
  const uintptr_t bits = reinterpret_cast<uintptr_t>(c.y) | reinterpret_cast<uintptr_t>(c.out);
  const bool even = bits % 16 == 0 && c.y_row % 8 == 0 && c.out_row % 8 == 0;
  return tile_of(c.tokens) == 16 ? run_rank<16>(c, p, even) : run_rank<64>(c, p, even);
}

}  // namespace w4a16
