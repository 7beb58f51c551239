// Attention of drafted tokens over a paged key/value cache.
//
//   s_j = scale * q . k_j,  out = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m)
//
// over the positions j that the token sees (its row's context and, by its
// mask word, the row's new tokens). One pass over the keys with a running
// maximum m and sum; the sums are rescaled when m grows.
//
// This file: the kernel on mma.sync (m16n8k16) for up to 16 query rows per kv
// head (one token of any model, a few tokens of small head groups), and the
// kernel that joins partial results; tree_attn_tc.cu has more rows. 16 rows
// against the whole cache are bound by HBM: every key and value is read once.
// Measured against the copy peak of 6.78 TB/s: bf16 6.2 TB/s at 64 rows of
// 4,096 keys (dim 256: 6.5), e4m3 5.5 TB/s (the conversions take half of the
// integer pipe).
//
//  * 4 computing warps and a copying warp. A stage is 64 or 128 keys: the
//    copying warp's lanes each fetch one box (up to a page's rows by 128 bytes)
//    of keys or values by TMA, swizzled as ldmatrix wants it.
//  * Each computing warp takes its quarter of a stage's keys with all 16 rows,
//    with a maximum, sums and outputs of its own; they meet at the end of an
//    item, through shared memory.
//  * bf16 caches: products of bf16 are exact in float32; the weights e^(s - m)
//    go into the second product as two bf16 parts (hi + lo, 15 bits of
//    mantissa; neither is negative, and neither is 0 where the weight is not, so
//    an infinite value stays infinite), which the tensor cores have time for.
//  * e4m3 caches: codes become f16 exactly (one conversion per pair), q is
//    scaled by a power of two per row so that its largest element is near 2^14
//    and becomes f16 (elements below 2^-24 of the largest lose bits, no more
//    than float32 sums lose anyway), and the weights, times 2^15, are f16 with
//    11 bits (down to 2^-29 of the maximum; smaller ones have fewer).
//  * Only tiles that hold new tokens or the end of the context take the masked
//    path. There, values that are not finite are zeroed in shared memory
//    before the product (0 * NaN is NaN) and added at the end to the rows that
//    see them.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "tree_attn.cuh"

namespace w4a16 {
namespace {

// What beginning and ending an item costs, in key tiles: with 4 rather than 2, 48 ragged rows of an e4m3 cache 116.8 ->
// 112.3 us, 64 even rows of a bf16 cache 174 -> 171 us.
constexpr int kRowsLead = 4;
constexpr int kComputeWarps = 4;
constexpr int kThreads = (kComputeWarps + 1) * 32;

template <int DIM, bool E4M3>
struct RowsGeo {
  static constexpr int KW = kComputeWarps;     // warps that share a stage's keys
  static constexpr int ROWS = 16;
  // keys of a stage: 128 where three such stages fit (e4m3, 48 ragged rows of up to 16,384 keys: 117 us, with 64 keys
  // 138 us)
  static constexpr int KT = DIM * (E4M3 ? 1 : 2) <= 128 || (DIM == 256 && E4M3) ? 128 : 64;
  using Tiles = Tiling<ROWS, KT, ROWS, kRowsLead>;
  static constexpr int KPW = KT / KW;         // keys of a warp per stage
  static constexpr int ELT = E4M3 ? 1 : 2;
  static constexpr int ROWB = DIM * ELT;       // bytes of a cache row
  static constexpr int CW = ROWB < 128 ? ROWB : 128;  // box width
  static constexpr int CH = ROWB / CW;
  static constexpr int SUB = KT * CW;         // one box column of a stage
  static constexpr int SIDE = CH * SUB;
  static constexpr int STAGE = 2 * SIDE;
  static constexpr int CTAS = DIM == 256 ? 1 : 2;  // per SM
  static constexpr int STAGES = (DIM == 256 ? 192 : 96) * 1024 / STAGE;
  static constexpr int KS = DIM / 16;          // k steps of the first product
  static constexpr int NT = KPW / 8;           // 8-key tiles of a warp
  static constexpr int OT = DIM / 8;           // 8-wide output tiles
  static constexpr int Q_BYTES = ROWS * DIM * 2;
  static constexpr int RED_BYTES = ROWS * DIM * 4;
  static constexpr int OFF_Q = STAGES * STAGE;  // q fragments; then the sums that warps exchange
  static constexpr int OFF_ML = OFF_Q + (Q_BYTES > RED_BYTES ? Q_BYTES : RED_BYTES);
  static constexpr int OFF_QS = OFF_ML + KW * ROWS * 8;
  static constexpr int OFF_BAR = OFF_QS + (E4M3 ? ROWS * 4 : 0);
  static constexpr int OFF_INFO = OFF_BAR + 2 * STAGES * 8;
  static constexpr int OFF_MISC = OFF_INFO + STAGES * 4;
  static constexpr int OFF_PLAN = (OFF_MISC + 16 + 15) / 16 * 16;
  static constexpr int SMEM = OFF_PLAN + (int)sizeof(PlanShared);
  static_assert(CTAS * (SMEM + 1024) <= 228 * 1024 && SMEM <= 227 * 1024, "shared memory budget");
  static_assert(STAGES >= 3 && SUB % 512 == 0, "stages");
};

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}

template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&b);
}
// The lower parts of two weights whose upper ones are `hi` (cut off, so that these are not negative), at least 2^-24 of
// them: where a weight is above 0 both parts are, and an infinite value gives infinity in both products.
__device__ __forceinline__ uint32_t low_part(uint32_t lo, uint32_t hi) {
  const __nv_bfloat162 least = __hmul2(*reinterpret_cast<__nv_bfloat162 *>(&hi), __float2bfloat162_rn(5.9604645e-8f));
  const __nv_bfloat162 r = __hmax2(*reinterpret_cast<__nv_bfloat162 *>(&lo), least);
  return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&h);
}

// the 16-bit or 8-bit elements of x that are not finite, as a byte mask
template <bool E4M3>
__device__ __forceinline__ uint32_t not_finite(uint32_t x) {
  uint32_t m = 0;
  if (E4M3) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (((x >> (8 * i)) & 0x7Fu) == 0x7Fu) m |= 0xFFu << (8 * i);
  } else {
    if ((x & 0x7F80u) == 0x7F80u) m |= 0xFFFFu;
    if ((x & 0x7F800000u) == 0x7F800000u) m |= 0xFFFF0000u;
  }
  return m;
}

__device__ __forceinline__ void compute_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// byte offset of 16-byte chunk `c` of row `row` in a box column
template <int CW>
__device__ __forceinline__ uint32_t swz(uint32_t row, uint32_t c) {
  return row * CW + ((c ^ (CW == 128 ? row & 7u : (row >> 1) & 3u)) << 4);
}

// value element d of position `pos`, 0 where there is none
template <bool E4M3>
__device__ float value_at(const AttnParams &p, int b, int head, long long pos, int d) {
  const long long pi = pos >> p.c.page_shift;
  if (pi >= p.r.max_pages) return 0.f;
  const int id = p.r.table[(long long)b * p.r.max_pages + pi];
  if ((unsigned)id >= (unsigned)p.c.pages) return 0.f;
  const uint8_t *a = p.c.v.base + (long long)id * p.c.v.page + (long long)head * p.c.v.head +
                     (pos & (p.c.page_rows - 1)) * p.c.v.row;
  if (E4M3) return __half2float(__half(__nv_cvt_fp8_to_halfraw(a[d], __NV_E4M3)));
  return __uint_as_float((uint32_t) reinterpret_cast<const uint16_t *>(a)[d] << 16);
}

template <int DIM, bool E4M3>
__global__ void __launch_bounds__(kThreads, RowsGeo<DIM, E4M3>::CTAS)
    rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                const __grid_constant__ AttnParams p) {
  using G = RowsGeo<DIM, E4M3>;
  constexpr int KW = G::KW, NT = G::NT, OT = G::OT, KS = G::KS;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + G::OFF_MISC);
  uint32_t *odd_values = reinterpret_cast<uint32_t *>(smem + G::OFF_MISC + 8);  // new tokens with values not finite
  PlanShared &plan = *reinterpret_cast<PlanShared *>(smem + G::OFF_PLAN);
  if (sbase & 1023u) {  // the swizzle counts from multiples of 1,024 (dynamic shared memory starts at one)
    if (tid == 0) atomicOr(p.err, kErrTimeout);
    return;
  }
  auto full = [&](uint32_t s) { return sbase + G::OFF_BAR + 8 * s; };
  auto empty = [&](uint32_t s) { return sbase + G::OFF_BAR + 8 * (G::STAGES + s); };

  if (tid == 0) {
    for (int i = 0; i < G::STAGES; ++i) {
      mbar_init(full(i), 1);
      mbar_init(empty(i), kComputeWarps);
    }
    *abort_flag = 0;
    odd_values[0] = odd_values[1] = 0;
    fence_mbar_init();
  }
  grid_dependency_wait();
  grid_launch_dependents();
  plan_share<typename G::Tiles, kThreads>(p, plan);
  __syncthreads();
  Cursor cur{plan.at, plan.end, plan.at < plan.end ? plan.unit : plan.end, plan.b, plan.head, plan.rt};
  Segment sg;

  if (warp == kComputeWarps) {
    // ------------------------------------------------------------ copies
    const int br = min(p.c.page_rows, G::KT), parts = G::KT / br;
    const int part = lane % parts, col = lane / parts % G::CH, side = lane / parts / G::CH;
    const bool has_box = side < 2;
    uint64_t pol;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(pol));
    if (lane == 0) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    uint32_t st = 0;
    bool ok = true;
    while (ok && next_segment<typename G::Tiles>(p, cur, sg)) {
      const int32_t *ids = p.r.table + (long long)sg.b * p.r.max_pages;
      auto id_of = [&](int kt) {  // -1: past the keys
        const long long key = (long long)kt * G::KT + part * br;
        return kt < sg.kt1 && key < sg.i.keys ? ids[key >> p.c.page_shift] : -1;
      };
      int next = id_of(sg.kt0);
      for (int kt = sg.kt0; kt < sg.kt1; ++kt, ++st) {
        const int id = next;
        next = id_of(kt + 1);
        const uint32_t s = st % G::STAGES;
        ok = mbar_wait(empty(s), ((st / G::STAGES) & 1) ^ 1, abort_flag);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        const int key = kt * G::KT + part * br;
        const bool valid = (unsigned)id < (unsigned)p.c.pages;
        const bool load = has_box && valid;
        if (has_box && !valid && key < sg.i.keys && side == 0 && col == 0) attn_flag(p.err);
        const uint32_t loads = __ballot_sync(0xFFFFFFFFu, load);
        if (lane == 0) {
          // which 16-key groups are there: those of the parts that load
          uint32_t groups = 0;
          for (int i = 0; i < parts; ++i)
            if (loads >> i & 1) groups |= ((1u << (br / 16)) - 1) << (i * br / 16);
          *reinterpret_cast<volatile uint32_t *>(smem + G::OFF_INFO + 4 * s) = groups;
          mbar_arrive_expect_tx(full(s), __popc(loads) * br * G::CW);
        }
        __syncwarp();
        if (load)
          tma_load_4d(sbase + s * G::STAGE + side * G::SIDE + col * G::SUB + part * br * G::CW, side ? &tm_v : &tm_k,
                      col * (G::CW / G::ELT), key & (p.c.page_rows - 1), sg.head, id, full(s), pol);
        __syncwarp();
      }
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      atomicOr(p.err, kErrTimeout);
      // every copy issued lands before the CTA can exit
      for (uint32_t i = 0; i < (uint32_t)G::STAGES && i < st; ++i) {
        const uint32_t u = st - 1 - i;
        mbar_wait_drain(full(u % G::STAGES), (u / G::STAGES) & 1);
      }
    }
    return;
  }

  // -------------------------------------------------------------- products
  const int kw = warp;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t qaddr = sbase + G::OFF_Q + lane * 16;
  float *ml = reinterpret_cast<float *>(smem + G::OFF_ML);
  float *qscale = reinterpret_cast<float *>(smem + G::OFF_QS);
  uint32_t st = 0;
  bool ok = true;  // after a wait that gave up: no more waits, but every barrier below is still met

  while (next_segment<typename G::Tiles>(p, cur, sg)) {
    const int rows = sg.rows;
    // ---- q in the order of the A fragments (16 bytes per lane and k step)
    compute_sync();  // the last item's exchange is over
    if (E4M3) {
      // one row per 8 threads: its largest exponent, as the power of two that takes it to 2^14
      for (int r = tid >> 3; r < G::ROWS; r += kComputeWarps * 4) {
        const int rr = sg.rt * G::ROWS + r;
        uint32_t top = 0;
        if (r < rows) {
          const uint4 *src = reinterpret_cast<const uint4 *>(p.q + (sg.i.start + rr / p.group) * p.q_token +
                                                             (sg.head * p.group + rr % p.group) * p.q_head);
          for (int i = tid & 7; i < DIM / 8; i += 8) {
            const uint4 x = src[i];
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) top = max(top, max((w[e] >> 7) & 0xFFu, (w[e] >> 23) & 0xFFu));
          }
        }
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
        // 2^(14 - (top - 127)), within float32's exponents; a row that is not finite stays as it is
        const int e = top == 0xFFu ? 0 : min(141 - (int)top, 120);
        if ((tid & 7) == 0) qscale[r] = __uint_as_float((uint32_t)(127 + e) << 23);
      }
      compute_sync();
    }
    for (int i = tid; i < G::ROWS * (DIM / 8); i += kComputeWarps * 32) {
      const int r = i / (DIM / 8), c8 = i % (DIM / 8);  // 8 elements from 8 * c8
      const int rr = sg.rt * G::ROWS + r;
      uint4 x = make_uint4(0, 0, 0, 0);
      if (r < rows)
        x = *reinterpret_cast<const uint4 *>(p.q + (sg.i.start + rr / p.group) * p.q_token +
                                             (sg.head * p.group + rr % p.group) * p.q_head + 8 * c8);
      uint32_t w[4] = {x.x, x.y, x.z, x.w};
      const int step = c8 >> 1, half = c8 & 1, hi = (r >> 3) & 1;
      const uint32_t base = sbase + G::OFF_Q + step * 512 + (r & 7) * 64;
      if (E4M3) {
        const float f = qscale[r];
        // a lane's four k of a step are d = 4t .. 4t + 3, as four codes of a key come
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t y = pack_f16(bf16lo_to_f32(w[e]) * f, bf16hi_to_f32(w[e]) * f);
          const int tt = half * 2 + (e >> 1);
          asm volatile("st.shared.u32 [%0], %1;" ::"r"(base + tt * 16 + (hi + 2 * (e & 1)) * 4), "r"(y) : "memory");
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          asm volatile("st.shared.u32 [%0], %1;" ::"r"(base + e * 16 + (hi + 2 * half) * 4), "r"(w[e]) : "memory");
      }
    }
    // this thread's two rows (g and g + 8 of the warp's 16): mask word, score factor
    unsigned long long word[2];
    float factor[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = g + 8 * i;
      const int tok = (sg.rt * G::ROWS + r) / p.group;
      word[i] = 0;
      if (r < rows) word[i] = p.mask ? (unsigned long long)p.mask[sg.i.start + tok] : (2ull << tok) - 1;
      factor[i] = p.scale_log2;
    }
    if (tid < 2) odd_values[tid] = 0;
    compute_sync();
    if (E4M3) {
      const float ks = p.c.k.scale[sg.head];
#pragma unroll
      for (int i = 0; i < 2; ++i) factor[i] = p.scale_log2 * ks / qscale[g + 8 * i];
    }
    constexpr bool QREG = KS <= 8;
    uint32_t qf[QREG ? KS : 1][4];
    if (QREG) {
#pragma unroll
      for (int c = 0; c < KS; ++c) {
        const uint4 x = lds128(qaddr + c * 512);
        qf[QREG ? c : 0][0] = x.x;
        qf[QREG ? c : 0][1] = x.y;
        qf[QREG ? c : 0][2] = x.z;
        qf[QREG ? c : 0][3] = x.w;
      }
    }
    float o[OT][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float lsum[4] = {0.f, 0.f, 0.f, 0.f};  // 8 bits: the sums of the weights as they were rounded, by one more product
#pragma unroll
    for (int i = 0; i < OT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

    for (int kt = sg.kt0; kt < sg.kt1; ++kt, ++st) {
      const uint32_t stage = st % G::STAGES;
      if (ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait<true>(full(stage), (st / G::STAGES) & 1, abort_flag));
      const uint32_t groups = *reinterpret_cast<volatile uint32_t *>(smem + G::OFF_INFO + 4 * stage);
      const uint32_t kbase = sbase + stage * G::STAGE, vbase = kbase + G::SIDE;
      const int key0 = kt * G::KT;
      const bool masked = key0 + G::KT > sg.i.len || groups != (1u << (G::KT / 16)) - 1;
      if (masked) {
        // values that must not meet a weight of 0, in the rows that this warp will read
        for (int i = lane; i < G::KPW * (G::ROWB / 16); i += 32) {
          const int j = kw * G::KPW + i / (G::ROWB / 16), c = i % (G::ROWB / 16);
          const int key = key0 + j;
          const bool there = key < sg.i.keys && (groups >> (j >> 4) & 1);
          if (there && key < sg.i.len) continue;
          const uint32_t a = vbase + (c / (G::CW / 16)) * G::SUB + swz<G::CW>(j, c % (G::CW / 16));
          uint4 x = make_uint4(0, 0, 0, 0);
          bool clean = false;
          if (there) {
            x = lds128(a);
            const uint32_t b0 = not_finite<E4M3>(x.x), b1 = not_finite<E4M3>(x.y), b2 = not_finite<E4M3>(x.z),
                           b3 = not_finite<E4M3>(x.w);
            clean = !(b0 | b1 | b2 | b3);
            if (!clean) {
              x = make_uint4(x.x & ~b0, x.y & ~b1, x.z & ~b2, x.w & ~b3);
              const int n = key - sg.i.len;
              atomicOr(&odd_values[n >> 5], 1u << (n & 31));
            }
          }
          if (!clean) sts128(a, x);
        }
        __syncwarp();
      }
      // ---- scores of the warp's keys
      float s[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
      const uint32_t krow = kw * G::KPW + (lane & 7);
      if constexpr (E4M3) {
        // one ldmatrix: 8 keys by 64 codes, 4 k steps
#pragma unroll
        for (int cc = 0; cc < DIM / 64; ++cc) {
          uint32_t a[4][4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            if constexpr (QREG) {
#pragma unroll
              for (int e = 0; e < 4; ++e) a[u][e] = qf[cc * 4 + u][e];
            } else {
              const uint4 x = lds128(qaddr + (cc * 4 + u) * 512);
              a[u][0] = x.x; a[u][1] = x.y; a[u][2] = x.z; a[u][3] = x.w;
            }
          }
          const uint32_t ch = cc * 4 + (lane >> 3);
          const uint32_t colb = kbase + (ch / (G::CW / 16)) * G::SUB;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            uint32_t b[4];
            ldsm4(colb + swz<G::CW>(krow + n * 8, ch % (G::CW / 16)), b);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              uint32_t lo, hi;
              e4m3x4_f16(b[u], lo, hi);
              mma16816<true>(s[n], a[u], lo, hi);
            }
          }
        }
      } else {
        // one ldmatrix: 8 keys by 32 elements, 2 k steps
#pragma unroll
        for (int cc = 0; cc < DIM / 32; ++cc) {
          uint32_t a[2][4];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            if constexpr (QREG) {
#pragma unroll
              for (int e = 0; e < 4; ++e) a[u][e] = qf[cc * 2 + u][e];
            } else {
              const uint4 x = lds128(qaddr + (cc * 2 + u) * 512);
              a[u][0] = x.x; a[u][1] = x.y; a[u][2] = x.z; a[u][3] = x.w;
            }
          }
          const uint32_t ch = cc * 4 + (lane >> 3);
          const uint32_t colb = kbase + (ch >> 3) * G::SUB;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            uint32_t b[4];
            ldsm4(colb + swz<128>(krow + n * 8, ch & 7), b);
            mma16816<false>(s[n], a[0], b[0], b[1]);
            mma16816<false>(s[n], a[1], b[2], b[3]);
          }
        }
      }
      // ---- softmax
      if (masked) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = kw * G::KPW + n * 8 + 2 * t + (e & 1), key = key0 + j, nw = key - sg.i.len;
            const bool sees = (groups >> (j >> 4) & 1) && key < sg.i.keys && (nw < 0 || (word[e >> 1] >> nw & 1));
            if (!sees) s[n][e] = -INFINITY;
          }
      }
      float base[2], alpha[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float top = -INFINITY;
#pragma unroll
        for (int n = 0; n < NT; ++n) top = fmaxf(top, fmaxf(s[n][2 * i], s[n][2 * i + 1]));
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        const float mn = fmaxf(m[i], top * factor[i]);
        base[i] = mn == -INFINITY ? 0.f : mn;
        alpha[i] = exp2_approx(m[i] - base[i]);
        m[i] = mn;
        if (E4M3) base[i] -= 15.f;  // weights times 2^15: f16 ends at 2^16, and loses bits below 2^-14
        l[i] *= alpha[i];
        lsum[2 * i] *= alpha[i];
      }
      if (__any_sync(0xFFFFFFFFu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
        for (int i = 0; i < OT; ++i) {
          o[i][0] *= alpha[0];
          o[i][1] *= alpha[0];
          o[i][2] *= alpha[1];
          o[i][3] *= alpha[1];
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = exp2_approx(fmaf(s[n][e], factor[e >> 1], -base[e >> 1]));
        if (!E4M3) {
          l[0] += s[n][0] + s[n][1];
          l[1] += s[n][2] + s[n][3];
        }
      }
      // ---- weights . values, 16 keys at a time
      const uint32_t vrow = kw * G::KPW + (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
      for (int n = 0; n < NT; n += 2) {
        if constexpr (E4M3) {
          const uint32_t a[4] = {pack_f16(s[n][0], s[n][1]), pack_f16(s[n][2], s[n][3]),
                                 pack_f16(s[n + 1][0], s[n + 1][1]), pack_f16(s[n + 1][2], s[n + 1][3])};
          mma16816<true>(lsum, a, 0x3C003C00u, 0x3C003C00u);
          // 16 keys by 32 codes; a register holds two codes of each of two keys: element 2u and 2u + 1 of a run of
          // 16, which go to two output tiles
#pragma unroll
          for (int cc = 0; cc < DIM / 32; ++cc) {
            const uint32_t ch = cc * 2 + (lane >> 4);
            uint32_t b[4];
            ldsm4t(vbase + (ch / (G::CW / 16)) * G::SUB + swz<G::CW>(vrow + n * 8, ch % (G::CW / 16)), b);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              uint32_t even[2], odd[2];
#pragma unroll
              for (int k = 0; k < 2; ++k) e4m3x4_f16(__byte_perm(b[2 * u + k], 0, 0x3120), even[k], odd[k]);
              mma16816<true>(o[cc * 4 + 2 * u], a, even[0], even[1]);
              mma16816<true>(o[cc * 4 + 2 * u + 1], a, odd[0], odd[1]);
            }
          }
        } else {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float x = s[n + (u >> 1)][2 * (u & 1)], y = s[n + (u >> 1)][2 * (u & 1) + 1];
            hi[u] = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);  // the upper halves
            lo[u] = low_part(pack_bf16(x - bf16lo_to_f32(hi[u]), y - bf16hi_to_f32(hi[u])), hi[u]);
          }
#pragma unroll
          for (int cc = 0; cc < DIM / 16; ++cc) {
            const uint32_t ch = cc * 2 + (lane >> 4);
            uint32_t b[4];
            ldsm4t(vbase + (ch >> 3) * G::SUB + swz<128>(vrow + n * 8, ch & 7), b);
            mma16816<false>(o[2 * cc], hi, b[0], b[1]);
            mma16816<false>(o[2 * cc + 1], hi, b[2], b[3]);
            mma16816<false>(o[2 * cc], lo, b[0], b[1]);
            mma16816<false>(o[2 * cc + 1], lo, b[2], b[3]);
          }
        }
      }
      if (masked) fence_proxy_async_smem();  // zeroed values, before the next copy into this stage
      __syncwarp();
      if (lane == 0) mbar_arrive(empty(stage));
    }

    // ---- the item's sums: over the quad, then over the warps that shared its keys
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 1);
      l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 2);
      if (E4M3) l[i] = lsum[2 * i];
    }
    constexpr int SLICE = OT / KW;  // output tiles that a warp ends up with
    {
      if (t == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float *x = ml + 2 * (kw * G::ROWS + g + 8 * i);
          x[0] = m[i];
          x[1] = l[i];
        }
      }
      compute_sync();
      float f[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float *x = ml + 2 * (g + 8 * i);
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int k = 0; k < KW; ++k) M = fmaxf(M, x[2 * k * G::ROWS]);
        const float b = M == -INFINITY ? 0.f : M;
#pragma unroll
        for (int k = 0; k < KW; ++k) L += x[2 * k * G::ROWS + 1] * exp2_approx(x[2 * k * G::ROWS] - b);
        f[i] = exp2_approx(m[i] - b);
        m[i] = M;
        l[i] = L;
      }
#pragma unroll
      for (int i = 0; i < OT; ++i) {
        o[i][0] *= f[0];
        o[i][1] *= f[0];
        o[i][2] *= f[1];
        o[i][3] *= f[1];
      }
      // round r: warp kw passes slice (kw + r) % KW on, and takes its own slice from warp (kw - r) % KW
      float4 *buf = reinterpret_cast<float4 *>(smem + G::OFF_Q);
#pragma unroll 1
      for (int r = 1; r < KW; ++r) {
        const int to = (kw + r) % KW;
#pragma unroll
        for (int sl = 0; sl < KW; ++sl)
          if (sl == to) {
#pragma unroll
            for (int i = 0; i < SLICE; ++i) {
              const float(&x)[4] = o[sl * SLICE + i];
              buf[(to * SLICE + i) * 32 + lane] = make_float4(x[0], x[1], x[2], x[3]);
            }
          }
        compute_sync();
#pragma unroll
        for (int sl = 0; sl < KW; ++sl)
          if (sl == kw) {
#pragma unroll
            for (int i = 0; i < SLICE; ++i) {
              const float4 x = buf[(kw * SLICE + i) * 32 + lane];
              float(&y)[4] = o[sl * SLICE + i];
              y[0] += x.x;
              y[1] += x.y;
              y[2] += x.z;
              y[3] += x.w;
            }
          }
        compute_sync();
      }
    }
    const uint32_t odd[2] = {odd_values[0], odd_values[1]};
    const bool whole = sg.whole();
    // slot 0: the item began before this share; slot 1: it goes on after it
    const int slot = sg.kt0 > 0 ? 0 : 1;
    const Partial<DIM, G::ROWS> part(p.partials, blockIdx.x, slot);
    if (tid == 0 && sg.kt0 > 0 && sg.kt1 == sg.ktiles) leave_record<typename G::Tiles>(p, sg, plan.share);
    const float vs = E4M3 ? p.c.v.scale[sg.head] : 1.f;
#pragma unroll
    for (int sl = 0; sl < KW; ++sl) {
      if (sl != kw) continue;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = g + 8 * i;
        if (r >= rows) continue;
        const int rr = sg.rt * G::ROWS + r, tok = sg.i.start + rr / p.group, h = sg.head * p.group + rr % p.group;
        const float inv = l[i] > 0.f || l[i] != l[i] ? vs / l[i] : 0.f;
        uint16_t *out = p.out + ((long long)tok * p.heads + h) * DIM;
#pragma unroll
        for (int n = 0; n < SLICE; n += (E4M3 ? 2 : 1)) {
          // the thread's columns: 8n + 2t, 8n + 2t + 1, or with 8-bit values 4 in a run over two tiles
          constexpr int NC = E4M3 ? 4 : 2;
          const int nt = sl * SLICE + n, d0 = E4M3 ? nt * 8 + 4 * t : nt * 8 + 2 * t;
          float x[NC];
          if constexpr (E4M3) {
            x[0] = o[nt][2 * i];
            x[1] = o[nt + 1][2 * i];
            x[2] = o[nt][2 * i + 1];
            x[3] = o[nt + 1][2 * i + 1];
          } else {
            x[0] = o[nt][2 * i];
            x[1] = o[nt][2 * i + 1];
          }
          if (odd[0] | odd[1]) {
            for (int j = 0; j < sg.i.n; ++j)
              if ((odd[j >> 5] >> (j & 31) & 1) && (word[i] >> j & 1))
#pragma unroll
                for (int e = 0; e < NC; ++e) {
                  const float v = value_at<E4M3>(p, sg.b, sg.head, (long long)sg.i.len + j, d0 + e);
                  if (!(fabsf(v) < INFINITY)) x[e] += v;
                }
          }
          if (whole) {
            if constexpr (E4M3)
              *reinterpret_cast<uint2 *>(out + d0) =
                  make_uint2(pack_bf16(x[0] * inv, x[1] * inv), pack_bf16(x[2] * inv, x[3] * inv));
            else
              *reinterpret_cast<uint32_t *>(out + d0) = pack_bf16(x[0] * inv, x[1] * inv);
          } else if constexpr (E4M3) {
            *reinterpret_cast<float4 *>(part.at(r, d0)) = make_float4(x[0], x[1], x[2], x[3]);
          } else {
            *reinterpret_cast<float2 *>(part.at(r, d0)) = make_float2(x[0], x[1]);
          }
        }
        if (!whole && t == 0 && sl == 0) *part.ml(r) = make_float2(m[i], l[i]);
      }
    }
  }
  if (!ok) {
    *abort_flag = 1;
    if (lane == 0) atomicOr(p.err, kErrTimeout);
  }
}

// ---------------------------------------------------------------------------
// Joining the partials of an item that was split. A block lists the records (a
// scan over one number per CTA) and takes its share of their groups of 8 query
// rows. A warp covers 8 rows by 16 elements, so that its loads are whole
// 128-byte lines of the partials and its stores whole sectors. The weights
// 2^(m_c - M) need maxima and sums alone, so the sums over partials are no
// chain of dependent loads. SPLIT: the block's eight warps share one such
// square's partials (few items, each over many CTAs); otherwise they stand side
// by side along the row. Bound by latency: counts, records, maxima and sums, and
// outputs are loads that wait for one another. (One lane after the other reading
// a row's maxima and sums: one 16-node tree over 8,191 keys 21.1 us, not 18.9;
// five tokens over 131,071 keys 96 and not 91.)
// ---------------------------------------------------------------------------
constexpr int kJoinThreads = 256;

template <int DIM, int ROWS, bool SPLIT>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ AttnParams p, int ctas) {
  constexpr int WARPS = kJoinThreads / 32, SQUARES = DIM / 16;  // squares along a row
  using Part = Partial<DIM, ROWS>;
  __shared__ int ends[kMaxCtas];  // work of records 0 .. c
  __shared__ int rows_of[kMaxCtas];
  __shared__ int4 records[kMaxCtas];
  __shared__ int sums[WARPS];
  __shared__ float4 acc[SPLIT ? WARPS : 1][32];
  grid_dependency_wait();
  grid_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int total = 0;
  for (int c0 = 0; c0 < ctas; c0 += kJoinThreads) {
    int v = 0;
    if (c0 + tid < ctas) {
      records[c0 + tid] = reinterpret_cast<const int4 *>(p.joins + kMaxCtas)[c0 + tid];  // (without rows: never looked at)
      rows_of[c0 + tid] = p.joins[c0 + tid];
      v = (rows_of[c0 + tid] + 7) / 8 * (SPLIT ? SQUARES : 1);
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, v, d);
      if (lane >= d) v += o;
    }
    if (lane == 31) sums[warp] = v;
    __syncthreads();
    int before = total;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      if (w < warp) before += sums[w];
      total += sums[w];
    }
    if (c0 + tid < ctas) ends[c0 + tid] = before + v;
    __syncthreads();
  }
  for (int e = blockIdx.x; e < total; e += gridDim.x) {  // (the whole block goes round together)
    int c1 = 0;
    for (int hi = ctas; c1 < hi;) {
      const int mid = (c1 + hi) >> 1;
      if (ends[mid] > e) hi = mid;
      else c1 = mid + 1;
    }
    const int local = e - (c1 ? ends[c1 - 1] : 0);
    const int4 rec = records[c1];
    const int rows = rows_of[c1], c0 = rec.x, n = c1 - c0 + 1;
    const int r0 = (SPLIT ? local / SQUARES : local) * 8 + (lane & 7), r = min(r0, rows - 1);
    // the first CTA ended its share inside the item (slot 1), the others began theirs in it (slot 0)
    auto part = [&](int c) { return Part(p.partials, c0 + c, c == 0 ? 1 : 0); };
    // maximum and sum: the four lanes of a row take the partials in turn, eight loads in flight
    float M = -INFINITY, L = 0.f;
    auto add = [&](float m, float l) {
      const float top = fmaxf(M, m), b = top == -INFINITY ? 0.f : top;
      L = L * exp2_approx(M - b) + l * exp2_approx(m - b);
      M = top;
    };
    for (int k = lane >> 3; k < n; k += 32) {
      float2 ml[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) ml[u] = k + 4 * u < n ? *part(k + 4 * u).ml(r) : make_float2(-INFINITY, 0.f);
      float top = ml[0].x;
#pragma unroll
      for (int u = 1; u < 8; ++u) top = fmaxf(top, ml[u].x);
      const float b = top == -INFINITY ? 0.f : top;
      float l = 0.f;
#pragma unroll
      for (int u = 0; u < 8; ++u) l += ml[u].y * exp2_approx(ml[u].x - b);
      add(top, l);
    }
#pragma unroll
    for (int d = 8; d < 32; d <<= 1) add(__shfl_xor_sync(0xFFFFFFFFu, M, d), __shfl_xor_sync(0xFFFFFFFFu, L, d));
    const float base = M == -INFINITY ? 0.f : M;
    const float inv = (L > 0.f || L != L) ? (p.c.e4m3 ? p.c.v.scale[rec.w] : 1.f) / L : 0.f;
    const int rr = rec.z + r, tok = rec.y + rr / p.group;
    uint16_t *out = p.out + ((long long)tok * p.heads + rec.w * p.group + rr % p.group) * DIM;
    for (int sq = SPLIT ? local % SQUARES : warp; sq < SQUARES; sq += SPLIT ? SQUARES : WARPS) {
      const int d = sq * 16 + (lane >> 3) * 4;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int c = SPLIT ? warp : 0; c < n; c += SPLIT ? WARPS : 1) {
        const Part s = part(c);
        const float w = exp2_approx(s.ml(r)->x - base);
        const float4 y = *reinterpret_cast<const float4 *>(s.at(r, d));
        x.x = fmaf(w, y.x, x.x);
        x.y = fmaf(w, y.y, x.y);
        x.z = fmaf(w, y.z, x.z);
        x.w = fmaf(w, y.w, x.w);
      }
      if constexpr (SPLIT) {
        acc[warp][lane] = x;
        __syncthreads();
        if (warp == 0) {
#pragma unroll
          for (int w = 1; w < WARPS; ++w) {
            const float4 y = acc[w][lane];
            x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
          }
        }
      }
      if (r0 < rows && (!SPLIT || warp == 0))
        *reinterpret_cast<uint2 *>(out + d) = make_uint2(pack_bf16(x.x * inv, x.y * inv), pack_bf16(x.z * inv, x.w * inv));
      if (SPLIT) __syncthreads();
    }
  }
}

// ---------------------------------------------------------------------------
// launch
// ---------------------------------------------------------------------------
constexpr size_t kJoinBytes = ((size_t)kMaxCtas * 5 * sizeof(int) + 255) / 256 * 256;

template <int DIM, int ROWS>
cudaError_t launch_join(const AttnCall &c, const AttnParams &p, int ctas) {
  // Few items: each is split over many CTAs, so a block's warps share the partials of a square
  const long long items = (long long)c.rows.rows * c.cache.kv_heads * ((c.max_tree * p.group + ROWS - 1) / ROWS);
  // at most one record per CTA and per item
  const long long groups = std::min((long long)ctas, items) * ((std::min(ROWS, c.max_tree * p.group) + 7) / 8);
  const bool split = items * 8 <= ctas;
  const unsigned grid = (unsigned)std::min(groups * (split ? DIM / 16 : 1), 8LL * c.sm_count);
  return split ? launch_dependent(join_kernel<DIM, ROWS, true>, grid, kJoinThreads, 0, c.stream, p, ctas)
               : launch_dependent(join_kernel<DIM, ROWS, false>, grid, kJoinThreads, 0, c.stream, p, ctas);
}

template <int DIM, bool E4M3>
cudaError_t launch_rows(const AttnCall &c, AttnParams &p) {
  using G = RowsGeo<DIM, E4M3>;
  auto kern = rows_kernel<DIM, E4M3>;
  static PerDevice configured;
  if (!configured.v[c.device].load(std::memory_order_relaxed)) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, G::SMEM);
    if (e != cudaSuccess) return e;
    configured.v[c.device].store(1, std::memory_order_relaxed);
  }
  CUtensorMap tk, tv;
  const int br = std::min(c.cache.page_rows, G::KT);
  if (!encode_cache(&tk, c.cache.k, c.cache, br, G::CW, true) || !encode_cache(&tv, c.cache.v, c.cache, br, G::CW, true))
    return cudaErrorInvalidValue;
  const int grid = std::min(G::CTAS * c.sm_count, kMaxCtas);
  cudaError_t e = launch_dependent(kern, grid, kThreads, G::SMEM, c.stream, tk, tv, p);
  if (e != cudaSuccess) return e;
  return p.whole ? cudaSuccess : launch_join<DIM, G::ROWS>(c, p, grid);
}

template <int DIM, bool E4M3>
cudaError_t launch_tc(const AttnCall &c, AttnParams &p) {
  cudaError_t e = launch_tree_tc(c, p);
  if (e != cudaSuccess) return e;
  return p.whole ? cudaSuccess : launch_join<DIM, tc_attn_rows(DIM, E4M3)>(c, p, std::min(c.sm_count, kTcMaxCtas));
}
// The tcgen05 kernel from 17 query rows per kv head on: its MMAs take 128 rows
// in the time of one. (When this file still had 32- and 64-row forms: 16
// sequences of 32 rows 63 us here, 55 there; 64 rows 121 and 57; 8-bit caches
// 77 and 61, 133 and 64.)
bool uses_tc(int rows) { return rows > 16; }

template <int DIM, bool E4M3>
cudaError_t launch_dim(const AttnCall &c, AttnParams &p) {
  return uses_tc(c.max_tree * p.group) ? launch_tc<DIM, E4M3>(c, p) : launch_rows<DIM, E4M3>(c, p);
}

}  // namespace

bool encode_cache(CUtensorMap *m, const KvSide &s, const KvCache &c, int box_rows, int box_bytes, bool swizzled) {
  const int elt = c.e4m3 ? 1 : 2;
  // an axis of one entry is never stepped along; its stride only has to be one that a map may have
  auto step = [&](int n, long long stride) { return (uint64_t)(n > 1 ? stride : c.row_bytes()); };
  const uint64_t dims[4] = {(uint64_t)c.dim, (uint64_t)c.page_rows, (uint64_t)c.kv_heads, (uint64_t)c.pages};
  const uint64_t strides[3] = {step(c.page_rows, s.row), step(c.kv_heads, s.head), step(c.pages, s.page)};
  const uint32_t box[4] = {(uint32_t)(box_bytes / elt), (uint32_t)box_rows, 1, 1};
  return encode_4d(m, c.e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, s.base, dims, strides,
                   box, !swizzled          ? CU_TENSOR_MAP_SWIZZLE_NONE
                         : box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                            : CU_TENSOR_MAP_SWIZZLE_64B);
}

size_t tree_attn_workspace_bytes(int heads, int kv_heads, int dim, int max_tree) {
  const int rows = max_tree * (heads / kv_heads);
  if (uses_tc(rows))  // (an 8-bit cache needs no more)
    return kJoinBytes + align_up((size_t)kTcMaxCtas * 2 * tc_attn_rows(dim, false) * (dim + 2) * sizeof(float), 256);
  return kJoinBytes + align_up((size_t)kMaxCtas * 2 * 16 * (dim + 2) * sizeof(float), 256);
}

cudaError_t launch_tree_attention(const AttnCall &c) {
  AttnParams p;
  p.q = c.q;
  p.q_token = c.q_token;
  p.q_head = c.q_head;
  p.c = c.cache;
  p.r = c.rows;
  p.mask = c.mask;
  p.heads = c.heads;
  p.group = c.heads / c.cache.kv_heads;
  p.max_tree = c.max_tree;
  p.whole = (long long)c.rows.max_pages * c.cache.page_rows <= (uses_tc(c.max_tree * p.group) ? kTcWholeKeys : kWholeKeys);
  p.scale_log2 = c.scale * kLog2e;
  p.out = c.out;
  p.joins = static_cast<int *>(c.workspace);
  p.partials = reinterpret_cast<float *>(static_cast<uint8_t *>(c.workspace) + kJoinBytes);
  p.err = c.err;
  switch (c.cache.dim) {
    case 64: return c.cache.e4m3 ? launch_dim<64, true>(c, p) : launch_dim<64, false>(c, p);
    case 128: return c.cache.e4m3 ? launch_dim<128, true>(c, p) : launch_dim<128, false>(c, p);
    default: return c.cache.e4m3 ? launch_dim<256, true>(c, p) : launch_dim<256, false>(c, p);
  }
}

}  // namespace w4a16
