// Attention of drafted tokens over a paged key/value cache.
//
//   s_j = scale * q . k_j,  out = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m)
//
// over the positions j that the token sees (its row's context and, by its
// mask word, the row's new tokens). One pass: a running maximum m and sum, the
// sums rescaled when m grows.
#include <cuda_fp8.h>

#include "w4a16_internal.h"

namespace w4a16 {
namespace {

constexpr int kThreads = 128;

struct SimpleParams {
  const uint16_t *q;
  long long q_token, q_head;
  KvCache c;
  KvRows r;
  const int64_t *mask;
  int heads, group, max_tree;
  float scale;
  uint16_t *out;
  int *err;
};

template <bool E4M3, int N>
__device__ __forceinline__ void load_row(const uint8_t *p, float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    if (E4M3) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(*reinterpret_cast<const uint16_t *>(p + i), __NV_E4M3);
      x[i] = __half2float(__half(__half_raw{h.x}));
      x[i + 1] = __half2float(__half(__half_raw{h.y}));
    } else {
      const uint32_t w = *reinterpret_cast<const uint32_t *>(p + 2 * i);
      x[i] = bf16lo_to_f32(w);
      x[i + 1] = bf16hi_to_f32(w);
    }
  }
}

// One CTA per (token, head), keys dealt to its warps; a lane holds DIM / 32
// consecutive elements.
template <int DIM, bool E4M3>
__global__ void __launch_bounds__(kThreads) simple_kernel(const SimpleParams p) {
  constexpr int N = DIM / 32, W = kThreads / 32;
  __shared__ float sm[W], sl[W], so[W][DIM];
  const int t = blockIdx.x, h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int b = 0;
  for (int hi = p.r.rows; b < hi;) {
    const int mid = (b + hi) >> 1;
    if (p.r.starts[mid + 1] > t) hi = mid;
    else b = mid + 1;
  }
  if (b >= p.r.rows) return;  // padding
  const int s0 = p.r.starts[b], n = p.r.starts[b + 1] - s0, len = p.r.lengths[b], i = t - s0;
  if (s0 < 0 || i < 0 || n > p.max_tree || len < 0) {
    if (threadIdx.x == 0) atomicOr(p.err, kErrIndex);
    return;
  }
  const unsigned long long word = p.mask ? (unsigned long long)p.mask[t] : (2ull << i) - 1;
  const int kh = h / p.group;
  float q[N], o[N], m = -INFINITY, l = 0.f;
  load_row<false>(reinterpret_cast<const uint8_t *>(p.q + t * p.q_token + h * p.q_head + lane * N), q);
#pragma unroll
  for (int e = 0; e < N; ++e) o[e] = 0.f;
  const float ks = E4M3 ? p.c.k.scale[kh] : 1.f, vs = E4M3 ? p.c.v.scale[kh] : 1.f;
  for (long long j = warp; j < (long long)len + n; j += W) {
    if (j >= len && !((word >> (j - len)) & 1)) continue;
    const long long pi = j >> p.c.page_shift;
    const int id = pi < p.r.max_pages ? p.r.table[(long long)b * p.r.max_pages + pi] : -1;
    if ((unsigned)id >= (unsigned)p.c.pages) {
      if (lane == 0) atomicOr(p.err, kErrIndex);
      continue;
    }
    const long long row = j & (p.c.page_rows - 1);
    float k[N], v[N], s = 0.f;
    load_row<E4M3>(p.c.k.base + id * p.c.k.page + kh * p.c.k.head + row * p.c.k.row + lane * N * (E4M3 ? 1 : 2), k);
    load_row<E4M3>(p.c.v.base + id * p.c.v.page + kh * p.c.v.head + row * p.c.v.row + lane * N * (E4M3 ? 1 : 2), v);
#pragma unroll
    for (int e = 0; e < N; ++e) s = fmaf(q[e], k[e], s);
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    s *= p.scale * ks;
    const float mn = fmaxf(m, s), a = __expf(m - mn), w = __expf(s - mn);
    l = l * a + w;
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] = fmaf(w, v[e], o[e] * a);
    m = mn;
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < N; ++e) so[warp][lane * N + e] = o[e];
  __syncthreads();
  float M = -INFINITY, L = 0.f;
  for (int w = 0; w < W; ++w) M = fmaxf(M, sm[w]);
  for (int w = 0; w < W; ++w) L += M == -INFINITY ? 0.f : sl[w] * __expf(sm[w] - M);
  for (int d = threadIdx.x; d < DIM; d += kThreads) {
    float x = 0.f;
    for (int w = 0; w < W; ++w) x += M == -INFINITY ? 0.f : so[w][d] * __expf(sm[w] - M);
    const __nv_bfloat16 y = __float2bfloat16_rn(L > 0.f ? x / L * vs : 0.f);
    p.out[((long long)t * p.heads + h) * DIM + d] = *reinterpret_cast<const uint16_t *>(&y);
  }
}

template <int DIM, bool E4M3>
cudaError_t run_simple(const AttnCall &c) {
  SimpleParams p{c.q, c.q_token, c.q_head, c.cache, c.rows, c.mask, c.heads, c.heads / c.cache.kv_heads,
                 c.max_tree, c.scale, c.out, c.err};
  simple_kernel<DIM, E4M3><<<dim3(c.rows.tokens, c.heads), kThreads, 0, c.stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

size_t tree_attn_workspace_bytes(int heads, int kv_heads, int dim, int max_tree) { return 256; }

cudaError_t launch_tree_attention(const AttnCall &c) {
  switch (c.cache.dim) {
    case 64: return c.cache.e4m3 ? run_simple<64, true>(c) : run_simple<64, false>(c);
    case 128: return c.cache.e4m3 ? run_simple<128, true>(c) : run_simple<128, false>(c);
    default: return c.cache.e4m3 ? run_simple<256, true>(c) : run_simple<256, false>(c);
  }
}

}  // namespace w4a16
