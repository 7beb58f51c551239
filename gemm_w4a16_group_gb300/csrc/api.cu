// C ABI (include/w4a16.h): argument checks, device checks and kernel choice.
// Nothing is launched when a check fails; every check that needs no GPU runs
// before the first CUDA call.
#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstdio>
#include <mutex>
#include <utility>

#include "w4a16.h"
#include "w4a16_internal.h"

using namespace w4a16;

namespace {

thread_local int t_last_cuda_error = 0;
std::atomic<int> g_override{0};
std::atomic<int> g_overlap{0};

// Device error word set by kernels whose bounded waits gave up.
__device__ int g_kernel_error;

// Fixed table of x group sums for w4a16_gemm_affine_noalloc (4 MiB per device,
// part of the module image: nothing is allocated at run time).
constexpr size_t kNoAllocXsumBytes = size_t(4) << 20;
static __device__ __align__(256) uint16_t g_noalloc_xsum[kNoAllocXsumBytes / sizeof(uint16_t)];

struct DeviceInfo {
  int device = 0;
  bool ready = false;
  int status = W4A16_OK;
  int sm_count = 0;
  int *err = nullptr;
  uint16_t *noalloc_xsum = nullptr;  // this device's copy of g_noalloc_xsum
};
DeviceInfo g_dev[kMaxDevices];
std::mutex g_dev_mu;

int cuda_fail(cudaError_t e) {
  t_last_cuda_error = (int)e;
  return W4A16_ERR_CUDA;
}

// Current device's properties and error-word address (looked up once per device).
int current_device(DeviceInfo &out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  if (dev < 0 || dev >= kMaxDevices) return W4A16_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lk(g_dev_mu);
  DeviceInfo &d = g_dev[dev];
  if (!d.ready) {
    int major = 0, minor = 0, sms = 0;
    if ((e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
      return cuda_fail(e);
    if (major != 10 || minor != 3) {
      d.status = W4A16_ERR_UNSUPPORTED;  // the kernels are built for sm_103a only
    } else {
      void *p = nullptr;
      if ((e = cudaGetSymbolAddress(&p, g_kernel_error)) != cudaSuccess) return cuda_fail(e);
      d.err = static_cast<int *>(p);
      if ((e = cudaGetSymbolAddress(&p, g_noalloc_xsum)) != cudaSuccess) return cuda_fail(e);
      d.noalloc_xsum = static_cast<uint16_t *>(p);
      d.sm_count = sms;
      d.status = W4A16_OK;
    }
    d.device = dev;
    d.ready = true;
  }
  out = d;
  return d.status;
}

bool sizes_ok(long long M, long long N, long long K, int group) {
  const long long lim = (1LL << 31) / 16;
  if (group != 64 && group != 128) return false;
  if (M < 1 || N < 1 || K < 64 || M >= lim || N >= lim || K >= lim) return false;
  return K % group == 0;
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int finish_launch(cudaError_t e) { return e == cudaSuccess ? W4A16_OK : cuda_fail(e); }

// The kernel override is read once per call (`ov`, from g_override) and that
// value decides both the argument checks and the launch, so a concurrent
// w4a16_set_kernel_override cannot send a call the checks did not accept.

// The decode kernels (M <= 32): override 2 keeps the per-warp-ring kernel, override 4
// forces the x-staged one, otherwise the x-staged kernel takes M <= 8 calls
// whose grid fills a wave and 9-16-row zero-point calls on grids of at least
// 1.5 CTAs per SM (launch_smallm_mma)
cudaError_t launch_decode_kernel(GemmCall &c, int sm_count, int ov) {
  c.xs_mode = ov == 4 ? 2 : ov == 2 ? 0 : 1;
  return launch_smallm_mma(c, sm_count);
}

// Rows that go to a decode kernel rather than the tcgen05 GEMM: M <= 32
// (graph-timed at N = 34816, K = 5120: M = 17-24 36.5 us against 66.8 on the
// tcgen05 GEMM, M = 32 47.6 against 66.8; 3.7-4.9x at N = 5120, where the
// GEMM has few tiles), unless the tcgen05 GEMM is forced (override 3)
constexpr int kDecodeMaxM = 32;
bool use_decode(int M, int ov) { return M <= kDecodeMaxM && ov != 3; }

bool form_ok(int form) { return form == kFormZero || form == kFormSym || form == kFormAffine; }
bool zero_form(int form) { return form == kFormZero || form == kFormSym; }

// The affine calls: the decode kernel for M <= 32 (it forms the x group sums
// itself), else the tcgen05 GEMM, which reads them from `xsum`.
bool affine_uses_tc(int M, int ov) { return !use_decode(M, ov); }

int launch_affine(GemmCall &c, const uint16_t *xsum, const DeviceInfo &d, int ov) {
  if (!affine_uses_tc(c.M, ov)) return finish_launch(launch_decode_kernel(c, d.sm_count, ov));
  c.xsum = xsum;
  return finish_launch(launch_prompt_tc(c, d.sm_count));
}

// b-bit affine weights: 2-4 bits widened into nibbles, 5-8 bits in two
// nibble planes over K' = 2K (x's groups each written twice)
bool bits_ok(int bits) { return bits >= 2 && bits <= 8; }
int bits_planes(int bits) { return bits > 4 ? 2 : 1; }
size_t widened_x_bytes(int M, int K, int bits) {
  return bits > 4 ? align_up((size_t)M * 2 * (size_t)K * sizeof(uint16_t), 256) : 0;
}

// rows of a gate/up buffer (each weight padded to 128 rows), or -1 if too many
long long gateup_rows(int N_each) {
  const long long rows = 2LL * ((N_each + 127) / 128 * 128);
  return rows >= (1LL << 31) / 16 ? -1 : rows;
}

// ---- paged cache calls ----
bool rows_ok(int rows, int max_pages) { return rows >= 1 && rows <= W4A16_MAX_SEQUENCES && max_pages >= 1; }
bool tokens_ok(long long tokens) { return tokens >= 1 && tokens < (1LL << 31) / 16; }
bool stride_ok(int64_t elements, int elt) { return elements >= 0 && elements * elt % 16 == 0; }

int page_shift_of(int page_rows) {
  for (int s = 4; s <= 8; ++s)
    if (page_rows == 1 << s) return s;
  return -1;
}

// ---- adapters ----
bool lora_sizes_ok(int rank, int inner) {
  return rank >= 8 && rank <= W4A16_MAX_RANK && rank % 8 == 0 && tokens_ok(inner) && inner % 8 == 0;
}

// Rows of `n` elements read at y and written at out: the same ones, or none
// in common (other buffers, or other columns of one). Rows whose strides
// differ must not lie in one range.
bool rows_apart(const uint16_t *y, int64_t y_row, const uint16_t *out, int64_t out_row, int tokens, int n) {
  const int64_t lim = int64_t(1) << 40;
  if (y_row >= lim || out_row >= lim) return false;
  const int64_t d = (reinterpret_cast<intptr_t>(out) - reinterpret_cast<intptr_t>(y)) / 2;
  if (d == 0 && (y_row == out_row || tokens == 1)) return true;
  if (d >= y_row * (tokens - 1) + n || -d >= out_row * (tokens - 1) + n) return true;
  if (y_row != out_row || y_row == 0) return false;
  const int64_t at = (d % y_row + y_row) % y_row;
  return at >= n && y_row - at >= n;
}

// No two elements of one side share an address: taken by ascending stride,
// each dimension steps past all that the smaller ones cover.
bool side_disjoint(int64_t dim, int64_t row, int64_t rows, int64_t head, int64_t heads, int64_t page, int64_t pages,
                   int64_t layer, int64_t layers) {
  std::pair<int64_t, int64_t> d[4] = {{row, rows}, {head, heads}, {page, pages}, {layer, layers}};
  std::sort(d, d + 4);
  int64_t extent = dim;
  for (const auto &x : d) {
    if (x.second == 1) continue;
    if (x.first < extent || x.first > (int64_t(1) << 60) / x.second) return false;
    extent += x.first * (x.second - 1);
  }
  return true;
}

// The checked form of a cache, strides in bytes; W4A16_OK or an error code.
// `values`: the call computes with the values (one layer, and scales for 8 bits); otherwise it moves rows.
int check_cache(const w4a16_kv_cache *c, bool values, KvCache &out) {
  if (!c || !c->k || !c->v) return W4A16_ERR_INVALID_ARG;
  if (c->type != W4A16_KV_BF16 && c->type != W4A16_KV_E4M3) return W4A16_ERR_INVALID_ARG;
  const bool e4m3 = c->type == W4A16_KV_E4M3;
  if (values && (e4m3 ? !c->k_scale || !c->v_scale : c->k_scale || c->v_scale)) return W4A16_ERR_INVALID_ARG;
  if (values && c->layers != 1) return W4A16_ERR_INVALID_ARG;
  if (c->layers < 1 || c->pages < 1 || c->kv_heads < 1 || c->kv_heads > 1024) return W4A16_ERR_INVALID_ARG;
  if (c->dim != 64 && c->dim != 128 && c->dim != 256) return W4A16_ERR_INVALID_ARG;
  const int shift = page_shift_of(c->page_rows);
  if (shift < 0) return W4A16_ERR_INVALID_ARG;
  const int elt = e4m3 ? 1 : 2;
  const int64_t strides[] = {c->k_layer, c->k_page, c->k_head, c->k_row, c->v_layer, c->v_page, c->v_head, c->v_row};
  for (int64_t s : strides)
    if (s < 0) return W4A16_ERR_INVALID_ARG;
  if (!side_disjoint(c->dim, c->k_row, c->page_rows, c->k_head, c->kv_heads, c->k_page, c->pages, c->k_layer, c->layers) ||
      !side_disjoint(c->dim, c->v_row, c->page_rows, c->v_head, c->kv_heads, c->v_page, c->pages, c->v_layer, c->layers))
    return W4A16_ERR_INVALID_ARG;
  for (int64_t s : strides)
    if (!stride_ok(s, elt)) return W4A16_ERR_MISALIGNED;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
    return W4A16_ERR_MISALIGNED;
  out.k = KvSide{static_cast<uint8_t *>(c->k), c->k_scale, c->k_layer * elt, c->k_page * elt, c->k_head * elt,
                 c->k_row * elt};
  out.v = KvSide{static_cast<uint8_t *>(c->v), c->v_scale, c->v_layer * elt, c->v_page * elt, c->v_head * elt,
                 c->v_row * elt};
  out.layers = c->layers;
  out.pages = c->pages;
  out.kv_heads = c->kv_heads;
  out.page_rows = c->page_rows;
  out.page_shift = shift;
  out.dim = c->dim;
  out.e4m3 = e4m3;
  return W4A16_OK;
}

bool attn_sizes_ok(int heads, int kv_heads, int dim, int max_tree) {
  return (dim == 64 || dim == 128 || dim == 256) && kv_heads >= 1 && kv_heads <= 1024 && heads >= kv_heads &&
         heads <= 65535 && heads % kv_heads == 0 && max_tree >= 1 && max_tree <= W4A16_MAX_TREE;
}

}  // namespace

extern "C" {

size_t w4a16_repacked_bytes(int N, int K, int group, int sym) {
  if (!sizes_ok(1, N, K, group) || !form_ok(sym)) return 0;
  return make_layout(N, K, group, sym).total;
}

size_t w4a16_gateup_repacked_bytes(int N_each, int K, int group, int sym) {
  if (!sizes_ok(1, N_each, K, group) || !form_ok(sym)) return 0;
  const long long rows = gateup_rows(N_each);
  if (rows < 0) return 0;
  return make_layout((int)rows, K, group, sym).total;
}

int w4a16_repack(const int32_t *qweight, const uint16_t *scales, const int32_t *zeros, int N, int K,
                 int group, int sym, void *packed, w4a16_stream_t stream) {
  if (sym != kFormZero && sym != kFormSym) return W4A16_ERR_INVALID_ARG;
  if (!qweight || !scales || !packed || (!sym && !zeros)) return W4A16_ERR_INVALID_ARG;
  if (!sizes_ok(1, N, K, group)) return W4A16_ERR_INVALID_ARG;
  if (!aligned(packed, 256) || !aligned(qweight, 4) || !aligned(scales, 2) || (zeros && !aligned(zeros, 4)))
    return W4A16_ERR_MISALIGNED;
  DeviceInfo d;
  int st = current_device(d);
  if (st != W4A16_OK) return st;
  const Layout L = make_layout(N, K, group, sym);
  return finish_launch(launch_repack(qweight, scales, sym ? nullptr : zeros, nullptr, nullptr, nullptr, nullptr,
                                     nullptr, N, false, L, static_cast<uint8_t *>(packed),
                                     reinterpret_cast<cudaStream_t>(stream)));
}

int w4a16_repack_affine(const int32_t *qweight, const uint16_t *scales, const uint16_t *biases, int N, int K,
                        int group, void *packed, w4a16_stream_t stream) {
  if (!qweight || !scales || !biases || !packed) return W4A16_ERR_INVALID_ARG;
  if (!sizes_ok(1, N, K, group)) return W4A16_ERR_INVALID_ARG;
  if (!aligned(packed, 256) || !aligned(qweight, 4) || !aligned(scales, 2) || !aligned(biases, 2))
    return W4A16_ERR_MISALIGNED;
  DeviceInfo d;
  int st = current_device(d);
  if (st != W4A16_OK) return st;
  const Layout L = make_layout(N, K, group, kFormAffine);
  return finish_launch(launch_repack(qweight, scales, nullptr, biases, nullptr, nullptr, nullptr, nullptr, N,
                                     false, L, static_cast<uint8_t *>(packed),
                                     reinterpret_cast<cudaStream_t>(stream)));
}

int w4a16_repack_affine_gateup(const int32_t *qw_gate, const uint16_t *sc_gate, const uint16_t *b_gate,
                               const int32_t *qw_up, const uint16_t *sc_up, const uint16_t *b_up, int N_each,
                               int K, int group, void *packed, w4a16_stream_t stream) {
  if (!qw_gate || !sc_gate || !b_gate || !qw_up || !sc_up || !b_up || !packed) return W4A16_ERR_INVALID_ARG;
  if (w4a16_gateup_repacked_bytes(N_each, K, group, kFormAffine) == 0) return W4A16_ERR_INVALID_ARG;
  if (!aligned(packed, 256) || !aligned(qw_gate, 4) || !aligned(qw_up, 4) || !aligned(sc_gate, 2) ||
      !aligned(sc_up, 2) || !aligned(b_gate, 2) || !aligned(b_up, 2))
    return W4A16_ERR_MISALIGNED;
  DeviceInfo d;
  int st = current_device(d);
  if (st != W4A16_OK) return st;
  const Layout L = make_layout((int)gateup_rows(N_each), K, group, kFormAffine);
  return finish_launch(launch_repack(qw_gate, sc_gate, nullptr, b_gate, qw_up, sc_up, nullptr, b_up, N_each, true,
                                     L, static_cast<uint8_t *>(packed), reinterpret_cast<cudaStream_t>(stream)));
}

int w4a16_repack_gateup(const int32_t *qw_gate, const uint16_t *sc_gate, const int32_t *z_gate,
                        const int32_t *qw_up, const uint16_t *sc_up, const int32_t *z_up, int N_each, int K,
                        int group, int sym, void *packed, w4a16_stream_t stream) {
  if (sym != kFormZero && sym != kFormSym) return W4A16_ERR_INVALID_ARG;
  if (!qw_gate || !sc_gate || !qw_up || !sc_up || !packed) return W4A16_ERR_INVALID_ARG;
  if (!sym && (!z_gate || !z_up)) return W4A16_ERR_INVALID_ARG;
  if (w4a16_gateup_repacked_bytes(N_each, K, group, sym) == 0) return W4A16_ERR_INVALID_ARG;
  if (!aligned(packed, 256) || !aligned(qw_gate, 4) || !aligned(qw_up, 4) || !aligned(sc_gate, 2) ||
      !aligned(sc_up, 2) || (z_gate && !aligned(z_gate, 4)) || (z_up && !aligned(z_up, 4)))
    return W4A16_ERR_MISALIGNED;
  DeviceInfo d;
  int st = current_device(d);
  if (st != W4A16_OK) return st;
  const Layout L = make_layout((int)gateup_rows(N_each), K, group, sym);
  return finish_launch(launch_repack(qw_gate, sc_gate, sym ? nullptr : z_gate, nullptr, qw_up, sc_up,
                                     sym ? nullptr : z_up, nullptr, N_each, true, L,
                                     static_cast<uint8_t *>(packed), reinterpret_cast<cudaStream_t>(stream)));
}

int w4a16_gemm(const uint16_t *x, const void *packed, const uint16_t *scales, const int32_t *zeros, int M,
               int N, int K, int group, int sym, uint16_t *y, w4a16_stream_t stream) {
  const int ov = g_override.load();
  if (!x || !packed || !y) return W4A16_ERR_INVALID_ARG;
  if (scales || zeros) return W4A16_ERR_INVALID_ARG;  // reserved: they travel inside `packed`
  if (!sizes_ok(M, N, K, group) || !zero_form(sym)) return W4A16_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(packed, 256)) return W4A16_ERR_MISALIGNED;
  DeviceInfo d;
  int st = current_device(d);
  if (st != W4A16_OK) return st;
  GemmCall c{x, static_cast<const uint8_t *>(packed), y, M, N, K, group, sym, false,
             reinterpret_cast<cudaStream_t>(stream), d.err, d.device, g_overlap.load() != 0};
  // M <= 32: a tensor-core decode kernel (measured faster than the CUDA-core
  // GEMV at M = 1 on every decode shape); the GEMV stays selectable.
  if (M == 1 && ov == 1) return finish_launch(launch_gemv_m1(c, d.sm_count));
  if (ov == 5 && smallm_tc_supports(c)) return finish_launch(launch_smallm_tc(c, d.sm_count));
  if (use_decode(M, ov)) return finish_launch(launch_decode_kernel(c, d.sm_count, ov));
  return finish_launch(launch_prompt_tc(c, d.sm_count));
}

int w4a16_gateup_silu(const uint16_t *x, const void *packed_gateup, int M, int N_each, int K, int group,
                      int sym, uint16_t *h, w4a16_stream_t stream) {
  const int ov = g_override.load();
  if (!x || !packed_gateup || !h) return W4A16_ERR_INVALID_ARG;
  if (!sizes_ok(M, N_each, K, group) || !zero_form(sym) || w4a16_gateup_repacked_bytes(N_each, K, group, sym) == 0)
    return W4A16_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(h, 16) || !aligned(packed_gateup, 256)) return W4A16_ERR_MISALIGNED;
  DeviceInfo d;
  int st = current_device(d);
  if (st != W4A16_OK) return st;
  GemmCall c{x, static_cast<const uint8_t *>(packed_gateup), h, M, N_each, K, group, sym, true,
             reinterpret_cast<cudaStream_t>(stream), d.err, d.device, g_overlap.load() != 0};
  if (use_decode(M, ov)) return finish_launch(launch_decode_kernel(c, d.sm_count, ov));
  return finish_launch(launch_prompt_tc(c, d.sm_count));
}

int w4a16_gemm_argmax(const uint16_t *x, const void *packed, int M, int N, int K, int group, int sym,
                      uint16_t *y, int64_t *argmax, w4a16_stream_t stream) {
  const int ov = g_override.load();
  const bool decode = use_decode(M, ov);
  if (!x || !packed || !argmax) return W4A16_ERR_INVALID_ARG;
  if (!sizes_ok(M, N, K, group) || !zero_form(sym) || (!decode && !y)) return W4A16_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(packed, 256) || !aligned(argmax, 8))
    return W4A16_ERR_MISALIGNED;
  DeviceInfo d;
  int st = current_device(d);
  if (st != W4A16_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool overlap = g_overlap.load() != 0;
  cudaError_t e = launch_argmax_init(argmax, M, overlap, s);
  if (e != cudaSuccess) return cuda_fail(e);
  GemmCall c{x, static_cast<const uint8_t *>(packed), y, M, N, K, group, sym, false, s, d.err, d.device, overlap};
  if (decode) {
    c.amax = argmax;  // keys from the decode kernel's epilogue; y may be NULL
    e = launch_decode_kernel(c, d.sm_count, ov);
  } else {
    e = launch_prompt_tc(c, d.sm_count);
    if (e == cudaSuccess) e = launch_row_argmax(y, M, N, argmax, s);
  }
  if (e == cudaSuccess) e = launch_argmax_finalize(argmax, M, overlap, s);
  return finish_launch(e);
}

int w4a16_topk(const uint16_t *y, int M, int N, int k, int64_t *idx, uint16_t *vals, w4a16_stream_t stream) {
  if (!y || !idx) return W4A16_ERR_INVALID_ARG;
  if (!sizes_ok(M, N, 64, 64) || k < 1 || k > N || k > kTopkMaxK) return W4A16_ERR_INVALID_ARG;
  if (!aligned(y, 2) || !aligned(idx, 8) || !aligned(vals, 2)) return W4A16_ERR_MISALIGNED;
  DeviceInfo d;
  int st = current_device(d);
  if (st != W4A16_OK) return st;
  return finish_launch(launch_topk(y, M, N, k, idx, vals, g_overlap.load() != 0, d.device,
                                   reinterpret_cast<cudaStream_t>(stream)));
}

int w4a16_gemm_topk(const uint16_t *x, const void *packed, int M, int N, int K, int group, int sym, int k,
                    uint16_t *y, int64_t *idx, uint16_t *vals, w4a16_stream_t stream) {
  if (k < 1 || k > N || k > kTopkMaxK || !idx) return W4A16_ERR_INVALID_ARG;
  if (!aligned(idx, 8) || !aligned(vals, 2)) return W4A16_ERR_MISALIGNED;
  const int st = w4a16_gemm(x, packed, nullptr, nullptr, M, N, K, group, sym, y, stream);
  if (st != W4A16_OK) return st;
  return w4a16_topk(y, M, N, k, idx, vals, stream);
}

size_t w4a16_xsum_bytes(int M, int K, int group) {
  if (!sizes_ok(M, 1, K, group)) return 0;
  return (size_t)M * (size_t)affine_kb3(K / group) * sizeof(uint16_t);
}

int w4a16_xsum(const uint16_t *x, int M, int K, int group, uint16_t *xsum, w4a16_stream_t stream) {
  if (!x || !xsum) return W4A16_ERR_INVALID_ARG;
  if (!sizes_ok(M, 1, K, group)) return W4A16_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(xsum, 16)) return W4A16_ERR_MISALIGNED;
  DeviceInfo d;
  int st = current_device(d);
  if (st != W4A16_OK) return st;
  return finish_launch(launch_xsum(x, M, K, group, xsum, reinterpret_cast<cudaStream_t>(stream)));
}

int w4a16_gemm_affine(const uint16_t *x, const uint16_t *xsum, const void *packed, int M, int N, int K, int group,
                      uint16_t *y, w4a16_stream_t stream) {
  const int ov = g_override.load();
  if (!x || !packed || !y || (!xsum && affine_uses_tc(M, ov))) return W4A16_ERR_INVALID_ARG;
  if (!sizes_ok(M, N, K, group)) return W4A16_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(packed, 256) || !aligned(xsum, 16))
    return W4A16_ERR_MISALIGNED;
  DeviceInfo d;
  int st = current_device(d);
  if (st != W4A16_OK) return st;
  GemmCall c{x, static_cast<const uint8_t *>(packed), y, M, N, K, group, kFormAffine, false,
             reinterpret_cast<cudaStream_t>(stream), d.err, d.device, g_overlap.load() != 0};
  return launch_affine(c, xsum, d, ov);
}

int w4a16_gemm_affine_noalloc(const uint16_t *x, const void *packed, int M, int N, int K, int group, uint16_t *y,
                              w4a16_stream_t stream) {
  const int ov = g_override.load();
  if (!x || !packed || !y) return W4A16_ERR_INVALID_ARG;
  if (!sizes_ok(M, N, K, group)) return W4A16_ERR_INVALID_ARG;
  const bool tc = affine_uses_tc(M, ov);
  if (tc && w4a16_xsum_bytes(M, K, group) > kNoAllocXsumBytes) return W4A16_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(packed, 256)) return W4A16_ERR_MISALIGNED;
  DeviceInfo d;
  int st = current_device(d);
  if (st != W4A16_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  GemmCall c{x, static_cast<const uint8_t *>(packed), y, M, N, K, group, kFormAffine, false, s, d.err, d.device,
             g_overlap.load() != 0};
  if (!tc) return launch_affine(c, nullptr, d, ov);
  // every entry the GEMM reads (padding included) is written by this pre-pass
  cudaError_t e = launch_xsum(x, M, K, group, d.noalloc_xsum, s);
  if (e != cudaSuccess) return cuda_fail(e);
  return launch_affine(c, d.noalloc_xsum, d, ov);
}

size_t w4a16_affine_bits_repacked_bytes(int N, int K, int group, int bits) {
  if (!bits_ok(bits) || !sizes_ok(1, N, K, group)) return 0;
  const long long Kp = (long long)K * bits_planes(bits);
  if (!sizes_ok(1, N, Kp, group)) return 0;
  return make_layout(N, (int)Kp, group, kFormAffine).total;
}

size_t w4a16_affine_bits_scratch_bytes(int M, int K, int group, int bits) {
  if (!bits_ok(bits) || !sizes_ok(M, 1, K, group)) return 0;
  const long long Kp = (long long)K * bits_planes(bits);
  if (!sizes_ok(M, 1, Kp, group)) return 0;
  return widened_x_bytes(M, K, bits) + (size_t)M * (size_t)affine_kb3((int)(Kp / group)) * sizeof(uint16_t);
}

int w4a16_repack_affine_bits(const uint32_t *qweight, const uint16_t *scales, const uint16_t *biases, int N, int K,
                             int group, int bits, void *packed, w4a16_stream_t stream) {
  if (!qweight || !scales || !biases || !packed) return W4A16_ERR_INVALID_ARG;
  if (w4a16_affine_bits_repacked_bytes(N, K, group, bits) == 0) return W4A16_ERR_INVALID_ARG;
  if (!aligned(packed, 256) || !aligned(qweight, 4) || !aligned(scales, 2) || !aligned(biases, 2))
    return W4A16_ERR_MISALIGNED;
  DeviceInfo d;
  int st = current_device(d);
  if (st != W4A16_OK) return st;
  const Layout L = make_layout(N, K * bits_planes(bits), group, kFormAffine);
  return finish_launch(launch_repack_affine_bits(reinterpret_cast<const uint32_t *>(qweight), scales, biases, N, K,
                                                 bits, L, static_cast<uint8_t *>(packed),
                                                 reinterpret_cast<cudaStream_t>(stream)));
}

int w4a16_gemm_affine_bits(const uint16_t *x, void *scratch, const void *packed, int M, int N, int K, int group,
                           int bits, uint16_t *y, w4a16_stream_t stream) {
  const int ov = g_override.load();
  if (!x || !scratch || !packed || !y) return W4A16_ERR_INVALID_ARG;
  if (!sizes_ok(M, N, K, group) || w4a16_affine_bits_scratch_bytes(M, K, group, bits) == 0 ||
      w4a16_affine_bits_repacked_bytes(N, K, group, bits) == 0)
    return W4A16_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(packed, 256) || !aligned(scratch, 256))
    return W4A16_ERR_MISALIGNED;
  DeviceInfo d;
  int st = current_device(d);
  if (st != W4A16_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint8_t *scr = static_cast<uint8_t *>(scratch);
  const uint16_t *xin = x;
  if (bits > 4) {
    uint16_t *xw = reinterpret_cast<uint16_t *>(scr);
    cudaError_t e = launch_widen_groups(x, M, K, group, xw, s);
    if (e != cudaSuccess) return cuda_fail(e);
    xin = xw;
  }
  const int Kp = K * bits_planes(bits);
  GemmCall c{xin, static_cast<const uint8_t *>(packed), y, M, N, Kp, group, kFormAffine, false, s, d.err, d.device,
             g_overlap.load() != 0};
  if (!affine_uses_tc(M, ov)) return launch_affine(c, nullptr, d, ov);
  uint16_t *xs = reinterpret_cast<uint16_t *>(scr + widened_x_bytes(M, K, bits));
  cudaError_t e = launch_xsum(xin, M, Kp, group, xs, s);
  if (e != cudaSuccess) return cuda_fail(e);
  return launch_affine(c, xs, d, ov);
}

int w4a16_dequantize_affine_bits(const void *packed, int N, int K, int group, int bits, float *w_out,
                                 w4a16_stream_t stream) {
  if (!packed || !w_out) return W4A16_ERR_INVALID_ARG;
  if (w4a16_affine_bits_repacked_bytes(N, K, group, bits) == 0) return W4A16_ERR_INVALID_ARG;
  if (!aligned(packed, 256) || !aligned(w_out, 16)) return W4A16_ERR_MISALIGNED;
  DeviceInfo d;
  int st = current_device(d);
  if (st != W4A16_OK) return st;
  const Layout L = make_layout(N, K * bits_planes(bits), group, kFormAffine);
  return finish_launch(launch_dequantize_affine_bits(static_cast<const uint8_t *>(packed), L, N, K, bits, w_out,
                                                     reinterpret_cast<cudaStream_t>(stream)));
}

int w4a16_gateup_silu_affine(const uint16_t *x, const uint16_t *xsum, const void *packed_gateup, int M, int N_each,
                             int K, int group, uint16_t *h, w4a16_stream_t stream) {
  const int ov = g_override.load();
  if (!x || !packed_gateup || !h || (!xsum && affine_uses_tc(M, ov))) return W4A16_ERR_INVALID_ARG;
  if (!sizes_ok(M, N_each, K, group) || w4a16_gateup_repacked_bytes(N_each, K, group, kFormAffine) == 0)
    return W4A16_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(h, 16) || !aligned(packed_gateup, 256) || !aligned(xsum, 16))
    return W4A16_ERR_MISALIGNED;
  DeviceInfo d;
  int st = current_device(d);
  if (st != W4A16_OK) return st;
  GemmCall c{x, static_cast<const uint8_t *>(packed_gateup), h, M, N_each, K, group, kFormAffine, true,
             reinterpret_cast<cudaStream_t>(stream), d.err, d.device, g_overlap.load() != 0};
  return launch_affine(c, xsum, d, ov);
}

int w4a16_dequantize(const void *packed, int N, int K, int group, int sym, float *w_out,
                     w4a16_stream_t stream) {
  if (!packed || !w_out) return W4A16_ERR_INVALID_ARG;
  if (!sizes_ok(1, N, K, group) || !form_ok(sym)) return W4A16_ERR_INVALID_ARG;
  if (!aligned(packed, 256) || !aligned(w_out, 16)) return W4A16_ERR_MISALIGNED;
  DeviceInfo d;
  int st = current_device(d);
  if (st != W4A16_OK) return st;
  const Layout L = make_layout(N, K, group, sym);
  return finish_launch(launch_dequantize(static_cast<const uint8_t *>(packed), L, N, w_out,
                                         reinterpret_cast<cudaStream_t>(stream)));
}

int w4a16_kv_append(const uint16_t *k, const uint16_t *v, int64_t k_token, int64_t k_head_stride, int64_t v_token,
                    int64_t v_head_stride, const w4a16_kv_cache *cache, const int32_t *page_table, int max_pages,
                    const int32_t *lengths, const int32_t *starts, int rows, int tokens, w4a16_stream_t stream) {
  AppendCall c;
  if (!k || !v || !page_table || !lengths || !starts) return W4A16_ERR_INVALID_ARG;
  if (!rows_ok(rows, max_pages) || !tokens_ok(tokens)) return W4A16_ERR_INVALID_ARG;
  int st = check_cache(cache, true, c.cache);
  if (st != W4A16_OK) return st;
  const int64_t strides[] = {k_token, k_head_stride, v_token, v_head_stride};
  for (int64_t s : strides)
    if (s < 0) return W4A16_ERR_INVALID_ARG;
  for (int64_t s : strides)
    if (!stride_ok(s, 2)) return W4A16_ERR_MISALIGNED;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(page_table, 4) || !aligned(lengths, 4) || !aligned(starts, 4))
    return W4A16_ERR_MISALIGNED;
  DeviceInfo d;
  st = current_device(d);
  if (st != W4A16_OK) return st;
  c.k = k;
  c.v = v;
  c.k_token = k_token;
  c.k_head = k_head_stride;
  c.v_token = v_token;
  c.v_head = v_head_stride;
  c.rows = KvRows{page_table, lengths, starts, max_pages, rows, tokens};
  c.err = d.err;
  c.stream = reinterpret_cast<cudaStream_t>(stream);
  return finish_launch(launch_kv_append(c));
}

size_t w4a16_tree_attention_workspace_bytes(int heads, int kv_heads, int dim, int max_tree) {
  if (!attn_sizes_ok(heads, kv_heads, dim, max_tree)) return 0;
  return tree_attn_workspace_bytes(heads, kv_heads, dim, max_tree);
}

int w4a16_tree_attention(const uint16_t *q, int64_t q_token, int64_t q_head, const w4a16_kv_cache *cache,
                         const int32_t *page_table, int max_pages, const int32_t *lengths, const int32_t *starts,
                         const int64_t *mask, int rows, int tokens, int heads, int max_tree, float scale,
                         uint16_t *out, void *workspace, w4a16_stream_t stream) {
  AttnCall c;
  if (!q || !page_table || !lengths || !starts || !out || !workspace) return W4A16_ERR_INVALID_ARG;
  if (!rows_ok(rows, max_pages) || !tokens_ok(tokens)) return W4A16_ERR_INVALID_ARG;
  int st = check_cache(cache, true, c.cache);
  if (st != W4A16_OK) return st;
  if (!attn_sizes_ok(heads, c.cache.kv_heads, c.cache.dim, max_tree)) return W4A16_ERR_INVALID_ARG;
  if ((long long)tokens * heads >= 1LL << 31) return W4A16_ERR_INVALID_ARG;
  if (q_token < 0 || q_head < 0 || !(scale > 0.f) || scale > 1e30f) return W4A16_ERR_INVALID_ARG;
  if (!stride_ok(q_token, 2) || !stride_ok(q_head, 2)) return W4A16_ERR_MISALIGNED;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 256) || !aligned(page_table, 4) ||
      !aligned(lengths, 4) || !aligned(starts, 4) || !aligned(mask, 8))
    return W4A16_ERR_MISALIGNED;
  DeviceInfo d;
  st = current_device(d);
  if (st != W4A16_OK) return st;
  c.q = q;
  c.q_token = q_token;
  c.q_head = q_head;
  c.rows = KvRows{page_table, lengths, starts, max_pages, rows, tokens};
  c.mask = mask;
  c.heads = heads;
  c.max_tree = max_tree;
  c.scale = scale;
  c.out = out;
  c.workspace = workspace;
  c.err = d.err;
  c.device = d.device;
  c.sm_count = d.sm_count;
  c.stream = reinterpret_cast<cudaStream_t>(stream);
  return finish_launch(launch_tree_attention(c));
}

int w4a16_tree_accept(const int64_t *target, const int64_t *draft, const int64_t *mask, const int32_t *starts,
                      int rows, int tokens, int max_tree, int32_t *path, int32_t *count, int64_t *token,
                      w4a16_stream_t stream) {
  if (!target || !draft || !starts || !path || !count || !token) return W4A16_ERR_INVALID_ARG;
  if (!rows_ok(rows, 1) || !tokens_ok(tokens) || max_tree < 1 || max_tree > W4A16_MAX_TREE)
    return W4A16_ERR_INVALID_ARG;
  if (!aligned(target, 8) || !aligned(draft, 8) || !aligned(mask, 8) || !aligned(starts, 4) || !aligned(path, 4) ||
      !aligned(count, 4) || !aligned(token, 8))
    return W4A16_ERR_MISALIGNED;
  DeviceInfo d;
  int st = current_device(d);
  if (st != W4A16_OK) return st;
  return finish_launch(launch_tree_accept(target, draft, mask, starts, rows, tokens, max_tree, path, count, token,
                                          d.err, reinterpret_cast<cudaStream_t>(stream)));
}

int w4a16_probabilities(const uint16_t *logits, int64_t logits_row, const float *temperature, const float *floor,
                        int tokens, int vocab, float *out, w4a16_stream_t stream) {
  if (!logits || !out) return W4A16_ERR_INVALID_ARG;
  if (!tokens_ok(tokens) || !tokens_ok(vocab) || logits_row < 0) return W4A16_ERR_INVALID_ARG;
  if (!aligned(logits, 2) || !aligned(temperature, 4) || !aligned(floor, 4) || !aligned(out, 4))
    return W4A16_ERR_MISALIGNED;
  DeviceInfo d;
  int st = current_device(d);
  if (st != W4A16_OK) return st;
  return finish_launch(launch_probabilities(logits, logits_row, temperature, floor, tokens, vocab, out, d.device,
                                            d.sm_count, reinterpret_cast<cudaStream_t>(stream)));
}

int w4a16_tree_sample(const float *p, int64_t p_row, const float *q, int64_t q_row, int vocab, const int64_t *draft,
                      const int64_t *mask, const int32_t *starts, const float *u, int rows, int tokens, int max_tree,
                      int32_t *path, int32_t *count, int64_t *token, w4a16_stream_t stream) {
  if (!p || !draft || !starts || !u || !path || !count || !token) return W4A16_ERR_INVALID_ARG;
  if (!rows_ok(rows, 1) || !tokens_ok(tokens) || !tokens_ok(vocab) || max_tree < 1 || max_tree > W4A16_MAX_TREE)
    return W4A16_ERR_INVALID_ARG;
  if (p_row < 0 || q_row < 0) return W4A16_ERR_INVALID_ARG;
  if (!aligned(p, 4) || !aligned(q, 4) || !aligned(draft, 8) || !aligned(mask, 8) || !aligned(starts, 4) ||
      !aligned(u, 4) || !aligned(path, 4) || !aligned(count, 4) || !aligned(token, 8))
    return W4A16_ERR_MISALIGNED;
  DeviceInfo d;
  int st = current_device(d);
  if (st != W4A16_OK) return st;
  return finish_launch(launch_tree_sample(SampleCall{p, q, p_row, q ? q_row : 0, draft, mask, starts, u, rows, tokens,
                                                     vocab, max_tree, path, count, token, d.err, d.device,
                                                     d.sm_count, reinterpret_cast<cudaStream_t>(stream)}));
}

size_t w4a16_lora_workspace_bytes(int tokens, int rank, int inner) {
  if (!tokens_ok(tokens) || !lora_sizes_ok(rank, inner)) return 0;
  return lora_workspace_bytes(tokens, rank, inner);
}

int w4a16_lora_add(const uint16_t *y, int64_t y_row, const uint16_t *x, int64_t x_row, const uint16_t *a,
                   int64_t a_adapter, int64_t a_row, const uint16_t *b, int64_t b_adapter, int64_t b_row,
                   const float *scale, const int32_t *adapter, const int32_t *starts, int rows, int tokens,
                   int adapters, int rank, int inner, int outer, uint16_t *out, int64_t out_row, void *workspace,
                   w4a16_stream_t stream) {
  if (!y || !x || !a || !b || !adapter || !out || !workspace) return W4A16_ERR_INVALID_ARG;
  if (!tokens_ok(tokens) || !tokens_ok(outer) || !lora_sizes_ok(rank, inner)) return W4A16_ERR_INVALID_ARG;
  if (adapters < 1 || adapters > W4A16_MAX_ADAPTERS) return W4A16_ERR_INVALID_ARG;
  if (starts ? rows < 1 || rows > W4A16_MAX_SEQUENCES : rows != tokens) return W4A16_ERR_INVALID_ARG;
  if (tokens == 1) y_row = x_row = out_row = 0;  // (a stride that takes no step)
  if (adapters == 1) a_adapter = b_adapter = 0;
  if (outer == 1) b_row = 0;
  const int64_t strides[] = {y_row, x_row, a_adapter, a_row, b_adapter, b_row, out_row};
  for (int64_t s : strides)
    if (s < 0) return W4A16_ERR_INVALID_ARG;
  if (y_row >= 1 << 30 || x_row >= 1 << 30 || out_row >= 1 << 30) return W4A16_ERR_INVALID_ARG;
  if (tokens > 1 && out_row < outer) return W4A16_ERR_INVALID_ARG;
  if (!rows_apart(y, y_row, out, out_row, tokens, outer)) return W4A16_ERR_INVALID_ARG;
  const int64_t wide[] = {x_row, a_adapter, a_row, b_adapter, b_row};
  for (int64_t s : wide)
    if (!stride_ok(s, 2)) return W4A16_ERR_MISALIGNED;
  if (!aligned(x, 16) || !aligned(a, 16) || !aligned(b, 16) || !aligned(workspace, 256) || !aligned(y, 2) ||
      !aligned(out, 2) || !aligned(scale, 4) || !aligned(adapter, 4) || !aligned(starts, 4))
    return W4A16_ERR_MISALIGNED;
  DeviceInfo d;
  int st = current_device(d);
  if (st != W4A16_OK) return st;
  LoraCall c;
  c.y = y;
  c.x = x;
  c.a = a;
  c.b = b;
  c.y_row = y_row;
  c.x_row = x_row;
  c.a_adapter = a_adapter;
  c.a_row = a_row;
  c.b_adapter = b_adapter;
  c.b_row = b_row;
  c.out_row = out_row;
  c.scale = scale;
  c.adapter = adapter;
  c.starts = starts;
  c.rows = rows;
  c.tokens = tokens;
  c.adapters = adapters;
  c.rank = rank;
  c.inner = inner;
  c.outer = outer;
  c.out = out;
  c.workspace = workspace;
  c.err = d.err;
  c.device = d.device;
  c.sm_count = d.sm_count;
  c.stream = reinterpret_cast<cudaStream_t>(stream);
  return finish_launch(launch_lora_add(c));
}

int w4a16_kv_compact(const w4a16_kv_cache *cache, const int32_t *page_table, int max_pages, const int32_t *lengths,
                     const int32_t *path, const int32_t *count, int rows, int max_tree, int32_t *lengths_out,
                     w4a16_stream_t stream) {
  KvCache c;
  if (!page_table || !lengths || !path || !count || !lengths_out) return W4A16_ERR_INVALID_ARG;
  if (!rows_ok(rows, max_pages) || max_tree < 1 || max_tree > W4A16_MAX_TREE) return W4A16_ERR_INVALID_ARG;
  if (lengths_out < lengths + rows && lengths < lengths_out + rows) return W4A16_ERR_INVALID_ARG;
  int st = check_cache(cache, false, c);
  if (st != W4A16_OK) return st;
  if (!aligned(page_table, 4) || !aligned(lengths, 4) || !aligned(path, 4) || !aligned(count, 4) ||
      !aligned(lengths_out, 4))
    return W4A16_ERR_MISALIGNED;
  DeviceInfo d;
  st = current_device(d);
  if (st != W4A16_OK) return st;
  return finish_launch(launch_kv_compact(c, KvRows{page_table, lengths, nullptr, max_pages, rows, 0}, path, count,
                                         max_tree, lengths_out, d.err, reinterpret_cast<cudaStream_t>(stream)));
}

int w4a16_kv_free(int32_t *page_table, int max_pages, int table_rows, int32_t *lengths, int32_t *refs, int pages,
                  const int32_t *rows, int n, w4a16_stream_t stream) {
  if (!page_table || !lengths || !refs || !rows) return W4A16_ERR_INVALID_ARG;
  if (max_pages < 1 || table_rows < 1 || pages < 1 || n < 1 || n > W4A16_MAX_ROWS) return W4A16_ERR_INVALID_ARG;
  if (!aligned(page_table, 4) || !aligned(lengths, 4) || !aligned(refs, 4) || !aligned(rows, 4))
    return W4A16_ERR_MISALIGNED;
  DeviceInfo d;
  int st = current_device(d);
  if (st != W4A16_OK) return st;
  return finish_launch(launch_kv_free(TableCall{page_table, lengths, refs, max_pages, table_rows, pages, d.err,
                                                reinterpret_cast<cudaStream_t>(stream)},
                                      rows, n));
}

int w4a16_kv_fork(const w4a16_kv_cache *cache, int32_t *page_table, int max_pages, int table_rows, int32_t *lengths,
                  int32_t *refs, const int32_t *src, const int32_t *dst, int n, int32_t *ok, w4a16_stream_t stream) {
  KvCache c;
  if (!page_table || !lengths || !refs || !src || !dst || !ok) return W4A16_ERR_INVALID_ARG;
  if (max_pages < 1 || table_rows < 1 || n < 1 || n > W4A16_MAX_ROWS) return W4A16_ERR_INVALID_ARG;
  int st = check_cache(cache, false, c);
  if (st != W4A16_OK) return st;
  if (!aligned(page_table, 4) || !aligned(lengths, 4) || !aligned(refs, 4) || !aligned(src, 4) || !aligned(dst, 4) ||
      !aligned(ok, 4))
    return W4A16_ERR_MISALIGNED;
  DeviceInfo d;
  st = current_device(d);
  if (st != W4A16_OK) return st;
  return finish_launch(launch_kv_fork(TableCall{page_table, lengths, refs, max_pages, table_rows, c.pages, d.err,
                                                reinterpret_cast<cudaStream_t>(stream)},
                                      c, src, dst, n, ok));
}

int w4a16_kv_reserve(int32_t *page_table, int max_pages, int table_rows, int32_t *refs, int pages, int page_rows,
                     const int32_t *rows, const int32_t *want, int n, int32_t *ok, w4a16_stream_t stream) {
  const int shift = page_shift_of(page_rows);
  if (!page_table || !refs || !rows || !want || !ok || shift < 0) return W4A16_ERR_INVALID_ARG;
  if (max_pages < 1 || table_rows < 1 || pages < 1 || n < 1 || n > W4A16_MAX_ROWS) return W4A16_ERR_INVALID_ARG;
  if (!aligned(page_table, 4) || !aligned(refs, 4) || !aligned(rows, 4) || !aligned(want, 4) || !aligned(ok, 4))
    return W4A16_ERR_MISALIGNED;
  DeviceInfo d;
  int st = current_device(d);
  if (st != W4A16_OK) return st;
  return finish_launch(launch_kv_reserve(TableCall{page_table, nullptr, refs, max_pages, table_rows, pages, d.err,
                                                   reinterpret_cast<cudaStream_t>(stream)},
                                         shift, rows, want, n, ok));
}

int w4a16_kernel_status(void) {
  DeviceInfo d;
  int st = current_device(d);
  if (st != W4A16_OK) return st;
  cudaError_t e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return cuda_fail(e);
  int v = 0;
  if ((e = cudaMemcpyFromSymbol(&v, g_kernel_error, sizeof(int))) != cudaSuccess) return cuda_fail(e);
  if (v != 0) {
    const int zero = 0;
    if ((e = cudaMemcpyToSymbol(g_kernel_error, &zero, sizeof(int))) != cudaSuccess) return cuda_fail(e);
    return v & kErrTimeout ? W4A16_ERR_TIMEOUT : W4A16_ERR_INDEX;
  }
  return W4A16_OK;
}

const char *w4a16_strerror(int status) {
  switch (status) {
    case W4A16_OK: return "ok";
    case W4A16_ERR_INVALID_ARG: return "invalid argument (size, group, null pointer or reserved argument)";
    case W4A16_ERR_MISALIGNED: return "misaligned pointer (x, y, h need 16 bytes; packed needs 256)";
    case W4A16_ERR_UNSUPPORTED: return "unsupported device (built for sm_103a)";
    case W4A16_ERR_CUDA: return "CUDA error (see w4a16_last_cuda_error)";
    case W4A16_ERR_TIMEOUT: return "a bounded wait inside a kernel gave up";
    case W4A16_ERR_INDEX: return "a kernel skipped an index outside its buffers (page id, position, row or offset)";
    default: return "unknown status";
  }
}

int w4a16_last_cuda_error(void) { return t_last_cuda_error; }

int w4a16_set_kernel_override(int which) {
  if (which < 0 || which > 5) return -1;
  return g_override.exchange(which);
}

int w4a16_set_programmatic_overlap(int on) {
  if (on != 0 && on != 1) return -1;
  return g_overlap.exchange(on);
}

}  // extern "C"
