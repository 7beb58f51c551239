// Attention of drafted tokens over a paged cache on the fifth-generation tensor
// cores (tcgen05), for rows of the page table with many query rows per kv head
// (wide draft trees, large head groups).
//
// An item is up to 256 query rows (tokens times the heads of one kv head; 128 at
// dim 256 and for 8-bit caches) of one kv head. S = Q . K^T and O += P . V are
// M = 128 MMAs with their accumulators in TMEM: a TMEM lane is one query row, so
// a softmax thread owns a row and needs no exchange. With up to 128 query rows
// HBM bounds the kernel (a 128-key tile at dim 128 is 64 KB, 2,800 clocks of an
// SM's share of HBM, against 1,024 clocks of MMA); with up to 256 the cache is
// still read once, and HBM, MMA time and softmax come near one another.
//
//   warp 0        copies: K and V tiles by TMA through the page table, into one
//                 ring of slots (K0, V0, K1, V1, ...)
//   warps 1, 2    one thread each issues the MMAs of a softmax group of a wide
//                 item, taking turns; otherwise warp 1 issues them all. TMEM
//                 allocation
//   warps 4-7     softmax group 0
//   warps 8-11    softmax group 1 (dim 64 and 128)
//   warps 12-15   8-bit caches: copied tiles of codes to f16, into the ring
//
// The two softmax groups keep maxima, sums and output accumulators of their
// own, so neither waits for the other. In an item of more than 128 rows ("wide")
// each has 128 of the rows and all tiles; else all rows, and every other tile:
// their outputs then meet at the item's end, where each group forms half of
// the columns (both can read the lanes of both). P (bf16; f16 for 8-bit caches)
// replaces S in TMEM and is the second MMA's A operand there; V, [key][dim] in
// shared memory, is its B operand as it lies (MN-major). At dim 256 the output
// takes half of TMEM, so there is one group, with two S buffers. An output
// accumulator is rescaled only when a row's maximum has grown by more than 2^8
// (8-bit caches: 2^3): until then the weights are up to 2^8, and the sums are float32.
//
// P is rounded once; sums use the unrounded weights. bf16: 2^-8 of a weight at
// most, as the output's own rounding. 8-bit caches: f16 times 2^12, so up to 2^15,
// 2^-11 of a weight down to 2^-26 of the maximum: many keys far below one other
// still count together. (Sums of the rounded weights cost registers: 16 rows of
// 4,096 keys, dim 128, 64 query rows 69.1 us; so 64.0.)
//
// Measured, dim 128, bf16: 16 rows of 4,096 keys and 8 kv heads (268 MB) with 32,
// 64 and 128 query rows per kv head 55, 57 and 61 us (4.9, 4.8, 4.6 TB/s); 4 rows
// of 16,384 keys with 256 72 us, 950 TFLOP/s; 8-bit caches 61 and 64 us with 32 and
// 64 query rows, 101 with 256 (converting bounds them). A wide tile takes some 3,500 clocks:
// a group's chain is 1,300 for its two products, 1,550 for its softmax and its
// stores, and 600 of waiting for the other's turn and of handing over. (Handing P
// over in two halves: 2 % slower. Fetching the next item's Q by a warp of its own
// during the output of the one before: 1 to 3 % slower.)
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "tree_attn.cuh"

namespace w4a16 {
namespace {

constexpr int kWarpCopy = 0, kWarpMma = 1, kWarpSoftmax = 4, kWarpConvert = 12;
// What beginning and ending an item costs (Q, filling and draining the pipeline, the output), in key tiles. 16 ragged
// trees of up to 64 nodes, 12 rows of up to 8 nodes, one 16-node tree: with 3 68.6, 28.9 and 25.2 us, with 4 65.4, 28.1
// and 25.1, with 5 66.5, 28.9 and 26.3.
constexpr int kTcLead = 4;
constexpr int kRows = 128;  // query rows of an MMA
constexpr int kInfo = 16;  // tiles whose key-group words are kept
constexpr int kOdd = 8;    // items whose words of odd values are kept: more than tiles converted ahead

template <int DIM, bool E4M3>
struct TcGeo {
  static constexpr int THREADS = E4M3 ? 512 : 384;
  static constexpr int STREAMS = DIM == 256 ? 1 : 2;  // softmax groups
  static constexpr int KT = tc_attn_keys(DIM);        // keys of a tile
  // How far (powers of two) a row's maximum may pass the one that its weights count from, and what the weights are
  // multiplied by: f16 ends at 2^16, and loses bits below 2^-14.
  static constexpr float LAG = E4M3 ? 3.f : 8.f, WEIGHT_LOG2 = E4M3 ? 12.f : 0.f;
  static constexpr int CH = DIM / 64;                 // 128-byte columns of a row
  static constexpr int SUB = KT * 128;                // one column of a K or V tile
  static constexpr int SLOT = CH * SUB;
  static constexpr int QSUB = kRows * 128;
  static constexpr int Q_TILE = CH * QSUB;
  static constexpr int ROWS = tc_attn_rows(DIM, E4M3);
  static constexpr int Q_BYTES = ROWS / kRows * Q_TILE;
  using Tiles = Tiling<ROWS, KT, kRows, kTcLead>;
  static constexpr int SLOTS = E4M3 ? (DIM == 64 ? 8 : 4) : DIM == 64 ? 12 : 5;
  // what is copied: boxes of BW bytes by up to KT rows, BCH of them side by side. 8-bit tiles go to slots of their own
  static constexpr int ELT = E4M3 ? 1 : 2;
  static constexpr int BW = DIM * ELT < 128 ? DIM * ELT : 128, BCH = DIM * ELT / BW, BSUB = KT * BW;
  static constexpr int RAW_SLOT = KT * DIM;
  static constexpr int RAW = E4M3 ? (DIM == 64 ? 8 : DIM == 128 ? 4 : 2) : 0;
  static constexpr int SBUFS = 2;                     // S buffers: one per stream, or two of the one
  // TMEM columns: S (P over its first half), then O
  static constexpr int COL_O = SBUFS * KT;
  static constexpr int OFF_SLOT = Q_BYTES;
  static constexpr int OFF_RAW = OFF_SLOT + SLOTS * SLOT;
  static constexpr int OFF_ML = OFF_RAW + RAW * RAW_SLOT;
  static constexpr int OFF_BAR = OFF_ML + 2 * kRows * 8;
  static constexpr int NBARS = 2 * SLOTS + 2 * SBUFS + 5 + 2 * RAW;
  static constexpr int OFF_INFO = OFF_BAR + NBARS * 8;
  static constexpr int OFF_MISC = OFF_INFO + kInfo * 4;  // TMEM address, abort flag, odd values
  static constexpr int OFF_PLAN = OFF_MISC + 8 + kOdd * 8;
  static constexpr int SMEM = OFF_PLAN + (int)sizeof(PlanShared);
  static_assert(COL_O + STREAMS * DIM <= 512, "TMEM budget");
  static_assert(SMEM <= 227 * 1024 && OFF_SLOT % 1024 == 0 && OFF_PLAN % 8 == 0, "shared memory budget");
  static_assert(SLOTS / 2 + 2 < kInfo, "a tile's word outlives its use");
};

// K-major (rows of 128 bytes, 8-row atoms 1,024 bytes apart) or MN-major (64
// elements of the long axis per 128-byte row, `mn_block` bytes to the next 64;
// 8 rows of the short axis per atom) operand with the 128-byte swizzle
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t mn_block) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(mn_block >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// B is MN-major
constexpr uint32_t kIdescBMn = 1u << 16;
// A and B are f16 (type 0) and not bf16 (type 1)
constexpr uint32_t kIdescF16 = ~((1u << 7) | (1u << 10));

__device__ __forceinline__ void tmem_ld32_nowait(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// 16 / 32 consecutive columns of this thread's lane
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float (&f)[32]) {
  const uint32_t *v = reinterpret_cast<const uint32_t *>(f);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,"
      "%30,%31,%32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
      "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
      "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}

__device__ __forceinline__ uint32_t pack2_f16(float lo, float hi) {
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&b);
}

template <int THREADS>
__device__ __forceinline__ void softmax_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
}

// e4m3 codes of NaN, as a byte mask
__device__ __forceinline__ uint32_t nan_codes(uint32_t x) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (((x >> (8 * i)) & 0x7Fu) == 0x7Fu) m |= 0xFFu << (8 * i);
  return m;
}
__device__ __forceinline__ uint32_t not_finite_bf16(uint32_t x) {
  return ((x & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u) | ((x & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u);
}

// Which of keys 32c .. 32c + 31 of a tile a row sees: `ctx` keys of the tile
// are cached ones, then the new tokens follow, by the row's mask word
__device__ __forceinline__ uint32_t seen_bits(int c, int ctx, unsigned long long word, uint32_t groups) {
  const int j0 = 32 * c, off = j0 - ctx;  // off: new-token index of the first key
  uint32_t v;
  if (off >= 0) v = off < 64 ? (uint32_t)(word >> off) : 0u;
  else if (off <= -32) v = 0xFFFFFFFFu;
  else v = ((1u << -off) - 1) | ((uint32_t)word << -off);
  const uint32_t g = groups >> (2 * c);
  return v & ((g & 1 ? 0xFFFFu : 0u) | (g & 2 ? 0xFFFF0000u : 0u));
}

template <int DIM, bool E4M3>
__global__ void __launch_bounds__(TcGeo<DIM, E4M3>::THREADS, 1)
    tree_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                   const __grid_constant__ AttnParams p) {
  using G = TcGeo<DIM, E4M3>;
  constexpr int KT = G::KT, STREAMS = G::STREAMS;
  constexpr int SOFT = STREAMS * 128;  // softmax threads
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + G::OFF_MISC);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + G::OFF_MISC + 4);
  uint32_t *odd_values = reinterpret_cast<uint32_t *>(smem + G::OFF_MISC + 8);
  volatile uint32_t *info = reinterpret_cast<volatile uint32_t *>(smem + G::OFF_INFO);
  PlanShared &plan = *reinterpret_cast<PlanShared *>(smem + G::OFF_PLAN);
  if (sbase & 1023u) {  // the swizzle counts from multiples of 1,024 (dynamic shared memory starts at one)
    if (tid == 0) atomicOr(p.err, kErrTimeout);
    return;
  }
  const uint32_t bars = sbase + G::OFF_BAR;
  auto full = [&](uint32_t s) { return bars + 8 * s; };
  auto empty = [&](uint32_t s) { return bars + 8 * (G::SLOTS + s); };
  auto s_full = [&](uint32_t b) { return bars + 8 * (2 * G::SLOTS + b); };               // S written
  auto p_full = [&](uint32_t b) { return bars + 8 * (2 * G::SLOTS + G::SBUFS + b); };    // P written, O rescaled
  const uint32_t q_full = bars + 8 * (2 * G::SLOTS + 2 * G::SBUFS);  // Q written, TMEM of the last item read
  const uint32_t o_full = q_full + 8;                                // the item's MMAs are done
  const uint32_t o_done = o_full + 24;                               // one group: a tile's output is in the accumulator
  auto raw_full = [&](uint32_t s) { return o_full + 32 + 8 * s; };   // 8 bits: copied
  auto raw_empty = [&](uint32_t s) { return o_full + 32 + 8 * (G::RAW + s); };  // ... and converted
  auto turn_of = [&](uint32_t w) { return o_full + 8 + 8 * w; };     // an MMA thread's turn to issue

  if (tid == 0) {
    for (int i = 0; i < G::SLOTS; ++i) {
      mbar_init(full(i), E4M3 ? 4 : 1);
      mbar_init(empty(i), STREAMS);
    }
    for (int i = 0; i < G::RAW; ++i) {
      mbar_init(raw_full(i), 1);
      mbar_init(raw_empty(i), 4);
    }
    for (int i = 0; i < G::SBUFS; ++i) {
      mbar_init(s_full(i), 1);
      mbar_init(p_full(i), 4);
    }
    mbar_init(q_full, SOFT / 32);
    mbar_init(o_full, STREAMS);
    mbar_init(o_done, 1);
    mbar_init(turn_of(0), 1);
    mbar_init(turn_of(1), 1);
    *abort_flag = 0;
    for (int i = 0; i < 2 * kOdd; ++i) odd_values[i] = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  grid_dependency_wait();
  grid_launch_dependents();
  plan_share<typename G::Tiles, G::THREADS>(p, plan);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Cursor cur{plan.at, plan.end, plan.at < plan.end ? plan.unit : plan.end, plan.b, plan.head, plan.rt};
  Segment sg;

  // A softmax thread holds a row's 128 scores. The block is launched with 384 x 168 (8 bits: 512 x 128) registers; the
  // first warpgroup (copies, MMAs) keeps 56 each, the converting one 72, and the softmax groups (at dim 256 one of them)
  // get 224 (192) each: 128 * 56 + 256 * 224 = 384 * 168, and 128 * (56 + 72) + 256 * 192 = 512 * 128.
  if (warp < kWarpSoftmax) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == kWarpCopy) {
      // ------------------------------------------------------------ copies
      const int br = min(p.c.page_rows, KT), parts = KT / br;
      const int part = lane % parts, col = lane / parts;
      const bool has_box = col < G::BCH;
      if (lane == 0) {
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
      }
      uint64_t pol;
      asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(pol));
      uint64_t keep;  // several row tiles come back for the same keys
      asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(keep));
      uint32_t ring = 0, tile = 0;
      bool ok = true;
      while (ok && next_segment<typename G::Tiles>(p, cur, sg)) {
        const int32_t *ids = p.r.table + (long long)sg.b * p.r.max_pages;
        const uint64_t policy = sg.i.n * p.group > G::ROWS ? keep : pol;
        auto id_of = [&](int kt) {  // -1: past the keys
          const long long key = (long long)kt * KT + part * br;
          return kt < sg.kt1 && key < sg.i.keys ? ids[key >> p.c.page_shift] : -1;
        };
        auto copy = [&](const CUtensorMap *tm, int kt, int id, bool load, uint32_t loads) {
          constexpr int N = E4M3 ? G::RAW : G::SLOTS;
          const uint32_t s = ring % N, bar = E4M3 ? raw_full(s) : full(s);
          ok = ok && mbar_wait(E4M3 ? raw_empty(s) : empty(s), ((ring / N) & 1) ^ 1, abort_flag);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) return;
          if (lane == 0) mbar_arrive_expect_tx(bar, __popc(loads) * br * G::BW);
          __syncwarp();
          if (load)
            tma_load_4d(sbase + (E4M3 ? G::OFF_RAW + s * G::RAW_SLOT : G::OFF_SLOT + s * G::SLOT) + col * G::BSUB + part * br * G::BW,
                        tm, col * (G::BW / G::ELT), (kt * KT + part * br) & (p.c.page_rows - 1), sg.head, id, bar, policy);
          __syncwarp();
          ++ring;
        };
        int next = id_of(sg.kt0);
        for (int kt = sg.kt0; ok && kt < sg.kt1; ++kt, ++tile) {
          const int id = next;
          next = id_of(kt + 1);
          const bool valid = (unsigned)id < (unsigned)p.c.pages, load = has_box && valid;
          if (col == 0 && !valid && kt * KT + part * br < sg.i.keys) attn_flag(p.err);
          const uint32_t loads = __ballot_sync(0xFFFFFFFFu, load);
          if (lane == 0) {
            uint32_t groups = 0;  // 16-key groups that are there (lanes 0 .. parts - 1: the first column's boxes)
            for (int i = 0; i < parts; ++i)
              if (loads >> i & 1) groups |= ((1u << (br / 16)) - 1) << (i * br / 16);
            info[tile % kInfo] = groups;
          }
          copy(&tm_k, kt, id, load, loads);
          copy(&tm_v, kt, id, load, loads);
        }
      }
      if (!ok && lane == 0) {
        *abort_flag = 1;
        atomicOr(p.err, kErrTimeout);
        // every copy issued lands before the CTA can exit
        constexpr uint32_t N = E4M3 ? G::RAW : G::SLOTS;
        for (uint32_t i = 0; i < N && i < ring; ++i) {
          const uint32_t u = ring - 1 - i;
          mbar_wait_drain(E4M3 ? raw_full(u % N) : full(u % N), (u / N) & 1);
        }
      }
    } else if (warp < kWarpMma + STREAMS) {
      // ------------------------------------------------------------ MMAs
      if (lane == 0) {
        constexpr uint32_t types = E4M3 ? kIdescF16 : ~0u;
        constexpr uint32_t idesc_s = idesc_bf16_f32(kRows, KT) & types;
        constexpr uint32_t idesc_o = (idesc_bf16_f32(kRows, DIM) & types) | kIdescBMn;
        const int mine = warp - kWarpMma;  // the softmax group served
        uint32_t ring = 0, item = 0, turn = 0;
        // Turns: a visit's two products are issued in one go. Left to themselves the two threads' MMAs mix, both groups
        // wait for both, and then both do softmax while the tensor core rests; in turn, one group's softmax runs under
        // the other's MMAs.
        uint32_t turns = 0;
        uint32_t made = 0;  // bit b: the parity of the scores written to S buffer b, the phase of its barriers
        bool ok = true;
        const uint64_t q_desc = smem_desc(sbase, 16);
        // Ring slot r has arrived. (A parity only tells two uses of a slot apart: whoever waits here has itself waited for
        // the slot's use before, or for the end of the item that it was part of.)
        auto arrived = [&](uint32_t r) {
          return mbar_wait<true>(full(r % G::SLOTS), (r / G::SLOTS) & 1, abort_flag);
        };
        // a slot is free once both threads' MMAs have read it; where one thread issues them all it gives it back for both
        auto release = [&](uint32_t slot, bool wide) {
          if (STREAMS == 2 && !wide) mbar_arrive(empty(slot));
          tc_commit(empty(slot));
        };
        // thread 0 goes first; later turns come from the other thread
        auto my_turn = [&]() {
          const uint32_t parity = mine == 0 ? (turns & 1) ^ 1 : turns & 1;
          ++turns;
          return mbar_wait<true>(turn_of(mine), parity, abort_flag);
        };
        while (ok && next_segment<typename G::Tiles>(p, cur, sg)) {
          ok = mbar_wait(q_full, item & 1, abort_flag);
          ++item;
          const int n = sg.kt1 - sg.kt0;
          const bool wide = STREAMS == 2 && sg.rows > kRows;
          // Visits to the S buffers in turn. Each first takes the P that the buffer holds (its last scores' weights) into
          // the output, then writes the next scores: tile v / 2 of group v % 2, or tile v.
          const int scores = wide ? 2 * n : n;
          const int step = wide ? 2 : 1, last = wide || mine == 0 ? scores + 2 : 0;
          for (int v = wide ? mine : 0; ok && v < last; v += step) {
            const uint32_t b = STREAMS == 2 ? v & 1 : (turn + v) & 1;
            const int was = v - 2;
            if (was >= 0) {
              const uint32_t r = ring + 2 * (wide ? was >> 1 : was) + 1;  // the values' ring slot
              ok = arrived(r) && mbar_wait<true>(p_full(b), (made >> b & 1) ^ 1, abort_flag);
              if (wide) ok = ok && (v >= scores || arrived(r + 1)) && my_turn();  // (r + 1: the keys that follow)
              if (!ok) break;
              tc_fence_after();
              uint64_t vd = smem_desc(sbase + G::OFF_SLOT + (r % G::SLOTS) * G::SLOT, G::SUB);
              uint32_t pa = tmem + b * KT;
              const uint32_t d = tmem + G::COL_O + (STREAMS == 2 ? b * DIM : 0);
              uint32_t add = was >= (wide ? 2 : STREAMS);  // the group's first output of the item overwrites
#pragma unroll
              for (int c = 0; c < KT / 64; ++c) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  tc_mma_f16_ts(d, pa + 8 * k, vd + k * (2048 >> 4), idesc_o, add);
                  add = 1;
                }
                pa += 32;
                vd += 4 * (2048 >> 4);
              }
              if (STREAMS == 1) tc_commit(o_done);
              release(r % G::SLOTS, wide);
            }
            if (v < scores) {
              const uint32_t r = ring + 2 * (wide ? v >> 1 : v);  // the keys' ring slot
              if (!wide || was < 0) {
                ok = arrived(r) && (!wide || my_turn());
                if (!ok) break;
                tc_fence_after();
              }
              uint64_t kd = smem_desc(sbase + G::OFF_SLOT + (r % G::SLOTS) * G::SLOT, 16);
              uint64_t qd = q_desc + (wide && b ? G::Q_TILE >> 4 : 0);
              const uint32_t d = tmem + b * KT;
              uint32_t add = 0;
#pragma unroll
              for (int c = 0; c < G::CH; ++c) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  tc_mma_f16(d, qd + 2 * k, kd + 2 * k, idesc_s, add);
                  add = 1;
                }
                qd += G::QSUB >> 4;
                kd += G::SUB >> 4;
              }
              tc_commit(s_full(b));
              made ^= 1u << b;
              release(r % G::SLOTS, wide);
            }
            if (wide) mbar_arrive(turn_of(mine ^ 1));
          }
          // the phases of the buffers that the other thread wrote
          if (wide) made ^= (n & 1u) << (mine ^ 1);
          else if (mine == 1) made ^= ((n + 1) / 2 & 1u) | (n / 2 & 1u) << 1;
          turn += n;
          ring += 2 * n;
          tc_commit(o_full);
        }
        if (!ok) {
          *abort_flag = 1;
          atomicOr(p.err, kErrTimeout);
          // every MMA issued has completed before TMEM is freed (the loop's last commit covers them)
          if (item > 0) mbar_wait_drain(o_full, (item - 1) & 1);
        }
      }
    }
  } else if (warp < kWarpSoftmax + 4 * STREAMS) {
    if constexpr (E4M3) asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    // ------------------------------------------------------------ softmax
    const int stream = (warp - kWarpSoftmax) >> 2, quarter = warp & 3;
    const int lane_row = quarter * 32 + lane;  // query row of the MMA: TMEM lane
    const int st = tid - kWarpSoftmax * 32;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t o_col = lanes + G::COL_O + stream * DIM;
    float2 *ml = reinterpret_cast<float2 *>(smem + G::OFF_ML);
    uint32_t tile = 0, item = 0, ring = 0;
    uint32_t took = 0;  // scores taken by this group (its S buffer, or the two in turn)
    bool ok = true;  // after a wait that gave up: no more waits, but the barriers below are still met
    while (next_segment<typename G::Tiles>(p, cur, sg)) {
      const int rows = sg.rows;
      const bool wide = STREAMS == 2 && rows > kRows;
      const int row = lane_row + (wide ? stream * kRows : 0);  // this thread's query row of the item
      // ---- Q: K-major, 128-byte swizzle; rows past the item's are zero
      long long *q_row = reinterpret_cast<long long *>(smem + G::OFF_ML);  // between two items' use of it
      float *q_scale = reinterpret_cast<float *>(q_row + kRows);  // 8 bits (items of 128 rows)
      const int q_rows = wide ? 2 * kRows : kRows;
      for (int r = st; r < q_rows; r += SOFT) {
        const int rr = sg.rt * G::ROWS + r;
        q_row[r] = r < rows ? (sg.i.start + rr / p.group) * p.q_token + (sg.head * p.group + rr % p.group) * p.q_head : -1;
      }
      softmax_sync<SOFT>();
      constexpr int QN = kRows * (DIM / 8) / SOFT, QB = QN < 8 ? QN : 8;  // 16-byte pieces of a thread, and per batch
      const int qn = q_rows / kRows * QN;
#pragma unroll 1
      for (int i0 = 0; i0 < qn; i0 += QB) {
        uint4 x[QB];
#pragma unroll
        for (int u = 0; u < QB; ++u) {
          const int e = st + (i0 + u) * SOFT;
          const long long q = q_row[e / (DIM / 8)];
          x[u] = q >= 0 ? *reinterpret_cast<const uint4 *>(p.q + q + 8 * (e % (DIM / 8))) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < QB; ++u) {
          const int e = st + (i0 + u) * SOFT, r = e / (DIM / 8), c = e % (DIM / 8);
          if constexpr (E4M3) {
            // f16, times the power of two that takes the row's largest element to 2^14 (a row's pieces are in
            // neighbouring lanes); a row that is not finite stays as it is
            uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w}, high = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) high = max(high, max((w[k] >> 7) & 0xFFu, (w[k] >> 23) & 0xFFu));
#pragma unroll
            for (int d = 1; d < DIM / 8; d <<= 1) high = max(high, __shfl_xor_sync(0xFFFFFFFFu, high, d));
            const int power = high == 0xFFu ? 0 : min(141 - (int)high, 120);
            const float f = __uint_as_float((uint32_t)(127 + power) << 23);
            if (c == 0) q_scale[r] = f;
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = pack2_f16(bf16lo_to_f32(w[k]) * f, bf16hi_to_f32(w[k]) * f);
            x[u] = make_uint4(w[0], w[1], w[2], w[3]);
          }
          sts128(sbase + (r / kRows) * G::Q_TILE + (c >> 3) * G::QSUB + (r % kRows) * 128 + (((c & 7) ^ (r & 7)) << 4), x[u]);
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      if (st < 2) odd_values[2 * ((item - 1) % kOdd) + st] = 0;  // the last item's
      softmax_sync<SOFT>();
      if (lane == 0) mbar_arrive(q_full);
      uint32_t *odd_of = odd_values + 2 * (item % kOdd);
      float factor = p.scale_log2, v_scale = 1.f;
      if constexpr (E4M3) {
        factor *= p.c.k.scale[sg.head] / q_scale[lane_row];
        v_scale = p.c.v.scale[sg.head];
      }
      const int rr = sg.rt * G::ROWS + row, tok = rr / p.group;
      unsigned long long word = 0;
      if (row < rows) {
        word = p.mask ? (unsigned long long)p.mask[sg.i.start + tok] : (2ull << tok) - 1;
        if (sg.i.n < 64) word &= (1ull << sg.i.n) - 1;
      }
      float m = -INFINITY, l = 0.f;
      const int n = sg.kt1 - sg.kt0;
      const bool idle = row - lane >= rows;  // a warp without rows: its P is never looked at
      for (int i = 0; i < n; ++i, ++tile) {
        if (STREAMS == 2 && !wide && (i & 1) != stream) continue;
        const uint32_t v_slot = ring + 2 * i + 1;
        const uint32_t b = STREAMS == 2 ? (uint32_t)stream : took & 1;
        const uint32_t phase = STREAMS == 2 ? took & 1 : (took >> 1) & 1;
        ++took;
        const uint32_t s_col = lanes + b * KT;
        if (ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait(s_full(b), phase, abort_flag));
        tc_fence_after();
        const uint32_t groups = info[tile % kInfo];
        const int key0 = (sg.kt0 + i) * KT;
        const bool masked = key0 + KT > sg.i.len || groups != (1u << (KT / 16)) - 1;
        if (!E4M3 && masked) {  // (8 bits: where they are converted)
          // Values that must not meet a weight of 0: zeroed before the MMA reads them. All threads of this group.
          const uint32_t v = v_slot % G::SLOTS;
          if (ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait(full(v), (v_slot / G::SLOTS) & 1, abort_flag));
          const uint32_t vbase = sbase + G::OFF_SLOT + v * G::SLOT;
          for (int e = st & 127; e < KT * (DIM / 8); e += 128) {
            const int j = e / (DIM / 8), c = e % (DIM / 8), key = key0 + j;
            const bool there = key < sg.i.keys && (groups >> (j >> 4) & 1);
            if (there && key < sg.i.len) continue;
            const uint32_t a = vbase + (c >> 3) * G::SUB + j * 128 + (((c & 7) ^ (j & 7)) << 4);
            uint4 x = make_uint4(0, 0, 0, 0);
            if (there) {
              x = lds128(a);
              const uint32_t b0 = not_finite_bf16(x.x), b1 = not_finite_bf16(x.y), b2 = not_finite_bf16(x.z),
                             b3 = not_finite_bf16(x.w);
              if (!(b0 | b1 | b2 | b3)) continue;
              x = make_uint4(x.x & ~b0, x.y & ~b1, x.z & ~b2, x.w & ~b3);
              const int nw = key - sg.i.len;
              atomicOr(&odd_of[nw >> 5], 1u << (nw & 31));
            }
            sts128(a, x);
          }
          fence_proxy_async_smem();
        }
        if (!idle) {
          // ---- the row's scores of the tile, all in registers, and their maximum
          float x[KT / 32][32];
#pragma unroll
          for (int c = 0; c < KT / 32; ++c) tmem_ld32_nowait(s_col + 32 * c, x[c]);
          tmem_wait_ld();
          if (masked) {
#pragma unroll
            for (int c = 0; c < KT / 32; ++c) {
              const uint32_t seen = seen_bits(c, sg.i.len - key0, word, groups);
#pragma unroll
              for (int e = 0; e < 32; ++e) x[c][e] = seen >> e & 1 ? x[c][e] : -INFINITY;
            }
          }
          float t4[4] = {x[0][0], x[0][1], x[0][2], x[0][3]};
#pragma unroll
          for (int c = 0; c < KT / 32; ++c)
#pragma unroll
            for (int e = 0; e < 32; e += 8)
#pragma unroll
              for (int k = 0; k < 4; ++k) t4[k] = fmaxf(fmaxf(t4[k], x[c][e + k]), x[c][e + 4 + k]);
          const float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
          const float mn = fmaxf(m, __fmul_rn(top, factor));
          const bool grow = mn > m + G::LAG;  // (or m was -inf)
          const bool first = i < (wide ? 1 : STREAMS);  // this group's first tile: no output yet
          if (__any_sync(0xFFFFFFFFu, grow)) {
            const float alpha = grow ? exp2_approx(m - mn) : 1.f;
            if (grow) m = mn;
            l *= alpha;
            if (!first) {
              // With two groups, these scores were made after the group's last output. The one group's were made ahead
              // of it: it may still be under way.
              if (STREAMS == 1 && ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait<true>(o_done, took & 1, abort_flag));
              if (STREAMS == 1) tc_fence_after();
#pragma unroll
              for (int c = 0; c < DIM / 32; ++c) {
                float y[32];
                tmem_ld32_nowait(o_col + 32 * c, y);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) y[e] *= alpha;
                tmem_st32(o_col + 32 * c, y);
              }
            }
          }
          // ---- weights, over the first half of S's columns
          const float base = (m == -INFINITY ? 0.f : m) - G::WEIGHT_LOG2;
          const f32x2 scale2 = f32_pair(factor, factor), base2 = f32_pair(-base, -base);
          f32x2 zero2;  // (not known to the compiler, which would make one fma of a product and a sum)
          asm volatile("mov.b64 %0, 0;" : "=l"(zero2));
          f32x2 sum[2] = {f32_pair(0.f, 0.f), f32_pair(0.f, 0.f)};
#pragma unroll
          for (int c = 0; c < KT / 32; ++c) {
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              // (8 bits: in two roundings, as the maximum was formed, so that its own weight is a power of two; it and the sums
              // then agree where one key has it all, although f16 rounds the weights alone)
              const f32x2 xx = f32_pair(x[c][e], x[c][e + 1]);
              const float2 y = f32_halves(E4M3 ? add2(fma2(xx, scale2, zero2), base2) : fma2(xx, scale2, base2));
              const float a = exp2_approx(y.x), d = exp2_approx(y.y);
              sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], f32_pair(a, d));
              w[e >> 1] = E4M3 ? pack2_f16(a, d) : pack2(a, d);
            }
            tmem_st16(s_col + 16 * c, w);
          }
          const float2 sums = f32_halves(add2(sum[0], sum[1]));
          l += sums.x + sums.y;
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(b));
      }
      ring += 2 * n;
      // ---- the item's output
      // (all MMAs are done, so all threads have begun their tiles and none still needs what lay here)
      if (ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait(o_full, item & 1, abort_flag));
      ml[stream * kRows + lane_row] = make_float2(m, l);
      ++item;
      softmax_sync<SOFT>();
      tc_fence_after();
      if (!idle) {
        // the group whose accumulator this thread reads, and the other one if it has a part of the same rows
        const int s0 = wide ? stream : 0;
        const bool both = STREAMS == 2 && !wide && n > 1;
        const float2 a = ml[s0 * kRows + lane_row], c2 = both ? ml[kRows + lane_row] : make_float2(-INFINITY, 0.f);
        const float M = fmaxf(a.x, c2.x), base = M == -INFINITY ? 0.f : M;
        const float f0 = exp2_approx(a.x - base), f1 = exp2_approx(c2.x - base);
        const float L = a.y * f0 + c2.y * f1;
        const bool whole = sg.whole(), mine = row < rows;
        const float inv = L > 0.f || L != L ? v_scale / L : 0.f;
        const float g0 = whole ? f0 * inv : f0, g1 = whole ? f1 * inv : f1;
        // slot 0: the item began before this share; slot 1: it goes on after it
        const Partial<DIM, G::ROWS> part(p.partials, blockIdx.x, sg.kt0 > 0 ? 0 : 1);
        if (st == 0 && sg.kt0 > 0 && sg.kt1 == sg.ktiles) leave_record<typename G::Tiles>(p, sg, plan.share);
        uint16_t *out = p.out + ((long long)(sg.i.start + tok) * p.heads + sg.head * p.group + rr % p.group) * DIM;
        const uint32_t odd[2] = {odd_of[0], odd_of[1]};
        const uint32_t oc = lanes + G::COL_O;
        const int cols = wide ? DIM : DIM / STREAMS, col0 = wide ? 0 : stream * cols;  // columns of this group
#pragma unroll 1
        for (int c = col0; c < col0 + cols; c += 32) {
          float x[32];
          tmem_ld32_nowait(oc + s0 * DIM + c, x);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) x[e] *= g0;
          if (both) {
            float y[32];
            tmem_ld32_nowait(oc + DIM + c, y);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = fmaf(y[e], g1, x[e]);
          }
          if (odd[0] | odd[1]) {
            for (int j = 0; j < sg.i.n; ++j) {
              if (!(odd[j >> 5] >> (j & 31) & 1) || !(word >> j & 1)) continue;
              const long long pos = (long long)sg.i.len + j;
              const int id = p.r.table[(long long)sg.b * p.r.max_pages + (pos >> p.c.page_shift)];
              const uint8_t *v = p.c.v.base + (long long)id * p.c.v.page + (long long)sg.head * p.c.v.head +
                                 (pos & (p.c.page_rows - 1)) * p.c.v.row + (long long)c * G::ELT;
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                if (E4M3) {
                  if ((v[e] & 0x7Fu) == 0x7Fu) x[e] = NAN;
                } else {
                  const float f = __uint_as_float((uint32_t) reinterpret_cast<const uint16_t *>(v)[e] << 16);
                  if (!(fabsf(f) < INFINITY)) x[e] += f;
                }
              }
            }
          }
          if (mine && whole) {
#pragma unroll
            for (int e = 0; e < 32; e += 8)
              *reinterpret_cast<uint4 *>(out + c + e) = make_uint4(pack2(x[e], x[e + 1]), pack2(x[e + 2], x[e + 3]),
                                                                   pack2(x[e + 4], x[e + 5]), pack2(x[e + 6], x[e + 7]));
          } else if (mine) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<float4 *>(part.at(row, c + e)) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
          }
        }
        if (mine && !whole && (wide || stream == 0)) *part.ml(row) = make_float2(M, L);
      }
      // the next item's Q, odd values and maxima: after everyone is here
      softmax_sync<SOFT>();
    }
    if (!ok) {
      *abort_flag = 1;
      if (lane == 0) atomicOr(p.err, kErrTimeout);
    }
  } else if constexpr (E4M3) {
    if (warp >= kWarpConvert) {
      // ---------------------------------------------------------- codes to f16
      asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
      const int ct = tid - kWarpConvert * 32;
      uint32_t ring = 0, tile = 0, item = 0;
      bool ok = true;
      while (ok && next_segment<typename G::Tiles>(p, cur, sg)) {
        for (int kt = sg.kt0; ok && kt < sg.kt1; ++kt, ++tile) {
#pragma unroll 1
          for (int side = 0; side < 2; ++side, ++ring) {
            const uint32_t rs = ring % G::RAW, s = ring % G::SLOTS;
            ok = ok && mbar_wait(raw_full(rs), (ring / G::RAW) & 1, abort_flag) &&
                 mbar_wait(empty(s), ((ring / G::SLOTS) & 1) ^ 1, abort_flag);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            const uint32_t groups = info[tile % kInfo];
            const int key0 = kt * KT;
            const bool clean = side == 0 || (key0 + KT <= sg.i.len && groups == (1u << (KT / 16)) - 1);
            // A thread takes 16-code pieces: of key j = ct / 4 + 32 (u / SUBS), the (ct % 4)-th of 64-element column
            // u % SUBS, so that all its addresses are constants apart.
            constexpr int SUBS = G::CH, N = KT / 32 * SUBS;
            const int j0 = ct >> 2, c4 = ct & 3;
            const uint32_t from = sbase + G::OFF_RAW + rs * G::RAW_SLOT + j0 * G::BW + c4 * 16;
            const uint32_t to = sbase + G::OFF_SLOT + s * G::SLOT + j0 * 128;
            const uint32_t lo16 = ((2 * c4) ^ (j0 & 7)) << 4, hi16 = ((2 * c4 + 1) ^ (j0 & 7)) << 4;
            uint4 x[N];
#pragma unroll
            for (int u = 0; u < N; ++u) {
              const int sub = u % SUBS;
              x[u] = lds128(from + (u / SUBS) * 32 * G::BW + sub * 64 / G::BW * G::BSUB + sub * 64 % G::BW);
            }
            if (!clean) {
              // values that must not meet a weight of 0
#pragma unroll
              for (int u = 0; u < N; ++u) {
                const int j = j0 + 32 * (u / SUBS), key = key0 + j;
                const bool there = key < sg.i.keys && (groups >> (j >> 4) & 1);
                if (there && key < sg.i.len) continue;
                const uint4 m = there ? make_uint4(nan_codes(x[u].x), nan_codes(x[u].y), nan_codes(x[u].z), nan_codes(x[u].w))
                                      : make_uint4(~0u, ~0u, ~0u, ~0u);
                if (there && (m.x | m.y | m.z | m.w)) {
                  const int nw = key - sg.i.len;
                  atomicOr(&odd_values[2 * (item % kOdd) + (nw >> 5)], 1u << (nw & 31));
                }
                x[u] = make_uint4(x[u].x & ~m.x, x[u].y & ~m.y, x[u].z & ~m.z, x[u].w & ~m.w);
              }
            }
#pragma unroll
            for (int u = 0; u < N; ++u) {
              // 16 codes are 32 bytes of a 128-byte row
              uint4 y[2];
              e4m3x4_f16(x[u].x, y[0].x, y[0].y);
              e4m3x4_f16(x[u].y, y[0].z, y[0].w);
              e4m3x4_f16(x[u].z, y[1].x, y[1].y);
              e4m3x4_f16(x[u].w, y[1].z, y[1].w);
              const uint32_t row = to + (u % SUBS) * G::SUB + (u / SUBS) * 32 * 128;
              sts128(row + lo16, y[0]);
              sts128(row + hi16, y[1]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(full(s));
              mbar_arrive(raw_empty(rs));
            }
          }
        }
        ++item;
      }
      if (!ok) {
        *abort_flag = 1;
        if (lane == 0) atomicOr(p.err, kErrTimeout);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int DIM, bool E4M3>
cudaError_t launch_tc_dim(const AttnCall &c, const AttnParams &p) {
  using G = TcGeo<DIM, E4M3>;
  auto kern = tree_tc_kernel<DIM, E4M3>;
  static PerDevice configured;
  if (!configured.v[c.device].load(std::memory_order_relaxed)) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, G::SMEM);
    if (e != cudaSuccess) return e;
    configured.v[c.device].store(1, std::memory_order_relaxed);
  }
  CUtensorMap tk, tv;
  const int br = std::min(c.cache.page_rows, G::KT);
  if (!encode_cache(&tk, c.cache.k, c.cache, br, G::BW, !E4M3) || !encode_cache(&tv, c.cache.v, c.cache, br, G::BW, !E4M3))
    return cudaErrorInvalidValue;
  return launch_dependent(kern, std::min(c.sm_count, kTcMaxCtas), G::THREADS, G::SMEM, c.stream, tk, tv, p);
}

template <bool E4M3>
cudaError_t launch_tc_type(const AttnCall &c, const AttnParams &p) {
  switch (c.cache.dim) {
    case 64: return launch_tc_dim<64, E4M3>(c, p);
    case 128: return launch_tc_dim<128, E4M3>(c, p);
    default: return launch_tc_dim<256, E4M3>(c, p);
  }
}

}  // namespace

cudaError_t launch_tree_tc(const AttnCall &c, const AttnParams &p) {
  return c.cache.e4m3 ? launch_tc_type<true>(c, p) : launch_tc_type<false>(c, p);
}

}  // namespace w4a16
