// The experts' products on E4M3 operands with one fp32 scale per block of 128, on the
// 5th-generation tensor cores (tcgen05.mma kind::f8f6f4, fp32 accumulation).
//   PRODUCT     out[i, j] = sum_b xs[i, b] ws[j / 128, b] sum_{k in b} xq[i, k] wq[j, k]
//   PRODUCT_DX  dx[i, k]  = sum_b dys[i, b] ws[b, k / 128] sum_{j in b} dyq[i, j] wq[j, k]
//   PRODUCT_DW  dw[j, k]  = sum_b dys[b, j] xs[b, k] sum_{i in b} dyq[i, j] xq[i, k]
// b runs over blocks of 128 along the contraction, i over an expert's rows.  The tensor
// cores have no fp32 block scales, so each block's 128 x 256 products are a fresh
// accumulator in tensor memory, and the epilogue warps add it, times its scales, to sums
// that stay in registers (128 a thread) until the tile is complete.  Two accumulators take
// turns, so the MMAs of block b + 1 run while block b is added.
//
// Roles of a CTA (384 threads, one CTA an SM): warp 0 issues the TMA loads of 128-deep
// k-blocks into a ring, warp 1 the MMAs (four 32-deep steps a block), warps 2 and 3 bring each
// block's scales to shared memory, warps 4-11 add and store: warp w owns TMEM lanes
// 32 (w % 4) .. and one half of the 256 columns; a thread's lane is one output row.  w and the
// operands of PRODUCT_DW are read in the layout they have (MN-major descriptors), nothing is
// transposed in memory.  Every wait is bounded.
//
// What bounds it (GB300, 131072 rows, 128 experts, K 4096, n 1536, 410 us at twice the measured
// bf16 rate, no more than a few launches in a row): 671 us, 2.46 PFLOP/s; PRODUCT_DX 727.  Loads
// and MMAs alone take 535, without the stores 616.  A block's MMAs are 540 cycles of the tensor
// pipe, but its 48 KB come into shared memory and go out again, 768 cycles at 128 bytes a cycle;
// adding its accumulator takes about 520, and each side waits for the other's barrier: 920 cycles
// a block.  PRODUCT_DW has a scale a column too, two operations a sum, and four bytes a result:
// 1240 us, 945 without its stores, 1013 without its sums, 634 without both.  Long runs are held
// by the power limit, 784 and 1316.  Measured against it: 16 epilogue warps +26 to +50%; paired
// fma (f32x2) +12%; pairs of CTAs (cta_group::2, 256 x 256 tiles) -5% to +4%, and slower by 6%
// where experts' rows do not fill their tiles; scales copied by the epilogue warps +40%.
#include <cudaTypedefs.h>

#include <stddef.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "product_fp8.cuh"
#include "rows.cuh"

namespace moe {

namespace {
constexpr int BM = 128, BN = 256, BK = 128;
constexpr int BOX = 128 * 128;                 // bytes of one loaded box
constexpr int EPI_WARPS = 8;
constexpr int CW = 4 * BN / EPI_WARPS;         // columns a warp
constexpr int SCALE_WARP0 = 2;                 // warps 0, 1: loads, MMAs; 2, 3: scales
constexpr int EPI_WARP0 = 4;
constexpr int THREADS = 32 * (EPI_WARP0 + EPI_WARPS);
// Registers: 384 threads are launched with 168 each (64512); warps 0-3 give some up, the
// epilogue warps, with 128 sums and 64 loaded values a thread, take them.
constexpr int REGS = 168, REGS_CONTROL = 72, REGS_EPI = 216;
static_assert(128 * REGS_CONTROL + 32 * EPI_WARPS * REGS_EPI == THREADS * REGS, "registers");
template <int N> __device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N> __device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
constexpr uint32_t TMEM_COLS = 512;
constexpr int MAX_E = 1024;
constexpr int kSms = 152;

constexpr int STAGES = 3;                      // of one box of A and two of B
constexpr int STAGE_BYTES = 3 * BOX;
// Blocks' scales in shared memory: for each of the CTA's 128 rows the product of both
// operands' scales, once for either half of the columns; PRODUCT_DW: the rows' scales and the
// 256 columns', in the order in which threads take them (column_slot).  A slot is written when
// the accumulator two blocks before it is full: every epilogue warp has then given back the one
// four blocks before, so it has read the scales of the one five blocks before.
template <int MODE> struct Ring {
  static constexpr int slots = 5;
  static constexpr int floats = 128 + (MODE == PRODUCT_DW ? 2 * 4 * 36 : 128);
  static constexpr int bytes = slots * floats * 4;
};
// PRODUCT_DW: a thread owns columns 2 q, 2 q + 1 of every eight (q = lane % 4) of its warp's
// 128, so theirs lie together, those of another q 36 floats on (no bank conflicts).
__device__ __forceinline__ int column_slot(int c) {   // c: even column of the 256
  return 128 + ((c >> 7) * 4 + (c >> 1 & 3)) * 36 + (c >> 3 & 15) * 2;
}
// Finished sums on their way out: two boxes of 32 rows of 128 bytes an epilogue warp.
constexpr int OUT_BOX = 32 * 128;
constexpr int OUT_BYTES = EPI_WARPS * 2 * OUT_BOX;
constexpr int CTL_BYTES = 9216;
// stages | boxes out | scales | control block with the tiles' schedule | slack for 1024-byte
// alignment
template <int MODE>
constexpr int kSmem = STAGES * STAGE_BYTES + OUT_BYTES + Ring<MODE>::bytes + CTL_BYTES + 1024;

struct alignas(8) Ctl {
  uint64_t full[STAGES];
  uint64_t empty[STAGES];
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort;
  int warp_sums[THREADS / 32];
  int start[MAX_E + 1];       // first row tile of each expert
  int row[MAX_E + 1];         // first row
};
static_assert(sizeof(Ctl) <= CTL_BYTES, "control block");

// n / d for 0 <= n < 2^31 by a multiplication: m = floor(2^32 (2^l - d) / d) + 1 with
// 2^(l-1) < d <= 2^l (Granlund and Montgomery, 1994).
struct Divisor {
  uint32_t d, m, l;
};
Divisor divisor(uint32_t d) {
  uint32_t l = 0;
  while ((1ull << l) < d) ++l;
  return {d, (uint32_t)(((1ull << 32) * ((1ull << l) - d)) / d + 1), l};
}
__device__ __forceinline__ int quotient(int n, const Divisor& v) {
  if (v.l == 0) return n;
  const uint32_t h = __umulhi((uint32_t)n, v.m);
  return (int)((h + (((uint32_t)n - h) >> 1)) >> (v.l - 1));
}

struct Args {
  int E, N, kblocks;          // kblocks: 128-deep blocks of the contraction (not PRODUCT_DW)
  int cols;                   // output columns
  int rows;                   // PRODUCT_DW: output rows an expert
  Divisor tiles_n;            // 256-wide tiles of the columns
  Divisor tiles_m;            // PRODUCT_DW: tiles of an expert's rows
  Divisor splits;             // CTAs that share a tile's contraction
  const int32_t* offsets;
  const float* sa;
  const float* sb;
  bool sa_vec;                // four scales of a row of A are an aligned vector
  int sa_ld;                  // scales of a row of A (PRODUCT_DW: of a block)
  int sb_ld;                  // scales of a row of tiles of w, or of a block of x
  int sb_plane;               // scales of an expert's w
  // The output's planes: one; PRODUCT_DW one an expert; as many again a split, whose parts
  // (fp32, dense) take the output's place.
  void* out;
  long long ld_out, plane;
  int out_align;              // 16 or the element's bytes
  bool accumulate;
  bool boxed;                 // outputs leave as boxes
  int* err;
};

struct Item {
  int e = 0;
  int row0, row_end;          // rows of the tile and the expert's end
  int nt, mt, split;
  int kb0, kb1;               // k-blocks (PRODUCT_DW: 128-row blocks of the whole matrix)
};

// 32 consecutive fp32 columns of this thread's TMEM lane; the values are there after
// tmem_ld_wait, and only asm volatile (add_scaled), which stays behind it, may use them: naming
// them as operands of the wait costs a move each.  (Two loads of 16: 32 registers in a row
// across a loop's end cost spills.)
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float* o = v + 16 * h;
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=f"(o[0]), "=f"(o[1]), "=f"(o[2]), "=f"(o[3]), "=f"(o[4]), "=f"(o[5]), "=f"(o[6]),
          "=f"(o[7]), "=f"(o[8]), "=f"(o[9]), "=f"(o[10]), "=f"(o[11]), "=f"(o[12]),
          "=f"(o[13]), "=f"(o[14]), "=f"(o[15])
        : "r"(taddr + 16 * h));
  }
}
// 32 columns of the warp's 32 lanes in fragments of 8 columns: element 16 h + 4 i + k is row
// 16 h + lane / 4 + 8 (k / 2), column 8 i + 2 (lane % 4) + k % 2.
__device__ __forceinline__ void tmem_ld_fragments(uint32_t taddr, float (&v)[32]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float* o = v + 16 * h;
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=f"(o[0]), "=f"(o[1]), "=f"(o[2]), "=f"(o[3]), "=f"(o[4]), "=f"(o[5]), "=f"(o[6]),
          "=f"(o[7]), "=f"(o[8]), "=f"(o[9]), "=f"(o[10]), "=f"(o[11]), "=f"(o[12]),
          "=f"(o[13]), "=f"(o[14]), "=f"(o[15])
        : "r"(taddr + ((uint32_t)(16 * h) << 16)));
  }
}
// a += b c, in the order of the loads around it.
__device__ __forceinline__ void add_scaled(float& a, float b, float c) {
  asm volatile("fma.rn.f32 %0, %1, %2, %0;" : "+f"(a) : "f"(b), "f"(c));
}
// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(e));
  return e != 0;
}

// At most one committed bulk group still reads shared memory.
__device__ __forceinline__ void bulk_wait_read_1() {
  asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
}
// fp32 box of shared memory added to (x, y, z), each element once: old + new, rounded to
// nearest, as an add by the thread would be.
__device__ __forceinline__ void tma_add_3d(const void* tmap, uint32_t src, int x, int y, int z) {
  asm volatile(
      "cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4}],"
      " [%1];"
      ::"l"(reinterpret_cast<uint64_t>(tmap)), "r"(src), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// The rows [r0, r1) of expert e; false where the offsets do not describe rows.
template <int MODE>
__device__ __forceinline__ bool expert_rows(const Args& g, int e, int& r0, int& r1) {
  r0 = 0;
  r1 = g.N;
  if (!g.offsets) return true;
  r0 = g.offsets[e];
  r1 = g.offsets[e + 1];
  if (r0 < 0 || r1 < r0 || r1 > g.N) return false;
  return MODE != PRODUCT_DW || r0 == r1 || (r0 % BK == 0 && (r1 % BK == 0 || r1 == g.N));
}

// Where part `i` of S of n blocks begins.
__device__ __forceinline__ int share(int n, int i, int S) {
  return S == 1 ? n * i : (int)((long long)n * i / S);
}

// Items in order: PRODUCT and PRODUCT_DX by row tile, column tile, split (activations
// shared by neighbours); PRODUCT_DW by expert, row tile, column tile, split.  it.e is the
// expert of this role's item before (0 at first): experts only move forward.
template <int MODE>
__device__ __forceinline__ void decode(const Args& g, const Ctl* ctl, int item, Item& it) {
  const int S = g.splits.d;
  const int tile = quotient(item, g.splits);
  it.split = item - tile * S;
  const int mi = quotient(tile, g.tiles_n);
  it.nt = tile - mi * g.tiles_n.d;
  if (MODE == PRODUCT_DW) {
    it.e = quotient(mi, g.tiles_m);
    it.mt = mi - it.e * g.tiles_m.d;
    const int r0 = ctl->row[it.e], r1 = ctl->row[it.e + 1];
    it.row0 = r0;
    it.row_end = r1;
    const int nkb = ceil_div(r1 - r0, BK);
    it.kb0 = r0 / BK + share(nkb, it.split, S);
    it.kb1 = r0 / BK + share(nkb, it.split + 1, S);
    return;
  }
  it.mt = mi;
  while (ctl->start[it.e + 1] <= mi) ++it.e;
  it.row0 = ctl->row[it.e] + (mi - ctl->start[it.e]) * BM;
  it.row_end = ctl->row[it.e + 1];
  it.kb0 = share(g.kblocks, it.split, S);
  it.kb1 = share(g.kblocks, it.split + 1, S);
}

// Every thread: the row tiles of each expert, in order; returns their number, or -1
// where the offsets are not valid (nothing is computed then).
template <int MODE>
__device__ __forceinline__ int schedule(const Args& g, Ctl* ctl) {
  constexpr int PER = (MAX_E + THREADS - 1) / THREADS;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int e0 = threadIdx.x * PER;
  int n[PER], sum = 0;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    n[i] = 0;
    if (e0 + i < g.E) {
      int r0, r1;
      if (!expert_rows<MODE>(g, e0 + i, r0, r1)) bad = true;
      else n[i] = ceil_div(r1 - r0, BM);
      ctl->row[e0 + i] = r0;
      if (e0 + i == g.E - 1) ctl->row[g.E] = r1;
    }
    sum += n[i];
  }
  int incl = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(kFull, incl, off);
    if (lane >= off) incl += o;
  }
  if (lane == 31) ctl->warp_sums[warp] = incl;
  bad = __syncthreads_or(bad);
  int at = incl - sum, total = 0;
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) at += ctl->warp_sums[w];
    total += ctl->warp_sums[w];
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (e0 + i < g.E) ctl->start[e0 + i] = at;
    at += n[i];
    if (e0 + i == g.E - 1) ctl->start[g.E] = at;
  }
  __syncthreads();
  return bad ? -1 : total;
}

// 16 finished sums of one row to `p`, in the widest stores that the alignment allows.
template <typename T>
__device__ __forceinline__ void store16(T* p, const float* v, int align) {
  T o[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) o[i] = from_f32<T>(v[i]);
  if (align >= 16) {
    uint4 r[sizeof(o) / 16];
    memcpy(r, o, sizeof(o));
#pragma unroll
    for (int i = 0; i < (int)(sizeof(o) / 16); ++i) reinterpret_cast<uint4*>(p)[i] = r[i];
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) p[i] = o[i];
  }
}

template <int MODE, typename T>
__global__ void __launch_bounds__(THREADS, 1)
product_fp8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmO, const __grid_constant__ Args g) {
  constexpr bool a_mn = MODE == PRODUCT_DW, b_mn = MODE != PRODUCT;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t tile_base = (raw_addr + 1023u) & ~1023u;
  uint8_t* boxes = smem_raw + (tile_base - raw_addr) + STAGES * STAGE_BYTES;
  uint8_t* after = boxes + OUT_BYTES;
  Ctl* ctl = reinterpret_cast<Ctl*>(after + Ring<MODE>::bytes);
  volatile int* abort_flag = &ctl->abort;
  const int warp = __shfl_sync(kFull, threadIdx.x >> 5, 0);   // known to be uniform
  const int lane = threadIdx.x & 31;
  const int first_item = blockIdx.x, item_step = gridDim.x;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(smem_u32(&ctl->full[s]), 1);
      mbar_init(smem_u32(&ctl->empty[s]), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&ctl->tfull[a]), 1 + EPI_WARP0 - SCALE_WARP0);   // MMAs, scales
      mbar_init(smem_u32(&ctl->tempty[a]), EPI_WARPS);
    }
    mbar_init(smem_u32(&ctl->mma_done), 1);
    ctl->abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    if (g.boxed) tma_prefetch_desc(&tmO);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&ctl->tmem_base), TMEM_COLS);
    tmem_relinquish();
  }
  const int row_tiles = schedule<MODE>(g, ctl);
  if (row_tiles < 0 && blockIdx.x == 0 && threadIdx.x == 0 && g.err)
    atomicOr(g.err, kErrBadRouting);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // below 2^30 for all sizes that a call may have
  const int total = row_tiles < 0 ? 0
                                  : (MODE == PRODUCT_DW ? g.E * (int)g.tiles_m.d : row_tiles) *
                                        (int)(g.tiles_n.d * g.splits.d);
  // warp-uniform, so that they stay in uniform registers
  const uint32_t tmem = __shfl_sync(kFull, ctl->tmem_base, 0);
  const uint32_t bars = __shfl_sync(kFull, smem_u32(ctl), 0);
  constexpr uint32_t kFullBar = offsetof(Ctl, full), kEmptyBar = offsetof(Ctl, empty),
                     kTfull = offsetof(Ctl, tfull), kTempty = offsetof(Ctl, tempty);

  if (warp < EPI_WARP0) fewer_registers<REGS_CONTROL>();
  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      uint32_t count = 0;
      bool ok = true;
      Item it;
      for (int item = first_item; item < total && ok; item += item_step) {
        decode<MODE>(g, ctl, item, it);
        for (int kb = it.kb0; kb < it.kb1; ++kb, ++count) {
          const int s = count % STAGES;
          if (!mbar_wait_bounded(smem_u32(&ctl->empty[s]), ((count / STAGES) & 1u) ^ 1u,
                                 abort_flag, g.err)) {
            ok = false;
            break;
          }
          const uint32_t bar = smem_u32(&ctl->full[s]);
          const uint32_t sa = tile_base + s * STAGE_BYTES;
          // the last tile of an odd number of 128-column halves has one of them
          const int c = it.nt * BN, halves = c + 128 < g.cols ? 2 : 1;
          mbar_arrive_expect_tx(bar, (1 + halves) * BOX);
          if (MODE == PRODUCT_DW) tma_load_3d(sa, &tmA, bar, it.mt * BM, kb * BK, 0);
          else tma_load_3d(sa, &tmA, bar, kb * BK, it.row0, 0);
          for (int j = 0; j < halves; ++j) {
            const uint32_t sb = sa + BOX + j * BOX;
            if (MODE == PRODUCT) tma_load_3d(sb, &tmB, bar, kb * BK, c + j * 128, it.e);
            else tma_load_3d(sb, &tmB, bar, c + j * 128, kb * BK, MODE == PRODUCT_DX ? it.e : 0);
          }
        }
      }
      if (!ok) {   // the loads in flight land before the CTA ends
        const uint32_t n = count < (uint32_t)STAGES ? count : (uint32_t)STAGES;
        for (uint32_t q = 0; q < n; ++q) {
          const uint32_t c = count - 1 - q;
          volatile int never = 0;
          mbar_wait_bounded(smem_u32(&ctl->full[c % STAGES]), (c / STAGES) & 1u, &never, nullptr);
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp walks the blocks, so that descriptors and addresses are warp-uniform
    // values (the MMA takes them from uniform registers); one elected thread issues.
    constexpr uint32_t idesc_full = idesc_f8(BM, BN, a_mn, b_mn),
                       idesc_half = idesc_f8(BM, BN / 2, a_mn, b_mn);
    // K-major: 32 codes further along each 128-byte row; MN-major: 32 rows of 128 bytes
    // further, blocks of 128 along MN one box apart
    constexpr uint32_t a_step = (a_mn ? 4096 : 32) >> 4, b_step = (b_mn ? 4096 : 32) >> 4;
    const uint32_t base = __shfl_sync(kFull, tile_base, 0);
    const uint64_t a_base = smem_desc_sw128(base, a_mn ? BOX : 16, 1024);
    const uint64_t b_base = smem_desc_sw128(base + BOX, b_mn ? BOX : 16, 1024);
    const bool issues = elect_one();
    uint32_t s = 0, ph = 0, count = 0;      // stage, its phase, blocks so far
    bool ok = true;
    Item it;
    for (int item = first_item; item < total && ok; item += item_step) {
      decode<MODE>(g, ctl, item, it);
      const int blocks = __shfl_sync(kFull, it.kb1 - it.kb0, 0);
      const uint32_t idesc =
          __shfl_sync(kFull, it.nt * BN + 128 < g.cols ? idesc_full : idesc_half, 0);
      for (int kb = 0; kb < blocks; ++kb) {
        const uint32_t buf = count & 1u;
        ok = mbar_wait_bounded(bars + kFullBar + 8 * s, ph, abort_flag, g.err) &&
             mbar_wait_bounded(bars + kTempty + 8 * buf, ((count >> 1) & 1u) ^ 1u, abort_flag,
                               g.err);
        ok = __all_sync(kFull, ok);
        if (!ok) break;
        tc_fence_after();
        const uint64_t ad = a_base + s * (STAGE_BYTES >> 4);
        const uint64_t bd = b_base + s * (STAGE_BYTES >> 4);
        const uint32_t d = tmem + buf * BN;
        if (issues) {
#pragma unroll
          for (uint32_t ks = 0; ks < BK / 32; ++ks)
            tc_mma_f8(d, ad + ks * a_step, bd + ks * b_step, idesc, ks > 0 ? 1u : 0u);
          tc_commit(bars + kTfull + 8 * buf);
          tc_commit(bars + kEmptyBar + 8 * s);
        }
        ++count;
        if (++s == STAGES) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    if (issues && count > 0) {   // no MMA is in flight when TMEM is released
      tc_commit(smem_u32(&ctl->mma_done));
      volatile int never = 0;
      mbar_wait_bounded(smem_u32(&ctl->mma_done), 0, &never, nullptr);
    }
    __syncwarp();
  } else if (warp >= SCALE_WARP0 && warp < EPI_WARP0) {
    // ------------------------------------------------------------ scales to shared memory
    using Rg = Ring<MODE>;
    constexpr int PT = 32 * (EPI_WARP0 - SCALE_WARP0);   // threads; each has rows tid, tid + 64
    const int tid = threadIdx.x - 32 * SCALE_WARP0;
    float* const ring = reinterpret_cast<float*>(after);
    uint32_t count = 0;
    bool ok = true;
    Item it;
    for (int item = first_item; item < total && ok; item += item_step) {
      decode<MODE>(g, ctl, item, it);
      const int row_end = MODE == PRODUCT_DW ? g.rows : it.row_end;
      const int row = (MODE == PRODUCT_DW ? it.mt * BM : it.row0) + tid;
      const float *pa[2], *pb[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = min(row + PT * i, row_end - 1);    // rows past the end: any
        if (MODE == PRODUCT_DW) {
          pa[i] = g.sa + (size_t)it.kb0 * g.sa_ld + r;
          pb[i] = g.sb + (size_t)it.kb0 * g.sb_ld + min(it.nt * BN + 4 * tid, g.cols - 4);
        } else {
          pa[i] = g.sa + (size_t)r * g.sa_ld + it.kb0;
          const int c = min(2 * it.nt + i, (g.cols - 1) / 128);
          pb[i] = g.sb + (size_t)it.e * g.sb_plane +
                  (MODE == PRODUCT ? (size_t)c * g.sb_ld + it.kb0 : (size_t)it.kb0 * g.sb_ld + c);
        }
      }
      float a[2][4], b[2][4];
      float4 cols = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int kb = it.kb0; kb < it.kb1 && ok; ++kb, ++count) {
        const uint32_t buf = count & 1u;
        const int left = it.kb1 - kb;
        if (MODE == PRODUCT_DW) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            a[i][0] = __ldg(pa[i]);
            pa[i] += g.sa_ld;
          }
          cols = __ldg(reinterpret_cast<const float4*>(pb[0]));
          pb[0] += g.sb_ld;
        } else if (((kb - it.kb0) & 3) == 0) {           // four blocks at a time
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (g.sa_vec && left >= 4) {
              const float4 v = __ldg(reinterpret_cast<const float4*>(pa[i]));
              a[i][0] = v.x; a[i][1] = v.y; a[i][2] = v.z; a[i][3] = v.w;
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j) a[i][j] = j < left ? __ldg(pa[i] + j) : 0.f;
            }
            pa[i] += 4;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              b[i][j] = j < left ? __ldg(pb[i] + (MODE == PRODUCT ? j : (size_t)j * g.sb_ld)) : 0.f;
            pb[i] += MODE == PRODUCT ? 4 : (size_t)4 * g.sb_ld;
          }
        }
        ok = mbar_wait_bounded(smem_u32(&ctl->tfull[buf]), ((count >> 1) & 1u) ^ 1u, abort_flag,
                               g.err);
        ok = __all_sync(kFull, ok);
        if (!ok) break;
        float* slot = ring + (count % Rg::slots) * Rg::floats;
        if (MODE == PRODUCT_DW) {
          slot[tid] = a[0][0];
          slot[tid + PT] = a[1][0];
          *reinterpret_cast<float2*>(slot + column_slot(4 * tid)) = make_float2(cols.x, cols.y);
          *reinterpret_cast<float2*>(slot + column_slot(4 * tid + 2)) = make_float2(cols.z, cols.w);
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) slot[128 * h + tid + PT * i] = a[i][0] * b[h][0];
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 3; ++j) {
              a[i][j] = a[i][j + 1];
              b[i][j] = b[i][j + 1];
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl->tfull[buf]));
      }
    }
  } else if (warp >= EPI_WARP0) {
    more_registers<REGS_EPI>();
    // ------------------------------------------------------------ scaled sums and stores
    using Rg = Ring<MODE>;
    const int q = warp & 3;                  // TMEM lane quadrant
    const int part = (warp - EPI_WARP0) >> 2;   // columns CW part .. of the tile
    const float* const ring = reinterpret_cast<const float*>(after);
    // this thread's output row of an item, whether it is there, and the first column
    struct Place {
      int row, row_end, c0;
      bool any;                              // the warp has something to do
    };
    auto place = [&](const Item& it) {
      Place p;
      const int row_w = (MODE == PRODUCT_DW ? it.mt * BM : it.row0) + q * 32;
      p.row = row_w + lane;
      p.row_end = MODE == PRODUCT_DW ? g.rows : it.row_end;
      p.c0 = it.nt * BN + part * CW;
      p.any = row_w < p.row_end && p.c0 < g.cols;
      return p;
    };
    uint32_t count = 0;
    bool ok = true;
    Item it;
    for (int item = first_item; item < total && ok; item += item_step) {
      decode<MODE>(g, ctl, item, it);
      const Place p = place(it);
      float acc[CW];
#pragma unroll
      for (int i = 0; i < CW; ++i) acc[i] = 0.f;
      float v0[32], v1[32];
      const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16) + part * CW;
      // The accumulator may be written again: the loads and their wait are the whole warp's.
      auto release = [&]() {
        tc_fence_before();
        if (lane == 0) mbar_arrive(bars + kTempty + 8 * (count & 1u));
      };
      auto load = [&](uint32_t t, float (&v)[32]) {
        if (MODE == PRODUCT_DW) tmem_ld_fragments(t, v);
        else tmem_ld32(t, v);
      };
      // f: the row's scale (PRODUCT_DW: its four rows'), w: this thread's columns' of the chunk
      constexpr int NF = MODE == PRODUCT_DW ? 4 : 1, NW = MODE == PRODUCT_DW ? 2 : 1;
      auto add = [&](float* to, const float (&v)[32], const float (&f)[NF], const float4 (&w)[NW]) {
        if constexpr (MODE == PRODUCT_DW) {
          const float ws[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
          for (int j = 0; j < 32; ++j)
            add_scaled(to[j], v[j], ws[(j >> 2 & 3) * 2 + (j & 1)] * f[(j >> 4) * 2 + (j >> 1 & 1)]);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) add_scaled(to[j], v[j], f[0]);
        }
      };
      // The last 32 columns of a block are added beside the first load of the next one.
      float f_last[NF];
      float4 w_last[NW];                      // (PRODUCT_DW)
#pragma unroll
      for (int i = 0; i < NF; ++i) f_last[i] = 0.f;
#pragma unroll
      for (int i = 0; i < NW; ++i) w_last[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 32; ++i) v1[i] = 0.f;
#pragma unroll 1
      for (int kb = it.kb0; kb < it.kb1 && ok; ++kb) {
        const uint32_t buf = count & 1u, t = lanes + buf * BN;
        ok = mbar_wait_bounded(bars + kTfull + 8 * buf, (count >> 1) & 1u, abort_flag, g.err);
        ok = __all_sync(kFull, ok);
        if (!ok) break;
        tc_fence_after();
        if (p.any) {
          load(t, v0);
          const float* slot = ring + (count % Rg::slots) * Rg::floats;
          float f[NF];
          float4 w[4][NW];                    // by 32 columns
          if constexpr (MODE == PRODUCT_DW) {
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = slot[q * 32 + lane / 4 + 8 * i];
            const float4* ws =
                reinterpret_cast<const float4*>(slot + column_slot(part * 128 + 2 * (lane & 3)));
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i / 2][i % 2] = ws[i];
          } else {
            f[0] = slot[part * 128 + q * 32 + lane];
          }
          add(acc + 96, v1, f_last, w_last);
          tmem_ld_wait();
          load(t + 32, v1);
          add(acc, v0, f, w[0]);
          tmem_ld_wait();
          load(t + 64, v0);
          add(acc + 32, v1, f, w[1]);
          tmem_ld_wait();
          load(t + 96, v1);
          add(acc + 64, v0, f, w[2]);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < NF; ++i) f_last[i] = f[i];
          if constexpr (MODE == PRODUCT_DW) {
            w_last[0] = w[3][0];
            w_last[1] = w[3][1];
          }
        }
        release();
        ++count;
      }
      if (p.any) add(acc + 96, v1, f_last, w_last);
      if (!ok) break;
      if (!p.any) continue;
      const int z = MODE == PRODUCT_DW ? it.split * g.E + it.e : it.split;   // the output's plane
      if (g.boxed && (MODE == PRODUCT_DW || p.row - lane + 32 <= p.row_end)) {
        // whole groups of 32 rows: boxes of 128 bytes a row through shared memory, sent by
        // bulk tensor stores (which clip at the matrix's edges)
        constexpr int BC = 128 / sizeof(T);   // columns a box
        const uint32_t box0 = smem_u32(boxes) + (warp - EPI_WARP0) * (2 * OUT_BOX);
        uint8_t* box_p = boxes + (warp - EPI_WARP0) * (2 * OUT_BOX);
#pragma unroll
        for (int c = 0; c < CW; c += BC) {
          if (p.c0 + c >= g.cols) break;
          const int slot = c / BC & 1;
          if (c != BC) {                      // the boxes before in both slots, or in this one,
            if (lane == 0) {                  // have been read
              if (c == 0) bulk_wait_read_0();
              else bulk_wait_read_1();
            }
            __syncwarp();
          }
          if (MODE == PRODUCT_DW) {
#pragma unroll
            for (int j = 0; j < BC; j += 2) { // pairs of a fragment, 128-byte swizzle
              const int ch = j / 32, h = j >> 4 & 1, i = j >> 2 & 3, up = j >> 1 & 1;
              const int r = 16 * h + lane / 4 + 8 * up;
              const int byte = (32 * ch + 8 * i + 2 * (lane & 3)) * (int)sizeof(T);
              T two[2] = {from_f32<T>(acc[c + j]), from_f32<T>(acc[c + j + 1])};
              using Pair = typename RawOf<2 * sizeof(T)>::type;
              Pair raw;
              memcpy(&raw, two, sizeof(raw));
              *reinterpret_cast<Pair*>(box_p + slot * OUT_BOX + r * 128 +
                                       (((byte >> 4) ^ (r & 7)) << 4) + (byte & 15)) = raw;
            }
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {     // 16 bytes each, 128-byte swizzle
              constexpr int W = 16 / sizeof(T);
              const typename Vec<T, W>::Raw r = Vec<T, W>::pack(acc + c + j * W);
              *reinterpret_cast<typename Vec<T, W>::Raw*>(box_p + slot * OUT_BOX + lane * 128 +
                                                          ((j ^ (lane & 7)) * 16)) = r;
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (MODE == PRODUCT_DW && g.accumulate)
              tma_add_3d(&tmO, box0 + slot * OUT_BOX, p.c0 + c, p.row, z);
            else
              tma_store_3d(&tmO, box0 + slot * OUT_BOX, p.c0 + c, p.row, z);
            bulk_commit();
          }
        }
        continue;
      }
      T* out = static_cast<T*>(g.out) + z * g.plane;
      // Added to 16-bit gradients: one rounding.  A load waits for the store before it, which
      // may be to the same address for all that is known here: 131072 rows, 128 x 1536 x 4096,
      // bf16 5340 us against 975 overwritten (fp32, as boxes, 1443 against 1243).
      if (MODE == PRODUCT_DW) {
#pragma unroll
        for (int j = 0; j < CW; ++j) {
          const int row = p.row - lane + 16 * (j >> 4 & 1) + lane / 4 + 8 * (j >> 1 & 1);
          const int col = p.c0 + 32 * (j >> 5) + 8 * (j >> 2 & 3) + 2 * (lane & 3) + (j & 1);
          if (row >= p.row_end || col >= g.cols) continue;
          T* o = out + row * g.ld_out + col;
          *o = from_f32<T>(acc[j] + to_f32(*o));
        }
        continue;
      }
      if (p.row >= p.row_end) continue;
#pragma unroll
      for (int c = 0; c < CW; c += 16) {
        if (p.c0 + c >= g.cols) break;
        store16(out + p.row * g.ld_out + p.c0 + c, acc + c, g.out_align);
      }
    }
    if (lane == 0) bulk_wait_all();          // the boxes have left before shared memory goes
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

// out = the splits' parts (g.out, see Args) added in order (and to what is there), for the
// rows that the product computed: [offsets[0], offsets[E]) of the N, or all (PRODUCT_DW).  A
// thread takes four columns.
template <typename T, bool DW>
__global__ void __launch_bounds__(256)
join_parts_kernel(const Args g, long long rows, T* __restrict__ out, long long ld_out,
                  bool accumulate) {
  wait_for_previous();
  const float* parts = static_cast<const float*>(g.out);
  const int splits = g.splits.d, cols = g.cols;
  long long r0 = 0, r1 = rows;
  if (g.offsets) {   // offsets that are not valid: nothing was computed, nothing is written
    bool bad = false;
    for (int e = threadIdx.x; e < g.E; e += blockDim.x) {
      int a, b;
      bad |= !expert_rows<DW ? PRODUCT_DW : PRODUCT>(g, e, a, b);
    }
    if (__syncthreads_or(bad)) return;
    if (!DW) {
      r0 = g.offsets[0];
      r1 = g.offsets[g.E];
    }
  }
  const int per_row = cols / 4;
  const long long n = (r1 - r0) * per_row;
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < n; i += gridDim.x * 256LL) {
    const long long r = r0 + i / per_row;
    const int c = (int)(i % per_row) * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s = 0; s < splits; ++s) {
      const float4 p = *reinterpret_cast<const float4*>(parts + (s * rows + r) * cols + c);
      v.x += p.x; v.y += p.y; v.z += p.z; v.w += p.w;
    }
    T* o = out + r * ld_out + c;
    const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      o[j] = from_f32<T>(DW && accumulate ? x[j] + to_f32(o[j]) : x[j]);
  }
}

int device_sms(int dev) {
  static int n[64] = {0};
  if (n[dev] == 0) cudaDeviceGetAttribute(&n[dev], cudaDevAttrMultiProcessorCount, dev);
  return n[dev] > 0 ? n[dev] : kSms;
}

template <int MODE, typename T>
cudaError_t launch(const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& mo,
                   const Args& g, long long items, cudaStream_t s) {
  auto kernel = product_fp8_kernel<MODE, T>;
  static bool attr_done[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_done[dev]) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem<MODE>);
    if (e != cudaSuccess) return e;
    cudaFuncAttributes fa;             // more_registers waits for what the launch brings
    e = cudaFuncGetAttributes(&fa, kernel);
    if (e != cudaSuccess) return e;
    if (fa.numRegs != REGS) return cudaErrorInvalidConfiguration;
    attr_done[dev] = true;
  }
  const int grid = (int)std::min<long long>(device_sms(dev), items);
  kernel<<<grid, THREADS, kSmem<MODE>, s>>>(ma, mb, mo, g);
  count_launches(1);
  return cudaGetLastError();
}

template <int MODE>
cudaError_t launch_typed(int dtype, const CUtensorMap& ma, const CUtensorMap& mb,
                         const CUtensorMap& mo, const Args& g, long long items, cudaStream_t s) {
  switch (dtype) {
    case MOE_BF16: return launch<MODE, __nv_bfloat16>(ma, mb, mo, g, items, s);
    case MOE_F16: return launch<MODE, __half>(ma, mb, mo, g, items, s);
    default: return launch<MODE, float>(ma, mb, mo, g, items, s);
  }
}

template <typename T>
cudaError_t join(const ProductArgs& a, const Args& g, long long rows, cudaStream_t s) {
  const long long quads = rows * (g.cols / 4);
  const int blocks = (int)std::max<long long>(1, std::min<long long>((quads + 255) / 256, kSms * 8));
  T* out = static_cast<T*>(a.out);
  const cudaError_t e = a.mode == PRODUCT_DW
      ? launch_after(join_parts_kernel<T, true>, blocks, 256, s, g, rows, out, a.ld_out, a.accumulate)
      : launch_after(join_parts_kernel<T, false>, blocks, 256, s, g, rows, out, a.ld_out, false);
  count_launches(1);
  return e;
}

// Over how many CTAs a tile's contraction is split, and the items' number at most.  Known
// from the sizes alone: the split with the least estimated time, counting half a microsecond a
// block of 128 in a CTA, 3 us for the second kernel and 4 TB/s for writing and reading the
// parts.  Measured without and with a split: 1 row, n = K = 4096: 16.9 and 10.0 us (9 CTAs a
// tile; 9.2 to 11.5 with 4 to 18); 1 row, n 2048, K 7168: 26.3 and 11.3; 1001 rows, n 2064, K
// 1040: 10.3 and 17.9 (3 CTAs a tile; not taken).
struct Cut {
  int splits;
  long long items;
};

Cut cut_of(int mode, int N, int n, int K, int E) {
  const int cols = mode == PRODUCT ? n : K, nt = ceil_div(cols, BN);
  long long tiles = (long long)E * ceil_div(n, BM) * nt;
  if (mode != PRODUCT_DW)
    tiles = std::min<long long>(N, ((long long)N + (long long)std::min(E, N) * (BM - 1)) / BM) * nt;
  const int kblocks = ceil_div(mode == PRODUCT_DW ? N : (mode == PRODUCT ? K : n), BK);
  Cut c{1, tiles};
  if (tiles > 0 && 2 * tiles <= kSms) {
    const double part_us = (double)(mode == PRODUCT_DW ? (long long)E * n : N) * cols * 8 / 4e6;
    double best = 0.5 * kblocks;
    for (int s = 2; s <= kblocks && s * tiles <= kSms; ++s) {
      const double t = 0.5 * ceil_div(kblocks, s) + 3.0 + s * part_us;
      if (t < best) {
        best = t;
        c.splits = s;
      }
    }
  }
  c.items *= c.splits;
  return c;
}

size_t parts_bytes(int mode, int N, int n, int K, int E) {
  const Cut c = cut_of(mode, N, n, K, E);
  if (c.splits == 1) return 0;
  const size_t rows = mode == PRODUCT_DW ? (size_t)E * n : (size_t)N;
  return align_up(c.splits * rows * (mode == PRODUCT ? n : K) * 4, 256);
}
}  // namespace

size_t product_fp8_parts_bytes(int N, int n, int K, int E) {
  return std::max(parts_bytes(PRODUCT, N, n, K, E),
                  std::max(parts_bytes(PRODUCT_DX, N, n, K, E), parts_bytes(PRODUCT_DW, N, n, K, E)));
}

cudaError_t launch_product_fp8(const ProductArgs& a, float* parts, int* err, cudaStream_t s) {
  const bool dw = a.mode == PRODUCT_DW;
  const int cols = a.mode == PRODUCT ? a.n : a.K;
  const int inner = a.mode == PRODUCT ? a.K : a.n;   // columns of a
  if (a.N == 0 && !dw) return cudaSuccess;
  const Cut cut = cut_of(a.mode, a.N, a.n, a.K, a.E);
  Args g{};
  g.E = a.E; g.N = a.N;
  g.kblocks = ceil_div(inner, BK);
  g.cols = cols;
  g.tiles_n = divisor(ceil_div(cols, BN));
  g.rows = a.n;
  g.tiles_m = divisor(ceil_div(a.n, BM));
  g.splits = divisor(cut.splits);
  g.offsets = a.offsets;
  g.sa = a.sa;
  g.sb = a.sb;
  g.sa_ld = dw ? a.n : ceil_div(inner, BK);
  g.sb_ld = dw ? a.K : ceil_div(a.K, BK);
  g.sa_vec = g.sa_ld % 4 == 0 && reinterpret_cast<uintptr_t>(a.sa) % 16 == 0 &&
             cut.splits == 1;
  g.sb_plane = ceil_div(a.n, BK) * ceil_div(a.K, BK);
  const int planes = dw ? a.E : 1;
  const long long all = dw ? (long long)a.E * a.n : (long long)a.N;   // rows of the output
  const bool split = cut.splits > 1;
  const int dtype = split ? MOE_F32 : a.out_dtype, es = dtype_bytes(dtype);
  g.out = split ? parts : a.out;
  g.ld_out = split ? cols : a.ld_out;
  g.plane = (dw ? a.n : a.N) * g.ld_out;
  const unsigned long long low =
      reinterpret_cast<uintptr_t>(g.out) | (unsigned long long)(g.ld_out * es);
  g.out_align = low % 16 == 0 ? 16 : es;
  g.accumulate = a.accumulate && !split;
  g.err = err;
  // boxes out: rows of 16-byte aligned pieces (apart by less than a tensor map's limit); sums
  // added to 16-bit outputs are rounded once, by the thread that reads them
  g.boxed = g.out_align == 16 && !(g.accumulate && es == 2) && g.ld_out < (1LL << 37);
  CUtensorMap ma, mb, mo;
  // a: [N, inner]; b: w [E, n, K], or x [N, K].  A matrix without rows is not read.
  const void* pa = a.N > 0 ? a.a : a.out;
  const void* pb = a.N > 0 || !dw ? a.b : a.out;
  const int rows = std::max(a.N, 1);
  if (!encode_map_codes(&ma, pa, 1, rows, inner, 128, 128) ||
      !encode_map_codes(&mb, pb, dw ? 1 : a.E, dw ? rows : a.n, a.K, 128, 128))
    return cudaErrorInvalidValue;
  mo = ma;
  if (g.boxed &&
      !encode_map_out(&mo, dtype, g.out, (long long)planes * cut.splits, dw ? a.n : rows, cols,
                      g.ld_out))
    return cudaErrorInvalidValue;
  cudaError_t e;
  switch (a.mode) {
    case PRODUCT: e = launch_typed<PRODUCT>(dtype, ma, mb, mo, g, cut.items, s); break;
    case PRODUCT_DX: e = launch_typed<PRODUCT_DX>(dtype, ma, mb, mo, g, cut.items, s); break;
    default: e = launch_typed<PRODUCT_DW>(dtype, ma, mb, mo, g, cut.items, s); break;
  }
  if (e != cudaSuccess || !split) return e;
  switch (a.out_dtype) {
    case MOE_BF16: return join<__nv_bfloat16>(a, g, all, s);
    case MOE_F16: return join<__half>(a, g, all, s);
    default: return join<float>(a, g, all, s);
  }
}

}  // namespace moe
