// Global gradient norm and the AdamW step over many tensors.
//   g' = coef g
//   m  = beta1 m + (1 - beta1) g'            v = beta2 v + (1 - beta2) g'^2
//   p  = p (1 - lr wd) - lr m / (1 - beta1^t) / (sqrt(v / (1 - beta2^t)) + eps)
//
// The tensors' pointers travel as a kernel parameter, so a call needs no device
// copy of its list and can be captured in a graph; a list longer than one
// parameter holds becomes several launches.  lr, the step's number and the seed
// travel with them: a replay is the captured step again (its bias correction, its
// dither), not the next one, so a training loop launches this call itself or
// updates the captured graph each step.  Work is cut into blocks of 256
// elements, `run` consecutive ones a warp, eight warps a chunk, a CTA per chunk.
//
// 8-bit states.  Each block of 256 elements keeps one fp32 scale and E4M3 codes:
// m as code * m_scale, v through its root, sqrt(v) as code * v_scale (the root
// halves the exponent range v needs).  The scale is the block's largest
// magnitude / 448.  A value is rounded to one of its two E4M3 neighbours by a
// dither: with rounding to nearest, v would stand still, since one step moves it
// by (1 - beta2) (g'^2 - v), far less than half a code's spacing of 1/8 to 1/16.
// The dither is a hash of the seed, the tensor's place in the list and the
// element's place, so a step is reproducible.  sqrt(v) > 0 never rounds to zero
// (least code 2^-9): m / eps would follow.  The update itself uses m and v
// before they are rounded.
//
// Bound by HBM: 24 B an element with 32-bit states (bf16 p, fp32 g), 12 B with
// 8-bit ones, where some 50 instructions an element come close to it.
#include <float.h>
#include <math.h>

#include <algorithm>

#include "adamw.cuh"
#include "kernels.h"
#include "rows.cuh"

namespace moe {

namespace {
constexpr int AT = 256;
constexpr int kBlock = 256;                  // elements per scale, one warp's share
constexpr int kRow = kBlock * (AT / 32);     // a block for each warp
constexpr int kPerLaunch = 256;              // tensors in one launch's parameter
constexpr int kNormBlocks = 152 * 32;        // partial sums of a launch
constexpr int kNormThreads = 1024;
constexpr int kMostRun = 8, kRun32 = 2, kNormRun = 4;   // blocks a warp takes at most
// Bits of AdamEntry::kind.
constexpr int kP16 = 1, kG16 = 2, kWide = 4;

struct AdamEntry {
  void* p;
  float* master;
  const void* g;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  long long n;
  float decay;        // 1 - lr * weight decay
  uint32_t place;     // hash of the seed and the tensor's place in the list
  int kind;
  int first;          // its first chunk in this launch
};
struct AdamTable {
  AdamEntry e[kPerLaunch];
  int count, chunks, run;       // a chunk: run blocks a warp
  float b1, b2, c1, c2;         // beta1, beta2, 1 - beta1, 1 - beta2
  float one;                    // 1
  float step_size, root, eps;   // lr / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
  const float* norm;            // {norm, coef, finite, -} or null
};

struct NormEntry {
  const void* g;
  long long n;
  int kind, first;
};
struct NormTable {
  NormEntry e[kPerLaunch];
  int count, chunks, run;
};

template <typename Table>
__device__ __forceinline__ int entry_of(const Table& t, int chunk) {
  int lo = 0, hi = t.count - 1;        // last entry whose first chunk is <= chunk
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (t.e[mid].first <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// A warp's walk over its runs of blocks.
struct Walk {
  int c, k = 0, end = 0;       // chunk, its tensor, the tensor's first chunk past it
  long long base;              // first element of the run
  int left;                    // its elements; <= 0: none
  template <typename Table>
  __device__ __forceinline__ bool at(const Table& t) {   // settles c; false past the end
    if (c >= t.chunks) return false;
    if (c >= end) {
      k = entry_of(t, c);
      end = k + 1 < t.count ? t.e[k + 1].first : t.chunks;
    }
    const auto& e = t.e[k];
    base = (long long)(c - e.first) * (kRow * t.run) + (threadIdx.x >> 5) * (kBlock * t.run);
    left = (int)min((long long)(kBlock * t.run), e.n - base);
    return true;
  }
};

// A 32-bit hash: two rounds of xor-shift and multiplication by an odd number
// (the fractions of the square roots of 2 and 3).
__host__ __device__ __forceinline__ uint32_t mix(uint32_t x) {
  x = (x ^ (x >> 16)) * 0x6A09E667u;
  x = (x ^ (x >> 15)) * 0xBB67AE85u;
  return x ^ (x >> 16);
}
constexpr uint32_t kGolden = 0x9E3779B1u;   // 2^32 / golden ratio

// r / 2^120 in fp32 has E4M3's exponent field (bias 7 against 127) and, below
// 2^-6, its fixed spacing, since fp32 becomes subnormal at 2^-126: the bits'
// upper end is the code.  20 dither bits added below the three kept mantissa bits
// carry into them with probability equal to the cut fraction.  Multiplying by 16
// moves the code to the top byte and drops the sign; `dither` comes times 16.
// r <= 448 (1 + 3 * 2^-24) cannot carry past 448: the dither's last bits are 1000.
constexpr float kToCode = 0x1p-120f;
constexpr float kLeast = 0x1p-129f;         // of code 1
__device__ __forceinline__ uint32_t code_top(float scaled, uint32_t dither) {
  return __float_as_uint(scaled) * 16u + dither;
}

// The top bytes of four words.
__device__ __forceinline__ uint32_t top_bytes(const uint32_t* w) {
  return __byte_perm(__byte_perm(w[0], w[1], 0x0073), __byte_perm(w[2], w[3], 0x0073), 0x5410);
}

// Codes to values, two at a time (exact).
__device__ __forceinline__ float2 e4m3x2_values(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

__device__ __forceinline__ float reciprocal(float v) {   // v normal; within 2^-23 of itself
  float u;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(u) : "f"(v));
  return u;
}

__device__ __forceinline__ float root_of(float v) {   // within 2^-23 of itself; 0 at 0
  float u;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(u) : "f"(v));
  return u;
}

// Largest of the warp's values (all >= 0: their bits order as they do).
__device__ __forceinline__ float warp_max(float v) {
  return __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(v)));
}

__device__ __forceinline__ void ld8(const float* p, float* f) {   // 32-byte aligned
  asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]), "=f"(f[4]), "=f"(f[5]),
                 "=f"(f[6]), "=f"(f[7])
               : "l"(p));
}

// This lane's eight elements of a block, as fp32.  In a block that is whole and
// aligned (WIDE) lane l holds elements 8 l .. 8 l + 7, one access per array;
// otherwise elements l + 32 j, single accesses, `left` of them in the block.
template <bool WIDE>
struct Lane {
  int lane, left;
  __device__ __forceinline__ int at(int j) const { return WIDE ? lane * 8 + j : lane + 32 * j; }
  __device__ __forceinline__ bool has(int j) const { return WIDE || lane + 32 * j < left; }

  __device__ __forceinline__ void get(const float* p, float* f) const {
    if (WIDE) {
      ld8(p + lane * 8, f);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = has(j) ? p[at(j)] : 0.f;
    }
  }
  __device__ __forceinline__ void put(float* p, const float* f) const {
    if (WIDE) {
      st_global_v8(p + lane * 8, f);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (has(j)) p[at(j)] = f[j];
    }
  }
  __device__ __forceinline__ void get(const uint16_t* p, float* f) const {   // bf16
    if (WIDE) {
      unpack8(*reinterpret_cast<const uint4*>(p + lane * 8), f);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = has(j) ? __uint_as_float((uint32_t)p[at(j)] << 16) : 0.f;
    }
  }
  __device__ __forceinline__ void put(uint16_t* p, const float* f) const {
    if (WIDE) {
      *reinterpret_cast<uint4*>(p + lane * 8) = pack8(f);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (has(j)) p[at(j)] = __bfloat16_as_ushort(__float2bfloat16_rn(f[j]));
    }
  }
  __device__ __forceinline__ uint2 get(const uint8_t* p) const {   // codes
    if (WIDE) return *reinterpret_cast<const uint2*>(p + lane * 8);
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (has(j)) w[j / 4] |= (uint32_t)p[at(j)] << (8 * (j % 4));
    return make_uint2(w[0], w[1]);
  }
  __device__ __forceinline__ void put(uint8_t* p, const uint2& c) const {
    if (WIDE) {
      *reinterpret_cast<uint2*>(p + lane * 8) = c;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (has(j)) p[at(j)] = (uint8_t)((j < 4 ? c.x : c.y) >> (8 * (j % 4)));
    }
  }
  // Each element's dither times 16, for the block's first element `base`.
  __device__ __forceinline__ void dithers(long long base, uint32_t place, uint32_t* d) const {
    const uint32_t first = (uint32_t)((unsigned long long)base >> 1);   // base is even
    if (WIDE) {
      const uint32_t x = (first + lane * 4) * kGolden + place;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t h = mix(x + j * kGolden);
        d[2 * j] = __byte_perm(h, 0x80, 0x5104);       // (h & 0xffff) << 8 | 0x80
        d[2 * j + 1] = __byte_perm(h, 0x80, 0x5324);   // (h >> 16) << 8 | 0x80
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t h = mix((first + (lane >> 1) + 16 * j) * kGolden + place);
        d[j] = (lane & 1 ? h >> 16 : h & 0xffffu) << 8 | 0x80u;
      }
    }
  }
};

__device__ __forceinline__ void values8(const uint2& c, float* f) {
  const uint32_t w[4] = {c.x & 0xffffu, c.x >> 16, c.y & 0xffffu, c.y >> 16};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 v = e4m3x2_values(w[j]);
    f[2 * j] = v.x;
    f[2 * j + 1] = v.y;
  }
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// The step's factors as pairs.  The arithmetic goes two elements an instruction:
// with 8-bit states the instructions, not the bytes, are what a plain form runs
// out of.
struct Factors {
  float2 b1, b2, c1, c2, k, one, root, eps, step, decay;   // k: the gradients' factor
  __device__ __forceinline__ Factors(const AdamTable& t, const AdamEntry& e, float coef)
      : b1(both(t.b1)), b2(both(t.b2)), c1(both(t.c1)), c2(both(t.c2)), k(both(coef)),
        one(both(t.one)), root(both(t.root)), eps(both(t.eps)), step(both(-t.step_size)), decay(both(e.decay)) {}
};

// Eight elements' step.  S8: m and v come as code values and are scaled by ms
// and vs (v the root's), and u gets sqrt(v).  There every operation that reaches
// the codes rounds by itself, in the order of the formulas: one bit more or less
// under the dither can turn a code, so results that are to be met bit for bit
// elsewhere cannot have their factors gathered or their sums fused.  (A sum of two
// paired products is compiled to a fused one, whatever rounding it names; times
// `one`, a 1 the compiler does not know, it is fused with that.)
template <bool S8>
__device__ __forceinline__ void step8(const Factors& f, const float* g, float* p, float* m,
                                      float* v, float* u, float ms, float vs) {
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const float2 gj = make_float2(g[j], g[j + 1]);
    float2 mj = make_float2(m[j], m[j + 1]), vj = make_float2(v[j], v[j + 1]), uj;
    if (S8) {
      const float2 gc = __fmul2_rn(gj, f.k), q = __fmul2_rn(vj, both(vs));
      mj = __ffma2_rn(__fmul2_rn(__fmul2_rn(mj, both(ms)), f.b1), f.one, __fmul2_rn(gc, f.c1));
      vj = __ffma2_rn(__fmul2_rn(__fmul2_rn(q, q), f.b2), f.one,
                      __fmul2_rn(__fmul2_rn(gc, gc), f.c2));
      uj = make_float2(__fsqrt_rn(vj.x), __fsqrt_rn(vj.y));
    } else {
      const float2 gc = __fmul2_rn(gj, f.k);
      mj = __ffma2_rn(gc, f.c1, __fmul2_rn(mj, f.b1));
      vj = __ffma2_rn(gc, __fmul2_rn(gc, f.c2), __fmul2_rn(vj, f.b2));
      uj = make_float2(root_of(vj.x), root_of(vj.y));
    }
    const float2 den = __ffma2_rn(uj, f.root, f.eps);
    const float2 ratio = __fmul2_rn(mj, make_float2(reciprocal(den.x), reciprocal(den.y)));
    const float2 pj = __ffma2_rn(ratio, f.step, __fmul2_rn(make_float2(p[j], p[j + 1]), f.decay));
    p[j] = pj.x, p[j + 1] = pj.y;
    m[j] = mj.x, m[j + 1] = mj.y;
    v[j] = vj.x, v[j + 1] = vj.y;
    u[j] = uj.x, u[j + 1] = uj.y;
  }
}

// Codes of eight elements of each state, given the block's scales.
__device__ __forceinline__ void encode8(const float* m, const float* u, float im, float iu,
                                        const uint32_t* d, uint2* mc, uint2* vc) {
  uint32_t wm[8], wu[8];
  const float2 to = both(kToCode);
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const float2 rm = __fmul2_rn(__fmul2_rn(make_float2(m[j], m[j + 1]), both(im)), to);
    const float2 qu = __fmul2_rn(make_float2(u[j], u[j + 1]), both(iu)), ru = __fmul2_rn(qu, to);
    wm[j] = code_top(rm.x, d[j]) | (__float_as_uint(rm.x) & 0x80000000u);
    wm[j + 1] = code_top(rm.y, d[j + 1]) | (__float_as_uint(rm.y) & 0x80000000u);
    // a root above zero is at least 2^-9, of its scale: decided before the factor, below
    // 2^-30 of the scale ru is zero (max of the codes instead spilled twice as much)
    wu[j] = code_top(fmaxf(ru.x, qu.x > 0.f ? kLeast : 0.f), d[j]);
    wu[j + 1] = code_top(fmaxf(ru.y, qu.y > 0.f ? kLeast : 0.f), d[j + 1]);
  }
  *mc = make_uint2(top_bytes(wm), top_bytes(wm + 4));
  *vc = make_uint2(top_bytes(wu), top_bytes(wu + 4));
}

// A block's new scales from its largest values, and their reciprocals (0 for a
// block of zeros).
struct Scales {
  float m, v, im, iu;
  __device__ __forceinline__ Scales(const float* mj, const float* uj) {
    float am = 0.f, au = 0.f;
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      am = fmaxf(fmaxf(am, fabsf(mj[j])), fabsf(mj[j + 1]));
      au = fmaxf(fmaxf(au, uj[j]), uj[j + 1]);
    }
    m = __fmul_rn(warp_max(am), 1.f / 448.f);
    v = __fmul_rn(warp_max(au), 1.f / 448.f);
    im = m >= 0x1p-126f ? __fdiv_rn(1.f, m) : 0.f;
    iu = v >= 0x1p-126f ? __fdiv_rn(1.f, v) : 0.f;
    if (im == 0.f) m = 0.f;
    if (iu == 0.f) v = 0.f;
  }
};

// One block of up to 256 elements of one tensor, one warp.
template <bool S8, bool WIDE>
__device__ __forceinline__ void step_block(const AdamEntry& e, const Factors& f, long long base,
                                           int left) {
  Lane<WIDE> l;
  l.lane = threadIdx.x & 31;
  l.left = left;
  float p[8], g[8], m[8], v[8], u[8];
  float ms = 1.f, vs = 1.f;
  const long long blk = base / kBlock;
  if (e.kind & kG16) l.get((const uint16_t*)e.g + base, g);
  else l.get((const float*)e.g + base, g);
  if (S8) {
    values8(l.get((const uint8_t*)e.m + base), m);
    values8(l.get((const uint8_t*)e.v + base), v);
    ms = e.m_scale[blk];
    vs = e.v_scale[blk];
  } else {
    l.get((const float*)e.m + base, m);
    l.get((const float*)e.v + base, v);
  }
  if (e.master) l.get(e.master + base, p);
  else if (e.kind & kP16) l.get((const uint16_t*)e.p + base, p);
  else l.get((const float*)e.p + base, p);
  step8<S8>(f, g, p, m, v, u, ms, vs);
  if (e.master) l.put(e.master + base, p);
  if (e.kind & kP16) l.put((uint16_t*)e.p + base, p);
  else l.put((float*)e.p + base, p);
  if (!S8) {
    l.put((float*)e.m + base, m);
    l.put((float*)e.v + base, v);
    return;
  }
  const Scales s(m, u);   // elements past the end hold zeros: they do not touch the maxima
  uint32_t d[8];
  uint2 mc, vc;
  l.dithers(base, e.place, d);
  encode8(m, u, s.im, s.iu, d, &mc, &vc);
  l.put((uint8_t*)e.m + base, mc);
  l.put((uint8_t*)e.v + base, vc);
  if (l.lane == 0) {
    e.m_scale[blk] = s.m;
    e.v_scale[blk] = s.v;
  }
}

// A run of whole aligned blocks with 8-bit states, no branch in its loop.  Lane
// b of the first 32 gets the new scale of m of block b in *sm, that of v in *sv.
template <bool G16, bool P16, bool MASTER>
__device__ __forceinline__ void step_run8(const AdamEntry& e, const Factors& f, long long base,
                                          int run, float* sm, float* sv) {
  Lane<true> l;
  l.lane = threadIdx.x & 31;
  l.left = kBlock;
  float ms = 0.f, vs = 0.f;        // the blocks' old scales, a lane each
  if (l.lane < run) {
    ms = e.m_scale[base / kBlock + l.lane];
    vs = e.v_scale[base / kBlock + l.lane];
  }
#pragma unroll 1
  for (int b = 0; b < run; ++b, base += kBlock) {
    float p[8], g[8], m[8], v[8], u[8];
    if (G16) l.get((const uint16_t*)e.g + base, g);
    else l.get((const float*)e.g + base, g);
    const uint2 mc = l.get((const uint8_t*)e.m + base);
    const uint2 vc = l.get((const uint8_t*)e.v + base);
    if (MASTER) l.get(e.master + base, p);
    else if (P16) l.get((const uint16_t*)e.p + base, p);
    else l.get((const float*)e.p + base, p);
    values8(mc, m);
    values8(vc, v);
    step8<true>(f, g, p, m, v, u, __shfl_sync(kFull, ms, b), __shfl_sync(kFull, vs, b));
    if (MASTER) l.put(e.master + base, p);
    if (P16) l.put((uint16_t*)e.p + base, p);
    else l.put((float*)e.p + base, p);
    const Scales s(m, u);
    uint32_t d[8];
    uint2 mn, vn;
    l.dithers(base, e.place, d);
    encode8(m, u, s.im, s.iu, d, &mn, &vn);
    l.put((uint8_t*)e.m + base, mn);
    l.put((uint8_t*)e.v + base, vn);
    if (l.lane == b) {
      *sm = s.m;
      *sv = s.v;
    }
  }
}

__device__ __forceinline__ bool clip_of(const AdamTable& t, float* coef) {
  *coef = 1.f;
  if (!t.norm) return true;
  *coef = t.norm[1];
  return t.norm[2] != 0.f;       // some gradient is not finite: the step is skipped
}

template <bool S8>
__device__ __noinline__ void step_ragged(const AdamEntry& e, const AdamTable& t, float coef,
                                         long long base, int left) {
  const Factors f(t, e, coef);
  for (; left > 0; left -= kBlock, base += kBlock)
    step_block<S8, false>(e, f, base, min(left, kBlock));
}

// 32-bit states.  254M elements with master copies and bf16 gradients (28 B an
// element, 7.1 GB): 1.00 ms, 7.05 TB/s (a copy 6.78).  Two blocks a warp in a
// CTA per chunk; persistent CTAs took 1.06 ms.
__global__ void __launch_bounds__(AT) adamw32_kernel(const __grid_constant__ AdamTable t) {
  float coef;
  Walk w;
  w.c = blockIdx.x;
  if (!clip_of(t, &coef) || !w.at(t) || w.left <= 0) return;
  const AdamEntry& e = t.e[w.k];
  const Factors f(t, e, coef);
  if (e.kind & kWide)
    for (; w.left >= kBlock; w.left -= kBlock, w.base += kBlock)
      step_block<false, true>(e, f, w.base, kBlock);
  if (w.left > 0) step_ragged<false>(e, t, coef, w.base, w.left);
}

// 8-bit states.  553M elements (bf16 p, fp32 g, 6.7 GB): 0.99 ms, 6.7 TB/s.  The
// new scales of a whole chunk go out as lines from shared memory: written block
// by block, 4 bytes at a time into lines that other CTAs read and write at the
// same moment, the kernel took 2.3 ms.  Eight blocks a warp, loads not issued
// ahead: the other warps cover them.  Five CTAs an SM although 48 registers spill
// a little (four with 64: 1.04 ms, three: 1.15, six: 1.09).
__global__ void __launch_bounds__(AT, 5) adamw8_kernel(const __grid_constant__ AdamTable t) {
  __shared__ float scales[2][kMostRun * (AT / 32)];
  float coef;
  Walk w;
  w.c = blockIdx.x;
  if (!clip_of(t, &coef) || !w.at(t)) return;
  const AdamEntry& e = t.e[w.k];
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const long long first = (long long)(w.c - e.first) * kRow * t.run;
  const Factors f(t, e, coef);
  if (!(e.kind & kWide) || first + kRow * t.run > e.n) {
    if (e.kind & kWide)
      for (; w.left >= kBlock; w.left -= kBlock, w.base += kBlock)
        step_block<true, true>(e, f, w.base, kBlock);
    if (w.left > 0) step_ragged<true>(e, t, coef, w.base, w.left);
    return;
  }
  float sm = 0.f, sv = 0.f;
  if (e.kind & kG16) {
    if (e.master) step_run8<true, true, true>(e, f, w.base, t.run, &sm, &sv);
    else if (e.kind & kP16) step_run8<true, true, false>(e, f, w.base, t.run, &sm, &sv);
    else step_run8<true, false, false>(e, f, w.base, t.run, &sm, &sv);
  } else {
    if (e.master) step_run8<false, true, true>(e, f, w.base, t.run, &sm, &sv);
    else if (e.kind & kP16) step_run8<false, true, false>(e, f, w.base, t.run, &sm, &sv);
    else step_run8<false, false, false>(e, f, w.base, t.run, &sm, &sv);
  }
  if (lane < t.run) {
    scales[0][wid * t.run + lane] = sm;
    scales[1][wid * t.run + lane] = sv;
  }
  __syncthreads();
  const int all = t.run * (AT / 32);
  if ((int)threadIdx.x < 2 * all) {
    const int k = threadIdx.x / all, j = threadIdx.x % all;
    (k ? e.v_scale : e.m_scale)[first / kBlock + j] = scales[k][j];
  }
}

// ---------------------------------------------------------------- norm
// 553M fp32 gradients (2.2 GB) in 0.314 ms, 7.05 TB/s.
__device__ __forceinline__ float square_add(float s, float g) { return fmaf(g, g, s); }

// A sum as two fp32 numbers, hi + lo: an addition's rounding error is itself an
// fp32 number and goes into lo, which leaves some 46 bits.  The card adds 64
// fp32 numbers in the time of one fp64: with fp64 sums the norm of 12.6M gradients
// spent 5 of its 18 us in them.
struct Sum {
  float hi, lo;
  __device__ __forceinline__ void add(float x) {
    const float s = __fadd_rn(hi, x), t = __fadd_rn(s, -hi);
    lo += __fadd_rn(__fadd_rn(hi, -__fadd_rn(s, -t)), __fadd_rn(x, -t));
    hi = s;
  }
  __device__ __forceinline__ void add(const Sum& o) {
    add(o.hi);
    lo += o.lo;
  }
  __device__ __forceinline__ void add_over_warp() {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      Sum o;
      o.hi = __shfl_xor_sync(kFull, hi, off);
      o.lo = __shfl_xor_sync(kFull, lo, off);
      // both lanes of a pair must add in the same order
      Sum a = threadIdx.x & off ? o : *this;
      a.add(threadIdx.x & off ? *this : o);
      *this = a;
    }
  }
};

// Squares of four blocks' eight elements a lane (fp32: block b at p + 256 b), all
// loads issued before the first is used: one instruction block, since the
// compiler, free to choose, waits for each to save registers.
__device__ __forceinline__ void squares32(const float* p, Sum& sum) {
  float f[4][8];
  asm volatile(
      "ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%32];\n\t"
      "ld.global.v8.f32 {%8, %9, %10, %11, %12, %13, %14, %15}, [%32+1024];\n\t"
      "ld.global.v8.f32 {%16, %17, %18, %19, %20, %21, %22, %23}, [%32+2048];\n\t"
      "ld.global.v8.f32 {%24, %25, %26, %27, %28, %29, %30, %31}, [%32+3072];"
      : "=f"(f[0][0]), "=f"(f[0][1]), "=f"(f[0][2]), "=f"(f[0][3]), "=f"(f[0][4]), "=f"(f[0][5]),
        "=f"(f[0][6]), "=f"(f[0][7]), "=f"(f[1][0]), "=f"(f[1][1]), "=f"(f[1][2]), "=f"(f[1][3]),
        "=f"(f[1][4]), "=f"(f[1][5]), "=f"(f[1][6]), "=f"(f[1][7]), "=f"(f[2][0]), "=f"(f[2][1]),
        "=f"(f[2][2]), "=f"(f[2][3]), "=f"(f[2][4]), "=f"(f[2][5]), "=f"(f[2][6]), "=f"(f[2][7]),
        "=f"(f[3][0]), "=f"(f[3][1]), "=f"(f[3][2]), "=f"(f[3][3]), "=f"(f[3][4]), "=f"(f[3][5]),
        "=f"(f[3][6]), "=f"(f[3][7])
      : "l"(p));
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) s = square_add(s, f[b][j]);
    sum.add(s);
  }
}

__device__ __forceinline__ void squares32(const uint16_t* p, Sum& sum) {   // bf16
  uint4 q[4];
  asm volatile(
      "ld.global.v4.u32 {%0, %1, %2, %3}, [%16];\n\t"
      "ld.global.v4.u32 {%4, %5, %6, %7}, [%16+512];\n\t"
      "ld.global.v4.u32 {%8, %9, %10, %11}, [%16+1024];\n\t"
      "ld.global.v4.u32 {%12, %13, %14, %15}, [%16+1536];"
      : "=r"(q[0].x), "=r"(q[0].y), "=r"(q[0].z), "=r"(q[0].w), "=r"(q[1].x), "=r"(q[1].y),
        "=r"(q[1].z), "=r"(q[1].w), "=r"(q[2].x), "=r"(q[2].y), "=r"(q[2].z), "=r"(q[2].w),
        "=r"(q[3].x), "=r"(q[3].y), "=r"(q[3].z), "=r"(q[3].w)
      : "l"(p));
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    float f[8], s = 0.f;
    unpack8(q[b], f);
#pragma unroll
    for (int j = 0; j < 8; ++j) s = square_add(s, f[j]);
    sum.add(s);
  }
}

template <bool WIDE>
__device__ __forceinline__ float squares8(const NormEntry& e, long long base, int left) {
  const Lane<WIDE> l{(int)(threadIdx.x & 31), left};
  float g[8], s = 0.f;
  if (e.kind & kG16) l.get((const uint16_t*)e.g + base, g);
  else l.get((const float*)e.g + base, g);
#pragma unroll
  for (int j = 0; j < 8; ++j) s = square_add(s, g[j]);
  return s;
}

// Block b's sum of squares over its chunks.
__global__ void __launch_bounds__(AT) square_sums_kernel(const __grid_constant__ NormTable t,
                                                         float2* __restrict__ sums) {
  __shared__ Sum red[AT / 32];
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  let_next_start();
  Sum sum{0.f, 0.f};
  Walk w;
  for (w.c = blockIdx.x; w.at(t); w.c += gridDim.x) {
    const NormEntry& e = t.e[w.k];
    const bool wide = e.kind & kWide;
    if (wide && w.left == kBlock * kNormRun) {
      const long long i = w.base + lane * 8;
      if (e.kind & kG16) squares32((const uint16_t*)e.g + i, sum);
      else squares32((const float*)e.g + i, sum);
      continue;
    }
    for (; w.left > 0; w.left -= kBlock, w.base += kBlock)
      sum.add(wide && w.left >= kBlock ? squares8<true>(e, w.base, kBlock)
                                       : squares8<false>(e, w.base, w.left));
  }
  sum.add_over_warp();
  if (lane == 0) red[wid] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int k = 1; k < AT / 32; ++k) sum.add(red[k]);
    sums[blockIdx.x] = make_float2(sum.hi, sum.lo);
  }
}

__global__ void __launch_bounds__(kNormThreads) norm_kernel(const float2* sums, int n, bool clip,
                                                            float max_norm, float* norm) {
  __shared__ Sum red[kNormThreads / 32];
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  wait_for_previous();
  Sum sum{0.f, 0.f};
#pragma unroll 4
  for (int i = threadIdx.x; i < n; i += kNormThreads) {
    const float2 s = sums[i];
    sum.add(s.x);
    sum.lo += s.y;
  }
  sum.add_over_warp();
  if (lane == 0) red[wid] = sum;
  __syncthreads();
  if (wid > 0) return;
  sum = red[lane];
  sum.add_over_warp();
  if (lane == 0) {
    // past the fp32 range hi is inf, of a NaN it is NaN, and lo has no meaning
    const float v = isfinite(sum.hi) ? (float)sqrt((double)sum.hi + (double)sum.lo) : sum.hi;
    const float coef = max_norm / (v + 1e-6f);
    norm[0] = v;
    norm[1] = !clip || coef > 1.f ? 1.f : coef;   // a NaN stays
    norm[2] = isfinite(v) ? 1.f : 0.f;
    norm[3] = 0.f;
  }
}

int chunks_of(long long n, int run) {
  return (int)((n + (long long)kRow * run - 1) / ((long long)kRow * run));
}

// Blocks a warp takes in a row: the most up to `most` that leaves eight chunks
// an SM.  Clipped step with 8-bit states: 12.6M elements 41.9 us (four chunks 45.5,
// sixteen 43.7), 6.3M 26.2 (26.0, 28.0), 3.1M 15.0 (14.1, 15.0), 25M 77 (77, 75).
int run_for(const moe_adamw_tensor_t* x, int i, int j, int most) {
  long long total = 0;
  for (int k = i; k < j; ++k) total += x[k].n;
  int run = most;
  while (run > 1 && total < (long long)run * kRow * 152 * 8) run /= 2;
  return run;
}
int grad_bits(const moe_adamw_tensor_t& x) { return x.g_dtype == MOE_BF16 ? kG16 : 0; }

// Eight elements of each array from any multiple of eight are one access.  A tensor
// with an array that is not takes single accesses throughout: 185M elements at an odd
// offset, 8-bit states 735 us (aligned 335); 92M, 32-bit states 364 (323).
bool wide_at(const void* p, int element_bytes) {
  return reinterpret_cast<uintptr_t>(p) % (8 * element_bytes) == 0;
}

// Calls launch(first tensor, past the last) for stretches of the list that fit one
// launch's parameter and chunk count.
template <typename F>
cudaError_t in_runs(const moe_adamw_tensor_t* x, int n, F launch) {
  for (int i = 0; i < n;) {
    int j = i;
    long long chunks = 0;
    while (j < n && j - i < kPerLaunch && chunks + chunks_of(x[j].n, 1) < (1LL << 30))
      chunks += chunks_of(x[j++].n, 1);
    if (chunks > 0) {
      const cudaError_t e = launch(i, j);
      if (e != cudaSuccess) return e;
    }
    i = j;
  }
  return cudaSuccess;
}
}  // namespace

size_t grad_norm_ws_bytes(const moe_adamw_tensor_t* x, int n) {
  int runs = 0;
  (void)in_runs(x, n, [&](int, int) { ++runs; return cudaSuccess; });
  return align_up(sizeof(float2) * kNormBlocks * (size_t)(runs > 0 ? runs : 1), 256);
}

cudaError_t launch_grad_norm(const moe_adamw_tensor_t* x, int n, double max_norm, float* norm,
                             void* ws, cudaStream_t s) {
  float2* sums = static_cast<float2*>(ws);
  int used = 0;
  const cudaError_t e = in_runs(x, n, [&](int i, int j) {
    NormTable t;
    t.count = t.chunks = 0;
    t.run = run_for(x, i, j, kNormRun);
    for (int k = i; k < j; ++k) {
      if (x[k].n == 0) continue;
      const bool wide = wide_at(x[k].g, dtype_bytes(x[k].g_dtype));
      t.e[t.count++] = {x[k].g, x[k].n, grad_bits(x[k]) | (wide ? kWide : 0), t.chunks};
      t.chunks += chunks_of(x[k].n, t.run);
    }
    const int blocks = std::min(t.chunks, kNormBlocks);
    square_sums_kernel<<<blocks, AT, 0, s>>>(t, sums + used);
    used += blocks;
    count_launches(1);
    return cudaGetLastError();
  });
  if (e != cudaSuccess) return e;
  count_launches(1);
  // a limit above zero may be zero in fp32: then the factor is, too; one above the fp32
  // range does not meet an infinite norm as another infinity
  return launch_after(norm_kernel, 1, kNormThreads, s, sums, used, max_norm > 0,
                      (float)std::min(max_norm, (double)FLT_MAX), norm);
}

cudaError_t launch_adamw(const moe_adamw_tensor_t* x, int n, const moe_adamw_t& h,
                         const float* norm, cudaStream_t s) {
  return in_runs(x, n, [&](int i, int j) {
    AdamTable t;
    t.one = 1.f;
    t.b1 = (float)h.beta1;
    t.b2 = (float)h.beta2;
    t.c1 = (float)(1.0 - h.beta1);
    t.c2 = (float)(1.0 - h.beta2);
    t.step_size = (float)(h.lr / (1.0 - pow(h.beta1, (double)h.step)));
    t.root = (float)(1.0 / sqrt(1.0 - pow(h.beta2, (double)h.step)));
    t.eps = (float)h.eps;
    t.norm = norm;
    for (const int bits : {8, 32}) {   // a launch for each kind of state in the run
      t.count = t.chunks = 0;
      t.run = run_for(x, i, j, bits == 8 ? kMostRun : kRun32);
      for (int k = i; k < j; ++k) {
        if (x[k].n == 0 || x[k].state_bits != bits) continue;
        AdamEntry& e = t.e[t.count++];
        e.p = x[k].p;
        e.master = x[k].master;
        e.g = x[k].g;
        e.m = x[k].m;
        e.v = x[k].v;
        e.m_scale = x[k].m_scale;
        e.v_scale = x[k].v_scale;
        e.n = x[k].n;
        e.decay = (float)(1.0 - h.lr * x[k].weight_decay);
        e.place = mix(h.seed + (uint32_t)k * kGolden);
        const bool wide = wide_at(e.p, dtype_bytes(x[k].p_dtype)) && wide_at(e.master, 4) &&
                          wide_at(e.g, dtype_bytes(x[k].g_dtype)) && wide_at(e.m, bits / 8) &&
                          wide_at(e.v, bits / 8);
        e.kind = grad_bits(x[k]) | (x[k].p_dtype == MOE_BF16 ? kP16 : 0) | (wide ? kWide : 0);
        e.first = t.chunks;
        t.chunks += chunks_of(x[k].n, t.run);
      }
      if (t.count == 0) continue;
      if (bits == 8) adamw8_kernel<<<t.chunks, AT, 0, s>>>(t);
      else adamw32_kernel<<<t.chunks, AT, 0, s>>>(t);
      count_launches(1);
      const cudaError_t e = cudaGetLastError();
      if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
  });
}

}  // namespace moe
