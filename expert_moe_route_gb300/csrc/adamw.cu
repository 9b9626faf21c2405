// Global gradient norm and the AdamW step over many tensors.
//   g' = coef g
//   m  = beta1 m + (1 - beta1) g'            v = beta2 v + (1 - beta2) g'^2
//   p  = p (1 - lr wd) - lr m / (1 - beta1^t) / (sqrt(v / (1 - beta2^t)) + eps)
//
// The tensors' pointers travel as a kernel parameter, so a call needs no device
// copy of its list and can be captured in a graph; a list longer than one
// parameter holds becomes several launches.  Work is cut into chunks of 2048
// elements, eight blocks of 256, one per warp; a persistent grid walks them.
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
// 8-bit ones.
#include <math.h>

#include "adamw.cuh"
#include "kernels.h"

namespace moe {

namespace {
constexpr int AT = 256;
constexpr int kBlock = 256;                  // elements per scale, one warp's share
constexpr int kChunk = kBlock * (AT / 32);   // elements per CTA pass
constexpr int kPerLaunch = 256;              // tensors in one launch's parameter
constexpr int kNormBlocks = 152 * 8;

// Bits of AdamEntry::kind.
constexpr int kP16 = 1, kG16 = 2, kS8 = 4, kWide = 8;

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
  int count, chunks;
  float b1, b2, c1, c2;         // beta1, beta2, 1 - beta1, 1 - beta2
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
  int count, chunks;
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

// A 32-bit hash: two rounds of xor-shift and multiplication by an odd number
// (the fractions of the square roots of 2 and 3).
__host__ __device__ __forceinline__ uint32_t mix(uint32_t x) {
  x = (x ^ (x >> 16)) * 0x6A09E667u;
  x = (x ^ (x >> 15)) * 0xBB67AE85u;
  return x ^ (x >> 16);
}
constexpr uint32_t kGolden = 0x9E3779B1u;   // 2^32 / golden ratio

// r in [0, 448] rounded to an E4M3 value by 20 dither bits: adding them below
// the kept mantissa bits and cutting rounds up with probability equal to the
// fraction.  Below 2^-6 the spacing is 2^-9; adding 2^-6 moves r to a binade
// with that spacing.
__device__ __forceinline__ float round_e4m3(float r, uint32_t dither) {
  const float shift = r < 0.015625f ? 0.015625f : 0.f;
  const uint32_t b = (__float_as_uint(__fadd_rn(r, shift)) + dither) & 0xFFF00000u;
  return fminf(__uint_as_float(b) - shift, 448.f);
}

__device__ __forceinline__ float e4m3_value(uint8_t c) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, off));
  return v;
}

// One block of 256 elements of one tensor, elements lane + 32 j.
__device__ __forceinline__ void step_block(const AdamEntry& e, const AdamTable& t, long long base,
                                           float coef) {
  const int lane = threadIdx.x & 31;
  const long long blk = base / kBlock;
  float ms = 0.f, vs = 0.f;
  if (e.kind & kS8) {
    ms = e.m_scale[blk];
    vs = e.v_scale[blk];
  }
  float m[8], u[8];
  float am = 0.f, au = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const long long i = base + lane + 32 * j;
    m[j] = u[j] = 0.f;
    if (i >= e.n) continue;
    const float g0 = e.kind & kG16 ? __bfloat162float(((const __nv_bfloat16*)e.g)[i])
                                   : ((const float*)e.g)[i];
    const float g = __fmul_rn(g0, coef);
    float m0, v0;
    if (e.kind & kS8) {
      m0 = __fmul_rn(e4m3_value(((const uint8_t*)e.m)[i]), ms);
      const float q = __fmul_rn(e4m3_value(((const uint8_t*)e.v)[i]), vs);
      v0 = __fmul_rn(q, q);
    } else {
      m0 = ((const float*)e.m)[i];
      v0 = ((const float*)e.v)[i];
    }
    m[j] = __fadd_rn(__fmul_rn(m0, t.b1), __fmul_rn(g, t.c1));
    const float v = __fadd_rn(__fmul_rn(v0, t.b2), __fmul_rn(__fmul_rn(g, g), t.c2));
    u[j] = __fsqrt_rn(v);
    float p;
    if (e.master) p = e.master[i];
    else p = e.kind & kP16 ? __bfloat162float(((const __nv_bfloat16*)e.p)[i]) : ((const float*)e.p)[i];
    p = p * e.decay - m[j] * t.step_size / (u[j] * t.root + t.eps);
    if (e.master) e.master[i] = p;
    if (e.kind & kP16) ((__nv_bfloat16*)e.p)[i] = __float2bfloat16_rn(p);
    else ((float*)e.p)[i] = p;
    if (!(e.kind & kS8)) {
      ((float*)e.m)[i] = m[j];
      ((float*)e.v)[i] = v;
    }
    am = fmaxf(am, fabsf(m[j]));
    au = fmaxf(au, u[j]);
  }
  if (!(e.kind & kS8)) return;
  ms = __fdiv_rn(warp_max(am), 448.f);
  vs = __fdiv_rn(warp_max(au), 448.f);
  const float im = ms >= 0x1p-126f ? __fdiv_rn(1.f, ms) : 0.f;
  const float iu = vs >= 0x1p-126f ? __fdiv_rn(1.f, vs) : 0.f;
  if (lane == 0) {
    e.m_scale[blk] = im > 0.f ? ms : 0.f;
    e.v_scale[blk] = iu > 0.f ? vs : 0.f;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const long long i = base + lane + 32 * j;
    if (i >= e.n) continue;
    const uint32_t h = mix((uint32_t)((unsigned long long)i >> 1) * kGolden + e.place);
    const uint32_t dither = ((i & 1 ? h >> 16 : h & 0xffffu) << 4) | 8u;
    const float rm = fminf(__fmul_rn(fabsf(m[j]), im), 448.f);
    const float ru = fminf(__fmul_rn(u[j], iu), 448.f);
    const float qm = rm > 0.f ? round_e4m3(rm, dither) : 0.f;
    const float qu = ru > 0.f ? fmaxf(round_e4m3(ru, dither), 0x1p-9f) : 0.f;
    ((uint8_t*)e.m)[i] = __nv_cvt_float_to_fp8(copysignf(qm, m[j]), __NV_SATFINITE, __NV_E4M3);
    ((uint8_t*)e.v)[i] = __nv_cvt_float_to_fp8(qu, __NV_SATFINITE, __NV_E4M3);
  }
}

__global__ void __launch_bounds__(AT) adamw_kernel(const __grid_constant__ AdamTable t) {
  float coef = 1.f;
  if (t.norm) {
    if (t.norm[2] == 0.f) return;      // some gradient is not finite: the step is skipped
    coef = t.norm[1];
  }
  const int wid = threadIdx.x >> 5;
  for (int c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const AdamEntry& e = t.e[entry_of(t, c)];
    const long long base = (long long)(c - e.first) * kChunk + wid * kBlock;
    if (base < e.n) step_block(e, t, base, coef);
  }
}

// ---------------------------------------------------------------- norm
// Block b's sum of squares over its chunks: fp32 over a thread's eight elements
// of a chunk, double from there.
__global__ void __launch_bounds__(AT) square_sums_kernel(const __grid_constant__ NormTable t,
                                                         double* __restrict__ sums) {
  __shared__ double red[AT / 32];
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  double sum = 0.0;
  for (int c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const NormEntry& e = t.e[entry_of(t, c)];
    const long long base = (long long)(c - e.first) * kChunk;
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const long long i = base + threadIdx.x + AT * j;
      if (i >= e.n) break;
      const float g = e.kind & kG16 ? __bfloat162float(((const __nv_bfloat16*)e.g)[i])
                                    : ((const float*)e.g)[i];
      s = fmaf(g, g, s);
    }
    sum += (double)s;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(kFull, sum, off);
  if (lane == 0) red[wid] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    double total = 0.0;
    for (int w = 0; w < AT / 32; ++w) total += red[w];
    sums[blockIdx.x] = total;
  }
}

__global__ void __launch_bounds__(AT) norm_kernel(const double* __restrict__ sums, int n,
                                                  float max_norm, float* __restrict__ norm) {
  __shared__ double red[AT];
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += AT) s += sums[i];
  red[threadIdx.x] = s;
  __syncthreads();
  for (int k = AT / 2; k > 0; k >>= 1) {
    if (threadIdx.x < k) red[threadIdx.x] += red[threadIdx.x + k];
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    const float v = (float)sqrt(red[0]);
    norm[0] = v;
    norm[1] = max_norm > 0.f ? fminf(max_norm / (v + 1e-6f), 1.f) : 1.f;
    norm[2] = isfinite(v) ? 1.f : 0.f;
    norm[3] = 0.f;
  }
}

int chunks_of(long long n) { return (int)((n + kChunk - 1) / kChunk); }
int grid_for(int chunks) { return chunks < kNormBlocks ? chunks : kNormBlocks; }
int grad_bits(const moe_adamw_tensor_t& x) { return x.g_dtype == MOE_BF16 ? kG16 : 0; }

// Calls launch(first tensor, past the last, chunks) for runs of tensors that fit
// one launch's parameter and chunk count.
template <typename F>
cudaError_t in_runs(const moe_adamw_tensor_t* x, int n, F launch) {
  for (int i = 0; i < n;) {
    int j = i;
    long long chunks = 0;
    while (j < n && j - i < kPerLaunch && chunks + chunks_of(x[j].n) < (1LL << 30))
      chunks += chunks_of(x[j++].n);
    if (chunks > 0) {
      const cudaError_t e = launch(i, j, (int)chunks);
      if (e != cudaSuccess) return e;
    }
    i = j;
  }
  return cudaSuccess;
}
}  // namespace

size_t grad_norm_ws_bytes(const moe_adamw_tensor_t* x, int n) {
  int runs = 0;
  (void)in_runs(x, n, [&](int, int, int) { ++runs; return cudaSuccess; });
  return align_up(sizeof(double) * kNormBlocks * (size_t)(runs > 0 ? runs : 1), 256);
}

cudaError_t launch_grad_norm(const moe_adamw_tensor_t* x, int n, float max_norm, float* norm,
                             void* ws, cudaStream_t s) {
  double* sums = static_cast<double*>(ws);
  int used = 0;
  const cudaError_t e = in_runs(x, n, [&](int i, int j, int chunks) {
    NormTable t;
    t.count = 0;
    t.chunks = chunks;
    int first = 0;
    for (int k = i; k < j; ++k) {
      if (x[k].n == 0) continue;
      t.e[t.count++] = {x[k].g, x[k].n, grad_bits(x[k]), first};
      first += chunks_of(x[k].n);
    }
    const int blocks = grid_for(chunks);
    square_sums_kernel<<<blocks, AT, 0, s>>>(t, sums + used);
    used += blocks;
    count_launches(1);
    return cudaGetLastError();
  });
  if (e != cudaSuccess) return e;
  norm_kernel<<<1, AT, 0, s>>>(sums, used, max_norm, norm);
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_adamw(const moe_adamw_tensor_t* x, int n, const moe_adamw_t& h,
                         const float* norm, cudaStream_t s) {
  return in_runs(x, n, [&](int i, int j, int chunks) {
    AdamTable t;
    t.count = 0;
    t.chunks = chunks;
    t.b1 = (float)h.beta1;
    t.b2 = (float)h.beta2;
    t.c1 = (float)(1.0 - h.beta1);
    t.c2 = (float)(1.0 - h.beta2);
    t.step_size = (float)(h.lr / (1.0 - pow(h.beta1, (double)h.step)));
    t.root = (float)(1.0 / sqrt(1.0 - pow(h.beta2, (double)h.step)));
    t.eps = (float)h.eps;
    t.norm = norm;
    int first = 0;
    for (int k = i; k < j; ++k) {
      if (x[k].n == 0) continue;
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
      e.kind = grad_bits(x[k]) | (x[k].p_dtype == MOE_BF16 ? kP16 : 0) |
               (x[k].state_bits == 8 ? kS8 : 0);
      e.first = first;
      first += chunks_of(x[k].n);
    }
    adamw_kernel<<<grid_for(chunks), AT, 0, s>>>(t);
    count_launches(1);
    return cudaGetLastError();
  });
}

}  // namespace moe
