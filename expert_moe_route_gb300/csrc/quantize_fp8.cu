// E4M3 codes and fp32 scales of a matrix, one scale per block of 128:
//   scale = largest |x| of the block / 448,   code = E4M3(x / scale)   (nearest even)
// A block is 128 elements of a row, 128 of a column, or a tile of 128 x 128.  Bound by HBM.
// A block of 256 threads takes one 128 x 128 tile: a thread holds eight neighbouring
// columns of eight rows, so the matrix is read once whichever forms are wanted, rows' maxima
// are shuffles among 16 lanes and columns' go through 4 KB of shared memory.
//
// The quotient is computed as q = x r, q + (x - q s) r with r = 1/s rounded to nearest
// (Markstein's correction of a quotient, 1990: the remainder is exact under fma): the
// rounded quotient, three operations where the compiler's division takes about ten, which
// would be more than the memory allows.  Scales whose remainders could leave the normal
// range are divided.
#include <algorithm>

#include "kernels.h"
#include "product_fp8.cuh"
#include "rows.cuh"

namespace moe {

namespace {
constexpr int QT = 256;
constexpr int BLK = 128;
constexpr float kMax = 448.f;
enum Form : int { ROWS = 1, COLS = 2, TILES = 4 };

// 1 / s for the quotients of a block, 0 for a scale of zero (all codes are 0 then, or NaN).
__device__ __forceinline__ float inverse(float s) { return s == 0.f ? 0.f : __frcp_rn(s); }
__device__ __forceinline__ bool plain_range(float s) {
  return s == 0.f || (s >= 0x1p-69f && s <= 0x1p69f);
}
__device__ __forceinline__ float quotient(float x, float s, float r) {
  const float q = x * r;
  return fmaf(fmaf(-q, s, x), r, q);
}

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// Eight codes of v with one scale.
__device__ __forceinline__ uint2 codes8(const float* v, float s, float r) {
  float q[8];
  if (plain_range(s)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = quotient(v[i], s, r);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = v[i] / s;
  }
  return make_uint2(codes4(q[0], q[1], q[2], q[3]), codes4(q[4], q[5], q[6], q[7]));
}

// Eight codes of v with a scale each.
__device__ __forceinline__ uint2 codes8(const float* v, const float* s, const float* r,
                                        bool plain) {
  float q[8];
  if (plain) {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = quotient(v[i], s[i], r[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (plain_range(s[i])) q[i] = quotient(v[i], s[i], r[i]);
      else q[i] = v[i] / s[i];
    }
  }
  return make_uint2(codes4(q[0], q[1], q[2], q[3]), codes4(q[4], q[5], q[6], q[7]));
}

// VEC: eight elements of x are one or two aligned accesses.
template <typename T, int FORM, bool VEC>
__global__ void __launch_bounds__(QT)
quantize_fp8_kernel(const T* __restrict__ x, long long ldx, long long n, int K, long long plane,
                    int row_tiles, int col_tiles, uint8_t* __restrict__ row_codes,
                    float* __restrict__ row_scales, uint8_t* __restrict__ col_codes,
                    float* __restrict__ col_scales) {
  using V = Vec<T, 8>;
  __shared__ float part[QT / 32][BLK];
  __shared__ float scales[BLK];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const long long id = blockIdx.x;
  const int ct = (int)(id % col_tiles);
  const long long rest = id / col_tiles;
  const int rt = (int)(rest % row_tiles);
  const long long e = rest / row_tiles;            // TILES: the matrix of the stack
  const long long r0 = (long long)rt * BLK;
  const int c = ct * BLK + (t & 15) * 8;
  const bool in_cols = c < K;
  const T* xe = x + e * plane;

  typename V::Raw raw[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const long long r = r0 + (t >> 4) + 16 * i;
    raw[i] = V::zero();
    if (in_cols && r < n) {
      const T* p = xe + r * ldx + c;
      if (VEC) {
        raw[i] = V::load(p);
      } else {
        T one[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) one[j] = p[j];
        memcpy(&raw[i], one, sizeof(one));
      }
    }
  }

  float top[8];                                    // per column (COLS), or top[0] (TILES)
#pragma unroll
  for (int j = 0; j < 8; ++j) top[j] = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float v[8];
    V::unpack(raw[i], v);
    if (FORM & COLS) {
#pragma unroll
      for (int j = 0; j < 8; ++j) top[j] = fmaxf(top[j], fabsf(v[j]));
    }
    if (FORM & (ROWS | TILES)) {
      float m = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[j]));
      if (FORM & TILES) {
        top[0] = fmaxf(top[0], m);
      } else {
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, off));
        const long long r = r0 + (t >> 4) + 16 * i;
        const float s = m / kMax;
        const uint2 q = codes8(v, s, inverse(s));
        if (in_cols && r < n) {
          *reinterpret_cast<uint2*>(row_codes + r * K + c) = q;
          if ((t & 15) == 0) row_scales[r * col_tiles + ct] = s;
        }
      }
    }
  }

  if (FORM & TILES) {
    float m = top[0];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, off));
    if (lane == 0) part[warp][0] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < QT / 32; ++w) m = fmaxf(m, part[w][0]);
    const float s = m / kMax, inv = inverse(s);
    if (t == 0) row_scales[id] = s;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const long long r = r0 + (t >> 4) + 16 * i;
      float v[8];
      V::unpack(raw[i], v);
      const uint2 q = codes8(v, s, inv);
      if (in_cols && r < n) *reinterpret_cast<uint2*>(row_codes + e * plane + r * K + c) = q;
    }
  }

  if (FORM & COLS) {
#pragma unroll
    for (int j = 0; j < 8; ++j) top[j] = fmaxf(top[j], __shfl_xor_sync(kFull, top[j], 16));
    if (lane < 16) {
#pragma unroll
      for (int j = 0; j < 8; j += 4)
        *reinterpret_cast<float4*>(&part[warp][lane * 8 + j]) =
            make_float4(top[j], top[j + 1], top[j + 2], top[j + 3]);
    }
    __syncthreads();
    if (t < BLK) {
      float m = 0.f;
#pragma unroll
      for (int w = 0; w < QT / 32; ++w) m = fmaxf(m, part[w][t]);
      const float s = m / kMax;
      scales[t] = s;
      if (ct * BLK + t < K) col_scales[(size_t)rt * K + ct * BLK + t] = s;
    }
    __syncthreads();
    float s[8], inv[8];
    bool plain = true;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      s[j] = scales[(t & 15) * 8 + j];
      inv[j] = inverse(s[j]);
      plain = plain && plain_range(s[j]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const long long r = r0 + (t >> 4) + 16 * i;
      float v[8];
      V::unpack(raw[i], v);
      const uint2 q = codes8(v, s, inv, plain);
      if (in_cols && r < n) *reinterpret_cast<uint2*>(col_codes + r * K + c) = q;
    }
  }
}

struct Call {
  const void* x;
  long long ldx, n, plane;
  int K, E;
  uint8_t* rc;
  float* rs;
  uint8_t* cc;
  float* cs;
};

template <typename T, int FORM>
cudaError_t launch_form(const Call& a, cudaStream_t s) {
  const int rt = (int)((a.n + BLK - 1) / BLK), ct = ceil_div(a.K, BLK);
  const long long blocks = (long long)a.E * rt * ct;
  if (blocks == 0) return cudaSuccess;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  const int align = sizeof(T) == 4 ? 32 : 16;      // of eight elements
  const bool vec = reinterpret_cast<uintptr_t>(a.x) % align == 0 &&
                   a.ldx * (long long)sizeof(T) % align == 0;
  const T* x = static_cast<const T*>(a.x);
  if (vec)
    quantize_fp8_kernel<T, FORM, true><<<(unsigned)blocks, QT, 0, s>>>(
        x, a.ldx, a.n, a.K, a.plane, rt, ct, a.rc, a.rs, a.cc, a.cs);
  else
    quantize_fp8_kernel<T, FORM, false><<<(unsigned)blocks, QT, 0, s>>>(
        x, a.ldx, a.n, a.K, a.plane, rt, ct, a.rc, a.rs, a.cc, a.cs);
  count_launches(1);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_typed(const Call& a, int form, cudaStream_t s) {
  switch (form) {
    case ROWS: return launch_form<T, ROWS>(a, s);
    case COLS: return launch_form<T, COLS>(a, s);
    case ROWS | COLS: return launch_form<T, ROWS | COLS>(a, s);
    default: return launch_form<T, TILES>(a, s);
  }
}

cudaError_t launch_any(const Call& a, int dtype, int form, cudaStream_t s) {
  switch (dtype) {
    case MOE_BF16: return launch_typed<__nv_bfloat16>(a, form, s);
    case MOE_F16: return launch_typed<__half>(a, form, s);
    default: return launch_typed<float>(a, form, s);
  }
}
}  // namespace

cudaError_t launch_quantize_fp8(const QuantizeArgs& a, cudaStream_t s) {
  const int form = (a.row_codes ? ROWS : 0) | (a.col_codes ? COLS : 0);
  if (form == 0 || a.n == 0) return cudaSuccess;
  const Call c{a.x, a.ldx, a.n, 0, a.K, 1, a.row_codes, a.row_scales, a.col_codes, a.col_scales};
  return launch_any(c, a.dtype, form, s);
}

cudaError_t launch_quantize_fp8_tiles(const void* x, int dtype, int E, int n, int K,
                                      uint8_t* codes, float* scales, cudaStream_t s) {
  const Call c{x, K, n, (long long)n * K, K, E, codes, scales, nullptr, nullptr};
  return launch_any(c, dtype, TILES, s);
}

}  // namespace moe
