// E4M3 codes and fp32 scales of a matrix, one scale per block of 128:
//   scale = largest |x| of the block / 448,   code = E4M3(x / scale)   (nearest even)
// A block is 128 elements of a row, 128 of a column, or a tile of 128 x 128.  Bound by HBM.
// A block of 256 threads takes one 128 x 128 tile: a thread holds 16 neighbouring columns of
// four rows, so the matrix is read once whichever forms are wanted, rows' maxima are shuffles
// among eight lanes (16-bit types: two rows a shuffle, two elements a maximum) and columns' go
// through 4 KB of shared memory.
//
// The quotient is computed as q = x r, q - (q s - x) r with r = 1/s rounded to nearest
// (Markstein's correction of a quotient, 1990: the remainder is exact under fma): the
// rounded quotient, three operations where the compiler's division takes about ten, which
// would be more than the memory allows.  The remainder has the sign with which a zero keeps its
// own: q s - x is +0, so that -0 is added to q.  Scales whose remainders could leave the normal
// range are divided.  Under a scale of 0 codes are zeros with the elements' signs, or NaN.
#include <type_traits>

#include "kernels.h"
#include "product_fp8.cuh"
#include "rows.cuh"

namespace moe {

namespace {
constexpr int QT = 256;
constexpr int BLK = 128;
constexpr float kMax = 448.f;
enum Form : int { ROWS = 1, COLS = 2, TILES = 4 };

// 1 / s for the quotients of a block, 0 for a scale of zero.  PAIRS: negative, see quotients.
template <bool PAIRS> __device__ __forceinline__ float inverse(float s) {
  const float r = s == 0.f ? 0.f : __frcp_rn(s);
  return PAIRS ? -r : r;
}
__device__ __forceinline__ bool plain_range(float s) {
  return s == 0.f || (s >= 0x1p-69f && s <= 0x1p69f);
}
__device__ __forceinline__ float quotient(float x, float s, float r) {
  const float q = x * r;
  return fmaf(-fmaf(q, s, -x), r, q);
}

// Two of them, negated: a pair of products or sums is one instruction, whose operands cannot
// change sign on their way in.  With r the negated inverses q is the negated quotient, x + q s is
// +0 for a zero, and times r -0.
__device__ __forceinline__ void quotients(const float* x, float s0, float s1, float r0, float r1,
                                          float* q) {
  asm("{\n\t.reg .b64 x, s, r, q;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 s, {%4, %5};\n\tmov.b64 r, {%6, %7};\n\t"
      "mul.rn.f32x2 q, x, r;\n\t"
      "fma.rn.f32x2 x, q, s, x;\n\t"
      "fma.rn.f32x2 q, x, r, q;\n\t"
      "mov.b64 {%0, %1}, q;\n\t}"
      : "=f"(q[0]), "=f"(q[1])
      : "f"(x[0]), "f"(x[1]), "f"(s0), "f"(s1), "f"(r0), "f"(r1));
}

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// x / s, a zero under a scale of zero (rare: kept out of the way of the kernel's registers).
__device__ __noinline__ float divided(float x, float s) { return s == 0.f ? x * 0.f : x / s; }

// Four codes of v with a scale each.  PAIRS: quotients two at a time, where both forms are made
// and instructions are what is short: bf16 131072 x 4096 403 us against 421.  With one form, bound by
// memory, the pairs' registers cost more than that: by row 263 against 240, by column 276 against 269.
// The pairs' negated quotients have their signs put right in the codes, four at a time; negated
// one by one before they are converted the two forms take 421 us.
template <bool PAIRS>
__device__ __forceinline__ uint32_t codes4_of(const float* v, const float4& s, const float4& r,
                                              bool plain) {
  if (plain && PAIRS) {
    float q[4];
    quotients(v, s.x, s.y, r.x, r.y, q);
    quotients(v + 2, s.z, s.w, r.z, r.w, q + 2);
    return codes4(q[0], q[1], q[2], q[3]) ^ 0x80808080u;
  }
  if (plain)
    return codes4(quotient(v[0], s.x, r.x), quotient(v[1], s.y, r.y), quotient(v[2], s.z, r.z),
                  quotient(v[3], s.w, r.w));
  return codes4(divided(v[0], s.x), divided(v[1], s.y), divided(v[2], s.z), divided(v[3], s.w));
}

// 16 codes of v with one scale.
template <bool PAIRS>
__device__ __forceinline__ uint4 codes16(const float* v, float s, float r) {
  const float4 s4 = make_float4(s, s, s, s), r4 = make_float4(r, r, r, r);
  const bool plain = plain_range(s);
  return make_uint4(codes4_of<PAIRS>(v, s4, r4, plain), codes4_of<PAIRS>(v + 4, s4, r4, plain),
                    codes4_of<PAIRS>(v + 8, s4, r4, plain), codes4_of<PAIRS>(v + 12, s4, r4, plain));
}

// 16 elements as 32-bit words, and maxima of magnitudes on words: two elements of a 16-bit
// type or one float.  NaN never wins.
template <typename T> struct Words {
  static constexpr int n = 16 * sizeof(T) / 4;
  static constexpr int per = 4 / sizeof(T);      // elements a word
  static __device__ __forceinline__ uint32_t magnitude(uint32_t w) {
    return w & (per == 2 ? 0x7fff7fffu : 0x7fffffffu);
  }
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
    if constexpr (per == 1) {
      return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    } else {
      using P = typename std::conditional<std::is_same<T, __half>::value, __half2,
                                          __nv_bfloat162>::type;
      const P m = __hmax2(*reinterpret_cast<const P*>(&a), *reinterpret_cast<const P*>(&b));
      return *reinterpret_cast<const uint32_t*>(&m);
    }
  }
  // element i (0 or 1) of a word
  static __device__ __forceinline__ float value(uint32_t w, int i) {
    if constexpr (per == 1) {
      return __uint_as_float(w);
    } else {
      const uint16_t h = (uint16_t)(w >> (16 * i));
      return to_f32(*reinterpret_cast<const T*>(&h));
    }
  }
  static __device__ __forceinline__ void unpack(const uint32_t* w, float* f) {
#pragma unroll
    for (int i = 0; i < 16; ++i) f[i] = value(w[i / per], i % per);
  }
};

__device__ __forceinline__ void ldg_nc_32(const void* p, uint32_t* v) {
  asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]),
                 "=r"(v[6]), "=r"(v[7])
               : "l"(p));
}

// VEC: 16 elements of x are aligned vectors of so many bytes, 32 or 16; 0: they are read one by
// one.  Vectors of 32 bytes read whole sectors: bf16 131072 x 4096 in both forms 403 us against 416,
// fp32 65536 x 4096 294 against 321.
template <typename T, int FORM, int VEC>
__global__ void __launch_bounds__(QT, sizeof(T) == 2 ? 4 : (FORM == ROWS ? 3 : 2))
quantize_fp8_kernel(const T* __restrict__ x, long long ldx, long long n, int K, long long plane,
                    int row_tiles, int col_tiles, uint8_t* __restrict__ row_codes,
                    float* __restrict__ row_scales, uint8_t* __restrict__ col_codes,
                    float* __restrict__ col_scales) {
  using W = Words<T>;
  constexpr bool kBoth = FORM == (ROWS | COLS);
  __shared__ float part[QT / 32][BLK];
  __shared__ float4 scales[BLK / 4], inverses[BLK / 4];   // of the columns
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const long long id = blockIdx.x;
  const int ct = (int)(id % col_tiles);
  const long long rest = id / col_tiles;
  const int rt = (int)(rest % row_tiles);
  const long long e = rest / row_tiles;            // TILES: the matrix of the stack
  const int c = ct * BLK + (t & 7) * 16;
  const bool in_cols = c < K;
  const long long r0 = (long long)rt * BLK + (t >> 3);   // rows r0, r0 + 32, ...
  const T* xe = x + e * plane + r0 * ldx + c;

  uint32_t raw[4][W::n];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int j = 0; j < W::n; ++j) raw[i][j] = 0;
    if (in_cols && r0 + 32 * i < n) {
      const T* p = xe + 32 * i * ldx;
      if constexpr (VEC > 0) {
#pragma unroll
        for (int j = 0; j < W::n; j += VEC / 4) {
          if constexpr (VEC == 32) {
            ldg_nc_32(p + j * W::per, raw[i] + j);
          } else {
            const uint4 v = ldg_nc_v4(p + j * W::per);
            raw[i][j] = v.x; raw[i][j + 1] = v.y; raw[i][j + 2] = v.z; raw[i][j + 3] = v.w;
          }
        }
      } else {
        T one[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) one[j] = p[j];
        memcpy(raw[i], one, sizeof(one));
      }
    }
  }

  if (FORM & (ROWS | TILES)) {
    float m[4];                                    // each row's largest magnitude
    {
      uint32_t top[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        top[i] = 0;
#pragma unroll
        for (int j = 0; j < W::n; ++j) top[i] = W::larger(top[i], W::magnitude(raw[i][j]));
      }
      if (W::per == 2) {                           // rows in pairs, one a half of a word
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          uint32_t both = W::larger(__byte_perm(top[i], top[i + 1], 0x5410),
                                    __byte_perm(top[i], top[i + 1], 0x7632));
#pragma unroll
          for (int off = 4; off > 0; off >>= 1)
            both = W::larger(both, __shfl_xor_sync(kFull, both, off));
          m[i] = W::value(both, 0);
          m[i + 1] = W::value(both, 1);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
          for (int off = 4; off > 0; off >>= 1)
            top[i] = W::larger(top[i], __shfl_xor_sync(kFull, top[i], off));
          m[i] = W::value(top[i], 0);
        }
      }
    }
    if (FORM & TILES) {
      float all = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
#pragma unroll
      for (int off = 16; off >= 8; off >>= 1) all = fmaxf(all, __shfl_xor_sync(kFull, all, off));
      if (lane == 0) part[warp][0] = all;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < QT / 32; ++w) all = fmaxf(all, part[w][0]);
#pragma unroll
      for (int i = 0; i < 4; ++i) m[i] = all;
    }
    float s = m[0] / kMax, inv = inverse<kBoth>(s);
    if ((FORM & TILES) && t == 0) row_scales[id] = s;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long r = r0 + 32 * i;
      if (i > 0 && !(FORM & TILES)) {
        s = m[i] / kMax;
        inv = inverse<kBoth>(s);
      }
      float v[16];
      W::unpack(raw[i], v);
      const uint4 q = codes16<kBoth>(v, s, inv);
      if (in_cols && r < n) {
        *reinterpret_cast<uint4*>(row_codes + e * plane + r * K + c) = q;
        if (!(FORM & TILES) && (t & 7) == 0) row_scales[r * col_tiles + ct] = s;
      }
    }
  }

  if (FORM & COLS) {
    // the words anew: the floats of the rows' codes are not kept (about 150 registers instead of 80)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < W::n; ++j) asm volatile("" : "+r"(raw[i][j]));
    uint32_t top[W::n];
#pragma unroll
    for (int j = 0; j < W::n; ++j) {
      top[j] = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) top[j] = W::larger(top[j], W::magnitude(raw[i][j]));
      top[j] = W::larger(top[j], __shfl_xor_sync(kFull, top[j], 8));
      top[j] = W::larger(top[j], __shfl_xor_sync(kFull, top[j], 16));
    }
    if (lane < 8) {
      float f[16];
      W::unpack(top, f);
#pragma unroll
      for (int j = 0; j < 16; j += 4)
        *reinterpret_cast<float4*>(&part[warp][lane * 16 + j]) =
            make_float4(f[j], f[j + 1], f[j + 2], f[j + 3]);
    }
    __syncthreads();
    bool plain = true;
    if (t < BLK) {
      float m = 0.f;
#pragma unroll
      for (int w = 0; w < QT / 32; ++w) m = fmaxf(m, part[w][t]);
      const float s = m / kMax;
      reinterpret_cast<float*>(scales)[t] = s;
      reinterpret_cast<float*>(inverses)[t] = inverse<kBoth>(s);
      plain = plain_range(s);
      if (ct * BLK + t < K) col_scales[(size_t)rt * K + ct * BLK + t] = s;
    }
    plain = __syncthreads_and(plain);
    uint32_t out[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {                  // four columns of the four rows
      const float4 s = scales[(t & 7) * 4 + j], inv = inverses[(t & 7) * 4 + j];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = W::value(raw[i][(4 * j + k) / W::per], (4 * j + k) % W::per);
        out[i][j] = codes4_of<kBoth>(v, s, inv, plain);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long r = r0 + 32 * i;
      if (in_cols && r < n)
        *reinterpret_cast<uint4*>(col_codes + r * K + c) =
            make_uint4(out[i][0], out[i][1], out[i][2], out[i][3]);
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
  const unsigned long long low =
      reinterpret_cast<uintptr_t>(a.x) | (unsigned long long)(a.ldx * (long long)sizeof(T));
  const T* x = static_cast<const T*>(a.x);
  auto kernel = low % 32 == 0   ? quantize_fp8_kernel<T, FORM, 32>
                : low % 16 == 0 ? quantize_fp8_kernel<T, FORM, 16>
                                : quantize_fp8_kernel<T, FORM, 0>;
  kernel<<<(unsigned)blocks, QT, 0, s>>>(x, a.ldx, a.n, a.K, a.plane, rt, ct, a.rc, a.rs, a.cc,
                                         a.cs);
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
