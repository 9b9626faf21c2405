// Routing by scores and its gradient.
//   s = sigmoid(l) or softmax(l) over the experts;  c = s + bias (without a bias: l, which
//   orders alike)
//   groups of E / G neighbouring experts: worth = sum of the 1 or 2 largest s + bias; the
//   experts of the top_groups best groups take part
//   idx = the R largest c, ties to the lower expert;  w = scale s_idx [/ sum of s_idx]
// An expert with logit -inf is closed: score 0, never chosen.  Where none is left, idx = -1
// and w = 0.
//
// The choice is that of c in 64 bits: two scores can lie closer to each other than 32 bits
// tell, about one token in two thousand at 256 experts.  The scores are computed in 32
// bits; a token two of whose values that decide lie within the error bound of each other
// (kNear below) is done again in 64 bits by choose_exact.  Equal logits under equal biases
// are equal in any precision and need no second look.
//
// A warp takes a token, a lane ceil(E/32) neighbouring experts, so the lower lane holds the
// lower experts and a ballot's first lane is the tie's winner.  Keys are compared as
// integers in the order of the floats (redux.sync).
#include <math.h>

#include <algorithm>

#include "kernels.h"
#include "route_scores.cuh"
#include "rows.cuh"

namespace moe {

namespace {
constexpr int RT = 256;                 // threads per block: eight tokens
constexpr int RW = RT / 32;

// Integers in the order of the floats; NaN first of all, -inf (closed) 0.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);   // -0 and 0 are equal
  const uint32_t o = b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
  return v != v ? 0xffffffffu : (v == -INFINITY ? 0u : o);
}
__device__ __forceinline__ float unordered(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ unsigned long long ordered(double v) {
  const unsigned long long b = (unsigned long long)__double_as_longlong(v + 0.0);
  const unsigned long long o = b ^ ((unsigned long long)((long long)b >> 63) | (1ull << 63));
  return v != v ? ~0ull : (v == -INFINITY ? 0ull : o);
}
__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(kFull, v); }
__device__ __forceinline__ unsigned long long warp_max(unsigned long long v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const unsigned long long o = __shfl_xor_sync(kFull, v, off);
    v = o > v ? o : v;
  }
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
  return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
  return v;
}

// Error bounds of the 32-bit keys.  A sigmoid by __expf and a fast quotient is within
// 2.5e-7 + 6e-8 of itself, a softmax within 9e-7 of the token's largest score; the bias's
// addition rounds by 2^-24 of the key.  Two keys whose distance is above
//   kNear * (largest score) + kRound * (larger key)
// are in the right order.
constexpr float kNearSigmoid = 1.0e-6f, kNearSoftmax = 2.5e-6f, kRound = 2.5e-7f;

struct RouteParams {
  long long ld;
  int T, E, R;
  int per;              // experts a lane
  int sigmoid, groups, top_groups, group_keys, renormalise;
  float scale;
  const float* bias;
};

// The whole choice in 64 bits, lane r < R receives its expert (or -1).
template <typename T, int EPL>
__device__ __noinline__ int choose_exact(const T* row, const RouteParams& p) {
  const int lane = threadIdx.x & 31;
  const int e0 = lane * p.per;
  double key[EPL], by[EPL];     // what groups are worth by, what experts are ordered by
  double top = -INFINITY;
  bool nan = false;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const bool here = j < p.per && e0 + j < p.E;
    by[j] = here ? (double)to_f32(row[e0 + j]) : -INFINITY;
    nan |= by[j] != by[j];
    top = fmax(top, by[j]);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) top = fmax(top, __shfl_xor_sync(kFull, top, off));
  if (__any_sync(kFull, nan)) top = NAN;
  double sum = 0.0;
  if (!p.sigmoid) {
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      key[j] = by[j] == -INFINITY ? 0.0 : exp(by[j] - top);
      sum += key[j];
    }
    sum = warp_sum(sum);
  }
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    double k = by[j];
    if (p.bias || p.group_keys == 2) {
      k = p.sigmoid ? 1.0 / (1.0 + exp(-by[j])) : key[j] / sum;
      if (p.bias && j < p.per && e0 + j < p.E) k += (double)p.bias[e0 + j];
      if (by[j] == -INFINITY) k = -INFINITY;
    }
    key[j] = k;
    if (p.bias) by[j] = k;
  }
  if (p.groups > 1) {
    const int per_group = p.E / p.groups;
    unsigned long long mine = 0;          // worth of group `lane`
    for (int g = 0; g < p.groups; ++g) {
      double a = -INFINITY, b = -INFINITY;
      bool bad = false;
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        const int e = e0 + j;
        if (j < p.per && e < p.E && e / per_group == g) {
          bad |= key[j] != key[j];
          b = fmax(b, fmin(a, key[j]));
          a = fmax(a, key[j]);
        }
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        const double oa = __shfl_xor_sync(kFull, a, off), ob = __shfl_xor_sync(kFull, b, off);
        b = fmax(fmin(a, oa), fmax(b, ob));
        a = fmax(a, oa);
      }
      bad = __any_sync(kFull, bad);
      const double worth = bad ? (double)NAN : (p.group_keys == 2 ? a + b : a);
      if (lane == g) mine = ordered(worth);
    }
    int before = 0;
    for (int g = 0; g < p.groups; ++g) {
      const unsigned long long o = __shfl_sync(kFull, mine, g);
      before += o > mine || (o == mine && g < lane);
    }
    const uint32_t kept = __ballot_sync(kFull, lane < p.groups && before < p.top_groups);
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const int e = e0 + j;
      if (j < p.per && e < p.E && !((kept >> (e / per_group)) & 1u)) by[j] = -INFINITY;
    }
  }
  uint32_t taken = 0;
  int mine = -1;
  for (int r = 0; r < p.R; ++r) {
    unsigned long long best = 0;
    int at = 0;
#pragma unroll
    for (int j = EPL - 1; j >= 0; --j) {
      const unsigned long long o = (taken >> j) & 1u ? 0ull : ordered(by[j]);
      if (o != 0 && o >= best) {
        best = o;
        at = j;
      }
    }
    const unsigned long long all = warp_max(best);
    if (all == 0) break;
    const int src = __ffs(__ballot_sync(kFull, best == all)) - 1;
    if (lane == src) taken |= 1u << at;
    const int e = __shfl_sync(kFull, e0 + at, src);
    if (lane == r) mine = e;
  }
  return mine;
}

// w of lane r < R's expert with logit x (here: it has one); m, sum: the token's largest
// logit and sum of exp(l - m), for a softmax over all experts.
__device__ __forceinline__ float weight_of(const RouteParams& p, float x, bool here, float m,
                                           float sum) {
  if (!p.renormalise) {
    float v;
    if (p.sigmoid) {
      const float z = expf(-fabsf(x));
      v = (x < 0.f ? z : 1.f) / (1.f + z);
    } else {
      v = expf(x - m) / sum;
    }
    return here ? v * p.scale : 0.f;
  }
  // shares of the chosen scores, scaled by the largest one's exponential: no sum underflows
  const float y = p.sigmoid ? fminf(x, 0.f) : x;
  float top = here ? y : -INFINITY;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
  float v = here ? expf(y - top) : 0.f;
  if (p.sigmoid && here) v = v / (1.f + expf(-fabsf(x)));
  const float total = warp_sum(v);
  return here ? v / total * p.scale : 0.f;
}

// VEC: a lane's experts are EPL = per elements in aligned vectors of four.
template <typename T, int EPL, bool VEC>
__device__ __forceinline__ void load_row(const T* row, const RouteParams& p, float (&x)[EPL]) {
  const int e0 = (threadIdx.x & 31) * p.per;
  if constexpr (VEC) {
#pragma unroll
    for (int j = 0; j < EPL; j += 4) Vec<T, 4>::unpack(Vec<T, 4>::load(row + e0 + j), x + j);
  } else {
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      x[j] = j < p.per && e0 + j < p.E ? to_f32(row[e0 + j]) : -INFINITY;
  }
}

// Largest logit of the token and the sum of exp(l - m), as needed for softmax scores.
template <int EPL>
__device__ __forceinline__ void softmax_parts(const float (&x)[EPL], float& m, float& sum) {
  m = -INFINITY;
  bool nan = false;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    m = fmaxf(m, x[j]);
    nan |= x[j] != x[j];
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, off));
  if (__any_sync(kFull, nan)) m = NAN;
  sum = 0.f;
#pragma unroll
  for (int j = 0; j < EPL; ++j) sum += x[j] == -INFINITY ? 0.f : expf(x[j] - m);
  sum = warp_sum(sum);
}

template <typename T, int EPL, bool VEC>
__global__ void __launch_bounds__(RT)
route_scores_kernel(const T* __restrict__ logits, const RouteParams p, int32_t* __restrict__ idx,
                    float* __restrict__ w) {
  extern __shared__ float group_keys_s[];    // groups > 1: a token's keys, E + 32 a warp
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int e0 = lane * p.per;
  const bool scored = p.bias != nullptr || p.group_keys == 2;   // keys are scores, not logits
  for (long long t = blockIdx.x * RW + warp; t < p.T; t += gridDim.x * RW) {
    const T* row = logits + t * p.ld;
    float x[EPL];
    load_row<T, EPL, VEC>(row, p, x);
    float m = 0.f, sum = 1.f;
    if (!p.sigmoid && (scored || !p.renormalise)) softmax_parts<EPL>(x, m, sum);
    // keys: what experts are ordered by (o), what groups are worth by (k)
    float k[EPL];
    uint32_t o[EPL];
    bool nan = false;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      k[j] = x[j];
      nan |= x[j] != x[j] || x[j] == INFINITY;
    }
    if (scored) {
      const float inv = 1.f / sum;
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        float v = p.sigmoid ? __fdividef(1.f, 1.f + __expf(-x[j])) : __expf(x[j] - m) * inv;
        if (p.bias && j < p.per && e0 + j < p.E) v += __ldg(p.bias + e0 + j);
        k[j] = x[j] == -INFINITY ? -INFINITY : v;
        nan |= k[j] != k[j];
      }
    }
    const float near = !scored ? -1.f : (p.sigmoid ? kNearSigmoid : kNearSoftmax / sum);
    bool again = __any_sync(kFull, nan);       // NaN and +inf: by the definition's arithmetic
#pragma unroll
    for (int j = 0; j < EPL; ++j) o[j] = ordered(p.bias ? k[j] : x[j]);

    if (p.groups > 1 && !again) {
      const int per_group = p.E / p.groups;
      int P = 1;                                // lanes a group
      while (2 * P * p.groups <= 32) P *= 2;
      float* ks = group_keys_s + warp * (p.E + 32);
      // a group's keys start P words apart from a multiple of its length: no bank conflicts
      {
        int g = e0 / per_group, left = per_group - (e0 - g * per_group);
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
          if (j < p.per && e0 + j < p.E) ks[e0 + j + g * P] = k[j];
          if (--left == 0) {
            ++g;
            left = per_group;
          }
        }
      }
      __syncwarp();
      const int g = lane / P;
      float a = -INFINITY, b = -INFINITY;
      if (g < p.groups)
        for (int i = lane % P; i < per_group; i += P) {
          const float v = ks[g * (per_group + P) + i];
          b = fmaxf(b, fminf(a, v));
          a = fmaxf(a, v);
        }
      for (int off = P / 2; off > 0; off >>= 1) {
        const float oa = __shfl_xor_sync(kFull, a, off), ob = __shfl_xor_sync(kFull, b, off);
        b = fmaxf(fminf(a, oa), fmaxf(b, ob));
        a = fmaxf(a, oa);
      }
      __syncwarp();
      const float worth = p.group_keys == 2 ? a + b : a;
      int before = 0;
      for (int j = 0; j < p.groups; ++j) {
        const float other = __shfl_sync(kFull, worth, j * P);
        before += other > worth || (other == worth && j < g);
      }
      const bool first = lane % P == 0 && g < p.groups;
      const uint32_t kept = __ballot_sync(kFull, first && before < p.top_groups);
      if (scored && p.top_groups < p.groups) {
        const int in = __ffs(__ballot_sync(kFull, first && before == p.top_groups - 1)) - 1;
        const int out = __ffs(__ballot_sync(kFull, first && before == p.top_groups)) - 1;
        const float hi = __shfl_sync(kFull, worth, in), lo = __shfl_sync(kFull, worth, out);
        again = lo > -INFINITY && hi - lo <= 2.f * near + 2.f * kRound * fmaxf(fabsf(hi), fabsf(lo));
      }
      int ge = e0 / per_group, left = per_group - (e0 - ge * per_group);
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        if (j < p.per && ge < p.groups && !((kept >> (ge * P)) & 1u)) o[j] = 0;
        if (--left == 0) {
          ++ge;
          left = per_group;
        }
      }
    }

    int mine = -1;
    if (!again) {
      uint32_t last = 0;
      int last_e = 0;
      for (int r = 0; r <= p.R; ++r) {          // one more: the first that is left out
        uint32_t best = 0;
#pragma unroll
        for (int j = 0; j < EPL; ++j) best = max(best, o[j]);
        const uint32_t all = warp_max(best);
        if (all == 0) break;
        const int src = __ffs(__ballot_sync(kFull, best == all)) - 1;
        int at = 0;
#pragma unroll
        for (int j = EPL - 1; j >= 0; --j)
          if (o[j] == all) at = j;
        const int e = __shfl_sync(kFull, e0 + at, src);
        if (p.bias && r > 0) {
          const float hi = unordered(last), lo = unordered(all);
          if (hi - lo <= near + kRound * fmaxf(fabsf(hi), fabsf(lo)) &&
              (to_f32(row[e]) != to_f32(row[last_e]) || p.bias[e] != p.bias[last_e])) {
            again = true;
            break;
          }
        }
        if (lane == src) {
#pragma unroll
          for (int j = 0; j < EPL; ++j)
            if (j == at) o[j] = 0;
        }
        if (lane == r && r < p.R) mine = e;
        last = all;
        last_e = e;
      }
    }
    if (again) mine = choose_exact<T, EPL>(row, p);
    const bool here = lane < p.R && mine >= 0;
    const float xm = here ? to_f32(row[mine]) : 0.f;
    const float v = weight_of(p, xm, here, m, sum);
    if (lane < p.R) {
      idx[t * p.R + lane] = mine;
      w[t * p.R + lane] = v;
    }
  }
}

// dlogits of a token, all E of them.  DENSE (softmax over all experts, not renormalised):
// p_e (g_e - sum_j g_j p_j), every expert.  Otherwise the chosen experts alone have one:
//   renormalised: scale u_r (g_r - sum_j g_j u_j) with shares u, times 1 - sigmoid(l) for a
//   sigmoid;  a sigmoid alone: scale g s (1 - s)
template <typename T, int EPL, bool VEC, bool DENSE>
__global__ void __launch_bounds__(RT)
route_scores_bwd_kernel(const T* __restrict__ logits, const RouteParams p,
                        const int32_t* __restrict__ idx, const float* __restrict__ dw,
                        T* __restrict__ dlogits, long long ld_out) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int e0 = lane * p.per;
  for (long long t = blockIdx.x * RW + warp; t < p.T; t += gridDim.x * RW) {
    const T* row = logits + t * p.ld;
    T* out = dlogits + t * ld_out;
    int e = lane < p.R ? idx[t * p.R + lane] : -1;
    if ((unsigned)e >= (unsigned)p.E) e = -1;
    float x = e >= 0 ? to_f32(row[e]) : -INFINITY;
    const bool here = x != -INFINITY;       // an empty slot or a closed expert: no gradient
    if (!here) x = 0.f;
    const float g = here ? dw[t * p.R + lane] * p.scale : 0.f;
    float d, m = 0.f, sum = 1.f;
    float v[EPL];
    float dot = 0.f;
    if (DENSE) {
      load_row<T, EPL, VEC>(row, p, v);
      softmax_parts<EPL>(v, m, sum);
      const float s = here ? expf(x - m) / sum : 0.f;
      dot = warp_sum(here ? g * s : 0.f);
      d = s * g;
      const float inv = 1.f / sum;
#pragma unroll
      for (int j = 0; j < EPL; ++j) v[j] = v[j] == -INFINITY ? 0.f : -expf(v[j] - m) * inv * dot;
    } else if (p.renormalise) {
      RouteParams one = p;
      one.scale = 1.f;
      const float u = weight_of(one, x, here, m, sum);
      dot = warp_sum(here ? g * u : 0.f);
      d = u * (g - dot);
      if (p.sigmoid) d /= 1.f + expf(x);
    } else {
      const float z = expf(-fabsf(x));
      d = g * z / ((1.f + z) * (1.f + z));
    }
    // an expert named twice gets both
    float all = 0.f;
    bool first = here;      // the lowest slot that names this expert
    for (int r = 0; r < p.R; ++r) {
      const int er = __shfl_sync(kFull, e, r);
      const float dr = __shfl_sync(kFull, d, r);
      if (er == e && here) {
        all += dr;
        if (r < lane) first = false;
      }
    }
    if (DENSE) {
      if constexpr (VEC) {
#pragma unroll
        for (int j = 0; j < EPL; j += 4)
          Vec<T, 4>::store(out + e0 + j, Vec<T, 4>::pack(v + j));
      } else {
#pragma unroll
        for (int j = 0; j < EPL; ++j)
          if (j < p.per && e0 + j < p.E) out[e0 + j] = from_f32<T>(v[j]);
      }
      if (first) all -= expf(x - m) / sum * dot;
    } else {
      for (int j = lane; j < p.E; j += 32) out[j] = from_f32<T>(0.f);
    }
    __syncwarp();     // the chosen experts' values come after the row's
    if (first) out[e] = from_f32<T>(all);
  }
}

RouteParams params_of(const ScoresArgs& a) {
  const moe_router_t& r = a.router;
  return {a.ld, a.T, a.E, a.R, ceil_div(a.E, 32), r.score == MOE_SCORE_SIGMOID, r.groups,
          r.top_groups, r.group_keys, r.renormalise != 0, r.scale, a.bias};
}

int blocks_of(int T) { return (int)std::min<long long>(((long long)T + RW - 1) / RW, 152 * 16); }

// A row's experts in vectors of four: E = 32 EPL, rows and base aligned to four elements.
template <typename T>
bool vectors(const void* p, long long ld, int E) {
  return E % 128 == 0 && reinterpret_cast<uintptr_t>(p) % (4 * sizeof(T)) == 0 && ld % 4 == 0;
}

// Calls f(std::integral_constant EPL, vec) for the smallest EPL that holds E experts.
#define MOE_EPL(E, CALL)                      \
  do {                                        \
    const int per_ = ceil_div(E, 32);         \
    if (per_ <= 2) { CALL(2); }               \
    else if (per_ <= 4) { CALL(4); }          \
    else if (per_ <= 8) { CALL(8); }          \
    else if (per_ <= 12) { CALL(12); }        \
    else if (per_ <= 16) { CALL(16); }        \
    else { CALL(32); }                        \
  } while (0)

template <typename T>
cudaError_t route_typed(const ScoresArgs& a, int32_t* idx, float* w, cudaStream_t s) {
  const RouteParams p = params_of(a);
  const T* l = static_cast<const T*>(a.logits);
  const size_t smem = p.groups > 1 ? (size_t)RW * (a.E + 32) * sizeof(float) : 0;
  const bool vec = vectors<T>(a.logits, a.ld, a.E);
#define MOE_ROUTE(N)                                                                       \
  if (vec && p.per == N && N % 4 == 0)                                                     \
    route_scores_kernel<T, N, N % 4 == 0><<<blocks_of(a.T), RT, smem, s>>>(l, p, idx, w);  \
  else                                                                                     \
    route_scores_kernel<T, N, false><<<blocks_of(a.T), RT, smem, s>>>(l, p, idx, w)
  MOE_EPL(a.E, MOE_ROUTE);
#undef MOE_ROUTE
  count_launches(1);
  return cudaGetLastError();
}

template <typename T>
cudaError_t bwd_typed(const ScoresArgs& a, const int32_t* idx, const float* dw, void* out,
                      long long ld_out, cudaStream_t s) {
  const RouteParams p = params_of(a);
  const T* l = static_cast<const T*>(a.logits);
  T* o = static_cast<T*>(out);
  if (p.sigmoid || p.renormalise) {
    route_scores_bwd_kernel<T, 1, false, false>
        <<<blocks_of(a.T), RT, 0, s>>>(l, p, idx, dw, o, ld_out);
  } else {
    const bool vec = vectors<T>(a.logits, a.ld, a.E) && vectors<T>(out, ld_out, a.E);
#define MOE_ROUTE(N)                                                                      \
  if (vec && p.per == N && N % 4 == 0)                                                    \
    route_scores_bwd_kernel<T, N, N % 4 == 0, true>                                       \
        <<<blocks_of(a.T), RT, 0, s>>>(l, p, idx, dw, o, ld_out);                         \
  else                                                                                    \
    route_scores_bwd_kernel<T, N, false, true>                                            \
        <<<blocks_of(a.T), RT, 0, s>>>(l, p, idx, dw, o, ld_out)
    MOE_EPL(a.E, MOE_ROUTE);
#undef MOE_ROUTE
  }
  count_launches(1);
  return cudaGetLastError();
}
}  // namespace

cudaError_t launch_route_scores(const ScoresArgs& a, int32_t* idx, float* w, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  switch (a.dtype) {
    case MOE_BF16: return route_typed<__nv_bfloat16>(a, idx, w, s);
    case MOE_F16: return route_typed<__half>(a, idx, w, s);
    default: return route_typed<float>(a, idx, w, s);
  }
}

cudaError_t launch_route_scores_bwd(const ScoresArgs& a, const int32_t* idx, const float* dw,
                                    void* dlogits, long long ld_dlogits, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  switch (a.dtype) {
    case MOE_BF16: return bwd_typed<__nv_bfloat16>(a, idx, dw, dlogits, ld_dlogits, s);
    case MOE_F16: return bwd_typed<__half>(a, idx, dw, dlogits, ld_dlogits, s);
    default: return bwd_typed<float>(a, idx, dw, dlogits, ld_dlogits, s);
  }
}

}  // namespace moe
