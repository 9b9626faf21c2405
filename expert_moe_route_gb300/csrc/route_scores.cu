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
// tell, about one token in five hundred of 384 normal logits.  The scores are computed in 32 bits;
// where two that follow each other lie within the error bound (kNear below), experts are taken
// on until a gap, and those taken are put in order by their keys in 64 bits, a lane each.
// Equal logits under equal biases are equal in any precision and need no second look.
//
// A warp takes a token, a lane up to EPL of its experts.  A key becomes one 32-bit integer:
// its distance below the largest in 2^23 steps of the keys' range (2^22 where a lane holds 32),
// then the expert, so that the warp's smallest integer (redux.sync) is the next expert and ties
// go to the lower one by themselves.  A lane keeps its three smallest in order and finds the
// next three when they are taken (4% of the tokens, 8 of 384 experts).  Groups whose worths lie
// within the error bound are put in order in 64 bits (groups_exact, a lane an expert at a time).
// A token whose keys are not finite or with more than 32 experts in a row within the bound goes to
// choose_exact, all of it in 64 bits, and takes 37 us there: kernels that send it one late end
// late (65536 x 256 in 8 groups: 93 us; without groups_exact 4 to 31 more).  A bias that is not
// finite sends every token there, as does a finite key so far below the others that these share
// the steps of the range: 65536 x 256, one bias of -inf 1678 us against 49, a tenth of the logits
// at -1e9 and no bias 1583 against 50 (52 with them at -inf).
// Bound by the issue of instructions: 65536 tokens x 384 experts, sigmoid and bias, 56 us (15.6
// at the copy rate).
#include <float.h>
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
__device__ __forceinline__ uint32_t sortable(float v) {   // of numbers; -0 below 0
  const uint32_t b = __float_as_uint(v);
  return b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t o = sortable(v + 0.f);   // -0 and 0 are equal
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
// are in the right order.  A group's worth is within kNear * (largest score) + kRound * (the
// magnitudes of its one or two keys) of itself: of its keys, which may cancel in the sum.
constexpr float kNearSigmoid = 1.0e-6f, kNearSoftmax = 2.5e-6f, kRound = 2.5e-7f;
constexpr uint32_t kNone = 0xffffffffu;   // no expert
constexpr uint32_t kMinusInf = 0x007fffffu;   // sortable(-inf)

struct RouteParams {
  long long ld;
  int T, E, R;
  int sigmoid, groups, top_groups, group_keys, renormalise;
  float scale;
  const float* bias;
};

// A lane's expert j.  VEC: vectors of four neighbours, 128 experts a warp's load; else 32.
template <bool VEC> __device__ __forceinline__ int expert_of(int j) {
  const int lane = threadIdx.x & 31;
  return VEC ? (j / 4) * 128 + lane * 4 + j % 4 : j * 32 + lane;
}

// The whole choice in 64 bits, lane r < R receives its expert (or -1).
template <typename T>
__device__ __noinline__ int choose_exact(const T* row, const RouteParams& p) {
  const int lane = threadIdx.x & 31;
  const int n = (p.E + 31) / 32;          // this lane's experts are lane, lane + 32, ...
  double key[32], by[32];       // what groups are worth by, what experts are ordered by
  double top = -INFINITY;
  bool nan = false;
#pragma unroll 1
  for (int j = 0; j < n; ++j) {
    const int e = j * 32 + lane;
    by[j] = e < p.E ? (double)to_f32(row[e]) : -INFINITY;
    nan |= by[j] != by[j];
    top = fmax(top, by[j]);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) top = fmax(top, __shfl_xor_sync(kFull, top, off));
  if (__any_sync(kFull, nan)) top = NAN;
  double sum = 0.0;
  if (!p.sigmoid) {
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
      key[j] = by[j] == -INFINITY ? 0.0 : exp(by[j] - top);
      sum += key[j];
    }
    sum = warp_sum(sum);
  }
#pragma unroll 1
  for (int j = 0; j < n; ++j) {
    const int e = j * 32 + lane;
    double k = by[j];
    if (p.bias || p.group_keys == 2) {
      k = p.sigmoid ? 1.0 / (1.0 + exp(-by[j])) : key[j] / sum;
      if (p.bias && e < p.E) k += (double)p.bias[e];
      if (by[j] == -INFINITY) k = -INFINITY;
    }
    key[j] = k;
    if (p.bias) by[j] = k;
  }
  if (p.groups > 1) {
    const int per_group = p.E / p.groups;
    unsigned long long mine = 0;          // worth of group `lane`
#pragma unroll 1
    for (int g = 0; g < p.groups; ++g) {
      double a = -INFINITY, b = -INFINITY;
      bool bad = false;
#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        const int e = j * 32 + lane;
        if (e < p.E && e / per_group == g) {
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
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
      const int e = j * 32 + lane;
      if (e < p.E && !((kept >> (e / per_group)) & 1u)) by[j] = -INFINITY;
    }
  }
  uint32_t taken = 0;
  int mine = -1;
#pragma unroll 1
  for (int r = 0; r < p.R; ++r) {
    unsigned long long best = 0;
    int at = 0;                           // this lane's lowest expert with its best key
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
      const unsigned long long o = (taken >> j) & 1u ? 0ull : ordered(by[j]);
      if (o > best) {
        best = o;
        at = j;
      }
    }
    const unsigned long long all = warp_max(best);
    if (all == 0) break;
    const int e = __reduce_min_sync(kFull, best == all ? at * 32 + lane : 0x7fffffff);
    if (best == all && e == at * 32 + lane) taken |= 1u << at;
    if (lane == r) mine = e;
  }
  return mine;
}

// Largest logit of a token and the sum of exp(l - top), in 64 bits.
template <typename T>
__device__ __forceinline__ void softmax_parts64(const T* row, int E, double& top, double& sum) {
  const int lane = threadIdx.x & 31;
  top = -INFINITY;
  sum = 0.0;
#pragma unroll 1
  for (int e = lane; e < E; e += 32) top = fmax(top, (double)to_f32(row[e]));
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) top = fmax(top, __shfl_xor_sync(kFull, top, off));
#pragma unroll 1
  for (int e = lane; e < E; e += 32) sum += exp((double)to_f32(row[e]) - top);
  sum = warp_sum(sum);
}

// The groups that take part, bits P g of group g, where worths in 32 bits do not tell (lane P g:
// of group g): those that are `sure` do, the rest are the best of the `open`, in order in 64 bits.
template <typename T>
__device__ __noinline__ uint32_t groups_exact(const T* row, const RouteParams& p, int P, bool sure,
                                              bool open) {
  const int lane = threadIdx.x & 31, per_group = p.E / p.groups;
  const uint32_t in = __ballot_sync(kFull, sure);
  const uint32_t all = __ballot_sync(kFull, open);
  double top = 0.0, sum = 1.0;
  if (!p.sigmoid) softmax_parts64(row, p.E, top, sum);
  unsigned long long mine = 0;
  for (uint32_t left = all; left; left &= left - 1) {
    const int at = __ffs(left) - 1, e0 = at / P * per_group;
    double a = -INFINITY, b = -INFINITY;
#pragma unroll 1
    for (int e = e0 + lane; e < e0 + per_group; e += 32) {
      const double l = (double)to_f32(row[e]);
      double key = p.sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - top) / sum;
      if (p.bias) key += (double)p.bias[e];
      if (l == -INFINITY) key = -INFINITY;
      b = fmax(b, fmin(a, key));
      a = fmax(a, key);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const double oa = __shfl_xor_sync(kFull, a, off), ob = __shfl_xor_sync(kFull, b, off);
      b = fmax(fmin(a, oa), fmax(b, ob));
      a = fmax(a, oa);
    }
    if (lane == at) mine = ordered(p.group_keys == 2 ? a + b : a);
  }
  int before = __popc(in);
  for (uint32_t left = all; left; left &= left - 1) {
    const int at = __ffs(left) - 1;
    const unsigned long long o = __shfl_sync(kFull, mine, at);
    before += o > mine || (o == mine && at < lane);
  }
  return in | __ballot_sync(kFull, open && before < p.top_groups);
}

// Experts of the lanes (or -1) in the order of their keys in 64 bits: lane r receives the r-th.
template <typename T>
__device__ __noinline__ int order_exact(const T* row, const RouteParams& p, int e) {
  const int lane = threadIdx.x & 31;
  const double l = e >= 0 ? (double)to_f32(row[e]) : -INFINITY;
  double key = l;
  if (p.bias) {
    if (p.sigmoid) {
      key = 1.0 / (1.0 + exp(-l));
    } else {
      double top, sum;
      softmax_parts64(row, p.E, top, sum);
      key = exp(l - top) / sum;
    }
    key += e >= 0 ? (double)p.bias[e] : 0.0;
  }
  int place = 0;
  for (int j = 0; j < 32; ++j) {
    const double o = __shfl_sync(kFull, key, j);
    const int oe = __shfl_sync(kFull, e, j);
    place += oe >= 0 && (o > key || (o == key && oe < e));
  }
  int mine = -1;
  for (int j = 0; j < 32; ++j) {
    const int at = __shfl_sync(kFull, place, j), oe = __shfl_sync(kFull, e, j);
    if (oe >= 0 && at == lane) mine = oe;
  }
  return mine;
}

// Sum over a token's slots (lanes 0 .. R - 1, R <= 2 half), the same in every lane.
__device__ __forceinline__ float slot_sum(float v, int half) {
  for (int off = half; off > 0; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
  return __shfl_sync(kFull, v, 0);
}

// w of lane r < R's expert with logit x (here: it has one); m, sum: the token's largest
// logit and sum of exp(l - m), for a softmax over all experts.  half: see slot_sum.
__device__ __forceinline__ float weight_of(const RouteParams& p, float x, bool here, float m,
                                           float sum, int half) {
  float v = 0.f;
  if (p.sigmoid) {
    const float z = expf(-fabsf(x));
    v = here ? (x < 0.f ? z : 1.f) / (1.f + z) : 0.f;
    if (!p.renormalise) return v * p.scale;
  } else if (!p.renormalise) {
    return here ? expf(x - m) / sum * p.scale : 0.f;
  }
  float total = p.sigmoid ? slot_sum(v, half) : 0.f;
  if (!(total >= 1e-20f)) {
    // shares of the chosen scores (of a softmax, or so small that their sum underflows),
    // scaled by the largest one's exponential
    const float y = p.sigmoid ? fminf(x, 0.f) : x;
    float top = here ? y : -INFINITY;
    for (int off = half; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
    v = here ? expf(y - top) : 0.f;
    if (p.sigmoid && here) v = v / (1.f + expf(-fabsf(x)));
    total = slot_sum(v, half);
  }
  return here ? v / total * p.scale : 0.f;
}

template <typename T, int EPL, bool VEC>
__device__ __forceinline__ void load_row(const T* row, const RouteParams& p, float (&x)[EPL]) {
  if constexpr (VEC) {
#pragma unroll
    for (int j = 0; j < EPL; j += 4) {
      x[j] = x[j + 1] = x[j + 2] = x[j + 3] = -INFINITY;
      const int e = expert_of<VEC>(j);
      if (e < p.E) Vec<T, 4>::unpack(Vec<T, 4>::load(row + e), x + j);
    }
  } else {
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const int e = expert_of<VEC>(j);
      x[j] = e < p.E ? to_f32(row[e]) : -INFINITY;
    }
  }
}

// Largest logit of the token and the sum of exp(l - m), as needed for softmax scores; KEEP:
// x becomes exp(l - m).
template <int EPL, bool KEEP>
__device__ __forceinline__ void softmax_parts(float (&x)[EPL], float& m, float& sum) {
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
  for (int j = 0; j < EPL; ++j) {
    const float z = x[j] == -INFINITY ? 0.f : expf(x[j] - m);
    sum += z;
    if (KEEP) x[j] = z;
  }
  sum = warp_sum(sum);
}

// 1 / (1 + exp(-x)) within 2.5e-7 + 6e-8 of itself, 0 for -inf.
__device__ __forceinline__ float fast_sigmoid(float x) {
  float z, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(z) : "f"(x * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + z));
  return r;
}

// The three smallest of those of v that are above `floor` (all: floor = 0, for v > 0), in
// order.
template <int EPL>
__device__ __forceinline__ void smallest_three(const uint32_t (&v)[EPL], uint32_t floor,
                                               uint32_t (&s)[3]) {
  s[0] = s[1] = s[2] = kNone;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    uint32_t x = floor == 0 || v[j] > floor ? v[j] : kNone;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      if (i > j) break;
      const uint32_t lo = min(s[i], x);
      x = max(s[i], x);
      s[i] = lo;
    }
  }
}

// A bound of keys' distances in steps, as a difference of their integers.
__device__ __forceinline__ uint32_t within(float bound, float steps, int bits) {
  return bound < steps ? (uint32_t)bound << bits : 0xffffffffu;
}

// What a call's keys are: logits or scores of one group; of several groups; sigmoid scores
// with a bias and one group, whose integer is one fma of the score, since every token's keys
// are in [lowest bias, 1 + highest bias].
enum Keys : int { ANY = 0, GROUPED = 1, BIASED = 2 };

// Blocks an SM: choose_exact, rare, would else set the registers of all.
template <typename T, int EPL, bool VEC, int KEYS>
__global__ void __launch_bounds__(RT, EPL <= 8 || (EPL <= 12 && KEYS == BIASED) ? 4 : (EPL <= 16 ? 3 : 2))
route_scores_kernel(const T* __restrict__ logits, const RouteParams p, int32_t* __restrict__ idx,
                    float* __restrict__ w) {
  extern __shared__ float group_keys_s[];    // GROUPED: a token's keys, E + 32 a warp
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool biased = KEYS == BIASED || p.bias != nullptr;
  const bool scored = biased || p.group_keys == 2;   // keys are scores, not logits
  constexpr int bits = EPL <= 16 ? 9 : 10;   // of an expert's number
  constexpr float steps = (float)(1 << (32 - bits)) - 72.f;
  constexpr float kMagic = 8388608.f + 64.f; // distances start at 64: the first is near none
  int half = 1;
  while (2 * half < p.R) half *= 2;
  float bias[EPL];
  bool bad_bias = false;
  float b_hi = -INFINITY, b_lo = INFINITY;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = expert_of<VEC>(j);
    bias[j] = biased && e < p.E ? p.bias[e] : 0.f;
    bad_bias |= !(fabsf(bias[j]) < 1e30f);   // (sums of two are finite)
    if (e < p.E) {
      b_hi = fmaxf(b_hi, bias[j]);
      b_lo = fminf(b_lo, bias[j]);
    }
  }
  bad_bias = __any_sync(kFull, bad_bias);
  float f_scale = 0.f;
  uint32_t close = 0;                        // distances up to this may be in the wrong order
  if constexpr (KEYS == BIASED) {
    b_hi = unordered(__reduce_max_sync(kFull, ordered(b_hi)));
    b_lo = unordered(__reduce_min_sync(kFull, ordered(b_lo)));
    f_scale = steps / (1.f + (b_hi - b_lo));
#pragma unroll
    for (int j = 0; j < EPL; ++j) bias[j] = fmaf(1.f + (b_hi - bias[j]), f_scale, kMagic);
    // two keys' distances: the offsets' two roundings, theirs to whole steps and the sum's, each
    // half a step, are 4 steps; a key in 64 bits is rounded to 2^-53 of itself
    const float most = fmaxf(fabsf(b_hi), fabsf(b_lo)) + 1.f;
    close = within((kNearSigmoid + 1e-15f * most) * f_scale + 6.f, steps, bits);
  }
  int P = 1, per_group = p.E;                // groups: lanes each, and experts
  uint8_t place[KEYS == GROUPED ? EPL : 1];  // P times the expert's group
  if constexpr (KEYS == GROUPED) {
    per_group = p.E / p.groups;
    while (2 * P * p.groups <= 32) P *= 2;
#pragma unroll
    for (int j = 0; j < EPL; ++j) place[j] = (uint8_t)(expert_of<VEC>(j) / per_group * P);
  }
  for (long long t = blockIdx.x * RW + warp; t < p.T; t += gridDim.x * RW) {
    const T* row = logits + t * p.ld;
    float k[EPL];                            // keys, first of all the logits
    load_row<T, EPL, VEC>(row, p, k);
    float m = 0.f, sum = 1.f;
    if (KEYS != BIASED && !p.sigmoid && (scored || !p.renormalise))
      softmax_parts<EPL, false>(k, m, sum);
    bool odd = false;                        // NaN or +inf: by the definition's arithmetic
#pragma unroll
    for (int j = 0; j < EPL; ++j) odd |= !(k[j] < INFINITY);
    odd = __any_sync(kFull, odd);
    bool again = odd || bad_bias;

    uint32_t v[EPL];                         // keys as integers
    if constexpr (KEYS == BIASED) {
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        const uint32_t d = __float_as_uint(fmaf(fast_sigmoid(k[j]), -f_scale, bias[j]));
        v[j] = k[j] == -INFINITY ? kNone : d << bits | (uint32_t)expert_of<VEC>(j);
      }
    } else {
      float near = 0.f;                      // error bound of a difference of two keys
      if (scored) {
        const float inv = 1.f / sum;
        near = p.sigmoid ? kNearSigmoid : kNearSoftmax * inv;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
          const float s = p.sigmoid ? fast_sigmoid(k[j]) : __expf(k[j] - m) * inv;
          k[j] = k[j] == -INFINITY ? k[j] : s + bias[j];
        }
      }
      if constexpr (KEYS == GROUPED) {
        float* ks = group_keys_s + warp * (p.E + 32);
        // a group's keys start P words apart from a multiple of its length: no bank conflicts
#pragma unroll
        for (int j = 0; j < EPL; ++j)
          if (expert_of<VEC>(j) < p.E) ks[expert_of<VEC>(j) + place[j]] = k[j];
        __syncwarp();
        const int g = lane / P;
        float a = -INFINITY, b = -INFINITY;
        if (g < p.groups)
          for (int i = lane % P; i < per_group; i += P) {
            const float key = ks[g * (per_group + P) + i];
            b = fmaxf(b, fminf(a, key));
            a = fmaxf(a, key);
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
        // bits P g of the groups that take part
        uint32_t kept = __ballot_sync(kFull, first && before < p.top_groups);
        if (scored && p.top_groups < p.groups && !again) {
          // Each worth lies between `least` and `most` (-inf: the group is closed).  A group is
          // in for sure above all that are out, and out below all that are in.
          const float size = fabsf(a) + (p.group_keys == 2 ? fabsf(b) : 0.f);
          const float err = fminf(near + kRound * size, FLT_MAX);
          const uint32_t least = sortable(worth - err), most = sortable(worth + err);
          const bool in = first && (kept >> lane) & 1u;
          const uint32_t lo = __reduce_min_sync(kFull, in ? least : kNone);
          const uint32_t hi = __reduce_max_sync(kFull, first && !in ? most : 0u);
          if (hi > kMinusInf && lo <= hi)
            kept = groups_exact<T>(row, p, P, first && least > hi,
                                   first && least <= hi && most >= lo);
        }
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
          const int e = expert_of<VEC>(j);
          if (!biased && scored && e < p.E) k[j] = to_f32(row[e]);   // experts go by logit
          if (!((kept >> place[j]) & 1u)) k[j] = -INFINITY;
        }
      }
      // distance below the largest in steps of the range, then the expert
      float hi = -INFINITY, lo = INFINITY;
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        hi = fmaxf(hi, k[j]);
        lo = fminf(lo, k[j] == -INFINITY ? INFINITY : k[j]);
      }
      hi = unordered(__reduce_max_sync(kFull, ordered(hi)));
      lo = unordered(__reduce_min_sync(kFull, ordered(lo)));
      const float range = hi - lo;
      again |= range == INFINITY;
      const float scale = range > 1e-30f ? steps / range : 0.f;
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        // the sum's low 23 bits are the rounded distance; the shift leaves nothing else
        const uint32_t d = __float_as_uint(fmaf(hi - k[j], scale, kMagic));
        v[j] = k[j] == -INFINITY ? kNone : d << bits | (uint32_t)expert_of<VEC>(j);
      }
      const float bound =
          (biased ? near + kRound * fmaxf(fabsf(hi), fabsf(lo)) : 0.f) * scale + 4.f;
      close = within(bound, steps, bits);
    }

    int mine = -1;
    if (!again) {
      uint32_t s[3];
      smallest_three<EPL>(v, 0, s);
      // no lane has given its third while those taken are below every lane's third
      uint32_t thirds = __reduce_min_sync(kFull, s[2]);
      auto take = [&](uint32_t best) {        // the lane that holds it goes on to its next
        const bool popped = s[0] == best;
        if (popped) {
          s[0] = s[1]; s[1] = s[2]; s[2] = kNone;
        }
        if (EPL > 3 && best >= thirds && __any_sync(kFull, popped && s[0] == kNone)) {
          uint32_t more[3];
          smallest_three<EPL>(v, best, more);
          if (popped) {
            s[0] = more[0]; s[1] = more[1]; s[2] = more[2];
          }
        }
      };
      auto differ = [&](uint32_t a, uint32_t b) {   // not the same logit under the same bias
        const int x = a & ((1u << bits) - 1), y = b & ((1u << bits) - 1);
        return to_f32(row[x]) != to_f32(row[y]) || (biased && p.bias[x] != p.bias[y]);
      };
      uint32_t last = 0;
      int taken = 0;                          // experts in order; lane r holds the r-th
      bool unsure = false;                    // two that follow each other may be swapped
      for (; taken < p.R; ++taken) {
        const uint32_t best = __reduce_min_sync(kFull, s[0]);
        if (best == kNone) break;
        if (best - last <= close) unsure |= differ(best, last);
        if (lane == taken) mine = best & ((1u << bits) - 1);
        take(best);
        last = best;
      }
      // Those left out that may belong before one that was taken are within `close` of the last.
      // Where they all equal it, and no two of those taken may be swapped, they come after it.
      uint32_t best = taken == p.R ? __reduce_min_sync(kFull, s[0]) : kNone;
      if (best != kNone && best - last <= close && !unsure) {
        unsure = differ(best, last);
        if (!unsure) {
          bool other = false;
#pragma unroll
          for (int j = 0; j < EPL; ++j)
            if (v[j] != kNone && v[j] > last && v[j] - last <= close) other |= differ(v[j], last);
          unsure = __any_sync(kFull, other);
        }
      }
      if (unsure) {
        for (; best != kNone && best - last <= close; best = __reduce_min_sync(kFull, s[0])) {
          if (taken == 32) {
            again = true;
            break;
          }
          if (lane == taken) mine = best & ((1u << bits) - 1);
          take(best);
          ++taken;
        }
      }
      if (unsure && !again) mine = order_exact<T>(row, p, mine);
    }
    if (again) mine = choose_exact<T>(row, p);
    const bool here = lane < p.R && mine >= 0;
    const float xm = here ? to_f32(row[mine]) : 0.f;
    float weight = weight_of(p, xm, here, m, sum, half);
    // a softmax that is NaN: weight_of takes renormalised weights from the chosen logits alone
    if (KEYS != BIASED && !p.sigmoid && odd && here) weight = NAN;
    if (lane < p.R) {
      idx[t * p.R + lane] = mine;
      w[t * p.R + lane] = weight;
    }
  }
}

// dlogits of a token, all E of them.  DENSE (softmax over all experts, not renormalised):
// p_e (g_e - sum_j g_j p_j), every expert.  Otherwise the chosen experts alone have one:
//   renormalised: scale u_r (g_r - sum_j g_j u_j) with shares u, times 1 - sigmoid(l) for a
//   sigmoid;  a sigmoid alone: scale g s (1 - s)
// (EPL 8 in 32 registers instead of 40: 65536 x 256 30.2 us against 32.4.)
template <typename T, int EPL, bool VEC, bool DENSE>
__global__ void __launch_bounds__(RT, EPL == 8 ? 8 : 0)
route_scores_bwd_kernel(const T* __restrict__ logits, const RouteParams p,
                        const int32_t* __restrict__ idx, const float* __restrict__ dw,
                        T* __restrict__ dlogits, long long ld_out) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (long long t = blockIdx.x * RW + warp; t < p.T; t += gridDim.x * RW) {
    const T* row = logits + t * p.ld;
    T* out = dlogits + t * ld_out;
    float v[EPL];
    if (DENSE) load_row<T, EPL, VEC>(row, p, v);
    int e = lane < p.R ? idx[t * p.R + lane] : -1;
    if ((unsigned)e >= (unsigned)p.E) e = -1;
    // An expert named twice, while the row is on its way: two slots are up to R / 2 apart, around
    // the end (a __match_any_sync after the sums: 16384 x 128 7.8 us against 6.9).
    bool twice = false;
#pragma unroll 4
    for (int off = 1; off <= p.R / 2; ++off) {
      const int other = lane + off < p.R ? lane + off : lane + off - p.R;
      twice |= __shfl_sync(kFull, e, other) == e;
    }
    float x = e >= 0 ? to_f32(row[e]) : -INFINITY;
    const bool here = x != -INFINITY;       // an empty slot or a closed expert: no gradient
    if (!here) x = 0.f;
    const float g = here ? dw[t * p.R + lane] * p.scale : 0.f;
    float d, m = 0.f, sum = 1.f;
    float dot = 0.f;
    if (DENSE) {
      softmax_parts<EPL, true>(v, m, sum);
      const float s = here ? expf(x - m) / sum : 0.f;
      dot = warp_sum(here ? g * s : 0.f);
      d = s * g;
      const float inv = sum == 0.f ? 0.f : 1.f / sum;   // 0: every expert is closed
#pragma unroll
      for (int j = 0; j < EPL; ++j) v[j] = -(v[j] * inv) * dot;
    } else if (p.renormalise) {
      RouteParams one = p;
      one.scale = 1.f;
      const float u = weight_of(one, x, here, m, sum, 16);
      dot = warp_sum(here ? g * u : 0.f);
      d = u * (g - dot);
      if (p.sigmoid) d /= 1.f + expf(x);
    } else {
      const float z = expf(-fabsf(x));
      d = g * z / ((1.f + z) * (1.f + z));
    }
    float all = d;
    bool first = here;      // the lowest slot that names this expert
    if (__any_sync(kFull, twice && here)) {   // an expert named twice gets both
      all = 0.f;
      for (int r = 0; r < p.R; ++r) {
        const int er = __shfl_sync(kFull, e, r);
        const float dr = __shfl_sync(kFull, d, r);
        if (er == e && here) {
          all += dr;
          if (r < lane) first = false;
        }
      }
    }
    if (DENSE) {
      if constexpr (VEC) {
#pragma unroll
        for (int j = 0; j < EPL; j += 4)
          if (expert_of<VEC>(j) < p.E)
            Vec<T, 4>::store(out + expert_of<VEC>(j), Vec<T, 4>::pack(v + j));
      } else {
#pragma unroll
        for (int j = 0; j < EPL; ++j)
          if (expert_of<VEC>(j) < p.E) out[expert_of<VEC>(j)] = from_f32<T>(v[j]);
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
  return {a.ld, a.T, a.E, a.R, r.score == MOE_SCORE_SIGMOID, r.groups,
          r.top_groups, r.group_keys, r.renormalise != 0, r.scale, a.bias};
}

int blocks_of(int T) { return (int)std::min<long long>(((long long)T + RW - 1) / RW, 152 * 16); }

// A row's experts in vectors of four: their number, the rows and the base allow it.
template <typename T>
bool vectors(const void* p, long long ld, int E) {
  return E % 4 == 0 && reinterpret_cast<uintptr_t>(p) % (4 * sizeof(T)) == 0 && ld % 4 == 0;
}

// CALL(EPL, VEC) for the smallest EPL that holds E experts.
#define MOE_EPL(E, vec, CALL)                 \
  do {                                        \
    const int per_ = ceil_div(E, 32);         \
    if (vec) {                                \
      if (per_ <= 4) CALL(4, true);           \
      else if (per_ <= 8) CALL(8, true);      \
      else if (per_ <= 12) CALL(12, true);    \
      else if (per_ <= 16) CALL(16, true);    \
      else CALL(32, true);                    \
    } else {                                  \
      if (per_ <= 2) CALL(2, false);          \
      else if (per_ <= 8) CALL(8, false);     \
      else CALL(32, false);                   \
    }                                         \
  } while (0)

template <typename T>
cudaError_t route_typed(const ScoresArgs& a, int32_t* idx, float* w, cudaStream_t s) {
  const RouteParams p = params_of(a);
  const T* l = static_cast<const T*>(a.logits);
  const size_t smem = p.groups > 1 ? (size_t)RW * (a.E + 32) * sizeof(float) : 0;
  const bool vec = vectors<T>(a.logits, a.ld, a.E);
#define MOE_ROUTE(N, V)                                                                      \
  do {                                                                                       \
    if (p.groups > 1)                                                                        \
      route_scores_kernel<T, N, V, GROUPED><<<blocks_of(a.T), RT, smem, s>>>(l, p, idx, w);  \
    else if (p.sigmoid && p.bias)                                                            \
      route_scores_kernel<T, N, V, BIASED><<<blocks_of(a.T), RT, 0, s>>>(l, p, idx, w);      \
    else                                                                                     \
      route_scores_kernel<T, N, V, ANY><<<blocks_of(a.T), RT, 0, s>>>(l, p, idx, w);         \
  } while (0)
  MOE_EPL(a.E, vec, MOE_ROUTE);
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
#define MOE_ROUTE(N, V) \
  route_scores_bwd_kernel<T, N, V, true><<<blocks_of(a.T), RT, 0, s>>>(l, p, idx, dw, o, ld_out)
    MOE_EPL(a.E, vec, MOE_ROUTE);
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
