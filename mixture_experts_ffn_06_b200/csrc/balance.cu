// balance.cu -- routing with a per-expert bias for balance
// (moe_route_balanced).  Per token: scores s = softmax(z) or sigmoid(z), choice
// values c = s + bias ranked as real numbers, the topk_group groups whose
// group_top largest c sum highest, the k largest c inside them, weights from
// the s of the chosen.
//
// The definition ranks c in 64 bits.  Here c is formed in fp32 with a bound on its
// error, and the choice is taken as made only where every gap it rests on (between
// consecutive chosen values, to the runner-up, between groups) is wider than
// that bound; the few tokens where one is not are chosen again on fp64 values
// (exact_choice).  The weights of the k chosen are fp64 throughout.
//
// LT lanes take a token (8 or 16 where there are many tokens, a whole warp where there
// are few), each lane PER experts of one group: it sorts its values, packed with
// their place in the low bits, by a network, so that a round of the top-k is a
// maximum over the LT heads, and a group of one lane has its two largest in
// front.  Bound by the instructions per expert (score and sort) and their latencies,
// then by the k rounds; the bytes (4 E + 8 k per token) would take a fifteenth of
// the time.  B200, device time: T = 16384, E = 64, k = 6 11.2 us (446 GB/s; 5.7 million warp
// instructions, issued in 53 % of the cycles); T = 4095, E = 256, k = 8 in 8 groups
// 11.5 us (19 % of the issue slots: latency); T = 64, E = 128 4.6 us; T = 1, E = 256 in
// groups 5.1 us.
#include <cfloat>
#include <cmath>

#include "tc_ptx.cuh"

namespace moe {
namespace {

constexpr uint32_t kAll = 0xffffffffu;

struct BalanceOpt {
  int scoring, n_group, topk_group, group_top, renorm;
  float factor;
};

// Order-preserving key of a double, above 0; -0 is keyed as +0.
__device__ __forceinline__ unsigned long long key64(double v) {
  if (v == 0.0) v = 0.0;
  const unsigned long long u = (unsigned long long)__double_as_longlong(v);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

__device__ __forceinline__ unsigned long long warp_max64(unsigned long long v) {
  const uint32_t hi = __reduce_max_sync(kAll, (uint32_t)(v >> 32));
  const uint32_t lo = __reduce_max_sync(kAll, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
  return (unsigned long long)hi << 32 | lo;
}

// A logit as the score sees it: +inf as the largest finite value; -inf and
// NaN stay what they are (not available).
__device__ __forceinline__ float clamp_logit(float z) { return z > FLT_MAX ? FLT_MAX : z; }
__device__ __forceinline__ bool available(float z) { return z > -INFINITY; }

__device__ __forceinline__ double value64(unsigned long long k) {
  return __longlong_as_double((long long)((k >> 63) ? k & 0x7fffffffffffffffull : ~k));
}

__device__ __forceinline__ double score64(float z, float zmax, double inv, bool sigmoid) {
  if (!available(z)) return 0.0;
  return sigmoid ? 1.0 / (1.0 + exp(-(double)z)) : exp((double)z - (double)zmax) * inv;
}

// what the choice compares: -inf for an expert that is not available
__device__ __forceinline__ double choice64(float z, double s, float b) {
  if (!available(z)) return -INFINITY;
  const double c = s + (double)b;
  return c == c ? fmin(c, DBL_MAX) : -INFINITY;
}

// 1 / sum of exp(z - zmax) over a row, by the whole warp.
__device__ __forceinline__ double softmax_inverse64(const float* __restrict__ zr, int E,
                                                    float zmax) {
  double sum = 0.0;
#pragma unroll 4
  for (int e = threadIdx.x & 31; e < E; e += 32)
    sum += score64(clamp_logit(__ldg(zr + e)), zmax, 1.0, false);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(kAll, sum, off);
  return 1.0 / sum;
}

// c of an expert as the choice compares it, in fp32: ``term`` is the logit, or the
// softmax's exponential.
__device__ __forceinline__ float choice32(float term, float inv, float b, bool sigmoid) {
  const float c = (sigmoid ? __fdividef(1.0f, 1.0f + __expf(-term)) : term * inv) + b;
  return available(term) && c == c ? c : -INFINITY;
}

// A softmax's denominator as it is added up: hi + lo.
struct Sum2 {
  float2 hi, lo;
};

__device__ __forceinline__ float2 minus2(float2 a, float2 b) { return fma2(b, both(-1.0f), a); }

// a + b as the rounded sum and its error (2Sum).
__device__ __forceinline__ float2 two_sum(float2 a, float2 b, float2& err) {
  const float2 s = add2(a, b), bb = minus2(s, a);
  err = add2(minus2(a, minus2(s, bb)), minus2(b, bb));
  return s;
}

// e^(z - m), z <= m, of two logits, added to the sum without the roundings of the
// difference, of the exponential and of the sum.  With x + e = z - m exactly, n = rint(x / ln 2)
// and r + rl = x + e - n ln 2, a term is 2^n (1 + r + q)(1 + rl), q the series from r^2 / 2 to
// r^7 / 7! (the rest is below 2^-27 at |r| <= ln 2 / 2) and 1 + r split exactly.  What rounds is
// below a tenth of a term, so the sum is within 2^-25.  Below e^-87, and for NaN, a term
// counts as that.  (T = 16384, E = 64, k = 6 11.2 us, with terms from expf added in fp64,
// which left weights 1.7 roundings off, 10.9; E = 512, k = 8 43.3 and 46.1.)
__device__ __forceinline__ float2 exp_below(float2 z, float m, Sum2& sum) {
  float2 e, x = two_sum(z, both(-m), e);
  e.x = x.x > -87.0f ? e.x : 0.0f;
  e.y = x.y > -87.0f ? e.y : 0.0f;
  x = make_float2(fmaxf(x.x, -87.0f), fmaxf(x.y, -87.0f));
  const float2 k = fma2(x, both(1.44269504f), both(12582912.0f));  // 1.5 2^23: n in the low bits
  const float2 n = add2(k, both(-12582912.0f));
  // ln 2 in 16 bits and what is left of it
  const float2 r = fma2(n, both(-0.693145751953125f), x);
  const float2 rl = fma2(n, both(-1.42860682e-06f), e);
  float2 p = fma2(r, both(1.98412701e-04f), both(1.38888892e-03f));  // 1/7!, 1/6!
  p = fma2(p, r, both(8.33333377e-03f));
  p = fma2(p, r, both(4.16666679e-02f));
  p = fma2(p, r, both(1.66666672e-01f));
  p = fma2(p, r, both(0.5f));
  const float2 h = add2(both(1.0f), r);
  float2 l = add2(minus2(both(1.0f), h), r);  // 1 + r = h + l
  const float2 q = mul2(mul2(r, r), p);
  l = add2(l, fma2(rl, add2(h, q), q));
  const float2 f = make_float2(__int_as_float((__float_as_int(k.x) << 23) + 0x3f800000),
                               __int_as_float((__float_as_int(k.y) << 23) + 0x3f800000));
  const float2 hf = mul2(h, f), lf = mul2(l, f);
  sum.hi = two_sum(sum.hi, hf, e);
  sum.lo = add2(sum.lo, add2(e, lf));
  return add2(hf, lf);
}

// Puts n <= 32 candidates of a token in their order, by the whole warp: each lane
// forms one's value and counts those before it.  In fp32 first, without the
// packing's error; where two are still within err of each other, in fp64, equal
// values by id.
__device__ __noinline__ void rank_exactly(const float* __restrict__ zr,
                                          const float* __restrict__ bias, int E, float zmax,
                                          float inv, float err, bool sigmoid, int n,
                                          int16_t* list) {
  const int lane = threadIdx.x & 31;
  const int id = lane < n ? list[lane] : E;
  const float z = lane < n ? clamp_logit(__ldg(zr + id)) : 0.f;
  const float b = lane < n && bias ? __ldg(bias + id) : 0.f;
  const float c = choice32(sigmoid || !available(z) ? z : __expf(z - zmax), inv, b, sigmoid);
  int rank = 0;
  bool close = false;
  for (int i = 0; i < n; ++i) {
    const float ci = __shfl_sync(kAll, c, i);
    rank += ci > c;
    close |= i != lane && !(fabsf(ci - c) > err + 4.8e-07f * fabsf(c));
  }
  if (__any_sync(kAll, close && lane < n)) {
    const double all = sigmoid ? 1.0 : softmax_inverse64(zr, E, zmax);
    const double d = choice64(z, score64(z, zmax, all, sigmoid), b);
    rank = 0;
    for (int i = 0; i < n; ++i) {
      const double di = __shfl_sync(kAll, d, i);
      const int idi = __shfl_sync(kAll, id, i);
      rank += di > d || (di == d && idi < id);
    }
  }
  __syncwarp();  // every lane has read its entry
  if (lane < n) list[rank] = (int16_t)id;
}

// One token's choice values in fp64 as ordered keys in key[E] (shared memory), and the
// groups it keeps by them (a bit each), by the whole warp.
__device__ __noinline__ uint32_t exact_groups(const float* __restrict__ zr,
                                              const float* __restrict__ bias, int E, float zmax,
                                              const BalanceOpt& o, unsigned long long* key) {
  const int lane = threadIdx.x & 31;
  const bool sigmoid = o.scoring == MOE_SCORE_SIGMOID;
  const double inv = sigmoid ? 1.0 : softmax_inverse64(zr, E, zmax);
#pragma unroll 4
  for (int e = lane; e < E; e += 32) {
    const float z = clamp_logit(__ldg(zr + e));
    key[e] = key64(choice64(z, score64(z, zmax, inv, sigmoid), bias ? __ldg(bias + e) : 0.f));
  }
  __syncwarp();
  if (o.n_group <= 1) return kAll;
  // a power of two lanes to a group, each with every such expert of it
  int lanes = 32;
  while (lanes * o.n_group > 32) lanes >>= 1;
  const int gs = E / o.n_group, g = lane / lanes;
  unsigned long long k0 = 0, k1 = 0;  // the two largest
  if (g < o.n_group) {
#pragma unroll 4
    for (int e = lane % lanes; e < gs; e += lanes) {
      const unsigned long long v = key[g * gs + e];
      k1 = max(k1, min(k0, v));
      k0 = max(k0, v);
    }
  }
  for (int s = 1; s < lanes; s <<= 1) {
    const unsigned long long w0 = __shfl_xor_sync(kAll, k0, s), w1 = __shfl_xor_sync(kAll, k1, s);
    k1 = max(min(k0, w0), max(k1, w1));
    k0 = max(k0, w0);
  }
  const double score =
      g < o.n_group ? (o.group_top == 2 && gs > 1 ? value64(k0) + value64(k1) : value64(k0)) : 0.0;
  int rank = 0;
  for (int i = 0; i < o.n_group; ++i) {
    const double other = __shfl_sync(kAll, score, i * lanes);
    rank += other > score || (other == score && i < g);
  }
  const uint32_t b = __ballot_sync(kAll, g < o.n_group && rank < o.topk_group);
  uint32_t keep = 0;
  for (int i = 0; i < o.n_group; ++i) keep |= ((b >> (i * lanes)) & 1u) << i;
  return keep;
}

// The k chosen experts of one token on fp64 values alone, by the whole warp: rounds
// of a maximum over the keys, equal values to the lower id.
__device__ __noinline__ void exact_choice(const float* __restrict__ zr,
                                          const float* __restrict__ bias, int E, int k,
                                          float zmax, const BalanceOpt& o,
                                          unsigned long long* key, int16_t* out) {
  const int lane = threadIdx.x & 31;
  const uint32_t keep = exact_groups(zr, bias, E, zmax, o, key);
  if (o.n_group > 1) {
    const int gs = E / o.n_group;
    for (int e = lane; e < E; e += 32)
      if (!((keep >> (e / gs)) & 1u)) key[e] = 0;  // not a candidate
    __syncwarp();
  }
  for (int j = 0; j < k; ++j) {
    unsigned long long best = 0;
    uint32_t at = kAll;
#pragma unroll 4
    for (int e = lane; e < E; e += 32)
      if (key[e] > best) {
        best = key[e];
        at = (uint32_t)e;
      }
    const unsigned long long top = warp_max64(best);
    const int win = (int)__reduce_min_sync(kAll, best == top ? at : kAll);
    __syncwarp();
    if (lane == 0) {
      key[win] = 0;
      out[j] = (int16_t)win;
    }
    __syncwarp();
  }
}

// ---- sorting networks on packed keys, largest first

template <int N, int I, int J>
__device__ __forceinline__ void cas(uint32_t (&a)[N]) {
  const uint32_t hi = max(a[I], a[J]), lo = min(a[I], a[J]);
  a[I] = hi;
  a[J] = lo;
}

// Bitonic network: sorts a[B, B + S) whose first half falls and second half rises.
template <int N, int B, int S>
__device__ __forceinline__ void merge(uint32_t (&a)[N]) {
  if constexpr (S > 1) {
#pragma unroll
    for (int i = B; i < B + S / 2; ++i) {
      const uint32_t hi = max(a[i], a[i + S / 2]), lo = min(a[i], a[i + S / 2]);
      a[i] = hi;
      a[i + S / 2] = lo;
    }
    merge<N, B, S / 2>(a);
    merge<N, B + S / 2, S / 2>(a);
  }
}

template <int N, int B, int S>
__device__ __forceinline__ void sort(uint32_t (&a)[N]) {
  if constexpr (S == 8) {  // odd-even merge sort: 19 exchanges, the bitonic one has 24
    cas<N, B, B + 1>(a); cas<N, B + 2, B + 3>(a); cas<N, B + 4, B + 5>(a); cas<N, B + 6, B + 7>(a);
    cas<N, B, B + 2>(a); cas<N, B + 1, B + 3>(a); cas<N, B + 4, B + 6>(a); cas<N, B + 5, B + 7>(a);
    cas<N, B + 1, B + 2>(a); cas<N, B + 5, B + 6>(a);
    cas<N, B, B + 4>(a); cas<N, B + 1, B + 5>(a); cas<N, B + 2, B + 6>(a); cas<N, B + 3, B + 7>(a);
    cas<N, B + 2, B + 4>(a); cas<N, B + 3, B + 5>(a);
    cas<N, B + 1, B + 2>(a); cas<N, B + 3, B + 4>(a); cas<N, B + 5, B + 6>(a);
  } else if constexpr (S > 1) {
    sort<N, B, S / 2>(a);
    sort<N, B + S / 2, S / 2>(a);
    // turn the second half round: falling, then rising
    if constexpr (S > 2) {
#pragma unroll
      for (int i = 0; i < S / 4; ++i) {
        const uint32_t t = a[B + S / 2 + i];
        a[B + S / 2 + i] = a[B + S - 1 - i];
        a[B + S - 1 - i] = t;
      }
    }
    merge<N, B, S>(a);
  }
}

// The eight largest of a (runs of eight), sorted, in a[0, 8).
template <int N>
__device__ __forceinline__ void top8(uint32_t (&a)[N]) {
  if constexpr (N <= 8) {
    sort<N, 0, N>(a);
  } else {
    sort<N, 0, 8>(a);
    sort<N, 8, 8>(a);
    if constexpr (N == 32) {
      sort<N, 16, 8>(a);
      sort<N, 24, 8>(a);
    }
    // the larger of the i-th and the (7 - i)-th of two runs are their eight largest
#pragma unroll
    for (int h = 0; h < N; h += 16) {
#pragma unroll
      for (int i = 0; i < 8; ++i) a[h + i] = max(a[h + i], a[h + 15 - i]);
    }
    merge<N, 0, 8>(a);
    if constexpr (N == 32) {
      merge<N, 16, 8>(a);
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] = max(a[i], a[23 - i]);
      merge<N, 0, 8>(a);
    }
  }
}

template <int LT>
__device__ __forceinline__ uint32_t token_max(uint32_t v) {
  if constexpr (LT == 32) {
    v = __reduce_max_sync(kAll, v);
  } else {
#pragma unroll
    for (int off = LT / 2; off > 0; off >>= 1) v = max(v, __shfl_xor_sync(kAll, v, off));
  }
  return v;
}

template <int LT>
__device__ __forceinline__ float token_max(float v) {
#pragma unroll
  for (int off = LT / 2; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, off));
  return v;
}

template <int LT>
__device__ __forceinline__ double token_sum(double v) {
#pragma unroll
  for (int off = LT / 2; off > 0; off >>= 1) v += __shfl_xor_sync(kAll, v, off);
  return v;
}

// Experts of a lane.  The LT lanes of a token are dealt to the groups, ``lanes``
// (a power of two) each; a lane's i-th expert is i * lanes + sub places into its
// group, or with quads four at a time, read as 16-byte vectors.
struct Deal {
  int groups, size;  // 1 and E without groups
  int lanes, lg;     // lanes per group, and its logarithm
  int n;             // experts per lane, at most
  int quads;
};

constexpr int kRouteWarps = 8;

// TOP8: a lane keeps its eight largest alone, sorted by a shorter network; a token that
// wants more of a lane is chosen on fp64 values (eight_will_do: rare where it is used).
template <int LT, int PER, bool TOP8>
__global__ void __launch_bounds__(32 * kRouteWarps, PER <= 8 ? 4 : PER <= 16 ? 3 : 2)
balance_kernel(const float* __restrict__ logits, const float* __restrict__ bias,
               const float* __restrict__ scale, int64_t T, int E, int k,
               int32_t* __restrict__ ids, float* __restrict__ w, int32_t* __restrict__ load,
               const BalanceOpt o, const Deal d, const bool clustered) {
  constexpr int TW = 32 / LT;                // tokens per warp
  constexpr uint32_t LOW = PER - 1;          // place of an expert in its lane, reversed
  constexpr int M = TOP8 && PER > 8 ? 8 : PER;  // sorted entries a lane keeps
  constexpr int LIST = LT == 8 ? 16 : 32;       // candidates of a token, at most
  extern __shared__ unsigned long long keys_s[];  // [warps][E], exact_choice's
  __shared__ int hist[kMaxExperts];
  __shared__ int16_t list_s[kRouteWarps][TW][LIST];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int tl = lane % LT, tw = lane / LT;
  const uint32_t mask = LT == 32 ? kAll : ((1u << LT) - 1u) << (tw * LT);  // this token's lanes
  const uint32_t below = mask & ((1u << lane) - 1u);
  const bool sigmoid = o.scoring == MOE_SCORE_SIGMOID;
  const int g = tl >> d.lg, sub = tl & (d.lanes - 1);  // this lane's group and place in it
  const bool in = g < d.groups;
  // its first expert, and how many it has
  const int e0 = g * d.size + (d.quads ? 4 * sub : sub);
  int nv = 0;
  if (in)
    nv = d.quads ? 4 * ((d.size - 4 * sub + 4 * d.lanes - 1) >> (d.lg + 2))
                 : (d.size - sub + d.lanes - 1) >> d.lg;
  const int step = d.quads ? 4 * d.lanes : d.lanes;
  auto expert = [&](int i) { return d.quads ? e0 + (i >> 2) * step + (i & 3) : e0 + i * step; };
  int16_t* list = list_s[warp][tw];
  if (load) {
    for (int e = threadIdx.x; e < E; e += blockDim.x) hist[e] = 0;
    __syncthreads();
  }
  pdl_wait();
  pdl_trigger();
  for (int64_t base = ((int64_t)blockIdx.x * warps + warp) * TW; base < T;
       base += (int64_t)gridDim.x * warps * TW) {
    // lanes past the last token route it once more and store nothing
    const int64_t t = base + tw < T ? base + tw : T - 1;
    const float* zr = logits + t * E;
    float z[PER];
    float early[PER <= 8 ? PER : 1];  // the bias, requested beside the logits
    float zmax = -INFINITY;
    bool quads = false;
    if constexpr (PER >= 4) {
      quads = d.quads;
      if (quads) {
#pragma unroll
        for (int i = 0; i < PER; i += 4) {
          float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
          if (i < nv) v = __ldg(reinterpret_cast<const float4*>(zr + e0 + (i >> 2) * step));
          z[i] = v.x;
          z[i + 1] = v.y;
          z[i + 2] = v.z;
          z[i + 3] = v.w;
        }
      }
    }
    if (!quads) {
#pragma unroll
      for (int i = 0; i < PER; ++i) z[i] = i < nv ? __ldg(zr + e0 + i * step) : -INFINITY;
    }
    if constexpr (PER <= 8) {
#pragma unroll
      for (int i = 0; i < PER; ++i)
        early[i] = bias && i < nv ? __ldg(bias + expert(i)) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      z[i] = clamp_logit(z[i]);
      zmax = fmaxf(zmax, z[i]);  // a NaN is passed over
    }
    zmax = token_max<LT>(zmax);
    // Scores, and a bound on the error of a difference of two, in units of 2^-23.  __expf
    // is within 2 + 1.173 |x|.  A sigmoid: s (1 - s) (2 + 1.173 |z|) from it, s / 2 and 2 s from
    // the sum and the division, 2.67 at most: 5.4 for two, taken as 5.7.  A softmax's
    // term, with the rounding of z - zmax: 2 + 1.7 |x| of e^x, which never is above 2 of
    // the largest; half of the score for the product with inv: 5 for two.  The
    // denominator's error is common to both and so counts once, times their difference:
    // the mean of its terms' errors, 2 + 1.7 ln 512 = 12.7, half for each of up to 36
    // additions in a row, 2 for the division.  38 of the largest score, taken as 64.
    float err = 6.8e-07f;  // of two values
    float inv = 1.0f;
    double den = 0.0;
    if (!sigmoid) {
      if (o.renorm) {  // the denominator cancels out of the weights
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const bool a = available(z[i]);
          z[i] = a ? __expf(z[i] - zmax) : z[i];  // now the term, or -inf / NaN
          sum += a ? z[i] : 0.0f;
        }
#pragma unroll
        for (int s = LT / 2; s > 0; s >>= 1) sum += __shfl_xor_sync(kAll, sum, s);
        inv = __fdividef(1.0f, sum);
      } else {
        Sum2 sum{both(0.0f), both(0.0f)};
        const float m = fmaxf(zmax, -FLT_MAX);  // (-inf where no expert is available)
#pragma unroll
        for (int i = 0; i < PER; i += 2) {
          const float z1 = i + 1 < PER ? z[i + 1] : -INFINITY;
          const float2 term = exp_below(make_float2(z[i], z1), m, sum);
          if (available(z[i])) z[i] = term.x;
          if (i + 1 < PER && available(z1)) z[i + 1] = term.y;
        }
        den = token_sum<LT>(((double)sum.hi.x + (double)sum.hi.y) +
                            ((double)sum.lo.x + (double)sum.lo.y));
        inv = __fdividef(1.0f, (float)den);
      }
      err = 7.6293945e-06f * inv;  // 2^-17: inv is the largest score
    }
    uint32_t a[PER];
    float v0 = -INFINITY, v1 = -INFINITY;  // this lane's two largest c (for its group)
    auto pack = [&](int i, float b) {
      const float c = choice32(z[i], inv, b, sigmoid);
      if (d.groups > 1) {
        const float u = i < nv ? c : -INFINITY;
        v1 = fmaxf(v1, fminf(v0, u));
        v0 = fmaxf(v0, u);
      }
      const uint32_t u = __float_as_uint(c);
      const uint32_t key = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
      a[i] = i < nv ? (key & ~LOW) | (LOW - i) : 0u;
    };
    if constexpr (PER <= 8) {
#pragma unroll
      for (int i = 0; i < PER; ++i) pack(i, early[i]);
    } else if (quads) {
#pragma unroll
        for (int i = 0; i < PER; i += 4) {
          float4 b = make_float4(0.f, 0.f, 0.f, 0.f);
          if (bias && i < nv)
            b = __ldg(reinterpret_cast<const float4*>(bias + e0 + (i >> 2) * step));
          pack(i, b.x);
          pack(i + 1, b.y);
          pack(i + 2, b.z);
          pack(i + 3, b.w);
        }
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i) pack(i, bias && i < nv ? __ldg(bias + e0 + i * step) : 0.f);
    }
    if constexpr (TOP8)
      top8<PER>(a);
    else
      sort<PER, 0, PER>(a);
    auto value = [](uint32_t key) {
      key &= ~LOW;
      return __uint_as_float((key & 0x80000000u) ? key ^ 0x80000000u : ~key);
    };
    // a packed value is short of c by less than 2^-23 PER |c|; c itself rounds once
    constexpr float REL = 2.0f * (PER + 1) * 1.1920929e-07f;
    if (d.groups > 1) {
      const bool two = o.group_top == 2 && d.size > 1;
      for (int s = 1; s < d.lanes; s <<= 1) {
        const float w0 = __shfl_xor_sync(kAll, v0, s), w1 = __shfl_xor_sync(kAll, v1, s);
        v1 = fmaxf(fminf(v0, w0), fmaxf(v1, w1));
        v0 = fmaxf(v0, w0);
      }
      const float score = two ? v0 + v1 : v0;
      int rank = 0;
      for (int s = d.lanes; s < LT; s += d.lanes) {
        const float other = __shfl_xor_sync(kAll, score, s);
        const int og = (tl ^ s) >> d.lg;
        rank += og < d.groups && (other > score || (other == score && og < g));
      }
      bool kept = in && rank < o.topk_group;
      if (o.topk_group < d.groups) {
        // the lowest kept score against the highest other
        const float low = -token_max<LT>(kept ? -score : -INFINITY);
        const float high = token_max<LT>(in && !kept ? score : -INFINITY);
        const float mag = token_max<LT>(in ? fabsf(v0) + (two ? fabsf(v1) : 0.0f) : 0.0f);
        uint32_t open = __ballot_sync(kAll, !(low - high > 2.0f * err + 4.8e-07f * mag));
#pragma unroll 1
        while (open) {  // a token whose groups are open
          const int q = (__ffs(open) - 1) / LT;
          open &= LT == 32 ? 0u : ~(((1u << LT) - 1u) << (q * LT));
          const int64_t tq = base + q < T ? base + q : T - 1;
          const uint32_t keep = exact_groups(logits + tq * E, bias, E,
                                             __shfl_sync(kAll, zmax, q * LT), o,
                                             keys_s + warp * E);
          __syncwarp();
          if (tw == q) kept = in && ((keep >> g) & 1u);
        }
      }
      if (!kept) {
#pragma unroll
        for (int i = 0; i < M; ++i) a[i] = 0;
      }
    }
    // Candidates in falling order: k of them, and on until one is clearly below the
    // k-th: ``count`` of them then.  ``near``: a gap between two was too narrow to
    // tell their order.
    const int cand = d.groups > 1 ? o.topk_group * d.size : E;
    bool all_again = false;  // the whole choice has to be made on fp64 values
    auto pop = [&](int r, uint32_t top) {
      const uint32_t b = __ballot_sync(kAll, a[0] == top);
      if (a[0] == top && !(b & below) && top) {
        list[r] = (int16_t)expert((int)(LOW - (top & LOW)));
#pragma unroll
        for (int i = 0; i + 1 < M; ++i) a[i] = a[i + 1];
        a[M - 1] = 0;
        // more than it kept may be wanted of this lane
        if (M < PER && a[0] == 0 && nv > M) all_again = true;
      }
    };
    uint32_t top = token_max<LT>(a[0]);
    float v = value(top), last = v;
    bool near = false;
#pragma unroll 1
    for (int r = 0; r < k; ++r) {
      pop(r, top);
      top = token_max<LT>(a[0]);
      const float tol = err + REL * fabsf(v), before = v;
      v = value(top);
      if (r + 1 < k) near |= !(before - v > tol);
      else last = before;
    }
    int count = last - v > err + REL * fabsf(last) || k == cand ? k : 0;
#pragma unroll 1
    for (int r = k; r < LIST && __any_sync(kAll, count == 0); ++r) {
      near |= count == 0;
      pop(r, top);
      last = v;
      top = token_max<LT>(a[0]);
      v = value(top);
      if (count == 0 && (last - v > err + REL * fabsf(last) || r + 1 == cand)) count = r + 1;
    }
    all_again |= count == 0;
    // tokens whose order is open, one at a time
    const uint32_t wide = __ballot_sync(kAll, all_again), close = __ballot_sync(kAll, near);
    __syncwarp();
    if (wide | close) {
#pragma unroll 1
      for (int q = 0; q < TW; ++q) {
        const uint32_t lanes = LT == 32 ? kAll : ((1u << LT) - 1u) << (q * LT);
        const int64_t tq = base + q < T ? base + q : T - 1;
        const float top = __shfl_sync(kAll, zmax, q * LT);
        const int n = __shfl_sync(kAll, count, q * LT);
        const float invq = __shfl_sync(kAll, inv, q * LT), errq = __shfl_sync(kAll, err, q * LT);
        if (wide & lanes)
          exact_choice(logits + tq * E, bias, E, k, top, o, keys_s + warp * E, list_s[warp][q]);
        else if (close & lanes)
          rank_exactly(logits + tq * E, bias, E, top, invq, errq, sigmoid, n, list_s[warp][q]);
      }
      __syncwarp();
    }
    // weights in fp64
    const bool mine = tl < k && base + tw < T;
    const int id = mine ? list[tl] : 0;
    const float each = scale && mine ? __ldg(scale + id) : 1.0f;
    double s = 0.0;
    if (mine) {
      const float b = bias ? __ldg(bias + id) : 0.0f;
      if (b > -INFINITY)  // else (or NaN) not available, as by its logit
        s = score64(clamp_logit(__ldg(zr + id)), zmax, o.renorm ? 1.0 : 1.0 / den, sigmoid);
    }
    double wt = s;
    if (o.renorm) {
      const double sum = token_sum<LT>(s);
      wt = sum > 0.0 ? s / sum : 0.0;
    }
    wt *= (double)o.factor;
    if (mine) {
      ids[t * k + tl] = id;
      w[t * k + tl] = (float)(wt * (double)each);
      if (load) atomicAdd(&hist[id], 1);
    }
    __syncwarp();
  }
  if (load) {
    __syncthreads();
    if (clustered) {  // the blocks are one cluster: each sums a part of the counts over all
      cluster_sync();
      const uint32_t rank = cluster_ctarank(), counts = smem_u32(hist);
      for (int e = rank * blockDim.x + threadIdx.x; e < E; e += gridDim.x * blockDim.x) {
        int sum = 0;
        for (uint32_t r = 0; r < gridDim.x; ++r)
          sum += ld_cluster_s32(mapa_shared(counts + 4 * e, r));
        load[e] = sum;
      }
      cluster_sync();  // no block leaves while its counts are read
      return;
    }
    // alone, a block writes the counts; several add theirs to zeros
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
      if (gridDim.x == 1) load[e] = hist[e];
      else if (hist[e]) atomicAdd(load + e, hist[e]);
    }
  }
}

// Zeros ahead of a launch of several blocks, which starts beside it.
__global__ void zero_load_kernel(int32_t* load, int E) {
  pdl_trigger();
  pdl_wait();
  for (int e = threadIdx.x; e < E; e += blockDim.x) load[e] = 0;
}

template <int LT, bool TOP8>
cudaError_t launch_balance(int per, unsigned blocks, unsigned threads, const float* logits,
                           const float* bias, const float* scale, int64_t T, int E, int k,
                           int32_t* ids, float* w, int32_t* load, const BalanceOpt& o,
                           const Deal& d, bool clustered, cudaStream_t st) {
  auto kern = per <= 1    ? balance_kernel<LT, 1, TOP8>
              : per <= 2  ? balance_kernel<LT, 2, TOP8>
              : per <= 4  ? balance_kernel<LT, 4, TOP8>
              : per <= 8  ? balance_kernel<LT, 8, TOP8>
              : per <= 16 ? balance_kernel<LT, 16, TOP8>
                          : balance_kernel<LT, 32, TOP8>;
  const size_t smem = sizeof(unsigned long long) * (threads / 32) * E;  // at most 32 KB
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = blocks;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = clustered ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, logits, bias, scale, T, E, k, ids, w, load, o, d,
                            clustered);
}

// Deals E experts in groups to LT lanes; n > 32 where they do not fit.
Deal deal(int E, int groups, int LT, bool aligned) {
  Deal d{groups, E / groups, LT, 0, 0, 0};
  while (d.lanes * groups > LT) d.lanes /= 2;  // 0: more groups than lanes
  if (d.lanes == 0) {
    d.n = 1 << 20;
    return d;
  }
  while (1 << d.lg < d.lanes) ++d.lg;
  d.n = (d.size + d.lanes - 1) / d.lanes;
  const int quads = (d.size + 4 * d.lanes - 1) / (4 * d.lanes);
  if (aligned && d.size % 4 == 0 && d.n >= 4) {
    d.quads = 1;
    d.n = 4 * quads;
  }
  return d;
}

// Whether a lane's eight largest will do: fewer than eight are chosen, or they come from
// so many lanes that all eight of one are rarely wanted (C(k, 8) lanes^-7 (1 - 1 / lanes)^(k - 8)
// of the tokens): at most one token in 475, in 5000 where a lane has more than 16, whose
// tokens take longer to choose again.  Where one kept group was one lane's every token was
// chosen again: E = 256, 8 groups, 1 kept, k = 8, T = 4095 40.3 us, with all entries on 32 lanes
// 11.2; E = 512, 32 groups, 1 kept, T = 1 21.0 and 7.4.  With eight lanes in play and
// k = 16, sixteen lanes and all entries on 32: E = 256, T = 4500 14.0 and 14.6, T = 16384 29.3
// and 38.0; E = 512, T = 4095 14.7 and 18.6, T = 8192 36.8 and 28.3, T = 16384 53.0 and 49.9.
bool eight_will_do(const Deal& d, const BalanceOpt& o, int k, int LT) {
  const int lanes = d.groups > 1 ? d.lanes * o.topk_group : LT;
  return d.n <= 8 || k < 8 || lanes >= (d.n <= 16 ? (k + 1) / 2 : k - 4);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_route_balanced(const moe_shape* shape, const float* logits,
                                         const float* bias, const float* scale,
                                         const moe_balance_opts* opts, int32_t* ids, float* w,
                                         int32_t* load, cudaStream_t stream) {
  moe_status st = validate_shape(shape);
  if (st != MOE_OK) return st;
  const int E = shape->E, k = shape->k;
  BalanceOpt o{MOE_SCORE_SOFTMAX, 1, 1, 1, 1, 1.0f};
  if (opts) {
    if (opts->scoring != MOE_SCORE_SOFTMAX && opts->scoring != MOE_SCORE_SIGMOID)
      return MOE_ERR_INVALID_ARG;
    if (opts->n_group < 0 || !std::isfinite(opts->factor)) return MOE_ERR_INVALID_ARG;
    if (opts->n_group > MOE_MAX_GROUPS) return MOE_ERR_UNSUPPORTED;
    o.scoring = opts->scoring;
    o.renorm = opts->renorm != 0;
    o.factor = opts->factor;
    if (opts->n_group > 1) {
      if (E % opts->n_group != 0 || opts->topk_group < 1 || opts->topk_group > opts->n_group ||
          opts->group_top < 1 || opts->group_top > 2 ||
          k > opts->topk_group * (E / opts->n_group))
        return MOE_ERR_INVALID_ARG;
      o.n_group = opts->n_group;
      o.topk_group = opts->topk_group;
      o.group_top = opts->group_top;
    }
  }
  if (shape->T > 0 && (!logits || !ids || !w)) return MOE_ERR_INVALID_ARG;
  const int64_t T = shape->T;
  const bool vec = aligned(logits, 16) && aligned(bias, 16);
  // A warp per token while that leaves the SMs room; else the fewest lanes that the
  // groups, 32 experts a lane and eight_will_do allow.  A lane of a token writes one choice, so
  // k lanes at least.  Sigmoid, with 8, 16 and 32 lanes: E = 64, k = 8 T = 2000 6.0, 5.0 and 5.0,
  // T = 4500 6.5, 6.4 and 7.0, T = 8192 7.2, 7.9 and 10.5; E = 256, k = 8 in 8 groups T = 2000 10.3,
  // 7.5 and 7.4, T = 4500 10.8, 12.1 and 11.8, T = 16384 24.7, 25.4 and 30.3; with 16 and 32: E = 256,
  // k = 16 in 8 groups T = 2000 9.6 and 9.1, T = 3600 13.9 and 14.3, T = 6000 21.4 and 19.3,
  // T = 16384 29.3 and 38.0; E = 512, k = 16 T = 2000 11.0 and 12.8, T = 16384 40.0 and 45.7.
  int LT = 32;
  Deal d = deal(E, o.n_group, 32, vec);
  if (T > 24 * device_sm_count()) {
    for (int lt = k <= 8 ? 8 : 16; lt < 32 && k <= lt; lt *= 2) {
      const Deal c = deal(E, o.n_group, lt, vec);
      if (c.n > 32 || !eight_will_do(c, o, k, lt)) continue;
      LT = lt;
      d = c;
      break;
    }
  }
  const int tw = 32 / LT;
  const int64_t need = (T + tw - 1) / tw;  // warps
  const int warps = need < kRouteWarps ? (need > 0 ? (int)need : 1) : kRouteWarps;
  const int64_t all = (need + warps - 1) / warps, most = 8 * device_sm_count();
  const unsigned blocks = (unsigned)(all < most ? all : most);
  // Counts of several blocks: up to eight are one cluster and sum them there, more
  // add them to zeros that a launch of its own wrote; so do fewer in a graph, whose replay
  // hides that launch and not the cluster's barriers.  With a cluster and with two
  // launches, E = 128: a call 6.2 and 8.3 us at T = 9 to 64; replayed T = 9 4.4 and 4.3, T = 33 4.9
  // and 4.3, T = 64 4.5 and 4.3; E = 256 in groups, replayed T = 33 6.5 and 6.0.
  bool clustered = load && blocks > 1 && blocks <= 8;
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  if (clustered && cudaStreamIsCapturing(stream, &capture) == cudaSuccess &&
      capture == cudaStreamCaptureStatusActive)
    clustered = false;
  if (load && blocks != 1 && !clustered &&
      launch_ex(zero_load_kernel, dim3(1), dim3(256), 0, stream, true, load, E) != cudaSuccess)
    return MOE_ERR_CUDA;
  if (T == 0) return MOE_OK;
  const unsigned threads = 32 * warps;
  const bool top8 = LT < 32 || (k <= 8 && eight_will_do(d, o, k, 32));
  auto go = LT == 8 ? launch_balance<8, true> : LT == 16 ? launch_balance<16, true>
            : top8  ? launch_balance<32, true>
                    : launch_balance<32, false>;
  const cudaError_t e = go(d.n, blocks, threads, logits, bias, scale, T, E, k, ids, w, load, o, d,
                           clustered, stream);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
