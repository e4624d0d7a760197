// balance.cu -- routing with a per-expert bias for balance
// (moe_route_balanced).  Per token: scores s = softmax(z) or sigmoid(z), choice
// values c = s + bias ranked as real numbers, the topk_group groups whose
// group_top largest c sum highest, the k largest c inside them, weights from
// the s of the chosen.
//
// A warp per token; lane l holds experts l, l + 32, ... (PER per lane).  The
// choice is made on fp64 values, so that it is the one the definition gives
// and not one of an fp32 rounding; equal values go to the lower id.
#include <cfloat>
#include <cmath>

#include "internal.cuh"

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

template <int PER>
__global__ void __launch_bounds__(256)
balance_kernel(const float* __restrict__ logits, const float* __restrict__ bias,
               const float* __restrict__ scale, int64_t T, int E, int k,
               int32_t* __restrict__ ids, float* __restrict__ w, int32_t* __restrict__ load,
               const BalanceOpt o) {
  extern __shared__ int32_t hist[];  // [E] when load is given
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_trigger();
  if (load) {
    for (int e = threadIdx.x; e < E; e += blockDim.x) hist[e] = 0;
    __syncthreads();
  }
  const bool sigmoid = o.scoring == MOE_SCORE_SIGMOID;
  const int64_t t = (int64_t)blockIdx.x * (blockDim.x >> 5) + warp;
  if (t < T) {
    const float* zr = logits + t * E;
    float z[PER];
    float zmax = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = lane + 32 * i;
      z[i] = e < E ? clamp_logit(__ldg(zr + e)) : -INFINITY;
      if (available(z[i])) zmax = fmaxf(zmax, z[i]);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) zmax = fmaxf(zmax, __shfl_xor_sync(kAll, zmax, off));
    double inv = 1.0;
    if (!sigmoid) {
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < PER; ++i) sum += score64(z[i], zmax, 1.0, false);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(kAll, sum, off);
      inv = 1.0 / sum;
    }
    double c[PER];
    unsigned long long key[PER];  // 0: not a candidate
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = lane + 32 * i;
      c[i] = e < E ? choice64(z[i], score64(z[i], zmax, inv, sigmoid), bias ? __ldg(bias + e) : 0.f)
                   : -INFINITY;
      key[i] = e < E ? key64(c[i]) : 0ull;
    }
    if (o.n_group > 1) {
      const int gs = E / o.n_group;
      // lane g gets group g's score
      unsigned long long mine = 0;
      for (int g = 0; g < o.n_group; ++g) {
        unsigned long long best = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if ((lane + 32 * i) / gs == g) best = max(best, key[i]);
        const unsigned long long top = warp_max64(best);
        double sum = __longlong_as_double((top >> 63) ? top & 0x7fffffffffffffffull : ~top);
        if (o.group_top == 2) {
          // the second largest: drop one entry that holds the largest
          uint32_t cand = kAll;
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            const int e = lane + 32 * i;
            if (e < E && e / gs == g && key[i] == top) cand = min(cand, (uint32_t)e);
          }
          const uint32_t drop = __reduce_min_sync(kAll, cand);
          best = 0;
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            const int e = lane + 32 * i;
            if (e < E && e / gs == g && (uint32_t)e != drop) best = max(best, key[i]);
          }
          const unsigned long long second = warp_max64(best);
          if (second)
            sum += __longlong_as_double((second >> 63) ? second & 0x7fffffffffffffffull
                                                       : ~second);
        }
        if (lane == g) mine = key64(sum);
      }
      uint32_t keep = 0;
      for (int r = 0; r < o.topk_group; ++r) {
        const unsigned long long top = warp_max64(mine);
        const int win = __ffs(__ballot_sync(kAll, mine == top)) - 1;
        keep |= 1u << win;
        if (lane == win) mine = 0;
      }
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int e = lane + 32 * i;
        if (e < E && !((keep >> (e / gs)) & 1u)) key[i] = 0;
      }
    }
    int my_id = 0;
    bool usable = false;  // c above -inf
    for (int j = 0; j < k; ++j) {
      unsigned long long best = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) best = max(best, key[i]);
      const unsigned long long top = warp_max64(best);
      uint32_t cand = kAll;
#pragma unroll
      for (int i = PER - 1; i >= 0; --i)
        if (key[i] == top) cand = (uint32_t)(lane + 32 * i);
      const int win = (int)__reduce_min_sync(kAll, cand);
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (lane + 32 * i == win) key[i] = 0;
      if (lane == j) {
        my_id = win;
        usable = top > key64(-INFINITY);
      }
    }
    double s = 0.0;
    if (lane < k && usable) s = score64(clamp_logit(__ldg(zr + my_id)), zmax, inv, sigmoid);
    double wt = s;
    if (o.renorm) {
      double den = s;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) den += __shfl_xor_sync(kAll, den, off);
      wt = den > 0.0 ? s / den : 0.0;
    }
    wt *= (double)o.factor;
    if (lane < k) {
      if (scale) wt *= (double)__ldg(scale + my_id);
      ids[t * k + lane] = my_id;
      w[t * k + lane] = (float)wt;
      if (load) atomicAdd(&hist[my_id], 1);
    }
  }
  if (load) {
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x)
      if (hist[e]) atomicAdd(load + e, hist[e]);
  }
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
  if (load && cudaMemsetAsync(load, 0, sizeof(int32_t) * E, stream) != cudaSuccess)
    return MOE_ERR_CUDA;
  if (shape->T == 0) return MOE_OK;
  auto kern = E <= 32 ? balance_kernel<1> : E <= 64 ? balance_kernel<2> : E <= 128 ? balance_kernel<4>
              : E <= 256 ? balance_kernel<8> : balance_kernel<16>;
  const int64_t blocks = (shape->T + 7) / 8;
  const cudaError_t e =
      launch_ex(kern, dim3((unsigned)blocks), dim3(256), load ? sizeof(int32_t) * E : 0, stream,
                false, logits, bias, scale, shape->T, E, k, ids, w, load, o);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
