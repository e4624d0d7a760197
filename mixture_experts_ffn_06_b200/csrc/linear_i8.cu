// linear_i8.cu -- the 8-bit integer product with scales for each token and
// channel (moe_linear_i8): v[t,n] = fl(sum_k x[t,k] w[n,k]) fl(sx[t] sw[n]),
// plain or gated (Act(gate) up).  The sums are exact in 32-bit integers.
//
// A block of 256 threads takes 64 tokens and 64 channels (gated: 64 gate and
// the matching 64 up channels), staging 64 bytes of K at a time in shared
// memory; a thread sums 4 x 4 outputs with four-way integer dot products.
#include "internal.cuh"

namespace moe {
namespace {

constexpr int kLt = 64;   // tokens and channels per block
constexpr int kKw = 16;   // 32-bit words of K per stage

struct LinParams {
  const int8_t *x, *w;
  const float *xs, *ws;
  int64_t T;
  int N, K, act;  // N: rows of w
  __nv_bfloat16* out;
  float* out_f32;
};

// Both activations as g sigma(.): 0.5 (1 + tanh v) = sigma(2v) does not cancel
// where v is large and negative.
__device__ __forceinline__ float lin_act(int act, float g) {
  const float e = act == MOE_ACT_SILU
                      ? -g
                      : -1.5957691216057308f * fmaf(0.044715f * g, g * g, g);  // -2 v
  return g / (1.0f + expf(e));
}

template <bool GATED>
__global__ void __launch_bounds__(256) linear_i8_kernel(const LinParams p) {
  constexpr int NB = GATED ? 2 : 1;
  __shared__ int xs[kKw][kLt + 1];
  __shared__ int wsm[NB][kKw][kLt + 1];
  const int tid = threadIdx.x;
  const int NO = GATED ? p.N / 2 : p.N;
  const int64_t t0 = (int64_t)blockIdx.x * kLt;
  const int n0 = blockIdx.y * kLt;
  int acc[NB][4][4] = {};
  const int lr = tid >> 2, lq = tid & 3;  // row and 16-byte quarter this thread stages
  pdl_wait();
  pdl_trigger();
  for (int k0 = 0; k0 < p.K; k0 += 4 * kKw) {
    const int kb = k0 + 16 * lq;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (t0 + lr < p.T && kb < p.K)
      v = *reinterpret_cast<const uint4*>(p.x + (t0 + lr) * p.K + kb);
    xs[4 * lq][lr] = v.x;
    xs[4 * lq + 1][lr] = v.y;
    xs[4 * lq + 2][lr] = v.z;
    xs[4 * lq + 3][lr] = v.w;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      v = make_uint4(0, 0, 0, 0);
      if (n0 + lr < NO && kb < p.K)
        v = *reinterpret_cast<const uint4*>(p.w + ((int64_t)b * NO + n0 + lr) * p.K + kb);
      wsm[b][4 * lq][lr] = v.x;
      wsm[b][4 * lq + 1][lr] = v.y;
      wsm[b][4 * lq + 2][lr] = v.z;
      wsm[b][4 * lq + 3][lr] = v.w;
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < kKw; ++kk) {
      int a[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = xs[kk][(tid >> 4) * 4 + i];
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = wsm[b][kk][(tid & 15) + 16 * j];
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[b][i][j] = __dp4a(a[i], c, acc[b][i][j]);
        }
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t t = t0 + (tid >> 4) * 4 + i;
    if (t >= p.T) continue;
    const float sx = __ldg(p.xs + t);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + (tid & 15) + 16 * j;
      if (n >= NO) continue;
      float v = __fmul_rn((float)acc[0][i][j], __fmul_rn(sx, __ldg(p.ws + n)));
      if (GATED) {
        const float u = __fmul_rn((float)acc[NB - 1][i][j], __fmul_rn(sx, __ldg(p.ws + NO + n)));
        v = lin_act(p.act, v) * u;
      }
      if (p.out) p.out[t * NO + n] = __float2bfloat16_rn(v);
      if (p.out_f32) p.out_f32[t * NO + n] = v;
    }
  }
}

bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_linear_i8(int64_t T, int N, int K, const int8_t* x,
                                    const float* x_scale, const int8_t* w,
                                    const float* w_scale, int gate_act, moe_bf16* out,
                                    float* out_f32, void* ws, size_t ws_bytes,
                                    cudaStream_t stream) {
  if (T < 0 || N <= 0 || K <= 0) return MOE_ERR_INVALID_ARG;
  if (gate_act != MOE_LINEAR_PLAIN && gate_act != MOE_ACT_SILU && gate_act != MOE_ACT_GELU_TANH)
    return MOE_ERR_INVALID_ARG;
  const bool gated = gate_act != MOE_LINEAR_PLAIN;
  if (gated && N % 2 != 0) return MOE_ERR_INVALID_ARG;
  if (K % 16 != 0 || K > MOE_LINEAR_MAX_K || N >= (1 << 22) || T >= (int64_t(1) << 24))
    return MOE_ERR_UNSUPPORTED;
  if (!ws || !aligned(ws, 256)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < 256) return MOE_ERR_WORKSPACE;
  if (T == 0) return MOE_OK;
  if (!x || !x_scale || !w || !w_scale || (!out && !out_f32)) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(out, 16) || !aligned(out_f32, 16))
    return MOE_ERR_INVALID_ARG;
  LinParams p{x, w, x_scale, w_scale, T, N, K, gate_act,
              reinterpret_cast<__nv_bfloat16*>(out), out_f32};
  const int NO = gated ? N / 2 : N;
  const dim3 grid((unsigned)((T + kLt - 1) / kLt), (NO + kLt - 1) / kLt);
  const cudaError_t e = launch_ex(gated ? linear_i8_kernel<true> : linear_i8_kernel<false>, grid,
                                  dim3(256), 0, stream, false, p);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
