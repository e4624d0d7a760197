// norm.cu -- the norms around a block (moe_block_norm) and the int8 row
// quantiser (moe_quantize_rows_i8).  Per token row, each step one fp32
// operation:
//   t  = y (1 / sqrt(mean(y^2) + eps)) post_w        (t = y without post_w)
//   r' = bf16(alpha r + (beta token_gate) (t gate))
//   a  = bf16(r' (1 / sqrt(mean(r'^2) + eps)) pre_w)
//   codes: s = amax(a) / 127, rint(a / s)
// The quantiser is the last step alone, on the rows it is given.
//
// Bound: HBM.  A row is read once and kept in registers (8 bf16 values per
// 16-byte vector, VPT vectors per thread) through its up to three reductions,
// so every input byte is read once and every output byte written once.  B200:
// T = 8192, H = 2816, both norms 35.3 us (5.2 TB/s, 80 % of the measured copy bandwidth);
// T = 16383, H = 2048, with codes 58.6 us (5.1 TB/s; the instructions of the rounding to
// codes come next, issued in 68 % of the cycles); T = 1 2.6 us.
//
// The means are taken in double (a square of a bf16 value is exact in fp32), and with IEEE
// divisions and square roots the rows and their codes come out the same bits as the steps
// taken one by one.  The number of threads of a row, and with it the order of its sum,
// depends on how many rows there are: the fp64 sums then differ in their last bits, where
// a row's exponents span more than 53 bits hold, and round to the same fp32 mean but at a
// border (some 2^-27 of rows).
#include <algorithm>
#include <cmath>

#include "internal.cuh"

namespace moe {
namespace {

struct RowParams {
  const uint4 *y, *r, *post_w, *gate, *pre_w;
  const float* token_gate;
  float alpha, beta, post_eps, pre_eps;
  uint4 *r_out, *a;
  uint2* codes;
  float* scales;
  int64_t rows;
  int vec;        // 16-byte vectors per row
  double n, inv_n;  // values per row, 1 / n
};

__device__ __forceinline__ void unpack8(const uint4& v, float2 (&f)[4]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    f[i] = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
}

__device__ __forceinline__ uint4 pack8(const float2 (&f)[4]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(f[i].x, f[i].y);
    u[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

__device__ __forceinline__ double squares(const uint4& v) {
  float2 f[4];
  unpack8(v, f);
  double s = 0.0, t = 0.0;  // two chains
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s = fma((double)f[i].x, (double)f[i].x, s);
    t = fma((double)f[i].y, (double)f[i].y, t);
  }
  return s + t;
}

// The largest magnitude of eight bf16 values as its 15 bits, which order like the
// values, with infinity and then NaN above them.
__device__ __forceinline__ uint32_t abs_bits(const uint4& v) {
  const uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                              __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
  return max(m & 0xffffu, m >> 16);
}

// Sum and maximum over the block, for every thread; red holds one value per warp
// and is not used again, so one barrier does.
__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = blockDim.x >> 5;
  if (n == 1) return v;
  if (lane == 0) red[warp] = v;
  __syncthreads();
  if (n <= 4) {
    v = red[0] + red[1];
    if (n > 2) v += red[2];
    if (n > 3) v += red[3];
    return v;
  }
  v = lane < n ? red[lane] : 0.0;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* red) {
  v = __reduce_max_sync(0xffffffffu, v);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = blockDim.x >> 5;
  if (n == 1) return v;
  if (lane == 0) red[warp] = v;
  __syncthreads();
  return __reduce_max_sync(0xffffffffu, lane < n ? red[lane] : 0u);
}

// Sum of the row's squares over the block, from this thread's vectors.
template <int VPT>
__device__ __forceinline__ double block_squares(const uint4 (&v)[VPT], double* red) {
  double ss = 0.0;
#pragma unroll
  for (int j = 0; j < VPT; ++j) ss += squares(v[j]);
  return block_sum(ss, red);
}

// 1 / sqrt(mean + eps), IEEE fp32, of the mean of squares rounded to fp32.  The
// quotient in double by its reciprocal and one exact remainder: right to the last
// bit wherever it can lie halfway between two fp32 values.
__device__ __forceinline__ float rms_inverse(double ss, const RowParams& p, float eps) {
  double q = ss * p.inv_n;
  if (q < 1e300) q = fma(fma(-q, p.n, ss), p.inv_n, q);
  return 1.0f / sqrtf((float)q + eps);
}

// rint(fl(v / s)) of eight values, as bytes.  inv is 1 / s rounded, or 0 where s is
// outside [2^-60, 2^60] or not finite.  v inv is within 2.3e-5 of fl(v / s) (three
// roundings of 2^-24 of at most 127), so it has the same nearest integer unless
// it comes that near to a half; those, and every row without inv, divide.  Adding
// 1.5 2^23 rounds to an integer in the low bits.
__device__ __forceinline__ uint2 codes8(const float2 (&f)[4], float s, float inv) {
  uint32_t c[8];
  float off = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = mul2(f[i], both(inv));
    const float2 r = add2(t, both(12582912.0f));
    // t - (r - 1.5 2^23), both exact
    const float2 d = add2(add2(r, both(-12582912.0f)), make_float2(-t.x, -t.y));
    c[2 * i] = __float_as_uint(r.x);
    c[2 * i + 1] = __float_as_uint(r.y);
    off = fmaxf(off, fmaxf(fabsf(d.x), fabsf(d.y)));
  }
  if (off > 0.49993896f || inv == 0.0f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // a row that is not finite: 0 or NaN, code 0
      const float v = (i & 1) ? f[i / 2].y : f[i / 2].x;
      c[i] = (uint32_t)max(-127, min(127, __float2int_rn(__fdiv_rn(v, s))));
    }
  }
  uint2 o;
  o.x = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
  o.y = __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040), 0x5410);
  return o;
}

// AFTER: with the norm after a block and the residual; BEFORE: with the norm ahead of the
// next; neither: the quantiser alone.  (One kernel that branches on what it is given keeps
// more registers and fewer rows on an SM: T = 148, H = 2048 with codes 3.66 us and here
// 3.39; the quantiser at 8192 x 2816 18.8 and 17.7, 3.9 TB/s.)
template <int VPT, bool AFTER, bool BEFORE>
__global__ void __launch_bounds__(1024)
rows_kernel(const RowParams p) {
  __shared__ double red[2][32];
  __shared__ uint32_t redm[32];
  pdl_wait();
  pdl_trigger();
  // (blockDim.y rows to a block only where a row is one warp's: no barrier then)
  const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y, base = t * p.vec;
  if (t >= p.rows) return;
  const int tid = threadIdx.x, nt = blockDim.x;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint4 r[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) r[j] = tid + j * nt < p.vec ? p.r[base + tid + j * nt] : zero;
  if constexpr (AFTER) {
    uint4 y[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) y[j] = tid + j * nt < p.vec ? p.y[base + tid + j * nt] : zero;
    float inv = 1.0f;
    if (p.post_w) inv = rms_inverse(block_squares<VPT>(y, red[0]), p, p.post_eps);
    const float m = p.token_gate ? __fmul_rn(p.beta, p.token_gate[t]) : p.beta;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = tid + j * nt;
      if (c < p.vec) {
        float2 f[4], g[4], o[4];
        unpack8(y[j], f);
        if (p.post_w) {
          unpack8(__ldg(p.post_w + c), g);
#pragma unroll
          for (int i = 0; i < 4; ++i) f[i] = mul2(mul2(f[i], both(inv)), g[i]);
        }
        if (p.gate) {
          unpack8(__ldg(p.gate + c), g);
#pragma unroll
          for (int i = 0; i < 4; ++i) f[i] = mul2(f[i], g[i]);
        }
        unpack8(r[j], o);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          o[i] = add2(mul2(both(p.alpha), o[i]), mul2(both(m), f[i]));
        r[j] = pack8(o);
        p.r_out[base + c] = r[j];
      }
    }
  }
  if constexpr (BEFORE) {
    const float inv = rms_inverse(block_squares<VPT>(r, red[1]), p, p.pre_eps);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = tid + j * nt;
      if (c < p.vec) {
        float2 f[4], g[4];
        unpack8(r[j], f);
        unpack8(__ldg(p.pre_w + c), g);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = mul2(mul2(f[i], both(inv)), g[i]);
        r[j] = pack8(f);
        if (p.a) p.a[base + c] = r[j];
      }
    }
  }
  if (p.codes) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < VPT; ++j) m = max(m, abs_bits(r[j]));
    const float amax = __uint_as_float(block_max(m, redm) << 16);
    const float s = amax == 0.0f ? 1.0f : __fdiv_rn(amax, 127.0f);
    const float inv = s >= 8.6736174e-19f && s <= 1.1529215e18f ? __frcp_rn(s) : 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = tid + j * nt;
      if (c < p.vec) {
        float2 f[4];
        unpack8(r[j], f);
        p.codes[base + c] = codes8(f, s, inv);
      }
    }
    if (tid == 0) p.scales[t] = s;
  }
}

template <bool AFTER, bool BEFORE>
auto pick(int vpt) {
  return vpt == 1   ? rows_kernel<1, AFTER, BEFORE>
         : vpt == 2 ? rows_kernel<2, AFTER, BEFORE>
         : vpt == 3 ? rows_kernel<3, AFTER, BEFORE>
                    : rows_kernel<4, AFTER, BEFORE>;
}

cudaError_t launch_rows(int64_t rows, RowParams& p, cudaStream_t st) {
  p.rows = rows;
  // Few rows: a thread per vector.  Many: three or four vectors per thread, which
  // shares a row's fixed cost (two means, two inverse roots) between them and still
  // leaves enough rows on an SM (T = 8192, H = 4096, both norms: 47.5 us with 128
  // threads, 54.3 with 96, 52.5 with 256, 65.2 with 512; H = 2816: 35.6 us with three
  // on 128 threads, 36.3 with four on 96).  A row of up to 1024
  // values is one warp's; then eight of them share a block.
  int nt = std::min(1024, (p.vec + 31) / 32 * 32), per = 1;
  if (rows > 2 * device_sm_count()) {
    nt = (p.vec + 127) / 128 * 32;
    const int nt3 = (p.vec + 95) / 96 * 32;
    if (nt3 <= 1024 && 3 * nt3 <= 4 * nt) nt = nt3;
    if (p.vec <= 128) nt = 32, per = 8;
  }
  const int vpt = (p.vec + nt - 1) / nt;
  auto kern = p.y && p.pre_w ? pick<true, true>(vpt)
              : p.y          ? pick<true, false>(vpt)
              : p.pre_w      ? pick<false, true>(vpt)
                             : pick<false, false>(vpt);
  return launch_ex(kern, dim3((unsigned)((rows + per - 1) / per)), dim3(nt, per), 0, st, true, p);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_quantize_rows_i8(const moe_bf16* src, int64_t rows, int cols, int8_t* codes,
                                float* scales, cudaStream_t stream) {
  if (rows < 0 || cols <= 0 || cols % 8 != 0) return MOE_ERR_INVALID_ARG;
  if (cols > MOE_MAX_ROW || rows >= (int64_t(1) << 31)) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (!src || !codes || !scales || !aligned(src, 16) || !aligned(codes, 8))
    return MOE_ERR_INVALID_ARG;
  RowParams p{};
  p.r = reinterpret_cast<const uint4*>(src);
  p.codes = reinterpret_cast<uint2*>(codes);
  p.scales = scales;
  p.vec = cols / 8;
  p.n = cols;
  p.inv_n = 1.0 / cols;
  return launch_rows(rows, p, stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_block_norm(int64_t T, int H, const moe_block_norm_params* q,
                          cudaStream_t stream) {
  if (T < 0 || H <= 0 || !q) return MOE_ERR_INVALID_ARG;
  if (H % 8 != 0 || H > MOE_MAX_ROW || T >= (int64_t(1) << 24)) return MOE_ERR_UNSUPPORTED;
  if (!std::isfinite(q->alpha) || !std::isfinite(q->beta)) return MOE_ERR_INVALID_ARG;
  for (const float eps : {q->post_eps, q->pre_eps})
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return MOE_ERR_INVALID_ARG;
  // what a half that does not run would use, and a half without an output
  if (!q->y && (q->post_w || q->gate || q->token_gate || q->r_out)) return MOE_ERR_INVALID_ARG;
  if (!q->pre_w && (q->a || q->codes || q->scales)) return MOE_ERR_INVALID_ARG;
  if (!q->y && !q->pre_w) return MOE_ERR_INVALID_ARG;
  if ((q->codes == nullptr) != (q->scales == nullptr)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!q->r || (q->y && !q->r_out) || (q->pre_w && !q->a && !q->codes))
    return MOE_ERR_INVALID_ARG;
  for (const void* v : {(const void*)q->y, (const void*)q->r, (const void*)q->post_w,
                        (const void*)q->gate, (const void*)q->pre_w, (const void*)q->r_out,
                        (const void*)q->a})
    if (!aligned(v, 16)) return MOE_ERR_INVALID_ARG;
  if (!aligned(q->codes, 8)) return MOE_ERR_INVALID_ARG;
  auto vec = [](const moe_bf16* v) { return reinterpret_cast<const uint4*>(v); };
  RowParams p{};
  p.y = vec(q->y);
  p.r = vec(q->r);
  p.post_w = vec(q->post_w);
  p.gate = vec(q->gate);
  p.pre_w = vec(q->pre_w);
  p.token_gate = q->token_gate;
  p.alpha = q->alpha;
  p.beta = q->beta;
  p.post_eps = q->post_eps;
  p.pre_eps = q->pre_eps;
  p.r_out = reinterpret_cast<uint4*>(q->r_out);
  p.a = reinterpret_cast<uint4*>(q->a);
  p.codes = reinterpret_cast<uint2*>(q->codes);
  p.scales = q->scales;
  p.vec = H / 8;
  p.n = H;
  p.inv_n = 1.0 / H;
  return launch_rows(T, p, stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
