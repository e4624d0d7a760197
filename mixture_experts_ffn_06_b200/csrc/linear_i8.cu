// linear_i8.cu -- the 8-bit integer product with scales for each token and
// channel (moe_linear_i8): v[t,n] = fl(sum_k x[t,k] w[n,k]) fl(sx[t] sw[n]),
// plain or gated (Act(gate) up), on the sm_100a tensor cores
// (tcgen05.mma kind::i8, 32-bit integer accumulators).
//
// The weights are the M side of each MMA and the tokens its N side: a lane of
// the accumulator is a channel and a column a token, so a warp writes 32
// consecutive channels of a token at once, and few tokens cost few columns
// instead of padding a 128-row tile.  A gated tile of 128 weight rows holds, for
// each epilogue warp, 16 gate rows and then the matching 16 up rows (one 3D
// TMA box over w [2, I, K]), so lane l's partner is lane l + 16.
//
// Which form runs depends on what bounds it (linear_plan.cuh has the rules):
//   few tokens, streaming w: small independent blocks with mma.sync
//               (linear_i8_few_kernel; gated 4096 x 28672, T = 1: 20.5 us, 5.7 TB/s, 87 % of
//               the measured copy bandwidth);
//   fewer tiles than SMs and K long enough: a tile per cluster of up to 8 CTAs that
//               split K; each parks its partial sums in shared memory and adds
//               up a slice of the columns over all CTAs' (integers: the order
//               of the sum does not matter; gated 2816 x 4224, T = 64: 7.3 us, latency);
//   up to 128 tokens otherwise, streaming w: a CTA per tile, two or three to an SM
//               (gated 4096 x 28672, T = 64: 21.9 us, 5.4 TB/s);
//   more (bound by the tensor cores, under the power limit): persistent CTAs or
//               CTA pairs (M = 256) walk the tiles, two accumulators in TMEM so
//               that a tile's epilogue runs beside the next one's MMAs, or one of
//               twice the columns, which reads each weight tile half as often (gated
//               4096 x 28672, T = 4096: 284 to 341 us, 2.8 to 3.4 POPS, by the power limit).
// The tcgen05 forms have one TMA warp, one MMA warp and 4, 8 or 16 epilogue warps.
// Every mbarrier wait is bounded (tc_ptx.cuh); after a timeout the block
// records MOE_ERR_TIMEOUT, waits for its own copies and MMAs and frees TMEM.
#include <algorithm>
#include <atomic>

#include "linear_plan.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace {

constexpr uint64_t kTimeoutNs = 1000000000ull;  // 1 s per wait
constexpr int kMaxDev = 64;

struct LinParams {
  const float *xs, *ws;
  int64_t T;
  int N;        // rows of w
  int NO;       // channels of the output
  int KB;       // k-blocks of 128
  int act;
  int tn;       // token columns of one MMA (of the pair)
  int nsub;     // MMAs (token sub-tiles) that share a weight tile
  int nbuf;     // accumulators in TMEM
  int stages;
  uint32_t MT, TT;  // weight tiles (of CG x 128 rows) and token tiles (nsub x tn)
  int panel;    // token tiles per panel of the tile order
  uint32_t cols;  // TMEM columns
  __nv_bfloat16* out;
  float* out_f32;
  uint32_t* err;
};

struct LinCtl {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t tmem_full[2];
  uint64_t tmem_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int32_t abort_flag;
};
static_assert(sizeof(LinCtl) + 4096 <= kLinStatic, "with the token scales of sixteen warps");

// mbar_wait, with the first tries made here: the timed wait reads the global
// timer, which costs as much as several k-blocks.
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity,
                                         volatile int32_t* abort_flag, uint32_t* err) {
#pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (mbar_test(bar, parity)) return true;
  return mbar_wait(bar, parity, abort_flag, kTimeoutNs, err);
}
__device__ __forceinline__ bool wait_for_cluster(uint32_t bar, uint32_t parity,
                                                 volatile int32_t* abort_flag, uint32_t* err) {
#pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (mbar_test_cluster(bar, parity)) return true;
  return mbar_wait_cluster(bar, parity, abort_flag, kTimeoutNs, err);
}

// Both activations as g sigma(x): 0.5 (1 + tanh v) = sigma(2v) does not cancel
// where v is large and negative.  In units of 2^-23, __expf is within 2 + 1.173 |x|, GELU's x
// (six roundings) brings 3 |x|, the sum, the division and the product with the up value
// 3 together: 5 + 1.2 max(-x, 0) and 5 + 4.2 max(-x, 0), as the exponential counts by sigma(-x).
// At x = -8 that is a 400th of the rounding to bf16 (2^-9), and expf with an IEEE division,
// which leave 3 at any x, cost too much there: gated 4096 x 28672, T = 8 24.8 us and here
// 21.0, 1408 x 2816, T = 16384 65 and 56; an exponential with its argument's remainder
// (4 at any x) 21.0 and 61.
template <int ACT>
__device__ __forceinline__ float lin_act(float g) {
  const float e = ACT == MOE_ACT_SILU
                      ? -g
                      : -1.5957691216057308f * fmaf(0.044715f * g, g * g, g);  // -2 v
  return __fdividef(g, 1.0f + __expf(e));
}

// 16 bytes of a weight row, which pass through once
__device__ __forceinline__ int4 ld_stream(const int4* p) {
  int4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

struct LinTile {
  int mt;
  int64_t t0;  // first token
};

// Tile u: panels of ``panel`` token tiles, then the weight tile, then the token
// tile inside the panel, so that the tiles running at once share weight tiles
// and the panel's tokens stay in L2 while the weights pass by once per panel.
__device__ __forceinline__ LinTile lin_tile(uint32_t u, const LinParams& p) {
  const uint32_t per = (uint32_t)p.panel * p.MT;
  const uint32_t pn = u / per, in = u - pn * per;
  const uint32_t pw = min((uint32_t)p.panel, p.TT - pn * p.panel);
  const uint32_t mt = in / pw;
  return LinTile{(int)mt, (int64_t)(pn * p.panel + in - mt * pw) * p.nsub * p.tn};
}

// A lane of the epilogue: its channel and scales.  The lanes of a pair (plain:
// lanes 2i and 2i + 1, neighbouring channels; gated: l and l + 16, gate and up
// row of a channel) each finish one of two token columns for both their rows.
template <bool GATED>
struct LaneOut {
  int n;         // first output channel
  bool ok;       // it exists (plain: n; n + 1 is checked where it is stored)
  bool hi;       // second lane of the pair: takes the second column
  float s0, s1;  // scales of the pair's two rows

  __device__ __forceinline__ void init(const LinParams& p, int row, int lane) {
    if (GATED) {
      hi = lane >= 16;
      n = (row >> 5) * 16 + (lane & 15);
      ok = n < p.NO;
      s0 = ok ? __ldg(p.ws + n) : 0.f;
      s1 = ok ? __ldg(p.ws + p.NO + n) : 0.f;
    } else {
      hi = (lane & 1) != 0;
      n = row & ~1;
      ok = n < p.NO;
      s0 = ok ? __ldg(p.ws + n) : 0.f;
      s1 = n + 1 < p.NO ? __ldg(p.ws + n + 1) : 0.f;
    }
  }

  // NP pairs of columns of this lane's row: a[j], b[j] are columns of tokens
  // t + stride j and t + stride j + 1 (tokens from t_end on are not stored),
  // sx[j] the scale of the one this lane finishes.  No branch between the pairs, so
  // that their chains overlap.
  template <int NP>
  __device__ __forceinline__ void store(const LinParams& p, int64_t t, int64_t t_end, int stride,
                                        const int32_t (&a)[NP], const int32_t (&b)[NP],
                                        const float (&sx)[NP]) const {
    float v0[NP], v1[NP];
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const int32_t got = __shfl_xor_sync(0xffffffffu, hi ? a[j] : b[j], GATED ? 16 : 1);
      const float2 s = mul2(make_float2(sx[j], sx[j]), make_float2(s0, s1));
      const float2 v = mul2(make_float2((float)(hi ? got : a[j]), (float)(hi ? b[j] : got)), s);
      v0[j] = v.x;
      v1[j] = v.y;
    }
    if (GATED) {
      if (p.act == MOE_ACT_SILU) {
#pragma unroll
        for (int j = 0; j < NP; ++j) v0[j] = lin_act<MOE_ACT_SILU>(v0[j]) * v1[j];
      } else {
#pragma unroll
        for (int j = 0; j < NP; ++j) v0[j] = lin_act<MOE_ACT_GELU_TANH>(v0[j]) * v1[j];
      }
    }
    const int64_t tok = t + (hi ? 1 : 0);
    const int64_t step = (int64_t)stride * p.NO;
    const bool full = t + (NP - 1) * stride + 1 < t_end;
    if (GATED && NP % 2 == 0 && full && !p.out_f32 && (p.NO & 1) == 0) {
      // neighbouring channels swap one of two tokens, for 4-byte stores
      const bool odd = (n & 1) != 0;
      __nv_bfloat16* o = p.out + (tok + (odd ? stride : 0)) * p.NO + (n & ~1);
#pragma unroll
      for (int j = 0; j + 1 < NP; j += 2, o += 2 * step) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v0[j], v0[j + 1]);
        const uint32_t mine = *reinterpret_cast<const uint32_t*>(&h);
        const uint32_t other = __shfl_xor_sync(0xffffffffu, mine, 1);
        // even: (mine.lo, other.lo) of token j; odd: (other.hi, mine.hi) of j + 1
        const uint32_t w = __byte_perm(mine, other, odd ? 0x3276 : 0x5410);
        if (ok) *reinterpret_cast<uint32_t*>(o) = w;
      }
      return;
    }
    if (!ok) return;
    const int64_t at = tok * p.NO + n;
    if (full) {
      write<NP>(p, at, step, NP, v0, v1);
    } else {
      int64_t left = t_end - tok;  // pairs j < left / stride are real
      left = left > 0 ? (left + stride - 1) / stride : 0;
      write<NP>(p, at, step, (int)(left < NP ? left : NP), v0, v1);
    }
  }

  template <int NP>
  __device__ __forceinline__ void write(const LinParams& p, int64_t at, int64_t step, int nv,
                                        const float (&v0)[NP], const float (&v1)[NP]) const {
    if (p.out) {
      __nv_bfloat16* o = p.out + at;
#pragma unroll
      for (int j = 0; j < NP; ++j, o += step) {
        if (j >= nv) continue;
        if (GATED) {
          *o = __float2bfloat16_rn(v0[j]);
        } else if ((p.NO & 1) == 0) {
          *reinterpret_cast<__nv_bfloat162*>(o) = __floats2bfloat162_rn(v0[j], v1[j]);
        } else {
          o[0] = __float2bfloat16_rn(v0[j]);
          if (n + 1 < p.NO) o[1] = __float2bfloat16_rn(v1[j]);
        }
      }
    }
    if (p.out_f32) {
      float* o = p.out_f32 + at;
#pragma unroll
      for (int j = 0; j < NP; ++j, o += step) {
        if (j >= nv) continue;
        if (GATED) {
          *o = v0[j];
        } else if ((p.NO & 1) == 0) {
          *reinterpret_cast<float2*>(o) = make_float2(v0[j], v1[j]);
        } else {
          o[0] = v0[j];
          if (n + 1 < p.NO) o[1] = v1[j];
        }
      }
    }
  }
};

// CG = 2: CTA pairs walk the tiles.  CG = 1: single CTAs do, or with SPLIT > 1 a cluster
// of SPLIT CTAs that share K takes one tile.  EW epilogue warps: 16 beside the MMAs of
// the next tile (gated 1408 x 2816, T = 16384: 53 us, with eight 59), 8 where sums are
// handed over (2112 x 2816, T = 128: 6.9 us, with four 7.3), 4 where several CTAs share
// an SM.
template <int CG, bool GATED, int SPLIT, int EW>
__global__ void __launch_bounds__(64 + 32 * EW, 1)
linear_i8_kernel(const __grid_constant__ CUtensorMap tmW,
                 const __grid_constant__ CUtensorMap tmX, const LinParams p) {
  static_assert(CG == 1 || SPLIT == 1, "K is split over single CTAs");
  static_assert(EW == 4 || EW == 8 || EW == 16, "whole warps for each 32 accumulator lanes");
  extern __shared__ uint8_t smem_raw[];
  __shared__ LinCtl ctl_s;
  __shared__ __align__(16) float sx_s[SPLIT == 1 ? EW : 1][EW == 4 ? 4 : 32 / EW][32];
  LinCtl* ctl = &ctl_s;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t sub_bytes = (uint32_t)p.tn / CG * 128u;
  const uint32_t b_bytes = sub_bytes * p.nsub;
  const uint32_t sA = base;
  const uint32_t sB = base + p.stages * kABytes;
  volatile int32_t* abort_flag = &ctl->abort_flag;
  // (the warp index by a shuffle, so that the compiler knows it is one per warp)
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = (CG == 2 || SPLIT > 1) ? cluster_ctarank() : 0u;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(smem_u32(&ctl->full[s]), 1);
      mbar_init(smem_u32(&ctl->empty[s]), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&ctl->tmem_full[a]), 1);
      mbar_init(smem_u32(&ctl->tmem_empty[a]), EW * CG);  // one per epilogue warp
    }
    mbar_init(smem_u32(&ctl->drain), 1);
    ctl->abort_flag = 0;
    mbar_init_fence();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
  }
  if (warp == 1) {
    if (CG == 2)
      tmem_alloc_pair(smem_u32(&ctl->tmem_base), p.cols);
    else
      tmem_alloc(smem_u32(&ctl->tmem_base), p.cols);
  }
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();  // the peer's barriers are initialised
  tc_fence_after();
  const uint32_t tmem_base = ctl->tmem_base;
  pdl_trigger();  // not before the block owns its columns (pdl_trigger's comment)

  // (fewer than 2^31 tiles: the host checks)
  const uint32_t total = (uint32_t)p.MT * p.TT;
  const uint32_t unit0 = CG == 2 ? cluster_id_x() : blockIdx.x / SPLIT;
  const uint32_t step = CG == 2 ? nclusters_x() : SPLIT == 1 ? gridDim.x : total;
  const int kb0 = (int)(rank * p.KB / SPLIT) * (CG == 1);
  const int kb1 = CG == 1 ? (int)((rank + 1) * p.KB / SPLIT) : p.KB;

  if (warp == 0) {
    // ------------------------------------------------------ TMA producer
    int stage = 0;
    uint32_t phase = 0, filled = 0, last = 0;  // bit s: stage s filled, its parity
    bool ok = true;
    for (uint32_t u = unit0; ok && u < total; u += step) {
      const LinTile tl = lin_tile(u, p);
      const int mrow = (tl.mt * CG + (int)(CG == 2 ? rank : 0)) * (GATED ? 64 : 128);
      const int64_t tr = tl.t0 + (CG == 2 ? (int64_t)rank * (p.tn / 2) : 0);
      // each weight tile starts elsewhere in K and wraps round (integer sums
      // do not mind), so that the CTAs do not all read the same lines of x
      // at the same time
      int kb = kb0 + (int)(tl.mt * 5u % (uint32_t)(kb1 - kb0));
      for (int i = kb0; i < kb1; ++i, kb = kb + 1 < kb1 ? kb + 1 : kb0) {
        ok = __all_sync(0xffffffffu,
                        wait_for(smem_u32(&ctl->empty[stage]), phase ^ 1u, abort_flag, p.err));
        if (!ok) break;
        if (elect_one()) {
          uint32_t fb = smem_u32(&ctl->full[stage]);
          // with a pair both CTAs' bytes complete on CTA 0's barrier
          if (CG == 1 || rank == 0) mbar_expect_tx(fb, CG * (kABytes + b_bytes));
          if (CG == 2) fb &= kPeerBitMask;
          const uint32_t a = sA + stage * kABytes, b = sB + stage * b_bytes;
          const int32_t kx = kb * 128;
          if (GATED) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              if (CG == 2)
                tma_load_3d_pair(a + q * 4096, &tmW, kx, mrow + 16 * q, 0, fb);
              else
                tma_load_3d(a + q * 4096, &tmW, kx, mrow + 16 * q, 0, fb);
            }
          } else {
            if (CG == 2)
              tma_load_2d_pair(a, &tmW, kx, mrow, fb);
            else
              tma_load_2d(a, &tmW, kx, mrow, fb);
          }
          for (int s = 0; s < p.nsub; ++s) {
            if (CG == 2)
              tma_load_2d_pair(b + s * sub_bytes, &tmX, kx, (int32_t)(tr + s * p.tn), fb);
            else
              tma_load_2d(b + s * sub_bytes, &tmX, kx, (int32_t)(tr + s * p.tn), fb);
          }
        }
        __syncwarp();
        filled |= 1u << stage;
        last = (last & ~(1u << stage)) | (phase << stage);
        if (++stage == p.stages) { stage = 0; phase ^= 1u; }
      }
    }
    if (!ok && lane == 0 && (CG == 1 || rank == 0)) {
      // let the copies already issued land before the block exits
      int32_t none = 0;
      volatile int32_t* never = &none;
      for (int s = 0; s < p.stages; ++s)
        if ((filled >> s) & 1u)
          mbar_wait(smem_u32(&ctl->full[s]), (last >> s) & 1u, never, kTimeoutNs, p.err);
    }
    __syncwarp();
  } else if (warp == 1) {
    // --------------------------------------------------------- MMA issuer
    // The whole warp walks the k-blocks and one lane issues (elect_one): an MMA of up to
    // 192 columns would otherwise take longer to issue than to run.
    if (CG == 1 || rank == 0) {
      const uint32_t idesc = idesc_i8_s32(128 * CG, p.tn);
      int stage = 0, buf = 0;
      uint32_t phase = 0, buf_phase = 0;
      bool ok = true;
      for (uint32_t u = unit0; ok && u < total; u += step) {
        const uint32_t eb = smem_u32(&ctl->tmem_empty[buf]);
        ok = CG == 2 ? wait_for_cluster(eb, buf_phase ^ 1u, abort_flag, p.err)
                     : wait_for(eb, buf_phase ^ 1u, abort_flag, p.err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem_base + buf * 256;
        for (int kb = kb0; kb < kb1; ++kb) {
          ok = __all_sync(0xffffffffu,
                          wait_for(smem_u32(&ctl->full[stage]), phase, abort_flag, p.err));
          if (!ok) break;
          tc_fence_after();
          const uint64_t ad = sw128_kmajor_desc(sA + stage * kABytes);
          const uint64_t bd = sw128_kmajor_desc(sB + stage * b_bytes);
          const uint32_t first = kb != kb0 ? 1u : 0u;
          if (elect_one()) {
            // four MMAs of 32 bytes of K each for each sub-tile
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_i8<CG>(d, ad + 2u * kk, bd + 2u * kk, idesc, first | (kk != 0));
            if (p.nsub == 2) {
              const uint64_t b2 = bd + (sub_bytes >> 4);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                umma_i8<CG>(d + 256, ad + 2u * kk, b2 + 2u * kk, idesc, first | (kk != 0));
            }
            if (CG == 2)
              umma_commit_pair_mc(smem_u32(&ctl->empty[stage]), 0x3);
            else
              umma_commit(smem_u32(&ctl->empty[stage]));
          }
          __syncwarp();
          if (++stage == p.stages) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        if (elect_one()) {
          if (CG == 2)
            umma_commit_pair_mc(smem_u32(&ctl->tmem_full[buf]), 0x3);
          else
            umma_commit(smem_u32(&ctl->tmem_full[buf]));
        }
        __syncwarp();
        if (++buf == p.nbuf) { buf = 0; buf_phase ^= 1u; }
      }
      if (__any_sync(0xffffffffu, !ok || *abort_flag)) {
        // wait for the MMAs already issued before TMEM is released
        if (elect_one()) {
          int32_t none = 0;
          volatile int32_t* never = &none;
          if (CG == 2)
            umma_commit_pair(smem_u32(&ctl->drain));
          else
            umma_commit(smem_u32(&ctl->drain));
          mbar_wait(smem_u32(&ctl->drain), 0, never, kTimeoutNs, p.err);
        }
        __syncwarp();
      }
    }
  } else {
    // ----------------------------------------------------------- epilogue
    // Warp w reads TMEM lanes [32 (w % 4), 32 (w % 4) + 32); the EW / 4 warps of the
    // same lanes take their 32-column chunks in turn.
    const int q = warp & 3;
    constexpr int HALVES = EW / 4;
    constexpr int CHUNKS = EW == 4 ? 4 : 8 / HALVES;  // of a warp (EW = 4: tn <= 128)
    const int c_first = 32 * ((warp - 2) >> 2);
    const uint32_t lanes = (uint32_t)(q * 32) << 16;
    const uint32_t empty0 = CG == 2 ? mapa_shared(smem_u32(&ctl->tmem_empty[0]), 0) : 0u;
    const uint32_t empty1 = CG == 2 ? mapa_shared(smem_u32(&ctl->tmem_empty[1]), 0) : 0u;
    int buf = 0;
    uint32_t buf_phase = 0;
    for (uint32_t u = unit0; u < total; u += step) {
      const LinTile tl = lin_tile(u, p);
      LaneOut<GATED> lo;
      lo.init(p, (tl.mt * CG + (int)(CG == 2 ? rank : 0)) * 128 + q * 32 + lane, lane);
      // Token scales of this warp's chunks, brought to shared memory before the wait
      // and by the parity of their token: a lane reads the 16 of its own columns of
      // a chunk as four vectors.
      auto token_scales = [&](int64_t ts) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i) {
          const int64_t tok = ts + c_first + 32 * HALVES * i + lane;
          sx_s[warp - 2][i][(lane & 1) * 16 + (lane >> 1)] = tok < p.T ? __ldg(p.xs + tok) : 0.f;
        }
        __syncwarp();
      };
      if constexpr (SPLIT == 1) token_scales(tl.t0);
      const bool got = wait_for(smem_u32(&ctl->tmem_full[buf]), buf_phase, abort_flag, p.err);
      // warp-uniform decision; also reconverges the warp for tcgen05.ld
      if (!__all_sync(0xffffffffu, got)) break;
      tc_fence_after();
      const uint32_t tb = tmem_base + lanes + buf * 256;
      if constexpr (SPLIT > 1) {
        // partial sums [column][128 rows] over the ring, which is idle now
        int32_t* part = reinterpret_cast<int32_t*>(gbase) + q * 32 + lane;
#pragma unroll 1
        for (int c = c_first; c < p.tn; c += 32 * HALVES) {
          uint32_t v[32];
          tmem_ld32(tb + c, v);
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (c + j < p.tn) part[(c + j) * 128] = (int32_t)v[j];
        }
      } else {
        for (int s = 0; s < p.nsub; ++s) {
          const int64_t ts = tl.t0 + (int64_t)s * p.tn;
          // columns past tn belong to the next sub-tile or to nobody
          const int64_t t_end = ts + p.tn < p.T ? ts + p.tn : p.T;
          if (s > 0) token_scales(ts);
#pragma unroll
          for (int i = 0; i < CHUNKS; ++i) {
            const int c = c_first + 32 * HALVES * i;
            if (c >= p.tn || ts + c >= p.T) break;
            uint32_t v[32];
            tmem_ld32(tb + s * 256 + c, v);
            const float* sx_w = sx_s[warp - 2][i];
#pragma unroll
            for (int h = 0; h < 32; h += 16) {
              int32_t a[8], b[8];
              float sx[8];
#pragma unroll
              for (int j = 0; j < 8; j += 4)
                *reinterpret_cast<float4*>(sx + j) = *reinterpret_cast<const float4*>(
                    sx_w + (lo.hi ? 16 : 0) + h / 2 + j);
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                a[j] = (int32_t)v[h + 2 * j];
                b[j] = (int32_t)v[h + 2 * j + 1];
              }
              lo.template store<8>(p, ts + c + h, t_end, 2, a, b, sx);
            }
          }
        }
      }
      // this warp is done with the accumulator: one arrival per warp (on CTA
      // 0's barrier when the pair shares the MMA)
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CG == 2)
          mbar_arrive_cluster(buf ? empty1 : empty0);
        else
          mbar_arrive(smem_u32(&ctl->tmem_empty[buf]));
      }
      if (++buf == p.nbuf) { buf = 0; buf_phase ^= 1u; }
    }
  }

  if constexpr (SPLIT > 1) {
    __syncwarp();
    cluster_sync();  // every CTA's partial sums are in its shared memory
    if (warp >= 2 && !*abort_flag) {
      // CTA r finishes the column pairs r, r + SPLIT, ..., NP at a time; the
      // EW / 4 warps of a row quarter take turns
      constexpr int NP = 16 / SPLIT < 4 ? 16 / SPLIT : 4;
      const int q = warp & 3, row = q * 32 + lane, half = (warp - 2) >> 2;
      const LinTile tl = lin_tile(unit0, p);
      LaneOut<GATED> lo;
      lo.init(p, tl.mt * 128 + row, lane);
      uint32_t src[SPLIT];
#pragma unroll
      for (int r = 0; r < SPLIT; ++r) src[r] = mapa_shared(smem_u32(gbase) + row * 4, r);
      constexpr int GROUP = 2 * SPLIT * NP;  // columns of one turn, at most 32
      const int64_t t_end = tl.t0 + p.tn < p.T ? tl.t0 + p.tn : p.T;
      for (int c0 = GROUP * half; c0 < p.tn && tl.t0 + c0 < p.T; c0 += GROUP * (EW / 4)) {
        const int c = c0 + 2 * (int)rank;
        int32_t a[NP], b[NP];
        float sx[NP];
#pragma unroll
        for (int j = 0; j < NP; ++j) {
          const int64_t tok = tl.t0 + c + 2 * SPLIT * j + (lo.hi ? 1 : 0);
          sx[j] = tok < p.T ? __ldg(p.xs + tok) : 0.f;
          a[j] = b[j] = 0;
        }
#pragma unroll
        for (int r = 0; r < SPLIT; ++r) {
          int32_t ua[NP], ub[NP];
#pragma unroll
          for (int j = 0; j < NP; ++j) {
            const uint32_t at = src[r] + (uint32_t)(c + 2 * SPLIT * j) * 512u;
            ua[j] = ub[j] = 0;
            if (tl.t0 + c + 2 * SPLIT * j < t_end) {
              ua[j] = ld_cluster_s32(at);
              ub[j] = ld_cluster_s32(at + 512u);
            }
          }
#pragma unroll
          for (int j = 0; j < NP; ++j) {
            a[j] += ua[j];
            b[j] += ub[j];
          }
        }
        lo.template store<NP>(p, tl.t0 + c, t_end, 2 * SPLIT, a, b, sx);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (CG == 2 || SPLIT > 1) cluster_sync();  // no peer still uses this CTA's memory or TMEM
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    if (CG == 2)
      tmem_dealloc_pair(tmem_base, p.cols);
    else
      tmem_dealloc(tmem_base, p.cols);
  }
}

// --------------------------------------------------------- at most 16 tokens
// A block of W warps takes 16 weight rows (gated: 8 gate rows and the
// matching 8 up rows) and all tokens; the warps take 64-byte steps of K in turn.
// mma.sync m16n8k32 with the weights as A and the tokens as B, both read
// straight into fragments: lane (g, q) loads 16 bytes at 16 q of a step, of the
// rows g and g + 8 and of token g, and uses the four words as the K slots of two
// MMAs.  That permutes K the same way on both sides.  U steps are requested
// before the first is used; nothing but the final sum over the warps meets at a
// barrier.

__device__ __forceinline__ void mma_i8(int (&d)[4], int a0, int a1, int a2, int a3, int b0,
                                       int b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int NB, bool GATED, int W>  // NB tiles of 8 tokens
__global__ void __launch_bounds__(32 * W)
linear_i8_few_kernel(const int4* __restrict__ x, const int4* __restrict__ w, int vec,
                     const LinParams p) {
  constexpr int U = W == 16 ? 3 : 4;
  __shared__ int part[W][NB * 4][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int n0 = blockIdx.x * (GATED ? 8 : 16);
  const int T = (int)p.T;
  // rows past the end: read the last one, store nothing
  const int ra = min(n0 + g, p.NO - 1);
  const int rb = GATED ? p.NO + ra : min(n0 + g + 8, p.NO - 1);
  const int4* wa = w + (int64_t)ra * vec;
  const int4* wb = w + (int64_t)rb * vec;
  pdl_wait();
  pdl_trigger();
  int acc[NB][4];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[b][i] = 0;
  const int4 zero = make_int4(0, 0, 0, 0);
  for (int v0 = 4 * warp + q; v0 - q < vec; v0 += 4 * W * U) {
    int4 a[U], c[U], t[U][NB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int v = v0 + 4 * W * u;
      a[u] = v < vec ? ld_stream(wa + v) : zero;
      c[u] = v < vec ? ld_stream(wb + v) : zero;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int v = v0 + 4 * W * u;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int tok = 8 * b + g;
        t[u][b] = v < vec && tok < T ? __ldg(x + (int64_t)tok * vec + v) : zero;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        mma_i8(acc[b], a[u].x, c[u].x, a[u].y, c[u].y, t[u][b].x, t[u][b].y);
        mma_i8(acc[b], a[u].z, c[u].z, a[u].w, c[u].w, t[u][b].z, t[u][b].w);
      }
  }
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) part[warp][b * 4 + i][lane] = acc[b][i];
  __syncthreads();
  // a thread finishes one token of rows g and g + 8: entries i and i + 2
  if (threadIdx.x >= NB * 64) return;
  const int b = threadIdx.x >> 6, i = (threadIdx.x >> 5) & 1;
  int s0 = 0, s1 = 0;
#pragma unroll
  for (int k = 0; k < W; ++k) {
    s0 += part[k][b * 4 + i][lane];
    s1 += part[k][b * 4 + i + 2][lane];
  }
  const int tok = 8 * b + 2 * q + i, n = n0 + g;
  if (tok >= T || n >= p.NO) return;
  const float sx = __ldg(p.xs + tok);
  const int64_t at = (int64_t)tok * p.NO + n;
  float v = __fmul_rn((float)s0, __fmul_rn(sx, __ldg(p.ws + n)));
  if (GATED) {
    const float u = __fmul_rn((float)s1, __fmul_rn(sx, __ldg(p.ws + p.NO + n)));
    v = (p.act == MOE_ACT_SILU ? lin_act<MOE_ACT_SILU>(v) : lin_act<MOE_ACT_GELU_TANH>(v)) * u;
  } else if (n + 8 < p.NO) {
    const float u = __fmul_rn((float)s1, __fmul_rn(sx, __ldg(p.ws + n + 8)));
    if (p.out) p.out[at + 8] = __float2bfloat16_rn(u);
    if (p.out_f32) p.out_f32[at + 8] = u;
  }
  if (p.out) p.out[at] = __float2bfloat16_rn(v);
  if (p.out_f32) p.out_f32[at] = v;
}

// ------------------------------------------------------------------- host

// Map of the gated weight as [2, I, K] bytes: box {128, 16, 2}, 16 gate rows and
// then the matching 16 up rows (rows past I read as zero).
cudaError_t make_gated_map(CUtensorMap* m, const void* ptr, uint64_t K, uint64_t I) {
  const EncodeTiledFn enc = encode_tiled();
  if (!enc) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {K, I, 2};
  const cuuint64_t strides[2] = {K, K * I};
  const cuuint32_t box[3] = {128, 16, 2};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(ptr), dims,
                         strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// The shared-memory opt-in of a kernel, once per device.
template <int CG, bool GATED, int SPLIT, int EW>
cudaError_t set_smem(int dev) {
  static std::atomic<bool> ready[kMaxDev];
  if (dev >= 0 && dev < kMaxDev && ready[dev].load()) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(linear_i8_kernel<CG, GATED, SPLIT, EW>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kSmemMax - kLinStatic);
  if (e == cudaSuccess && dev >= 0 && dev < kMaxDev) ready[dev].store(true);
  return e;
}

template <int CG, bool GATED, int SPLIT, int EW>
cudaError_t launch_linear(const LinParams& p, const int8_t* x, const int8_t* w, int K,
                          const LinPlan& pl, cudaStream_t st) {
  auto kern = linear_i8_kernel<CG, GATED, SPLIT, EW>;
  CUtensorMap mw, mx;
  cudaError_t e = GATED ? make_gated_map(&mw, w, K, p.NO) : make_tma_map_e4m3(&mw, w, K, p.N, 128);
  if (e == cudaSuccess) e = make_tma_map_e4m3(&mx, x, K, p.T, p.tn / CG);
  if (e != cudaSuccess) return e;
  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if ((e = set_smem<CG, GATED, SPLIT, EW>(dev)) != cudaSuccess) return e;
  constexpr int per = CG * SPLIT;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(pl.blocks * per));
  cfg.blockDim = dim3(64 + 32 * EW);
  cfg.dynamicSmemBytes = pl.smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = per;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = per > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, mw, mx, p);
}

template <int NB, bool GATED, int W>
cudaError_t launch_few(const LinParams& p, int blocks, const int8_t* x, const int8_t* w, int K,
                       cudaStream_t st) {
  return launch_ex(linear_i8_few_kernel<NB, GATED, W>, dim3(blocks), dim3(32 * W), 0, st, true,
                   reinterpret_cast<const int4*>(x), reinterpret_cast<const int4*>(w), K / 16, p);
}

// Clusters of SPLIT CTAs that run at once on the current device, a CTA to an SM.
template <int SPLIT>
int clusters_at_once() {
  static std::atomic<int> known[kMaxDev];  // plus 1
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return 0;
  if (const int n = known[dev].load()) return n - 1;
  auto kern = linear_i8_kernel<1, false, SPLIT, 8>;
  const int smem = 128 * 1024;  // two do not fit an SM
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = SPLIT;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(SPLIT);
  cfg.blockDim = dim3(64 + 32 * 8);
  cfg.dynamicSmemBytes = smem;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (set_smem<1, false, SPLIT, 8>(dev) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess)
    return 0;
  known[dev].store(n + 1);
  return n;
}

template <bool GATED>
cudaError_t run_linear(LinParams p, const int8_t* x, const int8_t* w, int K, cudaStream_t st) {
  const LinPlan pl = plan_linear(p.T, p.NO, K, GATED, device_sm_count(), [](int split) {
    return split == 8 ? clusters_at_once<8>() : clusters_at_once<4>();
  });
  if (pl.few == 16)
    return p.T <= 8 ? launch_few<1, GATED, 16>(p, pl.blocks, x, w, K, st)
                    : launch_few<2, GATED, 16>(p, pl.blocks, x, w, K, st);
  if (pl.few) return launch_few<1, GATED, 8>(p, pl.blocks, x, w, K, st);
  if (pl.blocks == 0) return cudaErrorInvalidValue;
  p.KB = pl.KB;
  p.tn = pl.tn;
  p.nsub = pl.nsub;
  p.nbuf = pl.nbuf;
  p.stages = pl.stages;
  p.MT = pl.MT;
  p.TT = pl.TT;
  p.panel = pl.panel;
  p.cols = pl.cols;
  if (pl.cg == 2) return launch_linear<2, GATED, 1, 16>(p, x, w, K, pl, st);
  if (pl.ew == 16) return launch_linear<1, GATED, 1, 16>(p, x, w, K, pl, st);
  if (pl.split == 1) return launch_linear<1, GATED, 1, 4>(p, x, w, K, pl, st);
  if (pl.split == 2) return launch_linear<1, GATED, 2, 8>(p, x, w, K, pl, st);
  if (pl.split == 4) return launch_linear<1, GATED, 4, 8>(p, x, w, K, pl, st);
  return launch_linear<1, GATED, 8, 8>(p, x, w, K, pl, st);
}

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
  LinParams p{};
  p.xs = x_scale;
  p.ws = w_scale;
  p.T = T;
  p.N = N;
  p.NO = gated ? N / 2 : N;
  p.act = gate_act;
  p.out = reinterpret_cast<__nv_bfloat16*>(out);
  p.out_f32 = out_f32;
  p.err = reinterpret_cast<uint32_t*>(ws);
  const cudaError_t e = gated ? run_linear<true>(p, x, w, K, stream)
                              : run_linear<false>(p, x, w, K, stream);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
