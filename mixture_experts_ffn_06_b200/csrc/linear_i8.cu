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
// Two forms, both with one TMA warp, one MMA warp and four epilogue warps:
//   few tokens  (bound by streaming w): a tile per cluster of up to 8 CTAs that
//               split K; each parks its partial sums in shared memory and adds
//               up a slice of the columns over all CTAs' (integers: the order
//               of the sum does not matter);
//   many tokens (bound by the tensor cores and by L2 -> shared memory): CTA
//               pairs (M = 256) walk the tiles, two accumulators in TMEM so that
//               a tile's epilogue runs beside the next one's MMAs.
// Every mbarrier wait is bounded (tc_ptx.cuh); after a timeout the block
// records MOE_ERR_TIMEOUT, waits for its own copies and MMAs and frees TMEM.
#include <algorithm>
#include <atomic>
#include <mutex>

#include "tc_ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 192;
constexpr int kABytes = 128 * 128;   // 128 weight rows x 128 bytes of K
constexpr int kMaxStages = 12;
constexpr uint64_t kTimeoutNs = 1000000000ull;  // 1 s per wait
constexpr int kSmemMax = 227 * 1024;
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
  int MT, TT;   // weight tiles (of CG x 128 rows) and token tiles (nsub x tn)
  int panel;    // token tiles per panel of the tile order
  int split;    // CTAs that share K
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

// Both activations as g sigma(.): 0.5 (1 + tanh v) = sigma(2v) does not cancel
// where v is large and negative.
__device__ __forceinline__ float lin_act(int act, float g) {
  const float e = act == MOE_ACT_SILU
                      ? -g
                      : -1.5957691216057308f * fmaf(0.044715f * g, g * g, g);  // -2 v
  return __fdividef(g, 1.0f + __expf(e));
}

struct LinTile {
  int mt;
  int64_t t0;  // first token
};

// Tile u: panels of ``panel`` token tiles, then the weight tile, then the token
// tile inside the panel, so that the tiles running at once share weight tiles
// and the panel's tokens stay in L2 while the weights pass by once per panel.
__device__ __forceinline__ LinTile lin_tile(int64_t u, const LinParams& p) {
  const int64_t per = (int64_t)p.panel * p.MT;
  const int64_t pn = u / per, in = u - pn * per;
  const int64_t left = p.TT - pn * p.panel;
  const int64_t pw = left < p.panel ? left : p.panel;
  const int64_t mt = in / pw;
  return LinTile{(int)mt, (pn * p.panel + in - mt * pw) * p.nsub * p.tn};
}

// What the epilogue needs of a lane: its channel and scales.
template <bool GATED>
struct LaneOut {
  int n;        // output channel
  bool ok;
  float s0, s1;  // plain: scales of channels n, n + 1 of the even lane; gated: gate, up
  int lane;

  __device__ __forceinline__ void init(const LinParams& p, int row, int ln) {
    lane = ln;
    if (GATED) {
      n = (row >> 5) * 16 + (ln & 15);
      ok = n < p.NO;
      s0 = ok ? __ldg(p.ws + n) : 0.f;
      s1 = ok ? __ldg(p.ws + p.NO + n) : 0.f;
    } else {
      n = row;
      ok = n < p.N;
      const float own = ok ? __ldg(p.ws + n) : 0.f;
      const float other = __shfl_xor_sync(0xffffffffu, own, 1);
      s0 = (ln & 1) ? other : own;
      s1 = (ln & 1) ? own : other;
    }
  }

  // Two token columns c and c + 1 of this lane's row; t: token of column c; the
  // token scales sx (of c) and sy (of c + 1).
  __device__ __forceinline__ void store2(const LinParams& p, int64_t t, int32_t a, int32_t b,
                                         float sx, float sy) const {
    // partners swap one value, so that each lane holds both rows of one token
    const bool up = GATED ? lane >= 16 : (lane & 1) != 0;
    const int32_t got = __shfl_xor_sync(0xffffffffu, up ? a : b, GATED ? 16 : 1);
    const int64_t tok = t + (up ? 1 : 0);
    const float s = up ? sy : sx;
    const float v0 = __fmul_rn((float)(up ? got : a), __fmul_rn(s, s0));
    const float v1 = __fmul_rn((float)(up ? b : got), __fmul_rn(s, s1));
    if (tok >= p.T) return;
    if (GATED) {
      if (!ok) return;
      const float v = lin_act(p.act, v0) * v1;
      const int64_t at = tok * p.NO + n;
      if (p.out) p.out[at] = __float2bfloat16_rn(v);
      if (p.out_f32) p.out_f32[at] = v;
    } else {
      const int m = n & ~1;  // channels m, m + 1
      const int64_t at = tok * p.NO + m;
      if (m + 1 < p.N && (p.NO & 1) == 0) {
        if (p.out) *reinterpret_cast<__nv_bfloat162*>(p.out + at) = __floats2bfloat162_rn(v0, v1);
        if (p.out_f32) *reinterpret_cast<float2*>(p.out_f32 + at) = make_float2(v0, v1);
      } else {
        if (m < p.N) {
          if (p.out) p.out[at] = __float2bfloat16_rn(v0);
          if (p.out_f32) p.out_f32[at] = v0;
        }
        if (m + 1 < p.N) {
          if (p.out) p.out[at + 1] = __float2bfloat16_rn(v1);
          if (p.out_f32) p.out_f32[at + 1] = v1;
        }
      }
    }
  }
};

template <int CG, bool GATED, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
linear_i8_kernel(const __grid_constant__ CUtensorMap tmW,
                 const __grid_constant__ CUtensorMap tmX, const LinParams p) {
  static_assert(!(SPLIT && CG == 2), "K is split over single CTAs");
  extern __shared__ uint8_t smem_raw[];
  __shared__ LinCtl ctl_s;
  LinCtl* ctl = &ctl_s;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t sub_bytes = (uint32_t)p.tn / CG * 128u;
  const uint32_t b_bytes = sub_bytes * p.nsub;
  const uint32_t sA = base;
  const uint32_t sB = base + p.stages * kABytes;
  volatile int32_t* abort_flag = &ctl->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = (CG == 2 || SPLIT) ? cluster_ctarank() : 0u;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(smem_u32(&ctl->full[s]), 1);
      mbar_init(smem_u32(&ctl->empty[s]), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&ctl->tmem_full[a]), 1);
      mbar_init(smem_u32(&ctl->tmem_empty[a]), 4 * CG);  // one per epilogue warp
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
  pdl_trigger();
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();  // the peer's barriers are initialised
  tc_fence_after();
  const uint32_t tmem_base = ctl->tmem_base;

  // tiles: one per cluster with SPLIT (grid = tiles x split), else a walk
  const int64_t unit0 = SPLIT ? (int64_t)(blockIdx.x / p.split)
                        : CG == 2 ? (int64_t)cluster_id_x() : (int64_t)blockIdx.x;
  const int64_t total = (int64_t)p.MT * p.TT;
  const int64_t step = SPLIT ? total
                       : CG == 2 ? (int64_t)nclusters_x() : (int64_t)gridDim.x;
  const int kb0 = SPLIT ? (int)(rank * p.KB / p.split) : 0;
  const int kb1 = SPLIT ? (int)((rank + 1) * p.KB / p.split) : p.KB;

  if (warp == 0) {
    // ------------------------------------------------------ TMA producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, filled = 0, last = 0;  // bit s: stage s filled, its parity
      bool ok = true;
      for (int64_t u = unit0; ok && u < total; u += step) {
        const LinTile tl = lin_tile(u, p);
        const int mrow = (tl.mt * CG + (int)(CG == 2 ? rank : 0)) * (GATED ? 64 : 128);
        const int64_t tr = tl.t0 + (CG == 2 ? (int64_t)rank * (p.tn / 2) : 0);
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait(smem_u32(&ctl->empty[stage]), phase ^ 1u, abort_flag, kTimeoutNs,
                         p.err)) {
            ok = false;
            break;
          }
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
          filled |= 1u << stage;
          last = (last & ~(1u << stage)) | (phase << stage);
          if (++stage == p.stages) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok && (CG == 1 || rank == 0)) {
        // let the copies already issued land before the block exits
        int32_t none = 0;
        volatile int32_t* never = &none;
        for (int s = 0; s < p.stages; ++s)
          if ((filled >> s) & 1u)
            mbar_wait(smem_u32(&ctl->full[s]), (last >> s) & 1u, never, kTimeoutNs, p.err);
      }
    }
  } else if (warp == 1) {
    // --------------------------------------------------------- MMA issuer
    if (lane == 0 && (CG == 1 || rank == 0)) {
      const uint32_t idesc = idesc_i8_s32(128 * CG, p.tn);
      int stage = 0, buf = 0;
      uint32_t phase = 0, buf_phase = 0;
      bool ok = true;
      for (int64_t u = unit0; ok && u < total; u += step) {
        const uint32_t eb = smem_u32(&ctl->tmem_empty[buf]);
        ok = CG == 2 ? mbar_wait_cluster(eb, buf_phase ^ 1u, abort_flag, kTimeoutNs, p.err)
                     : mbar_wait(eb, buf_phase ^ 1u, abort_flag, kTimeoutNs, p.err);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem_base + buf * 256;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait(smem_u32(&ctl->full[stage]), phase, abort_flag, kTimeoutNs, p.err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t ad = sw128_kmajor_desc(sA + stage * kABytes);
          for (int s = 0; s < p.nsub; ++s) {
            const uint64_t bd = sw128_kmajor_desc(sB + stage * b_bytes + s * sub_bytes);
            // four MMAs of 32 bytes of K each
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_i8<CG>(d + s * 256, ad + 2u * kk, bd + 2u * kk, idesc,
                          (kb != kb0 || kk != 0) ? 1u : 0u);
          }
          if (CG == 2)
            umma_commit_pair_mc(smem_u32(&ctl->empty[stage]), 0x3);
          else
            umma_commit(smem_u32(&ctl->empty[stage]));
          if (++stage == p.stages) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        if (CG == 2)
          umma_commit_pair_mc(smem_u32(&ctl->tmem_full[buf]), 0x3);
        else
          umma_commit(smem_u32(&ctl->tmem_full[buf]));
        if (++buf == p.nbuf) { buf = 0; buf_phase ^= 1u; }
      }
      if (!ok || *abort_flag) {
        // wait for the MMAs already issued before TMEM is released
        int32_t none = 0;
        volatile int32_t* never = &none;
        if (CG == 2)
          umma_commit_pair(smem_u32(&ctl->drain));
        else
          umma_commit(smem_u32(&ctl->drain));
        mbar_wait(smem_u32(&ctl->drain), 0, never, kTimeoutNs, p.err);
      }
    }
  } else {
    // ----------------------------------------------------------- epilogue
    // Warp w reads TMEM lanes [32 (w % 4), 32 (w % 4) + 32).
    const int q = warp & 3;
    const uint32_t lanes = (uint32_t)(q * 32) << 16;
    const uint32_t empty0 = CG == 2 ? mapa_shared(smem_u32(&ctl->tmem_empty[0]), 0) : 0u;
    const uint32_t empty1 = CG == 2 ? mapa_shared(smem_u32(&ctl->tmem_empty[1]), 0) : 0u;
    int buf = 0;
    uint32_t buf_phase = 0;
    for (int64_t u = unit0; u < total; u += step) {
      const LinTile tl = lin_tile(u, p);
      LaneOut<GATED> lo;
      lo.init(p, (tl.mt * CG + (int)(CG == 2 ? rank : 0)) * 128 + q * 32 + lane, lane);
      const bool got = mbar_wait(smem_u32(&ctl->tmem_full[buf]), buf_phase, abort_flag,
                                 kTimeoutNs, p.err);
      // warp-uniform decision; also reconverges the warp for tcgen05.ld
      if (!__all_sync(0xffffffffu, got)) break;
      tc_fence_after();
      const uint32_t tb = tmem_base + lanes + buf * 256;
      if constexpr (SPLIT) {
        // partial sums [column][128 rows] over the ring, which is idle now
        int32_t* part = reinterpret_cast<int32_t*>(gbase);
        for (int c = 0; c < p.tn; c += 32) {
          uint32_t v[32];
          tmem_ld32(tb + c, v);
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (c + j < p.tn) part[(c + j) * 128 + q * 32 + lane] = (int32_t)v[j];
        }
        break;  // one tile per cluster; finished below
      } else {
      for (int s = 0; s < p.nsub; ++s) {
        const int64_t ts = tl.t0 + (int64_t)s * p.tn;
        for (int c = 0; c < p.tn; c += 32) {
          if (ts + c >= p.T) break;
          uint32_t v[32];
          tmem_ld32(tb + s * 256 + c, v);
          const float sx = ts + c + lane < p.T ? __ldg(p.xs + ts + c + lane) : 0.f;
#pragma unroll
          for (int j = 0; j < 32; j += 2)
            if (c + j < p.tn)
              lo.store2(p, ts + c + j, (int32_t)v[j], (int32_t)v[j + 1],
                        __shfl_sync(0xffffffffu, sx, j), __shfl_sync(0xffffffffu, sx, j + 1));
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
  }

  if (SPLIT) {
    __syncwarp();
    cluster_sync();  // every CTA's partial sums are in its shared memory
    if (warp >= 2 && !*abort_flag) {
      // columns c = 2 rank, 2 rank + 1, then 2 split further on
      const int q = warp & 3, row = q * 32 + lane;
      const LinTile tl = lin_tile(unit0, p);
      LaneOut<GATED> lo;
      lo.init(p, tl.mt * 128 + row, lane);
      const uint32_t mine = smem_u32(gbase) + row * 4;
      for (int c = 2 * (int)rank; c < p.tn && tl.t0 + c < p.T; c += 2 * p.split) {
        int32_t a = 0, b = 0;
        for (int r = 0; r < p.split; ++r) {
          const uint32_t src = mapa_shared(mine + c * 512, r);
          int32_t u, v;
          asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(u) : "r"(src));
          asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(src + 512));
          a += u;
          b += v;
        }
        const float sx = __ldg(p.xs + tl.t0 + c);
        const float sy = tl.t0 + c + 1 < p.T ? __ldg(p.xs + tl.t0 + c + 1) : 0.f;
        lo.store2(p, tl.t0 + c, a, b, sx, sy);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (CG == 2 || SPLIT) cluster_sync();  // no peer still uses this CTA's memory or TMEM
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    if (CG == 2)
      tmem_dealloc_pair(tmem_base, p.cols);
    else
      tmem_dealloc(tmem_base, p.cols);
  }
}

// ------------------------------------------------------------------- host

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion,
                                  CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(ptr);
  });
  return fn;
}

// Map of the gated weight as [2, I, K] bytes: box {128, 16, 2}, 16 gate rows and
// then the matching 16 up rows (rows past I read as zero).
cudaError_t make_gated_map(CUtensorMap* m, const void* ptr, uint64_t K, uint64_t I) {
  EncodeTiledFn enc = encode_fn();
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

template <int CG, bool GATED, bool SPLIT>
cudaError_t launch_linear(LinParams& p, const int8_t* x, const int8_t* w, int K, int clusters,
                          cudaStream_t st) {
  auto kern = linear_i8_kernel<CG, GATED, SPLIT>;
  CUtensorMap mw, mx;
  cudaError_t e = GATED ? make_gated_map(&mw, w, K, p.NO) : make_tma_map_e4m3(&mw, w, K, p.N, 128);
  if (e == cudaSuccess) e = make_tma_map_e4m3(&mx, x, K, p.T, p.tn / CG);
  if (e != cudaSuccess) return e;
  // the shared-memory opt-in is a per-device attribute
  static std::atomic<bool> ready[kMaxDev];
  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDev || !ready[dev].load()) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSmemMax - (int)sizeof(LinCtl));
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < kMaxDev) ready[dev].store(true);
  }
  const int per = SPLIT ? p.split : CG;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(clusters * per));
  cfg.blockDim = dim3(kThreads);
  const size_t ring = (size_t)p.stages * (kABytes + (size_t)p.tn / CG * 128 * p.nsub);
  cfg.dynamicSmemBytes = 1024 + std::max(ring, SPLIT ? (size_t)p.tn * 512 : (size_t)0);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)per;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = per > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, mw, mx, (const LinParams)p);
}

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

template <bool GATED>
cudaError_t run_linear(LinParams p, const int8_t* x, const int8_t* w, int K, cudaStream_t st) {
  const int sms = device_sm_count();
  const int rows = GATED ? 64 : 128;  // output channels of 128 weight rows
  p.KB = ceil_div(K, 128);
  p.nsub = 1;
  if (p.T <= 128) {
    p.tn = 16 * ceil_div(p.T, 16);
    p.nbuf = 1;
    p.TT = 1;
    p.panel = 1;
    p.MT = ceil_div(p.NO, rows);
    p.cols = p.tn <= 32 ? 32 : p.tn <= 64 ? 64 : 128;
    int split = 1;
    while (split < 8 && p.MT * split < sms && 2 * split <= p.KB) split *= 2;
    p.split = split;
    const int stage = kABytes + p.tn * 128;
    p.stages = std::min({kMaxStages, (kSmemMax - 2048) / stage, ceil_div(p.KB, split)});
    return launch_linear<1, GATED, true>(p, x, w, K, p.MT, st);
  }
  p.split = 1;
  p.TT = ceil_div(p.T, 256);
  p.tn = 32 * ceil_div(ceil_div(p.T, p.TT), 32);
  p.nbuf = 2;
  p.panel = 16;
  p.MT = ceil_div(p.NO, 2 * rows);
  p.cols = 512;
  const int stage = kABytes + p.tn / 2 * 128;
  p.stages = std::min(kMaxStages, (kSmemMax - 2048) / stage);
  const int64_t tiles = (int64_t)p.MT * p.TT;
  return launch_linear<2, GATED, false>(p, x, w, K, (int)std::min<int64_t>(sms / 2, tiles), st);
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
