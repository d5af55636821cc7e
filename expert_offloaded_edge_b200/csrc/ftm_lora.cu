// The shared projection with low-rank adapters of many requests:
//   y[t] = x[t] W^T + s[a] (x[t] A[a]^T) B[a]^T
// in two launches, the second started early (programmatic dependent launch):
//   1. lora_shrink_kernel: v[t] = s[a] (x[t] A[a]^T), rounded to bf16 (the
//      operand type of the second product; a relative 2^-9 of the adapter's
//      part of y alone);
//   2. the projection over K = d_in and the adapters' K range (ftm_lora.cuh):
//      lora_proj_kernel below for few tokens (bound by the bytes of W: weights
//      on the MMA's M side, split over a cluster along K), the CTA-pair engine
//      of ftm_dense.cuh for many.
#include "ftm_dense.cuh"

namespace ftm {

// ---------------------------------------------------------------------------
// v = s (x A^T).  A block takes 16 MI tokens and one share of K (a cluster of
// blocks splits K) and walks over the adapters that occur among its tokens:
// tensor-core products of all its rows with 32 rows of A[a] at a time, kept for
// the tokens whose adapter it is.  blockIdx.y shares out the adapters of a tile,
// since a decode batch may bring 16 of them to 16 tokens.  mma.sync on purpose:
// the product reads A once per tile and does 2 rank flops per value of x, far
// below the tensor rate, and takes any mixture of adapters without a layout.
// Each thread loads 16 consecutive bytes of a row per operand: the depths of
// one 32-deep step are dealt to the two MMAs in the same order on both sides.
// ---------------------------------------------------------------------------
constexpr int kShrinkWarps = 8;
constexpr int kShrinkCols = 32;                // rows of A (columns of v) per pass

__device__ __forceinline__ void mma_bf16_16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int MI, int KS>
__global__ void __launch_bounds__(kShrinkWarps * 32)
    lora_shrink_kernel(const uint16_t* __restrict__ x, int64_t ldx, int T, int K, const uint16_t* __restrict__ a_pool,
                       const float* __restrict__ scale, const int32_t* __restrict__ ids, int n, int rank, int rp,
                       uint16_t* __restrict__ v) {
  constexpr int MT = 16 * MI;
  constexpr int kOut = MT * kShrinkCols;
  __shared__ float red[kShrinkWarps][kOut];
  __shared__ float part[KS > 1 ? 2 * KS * kOut : 1];   // rank 0: the ranks' sums, by pass parity
  __shared__ int32_t s_id[MT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, tq = lane & 3;
  const int kr = KS > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int m0 = static_cast<int>(blockIdx.x / KS) * MT;
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x < 32) {
    const int id = lane < MT ? lora_id(ids, T, n, m0 + lane) : -1;
    if (lane < MT) s_id[lane] = id;
  }
  __syncthreads();
  if (KS > 1) cluster_sync_all();       // every rank runs before the first remote store
  // distinct adapters: bit i of `heads` where token i is the first of its adapter
  const int my = lane < MT ? s_id[lane] : -1;
  uint32_t heads = __ballot_sync(0xffffffffu, (__ffs(__match_any_sync(0xffffffffu, my)) - 1) == lane && my >= 0);
  const int steps = (K + 31) / 32;
  const int c_lo = steps * kr / KS, c_hi = steps * (kr + 1) / KS;
  int pass = 0;
  for (int li = 0; heads; ++li) {
    const int head = __ffs(heads) - 1;
    heads &= heads - 1;
    if (li % static_cast<int>(gridDim.y) != static_cast<int>(blockIdx.y)) continue;
    const int id = s_id[head];
    const uint16_t* A = a_pool + static_cast<size_t>(id) * rank * K;
    for (int n0 = 0; n0 < rp; n0 += kShrinkCols, ++pass) {
      float acc[MI][4][4] = {};
#pragma unroll 4
      for (int c = c_lo + warp; c < c_hi; c += kShrinkWarps) {
        const int k = c * 32 + tq * 8;
        uint4 xv[MI][2], av[4];
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int t = m0 + i * 16 + h * 8 + g;
            xv[i][h] = t < T && k < K ? __ldg(reinterpret_cast<const uint4*>(x + t * ldx + k)) : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = n0 + j * 8 + g;
          av[j] = r < rank && k < K ? __ldg(reinterpret_cast<const uint4*>(A + static_cast<size_t>(r) * K + k))
                                    : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            mma_bf16_16816(acc[i][j], xv[i][0].x, xv[i][1].x, xv[i][0].y, xv[i][1].y, av[j].x, av[j].y);
            mma_bf16_16816(acc[i][j], xv[i][0].z, xv[i][1].z, xv[i][0].w, xv[i][1].w, av[j].z, av[j].w);
          }
      }
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            *reinterpret_cast<float2*>(&red[warp][(i * 16 + h * 8 + g) * kShrinkCols + j * 8 + 2 * tq]) =
                make_float2(acc[i][j][2 * h], acc[i][j][2 * h + 1]);
      __syncthreads();
      float* mine = part + (pass & 1) * KS * kOut;
      float sum[kOut / 256];
#pragma unroll
      for (int o = 0; o < kOut / 256; ++o) {
        const int at = o * 256 + threadIdx.x;
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kShrinkWarps; ++w) s += red[w][at];
        sum[o] = s;
        if (KS > 1)
          asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(mapa_rank(smem_u32(mine + kr * kOut + at), 0)), "f"(s)
                       : "memory");
      }
      if (KS > 1) cluster_sync_all();
      else __syncthreads();             // red is free again
      if (kr == 0) {
        const float sc = scale ? scale[id] : 1.f;
#pragma unroll
        for (int o = 0; o < kOut / 256; ++o) {
          const int at = o * 256 + threadIdx.x;
          const int i = at / kShrinkCols, r = n0 + at % kShrinkCols;
          float s = sum[o];
          if (KS > 1) {
            s = 0.f;
#pragma unroll
            for (int p = 0; p < KS; ++p) s += mine[p * kOut + at];
          }
          if (s_id[i] == id && r < rp) {
            // columns that pad the rank to 16 are zero whatever the scale
            const __nv_bfloat16 b = __float2bfloat16_rn(r < rank ? sc * s : 0.f);
            v[static_cast<size_t>(m0 + i) * rp + r] = *reinterpret_cast<const uint16_t*>(&b);
          }
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// The projection for few tokens.  One cluster of ks CTAs per (128 outputs, BN
// tokens) tile, each CTA a share of K and of the adapters' slices; the partial
// sums meet in shared memory (CTA s sums the token columns it owns in rank
// order, so the result does not depend on timing).  W is read once per token
// tile; its loads are issued before the shrink's results are waited for.
// ---------------------------------------------------------------------------
template <int BN>
struct ProjShape {
  static constexpr uint32_t kBBytes = ((BN * 128 + 1023) / 1024) * 1024;
  static constexpr uint32_t kStage = kATileBytes + kBBytes;
  static constexpr int kStages = BN <= 32 ? 7 : BN == 64 ? 5 : 3;
  static constexpr uint32_t kBuf = 128 * 32 + BN * 32;               // a slice of B[a] and one of v
  static constexpr uint32_t kTmemCols = BN < 32 ? 32 : BN;
  static size_t red_bytes(int ks) { return ks > 1 ? static_cast<size_t>(ks) * ((BN + ks - 1) / ks) * 512 : 0; }
  static size_t smem(int ks) { return 1024 + static_cast<size_t>(kStages) * kStage + kLoraRing * kBuf + red_bytes(ks); }
};

template <int BN>
__global__ void __launch_bounds__(192, 1)
    lora_proj_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                     const __grid_constant__ LoraArgs a, int K, uint16_t* __restrict__ y, int64_t ldy) {
  using S = ProjShape<BN>;
  constexpr uint32_t kIdesc = idesc_bf16_f32(128, BN);
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[S::kStages], empty_bar[S::kStages], tfull_bar, count_bar;
  __shared__ uint32_t tmem_holder, slices;
  __shared__ LoraShared<true> ls;

  const uint32_t smem_base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (smem_base - smem_u32(smem_raw));
  uint8_t* ext = smem + static_cast<size_t>(S::kStages) * S::kStage;
  float* red = reinterpret_cast<float*>(ext + kLoraRing * S::kBuf);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int ks = static_cast<int>(cluster_nranks()), kr = static_cast<int>(cluster_rank());
  const int n0 = blockIdx.y * BN, w0 = blockIdx.z * 128;
  const int KB = (K + 63) / 64;
  const int kb0 = kr * KB / ks, kb1 = (kr + 1) * KB / ks;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) { mbar_init(&full_bar[s], 1); mbar_init(&empty_bar[s], 1); }
    mbar_init(&tfull_bar, 1);
    mbar_init(&count_bar, 1);
    ls.init(1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_holder, S::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  if (ks > 1) cluster_sync_all();       // every rank's shared memory may be written from here on
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = tmem_holder;

  if (warp == 0) {
    // The launch before this one is always the shrink, which started this one
    // after its own wait for everything earlier: x and W are final.
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(&empty_bar[stage], phase ^ 1u)) break;
        mbar_arrive_expect_tx(&full_bar[stage], kATileBytes + BN * 128);
        uint8_t* sa = smem + static_cast<size_t>(stage) * S::kStage;
        tma_load_2d(sa, &tmW, &full_bar[stage], kb * 64, w0);
        tma_load_2d(sa + kATileBytes, &tmX, &full_bar[stage], kb * 64, n0);
        if (++stage == S::kStages) { stage = 0; phase ^= 1u; }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(&full_bar[stage], phase)) { ok = false; break; }
        tc_fence_after();
        const uint32_t sa = smem_u32(smem + static_cast<size_t>(stage) * S::kStage);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_f16(tmem_base, smem_desc_sw128(sa + kk * 32), smem_desc_sw128(sa + kATileBytes + kk * 32), kIdesc,
                   kb != kb0 || kk != 0 ? 1u : 0u);
        umma_commit(&empty_bar[stage]);
        if (++stage == S::kStages) { stage = 0; phase ^= 1u; }
      }
      ok = ok && mbar_wait(&count_bar, 0);
      const uint32_t cnt = ok ? slices : 0;
      for (uint32_t c = 0; c < cnt; ++c) {
        const uint32_t slot = c % kLoraRing;
        if (!mbar_wait_cl(&ls.full[slot], (c / kLoraRing) & 1u)) { ok = false; break; }
        tc_fence_after();
        const uint32_t sb = smem_u32(ext + slot * S::kBuf);
        umma_f16(tmem_base, smem_desc_k32(sb), smem_desc_k32(sb + 128 * 32), kIdesc, 1u);
        umma_commit(&ls.empty[slot]);
      }
      if (ok) umma_commit(&tfull_bar);
    }
    __syncwarp();
  } else {
    // the adapters' slices of this rank
    const int e = threadIdx.x - 64;
    const int i0 = e < BN ? lora_id(a.ids, a.T, a.n, n0 + e) : -1;
    const int nl = lora_list<128>(ls, e, i0, -1);
    const int total = nl * (a.rp >> 4);
    if (e == 0) {
      slices = total > kr ? (total - kr - 1) / ks + 1 : 0;
      mbar_arrive(&count_bar);
    }
    pdl_wait();
    pdl_trigger();
    LoraRing ring;
    auto send = [&](uint32_t slot, bool, bool bad) {
      if (bad)      // every rank's epilogue looks at its own flag
        for (int r = 0; r < ks; ++r)
          asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_rank(smem_u32(&ls.poison[0]), r)), "r"(kLoraPoison)
                       : "memory");
      mbar_arrive(&ls.full[slot]);
    };
    bool ok = lora_feed<BN, 128>(a, ls, ring, ext, 128 * 32, 0, S::kBuf, e, nl, kr, ks, n0 + e, i0, w0, send);
    // the partial sums: lane = output, TMEM column = token
    const int q = warp % 4, er = q * 32 + lane;
    ok = ok && mbar_wait(&tfull_bar, 0);
    if (__all_sync(0xffffffffu, ok)) {
      tc_fence_after();
      const uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
      const int ncmax = (BN + ks - 1) / ks;
#pragma unroll 1
      for (int c0 = 0; c0 < BN && n0 + c0 < a.T; c0 += 16) {
        float f[16];
        tmem_ld16(tb + c0, f);
        tmem_ld_wait();
        if (ks == 1) {
          const bool poison = *reinterpret_cast<volatile uint32_t*>(&ls.poison[0]) != 0;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int t = n0 + c0 + j;
            if (t < a.T && w0 + er < a.d_out) {
              if (poison) f[j] += lora_nonfinite_term(a, t, w0 + er);
              const __nv_bfloat16 b = __float2bfloat16_rn(f[j]);
              y[t * ldy + w0 + er] = *reinterpret_cast<const uint16_t*>(&b);
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int c = c0 + j, s = ((c + 1) * ks - 1) / BN;       // the rank that owns column c
            float* at = red + (kr * ncmax + c - s * BN / ks) * 128 + er;
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(mapa_rank(smem_u32(at), s)), "f"(f[j]) : "memory");
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncwarp();
  if (ks > 1) cluster_sync_all();       // all partial sums and flags are in place
  else __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, S::kTmemCols);
  if (ks > 1 && warp >= 2) {
    const int er = (warp % 4) * 32 + lane;
    const int ncmax = (BN + ks - 1) / ks;
    const int lo = kr * BN / ks, hi = (kr + 1) * BN / ks;
    const bool poison = ls.poison[0] != 0;
    for (int c = lo; c < hi && n0 + c < a.T; ++c) {
      float s = 0.f;
      for (int r = 0; r < ks; ++r) s += red[(r * ncmax + c - lo) * 128 + er];
      if (w0 + er < a.d_out) {
        if (poison) s += lora_nonfinite_term(a, n0 + c, w0 + er);
        const __nv_bfloat16 b = __float2bfloat16_rn(s);
        y[(n0 + c) * ldy + w0 + er] = *reinterpret_cast<const uint16_t*>(&b);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
template <int MI, int KS>
static cudaError_t launch_shrink(const LoraCall& c, int rp, int split, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(KS * ((c.T + 16 * MI - 1) / (16 * MI)), split);
  cfg.blockDim = dim3(kShrinkWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = KS;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return count_launch(cudaLaunchKernelEx(&cfg, lora_shrink_kernel<MI, KS>, c.x, c.ldx, c.T, c.d_in, c.a, c.scale, c.ids,
                                         c.n, c.rank, rp, c.v));
}

template <int BN>
static cudaError_t launch_proj(const LoraCall& c, const CUtensorMap& mW, const CUtensorMap& mX, const LoraArgs& la,
                               cudaStream_t st) {
  using S = ProjShape<BN>;
  const int KB = (c.d_in + 63) / 64;
  const int mt = (c.d_out + 127) / 128, nt = (c.T + BN - 1) / BN;
  int ks = num_sms() / (mt * nt);
  ks = ks < 1 ? 1 : ks > 8 ? 8 : ks;
  if (ks > KB) ks = KB;
  auto kern = lora_proj_kernel<BN>;
  const size_t smem = S::smem(ks);
  cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ks, nt, mt);
  cfg.blockDim = dim3(192);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return count_launch(cudaLaunchKernelEx(&cfg, kern, mW, mX, la, c.d_in, c.y, c.ldy));
}

// Returns a message on failure, nullptr on success.
const char* launch_lora(const LoraCall& c, cudaStream_t st, cudaError_t* cerr) {
  const int rp = (c.rank + 15) / 16 * 16;
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return "cuTensorMapEncodeTiled not found";
  // v first
  const int tiles16 = (c.T + 15) / 16;
  if (c.T <= 512) {
    int split = 600 / (tiles16 * 4);
    split = split < 1 ? 1 : split > 16 ? 16 : split;
    *cerr = launch_shrink<1, 4>(c, rp, split, st);
  } else {
    const int tiles = (c.T + 31) / 32;
    int split = 600 / tiles;
    split = split < 1 ? 1 : split > 16 ? 16 : split;
    *cerr = launch_shrink<2, 1>(c, rp, split, st);
  }
  if (*cerr != cudaSuccess) return "adapter shrink launch failed";

  const int BNp = 256;     // the pair engine's column tile
  const long pair_tiles = static_cast<long>((c.T + 255) / 256) * ((c.d_out + BNp - 1) / BNp);
  const bool pairs = pair_tiles >= num_sms() / 4;
  const uint32_t b_rows = pairs ? BNp / 2 : 128;
  LoraArgs la;
  {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(c.rank), static_cast<cuuint64_t>(c.d_out), static_cast<cuuint64_t>(c.n)};
    const cuuint64_t strides[2] = {2ull * c.rank, 2ull * c.rank * c.d_out};
    const cuuint32_t box[3] = {16, b_rows, 1}, es[3] = {1, 1, 1};
    if (enc(&la.b, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(c.b), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_32B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return "cuTensorMapEncodeTiled of the adapters failed";
  }
  la.ids = c.ids;
  la.v = c.v;
  la.b_pool = c.b;
  la.T = c.T;
  la.n = c.n;
  la.rank = c.rank;
  la.rp = rp;
  la.d_out = c.d_out;

  if (pairs) {
    DenseArgs g = {};
    g.n = 1;
    DenseProblem& P = g.p[0];
    dense_tiles(P, c.T, c.d_out, c.d_in, BNp);
    if (!dense_operand_map(&P.a, c.x, false, c.T, c.d_in, 2ull * c.ldx, 128) ||
        !dense_operand_map(&P.b, c.w, false, c.d_out, c.d_in, 2ull * c.d_in, BNp / 2) ||
        !dense_store_map(&P.c0, c.y, c.d_out, c.T, 2ull * c.ldy))
      return "cuTensorMapEncodeTiled failed";
    g.lora = la;
    *cerr = launch_dense<kEpiStore, 256, true>(g, st);
    return *cerr == cudaSuccess ? nullptr : "projection launch failed";
  }
  const int bn = c.T <= 16 ? 16 : c.T <= 32 ? 32 : c.T <= 64 ? 64 : 128;
  CUtensorMap mW, mX;
  if (!dense_operand_map(&mW, c.w, false, c.d_out, c.d_in, 2ull * c.d_in, 128) ||
      !dense_operand_map(&mX, c.x, false, c.T, c.d_in, 2ull * c.ldx, bn))
    return "cuTensorMapEncodeTiled failed";
  switch (bn) {
    case 16: *cerr = launch_proj<16>(c, mW, mX, la, st); break;
    case 32: *cerr = launch_proj<32>(c, mW, mX, la, st); break;
    case 64: *cerr = launch_proj<64>(c, mW, mX, la, st); break;
    default: *cerr = launch_proj<128>(c, mW, mX, la, st); break;
  }
  return *cerr == cudaSuccess ? nullptr : "projection launch failed";
}

}  // namespace ftm
