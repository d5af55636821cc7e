// The shared projection with adapters for a handful of tokens, in one launch
// (device part and launcher; ftm_lora.cu chooses it).
//
// Half of a CTA's warps sum its 16 rows of W over all of K, the other half 16
// rows of the adapters' A: the groups of 16 rows of the adapters that
// occur are dealt out to the CTAs of a cluster, which hand v = s (x A^T) to all
// of them through shared memory.  So every CTA has v without a second launch, and
// A is read once per cluster.  A CTA then adds B[a] v of its own outputs, a
// token's own adapter only, in fp32: v is no tensor-core operand here and is not
// rounded.
//
// The products are those of ftm_token.cuh.  (Asking W into L2 first: 5.0 us for
// one token of 2048 to 2048, 4.8 without; all warps at W and then at A: 5.5.)
#pragma once

#include "ftm_token.cuh"

namespace ftm {

constexpr int kTokenHalf = kTokenThreads / 64;           // warps at W, and at A

struct TokenArgs {
  const uint16_t *x, *w, *a_pool, *b_pool;
  const float* scale;
  const int32_t* ids;
  uint16_t* y;
  int64_t ldx, ldy;
  int T, K, M, n, rank;
};

__global__ void __launch_bounds__(kTokenThreads, 2) lora_token_kernel(const TokenArgs p) {
  constexpr int kLanes = kTokenThreads / (kTokenRows * kTokenTile);     // threads of an output at the end
  __shared__ float red[2][kTokenHalf][kTokenTile * kTokenPitch];        // [half][warp][token][row]
  __shared__ __align__(16) float s_v[kTokenTile][128];
  const int lane = threadIdx.x % 32, half = threadIdx.x / 32 / kTokenHalf, warp = threadIdx.x / 32 % kTokenHalf;
  const int g = lane >> 2;
  const int m0 = blockIdx.x * kTokenRows;
  const int nc = static_cast<int>(cluster_nranks());
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  pdl_wait();
  pdl_trigger();

  const uint16_t* const xr[1] = {g < p.T ? p.x + g * p.ldx : nullptr};
  auto dot = [&](const uint16_t* r0, const uint16_t* r1) {
    token_dot<1, false>(r0, r1, xr, p.K, warp, kTokenHalf, red[half][warp], [] {});
  };
  auto sum = [&](int h, int t, int row) {
    float f = 0.f;
#pragma unroll
    for (int w = 0; w < kTokenHalf; ++w) f += red[h][w][t * kTokenPitch + row];
    return f;
  };

  const int id = lane < kTokenTile ? lora_id(p.ids, p.T, p.n, lane) : -1;      // of token `lane`
  if (half == 0) {
    const int r = m0 + g;
    dot(r < p.M ? p.w + static_cast<size_t>(r) * p.K : nullptr,
        r + 8 < p.M ? p.w + static_cast<size_t>(r + 8) * p.K : nullptr);
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  } else {
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");   // every CTA runs: its s_v may be written
    const uint32_t same = __match_any_sync(0xffffffffu, id);
    const uint32_t heads = __ballot_sync(0xffffffffu, id >= 0 && __ffs(same) - 1 == lane);
    const int per = (p.rank + 15) / 16, groups = __popc(heads) * per;
    for (int grp = static_cast<int>(cluster_rank()); grp < groups; grp += nc) {
      const int li = grp / per, n0 = (grp - li * per) * 16;
      const int aid = __shfl_sync(0xffffffffu, id, __fns(heads, 0, li + 1));
      const uint16_t* A = p.a_pool + (static_cast<size_t>(aid) * p.rank + n0) * p.K;
      dot(n0 + g < p.rank ? A + static_cast<size_t>(g) * p.K : nullptr,
          n0 + g + 8 < p.rank ? A + static_cast<size_t>(g + 8) * p.K : nullptr);
      asm volatile("bar.sync 1, 256;" ::: "memory");
      // a warp of the first four takes two tokens
      const int t = warp * 2 + (lane >> 4), row = lane & 15;
      const int mine = __shfl_sync(0xffffffffu, id, t);
      if (t < p.T && mine == aid && n0 + row < p.rank) {
        const float v = (p.scale ? p.scale[aid] : 1.f) * sum(1, t, row);
        const uint32_t at = smem_u32(&s_v[t][n0 + row]);
        for (int c = 0; c < nc; ++c)
          asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(mapa_rank(at, c)), "f"(v) : "memory");
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");              // the sums are read
    }
  }
  // an output's threads ask for their pieces of B ahead of the exchange
  const int o = threadIdx.x / kLanes, sub = threadIdx.x % kLanes;
  const int t = o / kTokenRows, m = m0 + o % kTokenRows, pieces = p.rank / 8;
  const int mine = __shfl_sync(0xffffffffu, id, t);
  const bool low = m < p.M && mine >= 0;
  const uint4* B = reinterpret_cast<const uint4*>(p.b_pool + (static_cast<size_t>(max(mine, 0)) * p.M + m) * p.rank);
  constexpr int kPieces = 128 / 8 / kLanes;
  uint4 b[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i)
    if (low && sub + i * kLanes < pieces) b[i] = __ldg(B + sub + i * kLanes);
  cluster_sync_all();                 // v is complete in every CTA, and no CTA writes to another any more
  float f = 0.f;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int at = sub + i * kLanes;
    if (!low || at >= pieces) break;
    const float4 v0 = *reinterpret_cast<const float4*>(&s_v[t][at * 8]);
    const float4 v1 = *reinterpret_cast<const float4*>(&s_v[t][at * 8 + 4]);
    const float v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
    const uint32_t bw[4] = {b[i].x, b[i].y, b[i].z, b[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f = fmaf(v[2 * j], __uint_as_float(bw[j] << 16), f);
      f = fmaf(v[2 * j + 1], __uint_as_float(bw[j] & 0xffff0000u), f);
    }
  }
#pragma unroll
  for (int d = kLanes / 2; d > 0; d /= 2) f += __shfl_xor_sync(0xffffffffu, f, d);
  if (t < p.T && m < p.M && sub == 0) p.y[t * p.ldy + m] = static_cast<uint16_t>(pack_bf16(sum(0, t, o % kTokenRows) + f, 0.f));
}

// Whether the call runs here, and its cluster's size: the rows of A are one
// pass of the cluster's CTAs, and the outputs one wave of CTAs, or two of a depth
// that costs little more than a launch.  In a replayed graph, here and in the
// two launches of ftm_lora.cu:
//   1 token,  2048 -> 2048, rank 8      4.3   7.4 us
//   1 token,  4096 -> 4096, rank 16     9.6  13.1
//   4 tokens, 4096 -> 4096, rank 16    11.1  13.8
//   8 tokens, 2048 -> 2048, rank 16     6.8   8.2
//   8 tokens, 4096 -> 4096, rank 16    14.2  14.3   (two passes of a cluster of 4: 16.6)
//   2 tokens, 1024 -> 6144, rank 32     8.0   8.4   (two waves)
//   2 tokens, 4096 -> 6144, rank 64    19.2  17.0   (two waves, not taken)
inline bool lora_token_fits(const TokenArgs& p, int& cluster) {
  const int groups = p.T * ((p.rank + 15) / 16);
  if (p.T > kTokenTile || groups > 8) return false;
  cluster = groups <= 4 ? 4 : 8;          // of 8: fewer fit beside one another
  struct Fit { int n[2]; };
  static const Fit fit = [] {
    Fit f = {};
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.blockDim = dim3(kTokenThreads);
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    for (int i = 0; i < 2; ++i) {
      attr.val.clusterDim.x = 4 << i;
      cfg.gridDim = dim3(num_sms() * 2 / (4 << i) * (4 << i));
      if (cudaOccupancyMaxActiveClusters(&f.n[i], lora_token_kernel, &cfg) != cudaSuccess) f.n[i] = 0;
    }
    (void)cudaGetLastError();
    return f;
  }();
  const int ctas = (p.M + kTokenRows - 1) / kTokenRows, wave = cluster * fit.n[cluster == 8];
  return ctas <= wave || (ctas <= 2 * wave && p.K <= 1024);
}

inline cudaError_t launch_lora_token(const TokenArgs& p, int cluster, cudaStream_t st) {
  const int span = kTokenRows * cluster;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((p.M + span - 1) / span * cluster);
  cfg.blockDim = dim3(kTokenThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return count_launch(cudaLaunchKernelEx(&cfg, lora_token_kernel, p));
}

}  // namespace ftm
