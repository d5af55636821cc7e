// The shared projection with low-rank adapters of many requests:
//   y[t] = x[t] W^T + s[a] (x[t] A[a]^T) B[a]^T
// a handful of tokens in one launch (ftm_lora_token.cuh), others in two, the
// second started early (programmatic dependent launch):
//   1. lora_shrink_kernel: v[t] = s[a] (x[t] A[a]^T), rounded to bf16 (the
//      operand type of the second product; at most 2^-8 of the adapter's
//      part of y alone; one launch keeps it in fp32);
//   2. the projection over K = d_in and the adapters' K range (ftm_lora.cuh):
//      ftm_proj.cuh for few tokens (bound by the bytes of W), the CTA-pair
//      engine of ftm_dense.cuh for many.
#include "ftm_lora_token.cuh"
#include "ftm_proj.cuh"

namespace ftm {

// ---------------------------------------------------------------------------
// v = s (x A^T).  A block takes MT tokens and one share of K (a cluster of
// blocks splits K) and walks over the adapters that occur among its tokens:
// tensor-core products of all its rows with the rows of A[a], kept for the
// tokens whose adapter it is.  blockIdx.y shares out the adapters of a tile,
// since a decode batch may bring 16 of them to 16 tokens.
//
// Within a window of 512, tokens whose adapters change often are tiled in the
// order of their adapters, so that A[a] is read once per MT tokens of adapter a
// however the requests are mixed (every block ranks its window's ids by
// counting: 1.4 us at 64 tokens, 3.3 at 256); packed prompts are tiled as they
// come.
//
// mma.sync on purpose: the product reads x and A once and does 2 rank flops per
// value of x, far below the tensor rate, and takes any mixture of adapters
// without a layout.
// ---------------------------------------------------------------------------
constexpr int kShrinkThreads = 256;
constexpr int kShrinkWindow = 512;

struct ShrinkArgs {
  const uint16_t* x;
  int64_t ldx;
  int T, K;
  const uint16_t* a_pool;
  const float* scale;
  const int32_t* ids;
  int n, rank, rp;
  uint16_t* v;
};

// A block's tile: the tokens in its places and the distinct adapters among them.
template <int MT>
struct ShrinkTile {
  __align__(16) uint32_t key[kShrinkWindow];
  int32_t id[MT], tok[MT];                             // adapter and token of a place; tok -1: none
  int32_t list[MT];                                    // the adapters of its runs
  uint32_t heads[(MT + 31) / 32];                      // places at which an adapter begins
};

// Fills the tile at place m0 of the window that starts at token `base`, after
// the wait for the launch before; returns the length of its list.  Ends with a
// barrier of the cluster.
template <int MT>
__device__ __forceinline__ int shrink_tile(const ShrinkArgs& p, ShrinkTile<MT>& s, int base, int m0, int ks) {
  pdl_wait();
  pdl_trigger();
  // Every adapter (n for none) and token of the window make one key.  Where the ids change often (a mixed
  // decode batch) the places are in the order of the keys: a token's place is the number of lower keys.
  const int Tw = min(kShrinkWindow, p.T - base), Tp = (Tw + 3) & ~3;
  int changes = 0;
  for (int t = threadIdx.x; t < Tp; t += kShrinkThreads) {
    const int id = lora_id(p.ids, p.T, p.n, t < Tw ? base + t : p.T);
    s.key[t] = t < Tw ? static_cast<uint32_t>(id < 0 ? p.n : id) * kShrinkWindow + t : 0xffffffffu;
  }
  if (threadIdx.x < MT) s.id[threadIdx.x] = s.tok[threadIdx.x] = -1;
  __syncthreads();
  for (int t = threadIdx.x; t + 1 < Tw; t += kShrinkThreads)
    changes += s.key[t] / kShrinkWindow != s.key[t + 1] / kShrinkWindow;
  const bool mixed = Tw > MT && __syncthreads_count(changes) * 16 > Tw;
  // this thread's two tokens at once
  static_assert(kShrinkWindow == 2 * kShrinkThreads, "two tokens per thread");
  const int t0 = threadIdx.x, t1 = t0 + kShrinkThreads;
  const uint32_t me0 = t0 < Tw ? s.key[t0] : 0u, me1 = t1 < Tw ? s.key[t1] : 0u;
  int place0 = t0, place1 = t1;
  if (mixed) {
    place0 = place1 = 0;
    if (Tw > kShrinkThreads) {
#pragma unroll 8
      for (int o = 0; o < Tp; o += 4) {
        const uint4 k = *reinterpret_cast<const uint4*>(&s.key[o]);
        place0 += (k.x < me0) + (k.y < me0) + (k.z < me0) + (k.w < me0);
        place1 += (k.x < me1) + (k.y < me1) + (k.z < me1) + (k.w < me1);
      }
    } else {
#pragma unroll 8
      for (int o = 0; o < Tp; o += 4) {
        const uint4 k = *reinterpret_cast<const uint4*>(&s.key[o]);
        place0 += (k.x < me0) + (k.y < me0) + (k.z < me0) + (k.w < me0);
      }
    }
  }
  auto put = [&](int t, uint32_t me, int place) {
    if (t < Tw && place >= m0 && place < m0 + MT) {
      const int id = static_cast<int>(me / kShrinkWindow);
      s.id[place - m0] = id < p.n ? id : -1;
      s.tok[place - m0] = base + t;
    }
  };
  put(t0, me0, place0);
  put(t1, me1, place1);
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int i = threadIdx.x;
  int id = -1;
  bool head = false;
  if (i < MT) {
    id = s.id[i];
    head = id >= 0 && (i == 0 || s.id[i - 1] != id);   // an adapter of two runs is listed, and computed, twice
  }
  if (i < (MT + 31) / 32 * 32) {
    const uint32_t m = __ballot_sync(0xffffffffu, head);
    if (lane == 0) s.heads[warp] = m;
  }
  __syncthreads();
  int n = 0;
#pragma unroll
  for (int w = 0; w < (MT + 31) / 32; ++w) {
    if (w == warp && head) s.list[n + __popc(s.heads[w] & ((1u << lane) - 1u))] = id;
    n += __popc(s.heads[w]);
  }
  if (ks > 1) cluster_sync_all();       // also: every rank runs before the first remote store
  else __syncthreads();
  return n;
}

// A pass's outputs, MT places x NC columns in pieces of 8 columns (16 bytes of
// v): `sums(at, f)` gives this block's sums of the piece that starts at output
// `at`; the cluster's ranks each add up their share of the pieces in rank order,
// scale, round and store.  column(c, r): the adapter of the piece at column c
// (-1: none), and its place r in v.
template <int MT, int NC, typename Sums, typename Column>
__device__ __forceinline__ void shrink_store(const ShrinkArgs& p, const ShrinkTile<MT>& s, float* part, int ks, int kr,
                                             Sums sums, Column column) {
  constexpr int kPieces = MT * NC / 8;
  const int own = (kPieces + ks - 1) / ks;
  if (ks > 1) {
    for (int at = threadIdx.x; at < kPieces; at += kShrinkThreads) {
      float f[8];
      sums(at * 8, f);
      const int owner = at / own;
      const uint32_t to = mapa_rank(smem_u32(part + (kr * own + at - owner * own) * 8), owner);
      st_cluster_v4(to, f[0], f[1], f[2], f[3]);
      st_cluster_v4(to + 16, f[4], f[5], f[6], f[7]);
    }
    cluster_sync_all();
  }
  for (int o = threadIdx.x; o < own; o += kShrinkThreads) {
    const int at = kr * own + o;
    if (at >= kPieces) break;
    const int i = at * 8 / NC;
    int r;
    const int id = column(at * 8 % NC, r);
    if (id < 0 || s.tok[i] < 0 || s.id[i] != id) continue;
    const float scale = p.scale ? p.scale[id] : 1.f;
    float f[8] = {};
    if (ks > 1) {
      for (int q = 0; q < ks; ++q) {
        const float4* u = reinterpret_cast<const float4*>(part + (q * own + o) * 8);
        const float4 a = u[0], b = u[1];
        f[0] += a.x; f[1] += a.y; f[2] += a.z; f[3] += a.w;
        f[4] += b.x; f[5] += b.y; f[6] += b.z; f[7] += b.w;
      }
    } else {
      sums(at * 8, f);
    }
    // rank is a multiple of 8: a piece is all rank or all padding, which is zero whatever the scale
    uint4 w = make_uint4(0, 0, 0, 0);
    if (r < p.rank)
      w = make_uint4(pack_bf16(scale * f[0], scale * f[1]), pack_bf16(scale * f[2], scale * f[3]),
                     pack_bf16(scale * f[4], scale * f[5]), pack_bf16(scale * f[6], scale * f[7]));
    *reinterpret_cast<uint4*>(p.v + static_cast<size_t>(s.tok[i]) * p.rp + r) = w;
  }
  if (ks == 1) __syncthreads();         // the sums' buffer is free again
}

// Few tokens: tiles of 16, the 8 warps split the block's depth, operands straight
// into registers.  Each thread loads 16 consecutive bytes of a row per operand:
// the depths of one 32-deep step are dealt to the two MMAs in the same order on
// both sides, and a warp takes two neighbouring steps (128 bytes of a row) at once.
template <int NJ>
struct ShrinkFew {
  static constexpr int MT = 16, NC = 8 * NJ, kOut = MT * NC, kPart = kOut + 64;
  static constexpr size_t kSmem = static_cast<size_t>(8 * kOut + 2 * kPart) * 4;
};

template <int NJ>
__global__ void __launch_bounds__(kShrinkThreads, 2) lora_shrink_few_kernel(const ShrinkArgs p) {
  using S = ShrinkFew<NJ>;
  constexpr int NC = S::NC, kOut = S::kOut;
  extern __shared__ __align__(16) float s_dyn[];
  float* red = s_dyn;                                  // [warp][place][column]
  float* part = s_dyn + 8 * kOut;                      // [pass parity][rank][its share of the outputs]
  __shared__ ShrinkTile<16> s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, tq = lane & 3;
  const int ks = static_cast<int>(cluster_nranks()), kr = static_cast<int>(cluster_rank());
  const int n_list = shrink_tile(p, s, 0, static_cast<int>(blockIdx.x / ks) * 16, ks);
  const int steps = (p.K + 31) / 32;
  const int c_lo = steps * kr / ks, c_hi = steps * (kr + 1) / ks;
  const int t0 = s.tok[g], t1 = s.tok[g + 8];
  const uint16_t* x0 = t0 >= 0 ? p.x + t0 * p.ldx : nullptr;
  const uint16_t* x1 = t1 >= 0 ? p.x + t1 * p.ldx : nullptr;
  // items (adapter of the list, NC rows of it) are shared out over blockIdx.y
  const int groups = (p.rp + NC - 1) / NC;
  int pass = 0;
  for (int item = blockIdx.y; item < n_list * groups; item += gridDim.y, ++pass) {
    {
      const int li = item / groups, n0 = (item - li * groups) * NC;
      const int id = s.list[li];
      const uint16_t* A = p.a_pool + static_cast<size_t>(id) * p.rank * p.K;
      float acc[NJ][4] = {};
      for (int c2 = c_lo + 2 * warp; c2 < c_hi; c2 += 16) {
        uint4 xv[2][2], av[2][NJ];
        const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int k = (c2 + u) * 32 + tq * 8;
          const bool in = c2 + u < c_hi && k < p.K;
          xv[u][0] = in && x0 ? __ldg(reinterpret_cast<const uint4*>(x0 + k)) : zero;
          xv[u][1] = in && x1 ? __ldg(reinterpret_cast<const uint4*>(x1 + k)) : zero;
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            const int r = n0 + j * 8 + g;
            av[u][j] = in && r < p.rank ? __ldg(reinterpret_cast<const uint4*>(A + static_cast<size_t>(r) * p.K + k)) : zero;
          }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            mma_bf16_16816(acc[j], xv[u][0].x, xv[u][1].x, xv[u][0].y, xv[u][1].y, av[u][j].x, av[u][j].y);
            mma_bf16_16816(acc[j], xv[u][0].z, xv[u][1].z, xv[u][0].w, xv[u][1].w, av[u][j].z, av[u][j].w);
          }
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<float2*>(&red[warp * kOut + (h * 8 + g) * NC + j * 8 + 2 * tq]) =
              make_float2(acc[j][2 * h], acc[j][2 * h + 1]);
      __syncthreads();
      auto warps = [&](int at, float* f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
          const float4* u = reinterpret_cast<const float4*>(red + w * kOut + at);
          const float4 a = u[0], b = u[1];
          f[0] += a.x; f[1] += a.y; f[2] += a.z; f[3] += a.w;
          f[4] += b.x; f[5] += b.y; f[6] += b.z; f[7] += b.w;
        }
      };
      shrink_store<16, NC>(p, s, part + (pass & 1) * S::kPart, ks, kr, warps, [&](int c, int& r) {
        r = n0 + c;
        return r < p.rp ? id : -1;
      });
    }
  }
}

// Many tokens: tiles of 64 places and NC columns, which hold as many of the
// tile's adapters as fit (a tile over the border of two requests takes no longer
// than another), so that x is read once: bound by its bytes.  A ring of 128-deep
// stages filled by cp.async (rows are gathered, so no TMA box), four warps over
// the rows times two over each stage's depth.
template <int NJ>
struct ShrinkMany {
  static constexpr int MT = 64, NC = 8 * NJ, kOut = MT * NC, kPart = kOut + 64;
  static constexpr int kHalf = (MT + NC) * 128;                      // 64 deep of a stage
  static constexpr int kStages = NJ == 16 ? 4 : 6;
  static constexpr size_t kSmem = static_cast<size_t>(kStages) * 2 * kHalf;
  static_assert((2 * kOut + kPart) * 4 <= kSmem, "the sums take the ring's place");
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

template <int NJ>
__global__ void __launch_bounds__(kShrinkThreads, 1) lora_shrink_many_kernel(const ShrinkArgs p) {
  using S = ShrinkMany<NJ>;
  constexpr int MT = S::MT, NC = S::NC, kOut = S::kOut, kStages = S::kStages;
  extern __shared__ __align__(128) uint8_t s_ring[];
  float* red = reinterpret_cast<float*>(s_ring);                     // [depth half][place][column], when the ring is done
  float* part = red + 2 * kOut;                                      // [rank][its share of the outputs]
  __shared__ ShrinkTile<MT> s;
  __shared__ int32_t s_col[NJ], s_r[NJ];                             // 8 columns' adapter (-1: none) and place in v
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wm = warp & 3, wk = warp >> 2;
  const int ks = static_cast<int>(cluster_nranks()), kr = static_cast<int>(cluster_rank());
  const int tile = blockIdx.x / ks;
  constexpr int kTiles = kShrinkWindow / MT;
  const int n_ad = shrink_tile(p, s, tile / kTiles * kShrinkWindow, tile % kTiles * MT, ks);
  const int KB = (p.K + 127) / 128;
  const int kb0 = kr * KB / ks, kb1 = (kr + 1) * KB / ks;
  const uint32_t ring = smem_u32(s_ring);
  // this thread's 16-byte pieces of a stage: piece lc of each half of rows lr, lr + 32, ...
  const int lr = threadIdx.x >> 3, lc = threadIdx.x & 7;
  const uint16_t* xr[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) xr[i] = s.tok[lr + i * 32] >= 0 ? p.x + s.tok[lr + i * 32] * p.ldx : nullptr;
  const int fit = NC / p.rp;             // adapters of a pass
  for (int l0 = blockIdx.y * fit; l0 < n_ad; l0 += fit * gridDim.y) {
    if (threadIdx.x < NJ) {
      const int a = 8 * threadIdx.x / p.rp, l = l0 + a;
      s_col[threadIdx.x] = a < fit && l < n_ad ? s.list[l] : -1;
      s_r[threadIdx.x] = 8 * threadIdx.x - a * p.rp;
    }
    __syncthreads();
    const int cols = min(fit, n_ad - l0) * p.rp;
    const uint16_t* ar[(NC + 31) / 32];
#pragma unroll
    for (int i = 0; i < (NC + 31) / 32; ++i) {
      const int row = lr + i * 32, id = s_col[row >> 3], r = s_r[row >> 3] + (row & 7);
      ar[i] = id >= 0 && r < p.rank ? p.a_pool + (static_cast<size_t>(id) * p.rank + r) * p.K : nullptr;
    }
    auto load = [&](int kb) {
      const uint32_t st = ring + static_cast<uint32_t>((kb - kb0) % kStages) * (2 * S::kHalf);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = kb * 128 + h * 64 + lc * 8;
        const uint32_t sh = st + h * S::kHalf;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = lr + i * 32;
          const bool in = xr[i] && k < p.K;
          cp_async16(sh + row * 128 + ((lc ^ (row & 7)) << 4), in ? xr[i] + k : p.x, in);
        }
#pragma unroll
        for (int i = 0; i < (NC + 31) / 32; ++i) {
          const int row = lr + i * 32;
          const bool in = ar[i] && k < p.K;
          if (row < cols) cp_async16(sh + (MT + row) * 128 + ((lc ^ (row & 7)) << 4), in ? ar[i] + k : p.a_pool, in);
        }
      }
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      if (kb0 + i < kb1) load(kb0 + i);
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
    float acc[NJ][4] = {};
    for (int kb = kb0; kb < kb1; ++kb) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
      __syncthreads();                   // stage kb has landed; stage kb - 1 is no longer read
      if (kb + kStages - 1 < kb1) load(kb + kStages - 1);
      asm volatile("cp.async.commit_group;" ::: "memory");
      const uint32_t sh = ring + static_cast<uint32_t>((kb - kb0) % kStages) * (2 * S::kHalf) + wk * S::kHalf;
      const int arow = wm * 16 + (lane & 15), hi = lane >> 4;
      uint32_t a[4][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) ldmatrix_x4(sh + arow * 128 + (((2 * k + hi) ^ (arow & 7)) << 4), a[k]);
#pragma unroll
      for (int j = 0; j < NJ; j += 2) {
        if (j * 8 < cols) {
          // rows j * 8 .. j * 8 + 15: matrices (rows 0-7, depth 0-7), (8-15, 0-7), (0-7, 8-15), (8-15, 8-15)
          const int brow = j * 8 + (lane & 15);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t b[4];
            ldmatrix_x4(sh + (MT + brow) * 128 + (((2 * k + hi) ^ (brow & 7)) << 4), b);
            mma_bf16_16816(acc[j], a[k][0], a[k][1], a[k][2], a[k][3], b[0], b[2]);
            mma_bf16_16816(acc[j + 1], a[k][0], a[k][1], a[k][2], a[k][3], b[1], b[3]);
          }
        }
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    const int g = lane >> 2, tq = lane & 3;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<float2*>(&red[wk * kOut + (wm * 16 + h * 8 + g) * NC + j * 8 + 2 * tq]) =
            make_float2(acc[j][2 * h], acc[j][2 * h + 1]);
    if (ks > 1) cluster_sync_all();      // every rank's ring is idle: sums may cross
    else __syncthreads();
    auto halves = [&](int at, float* f) {
      const float4* u = reinterpret_cast<const float4*>(red + at);
      const float4* v = reinterpret_cast<const float4*>(red + kOut + at);
      const float4 a = u[0], b = u[1], c = v[0], d = v[1];
      f[0] = a.x + c.x; f[1] = a.y + c.y; f[2] = a.z + c.z; f[3] = a.w + c.w;
      f[4] = b.x + d.x; f[5] = b.y + d.y; f[6] = b.z + d.z; f[7] = b.w + d.w;
    };
    shrink_store<MT, NC>(p, s, part, ks, kr, halves, [&](int c, int& r) {
      r = s_r[c >> 3];
      return s_col[c >> 3];
    });
    if (ks > 1) __syncthreads();         // the ring and the list of columns are free again
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
// clusters: of ks blocks, that run at once; what the tiles leave of them, at
// least `least` blocks a tile, shares out a tile's adapters.
template <typename S>
static cudaError_t launch_shrink(void (*kern)(ShrinkArgs), const ShrinkArgs& p, int ks, int clusters, int least,
                                 cudaStream_t st) {
  cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(S::kSmem));
  if (err != cudaSuccess) return err;
  const int tiles = (p.T + S::MT - 1) / S::MT;
  int split = clusters / tiles;
  split = split < least ? least : split > 16 ? 16 : split;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ks * tiles, split);
  cfg.blockDim = dim3(kShrinkThreads);
  cfg.dynamicSmemBytes = S::kSmem;
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
  return count_launch(cudaLaunchKernelEx(&cfg, kern, p));
}

// Few tokens (a window): K over 8 or 4 blocks (two blocks per SM: 30 clusters of
// 8, 66 of 4 at once).  Many: K split only as far as the tiles leave SMs idle
// (one block per SM: 15 clusters of 8, 33 of 4, 74 of 2).
static cudaError_t launch_shrink_for(const ShrinkArgs& p, cudaStream_t st) {
  if (p.T <= kShrinkWindow) {
    const int ks = p.T <= 64 ? 8 : 4, clusters = p.T <= 64 ? 28 : 64;
    return p.rp <= 16 ? launch_shrink<ShrinkFew<2>>(lora_shrink_few_kernel<2>, p, ks, clusters, 1, st)
                      : launch_shrink<ShrinkFew<4>>(lora_shrink_few_kernel<4>, p, ks, clusters, 1, st);
  }
  const int tiles = (p.T + 63) / 64;
  const int ks = tiles <= 15 ? 8 : tiles <= 33 ? 4 : tiles <= 74 ? 2 : 1;
  const int clusters = ks == 8 ? 15 : ks == 4 ? 33 : ks == 2 ? 74 : 148;
  // above 64 columns a pass holds one adapter: a tile over the border of two requests gives the second to a block
  // of its own (most find none: 2 us, against 57 us of one 128-column pass over 4096)
  return p.rp <= 32   ? launch_shrink<ShrinkMany<8>>(lora_shrink_many_kernel<8>, p, ks, clusters, 1, st)
         : p.rp <= 64 ? launch_shrink<ShrinkMany<16>>(lora_shrink_many_kernel<16>, p, ks, clusters, 1, st)
                      : launch_shrink<ShrinkMany<16>>(lora_shrink_many_kernel<16>, p, ks, clusters, 2, st);
}

// Returns a message on failure, nullptr on success.
const char* launch_lora(const LoraCall& c, cudaStream_t st, cudaError_t* cerr) {
  const int rp = (c.rank + 15) / 16 * 16;
  *cerr = cudaSuccess;
  const TokenArgs few = {c.x, c.w, c.a, c.b, c.scale, c.ids, c.y, c.ldx, c.ldy, c.T, c.d_in, c.d_out, c.n, c.rank};
  int cluster = 0;
  if (lora_token_fits(few, cluster)) {
    *cerr = launch_lora_token(few, cluster, st);
    return *cerr == cudaSuccess ? nullptr : "adapter projection launch failed";
  }
  const bool pairs = !proj_fits(c.T, c.d_out, 128, c.d_in, true);

  // v first
  const ShrinkArgs p = {c.x, c.ldx, c.T, c.d_in, c.a, c.scale, c.ids, c.n, c.rank, rp, c.v};
  *cerr = launch_shrink_for(p, st);
  if (*cerr != cudaSuccess) return "adapter shrink launch failed";

  const LoraArgs la = {c.ids, c.v, c.b, c.T, c.n, c.rank, rp, c.d_out};
  if (pairs) {
    DenseArgs g = {};
    g.n = 1;
    DenseProblem& P = g.p[0];
    dense_tiles(P, c.T, c.d_out, c.d_in, 256);
    if (!dense_operand_map(&P.a, c.x, false, c.T, c.d_in, 2ull * c.ldx, 128) ||
        !dense_operand_map(&P.b, c.w, false, c.d_out, c.d_in, 2ull * c.d_in, 128) ||
        !dense_store_map(&P.c0, c.y, c.d_out, c.T, 2ull * c.ldy))
      return "cuTensorMapEncodeTiled failed";
    g.lora = la;
    *cerr = launch_dense<kEpiStore, true>(g, true, st);
    return *cerr == cudaSuccess ? nullptr : "projection launch failed";
  }
  ProjArgs g = {};
  g.T = c.T;
  g.M = c.d_out;
  g.early = 1;
  g.out = c.y;
  g.ld = c.ldy;
  g.lora = la;
  if (!proj_maps(g, c.w, false, c.d_out, c.d_in, 2ull * c.d_in, c.x, 2ull * c.ldx)) return "cuTensorMapEncodeTiled failed";
  *cerr = launch_proj<kEpiStore, true>(g, st);
  return *cerr == cudaSuccess ? nullptr : "projection launch failed";
}

}  // namespace ftm
