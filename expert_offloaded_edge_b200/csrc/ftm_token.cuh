// Products of a handful of tokens with dense weights, bf16, from registers: 16
// rows of weights on the M side of mma.sync and 8 or 16 tokens on the N side.
// What bounds such a product is the latency of the weights' bytes, which wants
// many loads in flight and little around them: no ring, no tensor memory, no
// cluster.  Each thread loads 16 consecutive bytes of a row per operand; the
// depths of one 32-deep step are dealt to the two MMAs in the same order on both
// sides.  Two blocks of 64 registers a thread per SM: four steps at a time, or
// one block per SM with room for eight, was slower (a projection of one token,
// 2048 x 2048, with its adapter: 4.8 us, 5.4 and 6.5).
//
// Every block reads all tokens: beyond 16 that is more than its weights, and for
// 16 of large weights as many bytes from L2.  The gated block in a replayed
// graph, here and on ftm_proj.cuh, us:
//    1 token,  2048 x 768     4.2   7.8      16 tokens,  2048 x 768     5.5   8.2
//    1 token,  4096 x 2048   11.5  16.0      16 tokens,  4096 x 2048   14.9  16.6
//    8 tokens, 6144 x 2048   17.5  20.5      16 tokens,  6144 x 2048   21.7  20.9
//    1 token,  6144 x 256     6.4   9.4      16 tokens,  6144 x 256     9.6   9.9
#pragma once

#include "ftm_dense.cuh"

namespace ftm {

constexpr int kTokenThreads = 512;
constexpr int kTokenRows = 16;                           // rows of weights of a tile
constexpr int kTokenTile = 8;                            // tokens of a tile
constexpr int kTokenPitch = 20;                          // of a token's 16 sums: a quad's stores fall into different banks

__device__ __forceinline__ void mma_bf16_16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The products of a tile's 16 rows with NT tiles of tokens over one of `warps`
// warps' share of K, into to[token * kTokenPitch + row].  r0, r1: rows lane / 4
// and that + 8 of the tile; xr: token lane / 4 of each tile (NULL: zeros).
// ready() is called once, before the tokens are first read.  EARLY: the weights
// are read before the launch's wait (ftm_common.cuh).
template <int NT, bool EARLY, typename Ready>
__device__ __forceinline__ void token_dot(const uint16_t* r0, const uint16_t* r1, const uint16_t* const (&xr)[NT], int K, int warp,
                                          int warps, float* to, Ready ready) {
  constexpr int U = 2;                                   // steps at a time
  const int lane = threadIdx.x % 32, g = lane >> 2, tq = lane & 3;
  const int steps = (K + 31) / 32;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  auto weight = [](const uint16_t* p) {
    return EARLY ? ld_early(reinterpret_cast<const uint4*>(p)) : __ldg(reinterpret_cast<const uint4*>(p));
  };
  float acc[NT][4] = {};
  bool waited = false;
  // two neighbouring steps (128 bytes of a row) are a warp's, then the next warp's
  for (int c = U * warp; c < steps; c += warps * U) {
    uint4 a0[U], a1[U], b[U][NT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = (c + u) * 32 + tq * 8;
      const bool in = k < K;
      a0[u] = in && r0 ? weight(r0 + k) : zero;
      a1[u] = in && r1 ? weight(r1 + k) : zero;
    }
    if (!waited) ready();
    waited = true;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = (c + u) * 32 + tq * 8;
#pragma unroll
      for (int j = 0; j < NT; ++j) b[u][j] = k < K && xr[j] ? *reinterpret_cast<const uint4*>(xr[j] + k) : zero;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        mma_bf16_16816(acc[j], a0[u].x, a1[u].x, a0[u].y, a1[u].y, b[u][j].x, b[u][j].y);
        mma_bf16_16816(acc[j], a0[u].z, a1[u].z, a0[u].w, a1[u].w, b[u][j].z, b[u][j].w);
      }
    }
  }
  if (!waited) ready();
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) to[(j * kTokenTile + 2 * tq + (i & 1)) * kTokenPitch + (i >> 1) * 8 + g] = acc[j][i];
}

// out[t][m] = sum_k A[m][k] x[t][k]; gated: of 8 gate rows and the 8 up rows of
// the same outputs, out = act(g) u, with g and u kept on request.
struct TokenProduct {
  const uint16_t *a, *x;     // [rows][K], [T][K]
  uint16_t *out, *pre;       // [T][M]; gated: g, u [T][2M] or NULL
  int T, K, M, act;
  int early;                 // the launch before is this call's own, and waited: A may be read before it ends
};

template <bool GATED, int NT>
__global__ void __launch_bounds__(kTokenThreads, 2) token_product_kernel(const TokenProduct p) {
  constexpr int kWarps = kTokenThreads / 32, kOut = GATED ? kTokenRows / 2 : kTokenRows;
  __shared__ float red[kWarps][NT * kTokenTile * kTokenPitch];    // [warp][token][row]
  const int warp = threadIdx.x / 32, g = threadIdx.x % 32 / 4;
  const int m0 = blockIdx.x * kOut;
  auto ready = [] { pdl_wait(); pdl_trigger(); };
  if (!p.early) ready();
  const int r0 = m0 + g, r1 = GATED ? p.M + r0 : r0 + 8;
  const bool in0 = r0 < p.M, in1 = GATED ? in0 : r1 < p.M;
  const uint16_t* xr[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int t = j * kTokenTile + g;
    xr[j] = t < p.T ? p.x + static_cast<size_t>(t) * p.K : nullptr;
  }
  token_dot<NT, !GATED>(in0 ? p.a + static_cast<size_t>(r0) * p.K : nullptr, in1 ? p.a + static_cast<size_t>(r1) * p.K : nullptr,
                xr, p.K, warp, kWarps, red[warp], [&] {
                  if (p.early) ready();
                });
  __syncthreads();
  if (threadIdx.x >= NT * kTokenTile * kOut) return;
  const int t = threadIdx.x / kOut, i = threadIdx.x % kOut, m = m0 + i;
  if (t >= p.T || m >= p.M) return;
  auto sum = [&](int row) {
    float f = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) f += red[w][t * kTokenPitch + row];
    return f;
  };
  auto bf16 = [](float f) { return static_cast<uint16_t>(pack_bf16(f, 0.f)); };
  float v = sum(i);
  if constexpr (GATED) {
    const float u = sum(kOut + i);
    if (p.pre) {
      uint16_t* q = p.pre + static_cast<size_t>(t) * 2 * p.M + m;
      q[0] = bf16(v);
      q[p.M] = bf16(u);
    }
    v = act_value(v, p.act) * u;
  }
  p.out[static_cast<size_t>(t) * p.M + m] = bf16(v);
}

// Whether a gated block runs here (the figures above), both products: the down
// product here behind a gate/up product of ftm_proj.cuh took 27 us for the 21 of
// the largest case, since its blocks move in early beside it.
inline bool token_fits(int T, int d, int I) {
  return T <= kTokenTile || (T <= 2 * kTokenTile && 4ull * d * I <= (40u << 20));
}

template <bool GATED>
cudaError_t launch_token_product(const TokenProduct& p, cudaStream_t st) {
  const int out = GATED ? kTokenRows / 2 : kTokenRows;
  return launch_pdl(p.T <= kTokenTile ? token_product_kernel<GATED, 1> : token_product_kernel<GATED, 2>,
                    dim3((p.M + out - 1) / out), dim3(kTokenThreads), 0, st, p);
}

}  // namespace ftm
