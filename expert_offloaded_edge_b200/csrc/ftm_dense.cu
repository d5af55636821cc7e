// The dense gated feed-forward block (an MoE model's leading dense layers, its
// shared expert) and its backward pass:
//
//   forward   h = act(x Wg^T) * (x Wu^T)     one launch: both projections, activation, product
//             y = h Wd^T                     one launch
//   backward  dh = dy Wd; dg = dh u act'(g); du = dh act(g); h = act(g) u
//                                            one launch: the product and its epilogue
//             dx = [dg du] Wgu, dWgu = [dg du]^T x, dWd = dy^T h
//                                            independent products, one launch where they fill the GPU
//
// The forward pass of a training step keeps g and u rounded to bf16 (4 T I
// bytes): recomputing them instead costs a third of the backward's products.
// dg, du and h are rounded to bf16 between the two backward launches, as the
// operands of the next products; every sum is fp32.
//
// Each product runs on one of two engines: tiles of 256 x 256 on CTA pairs
// (ftm_dense.cuh), bound by the tensor cores, or, where those tiles are too few
// to occupy the GPU, 128-row tiles split along K over a cluster (ftm_proj.cuh),
// bound by the bytes.
#include "ftm_proj.cuh"

namespace ftm {

// Whether an [M][N] product has too few of the pair engine's tiles to occupy the GPU.
static bool few_tiles(int M, int N, int cols) {
  return static_cast<long>((M + kDTileM - 1) / kDTileM) * ((N + cols - 1) / cols) < num_sms() / 4;
}

const char* launch_gated_ffn(int act, const void* x, int T, int d, int I, const void* bank, size_t w_d_off, void* pre,
                             void* h, void* y, cudaStream_t st, cudaError_t* cerr) {
  static const char* maps = "cuTensorMapEncodeTiled failed";
  const uint8_t* w = static_cast<const uint8_t*>(bank);
  uint8_t* pp = static_cast<uint8_t*>(pre);
  const uint64_t rd = 2ull * d, rI = 2ull * I;          // bytes of a row
  *cerr = cudaSuccess;
  prof_mark(FTM_K_GEMM1, st, false);
  if (few_tiles(T, I, 128)) {
    ProjArgs g = {};
    g.T = T;
    g.M = I;
    g.up_row0 = I;
    g.act = act;
    g.keep = pre != nullptr;
    g.out = static_cast<uint16_t*>(h);
    g.ld = I;
    g.pre = static_cast<uint16_t*>(pre);
    if (!proj_maps(g, w, false, 2ull * I, d, rd, x, rd)) return maps;
    *cerr = launch_proj<kEpiGated, false>(g, st);
  } else {
    DenseArgs g = {};
    g.n = 1;
    g.act = act;
    g.keep = pre != nullptr;
    DenseProblem& P = g.p[0];
    dense_tiles(P, T, I, d, 128);
    P.up_row0 = I;
    if (!dense_operand_map(&P.a, x, false, T, d, rd, 128) || !dense_operand_map(&P.b, w, false, 2ull * I, d, rd, 128) ||
        !dense_store_map(&P.c0, h, I, T, rI))
      return maps;
    if (pre && (!dense_store_map(&P.c1, pp, I, T, 2 * rI) || !dense_store_map(&P.c2, pp + rI, I, T, 2 * rI))) return maps;
    *cerr = launch_dense<kEpiGated, 256, false>(g, st);
  }
  prof_mark(FTM_K_GEMM1, st, true);
  if (*cerr != cudaSuccess) return "gate/up launch failed";
  prof_mark(FTM_K_GEMM2, st, false);
  if (few_tiles(T, d, 256)) {
    ProjArgs g = {};
    g.T = T;
    g.M = d;
    g.early = 1;
    g.out = static_cast<uint16_t*>(y);
    g.ld = d;
    if (!proj_maps(g, w + w_d_off, false, d, I, rI, h, rI)) return maps;
    *cerr = launch_proj<kEpiStore, false>(g, st);
  } else {
    DenseArgs g = {};
    g.n = 1;
    DenseProblem& Q = g.p[0];
    dense_tiles(Q, T, d, I, 256);
    if (!dense_operand_map(&Q.a, h, false, T, I, rI, 128) ||
        !dense_operand_map(&Q.b, w + w_d_off, false, d, I, rI, 128) || !dense_store_map(&Q.c0, y, d, T, rd))
      return maps;
    *cerr = launch_dense<kEpiStore, 256, false>(g, st);
  }
  prof_mark(FTM_K_GEMM2, st, true);
  return *cerr == cudaSuccess ? nullptr : "down launch failed";
}

// dgu [T][2I] and h [T][I] are workspace; dx or (dw_gu, dw_d) may be NULL.
const char* launch_gated_ffn_backward(int act, const void* x, int T, int d, int I, const void* bank, size_t w_d_off,
                                      const void* pre, const void* dy, void* dx, void* dw_gu, void* dw_d, void* dgu,
                                      void* h, cudaStream_t st, cudaError_t* cerr) {
  static const char* maps = "cuTensorMapEncodeTiled failed";
  const uint8_t* w = static_cast<const uint8_t*>(bank);
  uint8_t* dg = static_cast<uint8_t*>(dgu);
  const uint64_t rd = 2ull * d, rI = 2ull * I;
  *cerr = cudaSuccess;
  if (few_tiles(T, I, 256)) {
    ProjArgs g = {};
    g.T = T;
    g.M = I;
    g.act = act;
    g.keep = dw_d != nullptr;
    g.out = static_cast<uint16_t*>(dgu);
    g.ld = 2ll * I;
    g.pre = static_cast<uint16_t*>(const_cast<void*>(pre));
    g.h = static_cast<uint16_t*>(h);
    if (!proj_maps(g, w + w_d_off, true, I, d, rI, dy, rd)) return maps;
    *cerr = launch_proj<kEpiDgate, false>(g, st);
  } else {
    DenseArgs g = {};
    g.n = 1;
    g.act = act;
    g.keep = dw_d != nullptr;
    g.pre = static_cast<const uint16_t*>(pre);
    DenseProblem& P = g.p[0];
    dense_tiles(P, T, I, d, 256);
    P.b_mn = 1;
    if (!dense_operand_map(&P.a, dy, false, T, d, rd, 128) || !dense_operand_map(&P.b, w + w_d_off, true, I, d, rI, 0) ||
        !dense_store_map(&P.c0, dg, I, T, 2 * rI) || !dense_store_map(&P.c1, dg + rI, I, T, 2 * rI) ||
        !dense_store_map(&P.c2, h, I, T, rI))
      return maps;
    *cerr = launch_dense<kEpiDgate, 256, false>(g, st);
  }
  if (*cerr != cudaSuccess) return "activation gradient launch failed";
  DenseArgs g = {};
  bool ok = true;
  if (dw_d) {
    DenseProblem& Q = g.p[g.n++];        // dWgu [2I][d] = dgu^T x
    dense_tiles(Q, 2 * I, d, T, 256);
    Q.a_mn = Q.b_mn = 1;
    ok = ok && dense_operand_map(&Q.a, dgu, true, 2ull * I, T, 2 * rI, 0) &&
         dense_operand_map(&Q.b, x, true, d, T, rd, 0) && dense_store_map(&Q.c0, dw_gu, d, 2ull * I, rd);
    DenseProblem& R = g.p[g.n++];        // dWd [d][I] = dy^T h
    dense_tiles(R, d, I, T, 256);
    R.a_mn = R.b_mn = 1;
    ok = ok && dense_operand_map(&R.a, dy, true, d, T, rd, 0) && dense_operand_map(&R.b, h, true, I, T, rI, 0) &&
         dense_store_map(&R.c0, dw_d, I, d, rI);
  }
  if (dx) {
    DenseProblem& Q = g.p[g.n++];        // dx = dgu Wgu
    dense_tiles(Q, T, d, 2 * I, 256);
    Q.b_mn = 1;
    ok = ok && dense_operand_map(&Q.a, dgu, false, T, 2ull * I, 2 * rI, 128) &&
         dense_operand_map(&Q.b, w, true, d, 2ull * I, rd, 0) && dense_store_map(&Q.c0, dx, d, T, rd);
  }
  if (!ok) return maps;
  *cerr = launch_dense<kEpiStore, 256, false>(g, st);
  return *cerr == cudaSuccess ? nullptr : "gradient products launch failed";
}

}  // namespace ftm
