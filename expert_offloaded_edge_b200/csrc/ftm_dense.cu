// The dense gated feed-forward block (an MoE model's leading dense layers, its
// shared expert) and its backward pass, on the CTA-pair engine of ftm_dense.cuh:
//
//   forward   h = act(x Wg^T) * (x Wu^T)     one launch: both projections, activation, product
//             y = h Wd^T                     one launch
//   backward  dh = dy Wd; dg = dh u act'(g); du = dh act(g); h = act(g) u
//                                            one launch: the product and its epilogue
//             dx = [dg du] Wgu, dWgu = [dg du]^T x, dWd = dy^T h
//                                            one launch: three independent products
//
// The forward pass of a training step keeps g and u rounded to bf16 (4 T I
// bytes): recomputing them instead costs a third of the backward's products.
// dg, du and h are rounded to bf16 between the two backward launches, as the
// operands of the next products; every sum is fp32.
#include "ftm_dense.cuh"

namespace ftm {

const char* launch_gated_ffn_small(int act, const void* x, int T, int d, int I, const void* bank, size_t w_d_off,
                                   void* h, void* y, cudaStream_t st, cudaError_t* cerr);

const char* launch_gated_ffn(int act, const void* x, int T, int d, int I, const void* bank, size_t w_d_off, void* pre,
                             void* h, void* y, cudaStream_t st, cudaError_t* cerr) {
  if (!pre && T <= 256) return launch_gated_ffn_small(act, x, T, d, I, bank, w_d_off, h, y, st, cerr);
  const uint8_t* w = static_cast<const uint8_t*>(bank);
  uint8_t* pp = static_cast<uint8_t*>(pre);
  *cerr = cudaSuccess;
  DenseArgs g = {};
  g.n = 1;
  g.act = act;
  g.keep = pre != nullptr;
  DenseProblem& P = g.p[0];
  dense_tiles(P, T, I, d, 128);
  P.up_row0 = I;
  bool ok = dense_operand_map(&P.a, x, false, T, d, 2ull * d, 128) &&
            dense_operand_map(&P.b, w, false, 2ull * I, d, 2ull * d, 128) && dense_store_map(&P.c0, h, I, T, 2ull * I);
  if (ok && pre) ok = dense_store_map(&P.c1, pp, I, T, 4ull * I) && dense_store_map(&P.c2, pp + 2ull * I, I, T, 4ull * I);
  DenseArgs g2 = {};
  g2.n = 1;
  DenseProblem& Q = g2.p[0];
  dense_tiles(Q, T, d, I, 256);
  ok = ok && dense_operand_map(&Q.a, h, false, T, I, 2ull * I, 128) &&
       dense_operand_map(&Q.b, w + w_d_off, false, d, I, 2ull * I, 128) && dense_store_map(&Q.c0, y, d, T, 2ull * d);
  if (!ok) return "cuTensorMapEncodeTiled failed";
  prof_mark(FTM_K_GEMM1, st, false);
  *cerr = launch_dense<kEpiGated, 256, false>(g, st);
  prof_mark(FTM_K_GEMM1, st, true);
  if (*cerr != cudaSuccess) return "gate/up launch failed";
  prof_mark(FTM_K_GEMM2, st, false);
  *cerr = launch_dense<kEpiStore, 256, false>(g2, st);
  prof_mark(FTM_K_GEMM2, st, true);
  return *cerr == cudaSuccess ? nullptr : "down launch failed";
}

// dgu [T][2I] and h [T][I] are workspace; dx or (dw_gu, dw_d) may be NULL.
const char* launch_gated_ffn_backward(int act, const void* x, int T, int d, int I, const void* bank, size_t w_d_off,
                                      const void* pre, const void* dy, void* dx, void* dw_gu, void* dw_d, void* dgu,
                                      void* h, cudaStream_t st, cudaError_t* cerr) {
  const uint8_t* w = static_cast<const uint8_t*>(bank);
  uint8_t* dg = static_cast<uint8_t*>(dgu);
  *cerr = cudaSuccess;
  DenseArgs g = {};
  g.n = 1;
  g.act = act;
  g.keep = dw_d != nullptr;
  g.pre = static_cast<const uint16_t*>(pre);
  DenseProblem& P = g.p[0];
  dense_tiles(P, T, I, d, 256);
  P.b_mn = 1;
  bool ok = dense_operand_map(&P.a, dy, false, T, d, 2ull * d, 128) &&
            dense_operand_map(&P.b, w + w_d_off, true, I, d, 2ull * I, 0) && dense_store_map(&P.c0, dg, I, T, 4ull * I) &&
            dense_store_map(&P.c1, dg + 2ull * I, I, T, 4ull * I) && dense_store_map(&P.c2, h, I, T, 2ull * I);
  DenseArgs g2 = {};
  if (dw_d) {
    DenseProblem& Q = g2.p[g2.n++];        // dWgu [2I][d] = dgu^T x
    dense_tiles(Q, 2 * I, d, T, 256);
    Q.a_mn = Q.b_mn = 1;
    ok = ok && dense_operand_map(&Q.a, dgu, true, 2ull * I, T, 4ull * I, 0) &&
         dense_operand_map(&Q.b, x, true, d, T, 2ull * d, 0) && dense_store_map(&Q.c0, dw_gu, d, 2ull * I, 2ull * d);
    DenseProblem& R = g2.p[g2.n++];        // dWd [d][I] = dy^T h
    dense_tiles(R, d, I, T, 256);
    R.a_mn = R.b_mn = 1;
    ok = ok && dense_operand_map(&R.a, dy, true, d, T, 2ull * d, 0) &&
         dense_operand_map(&R.b, h, true, I, T, 2ull * I, 0) && dense_store_map(&R.c0, dw_d, I, d, 2ull * I);
  }
  if (dx) {
    DenseProblem& Q = g2.p[g2.n++];        // dx = dgu Wgu
    dense_tiles(Q, T, d, 2 * I, 256);
    Q.b_mn = 1;
    ok = ok && dense_operand_map(&Q.a, dgu, false, T, 2ull * I, 4ull * I, 128) &&
         dense_operand_map(&Q.b, w, true, d, 2ull * I, 2ull * d, 0) && dense_store_map(&Q.c0, dx, d, T, 2ull * d);
  }
  if (!ok) return "cuTensorMapEncodeTiled failed";
  *cerr = launch_dense<kEpiDgate, 256, false>(g, st);
  if (*cerr != cudaSuccess) return "activation gradient launch failed";
  *cerr = launch_dense<kEpiStore, 256, false>(g2, st);
  return *cerr == cudaSuccess ? nullptr : "gradient products launch failed";
}

}  // namespace ftm
