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
// Each product runs on one of three engines: tiles of 256 x 256 on CTA pairs
// (ftm_dense.cuh), for few tokens 128 rows of weights at a time (ftm_proj.cuh),
// and for a handful 16 rows from registers (ftm_token.cuh).
#include <initializer_list>

#include "ftm_proj.cuh"
#include "ftm_token.cuh"

namespace ftm {

static const char* kMapsFailed = "cuTensorMapEncodeTiled failed";

const char* launch_gated_ffn(int act, const void* x, int T, int d, int I, const void* bank, size_t w_d_off, void* pre,
                             void* h, void* y, cudaStream_t st, cudaError_t* cerr) {
  const uint8_t* w = static_cast<const uint8_t*>(bank);
  uint8_t* pp = static_cast<uint8_t*>(pre);
  const uint64_t rd = 2ull * d, rI = 2ull * I;          // bytes of a row
  *cerr = cudaSuccess;
  prof_mark(FTM_K_GEMM1, st, false);
  const TokenProduct gate_up = {static_cast<const uint16_t*>(bank), static_cast<const uint16_t*>(x),
                                static_cast<uint16_t*>(h), static_cast<uint16_t*>(pre), T, d, I, act, 0};
  const bool handful = token_fits(T, d, I);
  if (handful) {
    *cerr = launch_token_product<true>(gate_up, st);
  } else if (proj_fits(T, I, 64, d)) {
    ProjArgs g = {};
    g.T = T;
    g.M = I;
    g.up_row0 = I;
    g.act = act;
    g.keep = pre != nullptr;
    g.out = static_cast<uint16_t*>(h);
    g.ld = I;
    g.pre = static_cast<uint16_t*>(pre);
    if (!proj_maps(g, w, false, 2ull * I, d, rd, x, rd)) return kMapsFailed;
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
        !dense_half_map(&P.c0, h, I, T, rI))
      return kMapsFailed;
    if (pre && (!dense_half_map(&P.c1, pp, I, T, 2 * rI) || !dense_half_map(&P.c2, pp + rI, I, T, 2 * rI))) return kMapsFailed;
    *cerr = launch_dense<kEpiGated, false>(g, true, st);
  }
  prof_mark(FTM_K_GEMM1, st, true);
  if (*cerr != cudaSuccess) return "gate/up launch failed";
  prof_mark(FTM_K_GEMM2, st, false);
  const TokenProduct down = {reinterpret_cast<const uint16_t*>(w + w_d_off), static_cast<const uint16_t*>(h),
                             static_cast<uint16_t*>(y), nullptr, T, I, d, act, 1};
  if (handful) {
    *cerr = launch_token_product<false>(down, st);
  } else if (proj_fits(T, d, 128, I)) {
    ProjArgs g = {};
    g.T = T;
    g.M = d;
    g.early = 1;
    g.out = static_cast<uint16_t*>(y);
    g.ld = d;
    if (!proj_maps(g, w + w_d_off, false, d, I, rI, h, rI)) return kMapsFailed;
    *cerr = launch_proj<kEpiStore, false>(g, st);
  } else {
    DenseArgs g = {};
    g.n = 1;
    DenseProblem& Q = g.p[0];
    dense_tiles(Q, T, d, I, 256);
    if (!dense_operand_map(&Q.a, h, false, T, I, rI, 128) ||
        !dense_operand_map(&Q.b, w + w_d_off, false, d, I, rI, 128) || !dense_store_map(&Q.c0, y, d, T, rd))
      return kMapsFailed;
    *cerr = launch_dense<kEpiStore, false>(g, true, st);
  }
  prof_mark(FTM_K_GEMM2, st, true);
  return *cerr == cudaSuccess ? nullptr : "down launch failed";
}

// dgu [T][2I] and h [T][I] are workspace; dx or (dw_gu, dw_d) may be NULL.
const char* launch_gated_ffn_backward(int act, const void* x, int T, int d, int I, const void* bank, size_t w_d_off,
                                      const void* pre, const void* dy, void* dx, void* dw_gu, void* dw_d, void* dgu,
                                      void* h, cudaStream_t st, cudaError_t* cerr) {
  const uint8_t* w = static_cast<const uint8_t*>(bank);
  uint8_t* dg = static_cast<uint8_t*>(dgu);
  const uint64_t rd = 2ull * d, rI = 2ull * I;
  *cerr = cudaSuccess;
  if (proj_fits(T, I, 128, d)) {
    ProjArgs g = {};
    g.T = T;
    g.M = I;
    g.act = act;
    g.keep = dw_d != nullptr;
    g.out = static_cast<uint16_t*>(dgu);
    g.ld = 2ll * I;
    g.pre = static_cast<uint16_t*>(const_cast<void*>(pre));
    g.h = static_cast<uint16_t*>(h);
    if (!proj_maps(g, w + w_d_off, true, I, d, rI, dy, rd)) return kMapsFailed;
    *cerr = launch_proj<kEpiDgate, false>(g, st);
  } else {
    DenseArgs g = {};
    g.n = 1;
    g.act = act;
    g.keep = dw_d != nullptr;
    const uint8_t* pp = static_cast<const uint8_t*>(pre);
    DenseProblem& P = g.p[0];
    dense_tiles(P, T, I, d, 256);
    P.b_mn = 1;
    if (!dense_operand_map(&P.a, dy, false, T, d, rd, 128) || !dense_operand_map(&P.b, w + w_d_off, true, I, d, rI, 0) ||
        !dense_half_map(&P.c0, dg, I, T, 2 * rI) || !dense_half_map(&P.c1, dg + rI, I, T, 2 * rI) ||
        !dense_half_map(&P.c2, h, I, T, rI) || !dense_half_map(&P.p0, pp, I, T, 2 * rI) ||
        !dense_half_map(&P.p1, pp + rI, I, T, 2 * rI))
      return kMapsFailed;
    *cerr = launch_dense<kEpiDgate, false>(g, true, st);
  }
  if (*cerr != cudaSuccess) return "activation gradient launch failed";
  // The products.  Each is out[rows][cols] = P Q^T over depth K.
  struct Product {
    const void *p, *q;                 // [rows][K] and [cols][K], or stored [K][...] where mn
    bool p_mn, q_mn;
    int rows, cols, K;
    uint64_t p_pitch, q_pitch;
    void* out;
  };
  const Product all[3] = {
      {dgu, x, true, true, 2 * I, d, T, 2 * rI, rd, dw_gu},      // dWgu = dgu^T x
      {dy, h, true, true, d, I, T, rd, rI, dw_d},                // dWd = dy^T h
      {dgu, w, false, true, T, d, 2 * I, 2 * rI, rd, dx},        // dx = dgu Wgu
  };
  // One launch holds all, but for a product of few tiles that is deeper than the
  // others keep the pairs busy for: in a launch of its own it is split along K
  // (worth it from 24 blocks of 64: a pair takes 0.42 us for one, a launch 6 us).
  // The choice looks at all three, so that a gradient has the same bits whichever
  // others are asked for.
  DenseProblem problems[3];
  bool alone[3];
  long work = 0;
  for (int i = 0; i < 3; ++i) {
    const Product& P = all[i];
    DenseProblem& Q = problems[i];
    Q = {};
    dense_tiles(Q, P.rows, P.cols, P.K, 256);
    Q.a_mn = P.p_mn;
    Q.b_mn = P.q_mn;
    work += static_cast<long>(Q.tiles) * Q.kb;
    if (P.out && (!dense_operand_map(&Q.a, P.p, P.p_mn, P.rows, P.K, P.p_pitch, 128) ||
                  !dense_operand_map(&Q.b, P.q, P.q_mn, P.cols, P.K, P.q_pitch, 128) ||
                  !dense_store_map(&Q.c0, P.out, P.cols, P.rows, 2ull * P.cols)))
      return kMapsFailed;
  }
  const int pairs = num_sms() / 2;
  for (int i = 0; i < 3; ++i) alone[i] = problems[i].tiles <= pairs / 2 && problems[i].kb - work / pairs >= 24;
  // In order: split weight gradients, which leave pairs idle for those behind
  // them, the common launch, a split dx.  The first waits for dg, du and h, those
  // behind it for nothing but the end.
  bool launched = false;
  auto launch = [&](std::initializer_list<int> which, bool split) -> cudaError_t {
    DenseArgs g = {};
    for (int i : which)
      if (all[i].out && alone[i] == split) g.p[g.n++] = problems[i];
    if (!g.n) return cudaSuccess;
    g.early = launched;
    launched = true;
    return launch_dense<kEpiStore, false>(g, split, st);
  };
  if (alone[0] && alone[1] && problems[0].tiles + problems[1].tiles <= pairs / 2) {
    *cerr = launch({0, 1}, true);
  } else {
    *cerr = launch({0}, true);
    if (*cerr == cudaSuccess) *cerr = launch({1}, true);
  }
  if (*cerr == cudaSuccess) *cerr = launch({0, 1, 2}, false);
  if (*cerr != cudaSuccess) return "gradient products launch failed";
  if (dx && alone[2]) {
    if (proj_fits(T, d, 128, 2 * I)) {
      ProjArgs s = {};
      s.T = T;
      s.M = d;
      s.early = launched ? 2 : 0;
      s.out = static_cast<uint16_t*>(dx);
      s.ld = d;
      if (!proj_maps(s, w, true, d, 2ull * I, rd, dgu, 2 * rI)) return kMapsFailed;
      *cerr = launch_proj<kEpiStore, false>(s, st);
    } else {
      *cerr = launch({2}, true);
    }
    if (*cerr != cudaSuccess) return "gradient product launch failed";
  }
  return nullptr;
}

}  // namespace ftm
