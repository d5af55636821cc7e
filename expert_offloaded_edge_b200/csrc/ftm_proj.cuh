// Dense bf16 projections of few tokens, bound by the bytes of the weights:
// out[t][m] = sum_k A[m][k] X[t][k] with the weight rows on the MMA's M side
// (128 per tile) and BN tokens on its N side, so one token streams full weight
// tiles.  A cluster of ks CTAs splits each tile's K; the partial sums cross
// shared memory once, 16 bytes a store (every rank sums the outputs it owns, in
// rank order, so the result does not depend on timing), and the epilogue runs
// from there on pieces of 2 outputs of 4 tokens: a warp covers 64 outputs, 128
// bytes of a token's row.
//
//   kEpiStore  out = D
//   kEpiGated  64 gate rows and the 64 up rows of the same outputs per tile:
//              out = act(g) * u, and g, u kept on request
//   kEpiDgate  D = dh: dg, du and h from the kept g and u (A read rows-innermost)
//   LORA       kEpiStore over K and the adapters' K range (ftm_lora.cuh); the
//              slices are shared out over the cluster's ranks like K, by their
//              place in the tile's list of adapters (a token's last bits may
//              depend on which adapters its tile holds, never on their values)
//
// Without LORA, shared memory stays under half an SM's for BN <= 64, so that the
// next launch of the chain may move in early and load its weights while this one
// drains.  With LORA (136 to 194 KB) registers (two blocks' share; 103 a thread
// for 128 tokens) and shared memory let a block in beside one of the shrink's, to
// run over x and W while v is computed: 256 tokens of 256 requests, 6144 to 2048
// at rank 64, 36.0 -> 34.3 us.
#pragma once

#include "ftm_dense.cuh"

namespace ftm {

struct ProjArgs {
  CUtensorMap a, x;        // weights (boxes of 64 rows x 64 deep, either majorness), tokens {K, T}
  int T, M, kb;            // tokens, outputs, 64-deep blocks
  int a_mn;                // A stored rows-innermost
  int up_row0;             // gated: first up row of A
  int act, keep;
  int early;               // the launch before is this call's own, and waited: 1: A may be read before it ends, 2: X too
  uint16_t* out;           // [T][ld]
  int64_t ld;
  uint16_t* pre;           // gated: g, u [T][2M] when kept; dgate: read
  uint16_t* h;             // dgate: [T][M] when kept
  LoraArgs lora;
};

template <int BN, bool LORA>
struct ProjShape {
  static constexpr uint32_t kBBytes = ((BN * 128 + 1023) / 1024) * 1024;
  static constexpr uint32_t kStage = kATileBytes + kBBytes;
  static constexpr int kStages = BN == 16 ? 5 : BN == 32 ? 4 : 3;
  // adapter slices per message; two for 128 tokens, whose shared memory leaves room for a block of the shrink then
  static constexpr int kGroup = BN == 128 ? 2 : 4;
  static constexpr uint32_t kBuf = LORA ? 128 * 32 + BN * 32 : 0;      // a slice of B[a] and one of v
  static constexpr uint32_t kRed = BN * 512 + 8 * 64;                  // partial sums of every rank, each rounded up
  static constexpr uint32_t kTmemCols = BN < 32 ? 32 : BN;
  // warp 0 TMA, warp 1 MMA, then the warps that drain the accumulator and write the outputs, the first four also the
  // adapters' feed.  Sixteen for 128 tokens, a quadrant's four with 32 columns each: there the drain and the outputs
  // take longer than the MMAs (on four warps 333 tokens x 768 outputs, 2048 deep, 1.8 us of MMAs, 2 and 2; a training
  // step of 333 tokens 41.3 us, 40.1 on eight, 37.6 on sixteen).  Eight of them with LORA (200 tokens, 2048 to 2048,
  // 13.8 -> 13.2 us), whose registers still let a block of the shrink in.  Not for 64 tokens: a second block moves in
  // there (50 tokens, 4096 x 2048, on eight: 61 -> 66 us).
  static constexpr int kDrain = BN == 128 ? (LORA ? 8 : 16) : 4;
  static constexpr int kBlocks = LORA && BN < 128 ? 2 : 1;             // that registers are held to
  static constexpr int kThreads = 64 + 32 * kDrain;
  static constexpr size_t kSmem = 1024 + static_cast<size_t>(kStages) * kStage + kLoraRing * kGroup * kBuf + kRed;
  static constexpr int kPerSm = 2 * (kSmem + 2048) <= 228 * 1024 ? 2 : 1;   // blocks that shared memory lets in
  static_assert(LORA || BN > 64 || kPerSm == 2, "the next launch moves in beside this one");
};

__device__ __forceinline__ void st_cluster_f32x4(uint32_t addr, const float* f) {
  st_cluster_v4(addr, f[0], f[1], f[2], f[3]);
}

template <int EPI, int BN, bool LORA>
__global__ void __launch_bounds__(ProjShape<BN, LORA>::kThreads, ProjShape<BN, LORA>::kBlocks)
    proj_kernel(const __grid_constant__ ProjArgs a) {
  using S = ProjShape<BN, LORA>;
  constexpr int kProjThreads = S::kThreads;
  constexpr uint32_t kIdesc = idesc_bf16_f32(128, BN);
  constexpr int kRows = EPI == kEpiGated ? 64 : 128;      // outputs per tile
  constexpr int kPairs = kRows / 2;                       // pieces (2 outputs, 4 tokens) of 4 tokens
  constexpr int kParts = EPI == kEpiGated ? 2 : 1;        // gate and up values of a piece

  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[S::kStages], empty_bar[S::kStages], tfull_bar, count_bar;
  __shared__ uint32_t tmem_holder, messages;
  __shared__ LoraShared<LORA> ls;

  const uint32_t smem_base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (smem_base - smem_u32(smem_raw));
  uint8_t* ext = smem + static_cast<size_t>(S::kStages) * S::kStage;
  uint8_t* red = ext + kLoraRing * S::kGroup * S::kBuf;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int ks = static_cast<int>(cluster_nranks()), kr = static_cast<int>(cluster_rank());
  const int n0 = blockIdx.y * BN, w0 = blockIdx.z * kRows;
  const int valid = min(BN, a.T - n0);
  const int kb0 = kr * a.kb / ks, kb1 = (kr + 1) * a.kb / ks;
  // pieces of the tile, `share` of them summed by each rank; a piece is 32 bytes: [output][token]
  const int pieces = (valid + 3) / 4 * kPairs, share = (pieces + ks - 1) / ks;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) { mbar_init(&full_bar[s], 1); mbar_init(&empty_bar[s], 1); }
    mbar_init(&tfull_bar, 1);
    mbar_init(&count_bar, 1);
    if constexpr (LORA) ls.init(1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_holder, S::kTmemCols);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) { tma_prefetch_desc(&a.a); tma_prefetch_desc(&a.x); }
  tc_fence_before();
  if (ks > 1) cluster_sync_all();       // every rank's shared memory may be written from here on
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = tmem_holder;

  if (warp == 0) {
    if (lane == 0) {
      auto load_a = [&](int kb, int stage) {
        uint8_t* sa = smem + static_cast<size_t>(stage) * S::kStage;
        const int r1 = EPI == kEpiGated ? a.up_row0 + w0 : w0 + 64;
        if (a.a_mn) {
          tma_load_2d(sa, &a.a, &full_bar[stage], w0, kb * 64);
          tma_load_2d(sa + 8192, &a.a, &full_bar[stage], r1, kb * 64);
        } else {
          tma_load_2d(sa, &a.a, &full_bar[stage], kb * 64, w0);
          tma_load_2d(sa + 8192, &a.a, &full_bar[stage], kb * 64, r1);
        }
      };
      // The launch before waited for everything earlier before it let this one
      // start, and does not write A: the first stages' weights need no wait.
      // (LORA: nor does the shrink write x.)
      int ahead = 0;
      if (a.early)
        for (; ahead < S::kStages && kb0 + ahead < kb1; ++ahead) {
          mbar_arrive_expect_tx(&full_bar[ahead], kATileBytes + BN * 128);
          load_a(kb0 + ahead, ahead);
        }
      if (!LORA) {
        if (a.early < 2) pdl_wait();
        pdl_trigger();
      }
      int stage = 0;
      uint32_t phase = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (kb - kb0 >= ahead) {
          if (!mbar_wait(&empty_bar[stage], phase ^ 1u)) break;
          mbar_arrive_expect_tx(&full_bar[stage], kATileBytes + BN * 128);
          load_a(kb, stage);
        }
        tma_load_2d(smem + static_cast<size_t>(stage) * S::kStage + kATileBytes, &a.x, &full_bar[stage], kb * 64, n0);
        if (++stage == S::kStages) { stage = 0; phase ^= 1u; }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      // the bounded waits begin when what they wait for may: not while an earlier launch still runs
      if (!LORA && a.early < 2) pdl_wait();
      const bool amn = a.a_mn;
      const uint32_t idesc = kIdesc | (amn ? 1u << 15 : 0u);
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(&full_bar[stage], phase)) { ok = false; break; }
        tc_fence_after();
        const uint32_t sa = smem_u32(smem + static_cast<size_t>(stage) * S::kStage);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_f16(tmem_base, amn ? smem_desc_mn_sw128(sa + kk * 2048) : smem_desc_sw128(sa + kk * 32),
                   smem_desc_sw128(sa + kATileBytes + kk * 32), idesc, kb != kb0 || kk != 0 ? 1u : 0u);
        umma_commit(&empty_bar[stage]);
        if (++stage == S::kStages) { stage = 0; phase ^= 1u; }
      }
      if constexpr (LORA) {
        ok = ok && mbar_wait(&count_bar, 0);
        const uint32_t cnt = ok ? messages : 0;
        for (uint32_t c = 0; c < cnt; ++c) {
          const uint32_t slot = c % kLoraRing;
          if (!mbar_wait_cl(&ls.full[slot], (c / kLoraRing) & 1u)) { ok = false; break; }
          tc_fence_after();
          const uint32_t n = ls.msg[slot];
          for (uint32_t s = 0; s < n; ++s) {
            const uint32_t sb = smem_u32(ext + (slot * S::kGroup + s) * S::kBuf);
            umma_f16(tmem_base, smem_desc_k32(sb), smem_desc_k32(sb + 128 * 32), kIdesc, 1u);
          }
          umma_commit(&ls.empty[slot]);
        }
      }
      if (ok) umma_commit(&tfull_bar);
    }
    __syncwarp();
  } else {
    bool ok = true;
    if (!LORA && a.early < 2) pdl_wait();
    if constexpr (LORA) {
      if (warp < 6) {
        const int e = threadIdx.x - 64;
        const int i0 = e < BN ? lora_id<true>(a.lora.ids, a.T, a.lora.n, n0 + e) : -1;
        int at;
        const int nl = lora_list<128>(ls, e, i0, -1, 0, at);
        if (e == 0) {
          messages = lora_messages(nl, a.lora.rp, S::kGroup, kr, ks);
          mbar_arrive(&count_bar);
        }
        LoraRing ring;
        auto ready = [] { pdl_wait(); pdl_trigger(); };
        auto send = [&](uint32_t slot, uint32_t n, bool, bool bad) {
          ls.msg[slot] = n;
          if (bad)      // every rank's epilogue looks at its own flag
            for (int r = 0; r < ks; ++r)
              asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_rank(smem_u32(&ls.poison[0]), r)), "r"(kLoraPoison)
                           : "memory");
          mbar_arrive(&ls.full[slot]);
        };
        ok = lora_feed<BN, 128, S::kGroup>(a.lora, ls, ring, ext, 128 * 32, 0, S::kBuf, e, nl, kr, ks, n0 + e,
                                           i0 >= 0 ? at : -1, w0, ready, send);
      }
    }
    // this rank's partial sums to the ranks that own them: lane = weight row, TMEM column = token
    const int q = warp % 4, er = q * 32 + lane;
    ok = ok && mbar_wait(&tfull_bar, 0);
    if (__all_sync(0xffffffffu, ok)) {
      tc_fence_after();
      const uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
      // piece (tokens 4 g .. 4 g + 3, outputs of this row's pair): its owner and its place there
      const uint32_t mine = smem_u32(red) + (kr * kParts + er / kRows) * share * 32 + (er & 1) * 16;
      constexpr int kStep = BN < 32 ? BN : 32, kTurns = S::kDrain / 4;
      const int turn = (warp - 2) / 4;
      int local = (er % kRows) / 2 + turn * (kStep / 4) * kPairs, owner = 0;
#pragma unroll 1
      for (int c0 = turn * kStep; c0 < valid; c0 += kTurns * kStep) {
        float f[kStep];
#pragma unroll
        for (int j = 0; j < kStep; j += 16) tmem_ld16(tb + c0 + j, f + j);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < kStep; j += 4) {
          if (c0 + j < valid) {
            while (local >= share) { local -= share; ++owner; }
            st_cluster_f32x4(mapa_rank(mine + local * 32, owner), f + j);
            local += kPairs;
          }
        }
        local += (kTurns - 1) * (kStep / 4) * kPairs;
      }
    }
  }
  // This thread's pieces, and for the activation's gradient the g and u of the first two, asked for ahead of
  // the exchange (their latency was 4 us of a 15 us launch).
  auto place = [&](int i, int& t0, int& m) {
    const int piece = kr * share + i;
    t0 = n0 + piece / kPairs * 4;
    m = w0 + piece % kPairs * 2;
    return i < share && piece < pieces && m < a.M;
  };
  constexpr int kAhead = EPI == kEpiDgate ? 2 : 1;
  uint32_t kept[kAhead][4][2];
  if (EPI == kEpiDgate) {
    pdl_wait();                         // over since the loads began; every thread that reads `pre` asks for itself
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      int t0, m;
      const bool in = place(threadIdx.x + k * kProjThreads, t0, m);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint16_t* p = a.pre + static_cast<size_t>(t0 + j) * (2 * static_cast<size_t>(a.M)) + m;
        const bool on = in && t0 + j < a.T;
        kept[k][j][0] = on ? __ldg(reinterpret_cast<const uint32_t*>(p)) : 0u;
        kept[k][j][1] = on ? __ldg(reinterpret_cast<const uint32_t*>(p + a.M)) : 0u;
      }
    }
  }
  tc_fence_before();
  __syncwarp();
  if (ks > 1) cluster_sync_all();       // all partial sums and flags are in place
  else __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, S::kTmemCols);

  if (!LORA) pdl_wait();                // this launch's end stands for the end of the one before
  bool poison = false;
  if constexpr (LORA) poison = ls.poison[0] != 0;
  auto finish = [&](int i, const uint32_t (*z)[2]) {
    int t0, m;
    if (!place(i, t0, m)) return;
    auto sum = [&](int part, float* f) {       // f[output * 4 + token]
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = 0.f;
      for (int r = 0; r < ks; ++r) {
        const float4* p = reinterpret_cast<const float4*>(red + ((r * kParts + part) * share + i) * 32);
        const float4 u = p[0], v = p[1];
        f[0] += u.x; f[1] += u.y; f[2] += u.z; f[3] += u.w;
        f[4] += v.x; f[5] += v.y; f[6] += v.z; f[7] += v.w;
      }
    };
    float f[8], u[8];
    sum(0, f);
    if (EPI == kEpiGated) sum(1, u);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int t = t0 + j;
      if (t >= a.T) break;
      float v0 = f[j], v1 = f[4 + j];
      uint16_t* o = a.out + t * a.ld + m;
      uint16_t* p = a.pre + static_cast<size_t>(t) * (2 * static_cast<size_t>(a.M)) + m;
      if constexpr (EPI == kEpiStore) {
        if constexpr (LORA) {
          if (poison) {
            v0 += lora_nonfinite_term(a.lora, t, m);
            v1 += lora_nonfinite_term(a.lora, t, m + 1);
          }
        }
        *reinterpret_cast<uint32_t*>(o) = pack_bf16(v0, v1);
      } else if constexpr (EPI == kEpiGated) {
        const float u0 = u[j], u1 = u[4 + j];
        *reinterpret_cast<uint32_t*>(o) = pack_bf16(act_value(v0, a.act) * u0, act_value(v1, a.act) * u1);
        if (a.keep) {
          *reinterpret_cast<uint32_t*>(p) = pack_bf16(v0, v1);
          *reinterpret_cast<uint32_t*>(p + a.M) = pack_bf16(u0, u1);
        }
      } else {
        const uint32_t gw = z ? z[j][0] : __ldg(reinterpret_cast<const uint32_t*>(p));
        const uint32_t uw = z ? z[j][1] : __ldg(reinterpret_cast<const uint32_t*>(p + a.M));
        float dg0, dg1, du0, du1, h0, h1;
        act_gradient(__uint_as_float(gw << 16), __uint_as_float(uw << 16), v0, a.act, dg0, du0, h0);
        act_gradient(__uint_as_float(gw & 0xffff0000u), __uint_as_float(uw & 0xffff0000u), v1, a.act, dg1, du1, h1);
        *reinterpret_cast<uint32_t*>(o) = pack_bf16(dg0, dg1);
        *reinterpret_cast<uint32_t*>(o + a.M) = pack_bf16(du0, du1);
        if (a.keep) *reinterpret_cast<uint32_t*>(a.h + static_cast<size_t>(t) * a.M + m) = pack_bf16(h0, h1);
      }
    }
  };
  int i = threadIdx.x;
  if constexpr (EPI == kEpiDgate) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k, i += kProjThreads) finish(i, kept[k]);
  }
  for (; i < share; i += kProjThreads) finish(i, nullptr);
}

// ---- host ------------------------------------------------------------------------

template <int EPI, int BN, bool LORA>
cudaError_t launch_proj_bn(const ProjArgs& a, cudaStream_t st) {
  using S = ProjShape<BN, LORA>;
  const int mt = (a.M + (EPI == kEpiGated ? 63 : 127)) / (EPI == kEpiGated ? 64 : 128), nt = (a.T + BN - 1) / BN;
  const long tiles = static_cast<long>(mt) * nt;
  auto kern = proj_kernel<EPI, BN, LORA>;
  cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(S::kSmem));
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(S::kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // The widest split whose clusters all run at once: a second wave doubles the
  // time, and clusters do not fill every GPC (15 of 8 CTAs on 148 SMs at one
  // CTA per SM, which is what the query reports).
  struct Fit { int n[9]; };
  static const Fit fit = [&] {
    Fit f = {};
    for (int c = 2; c <= 8; ++c) {
      attr[0].val.clusterDim.x = c;
      cfg.gridDim = dim3(num_sms() / c * c);
      if (cudaOccupancyMaxActiveClusters(&f.n[c], kern, &cfg) != cudaSuccess) f.n[c] = 0;
    }
    (void)cudaGetLastError();
    return f;
  }();
  int ks = 1;
  for (int c = 2; c <= 8 && c <= a.kb && c * tiles <= num_sms(); ++c)
    if (tiles <= S::kPerSm * fit.n[c]) ks = c;
  cfg.gridDim = dim3(ks, nt, mt);
  attr[0].val.clusterDim.x = ks;
  cfg.numAttrs = 2;
  return count_launch(cudaLaunchKernelEx(&cfg, kern, a));
}

// Token tile: the smallest that holds all tokens, 128 beyond.
inline int proj_tile(int T) { return T <= 16 ? 16 : T <= 32 ? 32 : T <= 64 ? 64 : 128; }

template <int EPI, bool LORA>
cudaError_t launch_proj(const ProjArgs& a, cudaStream_t st) {
  switch (proj_tile(a.T)) {
    case 16: return launch_proj_bn<EPI, 16, LORA>(a, st);
    case 32: return launch_proj_bn<EPI, 32, LORA>(a, st);
    case 64: return launch_proj_bn<EPI, 64, LORA>(a, st);
    default: return launch_proj_bn<EPI, 128, LORA>(a, st);
  }
}

// Whether a product of T tokens and M outputs (`rows` of them to a tile), K
// deep, runs here: while its tiles leave room for a split over at least two CTAs
// each, and up to one a CTA where K is short.  Beyond, the pair engine does four
// times the products in an MMA of the same time and reads half as much from L2
// for each: 512 tokens x 4096 outputs x 4096 take 45 us here, 33 there; 200 x 4096
// x 2048 takes 10 here, 12 there.  Between one and two tiles for two CTAs, whole
// calls: gated blocks of 700 tokens, 2048 x 1024, 25.1 here, 27.0 there; 1000,
// 1024 x 768, 17.0 and 19.4; 300, 4096 x 2048, 43.8 and 36.7; with adapters (which
// four warps feed and drain) 700 tokens, 2048 to 2048, 28.1 and 26.8.  Measured up
// to widths of 4096: beyond, few tokens leave this engine while most of a tile there
// is padding (32 tokens, gate/up 2176 x 5120, 20 us there for 6.8 us of bytes).
inline bool proj_fits(int T, int M, int rows, int K, bool lora = false) {
  const int bn = proj_tile(T);
  const long tiles = static_cast<long>((M + rows - 1) / rows) * ((T + bn - 1) / bn);
  return tiles <= num_sms() / 2 || (!lora && K <= 2048 && tiles <= num_sms());
}

// Maps of the weights [w_rows][K] (a_mn: stored [K][w_rows]) and the tokens [T][K].
inline bool proj_maps(ProjArgs& a, const void* w, bool a_mn, uint64_t w_rows, uint64_t K, uint64_t w_pitch,
                      const void* x, uint64_t x_pitch) {
  a.a_mn = a_mn;
  a.kb = static_cast<int>((K + 63) / 64);
  return dense_operand_map(&a.a, w, a_mn, w_rows, K, w_pitch, 64) &&
         dense_operand_map(&a.x, x, false, a.T, K, x_pitch, proj_tile(a.T));
}

}  // namespace ftm
