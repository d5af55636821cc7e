// The dense (ungrouped) bf16 GEMM engine on CTA pairs: D = A B^T over tiles of
// 256 rows x 256 columns, one tile per pair of CTAs (tcgen05 cta_group::2).
// Narrower tiles do not pay: an MMA of 128 accumulator columns takes as long as
// one of 256 (a 4096 x 4096 x 2048 product took 1.9x as long in 256 x 128 tiles).
// Rows (tokens, or the rows of a weight gradient) are on the MMA's M side, so
// that a thread of the epilogue owns one row and consecutive columns: the
// gate/up pairing, the activation's gradient and the stores need no exchange
// between threads.  Either operand may be stored with its depth innermost
// (K-major: activations and weights of a forward product) or with its rows
// innermost (MN-major: what a transposed product reads), which is a choice of
// tensor-map box and matrix descriptor, never a transposing copy:
//   K-major  stage tile: [rows][64 deep], one box {64 deep, rows}
//   MN-major stage tile: boxes {64 rows, 64 deep}, 8 KB each, one per 64 rows
// A launch takes up to three products ("problems"), so the independent
// products of a backward pass fill the GPU together.  A single product of few
// tiles is split along K over the 2 to 4 pairs of a cluster (SPLIT): each pair
// sums its share of the depth, hands the columns that another pair owns to it
// through shared memory, and finishes its own, adding in pair order.
//
// Roles: warp 0 issues the TMA loads, warp 1 of the even CTA the MMAs, warps
// 2-5 (or 2-9) drain the accumulators (double-buffered in all 512 columns of
// TMEM) through swizzled staging rows and TMA stores, which clip the ragged
// rows and columns.  With LORA, warps 6-9 feed the adapters' K range (see
// ftm_lora.cuh).  No TMA multicast.
#pragma once

#include "ftm_gemm.cuh"
#include "ftm_lora.cuh"

namespace ftm {

constexpr int kDTileM = 256;                   // rows per tile (128 per CTA)
constexpr int kDTileN = 256;                   // accumulator columns per tile
constexpr int kDBK = 64;                       // depth per stage
constexpr uint32_t kDABytes = 128 * 128;       // 128 rows x 64 deep of bf16 per CTA
constexpr int kDSlotBytes = 32 * 128;          // one warp's staging slot: 32 rows x 64 columns of bf16
constexpr int kDHalfBytes = 32 * 64;           // the epilogues with several tensors: 32 rows x 32 columns each
constexpr int kDProblems = 3;

enum DenseEpi {
  kEpiStore = 0,   // c0 = D
  kEpiGated = 1,   // D holds gate and up columns: c0 = act(g) * u; c1 = g, c2 = u when kept
  kEpiDgate = 2    // D = dh: c0 = dg, c1 = du, c2 = h, from the kept g and u
};

struct DenseProblem {
  CUtensorMap a, b, c0, c1, c2, p0, p1;      // operands, outputs; dgate: the kept g and u
  int M, N;          // rows, output columns (gated: columns of h)
  int nt;            // column tiles
  int kb;            // 64-deep blocks
  int tiles;
  int a_mn, b_mn;    // operand stored rows-innermost
  int up_row0;       // gated: row of B where the up projection starts
};

struct DenseArgs {
  DenseProblem p[kDProblems];
  int n;             // problems, deepest first
  int early;         // the launches since the operands were written are this call's own, and waited: do not wait again
  int act;           // ftm_act
  int keep;          // gated: store g and u; dgate: store h
  // tile schedule (see dense_tile_at)
  int n_long, n_short, short_extra;
  LoraArgs lora;
};

// ---- descriptors ---------------------------------------------------------------
// MN-major operand, 128-byte swizzle: atoms of 64 rows (128 bytes) x 8 deep, the
// next 8 deep 1024 bytes on, the next 64 rows one box (8 KB) on.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(8192u >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* m, const void* src, int32_t c0, int32_t c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(smem_u32(src)), "r"(c0), "r"(c1)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// One row's 32 columns into half (0: columns 0-31, 1: 32-63) of a staging slot
// in the layout the 128-byte-swizzled store map reads.
__device__ __forceinline__ void stage_half(uint8_t* slot, int row, int half, const uint32_t* w) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int chunk = (half * 4 + c) ^ (row & 7);
    *reinterpret_cast<uint4*>(slot + row * 128 + chunk * 16) = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
  }
}

// One row's 32 columns in a half slot, whose maps swizzle over 64 bytes.
__device__ __forceinline__ uint4* half_piece(uint8_t* slot, int row, int c) {
  return reinterpret_cast<uint4*>(slot + row * 64 + ((c ^ ((row >> 1) & 3)) << 4));
}
__device__ __forceinline__ void stage_row(uint8_t* slot, int row, const uint32_t* w) {
#pragma unroll
  for (int c = 0; c < 4; ++c) *half_piece(slot, row, c) = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
}

// ---- tile schedule ---------------------------------------------------------------
// The pair's i-th tile, or -1.  Tiles [0, n_long) have the deepest K and go
// round the pairs first; a pair that got one fewer takes short_extra shallow
// tiles in its place, and the rest go round from the last pair down.  All from
// sizes: the assignment never depends on timing.
__device__ __forceinline__ int dense_tile_at(const DenseArgs& g, int pair, int np, int i) {
  const int rem = g.n_long % np;
  const int mine = g.n_long / np + (pair < rem ? 1 : 0);
  if (i < mine) return pair + i * np;
  i -= mine;
  const int room = np - rem;
  const int s1 = rem ? min(g.n_short, g.short_extra * room) : 0;
  if (pair >= rem && s1) {
    const int first = pair - rem;
    const int have = first < s1 ? (s1 - first - 1) / room + 1 : 0;
    if (i < have) return g.n_long + first + i * room;
    i -= have;
  }
  const int s = s1 + (np - 1 - pair) + i * np;
  return s < g.n_short ? g.n_long + s : -1;
}

struct DenseTile {
  int p, m, n;
};

// Tiles of a problem run down bands of 8 row tiles, so that the tiles in
// flight share both operands' blocks in L2.
__device__ __forceinline__ DenseTile dense_decode(const DenseArgs& g, int t) {
  int p = 0;
  while (p + 1 < g.n && t >= g.p[p].tiles) { t -= g.p[p].tiles; ++p; }
  const int nt = g.p[p].nt, mt = g.p[p].tiles / nt;
  const int band = t / (8 * nt);
  const int rows = min(8, mt - band * 8);
  const int in = t - band * 8 * nt;
  DenseTile d;
  d.p = p;
  d.m = band * 8 + in % rows;
  d.n = in / rows;
  return d;
}

// Epilogue warps and their staging.  kEpiStore: four warps, two slots each in
// turn.  The others, whose arithmetic takes as long as a shallow product's MMAs
// (with four warps the activation gradient took 18 us a tile at 640 deep, a
// product of 4 us), run eight, two to a quadrant of rows with every other chunk
// of 32 columns: kEpiGated one set of three half slots (h, g, u); kEpiDgate two
// sets in turn, into which g and u are loaded a chunk ahead and which dg, du and
// h leave from.
template <int EPI, bool LORA>
struct DenseShape {
  static constexpr uint32_t kStage = 2 * kDABytes;                 // 128 rows of A and 128 of B, 64 deep
  static constexpr int kEpiWarps = EPI == kEpiStore ? 4 : 8;
  static constexpr uint32_t kWarpStaging = EPI == kEpiStore ? 2 * kDSlotBytes : (EPI == kEpiGated ? 3 : 6) * kDHalfBytes;
  static constexpr uint32_t kStaging = kEpiWarps * kWarpStaging;
  static constexpr int kGroup = 4;                                 // adapter slices per message
  static constexpr uint32_t kBuf = 2 * 128 * 32;                   // a slice of v and one of B[a]
  static constexpr uint32_t kExt = LORA ? kLoraRing * kGroup * kBuf : 0;
  static constexpr int kStages = EPI == kEpiDgate || LORA ? 4 : 5;
  static constexpr size_t kSmem = 1024 + static_cast<size_t>(kStages) * kStage + kStaging + kExt;
  static constexpr int kThreads = 64 + 32 * kEpiWarps + (LORA ? 128 : 0);
};

// 32 accumulator columns of this thread's row.
__device__ __forceinline__ void tmem_ld32(uint32_t t, float* v) {
  tmem_ld16(t, v);
  tmem_ld16(t + 16, v + 16);
}

// SPLIT: the pair that finishes the 32 accumulator columns of chunk c (0 to 7),
// in units of what is finished together: two neighbouring chunks, a gate chunk
// and its up chunk, or one.  And where another pair finds room for its sums of
// them in the owner's idle ring: [pair][the owner's chunks][4 columns][row].
template <int EPI>
struct SplitUnits {
  static constexpr int kUnits = EPI == kEpiDgate ? 8 : 4, kPer = 8 / kUnits;
  static __device__ __forceinline__ int unit(int c) { return EPI == kEpiStore ? c >> 1 : EPI == kEpiGated ? c & 3 : c; }
  static __device__ __forceinline__ int owner(int c, int ks) { return unit(c) * ks / kUnits; }
  static __device__ __forceinline__ uint32_t place(int c, int from, int own, int ks) {
    const int base = (own * kUnits + ks - 1) / ks, stride = kPer * ((kUnits + ks - 1) / ks);
    const int at = (unit(c) - base) * kPer + (EPI == kEpiStore ? c & 1 : EPI == kEpiGated ? c >> 2 : 0);
    return ((from - (from > own ? 1 : 0)) * stride + at) * (128 * 32 * 4);
  }
};

template <int EPI, bool LORA, bool SPLIT>
__global__ void __launch_bounds__(DenseShape<EPI, LORA>::kThreads, 1)
    dense_kernel(const __grid_constant__ DenseArgs g) {
  using S = DenseShape<EPI, LORA>;
  constexpr int BN = kDTileN;
  constexpr int kStages = S::kStages;
  constexpr uint32_t kTmemCols = 2 * BN;
  constexpr int kOutCols = EPI == kEpiGated ? BN / 2 : BN;   // output columns per tile

  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[kStages], empty_bar[kStages], tfull_bar[2], tempty_bar[2];
  __shared__ __align__(8) uint64_t pre_bar[EPI == kEpiDgate ? 16 : 1];     // [warp][set]: g and u of a chunk
  __shared__ uint32_t tmem_holder;
  __shared__ LoraShared<LORA> ls;

  const uint32_t smem_base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (smem_base - smem_u32(smem_raw));
  uint8_t* staging = smem + static_cast<size_t>(kStages) * S::kStage;
  uint8_t* ext = staging + S::kStaging;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t crank = cluster_rank();
  const uint32_t even = crank & ~1u;                         // the pair's even CTA: its barriers count for both
  const uint32_t rank = crank & 1u;
  const bool leader = rank == 0;
  const int ks = SPLIT ? static_cast<int>(cluster_nranks()) / 2 : 1, kr = static_cast<int>(crank) / 2;
  const int np = gridDim.x / (2 * ks), pair = blockIdx.x / (2 * ks);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) { mbar_init(&full_bar[s], 1); mbar_init(&empty_bar[s], 1); }
    for (int a = 0; a < 2; ++a) { mbar_init(&tfull_bar[a], LORA ? 2 : 1); mbar_init(&tempty_bar[a], 2 * S::kEpiWarps); }
    if (EPI == kEpiDgate)
      for (int i = 0; i < 16; ++i) mbar_init(&pre_bar[i], 1);
    if constexpr (LORA) ls.init();
    fence_mbar_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_holder)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  if (warp == 0 && lane == 0) {
    for (int p = 0; p < g.n; ++p) { tma_prefetch_desc(&g.p[p].a); tma_prefetch_desc(&g.p[p].b); }
  }
  // LORA: the launch before is always the shrink, which waited for everything
  // earlier before it let this one start: x and W are final, only v is waited
  // for, by the warps that feed it.  Pairs on SMs that the shrink leaves idle
  // (the first pairs, which have the most tiles) start at once.
  if (!LORA) {
    if (!g.early) pdl_wait();
    pdl_trigger();
  }
  tc_fence_before();
  cluster_sync_all();     // barriers initialised and TMEM allocated in every CTA
  tc_fence_after();
  const uint32_t tmem_base = tmem_holder;

  const int q = warp % 4;                                // TMEM lane quadrant of an epilogue warp
  uint8_t* slots = staging + (warp >= 2 ? warp - 2 : 0) * S::kWarpStaging;
  constexpr int kCols = EPI == kEpiStore ? 64 : 32;      // columns of a chunk
  constexpr int kTurns = S::kEpiWarps / 4;               // warps that share a quadrant's chunks
  const int first = (warp - 2) / 4;
  uint32_t chunk = 0;                                    // chunks of this warp so far: slots and sets take turns
  uint64_t* pbar = pre_bar + (EPI == kEpiDgate && warp >= 2 ? (warp - 2) * 2 : 0);

  // The finishing of a tile by one epilogue warp: load(c, v) gives the 32 accumulator columns from c of the
  // thread's row; mine(cc): whether this pair finishes chunk cc; poison is valid after wait().  False when a
  // wait gave up.
  auto finish = [&](const DenseProblem& P, const DenseTile& ti, const bool& poison, auto wait, auto load,
                    auto mine) -> bool {
    const int row0 = ti.m * kDTileM + static_cast<int>(rank) * 128 + q * 32;   // this warp's 32 rows
    [[maybe_unused]] const int row = row0 + lane;
    const int col0 = ti.n * kOutCols;
    const int chunks = row0 < P.M ? (min(kOutCols, P.N - col0) + kCols - 1) / kCols : 0;
    auto next = [&](int cc) {
      while (SPLIT && cc < chunks && !mine(cc)) cc += kTurns;
      return cc;
    };
    auto ask = [&](int c, uint32_t n) {      // lane 0: g and u of the tile's chunk c into the set of this warp's n-th
      uint8_t* in = slots + (n & 1) * 3 * kDHalfBytes;
      mbar_arrive_expect_tx(&pbar[n & 1], 2 * kDHalfBytes);
      tma_load_2d(in, &P.p0, &pbar[n & 1], col0 + c * kCols, row0);
      tma_load_2d(in + kDHalfBytes, &P.p1, &pbar[n & 1], col0 + c * kCols, row0);
    };
    if (EPI == kEpiDgate && lane == 0 && next(first) < chunks) {
      bulk_wait_read<0>();
      ask(next(first), chunk);
    }
    bool ok = wait();
    if (!__all_sync(0xffffffffu, ok)) return false;
#pragma unroll 1
    for (int cc = next(first); cc < chunks; cc = next(cc + kTurns), ++chunk) {
      const int c0 = cc * kCols;
      if constexpr (EPI == kEpiStore) {
        if (lane == 0) bulk_wait_read<1>();    // the store before last has read its slot
        __syncwarp();
        uint8_t* s0 = slots + (chunk & 1) * kDSlotBytes;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const int c = c0 + hf * 32;
          float v[32];
          load(c, v);
          tmem_ld_wait();
          if constexpr (LORA) {
            if (poison && row < P.M) {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (col0 + c + j < P.N) v[j] += lora_nonfinite_term(g.lora, row, col0 + c + j);
            }
          }
          uint32_t w[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) w[j] = pack_bf16(v[2 * j], v[2 * j + 1]);
          stage_half(s0, lane, hf, w);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(&P.c0, s0, col0 + c0, row0);
          bulk_commit();
        }
      } else {
        uint8_t* set = slots + (EPI == kEpiDgate ? (chunk & 1) * 3 * kDHalfBytes : 0);
        float v[32];
        load(c0, v);
        uint32_t w0[16], w1[16], w2[16];
        if constexpr (EPI == kEpiGated) {
          float u[32];
          load(BN / 2 + c0, u);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            w1[j] = pack_bf16(v[2 * j], v[2 * j + 1]);
            w2[j] = pack_bf16(u[2 * j], u[2 * j + 1]);
            w0[j] = pack_bf16(act_value(v[2 * j], g.act) * u[2 * j], act_value(v[2 * j + 1], g.act) * u[2 * j + 1]);
          }
          if (lane == 0) bulk_wait_read<0>();  // the last chunk has left its slots
        } else {
          ok = mbar_wait(&pbar[chunk & 1], (chunk >> 1) & 1);
          if (!__all_sync(0xffffffffu, ok)) return false;
          uint4 gv[4], uv[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            gv[k] = *half_piece(set, lane, k);
            uv[k] = *half_piece(set + kDHalfBytes, lane, k);
          }
          tmem_ld_wait();
          const uint32_t* gw = reinterpret_cast<const uint32_t*>(gv);
          const uint32_t* uw = reinterpret_cast<const uint32_t*>(uv);
          if (lane == 0 && next(cc + kTurns) < chunks) {
            bulk_wait_read<0>();               // the last chunk has left the other set
            ask(next(cc + kTurns), chunk + 1);
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float dg[2], du[2], h[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float z = __uint_as_float(e ? gw[j] & 0xffff0000u : gw[j] << 16);
              const float u = __uint_as_float(e ? uw[j] & 0xffff0000u : uw[j] << 16);
              act_gradient(z, u, v[2 * j + e], g.act, dg[e], du[e], h[e]);
            }
            w0[j] = pack_bf16(dg[0], dg[1]);
            w1[j] = pack_bf16(du[0], du[1]);
            w2[j] = pack_bf16(h[0], h[1]);
          }
        }
        __syncwarp();                          // every lane has read its g and u; the slots are free
        stage_row(set, lane, w0);
        if (EPI == kEpiDgate || g.keep) stage_row(set + kDHalfBytes, lane, w1);
        if (g.keep) stage_row(set + 2 * kDHalfBytes, lane, w2);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(&P.c0, set, col0 + c0, row0);
          if (EPI == kEpiDgate || g.keep) tma_store_2d(&P.c1, set + kDHalfBytes, col0 + c0, row0);
          if (g.keep) tma_store_2d(&P.c2, set + 2 * kDHalfBytes, col0 + c0, row0);
          bulk_commit();
        }
      }
    }
    return true;
  };

  bool summed = true;     // SPLIT: an epilogue warp's accumulator is complete

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int i = 0, t; ok && (t = dense_tile_at(g, pair, np, i)) >= 0; ++i) {
        const DenseTile ti = dense_decode(g, t);
        const DenseProblem& P = g.p[ti.p];
        const int ar = ti.m * kDTileM + static_cast<int>(rank) * 128;
        // gated: the even CTA stages gate rows, the odd CTA the matching up rows
        const int br = EPI == kEpiGated ? ti.n * kOutCols + (leader ? 0 : P.up_row0)
                                        : ti.n * BN + static_cast<int>(rank) * (BN / 2);
        for (int kb = kr * P.kb / ks; kb < (kr + 1) * P.kb / ks; ++kb) {
          if (!mbar_wait_cl(&empty_bar[stage], phase ^ 1u)) { ok = false; break; }
          if (leader) mbar_arrive_expect_tx(&full_bar[stage], 2 * S::kStage);
          const uint32_t lbar = mapa_rank(smem_u32(&full_bar[stage]), even);
          uint8_t* sa = smem + static_cast<size_t>(stage) * S::kStage;
          uint8_t* sb = sa + kDABytes;
          const int kc = kb * kDBK;
          if (P.a_mn) {
            tma2_load_2d(sa, &P.a, lbar, ar, kc);
            tma2_load_2d(sa + 8192, &P.a, lbar, ar + 64, kc);
          } else {
            tma2_load_2d(sa, &P.a, lbar, kc, ar);
          }
          if (P.b_mn) {
            tma2_load_2d(sb, &P.b, lbar, br, kc);
            tma2_load_2d(sb + 8192, &P.b, lbar, br + 64, kc);
          } else {
            tma2_load_2d(sb, &P.b, lbar, kc, br);
          }
          if (++stage == kStages) { stage = 0; phase ^= 1u; }
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (leader && lane == 0) {
      int stage = 0, es = 0;
      uint32_t phase = 0, ephase = 0;
      bool ok = true;
      for (int i = 0, t; ok && (t = dense_tile_at(g, pair, np, i)) >= 0; ++i) {
        const DenseTile ti = dense_decode(g, t);
        const DenseProblem& P = g.p[ti.p];
        const int ab = i & 1;
        if (!mbar_wait_cl(&tempty_bar[ab], ((i >> 1) & 1) ^ 1u)) break;
        tc_fence_after();
        const uint32_t d = tmem_base + ab * BN;
        const bool amn = P.a_mn, bmn = P.b_mn;
        const uint32_t idesc = idesc_bf16_f32(256, BN) | (amn ? 1u << 15 : 0u) | (bmn ? 1u << 16 : 0u);
        // a 16-deep step: 32 bytes along a K-major row, 16 rows of 128 bytes of an MN-major box
        const uint32_t astep = amn ? 2048 : 32, bstep = bmn ? 2048 : 32;
        const int kb0 = kr * P.kb / ks, kb1 = (kr + 1) * P.kb / ks;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait_cl(&full_bar[stage], phase)) { ok = false; break; }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + static_cast<size_t>(stage) * S::kStage);
          const uint32_t sb = sa + kDABytes;
#pragma unroll
          for (int kk = 0; kk < kDBK / 16; ++kk) {
            const uint64_t da = amn ? smem_desc_mn_sw128(sa + kk * astep) : smem_desc_sw128(sa + kk * astep);
            const uint64_t db = bmn ? smem_desc_mn_sw128(sb + kk * bstep) : smem_desc_sw128(sb + kk * bstep);
            umma2_f16(d, da, db, idesc, kb != kb0 || kk != 0 ? 1u : 0u);
          }
          umma2_commit_pair(&empty_bar[stage], even);
          if (++stage == kStages) { stage = 0; phase ^= 1u; }
        }
        if constexpr (LORA) {
          // the adapters' K range, message by message until the tile's last
          uint32_t poison = 0;
          bool last = false;
          while (ok && !last) {
            if (!mbar_wait_cl(&ls.full[es], ephase)) { ok = false; break; }
            tc_fence_after();
            const uint32_t msg = ls.msg[es], n = msg & kLoraCount;
            last = (msg & kLoraLast) != 0;
            if (n) poison |= (msg | ls.msg_peer[es]) & kLoraPoison;
            for (uint32_t s = 0; s < n; ++s) {
              const uint32_t sv = smem_u32(ext + (es * S::kGroup + s) * S::kBuf);
              umma2_f16(d, smem_desc_k32(sv), smem_desc_k32(sv + 128 * 32), idesc_bf16_f32(256, BN), 1u);
            }
            umma2_commit_pair(&ls.empty[es], even);
            if (++es == kLoraRing) { es = 0; ephase ^= 1u; }
          }
          if (ok) {
            // The epilogue learns whether a slice held non-finite weights: that of both CTAs before they start on
            // the tile, or of the whole cluster (only ever set) before its barrier.
            if (!SPLIT || poison)
              for (uint32_t r = SPLIT ? 0 : even; r < (SPLIT ? 2 * ks : even + 2); ++r)
                asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_rank(smem_u32(&ls.poison[ab]), r)), "r"(poison)
                             : "memory");
            mbar_arrive(&tfull_bar[ab]);
            mbar_arrive_remote(mapa_rank(smem_u32(&tfull_bar[ab]), even + 1));
          }
        }
        if (ok) umma2_commit_pair(&tfull_bar[ab], even);
      }
    }
    __syncwarp();
  } else if (warp < 2 + S::kEpiWarps) {
    if constexpr (SPLIT) {
      summed = __all_sync(0xffffffffu, mbar_wait_cl(&tfull_bar[0], 0));
    } else {
      const uint32_t tempty0 = mapa_rank(smem_u32(&tempty_bar[0]), even);
      const uint32_t tempty1 = mapa_rank(smem_u32(&tempty_bar[1]), even);
      for (int i = 0, t; (t = dense_tile_at(g, pair, np, i)) >= 0; ++i) {
        const DenseTile ti = dense_decode(g, t);
        const int ab = i & 1;
        const uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + ab * BN;
        bool poison = false;
        auto wait = [&] {
          const bool ok = mbar_wait_cl(&tfull_bar[ab], (i >> 1) & 1);
          tc_fence_after();
          if constexpr (LORA) poison = ls.poison[ab] != 0;
          return ok;
        };
        if (!finish(g.p[ti.p], ti, poison, wait, [&](int c, float* v) { tmem_ld32(tb + c, v); }, [](int) { return true; }))
          break;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (leader) mbar_arrive(&tempty_bar[ab]);
          else mbar_arrive_remote(ab ? tempty1 : tempty0);
        }
      }
      if (lane == 0) bulk_wait_all();
      __syncwarp();
    }
  } else {
    if constexpr (LORA) {
      // one row of the tile per thread; both CTAs list the adapters of all 256 rows and feed the same slices,
      // each its own 128 rows of v and its own half of the output columns (SPLIT: every ks-th message)
      LoraRing ring;
      const LoraArgs& L = g.lora;
      const int e = threadIdx.x - 192;
      bool ok = true, waited = false;
      auto ready = [&] {
        if (!waited) { pdl_wait(); pdl_trigger(); }
        waited = true;
      };
      for (int i = 0, t; ok && (t = dense_tile_at(g, pair, np, i)) >= 0; ++i) {
        const DenseTile ti = dense_decode(g, t);
        const int m0 = ti.m * kDTileM;
        const int i0 = lora_id<true>(L.ids, L.T, L.n, m0 + e), i1 = lora_id<true>(L.ids, L.T, L.n, m0 + 128 + e);
        int at;
        const int nl = lora_list<256>(ls, e, i0, i1, static_cast<int>(rank), at);
        auto send = [&](uint32_t slot, uint32_t n, bool last, bool bad) {
          if (leader) {
            ls.msg[slot] = n | (last ? kLoraLast : 0u) | (bad ? kLoraPoison : 0u);
            mbar_arrive(&ls.full[slot]);
          } else {
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_rank(smem_u32(&ls.msg_peer[slot]), even)),
                         "r"(bad ? kLoraPoison : 0u)
                         : "memory");
            mbar_arrive_remote(mapa_rank(smem_u32(&ls.full[slot]), even));
          }
        };
        if (lora_messages(nl, L.rp, S::kGroup, kr, ks) == 0) {
          // no slice for this pair: one message without data
          ready();
          const uint32_t slot = ring.count % kLoraRing;
          ok = mbar_wait_cl(&ls.empty[slot], ((ring.count / kLoraRing) & 1u) ^ 1u);
          ok = feed_all(ok);
          if (ok && e == 0) {
            if (leader) {
              ls.msg[slot] = kLoraLast;
              mbar_arrive(&ls.full[slot]);
            } else {
              mbar_arrive_remote(mapa_rank(smem_u32(&ls.full[slot]), even));
            }
          }
          ring.count += 1;
          continue;
        }
        ok = lora_feed<128, BN / 2, S::kGroup>(L, ls, ring, ext, 0, 128 * 32, S::kBuf, e, nl, kr, ks,
                                               m0 + static_cast<int>(rank) * 128 + e, (leader ? i0 : i1) >= 0 ? at : -1,
                                               ti.n * BN + static_cast<int>(rank) * (BN / 2), ready, send);
      }
    }
  }

  if constexpr (SPLIT) {
    // one tile per cluster: the ring is idle once every pair has its sum
    const DenseTile ti = dense_decode(g, pair);
    const bool epi = warp >= 2 && warp < 2 + S::kEpiWarps;
    const uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
    const uint32_t mine_row = (q * 32 + lane) * 16;
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    if (epi && summed) {
#pragma unroll 1
      for (int c = first; c < BN / 32; c += kTurns) {
        const int owner = SplitUnits<EPI>::owner(c, ks);
        if (owner == kr) continue;
        float v[32];
        tmem_ld32(tb + c * 32, v);
        tmem_ld_wait();
        const uint32_t to = mapa_rank(smem_u32(smem) + SplitUnits<EPI>::place(c, kr, owner, ks) + mine_row, owner * 2 + rank);
#pragma unroll
        for (int j = 0; j < 8; ++j) st_cluster_v4(to + j * 2048, v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
      }
    }
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    if (epi && summed) {
      bool poison = false;
      if constexpr (LORA) poison = ls.poison[0] != 0;
      auto load = [&](int c, float* v) {       // the pairs' sums of 32 columns, added in their order
        float own[32];
        tmem_ld32(tb + c, own);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = 0.f;
        for (int r = 0; r < ks; ++r) {
          if (r == kr) {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] += own[j];
          } else {
            const uint8_t* at = smem + SplitUnits<EPI>::place(c / 32, r, kr, ks) + mine_row;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float4 u = *reinterpret_cast<const float4*>(at + j * 2048);
              v[4 * j] += u.x; v[4 * j + 1] += u.y; v[4 * j + 2] += u.z; v[4 * j + 3] += u.w;
            }
          }
        }
      };
      finish(g.p[ti.p], ti, poison, [] { return true; }, load,
             [&](int cc) { return SplitUnits<EPI>::owner(EPI == kEpiStore ? 2 * cc : cc, ks) == kr; });
      if (lane == 0) bulk_wait_all();
      __syncwarp();
    }
  }
  tc_fence_before();
  cluster_sync_all();     // no CTA leaves while its pair may still signal it
  tc_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(kTmemCols) : "memory");
  if (g.early) pdl_wait();     // this launch's end stands for the end of those before it
}

// ---- host ------------------------------------------------------------------------

// Operand map: K-major dims {K, rows}, box {64, box_rows}; MN-major dims {rows, K}, box {64, 64}.
inline bool dense_operand_map(CUtensorMap* m, const void* base, bool mn, uint64_t rows, uint64_t K, uint64_t pitch_bytes,
                              uint32_t box_rows) {
  return make_map_sw128(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, mn ? rows : K, mn ? K : rows, pitch_bytes, 0, 0,
                        mn ? 64 : box_rows);
}

// Store map of kEpiStore: dims {cols, rows}, box {64 columns, 32 rows}; clips what lies outside.
inline bool dense_store_map(CUtensorMap* m, void* base, uint64_t cols, uint64_t rows, uint64_t pitch_bytes) {
  return make_map_sw128(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, cols, rows, pitch_bytes, 0, 0, 32);
}

// Map of a half slot: box {32 columns, 32 rows}, 64-byte swizzle.
inline bool dense_half_map(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint64_t pitch_bytes) {
  const cuuint64_t dims[2] = {cols, rows}, strides[1] = {pitch_bytes};
  const cuuint32_t box[2] = {32, 32};
  return encode_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_64B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

// A problem's sizes: out_cols output columns per tile.
inline void dense_tiles(DenseProblem& P, int M, int N, int K, int out_cols) {
  P.M = M;
  P.N = N;
  P.kb = (K + kDBK - 1) / kDBK;
  P.nt = (N + out_cols - 1) / out_cols;
  P.tiles = (M + kDTileM - 1) / kDTileM * P.nt;
}

// Orders the problems by depth and sets the schedule.
inline void dense_schedule(DenseArgs& a) {
  for (int i = 1; i < a.n; ++i)
    for (int j = i; j > 0 && a.p[j].kb > a.p[j - 1].kb; --j) { DenseProblem t = a.p[j]; a.p[j] = a.p[j - 1]; a.p[j - 1] = t; }
  a.n_long = a.n_short = 0;
  int kshort = 1;
  for (int i = 0; i < a.n; ++i) {
    if (a.p[i].kb == a.p[0].kb) a.n_long += a.p[i].tiles;
    else { a.n_short += a.p[i].tiles; kshort = kshort > a.p[i].kb ? kshort : a.p[i].kb; }
  }
  a.short_extra = (a.p[0].kb + kshort / 2) / kshort;
}

template <int EPI, bool LORA, bool SPLIT>
cudaError_t launch_dense_split(DenseArgs& a, cudaStream_t st) {
  using S = DenseShape<EPI, LORA>;
  dense_schedule(a);
  auto kern = dense_kernel<EPI, LORA, SPLIT>;
  cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(S::kSmem));
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(S::kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // clusters of 1 to 4 pairs that run at once: as many as the GPCs can hold
  struct Fit { int n[5]; };
  static const Fit fit = [&] {
    Fit f = {};
    for (int c = 1; c <= 4; ++c) {
      attr[0].val.clusterDim.x = 2 * c;
      cfg.gridDim = dim3(num_sms() / (2 * c) * (2 * c));
      if (cudaOccupancyMaxActiveClusters(&f.n[c], kern, &cfg) != cudaSuccess) f.n[c] = 0;
    }
    (void)cudaGetLastError();
    if (f.n[1] <= 0 || f.n[1] > num_sms() / 2) f.n[1] = num_sms() / 2;
    return f;
  }();
  const int tiles = a.n_long + a.n_short;
  int ks = 1;
  if (SPLIT)
    for (int c = 2; c <= 4 && c <= a.p[a.n - 1].kb; ++c)
      if (tiles <= fit.n[c]) ks = c;
  attr[0].val.clusterDim.x = 2 * ks;
  cfg.gridDim = dim3(SPLIT ? 2 * ks * tiles : 2 * (tiles < fit.n[1] ? tiles : fit.n[1]));
  cfg.numAttrs = 2;
  return count_launch(cudaLaunchKernelEx(&cfg, kern, a));
}

// One product whose tiles leave half the pairs idle may be split along K, from 4
// blocks of 64 a pair (an exchange costs as much as 4 blocks).
template <int EPI, bool LORA>
cudaError_t launch_dense(DenseArgs& a, bool may_split, cudaStream_t st) {
  int tiles = 0, kb = 8;
  for (int i = 0; i < a.n; ++i) {
    tiles += a.p[i].tiles;
    kb = a.p[i].kb < kb ? a.p[i].kb : kb;
  }
  const bool split = may_split && tiles <= num_sms() / 4 && kb >= 8;
  return split ? launch_dense_split<EPI, LORA, true>(a, st) : launch_dense_split<EPI, LORA, false>(a, st);
}

}  // namespace ftm
