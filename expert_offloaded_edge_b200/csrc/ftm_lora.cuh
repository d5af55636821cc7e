// Low-rank adapters of many requests beside a shared projection (device parts).
//
//   y[t] = x[t] W^T + s[a] (x[t] A[a]^T) B[a]^T,   a = adapter id of token t
//
// The projection kernels run over K = d_in and then over an extra K range: for
// every adapter that occurs in the token tile, the products v B[a]^T with
// v = s (x A[a]^T) of that adapter's tokens and zeros for all others, added in
// the same accumulator.  So a tile may mix any requests, nothing is sorted, W
// is read once, and B[a] is read by the tiles that hold one of its tokens.  The
// extra range is fed in slices of 16 (one MMA deep), a few to a message, which
// four warps write to shared memory.
//
// A zero row does not mask an infinity or NaN of another request's adapter
// (0 * inf = NaN).  The feeding threads see every slice of B[a], so they put a
// tiny weight of the same sign in a non-finite one's place and flag the tile; the
// epilogue of a flagged tile adds the non-finite terms to the adapter's own tokens
// only.  (Tiny and not zero: an infinite v times it is the infinity that the term
// is; a finite v adds next to nothing to what will be infinite or NaN.)
#pragma once

#include "ftm_gemm.cuh"

namespace ftm {

constexpr int kLoraRing = 2;              // messages (groups of slices) in flight
// a message: slices in it (low bits, 0: none), and
constexpr uint32_t kLoraCount = 7, kLoraLast = 8, kLoraPoison = 16;

struct LoraArgs {
  const int32_t* ids;        // [T] adapter of each token, -1: none
  const uint16_t* v;         // [T][rp] bf16, s (x A^T); rows of tokens without an adapter are never read
  const uint16_t* b_pool;    // [adapters][d_out][rank]
  int T, n, rank, rp, d_out; // rp: rank rounded up to 16
};

// K-major operand slice, 16 deep: rows of 32 bytes, 32-byte swizzle (the two
// 16-byte halves of a row change places where bit 2 of the row is set), 8 rows = 256 bytes.
__device__ __forceinline__ uint64_t smem_desc_k32(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(1u) << 16;
  d |= static_cast<uint64_t>(256u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(6u) << 61;
  return d;
}

// Barrier of the four feeding warps (the even and odd CTA have their own).
__device__ __forceinline__ void feed_bar() { asm volatile("bar.sync 2, 128;" ::: "memory"); }
__device__ __forceinline__ bool feed_all(bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred pi, po;\n\t"
      "setp.ne.u32 pi, %1, 0;\n\t"
      "bar.red.and.pred po, 2, 128, pi;\n\t"
      "selp.u32 %0, 1, 0, po;\n\t}\n"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(p))
      : "memory");
  return r != 0;
}

// The adapter of token t: -1 outside the batch, and for an id out of range
// (reported in the device status word).  EARLY: read before the launch's wait.
template <bool EARLY = false>
__device__ __forceinline__ int lora_id(const int32_t* ids, int T, int n, int t) {
  if (t >= T) return -1;
  const int id = EARLY ? ld_early(ids + t) : ids[t];
  if (id >= -1 && id < n) return id;
  report_bad_index();
  return -1;
}

// Nonzero where a bf16 of the pair is an infinity or NaN: an exponent of all ones carries into the sign's place.
__device__ __forceinline__ uint32_t bf16_pair_nonfinite(uint32_t w) {
  return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
}
__device__ __forceinline__ uint32_t bf16x8_nonfinite(uint4 w) {
  return bf16_pair_nonfinite(w.x) | bf16_pair_nonfinite(w.y) | bf16_pair_nonfinite(w.z) | bf16_pair_nonfinite(w.w);
}
// The smallest normal of the same sign for each infinity and NaN of the pair.
__device__ __forceinline__ uint32_t bf16_pair_finite(uint32_t w) {
  if ((w & 0x7f80u) == 0x7f80u) w = (w & 0xffff8000u) | 0x0080u;
  if ((w & 0x7f800000u) == 0x7f800000u) w = (w & 0x8000ffffu) | 0x00800000u;
  return w;
}

// What the non-finite weights of output `col` of token t's own adapter add.
inline __device__ __noinline__ float lora_nonfinite_term(const LoraArgs& a, int t, int col) {
  const int id = lora_id(a.ids, a.T, a.n, t);
  if (id < 0) return 0.f;
  const uint16_t* b = a.b_pool + (static_cast<size_t>(id) * a.d_out + col) * a.rank;
  const uint16_t* v = a.v + static_cast<size_t>(t) * a.rp;
  float s = 0.f;
  for (int r = 0; r < a.rank; ++r)
    if ((b[r] & 0x7f80u) == 0x7f80u) s += bf16_bits_to_f32(v[r]) * bf16_bits_to_f32(b[r]);
  return s;
}

// Shared state of the feed (barriers, the tile's adapter list, messages).
template <bool ON>
struct LoraShared {};

template <>
struct LoraShared<true> {
  uint64_t full[kLoraRing], empty[kLoraRing];
  uint32_t msg[kLoraRing];        // the message (even CTA)
  uint32_t msg_peer[kLoraRing];   // the odd CTA's kLoraPoison
  uint32_t bad[kLoraRing];
  uint32_t poison[2];
  uint32_t heads[8];
  alignas(16) int32_t id[256];    // read 16 bytes at a time
  uint8_t list[256];              // rows at which an adapter occurs first

  // full: one arrival of each CTA's feed
  __device__ __forceinline__ void init(int ctas = 2) {
    for (int s = 0; s < kLoraRing; ++s) {
      mbar_init(&full[s], ctas);
      mbar_init(&empty[s], 1);
      msg_peer[s] = 0;
      bad[s] = 0;
    }
    poison[0] = poison[1] = 0;
  }
};

// Lists the distinct adapters of `ROWS` (128 or 256) tile rows in the order of
// their first row: ls.id and ls.list are set, the count is returned.  Called by
// the 128 feeding threads; e = thread.  i0 / i1: the ids of rows e and e + 128.
// at: the list position of row e + 128 * which (meaningless for id -1).
template <int ROWS>
__device__ __forceinline__ int lora_list(LoraShared<true>& ls, int e, int i0, int i1, int which, int& at) {
  feed_bar();                     // the previous tile's list is no longer read
  ls.id[e] = i0;
  if (ROWS == 256) ls.id[e + 128] = i1;
  feed_bar();
  const int w = e >> 5, lane = e & 31;
  int first = 0;                  // first row with the id of row e + 128 * which
#pragma unroll
  for (int half = 0; half < ROWS / 128; ++half) {
    const int id = half ? i1 : i0;
    const int wrow = half * 128 + w * 32;              // first row of this warp's 32
    const int wfirst = __ffs(__match_any_sync(0xffffffffu, id)) - 1;
    int at_row = wrow + wfirst;
    if (wfirst == lane && id >= 0) {
      for (int j = 0; j < wrow; j += 4) {
        const int4 o = *reinterpret_cast<const int4*>(&ls.id[j]);
        if (o.x == id || o.y == id || o.z == id || o.w == id) {
          at_row = o.x == id ? j : o.y == id ? j + 1 : o.z == id ? j + 2 : j + 3;
          break;
        }
      }
    }
    __syncwarp();
    const uint32_t m = __ballot_sync(0xffffffffu, id >= 0 && at_row == wrow + lane);
    if (lane == 0) ls.heads[half * 4 + w] = m;
    at_row = __shfl_sync(0xffffffffu, at_row, wfirst);
    if (half == which) first = at_row;
  }
  feed_bar();
  int n = 0;
  at = 0;
#pragma unroll
  for (int k = 0; k < ROWS / 32; ++k) {
    const uint32_t m = ls.heads[k];
    if ((k & 3) == w && (m >> lane & 1u)) ls.list[n + __popc(m & ((1u << lane) - 1u))] = static_cast<uint8_t>(k * 32 + lane);
    if (first >> 5 == k) at = n + __popc(m & ((1u << (first & 31)) - 1u));
    n += __popc(m);
  }
  feed_bar();
  return n;
}

// Position in the ring of message buffers.
struct LoraRing {
  uint32_t count = 0;             // messages passed so far
  uint32_t dirty = ~0u;           // slots that may hold something else than zeros in this thread's row of v
};

// Feeds one tile's slices, the list's adapters x rank / 16, G neighbouring ones to
// a message, so that one round of barriers serves G MMAs and a row's 128 bytes
// are read together; this feed takes messages first, first + stride, ...  Row
// `e` of a v slice is token `tok` when e < NV (`mine`: its adapter's list
// position, -1 for none); row e of a slice of B is output n0 + e when e < NB.  A
// slice takes buf_bytes of the message's buffer, the operands at v_at and b_at.
// `ready()` is called before v is first read, `send(slot, slices, last, poison)`
// by thread 0 for a finished message.
//
// Each thread moves its rows of both operands through registers, loaded two
// messages ahead, and asks all its rows of B into L2 while it waits for v: what
// a mixed batch reads here comes from DRAM, and is all that is left to do by
// then.  (TMA boxes of 32-byte rows took 2 us a message.)
__device__ __forceinline__ int lora_messages(int n_list, int rp, int G, int first, int stride) {
  const int total = (n_list * (rp >> 4) + G - 1) / G;
  return total > first ? (total - first - 1) / stride + 1 : 0;
}

template <int NV, int NB, int G, typename Ready, typename Send>
__device__ __forceinline__ bool lora_feed(const LoraArgs& a, LoraShared<true>& ls, LoraRing& ring, uint8_t* ext,
                                          uint32_t v_at, uint32_t b_at, uint32_t buf_bytes, int e, int n_list,
                                          int first, int stride, int tok, int mine, int n0, Ready ready, Send send) {
  const int per = a.rp >> 4;
  const int total = n_list * per;
  const int msgs = lora_messages(n_list, a.rp, G, first, stride);
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const uint4* vrow = reinterpret_cast<const uint4*>(a.v + static_cast<size_t>(tok) * a.rp);
  const bool has_b = e < NB && n0 + e < a.d_out;
  const uint16_t* brow = a.b_pool + (static_cast<size_t>(n0) + e) * a.rank;
  const size_t b_pitch = static_cast<size_t>(a.d_out) * a.rank;      // between adapters
  auto slices = [&](int m) { return min(G, total - (first + m * stride) * G); };
  if (has_b)
    for (int m = 0; m < msgs; ++m) {
      const int sl0 = (first + m * stride) * G, n = slices(m);
      int l = sl0 / per, k = sl0 - l * per;
      for (int s = 0; s < n; ++s) {          // once per adapter: G slices of one are 32 G bytes of a row
        if (s == 0 || k == 0)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(brow + ls.id[ls.list[l]] * b_pitch + k * 16));
        if (++k == per) { k = 0; ++l; }
      }
    }
  ready();
  struct Set { uint4 v[G][2], b[G][2]; };
  Set set[2];
  auto load = [&](Set& r, int m) {
    if (m >= msgs) return;
    const int sl0 = (first + m * stride) * G;
    int l = sl0 / per, k = sl0 - l * per;
    const int n = slices(m);
#pragma unroll
    for (int s = 0; s < G; ++s) {
      r.b[s][0] = r.b[s][1] = r.v[s][0] = r.v[s][1] = zero;
      if (s < n) {
        if (has_b) {
          const uint4* p = reinterpret_cast<const uint4*>(brow + ls.id[ls.list[l]] * b_pitch + k * 16);
          r.b[s][0] = __ldg(p);
          if (k * 16 + 8 < a.rank) r.b[s][1] = __ldg(p + 1);
        }
        if (e < NV && mine == l) {
          r.v[s][0] = vrow[2 * k];
          r.v[s][1] = vrow[2 * k + 1];
        }
        if (++k == per) { k = 0; ++l; }
      }
    }
  };
  load(set[0], 0);
  load(set[1], 1);
  bool ok = true;
  uint32_t dirty = ring.dirty;               // slots in which this row of v is not all zero
  auto pass = [&](Set& r, int m) -> bool {
    const uint32_t slot = ring.count % kLoraRing, phase = (ring.count / kLoraRing) & 1u;
    ring.count += 1;
    const int n = slices(m);
    ok = ok && mbar_wait_cl(&ls.empty[slot], phase ^ 1u);
    uint8_t* buf = ext + slot * G * buf_bytes;
    if (ok) {
      const int sw = (e >> 2) & 1;
      // v: where the token has no slice here and the row is still zero from before, nothing is written
      const int sl0 = (first + m * stride) * G;
      const bool any_v = e < NV && mine >= 0 && mine * per < sl0 + n && (mine + 1) * per > sl0;
      if (e < NV && (any_v || (dirty >> slot & 1u))) {
#pragma unroll
        for (int s = 0; s < G; ++s) {
          uint8_t* row = buf + s * buf_bytes + v_at + e * 32;
          *reinterpret_cast<uint4*>(row + sw * 16) = r.v[s][0];
          *reinterpret_cast<uint4*>(row + (sw ^ 1) * 16) = r.v[s][1];
        }
        dirty = (dirty & ~(1u << slot)) | (any_v ? 1u << slot : 0u);
      }
      if (e < NB) {
        uint32_t bad = 0;
#pragma unroll
        for (int s = 0; s < G; ++s) bad |= bf16x8_nonfinite(r.b[s][0]) | bf16x8_nonfinite(r.b[s][1]);
        if (bad) {
          ls.bad[slot] = 1;
#pragma unroll
          for (int s = 0; s < G; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint4 w = r.b[s][h];
              r.b[s][h] = make_uint4(bf16_pair_finite(w.x), bf16_pair_finite(w.y), bf16_pair_finite(w.z), bf16_pair_finite(w.w));
            }
        }
#pragma unroll
        for (int s = 0; s < G; ++s) {
          uint8_t* row = buf + s * buf_bytes + b_at + e * 32;
          *reinterpret_cast<uint4*>(row + sw * 16) = r.b[s][0];
          *reinterpret_cast<uint4*>(row + (sw ^ 1) * 16) = r.b[s][1];
        }
      }
    }
    load(r, m + 2);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    if (!feed_all(ok)) return false;
    if (e == 0) {
      const bool any = ls.bad[slot] != 0;
      ls.bad[slot] = 0;
      send(slot, static_cast<uint32_t>(n), m + 1 == msgs, any);
    }
    return true;
  };
  for (int m = 0; m < msgs; m += 2) {
    if (!pass(set[0], m)) return false;
    if (m + 1 < msgs && !pass(set[1], m + 1)) return false;
  }
  ring.dirty = dirty;
  return true;
}

}  // namespace ftm
