// pattn.cu — attention of up to 16 rows over a paged cache, bf16 or 4-bit, with
// an optional window and sinks.
//
// Row i sits at position p = seq_len - M + i and sees the keys t <= p with
// t > p - window or t < sinks (window 0: every t <= p).
// s_t = q.k_t / sqrt(128), o = sum_t exp(s_t - m) v_t / sum_t exp(s_t - m).
//
// Decomposition (flash-decoding).  Keys are taken in tiles of 128 at absolute
// positions; the M * group query rows of a KV head (group query heads read it)
// are cut into row tiles of up to N = 16, 32 or 64 rows.  The keys are the 128
// rows of the tcgen05 MMAs and the query rows their N dimension, so the work of
// a tile follows the number of query rows (13 for one decoded token of the
// 52-head target), not a padded 128:
//   S^T[128 keys x 2N]  = K[128 x 128 d] . [Q_hi; Q_lo]^T
//   O^T[128 d x 2N]     = V^T[128 x 128 keys] . [P_hi; P_lo]^T
// The two operand parts of q and p are stacked along N: K and V are read from
// shared memory once per tile.  A thread of the softmax owns one key and half
// of the rows, and one d of O.  A CTA (slot, KV head, row tile) walks one chunk
// of L key tiles and writes (O, max, sum); a merge kernel joins the chunks.
//
// The split of the keys is a function of the row's own position alone (chunk_len
// below): chunks are whole multiples of L tiles from position 0, so a row has
// the same bits alone and in any block (batch-height invariance).  L grows
// with the position such that there are never more chunks than SMs per KV head;
// a block that crosses such a step runs its two groups of rows one after the
// other.  Tiles that no row sees are skipped: they would add exact zeros.
//
// Precision: all operands are binary16.  A 4-bit value is exact in it; a bf16
// value times 32 is exact when 2^-22 <= |x| < 2^11 (below: off by at most 2^-30
// absolute; keys with a larger or non-finite element are worked on in fp32, see
// `odd` below).  q and p are split into two parts, 22 significant bits.  Each
// tile's O starts afresh in TMEM and is added up in fp32 registers: the tensor
// core's own additions truncate, and 27 tiles of them were off by 8e-6.
#include <type_traits>

#include "attn_mma.cuh"
#include "common.cuh"
#include "internal.h"
#include "kv4.cuh"

namespace spec {

constexpr int kKeys = 128;                          // keys of a tile
constexpr int kPagesPerTile = kKeys / 16;
constexpr int kHalf = kKeys * 128;                  // one d half of a K or V tile: [keys][64 values]
constexpr int kStageBytes = 4 * kHalf;              // K then V, 64 KB
constexpr uint64_t kPattnWaitNs = 2000000000ull;

// Shared memory: K/V stages ([d half][key][128 B] with the 128-byte swizzle),
// Q and P.  Q: 16-byte chunk d / 8 of row r (hi rows, then lo rows) at
// (d / 8) * 32 N + 16 r.  P: 8 rows of a key at (r / 8) * 2048 + 16 key.
// TMEM columns: two S buffers of 2N, O of 2N.
template <int N>
struct Cfg {
  static_assert(N == 16 || N == 32 || N == 64, "rows of a row tile");
  static constexpr int kCols = N / 2;               // rows of a softmax thread
  static constexpr int kStages = N == 64 ? 2 : 3;
  static constexpr int kQBytes = 2 * N * 256;
  static constexpr size_t kSmem = 1024 + (size_t)kStages * kStageBytes + 2 * kQBytes;
  static constexpr uint32_t kTmO = 4 * N;
  static constexpr int kTmAlloc = N == 16 ? 128 : (N == 32 ? 256 : 512);
};

// warps: 0-7 softmax (warp w: keys and d's 32 (w % 4).., rows (N / 2) (w / 4)..),
// 8 issues the QK MMAs, 9 the PV MMAs, 10-15 unpack pages of K and V in turn.
// 16 warps: a 17th would leave each thread 96 registers instead of 128.
constexpr int kSoftWarps = 8, kWQk = 8, kWPv = 9, kWLoad = 10, kUnpackWarps = 6;
constexpr int kPattnThreads = 32 * (kWLoad + kUnpackWarps);

struct PattnPlan {
  int M, nq, nkv, group, window, sinks;
  int C;                     // chunks of a KV head at most
  int slots;                 // chunk slots launched (<= C)
  int Lw;                    // tiles per chunk at most (what the window needs)
  int tile_rows;             // rows per row tile
};

// tiles per chunk of a row at position p
SPEC_DEV int chunk_len(const PattnPlan& pl, int p) {
  const int l = p > 0 ? (p >> 7) / pl.C + 1 : 1;
  return l < pl.Lw ? l : pl.Lw;
}
// the first position that a row at p sees through its window
SPEC_DEV int window_low(const PattnPlan& pl, int p) { return pl.window > 0 && p >= pl.window ? p - pl.window + 1 : 0; }

// The rows of a block that share a chunk length (all of them, or the rows
// before and after a step of chunk_len), and their chunk slots: the sinks'
// chunks that end before the window, then the window's.
struct Span {
  int i0, i1;                // block rows [i0, i1)
  int L, lo, last;           // tiles per chunk; first window key; last key
  int sink_tiles, ns, cbase, nslots;
};
SPEC_DEV int span_count(const PattnPlan& pl, int n_past) {
  return chunk_len(pl, n_past) == chunk_len(pl, n_past + pl.M - 1) ? 1 : 2;
}
SPEC_DEV Span span_of(const PattnPlan& pl, int n_past, int pass) {
  Span s;
  const int la = chunk_len(pl, n_past), lb = chunk_len(pl, n_past + pl.M - 1);
  const int cut = la == lb ? pl.M : la * pl.C * kKeys - n_past;      // rows before the step
  s.i0 = pass == 0 ? 0 : cut;
  s.i1 = pass == 0 ? cut : pl.M;
  s.L = pass == 0 ? la : lb;
  s.lo = window_low(pl, n_past + s.i0);
  s.last = n_past + s.i1 - 1;
  s.sink_tiles = s.ns = s.cbase = s.nslots = 0;
  if (s.last >= 0) {
    const int keys = s.L * kKeys, sk = pl.window > 0 ? min(pl.sinks, s.last + 1) : 0;
    s.sink_tiles = (sk + kKeys - 1) / kKeys;
    s.cbase = s.lo / keys;
    s.ns = min((s.sink_tiles + s.L - 1) / s.L, s.cbase);
    s.nslots = s.ns + s.last / keys - s.cbase + 1;
  }
  return s;
}
// the key tiles of slot c: n0 from a0, then n - n0 from a1
struct TileList {
  int a0 = 0, n0 = 0, a1 = 0, n = 0;
  SPEC_DEV int at(int j) const { return j < n0 ? a0 + j : a1 + (j - n0); }
};
SPEC_DEV TileList tiles_of(const Span& s, int c) {
  TileList t;
  if (c >= s.nslots) return t;
  const int x = c < s.ns ? c : s.cbase + c - s.ns, from = x * s.L, to = from + s.L;
  t.a0 = from;
  t.n0 = max(0, min(to, s.sink_tiles) - from);
  t.a1 = max(max(from, s.lo >> 7), from + t.n0);
  t.n = t.n0 + max(0, min(to, (s.last >> 7) + 1) - t.a1);
  return t;
}

SPEC_DEV uint32_t low_bits(int n) { return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u); }

// binary16 parts of a pair: hi nearest, lo what is left (x0 in the low half)
SPEC_DEV void split_pair(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x0, x1);
  const float2 f = __half22float2(h);
  const __half2 l = __floats2half2_rn(x0 - f.x, x1 - f.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}
// C consecutive TMEM columns of this warp's 32 lanes
template <int C>
SPEC_DEV void tmem_ld(uint32_t taddr, float (&v)[C]) {
  uint32_t r[C];
  if constexpr (C == 8) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
  } else if constexpr (C == 16) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
  } else {
    static_assert(C == 32, "8, 16 or 32 columns");
    tmem_ld32(taddr, r);
  }
#pragma unroll
  for (int i = 0; i < C; ++i) v[i] = __uint_as_float(r[i]);
}
// maximum of a value over the warp (one reduction instruction)
SPEC_DEV float warp_max_f32(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;\n" : "=f"(r) : "f"(x));
  return r;
}
SPEC_DEV void named_bar(int id, int count) { asm volatile("bar.sync %0, %1;\n" ::"r"(id), "r"(count) : "memory"); }
SPEC_DEV bool named_bar_or(int id, int count, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, %2, %3, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)pred), "r"(id), "r"(count)
      : "memory");
  return r != 0;
}

SPEC_DEV int page_at(const KvView& kv, int lp) {
  const int page = lp < kv.max_seq_pages ? __ldg(kv.page_table + lp) : -1;
  return page < kv.num_pages ? page : -1;
}

// One page of a tile as an unpacking warp holds it.
// 4-bit: lane = key % 16 + 16 * d half; 64 codes and 4 scale bytes of K and V.
struct Raw4 {
  uint4 k[2], v[2];
  uint32_t ks, vs;
};
SPEC_DEV void load_page(const KvView& kv, int layer, int kvh, int page, int lane, Raw4& r) {
  const uint4 z = make_uint4(0, 0, 0, 0);
  r.k[0] = r.k[1] = r.v[0] = r.v[1] = z;                  // an unmapped page: zeros (its keys are masked)
  r.ks = r.vs = 0;
  if (page < 0) return;
  const int t = lane & 15, half = lane >> 4;
  const uint8_t* kp = reinterpret_cast<const uint8_t*>(kv.pool) +
                      (((size_t)page * kv.n_layers + layer) * 2 * kv.n_kv + kvh) * kKv4PageBytes;
  const uint8_t* vp = kp + (size_t)kv.n_kv * kKv4PageBytes;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    r.k[c] = __ldg(reinterpret_cast<const uint4*>(kp + kv4_chunk(t, 2 * half + c)));
    r.v[c] = __ldg(reinterpret_cast<const uint4*>(vp + kv4_chunk(t, 2 * half + c)));
  }
  r.ks = __ldg(reinterpret_cast<const uint32_t*>(kp + kKv4Scales + 8 * t + 4 * half));
  r.vs = __ldg(reinterpret_cast<const uint32_t*>(vp + kKv4Scales + 8 * t + 4 * half));
}
// the 64 values of one key and d half as binary16 into a tile's row (128
// bytes, 16-byte chunk j at j ^ (row % 8)); the eight lanes of a store phase
// hold different rows % 8, so no two meet in a bank
SPEC_DEV void unpack_row(const uint4 (&codes)[2], uint32_t scales, uint8_t* row, int r7) {
  const uint32_t sc = __vminu4(scales, 0xE2E2E2E2u);
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const uint32_t w[4] = {codes[c].x, codes[c].y, codes[c].z, codes[c].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t s2 = ((sc >> (8 * (2 * c + (j >> 1)))) & 0xFFu) * 0x00800080u;   // (byte << 7) in both halves
      uint32_t f[4];
      e2m1_word(w[j], f);
      const int ch = 4 * c + j;
      *reinterpret_cast<uint4*>(row + ((ch ^ r7) << 4)) =
          make_uint4(hmul2_u32(f[0], s2), hmul2_u32(f[1], s2), hmul2_u32(f[2], s2), hmul2_u32(f[3], s2));
    }
  }
}
// bf16: load j of K or V is the 16-byte chunk lane % 16 of row 2j + lane / 16
struct Raw16 {
  uint4 x[8];
};
SPEC_DEV void load_rows(const KvView& kv, int layer, int which, int kvh, int page, int lane, Raw16& r) {
  if (page < 0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) r.x[j] = make_uint4(0, 0, 0, 0);
    return;
  }
  const uint4* p = reinterpret_cast<const uint4*>(
      kv.pool + ((((size_t)page * kv.n_layers + layer) * 2 + which) * kv.n_kv + kvh) * 2048);
#pragma unroll
  for (int j = 0; j < 8; ++j) r.x[j] = __ldg(p + 32 * j + lane);
}
// bf16 pair times 32 as binary16 (exact in its normal range): 5 is added to
// both exponents; |x| >= 2^11, infinities and NaN are the caller's business
SPEC_DEV uint32_t bf16x2_to_f16x2(uint32_t w) {
  const uint32_t y = w + 0x02800280u;
  const __half2 h = __floats2half2_rn(__uint_as_float(y << 16), __uint_as_float(y & 0xFFFF0000u));
  return *reinterpret_cast<const uint32_t*>(&h);
}
constexpr float kBf16Scale = 32.f;
constexpr uint32_t kBf16Limit = 0x4500u;            // bf16 bits of 2^11

// ---------------------------------------------------------------------------
// partials: grid (slot, KV head, row tile)
// ---------------------------------------------------------------------------
template <bool k4, int N>
__global__ void __launch_bounds__(kPattnThreads, 1)
pattn_kernel(const float* __restrict__ q, PattnPlan pl, KvView kv, int layer, float* __restrict__ part_o,
             float2* __restrict__ part_ml, int32_t* status) {
  using G = Cfg<N>;
  constexpr int NC = G::kCols, kStages = G::kStages;
  extern __shared__ __align__(128) uint8_t dsm[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dsm) + 1023) & ~(uintptr_t)1023);
  uint8_t* qs = sm + (size_t)kStages * kStageBytes;
  uint8_t* ps = qs + G::kQBytes;
  __shared__ uint32_t tmem_slot;
  __shared__ __align__(8) uint64_t q_full, k_full[kStages], v_full[kStages], k_free[kStages], v_free[kStages],
      s_full[2], s_free[2], p_full, pv_done;
  __shared__ __align__(16) float2 scale[N];             // per row: {score to base-2 units, exponent of p = 1}
  __shared__ float red[2][4][NC], alpha_s[2][NC];
  __shared__ __align__(16) uint16_t odd[kStages][2][kPagesPerTile];   // bf16: keys of K, V with an element out of range
  __shared__ int gave_up[2];                            // a wait of this softmax group ran out

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slot = blockIdx.x, kvh = blockIdx.y, R = pl.M * pl.group;
  const int r0 = blockIdx.z * pl.tile_rows, nr = min(pl.tile_rows, R - r0);
  if (warp == kWQk) tmem_alloc(&tmem_slot, G::kTmAlloc);
  if (tid == 32 * kWPv) {
    mbar_init(&q_full, 32 * kSoftWarps);
    for (int b = 0; b < kStages; ++b) {
      mbar_init(&k_full[b], kPagesPerTile);
      mbar_init(&v_full[b], kPagesPerTile);
      mbar_init(&k_free[b], 1);
      mbar_init(&v_free[b], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&s_full[b], 1);
      mbar_init(&s_free[b], 32 * kSoftWarps);
    }
    mbar_init(&p_full, 32 * kSoftWarps);
    mbar_init(&pv_done, 1);
    gave_up[0] = gave_up[1] = 0;
    fence_mbarrier_init();
  }
  pdl_trigger();
  pdl_wait();
  const int n_past = __ldcg(kv.seq_len) - pl.M;
  const int passes = span_count(pl, n_past);
  TileList tl0 = tiles_of(span_of(pl, n_past, 0), slot), tl1;
  if (passes == 2) tl1 = tiles_of(span_of(pl, n_past, 1), slot);
  const int total = tl0.n + tl1.n;
  auto tile_at = [&](int it) { return it < tl0.n ? tl0.at(it) : tl1.at(it - tl0.n); };
  const int b_last = n_past + pl.M - 1;                 // the block's last position
  const int low0 = window_low(pl, n_past), low1 = window_low(pl, b_last), sinks = pl.window > 0 ? pl.sinks : 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  if (total == 0) {
    // nothing of this chunk is seen
  } else if (warp >= kWLoad) {
    // -------------------------------------------------------------- unpack
    // item g is page g % 8 of tile g / 8; this warp takes every sixth
    const int items = total * kPagesPerTile, g0 = warp - kWLoad;
    auto page_of = [&](int g) { return g < items ? page_at(kv, tile_at(g >> 3) * kPagesPerTile + (g & 7)) : -1; };
    auto free_k = [&](int it) {
      return it < kStages || __all_sync(0xffffffffu, mbar_wait_ns(&k_free[it % kStages], ((it / kStages) - 1) & 1, kPattnWaitNs));
    };
    auto free_v = [&](int it) {
      return it < kStages || __all_sync(0xffffffffu, mbar_wait_ns(&v_free[it % kStages], ((it / kStages) - 1) & 1, kPattnWaitNs));
    };
    auto done = [&](uint64_t* bar) {
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    bool ok = true;
    if constexpr (k4) {
      // registers hold the next two items: about 27 KB per SM in flight
      const int t = lane & 15, half = lane >> 4;
      Raw4 a, b;
      load_page(kv, layer, kvh, page_of(g0), lane, a);
      load_page(kv, layer, kvh, page_of(g0 + kUnpackWarps), lane, b);
      int next = page_of(g0 + 2 * kUnpackWarps);
      auto put = [&](int g, Raw4& r) -> bool {
        const int it = g >> 3, st = it % kStages, key = 16 * (g & 7) + t;
        uint8_t* row = sm + (size_t)st * kStageBytes + half * kHalf + key * 128;
        if (!free_k(it)) return false;
        unpack_row(r.k, r.ks, row, key & 7);
        done(&k_full[st]);
        if (!free_v(it)) return false;
        unpack_row(r.v, r.vs, row + 2 * kHalf, key & 7);
        done(&v_full[st]);
        const int page = next;
        next = page_of(g + 3 * kUnpackWarps);
        load_page(kv, layer, kvh, page, lane, r);       // item g + 12
        return true;
      };
      for (int g = g0; ok && g < items; g += 2 * kUnpackWarps) {
        ok = put(g, a);
        if (ok && g + kUnpackWarps < items) ok = put(g + kUnpackWarps, b);
      }
    } else {
      // registers hold the next item: up to 48 KB per SM in flight
      Raw16 k, v;
      int page = page_of(g0);
      load_rows(kv, layer, 0, kvh, page, lane, k);
      load_rows(kv, layer, 1, kvh, page, lane, v);
      auto put = [&](Raw16& r, int st, int u, int which, int t0, bool there) -> uint32_t {
        uint32_t far = 0;                               // rows (of the 16) with an element out of range
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int row = 2 * j + (lane >> 4), key = 16 * u + row, t = t0 + 16 * u + row, ch = lane & 15;
          uint32_t w[4] = {r.x[j].x, r.x[j].y, r.x[j].z, r.x[j].w};
          uint32_t top = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) top = __vmaxu2(top, w[e] & 0x7FFF7FFFu);
          // a key that some row sees; others are masked, and their V is zeroed
          // (stale bytes may be anything, and 0 * NaN is NaN)
          const bool seen = there && t <= b_last && (t >= low0 || t < sinks);
          const bool big = seen && ((top & 0xFFFFu) >= kBf16Limit || (top >> 16) >= kBf16Limit);
          const uint32_t m = __ballot_sync(0xffffffffu, big);
          far |= ((m & 0xFFFFu ? 1u : 0u) | (m >> 16 ? 2u : 0u)) << (2 * j);
          if (big) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] &= ((w[e] & 0x7FFFu) >= kBf16Limit ? 0xFFFF0000u : 0xFFFFFFFFu) &
                      ((w[e] >> 16 & 0x7FFFu) >= kBf16Limit ? 0xFFFFu : 0xFFFFFFFFu);
          }
          uint4 y = make_uint4(bf16x2_to_f16x2(w[0]), bf16x2_to_f16x2(w[1]), bf16x2_to_f16x2(w[2]), bf16x2_to_f16x2(w[3]));
          if (which == 1 && !seen) y = make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>(sm + (size_t)st * kStageBytes + (2 * which + (ch >> 3)) * kHalf + key * 128 +
                                    (((ch & 7) ^ (key & 7)) << 4)) = y;
        }
        return far;
      };
      for (int g = g0; g < items; g += kUnpackWarps) {
        const int it = g >> 3, u = g & 7, st = it % kStages, t0 = tile_at(it) * kKeys;
        const int next = page_of(g + kUnpackWarps);
        ok = free_k(it);
        if (!ok) break;
        const uint32_t fk = put(k, st, u, 0, t0, page >= 0);
        done(&k_full[st]);
        load_rows(kv, layer, 0, kvh, next, lane, k);
        ok = free_v(it);
        if (!ok) break;
        const uint32_t fv = put(v, st, u, 1, t0, page >= 0);
        if (lane == 0) {
          odd[st][0][u] = (uint16_t)fk;                 // read after v_full
          odd[st][1][u] = (uint16_t)fv;
        }
        done(&v_full[st]);
        load_rows(kv, layer, 1, kvh, next, lane, v);
        page = next;
      }
    }
    if (!ok && lane == 0) atomicOr(status, SPEC_ST_DEVICE_WAIT);
  } else if (warp == kWQk) {
    // -------------------------------------------------- S^T = K . [Q_hi; Q_lo]^T
    // D f32 (bit 4), A and B f16, N >> 3 at 17, M >> 4 at 24; 8 d steps of 16
    constexpr uint32_t kId = (1u << 4) | ((2u * N >> 3) << 17) | ((128u >> 4) << 24);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t dk0 = desc_sw128(__shfl_sync(0xffffffffu, smem_u32(sm), 0), 16, 1024);
    const uint64_t dq0 = smem_desc(__shfl_sync(0xffffffffu, smem_u32(qs), 0), 32 * N, 128);
    bool ok = __all_sync(0xffffffffu, mbar_wait_ns(&q_full, 0, kPattnWaitNs));
    int last = -1;
    for (int it = 0; ok && it < total; ++it) {
      const int st = it % kStages, sb = it & 1;
      bool w = mbar_wait_ns(&k_full[st], (it / kStages) & 1, kPattnWaitNs);
      if (it >= 2) w = w && mbar_wait_ns(&s_free[sb], ((it >> 1) - 1) & 1, kPattnWaitNs);
      ok = __all_sync(0xffffffffu, w);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t dk = dk0 + (uint64_t)((st * kStageBytes) >> 4);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          mma_f16_ss(tm + 2u * N * sb, dk + (uint64_t)(((ks >> 2) * kHalf + (ks & 3) * 32) >> 4),
                     dq0 + (uint64_t)((ks * 64 * N) >> 4), kId, ks != 0);
        mma_commit(&s_full[sb]);
        mma_commit(&k_free[st]);
      }
      __syncwarp();
      last = it;
    }
    if (!ok && lane == 0) atomicOr(status, SPEC_ST_DEVICE_WAIT);
    if (last >= 0) mbar_wait_ns(&s_full[last & 1], (last >> 1) & 1, kPattnWaitNs);   // before TMEM is released
  } else if (warp == kWPv) {
    // -------------------------------------------------- O^T = V^T . [P_hi; P_lo]^T
    // 8 key steps of 16.  A (V) is MN-major (bit 15): lbo = the d-half stride,
    // sbo = 1 KB between 8-key groups.  B (P) is MN-major (bit 16), no swizzle:
    // lbo = 128 between 8-key groups, sbo = 2 KB between 8-row groups.
    constexpr uint32_t kId = (1u << 4) | (1u << 15) | (1u << 16) | ((2u * N >> 3) << 17) | ((128u >> 4) << 24);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t dv0 = desc_sw128(__shfl_sync(0xffffffffu, smem_u32(sm), 0) + 2 * kHalf, kHalf, 1024);
    const uint64_t dp0 = smem_desc(__shfl_sync(0xffffffffu, smem_u32(ps), 0), 128, 2048);
    bool ok = true;
    int last = -1;
    for (int it = 0; ok && it < total; ++it) {
      const int st = it % kStages;
      ok = __all_sync(0xffffffffu, mbar_wait_ns(&p_full, it & 1, kPattnWaitNs) &&
                                       mbar_wait_ns(&v_full[st], (it / kStages) & 1, kPattnWaitNs));
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t dv = dv0 + (uint64_t)((st * kStageBytes) >> 4);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_f16_ss(tm + G::kTmO, dv + (uint64_t)((kk * 2048) >> 4), dp0 + (uint64_t)((kk * 256) >> 4), kId, kk != 0);
        mma_commit(&pv_done);
        mma_commit(&v_free[st]);
      }
      __syncwarp();
      last = it;
    }
    if (!ok && lane == 0) atomicOr(status, SPEC_ST_DEVICE_WAIT);
    if (last >= 0) mbar_wait_ns(&pv_done, last & 1, kPattnWaitNs);
  } else {
    // -------------------------------------------------------------- softmax
    const int h = warp >> 2, ww = warp & 3, tw = tid & 127;
    const int key = 32 * ww + lane, c0 = NC * h;        // this thread's key (and d) and first row
    const uint32_t lane_base = (uint32_t)(32 * ww) << 16;
    constexpr float kBias = 7.f;                        // p = 2^(7 + s - max): binary16 keeps 2^-24 of 2^7
    // Q: 16 threads per row, 8 values each.  The row is scaled by a power of
    // two to at most 2 in magnitude, and the scores are scaled back.
    for (int x = tid; x < N * 16; x += 32 * kSoftWarps) {
      const int r = x >> 4, ch = x & 15;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
      if (r < nr) {
        const int i = (r0 + r) / pl.group, hd = (r0 + r) - i * pl.group;
        const float4* src = reinterpret_cast<const float4*>(q + ((size_t)i * pl.nq + kvh * pl.group + hd) * 128 + 8 * ch);
        a = src[0];
        b = src[1];
      }
      float mx = fmaxf(fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(a.z), fabsf(a.w))),
                       fmaxf(fmaxf(fabsf(b.x), fabsf(b.y)), fmaxf(fabsf(b.z), fabsf(b.w))));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const int e = min(max((int)((__float_as_uint(mx) >> 23) & 255u) - 127, -100), 100);
      const float mul = __uint_as_float((uint32_t)(127 - e) << 23);
      uint4 hi, lo;
      split_pair(a.x * mul, a.y * mul, hi.x, lo.x);
      split_pair(a.z * mul, a.w * mul, hi.y, lo.y);
      split_pair(b.x * mul, b.y * mul, hi.z, lo.z);
      split_pair(b.z * mul, b.w * mul, hi.w, lo.w);
      *reinterpret_cast<uint4*>(qs + ch * 32 * N + r * 16) = hi;
      *reinterpret_cast<uint4*>(qs + ch * 32 * N + (N + r) * 16) = lo;
      // log2(e) / sqrt(d) times the row's power of two (and the 32 of a bf16 K)
      if (ch == 0)
        scale[r] = make_float2((1.4426950408889634f / sqrtf(128.0f)) * (k4 ? 1.f : 1.f / kBf16Scale) *
                                   __uint_as_float((uint32_t)(127 + e) << 23),
                               r < nr ? -INFINITY : 0.f);
    }
    fence_proxy_async();
    mbar_arrive(&q_full);
    named_bar(3, 32 * kSoftWarps);                      // `scale` is written
    auto page_lane = [&](int it) { return it < total && lane < kPagesPerTile ? page_at(kv, tile_at(it) * kPagesPerTile + lane) : -1; };
    int pg = page_lane(0);
    bool ok = true, left = false;
    int it = 0;
#pragma unroll 1
    for (int pass = 0; !left && pass < passes; ++pass) {
      const Span sp = span_of(pl, n_past, pass);
      const int n = pass == 0 ? tl0.n : tl1.n;
      float acc[NC], lsum[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) acc[c] = lsum[c] = 0.f;
      if (pass > 0) {
        // new maxima; the threads that still read the old ones are behind this barrier
        named_bar(1 + h, 128);
        if (tw < NC && c0 + tw < nr) scale[c0 + tw].y = -INFINITY;
        named_bar(1 + h, 128);
      }
      auto drain = [&]() -> bool {                      // O of tile it - 1 (this pass), added in fp32
        if (!__all_sync(0xffffffffu, mbar_wait_ns(&pv_done, (it - 1) & 1, kPattnWaitNs))) return false;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < NC; c += 8) {
          float hi[8], lo[8];
          tmem_ld<8>(tmem + lane_base + G::kTmO + c0 + c, hi);
          tmem_ld<8>(tmem + lane_base + G::kTmO + N + c0 + c, lo);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[c + e] += hi[e] + lo[e];
        }
        tc_fence_before();
        return true;
      };
#pragma unroll 1
      for (int sc = 0; sc < n; ++sc, ++it) {
        const int sb = it & 1, st = it % kStages, t0 = tile_at(it) * kKeys, t = t0 + key;
        const uint32_t pages = __ballot_sync(0xffffffffu, pg >= 0) & 0xffu;
        pg = page_lane(it + 1);
        // rows of this thread that see its key; `masked`: some row of the
        // block does not see some key of the tile
        uint32_t vis = 0xffffffffu;
        const bool masked = pages != 0xffu || t0 + kKeys - 1 > n_past || (t0 < low1 && t0 + kKeys > sinks) || passes > 1;
        if (masked) {
          const long long d = (long long)t - n_past;    // rows i >= d, and i < d + window
          const int from = (int)(d < sp.i0 ? sp.i0 : (d > sp.i1 ? sp.i1 : d));
          const long long e = pl.window > 0 && t >= sinks ? d + pl.window : pl.M;
          const int to = (int)(e < sp.i1 ? (e < 0 ? 0 : e) : sp.i1);
          vis = low_bits(min(to * pl.group - r0, nr) - c0) & ~low_bits(from * pl.group - r0 - c0);
          if (!((pages >> (key >> 4)) & 1u)) vis = 0u;
        }
        bool got = __all_sync(0xffffffffu, mbar_wait_ns(&s_full[sb], (it >> 1) & 1, kPattnWaitNs));
        if (!k4) got = got && __all_sync(0xffffffffu, mbar_wait_ns(&v_full[st], (it / kStages) & 1, kPattnWaitNs));
        tc_fence_after();
        float x[NC];
        auto scores = [&]() {
#pragma unroll
          for (int c = 0; c < NC; c += 8) {
            float hi[8], lo[8];
            tmem_ld<8>(tmem + lane_base + 2u * N * sb + c0 + c, hi);
            tmem_ld<8>(tmem + lane_base + 2u * N * sb + N + c0 + c, lo);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e) x[c + e] = hi[e] + lo[e];
          }
          if (!k4 && ((odd[st][0][key >> 4] >> (key & 15)) & 1u)) {
            // a key with an element past binary16: its scores in fp32
            const uint16_t* kr = kv.pool + ((((size_t)page_at(kv, t >> 4) * kv.n_layers + layer) * 2) * kv.n_kv + kvh) * 2048 +
                                 (t & 15) * 128;
#pragma unroll 1
            for (int c = 0; c < NC; ++c) {
              const int fr = r0 + min(c0 + c, nr - 1), i = fr / pl.group;
              const float* qr = q + ((size_t)i * pl.nq + kvh * pl.group + fr - i * pl.group) * 128;
              float y = 0.f;
#pragma unroll 4
              for (int d = 0; d < 128; ++d) y = fmaf(qr[d], __uint_as_float((uint32_t)kr[d] << 16), y);
              y *= (1.4426950408889634f / sqrtf(128.0f)) / scale[c0 + c].x;
#pragma unroll
              for (int e = 0; e < NC; ++e)
                if (e == c) x[e] = y;
            }
          }
        };
        // exponents of the visible scores over the rows' references
        auto exponents = [&]() {
#pragma unroll
          for (int c = 0; c < NC; c += 2) {
            const float4 f = *reinterpret_cast<const float4*>(&scale[c0 + c]);
            x[c] = fmaf(x[c], f.x, -f.y);
            x[c + 1] = fmaf(x[c + 1], f.z, -f.w);
          }
          if (masked) {
#pragma unroll
            for (int c = 0; c < NC; ++c)
              if (!((vis >> c) & 1u)) x[c] = -INFINITY;
          }
        };
        if (got) scores();
        exponents();
        bool over = false;                              // some p would exceed 2^15
#pragma unroll
        for (int c = 0; c < NC; ++c) over = over || x[c] > 8.f + kBias;
        // a wait that ran out is carried to this barrier, where the group of
        // 128 threads leaves together
        if (!got || !ok) *reinterpret_cast<volatile int*>(&gave_up[h]) = 1;
        bool drained = sc == 0;
        if (named_bar_or(1 + h, 128, over || !got || !ok)) {
          left = *reinterpret_cast<volatile int*>(&gave_up[h]) != 0;
          if (left) break;
          // each row's largest score of the tile; where it exceeds the
          // reference by more than 8 it becomes the reference
          scores();
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const float m = warp_max_f32((vis >> c) & 1u ? x[c] * scale[c0 + c].x : -INFINITY);
            if (lane == 0) red[h][ww][c] = m;
          }
          if (!drained) ok = drain();                   // O so far is in the old units
          drained = true;
          named_bar(1 + h, 128);
          if (tw < NC) {
            const float m = fmaxf(fmaxf(red[h][0][tw], red[h][1][tw]), fmaxf(red[h][2][tw], red[h][3][tw]));
            const float old = scale[c0 + tw].y;         // reference - 7; -inf at first
            float a = 1.f;
            if (m - kBias > old + 8.f) {
              if (old != -INFINITY) a = exp2_approx(old - (m - kBias));
              scale[c0 + tw].y = m - kBias;
            }
            alpha_s[h][tw] = a;
          }
          named_bar(1 + h, 128);
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const float a = alpha_s[h][c];
            acc[c] *= a;
            lsum[c] *= a;
          }
          exponents();
        }
        mbar_arrive(&s_free[sb]);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          x[c] = exp2_approx(x[c]);
          lsum[c] += x[c];
        }
        // P and O are free once P.V of the tile before has finished
        if (!drained) {
          ok = ok && drain();
        } else if (it > 0) {
          ok = ok && __all_sync(0xffffffffu, mbar_wait_ns(&pv_done, (it - 1) & 1, kPattnWaitNs));
        }
#pragma unroll
        for (int c = 0; c < NC; c += 8) {
          uint4 hi, lo;
          split_pair(x[c], x[c + 1], hi.x, lo.x);
          split_pair(x[c + 2], x[c + 3], hi.y, lo.y);
          split_pair(x[c + 4], x[c + 5], hi.z, lo.z);
          split_pair(x[c + 6], x[c + 7], hi.w, lo.w);
          *reinterpret_cast<uint4*>(ps + ((c0 + c) >> 3) * 2048 + key * 16) = hi;
          *reinterpret_cast<uint4*>(ps + ((N + c0 + c) >> 3) * 2048 + key * 16) = lo;
        }
        fence_proxy_async();
        if (ok) mbar_arrive(&p_full);
        if (!k4) {
          // V elements past binary16 are zero in the tile: their p v is added
          // here in fp32, to the rows that see them
          const uint4 m = *reinterpret_cast<const uint4*>(&odd[st][1][0]);
          if (m.x | m.y | m.z | m.w) {
            const uint32_t mw[4] = {m.x, m.y, m.z, m.w};
#pragma unroll 1
            for (int k = 0; k < kKeys; ++k) {
              if (!((mw[k >> 5] >> (k & 31)) & 1u)) continue;
              if (key == k) {
#pragma unroll
                for (int c = 0; c < NC; ++c) red[h][0][c] = (vis >> c) & 1u ? x[c] : -1.f;
              }
              named_bar(1 + h, 128);
              const int tk = t0 + k;
              const uint32_t b = kv.pool[((((size_t)page_at(kv, tk >> 4) * kv.n_layers + layer) * 2 + 1) * kv.n_kv + kvh) * 2048 +
                                         (tk & 15) * 128 + key];
              if ((b & 0x7FFFu) >= kBf16Limit) {
#pragma unroll
                for (int c = 0; c < NC; ++c)
                  if (!(red[h][0][c] < 0.f)) acc[c] += red[h][0][c] * (__uint_as_float(b << 16) * kBf16Scale);
              }
              named_bar(1 + h, 128);
            }
          }
        }
      }
      if (left || n == 0) continue;
      ok = ok && drain();
      left = named_bar_or(1 + h, 128, !ok);
      if (left) break;
      // the row sums over the 128 keys: lanes, then the four warps in order
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const float l = warp_sum(lsum[c]);
        if (lane == 0) red[h][ww][c] = l;
      }
      named_bar(1 + h, 128);
      const int lim = min(nr, sp.i1 * pl.group - r0), from = sp.i0 * pl.group - r0;
      const size_t at = ((size_t)slot * pl.nkv + kvh) * R + r0;
      if (tw < NC && c0 + tw < lim && c0 + tw >= from)
        part_ml[at + c0 + tw] = make_float2(scale[c0 + tw].y, ((red[h][0][tw] + red[h][1][tw]) + red[h][2][tw]) + red[h][3][tw]);
#pragma unroll
      for (int c = 0; c < NC; ++c)
        if (c0 + c < lim && c0 + c >= from) part_o[(at + c0 + c) * 128 + key] = acc[c] * (k4 ? 1.f : 1.f / kBf16Scale);
      named_bar(1 + h, 128);
    }
    if (left && lane == 0) atomicOr(status, SPEC_ST_DEVICE_WAIT);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWQk) {
    tc_fence_after();
    tmem_dealloc(tmem, G::kTmAlloc);
  }
}

// ---------------------------------------------------------------------------
// merge: one warp per (row, head), 4 output elements per lane.  With m the
// largest chunk maximum (base 2) and w_c = 2^(m_c - m):
//   out = sum_c w_c o_c / sum_c w_c l_c, both in chunk order over the chunks in
// which the row sees a key, so the order does not depend on the block.
// ---------------------------------------------------------------------------
constexpr int kMergeWarps = 4;

__global__ void __launch_bounds__(32 * kMergeWarps)
pattn_merge_kernel(const float* __restrict__ part_o, const float2* __restrict__ part_ml, PattnPlan pl,
                   const int32_t* __restrict__ seq_len, float* __restrict__ out) {
  pdl_trigger();
  pdl_wait();
  const int item = blockIdx.x * kMergeWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (item >= pl.M * pl.nq) return;
  const int i = item / pl.nq, head = item % pl.nq, kvh = head / pl.group;
  const int n_past = __ldcg(seq_len) - pl.M;
  Span s = span_of(pl, n_past, 0);
  if (i >= s.i1) s = span_of(pl, n_past, 1);
  const int n = n_past + i < 0 ? 0 : min(s.nslots, pl.slots);
  const size_t stride = (size_t)pl.nkv * pl.M * pl.group;
  const size_t at = (size_t)kvh * pl.M * pl.group + i * pl.group + head % pl.group;
  float m = -INFINITY;
  for (int c = lane; c < n; c += 32) {
    const float2 x = part_ml[at + c * stride];
    if (x.y != 0.f) m = fmaxf(m, x.x);
  }
  m = warp_max(m);
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float L = 0.f;
  for (int c0 = 0; c0 < n; c0 += 32) {
    const float2 x = c0 + lane < n ? part_ml[at + (c0 + lane) * stride] : make_float2(0.f, 0.f);
    const float wl = x.y != 0.f ? exp2f(x.x - m) : 0.f;
#pragma unroll 8
    for (int k = 0; k < min(32, n - c0); ++k) {
      const float w = __shfl_sync(0xffffffffu, wl, k), l = __shfl_sync(0xffffffffu, x.y, k);
      const float4 y = reinterpret_cast<const float4*>(part_o + (at + (c0 + k) * stride) * 128)[lane];
      if (l != 0.f) {
        L += w * l;
        o.x += w * y.x;
        o.y += w * y.y;
        o.z += w * y.z;
        o.w += w * y.w;
      }
    }
  }
  const bool none = L == 0.f;                          // nothing visible: zero
  reinterpret_cast<float4*>(out + ((size_t)i * pl.nq + head) * 128)[lane] =
      none ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o.x / L, o.y / L, o.z / L, o.w / L);
}

// chunks of a KV head at most: one per SM and KV head.  At least 4, so that a
// window's chunks (one of sinks, and one more than the window's own) fit.
static int pattn_chunks(int nkv, int num_sms) { return num_sms / nkv > 4 ? num_sms / nkv : 4; }

size_t paged_attention_floats(int nq, int nkv, int max_rows, int num_sms) {
  return (size_t)pattn_chunks(nkv, num_sms) * nq * max_rows * 130;
}

template <bool k4, int N>
static cudaError_t launch_pattn(const PattnPlan& pl, const KvView& kv, int layer, const float* q, int row_tiles,
                                float* part_o, float2* part_ml, int32_t* status, cudaStream_t st) {
  // the shared-memory limit is a per-device attribute
  constexpr int kMaxDevices = 64;
  static bool have[kMaxDevices] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool known = dev >= 0 && dev < kMaxDevices;
  if (!known || !have[dev]) {
    e = cudaFuncSetAttribute(pattn_kernel<k4, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg<N>::kSmem);
    if (e != cudaSuccess) return e;
    if (known) have[dev] = true;
  }
  pattn_kernel<k4, N><<<dim3(pl.slots, pl.nkv, row_tiles), kPattnThreads, Cfg<N>::kSmem, st>>>(q, pl, kv, layer, part_o,
                                                                                              part_ml, status);
  return cudaGetLastError();
}

cudaError_t launch_paged_attention(bool k4, const KvView& kv, int layer, const float* q, int M, int nq, int window,
                                   int sinks, int num_sms, float* part, float* out, int32_t* status, cudaStream_t st) {
  PattnPlan pl;
  pl.M = M;
  pl.nq = nq;
  pl.nkv = kv.n_kv;
  pl.group = nq / kv.n_kv;
  pl.window = window;
  pl.sinks = sinks;
  pl.C = pattn_chunks(kv.n_kv, num_sms);
  // chunk slots: never more than the cache has tiles; the window's longest
  // chunk is the shortest with which sinks and window fit into C chunks
  const long long tiles = ((long long)kv.max_seq_pages * 16 + kKeys - 1) / kKeys;
  pl.Lw = INT32_MAX;
  pl.slots = (int)(tiles < pl.C ? tiles : pl.C);
  if (window > 0) {
    const long long ws = ((long long)window + 14 + kKeys - 1) / kKeys + 1;       // tiles of window + 15 keys
    const long long ss = ((long long)sinks + kKeys - 1) / kKeys;
    long long L = (ws + ss) / pl.C > 1 ? (ws + ss) / pl.C : 1;
    while ((ss + L - 1) / L + (ws + L - 2) / L + 1 > pl.C) ++L;
    pl.Lw = (int)(L < INT32_MAX ? L : INT32_MAX);
    if (pl.Lw == 1 && ss + ws < pl.slots) pl.slots = (int)(ss + ws);
  }
  const int R = M * pl.group, row_tiles = (R + 63) / 64;
  pl.tile_rows = (R + row_tiles - 1) / row_tiles;
  float2* ml = reinterpret_cast<float2*>(part);        // [slots][nkv][R], then the outputs
  float* po = part + 2 * (size_t)pl.C * nq * 16;
  auto run = [&](auto k4c) {
    constexpr bool k = decltype(k4c)::value;
    return pl.tile_rows <= 16   ? launch_pattn<k, 16>(pl, kv, layer, q, row_tiles, po, ml, status, st)
           : pl.tile_rows <= 32 ? launch_pattn<k, 32>(pl, kv, layer, q, row_tiles, po, ml, status, st)
                                : launch_pattn<k, 64>(pl, kv, layer, q, row_tiles, po, ml, status, st);
  };
  cudaError_t e = k4 ? run(std::true_type{}) : run(std::false_type{});
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((M * nq + kMergeWarps - 1) / kMergeWarps);
  cfg.blockDim = dim3(32 * kMergeWarps);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, pattn_merge_kernel, (const float*)po, (const float2*)ml, pl,
                            (const int32_t*)kv.seq_len, out);
}

}  // namespace spec
