// pattn.cu — attention of up to 16 rows over a paged cache, bf16 or 4-bit, with
// an optional window and sinks.
//
// Row i sits at position p = seq_len - M + i and sees the keys t <= p with
// t > p - window or t < sinks (window 0: every t <= p).
// s_t = q.k_t / sqrt(128), o = sum_t exp(s_t - m) v_t / sum_t exp(s_t - m).
//
// Decomposition (flash-decoding).  The M * group query rows of a KV head (group
// query heads read it) are packed into tiles of up to 128 rows, the rows of the
// tcgen05 MMAs, so that one decoded token of 13 heads and a block of 104 rows
// both take one tile.  Keys are taken in tiles of 128 at absolute positions:
//   S[128 x 128 keys] = Q[128 x 128 d] . K^T      (A = Q in TMEM, B = K)
//   O[128 x 128 d]    = P[128 x 128 keys] . V     (A = P in TMEM, B = V)
// with a running (max, sum) per row.  A CTA (slot, KV head, row tile) walks one
// chunk of L key tiles and writes (O, max, sum); a merge kernel joins the chunks.
// Q and P live in TMEM because shared memory is the busiest unit: a tile's K
// and V are written once and read twice, 192 KB.  With the keys on the MMA's
// rows and Q and P in shared memory (a tile's work then follows the number of
// query rows) 52 rows cost as much as 128 do here: 113 against 24 us for 208
// rows over 32k keys, and one token behind 128k keys was no faster.
//
// The split of the keys is a function of the row's own position alone (chunk_len
// below): chunks are whole multiples of L tiles from position 0, so a row has
// the same bits alone and in any block (batch-height invariance).  L grows
// with the position such that there are never more chunks than SMs per KV head;
// a block that crosses such a step runs its two groups of rows one after the
// other.  Tiles that no row sees are skipped: they would add exact zeros.
//
// Precision: all operands are binary16.  A 4-bit value is exact in it; a bf16
// value is exact when 2^-17 <= |x| < 2^15 (below: off by at most 2^-25 absolute;
// larger and non-finite elements are worked on in fp32, see `odd` below).  q and
// p are split into two parts, 22 significant bits.  The tensor core truncates
// its additions, so the small parts go first, and each tile's O starts afresh
// and is added up in fp32 registers: left in TMEM over 27 tiles it was off by
// 8e-6.
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

constexpr int kStages = 3;                          // [d half][key][128 B], 128-byte swizzle; K, then V
constexpr size_t kPattnSmem = 1024 + (size_t)kStages * kStageBytes;
// TMEM columns: two score buffers, each overwritten in place by its P parts
// (16 columns of high and 16 of low parts per 32 keys); O; Q (64 columns of high
// parts, then 64 of low ones)
constexpr uint32_t kTmS = 0, kTmO = 256, kTmQ = 384;
constexpr int kTmAll = 512;

// warps: 0-7 softmax, two threads per row (warp w: rows 32 (w % 4).., keys and
// d's 64 (w / 4)..), 8 issues the QK MMAs, 9 the PV MMAs, 10-15 unpack pages of K
// and V in turn.  The launch gives every thread
// 128 registers, 65,536 in all; the softmax threads take 176 (bf16: 160) of them
// and the others 80 (96).
constexpr int kSoftWarps = 8, kWQk = 8, kWPv = 9, kWLoad = 10, kUnpackWarps = 6;
constexpr int kPattnThreads = 512;

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

using f2 = unsigned long long;                      // two floats for the packed fp32 instructions
// binary16 parts of a pair: hi nearest, lo what is left (the first in the low half)
SPEC_DEV void split_pair(f2 x, uint32_t& hi, uint32_t& lo) {
  float x0, x1, r0, r1;
  f2unpack(x, x0, x1);
  const __half2 h = __floats2half2_rn(x0, x1);
  const float2 f = __half22float2(h);
  f2unpack(f2sub(x, f2pack(f.x, f.y)), r0, r1);
  const __half2 l = __floats2half2_rn(r0, r1);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}
// 32 consecutive TMEM columns of this warp's 32 lanes, as pairs (to be waited for)
SPEC_DEV void tmem_ld32_f2(uint32_t taddr, f2* v) {
  uint32_t r[32];
  tmem_ld32(taddr, r);
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = f2pack(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
}
SPEC_DEV void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]));
}

SPEC_DEV void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]));
}

// wait for a phase, giving up after kPattnWaitNs
SPEC_DEV bool mbar_wait(uint64_t* mbar, uint32_t parity) {
#pragma unroll 1
  for (int i = 0; i < 64; ++i) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(smem_u32(mbar)), "r"(parity)
        : "memory");
    if (done) return true;
  }
  return mbar_wait_ns(mbar, parity, kPattnWaitNs);
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

// loads issued where they stand (a plain load may be moved down to its use,
// behind a wait)
SPEC_DEV uint4 ldg_now(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
SPEC_DEV uint32_t ldg_now(const void* p) {
  uint32_t v;
  asm volatile("ld.global.nc.u32 %0, [%1];\n" : "=r"(v) : "l"(p));
  return v;
}
SPEC_DEV int page_at(const KvView& kv, int lp) {
  const int page = lp < kv.max_seq_pages ? (int)ldg_now((const void*)(kv.page_table + lp)) : -1;
  return page < kv.num_pages ? page : -1;
}

// One page of a tile as an unpacking warp holds it.
// 4-bit: lane = key % 16 + 16 * d half; 64 codes and 4 scale bytes of K or V.
struct Raw4 {
  uint4 c[2];
  uint32_t s;
};
// base: this lane's first chunk of page 0 of the layer and head; stride: bytes
// of a page of the pool
SPEC_DEV void load_page(const uint8_t* base, uint32_t stride, int page, int scales, Raw4& r) {
  if (page < 0) {                                        // unmapped: zeros (its keys are masked)
    r.c[0] = r.c[1] = make_uint4(0, 0, 0, 0);
    r.s = 0;
    return;
  }
  const uint8_t* p = base + (uint64_t)(uint32_t)page * stride;
  r.c[0] = ldg_now(reinterpret_cast<const uint4*>(p));
  r.c[1] = ldg_now(reinterpret_cast<const uint4*>(p + 256));
  r.s = ldg_now((const void*)(p + scales));
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
SPEC_DEV void load_rows(const uint4* base, uint32_t stride, int page, Raw16& r) {
  if (page < 0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) r.x[j] = make_uint4(0, 0, 0, 0);
    return;
  }
  const uint4* p = base + (uint64_t)(uint32_t)page * stride;
#pragma unroll
  for (int j = 0; j < 8; ++j) r.x[j] = ldg_now(p + 32 * j);
}
// bf16 pair as binary16; |x| >= 2^15, infinities and NaN are the caller's business
SPEC_DEV uint32_t bf16x2_to_f16x2(uint32_t w) {
  const __half2 h = __floats2half2_rn(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return *reinterpret_cast<const uint32_t*>(&h);
}
constexpr uint32_t kBf16Limit = 0x4700u;            // bf16 bits of 2^15

// ---------------------------------------------------------------------------
// partials: grid (slot, KV head, row tile)
// ---------------------------------------------------------------------------
template <bool k4>
__global__ void __launch_bounds__(kPattnThreads, 1)
pattn_kernel(const float* __restrict__ q, PattnPlan pl, KvView kv, int layer, float* __restrict__ part_o,
             float2* __restrict__ part_ml, int32_t* status) {
  extern __shared__ __align__(128) uint8_t dsm[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dsm) + 1023) & ~(uintptr_t)1023);
  __shared__ uint32_t tmem_slot;
  __shared__ __align__(8) uint64_t q_full, k_full[kStages], v_full[kStages], k_free[kStages], v_free[kStages],
      s_full[2], p_full[2], pv_done[2];
  __shared__ float pair[2][128];                        // what the two threads of a row exchange
  // per tile (a ring of 8: a tile's entries are rewritten eight tiles later,
  // when its softmax has long been passed): mapped pages, and for bf16 the keys
  // whose K or V has an element out of range
  __shared__ __align__(16) uint16_t odd[2][8][kPagesPerTile];
  __shared__ __align__(8) uint8_t mapped[8][kPagesPerTile];
  __shared__ int gave_up[4];                            // a wait of this pair of softmax warps ran out

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slot = blockIdx.x, kvh = blockIdx.y, R = pl.M * pl.group;
  const int r0 = blockIdx.z * pl.tile_rows, nr = min(pl.tile_rows, R - r0);
  const int row_warps = (nr + 31) >> 5;                 // pairs of softmax warps with rows
  if (warp == kWQk) tmem_alloc(&tmem_slot, kTmAll);
  if (tid == 32 * kWPv) {
    mbar_init(&q_full, 2 * row_warps);
    for (int b = 0; b < kStages; ++b) {
      mbar_init(&k_full[b], kPagesPerTile);
      mbar_init(&v_full[b], kPagesPerTile);
      mbar_init(&k_free[b], 1);
      mbar_init(&v_free[b], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&s_full[b], 1);
      mbar_init(&p_full[b], 2 * row_warps);
      mbar_init(&pv_done[b], 1);
    }
    for (int g = 0; g < 4; ++g) gave_up[g] = 0;
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
  // (total == 0: nothing of this chunk is seen)
  if (warp >= kSoftWarps) {
  if constexpr (k4)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;\n");
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 96;\n");
  if (total == 0) {
  } else if (warp >= kWLoad) {
    // -------------------------------------------------------------- unpack
    // item g is page g % 8 of tile g / 8; this warp takes every sixth
    const int items = total * kPagesPerTile, g0 = warp - kWLoad;
    auto page_of = [&](int g) { return g < items ? page_at(kv, tile_at(g >> 3) * kPagesPerTile + (g & 7)) : -1; };
    auto free_k = [&](int it) {
      return it < kStages || __all_sync(0xffffffffu, mbar_wait(&k_free[it % kStages], ((it / kStages) - 1) & 1));
    };
    auto free_v = [&](int it) {
      return it < kStages || __all_sync(0xffffffffu, mbar_wait(&v_free[it % kStages], ((it / kStages) - 1) & 1));
    };
    auto done = [&](uint64_t* bar) {
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    bool ok = true;
    if constexpr (k4) {
      // K runs one item ahead of V, whose stage is freed later; the registers
      // hold the next item of each besides
      const int t = lane & 15, half = lane >> 4;
      auto row_of = [&](int g) {
        return sm + (size_t)((g >> 3) % kStages) * kStageBytes + half * kHalf + (16 * (g & 7) + t) * 128;
      };
      auto put_k = [&](int g, const Raw4& r, int page) {
        if (!free_k(g >> 3)) return false;
        unpack_row(r.c, r.s, row_of(g), t & 7);
        if (lane == 0) mapped[(g >> 3) & 7][g & 7] = page >= 0;
        done(&k_full[(g >> 3) % kStages]);
        return true;
      };
      auto put_v = [&](int g, const Raw4& r) {
        if (!free_v(g >> 3)) return false;
        unpack_row(r.c, r.s, row_of(g) + 2 * kHalf, t & 7);
        done(&v_full[(g >> 3) % kStages]);
        return true;
      };
      const uint32_t stride = (uint32_t)(kv.n_layers * 2 * kv.n_kv) * kKv4PageBytes;
      const uint8_t* kb0 = reinterpret_cast<const uint8_t*>(kv.pool) +
                           (size_t)(layer * 2 * kv.n_kv + kvh) * kKv4PageBytes + kv4_chunk(t, 2 * half);
      const uint8_t* vb0 = kb0 + kv.n_kv * kKv4PageBytes;
      const int scales = kKv4Scales + 8 * t + 4 * half - kv4_chunk(t, 2 * half);
      Raw4 ka, kb, va, vb;
      const int p0 = page_of(g0), p1 = page_of(g0 + kUnpackWarps);
      // the pages whose K is next, loaded next and loaded after that: a page
      // id is fetched a step before its page
      int held = p1, next = page_of(g0 + 2 * kUnpackWarps), after = page_of(g0 + 3 * kUnpackWarps);
      load_page(kb0, stride, p0, scales, ka);
      load_page(kb0, stride, p1, scales, kb);
      load_page(vb0, stride, p0, scales, va);
      load_page(vb0, stride, p1, scales, vb);
      if (g0 < items) ok = put_k(g0, ka, p0);
      // one item: V of g, K of the item after it (whose K is in kn), loads of
      // the item after that into the registers that become free
      auto step = [&](int g, Raw4& vg, Raw4& kg, const Raw4& kn) {
        const int id = page_of(g + 4 * kUnpackWarps);
        load_page(kb0, stride, next, scales, kg);       // kg's page has been unpacked
        if (g + kUnpackWarps < items && !put_k(g + kUnpackWarps, kn, held)) return false;
        if (!put_v(g, vg)) return false;
        load_page(vb0, stride, next, scales, vg);
        held = next;
        next = after;
        after = id;
        return true;
      };
      for (int g = g0; ok && g < items; g += 2 * kUnpackWarps) {
        ok = step(g, va, ka, kb);
        if (ok && g + kUnpackWarps < items) ok = step(g + kUnpackWarps, vb, kb, ka);
      }
    } else {
      // registers hold the next item of K and of V
      Raw16 k, v;
      // (16-byte units; a page of one head is 256 of them)
      const uint32_t stride = (uint32_t)(kv.n_layers * 2 * kv.n_kv) * 256u;
      const uint4* kb0 = reinterpret_cast<const uint4*>(kv.pool) + (size_t)(layer * 2 * kv.n_kv + kvh) * 256 + lane;
      const uint4* vb0 = kb0 + kv.n_kv * 256;
      // the pages in v, in k, and of the K after that
      int page = page_of(g0), next = page_of(g0 + kUnpackWarps), after = page_of(g0 + 2 * kUnpackWarps);
      load_rows(kb0, stride, page, k);
      load_rows(vb0, stride, page, v);
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
      // K runs one item ahead of V, whose stage is freed later
      auto put_k = [&](int g, int pg) {
        const uint32_t far = put(k, (g >> 3) % kStages, g & 7, 0, tile_at(g >> 3) * kKeys, pg >= 0);
        if (lane == 0) {
          mapped[(g >> 3) & 7][g & 7] = pg >= 0;
          odd[0][(g >> 3) & 7][g & 7] = (uint16_t)far;
        }
        done(&k_full[(g >> 3) % kStages]);
      };
      if (g0 < items) put_k(g0, page);
      load_rows(kb0, stride, next, k);
      for (int g = g0; g < items; g += kUnpackWarps) {
        const int it = g >> 3, st = it % kStages, gn = g + kUnpackWarps, id = page_of(gn + 2 * kUnpackWarps);
        if (gn < items) {
          ok = free_k(gn >> 3);
          if (!ok) break;
          put_k(gn, next);
          load_rows(kb0, stride, after, k);
        }
        ok = free_v(it);
        if (!ok) break;
        const uint32_t far = put(v, st, g & 7, 1, tile_at(it) * kKeys, page >= 0);
        if (lane == 0) odd[1][it & 7][g & 7] = (uint16_t)far;
        done(&v_full[st]);
        load_rows(vb0, stride, next, v);
        page = next;
        next = after;
        after = id;
      }
    }
    if (!ok && lane == 0) atomicOr(status, SPEC_ST_DEVICE_WAIT);
  } else if (warp == kWQk) {
    // ------------------------------------------------------------ S = Q . K^T
    // D f32 (bit 4), A and B f16, N >> 3 at 17, M >> 4 at 24; 8 d steps of 16,
    // the low parts of Q first
    constexpr uint32_t kId = (1u << 4) | ((kKeys >> 3) << 17) | ((128u >> 4) << 24);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t dk0 = desc_sw128(__shfl_sync(0xffffffffu, smem_u32(sm), 0), 16, 1024);
    bool ok = __all_sync(0xffffffffu, mbar_wait(&q_full, 0));
    int last = -1;
    for (int it = 0; ok && it < total; ++it) {
      const int st = it % kStages, sb = it & 1;
      bool w = mbar_wait(&k_full[st], (it / kStages) & 1);
      // the buffer's P of two tiles ago has been read
      if (it >= 2) w = w && mbar_wait(&pv_done[sb], ((it >> 1) - 1) & 1);
      ok = __all_sync(0xffffffffu, w);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t dk = dk0 + (uint64_t)((st * kStageBytes) >> 4);
#pragma unroll
        for (int pt = 1; pt >= 0; --pt)
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            mma_f16_ts(tm + kTmS + 128u * sb, tm + kTmQ + 64u * pt + 8u * ks,
                       dk + (uint64_t)(((ks >> 2) * kHalf + (ks & 3) * 32) >> 4), kId, pt == 0 || ks != 0);
        mma_commit(&s_full[sb]);
        mma_commit(&k_free[st]);
      }
      __syncwarp();
      last = it;
    }
    if (!ok && lane == 0) atomicOr(status, SPEC_ST_DEVICE_WAIT);
    if (last >= 0) mbar_wait(&s_full[last & 1], (last >> 1) & 1);   // before TMEM is released
  } else {
    // ------------------------------------------------------------ O = P . V
    // key steps of 16; V MN-major (bit 16): lbo = the d-half stride, sbo = 1 KB
    // between 8-key groups; the low parts of P first
    constexpr uint32_t kId = (1u << 4) | (1u << 16) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t dv0 = desc_sw128(__shfl_sync(0xffffffffu, smem_u32(sm), 0) + 2 * kHalf, kHalf, 1024);
    bool ok = true;
    int last = -1;
    for (int it = 0; ok && it < total; ++it) {
      const int st = it % kStages, sb = it & 1;
      ok = __all_sync(0xffffffffu, mbar_wait(&v_full[st], (it / kStages) & 1) && mbar_wait(&p_full[sb], (it >> 1) & 1));
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t dv = dv0 + (uint64_t)((st * kStageBytes) >> 4);
#pragma unroll
        for (int pt = 1; pt >= 0; --pt)
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_f16_ts(tm + kTmO, tm + kTmS + 128u * sb + 32u * (kk >> 1) + 16u * pt + 8u * (kk & 1),
                       dv + (uint64_t)((kk * 2048) >> 4), kId, pt == 0 || kk != 0);
        mma_commit(&pv_done[sb]);
        mma_commit(&v_free[st]);
      }
      __syncwarp();
      last = it;
    }
    if (!ok && lane == 0) atomicOr(status, SPEC_ST_DEVICE_WAIT);
    if (last >= 0) mbar_wait(&pv_done[last & 1], (last >> 1) & 1);
  }
  } else {
  if constexpr (k4)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 176;\n");
  else
    asm volatile("setmaxnreg.inc.sync.aligned.u32 160;\n");
  if (total > 0 && (warp & 3) < row_warps) {
    // ------------------------------------------------------------ softmax
    const int h = warp >> 2, ww = warp & 3;
    const int r = 32 * ww + lane, fr = r0 + r;          // tile row, row of the KV head
    const bool live = r < nr;
    const int i = live ? fr / pl.group : 0, hd = live ? fr - i * pl.group : 0;
    const uint32_t tl = tmem + ((uint32_t)(32 * ww) << 16);
    constexpr float kBias = 7.f;                        // p = 2^(7 + s - max): binary16 keeps 2^-24 of 2^7
    const float* qr = q + ((size_t)i * pl.nq + kvh * pl.group + hd) * 128;
    // one lane arrives for the warp: the warp barrier orders the others' writes
    auto arrive = [&](uint64_t* bar) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    // log2(e) / sqrt(d) times the row's power of two: scores in base-2 units
    float unit = 1.4426950408889634f / sqrtf(128.0f);
    {
      // the row is scaled by a power of two to at most 2 in magnitude, and the
      // scores are scaled back
      float4 y[16];
      float mx = 0.f;
#pragma unroll
      for (int d = 0; d < 16; ++d) {
        y[d] = live ? reinterpret_cast<const float4*>(qr)[16 * h + d] : make_float4(0.f, 0.f, 0.f, 0.f);
        mx = fmaxf(mx, fmaxf(fmaxf(fabsf(y[d].x), fabsf(y[d].y)), fmaxf(fabsf(y[d].z), fabsf(y[d].w))));
      }
      pair[h][r] = mx;
      named_bar(1 + ww, 64);
      mx = fmaxf(mx, pair[1 - h][r]);
      const int e = min(max((int)((__float_as_uint(mx) >> 23) & 255u) - 127, -100), 100);
      const float mul = __uint_as_float((uint32_t)(127 - e) << 23);
      unit *= __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int d = 0; d < 8; ++d) {
          split_pair(f2pack(y[8 * c + d].x * mul, y[8 * c + d].y * mul), hi[2 * d], lo[2 * d]);
          split_pair(f2pack(y[8 * c + d].z * mul, y[8 * c + d].w * mul), hi[2 * d + 1], lo[2 * d + 1]);
        }
        tmem_st16(tl + kTmQ + 32u * h + 16u * c, hi);
        tmem_st16(tl + kTmQ + 64u + 32u * h + 16u * c, lo);
      }
      tmem_wait_st();
      tc_fence_before();
      arrive(&q_full);
    }
    const int p = n_past + i, plow = window_low(pl, p);
    bool ok = true, left = false;
    int it = 0;
#pragma unroll 1
    for (int pass = 0; !left && pass < passes; ++pass) {
      const Span sp = span_of(pl, n_past, pass);
      const bool mine = live && i >= sp.i0 && i < sp.i1;
      const int n = pass == 0 ? tl0.n : tl1.n;
      f2 acc[32];                                       // O of this row, d's 64 h .., in pairs
#pragma unroll
      for (int c = 0; c < 32; ++c) acc[c] = f2pack(0.f, 0.f);
      float ref = -INFINITY, lsum = 0.f;                // reference of the exponents (both threads agree)
      bool pending = false;                             // O of tile it - 1 is not in acc yet
      auto drain = [&]() -> bool {
        pending = false;
        if (!__all_sync(0xffffffffu, mbar_wait(&pv_done[(it - 1) & 1], ((it - 1) >> 1) & 1))) return false;
        tc_fence_after();
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          f2 o[16];
          tmem_ld32_f2(tl + kTmO + 64u * h + 32u * g, o);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 16; ++c) acc[16 * g + c] = f2add(acc[16 * g + c], o[c]);
        }
        return true;
      };
#pragma unroll 1
      for (int sc = 0; sc < n; ++sc, ++it) {
        const int sb = it & 1, st = it % kStages, t0 = tile_at(it) * kKeys;
        bool got = __all_sync(0xffffffffu, mbar_wait(&s_full[sb], (it >> 1) & 1));
        tc_fence_after();
        const uint32_t sa = tl + kTmS + 128u * sb + 64u * h;
        f2 x[32];                                       // scores of keys t0 + 64 h ..
        tmem_ld32_f2(sa, x);
        tmem_ld32_f2(sa + 32u, x + 16);
        // `masked`: some row of the block does not see some key of the tile
        const uint2 mp = *reinterpret_cast<const uint2*>(&mapped[it & 7][0]);
        const bool masked = (mp.x & mp.y) != 0x01010101u || t0 + kKeys - 1 > n_past || (t0 < low1 && t0 + kKeys > sinks) ||
                            passes > 1;
        tmem_wait_ld();
        if (!k4) {
          // keys with an element past binary16: their scores in fp32
          const uint2 m = *reinterpret_cast<const uint2*>(&odd[0][it & 7][4 * h]);
          if (m.x | m.y) {
#pragma unroll 1
            for (int c = 0; c < 64; ++c) {
              if (!(((c < 32 ? m.x : m.y) >> (c & 31)) & 1u)) continue;
              const int t = t0 + 64 * h + c;
              const uint16_t* kr = kv.pool + ((((size_t)page_at(kv, t >> 4) * kv.n_layers + layer) * 2) * kv.n_kv + kvh) * 2048 +
                                   (t & 15) * 128;
              float y = 0.f;
#pragma unroll 4
              for (int d = 0; d < 128; ++d) y = fmaf(qr[d], __uint_as_float((uint32_t)kr[d] << 16), y);
              y *= (1.4426950408889634f / sqrtf(128.0f)) / unit;
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                float a, b;
                f2unpack(x[e], a, b);
                x[e] = f2pack(2 * e == c ? y : a, 2 * e + 1 == c ? y : b);
              }
            }
          }
        }
        if (masked) {
          // keys of this thread that its row sees
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int k0 = t0 + 64 * h + 32 * c;
            const uint32_t two = (h ? mp.y : mp.x) >> (16 * c);
            const uint32_t vis = !mine ? 0u
                                       : low_bits(p + 1 - k0) & (~low_bits(plow - k0) | low_bits(sinks - k0)) &
                                             ((two & 1u ? 0xffffu : 0u) | (two & 0x100u ? 0xffff0000u : 0u));
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float a, b;
              f2unpack(x[16 * c + e], a, b);
              x[16 * c + e] = f2pack((vis >> (2 * e)) & 1u ? a : -INFINITY, (vis >> (2 * e + 1)) & 1u ? b : -INFINITY);
            }
          }
        }
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          float a, b;
          f2unpack(x[e], a, b);
          m4[e & 3] = fmaxf(m4[e & 3], fmaxf(a, b));
        }
        float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * unit;
        // The reference moves only when a score exceeds it by more than 8 (p
        // would exceed 2^15).  A wait that ran out is carried to this barrier,
        // where the pair of warps leaves together.
        if (!got || !ok) *reinterpret_cast<volatile int*>(&gave_up[ww]) = 1;
        if (named_bar_or(1 + ww, 64, mx > ref + 8.f || !got || !ok)) {
          left = *reinterpret_cast<volatile int*>(&gave_up[ww]) != 0;
          if (left) break;
          pair[h][r] = mx;
          named_bar(1 + ww, 64);
          mx = fmaxf(mx, pair[1 - h][r]);
          if (pending) ok = drain();                    // O so far is in the old units
          if (mx > ref + 8.f) {
            const float a = ref == -INFINITY ? 1.f : exp2_approx(ref - mx);
            ref = mx;
            lsum *= a;
            const f2 a2 = f2pack(a, a);
#pragma unroll
            for (int c = 0; c < 32; ++c) acc[c] = f2mul(acc[c], a2);
          }
        }
        const float base = kBias - (ref == -INFINITY ? 0.f : ref);
        const f2 un = f2pack(unit, unit), bs = f2pack(base, base);
        f2 sum = f2pack(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < 4; ++c) {                   // 16 keys each
          uint32_t hi[8], lo[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float a, b;
            f2unpack(f2fma(x[8 * c + e], un, bs), a, b);
            x[8 * c + e] = f2pack(exp2_approx(a), exp2_approx(b));
            sum = f2add(sum, x[8 * c + e]);
            split_pair(x[8 * c + e], hi[e], lo[e]);
          }
          tmem_st8(sa + 32u * (c >> 1) + 8u * (c & 1), hi);
          tmem_st8(sa + 32u * (c >> 1) + 8u * (c & 1) + 16u, lo);
        }
        float s0, s1;
        f2unpack(sum, s0, s1);
        lsum += s0 + s1;
        if (!k4) {
          // V elements past binary16 are zero in the tile: their p v is added
          // here in fp32, to the rows that see them
          got = __all_sync(0xffffffffu, mbar_wait(&v_full[st], (it / kStages) & 1));
          const uint4 m = *reinterpret_cast<const uint4*>(&odd[1][it & 7][0]);
          if (!got || !ok) *reinterpret_cast<volatile int*>(&gave_up[ww]) = 1;
          if (named_bar_or(1 + ww, 64, (m.x | m.y | m.z | m.w) != 0 || !got || !ok)) {
            left = *reinterpret_cast<volatile int*>(&gave_up[ww]) != 0;
            if (left) break;
            const uint32_t mw[4] = {m.x, m.y, m.z, m.w};
#pragma unroll 1
            for (int k = 0; k < kKeys; ++k) {
              if (!((mw[k >> 5] >> (k & 31)) & 1u)) continue;
              const int t = t0 + k;
              if ((k >> 6) == h) {
                float y = 0.f;
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                  float a, b;
                  f2unpack(x[e], a, b);
                  if (2 * e == (k & 63)) y = a;
                  if (2 * e + 1 == (k & 63)) y = b;
                }
                pair[0][r] = mine && t <= p && (t >= plow || t < sinks) ? y : -1.f;
              }
              named_bar(1 + ww, 64);
              const float y = pair[0][r];
              const uint16_t* vr = kv.pool + ((((size_t)page_at(kv, t >> 4) * kv.n_layers + layer) * 2 + 1) * kv.n_kv + kvh) * 2048 +
                                   (t & 15) * 128 + 64 * h;
              if (!(y < 0.f)) {
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                  float a, b;
                  f2unpack(acc[c], a, b);
                  const uint32_t w0 = vr[2 * c], w1 = vr[2 * c + 1];
                  if ((w0 & 0x7FFFu) >= kBf16Limit) a += y * __uint_as_float(w0 << 16);
                  if ((w1 & 0x7FFFu) >= kBf16Limit) b += y * __uint_as_float(w1 << 16);
                  acc[c] = f2pack(a, b);
                }
              }
              named_bar(1 + ww, 64);
            }
          }
        }
        // O may be rewritten once the tile before has been added up
        if (pending) ok = ok && drain();
        pending = true;
        tmem_wait_st();
        tc_fence_before();
        if (ok) arrive(&p_full[sb]);
      }
      if (left || n == 0) continue;
      ok = ok && drain();
      pair[h][r] = lsum;
      if (!ok) *reinterpret_cast<volatile int*>(&gave_up[ww]) = 1;
      named_bar(1 + ww, 64);
      left = *reinterpret_cast<volatile int*>(&gave_up[ww]) != 0;
      if (left) break;
      const size_t at = ((size_t)slot * pl.nkv + kvh) * R + fr;
      if (mine) {
        if (h == 0) part_ml[at] = make_float2(ref - kBias, lsum + pair[1][r]);
        float4* dst = reinterpret_cast<float4*>(part_o + at * 128 + 64 * h);
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          float4 y;
          f2unpack(acc[2 * c], y.x, y.y);
          f2unpack(acc[2 * c + 1], y.z, y.w);
          dst[c] = y;
        }
      }
      named_bar(1 + ww, 64);                            // `pair` is free
    }
    if (left && lane == 0) atomicOr(status, SPEC_ST_DEVICE_WAIT);
  }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWQk) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmAll);
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
  constexpr int kBatch = 16;                            // loads in flight
  for (int c0 = 0; c0 < n; c0 += kBatch) {
    float4 y[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (c0 + k < n) y[k] = reinterpret_cast<const float4*>(part_o + (at + (c0 + k) * stride) * 128)[lane];
    const float2 x = lane < kBatch && c0 + lane < n ? part_ml[at + (c0 + lane) * stride] : make_float2(0.f, 0.f);
    const float wl = x.y != 0.f ? exp2f(x.x - m) : 0.f;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const float w = __shfl_sync(0xffffffffu, wl, k), l = __shfl_sync(0xffffffffu, x.y, k);
      if (c0 + k < n && l != 0.f) {
        L += w * l;
        o.x += w * y[k].x;
        o.y += w * y[k].y;
        o.z += w * y[k].z;
        o.w += w * y[k].w;
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

template <bool k4>
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
    e = cudaFuncSetAttribute(pattn_kernel<k4>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPattnSmem);
    if (e != cudaSuccess) return e;
    if (known) have[dev] = true;
  }
  pattn_kernel<k4><<<dim3(pl.slots, pl.nkv, row_tiles), kPattnThreads, kPattnSmem, st>>>(q, pl, kv, layer, part_o, part_ml,
                                                                                        status);
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
  const int R = M * pl.group, row_tiles = (R + 127) / 128;
  pl.tile_rows = (R + row_tiles - 1) / row_tiles;
  float2* ml = reinterpret_cast<float2*>(part);        // [slots][nkv][R], then the outputs
  float* po = part + 2 * (size_t)pl.C * nq * 16;
  cudaError_t e = k4 ? launch_pattn<true>(pl, kv, layer, q, row_tiles, po, ml, status, st)
                     : launch_pattn<false>(pl, kv, layer, q, row_tiles, po, ml, status, st);
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
