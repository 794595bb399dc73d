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
//   S[128 x 128 keys]  = Q[128 x 128 d] . K^T     (A = Q in TMEM, B = K)
//   O[128 x 128 d]    += P[128 x 128 keys] . V    (A = P in TMEM, B = V)
// with a running (max, sum) per row and O accumulated in TMEM.  A CTA (slot, KV
// head, row tile) walks one chunk of L key tiles and writes (O, max, sum); a
// merge kernel joins the chunks in order.
//
// The split of the keys is a function of the row's own position alone (chunk_len
// below): chunks are whole multiples of L tiles from position 0, so a row has
// the same bits alone and in any block (batch-height invariance).  L grows
// with the position such that there are never more chunks than SMs per KV head;
// a block that crosses such a step runs its two groups of rows one after the
// other.  Tiles that no row sees are skipped: they would add exact zeros.
//
// Precision: K and V are exact operands (bf16, or binary16 for the 4-bit
// cache); q and p are split into two operand-precision parts (two MMAs each),
// 16 (bf16) or 22 (binary16) significant bits; accumulation is fp32.
#include "attn_mma.cuh"
#include "common.cuh"
#include "internal.h"
#include "kv4.cuh"

namespace spec {

constexpr int kKeys = 128;                          // keys of a tile
constexpr int kPagesPerTile = kKeys / 16;
constexpr int kHalf = kKeys * 128;                  // one d half of a K or V tile: [keys][64 values]
constexpr int kStageBytes = 4 * kHalf;              // K then V, 64 KB
constexpr int kStages = 3;
constexpr size_t kPattnSmem = 1024 + (size_t)kStages * kStageBytes;
// TMEM columns: two score buffers, each overwritten in place by its P parts;
// O; Q (64 columns of hi parts, then 64 of lo parts)
constexpr uint32_t kTmS0 = 0, kTmO0 = 256, kTmQ0 = 384;
constexpr int kTmAll = 512;
constexpr uint64_t kPattnWaitNs = 2000000000ull;

// warps: 0-3 own one tile row per thread (softmax, O rescale, partials), 4
// issues the QK MMAs, 5 the PV MMAs; bf16: 6 copies K and 7 V pages by TMA;
// 4-bit: 6-13 unpack one page of K and V each
constexpr int kWQk = 4, kWPv = 5, kWLoad = 6, kUnpackWarps = 8;
template <bool k4>
constexpr int pattn_warps() { return k4 ? kWLoad + kUnpackWarps : kWLoad + 2; }

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

// (x0, x1) rounded to the operand type, packed with x0 in the low half, and
// what the rounding left
template <bool k4>
SPEC_DEV uint32_t pack_hi(float x0, float x1, float& r0, float& r1) {
  if (k4) {
    const __half2 h = __floats2half2_rn(x0, x1);
    const float2 f = __half22float2(h);
    r0 = x0 - f.x;
    r1 = x1 - f.y;
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(x0, x1);
  const uint32_t u = *reinterpret_cast<const uint32_t*>(&h);
  r0 = x0 - __uint_as_float(u << 16);
  r1 = x1 - __uint_as_float(u & 0xFFFF0000u);
  return u;
}
template <bool k4>
SPEC_DEV uint32_t pack_lo(float x0, float x1) {
  if (k4) {
    const __half2 h = __floats2half2_rn(x0, x1);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(x0, x1);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// 16 operand pairs of 32 values: hi parts and lo parts
template <bool k4>
SPEC_DEV void split32(const float (&x)[32], uint32_t (&hi)[16], uint32_t (&lo)[16]) {
#pragma unroll
  for (int c = 0; c < 16; ++c) {
    float r0, r1;
    hi[c] = pack_hi<k4>(x[2 * c], x[2 * c + 1], r0, r1);
    lo[c] = pack_lo<k4>(r0, r1);
  }
}
SPEC_DEV void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]));
}

SPEC_DEV int page_at(const KvView& kv, int lp) {
  const int page = lp < kv.max_seq_pages ? __ldg(kv.page_table + lp) : -1;
  return page < kv.num_pages ? page : -1;
}

// One page of a tile as an unpacking warp holds it: lane = key % 16 + 16 * d
// half; 64 codes and 4 scale bytes of K and of V
struct RawPage {
  uint4 k[2], v[2];
  uint32_t ks, vs;
};
SPEC_DEV void load_page(const KvView& kv, int layer, int kvh, int page, int lane, RawPage& r) {
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

// ---------------------------------------------------------------------------
// partials: grid (slot, KV head, row tile)
// ---------------------------------------------------------------------------
template <bool k4>
__global__ void __launch_bounds__(32 * pattn_warps<k4>(), 1)
pattn_kernel(const float* __restrict__ q, PattnPlan pl, KvView kv, const __grid_constant__ CUtensorMap kvmap, int layer,
             float* __restrict__ part_o, float2* __restrict__ part_ml, int32_t* status) {
  extern __shared__ __align__(128) uint8_t dsm[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dsm) + 1023) & ~(uintptr_t)1023);
  __shared__ uint32_t tmem_slot, poison;
  __shared__ __align__(8) uint64_t q_full, k_full[kStages], v_full[kStages], k_free[kStages], v_free[kStages],
      s_full[2], p_full[2], pv_done[2];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slot = blockIdx.x, kvh = blockIdx.y, R = pl.M * pl.group;
  const int r0 = blockIdx.z * pl.tile_rows, nr = min(pl.tile_rows, R - r0);
  const int row_warps = (nr + 31) >> 5;                 // softmax warps with rows
  if (warp == 0) tmem_alloc(&tmem_slot, kTmAll);
  if (tid == 32) {
    mbar_init(&q_full, 32 * row_warps);
    for (int b = 0; b < kStages; ++b) {
      mbar_init(&k_full[b], k4 ? kUnpackWarps : 1);
      mbar_init(&v_full[b], k4 ? kUnpackWarps : 1);
      mbar_init(&k_free[b], 1);
      mbar_init(&v_free[b], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&s_full[b], 1);
      mbar_init(&p_full[b], 128);
      mbar_init(&pv_done[b], 1);
    }
    poison = 0;
    fence_mbarrier_init();
  }
  pdl_trigger();
  pdl_wait();
  const int n_past = __ldcg(kv.seq_len) - pl.M;
  const int passes = span_count(pl, n_past);
  TileList tl[2];
  tl[0] = tiles_of(span_of(pl, n_past, 0), slot);
  if (passes == 2) tl[1] = tiles_of(span_of(pl, n_past, 1), slot);
  const int total = tl[0].n + tl[1].n;
  auto tile_at = [&](int it) { return it < tl[0].n ? tl[0].at(it) : tl[1].at(it - tl[0].n); };
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  if (total == 0) {
    // nothing of this chunk is seen
  } else if (warp >= kWLoad) {
    if (k4) {
      // ------------------------------------------------------------ unpack
      // registers hold the pages of the next two tiles: with 8 warps about
      // 36 KB per SM in flight
      const int w = warp - kWLoad, t = lane & 15, half = lane >> 4;
      const int key = 16 * w + t;
      auto page_of = [&](int it) { return it < total ? page_at(kv, tile_at(it) * kPagesPerTile + w) : -1; };
      RawPage a, b;
      load_page(kv, layer, kvh, page_of(0), lane, a);
      load_page(kv, layer, kvh, page_of(1), lane, b);
      int next = page_of(2);
      auto put = [&](int it, RawPage& r) -> bool {
        const int st = it % kStages;
        uint8_t* row = sm + (size_t)st * kStageBytes + half * kHalf + key * 128;
        if (it >= kStages && !__all_sync(0xffffffffu, mbar_wait_ns(&k_free[st], ((it / kStages) - 1) & 1, kPattnWaitNs)))
          return false;
        unpack_row(r.k, r.ks, row, key & 7);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&k_full[st]);
        if (it >= kStages && !__all_sync(0xffffffffu, mbar_wait_ns(&v_free[st], ((it / kStages) - 1) & 1, kPattnWaitNs)))
          return false;
        unpack_row(r.v, r.vs, row + 2 * kHalf, key & 7);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_full[st]);
        const int page = next;
        next = page_of(it + 3);
        load_page(kv, layer, kvh, page, lane, r);       // tile it + 2
        return true;
      };
      bool ok = true;
      for (int it = 0; ok && it < total; it += 2) {
        ok = put(it, a);
        if (ok && it + 1 < total) ok = put(it + 1, b);
      }
      if (!ok && lane == 0) atomicOr(status, SPEC_ST_DEVICE_WAIT);
    } else if (warp < kWLoad + 2) {
      // ------------------------------------------------------------ copies
      // lane l < 16: page l / 2, d half l % 2
      const int which = warp - kWLoad, pp = (lane >> 1) & 7, half = lane & 1;
      uint64_t* full = which ? v_full : k_full;
      uint64_t* freed = which ? v_free : k_free;
      if (lane == 0) asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&kvmap)) : "memory");
      bool ok = true;
      int issued = 0;
      int page = page_at(kv, tile_at(0) * kPagesPerTile + pp);
      for (int it = 0; it < total; ++it) {
        const int st = it % kStages;
        const int next = it + 1 < total ? page_at(kv, tile_at(it + 1) * kPagesPerTile + pp) : -1;
        if (it >= kStages)
          ok = __all_sync(0xffffffffu, mbar_wait_ns(&freed[st], ((it / kStages) - 1) & 1, kPattnWaitNs));
        if (!ok) break;
        // pages past the last key are masked, not copied
        const bool go = lane < 16 && page >= 0 && tile_at(it) * kKeys + 16 * pp < n_past + pl.M;
        const uint32_t ops = __popc(__ballot_sync(0xffffffffu, go));
        if (lane == 0) mbar_arrive_expect_tx(&full[st], ops * 2048u);
        __syncwarp();
        if (go)
          tma_load_2d(sm + (size_t)st * kStageBytes + (2 * which + half) * kHalf + pp * 2048, &kvmap, 64 * half,
                      (((page * kv.n_layers + layer) * 2 + which) * kv.n_kv + kvh) * 16, &full[st]);
        issued = it + 1;
        page = next;
      }
      if (!ok && lane == 0) atomicOr(status, SPEC_ST_DEVICE_WAIT);
      // no copy may still be writing shared memory when the CTA exits
      if (lane == 0)
        for (int x = max(0, issued - kStages); x < issued; ++x)
          mbar_wait_ns(&full[x % kStages], (x / kStages) & 1, kPattnWaitNs);
    }
  } else if (warp == kWQk) {
    // ------------------------------------------------------------ S = Q . K^T
    // D f32 (bit 4); A, B bf16 (bits 7, 10) or f16; N >> 3 at 17, M >> 4 at 24;
    // 8 d steps of 16, hi and lo parts of Q
    constexpr uint32_t kId = (1u << 4) | (k4 ? 0u : (1u << 7) | (1u << 10)) | ((kKeys >> 3) << 17) | ((128u >> 4) << 24);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t dk0 = desc_sw128(__shfl_sync(0xffffffffu, smem_u32(sm), 0), 16, 1024);
    bool ok = __all_sync(0xffffffffu, mbar_wait_ns(&q_full, 0, kPattnWaitNs));
    int last = -1;
    for (int it = 0; ok && it < total; ++it) {
      const int st = it % kStages, sb = it & 1;
      bool w = mbar_wait_ns(&k_full[st], (it / kStages) & 1, kPattnWaitNs);
      // the buffer's P of two tiles ago has been read
      if (it >= 2) w = w && mbar_wait_ns(&pv_done[sb], ((it >> 1) - 1) & 1, kPattnWaitNs);
      ok = __all_sync(0xffffffffu, w);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t dk = dk0 + (uint64_t)((st * kStageBytes) >> 4);
        const uint32_t d = tm + kTmS0 + 128u * sb;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
#pragma unroll
          for (int pt = 0; pt < 2; ++pt)
            mma_f16_ts(d, tm + kTmQ0 + 64u * pt + 8u * ks, dk + (uint64_t)(((ks >> 2) * kHalf + (ks & 3) * 32) >> 4), kId,
                       (ks | pt) != 0);
        mma_commit(&s_full[sb]);
        mma_commit(&k_free[st]);
      }
      __syncwarp();
      last = it;
    }
    if (!ok && lane == 0) atomicOr(status, SPEC_ST_DEVICE_WAIT);
    if (last >= 0) mbar_wait_ns(&s_full[last & 1], (last >> 1) & 1, kPattnWaitNs);   // before TMEM is released
  } else if (warp == kWPv) {
    // ------------------------------------------------------------ O += P . V
    // key steps of 16; V MN-major (bit 16): lbo = the d-half stride, sbo = 1 KB
    // between 8-key groups; P parts interleaved, 16 columns of hi and of lo per
    // 32 keys
    constexpr uint32_t kId = (1u << 4) | (k4 ? 0u : (1u << 7) | (1u << 10)) | (1u << 16) | ((128u >> 3) << 17) |
                             ((128u >> 4) << 24);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t dv0 = desc_sw128(__shfl_sync(0xffffffffu, smem_u32(sm), 0) + 2 * kHalf, kHalf, 1024);
    bool ok = true;
    int last = -1;
    for (int it = 0; ok && it < total; ++it) {
      const int st = it % kStages, sb = it & 1;
      ok = __all_sync(0xffffffffu, mbar_wait_ns(&p_full[sb], (it >> 1) & 1, kPattnWaitNs) &&
                                       mbar_wait_ns(&v_full[st], (it / kStages) & 1, kPattnWaitNs));
      if (!ok) break;
      tc_fence_after();
      const bool fresh = it == 0 || it == tl[0].n;
      if (elect_one()) {
        const uint64_t dv = dv0 + (uint64_t)((st * kStageBytes) >> 4);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
#pragma unroll
          for (int pt = 0; pt < 2; ++pt)
            mma_f16_ts(tm + kTmO0, tm + kTmS0 + 128u * sb + 32u * (kk >> 1) + 16u * pt + 8u * (kk & 1),
                       dv + (uint64_t)((kk * 2048) >> 4), kId, !(fresh && (kk | pt) == 0));
        mma_commit(&pv_done[sb]);
        mma_commit(&v_free[st]);
      }
      __syncwarp();
      last = it;
    }
    if (!ok && lane == 0) atomicOr(status, SPEC_ST_DEVICE_WAIT);
    if (last >= 0) mbar_wait_ns(&pv_done[last & 1], (last >> 1) & 1, kPattnWaitNs);
  } else {
    // ------------------------------------------------------------ tile rows
    const bool rows = warp < row_warps;                 // warps without rows only help to clean V
    const int r = 32 * warp + lane, fr = r0 + r;
    const bool live = r < nr;
    const int i = live ? fr / pl.group : 0, h = live ? fr - i * pl.group : 0;
    const uint32_t lane_base = (uint32_t)(32 * warp) << 16;
    float rowc = 1.4426950408889634f / sqrtf(128.0f);   // log2(e) / sqrt(d): scores in base-2 units
    if (rows) {
      const float* src = q + ((size_t)i * pl.nq + kvh * pl.group + h) * 128;
      float qmul = 1.f;
      if (k4 && live) {
        // binary16 parts: the row is scaled by a power of two to at most 2 in
        // magnitude and the scores are scaled back
        float mx = 0.f;
#pragma unroll 8
        for (int d = 0; d < 32; ++d) {
          const float4 x = reinterpret_cast<const float4*>(src)[d];
          mx = fmaxf(mx, fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w))));
        }
        const int e = min(max((int)((__float_as_uint(mx) >> 23) & 255u) - 127, -100), 100);
        qmul = __uint_as_float((uint32_t)(127 - e) << 23);
        rowc *= __uint_as_float((uint32_t)(127 + e) << 23);
      }
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        float x[32];
#pragma unroll
        for (int d = 0; d < 8; ++d) {
          const float4 y = live ? reinterpret_cast<const float4*>(src)[8 * c + d] : make_float4(0.f, 0.f, 0.f, 0.f);
          x[4 * d] = y.x * qmul;
          x[4 * d + 1] = y.y * qmul;
          x[4 * d + 2] = y.z * qmul;
          x[4 * d + 3] = y.w * qmul;
        }
        uint32_t hi[16], lo[16];
        split32<k4>(x, hi, lo);
        tmem_st16(tmem + lane_base + kTmQ0 + 16u * c, hi);
        tmem_st16(tmem + lane_base + kTmQ0 + 64u + 16u * c, lo);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&q_full);
    }
    const int p = n_past + i, plow = window_low(pl, p), sinks = pl.window > 0 ? pl.sinks : 0;
    const int b_last = n_past + pl.M - 1;                             // the block's last position
    const int low0 = window_low(pl, n_past), low1 = window_low(pl, b_last);
    auto page_lane = [&](int it) { return it < total && lane < kPagesPerTile ? page_at(kv, tile_at(it) * kPagesPerTile + lane) : -1; };
    int pg = page_lane(0);
    bool ok = true;
    int it = 0;
#pragma unroll 1
    for (int pass = 0; ok && pass < passes; ++pass) {
      const Span sp = span_of(pl, n_past, pass);
      const bool mine = live && i >= sp.i0 && i < sp.i1;
      float mref = -INFINITY, lsum = 0.f;
      const int n = tl[pass].n;
#pragma unroll 1
      for (int sc = 0; sc < n; ++sc, ++it) {
        const int sb = it & 1, t0 = tl[pass].at(sc) * kKeys;
        const uint32_t pages = __ballot_sync(0xffffffffu, pg >= 0) & 0xffu;
        pg = page_lane(it + 1);
        // every key of the tile is seen by every row of the block
        const bool full = pages == 0xffu && t0 + kKeys - 1 <= n_past && (t0 >= low1 || t0 + kKeys <= sinks);
        ok = __all_sync(0xffffffffu, mbar_wait_ns(&s_full[sb], (it >> 1) & 1, kPattnWaitNs));
        if (!ok) break;
        if (rows) {
          tc_fence_after();
          const uint32_t sa = tmem + lane_base + kTmS0 + 128u * sb;
          uint32_t vis[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int k0 = t0 + 32 * c;
            const uint32_t pm = ((pages >> (2 * c)) & 1u ? 0xffffu : 0u) | ((pages >> (2 * c)) & 2u ? 0xffff0000u : 0u);
            vis[c] = mine ? low_bits(p + 1 - k0) & (~low_bits(plow - k0) | low_bits(sinks - k0)) & pm : 0u;
          }
          float mx = -INFINITY;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t s[32];
            tmem_ld32(sa + 32u * c, s);
            tmem_wait_ld();
            if (full) {
#pragma unroll
              for (int j = 0; j < 32; ++j) mx = fmaxf(mx, __uint_as_float(s[j]));
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j) mx = fmaxf(mx, (vis[c] >> j) & 1u ? __uint_as_float(s[j]) : -INFINITY);
            }
          }
          mx *= rowc;
          // the reference max moves only when a score exceeds it by more than 8
          // (p <= 2^8 of it): O is rescaled rarely
          float alpha = 1.f;
          if (mx > mref + 8.f) {
            if (mref != -INFINITY) alpha = exp2_approx(mref - mx);
            mref = mx;
            lsum *= alpha;
          }
          if (__any_sync(0xffffffffu, alpha != 1.f)) {
            ok = __all_sync(0xffffffffu, mbar_wait_ns(&pv_done[sb ^ 1], ((it - 1) >> 1) & 1, kPattnWaitNs));
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t o[32];
              const uint32_t oa = tmem + lane_base + kTmO0 + 32u * c;
              tmem_ld32(oa, o);
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
              tmem_st32(oa, o);
            }
          }
          // p = 2^(s - base); binary16 keeps p below its range's bottom by
          // working 7 binary places up (p <= 2^15)
          const float base = mref == -INFINITY ? 0.f : (k4 ? mref - 7.f : mref);
          float ps[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t s[32];
            float x[32];
            tmem_ld32(sa + 32u * c, s);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const float e = exp2_approx(fmaf(__uint_as_float(s[j]), rowc, -base));
              x[j] = full || ((vis[c] >> j) & 1u) ? e : 0.f;
              ps[j & 3] += x[j];
            }
            uint32_t hi[16], lo[16];
            split32<k4>(x, hi, lo);
            tmem_st16(sa + 32u * c, hi);
            tmem_st16(sa + 32u * c + 16u, lo);
          }
          lsum += (ps[0] + ps[1]) + (ps[2] + ps[3]);
        }
        if (!k4 && !full) {
          // V rows that no row sees read as zero (stale bytes may be anything,
          // and 0 * NaN is NaN); a non-finite element that only some rows see
          // is taken out of the product and added to those rows at the end
          const int st = it % kStages;
          ok = __all_sync(0xffffffffu, mbar_wait_ns(&v_full[st], (it / kStages) & 1, kPattnWaitNs));
          if (!ok) break;
          uint8_t* vb = sm + (size_t)st * kStageBytes + 2 * kHalf;
#pragma unroll 1
          for (int x = tid; x < kKeys * 16; x += 128) {               // (key, d half, 16-byte chunk)
            const int key = x >> 4, t = t0 + key;
            const bool there = (pages >> (key >> 4)) & 1u;
            if (there && t <= n_past && (t >= low1 || t < sinks)) continue;      // all rows see it
            uint4* at = reinterpret_cast<uint4*>(vb + ((x >> 3) & 1) * kHalf + key * 128 + (x & 7) * 16);
            if (!there || t > b_last || (t < low0 && t >= sinks)) {
              *at = make_uint4(0, 0, 0, 0);                                      // no row does
              continue;
            }
            uint4 y = *at;
            uint32_t* w = reinterpret_cast<uint32_t*>(&y);
            bool found = false;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const bool b0 = (w[j] & 0x7F80u) == 0x7F80u, b1 = (w[j] & 0x7F800000u) == 0x7F800000u;
              found = found || b0 || b1;
              w[j] &= (b0 ? 0xFFFF0000u : 0xFFFFFFFFu) & (b1 ? 0x0000FFFFu : 0xFFFFFFFFu);
            }
            if (found) {
              *at = y;
              // bit e: key n_past + 1 + e (e < 16) or low0 + e - 16
              atomicOr(&poison, 1u << (t > n_past ? t - n_past - 1 : 16 + t - low0));
            }
          }
          fence_proxy_async();
        }
        if (rows) {
          tmem_wait_st();
          tc_fence_before();
        }
        mbar_arrive(&p_full[sb]);
      }
      if (!ok || n == 0 || !rows) continue;
      ok = __all_sync(0xffffffffu, mbar_wait_ns(&pv_done[(it - 1) & 1], ((it - 1) >> 1) & 1, kPattnWaitNs));
      if (!ok) break;
      tc_fence_after();
      const size_t at = ((size_t)slot * pl.nkv + kvh) * R + fr;
      const uint32_t bad = k4 ? 0u : *reinterpret_cast<volatile uint32_t*>(&poison);
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t o[32];
        tmem_ld32(tmem + lane_base + kTmO0 + 32u * c, o);
        tmem_wait_ld();
        if (!mine) continue;
        for (uint32_t left = bad; left; left &= left - 1) {
          const int e = __ffs(left) - 1, t = e < 16 ? n_past + 1 + e : low0 + e - 16;
          if (t > p || (t < plow && t >= sinks)) continue;
          const uint16_t* v = kv.pool + ((((size_t)page_at(kv, t >> 4) * kv.n_layers + layer) * 2 + 1) * kv.n_kv + kvh) * 2048 +
                              (t & 15) * 128 + 32 * c;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const uint32_t w = (uint32_t)v[j] << 16;
            if ((w & 0x7F800000u) == 0x7F800000u) o[j] = __float_as_uint(__uint_as_float(o[j]) + __uint_as_float(w));
          }
        }
        float4* dst = reinterpret_cast<float4*>(part_o + at * 128 + 32 * c);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          dst[j] = make_float4(__uint_as_float(o[4 * j]), __uint_as_float(o[4 * j + 1]), __uint_as_float(o[4 * j + 2]),
                               __uint_as_float(o[4 * j + 3]));
      }
      if (mine) part_ml[at] = make_float2(k4 ? mref - 7.f : mref, lsum);
      tc_fence_before();
    }
    if (!ok && lane == 0) atomicOr(status, SPEC_ST_DEVICE_WAIT);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
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

template <bool k4>
static cudaError_t launch_pattn(const PattnPlan& pl, const KvView& kv, const CUtensorMap& map, int layer, const float* q,
                                int row_tiles, float* part_o, float2* part_ml, int32_t* status, cudaStream_t st) {
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
  pattn_kernel<k4><<<dim3(pl.slots, pl.nkv, row_tiles), 32 * pattn_warps<k4>(), kPattnSmem, st>>>(
      q, pl, kv, map, layer, part_o, part_ml, status);
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
  alignas(64) CUtensorMap map = {};
  if (!k4) {
    const cudaError_t e = make_kv_tmap(kv, &map);
    if (e != cudaSuccess) return e;
  }
  cudaError_t e = k4 ? launch_pattn<true>(pl, kv, map, layer, q, row_tiles, po, ml, status, st)
                     : launch_pattn<false>(pl, kv, map, layer, q, row_tiles, po, ml, status, st);
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
