// pattn.cu — attention of up to 16 rows over a paged cache, bf16 or 4-bit, with
// an optional window and sinks.
//
// Row i sits at position p = seq_len - M + i and sees the keys t <= p with
// t > p - window or t < sinks (window 0: every t <= p).
// s_t = q.k_t / sqrt(128), o = sum_t exp(s_t - m) v_t / sum_t exp(s_t - m).
//
// Decomposition (flash-decoding).  The M * group query rows of a KV head (group
// query heads read it) are packed into tiles of up to 128 rows.  Keys are taken in
// tiles of 128 at absolute positions, and chunks of L tiles are worked on by one
// CTA each (slot, KV head, row tile) with a running (max, sum) per row; a merge
// kernel joins the chunks.
// Three kernels write the chunks' (O, max, sum): pattn_few.cu for at most 16 query
// rows per KV head, and for more the one here (4-bit) or pattn_bf16.cu.
//
// The split of the keys is a function of the row's own position and the number of
// row tiles (chunk_len, pattn_plan.cuh): chunks are whole multiples of L tiles
// from position 0, so a row has the same bits in every block of as many row tiles
// (batch-height invariance).  L grows with the position such that there are never
// more chunks than SMs per KV head and row tile; a block that crosses such a step
// runs its two groups of rows one after the other.  Tiles that no row sees are
// skipped: they would add exact zeros.
//
// The 4-bit kernel for many rows, on tcgen05:
//   S[128 x 128 keys] = Q[128 x 128 d] . K^T      (A = Q in TMEM, B = K)
//   O[128 x 128 d]    = P[128 x 128 keys] . V     (A = P in TMEM, B = V)
// Pages are unpacked into binary16 tiles in shared memory.  Q and P live in TMEM:
// with the keys on the MMA's rows and Q and P in shared memory, which then carries
// 192 KB and more per tile, 208 rows over 32k keys took 100 us when this layout
// took 57.
//
// What bounds it: 32 MMAs of 128 x 128 x 16 take 2,600 cycles a tile, 8,750 warp
// instructions, most of them softmax and unpacking, 2,190 cycles of four schedulers
// at best (half of the slots are used): 3,200 cycles a tile.  A call of one tile per
// CTA is latency: 3,000 cycles to the sequence length and the plan, 4,700 to page
// ids, pages and the unpacked K, 3,900 for the tile, 2,500 to store.  16 rows of 52
// heads on 4: 11.5 us behind 2k keys, 34.1 behind 32k (410 TFLOP/s, counting each
// product once; two parts make it two).  Both row tiles of a KV head unpack every
// page, each in its own CTA.  128 bytes a thread are spilled.
//
// Precision: all operands are binary16.  A 4-bit value is exact in it; q and p are
// split into two parts, 22 significant bits.  q is first multiplied by log2(e) /
// sqrt(d), rounded once, so that the scores come in base-2 units times a power of two
// and the largest less itself is exactly 0.  The tensor core truncates its
// additions, so the small parts go first, and each tile's O starts afresh and is
// added up in fp32 registers: left in TMEM over 27 tiles it was off by 8e-6.
#include "attn_mma.cuh"
#include "common.cuh"
#include "internal.h"
#include "pattn_plan.cuh"
#include "pattn_unpack.cuh"

namespace spec {

constexpr int kUnpackWarps = 6;
constexpr size_t kPattnSmem = 1024 + (size_t)kStages * kStageBytes;
// TMEM columns: two score buffers, each overwritten in place by its P parts
// (16 columns of high and 16 of low parts per 32 keys); O; Q (64 columns of high
// parts, then 64 of low ones)
constexpr uint32_t kTmS = 0, kTmO = 256, kTmQ = 384;
constexpr int kTmAll = 512;

// warps: 0-7 softmax, two threads per row (warp w: rows 32 (w % 4).., keys and
// d's 64 (w / 4)..), 8 issues the QK MMAs, 9 the PV MMAs, 10-15 unpack pages of K
// and V in turn.  The launch gives every thread 128 registers, 65,536 in all; the
// softmax threads take 184 of them and the others 72.
constexpr int kSoftWarps = 8, kWQk = 8, kWPv = 9, kWLoad = 10;
constexpr int kPattnThreads = 512;

using f2 = unsigned long long;                      // two floats for the packed fp32 instructions
// binary16 parts of a pair: hi nearest, lo what is left (the first in the low half)
SPEC_DEV void split_pair(f2 x, uint32_t& hi, uint32_t& lo) {
  float x0, x1;
  f2unpack(x, x0, x1);
  const __half2 h = __floats2half2_rn(x0, x1);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  minus_f16x2(x0, x1, hi);
  const __half2 l = __floats2half2_rn(x0, x1);
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

// ---------------------------------------------------------------------------
// partials: grid (slot, KV head, row tile)
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kPattnThreads, 1)
pattn_kernel(const float* __restrict__ q, PattnPlan pl, KvView kv, int layer, float* __restrict__ part_o,
             float2* __restrict__ part_ml, int32_t* status) {
  extern __shared__ __align__(128) uint8_t dsm[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dsm) + 1023) & ~(uintptr_t)1023);
  __shared__ uint32_t tmem_slot;
  __shared__ __align__(8) uint64_t q_full, s_full[2], p_full[2], pv_done[2];
  __shared__ __align__(8) StageBars bar;
  __shared__ float pair[2][128];                        // what the two threads of a row exchange
  // mapped pages per tile (a ring of 8: a tile's entries are rewritten eight tiles
  // later, when its softmax has long been passed)
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
      mbar_init(&bar.k_full[b], kItemsPerTile);
      mbar_init(&bar.v_full[b], kItemsPerTile);
      mbar_init(&bar.k_free[b], 1);
      mbar_init(&bar.v_free[b], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&s_full[b], 1);
      mbar_init(&p_full[b], 2 * row_warps);
      mbar_init(&pv_done[b], 1);
    }
    for (int g = 0; g < 4; ++g) gave_up[g] = 0;
    fence_mbarrier_init();
  }
  pdl_wait();
  pdl_trigger();                                        // not before: see the merge
  const int n_past = ldg_now(kv.seq_len) - pl.M;
  // the rows of Q, whole rows by a warp, into the last stage (which tile 2 is the
  // first to use), 16-byte chunk j at j ^ (row % 8)
  uint8_t* q_rows = sm + (kStages - 1) * kStageBytes;
  {
    constexpr int kRows = 128 / (kPattnThreads / 32);
    const int fr = r0 + kRows * warp;
    int i = div24(fr, pl.group), hd = fr - i * pl.group;
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const int r = kRows * warp + j;
      if (r < nr)
        copy16(q_rows + 512 * r + ((lane ^ (r & 7)) << 4),
               reinterpret_cast<const uint8_t*>(q + ((size_t)i * pl.nq + kvh * pl.group + hd) * 128) + 16 * lane);
      if (++hd == pl.group) {
        hd = 0;
        ++i;
      }
    }
  }
  copy_commit();
  const int passes = span_count(pl, n_past);
  TileList tl0 = tiles_of(span_of(pl, n_past, 0), slot), tl1;
  if (passes == 2) tl1 = tiles_of(span_of(pl, n_past, 1), slot);
  const int total = tl0.n + tl1.n;
  auto tile_at = [&](int it) { return it < tl0.n ? tl0.at(it) : tl1.at(it - tl0.n); };
  const int b_last = n_past + pl.M - 1;                 // the block's last position
  const int low0 = window_low(pl, n_past), low1 = window_low(pl, b_last), sinks = pl.window > 0 ? pl.sinks : 0;
  copy_wait<0>();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  // (total == 0: nothing of this chunk is seen)
  if (warp >= kSoftWarps) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 72;\n");
  if (total == 0) {
  } else if (warp >= kWLoad) {
    // Q's rows lie in the last stage until they have been read
    if (!unpack_tiles<kUnpackWarps>(warp - kWLoad, total, tile_at, kv, layer, kvh, sm, bar, mapped, &q_full) && lane == 0)
      atomicOr(status, SPEC_ST_DEVICE_WAIT);
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
      bool w = mbar_wait(&bar.k_full[st], (it / kStages) & 1);
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
        mma_commit(&bar.k_free[st]);
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
      ok = __all_sync(0xffffffffu, mbar_wait(&bar.v_full[st], (it / kStages) & 1) && mbar_wait(&p_full[sb], (it >> 1) & 1));
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
        mma_commit(&bar.v_free[st]);
      }
      __syncwarp();
      last = it;
    }
    if (!ok && lane == 0) atomicOr(status, SPEC_ST_DEVICE_WAIT);
    if (last >= 0) mbar_wait(&pv_done[last & 1], (last >> 1) & 1);
  }
  } else {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 184;\n");
  if (total > 0 && (warp & 3) < row_warps) {
    // ------------------------------------------------------------ softmax
    const int h = warp >> 2, ww = warp & 3;
    const int r = 32 * ww + lane, fr = r0 + r;          // tile row, row of the KV head
    const bool live = r < nr;
    const int i = live ? div24(fr, pl.group) : 0;
    const uint32_t tl = tmem + ((uint32_t)(32 * ww) << 16);
    constexpr float kBias = 7.f;                        // p = 2^(7 + s - max): binary16 keeps 2^-24 of 2^7
    // one lane arrives for the warp: the warp barrier orders the others' writes
    auto arrive = [&](uint64_t* bar) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    // what turns scores into base-2 units: a power of two, so that its products are
    // exact and the largest score less itself is 0 however large it is
    float unit;
    {
      // the row times log2(e) / sqrt(d), by a power of two to about 2 in magnitude at
      // most, and the scores are scaled back
      float4 y[16];
      float mx = 0.f;
#pragma unroll
      for (int d = 0; d < 16; ++d) {
        y[d] = live ? *reinterpret_cast<const float4*>(q_rows + 512 * r + (((16 * h + d) ^ (r & 7)) << 4))
                    : make_float4(0.f, 0.f, 0.f, 0.f);
        mx = fmaxf(mx, fmaxf(fmaxf(fabsf(y[d].x), fabsf(y[d].y)), fmaxf(fabsf(y[d].z), fabsf(y[d].w))));
      }
      pair[h][r] = mx;
      named_bar(1 + ww, 64);
      mx = fmaxf(mx, pair[1 - h][r]);
      const int e = min(max((int)((__float_as_uint(mx) >> 23) & 255u) - 127, -100), 126);
      const float mul = 8.f * kScoreScale * __uint_as_float((uint32_t)(127 - e) << 23);
      unit = __uint_as_float((uint32_t)(124 + e) << 23);
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
        const int sb = it & 1, t0 = tile_at(it) * kKeys;
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
        // The reference moves only when a score exceeds it by more than 7: p stays
        // within 2^15 with the bias, which rounds to at most 8 beside large scores.
        // A wait that ran out is carried to this barrier, where the pair of warps
        // leaves together.
        if (!got || !ok) *reinterpret_cast<volatile int*>(&gave_up[ww]) = 1;
        if (named_bar_or(1 + ww, 64, mx - ref > 7.f || !got || !ok)) {
          left = *reinterpret_cast<volatile int*>(&gave_up[ww]) != 0;
          if (left) break;
          pair[h][r] = mx;
          named_bar(1 + ww, 64);
          mx = fmaxf(mx, pair[1 - h][r]);
          if (pending) ok = drain();                    // O so far is in the old units
          if (mx - ref > 7.f) {
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
        // [slot][KV head][d / 4][row]: a warp's rows side by side
        float4* dst = reinterpret_cast<float4*>(part_o) + (((size_t)slot * pl.nkv + kvh) * 32 + 16 * h) * R + fr;
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          float4 y;
          f2unpack(acc[2 * c], y.x, y.y);
          f2unpack(acc[2 * c + 1], y.z, y.w);
          dst[(size_t)c * R] = y;
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
// merge: four threads per 4 output elements, one per residue of the chunk number
// mod 4; a warp takes 32 neighbouring rows, which lie side by side in the
// partials.  With m the largest chunk maximum (base 2) and w_c = 2^(m_c - m):
//   out = sum_c w_c o_c / sum_c w_c l_c, over the chunks in which the row sees a
// key: within each residue its largest maximum, then the sums in chunk order, then
// the same over the residues.  Every step is one of the row's own chunks, so a row's
// bits do not depend on the block.
// ---------------------------------------------------------------------------
constexpr int kMergeParts = 4;

__global__ void __launch_bounds__(32 * kMergeParts)
pattn_merge_kernel(const float4* __restrict__ part_o, const float2* __restrict__ part_ml, PattnPlan pl,
                   const int32_t* __restrict__ seq_len, float4* __restrict__ out) {
  __shared__ float4 o_sm[kMergeParts][32];
  __shared__ float2 ml_sm[kMergeParts][32];
  pdl_trigger();
  const int lane = threadIdx.x & 31, res = threadIdx.x >> 5;
  const int R = pl.M * pl.group, item = blockIdx.x * 32 + lane;       // ((KV head, d / 4), row); a grid of whole warps
  const int hd = div24(item, R), r = item - hd * R, kvh = hd >> 5, d4 = hd & 31;
  const int i = div24(r, pl.group), head = kvh * pl.group + r - i * pl.group;
  // The length may be read before the wait: the kernel before this one lets it start
  // only once its own wait is over, so whatever wrote the length has finished.
  const int n_past = ldg_now(seq_len) - pl.M;
  Span s = span_of(pl, n_past, 0);
  if (i >= s.i1) s = span_of(pl, n_past, 1);
  const int slots = n_past + i < 0 ? 0 : min(s.nslots, pl.slots);
  // this residue's slots: n0 of the sinks' from slot res on, then those from c1 on
  const int ns = min(s.ns, slots), n0 = (ns + kMergeParts - 1 - res) / kMergeParts;
  const int c1 = ns + ((res - s.cbase) & (kMergeParts - 1));
  const int n = n0 + max(0, slots - c1 + kMergeParts - 1) / kMergeParts;
  auto slot = [&](int j) { return j < n0 ? res + kMergeParts * j : c1 + kMergeParts * (j - n0); };
  const size_t step = (size_t)pl.nkv * R, at = (size_t)kvh * R + r;
  const float4* po = part_o + (size_t)hd * R + r;
  pdl_wait();
  constexpr int kBatch = 8;                             // loads in flight
  float4 y[kBatch];
  float2 x[kBatch];
  auto load = [&](int j0) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      x[k] = make_float2(0.f, 0.f);
      if (j0 + k < n) {
        const size_t c = slot(j0 + k);
        x[k] = ldg_now(part_ml + at + c * step);
        y[k] = ldg_now(po + 32 * c * step);
      }
    }
  };
  load(0);
  float m = -INFINITY, L = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  // the largest maximum of all batches first: sums that were rescaled from batch to
  // batch would depend on where the block's list starts
#pragma unroll 4
  for (int j = kBatch; j < n; ++j) {
    const float2 z = ldg_now(part_ml + at + (size_t)slot(j) * step);
    if (z.y != 0.f) m = fmaxf(m, z.x);
  }
#pragma unroll
  for (int k = 0; k < kBatch; ++k)
    if (x[k].y != 0.f) m = fmaxf(m, x[k].x);
  for (int j0 = 0;;) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (x[k].y != 0.f) {
        const float w = exp2_approx(x[k].x - m);
        L = fmaf(w, x[k].y, L);
        o.x = fmaf(w, y[k].x, o.x);
        o.y = fmaf(w, y[k].y, o.y);
        o.z = fmaf(w, y[k].z, o.z);
        o.w = fmaf(w, y[k].w, o.w);
      }
    j0 += kBatch;
    if (j0 >= n) break;
    load(j0);
  }
  o_sm[res][lane] = o;
  ml_sm[res][lane] = make_float2(m, L);
  __syncthreads();
  if (res != 0) return;
  m = -INFINITY;
#pragma unroll
  for (int k = 0; k < kMergeParts; ++k) m = fmaxf(m, ml_sm[k][lane].x);
  o = make_float4(0.f, 0.f, 0.f, 0.f);
  L = 0.f;
#pragma unroll
  for (int k = 0; k < kMergeParts; ++k) {
    const float2 x = ml_sm[k][lane];
    if (x.y == 0.f) continue;
    const float w = exp2_approx(x.x - m);
    const float4 y = o_sm[k][lane];
    L += w * x.y;
    o.x += w * y.x;
    o.y += w * y.y;
    o.z += w * y.z;
    o.w += w * y.w;
  }
  out[((size_t)i * pl.nq + head) * 32 + d4] =           // nothing visible: zero
      L == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o.x / L, o.y / L, o.z / L, o.w / L);
}

// chunks of a KV head at most: one per SM, KV head and row tile, so that the
// grid is one wave.  (With as many for two row tiles, two waves, 16 rows of 13
// heads took 57 instead of 45 us behind 32k keys.)  At least 4, so that
// a window's chunks (one of sinks, and one more than the window's own) fit.
static int pattn_chunks(int nkv, int row_tiles, int num_sms) {
  const int c = num_sms / (nkv * row_tiles);
  return c > 4 ? c : 4;
}

size_t paged_attention_floats(int nq, int nkv, int max_rows, int num_sms) {
  // rows * chunks is largest for one row tile or, below 4 chunks, for all rows
  return (size_t)pattn_chunks(nkv, 1, num_sms) * nq * max_rows * 130;
}

static cudaError_t launch_pattn_kv4(const PattnPlan& pl, const KvView& kv, int layer, const float* q, int row_tiles,
                                float* part_o, float2* part_ml, int32_t* status, cudaStream_t st) {
  // the shared-memory limit is a per-device attribute
  constexpr int kMaxDevices = 64;
  static bool have[kMaxDevices] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool known = dev >= 0 && dev < kMaxDevices;
  if (!known || !have[dev]) {
    e = cudaFuncSetAttribute(pattn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPattnSmem);
    if (e != cudaSuccess) return e;
    if (known) have[dev] = true;
  }
  return launch_early(pattn_kernel, dim3(pl.slots, pl.nkv, row_tiles), dim3(kPattnThreads), kPattnSmem, st, q, pl, kv, layer,
                      part_o, part_ml, status);
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
  const int R = M * pl.group, row_tiles = (R + 127) / 128;
  pl.C = pattn_chunks(kv.n_kv, row_tiles, num_sms);
  pl.c_inv = ((1ull << 40) + pl.C - 1) / pl.C;
  // chunk slots: never more than the cache has tiles; the window's longest
  // chunk is the shortest with which sinks and window fit into C chunks
  const long long tiles = ((long long)kv.max_seq_pages * 16 + kKeys - 1) / kKeys;
  pl.Lw = INT32_MAX;
  pl.slots = (int)(tiles < pl.C ? tiles : pl.C);
  if (window > 0) {
    const long long ws = ((long long)window + 14 + kKeys - 1) / kKeys + 1;       // tiles of window + 15 keys
    const long long ss = ((long long)sinks + kKeys - 1) / kKeys;
    long long L = (ws + ss) / pl.C > 1 ? (ws + ss) / pl.C : 1;
    // bisected: a window without an end (2^31 - 1) would take millions of steps
    for (long long most = ws + ss; L < most;) {
      const long long mid = (L + most) / 2;
      if ((ss + mid - 1) / mid + (ws + mid - 2) / mid + 1 > pl.C)
        L = mid + 1;
      else
        most = mid;
    }
    pl.Lw = (int)(L < INT32_MAX ? L : INT32_MAX);
    if (pl.Lw == 1 && ss + ws < pl.slots) pl.slots = (int)(ss + ws);
  }
  pl.tile_rows = (R + row_tiles - 1) / row_tiles;
  float2* ml = reinterpret_cast<float2*>(part);        // [slots][nkv][R], then the outputs
  float* po = part + 2 * (size_t)pl.C * nq * 16;
  cudaError_t e = R <= kFewRows ? launch_pattn_few(k4, pl, kv, layer, q, po, ml, st)
                  : k4          ? launch_pattn_kv4(pl, kv, layer, q, row_tiles, po, ml, status, st)
                                : launch_pattn_bf16(pl, kv, layer, q, row_tiles, po, ml, status, st);
  if (e != cudaSuccess) return e;
  return launch_early(pattn_merge_kernel, dim3(M * nq), dim3(32 * kMergeParts), 0, st, reinterpret_cast<const float4*>(po), ml,
                      pl, kv.seq_len, reinterpret_cast<float4*>(out));
}

}  // namespace spec
