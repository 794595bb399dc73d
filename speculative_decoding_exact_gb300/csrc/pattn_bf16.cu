// pattn_bf16.cu — the partials of attention over the bf16 paged cache (pattn.cu) for
// calls of more than 16 query rows per KV head.
//
// The decomposition is that of pattn.cu: tiles of up to 128 packed query rows and
// 128 keys, S = Q . K^T and O = P . V on tcgen05 with a running (max, sum) per
// row, each tile's O added in registers, a chunk of L tiles per CTA.
//
// K and V pages are operands as they are: TMA lays them down swizzled, and no
// thread touches K.  Q and P go in three bf16 parts by truncation, 24 bits, so no
// value is out of range and nothing is rounded but q's product with log2(e) /
// sqrt(d), once.  Binary16 operands (two parts)
// took conversions of every page and a second path for elements past binary16;
// 104 rows over 32k keys took 48 us with them when this took 39 (now 35).
//
// What bounds it: the MMAs.  A 128 x 128 x 16 product takes 121 cycles with both
// operands in shared memory (Q . K^T) and 81 with one in TMEM (P . V), 48 of them
// 4,850 cycles a tile; the tile's 64 KB come in 2,850 at the SM's share of HBM.  O, S
// and P take 448 of the 512 columns of the TMEM: one of Q's three parts would fit in
// the rest and save 8 x 40 cycles a tile (not tried).  140 bytes a thread are
// spilled.  16 rows of 52 heads on 4 with a window of 4096: 16.4 us, of which the
// MMAs of a CTA's two tiles are 4.7; 8 rows and a window of 32768: 35.2.
//
// 0 * NaN is NaN, so an element of V that is not finite would reach rows that do
// not see its key.  Four warps look through each V tile before its MMAs; such
// elements are zeroed there and their p v added in fp32 to the rows that see them.
//
// Q lies in shared memory (96 KB) next to two stages of K and V; P (192 columns),
// S and O fill the tensor memory.
#include "attn_mma.cuh"
#include "common.cuh"
#include "internal.h"
#include "pattn_plan.cuh"

namespace spec {

constexpr int kHalf = kKeys * 128;                  // one d half of a tile of 128 rows: [row][64 values]
constexpr int kParts = 3;
constexpr int kQBytes = kParts * 2 * kHalf;
constexpr int kStages = 2, kStageBytes = 4 * kHalf; // K then V, 64 KB
constexpr size_t kBf16Smem = 1024 + kQBytes + (size_t)kStages * kStageBytes;
constexpr uint32_t kTmO = 0, kTmS = 128, kTmP = 256;   // TMEM columns; P: 64 per part
constexpr int kTmAll = 512;

// warps: 0-7 softmax, two threads per row (warp w: rows 32 (w % 4).., keys and
// d's 64 (w / 4)..), 8 issues the QK MMAs, 9 the PV MMAs, 10 and 11 copy K and V,
// 12-15 look through V.  The launch gives every thread 128 registers, 65,536 in
// all; the softmax threads take 200 of them and the others 56.
constexpr int kSoftWarps = 8, kWQk = 8, kWPv = 9, kWLoadK = 10, kWLoadV = 11, kWScan = 12;
constexpr int kThreads = 512;
constexpr int kQWarps = 14;                         // all but the copying ones lay down Q
constexpr int kQRows = (128 + kQWarps - 1) / kQWarps;

// one TMEM column (to be waited for)
SPEC_DEV uint32_t tmem_ld1(uint32_t taddr) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n" : "=r"(r) : "r"(taddr));
  return r;
}
// an element of a bf16 pair is infinite or NaN
SPEC_DEV bool nonfinite(uint32_t w) { return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u; }

__global__ void __launch_bounds__(kThreads, 1)
pattn_bf16_kernel(const float* __restrict__ q, PattnPlan pl, KvView kv, const __grid_constant__ CUtensorMap map, int layer,
                  float4* __restrict__ part_o, float2* __restrict__ part_ml, int32_t* status) {
  extern __shared__ __align__(128) uint8_t dsm[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dsm) + 1023) & ~(uintptr_t)1023);
  uint8_t* stages = sm + kQBytes;
  __shared__ uint32_t tmem_slot;
  __shared__ __align__(8) uint64_t k_full[kStages], v_here[kStages], v_full[kStages], k_free[kStages], v_free[kStages],
      s_full, s_free, p_full, pv_done;
  __shared__ float pair[2][128];                        // what the two threads of a row exchange
  // per tile (a ring of 8: a tile's entries are rewritten eight tiles later,
  // when its softmax has long been passed): mapped pages, and the keys whose V
  // has an element that is not finite
  __shared__ __align__(16) uint16_t odd[8][kPagesPerTile];
  __shared__ __align__(8) uint8_t mapped[8][kPagesPerTile];
  __shared__ int gave_up[4];                            // a wait of this pair of softmax warps ran out

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slot = blockIdx.x, kvh = blockIdx.y, R = pl.M * pl.group;
  const int r0 = blockIdx.z * pl.tile_rows, nr = min(pl.tile_rows, R - r0);
  const int row_warps = (nr + 31) >> 5;                 // pairs of softmax warps with rows
  if (warp == kWQk) tmem_alloc(&tmem_slot, kTmAll);
  if (tid == 32 * kWPv) {
    for (int b = 0; b < kStages; ++b) {
      mbar_init(&k_full[b], 1);
      mbar_init(&v_here[b], 1);
      mbar_init(&v_full[b], 4);
      mbar_init(&k_free[b], 1);
      mbar_init(&v_free[b], 1);
    }
    mbar_init(&s_full, 1);
    mbar_init(&s_free, 2 * row_warps);
    mbar_init(&p_full, 2 * row_warps);
    mbar_init(&pv_done, 1);
    for (int g = 0; g < 4; ++g) gave_up[g] = 0;
    fence_mbarrier_init();
  }
  pdl_wait();
  pdl_trigger();                                        // not before: see the merge in pattn.cu
  const int n_past = ldg_now(kv.seq_len) - pl.M;
  // Q, whole rows by a warp, as swizzled K-major tiles: [part][d half][row][128 B]
  const int qw = warp < kWLoadK ? warp : warp - 2;
  float4 y[kQRows];
  if (warp != kWLoadK && warp != kWLoadV) {
    const int fr = r0 + kQRows * qw;
    int i = div24(fr, pl.group), hd = fr - i * pl.group;
#pragma unroll
    for (int j = 0; j < kQRows; ++j) {
      y[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (kQRows * qw + j < nr)
        y[j] = ldg_now(reinterpret_cast<const float4*>(q + ((size_t)i * pl.nq + kvh * pl.group + hd) * 128) + lane);
      if (++hd == pl.group) {
        hd = 0;
        ++i;
      }
    }
  }
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

  // one tile's K (V) pages; lane l < 16 copies d half l % 2 of page l / 2.  An
  // unmapped page is a box outside the tensor, which reads as zeros.
  auto page_of = [&](int it) { return it < total ? page_at(kv, tile_at(it) * kPagesPerTile + ((lane >> 1) & 7)) : -1; };
  auto issue = [&](int it, bool is_v, int page) {
    const int st = it % kStages;
    uint64_t* full = is_v ? &v_here[st] : &k_full[st];
    const int pp = (lane >> 1) & 7, half = lane & 1;
    const bool ok = page_ok(kv, page);
    if (!is_v && lane < 16 && half == 0) mapped[it & 7][pp] = ok;
    __syncwarp();
    if (lane == 0) mbar_arrive_expect_tx(full, 2 * kHalf);
    __syncwarp();
    if (lane < 16)
      tma_load_2d(stages + st * kStageBytes + (is_v ? 2 : 0) * kHalf + half * kHalf + pp * 2048, &map, 64 * half,
                  ok ? (((page * kv.n_layers + layer) * 2 + is_v) * kv.n_kv + kvh) * 16 : -16, full);
  };
  int next_page = -1;                                   // of a copying warp: the ids of its next tile
  if (warp == kWLoadK || warp == kWLoadV) {
    int ids[kStages];
#pragma unroll
    for (int it = 0; it < kStages; ++it) ids[it] = page_of(it);
    next_page = page_of(kStages);
#pragma unroll
    for (int it = 0; it < kStages; ++it)
      if (it < total) issue(it, warp == kWLoadV, ids[it]);
  } else if (total > 0) {
#pragma unroll
    for (int j = 0; j < kQRows; ++j) {
      const int r = kQRows * qw + j;
      if (r >= 32 * row_warps) break;
      uint8_t* dst = sm + (lane >> 4) * kHalf + r * 128 + ((((lane & 15) >> 1) ^ (r & 7)) << 4) + 8 * (lane & 1);
      // log2(e) / sqrt(d) goes into Q: the scores come in base-2 units, and the largest
      // less itself is 0 however large it is
      y[j] = make_float4(y[j].x * kScoreScale, y[j].y * kScoreScale, y[j].z * kScoreScale, y[j].w * kScoreScale);
#pragma unroll
      for (int pt = 0; pt < kParts; ++pt) {
        uint2 w;
        w.x = take_bf16(y[j].x, y[j].y);
        w.y = take_bf16(y[j].z, y[j].w);
        *reinterpret_cast<uint2*>(dst + pt * 2 * kHalf) = w;
      }
    }
    fence_proxy_async();
  }
  __syncthreads();

  // (total == 0: nothing of this chunk is seen)
  if (warp >= kSoftWarps) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 56;\n");
  bool ok = true;
  if (total == 0) {
  } else if (warp == kWQk) {
    // ------------------------------------------------------------ S = Q . K^T
    // D f32 (bit 4), A and B bf16 (7, 10), N >> 3 at 17, M >> 4 at 24; 8 d steps
    // of 16, the small parts of Q first (the tensor core truncates its additions)
    constexpr uint32_t kId = (1u << 4) | (1u << 7) | (1u << 10) | ((kKeys >> 3) << 17) | ((128u >> 4) << 24);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t dq0 = desc_sw128(__shfl_sync(0xffffffffu, smem_u32(sm), 0), 16, 1024);
    const uint64_t dk0 = dq0 + (uint64_t)(kQBytes >> 4);
    int last = -1;
    for (int it = 0; ok && it < total; ++it) {
      const int st = it % kStages;
      bool w = mbar_wait(&k_full[st], (it / kStages) & 1);
      if (it >= 1) w = w && mbar_wait(&s_free, (it - 1) & 1);
      ok = __all_sync(0xffffffffu, w);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t dk = dk0 + (uint64_t)((st * kStageBytes) >> 4);
#pragma unroll
        for (int pt = kParts - 1; pt >= 0; --pt)
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) {
            const uint64_t off = (uint64_t)(((ks >> 2) * kHalf + (ks & 3) * 32) >> 4);
            mma_f16_ss(tm + kTmS, dq0 + (uint64_t)((pt * 2 * kHalf) >> 4) + off, dk + off, kId,
                       pt != kParts - 1 || ks != 0);
          }
        mma_commit(&s_full);
        mma_commit(&k_free[st]);
      }
      __syncwarp();
      last = it;
    }
    if (last >= 0) mbar_wait(&s_full, last & 1);        // before TMEM is released
  } else if (warp == kWPv) {
    // ------------------------------------------------------------ O = P . V
    // key steps of 16; V MN-major (bit 16): lbo = the d-half stride, sbo = 1 KB
    // between 8-key groups; the small parts of P first
    constexpr uint32_t kId =
        (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t dv0 = desc_sw128(__shfl_sync(0xffffffffu, smem_u32(stages), 0) + 2 * kHalf, kHalf, 1024);
    int last = -1;
    for (int it = 0; ok && it < total; ++it) {
      const int st = it % kStages;
      ok = __all_sync(0xffffffffu, mbar_wait(&v_full[st], (it / kStages) & 1) && mbar_wait(&p_full, it & 1));
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t dv = dv0 + (uint64_t)((st * kStageBytes) >> 4);
#pragma unroll
        for (int pt = kParts - 1; pt >= 0; --pt)
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_f16_ts(tm + kTmO, tm + kTmP + 64u * pt + 8u * kk, dv + (uint64_t)((kk * 2048) >> 4), kId,
                       pt != kParts - 1 || kk != 0);
        mma_commit(&pv_done);
        mma_commit(&v_free[st]);
      }
      __syncwarp();
      last = it;
    }
    if (last >= 0) mbar_wait(&pv_done, last & 1);
  } else if (warp < kWScan) {
    // ------------------------------------------------------------ copies
    const bool is_v = warp == kWLoadV;
    int it = kStages;
    for (; ok && it < total; ++it) {
      ok = __all_sync(0xffffffffu, mbar_wait(is_v ? &v_free[it % kStages] : &k_free[it % kStages], ((it / kStages) - 1) & 1));
      if (!ok) break;
      const int page = next_page;
      next_page = page_of(it + 1);
      issue(it, is_v, page);
    }
    // no copy is in flight when the CTA ends
    const int issued = min(it, total);
    for (int j = max(0, issued - kStages); j < issued; ++j)
      mbar_wait(is_v ? &v_here[j % kStages] : &k_full[j % kStages], (j / kStages) & 1);
  } else {
    // ------------------------------------------------------------ V looked through
    const int w = warp - kWScan;                        // pages 2 w and 2 w + 1 of a tile
    for (int it = 0; ok && it < total; ++it) {
      const int st = it % kStages;
      ok = __all_sync(0xffffffffu, mbar_wait(&v_here[st], (it / kStages) & 1));
      if (!ok) break;
      uint8_t* vt = stages + st * kStageBytes + 2 * kHalf + 2 * w * 2048;
      // a lane's pieces: 16 bytes at 512 c of d half 0, then of half 1
      __nv_bfloat162 top = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        const uint4 x = *reinterpret_cast<const uint4*>(vt + (c >> 3) * kHalf + (c & 7) * 512 + 16 * lane);
        const uint32_t e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) top = __hmax2_nan(top, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&e[k])));
      }
      uint32_t far = 0;                                 // of the two pages
      if (__any_sync(0xffffffffu, nonfinite(*reinterpret_cast<const uint32_t*>(&top)))) {
#pragma unroll 1
        for (int c = 0; c < 16; ++c) {
          uint4* at = reinterpret_cast<uint4*>(vt + (c >> 3) * kHalf + (c & 7) * 512 + 16 * lane);
          uint4 x = *at;
          uint32_t e[4] = {x.x, x.y, x.z, x.w};
          bool bad = false;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            bad = bad || nonfinite(e[k]);
            e[k] &= ((e[k] & 0x7F80u) == 0x7F80u ? 0xFFFF0000u : 0xFFFFFFFFu) &
                    ((e[k] & 0x7F800000u) == 0x7F800000u ? 0x0000FFFFu : 0xFFFFFFFFu);
          }
          if (bad) *at = make_uint4(e[0], e[1], e[2], e[3]);
          // 8 lanes hold a row: rows 4 (c % 8) .. + 3 of the two pages
          const uint32_t m = __ballot_sync(0xffffffffu, bad);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if ((m >> (8 * k)) & 0xFFu) far |= 1u << (4 * (c & 7) + k);
        }
        // only keys that a row of the block may see
        const int t = tile_at(it) * kKeys + 32 * w + lane;
        far &= __ballot_sync(0xffffffffu, t <= b_last && (t >= low0 || t < sinks));
        fence_proxy_async();
      }
      if (lane < 2) odd[it & 7][2 * w + lane] = (uint16_t)(far >> (16 * lane));
      __syncwarp();
      if (lane == 0) mbar_arrive(&v_full[st]);
    }
  }
  if (!ok && lane == 0) atomicOr(status, SPEC_ST_DEVICE_WAIT);
  } else {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 200;\n");
  if (total > 0 && (warp & 3) < row_warps) {
    // ------------------------------------------------------------ softmax
    const int h = warp >> 2, ww = warp & 3;
    const int r = 32 * ww + lane, fr = r0 + r;          // tile row, row of the KV head
    const bool live = r < nr;
    const int i = live ? div24(fr, pl.group) : 0;
    const uint32_t tl = tmem + ((uint32_t)(32 * ww) << 16);
    // one lane arrives for the warp: the warp barrier orders the others' writes
    auto arrive = [&](uint64_t* bar) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    const int p = n_past + i, plow = window_low(pl, p);
    bool ok = true, left = false;
    int it = 0;
#pragma unroll 1
    for (int pass = 0; !left && pass < passes; ++pass) {
      const Span sp = span_of(pl, n_past, pass);
      const bool mine = live && i >= sp.i0 && i < sp.i1;
      const int n = pass == 0 ? tl0.n : tl1.n;
      float acc[64];                                    // O of this row, d's 64 h ..
#pragma unroll
      for (int c = 0; c < 64; ++c) acc[c] = 0.f;
      float ref = -INFINITY, lsum = 0.f;                // reference of the exponents (both threads agree)
      bool pending = false;                             // O of tile it - 1 is not in acc yet
      auto pv_wait = [&]() { return (bool)__all_sync(0xffffffffu, mbar_wait(&pv_done, (it - 1) & 1)); };
      auto drain = [&]() {
        pending = false;
        tc_fence_after();
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          uint32_t o[32];
          tmem_ld32(tl + kTmO + 64u * h + 32u * g, o);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 32; ++c) acc[32 * g + c] += __uint_as_float(o[c]);
        }
      };
#pragma unroll 1
      for (int sc = 0; sc < n; ++sc, ++it) {
        const int st = it % kStages, t0 = tile_at(it) * kKeys;
        ok = ok && __all_sync(0xffffffffu, mbar_wait(&s_full, it & 1));
        tc_fence_after();
        float x[64];                                    // scores of keys t0 + 64 h ..
        {
          uint32_t y0[32], y1[32];
          tmem_ld32(tl + kTmS + 64u * h, y0);
          tmem_ld32(tl + kTmS + 64u * h + 32u, y1);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            x[c] = __uint_as_float(y0[c]);
            x[32 + c] = __uint_as_float(y1[c]);
          }
        }
        tc_fence_before();
        if (ok) arrive(&s_free);
        // `masked`: some row of the block does not see some key of the tile
        const uint2 mp = *reinterpret_cast<const uint2*>(&mapped[it & 7][0]);
        if ((mp.x & mp.y) != 0x01010101u || t0 + kKeys - 1 > n_past || (t0 < low1 && t0 + kKeys > sinks) || passes > 1) {
          // keys of this thread that its row sees
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int k0 = t0 + 64 * h + 32 * c;
            const uint32_t two = (h ? mp.y : mp.x) >> (16 * c);
            const uint32_t vis = !mine ? 0u
                                       : low_bits(p + 1 - k0) & (~low_bits(plow - k0) | low_bits(sinks - k0)) &
                                             ((two & 1u ? 0xffffu : 0u) | (two & 0x100u ? 0xffff0000u : 0u));
#pragma unroll
            for (int e = 0; e < 32; ++e) x[32 * c + e] = (vis >> e) & 1u ? x[32 * c + e] : -INFINITY;
          }
        }
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < 64; ++e) m4[e & 3] = fmaxf(m4[e & 3], x[e]);
        float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        // The reference moves only when a score exceeds it by more than 8 (a
        // difference, which is exact for large scores too).  A wait
        // that ran out is carried to this barrier, where the pair of warps leaves
        // together.
        if (!ok) *reinterpret_cast<volatile int*>(&gave_up[ww]) = 1;
        if (named_bar_or(1 + ww, 64, mx - ref > 8.f || !ok)) {
          left = *reinterpret_cast<volatile int*>(&gave_up[ww]) != 0;
          if (left) break;
          pair[h][r] = mx;
          named_bar(1 + ww, 64);
          mx = fmaxf(mx, pair[1 - h][r]);
          if (pending) {                                // O so far is in the old units
            ok = pv_wait();
            if (ok) drain();
          }
          if (mx - ref > 8.f) {
            const float a = ref == -INFINITY ? 1.f : exp2_approx(ref - mx);
            ref = mx;
            lsum *= a;
#pragma unroll
            for (int c = 0; c < 64; ++c) acc[c] *= a;
          }
        }
        const float base = ref == -INFINITY ? 0.f : -ref;
        // P may be rewritten, and O read, once the tile before is done
        if (pending) ok = pv_wait();
        float sum = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {                   // 16 keys each
          uint32_t w[kParts][8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float& a = x[16 * c + 2 * e];
            float& b = x[16 * c + 2 * e + 1];
            a = exp2_approx(a + base);
            b = exp2_approx(b + base);
            sum += a + b;
            float a1 = a, b1 = b;
#pragma unroll
            for (int pt = 0; pt < kParts; ++pt) w[pt][e] = take_bf16(a1, b1);
          }
#pragma unroll
          for (int pt = 0; pt < kParts; ++pt) tmem_st8(tl + kTmP + 64u * pt + 32u * h + 8u * c, w[pt]);
        }
        lsum += sum;
        // V elements that are not finite are zero in the tile: their p v is added
        // here, to the rows that see them
        ok = ok && __all_sync(0xffffffffu, mbar_wait(&v_full[st], (it / kStages) & 1));
        const uint4 far = *reinterpret_cast<const uint4*>(&odd[it & 7][0]);
        if (!ok) *reinterpret_cast<volatile int*>(&gave_up[ww]) = 1;
        if (named_bar_or(1 + ww, 64, (far.x | far.y | far.z | far.w) != 0 || !ok)) {
          left = *reinterpret_cast<volatile int*>(&gave_up[ww]) != 0;
          if (left) break;
          const uint32_t mw[4] = {far.x, far.y, far.z, far.w};
          tmem_wait_st();
          tc_fence_before();
          named_bar(1 + ww, 64);                        // both warps' p are in P
          tc_fence_after();
#pragma unroll 1
          for (int k = 0; k < kKeys; ++k) {
            if (!((mw[k >> 5] >> (k & 31)) & 1u)) continue;
            uint32_t w[kParts];
#pragma unroll
            for (int pt = 0; pt < kParts; ++pt) w[pt] = tmem_ld1(tl + kTmP + 64u * pt + (k >> 1));
            tmem_wait_ld();
            float y1 = 0.f;
#pragma unroll
            for (int pt = 0; pt < kParts; ++pt)
              y1 += __uint_as_float(k & 1 ? w[pt] & 0xFFFF0000u : w[pt] << 16);
            const int t = t0 + k;
            if (mine && t <= p && (t >= plow || t < sinks)) {
              const uint16_t* vr = kv.pool + ((((size_t)page_at(kv, t >> 4) * kv.n_layers + layer) * 2 + 1) * kv.n_kv + kvh) * 2048 +
                                   (t & 15) * 128 + 64 * h;
#pragma unroll
              for (int c = 0; c < 64; ++c) {
                const uint32_t w0 = vr[c];
                if ((w0 & 0x7F80u) == 0x7F80u) acc[c] += y1 * __uint_as_float(w0 << 16);
              }
            }
            __syncwarp();
          }
        }
        if (pending && ok) drain();
        pending = true;
        tmem_wait_st();
        tc_fence_before();
        if (ok) arrive(&p_full);
      }
      if (left || n == 0) continue;
      ok = ok && pv_wait();
      if (ok) drain();
      pair[h][r] = lsum;
      if (!ok) *reinterpret_cast<volatile int*>(&gave_up[ww]) = 1;
      named_bar(1 + ww, 64);
      left = *reinterpret_cast<volatile int*>(&gave_up[ww]) != 0;
      if (left) break;
      if (mine) {
        if (h == 0) part_ml[((size_t)slot * pl.nkv + kvh) * R + fr] = make_float2(ref, lsum + pair[1][r]);
        float4* dst = part_o + (((size_t)slot * pl.nkv + kvh) * 32 + 16 * h) * R + fr;
#pragma unroll
        for (int c = 0; c < 16; ++c) dst[(size_t)c * R] = make_float4(acc[4 * c], acc[4 * c + 1], acc[4 * c + 2], acc[4 * c + 3]);
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

cudaError_t launch_pattn_bf16(const PattnPlan& pl, const KvView& kv, int layer, const float* q, int row_tiles, float* part_o,
                              float2* part_ml, int32_t* status, cudaStream_t st) {
  // the shared-memory limit is a per-device attribute
  constexpr int kMaxDevices = 64;
  static bool have[kMaxDevices] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool known = dev >= 0 && dev < kMaxDevices;
  if (!known || !have[dev]) {
    e = cudaFuncSetAttribute(pattn_bf16_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kBf16Smem);
    if (e != cudaSuccess) return e;
    if (known) have[dev] = true;
  }
  CUtensorMap map;
  e = make_kv_tmap(kv, &map);
  if (e != cudaSuccess) return e;
  return launch_early(pattn_bf16_kernel, dim3(pl.slots, pl.nkv, row_tiles), dim3(kThreads), kBf16Smem, st, q, pl, kv, map, layer,
                      reinterpret_cast<float4*>(part_o), part_ml, status);
}

}  // namespace spec
