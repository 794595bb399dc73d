// pattn_unpack.cuh — pages of a 4-bit cache into the binary16 operand tiles of
// attention for many rows (pattn.cu).
#pragma once
#include "common.cuh"
#include "internal.h"
#include "kv4.cuh"
#include "pattn_plan.cuh"

namespace spec {

constexpr int kHalf = kKeys * 128;                  // one d half of a K or V tile: [key][64 values], 128-byte swizzle
constexpr int kStageBytes = 4 * kHalf;              // K then V, 64 KB
constexpr int kStages = 3;
constexpr int kItemsPerTile = kPagesPerTile / 2;    // what an unpacking warp takes at once: two pages, 32 keys

// barriers of the stages; `_full` counts kItemsPerTile arrivals
struct StageBars {
  uint64_t k_full[kStages], v_full[kStages], k_free[kStages], v_free[kStages];
};

// One key of K or V: codes and scale bytes
struct Raw4 {
  uint4 c[4];
  uint2 s;
};
// p: the page's chunk 0 of the key; scales: from there to its scale bytes
SPEC_DEV void load_key(const uint8_t* p, int scales, bool there, Raw4& r) {
  if (!there) {                                          // unmapped: zeros (its keys are masked)
#pragma unroll
    for (int c = 0; c < 4; ++c) r.c[c] = make_uint4(0, 0, 0, 0);
    r.s = make_uint2(0, 0);
    return;
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) r.c[c] = ldg_now(reinterpret_cast<const uint4*>(p + 256 * c));
  r.s = ldg_now(reinterpret_cast<const uint2*>(p + scales));
}
// the 128 values of a key as binary16 into its row of the tile's d halves (128
// bytes each, 16-byte chunk j at j ^ (row % 8)); the eight lanes of a store phase
// hold different rows % 8, so no two meet in a bank
SPEC_DEV void unpack_key(const Raw4& r, uint8_t* row, int r7) {
  const uint32_t sc[2] = {__vminu4(r.s.x, 0xE2E2E2E2u), __vminu4(r.s.y, 0xE2E2E2E2u)};
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const uint32_t w[4] = {r.c[c].x, r.c[c].y, r.c[c].z, r.c[c].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t s2 = ((sc[c >> 1] >> (8 * (2 * (c & 1) + (j >> 1)))) & 0xFFu) * 0x00800080u;   // (byte << 7) in both halves
      uint32_t f[4];
      e2m1_word(w[j], f);
      *reinterpret_cast<uint4*>(row + (c >> 1) * kHalf + (((4 * (c & 1) + j) ^ r7) << 4)) =
          make_uint4(hmul2_u32(f[0], s2), hmul2_u32(f[1], s2), hmul2_u32(f[2], s2), hmul2_u32(f[3], s2));
    }
  }
}

// Unpacks the tiles of a CTA, warp id of kWarps.  Item g is pages 2 (g % 4) and the
// next of tile g / 4, a key per lane; a warp takes every kWarps-th.  A step waits,
// unpacks and signals for K of one item and V of the item before (whose stage is
// freed later).  The registers hold the next step's keys.  (With items of one page,
// where the bookkeeping weighs more than the unpacking, 208 rows over 32k keys took
// 43 instead of 39 us; filling slots in shared memory by cp.async two steps ahead
// was no faster.)
// mapped: per tile mod 8 and page, whether it is; last_stage: to be waited for
// before the last stage is first written.  False when a wait ran out.
template <int kWarps, class TileAt>
SPEC_DEV bool unpack_tiles(int id, int total, TileAt tile_at, const KvView& kv, int layer, int kvh, uint8_t* stages,
                           StageBars& bar, uint8_t (*mapped)[kPagesPerTile], uint64_t* last_stage) {
  const int lane = threadIdx.x & 31;
  const int items = total * kItemsPerTile;
  auto page_of = [&](int g) {
    return g < items ? page_at(kv, tile_at(g / kItemsPerTile) * kPagesPerTile + 2 * (g % kItemsPerTile) + (lane >> 4)) : -1;
  };
  const uint32_t stride = (uint32_t)(kv.n_layers * 2 * kv.n_kv) * kKv4PageBytes;
  const int t = lane & 15, scales = kKv4Scales + 8 * t - 16 * t;
  const uint8_t* kb = reinterpret_cast<const uint8_t*>(kv.pool) + (size_t)(layer * 2 * kv.n_kv + kvh) * kKv4PageBytes + 16 * t;
  const uint8_t* vb = kb + kv.n_kv * kKv4PageBytes;
  auto load = [&](const uint8_t* base, int page, Raw4& r) {
    load_key(base + (uint64_t)(uint32_t)page * stride, scales, page_ok(kv, page), r);
  };
  // the pages of this V, of this step's K, and of the K after that
  int page = page_of(id), next = page_of(id + kWarps), after = page_of(id + 2 * kWarps);
  bool ok = true;
  Raw4 k, v;
  load(kb, page, k);
  load(vb, page, v);
  for (int g = id - kWarps; ok && g < items; g += kWarps) {
    const int gk = g + kWarps, itk = gk / kItemsPerTile, stk = itk % kStages, it = g / kItemsPerTile, st = it % kStages;
    const bool has_k = gk < items, has_v = g >= 0;
    // the stage, once its former K (V) has been read
    if (has_k && itk >= kStages) ok = mbar_wait(&bar.k_free[stk], ((itk / kStages) - 1) & 1);
    if (has_k && itk == kStages - 1) ok = mbar_wait(last_stage, 0);
    if (has_v && it >= kStages) ok = ok && mbar_wait(&bar.v_free[st], ((it / kStages) - 1) & 1);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    if (has_k) unpack_key(k, stages + stk * kStageBytes + (gk % kItemsPerTile) * 4096 + lane * 128, lane & 7);
    if (has_v) unpack_key(v, stages + st * kStageBytes + 2 * kHalf + (g % kItemsPerTile) * 4096 + lane * 128, lane & 7);
    fence_proxy_async();
    if (has_k && t == 0) mapped[itk & 7][2 * (gk % kItemsPerTile) + (lane >> 4)] = page_ok(kv, has_v ? next : page);
    __syncwarp();
    if (lane == 0) {
      if (has_k) mbar_arrive(&bar.k_full[stk]);
      if (has_v) mbar_arrive(&bar.v_full[st]);
    }
    // K of the step after; V of the item whose K was just unpacked
    load(kb, has_v ? after : next, k);
    if (has_v) {
      load(vb, next, v);
      page = next;
      next = after;
      after = page_of(gk + 2 * kWarps);
    }
  }
  return ok;
}

}  // namespace spec
