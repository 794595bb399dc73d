// pattn_kv4_few.cu — the partials of attention over a 4-bit paged cache (pattn.cu) for
// calls of at most 16 query rows per KV head: one decoded token of a group of up
// to 16 heads, a few rows of smaller groups.
//
// The roles of the MMAs' dimensions are swapped against pattn.cu, whose softmax and
// MMAs cost the same for 13 rows as for 128: keys (and d's) are the 128 rows, the
// query rows are columns, high and low parts side by side (N = 32):
//   S^T[128 keys x 32] = K . [Q_hi; Q_lo]^T,   O^T[128 d x 32] = V^T . [P_hi; P_lo]^T
// A thread of the softmax owns one key and, of O, one d.  A tile's softmax is then
// four warps' work on 16 scores each, and what bounds a tile is unpacking it: 64 KB
// into shared memory and out of it again, on ten warps.
// One token of 52 heads behind 128k keys: XX us (mma.sync on pages unpacked in
// registers: 43; the layout of pattn.cu: 64).
//
// Precision: as pattn.cu.
#include "attn_mma.cuh"
#include "common.cuh"
#include "internal.h"
#include "pattn_plan.cuh"
#include "pattn_unpack.cuh"

namespace spec {

constexpr int N = kFewRows;
// Shared memory: the stages, Q and two P buffers.  Q: 16-byte chunk d / 8 of row r
// (high rows, then low rows) at (d / 8) * 32 N + 16 r.  P: 8 rows of a key at
// (r / 8) * 2048 + 16 key.  TMEM columns: two S buffers of 2N, two O buffers of 2N.
constexpr int kQBytes = 2 * N * 256;
constexpr size_t kSmem = 1024 + (size_t)kStages * kStageBytes + 3 * kQBytes;
constexpr uint32_t kTmO = 4 * N;
constexpr int kTmAll = 8 * N;
// warps: 0-3 softmax (keys and d's 32 w ..), 4 issues the QK MMAs, 5 the PV MMAs,
// 6-15 unpack
constexpr int kSoftWarps = 4, kWQk = 4, kWPv = 5, kWLoad = 6, kUnpackWarps = 10;
constexpr int kThreads = 512;

// 16 consecutive TMEM columns of this warp's 32 lanes (to be waited for)
SPEC_DEV void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
// sum of 2 x 16 columns: high and low parts
SPEC_DEV void tmem_ld_parts(uint32_t taddr, float (&v)[16]) {
  float lo[16];
  tmem_ld16(taddr, v);
  tmem_ld16(taddr + N, lo);
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] += lo[i];
}
// f over the warp's lanes of 16 columns, column lane / 2 in this lane
template <class F>
SPEC_DEV float reduce_columns(const float (&v)[16], int lane, F f) {
  float w[16];
#pragma unroll
  for (int c = 0; c < 16; ++c) w[c] = v[c];
#pragma unroll
  for (int n = 8; n >= 1; n /= 2) {
    const int s = 2 * n;
    const bool up = lane & s;
#pragma unroll
    for (int c = 0; c < n; ++c) {
      const float send = up ? w[c] : w[c + n], keep = up ? w[c + n] : w[c];
      w[c] = f(keep, __shfl_xor_sync(0xffffffffu, send, s));
    }
  }
  return f(w[0], __shfl_xor_sync(0xffffffffu, w[0], 1));
}
// binary16 parts of a pair: hi nearest, lo what is left
SPEC_DEV void split_pair(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x0, x1);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  minus_f16x2(x0, x1, hi);
  const __half2 l = __floats2half2_rn(x0, x1);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}

// grid (slot, KV head)
__global__ void __launch_bounds__(kThreads, 1)
pattn_kv4_few_kernel(const float* __restrict__ q, PattnPlan pl, KvView kv, int layer, float* __restrict__ part_o,
                     float2* __restrict__ part_ml, int32_t* status) {
  extern __shared__ __align__(128) uint8_t dsm[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dsm) + 1023) & ~(uintptr_t)1023);
  uint8_t* qs = sm + kStages * kStageBytes;
  uint8_t* ps = qs + kQBytes;
  __shared__ uint32_t tmem_slot;
  __shared__ __align__(8) uint64_t q_full, s_full[2], p_full[2], pv_done[2];
  __shared__ __align__(8) StageBars bar;
  // per row: score to base-2 units, and minus the exponent of p = 1
  __shared__ __align__(16) float unit[N], nref[N];
  __shared__ float red[4][N];
  // mapped pages per tile (a ring of 8: a tile's entries are rewritten eight tiles
  // later, when its softmax has long been passed)
  __shared__ __align__(8) uint8_t mapped[8][kPagesPerTile];
  __shared__ int gave_up;                               // a wait of the softmax ran out

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slot = blockIdx.x, kvh = blockIdx.y, R = pl.M * pl.group;
  if (warp == kWQk) tmem_alloc(&tmem_slot, kTmAll);
  if (tid == 32 * kWPv) {
    mbar_init(&q_full, kSoftWarps);
    for (int b = 0; b < kStages; ++b) {
      mbar_init(&bar.k_full[b], kItemsPerTile);
      mbar_init(&bar.v_full[b], kItemsPerTile);
      mbar_init(&bar.k_free[b], 1);
      mbar_init(&bar.v_free[b], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&s_full[b], 1);
      mbar_init(&p_full[b], kSoftWarps);
      mbar_init(&pv_done[b], 1);
    }
    gave_up = 0;
    fence_mbarrier_init();
  }
  pdl_trigger();
  pdl_wait();
  const int n_past = __ldcg(kv.seq_len) - pl.M;
  // Q: 16 threads per row, 8 values each (softmax threads: two rows of theirs)
  float4 qa[2], qb[2];
  if (warp < kSoftWarps) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = (tid >> 4) + 8 * j;
      qa[j] = qb[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < R) {
        const int i = div24(r, pl.group);
        const float4* src = reinterpret_cast<const float4*>(
            q + ((size_t)i * pl.nq + kvh * pl.group + r - i * pl.group) * 128 + 8 * (tid & 15));
        qa[j] = src[0];
        qb[j] = src[1];
      }
    }
  }
  const int passes = span_count(pl, n_past);
  TileList tl0 = tiles_of(span_of(pl, n_past, 0), slot), tl1;
  if (passes == 2) tl1 = tiles_of(span_of(pl, n_past, 1), slot);
  const int total = tl0.n + tl1.n;
  auto tile_at = [&](int it) { return it < tl0.n ? tl0.at(it) : tl1.at(it - tl0.n); };
  const int low1 = window_low(pl, n_past + pl.M - 1), sinks = pl.window > 0 ? pl.sinks : 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  if (total == 0) {
    // nothing of this chunk is seen
  } else if (warp >= kWLoad) {
    if (!unpack_tiles<kUnpackWarps>(warp - kWLoad, total, tile_at, kv, layer, kvh, sm, bar, mapped, nullptr) && lane == 0)
      atomicOr(status, SPEC_ST_DEVICE_WAIT);
  } else if (warp == kWQk) {
    // -------------------------------------------------- S^T = K . [Q_hi; Q_lo]^T
    // D f32 (bit 4), A and B f16, N >> 3 at 17, M >> 4 at 24; 8 d steps of 16
    constexpr uint32_t kId = (1u << 4) | ((2u * N >> 3) << 17) | ((128u >> 4) << 24);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t dk0 = desc_sw128(__shfl_sync(0xffffffffu, smem_u32(sm), 0), 16, 1024);
    const uint64_t dq0 = smem_desc(__shfl_sync(0xffffffffu, smem_u32(qs), 0), 32 * N, 128);
    bool ok = __all_sync(0xffffffffu, mbar_wait(&q_full, 0));
    int last = -1;
    for (int it = 0; ok && it < total; ++it) {
      const int st = it % kStages, sb = it & 1;
      bool w = mbar_wait(&bar.k_full[st], (it / kStages) & 1);
      // S of two tiles ago has been read (its P is written).  Its P.V is done
      // too, so S of this tile tells the softmax that that O may be read and
      // that P buffer rewritten.
      if (it >= 2) w = w && mbar_wait(&pv_done[sb], ((it >> 1) - 1) & 1);
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
        mma_commit(&bar.k_free[st]);
      }
      __syncwarp();
      last = it;
    }
    if (!ok && lane == 0) atomicOr(status, SPEC_ST_DEVICE_WAIT);
    if (last >= 0) mbar_wait(&s_full[last & 1], (last >> 1) & 1);   // before TMEM is released
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
      const int st = it % kStages, pb = it & 1;
      ok = __all_sync(0xffffffffu, mbar_wait(&bar.v_full[st], (it / kStages) & 1) && mbar_wait(&p_full[pb], (it >> 1) & 1));
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t dv = dv0 + (uint64_t)((st * kStageBytes) >> 4);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_f16_ss(tm + kTmO + 2u * N * pb, dv + (uint64_t)((kk * 2048) >> 4),
                     dp0 + (uint64_t)((pb * kQBytes + kk * 256) >> 4), kId, kk != 0);
        mma_commit(&pv_done[pb]);
        mma_commit(&bar.v_free[st]);
      }
      __syncwarp();
      last = it;
    }
    if (!ok && lane == 0) atomicOr(status, SPEC_ST_DEVICE_WAIT);
    if (last >= 0) mbar_wait(&pv_done[last & 1], (last >> 1) & 1);
  } else {
    // -------------------------------------------------------------- softmax
    const int key = tid;                                // this thread's key and d
    const uint32_t tl = tmem + ((uint32_t)(32 * warp) << 16);
    constexpr float kBias = 7.f;                        // p = 2^(7 + s - max): binary16 keeps 2^-24 of 2^7
    // A row of Q is scaled by a power of two to at most 2 in magnitude, and its
    // scores are scaled back.
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = (tid >> 4) + 8 * j, ch = tid & 15;
      const float4 a = qa[j], b = qb[j];
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
      // log2(e) / sqrt(d) times the row's power of two; no reference yet
      if (ch == 0) {
        unit[r] = (1.4426950408889634f / sqrtf(128.0f)) * __uint_as_float((uint32_t)(127 + e) << 23);
        nref[r] = r < R ? INFINITY : 0.f;
      }
    }
    // the warps' arrivals: every lane's writes are ordered by the warp barrier
    auto arrive = [&](uint64_t* b) {
      __syncwarp();
      if (lane == 0) mbar_arrive(b);
    };
    fence_proxy_async();
    arrive(&q_full);
    named_bar(1, 128);                                  // `unit` and `nref` are written
    bool ok = true, left = false;
    int it = 0;
#pragma unroll 1
    for (int pass = 0; !left && pass < passes; ++pass) {
      const Span sp = span_of(pl, n_past, pass);
      const int n = pass == 0 ? tl0.n : tl1.n;
      float acc[N], lsum[N];                            // by row
#pragma unroll
      for (int c = 0; c < N; ++c) acc[c] = lsum[c] = 0.f;
      if (pass > 0) {
        // new maxima; the threads that still read the old ones are behind this barrier
        named_bar(1, 128);
        if (tid < R) nref[tid] = INFINITY;
        named_bar(1, 128);
      }
      int drained = it;                                 // tiles before this one are in acc
      // adds O of a finished tile in fp32
      auto add_o = [&]() {
        float o[16];
        tmem_ld_parts(tl + kTmO + 2u * N * (drained & 1), o);
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] += o[e];
        ++drained;
      };
      // the tiles whose P.V may still run
      auto drain = [&](int upto) -> bool {
        while (drained < upto) {
          if (!__all_sync(0xffffffffu, mbar_wait(&pv_done[drained & 1], (drained >> 1) & 1))) return false;
          tc_fence_after();
          add_o();
        }
        return true;
      };
#pragma unroll 1
      for (int sc = 0; sc < n; ++sc, ++it) {
        const int sb = it & 1, t0 = tile_at(it) * kKeys, t = t0 + key;
        const bool got = __all_sync(0xffffffffu, mbar_wait(&s_full[sb], (it >> 1) & 1));
        tc_fence_after();
        // rows that see this thread's key; `masked`: some row of the block does
        // not see some key of the tile
        const uint2 mp = *reinterpret_cast<const uint2*>(&mapped[it & 7][0]);
        uint32_t vis = 0xffffffffu;
        const bool masked = (mp.x & mp.y) != 0x01010101u || t0 + kKeys - 1 > n_past || (t0 < low1 && t0 + kKeys > sinks) ||
                            passes > 1;
        if (masked) {
          const long long d = (long long)t - n_past;    // rows i >= d, and i < d + window
          const int from = (int)(d < sp.i0 ? sp.i0 : (d > sp.i1 ? sp.i1 : d));
          const long long e = pl.window > 0 && t >= sinks ? d + pl.window : pl.M;
          const int to = (int)(e < sp.i1 ? (e < 0 ? 0 : e) : sp.i1);
          vis = low_bits(min(to * pl.group, R)) & ~low_bits(from * pl.group);
          if (!mapped[it & 7][key >> 4]) vis = 0u;
        }
        float x[N];
        // exponents of the visible scores over the rows' references
        auto exponents = [&]() {
#pragma unroll
          for (int e = 0; e < N; e += 4) {
            const float4 un = *reinterpret_cast<const float4*>(&unit[e]), nf = *reinterpret_cast<const float4*>(&nref[e]);
            x[e] = fmaf(x[e], un.x, nf.x);
            x[e + 1] = fmaf(x[e + 1], un.y, nf.y);
            x[e + 2] = fmaf(x[e + 2], un.z, nf.z);
            x[e + 3] = fmaf(x[e + 3], un.w, nf.w);
          }
          if (masked) {
#pragma unroll
            for (int e = 0; e < N; ++e) x[e] = (vis >> e) & 1u ? x[e] : -INFINITY;
          }
        };
        // does some p exceed 2^15?  The first tile has no references yet.
        tmem_ld_parts(tl + 2u * N * sb, x);
        if (drained < it - 1) add_o();                  // two tiles ago: done when S is (see the QK warp)
        bool over = sc == 0;
        if (sc > 0) {
          exponents();
          float top = -INFINITY;
#pragma unroll
          for (int e = 0; e < N; ++e) top = fmaxf(top, x[e]);
          over = top > 8.f + kBias;
        }
        // a wait that ran out is carried to this barrier, where the four warps
        // leave together
        if (!got || !ok) *reinterpret_cast<volatile int*>(&gave_up) = 1;
        if (named_bar_or(1, 128, over || !got || !ok)) {
          left = *reinterpret_cast<volatile int*>(&gave_up) != 0;
          if (left) break;
          // each row's largest score of the tile; where it exceeds the
          // reference by more than 8 it becomes the reference
          if (sc > 0) tmem_ld_parts(tl + 2u * N * sb, x);
          float y[N];
#pragma unroll
          for (int e = 0; e < N; ++e) y[e] = (vis >> e) & 1u ? x[e] * unit[e] : -INFINITY;
          red[warp][lane >> 1] = reduce_columns(y, lane, [](float a, float b) { return fmaxf(a, b); });
          ok = drain(it);                               // O so far is in the old units
          named_bar(1, 128);
          if (tid < N) {
            const float m = fmaxf(fmaxf(red[0][tid], red[1][tid]), fmaxf(red[2][tid], red[3][tid]));
            const float old = -nref[tid];               // reference - 7; -inf at first
            float a = 1.f;
            if (m - kBias > old + 8.f) {
              if (old != -INFINITY) a = exp2_approx(old - (m - kBias));
              nref[tid] = kBias - m;
            }
            red[0][tid] = a;
          }
          named_bar(1, 128);
          if (sc > 0) {
#pragma unroll
            for (int c = 0; c < N; ++c) {
              const float a = red[0][c];
              acc[c] *= a;
              lsum[c] *= a;
            }
          }
          exponents();
        }
        uint8_t* pt = ps + sb * kQBytes + key * 16;
#pragma unroll
        for (int e = 0; e < N; ++e) x[e] = exp2_approx(x[e]);
#pragma unroll
        for (int e = 0; e < N; e += 8) {
          uint4 hi, lo;
          split_pair(x[e], x[e + 1], hi.x, lo.x);
          split_pair(x[e + 2], x[e + 3], hi.y, lo.y);
          split_pair(x[e + 4], x[e + 5], hi.z, lo.z);
          split_pair(x[e + 6], x[e + 7], hi.w, lo.w);
          *reinterpret_cast<uint4*>(pt + (e >> 3) * 2048) = hi;
          *reinterpret_cast<uint4*>(pt + ((N + e) >> 3) * 2048) = lo;
        }
        tc_fence_before();
        fence_proxy_async();
        if (ok) arrive(&p_full[sb]);
#pragma unroll
        for (int e = 0; e < N; ++e) lsum[e] += x[e];
      }
      if (left || n == 0) continue;
      ok = ok && drain(it);
      left = named_bar_or(1, 128, !ok);
      if (left) break;
      // the row sums over the 128 keys: lanes, then the four warps in order
      red[warp][lane >> 1] = reduce_columns(lsum, lane, [](float a, float b) { return a + b; });
      named_bar(1, 128);
      const int from = sp.i0 * pl.group, lim = min(R, sp.i1 * pl.group);
      if (tid < lim && tid >= from)
        part_ml[((size_t)slot * pl.nkv + kvh) * R + tid] =
            make_float2(-nref[tid], ((red[0][tid] + red[1][tid]) + red[2][tid]) + red[3][tid]);
      // [slot][KV head][d / 4][row][d % 4]
      float* dst = part_o + (((size_t)slot * pl.nkv + kvh) * 32 + (key >> 2)) * R * 4 + (key & 3);
#pragma unroll
      for (int c = 0; c < N; ++c)
        if (c < lim && c >= from) dst[4 * c] = acc[c];
      named_bar(1, 128);
    }
    if (left && lane == 0) atomicOr(status, SPEC_ST_DEVICE_WAIT);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWQk) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmAll);
  }
}

cudaError_t launch_pattn_kv4_few(const PattnPlan& pl, const KvView& kv, int layer, const float* q, float* part_o,
                                 float2* part_ml, int32_t* status, cudaStream_t st) {
  // the shared-memory limit is a per-device attribute
  constexpr int kMaxDevices = 64;
  static bool have[kMaxDevices] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool known = dev >= 0 && dev < kMaxDevices;
  if (!known || !have[dev]) {
    e = cudaFuncSetAttribute(pattn_kv4_few_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
    if (known) have[dev] = true;
  }
  pattn_kv4_few_kernel<<<dim3(pl.slots, pl.nkv), kThreads, kSmem, st>>>(q, pl, kv, layer, part_o, part_ml, status);
  return cudaGetLastError();
}

}  // namespace spec
