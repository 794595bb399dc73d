// pattn_few.cu — the partials of attention over a paged cache (pattn.cu) for calls
// of at most 16 query rows per KV head: one decoded token of a group of up to 16
// heads, a few rows of smaller groups.
//
// The tcgen05 kernels pay for 128 rows whatever their number.  Here the 16 rows are
// one m16n8k16 fragment: 512 (bf16: 768) warp MMAs a tile of 128 keys.
//
// The warps of a CTA (slot, KV head) take the pages of its chunk in turn, 4-bit ones
// two at a time, with a running (max, sum) and O of their own in registers; they are
// joined in order at the end.  Pages fall to warps by their number, so a row's bits
// do not depend on the block.  Each warp has a ring of pages in shared memory that
// it fills by cp.async (16 bytes per lane; bulk copies to padded places are issued
// lane by lane and cost 150 instructions a page).
//
// What bounds it: the dependent steps of a few warps.  A 4-bit page is 520 warp
// instructions, 64 of them MMAs of 8 cycles; two warps per scheduler fill 42 % of the
// slots, 2,300 cycles a tile against 800 at the SM's share of HBM.  One token of 52
// heads on 4 behind 128k keys: 40.3 us in 4 bits, 59.7 in bf16; 7.8 us behind 2k keys,
// 8.5 for a bf16 window of 1024.  (An earlier build took 41, 61, 8.1, of which the
// join was 3, and 9.4; with 12 warps of 168 registers 40, 60, 8.7 and 10.4.  One
// 4-bit page at a time: 5 % slower.  Pages loaded into registers in fragment order: 52
// when this took 43.  Keys on the 128 rows of tcgen05 MMAs and query rows as columns:
// 42, with twice the code.)
//
// The d's of a K row and the d's and keys of a V page may be visited in any
// order.  Lane 4n + g (g < 4) takes d's 32 g .. of K (one 16-byte chunk of codes, 64
// bytes of bf16), and d's 16 n .. of keys 4 g .. of V:
//   S: B fragment of MMA ks: elements 4 ks .. 4 ks + 3 of the lane's chunk (bf16:
//      with its 16-byte pieces in the order c ^ (g / 2), for the banks); column n
//      of key tile nt (of two) is key 4 (n / 2) + n % 2 + 2 nt, so that a lane's
//      scores are those of keys 4 g .. 4 g + 3, its V rows
//   O: column n of MMA j is d 16 n + j
//
// Precision: as pattn.cu for the 4-bit cache (binary16, q and p in two parts,
// row-wise powers of two).  bf16 pages are operands as they are, with q and p in
// three bf16 parts by truncation (24 significant bits): no value is out of range.
// A unit's O is added up in fp32, since the MMAs truncate: left in their accumulators
// over the 27 pages of a warp it was off by 1.2e-6 instead of 4e-7 (and 2.5 us faster).
#include "attn_mma.cuh"
#include "common.cuh"
#include "internal.h"
#include "kv4.cuh"
#include "pattn_plan.cuh"

namespace spec {

constexpr int kFewWarps = 8;
constexpr int kOPitch = 132;               // floats between rows of a warp's O in shared memory
// A warp's ring of pages in shared memory.  Where a piece of 16 bytes lies keeps
// the eight lanes of a load phase in different banks:
//   4-bit: piece 16 c + t (chunk column c, key t) at 288 c + 16 t, then the scales
//   bf16:  K row t at 288 t, V row t at 272 t + 16 (t / 8)
template <bool k4>
struct FewRing {
  static constexpr int kPg = k4 ? 2 : 1;                // pages of a unit
  static constexpr int kK = k4 ? 4 * 288 + 128 : 16 * 288, kV = k4 ? kK : 16 * 272 + 16;
  static constexpr int kSlots = 3;
  static constexpr int kWarp = kSlots * kPg * (kK + kV), kO = 4 * kFewWarps * kFewRows * kOPitch;
  static constexpr size_t kSmem = kFewWarps * kWarp > kO ? kFewWarps * kWarp : kO;
};
template <bool k4>
SPEC_DEV void mma16816(float (&c)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  if constexpr (k4)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
// the same onto zero
template <bool k4>
SPEC_DEV void mma16816_first(float (&c)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  if constexpr (k4)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1), "f"(0.f));
}
// the operand part of a pair (x0 in the low half); x becomes what is left
template <bool k4>
SPEC_DEV uint32_t take_part(float& x0, float& x1) {
  if constexpr (k4) {
    const __half2 h = __floats2half2_rn(x0, x1);
    minus_f16x2(x0, x1, *reinterpret_cast<const uint32_t*>(&h));
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    return take_bf16(x0, x1);
  }
}

SPEC_DEV uint32_t word_of(const uint4& x, int i) { return i == 0 ? x.x : (i == 1 ? x.y : (i == 2 ? x.z : x.w)); }
// f16 pair of byte b of w
template <int B>
SPEC_DEV uint32_t e2m1_byte(uint32_t w) {
  uint32_t r;
  if constexpr (B == 0)
    asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %1;\n cvt.rn.f16x2.e2m1x2 %0, a;\n}\n" : "=r"(r) : "r"(w));
  if constexpr (B == 1)
    asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %1;\n cvt.rn.f16x2.e2m1x2 %0, b;\n}\n" : "=r"(r) : "r"(w));
  if constexpr (B == 2)
    asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %1;\n cvt.rn.f16x2.e2m1x2 %0, c;\n}\n" : "=r"(r) : "r"(w));
  if constexpr (B == 3)
    asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %1;\n cvt.rn.f16x2.e2m1x2 %0, d;\n}\n" : "=r"(r) : "r"(w));
  return r;
}
SPEC_DEV uint32_t e2m1_pick(uint32_t w, int b) {        // b known at compile time after unrolling
  return b == 0 ? e2m1_byte<0>(w) : (b == 1 ? e2m1_byte<1>(w) : (b == 2 ? e2m1_byte<2>(w) : e2m1_byte<3>(w)));
}
// the scale of a byte in both halves
SPEC_DEV uint32_t scale_pair(uint32_t byte) { return byte * 0x00800080u; }

template <bool k4>
__global__ void __launch_bounds__(32 * kFewWarps, 1)
pattn_few_kernel(const float* __restrict__ q, PattnPlan pl, KvView kv, int layer, float* __restrict__ part_o,
                 float2* __restrict__ part_ml) {
  constexpr int kParts = k4 ? 2 : 3;                    // of q and p
  // p = 2^(bias + s - max), s - max at most the lag: 2^15 in binary16, where the bias
  // rounds to at most 8 beside large scores
  constexpr float kBias = k4 ? 7.f : 0.f, kLag = k4 ? 7.f : 8.f;
  constexpr int kPageBytes = k4 ? kKv4PageBytes : 4096;
  using Ring = FewRing<k4>;
  constexpr int kWarps = kFewWarps, kPg = Ring::kPg, kUnitsPerTile = kPagesPerTile / kPg;
  extern __shared__ __align__(128) uint8_t sm[];
  float* o_sm = reinterpret_cast<float*>(sm);           // [warp][row][kOPitch], where the rings were
  __shared__ uint4 qs[kParts][8][32];                   // A fragments
  __shared__ int qmax[kFewRows];
  __shared__ float2 ml_sm[kWarps][kFewRows];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, n = lane >> 2, g = lane & 3;
  const int slot = blockIdx.x, kvh = blockIdx.y, R = pl.M * pl.group;
  if (tid < kFewRows) qmax[tid] = 0;
  uint8_t* ring = sm + warp * Ring::kWarp;
  pdl_wait();
  pdl_trigger();                                        // not before: see the merge in pattn.cu
  const int n_past = ldg_now(kv.seq_len) - pl.M;
  // this thread's rows n and n + 8; in the first 8 warps the Q elements of MMA
  // `warp` (bf16: the 16-byte pieces of a K row in an order that depends on g)
  const int q_at = k4 ? 32 * g + 4 * warp : 32 * g + 8 * ((warp >> 1) ^ (g >> 1)) + 4 * (warp & 1);
  float4 qv[2];
  int pos[2], plow[2], row_i[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = n + 8 * h;
    row_i[h] = r < R ? div24(r, pl.group) : -1;
    pos[h] = n_past + row_i[h];
    plow[h] = window_low(pl, pos[h]);
    qv[h] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < R && warp < 8)
      qv[h] = ldg_now(reinterpret_cast<const float4*>(
          q + ((size_t)row_i[h] * pl.nq + kvh * pl.group + r - row_i[h] * pl.group) * 128 + q_at));
  }
  const int passes = span_count(pl, n_past);
  TileList tl0 = tiles_of(span_of(pl, n_past, 0), slot), tl1;
  if (passes == 2) tl1 = tiles_of(span_of(pl, n_past, 1), slot);
  if (tl0.n + tl1.n == 0) return;
  const int b_last = n_past + pl.M - 1;                 // the block's last position
  const int low0 = window_low(pl, n_past), low1 = window_low(pl, b_last), sinks = pl.window > 0 ? pl.sinks : 0;

  const uint32_t stride = (uint32_t)(kv.n_layers * 2 * kv.n_kv * kPageBytes);
  const uint8_t* kbase = reinterpret_cast<const uint8_t*>(kv.pool) + (size_t)(layer * 2 * kv.n_kv + kvh) * kPageBytes;
  const uint8_t* vbase = kbase + (size_t)kv.n_kv * kPageBytes;

  // This warp's units of kPg pages: those of the chunk whose number is `warp` mod
  // kWarps.
  TileList tl;
  int f0, f1, c0, units;
  auto page_no = [&](int j) {                           // first page of unit j
    return kPg * (j < c0 ? tl.a0 * kUnitsPerTile + f0 + kWarps * j : tl.a1 * kUnitsPerTile + f1 + kWarps * (j - c0));
  };
  struct Ids {
    int id[kPg];
  };
  auto ids_of = [&](int j) {
    Ids r;
#pragma unroll
    for (int pg = 0; pg < kPg; ++pg) r.id[pg] = j < units ? page_at(kv, page_no(j) + pg) : -1;
    return r;
  };
  // Copies page pg of unit j into slot b if it is mapped and some row of the block
  // sees a key of it; whether it was.
  auto fetch_page = [&](int j, int id, int b, int pg) {
    if (!page_ok(kv, id)) return false;
    const int k0 = 16 * (page_no(j) + pg);
    if (k0 > b_last || (k0 + 15 < low0 && k0 >= sinks)) return false;
    uint8_t* dst = ring + (b * kPg + pg) * (Ring::kK + Ring::kV);
    const uint8_t* kp = kbase + (uint64_t)(uint32_t)id * stride;
    const uint8_t* vp = vbase + (uint64_t)(uint32_t)id * stride;
    if constexpr (k4) {
      const int at = 288 * (lane >> 4) + 16 * (lane & 15);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        copy16(dst + at + 576 * i, kp + 16 * lane + 512 * i);
        copy16(dst + Ring::kK + at + 576 * i, vp + 16 * lane + 512 * i);
      }
      if (lane < 16)                                    // the scales of K, of V
        copy16(dst + (lane < 8 ? 0 : Ring::kK) + 4 * 288 + 16 * (lane & 7), (lane < 8 ? kp : vp) + kKv4Scales + 16 * (lane & 7));
    } else {
      const int t0 = lane >> 4, at = 16 * (lane & 15);
#pragma unroll
      for (int i = 0; i < 8; ++i) {                     // rows 2 i + t0
        copy16(dst + 288 * (2 * i + t0) + at, kp + 16 * lane + 512 * i);
        copy16(dst + Ring::kK + 272 * (2 * i + t0) + 16 * (i >> 2) + at, vp + 16 * lane + 512 * i);
      }
    }
    return true;
  };
  uint32_t have = 0;                                    // bit kPg b + pg: slot b holds that page, or will
  auto fetch = [&](int j, const Ids& ids, int b) {
    have &= ~(((1u << kPg) - 1u) << (kPg * b));
    if (j < units) {
#pragma unroll
      for (int pg = 0; pg < kPg; ++pg)
        if (fetch_page(j, ids.id[pg], b, pg)) have |= 1u << (kPg * b + pg);
    }
    copy_commit();
  };
  Ids id_next, id_after;                                // of the two units behind those of the ring
  auto start = [&](int pass) {
    tl = pass == 0 ? tl0 : tl1;
    const int n0 = tl.n0 * kUnitsPerTile, n1 = (tl.n - tl.n0) * kUnitsPerTile;
    auto first_of = [&](int from) { return (int)((unsigned)(warp + kWarps - (unsigned)from % kWarps) % kWarps); };
    f0 = first_of(tl.a0 * kUnitsPerTile);
    f1 = first_of(tl.a1 * kUnitsPerTile);
    c0 = n0 > f0 ? (n0 - f0 + kWarps - 1) / kWarps : 0;
    units = c0 + (n1 > f1 ? (n1 - f1 + kWarps - 1) / kWarps : 0);
    Ids id[Ring::kSlots];
#pragma unroll
    for (int b = 0; b < Ring::kSlots; ++b) id[b] = ids_of(b);
    id_next = ids_of(Ring::kSlots);
    id_after = ids_of(Ring::kSlots + 1);
#pragma unroll
    for (int b = 0; b < Ring::kSlots; ++b) fetch(b, id[b], b);
  };
  start(0);

  // log2(e) / sqrt(d), for the 4-bit cache times the row's power of two
  float unit[2];
  unit[0] = unit[1] = 1.4426950408889634f / sqrtf(128.0f);
  __syncthreads();
  if (k4) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float m = fmaxf(fmaxf(fabsf(qv[h].x), fabsf(qv[h].y)), fmaxf(fabsf(qv[h].z), fabsf(qv[h].w)));
      atomicMax(&qmax[n + 8 * h], __float_as_int(m));   // magnitudes order as integers
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int e = min(max(((qmax[n + 8 * h] >> 23) & 255) - 127, -100), 126);
      const float mul = __uint_as_float((uint32_t)(127 - e) << 23);
      unit[h] *= __uint_as_float((uint32_t)(127 + e) << 23);
      qv[h].x *= mul;
      qv[h].y *= mul;
      qv[h].z *= mul;
      qv[h].w *= mul;
    }
  }
#pragma unroll
  for (int pt = 0; pt < kParts; ++pt) {
    uint4 a;
    a.x = take_part<k4>(qv[0].x, qv[0].y);
    a.y = take_part<k4>(qv[1].x, qv[1].y);
    a.z = take_part<k4>(qv[0].z, qv[0].w);
    a.w = take_part<k4>(qv[1].z, qv[1].w);
    if (warp < 8) qs[pt][warp][lane] = a;
  }
  __syncthreads();

  // An element of V that is not finite makes every row of its MMA infinite or NaN,
  // the rows that do not see its key too.  Where that happened the pass is run again
  // without such elements, and each is then added to the rows that see it: one rule
  // for every row, whatever the others of its block see.
  bool again = false;
#pragma unroll 1
  for (int pass = 0; pass < passes;) {
    const Span sp = span_of(pl, n_past, pass);
    bool mine[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) mine[h] = row_i[h] >= sp.i0 && row_i[h] < sp.i1;
    float o[16][4];
#pragma unroll
    for (int j = 0; j < 16; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    float ref[2] = {-INFINITY, -INFINITY}, lsum[2] = {0.f, 0.f};

    int b = 0;                                          // slot of unit j
#pragma unroll 1
    for (int j = 0; j < units; ++j) {
      copy_wait<Ring::kSlots - 1>();
      __syncwarp();
      const uint32_t there = (have >> (kPg * b)) & ((1u << kPg) - 1u);
      if (there) {
        const uint8_t* kp = ring + b * kPg * (Ring::kK + Ring::kV);
        const uint8_t* vp = kp + Ring::kK;
        constexpr int kPgBytes = Ring::kK + Ring::kV;
        const int k0 = 16 * page_no(j);
        // ------------------------------------------------ S = Q . K^T
        float s[kPg][2][2][4] = {};                     // [page][key tile][high part, low parts]
        uint32_t ksc[kPg][2][2], vs_word[kPg];          // vs_word: word `lane` of V's scales, groups 4 (lane % 2).. of key lane / 2
        uint4 kc[kPg][2];
        if constexpr (k4) {
#pragma unroll
          for (int pg = 0; pg < kPg; ++pg) {
            const uint32_t ks_word =
                __vminu4(*reinterpret_cast<const uint32_t*>(kp + pg * kPgBytes + 4 * 288 + 4 * lane), 0x01010101u * kKv4TopScale);
            vs_word[pg] =
                __vminu4(*reinterpret_cast<const uint32_t*>(vp + pg * kPgBytes + 4 * 288 + 4 * lane), 0x01010101u * kKv4TopScale);
            // scales 2 g and 2 g + 1 of this lane's keys
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
              const uint32_t w =
                  __shfl_sync(0xffffffffu, ks_word, 2 * (4 * (n >> 1) + (n & 1) + 2 * nt) + (g >> 1)) >> (16 * (g & 1));
              ksc[pg][nt][0] = scale_pair(w & 0xFFu);
              ksc[pg][nt][1] = scale_pair((w >> 8) & 0xFFu);
            }
          }
        }
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          uint32_t kb[kPg][2][2];
#pragma unroll
          for (int pg = 0; pg < kPg; ++pg)
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
              const int t = 4 * (n >> 1) + (n & 1) + 2 * nt;      // this lane's key
              const uint8_t* at = kp + pg * kPgBytes;
              if constexpr (k4) {
                if (ks == 0) kc[pg][nt] = *reinterpret_cast<const uint4*>(at + 288 * g + 16 * t);
                const uint32_t w = word_of(kc[pg][nt], ks >> 1), s2 = ksc[pg][nt][ks >> 2];
                kb[pg][nt][0] = hmul2_u32(e2m1_pick(w, 2 * (ks & 1)), s2);
                kb[pg][nt][1] = hmul2_u32(e2m1_pick(w, 2 * (ks & 1) + 1), s2);
              } else {
                if ((ks & 1) == 0)
                  kc[pg][nt] = *reinterpret_cast<const uint4*>(at + 288 * t + 64 * g + 16 * ((ks >> 1) ^ (g >> 1)));
                kb[pg][nt][0] = word_of(kc[pg][nt], 2 * (ks & 1));
                kb[pg][nt][1] = word_of(kc[pg][nt], 2 * (ks & 1) + 1);
              }
            }
#pragma unroll
          for (int pt = kParts - 1; pt >= 0; --pt) {
            const uint4 a = qs[pt][ks][lane];
#pragma unroll
            for (int pg = 0; pg < kPg; ++pg)
#pragma unroll
              for (int nt = 0; nt < 2; ++nt) mma16816<k4>(s[pg][nt][pt > 0], a, kb[pg][nt][0], kb[pg][nt][1]);
          }
        }
        // x[pg][h][e]: row n + 8 h, key k0 + 16 pg + 4 g + e
        float x[kPg][2][4];
#pragma unroll
        for (int pg = 0; pg < kPg; ++pg)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              x[pg][h][e] = (s[pg][e >> 1][0][2 * h + (e & 1)] + s[pg][e >> 1][1][2 * h + (e & 1)]) * unit[h];
        uint2 v4[kPg][4];                               // V pieces of this lane's four keys
        uint4 v16[4][2];
#pragma unroll
        for (int pg = 0; pg < kPg; ++pg)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int t = 4 * g + e;
            const uint8_t* at = vp + pg * kPgBytes;
            if constexpr (k4)
              v4[pg][e] = *reinterpret_cast<const uint2*>(at + 288 * (n >> 1) + 16 * t + 8 * (n & 1));
            else
#pragma unroll
              for (int c = 0; c < 2; ++c)
                v16[e][c] = *reinterpret_cast<const uint4*>(at + 272 * t + 16 * (g >> 1) + 32 * n + 16 * c);
          }
        // some row of the block does not see some key of the pages
        const bool masked = there != (1u << kPg) - 1u || k0 + 16 * kPg - 1 > n_past || (k0 < low1 && k0 + 16 * kPg > sinks) ||
                            passes > 1;
        if (masked) {
#pragma unroll
          for (int pg = 0; pg < kPg; ++pg)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int t = k0 + 16 * pg + 4 * g + e;
                if (!(((there >> pg) & 1u) && mine[h] && t <= pos[h] && (t >= plow[h] || t < sinks))) x[pg][h][e] = -INFINITY;
              }
        }
        if constexpr (!k4) {
          // V rows that no row sees are zeroed (stale bytes may be anything, and
          // 0 * NaN is NaN), on a second pass every element that is not finite
          if (masked || again) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int t = k0 + 4 * g + e;
              const bool seen = t <= b_last && (t >= low0 || t < sinks);
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                uint32_t* w = reinterpret_cast<uint32_t*>(&v16[e][c]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const bool lo = (w[i] & 0x7F80u) == 0x7F80u, hi = (w[i] & 0x7F800000u) == 0x7F800000u;
                  w[i] = !seen ? 0u : !again ? w[i] : w[i] & (lo ? 0xFFFF0000u : 0xFFFFFFFFu) & (hi ? 0x0000FFFFu : 0xFFFFFFFFu);
                }
              }
            }
          }
        }
        float mx[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          mx[h] = -INFINITY;
#pragma unroll
          for (int pg = 0; pg < kPg; ++pg)
            mx[h] = fmaxf(mx[h], fmaxf(fmaxf(x[pg][h][0], x[pg][h][1]), fmaxf(x[pg][h][2], x[pg][h][3])));
        }
        // the reference moves only when a score exceeds it by more than kLag (a
        // difference, which is exact for large scores too)
        if (__any_sync(0xffffffffu, mx[0] - ref[0] > kLag || mx[1] - ref[1] > kLag)) {
          float a[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
            mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
            a[h] = 1.f;
            if (mx[h] - ref[h] > kLag) {
              if (ref[h] != -INFINITY) a[h] = exp2_approx(ref[h] - mx[h]);
              ref[h] = mx[h];
            }
            lsum[h] *= a[h];
          }
#pragma unroll
          for (int jj = 0; jj < 16; ++jj) {
            o[jj][0] *= a[0];
            o[jj][1] *= a[0];
            o[jj][2] *= a[1];
            o[jj][3] *= a[1];
          }
        }
        uint4 pa[kPg][kParts];
#pragma unroll
        for (int pg = 0; pg < kPg; ++pg) {
          float (&xp)[2][4] = x[pg];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float base = kBias - (ref[h] == -INFINITY ? 0.f : ref[h]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              xp[h][e] = exp2_approx(xp[h][e] + base);
              lsum[h] += xp[h][e];
            }
          }
#pragma unroll
          for (int pt = 0; pt < kParts; ++pt) {
            pa[pg][pt].x = take_part<k4>(xp[0][0], xp[0][1]);
            pa[pg][pt].y = take_part<k4>(xp[1][0], xp[1][1]);
            pa[pg][pt].z = take_part<k4>(xp[0][2], xp[0][3]);
            pa[pg][pt].w = take_part<k4>(xp[1][2], xp[1][3]);
          }
        }
        // ------------------------------------------------ O += P . V
        uint32_t s2[kPg][4];
        if constexpr (k4) {
#pragma unroll
          for (int pg = 0; pg < kPg; ++pg)
#pragma unroll
            for (int e = 0; e < 4; ++e)                 // scale byte n of keys 4 g + e
              s2[pg][e] =
                  scale_pair((__shfl_sync(0xffffffffu, vs_word[pg], 2 * (4 * g + e) + (n >> 2)) >> (8 * (n & 3))) & 0xFFu);
        }
#pragma unroll
        for (int i = 0; i < 8; i += 2) {                // d's 16 n + 2i .. 2i + 3: four independent sums
          float oi[4][4];                               // of this unit
#pragma unroll
          for (int pg = 0; pg < kPg; ++pg) {
            uint32_t vb[4][2];
#pragma unroll
            for (int ii = 0; ii < 2; ++ii) {
              uint32_t v[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if constexpr (k4)
                  v[e] = hmul2_u32(e2m1_pick(i < 4 ? v4[pg][e].x : v4[pg][e].y, (i & 3) + ii), s2[pg][e]);
                else
                  v[e] = word_of(v16[e][i >> 2], (i & 3) + ii);
              }
#pragma unroll
              for (int hl = 0; hl < 2; ++hl) {
                const uint32_t sel = hl ? 0x7632u : 0x5410u;
                vb[2 * ii + hl][0] = __byte_perm(v[0], v[1], sel);
                vb[2 * ii + hl][1] = __byte_perm(v[2], v[3], sel);
              }
            }
#pragma unroll
            for (int pt = kParts - 1; pt >= 0; --pt)
#pragma unroll
              for (int jj = 0; jj < 4; ++jj) {
                if (pg == 0 && pt == kParts - 1)
                  mma16816_first<k4>(oi[jj], pa[pg][pt], vb[jj][0], vb[jj][1]);
                else
                  mma16816<k4>(oi[jj], pa[pg][pt], vb[jj][0], vb[jj][1]);
              }
          }
#pragma unroll
          for (int jj = 0; jj < 4; ++jj)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[2 * i + jj][c] += oi[jj][c];
        }
      }
      // the slot takes unit j + kSlots
      __syncwarp();
      fetch(j + Ring::kSlots, id_next, b);
      id_next = id_after;
      id_after = ids_of(j + Ring::kSlots + 2);
      b = b + 1 == Ring::kSlots ? 0 : b + 1;
    }
    __syncthreads();                                    // the rings are free
    // ---- join the warps, in order.  Row n + 8 h, d's 32 g + 16 e + (MMA index).
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      lsum[h] += __shfl_xor_sync(0xffffffffu, lsum[h], 1);
      lsum[h] += __shfl_xor_sync(0xffffffffu, lsum[h], 2);
      if (g == 0) ml_sm[warp][n + 8 * h] = make_float2(ref[h] - kBias, lsum[h]);
      float* dst = o_sm + ((size_t)warp * kFewRows + n + 8 * h) * kOPitch + 32 * g;
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          // the lanes of a store phase are two rows and four g: pieces in an
          // order rotated by g fall into different banks
          const int cc = (c + g) & 3;
          float4 y;
          y.x = cc == 0 ? o[0][2 * h + e] : (cc == 1 ? o[4][2 * h + e] : (cc == 2 ? o[8][2 * h + e] : o[12][2 * h + e]));
          y.y = cc == 0 ? o[1][2 * h + e] : (cc == 1 ? o[5][2 * h + e] : (cc == 2 ? o[9][2 * h + e] : o[13][2 * h + e]));
          y.z = cc == 0 ? o[2][2 * h + e] : (cc == 1 ? o[6][2 * h + e] : (cc == 2 ? o[10][2 * h + e] : o[14][2 * h + e]));
          y.w = cc == 0 ? o[3][2 * h + e] : (cc == 1 ? o[7][2 * h + e] : (cc == 2 ? o[11][2 * h + e] : o[15][2 * h + e]));
          *reinterpret_cast<float4*>(dst + 16 * e + 4 * cc) = y;
        }
    }
    __syncthreads();
    bool odd = false;                                   // a row is not finite
    const int r_lo = sp.i0 * pl.group, r_hi = min(sp.i1 * pl.group, R);
    for (int r = r_lo + (tid >> 5); r < r_hi; r += kWarps) {        // a warp per row, 4 d's per lane
      float m = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 v = ml_sm[w][r];
        if (v.y != 0.f) m = fmaxf(m, v.x);
      }
      float L = 0.f;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 v = ml_sm[w][r];
        if (v.y == 0.f) continue;                       // the row sees no key of this warp
        const float a = exp2_approx(v.x - m);
        const float4 z = *reinterpret_cast<const float4*>(o_sm + ((size_t)w * kFewRows + r) * kOPitch + 4 * lane);
        L += a * v.y;
        y.x += a * z.x;
        y.y += a * z.y;
        y.z += a * z.z;
        y.w += a * z.w;
      }
      if constexpr (!k4) {
        odd = odd || !(fabsf(y.x) + fabsf(y.y) + fabsf(y.z) + fabsf(y.w) < INFINITY);
        if (again) {
          const int p = n_past + div24(r, pl.group), low = window_low(pl, p);
          for (int j = 0; j < tl.n * kPagesPerTile; ++j) {
            const int lp = tl.at(j / kPagesPerTile) * kPagesPerTile + j % kPagesPerTile, id = page_at(kv, lp);
            if (!page_ok(kv, id)) continue;
            const uint8_t* vp = vbase + (uint64_t)(uint32_t)id * stride + 8 * lane;
            for (int t = 16 * lp; t < 16 * lp + 16; ++t, vp += 256) {
              if (t > p || (t < low && t >= sinks)) continue;
              const uint2 w = ldg_now(reinterpret_cast<const uint2*>(vp));
              if ((w.x & 0x7F80u) == 0x7F80u) y.x += __uint_as_float(w.x << 16);
              if ((w.x & 0x7F800000u) == 0x7F800000u) y.y += __uint_as_float(w.x & 0xFFFF0000u);
              if ((w.y & 0x7F80u) == 0x7F80u) y.z += __uint_as_float(w.y << 16);
              if ((w.y & 0x7F800000u) == 0x7F800000u) y.w += __uint_as_float(w.y & 0xFFFF0000u);
            }
          }
        }
      }
      const size_t at = ((size_t)slot * pl.nkv + kvh) * R + r;
      reinterpret_cast<float4*>(part_o)[(((size_t)slot * pl.nkv + kvh) * 32 + lane) * R + r] = y;
      if (lane == 0) part_ml[at] = make_float2(m, L);
    }
    // the barrier also frees the shared memory for the next pass
    const bool found = __syncthreads_or(odd);
    again = found && !again;
    if (!again) ++pass;
    if (pass < passes) start(pass);
  }
}

template <bool k4>
static cudaError_t launch_few(const PattnPlan& pl, const KvView& kv, int layer, const float* q, float* part_o, float2* part_ml,
                              cudaStream_t st) {
  // the shared-memory limit is a per-device attribute
  constexpr int kMaxDevices = 64;
  static bool have[kMaxDevices] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool known = dev >= 0 && dev < kMaxDevices;
  if (!known || !have[dev]) {
    e = cudaFuncSetAttribute(pattn_few_kernel<k4>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)FewRing<k4>::kSmem);
    if (e != cudaSuccess) return e;
    if (known) have[dev] = true;
  }
  return launch_early(pattn_few_kernel<k4>, dim3(pl.slots, pl.nkv), dim3(32 * kFewWarps), FewRing<k4>::kSmem, st, q,
                      pl, kv, layer, part_o, part_ml);
}

cudaError_t launch_pattn_few(bool k4, const PattnPlan& pl, const KvView& kv, int layer, const float* q, float* part_o,
                             float2* part_ml, cudaStream_t st) {
  return k4 ? launch_few<true>(pl, kv, layer, q, part_o, part_ml, st) : launch_few<false>(pl, kv, layer, q, part_o, part_ml, st);
}

}  // namespace spec
