// pattn_plan.cuh — how attention over a paged cache is cut into chunks of keys,
// shared by its two kernels (pattn.cu, pattn_few.cu).
#pragma once
#include "common.cuh"
#include "internal.h"

namespace spec {

constexpr int kKeys = 128;                          // keys of a tile
constexpr int kPagesPerTile = kKeys / 16;
constexpr float kScoreScale = (float)(1.4426950408889634 / 11.313708498984761);   // log2(e) / sqrt(128)

struct PattnPlan {
  int M, nq, nkv, group, window, sinks;
  int C;                     // chunks of a KV head at most
  unsigned long long c_inv;  // ceil(2^40 / C): t / C = t * c_inv >> 40 for t < 2^24
  int slots;                 // chunk slots launched (<= C)
  int Lw;                    // tiles per chunk at most (what the window needs)
  int tile_rows;             // rows per row tile
};

// tiles per chunk of a row at position p
SPEC_DEV int chunk_len(const PattnPlan& pl, int p) {
  const int l = p > 0 ? (int)(((unsigned long long)(p >> 7) * pl.c_inv) >> 40) + 1 : 1;
  return l < pl.Lw ? l : pl.Lw;
}
// the first position that a row at p sees through its window
SPEC_DEV int window_low(const PattnPlan& pl, int p) { return pl.window > 0 && p >= pl.window ? p - pl.window + 1 : 0; }

// x / d for 0 <= x < 2^24: the quotient in fp32 is off by less than one
SPEC_DEV int div24(int x, int d) {
  int q = (int)__fdividef((float)x, (float)d);
  const int r = x - q * d;
  return r < 0 ? q - 1 : (r >= d ? q + 1 : q);
}

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
    const int sk = pl.window > 0 ? min(pl.sinks, s.last + 1) : 0;
    s.sink_tiles = (int)(((unsigned)sk + kKeys - 1) / kKeys);
    s.cbase = div24(s.lo >> 7, s.L);
    s.ns = min(div24(s.sink_tiles + s.L - 1, s.L), s.cbase);
    s.nslots = s.ns + div24(s.last >> 7, s.L) - s.cbase + 1;
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

// x0 and x1 less the halves of a binary16 pair
SPEC_DEV void minus_f16x2(float& x0, float& x1, uint32_t h) {
  asm("{\n .reg .f16 a, b, m;\n mov.b32 {a, b}, %2;\n mov.b16 m, 0xBC00U;\n"      // m = -1
      " fma.rn.f32.f16 %0, a, m, %0;\n fma.rn.f32.f16 %1, b, m, %1;\n}\n"
      : "+f"(x0), "+f"(x1)
      : "r"(h));
}
// the upper 16 bits of two values, x0's in the low half; x becomes what is left
// (by truncation: rounding would turn the largest numbers into infinities)
SPEC_DEV uint32_t take_bf16(float& x0, float& x1) {
  const uint32_t a = __float_as_uint(x0), b = __float_as_uint(x1);
  x0 -= __uint_as_float(a & 0xFFFF0000u);
  x1 -= __uint_as_float(b & 0xFFFF0000u);
  return __byte_perm(a, b, 0x7632);
}
SPEC_DEV uint32_t low_bits(int n) { return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u); }

// Loads issued where they stand (a plain load may be moved down to its use, behind a
// wait, and one that the compiler takes for invariant up, before the wait for the
// kernel's predecessors).  Not the non-coherent kind: a kernel here may start before
// the writers of its data have ended.
SPEC_DEV uint4 ldg_now(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.cg.v4.u32 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
SPEC_DEV uint2 ldg_now(const uint2* p) {
  uint2 v;
  asm volatile("ld.global.cg.v2.u32 {%0,%1}, [%2];\n" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
SPEC_DEV int ldg_now(const int32_t* p) {
  int v;
  asm volatile("ld.global.cg.u32 %0, [%1];\n" : "=r"(v) : "l"(p));
  return v;
}
SPEC_DEV float4 ldg_now(const float4* p) {
  const uint4 v = ldg_now(reinterpret_cast<const uint4*>(p));
  return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
}
SPEC_DEV float2 ldg_now(const float2* p) {
  const uint2 v = ldg_now(reinterpret_cast<const uint2*>(p));
  return make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
}
// 16 bytes global -> shared, completion by group
SPEC_DEV void copy16(uint8_t* dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
SPEC_DEV void copy_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int kPending>
SPEC_DEV void copy_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(kPending) : "memory");
}

// the page id of a logical page, -1 past the table; to be checked where it is
// used (a check here would wait for the load).  Through L1, where neighbouring ids
// are found: from L2 alone one token behind 128k keys takes 42 instead of 41 us.
SPEC_DEV int page_at(const KvView& kv, int lp) {
  int v = -1;
  if (lp < kv.max_seq_pages) asm volatile("ld.global.u32 %0, [%1];\n" : "=r"(v) : "l"(kv.page_table + lp));
  return v;
}
SPEC_DEV bool page_ok(const KvView& kv, int page) { return (uint32_t)page < (uint32_t)kv.num_pages; }

constexpr uint64_t kPattnWaitNs = 2000000000ull;
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

// attention for a call of at most kFewRows query rows per KV head
constexpr int kFewRows = 16;
cudaError_t launch_pattn_few(bool k4, const PattnPlan& pl, const KvView& kv, int layer, const float* q, float* part_o,
                             float2* part_ml, cudaStream_t st);

// attention over a bf16 cache for more rows
cudaError_t launch_pattn_bf16(const PattnPlan& pl, const KvView& kv, int layer, const float* q, int row_tiles, float* part_o,
                              float2* part_ml, int32_t* status, cudaStream_t st);

}  // namespace spec
