// kv4.cu — writing and reading the rows of a 4-bit KV cache (page layout and
// arithmetic: kv4.cuh).
//
// Both kernels make one pass over their data: 4 bytes per value on the fp32
// side and 9/16 on the paged side, so they are bound by memory traffic.  A CTA
// takes the 16 positions of one page and KV head, K and V, so that the pages are
// written and read whole.  32761 rows of 4 KV heads: 48 us to append (134 MB read)
// and read back (134 MB written), 6.4 TB/s; alone 27 and 28.  Appending with a CTA
// per item instead of a loop that loads ahead took 30; reading back in such a loop,
// or with 256 threads instead of 128, 31 and 29.
#include "common.cuh"
#include "internal.h"
#include "kv4.cuh"

namespace spec {

constexpr int kKv4Threads = 256, kAppendCtas = 4;     // CTAs per SM
constexpr int kReadThreads = 128;

// the id of a logical page, -1 when it is not mapped
SPEC_DEV int kv4_page_id(const KvView& kv, long long lp) {
  if (lp < 0 || lp >= kv.max_seq_pages) return -1;
  const int page = kv.page_table[lp];
  return page < kv.num_pages ? page : -1;
}
// the K page of (page id, layer, head); V's is n_kv pages behind it
SPEC_DEV uint8_t* kv4_page(const KvView& kv, int page, int layer, int head) {
  return reinterpret_cast<uint8_t*>(kv.pool) +
         (((size_t)page * kv.n_layers + layer) * 2 * kv.n_kv + head) * kKv4PageBytes;
}

// 16 lanes per position, 8 values of K and 8 of V each; two lanes share a group
// of 16 and its scale.
//
// The code of x under scale s is the e2m1 number nearest to x / s, ties to the
// even code.  x (1/s) in fp32 is off by less than 2^-22 of itself.  The
// conversion is monotone, so where x (1/s) (1 - 2^-20) and x (1/s) (1 + 2^-20)
// have the same code it is that of x / s; where they differ x / s is next to a
// tie, and the comparisons of kv4_code decide.
// A CTA works on every gridDim.x-th item, (tile, head), and loads the next one's
// rows before it quantises this one's.
__global__ void __launch_bounds__(kKv4Threads, kAppendCtas)
kv4_append_kernel(const float* k, const float* v, long long ld, int n, uint32_t items, KvView kv,
                  int layer, int32_t* status) {
  pdl_trigger();
  const int sub = threadIdx.x & 15, t = threadIdx.x >> 4;
  pdl_wait();
  const long long pos0 = (long long)*kv.seq_len - n;    // may lie below 0
  struct Item {
    float4 x[2][2];
    int page, head;
    bool in;
  };
  auto load = [&](uint32_t item) {
    Item r;
    const uint32_t tile = item / (uint32_t)kv.n_kv;
    r.head = item - tile * kv.n_kv;
    const long long lp = (pos0 >> 4) + tile, row = lp * 16 + t - pos0;
    r.in = row >= 0 && row < n;
    r.page = kv4_page_id(kv, lp);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      r.x[which][0] = r.x[which][1] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r.in) {
        const float4* src = reinterpret_cast<const float4*>((which ? v : k) + (size_t)row * ld + r.head * 128 + 8 * sub);
        r.x[which][0] = __ldcs(src);
        r.x[which][1] = __ldcs(src + 1);
      }
    }
    return r;
  };
  uint32_t item = blockIdx.x;
  Item next = load(item);
  for (; item < items; item += gridDim.x) {
    const Item cur = next;
    if (item + gridDim.x < items) next = load(item + gridDim.x);
    if (cur.in && cur.page < 0 && sub == 0) atomicOr(status, SPEC_ST_CTX_FULL);
    uint8_t* pg = kv4_page(kv, cur.page, layer, cur.head);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const float4 a = cur.x[which][0], b = cur.x[which][1];
      float y[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      float amax = 0.f;                                 // NaN if there is one
#pragma unroll
      for (int i = 0; i < 8; ++i) asm("max.NaN.f32 %0, %0, %1;\n" : "+f"(amax) : "f"(fabsf(y[i])));
      const bool bad = !(amax <= 3.40282347e38f);
      if (bad) {
        atomicOr(status, SPEC_ST_NONFINITE);
        amax = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (y[i] != y[i]) y[i] = 0.f;                 // a NaN is stored as 0
          amax = fmaxf(amax, fabsf(y[i]));
        }
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      const uint32_t sb = kv4_scale_byte(amax);
      const float s = kv4_scale(sb), inv = 1.0f / s;
      const float up = inv * (1.f + 0x1p-20f), down = inv * (1.f - 0x1p-20f);
      float y0[8], y1[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        y0[i] = y[i] * down;
        y1[i] = y[i] * up;
      }
      uint32_t w = e2m1_word(y0);
      if (w != e2m1_word(y1) || sb == 0) {
        w = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) w |= (sb ? kv4_code(y[i], s) : (__float_as_uint(y[i]) >> 28) & 8u) << (4 * i);
      }
      if (cur.in && cur.page >= 0) {
        uint8_t* dst = pg + (which ? (size_t)kv.n_kv * kKv4PageBytes : 0);
        *reinterpret_cast<uint32_t*>(dst + kv4_chunk(t, sub >> 2) + 4 * (sub & 3)) = w;
        if ((sub & 1) == 0) dst[kKv4Scales + 8 * t + (sub >> 1)] = (uint8_t)sb;
      }
    }
  }
}

// A warp per position, K then V, 4 values per lane, so that a store is a whole
// row of 512 bytes; all of a lane's loads come before its first store.
__global__ void __launch_bounds__(kReadThreads)
kv4_read_kernel(KvView kv, int layer, int pos0, int n, float* __restrict__ k, float* __restrict__ v, long long ld) {
  pdl_trigger();
  const uint32_t tile = blockIdx.x / (uint32_t)kv.n_kv, head = blockIdx.x - tile * kv.n_kv;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kWarps = kReadThreads / 32, kRows = 16 / kWarps;
  const long long lp = (pos0 >> 4) + tile;
  pdl_wait();
  const int seq_len = *kv.seq_len;
  const int page = kv4_page_id(kv, lp);
  const uint8_t* pg = kv4_page(kv, page, layer, head);
  uint32_t code[kRows][2], sb[kRows][2];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int t = warp + kWarps * r;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      code[r][which] = sb[r][which] = 0;
      if (page >= 0 && lp * 16 + t < seq_len) {
        const uint8_t* src = pg + (which ? (size_t)kv.n_kv * kKv4PageBytes : 0);
        code[r][which] = *reinterpret_cast<const uint16_t*>(src + kv4_chunk(t, lane >> 3) + 2 * (lane & 7));
        sb[r][which] = src[kKv4Scales + 8 * t + (lane >> 2)];
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const long long row = lp * 16 + warp + kWarps * r - pos0;
    if (row < 0 || row >= n) continue;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      uint32_t f0, f1;
      e2m1_pairs(code[r][which], f0, f1);
      const uint32_t s2 = min(sb[r][which], (uint32_t)kKv4TopScale) * 0x00800080u;      // the scale in both halves
      f0 = hmul2_u32(f0, s2);
      f1 = hmul2_u32(f1, s2);
      const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&f0));
      const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&f1));
      __stcs(reinterpret_cast<float4*>((which ? v : k) + (size_t)row * ld + head * 128 + 4 * lane),
             make_float4(a.x, a.y, b.x, b.y));
    }
  }
}

// (tile, head) items of the pages that n rows touch, at most; the kernels count
// them, and the steps through them, in 32 bits
static bool kv4_items(const KvView& kv, long long tiles, uint32_t& items) {
  items = (uint32_t)(tiles * kv.n_kv);
  return tiles * kv.n_kv <= 0x3FFFFFFFll;
}
cudaError_t launch_kv4_append(const float* k, const float* v, int ld, int n, const KvView& kv, int layer, int num_sms,
                              int32_t* status, cudaStream_t st) {
  uint32_t items;
  if (!kv4_items(kv, ((long long)n + 15) / 16 + 1, items)) return cudaErrorInvalidConfiguration;
  const uint32_t most = (uint32_t)(kAppendCtas * num_sms);
  return launch_early(kv4_append_kernel, dim3(items < most ? items : most), dim3(kKv4Threads), 0, st, k, v, ld, n, items, kv,
                      layer, status);
}

cudaError_t launch_kv4_read(const KvView& kv, int layer, int pos0, int n, float* k, float* v, int ld, cudaStream_t st) {
  uint32_t items;
  if (!kv4_items(kv, ((long long)pos0 + n + 15) / 16 - pos0 / 16, items)) return cudaErrorInvalidConfiguration;
  return launch_early(kv4_read_kernel, dim3(items), dim3(kReadThreads), 0, st, kv, layer, pos0, n, k, v, ld);
}

}  // namespace spec
