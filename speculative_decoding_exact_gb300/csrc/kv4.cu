// kv4.cu — writing and reading the rows of a 4-bit KV cache (page layout and
// arithmetic: kv4.cuh).
//
// Both kernels move one pass over their data: 4 bytes per value on the fp32
// side and 9/16 on the paged side, so they are bound by memory traffic.
#include "common.cuh"
#include "internal.h"
#include "kv4.cuh"

namespace spec {

constexpr int kKv4Threads = 256;

// the page of (lp, layer, which, head), nullptr when lp is not mapped
SPEC_DEV uint8_t* kv4_page(const KvView& kv, int lp, int layer, int which, int head) {
  if (lp < 0 || lp >= kv.max_seq_pages) return nullptr;
  const int page = kv.page_table[lp];
  if (page < 0 || page >= kv.num_pages) return nullptr;
  return reinterpret_cast<uint8_t*>(kv.pool) +
         ((((size_t)page * kv.n_layers + layer) * 2 + which) * kv.n_kv + head) * kKv4PageBytes;
}

// 16 lanes per (row, K or V, head), 8 values each; two lanes share a group of
// 16 and its scale.
__global__ void __launch_bounds__(kKv4Threads)
kv4_append_kernel(const float* __restrict__ k, const float* __restrict__ v, long long ld, int n, KvView kv, int layer,
                  int32_t* status) {
  pdl_trigger();
  pdl_wait();
  const int sub = threadIdx.x & 15;
  const long long item = ((long long)blockIdx.x * kKv4Threads + threadIdx.x) >> 4;
  const int per_row = 2 * kv.n_kv;
  const int row = (int)(item / per_row), rest = (int)(item % per_row);
  const bool in = row < n;
  const int which = rest / kv.n_kv, head = rest % kv.n_kv;
  float x[8] = {};
  if (in) {
    const float* src = (which ? v : k) + (size_t)row * ld + head * 128 + 8 * sub;
    const float4 a = reinterpret_cast<const float4*>(src)[0], b = reinterpret_cast<const float4*>(src)[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  float amax = 0.f;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    bad = bad || !(fabsf(x[i]) <= 3.40282347e38f);
    if (x[i] != x[i]) x[i] = 0.f;                    // a NaN is stored as 0
    amax = fmaxf(amax, fabsf(x[i]));
  }
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  if (!in) return;
  if (bad) atomicOr(status, SPEC_ST_NONFINITE);
  const int pos = *kv.seq_len - n + row;
  uint8_t* pg = pos >= 0 ? kv4_page(kv, pos >> 4, layer, which, head) : nullptr;
  if (!pg) {
    if (sub == 0) atomicOr(status, SPEC_ST_CTX_FULL);
    return;
  }
  const uint32_t sb = kv4_scale_byte(amax);
  const float s = kv4_scale(sb);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) w |= (sb ? kv4_code(x[i], s) : (__float_as_uint(x[i]) >> 28) & 8u) << (4 * i);
  const int t = pos & 15;
  *reinterpret_cast<uint32_t*>(pg + kv4_chunk(t, sub >> 2) + 4 * (sub & 3)) = w;
  if ((sub & 1) == 0) pg[kKv4Scales + 8 * t + (sub >> 1)] = (uint8_t)sb;
}

__global__ void __launch_bounds__(kKv4Threads)
kv4_read_kernel(KvView kv, int layer, int pos0, int n, float* __restrict__ k, float* __restrict__ v, long long ld) {
  pdl_trigger();
  pdl_wait();
  const int sub = threadIdx.x & 15;
  const long long item = ((long long)blockIdx.x * kKv4Threads + threadIdx.x) >> 4;
  const int per_row = 2 * kv.n_kv;
  const int row = (int)(item / per_row), rest = (int)(item % per_row);
  if (row >= n) return;
  const int which = rest / kv.n_kv, head = rest % kv.n_kv;
  const int pos = pos0 + row, t = pos & 15;
  const uint8_t* pg = pos < *kv.seq_len ? kv4_page(kv, pos >> 4, layer, which, head) : nullptr;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
  if (pg) {
    uint32_t c[4];
    e2m1_word(*reinterpret_cast<const uint32_t*>(pg + kv4_chunk(t, sub >> 2) + 4 * (sub & 3)), c);
    const float s = kv4_scale(pg[kKv4Scales + 8 * t + (sub >> 1)]);
    float y[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&c[i]));
      y[2 * i] = f.x * s;
      y[2 * i + 1] = f.y * s;
    }
    a = make_float4(y[0], y[1], y[2], y[3]);
    b = make_float4(y[4], y[5], y[6], y[7]);
  }
  float4* dst = reinterpret_cast<float4*>((which ? v : k) + (size_t)row * ld + head * 128 + 8 * sub);
  dst[0] = a;
  dst[1] = b;
}

static unsigned kv4_grid(const KvView& kv, int n) {
  return (unsigned)(((long long)n * 2 * kv.n_kv * 16 + kKv4Threads - 1) / kKv4Threads);
}

cudaError_t launch_kv4_append(const float* k, const float* v, int ld, int n, const KvView& kv, int layer,
                              int32_t* status, cudaStream_t st) {
  kv4_append_kernel<<<kv4_grid(kv, n), kKv4Threads, 0, st>>>(k, v, ld, n, kv, layer, status);
  return cudaGetLastError();
}

cudaError_t launch_kv4_read(const KvView& kv, int layer, int pos0, int n, float* k, float* v, int ld,
                            cudaStream_t st) {
  kv4_read_kernel<<<kv4_grid(kv, n), kKv4Threads, 0, st>>>(kv, layer, pos0, n, k, v, ld);
  return cudaGetLastError();
}

}  // namespace spec
