// pattn.cu — attention of up to 16 rows over a paged cache, bf16 or 4-bit, with
// an optional window and sinks.
//
// Row i sits at position p = seq_len - M + i and sees the keys t <= p with
// t > p - window or t < sinks (window 0: every t <= p).
// s_t = q.k_t / sqrt(128), o = sum_t exp(s_t - m) v_t / sum_t exp(s_t - m).
#include "common.cuh"
#include "internal.h"
#include "kv4.cuh"

namespace spec {

constexpr int kSimpleWarps = 8;

// elements 4l .. 4l + 3 of the key (which = 0) or value row at position t
template <bool k4>
SPEC_DEV bool row4(const KvView& kv, int layer, int which, int head, int t, int lane, float (&y)[4]) {
  const int lp = t >> 4;
  const int page = lp < kv.max_seq_pages ? kv.page_table[lp] : -1;
  if (page < 0 || page >= kv.num_pages) return false;
  const size_t block = (((size_t)page * kv.n_layers + layer) * 2 + which) * kv.n_kv + head;
  const int s = t & 15;
  if (k4) {
    const uint8_t* pg = reinterpret_cast<const uint8_t*>(kv.pool) + block * kKv4PageBytes;
    const uint32_t w = *reinterpret_cast<const uint16_t*>(pg + kv4_chunk(s, lane >> 3) + 2 * (lane & 7));
    uint32_t c[4];
    e2m1_word(w, c);
    const float sc = kv4_scale(pg[kKv4Scales + 8 * s + (lane >> 2)]);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&c[0]));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&c[1]));
    y[0] = a.x * sc; y[1] = a.y * sc; y[2] = b.x * sc; y[3] = b.y * sc;
  } else {
    const uint2 w = *reinterpret_cast<const uint2*>(kv.pool + block * 2048 + s * 128 + 4 * lane);
    y[0] = __uint_as_float(w.x << 16); y[1] = __uint_as_float(w.x & 0xFFFF0000u);
    y[2] = __uint_as_float(w.y << 16); y[3] = __uint_as_float(w.y & 0xFFFF0000u);
  }
  return true;
}

// grid (head, row): warp w takes the visible keys w, w + 8, ... with a running
// maximum and sum; the warps are joined in order
template <bool k4>
__global__ void __launch_bounds__(32 * kSimpleWarps)
pattn_simple_kernel(const float* __restrict__ q, int M, int nq, KvView kv, int layer, int window, int sinks,
                    float* __restrict__ out) {
  __shared__ float so[kSimpleWarps][128], sm[kSimpleWarps], sl[kSimpleWarps];
  const int h = blockIdx.x, i = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int p = *kv.seq_len - M + i, kvh = h / (nq / kv.n_kv);
  const int lo = window > 0 ? max(0, p - window + 1) : 0;
  const int first = window > 0 ? min(sinks, lo) : 0;         // sinks before the window
  const float4 qv = *reinterpret_cast<const float4*>(q + ((size_t)i * nq + h) * 128 + 4 * lane);
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int j = warp; j < first + (p + 1 - lo); j += kSimpleWarps) {
    const int t = j < first ? j : lo + j - first;
    float k[4], v[4];
    if (!row4<k4>(kv, layer, 0, kvh, t, lane, k)) continue;
    row4<k4>(kv, layer, 1, kvh, t, lane, v);
    const float s = warp_sum(qv.x * k[0] + qv.y * k[1] + qv.z * k[2] + qv.w * k[3]) / sqrtf(128.f);
    const float mn = fmaxf(m, s), a = expf(m - mn), w = expf(s - mn);
    m = mn;
    l = l * a + w;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = o[e] * a + w * v[e];
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) so[warp][4 * lane + e] = o[e];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  __syncthreads();
  if (threadIdx.x >= 128) return;
  float mm = -INFINITY, L = 0.f, O = 0.f;
  for (int w = 0; w < kSimpleWarps; ++w) mm = fmaxf(mm, sm[w]);
  for (int w = 0; w < kSimpleWarps; ++w) {
    const float a = sl[w] == 0.f ? 0.f : expf(sm[w] - mm);
    L += a * sl[w];
    O += a * so[w][threadIdx.x];
  }
  out[((size_t)i * nq + h) * 128 + threadIdx.x] = L == 0.f ? 0.f : O / L;   // nothing visible: zero
}

cudaError_t launch_paged_attention(bool k4, const KvView& kv, int layer, const float* q, int M, int nq, int window,
                                   int sinks, float* out, cudaStream_t st) {
  const dim3 grid(nq, M);
  if (k4)
    pattn_simple_kernel<true><<<grid, 32 * kSimpleWarps, 0, st>>>(q, M, nq, kv, layer, window, sinks, out);
  else
    pattn_simple_kernel<false><<<grid, 32 * kSimpleWarps, 0, st>>>(q, M, nq, kv, layer, window, sinks, out);
  return cudaGetLastError();
}

}  // namespace spec
