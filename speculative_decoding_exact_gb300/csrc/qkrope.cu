// qkrope.cu — QK-norm and rotary embedding of the q and k heads of n rows.
//
// One warp per (row, head): lane l holds elements 2l, 2l + 1 and 64 + 2l,
// 64 + 2l + 1, so that the pair (i, i + 64) that the rotation turns is in one
// lane.  y = x * g / sqrt(mean(x^2) + eps) with the mean of the 128 elements
// in fp32 (lane sums, then a butterfly), then
//   (y_i, y_{i+64}) -> (y_i cos - y_{i+64} sin, y_{i+64} cos + y_i sin).
// Bound by memory traffic: 8 bytes per element.
#include "common.cuh"
#include "internal.h"

namespace spec {

constexpr int kQkWarps = 8;

__global__ void __launch_bounds__(32 * kQkWarps)
qk_norm_rope_kernel(const float* x, long long ldx, int n, int nq, int nkv, const int32_t* __restrict__ pos,
                    QkTransform t, float* out, long long ldo, int32_t* status) {
  pdl_trigger();
  pdl_wait();
  const int heads = nq + nkv, lane = threadIdx.x & 31;
  const long long item = (long long)blockIdx.x * kQkWarps + (threadIdx.x >> 5);
  const int row = (int)(item / heads), head = (int)(item % heads);
  if (row >= n) return;
  const float* src = x + (size_t)row * ldx + head * 128 + 2 * lane;
  float2 a = *reinterpret_cast<const float2*>(src), b = *reinterpret_cast<const float2*>(src + 64);
  const float* g = head < nq ? t.gq : t.gk;
  if (g) {
    const float ss = warp_sum(a.x * a.x + a.y * a.y + b.x * b.x + b.y * b.y);
    const float r = 1.0f / sqrtf(ss / 128.0f + t.eps);
    const float2 g0 = *reinterpret_cast<const float2*>(g + 2 * lane);
    const float2 g1 = *reinterpret_cast<const float2*>(g + 64 + 2 * lane);
    a = make_float2(a.x * r * g0.x, a.y * r * g0.y);
    b = make_float2(b.x * r * g1.x, b.y * r * g1.y);
  }
  if (t.cs) {
    const int p = pos[row];
    if (p >= 0 && p < t.cs_len) {
      const float4 c = *reinterpret_cast<const float4*>(t.cs + (size_t)p * 64 + 2 * lane);   // cos, sin of 2l, 2l + 1
      const float2 u = a, w = b;
      a = make_float2(u.x * c.x - w.x * c.y, u.y * c.z - w.y * c.w);
      b = make_float2(w.x * c.x + u.x * c.y, w.y * c.z + u.y * c.w);
    } else {
      // no angle for this position: the row is zero, and the status says so
      a = b = make_float2(0.f, 0.f);
      if (lane == 0) atomicOr(status, SPEC_ST_CTX_FULL);
    }
  }
  float* dst = out + (size_t)row * ldo + head * 128 + 2 * lane;
  *reinterpret_cast<float2*>(dst) = a;
  *reinterpret_cast<float2*>(dst + 64) = b;
}

cudaError_t launch_qk_norm_rope(const float* x, int ldx, int n, int nq, int nkv, const int32_t* pos,
                                const QkTransform& t, float* out, int ldo, int32_t* status, cudaStream_t st) {
  const long long warps = (long long)n * (nq + nkv);
  qk_norm_rope_kernel<<<(unsigned)((warps + kQkWarps - 1) / kQkWarps), 32 * kQkWarps, 0, st>>>(
      x, ldx, n, nq, nkv, pos, t, out, ldo, status);
  return cudaGetLastError();
}

}  // namespace spec
