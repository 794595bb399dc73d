// qkrope.cu — QK-norm and rotary embedding of the q and k heads of n rows.
//
// y = x * g / sqrt(mean(x^2) + eps) with the mean of the head's 128 elements in
// fp32, then
//   (y_i, y_{i+64}) -> (y_i cos - y_{i+64} sin, y_{i+64} cos + y_i sin).
//
// A warp takes up to 8 q heads or 8 k heads of one row, two at a time: 16 lanes
// of 4 + 4 elements each, l's being 4l .. and 64 + 4l .., so that the pairs that
// the rotation turns are in one lane, the mean is a butterfly of four steps, and
// the gains and angles are read once for all heads.
//
// Bound by memory traffic, 8 bytes per element.  All of a warp's loads are in
// flight at once, 4 KB: 8191 rows of 56 heads take 72 us, 6.6 TB/s (a warp per
// head, 512 bytes in flight: 108); one row 4.3 us, a launch.
#include "common.cuh"
#include "internal.h"

namespace spec {

constexpr int kQkHeads = 8;                // heads of a warp
constexpr int kQkWarps = 8;                // warps of a CTA at most

__global__ void __launch_bounds__(32 * kQkWarps)
qk_norm_rope_kernel(const float* x, long long ldx, int nq, int nkv, const int32_t* pos, QkTransform t,
                    float* out, long long ldo, int32_t* status) {
  pdl_trigger();
  const int lane = threadIdx.x & 31, half = lane >> 4, l = lane & 15, row = blockIdx.x;
  const int q_groups = (nq + kQkHeads - 1) / kQkHeads;
  const int group = blockIdx.y * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const bool is_q = group < q_groups;
  const int first = is_q ? group * kQkHeads : nq + (group - q_groups) * kQkHeads;
  const int heads = min(kQkHeads, (is_q ? nq : nq + nkv) - first);
  pdl_wait();
  if (heads <= 0) return;
  const float* src = x + (size_t)row * ldx + (first + half) * 128 + 4 * l;
  float* dst = out + (size_t)row * ldo + (first + half) * 128 + 4 * l;
  const int p = t.cs ? pos[row] : 0;
  float4 a[kQkHeads / 2], b[kQkHeads / 2];
#pragma unroll
  for (int h = 0; h < kQkHeads / 2; ++h) {
    a[h] = b[h] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (2 * h + half < heads) {
      a[h] = *reinterpret_cast<const float4*>(src + 256 * h);
      b[h] = *reinterpret_cast<const float4*>(src + 256 * h + 64);
    }
  }
  const float* g = is_q ? t.gq : t.gk;
  float4 ga = make_float4(1.f, 1.f, 1.f, 1.f), gb = ga;
  if (g) {
    ga = *reinterpret_cast<const float4*>(g + 4 * l);
    gb = *reinterpret_cast<const float4*>(g + 64 + 4 * l);
  }
  // cos and sin of elements 4l .. 4l + 3; without an angle for this position
  // the row is zero, and the status says so
  float4 c0 = make_float4(1.f, 0.f, 1.f, 0.f), c1 = c0;
  const bool angle = !t.cs || (p >= 0 && p < t.cs_len);
  if (t.cs && angle) {
    c0 = *reinterpret_cast<const float4*>(t.cs + (size_t)p * 64 + 4 * l);
    c1 = *reinterpret_cast<const float4*>(t.cs + (size_t)p * 64 + 4 * l + 2);
  } else if (!angle && threadIdx.x == 0) {
    atomicOr(status, SPEC_ST_CTX_FULL);
  }
#pragma unroll
  for (int h = 0; h < kQkHeads / 2; ++h) {
    if (2 * h >= heads) break;
    float4 u = a[h], w = b[h];
    if (g) {
      float ss = (u.x * u.x + u.y * u.y) + (u.z * u.z + u.w * u.w) + ((w.x * w.x + w.y * w.y) + (w.z * w.z + w.w * w.w));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float r = 1.0f / sqrtf(ss / 128.0f + t.eps);
      u = make_float4(u.x * r * ga.x, u.y * r * ga.y, u.z * r * ga.z, u.w * r * ga.w);
      w = make_float4(w.x * r * gb.x, w.y * r * gb.y, w.z * r * gb.z, w.w * r * gb.w);
    }
    float4 y = u, z = w;
    if (t.cs) {
      y = make_float4(u.x * c0.x - w.x * c0.y, u.y * c0.z - w.y * c0.w, u.z * c1.x - w.z * c1.y, u.w * c1.z - w.w * c1.w);
      z = make_float4(w.x * c0.x + u.x * c0.y, w.y * c0.z + u.y * c0.w, w.z * c1.x + u.z * c1.y, w.w * c1.z + u.w * c1.w);
    }
    if (!angle) y = z = make_float4(0.f, 0.f, 0.f, 0.f);
    if (2 * h + half < heads) {
      *reinterpret_cast<float4*>(dst + 256 * h) = y;
      *reinterpret_cast<float4*>(dst + 256 * h + 64) = z;
    }
  }
}

cudaError_t launch_qk_norm_rope(const float* x, int ldx, int n, int nq, int nkv, const int32_t* pos,
                                const QkTransform& t, float* out, int ldo, int32_t* status, cudaStream_t st) {
  const int groups = (nq + kQkHeads - 1) / kQkHeads + (nkv + kQkHeads - 1) / kQkHeads;
  const int warps = groups < kQkWarps ? groups : kQkWarps;
  return launch_early(qk_norm_rope_kernel, dim3(n, (groups + warps - 1) / warps), dim3(32 * warps), 0, st, x, ldx, nq, nkv,
                      pos, t, out, ldo, status);
}

}  // namespace spec
