// gkd_linear on the fp32 units, fp32 operands: out = residual + scale * act(x weight^T + bias).
#include "blocks_common.cuh"
#include "gkd_internal.h"

namespace gkd {
namespace lin {

constexpr int kTile = 64, kStep = 16;

// One 64 x 64 tile of the output per CTA, a 4 x 4 patch per thread; the channels
// go through shared memory 16 at a time.
__global__ void __launch_bounds__(256) linear_kernel(const __grid_constant__ LinearArgs a) {
  __shared__ float xs[kStep][kTile + 4], ws[kStep][kTile + 4];
  const int t0 = blockIdx.x * kTile, n0 = blockIdx.y * kTile;
  const int tid = threadIdx.x, tr = tid >> 4, tc = tid & 15;
  const float* x = static_cast<const float*>(a.x);
  const float* w = static_cast<const float*>(a.weight);
  float acc[4][4] = {};
  const int lr = tid >> 2, lc = (tid & 3) * 4;
  for (int c0 = 0; c0 < a.Cin; c0 += kStep) {
    float4 xv = make_float4(0.f, 0.f, 0.f, 0.f), wv = xv;
    if (c0 + lc < a.Cin) {
      if (t0 + lr < a.T) xv = load4(x + static_cast<long long>(t0 + lr) * a.x_stride + c0 + lc);
      if (n0 + lr < a.Cout) wv = load4(w + static_cast<long long>(n0 + lr) * a.Cin + c0 + lc);
    }
    __syncthreads();
    xs[lc][lr] = xv.x; xs[lc + 1][lr] = xv.y; xs[lc + 2][lr] = xv.z; xs[lc + 3][lr] = xv.w;
    ws[lc][lr] = wv.x; ws[lc + 1][lr] = wv.y; ws[lc + 2][lr] = wv.z; ws[lc + 3][lr] = wv.w;
    __syncthreads();
#pragma unroll
    for (int c = 0; c < kStep; ++c) {
      const float4 p = *reinterpret_cast<const float4*>(&xs[c][tr * 4]);
      const float4 q = *reinterpret_cast<const float4*>(&ws[c][tc * 4]);
      const float pv[4] = {p.x, p.y, p.z, p.w}, qv[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(pv[i], qv[j], acc[i][j]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = t0 + tr * 4 + i, n = n0 + tc * 4;
    if (t >= a.T || n >= a.Cout) continue;                         // Cout is a multiple of 8
    float4 res = make_float4(0.f, 0.f, 0.f, 0.f);
    if (a.residual)
      res = load4(static_cast<const float*>(a.residual) + static_cast<long long>(t) * a.residual_stride + n);
    const float rv[4] = {res.x, res.y, res.z, res.w};
    float y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      y[j] = acc[i][j] + (a.bias ? a.bias[n + j] : 0.f);
    }
    activate(y, a.act);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (a.scale) y[j] *= a.scale[n + j];
      y[j] += rv[j];
    }
    store4(static_cast<float*>(a.out) + static_cast<long long>(t) * a.out_stride + n, make_float4(y[0], y[1], y[2], y[3]));
  }
}

}  // namespace lin

cudaError_t launch_linear(LinearArgs& a, int num_sms, cudaStream_t stream, const char** why) {
  if (a.in_bf16) return launch_linear_tc(a, num_sms, stream, why);
  const dim3 grid((a.T + lin::kTile - 1) / lin::kTile, (a.Cout + lin::kTile - 1) / lin::kTile);
  lin::linear_kernel<<<grid, 256, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace gkd
