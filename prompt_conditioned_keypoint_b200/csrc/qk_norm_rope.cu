// gkd_qk_norm_rope: RMS norm of every query and key head and its rotation by
// position (one to three axes), one pass over q and k.
//
// y = x w / sqrt(mean x^2 + eps); pair p of a head turns by pos[t, axis[p]] freq[p].
// Bound by HBM: q and k are read once and written once; everything else is small.
// A CTA takes a few consecutive rows with all of their heads, so each (row, pair)
// angle is formed once and serves every head: turns = pos * freq / (2 pi) in fp64
// (the product of two fp32 numbers is exact there), minus its nearest whole
// number, then sine and cosine in fp32. A thread holds both halves of V pairs, so
// the rotation needs no exchange between threads; the norm's sum goes over the G
// lanes of a head by shuffles. A thread's loads (IT items of two vectors) are all
// issued before the angles are formed and are in flight meanwhile.
#include "blocks_common.cuh"
#include "gkd_internal.h"

namespace gkd {
namespace rope {

constexpr int kThreads = 256, kItems = 4, kMaxTok = 16, kMaxPairs = 128;

template <typename T, int V>
__device__ __forceinline__ void loadv(const T* p, float (&v)[V]) {
  if constexpr (sizeof(T) == 2 && V == 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    v[0] = bf16_lo(u.x); v[1] = bf16_hi(u.x); v[2] = bf16_lo(u.y); v[3] = bf16_hi(u.y);
    v[4] = bf16_lo(u.z); v[5] = bf16_hi(u.z); v[6] = bf16_lo(u.w); v[7] = bf16_hi(u.w);
  } else {
    const float4 u = load4(p);
    v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
  }
}
template <typename T, int V>
__device__ __forceinline__ void storev(T* p, const float (&v)[V]) {
  if constexpr (sizeof(T) == 2 && V == 8) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                              pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  } else {
    store4(p, make_float4(v[0], v[1], v[2], v[3]));
  }
}

// Where item `item` of the CTA (row, head, lane of the head) lies.
struct Place {
  int tok, side, a, b, u;   // row of the CTA, 0 = q / 1 = k, element offsets of the two vectors, unit
  long long in, out;        // element offset of the head in the input and in the output
  bool live;
};

template <typename T, int V, bool PAIRS>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const __grid_constant__ RopeArgs g) {
  __shared__ float2 cs[kMaxTok * kMaxPairs];
  __shared__ __align__(16) float wt[2][256];
  const int heads = g.side[0].heads + g.side[1].heads;
  const int units = g.D / (2 * V), rot_units = g.pairs / V;
  const long long rows = static_cast<long long>(g.B) * g.T;
  const long long row0 = static_cast<long long>(blockIdx.x) * g.tok;
  const int ntok = static_cast<int>(min(static_cast<long long>(g.tok), rows - row0));
  const int per_tok = heads << g.log_lanes;
  const int total = ntok * per_tok;
  const bool norm = g.side[0].weight != nullptr;

  auto place = [&](int item) {
    Place p;
    p.live = item < total;
    p.tok = item / per_tok;
    const int r = item - p.tok * per_tok;
    int h = r >> g.log_lanes;
    p.u = r & ((1 << g.log_lanes) - 1);
    p.live = p.live && p.u < units;
    p.side = h >= g.side[0].heads ? 1 : 0;
    if (p.side) h -= g.side[0].heads;
    const long long row = row0 + p.tok, b = row / g.T, t = row - b * g.T;
    const RopeSide& s = g.side[p.side];
    p.in = b * s.in_bs + t * s.in_rs + h * s.in_hs;
    p.out = b * s.out_bs + t * s.out_rs + h * s.out_hs;
    if (p.u < rot_units) {
      p.a = PAIRS ? 2 * p.u * V : p.u * V;
      p.b = PAIRS ? p.a + V : g.pairs + p.a;
    } else {
      p.a = 2 * p.u * V;                                     // behind the rotated elements: two vectors in a row
      p.b = p.a + V;
    }
    return p;
  };

  float va[kItems][V], vb[kItems][V];
  auto load = [&](int base) {
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const Place p = place(base + i * kThreads + threadIdx.x);
#pragma unroll
      for (int e = 0; e < V; ++e) va[i][e] = vb[i][e] = 0.f;
      if (p.live) {
        const T* x = static_cast<const T*>(g.side[p.side].in) + p.in;
        loadv<T, V>(x + p.a, va[i]);
        loadv<T, V>(x + p.b, vb[i]);
      }
    }
  };
  load(0);
  for (int e = threadIdx.x; e < ntok * g.pairs; e += kThreads) {
    const int tok = e / g.pairs, pr = e - tok * g.pairs;
    const long long row = row0 + tok, b = row / g.T, t = row - b * g.T;
    int axis = g.pair_axis[pr];
    if (axis >= g.axes) axis = 0;
    const double turns = static_cast<double>(g.pos[b * g.pos_bs + t * g.axes + axis]) *
                         static_cast<double>(g.pair_freq[pr]) * 0.15915494309189535;
    float s, c;
    sincospif(2.f * static_cast<float>(turns - rint(turns)), &s, &c);
    cs[e] = make_float2(c, s);
  }
  if (norm)
    for (int e = threadIdx.x; e < 2 * g.D; e += kThreads) {
      const int s = e >= g.D;
      if (g.side[s].weight) wt[s][e - s * g.D] = g.side[s].weight[e - s * g.D];
    }
  __syncthreads();
  for (int base = 0; base < total; base += kItems * kThreads) {
    if (base) load(base);
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const Place p = place(base + i * kThreads + threadIdx.x);
      if (norm) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) ss = fmaf(va[i][e], va[i][e], fmaf(vb[i][e], vb[i][e], ss));
        for (int o = (1 << g.log_lanes) >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float r = 1.f / sqrtf(ss / static_cast<float>(g.D) + g.eps);
        if (p.live) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            va[i][e] *= r * wt[p.side][p.a + e];
            vb[i][e] *= r * wt[p.side][p.b + e];
          }
        }
      }
      if (!p.live) continue;
      if (p.u < rot_units) {
        const float2* c = cs + p.tok * g.pairs + p.u * V;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          if constexpr (PAIRS) {                             // pair e of the unit: elements 2 e, 2 e + 1 of the 2 V
            float& x = 2 * e < V ? va[i][2 * e % V] : vb[i][2 * e % V];
            float& y = 2 * e < V ? va[i][(2 * e + 1) % V] : vb[i][(2 * e + 1) % V];
            const float x0 = x;
            x = x0 * c[e].x - y * c[e].y;
            y = y * c[e].x + x0 * c[e].y;
          } else {
            const float x0 = va[i][e];
            va[i][e] = x0 * c[e].x - vb[i][e] * c[e].y;
            vb[i][e] = vb[i][e] * c[e].x + x0 * c[e].y;
          }
        }
      }
      T* o = static_cast<T*>(g.side[p.side].out) + p.out;
      storev<T, V>(o + p.a, va[i]);
      storev<T, V>(o + p.b, vb[i]);
    }
  }
}

template <typename T, int V>
cudaError_t go(RopeArgs& g, int num_sms, cudaStream_t stream) {
  const int heads = g.side[0].heads + g.side[1].heads, units = g.D / (2 * V);
  g.log_lanes = 0;
  while ((1 << g.log_lanes) < units) ++g.log_lanes;
  const long long rows = static_cast<long long>(g.B) * g.T;
  // rows per CTA: as many as fill a thread's items, fewer while that leaves SMs without a CTA
  long long tok = (kItems * kThreads) / (heads << g.log_lanes);
  const long long spread = rows / (2 * num_sms);
  if (tok > spread) tok = spread;
  if (tok > kMaxTok) tok = kMaxTok;
  if (tok < 1) tok = 1;
  g.tok = static_cast<int>(tok);
  const long long grid = (rows + tok - 1) / tok;
  if (g.interleaved)
    qk_norm_rope_kernel<T, V, true><<<static_cast<unsigned>(grid), kThreads, 0, stream>>>(g);
  else
    qk_norm_rope_kernel<T, V, false><<<static_cast<unsigned>(grid), kThreads, 0, stream>>>(g);
  return cudaGetLastError();
}

}  // namespace rope

cudaError_t launch_qk_norm_rope(RopeArgs& g, bool bf16, int num_sms, cudaStream_t stream) {
  if (!bf16) return rope::go<float, 4>(g, num_sms, stream);
  // 16-byte vectors of bf16 where both runs of elements divide into them, 8-byte ones else
  if (g.pairs % 8 == 0 && (g.D - 2 * g.pairs) % 16 == 0) return rope::go<__nv_bfloat16, 8>(g, num_sms, stream);
  return rope::go<__nv_bfloat16, 4>(g, num_sms, stream);
}

}  // namespace gkd
