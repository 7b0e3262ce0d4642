// gkd_qk_norm_rope: RMS norm of every query and key head and its rotation by
// position (one to three axes), one pass over q and k.
//
// y = x w / sqrt(mean x^2 + eps); pair p of a head turns by pos[t, axis[p]] freq[p].
// Bound by HBM: q and k are read once and written once; everything else is small.
// A CTA takes a few consecutive rows with all of their heads, so each (row, pair)
// angle is formed once and serves every head: turns = pos * freq / (2 pi) in fp64
// (the product of two fp32 numbers is exact there), minus its nearest whole
// number, then sine and cosine in fp32. A thread holds both halves of V pairs, so
// the rotation needs no exchange between threads; a head has D / (2 V) lanes, next to
// one another in a warp, and the norm's sum goes over them by shuffles. Which
// elements a thread takes is the same for all of its heads. Its loads (kItems heads
// of two vectors each) are all issued before the angles are formed and are in flight
// meanwhile.
//
// Measured (B200, in a graph): 64 x 581 rows of 2 x 20 heads of 64 63 us = 6.0 TB/s (92% of
// the copy rate), 80 us with norms (73% of the issue slots taken); 2 x 4608 rows of 20 fp32 heads of 80 with norms 29 us
// = 4.1 TB/s. CTAs of 256 threads took 68, 87 and 32 us; a warp per row with its angles
// and weights in registers 73, 104 and 35.
#include "blocks_common.cuh"
#include "gkd_internal.h"

namespace gkd {
namespace rope {

constexpr int kThreads = 128, kItems = 4, kMaxTok = 16, kMaxPairs = 128;

// V elements as they lie in memory, and as fp32.
template <typename T, int V>
struct Vec;
template <>
struct Vec<float, 4> {
  using Raw = float4;
  static __device__ __forceinline__ void open(const Raw& r, float (&v)[4]) {
    v[0] = r.x; v[1] = r.y; v[2] = r.z; v[3] = r.w;
  }
  static __device__ __forceinline__ Raw close(const float (&v)[4]) { return make_float4(v[0], v[1], v[2], v[3]); }
};
template <>
struct Vec<__nv_bfloat16, 4> {
  using Raw = uint2;
  static __device__ __forceinline__ void open(const Raw& r, float (&v)[4]) {
    v[0] = bf16_lo(r.x); v[1] = bf16_hi(r.x); v[2] = bf16_lo(r.y); v[3] = bf16_hi(r.y);
  }
  static __device__ __forceinline__ Raw close(const float (&v)[4]) {
    return make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  }
};
template <>
struct Vec<__nv_bfloat16, 8> {
  using Raw = uint4;
  static __device__ __forceinline__ void open(const Raw& r, float (&v)[8]) {
    v[0] = bf16_lo(r.x); v[1] = bf16_hi(r.x); v[2] = bf16_lo(r.y); v[3] = bf16_hi(r.y);
    v[4] = bf16_lo(r.z); v[5] = bf16_hi(r.z); v[6] = bf16_lo(r.w); v[7] = bf16_hi(r.w);
  }
  static __device__ __forceinline__ Raw close(const float (&v)[8]) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
};

template <typename T, int V, bool PAIRS, bool NORM>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const __grid_constant__ RopeArgs g) {
  using X = Vec<T, V>;
  using Raw = typename X::Raw;
  // Both so that the lanes of a head read consecutive 16-byte words: cosine and sine of pairs
  // (V u + 2 c, V u + 2 c + 1) of row tok at (tok V / 2 + c) rot_units + u; the weights of elements
  // 4 c ... of lane u's first (second) vector at c (V / 4 + c) of q (k).
  __shared__ float4 cs[kMaxTok * kMaxPairs / 2];
  __shared__ float4 wt[2][V / 2][32];
  const int lane = threadIdx.x & 31;
  const int units = g.D / (2 * V), rot_units = g.pairs / V;
  const int per_warp = 32 / units, slots = per_warp * (kThreads / 32);   // heads that the CTA takes at a time
  const int u = lane % units, slot = (threadIdx.x >> 5) * per_warp + lane / units;
  const bool idle = lane >= per_warp * units;
  const bool turn = u < rot_units;
  // element offsets of the thread's two vectors in a head; behind the rotated elements two in a row
  auto first_of = [&](int lu) { return lu < rot_units && !PAIRS ? lu * V : 2 * lu * V; };
  auto second_of = [&](int lu) { return lu < rot_units && !PAIRS ? g.pairs + lu * V : 2 * lu * V + V; };
  const int ea = first_of(u), eb = second_of(u);
  const int b = blockIdx.y;
  const long long t0 = static_cast<long long>(blockIdx.x) * g.tok;
  const int ntok = static_cast<int>(min(static_cast<long long>(g.tok), g.T - t0));
  const int hq = g.side[0].heads, heads = hq + g.side[1].heads;
  const int total = ntok * heads;
  // the n-th head of the CTA's rows: its row, whether it is of q (0) or k (1), its number there
  auto head = [&](int n, int& tok, int& s, int& h) {
    tok = heads == 1 ? n : static_cast<int>(__umulhi(n, g.heads_magic));
    h = n - tok * heads;
    s = h >= hq;
    if (s) h -= hq;
  };

  Raw ra[kItems], rb[kItems];
  auto load = [&](int base) {
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int n = base + i * slots + slot;
      if (idle || n >= total) {
        ra[i] = rb[i] = Raw{};
        continue;
      }
      int tok, s, h;
      head(n, tok, s, h);
      const RopeSide& side = g.side[s];
      const T* x = static_cast<const T*>(side.in) + b * side.in_bs + (t0 + tok) * side.in_rs + h * side.in_hs;
      ra[i] = *reinterpret_cast<const Raw*>(x + ea);
      rb[i] = *reinterpret_cast<const Raw*>(x + eb);
    }
  };
  load(0);
  for (int e = threadIdx.x; e < ntok * g.pairs; e += kThreads) {
    const int tok = e / g.pairs, pr = e - tok * g.pairs;
    // all axes' positions, so that no load waits for the axis
    const float* pos = g.pos + b * g.pos_bs + (t0 + tok) * g.axes;
    const int axis = g.pair_axis[pr];
    float p = pos[0];
    const float p1 = g.axes > 1 ? pos[1] : p, p2 = g.axes > 2 ? pos[2] : p;
    if (axis == 1) p = p1;
    if (axis == 2) p = p2;
    const double turns = static_cast<double>(p) * static_cast<double>(g.pair_freq[pr]) * 0.15915494309189535;
    float s, c;
    sincospif(2.f * static_cast<float>(turns - rint(turns)), &s, &c);
    reinterpret_cast<float2*>(cs)[2 * ((tok * (V / 2) + pr % V / 2) * rot_units + pr / V) + (pr & 1)] = make_float2(c, s);
  }
  if (NORM)
    for (int e = threadIdx.x; e < V * units; e += kThreads) {
      const int lu = e % units, c = e / units % (V / 2), sd = e / units / (V / 2);
      if (g.side[sd].weight) {
        const float* w = g.side[sd].weight + (c < V / 4 ? first_of(lu) + 4 * c : second_of(lu) + 4 * c - V);
        wt[sd][c][lu] = make_float4(w[0], w[1], w[2], w[3]);
      }
    }
  __syncthreads();
  for (int base = 0; base < total; base += kItems * slots) {
    if (base) load(base);
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int n = base + i * slots + slot;
      int tok, s, h;
      head(n, tok, s, h);
      float va[V], vb[V];
      X::open(ra[i], va);
      X::open(rb[i], vb);
      if (NORM) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) ss = fmaf(va[e], va[e], fmaf(vb[e], vb[e], ss));
        // the head's lanes fold onto its first one: after a step of o the lanes below o have all of it
        for (int o = g.fold; o > 0; o >>= 1) {
          const float other = __shfl_down_sync(0xffffffffu, ss, o);
          if (u + o < units && u < o) ss += other;
        }
        ss = __shfl_sync(0xffffffffu, ss, lane - u);
        const float r = rsqrtf(ss * g.inv_d + g.eps);
#pragma unroll
        for (int e = 0; e < V; e += 4) {
          const float4 wa = wt[s][e / 4][u], wb = wt[s][V / 4 + e / 4][u];
          va[e] *= r * wa.x; va[e + 1] *= r * wa.y; va[e + 2] *= r * wa.z; va[e + 3] *= r * wa.w;
          vb[e] *= r * wb.x; vb[e + 1] *= r * wb.y; vb[e + 2] *= r * wb.z; vb[e + 3] *= r * wb.w;
        }
      }
      if (idle || n >= total) continue;
      if (turn) {
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          const float4 c = cs[(tok * (V / 2) + e / 2) * rot_units + u];   // cosine and sine of two pairs
          if constexpr (PAIRS) {                             // pair e of the unit: elements 2 e, 2 e + 1 of the 2 V
#pragma unroll
            for (int d = 0; d < 2; ++d) {
              float& x = 2 * (e + d) < V ? va[2 * (e + d) % V] : vb[2 * (e + d) % V];
              float& y = 2 * (e + d) < V ? va[(2 * (e + d) + 1) % V] : vb[(2 * (e + d) + 1) % V];
              const float x0 = x, co = d ? c.z : c.x, si = d ? c.w : c.y;
              x = x0 * co - y * si;
              y = y * co + x0 * si;
            }
          } else {
            const float x0 = va[e], x1 = va[e + 1];
            va[e] = x0 * c.x - vb[e] * c.y;
            vb[e] = vb[e] * c.x + x0 * c.y;
            va[e + 1] = x1 * c.z - vb[e + 1] * c.w;
            vb[e + 1] = vb[e + 1] * c.z + x1 * c.w;
          }
        }
      }
      const RopeSide& side = g.side[s];
      T* o = static_cast<T*>(side.out) + b * side.out_bs + (t0 + tok) * side.out_rs + h * side.out_hs;
      *reinterpret_cast<Raw*>(o + ea) = X::close(va);
      *reinterpret_cast<Raw*>(o + eb) = X::close(vb);
    }
  }
}

template <typename T, int V>
cudaError_t go(RopeArgs& g, int num_sms, cudaStream_t stream) {
  const int heads = g.side[0].heads + g.side[1].heads, units = g.D / (2 * V);
  const int slots = 32 / units * (kThreads / 32);
  g.fold = 0;
  for (int o = 1; o < units; o <<= 1) g.fold = o;
  g.heads_magic = 0xffffffffu / heads + 1;                   // n / heads = (n * magic) >> 32 for n < 2^32 / heads
  g.inv_d = 1.f / static_cast<float>(g.D);
  // rows per CTA: as many as fill a thread's items, fewer while that leaves SMs without a CTA
  long long tok = kItems * slots / heads;
  const long long spread = static_cast<long long>(g.B) * g.T / (2 * num_sms);
  if (tok > spread) tok = spread;
  if (tok > kMaxTok) tok = kMaxTok;
  if (tok < 1) tok = 1;
  g.tok = static_cast<int>(tok);
  const dim3 grid(static_cast<unsigned>((g.T + tok - 1) / tok), g.B);
  const bool norm = g.side[0].weight != nullptr;
  if (g.interleaved)
    norm ? qk_norm_rope_kernel<T, V, true, true><<<grid, kThreads, 0, stream>>>(g)
         : qk_norm_rope_kernel<T, V, true, false><<<grid, kThreads, 0, stream>>>(g);
  else
    norm ? qk_norm_rope_kernel<T, V, false, true><<<grid, kThreads, 0, stream>>>(g)
         : qk_norm_rope_kernel<T, V, false, false><<<grid, kThreads, 0, stream>>>(g);
  return cudaGetLastError();
}

}  // namespace rope

cudaError_t launch_qk_norm_rope(RopeArgs& g, bool bf16, int num_sms, cudaStream_t stream) {
  // 16-byte vectors: 4 of fp32 (8 measured slower: 36.7 against 32.2 us for 2 x 4608 rows of 20
  // heads of 80), 8 of bf16 where both runs of elements divide into them, 4 else
  if (!bf16) return rope::go<float, 4>(g, num_sms, stream);
  if (g.pairs % 8 == 0 && (g.D - 2 * g.pairs) % 16 == 0) return rope::go<__nv_bfloat16, 8>(g, num_sms, stream);
  return rope::go<__nv_bfloat16, 4>(g, num_sms, stream);
}

}  // namespace gkd
