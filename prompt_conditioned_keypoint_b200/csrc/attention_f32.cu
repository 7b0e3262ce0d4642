// gkd_attention on the fp32 units, fp32: out = softmax(scale q k^T) v under a key mask.
//
// One CTA per (batch, head, 64 query rows). Keys come 64 at a time: a thread has
// 4 rows (16 apart) x 8 keys (8 apart) of the scores and 4 rows x (D / 8) columns of the output, with
// the running maximum and sum of its rows (the eight threads of a row group agree
// on them by shuffles). Scores are kept in units of log 2. Key tiles that the
// mask or the diagonal leaves empty are skipped; hidden keys and values are
// replaced by zeros on their way into shared memory, so what they hold never
// meets a product. Few query tiles: a cluster of S CTAs shares the key tiles of one.
#include <type_traits>

#include "blocks_common.cuh"
#include "gkd_internal.h"

namespace gkd {
namespace att {

constexpr int kRows = 64, kKeys = 64, kThreads = 128;
constexpr int kPitch = 72;   // floats between rows of weights: a warp's 4 rows x 8 keys fall on 32 banks

template <int DC>   // DC: head columns in units of 32, rounded up
__global__ void __launch_bounds__(kThreads, DC <= 2 ? 3 : DC == 3 ? 2 : 1) attention_f32_kernel(const __grid_constant__ AttentionArgs a, int S) {
  extern __shared__ float sm[];
  constexpr int DP = 32 * DC + 4;
  float* qs = sm;
  float* ks = qs + kRows * DP;
  float* vs = ks + kKeys * DP;
  float* ps = vs + kKeys * DP;                       // [64][kPitch]
  __shared__ uint8_t ok[kKeys];
  __shared__ uint32_t words[2];
  const int tid = threadIdx.x, rg = tid >> 3, cg = tid & 7;
  const int ntiles = (a.Tq + kRows - 1) / kRows;
  const int rank = blockIdx.x % S, work = blockIdx.x / S;         // = the rank in the cluster, the query tile
  const int tile = work % ntiles;
  const int bh = work / ntiles, h = bh % a.q.heads, b = bh / a.q.heads;
  const int hk = h / (a.q.heads / a.k.heads);
  const int r0 = tile * kRows;
  const float* q = static_cast<const float*>(a.q.data) + b * a.q.batch_stride + h * a.q.head_stride;
  const float* k = static_cast<const float*>(a.k.data) + b * a.k.batch_stride + hk * a.k.head_stride;
  const float* v = static_cast<const float*>(a.v.data) + b * a.v.batch_stride + hk * a.v.head_stride;
  float* o = static_cast<float*>(a.out.data) + b * a.out.batch_stride + h * a.out.head_stride;
  const uint8_t* mask = a.mask ? a.mask + b * a.mask_batch_stride : nullptr;
  const int nq4 = a.D / 4;
  const float qscale = a.scale * 1.4426950408889634f;
#pragma unroll 8
  for (int e = tid; e < kRows * 8 * DC; e += kThreads) {
    const int r = e / (8 * DC), c = e % (8 * DC);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r0 + r < a.Tq && c < nq4) x = load4(q + (r0 + r) * a.q.row_stride + 4 * c);
    *reinterpret_cast<float4*>(qs + r * DP + 4 * c) = x;
  }
  float m[4], l[4], acc[4][4 * DC];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < 4 * DC; ++c) acc[i][c] = 0.f;
  }
  const long long shift = static_cast<long long>(a.Tk) - a.Tq;   // causal: key j for row i iff j <= i + shift
  long long klast = a.Tk;
  if (a.causal) klast = min(klast, min(static_cast<long long>(r0) + kRows, static_cast<long long>(a.Tq)) + shift);
  // this CTA's share of the key tiles
  const long long ktiles = klast > 0 ? (klast + kKeys - 1) / kKeys : 0;
  const long long kend = min(klast, ktiles * (rank + 1) / S * kKeys);
  for (long long k0 = ktiles * rank / S * kKeys; k0 < kend; k0 += kKeys) {
    bool mine = false;
    if (tid < kKeys) {
      mine = k0 + tid < a.Tk && (!mask || mask[k0 + tid] != 0);
    }
    // keys up to the last visible one, in eights
    const uint32_t bits = __ballot_sync(0xffffffffu, mine);
    if ((tid & 31) == 0 && tid < kKeys) words[tid >> 5] = bits;
    if (tid < kKeys) ok[tid] = mine;
    __syncthreads();
    const uint32_t w0 = words[0], w1 = words[1];
    if (!(w0 | w1)) {
      __syncthreads();
      continue;
    }
    const int groups = w1 ? 8 - (__clz(w1) >> 3) : 4 - (__clz(w0) >> 3);
#pragma unroll 4
    for (int e = tid; e < 8 * groups * 8 * DC; e += kThreads) {
      const int r = e / (8 * DC), c = e % (8 * DC);
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
      if (ok[r] && c < nq4) {
        x = load4(k + (k0 + r) * a.k.row_stride + 4 * c);
        y = load4(v + (k0 + r) * a.v.row_stride + 4 * c);
      }
      *reinterpret_cast<float4*>(ks + r * DP + 4 * c) = x;
      *reinterpret_cast<float4*>(vs + r * DP + 4 * c) = y;
    }
    __syncthreads();
    float s[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) s[i][j] = 0.f;
    auto dots = [&](auto half) {                                  // of the first 4 or all 8 groups of keys
      constexpr int kGroups = decltype(half)::value ? 4 : 8;
      for (int c = 0; c < nq4; ++c) {
        float4 qv[4], kv[kGroups];
#pragma unroll
        for (int i = 0; i < 4; ++i) qv[i] = *reinterpret_cast<const float4*>(qs + (rg + 16 * i) * DP + 4 * c);
#pragma unroll
        for (int j = 0; j < kGroups; ++j) kv[j] = *reinterpret_cast<const float4*>(ks + (cg + 8 * j) * DP + 4 * c);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < kGroups; ++j)
            s[i][j] = fmaf(qv[i].x, kv[j].x, fmaf(qv[i].y, kv[j].y, fmaf(qv[i].z, kv[j].z, fmaf(qv[i].w, kv[j].w, s[i][j]))));
      }
    };
    if (groups <= 4)
      dots(std::true_type{});
    else
      dots(std::false_type{});
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long row = r0 + rg + 16 * i;
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool live = ok[cg + 8 * j] && (!a.causal || k0 + cg + 8 * j <= row + shift);
        s[i][j] = live ? s[i][j] * qscale : -INFINITY;
        top = fmaxf(top, s[i][j]);
      }
#pragma unroll
      for (int x = 1; x < 8; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      const float mn = fmaxf(m[i], top);
      const float base = mn == -INFINITY ? 0.f : mn;             // nothing seen yet: every weight is 0
      const float f = ex2_approx(m[i] - base);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float p = ex2_approx(s[i][j] - base);
        sum += p;
        ps[(rg + 16 * i) * kPitch + cg + 8 * j] = p;
      }
#pragma unroll
      for (int x = 1; x < 8; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
      l[i] = l[i] * f + sum;
      m[i] = mn;
#pragma unroll
      for (int c = 0; c < 4 * DC; ++c) acc[i][c] *= f;
    }
    __syncwarp();                                                 // a row's weights come from its own warp
#pragma unroll 2
    for (int j4 = 0; j4 < 2 * groups; ++j4) {
      float4 pv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) pv[i] = *reinterpret_cast<const float4*>(ps + (rg + 16 * i) * kPitch + 4 * j4);
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
#pragma unroll
        for (int d = 0; d < DC; ++d) {
          const float4 x = *reinterpret_cast<const float4*>(vs + (4 * j4 + jj) * DP + 32 * d + 4 * cg);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float p = jj == 0 ? pv[i].x : jj == 1 ? pv[i].y : jj == 2 ? pv[i].z : pv[i].w;
            acc[i][4 * d] = fmaf(p, x.x, acc[i][4 * d]);
            acc[i][4 * d + 1] = fmaf(p, x.y, acc[i][4 * d + 1]);
            acc[i][4 * d + 2] = fmaf(p, x.z, acc[i][4 * d + 2]);
            acc[i][4 * d + 3] = fmaf(p, x.w, acc[i][4 * d + 3]);
          }
        }
      }
    }
    __syncthreads();
  }
  if (S == 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long row = r0 + rg + 16 * i;
      if (row >= a.Tq) continue;
      const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
#pragma unroll
      for (int d = 0; d < DC; ++d)
        if (32 * d + 4 * cg < a.D)
          store4(o + row * a.out.row_stride + 32 * d + 4 * cg,
                 make_float4(acc[i][4 * d] * inv, acc[i][4 * d + 1] * inv, acc[i][4 * d + 2] * inv,
                             acc[i][4 * d + 3] * inv));
    }
    return;
  }
  // The shares meet in shared memory, where the keys were: (O, m, l) of every row, in rank order.
  float* ml = ps;                                                  // [64][2]
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = rg + 16 * i;
#pragma unroll
    for (int d = 0; d < DC; ++d)
      *reinterpret_cast<float4*>(ks + r * DP + 32 * d + 4 * cg) =
          make_float4(acc[i][4 * d], acc[i][4 * d + 1], acc[i][4 * d + 2], acc[i][4 * d + 3]);
    if (cg == 0) {
      ml[2 * r] = m[i];
      ml[2 * r + 1] = l[i];
    }
  }
  cluster_sync();
  const uint32_t oo = smem_u32(ks), om = smem_u32(ml);
  const int share = kRows / S;
  for (int e = tid; e < share * nq4; e += kThreads) {
    const int r = rank * share + e / nq4, c = e % nq4;
    if (r0 + r >= a.Tq) continue;
    float top = -INFINITY;
    for (int s = 0; s < S; ++s) top = fmaxf(top, cluster_load1(cluster_map(om + 8 * r, s)));
    float total = 0.f;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s = 0; s < S; ++s) {
      const float ms = cluster_load1(cluster_map(om + 8 * r, s));
      if (ms == -INFINITY) continue;                               // a share without a key for this row
      const float f = ex2_approx(ms - top);
      const float4 v = cluster_load4(cluster_map(oo + 4 * (r * DP + 4 * c), s));
      total = fmaf(f, cluster_load1(cluster_map(om + 8 * r + 4, s)), total);
      y.x = fmaf(f, v.x, y.x);
      y.y = fmaf(f, v.y, y.y);
      y.z = fmaf(f, v.z, y.z);
      y.w = fmaf(f, v.w, y.w);
    }
    const float inv = total == 0.f ? 0.f : 1.f / total;
    store4(o + (r0 + r) * a.out.row_stride + 4 * c, make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
  }
  __syncwarp();
  cluster_sync();                                                  // nobody leaves while its shared memory is read
}

template <int DC>
cudaError_t go(const AttentionArgs& a, unsigned work, int S, cudaStream_t stream) {
  constexpr size_t bytes = sizeof(float) * ((kRows + 2 * kKeys) * (32 * DC + 4) + kRows * kPitch);
  cudaError_t e = allow_smem<attention_f32_kernel<DC>>(bytes);
  if (e != cudaSuccess) return e;
  return launch_cluster(attention_f32_kernel<DC>, dim3(work * S), kThreads, bytes, S, stream, a, S);
}

}  // namespace att

cudaError_t launch_attention_f32(const AttentionArgs& a, int num_sms, cudaStream_t stream) {
  const long long ntiles = (static_cast<long long>(a.Tq) + att::kRows - 1) / att::kRows;
  const unsigned work = static_cast<unsigned>(ntiles * a.q.heads * a.B);
  // few query tiles: a cluster shares the keys of one, while that keeps to two CTAs per SM
  const int ktiles = static_cast<int>((static_cast<long long>(a.Tk) + att::kKeys - 1) / att::kKeys);
  int S = 1;
  while (S < 8 && static_cast<long long>(work) * S * 2 <= 2 * num_sms && ktiles >= 2 * S) S *= 2;
  switch ((a.D + 31) / 32) {
    case 1:
      return att::go<1>(a, work, S, stream);
    case 2:
      return att::go<2>(a, work, S, stream);
    case 3:
      return att::go<3>(a, work, S, stream);
    default:
      return att::go<4>(a, work, S, stream);
  }
}

}  // namespace gkd
