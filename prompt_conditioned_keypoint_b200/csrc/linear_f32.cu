// gkd_linear for fp32 operands: out = residual + scale * act(x weight^T + bias) on the
// tensor cores, with fp32 accuracy from TF32 products.
//
// Every operand is taken as x = hi + lo: hi is x without its low 13 bits (which
// kind::tf32 does not read, so hi needs no copy), lo = x - hi rounded to TF32. Then
// x w = hi hi + hi lo + lo hi to within 2^-19 of |x w| (lo lo, below 2^-20, and twice
// the rounding of lo), three products per term, where the fp32 units have a sixth of one
// product's rate. lo has its operand's sign, so lo lo has the product's: sums of one sign
// come out 1.5e-7 low at any length.
// The tensor core truncates each step's sum, so a long sum drifts towards zero (at 1024
// channels by 2.4e-6 of the result for plain TF32): an accumulator holds 32 channels,
// small products first, and warps of their own add the accumulators up in fp32. Measured
// error (rms, of the results' rms, normal operands) at 8, 64, 256, 1024 and 4096 channels: 1.8,
// 2.2, 2.2, 2.3 and 2.4e-7 (fp32 products by the library: 0.5, 1.4, 2.9, 5.7 and 11e-7).
//
// A CTA has a 128 x 128 tile of the output, 18 warps:
//   warp 0       TMA: stages of 32 channels of x and of weight (128B-swizzled);
//   warp 1       products, 12 per stage, into two accumulators in turn;
//   warps 2-5    x into tensor memory (a row per lane), as it is and its lo part;
//   warps 6-9    lo parts of weight: 16 bytes in, 16 bytes out at the same place of the
//                next tile, whatever the swizzle;
//   warps 10-17  sums in registers (a thread: one row, 64 columns).
// Few tiles: a cluster of S CTAs shares a tile's channels; the sums meet in shared
// memory in rank order and every CTA finishes its share of the rows.
//
// Measured (B200, in a graph): 1360 x 1024 -> 1024 28 us, 80 rows 9.6 us, 9296 x 1280 -> 5120
// 645 us = 189 TFLOP/s. 64 x 64 tiles on the fp32 units took 120 us for the first; both lo
// parts in shared memory (160 KB through it per stage instead of 96), two accumulators of
// 64 channels, 35. Bound by the stage's chain: some 1300 clocks where its products and
// its shared-memory traffic need 768 each.
#include "blocks_common.cuh"
#include "gkd_internal.h"

namespace gkd {
namespace lin32 {

constexpr int kTile = 128, kChunk = 32, kStages = 4;
constexpr int kOpBytes = kTile * 128;                              // one operand's tile of a stage
constexpr int kStageBytes = 3 * kOpBytes;                          // x, weight, weight's lo part
constexpr uint32_t kColA = 256;                                    // accumulators at 0 and 128, x's stages (hi, lo) at 256 + 64 s
constexpr int kConvWarps = 8, kSumWarps = 8, kThreads = 32 * (2 + kConvWarps + kSumWarps);

struct Args {
  CUtensorMap x, w;
  const float* bias;
  const float* scale;
  const float* residual;
  float* out;
  long long residual_stride, out_stride;
  int T, Cin, Cout;
  short act;
  bool withhold;             // in a word that is read anyway: at the end it was fetched by itself, 0.5 us
  unsigned* err;
  unsigned long long wait_limit_ns;
};

struct Ctl {
  uint64_t full[kStages], ready[kStages], empty[kStages], accfull[2], accempty[2], drain;
  uint32_t tmem_base;
  int abort_flag;
};
constexpr size_t kSmem = 1024 + kStages * static_cast<size_t>(kStageBytes) + sizeof(Ctl);
static_assert(kTile * kTile * 4 <= kStages * kStageBytes, "the sums take the ring's place");

__device__ __forceinline__ float lo_part(float x) {
  const float lo = x - __uint_as_float(__float_as_uint(x) & 0xffffe000u);
  uint32_t r;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(lo));
  return __uint_as_float(r);
}

__global__ void __launch_bounds__(kThreads, 1) linear_f32_kernel(const __grid_constant__ Args a, int S) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + kStages * kStageBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x % S;                                 // = the rank in the cluster
  const int ncol = (a.Cout + kTile - 1) / kTile;
  const int tile = blockIdx.x / S;
  const int t0 = tile / ncol * kTile, n0 = tile % ncol * kTile;
  const int nkall = (a.Cin + kChunk - 1) / kChunk;
  const int kb = static_cast<int>(static_cast<long long>(nkall) * rank / S);
  const int nk = static_cast<int>(static_cast<long long>(nkall) * (rank + 1) / S) - kb;   // may be 0
  const uint64_t lim = a.wait_limit_ns;
  volatile int* abortp = &ctl->abort_flag;
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    const bool okw = mbar_wait_bounded(bar, parity, lim, abortp);
    ok = __all_sync(0xffffffffu, okw) && ok;
    return ok;
  };
  auto give_up = [&] {
    if (lane == 0) {
      ctl->abort_flag = 1;
      atomicOr(a.err, kErrTimeout);
    }
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&ctl->full[s], 1);
      mbar_init(&ctl->ready[s], kConvWarps);
      mbar_init(&ctl->empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ctl->accfull[s], 1);
      mbar_init(&ctl->accempty[s], kSumWarps);
    }
    mbar_init(&ctl->drain, 1);
    ctl->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&ctl->tmem_base, 512);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;

  if (warp == 0) {
    int it = 0;
    for (; it < nk; ++it) {
      const int s = it % kStages;
      if (it >= kStages && !wait(&ctl->empty[s], ((it / kStages) & 1) ^ 1)) break;
      if (lane == 0 && !(a.withhold && it == 0)) {
        mbar_arrive_expect_tx(&ctl->full[s], 2 * kOpBytes);
        tma_load_2d(smem + s * kStageBytes, &a.x, &ctl->full[s], (kb + it) * kChunk, t0);
        tma_load_2d(smem + s * kStageBytes + kOpBytes, &a.w, &ctl->full[s], (kb + it) * kChunk, n0);
      }
      __syncwarp();
    }
    if (!ok) give_up();
    for (int k = 0; k < kStages && k < it; ++k) {
      const int last = it - 1 - k;
      if (!mbar_wait_drain(&ctl->full[last % kStages], (last / kStages) & 1, lim) && lane == 0) atomicOr(a.err, kErrTimeout);
    }
    __syncwarp();
  } else if (warp == 1) {
    // fp32 accumulator, tf32 x tf32, both K-major, M = N = 128
    constexpr uint32_t idesc = (1u << 4) | (2u << 7) | (2u << 10) | (static_cast<uint32_t>(kTile >> 3) << 17) | (8u << 24);
    const uint64_t base = umma_desc_sw128(smem_u32(smem));
    int it = 0;
    for (; it < nk; ++it) {
      const int s = it % kStages, buf = it & 1;
      if (it >= 2 && !wait(&ctl->accempty[buf], ((it >> 1) & 1) ^ 1)) break;
      if (!wait(&ctl->ready[s], (it / kStages) & 1)) break;
      tc_fence_after();
      const uint64_t w = base + ((s * kStageBytes + kOpBytes) >> 4), wl = w + (kOpBytes >> 4);
      const uint32_t d = tmem + 128 * buf, hi = tmem + kColA + 64 * s, lo = hi + 32;
      umma_ts_tf32_x4_elect(d, hi, wl, idesc, 0u);                 // small products first
      umma_ts_tf32_x4_elect(d, lo, w, idesc, 1u);
      umma_ts_tf32_x4_elect(d, hi, w, idesc, 1u);
      umma_commit_elect(&ctl->empty[s]);
      umma_commit_elect(&ctl->accfull[buf]);
    }
    if (!ok) give_up();
    if (it > 0) {                                                  // what was issued ends before the CTA does
      umma_commit_elect(&ctl->drain);
      if (!mbar_wait_drain(&ctl->drain, 0, lim) && lane == 0) atomicOr(a.err, kErrTimeout);
    }
    __syncwarp();
  } else if (warp < 6) {
    // x: a row per lane of tensor memory, as it is (hi) and its lo part
    const int q = warp & 3, r = 32 * q + lane;
    const uint32_t dst = tmem + (static_cast<uint32_t>(32 * q) << 16) + kColA;
    for (int it = 0; it < nk; ++it) {
      const int s = it % kStages;
      if (!wait(&ctl->full[s], (it / kStages) & 1)) break;         // the last products that read the stage have ended
      const uint8_t* p = smem + s * kStageBytes + r * 128;
      uint32_t hi[32], lo[32];
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float4 v = *reinterpret_cast<const float4*>(p + ((c ^ (r & 7)) << 4));
        hi[4 * c] = __float_as_uint(v.x);
        hi[4 * c + 1] = __float_as_uint(v.y);
        hi[4 * c + 2] = __float_as_uint(v.z);
        hi[4 * c + 3] = __float_as_uint(v.w);
      }
#pragma unroll
      for (int c = 0; c < 32; ++c) lo[c] = __float_as_uint(lo_part(__uint_as_float(hi[c])));
      tmem_st_32x32b_x32(dst + 64 * s, hi);
      tmem_st_32x32b_x32(dst + 64 * s + 32, lo);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->ready[s]);
    }
    if (!ok) give_up();
  } else if (warp < 2 + kConvWarps) {
    // weight: lo parts, 16 bytes in, 16 bytes out at the same place of the next tile
    const int tid = threadIdx.x - 32 * 6;
    for (int it = 0; it < nk; ++it) {
      const int s = it % kStages;
      if (!wait(&ctl->full[s], (it / kStages) & 1)) break;
      uint8_t* p = smem + s * kStageBytes + kOpBytes + tid * 16;
#pragma unroll
      for (int i = 0; i < kOpBytes / (16 * 128); ++i) {
        const float4 v = *reinterpret_cast<const float4*>(p + i * (16 * 128));
        *reinterpret_cast<float4*>(p + i * (16 * 128) + kOpBytes) =
            make_float4(lo_part(v.x), lo_part(v.y), lo_part(v.z), lo_part(v.w));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->ready[s]);
    }
    if (!ok) give_up();
  } else {
    const int q = warp & 3, half = (warp - 2 - kConvWarps) >> 2, r = 32 * q + lane;
    const uint32_t src0 = tmem + (static_cast<uint32_t>(32 * q) << 16) + 64 * half;
    float v[64];
#pragma unroll
    for (int j = 0; j < 64; ++j) v[j] = 0.f;
    for (int it = 0; it < nk; ++it) {
      const int buf = it & 1;
      if (!wait(&ctl->accfull[buf], (it >> 1) & 1)) break;
      tc_fence_after();
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        uint32_t d[16];
        tmem_ld_32x32b_x16(src0 + 128 * buf + 16 * g, d);
        tmem_wait_ld_regs(d);
#pragma unroll
        for (int j = 0; j < 16; ++j) v[16 * g + j] += __uint_as_float(d[j]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->accempty[buf]);
    }
    if (!ok) {
      give_up();
    } else {
      // over the ring, which the last product has left; row r's 16-byte pieces c at c ^ (r & 31)
#pragma unroll
      for (int c = 0; c < 16; ++c)
        *reinterpret_cast<float4*>(smem + r * 512 + (((16 * half + c) ^ (r & 31)) << 4)) =
            make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
    }
  }
  tc_fence_before();
  __syncthreads();
  // tensor memory is given back before any wait for another CTA
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (S > 1) cluster_sync();
  const int c = n0 + 4 * lane;
  if (c < a.Cout) {
    const uint32_t base = smem_u32(smem);
    float4 b = make_float4(0.f, 0.f, 0.f, 0.f), sc = make_float4(1.f, 1.f, 1.f, 1.f);
    if (a.bias) b = *reinterpret_cast<const float4*>(a.bias + c);
    if (a.scale) sc = *reinterpret_cast<const float4*>(a.scale + c);
    // a warp's rows, their residuals in flight together
    constexpr int kMine = (kTile + kThreads / 32 - 1) / (kThreads / 32);
    const int last = min((rank + 1) * (kTile / S), a.T - t0);
    auto row = [&](int i) { return rank * (kTile / S) + warp + i * (kThreads / 32); };
    float4 res[kMine];
#pragma unroll
    for (int i = 0; i < kMine; ++i)
      res[i] = a.residual && row(i) < last ? load4(a.residual + static_cast<long long>(t0 + row(i)) * a.residual_stride + c)
                                           : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int r = row(i);
      if (r >= last) break;
      const uint32_t at = r * 512 + ((lane ^ (r & 31)) << 4);
      float z[4] = {b.x, b.y, b.z, b.w};
#pragma unroll 8
      for (int s = 0; s < S; ++s) {
        const float4 v = S > 1 ? cluster_load4(cluster_map(base + at, s)) : *reinterpret_cast<const float4*>(smem + at);
        z[0] += v.x;
        z[1] += v.y;
        z[2] += v.z;
        z[3] += v.w;
      }
      activate(z, a.act);
      store4(a.out + static_cast<long long>(t0 + r) * a.out_stride + c,
             make_float4(fmaf(sc.x, z[0], res[i].x), fmaf(sc.y, z[1], res[i].y), fmaf(sc.z, z[2], res[i].z),
                         fmaf(sc.w, z[3], res[i].w)));
    }
  }
  __syncwarp();
  if (S > 1) cluster_sync();                                       // nobody leaves while its shared memory is read
}

}  // namespace lin32

cudaError_t launch_linear_f32(const LinearArgs& a, int num_sms, cudaStream_t stream, const char** why) {
  using namespace lin32;
  Args p{};
  if (!encode_rows(&p.x, false, a.x, a.Cin, a.T, a.x_stride, kChunk, kTile) ||
      !encode_rows(&p.w, false, a.weight, a.Cin, a.Cout, a.Cin, kChunk, kTile)) {
    *why = "tensor map encoding failed";
    return cudaErrorInvalidValue;
  }
  p.bias = a.bias;
  p.scale = a.scale;
  p.residual = static_cast<const float*>(a.residual);
  p.out = static_cast<float*>(a.out);
  p.residual_stride = a.residual_stride;
  p.out_stride = a.out_stride;
  p.T = a.T;
  p.Cin = a.Cin;
  p.Cout = a.Cout;
  p.act = static_cast<short>(a.act);
  p.err = a.err;
  p.wait_limit_ns = a.wait_limit_ns;
  p.withhold = a.withhold;
  const long long tiles = (static_cast<long long>(a.T) + kTile - 1) / kTile * ((a.Cout + kTile - 1) / kTile);
  const int nk = (a.Cin + kChunk - 1) / kChunk;
  // Few tiles: the channels are split, up to one CTA per SM; clusters of 8 up to two thirds of
  // that, since a group of SMs that shares clusters has places left over (16 clusters of 8 ran
  // in two waves: 17 x 1280 -> 2048 took 19.1 us, with clusters of 4 13.1).
  int S = 1;
  while (S < 8 && tiles * S * 2 <= (S == 4 ? 2 * num_sms / 3 : num_sms) && nk >= 4 * S) S *= 2;
  cudaError_t e = allow_smem<linear_f32_kernel>(kSmem);
  if (e != cudaSuccess) return e;
  return launch_cluster(linear_f32_kernel, dim3(static_cast<unsigned>(tiles * S)), kThreads, kSmem, S, stream, p, S);
}

}  // namespace gkd
