// gkd_linear on the tensor cores, bf16 operands:
//   out = residual + scale * act(x weight^T + bias).
// Two kernels. Both feed tcgen05.mma from a ring of 64-channel stages that TMA
// fills (128B-swizzled K-major tiles, zeros past every edge) and accumulate in
// fp32 in tensor memory.
//
//   rows_kernel    many rows: 128 rows x 256 (192, 128) columns per tile, rows on the lanes.
//                  One CTA per SM walks over the tiles; two accumulators, so that
//                  the next tile's products run under this tile's epilogue.
//   split_kernel   few rows: 128 columns (the weights, which are the large operand,
//                  on the lanes) x N <= 64 rows per tile; a cluster of S CTAs
//                  shares a tile's channels, and their partial sums meet in
//                  shared memory (rank order, so the result is always the same);
//                  for fp32 outputs four accumulators in turn.
//
// Measured (B200, in a graph): 36864 x 1280 -> 5120 353 us = 1367 TFLOP/s without an
// activation (the rate that the power limit sustains), 370 to 391 with GELU; 9296 x 4096 ->
// 1024 58 us = 1334 TFLOP/s, 73 with scale and residual onto fp32; 17 x 1280 -> 2048 6.1 us.
//
// The tensor core truncates each K = 16 step's sum, so a sum of Cin products
// drifts towards zero (sums of positive products: 3.7e-7 of the result at 512 channels,
// 1.1e-6 at 1024, 3.4e-6 at 2048). A bf16 output (half a step is 2e-3 and more) does not see
// that at any Cin; for an fp32 output sums of at most 512 channels stay in an accumulator and
// are added up in fp32 by the epilogue's warps, in both kernels and for every Cin.
#include "blocks_common.cuh"
#include "gkd_internal.h"

namespace gkd {
namespace lintc {

constexpr int kChunk = 64;                         // channels per stage: one 128-byte row of bf16
constexpr int kFlush = 8;                          // stages per accumulator for fp32 outputs (512 channels)

__device__ __forceinline__ uint32_t idesc_bf16(int n) {   // fp32 accumulator, bf16 x bf16, both K-major, M = 128
  return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | ((128u >> 4) << 24);
}

// ---------------------------------------------------------------------------
// Many rows
// ---------------------------------------------------------------------------
constexpr int kM = 128, kABytes = kM * 128;
constexpr int kEpiWarps = 8, kWarps = 2 + kEpiWarps, kThreads = 32 * kWarps;
constexpr int kBufBytes = 2048;                    // 32 rows x 64 bytes of output (or residual); two per epilogue warp
constexpr int kMaxStages = 6;

// NT: columns of a tile.
template <int NT>
struct Tile {
  static constexpr int kBBytes = NT * 128, kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = NT == 128 ? 6 : 4;
  static constexpr size_t kSmem = 1024 + kStages * static_cast<size_t>(kStageBytes) + kEpiWarps * 2 * kBufBytes + 512;
  static_assert(kStages <= kMaxStages && kSmem <= 227 * 1024, "ring");
};

struct RowsArgs {
  CUtensorMap x, w, out, res;
  const float* bias;
  const float* scale;
  int T, Cin, Cout;
  short act;
  bool withhold;             // in a word that is read anyway: at the end it was fetched by itself, 0.5 us
  unsigned* err;
  unsigned long long wait_limit_ns;
};

struct RowsCtl {
  uint64_t full[kMaxStages], empty[kMaxStages], accfull[2], accempty[2], res[kEpiWarps][2], drain;
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(RowsCtl) <= 512, "control block");

template <int NT, bool F32OUT, bool RES>
__global__ void __launch_bounds__(kThreads, 1) rows_kernel(const __grid_constant__ RowsArgs a) {
  using R = Tile<NT>;
  constexpr int kStageBytes = R::kStageBytes, kStages = R::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* bufs = smem + kStages * kStageBytes;
  RowsCtl* ctl = reinterpret_cast<RowsCtl*>(bufs + kEpiWarps * 2 * kBufBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ncol = (a.Cout + NT - 1) / NT;
  const long long ntiles = (static_cast<long long>(a.T) + kM - 1) / kM * ncol;
  const int nk = (a.Cin + kChunk - 1) / kChunk;
  const int flush = F32OUT ? kFlush : nk;            // stages per accumulator
  const uint64_t lim = a.wait_limit_ns;
  volatile int* abortp = &ctl->abort_flag;
  auto give_up = [&] {
    ctl->abort_flag = 1;
    atomicOr(a.err, kErrTimeout);
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&ctl->full[s], 1);
      mbar_init(&ctl->empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ctl->accfull[s], 1);
      mbar_init(&ctl->accempty[s], kEpiWarps);
      for (int w = 0; w < kEpiWarps; ++w) mbar_init(&ctl->res[w][s], 1);
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
    // ---------------------------------------------------------------- TMA (one thread)
    if (lane == 0) {
      uint32_t it = 0;
      const uint32_t skip = a.withhold ? 0u : 0xffffffffu;   // the stage that the test hook withholds
      bool ok = true;
      for (long long tile = blockIdx.x; tile < ntiles && ok; tile += gridDim.x) {
        const int t0 = static_cast<int>(tile / ncol) * kM, n0 = static_cast<int>(tile % ncol) * NT;
        for (int k = 0; k < nk; ++k, ++it) {
          const uint32_t s = it % kStages, ph = (it / kStages) & 1;
          if (it >= kStages && !mbar_wait_bounded(&ctl->empty[s], ph ^ 1, lim, abortp)) {
            give_up();
            ok = false;
            break;
          }
          if (it == skip) continue;
          mbar_arrive_expect_tx(&ctl->full[s], kStageBytes);
          tma_load_2d(smem + s * kStageBytes, &a.x, &ctl->full[s], k * kChunk, t0);
          tma_load_2d(smem + s * kStageBytes + kABytes, &a.w, &ctl->full[s], k * kChunk, n0);
        }
      }
      for (uint32_t k = 0; k < kStages && k < it; ++k) {
        const uint32_t last = it - 1 - k;
        if (!mbar_wait_drain(&ctl->full[last % kStages], (last / kStages) & 1, lim)) atomicOr(a.err, kErrTimeout);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA
    // The warp stays converged and one elected lane issues: descriptors then live in
    // uniform registers (a lone thread takes some 230 clocks per product).
    const uint32_t idesc = idesc_bf16(NT);
    const uint64_t adesc = umma_desc_sw128(smem_u32(smem)), bdesc = umma_desc_sw128(smem_u32(smem) + kABytes);
    uint32_t it = 0, acc = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      const bool okw = mbar_wait_bounded(bar, parity, lim, abortp);
      ok = __all_sync(0xffffffffu, okw) && ok;
      return ok;
    };
    for (long long tile = blockIdx.x; tile < ntiles && ok; tile += gridDim.x) {
      for (int k = 0; k < nk; ++k, ++it) {
        const uint32_t s = it % kStages, ph = (it / kStages) & 1;
        const uint32_t buf = acc & 1;
        const bool fresh = k % flush == 0;
        if (fresh && acc >= 2 && !wait(&ctl->accempty[buf], ((acc >> 1) & 1) ^ 1)) break;
        if (!wait(&ctl->full[s], ph)) break;
        tc_fence_after();
        const uint64_t off = static_cast<uint64_t>((s * kStageBytes) >> 4);
        umma_ss_f16_x4_elect(tmem + buf * 256, adesc + off, bdesc + off, idesc, fresh ? 0u : 1u);
        umma_commit_elect(&ctl->empty[s]);
        if (k % flush == flush - 1 || k == nk - 1) {
          umma_commit_elect(&ctl->accfull[buf]);
          ++acc;
        }
      }
    }
    if (!ok && lane == 0) give_up();
    if (it > 0) {                                     // what was issued ends before the CTA does
      umma_commit_elect(&ctl->drain);
      if (!mbar_wait_drain(&ctl->drain, 0, lim) && lane == 0) atomicOr(a.err, kErrTimeout);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- epilogue: 32 rows x NT / 2 columns per warp
    const int q = warp & 3, half = (warp - 2) >> 2, ew = warp - 2;
    uint8_t* mybuf = bufs + ew * 2 * kBufBytes;
    constexpr int kHalf = NT / 2;
    constexpr int kCols = F32OUT ? 16 : 32;          // columns of one 64-byte buffer row
    constexpr int kPieces = kHalf / kCols;
    uint32_t acc = 0, piece = 0;                     // accumulators read, output pieces written
    bool ok = true;
    for (long long tile = blockIdx.x; tile < ntiles && ok; tile += gridDim.x) {
      const int t0 = static_cast<int>(tile / ncol) * kM + 32 * q, n0 = static_cast<int>(tile % ncol) * NT + kHalf * half;
      const int pieces = (t0 < a.T && n0 < a.Cout) ? min(kPieces, (a.Cout - n0 + kCols - 1) / kCols) : 0;
      // the residual is on its way while the products run: to L2, the first piece to its buffer
      if (RES && lane > 0 && lane < pieces) tma_prefetch_2d(&a.res, n0 + lane * kCols, t0);
      if (RES && pieces > 0 && lane == 0) {
        tma_store_wait_read<1>();
        mbar_arrive_expect_tx(&ctl->res[ew][piece & 1], kBufBytes);
        tma_load_2d(mybuf + (piece & 1) * kBufBytes, &a.res, &ctl->res[ew][piece & 1], n0, t0);
      }
      float v[kHalf];
      if (F32OUT) {
#pragma unroll
        for (int j = 0; j < kHalf; ++j) v[j] = 0.f;
      }
      for (int k0 = 0; k0 < nk; k0 += flush, ++acc) {
        const uint32_t buf = acc & 1;
        const bool okw = mbar_wait_bounded(&ctl->accfull[buf], (acc >> 1) & 1, lim, abortp);
        if (!__all_sync(0xffffffffu, okw)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t src = tmem + (static_cast<uint32_t>(32 * q) << 16) + buf * 256 + kHalf * half;
#pragma unroll
        for (int g = 0; g < kHalf / 16; ++g) {
          uint32_t r[16];
          tmem_ld_32x32b_x16(src + 16 * g, r);
          tmem_wait_ld_regs(r);
#pragma unroll
          for (int j = 0; j < 16; ++j) v[16 * g + j] = F32OUT ? v[16 * g + j] + __uint_as_float(r[j]) : __uint_as_float(r[j]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->accempty[buf]);
      }
      if (!ok) {
        if (lane == 0) {
          give_up();
          // a residual load in flight lands before the CTA ends
          if (RES && pieces > 0 && !mbar_wait_drain(&ctl->res[ew][piece & 1], (piece >> 1) & 1, lim))
            atomicOr(a.err, kErrTimeout);
        }
        __syncwarp();
        break;
      }
#pragma unroll
      for (int p = 0; p < kPieces; ++p) {
        if (p >= pieces || !ok) continue;
        uint8_t* buf = mybuf + (piece & 1) * kBufBytes;
        const int c0 = n0 + p * kCols;
        // Bias and activation for the whole piece at once, without branches per vector: columns
        // past Cout (a multiple of 8) take the last ones' values and are clipped by the store.
        float(&y)[kCols] = reinterpret_cast<float(&)[kCols]>(v[p * kCols]);
        auto column = [&](int j) { return min(c0 + 4 * j, a.Cout - 4); };
        if (a.bias) {
#pragma unroll
          for (int j = 0; j < kCols / 4; ++j) {
            const float4 b = __ldg(reinterpret_cast<const float4*>(a.bias + column(j)));
            y[4 * j] += b.x;
            y[4 * j + 1] += b.y;
            y[4 * j + 2] += b.z;
            y[4 * j + 3] += b.w;
          }
        }
        activate(y, a.act);
        if (a.scale) {
#pragma unroll
          for (int j = 0; j < kCols / 4; ++j) {
            const float4 b = __ldg(reinterpret_cast<const float4*>(a.scale + column(j)));
            y[4 * j] *= b.x;
            y[4 * j + 1] *= b.y;
            y[4 * j + 2] *= b.z;
            y[4 * j + 3] *= b.w;
          }
        }
        if (RES) {
          if (p + 1 < pieces && lane == 0) {          // the next piece's residual
            tma_store_wait_read<0>();
            mbar_arrive_expect_tx(&ctl->res[ew][(piece + 1) & 1], kBufBytes);
            tma_load_2d(mybuf + ((piece + 1) & 1) * kBufBytes, &a.res, &ctl->res[ew][(piece + 1) & 1], c0 + kCols, t0);
          }
          const bool okw = mbar_wait_bounded(&ctl->res[ew][piece & 1], (piece >> 1) & 1, lim, abortp);
          if (!__all_sync(0xffffffffu, okw)) {
            ok = false;
            if (lane == 0) {
              give_up();
              for (uint32_t i = 0; i < 2; ++i)
                if (!i || p + 1 < pieces)
                  if (!mbar_wait_drain(&ctl->res[ew][(piece + i) & 1], ((piece + i) >> 1) & 1, lim))
                    atomicOr(a.err, kErrTimeout);
            }
            __syncwarp();
            continue;
          }
        } else {
          if (lane == 0) tma_store_wait_read<1>();
          __syncwarp();
        }
        const uint32_t row = smem_u32(buf) + lane * 64u;
#pragma unroll
        for (int j = 0; j < 4; ++j) {                 // 16-byte vectors of the 64-byte row, 64B-swizzled
          constexpr int kE = F32OUT ? 4 : 8;
          const uint32_t at = row + ((static_cast<uint32_t>(j) ^ ((lane >> 1) & 3u)) << 4);
          uint32_t o[4];
          if (RES) {
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]) : "r"(at) : "memory");
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (F32OUT) {
                y[kE * j + e] += __uint_as_float(o[e]);
              } else {
                y[(kE * j + 2 * e) % kCols] += bf16_lo(o[e]);
                y[(kE * j + 2 * e + 1) % kCols] += bf16_hi(o[e]);
              }
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e)
            o[e] = F32OUT ? __float_as_uint(y[kE * j + e])
                          : pack_bf16x2(y[(kE * j + 2 * e) % kCols], y[(kE * j + 2 * e + 1) % kCols]);
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                       ::"r"(at), "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3]) : "memory");
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(buf, &a.out, c0, t0);
          tma_store_commit();
        }
        ++piece;
      }
    }
    if (lane == 0) tma_store_wait<0>();
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// Few rows
// ---------------------------------------------------------------------------
constexpr int kSplitThreads = 256;
// Stages of 64 channels: as many as let two CTAs share an SM (one CTA's latencies under the
// other's), six at most.
template <int N>
constexpr int kSplitStagesOf = N <= 16 ? 6 : N <= 32 ? 5 : 4;
constexpr int kWBytes = 128 * 128;                 // a stage's weights: 128 columns x 64 channels

struct SplitArgs {
  CUtensorMap x, w;
  const float* bias;
  const float* scale;
  const void* residual;
  void* out;
  long long residual_stride, out_stride;
  int T, Cin, Cout;
  short act;
  bool withhold;             // in a word that is read anyway: at the end it was fetched by itself, 0.5 us
  unsigned* err;
  unsigned long long wait_limit_ns;
};

constexpr int kAccs = 4;                           // accumulators in turn for fp32 outputs (256 columns at N = 64: two CTAs fit)

struct SplitCtl {
  uint64_t full[6], empty[6], accfull[kAccs], accempty[kAccs], drain;
  uint32_t tmem_base;
  int abort_flag;
};

template <int N>
constexpr size_t split_smem() {
  return 1024 + kSplitStagesOf<N> * static_cast<size_t>(kWBytes + N * 128) + sizeof(SplitCtl);
}

template <int N, typename TO>
__global__ void __launch_bounds__(kSplitThreads, 2) split_kernel(const __grid_constant__ SplitArgs a, int S) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr int kBytes = kWBytes + N * 128, kSplitStages = kSplitStagesOf<N>;
  static_assert(N * 512 <= kSplitStages * kBytes, "the partial sums take the ring's place");
  SplitCtl* ctl = reinterpret_cast<SplitCtl*>(smem + kSplitStages * kBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x % S;                   // = the rank in the cluster
  const int n0 = (blockIdx.x / S) * 128, t0 = blockIdx.y * N;
  const int nkall = (a.Cin + kChunk - 1) / kChunk;
  const int kb = static_cast<int>(static_cast<long long>(nkall) * rank / S);
  const int nk = static_cast<int>(static_cast<long long>(nkall) * (rank + 1) / S) - kb;   // may be 0
  constexpr bool kTurns = sizeof(TO) == 4;           // accumulators of kFlush stages in turn, else one for all
  const int parts = kTurns ? (nk + kFlush - 1) / kFlush : min(nk, 1);
  constexpr uint32_t ncols = kTurns ? kAccs * N : N < 32 ? 32 : N;
  const uint64_t lim = a.wait_limit_ns;
  volatile int* abortp = &ctl->abort_flag;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kSplitStages; ++s) {
      mbar_init(&ctl->full[s], 1);
      mbar_init(&ctl->empty[s], 1);
    }
    for (int s = 0; s < kAccs; ++s) {
      mbar_init(&ctl->accfull[s], 1);
      mbar_init(&ctl->accempty[s], 4);
    }
    mbar_init(&ctl->drain, 1);
    ctl->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&ctl->tmem_base, ncols);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;

  if (warp == 0) {
    if (lane == 0) {
      uint32_t it = 0;
      const uint32_t skip = a.withhold ? 0u : 0xffffffffu;
      for (; it < static_cast<uint32_t>(nk); ++it) {
        const uint32_t s = it % kSplitStages, ph = (it / kSplitStages) & 1;
        if (it >= kSplitStages && !mbar_wait_bounded(&ctl->empty[s], ph ^ 1, lim, abortp)) {
          ctl->abort_flag = 1;
          atomicOr(a.err, kErrTimeout);
          break;
        }
        if (it == skip) continue;
        mbar_arrive_expect_tx(&ctl->full[s], kBytes);
        tma_load_2d(smem + s * kBytes, &a.w, &ctl->full[s], (kb + static_cast<int>(it)) * kChunk, n0);
        tma_load_2d(smem + s * kBytes + kWBytes, &a.x, &ctl->full[s], (kb + static_cast<int>(it)) * kChunk, t0);
      }
      for (uint32_t k = 0; k < kSplitStages && k < it; ++k) {
        const uint32_t last = it - 1 - k;
        if (!mbar_wait_drain(&ctl->full[last % kSplitStages], (last / kSplitStages) & 1, lim)) atomicOr(a.err, kErrTimeout);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    const uint32_t idesc = idesc_bf16(N);
    const uint64_t wdesc = umma_desc_sw128(smem_u32(smem)), xdesc = umma_desc_sw128(smem_u32(smem) + kWBytes);
    bool ok = true;
    uint32_t it = 0;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      const bool okw = mbar_wait_bounded(bar, parity, lim, abortp);
      ok = __all_sync(0xffffffffu, okw) && ok;
      return ok;
    };
    for (; it < static_cast<uint32_t>(nk); ++it) {
      const uint32_t s = it % kSplitStages, ph = (it / kSplitStages) & 1;
      const uint32_t acc = kTurns ? it / kFlush % kAccs : 0, turn = kTurns ? it / (kFlush * kAccs) : 0;
      const bool fresh = kTurns ? it % kFlush == 0 : it == 0;
      if (fresh && turn > 0 && !wait(&ctl->accempty[acc], (turn & 1) ^ 1)) break;
      if (!wait(&ctl->full[s], ph)) break;
      tc_fence_after();
      const uint64_t off = static_cast<uint64_t>((s * kBytes) >> 4);
      umma_ss_f16_x4_elect(tmem + acc * N, wdesc + off, xdesc + off, idesc, fresh ? 0u : 1u);
      umma_commit_elect(&ctl->empty[s]);
      if ((kTurns && it % kFlush == kFlush - 1) || it + 1 == static_cast<uint32_t>(nk))
        umma_commit_elect(&ctl->accfull[acc]);
    }
    if (!ok && lane == 0) {
      ctl->abort_flag = 1;
      atomicOr(a.err, kErrTimeout);
    }
    if (it > 0) {                                     // what was issued ends before the CTA does
      umma_commit_elect(&ctl->drain);
      if (!mbar_wait_drain(&ctl->drain, 0, lim) && lane == 0) atomicOr(a.err, kErrTimeout);
    }
    __syncwarp();
  }
  // a CTA's own partial sums, [N rows][128 columns] fp32, over the ring (no product reads it any more)
  float* part = reinterpret_cast<float*>(smem);
  if (warp >= 4) {
    const int q = warp & 3;
    const uint32_t src = tmem + (static_cast<uint32_t>(32 * q) << 16);
    float v[N];
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = 0.f;
    bool ok = true;
    for (int p = 0; p < parts; ++p) {
      const int acc = p % kAccs;
      const bool okw = mbar_wait_bounded(&ctl->accfull[acc], (p / kAccs) & 1, lim, abortp);
      ok = __all_sync(0xffffffffu, okw);
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int g = 0; g < N / 16; ++g) {
        uint32_t r[16];
        tmem_ld_32x32b_x16(src + acc * N + 16 * g, r);
        tmem_wait_ld_regs(r);
#pragma unroll
        for (int j = 0; j < 16; ++j) v[16 * g + j] += __uint_as_float(r[j]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->accempty[acc]);
    }
    if (ok) {                                          // the last products have ended: nothing reads the ring any more
#pragma unroll
      for (int j = 0; j < N; ++j) part[j * 128 + 32 * q + lane] = v[j];
    } else if (lane == 0) {
      ctl->abort_flag = 1;
      atomicOr(a.err, kErrTimeout);
    }
    tc_fence_before();
  }
  __syncthreads();
  // tensor memory is given back before any wait for another CTA, so that no CTA
  // holds it while it waits
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, ncols);
  }
  if (S > 1) cluster_sync();
  const uint32_t base = smem_u32(part);
  const int c = n0 + 4 * lane;
  if (c < a.Cout) {
    float4 b = make_float4(0.f, 0.f, 0.f, 0.f), sc = make_float4(1.f, 1.f, 1.f, 1.f);
    if (a.bias) b = *reinterpret_cast<const float4*>(a.bias + c);
    if (a.scale) sc = *reinterpret_cast<const float4*>(a.scale + c);
    // a warp's rows, their residuals in flight together
    constexpr int kMine = (N + kSplitThreads / 32 - 1) / (kSplitThreads / 32);
    const int last = min((rank + 1) * (N / S), a.T - t0);
    auto row = [&](int i) { return rank * (N / S) + warp + i * (kSplitThreads / 32); };
    float4 res[kMine];
#pragma unroll
    for (int i = 0; i < kMine; ++i)
      res[i] = a.residual && row(i) < last
                   ? load4(static_cast<const TO*>(a.residual) + static_cast<long long>(t0 + row(i)) * a.residual_stride + c)
                   : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int n = row(i);
      if (n >= last) break;
      float z[4] = {b.x, b.y, b.z, b.w};
      const uint32_t at = base + (n * 128 + 4 * lane) * 4;
#pragma unroll 8
      for (int s = 0; s < S; ++s) {
        const float4 v = S > 1 ? cluster_load4(cluster_map(at, s)) : *reinterpret_cast<const float4*>(part + n * 128 + 4 * lane);
        z[0] += v.x;
        z[1] += v.y;
        z[2] += v.z;
        z[3] += v.w;
      }
      activate(z, a.act);
      store4(static_cast<TO*>(a.out) + static_cast<long long>(t0 + n) * a.out_stride + c,
             make_float4(fmaf(sc.x, z[0], res[i].x), fmaf(sc.y, z[1], res[i].y), fmaf(sc.z, z[2], res[i].z),
                         fmaf(sc.w, z[3], res[i].w)));
    }
  }
  __syncwarp();
  if (S > 1) cluster_sync();                         // nobody leaves while its shared memory is read
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
template <int NT, bool F32OUT, bool RES>
cudaError_t go_rows(const RowsArgs& r, unsigned grid, cudaStream_t stream) {
  cudaError_t e = allow_smem<rows_kernel<NT, F32OUT, RES>>(Tile<NT>::kSmem);
  if (e != cudaSuccess) return e;
  rows_kernel<NT, F32OUT, RES><<<grid, kThreads, Tile<NT>::kSmem, stream>>>(r);
  return cudaGetLastError();
}

template <int NT>
cudaError_t launch_rows(const LinearArgs& a, int num_sms, cudaStream_t stream, const char** why) {
  RowsArgs r{};
  const int cols = a.out_bf16 ? 32 : 16;             // 64 bytes
  if (!encode_rows(&r.x, true, a.x, a.Cin, a.T, a.x_stride, kChunk, kM) ||
      !encode_rows(&r.w, true, a.weight, a.Cin, a.Cout, a.Cin, kChunk, NT) ||
      !encode_rows(&r.out, a.out_bf16, a.out, a.Cout, a.T, a.out_stride, cols, 32) ||
      (a.residual && !encode_rows(&r.res, a.out_bf16, a.residual, a.Cout, a.T, a.residual_stride, cols, 32))) {
    *why = "tensor map encoding failed";
    return cudaErrorInvalidValue;
  }
  r.bias = a.bias;
  r.scale = a.scale;
  r.T = a.T;
  r.Cin = a.Cin;
  r.Cout = a.Cout;
  r.act = static_cast<short>(a.act);
  r.err = a.err;
  r.wait_limit_ns = a.wait_limit_ns;
  r.withhold = a.withhold;
  const long long tiles = (static_cast<long long>(a.T) + kM - 1) / kM * ((a.Cout + NT - 1) / NT);
  const unsigned grid = static_cast<unsigned>(tiles < num_sms ? tiles : num_sms);
  if (a.out_bf16) return a.residual ? go_rows<NT, false, true>(r, grid, stream) : go_rows<NT, false, false>(r, grid, stream);
  return a.residual ? go_rows<NT, true, true>(r, grid, stream) : go_rows<NT, true, false>(r, grid, stream);
}

template <int N, typename TO>
cudaError_t go_split(const SplitArgs& p, int S, unsigned ctiles, unsigned rtiles, cudaStream_t stream) {
  constexpr size_t bytes = split_smem<N>();
  cudaError_t e = allow_smem<split_kernel<N, TO>>(bytes);
  if (e != cudaSuccess) return e;
  return launch_cluster(split_kernel<N, TO>, dim3(ctiles * S, rtiles), kSplitThreads, bytes, S, stream, p, S);
}

template <int N>
cudaError_t launch_split(const LinearArgs& a, int S, cudaStream_t stream, const char** why) {
  SplitArgs p{};
  if (!encode_rows(&p.x, true, a.x, a.Cin, a.T, a.x_stride, kChunk, N) ||
      !encode_rows(&p.w, true, a.weight, a.Cin, a.Cout, a.Cin, kChunk, 128)) {
    *why = "tensor map encoding failed";
    return cudaErrorInvalidValue;
  }
  p.bias = a.bias;
  p.scale = a.scale;
  p.residual = a.residual;
  p.out = a.out;
  p.residual_stride = a.residual_stride;
  p.out_stride = a.out_stride;
  p.T = a.T;
  p.Cin = a.Cin;
  p.Cout = a.Cout;
  p.act = static_cast<short>(a.act);
  p.err = a.err;
  p.wait_limit_ns = a.wait_limit_ns;
  p.withhold = a.withhold;
  const unsigned ctiles = (a.Cout + 127) / 128, rtiles = (static_cast<unsigned>(a.T) + N - 1) / N;
  return a.out_bf16 ? go_split<N, __nv_bfloat16>(p, S, ctiles, rtiles, stream)
                    : go_split<N, float>(p, S, ctiles, rtiles, stream);
}

}  // namespace lintc

bool encode_rows(CUtensorMap* m, bool bf16, const void* base, long long cols, long long rows, long long stride, int box_cols,
            int box_rows) {
  EncodeTiledFn enc = get_encode_tiled();
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride) * (bf16 ? 2 : 4)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)}, es[2] = {1, 1};
  return enc && enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2,
                    const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    box_cols * (bf16 ? 2 : 4) == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_linear_tc(const LinearArgs& a, int num_sms, cudaStream_t stream, const char** why) {
  using namespace lintc;
  const long long rtiles = (static_cast<long long>(a.T) + kM - 1) / kM;
  auto ctiles = [&](int n) { return static_cast<long long>((a.Cout + n - 1) / n); };
  if (2 * rtiles * ctiles(128) > num_sms) {
    // The width whose waves of tiles cost least. A wave takes 1.00 : 0.80 : 0.63 of the time
    // for 256 : 192 : 128 columns (36864 x 1280 -> 5120: 363, 396, 460 us; 5120 x 1024 -> 1024,
    // where 256 leaves its second wave nearly empty: 19.3, 17.5, 18.2 us).
    auto cost = [&](int n, int weight) { return (rtiles * ctiles(n) + num_sms - 1) / num_sms * weight; };
    const long long c256 = cost(256, 100), c192 = cost(192, 80), c128 = cost(128, 63);
    if (c256 <= c192 && c256 <= c128) return launch_rows<256>(a, num_sms, stream, why);
    return c192 <= c128 ? launch_rows<192>(a, num_sms, stream, why) : launch_rows<128>(a, num_sms, stream, why);
  }
  // Fewer than half as many tiles as SMs: the channels are split too, while that keeps to about
  // one CTA per SM and leaves each CTA some stages (80 x 4096 -> 1024: 21.1, 14.2, 10.2, 9.7 us
  // with 1, 2, 4, 8; 80 x 1024 -> 1024: 9.8, 8.5, 7.3, 7.8 us; 256 x 1024 -> 1024, where 8 would
  // be two CTAs per SM: 7.8 us with 4, 9.8 with 8; one tile of 128 columns instead: 10.1 us).
  const int nk = (a.Cin + kChunk - 1) / kChunk;
  const int N = a.T <= 32 ? 16 : a.T <= 64 ? 32 : 64;
  const long long tiles = (static_cast<long long>(a.T) + N - 1) / N * ctiles(128);
  int S = 1;
  while (S < 8 && tiles * 2 * S <= num_sms + num_sms / 8 && nk >= (tiles * 4 * S <= num_sms ? 4 : 8) * S) S *= 2;
  switch (N) {
    case 16:
      return launch_split<16>(a, S, stream, why);
    case 32:
      return launch_split<32>(a, S, stream, why);
    default:
      return launch_split<64>(a, S, stream, why);
  }
}

}  // namespace gkd
