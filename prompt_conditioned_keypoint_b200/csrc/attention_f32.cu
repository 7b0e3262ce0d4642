// gkd_attention for fp32: out = softmax(scale q k^T) v under a key mask. Three kernels: one
// on the tensor cores, with fp32 accuracy from bf16 products, which this comment describes, and
// below it two on the fma units, for up to 24 keys and for up to 12 or 16 queries.
//
// Every operand is taken as x = b0 + b1 + b2, b0 = bf16(x), b1 = bf16(x - b0), b2 =
// bf16(x - b0 - b1): 24 bits. Of the nine products per term the six with i + j <= 2 are
// formed (the others are below 2^-24 of the term), small ones first. bf16 planes rather
// than TF32 pairs because the second product reads V across its rows, which 16-bit
// operands allow in place. A fp32 unit version of this kernel (64 x 64 tiles in
// shared memory) took 168 us for 64 x 160 padded rows of 16 heads of 64 and 1746 us
// for 2 x 2309 rows of 20 heads.
//
// The tensor core truncates each step's sum, which over a long row of keys would drift
// by 2^-23 per 32 keys: an output accumulator holds one tile of 64 keys, and the softmax
// threads add the tiles up in fp32 registers, where rescaling them costs nothing either.
//
// A CTA has 128 query rows of one head, one CTA per SM, 16 warps:
//   warp 0       decides which tiles of 64 keys are worth doing (mask and diagonal) and
//                hands their key bits to the others through a small ring;
//   warp 1       issues the products: the next tile's scores ahead of this tile's output;
//   warps 4-7    softmax, one row per thread: maximum, weights, their three planes into
//                tensor memory, and the last tile's output added up;
//   warps 8-15   fetch K and V (the next tile's on their way meanwhile) and write their
//                planes as 128B-swizzled tiles. Hidden keys and values become zeros.
// Few query tiles: a cluster of S CTAs shares the key tiles of one and joins (O, m, l)
// through shared memory in rank order.
//
// Measured (B200, in a graph): 64 x 160 padded rows of 16 heads of 64 152 us, 2 x 2309 rows of 20 heads
// 722, 8 x 581 rows of 16 heads of 128 320. Neither memory nor products bound it: the tensor pipe is busy
// 11% (heads of 128: 24%), 27% of the issue slots are taken; one CTA per SM waits at its own barriers.
#include "blocks_common.cuh"
#include "gkd_internal.h"

namespace gkd {
namespace att32 {

constexpr int kThreads = 512, kRows = 128, BN = 64, W = 2, kInfo = 4, kConvThreads = 256;
// 512 threads have 128 registers each; the softmax warps hold a row of scores and one of outputs:
// 64 + 240 + 2 x 104 <= 4 x 128. Each group changes its share once, at the start of its role: a second
// change would need the group's warps to meet before it. The compiler allots registers for 128 a thread all
// the same: heads above 64 spill 484 bytes a thread (804 read back), heads up to 64 4 (36).
constexpr int kRegsIssue = 64, kRegsSoft = 240, kRegsConv = 104;

struct Info {                                       // one key tile
  int k0;                                           // first key, or -1: no more tiles
  int plain;                                        // every key of the tile is visible to every row of the CTA
  int words;                                        // 32-key groups up to the last visible key
  uint32_t bits[W];                                 // keys that the mask and Tk leave
};

template <int DCH>
struct Plan {
  static constexpr int kStages = DCH == 1 ? 2 : 1, kOBufs = DCH == 1 ? 2 : 1;
  static constexpr int kQPlane = kRows * 128 * DCH, kPlane = BN * 128 * DCH;        // bytes
  static constexpr int kKvBytes = 3 * kPlane, kStageBytes = 2 * kKvBytes;           // K's planes, then V's
  struct Ctl {
    uint64_t qready, kready[kStages], kempty[kStages], vready[kStages], vempty[kStages];
    uint64_t ifull[kInfo], iempty[kInfo], sfull[2], pready[2], odone[2], drain;
    Info info[kInfo];
    int first;                                      // the first key that the mask leaves in this CTA's tiles (none: INT_MAX)
    uint32_t tmem_base;
    int abort_flag;
    float m[kRows], l[kRows];                       // of the rows, for the other CTAs of the cluster
  };
  static constexpr size_t kSmem = 1024 + 3 * kQPlane + kStages * kStageBytes + sizeof(Ctl);
};

// Tensor memory: scores at 0 and 64, P's three planes of 32 columns twice, the tile's output (twice for heads
// up to 64: the next tile's product then need not wait until it is added up). Buffers and barriers go by the
// parity of the tile: a softmax warp may be a tile ahead of another.
constexpr uint32_t kColP = 128, kColO = 320;

// Two values as their planes' bf16 pairs.
__device__ __forceinline__ void planes(float x, float y, uint32_t (&p)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    p[i] = pack_bf16x2(x, y);
    x -= bf16_lo(p[i]);
    y -= bf16_hi(p[i]);
  }
}

template <int DCH>
__global__ void __launch_bounds__(kThreads, 1) attention_f32_kernel(const __grid_constant__ AttentionArgs a, int S) {
  using P = Plan<DCH>;
  constexpr int kStages = P::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* qs = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* kv = qs + 3 * P::kQPlane;
  auto* ctl = reinterpret_cast<typename P::Ctl*>(kv + kStages * P::kStageBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ntiles = static_cast<int>((static_cast<long long>(a.Tq) + kRows - 1) / kRows);
  const int rank = blockIdx.x % S, work = blockIdx.x / S;          // = the rank in the cluster, the query tile
  const int tile = ntiles - 1 - work % ntiles;                     // with a diagonal the last rows have the most keys: first
  const int bh = work / ntiles, h = bh % a.q.heads, b = bh / a.q.heads, hk = h / (a.q.heads / a.k.heads);
  const int r0 = tile * kRows;
  const long long shift = static_cast<long long>(a.Tk) - a.Tq;     // causal: key j for row i iff j <= i + shift
  const float scale_log2 = a.scale.c;
  const int dk = (a.D + 15) / 16;
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

  // What a row's output is multiplied by whose sum is 0, having no score above -inf: 0 without a key, but 0 / 0 if it
  // sees one, of score -inf.
  auto empty = [&](int first, int r) { return first <= (a.causal ? r0 + r + shift : static_cast<long long>(a.Tk)) ? NAN : 0.f; };

  if (threadIdx.x == 0) {
    mbar_init(&ctl->qready, kConvThreads / 32);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&ctl->kready[s], kConvThreads / 32);
      mbar_init(&ctl->kempty[s], 1);
      mbar_init(&ctl->vready[s], kConvThreads / 32);
      mbar_init(&ctl->vempty[s], 1);
    }
    for (int s = 0; s < kInfo; ++s) {
      mbar_init(&ctl->ifull[s], 1);
      mbar_init(&ctl->iempty[s], 1 + 4 + kConvThreads / 32);       // products, softmax, converters
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ctl->sfull[s], 1);
      mbar_init(&ctl->pready[s], 4);
      mbar_init(&ctl->odone[s], 1);
    }
    mbar_init(&ctl->drain, 1);
    ctl->abort_flag = 0;
    ctl->first = 0x7fffffff;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&ctl->tmem_base, 512);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  // tile j's info, the slot given back; k0 < 0: no more tiles (or a wait ran out)
  auto next = [&](uint32_t j) {
    Info f;
    f.k0 = -1;
    const uint32_t is = j % kInfo;
    if (wait(&ctl->ifull[is], (j / kInfo) & 1)) {
      f = ctl->info[is];
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->iempty[is]);
    }
    return f;
  };

  if (warp < 4) {
    regs_give_up<kRegsIssue>();
    if (warp == 0) {
      // -------------------------------------------------------------- tiles and key bits
      long long klast = a.Tk;                       // keys that some row of this CTA may see
      if (a.causal) klast = max(0ll, min(klast, min(static_cast<long long>(r0) + kRows, static_cast<long long>(a.Tq)) + shift));
      long long full = a.Tk;                        // and those that every row sees (but for the mask)
      if (a.causal) full = max(0ll, min(full, r0 + shift + 1));
      const int all = static_cast<int>((klast + BN - 1) / BN), seen = static_cast<int>(full / BN);
      const int lo = static_cast<int>(static_cast<long long>(all) * rank / S);
      const int hi = static_cast<int>(static_cast<long long>(all) * (rank + 1) / S);
      const uint8_t* mask = a.mask ? a.mask + b * a.mask_batch_stride : nullptr;
      uint8_t ahead[W];                             // mask bytes of the coming tile
      auto fetch = [&](int t) {
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const long long key = static_cast<long long>(t) * BN + 32 * w + lane;
          ahead[w] = t < hi && key < a.Tk ? (mask ? mask[key] : 1) : 0;
        }
      };
      fetch(lo);
      uint32_t n = 0;                               // tiles handed on
      for (int t = lo; t <= hi && ok; ++t) {
        const bool end = t == hi;
        uint32_t bits[W], any = 0, every = 0xffffffffu;
#pragma unroll
        for (int w = 0; w < W; ++w) {
          bits[w] = __ballot_sync(0xffffffffu, ahead[w] != 0);
          any |= bits[w];
          every &= bits[w];
        }
        if (!end) fetch(t + 1);
        if (!end && !any) continue;
        const uint32_t is = n % kInfo;
        if (n >= kInfo && !wait(&ctl->iempty[is], ((n / kInfo) & 1) ^ 1)) break;
        if (lane == 0) {
          Info& f = ctl->info[is];
          f.k0 = end ? -1 : t * BN;
          f.plain = every == 0xffffffffu && t < seen;
          f.words = bits[1] ? 2 : 1;
          if (n == 0 && !end) ctl->first = t * BN + (bits[0] ? __ffs(bits[0]) : 32 + __ffs(bits[1])) - 1;
          f.bits[0] = bits[0];
          f.bits[1] = bits[1];
          mbar_arrive(&ctl->ifull[is]);
        }
        __syncwarp();
        ++n;
      }
      if (!ok) give_up();
    } else if (warp == 1) {
      // -------------------------------------------------------------- products
      constexpr int kTerms[6][2] = {{2, 0}, {0, 2}, {1, 1}, {1, 0}, {0, 1}, {0, 0}};   // planes, small products first
      const uint32_t idesc_s = (1u << 4) | (1u << 7) | (1u << 10) | (8u << 24);        // and N = the keys taken
      const uint32_t idesc_o = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | (static_cast<uint32_t>(dk * 2) << 17) | (8u << 24);
      const uint64_t qd = umma_desc_sw128(smem_u32(qs)), kd = umma_desc_sw128(smem_u32(kv));
      const uint64_t vd = umma_desc_mn_sw128(smem_u32(kv) + P::kKvBytes, BN * 128);
      bool issued = false;
      auto scores = [&](uint32_t j, int words) {
        const uint32_t s = j % kStages;
        if (!wait(&ctl->kready[s], (j / kStages) & 1)) return;
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < 6; ++i)
#pragma unroll
          for (int c = 0; c < DCH; ++c)
            umma_ss_f16_x4_elect(tmem + 64 * (j & 1), qd + ((kTerms[i][0] * P::kQPlane + c * kRows * 128) >> 4),
                                 kd + ((s * P::kStageBytes + kTerms[i][1] * P::kPlane + c * BN * 128) >> 4),
                                 idesc_s | (static_cast<uint32_t>(words * 4) << 17), (i > 0 || c > 0) ? 1u : 0u);
        issued = true;
        umma_commit_elect(&ctl->sfull[j & 1]);
        umma_commit_elect(&ctl->kempty[s]);
      };
      Info f = next(0);
      if (f.k0 >= 0 && wait(&ctl->qready, 0)) scores(0, f.words);
      for (uint32_t j = 0; f.k0 >= 0 && ok; ++j) {
        const uint32_t s = j % kStages;
        const Info g = next(j + 1);
        if (ok && g.k0 >= 0) scores(j + 1, g.words);               // its buffer was read before P of tile j - 1 was ready
        if (!ok || !wait(&ctl->vready[s], (j / kStages) & 1) || !wait(&ctl->pready[j & 1], (j >> 1) & 1)) break;
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < 6; ++i)
#pragma unroll
          for (int w = 0; w < W; ++w)
            if (w < f.words)
              umma_ts_f16_x2_elect(tmem + kColO + 64 * (j % P::kOBufs), tmem + kColP + 96 * (j & 1) + 32 * kTerms[i][0] + 16 * w,
                                   vd + ((s * P::kStageBytes + kTerms[i][1] * P::kPlane + w * 4096) >> 4), 2048 >> 4,
                                   idesc_o, (i > 0 || w > 0) ? 1u : 0u);
        umma_commit_elect(&ctl->odone[j & 1]);
        umma_commit_elect(&ctl->vempty[s]);
        f = g;
      }
      if (!ok) give_up();
      if (issued) {                                                // what was issued ends before the CTA does
        umma_commit_elect(&ctl->drain);
        if (!mbar_wait_drain(&ctl->drain, 0, lim) && lane == 0) atomicOr(a.err, kErrTimeout);
      }
      __syncwarp();
    }
  } else if (warp < 8) {
    regs_take<kRegsSoft>();
    // ---------------------------------------------------------------- softmax: one row per thread
    const int q = warp & 3, r = 32 * q + lane;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(32 * q) << 16);
    const bool active = r0 + 32 * q < a.Tq;
    float m = -INFINITY, l = 0.f, acc[64 * DCH];
#pragma unroll
    for (int e = 0; e < 64 * DCH; ++e) acc[e] = 0.f;
    // the last tile's output, once its product is done, and the rescaling of all so far
    auto gather = [&](uint32_t j, float f) {
      if (!wait(&ctl->odone[j & 1], (j >> 1) & 1)) return;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < 4 * DCH; ++c) {
        if (c >= dk) continue;
        uint32_t o[16];
        tmem_ld_32x32b_x16(lane_base + kColO + 64 * (j % P::kOBufs) + 16 * c, o);
        tmem_wait_ld_regs(o);
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[16 * c + e] = (acc[16 * c + e] + __uint_as_float(o[e])) * f;
      }
    };
    uint32_t j = 0;
    for (;; ++j) {
      const Info t = next(j);
      if (t.k0 < 0) break;
      uint32_t bits[W] = {t.bits[0], t.bits[1]};
      if (a.causal && !t.plain) {                                  // keys up to the diagonal
        const int v = static_cast<int>(max(0ll, min(r0 + r + shift - t.k0 + 1, static_cast<long long>(BN))));
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const int c = min(max(v - 32 * w, 0), 32);
          bits[w] &= c == 32 ? 0xffffffffu : (1u << c) - 1u;
        }
      }
      if (!wait(&ctl->sfull[j & 1], (j >> 1) & 1)) break;
      tc_fence_after();
      if (!active) {                                // no row inside Tq: barriers alone
        if (j > 0 && !wait(&ctl->odone[(j - 1) & 1], ((j - 1) >> 1) & 1)) break;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->pready[j & 1]);
        continue;
      }
      float x[BN];
#pragma unroll
      for (int w = 0; w < W; ++w) {
        uint32_t(&v)[32] = *reinterpret_cast<uint32_t(*)[32]>(&x[32 * w]);
        if (w < t.words) tmem_ld_32x32b_x32(lane_base + 64 * (j & 1) + 32 * w, v);
      }
#pragma unroll
      for (int w = 0; w < W; ++w) {
        tmem_wait_ld_regs(*reinterpret_cast<uint32_t(*)[32]>(&x[32 * w]));
        if (!t.plain) {
#pragma unroll
          for (int e = 0; e < 32; ++e) x[32 * w + e] = (bits[w] >> e) & 1u ? x[32 * w + e] : -INFINITY;
        }
      }
      float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int e = 0; e < BN; e += 2) t4[(e >> 1) & 3] = max3_nan(t4[(e >> 1) & 3], x[e], x[e + 1]);
      const float top = max3_nan(max3_nan(t4[0], t4[1], t4[2]), t4[3], m);   // NaN if any score was
      const float factor = score_factor(a.scale, top), base = score_offset(a.scale, top);
      const float f = m == -INFINITY ? 0.f : ex2_approx((m - top) * scale_log2);
      m = top;
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int e = 0; e < BN; ++e) {
        x[e] = ex2_approx(fmaf(x[e], factor, -base));
        sum[e & 3] += x[e];
      }
      l = fmaf(l, f, (sum[0] + sum[1]) + (sum[2] + sum[3]));
      // this buffer of P is free: the product that read it last, of tile j - 2, has been gathered
      const uint32_t pcol = lane_base + kColP + 96 * (j & 1);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        if (w >= t.words) continue;
        uint32_t p0[16], p1[16], p2[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          uint32_t p[3];
          planes(x[32 * w + 2 * e], x[32 * w + 2 * e + 1], p);
          p0[e] = p[0];
          p1[e] = p[1];
          p2[e] = p[2];
        }
        tmem_st_32x32b_x16(pcol + 16 * w, p0);
        tmem_st_32x32b_x16(pcol + 32 + 16 * w, p1);
        tmem_st_32x32b_x16(pcol + 64 + 16 * w, p2);
      }
      tmem_wait_st();
      if (P::kOBufs == 1 && j > 0) {                // the product overwrites the last tile's output
        gather(j - 1, f);
        if (!ok) break;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->pready[j & 1]);
      if (P::kOBufs == 2 && j > 0) {                // under this tile's product
        gather(j - 1, f);
        if (!ok) break;
      }
    }
    if (ok && j > 0 && active) gather(j - 1, 1.f);
    if (S > 1 && j == 0) wait(&ctl->qready, 0);     // no tile: Q's planes, which the share overwrites, may still be written
    if (!ok) give_up();
    if (S == 1) {
      const float inv = l == 0.f ? empty(ctl->first, r) : 1.f / l;
      float* o = static_cast<float*>(a.out.data) + b * a.out.batch_stride + (r0 + r) * a.out.row_stride + h * a.out.head_stride;
      if (ok && r0 + r < a.Tq) {
#pragma unroll
        for (int c = 0; c < 16 * DCH; ++c)
          if (4 * c < a.D)
            store4(o + 4 * c, make_float4(acc[4 * c] * inv, acc[4 * c + 1] * inv, acc[4 * c + 2] * inv, acc[4 * c + 3] * inv));
      }
    } else {
      // this CTA's share, over Q's planes (written, and their last reader is done): row r's 16-byte pieces c at c ^ (r & 15)
      ctl->m[r] = m;
      ctl->l[r] = l;
#pragma unroll
      for (int c = 0; c < 16 * DCH; ++c)
        *reinterpret_cast<float4*>(qs + r * (256 * DCH) + ((c ^ (r & 15)) << 4)) =
            make_float4(acc[4 * c], acc[4 * c + 1], acc[4 * c + 2], acc[4 * c + 3]);
    }
  } else {
    regs_give_up<kRegsConv>();
    // ---------------------------------------------------------------- converters
    constexpr int kRow4 = 16 * DCH;                 // 16-byte pieces of a row, 64 columns each chunk
    const int t = threadIdx.x - 256;
    const int c4 = t % kRow4, nq4 = a.D / 4;
    // piece (row, c4) of a plane: four bf16 of a 128-byte swizzled row
    auto put = [&](uint8_t* tile0, int plane_bytes, int chunk_bytes, int row, const float4& v) {
      uint32_t lo[3], hi[3];
      planes(v.x, v.y, lo);
      planes(v.z, v.w, hi);
      const int c = c4 & 15;
      uint8_t* at = tile0 + (c4 >> 4) * chunk_bytes + row * 128 + (((c >> 1) ^ (row & 7)) << 4) + (c & 1) * 8;
#pragma unroll
      for (int i = 0; i < 3; ++i) *reinterpret_cast<uint2*>(at + i * plane_bytes) = make_uint2(lo[i], hi[i]);
    };
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kStep = kConvThreads / kRow4;     // rows between a thread's pieces
    const float* q = static_cast<const float*>(a.q.data) + b * a.q.batch_stride + h * a.q.head_stride;
    const float* k = static_cast<const float*>(a.k.data) + b * a.k.batch_stride + hk * a.k.head_stride;
    const float* v = static_cast<const float*>(a.v.data) + b * a.v.batch_stride + hk * a.v.head_stride;
    float4 kr[BN / kStep], vr[BN / kStep];
    auto fetch = [&](const Info& f) {
#pragma unroll
      for (int i = 0; i < BN / kStep; ++i) {
        const int row = t / kRow4 + i * kStep;
        const bool live = f.k0 >= 0 && c4 < nq4 && ((f.bits[row >> 5] >> (row & 31)) & 1u);
        kr[i] = live ? load4(k + (f.k0 + static_cast<long long>(row)) * a.k.row_stride + 4 * c4) : zero;
        vr[i] = live ? load4(v + (f.k0 + static_cast<long long>(row)) * a.v.row_stride + 4 * c4) : zero;
      }
    };
    // Q first, half of it at a time: its loads wait for no mask
    auto fetch_q = [&](float4* to, int half) {
#pragma unroll
      for (int i = 0; i < BN / kStep; ++i) {
        const int row = 64 * half + t / kRow4 + i * kStep;
        to[i] = r0 + row < a.Tq && c4 < nq4 ? load4(q + (r0 + static_cast<long long>(row)) * a.q.row_stride + 4 * c4) : zero;
      }
    };
    auto put_q = [&](const float4* from, int half) {
#pragma unroll
      for (int i = 0; i < BN / kStep; ++i) put(qs, P::kQPlane, kRows * 128, 64 * half + t / kRow4 + i * kStep, from[i]);
    };
    fetch_q(kr, 0);
    fetch_q(vr, 1);
    put_q(kr, 0);
    put_q(vr, 1);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctl->qready);
    Info f = next(0);
    fetch(f);
    for (uint32_t j = 0; f.k0 >= 0 && ok; ++j) {
      const uint32_t s = j % kStages, ph = (j / kStages) & 1;
      uint8_t* ks = kv + s * P::kStageBytes;
      if (j >= kStages && !wait(&ctl->kempty[s], ph ^ 1)) break;
#pragma unroll
      for (int i = 0; i < BN / kStep; ++i) put(ks, P::kPlane, BN * 128, t / kRow4 + i * kStep, kr[i]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0 && !(a.withhold && j == 0)) mbar_arrive(&ctl->kready[s]);
      if (j >= kStages && !wait(&ctl->vempty[s], ph ^ 1)) break;
#pragma unroll
      for (int i = 0; i < BN / kStep; ++i) put(ks + P::kKvBytes, P::kPlane, BN * 128, t / kRow4 + i * kStep, vr[i]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->vready[s]);
      f = next(j + 1);
      fetch(f);
    }
    if (!ok) give_up();
  }
  tc_fence_before();
  __syncthreads();
  // tensor memory is given back before any wait for another CTA
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (S > 1) {
    cluster_sync();
    const uint32_t om = smem_u32(ctl->m), ol = smem_u32(ctl->l), oo = smem_u32(qs);
    // by the softmax warps, which have the registers for it: the others keep to the barriers from here
    const int pieces = a.D / 4, share = kRows / S;
    for (int i = warp >= 4 && warp < 8 ? threadIdx.x - 128 : share * pieces; i < share * pieces; i += 128) {
      const int r = rank * share + i / pieces, c = i % pieces;
      if (r0 + r >= a.Tq) continue;
      float top = -INFINITY;                        // loops without branches: the loads are in flight together
#pragma unroll 8
      for (int s = 0; s < S; ++s) top = fmaxf(top, cluster_load1(cluster_map(om + 4 * r, s)));
      float l = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
      for (int s = 0; s < S; ++s) {
        const float ms = cluster_load1(cluster_map(om + 4 * r, s));
        const float f = ms == -INFINITY ? 0.f : ex2_approx((ms - top) * scale_log2);   // 0: a share without a key for this row
        const float4 v = cluster_load4(cluster_map(oo + r * (256 * DCH) + ((c ^ (r & 15)) << 4), s));
        l = fmaf(f, cluster_load1(cluster_map(ol + 4 * r, s)), l);
        o.x = fmaf(f, v.x, o.x);
        o.y = fmaf(f, v.y, o.y);
        o.z = fmaf(f, v.z, o.z);
        o.w = fmaf(f, v.w, o.w);
      }
      float inv = 1.f / l;
      if (l == 0.f) {
        int first = 0x7fffffff;
#pragma unroll 1
        for (int s = 0; s < S; ++s)
          first = min(first, __float_as_int(cluster_load1(cluster_map(smem_u32(&ctl->first), s))));
        inv = empty(first, r);
      }
      store4(static_cast<float*>(a.out.data) + b * a.out.batch_stride + (r0 + r) * a.out.row_stride + h * a.out.head_stride + 4 * c,
             make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
    }
    __syncwarp();
    cluster_sync();                                 // nobody leaves while its shared memory is read
  }
}

template <int DCH>
cudaError_t go(const AttentionArgs& a, unsigned work, int S, cudaStream_t stream) {
  static_assert(Plan<DCH>::kSmem <= 227 * 1024, "shared memory");
  cudaError_t e = allow_smem<attention_f32_kernel<DCH>>(Plan<DCH>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_cluster(attention_f32_kernel<DCH>, dim3(work * S), kThreads, Plan<DCH>::kSmem, S, stream, a, S);
}

}  // namespace att32

// Up to 24 keys: scores, softmax and output by fp32 fmas. The tensor-core kernel's CTA, one per SM, spends
// such a call on its set-up; here a CTA of 64 rows needs about 100 registers a thread, so that four or more
// share an SM. Four lanes share a row (16-byte pieces l, l + 4, .. each: a row's loads and stores fill whole
// sectors), a thread has two rows and keeps their scores in registers; K and V, zeros where hidden, lie in
// shared memory, and a read of 64 bytes of it serves the warp's 16 rows. Two shuffles add up a score.
// Bound by HBM at a few keys, by those reads from 16 on. Measured (B200, us, keys 3 / 8 / 16 / 24, the
// tensor-core kernel in brackets): 54 x 131 rows of 20 heads of 64 19.0 / 23.5 / 36.3 / 52.0 (122 to 123),
// 4 x 1024 rows of 8 heads of 128 7.8 / 10.0 / 19 / 24 to 26 (25), 2304 rows of 16 heads of 64
// 5.3 / 6.4 / 9.2 / 12.0 (17.6), one row of 16 heads of 128 4.2 / 4.8 / 7.0 / 8.7 (10). At 32 keys it took
// 85 (123), 31 (25), 20 (17.7) and 11.2 (10).
namespace att32few {

constexpr int kThreads = 128, R = 2, kRows = R * kThreads / 4;

template <int NP, int KMAX>                         // 16-byte pieces of a row per lane: D <= 16 NP; Tk <= KMAX
__global__ void __launch_bounds__(kThreads) attention_few_keys_kernel(const __grid_constant__ AttentionArgs a) {
  __shared__ float4 ks[KMAX * 4 * NP], vs[KMAX * 4 * NP];
  const int ntiles = static_cast<int>((static_cast<long long>(a.Tq) + kRows - 1) / kRows);
  const int tile = blockIdx.x % ntiles, bh = blockIdx.x / ntiles;
  const int h = bh % a.q.heads, b = bh / a.q.heads, hk = h / (a.q.heads / a.k.heads);
  const int lane = threadIdx.x & 31, l4 = lane & 3, nq4 = a.D / 4;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  const float* q = static_cast<const float*>(a.q.data) + b * a.q.batch_stride + h * a.q.head_stride;
  const float* k = static_cast<const float*>(a.k.data) + b * a.k.batch_stride + hk * a.k.head_stride;
  const float* v = static_cast<const float*>(a.v.data) + b * a.v.batch_stride + hk * a.v.head_stride;
  const uint8_t* mask = a.mask ? a.mask + b * a.mask_batch_stride : nullptr;

  // every load before the first use of one
  const uint8_t mine = lane < a.Tk ? (mask ? mask[lane] : 1) : 0;
  constexpr int kPieces = (KMAX * 4 * NP + kThreads - 1) / kThreads;
  float4 kr[kPieces], vr[kPieces];
#pragma unroll
  for (int n = 0; n < kPieces; ++n) {
    const int i = threadIdx.x + n * kThreads, j = i / (4 * NP), c = i % (4 * NP);
    kr[n] = j < a.Tk && c < nq4 ? load4(k + j * a.k.row_stride + 4 * c) : zero;
    vr[n] = j < a.Tk && c < nq4 ? load4(v + j * a.v.row_stride + 4 * c) : zero;
  }
  long long row[R];
  float4 x[R][NP];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    row[i] = static_cast<long long>(tile) * kRows + i * (kThreads / 4) + (threadIdx.x >> 2);
#pragma unroll
    for (int c = 0; c < NP; ++c)
      x[i][c] = row[i] < a.Tq && 4 * c + l4 < nq4 ? load4(q + row[i] * a.q.row_stride + 4 * (4 * c + l4)) : zero;
  }
  const uint32_t seen = __ballot_sync(0xffffffffu, mine != 0);
#pragma unroll
  for (int n = 0; n < kPieces; ++n) {
    const int i = threadIdx.x + n * kThreads;
    const bool live = (seen >> ((i / (4 * NP)) & 31)) & 1u;        // a hidden key's row becomes zeros
    if (i < KMAX * 4 * NP) {
      ks[i] = live ? kr[n] : zero;
      vs[i] = live ? vr[n] : zero;
    }
  }
  __syncthreads();
  if (static_cast<long long>(tile) * kRows + (threadIdx.x >> 5) * 8 >= a.Tq) return;   // a warp without a row

  float w[R][KMAX], inv[R];
#pragma unroll
  for (int j0 = 0; j0 < KMAX; j0 += 4) {            // four keys at a time: their sums in flight together
#pragma unroll
    for (int j = j0; j < j0 + 4; ++j)
#pragma unroll
      for (int i = 0; i < R; ++i) w[i][j] = 0.f;
    if (j0 >= a.Tk) continue;
#pragma unroll
    for (int c = 0; c < NP; ++c)
#pragma unroll
      for (int j = j0; j < j0 + 4; ++j) {
        const float4 y = ks[j * 4 * NP + 4 * c + l4];
#pragma unroll
        for (int i = 0; i < R; ++i)
          w[i][j] = fmaf(x[i][c].x, y.x, fmaf(x[i][c].y, y.y, fmaf(x[i][c].z, y.z, fmaf(x[i][c].w, y.w, w[i][j]))));
      }
#pragma unroll
    for (int m = 1; m <= 2; ++m)
#pragma unroll
      for (int j = j0; j < j0 + 4; ++j)
#pragma unroll
        for (int i = 0; i < R; ++i) w[i][j] += __shfl_xor_sync(0xffffffffu, w[i][j], m);
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    uint32_t bits = seen;
    if (a.causal) {                                 // keys up to the diagonal
      const int n = static_cast<int>(max(0ll, min(row[i] + a.Tk - a.Tq + 1, 32ll)));
      bits &= n == 32 ? 0xffffffffu : (1u << n) - 1u;
    }
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < KMAX; j += 2) {
      w[i][j] = (bits >> j) & 1u ? w[i][j] : -INFINITY;
      w[i][j + 1] = (bits >> (j + 1)) & 1u ? w[i][j + 1] : -INFINITY;
      top = max3_nan(top, w[i][j], w[i][j + 1]);    // NaN if any score was
    }
    const float factor = score_factor(a.scale, top), base = score_offset(a.scale, top);
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < KMAX; ++j) {
      w[i][j] = ex2_approx(fmaf(w[i][j], factor, -base));
      sum[j & 3] += w[i][j];
    }
    const float l = (sum[0] + sum[1]) + (sum[2] + sum[3]);
    // no score above -inf: 0 / 0 for a row that sees a key, 0 for one without
    inv[i] = top == -INFINITY ? (bits ? NAN : 0.f) : 1.f / l;
  }
#pragma unroll
  for (int c = 0; c < NP; ++c) {
    float4 o[R];
#pragma unroll
    for (int i = 0; i < R; ++i) o[i] = zero;
#pragma unroll
    for (int j0 = 0; j0 < KMAX; j0 += 4) {
      if (j0 >= a.Tk) continue;
#pragma unroll
      for (int j = j0; j < j0 + 4; ++j) {
        const float4 y = vs[j * 4 * NP + 4 * c + l4];
#pragma unroll
        for (int i = 0; i < R; ++i)
          o[i] = make_float4(fmaf(w[i][j], y.x, o[i].x), fmaf(w[i][j], y.y, o[i].y), fmaf(w[i][j], y.z, o[i].z),
                             fmaf(w[i][j], y.w, o[i].w));
      }
    }
    if (4 * c + l4 >= nq4) continue;
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (row[i] < a.Tq)
        store4(static_cast<float*>(a.out.data) + b * a.out.batch_stride + row[i] * a.out.row_stride + h * a.out.head_stride +
                   4 * (4 * c + l4),
               make_float4(o[i].x * inv[i], o[i].y * inv[i], o[i].z * inv[i], o[i].w * inv[i]));
  }
}

template <int NP, int KMAX>
cudaError_t go(const AttentionArgs& a, cudaStream_t stream) {
  const long long work = (static_cast<long long>(a.Tq) + kRows - 1) / kRows * a.q.heads * a.B;   // fits: the caller's check
  attention_few_keys_kernel<NP, KMAX><<<static_cast<unsigned>(work), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

template <int KMAX>
cudaError_t go(const AttentionArgs& a, cudaStream_t stream) {
  return a.D <= 64 ? go<4, KMAX>(a, stream) : go<8, KMAX>(a, stream);
}

}  // namespace att32few

// Up to 16 queries (decoding, pooled tokens): K and V go from memory straight into registers and the products
// are fp32 fmas. A CTA has R rows, of all query heads that share a key head (row u is query u / g of head
// u % g): 4, or 1 for a single query without shared heads. L lanes share a key (16-byte pieces l, l + L, ..),
// the groups of a CTA stride through the keys, two at a time, and each keeps its own running maximum, sum and
// output, so that no group waits for another. They are joined at the end: a warp's by shuffles, the warps'
// and those of a cluster of S CTAs (while the GPU has places left) through shared memory, in a fixed order.
// With four rows a thread needs 245 registers (two CTAs per SM); held to 168, or one key at a time in 128,
// it spilled and took twice as long.
// One row is bound by HBM, four by fmas and issue. Measured (B200, us, 1 / 5 / 16 queries, the tensor-core
// kernel, which has 128 rows whatever it gets, in brackets): 57 batches of 20 heads of 64 over 4358 keys with
// holes 222 / 581 / 1112 (1502 to 1506), 64 of 16 heads over 581 55.5 / 111 / 217 (254), one batch over
// 2304 9.1 / 13.7 / 16.1 (28), 8 of 8 heads of 128 over 581 8.4 / 15.7 / 27.7 (37 to 39), 16 batches of
// 16 heads on 4 key heads 10.0 / 25.8 / 51 (70). The time grows with the tiles of four rows; fits() below has the other side.
namespace att32rows {

constexpr int kThreads = 128, kWarps = kThreads / 32, NP = 4, U = 2;

// The first of the keys k0, k0 + step, .. below hi that the mask leaves, or INT_MAX. Out of line: inside the kernel it
// stood between code that every call runs (0.3 of 10 us); noted in the loop over the keys it took 2% of 5 and 16 rows' time.
__device__ __noinline__ int first_key(const uint8_t* mask, long long k0, int hi, int step) {
  for (; k0 < hi; k0 += 8 * step) {
    uint8_t seen[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) seen[e] = k0 + e * step < hi ? (mask ? mask[k0 + e * step] : 1) : 0;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (seen[e]) return static_cast<int>(k0 + e * step);
  }
  return 0x7fffffff;
}

template <int L, int R>                             // lanes per key, NP pieces of 16 bytes each: D <= 16 L; rows
__global__ void __launch_bounds__(kThreads, 2) attention_few_rows_kernel(const __grid_constant__ AttentionArgs a, int S) {
  constexpr int kGroups = kThreads / L, kRow = L * NP;             // pieces of a row
  __shared__ float4 qs[R * kRow], part[kWarps * R * kRow];
  __shared__ float pm[kWarps * R], pl[kWarps * R];
  const int g = a.q.heads / a.k.heads;
  const long long rows = static_cast<long long>(a.Tq) * g;
  const int ntiles = static_cast<int>((rows + R - 1) / R);
  const int rank = blockIdx.x % S, work = blockIdx.x / S;          // = the rank in the cluster
  const int tile = work % ntiles, hk = work / ntiles % a.k.heads, b = work / ntiles / a.k.heads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, piece = lane % L, group = threadIdx.x / L, nq4 = a.D / 4;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  const float* k = static_cast<const float*>(a.k.data) + b * a.k.batch_stride + hk * a.k.head_stride;
  const float* v = static_cast<const float*>(a.v.data) + b * a.v.batch_stride + hk * a.v.head_stride;
  const uint8_t* mask = a.mask ? a.mask + b * a.mask_batch_stride : nullptr;
  const float scale_log2 = a.scale.c;

  for (int i = threadIdx.x; i < R * kRow; i += kThreads) {
    const long long u = static_cast<long long>(tile) * R + i / kRow;
    const int c = i % kRow;
    qs[i] = u < rows && c < nq4 ? load4(static_cast<const float*>(a.q.data) + b * a.q.batch_stride + u / g * a.q.row_stride +
                                        (hk * g + u % g) * a.q.head_stride + 4 * c)
                                : zero;
  }
  int see[R], most = 0;                             // keys up to each row's diagonal
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const long long u = static_cast<long long>(tile) * R + r;
    see[r] = u >= rows    ? 0
             : a.causal   ? static_cast<int>(max(0ll, min(u / g + a.Tk - a.Tq + 1, static_cast<long long>(a.Tk))))
                          : a.Tk;
    most = max(most, see[r]);
  }
  const int lo = static_cast<int>(static_cast<long long>(most) * rank / S);
  const int hi = static_cast<int>(static_cast<long long>(most) * (rank + 1) / S);
  const int turns = (hi - lo + kGroups * U - 1) / (kGroups * U);   // the same for all: the shuffles want whole warps
  float m[R], l[R], off[R];                         // off: m, but 0 where there was no key yet; (s - off) c needs no ScoreScale
  float4 acc[R][NP];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    m[r] = -INFINITY;
    l[r] = off[r] = 0.f;
#pragma unroll
    for (int c = 0; c < NP; ++c) acc[r][c] = zero;
  }
  uint8_t ahead[U];                                 // mask bytes of the coming keys
  auto fetch = [&](int n) {
#pragma unroll
    for (int e = 0; e < U; ++e) {
      const long long key = lo + static_cast<long long>(n * U + e) * kGroups + group;
      ahead[e] = key < hi ? (mask ? mask[key] : 1) : 0;
    }
  };
  fetch(0);
  __syncthreads();
  for (int n = 0; n < turns; ++n) {
    float4 y[U][NP], z[U][NP];
    bool live[U];
#pragma unroll
    for (int e = 0; e < U; ++e) {
      const long long key = lo + static_cast<long long>(n * U + e) * kGroups + group;
      live[e] = ahead[e] != 0;                      // hidden keys and values are not read
#pragma unroll
      for (int c = 0; c < NP; ++c) y[e][c] = live[e] && L * c + piece < nq4 ? load4(k + key * a.k.row_stride + 4 * (L * c + piece)) : zero;
#pragma unroll
      for (int c = 0; c < NP; ++c) z[e][c] = live[e] && L * c + piece < nq4 ? load4(v + key * a.v.row_stride + 4 * (L * c + piece)) : zero;
    }
    fetch(n + 1);
    float s[R][U];
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int e = 0; e < U; ++e) s[r][e] = 0.f;
#pragma unroll
      for (int c = 0; c < NP; ++c) {
        const float4 x = qs[r * kRow + L * c + piece];
#pragma unroll
        for (int e = 0; e < U; ++e)
          s[r][e] = fmaf(x.x, y[e][c].x, fmaf(x.y, y[e][c].y, fmaf(x.z, y[e][c].z, fmaf(x.w, y[e][c].w, s[r][e]))));
      }
    }
#pragma unroll
    for (int d = 1; d < L; d *= 2)
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int e = 0; e < U; ++e) s[r][e] += __shfl_xor_sync(0xffffffffu, s[r][e], d);
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int e = 0; e < U; ++e)
        if (!live[e] || lo + (n * U + e) * kGroups + group >= see[r]) s[r][e] = -INFINITY;
      const float top = max3_nan(m[r], s[r][0], s[r][U - 1]);      // NaN if any score was
      if (top != m[r]) {
        const float f = m[r] == -INFINITY ? 0.f : ex2_approx((m[r] - top) * scale_log2);
        m[r] = off[r] = top;
        l[r] *= f;
#pragma unroll
        for (int c = 0; c < NP; ++c)
          acc[r][c] = make_float4(acc[r][c].x * f, acc[r][c].y * f, acc[r][c].z * f, acc[r][c].w * f);
      }
#pragma unroll
      for (int e = 0; e < U; ++e) {
        const float p = ex2_approx((s[r][e] - off[r]) * scale_log2);
        l[r] += p;
#pragma unroll
        for (int c = 0; c < NP; ++c)
          acc[r][c] = make_float4(fmaf(p, z[e][c].x, acc[r][c].x), fmaf(p, z[e][c].y, acc[r][c].y),
                                  fmaf(p, z[e][c].z, acc[r][c].z), fmaf(p, z[e][c].w, acc[r][c].w));
      }
    }
  }
  // A row without a score above -inf may see a key all the same: the first one that the mask leaves in the group.
  int first = 0x7fffffff;
  bool low = false;
#pragma unroll
  for (int r = 0; r < R; ++r) low |= m[r] == -INFINITY;
  if (low) first = first_key(mask, lo + group, hi, kGroups);
  // the warp's groups
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float top = m[r];
#pragma unroll
    for (int d = L; d <= 16; d *= 2) {
      const float t = __shfl_xor_sync(0xffffffffu, top, d);
      top = max3_nan(top, t, t);
    }
    const float f = m[r] == -INFINITY ? 0.f : ex2_approx((m[r] - top) * scale_log2);
    // no score above -inf in the warp: 1 marks that the row sees a key all the same
    float sum = top == -INFINITY ? (first < see[r] ? 1.f : 0.f) : l[r] * f;
#pragma unroll
    for (int d = L; d <= 16; d *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
#pragma unroll
    for (int c = 0; c < NP; ++c) {
      float4 o = make_float4(acc[r][c].x * f, acc[r][c].y * f, acc[r][c].z * f, acc[r][c].w * f);
#pragma unroll
      for (int d = L; d <= 16; d *= 2) {
        o.x += __shfl_xor_sync(0xffffffffu, o.x, d);
        o.y += __shfl_xor_sync(0xffffffffu, o.y, d);
        o.z += __shfl_xor_sync(0xffffffffu, o.z, d);
        o.w += __shfl_xor_sync(0xffffffffu, o.w, d);
      }
      if (lane < L) part[(warp * R + r) * kRow + L * c + piece] = o;
    }
    if (lane == 0) {
      pm[warp * R + r] = top;
      pl[warp * R + r] = sum;
    }
  }
  __syncthreads();
  if (S > 1) cluster_sync();
  const uint32_t om = smem_u32(pm), ol = smem_u32(pl), oo = smem_u32(part);
  for (int i = threadIdx.x * S + rank; i < R * nq4; i += kThreads * S) {
    const int r = i / nq4, c = i % nq4;
    const long long u = static_cast<long long>(tile) * R + r;
    if (u >= rows) continue;
    float top = -INFINITY, sum = 0.f;
    float4 o = zero;
#pragma unroll 4
    for (int w = 0; w < S * kWarps; ++w) {          // a NaN among them comes back through its own weight
      const uint32_t at = om + 4 * (w % kWarps * R + r);
      top = fmaxf(top, S > 1 ? cluster_load1(cluster_map(at, w / kWarps)) : pm[w * R + r]);
    }
#pragma unroll 4
    for (int w = 0; w < S * kWarps; ++w) {
      const int own = w % kWarps * R + r;
      const float mw = S > 1 ? cluster_load1(cluster_map(om + 4 * own, w / kWarps)) : pm[own];
      const float lw = S > 1 ? cluster_load1(cluster_map(ol + 4 * own, w / kWarps)) : pl[own];
      const float4 ow = S > 1 ? cluster_load4(cluster_map(oo + 16 * (own * kRow + c), w / kWarps)) : part[own * kRow + c];
      const float f = mw == -INFINITY ? 0.f : ex2_approx((mw - top) * scale_log2);
      sum = fmaf(f, lw, sum);
      o = make_float4(fmaf(f, ow.x, o.x), fmaf(f, ow.y, o.y), fmaf(f, ow.z, o.z), fmaf(f, ow.w, o.w));
    }
    float inv = 1.f / sum;
    if (sum == 0.f) {                               // no score above -inf in any warp: 0 / 0 for a row that sees a key, 0 for one without
      float marks = 0.f;
#pragma unroll 1
      for (int w = 0; w < S * kWarps; ++w) {
        const int own = w % kWarps * R + r;
        marks += S > 1 ? cluster_load1(cluster_map(ol + 4 * own, w / kWarps)) : pl[own];
      }
      inv = marks > 0.f ? NAN : 0.f;
    }
    store4(static_cast<float*>(a.out.data) + b * a.out.batch_stride + u / g * a.out.row_stride + (hk * g + u % g) * a.out.head_stride +
               4 * c,
           make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
  }
  __syncwarp();
  if (S > 1) cluster_sync();                        // nobody leaves while its shared memory is read
}

// Up to 12 queries always (2 to 12 took 0.12 to 1.00 of the tensor-core kernel's time over 25 to 400 keys, alone or on
// shared heads, 16 to 1024 heads in the batch), and so 16 over long rows of keys or where the tiles of four rows are one
// wave of CTAs (0.43 to 0.72). Between, those tiles read all keys for less work than that costs: 13 to 16 queries of 1024
// heads of 64 took 1.21 of its time over 25 keys, 1.14 over 48, 1.31 over 128, 1.12 over 256, 0.93 over 400; on shared heads
// 0.98 and 1.21 (13 and 16) over 25 to 128 keys, 0.88 and 1.08 over 192. Heads of 128, 1024 of them: 0.83 over 32 keys, 0.97
// over 48, 1.09 over 64, 1.15 over 128, 1.02 over 192, 0.95 over 256; on shared heads 0.68 to 1.01; 80 and 128 of them
// 0.83 to 1.01.
bool fits(const AttentionArgs& a, int num_sms) {
  if (a.Tq > 16) return false;
  const long long group = a.q.heads / a.k.heads, tiles = (a.Tq * group + 3) / 4 * a.k.heads * a.B;
  if (a.Tq <= 12 || tiles <= 2 * num_sms) return true;
  if (a.D <= 64) return a.Tk > (group > 1 ? 128 : 256);
  return group > 1 || tiles <= 8 * num_sms || a.Tk <= 48 || a.Tk > 192;
}

template <int L, int R>
cudaError_t go(const AttentionArgs& a, int num_sms, cudaStream_t stream) {
  const long long rows = static_cast<long long>(a.Tq) * (a.q.heads / a.k.heads);
  const long long work = (rows + R - 1) / R * a.k.heads * a.B;     // below 2^31: at most 16 x 1024 x 65535 rows
  int S = 1;                                        // up to two CTAs per SM, at least 128 keys each
  while (S < 8 && work * S * 2 <= 2 * num_sms && a.Tk >= 256 * S) S *= 2;
  return launch_cluster(attention_few_rows_kernel<L, R>, dim3(static_cast<unsigned>(work * S)), kThreads, 0, S, stream, a, S);
}

}  // namespace att32rows

cudaError_t launch_attention_f32(const AttentionArgs& a, int num_sms, cudaStream_t stream) {
  // few keys: fma units, above 24 tensor cores (both sides beside that kernel)
  if (a.Tk <= 8) return att32few::go<8>(a, stream);
  if (a.Tk <= 16) return att32few::go<16>(a, stream);
  if (a.Tk <= 24) return att32few::go<24>(a, stream);
  if (att32rows::fits(a, num_sms)) {
    using namespace att32rows;
    if (a.Tq == 1 && a.q.heads == a.k.heads) return a.D <= 64 ? go<4, 1>(a, num_sms, stream) : go<8, 1>(a, num_sms, stream);
    return a.D <= 64 ? go<4, 4>(a, num_sms, stream) : go<8, 4>(a, num_sms, stream);
  }
  using namespace att32;
  const long long work = (static_cast<long long>(a.Tq) + kRows - 1) / kRows * a.q.heads * a.B;
  // few query tiles: a cluster shares the keys of one, while that keeps to one CTA per SM (and to
  // two thirds of them for clusters of 8, of which 16 run in two waves)
  const int ktiles = static_cast<int>((static_cast<long long>(a.Tk) + BN - 1) / BN);
  int S = 1;
  while (S < 8 && work * S * 2 <= (S == 4 ? 2 * num_sms / 3 : num_sms) && ktiles >= 2 * S) S *= 2;
  const unsigned w = static_cast<unsigned>(work);
  return a.D <= 64 ? go<1>(a, w, S, stream) : go<2>(a, w, S, stream);
}

}  // namespace gkd
