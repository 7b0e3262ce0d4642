// gkd_attention on the tensor cores, bf16: out = softmax(scale q k^T) v under a
// key mask, one pass over the keys with a running maximum and sum.
//
// A CTA has 128 query rows of one head (a row per tensor-memory lane) and walks
// over tiles of 64 keys: S = Q K^T into tensor memory (fp32), p = 2^(s - m) by one
// thread per row, P as bf16 over the scores it came from, O += P V with P as the
// tensor-memory operand and V as a shared-memory operand read across its rows
// (head columns contiguous).
//
// A tile is a chain of steps that wait for one another (product, scores to
// registers, exponentials, weights back, product), so what fills an SM is other
// chains: heads of up to 64 columns take 128 columns of tensor memory and four
// CTAs share an SM; wider heads take 256 with two buffers of scores (the next
// tile's product runs under this tile's exponentials) and two CTAs share it.
//
//   warp 0     loads Q, K and V by TMA (128B-swizzled, zeros past every edge). With a
//              mask it decides which key tiles are worth doing and hands their key
//              bits to the others through a small ring;
//   warp 1     issues the products;
//   warps 2-5  softmax, one row per thread. O is rescaled only when a row's maximum has
//              grown by more than 2^8 since the last time; until then the weights are
//              taken against the older maximum, which changes nothing but their
//              common scale (they stay below 2^8).
//
// Hidden keys: their scores are replaced by -inf, and their rows of V in shared
// memory are zeroed before the product (0 x NaN would be NaN).
// Few query tiles: a cluster of S CTAs shares the key tiles of one query tile and
// joins (O, m, l) through shared memory in rank order.
// The weights are rounded to bf16 for the second product (the operand type); their
// sum l is taken from the fp32 values.
//
// Measured (B200, in a graph): 8 x 2309 rows of 20 heads of 64 332 us = 658 TFLOP/s; 12
// heads of 128 276 us = 950; 64 x 80 rows over 576 keys 38.7 us; one row over 2304 keys
// 11.4 us. Bound by the chain's instructions and latencies: on 2 x 2309 rows the
// exponentials keep the special-function unit 53% busy, the tensor pipe is at 27%, 44% of
// the issue slots are taken (heads of 128: 42%, 43%, 36%). Heads up to 64 spill 12 bytes a
// thread in 80 registers, 16 with a mask. Tried and slower for heads of 64: tiles of 128 keys at two
// CTAs per SM (394 to 420 us in six forms: one or two threads per row, weights beside the
// scores, a share of the exponentials on the fma units, 200 registers by giving up the
// others'); scores held in registers at three CTAs per SM (406 us).
#include "blocks_common.cuh"
#include "gkd_internal.h"

namespace gkd {
namespace atc {

constexpr int kSoftWarps = 4, kThreads = 32 * (2 + kSoftWarps), kRows = 128, kKvStages = 2, kInfo = 4;
constexpr int BN = 64, W = BN / 32;                 // keys per tile, words of key bits
constexpr int kMaxSplit = 16;                       // CTAs of a cluster (above 8 the kernel asks for it)
constexpr float kGrow = 8.f;                        // rescale O when a maximum grew by more than this (log2)

struct Args {
  CUtensorMap q, k, v;                              // {D, rows, heads, batch}
  void* out;
  long long out_bs, out_rs, out_hs;
  int heads, group;                                 // query heads, query heads per key head
  int kb_shared;                                    // bit 0: q, 1: k, 2: v has one batch for all
  int Tq, Tk, D, ntiles;
  bool causal, withhold;
  ScoreScale scale;
  const uint8_t* mask;                              // MASK kernels
  long long mask_bs;
  unsigned* err;
  unsigned long long wait_limit_ns;
};

struct Info {                                       // one key tile
  int k0;                                           // first key, or -1: no more tiles
  int plain;                                        // every key of the tile is visible to every row of the CTA
  int words;                                        // 32-key groups up to the last visible key; the rest is left out
  uint32_t bits[W];                                 // keys that the mask and Tk leave
};

struct Ctl {
  uint64_t qfull, kfull[kKvStages], kempty[kKvStages], vfull[kKvStages], vempty[kKvStages];
  uint64_t ifull[kInfo], iempty[kInfo], sfull[2], pready[2], pvdone, odone, drain;
  Info info[kInfo];
  int first;                                        // the first key that the mask leaves in this CTA's tiles (none: INT_MAX)
  uint32_t tmem_base;
  int abort_flag;
  float m[kRows], l[kRows];                         // of the rows, for the other CTAs of the cluster
};

template <int DCH, bool MASK>
__global__ void __launch_bounds__(kThreads, DCH == 1 ? 4 : 2) attention_kernel(const __grid_constant__ Args a, int S) {
  constexpr int kBufs = DCH;                                         // buffers of scores
  constexpr bool kHold = DCH == 2;                                   // 128 registers and more a thread
  constexpr uint32_t kCols = 128 * DCH, kColO = 64 * kBufs;          // scores at 0 (and 64)
  constexpr int kQBytes = kRows * 128 * DCH, kKvBytes = BN * 128 * DCH;
  static_assert(kRows * DCH * 64 * 4 <= 2 * kKvStages * kKvBytes, "the partial output takes the ring's place");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ks = smem + kQBytes;
  uint8_t* vs = ks + kKvStages * kKvBytes;
  Ctl* ctl = reinterpret_cast<Ctl*>(vs + kKvStages * kKvBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x % S;
  const int work = blockIdx.x / S;
  const int tile = a.ntiles - 1 - work % a.ntiles;  // with a diagonal the last rows have the most keys: first
  const int bh = work / a.ntiles, h = bh % a.heads, b = bh / a.heads, hk = h / a.group;
  const int r0 = tile * kRows;
  const long long shift = static_cast<long long>(a.Tk) - a.Tq;       // causal: key j for row i iff j <= i + shift
  const uint64_t lim = a.wait_limit_ns;
  volatile int* abortp = &ctl->abort_flag;
  auto give_up = [&] {
    ctl->abort_flag = 1;
    atomicOr(a.err, kErrTimeout);
  };
  long long klast = a.Tk;                           // keys that some row of this CTA may see
  if (a.causal) klast = max(0ll, min(klast, min(static_cast<long long>(r0) + kRows, static_cast<long long>(a.Tq)) + shift));
  const int all = static_cast<int>((klast + BN - 1) / BN);
  const int lo = static_cast<int>(static_cast<long long>(all) * rank / S);       // this CTA's tiles of keys
  const int hi = static_cast<int>(static_cast<long long>(all) * (rank + 1) / S);
  // without a mask every tile is taken, and what there is to know of it follows from its number
  const int tail = static_cast<int>(klast - static_cast<long long>(all - 1) * BN);   // keys of the last tile of all
  auto words_of = [&](int t) { return t < all - 1 ? W : (tail + 31) / 32; };
  // tiles below this one hold keys that every row of the CTA sees (but for the mask)
  long long full = a.Tk;
  if (a.causal) full = max(0ll, min(full, r0 + shift + 1));
  const int seen = static_cast<int>(full / BN);

  // What a row's output is multiplied by whose sum is 0, having no score above -inf: 0 without a key, but 0 / 0 if it
  // sees one, of score -inf.
  auto empty = [&](int first, int r) {
    return first <= (a.causal ? r0 + r + static_cast<long long>(a.Tk) - a.Tq : static_cast<long long>(a.Tk)) ? NAN : 0.f;
  };

  if (threadIdx.x == 0) {
    mbar_init(&ctl->qfull, 1);
    for (int s = 0; s < kKvStages; ++s) {
      mbar_init(&ctl->kfull[s], 1);
      mbar_init(&ctl->kempty[s], 1);
      mbar_init(&ctl->vfull[s], 1);
      mbar_init(&ctl->vempty[s], 1);
    }
    for (int s = 0; s < kInfo; ++s) {
      mbar_init(&ctl->ifull[s], 1);
      mbar_init(&ctl->iempty[s], kSoftWarps + 1);   // and the one that issues the products
    }
    for (int s = 0; s < kBufs; ++s) {
      mbar_init(&ctl->sfull[s], 1);
      mbar_init(&ctl->pready[s], kSoftWarps);       // one per buffer: a warp may be a tile ahead of another
    }
    mbar_init(&ctl->pvdone, 1);
    mbar_init(&ctl->odone, 1);
    mbar_init(&ctl->drain, 1);
    ctl->abort_flag = 0;
    ctl->first = MASK || lo >= hi ? 0x7fffffff : lo * BN;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&ctl->tmem_base, kCols);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;

  if (warp == 0) {
    // ---------------------------------------------------------------- tiles, key bits, TMA
    const uint8_t* mask = MASK ? a.mask + b * a.mask_bs : nullptr;
    const int bq = a.kb_shared & 1 ? 0 : b, bk = a.kb_shared & 2 ? 0 : b, bv = a.kb_shared & 4 ? 0 : b;
    uint32_t n = 0;                                 // tiles handed on
    bool ok = true;
    uint8_t next[W];                                // mask bytes of the coming tile, loaded ahead
    auto fetch = [&](int t) {
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const long long key = static_cast<long long>(t) * BN + 32 * w + lane;
        next[w] = t < hi && key < a.Tk ? mask[key] : 0;
      }
    };
    if (MASK) fetch(lo);
    for (int t = lo; t <= hi && ok; ++t) {
      const bool end = t == hi;
      const int k0 = t * BN;
      if (MASK) {
        uint32_t bits[W], any = 0, every = 0xffffffffu;
        if (!end) {
#pragma unroll
          for (int w = 0; w < W; ++w) {
            bits[w] = __ballot_sync(0xffffffffu, next[w] != 0);
            any |= bits[w];
            every &= bits[w];
          }
          fetch(t + 1);
          if (!any) continue;
        }
        const uint32_t is = n % kInfo;
        if (n >= kInfo) {
          const bool okw = mbar_wait_bounded(&ctl->iempty[is], ((n / kInfo) & 1) ^ 1, lim, abortp);
          if (!__all_sync(0xffffffffu, okw)) ok = false;
        }
        if (ok && lane == 0) {
          Info& f = ctl->info[is];
          f.k0 = end ? -1 : k0;
          if (!end) {
            if (n == 0) ctl->first = k0 + (bits[0] ? __ffs(bits[0]) : 32 + __ffs(bits[W - 1])) - 1;
            f.plain = every == 0xffffffffu && t < seen;
            f.words = 1;
#pragma unroll
            for (int w = 0; w < W; ++w) {
              f.bits[w] = bits[w];
              if (bits[w]) f.words = w + 1;
            }
          }
          mbar_arrive(&ctl->ifull[is]);
        }
        __syncwarp();
      }
      if (end || !ok) break;
      if (lane == 0) {
        if (n == 0) {
          mbar_arrive_expect_tx(&ctl->qfull, kQBytes);
          for (int c = 0; c < DCH; ++c)
            tma_load_4d(smem + c * kRows * 128, &a.q, &ctl->qfull, 64 * c, r0, h, bq);
        }
        const uint32_t s = n % kKvStages, ph = (n / kKvStages) & 1;
        if (n < kKvStages || mbar_wait_bounded(&ctl->kempty[s], ph ^ 1, lim, abortp)) {
          if (!(a.withhold && n == 0)) mbar_arrive_expect_tx(&ctl->kfull[s], kKvBytes);
          for (int c = 0; c < DCH && !(a.withhold && n == 0); ++c)
            tma_load_4d(ks + s * kKvBytes + c * BN * 128, &a.k, &ctl->kfull[s], 64 * c, k0, hk, bk);
          if (n < kKvStages || mbar_wait_bounded(&ctl->vempty[s], ph ^ 1, lim, abortp)) {
            mbar_arrive_expect_tx(&ctl->vfull[s], kKvBytes);
            for (int c = 0; c < DCH; ++c)
              tma_load_4d(vs + s * kKvBytes + c * BN * 128, &a.v, &ctl->vfull[s], 64 * c, k0, hk, bv);
          } else {
            if (!mbar_wait_drain(&ctl->kfull[s], ph, lim)) atomicOr(a.err, kErrTimeout);
            ok = false;
          }
        } else {
          ok = false;
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (ok) ++n;
    }
    if (lane == 0) {
      if (!ok) give_up();
      if (n > 0 && !mbar_wait_drain(&ctl->qfull, 0, lim)) atomicOr(a.err, kErrTimeout);
      for (uint32_t i = 0; i < kKvStages && i < n; ++i) {
        const uint32_t last = n - 1 - i, s = last % kKvStages, ph = (last / kKvStages) & 1;
        if (!mbar_wait_drain(&ctl->kfull[s], ph, lim) || !mbar_wait_drain(&ctl->vfull[s], ph, lim))
          atomicOr(a.err, kErrTimeout);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- products
    // The warp stays converged and one elected lane issues: descriptors then live in
    // uniform registers (a lone thread needed 900 clocks to issue four products).
    const int dk = (a.D + 15) / 16;
    const uint32_t idesc_s = (1u << 4) | (1u << 7) | (1u << 10) | (8u << 24);        // and N = the keys taken
    const uint32_t idesc_o = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | (static_cast<uint32_t>(dk * 2) << 17) | (8u << 24);
    const uint64_t qd = umma_desc_sw128(smem_u32(smem)), kd = umma_desc_sw128(smem_u32(ks));
    const uint64_t vd = umma_desc_mn_sw128(smem_u32(vs), BN * 128);
    bool ok = true, issued = false;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      const bool okw = mbar_wait_bounded(bar, parity, lim, abortp);
      ok = __all_sync(0xffffffffu, okw) && ok;
      return ok;
    };
    auto more = [&](uint32_t j) {                                    // words of tile j, 0: no more (its info slot is then done with)
      if (!MASK) return lo + static_cast<int>(j) < hi ? words_of(lo + static_cast<int>(j)) : 0;
      const uint32_t is = j % kInfo;
      if (!wait(&ctl->ifull[is], (j / kInfo) & 1)) return 0;
      const int words = ctl->info[is].k0 >= 0 ? ctl->info[is].words : 0;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->iempty[is]);
      return words;
    };
    // Scores of tile j, in order behind the output product that last read their buffer.
    auto scores = [&](uint32_t j, int words) {
      const uint32_t s = j % kKvStages;
      // columns past D are zeros in both operands, so whole 64-column chunks are multiplied
#pragma unroll
      for (int c = 0; c < DCH; ++c)
        umma_ss_f16_x4_elect(tmem + 64 * (j % kBufs), qd + ((c * kRows * 128) >> 4), kd + ((s * kKvBytes + c * BN * 128) >> 4),
                             idesc_s | (static_cast<uint32_t>(words * 4) << 17), c > 0 ? 1u : 0u);
      issued = true;
      umma_commit_elect(&ctl->sfull[j % kBufs]);
      umma_commit_elect(&ctl->kempty[s]);
    };
    int words = more(0);
    if (words && wait(&ctl->qfull, 0) && wait(&ctl->kfull[0], 0)) scores(0, words);
    for (uint32_t j = 0; words && ok; ++j) {
      const uint32_t s = j % kKvStages, ph = (j / kKvStages) & 1, sn = (j + 1) % kKvStages, phn = ((j + 1) / kKvStages) & 1;
      const int ahead = more(j + 1);
      if (!ok || (ahead && !wait(&ctl->kfull[sn], phn))) break;
      if (kBufs == 2 && ahead) scores(j + 1, ahead);
      if (!wait(&ctl->vfull[s], ph) || !wait(&ctl->pready[j % kBufs], (j / kBufs) & 1)) break;
      tc_fence_after();
#pragma unroll
      for (int w = 0; w < W; ++w)
        if (w < words)
          umma_ts_f16_x2_elect(tmem + kColO, tmem + 64 * (j % kBufs) + 16 * w, vd + ((s * kKvBytes + w * 4096) >> 4),
                               2048 >> 4, idesc_o, (j > 0 || w > 0) ? 1u : 0u);
      if (!ahead) umma_commit_elect(&ctl->odone);
      if (kBufs == 2) umma_commit_elect(&ctl->pvdone);               // else the next tile's scores say it
      if (kBufs == 1 && ahead) scores(j + 1, ahead);
      umma_commit_elect(&ctl->vempty[s]);
      words = ahead;
    }
    if (!ok && lane == 0) give_up();
    if (issued) {                                                    // what was issued ends before the CTA does
      umma_commit_elect(&ctl->drain);
      if (!mbar_wait_drain(&ctl->drain, 0, lim) && lane == 0) atomicOr(a.err, kErrTimeout);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- softmax: one row per thread
    const int q = warp & 3, r = 32 * q + lane;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(32 * q) << 16);
    const int ochunks = (a.D + 15) / 16;
    // A warp without a row inside Tq keeps to the barriers: what its lanes of tensor memory hold meets no other row.
    const bool active = r0 + 32 * q < a.Tq;
    float m = -INFINITY, l = 0.f;                   // the maximum that the weights are taken against, their sum
    uint32_t j = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      const bool okw = mbar_wait_bounded(bar, parity, lim, abortp);
      ok = __all_sync(0xffffffffu, okw) && ok;
      return ok;
    };
    for (;; ++j) {
      bool plain;
      int words, k0;
      uint32_t bits[W], hidden = 0;
      if (MASK) {
        const uint32_t is = j % kInfo;
        if (!wait(&ctl->ifull[is], (j / kInfo) & 1)) break;
        const Info& f = ctl->info[is];
        k0 = f.k0;
        plain = f.plain != 0;
        words = f.words;
        if (k0 >= 0 && !plain) {
#pragma unroll
          for (int w = 0; w < W; ++w) bits[w] = f.bits[w];
          hidden = r < BN ? !((f.bits[r >> 5 & (W - 1)] >> lane) & 1u) : 0u;   // this thread's row of V goes
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->iempty[is]);
        if (k0 < 0) break;
      } else {
        const int t = lo + static_cast<int>(j);
        if (t >= hi) break;
        k0 = t * BN;
        words = words_of(t);
        plain = t < seen;
#pragma unroll
        for (int w = 0; w < W; ++w) bits[w] = 0xffffffffu;
      }
      if (!plain) {                                 // keys of the tile up to the last one, and up to the diagonal
        long long vis = static_cast<long long>(a.Tk) - k0;
        if (a.causal) vis = min(vis, r0 + r + shift - k0 + 1);
        const int v = static_cast<int>(max(0ll, min(vis, static_cast<long long>(BN))));
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const int c = min(max(v - 32 * w, 0), 32);
          bits[w] &= c == 32 ? 0xffffffffu : (1u << c) - 1u;
        }
      }
      if (!wait(&ctl->sfull[j % kBufs], (j / kBufs) & 1)) break;
      tc_fence_after();
      const uint32_t scores = lane_base + 64 * (j % kBufs);
      if (active) {
        // Hidden keys: -inf over their scores first, so that what follows is the same code
        // without tests for every tile. (With the tests inside it 8 x 2309 rows took 386 us
        // against 344; a second copy of it for whole tiles took 335, but 80 x 77 causal rows
        // under a mask 35.8 against 30.9.)
        if (!plain) {
#pragma unroll 1
          for (int g = 0; g < 2 * W; ++g) {
            uint32_t x[16] = {};
            if (g < 2 * words) {
              tmem_ld_32x32b_x16(scores + 16 * g, x);
              tmem_wait_ld_regs(x);
            }
            const uint32_t b16 = (g < 2 ? bits[0] : bits[1]) >> (16 * (g & 1));
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (!((b16 >> e) & 1u)) x[e] = 0xff800000u;
            tmem_st_32x32b_x16(scores + 16 * g, x);
          }
          tmem_wait_st();
        }
        // Groups of 16 scores. With two CTAs per SM a tile's scores stay in registers; with
        // four they are read twice, for the maximum and for the weights, and a group is on
        // its way while the one before is worked on.
        uint32_t v[kHold ? 2 * W : 2][16];
        float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        auto load = [&](int g) { tmem_ld_32x32b_x16(scores + 16 * g, v[kHold ? g : g & 1]); };
        load(0);
        if (kHold) {
#pragma unroll
          for (int g = 1; g < 2 * W; ++g) load(g);
        }
#pragma unroll
        for (int g = 0; g < 2 * W; ++g) {
          uint32_t(&x)[16] = v[kHold ? g : g & 1];
          tmem_wait_ld_regs(x);
          if (!kHold && g + 1 < 2 * W) load(g + 1);
#pragma unroll
          for (int e = 0; e < 16; e += 2)
            t4[(e >> 1) & 3] = max3_nan(t4[(e >> 1) & 3], __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
        }
        const float top = max3_nan(max3_nan(t4[0], t4[1], t4[2]), t4[3], t4[3]);   // NaN if any score is
        const bool grow = !((top - m) * a.scale.c <= kGrow);   // also for NaN, and where there was no key before
        if (__any_sync(0xffffffffu, grow)) {
          float mn = max3_nan(m, top, top);
          if (mn == INFINITY) mn = NAN;               // infinity against infinity: the row is NaN
          const float f = m == -INFINITY ? 0.f : ex2_approx((m - mn) * a.scale.c);
          m = mn;
          l *= f;
          if (j > 0) {
            // O is at rest: the product before the last ended before these scores were
            // formed, and with one buffer the last one did too
            if (kBufs == 2 && !wait(&ctl->pvdone, (j - 1) & 1)) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < ochunks; ++c) {
              uint32_t o[16];
              tmem_ld_32x32b_x16(lane_base + kColO + 16 * c, o);
              tmem_wait_ld_regs(o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st_32x32b_x16(lane_base + kColO + 16 * c, o);
            }
          }
        }
        const float factor = score_factor(a.scale, m), base = score_offset(a.scale, m);
        const float2 scale2 = make_float2(factor, factor), base2 = make_float2(-base, -base);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        if (!kHold) load(0);
#pragma unroll
        for (int g = 0; g < 2 * W; ++g) {
          uint32_t(&x)[16] = v[kHold ? g : g & 1];
          if (!kHold) {
            tmem_wait_ld_regs(x);
            if (g + 1 < 2 * W) load(g + 1);
          }
          uint32_t p[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float2 y = fma2(make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), scale2, base2);
            y.x = ex2_approx(y.x);
            y.y = ex2_approx(y.y);
            sum[e & 1] = add2(sum[e & 1], y);
            p[e] = pack_bf16x2(y.x, y.y);
          }
          tmem_st_32x32b_x8(scores + 8 * g, p);       // over scores that are done with: 8 g + 8 <= 16 g + 16
        }
        sum[0] = add2(sum[0], sum[1]);
        l += sum[0].x + sum[0].y;
        tmem_wait_st();
      }
      if (MASK && !plain) {                         // rows of V that no row may see
        const uint32_t s = j % kKvStages;
        if (!wait(&ctl->vfull[s], (j / kKvStages) & 1)) break;
        if (hidden) {
          for (int c = 0; c < DCH; ++c)
#pragma unroll
            for (int e = 0; e < 8; ++e)
              *reinterpret_cast<uint4*>(vs + s * kKvBytes + c * BN * 128 + r * 128 + 16 * e) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->pready[j % kBufs]);
    }
    if (ok && j > 0) {
      wait(&ctl->odone, 0);
      tc_fence_after();
    }
    if (!ok && lane == 0) give_up();
    const bool mine = ok && r0 + r < a.Tq;
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.out) + b * a.out_bs + (r0 + r) * a.out_rs + h * a.out_hs;
    if (S > 1) {
      ctl->m[r] = m;
      ctl->l[r] = l;
    }
    for (int c = 0; active && c < ochunks; ++c) {
      uint32_t v[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = 0u;
      if (ok && j > 0) {
        tmem_ld_32x32b_x16(lane_base + kColO + 16 * c, v);
        tmem_wait_ld_regs(v);
      }
      if (S == 1) {
        if (!mine) continue;
        const float inv = l == 0.f ? empty(ctl->first, r) : 1.f / l;
#pragma unroll
        for (int e = 0; e < 16; e += 8) {
          if (16 * c + e >= a.D) continue;
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = pack_bf16x2(__uint_as_float(v[e + 2 * i]) * inv, __uint_as_float(v[e + 2 * i + 1]) * inv);
          *reinterpret_cast<uint4*>(o + 16 * c + e) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      } else {
        // this CTA's share, over the K and V ring (its last reader, the last product, is done):
        // row r's 16-byte pieces c at c ^ (r & 15), so that the 32 rows of a store spread over the banks
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *reinterpret_cast<uint4*>(ks + r * (256 * DCH) + (((4 * c + e) ^ (r & 15)) << 4)) =
              make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  // tensor memory is given back before any wait for another CTA
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
  if (S > 1) {
    cluster_sync();
    const uint32_t om = smem_u32(ctl->m), ol = smem_u32(ctl->l), oo = smem_u32(ks);
    const int pieces = a.D / 4, share = kRows / S;
    for (int i = threadIdx.x; i < share * pieces; i += kThreads) {
      const int r = rank * share + i / pieces, c = i % pieces;
      if (r0 + r >= a.Tq) continue;
      float m = -INFINITY;                          // loops without branches: the loads are in flight together
#pragma unroll 8
      for (int s = 0; s < S; ++s) m = fmaxf(m, cluster_load1(cluster_map(om + 4 * r, s)));
      float l = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
      for (int s = 0; s < S; ++s) {
        const float ms = cluster_load1(cluster_map(om + 4 * r, s));
        const float f = ms == -INFINITY ? 0.f : ex2_approx((ms - m) * a.scale.c);   // 0: a share without a key for this row
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
      store4(static_cast<__nv_bfloat16*>(a.out) + b * a.out_bs + (r0 + r) * a.out_rs + h * a.out_hs + 4 * c,
             make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
    }
    __syncwarp();
    cluster_sync();                                 // nobody leaves while its shared memory is read
  }
}

bool encode(CUtensorMap* m, const HeadsView& t, int B, int rows, int D, int box_rows) {
  EncodeTiledFn enc = get_encode_tiled();
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(t.heads),
                              static_cast<cuuint64_t>(t.batch_stride ? B : 1)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(t.row_stride) * 2, static_cast<cuuint64_t>(t.head_stride) * 2,
                                 static_cast<cuuint64_t>(t.batch_stride ? t.batch_stride : t.row_stride) * 2};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(box_rows), 1, 1}, es[4] = {1, 1, 1, 1};
  return enc && enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, t.data, dims, strides, box, es,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DCH, bool MASK>
cudaError_t go(const Args& a, int S, unsigned work, cudaStream_t stream) {
  constexpr size_t bytes = 1024 + kRows * 128 * DCH + 2 * kKvStages * BN * 128 * DCH + sizeof(Ctl);
  static_assert((DCH == 1 ? 4 : 2) * (bytes + 1024) <= 228 * 1024, "CTAs per SM");
  cudaError_t e = allow_smem<attention_kernel<DCH, MASK>>(bytes, true);
  if (e != cudaSuccess) return e;
  return launch_cluster(attention_kernel<DCH, MASK>, dim3(work * S), kThreads, bytes, S, stream, a, S);
}

// Attention over no keys: zeros. `row16`: 16-byte pieces of a head's row; strides in bytes.
__global__ void __launch_bounds__(128) zero_kernel(uint8_t* out, long long bs, long long rs, long long hs, int B, int T,
                                                   int heads, int row16) {
  for (long long row = blockIdx.x; row < static_cast<long long>(B) * T; row += gridDim.x)
    for (int i = threadIdx.x; i < heads * row16; i += blockDim.x)
      *reinterpret_cast<uint4*>(out + row / T * bs + row % T * rs + i / row16 * hs + i % row16 * 16) =
          make_uint4(0u, 0u, 0u, 0u);
}

}  // namespace atc

cudaError_t launch_attention_none(const AttentionArgs& a, int size, cudaStream_t stream) {
  const long long rows = static_cast<long long>(a.B) * a.Tq;
  atc::zero_kernel<<<static_cast<unsigned>(rows < 65536 ? rows : 65536), 128, 0, stream>>>(
      static_cast<uint8_t*>(a.out.data), a.out.batch_stride * size, a.out.row_stride * size, a.out.head_stride * size, a.B,
      a.Tq, a.q.heads, a.D * size / 16);
  return cudaGetLastError();
}

cudaError_t launch_attention_tc(const AttentionArgs& a, int num_sms, cudaStream_t stream, const char** why) {
  using namespace atc;
  Args p{};
  if (!encode(&p.q, a.q, a.B, a.Tq, a.D, kRows) || !encode(&p.k, a.k, a.B, a.Tk, a.D, BN) ||
      !encode(&p.v, a.v, a.B, a.Tk, a.D, BN)) {
    *why = "tensor map encoding failed";
    return cudaErrorInvalidValue;
  }
  p.out = a.out.data;
  p.out_bs = a.out.batch_stride;
  p.out_rs = a.out.row_stride;
  p.out_hs = a.out.head_stride;
  p.heads = a.q.heads;
  p.group = a.q.heads / a.k.heads;
  p.kb_shared = (a.q.batch_stride ? 0 : 1) | (a.k.batch_stride ? 0 : 2) | (a.v.batch_stride ? 0 : 4);
  p.Tq = a.Tq;
  p.Tk = a.Tk;
  p.D = a.D;
  p.causal = a.causal;
  p.ntiles = static_cast<int>((static_cast<long long>(a.Tq) + kRows - 1) / kRows);
  p.scale = a.scale;
  p.mask = a.mask;
  p.mask_bs = a.mask_batch_stride;
  p.err = a.err;
  p.wait_limit_ns = a.wait_limit_ns;
  p.withhold = a.withhold;
  const long long work = static_cast<long long>(p.ntiles) * a.q.heads * a.B;
  const int ktiles = static_cast<int>((static_cast<long long>(a.Tk) + BN - 1) / BN);
  int S = 1;
  while (S < kMaxSplit && work * S * 2 <= 2 * num_sms && ktiles >= 2 * S) S *= 2;
  const unsigned w = static_cast<unsigned>(work);
  if (a.mask) return a.D <= 64 ? go<1, true>(p, S, w, stream) : go<2, true>(p, S, w, stream);
  return a.D <= 64 ? go<1, false>(p, S, w, stream) : go<2, false>(p, S, w, stream);
}

}  // namespace gkd
