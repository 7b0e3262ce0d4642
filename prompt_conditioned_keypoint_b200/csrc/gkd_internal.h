// Internal launch interface between the C-ABI layer (api.cu) and the kernels.
// Every launcher assumes its arguments were validated by the caller and only
// enqueues work on `stream`; it returns the CUDA launch status.
#pragma once
#include <atomic>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace gkd {

// Device error word bits (written by kernels, read by gkd_check_device_error).
enum : unsigned {
  kErrTimeout = 1u << 0,   // a bounded wait ran out
  kErrBounds = 1u << 1,    // a bounds or placement check fired (the kernel did no work)
};

// Test hooks for the forced-timeout path (host-set, consumed by the next launch).
enum : unsigned {
  kDbgSkipProducerArrive = 1u << 0,   // upsample producers never signal their first stage
};

cudaError_t launch_norm(const float* rows, const uint8_t* mask, long long nrows, int C, float eps,
                        bool out_bf16, void* out, cudaStream_t stream);

cudaError_t launch_norm_fuse(const float* rows, const uint8_t* mask, int Bk, int M, int K, int C, float eps,
                             bool out_bf16, void* out, uint8_t* out_mask, cudaStream_t stream);

// Image preprocessing of B boxes of one image and the ROI -> image coordinate map (preprocess.cu).
cudaError_t launch_preprocess(const uint8_t* img, int H, int W, const float* boxes, int B, int canvas, float* out,
                              cudaStream_t stream);
cudaError_t launch_roi_to_image(const float* xy, const float* boxes, int B, int K, int canvas, float* out,
                                cudaStream_t stream);

cudaError_t launch_fuse_decode(const float* heat, const uint8_t* mask, long long mask_batch_stride,
                               int B, int M, int K, int H, int W, float* fused, float* xy, float* score,
                               int32_t* idx, uint8_t* valid, cudaStream_t stream);

// keys non-null: decode mode (no heatmap; one peak key per (crop, row) merged into keys)
cudaError_t launch_heatmap_f32(const float* feat, int B, int h, int w, int C, const float* kern,
                               long long kern_batch_stride, const uint8_t* mask, long long mask_batch_stride,
                               int M, int K, float* heat, unsigned long long* keys, int num_sms,
                               cudaStream_t stream);

// Turns peak keys [B][K] into idx / xy / score / valid (decode fused into the heatmap kernels).
cudaError_t launch_finalize_keys(const unsigned long long* keys, const uint8_t* mask, long long mask_batch_stride,
                                 int B, int M, int K, int H, int W, float* xy, float* score, int32_t* idx,
                                 uint8_t* valid, cudaStream_t stream);

constexpr int kKernMaps = 16;   // kernel-row boxes of 8, 16, ..., 128 rows

struct HeatmapTcArgs {
  CUtensorMap tmap_feat;                 // feature slabs: fp32 {32, w, h, C/32, B} or {C, w, h, B}
  CUtensorMap tmap_kern[kKernMaps];      // kernel rows {C, K, M, Bk}, box {64, 8 (i + 1), 1, 1}
  const uint8_t* mask;
  long long mask_batch_stride;
  float* heat;                           // heatmaps (heatmap mode), unused in decode mode
  unsigned long long* dec_keys;          // decode mode: per (crop, row) peak key, zeroed before launch; else null
  int B, h, w, C, M, K;
  int feat_bf16;
  int feat_5d;               // fp32 slab as one 5-D box (C % 32 == 0), else two 4-D boxes
  int kern_shared;           // kernels shared by all crops (batch stride 0)
  unsigned* err;             // device error word
  unsigned long long wait_limit_ns;
  unsigned debug_flags;
};

// Encodes the tensor maps and launches the persistent tcgen05 kernel.
cudaError_t launch_heatmap_tc(HeatmapTcArgs& a, const void* feat, const void* kern,
                              long long kern_batch_stride, int num_sms, cudaStream_t stream,
                              const char** why);

// Contract-then-upsample variant (contract_tc.cu).
struct ContractArgs {
  CUtensorMap tmap_feat;                 // features as [B*h*w][C], box {32 (fp32) or 64 (bf16), 128}
  CUtensorMap tmap_kern[kKernMaps];      // kernel rows, as for HeatmapTcArgs
  const uint8_t* mask;
  long long mask_batch_stride;
  float* G;                              // [B][M][K][h*w] fp32 contraction on the source grid (scratch)
  int B, h, w, C, M, K;
  int feat_bf16;
  int kern_shared;
  unsigned* err;
  unsigned long long wait_limit_ns;
};

cudaError_t launch_contract_first(ContractArgs& a, const void* feat, const void* kern, long long kern_batch_stride,
                                  float* heat, cudaStream_t stream, const char** why);

// Gaussian prototype pooling on the tensor cores (pool_tc.cu).
struct PoolTcArgs {
  CUtensorMap tmap;                      // support features as {C, h*w, B} fp32, box {32, 32, 1}
  const float* kpts;                     // [B][K][2]
  const uint8_t* kmask;                  // [B][K]
  float* proto;
  long long proto_bs;
  int h, w, C, K;
  int N;                                 // channels per CTA (32..256, a multiple of 32)
  float sigma, stride;
  unsigned* err;
  unsigned long long wait_limit_ns;
};

cudaError_t launch_pool_tc(const float* support, int B, int h, int w, int C, const float* kpts,
                           const uint8_t* kmask, int K, float sigma, float stride, float* proto,
                           long long proto_batch_stride, unsigned* err, unsigned long long wait_limit_ns,
                           int num_sms, cudaStream_t stream, const char** why);

// ---------------------------------------------------------------------------
// Operators of the transformer blocks (gkd_blocks.h)
// ---------------------------------------------------------------------------
// Allows a kernel its dynamic shared memory (and clusters of 16 CTAs), once per kernel and device.
template <auto* Kernel>
cudaError_t allow_smem(size_t bytes, bool cluster16 = false) {
  static std::atomic<unsigned long long> done{0};    // one bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  if (e == cudaSuccess && cluster16) e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// Launches clusters of S CTAs along x.
template <typename... Params, typename... Given>
cudaError_t launch_cluster(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, int S, cudaStream_t stream,
                           const Given&... given) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = S;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(given)...);
}

// Tensor map of a [rows][cols] tensor whose rows are `stride` elements apart; boxes of 128 (64) bytes a
// row, 128B- (64B-)swizzled.
bool encode_rows(CUtensorMap* m, bool bf16, const void* base, long long cols, long long rows, long long stride,
                 int box_cols, int box_rows);

struct LinearArgs {
  const void* x;
  const void* weight;        // [Cout][Cin]
  const float* bias;         // [Cout] or null
  const float* scale;        // [Cout] or null
  const void* residual;      // of the output's type, or null
  void* out;
  long long x_stride, residual_stride, out_stride;   // elements between rows
  int T, Cin, Cout, act;
  bool out_bf16;
  bool withhold;             // test hook: the first stage of every CTA is not handed to the products
  unsigned* err;
  unsigned long long wait_limit_ns;
};
cudaError_t launch_linear_f32(const LinearArgs& a, int num_sms, cudaStream_t stream, const char** why);
cudaError_t launch_linear_tc(const LinearArgs& a, int num_sms, cudaStream_t stream, const char** why);   // bf16 operands

struct RopeSide {            // q or k
  const void* in;
  void* out;
  long long in_bs, in_rs, in_hs, out_bs, out_rs, out_hs;   // elements between batches, rows, heads
  int heads;                 // 0: no such side
  const float* weight;       // [D] or null (no norm)
};
struct RopeArgs {
  RopeSide side[2];
  int B, T, D, axes, pairs, interleaved;
  float eps;
  const float* pos;          // [T][axes] per batch
  long long pos_bs;
  const uint8_t* pair_axis;
  const float* pair_freq;
  int tok, fold;             // set by the launcher: rows per CTA, first step of the sum over a head's lanes
  unsigned heads_magic;      // to divide by the heads of a row
  float inv_d;
};
cudaError_t launch_qk_norm_rope(RopeArgs& g, bool bf16, int num_sms, cudaStream_t stream);

struct HeadsView {           // element (b, t, h, i) at data + b batch_stride + t row_stride + h head_stride + i
  void* data;
  long long batch_stride, row_stride, head_stride;
  int heads;
};
// A row's weights are 2^(s f - m f) for its scores s and the largest of them m, by one fused multiply-add on the rounded
// m f, with f = c = scale log2(e). That rounding, common to the row's weights, takes them out of the exponent's range
// once |m c| passes 2^31. But from |m| pow2 = 2^30 on, pow2 the power of two below c, the scores next to m are 2^6 and
// more away from it (in units of 1 / pow2): whatever is below m has no weight, and f = pow2, with which m f is exact,
// serves as well. (factor and offset of a row: blocks_common.cuh. Formed here, since code in the kernels that ran once
// took 0.2 of 13 us of a one-row call.)
struct ScoreScale {
  float c, pow2, far;        // far = 2^30 / pow2
};
ScoreScale score_scale(float scale);

struct AttentionArgs {
  HeadsView q, k, v, out;
  int B, Tq, Tk, D;
  bool causal;
  bool withhold;             // test hook: the first tile of keys of every CTA is not handed to the products
  ScoreScale scale;
  const uint8_t* mask;       // batch b's [Tk] at mask + b * mask_batch_stride, or null
  long long mask_batch_stride;
  unsigned* err;
  unsigned long long wait_limit_ns;
};
cudaError_t launch_attention_none(const AttentionArgs& a, int size, cudaStream_t stream);   // Tk = 0: zeros
cudaError_t launch_attention_f32(const AttentionArgs& a, int num_sms, cudaStream_t stream);
cudaError_t launch_attention_tc(const AttentionArgs& a, int num_sms, cudaStream_t stream, const char** why);   // bf16

// cuTensorMapEncodeTiled resolved through the runtime's driver entry point.
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn get_encode_tiled();

}  // namespace gkd
