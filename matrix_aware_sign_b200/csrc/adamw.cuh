// adamw.cuh -- tables and launchers of the AdamW kernels (k_adamw.cu), shared with the host ABI.
#pragma once

#include <stdint.h>

#include "smuon.h"
#include <cuda_runtime.h>

namespace smuon {

constexpr int kAdBlock = 256;  // entries per block, the 8-bit moments' scale group
constexpr int kAdTile = 512;   // two blocks: what a warp steps at once

// One tensor of a launch. States and master are contiguous; W and G may have a row stride.
struct AdTensor {
  void* w;
  const void* g;
  float* master;          // nullable: W's float32 original
  void* m;                // F32, or E4M3 codes
  void* v;                // F32, or E4M3 codes of its square root
  uint8_t* scales;        // 8-bit states: two exponent bytes per block (m, root of v)
  int64_t n, w_ld, g_ld;
  int32_t cols;
  int32_t tile_begin;     // first tile of this tensor in the launch
  float lr_scale, wd;
  uint32_t id;            // index in the call's lists: key word 1 of its rounding stream
  int32_t flags;          // kAd*
};
// a lane's entries (eight, with 8-bit moments sixteen) are aligned vectors in the moments and the master, in W, in G
constexpr int32_t kAdVecState = 1, kAdVecW = 2, kAdVecG = 4, kAdVec = 7;
constexpr int32_t kAdWStride = 8, kAdGStride = 16;  // W, G has a row stride

// What changes from call to call, beside the table (which a plan keeps).
struct AdHyper {
  const int32_t* skip;    // nullable
  const float* d_lr;      // nullable: the learning rate, else lr
  const float* d_gscale;  // nullable: factor on the gradients
  int64_t* d_t;           // nullable {steps taken, arrivals}: the step is d_t[0] + 1, else t
  int64_t t;
  double log_b1, log_b2;  // 1 - b^t = -expm1(t log b)
  float lr, b1, c1, b2, c2, eps;
  float2 one2, c1_2, c2_2, eps2;  // both halves alike: operands of the packed operations
  uint32_t seed;          // key word 0 of the rounding stream, and its ten rounds' values
  uint32_t k0[10];
  int32_t advance;        // last launch of the call: the last CTA to read d_t[0] adds one to it
};

// Tables travel as kernel parameters (32,764 bytes at most) or, with a plan of more than kAdFew tensors, lie in its
// workspace. Launching with the large parameter block costs the host 4 us more and the GPU 2 us more than with the small
// one or a table in memory; the small one is 0.1 to 0.3 us quicker on the GPU than a table in memory with 2 tensors, even
// with 16, and needs no upload.
constexpr int kAdFew = 16, kAdMany = 320;
template <int kCap>
struct AdTable {
  int32_t n_tensors, total_tiles;
  AdTensor t[kCap];
};
// Where to look in a table in memory: the tensor of each 2^shift-th tile, and of the last. It travels with the launch, so
// that finding a tile's tensor takes one load from the table instead of two (and none inside a large tensor).
struct Guide {
  static constexpr int kParts = 64;
  int32_t shift;
  int32_t at[kParts + 1];
};
struct AdDevTable {
  int32_t n_tensors, total_tiles;
  const AdTensor* t;
  Guide guide;
};

enum AdKind { AD_W_F32 = 0, AD_W_BF16 = 1, AD_W_MASTER = 2, AD_G_BF16 = 4, AD_8BIT = 8, AD_KINDS = 16 };

template <class Table>
cudaError_t launch_adamw(int kind, const Table& tb, const AdHyper& h, int sms, cudaStream_t s);

// gradient norm: per-CTA sums of squares; the last CTA to finish takes the norm, the clip factor and the flags
constexpr int kNormTile = 1024;  // entries that a warp squares at once
struct NormTensor {
  const void* g;
  int64_t n, ld;
  int32_t cols;
  int32_t tile_begin;
  int32_t bf16, vec;
};
constexpr int kNormMaxGrid = 592;  // four CTAs an SM (64 registers a thread)
struct NormArgs {
  const NormTensor* t;
  int32_t n_tensors, total_tiles;
  Guide guide;
  double* partials;   // one per CTA
  uint32_t* arrived;  // zero before a launch, and after it
  double max_norm;
  float* out;         // {norm, factor}
  int32_t* skip;      // nullable: 1 where the norm is not finite, else 0
  int32_t* status;    // nullable
};
cudaError_t launch_grad_norm(const NormArgs& a, cudaStream_t s);

// moments from float32 to 8 bits (to8) or back
struct ConvTensor {
  void *m32, *v32, *m8, *v8;
  uint8_t* scales;
  int64_t n;
  int32_t tile_begin;
  int32_t vec;
};
struct ConvTable {
  int32_t n_tensors, total_tiles, to8, pad;
  ConvTensor t[kAdMany];
};
cudaError_t launch_adamw_convert(const ConvTable& tb, cudaStream_t s);

}  // namespace smuon
