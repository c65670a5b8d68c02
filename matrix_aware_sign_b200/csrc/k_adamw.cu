// k_adamw.cu -- the AdamW step for the parameters beside the Muon matrices.
//
//  * k_adamw              one step over many tensors, moments in float32 or in 8 bits
//  * k_grad_sumsq         sums of squares of many gradients
//  * k_grad_norm_finish   their norm, the clip factor made from it, the skip flag
//  * k_adamw_convert      moments from float32 to 8 bits and back
//
// The step is Loshchilov and Hutter's ("Decoupled Weight Decay Regularization"):
//   g = s G,  m' = b1 m + (1 - b1) g,  v' = b2 v + (1 - b2) g^2,  r' = sqrt(v')
//   W' = W - lr (wd W + (m' / (1 - b1^t)) / (r' / sqrt(1 - b2^t) + eps))
// All arithmetic is float32. m', v' and r' are formed with every operation
// rounded on its own (no fused multiply-add), so that any IEEE evaluation of
// the same steps gives the same bits; the 8-bit codes depend on them.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "adamw.cuh"
#include "counter_rng.cuh"

namespace smuon {
namespace {

// ---------------------------------------------------------------- eight entries of a lane
__device__ __forceinline__ void ld256(const void* p, uint32_t (&u)[8]) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
               : "l"(p));
}
__device__ __forceinline__ void st256(void* p, const uint32_t (&u)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
               ::"l"(p), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
               : "memory");
}

__device__ __forceinline__ void ld8(const float* p, float (&x)[8]) {
  uint32_t u[8];
  ld256(p, u);
#pragma unroll
  for (int k = 0; k < 8; ++k) x[k] = __uint_as_float(u[k]);
}
__device__ __forceinline__ void ld8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 w = *reinterpret_cast<const uint4*>(p);
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[2 * k] = __uint_as_float(u[k] << 16);
    x[2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
  }
}
__device__ __forceinline__ void st8(float* p, const float (&x)[8]) {
  uint32_t u[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) u[k] = __float_as_uint(x[k]);
  st256(p, u);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&t);
}
__device__ __forceinline__ void st8(__nv_bfloat16* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
}
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// entry e of a tensor with a row stride
__device__ __forceinline__ int64_t strided(int64_t e, int32_t cols, int64_t ld) {
  const int64_t r = e / cols;
  return r * ld + (e - r * cols);
}

template <class T>
__device__ __forceinline__ void load(const T* p, int64_t e0, int64_t n, int32_t cols, int64_t ld, bool stride, bool vec,
                                     float (&x)[8]) {
  if (vec) {
    ld8(p + (stride ? strided(e0, cols, ld) : e0), x);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      x[k] = e0 + k < n ? to_f32(p[stride ? strided(e0 + k, cols, ld) : e0 + k]) : 0.f;
  }
}
template <class T>
__device__ __forceinline__ void store(T* p, int64_t e0, int64_t n, int32_t cols, int64_t ld, bool stride, bool vec,
                                      const float (&x)[8]) {
  if (vec) {
    st8(p + (stride ? strided(e0, cols, ld) : e0), x);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (e0 + k < n) put(p + (stride ? strided(e0 + k, cols, ld) : e0 + k), x[k]);
  }
}

// ---------------------------------------------------------------- 8-bit states
// A block of 256 values x is held as E4M3 codes (x 2^(127 - byte), below 256 in
// magnitude) and one exponent byte: the exponent field of the largest magnitude
// less 7, 0 for a block of zeros (largest below 2^-119), 255 if it is not finite
// (every value then reads back as NaN). float(byte << 23) is the scale in all
// three cases: 2^(byte - 127), 0 and infinity (times a zero code: NaN).
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

__device__ __forceinline__ void decode8(const uint2 c, float scale, float (&x)[8]) {
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[k >> 1] >> (16 * (k & 1))), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    x[2 * k] = __fmul_rn(f.x, scale);
    x[2 * k + 1] = __fmul_rn(f.y, scale);
  }
}

__device__ __forceinline__ uint2 load_codes(const uint8_t* p, int64_t e0, int64_t n, bool vec) {
  if (vec) return *reinterpret_cast<const uint2*>(p + e0);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (e0 + k < n) w[k >> 2] |= (uint32_t)p[e0 + k] << (8 * (k & 3));
  return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void store_codes(uint8_t* p, int64_t e0, int64_t n, bool vec, const uint2 c) {
  if (vec) {
    *reinterpret_cast<uint2*>(p + e0) = c;
    return;
  }
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (e0 + k < n) p[e0 + k] = (uint8_t)(w[k >> 2] >> (8 * (k & 3)));
}

// exponent byte of the warp's block (all lanes take part)
__device__ __forceinline__ uint32_t block_exponent(const float (&x)[8]) {
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(x[k]) & 0x7fffffffu);  // NaN above infinity above all
  top = __reduce_max_sync(0xffffffffu, top) >> 23;
  return top == 255u ? 255u : (top > 7u ? top - 7u : 0u);
}

// Codes of eight values. kRandom: 16 random bits added below the three mantissa bits that a code keeps,
// then cut there (halves of rnd[4], low first), so that a code's mean is the value: the moments move by
// far less than a code step (a second moment with b2 = 0.999 by 0.05% a step, a code step is 6 to 12%),
// which rounding to nearest would lose every time. Else to nearest.
template <bool kRandom>
__device__ __forceinline__ uint2 encode8(const float (&x)[8], uint32_t byte, const uint4 rnd) {
  if (byte == 0u || byte == 255u) return make_uint2(0u, 0u);
  const float up = __uint_as_float((254u - byte) << 23);
  const uint32_t rw[4] = {rnd.x, rnd.y, rnd.z, rnd.w};
  uint32_t out[2];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float2 y = make_float2(x[2 * k] * up, x[2 * k + 1] * up);
    if (kRandom) {
      y.x = __uint_as_float((__float_as_uint(y.x) + ((rw[k] & 0xffffu) << 4)) & 0xfff00000u);
      y.y = __uint_as_float((__float_as_uint(y.y) + ((rw[k] >> 16) << 4)) & 0xfff00000u);
    }
    const uint32_t two = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
    out[k >> 1] = (k & 1) ? (out[k >> 1] | two << 16) : two;
  }
  return make_uint2(out[0], out[1]);
}

// last tensor whose first block is at or before b; monotonic from `li` on
template <class Table>
__device__ __forceinline__ int tensor_of(const Table& tb, int b, int li) {
  if (li < 0) {
    int lo = 0, hi = tb.n_tensors - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (tb.t[mid].block_begin <= b) lo = mid; else hi = mid - 1;
    }
    return lo;
  }
  while (li + 1 < tb.n_tensors && tb.t[li + 1].block_begin <= b) ++li;
  return li;
}

}  // namespace

// ---------------------------------------------------------------- the step
template <int kKind, int kCap>
__global__ void __launch_bounds__(256) k_adamw(const __grid_constant__ AdTable<kCap> tb, const __grid_constant__ AdHyper h) {
  constexpr bool kMaster = (kKind & 3) == AD_W_MASTER, k8 = (kKind & AD_8BIT) != 0;
  using WT = typename std::conditional<(kKind & 3) == AD_W_F32, float, __nv_bfloat16>::type;
  using GT = typename std::conditional<(kKind & AD_G_BF16) != 0, __nv_bfloat16, float>::type;
  if (h.skip && *h.skip) return;
  const int64_t t = h.d_t ? *h.d_t + 1 : h.t;
  const float lr = h.d_lr ? *h.d_lr : h.lr;
  const float gs = h.d_gscale ? *h.d_gscale : 1.f;
  const float ic1 = -1.f / expm1f((float)((double)t * h.log_b1));         // 1 / (1 - b1^t)
  const float ic2 = rsqrtf(-expm1f((float)((double)t * h.log_b2)));       // 1 / sqrt(1 - b2^t)
  if (h.d_t && h.advance) {  // the last CTA to have read the count steps it
    __syncthreads();
    if (threadIdx.x == 0) {
      __threadfence();
      if (atomicAdd(reinterpret_cast<unsigned long long*>(h.d_t + 1), 1ull) + 1 == gridDim.x) {
        h.d_t[1] = 0;
        h.d_t[0] = t;
      }
    }
  }
  const int lane = threadIdx.x & 31;
  int li = -1;
  for (int b = blockIdx.x * 8 + (threadIdx.x >> 5); b < tb.total_blocks; b += gridDim.x * 8) {
    li = tensor_of(tb, b, li);
    const AdTensor& T = tb.t[li];
    const int64_t n = T.n, blk = b - T.block_begin, e0 = blk * kAdBlock + lane * 8;
    const bool vec = (T.flags & kAdVec) && e0 + 8 <= n;
    const bool ws = T.flags & kAdWStride, gst = T.flags & kAdGStride;
    float g[8], w[8], m[8], v[8];
    load(reinterpret_cast<const GT*>(T.g), e0, n, T.cols, T.g_ld, gst, vec, g);
    if (kMaster) load(T.master, e0, n, T.cols, 0, false, vec, w);
    else load(reinterpret_cast<const WT*>(T.w), e0, n, T.cols, T.w_ld, ws, vec, w);
    if (k8) {
      const uint32_t sc = *reinterpret_cast<const uint16_t*>(T.scales + 2 * blk);
      decode8(load_codes(reinterpret_cast<const uint8_t*>(T.m), e0, n, vec), scale_of(sc & 255u), m);
      decode8(load_codes(reinterpret_cast<const uint8_t*>(T.v), e0, n, vec), scale_of(sc >> 8), v);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = __fmul_rn(v[k], v[k]);  // exact: a code has four significant bits
    } else {
      load(reinterpret_cast<const float*>(T.m), e0, n, T.cols, 0, false, vec, m);
      load(reinterpret_cast<const float*>(T.v), e0, n, T.cols, 0, false, vec, v);
    }
    const float wd = T.wd, step = lr * T.lr_scale;
    float r[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      g[k] = __fmul_rn(gs, g[k]);
      m[k] = __fadd_rn(__fmul_rn(h.b1, m[k]), __fmul_rn(h.c1, g[k]));
      v[k] = __fadd_rn(__fmul_rn(h.b2, v[k]), __fmul_rn(h.c2, __fmul_rn(g[k], g[k])));
      r[k] = __fsqrt_rn(v[k]);
      const float u = (m[k] * ic1) / fmaf(r[k], ic2, h.eps);
      w[k] = fmaf(-step, fmaf(wd, w[k], u), w[k]);
    }
    if (kMaster) store(T.master, e0, n, T.cols, 0, false, vec, w);
    store(reinterpret_cast<WT*>(T.w), e0, n, T.cols, T.w_ld, ws, vec, w);
    if (k8) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (!vec && e0 + k >= n) m[k] = r[k] = 0.f;  // entries past a short last block
      const uint32_t bm = block_exponent(m), br = block_exponent(r);
      const uint64_t grp = (uint64_t)e0 >> 3;
      const uint4 rnd =
          crng::philox4x32_10(make_uint4((uint32_t)grp, (uint32_t)(grp >> 32), (uint32_t)t, 1u), h.seed, T.id);
      store_codes(reinterpret_cast<uint8_t*>(T.m), e0, n, vec, encode8<true>(m, bm, rnd));
      store_codes(reinterpret_cast<uint8_t*>(T.v), e0, n, vec, encode8<true>(r, br, rnd));
      if (lane == 0) *reinterpret_cast<uint16_t*>(T.scales + 2 * blk) = (uint16_t)(bm | br << 8);
    } else {
      store(reinterpret_cast<float*>(T.m), e0, n, T.cols, 0, false, vec, m);
      store(reinterpret_cast<float*>(T.v), e0, n, T.cols, 0, false, vec, v);
    }
  }
}

namespace {
template <int kKind, int kCap>
cudaError_t launch_kind(const AdTable<kCap>& tb, const AdHyper& h, int sms, cudaStream_t s) {
  const int want = (tb.total_blocks + 7) / 8;
  const int grid = want < 1 ? 1 : (want < sms * 8 ? want : sms * 8);
  k_adamw<kKind, kCap><<<grid, 256, 0, s>>>(tb, h);
  return cudaGetLastError();
}
}  // namespace

template <int kCap>
cudaError_t launch_adamw(int kind, const AdTable<kCap>& tb, const AdHyper& h, int sms, cudaStream_t s) {
  switch (kind) {
    case AD_W_F32: return launch_kind<AD_W_F32, kCap>(tb, h, sms, s);
    case AD_W_BF16: return launch_kind<AD_W_BF16, kCap>(tb, h, sms, s);
    case AD_W_MASTER: return launch_kind<AD_W_MASTER, kCap>(tb, h, sms, s);
    case AD_W_F32 | AD_G_BF16: return launch_kind<AD_W_F32 | AD_G_BF16, kCap>(tb, h, sms, s);
    case AD_W_BF16 | AD_G_BF16: return launch_kind<AD_W_BF16 | AD_G_BF16, kCap>(tb, h, sms, s);
    case AD_W_MASTER | AD_G_BF16: return launch_kind<AD_W_MASTER | AD_G_BF16, kCap>(tb, h, sms, s);
    case AD_W_F32 | AD_8BIT: return launch_kind<AD_W_F32 | AD_8BIT, kCap>(tb, h, sms, s);
    case AD_W_BF16 | AD_8BIT: return launch_kind<AD_W_BF16 | AD_8BIT, kCap>(tb, h, sms, s);
    case AD_W_MASTER | AD_8BIT: return launch_kind<AD_W_MASTER | AD_8BIT, kCap>(tb, h, sms, s);
    case AD_W_F32 | AD_G_BF16 | AD_8BIT: return launch_kind<AD_W_F32 | AD_G_BF16 | AD_8BIT, kCap>(tb, h, sms, s);
    case AD_W_BF16 | AD_G_BF16 | AD_8BIT: return launch_kind<AD_W_BF16 | AD_G_BF16 | AD_8BIT, kCap>(tb, h, sms, s);
    case AD_W_MASTER | AD_G_BF16 | AD_8BIT: return launch_kind<AD_W_MASTER | AD_G_BF16 | AD_8BIT, kCap>(tb, h, sms, s);
    default: return cudaErrorInvalidValue;
  }
}
template cudaError_t launch_adamw<kAdFew>(int, const AdTable<kAdFew>&, const AdHyper&, int, cudaStream_t);
template cudaError_t launch_adamw<kAdMany>(int, const AdTable<kAdMany>&, const AdHyper&, int, cudaStream_t);

// ---------------------------------------------------------------- gradient norm
// Sum of squares of a lane's eight entries in float32, added up in float64 in a fixed order. Where the
// float32 sum leaves [2^-90, 2^120] (squares that underflow or overflow, NaN, zeros) it is formed in
// float64 instead, so every finite gradient has its norm.
__global__ void __launch_bounds__(256) k_grad_sumsq(const __grid_constant__ NormTable tb) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  double acc = 0.0;
  int li = -1;
  for (int b = blockIdx.x * 8 + warp; b < tb.total_blocks; b += gridDim.x * 8) {
    li = tensor_of(tb, b, li);
    const NormTensor& T = tb.t[li];
    const int64_t n = T.n, e0 = (int64_t)(b - T.block_begin) * kAdBlock + lane * 8;
    const bool vec = T.vec && e0 + 8 <= n, st = T.ld != T.cols;
    float g[8];
    if (T.bf16) load(reinterpret_cast<const __nv_bfloat16*>(T.g), e0, n, T.cols, T.ld, st, vec, g);
    else load(reinterpret_cast<const float*>(T.g), e0, n, T.cols, T.ld, st, vec, g);
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s = fmaf(g[k], g[k], s);
    double d = (double)s;
    if (!(s >= 0x1p-90f && s <= 0x1p120f)) {
      d = 0.0;
#pragma unroll
      for (int k = 0; k < 8; ++k) d = fma((double)g[k], (double)g[k], d);
    }
    acc += d;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  __shared__ double part[8];
  if (lane == 0) part[warp] = acc;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0.0;
    for (int k = 0; k < 8; ++k) s += part[k];
    tb.partials[blockIdx.x] = s;
  }
}

__global__ void __launch_bounds__(256) k_grad_norm_finish(const __grid_constant__ NormOut o) {
  __shared__ double part[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  double acc = 0.0;
  for (int i = threadIdx.x; i < o.n_partials; i += 256) acc += o.partials[i];
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, k);
  if (lane == 0) part[warp] = acc;
  __syncthreads();
  if (threadIdx.x) return;
  double s = 0.0;
  for (int k = 0; k < 8; ++k) s += part[k];
  const double norm = sqrt(s);
  const float f = (float)norm;
  const bool bad = !(f <= 3.402823466e38f);
  o.out[0] = f;
  o.out[1] = bad ? 0.f : (float)fmin(1.0, o.max_norm / (norm + 1e-6));
  if (o.skip) *o.skip = bad;
  if (o.status && bad) atomicOr(o.status, SMUON_DEV_NONFINITE_NORM);
}

int norm_grid(int total_blocks) {
  const int want = (total_blocks + 7) / 8;
  return want < 1 ? 1 : (want < kNormMaxGrid ? want : kNormMaxGrid);
}

cudaError_t launch_grad_norm(const NormTable& tb, cudaStream_t s) {
  k_grad_sumsq<<<norm_grid(tb.total_blocks), 256, 0, s>>>(tb);
  return cudaGetLastError();
}

cudaError_t launch_grad_norm_finish(const NormOut& o, cudaStream_t s) {
  k_grad_norm_finish<<<1, 256, 0, s>>>(o);
  return cudaGetLastError();
}

// ---------------------------------------------------------------- conversion
__global__ void __launch_bounds__(256) k_adamw_convert(const __grid_constant__ ConvTable tb) {
  const int lane = threadIdx.x & 31;
  int li = -1;
  for (int b = blockIdx.x * 8 + (threadIdx.x >> 5); b < tb.total_blocks; b += gridDim.x * 8) {
    li = tensor_of(tb, b, li);
    const ConvTensor& T = tb.t[li];
    const int64_t n = T.n, blk = b - T.block_begin, e0 = blk * kAdBlock + lane * 8;
    const bool vec = T.vec && e0 + 8 <= n;
    float m[8], r[8];
    if (tb.to8) {
      load(reinterpret_cast<const float*>(T.m32), e0, n, 1, 1, false, vec, m);
      load(reinterpret_cast<const float*>(T.v32), e0, n, 1, 1, false, vec, r);
#pragma unroll
      for (int k = 0; k < 8; ++k) r[k] = __fsqrt_rn(r[k]);
      const uint32_t bm = block_exponent(m), br = block_exponent(r);
      store_codes(reinterpret_cast<uint8_t*>(T.m8), e0, n, vec, encode8<false>(m, bm, make_uint4(0, 0, 0, 0)));
      store_codes(reinterpret_cast<uint8_t*>(T.v8), e0, n, vec, encode8<false>(r, br, make_uint4(0, 0, 0, 0)));
      if (lane == 0) *reinterpret_cast<uint16_t*>(T.scales + 2 * blk) = (uint16_t)(bm | br << 8);
    } else {
      const uint32_t sc = *reinterpret_cast<const uint16_t*>(T.scales + 2 * blk);
      decode8(load_codes(reinterpret_cast<const uint8_t*>(T.m8), e0, n, vec), scale_of(sc & 255u), m);
      decode8(load_codes(reinterpret_cast<const uint8_t*>(T.v8), e0, n, vec), scale_of(sc >> 8), r);
#pragma unroll
      for (int k = 0; k < 8; ++k) r[k] = __fmul_rn(r[k], r[k]);
      store(reinterpret_cast<float*>(T.m32), e0, n, 1, 1, false, vec, m);
      store(reinterpret_cast<float*>(T.v32), e0, n, 1, 1, false, vec, r);
    }
  }
}

cudaError_t launch_adamw_convert(const ConvTable& tb, int sms, cudaStream_t s) {
  const int want = (tb.total_blocks + 7) / 8;
  const int grid = want < 1 ? 1 : (want < sms * 8 ? want : sms * 8);
  k_adamw_convert<<<grid, 256, 0, s>>>(tb);
  return cudaGetLastError();
}

}  // namespace smuon
