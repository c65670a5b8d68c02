// k_adamw.cu -- the AdamW step for the parameters beside the Muon matrices.
//
//  * k_adamw32, k_adamw8  one step over many tensors, moments in float32 or in 8 bits
//  * k_grad_norm          norm of many gradients, the clip factor made from it, the skip flag
//  * k_adamw_convert      moments from float32 to 8 bits and back
//
// The step is Loshchilov and Hutter's ("Decoupled Weight Decay Regularization"):
//   g = s G,  m' = b1 m + (1 - b1) g,  v' = b2 v + (1 - b2) g^2,  r' = sqrt(v')
//   W' = W - lr (wd W + (m' / (1 - b1^t)) / (r' / sqrt(1 - b2^t) + eps))
// All arithmetic is float32. m', v' and r' are formed with every operation
// rounded on its own (no fused multiply-add), so that any IEEE evaluation of
// the same steps gives the same bits; the 8-bit codes depend on them.
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "adamw.cuh"
#include "counter_rng.cuh"

namespace smuon {
namespace {

// ---------------------------------------------------------------- launches
// These kernels are launched so that they may begin while the kernel before them in the stream ends (programmatic
// dependent launch): the next one's CTAs are let in at once, and memory is touched only after what came before is done.
// A chain of small calls takes one launch latency less each.
__device__ __forceinline__ void follow_previous() {
  asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
}
template <class... P, class... A>
cudaError_t launch(void (*kernel)(P...), int grid, int block, int smem, cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

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
// bf16 halves to float32 by the mixed-precision add, which leaves the integer pipe to the codes and random bits
__device__ __forceinline__ float add_bf16(uint16_t a) {
  float d;
  asm("add.f32.bf16 %0, %1, %2;" : "=f"(d) : "h"(a), "f"(-0.f));
  return d;
}
__device__ __forceinline__ void ld8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 w = *reinterpret_cast<const uint4*>(p);
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[2 * k] = add_bf16((uint16_t)u[k]);
    x[2 * k + 1] = add_bf16((uint16_t)(u[k] >> 16));
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

// element offsets of entries e, e + 32, e + 64, ... (cols 0: no row stride)
struct Places {
  int64_t at, ld;
  int32_t col, cols;
  __device__ __forceinline__ Places(int64_t e, int32_t cols_, int64_t ld_) : at(e), ld(ld_), col(0), cols(cols_) {
    if (cols) {
      const int64_t r = e / cols;
      col = (int32_t)(e - r * cols);
      at = r * ld + col;
    }
  }
  __device__ __forceinline__ int64_t take() {
    const int64_t here = at;
    at += 32;
    if (cols) {
      col += 32;
      while (col >= cols) {
        col -= cols;
        at += ld - cols;
      }
    }
    return here;
  }
};

// eight entries from entry e0 on, which lies at element `at` (all eight in one row, where there are eight)
template <class T>
__device__ __forceinline__ void load(const T* p, int64_t e0, int64_t n, int64_t at, bool vec, float (&x)[8]) {
  if (vec) {
    ld8(p + at, x);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = e0 + k < n ? to_f32(p[at + k]) : 0.f;
  }
}
template <class T>
__device__ __forceinline__ void store(T* p, int64_t e0, int64_t n, int64_t at, bool vec, const float (&x)[8]) {
  if (vec) {
    st8(p + at, x);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (e0 + k < n) put(p + at + k, x[k]);
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

__device__ __forceinline__ float decode1(uint8_t code) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(code, __NV_E4M3)));
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

// A root that is not zero keeps at least the smallest code. Cut to zero beside a first moment that is held, it would leave
// eps alone under that moment: a step of a thousand learning rates where a gradient is 1e-5 of its block's largest. x:
// the roots, or their squares; few lanes have a code of zero to look at (zero_codes).
template <int N>
__device__ __forceinline__ void keep_roots(const float (&x)[N], uint32_t (&codes)[N / 4]) {
#pragma unroll
  for (int k = 0; k < N; ++k)
    if (x[k] > 0.f && !(codes[k >> 2] & 0x7fu << (8 * (k & 3)))) codes[k >> 2] |= 1u << (8 * (k & 3));
}
// high bits where one of four codes (none of them negative) is zero, or stands behind one that is
__device__ __forceinline__ uint32_t zero_codes(uint32_t codes) { return codes - 0x01010101u; }

// Codes of eight values. kRandom: a code goes up with the probability of its remainder, so that its mean is the value: the
// moments move by far less than a code step (a second moment with b2 = 0.999 by 0.05% a step, a code step is 6 to 12%, and
// as much as the value itself at the smallest codes), which rounding to nearest would lose every time. The values are
// brought to 2^-120 times what the codes stand for, where float32's subnormal numbers begin with the codes' (below 2^-6,
// 2^-9 apart): a pattern's sign bit and bits 20 to 26 are then the code at every size, and 16 random bits (halves of
// rnd[4], low first) added at bit 4 carry into it. Else to nearest.
template <bool kRandom, bool kRoot>
__device__ __forceinline__ uint2 encode8(const float (&x)[8], uint32_t byte, const uint4 rnd) {
  if (byte == 0u || byte == 255u) return make_uint2(0u, 0u);
  const float up = __uint_as_float((254u - byte) << 23);
  const uint32_t rw[4] = {rnd.x, rnd.y, rnd.z, rnd.w};
  uint32_t out[2] = {0u, 0u};
#pragma unroll
  for (int k = 0; k < 8; k += 2) {
    const float2 y = make_float2(x[k] * up, x[k + 1] * up);
    uint32_t two;
    if (kRandom) {
      const uint32_t a = __float_as_uint(y.x * 0x1p-120f) + ((rw[k >> 1] & 0xffffu) << 4);
      const uint32_t b = __float_as_uint(y.y * 0x1p-120f) + ((rw[k >> 1] >> 16) << 4);
      two = (a >> 24 & 0x80u) | (a >> 20 & 0x7fu) | (b >> 16 & 0x8000u) | (b >> 12 & 0x7f00u);
    } else {
      two = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
    }
    out[k >> 2] |= two << (8 * (k & 2));
  }
  if (kRoot && ((zero_codes(out[0]) | zero_codes(out[1])) & 0x80808080u)) keep_roots(x, out);
  return make_uint2(out[0], out[1]);
}

// last tensor that begins at or before tile b; li: one known to. Binary in a table of kernel parameters
template <class Table>
__device__ __forceinline__ int tensor_of(const Table& tb, int b, int li) {
  int lo = li, hi = tb.n_tensors - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tb.t[mid].tile_begin <= b) lo = mid; else hi = mid - 1;
  }
  return lo;
}
// in a table in memory: between two places of the guide, the warp looking at 32 tensors at once
template <class Tensor>
__device__ __forceinline__ int tensor_of_warp(const Tensor* t, const Guide& guide, int b) {
  const int part = b >> guide.shift, lane = threadIdx.x & 31;
  int li = guide.at[part];
  for (int len = guide.at[part + 1] - li + 1; len > 1;) {
    const int step = (len + 31) >> 5, at = li + lane * step;
    const bool ok = lane * step < len && t[at].tile_begin <= b;
    const int k = __popc(__ballot_sync(0xffffffffu, ok)) - 1;
    li += k * step;
    len = min(step, len - k * step);
  }
  return li;
}
__device__ __forceinline__ int tensor_of(const AdDevTable& tb, int b, int) { return tensor_of_warp(tb.t, tb.guide, b); }

// A warp's walk over the tiles of a launch.
template <class Table>
struct Walk {
  int b, stop;          // tile, and where the walk stops
  int li = 0, end = 0;  // the tile's tensor, and the first tile after that tensor
  int which = 1;        // of the warp's two places in shared memory for tensors of a table in memory, taken in turn (0 first)
  __device__ __forceinline__ Walk(int first, int after) : b(first), stop(after) {}
  __device__ __forceinline__ bool seek(const Table& tb, AdTensor* slots) {
    if (b >= stop) return false;
    if (b >= end) {
      li = tensor_of(tb, b, li);
      end = li + 1 < tb.n_tensors ? tb.t[li + 1].tile_begin : tb.total_tiles;
      if constexpr (std::is_same<Table, AdDevTable>::value) {
        which ^= 1;
        const int lane = threadIdx.x & 31;
        __syncwarp();  // every lane is done with the tensor that lay there
        if (lane < (int)(sizeof(AdTensor) / 4))
          reinterpret_cast<uint32_t*>(slots + which)[lane] = reinterpret_cast<const uint32_t*>(tb.t + li)[lane];
        __syncwarp();
      }
    }
    return true;
  }
};
// tensor `li` of a table: in the kernel parameters, or the copy in shared memory
template <class Table>
__device__ __forceinline__ const AdTensor& tensor_at(const Table& tb, int li, const AdTensor* slots, int which) {
  if constexpr (std::is_same<Table, AdDevTable>::value) return slots[which];
  else return tb.t[li];
}

// ---------------------------------------------------------------- the step
// per-call numbers, the same for every entry
struct Consts {
  float b1, c1, b2, c2, eps, gs, lr, ic1, ic2;  // ic1 = 1 / (1 - b1^t), ic2 = 1 / sqrt(1 - b2^t)
  uint32_t t, seed;
};

template <int kKind>
struct Kind {
  static constexpr bool master = (kKind & 3) == AD_W_MASTER, eight = (kKind & AD_8BIT) != 0;
  using W = typename std::conditional<(kKind & 3) == AD_W_F32, float, __nv_bfloat16>::type;
  using G = typename std::conditional<(kKind & AD_G_BF16) != 0, __nv_bfloat16, float>::type;
};

__device__ __forceinline__ float rcp_approx(float x) {
  float d;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(x));
  return d;
}

// W' from m' and r' = sqrt(v'); the reciprocal is an approximation within a unit in the last place: the direction is a
// small part of W, which is rounded to 2^-24 of itself afterwards
__device__ __forceinline__ float weight_step(float w, float m, float r, float decay, float step, const Consts& c) {
  return fmaf(-step, m * rcp_approx(fmaf(r, c.ic2, c.eps)), fmaf(-decay, w, w));  // step = lr / (1 - b1^t), decay = lr wd
}

__device__ __forceinline__ float sqrt_approx(float v) {
  float r;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// A block of any alignment or stride, float32 moments: the lanes' entries lie side by side, so the accesses coalesce.
template <int kKind>
__device__ __noinline__ void step_block32(const AdTensor& T, int64_t blk, int lane, const Consts& c) {
  using K = Kind<kKind>;
  using WT = typename K::W;
  using GT = typename K::G;
  const float lr = c.lr * T.lr_scale, step = lr * c.ic1, decay = lr * T.wd;
  const int64_t first = blk * kAdBlock + lane;
  const int left = (int)min(T.n - first, (int64_t)kAdBlock);
  float* const pm = reinterpret_cast<float*>(T.m) + first;
  float* const pv = reinterpret_cast<float*>(T.v) + first;
  Places wp(first, T.flags & kAdWStride ? T.cols : 0, T.w_ld), gp(first, T.flags & kAdGStride ? T.cols : 0, T.g_ld);
#pragma unroll 1
  for (int k0 = 0; k0 < 8; k0 += 4) {  // four entries' loads before the first use
    float w[4], g[4], m[4], v[4];
    WT* to[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int d = 32 * (k0 + j);
      to[j] = reinterpret_cast<WT*>(T.w) + wp.take();
      const GT* const from = reinterpret_cast<const GT*>(T.g) + gp.take();
      w[j] = g[j] = m[j] = v[j] = 0.f;
      if (d < left) {
        g[j] = to_f32(*from);
        w[j] = K::master ? T.master[first + d] : to_f32(*to[j]);
        m[j] = pm[d];
        v[j] = pv[d];
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int d = 32 * (k0 + j);
      if (d < left) {
        const float x = __fmul_rn(c.gs, g[j]);
        m[j] = __fadd_rn(__fmul_rn(c.b1, m[j]), __fmul_rn(c.c1, x));
        v[j] = __fadd_rn(__fmul_rn(c.b2, v[j]), __fmul_rn(c.c2, __fmul_rn(x, x)));
        w[j] = weight_step(w[j], m[j], __fsqrt_rn(v[j]), decay, step, c);
        if (K::master) T.master[first + d] = w[j];
        put(to[j], w[j]);
        pm[d] = m[j];
        pv[d] = v[j];
      }
    }
  }
}

// A block with 8-bit moments of any alignment, or whose scales leave the range of the fast form, or whose values are not
// finite: entry by entry.
template <int kKind>
__device__ __noinline__ void step_block8(const AdTensor& T, int64_t blk, int lane, const Consts& c) {
  using K = Kind<kKind>;
  using WT = typename K::W;
  using GT = typename K::G;
  const int64_t n = T.n, first = blk * kAdBlock + lane * 8;
  const bool ws = T.flags & kAdWStride, gst = T.flags & kAdGStride;
  const float lr = c.lr * T.lr_scale, step = lr * c.ic1, decay = lr * T.wd;
  const uint32_t sc = *reinterpret_cast<const uint16_t*>(T.scales + 2 * blk);
  float m[8], r[8];
#pragma unroll
  for (int k0 = 0; k0 < 8; k0 += 4) {  // four entries' loads before the first use
    float w[4], g[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = k0 + j;
      const int64_t e = first + k;
      w[j] = g[j] = m[k] = r[k] = 0.f;
      if (e < n) {
        g[j] = to_f32(reinterpret_cast<const GT*>(T.g)[gst ? strided(e, T.cols, T.g_ld) : e]);
        w[j] = K::master ? T.master[e] : to_f32(reinterpret_cast<const WT*>(T.w)[ws ? strided(e, T.cols, T.w_ld) : e]);
        m[k] = decode1(reinterpret_cast<const uint8_t*>(T.m)[e]);
        r[k] = decode1(reinterpret_cast<const uint8_t*>(T.v)[e]);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = k0 + j;
      const int64_t e = first + k;
      m[k] = __fmul_rn(m[k], scale_of(sc & 255u));
      r[k] = __fmul_rn(r[k], scale_of(sc >> 8));
      const float x = __fmul_rn(c.gs, g[j]);
      m[k] = __fadd_rn(__fmul_rn(c.b1, m[k]), __fmul_rn(c.c1, x));
      r[k] = __fsqrt_rn(__fadd_rn(__fmul_rn(c.b2, __fmul_rn(r[k], r[k])), __fmul_rn(c.c2, __fmul_rn(x, x))));
      if (e < n) {
        w[j] = weight_step(w[j], m[k], r[k], decay, step, c);
        if (K::master) T.master[e] = w[j];
        put(reinterpret_cast<WT*>(T.w) + (ws ? strided(e, T.cols, T.w_ld) : e), w[j]);
      } else {
        m[k] = r[k] = 0.f;  // past a short last block
      }
    }
  }
  const uint32_t bm = block_exponent(m), br = block_exponent(r);
  const uint64_t grp = (uint64_t)first >> 3;
  const uint4 rnd = crng::philox4x32_10(make_uint4((uint32_t)grp, (uint32_t)(grp >> 32), c.t, 1u), c.seed, T.id);
  store_codes(reinterpret_cast<uint8_t*>(T.m), first, n, false, encode8<true, false>(m, bm, rnd));
  store_codes(reinterpret_cast<uint8_t*>(T.v), first, n, false, encode8<true, true>(r, br, rnd));
  if (lane == 0) *reinterpret_cast<uint16_t*>(T.scales + 2 * blk) = (uint16_t)(bm | br << 8);
}

// Eight entries of a lane, float32 moments, vector operands.
template <int kKind>
__device__ __forceinline__ void step_lane32(const AdTensor& T, int64_t e0, const Consts& c) {
  using K = Kind<kKind>;
  using WT = typename K::W;
  using GT = typename K::G;
  const int64_t wo = T.flags & kAdWStride ? strided(e0, T.cols, T.w_ld) : e0;
  const int64_t go = T.flags & kAdGStride ? strided(e0, T.cols, T.g_ld) : e0;
  float g[8], w[8], m[8], v[8];
  ld8(reinterpret_cast<const GT*>(T.g) + go, g);
  if (K::master) ld8(T.master + e0, w);
  else ld8(reinterpret_cast<const WT*>(T.w) + wo, w);
  ld8(reinterpret_cast<const float*>(T.m) + e0, m);
  ld8(reinterpret_cast<const float*>(T.v) + e0, v);
  const float lr = c.lr * T.lr_scale, step = lr * c.ic1, decay = lr * T.wd;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    g[k] = __fmul_rn(c.gs, g[k]);
    m[k] = __fadd_rn(__fmul_rn(c.b1, m[k]), __fmul_rn(c.c1, g[k]));
    v[k] = __fadd_rn(__fmul_rn(c.b2, v[k]), __fmul_rn(c.c2, __fmul_rn(g[k], g[k])));
    w[k] = weight_step(w[k], m[k], __fsqrt_rn(v[k]), decay, step, c);
  }
  if (K::master) st8(T.master + e0, w);
  st8(reinterpret_cast<WT*>(T.w) + wo, w);
  st8(reinterpret_cast<float*>(T.m) + e0, m);
  st8(reinterpret_cast<float*>(T.v) + e0, v);
}

// two float32 numbers in one register pair: one instruction for both, each rounded on its own as ever
struct F2 {
  unsigned long long x;
};
__device__ __forceinline__ F2 two(float a, float b) {
  F2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d.x) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ F2 both(float a) { return two(a, a); }
__device__ __forceinline__ void split(F2 a, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a.x));
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.x) : "l"(a.x), "l"(b.x));
  return d;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.x) : "l"(a.x), "l"(b.x), "l"(c.x));
  return d;
}
// a + b as a 1 + b, with a one that the assembler does not know to be one: it contracts mul.rn.f32x2 and add.rn.f32x2
// into a single rounding (with -fmad=false, too), and the moments need both
__device__ __forceinline__ F2 add2(F2 a, F2 b, float2 one) { return fma2(a, two(one.x, one.y), b); }
// two codes (in the low half) to their values without scale
__device__ __forceinline__ F2 values_of(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return two(f.x, f.y);
}
// codes of four entries from the patterns of encode8 with their random bits added; sign: a code's sign bits, where it has any
__device__ __forceinline__ uint32_t codes_of(const uint32_t (&p)[4], uint32_t sign) {
  constexpr uint32_t even = 0x00ff00ffu;  // entries 0 and 2 of the packed four
  const uint32_t x = __byte_perm(p[0], p[2], 0x7632), y = __byte_perm(p[1], p[3], 0x7632);
  return ((x >> 4) & even) | ((y << 4) & ~even) | ((((x >> 8) & even) | (y & ~even)) & sign);
}

// sixteen consecutive entries as loaded, and pairs of them as float32
template <class E>
struct Raw16;
template <>
struct Raw16<float> {
  uint32_t lo[8], hi[8];
  __device__ __forceinline__ void from(const char* p) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint4 x = reinterpret_cast<const uint4*>(p)[k];
      uint32_t* u = k < 2 ? lo + 4 * k : hi + 4 * k - 8;
      u[0] = x.x; u[1] = x.y; u[2] = x.z; u[3] = x.w;
    }
  }
  __device__ __forceinline__ void store(float* p) const { st256(p, lo); st256(p + 8, hi); }
  __device__ __forceinline__ F2 pair(int k) const {
    const uint32_t* u = k < 8 ? lo + k : hi + k - 8;
    return two(__uint_as_float(u[0]), __uint_as_float(u[1]));
  }
  __device__ __forceinline__ void put(int k, float a, float b) {
    uint32_t* u = k < 8 ? lo + k : hi + k - 8;
    u[0] = __float_as_uint(a);
    u[1] = __float_as_uint(b);
  }
};
template <>
struct Raw16<__nv_bfloat16> {
  uint32_t u[8];
  __device__ __forceinline__ void from(const char* p) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint4 x = reinterpret_cast<const uint4*>(p)[k];
      u[4 * k] = x.x; u[4 * k + 1] = x.y; u[4 * k + 2] = x.z; u[4 * k + 3] = x.w;
    }
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { st256(p, u); }
  __device__ __forceinline__ F2 pair(int k) const {
    return two(add_bf16((uint16_t)u[k >> 1]), add_bf16((uint16_t)(u[k >> 1] >> 16)));
  }
  __device__ __forceinline__ void put(int k, float a, float b) { u[k >> 1] = pack2(a, b); }
};

// largest of three magnitudes; NaN if one is
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// largest magnitude of the sixteen lanes' sixteen values each that this lane belongs to
__device__ __forceinline__ float half_warp_max(const float (&x)[16], bool upper) {
  float t = fabsf(x[0]);
#pragma unroll
  for (int k = 1; k < 15; k += 2) t = max_abs3(t, x[k], x[k + 1]);
  const uint32_t u = __float_as_uint(max_abs3(t, x[15], x[15]));  // NaN above infinity above all, as integers too
  const uint32_t lo = __reduce_max_sync(0xffffffffu, upper ? 0u : u), hi = __reduce_max_sync(0xffffffffu, upper ? u : 0u);
  return __uint_as_float(upper ? hi : lo);
}

// random words of a group of eight entries: Philox4x32-10 with the seed's key schedule from the parameters
__device__ __forceinline__ uint4 group_words(uint64_t grp, uint32_t t, const uint32_t (&k0)[10], uint32_t k1) {
  uint4 x = make_uint4((uint32_t)grp, (uint32_t)(grp >> 32), t, 1u);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    if (r) k1 += 0xBB67AE85u;
    const uint64_t p0 = (uint64_t)x.x * 0xD2511F53u, p1 = (uint64_t)x.z * 0xCD9E8D57u;
    x = make_uint4((uint32_t)(p1 >> 32) ^ x.y ^ k0[r], (uint32_t)p1, (uint32_t)(p0 >> 32) ^ x.w ^ k1, (uint32_t)p0);
  }
  return x;
}

// A warp's stage of shared memory: the operands of one tile as they lie in global memory.
template <int kKind>
struct Stage {
  using K = Kind<kKind>;
  using ST = typename std::conditional<K::master, float, typename K::W>::type;  // the weights that are stepped
  static constexpr int w = 0, g = w + kAdTile * (int)sizeof(ST), m = g + kAdTile * (int)sizeof(typename K::G),
                       v = m + kAdTile, bytes = v + kAdTile;
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// tile of a contiguous operand, 16 bytes a lane at a time
template <class E>
__device__ __forceinline__ void copy_operand(uint32_t dst, const void* base, int tile, uint32_t lane16) {
  const char* src = reinterpret_cast<const char*>(base) + lane16 + (uint64_t)(uint32_t)tile * (kAdTile * sizeof(E));
#pragma unroll
  for (int k = 0; k < kAdTile * (int)sizeof(E); k += 512) copy16(dst + lane16 + k, src + k);
}
// the same where the tensor ends inside the tile (zeros past its end) or the operand has a row stride
template <class E>
__device__ __noinline__ void copy_rows(uint32_t dst, const E* base, int64_t e0, int64_t n, int lane, int32_t cols, int64_t ld) {
  constexpr int per = 16 / sizeof(E);
#pragma unroll 1
  for (int k = lane * per; k < kAdTile; k += 32 * per) {
    const int64_t e = e0 + k, left = n - e;
    const int bytes = left >= per ? 16 : left > 0 ? (int)left * (int)sizeof(E) : 0;
    const E* const src = base + (bytes == 0 ? 0 : cols ? strided(e, cols, ld) : e);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + k * (int)sizeof(E)), "l"(src), "r"(bytes) : "memory");
  }
}

// the same for an operand off its vector addresses, entry by entry
template <class E>
__device__ __noinline__ void copy_entries(E* dst, const E* base, int64_t e0, int64_t n, int lane, int32_t cols, int64_t ld) {
  const int left = (int)min(n - e0, (int64_t)kAdTile);
  Places p(e0 + lane, cols, ld);
#pragma unroll 1
  for (int k0 = lane; k0 < kAdTile; k0 += 8 * 32) {
    E x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t at = p.take();
      x[j] = k0 + 32 * j < left ? base[at] : E(0.f);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) dst[k0 + 32 * j] = x[j];
  }
}

// starts the copies of a tile; returns the exponent bytes of the lane's block
template <int kKind>
__device__ __forceinline__ uint32_t fetch_tile8(const AdTensor& T, int tile, int lane, char* stage_ptr) {
  using L = Stage<kKind>;
  using K = Kind<kKind>;
  using ST = typename L::ST;
  using GT = typename K::G;
  const uint32_t stage = (uint32_t)__cvta_generic_to_shared(stage_ptr);
  const void* const w = K::master ? T.master : T.w;
  if ((int64_t)(tile + 1) * kAdTile <= T.n && (T.flags & (kAdVec | kAdWStride | kAdGStride)) == kAdVec) {
    const uint32_t lane16 = lane * 16;
    copy_operand<GT>(stage + L::g, T.g, tile, lane16);
    copy_operand<uint8_t>(stage + L::m, T.m, tile, lane16);
    copy_operand<uint8_t>(stage + L::v, T.v, tile, lane16);
    copy_operand<ST>(stage + L::w, w, tile, lane16);
    return reinterpret_cast<const uint16_t*>(T.scales)[2 * (int64_t)tile + (lane >> 4)];
  }
  if (!(T.flags & kAdVecState)) return 0;
  const int64_t e0 = (int64_t)tile * kAdTile, n = T.n, blk = 2 * (int64_t)tile + (lane >> 4);
  const GT* const g = reinterpret_cast<const GT*>(T.g);
  const int32_t g_cols = T.flags & kAdGStride ? T.cols : 0, w_cols = !K::master && (T.flags & kAdWStride) ? T.cols : 0;
  if (T.flags & kAdVecG) copy_rows(stage + L::g, g, e0, n, lane, g_cols, T.g_ld);
  else copy_entries(reinterpret_cast<GT*>(stage_ptr + L::g), g, e0, n, lane, g_cols, T.g_ld);
  const ST* const ws = reinterpret_cast<const ST*>(w);
  if (K::master || (T.flags & kAdVecW)) copy_rows(stage + L::w, ws, e0, n, lane, w_cols, T.w_ld);
  else copy_entries(reinterpret_cast<ST*>(stage_ptr + L::w), ws, e0, n, lane, w_cols, T.w_ld);
  copy_rows(stage + L::m, reinterpret_cast<const uint8_t*>(T.m), e0, n, lane, 0, 0);
  copy_rows(stage + L::v, reinterpret_cast<const uint8_t*>(T.v), e0, n, lane, 0, 0);
  return blk * kAdBlock < n ? reinterpret_cast<const uint16_t*>(T.scales)[blk] : 0u;
}

// A tile with vector moments, 8-bit, a block to each half of the warp (sixteen entries a lane: what a block
// costs beside its entries is then paid once for two): the same values as step_block8 with fewer instructions (395 a warp
// for 256 entries, the first form took 770), which are what bounds it.
//  - b1 m = (b1 2^k) code and b2 v = (b2 2^2k) code^2: a power of two commutes with the rounding, so the factor is
//    formed once a block (while it is a normal number).
//  - r' only goes into W' and into its code, which depends on r' through the carry out of its 20 low bits. An
//    approximate root, made smaller by 2^-21 of itself, is below r' by less than 16 units in the last place (by fewer
//    where the pattern is subnormal, whose units are wider) and gives the same code unless those bits are within 16 of a
//    carry: the warp then (one tile in 125) takes exact roots. The block's exponent comes from the exact root of the
//    largest v' (rounding is monotonic).
// false where a value leaves the range in which this holds (nothing is written then).
template <int kKind>
__device__ __forceinline__ bool step_tile8(const AdTensor& T, int tile, int lane, const Consts& c, const AdHyper& h,
                                           char* stage, uint32_t sc) {
  using K = Kind<kKind>;
  using L = Stage<kKind>;
  using WT = typename K::W;
  const bool upper = lane >= 16;
  const int at = lane * 16;
  const int64_t e0 = (int64_t)tile * kAdTile + at;  // entries past the tensor's end are zeros
  float m[16], v[16];
  {
    Raw16<typename K::G> g;
    const uint4 cm = *reinterpret_cast<const uint4*>(stage + L::m + at), cr = *reinterpret_cast<const uint4*>(stage + L::v + at);
    g.from(stage + L::g + at * (int)sizeof(typename K::G));
    const float sm = scale_of(sc & 255u), sr = scale_of(sc >> 8);
    const float b1s = c.b1 * sm, b2s = c.b2 * (sr * sr);
    // exact factors: zero, or normal with room on both sides
    const bool ok = (sm == 0.f || c.b1 == 0.f || (b1s >= 0x1p-100f && b1s <= 0x1p100f)) && sm <= 0x1p100f &&
                    (sr == 0.f || c.b2 == 0.f || (b2s >= 0x1p-100f && b2s <= 0x1p100f)) && sr <= 0x1p50f;
    if (!__all_sync(0xffffffffu, ok)) return false;
    const uint32_t wm[4] = {cm.x, cm.y, cm.z, cm.w}, wr[4] = {cr.x, cr.y, cr.z, cr.w};
    const F2 gs = both(c.gs), b1 = both(b1s), c1 = two(h.c1_2.x, h.c1_2.y), b2 = both(b2s), c2 = two(h.c2_2.x, h.c2_2.y);
#pragma unroll
    for (int k = 0; k < 16; k += 2) {
      const F2 g2 = mul2(gs, g.pair(k)), m2 = values_of(wm[k >> 2] >> (8 * (k & 2))), r2 = values_of(wr[k >> 2] >> (8 * (k & 2)));
      split(add2(mul2(b1, m2), mul2(c1, g2), h.one2), m[k], m[k + 1]);
      split(add2(mul2(b2, mul2(r2, r2)), mul2(c2, mul2(g2, g2)), h.one2), v[k], v[k + 1]);
    }
  }
  const float tm = half_warp_max(m, upper), tv = half_warp_max(v, upper);
  // Finite, within what one factor brings to the codes' patterns (2^(7 - byte), 2^-149 at least), and so large (or zero)
  // that a root flushed to zero (below 2^-63) is far below the codes: its random bits bring it to the smallest at most,
  // which it gets in any case.
  if (!__all_sync(0xffffffffu, tm <= 0x1p36f && tv <= 0x1p72f && (tv == 0.f || tv >= 0x1p-80f))) return false;
  // A root flushed to zero (below 2^-63) leaves out up to 2^-63 ic2 of a denominator of at least eps: 2^-24 of it, unless
  if (c.eps < 0x1p-39f * c.ic2) {
    bool tiny = false;
#pragma unroll
    for (int k = 0; k < 16; ++k) tiny |= v[k] > 0.f && v[k] < 0x1p-126f;
    if (__any_sync(0xffffffffu, tiny)) return false;
  }
  const uint32_t fm = __float_as_uint(tm) >> 23, fr = __float_as_uint(__fsqrt_rn(tv)) >> 23;
  const uint32_t bm = fm > 7u ? fm - 7u : 0u, br = fr > 7u ? fr - 7u : 0u;
  const F2 um = both(bm ? __uint_as_float((158u - bm) << 23) * 0x1p-24f : 0.f);  // 2^(7 - byte), subnormal or not
  const F2 ur = both(br ? __uint_as_float((158u - br) << 23) * 0x1p-24f : 0.f);
  const F2 low = both(1.f - 0x1p-21f), ic2 = both(c.ic2 * (1.f + 0x1p-21f));  // the root that is made smaller, and its weight
  const uint32_t sign = bm ? 0x80808080u : 0u;  // a block held as zeros has no signs
  const uint64_t grp = (uint64_t)e0 >> 3;
  const uint4 ra = group_words(grp, c.t, h.k0, T.id), rb = group_words(grp + 1, c.t, h.k0, T.id);
  const uint32_t rw[8] = {ra.x, ra.y, ra.z, ra.w, rb.x, rb.y, rb.z, rb.w};
  const float lr = c.lr * T.lr_scale;
  const F2 step = both(-lr * c.ic1), decay = both(-lr * T.wd), eps = two(h.eps2.x, h.eps2.y);
  Raw16<typename L::ST> w;
  w.from(stage + L::w + at * (int)sizeof(typename L::ST));
  uint32_t om[4], orr[4], near = 0xffffffffu, zero = 0;
#pragma unroll
  for (int k0 = 0; k0 < 16; k0 += 4) {
    uint32_t pm[4], pr[4];
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
      const int k = k0 + j;
      const F2 m2 = two(m[k], m[k + 1]), r2 = mul2(two(sqrt_approx(v[k]), sqrt_approx(v[k + 1])), low), w2 = w.pair(k);
      float d0, d1, a0, a1, b0, b1;
      split(fma2(r2, ic2, eps), d0, d1);
      split(fma2(step, mul2(m2, two(rcp_approx(d0), rcp_approx(d1))), fma2(decay, w2, w2)), a0, a1);
      w.put(k, a0, a1);
      split(mul2(m2, um), a0, a1);
      split(mul2(r2, ur), b0, b1);
      const uint32_t h0 = __byte_perm(rw[k >> 1], 0, 0x4410), h1 = __byte_perm(rw[k >> 1], 0, 0x4432);
      pm[j] = h0 * 16u + __float_as_uint(a0);
      pm[j + 1] = h1 * 16u + __float_as_uint(a1);
      pr[j] = h0 * 16u + __float_as_uint(b0);
      pr[j + 1] = h1 * 16u + __float_as_uint(b1);
      near = min(near, min(~pr[j] & 0xffff0u, ~pr[j + 1] & 0xffff0u));
    }
    om[k0 >> 2] = codes_of(pm, sign);
    orr[k0 >> 2] = codes_of(pr, 0u);
    zero |= zero_codes(orr[k0 >> 2]);
  }
  if (__any_sync(0xffffffffu, near == 0u)) {
#pragma unroll
    for (int k = 0; k < 16; k += 8) {
      float r[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) r[j] = __fsqrt_rn(v[k + j]);
      const uint2 x = encode8<true, true>(r, br, k ? rb : ra);
      orr[k >> 2] = x.x;
      orr[(k >> 2) + 1] = x.y;
    }
  }
  if (br && (zero & 0x80808080u)) keep_roots(v, orr);
  if (!(T.flags & kAdVecW)) {  // W off its vector addresses: through the stage, entry by entry
    __syncwarp();  // its own copy has been read
    WT* const out = reinterpret_cast<WT*>(stage + L::w);
#pragma unroll
    for (int k = 0; k < 16; k += 2) {
      float x, y;
      split(w.pair(k), x, y);
      put(out + at + k, x);
      put(out + at + k + 1, y);
    }
    __syncwarp();
    const int64_t t0 = (int64_t)tile * kAdTile;
    Places p(t0 + lane, T.flags & kAdWStride ? T.cols : 0, T.w_ld);
    for (int k = lane; k < kAdTile; k += 32) {
      const int64_t to = p.take();
      if (t0 + k < T.n) reinterpret_cast<WT*>(T.w)[to] = out[k];
    }
  }
  if (e0 >= T.n) return true;
  if ((lane & 15) == 0) reinterpret_cast<uint16_t*>(T.scales)[2 * (int64_t)tile + upper] = (uint16_t)(bm | br << 8);
  const bool vw = T.flags & kAdVecW;
  WT* const pw = reinterpret_cast<WT*>(T.w) + (T.flags & kAdWStride ? strided(e0, T.cols, T.w_ld) : e0);
  uint8_t *const pm = reinterpret_cast<uint8_t*>(T.m) + e0, *const pr = reinterpret_cast<uint8_t*>(T.v) + e0;
  if (e0 + 16 <= T.n) {
    if constexpr (K::master) w.store(T.master + e0);
    if (vw) {
      if constexpr (K::master) {
        Raw16<WT> b;
#pragma unroll
        for (int k = 0; k < 16; k += 2) {
          float x, y;
          split(w.pair(k), x, y);
          b.put(k, x, y);
        }
        b.store(pw);
      } else {
        w.store(pw);
      }
    }
    *reinterpret_cast<uint4*>(pm) = make_uint4(om[0], om[1], om[2], om[3]);
    *reinterpret_cast<uint4*>(pr) = make_uint4(orr[0], orr[1], orr[2], orr[3]);
  } else {  // the lane with the tensor's last entries
    const int left = (int)(T.n - e0);
#pragma unroll
    for (int k = 0; k < 16; k += 2) {
      float x[2];
      split(w.pair(k), x[0], x[1]);
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (k + j < left) {
          if constexpr (K::master) T.master[e0 + k + j] = x[j];
          if (vw) put(pw + k + j, x[j]);
          pm[k + j] = (uint8_t)(om[k >> 2] >> (8 * ((k + j) & 3)));
          pr[k + j] = (uint8_t)(orr[k >> 2] >> (8 * ((k + j) & 3)));
        }
    }
  }
  return true;
}

__device__ __forceinline__ Consts consts_of(const AdHyper& h) {
  const int64_t t = h.d_t ? *h.d_t + 1 : h.t;
  Consts c;
  c.b1 = h.b1; c.c1 = h.c1; c.b2 = h.b2; c.c2 = h.c2; c.eps = h.eps;
  c.lr = h.d_lr ? *h.d_lr : h.lr;
  c.gs = h.d_gscale ? *h.d_gscale : 1.f;
  c.ic1 = -1.f / expm1f((float)((double)t * h.log_b1));
  c.ic2 = rsqrtf(-expm1f((float)((double)t * h.log_b2)));
  c.t = (uint32_t)t;
  c.seed = h.seed;
  return c;
}

// at a kernel's end, in the call's last launch: the last CTA to come here counts the step
__device__ __forceinline__ void advance(const AdHyper& h, int skip) {
  if (!h.d_t || !h.advance || skip) return;
  __syncthreads();  // every thread of the CTA has read the count
  if (threadIdx.x == 0) {
    __threadfence();
    if (atomicAdd(reinterpret_cast<unsigned long long*>(h.d_t + 1), 1ull) + 1 == gridDim.x) {
      h.d_t[1] = 0;
      h.d_t[0] += 1;
    }
  }
}

}  // namespace

// A warp takes one block and ends: a grid of as many CTAs as that needs moved 98% of the copy rate on the 774M-entry
// case (3.38 ms), a grid of resident CTAs that walk on 89 to 93% (3.56 to 3.73 ms): its warps load and store in step.
constexpr int kAd32Warps = 4;
template <int kKind, class Table>
__global__ void __launch_bounds__(32 * kAd32Warps, 8) k_adamw32(const __grid_constant__ Table tb, const __grid_constant__ AdHyper h) {
  __shared__ AdTensor slots[kAd32Warps][1];  // a warp looks up one tensor
  follow_previous();
  const int skip = h.skip ? *h.skip : 0;
  const Consts c = consts_of(h);
  const int lane = threadIdx.x & 31;
  const unsigned unit = blockIdx.x * kAd32Warps + (threadIdx.x >> 5);  // block of the launch, two for each tile
  AdTensor* const mine = slots[threadIdx.x >> 5];
  Walk<Table> at((int)(unit >> 1), tb.total_tiles);
  if (at.seek(tb, mine)) {
    const AdTensor& T = tensor_at(tb, at.li, mine, at.which);
    const int64_t blk = 2 * (int64_t)(at.b - T.tile_begin) + (unit & 1);
    if (skip) {  // nothing
    } else if ((T.flags & kAdVec) == kAdVec && (blk + 1) * kAdBlock <= T.n) {
      step_lane32<kKind>(T, blk * kAdBlock + lane * 8, c);
    } else if (blk * kAdBlock < T.n) {
      step_block32<kKind>(T, blk, lane, c);
    }
  }
  advance(h, skip);
}

// Each warp has two stages of its own: the next tile's operands are on their way into one (cp.async) while the other is
// stepped. A CTA walks over a stretch of its own: tiles dealt out in turn over the grid took 2.35 ms instead of 2.20 on
// the 774M-entry case with master (all CTAs load and store in step). Deeper rings (up to four stages: 2.35, 2.47 and 2.51
// ms with two, three and four) and more warps with fewer registers measured slower. bf16 weights without a master: 65.6M
// entries take 137 to 141 us (4.7 to 4.8 TB/s), and no unit is full (issue slots 65%, FMA pipe 56%, ALU 49%, DRAM 51%). With
// 16 warps an SM a third of the cycles has none to issue: of the 5.2 cycles between two instructions of a warp 1.3 are
// the first one's latency, 0.7 a busy pipe, 1.0 other warps' turns. Data that stays in L2 would take 114 us.
constexpr int kAd8Warps = 2, kAd8Ctas = 8;
constexpr int kAd8Run = 24;  // tiles of a warp in a long run of CTAs
template <int kKind, class Table>
__global__ void __launch_bounds__(32 * kAd8Warps, kAd8Ctas) k_adamw8(const __grid_constant__ Table tb,
                                                                     const __grid_constant__ AdHyper h) {
  using L = Stage<kKind>;
  extern __shared__ __align__(16) char smem[];
  __shared__ AdTensor slots[kAd8Warps][2];
  follow_previous();
  const int skip = h.skip ? *h.skip : 0;
  const Consts c = consts_of(h);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  char* const ring = smem + warp * 2 * L::bytes;
  AdTensor* const mine = slots[warp];
  const int first = (int)((int64_t)tb.total_tiles * blockIdx.x / gridDim.x);
  Walk<Table> next(first + warp, (int)((int64_t)tb.total_tiles * (blockIdx.x + 1) / gridDim.x));
  bool more = next.seek(tb, mine);
  uint32_t sc_next = 0;
  if (more) {
    const AdTensor& N = tensor_at(tb, next.li, mine, next.which);
    sc_next = fetch_tile8<kKind>(N, next.b - N.tile_begin, lane, ring);
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
  if (skip) {
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    more = false;
  }
  for (int turn = 0; more; turn ^= 1) {
    const AdTensor& T = tensor_at(tb, next.li, mine, next.which);
    const int tile = next.b - T.tile_begin;
    const uint32_t sc = sc_next;
    next.b += kAd8Warps;
    more = next.seek(tb, mine);
    __syncwarp();  // every lane has read the stage that is filled now
    if (more) {
      const AdTensor& N = tensor_at(tb, next.li, mine, next.which);
      sc_next = fetch_tile8<kKind>(N, next.b - N.tile_begin, lane, ring + (turn ^ 1) * L::bytes);
    }
    asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 1;" ::: "memory");
    __syncwarp();
    if ((T.flags & kAdVecState) && step_tile8<kKind>(T, tile, lane, c, h, ring + turn * L::bytes, sc)) continue;
    for (int k = 0; k < 2 && (2 * (int64_t)tile + k) * kAdBlock < T.n; ++k) step_block8<kKind>(T, 2 * (int64_t)tile + k, lane, c);
  }
  advance(h, skip);
}

namespace {
template <int kKind, class Table>
cudaError_t launch_kind(const Table& tb, const AdHyper& h, int sms, cudaStream_t s) {
  if constexpr (Kind<kKind>::eight) {
    // As many CTAs as are resident, with equal stretches; from four times what those do at 24 tiles a warp on (117M entries
    // on 148 SMs), CTAs of 24 tiles a warp that follow one another, whose stretches stay close together in memory. Both
    // forms on one box, us (resident / following), bf16 without a master: 33M entries 72 / 84, 66M 138 / 146, 90M 186 /
    // 189, 118M 242 / 242, 131M 268 / 266, 233M 472 / 455, 774M 1,578 / 1,506; bf16 with a master: 33M 100 / 114, 66M 194 /
    // 188, 118M 341 / 312, 233M 667 / 592, 774M 2,177 / 1,913; float32: 33M 101 / 112, 66M 199 / 183, 118M 341 / 309, 774M
    // 2,116 / 1,866. What crosses is the round of CTAs that is left over at the end, so the latest type sets the border.
    const int want = (tb.total_tiles + kAd8Warps - 1) / kAd8Warps, resident = sms * kAd8Ctas;
    const int grid = want < 1 ? 1 : want < resident ? want : want / kAd8Run >= 4 * resident ? want / kAd8Run : resident;
    return launch(k_adamw8<kKind, Table>, grid, 32 * kAd8Warps, kAd8Warps * 2 * Stage<kKind>::bytes, s, tb, h);
  } else {
    const int want = (int)((2 * (int64_t)tb.total_tiles + kAd32Warps - 1) / kAd32Warps);
    return launch(k_adamw32<kKind, Table>, want < 1 ? 1 : want, 32 * kAd32Warps, 0, s, tb, h);
  }
}
}  // namespace

template <class Table>
cudaError_t launch_adamw(int kind, const Table& tb, const AdHyper& h, int sms, cudaStream_t s) {
  switch (kind) {
    case AD_W_F32: return launch_kind<AD_W_F32, Table>(tb, h, sms, s);
    case AD_W_BF16: return launch_kind<AD_W_BF16, Table>(tb, h, sms, s);
    case AD_W_MASTER: return launch_kind<AD_W_MASTER, Table>(tb, h, sms, s);
    case AD_W_F32 | AD_G_BF16: return launch_kind<AD_W_F32 | AD_G_BF16, Table>(tb, h, sms, s);
    case AD_W_BF16 | AD_G_BF16: return launch_kind<AD_W_BF16 | AD_G_BF16, Table>(tb, h, sms, s);
    case AD_W_MASTER | AD_G_BF16: return launch_kind<AD_W_MASTER | AD_G_BF16, Table>(tb, h, sms, s);
    case AD_W_F32 | AD_8BIT: return launch_kind<AD_W_F32 | AD_8BIT, Table>(tb, h, sms, s);
    case AD_W_BF16 | AD_8BIT: return launch_kind<AD_W_BF16 | AD_8BIT, Table>(tb, h, sms, s);
    case AD_W_MASTER | AD_8BIT: return launch_kind<AD_W_MASTER | AD_8BIT, Table>(tb, h, sms, s);
    case AD_W_F32 | AD_G_BF16 | AD_8BIT: return launch_kind<AD_W_F32 | AD_G_BF16 | AD_8BIT, Table>(tb, h, sms, s);
    case AD_W_BF16 | AD_G_BF16 | AD_8BIT: return launch_kind<AD_W_BF16 | AD_G_BF16 | AD_8BIT, Table>(tb, h, sms, s);
    case AD_W_MASTER | AD_G_BF16 | AD_8BIT: return launch_kind<AD_W_MASTER | AD_G_BF16 | AD_8BIT, Table>(tb, h, sms, s);
    default: return cudaErrorInvalidValue;
  }
}
template cudaError_t launch_adamw(int, const AdTable<kAdFew>&, const AdHyper&, int, cudaStream_t);
template cudaError_t launch_adamw(int, const AdTable<kAdMany>&, const AdHyper&, int, cudaStream_t);
template cudaError_t launch_adamw(int, const AdDevTable&, const AdHyper&, int, cudaStream_t);

// ---------------------------------------------------------------- gradient norm
// A lane squares eight entries at a time: their sum in float32 (one rounding an entry), added up in float64 in a fixed
// order. Where the float32 sum leaves [2^-90, 2^120] (squares that underflow or overflow, NaN, zeros) it is formed in
// float64 instead, so every gradient whose norm float32 holds gets it. It reads 2 or 4 bytes an entry and writes nothing:
// 774M bf16 entries take 257 to 276 us (86 to 92% of the copy rate); 290 short tensors 5.6 us, which are latencies (table,
// tensor, data, the CTAs' sums). One launch: the last CTA to arrive adds the others' sums, in their order.
namespace {
constexpr float kNormLow = 0x1p-90f, kNormHigh = 0x1p120f;
__device__ __noinline__ double sumsq_f64(const float (&g)[8]) {
  double d = 0.0;
#pragma unroll 1
  for (int k = 0; k < 8; ++k) d = fma((double)g[k], (double)g[k], d);
  return d;
}

template <class E>
struct Raw8;
template <>
struct Raw8<float> {
  uint32_t u[8];
  __device__ __forceinline__ void load(const float* p) { ld256(p, u); }
  __device__ __forceinline__ float sum() const {
    F2 a{0};
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      const F2 x = two(__uint_as_float(u[k]), __uint_as_float(u[k + 1]));
      a = k ? fma2(x, x, a) : mul2(x, x);
    }
    float lo, hi;
    split(a, lo, hi);
    return __fadd_rn(lo, hi);
  }
  __device__ __forceinline__ void values(float (&g)[8]) const {
#pragma unroll
    for (int k = 0; k < 8; ++k) g[k] = __uint_as_float(u[k]);
  }
};
template <>
struct Raw8<__nv_bfloat16> {
  uint32_t u[4];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    const uint4 x = *reinterpret_cast<const uint4*>(p);
    u[0] = x.x; u[1] = x.y; u[2] = x.z; u[3] = x.w;
  }
  __device__ __forceinline__ float sum() const {  // bf16 factors, float32 sum: nothing to unpack
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      asm("fma.rn.f32.bf16 %0, %1, %1, %0;" : "+f"(s) : "h"((uint16_t)u[k]));
      asm("fma.rn.f32.bf16 %0, %1, %1, %0;" : "+f"(s) : "h"((uint16_t)(u[k] >> 16)));
    }
    return s;
  }
  __device__ __forceinline__ void values(float (&g)[8]) const {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      g[2 * k] = __uint_as_float(u[k] << 16);
      g[2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
    }
  }
};
template <class E>
__device__ __forceinline__ double sumsq(const Raw8<E>& x) {
  const float s = x.sum();
  if (s >= kNormLow && s <= kNormHigh) return (double)s;
  uint32_t any = 0;  // rows without a gradient are common: no float64 for them
#pragma unroll
  for (int k = 0; k < (int)(sizeof(x.u) / 4); ++k) any |= x.u[k];
  if (any == 0) return 0.0;
  float g[8];
  x.values(g);
  return sumsq_f64(g);
}

// what a warp keeps of the tensor it is in
struct NormAt {
  const void* g;
  int64_t n;
  int begin;
  bool fast;  // contiguous and aligned
};

// a lane's part of a tile, its first entry e0: four loads of eight under way at once (with eight 774M bf16 entries took
// 291 us instead of 257)
template <class E>
__device__ __forceinline__ double run_sumsq(const NormAt& A, const NormTensor& T, int64_t e0, int lane) {
  constexpr int kLoads = kNormTile / kAdBlock;
  const E* const p = reinterpret_cast<const E*>(A.g);
  double d = 0.0;
  if (A.fast) {
    Raw8<E> x[kLoads];
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      x[k] = Raw8<E>{};
      if (e0 + k * kAdBlock + 8 <= A.n) x[k].load(p + e0 + k * kAdBlock);
    }
#pragma unroll
    for (int k = 0; k < kLoads; ++k) d += sumsq(x[k]);
    const int64_t tail = A.n & ~(int64_t)7;  // the last entries, short of eight: one lane's
    if (tail < A.n && tail >= e0 && tail < e0 + kLoads * kAdBlock && (tail - e0) % kAdBlock == 0) {
      for (int64_t e = tail; e < A.n; ++e) d = fma((double)to_f32(p[e]), (double)to_f32(p[e]), d);
    }
    return d;
  }
  const bool stride = T.ld != T.cols;
  if (T.vec) {  // a row stride, eight in one row
#pragma unroll 1
    for (int k = 0; k < kLoads; ++k) {
      const int64_t e = e0 + k * kAdBlock;
      if (e + 8 > A.n) break;
      Raw8<E> x;
      x.load(p + strided(e, T.cols, T.ld));
      d += sumsq(x);
    }
    return d;
  }
  // off the vector addresses: entries 32 apart, which the lanes' accesses cover side by side
  const int64_t first = e0 - lane * 7;
  Places at(first, stride ? T.cols : 0, T.ld);
#pragma unroll 1
  for (int k = 0; k < kLoads; ++k) {
    float g[8], s = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t to = at.take();
      g[j] = first + 256 * k + 32 * j < A.n ? to_f32(p[to]) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) s = fmaf(g[j], g[j], s);
    d += s >= kNormLow && s <= kNormHigh ? (double)s : sumsq_f64(g);
  }
  return d;
}

// sum over the CTA, in a fixed order, in thread 0
__device__ __forceinline__ double cta_sum(double acc) {
  __shared__ double part[8];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = acc;
  __syncthreads();
  double s = 0.0;
  if (threadIdx.x == 0)
    for (int k = 0; k < 8; ++k) s += part[k];
  return s;
}
}  // namespace

__global__ void __launch_bounds__(256, 4) k_grad_norm(const __grid_constant__ NormArgs a) {
  const int lane = threadIdx.x & 31;
  double acc = 0.0;
  int li = 0, end = 0;
  follow_previous();
  NormAt A{};
  bool bf16 = false;
  // a stretch of its own for each CTA: 774M bf16 entries 268 us, dealt out in turn 284
  const int stop = (int)((int64_t)a.total_tiles * (blockIdx.x + 1) / gridDim.x);
  for (int b = (int)((int64_t)a.total_tiles * blockIdx.x / gridDim.x) + (threadIdx.x >> 5); b < stop; b += 8) {
    if (b >= end) {
      li = tensor_of_warp(a.t, a.guide, b);
      const NormTensor& T = a.t[li];
      A = NormAt{T.g, T.n, T.tile_begin, T.vec && T.ld == T.cols};
      bf16 = T.bf16;
      end = li + 1 < a.n_tensors ? a.t[li + 1].tile_begin : a.total_tiles;
    }
    const int64_t e0 = (int64_t)(b - A.begin) * kNormTile + lane * 8;
    acc += bf16 ? run_sumsq<__nv_bfloat16>(A, a.t[li], e0, lane) : run_sumsq<float>(A, a.t[li], e0, lane);
  }
  const double mine = cta_sum(acc);
  __shared__ bool last;
  if (threadIdx.x == 0) {
    a.partials[blockIdx.x] = mine;
    __threadfence();
    last = atomicInc(a.arrived, gridDim.x - 1) == gridDim.x - 1;  // wraps to zero for the next launch
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  acc = 0.0;
#pragma unroll
  for (int k = 0; k < (kNormMaxGrid + 255) / 256; ++k) {
    const int i = threadIdx.x + 256 * k;
    if (i < gridDim.x) acc += *(volatile double*)(a.partials + i);
  }
  const double s = cta_sum(acc);
  if (threadIdx.x) return;
  const double norm = sqrt(s);
  const float f = (float)norm;
  const bool bad = !(f <= 3.402823466e38f);
  a.out[0] = f;
  a.out[1] = bad ? 0.f : (float)fmin(1.0, a.max_norm / (norm + 1e-6));
  if (a.skip) *a.skip = bad;
  if (a.status && bad) atomicOr(a.status, SMUON_DEV_NONFINITE_NORM);
}

cudaError_t launch_grad_norm(const NormArgs& a, cudaStream_t s) {
  const int want = (a.total_tiles + 7) / 8;
  return launch(k_grad_norm, want < 1 ? 1 : (want < kNormMaxGrid ? want : kNormMaxGrid), 256, 0, s, a);
}

// ---------------------------------------------------------------- conversion
// Reads 8 and writes 2 bytes an entry, or the other way round; one block a warp, as in k_adamw32 (65.6M entries to 32
// bits: 99 us; with a grid of resident CTAs 118 us).
namespace {
__device__ __forceinline__ void convert_to8(const ConvTensor& T, int64_t blk, int lane, const float (&m)[8], float (&r)[8]) {
  const int64_t e0 = blk * kAdBlock + lane * 8;
  const bool vec = T.vec && e0 + 8 <= T.n;
#pragma unroll
  for (int k = 0; k < 8; ++k) r[k] = __fsqrt_rn(r[k]);
  const uint32_t bm = block_exponent(m), br = block_exponent(r);
  store_codes(reinterpret_cast<uint8_t*>(T.m8), e0, T.n, vec, encode8<false, false>(m, bm, make_uint4(0, 0, 0, 0)));
  store_codes(reinterpret_cast<uint8_t*>(T.v8), e0, T.n, vec, encode8<false, true>(r, br, make_uint4(0, 0, 0, 0)));
  if (lane == 0) *reinterpret_cast<uint16_t*>(T.scales + 2 * blk) = (uint16_t)(bm | br << 8);
}
__device__ __forceinline__ void convert_to32(const ConvTensor& T, int64_t blk, int lane, uint32_t sc, uint2 cm, uint2 cr) {
  const int64_t e0 = blk * kAdBlock + lane * 8;
  const bool vec = T.vec && e0 + 8 <= T.n;
  float m[8], r[8];
  decode8(cm, scale_of(sc & 255u), m);
  decode8(cr, scale_of(sc >> 8), r);
#pragma unroll
  for (int k = 0; k < 8; ++k) r[k] = __fmul_rn(r[k], r[k]);
  store(reinterpret_cast<float*>(T.m32), e0, T.n, e0, vec, m);
  store(reinterpret_cast<float*>(T.v32), e0, T.n, e0, vec, r);
}
}  // namespace

constexpr int kConvWarps = 8;
__global__ void __launch_bounds__(32 * kConvWarps) k_adamw_convert(const __grid_constant__ ConvTable tb) {
  follow_previous();
  const int lane = threadIdx.x & 31;
  const unsigned unit = blockIdx.x * kConvWarps + (threadIdx.x >> 5);  // block of the launch, two for each tile
  const int tile = (int)(unit >> 1);
  if (tile >= tb.total_tiles) return;
  const ConvTensor& T = tb.t[tensor_of(tb, tile, 0)];
  const int64_t n = T.n, blk = 2 * (int64_t)(tile - T.tile_begin) + (unit & 1), e0 = blk * kAdBlock + lane * 8;
  if (blk * kAdBlock >= n) return;
  const bool vec = T.vec && e0 + 8 <= n;
  if (tb.to8) {
    float m[8], r[8];
    load(reinterpret_cast<const float*>(T.m32), e0, n, e0, vec, m);
    load(reinterpret_cast<const float*>(T.v32), e0, n, e0, vec, r);
    convert_to8(T, blk, lane, m, r);
  } else {
    const uint32_t sc = reinterpret_cast<const uint16_t*>(T.scales)[blk];
    const uint2 cm = load_codes(reinterpret_cast<const uint8_t*>(T.m8), e0, n, vec);
    const uint2 cr = load_codes(reinterpret_cast<const uint8_t*>(T.v8), e0, n, vec);
    convert_to32(T, blk, lane, sc, cm, cr);
  }
}

cudaError_t launch_adamw_convert(const ConvTable& tb, cudaStream_t s) {
  const int want = (int)((2 * (int64_t)tb.total_tiles + kConvWarps - 1) / kConvWarps);
  return launch(k_adamw_convert, want < 1 ? 1 : want, 32 * kConvWarps, 0, s, tb);
}

}  // namespace smuon
