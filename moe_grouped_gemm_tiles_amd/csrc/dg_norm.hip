// dg_norm.hip -- residual addition, RMS norm and the per-token FP8 cast in one
// pass, and the gradient of the norm, on gfx950.
//
// Forward, per row of K values (all in FP32, every output rounded once):
//     s = x + residual,  rstd = 1 / sqrt(mean(s^2) + eps),  y = s * rstd * w,
//     per 128 values:  sf = amax(|y|) / 448 (or the UE8M0 form),  q = E4M3(y / sf),
// the same scale rule and quotient as the plain cast (dg_cast.hpp).
//
// Backward, with xhat = s * rstd and g = dy * w:
//     dx = rstd * (g - xhat * mean(g * xhat)) + dresidual,   dw = sum over rows of dy * xhat
// (the cast passes its gradient through unchanged).
#include <hip/hip_runtime.h>

#include <cstdint>

#include "dg.h"
#include "dg_cast.hpp"
#include "dg_common.hpp"

namespace {

namespace norm {

using namespace dg::cast;

constexpr int kMaxThreads = 512;
constexpr int kMaxChunks = 4;                        // 8-value chunks a thread holds
constexpr int kMaxK = 8 * kMaxChunks * kMaxThreads;  // 16384

// BF16 bits of a float, round to nearest even (NaN stays NaN), two to a word.
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}

template <bool BF16>
__device__ __forceinline__ void store8(void* p, const float (&v)[8]) {
  if constexpr (BF16) {
    *reinterpret_cast<uint4*>(p) = make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]),
                                              bf16_pair(v[6], v[7]));
  } else {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *(reinterpret_cast<float4*>(p) + 1) = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// Eight values of the norm's weight (chunk ch of the row).
__device__ __forceinline__ void load_weight(const uint8_t* w, int bf16, int ch, float (&v)[8]) {
  if (bf16) load8<true>(w + (int64_t)ch * 16, v);
  else load8<false>(w + (int64_t)ch * 32, v);
}

// Sum over the workgroup, the same on every thread and in a fixed order.
// `slot` holds one float per wave; calls in turn use different slots, so one
// barrier per call is enough.
__device__ __forceinline__ float block_sum(float v, float* slot) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
  const int waves = blockDim.x >> 6;
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
  __syncthreads();
  float t = 0.f;
  for (int i = 0; i < waves; ++i) t += slot[i];
  return t;
}

struct FwdParams {
  const uint8_t* x;
  const uint8_t* res;
  uint8_t* res_out;
  const uint8_t* w;
  uint8_t* q;
  void* sf;
  uint8_t* y;
  float* rstd;
  int64_t ldx, ldr, ldro, ldq, ld_sf, ldy;  // bytes, except ld_sf (words)
  float eps;
  int m, k, rows_per_wg;
  int w_bf16;
};

// Codes of eight values of a block whose amax bits are `amax` (as an unsigned
// integer, so that a NaN is the largest).  A block with an Inf or NaN keeps it:
// its scale is not finite, and neither are its NaN elements' codes.
template <bool UE8M0>
__device__ __forceinline__ uint2 codes8(const float (&v)[8], uint32_t amax, float& s, uint32_t& byte) {
  if (amax >= 0x7f800000u) {
    byte = 255;
    s = amax > 0x7f800000u ? __builtin_nanf("") : __builtin_inff();
    uint2 c = make_uint2(0, 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t nan = !(fabsf(v[i]) < __builtin_inff());
      (i < 4 ? c.x : c.y) |= (nan ? 0x7fu : 0u) << (8 * (i & 3));
    }
    return c;
  }
  const float a = __uint_as_float(amax);
  if constexpr (UE8M0) {
    byte = ue8m0_byte(a);
    s = ue8m0_value(byte);
  } else {
    byte = 0;
    s = fp32_scale(a);
  }
  return quant8<UE8M0>(v, s);
}

// One workgroup takes rows_per_wg rows in turn; a thread holds chunks
// c * blockDim + tid of eight values of a row, so 16 adjacent lanes hold one
// 128-value block and a wave four adjacent ones (one packed UE8M0 word).
template <bool BF16, bool UE8M0, int C>
__global__ void __launch_bounds__(kMaxThreads) fwd_kernel(const FwdParams p) {
  __shared__ float s_sum[2][2][kMaxThreads / 64];  // [scaled again][row parity]
  constexpr int ES = BF16 ? 2 : 4;
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 63;
  const int chunks = p.k >> 3;
  const int row0 = blockIdx.x * p.rows_per_wg;
  const int row1 = min(row0 + p.rows_per_wg, p.m);
  for (int row = row0; row < row1; ++row) {
    float v[C][8];
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int ch = c * nt + tid;
      if (ch >= chunks) continue;
      load8<BF16>(p.x + row * p.ldx + (int64_t)ch * 8 * ES, v[c]);
      if (p.res != nullptr) {
        float r[8];
        load8<BF16>(p.res + row * p.ldr + (int64_t)ch * 8 * ES, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] += r[i];
        store8<BF16>(p.res_out + row * p.ldro + (int64_t)ch * 8 * ES, v[c]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) ss += v[c][i] * v[c][i];
    }
    ss = block_sum(ss, s_sum[0][row & 1]);
    float rstd = 1.0f / sqrtf(ss / (float)p.k + p.eps);
    if (!(ss >= 0x1p-100f && ss < __builtin_inff())) {
      // squares past FP32's range on either side (the same branch on every thread): again, scaled
      const float c = ss < 1.0f ? 0x1p60f : 0x1p-64f;
      ss = 0.f;
#pragma unroll
      for (int j = 0; j < C; ++j) {
        if (j * nt + tid >= chunks) continue;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += (v[j][i] * c) * (v[j][i] * c);
      }
      ss = block_sum(ss, s_sum[1][row & 1]);
      rstd = (float)(1.0 / sqrt((double)ss / ((double)c * (double)c) / p.k + (double)p.eps));
    }
    if (p.rstd != nullptr && tid == 0) p.rstd[row] = rstd;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int ch = c * nt + tid;
      if (c * nt + (tid & ~63) >= chunks) continue;  // a wave past the row's end; its last blocks may be too
      uint32_t amax = 0;
      if (ch < chunks) {
        float w[8];
        load_weight(p.w, p.w_bf16, ch, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[c][i] = v[c][i] * rstd * w[i];
          amax = max(amax, __float_as_uint(v[c][i]) & 0x7fffffffu);
        }
        if (p.y != nullptr) store8<BF16>(p.y + row * p.ldy + (int64_t)ch * 8 * ES, v[c]);
      }
#pragma unroll
      for (int off = 8; off >= 1; off >>= 1) amax = max(amax, (uint32_t)__shfl_xor((int)amax, off, 16));
      float s = 1.0f;
      uint32_t byte = 127;
      if (ch < chunks) {
        *reinterpret_cast<uint2*>(p.q + row * p.ldq + (int64_t)ch * 8) = codes8<UE8M0>(v[c], amax, s, byte);
      }
      if constexpr (UE8M0) {
        const uint32_t b1 = __shfl((int)byte, 16), b2 = __shfl((int)byte, 32), b3 = __shfl((int)byte, 48);
        if (lane == 0)
          static_cast<uint32_t*>(p.sf)[(int64_t)(ch >> 6) * p.ld_sf + row] = byte | b1 << 8 | b2 << 16 | b3 << 24;
      } else {
        if ((lane & 15) == 0 && ch < chunks) static_cast<float*>(p.sf)[(int64_t)(ch >> 4) * p.ld_sf + row] = s;
      }
    }
  }
}

struct BwdParams {
  const uint8_t* dy;
  const uint8_t* s;
  const uint8_t* w;
  const uint8_t* dres;
  const float* rstd;
  uint8_t* dx;
  float* part;
  int64_t lddy, lds, lddres, lddx;  // bytes
  int m, k;
  int w_bf16;
};

// One workgroup takes rows blockIdx, blockIdx + gridDim, ... and keeps its sum
// of dy * xhat per column in registers; it leaves that as one row of `part`.
template <bool BF16, int C>
__global__ void __launch_bounds__(kMaxThreads) bwd_kernel(const BwdParams p) {
  __shared__ float s_sum[2][kMaxThreads / 64];
  constexpr int ES = BF16 ? 2 : 4;
  const int tid = threadIdx.x, nt = blockDim.x;
  const int chunks = p.k >> 3;
  float dw[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[c][i] = 0.f;
  const float inv_k = 1.0f / (float)p.k;
  int turn = 0;
  for (int row = blockIdx.x; row < p.m; row += gridDim.x, turn ^= 1) {
    const float rstd = p.rstd[row];
    float g[C][8], xh[C][8];
    float dot = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int ch = c * nt + tid;
      if (ch >= chunks) continue;
      load8<BF16>(p.dy + row * p.lddy + (int64_t)ch * 8 * ES, g[c]);
      load8<BF16>(p.s + row * p.lds + (int64_t)ch * 8 * ES, xh[c]);
      float w[8];
      load_weight(p.w, p.w_bf16, ch, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        xh[c][i] *= rstd;
        dw[c][i] += g[c][i] * xh[c][i];
        g[c][i] *= w[i];
        dot += g[c][i] * xh[c][i];
      }
    }
    dot = block_sum(dot, s_sum[turn]) * inv_k;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int ch = c * nt + tid;
      if (ch >= chunks) continue;
      float d[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] = rstd * (g[c][i] - xh[c][i] * dot);
      if (p.dres != nullptr) {
        float r[8];
        load8<BF16>(p.dres + row * p.lddres + (int64_t)ch * 8 * ES, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] += r[i];
      }
      store8<BF16>(p.dx + row * p.lddx + (int64_t)ch * 8 * ES, d);
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int ch = c * nt + tid;
    if (ch < chunks) store8<false>(p.part + (int64_t)blockIdx.x * p.k + (int64_t)ch * 8, dw[c]);
  }
}

constexpr int kDwCols = 32;  // columns of one workgroup of the column sum

// dw[col] (+)= sum over rows of part[row][col]: eight lanes take 32 columns of
// a row, 32 rows at a time, and the 32 sums of a column are added in order.
__global__ void __launch_bounds__(256) dw_kernel(const float* part, int rows, int k, float* dw, int accumulate) {
  __shared__ float t[32][kDwCols];
  const int tid = threadIdx.x, r = tid >> 3, c4 = (tid & 7) * 4;
  const int col = blockIdx.x * kDwCols + c4;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = r; i < rows; i += 32) {
    const float4 v = *reinterpret_cast<const float4*>(part + (int64_t)i * k + col);
    a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
  }
  *reinterpret_cast<float4*>(&t[r][c4]) = a;
  __syncthreads();
  if (tid < kDwCols) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) sum += t[i][tid];
    float* o = dw + blockIdx.x * kDwCols + tid;
    *o = accumulate ? *o + sum : sum;
  }
}

// Threads and chunks per thread for rows of k values.
struct Shape {
  int threads, chunks;
};
Shape shape_for(int k, int want_chunks) {
  const int n = k / 8;
  int c = want_chunks;
  while (c < kMaxChunks && (n + c - 1) / c > kMaxThreads) c *= 2;
  const int threads = ((n + c - 1) / c + 63) / 64 * 64;
  return {threads, c};
}

// Workgroups of the backward's row loop: each leaves a row of partial sums.
int bwd_grid(int m) {
  constexpr int kMost = 1024;
  return m < kMost ? m : kMost;
}

inline bool aligned_to(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// A row-major operand: rows 16-byte aligned and at least k elements apart.
inline bool rows_ok(const void* p, int64_t ld, int64_t es, int k) {
  return p != nullptr && aligned_to(p, 16) && ld >= k && (ld * es) % 16 == 0;
}

template <bool BF16, bool UE8M0>
void launch_fwd(const FwdParams& p, Shape s, dim3 grid, hipStream_t stream) {
  switch (s.chunks) {
    case 1: hipLaunchKernelGGL((fwd_kernel<BF16, UE8M0, 1>), grid, dim3(s.threads), 0, stream, p); break;
    case 2: hipLaunchKernelGGL((fwd_kernel<BF16, UE8M0, 2>), grid, dim3(s.threads), 0, stream, p); break;
    default: hipLaunchKernelGGL((fwd_kernel<BF16, UE8M0, 4>), grid, dim3(s.threads), 0, stream, p); break;
  }
}

template <bool BF16>
void launch_bwd(const BwdParams& p, Shape s, dim3 grid, hipStream_t stream) {
  switch (s.chunks) {
    case 1: hipLaunchKernelGGL((bwd_kernel<BF16, 1>), grid, dim3(s.threads), 0, stream, p); break;
    case 2: hipLaunchKernelGGL((bwd_kernel<BF16, 2>), grid, dim3(s.threads), 0, stream, p); break;
    default: hipLaunchKernelGGL((bwd_kernel<BF16, 4>), grid, dim3(s.threads), 0, stream, p); break;
  }
}

dg_status launch_status() {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? DG_SUCCESS : dg::record_hip_error(e);
}

}  // namespace norm

}  // namespace

extern "C" {

dg_status dg_add_rms_norm_cast_to_fp8(const void* x, int64_t ldx, const void* residual, int64_t ld_residual,
                                      void* residual_out, int64_t ld_residual_out, dg_dtype dtype,
                                      const void* weight, dg_dtype weight_dtype, float eps, void* q, int64_t ldq,
                                      void* sf, int64_t ld_sf, int ue8m0, void* y, int64_t ldy, float* rstd, int m,
                                      int k, hipStream_t stream) {
  using namespace norm;
  if (m < 0 || k < 0 || (dtype != DG_DTYPE_BF16 && dtype != DG_DTYPE_FP32) ||
      (weight_dtype != DG_DTYPE_BF16 && weight_dtype != DG_DTYPE_FP32) || !(eps >= 0.f))
    return DG_ERROR_INVALID_VALUE;
  if (k % 128 != 0 || k > kMaxK) return DG_ERROR_NOT_SUPPORTED;
  if (m == 0 || k == 0) return DG_SUCCESS;
  const int64_t es = dtype == DG_DTYPE_BF16 ? 2 : 4;
  if (!rows_ok(x, ldx, es, k)) return DG_ERROR_INVALID_VALUE;
  if ((residual == nullptr) != (residual_out == nullptr)) return DG_ERROR_INVALID_VALUE;
  if (residual != nullptr && (!rows_ok(residual, ld_residual, es, k) || !rows_ok(residual_out, ld_residual_out, es, k)))
    return DG_ERROR_INVALID_VALUE;
  if (y != nullptr && !rows_ok(y, ldy, es, k)) return DG_ERROR_INVALID_VALUE;
  if (weight == nullptr || !aligned_to(weight, 16)) return DG_ERROR_INVALID_VALUE;
  if (q == nullptr || !aligned_to(q, 8) || ldq < k || ldq % 8 != 0) return DG_ERROR_INVALID_VALUE;
  if (sf == nullptr || !aligned_to(sf, 16) || ld_sf < m || ld_sf % 4 != 0) return DG_ERROR_INVALID_VALUE;
  if (!aligned_to(rstd, 4)) return DG_ERROR_INVALID_VALUE;
  FwdParams p{static_cast<const uint8_t*>(x), static_cast<const uint8_t*>(residual),
              static_cast<uint8_t*>(residual_out), static_cast<const uint8_t*>(weight), static_cast<uint8_t*>(q),
              sf, static_cast<uint8_t*>(y), rstd, ldx * es, ld_residual * es, ld_residual_out * es, ldq, ld_sf,
              ldy * es, eps, m, k, 1, weight_dtype == DG_DTYPE_BF16};
  const Shape s = shape_for(k, m < 1024 ? 1 : 4);
  p.rows_per_wg = m < 8192 ? 1 : 4;
  const dim3 grid((m + p.rows_per_wg - 1) / p.rows_per_wg);
  if (dtype == DG_DTYPE_BF16) {
    if (ue8m0) launch_fwd<true, true>(p, s, grid, stream);
    else launch_fwd<true, false>(p, s, grid, stream);
  } else {
    if (ue8m0) launch_fwd<false, true>(p, s, grid, stream);
    else launch_fwd<false, false>(p, s, grid, stream);
  }
  return launch_status();
}

size_t dg_get_rms_norm_backward_workspace_size(int m, int k) {
  if (m <= 0 || k <= 0 || k % 128 != 0 || k > norm::kMaxK) return 0;
  return (size_t)norm::bwd_grid(m) * (size_t)k * sizeof(float);
}

dg_status dg_rms_norm_backward(const void* dy, int64_t ld_dy, const void* s, int64_t ld_s, dg_dtype dtype,
                               const void* weight, dg_dtype weight_dtype, const float* rstd, const void* dresidual,
                               int64_t ld_dresidual, void* dx, int64_t ld_dx, float* dw, int accumulate_dw, int m,
                               int k, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  using namespace norm;
  if (m < 0 || k < 0 || (dtype != DG_DTYPE_BF16 && dtype != DG_DTYPE_FP32) ||
      (weight_dtype != DG_DTYPE_BF16 && weight_dtype != DG_DTYPE_FP32))
    return DG_ERROR_INVALID_VALUE;
  if (k % 128 != 0 || k > kMaxK) return DG_ERROR_NOT_SUPPORTED;
  if (k == 0) return DG_SUCCESS;
  if (dw == nullptr || !aligned_to(dw, 16)) return DG_ERROR_INVALID_VALUE;
  const int grid = bwd_grid(m);
  if (m > 0) {
    const int64_t es = dtype == DG_DTYPE_BF16 ? 2 : 4;
    if (!rows_ok(dy, ld_dy, es, k) || !rows_ok(s, ld_s, es, k) || !rows_ok(dx, ld_dx, es, k))
      return DG_ERROR_INVALID_VALUE;
    if (dresidual != nullptr && !rows_ok(dresidual, ld_dresidual, es, k)) return DG_ERROR_INVALID_VALUE;
    if (weight == nullptr || !aligned_to(weight, 16) || rstd == nullptr || !aligned_to(rstd, 4))
      return DG_ERROR_INVALID_VALUE;
    if (workspace == nullptr || !aligned_to(workspace, 256) ||
        workspace_bytes < dg_get_rms_norm_backward_workspace_size(m, k))
      return DG_ERROR_WORKSPACE;
    const BwdParams p{static_cast<const uint8_t*>(dy), static_cast<const uint8_t*>(s),
                      static_cast<const uint8_t*>(weight), static_cast<const uint8_t*>(dresidual), rstd,
                      static_cast<uint8_t*>(dx), static_cast<float*>(workspace), ld_dy * es, ld_s * es,
                      ld_dresidual * es, ld_dx * es, m, k, weight_dtype == DG_DTYPE_BF16};
    const Shape sh = shape_for(k, 4);
    if (dtype == DG_DTYPE_BF16) launch_bwd<true>(p, sh, dim3(grid), stream);
    else launch_bwd<false>(p, sh, dim3(grid), stream);
    const dg_status st = launch_status();
    if (st != DG_SUCCESS) return st;
  }
  hipLaunchKernelGGL(dw_kernel, dim3(k / kDwCols), dim3(256), 0, stream, static_cast<const float*>(workspace), grid, k,
                     dw, accumulate_dw != 0);
  return launch_status();
}

}  // extern "C"
