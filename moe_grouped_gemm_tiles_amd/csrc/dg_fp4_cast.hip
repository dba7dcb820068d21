// dg_fp4_cast.hip -- microscaled 4-bit quantisation of GEMM operands on gfx950: E2M1 codes, one
// power-of-two scale (E8M0) for each row and 32 consecutive K values, the scales written in the
// layout the MXFP4 GEMMs take.
//
//   s    = the smallest power of two with amax <= 6 s (6 = E2M1's largest value; 1 for a block of
//          zeros), held in [2^-127, 2^127]; a block with an Inf or NaN gets the NaN scale and zero codes
//   code = E2M1(x / s), nearest, ties to even; x / s is exact, so this is the only rounding
//   y    = code * s, exact in BF16 (two significant bits)
//
// The scale comes from amax's bits alone: amax = 1.f * 2^E is at most 1.5 * 2^(e + 2) for e = E - 2
// where f <= 0.5 and for e = E - 1 above, which is one addition that carries into the exponent.
// Largest magnitudes are compared as integers, so that Inf and NaN win.  The codes and y are the
// conversion instructions with a scale (checked against the definition for every BF16 value and
// scale byte).
//
// HBM-bound: reads 2 or 4 bytes, writes half a byte, 1/32 and, with y, 2 or 4 per value.  A workgroup owns 16 rows x 512
// columns; a lane takes 8 values of a row, so a wave reads 1 KiB (BF16) runs, its four rows in flight at once, and a block's
// amax is two exchanges among four lanes.  The 4 x 16 scale words go through LDS and leave as 64-byte runs of the transposed
// layout.  8 x 4096 x 7168 BF16 with y, 1.06 GB: 171 us, 6.2 TB/s (32 rows per workgroup 185, 64 rows 207: fewer rows keep a
// workgroup's reads and writes close together in time).
#include <hip/hip_runtime.h>

#include <cstdint>

#include "dg.h"
#include "dg_common.hpp"

namespace {

namespace fp4c {

constexpr int kRows = 16;   // rows per workgroup, kBatch for each wave
constexpr int kCols = 512;  // columns per workgroup (four scale words)
constexpr int kBatch = 4;   // rows a wave has in flight
constexpr int kMaxBlocks = 1 << 23;  // workgroups of a launch and group

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// v with the lanes of each group of four exchanged by a quad permutation.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}
constexpr int kQuadXor1 = 0xB1, kQuadXor2 = 0x4E, kRowRor4 = 0x124, kRowRor8 = 0x128;

// 16-byte accesses, marked as streaming where NT.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
template <bool NT>
__device__ __forceinline__ u32x4 load16(const uint8_t* p) {
  if constexpr (NT) return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
  else return *reinterpret_cast<const u32x4*>(p);
}
template <bool NT, typename T>
__device__ __forceinline__ void store(uint8_t* p, T v) {
  if constexpr (NT) __builtin_nontemporal_store(v, reinterpret_cast<T*>(p));
  else *reinterpret_cast<T*>(p) = v;
}

// Eight values as the conversion instructions take them.
template <bool BF16, bool NT>
struct Eight;
template <bool NT>
struct Eight<true, NT> {
  u32x4 w;
  __device__ __forceinline__ void load(const uint8_t* p) { w = load16<NT>(p); }
  // Bits of the largest magnitude, as FP32.
  __device__ __forceinline__ uint32_t amax() const {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
    uint32_t hi = 0, lo = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      hi = max(hi, v[i] & 0x7fff0000u);
      lo = max(lo, (v[i] << 16) & 0x7fff0000u);
    }
    return max(hi, lo);
  }
  __device__ __forceinline__ uint32_t codes(float s) const {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
    uint32_t r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, v[0]), s, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, v[1]), s, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, v[2]), s, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, v[3]), s, 3);
    return r;
  }
  static __device__ __forceinline__ void store_values(uint8_t* p, uint32_t r, float s, bool nan) {
    u32x4 o;
    o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r, s, 0));
    o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r, s, 1));
    o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r, s, 2));
    o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r, s, 3));
    if (nan) o = u32x4{0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u};
    store<NT>(p, o);
  }
};
template <bool NT>
struct Eight<false, NT> {
  f32x4 lo, hi;
  __device__ __forceinline__ void load(const uint8_t* p) {
    lo = __builtin_bit_cast(f32x4, load16<NT>(p));
    hi = __builtin_bit_cast(f32x4, load16<NT>(p + 16));
  }
  __device__ __forceinline__ uint32_t amax() const {
    const float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = max(a, __float_as_uint(v[i]) & 0x7fffffffu);
    return a;
  }
  __device__ __forceinline__ uint32_t codes(float s) const {
    uint32_t r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, lo.x, lo.y, s, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, lo.z, lo.w, s, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, hi.x, hi.y, s, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, hi.z, hi.w, s, 3);
    return r;
  }
  static __device__ __forceinline__ void store_values(uint8_t* p, uint32_t r, float s, bool nan) {
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(r, s, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(r, s, 1);
    const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(r, s, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(r, s, 3);
    const float q = __uint_as_float(0x7fc00000u);
    store<NT>(p, nan ? f32x4{q, q, q, q} : f32x4{a[0], a[1], b[0], b[1]});
    store<NT>(p + 16, nan ? f32x4{q, q, q, q} : f32x4{c[0], c[1], d[0], d[1]});
  }
};

struct Args {
  const uint8_t* x;
  uint8_t* q;
  int32_t* sf;
  uint8_t* y;
  const int32_t* masked_m;
  int64_t ldx_bytes, ldq, ld_sf, ldy_bytes;
  int m, k, first;  // first: of the rows of each group that this launch takes
};

// Scale byte of a block from the bits of its amax.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  const int e = (int)((amax + 0x3fffffu) >> 23) - 2;
  return amax == 0u ? 127u : (amax >= 0x7f800000u ? 255u : (uint32_t)max(e, 0));
}

template <bool BF16, bool VALUES, bool NT>
__global__ void __launch_bounds__(256) cast_kernel(const Args a) {
  __shared__ uint32_t s_word[4][kRows];
  constexpr int ES = BF16 ? 2 : 4;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int g = blockIdx.y;
  const int col_blocks = (a.k + kCols - 1) / kCols;  // neighbours take the same rows' next columns
  const int row_block = blockIdx.x / col_blocks;
  const int m0 = a.first + row_block * kRows, c0 = (blockIdx.x - row_block * col_blocks) * kCols;
  const int rows = min(a.masked_m != nullptr ? min(max(a.masked_m[g], 0), a.m) : a.m, m0 + kRows);
  if (m0 >= rows) return;
  const int col = c0 + 8 * lane;
  const bool in = col < a.k;
  const int kw = a.k >> 7;
  const uint8_t* x = a.x + (int64_t)g * a.m * a.ldx_bytes + (int64_t)col * ES;
  uint8_t* q = a.q + (int64_t)g * a.m * a.ldq + (col >> 1);
  uint8_t* y = VALUES ? a.y + (int64_t)g * a.m * a.ldy_bytes + (int64_t)col * ES : nullptr;
  static_assert(kRows == 4 * kBatch, "a wave takes its rows at once");
  {
    const int r0 = wave * kBatch;
    Eight<BF16, NT> v[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int row = m0 + r0 + i;
      if (in && row < rows) v[i].load(x + (int64_t)row * a.ldx_bytes);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int row = m0 + r0 + i;
      if (row >= rows) break;
      uint32_t amax = v[i].amax();
      amax = max(amax, dpp<kQuadXor1>(amax));
      amax = max(amax, dpp<kQuadXor2>(amax));
      const uint32_t byte = scale_byte(amax);
      const bool nan = byte == 255u;
      // 2^(byte - 127): the exponent alone (byte 0 is 2^-127, a denormal)
      const float s = byte == 0u ? 0x1p-127f : __uint_as_float((nan ? 127u : byte) << 23);
      uint32_t codes = v[i].codes(s);
      codes = nan ? 0u : codes;
      uint32_t word = byte << (8 * ((lane >> 2) & 3));
      word |= dpp<kRowRor4>(word);
      word |= dpp<kRowRor8>(word);
      if (in) {
        store<NT>(q + (int64_t)row * a.ldq, codes);
        if (VALUES) Eight<BF16, NT>::store_values(y + (int64_t)row * a.ldy_bytes, codes, s, nan);
        if ((lane & 15) == 0) s_word[lane >> 4][r0 + i] = word;
      }
    }
  }
  __syncthreads();
  const int w = tid / kRows, r = tid % kRows;
  const int wk = (c0 >> 7) + w;
  if (w < 4 && wk < kw && m0 + r < rows)
    a.sf[((int64_t)g * kw + wk) * a.ld_sf + m0 + r] = (int32_t)s_word[w][r];
}

}  // namespace fp4c

inline bool aligned_to(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace

extern "C" {

dg_status dg_cast_to_mxfp4(const void* x, int64_t ldx, dg_dtype x_dtype, void* q, int64_t ldq, int32_t* sf,
                           int64_t ld_sf, void* y, int64_t ldy, const int32_t* masked_m, int num_groups, int m, int k,
                           hipStream_t stream) {
  if (m < 0 || k < 0 || num_groups < 0 || (x_dtype != DG_DTYPE_BF16 && x_dtype != DG_DTYPE_FP32))
    return DG_ERROR_INVALID_VALUE;
  if (k % 128 != 0) return DG_ERROR_NOT_SUPPORTED;
  if (m == 0 || k == 0 || num_groups == 0) return DG_SUCCESS;
  const int64_t es = x_dtype == DG_DTYPE_BF16 ? 2 : 4;
  if (x == nullptr || q == nullptr || sf == nullptr) return DG_ERROR_INVALID_VALUE;
  if (!aligned_to(x, 16) || !aligned_to(q, 4) || !aligned_to(sf, 4) || !aligned_to(masked_m, 4))
    return DG_ERROR_INVALID_VALUE;
  if (ldx < k || (ldx * es) % 16 != 0 || ldq < k / 2 || ldq % 4 != 0 || ld_sf < m) return DG_ERROR_INVALID_VALUE;
  if (y != nullptr && (!aligned_to(y, 16) || ldy < k || (ldy * es) % 16 != 0)) return DG_ERROR_INVALID_VALUE;
  if (y == x && ldy != ldx && (m > 1 || num_groups > 1)) return DG_ERROR_INVALID_VALUE;  // rows over other rows not yet read
  const int64_t col_blocks = (static_cast<int64_t>(k) + fp4c::kCols - 1) / fp4c::kCols;
  const int64_t row_blocks = (static_cast<int64_t>(m) + fp4c::kRows - 1) / fp4c::kRows;
  if (k > (1 << 25) || static_cast<int64_t>(m) * k >= (1ll << 36) || num_groups > 65535) return DG_ERROR_NOT_SUPPORTED;
  fp4c::Args a{static_cast<const uint8_t*>(x), static_cast<uint8_t*>(q), sf, static_cast<uint8_t*>(y), masked_m,
               ldx * es, ldq, ld_sf, ldy * es, m, k, 0};
  // operands past the last-level cache's 256 MiB are streamed (smaller ones are left there for their readers: 4099 x 1408 FP32
  // with y, called again and again, takes 12 us, streamed 18)
  const int64_t bytes = static_cast<int64_t>(num_groups) * m * k * (y ? 2 * es + 1 : es + 1);
  const bool nt = bytes > (int64_t)256 << 20;
  void (*fn)(fp4c::Args);
  if (x_dtype == DG_DTYPE_BF16)
    fn = y ? (nt ? fp4c::cast_kernel<true, true, true> : fp4c::cast_kernel<true, true, false>)
           : (nt ? fp4c::cast_kernel<true, false, true> : fp4c::cast_kernel<true, false, false>);
  else
    fn = y ? (nt ? fp4c::cast_kernel<false, true, true> : fp4c::cast_kernel<false, true, false>)
           : (nt ? fp4c::cast_kernel<false, false, true> : fp4c::cast_kernel<false, false, false>);
  // a grid holds fewer than 2^32 threads: rows past its share take another launch
  const int64_t most = fp4c::kMaxBlocks / col_blocks;
  for (int64_t at = 0; at < row_blocks; at += most) {
    a.first = static_cast<int>(at) * fp4c::kRows;
    const int64_t blocks = (row_blocks - at < most ? row_blocks - at : most) * col_blocks;
    hipLaunchKernelGGL(fn, dim3(static_cast<unsigned>(blocks), num_groups), dim3(256), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return dg::record_hip_error(e);
  }
  return DG_SUCCESS;
}

}  // extern "C"
