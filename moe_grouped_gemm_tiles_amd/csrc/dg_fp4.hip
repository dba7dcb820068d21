// dg_fp4.hip -- GEMMs of microscaled 4-bit operands (OCP MXFP4) on gfx950: D = C + A @ B.T, A and B
// E2M1 codes, two to a byte along K, with one E8M0 scale for each row and 32 K values; dense,
// M-grouped contiguous and M-grouped masked.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 takes both operands' scales: lane l holds the 32 values of one
// block of row l % 16, and a byte of its scale register is that block's scale.  So the scales cost
// no arithmetic, and all K accumulates in the matrix cores' FP32 accumulators.
//
//   * A workgroup owns a BM x BN tile and walks K in slabs of 256 values: 128 bytes a row, eight
//     blocks, two scale words.  Direct global -> LDS loads bring the slab's rows of A and B and its
//     scale words; the descriptors end at the last valid row, so rows past it read as zero.  In a last
//     slab that K fills by half, the lanes that hold its second half are pointed past the descriptor.
//   * K order is free as long as A and B agree.  Lane group q = lane / 16 takes blocks 2q and 2q + 1
//     in the slab's two products, so that their scale bytes are one 16-bit LDS read.  16-byte chunk c
//     of row r sits at chunk c ^ f(r), f(r) = (r >> 1 & 1) | (r >> 3 & 1) << 2, which makes those
//     reads free of bank conflicts.
//   * B is the product's first operand, so a lane's four results are four consecutive columns.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "dg.h"
#include "dg_common.hpp"
#include "dg_kernels.hpp"

namespace {

using dg::f32x4;
using dg::i32x4;
using dg::i32x8;

namespace fp4 {

struct Params {
  dg::Params g;      // sizes, strides (A and B in bytes) and outputs, as the FP8 GEMMs have them
  int64_t ld_sfb;    // words between the rows of B's scales
  int kw;            // scale words along K (k / 128)
};

constexpr int kE2M1 = 4;  // operand format code of the scaled MFMA

// x, y: the lane's 16 bytes; byte T of sx / sy scales them.
template <int T>
__device__ __forceinline__ f32x4 mfma(i32x4 x, i32x4 y, f32x4 c, int sx, int sy) {
  const i32x8 a = {x[0], x[1], x[2], x[3], 0, 0, 0, 0}, b = {y[0], y[1], y[2], y[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, kE2M1, kE2M1, T, sx, T, sy);
}

template <int BM, int BN, int WM, int WN, int MODE, bool BF16_OUT, bool HAS_C>
__global__ void __launch_bounds__(WM * WN * 64) gemm_kernel(const Params pp) {
  const dg::Params& p = pp.g;
  constexpr int NW = WM * WN;
  constexpr int TM = BM / WM, TN = BN / WN;
  constexpr int FM = TM / 16, FN = TN / 16;
  constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;
  constexpr int SA_OFF = A_BYTES + B_BYTES, SB_OFF = SA_OFF + 2 * BM * 4;
  constexpr int STAGE = SB_OFF + 2 * BN * 4;
  constexpr int A_LOADS = BM / 8 / NW, B_LOADS = BN / 8 / NW;
  static_assert(A_LOADS * NW * 8 == BM && B_LOADS * NW * 8 == BN, "whole loads");
  static_assert(NW >= 4, "the four scale loads ride on different waves");
  static_assert(BM <= 256 && BN <= 256, "a scale row is one load");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * STAGE];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int r16 = lane & 15, q4 = lane >> 4;
  const int slabs = (pp.kw + 1) >> 1;
  const int tiles_mn = p.tiles_m * p.tiles_n;
  // chunks 2 * q4 and 2 * q4 + 1 of a fragment's row, swizzled (rows of one fragment share r & 15)
  const int f = ((r16 >> 1) & 1) | ((r16 >> 3) << 2);
  const int ch0 = ((2 * q4) ^ f) << 4, ch1 = ((2 * q4 + 1) ^ f) << 4;
  // direct loads: LDS byte 16 * lane of a 1 KiB block (8 rows) is row lane / 8, chunk lane % 8
  const int ld_row = lane >> 3;
  const int vb = dg::xcd_remap(blockIdx.x, gridDim.x);
  for (int unit = vb; unit < p.num_tiles; unit += gridDim.x) {
    int g = 0, t = unit;
    if (MODE == dg::MODE_MASKED) {
      g = t / tiles_mn;
      t -= g * tiles_mn;
    }
    int mb, nb;
    dg::raster<4>(t, p.tiles_m, p.tiles_n, mb, nb);
    const int m0 = mb * BM, n0 = nb * BN;
    int row_end = p.m;
    if (MODE == dg::MODE_MASKED) {
      row_end = min(max(p.grp[g], 0), p.m);
      if (m0 >= row_end) continue;
    } else if (MODE == dg::MODE_CONTIG) {
      g = p.grp[m0];
      if (g < 0 || g >= p.num_groups) continue;
    }
    const uint8_t* A = p.a + (MODE == dg::MODE_MASKED ? g * p.a_gs : 0) + (int64_t)m0 * p.lda;
    const uint8_t* B = p.b + (MODE != dg::MODE_DENSE ? g * p.b_gs : 0) + (int64_t)n0 * p.ldb;
    const float* SA = p.sfa + (MODE == dg::MODE_MASKED ? g * p.sfa_gs : 0) + m0;
    const float* SB = p.sfb + (MODE != dg::MODE_DENSE ? g * p.sfb_gs : 0) + n0;
    const int a_rows = min(row_end - m0, BM), b_rows = min(p.n - n0, BN);

    auto issue = [&](int slab, int stage) {
      uint8_t* base = lds + stage * STAGE;
      const bool half = 2 * slab + 2 > pp.kw;  // the slab's second 128 values are past K
      const auto ra = dg::make_rsrc(A + slab * 128, dg::clamp_bytes(a_rows * p.lda - slab * 128));
      const auto rb = dg::make_rsrc(B + slab * 128, dg::clamp_bytes(b_rows * p.ldb - slab * 128));
#pragma unroll
      for (int i = 0; i < A_LOADS; ++i) {
        const int blk = wave * A_LOADS + i, chunk = (lane & 7) ^ (((ld_row >> 1) & 1) | ((blk & 1) << 2));
        uint32_t off = (uint32_t)((blk * 8 + ld_row) * p.lda) + chunk * 16;
        if (half && chunk >= 4) off = 0x80000000u;
        dg::load_to_lds<16, false>(ra, base + blk * 1024, off);
      }
#pragma unroll
      for (int i = 0; i < B_LOADS; ++i) {
        const int blk = wave * B_LOADS + i, chunk = (lane & 7) ^ (((ld_row >> 1) & 1) | ((blk & 1) << 2));
        uint32_t off = (uint32_t)((blk * 8 + ld_row) * p.ldb) + chunk * 16;
        if (half && chunk >= 4) off = 0x80000000u;
        dg::load_to_lds<16, false>(rb, base + A_BYTES + blk * 1024, off);
      }
      if (wave < 4) {
        const int w = 2 * slab + (wave & 1), rows = wave < 2 ? a_rows : b_rows, bl = wave < 2 ? BM : BN;
        const auto rs = dg::make_rsrc((wave < 2 ? SA + w * p.ld_sfa : SB + w * pp.ld_sfb),
                                      w < pp.kw ? dg::clamp_bytes(rows * 4) : 0u);
        if (lane < bl / 4)
          dg::load_to_lds<16, false>(rs, base + (wave < 2 ? SA_OFF : SB_OFF) + (wave & 1) * bl * 4, lane * 16);
      }
    };

    f32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    __syncthreads();  // the last tile's reads are done
    if (slabs > 0) issue(0, 0);
    for (int it = 0; it < slabs; ++it) {
      __syncthreads();  // slab it has landed (all loads waited for), slab it - 1 has been read
      if (it + 1 < slabs) issue(it + 1, (it + 1) & 1);
      const uint8_t* st = lds + (it & 1) * STAGE;
      i32x4 b0[FN], b1[FN];
      int sb[FN];
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int row = wn * TN + j * 16 + r16;
        b0[j] = *reinterpret_cast<const i32x4*>(st + A_BYTES + row * 128 + ch0);
        b1[j] = *reinterpret_cast<const i32x4*>(st + A_BYTES + row * 128 + ch1);
        sb[j] = *reinterpret_cast<const uint16_t*>(st + SB_OFF + (q4 >> 1) * BN * 4 + row * 4 + (q4 & 1) * 2);
      }
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const int row = wm * TM + i * 16 + r16;
        const i32x4 a0 = *reinterpret_cast<const i32x4*>(st + row * 128 + ch0);
        const i32x4 a1 = *reinterpret_cast<const i32x4*>(st + row * 128 + ch1);
        const int sa = *reinterpret_cast<const uint16_t*>(st + SA_OFF + (q4 >> 1) * BM * 4 + row * 4 + (q4 & 1) * 2);
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = mfma<0>(b0[j], a0, acc[i][j], sb[j], sa);
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = mfma<1>(b1[j], a1, acc[i][j], sb[j], sa);
      }
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int gm = m0 + wm * TM + i * 16 + r16;
      if (gm >= row_end || (MODE == dg::MODE_CONTIG && p.grp[gm] != g)) continue;
      const int64_t drow = (MODE == dg::MODE_MASKED ? g * p.d_gs : 0) + (int64_t)gm * p.ldd;
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int gn = n0 + wn * TN + j * 16 + 4 * q4;
        if (gn < p.n) dg::store_out<BF16_OUT, HAS_C>(p, (int64_t)gm * p.ldc, gn, drow, acc[i][j]);
      }
    }
  }
}

}  // namespace fp4

inline bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline int cdiv(int a, int b) { return (a + b - 1) / b; }

template <int MODE>
dg_status launch(fp4::Params& pp, dg_dtype t, int groups_for_tiles, hipStream_t stream) {
  dg::Params& p = pp.g;
  constexpr int BM = 128, BN = 128;
  p.tiles_m = cdiv(p.m, BM);
  p.tiles_n = cdiv(p.n, BN);
  const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n * groups_for_tiles;
  if (tiles > 0x7fffffff) return DG_ERROR_NOT_SUPPORTED;
  p.num_tiles = static_cast<int>(tiles);
  const int slots = 2 * dg_get_num_cus();
  const int grid = p.num_tiles < slots ? p.num_tiles : slots;
  void (*fn)(fp4::Params);
  if constexpr (MODE == dg::MODE_DENSE) {
    if (p.c != nullptr)
      fn = t == DG_DTYPE_BF16 ? fp4::gemm_kernel<BM, BN, 2, 2, MODE, true, true> : fp4::gemm_kernel<BM, BN, 2, 2, MODE, false, true>;
    else
      fn = t == DG_DTYPE_BF16 ? fp4::gemm_kernel<BM, BN, 2, 2, MODE, true, false> : fp4::gemm_kernel<BM, BN, 2, 2, MODE, false, false>;
  } else {
    fn = t == DG_DTYPE_BF16 ? fp4::gemm_kernel<BM, BN, 2, 2, MODE, true, false> : fp4::gemm_kernel<BM, BN, 2, 2, MODE, false, false>;
  }
  hipLaunchKernelGGL(fn, dim3(grid), dim3(256), 0, stream, pp);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? DG_SUCCESS : dg::record_hip_error(e);
}

// Operand checks shared by the entry points; rows = rows of A (M, M_total or M_max).
dg_status check(const void* a, int64_t lda, const void* sfa, int64_t ld_sfa, const void* b, int64_t ldb, const void* sfb,
                int64_t ld_sfb, const void* d, int64_t ldd, dg_dtype t, int rows, int n, int k) {
  if (rows < 0 || n < 0 || k < 0 || (t != DG_DTYPE_BF16 && t != DG_DTYPE_FP32)) return DG_ERROR_INVALID_VALUE;
  if (k % 128 != 0) return DG_ERROR_NOT_SUPPORTED;
  if (rows == 0 || n == 0) return DG_SUCCESS;  // empty tensors may have no address
  const int64_t es = t == DG_DTYPE_BF16 ? 2 : 4;
  if (d == nullptr || !aligned(d, 16) || ldd < n || (ldd * es) % 16 != 0) return DG_ERROR_INVALID_VALUE;
  if (k > 0) {
    if (a == nullptr || b == nullptr || sfa == nullptr || sfb == nullptr) return DG_ERROR_INVALID_VALUE;
    if (!aligned(a, 16) || !aligned(b, 16) || !aligned(sfa, 16) || !aligned(sfb, 16)) return DG_ERROR_INVALID_VALUE;
    if (lda < k / 2 || ldb < k / 2 || lda % 16 != 0 || ldb % 16 != 0) return DG_ERROR_INVALID_VALUE;
    if (ld_sfa < rows || ld_sfa % 4 != 0 || ld_sfb < n || ld_sfb % 4 != 0) return DG_ERROR_INVALID_VALUE;
    if (lda * 256 >= (1ll << 31) || ldb * 256 >= (1ll << 31)) return DG_ERROR_NOT_SUPPORTED;
  }
  return DG_SUCCESS;
}

fp4::Params params(const void* a, int64_t lda, const int32_t* sfa, int64_t ld_sfa, const void* b, int64_t ldb,
                   const int32_t* sfb, int64_t ld_sfb, void* d, int64_t ldd, int m, int n, int k) {
  fp4::Params pp{};
  dg::Params& p = pp.g;
  p.a = static_cast<const uint8_t*>(a);
  p.b = static_cast<const uint8_t*>(b);
  p.sfa = reinterpret_cast<const float*>(sfa);
  p.sfb = reinterpret_cast<const float*>(sfb);
  p.d = d;
  p.lda = lda;
  p.ldb = ldb;
  p.ldd = ldd;
  p.ld_sfa = ld_sfa;
  p.m = m;
  p.n = n;
  p.k = k;
  p.num_groups = 1;
  p.splits = 1;
  pp.ld_sfb = ld_sfb;
  pp.kw = k / 128;
  return pp;
}

}  // namespace

extern "C" {

size_t dg_get_mxfp4_workspace_size(int m, int n, int k) {
  (void)m;
  (void)n;
  (void)k;
  return 0;
}

dg_status dg_mxfp4_gemm_nt(const void* a, int64_t lda, const int32_t* sfa, int64_t ld_sfa, const void* b, int64_t ldb,
                           const int32_t* sfb, int64_t ld_sfb, const void* c, int64_t ldc, void* d, int64_t ldd,
                           dg_dtype d_dtype, int m, int n, int k, void* workspace, size_t workspace_bytes,
                           hipStream_t stream) {
  (void)workspace;
  (void)workspace_bytes;
  const dg_status st = check(a, lda, sfa, ld_sfa, b, ldb, sfb, ld_sfb, d, ldd, d_dtype, m, n, k);
  if (st != DG_SUCCESS || m == 0 || n == 0) return st;
  const int64_t es = d_dtype == DG_DTYPE_BF16 ? 2 : 4;
  if (c != nullptr && (!aligned(c, 16) || ldc < n || (ldc * es) % 16 != 0)) return DG_ERROR_INVALID_VALUE;
  fp4::Params pp = params(a, lda, sfa, ld_sfa, b, ldb, sfb, ld_sfb, d, ldd, m, n, k);
  pp.g.c = c;
  pp.g.ldc = ldc;
  return launch<dg::MODE_DENSE>(pp, d_dtype, 1, stream);
}

dg_status dg_m_grouped_mxfp4_gemm_nt_contiguous(const void* a, const int32_t* sfa, int64_t ld_sfa, const void* b,
                                                const int32_t* sfb, int64_t ld_sfb, void* d, dg_dtype d_dtype,
                                                const int32_t* m_indices, int m_total, int n, int k, int num_groups,
                                                hipStream_t stream) {
  if (num_groups < 0) return DG_ERROR_INVALID_VALUE;
  const dg_status st = check(a, k / 2, sfa, ld_sfa, b, k / 2, sfb, ld_sfb, d, n, d_dtype, m_total, n, k);
  if (st != DG_SUCCESS) return st;
  if (m_total % 128 != 0) return DG_ERROR_NOT_SUPPORTED;
  if (m_total == 0 || n == 0 || num_groups == 0) return DG_SUCCESS;
  if (m_indices == nullptr || !aligned(m_indices, 4)) return DG_ERROR_INVALID_VALUE;
  fp4::Params pp = params(a, k / 2, sfa, ld_sfa, b, k / 2, sfb, ld_sfb, d, n, m_total, n, k);
  pp.g.grp = m_indices;
  pp.g.num_groups = num_groups;
  pp.g.b_gs = static_cast<int64_t>(n) * (k / 2);
  pp.g.sfb_gs = pp.kw * ld_sfb;
  return launch<dg::MODE_CONTIG>(pp, d_dtype, 1, stream);
}

dg_status dg_m_grouped_mxfp4_gemm_nt_masked(const void* a, const int32_t* sfa, int64_t ld_sfa, const void* b,
                                            const int32_t* sfb, int64_t ld_sfb, void* d, dg_dtype d_dtype,
                                            const int32_t* masked_m, int num_groups, int m_max, int n, int k,
                                            int expected_m, hipStream_t stream) {
  (void)expected_m;
  if (num_groups < 0) return DG_ERROR_INVALID_VALUE;
  const dg_status st = check(a, k / 2, sfa, ld_sfa, b, k / 2, sfb, ld_sfb, d, n, d_dtype, m_max, n, k);
  if (st != DG_SUCCESS) return st;
  if (m_max == 0 || n == 0 || num_groups == 0) return DG_SUCCESS;
  if (masked_m == nullptr || !aligned(masked_m, 4)) return DG_ERROR_INVALID_VALUE;
  fp4::Params pp = params(a, k / 2, sfa, ld_sfa, b, k / 2, sfb, ld_sfb, d, n, m_max, n, k);
  pp.g.grp = masked_m;
  pp.g.num_groups = num_groups;
  pp.g.a_gs = static_cast<int64_t>(m_max) * (k / 2);
  pp.g.sfa_gs = pp.kw * ld_sfa;
  pp.g.b_gs = static_cast<int64_t>(n) * (k / 2);
  pp.g.sfb_gs = pp.kw * ld_sfb;
  pp.g.d_gs = static_cast<int64_t>(m_max) * n;
  return launch<dg::MODE_MASKED>(pp, d_dtype, num_groups, stream);
}

}  // extern "C"
