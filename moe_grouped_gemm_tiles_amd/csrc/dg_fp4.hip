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

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "dg.h"
#include "dg_common.hpp"
#include "dg_internal.h"
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

// A lane's part of a 16-row fragment of a slab: blocks 2q and 2q + 1 of its row, and their two scale bytes.
struct Frag {
  i32x4 lo, hi;
  int s;
};

// Masked groups: the tiles that have rows, numbered through, so that they spread evenly over the workgroups whatever the
// groups' row counts are (numbering all tiles instead leaves the rows that are there to the same few workgroups: 8 rows of 16
// groups in 32-row tiles took 228 us, numbered through 55).  first[i] = the row tiles of the groups before i * per.
constexpr int kGroupSlots = 1024;
struct LiveTiles {
  int first[kGroupSlots + 1];
  int wave_total[8];
};
template <int BM, int NW>
__device__ __forceinline__ void number_live_tiles(LiveTiles& t, const dg::Params& p) {
  constexpr int MINE = kGroupSlots / (NW * 64);
  const int per = (p.num_groups + kGroupSlots - 1) / kGroupSlots;
  const int tid = threadIdx.x, lane = tid & 63;
  int n[MINE], sum = 0;
#pragma unroll
  for (int i = 0; i < MINE; ++i) {
    const int at = (tid * MINE + i) * per;
    n[i] = 0;
    for (int g = at; g < min(at + per, p.num_groups); ++g) n[i] += (min(max(p.grp[g], 0), p.m) + BM - 1) / BM;
    sum += n[i];
  }
  int upto = sum;  // of the wave's lanes up to this one
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == 63) t.wave_total[tid >> 6] = upto;
  __syncthreads();
  int before = upto - sum;
  for (int w = 0; w < (tid >> 6); ++w) before += t.wave_total[w];
#pragma unroll
  for (int i = 0; i < MINE; ++i) {
    t.first[tid * MINE + i] = before;
    before += n[i];
  }
  if (tid == NW * 64 - 1) t.first[kGroupSlots] = before;
  __syncthreads();
}
// The group of live tile `id` (of tiles_n for each row tile), its number within the group and the group's row tiles; false
// past the last one.
template <int BM>
__device__ __forceinline__ bool live_tile(const LiveTiles& t, const dg::Params& p, int id, int& g, int& local, int& tiles_m) {
  const __attribute__((address_space(4))) int32_t* grp = (const __attribute__((address_space(4))) int32_t*)p.grp;
  const int per = (p.num_groups + kGroupSlots - 1) / kGroupSlots;
  const int row_tile = id / p.tiles_n;
  if (row_tile >= __builtin_amdgcn_readfirstlane(t.first[kGroupSlots])) return false;
  int at = 0;  // the last slot that starts at or before row_tile (of empty ones the last: it is the one with rows)
  for (int step = kGroupSlots / 2; step >= 1; step >>= 1)
    if (__builtin_amdgcn_readfirstlane(t.first[at + step]) <= row_tile) at += step;
  int before = __builtin_amdgcn_readfirstlane(t.first[at]);
  for (g = at * per;; ++g) {
    if (g >= p.num_groups) return false;
    tiles_m = (min(max(grp[g], 0), p.m) + BM - 1) / BM;
    if (row_tile < before + tiles_m) break;
    before += tiles_m;
  }
  local = id - before * p.tiles_n;
  return true;
}

// One persistent kernel for every entry point.  The schedule of a slab is the FP8 GEMM's: the operand with fewer fragments
// per wave ("outer") stays in registers for the slab, the other ("inner") is streamed from LDS; the last HOLD inner fragments
// are held back, so that after the slab's one barrier, placed between part 1 and part 2, the matrix cores run from registers
// while the next slab's outer fragments are read and the loads of the slab after it go out.  Each step is two MFMAs on an
// accumulator, the first halves of a fragment's products before the second ones, so that none waits for the one before.
// Bound by the matrix cores' schedule: 4096 x 7168 x 16384 takes 218 us, 4.4 PFLOP/s, with them 0.53 busy at 1.98 GHz (the
// power limit; the peak is 10 PFLOP/s at 2.4), 4096 x 8192 x 16384 240 us, 4.6 PFLOP/s; contiguous 8 x 4096 x 7168 3.9 PFLOP/s,
// masked 16 x 4096 x 7168 with 103 rows a group on average 68 us (its weights alone are 40 us of HBM).
template <int BM, int BN, int WM, int WN, int MODE, bool BF16_OUT, bool HAS_C>
__global__ void __launch_bounds__(WM * WN * 64) gemm_kernel(const Params pp) {
  const dg::Params& p = pp.g;
  constexpr int NW = WM * WN;
  constexpr int TM = BM / WM, TN = BN / WN;
  constexpr int FM = TM / 16, FN = TN / 16;
  constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;
  constexpr int SA_OFF = A_BYTES + B_BYTES, SB_OFF = SA_OFF + 2 * BM * 4;
  constexpr int STAGE = (SB_OFF + 2 * BN * 4 + 255) / 256 * 256;
  constexpr int A_TOTAL = BM / 8, B_TOTAL = BN / 8;  // 1 KiB (8-row) direct loads of a slab
  constexpr int A_LOADS = (A_TOTAL + NW - 1) / NW, B_LOADS = (B_TOTAL + NW - 1) / NW, LOADS = A_LOADS + B_LOADS;
  constexpr bool A_OUTER = FM < FN;
  constexpr int NO = A_OUTER ? FM : FN, NI = A_OUTER ? FN : FM;
  constexpr int HOLD = 2, FIRST = NI - HOLD;
  // the first half of a slab's loads goes out in part 2 of the slab two before it, the rest in the next part 1
  constexpr int P1L = LOADS / 2, P2L = LOADS - P1L;
  static_assert(TM % 16 == 0 && TN % 16 == 0 && BM % 8 == 0 && BN % 8 == 0, "whole MFMA tiles and loads");
  static_assert(NW >= 4, "the four scale loads ride on different waves");
  static_assert(BM <= 256 && BN <= 256, "a scale row is one load");
  static_assert(FIRST >= HOLD && NO >= 2 && P2L <= 2 * NO * HOLD && P1L <= 2 * NO * FIRST, "two-part slab schedule");
  static_assert(MODE != dg::MODE_CONTIG || BM == 128 || BM == 256, "contiguous tiles cover one or two 128-row blocks");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * STAGE];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int r16 = lane & 15, q4 = lane >> 4;
  const int slabs = (pp.kw + 1) >> 1;
  __shared__ LiveTiles live;
  if constexpr (MODE == dg::MODE_MASKED) number_live_tiles<BM, NW>(live, p);
  // chunks 2 * q4 and 2 * q4 + 1 of a fragment's row, swizzled (the rows of a fragment share r16)
  const int f = ((r16 >> 1) & 1) | ((r16 >> 3) << 2);
  const int ch0 = ((2 * q4) ^ f) << 4, ch1 = ((2 * q4 + 1) ^ f) << 4;
  // direct loads: LDS byte 16 * lane of a 1 KiB block is row lane / 8, chunk lane % 8
  const int ld_row = lane >> 3;
  // (masked: the loads are issued where the compiler does not see them; in a kernel that also loads into registers and reads
  // other LDS, it has each LDS read wait for all of them)

  // Work units: (tile, pass); a contiguous tile whose two 128-row halves belong to different groups takes one pass per group.
  // Group data is read through the constant address space: scalar loads do not share the vector-memory counter with the
  // slabs in flight.
  const __attribute__((address_space(4))) int32_t* grp_s = (const __attribute__((address_space(4))) int32_t*)p.grp;
  struct Unit {
    int tile, more, g, halves, m0, n0, row_end;  // tile < 0: no unit; more: a second pass follows; halves: whose rows are g's
  };
  auto find_unit = [&](int tile, int pass) {
    Unit u;
    u.tile = -1;
    for (; tile < p.num_tiles; tile += gridDim.x, pass = 0) {
      int g = 0, t = tile, tiles_m = p.tiles_m;
      if constexpr (MODE == dg::MODE_MASKED) {
        if (!live_tile<BM>(live, p, tile, g, t, tiles_m)) break;
      }
      int mb, nb;
      dg::raster<4>(t, tiles_m, p.tiles_n, mb, nb);
      const int m0 = mb * BM;
      int row_end = p.m, halves = 3, more = 0;
      if (MODE == dg::MODE_MASKED) {
        row_end = min(max(grp_s[g], 0), p.m);
      } else if (MODE == dg::MODE_CONTIG) {
        int g0 = grp_s[m0];
        int g1 = (BM == 256 && m0 + 128 < p.m) ? grp_s[m0 + 128] : -1;
        if (g0 < 0 || g0 >= p.num_groups) g0 = -1;
        if (g1 < 0 || g1 >= p.num_groups) g1 = -1;
        if (g0 < 0 && g1 < 0) continue;
        if (g0 < 0) g0 = g1;
        if (g1 < 0) g1 = g0;
        more = pass == 0 && g0 != g1;
        g = pass == 0 ? g0 : g1;
        halves = (g0 == g ? 1 : 0) | (g1 == g ? 2 : 0);
      }
      u.tile = tile;
      u.more = more;
      u.g = g;
      u.halves = halves;
      u.m0 = m0;
      u.n0 = nb * BN;
      u.row_end = row_end;
      break;
    }
    return u;
  };
  auto next_unit = [&](const Unit& u) {
    return u.more ? find_unit(u.tile, 1) : find_unit(u.tile + (int)gridDim.x, 0);
  };

  // A unit's descriptors, fixed over K: slab, block and scale row are part of the offsets.  Each ends at the unit's last row
  // (its last scale), below 2^31, so that offsets from kPast on read zero.
  constexpr uint32_t kPast = 0x80000000u;
  struct Src {
    __amdgpu_buffer_rsrc_t ra, rb, rs;  // rs: the scales that this wave loads, A's on waves 0 and 1, B's on 2 and 3
  };
  const uint32_t ld_s = (uint32_t)(wave < 2 ? p.ld_sfa : pp.ld_sfb) * 4;
  auto src_of = [&](const Unit& u) {
    Src r;
    // (rows past masked_m are read as zeros, without memory)
    const int a_rows = min(u.row_end - u.m0, BM), b_rows = min(p.n - u.n0, BN);
    r.ra = dg::make_rsrc(p.a + (MODE == dg::MODE_MASKED ? u.g * p.a_gs : 0) + (int64_t)u.m0 * p.lda, (uint32_t)(a_rows * p.lda));
    r.rb = dg::make_rsrc(p.b + (MODE != dg::MODE_DENSE ? u.g * p.b_gs : 0) + (int64_t)u.n0 * p.ldb, (uint32_t)(b_rows * p.ldb));
    const float* s = wave < 2 ? p.sfa + (MODE == dg::MODE_MASKED ? u.g * p.sfa_gs : 0) + u.m0
                              : p.sfb + (MODE != dg::MODE_DENSE ? u.g * p.sfb_gs : 0) + u.n0;
    r.rs = dg::make_rsrc(s, pp.kw > 0 ? (uint32_t)(pp.kw - 1) * ld_s + 4u * (wave < 2 ? a_rows : b_rows) : 0u);
    return r;
  };

  // Direct loads: the lane's row and chunk within an 8-row block; blocks alternate in the swizzle's upper bit.
  const int chunk0 = (lane & 7) ^ ((ld_row >> 1) & 1);
  const uint32_t a_off = (uint32_t)(ld_row * p.lda) + chunk0 * 16, b_off = (uint32_t)(ld_row * p.ldb) + chunk0 * 16;
  const uint32_t a_blk = (uint32_t)(8 * p.lda), b_blk = (uint32_t)(8 * p.ldb);
  const uint32_t odd_flip = chunk0 >= 4 ? (uint32_t)-64 : 64u;  // from chunk c to c ^ 4
  // A slab past K is loaded too, from offsets that read zero, so that each slab issues the same loads; of a slab that K
  // fills by half, so are the lanes that hold the second half (chunk >= 4).
  auto load16 = [&](__amdgpu_buffer_rsrc_t r, uint8_t* to, uint32_t off, int blk, uint32_t blk_bytes, int slab) {
    const bool odd = blk & 1;
    uint32_t at = slab < slabs ? (uint32_t)blk * blk_bytes + (uint32_t)slab * 128 : kPast;
    asm volatile("" : "+s"(at));  // added here, not kept as one sum per load in registers
    uint32_t v = (odd ? off + odd_flip : off) + at;
    if (2 * slab + 2 > pp.kw && ((chunk0 >= 4) != odd)) v = kPast;
    dg::load_to_lds<16, MODE == dg::MODE_MASKED>(r, to, v);
  };
  auto issue_load = [&](const Src& r, int slab, int stage, int idx) {
    uint8_t* base = lds + stage * STAGE;
    if (idx < A_LOADS) {
      const int blk = wave * A_LOADS + idx;
      if (A_LOADS * NW == A_TOTAL || blk < A_TOTAL) load16(r.ra, base + blk * 1024, a_off, blk, a_blk, slab);
    } else {
      const int blk = wave * B_LOADS + idx - A_LOADS;
      if (B_LOADS * NW == B_TOTAL || blk < B_TOTAL) load16(r.rb, base + A_BYTES + blk * 1024, b_off, blk, b_blk, slab);
    }
    if (idx == 0 && wave < 4) {
      const int w = 2 * slab + (wave & 1), len = wave < 2 ? BM : BN;
      if (lane < len / 4)
        dg::load_to_lds<16, MODE == dg::MODE_MASKED>(r.rs, base + (wave < 2 ? SA_OFF : SB_OFF) + (wave & 1) * len * 4,
                                   (w < pp.kw ? (uint32_t)w * ld_s : kPast) + lane * 16);
    }
  };
  auto issue_slab = [&](const Src& r, int slab, int stage) {
#pragma unroll
    for (int idx = 0; idx < LOADS; ++idx) issue_load(r, slab, stage, idx);
  };

  const uint8_t* As0 = lds + (wm * TM + r16) * 128;
  const uint8_t* Bs0 = lds + A_BYTES + (wn * TN + r16) * 128;
  const uint8_t* Sa0 = lds + SA_OFF + (q4 >> 1) * BM * 4 + (wm * TM + r16) * 4 + (q4 & 1) * 2;
  const uint8_t* Sb0 = lds + SB_OFF + (q4 >> 1) * BN * 4 + (wn * TN + r16) * 4 + (q4 & 1) * 2;
  auto read_frag = [&](const uint8_t* rows, const uint8_t* scales, int i) {
    Frag r;
    r.lo = *reinterpret_cast<const i32x4*>(rows + i * 2048 + ch0);
    r.hi = *reinterpret_cast<const i32x4*>(rows + i * 2048 + ch1);
    r.s = *reinterpret_cast<const uint16_t*>(scales + i * 64);
    return r;
  };
  const uint8_t *Is0 = A_OUTER ? Bs0 : As0, *Os0 = A_OUTER ? As0 : Bs0;
  const uint8_t *Si0 = A_OUTER ? Sb0 : Sa0, *So0 = A_OUTER ? Sa0 : Sb0;

  const int vb = dg::xcd_remap(blockIdx.x, gridDim.x);
  Unit u = find_unit(vb, 0), nx;
  bool pre = false;  // slabs 0 and 1 of this unit have been issued
  while (u.tile >= 0) {
    const int g = u.g, m0 = u.m0, n0 = u.n0, row_end = u.row_end;
    const int wrow0 = m0 + wm * TM;
    bool wave_live = wrow0 < row_end;
    if (MODE == dg::MODE_CONTIG && BM == 256) wave_live = wave_live && (u.halves >> ((wm * TM) >> 7) & 1);
    const Src sr = src_of(u);
    f32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto mma = [&](int o, int n, int half, const Frag& x, const Frag& y) {
      const int i = A_OUTER ? o : n, j = A_OUTER ? n : o;
      const Frag &b = A_OUTER ? y : x, &a = A_OUTER ? x : y;
      if (half == 0) acc[i][j] = mfma<0>(b.lo, a.lo, acc[i][j], b.s, a.s);
      else acc[i][j] = mfma<1>(b.hi, a.hi, acc[i][j], b.s, a.s);
    };
    if (slabs > 0) {
      if (!pre) {
        issue_slab(sr, 0, 0);
        dg::wait_vmcnt<0>();
      } else {
        dg::wait_vmcnt<0>();
      }
      dg::stage_barrier();
      if (!pre) issue_slab(sr, 1, 1);
      dg::debug_fence();
      Frag fo[NO], fh[HOLD];
      fo[0] = read_frag(Os0, So0, 0);
      Frag fi = read_frag(Is0, Si0, 0), fi_next = fi;
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int o = 1; o < NO; ++o) {
        fo[o] = read_frag(Os0, So0, o);
        __builtin_amdgcn_sched_barrier(0);
      }
      for (int it = 0; it < slabs; ++it) {
        const int cur = it & 1, nxt = cur ^ 1;
        const uint8_t *Is = Is0 + cur * STAGE, *Si = Si0 + cur * STAGE;
        // the last P1L loads of slab it + 1 (slab 1 went out whole)
        const bool late = it > 0;
        if (wave_live) {
#pragma unroll
          for (int n = 0; n < FIRST; ++n) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int o = 0; o < NO; ++o) {
                const int t = (n * 2 + h) * NO + o;
                if (h == 0 && o == 0 && n + 1 < FIRST) fi_next = read_frag(Is, Si, n + 1);
                if (h == 1 && o == 0 && n < HOLD) fh[n] = read_frag(Is, Si, FIRST + n);
                mma(o, n, h, fo[o], fi);
                if (t % 2 == 0 && t / 2 < P1L && late) issue_load(sr, it + 1, nxt, P2L + t / 2);
              }
            if (n + 1 < FIRST) fi = fi_next;
            __builtin_amdgcn_sched_barrier(0);
          }
        } else if (late) {
#pragma unroll
          for (int idx = P2L; idx < LOADS; ++idx) issue_load(sr, it + 1, nxt, idx);
        }
        dg::debug_fence();
        dg::wait_vmcnt<0>();  // slab it + 1 has landed (this wave's part of it)
        dg::stage_barrier();
        if (wave_live) {
          // (after the last slab the reads of the next stage are stale and unused)
#pragma unroll
          for (int o = 0; o < NO; ++o) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int n = 0; n < HOLD; ++n) {
                const int t = (o * 2 + h) * HOLD + n;
                mma(o, FIRST + n, h, fo[o], fh[n]);
                if (t % 2 == 0 && t / 2 < P2L) issue_load(sr, it + 2, cur, t / 2);
              }
            fo[o] = read_frag(Os0 + nxt * STAGE, So0 + nxt * STAGE, o);
            if (o == 0) fi = read_frag(Is0 + nxt * STAGE, Si0 + nxt * STAGE, 0);
            __builtin_amdgcn_sched_barrier(0);
          }
#pragma unroll
          for (int idx = NO * HOLD; idx < P2L; ++idx) issue_load(sr, it + 2, cur, idx);
        } else {
#pragma unroll
          for (int idx = 0; idx < P2L; ++idx) issue_load(sr, it + 2, cur, idx);
        }
        dg::debug_fence();
      }
    }
    dg::stage_barrier();  // all LDS reads of this unit are done before the next unit's loads
    dg::debug_fence();

    // Contiguous: the group of each row this lane stores, loaded before the next unit's slabs (the vector-memory counter
    // completes in order), at a clamped row, so that no load sits in a branch.
    int row_grp[MODE == dg::MODE_CONTIG ? FM : 1];
    if constexpr (MODE == dg::MODE_CONTIG) {
#pragma unroll
      for (int i = 0; i < FM; ++i) row_grp[i] = p.grp[min(wrow0 + r16 + i * 16, row_end - 1)];
      asm volatile("" ::: "memory");
    }
    // The next unit's first two slabs go out before this unit's stores (slabs past K, which read nothing, if there is none).
    nx = next_unit(u);
    pre = nx.tile >= 0;
    const Src ns = src_of(pre ? nx : u);
    issue_slab(ns, pre ? 0 : slabs, 0);
    issue_slab(ns, pre ? 1 : slabs + 1, 1);
    asm volatile("" ::: "memory");
    if (wave_live) {
      int row0 = wrow0 + r16;
      asm volatile("" : "+v"(row0));  // row addresses are worked out here, not above the K loop
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const int gm = row0 + i * 16;
        bool row_ok = gm < row_end;
        if constexpr (MODE == dg::MODE_CONTIG) row_ok = row_ok && row_grp[i] == g;
        const int64_t drow = (MODE == dg::MODE_MASKED ? g * p.d_gs : 0) + (int64_t)gm * p.ldd;
        const int64_t crow = (int64_t)gm * p.ldc;
        if constexpr (BF16_OUT) {
          // Column fragments j, j + 1: a permlane16 swap per pair of words leaves each lane eight consecutive columns, one
          // 16-byte store (as in the FP8 GEMM).  C is added in the MFMA layout first.
#pragma unroll
          for (int j = 0; j + 1 < FN; j += 2) {
            if (HAS_C && row_ok) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int gc = n0 + wn * TN + (j + h) * 16 + 4 * q4;
                if (gc < p.n) dg::add_c_bf16(p, crow, gc, acc[i][j + h]);
              }
            }
            const auto s0 = __builtin_amdgcn_permlane16_swap(dg::bf16x2_rne_bits(acc[i][j][0], acc[i][j][1]),
                                                             dg::bf16x2_rne_bits(acc[i][j + 1][0], acc[i][j + 1][1]), false, false);
            const auto s1 = __builtin_amdgcn_permlane16_swap(dg::bf16x2_rne_bits(acc[i][j][2], acc[i][j][3]),
                                                             dg::bf16x2_rne_bits(acc[i][j + 1][2], acc[i][j + 1][3]), false, false);
            const int gn = n0 + wn * TN + (j + (q4 & 1)) * 16 + 8 * (q4 >> 1);
            if (!row_ok || gn >= p.n) continue;
            uint16_t* D = reinterpret_cast<uint16_t*>(p.d) + drow + gn;
            const uint32_t w[4] = {s0[0], s1[0], s0[1], s1[1]};
            if (gn + 8 <= p.n) {
              *reinterpret_cast<uint4*>(D) = make_uint4(w[0], w[1], w[2], w[3]);
            } else {
#pragma unroll
              for (int c = 0; c < 8; ++c)
                if (gn + c < p.n) D[c] = (uint16_t)(w[c >> 1] >> (16 * (c & 1)));
            }
          }
          if constexpr (FN % 2 == 1) {
            const int gn = n0 + wn * TN + (FN - 1) * 16 + 4 * q4;
            if (row_ok && gn < p.n) dg::store_out<BF16_OUT, HAS_C>(p, crow, gn, drow, acc[i][FN - 1]);
          }
        } else {
          if (!row_ok) continue;
#pragma unroll
          for (int j = 0; j < FN; ++j) {
            const int gn = n0 + wn * TN + j * 16 + 4 * q4;
            if (gn < p.n) dg::store_out<BF16_OUT, HAS_C>(p, crow, gn, drow, acc[i][j]);
          }
        }
      }
    }
    asm volatile("" ::: "memory");  // every store precedes the next unit's first wait
    dg::debug_fence();
    u = nx;
  }
  dg::wait_vmcnt<0>();  // no direct load into this workgroup's LDS outlives it
}

// For calls that wait for memory rather than for the matrix cores: few rows, so that the reading of B is the work, or few
// tiles.  BM x 128 tiles (BM = 32, 64 or 128) on four or eight waves, a ring of STAGES slabs in all of a CU's LDS and
// counted waits, so that STAGES - 1 slabs are always on their way (the 256-row tile waits for the slab it has just asked
// for unless its products take as long as a memory access: 8 rows of 16 experts of 4096 x 7168 took 77 us with it).  Dense
// calls split K over workgroups: each writes its FP32 partial tile to the workspace and counts itself; the one that
// completes a tile adds the partials in the order of the splits, so the result does not depend on who comes last.  Bound by
// memory: 5 x 7168 x 16384 (62 MB) 16 us, 128 x 7168 x 16384 25 us, 512 x 4096 x 7168 19 us; 8 rows of 16 experts of
// 4096 x 7168 (249 MB) 50 us.
template <int BM, int WM, int STAGES, int MODE, bool BF16_OUT, bool HAS_C>
__global__ void __launch_bounds__(WM * 256) stream_kernel(const Params pp) {
  const dg::Params& p = pp.g;
  constexpr int BN = 128, WN = 4, NW = WM * WN, TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
  constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;
  constexpr int SA_OFF = A_BYTES + B_BYTES, SB_OFF = SA_OFF + 2 * BM * 4;
  constexpr int STAGE = (SB_OFF + 2 * BN * 4 + 255) / 256 * 256;
  constexpr int A_LOADS = BM / 8 / NW, B_LOADS = BN / 8 / NW, LOADS = A_LOADS + B_LOADS + 1;  // and one of scales
  static_assert(A_LOADS * NW * 8 == BM && B_LOADS * NW * 8 == BN, "the same loads on each wave");
  static_assert((STAGES - 2) * LOADS < 64, "counted waits");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[STAGES * STAGE];
  __shared__ int s_last;
  __shared__ LiveTiles live;
  if constexpr (MODE == dg::MODE_MASKED) number_live_tiles<BM, NW>(live, p);

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int r16 = lane & 15, q4 = lane >> 4, ld_row = lane >> 3;
  const int all_slabs = (pp.kw + 1) >> 1;
  const int tiles_mn = p.tiles_m * p.tiles_n;
  const int f = ((r16 >> 1) & 1) | ((r16 >> 3) << 2);
  const int ch0 = ((2 * q4) ^ f) << 4, ch1 = ((2 * q4 + 1) ^ f) << 4;
  const __attribute__((address_space(4))) int32_t* grp_s = (const __attribute__((address_space(4))) int32_t*)p.grp;

  constexpr uint32_t kPast = 0x80000000u;  // from here on every descriptor reads zero
  const bool a_scales = wn < 2;  // waves wn = 0, 1 load A's two scale rows of a slab, 2 and 3 B's; wm halves a row
  const uint32_t ld_s = (uint32_t)(a_scales ? p.ld_sfa : pp.ld_sfb) * 4;
  const int chunk0 = (lane & 7) ^ ((ld_row >> 1) & 1);
  const uint32_t a_off = (uint32_t)(ld_row * p.lda) + chunk0 * 16, b_off = (uint32_t)(ld_row * p.ldb) + chunk0 * 16;
  const uint32_t a_blk = (uint32_t)(8 * p.lda), b_blk = (uint32_t)(8 * p.ldb);
  const uint32_t odd_flip = chunk0 >= 4 ? (uint32_t)-64 : 64u;

  struct Unit {
    int tile, g, m0, n0, row_end, begin, end, split, tmn;  // tile < 0: no unit
  };
  auto find_unit = [&](int tile) {
    Unit u;
    u.tile = -1;
    for (; tile < p.num_tiles; tile += gridDim.x) {
      int g = 0, t = tile, split = 0;
      int tiles_m = p.tiles_m;
      if constexpr (MODE == dg::MODE_MASKED) {
        if (!live_tile<BM>(live, p, tile, g, t, tiles_m)) break;
      }
      if (MODE == dg::MODE_DENSE) split = t / tiles_mn, t -= split * tiles_mn;
      int mb, nb;
      dg::raster<4>(t, tiles_m, p.tiles_n, mb, nb);
      u.m0 = mb * BM;
      u.row_end = MODE == dg::MODE_MASKED ? min(max(grp_s[g], 0), p.m) : p.m;
      u.tile = tile;
      u.g = g;
      u.n0 = nb * BN;
      u.begin = split * p.slabs_per_split;
      u.end = min(all_slabs, u.begin + p.slabs_per_split);
      u.split = split;
      u.tmn = t;
      break;
    }
    return u;
  };
  struct Src {
    __amdgpu_buffer_rsrc_t ra, rb, rs;
  };
  auto src_of = [&](const Unit& u) {
    Src r;
    const int a_rows = min(u.row_end - u.m0, BM), b_rows = min(p.n - u.n0, BN);
    r.ra = dg::make_rsrc(p.a + (MODE == dg::MODE_MASKED ? u.g * p.a_gs : 0) + (int64_t)u.m0 * p.lda, (uint32_t)(a_rows * p.lda));
    r.rb = dg::make_rsrc(p.b + (MODE != dg::MODE_DENSE ? u.g * p.b_gs : 0) + (int64_t)u.n0 * p.ldb, (uint32_t)(b_rows * p.ldb));
    const float* s = a_scales ? p.sfa + (MODE == dg::MODE_MASKED ? u.g * p.sfa_gs : 0) + u.m0
                              : p.sfb + (MODE != dg::MODE_DENSE ? u.g * p.sfb_gs : 0) + u.n0;
    r.rs = dg::make_rsrc(s, (uint32_t)(pp.kw - 1) * ld_s + 4u * (a_scales ? a_rows : b_rows));
    return r;
  };
  auto load16 = [&](__amdgpu_buffer_rsrc_t r, uint8_t* to, uint32_t off, int blk, uint32_t blk_bytes, int slab, bool live) {
    const bool odd = blk & 1;
    uint32_t at = live ? (uint32_t)blk * blk_bytes + (uint32_t)slab * 128 : kPast;
    asm volatile("" : "+s"(at));
    uint32_t v = (odd ? off + odd_flip : off) + at;
    if (2 * slab + 2 > pp.kw && ((chunk0 >= 4) != odd)) v = kPast;
    dg::load_to_lds<16, true>(r, to, v);
  };
  // Slab number `slab` of K into its stage; one that is not live is loaded from offsets that read zero.
  auto issue = [&](const Src& r, int slab, int stage, bool live) {
    uint8_t* base = lds + stage * STAGE;
#pragma unroll
    for (int i = 0; i < B_LOADS; ++i) {
      const int blk = wave * B_LOADS + i;
      load16(r.rb, base + A_BYTES + blk * 1024, b_off, blk, b_blk, slab, live);
    }
#pragma unroll
    for (int i = 0; i < A_LOADS; ++i) {
      const int blk = wave * A_LOADS + i;
      load16(r.ra, base + blk * 1024, a_off, blk, a_blk, slab, live);
    }
    const int w = 2 * slab + (wn & 1), len = a_scales ? BM : BN, part = len * 4 / WM;
    if (lane < part / 16)
      dg::load_to_lds<16, true>(r.rs, base + (a_scales ? SA_OFF : SB_OFF) + (wn & 1) * len * 4 + wm * part,
                                (live && w < pp.kw ? (uint32_t)w * ld_s : kPast) + wm * part + lane * 16);
  };

  const uint8_t* As0 = lds + (wm * TM + r16) * 128;
  const uint8_t* Bs0 = lds + A_BYTES + (wn * TN + r16) * 128;
  const uint8_t* Sa0 = lds + SA_OFF + (q4 >> 1) * BM * 4 + (wm * TM + r16) * 4 + (q4 & 1) * 2;
  const uint8_t* Sb0 = lds + SB_OFF + (q4 >> 1) * BN * 4 + (wn * TN + r16) * 4 + (q4 & 1) * 2;
  auto read_frag = [&](const uint8_t* rows, const uint8_t* scales, int i) {
    Frag r;
    r.lo = *reinterpret_cast<const i32x4*>(rows + i * 2048 + ch0);
    r.hi = *reinterpret_cast<const i32x4*>(rows + i * 2048 + ch1);
    r.s = *reinterpret_cast<const uint16_t*>(scales + i * 64);
    return r;
  };

  Unit u = find_unit(dg::xcd_remap(blockIdx.x, gridDim.x)), nx;
  bool pre = false;
  while (u.tile >= 0) {
    const int g = u.g, m0 = u.m0, n0 = u.n0, row_end = u.row_end, slabs = u.end - u.begin;
    const Src sr = src_of(u);
    f32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (!pre) {
#pragma unroll
      for (int i = 0; i < STAGES - 1; ++i) issue(sr, u.begin + i, i, i < slabs);
    }
    int stage = 0, fill = STAGES - 1;
    for (int it = 0; it < slabs; ++it) {
      // this wave's part of slab it has landed (with stores in between, all of what is on its way)
      if (pre && it == 0) dg::wait_vmcnt<0>();
      else dg::wait_vmcnt<(STAGES - 2) * LOADS>();
      dg::stage_barrier();  // everybody's; and slab it - 1 has been read, so its stage is free
      issue(sr, u.begin + it + STAGES - 1, fill, it + STAGES - 1 < slabs);
      const int at = stage * STAGE;
      // all fragments first, so that their latency passes once a slab (rows that are not there too)
      Frag a[FM], b[FN];
#pragma unroll
      for (int j = 0; j < FN; ++j) b[j] = read_frag(Bs0 + at, Sb0 + at, j);
#pragma unroll
      for (int i = 0; i < FM; ++i) a[i] = read_frag(As0 + at, Sa0 + at, i);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = mfma<0>(b[j].lo, a[i].lo, acc[i][j], b[j].s, a[i].s);
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = mfma<1>(b[j].hi, a[i].hi, acc[i][j], b[j].s, a[i].s);
      stage = stage + 1 == STAGES ? 0 : stage + 1;
      fill = fill + 1 == STAGES ? 0 : fill + 1;
      dg::debug_fence();
    }
    dg::stage_barrier();  // all LDS reads of this unit are done before the next unit's loads
    nx = find_unit(u.tile + (int)gridDim.x);
    pre = nx.tile >= 0;
    if (pre) {
      dg::wait_vmcnt<0>();  // (the last slabs' empty loads write to the stages too)
      const Src ns = src_of(nx);
#pragma unroll
      for (int i = 0; i < STAGES - 1; ++i) issue(ns, nx.begin + i, i, i < nx.end - nx.begin);
    }

    bool finish = true;
    if (MODE == dg::MODE_DENSE && p.splits > 1) {
      // Partials go through device-scope accesses (sc1), so that workgroups on different XCDs may share a tile; one is
      // complete once its stores have been acknowledged.
      constexpr int SC1 = 16;
      constexpr int64_t TILE = (int64_t)BM * BN;
      const uint32_t loff = (uint32_t)(wave * FM * FN * 64 + lane) * 16;
      auto part = [&](int s) { return dg::make_rsrc(p.ws + ((int64_t)s * tiles_mn + u.tmn) * TILE, (uint32_t)(TILE * 4)); };
      {
        const auto rw = part(u.split);
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j)
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(i32x4, acc[i][j]), rw, loff + (i * FN + j) * 1024, 0, SC1);
      }
      dg::wait_vmcnt<0>();
      __syncthreads();
      if (tid == 0) {
        const uint32_t arrived = __hip_atomic_fetch_add(p.ctr + u.tmn, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1u;
        const int last = arrived >= (uint32_t)p.splits;
        if (last) __hip_atomic_store(p.ctr + u.tmn, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        s_last = last;
      }
      __syncthreads();
      finish = s_last != 0;
      if (finish) {
        constexpr int RD = BM == 32 ? 8 : (BM == 64 ? 4 : 2);  // partials in flight
        f32x4 buf[RD][FM][FN];
        for (int s0 = 0; s0 < p.splits; s0 += RD) {
#pragma unroll
          for (int r = 0; r < RD; ++r) {
            const auto rs = s0 + r < p.splits ? part(s0 + r) : dg::make_rsrc(p.ws, 0u);
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
              for (int j = 0; j < FN; ++j)
                buf[r][i][j] = __builtin_bit_cast(
                    f32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, loff + (i * FN + j) * 1024, 0, SC1));
          }
#pragma unroll
          for (int r = 0; r < RD; ++r)
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
              for (int j = 0; j < FN; ++j)  // (partials past the last are zeros)
                acc[i][j] = s0 + r == 0 ? buf[r][i][j] : acc[i][j] + buf[r][i][j];
        }
      }
    }
    if (finish) {
      int row0 = m0 + wm * TM + r16;
      asm volatile("" : "+v"(row0));
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const int gm = row0 + i * 16;
        if (gm >= row_end) continue;
        const int64_t drow = (MODE == dg::MODE_MASKED ? g * p.d_gs : 0) + (int64_t)gm * p.ldd;
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          const int gn = n0 + wn * TN + j * 16 + 4 * q4;
          if (gn < p.n) dg::store_out<BF16_OUT, HAS_C>(p, (int64_t)gm * p.ldc, gn, drow, acc[i][j]);
        }
      }
    }
    asm volatile("" ::: "memory");
    dg::debug_fence();
    u = nx;
  }
  dg::wait_vmcnt<0>();  // no direct load into this workgroup's LDS outlives it
}

}  // namespace fp4

inline bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline int cdiv(int a, int b) { return (a + b - 1) / b; }

// Tile configurations: 256-row tiles on 8 waves, one workgroup per CU (136, 127 and 119 KiB of LDS at 256, 224 and 192
// columns), and 128 x 128 on 4 waves, two per CU (68 KiB), on two slab stages; and the streaming tiles, one per CU, on a ring
// of 7, 6 or 4 (149, 153 and 136 KiB at 32, 64 and 128 rows).
struct Cfg {
  int bm, bn, per_cu, threads;
  double alone_us, full_us;  // per slab with few and with all CUs at work (the clock falls); streaming tiles: 0
};
constexpr Cfg kWide[4] = {{256, 256, 1, 512, 1.4, 1.9}, {256, 224, 1, 512, 1.35, 1.7}, {256, 192, 1, 512, 1.1, 1.5},
                          {128, 128, 2, 256, 0.84, 1.25}};
constexpr Cfg kStream[3] = {{32, 128, 1, 256, 0, 0}, {64, 128, 1, 512, 0, 0}, {128, 128, 1, 512, 0, 0}};
inline bool is_stream(const Cfg& c) { return c.full_us == 0; }

using Kernel = void (*)(fp4::Params);

template <int BM, int BN, int WM, int WN, int MODE>
Kernel pick_wide(bool bf16, bool has_c) {
  if constexpr (MODE == dg::MODE_DENSE) {
    if (has_c) return bf16 ? fp4::gemm_kernel<BM, BN, WM, WN, MODE, true, true> : fp4::gemm_kernel<BM, BN, WM, WN, MODE, false, true>;
  }
  return bf16 ? fp4::gemm_kernel<BM, BN, WM, WN, MODE, true, false> : fp4::gemm_kernel<BM, BN, WM, WN, MODE, false, false>;
}
template <int BM, int WM, int STAGES, int MODE>
Kernel pick_stream(bool bf16, bool has_c) {
  if constexpr (MODE == dg::MODE_DENSE) {
    if (has_c) return bf16 ? fp4::stream_kernel<BM, WM, STAGES, MODE, true, true> : fp4::stream_kernel<BM, WM, STAGES, MODE, false, true>;
  }
  return bf16 ? fp4::stream_kernel<BM, WM, STAGES, MODE, true, false> : fp4::stream_kernel<BM, WM, STAGES, MODE, false, false>;
}
template <int MODE>
Kernel pick(const Cfg& c, bool bf16, bool has_c) {
  if constexpr (MODE != dg::MODE_CONTIG) {
    if (is_stream(c) && c.bm == 32) return pick_stream<32, 1, 7, MODE>(bf16, has_c);
    if (is_stream(c) && c.bm == 64) return pick_stream<64, 2, 6, MODE>(bf16, has_c);
    if (is_stream(c)) return pick_stream<128, 2, 4, MODE>(bf16, has_c);
  }
  if (c.bm == 128) return pick_wide<128, 128, 2, 2, MODE>(bf16, has_c);
  if (c.bn == 224) return pick_wide<256, 224, 4, 2, MODE>(bf16, has_c);
  if (c.bn == 192) return pick_wide<256, 192, 4, 2, MODE>(bf16, has_c);
  return pick_wide<256, 256, 2, 4, MODE>(bf16, has_c);
}

// Split-K workspace of a dense call: counters (zero between calls) at a fixed place, then the partial tiles.
constexpr int kCtrWords = 16384;
constexpr size_t kCtrBytes = kCtrWords * sizeof(uint32_t);
constexpr size_t kMaxPartialBytes = size_t(32) << 20;

struct Plan {
  Cfg cfg;
  int splits, slabs_per_split;
  size_t ws_bytes;  // 0: no split
};

// The configuration (and, for a dense call, the K split) with the least estimated time, in microseconds, its constants set by
// hand from timings on MI355X: 4 us from launch to the first slab and for the last stores, 1 us a round of workgroups, the slabs
// at a rate of the tile's own (streaming tiles: 40 GB/s a CU), and not less than the operands' bytes at 5.5 TB/s.  A split adds
// 1.2 us to publish and count partials, their bytes at 6 TB/s twice, and the last workgroup's reading of a tile's at 85 GB/s.
// rows: of A, or of a group's (masked: the expected number, taken to be the mean of evenly spread ones, from 0 up to twice it,
// or of as wide a spread below most_rows).  Against every configuration forced, the choice is within 15 % of the best one's time
// in 30 dense calls (23 within 5 %) and in 9 of 12 masked ones (17, 23 and 33 % over it in the others).
Plan plan(int mode, int64_t groups, int rows, int most_rows, int n, int k, int cus) {
  const int slabs = (k / 128 + 1) / 2;
  const bool masked = mode == dg::MODE_MASKED;
  const double bytes = (static_cast<double>(groups) * n + static_cast<double>(masked ? groups : 1) * rows) * k * 0.53;
  Plan best{kWide[0], 1, slabs, 0};
  double least = 1e300;
  // row tiles of a call
  auto row_tiles = [&](int bm) {
    if (!masked) return static_cast<double>(cdiv(rows, bm));
    const double up_to = std::min<double>(2.0 * rows, most_rows), from = 2.0 * rows - up_to;
    double t = 0;
    for (int j = 0; j * static_cast<double>(bm) < up_to && j < 4096; ++j)
      t += j * bm < from ? 1.0 : (up_to - j * bm) / std::max(up_to - from, 1.0);
    return groups * t;
  };
  auto consider = [&](const Cfg& c, int s) {
    const double units = std::ceil(row_tiles(c.bm)) * cdiv(n, c.bn) * s, slots = static_cast<double>(cus) * c.per_cu;
    const double rounds = std::ceil(units / slots), busy = std::min(1.0, units / cus);
    const int sps = cdiv(slabs, s);
    double slab_us = is_stream(c) ? (std::min(c.bm, rows) + 128) * 136 / 40e3 : c.alone_us + (c.full_us - c.alone_us) * busy;
    if (c.per_cu == 2 && units <= cus) slab_us = c.alone_us;  // one to a CU
    if (!is_stream(c) && masked)                              // B from memory, waited for
      slab_us = std::max(slab_us, c.per_cu == 2 ? 2.4 : c.bn / 256.0 * (1.8 + 0.65 * std::min(rows, 256) / 256));
    const double part = s > 1 ? units * c.bm * c.bn * 4 : 0;
    const double us = 4.0 + std::max(rounds * (1.0 + sps * slab_us), bytes / 5.5e6) +
                      (s > 1 ? 1.2 + s * (c.bm * c.bn * 4 / 85e3) + 2 * part / 6e6 : 0.0);
    if (us < least - 1e-9) {
      least = us;
      best = Plan{c, s, sps, s > 1 ? kCtrBytes + static_cast<size_t>(part) : 0};
    }
  };
  for (const Cfg& c : kWide) consider(c, 1);
  if (mode == dg::MODE_CONTIG || k == 0) return best;
  for (const Cfg& c : kStream) {
    consider(c, 1);
    const int64_t tiles = static_cast<int64_t>(cdiv(rows, c.bm)) * cdiv(n, c.bn);
    if (masked || tiles > kCtrWords) continue;
    for (int s = 2; s <= slabs && tiles * s <= 2ll * cus; ++s) {
      if (cdiv(slabs, cdiv(slabs, s)) != s) continue;  // each split once, as its slabs per split
      if (static_cast<size_t>(s) * tiles * c.bm * c.bn * 4 > kMaxPartialBytes) break;
      consider(c, s);
    }
  }
  return best;
}

// Rows of a masked call's groups, as the caller expects them; half of the room where it does not say.
inline int rows_of_group(int expected_m, int m_max) {
  return expected_m > 0 ? std::min(expected_m, m_max) : (m_max + 1) / 2;
}

template <int MODE>
dg_status launch(fp4::Params& pp, const Plan& pl, dg_dtype t, int groups_for_tiles, int cus, hipStream_t stream) {
  dg::Params& p = pp.g;
  p.tiles_m = cdiv(p.m, pl.cfg.bm);
  p.tiles_n = cdiv(p.n, pl.cfg.bn);
  p.splits = pl.splits;
  p.slabs_per_split = pl.slabs_per_split;
  const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n * groups_for_tiles * pl.splits;
  if (tiles > (1 << 30)) return DG_ERROR_NOT_SUPPORTED;  // a tile's number and the grid's workgroups are added
  p.num_tiles = static_cast<int>(tiles);
  const int slots = cus * pl.cfg.per_cu;
  const int grid = p.num_tiles < slots ? p.num_tiles : slots;
  hipLaunchKernelGGL(pick<MODE>(pl.cfg, t == DG_DTYPE_BF16, p.c != nullptr), dim3(grid), dim3(pl.cfg.threads), 0, stream, pp);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? DG_SUCCESS : dg::record_hip_error(e);
}

inline int usable_cus() {
  const int c = dg_get_num_cus();
  return c > 0 ? c : 256;
}

// Operand checks shared by the entry points; rows = rows of A (M, M_total or M_max).
dg_status check(const void* a, int64_t lda, const void* sfa, int64_t ld_sfa, const void* b, int64_t ldb, const void* sfb,
                int64_t ld_sfb, const void* d, int64_t ldd, dg_dtype t, int rows, int n, int k) {
  if (rows < 0 || n < 0 || k < 0 || (t != DG_DTYPE_BF16 && t != DG_DTYPE_FP32)) return DG_ERROR_INVALID_VALUE;
  if (k % 128 != 0) return DG_ERROR_NOT_SUPPORTED;
  if (rows == 0 || n == 0) return DG_SUCCESS;  // empty tensors may have no address
  const int64_t es = t == DG_DTYPE_BF16 ? 2 : 4;
  if (d == nullptr || !aligned(d, 16) || ldd < n || (ldd * es) % 16 != 0) return DG_ERROR_INVALID_VALUE;
  // for any K: an empty product's kernel builds its descriptors from the strides too
  if (lda < k / 2 || ldb < k / 2 || lda % 16 != 0 || ldb % 16 != 0) return DG_ERROR_INVALID_VALUE;
  // offsets within a tile's rows, among a group's scales, and row and column numbers of the tiles stay below 2^31
  if (lda >= (1ll << 23) || ldb >= (1ll << 23) || rows >= (1 << 29) || n >= (1 << 29)) return DG_ERROR_NOT_SUPPORTED;
  if (k > 0) {
    if (a == nullptr || b == nullptr || sfa == nullptr || sfb == nullptr) return DG_ERROR_INVALID_VALUE;
    if (!aligned(a, 16) || !aligned(b, 16) || !aligned(sfa, 16) || !aligned(sfb, 16)) return DG_ERROR_INVALID_VALUE;
    if (ld_sfa < rows || ld_sfa % 4 != 0 || ld_sfb < n || ld_sfb % 4 != 0) return DG_ERROR_INVALID_VALUE;
    const int64_t most = ((1ll << 31) - 1) / (k / 128 * 4);
    if (ld_sfa > most || ld_sfb > most) return DG_ERROR_NOT_SUPPORTED;
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
  p.lda = k > 0 ? lda : 0;  // k == 0: descriptors of no bytes, whatever the pointers are
  p.ldb = k > 0 ? ldb : 0;
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
  if (m <= 0 || n <= 0 || k <= 0 || k % 128 != 0 || m >= (1 << 29) || n >= (1 << 29)) return 0;
  return plan(dg::MODE_DENSE, 1, m, m, n, k, usable_cus()).ws_bytes;
}

dg_status dg_mxfp4_gemm_nt(const void* a, int64_t lda, const int32_t* sfa, int64_t ld_sfa, const void* b, int64_t ldb,
                           const int32_t* sfb, int64_t ld_sfb, const void* c, int64_t ldc, void* d, int64_t ldd,
                           dg_dtype d_dtype, int m, int n, int k, void* workspace, size_t workspace_bytes,
                           hipStream_t stream) {
  const dg_status st = check(a, lda, sfa, ld_sfa, b, ldb, sfb, ld_sfb, d, ldd, d_dtype, m, n, k);
  if (st != DG_SUCCESS || m == 0 || n == 0) return st;
  const int64_t es = d_dtype == DG_DTYPE_BF16 ? 2 : 4;
  if (c != nullptr && (!aligned(c, 16) || ldc < n || (ldc * es) % 16 != 0)) return DG_ERROR_INVALID_VALUE;
  fp4::Params pp = params(a, lda, sfa, ld_sfa, b, ldb, sfb, ld_sfb, d, ldd, m, n, k);
  pp.g.c = c;
  pp.g.ldc = ldc;
  const int cus = usable_cus();
  const Plan pl = plan(dg::MODE_DENSE, 1, m, m, n, k, cus);
  if (pl.ws_bytes > 0) {
    if (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < pl.ws_bytes) return DG_ERROR_WORKSPACE;
    pp.g.ctr = static_cast<uint32_t*>(workspace);
    pp.g.ws = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kCtrBytes);
  }
  return launch<dg::MODE_DENSE>(pp, pl, d_dtype, 1, cus, stream);
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
  const int cus = usable_cus();
  return launch<dg::MODE_CONTIG>(pp, plan(dg::MODE_CONTIG, 1, m_total, m_total, n, k, cus), d_dtype, 1, cus, stream);
}

dg_status dg_m_grouped_mxfp4_gemm_nt_masked(const void* a, const int32_t* sfa, int64_t ld_sfa, const void* b,
                                            const int32_t* sfb, int64_t ld_sfb, void* d, dg_dtype d_dtype,
                                            const int32_t* masked_m, int num_groups, int m_max, int n, int k,
                                            int expected_m, hipStream_t stream) {
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
  const int cus = usable_cus();
  const Plan pl = plan(dg::MODE_MASKED, num_groups, rows_of_group(expected_m, m_max), m_max, n, k, cus);
  return launch<dg::MODE_MASKED>(pp, pl, d_dtype, num_groups, cus, stream);
}

dg_status dg_internal_mxfp4_plan(int mode, int groups, int rows, int most_rows, int n, int k, int cus, int* bm, int* bn,
                                 int* streaming, int* splits, size_t* ws_bytes) {
  if (mode < 0 || mode > 2 || groups <= 0 || (rows <= 0 && mode != dg::MODE_MASKED) || most_rows < rows || most_rows <= 0 || n <= 0 || k <= 0 || k % 128 != 0 || cus <= 0 ||
      bm == nullptr || bn == nullptr || streaming == nullptr || splits == nullptr || ws_bytes == nullptr)
    return DG_ERROR_INVALID_VALUE;
  const Plan pl = plan(mode, groups, mode == dg::MODE_MASKED ? rows_of_group(rows, most_rows) : rows, most_rows, n, k, cus);
  *bm = pl.cfg.bm;
  *bn = pl.cfg.bn;
  *streaming = is_stream(pl.cfg);
  *splits = pl.splits;
  *ws_bytes = pl.ws_bytes;
  return DG_SUCCESS;
}

}  // extern "C"
