// dg_router.hip -- the router of an expert layer on gfx950: scores, the choice of top_k experts and
// their weights, tokens per expert and the balance loss in one pass over the logits, and its gradient.
//
//   p      = softmax(x) or sigmoid(x)             (an expert whose logit is -inf has p = 0 and is never chosen)
//   ids    = the top_k largest keys, ties to the lower index; key = x, or p + bias where there is a bias
//   w_j    = scale * p_j / (sum over the chosen + 1e-20), or scale * p_j
//   share  = p / (sum over all + 1e-20)           (softmax: p itself)
//   counts = how often an expert is chosen, prob_sum = sum over rows of share
//   loss   = E * sum_e counts_e prob_sum_e / (sum counts * sum prob_sum)
//
// Forward: 16 lanes hold a row of up to 256 experts (32 or 64 lanes past that, or for more than 15 chosen), so that a wave
// works on four rows and reductions stay in a DPP row.  A key is one register: the value's leading bits in an unsigned order,
// and the index below them, so that a maximum finds value and tie-break at once.  Each lane sorts its keys and keeps five; the
// largest head is taken top_k times.  Where the bits that the index pushed out, or FP32's errors in score + bias, leave the
// order open, more are taken and sorted by full values, and at last all keys are compared in FP64 by the whole wave.
// Sums of scores are held in FP32 registers per lane and expert (one rounding for each of the lane's rows, 20480 rows apart,
// and for the 16 rows that a workgroup has at work); each workgroup leaves one partial row, which a second kernel adds in FP64
// in a fixed order (integer atomics would do for the counts, but FP ones would change the sums from run to run).
//
// 33280 x 256 FP32, sigmoid, bias, mask, top 8, loss: 21 us and 7 us for the second kernel (a wave per row with FP64 keys: 258);
// 34 MB of logits are 5 us of HBM, so the 720 vector instructions for four rows bound it (8 us of them issue alone).  Gradient,
// BF16: 15 us (530 instructions for four rows).  A batch of rows that all need the exact choice (with a bias, scores that
// saturate or lie closer than kNear) takes up to four times as long: 33280 x 256 93 us sigmoid, 102 us softmax.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "dg.h"
#include "dg_common.hpp"

namespace {

namespace route {

constexpr float kTiny = 1e-20f;
constexpr int kWaves = 4;         // waves per workgroup
constexpr int kMaxBlocks = 1280;  // workgroups of a large batch, each with its own partial sums
constexpr int kMaxAlone = 1 << 20;  // and of one without sums: a grid holds fewer than 2^32 threads
constexpr int kFinishCols = 16;  // experts per workgroup of the second kernel

// Workspace: a header (the count of finished workgroups, then three sums for each workgroup of the second kernel),
// counts [blocks][E] and probability sums [blocks][E].
constexpr size_t kHeader = 2048;

struct Args {
  const uint8_t* logits;
  const float* bias;
  const uint8_t* mask;
  int32_t* ids;
  float* weights;
  int32_t* counts;
  float* prob_sum;
  float* loss;
  uint8_t* ws;
  int64_t ld;  // bytes
  float scale;
  int m, e, k, normalize, blocks, vec;
};

struct GradArgs {
  const uint8_t* logits;
  const int32_t* ids;
  const float* dw;
  const int32_t* counts;
  const float* prob_sum;
  const float* dloss;
  uint8_t* dx;
  int64_t ld, ld_dx;  // bytes
  float scale;
  int m, e, k, normalize, vec;
};

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}

// Reduction over the L lanes (16, 32 or 64) of a row, the result in each of them: rotations within 16 lanes, then
// exchanges of whole 16-lane rows.  Every lane adds the same pairs, so all get the same bits.
template <int L, typename T, typename Op>
__device__ __forceinline__ T reduce(T v, Op op) {
  static_assert(sizeof(T) == 4, "one register");
  auto step = [&](uint32_t o) { v = op(v, __builtin_bit_cast(T, o)); };
  step(dpp<0x128>(__builtin_bit_cast(uint32_t, v)));  // row_ror 8, 4, 2, 1
  step(dpp<0x124>(__builtin_bit_cast(uint32_t, v)));
  step(dpp<0x122>(__builtin_bit_cast(uint32_t, v)));
  step(dpp<0x121>(__builtin_bit_cast(uint32_t, v)));
  if constexpr (L >= 32) {
    const auto s = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
    v = op(__builtin_bit_cast(T, (uint32_t)s[0]), __builtin_bit_cast(T, (uint32_t)s[1]));
  }
  if constexpr (L >= 64) {
    const auto s = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
    v = op(__builtin_bit_cast(T, (uint32_t)s[0]), __builtin_bit_cast(T, (uint32_t)s[1]));
  }
  return v;
}
template <int L>
__device__ __forceinline__ float sum_of(float v) {
  return reduce<L>(v, [](float a, float b) { return a + b; });
}
template <int L>
__device__ __forceinline__ float max_of(float v) {
  return reduce<L>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int L>
__device__ __forceinline__ uint32_t max_of(uint32_t v) {
  return reduce<L>(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}
// Whether any of a row's lanes says so.
template <int L>
__device__ __forceinline__ bool any_of(bool v, int lane) {
  const uint64_t b = __ballot(v);
  if constexpr (L == 64) return b != 0;
  return ((b >> (lane & ~(L - 1))) & ((1ull << L) - 1)) != 0;
}

// Orders a wave's LDS accesses before this point with those after it, for all its lanes.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Value i of lane l (of a row's L) is expert 4 * (l + L * (i / 4)) + i % 4: four in a row, so that a lane's loads
// and stores are vectors and a row's lanes cover whole runs.
template <int L>
__device__ __forceinline__ int expert(int l, int i) {
  return 4 * (l + L * (i >> 2)) + (i & 3);
}

template <bool BF16>
__device__ __forceinline__ float load1(const uint8_t* row, int e) {
  if constexpr (BF16) return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(row)[e] << 16);
  else return reinterpret_cast<const float*>(row)[e];
}

// A row's values of a lane, -inf past the last expert (loaded at a clamped place, so that no load sits in a branch).
// vec: rows are aligned to four values and hold whole fours.
template <int L, int V, bool BF16>
__device__ __forceinline__ void load_row(const uint8_t* row, int e, int vec, int l, float (&x)[V]) {
  asm volatile("" : "+v"(l));  // places are worked out here, not kept in registers over the loop around
  if (vec) {
    float4 v[V / 4];
#pragma unroll
    for (int c = 0; c < V / 4; ++c) {
      const int at = min(4 * (l + L * c), e - 4);
      if constexpr (BF16) {
        const uint2 w = *reinterpret_cast<const uint2*>(row + 2 * at);
        v[c] = make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                           __uint_as_float(w.y & 0xffff0000u));
      } else {
        v[c] = *reinterpret_cast<const float4*>(row + 4 * at);
      }
    }
#pragma unroll
    for (int c = 0; c < V / 4; ++c) x[4 * c] = v[c].x, x[4 * c + 1] = v[c].y, x[4 * c + 2] = v[c].z, x[4 * c + 3] = v[c].w;
    if (e == L * V) return;
#pragma unroll
    for (int c = 0; c < V / 4; ++c) {
      const bool in = 4 * (l + L * c) < e;
      x[4 * c] = in ? v[c].x : -INFINITY, x[4 * c + 1] = in ? v[c].y : -INFINITY;
      x[4 * c + 2] = in ? v[c].z : -INFINITY, x[4 * c + 3] = in ? v[c].w : -INFINITY;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = load1<BF16>(row, min(expert<L>(l, i), e - 1));
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = expert<L>(l, i) < e ? x[i] : -INFINITY;
  }
}

// What turns a row's logits into scores: the largest (0 for a row of -inf alone), the sum of the exponentials and 1 / sum.
struct Norm {
  float top, sum, inv;
};
// exp(x), x <= 0, within 3 steps of 2^-24 however far below: the instruction's result for an argument that has been rounded,
// t = x log2(e), times exp(r) = 1 + r, where r = x - t ln 2 (ln 2 in two parts) is what that rounding lost.  (Of -inf, r is NaN
// and any number does for it.)  Below 2^-126 the instruction gives 0.
__device__ __forceinline__ float exp32(float x) {
  const float t = x * 0x1.715476p+0f, e = __builtin_amdgcn_exp2f(t);
  const float r = __builtin_fmaf(t, 0x1.05c610p-29f, __builtin_fmaf(-t, 0x1.62e430p-1f, x));
  return __builtin_fmaf(e, fminf(r, 1.0f), e);
}
// Scores in a row's sums and in keys, whose distance is looked at (kNear): an exponential without that correction is off by
// 2 |x| steps of itself, which is less than one step of the row's largest.  exp(-x) overflows to Inf where the sigmoid is
// below 2^-126: 0.
__device__ __forceinline__ float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.0f + __expf(-x)); }
// The score of one logit, as weights have it, to a few steps.
template <bool SIGMOID>
__device__ __forceinline__ float score(float x, Norm n) {
  if constexpr (!SIGMOID) return exp32(x - n.top) / n.sum;
  const float e = exp32(-fabsf(x));
  return (x >= 0.f ? 1.0f : e) / (1.0f + e);
}
template <int L, int V>
__device__ __forceinline__ float top_of(const float (&x)[V]) {
  float top = x[0];
#pragma unroll
  for (int i = 1; i < V; ++i) top = fmaxf(top, x[i]);
  top = max_of<L>(top);
  return top == -INFINITY ? 0.f : top;
}
// A row's exponentials (a softmax is n.inv times them), or its sigmoids, for which n.inv is 1 / (their sum + 1e-20).
template <int L, int V, bool SIGMOID, bool CLOSE = false>
__device__ __forceinline__ Norm scores(const float (&x)[V], float (&p)[V]) {
  Norm n{0.f, 0.f, 0.f};
  float sum = 0.f;
  if constexpr (SIGMOID) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      p[i] = sigmoid(x[i]);
      sum += p[i];
    }
    n.inv = 1.0f / (sum_of<L>(sum) + kTiny);
  } else {
    n.top = top_of<L, V>(x);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      p[i] = CLOSE ? exp32(x[i] - n.top) : __expf(x[i] - n.top);
      sum += p[i];
    }
    n.sum = sum_of<L>(sum);
    n.inv = n.sum == 0.f ? 0.f : 1.0f / n.sum;
  }
  return n;
}

// For the gradient: a softmax's scores, or the slopes p (1 - p) of a row's sigmoids in their logits' place and dot = the sum of
// g p over the lane's.  With e = exp(-|x|) and r = 1 / (1 + e) a sigmoid is r or e r, its slope e r^2.  FP32 gradients have them
// to a few steps: the exponential with its correction, a Newton step on the reciprocal, with what 1 + e lost, and on the
// quotient by a softmax's sum.  One that is rounded to BF16, 2^-9 of itself at most, does without: 2 |x| steps are 2^-16.
template <int L, int V, bool BF16, bool SIGMOID>
__device__ __forceinline__ Norm scores_for_gradient(float (&x)[V], float (&p)[V], const float (&g)[V], float& dot) {
  Norm n{0.f, 0.f, 0.f};
  if constexpr (SIGMOID) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float e = BF16 ? __expf(-fabsf(x[i])) : exp32(-fabsf(x[i])), d = 1.0f + e;
      float r = __builtin_amdgcn_rcpf(d);
      if (!BF16) r = __builtin_fmaf(__builtin_fmaf(d - 1.0f - e, r, __builtin_fmaf(-d, r, 1.0f)), r, r);
      const float er = e * r, v = x[i] >= 0.f ? r : er;
      x[i] = er * r;
      sum += v;
      dot += g[i] * v;
      asm volatile("" : "+v"(x[i]), "+v"(dot), "+v"(sum));  // now, not where the slopes are used: fewer registers are held
    }
    n.inv = 1.0f / (sum_of<L>(sum) + kTiny);
  } else {
    n = scores<L, V, false, !BF16>(x, p);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float q = p[i] * n.inv;
      p[i] = BF16 ? q : __builtin_fmaf(__builtin_fmaf(-q, n.sum, p[i]), n.inv, q);
    }
  }
  return n;
}

// Floats as unsigned integers of the same order, and back.  -0 and 0 are one value; -inf and NaN are kDead at most.
constexpr uint32_t kDead = 0x007fffffu;
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(fmaxf(v, -INFINITY) + 0.0f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) { return __uint_as_float((u >> 31) ? u ^ 0x80000000u : ~u); }

// Scores plus bias further apart than kNear * (1 + |key|) are in the order of their FP32 values.  A sigmoid is off by at
// most 6 steps of 2^-24 (the exponential's own and its argument's, each damped by p (1 - p), the sum, the reciprocal); a
// softmax p by p (24 + 2 |ln p|) steps (a sum of 22 roundings at most), which for two scores of one row is under 26 steps
// together; adding the bias rounds by half a step of the key: under 30 * 2^-24 < 2^-19.
constexpr float kNear = 0x1p-19f;

// The value one lane before (lane 0 of a row: its own).
template <int L>
__device__ __forceinline__ uint32_t before(uint32_t v) {
  if constexpr (L == 16) return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x111, 0xF, 0xF, false);
  else return __shfl_up(v, 1, L);
}
template <int L>
__device__ __forceinline__ float before(float v) {
  return __uint_as_float(before<L>(__float_as_uint(v)));
}

// Descending sort of V registers (odd-even merges: V = 4, 8, 16 take 5, 19, 63 exchanges).
template <int V>
__device__ __forceinline__ void sort_desc(uint32_t (&k)[V]) {
#pragma unroll
  for (int p = 1; p < V; p <<= 1)
#pragma unroll
    for (int q = p; q >= 1; q >>= 1)
#pragma unroll
      for (int j = q % p; j + q < V; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (i + j + q < V && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
            const uint32_t a = k[i + j], b = k[i + j + q];
            k[i + j] = max(a, b);
            k[i + j + q] = min(a, b);
          }
}

// exp(x) in FP64 for the exact choice: x = n ln 2 + r with |r| <= ln 2 / 2 (ln 2 in two parts, the first with 31 bits so that
// n times it is exact), the series of exp(r) to r^13 / 13! (the next term is below 2^-57), times 2^n.  The coefficients
// are read where they are used: as constants in the code they would fill registers all over the kernel.
__device__ const double kInverseFactorials[14] = {1.0, 1.0, 1.0 / 2, 1.0 / 6, 1.0 / 24, 1.0 / 120, 1.0 / 720, 1.0 / 5040,
                                                  1.0 / 40320, 1.0 / 362880, 1.0 / 3628800, 1.0 / 39916800,
                                                  1.0 / 479001600, 1.0 / 6227020800};
__device__ __forceinline__ double exp64(double x) {
  typedef const __attribute__((address_space(4))) double* table_t;
  uint64_t at = (uint64_t)(uintptr_t)kInverseFactorials;
  asm volatile("" : "+s"(at));
  const table_t c = (table_t)at;
  x = fmin(fmax(x, -800.0), 800.0);  // 0 and Inf past that
  const double n = rint(x * 0x1.71547652b82fep+0);
  double r = __builtin_fma(n, -0x1.62e42fec00000p-1, x);
  r = __builtin_fma(n, -0x1.d1cf79abc9e3bp-32, r);
  double p = c[13];
#pragma unroll
  for (int k = 12; k >= 0; --k) p = __builtin_fma(p, r, c[k]);
  return ldexp(p, (int)n);
}

// The choice for a row whose order FP32 leaves open, by a whole wave: every key in FP64, the largest taken k times.
// Lane j gets the j-th one's expert (-1: none).
template <int E, bool SIGMOID>
__device__ __forceinline__ int choose_exact(const float* row, const float* bias, int e, int k, int lane) {
  constexpr int N = (E + 63) / 64;
  double key[N], top = -INFINITY;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int at = lane + 64 * i;
    const float x = at < e ? row[at] : -INFINITY;
    key[i] = x > -INFINITY ? (double)x : -INFINITY;
    top = key[i] > top ? key[i] : top;
  }
  auto wave_max = [](double v) {
    for (int o = 32; o >= 1; o >>= 1) {
      const double w = __shfl_xor(v, o);
      v = w > v ? w : v;
    }
    return v;
  };
  if (bias != nullptr) {
    double total = 0.0;
    top = SIGMOID ? 0.0 : wave_max(top);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const bool live = key[i] > -INFINITY;
      const double t = exp64(SIGMOID ? -key[i] : key[i] - top);
      key[i] = live ? (SIGMOID ? 1.0 / (1.0 + t) : t) : -INFINITY;
      total += live ? t : 0.0;
    }
    if constexpr (!SIGMOID)
      for (int o = 32; o >= 1; o >>= 1) total += __shfl_xor(total, o);
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (key[i] > -INFINITY) {
        key[i] = (SIGMOID ? key[i] : key[i] / total) + (double)bias[lane + 64 * i];
        if (!(key[i] > -INFINITY)) key[i] = -INFINITY;  // a bias of NaN
      }
  }
  // the largest key as an unsigned integer of the same order, its upper word first, and of equal ones the lowest index
  uint32_t hi[N], lo[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint64_t b = __builtin_bit_cast(uint64_t, key[i] + 0.0);
    const uint64_t u = key[i] > -INFINITY ? b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull) : 0ull;
    hi[i] = (uint32_t)(u >> 32), lo[i] = (uint32_t)u;
  }
  int mine = -1;
  for (int j = 0; j < k; ++j) {
    uint32_t top_hi = hi[0], top_lo = 0, at = 0;
#pragma unroll
    for (int i = 1; i < N; ++i) top_hi = max(top_hi, hi[i]);
    top_hi = max_of<64>(top_hi);
    if (top_hi == 0) break;  // none is left
#pragma unroll
    for (int i = 0; i < N; ++i) top_lo = max(top_lo, hi[i] == top_hi ? lo[i] : 0u);
    top_lo = max_of<64>(top_lo);
#pragma unroll
    for (int i = 0; i < N; ++i)
      at = max(at, hi[i] == top_hi && lo[i] == top_lo ? (uint32_t)(64 * N - (lane + 64 * i)) : 0u);
    at = 64 * N - max_of<64>(at);
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (lane + 64 * i == (int)at) hi[i] = lo[i] = 0;
    if (lane == j) mine = (int)at;
  }
  return mine;
}

template <int L, int V, bool BF16, bool SIGMOID>
__global__ void __launch_bounds__(kWaves * 64) __attribute__((amdgpu_waves_per_eu(L > 16 ? 2 : (SIGMOID ? 5 : 4)))) forward_kernel(const Args a) {
  constexpr int R = 64 / L;             // rows a wave works on
  constexpr int E = L * V;              // experts a row has room for
  constexpr int D = V < 6 ? V : 5;      // how many of its largest keys a lane keeps
  constexpr uint32_t IDX = E - 1;       // low bits of a key: E - 1 - expert, so that ties go to the lower one
  __shared__ float s_x[kWaves * R][E];  // the rows at work; at the end their sums of scores
  __shared__ __attribute__((aligned(16))) float s_bias[E];
  __shared__ uint32_t s_counts[E];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int grp = lane / L, l = lane % L;
  const bool stats = a.counts != nullptr;
  if (stats) {
    for (int e = tid; e < E; e += kWaves * 64) s_counts[e] = 0;
    if (blockIdx.x == 0 && tid == 0 && a.blocks > 1) *reinterpret_cast<uint32_t*>(a.ws) = 0;
  }
  if (a.bias != nullptr)
    for (int e = tid; e < E; e += kWaves * 64) s_bias[e] = e < a.e ? a.bias[e] : 0.f;
  if (stats || a.bias != nullptr) __syncthreads();
  float* xs = s_x[wave * R + grp];
  float ps[V];
#pragma unroll
  for (int i = 0; i < V; ++i) ps[i] = 0.f;
  // unsigned: a row number plus the grid's rows passes 2^31 in a batch near that
  const uint32_t m = a.m, stride = gridDim.x * kWaves * R;
  // rows past the end repeat the last one and store nothing
  for (uint32_t base = (blockIdx.x * kWaves + wave) * R; base < m; base += stride) {
    const uint32_t row = base + grp;
    float x[V], p[V];
    const uint8_t there = a.mask != nullptr ? a.mask[min(row, m - 1)] : 1;
    const bool on = row < m && there != 0;
    load_row<L, V, BF16>(a.logits + (int64_t)min(row, m - 1) * a.ld, a.e, a.vec, l, x);
    wave_sync();  // the last rows' reads are done
#pragma unroll
    for (int c = 0; c < V / 4; ++c)
      *reinterpret_cast<float4*>(xs + 4 * (l + L * c)) = make_float4(x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
    const Norm n = scores<L, V, SIGMOID>(x, p);
    if (stats && on) {
#pragma unroll
      for (int i = 0; i < V; ++i) ps[i] += p[i] * n.inv;
    }
    // Keys: the value's leading bits, then the index.  What the index pushed out is looked at below.
    uint32_t key[V], lost = 0;
    int lk = l;
    asm volatile("" : "+v"(lk));
    if (a.bias != nullptr) {
#pragma unroll
      for (int c = 0; c < V / 4; ++c) {
        const float4 b = *reinterpret_cast<const float4*>(s_bias + 4 * (l + L * c));
        const float v[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 4 * c; i < 4 * c + 4; ++i)
          key[i] = (ordered(x[i] > -INFINITY ? (SIGMOID ? p[i] : p[i] * n.inv) + v[i & 3] : -INFINITY) & ~IDX) | (IDX - expert<L>(lk, i));
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (!BF16) lost |= __float_as_uint(x[i]);
        key[i] = (ordered(x[i]) & ~IDX) | (IDX - expert<L>(lk, i));
      }
    }
    sort_desc<V>(key);
    wave_sync();
    uint32_t mine = 0, last = 0, kth = 0;
    int taken = 0;
    auto take = [&]() {
      last = max_of<L>(key[0]);
      if (l == taken) mine = last;
      const bool won = key[0] == last;
#pragma unroll
      for (int i = 0; i + 1 < D; ++i) key[i] = won ? key[i + 1] : key[i];
      if (won) key[D - 1] = 0;
      ++taken;
    };
    for (int j = 0; j < a.k; ++j) take();
    kth = last;
    int id = mine > kDead ? (int)(IDX - (mine & IDX)) : -1;
    // BF16 logits lose nothing, nor do FP32 ones whose last bits are zero
    const bool rough = a.bias != nullptr || (!BF16 && any_of<L>((lost & IDX) != 0, lane));
    // A lane whose kept keys are all taken may hide one that belongs to the chosen: left to the exact choice.
    bool slow = D < V && any_of<L>(key[0] == 0, lane);
    if (__any(rough || slow)) {
      // Take more until none of the rest can belong to the first k, as far as there are lanes for them.
      auto open = [&]() {
        if (kth <= kDead || last <= kDead) return false;
        if (a.bias == nullptr) return (last | IDX) >= (kth & ~IDX);
        const float lo = unordered(kth & ~IDX), hi = unordered(last | IDX);
        return !(lo - hi > kNear * (1.0f + fabsf(lo)));
      };
      if (__any(rough)) {
        do take();
        while (taken < L && __any(rough && open()));
        slow = slow || (rough && (open() || (D < V && any_of<L>(key[0] == 0, lane))));
      }
      // the order of what was taken, by full FP32 values
      id = mine > kDead ? (int)(IDX - (mine & IDX)) : -1;
      float xv = id >= 0 ? xs[id] : -INFINITY, bv = 0.f, v = xv;
      if (a.bias != nullptr && id >= 0) {
        bv = s_bias[id];
        v = (SIGMOID ? sigmoid(xv) : __expf(xv - n.top) * n.inv) + bv;
      }
      for (int turn = 0; turn <= L; ++turn) {
        const float up = before<L>(v);
        const int uid = (int)before<L>((uint32_t)id);
        const bool wrong = l > 0 && id >= 0 && (v > up || (v == up && id < uid));
        if (!__any(rough && wrong)) break;
        const bool high = (l + turn) & 1;  // of the pairs (odd, even) and (even, odd) by turns
        const int other = high ? l - 1 : l + 1;
        const bool pair = other >= 0 && other < L;
        const float ov = __shfl(v, pair ? other : l, L), ox = __shfl(xv, pair ? other : l, L), ob = __shfl(bv, pair ? other : l, L);
        const int oid = __shfl(id, pair ? other : l, L);
        const bool ahead = oid >= 0 && (id < 0 || ov > v || (ov == v && oid < id));  // the other one goes first
        if (rough && pair && oid != id && (high ? !ahead : ahead)) v = ov, xv = ox, bv = ob, id = oid;
      }
      if (a.bias != nullptr) {
        const float up = before<L>(v), ux = before<L>(xv), ub = before<L>(bv);
        const bool near = l > 0 && id >= 0 && !(up - v > kNear * (1.0f + fabsf(v))) && !(xv == ux && bv == ub);
        slow = slow || any_of<L>(near, lane);
      }
      for (uint64_t left = __ballot(slow && on && l == 0); left != 0; left &= left - 1) {
        const int g = __builtin_ctzll(left) / L;
        const int exact = __shfl(choose_exact<E, SIGMOID>(s_x[wave * R + g], a.bias, a.e, a.k, lane), l);
        if (grp == g) id = exact;
      }
    }
    if (l >= a.k || !on) id = -1;
    const float w = id >= 0 ? score<SIGMOID>(xs[id], n) : 0.f;
    const float chosen = a.normalize ? sum_of<L>(w) + kTiny : 1.0f;
    if (l < a.k && row < m) {
      a.ids[(int64_t)row * a.k + l] = id;
      a.weights[(int64_t)row * a.k + l] = id >= 0 ? a.scale * w / chosen : 0.f;  // (the sum may be NaN)
    }
    if (stats && id >= 0) atomicAdd(&s_counts[id], 1u);
  }
  if (!stats) return;
  wave_sync();
#pragma unroll
  for (int c = 0; c < V / 4; ++c)
    *reinterpret_cast<float4*>(xs + 4 * (l + L * c)) = make_float4(ps[4 * c], ps[4 * c + 1], ps[4 * c + 2], ps[4 * c + 3]);
  __syncthreads();
  uint32_t* part_counts = reinterpret_cast<uint32_t*>(a.ws + kHeader);
  float* part_probs = reinterpret_cast<float*>(part_counts + (size_t)a.blocks * a.e);
  double c = 0, s = 0, cs = 0;
  for (int e = tid; e < a.e; e += kWaves * 64) {
    float t = 0.f;
#pragma unroll 8
    for (int w = 0; w < kWaves * R; ++w) t += s_x[w][e];
    const uint32_t cnt = s_counts[e];
    if (a.blocks > 1) {
      part_counts[(size_t)blockIdx.x * a.e + e] = cnt;
      part_probs[(size_t)blockIdx.x * a.e + e] = t;
    } else {
      a.counts[e] = (int32_t)cnt;
      if (a.prob_sum != nullptr) a.prob_sum[e] = t;
      c += cnt;
      s += t;
      cs += (double)cnt * t;
    }
  }
  if (a.blocks == 1 && a.loss != nullptr) {
    __shared__ double s_red[3][kWaves];
    for (int o = 32; o >= 1; o >>= 1) {
      c += __shfl_xor(c, o);
      s += __shfl_xor(s, o);
      cs += __shfl_xor(cs, o);
    }
    if (lane == 0) s_red[0][wave] = c, s_red[1][wave] = s, s_red[2][wave] = cs;
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < kWaves; ++w) c += s_red[0][w], s += s_red[1][w], cs += s_red[2][w];
      *a.loss = c == 0 || s == 0 ? 0.f : (float)(a.e * cs / (c * s));
    }
  }
}

// The workgroups' partial sums, kFinishCols experts to a workgroup; the last one to finish adds up the loss.
__global__ void __launch_bounds__(1024) finish_kernel(const Args a) {
  constexpr int PARTS = 1024 / kFinishCols;
  __shared__ uint32_t s_c[16][kFinishCols];
  __shared__ double s_p[16][kFinishCols];
  const int tid = threadIdx.x, col = tid % kFinishCols, part = tid / kFinishCols;
  const int e = blockIdx.x * kFinishCols + col;
  const uint32_t* part_counts = reinterpret_cast<const uint32_t*>(a.ws + kHeader);
  const float* part_probs = reinterpret_cast<const float*>(part_counts + (size_t)a.blocks * a.e);
  uint32_t n = 0;
  double p = 0;
  if (e < a.e) {
#pragma unroll 8
    for (int b = part; b < a.blocks; b += PARTS) {
      n += part_counts[(size_t)b * a.e + e];
      p += (double)part_probs[(size_t)b * a.e + e];
    }
  }
  // the parts of a wave (lanes 16 and 32 apart), then the waves'
  auto fold = [&]() {
    for (int o = kFinishCols; o < 64; o <<= 1) n += __shfl_xor(n, o), p += __shfl_xor(p, o);
  };
  fold();
  if ((tid & 63) < kFinishCols) s_c[tid >> 6][col] = n, s_p[tid >> 6][col] = p;
  __syncthreads();
  if (tid >= 64) return;
  n = 0, p = 0;
#pragma unroll
  for (int i = 0; i < 16 / (64 / kFinishCols); ++i) {
    const int w = part + i * (64 / kFinishCols);
    n += s_c[w][col], p += s_p[w][col];
  }
  fold();
  double c = 0, cs = 0;
  if (tid < kFinishCols && e < a.e) {
    a.counts[e] = (int32_t)n;
    if (a.prob_sum != nullptr) a.prob_sum[e] = (float)p;
    c = n;
    cs = c * p;
  } else {
    p = 0;
  }
  if (a.loss == nullptr) return;
  for (int o = 32; o >= 1; o >>= 1) {
    c += __shfl_xor(c, o);
    p += __shfl_xor(p, o);
    cs += __shfl_xor(cs, o);
  }
  double* sums = reinterpret_cast<double*>(a.ws + 64);
  int last = 0;
  if (tid == 0) {
    double* mine = sums + 3 * blockIdx.x;
    __hip_atomic_store(mine, c, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_store(mine + 1, p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_store(mine + 2, cs, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    last = __hip_atomic_fetch_add(reinterpret_cast<uint32_t*>(a.ws), 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) + 1 ==
           gridDim.x;
  }
  if (!__builtin_amdgcn_readfirstlane(last)) return;
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
  c = p = cs = 0;
  if (tid < (int)gridDim.x) {  // at most 64 workgroups
    c = __hip_atomic_load(sums + 3 * tid, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    p = __hip_atomic_load(sums + 3 * tid + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    cs = __hip_atomic_load(sums + 3 * tid + 2, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  for (int o = 32; o >= 1; o >>= 1) {
    c += __shfl_xor(c, o);
    p += __shfl_xor(p, o);
    cs += __shfl_xor(cs, o);
  }
  if (tid == 0) *a.loss = c == 0 || p == 0 ? 0.f : (float)(a.e * cs / (c * p));
}

// A batch of no rows.
__global__ void __launch_bounds__(1024) zero_kernel(const Args a) {
  if ((int)threadIdx.x < a.e) {
    a.counts[threadIdx.x] = 0;
    if (a.prob_sum != nullptr) a.prob_sum[threadIdx.x] = 0.f;
  }
  if (threadIdx.x == 0 && a.loss != nullptr) *a.loss = 0.f;
}

template <int L, int V, bool BF16, bool SIGMOID>
__global__ void __launch_bounds__(kWaves * 64) __attribute__((amdgpu_waves_per_eu(L > 16 ? 2 : 5))) backward_kernel(const GradArgs a) {
  constexpr int R = 64 / L, E = L * V;
  __shared__ float s_d[kWaves * R][E];  // the gradient by the chosen scores, 0 elsewhere
  __shared__ double s_red[2][kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int grp = lane / L, l = lane % L;
  float* ds = s_d[wave * R + grp];
  float g[V];
#pragma unroll
  for (int i = 0; i < V; ++i) g[i] = 0.f;
  const uint32_t m = a.m, stride = gridDim.x * kWaves * R;
  if (a.counts != nullptr) {  // g_e = dloss * E * counts_e / (sum counts * sum prob_sum)
    double c = 0, s = 0;
    for (int e = tid; e < a.e; e += kWaves * 64) {
      c += a.counts[e];
      s += (double)a.prob_sum[e];
    }
    for (int o = 32; o >= 1; o >>= 1) {
      c += __shfl_xor(c, o);
      s += __shfl_xor(s, o);
    }
    if (lane == 0) s_red[0][wave] = c, s_red[1][wave] = s;
    __syncthreads();
    c = s = 0;
    for (int w = 0; w < kWaves; ++w) c += s_red[0][w], s += s_red[1][w];
    const float f = c * s == 0 ? 0.f : (float)((double)*a.dloss * a.e / (c * s));
#pragma unroll
    for (int i = 0; i < V; ++i) g[i] = (float)a.counts[min(expert<L>(l, i), a.e - 1)];
#pragma unroll
    for (int i = 0; i < V; ++i) g[i] = expert<L>(l, i) < a.e ? f * g[i] : 0.f;
  }
  for (uint32_t base = (blockIdx.x * kWaves + wave) * R; base < m; base += stride) {
    const uint32_t row = min(base + grp, m - 1);
    float x[V], p[V];
    const int64_t slot = (int64_t)row * a.k + min(l, a.k - 1);
    const int slot_id = a.ids[slot];
    const float slot_dw = a.dw[slot];
    load_row<L, V, BF16>(a.logits + row * a.ld, a.e, a.vec, l, x);
    const int id = l < a.k && (uint32_t)slot_id < (uint32_t)a.e ? slot_id : -1;
    float d = id >= 0 ? a.scale * slot_dw : 0.f;
    wave_sync();
    if (a.normalize) {
#pragma unroll
      for (int c = 0; c < V / 4; ++c)
        *reinterpret_cast<float4*>(ds + 4 * (l + L * c)) = make_float4(x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
      wave_sync();
    }
    const float xv = a.normalize && id >= 0 ? ds[id] : -INFINITY;
    wave_sync();
#pragma unroll
    for (int c = 0; c < V / 4; ++c) *reinterpret_cast<float4*>(ds + 4 * (l + L * c)) = make_float4(0.f, 0.f, 0.f, 0.f);
    float dot = 0.f;
    const Norm n = scores_for_gradient<L, V, BF16, SIGMOID>(x, p, g, dot);
    const bool on = any_of<L>(id >= 0, lane);
    if (a.normalize) {
      const float w = score<SIGMOID>(xv, n);  // 0 where there is no expert
      const float chosen = sum_of<L>(w) + kTiny;
      d = (d - sum_of<L>(d * w) / chosen) / chosen;
    }
    wave_sync();
    if (id >= 0) atomicAdd(&ds[id], d);
    wave_sync();
    float dp[V];
#pragma unroll
    for (int c = 0; c < V / 4; ++c) {
      const float4 v = *reinterpret_cast<const float4*>(ds + 4 * (l + L * c));
      dp[4 * c] = v.x, dp[4 * c + 1] = v.y, dp[4 * c + 2] = v.z, dp[4 * c + 3] = v.w;
    }
    if constexpr (SIGMOID) {
      // without the loss nothing depends on the row's sum, which may be NaN
      const float inv = a.counts != nullptr ? n.inv : 0.f;
      dot = a.counts != nullptr ? sum_of<L>(dot) * inv : 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        dp[i] = (dp[i] + (g[i] - dot) * inv) * x[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        dp[i] += g[i];
        dot += dp[i] * p[i];
      }
      dot = sum_of<L>(dot);
#pragma unroll
      for (int i = 0; i < V; ++i) dp[i] = p[i] * (dp[i] - dot);
    }
    if (base + grp < m) {
      uint8_t* out = a.dx + (int64_t)row * a.ld_dx;
#pragma unroll
      for (int i = 0; i < V; ++i) dp[i] = on ? dp[i] : 0.f;
      if (a.vec) {
#pragma unroll
        for (int c = 0; c < V / 4; ++c) {
          const int at = 4 * (l + L * c);
          if (at >= a.e) continue;
          if constexpr (BF16) {
            typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
            typedef float f32x4 __attribute__((ext_vector_type(4)));
            const f32x4 v = {dp[4 * c], dp[4 * c + 1], dp[4 * c + 2], dp[4 * c + 3]};
            *reinterpret_cast<bf16x4*>(out + 2 * at) = __builtin_convertvector(v, bf16x4);
          } else {
            *reinterpret_cast<float4*>(out + 4 * at) = make_float4(dp[4 * c], dp[4 * c + 1], dp[4 * c + 2], dp[4 * c + 3]);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int e = expert<L>(l, i);
          if (e >= a.e) continue;
          if constexpr (BF16) reinterpret_cast<__bf16*>(out)[e] = (__bf16)dp[i];
          else reinterpret_cast<float*>(out)[e] = dp[i];
        }
      }
    }
  }
}

// Rows a workgroup works on at a time, by the lanes of a row.
inline int rows_at_once(int lanes) { return kWaves * (64 / lanes); }

// Lanes and values of a row: 16 lanes of 4, 8 or 16 values up to 256 experts (reductions stay within a DPP row and a
// wave works on four rows), more lanes past that, or where the chosen and one more do not fit the lanes.
inline int lanes_of(int e, int k) { return e <= 256 && k < 16 ? 16 : (e <= 512 && k < 32 ? 32 : 64); }
inline int values_of(int e, int lanes) {
  const int v = (e + lanes - 1) / lanes;
  return v <= 4 ? 4 : (v <= 8 ? 8 : 16);
}

}  // namespace route

inline bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

dg_status sizes(int m, int e, int k, dg_dtype t, dg_score s) {
  if (m < 0 || e < 0 || k < 0 || (t != DG_DTYPE_BF16 && t != DG_DTYPE_FP32)) return DG_ERROR_INVALID_VALUE;
  if (s != DG_SCORE_SOFTMAX && s != DG_SCORE_SIGMOID) return DG_ERROR_INVALID_VALUE;
  if (e == 0 || e > 1024 || k == 0 || k > 64 || k > e) return DG_ERROR_NOT_SUPPORTED;
  return DG_SUCCESS;
}

inline int ceil_div(int a, int b) { return static_cast<int>((static_cast<int64_t>(a) + b - 1) / b); }

inline int blocks_of(int m, int e) {
  const int b = ceil_div(m, route::rows_at_once(route::lanes_of(e, 1)));
  return b < 1 ? 1 : (b > route::kMaxBlocks ? route::kMaxBlocks : b);
}

// Calls f(lanes, values, bf16?, sigmoid?) with compile-time constants.
template <int L, int V, typename F>
void with_types(dg_dtype t, dg_score s, F f) {
  using std::integral_constant;
  auto lv = [&](auto bf, auto sg) { f(integral_constant<int, L>{}, integral_constant<int, V>{}, bf, sg); };
  if (t == DG_DTYPE_BF16) s == DG_SCORE_SIGMOID ? lv(std::true_type{}, std::true_type{}) : lv(std::true_type{}, std::false_type{});
  else s == DG_SCORE_SIGMOID ? lv(std::false_type{}, std::true_type{}) : lv(std::false_type{}, std::false_type{});
}
template <typename F>
void with_variant(int e, int k, dg_dtype t, dg_score s, F f) {
  const int l = route::lanes_of(e, k), v = route::values_of(e, l);
  if (l == 16) v == 4 ? with_types<16, 4>(t, s, f) : (v == 8 ? with_types<16, 8>(t, s, f) : with_types<16, 16>(t, s, f));
  else if (l == 32) v == 4 ? with_types<32, 4>(t, s, f) : (v == 8 ? with_types<32, 8>(t, s, f) : with_types<32, 16>(t, s, f));
  else v == 4 ? with_types<64, 4>(t, s, f) : (v == 8 ? with_types<64, 8>(t, s, f) : with_types<64, 16>(t, s, f));
}

}  // namespace

extern "C" {

size_t dg_get_moe_router_workspace_size(int m, int num_experts) {
  if (m <= 0 || num_experts <= 0 || num_experts > 1024) return 0;
  return route::kHeader + static_cast<size_t>(blocks_of(m, num_experts)) * num_experts * 8;
}

dg_status dg_moe_router(const void* logits, int64_t ld, dg_dtype dtype, const float* bias, const void* mask, dg_score score,
                        int normalize, float scale, int32_t* topk_ids, float* topk_weights, int32_t* counts, float* prob_sum,
                        float* loss, int m, int num_experts, int top_k, void* workspace, size_t workspace_bytes,
                        hipStream_t stream) {
  const dg_status st = sizes(m, num_experts, top_k, dtype, score);
  if (st != DG_SUCCESS) return st;
  const int64_t es = dtype == DG_DTYPE_BF16 ? 2 : 4;
  if (!(scale >= 0.f) || (prob_sum == nullptr) != (loss == nullptr) || (loss != nullptr && counts == nullptr))
    return DG_ERROR_INVALID_VALUE;
  if (!aligned(counts, 4) || !aligned(prob_sum, 4) || !aligned(loss, 4) || !aligned(bias, 4)) return DG_ERROR_INVALID_VALUE;
  if (m > 0 && (logits == nullptr || !aligned(logits, es) || topk_ids == nullptr || !aligned(topk_ids, 4) ||
                topk_weights == nullptr || !aligned(topk_weights, 4) || ld < num_experts))
    return DG_ERROR_INVALID_VALUE;
  if (m > 0 && counts != nullptr && (workspace == nullptr || !aligned(workspace, 256) ||
                                     workspace_bytes < dg_get_moe_router_workspace_size(m, num_experts)))
    return DG_ERROR_WORKSPACE;
  if (m == 0 && counts == nullptr) return DG_SUCCESS;
  const int64_t ldb = ld * es;
  const int vec = num_experts % 4 == 0 && aligned(logits, 4 * es) && ldb % (4 * es) == 0;
  route::Args a{static_cast<const uint8_t*>(logits), bias, static_cast<const uint8_t*>(mask), topk_ids, topk_weights, counts,
                prob_sum, loss, static_cast<uint8_t*>(workspace), ldb, scale, m, num_experts, top_k, normalize, 0, vec};
  if (m == 0) {
    hipLaunchKernelGGL(route::zero_kernel, dim3(1), dim3(1024), 0, stream, a);
  } else {
    with_variant(num_experts, top_k, dtype, score, [&](auto l, auto v, auto bf, auto sg) {
      const int need = ceil_div(m, route::rows_at_once(l));
      // as many workgroups as give each the same number of rounds, at most
      const int most = counts == nullptr ? route::kMaxAlone : blocks_of(m, num_experts), rounds = ceil_div(need, most);
      a.blocks = ceil_div(need, rounds);
      hipLaunchKernelGGL((route::forward_kernel<l, v, bf, sg>), dim3(a.blocks), dim3(route::kWaves * 64), 0, stream, a);
    });
    if (counts != nullptr && a.blocks > 1)
      hipLaunchKernelGGL(route::finish_kernel, dim3((num_experts + route::kFinishCols - 1) / route::kFinishCols), dim3(1024), 0,
                         stream, a);
  }
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? DG_SUCCESS : dg::record_hip_error(e);
}

dg_status dg_moe_router_backward(const void* logits, int64_t ld, dg_dtype dtype, dg_score score, int normalize, float scale,
                                 const int32_t* topk_ids, const float* dweights, const int32_t* counts,
                                 const float* prob_sum, const float* dloss, void* dlogits, int64_t ld_dlogits, int m,
                                 int num_experts, int top_k, hipStream_t stream) {
  const dg_status st = sizes(m, num_experts, top_k, dtype, score);
  if (st != DG_SUCCESS) return st;
  const int64_t es = dtype == DG_DTYPE_BF16 ? 2 : 4;
  if (!(scale >= 0.f) || (counts == nullptr) != (dloss == nullptr) || (prob_sum == nullptr) != (dloss == nullptr))
    return DG_ERROR_INVALID_VALUE;
  if (!aligned(counts, 4) || !aligned(prob_sum, 4) || !aligned(dloss, 4)) return DG_ERROR_INVALID_VALUE;
  if (m == 0) return DG_SUCCESS;
  if (logits == nullptr || !aligned(logits, es) || dlogits == nullptr || !aligned(dlogits, es) || topk_ids == nullptr ||
      !aligned(topk_ids, 4) || dweights == nullptr || !aligned(dweights, 4) || ld < num_experts || ld_dlogits < num_experts)
    return DG_ERROR_INVALID_VALUE;
  if (dlogits == logits && m > 1 && ld != ld_dlogits) return DG_ERROR_INVALID_VALUE;  // rows over other rows not yet read
  const int64_t ldb = ld * es, ldd = ld_dlogits * es;
  const int vec = num_experts % 4 == 0 && aligned(logits, 4 * es) && ldb % (4 * es) == 0 && aligned(dlogits, 4 * es) &&
                  ldd % (4 * es) == 0;
  const route::GradArgs a{static_cast<const uint8_t*>(logits), topk_ids, dweights, counts, prob_sum, dloss,
                          static_cast<uint8_t*>(dlogits), ldb, ldd, scale, m, num_experts, top_k, normalize, vec};
  with_variant(num_experts, top_k, dtype, score, [&](auto l, auto v, auto bf, auto sg) {
    const int need = ceil_div(m, route::rows_at_once(l)), rounds = ceil_div(need, route::kMaxBlocks);
    hipLaunchKernelGGL((route::backward_kernel<l, v, bf, sg>), dim3(ceil_div(need, rounds)), dim3(route::kWaves * 64), 0,
                       stream, a);
  });
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? DG_SUCCESS : dg::record_hip_error(e);
}

}  // extern "C"
