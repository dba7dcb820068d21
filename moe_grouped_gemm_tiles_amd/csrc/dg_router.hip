// dg_router.hip -- the router of an expert layer on gfx950: scores, the choice of top_k experts and
// their weights, tokens per expert and the balance loss in one pass over the logits, and its gradient.
//
//   p      = softmax(x) or sigmoid(x)             (an expert whose logit is -inf has p = 0 and is never chosen)
//   ids    = the top_k largest keys, ties to the lower index; key = x, or p + bias where there is a bias
//   w_j    = scale * p_j / (sum over the chosen + 1e-20), or scale * p_j
//   share  = p / (sum over all + 1e-20)           (softmax: p itself)
//   counts = how often an expert is chosen, prob_sum = sum over rows of share
//   loss   = E * sum_e counts_e prob_sum_e / (sum counts * sum prob_sum)
#include <hip/hip_runtime.h>

#include <cstdint>

#include "dg.h"
#include "dg_common.hpp"

namespace {

namespace route {

constexpr float kTiny = 1e-20f;
constexpr int kWaves = 4;       // waves per workgroup, one row each at a time
constexpr int kMaxBlocks = 512;

struct Args {
  const uint8_t* logits;
  const float* bias;
  const uint8_t* mask;
  int32_t* ids;
  float* weights;
  int32_t* counts;
  float* prob_sum;
  float* loss;
  uint32_t* part_counts;  // [blocks][E]
  float* part_probs;      // [blocks][E]
  int64_t ld;
  float scale;
  int m, e, k, normalize, blocks;
};

struct GradArgs {
  const uint8_t* logits;
  const int32_t* ids;
  const float* dw;
  const int32_t* counts;
  const float* prob_sum;
  const float* dloss;
  uint8_t* dx;
  int64_t ld, ld_dx;
  float scale;
  int m, e, k, normalize;
};

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
template <typename T>
__device__ __forceinline__ T wave_max(T v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    const T w = __shfl_xor(v, o);
    v = w > v ? w : v;
  }
  return v;
}
__device__ __forceinline__ int wave_min(int v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = min(v, __shfl_xor(v, o));
  return v;
}

// Orders a wave's LDS accesses before this point with those after it, for all its lanes.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

template <bool BF16>
__device__ __forceinline__ float load(const uint8_t* row, int e) {
  if constexpr (BF16) return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(row)[e] << 16);
  return reinterpret_cast<const float*>(row)[e];
}

// Scores of a row's V experts per lane (0 past the last one), and the sum over all.
template <int V, bool SIGMOID>
__device__ __forceinline__ float scores(const float (&x)[V], float (&p)[V]) {
  float sum = 0.f;
  if constexpr (SIGMOID) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float t = __expf(-fabsf(x[i])), r = 1.0f / (1.0f + t);
      p[i] = x[i] >= 0.f ? r : t * r;
      sum += p[i];
    }
    return wave_sum(sum);
  } else {
    float top = x[0];
#pragma unroll
    for (int i = 1; i < V; ++i) top = fmaxf(top, x[i]);
    top = wave_max(top);
    if (top == -INFINITY) top = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      p[i] = __expf(x[i] - top);
      sum += p[i];
    }
    sum = wave_sum(sum);
    const float r = sum > 0.f ? 1.0f / sum : (sum == 0.f ? 0.f : sum);
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] *= r;
    return sum > 0.f ? 1.f : sum;
  }
}

// expert of value i of a lane
__device__ __forceinline__ int expert(int lane, int i) { return lane + 64 * i; }

template <int V, bool BF16, bool SIGMOID, bool BIAS, bool STATS>
__global__ void __launch_bounds__(kWaves * 64) forward_kernel(const Args a) {
  extern __shared__ uint32_t s_mem[];  // counts [E], then per wave probability sums [kWaves][E]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t* s_counts = s_mem;
  float* s_probs = reinterpret_cast<float*>(s_mem + a.e);
  if (STATS) {
    for (int e = threadIdx.x; e < a.e; e += kWaves * 64) s_counts[e] = 0;
    __syncthreads();
  }
  float ps[V];
#pragma unroll
  for (int i = 0; i < V; ++i) ps[i] = 0.f;
  for (int row = blockIdx.x * kWaves + wave; row < a.m; row += gridDim.x * kWaves) {
    const bool on = a.mask == nullptr || a.mask[row] != 0;
    const uint8_t* src = a.logits + row * a.ld;
    float x[V], p[V];
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = expert(lane, i) < a.e ? load<BF16>(src, expert(lane, i)) : -INFINITY;
    const float sum = scores<V, SIGMOID>(x, p);
    if (STATS && on) {
      const float r = SIGMOID ? 1.0f / (sum + kTiny) : 1.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) ps[i] += p[i] * r;
    }
    double key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      key[i] = x[i];
      if (BIAS && x[i] > -INFINITY) {
        const double b = a.bias[expert(lane, i)];
        if constexpr (SIGMOID) key[i] = 1.0 / (1.0 + exp(-(double)x[i])) + b;
      }
    }
    if constexpr (BIAS && !SIGMOID) {
      double top = key[0];
#pragma unroll
      for (int i = 1; i < V; ++i) top = key[i] > top ? key[i] : top;
      top = wave_max(top);
      double total = 0.0, ex[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        ex[i] = x[i] > -INFINITY ? exp(key[i] - top) : 0.0;
        total += ex[i];
      }
      total = wave_sum(total);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (x[i] > -INFINITY) key[i] = ex[i] / total + (double)a.bias[expert(lane, i)];
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (!(key[i] > -INFINITY)) key[i] = -INFINITY;  // NaN too
    int my_id = -1;
    float my_w = 0.f, chosen = 0.f;
    for (int j = 0; j < a.k; ++j) {
      double best = key[0];
#pragma unroll
      for (int i = 1; i < V; ++i) best = key[i] > best ? key[i] : best;
      best = wave_max(best);
      if (!(best > -INFINITY) || !on) break;
      int at = 0x7fffffff;
#pragma unroll
      for (int i = V - 1; i >= 0; --i)
        if (key[i] == best) at = expert(lane, i);
      at = wave_min(at);
      float w = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (expert(lane, i) == at) {
          w = p[i];
          key[i] = -INFINITY;
        }
      w = __shfl(w, at & 63);
      chosen += w;
      if (lane == j) {
        my_id = at;
        my_w = w;
      }
      if (STATS && lane == 0) atomicAdd(&s_counts[at], 1u);
    }
    if (lane < a.k) {
      a.ids[(int64_t)row * a.k + lane] = my_id;
      a.weights[(int64_t)row * a.k + lane] = my_id < 0 ? 0.f : a.scale * (a.normalize ? my_w / (chosen + kTiny) : my_w);
    }
  }
  if (STATS) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (expert(lane, i) < a.e) s_probs[wave * a.e + expert(lane, i)] = ps[i];
    __syncthreads();
    for (int e = threadIdx.x; e < a.e; e += kWaves * 64) {
      float s = 0.f;
      for (int w = 0; w < kWaves; ++w) s += s_probs[w * a.e + e];
      a.part_counts[(int64_t)blockIdx.x * a.e + e] = s_counts[e];
      a.part_probs[(int64_t)blockIdx.x * a.e + e] = s;
    }
  }
}

__global__ void __launch_bounds__(1024) finish_kernel(const Args a) {
  __shared__ double s_red[3][16];
  double c = 0, s = 0, cs = 0;
  for (int e = threadIdx.x; e < a.e; e += 1024) {
    uint32_t n = 0;
    double p = 0;
    for (int b = 0; b < a.blocks; ++b) {
      n += a.part_counts[(int64_t)b * a.e + e];
      p += (double)a.part_probs[(int64_t)b * a.e + e];
    }
    a.counts[e] = (int32_t)n;
    if (a.prob_sum != nullptr) a.prob_sum[e] = (float)p;
    c += n;
    s += p;
    cs += n * p;
  }
  c = wave_sum(c);
  s = wave_sum(s);
  cs = wave_sum(cs);
  if ((threadIdx.x & 63) == 0) {
    s_red[0][threadIdx.x >> 6] = c;
    s_red[1][threadIdx.x >> 6] = s;
    s_red[2][threadIdx.x >> 6] = cs;
  }
  __syncthreads();
  if (threadIdx.x == 0 && a.loss != nullptr) {
    double t[3] = {0, 0, 0};
    for (int w = 0; w < 16; ++w)
      for (int i = 0; i < 3; ++i) t[i] += s_red[i][w];
    const double den = t[0] * t[1];
    *a.loss = den == 0 ? 0.f : (float)(a.e * t[2] / den);
  }
}

template <int V, bool BF16, bool SIGMOID>
__global__ void __launch_bounds__(kWaves * 64) backward_kernel(const GradArgs a) {
  __shared__ float s_dp[kWaves][V * 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  // g_e = dloss * E * counts_e / (sum counts * sum prob_sum)
  float g[V];
  {
    double c = 0, s = 0;
    float mine[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = expert(lane, i);
      mine[i] = 0.f;
      if (a.counts != nullptr && e < a.e) {
        mine[i] = (float)a.counts[e];
        c += a.counts[e];
        s += (double)a.prob_sum[e];
      }
    }
    c = wave_sum(c);
    s = wave_sum(s);
    const double den = c * s;
    const float f = (a.counts == nullptr || den == 0) ? 0.f : (float)((double)*a.dloss * a.e / den);
#pragma unroll
    for (int i = 0; i < V; ++i) g[i] = f * mine[i];
  }
  for (int row = blockIdx.x * kWaves + wave; row < a.m; row += gridDim.x * kWaves) {
    const uint8_t* src = a.logits + row * a.ld;
    float x[V], p[V], dp[V];
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = expert(lane, i) < a.e ? load<BF16>(src, expert(lane, i)) : -INFINITY;
    const float sum = scores<V, SIGMOID>(x, p);
    int id = -1;
    float dw = 0.f;
    if (lane < a.k) {
      id = a.ids[(int64_t)row * a.k + lane];
      if (id < 0 || id >= a.e) id = -1;
      if (id >= 0) dw = a.dw[(int64_t)row * a.k + lane];
    }
    const bool on = __any(id >= 0);
#pragma unroll
    for (int i = 0; i < V; ++i) s_dp[wave][expert(lane, i)] = p[i];
    wave_sync();
    const float chosen = id >= 0 ? s_dp[wave][id] : 0.f;
    float d = a.scale * dw;
    if (a.normalize) {
      const float total = wave_sum(chosen) + kTiny;
      d = (d - wave_sum(d * chosen) / total) / total;
    }
    wave_sync();
#pragma unroll
    for (int i = 0; i < V; ++i) s_dp[wave][expert(lane, i)] = 0.f;
    wave_sync();
    if (id >= 0) atomicAdd(&s_dp[wave][id], d);
    wave_sync();
    float dot = 0.f;
    if constexpr (SIGMOID) {
      const float r = 1.0f / (sum + kTiny);
#pragma unroll
      for (int i = 0; i < V; ++i) dot += g[i] * p[i];
      dot = wave_sum(dot) * r;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float t = __expf(-fabsf(x[i])), q = 1.0f / (1.0f + t);
        dp[i] = (s_dp[wave][expert(lane, i)] + (g[i] - dot) * r) * p[i] * (x[i] >= 0.f ? t * q : q);
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        dp[i] = s_dp[wave][expert(lane, i)] + g[i];
        dot += dp[i] * p[i];
      }
      dot = wave_sum(dot);
#pragma unroll
      for (int i = 0; i < V; ++i) dp[i] = p[i] * (dp[i] - dot);
    }
    wave_sync();
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = expert(lane, i);
      if (e >= a.e) continue;
      const float v = on ? dp[i] : 0.f;
      if constexpr (BF16) reinterpret_cast<__bf16*>(a.dx + row * a.ld_dx)[e] = (__bf16)v;
      else reinterpret_cast<float*>(a.dx + row * a.ld_dx)[e] = v;
    }
  }
}

template <int V, bool BF16, bool SIGMOID>
void run_forward(const Args& a, hipStream_t stream) {
  const bool stats = a.counts != nullptr;
  const dim3 grid(a.blocks), block(kWaves * 64);
  const size_t lds = stats ? (size_t)a.e * 4 * (1 + kWaves) : 0;
  if (a.bias != nullptr) {
    if (stats) hipLaunchKernelGGL((forward_kernel<V, BF16, SIGMOID, true, true>), grid, block, lds, stream, a);
    else hipLaunchKernelGGL((forward_kernel<V, BF16, SIGMOID, true, false>), grid, block, lds, stream, a);
  } else {
    if (stats) hipLaunchKernelGGL((forward_kernel<V, BF16, SIGMOID, false, true>), grid, block, lds, stream, a);
    else hipLaunchKernelGGL((forward_kernel<V, BF16, SIGMOID, false, false>), grid, block, lds, stream, a);
  }
  if (stats) hipLaunchKernelGGL(finish_kernel, dim3(1), dim3(1024), 0, stream, a);
}

template <int V, bool BF16, bool SIGMOID>
void run_backward(const GradArgs& a, hipStream_t stream) {
  const int blocks = min((a.m + kWaves - 1) / kWaves, 2048);
  hipLaunchKernelGGL((backward_kernel<V, BF16, SIGMOID>), dim3(blocks), dim3(kWaves * 64), 0, stream, a);
}

}  // namespace route

inline bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

dg_status sizes(int m, int e, int k, dg_dtype t, dg_score s) {
  if (m < 0 || e < 0 || k < 0 || (t != DG_DTYPE_BF16 && t != DG_DTYPE_FP32)) return DG_ERROR_INVALID_VALUE;
  if (s != DG_SCORE_SOFTMAX && s != DG_SCORE_SIGMOID) return DG_ERROR_INVALID_VALUE;
  if (e == 0 || e > 1024 || k == 0 || k > 64 || k > e) return DG_ERROR_NOT_SUPPORTED;
  return DG_SUCCESS;
}

inline int blocks_of(int m) {
  const int b = (m + route::kWaves - 1) / route::kWaves;
  return b < 1 ? 1 : (b > route::kMaxBlocks ? route::kMaxBlocks : b);
}

#define DG_ROUTE_DISPATCH(FN, ARGS)                                                       \
  do {                                                                                    \
    const int v = (ARGS.e + 63) / 64;                                                     \
    const bool bf = dtype == DG_DTYPE_BF16, sg = score == DG_SCORE_SIGMOID;               \
    if (v <= 1) bf ? (sg ? FN<1, true, true>(ARGS, stream) : FN<1, true, false>(ARGS, stream))      \
                   : (sg ? FN<1, false, true>(ARGS, stream) : FN<1, false, false>(ARGS, stream));   \
    else if (v <= 4) bf ? (sg ? FN<4, true, true>(ARGS, stream) : FN<4, true, false>(ARGS, stream)) \
                   : (sg ? FN<4, false, true>(ARGS, stream) : FN<4, false, false>(ARGS, stream));   \
    else bf ? (sg ? FN<16, true, true>(ARGS, stream) : FN<16, true, false>(ARGS, stream))           \
                   : (sg ? FN<16, false, true>(ARGS, stream) : FN<16, false, false>(ARGS, stream)); \
  } while (0)

}  // namespace

extern "C" {

size_t dg_get_moe_router_workspace_size(int m, int num_experts) {
  if (m <= 0 || num_experts <= 0 || num_experts > 1024) return 0;
  return static_cast<size_t>(blocks_of(m)) * num_experts * 8;
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
  route::Args a{static_cast<const uint8_t*>(logits), bias, static_cast<const uint8_t*>(mask), topk_ids, topk_weights, counts,
                prob_sum, loss, static_cast<uint32_t*>(workspace),
                reinterpret_cast<float*>(static_cast<uint32_t*>(workspace) + (size_t)blocks_of(m) * num_experts), ld * es,
                scale, m, num_experts, top_k, normalize, blocks_of(m)};
  if (m == 0) {
    a.blocks = 0;
    hipLaunchKernelGGL(route::finish_kernel, dim3(1), dim3(1024), 0, stream, a);
  } else {
    DG_ROUTE_DISPATCH(route::run_forward, a);
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
  const route::GradArgs a{static_cast<const uint8_t*>(logits), topk_ids, dweights, counts, prob_sum, dloss,
                          static_cast<uint8_t*>(dlogits), ld * es, ld_dlogits * es, scale, m, num_experts, top_k, normalize};
  DG_ROUTE_DISPATCH(route::run_backward, a);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? DG_SUCCESS : dg::record_hip_error(e);
}

}  // extern "C"
