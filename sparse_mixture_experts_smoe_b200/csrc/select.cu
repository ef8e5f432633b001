// select.cu -- routing from given logits (smoe_route_select, smoe_route_select_bwd):
// softmax or sigmoid scores, a selection bias, expert groups, top-k and gates.
//
//   s_e  = 1 / (1 + exp(-l_e))  or  exp(l_e) / sum_u exp(l_u)
//   c_e  = s_e + b_e                       (what is ranked; without b: the logits)
//   best k of c_e, inside the best top_groups groups when there are groups
//   gate = scale * s_e, or scale * s_e / (sum of the selected s)
//
// Selected ids are whole numbers: they are those of scores compared in 64 bits, ties
// to the lower id.
#include <cfloat>

#include "common.cuh"

namespace smoe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kWarps = 4;

__device__ __forceinline__ double warp_max64(double v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = fmax(v, __shfl_xor_sync(kFull, v, off));
  return v;
}
template <typename V>
__device__ __forceinline__ V warp_sum(V v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
  return v;
}
// A logit as it is used: usable unless NaN or -inf; +inf counts as the largest
// finite value.
__device__ __forceinline__ bool usable(float l) { return l > -INFINITY; }
__device__ __forceinline__ float finite_top(float l) { return fminf(l, FLT_MAX); }

// One row, one warp, all scores in 64 bits.  sc: E + groups doubles of this warp.
// Returns in lane j < k the j-th selected expert (-1 elsewhere).
template <typename T>
__device__ int select_row64(const T* __restrict__ row, const SelectArgs& a, double* sc, int lane) {
  const bool soft = a.score == SMOE_SCORE_SOFTMAX;
  double mx = -INFINITY, den = 1.0;
  if (soft) {
    for (int e = lane; e < a.E; e += 32) {
      const float l = to_f(row[e]);
      if (usable(l)) mx = fmax(mx, (double)finite_top(l));
    }
    mx = warp_max64(mx);
    double sum = 0.0;
    for (int e = lane; e < a.E; e += 32) {
      const float l = to_f(row[e]);
      if (usable(l)) sum += exp((double)finite_top(l) - mx);
    }
    den = warp_sum(sum);
  }
  double* gs = sc + a.E;
  for (int e = lane; e < a.E; e += 32) {
    const float lf = to_f(row[e]);
    const double l = (double)finite_top(lf);
    const double s = soft ? exp(l - mx) / den : 1.0 / (1.0 + exp(-l));
    const float b = a.bias ? a.bias[e] : 0.0f;
    const bool ok = usable(lf) && b > -INFINITY;
    sc[e] = ok ? s + (double)b : -INFINITY;
  }
  __syncwarp();
  unsigned long long open = ~0ull;  // bit g: group g is kept
  const int n = a.E / a.groups;
  if (a.groups > 1) {
    for (int g = 0; g < a.groups; ++g) {
      double v1 = -INFINITY, v2 = -INFINITY;  // the two best of this lane, then of the group
      for (int i = lane; i < n; i += 32) {
        const double c = sc[g * n + i];
        if (c > v1) { v2 = v1; v1 = c; }
        else if (c > v2) v2 = c;
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        const double o1 = __shfl_xor_sync(kFull, v1, off), o2 = __shfl_xor_sync(kFull, v2, off);
        v2 = fmax(fmin(v1, o1), fmax(v2, o2));
        v1 = fmax(v1, o1);
      }
      if (lane == 0) gs[g] = a.group_top == 2 && v2 > -INFINITY ? v1 + v2 : v1;
    }
    __syncwarp();
    open = 0ull;
    for (int r = 0; r < a.top_groups; ++r) {
      double bv = 0.0;
      int bi = -1;
      for (int g = lane; g < a.groups; g += 32)
        if (!((open >> g) & 1ull) && (bi < 0 || gs[g] > bv)) { bv = gs[g]; bi = g; }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        const double ov = __shfl_xor_sync(kFull, bv, off);
        const int oi = __shfl_xor_sync(kFull, bi, off);
        if (oi >= 0 && (bi < 0 || ov > bv || (ov == bv && oi < bi))) { bv = ov; bi = oi; }
      }
      open |= 1ull << bi;
    }
  }
  unsigned taken = 0;  // bit i: expert lane + 32 i is taken
  int mine = -1;
  for (int j = 0; j < a.k; ++j) {
    double bv = 0.0;
    int bi = -1;
    for (int e = lane, i = 0; e < a.E; e += 32, ++i) {
      if ((taken >> i) & 1u) continue;
      if (a.groups > 1 && !((open >> (e / n)) & 1ull)) continue;
      double c = sc[e];
      if (!a.bias && c > -INFINITY) c = (double)finite_top(to_f(row[e]));  // the order of the logits
      if (bi < 0 || c > bv) { bv = c; bi = e; }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const double ov = __shfl_xor_sync(kFull, bv, off);
      const int oi = __shfl_xor_sync(kFull, bi, off);
      if (oi >= 0 && (bi < 0 || ov > bv || (ov == bv && oi < bi))) { bv = ov; bi = oi; }
    }
    if ((bi & 31) == lane) taken |= 1u << (bi >> 5);
    if (lane == j) mine = bi;
  }
  __syncwarp();
  return mine;
}

// Gates of the selected experts: lane j < k holds expert e (any lane order), W lanes
// from lane 0 on take part.  Renormalised gates divide out the row's largest factor
// first, so that a row of very negative logits does not lose its sum:
//   1 / (1 + exp(-l)) = exp(min(l, 0)) / (1 + exp(-|l|)).
// lse: log-sum-exp of the row (softmax without renormalisation).
template <int W>
__device__ __forceinline__ float gate_of(const SelectArgs& a, float lf, float b, bool live,
                                         float row_max, float row_den) {
  const bool ok = live && usable(lf) && b > -INFINITY;
  const float l = finite_top(lf);
  float w;
  if (!a.renorm) {
    w = !ok ? 0.0f
            : a.score == SMOE_SCORE_SOFTMAX ? expf(l - row_max) / row_den : 1.0f / (1.0f + expf(-l));
    return a.scale * w;
  }
  const float top = a.score == SMOE_SCORE_SOFTMAX ? l : fminf(l, 0.0f);
  float m = ok ? top : -INFINITY;
#pragma unroll
  for (int off = W / 2; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, off));
  w = ok ? expf(top - m) : 0.0f;
  if (a.score == SMOE_SCORE_SIGMOID && ok) w /= 1.0f + expf(-fabsf(l));
  float sum = w;
#pragma unroll
  for (int off = W / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(kFull, sum, off);
  return w > 0.0f ? a.scale * (w / sum) : 0.0f;
}

template <typename T>
__global__ void __launch_bounds__(kWarps * 32)
select64_kernel(const T* __restrict__ logits, SelectArgs a, int32_t* __restrict__ idx,
                float* __restrict__ gates) {
  extern __shared__ double smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  double* sc = smem + (size_t)warp * (a.E + a.groups);
  const int t = blockIdx.x * kWarps + warp;
  if (t >= a.T) return;
  const T* row = logits + (size_t)t * a.ld;
  const int e = select_row64(row, a, sc, lane);
  float mx = -INFINITY, den = 0.0f;
  if (a.score == SMOE_SCORE_SOFTMAX && !a.renorm) {
    for (int i = lane; i < a.E; i += 32) {
      const float l = to_f(row[i]);
      if (usable(l)) mx = fmaxf(mx, finite_top(l));
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, off));
    for (int i = lane; i < a.E; i += 32) {
      const float l = to_f(row[i]);
      if (usable(l)) den += expf(finite_top(l) - mx);
    }
    den = warp_sum(den);
  }
  const float lf = e >= 0 ? to_f(row[e]) : 0.0f;
  const float b = e >= 0 && a.bias ? a.bias[e] : 0.0f;
  const float g = gate_of<32>(a, lf, b, e >= 0, mx, den);
  if (e >= 0) {
    idx[(size_t)t * a.k + lane] = e;
    gates[(size_t)t * a.k + lane] = g;
  }
}

// Gradient of the logits, one warp per row.  With A = sum_i g_i dg_i:
//   renormalised:  dl_j = (g_j dg_j - g_j A / scale) (1 - s_j if sigmoid)
//   sigmoid:       dl_j = g_j dg_j (1 - s_j)
//   softmax:       dl_e = [e selected] g_e dg_e - p_e A      (every expert)
// 1 - s = 1 / (1 + exp(l)).  A gate of 0 (an expert that was not available) passes
// nothing on.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32)
select_bwd_kernel(const T* __restrict__ logits, SelectArgs a, const int32_t* __restrict__ idx,
                  const float* __restrict__ gates, const float* __restrict__ dgates,
                  T* __restrict__ dl, unsigned* err) {
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= a.T) return;
  const T* row = logits + (size_t)t * a.ld;
  T* out = dl + (size_t)t * a.E;
  int e = -1;
  float gd = 0.0f, g = 0.0f;
  if (lane < a.k) {
    e = idx[(size_t)t * a.k + lane];
    g = gates[(size_t)t * a.k + lane];
    if (e < 0 || e >= a.E) {
      report_error(err, ERRBIT_DATA);
      e = -1;
    }
    gd = e >= 0 && g != 0.0f ? g * dgates[(size_t)t * a.k + lane] : 0.0f;
  }
  const float A = warp_sum(gd);
  const bool dense = a.score == SMOE_SCORE_SOFTMAX && !a.renorm;
  float mx = -INFINITY, den = 0.0f;
  if (dense) {
    for (int i = lane; i < a.E; i += 32) {
      const float l = to_f(row[i]);
      if (usable(l)) mx = fmaxf(mx, finite_top(l));
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, off));
    for (int i = lane; i < a.E; i += 32) {
      const float l = to_f(row[i]);
      if (usable(l)) den += expf(finite_top(l) - mx);
    }
    den = warp_sum(den);
  }
  for (int i = lane; i < a.E; i += 32) {
    float d = 0.0f;
    if (dense) {
      const float l = to_f(row[i]);
      if (usable(l)) d = -(expf(finite_top(l) - mx) / den) * A;
    }
    out[i] = from_f<T>(d);
  }
  __syncwarp();
  if (e >= 0) {
    float d = 0.0f;
    const float l = to_f(row[e]);
    if (dense) {
      d = gd - (usable(l) ? (expf(finite_top(l) - mx) / den) * A : 0.0f);
    } else if (g != 0.0f) {
      d = a.renorm ? gd - g * (A / a.scale) : gd;
      if (a.score == SMOE_SCORE_SIGMOID) d *= 1.0f / (1.0f + expf(l));
    }
    out[e] = from_f<T>(d);
  }
}

}  // namespace

cudaError_t launch_select(const void* logits, const SelectArgs& a, smoe_dtype dt, int32_t* idx,
                          float* gates, cudaStream_t s) {
  const size_t smem = (size_t)kWarps * (a.E + a.groups) * sizeof(double);
  const int grid = cdiv(a.T, kWarps);
  if (dt == SMOE_BF16)
    select64_kernel<bf16><<<grid, kWarps * 32, smem, s>>>((const bf16*)logits, a, idx, gates);
  else
    select64_kernel<float><<<grid, kWarps * 32, smem, s>>>((const float*)logits, a, idx, gates);
  return cudaGetLastError();
}

cudaError_t launch_select_bwd(const void* logits, const SelectArgs& a, smoe_dtype dt,
                              const int32_t* idx, const float* gates, const float* dgates, void* dl,
                              unsigned* err, cudaStream_t s) {
  const int grid = cdiv(a.T, kWarps);
  if (dt == SMOE_BF16)
    select_bwd_kernel<bf16><<<grid, kWarps * 32, 0, s>>>((const bf16*)logits, a, idx, gates, dgates,
                                                         (bf16*)dl, err);
  else
    select_bwd_kernel<float><<<grid, kWarps * 32, 0, s>>>((const float*)logits, a, idx, gates,
                                                          dgates, (float*)dl, err);
  return cudaGetLastError();
}

}  // namespace smoe
