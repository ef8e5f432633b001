// select.cu -- routing from given logits (smoe_route_select, smoe_route_select_bwd):
// softmax or sigmoid scores, a selection bias, expert groups, top-k and gates.
//
//   s_e  = 1 / (1 + exp(-l_e))  or  exp(l_e) / sum_u exp(l_u)
//   c_e  = s_e + b_e                       (what is ranked; without b: the logits)
//   best k of c_e, inside the best top_groups groups when there are groups
//   gate = scale * s_e, or scale * s_e / (sum of the selected s)
//
// Selected ids are whole numbers: they are those of scores compared in 64 bits, ties to
// the lower id.  One warp has a row.  It ranks in 32 bits with scores whose error is
// bounded, and where two ranks that decide the outcome lie closer together than that
// bound (and are not equal because logit and bias are), it ranks the row again in 64 bits.
// Logits of a normal distribution bring that about in one row of 1300.
//
// Bound: instructions, and the rows in 64 bits at the end.  16384 rows of 256 fp32 logits in
// 8 groups are 18 MB, 2.8 us at the copy rate; they take 25 us, 23 with the logits in L2,
// and 970 instructions a row, issued in 73% of the cycles that SMs are active.  Without
// groups 18 us, without bias too 14, and then with k = 1 11.  Rows without a near tie (one
// row repeated) take 19: a row in 64 bits waits for its own exponentials and rounds while
// the rest of the GPU has finished.
#include <cfloat>
#include <climits>

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
// Largest value of the warp; NaN is no value.
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float warp_min(float v) {
  float r;
  asm volatile("redux.sync.min.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// How far apart two ranks of a row have to be in 32 bits to rank so in 64: kNear times the
// largest score there can be and kRound times the ranks' size; twice that for the sums of
// two that groups are ranked by.  ex2 and rcp are within 2^-22 and 2^-23 of their value and
// an exponent x loses 2^-23 |x|; times s (1 - s) that is under 2^-24 each, with rcp's own
// and two roundings 2^-22 for a sigmoid, 2^-21 for two.  A softmax is within 2^-18.4 of
// itself (its sum has up to 1024 terms, 32 in a lane and 5 steps across), two within 2^-17
// of the largest.  The bias added rounds by 2^-24 of each rank, and the place that takes up
// to three bits of it moves it by 7 units of 2^-23.
constexpr float kNearSigmoid = 1.0f / (1 << 21), kNearSoftmax = 1.0f / (1 << 17), kRound = 1.0f / (1 << 20);

// The lane that holds the warp's largest (v, then lowest e) of 64-bit values; e < 0: none.
__device__ __forceinline__ int best_lane64(double v, int e) {
  long long k = __double_as_longlong(v + 0.0);  // -0 is 0
  k ^= (k >> 63) & 0x7fffffffffffffffll;        // integer order
  const int hi = e < 0 ? INT_MIN : (int)(k >> 32);
  const int top = __reduce_max_sync(kFull, hi);
  bool in = e >= 0 && hi == top;
  const unsigned low = __reduce_max_sync(kFull, in ? (unsigned)k : 0u);
  in = in && (unsigned)k == low;
  const unsigned first = __reduce_min_sync(kFull, in ? (unsigned)e : 0xffffffffu);
  return __ffs(__ballot_sync(kFull, in && (unsigned)e == first)) - 1;
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
      open |= 1ull << __shfl_sync(kFull, bi, best_lane64(bv, bi));
    }
  }
  unsigned taken = 0;  // bit i: expert lane + 32 i is taken
  int mine = -1, bi = -1;
  double bv = 0.0;
  bool stale = true;
  for (int j = 0; j < a.k; ++j) {
    if (stale) {  // this lane's best expert that is left
      bi = -1;
      for (int e = lane, i = 0; e < a.E; e += 32, ++i) {
        if ((taken >> i) & 1u) continue;
        if (a.groups > 1 && !((open >> (e / n)) & 1ull)) continue;
        double c = sc[e];
        if (!a.bias && c > -INFINITY) c = (double)finite_top(to_f(row[e]));  // the order of the logits
        if (bi < 0 || c > bv) { bv = c; bi = e; }
      }
    }
    __syncwarp();
    const int src = best_lane64(bv, bi), e = __shfl_sync(kFull, bi, src);
    stale = lane == src;
    if (stale) taken |= 1u << (e >> 5);
    if (lane == j) mine = e;
  }
  __syncwarp();
  return mine;
}

// Gates of the selected experts: lane j < k holds expert e (any lane order), W lanes
// from lane 0 on take part.  Renormalised gates divide out the row's largest factor
// first, so that a row of very negative logits does not lose its sum:
//   1 / (1 + exp(-l)) = exp(min(l, 0)) / (1 + exp(-|l|)).
// row_max, row_den: largest logit and sum of the row (softmax without renormalisation).
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
  const float m = warp_max(ok ? top : -INFINITY);
  w = ok ? expf(top - m) : 0.0f;
  if (a.score == SMOE_SCORE_SIGMOID && ok) w /= 1.0f + expf(-fabsf(l));
  float sum = w;
#pragma unroll
  for (int off = W / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(kFull, sum, off);
  return w > 0.0f ? a.scale * (w / sum) : 0.0f;
}

// Logits of this lane's experts as they lie in memory.
template <typename T, int NV>
__device__ __forceinline__ void load_experts(const T* __restrict__ at, int have, bool wide, float* l) {
  constexpr int VB = NV * sizeof(T) < 16 ? NV * sizeof(T) : 16, VE = VB / sizeof(T);  // of a wide load
#pragma unroll
  for (int i = 0; i < NV; ++i) l[i] = -INFINITY;
  if (wide) {
#pragma unroll
    for (int i = 0; i < NV; i += VE) {
      T w[VE];
      if (VB == 16) *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(at + i);
      if (VB == 8) *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(at + i);
      if (VB == 4) *reinterpret_cast<unsigned*>(w) = *reinterpret_cast<const unsigned*>(at + i);
      if (VB == 2) w[0] = at[i];
#pragma unroll
      for (int j = 0; j < VE; ++j) l[i + j] = to_f(w[j]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (i < have) l[i] = to_f(at[i]);
  }
}

// Where a lane's experts are: those of a group lie in `lpg` lanes (a power of two, one
// group: the warp), C <= NV neighbours in a lane, so that a group's best are found in
// log2(lpg) steps and lanes are in the order of the ids.
struct Lane {
  int lane, lpg, group, e0, have;
};

// select_row64 with the row's scores in registers, so that a lane's exponentials overlap.
template <typename T, int NV>
__device__ __noinline__ int select_row64_wide(const T* __restrict__ row, const SelectArgs& a, const Lane p) {
  float lf[NV], b[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const float l = i < p.have ? to_f(row[p.e0 + i]) : -INFINITY;
    lf[i] = usable(l) ? finite_top(l) : -INFINITY;
    b[i] = a.bias && i < p.have ? a.bias[p.e0 + i] : 0.0f;
  }
  const bool soft = a.score == SMOE_SCORE_SOFTMAX;
  double c[NV];
  double mx = -INFINITY, den = 1.0;
  if (soft) {
#pragma unroll
    for (int i = 0; i < NV; ++i) mx = fmax(mx, (double)lf[i]);
    mx = warp_max64(mx);
    den = 0.0;
#pragma unroll
    for (int i = 0; i < NV; ++i) den += lf[i] > -INFINITY ? exp((double)lf[i] - mx) : 0.0;
    den = warp_sum(den);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const double l = lf[i];
    const double s = soft ? exp(l - mx) / den : 1.0 / (1.0 + exp(-l));
    c[i] = i < p.have && lf[i] > -INFINITY && b[i] > -INFINITY ? s + (double)b[i] : -INFINITY;
  }
  bool open = p.group < a.groups;
  if (a.groups > 1) {
    double v1 = -INFINITY, v2 = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      v2 = fmax(v2, fmin(v1, c[i]));
      v1 = fmax(v1, c[i]);
    }
    for (int off = 1; off < p.lpg; off <<= 1) {
      const double o1 = __shfl_xor_sync(kFull, v1, off), o2 = __shfl_xor_sync(kFull, v2, off);
      v2 = fmax(fmin(v1, o1), fmax(v2, o2));
      v1 = fmax(v1, o1);
    }
    const double gs = a.group_top == 2 && v2 > -INFINITY ? v1 + v2 : v1;
    int ahead = 0;
    for (int g = 0; g < a.groups; ++g) {
      const double o = __shfl_sync(kFull, gs, g * p.lpg);
      ahead += o > gs || (o == gs && g < p.group);
    }
    open = open && ahead < a.top_groups;
  }
  unsigned left = open ? (1u << p.have) - 1 : 0;
  if (!a.bias) {
#pragma unroll
    for (int i = 0; i < NV; ++i) c[i] = lf[i];  // the order of the logits
  }
  int mine = -1, be = -1;
  double bv = 0.0;
  bool stale = true;
  for (int j = 0; j < a.k; ++j) {
    if (stale) {
      be = -1;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (((left >> i) & 1u) && (be < 0 || c[i] > bv)) { bv = c[i]; be = p.e0 + i; }
    }
    __syncwarp();
    const int src = best_lane64(bv, be), e = __shfl_sync(kFull, be, src);
    stale = p.lane == src;
    if (stale) left &= ~(1u << (e - p.e0));
    if (p.lane == j) mine = e;
  }
  return mine;
}

// One row in 32 bits: l: this lane's logits (usable or -inf), b: its biases (-inf: expert
// not available).  Returns as select_row64; -2 in every lane if two ranks lie too close
// together.
template <typename T, int NV, bool BIAS>
__device__ __forceinline__ int select_row32(const T* __restrict__ row, const SelectArgs& a, const Lane& p,
                                            const float* l, const float* b, float* row_max, float* row_den) {
  const bool soft = a.score == SMOE_SCORE_SOFTMAX;
  // A rank is an integer in the order of the floats.  Where its low bits are to spare they
  // hold the place in the lane, the first highest: with scores, whose last bits are not
  // exact, and with bf16 logits.
  constexpr bool SORT = NV <= 8, PACK = SORT && (BIAS || sizeof(T) == 2);
  float c[NV];
  float mx = 0.0f, inv = 1.0f;
  if (soft && (BIAS || a.groups > 1 || !a.renorm)) {
    mx = l[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) mx = fmaxf(mx, l[i]);
    mx = warp_max(mx);
    float den = 0.0f;
    if (mx > -INFINITY) {
#pragma unroll
      for (int i = 0; i < NV; ++i) den += ex2((l[i] - mx) * 1.4426950408889634f);
    }
    den = warp_sum(den);
    inv = rcp(den);
    *row_max = mx;
    *row_den = den;
  }
  const float near = soft ? kNearSoftmax * fminf(inv, 1.0f) : kNearSigmoid;
  // scores, with the bias; without one what is ranked in the end is the logits
  if (BIAS || a.groups > 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const float s = soft ? ex2((l[i] - mx) * 1.4426950408889634f) * inv
                           : rcp(1.0f + ex2(l[i] * -1.4426950408889634f));
      c[i] = l[i] > -INFINITY ? (BIAS ? s + b[i] : s) : -INFINITY;
    }
  }
  bool open = p.group < a.groups, close_by = false;
  if (a.groups > 1) {
    float v1 = -INFINITY, v2 = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      v2 = fmaxf(v2, fminf(v1, c[i]));
      v1 = fmaxf(v1, c[i]);
    }
    for (int off = 1; off < p.lpg; off <<= 1) {
      const float o1 = __shfl_xor_sync(kFull, v1, off), o2 = __shfl_xor_sync(kFull, v2, off);
      v2 = fmaxf(fminf(v1, o1), fmaxf(v2, o2));
      v1 = fmaxf(v1, o1);
    }
    const float gs = a.group_top == 2 && v2 > -INFINITY ? v1 + v2 : v1;
    int ahead = 0;
    for (int g = 0; g < a.groups; ++g) {
      const float o = __shfl_sync(kFull, gs, g * p.lpg);
      ahead += o > gs || (o == gs && g < p.group);
    }
    const bool there = open;
    open = open && ahead < a.top_groups;
    if (a.top_groups < a.groups) {
      const float in = warp_min(open ? gs : INFINITY), out = warp_max(there && !open ? gs : -INFINITY);
      const float size = fmaxf(fabsf(v1), v2 > -INFINITY ? fabsf(v2) : 0.0f);
      const float most = warp_max(there && v1 > -INFINITY ? size : 0.0f);
      close_by = out > -INFINITY && !(in - out > 2.0f * (near + kRound * most));
      // a sum that leaves fp32's range still ranks before a group without experts
      close_by = close_by || (v2 > -INFINITY && gs == -INFINITY);
    }
  }
  // INT_MIN: not to be chosen (an unavailable expert's -inf ranks above that)
  int key[NV], place[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int f = __float_as_int((BIAS ? c[i] : l[i]) + 0.0f);  // -0 is 0
    const int o = f ^ ((f >> 31) & 0x7fffffff);
    key[i] = open && i < p.have ? (PACK ? (o & ~7) | (7 - i) : o) : INT_MIN;
    place[i] = i;
  }
  // a lane of few experts puts them in order (neighbours change places, so equal ones stay
  // as they are); one of many looks for its best each time
  int best = INT_MIN;
  if (SORT) {
#pragma unroll
    for (int r = NV - 1; r > 0; --r)
#pragma unroll
      for (int i = 0; i < r; ++i) {
        const int x = max(key[i], key[i + 1]), y = min(key[i], key[i + 1]);
        if (!PACK) {
          const bool swap = key[i + 1] > key[i];
          const int u = swap ? place[i + 1] : place[i], v = swap ? place[i] : place[i + 1];
          place[i] = u; place[i + 1] = v;
        }
        key[i] = x; key[i + 1] = y;
      }
    best = key[0];
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) best = max(best, key[i]);
  }
  const int rounds = BIAS ? a.k + 1 : a.k;  // with scores the next one too, to be compared
  int mine = -1, rank = INT_MIN;
  for (int j = 0; j < rounds; ++j) {
    const int head = PACK ? best & ~7 : best;  // equal ones in two lanes: the first lane's
    const int top = __reduce_max_sync(kFull, head);
    if (top == INT_MIN) break;  // no candidate left (only after the k-th)
    const int src = __ffs(__ballot_sync(kFull, head == top)) - 1;
    int e = p.e0 + (PACK ? 7 - (best & 7) : place[0]);
    if (p.lane == src) {
      if (SORT) {
#pragma unroll
        for (int i = 0; i + 1 < NV; ++i) {
          key[i] = key[i + 1];
          if (!PACK) place[i] = place[i + 1];
        }
        key[NV - 1] = INT_MIN;
        best = key[0];
      } else {
        bool found = false;
        best = INT_MIN;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (!found && key[i] == top) {
            found = true;
            e = p.e0 + i;
            key[i] = INT_MIN;
          }
          best = max(best, key[i]);
        }
      }
    }
    e = __shfl_sync(kFull, e, src);
    if (p.lane == j) {
      mine = e;
      rank = top;
    }
  }
  if (BIAS) {
    const int below = __shfl_down_sync(kFull, rank, 1);
    auto value = [](int r) -> float { return __int_as_float(r ^ ((r >> 31) & 0x7fffffff)); };
    // (a rank of -inf loses its last bits to NaN, no rank is one too: neither is near)
    auto near_each = [&](float hi, float lo) -> bool {
      return lo > -INFINITY && !(hi - lo > near + kRound * fabsf(hi));
    };
    const bool near_by = p.lane < a.k && near_each(value(rank), value(below));
    if (__any_sync(kFull, near_by)) {  // equal logits and biases are equal in 64 bits as well
      float lm = 0.0f, bm = 0.0f;
      if (mine >= 0) {
        lm = finite_top(to_f(row[mine]));
        bm = a.bias[mine];
      }
      const float ln = __shfl_down_sync(kFull, lm, 1), bn = __shfl_down_sync(kFull, bm, 1);
      const bool equal = lm == ln && bm == bn;
      close_by = close_by || (near_by && !equal);
      // the last selected rank and the next are equal: so must be all that are near them
      if (__any_sync(kFull, near_by && equal && p.lane == a.k - 1)) {
        const float last = value(__shfl_sync(kFull, rank, a.k - 1));
        lm = __shfl_sync(kFull, lm, a.k - 1);
        bm = __shfl_sync(kFull, bm, a.k - 1);
#pragma unroll
        for (int i = 0; i < NV; ++i) {  // what is left in this lane
          if (key[i] == INT_MIN || !near_each(last, value(PACK ? key[i] & ~7 : key[i]))) continue;
          const int e = p.e0 + (PACK ? 7 - (key[i] & 7) : place[i]);
          close_by = close_by || finite_top(to_f(row[e])) != lm || a.bias[e] != bm;
        }
      }
    }
  }
  if (__any_sync(kFull, close_by)) return -2;
  return p.lane < a.k ? mine : -1;
}

// One warp per row, with many experts to a lane for several, whose logits are asked for a
// row ahead; lpg = 0: every row in 64 bits.
// The ranking in 64 bits is rare, so it may spill: nine CTAs of the common path fit an SM.
constexpr int per_sm(int nv) { return nv <= 8 ? 9 : 4; }
template <typename T, int NV, bool BIAS>
__global__ void __launch_bounds__(kWarps * 32, per_sm(NV))
select_kernel(const T* __restrict__ logits, SelectArgs a, int lpg, int lpg_log2, int n, int C,
              int32_t* __restrict__ idx, float* __restrict__ gates) {
  extern __shared__ double smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int in0 = lpg ? (lane & (lpg - 1)) * C : 0;
  Lane p;
  p.lane = lane;
  p.lpg = lpg;
  p.group = lane >> lpg_log2;
  p.e0 = p.group * n + in0;
  p.have = p.group < a.groups && lpg ? max(0, min(C, n - in0)) : 0;
  constexpr int VE = NV * sizeof(T) < 16 ? NV : 16 / sizeof(T);
  const bool wide = p.have == NV && ((a.ld | p.e0) & (VE - 1)) == 0;
  float b[NV], next[NV];
  if (BIAS) {
    constexpr int VB = NV < 4 ? NV : 4;
    const bool wide_bias = p.have == NV && (p.e0 & (VB - 1)) == 0 && ((uintptr_t)a.bias & (4 * VB - 1)) == 0;
    load_experts<float, NV>(a.bias + p.e0, p.have, wide_bias, b);
#pragma unroll
    for (int i = 0; i < NV; ++i) b[i] = usable(b[i]) ? b[i] : -INFINITY;
  }
  constexpr bool SEVERAL = NV > 8;  // rows to a warp: of over 100 experts, so t + step fits
  const int step = SEVERAL ? gridDim.x * kWarps : 0;
  int t = blockIdx.x * kWarps + warp;
  if (t < a.T && lpg) load_experts<T, NV>(logits + (size_t)t * a.ld + p.e0, p.have, wide, next);
  for (; t < a.T; t = SEVERAL ? t + step : a.T) {
    const T* row = logits + (size_t)t * a.ld;
    float mx = -INFINITY, den = 0.0f;
    int e = -2;
    if (lpg > 0) {
      float l[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) l[i] = usable(next[i]) ? finite_top(next[i]) : -INFINITY;
      if (SEVERAL && t + step < a.T) load_experts<T, NV>(row + (size_t)step * a.ld + p.e0, p.have, wide, next);
      e = select_row32<T, NV, BIAS>(row, a, p, l, b, &mx, &den);
      if (NV <= 8 && e == -2) e = select_row64_wide<T, NV>(row, a, p);
    }
    if ((NV > 8 || lpg == 0) && e == -2)
      e = select_row64(row, a, smem + (size_t)warp * (a.E + a.groups), lane);
    if (lpg == 0 && a.score == SMOE_SCORE_SOFTMAX && !a.renorm) {
      for (int i = lane; i < a.E; i += 32) {
        const float l = to_f(row[i]);
        if (usable(l)) mx = fmaxf(mx, finite_top(l));
      }
      mx = warp_max(mx);
      for (int i = lane; i < a.E; i += 32) {
        const float l = to_f(row[i]);
        if (usable(l)) den += expf(finite_top(l) - mx);
      }
      den = warp_sum(den);
    }
    const float lf = e >= 0 ? to_f(row[e]) : 0.0f;
    const float bm = BIAS && e >= 0 ? a.bias[e] : 0.0f;
    const float g = gate_of<SMOE_MAX_TOPK>(a, lf, bm, e >= 0, mx, den);
    if (e >= 0) {
      idx[(size_t)t * a.k + lane] = e;
      gates[(size_t)t * a.k + lane] = g;
    }
  }
}

// Gradient of the logits, one warp per row.  With A = sum_i g_i dg_i:
//   renormalised:  dl_j = (g_j dg_j - g_j A / scale) (1 - s_j if sigmoid)
//   sigmoid:       dl_j = g_j dg_j (1 - s_j)
//   softmax:       dl_e = [e selected] g_e dg_e - p_e A      (every expert)
// 1 - s = 1 / (1 + exp(l)).  A gate of 0 (an expert that was not available) passes
// nothing on, and an expert whose p is 0 gets 0 even where A is NaN or infinite.
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
      const float l = to_f(row[i]), p = usable(l) ? expf(finite_top(l) - mx) / den : 0.0f;
      if (p > 0.0f) d = -p * A;
    }
    out[i] = from_f<T>(d);
  }
  __syncwarp();
  if (e >= 0) {
    float d = 0.0f;
    const float l = to_f(row[e]);
    if (dense) {
      const float p = usable(l) ? expf(finite_top(l) - mx) / den : 0.0f;
      d = gd - (p > 0.0f ? p * A : 0.0f);
    } else if (g != 0.0f) {
      d = a.renorm ? gd - g * (A / a.scale) : gd;
      if (a.score == SMOE_SCORE_SIGMOID) d *= 1.0f / (1.0f + expf(l));
    }
    out[e] = from_f<T>(d);
  }
}

// The same with LPR lanes for a row, which hold it in registers: 16-byte pieces p * LPR +
// sub (p < NP) of V values.  Every value is written once; a row's selected experts are
// passed round among its lanes.
template <typename T, int LPR, int NP>
__global__ void __launch_bounds__(kWarps * 32)
select_bwd_wide_kernel(const T* __restrict__ logits, SelectArgs a, const int32_t* __restrict__ idx,
                       const float* __restrict__ gates, const float* __restrict__ dgates,
                       T* __restrict__ dl, unsigned* err) {
  constexpr int V = 16 / sizeof(T), NK = SMOE_MAX_TOPK / LPR > 1 ? SMOE_MAX_TOPK / LPR : 1;
  const int lane = threadIdx.x & 31, sub = lane & (LPR - 1);
  const int t = (int)(((long long)blockIdx.x * kWarps * 32 + threadIdx.x) / LPR);
  const bool live = t < a.T;
  const T* row = logits + (size_t)(live ? t : 0) * a.ld;
  const bool dense = a.score == SMOE_SCORE_SOFTMAX && !a.renorm;
  float x[NP][V];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int at = (p * LPR + sub) * V;
#pragma unroll
    for (int i = 0; i < V; ++i) x[p][i] = -INFINITY;
    if (dense && live && at < a.E) {
      T w[V];
      *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(row + at);
#pragma unroll
      for (int i = 0; i < V; ++i) x[p][i] = usable(to_f(w[i])) ? finite_top(to_f(w[i])) : -INFINITY;
    }
  }
  // this lane's selected experts: slots sub, sub + LPR
  int e[NK];
  float g[NK], d[NK], lsel[NK], A = 0.0f;
#pragma unroll
  for (int q = 0; q < NK; ++q) {
    const int j = q * LPR + sub;
    e[q] = -1;
    g[q] = d[q] = lsel[q] = 0.0f;
    if (live && j < a.k) {
      e[q] = idx[(size_t)t * a.k + j];
      g[q] = gates[(size_t)t * a.k + j];
      if (e[q] < 0 || e[q] >= a.E) {
        report_error(err, ERRBIT_DATA);
        e[q] = -1;
      }
      if (e[q] >= 0 && g[q] != 0.0f) {
        d[q] = g[q] * dgates[(size_t)t * a.k + j];
        if (a.score == SMOE_SCORE_SIGMOID) lsel[q] = to_f(row[e[q]]);
      }
    }
    A += d[q];
  }
#pragma unroll
  for (int off = LPR / 2; off > 0; off >>= 1) A += __shfl_xor_sync(kFull, A, off);
  if (dense) {
    float mx = -INFINITY;
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int i = 0; i < V; ++i) mx = fmaxf(mx, x[p][i]);
#pragma unroll
    for (int off = LPR / 2; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, off));
    float den = 0.0f;
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        x[p][i] = x[p][i] > -INFINITY ? expf(x[p][i] - mx) : 0.0f;
        den += x[p][i];
      }
#pragma unroll
    for (int off = LPR / 2; off > 0; off >>= 1) den += __shfl_xor_sync(kFull, den, off);
    const float f = den > 0.0f ? -A / den : 0.0f;
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int i = 0; i < V; ++i) x[p][i] = x[p][i] > 0.0f ? x[p][i] * f : 0.0f;
  } else {
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int i = 0; i < V; ++i) x[p][i] = 0.0f;
#pragma unroll
    for (int q = 0; q < NK; ++q) {
      if (a.renorm) d[q] -= g[q] * (A / a.scale);
      if (a.score == SMOE_SCORE_SIGMOID) d[q] *= 1.0f / (1.0f + expf(lsel[q]));
      if (g[q] == 0.0f) d[q] = 0.0f;
    }
  }
#pragma unroll
  for (int q = 0; q < NK; ++q)
    for (int j = 0; j < LPR && q * LPR + j < a.k; ++j) {
      const int ej = __shfl_sync(kFull, e[q], j, LPR);
      const float dj = __shfl_sync(kFull, d[q], j, LPR);
      const int at = ej / V;  // -1 / V = 0, but then dj = 0
      if ((at & (LPR - 1)) == sub) {
#pragma unroll
        for (int p = 0; p < NP; ++p)
#pragma unroll
          for (int i = 0; i < V; ++i)
            if ((p * LPR + sub) * V + i == ej) x[p][i] += dj;
      }
    }
  if (!live) return;
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int at = (p * LPR + sub) * V;
    if (at >= a.E) continue;
    T w[V];
#pragma unroll
    for (int i = 0; i < V; ++i) w[i] = from_f<T>(x[p][i]);
    *reinterpret_cast<uint4*>(dl + (size_t)t * a.E + at) = *reinterpret_cast<const uint4*>(w);
  }
}

// Blocks of n rows each for T rows, up to 2^31 - 1 of them.
int blocks(int T, int n) { return (int)(((long long)T + n - 1) / n); }

template <typename T>
cudaError_t select(const T* logits, const SelectArgs& a, int32_t* idx, float* gates, cudaStream_t s) {
  const size_t smem = (size_t)kWarps * (a.E + a.groups) * sizeof(double);
  int lpg = a.groups <= 32 ? 32 : 0;
  while (lpg * a.groups > 32) lpg >>= 1;
  int lg = 0;
  while ((1 << lg) < lpg) ++lg;
  const int n = a.E / a.groups, C = lpg ? cdiv(n, lpg) : 0;
  // 32 values are what fits a lane's registers beside their scores
  // One row for each warp, so that CTAs come and go while a row is ranked in 64 bits; with
  // many experts a lane several, whose logits are asked for a row ahead (when this rule was
  // made: 16384 rows of 256 experts in groups 27 us, with several rows a warp 31; of 1024
  // experts 135 and 119).
  // More than 32 groups, or 32 experts to a lane, rank every row in 64 bits from loops (256
  // experts in 64 groups: 336 us).
#define SELECT(NV, L)                                                                             \
  const int rows = NV <= 8 ? 1 : blocks(a.T, 148 * per_sm(NV) * kWarps);                          \
  const int grid = blocks(a.T, kWarps * rows);                                                    \
  a.bias ? select_kernel<T, NV, true><<<grid, kWarps * 32, smem, s>>>(logits, a, L, lg, n, C, idx, gates) \
         : select_kernel<T, NV, false><<<grid, kWarps * 32, smem, s>>>(logits, a, L, lg, n, C, idx, gates)
  if (lpg == 0 || C > 32) { SELECT(1, 0); }
  else if (C == 1) { SELECT(1, lpg); }
  else if (C == 2) { SELECT(2, lpg); }
  else if (C <= 4) { SELECT(4, lpg); }
  else if (C <= 8) { SELECT(8, lpg); }
  else if (C <= 16) { SELECT(16, lpg); }
  else { SELECT(32, lpg); }
#undef SELECT
  return cudaGetLastError();
}

template <typename T>
cudaError_t select_bwd(const T* logits, const SelectArgs& a, const int32_t* idx, const float* gates,
                       const float* dgates, T* dl, unsigned* err, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const int pieces = a.E / V;
  if (a.E % V || a.ld % V || pieces > 8 * 32) {  // rows that are not whole 16-byte pieces
    select_bwd_kernel<T><<<blocks(a.T, kWarps), kWarps * 32, 0, s>>>(logits, a, idx, gates, dgates, dl, err);
    return cudaGetLastError();
  }
#define SELECT_BWD(LPR, NP)                                                                              \
  select_bwd_wide_kernel<T, LPR, NP><<<blocks(a.T, kWarps * 32 / LPR), kWarps * 32, 0, s>>>(logits, a, idx, \
                                                                                          gates, dgates, dl, err)
  if (pieces <= 8) SELECT_BWD(8, 1);
  else if (pieces <= 16) SELECT_BWD(16, 1);
  else if (pieces <= 32) SELECT_BWD(32, 1);
  else if (pieces <= 64) SELECT_BWD(32, 2);
  else if (pieces <= 128) SELECT_BWD(32, 4);
  else SELECT_BWD(32, 8);
#undef SELECT_BWD
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_select(const void* logits, const SelectArgs& a, smoe_dtype dt, int32_t* idx,
                          float* gates, cudaStream_t s) {
  return dt == SMOE_BF16 ? select((const bf16*)logits, a, idx, gates, s)
                         : select((const float*)logits, a, idx, gates, s);
}

cudaError_t launch_select_bwd(const void* logits, const SelectArgs& a, smoe_dtype dt,
                              const int32_t* idx, const float* gates, const float* dgates, void* dl,
                              unsigned* err, cudaStream_t s) {
  return dt == SMOE_BF16 ? select_bwd((const bf16*)logits, a, idx, gates, dgates, (bf16*)dl, err, s)
                         : select_bwd((const float*)logits, a, idx, gates, dgates, (float*)dl, err, s);
}

}  // namespace smoe
