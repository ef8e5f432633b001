// qk_norm.cu -- RMS norm of queries and keys for each head with the position rotation
// in the same pass, forward and backward (smoe_moa_qk_norm_rope_fwd / _bwd), and its
// serving form, which stores keys and values in a paged cache (smoe_moa_cache_append).
//
//   u = w x / sqrt(mean(x^2) + eps)      per head of head_dim values, fp32
//   (y_a, y_b) = (u_a cos t - u_b sin t, u_b cos t + u_a sin t),  t = position * inv_freq
//   backward, with du = the upstream gradient turned back by t and r = 1/sqrt(...):
//   dw = sum du x r,   dx = r (w du - x r mean(w du x r))
//
// One pass over the data: a lane holds two 16-byte pieces of a head, V values from its
// first half and V from its second (V = 8 bf16, 4 fp32), so that a pair is always in one
// lane: (i, head_dim/2 + i), or (2i, 2i + 1) when interleaved.  head_dim / (2V) lanes
// share a head; the mean is log2 of that many shuffles.  A lane keeps its row's cosines
// and sines for all heads of the row.
//
// Forward, a lane asks for the pieces of kBatch heads before it uses the first, and for a
// row's pieces before its position: outputs may be the inputs, so the compiler does not move
// loads across stores by itself.  Backward, whose sums and weights fill the registers, it
// copies its pieces with cp.async into places of its own in shared memory, kSteps - 1 heads
// ahead and across rows; no lane waits for another.
//
// Angles: far positions need more than fp32.  inv_freq / (2 pi) is held as a 64-bit
// fixed-point fraction of a turn, so position * fraction modulo 2^64 is the angle with
// whole turns dropped exactly; its upper 32 bits go to sincospif (bf16: to sin.approx).
//
// Bound: latency, then instructions.  A pass over 84 MB (8192 tokens, 4 slots, 4 heads of 128
// bf16; 13 us at the copy rate) takes 20.5 us, 14 with the input in L2: SMs are active for
// 74% of the launch and issue in 53% of those cycles; warps wait for loads and for fixed
// latencies.  The backward (126 MB, 19.5 us) takes 30 us, 27 with the input in L2, at 83%
// and 63%.  Two fp32 values go to an instruction, blocks are one wave.
#include <atomic>

#include "tc_ptx.cuh"

namespace smoe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
// One wave of blocks on 148 SMs.  The backward's number fixes the order of dw's sums.
constexpr int kFwdThreads = 128, kFwdBlocks = 4 * 148;
constexpr int kThreads = 256, kBlocks = 2 * 148;

template <typename T>
struct Geo {
  static constexpr int V = 16 / sizeof(T);  // values per 16-byte piece
  static constexpr int kBatch = 4;          // heads loaded ahead, forward
  static constexpr int kSteps = 3;          // of the backward's rings, a head each
};

// Two neighbouring fp32 values in one register pair: products and sums of both in one
// instruction, which halves what bounds these kernels.
typedef unsigned long long f2;
__device__ __forceinline__ f2 pair(float lo, float hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 halves(f2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

__device__ __forceinline__ void unpack_piece(const uint4& u, f2* v, const float*) {
  v[0] = pair(__uint_as_float(u.x), __uint_as_float(u.y));
  v[1] = pair(__uint_as_float(u.z), __uint_as_float(u.w));
}
__device__ __forceinline__ void unpack_piece(const uint4& u, f2* v, const bf16*) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ void store_piece(float* p, const f2* v) {
  const float2 a = halves(v[0]), b = halves(v[1]);
  *reinterpret_cast<float4*>(p) = make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void store_piece(bf16* p, const f2* v) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 h = halves(v[i]);
    f[2 * i] = h.x;
    f[2 * i + 1] = h.y;
  }
  *reinterpret_cast<uint4*>(p) = pack8(f);
}

__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <int LPH>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int off = LPH / 2; off > 0; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
  return v;
}
template <int LPH>
__device__ __forceinline__ float head_max(float v) {
#pragma unroll
  for (int off = LPH / 2; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, off));
  return v;
}

// Fraction of a turn per position, modulo one turn, in units of 2^-64.
__device__ __forceinline__ unsigned long long turn_fraction(float inv_freq) {
  double t = (double)inv_freq * 0.15915494309189533577;  // 1 / (2 pi)
  t -= floor(t);
  return (unsigned long long)(t * 18446744073709551616.0);
}
template <typename T>
__device__ __forceinline__ void turn(unsigned long long f, int pos, float* c, float* s) {
  const unsigned long long a = f * (unsigned long long)(long long)pos;
  const int hi = (int)(unsigned)((a + 0x80000000ull) >> 32);  // turns * 2^32, in [-1/2, 1/2)
  if (sizeof(T) == 2) {  // values of 8 bits: sin.approx is within 2^-20.5 between -pi and pi
    const float r = (float)hi * 1.4629180792671596e-9f;  // hi 2 pi / 2^32
    *s = __sinf(r);
    *c = __cosf(r);
  } else {
    sincospif((float)hi * 4.656612873077393e-10f, s, c);  // hi 2^-31 = turns * 2
  }
}

// Frequency index of pair i (i < V) of lane `sub`.
template <typename T, int DH, bool kInter>
__device__ __forceinline__ int pair_freq(int sub, int i) {
  constexpr int V = Geo<T>::V;
  if (!kInter) return sub * V + i;
  return i < V / 2 ? sub * (V / 2) + i : DH / 4 + sub * (V / 2) + i - V / 2;
}
// Cosines and sines of the lane's V pairs, and minus the sines (in the order of the values
// when pairs are halves apart).
template <int V>
struct Turn {
  f2 c[V / 2], s[V / 2], n[V / 2];
};
template <typename T, int V>
__device__ __forceinline__ void turns(const unsigned long long* fr, bool rot, int pos, float sign, Turn<V>& t) {
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    float c0 = 1.0f, s0 = 0.0f, c1 = 1.0f, s1 = 0.0f;
    if (rot) {
      turn<T>(fr[2 * i], pos, &c0, &s0);
      turn<T>(fr[2 * i + 1], pos, &c1, &s1);
    }
    t.c[i] = pair(c0, c1);
    t.s[i] = pair(sign * s0, sign * s1);
    t.n[i] = pair(-sign * s0, -sign * s1);
  }
}
// Turns the lane's 2V values x (first V: piece a, last V: piece b) by its V pairs.
template <int V, bool kInter>
__device__ __forceinline__ void rotate(f2* x, const Turn<V>& t) {
  if (!kInter) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const f2 a = x[i], b = x[V / 2 + i];
      x[i] = fma2(b, t.n[i], mul2(a, t.c[i]));
      x[V / 2 + i] = fma2(a, t.s[i], mul2(b, t.c[i]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float2 c = halves(t.c[i / 2]), s = halves(t.s[i / 2]), v = halves(x[i]);
      const float ci = i % 2 ? c.y : c.x, si = i % 2 ? s.y : s.x;
      x[i] = pair(v.x * ci - v.y * si, v.y * ci + v.x * si);
    }
  }
}
template <int V>
__device__ __forceinline__ void load_weights(const float* wp, int at_a, int at_b, f2* w) {
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    w[i] = wp ? pair(wp[at_a + 2 * i], wp[at_a + 2 * i + 1]) : pair(1.0f, 1.0f);
    w[V / 2 + i] = wp ? pair(wp[at_b + 2 * i], wp[at_b + 2 * i + 1]) : pair(1.0f, 1.0f);
  }
}

// Where the rows of a part come from and what happens to them.
enum Part : int { PART_Q = 0, PART_K = 1, PART_V = 2 };

struct KArgs {
  QkArgs a;
  smoe_kv_cache c;  // serving form
  int nb[3];        // blocks of each part
  int hpu;          // heads a unit (a group of lanes) walks through
};

__device__ __forceinline__ int unit_row(int u, int chunks) { return chunks == 1 ? u : u / chunks; }

constexpr int kListed = 512;  // sequences whose starts and lengths a block holds
// Position (and cache slot) of token t in the serving form.  False: leave the row as
// it is (padding, or a data error, which is reported).
__device__ __forceinline__ bool serving_place(const KArgs& g, const int* starts, const int* lens, int t, int* pos,
                                              int64_t* page, int* off) {
  const smoe_kv_cache& c = g.c;
  int b = t, after = 1;  // rows of the sequence from this one on
  if (g.a.starts) {
    if (t < starts[0] || t >= starts[c.B]) return false;  // rows outside every sequence
    int lo = 0, hi = c.B - 1;  // the last sequence that starts at or before t
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (starts[mid] <= t) lo = mid; else hi = mid - 1;
    }
    b = lo;
    after = starts[b + 1] - t;
  } else if (lens[b] == 0) {
    return false;  // an unused row of the batch
  }
  const int len = lens[b];
  const long long p = (long long)len - after;
  if (after <= 0 || p < 0 || len > (long long)c.max_pages * c.page_size) {
    report_error(g.a.err, ERRBIT_DATA);
    return false;
  }
  *pos = (int)p;
  const int in_table = (int)p / c.page_size;
  const int id = c.block_table[(int64_t)b * c.table_stride + in_table];
  if (id < 0 || id >= c.num_pages) {
    report_error(g.a.err, ERRBIT_DATA);
    return false;
  }
  *page = id;
  *off = (int)p - in_table * c.page_size;
  return true;
}

__device__ __forceinline__ uint16_t e4m3_pair(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

template <typename T, int DH, bool kInter, bool kServe>
__global__ void __launch_bounds__(kFwdThreads, 4)
qk_fwd_kernel(const __grid_constant__ KArgs g) {
  constexpr int V = Geo<T>::V, LPH = DH / (2 * V), UPB = kFwdThreads / LPH, HB = Geo<T>::kBatch;
  const QkArgs& a = g.a;
  int part = PART_Q, blk = blockIdx.x;
  while (part < PART_V && blk >= g.nb[part]) blk -= g.nb[part++];
  const int heads = part == PART_Q ? a.q_heads : a.kv_heads;
  const int rows = part == PART_Q ? a.T * a.kslots : a.T;
  const T* x = (const T*)(part == PART_Q ? a.q : part == PART_K ? a.k : a.v);
  const int64_t ldx = part == PART_Q ? a.ldq : part == PART_K ? a.ldk : a.ldv;
  const float* wp = part == PART_Q ? a.wq : a.wk;
  const bool norm = a.norm && part != PART_V, rot = a.inv_freq && part != PART_V;
  const int sub = threadIdx.x % LPH, chunks = cdiv(heads, g.hpu);
  const int units = rows * chunks;  // at most the rows' heads: below 2^31 / head_dim

  f2 w[V];
  load_weights<V>(norm ? wp : nullptr, sub * V, DH / 2 + sub * V, w);
  unsigned long long fr[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    fr[i] = rot ? turn_fraction(a.inv_freq[pair_freq<T, DH, kInter>(sub, i)]) : 0ull;
  }

  __shared__ int listed[kServe ? 2 * kListed + 1 : 1];
  const int *starts = a.starts, *lens = g.c.seq_lens;
  if (kServe && starts && g.c.B <= kListed) {  // the search for a row's sequence is a chain of reads
    for (int i = threadIdx.x; i <= g.c.B; i += kFwdThreads) {
      listed[i] = starts[i];
      if (i < g.c.B) listed[g.c.B + 1 + i] = lens[i];
    }
    __syncthreads();
    starts = listed;
    lens = listed + g.c.B + 1;
  }

  // the loop count is the same for all lanes of a block: the head sums shuffle whole warps
  const int first = blk * UPB, step = g.nb[part] * UPB;
  const bool slots = part == PART_Q && a.sorted_slot;
  int next = first + threadIdx.x / LPH;  // the next unit, and its row's slot
  int next_slot = slots && next < units ? a.sorted_slot[unit_row(next, chunks)] : 0;
  for (int u0 = first; u0 < units; u0 += step) {
    const int u = next;
    bool live = u < units;
    const int row = live ? unit_row(u, chunks) : 0;
    const int h0 = live ? (u - row * chunks) * g.hpu : 0;
    const int slot = slots ? next_slot : row;
    next = u <= units - step ? u + step : units;
    if (slots && next < units) next_slot = a.sorted_slot[unit_row(next, chunks)];
    const T* xr = x + row * ldx;
    uint4 raw[HB][2];
    auto fetch = [&](int hh) {
#pragma unroll
      for (int j = 0; j < HB; ++j) {
        raw[j][0] = raw[j][1] = make_uint4(0, 0, 0, 0);
        if (live && hh + j < g.hpu && h0 + hh + j < heads) {
          const T* p = xr + (h0 + hh + j) * DH + sub * V;
          raw[j][0] = *reinterpret_cast<const uint4*>(p);
          raw[j][1] = *reinterpret_cast<const uint4*>(p + DH / 2);
        }
      }
    };
    fetch(0);
    int t = row, pos = 0, off = 0;
    int64_t page = 0;
    if (live && part == PART_Q) {
      if (slot < 0 || slot >= rows) {
        report_error(a.err, ERRBIT_DATA);
        live = false;
      }
      t = slot / a.kslots;
    }
    if (kServe) live = live && serving_place(g, starts, lens, t, &pos, &page, &off);
    else if (live && rot) pos = a.positions[t];
    Turn<V> cs;
    turns<T, V>(fr, rot, pos, 1.0f, cs);
    for (int h4 = 0; h4 < g.hpu; h4 += HB) {
      if (h4 > 0) fetch(h4);
#pragma unroll
      for (int j = 0; j < HB; ++j) {
        const int hh = h4 + j;
        if (hh >= g.hpu) break;
        const int h = h0 + hh;
        const bool on = live && h < heads;
        f2 v[V];
        unpack_piece(raw[j][0], v, (const T*)nullptr);
        unpack_piece(raw[j][1], v + V / 2, (const T*)nullptr);
        if (norm) {
          f2 ss = 0;
#pragma unroll
          for (int i = 0; i < V; ++i) ss = fma2(v[i], v[i], ss);
          const float2 sh = halves(ss);
          const float r = rsqrtf(head_sum<LPH>(sh.x + sh.y) * (1.0f / DH) + a.eps);
          const f2 rr = pair(r, r);
#pragma unroll
          for (int i = 0; i < V; ++i) v[i] = mul2(v[i], mul2(rr, w[i]));
        }
        if (rot) rotate<V, kInter>(v, cs);
        if (!kServe || part == PART_Q) {
          if (on) {
            T* out = (T*)(part == PART_Q ? a.q_out : a.k_out) + ((int64_t)row * heads + h) * DH;
            store_piece(out + sub * V, v);
            store_piece(out + DH / 2 + sub * V, v + V / 2);
          }
        } else {
          const bool is_k = part == PART_K;
          const int64_t at = page * (is_k ? g.c.k_page_stride : g.c.v_page_stride) +
                             off * (is_k ? g.c.k_token_stride : g.c.v_token_stride) +
                             h * (is_k ? g.c.k_head_stride : g.c.v_head_stride);
          if (g.c.k_scale == nullptr) {
            if (on) {
              T* out = (T*)(is_k ? g.c.k : g.c.v) + at;
              store_piece(out + sub * V, v);
              store_piece(out + DH / 2 + sub * V, v + V / 2);
            }
          } else {  // one scale per (token, head): its largest magnitude maps to 448
            float m = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
              const float2 f = halves(v[i]);
              m = fmaxf(m, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
            m = head_max<LPH>(m);
            // (and at least the smallest normal number)
            const float sc = m > 0.0f ? fmaxf(m / 448.0f, 1.17549435e-38f) : 1.0f;
            // Codes are those of the quotients x / sc: with bf16 rows many lie half way between
            // two codes, where a product with the reciprocal alone may be off the middle.  A
            // product q with the rounded reciprocal, the remainder x - q sc (exact) and
            // q + remainder / sc round as the quotient does (P. Markstein, IBM J. Res. Dev. 34,
            // 1990), here at sizes that keep the remainder from underflow.  Prompts of up to 1400
            // tokens: 22.5 us, with the one product 20.9.
            float s1 = sc;
            if (sc < 0x1p-60f) {
              s1 = sc * 0x1p64f;
#pragma unroll
              for (int i = 0; i < V; ++i) v[i] = mul2(v[i], pair(0x1p64f, 0x1p64f));
            }
            const float inv = 1.0f / s1, minus = s1 < INFINITY ? -s1 : 0.0f;
            const f2 inv2 = pair(inv, inv), minus2 = pair(minus, minus);
            if (on) {
              uint8_t* out = (uint8_t*)(is_k ? g.c.k : g.c.v) + at;
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                uint16_t q[V / 2];
#pragma unroll
                for (int i = 0; i < V / 2; ++i) {
                  const f2 x = v[half * (V / 2) + i], q1 = mul2(x, inv2);
                  const float2 f = halves(fma2(fma2(q1, minus2, x), inv2, q1));
                  q[i] = e4m3_pair(f.x, f.y);
                }
                uint2 u8;
                u8.x = q[0] | ((uint32_t)q[1] << 16);
                u8.y = q[V / 2 - 2] | ((uint32_t)q[V / 2 - 1] << 16);
                *reinterpret_cast<uint2*>(out + half * (DH / 2) + sub * V) = u8;
              }
              if (sub == 0)
                (is_k ? g.c.k_scale : g.c.v_scale)[(page * g.c.page_size + off) * heads + h] = sc;
            }
          }
        }
      }
    }
  }
}

template <typename T, int DH, bool kInter>
__global__ void __launch_bounds__(kThreads, 2)
qk_bwd_kernel(const __grid_constant__ KArgs g) {
  constexpr int V = Geo<T>::V, LPH = DH / (2 * V), UPB = kThreads / LPH, S = Geo<T>::kSteps;
  extern __shared__ uint4 places[];  // [S][4][kThreads]
  __shared__ float red[kThreads / 32][DH];
  const QkArgs& a = g.a;
  const int part = (int)blockIdx.x < g.nb[0] ? PART_Q : PART_K;
  const int blk = part == PART_Q ? blockIdx.x : blockIdx.x - g.nb[0];
  const int heads = part == PART_Q ? a.q_heads : a.kv_heads;
  const int rows = part == PART_Q ? a.T * a.kslots : a.T;
  const T* x = (const T*)(part == PART_Q ? a.q : a.k);
  const T* dy = (const T*)(part == PART_Q ? a.dyq : a.dyk);
  const int64_t ldx = part == PART_Q ? a.ldq : a.ldk, ldy = part == PART_Q ? a.lddyq : a.lddyk;
  T* dx = (T*)(part == PART_Q ? a.q_out : a.k_out);
  const float* wp = part == PART_Q ? a.wq : a.wk;
  const bool want_dw = (part == PART_Q ? a.dwq : a.dwk) != nullptr;
  const bool rot = a.inv_freq != nullptr;
  const int sub = threadIdx.x % LPH, chunks = cdiv(heads, g.hpu);
  const int units = rows * chunks;  // at most the rows' heads: below 2^31 / head_dim

  f2 w[V], dw[V];
  load_weights<V>(wp, sub * V, DH / 2 + sub * V, w);
  unsigned long long fr[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    dw[i] = 0;
    fr[i] = rot ? turn_fraction(a.inv_freq[pair_freq<T, DH, kInter>(sub, i)]) : 0ull;
  }
  const int first = blk * UPB, step = g.nb[part] * UPB;
  const bool slots = part == PART_Q && a.sorted_slot;
  int next = first + threadIdx.x / LPH;  // the next unit, and its row's slot
  int next_slot = slots && next < units ? a.sorted_slot[unit_row(next, chunks)] : 0;
  int put_unit = next, put_head = 0, put = 0, get = 0;  // the step that is asked for next; stages
  auto ask = [&]() {
    const bool there = put_unit < units;
    const int row = there ? unit_row(put_unit, chunks) : 0, h = (put_unit - row * chunks) * g.hpu + put_head;
    const bool on = there && h < heads;
    const T* yp = on ? dy + row * ldy + h * DH + sub * V : dy;
    const T* xp = on && a.norm ? x + row * ldx + h * DH + sub * V : dy;
    const uint32_t at = smem_u32(&places[(4 * put) * kThreads + threadIdx.x]);
    cp_async16(at, yp, on ? 16u : 0u);
    cp_async16(at + 16 * kThreads, on ? yp + DH / 2 : yp, on ? 16u : 0u);
    cp_async16(at + 32 * kThreads, xp, on && a.norm ? 16u : 0u);
    cp_async16(at + 48 * kThreads, on && a.norm ? xp + DH / 2 : xp, on && a.norm ? 16u : 0u);
    cp_commit();
    put = put + 1 == S ? 0 : put + 1;
    if (++put_head == g.hpu) {
      put_head = 0;
      put_unit = put_unit <= units - step ? put_unit + step : units;
    }
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) ask();
  for (int u0 = first; u0 < units; u0 += step) {
    const int u = next;
    bool live = u < units;
    const int row = live ? unit_row(u, chunks) : 0;
    const int h0 = live ? (u - row * chunks) * g.hpu : 0;
    const int slot = slots ? next_slot : row;
    next = u <= units - step ? u + step : units;
    if (slots && next < units) next_slot = a.sorted_slot[unit_row(next, chunks)];
    int t = row;
    if (live && part == PART_Q) {
      if (slot < 0 || slot >= rows) {
        report_error(a.err, ERRBIT_DATA);
        live = false;
      }
      t = slot / a.kslots;
    }
    const int pos = live && rot ? a.positions[t] : 0;
    Turn<V> cs;
    turns<T, V>(fr, rot, pos, -1.0f, cs);
    for (int hh = 0; hh < g.hpu; ++hh) {
      const int h = h0 + hh;
      const bool on = live && h < heads;
      f2 v[V], d[V];
      cp_wait<S - 2>();
      uint4* mine = places + (4 * get) * kThreads + threadIdx.x;
      if (!live) {  // a skipped row, whatever it holds, adds nothing to dw
#pragma unroll
        for (int i = 0; i < 4; ++i) mine[i * kThreads] = make_uint4(0, 0, 0, 0);
      }
      unpack_piece(mine[0], d, (const T*)nullptr);
      unpack_piece(mine[kThreads], d + V / 2, (const T*)nullptr);
      unpack_piece(mine[2 * kThreads], v, (const T*)nullptr);
      unpack_piece(mine[3 * kThreads], v + V / 2, (const T*)nullptr);
      get = get + 1 == S ? 0 : get + 1;
      ask();  // into the stage of the step before this one
      if (rot) rotate<V, kInter>(d, cs);
      if (a.norm) {
        // with r = 1 / sqrt(...) and wd = w du: dx = r wd - x r^3 mean(wd x)
        f2 ss = 0, dot = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          ss = fma2(v[i], v[i], ss);
          dot = fma2(mul2(w[i], d[i]), v[i], dot);
        }
        const float2 sh = halves(ss), dh = halves(dot);
        const float r = rsqrtf(head_sum<LPH>(sh.x + sh.y) * (1.0f / DH) + a.eps);
        const float m = -(r * head_sum<LPH>(dh.x + dh.y)) * (1.0f / DH) * r * r;
        const f2 rr = pair(r, r), mm = pair(m, m);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const f2 rd = mul2(rr, d[i]);
          dw[i] = fma2(rd, v[i], dw[i]);
          d[i] = fma2(v[i], mm, mul2(rd, w[i]));
        }
      }
      if (on && dx) {
        T* out = dx + ((int64_t)row * heads + h) * DH;
        store_piece(out + sub * V, d);
        store_piece(out + DH / 2 + sub * V, d + V / 2);
      }
    }
  }
  cp_wait<0>();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!want_dw) return;
  // this block's share of dw: lanes of equal `sub`, then the warps in order
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int i = 0; i < 2 * V; ++i) {
    const float2 f = halves(dw[i / 2]);
    float v = i % 2 ? f.y : f.x;
#pragma unroll
    for (int off = LPH; off < 32; off <<= 1) v += __shfl_xor_sync(kFull, v, off);
    if (lane < LPH) red[warp][(i < V ? 0 : DH / 2 - V) + sub * V + i] = v;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < DH; i += kThreads) {
    float v = 0.0f;
#pragma unroll
    for (int j = 0; j < kThreads / 32; ++j) v += red[j][i];
    a.partial[(size_t)blockIdx.x * DH + i] = v;
  }
}

// dw[i] = sum of the blocks' shares: 32 columns by 32 block slices, joined in order.
__global__ void __launch_bounds__(1024)
qk_dw_sum_kernel(const float* __restrict__ partial, int nq, int nk, int DH, float* dwq, float* dwk) {
  __shared__ float red[32][33];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int per = DH / 32, part = blockIdx.x / per;
  const int col = (blockIdx.x % per) * 32 + threadIdx.x;
  float* out = part == 0 ? dwq : dwk;
  const int b0 = part == 0 ? 0 : nq, nb = part == 0 ? nq : nk;
  if (!out) return;
  float v = 0.0f;
#pragma unroll 8
  for (int b = threadIdx.y; b < nb; b += 32) v += partial[(size_t)(b0 + b) * DH + col];
  red[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y == 0) {
    v = 0.0f;
#pragma unroll
    for (int j = 0; j < 32; ++j) v += red[j][threadIdx.x];
    out[col] = v;
  }
}

// Heads a unit walks through: all of the row's heads share its cosines and sines, but a
// small batch spreads its heads over more lanes (148 SMs x 8 warps filled first).
int heads_per_unit(long long rows, int heads, int lph) {
  return rows * lph >= 148 * 256 ? heads : 1;
}
int lanes_per_head(int head_dim, int es) { return head_dim * es / 32; }

// All blocks are resident at once and share out the parts' units in proportion.
void plan(KArgs& g, int head_dim, int es, int threads, int most) {
  const QkArgs& a = g.a;
  const int lph = lanes_per_head(head_dim, es), upb = threads / lph;
  const int heads = a.q_heads > a.kv_heads ? a.q_heads : a.kv_heads;
  g.hpu = heads_per_unit((long long)a.T * a.kslots, heads, lph);
  const long long rows[3] = {a.q ? (long long)a.T * a.kslots : 0, a.k ? a.T : 0, a.v ? a.T : 0};
  long long blocks[3], all = 0;
  for (int p = 0; p < 3; ++p) {
    blocks[p] = (rows[p] * cdiv(p == 0 ? a.q_heads : a.kv_heads, g.hpu) + upb - 1) / upb;
    all += blocks[p];
  }
  for (int p = 0; p < 3; ++p)
    g.nb[p] = (int)(all <= most || blocks[p] == 0 ? blocks[p] : 1 + blocks[p] * (most - 3) / all);
}

template <typename T, int DH>
cudaError_t fwd(const KArgs& g, cudaStream_t s) {
  const int grid = g.nb[0] + g.nb[1] + g.nb[2];
  if (g.a.interleaved) qk_fwd_kernel<T, DH, true, false><<<grid, kFwdThreads, 0, s>>>(g);
  else qk_fwd_kernel<T, DH, false, false><<<grid, kFwdThreads, 0, s>>>(g);
  return cudaGetLastError();
}
template <int DH>
cudaError_t append(const KArgs& g, cudaStream_t s) {
  const int grid = g.nb[0] + g.nb[1] + g.nb[2];
  if (g.a.interleaved) qk_fwd_kernel<bf16, DH, true, true><<<grid, kFwdThreads, 0, s>>>(g);
  else qk_fwd_kernel<bf16, DH, false, true><<<grid, kFwdThreads, 0, s>>>(g);
  return cudaGetLastError();
}
// The attribute that allows the rings belongs to the kernel on a device and stays: set once
// for each.
template <void (*Kern)(KArgs)>
cudaError_t launch_rings(const KArgs& g, int grid, cudaStream_t s) {
  constexpr size_t smem = (size_t)Geo<bf16>::kSteps * 4 * kThreads * sizeof(uint4);
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (e == cudaSuccess && !(done.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  }
  if (e != cudaSuccess) return e;
  Kern<<<grid, kThreads, smem, s>>>(g);
  return cudaGetLastError();
}
template <typename T, int DH>
cudaError_t bwd(const KArgs& g, cudaStream_t s) {
  const int grid = g.nb[0] + g.nb[1];
  const cudaError_t e = g.a.interleaved ? launch_rings<qk_bwd_kernel<T, DH, true>>(g, grid, s)
                                        : launch_rings<qk_bwd_kernel<T, DH, false>>(g, grid, s);
  if (e != cudaSuccess || (!g.a.dwq && !g.a.dwk)) return e;
  // starts early and waits for the shares on the device
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2 * (DH / 32));
  cfg.blockDim = dim3(32, 32);
  cfg.stream = s;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, qk_dw_sum_kernel, (const float*)g.a.partial, g.nb[0], g.nb[1], DH, g.a.dwq,
                            g.a.dwk);
}

}  // namespace

size_t qk_bwd_partial_floats(int T, int kslots, int q_heads, int kv_heads, int head_dim) {
  (void)T; (void)kslots; (void)q_heads; (void)kv_heads;
  return (size_t)kBlocks * head_dim;
}

cudaError_t launch_qk_fwd(const QkArgs& a, int head_dim, smoe_dtype dt, cudaStream_t s) {
  KArgs g{};
  g.a = a;
  plan(g, head_dim, dt == SMOE_BF16 ? 2 : 4, kFwdThreads, kFwdBlocks);
  if (dt == SMOE_BF16) return head_dim == 64 ? fwd<bf16, 64>(g, s) : fwd<bf16, 128>(g, s);
  return head_dim == 64 ? fwd<float, 64>(g, s) : fwd<float, 128>(g, s);
}

cudaError_t launch_cache_append(const QkArgs& a, cudaStream_t s) {
  KArgs g{};
  g.a = a;
  g.c = *a.cache;
  plan(g, g.c.head_dim, 2, kFwdThreads, kFwdBlocks);
  return g.c.head_dim == 64 ? append<64>(g, s) : append<128>(g, s);
}

cudaError_t launch_qk_bwd(const QkArgs& a, int head_dim, smoe_dtype dt, cudaStream_t s) {
  KArgs g{};
  g.a = a;
  plan(g, head_dim, dt == SMOE_BF16 ? 2 : 4, kThreads, kBlocks);
  if (dt == SMOE_BF16) return head_dim == 64 ? bwd<bf16, 64>(g, s) : bwd<bf16, 128>(g, s);
  return head_dim == 64 ? bwd<float, 64>(g, s) : bwd<float, 128>(g, s);
}

}  // namespace smoe
