// decode.cu -- attention of one new token for each sequence over a paged key/value
// cache (smoe_moa_decode): the serving form of the Mixture-of-Attention core.
//
//   o = sum_u softmax_u(<q, k_u> / sqrt(head_dim)) v_u,  lse = log sum_u exp(...)
// over the seq_len cached tokens u of the query's sequence, for the G = kslots *
// (q_heads / kv_heads) query rows that share a key head.
//
// The cache is read once, so bytes bound it: 4 G head_dim operations against
// 4 head_dim bytes (bf16) per key and head leave the tensor pipe far from busy.
//
// Split: the work is cut into units of 64 keys of one (sequence, key head) item; the
// items' units in a row are dealt out in equal runs to a fixed number of CTAs, so a
// ragged batch and a single long sequence load the GPU alike.  An item that a CTA holds
// whole is finished there; the shares of the others go to the workspace and a second
// kernel joins them in CTA order.  No atomics: a batch gives the same bits every time.
//
// A CTA's four warps each take 16 keys of a unit and are independent until the item
// ends: a warp copies its keys' rows with cp.async into its own ring in shared memory,
// a few units ahead and across items, and keeps a running maximum m, sum l and
// accumulator O of its own (one pass over the data):
//   S^T = K Q^T      mma m16n8k16, keys as rows, 8 queries as columns
//   m' = max(m, S), P = exp(S - m'), l = l e^(m-m') + sum P, O^T = O^T e^(m-m') + V^T P^T
// Keys as rows cost ceil(G/8) 8-column products instead of a 16-row tile padded with
// empty queries; P^T turns from accumulator to operand layout by movmatrix.
//
// P is rounded to bf16 for the second product (bf16 values need a bf16 operand): half
// a step is at most 2^-8 of each weight, the size of the rounding of the output itself.
#include <cuda_fp16.h>

#include "tc_ptx.cuh"

namespace smoe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kKeys = 16;                    // keys of a warp's share of a unit
constexpr int kUnit = kKeys * kWarps;        // keys of a unit

struct DecArgs {
  const bf16* q;
  int64_t ldq;
  const int32_t* inv;  // grouped row of each slot, or null: row = slot
  smoe_kv_cache c;
  int kslots, q_heads, group, G, mts;  // mts: query tiles of 8 NT rows
  float scale_log2;                    // log2(e) / sqrt(head_dim)
  bf16* o;
  float* lse;  // nullable
  // shares of split items: [grid][2] slots of R rows, R = 8 NT
  float* part_o;   // [grid][2][R][DH]
  float* part_ml;  // [grid][2][R][2]
  int4* desc;      // [grid]: item started and not ended here (b, item), last CTA of it or -1
  unsigned* err;
};

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, uint32_t src_bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(src_bytes)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
                 "{%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
                 "{%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t e4m3_to_half2(uint16_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// 2^x, to 2 ulp; -inf gives 0.
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

template <int DH, bool F8>
struct Tile {
  static constexpr int kRow = F8 ? DH : 2 * DH;    // bytes of a cached row of a head
  static constexpr int kChunks = kRow / 16;
  static constexpr int kRows = 2 * kKeys * kRow;   // a warp's K rows, then its V rows
  static constexpr int kStage = kRows + (F8 ? 2 * kKeys * 4 : 0);  // and their scales
  // Byte of 16-byte chunk c of row r: eight rows of one chunk lie in eight different
  // 16-byte bank groups, so that ldmatrix reads without conflicts.
  static __device__ __forceinline__ uint32_t at(int r, int c) {
    return (uint32_t)(r * kRow + ((c ^ (kChunks >= 8 ? (r & 7) : ((r >> 1) & 3))) << 4));
  }
};

// A place in the row of units: unit `tile` of item `it` of sequence b.
struct Cursor {
  int b, it, tile, tiles, len;
};

__device__ __forceinline__ int seq_len(const smoe_kv_cache& c, int b) {
  const long long cap = (long long)c.max_pages * c.page_size;
  const int n = c.seq_lens[b];
  return n < 0 ? 0 : (int)(n < cap ? n : cap);
}
__device__ __forceinline__ void next_unit(Cursor& p, const smoe_kv_cache& c, int items) {
  if (++p.tile < p.tiles) return;
  p.tile = 0;
  if (++p.it < items) return;
  p.it = 0;
  do {
    if (++p.b >= c.B) { p.len = 0; p.tiles = 1 << 30; return; }
    p.len = seq_len(c, p.b);
    p.tiles = (p.len + kUnit - 1) / kUnit;
  } while (p.tiles == 0);
}

// Row of o, q and lse of query n of query tile mt, key head kvh, sequence b; -1 for a
// column that stands for no query (or a slot that sorted_slot leaves out: reported).
__device__ __forceinline__ int query_row(const DecArgs& a, int b, int qi, int kvh, int* head) {
  if (qi >= a.G) return -1;
  *head = kvh * a.group + qi % a.group;
  const int slot = b * a.kslots + qi / a.group;
  if (!a.inv) return slot;
  const int r = a.inv[slot];
  if (r < 0 || r >= a.c.B * a.kslots) {
    report_error(a.err, ERRBIT_DATA);
    return -1;
  }
  return r;
}

template <int DH, int NT, bool F8, int STAGES>
__global__ void __launch_bounds__(kThreads)
decode_kernel(const __grid_constant__ DecArgs a) {
  using TL = Tile<DH, F8>;
  constexpr int R = 8 * NT, KS = DH / 16;
  constexpr int RED = DH + 4;  // row pitch of the joining buffer: conflict-free
  extern __shared__ __align__(128) uint8_t smem[];
  float* red = reinterpret_cast<float*>(smem + (size_t)kWarps * STAGES * TL::kStage);  // [R][RED]
  float* mls = red + R * RED;                                                          // [warps][R][2]
  __shared__ unsigned masks[kWarps][STAGES];
  __shared__ long long wsum[kWarps];
  __shared__ int s_b;
  __shared__ long long s_rem;

  const smoe_kv_cache& c = a.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int items = c.kv_heads * a.mts;
  const int cta = blockIdx.x;

  // ---- this CTA's run of units: [u0, u1) of all ------------------------------
  const int per = (c.B + kThreads - 1) / kThreads;
  const int bb0 = threadIdx.x * per, bb1 = min(c.B, bb0 + per);
  long long mine = 0;
  for (int b = bb0; b < bb1; ++b) {
    const int n = c.seq_lens[b];
    if (cta == 0 && (n < 0 || n > (long long)c.max_pages * c.page_size)) report_error(a.err, ERRBIT_DATA);
    mine += (seq_len(c, b) + kUnit - 1) / kUnit;
  }
  long long incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long v = __shfl_up_sync(kFull, incl, off);
    if (lane >= off) incl += v;
  }
  if (lane == 31) wsum[warp] = incl;
  __syncthreads();
  long long before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += wsum[w];
    total += wsum[w];
  }
  const long long U = total * items;
  const int ctas = (int)min((long long)gridDim.x, U);  // those with a run: no run is empty
  const long long u0 = cta < ctas ? U * cta / ctas : 0;
  const long long n_units = cta < ctas ? U * (cta + 1) / ctas - u0 : 0;
  if (n_units > 0 && u0 >= before * items && u0 < (before + mine) * items) {
    long long rem = u0 - before * items;
    for (int b = bb0; b < bb1; ++b) {
      const long long tu = (long long)((seq_len(c, b) + kUnit - 1) / kUnit) * items;
      if (rem < tu) { s_b = b; s_rem = rem; break; }
      rem -= tu;
    }
  }
  __syncthreads();

  // sequences without a cached token: o = 0, lse = -inf
  for (int b = cta; b < c.B; b += gridDim.x) {
    if (seq_len(c, b) > 0) continue;
    for (int i = threadIdx.x; i < a.G * c.kv_heads * (DH / 8); i += kThreads) {
      int head;
      const int row = query_row(a, b, i / (DH / 8) % a.G, i / (DH / 8) / a.G, &head);
      if (row < 0) continue;
      *reinterpret_cast<uint4*>(a.o + ((int64_t)row * a.q_heads + head) * DH + 8 * (i % (DH / 8))) =
          make_uint4(0, 0, 0, 0);
      if (a.lse && i % (DH / 8) == 0) a.lse[(int64_t)row * a.q_heads + head] = -INFINITY;
    }
  }
  if (threadIdx.x == 0) a.desc[cta] = make_int4(0, 0, -1, 0);
  if (n_units <= 0) return;

  Cursor cp;
  {
    const long long rem = s_rem;
    cp.b = s_b;
    cp.len = seq_len(c, cp.b);
    cp.tiles = (cp.len + kUnit - 1) / kUnit;
    cp.it = (int)(rem / cp.tiles);
    cp.tile = (int)(rem - (long long)cp.it * cp.tiles);
  }
  Cursor ld = cp;

  // ---- loads: lane r and lane 16 + r own key r of the warp's share --------------
  const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * STAGES) * TL::kStage;
  const int kr = lane & 15;
  auto page_of = [&](const Cursor& p) -> int {  // page of this lane's key, -1: none
    const int pos = p.tile * kUnit + warp * kKeys + kr;
    if (pos >= p.len) return -1;
    const int id = c.block_table[(int64_t)p.b * c.table_stride + pos / c.page_size];
    if (id < 0 || id >= c.num_pages) {
      report_error(a.err, ERRBIT_DATA);
      return -1;
    }
    return id;
  };
  auto issue = [&](const Cursor& p, int page, int stage) {
    const uint32_t base = ring + stage * TL::kStage;
    const int pos = p.tile * kUnit + warp * kKeys + kr;
    const int off = pos % c.page_size, kvh = p.it / a.mts;
    const int es = F8 ? 1 : 2;
    const bool ok = page >= 0;
    const int64_t pg = ok ? page : 0;
    const int64_t of = ok ? off : 0;
    const unsigned mask = __ballot_sync(kFull, ok) & 0xffffu;
    if (lane == 0) masks[warp][stage] = mask;
    const bool is_v = lane >= 16;
    const char* src = (const char*)(is_v ? c.v : c.k) +
                      (pg * (is_v ? c.v_page_stride : c.k_page_stride) +
                       of * (is_v ? c.v_token_stride : c.k_token_stride) +
                       kvh * (is_v ? c.v_head_stride : c.k_head_stride)) * es;
    if (F8) {
      const float* sc = (is_v ? c.v_scale : c.k_scale) + (pg * c.page_size + of) * c.kv_heads + kvh;
      cp_async4(base + TL::kRows + lane * 4, sc, ok ? 4u : 0u);
    }
    constexpr int RPI = 32 / TL::kChunks;  // rows per instruction
    const int sub = lane % TL::kChunks, rr = lane / TL::kChunks;
#pragma unroll
    for (int i = 0; i < 32 / RPI; ++i) {
      const int r = i * RPI + rr;  // 0..15: K rows, 16..31: V rows
      const char* s = (const char*)__shfl_sync(kFull, (unsigned long long)src, r);
      const uint32_t bytes = (mask >> (r & 15)) & 1u ? 16u : 0u;
      cp_async16(base + (r >> 4) * (kKeys * TL::kRow) + TL::at(r & 15, sub), s + sub * 16, bytes);
    }
  };

  int page = page_of(ld);
  long long loaded = 0;
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) {
    if (loaded < n_units) {
      issue(ld, page, s);
      ++loaded;
      next_unit(ld, c, items);
      if (loaded < n_units) page = page_of(ld);
    }
    cp_commit();
  }

  uint32_t qf[NT][KS][2];
  float qs[NT][2];  // F8: factor of this thread's two query columns
  float m[NT][2], l[NT][2];
  float oacc[NT][KS][4];
  const int tg = lane & 3, gr = lane >> 2;
  bool fresh = true;
  int t0 = cp.tile, stage = 0;

  for (long long i = 0; i < n_units; ++i) {
    if (fresh) {  // first unit of an item here
      fresh = false;
      t0 = cp.tile;
      const int mt = cp.it % a.mts, kvh = cp.it / a.mts;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        int head = 0;
        const int row = query_row(a, cp.b, mt * R + 8 * t + gr, kvh, &head);
        const bf16* qr = a.q + (row < 0 ? 0 : (int64_t)row * a.ldq + (int64_t)head * DH);
        float amax = 0.0f;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          // bf16: dims 2 tg + {0, 1} and + 8; e4m3 cache: the four dims 4 tg .. 4 tg + 3,
          // which is how ldmatrix deals out 8-bit rows
          const int d0 = 16 * k + (F8 ? 4 * tg : 2 * tg), d1 = d0 + (F8 ? 2 : 8);
          qf[t][k][0] = row < 0 ? 0u : *reinterpret_cast<const uint32_t*>(qr + d0);
          qf[t][k][1] = row < 0 ? 0u : *reinterpret_cast<const uint32_t*>(qr + d1);
          if (F8) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&qf[t][k][j]));
              amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
          }
        }
        if (F8) {  // queries as fp16, scaled by a power of two so that the largest is in [1, 2)
          amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
          amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
          int ex = (int)((__float_as_uint(amax) >> 23) & 0xff) - 127;
          ex = max(-100, min(100, ex));
          const float down = __uint_as_float((unsigned)(127 - ex) << 23);
          const float up = __uint_as_float((unsigned)(127 + ex) << 23);
#pragma unroll
          for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&qf[t][k][j]));
              qf[t][k][j] = pack_f16(f.x * down, f.y * down);
            }
          qs[t][0] = __shfl_sync(kFull, up, (2 * tg) * 4) * a.scale_log2;
          qs[t][1] = __shfl_sync(kFull, up, (2 * tg + 1) * 4) * a.scale_log2;
        } else {
          qs[t][0] = qs[t][1] = a.scale_log2;
        }
        m[t][0] = m[t][1] = -INFINITY;
        l[t][0] = l[t][1] = 0.0f;
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int j = 0; j < 4; ++j) oacc[t][k][j] = 0.0f;
      }
    }

    cp_wait<STAGES - 2>();
    __syncwarp();
    const uint32_t base = ring + stage * TL::kStage;
    const unsigned mask = masks[warp][stage];
    if (mask) {
      float s[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[t][j] = 0.0f;
      float ks0 = 1.0f, ks1 = 1.0f, vs0 = 1.0f, vs1 = 1.0f;
      if (!F8) {
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          uint32_t f[4];
          ldsm4(f, base + TL::at(((lane >> 3) & 1) * 8 + (lane & 7), 2 * k + (lane >> 4)));
#pragma unroll
          for (int t = 0; t < NT; ++t) mma16816<false>(s[t], f, qf[t][k][0], qf[t][k][1]);
        }
      } else {
#pragma unroll
        for (int k = 0; k < KS; k += 2) {  // 32 dims: two 16-byte chunks
          uint32_t f[4];
          ldsm4(f, base + TL::at(((lane >> 3) & 1) * 8 + (lane & 7), k + (lane >> 4)));
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t g[4];
            g[0] = e4m3_to_half2((uint16_t)f[2 * h]);
            g[1] = e4m3_to_half2((uint16_t)f[2 * h + 1]);
            g[2] = e4m3_to_half2((uint16_t)(f[2 * h] >> 16));
            g[3] = e4m3_to_half2((uint16_t)(f[2 * h + 1] >> 16));
#pragma unroll
            for (int t = 0; t < NT; ++t) mma16816<true>(s[t], g, qf[t][k + h][0], qf[t][k + h][1]);
          }
        }
        const float* sc = reinterpret_cast<const float*>(smem + (size_t)(warp * STAGES + stage) * TL::kStage + TL::kRows);
        ks0 = sc[gr]; ks1 = sc[gr + 8];
        vs0 = sc[16 + gr]; vs1 = sc[24 + gr];
      }
      // The reference m of a query's weights: its largest score; with scaled values the
      // largest score times the value's scale, so that the weights times the scales, which
      // are rounded to fp16 for the second product, are at most 1.
      const float ls0 = F8 ? fmaxf(log2f(vs0), -100.0f) : 0.0f, ls1 = F8 ? fmaxf(log2f(vs1), -100.0f) : 0.0f;
      const bool on0 = (mask >> gr) & 1u, on1 = (mask >> (gr + 8)) & 1u;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        uint32_t pf[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          s[t][j] = on0 ? s[t][j] * qs[t][j] * ks0 : -INFINITY;
          s[t][2 + j] = on1 ? s[t][2 + j] * qs[t][j] * ks1 : -INFINITY;
          float top = fmaxf(s[t][j] + ls0, s[t][2 + j] + ls1);
          top = fmaxf(top, __shfl_xor_sync(kFull, top, 4));
          top = fmaxf(top, __shfl_xor_sync(kFull, top, 8));
          top = fmaxf(top, __shfl_xor_sync(kFull, top, 16));
          const float mn = fmaxf(m[t][j], top);
          const float ref = mn == -INFINITY ? 0.0f : mn;
          const float al = ex2(m[t][j] - ref);
          m[t][j] = mn;
          s[t][j] = ex2(s[t][j] - ref);
          s[t][2 + j] = ex2(s[t][2 + j] - ref);
          l[t][j] = l[t][j] * al + (s[t][j] + s[t][2 + j]);
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            oacc[t][k][j] *= al;
            oacc[t][k][2 + j] *= al;
          }
        }
        if (F8) {
          pf[0] = transpose8(pack_f16(s[t][0] * vs0, s[t][1] * vs0));
          pf[1] = transpose8(pack_f16(s[t][2] * vs1, s[t][3] * vs1));
        } else {
          pf[0] = transpose8(pack_bf16(s[t][0], s[t][1]));
          pf[1] = transpose8(pack_bf16(s[t][2], s[t][3]));
        }
        s[t][0] = __uint_as_float(pf[0]);
        s[t][1] = __uint_as_float(pf[1]);
      }
      const uint32_t vb = base + kKeys * TL::kRow;
      if (!F8) {
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          uint32_t f[4];
          ldsm4_t(f, vb + TL::at((lane >> 4) * 8 + (lane & 7), 2 * k + ((lane >> 3) & 1)));
#pragma unroll
          for (int t = 0; t < NT; ++t)
            mma16816<false>(oacc[t][k], f, __float_as_uint(s[t][0]), __float_as_uint(s[t][1]));
        }
      } else {
#pragma unroll
        for (int k = 0; k < KS; k += 2) {
          // transposed pairs of bytes: keys 2 tg, 2 tg + 1 of dims 2 gr, 2 gr + 1
          uint32_t f[4];
          ldsm4_t(f, vb + TL::at(((lane >> 3) & 1) * 8 + (lane & 7), k + (lane >> 4)));
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t g[4];  // rows gr: even dims, rows gr + 8: odd dims
            const uint32_t lo = f[2 * h], hi = f[2 * h + 1];
            g[0] = e4m3_to_half2((uint16_t)__byte_perm(lo, 0, 0x0020));
            g[1] = e4m3_to_half2((uint16_t)__byte_perm(lo, 0, 0x0031));
            g[2] = e4m3_to_half2((uint16_t)__byte_perm(hi, 0, 0x0020));
            g[3] = e4m3_to_half2((uint16_t)__byte_perm(hi, 0, 0x0031));
#pragma unroll
            for (int t = 0; t < NT; ++t)
              mma16816<true>(oacc[t][k + h], g, __float_as_uint(s[t][0]), __float_as_uint(s[t][1]));
          }
        }
      }
    }
    __syncwarp();  // the stage before this one is free: every lane has read it
    if (loaded < n_units) {
      issue(ld, page, stage == 0 ? STAGES - 1 : stage - 1);
      ++loaded;
      next_unit(ld, c, items);
      if (loaded < n_units) page = page_of(ld);
    }
    cp_commit();
    stage = stage + 1 == STAGES ? 0 : stage + 1;

    const bool ends = cp.tile + 1 == cp.tiles;
    if (ends || i + 1 == n_units) {
      // ---- join the four warps --------------------------------------------------
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float v = l[t][j];
          v += __shfl_xor_sync(kFull, v, 4);
          v += __shfl_xor_sync(kFull, v, 8);
          v += __shfl_xor_sync(kFull, v, 16);
          l[t][j] = v;
          if (lane < 4) {
            mls[(warp * R + 8 * t + 2 * tg + j) * 2] = m[t][j];
            mls[(warp * R + 8 * t + 2 * tg + j) * 2 + 1] = v;
          }
        }
      __syncthreads();
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int n = 8 * t + 2 * tg + j;
          float top = -INFINITY;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) top = fmaxf(top, mls[(w * R + n) * 2]);
          const float f = top == -INFINITY ? 0.0f : ex2(m[t][j] - top);
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            oacc[t][k][j] *= f;
            oacc[t][k][2 + j] *= f;
          }
        }
      for (int w = 0; w < kWarps; ++w) {
        if (w == warp) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const int dim = 16 * k + (F8 ? 2 * gr + (j >> 1) : gr + 8 * (j >> 1));
                float* d = red + (8 * t + 2 * tg + (j & 1)) * RED + dim;
                *d = (w == 0 ? 0.0f : *d) + oacc[t][k][j];
              }
        }
        __syncthreads();
      }
      const int mt = cp.it % a.mts, kvh = cp.it / a.mts;
      const bool whole = t0 == 0 && ends;
      const int slot = t0 > 0 ? 0 : 1;  // 0: an item started before, 1: one that goes on after
      for (int e = threadIdx.x; e < R * (DH / 8); e += kThreads) {
        const int n = e / (DH / 8), d0 = 8 * (e % (DH / 8));
        if (mt * R + n >= a.G) continue;
        float top = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, mls[(w * R + n) * 2]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float mw = mls[(w * R + n) * 2];
          if (mw != -INFINITY) sum += mls[(w * R + n) * 2 + 1] * ex2(mw - top);
        }
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = red[n * RED + d0 + j];
        if (whole) {
          int head;
          const int row = query_row(a, cp.b, mt * R + n, kvh, &head);
          if (row < 0) continue;
          const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] *= inv;
          const int64_t at = (int64_t)row * a.q_heads + head;
          *reinterpret_cast<uint4*>(a.o + at * DH + d0) = pack8(v);
          if (a.lse && d0 == 0)
            a.lse[at] = sum == 0.0f ? -INFINITY : (log2f(sum) + top) * 0.6931471805599453f;
        } else {
          const int64_t at = ((int64_t)cta * 2 + slot) * R + n;
          float* po = a.part_o + at * DH + d0;
          *reinterpret_cast<float4*>(po) = make_float4(v[0], v[1], v[2], v[3]);
          *reinterpret_cast<float4*>(po + 4) = make_float4(v[4], v[5], v[6], v[7]);
          if (d0 == 0) {
            a.part_ml[at * 2] = top;
            a.part_ml[at * 2 + 1] = sum;
          }
        }
      }
      if (slot == 1 && !whole && threadIdx.x == 0) {
        // the CTA that holds the item's last unit: the one whose run contains it
        const long long last = u0 + i + (cp.tiles - 1 - cp.tile);
        a.desc[cta] = make_int4(cp.b, cp.it, (int)(((last + 1) * ctas - 1) / U), 0);
      }
      __syncthreads();
      fresh = true;
    }
    next_unit(cp, c, items);
  }
  cp_wait<0>();
}

// Joins the shares of the items that several CTAs hold: block c the item that CTA c
// started, from its second slot and the first slots of the CTAs after it, in order.
template <int DH>
__global__ void __launch_bounds__(256)
decode_join_kernel(const __grid_constant__ DecArgs a, int R) {
  const int cta = blockIdx.x;
  const int4 d = a.desc[cta];
  if (d.z < 0) return;
  const int mt = d.y % a.mts, kvh = d.y / a.mts;
  for (int e = threadIdx.x; e < R * (DH / 4); e += 256) {
    const int n = e / (DH / 4), d0 = 4 * (e % (DH / 4));
    int head;
    const int row = query_row(a, d.x, mt * R + n, kvh, &head);
    if (row < 0) continue;
    float top = -INFINITY;
    for (int j = cta; j <= d.z; ++j)
      top = fmaxf(top, a.part_ml[(((int64_t)j * 2 + (j == cta)) * R + n) * 2]);
    float sum = 0.0f;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (top != -INFINITY) {
      for (int j = cta; j <= d.z; ++j) {
        const int64_t at = ((int64_t)j * 2 + (j == cta)) * R + n;
        const float f = ex2(a.part_ml[at * 2] - top);
        sum += f * a.part_ml[at * 2 + 1];
        const float4 p = *reinterpret_cast<const float4*>(a.part_o + at * DH + d0);
        v.x += f * p.x; v.y += f * p.y; v.z += f * p.z; v.w += f * p.w;
      }
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const int64_t at = (int64_t)row * a.q_heads + head;
    uint2 out;
    out.x = pack_bf16(v.x * inv, v.y * inv);
    out.y = pack_bf16(v.z * inv, v.w * inv);
    *reinterpret_cast<uint2*>(a.o + at * DH + d0) = out;
    if (a.lse && d0 == 0) a.lse[at] = sum == 0.0f ? -INFINITY : (log2f(sum) + top) * 0.6931471805599453f;
  }
}

// Query tiles: 8 columns of the product for each 8 of the G rows, up to 32 in one pass
// over the keys.
int tiles_of(int G) { return G <= 8 ? 1 : G <= 16 ? 2 : 4; }
// CTAs: a fixed count, so that the split (and the workspace) is the same on any GPU;
// two on each of 148 SMs, one where 32 queries fill the registers.
int ctas_of(int NT) { return NT == 4 ? 148 : 296; }

template <int DH, int NT, bool F8>
cudaError_t run(const DecArgs& a, cudaStream_t s) {
  using TL = Tile<DH, F8>;
  constexpr int most = NT == 4 ? 49152 : 24576;  // ring bytes of a warp
  constexpr int STAGES = most / TL::kStage > 6 ? 6 : most / TL::kStage;
  static_assert(STAGES >= 3, "a ring needs three stages");
  constexpr int R = 8 * NT;
  constexpr size_t smem = (size_t)kWarps * STAGES * TL::kStage + (size_t)R * (DH + 4) * 4 +
                          (size_t)kWarps * R * 2 * 4;
  auto kern = decode_kernel<DH, NT, F8, STAGES>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int grid = ctas_of(NT);
  kern<<<grid, kThreads, smem, s>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  decode_join_kernel<DH><<<grid, 256, 0, s>>>(a, R);
  return cudaGetLastError();
}
template <int DH, bool F8>
cudaError_t run_nt(const DecArgs& a, cudaStream_t s) {
  switch (tiles_of(a.G)) {
    case 1: return run<DH, 1, F8>(a, s);
    case 2: return run<DH, 2, F8>(a, s);
    default: return run<DH, 4, F8>(a, s);
  }
}

}  // namespace

size_t decode_workspace_bytes(int G, int head_dim) {
  const int nt = tiles_of(G), R = 8 * nt;
  const size_t slots = (size_t)ctas_of(nt) * 2 * R;
  return slots * head_dim * 4 + slots * 2 * 4 + (size_t)ctas_of(nt) * sizeof(int4);
}

cudaError_t launch_decode(const void* q, int64_t ldq, const smoe_kv_cache& c, const int32_t* inv,
                          int kslots, int q_heads, void* o, float* lse, void* ws, unsigned* err,
                          cudaStream_t s) {
  DecArgs a;
  a.q = (const bf16*)q;
  a.ldq = ldq;
  a.inv = inv;
  a.c = c;
  a.kslots = kslots;
  a.q_heads = q_heads;
  a.group = q_heads / c.kv_heads;
  a.G = kslots * a.group;
  const int nt = tiles_of(a.G), R = 8 * nt;
  a.mts = cdiv(a.G, R);
  a.scale_log2 = (float)(1.4426950408889634 / sqrt((double)c.head_dim));
  a.o = (bf16*)o;
  a.lse = lse;
  const size_t slots = (size_t)ctas_of(nt) * 2 * R;
  a.part_o = (float*)ws;
  a.part_ml = a.part_o + slots * c.head_dim;
  a.desc = (int4*)(a.part_ml + slots * 2);
  a.err = err;
  if (c.k_scale)
    return c.head_dim == 64 ? run_nt<64, true>(a, s) : run_nt<128, true>(a, s);
  return c.head_dim == 64 ? run_nt<64, false>(a, s) : run_nt<128, false>(a, s);
}

}  // namespace smoe
