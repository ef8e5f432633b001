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
// Split: a sequence is cut into units of 16 H keys (H = 2 where a row is 128 bytes or
// less, which spreads a unit's own instructions over more keys; when chosen, e4m3, 128
// sequences of 8000 tokens: 123 us, with H = 1 160).  The sequences' units in a row, with
// kItemCost units' worth of time for a sequence's own start and end, are cut into ranges;
// a job is a range and an item (a key head and a tile of queries), and a warp's.
// Neighbouring warps have the items of one range, because the key heads' rows of a token
// lie next to one another in a page. No warp waits for another.
//
// Where a warp has 32 units and more, an eighth of the work goes in smaller ranges that a
// warp fetches from a counter when it has finished, because SMs do not get equal shares of
// the memory's rate: equal runs alone end up to 20% apart (when chosen, 64 sequences of up
// to 16384 tokens: 184 us, without fetched ranges 193, with a quarter 191).  So a ragged
// batch and a single long sequence load the GPU alike.  A sequence that lies in one range
// is finished there; the shares of the others go to the workspace and a second kernel
// joins them in the order of the ranges.  Ranges and the order of all sums follow from
// sizes and lengths alone: a batch gives the same bits every time.
//
// Time: 128 sequences of up to 4096 tokens, 537 MB, 83 us at the copy rate: 99 to 105 us, of
// which the units take 85 at 6.4 TB/s, the start up to the first keys 5 and the join 5
// (reads that wait for one another).  64 of up to 16384, 1107 MB, 171 us: 187 to 194.  48 of up
// to 8190 in e4m3, 105 MB, 16 us: 39.5; seven units a warp do not hide its start and end, and
// 32 keys take 1100 instructions, for half of the bytes that a bf16 cache loads beside 950.
// One sequence of 2048 tokens: 12 us, latency throughout.
//
// A warp copies its keys' rows with cp.async into its own ring in shared memory, units
// ahead and across items, and keeps a running maximum m, sum l and accumulator O (one
// pass over the data):
//   S^T = K Q^T      mma m16n8k16, keys as rows, 8 queries as columns
//   m' = max(m, S), P = exp(S - m'), l = l e^(m-m') + sum P, O^T = O^T e^(m-m') + V^T P^T
// Keys as rows cost ceil(G/8) 8-column products instead of a 16-row tile padded with
// empty queries; P^T turns from accumulator to operand layout by movmatrix.
//
// The second product takes P as two bf16 numbers, the rounded weight and what the rounding
// left, so that a weight keeps 16 bits (one alone would cost the output as much again as
// its own rounding; the second product's time is under 1%).  For an e4m3 cache P is the
// weight times the value's scale and the codes are turned into bf16, exactly: a product with
// fp16 would lose small weights beside the scale of another row, such as the 1 of a row of
// zeros, below 2^-24 (4096 tokens under a zero row 12 above them: 15% of the output).  Keys
// are multiplied in fp16, codes exact and queries scaled to [1, 2), where what falls below
// 2^-24 of the largest is within the fp32 sum's own rounding.
#include <cuda_fp16.h>

#include <atomic>

#include "tc_ptx.cuh"

namespace smoe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kHalf = 16;                    // keys of a product's tile
constexpr int kItemCost = 2;                 // an item's start and end, in units
constexpr int kLeast = 2;                    // units of a range, rather than more warps
constexpr int kFetch = 32;                   // units of a warp, from which on an eighth is fetched
constexpr int kSpread = kThreads;            // runs of sequences that the units are counted for
constexpr int kMostSlots = 128;              // slots of a token
constexpr int kDirectRows = 1024;            // rows that are looked for rather than listed first
constexpr int kFifo = 8;                     // ranges between a warp's loads and its products

struct DecArgs {
  const bf16* q;
  int64_t ldq;
  const int32_t* slots;  // sorted_slot, or null: row = slot
  const int32_t* inv;    // grouped row of each slot that a row names; null: rows are looked for
  int direct;            // no kernel runs before the decode kernel: nothing is fetched
  smoe_kv_cache c;
  int kslots, q_heads, group, G, mts;  // mts: query tiles of 8 NT rows
  unsigned long long page_mul;         // position / page_size = position * page_mul >> page_shift
  int page_shift;
  int one_page;                        // 16 divides page_size
  unsigned k_page, k_token, k_head, v_page, v_token, v_head;  // strides in 16-byte pieces
  float scale_log2;                    // log2(e) / sqrt(head_dim)
  bf16* o;
  float* lse;  // nullable
  // two shares for each job, of min(G, R) rows (R = 8 NT): of a sequence that an earlier
  // range started, and of one that goes on in the next
  int workers;         // warps
  float* part_o;       // [jobs][2][rows][DH]
  float* part_ml;      // [jobs][2][rows][2]
  int jobs;
  int4* split;         // [jobs] what the job starts and does not end: b, item, first and last range (-1)
  unsigned* fetched;   // jobs fetched
  unsigned* err;
};

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, uint32_t src_bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(src_bytes)
               : "memory");
}
// A whole piece of a row that is read once and should leave L2 first: what the warps hand
// to the joining kernel stays there.
__device__ __forceinline__ unsigned long long read_once() {
  unsigned long long policy;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  return policy;
}
__device__ __forceinline__ void cp_async16_once(uint32_t dst, const void* src, unsigned long long policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "l"(policy)
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
// Two e4m3 codes as bf16, which holds all of their values (NaN stays NaN).
__device__ __forceinline__ uint32_t e4m3_to_bf162(uint16_t v) {
  const uint32_t h = e4m3_to_half2(v);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack_bf16(f.x, f.y);
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

__device__ __forceinline__ void pdl_trigger() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Grouped row of each slot, no job fetched and none that starts a split item.  Entries of
// slots that no row names keep what they hold: a reader checks that the row it finds names
// the slot.
__global__ void __launch_bounds__(256)
decode_prepare_kernel(const int32_t* __restrict__ slots, int rows, int32_t* __restrict__ inv,
                      int4* __restrict__ split, int jobs, unsigned* __restrict__ fetched, unsigned* err) {
  pdl_trigger();
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i == 0) *fetched = 0;
  if (i < jobs) split[i] = make_int4(0, 0, 0, -1);
  if (slots == nullptr || i >= rows) return;
  const int p = slots[i];
  if (p >= 0 && p < rows) inv[p] = i;
  else report_error(err, ERRBIT_DATA);
}

template <int DH, bool F8>
struct Tile {
  static constexpr int kRow = F8 ? DH : 2 * DH;    // bytes of a cached row of a head
  static constexpr int H = kRow <= 128 ? 2 : 1;
  static constexpr int kUnit = kHalf * H;          // keys of a unit
  // Eight rows' chunks of one number lie in eight bank groups: rows 16 bytes further apart
  // than they are long, or (128 bytes, where room is short) chunk c of row r at c ^ (r & 7).
  static constexpr bool kSwizzle = kRow == 128;
  static constexpr int kPitch = kSwizzle ? kRow : kRow + 16;
  static constexpr int kRows = 2 * kUnit * kPitch;                 // K rows, then V rows
  static constexpr int kStage = kRows + (F8 ? 2 * kUnit * 4 : 0);  // and their scales
};

// A place in the row of units: unit `tile` of sequence b, for item it; `left` costs before
// the end of the range (none: the range has no further unit).
struct Cursor {
  int b, it, tile, tiles, len, left, range;
};

__device__ __forceinline__ int seq_len(const smoe_kv_cache& c, int b) {
  const long long cap = (long long)c.max_pages * c.page_size;
  const int n = c.seq_lens[b];
  return n < 0 ? 0 : (int)(n < cap ? n : cap);
}
template <int UNIT>
__device__ __forceinline__ int tiles_in(int len) { return (len + UNIT - 1) / UNIT; }

template <int UNIT>
__device__ __forceinline__ void next_unit(Cursor& p, const smoe_kv_cache& c) {
  --p.left;
  if (++p.tile < p.tiles) return;
  p.left -= kItemCost;
  p.tile = 0;
  do {
    if (++p.b >= c.B) { p.left = 0; return; }
    p.len = seq_len(c, p.b);
    p.tiles = tiles_in<UNIT>(p.len);
  } while (p.tiles == 0);
}
// Slot and query head of query qi of key head kvh of sequence b.
__device__ __forceinline__ int query_slot(const DecArgs& a, int b, int qi, int kvh, int* head) {
  *head = kvh * a.group + qi % a.group;
  return b * a.kslots + qi / a.group;
}
// Grouped row of a slot, for a whole warp; -1 for a slot that no row names (reported).
__device__ __forceinline__ int row_of(const DecArgs& a, int slot, int lane) {
  if (!a.slots) return slot;
  const int all = a.c.B * a.kslots;
  int row = -1;
  if (a.inv) {
    row = a.inv[slot];
    if (row < 0 || row >= all || a.slots[row] != slot) row = -1;
  } else {
#pragma unroll 16
    for (int i = lane; i < all; i += 32)
      if (a.slots[i] == slot) row = i;
    row = __reduce_max_sync(kFull, row);
  }
  if (row < 0 && lane == 0) report_error(a.err, ERRBIT_DATA);
  return row;
}

template <int DH, int NT, bool F8, int STAGES, int PER_SM>
__global__ void __launch_bounds__(kThreads, PER_SM)
decode_kernel(const __grid_constant__ DecArgs a) {
  using TL = Tile<DH, F8>;
  constexpr int R = 8 * NT, KS = DH / 16, H = TL::H, UNIT = TL::kUnit;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ unsigned masks[kWarps][STAGES];
  __shared__ int before[kSpread];  // costs before each run of sequences (all: below 2^31)
  __shared__ int wsum[kWarps];
  __shared__ Cursor fifo[kWarps][kFifo];
  __shared__ int16_t sequence_rows[kWarps][kMostSlots];  // of the slots of the sequence at hand (direct)

  const smoe_kv_cache& c = a.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int items = c.kv_heads * a.mts;
  const int cta = blockIdx.x;

  // ---- the row of units: costs of the runs of sequences --------------------------
  const int per = (c.B + kSpread - 1) / kSpread;
  int mine = 0;
  for (int i = 0; i < per; ++i) {
    const int b = threadIdx.x * per + i;
    if (b >= c.B) break;
    const int n = c.seq_lens[b];
    if (cta == 0 && (n < 0 || n > (long long)c.max_pages * c.page_size)) report_error(a.err, ERRBIT_DATA);
    const int t = tiles_in<UNIT>(seq_len(c, b));
    mine += t > 0 ? t + kItemCost : 0;
  }
  int incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int v = __shfl_up_sync(kFull, incl, off);
    if (lane >= off) incl += v;
  }
  if (lane == 31) wsum[warp] = incl;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) incl += wsum[w];
    total += wsum[w];
  }
  before[threadIdx.x] = incl - mine;
  __syncthreads();
  // costs of a range that is dealt out (nr of them, W jobs), and of one that is fetched
  const int W = a.workers, nr = max(1, W / items);
  const int share = total / nr;
  const bool fetch = share >= kFetch && !a.direct;
  const int dealt = fetch ? share - share / 8 : max(kLeast, share + 1);
  const int rest = total - nr * dealt;  // not above 0 without fetched ranges
  const int fetched = fetch ? cdiv(rest, nr) : 1;
  const int ranges = nr + (rest > 0 ? cdiv(rest, fetched) : 0);
  auto start_of = [&](int r) -> int { return r <= nr ? r * dealt : nr * dealt + (r - nr) * fetched; };
  auto range_of = [&](int x) -> int {
    const int y = x - nr * dealt;
    return y < 0 ? x / dealt : nr + y / fetched;
  };
  // The first unit of a job, for a whole warp.
  auto open_job = [&](unsigned job) -> Cursor {
    Cursor p{};
    p.range = job / items;
    p.it = job - p.range * items;
    if (p.range >= ranges) return p;
    const int x = start_of(p.range), end = min(total, start_of(p.range + 1));
    if (x >= end) return p;
    int n = 0;
#pragma unroll
    for (int i = 0; i < kSpread / 32; ++i) n += before[i * 32 + lane] <= x;
    const int t = (int)__reduce_add_sync(kFull, n) - 1;
    int rem = x - before[t];
    for (p.b = t * per;; ++p.b) {
      p.len = seq_len(c, p.b);
      p.tiles = tiles_in<UNIT>(p.len);
      const int cost = p.tiles > 0 ? p.tiles + kItemCost : 0;
      if (rem < cost) break;
      rem -= cost;
    }
    p.tile = max(0, rem - kItemCost);
    p.left = end - x - max(0, kItemCost - rem);
    return p;
  };
  const unsigned jobs = (unsigned)ranges * items;
  if (a.direct && lane == 0 && cta * kWarps + warp < a.jobs) a.split[cta * kWarps + warp] = make_int4(0, 0, 0, -1);
  Cursor cp = open_job(cta * kWarps + warp);
  Cursor ld = cp;

  // ---- loads: 16-byte chunk `sub` of rows rr, rr + RPI, ... of the unit ---------------
  constexpr int CH = TL::kRow / 16, RPI = 32 / CH;
  const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * STAGES) * TL::kStage;
  const int sub = lane % CH, rr = lane / CH;
  constexpr bool SWZ = TL::kSwizzle;
  const unsigned long long once = read_once();
  static_assert(!SWZ || RPI == 4, "rows 4 i + rr");
  const uint32_t dst0 = ring + rr * TL::kPitch + (SWZ ? sub ^ rr : sub) * 16;
  // row i * RPI + rr of a stage's part that starts at `part`
  auto row_at = [&](uint32_t part, int i) -> uint32_t {
    return (SWZ && (i & 1) ? part ^ 64 : part) + i * RPI * TL::kPitch;
  };
  auto page_index = [&](int pos) { return (int)(((unsigned long long)(unsigned)pos * a.page_mul) >> a.page_shift); };
  auto at16 = [](const void* base, unsigned long long pieces) { return (const char*)base + (pieces << 4); };
  // Page of a key, -1: none.  Where 16 divides the page size 16 keys share a page: lane 16 h
  // holds the h-th sixteen's; else lane r holds key r's (and lane 16 + r too when H = 1).
  auto page_of = [&](const Cursor& p) -> int {
    const int pos = p.tile * UNIT + (a.one_page ? (lane >> 4) * (H - 1) * kHalf : lane % UNIT);
    if (pos >= p.len) return -1;
    const int id = c.block_table[(int64_t)p.b * c.table_stride + page_index(pos)];
    if (id < 0 || id >= c.num_pages) {
      report_error(a.err, ERRBIT_DATA);
      return -1;
    }
    return id;
  };
  auto issue = [&](const Cursor& p, int page, int stage) {
    const uint32_t dst = dst0 + stage * TL::kStage;
    const uint32_t sdst = ring + stage * TL::kStage + TL::kRows + lane * 4;
    const int pos0 = p.tile * UNIT;
    const unsigned kvh = a.mts == 1 ? p.it : p.it / a.mts;
    if (a.one_page) {
      unsigned mask = 0;
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const int id = H == 1 ? page : __shfl_sync(kFull, page, h * 16);
        const int first = pos0 + h * kHalf;
        const int live = id < 0 ? 0 : min(kHalf, p.len - first);
        mask |= ((1u << live) - 1) << (h * kHalf);
        const unsigned pg = max(id, 0), off = live > 0 ? first - page_index(first) * c.page_size : 0;
        // rows behind the last key: a place of the page itself, never read
        const unsigned r0 = off + min(rr, max(live - 1, 0));
        const char* ks = at16(c.k, (unsigned long long)pg * a.k_page + ((unsigned long long)r0 * a.k_token + (kvh * (unsigned long long)a.k_head + sub)));
        const char* vs = at16(c.v, (unsigned long long)pg * a.v_page + ((unsigned long long)r0 * a.v_token + (kvh * (unsigned long long)a.v_head + sub)));
        const uint32_t d = dst + h * kHalf * TL::kPitch;
        if (live == kHalf) {
#pragma unroll
          for (int i = 0; i < kHalf / RPI; ++i)
            cp_async16_once(row_at(d, i), at16(ks, (unsigned long long)a.k_token * (i * RPI)), once);
#pragma unroll
          for (int i = 0; i < kHalf / RPI; ++i)
            cp_async16_once(row_at(d + UNIT * TL::kPitch, i), at16(vs, (unsigned long long)a.v_token * (i * RPI)), once);
        } else {
#pragma unroll
          for (int i = 0; i < kHalf / RPI; ++i) {
            const bool on = i * RPI + rr < live;
            cp_async16(row_at(d, i), on ? at16(ks, (unsigned long long)a.k_token * (i * RPI)) : ks, on ? 16u : 0u);
            cp_async16(row_at(d + UNIT * TL::kPitch, i), on ? at16(vs, (unsigned long long)a.v_token * (i * RPI)) : vs, on ? 16u : 0u);
          }
        }
        if (F8) {
          const int key = lane % kHalf;
          const bool on = key < live;
          const int64_t at = ((int64_t)pg * c.page_size + off + (on ? key : 0)) * c.kv_heads + kvh;
          // lanes 0-15: the keys' scales, lanes 16-31 the values'
          cp_async4(ring + stage * TL::kStage + TL::kRows + ((lane >> 4) * UNIT + h * kHalf + key) * 4,
                    (lane < 16 ? c.k_scale : c.v_scale) + at, on ? 4u : 0u);
        }
      }
      if (lane == 0) masks[warp][stage] = mask;
    } else {
      const bool ok = page >= 0;
      const unsigned mask = __ballot_sync(kFull, ok) & (UNIT == 32 ? kFull : 0xffffu);
      if (lane == 0) masks[warp][stage] = mask;
      const int pos = pos0 + lane % UNIT;
      const unsigned pg = ok ? page : 0, off = ok ? pos - page_index(pos) * c.page_size : 0;
      const unsigned long long ks = (unsigned long long)pg * a.k_page + (unsigned long long)off * a.k_token + (unsigned long long)kvh * a.k_head;
      const unsigned long long vs = (unsigned long long)pg * a.v_page + (unsigned long long)off * a.v_token + (unsigned long long)kvh * a.v_head;
      if (F8) {
        const int64_t at = ((int64_t)pg * c.page_size + off) * c.kv_heads + kvh;
        cp_async4(sdst, c.k_scale + at, ok ? 4u : 0u);
        cp_async4(sdst + UNIT * 4, c.v_scale + at, ok ? 4u : 0u);
      }
#pragma unroll
      for (int i = 0; i < UNIT / RPI; ++i) {
        const int r = i * RPI + rr;
        const unsigned bytes = (mask >> r) & 1u ? 16u : 0u;
        cp_async16(row_at(dst, i), at16(c.k, __shfl_sync(kFull, ks, r) + sub), bytes);
        cp_async16(row_at(dst + UNIT * TL::kPitch, i), at16(c.v, __shfl_sync(kFull, vs, r) + sub), bytes);
      }
    }
  };

  uint32_t qf[NT][KS][2];
  float qs[NT][2];  // factor of this thread's two query columns
  float m[NT][2], l[NT][2];
  float oacc[NT][KS][4];
  const int tg = lane & 3, gr = lane >> 2;
  bool fresh = true, waited = false, more = jobs > (unsigned)W;
  int stage = 0, into = 0, inflight = 0, t0 = 0;
  unsigned opened = 0, closed = 0;  // ranges put into and taken out of the fifo
  int page = ld.left > 0 ? page_of(ld) : -1;

  for (;;) {
    while (inflight < STAGES) {
      if (ld.left <= 0) {
        if (!more || !waited || opened - closed == kFifo) break;
        unsigned r = 0;
        if (lane == 0) r = atomicAdd(a.fetched, 1u);
        r = __shfl_sync(kFull, r, 0) + W;
        more = r < jobs;
        if (!more) break;
        ld = open_job(r);
        if (ld.left <= 0) continue;
        __syncwarp();  // every lane has read what the place held before
        if (lane == 0) fifo[warp][opened % kFifo] = ld;
        ++opened;
        page = page_of(ld);
      }
      issue(ld, page, into);
      cp_commit();
      ++inflight;
      into = into + 1 == STAGES ? 0 : into + 1;
      next_unit<UNIT>(ld, c);
      if (ld.left > 0) page = page_of(ld);
    }
    if (!waited) {  // from here on: the rows of the slots, and the count
      pdl_wait();
      waited = true;
      if (cp.left <= 0 && more) continue;
    }
    if (cp.left <= 0) {
      if (opened == closed) break;
      __syncwarp();
      cp = fifo[warp][closed++ % kFifo];
      fresh = true;
    }
    if (fresh) {  // first unit of an item here
      fresh = false;
      t0 = cp.tile;
      const int mt = cp.it % a.mts, kvh = cp.it / a.mts;
      if (a.slots && !a.inv) {
        __syncwarp();  // every lane has written the item before: it read its rows here
        for (int i = lane; i < a.kslots; i += 32) sequence_rows[warp][i] = -1;
        __syncwarp();
        const int all = c.B * a.kslots;
#pragma unroll 16
        for (int i = lane; i < all; i += 32) {
          const int of = a.slots[i] - cp.b * a.kslots;
          if (of >= 0 && of < a.kslots) sequence_rows[warp][of] = (int16_t)i;
        }
        __syncwarp();
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        int head = 0, row = -1;
        if (mt * R + 8 * t + gr < a.G) {
          row = query_slot(a, cp.b, mt * R + 8 * t + gr, kvh, &head);
          if (a.slots) row = a.inv ? a.inv[row] : sequence_rows[warp][row - cp.b * a.kslots];
          if (row >= c.B * a.kslots) row = -1;
        }
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
          ex = max(-100, min(126, ex));
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

    if (inflight == STAGES) {
      cp_wait<STAGES - 1>();
    } else if (STAGES > 2 && inflight == STAGES - 1) {
      cp_wait<STAGES - 2>();
    } else {
      cp_wait<0>();
    }
    __syncwarp();  // every lane's copies and the mask are seen by all
    const unsigned mask = masks[warp][stage];
    const uint32_t base = ring + stage * TL::kStage;
    if (mask) {
      float s[H][NT][4];
#pragma unroll
      for (int h = 0; h < H; ++h)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[h][t][j] = 0.0f;
      float ks[H][2], vs[H][2];
      const uint32_t kb = base + (lane & 15) * TL::kPitch + ((lane >> 4) ^ (SWZ ? lane & 7 : 0)) * 16;
      auto chunk = [](uint32_t at, int c) -> uint32_t { return SWZ ? at ^ (16 * c) : at + 16 * c; };  // c even
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const uint32_t kh = kb + h * kHalf * TL::kPitch;
        if (!F8) {
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            uint32_t f[4];
            ldsm4(f, chunk(kh, 2 * k));
#pragma unroll
            for (int t = 0; t < NT; ++t) mma16816<false>(s[h][t], f, qf[t][k][0], qf[t][k][1]);
          }
        } else {
#pragma unroll
          for (int k = 0; k < KS; k += 2) {  // 32 dims: two 16-byte chunks
            uint32_t f[4];
            ldsm4(f, chunk(kh, k));
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint32_t g[4];
              g[0] = e4m3_to_half2((uint16_t)f[2 * e]);
              g[1] = e4m3_to_half2((uint16_t)f[2 * e + 1]);
              g[2] = e4m3_to_half2((uint16_t)(f[2 * e] >> 16));
              g[3] = e4m3_to_half2((uint16_t)(f[2 * e + 1] >> 16));
#pragma unroll
              for (int t = 0; t < NT; ++t) mma16816<true>(s[h][t], g, qf[t][k + e][0], qf[t][k + e][1]);
            }
          }
          const float* sc = reinterpret_cast<const float*>(smem + (size_t)(warp * STAGES + stage) * TL::kStage + TL::kRows) + h * kHalf;
          ks[h][0] = sc[gr]; ks[h][1] = sc[gr + 8];
          vs[h][0] = sc[UNIT + gr]; vs[h][1] = sc[UNIT + gr + 8];
        }
      }
      if (mask != (UNIT == 32 ? kFull : 0xffffu)) {
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const bool on = (mask >> (h * kHalf + 8 * e + gr)) & 1u;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              if (!on) s[h][t][2 * e] = s[h][t][2 * e + 1] = -INFINITY;
            }
            if (F8 && !on) ks[h][e] = 1.0f;  // a scale that was not copied is 0
          }
      }
      // The reference m of a query's weights: its largest score.
      float top[NT][2];
      bool grows = false;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 2; ++j) top[t][j] = -INFINITY;
#pragma unroll
      for (int h = 0; h < H; ++h)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float& v = s[h][t][2 * e + j];
              if (F8) v *= qs[t][j] * ks[h][e];
              top[t][j] = fmaxf(top[t][j], v);
            }
#pragma unroll
      for (int off = 4; off <= 16; off <<= 1)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int j = 0; j < 2; ++j) top[t][j] = fmaxf(top[t][j], __shfl_xor_sync(kFull, top[t][j], off));
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (!F8) top[t][j] *= qs[t][j];
          grows |= top[t][j] > m[t][j];
        }
      if (__any_sync(kFull, grows)) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float mn = fmaxf(top[t][j], m[t][j]);
            const float al = m[t][j] == -INFINITY ? 0.0f : ex2(m[t][j] - mn);
            m[t][j] = mn;
            l[t][j] *= al;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              oacc[t][k][j] *= al;
              oacc[t][k][2 + j] *= al;
            }
          }
      }
      float ref[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 2; ++j) ref[t][j] = m[t][j] == -INFINITY ? 0.0f : m[t][j];
      const uint32_t vb = base + UNIT * TL::kPitch;
#pragma unroll
      for (int h = 0; h < H; ++h) {
        uint32_t pf[NT][2], pr[NT][2];  // pr: what the rounding of pf left
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float* w = s[h][t];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            w[j] = ex2(F8 ? w[j] - ref[t][j] : fmaf(w[j], qs[t][j], -ref[t][j]));
            w[2 + j] = ex2(F8 ? w[2 + j] - ref[t][j] : fmaf(w[2 + j], qs[t][j], -ref[t][j]));
            l[t][j] += w[j] + w[2 + j];
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float x = F8 ? w[2 * e] * vs[h][e] : w[2 * e], y = F8 ? w[2 * e + 1] * vs[h][e] : w[2 * e + 1];
            const uint32_t hi = pack_bf16(x, y);
            pr[t][e] = transpose8(pack_bf16(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xffff0000u)));
            pf[t][e] = transpose8(hi);
          }
        }
        const uint32_t vh = vb + h * kHalf * TL::kPitch;
        if (!F8) {
          const uint32_t va = vh + ((lane >> 4) * 8 + (lane & 7)) * TL::kPitch +
                              (((lane >> 3) & 1) ^ (SWZ ? lane & 7 : 0)) * 16;
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            uint32_t f[4];
            ldsm4_t(f, chunk(va, 2 * k));
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              mma16816<false>(oacc[t][k], f, pf[t][0], pf[t][1]);
              mma16816<false>(oacc[t][k], f, pr[t][0], pr[t][1]);
            }
          }
        } else {
          const uint32_t va = vh + (lane & 15) * TL::kPitch + ((lane >> 4) ^ (SWZ ? lane & 7 : 0)) * 16;
#pragma unroll
          for (int k = 0; k < KS; k += 2) {
            // transposed pairs of bytes: keys 2 tg, 2 tg + 1 of dims 2 gr, 2 gr + 1
            uint32_t f[4];
            ldsm4_t(f, chunk(va, k));
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint32_t g[4];  // rows gr: even dims, rows gr + 8: odd dims
              const uint32_t e0 = __byte_perm(f[2 * e], 0, 0x3120), e1 = __byte_perm(f[2 * e + 1], 0, 0x3120);
              g[0] = e4m3_to_bf162((uint16_t)e0);
              g[1] = e4m3_to_bf162((uint16_t)(e0 >> 16));
              g[2] = e4m3_to_bf162((uint16_t)e1);
              g[3] = e4m3_to_bf162((uint16_t)(e1 >> 16));
#pragma unroll
              for (int t = 0; t < NT; ++t) {
                mma16816<false>(oacc[t][k + e], g, pf[t][0], pf[t][1]);
                mma16816<false>(oacc[t][k + e], g, pr[t][0], pr[t][1]);
              }
            }
          }
        }
      }
    }
    __syncwarp();  // the stage is free: every lane has read it
    --inflight;
    stage = stage + 1 == STAGES ? 0 : stage + 1;

    const bool ends = cp.tile + 1 == cp.tiles;
    if (ends || cp.left <= 1) {
      // ---- the item ends, or its part in this range ----------------------------------
      const int mt = cp.it % a.mts, kvh = cp.it / a.mts;
      const bool whole = ends && t0 == 0;
      const int pitch = min(R, a.G), slot = t0 > 0 ? 0 : 1;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int n = 8 * t + 2 * tg + j;
          float v = l[t][j];
          v += __shfl_xor_sync(kFull, v, 4);
          v += __shfl_xor_sync(kFull, v, 8);
          v += __shfl_xor_sync(kFull, v, 16);
          if (mt * R + n >= a.G) continue;
          if (whole) {
            int head;
            const int sl = query_slot(a, cp.b, mt * R + n, kvh, &head);
            int row = sl;
            if (a.slots) {
              row = a.inv ? a.inv[sl] : sequence_rows[warp][sl - cp.b * a.kslots];
              if (row < 0 || row >= c.B * a.kslots || (a.inv && a.slots[row] != sl)) {
                report_error(a.err, ERRBIT_DATA);
                continue;
              }
            }
            const int place = row * a.q_heads + head;
            const float inv = v == 0.0f ? 0.0f : 1.0f / v;
            bf16* o = a.o + (int64_t)place * DH;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              const float e0 = oacc[t][k][j] * inv, e1 = oacc[t][k][2 + j] * inv;
              if (F8) {
                *reinterpret_cast<uint32_t*>(o + 16 * k + 2 * gr) = pack_bf16(e0, e1);
              } else {
                o[16 * k + gr] = __float2bfloat16_rn(e0);
                o[16 * k + gr + 8] = __float2bfloat16_rn(e1);
              }
            }
            if (a.lse && gr == 0)
              a.lse[place] = v == 0.0f ? -INFINITY : (log2f(v) + m[t][j]) * 0.6931471805599453f;
          } else {
            const int64_t at = (((int64_t)cp.range * items + cp.it) * 2 + slot) * pitch + n;
            float* po = a.part_o + at * DH;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              if (F8) {
                *reinterpret_cast<float2*>(po + 16 * k + 2 * gr) = make_float2(oacc[t][k][j], oacc[t][k][2 + j]);
              } else {
                po[16 * k + gr] = oacc[t][k][j];
                po[16 * k + gr + 8] = oacc[t][k][2 + j];
              }
            }
            if (gr == 0) *reinterpret_cast<float2*>(a.part_ml + at * 2) = make_float2(m[t][j], v);
          }
        }
      if (slot == 1 && !whole && lane == 0) {
        const int here = min(total, start_of(cp.range + 1)) - cp.left;
        a.split[cp.range * items + cp.it] =
            make_int4(cp.b, cp.it, cp.range, range_of(here + cp.tiles - 1 - cp.tile));
      }
      fresh = true;
    }
    next_unit<UNIT>(cp, c);
  }
  // sequences without a cached token: o = 0, lse = -inf
  for (int b = cta; b < c.B; b += gridDim.x) {
    if (seq_len(c, b) > 0) continue;
    for (int j = warp; j < a.kslots; j += kWarps) {
      const int row = row_of(a, b * a.kslots + j, lane);
      if (row < 0) continue;
      for (int i = lane; i < a.q_heads * (DH / 8); i += 32)
        *reinterpret_cast<uint4*>(a.o + (int64_t)row * a.q_heads * DH + 8 * i) = make_uint4(0, 0, 0, 0);
      if (a.lse)
        for (int i = lane; i < a.q_heads; i += 32) a.lse[(int64_t)row * a.q_heads + i] = -INFINITY;
    }
  }
  pdl_trigger();
  cp_wait<0>();
}

// Joins the shares of the items that several ranges hold, row by row (of 8 NT a query
// tile): the share of the range that started the item, then those of the ranges after it.
// A warp takes a row with up to kFew shares, else the CTA's warps take every kJoinWarps-th
// share each and their sums are joined in order.  A share without a score above -inf has the
// sum 0 or, where a query or all of its keys are NaN, NaN: it is added like the others, with
// the factor 0, so that NaN stays.
constexpr int kJoinWarps = 8, kFew = 48;

template <int DH>
struct Joined {
  float top, sum, v[DH / 32];  // value 32 k + lane
};
template <int DH>
__device__ __forceinline__ Joined<DH> join_shares(const DecArgs& a, int it, int first, int last, int n, int pitch,
                                                  int from, int step, int lane) {
  constexpr int N = DH / 32, kAhead = 8;
  const int items = a.c.kv_heads * a.mts;
  Joined<DH> r;
  r.top = -INFINITY;
  r.sum = 0.0f;
#pragma unroll
  for (int k = 0; k < N; ++k) r.v[k] = 0.0f;
  for (int j0 = first + from; j0 <= last; j0 += step * kAhead) {
    float2 s[kAhead];
    float p[kAhead][N];
#pragma unroll
    for (int h = 0; h < kAhead; ++h) {
      const int j = j0 + h * step;
      s[h] = make_float2(-INFINITY, 0.0f);
#pragma unroll
      for (int k = 0; k < N; ++k) p[h][k] = 0.0f;
      if (j <= last) {
        const int64_t at = (((int64_t)j * items + it) * 2 + (j == first)) * pitch + n;
        s[h] = *reinterpret_cast<const float2*>(a.part_ml + at * 2);
#pragma unroll
        for (int k = 0; k < N; ++k) p[h][k] = a.part_o[at * DH + 32 * k + lane];
      }
    }
    const float before = r.top;
#pragma unroll
    for (int h = 0; h < kAhead; ++h) r.top = fmaxf(r.top, s[h].x);
    const float up = r.top == -INFINITY ? 0.0f : r.top, al = ex2(before - up);
    r.sum *= al;
#pragma unroll
    for (int k = 0; k < N; ++k) r.v[k] *= al;
#pragma unroll
    for (int h = 0; h < kAhead; ++h) {
      const float f = ex2(s[h].x - up);
      r.sum += f * s[h].y;
#pragma unroll
      for (int k = 0; k < N; ++k) r.v[k] += f * p[h][k];
    }
  }
  return r;
}

template <int DH>
__global__ void __launch_bounds__(32 * kJoinWarps)
decode_join_kernel(const __grid_constant__ DecArgs a, int R) {
  constexpr int N = DH / 32, kListed = 256;
  __shared__ float2 ml[kJoinWarps];
  __shared__ float sums[kJoinWarps][DH];
  __shared__ int listed[kListed], n_listed;  // this CTA's rows of many shares
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int pitch = min(R, a.G);
  if (threadIdx.x == 0) n_listed = 0;
  __syncthreads();
  pdl_wait();
  // place of row n of a split item, -1: none
  auto place_of = [&](const int4& d, int n) -> int {
    int head;
    const int slot = query_slot(a, d.x, d.y % a.mts * R + n, d.y / a.mts, &head);
    const int row = row_of(a, slot, lane);
    return row < 0 ? -1 : row * a.q_heads + head;
  };
  // a lane looks at every 32nd of its warp's rows, the warp joins what they find
  const int all = a.jobs * pitch, step = kJoinWarps * gridDim.x, u0 = warp * gridDim.x + blockIdx.x;
  for (int base = u0; base < all; base += 32 * step) {
    int4 e = make_int4(0, 0, 0, -1);
    const int at = base + lane * step;
    if (at < all) e = a.split[at / pitch];
    unsigned todo = __ballot_sync(kFull, e.w >= 0 && e.y % a.mts * R + at % pitch < a.G);
    for (; todo; todo &= todo - 1) {
      const int from = __ffs(todo) - 1, u = base + from * step, n = u % pitch;
      const int4 d = make_int4(__shfl_sync(kFull, e.x, from), __shfl_sync(kFull, e.y, from),
                               __shfl_sync(kFull, e.z, from), __shfl_sync(kFull, e.w, from));
      if (d.w - d.z >= kFew) {
        int slot = 0;
        if (lane == 0) slot = atomicAdd(&n_listed, 1);
        slot = __shfl_sync(kFull, slot, 0);
        if (slot < kListed) {
          if (lane == 0) listed[slot] = u;
          continue;
        }
      }
      const int place = place_of(d, n);
      const Joined<DH> r = join_shares<DH>(a, d.y, d.z, d.w, n, pitch, 0, 1, lane);
      if (place < 0) continue;
      const float inv = r.sum == 0.0f ? 0.0f : 1.0f / r.sum;
#pragma unroll
      for (int k = 0; k < N; ++k) a.o[(int64_t)place * DH + 32 * k + lane] = __float2bfloat16_rn(r.v[k] * inv);
      if (a.lse && lane == 0)
        a.lse[place] = r.sum == 0.0f ? -INFINITY : (log2f(r.sum) + r.top) * 0.6931471805599453f;
    }
  }
  __syncthreads();
  const int many = min(n_listed, kListed);
  for (int i = 0; i < many; ++i) {
    const int u = listed[i], n = u % pitch;
    const int4 d = a.split[u / pitch];
    const Joined<DH> r = join_shares<DH>(a, d.y, d.z, d.w, n, pitch, warp, kJoinWarps, lane);
    if (lane == 0) ml[warp] = make_float2(r.top, r.sum);
#pragma unroll
    for (int k = 0; k < N; ++k) sums[warp][32 * k + lane] = r.v[k];
    __syncthreads();
    if (threadIdx.x < DH) {
      float top = -INFINITY, sum = 0.0f, v = 0.0f;
#pragma unroll
      for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, ml[w].x);
      const float up = top == -INFINITY ? 0.0f : top;
#pragma unroll
      for (int w = 0; w < kJoinWarps; ++w) {
        const float f = ex2(ml[w].x - up);
        sum += f * ml[w].y;
        v += f * sums[w][threadIdx.x];
      }
      const int place = place_of(d, n);
      if (place >= 0) {
        a.o[(int64_t)place * DH + threadIdx.x] = __float2bfloat16_rn(sum == 0.0f ? 0.0f : v / sum);
        if (a.lse && threadIdx.x == 0)
          a.lse[place] = sum == 0.0f ? -INFINITY : (log2f(sum) + top) * 0.6931471805599453f;
      }
    }
    __syncthreads();
  }
}

// 8-column products of a query tile: the G rows of a key head in as few tiles as have up to
// three each, of one size.  Four spill (32 queries: 69 us, as two tiles of two 63), fewer
// read the keys more often (24 queries: one of three 51 us, two of two 61, three of one 66).
int tiles_of(int G) {
  const int columns = cdiv(G, 8);
  return cdiv(columns, cdiv(columns, 3));
}
// CTAs on each of 148 SMs: three where the registers allow it (8 queries), else two.
int workers_of(int nt) { return 148 * kWarps * (nt == 1 ? 3 : 2); }

// early: starts while the kernel before it still runs, and waits for it on the device.
template <typename... P, typename... A>
cudaError_t launch(bool early, void (*kern)(P...), int grid, int threads, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = early;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Three on each of 148 SMs, or one row for each warp.
int join_blocks(const DecArgs& a, int R) {
  const long long rows = (long long)a.jobs * (a.G < R ? a.G : R), n = (rows + kJoinWarps - 1) / kJoinWarps;
  return (int)(n < 444 ? n : 444);
}

template <int DH, int NT, bool F8>
cudaError_t run(const DecArgs& a, cudaStream_t s) {
  using TL = Tile<DH, F8>;
  constexpr int PER_SM = NT == 1 ? 3 : 2;
  constexpr int kRing = (228 * 1024 / PER_SM - 3584) / (kWarps * TL::kStage);
  constexpr int STAGES = kRing > 4 ? 4 : kRing;
  static_assert(STAGES >= 2, "a ring needs two stages");
  constexpr size_t smem = (size_t)kWarps * STAGES * TL::kStage;
  auto kern = decode_kernel<DH, NT, F8, STAGES, PER_SM>;
  // the attribute belongs to the kernel on a device and stays: set once for each
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (e == cudaSuccess && !(done.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  }
  if (e == cudaSuccess) e = launch(!a.direct, kern, a.direct ? cdiv(a.jobs, kWarps) : 148 * PER_SM, kThreads, smem, s, a);
  if (e == cudaSuccess) e = launch(true, decode_join_kernel<DH>, join_blocks(a, 8 * NT), 32 * kJoinWarps, 0, s, a, 8 * NT);
  return e;
}
template <int DH, bool F8>
cudaError_t run_nt(const DecArgs& a, cudaStream_t s) {
  switch (tiles_of(a.G)) {
    case 1: return run<DH, 1, F8>(a, s);
    case 2: return run<DH, 2, F8>(a, s);
    default: return run<DH, 3, F8>(a, s);
  }
}

struct DecWorkspace {
  int workers, jobs;
  size_t part_o, part_ml, split, fetched, inv, bytes;
  DecWorkspace(int rows, int kv_heads, int G, int head_dim) {
    const int nt = tiles_of(G), items = kv_heads * cdiv(G, 8 * nt);
    workers = workers_of(nt);
    jobs = 2 * (workers > items ? workers : items);
    const size_t share_rows = (size_t)jobs * 2 * (G < 8 * nt ? G : 8 * nt);
    part_o = 0;
    part_ml = part_o + share_rows * head_dim * 4;
    split = (part_ml + share_rows * 2 * 4 + 15) / 16 * 16;
    fetched = split + (size_t)jobs * sizeof(int4);
    inv = fetched + 16;
    bytes = inv + (size_t)rows * 4;
  }
};

// Units, with the items' costs, of one item of every sequence that the tables can hold.
long long most_units(const smoe_kv_cache& c) {
  return (long long)c.B * (cdiv(c.max_pages * c.page_size, kHalf) + kItemCost);
}
// Without a kernel before it where no batch that the tables can hold has work to fetch, and
// its rows are few enough to be looked for (one sequence of 2048 tokens: 8.7 us of the host's
// time, with that kernel 11.8; on the device the same, where it runs beside the next one).
bool direct(const smoe_kv_cache& c, int workers, int items, int rows, bool slots) {
  const int nr = workers / items;
  return nr >= 1 && most_units(c) / nr < kFetch && (!slots || rows <= kDirectRows);
}
int items_of(const smoe_kv_cache& c, int G) { return c.kv_heads * cdiv(G, 8 * tiles_of(G)); }

}  // namespace

int decode_kernels(const smoe_kv_cache& c, int kslots, int q_heads, bool slots) {
  const int G = kslots * (q_heads / c.kv_heads);
  return direct(c, workers_of(tiles_of(G)), items_of(c, G), c.B * kslots, slots) ? 2 : 3;
}

size_t decode_workspace_bytes(int rows, int kv_heads, int G, int head_dim) {
  return DecWorkspace(rows, kv_heads, G, head_dim).bytes;
}

cudaError_t launch_decode(const void* q, int64_t ldq, const smoe_kv_cache& c, const int32_t* sorted_slot,
                          int kslots, int q_heads, void* o, float* lse, void* ws, unsigned* err,
                          cudaStream_t s) {
  DecArgs a;
  a.q = (const bf16*)q;
  a.ldq = ldq;
  a.slots = sorted_slot;
  a.c = c;
  a.kslots = kslots;
  a.q_heads = q_heads;
  a.group = q_heads / c.kv_heads;
  a.G = kslots * a.group;
  const int rows = c.B * kslots;
  a.mts = cdiv(a.G, 8 * tiles_of(a.G));
  // exact for positions below 2^31: 2^(31 + n) / page_size rounded up, 2^n >= page_size
  int n = 0;
  while ((1ll << n) < c.page_size) ++n;
  a.page_shift = 31 + n;
  a.page_mul = ((1ull << a.page_shift) + c.page_size - 1) / c.page_size;
  a.one_page = c.page_size % kHalf == 0;
  const int es = c.k_scale ? 1 : 2;
  a.k_page = (unsigned)(c.k_page_stride * es / 16);
  a.k_token = (unsigned)(c.k_token_stride * es / 16);
  a.k_head = (unsigned)(c.k_head_stride * es / 16);
  a.v_page = (unsigned)(c.v_page_stride * es / 16);
  a.v_token = (unsigned)(c.v_token_stride * es / 16);
  a.v_head = (unsigned)(c.v_head_stride * es / 16);
  a.scale_log2 = (float)(1.4426950408889634 / sqrt((double)c.head_dim));
  a.o = (bf16*)o;
  a.lse = lse;
  const DecWorkspace w(rows, c.kv_heads, a.G, c.head_dim);
  char* base = (char*)ws;
  a.part_o = (float*)(base + w.part_o);
  a.part_ml = (float*)(base + w.part_ml);
  a.workers = w.workers;
  a.split = (int4*)(base + w.split);
  a.fetched = (unsigned*)(base + w.fetched);
  a.inv = (int32_t*)(base + w.inv);
  a.err = err;
  const int items = items_of(c, a.G);
  a.direct = direct(c, a.workers, items, rows, sorted_slot != nullptr);
  a.jobs = w.jobs;
  if (a.direct) {  // no more jobs, and blocks for them, than can have a unit
    const long long ranges = most_units(c) / kLeast + 1, nr = a.workers / items;
    a.jobs = (int)(ranges < nr ? ranges : nr) * items;
  }
  if (a.direct) {
    a.inv = nullptr;
  } else {
    const int n = sorted_slot && rows > w.jobs ? rows : w.jobs;
    decode_prepare_kernel<<<cdiv(n, 256), 256, 0, s>>>(sorted_slot, rows, (int32_t*)a.inv, a.split, w.jobs,
                                                       a.fetched, err);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (c.k_scale)
    return c.head_dim == 64 ? run_nt<64, true>(a, s) : run_nt<128, true>(a, s);
  return c.head_dim == 64 ? run_nt<64, false>(a, s) : run_nt<128, false>(a, s);
}

}  // namespace smoe
