// Paged cache: causal attention of runs of new tokens, over the pages or over
// rows of their own (prompts).
#pragma once

#include <cuda.h>

#include "kvq_paged_rows.cuh"
#include "kvq_tc.cuh"

namespace kvq {
namespace chunk {

using rows::add2;
using rows::f2;
using rows::f2_get;
using rows::f2_of;
using rows::fma2;

constexpr int kTokens = 128;  // tokens of a key or value tile
constexpr int kM = 128;       // rows of a query tile: (token, query head) pairs of one kv head
constexpr int kStart = 2;     // what starting an item counts, in tiles
constexpr int kPlan = 1024;   // entries of the plan in shared memory
constexpr int kMostBad = 8;   // masked tiles of a segment (6 at the most: see Seg::masked)
constexpr int kSlots = 2;     // segments under way

// Weights are taken 2^room above the power of two that a running maximum stands
// for, and the maximum follows only scores kLazy above it: below 2^15, the
// greatest that fp16 holds, and as far as can be above its smallest steps.
constexpr float kRoom16 = 7.0f, kLazy = 8.0f;

// ---------------------------------------------------------------- sequences and items

// The rows of a sequence that a call has: tensor rows row0 .. row0 + m - 1 at
// positions pos0 .. .
struct Span {
  int row0, m, pos0;
};

__device__ __forceinline__ Span read_span(const PagedChunkParams& p, int s, bool report) {
  Span r = {0, 0, 0};
  const PagedBatch& b = p.batch;
  int64_t a = s, e = s + 1;
  if (b.cu) {
    a = b.cu[s];
    e = b.cu[s + 1];
  }
  bool bad = e < a;
  const int64_t lo = a > 0 ? a : 0, hi = e < p.n ? e : p.n;
  int64_t pos = 0;
  if (p.prompt) {
    bad = bad || (e > a && (a < 0 || e > p.n));  // rows that are not there
  } else {
    const int len = b.lens[s];
    if (!b.cu && len == 0) return r;  // a padded place of the batch
    pos = len - (e - lo);
    bad = bad || (e > a && (len < e - a || len > static_cast<int64_t>(b.max_pages) << p.pool.page_shift));
  }
  if (bad) {
    if (report) atomicExch(p.pool.err, kErrBadState);
    return r;
  }
  if (hi <= lo) return r;
  r.row0 = static_cast<int>(lo);
  r.m = static_cast<int>(hi - lo);
  r.pos0 = static_cast<int>(pos);
  return r;
}

// Item j of a sequence and kv head: rows j R .. of its (token, head) pairs.
struct Item {
  int tok, rem;    // first token; row 0 is its head `rem`
  int rows;
  int last;        // last token
  int t0, t1;      // tiles that its rows see: t0 .. t1 - 1
};

__device__ __forceinline__ int items_of(int m, int gqa, int R) {
  return static_cast<int>((static_cast<int64_t>(m) * gqa + R - 1) / R);
}

__device__ __forceinline__ Item item_of(const Span& s, int64_t j, int gqa, int R, int window) {
  Item it;
  const int64_t x = j * R, total = static_cast<int64_t>(s.m) * gqa;
  it.tok = static_cast<int>(x / gqa);
  it.rem = static_cast<int>(x - static_cast<int64_t>(it.tok) * gqa);
  it.rows = static_cast<int>(total - x < R ? total - x : R);
  it.last = it.tok + (it.rem + it.rows - 1) / gqa;
  const int first = s.pos0 + it.tok;
  it.t0 = window && first >= window ? (first - window + 1) / kTokens : 0;
  it.t1 = (s.pos0 + it.last) / kTokens + 1;
  return it;
}

// What a CTA does at a time: tiles t0 .. t1 - 1 of an item, written by the
// warp that plans, read by all.
struct Seg {
  const int32_t* table;  // the sequence's pages
  int done;              // 1: no more
  int row, pos;          // tensor row and position of the item's first token
  int rem, rows;
  int kvh;
  int t0, t1;
  int lo, hi;            // positions that any of the item's rows sees: lo .. hi - 1
  int whole;             // the item has no other segments
  int slot;              // else: where the partial result goes
  int bad_tiles;         // tiles with infinite or NaN values among the masked ones
  int bad_tile[kMostBad];
  uint32_t bad[kMostBad][4];  // their tokens
};

// Whether some row of the rows first .. (positions) to last sees only a part of
// tile t.  Those are the tiles of the last rows' positions and of the window's
// lower ends, at most three each: rows first .. last are 256 tokens at the most.
__device__ __forceinline__ bool masked_tile(int t, int first, int last, int window) {
  return t * kTokens + kTokens - 1 > first || (window && t * kTokens <= last - window);
}

// A CTA's note for the join.
struct Note {
  int rows;       // of the item whose first piece this CTA left in its slot 1; 0: none
  int row, rem, kvh;
  int cont;       // 1: its slot 0 continues the item of the CTA before, 2: and ends it
  int pad[3];
};

// Where a boundary at weight b cuts an item of nt tiles that starts at x: not
// within `tol` of its ends, where a partial result costs more than the uneven work.
__device__ __forceinline__ int cut_at(int64_t b, int64_t x, int nt, int tol) {
  const int64_t d = b - x;
  if (d <= tol) return 0;
  if (nt + kStart - d <= tol) return nt;
  return static_cast<int>(d) - kStart;
}

// ---------------------------------------------------------------- shape

template <int D, int NQ>
struct Shape {
  static constexpr int R = NQ * kM;
  static constexpr int H = D / 64;                 // 128-byte halves of a row
  static constexpr int half = kTokens * 128;       // bytes of a tile's half
  static constexpr int tile = H * half;
  static constexpr int softmax = NQ * 128;         // threads
  static constexpr int threads = softmax + 128;    // and the warps that load, multiply and look (two)
  static constexpr int NST = D == 128 ? (NQ == 2 ? 5 : 6) : 8;
  static constexpr int q = 0;
  static constexpr int ring = NQ * tile;           // (a query tile is as large as a key tile)
  static constexpr int ctl = ring + NST * tile;
  static constexpr int smem = ctl + 2048;
  static_assert(smem <= 227 * 1024 && NST * tile >= kPlan * 8, "shared memory");
  static constexpr int tS = 0, tO = 2 * kTokens;   // columns: two score tiles, then the outputs
};

struct Ctl {
  uint64_t full[8], empty[8];   // ring stages
  // one for each query tile, or where there is one for each of its score tiles, of which a role may be a tile ahead of
  // another: a wait tells a phase from the one before only
  uint64_t q_full[2], s_full[2], p_full[2], o_done[2];
  uint64_t group[2];            // a group's warps have read its results
  uint64_t looked[8];           // masked values of the stage have been looked through
  uint64_t seg_full[kSlots], seg_empty[kSlots];
  uint64_t fin;
  uint32_t tmem;
  int quit;
  Seg seg[kSlots];
};
static_assert(sizeof(Ctl) <= 2048, "control");

// A bounded wait that ends when another of the CTA's waits gave up.
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t phase, int32_t* err, volatile int* quit) {
  for (int i = 0; i < 1 << 12; ++i) {
    const uint32_t addr = smem_u32(bar);
    for (int k = 0; k < 1 << 10; ++k) {
      uint32_t done;
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(done)
          : "r"(addr), "r"(phase)
          : "memory");
      if (done) return true;
    }
    if (*quit) return false;
  }
  atomicExch(err, kErrWaitTimeout);
  *quit = 1;
  return false;
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t phase, int32_t* err, int* quit) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(phase)
      : "memory");
  return done || wait_slow(bar, phase, err, quit);
}

__device__ __forceinline__ void tma5(void* dst, const CUtensorMap* map, int c1, int c2, int c3, int c4, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma4(void* dst, const CUtensorMap* map, int c1, int c2, int c3, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
      : "memory");
}

struct Stage {  // place in a ring of N
  int i;
  uint32_t phase;
  template <int N>
  __device__ __forceinline__ void next() {
    if (++i == N) {
      i = 0;
      phase ^= 1;
    }
  }
};

template <typename T>
struct Fmt;
template <>
struct Fmt<__half> {
  static constexpr uint32_t code = 0, expo = 0x7c007c00u, carry = 0x04000400u;
  static constexpr float room = kRoom16;
};
template <>
struct Fmt<__nv_bfloat16> {
  static constexpr uint32_t code = 1, expo = 0x7f807f80u, carry = 0x00800080u;
  static constexpr float room = 0.0f;
};
__device__ __forceinline__ uint32_t pack2(__half*, float x, float y) { return h2_as_u32(__floats2half2_rn(x, y)); }
__device__ __forceinline__ uint32_t pack2(__nv_bfloat16*, float x, float y) {
  __nv_bfloat162 r = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<uint32_t*>(&r);
}

struct Launch {
  PagedChunkParams p;
  CUtensorMap km, vm;   // pages: km alone; prompts: keys, values
  int grid;
  int slot_rows;        // rows of a partial result
  int64_t partials;     // bytes of the workspace before them
};

// ---------------------------------------------------------------- planning

// Weight (tiles, and kStart an item) of a sequence's items of one kv head, by a warp.
__device__ __forceinline__ int64_t span_weight(const Span& s, int gqa, int R, int window, int lane) {
  const int q = items_of(s.m, gqa, R);
  int64_t w = 0;
  for (int j = lane; j < q; j += 32) {
    const Item it = item_of(s, j, gqa, R, window);
    w += it.t1 - it.t0 + kStart;
  }
  for (int o = 16; o; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
  return w;
}

// Entry e of the plan: the weight of sequences e k .. e k + k - 1, all kv heads.
__device__ __forceinline__ void plan_entries(const PagedChunkParams& p, int R, int64_t* plan, int entries, int k,
                                             int warp, int warps, int lane) {
  for (int e0 = warp * 32; e0 < entries; e0 += warps * 32) {
    const int e = e0 + lane;
    int64_t w = 0;
    for (int i = 0; i < k; ++i) {
      const int64_t s = static_cast<int64_t>(e) * k + i;
      Span sp = {0, 0, 0};
      if (e < entries && s < p.batch.seqs) sp = read_span(p, static_cast<int>(s), blockIdx.x == 0);
      // few items: by the lane itself; many: by the warp
      const int q = items_of(sp.m, p.gqa, R);
      if (q <= 4)
        for (int j = 0; j < q; ++j) {
          const Item it = item_of(sp, j, p.gqa, R, p.window);
          w += it.t1 - it.t0 + kStart;
        }
      uint32_t big = __ballot_sync(0xffffffffu, q > 4);
      while (big) {
        const int l = __ffs(big) - 1;
        big &= big - 1;
        const Span o = {__shfl_sync(0xffffffffu, sp.row0, l), __shfl_sync(0xffffffffu, sp.m, l),
                        __shfl_sync(0xffffffffu, sp.pos0, l)};
        const int64_t x = span_weight(o, p.gqa, R, p.window, lane);
        if (lane == l) w += x;
      }
    }
    if (e < entries) plan[e] = w * p.hkv;
  }
}

// Walks a CTA's items: all lanes of the warp hold the same state.
struct Walk {
  int64_t b0, b1;     // the CTA's range of weights
  int64_t x;          // where the present item starts
  int s, kvh, j, q;   // sequence, kv head, item of q
  Span sp;
  int tol;
};

__device__ __forceinline__ void walk_start(const PagedChunkParams& p, int R, const int64_t* plan, int entries, int k,
                                           int cta, int grid, int lane, Walk& w) {
  // each lane has a run of entries
  const int per = (entries + 31) / 32;
  int64_t sum = 0;
  for (int i = 0; i < per; ++i)
    if (lane * per + i < entries) sum += plan[lane * per + i];
  int64_t end = sum;
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, end, o);
    if (lane >= o) end += v;
  }
  const int64_t total = __shfl_sync(0xffffffffu, end, 31);
  int64_t quota = (total + grid - 1) / grid;
  if (quota < 3 * kStart) quota = 3 * kStart;
  w.tol = static_cast<int>(quota / 16 < kStart + 1 ? kStart + 1 : quota / 16 > 64 ? 64 : quota / 16);
  w.b0 = quota * cta;
  w.b1 = w.b0 + quota < total ? w.b0 + quota : total;
  w.s = p.batch.seqs;  // nothing to do
  if (w.b0 >= total) return;
  const bool mine = end > w.b0 && end - sum <= w.b0;
  const int src = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
  int e = 0;
  int64_t x = end - sum;
  if (mine)
    for (e = lane * per; e + 1 < entries && x + plan[e] <= w.b0; ++e) x += plan[e];
  e = __shfl_sync(0xffffffffu, e, src);
  x = __shfl_sync(0xffffffffu, x, src);
  // the sequence of the entry, its kv head, its item
  int64_t s = static_cast<int64_t>(e) * k;
  for (; s < p.batch.seqs; ++s) {
    w.sp = read_span(p, static_cast<int>(s), false);
    const int64_t one = span_weight(w.sp, p.gqa, R, p.window, lane), all = one * p.hkv;
    if (all > 0 && x + all > w.b0) {
      w.kvh = static_cast<int>((w.b0 - x) / one);
      x += one * w.kvh;
      break;
    }
    x += all;
  }
  if (s >= p.batch.seqs) return;
  w.s = static_cast<int>(s);
  w.q = items_of(w.sp.m, p.gqa, R);
  for (int j0 = 0; j0 < w.q; j0 += 32) {
    int64_t wt = 0;
    if (j0 + lane < w.q) {
      const Item it = item_of(w.sp, j0 + lane, p.gqa, R, p.window);
      wt = it.t1 - it.t0 + kStart;
    }
    int64_t e2 = wt;
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, e2, o);
      if (lane >= o) e2 += v;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, wt > 0 && x + e2 > w.b0);
    if (hit) {
      const int l = __ffs(hit) - 1;
      w.j = j0 + l;
      w.x = x + __shfl_sync(0xffffffffu, e2 - wt, l);
      return;
    }
    x += __shfl_sync(0xffffffffu, e2, 31);
  }
  w.s = p.batch.seqs;
}

// To the next item; false where there is none.
__device__ __forceinline__ bool walk_next(const PagedChunkParams& p, int R, int tiles, Walk& w) {
  w.x += tiles + kStart;
  if (++w.j < w.q) return true;
  w.j = 0;
  if (++w.kvh < p.hkv) return true;
  w.kvh = 0;
  while (++w.s < p.batch.seqs) {
    w.sp = read_span(p, w.s, false);
    w.q = items_of(w.sp.m, p.gqa, R);
    if (w.q) return true;
  }
  return false;
}

// ---------------------------------------------------------------- values that are no numbers

template <typename T, int D, bool PROMPT>
__device__ __forceinline__ const uint8_t* value_row(const PagedChunkParams& p, const Seg& sg, int t) {
  if (PROMPT)
    return p.v.data + 2 * ((static_cast<int64_t>(sg.row) - sg.pos + t) * p.v.token_stride + sg.kvh * p.v.head_stride);
  const int page = sg.table[t >> p.pool.page_shift];
  if (page < 0 || page >= p.pool.num_pages) return nullptr;
  const int in = t & ((1 << p.pool.page_shift) - 1);
  const uint8_t* tile = p.pool.pages + page * p.pool.page_stride + sg.kvh * p.pool.head_stride +
                        static_cast<int64_t>(in / kTile) * p.pool.tile_bytes;
  return pool_ok(p.pool, tile, p.pool.tile_bytes) ? tile : nullptr;
}

// The masked tiles' values that are not finite were left out of the products
// (times a weight of 0 they would be NaN); the rows that see them get them here.
template <typename T, int D, bool PROMPT>
__device__ __forceinline__ void add_bad(const PagedChunkParams& p, const Seg& sg, int first, int last, int c0, float (&o)[32]) {
  for (int i = 0; i < sg.bad_tiles && i < kMostBad; ++i)
    for (int b = 0; b < kTokens; ++b) {
      const int t = sg.bad_tile[i] * kTokens + b;
      if (!(sg.bad[i][b / 32] >> (b % 32) & 1) || t < first || t > last) continue;
      const uint8_t* v = value_row<T, D, PROMPT>(p, sg, t);
      if (!v) continue;
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        const int ch = c0 + c;
        const T* x = PROMPT ? reinterpret_cast<const T*>(v) + ch
                            : reinterpret_cast<const T*>(v + 32 * D + (t % kTile) * 2 * D +
                                                         16 * tile_chunk16(ch / 8, t % kTile) + ch % 8 * 2);
        const float f = Num<T>::to(*x);
        if (!isfinite(f)) o[c] += f;
      }
    }
}

// ---------------------------------------------------------------- the kernel

template <typename T, int D, int NQ, bool PROMPT>
__global__ void __launch_bounds__(Shape<D, NQ>::threads, 1) paged_chunk_kernel(const __grid_constant__ Launch a) {
  using S = Shape<D, NQ>;
  extern __shared__ __align__(1024) uint8_t sm[];
  Ctl& ctl = *reinterpret_cast<Ctl*>(sm + S::ctl);
  const PagedChunkParams& p = a.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int W0 = S::softmax / 32;  // the loading warp; W0 + 1 multiplies, W0 + 2 and W0 + 3 look
  int32_t* err = p.pool.err;
  int* quit = &ctl.quit;

  if (tid == 0) {
    for (int i = 0; i < S::NST; ++i) {
      mbar_init(&ctl.full[i], 1);
      mbar_init(&ctl.empty[i], 3);  // the products have read it, and the two warps that look have passed it
      mbar_init(&ctl.looked[i], 2);
    }
    for (int g = 0; g < NQ; ++g) {
      mbar_init(&ctl.q_full[g], 4);
      mbar_init(&ctl.s_full[g], 1);
      mbar_init(&ctl.p_full[g], 4);
      mbar_init(&ctl.o_done[g], 1);
      mbar_init(&ctl.group[g], 4);
    }
    if (NQ == 1) {
      mbar_init(&ctl.s_full[1], 1);
      mbar_init(&ctl.p_full[1], 4);
      mbar_init(&ctl.o_done[1], 1);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&ctl.seg_full[i], 1);
      mbar_init(&ctl.seg_empty[i], W0 + 3);
    }
    mbar_init(&ctl.fin, 1);
    ctl.quit = 0;
    fence_mbar_init();
  }
  if (warp == W0 + 1) tmem_alloc(&ctl.tmem, 512);
  grid_dep_wait();
  grid_dep_launch();
  const int per_entry = (p.batch.seqs - 1) / kPlan + 1, entries = (p.batch.seqs - 1) / per_entry + 1;
  int64_t* plan = reinterpret_cast<int64_t*>(sm + S::ring);
  plan_entries(p, S::R, plan, entries, per_entry, warp, S::threads / 32, lane);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tm = ctl.tmem;

  if (warp == W0) {
    // ================= plans, and loads keys and values
    Walk w;
    walk_start(p, S::R, plan, entries, per_entry, blockIdx.x, a.grid, lane, w);
    __syncwarp();
    fence_proxy_async_smem();  // the plan's bytes become the ring's
    Note note = {};
    Stage st = {0, 0}, slot = {0, 0};
    int issued = 0;
    bool ok = true;
    bool more = w.s < p.batch.seqs;
    while (more && ok && w.x < w.b1) {
      const Item it = item_of(w.sp, w.j, p.gqa, S::R, p.window);
      const int nt = it.t1 - it.t0;
      const int from = w.x < w.b0 ? cut_at(w.b0, w.x, nt, w.tol) : 0;
      const int to = w.x + nt + kStart > w.b1 ? cut_at(w.b1, w.x, nt, w.tol) : nt;
      if (from < to) {
        ok = wait(&ctl.seg_empty[slot.i], slot.phase ^ 1, err, quit);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const int pos = w.sp.pos0 + it.tok, hi = w.sp.pos0 + it.last + 1;
        const int lo = p.window && pos >= p.window ? pos - p.window + 1 : 0;
        const int32_t* table = PROMPT ? nullptr : p.batch.table + w.s * p.batch.table_stride;
        if (lane == 0) {
          Seg& sg = ctl.seg[slot.i];
          sg.table = table;
          sg.done = 0;
          sg.row = w.sp.row0 + it.tok;
          sg.pos = pos;
          sg.rem = it.rem;
          sg.rows = it.rows;
          sg.kvh = w.kvh;
          sg.t0 = it.t0 + from;
          sg.t1 = it.t0 + to;
          sg.lo = lo;
          sg.hi = hi;
          sg.whole = from == 0 && to == nt;
          sg.slot = 2 * blockIdx.x + (from == 0);
          sg.bad_tiles = 0;
          for (int i = 0; i < kMostBad; ++i)
            for (int k = 0; k < 4; ++k) sg.bad[i][k] = 0;
          mbar_arrive(&ctl.seg_full[slot.i]);
        }
        slot.next<kSlots>();
        if (from > 0) {
          note.cont = to == nt ? 2 : 1;
        } else if (to < nt) {
          note.rows = it.rows;
          note.row = w.sp.row0 + it.tok;
          note.rem = it.rem;
          note.kvh = w.kvh;
        }
        for (int t = it.t0 + from; t < it.t0 + to && ok; ++t) {
          // a lane's page (of both, where rows have two halves), the same for keys and values
          int page = -1;
          const int pages = kTokens >> p.pool.page_shift;
          const int at = t * kTokens + ((lane / S::H) << p.pool.page_shift);
          if (!PROMPT) {
            if (lane < pages * S::H && at < hi && at + (1 << p.pool.page_shift) > lo) {
              const int32_t* entry = table + (at >> p.pool.page_shift);
              if (table_ok(p.batch, entry, err)) {
                page = *entry;
                if (page < 0 || page >= p.pool.num_pages) {
                  atomicExch(err, kErrBadPage);
                  page = -1;
                } else if (!pool_ok(p.pool, p.pool.pages + page * p.pool.page_stride + w.kvh * p.pool.head_stride,
                                    p.pool.head_stride)) {
                  page = -1;
                }
              }
            }
          }
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            if (ok) ok = wait(&ctl.empty[st.i], st.phase ^ 1, err, quit);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            uint8_t* dst = sm + S::ring + st.i * S::tile;
            uint64_t* bar = &ctl.full[st.i];
            if (PROMPT) {
              if (lane == 0) mbar_arrive_expect_tx(bar, S::tile);
              __syncwarp();
              if (lane < S::H)
                tma4(dst + lane * S::half, kv ? &a.vm : &a.km, w.sp.row0 + t * kTokens, lane, w.kvh, bar);
            } else {
              const uint32_t bytes = 128u << p.pool.page_shift;  // of a page's half
              const int count = __popc(__ballot_sync(0xffffffffu, page >= 0));
              if (lane == 0) {
                if (count)
                  mbar_arrive_expect_tx(bar, count * bytes);
                else
                  mbar_arrive(bar);
              }
              __syncwarp();
              if (page >= 0) {
                const int tiles = 1 << (p.pool.page_shift - 4);
                tma5(dst + (lane % S::H) * S::half + (lane / S::H) * bytes, &a.km, 0, (page * p.hkv + w.kvh) * tiles,
                     lane % S::H, kv, bar);
              }
            }
            st.next<S::NST>();
            if (issued < S::NST) ++issued;
          }
        }
      }
      more = walk_next(p, S::R, nt, w);
    }
    // no more segments
    if (ok) ok = wait(&ctl.seg_empty[slot.i], slot.phase ^ 1, err, quit);
    ok = __all_sync(0xffffffffu, ok);
    if (ok && lane == 0) {
      ctl.seg[slot.i].done = 1;
      mbar_arrive(&ctl.seg_full[slot.i]);
    }
    if (lane == 0) {
      Note* notes = reinterpret_cast<Note*>(p.ws);
      if (in_range(notes + blockIdx.x, sizeof(Note), p.ws, p.ws_hi, err)) notes[blockIdx.x] = note;
    }
    // every copy has landed before the CTA ends
    for (int i = 0; i < issued; ++i) {
      st.i = st.i ? st.i - 1 : S::NST - 1;
      if (st.i == S::NST - 1) st.phase ^= 1;
      mbar_wait(&ctl.full[st.i], st.phase, err, 1u << 16);
    }
  } else if (warp == W0 + 1) {
    // ================= multiplies: scores into columns tS, weights times values into tO
    if (lane == 0) {
      constexpr uint32_t f = Fmt<T>::code << 7 | Fmt<T>::code << 10;
      constexpr uint32_t idO = idesc_f16_f32(kM, D) | f | 1u << 16;  // values run along channels
      const uint32_t idS = idesc_f16_f32(kM, kTokens) | f | (p.alpha < 0.0f ? 1u << 13 : 0u);  // -q for a scale below 0
      const uint32_t sq = smem_u32(sm + S::q), sr = smem_u32(sm + S::ring);
      Stage st = {0, 0}, slot = {0, 0};
      uint32_t qph[2] = {0, 0}, pph = 0, lookph = 0;
      bool ok = true;
      auto scores = [&](int g, int buf, int stage) {
        const uint64_t dq = smem_desc_sw128(sq + g * S::tile, 16, 1024), dk = smem_desc_sw128(sr + stage * S::tile, 16, 1024);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint64_t off = ((k / 4) * S::half + (k % 4) * 32) >> 4;
          umma_f16(tm + S::tS + kTokens * buf, dq + off, dk + off, idS, k > 0);
        }
        umma_commit(&ctl.s_full[buf]);
      };
      auto outputs = [&](int g, int buf, int stage, bool first) {
        const uint64_t dv = smem_desc_sw128(sr + stage * S::tile, S::half, 1024);
#pragma unroll
        for (int k = 0; k < kTokens / 16; ++k)
          umma_f16_ts(tm + S::tO + D * g, tm + S::tS + kTokens * buf + 8 * k, dv + ((2048 * k) >> 4), idO, !first || k > 0);
      };
      while (ok) {
        ok = wait(&ctl.seg_full[slot.i], slot.phase, err, quit);
        if (!ok) break;
        const Seg& sg = ctl.seg[slot.i];
        if (sg.done) break;
        const int t0 = sg.t0, nt = sg.t1 - t0, pos = sg.pos, rem = sg.rem, rows = sg.rows, hi = sg.hi;
        int ng[NQ];  // tiles of each query tile
#pragma unroll
        for (int g = 0; g < NQ; ++g) {
          const int r = rows < kM * (g + 1) ? rows : kM * (g + 1);
          const int end = (pos + (rem + r - 1) / p.gqa) / kTokens + 1;
          ng[g] = kM * g >= rows ? 0 : (end < sg.t1 ? end : sg.t1) - t0;
          if (ng[g] > 0) {
            ok = ok && wait(&ctl.q_full[g], qph[g], err, quit);
            qph[g] ^= 1;
          }
        }
        mbar_arrive(&ctl.seg_empty[slot.i]);
        slot.next<kSlots>();
        ok = ok && wait(&ctl.full[st.i], st.phase, err, quit);
        if (!ok) break;
        tc_fence_after_sync();
        int kst = st.i;  // the stage of the keys in hand
#pragma unroll
        for (int g = 0; g < NQ; ++g)
          if (ng[g] > 0) scores(g, NQ == 1 ? 0 : g, kst);
        umma_commit(&ctl.empty[kst]);
        st.next<S::NST>();
        for (int i = 0; i < nt && ok; ++i) {
          const Stage v = st;
          st.next<S::NST>();
          const bool next = i + 1 < nt;
          if (NQ == 1 && next) {
            ok = wait(&ctl.full[st.i], st.phase, err, quit);
            if (!ok) break;
            tc_fence_after_sync();
            scores(0, (i + 1) & 1, st.i);
            umma_commit(&ctl.empty[st.i]);
          }
          if (masked_tile(t0 + i, pos, hi - 1, p.window)) {
            ok = wait(&ctl.looked[v.i], lookph >> v.i & 1, err, quit);
            lookph ^= 1u << v.i;
          } else {
            ok = wait(&ctl.full[v.i], v.phase, err, quit);
          }
          if (!ok) break;
          tc_fence_after_sync();
          bool have = false;
#pragma unroll
          for (int g = 0; g < NQ; ++g) {
            if (i >= ng[g]) continue;
            const int buf = NQ == 1 ? i & 1 : g;
            ok = ok && wait(&ctl.p_full[buf], pph >> buf & 1, err, quit);
            pph ^= 1u << buf;
            if (!ok) break;
            tc_fence_after_sync();
            outputs(g, buf, v.i, i == 0);
            if (NQ == 1 || i + 1 == ng[g]) umma_commit(&ctl.o_done[buf]);
            if (NQ > 1 && i + 1 < ng[g]) {
              if (!have) {
                ok = wait(&ctl.full[st.i], st.phase, err, quit);
                have = true;
                if (!ok) break;
                tc_fence_after_sync();
              }
              scores(g, g, st.i);
            }
          }
          if (!ok) break;
          umma_commit(&ctl.empty[v.i]);
          if (next) {
            if (NQ > 1) umma_commit(&ctl.empty[st.i]);
            st.next<S::NST>();
          }
        }
      }
      umma_commit(&ctl.fin);  // nothing is under way when the columns are given back
      mbar_wait(&ctl.fin, 0, err, 1u << 20);
    }
    __syncwarp();
  } else if (warp > W0) {
    // ================= look through the values of masked tiles
    Stage st = {0, 0}, slot = {0, 0};
    bool ok = true;
    while (ok) {
      ok = __all_sync(0xffffffffu, wait(&ctl.seg_full[slot.i], slot.phase, err, quit));
      if (!ok) break;
      Seg& sg = ctl.seg[slot.i];
      if (sg.done) break;
      int seen = 0;
      for (int t = sg.t0; t < sg.t1 && ok; ++t) {
        // every stage in turn, so that none is mistaken for its last use
        ok = __all_sync(0xffffffffu, wait(&ctl.full[st.i], st.phase, err, quit));
        if (!ok) break;
        if (lane == 0) mbar_arrive(&ctl.empty[st.i]);
        st.next<S::NST>();
        const Stage v = st;
        st.next<S::NST>();
        ok = __all_sync(0xffffffffu, wait(&ctl.full[v.i], v.phase, err, quit));
        if (!ok) break;
        if (!masked_tile(t, sg.pos, sg.hi - 1, p.window)) {
          if (lane == 0) mbar_arrive(&ctl.empty[v.i]);
          continue;
        }
        uint8_t* tile = sm + S::ring + v.i * S::tile;
        const int me = tid - (W0 + 2) * 32;
#pragma unroll 8
        for (int i = me; i < S::tile / 16; i += 64) {
          uint4* at = reinterpret_cast<uint4*>(tile) + i;
          uint4 x = *at;
          constexpr uint32_t E = Fmt<T>::expo, C = Fmt<T>::carry;
          uint32_t any = ((x.x & E) + C) | ((x.y & E) + C) | ((x.z & E) + C) | ((x.w & E) + C);
          if (any & 0x80008000u) {
            uint32_t* w = reinterpret_cast<uint32_t*>(&x);
            for (int k = 0; k < 4; ++k) {
              if (((w[k] & E) + C) & 0x8000u) w[k] &= 0xffff0000u;
              if (((w[k] & E) + C) & 0x80000000u) w[k] &= 0xffffu;
            }
            *at = x;
            const int tok = (i * 16 % S::half) / 128;
            if (seen < kMostBad) atomicOr(&sg.bad[seen][tok / 32], 1u << (tok % 32));
          }
        }
        if (me == 0 && seen < kMostBad) sg.bad_tile[seen] = t;
        if (me == 0) sg.bad_tiles = seen + 1;
        ++seen;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&ctl.looked[v.i]);
          mbar_arrive(&ctl.empty[v.i]);
        }
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.seg_empty[slot.i]);
      slot.next<kSlots>();
    }
  } else {
    // ================= softmax: a thread a row
    const int g = NQ == 1 ? 0 : warp >> 2, r = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t tO = tm + S::tO + D * g + lanes;
    uint8_t* qs = sm + S::q + g * S::tile;
    const float alpha = fabsf(p.alpha);
    const f2 alpha2 = f2_of(alpha, alpha);
    Stage slot = {0, 0};
    uint32_t sph[2] = {0, 0}, oph = 0, gph = 0;  // phases
    bool ok = true;
    while (ok) {
      ok = __all_sync(0xffffffffu, wait(&ctl.seg_full[slot.i], slot.phase, err, quit));
      if (!ok) break;
      const Seg& sg = ctl.seg[slot.i];
      if (sg.done) break;
      const int rows = sg.rows - kM * g < kM ? sg.rows - kM * g : kM;
      if (rows > 0) {
        const int x0 = sg.rem + kM * g;  // row r is head (x0 + r) % gqa of token (x0 + r) / gqa
        const int pos = sg.pos, t0 = sg.t0;
        const int first_lim = pos + x0 / p.gqa, last_lim = pos + (x0 + rows - 1) / p.gqa;
        const int end = last_lim / kTokens + 1;
        const int nt = (end < sg.t1 ? end : sg.t1) - t0;
        const int lim = r < rows ? pos + (x0 + r) / p.gqa : last_lim;
        const int low = p.window ? lim - p.window + 1 : 0;
        float m = -INFINITY, l = 0.0f;
        if (nt > 0) {
          // ---- query rows into shared memory
#pragma unroll 4
          for (int i = r; i < kM * (D / 8); i += 128) {
            const int row = i / (D / 8), ch = i % (D / 8);
            uint4 v = make_uint4(0, 0, 0, 0);
            if (row < rows) {
              const int tk = (x0 + row) / p.gqa, hh = x0 + row - tk * p.gqa;
              const T* src = reinterpret_cast<const T*>(p.q.data) + (static_cast<int64_t>(sg.row) + tk) * p.q.token_stride +
                             (sg.kvh * p.gqa + hh) * p.q.head_stride + 8 * ch;
              if (rows_ok(p.q, src, 16, err)) rows::load8(src, p.q_vec, v);
            }
            *reinterpret_cast<uint4*>(qs + (ch / 8) * S::half + row * 128 + (((ch & 7) ^ (row & 7)) << 4)) = v;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl.q_full[g]);
          for (int i = 0; i < nt; ++i) {
            const int buf = NQ == 1 ? i & 1 : g;
            ok = __all_sync(0xffffffffu, wait(&ctl.s_full[buf], sph[NQ == 1 ? buf : 0], err, quit));
            sph[NQ == 1 ? buf : 0] ^= 1;
            if (!ok) break;
            tc_fence_after_sync();
            const uint32_t tS = tm + S::tS + kTokens * buf + lanes;
            uint32_t x[4][32];
#pragma unroll
            for (int k = 0; k < 4; ++k) tmem_ld32(tS + 32 * k, x[k]);
#pragma unroll
            for (int k = 0; k < 4; ++k) tmem_ld_wait(x[k]);
            const int tb = (t0 + i) * kTokens;
            if (tb + kTokens - 1 > first_lim || (p.window && tb <= last_lim - p.window)) {
              const int a0 = low - tb, a1 = lim - tb;  // columns a0 .. a1 are seen
#pragma unroll
              for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int c = 0; c < 32; ++c)
                  if (32 * k + c < a0 || 32 * k + c > a1) x[k][c] = 0xff800000u;
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < 32; c += 2)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mx[k] = fmaxf(fmaxf(mx[k], __uint_as_float(x[k][c])), __uint_as_float(x[k][c + 1]));
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * alpha;
            const bool need = top > m + kLazy;
            if (__any_sync(0xffffffffu, need)) {
              float f = 1.0f;
              if (need) {
                f = ex2(m - top);
                m = top;
              }
              l *= f;
              if (i > 0) {
                if (NQ == 1) {  // the product of the tile before (for two tiles s_full says so)
                  ok = __all_sync(0xffffffffu, wait(&ctl.o_done[buf ^ 1], (oph >> (buf ^ 1) & 1) ^ 1, err, quit));
                  if (!ok) break;
                  tc_fence_after_sync();
                }
#pragma unroll 1
                for (int c = 0; c < D; c += 16) {
                  uint32_t o[16];
                  tmem_ld16(tO + c, o);
                  tmem_ld_wait(o);
#pragma unroll
                  for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                  tmem_st16(tO + c, o);
                }
              }
            }
            if (NQ == 1) oph ^= 1u << buf;
            const float nm = Fmt<T>::room - (m == -INFINITY ? 0.0f : m);
            const f2 nm2 = f2_of(nm, nm);
            f2 sum[2] = {f2_of(0.0f, 0.0f), f2_of(0.0f, 0.0f)};
            T* const type = nullptr;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t w[32];
#pragma unroll
              for (int c = 0; c < 32; ++c) {
                const uint32_t *xx = &x[2 * h + c / 16][2 * (c % 16)];
                float u, v;
                f2_get(fma2(f2_of(__uint_as_float(xx[0]), __uint_as_float(xx[1])), alpha2, nm2), u, v);
                u = ex2(u);
                v = ex2(v);
                sum[c & 1] = add2(sum[c & 1], f2_of(u, v));
                w[c] = pack2(type, u, v);
              }
              tmem_st32(tS + 32 * h, w);
            }
            float s0, s1, s2, s3;
            f2_get(sum[0], s0, s1);
            f2_get(sum[1], s2, s3);
            l += (s0 + s1) + (s2 + s3);
            tmem_st_wait();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl.p_full[buf]);
          }
          if (!ok) break;
          if (NQ == 1) {
            const int buf = (nt - 1) & 1;
            ok = wait(&ctl.o_done[buf], (oph >> buf & 1) ^ 1, err, quit);
          } else {
            ok = wait(&ctl.o_done[g], oph, err, quit);
            oph ^= 1;
          }
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after_sync();
        }
        // ---- the rows' results
        const int tk = (x0 + r) / p.gqa, head = sg.kvh * p.gqa + x0 + r - tk * p.gqa;
        const int64_t at = (static_cast<int64_t>(sg.row) + tk) * p.hkv * p.gqa + head;
        if (sg.whole) {
          const float inv = l != 0.0f ? __fdividef(1.0f, l) : 0.0f;
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            tmem_ld32(tO + c, o);
            tmem_ld_wait(o);
            float y[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) y[k] = l != 0.0f ? __uint_as_float(o[k]) * inv : 0.0f;
            if (sg.bad_tiles && l != 0.0f) add_bad<T, D, PROMPT>(p, sg, low, lim, c, y);
            if (r < rows) {
              T* const type = nullptr;
              uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(p.out) + at * D + c);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                dst[k] = make_uint4(pack2(type, y[8 * k], y[8 * k + 1]), pack2(type, y[8 * k + 2], y[8 * k + 3]),
                                    pack2(type, y[8 * k + 4], y[8 * k + 5]), pack2(type, y[8 * k + 6], y[8 * k + 7]));
            }
          }
          if (p.lse && r < rows)
            p.lse[at] = l == 0.0f ? -INFINITY : ((m - Fmt<T>::room) + log2f(l)) * 0.69314718055994531f;
        } else {
          // m, l of every row, then the outputs, four channels of all rows together
          float* part = reinterpret_cast<float*>(p.ws + a.partials) + static_cast<int64_t>(sg.slot) * a.slot_rows * (D + 2);
          const int rr = kM * g + r;
          if (rr < a.slot_rows && in_range(part, a.slot_rows * (D + 2) * 4, p.ws, p.ws_hi, err)) {
            part[rr] = m;
            part[a.slot_rows + rr] = l;
          }
          if (nt > 0) {
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              tmem_ld32(tO + c, o);
              tmem_ld_wait(o);
              float y[32];
#pragma unroll
              for (int k = 0; k < 32; ++k) y[k] = __uint_as_float(o[k]);
              if (sg.bad_tiles && l != 0.0f) add_bad<T, D, PROMPT>(p, sg, low, lim, c, y);
              if (rr < a.slot_rows) {
                float4* dst = reinterpret_cast<float4*>(part + 2 * a.slot_rows) + rr;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                  dst[(c / 4 + k) * a.slot_rows] = make_float4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
              }
            }
          }
        }
        tc_fence_before_sync();
        // the query rows of the next segment are written by all of the group's threads
        // (a bounded wait: a warp whose wait gave up does not come)
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.group[g]);
        ok = __all_sync(0xffffffffu, wait(&ctl.group[g], gph, err, quit));
        gph ^= 1;
        if (!ok) break;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.seg_empty[slot.i]);
      slot.next<kSlots>();
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == W0 + 1) {
    tc_fence_after_sync();
    tmem_dealloc(tm, 512);
  }
}

// Rows that a tensor map cannot describe (odd alignment, strides of 0 or below),
// packed into the workspace: [n][hkv][D], keys then values.
template <int D>
__global__ void __launch_bounds__(256) pack_rows_kernel(const __grid_constant__ PagedChunkParams p, uint8_t* to) {
  grid_dep_wait();
  const int64_t chunks = static_cast<int64_t>(p.n) * p.hkv * (D / 8);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < 2 * chunks; i += static_cast<int64_t>(gridDim.x) * 256) {
    const PagedRows& x = i < chunks ? p.k : p.v;
    const int64_t k = i < chunks ? i : i - chunks, row = k / (D / 8);
    const int c = static_cast<int>(k % (D / 8)), head = static_cast<int>(row % p.hkv);
    const uint16_t* src = reinterpret_cast<const uint16_t*>(x.data) + row / p.hkv * x.token_stride + head * x.head_stride + 8 * c;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (rows_ok(x, src, 16, p.pool.err)) rows::load8(src, p.kv_vec, v);
    uint4* dst = reinterpret_cast<uint4*>(to) + i;
    if (in_range(dst, 16, p.ws, p.ws_hi, p.pool.err)) *dst = v;
  }
}

// Joins the pieces of the items that several CTAs shared: block (i, y) takes 32
// rows of the item whose first piece is CTA i's.
template <typename T, int D>
__global__ void __launch_bounds__(256) paged_chunk_join_kernel(const __grid_constant__ Launch a) {
  grid_dep_wait();
  const PagedChunkParams& p = a.p;
  const Note* notes = reinterpret_cast<const Note*>(p.ws);
  const Note n = notes[blockIdx.x];
  const int r = blockIdx.y * 32 + (threadIdx.x & 31), c0 = (threadIdx.x >> 5) * (D / 8);
  if (n.rows <= 0 || r >= n.rows || r >= a.slot_rows) return;
  const float* parts = reinterpret_cast<const float*>(p.ws + a.partials);
  const int64_t size = static_cast<int64_t>(a.slot_rows) * (D + 2);
  int last = blockIdx.x;
  while (last + 1 < a.grid) {
    const int c = notes[last + 1].cont;
    if (c != 1 && c != 2) break;
    ++last;
    if (c == 2) break;
  }
  const auto piece = [&](int i) { return parts + size * (2 * i + (i == static_cast<int>(blockIdx.x))); };
  float top = -INFINITY;
  for (int i = blockIdx.x; i <= last; ++i) top = fmaxf(top, piece(i)[r]);
  float o[D / 8], l = 0.0f;
#pragma unroll
  for (int c = 0; c < D / 8; ++c) o[c] = 0.0f;
  for (int i = blockIdx.x; i <= last; ++i) {
    const float* x = piece(i);
    const float li = x[a.slot_rows + r];
    if (li == 0.0f) continue;  // nothing that the row sees
    const float w = top == -INFINITY ? 1.0f : ex2(x[r] - top);
    l = fmaf(li, w, l);
    const float4* y = reinterpret_cast<const float4*>(x + 2 * a.slot_rows) + r;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      const float4 v = y[(c0 / 4 + c) * a.slot_rows];
      o[4 * c] = fmaf(v.x, w, o[4 * c]);
      o[4 * c + 1] = fmaf(v.y, w, o[4 * c + 1]);
      o[4 * c + 2] = fmaf(v.z, w, o[4 * c + 2]);
      o[4 * c + 3] = fmaf(v.w, w, o[4 * c + 3]);
    }
  }
  const int tk = (n.rem + r) / p.gqa, head = n.kvh * p.gqa + n.rem + r - tk * p.gqa;
  const int64_t row = static_cast<int64_t>(n.row) + tk;
  if (n.row < 0 || row >= p.n || head < 0 || head >= p.hkv * p.gqa) return;
  const int64_t at = row * p.hkv * p.gqa + head;
  const float inv = 1.0f / l;
  T* const type = nullptr;
  uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<T*>(p.out) + at * D + c0);
#pragma unroll
  for (int c = 0; c < D / 8; c += 2)
    dst[c / 2] = l == 0.0f ? 0u : pack2(type, o[c] * inv, o[c + 1] * inv);
  if (p.lse && c0 == 0) p.lse[at] = l == 0.0f ? -INFINITY : ((top - Fmt<T>::room) + log2f(l)) * 0.69314718055994531f;
}

}  // namespace chunk
}  // namespace kvq
