// Paged cache: attention of one query token per sequence, split over the
// cache's length and joined.
//
// Mathematics.  For the up to 8 query heads of a kv head, with t = scale
// log2(e) q.k, running maximum m and l = sum 2^(t - m), o = sum 2^(t - m) v.
// A key k = s c + z (c its codes) gives q.k = s (q.c) + z sum(q), a value row
// p v = (p s) c + p z, whose second part is the same for every channel: the codes
// go into the tensor cores as they are, the scales and zeros are one multiply-add
// per (token, head).  Weights go in as two 16-bit numbers, so that what is left
// of them, 22 bits (16 in bf16), is no less than the sums keep.
//
// Bound.  Every cached byte is read once; 2 * 8 heads * D products per token
// and kv head are far below the tensor rate, so the floor is the copy rate,
// and what competes with it is the issue rate (unpacking, softmax).
//
// Work split.  A chunk is S tiles of 16 tokens of one unit, a (sequence, kv
// head).  The chunks of all units in a row, with a few void places ahead of
// each unit for what starting it costs, are cut into equal ranges, one per CTA
// of one wave, so that neither many short sequences nor one long one leaves
// CTAs idle.  The four warps of a CTA take its chunks in turn, each with a ring
// of NST stages in shared memory that one bulk copy a page fills, and meet at
// the end of a unit to merge.  A unit that lies in one range is written by its
// CTA; one that several share leaves partial results, which a second kernel
// (a programmatic dependent, resident when the first drains) joins in a fixed
// order.  Nothing is counted across CTAs, so the workspace needs no clearing.
// Short tables are not split (see attn_as).
//
// Layout.  Products are taken transposed: keys are the 16 rows of an MMA and
// query heads its 8 columns, so that 8 heads fill it.  The score fragment,
// packed to 16 bits and transposed by movmatrix, is the P fragment of the
// second product, whose rows are channels.  The channel order inside each
// product is free: a thread takes the channels that its own bytes hold, and q
// is loaded in the same order.  Codes are taken as fp16 subnormals (code *
// 2^-24 * 2^field): exact, one AND for two codes; a key field's power of two is
// taken out of q, a value field's out of the result.  The tensor cores align
// sums by the exponent field, so that a sum of subnormals keeps fewer bits the
// lower the field; fields are therefore moved to bit 4 or higher first (one
// more shift for four codes).  At bits 0 .. 3 the scores of 4-bit keys were
// 8.5e-6 off (rms) instead of 1.4e-6, and those of 2-bit keys over 1e-5 of a
// short sequence's; the shifts cost 2 us of 42 (with weights in one part).
//
// Measured (GB300, device time with the join, copy rate 6771 GB/s): 8 x 32K
// tokens x 8 kv heads in fp16 121 us, 95% of the copy rate; K4V2 48 us, 48%;
// 16 x 4K x 8 in bf16 39 us, 76%, K8V4 22 us, 52%; one sequence of 256 tokens
// 5 us.  About 9 us of each are the way to the first chunk (lengths, page
// table, first copies: 3 dependent loads, 4.7 us), the uneven end of the CTAs
// (2 to 4 us) and the join (3 us).  In between 16-bit rows stream at the copy
// rate; narrow codes are bound by latency, at the 12 warps an SM that their
// registers leave: K4V2 issues 240 instructions a tile, 100 of them the masks,
// shifts and byte permutes that make registers of two codes, in 51% of the
// issue slots, with the ALU pipe 41% and the tensor cores 34% busy.
#pragma once

#include <cfloat>
#include <climits>
#include <type_traits>

#include "kvq_paged.cuh"

namespace kvq {
namespace paged {

// A running maximum m is kept kRoom below the greatest score that it was taken
// from, and follows only scores kLazy above itself.  So rescaling is rare (2^8
// past the last one), weights 2^(t - m) stay below 2^15, and in fp16, whose
// steps end at 2^-24, the greatest has kRoom more bits below it than it would at
// 1: there a weight under 2^-25 of the greatest would be 0 in the product with the
// values, yet counted in the sum, so that up to 2^-25 of the output for every such token
// were lost.
constexpr float kRoom = 7.0f, kLazy = kRoom + 8.0f;

constexpr int kMostCtas = 3;  // of an SM, in any shape: the workspace has room for their partial results

template <int KB, int VB, int D>
struct Shape {
  static constexpr bool quant = KB != 16;
  static constexpr int TB = paged_tile_bytes(D, KB, VB);
  // Tiles of a chunk, and CTAs per SM.  Codes: a chunk costs about 50
  // instructions beside its tiles (wait, maximum, next copy), so larger chunks
  // on 12 warps an SM beat smaller ones on 16 (K4V2, 8 x 32K tokens: 4 tiles on
  // 3 CTAs 48.3 us, 2 on 3 50.5, 2 on 4 53.8; K8V4, 16 x 4K: 2 tiles on 3 CTAs
  // 21.7 us, on 2 22.5; K8V8, 32 sequences of up to 8K, window 4096: 2 tiles on 2
  // CTAs 29.7 us, 1 on 3 32.2).  16 bits: one tile, and two CTAs, whose rings
  // have room for three tiles (head_dim 128) or four (64: fp16, 4 x 16K tokens x
  // 2 kv heads, 17.9 us on 2, 24.2 on 3, 27.4 on 4; 16 x 32K x 4, 66.4, 69.5, 67.7).
  static constexpr int S = !quant ? 1 : (TB > 1664 ? 2 : 4);  // tiles of a chunk
  static constexpr int stage = S * TB;
  static constexpr int W = 4;  // warps
  static constexpr int threads = 32 * W;
  // What starting another unit costs a CTA (the merge, the drained pipeline), in
  // chunks: a unit counts that many more when the work is cut.  (Measured 1.2 us
  // with 16 bits, 1.6 with K8V4, 2.9 with K4V2; 2 W was the best of 0, W, 2 W,
  // 3 W for all three: K8V4, 16 x 4K tokens, then 21.7, 21.2, 20.8, 20.7 us.)
  static constexpr int E = 2 * W;
  static constexpr int CPS = quant && TB <= 3200 ? 3 : 2;
  static_assert(CPS <= kMostCtas, "workspace");
  static constexpr int merge = (W - 1) * 32 * D;            // what each warp hands the others (D/4 fp32 a lane)
  static constexpr int queries = (quant ? 3 : 2) * 16 * D;  // rows of 8 heads (see fetch_q)
  static constexpr int extra = 1024;             // barriers, maxima and sums, q's factors, the search's sums
  static constexpr int head = extra + merge + queries;
  static constexpr int ring = ((228 / CPS - 1) * 1024 - head) / W;
  static constexpr int NST = ring / stage > 4 ? 4 : ring / stage;
  static constexpr int smem = head + W * NST * stage;
  static_assert(NST >= (quant ? 2 : 3), "ring");
};

// One partial result in the workspace: {m, l} of 8 heads, then the result in
// fragment order (register, lane).
__host__ __device__ constexpr int partial_floats(int D) { return 16 + 8 * D; }

struct Meta {     // start of the workspace: what the join needs of unit u
  int32_t first;  // first CTA of the unit
  int32_t count;  // CTAs that share it, 0: written already
  int32_t second; // 1: the first CTA's part is its second slot
  int32_t pad;
};

// One unit's part of a CTA's range.  A unit is `E` void places, which stand for
// what starting it costs, then its chunks lo .. hi - 1.
struct Seg {
  int b, h;
  int len, first;  // tokens attended: [first, len)
  int lo, hi;      // chunks of the unit
  int cbase;       // chunk at the range's i-th place: cbase + i (void below lo)
  int i0, i1;      // the range's places [i0, i1)
};

__device__ __forceinline__ int seq_len(const PagedAttnParams& p, int b) {
  const int room = p.batch.max_pages << p.pool.page_shift;
  const int len = __ldg(p.batch.lens + b);
  return len < 0 ? 0 : (len > room ? room : len);
}
__device__ __forceinline__ int seq_first(const PagedAttnParams& p, int len) {
  return p.window > 0 && len > p.window ? len - p.window : 0;
}
// Places of a unit with `len` tokens.
template <int S, int E>
__device__ __forceinline__ int place_count(const PagedAttnParams& p, int len) {
  return len ? E + (len + 16 * S - 1) / (16 * S) - seq_first(p, len) / (16 * S) : 0;  // (below 2^31, see open_call)
}

template <int S, int E>
__device__ __forceinline__ void seg_at(const PagedAttnParams& p, Seg& s, int len, int i0, int skip, int range) {
  s.len = len;
  s.first = seq_first(p, s.len);
  s.lo = s.first / (16 * S);
  s.hi = (s.len + 16 * S - 1) / (16 * S);
  s.i0 = i0;
  s.cbase = s.lo - E + skip - i0;
  const int left = s.hi - s.lo + E - skip;
  s.i1 = left < range - i0 ? i0 + left : range;
}
// The unit after s; there is one while s.i1 < range.  (Where there is none,
// because the lengths change under the call, the rest of the range is void.)
// WARP: a whole warp calls it, and takes the lengths that its first lane read.
template <int S, int E, bool WARP>
__device__ __forceinline__ void seg_next(const PagedAttnParams& p, Seg& s, int range) {
  const int i0 = s.i1;
  int len = s.len;
  if (++s.h == p.hkv) {
    s.h = 0;
    len = 0;
    while (len == 0 && ++s.b < p.batch.seqs) {
      len = seq_len(p, s.b);
      if (WARP) len = __shfl_sync(0xffffffffu, len, 0);
    }
    if (len == 0) {
      s = Seg{0, 0, 0, 0, INT_MAX / 2, INT_MAX / 2, 0, i0, range};
      return;
    }
  }
  seg_at<S, E>(p, s, len, i0, 0, range);
}

// D = A(16x16) B(16x8) + D.  Not volatile: the compiler may interleave chains.
template <typename T>
__device__ __forceinline__ void mma_t(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  } else {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
}

__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (std::is_same<T, __half>::value) return h2_as_u32(__floats2half2_rn(lo, hi));
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// bulk_g2s with the destination as a shared-memory address
__device__ __forceinline__ void bulk_g2s_at(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// Debug builds: row `row` of the output, and one partial result, lie in their buffers.
template <typename T>
__device__ __forceinline__ bool out_ok(const PagedAttnParams& p, int64_t row, int D) {
  const T* out = reinterpret_cast<const T*>(p.out);
  const int64_t rows = static_cast<int64_t>(p.batch.seqs) * p.hkv * p.gqa;
  return in_range(out + row * D, D * sizeof(T), out, out + rows * D, p.pool.err);
}
__device__ __forceinline__ bool part_ok(const PagedAttnParams& p, const float* part, int D) {
  return in_range(part, partial_floats(D) * 4, p.ws + p.ws_partials, p.ws_hi, p.pool.err);
}

// N words (1, 2 or 4) from shared memory in one load.
template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t* w) {
  if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

// ---------------------------------------------------------------- codes

// The thread column t of a key fragment owns D/4 channels: with 16-bit keys
// the MMA's own (16 j + 8 i + 2t, + 1 for register 2j + i), with codes the
// ones of its bytes, a run of D/4 (8 bits, D = 128: the runs of 16 channels at
// 16t and 16t + 64).  Of the run's channels, register r holds 2r and 2r + 1 with
// 8-bit codes, 8 (r / 4) + r % 4 and the fourth after it with 4-bit ones, 16 (r / 8) + r % 8
// and the eighth after it with 2-bit ones (what split_codes leaves in its halves).
// log2 of the power of two that the field of key register (value channel) r carries
template <int B>
__host__ __device__ constexpr int code_field(int r) {
  constexpr int two[8] = {4, 6, 4, 6, 8, 4, 6, 8};
  return B == 8 ? 0 : B == 4 ? 4 : two[r % 8];
}

// 32 bits of codes -> registers of two fp16 subnormals, one from each half.
template <int B>
__device__ __forceinline__ void split_codes(uint32_t x, uint32_t* r) {
  if (B == 4) {  // fields at bits 4 .. 7
    const uint32_t u = x >> 8;
    r[0] = (x << 4) & 0x00f000f0u;
    r[1] = x & 0x00f000f0u;
    r[2] = (u << 4) & 0x00f000f0u;
    r[3] = u & 0x00f000f0u;
  } else {  // fields at bits 4, 6 and 8
    const uint32_t y = x << 4, u = x >> 6;
    r[0] = y & 0x00300030u;
    r[1] = y & 0x00c000c0u;
    r[2] = x & 0x00300030u;
    r[3] = x & 0x00c000c0u;
    r[4] = x & 0x03000300u;
    r[5] = u & 0x00300030u;
    r[6] = u & 0x00c000c0u;
    r[7] = u & 0x03000300u;
  }
}
// A word of a key row; two tokens' 16 bits of value codes (low half one token,
// high half the other).
template <int B>
__device__ __forceinline__ void key_regs(uint32_t w, uint32_t* r) {
  if constexpr (B == 8) {
    r[0] = prmt(w, 0, 0x4140);
    r[1] = prmt(w, 0, 0x4342);
  } else {
    split_codes<B>(w, r);
  }
}
template <int B>
__device__ __forceinline__ void val_regs(uint32_t x, uint32_t* r) {
  if constexpr (B == 8) {
    r[0] = prmt(x, 0, 0x4240);
    r[1] = prmt(x, 0, 0x4341);
  } else {
    split_codes<B>(x, r);
  }
}

// ---------------------------------------------------------------- the kernel

template <typename T, int KB, int VB, int D>
__global__ void __launch_bounds__(Shape<KB, VB, D>::threads, Shape<KB, VB, D>::CPS) attn_kernel(PagedAttnParams p) {
  using C = Shape<KB, VB, D>;
  constexpr int S = C::S, E = C::E, kWarps = C::W, kThreads = C::threads;
  constexpr int NR = D / 8;   // key fragment registers of a thread, per row
  constexpr int MT = D / 16;  // m-tiles of 16 channels
  constexpr int QT = MT / C::W;  // of which a warp finishes
  using W = typename std::conditional<C::quant, __half, T>::type;  // of weights in the second product
  extern __shared__ __align__(128) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem);           // [warps][NST]
  float* ml = reinterpret_cast<float*>(smem + 256);             // [warps][m 8, l 8]
  int64_t* sums = reinterpret_cast<int64_t*>(smem + 768);       // [2][warps] of the search
  // This unit's part and the next one's.  One thread reads the lengths for all:
  // warps that read them for themselves, while something changed them, could
  // differ on how often they meet.
  Seg* segs = reinterpret_cast<Seg*>(smem + 896);
  float2* qstat = reinterpret_cast<float2*>(smem + 512);        // [2][8 heads]: fac, qs (below)
  float4* mergebuf = reinterpret_cast<float4*>(smem + C::extra);  // [warps][warps - 1][QT][32]
  // 16 bits: q rows [2][8][D].  Codes: rows as they come [8][D], then their
  // fragments [2][NR / 4][32 lanes][4 registers]
  uint8_t* const qbuf = smem + C::extra + C::merge;
  uint32_t* const qfrag = reinterpret_cast<uint32_t*>(qbuf + 16 * D);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + C::head + warp * C::NST * C::stage;
  uint64_t* bar = bars + warp * C::NST;

  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < C::NST; ++i) mbar_init(bar + i, 1);
    fence_mbar_init();
  }
  if constexpr (C::quant) {  // fragments of the heads that there are not stay 0
    for (int x = threadIdx.x; x < 8 * D; x += kThreads) qfrag[x] = 0;
    if (threadIdx.x < 16) qstat[threadIdx.x] = make_float2(0.0f, 0.0f);
  }
  grid_dep_wait();
  grid_dep_launch();

  Seg cs;
  int64_t per = 0, r0 = 0;
  int range = 0;
  if (p.solo) {
    // one CTA for each unit: no search, and nothing to join
    if (threadIdx.x == 0) {
      cs.b = blockIdx.x / p.hkv;
      cs.h = blockIdx.x - cs.b * p.hkv;
      const int len = seq_len(p, cs.b);
      if (len != __ldg(p.batch.lens + cs.b)) atomicExch(p.pool.err, kErrBadState);
      seg_at<S, E>(p, cs, len, 0, 0, INT_MAX);
      segs[0] = cs;
    }
    __syncthreads();
    cs = segs[0];
    if (cs.len == 0) {
      const int64_t row = static_cast<int64_t>(blockIdx.x) * p.gqa;
      if (!out_ok<T>(p, row, D) || !out_ok<T>(p, row + p.gqa - 1, D)) return;
      for (int x = threadIdx.x; x < p.gqa * D; x += kThreads) reinterpret_cast<T*>(p.out)[row * D + x] = Num<T>::from(0.0f);
      if (p.lse && threadIdx.x < p.gqa) p.lse[row + threadIdx.x] = -INFINITY;
      return;
    }
    range = cs.i1;
  } else {
    // ---- the CTA's range of places, and the unit it starts in: prefix sums of
    // the sequences' places, 128 sequences at a time
    const int B = p.batch.seqs;
    // the page table on its way into L2 while the lengths are: a small one whole
    {
      const int64_t lines = (static_cast<int64_t>(B - 1) * p.batch.table_stride + p.batch.max_pages + 31) / 32;
      const int line = blockIdx.x * kThreads + threadIdx.x;
      if (lines <= 2048 && line < lines)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(p.batch.table + 32 * line));
    }
    int len = 0;  // of the sequence looked at last
    auto chunks_of = [&](int b) {
      if (b >= B) return static_cast<int64_t>(0);
      len = seq_len(p, b);
      if (blockIdx.x == 0 && __ldg(p.batch.lens + b) != len) atomicExch(p.pool.err, kErrBadState);
      return static_cast<int64_t>(place_count<S, E>(p, len)) * p.hkv;
    };
    int64_t total = 0;
    for (int b0 = kThreads; b0 < B; b0 += kThreads) total += chunks_of(b0 + threadIdx.x);  // but the first 128
    int64_t held = chunks_of(threadIdx.x), incl = held;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (B > kThreads) {
#pragma unroll
      for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    }
    if (lane == 31) {
      sums[warp] = incl;
      sums[kWarps + warp] = total;
    }
    __syncthreads();
    int64_t before = 0;  // places of the sequences looked at so far
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      total += sums[w] + sums[kWarps + w];
      before += sums[w];
      if (w < warp) incl += sums[w];
    }
    per = total + gridDim.x - 1;
    per = per >> 32 ? per / gridDim.x : static_cast<uint32_t>(per) / gridDim.x;  // (64 bits cost over 100 instructions)
    if (per < kWarps) per = kWarps;
    r0 = per * blockIdx.x;
    if (r0 >= total) return;  // the same for every thread
    range = static_cast<int>(total - r0 < per ? total - r0 : per);
    for (int b0 = 0;;) {
      const int64_t at = incl - held;
      if (r0 >= at && r0 < incl) {
        const int64_t n = held / p.hkv, off = r0 - at;
        cs.b = b0 + threadIdx.x;
        cs.h = static_cast<int>(off / n);
        seg_at<S, E>(p, cs, len, 0, static_cast<int>(off % n), range);
        segs[0] = cs;
        if (cs.i1 < range) seg_next<S, E, false>(p, cs, range);
        segs[1] = cs;
      }
      __syncthreads();
      if (r0 < before) break;
      b0 += kThreads;
      if (b0 >= B) {  // the lengths change under the call
        if (threadIdx.x == 0) atomicExch(p.pool.err, kErrBadState);
        return;
      }
      held = incl = chunks_of(b0 + threadIdx.x);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      if (lane == 31) sums[warp] = incl;
      __syncthreads();
      incl += before;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        before += sums[w];
        if (w < warp) incl += sums[w];
      }
    }
    cs = segs[0];
  }
  Seg ns = segs[1];  // (of no meaning where cs is the range's last)

  // ---- q rows of a unit into shared memory: asked for ahead of the copies of
  // its chunks (behind them, the first came 3 us late), of the next unit while
  // this one is worked on.  A thread takes 16 bytes, 8 channels of a head.
  constexpr int RC = D / 8;  // 16-byte chunks of a row
  static_assert(8 * RC <= kThreads, "one chunk a thread");
  const int qhead = threadIdx.x / RC, qchunk = threadIdx.x % RC;
  uint8_t* const qraw = qbuf + threadIdx.x * 16;
  auto fetch_q = [&](const Seg& u, int which) {
    if (qhead >= p.gqa) return;
    const T* src = reinterpret_cast<const T*>(p.q.data) + u.b * p.q.token_stride +
                   (u.h * p.gqa + qhead) * p.q.head_stride + qchunk * 8;
    if (!rows_ok(p.q, src, 16, p.pool.err)) return;
    uint8_t* dst = qraw + (C::quant ? 0 : which * 16 * D);
    if (p.q_vec) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
    } else {
      T v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = src[i];
      *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(v);
    }
  };
  // Codes: the thread's 8 channels, which it fetched itself, into the order of
  // the key fragments.  A power of two takes the row's largest |q|, with the
  // fields' least power off it, to [2^15, 2^16), where 11 bits still fit fp16.
  // What fp16's steps of 2^-24 cut off is then at most 2^-40 of the row's largest for 8- and
  // 4-bit keys and 2^-36 for 2-bit ones, whose fields differ by up to 2^4: a bf16
  // q is exact down to 2^-32 (2^-28) of it.
  auto make_frags = [&](int which) {
    float x[8], mx = 0.0f, sum = 0.0f;
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (qhead < p.gqa) raw = *reinterpret_cast<const uint4*>(qraw);
    const T* v = reinterpret_cast<const T*>(&raw);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = Num<T>::to(v[i]);
      mx = fmaxf(mx, fabsf(x[i]));
      sum += x[i];
    }
#pragma unroll
    for (int o = 1; o < RC; o <<= 1) {
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    if (qhead >= p.gqa) return;
    int e = static_cast<int>(__float_as_uint(mx) >> 23) - 127;  // mx in [2^e, 2^(e+1))
    constexpr int top = 15 + code_field<KB>(0);  // (register 0 has the lowest field)
    e = mx < 1e-30f ? top : (e > 100 ? 100 : e);
    const float up = __uint_as_float(static_cast<uint32_t>(127 + top - e) << 23);
    const float down = __uint_as_float(static_cast<uint32_t>(127 - top + e) << 23);
    // channel 8 qchunk + i: thread column, register and half (see codes, above)
    constexpr bool two_runs = KB == 8 && D == 128;
    const int col = two_runs ? qchunk / 2 % 4 : qchunk / (RC / 4);
    const int in_run = two_runs ? 16 * (qchunk / 8) + 8 * (qchunk % 2) : 8 * (qchunk % (RC / 4));
    uint32_t* const f = qfrag + which * 4 * D + (qhead * 4 + col) * 4;  // register r at f[r / 4 * 128 + r % 4]
    if constexpr (KB == 2) {  // registers 0 .. 7 of 16 channels, one half each
      __half* h = reinterpret_cast<__half*>(f + in_run / 16 * 256) + in_run / 8 % 2;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        h[i / 4 * 256 + i % 4 * 2] = __float2half_rn(x[i] * (up * (1.0f / (1 << code_field<KB>(i)))));
    } else {
      uint32_t r[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = x[KB == 8 ? 2 * i : i], b = x[KB == 8 ? 2 * i + 1 : i + 4];
        const float u = up * (1.0f / (1 << code_field<KB>(i)));
        r[i] = h2_as_u32(__floats2half2_rn(a * u, b * u));
      }
      *reinterpret_cast<uint4*>(f + in_run / 8 * 128) = make_uint4(r[0], r[1], r[2], r[3]);
    }
    // score = fac s acc + qs z
    if (qchunk == 0) qstat[which * 8 + qhead] = make_float2(p.alpha * down * 16777216.0f, p.alpha * sum);
  };
  fetch_q(cs, 0);

  // ---- the producer's side of the ring: the addresses of the warp's next
  // copies are worked out one a lane, 32 / ppc chunks at a time (one alone
  // costs as many instructions as all of them); chunk `ip` is the next to copy.
  // The warp reads the lengths for itself here, ahead of thread 0 (segs).  Should
  // something change them in between, the two sides differ on the places, so
  // that a wait is for a copy that was started, whichever place it was for,
  // and all of them are waited for at the end.
  Seg ps = cs;
  // Copies started and not waited for yet; -1 less that many once a wait gave
  // up or had none to wait for: nothing more is copied or computed then.
  int flight = 0;
  const int tiles_page = 1 << (p.pool.page_shift - 4);
  const int ppc = S > tiles_page ? S / tiles_page : 1;  // pages of a chunk
  const int nb = 32 / ppc, mine = lane / ppc, piece = lane % ppc;
  int ip = warp, nxt = 0;
  const uint8_t* src = nullptr;
  uint32_t bytes = 0, chunk_bytes = 0, voids = 0;
  uint32_t dst = smem_u32(ring) + piece * tiles_page * C::TB;
  auto fill = [&]() {
    nxt = 0;
    bytes = 0;
    bool is_void = false;
    const int idx = ip + mine * kWarps;
    const int last = ip + (nb - 1) * kWarps < range ? ip + (nb - 1) * kWarps : range - 1;
    for (;;) {
      if (idx >= ps.i0 && idx < ps.i1 && ps.cbase + idx < ps.lo) {
        is_void = true;
      } else if (idx >= ps.i0 && idx < ps.i1) {
        const int tok0 = (ps.cbase + idx) * (16 * S);
        const int left = (ps.len - tok0 + 15) >> 4;
        const int ntiles = left < S ? left : S;
        const int skip = piece * tiles_page;  // tiles of the chunk before this piece
        int n = ntiles - skip;
        n = n < 0 ? 0 : (ppc > 1 && n > tiles_page ? tiles_page : n);
        chunk_bytes = static_cast<uint32_t>(ntiles * C::TB);
        bytes = static_cast<uint32_t>(n * C::TB);
        if (n > 0) {
          const int e = (tok0 >> p.pool.page_shift) + piece;
          // a page wholly before the window is masked, and its entry may be gone
          const int32_t* entry = p.batch.table + ps.b * p.batch.table_stride + e;
          int page = ((e + 1) << p.pool.page_shift) <= ps.first || !table_ok(p.batch, entry, p.pool.err) ? 0 : __ldg(entry);
          if (page < 0 || page >= p.pool.num_pages) {
            atomicExch(p.pool.err, kErrBadPage);
            page = 0;
          }
          src = p.pool.pages + page * p.pool.page_stride + ps.h * p.pool.head_stride +
                (ppc > 1 ? 0 : ((tok0 >> 4) & (tiles_page - 1)) * C::TB);
          if (!pool_ok(p.pool, src, bytes)) src = p.pool.pages;  // (a barrier counts on the bytes)
        }
      }
      if (last < ps.i1) break;
      seg_next<S, E, true>(p, ps, range);
    }
    voids = __ballot_sync(0xffffffffu, is_void);
  };
  auto issue = [&](int st) {
    for (;; ++nxt, ip += kWarps) {
      if (ip >= range) return;
      if (nxt == nb) fill();
      if (!(voids >> (nxt * ppc) & 1)) break;
    }
    const bool turn = mine == nxt;
    if (turn && piece == 0) mbar_arrive_expect_tx(bar + st, chunk_bytes);
    if (ppc > 1) __syncwarp();
    if (turn && bytes) bulk_g2s_at(dst + st * C::stage, src, bytes, bar + st);
    ++flight;
    ++nxt;
    ip += kWarps;
  };
  __syncwarp();
  if (ip < range) fill();
  for (int st = 0; st < C::NST; ++st) issue(st);
  asm volatile("cp.async.wait_all;" ::: "memory");
  if constexpr (C::quant) make_frags(0);

  // ---- where the thread reads in a tile.  Quantized: key rows g and g + 8 (the
  // second eight rows lie 8 rows on, with the same XOR), value tokens t, t + 4,
  // t + 8, t + 12 (alike).  16 bits: its ldmatrix row and chunk.
  constexpr int rk = D * KB / 8, rv = D * VB / 8, CB = rv / 8;
  constexpr int off_v = 16 * rk, off_sz = 16 * (rk + rv);
  const int koff = C::quant ? g * rk + ((rk / 4 >= 16 ? 16 * t : rk / 4 * t) ^ tile_key_xor(rk, g)) : 0;
  const int voff = C::quant ? off_v + t * rv + ((CB * g) ^ tile_val_xor(rv, t)) : 0;
  const int soff = off_sz + 8 * g;

  int ic = warp, st = 0, which = 0;
  uint32_t phase = 0;

  for (;;) {
    // ---- q of the unit, in the order of the key fragments
    __syncthreads();
    if (cs.i1 < range) {
      fetch_q(ns, which ^ 1);
      if (threadIdx.x == 0) {  // the unit after the next
        Seg after = ns;
        if (ns.i1 < range) seg_next<S, E, false>(p, after, range);
        segs[1] = after;
      }
    }
    uint32_t qf[NR];
    float fac[2], qs[2];  // of heads 2t, 2t + 1: score = fac s acc + qs z (codes), fac acc (16 bits)
    if constexpr (!C::quant) {
      const T* q = reinterpret_cast<const T*>(qbuf) + (which * 8 + g) * D;
#pragma unroll
      for (int r = 0; r < NR; ++r) qf[r] = g < p.gqa ? *reinterpret_cast<const uint32_t*>(q + 8 * r + 2 * t) : 0u;
      fac[0] = fac[1] = p.alpha;
      qs[0] = qs[1] = 0.0f;
    } else {
#pragma unroll
      for (int r = 0; r < NR; r += 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(qfrag + which * 4 * D + r / 4 * 128 + lane * 4);
        qf[r] = v.x, qf[r + 1] = v.y, qf[r + 2] = v.z, qf[r + 3] = v.w;
      }
#pragma unroll
      for (int hd = 0; hd < 2; ++hd) {
        const float2 v = qstat[which * 8 + 2 * t + hd];
        fac[hd] = v.x, qs[hd] = v.y;
      }
    }
    which ^= 1;
    // (the maximum begins at a number: from -infinity, scores that are all
    // -infinity would get weights of NaN instead of 0)
    float o[MT][4], m[2] = {-FLT_MAX, -FLT_MAX}, l[2] = {0.0f, 0.0f}, zs[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[j][i] = 0.0f;

    for (; ic < cs.i1; ic += kWarps) {
      if (flight < 0 || cs.cbase + ic < cs.lo) continue;
      if (flight == 0) {  // the lengths change under the call
        if (lane == 0) atomicExch(p.pool.err, kErrBadState);
        flight = -1;
        continue;
      }
      if (__any_sync(0xffffffffu, !mbar_wait(bar + st, phase, p.pool.err))) {
        flight = -1 - flight;
        continue;
      }
      --flight;
      uint8_t* buf = ring + st * C::stage;
      const int base = (cs.cbase + ic) * (16 * S);
      const bool edge = base < cs.first || base + 16 * S > cs.len;
      float sc[S][4];  // scores of (row g, heads 2t, 2t+1), (row g + 8, the same)
      float vs[S][2], vz[S][2];  // value scales and zeros of the two rows

      if constexpr (!C::quant) {
        const int r = (lane & 7) + ((lane >> 3) & 1) * 8, c = lane >> 4;
#pragma unroll
        for (int s = 0; s < S; ++s) {
          float acc[2][4] = {};
          const uint8_t* row = buf + s * C::TB + r * 2 * D;
#pragma unroll
          for (int j = 0; j < MT; ++j) {
            uint32_t a[4];
            ldsm_x4(a, row + 16 * tile_chunk16(2 * j + c, r));
            mma_t<T>(acc[j & 1], a[0], a[1], a[2], a[3], qf[2 * j], qf[2 * j + 1]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) sc[s][i] = (acc[0][i] + acc[1][i]) * p.alpha;
        }
        if (edge) {
          // rows outside [first, len) may hold anything: no score, and values set to 0
#pragma unroll
          for (int s = 0; s < S; ++s) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int tok = base + 16 * s + g + 8 * (i >> 1);
              if (tok < cs.first || tok >= cs.len) sc[s][i] = -INFINITY;
            }
            for (int x = lane; x < 16 * (D / 8); x += 32) {
              const int tok = base + 16 * s + x / (D / 8);
              if (tok < cs.first || tok >= cs.len)
                *reinterpret_cast<uint4*>(buf + s * C::TB + 32 * D + 16 * x) = make_uint4(0, 0, 0, 0);
            }
          }
          __syncwarp();
          fence_proxy_async_smem();  // the next copy into this stage comes after these stores
        }
      } else {
        // the words of rows g and g + 8, then the products word by word with the
        // tiles inside, so that their S chains of dependent MMAs interleave
        constexpr int NW = rk / 16;  // words of a thread's part of a row
        constexpr int R = 16 / KB;   // registers of a word
        uint32_t wa[S][NW], wb[S][NW];
        // Two sums for 8-bit keys: an MMA cuts each product at its sum's last bit, and theirs (19 bits) are
        // longer than those of fewer bits.  In one sum the log-sum-exp of one token was 1.2e-6 off, in two 7e-7,
        // as far as that of 4-bit keys in one (K8V4, 16 x 4K tokens, 22.4 instead of 22.2 us).
        constexpr int CH = KB == 8 ? 2 : 1;
        float acc[S][CH][4] = {};
#pragma unroll
        for (int s = 0; s < S; ++s) {
          const uint8_t* kp = buf + s * C::TB + koff;
          load_words<(NW < 4 ? NW : 4)>(kp, wa[s]);
          load_words<(NW < 4 ? NW : 4)>(kp + 8 * rk, wb[s]);
          if constexpr (NW == 8) {
            const uint8_t* kq = buf + s * C::TB + (koff ^ 64);
            load_words<4>(kq, wa[s] + 4);
            load_words<4>(kq + 8 * rk, wb[s] + 4);
          }
        }
#pragma unroll
        for (int w = 0; w < NW; ++w)
#pragma unroll
          for (int s = 0; s < S; ++s) {
            uint32_t x[R], y[R];
            key_regs<KB>(wa[s][w], x);
            key_regs<KB>(wb[s][w], y);
#pragma unroll
            for (int j = 0; j < R; j += 2)
              mma_t<__half>(acc[s][w % CH], x[j], y[j], x[j + 1], y[j + 1], qf[w * R + j], qf[w * R + j + 1]);
          }
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint2 raw = *reinterpret_cast<const uint2*>(buf + s * C::TB + soff + 64 * i);
            const float ks = __low2float(u32_as_h2(raw.x)), kz = __high2float(u32_as_h2(raw.x));
            vs[s][i] = __low2float(u32_as_h2(raw.y));
            vz[s][i] = __high2float(u32_as_h2(raw.y));
#pragma unroll
            for (int hd = 0; hd < 2; ++hd)
              sc[s][2 * i + hd] =
                  fmaf(ks * fac[hd], CH == 1 ? acc[s][0][2 * i + hd] : acc[s][0][2 * i + hd] + acc[s][CH - 1][2 * i + hd],
                       kz * qs[hd]);
          }
        if (edge) {  // rows outside [first, len) may hold anything
          const int lo = cs.first - base - tile_row_token(g), hi = cs.len - base - tile_row_token(g);
#pragma unroll
          for (int s = 0; s < S; ++s)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (16 * s + 8 * i < lo || 16 * s + 8 * i >= hi) {
                sc[s][2 * i] = sc[s][2 * i + 1] = -INFINITY;
                vs[s][i] = vz[s][i] = 0.0f;
              }
        }
      }

      // ---- running maximum.  For codes it is that of t + log2(s): what P holds
      // is 2^(t - m) s, which then stays in fp16's range whatever the scales are
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float lv = 0.0f;
          if constexpr (C::quant) lv = lg2(fmaxf(vs[s][i], 5.9604645e-8f));  // a scale of 0 counts as fp16's smallest
          mx[0] = fmaxf(mx[0], sc[s][2 * i] + lv);
          mx[1] = fmaxf(mx[1], sc[s][2 * i + 1] + lv);
        }
      if (__any_sync(0xffffffffu, mx[0] > m[0] + kLazy || mx[1] > m[1] + kLazy)) {
#pragma unroll
        for (int hd = 0; hd < 2; ++hd) {
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) mx[hd] = fmaxf(mx[hd], __shfl_xor_sync(0xffffffffu, mx[hd], x));
          const float mn = fmaxf(m[hd], mx[hd] - kRoom);
          const float f = m[hd] == mn ? 1.0f : ex2(m[hd] - mn);
          m[hd] = mn;
          l[hd] *= f;
          zs[hd] *= f;
#pragma unroll
          for (int j = 0; j < MT; ++j) {
            o[j][hd] *= f;
            o[j][2 + hd] *= f;
          }
        }
      }

      // ---- probabilities, transposed into the second product's fragments
      // weights as two numbers of 16 bits, 22 (bf16: 16) bits of them together
      uint32_t pb[S][2], rest[S][2];
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float p0 = ex2(sc[s][2 * i] - m[0]), p1 = ex2(sc[s][2 * i + 1] - m[1]);
          l[0] += p0;
          l[1] += p1;
          float w0 = p0, w1 = p1;
          if constexpr (C::quant) {
            zs[0] = fmaf(p0, vz[s][i], zs[0]);
            zs[1] = fmaf(p1, vz[s][i], zs[1]);
            w0 *= vs[s][i];
            w1 *= vs[s][i];
          }
          const uint32_t hi = pack2<W>(w0, w1);
          const W* h = reinterpret_cast<const W*>(&hi);
          pb[s][i] = transpose8(hi);
          rest[s][i] = transpose8(pack2<W>(w0 - Num<W>::to(h[0]), w1 - Num<W>::to(h[1])));
        }

      // ---- the second product
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const uint8_t* tile = buf + s * C::TB;
        if constexpr (!C::quant) {
          const int r = (lane & 7) + (lane >> 4) * 8, c = (lane >> 3) & 1;
          const uint8_t* row = tile + 32 * D + r * 2 * D;
#pragma unroll
          for (int j = 0; j < MT; ++j) {
            uint32_t a[4];
            ldsm_x4_t(a, row + 16 * tile_chunk16(2 * j + c, r));
            mma_t<T>(o[j], a[0], a[1], a[2], a[3], pb[s][0], pb[s][1]);
            mma_t<T>(o[j], a[0], a[1], a[2], a[3], rest[s][0], rest[s][1]);
          }
        } else {
          // [pair (t, t+4) or (t+8, t+12)][channel of the thread]
          uint32_t v[2][NR];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint8_t* ra = tile + voff + 8 * h * rv;
            const uint8_t* rb = ra + 4 * rv;
            if constexpr (CB >= 4) {
              uint32_t ua[CB / 4], ub[CB / 4];
              load_words<CB / 4>(ra, ua);
              load_words<CB / 4>(rb, ub);
              constexpr int R = 16 / VB;  // channels of 16 bits
#pragma unroll
              for (int w = 0; w < CB / 4; ++w) {
                val_regs<VB>(prmt(ua[w], ub[w], 0x5410), v[h] + 2 * w * R);
                val_regs<VB>(prmt(ua[w], ub[w], 0x7632), v[h] + (2 * w + 1) * R);
              }
            } else {
              const uint32_t x = *reinterpret_cast<const uint16_t*>(ra) |
                                 static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(rb)) << 16;
              val_regs<VB>(x, v[h]);
            }
          }
#pragma unroll
          for (int j = 0; j < MT; ++j) {
            mma_t<__half>(o[j], v[0][2 * j], v[0][2 * j + 1], v[1][2 * j], v[1][2 * j + 1], pb[s][0], pb[s][1]);
            mma_t<__half>(o[j], v[0][2 * j], v[0][2 * j + 1], v[1][2 * j], v[1][2 * j + 1], rest[s][0], rest[s][1]);
          }
        }
      }
      __syncwarp();
      issue(st);
      if (++st == C::NST) {
        st = 0;
        phase ^= 1;
      }
    }

    if (cs.cbase + cs.i1 <= cs.lo) break;  // the range ends before the unit's first chunk
    // ---- the unit's end: every warp finishes MT / W of the m-tiles, from what
    // the others hand it, in a fixed order
    if (cs.i1 < range) {
      asm volatile("cp.async.wait_all;" ::: "memory");
      if constexpr (C::quant) make_frags(which);
    }
#pragma unroll
    for (int hd = 0; hd < 2; ++hd) {
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) {
        l[hd] += __shfl_xor_sync(0xffffffffu, l[hd], x);
        zs[hd] += __shfl_xor_sync(0xffffffffu, zs[hd], x);
      }
      if (g == 0) {
        ml[warp * 16 + 2 * t + hd] = m[hd];
        ml[warp * 16 + 8 + 2 * t + hd] = l[hd];
      }
    }
    float4 mine4[QT];
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
#pragma unroll
      for (int q = 0; q < QT; ++q) {
        const int j = w * QT + q;
        float4 v = make_float4(o[j][0], o[j][1], o[j][2], o[j][3]);
        if constexpr (C::quant) {  // the field's power of two, and what all channels share
          const float u0 = 16777216.0f / (1 << code_field<VB>(2 * j)), u1 = 16777216.0f / (1 << code_field<VB>(2 * j + 1));
          v = make_float4(fmaf(v.x, u0, zs[0]), fmaf(v.y, u0, zs[1]), fmaf(v.z, u1, zs[0]), fmaf(v.w, u1, zs[1]));
        }
        if (warp == w)
          mine4[q] = v;
        else
          mergebuf[((warp * (kWarps - 1) + (w < warp ? w : w - 1)) * QT + q) * 32 + lane] = v;
      }
    __syncthreads();
    float top[2] = {-INFINITY, -INFINITY}, sum[2] = {0.0f, 0.0f}, f[kWarps][2];
#pragma unroll
    for (int hd = 0; hd < 2; ++hd) {
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top[hd] = fmaxf(top[hd], ml[w * 16 + 2 * t + hd]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float lw = ml[w * 16 + 8 + 2 * t + hd];
        f[w][hd] = lw == 0.0f ? 0.0f : ex2(ml[w * 16 + 2 * t + hd] - top[hd]);
        sum[hd] = fmaf(lw, f[w][hd], sum[hd]);
      }
    }
    float4 r[QT];
#pragma unroll
    for (int q = 0; q < QT; ++q) {
      r[q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 v = w == warp ? mine4[q]
                                   : mergebuf[((w * (kWarps - 1) + (warp < w ? warp : warp - 1)) * QT + q) * 32 + lane];
        r[q] = make_float4(fmaf(v.x, f[w][0], r[q].x), fmaf(v.y, f[w][1], r[q].y), fmaf(v.z, f[w][0], r[q].z),
                           fmaf(v.w, f[w][1], r[q].w));
      }
    }
    {
      const int64_t unit = static_cast<int64_t>(cs.b) * p.hkv + cs.h;
      const bool starts = cs.cbase + cs.i0 <= cs.lo, ends = cs.cbase + cs.i1 == cs.hi;
      if (starts && !p.solo && threadIdx.x == 0) {
        const int64_t last = (r0 + cs.hi - 1 - cs.cbase) / per;  // the CTA of the unit's last chunk
        Meta meta = {static_cast<int32_t>(blockIdx.x), static_cast<int32_t>(ends ? 0 : last - blockIdx.x + 1),
                     cs.i0 > 0 ? 1 : 0, 0};
        uint8_t* note = p.ws + unit * sizeof(Meta);
        if (in_range(note, sizeof(Meta), p.ws, p.ws + p.ws_partials, p.pool.err))
          *reinterpret_cast<int4*>(note) = *reinterpret_cast<int4*>(&meta);
      }
      if (starts && ends) {
#pragma unroll
        for (int hd = 0; hd < 2; ++hd) {
          const int head = 2 * t + hd;
          if (head < p.gqa) {
            const int64_t row = unit * p.gqa + head;
            if (!out_ok<T>(p, row, D)) continue;
            const float inv = sum[hd] == 0.0f ? 0.0f : 1.0f / sum[hd];
            T* out = reinterpret_cast<T*>(p.out) + row * D;
#pragma unroll
            for (int q = 0; q < QT; ++q)
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                const int j = warp * QT + q;
                const int c = C::quant ? NR * g + 2 * j + half : 16 * j + 8 * half + g;
                out[c] = Num<T>::from((half ? (hd ? r[q].w : r[q].z) : (hd ? r[q].y : r[q].x)) * inv);
              }
            if (p.lse && g == 0 && warp == 0) p.lse[row] = (top[hd] + log2f(sum[hd])) * 0.693147180559945f;
          }
        }
      } else {
        float* part = reinterpret_cast<float*>(p.ws + p.ws_partials) +
                      (2 * static_cast<int64_t>(blockIdx.x) + (cs.i0 > 0 ? 1 : 0)) * partial_floats(D);
        const bool in = part_ok(p, part, D);
        if (in && g == 0 && warp == 0) {
#pragma unroll
          for (int hd = 0; hd < 2; ++hd) {
            part[2 * t + hd] = top[hd];
            part[8 + 2 * t + hd] = sum[hd];
          }
        }
        // [m-tile][lane][4]
#pragma unroll
        for (int q = 0; in && q < QT; ++q) *reinterpret_cast<float4*>(part + 16 + ((warp * QT + q) * 32 + lane) * 4) = r[q];
      }
    }
    if (cs.i1 >= range) break;
    cs = ns;
    ns = segs[1];  // (written before the barrier of the merge)
  }
  if (flight < 0) flight = -1 - flight;
  for (; flight > 0; --flight) {  // copies under way must not outlive the CTA's shared memory
    mbar_wait(bar + st, phase, p.pool.err);
    if (++st == C::NST) {
      st = 0;
      phase ^= 1;
    }
  }
}

// Joins the parts of units that several CTAs shared, and writes the rows of
// sequences with no token.  One CTA per unit, a thread per four results.
template <typename T, bool QUANT, int D>
__global__ void __launch_bounds__(2 * D) join_kernel(PagedAttnParams p) {
  grid_dep_wait();
  grid_dep_launch();
  const int64_t unit = blockIdx.x;
  const int b = static_cast<int>(unit / p.hkv);
  const int j = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint8_t* note = p.ws + unit * sizeof(Meta);
  if (!in_range(note, sizeof(Meta), p.ws, p.ws + p.ws_partials, p.pool.err)) return;
  const int4 raw = *reinterpret_cast<const int4*>(note);  // (garbage where there is no token)
  if (seq_len(p, b) == 0) {
    if (!out_ok<T>(p, unit * p.gqa, D) || !out_ok<T>(p, (unit + 1) * p.gqa - 1, D)) return;
    for (int x = threadIdx.x; x < p.gqa * D; x += 2 * D)
      reinterpret_cast<T*>(p.out)[unit * p.gqa * D + x] = Num<T>::from(0.0f);
    if (p.lse && threadIdx.x < p.gqa) p.lse[unit * p.gqa + threadIdx.x] = -INFINITY;
    return;
  }
  const int first = raw.x, count = raw.y, second = raw.z;
  if (count == 0) return;
  if (first < 0 || count < 0 || second < 0 || second > 1 || first >= p.ctas || count > p.ctas - first) {
    // no CTA began the unit: the lengths changed under the call
    if (threadIdx.x == 0) atomicExch(p.pool.err, kErrBadState);
    return;
  }
  const float* base = reinterpret_cast<const float*>(p.ws + p.ws_partials);
  auto part = [&](int i) {
    return base + (2 * (static_cast<int64_t>(first) + i) + (i == 0 ? second : 0)) * partial_floats(D);
  };
  // parts are read eight at a time, all their loads under way together
  float top[2] = {-INFINITY, -INFINITY}, sum[2] = {0.0f, 0.0f}, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  constexpr int U = 8;
  for (int i0 = 0; i0 < count; i0 += U) {
    float2 mi[U], li[U];
    float4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      mi[u] = make_float2(-INFINITY, -INFINITY);
      li[u] = make_float2(0.0f, 0.0f);
      v[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (i0 + u < count) {
        const float* x = part(i0 + u);
        if (!part_ok(p, x, D)) continue;
        mi[u] = *reinterpret_cast<const float2*>(x + 2 * t);
        li[u] = *reinterpret_cast<const float2*>(x + 8 + 2 * t);
        v[u] = *reinterpret_cast<const float4*>(x + 16 + (j * 32 + lane) * 4);
      }
    }
    float mn[2] = {top[0], top[1]};
#pragma unroll
    for (int u = 0; u < U; ++u) {
      mn[0] = fmaxf(mn[0], mi[u].x);
      mn[1] = fmaxf(mn[1], mi[u].y);
    }
    const float g0 = sum[0] == 0.0f ? 0.0f : ex2(top[0] - mn[0]), g1 = sum[1] == 0.0f ? 0.0f : ex2(top[1] - mn[1]);
    sum[0] *= g0, sum[1] *= g1;
    o[0] *= g0, o[1] *= g1, o[2] *= g0, o[3] *= g1;
    top[0] = mn[0], top[1] = mn[1];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float f0 = li[u].x == 0.0f ? 0.0f : ex2(mi[u].x - top[0]);
      const float f1 = li[u].y == 0.0f ? 0.0f : ex2(mi[u].y - top[1]);
      sum[0] = fmaf(li[u].x, f0, sum[0]);
      sum[1] = fmaf(li[u].y, f1, sum[1]);
      o[0] = fmaf(v[u].x, f0, o[0]);
      o[1] = fmaf(v[u].y, f1, o[1]);
      o[2] = fmaf(v[u].z, f0, o[2]);
      o[3] = fmaf(v[u].w, f1, o[3]);
    }
  }
#pragma unroll
  for (int hd = 0; hd < 2; ++hd) {
    const int head = 2 * t + hd;
    const int64_t row = unit * p.gqa + head;
    if (head >= p.gqa || !out_ok<T>(p, row, D)) continue;
    const float inv = sum[hd] == 0.0f ? 0.0f : 1.0f / sum[hd];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int c = QUANT ? D / 8 * g + 2 * j + half : 16 * j + 8 * half + g;
      reinterpret_cast<T*>(p.out)[row * D + c] = Num<T>::from(o[2 * half + hd] * inv);
    }
    if (p.lse && g == 0 && j == 0) p.lse[row] = (top[hd] + log2f(sum[hd])) * 0.693147180559945f;
  }
}

// ---------------------------------------------------------------- launch

// Without parameters: makes the kernel ready on the current device.
template <typename T, int KB, int VB, int D>
cudaError_t attn_as(const PagedAttnParams* pp, int sms, cudaStream_t s) {
  using C = Shape<KB, VB, D>;
  if (!pp)
    return cudaFuncSetAttribute(attn_kernel<T, KB, VB, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem);
  PagedAttnParams p = *pp;
  // Short tables are not split: a CTA for each unit, and no join.  Measured with
  // 1, 8 and 64 sequences x 8 kv heads, unsplit against split, us: fp16, 512
  // tokens 7.7, 8.0, 26 against 7.5, 9.7, 30, 1024 tokens 11.7, 12.0, 44 against
  // 9.9, 10.5, 50; K8V4, 512 tokens 6.7, 6.9, 17 against 7.4, 9.1, 19, 1024
  // tokens 9.9, 10.3, 28 against 7.9, 10.6, 27; K4V2, 1024 tokens 9.1, 9.6, 23
  // against 8.2, 10.5, 25, 2048 tokens 14.7, 15.2, 38 against 8.7, 12.9, 38.
  // Otherwise one wave, or as many CTAs as the longest sequences that fit the
  // tables can fill.
  const int64_t tokens = static_cast<int64_t>(p.batch.max_pages) << p.pool.page_shift;
  const int64_t units = static_cast<int64_t>(p.hkv) * p.batch.seqs;
  p.solo = tokens <= (C::S == 4 ? 1024 : 512);
  const int64_t most = ((tokens / (16 * C::S) + 1 + C::E) * units + C::W - 1) / C::W;
  const int64_t wave = static_cast<int64_t>(sms) * C::CPS;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = s;
  p.ctas = static_cast<int>(p.solo ? units : most < wave ? most : wave);
  cfg.gridDim = dim3(static_cast<unsigned>(p.ctas));
  cfg.blockDim = dim3(C::threads);
  cfg.dynamicSmemBytes = C::smem;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, attn_kernel<T, KB, VB, D>, p);
  if (e != cudaSuccess || p.solo) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(units));
  cfg.blockDim = dim3(2 * D);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, join_kernel<T, C::quant, D>, p);
}

template <int KB, int VB>
cudaError_t attn_quant(const PagedAttnParams* p, int D, int dtype, int sms, cudaStream_t s) {
  if (dtype == 0) return D == 64 ? attn_as<__half, KB, VB, 64>(p, sms, s) : attn_as<__half, KB, VB, 128>(p, sms, s);
  return D == 64 ? attn_as<__nv_bfloat16, KB, VB, 64>(p, sms, s) : attn_as<__nv_bfloat16, KB, VB, 128>(p, sms, s);
}

}  // namespace paged

cudaError_t paged_attn_k16(const PagedAttnParams* p, int D, int dtype, int sms, cudaStream_t s);
cudaError_t paged_attn_k8(const PagedAttnParams* p, int vb, int D, int dtype, int sms, cudaStream_t s);
cudaError_t paged_attn_k4(const PagedAttnParams* p, int vb, int D, int dtype, int sms, cudaStream_t s);
cudaError_t paged_attn_k2(const PagedAttnParams* p, int vb, int D, int dtype, int sms, cudaStream_t s);

}  // namespace kvq
