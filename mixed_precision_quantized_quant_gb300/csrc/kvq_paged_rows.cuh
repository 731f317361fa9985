// Paged cache: what append and read share: where a row's place in the pages is
// found, the packed arithmetic, the division of a CTA's rows among its warps.
#pragma once

#include <climits>

#include "kvq_paged.cuh"

namespace kvq {
namespace rows {

constexpr int kRowThreads = 256;
constexpr int kRowTokens = 32;  // tokens of a CTA at the most, a lane each when their places are found

// Where a row of a call's tensors lives in the cache.
struct RowPlace {
  int64_t tile;   // byte offset of kv head 0's tile from the pool's start
  int tok;        // token inside the tile
  int rope;       // row of the rotation's table
  int ok;
};

// A warp finds the places of tensor rows row0 + lane, for lanes below `count`.
// The sequence of row0 is the number of ends cu[s + 1] at or before it, counted
// 32 at a time; the others' are found among the 32 ends from there on (more
// where sequences without rows lie between).  Every value that a load's
// address depends on is checked first.
__device__ __forceinline__ RowPlace find_places(const PagedBatch& b, const PagedPool& pool, int row0, int count,
                                                const float* rope, const int32_t* positions, int rope_rows, int lane) {
  RowPlace r;
  r.ok = 0;
  r.tile = 0;
  r.tok = 0;
  r.rope = 0;
  const int row = row0 + lane;
  const bool live = lane < count;
  int seq = row;
  int64_t back = 1;  // rows from this one to the end of its sequence, itself included
  if (b.cu) {
    int c = 0;
    for (int s = lane; s < b.seqs; s += 32) c += b.cu[s + 1] <= row0;
    int base = __reduce_add_sync(0xffffffffu, c);
    bool found = !live;
    while (__any_sync(0xffffffffu, !found)) {
      const int end = base + lane < b.seqs ? b.cu[base + lane + 1] : INT_MAX;
      int k = 0;
#pragma unroll 8
      for (int i = 0; i < 32; ++i) k += __shfl_sync(0xffffffffu, end, i) <= row;
      if (!found && k < 32) {
        seq = base + k;
        found = true;
      }
      base += 32;
    }
    if (!live || seq >= b.seqs || row < b.cu[0]) return r;
    const int end = b.cu[seq + 1];
    if (row < b.cu[seq] || row >= end) {  // not ascending: the count of ends is not the row's sequence
      atomicExch(pool.err, kErrBadState);
      return r;
    }
    back = static_cast<int64_t>(end) - row;
  } else if (!live || seq >= b.seqs) {
    return r;
  }
  const int len = b.lens[seq];
  if (!b.cu && len == 0) return r;  // a padded place of the batch
  const int64_t pos = len - back;
  const int64_t idx = pos >> pool.page_shift;
  if (pos < 0 || idx >= b.max_pages) {
    atomicExch(pool.err, kErrBadState);
    return r;
  }
  const int32_t* entry = b.table + seq * b.table_stride + idx;
  if (!table_ok(b, entry, pool.err)) return r;
  const int page = *entry;
  int rp = static_cast<int>(pos);
  if (rope) {
    if (positions) rp = positions[row];
    if (rp < 0 || rp >= rope_rows) {
      atomicExch(pool.err, kErrBadPosition);
      return r;
    }
  }
  if (page < 0 || page >= pool.num_pages) {
    atomicExch(pool.err, kErrBadPage);
    return r;
  }
  const int in_page = static_cast<int>(pos) & ((1 << pool.page_shift) - 1);
  r.tile = page * pool.page_stride + static_cast<int64_t>(in_page / kTile) * pool.tile_bytes;
  r.tok = in_page % kTile;
  r.rope = rp;
  r.ok = 1;
  return r;
}

template <typename T>
__device__ __forceinline__ void load8(const T* p, bool vec, uint4& v) {
  if (vec) {
    v = *reinterpret_cast<const uint4*>(p);
  } else {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = h[2 * i] | static_cast<uint32_t>(h[2 * i + 1]) << 16;
    v = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, bool vec, const uint4& v) {
  if (vec) {
    *reinterpret_cast<uint4*>(p) = v;
  } else {
    uint16_t* h = reinterpret_cast<uint16_t*>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1)));
  }
}

// Two fp32 values that one instruction works on; every operation rounds each
// of them by itself, as the scalar one does.
typedef unsigned long long f2;
__device__ __forceinline__ f2 f2_of(float x, float y) {
  f2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
  return d;
}
__device__ __forceinline__ void f2_get(f2 v, float& x, float& y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v)); }
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// Eight 16-bit values <-> four pairs.
template <typename T>
__device__ __forceinline__ void unpack8(const uint4& v, f2 (&f)[4]) {
  const T* h = reinterpret_cast<const T*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = f2_of(Num<T>::to(h[2 * i]), Num<T>::to(h[2 * i + 1]));
}
__device__ __forceinline__ uint32_t pack_pair(__half*, f2 v) {
  float x, y;
  f2_get(v, x, y);
  return h2_as_u32(__floats2half2_rn(x, y));
}
__device__ __forceinline__ uint32_t pack_pair(__nv_bfloat16*, f2 v) {
  float x, y;
  f2_get(v, x, y);
  __nv_bfloat162 r = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<uint32_t*>(&r);
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const f2 (&f)[4]) {
  T* const type = nullptr;
  return make_uint4(pack_pair(type, f[0]), pack_pair(type, f[1]), pack_pair(type, f[2]), pack_pair(type, f[3]));
}

// (a, b) -> (a cos - b sin, b cos + a sin); every product and sum rounds by
// itself, so that the result does not depend on how a compiler contracts it.
// The sums are scalar: a packed product and a packed sum were seen to be
// contracted in spite of their .rn.
__device__ __forceinline__ void turn2(f2& a, f2& b, f2 c, f2 s) {
  float ac[2], bs[2], bc[2], as[2];
  f2_get(mul2(a, c), ac[0], ac[1]);
  f2_get(mul2(b, s), bs[0], bs[1]);
  f2_get(mul2(b, c), bc[0], bc[1]);
  f2_get(mul2(a, s), as[0], as[1]);
  a = f2_of(__fsub_rn(ac[0], bs[0]), __fsub_rn(ac[1], bs[1]));
  b = f2_of(__fadd_rn(bc[0], as[0]), __fadd_rn(bc[1], as[1]));
}
// a pair of neighbouring channels
__device__ __forceinline__ void turn_within(f2& v, float c, float s) {
  float a, b;
  f2_get(v, a, b);
  v = f2_of(__fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s)), __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s)));
}

// The pair rounded to fp16 and clamped to its finite values (NaN stays).
__device__ __forceinline__ uint32_t half_pair(f2 v) {
  float x, y;
  f2_get(v, x, y);
  const __half2 lim = __floats2half2_rn(65504.0f, 65504.0f);
  return h2_as_u32(__hmax2_nan(__hmin2_nan(__floats2half2_rn(x, y), lim), __hneg2(lim)));
}

// Floats whose low bytes are min(rint(a / s), qmax) with IEEE division, for
// a >= 0, an fp16 s > 0 and inv = RN(1/s), a pair at a time; s = inv = 0 gives 0.
// One correction step (Markstein): q0 = RN(a inv) is within 2 ulp, r = a - q0 s
// is exact in one fma, and q0 + r inv is off a/s by under 2 ulp * 2^-24 before
// its one rounding.  a / s is nowhere near enough to the middle of two fp32
// numbers for that to matter: a middle m has 25 significant bits, s has 11, so
// m s has at most 36, and |a - m s| / s, which is never 0 (an odd 25-bit m
// needs more bits than a has), is at least 2^-13 ulp.  So it rounds as a / s does.
// Adding 1.5 * 2^23 rounds to a whole number, half to even, in the low bits.
__device__ __forceinline__ void codes_of(f2 a, f2 minus_s, f2 inv, float qmax, uint32_t& c0, uint32_t& c1) {
  const f2 q0 = mul2(a, inv);
  float x, y;
  f2_get(fma2(fma2(q0, minus_s, a), inv, q0), x, y);
  const f2 r = add2(f2_of(fminf(x, qmax), fminf(y, qmax)), f2_of(12582912.0f, 12582912.0f));
  f2_get(r, x, y);
  c0 = __float_as_uint(x);
  c1 = __float_as_uint(y);
}

// Stores eight codes of `bits` bits (8, 4 or 2), each the low byte of a word
// whose next 14 bits are 0, at p: `bits` bytes.
__device__ __forceinline__ void store_codes(uint8_t* p, int bits, const uint32_t (&c)[8]) {
  if (bits == 8) {
    uint2 w;
    w.x = prmt(prmt(c[0], c[1], 0x0040), prmt(c[2], c[3], 0x0040), 0x5410);
    w.y = prmt(prmt(c[4], c[5], 0x0040), prmt(c[6], c[7], 0x0040), 0x5410);
    *reinterpret_cast<uint2*>(p) = w;
  } else if (bits == 4) {
    uint32_t t[4];  // two codes in the low byte
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = c[2 * i] + 16 * c[2 * i + 1];
    *reinterpret_cast<uint32_t*>(p) = prmt(prmt(t[0], t[1], 0x0040), prmt(t[2], t[3], 0x0040), 0x5410);
  } else {
    uint32_t t[2];  // four codes in the low byte
#pragma unroll
    for (int i = 0; i < 2; ++i) t[i] = c[4 * i] + 4 * c[4 * i + 1] + 16 * c[4 * i + 2] + 64 * c[4 * i + 3];
    *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(prmt(t[0], t[1], 0x0040));
  }
}

// A warp's run of the CTA's (token, group) pairs of one kind of row.
struct Run {
  int tk, g, left;  // token and group of the next pair; pairs left
  int groups;
  __device__ __forceinline__ Run(int count, int groups_, int w) : groups(groups_) {
    const int per = (count * groups + 7) >> 3, i = w * per;
    tk = static_cast<int>(__fdividef(static_cast<float>(i) + 0.5f, static_cast<float>(groups)));  // i < 2^20: exact
    g = i - tk * groups;
    left = count * groups - i < per ? count * groups - i : per;
  }
  __device__ __forceinline__ void next() {
    --left;
    if (++g == groups) {
      g = 0;
      ++tk;
    }
  }
};

// ---------------------------------------------------------------- launch

// Tokens of a CTA, at most 32: as many as fill whole waves of `per_sm` CTAs an
// SM, so that the last wave runs as full as the others (an append of 8,000 rows
// took 44 us in 2.2 waves of 8 tokens a CTA, 42 us in 4.4 waves of 4, 39 us in one
// of 18).
inline int cta_tokens(int n, int sms, int per_sm) {
  const int64_t slots = static_cast<int64_t>(sms) * per_sm;
  const int64_t waves = (n - 1) / (slots * kRowTokens) + 1;
  return static_cast<int>((n - 1) / (waves * slots) + 1);
}

template <typename F, typename P>
cudaError_t launch_pdl(F fn, const P& p, dim3 grid, int threads, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, p);
}

}  // namespace rows
}  // namespace kvq
