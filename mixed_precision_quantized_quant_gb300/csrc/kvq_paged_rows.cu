// Paged cache: append (rotation, rounding or quantization, store) and read.
//
// Both move every byte once and compute little: their floor is the copy rate.
//   append: q, k, v rows in; turned q rows and stored rows out.
//   read:   stored rows in; dense rows out.
//
// A row (one token, one head, D channels) is handled by D/16 neighbouring
// lanes with two 16-byte chunks each, so a warp holds a group of 4 or 8 rows.
// The two chunks lie D/2 channels apart (in an append: as far apart as the
// channels that turn together, so that no lane needs another's), and one store
// of a row's lanes covers whole 32-byte sectors.  A CTA takes 1 to 32 tokens:
// its first warp finds their places, a lane each (three dependent loads, so
// they are paid once a CTA); then each of its eight warps takes a run of the
// (token, group) pairs of the queries, of the keys and of the values.
#include <climits>

#include "kvq_paged.cuh"

namespace kvq {
namespace {

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
    if (row < b.cu[seq]) {  // not ascending
      atomicExch(pool.err, kErrBadState);
      return r;
    }
    back = static_cast<int64_t>(b.cu[seq + 1]) - row;
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
  const int page = b.table[seq * b.table_stride + idx];
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
    tk = i / groups;
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

// ---------------------------------------------------------------- append

enum { kQueries, kKeys, kValues };

template <typename T, int D, bool QUANT>
struct Appender {
  static constexpr int LPR = D / 16, RPW = 32 / LPR;  // lanes of a row, rows of a group
  const PagedAppendParams& p;
  const RowPlace* places;
  int row0, count, lane, j, sub, c0, c1;
  bool turns;

  template <int KIND>
  __device__ __forceinline__ const PagedRows& rows() const {
    return KIND == kQueries ? p.q : KIND == kKeys ? p.k : p.v;
  }
  template <int KIND>
  __device__ __forceinline__ int heads() const {
    return KIND == kQueries ? p.hq : p.hkv;
  }
  template <int KIND>
  __device__ __forceinline__ Run run(int warp) const {
    return Run(count, (heads<KIND>() + RPW - 1) / RPW, KIND == kValues ? (warp + 4) & 7 : warp);
  }
  // the lane's chunks of the pair's row
  template <int KIND>
  __device__ __forceinline__ void load(const Run& r, uint4& a, uint4& b) const {
    const int head = r.g * RPW + sub;
    if (r.left <= 0 || head >= heads<KIND>()) return;
    const T* x = reinterpret_cast<const T*>(rows<KIND>().data) + (row0 + r.tk) * rows<KIND>().token_stride +
                 head * rows<KIND>().head_stride;
    load8(x + 8 * c0, p.vec, a);
    load8(x + 8 * c1, p.vec, b);
  }

  // a, b: the first pair's chunks, loaded already
  template <int KIND>
  __device__ __forceinline__ void work(Run r, uint4 a, uint4 b) const {
    int tk = -1;
    RowPlace pl;
    pl.ok = 0;
    f2 cs[4], sn[4];  // of the half-split pairs, or of the lane's two chunks
#pragma unroll 1
    while (r.left > 0) {
      Run n = r;
      n.next();
      uint4 na = make_uint4(0, 0, 0, 0), nb = na;
      load<KIND>(n, na, nb);  // under way while this pair is worked on
      if (r.tk != tk) {
        tk = r.tk;
        pl = places[tk];
        if (KIND != kValues && turns && pl.ok) {
          const float* t = p.rope + static_cast<int64_t>(pl.rope) * p.rope_dim;
          const float* u = t + p.rope_dim / 2;
          const int o0 = p.interleaved ? 4 * c0 : 8 * j, o1 = p.interleaved ? 4 * c1 : 8 * j + 4;
          float4 x = __ldg(reinterpret_cast<const float4*>(t + o0)), y = __ldg(reinterpret_cast<const float4*>(t + o1));
          cs[0] = f2_of(x.x, x.y), cs[1] = f2_of(x.z, x.w), cs[2] = f2_of(y.x, y.y), cs[3] = f2_of(y.z, y.w);
          x = __ldg(reinterpret_cast<const float4*>(u + o0)), y = __ldg(reinterpret_cast<const float4*>(u + o1));
          sn[0] = f2_of(x.x, x.y), sn[1] = f2_of(x.z, x.w), sn[2] = f2_of(y.x, y.y), sn[3] = f2_of(y.z, y.w);
        }
      }
      if (pl.ok) one<KIND>(r.tk, r.g * RPW + sub, pl, cs, sn, a, b);
      a = na;
      b = nb;
      r = n;
    }
  }

  template <int KIND>
  __device__ __forceinline__ void one(int tk, int head, const RowPlace& pl, const f2 (&cs)[4], const f2 (&sn)[4],
                                      uint4 a, uint4 b) const {
    f2 f[2][4];
    const bool turned = KIND != kValues && turns;
    if (turned || (QUANT && KIND != kQueries)) {
      unpack8<T>(a, f[0]);
      unpack8<T>(b, f[1]);
    }
    if (turned) {
      if (!p.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) turn2(f[0][i], f[1][i], cs[i], sn[i]);
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float c[2], s[2];
            f2_get(cs[2 * h + i / 2], c[0], c[1]);
            f2_get(sn[2 * h + i / 2], s[0], s[1]);
            turn_within(f[h][i], c[i % 2], s[i % 2]);
          }
      }
      if (!QUANT || KIND == kQueries) {
        a = pack8<T>(f[0]);
        b = pack8<T>(f[1]);
      }
    }
    const bool live = head < heads<KIND>();
    if constexpr (KIND == kQueries) {
      if (live) {
        T* y = reinterpret_cast<T*>(p.qo.data) + (row0 + tk) * p.qo.token_stride + head * p.qo.head_stride;
        store8(y + 8 * c0, p.vec, a);
        store8(y + 8 * c1, p.vec, b);
      }
    } else if constexpr (!QUANT) {
      if (live) {
        uint8_t* t = p.pool.pages + pl.tile + head * p.pool.head_stride;
        t += (KIND == kValues ? 32 * D : 0) + pl.tok * 2 * D;
        *reinterpret_cast<uint4*>(t + 16 * tile_chunk16(c0, pl.tok)) = a;
        *reinterpret_cast<uint4*>(t + 16 * tile_chunk16(c1, pl.tok)) = b;
      }
    } else {
      quantize<KIND>(f, head, live, pl);
    }
  }

  template <int KIND>
  __device__ __forceinline__ void quantize(const f2 (&f)[2][4], int head, bool live, const RowPlace& pl) const {
    // the row in fp16, its least and greatest value
    uint32_t h[2][4];
    __half2 mn2, mx2;
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        h[x][i] = half_pair(f[x][i]);
        const __half2 v = u32_as_h2(h[x][i]);
        mn2 = x + i ? __hmin2_nan(mn2, v) : v;
        mx2 = x + i ? __hmax2_nan(mx2, v) : v;
      }
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) {
      mn2 = __hmin2_nan(mn2, u32_as_h2(__shfl_xor_sync(0xffffffffu, h2_as_u32(mn2), o)));
      mx2 = __hmax2_nan(mx2, u32_as_h2(__shfl_xor_sync(0xffffffffu, h2_as_u32(mx2), o)));
    }
    const __half mnh = __hmin_nan(__low2half(mn2), __high2half(mn2));
    const float mn = __half2float(mnh), mx = __half2float(__hmax_nan(__low2half(mx2), __high2half(mx2)));
    const int bits = KIND == kValues ? p.pool.vb : p.pool.kb;
    const float qmax = static_cast<float>((1 << bits) - 1);
    const __half sh = __float2half_rn(__fdiv_rn(__fsub_rn(mx, mn), qmax));
    const float s = __half2float(sh);
    const float inv = s > 0.0f ? __frcp_rn(s) : 0.0f;
    if (!live) return;
    uint8_t* t = p.pool.pages + pl.tile + head * p.pool.head_stride;
    const int rk = D / 8 * p.pool.kb, rv = D / 8 * p.pool.vb;
    const int kr = tile_key_row(pl.tok);
    uint8_t* codes = t + (KIND == kValues ? 16 * rk + pl.tok * rv : kr * rk);
    const int xr = KIND == kValues ? tile_val_xor(rv, pl.tok) : tile_key_xor(rk, kr);
    const f2 minus_mn = f2_of(-mn, -mn), minus_s = f2_of(-s, -s), inv2 = f2_of(inv, inv);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 v = __half22float2(u32_as_h2(h[x][i]));
        codes_of(add2(f2_of(v.x, v.y), minus_mn), minus_s, inv2, qmax, w[2 * i], w[2 * i + 1]);
      }
      store_codes(codes + (((x ? c1 : c0) * bits) ^ xr), bits, w);
    }
    if (j == 0)
      *reinterpret_cast<__half2*>(t + 16 * (rk + rv) + kr * 8 + (KIND == kValues ? 4 : 0)) = __halves2half2(sh, mnh);
  }
};

template <typename T, int D, bool QUANT>
__global__ void __launch_bounds__(kRowThreads, 3) paged_append_kernel(const __grid_constant__ PagedAppendParams p) {
  using A = Appender<T, D, QUANT>;
  __shared__ RowPlace places[kRowTokens];
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row0 = blockIdx.x << p.tokens;  // (n is at most INT_MAX - 31, see kvq_paged_append)
  const int count = p.n - row0 < (1 << p.tokens) ? p.n - row0 : 1 << p.tokens;
  const int j = lane % A::LPR;
  const int pairs = p.rope ? p.rope_dim / 16 : 0;
  const bool turns = j < pairs;
  // the lane's chunks: a pair that turns together, or two that pass
  const int c0 = turns ? j : pairs + j, c1 = turns ? j + pairs : c0 + A::LPR - pairs;
  const A w = {p, places, row0, count, lane, j, lane / A::LPR, c0, c1, turns};
  uint4 a[3], b[3];  // first rows of each kind, on their way while the places are found
  const Run rk = w.template run<kKeys>(warp), rv = w.template run<kValues>(warp);
  const Run rq = p.hq ? w.template run<kQueries>(warp) : Run(0, 1, 0);
  w.template load<kQueries>(rq, a[0], b[0]);
  w.template load<kKeys>(rk, a[1], b[1]);
  w.template load<kValues>(rv, a[2], b[2]);
  if (warp == 0) {
    const RowPlace r = find_places(p.batch, p.pool, row0, count, p.rope, p.positions, p.rope_rows, lane);
    if (lane < count) places[lane] = r;
  }
  __syncthreads();
  w.template work<kQueries>(rq, a[0], b[0]);
  w.template work<kKeys>(rk, a[1], b[1]);
  w.template work<kValues>(rv, a[2], b[2]);
}

// ---------------------------------------------------------------- read

// Eight codes of B bits, in the low 8 B bits of {x, y}, times s plus z: the
// product is exact in fp32, so the fma rounds once.
template <int B>
__device__ __forceinline__ void dequant8(uint32_t x, uint32_t y, f2 s, f2 z, f2 (&f)[4]) {
  // bytes that hold one code each
  uint32_t w[4] = {x, y, 0, 0};
  if (B == 4) {
    w[0] = x & 0x0f0f0f0fu;
    w[1] = (x >> 4) & 0x0f0f0f0fu;
  } else if (B == 2) {
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = (x >> (2 * k)) & 0x0303u;
  }
  float c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t v = B == 8 ? w[i / 4] >> (8 * (i % 4)) : B == 4 ? w[i % 2] >> (8 * (i / 2)) : w[i % 4] >> (8 * (i / 4));
    c[i] = static_cast<float>(v & 0xffu);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = fma2(f2_of(c[2 * i], c[2 * i + 1]), s, z);
}

constexpr int kReadAhead = 4;  // groups whose loads are under way together

template <typename T, int D, bool QUANT, bool VALUES>
__device__ __forceinline__ void read_rows(const PagedReadParams& p, const RowPlace* places, int row0, int count,
                                          int warp, int lane) {
  constexpr int LPR = D / 16, RPW = 32 / LPR, U = kReadAhead;
  const PagedRows& dst = VALUES ? p.v : p.k;
  if (!dst.data) return;
  const int j = lane % LPR, sub = lane / LPR;
  const int bits = VALUES ? p.pool.vb : p.pool.kb;
  const int rk = D / 8 * p.pool.kb, rv = D / 8 * p.pool.vb;
  Run r(count, (p.hkv + RPW - 1) / RPW, VALUES ? (warp + 4) & 7 : warp);
#pragma unroll 1
  while (r.left > 0) {
    uint4 a[U], b[U];  // the lane's chunks j and j + LPR of the row, or their codes
    uint32_t sz[U];
    T* y[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      y[u] = nullptr;
      const int head = r.g * RPW + sub;
      if (r.left > 0 && head < p.hkv && places[r.tk].ok) {
        const RowPlace pl = places[r.tk];
        y[u] = reinterpret_cast<T*>(dst.data) + (row0 + r.tk) * dst.token_stride + head * dst.head_stride + 8 * j;
        const uint8_t* tile = p.pool.pages + pl.tile + head * p.pool.head_stride;
        if (!QUANT) {
          tile += (VALUES ? 32 * D : 0) + pl.tok * 2 * D;
          a[u] = *reinterpret_cast<const uint4*>(tile + 16 * tile_chunk16(j, pl.tok));
          b[u] = *reinterpret_cast<const uint4*>(tile + 16 * tile_chunk16(j + LPR, pl.tok));
        } else {
          const int kr = tile_key_row(pl.tok);
          const int x = VALUES ? tile_val_xor(rv, pl.tok) : tile_key_xor(rk, kr);
          sz[u] = *reinterpret_cast<const uint32_t*>(tile + 16 * (rk + rv) + kr * 8 + (VALUES ? 4 : 0));
          tile += VALUES ? 16 * rk + pl.tok * rv : kr * rk;
          const uint8_t *x0 = tile + ((j * bits) ^ x), *x1 = tile + (((j + LPR) * bits) ^ x);
          if (bits == 8) {
            *reinterpret_cast<uint2*>(&a[u]) = *reinterpret_cast<const uint2*>(x0);
            *reinterpret_cast<uint2*>(&b[u]) = *reinterpret_cast<const uint2*>(x1);
          } else if (bits == 4) {
            a[u].x = *reinterpret_cast<const uint32_t*>(x0);
            b[u].x = *reinterpret_cast<const uint32_t*>(x1);
          } else {
            a[u].x = *reinterpret_cast<const uint16_t*>(x0);
            b[u].x = *reinterpret_cast<const uint16_t*>(x1);
          }
        }
      }
      if (r.left > 0) r.next();
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!y[u]) continue;
      if (QUANT) {
        const float sf = __low2float(u32_as_h2(sz[u])), zf = __high2float(u32_as_h2(sz[u]));
        const f2 s = f2_of(sf, sf), z = f2_of(zf, zf);
        f2 f[2][4];
        if (bits == 8) {
          dequant8<8>(a[u].x, a[u].y, s, z, f[0]);
          dequant8<8>(b[u].x, b[u].y, s, z, f[1]);
        } else if (bits == 4) {
          dequant8<4>(a[u].x, 0, s, z, f[0]);
          dequant8<4>(b[u].x, 0, s, z, f[1]);
        } else {
          dequant8<2>(a[u].x, 0, s, z, f[0]);
          dequant8<2>(b[u].x, 0, s, z, f[1]);
        }
        a[u] = pack8<T>(f[0]);
        b[u] = pack8<T>(f[1]);
      }
      store8(y[u], p.vec, a[u]);
      store8(y[u] + 8 * LPR, p.vec, b[u]);
    }
  }
}

template <typename T, int D, bool QUANT>
__global__ void __launch_bounds__(kRowThreads, 3) paged_read_kernel(const __grid_constant__ PagedReadParams p) {
  __shared__ RowPlace places[kRowTokens];
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row0 = blockIdx.x << p.tokens;
  const int count = p.n - row0 < (1 << p.tokens) ? p.n - row0 : 1 << p.tokens;
  if (warp == 0) {
    const RowPlace r = find_places(p.batch, p.pool, row0, count, nullptr, nullptr, 0, lane);
    if (lane < count) places[lane] = r;
  }
  __syncthreads();
  read_rows<T, D, QUANT, false>(p, places, row0, count, warp, lane);
  read_rows<T, D, QUANT, true>(p, places, row0, count, warp, lane);
}

// log2 of the tokens of a CTA: 32, halved while the grid would be under eight
// CTAs an SM.
int cta_tokens(int n, int sms) {
  int t = 5;
  while (t > 0 && ((n - 1) >> t) + 1 < 8 * sms) --t;
  return t;
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

template <typename T, int D>
cudaError_t append_as(PagedAppendParams p, int sms, cudaStream_t s) {
  p.tokens = cta_tokens(p.n, sms);
  const dim3 grid(static_cast<unsigned>(((p.n - 1) >> p.tokens) + 1));
  return p.pool.kb == 16 ? launch_pdl(paged_append_kernel<T, D, false>, p, grid, kRowThreads, s)
                         : launch_pdl(paged_append_kernel<T, D, true>, p, grid, kRowThreads, s);
}

template <typename T, int D>
cudaError_t read_as(PagedReadParams p, int sms, cudaStream_t s) {
  p.tokens = cta_tokens(p.n, sms);
  const dim3 grid(static_cast<unsigned>(((p.n - 1) >> p.tokens) + 1));
  return p.pool.kb == 16 ? launch_pdl(paged_read_kernel<T, D, false>, p, grid, kRowThreads, s)
                         : launch_pdl(paged_read_kernel<T, D, true>, p, grid, kRowThreads, s);
}

}  // namespace

cudaError_t paged_append_launch(const PagedAppendParams& p, int D, int dtype, int sms, cudaStream_t s) {
  if (dtype == 0) return D == 64 ? append_as<__half, 64>(p, sms, s) : append_as<__half, 128>(p, sms, s);
  return D == 64 ? append_as<__nv_bfloat16, 64>(p, sms, s) : append_as<__nv_bfloat16, 128>(p, sms, s);
}

cudaError_t paged_read_launch(const PagedReadParams& p, int D, int dtype, int sms, cudaStream_t s) {
  if (dtype == 0) return D == 64 ? read_as<__half, 64>(p, sms, s) : read_as<__half, 128>(p, sms, s);
  return D == 64 ? read_as<__nv_bfloat16, 64>(p, sms, s) : read_as<__nv_bfloat16, 128>(p, sms, s);
}

}  // namespace kvq
