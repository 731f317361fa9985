// Paged cache: append (rotation, rounding or quantization, store) and read.
//
// Both move every byte once and compute little: their floor is the copy rate.
//   append: q, k, v rows in; turned q rows and stored rows out.
//   read:   stored rows in; dense rows out.
//
// A row (one token, one head, D channels) is handled by D/16 neighbouring
// lanes with two 16-byte chunks each, so a warp holds 4 or 8 rows.  In an
// append a lane's chunks are the two that the rotation pairs (c and
// c + dim/16): no exchange between lanes is needed but the row's min and max.
#include "kvq_paged.cuh"

namespace kvq {
namespace {

constexpr int kRowThreads = 256;

// Where a row of a call's tensors lives in the cache.
struct RowPlace {
  int64_t tile;   // byte offset of kv head 0's tile from the pool's start
  int tok;        // token inside the tile
  int rope;       // row of the rotation's table
  int ok;
};

// One warp finds the place of tensor row `row`.  The sequence is the number of
// ends cu[s + 1] at or before the row, counted 32 at a time, so that the
// search costs one round trip for up to 32 sequences instead of a chain of
// dependent loads.  Every value that a load's address depends on is checked first.
__device__ __forceinline__ RowPlace find_place(const PagedBatch& b, const PagedPool& pool, int row, const float* rope,
                                               const int32_t* positions, int rope_rows, int lane) {
  RowPlace r;
  r.ok = 0;
  r.tile = 0;
  r.tok = 0;
  r.rope = 0;
  int seq = row;
  int64_t back = 1;  // rows from this one to the end of its sequence, itself included
  if (b.cu) {
    int c = 0;
    for (int s = lane; s < b.seqs; s += 32) c += b.cu[s + 1] <= row;
    seq = __reduce_add_sync(0xffffffffu, c);
    if (seq >= b.seqs || row < b.cu[0]) return r;
    if (row < b.cu[seq]) {  // not ascending
      if (lane == 0) atomicExch(pool.err, kErrBadState);
      return r;
    }
    back = static_cast<int64_t>(b.cu[seq + 1]) - row;
  } else if (seq >= b.seqs) {
    return r;
  }
  const int len = b.lens[seq];
  if (!b.cu && len == 0) return r;  // a padded place of the batch
  const int64_t pos = len - back;
  const int64_t idx = pos >> pool.page_shift;
  if (pos < 0 || idx >= b.max_pages) {
    if (lane == 0) atomicExch(pool.err, kErrBadState);
    return r;
  }
  const int page = b.table[seq * b.table_stride + idx];
  int rp = static_cast<int>(pos);
  if (rope) {
    if (positions) rp = positions[row];
    if (rp < 0 || rp >= rope_rows) {
      if (lane == 0) atomicExch(pool.err, kErrBadPosition);
      return r;
    }
  }
  if (page < 0 || page >= pool.num_pages) {
    if (lane == 0) atomicExch(pool.err, kErrBadPage);
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

template <typename T>
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const T* h = reinterpret_cast<const T*>(&v);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = Num<T>::to(h[i]);
}

template <typename T>
__device__ __forceinline__ uint4 pack8f(const float (&f)[8]) {
  uint4 v;
  T* h = reinterpret_cast<T*>(&v);
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = Num<T>::from(f[i]);
  return v;
}

// (a, b) -> (a cos - b sin, b cos + a sin); every operation rounds by itself,
// so that the result does not depend on how a compiler contracts it.
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = x;
}

__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// The row's value as fp16, clamped to its range (NaN stays).
__device__ __forceinline__ float as_half(float x) {
  const float y = x != x ? x : fminf(fmaxf(x, -65504.0f), 65504.0f);
  return __half2float(__float2half_rn(y));
}

// rint(a / s) with IEEE division, for 0 <= a and an fp16 s > 0, inv = RN(1/s).
// One correction step (Markstein): q0 = RN(a inv) is within 2 ulp, r = a - q0 s
// is exact in one fma, and q0 + r inv is off a/s by under 2 ulp * 2^-24 before
// its one rounding.  a / s is nowhere near enough to the middle of two fp32
// numbers for that to matter: a middle m has 25 significant bits, s has 11, so
// m s has at most 36, and |a - m s| / s, which is never 0 (an odd 25-bit m
// needs more bits than a has), is at least 2^-13 ulp.  So it rounds as a / s does.
__device__ __forceinline__ uint32_t code_of(float a, float s, float inv, float qmax) {
  const float q0 = __fmul_rn(a, inv);
  const float q = __fmaf_rn(__fmaf_rn(-q0, s, a), inv, q0);
  return static_cast<uint32_t>(fminf(rintf(q), qmax));
}

// Stores eight codes of `bits` bits (8, 4 or 2) at p, `bits` bytes.
__device__ __forceinline__ void store_codes(uint8_t* p, int bits, const uint32_t (&c)[8]) {
  if (bits == 8) {
    uint2 w;
    w.x = c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24;
    w.y = c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24;
    *reinterpret_cast<uint2*>(p) = w;
  } else if (bits == 4) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) w |= c[i] << (4 * i);
    *reinterpret_cast<uint32_t*>(p) = w;
  } else {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) w |= c[i] << (2 * i);
    *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(w);
  }
}

// ---------------------------------------------------------------- append

// One CTA per token; its warps take the token's q, k and v rows 32 / (D/16) at
// a time.
template <typename T, int D, bool QUANT>
__global__ void __launch_bounds__(kRowThreads) paged_append_kernel(PagedAppendParams p) {
  constexpr int LPR = D / 16;      // lanes per row
  constexpr int RPW = 32 / LPR;    // rows per warp
  __shared__ RowPlace place_s;
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int row = blockIdx.x;
  const int j = lane % LPR;
  const int rows = p.hq + 2 * p.hkv;
  const int rot_pairs = p.rope ? p.rope_dim / 16 : 0;
  // the lane's chunks: a pair that turns together, or two that pass
  const int c0 = j < rot_pairs ? j : 2 * rot_pairs + 2 * (j - rot_pairs);
  const int c1 = j < rot_pairs ? j + rot_pairs : c0 + 1;

  if (warp == 0) {
    const RowPlace r = find_place(p.batch, p.pool, row, p.rope, p.positions, p.rope_rows, lane);
    if (lane == 0) place_s = r;
  }
  __syncthreads();
  const RowPlace pl = place_s;
  if (!pl.ok) return;

  float cs[2][8], sn[2][8];  // half-split pairs use [0] only
  if (j < rot_pairs) {
    const float* t = p.rope + static_cast<int64_t>(pl.rope) * p.rope_dim;
    if (!p.interleaved) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        cs[0][i] = __ldg(t + 8 * j + i);
        sn[0][i] = __ldg(t + p.rope_dim / 2 + 8 * j + i);
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = h ? c1 : c0;
          cs[h][i] = __ldg(t + 4 * c + i);
          sn[h][i] = __ldg(t + p.rope_dim / 2 + 4 * c + i);
        }
    }
  }

  for (int base = warp * RPW; base < rows; base += warps * RPW) {
    const int r = base + lane / LPR;
    const bool live = r < rows;
    const bool is_q = r < p.hq, is_v = r >= p.hq + p.hkv;
    const int head = is_q ? r : (is_v ? r - p.hq - p.hkv : r - p.hq);
    const PagedRows& src = is_q ? p.q : (is_v ? p.v : p.k);
    uint4 a = make_uint4(0, 0, 0, 0), b = a;
    if (live) {
      const T* x = reinterpret_cast<const T*>(src.data) + row * src.token_stride + head * src.head_stride;
      load8(x + 8 * c0, p.vec, a);
      load8(x + 8 * c1, p.vec, b);
    }
    const bool turns = !is_v && j < rot_pairs;
    float f[2][8];
    if (QUANT || turns) {
      unpack8<T>(a, f[0]);
      unpack8<T>(b, f[1]);
    }
    if (turns) {
      if (!p.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) turn(f[0][i], f[1][i], cs[0][i], sn[0][i]);
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i) turn(f[h][2 * i], f[h][2 * i + 1], cs[h][i], sn[h][i]);
      }
      if (!QUANT || is_q) {
        a = pack8f<T>(f[0]);
        b = pack8f<T>(f[1]);
      }
    }
    if (QUANT) {
      // every lane takes part in the exchange, also those of query rows
      float mn = INFINITY, mx = -INFINITY;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          f[h][i] = as_half(f[h][i]);
          mn = min_nan(mn, f[h][i]);
          mx = max_nan(mx, f[h][i]);
        }
#pragma unroll
      for (int o = 1; o < LPR; o <<= 1) {
        mn = min_nan(mn, __shfl_xor_sync(0xffffffffu, mn, o));
        mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      }
      if (live && !is_q) {
        const int bits = is_v ? p.pool.vb : p.pool.kb;
        const float qmax = static_cast<float>((1 << bits) - 1);
        const __half sh = __float2half_rn(__fdiv_rn(__fsub_rn(mx, mn), qmax));
        const float s = __half2float(sh);
        const float inv = s > 0.0f ? __frcp_rn(s) : 0.0f;
        uint32_t q0[8], q1[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          q0[i] = code_of(__fsub_rn(f[0][i], mn), s, inv, qmax);
          q1[i] = code_of(__fsub_rn(f[1][i], mn), s, inv, qmax);
        }
        uint8_t* t = p.pool.pages + pl.tile + head * p.pool.head_stride;
        const int rk = D * p.pool.kb / 8, rv = D * p.pool.vb / 8;
        const int kr = tile_key_row(pl.tok);
        uint8_t* codes = is_v ? t + 16 * rk + pl.tok * rv : t + kr * rk;
        const int x = is_v ? tile_val_xor(rv, pl.tok) : tile_key_xor(rk, kr);
        store_codes(codes + ((c0 * bits) ^ x), bits, q0);
        store_codes(codes + ((c1 * bits) ^ x), bits, q1);
        if (j == 0)
          *reinterpret_cast<__half2*>(t + 16 * (rk + rv) + kr * 8 + (is_v ? 4 : 0)) =
              __halves2half2(sh, __float2half_rn(mn));
      }
    }
    if (live && is_q) {
      T* y = reinterpret_cast<T*>(p.qo.data) + row * p.qo.token_stride + head * p.qo.head_stride;
      store8(y + 8 * c0, p.vec, a);
      store8(y + 8 * c1, p.vec, b);
    } else if (!QUANT && live) {
      uint8_t* t = p.pool.pages + pl.tile + head * p.pool.head_stride + (is_v ? 32 * D : 0) + pl.tok * 2 * D;
      *reinterpret_cast<uint4*>(t + 16 * tile_chunk16(c0, pl.tok)) = a;
      *reinterpret_cast<uint4*>(t + 16 * tile_chunk16(c1, pl.tok)) = b;
    }
  }
}

// ---------------------------------------------------------------- read

constexpr int kReadTokens = 8;  // tokens of a CTA, one per warp while their places are found

template <typename T, int D, bool QUANT>
__global__ void __launch_bounds__(kRowThreads) paged_read_kernel(PagedReadParams p) {
  constexpr int LPR = D / 16;
  __shared__ RowPlace place_s[kReadTokens];
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row0 = blockIdx.x * kReadTokens;
  if (row0 + warp < p.n) {
    const RowPlace r = find_place(p.batch, p.pool, row0 + warp, nullptr, nullptr, 0, lane);
    if (lane == 0) place_s[warp] = r;
  } else if (lane == 0) {
    place_s[warp].ok = 0;
  }
  __syncthreads();
  const int j = threadIdx.x % LPR;
  const int rk = D * p.pool.kb / 8, rv = D * p.pool.vb / 8;
  const int items = kReadTokens * p.hkv * 2;
#pragma unroll 4
  for (int it = threadIdx.x / LPR; it < items; it += kRowThreads / LPR) {
    const int t = it / (2 * p.hkv);
    const int rest = it - t * 2 * p.hkv;
    const bool is_v = rest >= p.hkv;
    const int head = is_v ? rest - p.hkv : rest;
    const PagedRows& dst = is_v ? p.v : p.k;
    if (!place_s[t].ok || !dst.data) continue;
    const int tok = place_s[t].tok;
    const uint8_t* tile = p.pool.pages + place_s[t].tile + head * p.pool.head_stride;
    T* y = reinterpret_cast<T*>(dst.data) + (row0 + t) * dst.token_stride + head * dst.head_stride + 16 * j;
    uint4 a, b;
    if (!QUANT) {
      const uint8_t* x = tile + (is_v ? 32 * D : 0) + tok * 2 * D;
      a = *reinterpret_cast<const uint4*>(x + 16 * tile_chunk16(2 * j, tok));
      b = *reinterpret_cast<const uint4*>(x + 16 * tile_chunk16(2 * j + 1, tok));
    } else {
      const int kr = tile_key_row(tok);
      const int bits = is_v ? p.pool.vb : p.pool.kb;
      const uint8_t* x = is_v ? tile + 16 * rk + tok * rv : tile + kr * rk;
      x += (2 * j * bits) ^ (is_v ? tile_val_xor(rv, tok) : tile_key_xor(rk, kr));
      const __half2 sz = *reinterpret_cast<const __half2*>(tile + 16 * (rk + rv) + kr * 8 + (is_v ? 4 : 0));
      const float s = __low2float(sz), z = __high2float(sz);
      uint32_t w[4];
      if (bits == 8) {
        const uint4 v = *reinterpret_cast<const uint4*>(x);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
      } else if (bits == 4) {
        const uint2 v = *reinterpret_cast<const uint2*>(x);
        w[0] = v.x, w[1] = v.x >> 16, w[2] = v.y, w[3] = v.y >> 16;
      } else {
        const uint32_t v = *reinterpret_cast<const uint32_t*>(x);
        w[0] = v, w[1] = v >> 8, w[2] = v >> 16, w[3] = v >> 24;
      }
      const uint32_t mask = (1u << bits) - 1;
      float f[2][8];
#pragma unroll
      for (int i = 0; i < 16; ++i)  // the product is exact in fp32, so the fma rounds once
        f[i / 8][i % 8] = __fmaf_rn(static_cast<float>((w[i / 4] >> (bits * (i % 4))) & mask), s, z);
      a = pack8f<T>(f[0]);
      b = pack8f<T>(f[1]);
    }
    store8(y, p.vec, a);
    store8(y + 8, p.vec, b);
  }
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
cudaError_t append_as(const PagedAppendParams& p, cudaStream_t s) {
  const int per_warp = 32 / (D / 16);
  int warps = (p.hq + 2 * p.hkv + per_warp - 1) / per_warp;
  if (warps > kRowThreads / 32) warps = kRowThreads / 32;
  const dim3 grid(static_cast<unsigned>(p.n));
  return p.pool.kb == 16 ? launch_pdl(paged_append_kernel<T, D, false>, p, grid, 32 * warps, s)
                         : launch_pdl(paged_append_kernel<T, D, true>, p, grid, 32 * warps, s);
}

template <typename T, int D>
cudaError_t read_as(const PagedReadParams& p, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((p.n + kReadTokens - 1) / kReadTokens));
  return p.pool.kb == 16 ? launch_pdl(paged_read_kernel<T, D, false>, p, grid, kRowThreads, s)
                         : launch_pdl(paged_read_kernel<T, D, true>, p, grid, kRowThreads, s);
}

}  // namespace

cudaError_t paged_append_launch(const PagedAppendParams& p, int D, int dtype, cudaStream_t s) {
  if (dtype == 0) return D == 64 ? append_as<__half, 64>(p, s) : append_as<__half, 128>(p, s);
  return D == 64 ? append_as<__nv_bfloat16, 64>(p, s) : append_as<__nv_bfloat16, 128>(p, s);
}

cudaError_t paged_read_launch(const PagedReadParams& p, int D, int dtype, cudaStream_t s) {
  if (dtype == 0) return D == 64 ? read_as<__half, 64>(p, s) : read_as<__half, 128>(p, s);
  return D == 64 ? read_as<__nv_bfloat16, 64>(p, s) : read_as<__nv_bfloat16, 128>(p, s);
}

}  // namespace kvq
