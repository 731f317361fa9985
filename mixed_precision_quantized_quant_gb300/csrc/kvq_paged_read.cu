// Paged cache: the newest rows of every sequence read back, dequantized.
//
// Every byte moves once and little is computed, so the floor is the copy rate:
// stored rows in, dense rows out, most of it the writing.  A row is handled by
// D/16 neighbouring lanes with two 16-byte chunks each, D/2 channels apart, so
// that one store of a row's lanes covers whole 32-byte sectors.  A CTA takes up to
// 32 tokens: its first warp finds their places, a lane each; then each
// of its eight warps takes a run of the (token, group of rows) pairs.
//
// Measured (GB300): 52,000 rows of 8 kv heads from K4V2 to bf16 45.5 us, 83% of
// the copy rate (a kernel for every pair of widths; one for all took 52), bound by
// the ALU pipe, 61% busy with converting codes; 515 rows 3.2 us.
#include "kvq_paged_rows.cuh"

namespace kvq {
namespace {

using namespace rows;

constexpr int kReadPerSm = 3;  // CTAs of an SM

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

template <typename T, int D, int BITS, bool VALUES>
__device__ __forceinline__ void read_rows(const PagedReadParams& p, const RowPlace* places, int row0, int count,
                                          int warp, int lane) {
  constexpr int LPR = D / 16, RPW = 32 / LPR, U = kReadAhead;
  const PagedRows& dst = VALUES ? p.v : p.k;
  if (!dst.data) return;
  const int j = lane % LPR, sub = lane / LPR;
  constexpr int bits = BITS;
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
        if (!pool_ok(p.pool, tile, p.pool.tile_bytes) || !rows_ok(dst, y[u], 32 * LPR - 16 * j, p.pool.err)) {
          y[u] = nullptr;
          r.next();
          continue;
        }
        if constexpr (BITS == 16) {
          tile += (VALUES ? 32 * D : 0) + pl.tok * 2 * D;
          a[u] = *reinterpret_cast<const uint4*>(tile + 16 * tile_chunk16(j, pl.tok));
          b[u] = *reinterpret_cast<const uint4*>(tile + 16 * tile_chunk16(j + LPR, pl.tok));
        } else {
          const int kr = tile_key_row(pl.tok);
          const int x = VALUES ? tile_val_xor(rv, pl.tok) : tile_key_xor(rk, kr);
          sz[u] = *reinterpret_cast<const uint32_t*>(tile + 16 * (rk + rv) + kr * 8 + (VALUES ? 4 : 0));
          tile += VALUES ? 16 * rk + pl.tok * rv : kr * rk;
          const uint8_t *x0 = tile + ((j * bits) ^ x), *x1 = tile + (((j + LPR) * bits) ^ x);
          if constexpr (bits == 8) {
            *reinterpret_cast<uint2*>(&a[u]) = *reinterpret_cast<const uint2*>(x0);
            *reinterpret_cast<uint2*>(&b[u]) = *reinterpret_cast<const uint2*>(x1);
          } else if constexpr (bits == 4) {
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
      if constexpr (BITS != 16) {
        const float sf = __low2float(u32_as_h2(sz[u])), zf = __high2float(u32_as_h2(sz[u]));
        const f2 s = f2_of(sf, sf), z = f2_of(zf, zf);
        f2 f[2][4];
        dequant8<BITS>(a[u].x, a[u].y, s, z, f[0]);
        dequant8<BITS>(b[u].x, b[u].y, s, z, f[1]);
        a[u] = pack8<T>(f[0]);
        b[u] = pack8<T>(f[1]);
      }
      store8(y[u], p.vec, a[u]);
      store8(y[u] + 8 * LPR, p.vec, b[u]);
    }
  }
}

template <typename T, int D, int KB, int VB>
__global__ void __launch_bounds__(kRowThreads, kReadPerSm) paged_read_kernel(const __grid_constant__ PagedReadParams p) {
  __shared__ RowPlace places[kRowTokens];
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row0 = blockIdx.x * p.tokens;  // (n is at most INT_MAX - 31)
  const int count = p.n - row0 < p.tokens ? p.n - row0 : p.tokens;
  if (warp == 0) {
    const RowPlace r = find_places(p.batch, p.pool, row0, count, nullptr, nullptr, 0, lane);
    if (lane < count) places[lane] = r;
  }
  __syncthreads();
  read_rows<T, D, KB, false>(p, places, row0, count, warp, lane);
  read_rows<T, D, VB, true>(p, places, row0, count, warp, lane);
}

template <typename T, int D, int KB, int VB>
cudaError_t read_as(PagedReadParams p, int sms, cudaStream_t s) {
  p.tokens = cta_tokens(p.n, sms, kReadPerSm);
  return launch_pdl(paged_read_kernel<T, D, KB, VB>, p, dim3(static_cast<unsigned>((p.n - 1) / p.tokens + 1)),
                    kRowThreads, s);
}

template <typename T, int D>
cudaError_t read_pair(const PagedReadParams& p, int sms, cudaStream_t s) {
  switch (p.pool.kb * 32 + p.pool.vb) {
    case 8 * 32 + 8: return read_as<T, D, 8, 8>(p, sms, s);
    case 8 * 32 + 4: return read_as<T, D, 8, 4>(p, sms, s);
    case 8 * 32 + 2: return read_as<T, D, 8, 2>(p, sms, s);
    case 4 * 32 + 8: return read_as<T, D, 4, 8>(p, sms, s);
    case 4 * 32 + 4: return read_as<T, D, 4, 4>(p, sms, s);
    case 4 * 32 + 2: return read_as<T, D, 4, 2>(p, sms, s);
    case 2 * 32 + 8: return read_as<T, D, 2, 8>(p, sms, s);
    case 2 * 32 + 4: return read_as<T, D, 2, 4>(p, sms, s);
    case 2 * 32 + 2: return read_as<T, D, 2, 2>(p, sms, s);
  }
  return read_as<T, D, 16, 16>(p, sms, s);
}

}  // namespace

cudaError_t paged_read_launch(const PagedReadParams& p, int D, int dtype, int sms, cudaStream_t s) {
  if (dtype == 0) return D == 64 ? read_pair<__half, 64>(p, sms, s) : read_pair<__half, 128>(p, sms, s);
  return D == 64 ? read_pair<__nv_bfloat16, 64>(p, sms, s) : read_pair<__nv_bfloat16, 128>(p, sms, s);
}

}  // namespace kvq
