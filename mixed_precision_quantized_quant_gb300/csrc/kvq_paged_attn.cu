// Paged cache: attention of one query token per sequence.
//
// One CTA per (sequence, kv head); its warps take every fourth token, a lane
// D/32 channels of it, with a running maximum and sum per query head.
#include "kvq_paged.cuh"

namespace kvq {
namespace {

constexpr int kWarps = 4;

template <typename T, int D>
__device__ __forceinline__ float tile_value(const uint8_t* tile, int kb, int vb, bool value, int tok, int c) {
  const int bits = value ? vb : kb;
  if (bits == 16) {
    const uint8_t* x = tile + (value ? 32 * D : 0) + tok * 2 * D + 16 * tile_chunk16(c / 8, tok) + 2 * (c % 8);
    return Num<T>::to(*reinterpret_cast<const T*>(x));
  }
  const int rk = D * kb / 8, rv = D * vb / 8, kr = tile_key_row(tok);
  const uint8_t* row = value ? tile + 16 * rk + tok * rv : tile + kr * rk;
  const int byte = (c * bits / 8) ^ (value ? tile_val_xor(rv, tok) : tile_key_xor(rk, kr));
  const float code = static_cast<float>((row[byte] >> (c * bits % 8)) & ((1 << bits) - 1));
  const __half2 sz = *reinterpret_cast<const __half2*>(tile + 16 * (rk + rv) + kr * 8 + (value ? 4 : 0));
  return code * __low2float(sz) + __high2float(sz);
}

template <typename T, int D>
__global__ void __launch_bounds__(32 * kWarps) paged_attn_kernel(PagedAttnParams p) {
  constexpr int C = D / 32;
  __shared__ float o_s[kWarps][8][D];
  __shared__ float m_s[kWarps][8], l_s[kWarps][8];
  grid_dep_wait();
  grid_dep_launch();
  const int seq = blockIdx.y, head = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t len = p.batch.lens[seq];
  const int64_t room = static_cast<int64_t>(p.batch.max_pages) << p.pool.page_shift;
  if (len < 0 || len > room) {
    if (threadIdx.x == 0) atomicExch(p.pool.err, kErrBadState);
    len = len < 0 ? 0 : room;
  }
  const int64_t first = p.window > 0 && len > p.window ? len - p.window : 0;
  float q[8][C], o[8][C], m[8], l[8];
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    m[g] = -INFINITY;
    l[g] = 0.0f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      o[g][i] = 0.0f;
      q[g][i] = g < p.gqa ? Num<T>::to(reinterpret_cast<const T*>(p.q.data)[seq * p.q.token_stride +
                                                                         (head * p.gqa + g) * p.q.head_stride +
                                                                         lane * C + i])
                          : 0.0f;
    }
  }
  for (int64_t t = first + warp; t < len; t += kWarps) {
    int page = p.batch.table[seq * p.batch.table_stride + (t >> p.pool.page_shift)];
    if (page < 0 || page >= p.pool.num_pages) {
      if (lane == 0) atomicExch(p.pool.err, kErrBadPage);
      page = 0;
    }
    const int in_page = static_cast<int>(t) & ((1 << p.pool.page_shift) - 1);
    const uint8_t* tile = p.pool.pages + page * p.pool.page_stride + head * p.pool.head_stride +
                          static_cast<int64_t>(in_page / kTile) * p.pool.tile_bytes;
    float k[C], v[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
      k[i] = tile_value<T, D>(tile, p.pool.kb, p.pool.vb, false, in_page % kTile, lane * C + i);
      v[i] = tile_value<T, D>(tile, p.pool.kb, p.pool.vb, true, in_page % kTile, lane * C + i);
    }
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      if (g >= p.gqa) break;
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < C; ++i) s += q[g][i] * k[i];
#pragma unroll
      for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
      s *= p.alpha;
      const float mn = fmaxf(m[g], s);
      const float old = m[g] == mn ? 1.0f : exp2f(m[g] - mn), e = exp2f(s - mn);
      m[g] = mn;
      l[g] = l[g] * old + e;
#pragma unroll
      for (int i = 0; i < C; ++i) o[g][i] = o[g][i] * old + e * v[i];
    }
  }
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    if (lane == 0) {
      m_s[warp][g] = m[g];
      l_s[warp][g] = l[g];
    }
#pragma unroll
    for (int i = 0; i < C; ++i) o_s[warp][g][lane * C + i] = o[g][i];
  }
  __syncthreads();
  for (int x = threadIdx.x; x < p.gqa * D; x += 32 * kWarps) {
    const int g = x / D, c = x % D;
    float mx = -INFINITY;
    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, m_s[w][g]);
    float sum = 0.0f, acc = 0.0f;
    for (int w = 0; w < kWarps; ++w) {
      const float f = l_s[w][g] > 0.0f ? exp2f(m_s[w][g] - mx) : 0.0f;
      sum += f * l_s[w][g];
      acc += f * o_s[w][g][c];
    }
    const int64_t row = static_cast<int64_t>(seq) * p.hkv * p.gqa + head * p.gqa + g;
    reinterpret_cast<T*>(p.out)[row * D + c] = Num<T>::from(len > first ? acc / sum : 0.0f);
    if (p.lse && c == 0) p.lse[row] = len > first ? (mx + log2f(sum)) * 0.69314718f : -INFINITY;
  }
}

template <typename T, int D>
cudaError_t launch(const PagedAttnParams& p, cudaStream_t s) {
  paged_attn_kernel<T, D><<<dim3(p.hkv, p.batch.seqs), 32 * kWarps, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t paged_attn_launch(const PagedAttnParams& p, int D, int dtype, int sms, cudaStream_t s) {
  if (dtype == 0) return D == 64 ? launch<__half, 64>(p, s) : launch<__half, 128>(p, s);
  return D == 64 ? launch<__nv_bfloat16, 64>(p, s) : launch<__nv_bfloat16, 128>(p, s);
}

size_t paged_attn_workspace(int D, int gqa, int hkv, int seqs, int sms) { return 256; }

}  // namespace kvq
