// Paged cache: causal attention of runs of new tokens, over the pages or over
// rows of their own.
//
// For a row at position p and a query head of kv head g, over the positions t it sees:
//   s_t = alpha q.k_t (base 2), m = max s_t, l = sum 2^(s_t - m),
//   out = sum 2^(s_t - m) v_t / l, lse = (m + log2 l) ln 2.
//
// The plainest form: a CTA takes a row, a warp one query head at a time, its
// lanes D / 32 channels each, one position after another with the running
// maximum and sum.
#include "kvq_paged_rows.cuh"

namespace kvq {
namespace {

using namespace rows;

constexpr int kChunkWarps = 4;

// What a row attends: positions lo .. p; key and value of position t are in
// row t + shift of the call's tensors (prompts), or in the pages of `table`.
struct Seen {
  const int32_t* table;
  int64_t shift;
  int lo, p, ok;
};

// The row's sequence is the number of ends at or before it, as for an append.
__device__ Seen find_row(const PagedChunkParams& p, int row, int lane) {
  Seen r = {nullptr, 0, 0, 0, 0};
  const PagedBatch& b = p.batch;
  int seq = row;
  int64_t first = row, end = row + 1;
  if (b.cu) {
    int c = 0;
    for (int s = lane; s < b.seqs; s += 32) c += b.cu[s + 1] <= row;
    seq = __reduce_add_sync(0xffffffffu, c);
    if (seq >= b.seqs || row < b.cu[0]) return r;
    first = b.cu[seq];
    end = b.cu[seq + 1];
    if (row < first || row >= end) {  // not ascending
      if (lane == 0) atomicExch(p.pool.err, kErrBadState);
      return r;
    }
  }
  int64_t pos = row - first;
  if (p.prompt) {
    if (first < 0 || end > p.n) {  // rows that are not there
      if (lane == 0) atomicExch(p.pool.err, kErrBadState);
      return r;
    }
    r.shift = first;
  } else {
    const int len = b.lens[seq];
    if (!b.cu && len == 0) return r;
    pos = len - (end - row);
    if (len - (end - first) < 0 || len > static_cast<int64_t>(b.max_pages) << p.pool.page_shift) {
      if (lane == 0) atomicExch(p.pool.err, kErrBadState);
      return r;
    }
    r.table = b.table + seq * b.table_stride;
  }
  r.p = static_cast<int>(pos);
  r.lo = p.window && pos >= p.window ? static_cast<int>(pos) - p.window + 1 : 0;
  r.ok = 1;
  return r;
}

// A lane's channels of a stored row, in fp32.
template <typename T, int C>
__device__ void stored(const uint8_t* tile, int tok, bool value, int kb, int vb, int D, int c0, float (&x)[C]) {
  const int bits = value ? vb : kb;
  if (bits == 16) {
    const uint8_t* row = tile + (value ? 32 * D : 0) + tok * 2 * D;
    for (int i = 0; i < C; ++i) {
      const int c = c0 + i;
      x[i] = Num<T>::to(*reinterpret_cast<const T*>(row + 16 * tile_chunk16(c / 8, tok) + c % 8 * 2));
    }
    return;
  }
  const int rk = D / 8 * kb, rv = D / 8 * vb, kr = tile_key_row(tok);
  const uint8_t* row = tile + (value ? 16 * rk + tok * rv : kr * rk);
  const int xr = value ? tile_val_xor(rv, tok) : tile_key_xor(rk, kr);
  const __half2 sz = *reinterpret_cast<const __half2*>(tile + 16 * (rk + rv) + kr * 8 + (value ? 4 : 0));
  const float s = __low2float(sz), z = __high2float(sz);
  for (int i = 0; i < C; ++i) {
    const int bit = (c0 + i) * bits;
    x[i] = fmaf(static_cast<float>((row[(bit / 8) ^ xr] >> (bit % 8)) & ((1 << bits) - 1)), s, z);
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(32 * kChunkWarps) paged_chunk_kernel(const __grid_constant__ PagedChunkParams p) {
  constexpr int C = D / 32;
  const int lane = threadIdx.x & 31, row = blockIdx.x, c0 = lane * C;
  const Seen r = find_row(p, row, lane);
  if (!r.ok) return;
  for (int h = threadIdx.x >> 5; h < p.hkv * p.gqa; h += kChunkWarps) {
    const int g = h / p.gqa;
    float q[C], o[C], m = -INFINITY, l = 0.0f;
    const T* qr = reinterpret_cast<const T*>(p.q.data) + row * p.q.token_stride + h * p.q.head_stride;
    for (int i = 0; i < C; ++i) q[i] = Num<T>::to(qr[c0 + i]), o[i] = 0.0f;
    for (int t = r.lo; t <= r.p; ++t) {
      float k[C], v[C];
      if (p.prompt) {
        const T* kr = reinterpret_cast<const T*>(p.k.data) + (t + r.shift) * p.k.token_stride + g * p.k.head_stride;
        const T* vr = reinterpret_cast<const T*>(p.v.data) + (t + r.shift) * p.v.token_stride + g * p.v.head_stride;
        for (int i = 0; i < C; ++i) k[i] = Num<T>::to(kr[c0 + i]), v[i] = Num<T>::to(vr[c0 + i]);
      } else {
        const int page = r.table[t >> p.pool.page_shift];
        if (page < 0 || page >= p.pool.num_pages) {
          if (lane == 0) atomicExch(p.pool.err, kErrBadPage);
          continue;
        }
        const int in_page = t & ((1 << p.pool.page_shift) - 1);
        const uint8_t* tile = p.pool.pages + page * p.pool.page_stride + g * p.pool.head_stride +
                              static_cast<int64_t>(in_page / kTile) * p.pool.tile_bytes;
        if (!pool_ok(p.pool, tile, p.pool.tile_bytes)) continue;
        stored<T>(tile, in_page % kTile, false, p.pool.kb, p.pool.vb, D, c0, k);
        stored<T>(tile, in_page % kTile, true, p.pool.kb, p.pool.vb, D, c0, v);
      }
      float s = 0.0f;
      for (int i = 0; i < C; ++i) s = fmaf(q[i], k[i], s);
      for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
      s *= p.alpha;
      if (s == -INFINITY) continue;
      const float top = fmaxf(m, s), f = exp2f(m - top), w = exp2f(s - top);
      m = top;
      l = fmaf(l, f, w);
      for (int i = 0; i < C; ++i) o[i] = fmaf(o[i], f, w * v[i]);
    }
    const int64_t at = static_cast<int64_t>(row) * p.hkv * p.gqa + h;
    const float inv = l > 0.0f ? 1.0f / l : l == 0.0f ? 0.0f : l;
    T* y = static_cast<T*>(p.out) + at * D;
    for (int i = 0; i < C; ++i) y[c0 + i] = Num<T>::from(l == 0.0f ? 0.0f : o[i] * inv);
    if (p.lse && lane == 0) p.lse[at] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
  }
}

}  // namespace

cudaError_t paged_chunk_launch(const PagedChunkParams& p, int D, int dtype, int, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(p.n));
  if (dtype == 0)
    D == 64 ? paged_chunk_kernel<__half, 64><<<grid, 32 * kChunkWarps, 0, s>>>(p)
            : paged_chunk_kernel<__half, 128><<<grid, 32 * kChunkWarps, 0, s>>>(p);
  else
    D == 64 ? paged_chunk_kernel<__nv_bfloat16, 64><<<grid, 32 * kChunkWarps, 0, s>>>(p)
            : paged_chunk_kernel<__nv_bfloat16, 128><<<grid, 32 * kChunkWarps, 0, s>>>(p);
  return cudaGetLastError();
}

size_t paged_chunk_workspace(int, int, int, int, int, int) { return 256; }

}  // namespace kvq
