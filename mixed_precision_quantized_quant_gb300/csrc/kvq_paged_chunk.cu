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
#include "kvq_paged_chunk.cuh"

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
__global__ void __launch_bounds__(32 * kChunkWarps) paged_chunk_plain_kernel(const __grid_constant__ PagedChunkParams p) {
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

using chunk::Launch;
using chunk::Shape;

constexpr int64_t kNoteBytes(int sms) { return (sms * static_cast<int64_t>(sizeof(chunk::Note)) + 255) / 256 * 256; }

int slot_rows(int64_t pairs) { return static_cast<int>(pairs < 256 ? (pairs + 31) / 32 * 32 : 256); }

int64_t packed_at(int D, int64_t pairs, int sms) {
  return kNoteBytes(sms) + 2LL * sms * slot_rows(pairs) * (D + 2) * 4;
}

template <typename F>
cudaError_t big_smem(F fn, int bytes) {
  return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <typename T, int D, int NQ, bool PROMPT>
cudaError_t launch_as(Launch& a, int sms, cudaStream_t s) {
  using S = Shape<D, NQ>;
  const PagedChunkParams& p = a.p;
  // no more CTAs than the work could give something to do
  const int64_t pairs = static_cast<int64_t>(p.n) * p.gqa;
  const int64_t items = (pairs / S::R + (p.batch.seqs < p.n ? p.batch.seqs : p.n)) * p.hkv;
  const int64_t longest = PROMPT ? p.n : static_cast<int64_t>(p.batch.max_pages) << p.pool.page_shift;
  const double work = static_cast<double>(items) * static_cast<double>(longest / chunk::kTokens + 1 + chunk::kStart);
  const double most = work / (3 * chunk::kStart) + 1;
  a.grid = most < sms ? static_cast<int>(most) : sms;
  const auto fn = chunk::paged_chunk_kernel<T, D, NQ, PROMPT>;
  cudaError_t e = big_smem(fn, S::smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.grid));
  cfg.blockDim = dim3(S::threads);
  cfg.dynamicSmemBytes = S::smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, fn, a);
  if (e != cudaSuccess) return e;
  if (a.grid == 1) return cudaSuccess;
  return rows::launch_pdl(chunk::paged_chunk_join_kernel<T, D>, a,
                          dim3(static_cast<unsigned>(a.grid), static_cast<unsigned>(a.slot_rows / 32)), 256, s);
}

// 16-bit rows [n][heads][D] as boxes of 128 tokens of one half of a head's channels.
bool rows_map(CUtensorMap* m, TensorMapEncode enc, const void* data, int64_t ts, int64_t hs, int n, int heads, int D, int dtype) {
  if (n == 1) ts = D;
  if (heads == 1) hs = D;
  if ((reinterpret_cast<uintptr_t>(data) & 15u) || ts % 8 || hs % 8 || ts <= 0 || hs <= 0 || ts >= int64_t{1} << 38 ||
      hs >= int64_t{1} << 38)
    return false;
  const cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(n), static_cast<cuuint64_t>(D / 64), static_cast<cuuint64_t>(heads)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(2 * ts), 128, static_cast<cuuint64_t>(2 * hs)};
  const cuuint32_t box[4] = {64, 128, 1, 1}, one[4] = {1, 1, 1, 1};
  return enc(m, dtype == 0 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
             const_cast<void*>(data), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D>
cudaError_t chunk_as(const PagedChunkParams& p, const CUtensorMap* pages, TensorMapEncode enc, int dtype, int sms, cudaStream_t s) {
  Launch a;
  a.p = p;
  const int64_t pairs = static_cast<int64_t>(p.n) * p.gqa;
  a.slot_rows = slot_rows(pairs);
  a.partials = kNoteBytes(sms);
  const bool wide = pairs > static_cast<int64_t>(chunk::kM) * p.batch.seqs;
  if (!p.prompt) {
    if (p.pool.kb != 16) {
      paged_chunk_plain_kernel<T, D><<<static_cast<unsigned>(p.n), 32 * kChunkWarps, 0, s>>>(p);
      return cudaGetLastError();
    }
    a.km = a.vm = *pages;
    return wide ? launch_as<T, D, 2, false>(a, sms, s) : launch_as<T, D, 1, false>(a, sms, s);
  }
  if (!rows_map(&a.km, enc, p.k.data, p.k.token_stride, p.k.head_stride, p.n, p.hkv, D, dtype) ||
      !rows_map(&a.vm, enc, p.v.data, p.v.token_stride, p.v.head_stride, p.n, p.hkv, D, dtype)) {
    uint8_t* to = p.ws + packed_at(D, pairs, sms);
    const int64_t bytes = 2LL * p.n * p.hkv * D;
    cudaError_t e;
    const int64_t blocks = (bytes / 8 + 255) / 256;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks < 8LL * sms ? blocks : 8LL * sms));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    if ((e = cudaLaunchKernelEx(&cfg, chunk::pack_rows_kernel<D>, p, to)) != cudaSuccess) return e;
    a.p.k.data = to;
    a.p.v.data = to + bytes;
    a.p.k.token_stride = a.p.v.token_stride = static_cast<int64_t>(p.hkv) * D;
    a.p.k.head_stride = a.p.v.head_stride = D;
    if (!rows_map(&a.km, enc, a.p.k.data, a.p.k.token_stride, D, p.n, p.hkv, D, dtype) ||
        !rows_map(&a.vm, enc, a.p.v.data, a.p.v.token_stride, D, p.n, p.hkv, D, dtype))
      return cudaErrorInvalidValue;
  }
  return wide ? launch_as<T, D, 2, true>(a, sms, s) : launch_as<T, D, 1, true>(a, sms, s);
}

}  // namespace

cudaError_t paged_chunk_launch(const PagedChunkParams& p, const CUtensorMap* pages, TensorMapEncode enc, int D, int dtype,
                               int sms, cudaStream_t s) {
  if (dtype == 0)
    return D == 64 ? chunk_as<__half, 64>(p, pages, enc, dtype, sms, s) : chunk_as<__half, 128>(p, pages, enc, dtype, sms, s);
  return D == 64 ? chunk_as<__nv_bfloat16, 64>(p, pages, enc, dtype, sms, s)
                 : chunk_as<__nv_bfloat16, 128>(p, pages, enc, dtype, sms, s);
}

// Notes, partial results, then room for a prompt's keys and values (see pack_rows_kernel).
size_t paged_chunk_workspace(int D, int hkv, int gqa, int n, int sms) {
  return static_cast<size_t>(packed_at(D, static_cast<int64_t>(n) * gqa, sms) + 4LL * n * hkv * D);
}

// A layer of 16-bit rows as boxes of one page: a half of a kv head's channels of its keys, or values.
bool paged_chunk_map(CUtensorMap* m, TensorMapEncode enc, void* pages, int64_t tiles, int page_size, int D, int dtype) {
  if (tiles > int64_t{1} << 31) return false;
  const cuuint64_t row = 2 * D;
  const cuuint64_t dims[5] = {64, 16, static_cast<cuuint64_t>(tiles), static_cast<cuuint64_t>(D / 64), 2};
  const cuuint64_t strides[4] = {row, 32 * row, 128, 16 * row};
  const cuuint32_t box[5] = {64, 16, static_cast<cuuint32_t>(page_size / 16), 1, 1}, one[5] = {1, 1, 1, 1, 1};
  return enc(m, dtype == 0 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, pages, dims, strides,
             box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace kvq
