// Paged cache: parameter blocks of its kernels and the layout of a tile
// (16 consecutive tokens of one kv head), shared by append, read and attention.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kvq_device.cuh"

namespace kvq {

// further device error codes (see kvq_device.cuh)
constexpr int32_t kErrBadPage = 4;
constexpr int32_t kErrBadPosition = 5;

constexpr int kTile = 16;  // tokens of a tile: the K extent of one tensor-core step

struct PagedBatch {
  const int32_t* table;   // [seqs][max_pages], rows table_stride apart
  int64_t table_stride;
  const int32_t* lens;
  const int32_t* cu;      // [seqs + 1] or null
  int seqs;
  int max_pages;
};

struct PagedPool {
  uint8_t* pages;
  int64_t page_stride;    // bytes from a page to the next
  int64_t head_stride;    // bytes from a kv head of a page to the next
  int tile_bytes;
  int num_pages;
  int page_shift;         // log2(page_size)
  int kb, vb;
  int32_t* err;
  const uint8_t* hi;      // end of the layer's pages (checked in debug builds)
};

struct PagedRows {
  uint8_t* data;
  int64_t token_stride;   // elements
  int64_t head_stride;
  const uint8_t *lo, *hi; // where the rows lie (checked in debug builds)
};

struct PagedAppendParams {
  PagedBatch batch;
  PagedPool pool;
  PagedRows k, v, q, qo;
  const float* rope;      // null: no rotation
  const int32_t* positions;
  int rope_rows, rope_dim, interleaved;
  int n, hq, hkv;         // hq = 0: no queries
  int vec;                // every row is 16-byte aligned
  int tokens;             // tokens of a CTA (set at launch)
};

struct PagedReadParams {
  PagedBatch batch;
  PagedPool pool;
  PagedRows k, v;
  int n, hkv;
  int vec;
  int tokens;
};

struct PagedAttnParams {
  PagedBatch batch;
  PagedPool pool;
  PagedRows q;
  void* out;              // [seqs][hq][D]
  float* lse;             // [seqs][hq] or null
  float alpha;            // scale * log2(e)
  int window;             // 0: all
  int hkv, gqa;
  int q_vec;              // every row of q is 16-byte aligned
  uint8_t* ws;             // what the join needs of every unit, then partial results
  int64_t ws_partials;    // where those start
  const uint8_t* ws_hi;   // end of the workspace (checked in debug builds)
  int solo;               // a CTA for each unit, no join (set at launch)
  int ctas;               // of the attention kernel (set at launch)
};

// ---------------------------------------------------------------- debug checks

// in_range (kvq_device.cuh) on what these calls were given; `true` in a release
// build.  A miss is reported, and the access skipped.
__device__ __forceinline__ bool pool_ok(const PagedPool& p, const void* a, size_t bytes) {
  return in_range(a, bytes, p.pages, p.hi, p.err);
}
__device__ __forceinline__ bool rows_ok(const PagedRows& r, const void* a, size_t bytes, int32_t* err) {
  return in_range(a, bytes, r.lo, r.hi, err);
}
__device__ __forceinline__ bool table_ok(const PagedBatch& b, const int32_t* a, int32_t* err) {
  return in_range(a, 4, b.table, b.table + (b.seqs - 1) * b.table_stride + b.max_pages, err);
}

// ---------------------------------------------------------------- tile layout

// Rows of a 16-bit tile keep the 16-byte chunk c of token i at c ^ (i & 7):
// eight tokens' rows of one ldmatrix then fall on eight bank groups.
__host__ __device__ constexpr int tile_chunk16(int c, int i) { return c ^ (i & 7); }

// Row of token i's key codes and scales in a quantized tile: the order in
// which the tensor-core fragments of the attention take the tokens (row r of
// an MMA is token r(i)^-1), so that a thread's four value tokens
// t, t+4, t+8, t+12 lie in four consecutive-row reads without bank conflicts.
__host__ __device__ constexpr int tile_key_row(int i) { return 2 * (i & 3) + ((i >> 2) & 1) + (i & 8); }
// its inverse: the token of MMA row r
__host__ __device__ constexpr int tile_row_token(int r) { return ((r >> 1) & 3) + 4 * (r & 1) + (r & 8); }

// XOR on the byte offset inside a key code row at row r / a value code row of
// token i (see kvq_paged_view in kvq.h)
__host__ __device__ constexpr int tile_key_xor(int row_bytes, int r) { return row_bytes == 128 ? (r & 1) << 6 : 0; }
__host__ __device__ constexpr int tile_val_xor(int row_bytes, int i) {
  return row_bytes == 128 ? (i & 3) << 5 : (row_bytes == 64 ? (i & 2) << 4 : 0);
}

__host__ __device__ constexpr int paged_tile_bytes(int D, int kb, int vb) {
  return 2 * D * (kb + vb) + (kb == 16 ? 0 : 128);
}

// ---------------------------------------------------------------- types

template <typename T>
struct Num;
template <>
struct Num<__half> {
  static __device__ __forceinline__ float to(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half from(float x) { return __float2half_rn(x); }
};
template <>
struct Num<__nv_bfloat16> {
  static __device__ __forceinline__ float to(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 from(float x) { return __float2bfloat16_rn(x); }
};

// ---------------------------------------------------------------- host entry points

cudaError_t paged_append_launch(const PagedAppendParams& p, int D, int dtype, int sms, cudaStream_t s);
cudaError_t paged_read_launch(const PagedReadParams& p, int D, int dtype, int sms, cudaStream_t s);
// Makes a layer's attention kernel ready on the current device; once, at creation.
cudaError_t paged_attn_prepare(int kb, int vb, int D, int dtype);
cudaError_t paged_attn_launch(PagedAttnParams p, int D, int dtype, int sms, cudaStream_t s);
size_t paged_attn_workspace(int D, int hkv, int seqs, int sms);

}  // namespace kvq
