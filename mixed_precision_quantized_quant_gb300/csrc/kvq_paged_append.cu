// Paged cache: append (rotation, rounding or quantization, store).
//
// Every byte moves once and little is computed, so the floor is the copy rate:
// q, k, v rows in; turned q rows and stored rows out.
//
// A row (one token, one head, D channels) is handled by D/16 neighbouring
// lanes with two 16-byte chunks each, so a warp holds a group of 4 or 8 rows.
// The two chunks are as far apart as the channels that turn together, so that
// no lane needs another's, and one store of a row's lanes covers whole 32-byte
// sectors.  Finding a token's place takes three dependent loads, which two
// forms of the kernel hide in two ways (see them below).
//
// Measured (GB300): 8,000 rows of 32 query and 8 kv heads in bf16 35 us, 84% of
// the copy rate; 9,500 rows of 64 and 8 heads into K4V2 72 us, 75%, bound by the
// issue slots (half used) and the latency of 24 warps an SM; one row 1.9 us.
#include "kvq_paged_rows.cuh"

namespace kvq {
namespace {

using namespace rows;

constexpr int kAppendPerSm = 3;  // CTAs of an SM

// ---------------------------------------------------------------- append

enum { kQueries, kKeys, kValues, kKinds };

constexpr int kDepth = 2;  // groups a warp has under way beside the one it works on

// cp.async of 16 bytes
__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ bool angles_ok(const PagedAppendParams& p, const void* a, size_t bytes) {  // (debug builds)
  return in_range(a, bytes, p.rope, p.rope + static_cast<int64_t>(p.rope_rows) * p.rope_dim, p.pool.err);
}

struct AppendSmem {
  RowPlace places[kRowTokens];
  uint4 ring[kRowThreads / 32][kDepth][2][32];  // each lane's two chunks of the groups under way
  float angles[kRowTokens][128];                // the tokens' cosines and sines
};

// What is done with a row once its two chunks are in registers.
template <typename T, int D, bool QUANT>
struct RowWork {
  static constexpr int LPR = D / 16, RPW = 32 / LPR;  // lanes of a row, rows of a group
  const PagedAppendParams& p;
  int j, sub, c0, c1;  // lane of the row, row of the group, the lane's chunks
  bool turns;

  __device__ __forceinline__ RowWork(const PagedAppendParams& p_, int lane) : p(p_), j(lane % LPR), sub(lane / LPR) {
    // a pair of chunks that turns together, or two that pass
    const int pairs = p.rope ? p.rope_dim / 16 : 0;
    turns = j < pairs;
    c0 = turns ? j : pairs + j;
    c1 = turns ? j + pairs : c0 + LPR - pairs;
  }
  template <int KIND>
  __device__ __forceinline__ const PagedRows& rows() const {
    return KIND == kQueries ? p.q : KIND == kKeys ? p.k : p.v;
  }
  template <int KIND>
  __device__ __forceinline__ int heads() const {
    return KIND == kQueries ? p.hq : p.hkv;
  }
  template <int KIND>
  __device__ __forceinline__ const T* row_of(int row, int head) const {
    return reinterpret_cast<const T*>(rows<KIND>().data) + row * rows<KIND>().token_stride +
           head * rows<KIND>().head_stride;
  }

  template <int KIND>
  __device__ __forceinline__ void one(int row, int head, const RowPlace& pl, const float* angles, uint4 a, uint4 b) const {
    f2 f[2][4];
    const bool turned = KIND != kValues && turns;
    if (turned || (QUANT && KIND != kQueries)) {
      unpack8<T>(a, f[0]);
      unpack8<T>(b, f[1]);
    }
    if (turned) {
      // angles of the half-split pairs, or of the lane's two chunks
      const float *t = angles, *u = t + p.rope_dim / 2;
      const int o0 = p.interleaved ? 4 * c0 : 8 * j, o1 = p.interleaved ? 4 * c1 : 8 * j + 4;
      float4 x = *reinterpret_cast<const float4*>(t + o0), y = *reinterpret_cast<const float4*>(t + o1);
      const f2 cs[4] = {f2_of(x.x, x.y), f2_of(x.z, x.w), f2_of(y.x, y.y), f2_of(y.z, y.w)};
      x = *reinterpret_cast<const float4*>(u + o0), y = *reinterpret_cast<const float4*>(u + o1);
      const f2 sn[4] = {f2_of(x.x, x.y), f2_of(x.z, x.w), f2_of(y.x, y.y), f2_of(y.z, y.w)};
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
    bool live = head < heads<KIND>();
    if constexpr (KIND == kQueries) {
      const T* y = reinterpret_cast<const T*>(p.qo.data) + row * p.qo.token_stride + head * p.qo.head_stride;
      live = live && rows_ok(p.qo, y, 2 * D, p.pool.err);
    } else {
      live = live && pool_ok(p.pool, p.pool.pages + pl.tile + head * p.pool.head_stride, p.pool.tile_bytes);
    }
    if constexpr (KIND == kQueries) {
      if (live) {
        T* y = reinterpret_cast<T*>(p.qo.data) + row * p.qo.token_stride + head * p.qo.head_stride;
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
    // by the reciprocal, rounded once: the scale's last bit may differ from a
    // division's, its error from the range over the codes hardly
    const float steps = bits == 8 ? 1.0f / 255.0f : bits == 4 ? 1.0f / 15.0f : 1.0f / 3.0f;
    const __half sh = __float2half_rn(__fmul_rn(__fsub_rn(mx, mn), steps));
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

// Streams a warp's pairs: their rows are fetched kDepth pairs ahead.
template <typename T, int D, bool QUANT>
struct Appender {
  using W = RowWork<T, D, QUANT>;
  const W& w;
  AppendSmem& sm;
  int row0, count, lane, warp;
  // the next pair to fetch
  int kind;
  Run ahead;

  __device__ __forceinline__ Run run(int k) const {
    const int h = k == kQueries ? w.p.hq : w.p.hkv;
    return h ? Run(count, (h + W::RPW - 1) / W::RPW, k == kValues ? (warp + 4) & 7 : warp) : Run(0, 1, 0);
  }
  // starts the copy of the lane's chunks of the pair's row into `slot`
  template <int KIND>
  __device__ __forceinline__ void load(int slot) const {
    const int head = ahead.g * W::RPW + w.sub;
    if (head >= w.template heads<KIND>()) return;
    const T* x = w.template row_of<KIND>(row0 + ahead.tk, head);
    if (!rows_ok(w.template rows<KIND>(), x, 2 * D, w.p.pool.err)) return;
    uint4* y = &sm.ring[warp][slot][0][lane];
    if (w.p.vec) {
      copy16(y, x + 8 * w.c0);
      copy16(y + 32, x + 8 * w.c1);
    } else {
      load8(x + 8 * w.c0, 0, y[0]);
      load8(x + 8 * w.c1, 0, y[32]);
    }
  }
  __device__ __forceinline__ void fetch(int slot) {
    while (kind < kKinds && ahead.left <= 0) {
      ++kind;
      if (kind < kKinds) ahead = run(kind);
    }
    if (kind == kQueries) load<kQueries>(slot);
    if (kind == kKeys) load<kKeys>(slot);
    if (kind == kValues) load<kValues>(slot);
    if (kind < kKinds) ahead.next();
    copy_commit();
  }

  // The warp's pairs of one kind, in the order they are fetched in.
  template <int KIND>
  __device__ __forceinline__ void work(int& slot) {
    Run r = run(KIND);
#pragma unroll 1
    for (; r.left > 0; r.next()) {
      copy_wait<kDepth - 1>();
      const uint4 a = sm.ring[warp][slot][0][lane], b = sm.ring[warp][slot][1][lane];
      fetch(slot);
      slot = slot + 1 == kDepth ? 0 : slot + 1;
      const RowPlace pl = sm.places[r.tk];
      if (pl.ok) w.template one<KIND>(row0 + r.tk, r.g * W::RPW + w.sub, pl, sm.angles[r.tk], a, b);
    }
  }
};

// Many tokens: a CTA takes up to 32.
template <typename T, int D, bool QUANT>
__global__ void __launch_bounds__(kRowThreads, kAppendPerSm) paged_append_kernel(const __grid_constant__ PagedAppendParams p) {
  __shared__ __align__(16) AppendSmem sm;
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row0 = blockIdx.x * p.tokens;  // (n is at most INT_MAX - 31)
  const int count = p.n - row0 < p.tokens ? p.n - row0 : p.tokens;
  const RowWork<T, D, QUANT> work(p, lane);
  Appender<T, D, QUANT> ap = {work, sm, row0, count, lane, warp, kQueries, Run(0, 1, 0)};
  ap.ahead = ap.run(kQueries);
#pragma unroll
  for (int i = 0; i < kDepth; ++i) ap.fetch(i);  // under way while the places are found
  if (warp == 0) {
    const RowPlace r = find_places(p.batch, p.pool, row0, count, p.rope, p.positions, p.rope_rows, lane);
    if (lane < count) sm.places[lane] = r;
  }
  __syncthreads();
  if (p.rope) {  // every token's angles once, for all its rows
    const int quads = p.rope_dim / 4;
    for (int tk = warp; tk < count; tk += kRowThreads / 32)
      if (sm.places[tk].ok && lane < quads) {
        const float4* x = reinterpret_cast<const float4*>(p.rope + static_cast<int64_t>(sm.places[tk].rope) * p.rope_dim) + lane;
        if (angles_ok(p, x, 16)) *reinterpret_cast<float4*>(&sm.angles[tk][4 * lane]) = __ldg(x);
      }
    __syncthreads();
  }
  int slot = 0;
  ap.template work<kQueries>(slot);
  ap.template work<kKeys>(slot);
  ap.template work<kValues>(slot);
}

// Few tokens, where latency counts: a CTA takes one, a warp one group of its
// rows (more where there are over 32), each finding the token's place by
// itself while its row is on its way; no shared memory and no barrier.  Against
// the form above, us (bf16, 32 query and 8 kv heads, D = 128): 1 row 2.2 and 3.6,
// 256 rows 4.5 and 5.0, 456 rows 4.6 and 5.1, 912 rows 8.2 and 6.2; codes (K4V2,
// with the read back): 1 row 4.8 and 6.2, 256 rows 7.5 and 9.1, 456 rows 10.6
// and 9.3.
template <typename T, int D, bool QUANT>
__global__ void __launch_bounds__(1024) paged_append_few_kernel(const __grid_constant__ PagedAppendParams p) {
  using W = RowWork<T, D, QUANT>;
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, row = blockIdx.x;
  const W w(p, lane);
  const int gq = (p.hq + W::RPW - 1) / W::RPW, gk = (p.hkv + W::RPW - 1) / W::RPW;
  RowPlace pl;
  bool found = false;
  for (int g = threadIdx.x >> 5; g < gq + 2 * gk; g += blockDim.x >> 5) {
    const bool q = g < gq, k = g < gq + gk;
    const int head = (q ? g : k ? g - gq : g - gq - gk) * W::RPW + w.sub;
    uint4 a = make_uint4(0, 0, 0, 0), b = a;
    if (head < (q ? p.hq : p.hkv)) {
      const T* x = q ? w.template row_of<kQueries>(row, head)
                     : k ? w.template row_of<kKeys>(row, head) : w.template row_of<kValues>(row, head);
      if (rows_ok(q ? p.q : k ? p.k : p.v, x, 2 * D, p.pool.err)) {
        load8(x + 8 * w.c0, p.vec, a);
        load8(x + 8 * w.c1, p.vec, b);
      }
    }
    if (!found) {
      pl = find_places(p.batch, p.pool, row, 1, p.rope, p.positions, p.rope_rows, lane);
      pl.tile = __shfl_sync(0xffffffffu, pl.tile, 0);
      pl.tok = __shfl_sync(0xffffffffu, pl.tok, 0);
      pl.rope = __shfl_sync(0xffffffffu, pl.rope, 0);
      pl.ok = __shfl_sync(0xffffffffu, pl.ok, 0);
      found = true;
    }
    if (!pl.ok) return;
    const float* angles = p.rope ? p.rope + static_cast<int64_t>(pl.rope) * p.rope_dim : nullptr;
    if (angles && !angles_ok(p, angles, 4 * p.rope_dim)) return;
    if (q)
      w.template one<kQueries>(row, head, pl, angles, a, b);
    else if (k)
      w.template one<kKeys>(row, head, pl, angles, a, b);
    else
      w.template one<kValues>(row, head, pl, angles, a, b);
  }
}

template <typename T, int D>
cudaError_t append_as(PagedAppendParams p, int sms, cudaStream_t s) {
  p.tokens = cta_tokens(p.n, sms, kAppendPerSm);
  const dim3 grid(static_cast<unsigned>((p.n - 1) / p.tokens + 1));
  if (p.n <= sms * (p.pool.kb == 16 ? 3 : 2)) {  // (p.tokens is 1)
    constexpr int RPW = 32 / (D / 16);
    const int groups = (p.hq + RPW - 1) / RPW + 2 * ((p.hkv + RPW - 1) / RPW);
    const int threads = groups < 32 ? 32 * groups : 1024;
    return p.pool.kb == 16 ? launch_pdl(paged_append_few_kernel<T, D, false>, p, grid, threads, s)
                           : launch_pdl(paged_append_few_kernel<T, D, true>, p, grid, threads, s);
  }
  return p.pool.kb == 16 ? launch_pdl(paged_append_kernel<T, D, false>, p, grid, kRowThreads, s)
                         : launch_pdl(paged_append_kernel<T, D, true>, p, grid, kRowThreads, s);
}

}  // namespace

cudaError_t paged_append_launch(const PagedAppendParams& p, int D, int dtype, int sms, cudaStream_t s) {
  if (dtype == 0) return D == 64 ? append_as<__half, 64>(p, sms, s) : append_as<__half, 128>(p, sms, s);
  return D == 64 ? append_as<__nv_bfloat16, 64>(p, sms, s) : append_as<__nv_bfloat16, 128>(p, sms, s);
}

}  // namespace kvq
