// Paged cache: append (rotation, rounding or quantization, store).
//
// Every byte moves once and little is computed, so the floor is the copy rate:
// q, k, v rows in; turned q rows and stored rows out.
//
// A row (one token, one head, D channels) is handled by D/16 neighbouring
// lanes with two 16-byte chunks each, so a warp holds a group of 4 or 8 rows.
// The two chunks lie D/2 channels apart (in an append: as far apart as the
// channels that turn together, so that no lane needs another's), and one store
// of a row's lanes covers whole 32-byte sectors.  A CTA takes up to 32
// tokens: its first warp finds their places, a lane each (three dependent loads, so
// they are paid once a CTA); then each of its eight warps takes a run of the
// (token, group) pairs of the queries, of the keys and of the values.
#include "kvq_paged_rows.cuh"

namespace kvq {
namespace {

using namespace rows;

constexpr int kAppendPerSm = 3;  // CTAs of an SM

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
__global__ void __launch_bounds__(kRowThreads, kAppendPerSm) paged_append_kernel(const __grid_constant__ PagedAppendParams p) {
  using A = Appender<T, D, QUANT>;
  __shared__ RowPlace places[kRowTokens];
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int j = lane % A::LPR;
  const int pairs = p.rope ? p.rope_dim / 16 : 0;
  const bool turns = j < pairs;
  // the lane's chunks: a pair that turns together, or two that pass
  const int c0 = turns ? j : pairs + j, c1 = turns ? j + pairs : c0 + A::LPR - pairs;
  const int row0 = blockIdx.x * p.tokens;  // (n is at most INT_MAX - 31)
  const int count = p.n - row0 < p.tokens ? p.n - row0 : p.tokens;
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

template <typename T, int D>
cudaError_t append_as(PagedAppendParams p, int sms, cudaStream_t s) {
  p.tokens = cta_tokens(p.n, sms, kAppendPerSm);
  const dim3 grid(static_cast<unsigned>((p.n - 1) / p.tokens + 1));
  return p.pool.kb == 16 ? launch_pdl(paged_append_kernel<T, D, false>, p, grid, kRowThreads, s)
                         : launch_pdl(paged_append_kernel<T, D, true>, p, grid, kRowThreads, s);
}

}  // namespace

cudaError_t paged_append_launch(const PagedAppendParams& p, int D, int dtype, int sms, cudaStream_t s) {
  if (dtype == 0) return D == 64 ? append_as<__half, 64>(p, sms, s) : append_as<__half, 128>(p, sms, s);
  return D == 64 ? append_as<__nv_bfloat16, 64>(p, sms, s) : append_as<__nv_bfloat16, 128>(p, sms, s);
}

}  // namespace kvq
