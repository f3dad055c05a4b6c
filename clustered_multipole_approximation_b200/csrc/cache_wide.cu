// Attention over the paged cache in fp32: fp32 queries, or an fp32 cache.
//
// One CTA of 256 threads takes a tile of R packed rows (64, or 16 where the
// call has no more) and one split of its keys, 64 at a time: K and V of a
// block stand in shared memory as fp32 (8-bit rows times their scale), the
// next block's are on their way in registers.  Thread (y, x) of 16 x 16 forms
// S of rows y R / 16 .. and keys x + 16 j, the row statistics are shuffles of
// its 16 lanes, and O of the same rows and columns 4 x + 64 j stays in
// registers.  fp32 FMAs throughout: with 64 rows bound by their rate (a logit
// has to keep 24 bits, and three products of a tensor-core split cost more
// moves than these save at such sizes), with 16 by shared memory's.
#include "cache_attn.cuh"
#include "kernels.h"
#include "mma_sync.cuh"

namespace muse {

namespace {

constexpr int kBlock = 64;  // keys

template <int D, int R>
struct WideL {
  static constexpr int Q = 0, QS = D + 4;          // [R][QS]
  static constexpr int K = Q + R * QS, KS = D + 4;  // [64][KS]
  static constexpr int V = K + kBlock * KS;         // [64][D]
  static constexpr int P = V + kBlock * D, PS = kBlock + 4;  // [R][PS]
  static constexpr int TOTAL = (P + R * PS) * 4;
};

template <typename T, int CT, int D, int R>
__global__ void __launch_bounds__(256) cache_wide_kernel(const __grid_constant__ CacheAttn a) {
  using L = WideL<D, R>;
  constexpr int RT = R / 16, CG = D / 64;  // rows and column groups of a thread
  constexpr int LPR = D / 8, PASS = 256 / LPR, NP = kBlock / PASS;
  extern __shared__ __align__(16) float wide_sm[];
  const long long tile = blockIdx.x / a.S;
  const int split = (int)(blockIdx.x - tile * a.S);
  const long long bh = tile / a.RT;
  const int r0 = (int)(tile - bh * a.RT) * R;
  const int b = (int)(bh / a.c.Hkv), h = (int)(bh - (long long)b * a.c.Hkv);
  const SeqLen s = seq_len(a.c, b);
  if (r0 >= s.nn * a.G) return;
  const RowTile rt = row_tile(a, s, r0, R);
  const int len = rt.hi - rt.lo, parts = split_count(a, len);
  if (split >= parts) return;
  const int keys = split_keys(a, len);
  const int t0 = rt.lo + split * keys, t1 = min(rt.hi, t0 + keys);

  const int tid = threadIdx.x, x = tid & 15, y = tid >> 4;
  const int lr = tid / LPR, lc = tid % LPR;  // row (of a pass) and columns of this thread's loads
  float kreg[NP][8], vreg[NP][8];
  auto fetch = [&](int tb) {
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int t = tb + p * PASS + lr;
      const long long row = t < t1 ? row_of(a.c, b, h, t) : -1;
      load8<CT>(a.c.k, a.c.ks, row, D, lc, kreg[p]);
      load8<CT>(a.c.v, a.c.vs, row, D, lc, vreg[p]);
    }
  };
  fetch(t0);
  for (int e = tid; e < R * (D / 8); e += 256) {
    const int r = e / (D / 8), c = e % (D / 8);
    float q[8] = {};
    if (r0 + r < rt.r1) load8_in(static_cast<const T*>(a.Q) + row_at(a, b, h, r0 + r).q + 8 * c, q);
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] *= a.scale * kLog2e;
    store8(wide_sm + L::Q + r * L::QS + 8 * c, q);
  }
  int2 see[RT];
  float m[RT], l[RT], o[RT][4 * CG];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int r = r0 + y * RT + i;
    see[i] = r < rt.r1 ? seen(a, s, s.pos0 + r / a.G) : make_int2(0, 0);
    see[i].y = min(see[i].y, t1);
    m[i] = kFloor;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < 4 * CG; ++c) o[i][c] = 0.f;
  }
  bool bad = false;
  for (int tb = t0; tb < t1; tb += kBlock) {
    const bool edge = tb < rt.alo || tb + kBlock > rt.ahi;
    __syncthreads();  // the last block is read
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int r = p * PASS + lr;
      store8(wide_sm + L::K + r * L::KS + 8 * lc, kreg[p]);
      store8(wide_sm + L::V + r * D + 8 * lc, vreg[p]);
      if (edge) {  // values that are not numbers would reach the rows that do not see them
#pragma unroll
        for (int e = 0; e < 8; ++e) bad = bad || !(fabsf(vreg[p][e]) <= 3.4028234e38f);
      }
    }
    __syncthreads();
    if (tb + kBlock < t1) fetch(tb + kBlock);
    float acc[RT][4] = {};
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
      float4 kk[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        kk[j] = *reinterpret_cast<const float4*>(wide_sm + L::K + (x + 16 * j) * L::KS + d);
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const float4 q = *reinterpret_cast<const float4*>(wide_sm + L::Q + (y * RT + i) * L::QS + d);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[i][j] = fmaf(q.x, kk[j].x, acc[i][j]);
          acc[i][j] = fmaf(q.y, kk[j].y, acc[i][j]);
          acc[i][j] = fmaf(q.z, kk[j].z, acc[i][j]);
          acc[i][j] = fmaf(q.w, kk[j].w, acc[i][j]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int t = tb + x + 16 * j;
        if (t < see[i].x || t >= see[i].y) acc[i][j] = -INFINITY;
        top = fmaxf(top, acc[i][j]);
      }
#pragma unroll
      for (int w = 1; w < 16; w <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
      const float mn = fmaxf(m[i], top), f = fast_exp2(m[i] - mn);
      m[i] = mn;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float e = fast_exp2(acc[i][j] - mn);
        sum += e;
        wide_sm[L::P + (y * RT + i) * L::PS + x + 16 * j] = e;
      }
      l[i] = l[i] * f + sum;  // this thread's share
#pragma unroll
      for (int c = 0; c < 4 * CG; ++c) o[i][c] *= f;
    }
    __syncwarp();  // a row's weights are written and read by the same half warp
#pragma unroll 2
    for (int t = 0; t < kBlock; t += 4) {
      float4 p[RT];
#pragma unroll
      for (int i = 0; i < RT; ++i)
        p[i] = *reinterpret_cast<const float4*>(wide_sm + L::P + (y * RT + i) * L::PS + t);
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int g = 0; g < CG; ++g) {
          const float4 v = *reinterpret_cast<const float4*>(wide_sm + L::V + (t + u) * D + 64 * g + 4 * x);
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            const float w = u == 0 ? p[i].x : u == 1 ? p[i].y : u == 2 ? p[i].z : p[i].w;
            o[i][4 * g] = fmaf(w, v.x, o[i][4 * g]);
            o[i][4 * g + 1] = fmaf(w, v.y, o[i][4 * g + 1]);
            o[i][4 * g + 2] = fmaf(w, v.z, o[i][4 * g + 2]);
            o[i][4 * g + 3] = fmaf(w, v.w, o[i][4 * g + 3]);
          }
        }
    }
  }
  if (__syncthreads_or(bad)) {
    for (int r = r0 + (tid >> 5); r < rt.r1; r += 8)
      redo_row<T, CT, D>(a, s, b, h, r, t0, t1, tile, split, parts, r0);
    return;
  }
#pragma unroll
  for (int i = 0; i < RT; ++i) {
#pragma unroll
    for (int w = 1; w < 16; w <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);
    const int r = r0 + y * RT + i;
    if (r >= rt.r1) continue;
    if (parts > 1) {
#pragma unroll
      for (int g = 0; g < CG; ++g)
        *reinterpret_cast<float4*>(part_o<D>(a, tile, split, r - r0) + 64 * g + 4 * x) =
            make_float4(o[i][4 * g], o[i][4 * g + 1], o[i][4 * g + 2], o[i][4 * g + 3]);
      if (x == 0) *part_ml(a, tile, split, r - r0) = make_float2(m[i], l[i]);
      continue;
    }
    const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
    const RowAt at = row_at(a, b, h, r);
#pragma unroll
    for (int g = 0; g < CG; ++g)
#pragma unroll
      for (int c = 0; c < 4; ++c) st(static_cast<T*>(a.O) + at.o + 64 * g + 4 * x + c, o[i][4 * g + c] * inv);
    if (a.lse && x == 0) a.lse[at.lse] = lse_of(m[i], l[i]);
  }
}

template <typename T, int CT, int D, int R>
void launch(const CacheAttn& a, cudaStream_t st) {
  const int smem = WideL<D, R>::TOTAL;
  static LargeShared allowed;
  allowed.ensure((const void*)cache_wide_kernel<T, CT, D, R>, smem);
  const long long blocks = (long long)a.B * a.c.Hkv * a.RT * a.S;
  cache_wide_kernel<T, CT, D, R><<<(unsigned)blocks, 256, smem, st>>>(a);
}
template <typename T, int CT>
void launch_as(const CacheAttn& a, cudaStream_t st) {
  if (a.c.D == 64)
    a.rows == 16 ? launch<T, CT, 64, 16>(a, st) : launch<T, CT, 64, 64>(a, st);
  else
    a.rows == 16 ? launch<T, CT, 128, 16>(a, st) : launch<T, CT, 128, 64>(a, st);
}

}  // namespace

void run_cache_wide(const CacheAttn& a, cudaStream_t st) {
  ProfScope ps(st, "cache_wide");
  switch (a.type * 2 + a.f32) {
    case 2 * kCacheF32: return launch_as<__nv_bfloat16, kCacheF32>(a, st);
    case 2 * kCacheF32 + 1: return launch_as<float, kCacheF32>(a, st);
    case 2 * kCacheBf16 + 1: return launch_as<float, kCacheBf16>(a, st);
    case 2 * kCacheE4m3 + 1: return launch_as<float, kCacheE4m3>(a, st);
    default: return launch_as<float, kCacheI8>(a, st);
  }
}

}  // namespace muse
