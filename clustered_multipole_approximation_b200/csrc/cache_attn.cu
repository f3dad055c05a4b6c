// Attention of a chunk of new tokens over the paged cache.
//
// Query i of sequence b, at position P = kv_len - new_len + i, sees the keys
// [lo, hi) of `seen` and takes
//   o = sum_t softmax_t(scale q.k_t) v_t,   lse = ln sum_t exp(scale q.k_t);
// a row that sees nothing has o = 0 and lse = -inf.  One online softmax: the
// running maximum m and sum l, and o rescaled when m moves.
#include "cache.cuh"
#include "kernels.h"
#include "mma_sync.cuh"

namespace muse {

namespace {

// One warp per query row; lane c of the first D / 8 lanes of each of two (four
// at D = 64) groups holds columns [8 c, 8 c + 8), a group takes every second
// (fourth) key.  fp32 throughout.
template <typename T, int CT, int D>
__global__ void __launch_bounds__(128) cache_attn_simt_kernel(CacheAttn a, long long rows) {
  constexpr int LPR = D / 8, GR = 32 / LPR;
  const long long r = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (r >= rows) return;
  const int lane = threadIdx.x & 31, col = lane % LPR, grp = lane / LPR;
  const long long bh = r / a.c.n;
  const int i = (int)(r - bh * a.c.n);
  const int b = (int)(bh / a.Hq), hq = (int)(bh - (long long)b * a.Hq);
  const SeqLen s = seq_len(a.c, b);
  if (i >= s.nn) return;
  const int2 ks = seen(a, s, s.pos0 + i);
  float q[8], o[8] = {}, m = -INFINITY, l = 0.f;
  load8_in(static_cast<const T*>(a.Q) + b * a.qs.b + hq * a.qs.h + i * a.qs.t + 8 * col, q);
#pragma unroll
  for (int e = 0; e < 8; ++e) q[e] *= a.scale;
  for (int t0 = ks.x; t0 < ks.y; t0 += GR) {
    const int t = t0 + grp;
    const long long row = t < ks.y ? row_of(a.c, b, hq / a.G, t) : -1;
    float k[8], v[8], x = 0.f;
    load8<CT>(a.c.k, a.c.ks, row, D, col, k);
    load8<CT>(a.c.v, a.c.vs, row, D, col, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) x = fmaf(q[e], k[e], x);
#pragma unroll
    for (int w = LPR / 2; w > 0; w >>= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
    if (t >= ks.y) continue;
    const float mn = fmaxf(m, x);
    // a logit of -inf before any other: nothing is added
    const float f = m == -INFINITY ? 0.f : expf(m - mn);
    const float p = x == -INFINITY ? 0.f : expf(x - mn);
    l = l * f + p;
    m = mn;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = fmaf(o[e], f, p * v[e]);
  }
#pragma unroll
  for (int w = LPR; w < 32; w <<= 1) {  // join the groups
    const float m2 = __shfl_xor_sync(0xffffffffu, m, w), l2 = __shfl_xor_sync(0xffffffffu, l, w);
    const float mn = fmaxf(m, m2);
    const float f = m == -INFINITY ? 0.f : expf(m - mn), f2 = m2 == -INFINITY ? 0.f : expf(m2 - mn);
    l = l * f + l2 * f2;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = o[e] * f + __shfl_xor_sync(0xffffffffu, o[e], w) * f2;
    m = mn;
  }
  if (grp) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] *= inv;
  store8(static_cast<T*>(a.O) + b * a.os.b + hq * a.os.h + i * a.os.t + 8 * col, o);
  if (a.lse && col == 0) a.lse[r] = l == 0.f ? -INFINITY : m + logf(l);
}

template <typename T, int CT>
void simt_as(const CacheAttn& a, cudaStream_t st) {
  const long long rows = (long long)a.B * a.Hq * a.c.n;
  const unsigned blocks = (unsigned)((rows + 3) / 4);
  if (a.c.D == 64)
    cache_attn_simt_kernel<T, CT, 64><<<blocks, 128, 0, st>>>(a, rows);
  else
    cache_attn_simt_kernel<T, CT, 128><<<blocks, 128, 0, st>>>(a, rows);
}

}  // namespace

size_t cache_attn_workspace(const CacheAttn&) { return 256; }

void run_cache_attn(const CacheAttn& a, cudaStream_t st) {
  ProfScope ps(st, "cache_attn");
  switch (a.type * 2 + a.f32) {
    case 0: return simt_as<__nv_bfloat16, kCacheBf16>(a, st);
    case 1: return simt_as<float, kCacheBf16>(a, st);
    case 2: return simt_as<__nv_bfloat16, kCacheF32>(a, st);
    case 3: return simt_as<float, kCacheF32>(a, st);
    case 4: return simt_as<__nv_bfloat16, kCacheE4m3>(a, st);
    case 5: return simt_as<float, kCacheE4m3>(a, st);
    case 6: return simt_as<__nv_bfloat16, kCacheI8>(a, st);
    default: return simt_as<float, kCacheI8>(a, st);
  }
}

}  // namespace muse
