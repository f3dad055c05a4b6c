// Attention of a chunk of new tokens over the paged cache: the choice of a
// kernel, the division of the keys and the join of the splits.
//
// Query i of sequence b, at position P = kv_len - new_len + i, sees the keys
// [lo, hi) of `seen` and takes
//   o = sum_t softmax_t(scale q.k_t) v_t,   lse = ln sum_t exp(scale q.k_t);
// a row that sees nothing has o = 0 and lse = -inf.  One online softmax: the
// running maximum m and sum l, and o rescaled when m moves.
#include "cache_attn.cuh"
#include "kernels.h"

namespace muse {

namespace {

// Joins the splits of one row: W warps take every W-th split each, then the
// CTA's first warp their sums, always in this order.
template <typename T, int D, int W>
__global__ void __launch_bounds__(32 * W) cache_join_kernel(const __grid_constant__ CacheAttn a) {
  constexpr int C = D / 32;  // columns of a lane
  __shared__ float so[W][D];
  __shared__ float2 sml[W];
  const int n = a.c.n, rows = n * a.G;
  const long long bh = blockIdx.x / rows;
  const int r = (int)(blockIdx.x - bh * rows);
  const int b = (int)(bh / a.c.Hkv), h = (int)(bh - (long long)b * a.c.Hkv);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const SeqLen s = seq_len(a.c, b);
  cudaGridDependencySynchronize();
  if (r >= s.nn * a.G) return;
  const int rt = r / a.rows;
  const RowTile t = row_tile(a, s, rt * a.rows, a.rows);
  const int parts = split_count(a, t.hi - t.lo);
  if (parts == 1) return;  // the tile wrote its rows itself
  const long long tile = bh * a.RT + rt;
  const int pr = r - t.r0;
  float m = kFloor, l = 0.f, o[C] = {};
#pragma unroll 4
  for (int p = warp; p < parts; p += W) {
    const float2 ml = *part_ml(a, tile, p, pr);
    const float* po = part_o<D>(a, tile, p, pr) + C * lane;
    float y[C];
#pragma unroll
    for (int c = 0; c < C; ++c) y[c] = po[c];
    // NaN maxima do not arise: they are maxima of the numbers among the logits
    const float mn = fmaxf(m, ml.x), f = exp2f(m - mn), g = exp2f(ml.x - mn);
    l = l * f + ml.y * g;
#pragma unroll
    for (int c = 0; c < C; ++c) o[c] = o[c] * f + y[c] * g;
    m = mn;
  }
  if (W > 1) {
#pragma unroll
    for (int c = 0; c < C; ++c) so[warp][C * lane + c] = o[c];
    if (lane == 0) sml[warp] = make_float2(m, l);
    __syncthreads();
    if (warp) return;
    m = kFloor;
    l = 0.f;
    for (int w = 0; w < W; ++w) m = fmaxf(m, sml[w].x);
#pragma unroll
    for (int c = 0; c < C; ++c) o[c] = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float f = exp2f(sml[w].x - m);
      l += sml[w].y * f;
#pragma unroll
      for (int c = 0; c < C; ++c) o[c] = fmaf(so[w][C * lane + c], f, o[c]);
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const RowAt at = row_at(a, b, h, r);
  T* op = static_cast<T*>(a.O) + at.o + C * lane;
#pragma unroll
  for (int c = 0; c < C; ++c) st(op + c, o[c] * inv);
  if (a.lse && lane == 0) a.lse[at.lse] = lse_of(m, l);
}

template <typename T, int D, int W>
void join_as(const CacheAttn& a, cudaStream_t st) {
  // launched while its predecessor drains: it waits for it on the device
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((long long)a.B * a.Hq * a.c.n));
  cfg.blockDim = dim3(32 * W);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, cache_join_kernel<T, D, W>, a);
}
template <typename T>
void run_join(const CacheAttn& a, cudaStream_t st) {
  ProfScope ps(st, "cache_join");
  if (a.c.D == 64)
    a.S <= 8 ? join_as<T, 64, 1>(a, st) : join_as<T, 64, 8>(a, st);
  else
    a.S <= 8 ? join_as<T, 128, 1>(a, st) : join_as<T, 128, 8>(a, st);
}

enum Path { kWide, kStep, kChunk };
Path path_of(const CacheAttn& a) {
  if (a.f32 || a.type == kCacheF32) return kWide;
  return (long long)a.c.n * a.G <= 32 ? kStep : kChunk;
}

constexpr int kSMs = 148;

// How the call's keys are divided, from its sizes alone (the lengths are on
// the device; each row tile then uses the splits that its own length asks
// for).
Path plan(CacheAttn& a) {
  const Path p = path_of(a);
  const long long cap = (long long)a.c.wide * a.c.page.d;
  const long long packed = (long long)a.c.n * a.G;
  auto quanta = [](long long x) { return (x + kQuantum - 1) / kQuantum * kQuantum; };
  a.rows = p == kChunk ? 256 : p == kStep && packed <= 8 ? 8 : packed <= 16 ? 16 : p == kStep ? 32 : 64;
  a.RT = (int)((packed + a.rows - 1) / a.rows);
  a.PR = (int)(packed < a.rows ? packed : a.rows);
  const long long units = (long long)a.B * a.c.Hkv * a.RT;
  a.S = a.minc = 1;
  a.cluster = 0;
  if (p != kChunk) {
    // keys of a split: enough splits for eight CTAs an SM, none of more than
    // 512 KB of cache, and no more than 128 a row
    const int size = a.type == kCacheF32 ? 4 : a.type == kCacheBf16 ? 2 : 1;
    long long c = quanta(cap * units / (kSMs * 8) + 1);
    const long long most = quanta((512 << 10) / (2 * a.c.D * size));
    if (c > most) c = most;
    if (c * 128 < cap) c = quanta((cap + 127) / 128);
    a.S = (int)((cap + c - 1) / c);
    while (a.S > 1 && units * a.S > 0x7FFFFFFF) a.S = (a.S + 1) / 2;  // the grid
    // a table far wider than its sequences: shorter splits while few rows fill the SMs
    const long long least = quanta(c * units / (2 * kSMs));
    a.minc = (int)(least < c ? least : c);
    if (p == kStep && a.S > 1 && a.S <= 16) {  // up to eight join without a second launch
      a.S = a.S < 8 ? a.S : 8;
      a.cluster = 1;
    }
  } else {
    // the number of splits whose last wave of CTAs wastes least, each split
    // charged with 3 % for its partials and start
    double best = 1e30;
    for (int S = 1; S <= 64 && (S == 1 || (long long)S * 512 <= cap); ++S) {
      const double w = (double)((units * S + kSMs - 1) / kSMs) / S * (1 + 0.03 * (S - 1));
      if (w < best - 1e-9) {
        best = w;
        a.S = S;
      }
      if (units * S > 8 * kSMs) break;
    }
    a.minc = 512;
  }
  return p;
}

// Bytes of the split partials: o, then (m, l).
size_t part_bytes(const CacheAttn& a, bool ml) {
  const size_t rows = (size_t)a.B * a.c.Hkv * a.RT * a.S * a.PR;
  return (rows * (ml ? 8 : (size_t)a.c.D * 4) + 255) / 256 * 256;
}

}  // namespace

size_t cache_attn_workspace(const CacheAttn& a0) {
  CacheAttn a = a0;
  plan(a);
  return a.S > 1 && !a.cluster ? part_bytes(a, false) + part_bytes(a, true) : 256;
}

void run_cache_attn(const CacheAttn& a0, cudaStream_t st) {
  CacheAttn a = a0;
  const Path p = plan(a);
  const bool join = a.S > 1 && !a.cluster;
  if (join) a.ml = reinterpret_cast<float2*>(static_cast<unsigned char*>(a.ws) + part_bytes(a, false));
  p == kWide ? run_cache_wide(a, st) : p == kStep ? run_cache_step(a, st) : run_cache_chunk(a, st);
  if (join) a.f32 ? run_join<float>(a, st) : run_join<__nv_bfloat16>(a, st);
}

}  // namespace muse
