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
#include "mma_sync.cuh"

namespace muse {

namespace {

// Joins the splits of a row: W warps take every W-th split each, then the first
// of them their sums, always in this order.  A CTA has eight warps.
template <typename T, int D, int W>
__global__ void __launch_bounds__(256) cache_join_kernel(const __grid_constant__ CacheAttn a, int total) {
  constexpr int C = D / 32;  // columns of a lane
  __shared__ float so[8][D];
  __shared__ float2 sml[8];
  const int rows = a.c.n * a.G;  // of a kv-head
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = warp % W;
  const long long gr = (long long)blockIdx.x * (8 / W) + warp / W;
  const int bh = (int)(gr / rows), r = (int)(gr - (long long)bh * rows);
  const int b = bh / a.c.Hkv, h = bh - b * a.c.Hkv;
  const bool there = gr < total;
  SeqLen s{};
  if (there) s = seq_len(a.c, b);
  cudaGridDependencySynchronize();
  bool live = there && r < s.nn * a.G;
  const int rt = a.RT == 1 ? 0 : r / a.rows;
  RowTile t{};
  int parts = 1;
  if (live) {
    t = row_tile(a, s, rt * a.rows, a.rows);
    parts = split_count(a, t.hi - t.lo);
    live = parts > 1;  // else the tile wrote its rows itself
  }
  const long long tile = (long long)bh * a.RT + rt;
  const int pr = r - t.r0;
  float m = kFloor, l = 0.f, o[C] = {};
  if (live) {
#pragma unroll 4
    for (int p = part; p < parts; p += W) {
      const float2 ml = *part_ml(a, tile, p, pr);
      const float* po = part_o<D>(a, tile, p, pr) + C * lane;
      float y[C];
#pragma unroll
      for (int c = 0; c < C; ++c) y[c] = po[c];
      // NaN maxima do not arise: they are maxima of the numbers among the logits
      const float mn = fmaxf(m, ml.x), f = fast_exp2(m - mn), g = fast_exp2(ml.x - mn);
      l = l * f + ml.y * g;
#pragma unroll
      for (int c = 0; c < C; ++c) o[c] = o[c] * f + y[c] * g;
      m = mn;
    }
  }
  if (W > 1) {
#pragma unroll
    for (int c = 0; c < C; ++c) so[warp][C * lane + c] = o[c];
    if (lane == 0) sml[warp] = make_float2(m, l);
    __syncthreads();
    if (part) return;
    m = kFloor;
    l = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) m = fmaxf(m, sml[warp + w].x);
#pragma unroll
    for (int c = 0; c < C; ++c) o[c] = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float f = fast_exp2(sml[warp + w].x - m);
      l += sml[warp + w].y * f;
#pragma unroll
      for (int c = 0; c < C; ++c) o[c] = fmaf(so[warp + w][C * lane + c], f, o[c]);
    }
  }
  if (!live) return;
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
  const int rows = a.B * a.Hq * a.c.n;  // < 2^31, checked
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(((long long)rows * W + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, cache_join_kernel<T, D, W>, a, rows);
}
template <typename T, int D>
void join_of(const CacheAttn& a, cudaStream_t st) {
  a.S <= 8 ? join_as<T, D, 1>(a, st) : a.S <= 32 ? join_as<T, D, 4>(a, st) : join_as<T, D, 8>(a, st);
}
template <typename T>
void run_join(const CacheAttn& a, cudaStream_t st) {
  ProfScope ps(st, "cache_join");
  a.c.D == 64 ? join_of<T, 64>(a, st) : join_of<T, 128>(a, st);
}

// Failure-path testing (muse_debug_inject_cache_fault).
int g_lost_load = -1;

enum Path { kWide, kStep, kChunk };
Path path_of(const CacheAttn& a) {
  if (a.f32 || a.type == kCacheF32) return kWide;
  return (long long)a.c.n * a.G <= 32 ? kStep : kChunk;
}

constexpr int kSMs = 148;

// How up to `cap` keys of a row tile are divided, from the call's sizes alone
// (the lengths are on the device; each row tile then uses the splits that its
// own length asks for).
Path plan_keys(CacheAttn& a, long long cap) {
  const Path p = path_of(a);
  const long long packed = (long long)a.c.n * a.G;
  auto quanta = [](long long x) { return (x + kQuantum - 1) / kQuantum * kQuantum; };
  a.rows = p == kChunk ? 256 : p == kStep && packed <= 8 ? 8 : packed <= 16 ? 16 : p == kStep ? 32 : 64;
  a.RT = (int)((packed + a.rows - 1) / a.rows);
  a.PR = (int)(packed < a.rows ? packed : a.rows);
  const long long units = (long long)a.B * a.c.Hkv * a.RT;
  a.S = a.minc = 1;
  a.cluster = 0;
  a.quantum = p == kWide ? 64 : kQuantum;
  if (p == kWide) {
    // in blocks of 64 keys: two CTAs an SM at a time (at D = 128 the kernel has one,
    // and the same division), half a wave lost at the end, 0.3 of a block for a split's
    // start and partials
    double best = 1e30;
    for (int S = 1; S <= 64 && (S == 1 || (long long)S * 64 < cap + 64); ++S) {
      if (S > 1 && units * S > 0x7FFFFFFF) break;
      const double waves = (double)(units * S) / (2 * kSMs);
      const double w = ((waves < 0.5 ? 0.5 : waves) + 0.5) * ((double)((cap + S * 64LL - 1) / (S * 64LL)) + 0.3);
      if (w < best - 1e-9) {
        best = w;
        a.S = S;
      }
    }
    a.minc = 64;
  } else if (p == kStep) {
    // Keys of a split.  Enough for eight CTAs an SM; but, as long as two an SM are
    // left, 256 KB of cache, which pays for a CTA's start (37 x 8 kv-heads of 128 at
    // 1265 in e4m3: one split 25 us, two 39); and 512 KB at most, for the tail.
    const int size = a.type == kCacheBf16 ? 2 : 1;
    const long long bytes = 2 * a.c.D * size, most = quanta((512 << 10) / bytes);
    long long c = quanta(cap * units / (kSMs * 8) + 1);
    const long long some = quanta((256 << 10) / bytes), two = quanta(cap * units / (kSMs * 2) + 1);
    if (c < some && c < two) c = some < two ? some : two;
    if (c > most) c = most;
    if (units >= 2 * kSMs && cap <= most) c = quanta(cap);  // one split, no join
    if (c * 128 < cap) c = quanta((cap + 127) / 128);
    // (and no more than 64 CTAs an SM in all: workspace for nothing)
    if (c * (kSMs * 64) < cap * units) c = quanta(cap * units / (kSMs * 64));
    a.S = (int)((cap + c - 1) / c);
    while (a.S > 1 && units * a.S > 0x7FFFFFFF) a.S = (a.S + 1) / 2;  // the grid
    // a table far wider than its sequences: shorter splits while few rows fill the SMs
    const long long least = quanta(c * units / (2 * kSMs));
    // (but a quantum at least: a row tile that sees nothing divides by it too)
    a.minc = (int)(least < c ? least : c);
    if (a.minc < kQuantum) a.minc = kQuantum;
    // Up to eight splits join as a cluster, without a second launch -- where the
    // grid fits the SMs at once: one token of 8 heads at 1000 8 us against 11, but
    // clusters that wait for one another's places took 485 us where 64 sequences of
    // 16384 take 389.
    const int S8 = a.S < 8 ? a.S : 8;
    if (a.S > 1 && units * S8 <= 2 * kSMs && (a.S <= 8 || cap <= 8 * 512)) {
      a.S = S8;
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

// The division for the call's keys: what its table can hold, or what a tile's
// rows can see through the window.  The workspace is sized without the window,
// so that a windowed call takes no more of it.
Path plan(CacheAttn& a) {
  const long long cap = (long long)a.c.wide * a.c.page.d;
  const Path p = plan_keys(a, cap);
  const long long reach = (long long)a.window + a.rows / a.G + 1;
  if (!a.window || reach >= cap) return p;
  const int S = a.S, cluster = a.cluster;
  plan_keys(a, reach);
  if (S == 1 || (cluster && !a.cluster)) {
    a.S = 1;
    a.cluster = 0;
  } else if (!a.cluster && a.S > S) {
    a.S = S;
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

void cache_attn_division(CacheAttn& a, int len, int* parts, int* keys) {
  plan(a);
  a.by_S = fast_div((uint32_t)a.S);
  *keys = split_keys(a, len);
  *parts = *keys > 0 ? split_count(a, len) : 0;
}

void set_cache_fault(int load) { g_lost_load = load; }

void run_cache_attn(const CacheAttn& a0, cudaStream_t st) {
  CacheAttn a = a0;
  const Path p = plan(a);
  a.by_G = fast_div((uint32_t)a.G);
  a.by_Hkv = fast_div((uint32_t)a.c.Hkv);
  a.by_RT = fast_div((uint32_t)a.RT);
  a.by_S = fast_div((uint32_t)a.S);
  a.lost = g_lost_load;
  const bool join = a.S > 1 && !a.cluster;
  if (join) a.ml = reinterpret_cast<float2*>(static_cast<unsigned char*>(a.ws) + part_bytes(a, false));
  p == kWide ? run_cache_wide(a, st) : p == kStep ? run_cache_step(a, st) : run_cache_chunk(a, st);
  if (join) a.f32 ? run_join<float>(a, st) : run_join<__nv_bfloat16>(a, st);
}

}  // namespace muse
