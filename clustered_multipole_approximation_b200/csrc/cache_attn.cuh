// What the attention kernels over the paged cache share: rows packed by
// kv-head, the division of a row tile's keys into splits, the split partials
// and one row over a range of keys in fp32.
//
// The queries of a kv-head are packed token by token: packed row r is new
// token r / G, q-head h G + r % G, so the G heads that share keys share every
// tile of them, and the rows of a tile end at neighbouring positions.
#pragma once

#include <cuda_fp16.h>

#include <atomic>

#include "cache.cuh"

namespace muse {

constexpr float kLn2 = 0.6931471805599453f, kLog2e = 1.4426950408889634f;
// Running maxima (base 2) start at a finite floor below every finite logit,
// so that a block without a seen key needs no case of its own:
// exp2(-inf - floor) = 0.
constexpr float kFloor = -3.0e38f;
constexpr float kSlack = 8.f;  // the maximum moves when a logit exceeds it by this (base 2)
constexpr int kQuantum = 128;  // keys: splits are multiples of it (64 on the fp32 path)

// A row tile: packed rows [r0, r1) of (b, h) and the keys that any (all) of
// them see.
struct RowTile {
  int r0, r1;
  int lo, hi;    // some row sees only keys of [lo, hi)
  int alo, ahi;  // every row sees all keys of [alo, ahi)
};
__device__ inline RowTile row_tile(const CacheAttn& a, const SeqLen& s, int r0, int rows) {
  RowTile t;
  t.r0 = r0;
  t.r1 = min(s.nn * a.G, r0 + rows);
  const int2 f = seen(a, s, s.pos0 + div_by(a.by_G, r0)), l = seen(a, s, s.pos0 + div_by(a.by_G, max(t.r1 - 1, 0)));
  t.lo = f.x;
  t.hi = max(l.y, f.x);
  t.alo = l.x;
  t.ahi = f.y;
  return t;
}
__host__ __device__ inline int round_up(int x, int m) { return (x + m - 1) / m * m; }

// Keys of one split of a range of len keys: the call has up to a.S splits for
// every row tile, a tile uses as many as its own length asks for.
__host__ __device__ inline int split_keys(const CacheAttn& a, int len) {
  const int keys = round_up(div_by(a.by_S, len + a.S - 1), a.quantum);
  return keys > a.minc ? keys : a.minc;
}
__host__ __device__ inline int split_count(const CacheAttn& a, int len) {
  const int c = split_keys(a, len), n = (len + c - 1) / c;  // c >= minc >= 1
  return n > 1 ? n : 1;
}

// Split partials in the workspace: o (relative to 2^m, not divided by l), m, l
// of PR rows per (tile, split).
template <int D>
__device__ inline float* part_o(const CacheAttn& a, long long tile, int split, int r) {
  return static_cast<float*>(a.ws) + ((tile * a.S + split) * a.PR + r) * D;
}
__device__ inline float2* part_ml(const CacheAttn& a, long long tile, int split, int r) {
  return a.ml + (tile * a.S + split) * a.PR + r;
}

// The CTA's place in a grid of (sequence, kv-head, row tile, split), the last
// fastest (fewer than 2^31 CTAs).
struct Place {
  int tile, split, rt, b, h;
};
__device__ inline Place place_of(const CacheAttn& a) {
  Place p;
  p.tile = div_by(a.by_S, (int)blockIdx.x);
  p.split = (int)blockIdx.x - p.tile * a.S;
  const int bh = div_by(a.by_RT, p.tile);
  p.rt = p.tile - bh * a.RT;
  p.b = div_by(a.by_Hkv, bh);
  p.h = bh - p.b * a.c.Hkv;
  return p;
}

struct RowAt {
  int hq, i;
  long long q, o, lse;  // element offsets
};
__device__ inline RowAt row_at(const CacheAttn& a, int b, int h, int r) {
  RowAt x;
  x.i = div_by(a.by_G, r);
  x.hq = h * a.G + (r - x.i * a.G);
  x.q = b * a.qs.b + x.hq * a.qs.h + x.i * a.qs.t;
  x.o = b * a.os.b + x.hq * a.os.h + x.i * a.os.t;
  x.lse = ((long long)b * a.Hq + x.hq) * a.c.n + x.i;
  return x;
}

// One row over its seen keys within [t0, t1) by one warp, in fp32, key by key:
// D / 8 lanes hold a key, eight columns each.  Its result lies in the first
// D / 8 lanes (m in base 2).  Also the road of tiles whose masked values are
// not numbers: a product with a zero weight would spread them.
template <typename T, int CT, int D>
__device__ __noinline__ void row_over_keys(const CacheAttn& a, const SeqLen& s, int b, int h, int r,
                                           int t0, int t1, float (&o)[8], float& m, float& l) {
  constexpr int LPR = D / 8, GR = 32 / LPR;
  const int lane = threadIdx.x & 31, col = lane % LPR, grp = lane / LPR;
  const RowAt at = row_at(a, b, h, r);
  int2 ks = seen(a, s, s.pos0 + at.i);
  ks.x = max(ks.x, t0);
  ks.y = min(ks.y, t1);
  float q[8];
  m = -INFINITY;
  l = 0.f;
  load8_in(static_cast<const T*>(a.Q) + at.q + 8 * col, q);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    q[e] *= a.scale * kLog2e;
    o[e] = 0.f;
  }
  for (int u = ks.x; u < ks.y; u += GR) {
    const int t = u + grp;
    const long long row = t < ks.y ? row_of(a.c, b, h, t) : -1;
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
    const float f = m == -INFINITY ? 0.f : exp2f(m - mn);
    const float p = x == -INFINITY ? 0.f : exp2f(x - mn);
    l = l * f + p;
    m = mn;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = fmaf(o[e], f, p * v[e]);
  }
#pragma unroll
  for (int w = LPR; w < 32; w <<= 1) {  // join the groups
    const float m2 = __shfl_xor_sync(0xffffffffu, m, w), l2 = __shfl_xor_sync(0xffffffffu, l, w);
    const float mn = fmaxf(m, m2);
    const float f = m == -INFINITY ? 0.f : exp2f(m - mn), f2 = m2 == -INFINITY ? 0.f : exp2f(m2 - mn);
    l = l * f + l2 * f2;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = o[e] * f + __shfl_xor_sync(0xffffffffu, o[e], w) * f2;
    m = mn;
  }
}

// lse of a row from its maximum (base 2) and sum; nothing seen: -inf.
__device__ inline float lse_of(float m, float l) {
  return l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// Row r of the tile, recomputed by this warp and stored (as a split's partial
// where parts > 1).
template <typename T, int CT, int D>
__device__ __noinline__ void redo_row(const CacheAttn& a, const SeqLen& s, int b, int h, int r, int t0,
                                      int t1, long long tile, int split, int parts, int r0) {
  float o[8], m, l;
  row_over_keys<T, CT, D>(a, s, b, h, r, t0, t1, o, m, l);
  const int lane = threadIdx.x & 31;
  if (lane >= D / 8) return;
  if (parts > 1) {
    store8(part_o<D>(a, tile, split, r - r0) + 8 * lane, o);
    if (lane == 0) *part_ml(a, tile, split, r - r0) = make_float2(l == 0.f ? kFloor : m, l);
    return;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] *= inv;
  const RowAt at = row_at(a, b, h, r);
  store8(static_cast<T*>(a.O) + at.o + 8 * lane, o);
  if (a.lse && lane == 0) a.lse[at.lse] = lse_of(m, l);
}

// e4m3 pairs in the low (high) half of x as fp16, exact.
__device__ inline uint32_t half_of_e4m3_lo(uint32_t x) {
  uint32_t y;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}\n" : "=r"(y) : "r"(x));
  return y;
}
__device__ inline uint32_t half_of_e4m3_hi(uint32_t x) {
  uint32_t y;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}\n" : "=r"(y) : "r"(x));
  return y;
}
// An fp16 pair of bf16 values as bf16: the upper halves of the fp32 forms.
__device__ inline uint32_t bf16_of_half(uint32_t x) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x));
  return __byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x7632);
}
// int8 pair in bytes 0 and 2 of w as bf16, exact: q = (128 + (q & 127)) -
// (128 + (q & 128)), both terms bf16 values made by OR with the bits of 128.
__device__ inline uint32_t bf16_of_i8(uint32_t w) {
  const uint32_t p = (w & 0x007F007Fu) | 0x43004300u, n = (w & 0x00800080u) | 0x43004300u;
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&p),
                                   *reinterpret_cast<const __nv_bfloat162*>(&n));
  return *reinterpret_cast<const uint32_t*>(&d);
}
// Byte i of x and of y, i = 0 .. 3, as four bf16 pairs.
template <int CT>
__device__ inline void bf16_pairs(uint32_t x, uint32_t y, uint32_t (&o)[4]) {
  if (CT == kCacheE4m3) {
    const uint32_t a = __byte_perm(x, y, 0x5140), b = __byte_perm(x, y, 0x7362);
    o[0] = bf16_of_half(half_of_e4m3_lo(a));
    o[1] = bf16_of_half(half_of_e4m3_hi(a));
    o[2] = bf16_of_half(half_of_e4m3_lo(b));
    o[3] = bf16_of_half(half_of_e4m3_hi(b));
  } else {
    o[0] = bf16_of_i8(__byte_perm(x, y, 0x0400));
    o[1] = bf16_of_i8(__byte_perm(x, y, 0x0501));
    o[2] = bf16_of_i8(__byte_perm(x, y, 0x0602));
    o[3] = bf16_of_i8(__byte_perm(x, y, 0x0703));
  }
}
// Bytes (0, 1) and (2, 3) of x as bf16 pairs, and as fp16 pairs (int8 from the
// bits of 1024 + 128 + q).
template <int CT>
__device__ inline uint2 bf16_of_word(uint32_t x) {
  if (CT == kCacheE4m3) return make_uint2(bf16_of_half(half_of_e4m3_lo(x)), bf16_of_half(half_of_e4m3_hi(x)));
  return make_uint2(bf16_of_i8(__byte_perm(x, x, 0x0100)), bf16_of_i8(__byte_perm(x, x, 0x0302)));
}
template <int CT>
__device__ inline uint2 half_of_word(uint32_t x) {
  if (CT == kCacheE4m3) return make_uint2(half_of_e4m3_lo(x), half_of_e4m3_hi(x));
  const uint32_t u = x ^ 0x80808080u;
  const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
  const __half2 c = __floats2half2_rn(1152.f, 1152.f);
  const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&a), c);
  const __half2 e = __hsub2(*reinterpret_cast<const __half2*>(&b), c);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&d), *reinterpret_cast<const uint32_t*>(&e));
}
// Powers of two (f, 1 / f) with f top in [2^14, 2^15), f at most 2^103 (1 / f
// times a softmax scale stays a normal number); (1, 1) where top is not finite.
__device__ inline float2 half_factor(float top) {
  const int e = (int)(__float_as_uint(top) >> 23);  // biased exponent
  if (e == 255) return make_float2(1.f, 1.f);
  const int n = min(127 + 14 - (e - 127), 127 + 103);
  return make_float2(__uint_as_float((uint32_t)n << 23), __uint_as_float((uint32_t)(254 - n) << 23));
}

// Whether a word of stored values (two bf16, or four e4m3) holds one that is
// not finite.
__device__ inline bool bf16_not_finite(uint32_t w) {
  return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}
__device__ inline bool e4m3_not_finite(uint32_t w) {
  return (((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0;
}

// A kernel's leave for more than 48 KB of shared memory, asked for once a device.
struct LargeShared {
  std::atomic<uint64_t> done{0};
  void ensure(const void* kernel, int bytes) {
    int dev = 0;
    cudaGetDevice(&dev);
    const uint64_t bit = 1ull << (dev & 63);
    if (done.load(std::memory_order_acquire) & bit) return;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess && dev < 64)
      done.fetch_or(bit, std::memory_order_release);
  }
};

void run_cache_step(const CacheAttn& a, cudaStream_t st);  // up to 32 packed rows, bf16 queries
void run_cache_chunk(const CacheAttn& a, cudaStream_t st);  // more
void run_cache_wide(const CacheAttn& a, cudaStream_t st);  // fp32 queries or cache

}  // namespace muse
