// Attention over the paged cache in fp32: fp32 queries, or an fp32 cache.
//
// One CTA of eight warps takes a tile of R packed rows (64, or 16 where the
// call has no more) and one split of its keys, 64 at a time: K and V of a
// block stand in shared memory as fp32 (8-bit rows times their scale), the
// next block's are on their way in registers.  Both products run on the tensor
// cores (mma.sync m16n8k8, tf32) with either operand x split in two, hi the
// tf32 value nearest to x and lo that nearest to x - hi: hi hi + hi lo + lo hi
// leaves out lo lo and what lo rounds off, 3 2^-22 of a product at most, less
// than the additions in fp32 lose over D = 64 terms.  The softmax between them
// is a thread's R / 16 rows and every 16th key, row statistics by shuffles,
// weights through shared memory.
// Two sequences of 130 tokens at 2100, 8 heads over 2 of 64: 40 us, of which the
// kernel takes 34 (tensor cores 28 % busy; the splitting's integer operations
// and the four barriers of a block bound it).  The same tile as fp32 FMAs was
// bound by shared memory's reads: 4 us more, and 58 us against 46 for single
// tokens over int8.
//
// An infinity has no such split (nor has the last step below one): a CTA that
// meets a value that is not finite forms its rows again key by key (redo_row).
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
  static constexpr int V = K + kBlock * KS, VS = D + 8;  // [64][VS]
  static constexpr int P = V + kBlock * VS, PS = kBlock + 4;  // [R][PS]: logits, then weights
  static constexpr int F = P + R * PS;                        // [R]: O's factor, then 1 / l
  static constexpr int TOTAL = (F + R) * 4;
};

// x = hi + lo to 2^-22: hi the nearest tf32 value, lo the rest (the tensor cores
// read the upper 19 bits of an operand; half a step is added for them).
struct Split {
  uint32_t hi, lo;
};
__device__ inline Split split_tf32(float x) {
  Split s;
  s.hi = (__float_as_uint(x) + 0x1000u) & 0xFFFFE000u;
  s.lo = __float_as_uint(x - __uint_as_float(s.hi)) + 0x1000u;
  return s;
}
__device__ inline void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// c[n] += A B: A the 16 rows at `pa` (stride as), B the NT n8 tiles whose element
// (k, n) is pb[k bk + n bn], k < K.  The strides keep a warp's reads on 32 banks.
// The small terms have accumulators of their own: shorter chains.
template <int NT, int K>
__device__ inline void product(float (&c)[NT][4], const float* pa, int as, const float* pb, int bk, int bn) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  pa += g * as + t;
  pb += t * bk + g * bn;
  float d[NT][4] = {};
#pragma unroll 2
  for (int k = 0; k < K; k += 8) {
    uint32_t ah[4], al[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const Split s = split_tf32(pa[k + 8 * as * (i & 1) + 4 * (i >> 1)]);
      ah[i] = s.hi;
      al[i] = s.lo;
    }
    Split b0[NT], b1[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      b0[n] = split_tf32(pb[k * bk + 8 * n * bn]);
      b1[n] = split_tf32(pb[(k + 4) * bk + 8 * n * bn]);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) mma_tf32(d[n], al, b0[n].hi, b1[n].hi);
#pragma unroll
    for (int n = 0; n < NT; ++n) mma_tf32(c[n], ah, b0[n].hi, b1[n].hi);
#pragma unroll
    for (int n = 0; n < NT; ++n) mma_tf32(d[n], ah, b0[n].lo, b1[n].lo);
  }
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) c[n][e] += d[n][e];
}

template <typename T, int CT, int D, int R>
__global__ void __launch_bounds__(256, D == 64 ? 2 : 1) cache_wide_kernel(const __grid_constant__ CacheAttn a) {
  using L = WideL<D, R>;
  constexpr int RT = R / 16;  // softmax rows of a thread
  // warps: R / 16 row tiles by 128 / R column groups of both products
  constexpr int WN = 128 / R, NS = kBlock / 8 / WN, NO = D / 8 / WN;
  constexpr int LPR = D / 8, PASS = 256 / LPR, NP = kBlock / PASS;
  extern __shared__ __align__(16) float wide_sm[];
  const Place at0 = place_of(a);
  const int tile = at0.tile, split = at0.split, b = at0.b, h = at0.h, r0 = at0.rt * R;
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
  uint32_t top = 0;  // largest magnitude met, as an integer
  for (int e = tid; e < R * (D / 8); e += 256) {
    const int r = e / (D / 8), c = e % (D / 8);
    float q[8] = {};
    if (r0 + r < rt.r1) load8_in(static_cast<const T*>(a.Q) + row_at(a, b, h, r0 + r).q + 8 * c, q);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      q[i] *= a.scale * kLog2e;
      top = max(top, __float_as_uint(q[i]) & 0x7FFFFFFFu);
    }
    store8(wide_sm + L::Q + r * L::QS + 8 * c, q);
  }
  const int lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
  const int wr = 16 * (warp / WN), wn = warp % WN;  // this warp's rows and column group
  int2 see[RT];
  float m[RT], l[RT], o[NO][4];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int r = r0 + y * RT + i;
    see[i] = r < rt.r1 ? seen(a, s, s.pos0 + div_by(a.by_G, r)) : make_int2(0, 0);
    see[i].y = min(see[i].y, t1);
    m[i] = kFloor;
    l[i] = 0.f;
  }
#pragma unroll
  for (int n = 0; n < NO; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
  for (int tb = t0; tb < t1; tb += kBlock) {
    __syncthreads();  // the last block is read
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int r = p * PASS + lr;
      store8(wide_sm + L::K + r * L::KS + 8 * lc, kreg[p]);
      store8(wide_sm + L::V + r * L::VS + 8 * lc, vreg[p]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        top = max(top, __float_as_uint(kreg[p][e]) & 0x7FFFFFFFu);
        top = max(top, __float_as_uint(vreg[p][e]) & 0x7FFFFFFFu);
      }
    }
    __syncthreads();
    if (tb + kBlock < t1) fetch(tb + kBlock);
    {
      float x4[NS][4] = {};
      product<NS, D>(x4, wide_sm + L::Q + wr * L::QS, L::QS, wide_sm + L::K + 8 * NS * wn * L::KS, 1, L::KS);
#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          *reinterpret_cast<float2*>(wide_sm + L::P + (wr + g + 8 * e) * L::PS + 8 * (NS * wn + n) + 2 * t4) =
              make_float2(x4[n][2 * e], x4[n][2 * e + 1]);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      float* row = wide_sm + L::P + (y * RT + i) * L::PS + x;
      float acc[4], mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int t = tb + x + 16 * j;
        acc[j] = t < see[i].x || t >= see[i].y ? -INFINITY : row[16 * j];
        mx = fmaxf(mx, acc[j]);
      }
#pragma unroll
      for (int w = 1; w < 16; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
      const float mn = fmaxf(m[i], mx), f = fast_exp2(m[i] - mn);
      m[i] = mn;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float e = fast_exp2(acc[j] - mn);
        sum += e;
        row[16 * j] = e;
      }
      l[i] = l[i] * f + sum;  // this thread's share
      if (x == 0) wide_sm[L::F + y * RT + i] = f;
    }
    __syncthreads();
    const float f0 = wide_sm[L::F + wr + g], f1 = wide_sm[L::F + wr + g + 8];
#pragma unroll
    for (int n = 0; n < NO; ++n) o[n][0] *= f0, o[n][1] *= f0, o[n][2] *= f1, o[n][3] *= f1;
    product<NO, kBlock>(o, wide_sm + L::P + wr * L::PS, L::PS, wide_sm + L::V + 8 * NO * wn, L::VS, 1);
  }
  if (__syncthreads_or(top >= 0x7F7FF000u)) {
    for (int r = r0 + warp; r < rt.r1; r += 8)
      redo_row<T, CT, D>(a, s, b, h, r, t0, t1, tile, split, parts, r0);
    return;
  }
#pragma unroll
  for (int i = 0; i < RT; ++i) {
#pragma unroll
    for (int w = 1; w < 16; w <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);
    const int r = r0 + y * RT + i;
    if (x != 0 || r >= rt.r1) continue;
    if (parts > 1)
      *part_ml(a, tile, split, r - r0) = make_float2(m[i], l[i]);
    else if (a.lse)
      a.lse[row_at(a, b, h, r).lse] = lse_of(m[i], l[i]);
    wide_sm[L::F + y * RT + i] = parts > 1 ? 1.f : l[i] == 0.f ? 0.f : 1.f / l[i];
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int r = r0 + wr + g + 8 * e;
    if (r >= rt.r1) continue;
    const float inv = wide_sm[L::F + r - r0];
    T* op = static_cast<T*>(a.O) + row_at(a, b, h, r).o;
#pragma unroll
    for (int n = 0; n < NO; ++n) {
      const int c = 8 * (NO * wn + n) + 2 * t4;
      const float u = o[n][2 * e] * inv, v = o[n][2 * e + 1] * inv;
      if (parts > 1) {
        *reinterpret_cast<float2*>(part_o<D>(a, tile, split, r - r0) + c) = make_float2(u, v);
      } else if (sizeof(T) == 4) {
        *reinterpret_cast<float2*>(op + c) = make_float2(u, v);
      } else {
        *reinterpret_cast<uint32_t*>(op + c) = bf16_bits2(u, v);
      }
    }
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
