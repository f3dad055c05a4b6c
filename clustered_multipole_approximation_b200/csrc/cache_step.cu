// Attention of single tokens (and of a few: up to 16 packed rows a kv-head)
// over the paged cache, bf16 queries.
//
// One CTA of four warps takes a split of one (sequence, kv-head)'s keys.  The
// bound is the cache's bytes: each warp streams blocks of keys of its own
// through a ring of shared memory (cp.async, several blocks in flight, no
// block-wide barrier in the loop) and keeps its own online softmax, so that
// warps drift apart and loads never stop; they join once, at the end, in a
// fixed order.  Products run on mma.sync m16n8k16: with at most 16 rows a
// tile of the fifth-generation tensor cores would be seven-eighths padding,
// and its results would take the way over TMEM.
//   S = Q K^T     K rows as the B operand.  The contraction's order is free,
//                 so an 8-bit row is read 16 bytes a lane and Q's columns are
//                 permuted to match; converted in registers.
//   o += P V      V as the B operand: ldmatrix.trans (bf16), or pairs of bytes
//                 from neighbouring keys' rows (8-bit) with the output columns
//                 permuted to match.
// Scales of 8-bit rows multiply S's columns and P's columns (before its one
// rounding to bf16).
#include "cache_attn.cuh"
#include "kernels.h"
#include "mma_sync.cuh"

namespace muse {

namespace {

constexpr int kWarps = 4;

template <int CT, int D>
struct StepL {
  static constexpr int SZ = CT == kCacheBf16 ? 2 : 1;
  static constexpr int KB = SZ * D > 128 ? 16 : 32;  // keys of a block
  static constexpr int RB = SZ * D;                  // bytes of a row
  static constexpr int LPR = RB / 16;                // lanes of a row's load
  static constexpr int HALF = KB * RB;               // K (or V) of a block
  static constexpr int SCALES = SZ == 1 ? 2 * KB * 4 : 0;
  static constexpr int STAGE = 2 * HALF + SCALES;
  static constexpr int NS = 3;
  static constexpr int RING = NS * STAGE;
  static constexpr int JOIN = 16 * D * 4 + 16 * 8;  // o, (m, l) of a warp
  static constexpr int WARP = RING > JOIN ? RING : JOIN;
  static constexpr int TOTAL = kWarps * WARP;
};

// Byte offset of 16-byte piece c of key row r.  Each pattern keeps the lanes
// of one shared-memory phase on other banks: bf16 rows for ldmatrix; 8-bit K
// (two keys, four pieces a phase); 8-bit V (keys 0, 2, 4, 6, two pieces).
template <int CT, int D, bool V>
__device__ inline int at16(int r, int c) {
  if (CT == kCacheBf16) return r * (2 * D) + ((c ^ (r & 7)) << 4);
  if (D == 128) return r * 128 + ((c ^ (V ? ((r >> 1) & 3) << 1 : (r & 1) << 2)) << 4);
  if (!V) return r * 64 + (c << 4);
  const int slot = (r & ~3) | ((r & 1) << 1) | ((r >> 1) & 1);
  return slot * 64 + ((c ^ (((r >> 2) & 1) << 1)) << 4);
}

template <int CT, int D>
__global__ void __launch_bounds__(32 * kWarps) cache_step_kernel(const __grid_constant__ CacheAttn a) {
  using L = StepL<CT, D>;
  constexpr int KB = L::KB, NT = KB / 8, DT = D / 8;
  extern __shared__ __align__(128) unsigned char step_sm[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  const long long tile = blockIdx.x / a.S;
  const int split = (int)(blockIdx.x - tile * a.S);
  const int b = (int)(tile / a.c.Hkv), h = (int)(tile - (long long)b * a.c.Hkv);
  const SeqLen s = seq_len(a.c, b);
  if (s.nn == 0) return;
  const RowTile rt = row_tile(a, s, 0, 16);
  const int len = rt.hi - rt.lo, parts = split_count(a, len);
  if (split >= parts) return;
  const int keys = split_keys(a, len);
  const int t0 = rt.lo + split * keys, t1 = min(rt.hi, t0 + keys);
  unsigned char* ring = step_sm + warp * L::WARP;

  // this warp's blocks: warp, warp + 4, ... of the split's
  const int nblk = (max(0, t1 - t0) + KB - 1) / KB;
  auto key0 = [&](int i) { return t0 + (warp + kWarps * i) * KB; };
  const int mine = nblk > warp ? (nblk - warp + kWarps - 1) / kWarps : 0;
  auto lookup = [&](int i) -> int {  // page row of key `lane` of block i
    const int t = i < mine ? key0(i) + lane : t1;
    return (KB == 32 || lane < KB) && t < t1 ? (int)row_of(a.c, b, h, t) : -1;
  };
  auto load = [&](int i, int row) {
    if (i < mine) {
      unsigned char* st = ring + (i % L::NS) * L::STAGE;
      const unsigned char* kp = static_cast<const unsigned char*>(a.c.k);
      const unsigned char* vp = static_cast<const unsigned char*>(a.c.v);
      constexpr int RPI = 32 / L::LPR;
      const int c = lane % L::LPR;
#pragma unroll
      for (int j = 0; j < KB / RPI; ++j) {
        const int r = j * RPI + lane / L::LPR;
        const int pr = __shfl_sync(0xffffffffu, row, r);
        const long long off = (long long)max(pr, 0) * L::RB + 16 * c;
        cp16(st + at16<CT, D, false>(r, c), kp + off, pr < 0 ? 0 : 16);
        cp16(st + L::HALF + at16<CT, D, true>(r, c), vp + off, pr < 0 ? 0 : 16);
      }
      if (L::SZ == 1) {
        float* sc = reinterpret_cast<float*>(st + 2 * L::HALF);
        cp4(sc + lane, a.c.ks + max(row, 0), row < 0 ? 0 : 4);
        cp4(sc + KB + lane, a.c.vs + max(row, 0), row < 0 ? 0 : 4);
      }
    }
    cp_commit();
  };
  int row = lookup(0);
#pragma unroll
  for (int i = 0; i < L::NS - 1; ++i) {
    const int next = lookup(i + 1);
    load(i, row);
    row = next;
  }

  // Q fragments (rows g and g + 8, zero past the tile)
  uint32_t q[D / 16][4];
  {
    const __nv_bfloat16* Q = static_cast<const __nv_bfloat16*>(a.Q);
    const bool lg = g < rt.r1, lh = g + 8 < rt.r1;
    const __nv_bfloat16* qg = Q + (lg ? row_at(a, b, h, g).q : 0);
    const __nv_bfloat16* qh = Q + (lh ? row_at(a, b, h, g + 8).q : 0);
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      // columns of the first and second half of the fragment's k = 16
      const int c0 = L::SZ == 2 ? 16 * k + 2 * t4 : (k >> 2) * 64 + 16 * t4 + 4 * (k & 3);
      const int c1 = c0 + (L::SZ == 2 ? 8 : 2);
      q[k][0] = lg ? *reinterpret_cast<const uint32_t*>(qg + c0) : 0;
      q[k][1] = lh ? *reinterpret_cast<const uint32_t*>(qh + c0) : 0;
      q[k][2] = lg ? *reinterpret_cast<const uint32_t*>(qg + c1) : 0;
      q[k][3] = lh ? *reinterpret_cast<const uint32_t*>(qh + c1) : 0;
    }
  }
  const int2 sg = seen(a, s, s.pos0 + g / a.G), sh = seen(a, s, s.pos0 + (g + 8) / a.G);
  const float sl2 = a.scale * kLog2e;

  float o[DT][4];
#pragma unroll
  for (int j = 0; j < DT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
  float m0 = kFloor, m1 = kFloor, l0 = 0.f, l1 = 0.f;  // l: this lane's share
  bool bad = false;

  for (int i = 0; i < mine; ++i) {
    {
      const int next = lookup(i + L::NS);
      load(i + L::NS - 1, row);
      row = next;
    }
    cp_wait<L::NS - 1>();
    __syncwarp();
    const unsigned char* sk = ring + (i % L::NS) * L::STAGE;
    const unsigned char* sv = sk + L::HALF;
    const float* sc = reinterpret_cast<const float*>(sk + 2 * L::HALF);
    const int tb = key0(i);
    float x[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      x[n][0] = x[n][1] = x[n][2] = x[n][3] = 0.f;
      if (L::SZ == 2) {
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t r0, r1, r2, r3;
          ldsm_x4(smem_u32(sk + at16<CT, D, false>(8 * n + (lane & 7), 4 * c + (lane >> 3))), r0, r1, r2, r3);
          mma_bf16(x[n], q[2 * c], r0, r1);
          mma_bf16(x[n], q[2 * c + 1], r2, r3);
        }
      } else {
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          const uint4 w = *reinterpret_cast<const uint4*>(sk + at16<CT, D, false>(8 * n + g, 4 * c + t4));
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            mma_bf16(x[n], q[4 * c + e], bf16_of_bytes<CT>(ww[e], ww[e], 0, 1),
                     bf16_of_bytes<CT>(ww[e], ww[e], 2, 3));
        }
      }
    }
    // logits in base 2, columns 8 n + 2 t4 + {0, 1}
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float2 ks = make_float2(sl2, sl2);
      if (L::SZ == 1) {
        const float2 f = *reinterpret_cast<const float2*>(sc + 8 * n + 2 * t4);
        x[n][0] *= f.x, x[n][1] *= f.y, x[n][2] *= f.x, x[n][3] *= f.y;
      }
      x[n][0] *= ks.x, x[n][1] *= ks.y, x[n][2] *= ks.x, x[n][3] *= ks.y;
    }
    const bool edge = tb < rt.alo || tb + KB > rt.ahi || tb + KB > t1;
    if (edge) {  // the same in the whole warp
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int t = tb + 8 * n + 2 * t4 + (e & 1);
          const int2 ks = e < 2 ? sg : sh;
          if (t < ks.x || t >= ks.y || t >= t1) x[n][e] = -INFINITY;
        }
      if (CT != kCacheI8 && (tb < rt.alo || tb + KB > rt.ahi)) {
        bool f = false;
        for (int e = lane; e < L::HALF / 4; e += 32) {
          const uint32_t w = reinterpret_cast<const uint32_t*>(sv)[e];
          f = f || (CT == kCacheBf16 ? bf16_not_finite(w) : e4m3_not_finite(w));
        }
        bad = bad || __any_sync(0xffffffffu, f);
      }
    }
    float n0 = -INFINITY, n1 = -INFINITY;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      n0 = fmaxf(n0, fmaxf(x[n][0], x[n][1]));
      n1 = fmaxf(n1, fmaxf(x[n][2], x[n][3]));
    }
#pragma unroll
    for (int w = 1; w < 4; w <<= 1) {
      n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, w));
      n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, w));
    }
    const bool v0 = n0 > m0 + kSlack, v1 = n1 > m1 + kSlack;
    if (__any_sync(0xffffffffu, v0 || v1)) {
      const float f0 = v0 ? fast_exp2(m0 - n0) : 1.f, f1 = v1 ? fast_exp2(m1 - n1) : 1.f;
      m0 = v0 ? n0 : m0;
      m1 = v1 ? n1 : m1;
      l0 *= f0;
      l1 *= f1;
#pragma unroll
      for (int j = 0; j < DT; ++j) o[j][0] *= f0, o[j][1] *= f0, o[j][2] *= f1, o[j][3] *= f1;
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      x[n][0] = fast_exp2(x[n][0] - m0);
      x[n][1] = fast_exp2(x[n][1] - m0);
      x[n][2] = fast_exp2(x[n][2] - m1);
      x[n][3] = fast_exp2(x[n][3] - m1);
      l0 += x[n][0] + x[n][1];
      l1 += x[n][2] + x[n][3];
    }
    if (L::SZ == 1) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float2 f = *reinterpret_cast<const float2*>(sc + KB + 8 * n + 2 * t4);
        x[n][0] *= f.x, x[n][1] *= f.y, x[n][2] *= f.x, x[n][3] *= f.y;
      }
      if (edge) {  // a masked key's scale need not be a number
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int t = tb + 8 * n + 2 * t4 + (e & 1);
            const int2 ks = e < 2 ? sg : sh;
            if (t < ks.x || t >= ks.y || t >= t1) x[n][e] = 0.f;
          }
      }
    }
#pragma unroll
    for (int u = 0; u < KB / 16; ++u) {
      const uint32_t p[4] = {bf16_bits2(x[2 * u][0], x[2 * u][1]), bf16_bits2(x[2 * u][2], x[2 * u][3]),
                             bf16_bits2(x[2 * u + 1][0], x[2 * u + 1][1]),
                             bf16_bits2(x[2 * u + 1][2], x[2 * u + 1][3])};
      if (L::SZ == 2) {
#pragma unroll
        for (int j = 0; j < DT; j += 2) {
          uint32_t r0, r1, r2, r3;
          ldsm_x4_t(smem_u32(sv + at16<CT, D, true>(16 * u + (lane & 15), j + (lane >> 4))), r0, r1, r2, r3);
          mma_bf16(o[j], p, r0, r1);
          mma_bf16(o[j + 1], p, r2, r3);
        }
      } else {
        // keys 2 t4, + 1, + 8, + 9 of the 16; output column D / 8 g + j
        constexpr int W = D / 32;  // words of a lane's columns
        uint32_t v[4][W];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = 16 * u + 2 * t4 + (e & 1) + 8 * (e >> 1);
          if (D == 128) {
            const uint4 w = *reinterpret_cast<const uint4*>(sv + at16<CT, D, true>(r, g));
            v[e][0] = w.x, v[e][1] = w.y, v[e][W - 2] = w.z, v[e][W - 1] = w.w;
          } else {
            const uint2 w = *reinterpret_cast<const uint2*>(sv + at16<CT, D, true>(r, g >> 1) + 8 * (g & 1));
            v[e][0] = w.x, v[e][1] = w.y;
          }
        }
#pragma unroll
        for (int j = 0; j < DT; ++j)
          mma_bf16(o[j], p, bf16_of_bytes<CT>(v[0][j >> 2], v[1][j >> 2], j & 3, j & 3),
                   bf16_of_bytes<CT>(v[2][j >> 2], v[3][j >> 2], j & 3, j & 3));
      }
    }
    __syncwarp();  // the block is read: its stage is loaded next
  }
  cp_wait<0>();

  // ---- join the warps --------------------------------------------------------
#pragma unroll
  for (int w = 1; w < 4; w <<= 1) {
    l0 += __shfl_xor_sync(0xffffffffu, l0, w);
    l1 += __shfl_xor_sync(0xffffffffu, l1, w);
  }
  __syncwarp();
  {
    float* jo = reinterpret_cast<float*>(ring);
    float2* jm = reinterpret_cast<float2*>(jo + 16 * D);
#pragma unroll
    for (int j = 0; j < DT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int n = 2 * t4 + (e & 1);
        const int d = L::SZ == 2 ? 8 * j + n : DT * n + j;
        jo[(g + 8 * (e >> 1)) * D + d] = o[j][e];
      }
    if (t4 == 0) {
      jm[g] = make_float2(m0, l0);
      jm[g + 8] = make_float2(m1, l1);
    }
  }
  if (__syncthreads_or(bad)) {
    for (int r = warp; r < rt.r1; r += kWarps)
      redo_row<__nv_bfloat16, CT, D>(a, s, b, h, r, t0, t1, tile, split, parts, 0);
    return;
  }
  for (int e = tid; e < rt.r1 * (D / 8); e += 32 * kWarps) {
    const int r = e / (D / 8), c = e % (D / 8);
    float2 ml[kWarps];
    float m = kFloor, l = 0.f, y[8] = {};
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      ml[w] = reinterpret_cast<const float2*>(step_sm + w * L::WARP + 16 * D * 4)[r];
      m = fmaxf(m, ml[w].x);
    }
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = fast_exp2(ml[w].x - m);
      l += ml[w].y * f;
      const float* jo = reinterpret_cast<const float*>(step_sm + w * L::WARP) + r * D + 8 * c;
#pragma unroll
      for (int u = 0; u < 8; ++u) y[u] = fmaf(jo[u], f, y[u]);
    }
    if (parts > 1) {
      store8(part_o<D>(a, tile, split, r) + 8 * c, y);
      if (c == 0) *part_ml(a, tile, split, r) = make_float2(m, l);
      continue;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int u = 0; u < 8; ++u) y[u] *= inv;
    const RowAt at = row_at(a, b, h, r);
    store8(static_cast<__nv_bfloat16*>(a.O) + at.o + 8 * c, y);
    if (a.lse && c == 0) a.lse[at.lse] = lse_of(m, l);
  }
}

template <int CT, int D>
void launch(const CacheAttn& a, cudaStream_t st) {
  const int smem = StepL<CT, D>::TOTAL;
  cudaFuncSetAttribute(cache_step_kernel<CT, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  const long long blocks = (long long)a.B * a.c.Hkv * a.S;
  cache_step_kernel<CT, D><<<(unsigned)blocks, 32 * kWarps, smem, st>>>(a);
}

}  // namespace

void run_cache_step(const CacheAttn& a, cudaStream_t st) {
  ProfScope ps(st, "cache_step");
  switch (a.type * 2 + (a.c.D == 128)) {
    case 2 * kCacheBf16: return launch<kCacheBf16, 64>(a, st);
    case 2 * kCacheBf16 + 1: return launch<kCacheBf16, 128>(a, st);
    case 2 * kCacheE4m3: return launch<kCacheE4m3, 64>(a, st);
    case 2 * kCacheE4m3 + 1: return launch<kCacheE4m3, 128>(a, st);
    case 2 * kCacheI8: return launch<kCacheI8, 64>(a, st);
    default: return launch<kCacheI8, 128>(a, st);
  }
}

}  // namespace muse
