// Attention of single tokens (and of a few: up to 32 packed rows a kv-head)
// over the paged cache, bf16 queries.
//
// One CTA of four warps takes a split of one (sequence, kv-head)'s keys.  The
// bound is the cache's bytes: each warp streams blocks of keys of its own
// through a ring of shared memory (cp.async, several blocks in flight, no
// block-wide barrier in the loop) and keeps its own online softmax, so that
// warps drift apart and loads never stop; they join once, at the end, in a
// fixed order.  Products run on mma.sync m16n8k16: with at most 32 rows a
// tile of the fifth-generation tensor cores would be three quarters padding,
// and its results would take the way over TMEM.
//   S = Q K^T     K rows as the B operand.  The contraction's order is free,
//                 so an 8-bit row is read 16 bytes a lane and Q's columns are
//                 permuted to match; converted in registers to fp16 (half the
//                 instructions of bf16), Q's rows brought into fp16's range by
//                 powers of two.
//   o += P V      V as the B operand: ldmatrix.trans (bf16), or pairs of bytes
//                 from neighbouring keys' rows (8-bit) with the output columns
//                 permuted to match.
// Scales of 8-bit rows multiply S's columns and P's columns (before its one
// rounding to bf16).  Up to eight splits are one thread-block cluster and join
// through its distributed shared memory (one launch, no workspace traffic);
// more leave partials for cache_join_kernel.
//
// Measured: 64 sequences of up to 16384 tokens, 32 heads over 8 of 128, bf16:
// 389 us, 6.6 TB/s of cache, a copy's rate.  8 sequences of up to 65536 of 64 in
// e4m3: 89 us, 63 %: conversions and masks fill the integer pipe.  Five tokens
// each (20 rows) over int8 of 128: 66 us, 26 %: two row tiles leave two warps a
// scheduler, whose latencies bound it.  One token at 1000: 8.2 us, the chain
// launch, lengths, pages, rows, join.
#include <cooperative_groups.h>

#include "cache_attn.cuh"
#include "kernels.h"
#include "mma_sync.cuh"

namespace muse {

namespace {

constexpr int kWarps = 4;

template <int CT, int D, int MT>
struct StepL {
  static constexpr int SZ = CT == kCacheBf16 ? 2 : 1;
  static constexpr int KB = SZ * D > 128 ? 16 : 32;  // keys of a block
  static constexpr int RB = SZ * D;                  // bytes of a row
  static constexpr int LPR = RB / 16;                // lanes of a row's load
  static constexpr int HALF = KB * RB;               // K (or V) of a block
  static constexpr int SCALES = SZ == 1 ? 2 * KB * 4 : 0;
  static constexpr int STAGE = 2 * HALF + SCALES;
  // stages of a warp's ring: two for 8-bit rows, so that one more CTA fits an SM
  // (5 ragged sequences of up to 33147, 16 heads of 128, e4m3: 93 -> 82 us; 26 of
  // 18349, 16 of 64: 236 -> 224)
  static constexpr int NS = SZ == 1 && MT == 1 ? 2 : 3;
  static constexpr int RING = NS * STAGE;
  static constexpr int ROWS = 16 * MT;
  static constexpr int JOIN = ROWS * D * 4 + ROWS * 8;  // o, (m, l) of a warp
  static constexpr int WARP = RING > JOIN ? RING : JOIN;
  static constexpr int Q = kWarps * WARP, QP = 2 * D + 16;  // query rows, padded against bank conflicts
  static constexpr int TOTAL = Q + ROWS * QP;
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

// Column of query element d: for an 8-bit cache the order in which a lane's 16
// bytes of a K row meet the k = 16 steps.
template <bool k8>
__device__ inline int q_column(int d) {
  if (!k8) return d;
  const int t = (d >> 4) & 3, k = (d >> 2) & 3, e = d & 3;
  return (d & 64) + 16 * k + 2 * t + (e & 1) + 8 * (e >> 1);
}

// MT m16 tiles of rows; with HR = 1 row half of the one tile (up to 8 rows): the
// lanes' second rows are left out.
template <int CT, int D, int MT, int HR, bool CL>
__global__ void __launch_bounds__(32 * kWarps) cache_step_kernel(const __grid_constant__ CacheAttn a) {
  using L = StepL<CT, D, MT>;
  constexpr int KB = L::KB, NT = KB / 8, DT = D / 8;
  constexpr bool k8 = L::SZ == 1;
  constexpr int XE = 2 * HR;  // a lane's logits of an n8 tile that are used
  extern __shared__ __align__(128) unsigned char step_sm[];
  __shared__ float qback[L::ROWS];  // 8-bit: the power of two that undoes a row's factor
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  const Place at0 = place_of(a);
  const int tile = at0.tile, split = at0.split, b = at0.b, h = at0.h;
  const SeqLen s = seq_len(a.c, b);
  if (s.nn == 0) return;
  const RowTile rt = row_tile(a, s, 0, L::ROWS);
  const int len = rt.hi - rt.lo, parts = split_count(a, len);
  if (split >= parts && (!CL || parts == 1)) return;
  const int keys = split_keys(a, len);
  const int t0 = min(rt.hi, rt.lo + split * keys), t1 = min(rt.hi, t0 + keys);
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

  // the query rows (zero past the tile), four threads a row
  for (int r = tid >> 2; r < L::ROWS; r += 8 * kWarps) {
    const bool live = r < rt.r1;
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.Q) + (live ? row_at(a, b, h, r).q : 0);
    unsigned char* dst = step_sm + L::Q + r * L::QP;
    uint4 v[D / 32];
    float top = 0.f;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {  // columns 8 t4 + 32 c ..
      v[c] = live ? *reinterpret_cast<const uint4*>(src + 8 * t4 + 32 * c) : make_uint4(0, 0, 0, 0);
      if (!k8) {
        *reinterpret_cast<uint4*>(dst + 16 * t4 + 64 * c) = v[c];
      } else {
        float x[8];
        load8_in(reinterpret_cast<const __nv_bfloat16*>(&v[c]), x);
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[e]));
      }
    }
    if (k8) {
      // a maximum in [2^14, 2^15): exact for values down to 2^-31 of it
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const float2 f = half_factor(top);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        float x[8];
        load8_in(reinterpret_cast<const __nv_bfloat16*>(&v[c]), x);
#pragma unroll
        for (int e = 0; e < 8; e += 2)
          *reinterpret_cast<uint32_t*>(dst + 2 * q_column<k8>(8 * t4 + 32 * c + e)) = pack_h2(x[e] * f.x, x[e + 1] * f.x);
      }
      if (t4 == 0) qback[r] = f.y;
    }
  }
  __syncthreads();
  int2 see[MT][HR];   // of rows 16 i + g and 16 i + g + 8
  float mul[MT][HR];  // their product to base-2 logit
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int e = 0; e < HR; ++e) {
      const int r = 16 * i + 8 * e + g;
      see[i][e] = seen(a, s, s.pos0 + div_by(a.by_G, r));
      see[i][e].y = min(see[i][e].y, t1);
      mul[i][e] = a.scale * kLog2e * (k8 ? qback[r] : 1.f);
    }

  float o[MT][DT][4], m[MT][HR], l[MT][HR];  // l: this lane's share
#pragma unroll
  for (int i = 0; i < MT; ++i) {
#pragma unroll
    for (int e = 0; e < HR; ++e) m[i][e] = kFloor, l[i][e] = 0.f;
#pragma unroll
    for (int j = 0; j < DT; ++j) o[i][j][0] = o[i][j][1] = o[i][j][2] = o[i][j][3] = 0.f;
  }
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
    float x[MT][NT][4] = {};
    // two (bf16) or four (8-bit) k = 16 steps at a time
    constexpr int KS = k8 ? 4 : 2;
#pragma unroll
    for (int c = 0; c < D / (16 * KS); ++c) {
      uint32_t q[MT][KS][4];
#pragma unroll
      for (int u = 0; u < MT; ++u)
#pragma unroll
        for (int e = 0; e < KS; ++e)
          ldsm_x4(smem_u32(step_sm + L::Q + (16 * u + (lane & 15)) * L::QP + 32 * (KS * c + e) + 16 * (lane >> 4)),
                  q[u][e][0], q[u][e][1], q[u][e][2], q[u][e][3]);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (!k8) {
          uint32_t r0, r1, r2, r3;
          ldsm_x4(smem_u32(sk + at16<CT, D, false>(8 * n + (lane & 7), 4 * c + (lane >> 3))), r0, r1, r2, r3);
#pragma unroll
          for (int u = 0; u < MT; ++u) {
            mma_bf16(x[u][n], q[u][0], r0, r1);
            mma_bf16(x[u][n], q[u][KS / 2], r2, r3);
          }
        } else {
          const uint4 w = *reinterpret_cast<const uint4*>(sk + at16<CT, D, false>(8 * n + g, 4 * c + t4));
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint2 kk = half_of_word<CT>(ww[e]);
#pragma unroll
            for (int u = 0; u < MT; ++u) mma_f16(x[u][n], q[u][e % KS], kk.x, kk.y);
          }
        }
      }
    }
    // logits in base 2, columns 8 n + 2 t4 + {0, 1}
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float2 f = make_float2(1.f, 1.f);
      if (k8) f = *reinterpret_cast<const float2*>(sc + 8 * n + 2 * t4);
#pragma unroll
      for (int u = 0; u < MT; ++u)
#pragma unroll
        for (int e = 0; e < XE; ++e) {
          x[u][n][e] *= k8 ? mul[u][e >> 1] * (e & 1 ? f.y : f.x) : mul[u][e >> 1];
        }
    }
    const bool edge = tb < rt.alo || tb + KB > rt.ahi || tb + KB > t1;
    auto masked = [&](int u, int n, int e) {
      const int t = tb + 8 * n + 2 * t4 + (e & 1);
      return t < see[u][e >> 1].x || t >= see[u][e >> 1].y;
    };
    if (edge) {  // the same in the whole warp
#pragma unroll
      for (int u = 0; u < MT; ++u)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < XE; ++e)
            if (masked(u, n, e)) x[u][n][e] = -INFINITY;
      if (CT != kCacheI8 && (tb < rt.alo || tb + KB > rt.ahi)) {
        bool f = false;
        for (int e = lane; e < L::HALF / 4; e += 32) {
          const uint32_t w = reinterpret_cast<const uint32_t*>(sv)[e];
          f = f || (CT == kCacheBf16 ? bf16_not_finite(w) : e4m3_not_finite(w));
        }
        bad = bad || __any_sync(0xffffffffu, f);
      }
    }
    float top[MT][HR];
    bool moves = false;
#pragma unroll
    for (int u = 0; u < MT; ++u)
#pragma unroll
      for (int e = 0; e < HR; ++e) {
        float y = -INFINITY;
#pragma unroll
        for (int n = 0; n < NT; ++n) y = max3(y, x[u][n][2 * e], x[u][n][2 * e + 1]);
        y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 1));
        y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 2));
        top[u][e] = y;
        moves = moves || y > m[u][e] + kSlack;
      }
    if (__any_sync(0xffffffffu, moves)) {
#pragma unroll
      for (int u = 0; u < MT; ++u) {
        float f[2] = {1.f, 1.f};
#pragma unroll
        for (int e = 0; e < HR; ++e) {
          const bool v = top[u][e] > m[u][e] + kSlack;
          f[e] = v ? fast_exp2(m[u][e] - top[u][e]) : 1.f;
          m[u][e] = v ? top[u][e] : m[u][e];
          l[u][e] *= f[e];
        }
#pragma unroll
        for (int j = 0; j < DT; ++j) {
          o[u][j][0] *= f[0], o[u][j][1] *= f[0];
          if (HR == 2) o[u][j][2] *= f[1], o[u][j][3] *= f[1];
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float2 f = make_float2(1.f, 1.f);
      if (k8) f = *reinterpret_cast<const float2*>(sc + KB + 8 * n + 2 * t4);
#pragma unroll
      for (int u = 0; u < MT; ++u)
#pragma unroll
        for (int e = 0; e < XE; ++e) {
          const float y = fast_exp2(x[u][n][e] - m[u][e >> 1]);
          l[u][e >> 1] += y;
          x[u][n][e] = k8 ? y * (e & 1 ? f.y : f.x) : y;
          // a masked key's scale need not be a number
          if (k8 && edge && masked(u, n, e)) x[u][n][e] = 0.f;
        }
    }
#pragma unroll
    for (int k = 0; k < KB / 16; ++k) {
      uint32_t p[MT][4];
#pragma unroll
      for (int u = 0; u < MT; ++u) {
        p[u][0] = bf16_bits2(x[u][2 * k][0], x[u][2 * k][1]);
        p[u][1] = HR == 2 ? bf16_bits2(x[u][2 * k][2], x[u][2 * k][3]) : 0;
        p[u][2] = bf16_bits2(x[u][2 * k + 1][0], x[u][2 * k + 1][1]);
        p[u][3] = HR == 2 ? bf16_bits2(x[u][2 * k + 1][2], x[u][2 * k + 1][3]) : 0;
      }
      if (!k8) {
#pragma unroll
        for (int j = 0; j < DT; j += 2) {
          uint32_t r0, r1, r2, r3;
          ldsm_x4_t(smem_u32(sv + at16<CT, D, true>(16 * k + (lane & 15), j + (lane >> 4))), r0, r1, r2, r3);
#pragma unroll
          for (int u = 0; u < MT; ++u) {
            mma_bf16(o[u][j], p[u], r0, r1);
            mma_bf16(o[u][j + 1], p[u], r2, r3);
          }
        }
      } else {
        // keys 2 t4, + 1, + 8, + 9 of the 16; output column D / 8 g + j
        constexpr int W = D / 32;  // words of a lane's columns
        uint32_t v[4][W];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = 16 * k + 2 * t4 + (e & 1) + 8 * (e >> 1);
          if (D == 128) {
            const uint4 w = *reinterpret_cast<const uint4*>(sv + at16<CT, D, true>(r, g));
            v[e][0] = w.x, v[e][1] = w.y, v[e][W - 2] = w.z, v[e][W - 1] = w.w;
          } else {
            const uint2 w = *reinterpret_cast<const uint2*>(sv + at16<CT, D, true>(r, g >> 1) + 8 * (g & 1));
            v[e][0] = w.x, v[e][1] = w.y;
          }
        }
#pragma unroll
        for (int w = 0; w < W; ++w) {
          uint32_t b0[4], b1[4];
          bf16_pairs<CT>(v[0][w], v[1][w], b0);
          bf16_pairs<CT>(v[2][w], v[3][w], b1);
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int u = 0; u < MT; ++u) mma_bf16(o[u][4 * w + j], p[u], b0[j], b1[j]);
        }
      }
    }
    __syncwarp();  // the block is read: its stage is loaded next
  }
  cp_wait<0>();

  // ---- join the warps --------------------------------------------------------
  __syncwarp();
  {
    float* jo = reinterpret_cast<float*>(ring);
    float2* jm = reinterpret_cast<float2*>(jo + L::ROWS * D);
#pragma unroll
    for (int u = 0; u < MT; ++u)
#pragma unroll
      for (int e = 0; e < HR; ++e) {
        l[u][e] += __shfl_xor_sync(0xffffffffu, l[u][e], 1);
        l[u][e] += __shfl_xor_sync(0xffffffffu, l[u][e], 2);
        const int r = 16 * u + 8 * e + g;
#pragma unroll
        for (int j = 0; j < DT; ++j)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int n = 2 * t4 + c;
            jo[r * D + (k8 ? DT * n + j : 8 * j + n)] = o[u][j][2 * e + c];
          }
        if (t4 == 0) jm[r] = make_float2(m[u][e], l[u][e]);
      }
  }
  // The CTA's o, m, l of columns [8 c, 8 c + 8) of row r: the result, a partial
  // in the workspace, or one for the cluster (in place of the first warp's).
  float* co = reinterpret_cast<float*>(step_sm);
  __shared__ float2 cml[L::ROWS];
  auto finish = [&](int r, int c, float (&y)[8], float mr, float lr) {
    const float inv = lr == 0.f ? 0.f : 1.f / lr;
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] *= inv;
    const RowAt at = row_at(a, b, h, r);
    store8(static_cast<__nv_bfloat16*>(a.O) + at.o + 8 * c, y);
    if (a.lse && c == 0) a.lse[at.lse] = lse_of(mr, lr);
  };
  auto emit = [&](int r, int c, float (&y)[8], float mr, float lr) {
    if (parts == 1) return finish(r, c, y, mr, lr);
    if (CL) {
      store8(co + r * D + 8 * c, y);
      if (c == 0) cml[r] = make_float2(mr, lr);
    } else {
      store8(part_o<D>(a, tile, split, r) + 8 * c, y);
      if (c == 0) *part_ml(a, tile, split, r) = make_float2(mr, lr);
    }
  };
  if (__syncthreads_or(bad)) {
    for (int r = warp; r < rt.r1; r += kWarps) {
      float y[8], mr, lr;
      row_over_keys<__nv_bfloat16, CT, D>(a, s, b, h, r, t0, t1, y, mr, lr);
      if (lane < D / 8) emit(r, lane, y, lr == 0.f ? kFloor : mr, lr);
    }
  } else {
    for (int e = tid; e < rt.r1 * (D / 8); e += 32 * kWarps) {
      const int r = e / (D / 8), c = e % (D / 8);
      float2 ml[kWarps];
      float mr = kFloor, lr = 0.f, y[8] = {};
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        ml[w] = reinterpret_cast<const float2*>(step_sm + w * L::WARP + L::ROWS * D * 4)[r];
        mr = fmaxf(mr, ml[w].x);
      }
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = fast_exp2(ml[w].x - mr);
        lr += ml[w].y * f;
        const float* jo = reinterpret_cast<const float*>(step_sm + w * L::WARP) + r * D + 8 * c;
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = fmaf(jo[i], f, y[i]);
      }
      emit(r, c, y, mr, lr);
    }
  }
  if (!CL || parts == 1) return;

  // ---- join the cluster's splits, every CTA a share of the columns -------------
  auto cluster = cooperative_groups::this_cluster();
  cluster.sync();
  for (int e = split * 32 * kWarps + tid; e < rt.r1 * (D / 8); e += a.S * 32 * kWarps) {
    const int r = e / (D / 8), c = e % (D / 8);
    float mr = kFloor, lr = 0.f, y[8] = {};
    float2 ml[8];
    float z[8][8];
#pragma unroll
    for (int p = 0; p < 8; ++p) {  // every load on its way before the first is used
      ml[p] = make_float2(kFloor, 0.f);
      if (p < parts) {
        ml[p] = cluster.map_shared_rank(cml, p)[r];
        load8_in(cluster.map_shared_rank(co, p) + r * D + 8 * c, z[p]);
      }
    }
#pragma unroll
    for (int p = 0; p < 8; ++p) mr = fmaxf(mr, ml[p].x);
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      if (p >= parts) break;
      const float f = fast_exp2(ml[p].x - mr);
      lr += ml[p].y * f;
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = fmaf(z[p][i], f, y[i]);
    }
    finish(r, c, y, mr, lr);
  }
  cluster.sync();  // no CTA leaves while another reads its shared memory
}

template <int CT, int D, int MT, int HR, bool CL>
void launch(const CacheAttn& a, cudaStream_t st) {
  const int smem = StepL<CT, D, MT>::TOTAL;
  auto* kernel = cache_step_kernel<CT, D, MT, HR, CL>;
  static LargeShared allowed;
  allowed.ensure((const void*)kernel, smem);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((long long)a.B * a.c.Hkv * a.S));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = a.S;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = CL ? 1 : 0;
  cudaLaunchKernelEx(&cfg, kernel, a);
}
template <int CT, int D>
void launch_as(const CacheAttn& a, cudaStream_t st) {
  if (a.rows == 8)
    a.cluster ? launch<CT, D, 1, 1, true>(a, st) : launch<CT, D, 1, 1, false>(a, st);
  else if (a.rows == 16)
    a.cluster ? launch<CT, D, 1, 2, true>(a, st) : launch<CT, D, 1, 2, false>(a, st);
  else
    a.cluster ? launch<CT, D, 2, 2, true>(a, st) : launch<CT, D, 2, 2, false>(a, st);
}

}  // namespace

void run_cache_step(const CacheAttn& a, cudaStream_t st) {
  ProfScope ps(st, "cache_step");
  switch (a.type * 2 + (a.c.D == 128)) {
    case 2 * kCacheBf16: return launch_as<kCacheBf16, 64>(a, st);
    case 2 * kCacheBf16 + 1: return launch_as<kCacheBf16, 128>(a, st);
    case 2 * kCacheE4m3: return launch_as<kCacheE4m3, 64>(a, st);
    case 2 * kCacheE4m3 + 1: return launch_as<kCacheE4m3, 128>(a, st);
    case 2 * kCacheI8: return launch_as<kCacheI8, 64>(a, st);
    default: return launch_as<kCacheI8, 128>(a, st);
  }
}

}  // namespace muse
