// Decode over the 4-bit cache (row format: kv4.cuh): one query row per (batch,
// query head) against the live slots [0, seqlens[b]) of its cache head,
//
//   x_j = scale log2(e) q . k_j,  m = max x_j,  l = sum 2^(x_j - m),
//   o = sum 2^(x_j - m) v_j / l,  lse = ln 2 (m + log2 l),
//   and, where asked for, w_j += sum over the heads of a cache head of
//   2^(x_j - lse log2(e)), the accumulated attention weight of a slot.
//
// Split-KV as in decode.cuh: each chunk of slots leaves a normalised partial
// result and its log-sum-exp, decode_kv4_combine_kernel merges them.  A weight
// needs the log-sum-exp of the whole row, so the split kernel leaves the
// scores x in the workspace and a last kernel turns them into weights.
#pragma once
#include <cuda_fp16.h>

#include "fwd_bf16.cuh"  // wait_bar_drain
#include "fwd_fp4.cuh"   // bulk_load
#include "kv4.cuh"

namespace ta {

struct DecKv4Params {
  const uint16_t* q;             // [B][Hq][D] bf16
  const uint8_t *kc, *vc;        // [B][Hkv][cap][D/2]
  const uint16_t *ks, *vs;       // [B][Hkv][cap][D/32] bf16
  float *o_part, *lse_part;      // [B*Hq][S][D], [B*Hq][S]
  float* x;                      // [B*Hq][cap] scores, or null
  const int* seqlens;            // [B]
  int Hkv, group, cap, S;
  int blocks;                    // blocks of <= 8 query heads per cache head
  float sl2;
  unsigned long long timeout_ns;
};

template <int NG>
struct DecKv4Cfg {
  static constexpr int D = 32 * NG;
  static constexpr int WARPS = 8, TILE = 32;          // slots per pipeline stage of a warp
  static constexpr int STAGES = NG == 4 ? 3 : 6;
  static constexpr int CODES = TILE * D / 2, SCALES = TILE * NG * 2;
  static constexpr int STAGE = 2 * (CODES + SCALES);  // K codes, V codes, K scales, V scales
  static constexpr int RING = WARPS * STAGES * STAGE;
  static constexpr int ML_OFF = RING;                 // running max and sum of each warp and head
  static constexpr int BAR_OFF = ML_OFF + WARPS * 8 * 8;
  static constexpr int SMEM = BAR_OFF + WARPS * STAGES * 8 + 16;
  // lazy rescale: the reference max moves when a score exceeds it by TAU (log2
  // units); probabilities are taken 2^-TAU smaller, so that none exceeds 1
  static constexpr float TAU = 8.f;
};
static_assert(DecKv4Cfg<4>::WARPS * 8 * 128 * 4 <= DecKv4Cfg<4>::RING, "partial outputs reuse the ring");
static_assert(DecKv4Cfg<2>::WARPS * 8 * 64 * 4 <= DecKv4Cfg<2>::RING, "partial outputs reuse the ring");

__device__ __forceinline__ void mma_f16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// transpose of an 8x8 matrix of 16-bit elements held two per lane
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ float bf2f(uint32_t w, int hi) { return __uint_as_float(hi ? (w & 0xFFFF0000u) : (w << 16)); }

// NG words of a row's scales as floats
__device__ __forceinline__ void kv4_scales(const uint2& w, float (&f)[4]) {
  f[0] = bf2f(w.x, 0), f[1] = bf2f(w.x, 1), f[2] = bf2f(w.y, 0), f[3] = bf2f(w.y, 1);
}
__device__ __forceinline__ void kv4_scales(const uint32_t& w, float (&f)[2]) { f[0] = bf2f(w, 0), f[1] = bf2f(w, 1); }

// One CTA: one block of <= 8 query heads of a cache head, one chunk of its slots.
// Each warp walks its own tiles of 32 slots (every 8th of the chunk) through its
// own ring of bulk copies and keeps its own running max, sum and output; the
// warps meet once, at the end.  Per 16 slots, r = lane / 4, t = lane % 4:
//
//   S^T = K Q^T   m16n8k16 f16, rows = slots, columns = heads, per channel group:
//     A is a code's offset form n = c + 8 straight in the low bits of an fp16, a
//     subnormal of value n 2^-24 (nibbles 0 and 2 of a halfword) or 16 n 2^-24
//     (nibbles 1 and 3, whose q carries 1/16): masking is all the conversion there
//     is.  B is q times a power of two per head that brings its largest channel
//     to [2^14, 2^15): exact in fp16 down to 2^-27 of that channel.  The
//     accumulators start from -8 sum q, which takes the offset out again.
//   O^T = V^T P^T  m16n8k16 bf16, rows = channels, columns = heads: A is c exactly
//     (128 + n by one logic operation, minus 136), B is p times the slot's scale
//     of the group, rounded to bf16: the one rounding of P, as in the bf16 decode
//     (fp16 would need a common exponent for the scales of V; the offset form
//     would cancel against a sum far larger than the result on long rows).
template <int NG>
__global__ void __launch_bounds__(256, 2) decode_kv4_kernel(const DecKv4Params p) {
  using C = DecKv4Cfg<NG>;
  using T = typename Kv4Piece<NG>::T;
  constexpr int D = C::D;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;

  const int c = blockIdx.x % p.S;
  const int hb = blockIdx.x / p.S;                     // (batch, cache head, block of heads)
  const int bhk = hb / p.blocks, blk = hb - bhk * p.blocks;
  const int heads = min(8, p.group - blk * 8);
  const size_t bh0 = (size_t)bhk * p.group + blk * 8;  // first query head (batch * Hq + head)
  const int len = min(max(p.seqlens[bhk / p.Hkv], 0), p.cap);
  const int tiles = (len + C::TILE - 1) / C::TILE;
  const int per = (tiles + p.S - 1) / p.S;             // tiles per chunk
  const int t0 = min(c * per, tiles), t1 = min(t0 + per, tiles);
  const int mine = max(0, (t1 - t0 - warp + C::WARPS - 1) / C::WARPS);

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF) + warp * C::STAGES;
  int* abort_flag = reinterpret_cast<int*>(smem + C::BAR_OFF + C::WARPS * C::STAGES * 8);
  uint8_t* ring = smem + warp * C::STAGES * C::STAGE;
  const size_t row0 = (size_t)bhk * p.cap;
  if (threadIdx.x == 0) *abort_flag = 0;
  if (lane == 0) {
    for (int s = 0; s < C::STAGES; ++s) mbar_init(smem_u32(&bars[s]), 1);
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  auto issue = [&](int i) {  // lane 0: tile i of this warp into stage i % STAGES
    const int slot = (t0 + warp + i * C::WARPS) * C::TILE;
    const uint32_t rows = (uint32_t)min(C::TILE, (len - slot + 15) & ~15);  // capacity is a multiple of 16
    const uint32_t dst = smem_u32(ring + (i % C::STAGES) * C::STAGE), bar = smem_u32(&bars[i % C::STAGES]);
    mbar_arrive_expect_tx(bar, rows * (D + 4 * NG));
    bulk_load(dst, p.kc + (row0 + slot) * (D / 2), rows * (D / 2), bar);
    bulk_load(dst + 2 * C::CODES, p.ks + (row0 + slot) * NG, rows * NG * 2, bar);
    bulk_load(dst + C::CODES, p.vc + (row0 + slot) * (D / 2), rows * (D / 2), bar);
    bulk_load(dst + 2 * C::CODES + C::SCALES, p.vs + (row0 + slot) * NG, rows * NG * 2, bar);
  };
  if (lane == 0)
    for (int i = 0; i < min(mine, C::STAGES); ++i) issue(i);

  // ---- queries: head r, channels 32 g + 8 t + 0..7 of each group, as B fragments
  uint32_t qb[NG][4];
  float c0[NG][2];  // accumulator start of heads 2t, 2t + 1
  float fa[2], fb[2];
  {
    uint4 w[NG];
    uint32_t m = 0;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      w[g] = r < heads ? *reinterpret_cast<const uint4*>(p.q + (bh0 + r) * D + 32 * g + 8 * t) : make_uint4(0, 0, 0, 0);
      const uint32_t a = __vmaxu2(__vmaxu2(w[g].x & 0x7FFF7FFFu, w[g].y & 0x7FFF7FFFu),
                                  __vmaxu2(w[g].z & 0x7FFF7FFFu, w[g].w & 0x7FFF7FFFu));
      m = max(m, max(a & 0xFFFFu, a >> 16));
    }
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    // largest channel in [2^e, 2^(e+1)) (below the normal numbers: e = -126); a
    // head with an infinity or a NaN is left as it is, its outputs are NaN anyway
    const int e = m >= 0x7F80u ? 14 : max(1, (int)(m >> 7)) - 127;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const uint32_t ww[4] = {w[g].x, w[g].y, w[g].z, w[g].w};
      float f[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = ldexpf(bf2f(ww[i], 0), 14 - e);
        f[2 * i + 1] = ldexpf(bf2f(ww[i], 1), 14 - e) * 0.0625f;
      }
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // nibble i of the two halfwords: channels i and 4 + i
        const __half2 h = __floats2half2_rn(f[i], f[4 + i]);
        qb[g][i] = *reinterpret_cast<const uint32_t*>(&h);
        sum += (__low2float(h) + __high2float(h)) * ((i & 1) ? 16.f : 1.f);
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      sum *= -8.f * 0x1p-24f;
      c0[g][0] = __shfl_sync(0xffffffffu, sum, 8 * t);
      c0[g][1] = __shfl_sync(0xffffffffu, sum, 8 * t + 4);
    }
    // x = score * sl2 * 2^(24 + e - 14), the power of two in two factors
    const int eh = (e + 10) / 2;
    const float a = ldexpf(1.f, eh), b = ldexpf(p.sl2, e + 10 - eh);
    fa[0] = __shfl_sync(0xffffffffu, a, 8 * t), fa[1] = __shfl_sync(0xffffffffu, a, 8 * t + 4);
    fb[0] = __shfl_sync(0xffffffffu, b, 8 * t), fb[1] = __shfl_sync(0xffffffffu, b, 8 * t + 4);
  }

  float acc[2 * NG][4];
#pragma unroll
  for (int i = 0; i < 2 * NG; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  __syncwarp();
  __syncthreads();  // the abort flag is set up

  bool ok = true;
  int done = 0;
  for (int i = 0; i < mine; ++i) {
    const int st = i % C::STAGES;
    ok = __all_sync(0xffffffffu, wait_bar(smem_u32(&bars[st]), (i / C::STAGES) & 1, abort_flag, p.timeout_ns));
    if (!ok) break;
    done = i + 1;
    const uint8_t* buf = ring + st * C::STAGE;
    const int slot0 = (t0 + warp + i * C::WARPS) * C::TILE;
#pragma unroll 1
    for (int sub = 0; sub < C::TILE; sub += 16) {
      const int left = len - slot0 - sub;  // live slots from here on
      if (left <= 0) break;
      // ---- scores of 16 slots
      float x[4] = {0.f, 0.f, 0.f, 0.f};
      {
        uint32_t kw[2][NG];
        float sc[2][NG];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = sub + r + 8 * h;
          if constexpr (NG == 4) {
            const uint4 w = *reinterpret_cast<const uint4*>(buf + row * 64 + t * 16);
            kw[h][0] = __byte_perm(w.x, w.z, 0x5410), kw[h][1] = __byte_perm(w.x, w.z, 0x7632);
            kw[h][2] = __byte_perm(w.y, w.w, 0x5410), kw[h][3] = __byte_perm(w.y, w.w, 0x7632);
          } else {
            const uint2 w = *reinterpret_cast<const uint2*>(buf + row * 32 + t * 8);
            kw[h][0] = __byte_perm(w.x, w.y, 0x5410), kw[h][1] = __byte_perm(w.x, w.y, 0x7632);
          }
          kv4_scales(*reinterpret_cast<const T*>(buf + 2 * C::CODES + row * NG * 2), sc[h]);
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          float s[4] = {c0[g][0], c0[g][1], c0[g][0], c0[g][1]};
          const uint32_t a = kw[0][g], b = kw[1][g], a8 = a >> 8, b8 = b >> 8;
          mma_f16_16816(s, (a & 0x000F000Fu) ^ 0x00080008u, (b & 0x000F000Fu) ^ 0x00080008u,
                        (a & 0x00F000F0u) ^ 0x00800080u, (b & 0x00F000F0u) ^ 0x00800080u, qb[g][0], qb[g][1]);
          mma_f16_16816(s, (a8 & 0x000F000Fu) ^ 0x00080008u, (b8 & 0x000F000Fu) ^ 0x00080008u,
                        (a8 & 0x00F000F0u) ^ 0x00800080u, (b8 & 0x00F000F0u) ^ 0x00800080u, qb[g][2], qb[g][3]);
          x[0] = fmaf(s[0], sc[0][g], x[0]);
          x[1] = fmaf(s[1], sc[0][g], x[1]);
          x[2] = fmaf(s[2], sc[1][g], x[2]);
          x[3] = fmaf(s[3], sc[1][g], x[3]);
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = x[e] * fa[e & 1] * fb[e & 1];
      float sc[2][NG];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        kv4_scales(*reinterpret_cast<const T*>(buf + 2 * C::CODES + C::SCALES + (sub + r + 8 * h) * NG * 2), sc[h]);
      if (left < 16) {  // slots behind the live ones: no score, and their scales may be anything
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (r + 8 * h >= left) {
            x[2 * h] = x[2 * h + 1] = -INFINITY;
#pragma unroll
            for (int g = 0; g < NG; ++g) sc[h][g] = 0.f;
          }
      }
      if (p.x) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (2 * t + (e & 1) < heads && r + 8 * (e >> 1) < left)
            p.x[(bh0 + 2 * t + (e & 1)) * p.cap + slot0 + sub + r + 8 * (e >> 1)] = x[e];
      }
      // ---- running max, moved only when it must
      const float h0 = fmaxf(x[0], x[2]), h1 = fmaxf(x[1], x[3]);
      if (__any_sync(0xffffffffu, h0 > m[0] + C::TAU || h1 > m[1] + C::TAU)) {
        float mx[2] = {h0, h1};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], o));
          mx[k] = fmaxf(mx[k], m[k]);
          const float f = mx[k] == -INFINITY ? 1.f : ex2(m[k] - mx[k]);
          l[k] *= f;
#pragma unroll
          for (int n = 0; n < 2 * NG; ++n) acc[n][k] *= f, acc[n][k + 2] *= f;
          m[k] = mx[k];
        }
      }
      float pr[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float mm = m[e & 1];
        pr[e] = ex2(x[e] - ((mm == -INFINITY ? 0.f : mm) + C::TAU));
      }
      l[0] += pr[0] + pr[2];
      l[1] += pr[1] + pr[3];
      // ---- values: piece r of slots 2t, 2t + 1, 2t + 8, 2t + 9
      T vw[4];
#pragma unroll
      for (int h = 0; h < 4; ++h)
        vw[h] = *reinterpret_cast<const T*>(buf + C::CODES + (sub + 2 * t + (h & 1) + 8 * (h >> 1)) * (D / 2) + r * 2 * NG);
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const uint32_t b0 = movmatrix_trans(pack_bf16(pr[0] * sc[0][g], pr[1] * sc[0][g]));
        const uint32_t b1 = movmatrix_trans(pack_bf16(pr[2] * sc[1][g], pr[3] * sc[1][g]));
        uint32_t a[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t w0, w1;
          if constexpr (NG == 4) {
            w0 = g < 2 ? vw[2 * h].x : vw[2 * h].y;
            w1 = g < 2 ? vw[2 * h + 1].x : vw[2 * h + 1].y;
          } else {
            w0 = vw[2 * h], w1 = vw[2 * h + 1];
          }
          a[h] = __byte_perm(w0, w1, (g & 1) ? 0x7632 : 0x5410);
        }
        uint32_t f[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int n = 0; n < 4; ++n)
            f[h][n] = sub_bf16x2(((a[h] >> (4 * n)) & 0x000F000Fu) ^ 0x43084308u, 0x43084308u);
        mma_bf16_16816(acc[2 * g], f[0][0], f[0][1], f[1][0], f[1][1], b0, b1);
        mma_bf16_16816(acc[2 * g + 1], f[0][2], f[0][3], f[1][2], f[1][3], b0, b1);
      }
    }
    __syncwarp();
    if (lane == 0 && i + C::STAGES < mine) issue(i + C::STAGES);
  }
  if (!ok) {  // never leave a copy in flight
    for (int i = done; i < min(mine, done + C::STAGES); ++i)
      wait_bar_drain(smem_u32(&bars[i % C::STAGES]), (i / C::STAGES) & 1, p.timeout_ns);
  }

  // ---- the warps' results meet: max, sums and outputs through shared memory
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) l[k] += __shfl_xor_sync(0xffffffffu, l[k], o);
  float2* ml = reinterpret_cast<float2*>(smem + C::ML_OFF);
  if (r == 0) {
    ml[warp * 8 + 2 * t] = make_float2(m[0], l[0]);
    ml[warp * 8 + 2 * t + 1] = make_float2(m[1], l[1]);
  }
  __syncthreads();  // and every warp is done with its ring
  float* op = reinterpret_cast<float*>(smem);  // [warp][head][channel]
#pragma unroll
  for (int n = 0; n < 2 * NG; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      op[(warp * 8 + 2 * t + (e & 1)) * D + 32 * (n >> 1) + 4 * r + 2 * (n & 1) + (e >> 1)] = acc[n][e];
  __syncthreads();
  for (int i = threadIdx.x; i < heads * D; i += 256) {
    const int h = i / D, ch = i % D;
    float mx = -INFINITY, tot = 0.f, o = 0.f;
#pragma unroll
    for (int w = 0; w < C::WARPS; ++w) mx = fmaxf(mx, ml[w * 8 + h].x);
#pragma unroll
    for (int w = 0; w < C::WARPS; ++w) {
      const float2 v = ml[w * 8 + h];
      // a warp without slots has sum 0; one whose scores are all NaN has no max but a NaN sum
      const float f = v.x == mx ? 1.f : ex2(v.x - mx);
      tot = fmaf(v.y, f, tot);
      o = fmaf(op[(w * 8 + h) * D + ch], f, o);
    }
    const size_t part = (bh0 + h) * p.S + c;
    const bool live = t1 > t0;
    p.o_part[part * D + ch] = live ? o / tot : 0.f;
    if (ch == 0) p.lse_part[part] = live ? ((mx == -INFINITY ? 0.f : mx) + C::TAU + log2f(tot)) * 0.69314718055994531f : -INFINITY;
  }
}

// Merge of a row's chunks: LSE = log sum_c exp(LSE_c), O = sum_c exp(LSE_c - LSE) O_c.
// A chunk without slots has LSE_c = -inf; a NaN in a live slot stays a NaN.
template <int D>
__global__ void __launch_bounds__(D)
    decode_kv4_combine_kernel(const float* __restrict__ o_part, const float* __restrict__ lse_part,
                              uint16_t* __restrict__ o, float* __restrict__ lse, int S) {
  const int bh = blockIdx.x, e = threadIdx.x;
  const float* lp = lse_part + (size_t)bh * S;
  float mx = -INFINITY;
  bool any = false;
  for (int c = 0; c < S; ++c) {
    any |= !(lp[c] == -INFINITY);
    mx = fmaxf(mx, lp[c]);
  }
  float tot = 0.f, acc = 0.f;
  for (int c = 0; any && c < S; ++c) {
    const float w = ex2((lp[c] - mx) * 1.4426950408889634f);
    tot += w;
    acc = fmaf(w, o_part[((size_t)bh * S + c) * D + e], acc);
  }
  o[(size_t)bh * D + e] = (uint16_t)(pack_bf16(any ? acc / tot : 0.f, 0.f) & 0xFFFFu);
  if (e == 0) lse[bh] = any ? mx + logf(tot) : -INFINITY;
}

// w_j += sum_h 2^(x_hj - lse_h log2 e) over the query heads of one cache head
__global__ void __launch_bounds__(256)
    decode_kv4_weights_kernel(const float* __restrict__ x, const float* __restrict__ lse, float* __restrict__ weights,
                              const int* __restrict__ seqlens, int Hq, int Hkv, int cap) {
  const int bhk = blockIdx.y, group = Hq / Hkv;
  const int j = blockIdx.x * 256 + threadIdx.x;
  if (j >= min(max(seqlens[bhk / Hkv], 0), cap)) return;
  float sum = 0.f;
  for (int h = 0; h < group; ++h) {
    const size_t bh = (size_t)bhk * group + h;
    sum += ex2(x[bh * cap + j] - lse[bh] * 1.4426950408889634f);
  }
  weights[(size_t)bhk * cap + j] += sum;
}

}  // namespace ta
