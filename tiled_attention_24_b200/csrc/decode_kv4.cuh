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

// d = a b + c, f16 operands, f32 accumulation
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1, float c0, float c1, float c2, float c3) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
// transpose of an 8x8 matrix of 16-bit elements held two per lane
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// (a & MASK) ^ flip in one logic operation
template <uint32_t MASK>
__device__ __forceinline__ uint32_t and_xor(uint32_t a, uint32_t flip) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(d) : "r"(a), "n"(MASK), "r"(flip));
  return d;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// two fp32 -> packed f16x2 (round to nearest even), `lo` in the low half
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ float bf2f(uint32_t w, int hi) { return __uint_as_float(hi ? (w & 0xFFFF0000u) : (w << 16)); }

// word i (two groups) of a row's scales
__device__ __forceinline__ uint32_t kv4_word(const uint2& w, int i) { return i ? w.y : w.x; }
__device__ __forceinline__ uint32_t kv4_word(const uint32_t& w, int) { return w; }

// One CTA: one block of <= 8 query heads of a cache head, one chunk of its slots.
// Each warp walks its own tiles of 32 slots (every 8th of the chunk) through its
// own ring of bulk copies and keeps its own running max, sum and output; the
// warps meet once, at the end.  Per 16 slots, r = lane / 4, t = lane % 4:
//
// Both products run on m16n8k16 f16 with the codes as the A operand.  A code's
// offset form n = c + 8 sits in the low bits of an fp16 and is one as it is: a
// subnormal of value n 2^-24 (nibbles 0 and 2 of a halfword) or 16 n 2^-24
// (nibbles 1 and 3).  Masking (with the flip of the sign bit, one logic operation)
// is all the conversion there is; one shift serves the two upper nibbles.
//
//   S^T = K Q^T, rows = slots, columns = heads, one channel group at a time:
//     B is q times a power of two per head that brings its largest channel to
//     [2^14, 2^15), exact in fp16 down to 2^-27 of that channel; the odd
//     nibbles' channels carry 1/16.  The accumulators start from -8 sum q, which
//     takes the offset out again, and each group's sum is scaled in fp32.
//   O^T = V^T P^T, rows = channels, columns = heads: B is p times the slot's scale
//     of the group, rounded to fp16 (the one rounding of P, 2^-11), with p
//     taken times a power of two that keeps p s below 2^15.  That power follows
//     the largest scale met so far as the running max follows the scores, so
//     a product counts from 2^-31 of the largest on.  The offset goes out tile by
//     tile through a second product with the constant -8: summed up over a long
//     row it would swamp the result.
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
  // per head 2t, 2t + 1: reference max of y (scores before fb), threshold above which
  // it moves, exponent M that probabilities are taken against; vref = 2^ev, bf16x2
  float my[2] = {-INFINITY, -INFINITY}, thr[2] = {-INFINITY, -INFINITY}, M[2] = {0.f, 0.f}, l[2] = {0.f, 0.f};
  int ev = -100;
  uint32_t vref = (uint32_t)((127 - 100) << 7) * 0x10001u;
  const uint32_t flip0 = 0x00080008u, flip1 = 0x00800080u;
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
    const int left = len - slot0;  // live slots from here on
    // ---- scores of 32 slots: [16-slot half][slot r or r + 8, head 2t or 2t + 1]
    float y[2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      uint32_t kw[2][NG];
      T sc[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = 16 * u + r + 8 * h;
        if constexpr (NG == 4) {
          const uint4 w = *reinterpret_cast<const uint4*>(buf + row * 64 + t * 16);
          kw[h][0] = __byte_perm(w.x, w.z, 0x5410), kw[h][1] = __byte_perm(w.x, w.z, 0x7632);
          kw[h][2] = __byte_perm(w.y, w.w, 0x5410), kw[h][3] = __byte_perm(w.y, w.w, 0x7632);
        } else {
          const uint2 w = *reinterpret_cast<const uint2*>(buf + row * 32 + t * 8);
          kw[h][0] = __byte_perm(w.x, w.y, 0x5410), kw[h][1] = __byte_perm(w.x, w.y, 0x7632);
        }
        sc[h] = *reinterpret_cast<const T*>(buf + 2 * C::CODES + row * NG * 2);
      }
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        float s[4];
        const uint32_t a = kw[0][g], b = kw[1][g], a8 = a >> 8, b8 = b >> 8;
        mma_f16_16816(s, and_xor<0x000F000Fu>(a, flip0), and_xor<0x000F000Fu>(b, flip0),
                      and_xor<0x00F000F0u>(a, flip1), and_xor<0x00F000F0u>(b, flip1), qb[g][0], qb[g][1], c0[g][0],
                      c0[g][1], c0[g][0], c0[g][1]);
        mma_f16_16816(s, and_xor<0x000F000Fu>(a8, flip0), and_xor<0x000F000Fu>(b8, flip0),
                      and_xor<0x00F000F0u>(a8, flip1), and_xor<0x00F000F0u>(b8, flip1), qb[g][2], qb[g][3], s[0], s[1],
                      s[2], s[3]);
        const float f0 = bf2f(kv4_word(sc[0], g >> 1), g & 1), f1 = bf2f(kv4_word(sc[1], g >> 1), g & 1);
        y[u][0] = g ? fmaf(s[0], f0, y[u][0]) : s[0] * f0;
        y[u][1] = g ? fmaf(s[1], f0, y[u][1]) : s[1] * f0;
        y[u][2] = g ? fmaf(s[2], f1, y[u][2]) : s[2] * f1;
        y[u][3] = g ? fmaf(s[3], f1, y[u][3]) : s[3] * f1;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) y[u][e] *= fa[e & 1];
    }
    T vs[2][2];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        vs[u][h] = *reinterpret_cast<const T*>(buf + 2 * C::CODES + C::SCALES + (16 * u + r + 8 * h) * NG * 2);
    if (left < C::TILE) {  // slots behind the live ones: no score, and their scales may be anything
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (16 * u + r + 8 * h >= left) {
            y[u][2 * h] = y[u][2 * h + 1] = -INFINITY;
            vs[u][h] = T{};
          }
    }
    if (p.x) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = 16 * u + r + 8 * (e >> 1);
          if (2 * t + (e & 1) < heads && j < left)
            p.x[(bh0 + 2 * t + (e & 1)) * p.cap + slot0 + j] = y[u][e] * fb[e & 1];
        }
    }
    // ---- references, moved only when they must
    const float h0 = fmaxf(fmaxf(y[0][0], y[0][2]), fmaxf(y[1][0], y[1][2]));
    const float h1 = fmaxf(fmaxf(y[0][1], y[0][3]), fmaxf(y[1][1], y[1][3]));
    uint32_t vm = vref;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int w = 0; w < NG / 2; ++w) vm = max_bf16x2(vm, kv4_word(vs[u][h], w));
    if (__any_sync(0xffffffffu, h0 > thr[0] || h1 > thr[1] || vm != vref)) {
      uint32_t v = max(vm & 0xFFFFu, vm >> 16);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
      const int ev_new = v > (vref & 0xFFFFu) ? (int)(v >> 7) - 126 : ev;
      float mx[2] = {h0, h1};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], o));
        if (!(mx[k] > my[k])) mx[k] = my[k];
        if (mx[k] != -INFINITY) {
          const float Mn = fmaf(mx[k], fb[k], C::TAU + (float)(ev_new - 15));
          const float f = my[k] == -INFINITY ? 0.f : ex2(M[k] - Mn);  // l and acc are 0 or NaN while my = -inf
          l[k] *= f;
#pragma unroll
          for (int n = 0; n < 2 * NG; ++n) acc[n][k] *= f, acc[n][k + 2] *= f;
          my[k] = mx[k];
          M[k] = Mn;
          thr[k] = mx[k] + C::TAU / fb[k];
        }
      }
      ev = ev_new;
      vref = (uint32_t)((127 + ev) << 7) * 0x10001u;
    }
    float pr[2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int e = 0; e < 4; ++e) pr[u][e] = ex2(fmaf(y[u][e], fb[e & 1], -M[e & 1]));
      l[0] += pr[u][0] + pr[u][2];
      l[1] += pr[u][1] + pr[u][3];
    }
    // ---- values: piece r of slots 2t, 2t + 1, 2t + 8, 2t + 9 of each half
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      T vw[4];
#pragma unroll
      for (int h = 0; h < 4; ++h)
        vw[h] = *reinterpret_cast<const T*>(buf + C::CODES + (16 * u + 2 * t + (h & 1) + 8 * (h >> 1)) * (D / 2) + r * 2 * NG);
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const float f0 = bf2f(kv4_word(vs[u][0], g >> 1), g & 1), f1 = bf2f(kv4_word(vs[u][1], g >> 1), g & 1);
        const uint32_t b0 = movmatrix_trans(pack_f16(pr[u][0] * f0, pr[u][1] * f0));
        const uint32_t b1 = movmatrix_trans(pack_f16(pr[u][2] * f1, pr[u][3] * f1));
        uint32_t a[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          a[h] = __byte_perm(kv4_word(vw[2 * h], g >> 1), kv4_word(vw[2 * h + 1], g >> 1), (g & 1) ? 0x7632 : 0x5410);
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          float(&o)[4] = acc[2 * g + n];
          mma_f16_16816(o, 0x80088008u, 0x80808080u, 0x80088008u, 0x80808080u, b0, b1, o[0], o[1], o[2], o[3]);
          const uint32_t w0 = n ? a[0] >> 8 : a[0], w1 = n ? a[1] >> 8 : a[1];
          mma_f16_16816(o, and_xor<0x000F000Fu>(w0, flip0), and_xor<0x00F000F0u>(w0, flip1),
                        and_xor<0x000F000Fu>(w1, flip0), and_xor<0x00F000F0u>(w1, flip1), b0, b1, o[0], o[1], o[2], o[3]);
        }
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
    ml[warp * 8 + 2 * t] = make_float2(my[0] == -INFINITY ? -INFINITY : M[0], l[0]);
    ml[warp * 8 + 2 * t + 1] = make_float2(my[1] == -INFINITY ? -INFINITY : M[1], l[1]);
  }
  __syncthreads();  // and every warp is done with its ring
  float* op = reinterpret_cast<float*>(smem);  // [warp][head][channel]
#pragma unroll
  for (int n = 0; n < 2 * NG; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      op[(warp * 8 + 2 * t + (e & 1)) * D + 32 * (n >> 1) + 4 * r + 2 * (n & 1) + (e >> 1)] =
          acc[n][e] * ((e >> 1) ? 0x1p20f : 0x1p24f);  // odd nibbles carry 16
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
    if (ch == 0) p.lse_part[part] = live ? ((mx == -INFINITY ? 0.f : mx) + log2f(tot)) * 0.69314718055994531f : -INFINITY;
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
