// Decode over the 4-bit cache (row format: kv4.cuh): one query row per (batch,
// query head) against the live slots [0, seqlens[b]) of its cache head,
//
//   x_j = scale log2(e) q . k_j,  m = max x_j,  l = sum 2^(x_j - m),
//   o = sum 2^(x_j - m) v_j / l,  lse = ln 2 (m + log2 l),
//   and, where asked for, w_j += sum over the heads of a cache head of
//   2^(x_j - lse log2(e)), the accumulated attention weight of a slot.
//
// Split-KV as in decode.cuh: each chunk of slots leaves a normalised partial
// result and its log-sum-exp, decode_combine_kernel merges them.  A weight
// needs the log-sum-exp of the whole row, so the split kernel leaves the
// scores x in the workspace and a last kernel turns them into weights.
#pragma once
#include "decode.cuh"
#include "kv4.cuh"

namespace ta {

struct DecKv4Params {
  const uint16_t* q;             // [B][Hq][D] bf16
  const uint8_t *kc, *vc;        // [B][Hkv][cap][D/2]
  const uint16_t *ks, *vs;       // [B][Hkv][cap][D/32] bf16
  float *o_part, *lse_part;      // [B*Hq][S][D], [B*Hq][S]
  float* x;                      // [B*Hq][cap] scores, or null
  const int* seqlens;            // [B]
  int Hq, group, cap, S;
  float sl2;
};

// One CTA per (query head, chunk): thread = slot for the scores, thread =
// channel for the values.
template <int NG>
__global__ void __launch_bounds__(128) decode_kv4_kernel(const DecKv4Params p) {
  constexpr int D = 32 * NG;
  using T = typename Kv4Piece<NG>::T;
  __shared__ float qs[D];
  __shared__ float ps[128];
  __shared__ float red[4];
  const int bh = blockIdx.x / p.S, c = blockIdx.x % p.S;
  const int tid = threadIdx.x;
  const int len = min(max(p.seqlens[bh / p.Hq], 0), p.cap);
  const int chunk = (len + p.S - 1) / p.S;
  const long long j0 = (long long)c * chunk;
  const int nk = (int)max(0LL, min((long long)len, j0 + chunk) - j0);
  const size_t base = (size_t)(bh / p.group) * p.cap + j0;
  if (tid < D) qs[tid] = __uint_as_float((uint32_t)p.q[(size_t)bh * D + tid] << 16);
  __syncthreads();
  float m = -INFINITY, l = 0.f, acc = 0.f;
  for (int s0 = 0; s0 < nk; s0 += 128) {
    const int ns = min(128, nk - s0);
    float x = -INFINITY;
    if (tid < ns) {
      const size_t row = base + s0 + tid;
      const T sc = *reinterpret_cast<const T*>(p.ks + row * NG);
      float a[NG];
#pragma unroll
      for (int g = 0; g < NG; ++g) a[g] = 0.f;
      for (int u = 0; u < 8; ++u) {
        const T w = reinterpret_cast<const T*>(p.kc + row * (D / 2))[u];
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
          for (int i = 0; i < 4; ++i) a[g] = fmaf(kv4_code(kv4_half(w, g), i), qs[32 * g + 4 * u + i], a[g]);
      }
      float s = 0.f;
#pragma unroll
      for (int g = 0; g < NG; ++g) s = fmaf(a[g], kv4_scale(kv4_half(sc, g)), s);
      x = s * p.sl2;
      if (p.x) p.x[(size_t)bh * p.cap + j0 + s0 + tid] = x;
    }
    float mx = x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if ((tid & 31) == 0) red[tid >> 5] = mx;
    __syncthreads();
    const float m_new = fmaxf(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])), m);
    const float f = (m == -INFINITY) ? 0.f : ex2(m - m_new);
    const float ref = (m_new == -INFINITY) ? 0.f : m_new;
    ps[tid] = tid < ns ? ex2(x - ref) : 0.f;
    m = m_new;
    __syncthreads();
    l *= f;
    acc *= f;
    for (int j = 0; j < ns; ++j) {
      l += ps[j];
      if (tid < D) {
        const size_t row = base + s0 + j;
        const int g = tid >> 5, u = (tid & 31) >> 2;
        const uint32_t h = reinterpret_cast<const uint16_t*>(p.vc + row * (D / 2))[u * NG + g];
        acc = fmaf(ps[j] * kv4_scale(p.vs[row * NG + g]), kv4_code(h, tid & 3), acc);
      }
    }
    __syncthreads();
  }
  const size_t part = (size_t)bh * p.S + c;
  if (tid < D) p.o_part[part * D + tid] = nk > 0 ? acc / l : 0.f;
  if (tid == 0) p.lse_part[part] = nk > 0 ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
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
