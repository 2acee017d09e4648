// Accumulated attention weight of a prompt's keys:
//
//   w_j = sum over the query heads h of a key/value head, over the query rows i,
//         of exp(scale q_hi . k_j - lse_hi)          (masked pairs count 0)
//
// with lse the forward's log-sum-exp: the column sums of the attention matrix,
// recomputed from q and k as in the backward, never stored.
#pragma once
#include "ptx.cuh"

namespace ta {

struct KeyWeightsParams {
  const uint16_t *q, *k;   // [B][Hq][Nq][D], [B][Hkv][Nkv][D] bf16
  const float* lse;        // [B][Hq][Nq]
  float* w;                // rows of `stride` floats, one per (batch, cache head)
  const int* seqlens;      // [B] or null
  int Hq, Hkv, Nq, Nkv, causal, accumulate;
  long long stride;
  float sl2;
};

// thread = key, its row in registers; query rows pass through shared memory
template <int D>
__global__ void __launch_bounds__(128) key_weights_kernel(const KeyWeightsParams p) {
  constexpr int QT = 16;
  __shared__ float qs[QT][D];
  __shared__ float ls[QT];
  const int bhk = blockIdx.y, b = bhk / p.Hkv, group = p.Hq / p.Hkv;
  const int j = blockIdx.x * 128 + threadIdx.x;
  const int off = p.Nkv - p.Nq;
  const int len = p.seqlens ? min(max(p.seqlens[b], 0), p.Nkv) : p.Nkv;
  const int rows = max(0, min(p.Nq, len - off));
  uint32_t kr[D / 2];
#pragma unroll
  for (int e = 0; e < D / 2; ++e)
    kr[e] = j < len ? reinterpret_cast<const uint32_t*>(p.k + ((size_t)bhk * p.Nkv + j) * D)[e] : 0u;
  float w = 0.f;
  const int first = p.causal ? max(0, (int)blockIdx.x * 128 - off) : 0;
  for (int h = 0; h < group; ++h) {
    const size_t bh = (size_t)b * p.Hq + (size_t)(bhk % p.Hkv) * group + h;
    for (int i0 = first; i0 < rows; i0 += QT) {
      const int n = min(QT, rows - i0);
      __syncthreads();
      for (int e = threadIdx.x; e < n * D; e += 128)
        qs[e / D][e % D] = __uint_as_float((uint32_t)p.q[(bh * p.Nq + i0) * D + e] << 16);
      if (threadIdx.x < n) {
        const float l = p.lse[bh * p.Nq + i0 + threadIdx.x];
        ls[threadIdx.x] = l == -INFINITY ? -INFINITY : -l * 1.4426950408889634f;  // a row that sees no key
      }
      __syncthreads();
      for (int i = 0; i < n; ++i) {
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < D / 2; ++e) {
          s = fmaf(__uint_as_float(kr[e] << 16), qs[i][2 * e], s);
          s = fmaf(__uint_as_float(kr[e] & 0xFFFF0000u), qs[i][2 * e + 1], s);
        }
        if (!p.causal || j <= i0 + i + off) w += ex2(fmaf(s, p.sl2, ls[i]));
      }
    }
  }
  if (j >= p.Nkv) return;
  float* out = p.w + bhk * p.stride + j;
  if (j >= len) w = 0.f;
  *out = p.accumulate ? *out + w : w;
}

}  // namespace ta
