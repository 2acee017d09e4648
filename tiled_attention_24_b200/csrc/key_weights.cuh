// Accumulated attention weight of a prompt's keys:
//
//   w_j = sum over the query heads h of a key/value head, over the query rows i,
//         of exp(scale q_hi . k_j - lse_hi)          (masked pairs count 0)
//
// with lse the forward's log-sum-exp: the column sums of the attention matrix,
// recomputed from q and k as in the backward, never stored.
//
// The scores are computed transposed, S^T = K Q^T on tcgen05 with keys as rows:
// an epilogue thread owns one key (its tensor-memory lane) and adds up its row,
// no value ever crosses a thread.  The heads of a group follow one another in
// memory, so the group's queries are one matrix of G Nq rows: a window of 32
// queries of 4 heads is one full tile.  A CTA holds one tile of 128 keys and
// streams the query tiles of its part; two CTAs share an SM, so that one's start
// hides behind the other's work.  Roles:
//   warps 0-3, 4-7  epilogue warpgroups, even and odd tiles (thread = key)
//   warp 8          TMA producer: K once, then query tiles, and for each query row
//                   -lse log2(e) and the last key it sees
//   warp 9          MMA issuer, tensor-memory owner
#pragma once
#include "fwd_bf16.cuh"  // wait_bar_drain
#include "ptx.cuh"

namespace ta {

struct KeyWeightsParams {
  const float* lse;        // [B][Hq][Nq]
  float* w;                // rows of `stride` floats, one per (batch, key/value head)
  float* parts_out;        // [parts][B*Hkv][Nkv] where parts > 1
  const int* seqlens;      // [B] or null
  int BHkv, Hkv, group, Nq, Nkv, causal, accumulate;
  int key_tiles, q_tiles, parts, per_part;  // q_tiles of group * Nq rows, per_part of them a part
  long long stride;
  float sl2;
  unsigned long long timeout_ns;
};

template <int D>
struct KeyWCfg {
  static constexpr int THREADS = 320;
  static constexpr int HALF = 128 * 128;                // 128 rows x 64 channels
  static constexpr int TILE = HALF * (D / 64);
  static constexpr int NQ = D == 128 ? 2 : 4, NL = 4;   // query ring, row-value ring
  static constexpr int Q_OFF = TILE;
  static constexpr int L_OFF = Q_OFF + NQ * TILE;       // NL x (128 floats, 128 ints)
  static constexpr int BAR_OFF = L_OFF + NL * 1024;
  static constexpr int SMEM = BAR_OFF + 256 + 1024;     // + alignment slack
  static constexpr uint32_t ID = idesc_bf16_f32(128, 128, false);
};

struct KeyWBars {
  uint64_t k_full, drain;
  uint64_t q_full[4], q_empty[4];
  uint64_t s_full[2], s_free[2];
  uint64_t l_full[4], l_empty[4];
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(KeyWBars) <= 256, "barrier block too large");

// What every role needs to know of a query tile: rows [n0, n1] of the group's matrix
struct KeyWTile {
  int lo, hi;  // smallest and largest query position + offset among its rows
  bool whole;  // 128 rows
};
__device__ __forceinline__ KeyWTile key_w_tile(int n, int Nq, int rows, int off) {
  const int n0 = n * 128, n1 = min(n0 + 128, rows) - 1;
  const int h0 = n0 / Nq, h1 = n1 / Nq;
  KeyWTile t;
  t.lo = (h0 == h1 ? n0 - h0 * Nq : 0) + off;
  t.hi = (h0 == h1 ? n1 - h0 * Nq : Nq - 1) + off;
  t.whole = n1 - n0 == 127;
  return t;
}

template <int D>
__global__ void __launch_bounds__(KeyWCfg<D>::THREADS, 2)
    key_weights_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const KeyWeightsParams p) {
  using C = KeyWCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  KeyWBars* bars = reinterpret_cast<KeyWBars*>(smem + C::BAR_OFF);
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &bars->abort;

  // the first key tiles see the most queries when causal: they come first
  const int bhk = blockIdx.x % p.BHkv;
  const int rest = blockIdx.x / p.BHkv;
  const int part = rest % p.parts, J = rest / p.parts * 128;
  const int b = bhk / p.Hkv, off = p.Nkv - p.Nq;
  const int len = p.seqlens ? min(max(p.seqlens[b], 0), p.Nkv) : p.Nkv;
  const int rows = p.group * p.Nq;
  const int q0 = part * p.per_part, q1 = J < len ? min(q0 + p.per_part, p.q_tiles) : q0;
  auto active = [&](const KeyWTile& t) { return t.lo < len && (!p.causal || t.hi >= J); };

  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&bars->k_full), 1);
    mbar_init(smem_u32(&bars->drain), 1);
    for (int i = 0; i < C::NQ; ++i) {
      mbar_init(smem_u32(&bars->q_full[i]), 1);
      mbar_init(smem_u32(&bars->q_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bars->s_full[i]), 1);
      mbar_init(smem_u32(&bars->s_free[i]), 4);
    }
    for (int i = 0; i < C::NL; ++i) {
      mbar_init(smem_u32(&bars->l_full[i]), 1);
      mbar_init(smem_u32(&bars->l_empty[i]), 4);
    }
    bars->abort = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(&bars->tmem_base), 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = bars->tmem_base;
  float w = 0.f, comp = 0.f;  // an epilogue thread's sum and its compensation

  if (warp == 8) {
    // ================================================================ producer
    const float* lse = p.lse + (size_t)bhk * rows;
    auto next = [&](int n) {  // first tile >= n that is computed
      while (n < q1 && !active(key_w_tile(n, p.Nq, rows, off))) ++n;
      return n;
    };
    float l[4];
    auto fetch = [&](int n) {  // the tile's lse, one tile ahead of its use
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = n * 128 + lane + 32 * e;
        l[e] = n < q1 && row < rows ? lse[row] : 0.f;
      }
    };
    int s = 0, n = next(q0);
    fetch(n);
    if (lane == 0 && n < q1) {
      prefetch_tmap(&tmQ);
      prefetch_tmap(&tmK);
      mbar_arrive_expect_tx(smem_u32(&bars->k_full), C::TILE);
      for (int h = 0; h < D / 64; ++h)
        tma_load_3d(sbase + h * C::HALF, &tmK, smem_u32(&bars->k_full), h * 64, J, bhk);
    }
    while (n < q1) {
      const int st = s % C::NQ, sl = s % C::NL;
      if (!__all_sync(0xffffffffu, wait_bar(smem_u32(&bars->q_empty[st]), ((s / C::NQ) & 1) ^ 1, abort_flag, p.timeout_ns)))
        break;
      if (lane == 0) {
        const uint32_t qb = smem_u32(&bars->q_full[st]);
        mbar_arrive_expect_tx(qb, C::TILE);
        for (int h = 0; h < D / 64; ++h)
          tma_load_2d(sbase + C::Q_OFF + st * C::TILE + h * C::HALF, &tmQ, qb, h * 64, bhk * rows + n * 128);
      }
      ++s;  // this tile's copy is in flight
      float v[4];
      int lim[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = n * 128 + lane + 32 * e, pos = row % p.Nq + off;
        const bool in = row < rows && pos < len;
        // a row that sees no key has lse = -inf: it gives nothing
        v[e] = !in || l[e] == -INFINITY ? -INFINITY : -l[e] * 1.4426950408889634f;
        lim[e] = !in ? -1 : p.causal ? pos : 0x7fffffff;
      }
      n = next(n + 1);
      fetch(n);
      if (!__all_sync(0xffffffffu, wait_bar(smem_u32(&bars->l_empty[sl]), (((s - 1) / C::NL) & 1) ^ 1, abort_flag, p.timeout_ns)))
        break;
      float* fv = reinterpret_cast<float*>(smem + C::L_OFF + sl * 1024);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        fv[lane + 32 * e] = v[e];
        reinterpret_cast<int*>(fv)[128 + lane + 32 * e] = lim[e];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->l_full[sl]));
    }
    // never leave a copy in flight (after a normal run these have all completed)
    if (lane == 0 && s > 0) {
      wait_bar_drain(smem_u32(&bars->k_full), 0, p.timeout_ns);
      for (int back = 1; back <= C::NQ && s - back >= 0; ++back)
        wait_bar_drain(smem_u32(&bars->q_full[(s - back) % C::NQ]), ((s - back) / C::NQ) & 1, p.timeout_ns);
    }
    __syncwarp();
  } else if (warp == 9) {
    // ================================================================ MMA issuer
    if (lane == 0) {
      bool ok = true;
      int s = 0;
      for (int n = q0; n < q1; ++n) {
        if (!active(key_w_tile(n, p.Nq, rows, off))) continue;
        if (s == 0 && !(ok = spin_bar(smem_u32(&bars->k_full), 0, abort_flag, p.timeout_ns))) break;
        const int st = s % C::NQ, buf = s & 1;
        if (!(ok = spin_bar(smem_u32(&bars->q_full[st]), (s / C::NQ) & 1, abort_flag, p.timeout_ns))) break;
        if (!(ok = spin_bar(smem_u32(&bars->s_free[buf]), ((s >> 1) & 1) ^ 1, abort_flag, p.timeout_ns))) break;
        tc_fence_after();
        const uint64_t dK = smem_desc(sbase, 16, 1024), dQ = smem_desc(sbase + C::Q_OFF + st * C::TILE, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t o = (uint64_t)(((kk >> 2) * C::HALF + (kk & 3) * 32) >> 4);
          mma_f16_ss(tbase + buf * 128, dK + o, dQ + o, C::ID, kk > 0);
        }
        tc_commit(smem_u32(&bars->s_full[buf]));
        tc_commit(smem_u32(&bars->q_empty[st]));
        ++s;
      }
      if (!ok) {  // every MMA issued so far must finish before TMEM is freed
        tc_commit(smem_u32(&bars->drain));
        wait_bar_drain(smem_u32(&bars->drain), 0, p.timeout_ns);
      }
    }
    __syncwarp();
  } else {
    // ================================================================ epilogue
    const int wg = warp >> 2, j = J + (warp & 3) * 32 + lane;
    const uint32_t tS = tbase + wg * 128 + ((uint32_t)((warp & 3) * 32) << 16);
    const uint64_t sc = f2(p.sl2, p.sl2);
    int s = 0;
    for (int n = q0; n < q1; ++n) {
      const KeyWTile t = key_w_tile(n, p.Nq, rows, off);
      if (!active(t)) continue;
      const int seq = s++;
      if ((seq & 1) != wg) continue;
      const int sl = seq % C::NL;
      bool ok = wait_bar(smem_u32(&bars->l_full[sl]), (seq / C::NL) & 1, abort_flag, p.timeout_ns) &&
                wait_bar(smem_u32(&bars->s_full[wg]), (seq >> 1) & 1, abort_flag, p.timeout_ns);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const float* fv = reinterpret_cast<const float*>(smem + C::L_OFF + sl * 1024);
      const int* lim = reinterpret_cast<const int*>(fv) + 128;
      const bool masked = !t.whole || t.hi >= len || (p.causal && t.lo < J + 127);
      // partial sums of 32 terms each; the tile's sum joins the running one with
      // compensation: over thousands of queries plain fp32 sums drift by 1e-6
      uint64_t a0 = f2(0.f, 0.f), a1 = a0;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t x[2][32];
        tmem_ld32(tS + half * 64, x[0]);
        tmem_ld32(tS + half * 64 + 32, x[1]);
        tmem_ld_wait(x[0]);
        tmem_ld_wait(x[1]);
        if (half == 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bars->s_free[wg]));
        }
#pragma unroll
        for (int i = 0; i < 64; i += 4) {
          const float4 v = *reinterpret_cast<const float4*>(fv + half * 64 + i);
          float e0, e1, e2, e3;
          const uint32_t* xi = &x[i >> 5][i & 31];
          f2_split(ffma2(f2(__uint_as_float(xi[0]), __uint_as_float(xi[1])), sc, f2(v.x, v.y)), e0, e1);
          f2_split(ffma2(f2(__uint_as_float(xi[2]), __uint_as_float(xi[3])), sc, f2(v.z, v.w)), e2, e3);
          e0 = ex2(e0), e1 = ex2(e1), e2 = ex2(e2), e3 = ex2(e3);
          if (masked) {
            const int4 m = *reinterpret_cast<const int4*>(lim + half * 64 + i);
            e0 = j <= m.x ? e0 : 0.f, e1 = j <= m.y ? e1 : 0.f, e2 = j <= m.z ? e2 : 0.f, e3 = j <= m.w ? e3 : 0.f;
          }
          a0 = fadd2(a0, f2(e0, e1));
          a1 = fadd2(a1, f2(e2, e3));
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->l_empty[sl]));
      float b0, b1;
      f2_split(fadd2(a0, a1), b0, b1);
      const float y = (b0 + b1) - comp, z = w + y;
      comp = (z - w) - y;
      w = z;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tbase, 256);
  }
  float* other = reinterpret_cast<float*>(smem + C::L_OFF);  // the ring is no longer read
  if (warp >= 4 && warp < 8) other[threadIdx.x - 128] = w;
  __syncthreads();
  if (warp < 4) {
    const int j = J + threadIdx.x;
    if (j < p.Nkv) {
      w += other[threadIdx.x];
      if (j >= len) w = 0.f;
      if (p.parts > 1) {
        p.parts_out[((size_t)part * p.BHkv + bhk) * p.Nkv + j] = w;
      } else {
        float* out = p.w + bhk * p.stride + j;
        *out = p.accumulate ? *out + w : w;
      }
    }
  }
}

// joins the parts, always in the same order
__global__ void __launch_bounds__(256) key_weights_join_kernel(const KeyWeightsParams p) {
  const int bhk = blockIdx.y, j = blockIdx.x * 256 + threadIdx.x;
  if (j >= p.Nkv) return;
  float w = 0.f;
  for (int k = 0; k < p.parts; ++k) w += p.parts_out[((size_t)k * p.BHkv + bhk) * p.Nkv + j];
  float* out = p.w + bhk * p.stride + j;
  *out = p.accumulate ? *out + w : w;
}

// no query at all
__global__ void __launch_bounds__(256) key_weights_none_kernel(float* w, long long stride, int Nkv) {
  const int j = blockIdx.x * 256 + threadIdx.x;
  if (j < Nkv) w[blockIdx.y * stride + j] = 0.f;
}

}  // namespace ta
