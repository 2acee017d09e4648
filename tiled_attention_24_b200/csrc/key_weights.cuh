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
// queries of 4 heads is one full tile.  An item is two tiles of 128 keys and a
// part of the query tiles; every query tile serves both key tiles.  CTAs are
// persistent, one to an SM, and the next item's keys load while this one's
// queries run, so that short items (a window) stream K at memory speed.  Roles:
//   warps 0-3, 4-7  epilogue warpgroups of key tile 0 and 1 (two score buffers each)
//   warp 8          TMA producer; per query row -lse log2(e) and the last key it
//                   sees, and what the other roles need to know of a step
//   warp 9          MMA issuer, tensor-memory owner
// Bound by the exponentials, one a score (MUFU 61 % busy; 64 us of them alone), and the
// hand-over of tiles: 4096 causal queries, 32 / 8 heads, d = 128: 110 us; the last 32
// queries of 4 x 16384 keys: 41 us, K at 3.4 TB/s.
#pragma once
#include <type_traits>

#include "exp2_poly5.cuh"
#include "fwd_bf16.cuh"  // wait_bar_drain
#include "ptx.cuh"

namespace ta {

struct KeyWeightsParams {
  const float* lse;        // [B][Hq][Nq]
  float* w;                // rows of `stride` floats, one per (batch, key/value head)
  float* parts_out;        // [parts][B*Hkv][Nkv] where parts > 1
  const int* seqlens;      // [B] or null
  int BHkv, Hkv, group, Nq, Nkv, causal, accumulate;
  int items, q_tiles, parts;  // q_tiles of group * Nq rows
  long long stride;
  float sl2;
  unsigned long long timeout_ns;
};

template <int D>
struct KeyWCfg {
  static constexpr int THREADS = 320;
  static constexpr int HALF = 128 * 128;                // 128 rows x 64 channels
  static constexpr int TILE = HALF * (D / 64);
  static constexpr int NS = D == 128 ? 6 : 12, NL = 4;  // tiles of K or Q, steps
  static constexpr int L_OFF = NS * TILE;               // NL x (128 floats, 128 ints)
  static constexpr int BAR_OFF = L_OFF + NL * 1024;
  static constexpr int SMEM = BAR_OFF + 512 + 1024;     // + alignment slack
  static constexpr uint32_t ID = idesc_bf16_f32(128, 128, false);
};

// One step of the ring that keeps the roles together: a query tile of an item, or
// (no key tile active) the whole of an item without any, or the end.
struct KeyWStep {
  int flags;  // KEYW_*
  int slots;  // shared-memory tiles: query tile, key tile 0 << 8, key tile 1 << 16
  int J, bhk, part;
};
enum { KEYW_ACTIVE = 1, KEYW_MASKED = 4, KEYW_FIRST = 16, KEYW_LAST = 32, KEYW_END = 64 };  // ACTIVE, MASKED << key tile

struct KeyWBars {
  uint64_t full[12], empty[12], drain;
  uint64_t s_full[4], s_free[4];    // [2 * key tile + parity]
  uint64_t l_full[4], l_empty[4];
  KeyWStep step[4];
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(KeyWBars) <= 512, "barrier block too large");

// What every role needs to know of a query tile: rows [n0, n1] of the group's matrix
struct KeyWTile {
  int head;    // head of the first row
  int lo, hi;  // smallest and largest query position + offset among its rows
  bool whole;  // 128 rows
};
__device__ __forceinline__ KeyWTile key_w_tile(int n, int Nq, int rows, int off) {
  const int n0 = n * 128, n1 = min(n0 + 128, rows) - 1;
  const int h0 = n0 / Nq, h1 = n1 < (h0 + 1) * Nq ? h0 : h0 + 1;  // or further on: all that counts is that it differs
  KeyWTile t;
  t.head = h0;
  t.lo = (h0 == h1 ? n0 - h0 * Nq : 0) + off;
  t.hi = (h0 == h1 ? n1 - h0 * Nq : Nq - 1) + off;
  t.whole = n1 - n0 == 127;
  return t;
}

__device__ __forceinline__ float max_nan(float a, float b) {  // a NaN stays one
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
// acc + 2^x of a pair on the FMA pipes: n = rint(x) by the magic add, f = x - n,
// a degree 5 polynomial for 2^f (2.1e-7, like the hardware's) and 2^n put together
// as a float, so that the accumulation's fma does the last product.  x >= -125
// after the clamp; below that the term is below 2^-125 anyway.
__device__ __forceinline__ uint64_t add_exp2_poly5(uint64_t acc, uint64_t x) {
  float x0, x1;
  f2_split(x, x0, x1);
  x = f2(max_nan(x0, -125.f), max_nan(x1, -125.f));
  const uint64_t t = fadd2(x, f2(12582912.f, 12582912.f));
  const uint64_t f = ffma2(fadd2(t, f2(-12582912.f, -12582912.f)), f2(-1.f, -1.f), x);
  uint64_t q = f2(kExp2P5C5, kExp2P5C5);
  q = ffma2(q, f, f2(kExp2P5C4, kExp2P5C4));
  q = ffma2(q, f, f2(kExp2P5C3, kExp2P5C3));
  q = ffma2(q, f, f2(kExp2P5C2, kExp2P5C2));
  q = ffma2(q, f, f2(kExp2P5C1, kExp2P5C1));
  q = ffma2(q, f, f2(kExp2P5C0, kExp2P5C0));
  float t0, t1;
  f2_split(t, t0, t1);
  const uint64_t e = f2(__uint_as_float((__float_as_uint(t0) << 23) + 0x3F800000u),
                        __uint_as_float((__float_as_uint(t1) << 23) + 0x3F800000u));
  return ffma2(q, e, acc);
}
// Which of 8 groups of 4 columns take half their exponentials from the polynomial:
// one (prompt of 4096, 32 heads, d = 128: 109 us; none 113, two 117, four 121).
constexpr unsigned KEYW_POLY = 0x10;

template <int D>
__global__ void __launch_bounds__(KeyWCfg<D>::THREADS, 1)
    key_weights_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ KeyWeightsParams p) {
  using C = KeyWCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  KeyWBars* bars = reinterpret_cast<KeyWBars*>(smem + C::BAR_OFF);
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &bars->abort;
  auto wait = [&](uint64_t& bar, int phase) {  // whole warp
    return __all_sync(0xffffffffu, wait_bar(smem_u32(&bar), (uint32_t)phase & 1u, abort_flag, p.timeout_ns)) != 0;
  };

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NS; ++i) {
      mbar_init(smem_u32(&bars->full[i]), 1);
      mbar_init(smem_u32(&bars->empty[i]), 1);
    }
    mbar_init(smem_u32(&bars->drain), 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&bars->s_full[i]), 1);
      mbar_init(smem_u32(&bars->s_free[i]), 4);
      mbar_init(smem_u32(&bars->l_full[i]), 1);
      mbar_init(smem_u32(&bars->l_empty[i]), 9);  // 8 epilogue warps and the MMA issuer
    }
    bars->abort = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(&bars->tmem_base), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = bars->tmem_base;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join may line up behind this grid

  if (warp == 8) {
    // ================================================================ producer
    if (lane == 0) {
      prefetch_tmap(&tmQ);
      prefetch_tmap(&tmK);
    }
    const int off = p.Nkv - p.Nq, rows = p.group * p.Nq;
    bool ok = true;
    int l = 0;  // steps so far
    // Shared-memory tiles go round, past the two that hold the item's keys.  Bit i
    // of `used` / `phase`: tile i was loaded before / an odd number of times.
    int at = -1, k0 = -1, k1 = -1;
    unsigned used = 0, phase = 0;
    auto load = [&](const CUtensorMap* m, bool three, int c1, int c2) {  // a tile; -1: gave up
      do {
        at = at + 1 == C::NS ? 0 : at + 1;
      } while (at == k0 || at == k1);
      if (((used >> at) & 1) && !wait(bars->empty[at], ((phase >> at) & 1) ^ 1)) return -1;
      if (lane == 0) {
        const uint32_t bar = smem_u32(&bars->full[at]);
        mbar_arrive_expect_tx(bar, C::TILE);
        for (int h = 0; h < D / 64; ++h) {
          if (three)
            tma_load_3d(sbase + at * C::TILE + h * C::HALF, m, bar, h * 64, c1, c2);
          else
            tma_load_2d(sbase + at * C::TILE + h * C::HALF, m, bar, h * 64, c1);
        }
      }
      used |= 1u << at;
      phase ^= 1u << at;
      return at;
    };
    for (int round = 0; round * (int)gridDim.x < p.items && ok; ++round) {
      // the first key tiles see the most queries when causal: they come first,
      // dealt out back and forth
      const int item = round * gridDim.x + ((round & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
      if (item >= p.items) continue;
      const int bhk = item % p.BHkv, rest = item / p.BHkv;
      const int part = rest % p.parts, J = rest / p.parts * 256;
      const int len = p.seqlens ? min(max(p.seqlens[bhk / p.Hkv], 0), p.Nkv) : p.Nkv;
      const float* lse = p.lse + (size_t)bhk * rows;
      // every p.parts-th query tile (so that the parts of a key pair weigh the same),
      // those of which some pair counts, 32 looked at together
      const int q1 = J < len ? p.q_tiles : 0;
      int base = part - 32 * p.parts;
      unsigned todo = 0;
      auto next = [&]() {
        while (todo == 0 && (base += 32 * p.parts) < q1) {
          bool is = false;
          if (base + lane * p.parts < q1) {
            const KeyWTile t = key_w_tile(base + lane * p.parts, p.Nq, rows, off);
            is = t.lo < len && (!p.causal || t.hi >= J);
          }
          todo = __ballot_sync(0xffffffffu, is);
        }
        if (todo == 0) return q1;
        const int n = base + (__ffs(todo) - 1) * p.parts;
        todo &= todo - 1;
        return n;
      };
      float v[4];
      auto fetch = [&](int n) {  // the tile's lse, one tile ahead of its use
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = n * 128 + lane + 32 * e;
          v[e] = n < q1 && row < rows ? lse[row] : 0.f;
        }
      };
      int n = next();
      fetch(n);
      if (n < q1) {
        const int n0 = load(&tmK, true, J, bhk);
        const int n1 = n0 < 0 ? -1 : load(&tmK, true, J + 128, bhk);
        if (!(ok = n1 >= 0)) break;
        k0 = n0, k1 = n1;
      }
      int flags = KEYW_FIRST;
      do {
        const int sl = l % C::NL;
        int lim[4], slot = 0;
        if (n < q1) {
          slot = load(&tmQ, false, bhk * rows + n * 128, 0);
          if (!(ok = slot >= 0)) break;
          const KeyWTile t = key_w_tile(n, p.Nq, rows, off);
#pragma unroll
          for (int kt = 0; kt < 2; ++kt) {
            const int Jk = J + kt * 128;
            if (Jk < len && (!p.causal || t.hi >= Jk)) flags |= KEYW_ACTIVE << kt;
            if (!t.whole || t.hi >= len || (p.causal && t.lo < Jk + 127)) flags |= KEYW_MASKED << kt;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int row = n * 128 + lane + 32 * e;
            int pos = row - t.head * p.Nq;  // at most one head on where a head has 128 rows
            pos = p.Nq < 128 ? pos % p.Nq : pos >= p.Nq ? pos - p.Nq : pos;
            pos += off;
            const bool in = row < rows && pos < len;
            // a row that sees no key has lse = -inf: it gives nothing
            v[e] = !in || v[e] == -INFINITY ? -INFINITY : -v[e] * 1.4426950408889634f;
            lim[e] = !in ? -1 : p.causal ? pos : 0x7fffffff;
          }
        }
        if (!(ok = wait(bars->l_empty[sl], (l / C::NL) ^ 1))) break;
        if (n < q1) {
          float* fv = reinterpret_cast<float*>(smem + C::L_OFF + sl * 1024);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            fv[lane + 32 * e] = v[e];
            reinterpret_cast<int*>(fv)[128 + lane + 32 * e] = lim[e];
          }
          n = next();
          fetch(n);
        }
        if (n == q1) flags |= KEYW_LAST;
        if (lane == 0) bars->step[sl] = KeyWStep{flags, slot | k0 << 8 | k1 << 16, J, bhk, part};
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->l_full[sl]));
        ++l;
        flags = 0;
      } while (n < q1);
    }
    if (ok && wait(bars->l_empty[l % C::NL], (l / C::NL) ^ 1) && lane == 0) {
      bars->step[l % C::NL] = KeyWStep{KEYW_END, 0, 0, 0, 0};
      mbar_arrive(smem_u32(&bars->l_full[l % C::NL]));
    }
    // never leave a copy in flight (after a normal run these have all completed)
    if (lane == 0)
      for (int i = 0; i < C::NS; ++i)
        if ((used >> i) & 1) wait_bar_drain(smem_u32(&bars->full[i]), ((phase >> i) & 1) ^ 1, p.timeout_ns);
    __syncwarp();
  } else if (warp == 9) {
    // ================================================================ MMA issuer
    if (lane == 0) {
      bool ok = true;
      int c[2] = {0, 0};   // products of each key tile so far
      unsigned phase = 0;  // bit i: tile i was waited for an odd number of times
      auto need = [&](uint64_t& bar, int ph) {
        return spin_bar(smem_u32(&bar), (uint32_t)ph & 1u, abort_flag, p.timeout_ns);
      };
      auto tile = [&](int i) {
        const bool r = need(bars->full[i], (phase >> i) & 1);
        phase ^= 1u << i;
        return r;
      };
      bool keys = false;  // whether the item has any product
      for (int l = 0;; ++l) {
        const int sl = l % C::NL;
        if (!(ok = need(bars->l_full[sl], l / C::NL))) break;
        const int flags = bars->step[sl].flags, slots = bars->step[sl].slots;
        mbar_arrive(smem_u32(&bars->l_empty[sl]));
        if (flags & KEYW_END) break;
        if (flags & KEYW_FIRST) keys = false;
        const int st = slots & 255;
        const int ks[2] = {(slots >> 8) & 255, (slots >> 16) & 255};
        if (flags & (3 * KEYW_ACTIVE)) {
          if (!keys && !(ok = tile(ks[0]) && tile(ks[1]))) break;
          keys = true;
          if (!(ok = tile(st))) break;
          const uint64_t dQ = smem_desc(sbase + st * C::TILE, 16, 1024);
          for (int kt = 0; kt < 2 && ok; ++kt) {
            if (!(flags & (KEYW_ACTIVE << kt))) continue;
            const int buf = 2 * kt + (c[kt] & 1);
            if (!(ok = need(bars->s_free[buf], (c[kt] >> 1) ^ 1))) break;
            tc_fence_after();
            const uint64_t dK = smem_desc(sbase + ks[kt] * C::TILE, 16, 1024);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint64_t o = (uint64_t)(((kk >> 2) * C::HALF + (kk & 3) * 32) >> 4);
              mma_f16_ss(tbase + buf * 128, dK + o, dQ + o, C::ID, kk > 0);
            }
            tc_commit(smem_u32(&bars->s_full[buf]));
            ++c[kt];
          }
          if (!ok) break;
          tc_commit(smem_u32(&bars->empty[st]));
        }
        if ((flags & KEYW_LAST) && keys) {
          tc_commit(smem_u32(&bars->empty[ks[0]]));
          tc_commit(smem_u32(&bars->empty[ks[1]]));
        }
      }
      if (!ok) {  // every MMA issued so far must finish before TMEM is freed
        tc_commit(smem_u32(&bars->drain));
        wait_bar_drain(smem_u32(&bars->drain), 0, p.timeout_ns);
      }
    }
    __syncwarp();
  } else {
    // ================================================================ epilogue
    const int kt = warp >> 2, row = threadIdx.x & 127;
    const uint64_t sc = f2(p.sl2, p.sl2);
    int c = 0;                  // products of the key tile so far
    float w = 0.f, comp = 0.f;  // this thread's sum and its compensation
    for (int l = 0;; ++l) {
      const int sl = l % C::NL;
      if (!wait(bars->l_full[sl], l / C::NL)) break;
      const KeyWStep step = bars->step[sl];
      if (step.flags & KEYW_END) break;
      const int j = step.J + kt * 128 + row;
      if (step.flags & (KEYW_ACTIVE << kt)) {
        const int buf = 2 * kt + (c & 1);
        if (!wait(bars->s_full[buf], c >> 1)) break;
        ++c;
        tc_fence_after();
        const uint32_t tS = tbase + buf * 128 + ((uint32_t)((warp & 3) * 32) << 16);
        uint32_t x[4][32];
#pragma unroll
        for (int k = 0; k < 4; ++k) tmem_ld32(tS + k * 32, x[k]);
#pragma unroll
        for (int k = 0; k < 4; ++k) tmem_ld_wait(x[k]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->s_free[buf]));
        const float* fv = reinterpret_cast<const float*>(smem + C::L_OFF + sl * 1024);
        const int* lim = reinterpret_cast<const int*>(fv) + 128;
        // partial sums of 32 terms each; the tile's sum joins the running one with
        // compensation: over thousands of queries plain fp32 sums drift by 1e-6
        uint64_t a0 = f2(0.f, 0.f), a1 = a0;
        auto columns = [&](auto mask) {
#pragma unroll
          for (int i = 0; i < 128; i += 4) {
            const float4 v = *reinterpret_cast<const float4*>(fv + i);
            const uint32_t* xi = &x[i >> 5][i & 31];
            const uint64_t y0 = ffma2(f2(__uint_as_float(xi[0]), __uint_as_float(xi[1])), sc, f2(v.x, v.y));
            const uint64_t y1 = ffma2(f2(__uint_as_float(xi[2]), __uint_as_float(xi[3])), sc, f2(v.z, v.w));
            float e0, e1, e2, e3;
            f2_split(y0, e0, e1);
            f2_split(y1, e2, e3);
            e0 = ex2(e0), e1 = ex2(e1);
            if (decltype(mask)::value || !((KEYW_POLY >> (i / 4 % 8)) & 1)) {
              e2 = ex2(e2), e3 = ex2(e3);
              if (decltype(mask)::value) {
                const int4 m = *reinterpret_cast<const int4*>(lim + i);
                e0 = j <= m.x ? e0 : 0.f, e1 = j <= m.y ? e1 : 0.f, e2 = j <= m.z ? e2 : 0.f, e3 = j <= m.w ? e3 : 0.f;
              }
              a1 = fadd2(a1, f2(e2, e3));
            } else {
              a1 = add_exp2_poly5(a1, y1);
            }
            a0 = fadd2(a0, f2(e0, e1));
          }
        };
        if (step.flags & (KEYW_MASKED << kt))
          columns(std::true_type{});
        else
          columns(std::false_type{});
        float b0, b1;
        f2_split(fadd2(a0, a1), b0, b1);
        const float y = (b0 + b1) - comp, z = w + y;
        comp = (z - w) - y;
        w = z;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->l_empty[sl]));
      if (!(step.flags & KEYW_LAST)) continue;
      if (j < p.Nkv) {
        const int len = p.seqlens ? p.seqlens[step.bhk / p.Hkv] : p.Nkv;
        if (j >= len) w = 0.f;
        if (p.parts > 1) {
          p.parts_out[((size_t)step.part * p.BHkv + step.bhk) * p.Nkv + j] = w;
        } else {
          float* out = p.w + step.bhk * p.stride + j;
          *out = p.accumulate ? *out + w : w;
        }
      }
      w = comp = 0.f;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// joins the parts, always in the same order
__global__ void __launch_bounds__(256) key_weights_join_kernel(const KeyWeightsParams p, int columns) {
  const int bhk = blockIdx.x / columns, j = blockIdx.x % columns * 256 + threadIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (j >= p.Nkv) return;
  float w = 0.f;
#pragma unroll 8
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
