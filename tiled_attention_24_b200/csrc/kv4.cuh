// The 4-bit key/value cache: row format, append (quantise and write), read
// back, eviction.
//
// A row (one token of one cache head, D channels) is D/2 bytes of signed 4-bit
// codes and NG = D/32 bf16 scales, one per group of 32 consecutive channels:
//
//   s = bf16(amax / 7)          (IEEE fp32 divide, both roundings to nearest even)
//   c = clamp(rne(x / s), -7, 7), value = c * s      (s = 0: every c = 0)
//   a group holding an infinity or a NaN: s = NaN, c = 0 (the row reads as NaN)
//
// Any rounding of s only moves the grid: the codes are taken against the
// rounded scale, so bf16 (the range of the inputs, 2 bytes per 32 channels)
// costs no accuracy beyond a grid at most 2^-8 coarser.
//
// Byte u * 2 NG + 2 g + h (u < 8, g < NG, h < 2) of a row holds channel
// 32 g + 4 u + 2 h (low nibble) and the next one (high nibble): piece u, 2 NG
// bytes, has four channels of EVERY group.  The decode kernel's matrix
// instructions need each lane to hold the same groups in the same registers;
// in channel order one lane's 16 bytes would be one whole group.
#pragma once
#include <cooperative_groups.h>

#include "ptx.cuh"

namespace ta {

constexpr int KV4_GROUP = 32;

// NG x 2 bytes (one piece of a row, or a row's scales) as one access
template <int NG>
struct Kv4Piece;
template <>
struct Kv4Piece<4> {
  using T = uint2;
};
template <>
struct Kv4Piece<2> {
  using T = uint32_t;
};
__device__ __forceinline__ uint32_t kv4_half(const uint2& w, int g) {
  const uint32_t v = (g & 2) ? w.y : w.x;
  return (g & 1) ? (v >> 16) : (v & 0xFFFFu);
}
__device__ __forceinline__ uint32_t kv4_half(const uint32_t& w, int g) { return (g & 1) ? (w >> 16) : (w & 0xFFFFu); }
// code i (0..3) of a halfword of four
__device__ __forceinline__ float kv4_code(uint32_t h, int i) { return (float)((int)(h << (28 - 4 * i)) >> 28); }
__device__ __forceinline__ float kv4_scale(uint32_t bits) { return __uint_as_float(bits << 16); }

// ------------------------------------------------------------------ append --
struct Kv4AppendParams {
  const uint16_t *k, *v;      // [B][Hkv][n][D] bf16
  uint8_t *kc, *vc;           // [B][Hkv][cap][D/2]
  uint16_t *ks, *vs;          // [B][Hkv][cap][D/32] bf16
  const int *starts, *counts; // [B]; counts may be null (n each)
  float* weights;             // [B][Hkv][cap] or null
  int* positions;             // [B][Hkv][cap] or null
  const int* next_pos;        // [B], with positions
  int Hkv, n, cap;
  unsigned rows;              // B * Hkv * n
};

// One K and one V row by the 8 lanes of their pieces (lane u: channels 4u..4u+3 of
// each of the 2 NG groups).  What a group needs once is done once: amax by a
// butterfly that halves the groups a lane holds at each step, on pairs of bf16 (a NaN
// wins; the sign of a maximum means nothing); the scale and its reciprocal by one lane
// (two where d = 64), which hands the reciprocal round.
//
// The codes need rne(x / s) exactly, without a divide per element: with
// r = rn(1/s), t = fma(x, r, 6144) is 6144 + x r rounded to a multiple of 2^-11.
// x and s have 8 significant bits, so a quotient of magnitude <= 7.6 is either
// exactly k + 1/2 or at least 2^-2 / 255 > 9e-4 away from it, and x r is within
// 5e-7 of the quotient: rounded to 2^-11 (at most 2.5e-4 away) the ties are
// ties again and nothing else is one.  t - 6144 + 8 + 1.5 * 2^23, one addition, then
// rounds to even and leaves c + 8 in the low bits of the number.  |x / s| <= 7 (1 +
// 2^-8), so c + 8 is 1 to 15: four make a halfword by shifts and sums, a nibble each,
// with the sign bits flipped.  Groups with an infinity or a NaN, and scales below
// 2^-100, where 1/s may overflow or s has lost bits, are redone with the divide.
//
// 4 x 16 heads x 4096 tokens, d = 128 (173 MB, 27 us at the copy bandwidth): 31 us.
// Maxima on unpacked halves and sums of c_i 16^i as floats took 36, a divide per group
// and lane with integer packing 53: the ALU pipe bounded both.
__device__ __forceinline__ uint32_t kv4_halfword(uint32_t lo, uint32_t hi, float r) {  // the bits above are not 0
  const uint64_t rr = f2(r, r), six = f2(6144.f, 6144.f), big = f2(12576776.f, 12576776.f);
  const uint64_t a = fadd2(ffma2(f2(__uint_as_float(lo << 16), __uint_as_float(lo & 0xFFFF0000u)), rr, six), big);
  const uint64_t b = fadd2(ffma2(f2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xFFFF0000u)), rr, six), big);
  float c0, c1, c2, c3;
  f2_split(a, c0, c1);
  f2_split(b, c2, c3);
  return __float_as_uint(c0) + (__float_as_uint(c1) << 4) + ((__float_as_uint(c2) + (__float_as_uint(c3) << 4)) << 8);
}
constexpr uint32_t KV4_FLIP = 0x88888888u;
__device__ __forceinline__ uint2 kv4_join_flipped(const uint32_t (&h)[4]) {
  return make_uint2(__byte_perm(h[0], h[1], 0x5410) ^ KV4_FLIP, __byte_perm(h[2], h[3], 0x5410) ^ KV4_FLIP);
}
__device__ __forceinline__ uint32_t kv4_join_flipped(const uint32_t (&h)[2]) {
  return __byte_perm(h[0], h[1], 0x5410) ^ KV4_FLIP;
}
// per half: the larger magnitude, NaN if either is; the sign may be either's
__device__ __forceinline__ uint32_t kv4_amax2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __noinline__ uint32_t kv4_halfword_slow(uint32_t lo, uint32_t hi, uint32_t scale_bits) {
  const float s = kv4_scale(scale_bits);
  const float x[4] = {__uint_as_float(lo << 16), __uint_as_float(lo & 0xFFFF0000u), __uint_as_float(hi << 16),
                      __uint_as_float(hi & 0xFFFF0000u)};
  uint32_t h = 0;
  if (s > 0.f)  // neither zero nor NaN
    for (int i = 0; i < 4; ++i) h |= ((uint32_t)max(-7, min(7, __float2int_rn(__fdiv_rn(x[i], s)))) & 15u) << (4 * i);
  return h;
}

template <int NG>
__global__ void __launch_bounds__(256) kv4_append_kernel(const Kv4AppendParams p) {
  constexpr int D = 32 * NG;
  using T = typename Kv4Piece<NG>::T;
  const unsigned row = blockIdx.x * 32u + (threadIdx.x >> 3);
  const int u = threadIdx.x & 7;
  const bool in = row < p.rows;
  const unsigned bh = (in ? row : 0u) / (unsigned)p.n;
  const int i = (int)((in ? row : 0u) - bh * (unsigned)p.n);
  const int b = (int)(bh / (unsigned)p.Hkv);
  uint2 w[2 * NG];  // K groups, V groups; loaded before the slot is known to be live
#pragma unroll
  for (int g = 0; g < 2 * NG; ++g) {
    const uint16_t* x = (g < NG ? p.k : p.v) + (size_t)row * D + 32 * (g % NG) + 4 * u;
    w[g] = in ? *reinterpret_cast<const uint2*>(x) : make_uint2(0, 0);
  }
  const int count = p.counts ? p.counts[b] : p.n;
  const long long slot = (long long)p.starts[b] + i;
  const bool live = in && i < count && slot >= 0 && slot < p.cap;

  uint32_t m[NG];  // amax of groups 2i (low half) and 2i + 1
#pragma unroll
  for (int g = 0; g < 2 * NG; g += 2) {
    const uint32_t a = kv4_amax2(w[g].x, w[g].y), c = kv4_amax2(w[g + 1].x, w[g + 1].y);
    m[g / 2] = kv4_amax2(__byte_perm(a, c, 0x5410), __byte_perm(a, c, 0x7632));
  }
  // halve the pairs held at each step; then lane u has pair `pair`, groups 2 pair, 2 pair + 1
  int pair = 0, bit = 4;
  if (NG == 4) {
    const bool up = u & 4;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t give = up ? m[e] : m[(e + 2) % NG], keep = up ? m[(e + 2) % NG] : m[e];
      m[e] = kv4_amax2(keep, __shfl_xor_sync(0xffffffffu, give, 4));
    }
    pair = up ? 2 : 0;
    bit = 2;
  }
  {
    const bool up = u & bit;
    const uint32_t give = up ? m[0] : m[1], keep = up ? m[1] : m[0];
    m[0] = kv4_amax2(keep, __shfl_xor_sync(0xffffffffu, give, bit));
    pair += up ? 1 : 0;
  }
#pragma unroll
  for (int o = NG == 4 ? 1 : 2; o > 0; o >>= 1) m[0] = kv4_amax2(m[0], __shfl_xor_sync(0xffffffffu, m[0], o));
  const int mine = 2 * pair + (u & 1);  // this lane's group
  const uint32_t top = ((u & 1) ? m[0] >> 16 : m[0]) & 0x7FFFu;
  uint32_t bits = pack_bf16(__fdiv_rn(__uint_as_float(top << 16), 7.f), 0.f) & 0xFFFFu;
  if (top >= 0x7F80u) bits = 0x7FC0u;
  const float s = kv4_scale(bits);
  const bool odd = !(s == 0.f || s >= 0x1p-100f);
  const float r = s == 0.f ? 0.f : __frcp_rn(s);

  uint32_t h[2 * NG];
  const int base = (threadIdx.x & 24);
#pragma unroll
  for (int g = 0; g < 2 * NG; ++g) {
    // the lane of the row that holds group g
    const int from = NG == 4 ? ((g & 4) ? 4 : 0) | ((g & 2) ? 2 : 0) | (g & 1) : ((g & 2) ? 4 : 0) | (g & 1);
    h[g] = kv4_halfword(w[g].x, w[g].y, __shfl_sync(0xffffffffu, r, base + from));
  }
  if (__any_sync(0xffffffffu, odd)) {
#pragma unroll
    for (int g = 0; g < 2 * NG; ++g) {
      const int from = NG == 4 ? ((g & 4) ? 4 : 0) | ((g & 2) ? 2 : 0) | (g & 1) : ((g & 2) ? 4 : 0) | (g & 1);
      const uint32_t sb = __shfl_sync(0xffffffffu, bits, base + from);
      if (__shfl_sync(0xffffffffu, (int)odd, base + from)) h[g] = kv4_halfword_slow(w[g].x, w[g].y, sb) ^ (KV4_FLIP & 0xFFFFu);
    }
  }
  if (!live) return;
  const size_t dst = (size_t)bh * p.cap + slot;
  uint32_t hk[NG], hv[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) hk[g] = h[g], hv[g] = h[NG + g];
  reinterpret_cast<T*>(p.kc + dst * (D / 2))[u] = kv4_join_flipped(hk);
  reinterpret_cast<T*>(p.vc + dst * (D / 2))[u] = kv4_join_flipped(hv);
  // every group's scale by the lane that made it (d = 64: by the first of the two)
  if (NG == 4 || !(u & 2)) (mine < NG ? p.ks : p.vs)[dst * NG + mine % NG] = (uint16_t)bits;
  if (u == 2 && p.weights) p.weights[dst] = 0.f;
  if (u == 3 && p.positions) p.positions[dst] = p.next_pos[b] + i;
}

// -------------------------------------------------------------------- read --
template <int NG>
__global__ void __launch_bounds__(256)
    kv4_read_kernel(const uint8_t* __restrict__ codes, const uint16_t* __restrict__ scales, uint16_t* __restrict__ out,
                    const int* __restrict__ starts, int Hkv, int n, int cap, unsigned rows) {
  constexpr int D = 32 * NG;
  using T = typename Kv4Piece<NG>::T;
  const unsigned row = blockIdx.x * 32u + (threadIdx.x >> 3);
  const int u = threadIdx.x & 7;
  if (row >= rows) return;
  const unsigned bh = row / (unsigned)n;
  const int i = (int)(row - bh * (unsigned)n);
  const long long slot = (long long)(starts ? starts[bh / (unsigned)Hkv] : 0) + i;
  const bool live = slot >= 0 && slot < cap;
  T c{}, s{};
  if (live) {
    const size_t src = (size_t)bh * cap + slot;
    c = reinterpret_cast<const T*>(codes + src * (D / 2))[u];
    s = *reinterpret_cast<const T*>(scales + src * NG);
  }
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const uint32_t h = kv4_half(c, g);
    const float f = kv4_scale(kv4_half(s, g));
    *reinterpret_cast<uint2*>(out + (size_t)row * D + 32 * g + 4 * u) =
        make_uint2(pack_bf16(kv4_code(h, 0) * f, kv4_code(h, 1) * f), pack_bf16(kv4_code(h, 2) * f, kv4_code(h, 3) * f));
  }
}

// ---------------------------------------------------------------- eviction --
struct Kv4EvictParams {
  uint8_t *kc, *vc;
  uint16_t *ks, *vs;
  const float* weights;      // [B][Hkv][cap]
  const int* positions;      // [B][Hkv][cap]
  const int *seqlens, *next_pos;  // [B]
  float* weights_out;        // may be weights
  int* positions_out;        // may be positions
  int* kept;                 // [B][Hkv][n_keep]
  int* lists;                // workspace: per (batch, head) n_keep holes, n_keep sources
  int Hkv, cap, n_keep, n_recent;
};

// Rank of a slot as an unsigned key: the newest slots on top, above +infinity (whose
// key is 0xFF800000), then by weight (-0 equals +0, a NaN ranks with -infinity).
__device__ __forceinline__ uint32_t kv4_rank_key(float w, int pos, long long first_recent) {
  if (pos >= first_recent) return 0xFFFFFFFFu;
  if (w != w) w = -INFINITY;
  const uint32_t b = __float_as_uint(w + 0.f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// The whole eviction of one (batch, cache head) by one cluster of up to 8 CTAs,
// each with a contiguous slice of the slots, keys kept in shared memory:
//   1. the n_keep-th largest key, 11 + 11 + 10 bits at a time: histograms per CTA,
//      which every CTA adds up, so that each finds the digit;
//   2. keys above it stay, and as many equal ones as are wanted, lowest slots first
//      (ranks by ballots, prefix sums over warps and CTAs);
//   3. the lists of holes (below n_keep, not kept) and sources (kept, at or beyond
//      n_keep), both in slot order, and the r-th source moves into the r-th hole.
// Rows move from slots >= n_keep into slots < n_keep only, so no row is read after
// it was overwritten and a repeated call moves the same rows again.
// 16 sequences of up to 32768 slots to 16384, 8 cache heads, d = 128 (138 MB, 21 us at
// the copy bandwidth): 60 us.  About 25 are a chain of barriers over a few slots a
// thread (load 5, each digit 3, places 2, lists 3), 25 the moves: rows of 64 + 8 + 8
// bytes picked out of sectors of 32 and written back.  Two CTAs of
// 512 threads on an SM: 3 spill (68 us), clusters of 2 or 8 leave SMs idle or wait for
// room (92, 97); two rows a lane in flight gain nothing (60).
constexpr int KV4_EVICT_THREADS = 512, KV4_EVICT_WARPS = KV4_EVICT_THREADS / 32;
constexpr int KV4_EVICT_CACHED = 16384;  // keys a CTA keeps; longer slices are ranked from memory each time
constexpr int KV4_EVICT_BINS = 2048;

struct Kv4EvictShared {
  int hist[2][KV4_EVICT_BINS];  // this CTA's, of one pass and the next; then the words' first list entries
  int2 warp[2][KV4_EVICT_WARPS];
  int2 cta[2][8];             // per CTA: equal keys; holes and sources
  uint32_t prefix;
  int need, ties;  // of the keys that match the prefix: to be kept, in all
};

template <int NG, bool CACHED>
__global__ void __launch_bounds__(KV4_EVICT_THREADS, 2) kv4_evict_kernel(const Kv4EvictParams p) {
  namespace cg = cooperative_groups;
  constexpr int D = 32 * NG;
  using T = typename Kv4Piece<NG>::T;
  extern __shared__ __align__(16) uint8_t smem[];
  Kv4EvictShared& sh = *reinterpret_cast<Kv4EvictShared*>(smem);
  uint32_t* keep_bits = reinterpret_cast<uint32_t*>(smem + sizeof(Kv4EvictShared));  // one bit a slot of the slice
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), CL = (int)cluster.num_blocks();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bh = blockIdx.x / CL, b = bh / p.Hkv;
  const int L = min(max(p.seqlens[b], 0), p.cap);
  int* kept = p.kept + (size_t)bh * p.n_keep;
  const size_t row0 = (size_t)bh * p.cap;
  const float* w = p.weights + row0;
  const int* pos = p.positions + row0;
  float* w_out = p.weights_out + row0;
  int* pos_out = p.positions_out + row0;
  if (L <= p.n_keep) {  // nothing to evict
    const int step = CL * KV4_EVICT_THREADS;
    for (int j0 = rank * KV4_EVICT_THREADS + tid; j0 < p.n_keep; j0 += 8 * step) {  // 8 slots a thread in flight
      float a[8];
      int c[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int j = j0 + k * step;
        a[k] = j < L ? w[j] : 0.f;
        c[k] = j < L ? pos[j] : 0;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int j = j0 + k * step;
        if (j < p.n_keep) kept[j] = j < L ? j : -1;
        if (j < L) w_out[j] = a[k], pos_out[j] = c[k];
      }
    }
    return;
  }
  const long long first_recent = (long long)p.next_pos[b] - p.n_recent;
  // this CTA's slots [j0, j0 + n), a warp's a contiguous run of them
  const int slice = ((L + CL - 1) / CL + KV4_EVICT_THREADS - 1) / KV4_EVICT_THREADS * KV4_EVICT_THREADS;
  const int j0 = min(rank * slice, L), n = min(slice, L - j0);
  uint32_t* keys = keep_bits + slice / 32;
  auto key_at = [&](int i) -> uint32_t {
    return CACHED ? keys[i] : kv4_rank_key(w[j0 + i], pos[j0 + i], first_recent);
  };
  // Slots below n_keep that stay keep their places; copied before it is known which
  // stay, since every other of them is a hole that a row is moved into later
  const int front = min(n, p.n_keep - j0);
  const bool copy = w_out != w || pos_out != pos;
  if (CACHED) {  // 8 slots a thread in flight
    for (int i = tid; i < n; i += 8 * KV4_EVICT_THREADS) {
      float a[8];
      int c[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int at = i + k * KV4_EVICT_THREADS;
        a[k] = at < n ? w[j0 + at] : 0.f;
        c[k] = at < n ? pos[j0 + at] : 0;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int at = i + k * KV4_EVICT_THREADS;
        if (at < n) keys[at] = kv4_rank_key(a[k], c[k], first_recent);
        if (copy && at < front) w_out[j0 + at] = a[k], pos_out[j0 + at] = c[k];
      }
    }
  }
  for (int i = tid; i < KV4_EVICT_BINS; i += KV4_EVICT_THREADS) sh.hist[0][i] = sh.hist[1][i] = 0;
  cluster.sync();

  // ---- 1. the threshold
  uint32_t prefix = 0, mask = 0;
  int need = p.n_keep;  // how many of the keys that match the prefix are kept
  for (int d = 0; d < 3; ++d) {
    const int shift = d == 0 ? 21 : d == 1 ? 10 : 0;
    const uint32_t digits = d == 2 ? 1023u : 2047u;
    int* hist = sh.hist[d & 1];
#pragma unroll 4
    for (int i = tid; i < n; i += KV4_EVICT_THREADS) {
      const uint32_t key = key_at(i);
      if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & digits], 1);
    }
    cluster.sync();
    if (d == 1)  // read by all before this pass's barrier, filled again in the next pass
      for (int i = tid; i < KV4_EVICT_BINS; i += KV4_EVICT_THREADS) sh.hist[0][i] = 0;
    // bins from the top, four to a thread: the one in which the need-th key lies
    constexpr int PER = 4;
    static_assert(PER * KV4_EVICT_THREADS == KV4_EVICT_BINS, "four bins a thread");
    const int top = KV4_EVICT_BINS - PER * (tid + 1);
    int c[PER] = {0, 0, 0, 0};
#pragma unroll 4
    for (int r = 0; r < CL; ++r) {
      const int4 v = *reinterpret_cast<const int4*>(cluster.map_shared_rank(hist, r) + top);
      c[0] += v.w, c[1] += v.z, c[2] += v.y, c[3] += v.x;
    }
    const int sum = c[0] + c[1] + c[2] + c[3];
    int before = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += v;
    }
    if (lane == 31) sh.warp[0][warp].x = before;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < KV4_EVICT_WARPS; ++k) {
      const int v = sh.warp[0][k].x;
      if (k < warp) before += v;
    }
    before -= sum;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      if (before < need && need <= before + c[k]) {
        sh.prefix = prefix | ((uint32_t)(top + PER - 1 - k) << shift);
        sh.need = need - before;
        sh.ties = c[k];
      }
      before += c[k];
    }
    __syncthreads();
    prefix = sh.prefix;
    need = sh.need;
    mask |= digits << shift;
    if (sh.ties == need) break;  // all keys of this digit stay, whatever their lower ones: no key is below the prefix
  }

  // ---- 2. who stays: a bit for each slot
  const int run = slice / KV4_EVICT_WARPS, i0 = warp * run, i1 = min(i0 + run, n);
  // exclusive sums over lower threads and CTAs of two per-thread counts; the cluster's totals
  auto before_me = [&](int2 c, int which, int2& total) {
    int2 up = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, up.x, o), y = __shfl_up_sync(0xffffffffu, up.y, o);
      if (lane >= o) up.x += x, up.y += y;
    }
    if (lane == 31) sh.warp[which][warp] = up;
    __syncthreads();
    int2 before = make_int2(up.x - c.x, up.y - c.y), mine = make_int2(0, 0);
#pragma unroll
    for (int k = 0; k < KV4_EVICT_WARPS; ++k) {
      const int2 v = sh.warp[which][k];
      if (k < warp) before.x += v.x, before.y += v.y;
      mine.x += v.x, mine.y += v.y;
    }
    if (tid < CL) cluster.map_shared_rank(&sh.cta[which][0], tid)[rank] = mine;
    cluster.sync();
    total = make_int2(0, 0);
    for (int r = 0; r < CL; ++r) {
      const int2 v = sh.cta[which][r];
      if (r < rank) before.x += v.x, before.y += v.y;
      total.x += v.x, total.y += v.y;
    }
    return before;
  };
  int2 all;
  if (sh.ties > need) {  // some of the equal keys go: which, by their order
    int count = 0;
    for (int i = i0; i < i1; i += 32)
      count += __popc(__ballot_sync(0xffffffffu, i + lane < i1 && key_at(i + lane) == prefix));
    int eq = __shfl_sync(0xffffffffu, before_me(make_int2(lane == 0 ? count : 0, 0), 0, all).x, 0);
    for (int i = i0; i < i1; i += 32) {
      const bool in = i + lane < i1;
      const uint32_t key = in ? key_at(i + lane) : 0u;
      const unsigned same = __ballot_sync(0xffffffffu, in && key == prefix);
      const bool stays = in && (key > prefix || (key == prefix && eq + __popc(same & ((1u << lane) - 1u)) < need));
      const unsigned keep = __ballot_sync(0xffffffffu, stays);
      eq += __popc(same);
      if (lane == 0) keep_bits[i / 32] = keep;
    }
  } else {
#pragma unroll 4
    for (int i = i0; i < i1; i += 32) {
      const unsigned keep = __ballot_sync(0xffffffffu, i + lane < i1 && key_at(i + lane) >= prefix);
      if (lane == 0) keep_bits[i / 32] = keep;
    }
  }
  __syncthreads();

  // ---- 3. the lists, then the rows.  A thread has `words` words of 32 slots
  int* hole_list = p.lists + (size_t)bh * 2 * p.n_keep;
  int* source_list = hole_list + p.n_keep;
  const int words = (slice / 32 + KV4_EVICT_THREADS - 1) / KV4_EVICT_THREADS, w0 = tid * words;
  auto low = [](int k) { return k <= 0 ? 0u : k >= 32 ? 0xffffffffu : (1u << k) - 1u; };  // bits [0, k)
  auto hole_bits = [&](int k) { return 32 * k < n ? ~keep_bits[k] & low(n - 32 * k) & low(p.n_keep - j0 - 32 * k) : 0u; };
  auto source_bits = [&](int k) { return 32 * k < n ? keep_bits[k] & ~low(p.n_keep - j0 - 32 * k) : 0u; };
  int2 count = make_int2(0, 0);
  for (int k = w0; k < w0 + words; ++k) count.x += __popc(hole_bits(k)), count.y += __popc(source_bits(k));
  int2 at = before_me(count, 1, all);
  const int moves = all.x;
  if constexpr (CACHED) {  // a warp per word.  No source lies before the word in which n_keep falls
    static_assert(KV4_EVICT_CACHED <= 32 * KV4_EVICT_THREADS, "a word a thread");
    int* first = sh.hist[0];
    if (tid < slice / 32) first[tid] = j0 + 32 * tid < p.n_keep ? at.x : at.y;
    __syncthreads();
    const unsigned below = (1u << lane) - 1u;
#pragma unroll 4
    for (int k = warp; k < slice / 32; k += KV4_EVICT_WARPS) {
      const unsigned holes = hole_bits(k), sources = source_bits(k);
      const int slot = j0 + 32 * k + lane;
      if (32 * k + lane < front && ((keep_bits[k] >> lane) & 1u)) kept[slot] = slot;
      if ((holes >> lane) & 1u) hole_list[first[k] + __popc(holes & below)] = slot;
      if ((sources >> lane) & 1u)
        source_list[(j0 + 32 * k < p.n_keep ? 0 : first[k]) + __popc(sources & below)] = slot;
    }
  } else {
    for (int k = w0; k < w0 + words; ++k) {
      for (unsigned m = hole_bits(k); m; m &= m - 1) hole_list[at.x++] = j0 + 32 * k + __ffs(m) - 1;
      for (unsigned m = source_bits(k); m; m &= m - 1) source_list[at.y++] = j0 + 32 * k + __ffs(m) - 1;
    }
    for (int i = tid; i < front; i += KV4_EVICT_THREADS)
      if ((keep_bits[i / 32] >> lane) & 1u) {
        const int slot = j0 + i;
        kept[slot] = slot;
        if (copy) w_out[slot] = w[slot], pos_out[slot] = pos[slot];
      }
  }
  cluster.sync();  // the lists are complete, and nobody reads weights or positions below n_keep any more
  constexpr int LANES = D / 32, ROWS = 32 / LANES, DEEP = 1;  // 16 bytes of codes a lane
  const int sub = lane % LANES;
  int to[DEEP], from[DEEP];
  auto pairs = [&](int m0) {
#pragma unroll
    for (int k = 0; k < DEEP; ++k) {
      const int m = m0 + k * ROWS + lane / LANES;
      to[k] = m < moves ? __ldcg(hole_list + m) : -1;
      from[k] = m < moves ? __ldcg(source_list + m) : 0;
    }
  };
  const int step = CL * KV4_EVICT_WARPS * ROWS * DEEP;
  int m0 = (rank * KV4_EVICT_WARPS + warp) * ROWS * DEEP;
  pairs(m0);
  for (; m0 < moves; m0 += step) {
    uint4 kc[DEEP], vc[DEEP];
    T sc[DEEP];
    uint32_t side[DEEP];
#pragma unroll
    for (int k = 0; k < DEEP; ++k)
      if (to[k] >= 0) {
        const size_t src = row0 + from[k];
        kc[k] = reinterpret_cast<const uint4*>(p.kc + src * (D / 2))[sub];
        vc[k] = reinterpret_cast<const uint4*>(p.vc + src * (D / 2))[sub];
        if (sub < 2) {
          sc[k] = *reinterpret_cast<const T*>((sub ? p.vs : p.ks) + src * NG);
          side[k] = sub ? (uint32_t)pos[from[k]] : __float_as_uint(w[from[k]]);
        }
      }
    int dsts[DEEP], srcs[DEEP];
#pragma unroll
    for (int k = 0; k < DEEP; ++k) dsts[k] = to[k], srcs[k] = from[k];
    pairs(m0 + step);  // the next rows' places, while these rows are on their way
#pragma unroll
    for (int k = 0; k < DEEP; ++k)
      if (dsts[k] >= 0) {
        const size_t dst = row0 + dsts[k];
        reinterpret_cast<uint4*>(p.kc + dst * (D / 2))[sub] = kc[k];
        reinterpret_cast<uint4*>(p.vc + dst * (D / 2))[sub] = vc[k];
        if (sub < 2) {
          *reinterpret_cast<T*>((sub ? p.vs : p.ks) + dst * NG) = sc[k];
          if (sub)
            pos_out[dsts[k]] = (int)side[k];
          else
            w_out[dsts[k]] = __uint_as_float(side[k]), kept[dsts[k]] = srcs[k];
        }
      }
  }
}

}  // namespace ta
