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
__device__ __forceinline__ uint2 kv4_join(const uint32_t (&h)[4]) {
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}
__device__ __forceinline__ uint32_t kv4_join(const uint32_t (&h)[2]) { return h[0] | (h[1] << 16); }
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

// One row by the 8 lanes of its pieces (lane u: channels 4u..4u+3 of each
// group).  amax is taken on the bf16 bit patterns (ordered like the values,
// infinities and NaNs on top).
//
// The codes need rne(x / s) exactly, without a divide per element: with
// r = rn(1/s), fma(x, r, 6144) - 6144 is x r rounded to a multiple of 2^-11.
// x and s have 8 significant bits, so a quotient of magnitude <= 7.6 is either
// exactly k + 1/2 or at least 2^-2 / 255 > 9e-4 away from it, and x r is within
// 5e-7 of the quotient: rounded to 2^-11 (at most 2.5e-4 away) the ties are
// ties again and nothing else is one.  Adding 1.5 * 2^23 then rounds to even
// and leaves the code in the low nibble.  |x / s| <= 7 (1 + 2^-8), so no code
// exceeds 7.  Scales below 2^-100, where 1/s may overflow or s has lost bits,
// take the divide and the clamp.
template <int NG>
__device__ __forceinline__ void kv4_quantize_row(const uint2 (&w)[NG], uint32_t (&half)[NG], uint32_t (&sc)[NG]) {
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const uint32_t a = w[g].x & 0x7FFF7FFFu, b = w[g].y & 0x7FFF7FFFu;
    const uint32_t m2 = __vmaxu2(a, b);
    uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    const uint32_t bits = pack_bf16(__fdiv_rn(__uint_as_float(m << 16), 7.f), 0.f) & 0xFFFFu;
    const float s = __uint_as_float(bits << 16);
    const float x[4] = {__uint_as_float(w[g].x << 16), __uint_as_float(w[g].x & 0xFFFF0000u),
                        __uint_as_float(w[g].y << 16), __uint_as_float(w[g].y & 0xFFFF0000u)};
    uint32_t h = 0;
    sc[g] = bits;
    if (m >= 0x7F80u) {
      sc[g] = 0x7FC0u;
    } else if (s >= 0x1p-100f) {
      const float r = __frcp_rn(s);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float y = (fmaf(x[i], r, 6144.f) - 6144.f) + 12582912.f;
        h |= (__float_as_uint(y) & 15u) << (4 * i);
      }
    } else if (s > 0.f) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        h |= ((uint32_t)max(-7, min(7, __float2int_rn(__fdiv_rn(x[i], s)))) & 15u) << (4 * i);
    }
    half[g] = h;
  }
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
  const int count = p.counts ? p.counts[b] : p.n;
  const long long slot = (long long)p.starts[b] + i;
  const bool live = in && i < count && slot >= 0 && slot < p.cap;
  uint2 wk[NG], wv[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const size_t at = (size_t)row * D + 32 * g + 4 * u;
    wk[g] = live ? *reinterpret_cast<const uint2*>(p.k + at) : make_uint2(0, 0);
    wv[g] = live ? *reinterpret_cast<const uint2*>(p.v + at) : make_uint2(0, 0);
  }
  uint32_t hk[NG], hv[NG], sk[NG], sv[NG];
  kv4_quantize_row<NG>(wk, hk, sk);
  kv4_quantize_row<NG>(wv, hv, sv);
  if (!live) return;
  const size_t dst = (size_t)bh * p.cap + slot;
  reinterpret_cast<T*>(p.kc + dst * (D / 2))[u] = kv4_join(hk);
  reinterpret_cast<T*>(p.vc + dst * (D / 2))[u] = kv4_join(hv);
  if (u == 0) *reinterpret_cast<T*>(p.ks + dst * NG) = kv4_join(sk);
  if (u == 1) *reinterpret_cast<T*>(p.vs + dst * NG) = kv4_join(sv);
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

// Rank of a slot as an unsigned key: the newest slots on top, then by weight
// (-0 equals +0, a NaN ranks with -infinity).
__device__ __forceinline__ uint32_t kv4_rank_key(float w, int pos, long long first_recent) {
  if (pos >= first_recent) w = INFINITY;
  if (w != w) w = -INFINITY;
  const uint32_t b = __float_as_uint(w + 0.f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// Which slots of one (batch, cache head) stay, one CTA each.  The n_keep-th
// largest key is found digit by digit; then one ordered walk gives every slot
// its place: kept slots below n_keep stay, the r-th kept slot at or beyond
// n_keep goes into the r-th hole below it.
constexpr int KV4_SEL_THREADS = 1024;
__global__ void __launch_bounds__(KV4_SEL_THREADS) kv4_select_kernel(const Kv4EvictParams p) {
  __shared__ int hist[256];
  __shared__ int wsum[2][32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  const int bh = blockIdx.x, b = bh / p.Hkv;
  const int L = min(max(p.seqlens[b], 0), p.cap);
  int* kept = p.kept + (size_t)bh * p.n_keep;
  if (L <= p.n_keep) {
    for (int j = threadIdx.x; j < p.n_keep; j += KV4_SEL_THREADS) kept[j] = j < L ? j : -1;
    return;
  }
  const float* w = p.weights + (size_t)bh * p.cap;
  const int* pos = p.positions + (size_t)bh * p.cap;
  const long long first_recent = (long long)p.next_pos[b] - p.n_recent;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

  uint32_t prefix = 0, mask = 0;
  int need = p.n_keep;  // how many of the keys that match the prefix are kept
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (threadIdx.x < 256) hist[threadIdx.x] = 0;
    __syncthreads();
    for (int j = threadIdx.x; j < L; j += KV4_SEL_THREADS) {
      const uint32_t key = kv4_rank_key(w[j], pos[j], first_recent);
      if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255u], 1);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      int above = 0, d = 255;
      while (d > 0 && above + hist[d] < need) above += hist[d--];
      s_prefix = prefix | ((uint32_t)d << shift);
      s_need = need - above;
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
    mask |= 255u << shift;
  }

  int* holes = p.lists + (size_t)bh * 2 * p.n_keep;
  int* sources = holes + p.n_keep;
  int eq_before = 0, holes_before = 0, sources_before = 0;
  // exclusive rank of this thread's flag in the CTA, and the CTA's count
  auto scan = [&](bool f, int which, int& total) {
    const unsigned m = __ballot_sync(0xffffffffu, f);
    if (lane == 0) wsum[which][warp] = __popc(m);
    __syncthreads();
    int before = 0;
    total = 0;
    for (int i = 0; i < 32; ++i) {
      if (i < warp) before += wsum[which][i];
      total += wsum[which][i];
    }
    return before + __popc(m & ((1u << lane) - 1u));
  };
  for (int j0 = 0; j0 < L; j0 += KV4_SEL_THREADS) {
    const int j = j0 + threadIdx.x;
    const bool in = j < L;
    const uint32_t key = in ? kv4_rank_key(w[j], pos[j], first_recent) : 0u;
    int n_eq, n_other;
    const bool eq = in && key == prefix;
    const int r = eq_before + scan(eq, 0, n_eq);
    const bool keep = in && (key > prefix || (eq && r < need));
    const bool front = j < p.n_keep;
    const bool hole = in && front && !keep, source = in && !front && keep;
    if (front && keep) kept[j] = j;
    __syncthreads();
    // a chunk may hold both kinds: holes first
    const int hr = holes_before + scan(hole, 1, n_other);
    if (hole) holes[hr] = j;
    holes_before += n_other;
    __syncthreads();
    const int sr = sources_before + scan(source, 0, n_other);
    if (source) sources[sr] = j;
    sources_before += n_other;
    eq_before += n_eq;
    __syncthreads();
  }
  for (int r = threadIdx.x; r < holes_before; r += KV4_SEL_THREADS) kept[holes[r]] = sources[r];
}

// Rows move from slots >= n_keep into slots < n_keep only, so no row is read
// after it was overwritten and a repeated call moves the same rows again.
template <int NG>
__global__ void __launch_bounds__(256) kv4_move_kernel(const Kv4EvictParams p, unsigned rows) {
  constexpr int D = 32 * NG;
  using T = typename Kv4Piece<NG>::T;
  const unsigned row = blockIdx.x * 32u + (threadIdx.x >> 3);
  const int u = threadIdx.x & 7;
  if (row >= rows) return;
  const unsigned bh = row / (unsigned)p.n_keep;
  const int j = (int)(row - bh * (unsigned)p.n_keep);
  const int from = p.kept[row];
  if (from < 0) return;
  const size_t src = (size_t)bh * p.cap + from, dst = (size_t)bh * p.cap + j;
  if (u == 0) p.weights_out[dst] = p.weights[src];
  if (u == 1) p.positions_out[dst] = p.positions[src];
  if (from == j) return;
  reinterpret_cast<T*>(p.kc + dst * (D / 2))[u] = reinterpret_cast<const T*>(p.kc + src * (D / 2))[u];
  reinterpret_cast<T*>(p.vc + dst * (D / 2))[u] = reinterpret_cast<const T*>(p.vc + src * (D / 2))[u];
  if (u == 2) *reinterpret_cast<T*>(p.ks + dst * NG) = *reinterpret_cast<const T*>(p.ks + src * NG);
  if (u == 3) *reinterpret_cast<T*>(p.vs + dst * NG) = *reinterpret_cast<const T*>(p.vs + src * NG);
}

}  // namespace ta
