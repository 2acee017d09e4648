// Decode over the 4-bit cache (row format: kv4.cuh): one query row per (batch,
// query head) against the live slots [0, seqlens[b]) of its cache head,
//
//   x_j = scale log2(e) q . k_j,  m = max x_j,  l = sum 2^(x_j - m),
//   o = sum 2^(x_j - m) v_j / l,  lse = ln 2 (m + log2 l),
//   and, where asked for, w_j += sum over the heads of a cache head of
//   2^(x_j - lse log2(e)), the accumulated attention weight of a slot.
//
// The live slots of the whole batch, 64 at a time, form one sequence of tiles
// (batch by batch, cache head by cache head), cut into equal pieces, one per
// warp: however lengths are spread, every warp streams the same number of bytes.
// A piece may begin and end inside a row; each (row, piece) leaves a partial
// output, its sum of probabilities and the exponent that is relative to, and a second
// kernel merges a row's partials.  A weight needs the log-sum-exp of the whole row, so
// the first kernel leaves the scores x in the workspace, fp32 (8 bytes a slot and
// head written and read, mostly in L2, against 4.5 bits a channel to read K
// again), and the second one turns them into weights.
//
// Bound by the chain of logic operations, products and conversions that makes 4-bit
// operands (2 warps on a scheduler: fixed latencies, then the ALU pipe at 44 %), not by
// memory: 64 sequences of 8192 slots, 8 cache heads of 4 query heads, d = 128 (605 MB)
// take 143 us (4.2 TB/s); 125 with the data in L2 and 106 streamed only where the whole took
// 140, before each group's scales had a power of two of their own.
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
  float* o_part;                 // [partial][head of the block][D], over the partial's sum
  float2* ml_part;               // [partial][head of the block]: exponent M, sum l of 2^(x - M)
  float* x;                      // [B*Hq][cap] scores, or null
  const int* seqlens;            // [B]
  int B, Hkv, group, cap;
  int blocks;                    // blocks of <= 8 query heads per cache head
  int per_block;                 // heads of a block: min(8, group)
  int pieces;
  float sl2;                     // scale log2(e) = sl2 2^sl2_exp
  int sl2_exp;
  unsigned long long timeout_ns;
};

// A tile of 64 slots is one straight run of instructions: with 2 warps on each
// scheduler and up to 255 registers the independent chains of its four 16-slot
// parts hide the latencies better than more warps do with shorter runs (64
// sequences of 8192 slots, 8 cache heads of 4 query heads, 605 MB, at the time: 148 us;
// 12 warps of 168 registers and 32 slots 161; 16 warps of 128 and 32 slots 159; 16
// slots at a time 169 to 178).
constexpr int KV4_TILE = 64;                // slots of a tile
constexpr int KV4_WARPS = 4, KV4_CTAS = 2;  // warps of a CTA, CTAs of an SM
// bf16x2 words of exponents: the least reference of V's scales, 2^-112 (2^15 over it
// is the largest power of two), and what a reference is taken from to give that quotient
constexpr uint32_t KV4_VREF0 = ((127 - 112) << 7) * 0x10001u, KV4_VUP = ((2 * 127 + 15) << 7) * 0x10001u;

template <int NG>
struct DecKv4Cfg {
  static constexpr int D = 32 * NG;
  static constexpr int WARPS = KV4_WARPS, CTAS = KV4_CTAS, TILE = KV4_TILE;
  static constexpr int U = TILE / 16, STAGES = NG == 4 ? 2 : 4;
  static constexpr int CODES = TILE * D / 2, SCALES = TILE * NG * 2;
  static constexpr int STAGE = 2 * (CODES + SCALES);  // K codes, V codes, K scales, V scales
  static constexpr int BAR_OFF = WARPS * STAGES * STAGE;
  static constexpr int SMEM = BAR_OFF + WARPS * STAGES * 8 + WARPS * 4;
  // lazy rescale: the reference max moves when a score exceeds it by TAU (log2
  // units); probabilities are taken 2^-TAU smaller, so that none exceeds 1 and a
  // piece's sum of them is from 2^-TAU to its number of slots, whatever the values
  static constexpr float TAU = 8.f;
};

// Where a row's tiles lie in the batch's sequence of tiles.  An item is one block
// of query heads of one cache head: item = (batch * Hkv + cache head) * blocks + block.
__device__ __forceinline__ int kv4_tiles(const int* __restrict__ seqlens, int b, int cap) {
  return (min(max(seqlens[b], 0), cap) + KV4_TILE - 1) / KV4_TILE;
}
// tiles of one item of each batch entry, summed over entries [0, n); whole warp
__device__ __forceinline__ int kv4_tiles_before(const int* __restrict__ seqlens, int n, int cap) {
  int s = 0;
  for (int b = threadIdx.x & 31; b < n; b += 32) s += kv4_tiles(seqlens, b, cap);
  return __reduce_add_sync(0xffffffffu, s);
}
__host__ __device__ inline int kv4_per_piece(int total, int pieces) { return max(1, (total + pieces - 1) / pieces); }

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
// d += a b
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// (a & MASK) ^ flip in one logic operation
template <uint32_t MASK>
__device__ __forceinline__ uint32_t and_xor(uint32_t a, uint32_t flip) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(d) : "r"(a), "n"(MASK), "r"(flip));
  return d;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
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

// half of a word of scales as a float, by a byte selector (0x1044 the low one, 0x3244 the high one)
__device__ __forceinline__ float kv4_half_float(uint32_t w, uint32_t pick) {
  return __uint_as_float(__byte_perm(w, 0u, pick));
}
// word i (two groups) of a row's scales
__device__ __forceinline__ uint32_t kv4_word(const uint2& w, int i) { return i ? w.y : w.x; }
__device__ __forceinline__ uint32_t kv4_word(const uint32_t& w, int) { return w; }

// the words of a row's scales times powers of two, exact as long as the product is normal
__device__ __forceinline__ void kv4_scale_words(uint2& w, const uint32_t (&up)[2]) {
  w.x = mul_bf16x2(w.x, up[0]), w.y = mul_bf16x2(w.y, up[1]);
}
__device__ __forceinline__ void kv4_scale_words(uint32_t& w, const uint32_t (&up)[1]) { w = mul_bf16x2(w, up[0]); }
// 2^n as a float, 0 below the normal numbers; n <= 127
__device__ __forceinline__ float kv4_exp2i(int n) { return n < -126 ? 0.f : __uint_as_float((uint32_t)(127 + n) << 23); }

// Each warp is on its own: it walks its piece tile by tile through its own ring
// of bulk copies, which runs ahead across the rows of the piece, and keeps its
// own running max, sum and output.  r = lane / 4, t = lane % 4 below.
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
//     of the group, rounded to fp16 (the one rounding of P, 2^-11), with the
//     scale taken times a power of two that keeps p s below 2^15.  That power follows
//     the largest scale of the group met so far as the running max follows the scores, so
//     a product counts from 2^-32 of its group's largest scale on; it never touches p or
//     the sum of p, which know nothing of the values.  The offset goes out 16
//     slots at a time through a second product with the constant -8: summed up over
//     a long row it would swamp the result.  What the cancellation leaves is below
//     2^-15 of p times the scale (a step of the grid), far inside the format's own
//     half step.
//
// PAIR, for up to 4 heads: the 8 columns are 4 heads for the even and 4 heads for
// the odd group of a pair.  A word of codes (4 channels of each group of the pair)
// then is an operand as it lies, without bringing a group's halves together, a
// lane works on the scales of one group of the pair only, and one more addition
// across lanes joins the scores of the two (64 x 8192 slots, 8 cache heads of 4, at the
// time: 141 us against 143, one row of 131072 slots 53 against 55).
template <int NG, bool PAIR>
__global__ void __launch_bounds__(32 * DecKv4Cfg<NG>::WARPS, DecKv4Cfg<NG>::CTAS)
    decode_kv4_kernel(const __grid_constant__ DecKv4Params p) {
  using C = DecKv4Cfg<NG>;
  using T = typename Kv4Piece<NG>::T;
  constexpr int D = C::D;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF) + warp * C::STAGES;
  int* abort_flag = reinterpret_cast<int*>(smem + C::BAR_OFF + C::WARPS * C::STAGES * 8) + warp;  // the warp's own
  uint8_t* ring = smem + warp * C::STAGES * C::STAGE;
  if (lane == 0) {
    *abort_flag = 0;
    for (int s = 0; s < C::STAGES; ++s) mbar_init(smem_u32(&bars[s]), 1);
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  __syncwarp();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the finish may line up behind this grid

  // ---- this warp's piece: tiles [first, first + mine) of the batch
  const int per_entry = p.Hkv * p.blocks;  // items of a batch entry
  const int total = kv4_tiles_before(p.seqlens, p.B, p.cap) * per_entry;
  const int per = kv4_per_piece(total, p.pieces);
  // 64 bits: pieces that start behind the last tile
  const long long first = (long long)(blockIdx.x * C::WARPS + warp) * per;
  const int mine = (int)max(0LL, min((long long)per, total - first));
  if (mine == 0) return;
  const int piece = blockIdx.x * C::WARPS + warp;
  int b = 0, before = 0;  // batch entry of the first tile, tiles before it
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int n = b0 + lane < p.B ? kv4_tiles(p.seqlens, b0 + lane, p.cap) * per_entry : 0;
    int sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    const unsigned beyond = __ballot_sync(0xffffffffu, before + sum > first);
    if (beyond) {
      const int at = __ffs(beyond) - 1;
      b = b0 + at;
      before += __shfl_sync(0xffffffffu, sum - n, at);
      break;
    }
    before += __shfl_sync(0xffffffffu, sum, 31);
  }
  // a place in the batch's tiles: entry b of length len, its item, tile of tiles
  struct Place {
    int b, len, tiles, item, tile;
    size_t row;  // first slot of the item's cache head
  };
  auto enter = [&](Place& c, int bb) {
    c.b = bb;
    c.len = min(max(p.seqlens[bb], 0), p.cap);
    c.tiles = (c.len + C::TILE - 1) / C::TILE;
  };
  auto next_item = [&](Place& c) {  // only where there is one with tiles
    c.tile = 0;
    if (++c.item == (c.b + 1) * per_entry) {
      do {
        enter(c, c.b + 1);
        c.item = c.b * per_entry;
      } while (c.tiles == 0);
    }
    c.row = (size_t)(c.item / p.blocks) * p.cap;
  };
  Place at, ahead;
  enter(at, b);
  {
    const int rem = (int)(first - before);
    at.item = b * per_entry + rem / at.tiles;
    at.tile = rem % at.tiles;
    at.row = (size_t)(at.item / p.blocks) * p.cap;
  }
  ahead = at;
  int issued = 0;
  auto issue = [&](int stage) {  // lane 0: the next tile of the piece into the next stage
    const int slot = ahead.tile * C::TILE;
    const uint32_t rows = (uint32_t)min(C::TILE, (ahead.len - slot + 15) & ~15);  // capacity is a multiple of 16
    const size_t row = ahead.row + slot;
    const uint32_t dst = smem_u32(ring + stage * C::STAGE), bar = smem_u32(&bars[stage]);
    mbar_arrive_expect_tx(bar, rows * (D + 4 * NG));
    bulk_load(dst, p.kc + row * (D / 2), rows * (D / 2), bar);
    bulk_load(dst + 2 * C::CODES, p.ks + row * NG, rows * NG * 2, bar);
    bulk_load(dst + C::CODES, p.vc + row * (D / 2), rows * (D / 2), bar);
    bulk_load(dst + 2 * C::CODES + C::SCALES, p.vs + row * NG, rows * NG * 2, bar);
    if (++issued < mine && ++ahead.tile == ahead.tiles) next_item(ahead);
  };
  if (lane == 0)
    while (issued < min(mine, C::STAGES)) issue(issued);

  bool ok = true;
  int i = 0;  // tiles of the piece done; the next one's stage and its phase
  int st = 0;
  uint32_t phase = 0;
  while (true) {
    const int bhk = at.item / p.blocks, blk = at.item - bhk * p.blocks;
    const int heads = min(8, p.group - blk * 8);
    const size_t bh0 = (size_t)bhk * p.group + blk * 8;  // first query head (batch * Hq + head)
  // ---- queries: head r, channels 32 g + 8 t + 0..7 of each group, as B fragments.
  // PAIR: head r % 4, of each pair of groups the even (r < 4) or the odd one
  constexpr int NQ = PAIR ? NG / 2 : NG;
  const int head = PAIR ? r & 3 : r, hi = t >> 1;  // hi: this lane's scores are the odd group's
  uint32_t qb[NQ][PAIR ? 8 : 4];
  float c0[NQ][4];  // accumulator start of heads 2t, 2t + 1, once for each slot of the lane
  float fx[2];
  int far_exp[2];
  {
    uint4 w[NG];
    uint32_t m = 0;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      w[g] = head < heads ? *reinterpret_cast<const uint4*>(p.q + (bh0 + head) * D + 32 * g + 8 * t) : make_uint4(0, 0, 0, 0);
      const uint32_t a = __vmaxu2(__vmaxu2(w[g].x & 0x7FFF7FFFu, w[g].y & 0x7FFF7FFFu),
                                  __vmaxu2(w[g].z & 0x7FFF7FFFu, w[g].w & 0x7FFF7FFFu));
      m = max(m, max(a & 0xFFFFu, a >> 16));
    }
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    // largest channel in [2^e, 2^(e+1)) (below the normal numbers: e = -126); a
    // head with an infinity or a NaN is left as it is, its outputs are NaN anyway; so is
    // one of zeros, whose scores are 0 at any size
    const int e = m == 0u || m >= 0x7F80u ? 14 : max(1, (int)(m >> 7)) - 127;
    const int e0 = (14 - e) / 2;  // 2^(14 - e) in two factors
    const float up0 = __uint_as_float((uint32_t)(127 + e0) << 23), up1 = __uint_as_float((uint32_t)(127 + 14 - e - e0) << 23);
#pragma unroll
    for (int g = 0; g < NQ; ++g) {
      const uint4 own = !PAIR ? w[g] : r < 4 ? w[2 * g] : w[2 * g + 1 < NG ? 2 * g + 1 : 0];
      const uint32_t ww[4] = {own.x, own.y, own.z, own.w};
      float f[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        f[2 * k] = bf2f(ww[k], 0) * up0 * up1;
        f[2 * k + 1] = bf2f(ww[k], 1) * up0 * (up1 * 0.0625f);
      }
      float sum = 0.f;
      if constexpr (PAIR) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {  // channel k: nibble k % 4 of piece 2t or 2t + 1
          const __half2 h = r < 4 ? __floats2half2_rn(f[k], 0.f) : __floats2half2_rn(0.f, f[k]);
          qb[g][k] = *reinterpret_cast<const uint32_t*>(&h);
          sum += (__low2float(h) + __high2float(h)) * ((k & 1) ? 16.f : 1.f);
        }
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // nibble k of the two halfwords: channels k and 4 + k
        const __half2 h = __floats2half2_rn(f[k], f[4 + k]);
        qb[g][k] = *reinterpret_cast<const uint32_t*>(&h);
        sum += (__low2float(h) + __high2float(h)) * ((k & 1) ? 16.f : 1.f);
      }
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      sum *= -8.f * 0x1p-24f;
      c0[g][0] = __shfl_sync(0xffffffffu, sum, 8 * t);
      c0[g][1] = __shfl_sync(0xffffffffu, sum, 8 * t + 4);
      c0[g][2] = c0[g][0], c0[g][3] = c0[g][1];
      // the instruction takes four registers in a row: four values of their own,
      // or every product would start with four moves
      asm volatile("" : "+f"(c0[g][0]), "+f"(c0[g][1]), "+f"(c0[g][2]), "+f"(c0[g][3]));
    }
    // x = y sl2 2^(sl2_exp + 24 + e - 14).  Of that power fx holds what keeps it far from
    // 0 and infinity; the rest, if any (queries or scales of extreme size), goes into
    // y as soon as it is there
    const int exponent = p.sl2_exp + 10 + e, near_exp = max(-60, min(60, exponent));
    const float f = p.sl2 * kv4_exp2i(near_exp);
    fx[0] = __shfl_sync(0xffffffffu, f, 8 * t), fx[1] = __shfl_sync(0xffffffffu, f, 8 * t + 4);
    far_exp[0] = __shfl_sync(0xffffffffu, exponent - near_exp, 8 * t);
    far_exp[1] = __shfl_sync(0xffffffffu, exponent - near_exp, 8 * t + 4);
  }
  const bool any_far = __any_sync(0xffffffffu, (far_exp[0] | far_exp[1]) != 0);

  float acc[2 * NG][4];
#pragma unroll
  for (int i = 0; i < 2 * NG; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
  // per head 2t, 2t + 1: reference max of y (scores before fx), threshold above which
  // it moves, exponent M that probabilities are taken against.  vref: 2^ev of each two
  // groups, bf16x2, no scale so far is larger; vup: 2^(15 - ev)
  float my[2] = {-INFINITY, -INFINITY}, thr[2] = {-INFINITY, -INFINITY}, M[2] = {0.f, 0.f}, l[2] = {0.f, 0.f};
  uint32_t vref[NG / 2], vup[NG / 2];
#pragma unroll
  for (int w = 0; w < NG / 2; ++w) vref[w] = KV4_VREF0, vup[w] = KV4_VUP - KV4_VREF0;
  const uint32_t flip0 = 0x00080008u, flip1 = 0x00800080u;
  const uint32_t pick = hi ? 0x3244u : 0x1044u;  // PAIR: this lane's half of a word of scales, as a float

  for (const int end = min(mine, i + at.tiles - at.tile); i < end; ++i, ++at.tile) {
    ok = __all_sync(0xffffffffu, wait_bar(smem_u32(&bars[st]), phase, abort_flag, p.timeout_ns));
    if (!ok) break;
    const uint8_t* buf = ring + st * C::STAGE;
    const int slot0 = at.tile * C::TILE;
    const int left = at.len - slot0;  // live slots from here on
    const uint8_t* ksb = buf + 2 * C::CODES;
    // ---- scores: [16-slot part][slot r or r + 8, head 2t or 2t + 1]
    float y[C::U][4];
#pragma unroll
    for (int u = 0; u < C::U; ++u) {
      if constexpr (PAIR) {
        uint32_t kw[2][NG];
        T sc[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = 16 * u + r + 8 * h;
          if constexpr (NG == 4) {
            const uint4 w = *reinterpret_cast<const uint4*>(buf + row * 64 + t * 16);
            kw[h][0] = w.x, kw[h][1] = w.z, kw[h][2] = w.y, kw[h][3] = w.w;
          } else {
            const uint2 w = *reinterpret_cast<const uint2*>(buf + row * 32 + t * 8);
            kw[h][0] = w.x, kw[h][1] = w.y;
          }
          sc[h] = *reinterpret_cast<const T*>(ksb + row * NG * 2);
        }
#pragma unroll
        for (int g = 0; g < NQ; ++g) {
          float s[4];
#pragma unroll
          for (int piece = 0; piece < 2; ++piece) {
            const uint32_t a = kw[0][2 * g + piece], b = kw[1][2 * g + piece], a8 = a >> 8, b8 = b >> 8;
            const uint32_t* q4 = &qb[g][4 * piece];
            if (piece == 0)
              mma_f16_16816(s, and_xor<0x000F000Fu>(a, flip0), and_xor<0x000F000Fu>(b, flip0),
                            and_xor<0x00F000F0u>(a, flip1), and_xor<0x00F000F0u>(b, flip1), q4[0], q4[1], c0[g][0],
                            c0[g][1], c0[g][2], c0[g][3]);
            else
              mma_f16_16816(s, and_xor<0x000F000Fu>(a, flip0), and_xor<0x000F000Fu>(b, flip0),
                            and_xor<0x00F000F0u>(a, flip1), and_xor<0x00F000F0u>(b, flip1), q4[0], q4[1]);
            mma_f16_16816(s, and_xor<0x000F000Fu>(a8, flip0), and_xor<0x000F000Fu>(b8, flip0),
                          and_xor<0x00F000F0u>(a8, flip1), and_xor<0x00F000F0u>(b8, flip1), q4[2], q4[3]);
          }
          const float f0 = kv4_half_float(kv4_word(sc[0], g), pick), f1 = kv4_half_float(kv4_word(sc[1], g), pick);
          y[u][0] = g ? fmaf(s[0], f0, y[u][0]) : s[0] * f0;
          y[u][1] = g ? fmaf(s[1], f0, y[u][1]) : s[1] * f0;
          y[u][2] = g ? fmaf(s[2], f1, y[u][2]) : s[2] * f1;
          y[u][3] = g ? fmaf(s[3], f1, y[u][3]) : s[3] * f1;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) y[u][e] += __shfl_xor_sync(0xffffffffu, y[u][e], 2);
        continue;
      }
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
        sc[h] = *reinterpret_cast<const T*>(ksb + row * NG * 2);
      }
#pragma unroll
      for (int g = 0; g < (PAIR ? 0 : NG); ++g) {
        float s[4];
        const uint32_t a = kw[0][g], b = kw[1][g], a8 = a >> 8, b8 = b >> 8;
        mma_f16_16816(s, and_xor<0x000F000Fu>(a, flip0), and_xor<0x000F000Fu>(b, flip0),
                      and_xor<0x00F000F0u>(a, flip1), and_xor<0x00F000F0u>(b, flip1), qb[g][0], qb[g][1], c0[g][0],
                      c0[g][1], c0[g][2], c0[g][3]);
        mma_f16_16816(s, and_xor<0x000F000Fu>(a8, flip0), and_xor<0x000F000Fu>(b8, flip0),
                      and_xor<0x00F000F0u>(a8, flip1), and_xor<0x00F000F0u>(b8, flip1), qb[g][2], qb[g][3]);
        const float f0 = bf2f(kv4_word(sc[0], g >> 1), g & 1), f1 = bf2f(kv4_word(sc[1], g >> 1), g & 1);
        y[u][0] = g ? fmaf(s[0], f0, y[u][0]) : s[0] * f0;
        y[u][1] = g ? fmaf(s[1], f0, y[u][1]) : s[1] * f0;
        y[u][2] = g ? fmaf(s[2], f1, y[u][2]) : s[2] * f1;
        y[u][3] = g ? fmaf(s[3], f1, y[u][3]) : s[3] * f1;
      }
    }
    if (any_far) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float f0 = kv4_exp2i(far_exp[k] / 2), f1 = kv4_exp2i(far_exp[k] - far_exp[k] / 2);
#pragma unroll
        for (int u = 0; u < C::U; ++u) y[u][k] = y[u][k] * f0 * f1, y[u][k + 2] = y[u][k + 2] * f0 * f1;
      }
    }
    T vs[C::U][2];
#pragma unroll
    for (int u = 0; u < C::U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        vs[u][h] = *reinterpret_cast<const T*>(ksb + C::SCALES + (16 * u + r + 8 * h) * NG * 2);
    if (left < C::TILE) {  // slots behind the live ones: no score, and their scales may be anything
#pragma unroll
      for (int u = 0; u < C::U; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (16 * u + r + 8 * h >= left) {
            y[u][2 * h] = y[u][2 * h + 1] = -INFINITY;
            vs[u][h] = T{};
          }
    }
    if (p.x) {
#pragma unroll
      for (int u = 0; u < C::U; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = 16 * u + r + 8 * (e >> 1);
          if (2 * t + (e & 1) < heads && j < left)
            p.x[(bh0 + 2 * t + (e & 1)) * p.cap + slot0 + j] = y[u][e] * fx[e & 1];
        }
    }
    // ---- references, moved only when they must
    float h0 = fmaxf(y[0][0], y[0][2]), h1 = fmaxf(y[0][1], y[0][3]);
#pragma unroll
    for (int u = 1; u < C::U; ++u) h0 = fmax3(h0, y[u][0], y[u][2]), h1 = fmax3(h1, y[u][1], y[u][3]);
    uint32_t vm[NG / 2];
    bool vmoved = false;
#pragma unroll
    for (int w = 0; w < NG / 2; ++w) {
      vm[w] = vref[w];
#pragma unroll
      for (int u = 0; u < C::U; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) vm[w] = max_bf16x2(vm[w], kv4_word(vs[u][h], w));
      vmoved |= vm[w] != vref[w];
    }
    if (__any_sync(0xffffffffu, h0 > thr[0] || h1 > thr[1] || vmoved)) {
      // what the outputs of each of the lane's groups shrink by for V's sake
      float fv[NQ];
#pragma unroll
      for (int w = 0; w < NG / 2; ++w) {
        uint32_t v = vm[w];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) v = max_bf16x2(v, __shfl_xor_sync(0xffffffffu, v, o));
        const uint32_t lo = (v & 0xFFFFu) > (vref[w] & 0xFFFFu) ? (v & 0x7F80u) + 0x80u : vref[w] & 0xFFFFu;
        const uint32_t up = (v >> 16) > (vref[w] >> 16) ? ((v >> 16) & 0x7F80u) + 0x80u : vref[w] >> 16;
        const float f0 = kv4_exp2i(((int)(vref[w] & 0xFFFFu) - (int)lo) >> 7);
        const float f1 = kv4_exp2i(((int)(vref[w] >> 16) - (int)up) >> 7);
        if constexpr (PAIR)
          fv[w] = hi ? f1 : f0;
        else
          fv[2 * w] = f0, fv[2 * w + 1] = f1;
        vref[w] = lo | up << 16;
        vup[w] = KV4_VUP - vref[w];
      }
      float mx[2] = {h0, h1};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], o));
        if (!(mx[k] > my[k])) mx[k] = my[k];
        float f = 1.f;
        if (mx[k] != -INFINITY) {
          const float Mn = fmaf(mx[k], fx[k], C::TAU);
          f = my[k] == -INFINITY ? 0.f : ex2(M[k] - Mn);  // l and acc are 0 or NaN while my = -inf
          l[k] *= f;
          my[k] = mx[k];
          M[k] = Mn;
          thr[k] = mx[k] + C::TAU / fx[k];
        }
#pragma unroll
        for (int n = 0; n < 2 * NG; ++n) {
          const float fn = f * fv[n / (PAIR ? 4 : 2)];
          acc[n][k] *= fn, acc[n][k + 2] *= fn;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < C::U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) kv4_scale_words(vs[u][h], vup);
    float pr[C::U][4];
#pragma unroll
    for (int u = 0; u < C::U; ++u) {
#pragma unroll
      for (int e = 0; e < 4; ++e) pr[u][e] = ex2(fmaf(y[u][e], fx[e & 1], -M[e & 1]));
      l[0] += pr[u][0] + pr[u][2];
      l[1] += pr[u][1] + pr[u][3];
    }
    // ---- values: piece r of slots 2t, 2t + 1, 2t + 8, 2t + 9 of each half
#pragma unroll
    for (int u = 0; u < C::U; ++u) {
      T vw[4];
#pragma unroll
      for (int h = 0; h < 4; ++h)
        vw[h] = *reinterpret_cast<const T*>(buf + C::CODES + (16 * u + 2 * t + (h & 1) + 8 * (h >> 1)) * (D / 2) + r * 2 * NG);
      if constexpr (PAIR) {
#pragma unroll
        for (int g = 0; g < NQ; ++g) {
          const float f0 = kv4_half_float(kv4_word(vs[u][0], g), pick), f1 = kv4_half_float(kv4_word(vs[u][1], g), pick);
          const uint32_t b0 = movmatrix_trans(pack_f16(pr[u][0] * f0, pr[u][1] * f0));
          const uint32_t b1 = movmatrix_trans(pack_f16(pr[u][2] * f1, pr[u][3] * f1));
          uint32_t a[4];  // even and odd group: slots 2t, 2t + 1, then 2t + 8, 2t + 9
#pragma unroll
          for (int h = 0; h < 4; ++h)
            a[h] = __byte_perm(kv4_word(vw[h & 2], g), kv4_word(vw[(h & 2) + 1], g), (h & 1) ? 0x7632 : 0x5410);
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            if (n == 1) {
#pragma unroll
              for (int h = 0; h < 4; ++h) a[h] >>= 8;
            }
            float(&o0)[4] = acc[4 * g + 2 * n];
            float(&o1)[4] = acc[4 * g + 2 * n + 1];
            mma_f16_16816(o0, 0x80088008u, 0x80088008u, 0x80088008u, 0x80088008u, b0, b1);
            mma_f16_16816(o1, 0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u, b0, b1);
            mma_f16_16816(o0, and_xor<0x000F000Fu>(a[0], flip0), and_xor<0x000F000Fu>(a[1], flip0),
                          and_xor<0x000F000Fu>(a[2], flip0), and_xor<0x000F000Fu>(a[3], flip0), b0, b1);
            mma_f16_16816(o1, and_xor<0x00F000F0u>(a[0], flip1), and_xor<0x00F000F0u>(a[1], flip1),
                          and_xor<0x00F000F0u>(a[2], flip1), and_xor<0x00F000F0u>(a[3], flip1), b0, b1);
          }
        }
        continue;
      }
#pragma unroll
      for (int g = 0; g < (PAIR ? 0 : NG); ++g) {
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
          mma_f16_16816(o, 0x80088008u, 0x80808080u, 0x80088008u, 0x80808080u, b0, b1);
          const uint32_t w0 = n ? a[0] >> 8 : a[0], w1 = n ? a[1] >> 8 : a[1];
          mma_f16_16816(o, and_xor<0x000F000Fu>(w0, flip0), and_xor<0x00F000F0u>(w0, flip1),
                        and_xor<0x000F000Fu>(w1, flip0), and_xor<0x00F000F0u>(w1, flip1), b0, b1);
        }
      }
    }
    __syncwarp();
    if (lane == 0 && issued < mine) issue(st);
    if (++st == C::STAGES) st = 0, phase ^= 1u;
  }
  if (!ok) break;

  // ---- the row's partial result of this piece
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) l[k] += __shfl_xor_sync(0xffffffffu, l[k], o);
  const size_t part = (size_t)(piece + at.item) * p.per_block;  // unique: the next piece or item has the next number
  // A partial output is divided by its own sum: a mean of values, which no number of
  // slots carries out of range.  2^(24 + ev - 15) over the sum, in three factors
  float inv[2], back[NQ][2];
#pragma unroll
  for (int g = 0; g < NQ; ++g) {
    const uint32_t v = PAIR ? vref[g] >> (hi ? 16 : 0) : vref[g / 2] >> (g & 1 ? 16 : 0);
    const int ev = (int)((v & 0xFFFFu) >> 7) - 127;
    back[g][0] = kv4_exp2i(ev / 2), back[g][1] = kv4_exp2i(ev - ev / 2);
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) inv[k] = l[k] == 0.f ? 0.f : 0x1p9f / l[k];
  if constexpr (PAIR) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int h = (2 * t + k) & 3;
      if (h >= heads) continue;
      float* o = p.o_part + (part + h) * D + 32 * hi + 4 * r;
#pragma unroll
      for (int g = 0; g < NQ; ++g) {
        float v[4];
#pragma unroll
        for (int i4 = 0; i4 < 4; ++i4)  // odd nibbles carry 16
          v[i4] = (hi ? acc[4 * g + i4][k + 2] : acc[4 * g + i4][k]) * ((i4 & 1) ? inv[k] * 0.0625f : inv[k]) * back[g][0] * back[g][1];
        *reinterpret_cast<float4*>(o + 64 * g) = make_float4(v[0], v[1], v[2], v[3]);
      }
      if (r == 0 && !hi) p.ml_part[part + h] = make_float2(my[k] == -INFINITY ? -INFINITY : M[k], l[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < (PAIR ? 0 : 2); ++k) {
    if (2 * t + k >= heads) continue;
    float* o = p.o_part + (part + 2 * t + k) * D + 4 * r;
#pragma unroll
    for (int g = 0; g < NG; ++g) {  // odd nibbles carry 16
      const float f[2] = {inv[k], inv[k] * 0.0625f};
      float v[4];
#pragma unroll
      for (int i4 = 0; i4 < 4; ++i4) v[i4] = acc[2 * g + i4 / 2][k + 2 * (i4 & 1)] * f[i4 & 1] * back[g][0] * back[g][1];
      *reinterpret_cast<float4*>(o + 32 * g) = make_float4(v[0], v[1], v[2], v[3]);
    }
    if (r == 0) p.ml_part[part + 2 * t + k] = make_float2(my[k] == -INFINITY ? -INFINITY : M[k], l[k]);
  }
  if (i == mine) break;
  next_item(at);
  }
  if (!ok) {  // never leave a copy in flight
    issued = __shfl_sync(0xffffffffu, issued, 0);
    for (; i < issued; ++i) wait_bar_drain(smem_u32(&bars[i % C::STAGES]), (i / C::STAGES) & 1, p.timeout_ns);
  }
}

// A row's partials: the first one's index and how many (none without slots); whole warp
struct Kv4Parts {
  size_t first;
  int n;
};
__device__ __forceinline__ Kv4Parts kv4_row_parts(const DecKv4Params& p, int row) {
  const int Hq = p.Hkv * p.group, b = row / Hq, h = row - b * Hq;
  const int tiles = kv4_tiles(p.seqlens, b, p.cap), per_entry = p.Hkv * p.blocks;
  const int per = kv4_per_piece(kv4_tiles_before(p.seqlens, p.B, p.cap) * per_entry, p.pieces);
  const int in_entry = h / p.group * p.blocks + h % p.group / 8, head = h % p.group % 8;
  const int t0 = kv4_tiles_before(p.seqlens, b, p.cap) * per_entry + in_entry * tiles, c0 = t0 / per;
  Kv4Parts r;
  r.first = (size_t)(c0 + b * per_entry + in_entry) * p.per_block + head;
  r.n = tiles == 0 ? 0 : (t0 + tiles - 1) / per - c0 + 1;
  return r;
}
__device__ __forceinline__ float kv4_part_factor(float M, float mx) { return M == mx ? 1.f : ex2(M - mx); }  // all NaN: no max
__device__ __forceinline__ float kv4_lse2(float mx, float l) { return (mx == -INFINITY ? 0.f : mx) + log2f(l); }
__device__ __forceinline__ float kv4_warp_max(float v) {
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, k));
  return v;
}
// max M and sum_c 2^(M_c - max M) l_c over a row's partials; whole warp
__device__ __forceinline__ float2 kv4_row_sum(const DecKv4Params& p, const Kv4Parts& parts) {
  const float2* ml = p.ml_part + parts.first;
  float m = -INFINITY, l = 0.f;
#pragma unroll 1
  for (int c = threadIdx.x & 31; c < parts.n; c += 128) {  // four in flight
    float2 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      v[k] = c + 32 * k < parts.n ? ml[(size_t)(c + 32 * k) * p.per_block] : make_float2(-INFINITY, 0.f);
    const float grown = fmaxf(fmaxf(m, fmax3(v[0].x, v[1].x, v[2].x)), v[3].x);
    l *= kv4_part_factor(m, grown);
#pragma unroll
    for (int k = 0; k < 4; ++k) l = fmaf(kv4_part_factor(v[k].x, grown), v[k].y, l);
    m = grown;
  }
  const float mx = kv4_warp_max(m);
  l *= kv4_part_factor(m, mx);
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
  return make_float2(mx, l);
}

// What the pieces left becomes the outputs, in one launch.  The first CTAs merge: with
// f = 2^(M_c - max M), L = sum f l_c, O = sum (f l_c / L) O_c, LSE = ln 2 (max M + log2 L);
// a row without slots has no partial, a NaN in a live slot stays one.  CTAS = 0: a
// warp per row, its partials in loads of 4 (d = 64: of 8); 1: a CTA per row, a warp (half a warp of
// d = 64) per partial; more: a CTA per 32 channels of a row, 32 partials at a time.
// The other CTAs, where weights are wanted, take 1024 slots of a cache head each:
// w_j += sum_h 2^(x_hj - lse_h log2 e), with the rows' log-sum-exps worked out again
// from the partials' (M, l), a few KB.  Every chain of loads costs about 1 us, so
// each is begun before the one it does not need: places from the lengths before the
// wait for the pieces, scores and partials before the maxima.  37 sequences of 4 cache
// heads, 8 partials a row: a CTA per 32 channels (4736 of them) took 15 us more than a
// warp per row with these loads (26 -> 11 us a call of one tile a warp).
constexpr int KV4_FINISH_THREADS = 256, KV4_FINISH_SLOTS = 4 * KV4_FINISH_THREADS;
constexpr int KV4_FINISH_WARPS = KV4_FINISH_THREADS / 32;
template <int D, int CTAS>
__global__ void __launch_bounds__(KV4_FINISH_THREADS)
    decode_kv4_finish_kernel(const __grid_constant__ DecKv4Params p, uint16_t* __restrict__ o, float* __restrict__ lse,
                             float* __restrict__ weights, int merge_blocks) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if ((int)blockIdx.x >= merge_blocks) {
    // ---- weights; a warp finds a head's log-sum-exp, 8 heads at a time
    __shared__ float s_lse2[KV4_FINISH_WARPS];
    const int per = (p.cap + KV4_FINISH_SLOTS - 1) / KV4_FINISH_SLOTS, at = blockIdx.x - merge_blocks;
    const int bhk = at / per, j = (at - bhk * per) * KV4_FINISH_SLOTS + 4 * tid;
    const int len = min(max(p.seqlens[bhk / p.Hkv], 0), p.cap);
    const bool any = j - 4 * tid < len;
    Kv4Parts parts = {0, 0};
    if (any && warp < p.group) parts = kv4_row_parts(p, bhk * p.group + warp);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!any) return;
    const float* x = p.x + (size_t)bhk * p.group * p.cap + j;
    float4* w4 = reinterpret_cast<float4*>(weights + (size_t)bhk * p.cap + j);  // j, capacity: multiples of 4
    float4 old = make_float4(0.f, 0.f, 0.f, 0.f), sum = old;
    if (j < len) old = *w4;
    float4 v[4];
    const auto load = [&](int h0) {
#pragma unroll
      for (int h = 0; h < 4; ++h)
        if (h0 + h < p.group && j < len) v[h] = *reinterpret_cast<const float4*>(x + (size_t)(h0 + h) * p.cap);
    };
    load(0);
    for (int h0 = 0; h0 < p.group; h0 += 4) {
      if (h0 % KV4_FINISH_WARPS == 0) {
        if (h0 > 0) {
          __syncthreads();
          if (h0 + warp < p.group) parts = kv4_row_parts(p, bhk * p.group + h0 + warp);
        }
        if (h0 + warp < p.group) {
          const float2 sum2 = kv4_row_sum(p, parts);
          if (lane == 0) s_lse2[warp] = kv4_lse2(sum2.x, sum2.y);
        }
        __syncthreads();
      }
#pragma unroll
      for (int h = 0; h < 4; ++h)
        if (h0 + h < p.group && j < len) {
          const float l2 = s_lse2[(h0 + h) % KV4_FINISH_WARPS];
          sum.x += ex2(v[h].x - l2), sum.y += ex2(v[h].y - l2), sum.z += ex2(v[h].z - l2), sum.w += ex2(v[h].w - l2);
        }
      load(h0 + 4);
    }
    old.x += sum.x, old.y += sum.y, old.z += sum.z, old.w += sum.w;
    if (j + 4 <= len) {
      *w4 = old;
    } else if (j < len) {
      float* w = reinterpret_cast<float*>(w4);
      w[0] = old.x;
      if (j + 1 < len) w[1] = old.y;
      if (j + 2 < len) w[2] = old.z;
    }
    return;
  }
  // ---- merge
  constexpr int LANES = CTAS > 1 ? 8 : D / 4;  // float4 of channels
  constexpr int GROUPS = (CTAS ? KV4_FINISH_THREADS : 32) / LANES, BATCH = 4;
  const int row = CTAS ? blockIdx.x / (CTAS ? CTAS : 1) : blockIdx.x * KV4_FINISH_WARPS + warp;
  const int first = CTAS > 1 ? blockIdx.x % (CTAS ? CTAS : 1) * 8 : 0;
  if (row >= p.B * p.Hkv * p.group) {
    asm volatile("griddepcontrol.wait;" ::: "memory");  // this grid never ends before the one it follows
    return;
  }
  const int lane4 = (CTAS ? tid : lane) % LANES, grp = (CTAS ? tid : lane) / LANES;
  uint2* out = reinterpret_cast<uint2*>(o + (size_t)row * D) + first + lane4;
  const Kv4Parts parts = kv4_row_parts(p, row);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (parts.n == 0) {
    if (grp == 0) *out = make_uint2(0, 0);
    if (grp == 0 && first + lane4 == 0) lse[row] = -INFINITY;
    return;
  }
  const float2* ml = p.ml_part + parts.first;
  const float4* op = reinterpret_cast<const float4*>(p.o_part + parts.first * D) + first + lane4;
  const int o_step = p.per_block * (D / 4);
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  float2 all = make_float2(0.f, 0.f);
  float inv = 0.f;
  for (int c0 = 0; c0 < parts.n; c0 += BATCH * GROUPS) {
    float2 v[BATCH];
    float4 w[BATCH];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int c = c0 + k * GROUPS + grp;
      if (c < parts.n) v[k] = ml[(size_t)c * p.per_block], w[k] = op[(size_t)c * o_step];
    }
    if (c0 == 0) {
      all = kv4_row_sum(p, parts);
      inv = 1.f / all.y;
    }
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      if (c0 + k * GROUPS + grp >= parts.n) break;
      const float f = kv4_part_factor(v[k].x, all.x) * v[k].y * inv;  // at most 1
      a.x = fmaf(f, w[k].x, a.x), a.y = fmaf(f, w[k].y, a.y), a.z = fmaf(f, w[k].z, a.z), a.w = fmaf(f, w[k].w, a.w);
    }
  }
#pragma unroll
  for (int k = LANES; k < 32; k <<= 1) {
    a.x += __shfl_xor_sync(0xffffffffu, a.x, k), a.y += __shfl_xor_sync(0xffffffffu, a.y, k);
    a.z += __shfl_xor_sync(0xffffffffu, a.z, k), a.w += __shfl_xor_sync(0xffffffffu, a.w, k);
  }
  if (CTAS) {
    __shared__ float4 s_o[KV4_FINISH_WARPS][LANES];
    if (lane < LANES) s_o[warp][lane] = a;
    __syncthreads();
    if (tid >= LANES) return;
    a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < KV4_FINISH_WARPS; ++k) {
      const float4 w = s_o[k][tid];
      a.x += w.x, a.y += w.y, a.z += w.z, a.w += w.w;
    }
  } else if (grp != 0) {
    return;
  }
  *out = make_uint2(pack_bf16(a.x, a.y), pack_bf16(a.z, a.w));
  if (first + lane4 == 0) lse[row] = kv4_lse2(all.x, all.y) * 0.69314718055994531f;
}

}  // namespace ta
