// Paged decode over the 8-bit cache (cache8.cuh): one new token a sequence.
//     s_t = scale * 2^ek_t * (q . kc_t),  O = sum_t softmax(s)_t 2^ev_t vc_t
// with kc, vc the codes of token t's key and value and ek, ev their exponents.
//
// Bound by the read of the cache.  The work is the tiles of 128 cached rows
// (16 tokens of 8 KV heads, or 128 / HB tokens of HB heads), in order of
// sequence, group of heads, position; every CTA takes an equal share of them,
// whatever the sequences' lengths (they are read and summed up on the device),
// so that all SMs finish together.  Where a share is many tiles, the begin of a
// sequence counts as up to 3 more: that is what it costs to write one result and
// set up the next (16 sequences of 4000 to 8200 tokens, 16 query heads a KV head of
// d = 128: 34.6 us without, 32.4 with it).  A run that covers the whole of a sequence's
// tiles writes its output; others write partial results, at most two a CTA,
// which decode8_merge_kernel joins.
//
// Few and short sequences go without the merge: a cluster of up to 8 CTAs has one
// sequence and KV head, and joins its results through its CTAs' shared memory
// (one sequence of 1000 tokens: 6.4 us against 8.1, and one launch less).
//
// A producer warp brings tiles into a ring (codes by TMA, scales by cp.async);
// each of the 8 consumer warps works on 16 of the tile's rows, 16 tokens of one
// KV head, for 8 NT of its query heads.  Both products run on mma.sync m16n8k16
// with the cache as the 16-row operand and the query heads as columns: S^T = K Q^T
// and O^T += V^T P^T.  There are a few FLOP per byte of cache, and a warp's operands
// go from its ring place to its registers and are converted there; a tcgen05 form
// would take 8-bit codes only against queries and weights of 8 bits, or as f16 that
// threads write back to shared or tensor memory first.  It has not been built.
//   - e4m3 codes become f16 exactly; q, scaled by a power of two of its row to
//     use f16's range, keeps its 8 bits (values 2^-28 below the row's largest
//     and less lose some).  The sum q . kc reaches 2^30 with q so scaled: times 2^ek
//     it would pass fp32's range long before the score does, so that factor is
//     2^(ek - b), and 2^b is in the other one, of scale and q's own power.  b is 22, or
//     less where the largest of the KV head's queries needs it; so nothing overflows on
//     the way to a score while scale max|q| max|k|, over a KV head's queries and its
//     rows, is below 2^127.
//   - V's scale goes into the weights before they are rounded:
//     p_t = 2^(s_t + ev_t - m), m a running bound of s_t + ev_t, so that no
//     weight overflows f16 however far apart the scales are; it is 2^8 off the
//     largest at most, and the stored weight has 11 bits down to 2^-20 of m.
//     The softmax's own sum takes 2^(s_t - n) in fp32, n a bound of s_t alone: m may
//     be 119 above the scores or 100 below, where a sum held against it would lose
//     its smaller terms or overflow.
//   - Both exponents come from one fma each.  Where n is far from 0 its rounding, and
//     that of m, would weigh more than the bf16 result's, and beyond 2^27 the fma's
//     unrounded product be far from n: there (above 2^9) scores are rounded first,
//     and m is taken as n + (m - n).
#pragma once

#include <cuda_fp16.h>

#include "cache8.cuh"
#include "decode_sm100.cuh"

namespace attn {

constexpr int kDecode8Parts = 8;                   // 16-row parts of a tile, a consumer warp each
constexpr int kDecode8RowsLog2 = 7;
constexpr int kDecode8Rows = 16 * kDecode8Parts;   // cached rows of a tile
static_assert(kDecode8Rows == 1 << kDecode8RowsLog2, "a tile is 8 warps of 16 rows");
constexpr int kDecode8MaxSeqs = 1024;              // sequences of one launch
constexpr float kDecode8PartScale = 0x1p-12f;      // of partial results: hundreds of the largest values still add up

struct Decode8Params {
  const __nv_bfloat16* q;      // [S, Hq, D]
  const int32_t* block_table;  // [S, max_pages]
  const int32_t* seq_lens;     // [S]
  __nv_bfloat16* o;            // [S, Hq, D]
  float* lse;                  // [S, Hq]
  const uint8_t* kv_scales;    // [num_pages, Hkv, page_size, 2]
  float* part_lse;             // workspace [2 ctas, HB * group], in log2
  float* part_o;               // workspace [2 ctas, HB * group, D]
  int S, Hq, Hkv, group, page_size, max_pages, num_pages, hb, hb_log2, ctas;
  int box;                     // tokens of one TMA box: 16 * 2^i, a divisor of page_size and of a tile's tokens
  uint32_t page_inverse;       // ceil(2^32 / (page_size / 16)); 0 for page_size = 16
  float scale_mantissa;        // scale * log2(e) = scale_mantissa * 2^scale_exp, 1 <= scale_mantissa <= 2
  int scale_exp;
};

template <int D, int STAGES>
struct Decode8Layout {
  static constexpr int kWarps = kDecode8Parts;            // consumers
  static constexpr int kThreads = 32 * (kWarps + 1);      // and the producer
  static constexpr int kPool = kDecode8Rows * D;          // codes of K (or V) of one tile
  static constexpr int kStage = 2 * kPool;
  static constexpr int kScales = STAGES * kStage;         // 32 bytes a warp and stage
  static constexpr int kBar = kScales + STAGES * 32 * kDecode8Parts;
  static constexpr int kWarpSums = kBar + 2 * STAGES * 8;
  static constexpr int kHeads = kWarpSums + 2 * kWarps * 4;   // of the warps: Decode8Heads [16 heads / 2], and Decode8Factors
  static constexpr int kJoin = kHeads + kWarps * (8 * 32 + 16);  // bounds and sums of the warps, [3][warp][16 heads]
  static constexpr int kTiles = kJoin + 3 * kWarps * 16 * 4;
  // Of a cluster's CTA instead: its share of the values of all CTAs' results (16
  // rows of D floats in all), and their LSEs [8][16].
  static constexpr int kOwn = kTiles, kOwnLse = kOwn + 16 * D * 4;
  static constexpr int kBytes = kTiles + (16 * D + 128 > kDecode8MaxSeqs + 1 ? 16 * D + 128 : kDecode8MaxSeqs + 1) * 4;
  static constexpr int kAlloc = kBytes + 1024;
};

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transposes an 8 x 8 matrix of 16-bit values held one row pair a lane.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Two e4m3 codes (the low or high half of w) as f16x2, exactly.
__device__ __forceinline__ uint32_t e4m3x2_f16x2_lo(uint32_t w) {
  uint32_t h;
  asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %1;\ncvt.rn.f16x2.e4m3x2 %0, a;\n}\n" : "=r"(h) : "r"(w));
  return h;
}
__device__ __forceinline__ uint32_t e4m3x2_f16x2_hi(uint32_t w) {
  uint32_t h;
  asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %1;\ncvt.rn.f16x2.e4m3x2 %0, b;\n}\n" : "=r"(h) : "r"(w));
  return h;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ uint4 lds_128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ uint32_t lds_u16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
  return v;
}

// Byte offset of 16-byte vector `c` of row `r` in a warp's 16 x D tile, as TMA
// swizzles it: 128-byte rows XOR the vector with r % 8, 64-byte rows with
// (r / 2) % 4.
template <int D>
__device__ __forceinline__ uint32_t decode8_offset(int r, int c) {
  return D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

template <int THREADS>
__device__ __forceinline__ void decode8_consumers_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
}

// Two 16 x 16 byte matrices (rows at the addresses of lanes 0-15 and 16-31),
// transposed: a lane holds bytes of column lane / 4 (r0, r2) and lane / 4 + 8
// (r1, r3), rows 4 (lane % 4) .. + 3.
__device__ __forceinline__ void ldmatrix_b8_trans(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr)
               : "memory");
}

// Token of the 16 in row r of the first product.  The second takes its tokens
// in the order in which ldmatrix hands out bytes: lane tig has tokens 4 tig ..
// + 3, as columns 2 tig, 2 tig + 1, 2 tig + 8, 2 tig + 9.
__device__ __forceinline__ int decode8_token(int r) { return 4 * ((r & 7) >> 1) + 2 * (r >> 3) + (r & 1); }

// Tiles (or chunks) of 2^log2 tokens that a length takes; no sum that could pass 2^31.
__device__ __forceinline__ int decode8_count(int len, int log2) { return (len >> log2) + ((len & ((1 << log2) - 1)) != 0); }

// Units of work: a sequence's tiles and, before them, `extra` for its begin.  CTA
// c of n takes total / n units, and one more if c < total % n.
struct Decode8Share {
  int extra, groups, ctas, each, more;
  Decode8Share() = default;
  // tiles, sequences: of one head group, all and those with tokens.
  __device__ __forceinline__ Decode8Share(int tiles, int sequences, int groups, int most) : groups(groups) {
    ctas = min(most, tiles * groups);
    extra = ctas > 0 ? min(3, tiles * groups / (8 * ctas)) : 0;
    const int total = units(tiles, sequences) * groups;
    each = ctas > 0 ? total / ctas : 0;
    more = total - each * ctas;
  }
  __device__ __forceinline__ int units(int tiles, int sequences) const { return tiles + extra * sequences; }
  __device__ __forceinline__ int begin(int c) const { return c * each + min(c, more); }
  __device__ __forceinline__ int owner(int unit) const {
    const int cut = more * (each + 1);
    return unit < cut ? unit / (each + 1) : more + (unit - cut) / each;
  }
};

// The tiles [from, to) of sequence s and head group hg, out of n (none if a share
// ends in the units of its begin), and the unit behind them.
struct Decode8Run {
  int s, hg, from, to, n, next;
};

// The run that begins at unit `at` of all, cut at `end`.  first: the units of one
// head group before each sequence.
__device__ __forceinline__ Decode8Run decode8_run(const int32_t* first, int S, const Decode8Share& share, int at, int end) {
  int lo = 0, hi = S;  // the last sequence that begins at or before unit `at`: it is not empty, since at < total
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] * share.groups <= at) lo = mid; else hi = mid;
  }
  Decode8Run r;
  r.s = lo;
  const int before = first[lo], units = first[lo + 1] - before;
  int in = at - before * share.groups;
  r.hg = 0;
  if (share.groups > 1) {
    r.hg = in / units;
    in -= r.hg * units;
  }
  const int to = min(units, in + (end - at));
  r.next = at + to - in;
  r.n = units - share.extra;
  r.from = max(in - share.extra, 0);
  r.to = max(to - share.extra, 0);
  return r;
}

// The cluster's barrier: every thread arrives and waits in turn.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// `addr` of this CTA's shared memory in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_map(uint32_t addr, int rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  return a;
}

__device__ __forceinline__ void cluster_store(uint32_t addr, float x) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(x) : "memory");
}

__device__ __forceinline__ void cluster_store4(uint32_t addr, const float (&x)[4]) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]) : "memory");
}

// The largest x of the warp's rows.
__device__ __forceinline__ float decode8_top(float x) {
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
  return x;
}

// Of two heads, 2 tig (low) and 2 tig + 1 (high): the scores' factor, minus the
// weights' bound m, minus the sum's bound n, and m - n.
struct alignas(16) Decode8Heads {
  uint64_t f, nm, nn, d;
};
// Of the run: 2^-b, and the V exponent (+ 6) below which the bounds have to be looked at.
struct alignas(8) Decode8Factors {
  float kb, v_low;
};

// One tile for one warp.
template <int D, int NT>
struct Decode8Warp {
  float acc[NT][D / 16][4];  // O^T: values 16 c + grp (0, 1) and + 8 (2, 3) of heads 2 tig (+ 1)
  uint64_t l[NT];            // this lane's share of the sums of heads 2 tig and 2 tig + 1
  uint32_t q[NT][D / 16][2];
  // Where registers are short the heads' values are in shared memory, a place for
  // each pair: loads cost less than what is spilled otherwise (64 sequences, d = 128:
  // 99.5 us against 102.1; 3 x 131072 tokens, two head tiles, d = 64: 29.5 against 34.0).
  static constexpr bool kShared = NT == 2 || D == 128;
  Decode8Heads* shared;
  Decode8Heads own[kShared ? 1 : NT];
  Decode8Factors* shared_factors;
  Decode8Factors own_factors;

  __device__ __forceinline__ Decode8Heads heads(int nt) const {
    if constexpr (kShared) return shared[4 * nt];
    else return own[nt];
  }
  // By the whole warp, all lanes of a pair alike; __syncwarp() before they are read.
  __device__ __forceinline__ void set_heads(int nt, const Decode8Heads& h, int grp) {
    if constexpr (!kShared) own[nt] = h;
    else if (grp == 0) shared[4 * nt] = h;
  }
  __device__ __forceinline__ Decode8Factors factors() const { return kShared ? *shared_factors : own_factors; }
  __device__ __forceinline__ void set_factors(const Decode8Factors& f, int lane) {
    if constexpr (!kShared) own_factors = f;
    else if (lane == 0) *shared_factors = f;
  }

  __device__ __forceinline__ void begin(const __nv_bfloat16* qrow, int group, float scale_mantissa, int scale_exp, int grp, int tig,
                                        uint8_t* heads_at) {
    shared = reinterpret_cast<Decode8Heads*>(heads_at) + tig;
    shared_factors = reinterpret_cast<Decode8Factors*>(heads_at + 8 * 32);
    int shifts[NT], least = 126;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int h = nt * 8 + grp;
      uint2 raw[D / 16];
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        // Step i of the product takes values 4 (i % 4) .. + 3 of 16-byte vector
        // (D / 64) tig + i / 4 of a key row: the same values of q.
        const int c = (D / 64) * tig + i / 4;
        raw[i] = make_uint2(0u, 0u);
        if (h < group) raw[i] = *reinterpret_cast<const uint2*>(qrow + h * D + 16 * c + 4 * (i % 4));
        amax = fmaxf(amax, fmaxf(fmaxf(fabsf(__uint_as_float(raw[i].x << 16)), fabsf(__uint_as_float(raw[i].x & 0xffff0000u))),
                                 fmaxf(fabsf(__uint_as_float(raw[i].y << 16)), fabsf(__uint_as_float(raw[i].y & 0xffff0000u)))));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // Largest magnitude to 2^13 .. 2^14, as far as 2^shift and scale 2^(22 - shift)
      // are normal floats (what smaller queries lose, 2^-25 of q so scaled, moves a
      // score by less than 2^-16 scale under the largest keys).
      int shift = 13 - (static_cast<int>(__float_as_uint(amax) >> 23) - 127);
      shift = amax > 3.4e38f ? 0 : min(amax == 0.f ? 126 : shift, min(126, scale_exp + 148));
      shifts[nt] = shift;
      least = min(least, shift);
      const float up = __int_as_float((shift + 127) << 23);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        q[nt][i][0] = pack_f16x2(__uint_as_float(raw[i].x << 16) * up, __uint_as_float(raw[i].x & 0xffff0000u) * up);
        q[nt][i][1] = pack_f16x2(__uint_as_float(raw[i].y << 16) * up, __uint_as_float(raw[i].y & 0xffff0000u) * up);
      }
      l[nt] = 0;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) acc[nt][c][0] = acc[nt][c][1] = acc[nt][c][2] = acc[nt][c][3] = 0.f;
    }
    // scale 2^(b - shift) < 2^127 for all heads.
    const int b = min(22, 126 - scale_exp + __reduce_min_sync(0xffffffffu, least));
    const uint64_t none = f2_pack(INFINITY, INFINITY);
    set_factors({__int_as_float((127 - b) << 23), -INFINITY}, 4 * grp + tig);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int e = scale_exp + b - shifts[nt], half = e >> 1;  // in two steps: 2^e may be out of range
      const float factor =  // of head grp; wanted: of heads 2 tig (+ 1)
          scale_mantissa * __int_as_float((127 + half) << 23) * __int_as_float((127 + e - half) << 23);
      set_heads(nt, {f2_pack(__shfl_sync(0xffffffffu, factor, 8 * tig), __shfl_sync(0xffffffffu, factor, 8 * tig + 4)), none, none, 0}, grp);
    }
    __syncwarp();
  }

  // valid: the tokens of the 16 that belong to the sequence (TAIL: fewer than 16).
  template <bool TAIL>
  __device__ __forceinline__ void tile(uint32_t k, uint32_t v, uint32_t scales, int valid, int lane) {
    const int grp = lane >> 2, tig = lane & 3;
    const int t0 = decode8_token(grp), t1 = t0 + 2;  // tokens of rows grp and grp + 8
    float sc[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
      const int c = (D / 64) * tig + j;
      const uint4 ka = lds_128(k + decode8_offset<D>(t0, c)), kb = lds_128(k + decode8_offset<D>(t1, c));
      const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t a0 = e4m3x2_f16x2_lo(wa[i]), a1 = e4m3x2_f16x2_lo(wb[i]);
        const uint32_t a2 = e4m3x2_f16x2_hi(wa[i]), a3 = e4m3x2_f16x2_hi(wb[i]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_f16_16816(sc[nt], a0, a1, a2, a3, q[nt][4 * j + i][0], q[nt][4 * j + i][1]);
      }
    }
    if (TAIL && valid < 16) {
      // Tokens past the end may hold NaN codes, and 0 * NaN is NaN: their
      // values are cleared (their scores below).
      for (int i = lane; i < (16 - valid) * (D / 16); i += 32)
        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(v + decode8_offset<D>(valid + i / (D / 16), i % (D / 16))),
                     "r"(0u)
                     : "memory");
      fence_proxy_async_smem();  // before the copies that will refill this place
      __syncwarp();
    }
    const uint32_t e0 = lds_u16(scales + 2 * t0), e1 = lds_u16(scales + 2 * t1);
    // K's scales times 2^-b, and V's exponents + 6 as floats (a byte in the last bits of 2^23).
    const Decode8Factors of_run = factors();
    const float k0 = cache8_scale(e0 & 255u) * of_run.kb, k1 = cache8_scale(e1 & 255u) * of_run.kb;
    const float v0 = __uint_as_float(0x4b000000u | e0 >> 8) - 8388729.f, v1 = __uint_as_float(0x4b000000u | e1 >> 8) - 8388729.f;
    const uint64_t k00 = f2_pack(k0, k0), k11 = f2_pack(k1, k1), v00 = f2_pack(v0, v0), v11 = f2_pack(v1, v1);
    uint64_t x[NT][2];  // scores of rows grp and grp + 8 but for f
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      x[nt][0] = f2_mul(f2_pack(sc[nt][0], sc[nt][1]), k00);
      x[nt][1] = f2_mul(f2_pack(sc[nt][2], sc[nt][3]), k11);
    }
    // Past the end -inf: a select, since what the slots there hold, their scales too,
    // may be NaN.
    auto within = [&](float (&out)[4]) {
      if (TAIL) {
#pragma unroll
        for (int e = 0; e < 4; ++e) out[e] = (e < 2 ? t0 : t1) < valid ? out[e] : -INFINITY;
      }
    };
    auto scores = [&](int nt, uint64_t f, uint64_t add0, uint64_t add1, float (&out)[4]) {
      f2_unpack(f2_fma(x[nt][0], f, add0), out[0], out[1]);
      f2_unpack(f2_fma(x[nt][1], f, add1), out[2], out[3]);
      within(out);
    };
    uint32_t p[NT][2];
    // From the log2 of the weights, 2^6 up, and of the sum's terms.
    auto weigh = [&](int nt, float (&w)[4], float (&s)[4]) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        w[e] = ex2_approx(w[e]);
        s[e] = ex2_approx(s[e]);
      }
      l[nt] = f2_add(l[nt], f2_add(f2_pack(s[0], s[1]), f2_pack(s[2], s[3])));
      p[nt][0] = movmatrix_trans(pack_f16x2(w[0], w[1]));
      p[nt][1] = movmatrix_trans(pack_f16x2(w[2], w[3]));
    };
    float w[NT][4];
    float top = -INFINITY;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const Decode8Heads h = heads(nt);
      scores(nt, h.f, f2_add(v00, h.nm), f2_add(v11, h.nm), w[nt]);
      top = max3(top, max3(w[nt][0], w[nt][1], w[nt][2]), w[nt][3]);
    }
    if (!__any_sync(0xffffffffu, top > 14.f || fminf(v0, v1) < of_run.v_low)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const Decode8Heads h = heads(nt);
        float s[4];
        scores(nt, h.f, h.nn, h.nn, s);
        weigh(nt, w[nt], s);
      }
    } else {
      // A weight more than 2^8 off its bound (or none yet), or a value so much smaller
      // than the largest that set a bound that a score may be far above n although its
      // weight is not above m: new bounds, the largest so far.  So a score is 105 above
      // n at most (8 - ev above m, and m that largest exponent above n), and 2^22 terms
      // of it still add up.  Once n or m is far from 0 every tile comes here.
      float far = 0.f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const Decode8Heads h = heads(nt);
        float s[4], n[2], d[2], b[2];
        f2_unpack(f2_mul(x[nt][0], h.f), s[0], s[1]);
        f2_unpack(f2_mul(x[nt][1], h.f), s[2], s[3]);
        within(s);
        f2_unpack(h.nn, n[0], n[1]);
        f2_unpack(h.d, d[0], d[1]);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float old = -n[u];
          n[u] = fmaxf(old, decode8_top(fmaxf(s[u], s[u + 2])));
          s[u] -= n[u];
          s[u + 2] -= n[u];
          b[u] = ex2_approx(old - n[u]);
          const float before = d[u] + (old - n[u]);  // the old m, seen from the new n
          w[nt][u] = s[u] + v0;
          w[nt][u + 2] = s[u + 2] + v1;
          d[u] = fmaxf(before, decode8_top(fmaxf(w[nt][u], w[nt][u + 2])) - 6.f);
          w[nt][u] -= d[u];
          w[nt][u + 2] -= d[u];
          const float a = ex2_approx(before - d[u]);
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            acc[nt][c][u] *= a;
            acc[nt][c][u + 2] *= a;
          }
          far = max3(far, fabsf(n[u]), fabsf(n[u] + d[u]));
        }
        l[nt] = f2_mul(l[nt], f2_pack(b[0], b[1]));
        __syncwarp();  // all lanes have read what is replaced
        set_heads(nt, {h.f, f2_pack(-n[0] - d[0], -n[1] - d[1]), f2_pack(-n[0], -n[1]), f2_pack(d[0], d[1])}, grp);
        weigh(nt, w[nt], s);
      }
      const float v = decode8_top(fmaxf(v0, v1)) - 97.f;
      set_factors({of_run.kb, __any_sync(0xffffffffu, far > 512.f) ? INFINITY : fmaxf(of_run.v_low, v)}, lane);
      __syncwarp();
    }
#pragma unroll
    for (int c = 0; c < D / 16; c += 2) {
      uint32_t r[4];  // of vectors c (r[0], r[1]) and c + 1: 4 tokens' codes of values lane / 4 and lane / 4 + 8
      ldmatrix_b8_trans(v + decode8_offset<D>(lane & 15, c + (lane >> 4)), r[0], r[1], r[2], r[3]);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t a0 = e4m3x2_f16x2_lo(r[2 * u]), a1 = e4m3x2_f16x2_lo(r[2 * u + 1]);
        const uint32_t a2 = e4m3x2_f16x2_hi(r[2 * u]), a3 = e4m3x2_f16x2_hi(r[2 * u + 1]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_f16_16816(acc[nt][c + u], a0, a1, a2, a3, p[nt][0], p[nt][1]);
      }
    }
  }
};

// NT tiles of 8 query heads a KV head.  PER_SM: CTAs an SM.  CLUSTER: p.ctas CTAs,
// a cluster, share the tiles of one sequence and KV head (hb = 1); else p.ctas
// share all there are.
template <int D, int NT, int PER_SM, int STAGES, bool CLUSTER>
__global__ void __launch_bounds__(Decode8Layout<D, STAGES>::kThreads, PER_SM)
    decode8_split_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                         const Decode8Params p) {
  using L = Decode8Layout<D, STAGES>;
  constexpr int kDecode8Warps = L::kWarps;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  auto full_bar = [&](int st) -> uint32_t { return base + L::kBar + 8u * st; };
  auto empty_bar = [&](int st) -> uint32_t { return base + L::kBar + 8u * (STAGES + st); };
  int32_t* first = reinterpret_cast<int32_t*>(smem + L::kTiles);
  int32_t* warp_sums = reinterpret_cast<int32_t*>(smem + L::kWarpSums);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tokens_log2 = kDecode8RowsLog2 - p.hb_log2, tokens = 1 << tokens_log2;  // of a tile

  if constexpr (CLUSTER) cluster_arrive();  // waited for before the first store to another CTA: it has begun by then
  if (threadIdx.x == 0) {
    for (int st = 0; st < STAGES; ++st) {
      mbar_init(full_bar(st), 1);
      mbar_init(empty_bar(st), kDecode8Warps);
    }
    fence_mbar_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  griddep_wait();  // what the call reads and writes: only behind the kernels before it
  // From here on the merge may be launched (it reads the lengths, then waits for
  // this grid): not earlier, so that what it reads is behind those kernels too.
  griddep_launch();

  int begin = 0, end = 0;
  Decode8Share share;
  Decode8Run mine;  // of a cluster's CTA
  int rank = 0, active = 0;
  if constexpr (CLUSTER) {
    const int index = blockIdx.x / p.ctas;
    rank = blockIdx.x - index * p.ctas;
    mine.s = index / p.Hkv;
    mine.hg = index - mine.s * p.Hkv;
    const int len = p.seq_lens[mine.s];
    const size_t head = static_cast<size_t>(mine.s) * p.Hq + mine.hg * p.group;
    if (len <= 0 || len > p.max_pages * p.page_size) {
      if (rank == 0) {
        if (threadIdx.x == 0 && mine.hg == 0 && len != 0) atomicOr(&g_attn_device_error, kErrCache8Table);
        for (int i = threadIdx.x; i < p.group * (D / 8); i += L::kThreads)
          reinterpret_cast<uint4*>(p.o + head * D)[i] = make_uint4(0u, 0u, 0u, 0u);
        for (int i = threadIdx.x; i < p.group; i += L::kThreads) p.lse[head + i] = -INFINITY;
      }
      return;  // all of the cluster
    }
    mine.n = decode8_count(len, tokens_log2);
    active = min(p.ctas, mine.n);
    const int each = mine.n / active, more = mine.n - each * active;
    mine.from = min(rank, active) * each + min(rank, more);
    mine.to = mine.from + (rank < active ? each + (rank < more) : 0);
    mine.next = end = 1;
    __syncthreads();  // the barriers are set up
  }

  if constexpr (!CLUSTER) {
    // Units before each sequence: every consumer thread sums up tiles and
    // sequences of a run of lengths, the warps' sums follow.
    const int per = (p.S + 32 * kDecode8Warps - 1) / (32 * kDecode8Warps);
    int tiles = 0, count = 0;  // of this thread's run; then of all before it
    if (warp < kDecode8Warps) {
      for (int i = 0; i < per; ++i) {
        const int s = threadIdx.x * per + i;
        if (s >= p.S) break;
        int len = p.seq_lens[s];
        if (len < 0 || len > p.max_pages * p.page_size) {
          if (blockIdx.x == 0) atomicOr(&g_attn_device_error, kErrCache8Table);
          len = 0;
        }
        first[s + 1] = decode8_count(len, tokens_log2);
        tiles += first[s + 1];
        count += len > 0;
      }
      const int own_tiles = tiles, own_count = count;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, tiles, off), y = __shfl_up_sync(0xffffffffu, count, off);
        if (lane >= off) {
          tiles += x;
          count += y;
        }
      }
      if (lane == 31) {
        warp_sums[warp] = tiles;
        warp_sums[kDecode8Warps + warp] = count;
      }
      tiles -= own_tiles;
      count -= own_count;
    }
    if (threadIdx.x == 0) first[0] = 0;
    __syncthreads();
    int all_tiles = 0, all_count = 0;
#pragma unroll
    for (int w = 0; w < kDecode8Warps; ++w) {
      if (w == warp) {
        tiles += all_tiles;
        count += all_count;
      }
      all_tiles += warp_sums[w];
      all_count += warp_sums[kDecode8Warps + w];
    }
    share = Decode8Share(all_tiles, all_count, p.Hkv >> p.hb_log2, p.ctas);
    if (warp < kDecode8Warps) {
      for (int i = 0; i < per; ++i) {
        const int s = threadIdx.x * per + i;
        if (s >= p.S) break;
        tiles += first[s + 1];
        count += first[s + 1] > 0;
        first[s + 1] = share.units(tiles, count);
      }
    }
    __syncthreads();
    if (static_cast<int>(blockIdx.x) >= share.ctas) return;
    begin = share.begin(blockIdx.x);
    end = share.begin(blockIdx.x + 1);
  }
  auto run_at = [&](int at) {
    if constexpr (CLUSTER) return mine;
    else return decode8_run(first, p.S, share, at, end);
  };

  if (warp == kDecode8Warps) {
    // ------------------------------------------------------------ producer
    const int chunks_per_tile = kDecode8Parts >> p.hb_log2;  // chunks of 16 tokens
    const int chunks_per_box = p.box / 16;
    const uint32_t box_bytes = p.hb * p.box * D;
    // Scales go by cp.async, 16 bytes a lane (a tensor copy of so few bytes
    // costs the copy engine as much as one of 16 KB): lanes 2 w and 2 w + 1
    // bring those of consumer w.
    const int w_hl = (lane >> 1) & (p.hb - 1), w_chunk = lane >> (1 + p.hb_log2);
    bool ok = true;
    int count = 0, st = 0;  // tiles issued, and the next one's place in the ring
    uint32_t phase = 1;     // of the empty barriers: the ring's first round finds every place free
    const int page_chunks = p.page_size / 16;
    for (int at = begin; at < end && ok;) {
      const Decode8Run run = run_at(at);
      at = run.next;
      if (run.from == run.to) continue;
      const int len = p.seq_lens[run.s];
      const int chunk_end = min(decode8_count(len, 4), run.to * chunks_per_tile);
      const int32_t* table = p.block_table + static_cast<size_t>(run.s) * p.max_pages;
      const int head = run.hg * p.hb;
      // Where 32 chunks lie, one a lane (page << 4 | chunk of the page); the
      // next 32 are under way while these are used.  The division by the
      // page's chunks is a product with its inverse, exact below 2^28 chunks.
      int window = run.from * chunks_per_tile;
      auto fetch = [&](int c) -> uint32_t {
        if (c >= chunk_end) return 0u;
        const int i = p.page_inverse ? static_cast<int>(__umulhi(c, p.page_inverse)) : c;
        const uint32_t page = static_cast<uint32_t>(table[i]);
        if (page < static_cast<uint32_t>(p.num_pages)) return page << 4 | static_cast<uint32_t>(c - i * page_chunks);
        atomicOr(&g_attn_device_error, kErrCache8Table);
        return 0u;  // keeps every copy inside the pool; the result is flagged
      };
      uint32_t here = fetch(window + lane), next = fetch(window + 32 + lane);
      for (int tile = run.from; tile < run.to; ++tile) {
        const int c0 = tile * chunks_per_tile;
        if (c0 >= window + 32) {
          window += 32;
          here = next;
          next = fetch(window + 32 + lane);
        }
        const uint32_t of_scale = __shfl_sync(0xffffffffu, here, c0 - window + w_chunk);
        const uint32_t of_box = __shfl_sync(0xffffffffu, here, c0 - window + lane * chunks_per_box);
        const int n = min(chunks_per_tile, chunk_end - c0), boxes = chunks_per_box == 1 ? n : (n + chunks_per_box - 1) / chunks_per_box;
        ok = mbar_wait(empty_bar(st), phase, kErrCache8Wait);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane < 2 * kDecode8Parts && w_chunk < n) {
          const size_t row = (static_cast<size_t>(of_scale >> 4) * p.Hkv + head + w_hl) * p.page_size + (of_scale & 15u) * 16;
          cp_async_16(base + L::kScales + (st * 2 * kDecode8Parts + lane) * 16, p.kv_scales + row * 2 + (lane & 1) * 16, 16);
        }
        cp_async_mbar_arrive(full_bar(st));  // holds the phase open until the lane's copies have landed
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(full_bar(st), 2 * boxes * box_bytes);
        __syncwarp();
        if (lane < boxes) {
          const uint32_t dst = base + st * L::kStage + lane * box_bytes;
          const int row = static_cast<int>((of_box >> 4) * p.page_size + (of_box & 15u) * 16);
          tma_load_3d(dst, &tm_k, full_bar(st), 0, row, head);
          tma_load_3d(dst + L::kPool, &tm_v, full_bar(st), 0, row, head);
        }
        ++count;
        if (++st == STAGES) {
          st = 0;
          phase ^= 1u;
        }
      }
      // The consumers write the run's result through NT places of the ring.
      for (int i = 0; i < NT && ok; ++i) {
        ok = __all_sync(0xffffffffu, mbar_wait(empty_bar(st), phase, kErrCache8Wait));
        if (!ok) break;
        if (lane == 0) mbar_arrive(full_bar(st));
        ++count;
        if (++st == STAGES) {
          st = 0;
          phase ^= 1u;
        }
      }
    }
    // No copy may be in flight when the CTA ends.
    for (int c = max(0, count - STAGES); c < count; ++c)
      mbar_wait(full_bar(c % STAGES), static_cast<uint32_t>(c / STAGES) & 1u, kErrCache8Wait);
    __syncwarp();
    if constexpr (CLUSTER) {
      cluster_wait();
      cluster_arrive();
    }
    return;
  }

  // -------------------------------------------------------------- consumers
  const int grp = lane >> 2, tig = lane & 3;
  const int hl = warp & (p.hb - 1), chunk = warp >> p.hb_log2, parts = kDecode8Parts >> p.hb_log2;
  const int chunks_per_box = p.box / 16;
  const uint32_t rows_at = ((chunk / chunks_per_box * p.hb + hl) * chunks_per_box + chunk % chunks_per_box) * 16 * D;
  float* join = reinterpret_cast<float*>(smem + L::kJoin);  // [3][warp][16 heads]: m - n, later factors; sums; n
  int st = 0;          // place in the ring, and phase of its full barriers
  uint32_t phase = 0;
  bool ok = true;  // false once a wait ran out (recorded): no more waits, and every barrier below is still met
  for (int at = begin; at < end;) {
    const Decode8Run run = run_at(at);
    at = run.next;
    if (run.from == run.to) continue;
    const int len = p.seq_lens[run.s];
    Decode8Warp<D, NT> w;
    w.begin(p.q + (static_cast<size_t>(run.s) * p.Hq + (run.hg * p.hb + hl) * p.group) * D, p.group, p.scale_mantissa, p.scale_exp,
            grp, tig, smem + L::kHeads + warp * (8 * 32 + 16));
    for (int tile = run.from; tile < run.to; ++tile) {
      if (ok) ok = mbar_wait(full_bar(st), phase, kErrCache8Wait);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) continue;
      const uint32_t k = base + st * L::kStage + rows_at, sc = base + L::kScales + (st * kDecode8Parts + warp) * 32;
      const int valid = len - tile * tokens - chunk * 16;
      // Two head tiles have a path without the selects; one loses by the code's size
      // (64 sequences: 100.6 us against 99.5; 16 of 4000 tokens: 33.9 against 32.4).
      if (NT == 2 && valid >= 16)
        w.template tile<false>(k, k + L::kPool, sc, 16, lane);
      else if (valid > 0)
        w.template tile<true>(k, k + L::kPool, sc, valid, lane);
      __syncwarp();
      if (lane == 0) mbar_arrive(empty_bar(st));
      if (++st == STAGES) {
        st = 0;
        phase ^= 1u;
      }
    }
    // The run's result.  Bounds, sums and O^T go to shared memory (O^T to the
    // ring's next NT places), one thread a head works out what each of the
    // head's warps counts, and all threads add up and write O, 8 values at a
    // time.
    float minus_n[NT][2], m_n[NT][2], sum[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const Decode8Heads h = w.heads(nt);
      f2_unpack(h.nn, minus_n[nt][0], minus_n[nt][1]);
      f2_unpack(h.d, m_n[nt][0], m_n[nt][1]);
      f2_unpack(w.l[nt], sum[nt][0], sum[nt][1]);
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) sum[nt][u] += __shfl_xor_sync(0xffffffffu, sum[nt][u], off);
    }
    uint32_t place[NT];
    decode8_consumers_sync<32 * kDecode8Warps>();  // the last run's factors have been read
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (ok) ok = mbar_wait(full_bar(st), phase, kErrCache8Wait);
      place[nt] = st;
      if (++st == STAGES) {
        st = 0;
        phase ^= 1u;
      }
      float* out = reinterpret_cast<float*>(smem + place[nt] * L::kStage) + warp * (D / 4) * 32;
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int k = 4 * c + e;  // rows of 32 lanes; lane ^ k keeps the readers below off one bank
          out[k * 32 + (lane ^ k)] = w.acc[nt][c][e];
        }
      if (grp == 0) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int at = warp * 16 + nt * 8 + 2 * tig + u;
          join[at] = m_n[nt][u];
          join[kDecode8Warps * 16 + at] = sum[nt][u];
          join[2 * kDecode8Warps * 16 + at] = -minus_n[nt][u];
        }
      }
    }
    ok = __all_sync(0xffffffffu, ok);
    decode8_consumers_sync<32 * kDecode8Warps>();
    const bool whole = run.from == 0 && run.to == run.n;
    const size_t row0 = (2 * static_cast<size_t>(blockIdx.x) + (run.from == 0 ? 1 : 0)) * p.hb * p.group;
    const size_t head0 = static_cast<size_t>(run.s) * p.Hq + static_cast<size_t>(run.hg) * p.hb * p.group;
    const int heads = p.hb * p.group;  // rows of the result
    // A thread a head and warp that holds tokens of it: 8 times the group in all.
    if (warp * 4 < p.group) {
      const bool on = static_cast<int>(threadIdx.x) < 8 * p.group;  // the others of the last warp repeat its last
      const int index = min(static_cast<int>(threadIdx.x), 8 * p.group - 1);
      const int part = index & (parts - 1), row = index >> (3 - p.hb_log2);
      const int g = row / p.group, mine_at = (part * p.hb + g) * 16 + row - g * p.group;
      const float d = join[mine_at], n = join[2 * kDecode8Warps * 16 + mine_at];
      float mx = n;
#pragma unroll
      for (int off = 1; off < 8; off <<= 1)
        if (off < parts) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
      float sum = join[kDecode8Warps * 16 + mine_at] * ex2_approx(n - mx);
#pragma unroll
      for (int off = 1; off < 8; off <<= 1)
        if (off < parts) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      __syncwarp();
      // O = sum over the warps of acc * 2^(m - mx - 6) / sum
      if (on) join[mine_at] = ex2_approx(n - mx + d - 6.f) / sum * (!CLUSTER && whole ? 1.f : kDecode8PartScale);
      const float lse2 = mx + log2f(sum);
      if constexpr (CLUSTER) {
        cluster_wait();  // (these warps here, the others below)
        // Every CTA of the cluster gets this one's: threads 8 a head, a CTA each.
        if (on && part < p.ctas) cluster_store(cluster_map(base + L::kOwnLse + (rank * 16 + row) * 4, part), lse2);
      } else if (on && part == 0) {
        if (whole)
          p.lse[head0 + row] = lse2 * 0.69314718055994530942f;
        else
          p.part_lse[row0 + row] = lse2;
      }
    } else if constexpr (CLUSTER) {
      cluster_wait();
    }
    decode8_consumers_sync<32 * kDecode8Warps>();
    // Values of a thread at a time: 4 in a cluster, whose CTAs have few heads, else 8.
    constexpr int kValues = CLUSTER ? 4 : 8;
    for (int i = threadIdx.x; i < heads * (D / kValues); i += 32 * kDecode8Warps) {
      const int row = i / (D / kValues), set = i % (D / kValues);
      const int g = row / p.group, h = row - g * p.group;
      const int k = 2 * (set * kValues / 8) + (h & 1), t = (CLUSTER ? 16 * (set & 1) : 0) + ((h & 7) >> 1);
      const float* src = reinterpret_cast<const float*>(smem + (NT == 1 || h < 8 ? place[0] : place[NT - 1]) * L::kStage);
      float x[kValues];
#pragma unroll
      for (int u = 0; u < kValues; ++u) x[u] = 0.f;
#pragma unroll 2
      for (int part = 0; part < parts; ++part) {
        const int from = part * p.hb + g;
        const float a = join[from * 16 + h];
#pragma unroll
        for (int u = 0; u < kValues; ++u) x[u] = fmaf(a, src[(from * (D / 4) + k) * 32 + ((4 * u + t) ^ k)], x[u]);
      }
      if constexpr (CLUSTER) {
        // To the CTA that has this share of the values.
        const int slot = (rank * 16 + row) * (D / 4 / p.ctas) + set / p.ctas;
        cluster_store4(cluster_map(base + L::kOwn + slot * 16, set % p.ctas), x);
      } else if (whole) {
        *reinterpret_cast<uint4*>(p.o + (head0 + row) * D + 8 * set) = pack_bf16x8(x);
      } else {
        float4* dst = reinterpret_cast<float4*>(p.part_o + (row0 + row) * D + 8 * set);
        dst[0] = make_float4(x[0], x[1], x[2], x[3]);
        dst[1] = make_float4(x[4], x[5], x[6], x[7]);
      }
    }
    fence_proxy_async_smem();  // before the copies that will refill these places
    __syncwarp();
    if (lane == 0) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mbar_arrive(empty_bar(place[nt]));
    }
  }
  if constexpr (CLUSTER) {
    // All results of the cluster for this CTA's share of the values are joined.
    __syncwarp();
    if (mine.from == mine.to) cluster_wait();  // (a CTA without tiles has not met the barrier's first round yet)
    cluster_arrive();
    cluster_wait();
    const size_t head = static_cast<size_t>(mine.s) * p.Hq + mine.hg * p.group;
    const int quads = D / 4 / p.ctas;
    for (int i = threadIdx.x; i < p.group * quads; i += 32 * kDecode8Warps) {
      const int row = i / quads, slot = i - row * quads;
      const float4* own = reinterpret_cast<const float4*>(smem + L::kOwn) + row * quads + slot;
      const float* own_lse = reinterpret_cast<const float*>(smem + L::kOwnLse) + row;
      float l[8], top = -INFINITY, sum = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
      float4 a[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const bool there = c < active;
        l[c] = there ? own_lse[c * 16] : -INFINITY;
        a[c] = there ? own[c * 16 * quads] : make_float4(0.f, 0.f, 0.f, 0.f);
        top = fmaxf(top, l[c]);
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float w = ex2_approx(l[c] - top);
        sum += w;
        x[0] = fmaf(w, a[c].x, x[0]);
        x[1] = fmaf(w, a[c].y, x[1]);
        x[2] = fmaf(w, a[c].z, x[2]);
        x[3] = fmaf(w, a[c].w, x[3]);
      }
      const float inv = 1.f / (kDecode8PartScale * sum);
      *reinterpret_cast<uint2*>(p.o + (head + row) * D + 4 * (slot * p.ctas + rank)) =
          make_uint2(pack_bf16x2(x[0] * inv, x[1] * inv), pack_bf16x2(x[2] * inv, x[3] * inv));
      if (slot == 0 && rank == 0) p.lse[head + row] = (top + log2f(sum)) * 0.69314718055994530942f;
    }
  }
}

// Joins the partial results of the heads of a sequence:
//     lse = log sum_i exp(lse_i),  O = sum_i exp(lse_i - lse) O_i.
// Which CTAs of the split pass hold them follows from the lengths, summed up as
// there; that part needs nothing of the split pass and runs before the wait for
// it.  Heads that one CTA held alone are written already.  PER warps share a
// head's partial rows, four or eight of each in flight at a time with their LSEs,
// so that the join costs one or two trips to memory (launch_decode8 chooses PER);
// the warps are added in their order.
constexpr int kMerge8Warps = 16;

template <int D, int PER>
__global__ void __launch_bounds__(32 * kMerge8Warps) decode8_merge_kernel(const Decode8Params p) {
  griddep_launch();  // all of this grid's CTAs are on the SMs by then: the next call may set itself up beside them
  constexpr int kPer = D / 32, kHeads = kMerge8Warps / PER;
  __shared__ float rows[PER > 1 ? kMerge8Warps : 1][D], bound[kMerge8Warps], sums[kMerge8Warps];
  __shared__ int sums_of[4][kMerge8Warps];
  const int s = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tokens_log2 = kDecode8RowsLog2 - p.hb_log2, most = p.max_pages * p.page_size;
  auto tiles_of = [&](int i) {
    const int len = p.seq_lens[i];
    return len < 0 || len > most ? 0 : decode8_count(len, tokens_log2);
  };
  // Tiles and sequences with tokens: of the sequences before s, of all.
  int x[4] = {0, 0, 0, 0};
  for (int i = threadIdx.x; i < p.S; i += 32 * kMerge8Warps) {
    const int n = tiles_of(i);
    x[2] += n;
    x[3] += n > 0;
    if (i < s) {
      x[0] += n;
      x[1] += n > 0;
    }
  }
  const int n = tiles_of(s);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x[i] += __shfl_xor_sync(0xffffffffu, x[i], off);
    if (lane == 0) sums_of[i][warp] = x[i];
    x[i] = 0;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kMerge8Warps; ++w)
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] += sums_of[i][w];
  const int h = blockIdx.x * kHeads + warp / PER, part = warp % PER;
  const bool on = h < p.Hq;
  const size_t head = static_cast<size_t>(s) * p.Hq + h;
  int pieces = 0;
  size_t slot0 = 0;
  const int hk = h / p.group, per_slot = p.hb * p.group, row0 = (hk & (p.hb - 1)) * p.group + h % p.group;
  if (n > 0) {
    const Decode8Share share(x[2], x[3], p.Hkv >> p.hb_log2, p.ctas);
    const int at = share.units(x[0], x[1]) * share.groups + (hk >> p.hb_log2) * share.units(n, 1) + share.extra;
    const int c0 = share.owner(at), c1 = share.owner(at + n - 1);
    pieces = on ? c1 - c0 + 1 : 0;
    slot0 = 2 * static_cast<size_t>(c0);
  }
  griddep_wait();
  if (n == 0) {  // no tokens (or a length that the split pass reported)
    if (on && part == 0) {
      if (lane < D / 8) reinterpret_cast<uint4*>(p.o + head * D)[lane] = make_uint4(0u, 0u, 0u, 0u);
      if (lane == 0) p.lse[head] = -INFINITY;
    }
    return;
  }
  if (PER == 1 && pieces <= 1) return;
  // The first piece ends its CTA (slot 1), the others begin theirs (slot 0).
  auto row_of = [&](int i) { return (slot0 + 2 * i + (i == 0 ? 1 : 0)) * per_slot + row0; };
  constexpr int kFlight = PER == 16 ? 8 : 4;
  float mx = -INFINITY, sum = 0.f, out[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) out[e] = 0.f;
  if (pieces > 1) {
    for (int i0 = part; i0 < pieces; i0 += PER * kFlight) {
      float l[kFlight], x[kFlight][kPer];
#pragma unroll
      for (int u = 0; u < kFlight; ++u) {
        const int i = i0 + u * PER;
        l[u] = -INFINITY;
#pragma unroll
        for (int e = 0; e < kPer; ++e) x[u][e] = 0.f;
        if (i < pieces) {
          const size_t row = row_of(i);
          l[u] = p.part_lse[row];
          const float* src = p.part_o + row * D + lane * kPer;
          if constexpr (kPer == 4) {
            const float4 y = *reinterpret_cast<const float4*>(src);
            x[u][0] = y.x; x[u][1] = y.y; x[u][2] = y.z; x[u][3] = y.w;
          } else {
            const float2 y = *reinterpret_cast<const float2*>(src);
            x[u][0] = y.x; x[u][1] = y.y;
          }
        }
      }
      float top = mx;
#pragma unroll
      for (int u = 0; u < kFlight; ++u) top = fmaxf(top, l[u]);
      const float a = ex2_approx(mx - top);  // 0 the first time: there is a row, so top is above -inf (or all is NaN)
      mx = top;
      sum *= a;
#pragma unroll
      for (int e = 0; e < kPer; ++e) out[e] *= a;
#pragma unroll
      for (int u = 0; u < kFlight; ++u) {
        const float w = ex2_approx(l[u] - mx);
        sum += w;
#pragma unroll
        for (int e = 0; e < kPer; ++e) out[e] = fmaf(w, x[u][e], out[e]);
      }
    }
  }
  if constexpr (PER > 1) {
#pragma unroll
    for (int e = 0; e < kPer; ++e) rows[warp][lane * kPer + e] = out[e];
    if (lane == 0) {
      bound[warp] = mx;
      sums[warp] = sum;
    }
    __syncthreads();
    if (part != 0 || pieces <= 1) return;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < PER; ++w) top = fmaxf(top, bound[warp + w]);
    sum = 0.f;
#pragma unroll
    for (int e = 0; e < kPer; ++e) out[e] = 0.f;
#pragma unroll
    for (int w = 0; w < PER; ++w) {
      const float a = ex2_approx(bound[warp + w] - top);  // 0 for a warp without rows
      sum = fmaf(a, sums[warp + w], sum);
#pragma unroll
      for (int e = 0; e < kPer; ++e) out[e] = fmaf(a, rows[warp + w][lane * kPer + e], out[e]);
    }
    mx = top;
  }
  const float inv = 1.f / (kDecode8PartScale * sum);
#pragma unroll
  for (int e = 0; e < kPer; e += 2)
    *reinterpret_cast<uint32_t*>(p.o + head * D + lane * kPer + e) = pack_bf16x2(out[e] * inv, out[e + 1] * inv);
  if (lane == 0) p.lse[head] = (mx + log2f(sum)) * 0.69314718055994530942f;
}

}  // namespace attn
