// A paged KV cache in 8 bits: quantising new keys and values as they are
// written, and reading the cache back.
//
// The pools hold e4m3 codes [num_pages, page_size, Hkv, D].  Each row of D
// values (one token, one KV head) has one power-of-two scale 2^e, kept as a
// byte e + 127 in kv_scales [num_pages, Hkv, page_size, 2] (the key's, then
// the value's):
//     e = the smallest exponent with max|x| <= 448 * 2^e, in [-100, 119]
//     code = e4m3(x * 2^-e), to nearest even, saturating; the value is code * 2^e.
// e4m3 is a floating format, so a scale that is not a power of two would round
// no better; this one is a single byte, its multiplication is exact, and every
// value of the cache is exact in bf16 (4 significant bits).  The limits keep
// 2^e and 2^-e normal floats and the largest value, 448 * 2^119, finite; only
// rows below 2^-91 lose bits to the lower one.
#pragma once

#include "ptx.cuh"
#include "rope.cuh"

namespace attn {

enum : unsigned int {
  kErrCache8Table = 1u << 14,  // 8-bit cache: a length or block-table entry out of range
  kErrCache8Wait = 1u << 15,   // 8-bit decode: a pipeline wait ran out
};

constexpr int kCache8MinExp = -100, kCache8MaxExp = 119;

// The exponent of a row whose largest magnitude is amax (448 = 1.75 * 2^8).
__device__ __forceinline__ int cache8_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = static_cast<int>(u >> 23) - 127 - ((u & 0x7fffffu) <= 0x600000u ? 8 : 7);
  return min(max(e, kCache8MinExp), kCache8MaxExp);
}

// 2^e for the exponents above and their opposites.
__device__ __forceinline__ float cache8_pow2(int e) { return __int_as_float((e + 127) << 23); }

// The sequence that packed row t belongs to: the last s with cu[s] <= t.  All
// lanes of the warp call it with the same t; 32 candidates a round, so that a
// thousand sequences take two trips to memory.
__device__ __forceinline__ int warp_find_sequence(const int32_t* cu, int num_seqs, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = num_seqs;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int s = lo + lane * step;
    const int below = __popc(__ballot_sync(0xffffffffu, s < hi && cu[s] <= t));
    lo += max(below - 1, 0) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

struct Append8Params {
  const __nv_bfloat16* q;      // [total_q, Hq, D] (with positions only)
  const __nv_bfloat16* k_new;  // [total_q, Hkv, D]
  const __nv_bfloat16* v_new;
  __nv_bfloat16* q_out;
  uint8_t* k_pool;             // [num_pages, page_size, Hkv, D] e4m3
  uint8_t* v_pool;
  uint8_t* kv_scales;          // [num_pages, Hkv, page_size, 2] e8m0
  const int32_t* positions;    // [axes, total_q]
  const int32_t* cu_q;         // [num_seqs + 1]
  const int32_t* seq_lens;     // [num_seqs], after the append
  const int32_t* block_table;  // [num_seqs, max_pages]
  int num_seqs, total_q, Hq, Hkv, page_size, max_pages, num_pages;
  int tokens_log2;             // of a block
  int one_wave;                // all blocks are on the SMs at once
};

// Largest magnitude of a row that LANES lanes hold, 16 values each (NaN aside).
template <int LANES>
__device__ __forceinline__ float row_amax(const float (&x)[8], const float (&y)[8]) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fmaxf(fabsf(x[i]), fabsf(y[i])));
#pragma unroll
  for (int off = LANES / 2; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
  return amax;
}

__device__ __forceinline__ uint2 cache8_codes(const float (&x)[8], float m) {
  return make_uint2(pack_e4m3x4(x[0] * m, x[1] * m, x[2] * m, x[3] * m), pack_e4m3x4(x[4] * m, x[5] * m, x[6] * m, x[7] * m));
}

constexpr int kAppend8Threads = 128;
constexpr int kAppend8Heads = 1;  // passes of an item

// Items of a warp: a token and kAppend8Heads passes over its KV heads, keys and
// values; D / 16 lanes a row as in rope_kernel.  All of an item's rows are
// requested before its place in the cache is looked up.
template <int D>
__global__ void __launch_bounds__(kAppend8Threads) append8_kernel(const Append8Params p) {
  constexpr int kLanes = D / 16, kRows = 32 / kLanes;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int groups = (p.Hkv + kRows * kAppend8Heads - 1) / (kRows * kAppend8Heads);
  const long long items = static_cast<long long>(p.total_q) * groups;
  const int off = 8 * (lane % kLanes);  // 8 values there and 8 at D / 2 behind: whole lines a pass
  if (p.one_wave) griddep_launch();
  griddep_wait();
  int s = -1, q0 = 0, q1 = 0, len = 0;  // the sequence of the last item, often this one's too
  for (long long item = static_cast<long long>(blockIdx.x) * (kAppend8Threads / 32) + warp; item < items;
       item += static_cast<long long>(gridDim.x) * (kAppend8Threads / 32)) {
    const int t = static_cast<int>(item / groups), group = static_cast<int>(item - static_cast<long long>(t) * groups);
    const int h0 = lane / kLanes + group * kRows * kAppend8Heads;
    uint4 v[kAppend8Heads][2][2];  // [pass][key, value][8 values]
#pragma unroll
    for (int u = 0; u < kAppend8Heads; ++u) {
      const int h = h0 + u * kRows;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const __nv_bfloat16* src = (kv == 0 ? p.k_new : p.v_new) + (static_cast<size_t>(t) * p.Hkv + h) * D + off;
        v[u][kv][0] = v[u][kv][1] = make_uint4(0u, 0u, 0u, 0u);
        if (h < p.Hkv) {
          v[u][kv][0] = reinterpret_cast<const uint4*>(src)[0];
          v[u][kv][1] = reinterpret_cast<const uint4*>(src)[D / 16];
        }
      }
    }
    if (s < 0 || t < q0 || t >= q1) {
      s = warp_find_sequence(p.cu_q, p.num_seqs, t);
      q0 = p.cu_q[s];
      q1 = p.cu_q[s + 1];
      len = p.seq_lens[s];
    }
    if (t >= q1) continue;  // padding behind the last sequence
    int page = -1, slot = 0;
    if (t >= q0 && q1 - q0 <= len && len <= p.max_pages * p.page_size) {
      const int pos = len - (q1 - t);
      const int i = pos / p.page_size;
      page = p.block_table[static_cast<size_t>(s) * p.max_pages + i];
      slot = pos - i * p.page_size;
    }
    if (page < 0 || page >= p.num_pages) {
      if (lane == 0) atomicOr(&g_attn_device_error, kErrCache8Table);
      continue;
    }
    const size_t at = (static_cast<size_t>(page) * p.page_size + slot) * p.Hkv;
#pragma unroll
    for (int u = 0; u < kAppend8Heads; ++u) {
      const int h = h0 + u * kRows;
      uint32_t scales = 0;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        float x[8], y[8];
        unpack_bf16x8(v[u][kv][0], x);
        unpack_bf16x8(v[u][kv][1], y);
        const int e = cache8_exponent(row_amax<kLanes>(x, y));
        scales |= static_cast<uint32_t>(e + 127) << (8 * kv);
        if (h < p.Hkv) {
          const float m = cache8_pow2(-e);
          uint2* dst = reinterpret_cast<uint2*>((kv == 0 ? p.k_pool : p.v_pool) + (at + h) * D + off);
          dst[0] = cache8_codes(x, m);
          dst[D / 16] = cache8_codes(y, m);
        }
      }
      if (h < p.Hkv && lane % kLanes == 0)
        *reinterpret_cast<uint16_t*>(p.kv_scales + ((static_cast<size_t>(page) * p.Hkv + h) * p.page_size + slot) * 2) =
            static_cast<uint16_t>(scales);
    }
  }
}

// A block's tokens, threads and angles are those of rope_kernel.  A row's largest
// magnitude is a reduction over its D / 16 lanes; a thread takes a head's key and
// value, so that both scales go in one store.  k is quantised from the 32-bit
// result of the rotation (one rounding, not two).
template <int D>
__global__ void __launch_bounds__(kRowThreads, 2) rope_append8_kernel(const __grid_constant__ RopeTable table, const Append8Params p) {
  using R = RowShape<D>;
  __shared__ __align__(16) float2 angles[kRowTokens][kRopeMaxHalf];
  __shared__ int pages[kRowTokens], slots[kRowTokens];  // page: -1 for a token that is left out
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int step = R::kSlots >> p.tokens_log2;  // heads at a time
  const int first = static_cast<int>(blockIdx.x) << p.tokens_log2;
  const int tokens = min(1 << p.tokens_log2, p.total_q - first);
  const int slot = threadIdx.x / R::kLanes;
  const int tok = slot / step, h0 = slot % step;
  const RopeLane rl = rope_lane(threadIdx.x % R::kLanes, table.half, table.adjacent);
  const bool in = tok < tokens;
  const size_t t = static_cast<size_t>(first) + tok;
  if (p.one_wave) griddep_launch();
  griddep_wait();
  uint4 v[2][kRowBatch][2];
  rows_load(v[0], p.q + t * p.Hq * D, D, h0, step, in ? p.Hq : 0, rl);
  rope_angles(table, p.positions + first, p.total_q, tokens, 1.f, angles);
  // Where each token goes, a warp a token.
  for (int i = warp; i < tokens; i += kRowThreads / 32) {
    const int row = first + i, s = warp_find_sequence(p.cu_q, p.num_seqs, row);
    const int q0 = p.cu_q[s], q1 = p.cu_q[s + 1], len = p.seq_lens[s];
    int page = -1;
    if (row < q1) {  // else padding behind the last sequence
      if (row >= q0 && q1 - q0 <= len && len <= p.max_pages * p.page_size) {
        const int pos = len - (q1 - row), at = pos / p.page_size;
        page = p.block_table[static_cast<size_t>(s) * p.max_pages + at];
        if (lane == 0) slots[i] = pos - at * p.page_size;
      }
      if (page < 0 || page >= p.num_pages) {
        if (lane == 0) atomicOr(&g_attn_device_error, kErrCache8Table);
        page = -1;
      }
    }
    if (lane == 0) pages[i] = page;
  }
  __syncthreads();
  const int page = in ? pages[tok] : -1, at_slot = page >= 0 ? slots[tok] : 0;
  const bool on = page >= 0;
  const int hq = on ? p.Hq : 0, hk = on ? p.Hkv : 0;
  float2 cs[8];
  const int more = kRowBatch * step;
  rope_take(angles[tok], rl, cs);
  const __nv_bfloat16* q = p.q + t * p.Hq * D;
  __nv_bfloat16* q_out = p.q_out + t * p.Hq * D;
  for (int h = h0; h < hq; h += 2 * more) {
    rows_load(v[1], q, D, h + more, step, hq, rl);
    rows_turn(v[0], q_out, D, h, step, hq, rl, cs, table.adjacent);
    rows_load(v[0], q, D, h + 2 * more, step, hq, rl);
    rows_turn(v[1], q_out, D, h + more, step, hq, rl, cs, table.adjacent);
  }
  // Keys and values: all lanes of a warp go round together (the reductions).
  const size_t row0 = (static_cast<size_t>(max(page, 0)) * p.page_size + at_slot) * p.Hkv;
  for (int h1 = 0; h1 < p.Hkv; h1 += more) {
    const int hb = h1 + h0;
    rows_load(v[0], p.k_new + t * p.Hkv * D, D, hb, step, hk, rl);
    rows_load(v[1], p.v_new + t * p.Hkv * D, D, hb, step, hk, rl);
#pragma unroll
    for (int u = 0; u < kRowBatch; ++u) {
      if (h1 + u * step >= p.Hkv) break;
      const int h = hb + u * step;
      uint32_t scales = 0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x[8], y[8];
        unpack_bf16x8(v[i][u][0], x);
        unpack_bf16x8(v[i][u][1], y);
        if (i == 0 && rl.turns) rope_turn(x, y, cs, table.adjacent);
        const int e = cache8_exponent(row_amax<R::kLanes>(x, y));
        const float m = cache8_pow2(-e);
        scales |= static_cast<uint32_t>(e + 127) << (8 * i);
        if (h >= hk) continue;
        uint8_t* dst = (i == 0 ? p.k_pool : p.v_pool) + (row0 + h) * D;
        *reinterpret_cast<uint2*>(dst + rl.off0) = cache8_codes(x, m);
        *reinterpret_cast<uint2*>(dst + rl.off1) = cache8_codes(y, m);
      }
      if (h < hk && threadIdx.x % R::kLanes == 0)
        *reinterpret_cast<uint16_t*>(p.kv_scales + ((static_cast<size_t>(page) * p.Hkv + h) * p.page_size + at_slot) * 2) =
            static_cast<uint16_t>(scales);
    }
  }
}

struct Gather8Params {
  const uint8_t* k_pool;
  const uint8_t* v_pool;
  const uint8_t* kv_scales;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* cu_k;         // [num_seqs + 1]: rows of the output
  __nv_bfloat16* k_out;        // [total_rows, Hkv, D]
  __nv_bfloat16* v_out;
  int num_seqs, total_rows, Hkv, page_size, max_pages, num_pages;
};

constexpr int kGather8Threads = 128;

// Two e4m3 codes (in the low half of a word) times 2^e as a pair of bf16 (exact;
// NaN codes stay NaN).
__device__ __forceinline__ uint32_t cache8_bf16x2(uint32_t codes16, float two_e) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(codes16)));
  float lo, hi;
  asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %2;\ncvt.f32.f16 %0, a;\ncvt.f32.f16 %1, b;\n}\n" : "=f"(lo), "=f"(hi) : "r"(h));
  return pack_bf16x2(lo * two_e, hi * two_e);
}

// 16 codes as bf16 in one 32-byte store.
__device__ __forceinline__ void cache8_store16(__nv_bfloat16* dst, const uint4& c, float e) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(cache8_bf16x2(c.x, e)),
               "r"(cache8_bf16x2(c.x >> 16, e)), "r"(cache8_bf16x2(c.y, e)), "r"(cache8_bf16x2(c.y >> 16, e)),
               "r"(cache8_bf16x2(c.z, e)), "r"(cache8_bf16x2(c.z >> 16, e)), "r"(cache8_bf16x2(c.w, e)),
               "r"(cache8_bf16x2(c.w >> 16, e))
               : "memory");
}

// The scale byte as a float.  0 and 255 are never written (e is limited), but
// a slot that no token was written to may hold them: such a row's values mean
// nothing, and 2^-127 or infinity serve as well as any.
__device__ __forceinline__ float cache8_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// One warp a row of the output (one token): 16 codes a lane, of keys and values,
// and kGather8Batch of each under way.
constexpr int kGather8Batch = 2;

template <int D>
__global__ void __launch_bounds__(kGather8Threads) gather8_kernel(const Gather8Params p) {
  // In warps, unsigned: threads would pass 32 bits at 2^27 rows.
  const unsigned warp = blockIdx.x * (kGather8Threads / 32) + (threadIdx.x >> 5);
  // Tokens that have no row have no warp that looks at them: the last block does.
  if (blockIdx.x == gridDim.x - 1) {
    for (int i = threadIdx.x; i < p.num_seqs; i += kGather8Threads) {
      const int n = p.seq_lens[i], first = p.cu_k[i];
      if ((n != 0 && p.cu_k[i + 1] <= first) || (n > 0 && first > p.total_rows - n)) atomicOr(&g_attn_device_error, kErrCache8Table);
    }
  }
  if (warp >= static_cast<unsigned>(p.total_rows)) return;
  const int row = static_cast<int>(warp);
  const int lane = threadIdx.x & 31;
  const int s = warp_find_sequence(p.cu_k, p.num_seqs, row);
  const int r0 = p.cu_k[s], r1 = p.cu_k[s + 1], len = p.seq_lens[s];
  if (row >= r1) return;  // behind the last sequence
  const int t = row - r0;
  if (t < 0 || len < 0 || len > p.max_pages * p.page_size || len > r1 - r0) {
    if (lane == 0) atomicOr(&g_attn_device_error, kErrCache8Table);
    return;
  }
  if (t >= len) return;  // room behind a sequence: left as it was
  const int page = p.block_table[static_cast<size_t>(s) * p.max_pages + t / p.page_size];
  const int slot = t % p.page_size;
  if (page < 0 || page >= p.num_pages) {
    if (lane == 0) atomicOr(&g_attn_device_error, kErrCache8Table);
    return;
  }
  const size_t src = (static_cast<size_t>(page) * p.page_size + slot) * p.Hkv * D;
  const size_t dst = static_cast<size_t>(row) * p.Hkv * D;
  const uint8_t* scales = p.kv_scales + (static_cast<size_t>(page) * p.Hkv * p.page_size + slot) * 2;
  for (int i0 = lane * 16; i0 < p.Hkv * D; i0 += 512 * kGather8Batch) {
    uint4 k[kGather8Batch], v[kGather8Batch];
    uint32_t e[kGather8Batch];
#pragma unroll
    for (int u = 0; u < kGather8Batch; ++u) {
      const int i = i0 + 512 * u;
      if (i < p.Hkv * D) {
        k[u] = *reinterpret_cast<const uint4*>(p.k_pool + src + i);
        v[u] = *reinterpret_cast<const uint4*>(p.v_pool + src + i);
        e[u] = *reinterpret_cast<const uint16_t*>(scales + static_cast<size_t>(i / D) * p.page_size * 2);
      }
    }
#pragma unroll
    for (int u = 0; u < kGather8Batch; ++u) {
      const int i = i0 + 512 * u;
      if (i < p.Hkv * D) {
        cache8_store16(p.k_out + dst + i, k[u], cache8_scale(e[u] & 255u));
        cache8_store16(p.v_out + dst + i, v[u], cache8_scale(e[u] >> 8));
      }
    }
  }
}

}  // namespace attn
