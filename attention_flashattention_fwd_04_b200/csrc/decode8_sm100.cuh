// Paged decode over the 8-bit cache (cache8.cuh): one new token a sequence,
// split over the cache's length and joined by decode_merge_kernel.
//     s_t = scale * 2^ek_t * (q . kc_t),  O = sum_t softmax(s)_t 2^ev_t vc_t
// with kc, vc the codes of token t's key and value and ek, ev their exponents.
#pragma once

#include "cache8.cuh"
#include "decode_sm100.cuh"

namespace attn {

struct Decode8Params {
  DecodeParams d;
  const uint8_t* k_pool;
  const uint8_t* v_pool;
  const uint8_t* kv_scales;
};

constexpr int kDecode8Threads = 128;

// CTA (split, sequence, query head): each warp takes every fourth token of the
// split with its own running maximum and sum; the four are joined at the end.
template <int D>
__global__ void __launch_bounds__(kDecode8Threads) decode8_split_kernel(const Decode8Params p) {
  constexpr int kPer = D / 32;
  constexpr int kWarps = kDecode8Threads / 32;
  __shared__ float so[kWarps][D], sm[kWarps], sl[kWarps];
  const DecodeParams& d = p.d;
  const int split = blockIdx.x, s = blockIdx.y, h = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int seq_len = d.seq_lens[s];
  if (seq_len < 0 || seq_len > d.max_pages * d.page_size) {
    if (split == 0 && h == 0 && threadIdx.x == 0) atomicOr(&g_attn_device_error, kErrCache8Table);
    return;
  }
  const int begin = split * d.split_tokens, end = min(seq_len, begin + d.split_tokens);
  if (begin >= end) return;
  const int hk = h / d.group;
  float q[kPer], o[kPer], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    q[i] = __bfloat162float(d.q[(static_cast<size_t>(s) * d.Hq + h) * D + lane * kPer + i]) * d.scale_log2;
    o[i] = 0.f;
  }
  for (int t = begin + warp; t < end; t += kWarps) {
    int page = d.block_table[static_cast<size_t>(s) * d.max_pages + t / d.page_size];
    if (page < 0 || page >= d.num_pages) {
      if (lane == 0) atomicOr(&g_attn_device_error, kErrCache8Table);
      page = 0;
    }
    const int slot = t % d.page_size;
    const size_t at = ((static_cast<size_t>(page) * d.page_size + slot) * d.Hkv + hk) * D + lane * kPer;
    const uint8_t* e = p.kv_scales + ((static_cast<size_t>(page) * d.Hkv + hk) * d.page_size + slot) * 2;
    const float ke = cache8_scale(e[0]), ve = cache8_scale(e[1]);
    float dot = 0.f;
    float v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; i += 2) {
      uint32_t kc = cache8_bf16x2(*reinterpret_cast<const uint16_t*>(p.k_pool + at + i), 1.f);
      uint32_t vc = cache8_bf16x2(*reinterpret_cast<const uint16_t*>(p.v_pool + at + i), 1.f);
      dot += q[i] * __uint_as_float(kc << 16) + q[i + 1] * __uint_as_float(kc & 0xffff0000u);
      v[i] = __uint_as_float(vc << 16) * ve;
      v[i + 1] = __uint_as_float(vc & 0xffff0000u) * ve;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
    dot *= ke;
    const float mn = fmaxf(m, dot);
    const float a = exp2f(m - mn), w = exp2f(dot - mn);
    m = mn;
    l = l * a + w;
#pragma unroll
    for (int i = 0; i < kPer; ++i) o[i] = o[i] * a + w * v[i];
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) so[warp][lane * kPer + i] = o[i];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  __syncthreads();
  float mx = sm[0];
  for (int w = 1; w < kWarps; ++w) mx = fmaxf(mx, sm[w]);
  float total = 0.f;
  for (int w = 0; w < kWarps; ++w) total += sl[w] * exp2f(sm[w] - mx);
  const size_t row = (static_cast<size_t>(s) * d.Hq + h) * d.max_splits + split;
  for (int i = threadIdx.x; i < D; i += kDecode8Threads) {
    float sum = 0.f;
    for (int w = 0; w < kWarps; ++w) sum += so[w][i] * exp2f(sm[w] - mx);
    d.part_o[row * D + i] = sum / total;
  }
  if (threadIdx.x == 0) d.part_lse[row] = (mx + log2f(total)) * 0.69314718055994530942f;
}

}  // namespace attn
