// Rotary positions with several axes (time, height, width, ...).
//
// Frequency j of a head's first R values belongs to one axis a(j), and a token
// at positions p turns the pair (x, y) of that frequency by the angle
// p[a(j)] * inv_freq[j]:
//     (x, y) -> (x cos - y sin, y cos + x sin).
// The pair is (j, j + R/2), or the adjacent (2j, 2j + 1).  The gradient of the
// rotation is the rotation by the opposite angle.
//
// Angles are kept in turns, as 64-bit fractions: the position times
// inv_freq / 2 pi modulo one turn is one integer product, exact for every
// 32-bit position, where a product in 32-bit floats is off by a whole radian
// near position 2^24.
#pragma once

#include "ptx.cuh"

namespace attn {

constexpr int kRopeMaxHalf = 64;  // frequencies: d <= 128

struct RopeTable {
  uint64_t turn[kRopeMaxHalf];  // inv_freq / 2 pi modulo 1, in units of 2^-64
  uint8_t axis[kRopeMaxHalf];
  int half;                     // R / 2, a multiple of 8
  int adjacent;
};

// cos and sin of `position` times frequency `turn`.  The signed 64-bit
// fraction is split into a 24-bit float and the rest, which is added back to
// first order: the result is good to the last bit or so of a float.
__device__ __forceinline__ float2 rope_cos_sin(int position, uint64_t turn) {
  const uint64_t t = static_cast<uint64_t>(static_cast<int64_t>(position)) * turn;
  const int hi = static_cast<int>(t >> 32);
  const float f = __int2float_rn(hi);
  const float rest = static_cast<float>(hi - __float2int_rn(f)) + __uint2float_rn(static_cast<uint32_t>(t)) * 0x1p-32f;
  float s, c;
  sincospif(f * 0x1p-31f, &s, &c);
  const float delta = rest * (6.2831853071795865f * 0x1p-32f);
  return make_float2(fmaf(-s, delta, c), fmaf(c, delta, s));
}

// A row of D values is held by D / 16 lanes, 16 values a lane, as two vectors
// of 8 at off0 and off1 such that both halves of every pair are in one lane.
struct RopeLane {
  int off0, off1;
  int freq;   // first of the lane's 8 frequencies
  bool turns; // false: values behind R, which pass through
};

__device__ __forceinline__ RopeLane rope_lane(int l, int half, bool adjacent) {
  RopeLane r;
  r.freq = 8 * l;
  r.turns = r.freq < half;
  if (adjacent || !r.turns) {
    // Behind R both pairings go on in order: lane half / 8 begins at 2 * half.
    r.off0 = 16 * l;
    r.off1 = 16 * l + 8;
  } else {
    r.off0 = 8 * l;
    r.off1 = half + 8 * l;
  }
  return r;
}

__device__ __forceinline__ void unpack_bf16x8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack_bf16x8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

// Turns a lane's 16 values (a at off0, b at off1) by its 8 angles.
__device__ __forceinline__ void rope_turn(float (&a)[8], float (&b)[8], const float2 (&cs)[8], bool adjacent) {
  if (adjacent) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = a[2 * i], y = a[2 * i + 1], z = b[2 * i], w = b[2 * i + 1];
      a[2 * i] = x * cs[i].x - y * cs[i].y;
      a[2 * i + 1] = y * cs[i].x + x * cs[i].y;
      b[2 * i] = z * cs[4 + i].x - w * cs[4 + i].y;
      b[2 * i + 1] = w * cs[4 + i].x + z * cs[4 + i].y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = a[i], y = b[i];
      a[i] = x * cs[i].x - y * cs[i].y;
      b[i] = y * cs[i].x + x * cs[i].y;
    }
  }
}

// Queries or keys [B, H, N, D] with their strides in elements.
struct RopeTensor {
  const __nv_bfloat16* x;
  __nv_bfloat16* out;
  long long b, h, n;      // strides of x
  long long ob, oh, on;   // strides of out
  int H;
};

struct RopeParams {
  RopeTensor q, k;        // k.H = 0: no keys
  const int32_t* positions;  // [axes, B, N]
  int B, N;
  float sign;             // -1: the gradient
};

// Kernels that turn rows work in items, a warp each: a token and up to
// kRopeRows passes over its heads, 32 / (D / 16) rows a pass.  All of an item's
// rows are requested first; its angles are worked out while they are under way,
// each once, by one lane, and handed round in shared memory.
constexpr int kRopeThreads = 128;
constexpr int kRopeRows = 4;

// A lane's frequencies in a warp: `lane`, and `lane` + 32 where there are so many.
struct RopeFreq {
  uint64_t turn[2];
  int axis[2];
};

__device__ __forceinline__ RopeFreq rope_freq(const RopeTable& table, int lane) {
  RopeFreq f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    f.turn[i] = table.turn[lane + 32 * i];
    f.axis[i] = table.axis[lane + 32 * i];
  }
  return f;
}

// cos and sin of a token's angles, to `cs` (shared memory of the warp).
template <int D>
__device__ __forceinline__ void rope_angles(const RopeFreq& f, const int32_t* positions, long long axis_stride, int half, float sign,
                                            float2* cs, int lane) {
  int pos[D / 64];
#pragma unroll
  for (int i = 0; i < D / 64; ++i) pos[i] = lane + 32 * i < half ? positions[f.axis[i] * axis_stride] : 0;
  __syncwarp();  // the last item's have been read
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    if (lane + 32 * i < half) {
      float2 v = rope_cos_sin(pos[i], f.turn[i]);
      v.y *= sign;
      cs[lane + 32 * i] = v;
    }
  }
  __syncwarp();
}

// The lane's 8 angles.
__device__ __forceinline__ void rope_take(const float2* cs, const RopeLane& rl, float2 (&out)[8]) {
  if (!rl.turns) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = reinterpret_cast<const float4*>(cs + rl.freq)[i];
    out[2 * i] = make_float2(v.x, v.y);
    out[2 * i + 1] = make_float2(v.z, v.w);
  }
}

// Items: (token, group of kRopeRows * 32 / (D / 16) heads, queries then keys).
template <int D>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeTable table, const RopeParams p) {
  constexpr int kLanes = D / 16, kRows = 32 / kLanes;
  __shared__ __align__(16) float2 angles[kRopeThreads / 32][kRopeMaxHalf];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rows = p.q.H + p.k.H, groups = (rows + kRows * kRopeRows - 1) / (kRows * kRopeRows);
  const long long tokens = static_cast<long long>(p.B) * p.N, items = tokens * groups;
  const RopeLane rl = rope_lane(lane % kLanes, table.half, table.adjacent);
  const RopeFreq freq = rope_freq(table, lane);
  for (long long item = static_cast<long long>(blockIdx.x) * (kRopeThreads / 32) + warp; item < items;
       item += static_cast<long long>(gridDim.x) * (kRopeThreads / 32)) {
    const long long token = item / groups;
    const int r0 = static_cast<int>(item - token * groups) * kRows * kRopeRows + lane / kLanes;
    const int b = static_cast<int>(token / p.N), n = static_cast<int>(token - static_cast<long long>(b) * p.N);
    uint4 v[kRopeRows][2];
    __nv_bfloat16* dst[kRopeRows];
#pragma unroll
    for (int u = 0; u < kRopeRows; ++u) {
      const int r = r0 + u * kRows;
      const bool is_q = r < p.q.H;
      const RopeTensor& t = is_q ? p.q : p.k;
      const int h = is_q ? r : r - p.q.H;
      dst[u] = r < rows ? t.out + b * t.ob + h * t.oh + n * t.on : nullptr;
      if (r < rows) {
        const __nv_bfloat16* src = t.x + b * t.b + h * t.h + n * t.n;
        v[u][0] = *reinterpret_cast<const uint4*>(src + rl.off0);
        v[u][1] = *reinterpret_cast<const uint4*>(src + rl.off1);
      }
    }
    rope_angles<D>(freq, p.positions + token, tokens, table.half, p.sign, angles[warp], lane);
    float2 cs[8];
    rope_take(angles[warp], rl, cs);
#pragma unroll
    for (int u = 0; u < kRopeRows; ++u) {
      if (dst[u] == nullptr) continue;
      if (rl.turns) {
        float x[8], y[8];
        unpack_bf16x8(v[u][0], x);
        unpack_bf16x8(v[u][1], y);
        rope_turn(x, y, cs, table.adjacent);
        v[u][0] = pack_bf16x8(x);
        v[u][1] = pack_bf16x8(y);
      }
      *reinterpret_cast<uint4*>(dst[u] + rl.off0) = v[u][0];
      *reinterpret_cast<uint4*>(dst[u] + rl.off1) = v[u][1];
    }
  }
}

}  // namespace attn
