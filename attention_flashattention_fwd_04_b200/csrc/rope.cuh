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

constexpr int kRopeThreads = 128;

// One warp a token: its lanes take D / 16 of a row each and go through the
// token's heads, queries then keys.
template <int D>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeTable table, const RopeParams p) {
  constexpr int kLanes = D / 16;
  constexpr int kRows = 32 / kLanes;
  const long long token = (static_cast<long long>(blockIdx.x) * kRopeThreads + threadIdx.x) >> 5;
  if (token >= static_cast<long long>(p.B) * p.N) return;
  const int lane = threadIdx.x & 31;
  const int b = static_cast<int>(token / p.N), n = static_cast<int>(token % p.N);
  const RopeLane rl = rope_lane(lane % kLanes, table.half, table.adjacent);
  float2 cs[8];
  if (rl.turns) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int pos = p.positions[static_cast<long long>(table.axis[rl.freq + i]) * p.B * p.N + token];
      cs[i] = rope_cos_sin(pos, table.turn[rl.freq + i]);
      cs[i].y *= p.sign;
    }
  }
  for (int r = lane / kLanes; r < p.q.H + p.k.H; r += kRows) {
    const bool is_q = r < p.q.H;
    const RopeTensor& t = is_q ? p.q : p.k;
    const int h = is_q ? r : r - p.q.H;
    const __nv_bfloat16* src = t.x + b * t.b + h * t.h + n * t.n;
    __nv_bfloat16* dst = t.out + b * t.ob + h * t.oh + n * t.on;
    uint4 v0 = *reinterpret_cast<const uint4*>(src + rl.off0);
    uint4 v1 = *reinterpret_cast<const uint4*>(src + rl.off1);
    if (rl.turns) {
      float x[8], y[8];
      unpack_bf16x8(v0, x);
      unpack_bf16x8(v1, y);
      rope_turn(x, y, cs, table.adjacent);
      v0 = pack_bf16x8(x);
      v1 = pack_bf16x8(y);
    }
    *reinterpret_cast<uint4*>(dst + rl.off0) = v0;
    *reinterpret_cast<uint4*>(dst + rl.off1) = v1;
  }
}

}  // namespace attn
