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

// Programmatic launches.  A kernel launched with the stream-serialisation
// attribute may begin once every CTA of the kernel before it has called
// griddep_launch (or ended); griddep_wait then waits for that kernel's end, with
// all it wrote visible.  Both return at once in a launch without the attribute.
__device__ __forceinline__ void griddep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void griddep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

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
  int tokens_log2;        // of a block
  int tokens_together;    // a head's tokens are nearer to one another than a token's heads
  float sign;             // -1: the gradient
};

// The kernels on rows (this one and the append to the 8-bit cache) give a block
// 2^tokens_log2 tokens.  Their angles are worked out once, by all threads, into
// shared memory, while the first rows are on their way; then a thread keeps to
// one token, its 16 values of a row and their angles, and goes through the heads.
// The block's D / 16 lanes a row cover kRowSlots rows at a time: heads of one
// token next to one another, or tokens of one head (whichever lie together).
constexpr int kRowThreads = 256;
constexpr int kRowTokens = 16;  // most tokens of a block
constexpr int kRowBatch = 4;    // rows that a thread has under way

template <int D>
struct RowShape {
  static constexpr int kLanes = D / 16;
  static constexpr int kSlots = kRowThreads / kLanes;
};

// cos and sin of the block's angles, [token][frequency].  kRowThreads is a
// multiple of kRopeMaxHalf, so a thread has one frequency.
__device__ __forceinline__ void rope_angles(const RopeTable& table, const int32_t* positions, long long axis_stride, int tokens,
                                            float sign, float2 (*cs)[kRopeMaxHalf]) {
  const int j = threadIdx.x % kRopeMaxHalf;
  if (j >= table.half) return;
  const uint64_t turn = table.turn[j];
  const int32_t* mine = positions + table.axis[j] * axis_stride;
  for (int t = threadIdx.x / kRopeMaxHalf; t < tokens; t += kRowThreads / kRopeMaxHalf) {
    float2 v = rope_cos_sin(mine[t], turn);
    v.y *= sign;
    cs[t][j] = v;
  }
}

// A lane's 8 angles.
__device__ __forceinline__ void rope_take(const float2* cs, const RopeLane& rl, float2 (&out)[8]) {
  if (!rl.turns) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = reinterpret_cast<const float4*>(cs + rl.freq)[i];
    out[2 * i] = make_float2(v.x, v.y);
    out[2 * i + 1] = make_float2(v.z, v.w);
  }
}

// Loads up to kRowBatch rows: heads h, h + step, ...
__device__ __forceinline__ void rows_load(uint4 (&v)[kRowBatch][2], const __nv_bfloat16* x, long long stride, int h, int step, int H,
                                          const RopeLane& rl) {
#pragma unroll
  for (int u = 0; u < kRowBatch; ++u) {
    if (h + u * step < H) {
      const __nv_bfloat16* src = x + (h + u * step) * stride;
      v[u][0] = *reinterpret_cast<const uint4*>(src + rl.off0);
      v[u][1] = *reinterpret_cast<const uint4*>(src + rl.off1);
    }
  }
}

// Turns them and stores them.
__device__ __forceinline__ void rows_turn(uint4 (&v)[kRowBatch][2], __nv_bfloat16* out, long long stride, int h, int step, int H,
                                          const RopeLane& rl, const float2 (&cs)[8], bool adjacent) {
#pragma unroll
  for (int u = 0; u < kRowBatch; ++u) {
    if (h + u * step >= H) continue;
    if (rl.turns) {
      float x[8], y[8];
      unpack_bf16x8(v[u][0], x);
      unpack_bf16x8(v[u][1], y);
      rope_turn(x, y, cs, adjacent);
      v[u][0] = pack_bf16x8(x);
      v[u][1] = pack_bf16x8(y);
    }
    __nv_bfloat16* dst = out + (h + u * step) * stride;
    *reinterpret_cast<uint4*>(dst + rl.off0) = v[u][0];
    *reinterpret_cast<uint4*>(dst + rl.off1) = v[u][1];
  }
}

template <int D>
__global__ void __launch_bounds__(kRowThreads, 2) rope_kernel(const __grid_constant__ RopeTable table, const RopeParams p) {
  using R = RowShape<D>;
  __shared__ __align__(16) float2 angles[kRowTokens][kRopeMaxHalf];
  const int per_block = 1 << p.tokens_log2, step = R::kSlots >> p.tokens_log2;  // heads at a time
  const long long first = static_cast<long long>(blockIdx.x) << p.tokens_log2, all = static_cast<long long>(p.B) * p.N;
  const int tokens = static_cast<int>(min(static_cast<long long>(per_block), all - first));
  const int slot = threadIdx.x / R::kLanes;
  const int tok = p.tokens_together ? slot & (per_block - 1) : slot / step;
  const int h0 = p.tokens_together ? slot >> p.tokens_log2 : slot % step;
  const RopeLane rl = rope_lane(threadIdx.x % R::kLanes, table.half, table.adjacent);
  const bool on = tok < tokens;
  const long long token = first + tok;
  const long long b = token / p.N, n = token - b * p.N;
  const int hq = on ? p.q.H : 0, hk = on ? p.k.H : 0;  // a thread behind the last token has no rows
  const __nv_bfloat16 *q = p.q.x + b * p.q.b + n * p.q.n, *k = p.k.x + b * p.k.b + n * p.k.n;
  __nv_bfloat16 *q_out = p.q.out + b * p.q.ob + n * p.q.on, *k_out = p.k.out + b * p.k.ob + n * p.k.on;
  uint4 v[2][kRowBatch][2];
  rows_load(v[0], q, p.q.h, h0, step, hq, rl);
  rope_angles(table, p.positions + first, all, tokens, p.sign, angles);
  __syncthreads();
  float2 cs[8];
  rope_take(angles[tok], rl, cs);
  const int more = kRowBatch * step;
  for (int h = h0; h < hq; h += 2 * more) {
    rows_load(v[1], q, p.q.h, h + more, step, hq, rl);
    rows_turn(v[0], q_out, p.q.oh, h, step, hq, rl, cs, table.adjacent);
    rows_load(v[0], q, p.q.h, h + 2 * more, step, hq, rl);
    rows_turn(v[1], q_out, p.q.oh, h + more, step, hq, rl, cs, table.adjacent);
  }
  for (int h = h0; h < hk; h += more) {
    rows_load(v[0], k, p.k.h, h, step, hk, rl);
    rows_turn(v[0], k_out, p.k.oh, h, step, hk, rl, cs, table.adjacent);
  }
}

}  // namespace attn
