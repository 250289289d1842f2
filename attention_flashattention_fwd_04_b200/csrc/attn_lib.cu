// The library's main translation unit: the entry points of attn_api.cu and,
// on top of its host helpers and its device error word (one word a translation
// unit), those of the rotary positions and of the 8-bit paged cache.
#include "attn_api.cu"

#include <algorithm>

#include "cache8.cuh"
#include "decode8_sm100.cuh"
#include "rope.cuh"

namespace {

// ----------------------------------------------------------------------------
// Rotary positions
// ----------------------------------------------------------------------------

// inv_freq / 2 pi modulo 1, in units of 2^-64, to the nearest, for |inv_freq| <
// 2^62: the product of the frequency's 53 bits and the first 128 of 1 / 2 pi, shifted.
// (A quotient in 64 bits would lose one of the fraction's for each bit of whole turns.)
uint64_t rope_turn(double inv_freq) {
  constexpr uint64_t kInverse[2] = {0x28be60db9391054aull, 0x7f09d5f47d4d3770ull};  // 1 / 2 pi
  int e;
  const uint64_t m = static_cast<uint64_t>(std::ldexp(std::frexp(std::fabs(inv_freq), &e), 53));
  const int shift = 53 - e + 64;  // inv_freq / 2 pi * 2^64 = m * kInverse / 2^shift, shift >= 55
  if (shift > 190) return 0;      // below half a unit
  const unsigned __int128 low = static_cast<unsigned __int128>(m) * kInverse[1];
  const unsigned __int128 high = static_cast<unsigned __int128>(m) * kInverse[0] + static_cast<uint64_t>(low >> 64);
  const uint64_t words[4] = {static_cast<uint64_t>(low), static_cast<uint64_t>(high), static_cast<uint64_t>(high >> 64), 0};
  auto from = [&](int bit) {  // 64 bits of the product
    const int w = bit / 64, b = bit % 64;
    if (w > 2) return uint64_t{0};
    return b == 0 ? words[w] : words[w] >> b | words[w + 1] << (64 - b);
  };
  const uint64_t turn = from(shift) + (from(shift - 1) & 1u);
  return inv_freq < 0 ? 0 - turn : turn;
}

// Checks a rotation and lays its table out for the kernels.
int rope_table(const attn_rope_spec* spec, int d, attn::RopeTable* out) {
  if (!spec) return ATTN_ERR_NULL;
  if (spec->rot_dim < 16 || spec->rot_dim > d || spec->rot_dim % 16 != 0) return ATTN_ERR_SHAPE;
  if (spec->num_axes < 1 || spec->num_axes > 255) return ATTN_ERR_SHAPE;
  if (spec->adjacent_pairs != 0 && spec->adjacent_pairs != 1) return ATTN_ERR_SHAPE;
  *out = attn::RopeTable{};
  out->half = spec->rot_dim / 2;
  out->adjacent = spec->adjacent_pairs;
  for (int j = 0; j < out->half; ++j) {
    if (!(std::fabs(spec->inv_freq[j]) < 0x1p62) || spec->axis[j] >= spec->num_axes) return ATTN_ERR_SHAPE;
    out->turn[j] = rope_turn(spec->inv_freq[j]);
    out->axis[j] = spec->axis[j];
  }
  return ATTN_OK;
}

// One of the two tensors of attn_rope.  Strides are in elements.
int rope_tensor(const attn_bf16* x, attn_bf16* out, const long long* strides, const long long* out_strides, int B, int H,
                int N, attn::RopeTensor* t) {
  if (!x || !out || !strides || !out_strides) return ATTN_ERR_NULL;
  if (H < 1) return ATTN_ERR_SHAPE;
  const int sizes[3] = {B, H, N};
  for (int i = 0; i < 3; ++i) {
    if (strides[i] < 0 || out_strides[i] < 0) return ATTN_ERR_SHAPE;
    if (sizes[i] > 1 && out_strides[i] == 0) return ATTN_ERR_SHAPE;  // rows of the output would fall together
  }
  for (int i = 0; i < 3; ++i)  // the stride of a size of 1 is never used
    if (sizes[i] > 1 && (strides[i] % 8 != 0 || out_strides[i] % 8 != 0)) return ATTN_ERR_ALIGN;
  if (misaligned16(x) || misaligned16(out)) return ATTN_ERR_ALIGN;
  t->x = reinterpret_cast<const __nv_bfloat16*>(x);
  t->out = reinterpret_cast<__nv_bfloat16*>(out);
  t->b = strides[0];
  t->h = strides[1];
  t->n = strides[2];
  t->ob = out_strides[0];
  t->oh = out_strides[1];
  t->on = out_strides[2];
  t->H = H;
  return ATTN_OK;
}

// ----------------------------------------------------------------------------
// The 8-bit cache
// ----------------------------------------------------------------------------

// Checks shared by the calls on the 8-bit cache (no CUDA call).
int validate_cache8(const void* k_pool, const void* v_pool, const void* kv_scales, const int32_t* block_table,
                    const int32_t* seq_lens, int num_seqs, int Hkv, int d, int page_size, int max_pages, int num_pages) {
  if (!k_pool || !v_pool || !kv_scales || !block_table || !seq_lens) return ATTN_ERR_NULL;
  if (num_seqs < 1 || Hkv < 1 || max_pages < 1 || num_pages < 1 || page_size < 1) return ATTN_ERR_SHAPE;
  if (d != 64 && d != 128) return ATTN_ERR_SHAPE;
  if (num_seqs > 65535 || Hkv > 65535) return ATTN_ERR_SHAPE;
  if (static_cast<long long>(num_pages) * page_size > INT_MAX || static_cast<long long>(max_pages) * page_size > INT_MAX)
    return ATTN_ERR_SHAPE;
  if (page_size % 16 != 0 || page_size > 256) return ATTN_ERR_UNSUPPORTED;
  if (misaligned16(k_pool) || misaligned16(v_pool) || misaligned16(kv_scales) || misaligned4(block_table) ||
      misaligned4(seq_lens))
    return ATTN_ERR_ALIGN;
  return ATTN_OK;
}

// Launches a kernel that may begin while the one before it ends
// (griddep_wait in rope.cuh).
template <typename... Params, typename... Args>
cudaError_t launch_early(void (*kernel)(Params...), unsigned grid_x, unsigned grid_y, unsigned threads, size_t smem, int cluster,
                         cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid_x, grid_y);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// SMs of a B200.  Plans, and with them workspaces, follow from the sizes alone and
// ask no device; on a part of one (fewer SMs) the same grids take more rounds.
constexpr int kPlanSms = 148;

// Tokens of a block of the kernels on rows: 16, so that their angles are shared
// by many rows and a head's tokens make long runs (4 x 16 + 16 heads x 2048
// tokens of d = 128: 24.1 us, with 8 tokens 26.4), but no more than leave two
// blocks for each SM; below 16 tokens that gives two to four.
int row_tokens_log2(long long tokens) {
  int n = 4;
  while (n > 0 && tokens >> n < 2 * kPlanSms) --n;
  return n;
}

template <int D>
int launch_append8(const attn::RopeTable& table, attn::Append8Params p, bool rope, cudaStream_t stream) {
  const int sms = sm_count();
  if (sms <= 0) return fail_cuda(cudaErrorInvalidDevice);
  cudaError_t e;
  if (rope) {
    p.tokens_log2 = row_tokens_log2(p.total_q);
    const unsigned grid = static_cast<unsigned>((static_cast<long long>(p.total_q) + (1 << p.tokens_log2) - 1) >> p.tokens_log2);
    p.one_wave = grid <= static_cast<unsigned>(sms);
    e = launch_early(attn::rope_append8_kernel<D>, grid, 1, attn::kRowThreads, 0, 1, stream, table, p);
  } else {
    // A warp an item, up to a few times what the SMs hold at once.
    constexpr int heads = 512 / D * attn::kAppend8Heads, warps = attn::kAppend8Threads / 32;
    const long long items = static_cast<long long>(p.total_q) * ((p.Hkv + heads - 1) / heads);
    const unsigned grid = static_cast<unsigned>(std::min<long long>((items + warps - 1) / warps, 16LL * sms));
    p.one_wave = grid <= static_cast<unsigned>(sms);
    e = launch_early(attn::append8_kernel<D>, grid, 1, attn::kAppend8Threads, 0, 1, stream, p);
  }
  if (e != cudaSuccess) return fail_cuda(e);
  e = cudaGetLastError();
  return e == cudaSuccess ? ATTN_OK : fail_cuda(e);
}

int append8(const attn_bf16* q, const attn_bf16* k_new, const attn_bf16* v_new, attn_bf16* q_out, const int32_t* positions,
            const attn_rope_spec* spec, bool rope, uint8_t* k_pool, uint8_t* v_pool, uint8_t* kv_scales,
            const int32_t* cu_seqlens_q, const int32_t* seq_lens, const int32_t* block_table, int num_seqs, int total_q,
            int Hq, int Hkv, int d, int page_size, int max_pages, int num_pages, void* stream) {
  const int st = validate_cache8(k_pool, v_pool, kv_scales, block_table, seq_lens, num_seqs, Hkv, d, page_size, max_pages,
                                 num_pages);
  if (st != ATTN_OK) return st;
  if (!cu_seqlens_q) return ATTN_ERR_NULL;
  if (total_q < 0) return ATTN_ERR_SHAPE;
  if (misaligned4(cu_seqlens_q)) return ATTN_ERR_ALIGN;
  attn::RopeTable table{};
  if (rope) {
    if (Hq < 1 || Hq > 65535) return ATTN_ERR_SHAPE;
    const int rs = rope_table(spec, d, &table);
    if (rs != ATTN_OK) return rs;
  }
  if (total_q == 0) return ATTN_OK;
  if (!k_new || !v_new || (rope && (!q || !q_out || !positions))) return ATTN_ERR_NULL;
  if (misaligned16(k_new) || misaligned16(v_new)) return ATTN_ERR_ALIGN;
  if (rope && (misaligned16(q) || misaligned16(q_out) || misaligned4(positions))) return ATTN_ERR_ALIGN;
  attn::Append8Params p{};
  p.q = reinterpret_cast<const __nv_bfloat16*>(q);
  p.k_new = reinterpret_cast<const __nv_bfloat16*>(k_new);
  p.v_new = reinterpret_cast<const __nv_bfloat16*>(v_new);
  p.q_out = reinterpret_cast<__nv_bfloat16*>(q_out);
  p.k_pool = k_pool;
  p.v_pool = v_pool;
  p.kv_scales = kv_scales;
  p.positions = positions;
  p.cu_q = cu_seqlens_q;
  p.seq_lens = seq_lens;
  p.block_table = block_table;
  p.num_seqs = num_seqs;
  p.total_q = total_q;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.page_size = page_size;
  p.max_pages = max_pages;
  p.num_pages = num_pages;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return d == 128 ? launch_append8<128>(table, p, rope, s) : launch_append8<64>(table, p, rope, s);
}

// The plan of a decode over the 8-bit cache, from the sizes alone: the group of
// heads a tile covers and the room for partial results.
struct Decode8Plan {
  int hb = 0;    // KV heads of a tile
  int ctas = 0;  // CTAs of the split pass, or of a cluster
  bool cluster = false;
  int box = 0;   // tokens of one TMA box
  size_t lse_offset = 0, total = 0;
};

bool decode8_plan(int num_seqs, int Hq, int Hkv, int d, int max_pages, int page_size, Decode8Plan* out) {
  if (num_seqs < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || max_pages < 1 || page_size < 1 || (d != 64 && d != 128)) return false;
  const long long max_tokens = static_cast<long long>(max_pages) * page_size;
  if (max_tokens > INT_MAX) return false;
  Decode8Plan pl;
  const int group = Hq / Hkv;
  // Clusters, where one a sequence and KV head fills no more than the SMs hold
  // and a CTA has few tiles: no partial results and no second launch, but no even
  // shares either.  Up to 8 tiles where they fill half the SMs or more (16
  // sequences of 2000 tokens, 8 KV heads: 17.7 us against 22.0; one of 2000 among
  // 15 of 100: 12.8 against 12.8; with up to 16, one of 4000 among 15: 20.2 against
  // 13.5), else 4 (one of 4000 tokens, 8 KV heads: 8.6 against 11.0; of 8000, 2 KV
  // heads, d = 64, 8 tiles: 12.5 against 9.6).
  // An SM group whose SMs do not divide by the cluster's leaves some out: 33
  // clusters of 8 are there at once with two CTAs an SM, 15 with one, 71 and 33 of
  // 4.  The rooms stay below that, as the last one to wait doubles the time (16
  // sequences of 1000 tokens, 16 query heads of one KV head: 15.4 us in clusters
  // of 8, 8.8 of 4).
  const long long heads = static_cast<long long>(num_seqs) * Hkv, head_tiles = (max_tokens + attn::kDecode8Rows - 1) / attn::kDecode8Rows;
  const int per_sm = group <= 8 || d == 64 ? 2 : 1;
  auto room = [&](int ctas) { return per_sm * (ctas == 8 ? 112 : 128); };
  int most = 8;
  while (most > 1 && (heads * most > room(most) || most / 2 >= head_tiles)) most /= 2;
  const int most_tiles = 2 * heads * most >= room(most) ? 8 : 4;
  pl.cluster = heads * most <= room(most) && head_tiles <= most_tiles * most;
  pl.hb = pl.cluster ? 1 : decode_heads_per_cta(Hkv);
  const int tokens = attn::kDecode8Rows / pl.hb;
  if (pl.cluster) {
    pl.ctas = most;
    pl.box = 16;
    while (pl.box < tokens && page_size % (2 * pl.box) == 0) pl.box *= 2;
    *out = pl;
    return true;
  }
  for (pl.box = 16; pl.box < tokens && page_size % (2 * pl.box) == 0;) pl.box *= 2;
  const long long tiles = std::min(num_seqs, attn::kDecode8MaxSeqs) * ((max_tokens + tokens - 1) / tokens) * (Hkv / pl.hb);
  if (tiles + 3LL * attn::kDecode8MaxSeqs * (Hkv / pl.hb) > INT_MAX) return false;  // units of work, in 32 bits
  // Every CTA that the SMs hold at once (see paged_attn_decode_fp8), or one a tile.
  pl.ctas = static_cast<int>(std::min<long long>(tiles, d == 64 || group <= 8 ? 2 * kPlanSms : kPlanSms));
  const size_t rows = 2 * static_cast<size_t>(pl.ctas) * pl.hb * group;
  pl.lse_offset = rows * d * sizeof(float);
  pl.total = (pl.lse_offset + rows * sizeof(float) + 15) & ~static_cast<size_t>(15);
  *out = pl;
  return true;
}

// 3-D map of codes; rows of 128 or 64 bytes, swizzled as wide.
bool encode_3d_bytes(CUtensorMap* map, const void* ptr, uint64_t d0, uint64_t d1, uint64_t d2, uint64_t stride1,
                     uint64_t stride2, uint32_t b0, uint32_t b1, uint32_t b2, CUtensorMapSwizzle swizzle) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {d0, d1, d2};
  const cuuint64_t strides[2] = {stride1, stride2};
  const cuuint32_t box[3] = {b0, b1, b2};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(ptr), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int NT, int PER_SM, int STAGES>
int launch_decode8(const CUtensorMap& tk, const CUtensorMap& tv, const attn::Decode8Params& p, bool cluster, cudaStream_t stream) {
  using L = attn::Decode8Layout<D, STAGES>;
  cudaError_t e;
  if (cluster) {
    e = ensure_smem_limit<attn::decode8_split_kernel<D, NT, PER_SM, STAGES, true>>(L::kAlloc);
    if (e != cudaSuccess) return fail_cuda(e);
    e = launch_early(attn::decode8_split_kernel<D, NT, PER_SM, STAGES, true>, static_cast<unsigned>(p.S * p.Hkv * p.ctas), 1, L::kThreads,
                     L::kAlloc, p.ctas, stream, tk, tv, p);
    if (e != cudaSuccess) return fail_cuda(e);
    e = cudaGetLastError();
    return e == cudaSuccess ? ATTN_OK : fail_cuda(e);
  }
  e = ensure_smem_limit<attn::decode8_split_kernel<D, NT, PER_SM, STAGES, false>>(L::kAlloc);
  if (e != cudaSuccess) return fail_cuda(e);
  e = launch_early(attn::decode8_split_kernel<D, NT, PER_SM, STAGES, false>, static_cast<unsigned>(p.ctas), 1, L::kThreads, L::kAlloc, 1,
                   stream, tk, tv, p);
  if (e != cudaSuccess) return fail_cuda(e);
  // Warps for a head's partial rows, about CTAs / (sequences x groups of heads) of
  // them: a warp takes 4 or 8 at a time, so one warp makes many trips to memory
  // where there are many (16 sequences of 1000 tokens, 18 rows: 20.3 us with 1,
  // 17.1 with 8), and many warps are idle blocks where there are few (the same
  // with 16: 24.9; 64 of 1000, 5 rows: 41.0 with 8, 33.1 with 2; 4 of 1000, 74
  // rows: 10.4 with 16, 15.7 with 2).
  const long long heads = static_cast<long long>(p.S) * (p.Hkv / p.hb);
  const int per = p.ctas > 48 * heads ? 16 : p.ctas > 12 * heads ? 8 : p.ctas > 2 * heads ? 2 : 1;
  auto* merge = per == 16  ? attn::decode8_merge_kernel<D, 16>
                : per == 8 ? attn::decode8_merge_kernel<D, 8>
                : per == 2 ? attn::decode8_merge_kernel<D, 2>
                           : attn::decode8_merge_kernel<D, 1>;
  const int heads_a_block = attn::kMerge8Warps / per;
  e = launch_early(merge, static_cast<unsigned>((p.Hq + heads_a_block - 1) / heads_a_block), static_cast<unsigned>(p.S),
                   32 * attn::kMerge8Warps, 0, 1, stream, p);
  if (e != cudaSuccess) return fail_cuda(e);
  e = cudaGetLastError();
  return e == cudaSuccess ? ATTN_OK : fail_cuda(e);
}

}  // namespace

extern "C" {

int attn_rope(const attn_bf16* q, attn_bf16* q_out, const long long* q_strides, const long long* q_out_strides, int Hq,
              const attn_bf16* k, attn_bf16* k_out, const long long* k_strides, const long long* k_out_strides, int Hkv,
              int B, int N, int d, const int32_t* positions, const attn_rope_spec* spec, int inverse, void* stream) {
  if (B < 0 || N < 0) return ATTN_ERR_SHAPE;
  if (d != 64 && d != 128) return ATTN_ERR_SHAPE;
  if (inverse != 0 && inverse != 1) return ATTN_ERR_SHAPE;
  const long long tokens = static_cast<long long>(B) * N;
  if (tokens > INT_MAX) return ATTN_ERR_SHAPE;
  attn::RopeTable table;
  const int st = rope_table(spec, d, &table);
  if (st != ATTN_OK) return st;
  if (tokens == 0) return ATTN_OK;
  if (!positions) return ATTN_ERR_NULL;
  attn::RopeParams p{};
  int ts = rope_tensor(q, q_out, q_strides, q_out_strides, B, Hq, N, &p.q);
  if (ts != ATTN_OK) return ts;
  if (k || k_out) {
    ts = rope_tensor(k, k_out, k_strides, k_out_strides, B, Hkv, N, &p.k);
    if (ts != ATTN_OK) return ts;
  }
  if (misaligned4(positions)) return ATTN_ERR_ALIGN;
  p.positions = positions;
  p.B = B;
  p.N = N;
  p.sign = inverse ? -1.f : 1.f;
  p.tokens_log2 = row_tokens_log2(tokens);
  p.tokens_together = p.q.n < p.q.h;
  const unsigned grid = static_cast<unsigned>((tokens + (1 << p.tokens_log2) - 1) >> p.tokens_log2);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d == 128)
    attn::rope_kernel<128><<<grid, attn::kRowThreads, 0, s>>>(table, p);
  else
    attn::rope_kernel<64><<<grid, attn::kRowThreads, 0, s>>>(table, p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? ATTN_OK : fail_cuda(e);
}

int paged_kv_append_fp8(const attn_bf16* k_new, const attn_bf16* v_new, uint8_t* k_pool, uint8_t* v_pool, uint8_t* kv_scales,
                        const int32_t* cu_seqlens_q, const int32_t* seq_lens, const int32_t* block_table, int num_seqs,
                        int total_q, int Hkv, int d, int page_size, int max_pages, int num_pages, void* stream) {
  return append8(nullptr, k_new, v_new, nullptr, nullptr, nullptr, false, k_pool, v_pool, kv_scales, cu_seqlens_q, seq_lens,
                 block_table, num_seqs, total_q, 0, Hkv, d, page_size, max_pages, num_pages, stream);
}

int paged_rope_append_fp8(const attn_bf16* q, const attn_bf16* k_new, const attn_bf16* v_new, attn_bf16* q_out,
                          const int32_t* positions, const attn_rope_spec* spec, uint8_t* k_pool, uint8_t* v_pool,
                          uint8_t* kv_scales, const int32_t* cu_seqlens_q, const int32_t* seq_lens,
                          const int32_t* block_table, int num_seqs, int total_q, int Hq, int Hkv, int d, int page_size,
                          int max_pages, int num_pages, void* stream) {
  return append8(q, k_new, v_new, q_out, positions, spec, true, k_pool, v_pool, kv_scales, cu_seqlens_q, seq_lens,
                 block_table, num_seqs, total_q, Hq, Hkv, d, page_size, max_pages, num_pages, stream);
}

int paged_kv_gather_fp8(const uint8_t* k_pool, const uint8_t* v_pool, const uint8_t* kv_scales, const int32_t* block_table,
                        const int32_t* seq_lens, const int32_t* cu_seqlens_k, attn_bf16* k_out, attn_bf16* v_out,
                        int num_seqs, int total_rows, int Hkv, int d, int page_size, int max_pages, int num_pages,
                        void* stream) {
  const int st = validate_cache8(k_pool, v_pool, kv_scales, block_table, seq_lens, num_seqs, Hkv, d, page_size, max_pages,
                                 num_pages);
  if (st != ATTN_OK) return st;
  if (!cu_seqlens_k) return ATTN_ERR_NULL;
  if (total_rows < 0) return ATTN_ERR_SHAPE;
  if (misaligned4(cu_seqlens_k)) return ATTN_ERR_ALIGN;
  if (total_rows == 0) return ATTN_OK;
  if (!k_out || !v_out) return ATTN_ERR_NULL;
  if (((reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) & 31u) != 0) return ATTN_ERR_ALIGN;
  attn::Gather8Params p{};
  p.k_pool = k_pool;
  p.v_pool = v_pool;
  p.kv_scales = kv_scales;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.cu_k = cu_seqlens_k;
  p.k_out = reinterpret_cast<__nv_bfloat16*>(k_out);
  p.v_out = reinterpret_cast<__nv_bfloat16*>(v_out);
  p.num_seqs = num_seqs;
  p.total_rows = total_rows;
  p.Hkv = Hkv;
  p.page_size = page_size;
  p.max_pages = max_pages;
  p.num_pages = num_pages;
  const unsigned grid = static_cast<unsigned>((static_cast<long long>(total_rows) * 32 + attn::kGather8Threads - 1) /
                                              attn::kGather8Threads);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d == 128)
    attn::gather8_kernel<128><<<grid, attn::kGather8Threads, 0, s>>>(p);
  else
    attn::gather8_kernel<64><<<grid, attn::kGather8Threads, 0, s>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? ATTN_OK : fail_cuda(e);
}

size_t paged_attn_decode_fp8_workspace_bytes(int num_seqs, int Hq, int Hkv, int d, int max_pages, int page_size) {
  Decode8Plan pl;
  if (!decode8_plan(num_seqs, Hq, Hkv, d, max_pages, page_size, &pl)) return 0;
  return pl.total;
}

int paged_attn_decode_fp8(const attn_bf16* q, const uint8_t* k_pool, const uint8_t* v_pool, const uint8_t* kv_scales,
                          const int32_t* block_table, const int32_t* seq_lens, int page_size, attn_bf16* o, float* lse,
                          int num_seqs, int Hq, int Hkv, int d, int max_pages, int num_pages, float scale, void* workspace,
                          size_t workspace_bytes, void* stream) {
  if (!q || !o || !lse) return ATTN_ERR_NULL;
  const int st = validate_cache8(k_pool, v_pool, kv_scales, block_table, seq_lens, num_seqs, Hkv, d, page_size, max_pages,
                                 num_pages);
  if (st != ATTN_OK && st != ATTN_ERR_UNSUPPORTED && st != ATTN_ERR_ALIGN) return st;
  if (Hq < 1 || Hq % Hkv != 0 || Hq > 65535) return ATTN_ERR_SHAPE;
  if (!(scale > 0.f) || !std::isfinite(scale)) return ATTN_ERR_SHAPE;
  if (st == ATTN_ERR_UNSUPPORTED || Hq / Hkv > 16) return ATTN_ERR_UNSUPPORTED;
  Decode8Plan pl;
  if (!decode8_plan(num_seqs, Hq, Hkv, d, max_pages, page_size, &pl)) return ATTN_ERR_SHAPE;
  if (pl.total > 0 && (!workspace || workspace_bytes < pl.total)) return ATTN_ERR_WORKSPACE;
  if (st == ATTN_ERR_ALIGN || misaligned16(q) || misaligned16(o) || misaligned16(workspace) || misaligned4(lse))
    return ATTN_ERR_ALIGN;

  CUtensorMap tk, tv;
  const uint64_t rows = static_cast<uint64_t>(num_pages) * page_size;
  const uint64_t token_bytes = static_cast<uint64_t>(Hkv) * d;
  const uint32_t hb = static_cast<uint32_t>(pl.hb);
  const CUtensorMapSwizzle sw = d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  // (value, token row, head)
  if (!encode_3d_bytes(&tk, k_pool, d, rows, Hkv, token_bytes, d, d, pl.box, hb, sw) ||
      !encode_3d_bytes(&tv, v_pool, d, rows, Hkv, token_bytes, d, d, pl.box, hb, sw))
    return fail_cuda(cudaErrorInvalidValue);

  attn::Decode8Params p{};
  p.part_o = static_cast<float*>(workspace);
  p.part_lse = reinterpret_cast<float*>(static_cast<char*>(workspace) + pl.lse_offset);
  p.kv_scales = kv_scales;
  p.box = pl.box;
  const uint32_t page_chunks = static_cast<uint32_t>(page_size / 16);
  p.page_inverse = page_chunks == 1 ? 0u : static_cast<uint32_t>(((1ull << 32) + page_chunks - 1) / page_chunks);
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.group = Hq / Hkv;
  p.page_size = page_size;
  p.max_pages = max_pages;
  p.num_pages = num_pages;
  p.hb = pl.hb;
  for (p.hb_log2 = 0; 1 << p.hb_log2 < pl.hb;) ++p.hb_log2;
  p.ctas = pl.ctas;
  p.scale_mantissa = static_cast<float>(2.0 * std::frexp(static_cast<double>(scale) * kLog2e, &p.scale_exp));  // whatever scale's exponent
  --p.scale_exp;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  for (int s0 = 0; s0 < num_seqs; s0 += attn::kDecode8MaxSeqs) {  // one launch for up to 1024 sequences
    p.S = std::min(num_seqs - s0, attn::kDecode8MaxSeqs);
    p.q = reinterpret_cast<const __nv_bfloat16*>(q) + static_cast<size_t>(s0) * Hq * d;
    p.o = reinterpret_cast<__nv_bfloat16*>(o) + static_cast<size_t>(s0) * Hq * d;
    p.lse = lse + static_cast<size_t>(s0) * Hq;
    p.block_table = block_table + static_cast<size_t>(s0) * max_pages;
    p.seq_lens = seq_lens + s0;
    // Two CTAs an SM, but one where 16 query heads of d = 128 need its registers.
    int rc;
    if (d == 128)
      rc = p.group <= 8 ? launch_decode8<128, 1, 2, 3>(tk, tv, p, pl.cluster, s) : launch_decode8<128, 2, 1, 6>(tk, tv, p, pl.cluster, s);
    else
      rc = p.group <= 8 ? launch_decode8<64, 1, 2, 6>(tk, tv, p, pl.cluster, s) : launch_decode8<64, 2, 2, 6>(tk, tv, p, pl.cluster, s);
    if (rc != ATTN_OK) return rc;
  }
  return ATTN_OK;
}

}  // extern "C"
