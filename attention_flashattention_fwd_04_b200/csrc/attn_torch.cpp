// Argument marshalling for the calls that a decode step makes once a layer: the
// checks, allocations and pointers of a call in C++, a few microseconds less
// each than in Python, where a small step's kernels take no longer than that.
// The work is done by the C ABI (include/attn_b200.h), whose functions api.py
// hands over by address; nothing of CUDA is called here but the current stream.
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/extension.h>

#include <array>
#include <cmath>
#include <optional>
#include <tuple>

#include "attn_b200.h"

namespace {

using at::Tensor;
using Maybe = std::optional<Tensor>;

struct Abi {
  decltype(&::attn_rope) rope = nullptr;
  decltype(&::paged_kv_append_fp8) append = nullptr;
  decltype(&::paged_rope_append_fp8) rope_append = nullptr;
  decltype(&::paged_kv_gather_fp8) gather = nullptr;
  decltype(&::paged_attn_decode_fp8_workspace_bytes) decode_bytes = nullptr;
  decltype(&::paged_attn_decode_fp8) decode = nullptr;
} abi;

void bind(uintptr_t rope, uintptr_t append, uintptr_t rope_append, uintptr_t gather, uintptr_t decode_bytes, uintptr_t decode) {
  abi.rope = reinterpret_cast<decltype(abi.rope)>(rope);
  abi.append = reinterpret_cast<decltype(abi.append)>(append);
  abi.rope_append = reinterpret_cast<decltype(abi.rope_append)>(rope_append);
  abi.gather = reinterpret_cast<decltype(abi.gather)>(gather);
  abi.decode_bytes = reinterpret_cast<decltype(abi.decode_bytes)>(decode_bytes);
  abi.decode = reinterpret_cast<decltype(abi.decode)>(decode);
}

void require(const Tensor& t, const char* name, at::ScalarType type, int64_t dims) {
  TORCH_CHECK_VALUE(t.scalar_type() == type, name, " must be ", type, ", got ", t.scalar_type());
  TORCH_CHECK_VALUE(t.dim() == dims, name, " must have ", dims, " dims, got shape ", t.sizes());
  TORCH_CHECK_VALUE(t.is_contiguous(), name, " must be contiguous");
}
void require(const Maybe& t, const char* name, at::ScalarType type, int64_t dims) {
  if (t) require(*t, name, type, dims);
}

void require_codes(const Tensor& t, const char* name, at::ScalarType type) {
  require(t, name, t.scalar_type() == at::kByte ? at::kByte : type, 4);
}

// After the shapes: every tensor on one CUDA device.
struct Device {
  const Tensor* first = nullptr;
  void add(const Tensor& t, const char* name) {
    TORCH_CHECK_VALUE(t.is_cuda(), name, " must be a CUDA tensor");
    if (!first) first = &t;
    TORCH_CHECK_VALUE(t.device() == first->device(), name, " is on ", t.device(), ", not on ", first->device());
  }
  void add(const Maybe& t, const char* name) {
    if (t) add(*t, name);
  }
};

int size32(int64_t n) {
  TORCH_CHECK_VALUE(n <= INT_MAX, "a size of ", n, " is out of range");
  return static_cast<int>(n);
}

const attn_bf16* in(const Tensor& t) { return static_cast<const attn_bf16*>(t.const_data_ptr()); }
attn_bf16* out(const Tensor& t) { return static_cast<attn_bf16*>(t.data_ptr()); }
const int32_t* ints(const Tensor& t) { return static_cast<const int32_t*>(t.const_data_ptr()); }
uint8_t* bytes(const Tensor& t) { return static_cast<uint8_t*>(t.data_ptr()); }

// The calling thread's device and stream for a call.
struct Call {
  c10::cuda::OptionalCUDAGuard guard;
  void* stream;
  explicit Call(const Device& d) : guard(d.first->device()) { stream = c10::cuda::getCurrentCUDAStream(d.first->device().index()).stream(); }
};

Tensor made(const Maybe& given, at::IntArrayRef shape, const Tensor& like, at::ScalarType type) {
  return given ? *given : at::empty(shape, like.options().dtype(type));
}

// ---------------------------------------------------------------- rotation

using Strides = std::array<long long, 3>;

Strides strides(const Tensor& x) {  // batch, head, token
  if (x.dim() == 4) return {x.stride(0), x.stride(1), x.stride(2)};
  return {0, x.stride(1), x.stride(0)};
}

void require_rows(const Tensor& x, const char* name, const Maybe& o, const char* o_name) {
  TORCH_CHECK_VALUE(x.scalar_type() == at::kBFloat16 && (x.dim() == 3 || x.dim() == 4), name,
                    " must be a 3-d or 4-d bfloat16 tensor, got ", x.scalar_type(), " ", x.sizes());
  TORCH_CHECK_VALUE(!o || (o->scalar_type() == at::kBFloat16 && o->sizes() == x.sizes()), o_name, " must be a bfloat16 tensor of ",
                    name, "'s shape");
  TORCH_CHECK_VALUE(x.numel() == 0 || x.stride(-1) == 1, "the rows of ", name, " must be contiguous");
  TORCH_CHECK_VALUE(!o || o->numel() == 0 || o->stride(-1) == 1, "the rows of ", o_name, " must be contiguous");
}

std::tuple<int, Tensor, Maybe> rope(const Tensor& q, const Maybe& k, const Tensor& positions, uintptr_t spec_at, bool inverse,
                                    const Maybe& q_out, const Maybe& k_out) {
  const auto* spec = reinterpret_cast<const attn_rope_spec*>(spec_at);
  require_rows(q, "q", q_out, "q_out");
  TORCH_CHECK_VALUE(k || !k_out, "k_out without k");
  if (k) require_rows(*k, "k", k_out, "k_out");
  const bool batched = q.dim() == 4;
  const int64_t B = batched ? q.size(0) : 1, N = q.size(batched ? 2 : 0), d = q.size(-1);
  if (k) {
    TORCH_CHECK_VALUE(k->dim() == q.dim() && k->size(0) == q.size(0) && (!batched || k->size(2) == N) && k->size(-1) == d, "k shape ",
                      k->sizes(), " does not match q ", q.sizes());
  }
  require(positions, "positions", at::kInt, batched ? 3 : 2);
  TORCH_CHECK_VALUE(positions.size(0) == spec->num_axes && positions.size(-1) == N && (!batched || positions.size(1) == B),
                    "positions must be one per axis (", spec->num_axes, ") and token, got ", positions.sizes());
  Device on;
  on.add(q, "q");
  on.add(k, "k");
  on.add(positions, "positions");
  on.add(q_out, "q_out");
  on.add(k_out, "k_out");
  const Call call(on);
  Tensor qo = made(q_out, q.sizes(), q, at::kBFloat16);
  Maybe ko;
  if (k) ko = made(k_out, k->sizes(), q, at::kBFloat16);
  const Strides qs = strides(q), qos = strides(qo), ks = k ? strides(*k) : Strides{}, kos = ko ? strides(*ko) : Strides{};
  const int rc = abi.rope(in(q), out(qo), qs.data(), qos.data(), size32(q.size(1)), k ? in(*k) : nullptr, ko ? out(*ko) : nullptr,
                          ks.data(), kos.data(), k ? size32(k->size(1)) : 0, size32(B), size32(N), size32(d), ints(positions), spec,
                          inverse, call.stream);
  return {rc, qo, ko};
}

// ---------------------------------------------------------------- 8-bit cache

struct Cache {
  const Tensor &k_pool, &v_pool, &kv_scales, &block_table, &seq_lens;
  int S, num_pages, page_size, Hkv, d, max_pages;

  Cache(const Tensor& k, const Tensor& v, const Tensor& s, const Tensor& table, const Tensor& lens)
      : k_pool(k), v_pool(v), kv_scales(s), block_table(table), seq_lens(lens) {
    require_codes(k, "k_pool", at::kFloat8_e4m3fn);
    require_codes(v, "v_pool", at::kFloat8_e4m3fn);
    require_codes(s, "kv_scales", at::kFloat8_e8m0fnu);
    require(table, "block_table", at::kInt, 2);
    require(lens, "seq_lens", at::kInt, 1);
    num_pages = size32(k.size(0));
    page_size = size32(k.size(1));
    Hkv = size32(k.size(2));
    d = size32(k.size(3));
    TORCH_CHECK_VALUE(v.sizes() == k.sizes(), "v_pool shape ", v.sizes(), " differs from k_pool's ", k.sizes());
    TORCH_CHECK_VALUE(s.size(0) == num_pages && s.size(1) == Hkv && s.size(2) == page_size && s.size(3) == 2, "kv_scales must be [",
                      num_pages, ", ", Hkv, ", ", page_size, ", 2], got ", s.sizes());
    S = size32(lens.size(0));
    max_pages = size32(table.size(1));
    TORCH_CHECK_VALUE(table.size(0) == S, "block_table ", table.sizes(), " does not have one row per sequence (", S, ")");
  }
  void add_to(Device& on) const {
    on.add(k_pool, "k_pool");
    on.add(v_pool, "v_pool");
    on.add(kv_scales, "kv_scales");
    on.add(block_table, "block_table");
    on.add(seq_lens, "seq_lens");
  }
  // Shapes of a step's new rows.
  void require_new(const Tensor& k_new, const Tensor& v_new, const Tensor& cu) const {
    require(k_new, "k_new", at::kBFloat16, 3);
    require(v_new, "v_new", at::kBFloat16, 3);
    require_cu(cu, "cu_seqlens_q");
    TORCH_CHECK_VALUE(k_new.size(1) == Hkv && k_new.size(2) == d && v_new.sizes() == k_new.sizes(), "k_new ", k_new.sizes(), " / v_new ",
                      v_new.sizes(), " do not match the pools");
  }
  void require_cu(const Tensor& cu, const char* name) const {
    require(cu, name, at::kInt, 1);
    TORCH_CHECK_VALUE(cu.size(0) == S + 1, name, " does not match the number of sequences");
  }
};

int append(const Tensor& k_new, const Tensor& v_new, const Tensor& k_pool, const Tensor& v_pool, const Tensor& kv_scales,
           const Tensor& block_table, const Tensor& cu, const Tensor& seq_lens) {
  const Cache c(k_pool, v_pool, kv_scales, block_table, seq_lens);
  c.require_new(k_new, v_new, cu);
  Device on;
  c.add_to(on);
  on.add(k_new, "k_new");
  on.add(v_new, "v_new");
  on.add(cu, "cu_seqlens_q");
  const Call call(on);
  return abi.append(in(k_new), in(v_new), bytes(k_pool), bytes(v_pool), bytes(kv_scales), ints(cu), ints(seq_lens), ints(block_table),
                    c.S, size32(k_new.size(0)), c.Hkv, c.d, c.page_size, c.max_pages, c.num_pages, call.stream);
}

std::tuple<int, Tensor> rope_append(const Tensor& q, const Tensor& k_new, const Tensor& v_new, const Tensor& positions,
                                    uintptr_t spec_at, const Tensor& k_pool, const Tensor& v_pool, const Tensor& kv_scales,
                                    const Tensor& block_table, const Tensor& cu, const Tensor& seq_lens, const Maybe& q_out) {
  const auto* spec = reinterpret_cast<const attn_rope_spec*>(spec_at);
  const Cache c(k_pool, v_pool, kv_scales, block_table, seq_lens);
  c.require_new(k_new, v_new, cu);
  require(q, "q", at::kBFloat16, 3);
  require(q_out, "q_out", at::kBFloat16, 3);
  require(positions, "positions", at::kInt, 2);
  const int64_t T = k_new.size(0);
  TORCH_CHECK_VALUE(q.size(0) == T && q.size(2) == c.d && (!q_out || q_out->sizes() == q.sizes()), "q / q_out do not match k_new");
  TORCH_CHECK_VALUE(positions.size(0) == spec->num_axes && positions.size(1) == T, "positions must be [", spec->num_axes, ", ", T,
                    "], got ", positions.sizes());
  Device on;
  c.add_to(on);
  on.add(q, "q");
  on.add(k_new, "k_new");
  on.add(v_new, "v_new");
  on.add(positions, "positions");
  on.add(cu, "cu_seqlens_q");
  on.add(q_out, "q_out");
  const Call call(on);
  Tensor qo = made(q_out, q.sizes(), q, at::kBFloat16);
  const int rc = abi.rope_append(in(q), in(k_new), in(v_new), out(qo), ints(positions), spec, bytes(k_pool), bytes(v_pool),
                                 bytes(kv_scales), ints(cu), ints(seq_lens), ints(block_table), c.S, size32(T), size32(q.size(1)), c.Hkv,
                                 c.d, c.page_size, c.max_pages, c.num_pages, call.stream);
  return {rc, qo};
}

std::tuple<int, Tensor, Tensor> gather(const Tensor& k_pool, const Tensor& v_pool, const Tensor& kv_scales, const Tensor& block_table,
                                       const Tensor& seq_lens, const Tensor& cu, std::optional<int64_t> total_rows, const Maybe& k_out,
                                       const Maybe& v_out) {
  const Cache c(k_pool, v_pool, kv_scales, block_table, seq_lens);
  c.require_cu(cu, "cu_seqlens_k");
  require(k_out, "k_out", at::kBFloat16, 3);
  require(v_out, "v_out", at::kBFloat16, 3);
  TORCH_CHECK_VALUE(k_out.has_value() == v_out.has_value(), "give both k_out and v_out, or neither");
  if (k_out) {
    TORCH_CHECK_VALUE(k_out->size(1) == c.Hkv && k_out->size(2) == c.d && v_out->sizes() == k_out->sizes() &&
                          (!total_rows || *total_rows == k_out->size(0)),
                      "k_out / v_out must be [rows, ", c.Hkv, ", ", c.d, "] alike, got ", k_out->sizes(), " / ", v_out->sizes());
  } else {
    TORCH_CHECK_VALUE(total_rows && *total_rows >= 0, "total_rows (or k_out and v_out) is needed");
  }
  const int64_t rows = k_out ? k_out->size(0) : *total_rows;
  Device on;
  c.add_to(on);
  on.add(cu, "cu_seqlens_k");
  on.add(k_out, "k_out");
  on.add(v_out, "v_out");
  const Call call(on);
  Tensor ko = made(k_out, {rows, c.Hkv, c.d}, k_pool, at::kBFloat16), vo = made(v_out, {rows, c.Hkv, c.d}, k_pool, at::kBFloat16);
  const int rc = abi.gather(bytes(k_pool), bytes(v_pool), bytes(kv_scales), ints(block_table), ints(seq_lens), ints(cu), out(ko), out(vo),
                            c.S, size32(rows), c.Hkv, c.d, c.page_size, c.max_pages, c.num_pages, call.stream);
  return {rc, ko, vo};
}

std::tuple<int, Tensor, Tensor> decode(const Tensor& q, const Tensor& k_pool, const Tensor& v_pool, const Tensor& kv_scales,
                                       const Tensor& block_table, const Tensor& seq_lens, std::optional<double> scale,
                                       const Maybe& workspace, const Maybe& o, const Maybe& lse) {
  const Cache c(k_pool, v_pool, kv_scales, block_table, seq_lens);
  require(q, "q", at::kBFloat16, 3);
  require(o, "out", at::kBFloat16, 3);
  require(lse, "lse", at::kFloat, 2);
  TORCH_CHECK_VALUE(q.size(0) == c.S && q.size(2) == c.d, "q must be [", c.S, ", Hq, ", c.d, "], got ", q.sizes());
  const int Hq = size32(q.size(1));
  TORCH_CHECK_VALUE(!o || o->sizes() == q.sizes(), "out's shape differs from q's ", q.sizes());
  TORCH_CHECK_VALUE(!lse || (lse->size(0) == c.S && lse->size(1) == Hq), "lse must be [", c.S, ", ", Hq, "]");
  TORCH_CHECK_VALUE(!workspace || workspace->is_contiguous(), "workspace must be contiguous");
  Device on;
  c.add_to(on);
  on.add(q, "q");
  on.add(workspace, "workspace");
  on.add(o, "out");
  on.add(lse, "lse");
  const Call call(on);
  Maybe ws = workspace;
  if (!ws) {
    const size_t need = abi.decode_bytes(c.S, Hq, c.Hkv, c.d, c.max_pages, c.page_size);
    if (need > 0) ws = at::empty({static_cast<int64_t>(need)}, q.options().dtype(at::kByte));
  }
  Tensor oo = made(o, q.sizes(), q, at::kBFloat16), ol = made(lse, {c.S, Hq}, q, at::kFloat);
  const float s = scale ? static_cast<float>(*scale) : static_cast<float>(1.0 / std::sqrt(static_cast<double>(c.d)));
  const int rc = abi.decode(in(q), bytes(k_pool), bytes(v_pool), bytes(kv_scales), ints(block_table), ints(seq_lens), c.page_size, out(oo),
                            static_cast<float*>(ol.data_ptr()), c.S, Hq, c.Hkv, c.d, c.max_pages, c.num_pages, s, ws ? ws->data_ptr() : nullptr,
                            ws ? ws->nbytes() : 0, call.stream);
  return {rc, oo, ol};
}

}  // namespace

PYBIND11_MODULE(_attn_torch, m) {
  m.def("bind", &bind);
  m.def("rope", &rope);
  m.def("append", &append);
  m.def("rope_append", &rope_append);
  m.def("gather", &gather);
  m.def("decode", &decode);
}
