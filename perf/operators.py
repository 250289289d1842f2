"""What is measured of the 8-bit paged cache and of the rotary positions with several axes.

Five operators, each a call a user makes next to the bf16 ones:

* ``rope``    ``api.attn_rope``: rotary positions with several axes on queries and keys (``inverse``: their gradient)
* ``append``  ``api.paged_kv_append_fp8``: new K/V quantised (e4m3, one power-of-two scale a row) as they are written
* ``step``    ``api.paged_rope_append_fp8``: the rotation of q and k, the quantisation and the write, in one call
* ``gather``  ``api.paged_kv_gather_fp8``: the 8-bit cache read back as bf16 rows
* ``decode``  ``api.paged_attn_decode_fp8``: attention of one new token a sequence over the 8-bit cache

The cache: pools [num_pages, page_size, Hkv, d] of e4m3 codes and kv_scales [num_pages, Hkv, page_size, 2] of e8m0
exponents (K's, then V's).  A row x of d values has the exponent e, the smallest with max|x| <= 448 * 2^e (limited to
-100 .. 119), and the codes RN(x * 2^-e).
"""

import math

import torch

own = False

E_MIN, E_MAX = -100, 119


# ----------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # rotary on the q and k of a prefill batch in [B, H, N, d] (the causal MHA prefill's shapes), text/image/video axes
        dict(name="rope prefill", op="rope", layout="bhnd", B=4, N=2048, Hq=16, Hkv=16, d=128, rot=128, axes=3, pairs="half",
             spread=False, inverse=False, far=4096),
        # the gradient of a vision tower's rotary: packed tokens, two axes, half of each head rotated, odd sizes
        dict(name="rope gradient", op="rope", layout="thd", B=1, N=1237, Hq=12, Hkv=4, d=64, rot=32, axes=2, pairs="adjacent",
             spread=False, inverse=True, far=700),
        # a decode step of 64 sequences: one new token each, rotated, quantised, written
        dict(name="step decode", op="step", S=64, q_min=1, q_max=1, ctx_min=511, ctx_max=8191, Hq=32, Hkv=8, d=128, page=16, rot=128,
             axes=3, pairs="half", spread=True, far=1 << 20),
        # a serving step that hands each of 16 sequences a prompt chunk (the chunked-prefill shapes)
        dict(name="step chunks", op="step", S=16, q_min=256, q_max=2048, ctx_min=0, ctx_max=6144, Hq=32, Hkv=8, d=128, page=16, rot=128,
             axes=3, pairs="half", spread=False, far=8192),
        # the same chunks where positions are already in K
        dict(name="append chunks", op="append", S=16, q_min=256, q_max=2048, ctx_min=0, ctx_max=6144, Hkv=8, d=128, page=16),
        # short ragged chunks into larger pages, small heads
        dict(name="append ragged", op="append", S=5, q_min=1, q_max=40, ctx_min=0, ctx_max=300, Hkv=2, d=64, page=64),
        # a whole 8-bit cache read back for a chunked prefill
        dict(name="gather batch", op="gather", S=16, len_min=512, len_max=8192, Hkv=8, d=128, page=16),
        # four short sequences read back
        dict(name="gather small", op="gather", S=4, len_min=1, len_max=1024, Hkv=4, d=64, page=32),
        # one sequence, one token: the lowest latency
        dict(name="decode one", op="decode", S=1, len_min=1000, len_max=1000, Hq=32, Hkv=8, d=128, page=16),
        # the small decode batch
        dict(name="decode small", op="decode", S=4, len_min=256, len_max=1024, Hq=32, Hkv=8, d=128, page=16),
        # the serving batch: 64 sequences of 512 to 8192 tokens
        dict(name="decode batch", op="decode", S=64, len_min=512, len_max=8192, Hq=32, Hkv=8, d=128, page=16),
        # long caches, few sequences, many query heads a KV head, d = 64, larger pages
        dict(name="decode long", op="decode", S=3, len_min=70001, len_max=131072, Hq=32, Hkv=2, d=64, page=64),
    ]


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))

    op = rng.choice(["rope", "step", "append", "gather", "decode", "decode"])
    d = rng.choice([64, 128, 128])
    page = rng.choice([16, 16, 32, 48, 64, 128, 256])
    Hkv = rng.choice([1, 2, 3, 4, 8, 8])
    group = rng.choice([1, 2, 4, 4, 7, 8, 16])
    turn = dict(rot=rng.choice([d, d, d // 2, 48]), axes=rng.choice([1, 2, 3, 3, 4]), pairs=rng.choice(["half", "half", "adjacent"]),
                spread=rng.random() < 0.4, far=log(16, 1 << 20))
    if op == "rope":
        B = rng.choice([1, 1, 2, 4])
        return dict(op=op, layout="thd" if B == 1 and rng.random() < 0.5 else "bhnd", B=B, N=log(1, 8192 // B), Hq=min(16, Hkv * group),
                    Hkv=Hkv, d=d, inverse=rng.random() < 0.4, **turn)
    S = log(1, 64)
    if op in ("step", "append"):
        most = log(1, max(1, 16384 // S))
        case = dict(op=op, S=S, q_min=max(1, most // 8), q_max=most, ctx_min=0, ctx_max=log(1, 4096), Hkv=Hkv, d=d, page=page)
        return dict(case, Hq=min(32, Hkv * group), **turn) if op == "step" else case
    if op == "gather":
        most = log(1, 65536 // S)
        return dict(op=op, S=S, len_min=max(1, most // 16), len_max=most, Hkv=Hkv, d=d, page=page)
    most = log(1, min(131072, 262144 // S))
    return dict(op=op, S=S, len_min=max(1, most // 8), len_max=most, Hq=Hkv * group, Hkv=Hkv, d=d, page=page)


def _between(lo, hi, n):
    """n lengths spread over lo .. hi, both ends among them where n > 1; the same for every seed, so that the work is known."""
    return [hi if n == 1 or i == n - 1 else lo + int((hi - lo + 1) * ((i * 0.6180339887498949) % 1.0)) for i in range(n)]


def _chunks(case):
    q = _between(case["q_min"], case["q_max"], case["S"])
    ctx = _between(case["ctx_min"], case["ctx_max"], case["S"])[::-1]
    return q, [a + b for a, b in zip(q, ctx)]


def work(case):
    d, op = case["d"], case["op"]
    if op == "rope":
        rows = case["B"] * case["N"] * (case["Hq"] + case["Hkv"])
        return {"bytes": 4.0 * rows * d + 4.0 * case["axes"] * case["B"] * case["N"], "flops": 3.0 * rows * case["rot"]}
    if op in ("step", "append"):
        q, lens = _chunks(case)
        T = sum(q)
        n = 2.0 * T * case["Hkv"] * (2 * d + d + 1) + 8.0 * case["S"] + 4.0 * T / case["page"]
        f = 4.0 * T * case["Hkv"] * d
        if op == "step":
            n += 4.0 * T * case["Hq"] * d + 4.0 * case["axes"] * T
            f += 3.0 * T * (case["Hq"] + case["Hkv"]) * case["rot"]
        return {"bytes": n, "flops": f}
    lens = _between(case["len_min"], case["len_max"], case["S"])
    L, pages = sum(lens), sum(-(-n // case["page"]) for n in lens)
    if op == "gather":
        return {"bytes": 2.0 * L * case["Hkv"] * (d + 1 + 2 * d) + 4.0 * pages, "flops": 2.0 * L * case["Hkv"] * d}
    return {"bytes": 2.0 * L * case["Hkv"] * (d + 1) + case["S"] * case["Hq"] * (4.0 * d + 4) + 4.0 * pages + 4.0 * case["S"],
            "flops": 4.0 * L * case["Hq"] * d}


# ----------------------------------------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _rows(g, *shape):
    """bf16 rows as attention meets them: normal values whose size differs from row to row."""
    x = torch.randn(*shape, generator=g, device="cuda")
    return x.mul_(torch.exp(0.5 * torch.randn(*shape[:-1], 1, generator=g, device="cuda"))).to(torch.bfloat16)


def _sections(case):
    """The frequencies of each axis: the first axis (time) a little fewer, as video models share them out."""
    half, a = case["rot"] // 2, case["axes"]
    rest = -(-half // a)
    return [half - rest * (a - 1)] + [rest] * (a - 1)


def _axis_of(case):
    s = _sections(case)
    if not case["spread"]:
        return [a for a, n in enumerate(s) for _ in range(n)]
    left, order = list(s), []  # in turn, while an axis has frequencies left
    while len(order) < sum(s):
        for a in range(len(s)):
            if left[a]:
                left[a] -= 1
                order.append(a)
    return order


def _tables(case, g, lens):
    """A block table over a seeded permutation of exactly the pages in use, with -1 behind each sequence's own."""
    page = case["page"]
    need = torch.tensor([-(-n // page) for n in lens])
    width = max(1, int(need.max()))
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    used = torch.arange(width)[None, :] < need[:, None]
    total = max(1, int(need.sum()))
    table[used.cuda()] = torch.randperm(total, generator=g, device="cuda")[:int(need.sum())].to(torch.int32)
    return table, total


def _pools(case, g, num_pages, filled):
    """8-bit pools and their scales; `filled`: with rows that were quantised, else with codes that nothing may read."""
    shape = (num_pages, case["page"], case["Hkv"], case["d"])
    scales = torch.full((num_pages, case["Hkv"], case["page"], 2), 255, dtype=torch.uint8, device="cuda")
    pools = []
    for i in range(2):
        if filled:
            codes, e = _quantise(_rows(g, *shape).float())
            scales[..., i] = (e + 127).to(torch.uint8).transpose(1, 2)
        else:
            codes = torch.full(shape, 0.5, device="cuda").to(torch.float8_e4m3fn)
            scales[..., i] = 127
        pools.append(codes)
    return pools[0], pools[1], scales.view(torch.float8_e8m0fnu)


def prepare(case, seed):
    g, d, op = _generator(seed), case["d"], case["op"]
    s = dict(case, scale=float(torch.tensor(d ** -0.5, dtype=torch.float32)))
    if "rot" in case:
        j = torch.arange(case["rot"] // 2, dtype=torch.float64)
        s["inv_freq"] = (10000.0 ** (-2.0 * j / case["rot"])).cuda()
        s["axis_of"] = torch.tensor(_axis_of(case), device="cuda")
        s["turn"] = {}  # the framework's description of the rotation, which a program makes once
    if op == "rope":
        B, N = case["B"], case["N"]
        shape = (lambda h: (N, h, d)) if case["layout"] == "thd" else (lambda h: (B, h, N, d))
        s["q"], s["k"] = _rows(g, *shape(case["Hq"])), _rows(g, *shape(case["Hkv"]))
        where = (case["axes"], N) if case["layout"] == "thd" else (case["axes"], B, N)
        s["positions"] = torch.randint(0, case["far"], where, generator=g, device="cuda", dtype=torch.int32)
        return s
    if op in ("step", "append"):
        q, lens = _chunks(case)
        T = sum(q)
        s["block_table"], pages = _tables(case, g, lens)
        s["cu"] = torch.tensor([sum(q[:i]) for i in range(len(q) + 1)], dtype=torch.int32, device="cuda")
        s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["k_new"], s["v_new"] = _rows(g, T, case["Hkv"], d), _rows(g, T, case["Hkv"], d)
        s["k_pool"], s["v_pool"], s["kv_scales"] = _pools(case, g, pages, False)
        if op == "step":
            s["q"] = _rows(g, T, case["Hq"], d)
            s["positions"] = torch.randint(0, case["far"], (case["axes"], T), generator=g, device="cuda", dtype=torch.int32)
        return s
    lens = _between(case["len_min"], case["len_max"], case["S"])
    s["block_table"], pages = _tables(case, g, lens)
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["k_pool"], s["v_pool"], s["kv_scales"] = _pools(case, g, pages, True)
    if op == "gather":
        s["cu"] = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
        s["rows"] = sum(lens)
    else:
        s["q"] = _rows(g, case["S"], case["Hq"], d)
    return s


# ----------------------------------------------------------------------------------------------- one pass

def run(state):
    return {"rope": _rope, "step": _step, "append": _append, "gather": _gather, "decode": _decode}[state["op"]](state)


def _spec(s):
    """The framework's description of the rotation: made once, and kept as a program keeps it."""
    if "spec" not in s["turn"]:
        from attention_flashattention_fwd_04_b200 import api
        sections = _sections(s)
        s["turn"]["spec"] = api.rope_spec(s["d"], sections, theta=10000.0, rot_dim=s["rot"], adjacent_pairs=s["pairs"] == "adjacent",
                                          interleaved_sections=s["spread"])
    return s["turn"]["spec"]


def _rope(s):
    if own:
        from attention_flashattention_fwd_04_b200 import api
        return api.attn_rope(s["q"], s["k"], s["positions"], _spec(s), inverse=s["inverse"])
    cos, sin = _angles(s)
    head = 1
    return _rotate(s["q"], cos, sin, s, head).to(torch.bfloat16), _rotate(s["k"], cos, sin, s, head).to(torch.bfloat16)


def _step(s):
    if own:
        from attention_flashattention_fwd_04_b200 import api
        q = api.paged_rope_append_fp8(s["q"], s["k_new"], s["v_new"], s["positions"], _spec(s), s["k_pool"], s["v_pool"], s["kv_scales"],
                                      s["block_table"], s["cu"], s["seq_lens"])
        return q, s["k_pool"], s["v_pool"], s["kv_scales"]
    cos, sin = _angles(s)
    _write(s, _rotate(s["k_new"], cos, sin, s, 1), s["v_new"].float())
    return _rotate(s["q"], cos, sin, s, 1).to(torch.bfloat16), s["k_pool"], s["v_pool"], s["kv_scales"]


def _append(s):
    if own:
        from attention_flashattention_fwd_04_b200 import api
        api.paged_kv_append_fp8(s["k_new"], s["v_new"], s["k_pool"], s["v_pool"], s["kv_scales"], s["block_table"], s["cu"], s["seq_lens"])
    else:
        _write(s, s["k_new"].float(), s["v_new"].float())
    return s["k_pool"], s["v_pool"], s["kv_scales"]


def _gather(s):
    if own:
        from attention_flashattention_fwd_04_b200 import api
        return api.paged_kv_gather_fp8(s["k_pool"], s["v_pool"], s["kv_scales"], s["block_table"], s["seq_lens"], s["cu"], s["rows"])
    row = torch.arange(s["rows"], device="cuda")
    seq = torch.searchsorted(s["cu"], row, right=True) - 1
    t = row - s["cu"][seq]
    page, slot = s["block_table"][seq, t // s["page"]].long(), t % s["page"]
    two = _two(s["kv_scales"].view(torch.uint8)[page, :, slot].to(torch.int32) - 127)  # [rows, Hkv, 2]
    k = s["k_pool"].view(torch.uint8)[page, slot].view(torch.float8_e4m3fn).float() * two[..., :1]
    v = s["v_pool"].view(torch.uint8)[page, slot].view(torch.float8_e4m3fn).float() * two[..., 1:]
    return k.to(torch.bfloat16), v.to(torch.bfloat16)


def _decode(s):
    if own:
        from attention_flashattention_fwd_04_b200 import api
        return api.paged_attn_decode_fp8(s["q"], s["k_pool"], s["v_pool"], s["kv_scales"], s["block_table"], s["seq_lens"], s["scale"])
    S, Hq, d = s["q"].shape
    Hkv, page = s["Hkv"], s["page"]
    table = s["block_table"].clamp(min=0).long()
    L = table.shape[1] * page
    two = _two(s["kv_scales"].view(torch.uint8)[table].to(torch.int32) - 127)  # [S, pages, Hkv, page, 2]
    two = two.transpose(1, 2).reshape(S, Hkv, L, 2)
    k = s["k_pool"].view(torch.uint8)[table].view(torch.float8_e4m3fn).reshape(S, L, Hkv, d).transpose(1, 2).float() * two[..., :1]
    scores = torch.matmul(s["q"].float().view(S, Hkv, Hq // Hkv, d), k.transpose(2, 3)) * s["scale"]  # [S, Hkv, group, L]
    del k
    hidden = torch.arange(L, device="cuda")[None, :] >= s["seq_lens"][:, None]
    scores = scores.masked_fill(hidden[:, None, None, :], float("-inf"))
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    v = s["v_pool"].view(torch.uint8)[table].view(torch.float8_e4m3fn).reshape(S, L, Hkv, d).transpose(1, 2).float() * two[..., 1:]
    v = v.masked_fill(hidden[:, None, :, None], 0.0)
    o = torch.matmul(p, v) / total
    return o.view(S, Hq, d).to(torch.bfloat16), (top + torch.log(total)).view(S, Hq)


def _angles(s):
    """cos and sin [..., rot / 2] of the angles positions[axis of j] * inv_freq[j]; the angles of far positions need 64 bits."""
    angle = s["positions"].double()[s["axis_of"]].movedim(0, -1) * s["inv_freq"]
    return torch.cos(angle).float(), torch.sin(angle).float()


def _rotate(x, cos, sin, s, head):
    """x with the pairs of its first rot values turned (back, where `inverse`), in 32 bits."""
    cos, sin = cos.unsqueeze(head), sin.unsqueeze(head)
    if s.get("inverse"):
        sin = -sin
    x, rot = x.float(), s["rot"]
    if s["pairs"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., rot:]], -1)
    a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), x[..., rot:]], -1)


def _quantise(x):
    """Codes and exponents [..., d], [...] of the rows of x (32 bits)."""
    m, e = torch.frexp(x.abs().amax(-1))  # amax = m * 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(m == 0, E_MIN, e).clamp(E_MIN, E_MAX)
    return (x * _two(-e).unsqueeze(-1)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn), e


def _two(e):
    """2^e (32 bits, -126 <= e <= 127) by the float's exponent: pow() and exp2() may be off in the last bit, and a bf16 value is often
    just between two codes."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _write(s, k, v):
    """Quantises the rows of k and v and puts them where the block table says."""
    row = torch.arange(k.shape[0], device="cuda")
    seq = torch.searchsorted(s["cu"], row, right=True) - 1
    t = s["seq_lens"][seq] - (s["cu"][seq + 1] - row)
    page, slot = s["block_table"][seq, t // s["page"]].long(), t % s["page"]
    scales = s["kv_scales"].view(torch.uint8)
    for i, (x, pool) in enumerate(((k, s["k_pool"]), (v, s["v_pool"]))):
        codes, e = _quantise(x)
        pool.view(torch.uint8)[page, slot] = codes.view(torch.uint8)
        scales[page, :, slot, i] = (e + 127).to(torch.uint8)


# ----------------------------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        thd = case["layout"] == "thd"
        return tuple(_exact_turn(s, x, 0 if thd else 2, -1.0 if case["inverse"] else 1.0) for x in (s["q"], s["k"]))
    if op in ("step", "append"):
        out = []
        k = s["k_new"].double()
        if op == "step":
            out.append(_exact_turn(s, s["q"], 0, 1.0))
            k = _exact_turn(s, s["k_new"], 0, 1.0)
        pools = [s["k_pool"].double(), s["v_pool"].double()]
        scales = s["kv_scales"].double()
        cu, lens, table = s["cu"].tolist(), s["seq_lens"].tolist(), s["block_table"].long()
        for i, n in enumerate(lens):
            new = cu[i + 1] - cu[i]
            at = torch.arange(n - new, n, device="cuda")
            page, slot = table[i, torch.div(at, case["page"], rounding_mode="floor")], torch.remainder(at, case["page"])
            for j, x in enumerate((k, s["v_new"].double())):
                codes, e = _exact_codes(x[cu[i]:cu[i + 1]])
                pools[j].index_put_((page, slot), codes)
                scales[page, :, slot, j] = _exact_two(e)
        return tuple(out + pools + [scales])
    lens, cu = s["seq_lens"].tolist(), 0
    o = []
    for i, n in enumerate(lens):
        pages = s["block_table"][i, :-(-n // case["page"])].long()
        e = s["kv_scales"].double()[pages].permute(0, 2, 1, 3).reshape(-1, case["Hkv"], 2)[:n]
        k = s["k_pool"][pages].double().reshape(-1, case["Hkv"], case["d"])[:n] * e[..., 0, None]
        v = s["v_pool"][pages].double().reshape(-1, case["Hkv"], case["d"])[:n] * e[..., 1, None]
        if op == "gather":
            o.append((k, v))
            continue
        q = s["q"][i].double().view(case["Hkv"], -1, case["d"])
        z = torch.einsum("hgd,lhd->hgl", q, k) * s["scale"]
        lse = torch.logsumexp(z, -1)
        o.append((torch.einsum("hgl,lhd->hgd", torch.exp(z - lse[..., None]), v).reshape(-1, case["d"]), lse.reshape(-1)))
    if op == "gather":
        return torch.cat([k for k, _ in o]), torch.cat([v for _, v in o])
    return torch.stack([a for a, _ in o]), torch.stack([b for _, b in o])


def _exact_turn(s, x, token, sign):
    """The rotation as complex numbers: pair j of a token at position p is multiplied by exp(i * sign * p * inv_freq[j])."""
    x = x.double()
    half = s["rot"] // 2
    angle = torch.stack([s["positions"][a].double() * s["inv_freq"][j] for j, a in enumerate(_axis_of(s))], -1)
    w = torch.polar(torch.ones_like(angle), sign * angle)
    w = w[:, None, :] if token == 0 else w[:, None, :, :]
    if s["pairs"] == "half":
        first, second = list(range(half)), list(range(half, 2 * half))
    else:
        first, second = list(range(0, 2 * half, 2)), list(range(1, 2 * half, 2))
    z = torch.complex(x[..., first], x[..., second]) * w
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_two(e):
    """2^e of whole numbers e, in 64 bits, by the number's exponent."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_codes(x):
    """The e4m3 values and the exponents of the rows of x, from the format's definition (nothing of the case is near its limits)."""
    top = x.abs().amax(-1)
    e = torch.ceil(torch.log2(top.clamp(min=1e-30) / 448.0))
    e = torch.where(top <= 448.0 * _exact_two(e - 1), e - 1, e)
    e = torch.where(top > 448.0 * _exact_two(e), e + 1, e)
    e = torch.where(top == 0, torch.full_like(e, float(E_MIN)), e)
    y = x / _exact_two(e)[..., None]
    binade = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    binade = torch.where(y.abs() < _exact_two(binade), binade - 1, binade).clamp(min=-6)
    binade = torch.where(y.abs() >= _exact_two(binade + 1), binade + 1, binade)
    step = _exact_two(binade - 3)
    return torch.round(y / step) * step, e
