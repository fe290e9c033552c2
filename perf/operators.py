"""Cases of the attention half of a decoder layer: the operators between the residual stream and the expert layer.

  norm       residual addition and root-mean-square norm, output in 16 bits or in e4m3 with a scale per 128 columns
  quantize   a 16-bit matrix to e4m3, a scale per row and 128 columns (activations) or per 128 x 128 block (weights)
  linear     product of two e4m3 matrices with those scales
  rope       rotary positions on q and k, with k and v appended to the paged cache
  attention  a chunk of new tokens of each sequence over the paged cache

Every operator has a plain form in elementary torch operations (32 bits, rounded once at the end) and `exact`, its
definition in 64 bits.  Sequence lengths and page orders of a case come from the case itself; values come from the seed.
"""
import math
import random

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
E4M3_MAX = 448.0
MIN_SCALE = 2.0 ** -100
GROUP = 128


def listed():
    return [
        # one token of the 8x7B-shaped layer: the norm before the experts at batch 1, where only latency counts
        {"name": "norm_one_token", "op": "norm", "rows": 1, "cols": 4096, "dtype": "fp16", "residual": True, "fp8": False},
        # a prefill batch of the 8x22B-shaped layer: the norm before the query/key/value projection
        {"name": "norm_fp8_prefill", "op": "norm", "rows": 8192, "cols": 6144, "dtype": "bf16", "residual": True,
         "fp8": True},
        # the attention's output of an odd decode batch, before the output projection
        {"name": "quantize_decode_odd", "op": "quantize", "rows": 97, "cols": 4096, "dtype": "fp16", "blocks": False},
        # the query/key/value weight of the 8x22B-shaped layer, as it is loaded
        {"name": "quantize_weight", "op": "quantize", "rows": 8192, "cols": 6144, "dtype": "bf16", "blocks": True},
        # the query/key/value projection (32 + 8 + 8 heads of 128) of a small decode batch
        {"name": "linear_decode", "op": "linear", "m": 8, "n": 6144, "k": 4096, "dtype": "fp16"},
        # the output projection of a ragged chunk
        {"name": "linear_chunk_odd", "op": "linear", "m": 509, "n": 4096, "k": 4096, "dtype": "bf16"},
        # the query/key/value projection (48 + 8 + 8 heads) of a prefill batch
        {"name": "linear_prefill", "op": "linear", "m": 8192, "n": 8192, "k": 6144, "dtype": "fp16"},
        # one new token of each of 128 sequences
        {"name": "rope_decode", "op": "rope", "batch": 128, "q_min": 1, "q_max": 1, "kv_min": 1, "kv_max": 8192, "lens": 1,
         "heads": 32, "kv_heads": 8, "head_dim": 128, "page_size": 16, "heads_first": False, "rotary_dim": 128,
         "interleaved": False, "scaling": "none", "dtype": "fp16"},
        # chunks of long prompts: interleaved pairs on half of the head, scaled for a long context
        {"name": "rope_prefill", "op": "rope", "batch": 5, "q_min": 1111, "q_max": 2048, "kv_min": 2048, "kv_max": 65536,
         "lens": 2, "heads": 48, "kv_heads": 8, "head_dim": 128, "page_size": 64, "heads_first": True, "rotary_dim": 64,
         "interleaved": True, "scaling": "yarn", "dtype": "bf16"},
        # one token of one short conversation: latency
        {"name": "attention_one_token", "op": "attention", "batch": 1, "q_min": 1, "q_max": 1, "kv_min": 1021,
         "kv_max": 1021, "lens": 3, "heads": 32, "kv_heads": 8, "head_dim": 128, "page_size": 16, "heads_first": False,
         "causal": True, "window": 0, "dtype": "fp16"},
        # a decode batch whose sequences run from a few tokens to a long document
        {"name": "attention_decode_ragged", "op": "attention", "batch": 24, "q_min": 1, "q_max": 1, "kv_min": 17,
         "kv_max": 65536, "lens": 4, "heads": 48, "kv_heads": 8, "head_dim": 128, "page_size": 64, "heads_first": True,
         "causal": True, "window": 0, "dtype": "bf16"},
        # chunks of prompts over what the cache holds already
        {"name": "attention_prefill", "op": "attention", "batch": 4, "q_min": 1500, "q_max": 2048, "kv_min": 4096,
         "kv_max": 16384, "lens": 5, "heads": 32, "kv_heads": 8, "head_dim": 128, "page_size": 32, "heads_first": False,
         "causal": True, "window": 0, "dtype": "fp16"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "quantize", "linear", "rope", "attention", "attention"])
    dtype = rng.choice(["fp16", "bf16"])
    if op == "norm":
        cols = rng.choice([_log(rng, 64, 8192), 8 * _log(rng, 8, 1024), rng.choice([2048, 4096, 6144])])
        return {"op": op, "rows": _log(rng, 1, 4096), "cols": cols, "dtype": dtype,
                "residual": rng.random() < 0.7, "fp8": rng.random() < 0.5}
    if op == "quantize":
        cols = rng.choice([_log(rng, 64, 8192), 8 * _log(rng, 8, 1024), rng.choice([2048, 4096, 6144])])
        return {"op": op, "rows": _log(rng, 1, 4096), "cols": cols, "dtype": dtype, "blocks": rng.random() < 0.4}
    if op == "linear":
        n = rng.choice([_log(rng, 128, 8192), 128 * rng.randint(1, 64)])
        k = rng.choice([16 * _log(rng, 4, 384), 128 * rng.randint(1, 48)])
        return {"op": op, "m": _log(rng, 1, 8192), "n": n, "k": k, "dtype": dtype}
    heads, kv_heads = rng.choice([(32, 8), (48, 8), (16, 16), (16, 2), (8, 1), (12, 4)])
    c = {"op": op, "batch": _log(rng, 1, 32), "lens": rng.randint(10, 1 << 20), "heads": heads, "kv_heads": kv_heads,
         "head_dim": rng.choice([64, 128, 128]), "page_size": rng.choice([16, 32, 64, 128]),
         "heads_first": rng.random() < 0.5, "dtype": dtype}
    # new tokens a sequence: one, a few (drafted tokens), or a chunk
    c["q_max"] = rng.choice([1, 1, rng.randint(2, 8), _log(rng, 16, 1024)])
    c["q_min"] = rng.randint(1, c["q_max"]) if c["q_max"] > 1 else 1
    # the plain form pads every sequence to the longest: at most 2^27 keys and 2^30 scores in all
    most = min(32768, (1 << 27) // (c["batch"] * kv_heads * c["head_dim"]) * 4, (1 << 30) // (c["batch"] * heads * c["q_max"]))
    c["kv_max"] = _log(rng, 64, max(65, most))
    c["kv_min"] = rng.randint(1, c["kv_max"])
    if op == "rope":
        c["rotary_dim"] = rng.choice([c["head_dim"], c["head_dim"], c["head_dim"] // 2, 24])
        c["interleaved"] = rng.random() < 0.5
        c["scaling"] = rng.choice(["none", "linear", "ntk", "yarn"])
        return c
    c["causal"] = rng.random() < 0.8
    c["window"] = rng.choice([0, 0, _log(rng, 8, 4096)]) if c["causal"] else 0
    return c


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _lens(case):
    """Sequence lengths: new tokens q and, with them, kv tokens in the cache.  A sequence that is shorter than its chunk
    is all new."""
    r = random.Random(case["lens"])
    kv = [_log(r, case["kv_min"], case["kv_max"]) for _ in range(case["batch"])]
    kv[r.randrange(len(kv))] = case["kv_max"]
    q = [min(n, r.randint(case["q_min"], case["q_max"])) for n in kv]
    return q, kv


def _frequencies(case):
    """Radians a position of each rotated pair, in 64 bits, and the factor on cos and sin."""
    d, base, s = case["rotary_dim"], 1e6, 8.0
    half = d // 2
    f = [base ** (-2.0 * i / d) for i in range(half)]
    if case["scaling"] == "linear":
        return [x / s for x in f], 1.0
    if case["scaling"] == "ntk":
        b = base * s ** (d / (d - 2.0))
        return [b ** (-2.0 * i / d) for i in range(half)], 1.0
    if case["scaling"] == "yarn":
        turn = lambda n: d * math.log(4096.0 / (n * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(turn(32.0)), 0), min(math.ceil(turn(1.0)), d - 1)
        ramp = [min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0) for i in range(half)]
        return [x / s * t + x * (1.0 - t) for x, t in zip(f, ramp)], 0.1 * math.log(s) + 1.0
    return f, 1.0


def _cache(case, g, q_lens, kv_lens):
    """The paged cache, [pages][page_size][kv_heads][head_dim] in either order of storage, its pages handed out at
    random, and the page table.  rope: of each sequence only the pages that take new tokens are at hand (what it writes
    is then most of the cache); the table says -1 for the others.  attention: past a sequence's end its last page holds
    nothing, not even numbers."""
    dt, ps, hk, d = DTYPES[case["dtype"]], case["page_size"], case["kv_heads"], case["head_dim"]
    need = [-(-n // ps) for n in kv_lens]
    skip = [(n - m) // ps if case["op"] == "rope" else 0 for m, n in zip(q_lens, kv_lens)]
    have = [n - m for m, n in zip(skip, need)]
    pages = sum(have) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    at = torch.arange(max(need), device="cuda")[None, :] - torch.tensor(skip, device="cuda")[:, None]
    used = (at >= 0) & (at < torch.tensor(have, device="cuda")[:, None])
    at = at + torch.tensor([sum(have[:b]) for b in range(len(have))], device="cuda")[:, None]
    table = torch.where(used, order[at.clamp(0, pages - 1)], torch.full_like(order[:1], -1)).contiguous()

    def one():
        shape = (pages, hk, ps, d) if case["heads_first"] else (pages, ps, hk, d)
        t = torch.empty(shape, dtype=dt, device="cuda").normal_(generator=g)
        return t.permute(0, 2, 1, 3) if case["heads_first"] else t
    kc, vc = one(), one()
    if case["op"] == "rope":
        return kc, vc, table
    last = torch.tensor([n % ps for n in kv_lens], device="cuda")
    page = table[torch.arange(len(need), device="cuda"), torch.tensor(need, device="cuda") - 1].long()
    empty = (torch.arange(ps, device="cuda")[None, :] >= last[:, None]) & (last[:, None] > 0)
    rows = page[:, None] * ps + torch.arange(ps, device="cuda")[None, :]
    rows = rows[empty]
    for t in (kc, vc):
        t[rows // ps, rows % ps] = float("nan")
    return kc, vc, table


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op in ("norm", "quantize"):
        dt, rows, cols = DTYPES[case["dtype"]], case["rows"], case["cols"]
        groups = -(-cols // GROUP)
        st = {"case": case, "x": torch.empty((rows, cols), dtype=dt, device="cuda").normal_(generator=g)}
        st["x"][:, :: 61] *= 20  # a few outlier channels, as activations have them
        if op == "norm":
            st["w"] = (1 + 0.1 * torch.randn(cols, generator=g, device="cuda")).to(dt)
            st["y"] = None if case["fp8"] else torch.empty_like(st["x"])
            if case["residual"]:
                st["res"] = torch.empty((rows, cols), dtype=dt, device="cuda").normal_(generator=g) * 4
                st["res_out"] = torch.empty_like(st["x"])
        if op == "quantize" or case["fp8"]:
            st["q"] = torch.empty((rows, cols), dtype=torch.float8_e4m3fn, device="cuda")
            srows = -(-rows // GROUP) if case.get("blocks") else rows
            st["scale"] = torch.empty((srows, groups), dtype=torch.float32, device="cuda")
        return st
    if op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        kb, nb = -(-k // GROUP), -(-n // GROUP)

        def codes(rows):
            t = torch.empty((rows, k), dtype=torch.float16, device="cuda").normal_(generator=g)
            return (t * 120).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        spread = lambda r, s: s * torch.exp(0.4 * torch.randn((r, kb), generator=g, device="cuda"))  # noqa: E731
        return {"case": case, "a": codes(m), "sa": spread(m, 1e-2), "b": codes(n), "sb": spread(nb, 2e-4),
                "y": torch.empty((m, n), dtype=DTYPES[case["dtype"]], device="cuda"),
                "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    q_lens, kv_lens = _lens(case)
    tokens, dt, d = sum(q_lens), DTYPES[case["dtype"]], case["head_dim"]
    hq, hk = case["heads"], case["kv_heads"]
    off = [0]
    for n in q_lens:
        off.append(off[-1] + n)
    st = {"case": case, "q_offsets": torch.tensor(off, dtype=torch.int32, device="cuda"),
          "kv_lens": torch.tensor(kv_lens, dtype=torch.int32, device="cuda"),
          "status": torch.zeros(1, dtype=torch.int32, device="cuda"), "max_q_len": max(q_lens), "max_kv_len": max(kv_lens)}
    st["k_cache"], st["v_cache"], st["page_table"] = _cache(case, g, q_lens, kv_lens)
    # token -> its sequence and its position there
    seq = torch.repeat_interleave(torch.arange(len(q_lens), device="cuda"), torch.tensor(q_lens, device="cuda"))
    st["seq"] = seq
    st["pos"] = (torch.arange(tokens, device="cuda") - st["q_offsets"][seq].long()
                 + (st["kv_lens"] - st["q_offsets"].diff())[seq].long())
    if op == "rope":
        st["qkv"] = torch.empty((tokens, hq + 2 * hk, d), dtype=dt, device="cuda").normal_(generator=g)
        f, st["factor"] = _frequencies(case)
        st["freq"] = torch.tensor(f, dtype=torch.float64, device="cuda")
        # the same table as fractions of a turn, in units of 2^-64
        st["turns"] = (st["freq"] / (2 * math.pi) * 2.0 ** 64).round().to(torch.int64)
        st["q_out"] = torch.empty((tokens, hq, d), dtype=dt, device="cuda")
        # the slots that the new tokens take
        ps = case["page_size"]
        st["slot"] = st["page_table"][seq, st["pos"] // ps].long() * ps + st["pos"] % ps
    else:
        st["q"] = torch.empty((tokens, hq, d), dtype=dt, device="cuda").normal_(generator=g) * 1.5
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty((tokens, hq), dtype=torch.float32, device="cuda")
    return st


# ---------------------------------------------------------------- one pass
def run(state):
    if own:
        return _run_own(state)
    return {"norm": _norm, "quantize": _quantize, "linear": _linear, "rope": _rope, "attention": _attention}[state["case"]["op"]](state)


def _run_own(s):
    from any_precision_bit_pw_gb300 import pw
    c = s["case"]
    if c["op"] == "norm":
        pw.pw_add_rmsnorm(s["x"], s["w"], 1e-5, residual=s.get("res"), residual_out=s.get("res_out"), y=s["y"],
                          q=s.get("q"), scale=s.get("scale"))
        return [t for t in (s.get("res_out"), s["y"], s.get("q"), s.get("scale")) if t is not None]
    if c["op"] == "quantize":
        pw.pw_quantize_fp8(s["x"], s["q"], s["scale"], block_rows=GROUP if c["blocks"] else 1)
        return [s["q"], s["scale"]]
    if c["op"] == "linear":
        pw.pw_fp8_linear(s["a"], s["sa"], s["b"], s["sb"], s["y"], s["status"])
        return s["y"]
    if c["op"] == "rope":
        hq, hk = c["heads"], c["kv_heads"]
        q, k, v = s["qkv"][:, :hq], s["qkv"][:, hq:hq + hk], s["qkv"][:, hq + hk:]
        pw.pw_rope_append(q, k, v, s["turns"], s["k_cache"], s["v_cache"], s["page_table"], s["q_offsets"], s["kv_lens"],
                          s["q_out"], s["status"], interleaved=c["interleaved"], factor=s["factor"])
        return [s["q_out"], s["k_cache"], s["v_cache"]]
    if "ws" not in s:  # kept by the caller beside its cache
        n = pw.pw_paged_attention_workspace(s["q"].shape[0], c["batch"], c["heads"], c["kv_heads"], c["head_dim"])
        s["ws"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
    pw.pw_paged_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["q_offsets"], s["kv_lens"], s["out"],
                          s["ws"], s["status"], scale=c["head_dim"] ** -0.5, causal=c["causal"], window=c["window"],
                          max_q_len=s["max_q_len"], max_kv_len=s["max_kv_len"], lse=s["lse"])
    return [s["out"], s["lse"]]


def _to_e4m3(y, blocks):
    """Codes and scales: s = max(largest of the group / 448, 2^-100), code = e4m3(y / s)."""
    rows, cols = y.shape
    gr = GROUP if blocks else 1
    pad = torch.nn.functional.pad(y, (0, -cols % GROUP, 0, -rows % gr))
    t = pad.view(pad.shape[0] // gr, gr, pad.shape[1] // GROUP, GROUP)
    scale = (t.abs().amax(dim=(1, 3)) / E4M3_MAX).clamp(min=MIN_SCALE)
    t = (t / scale[:, None, :, None]).view(pad.shape)[:rows, :cols]
    return t, scale


def _norm(s):
    r = s["x"].float()
    got = []
    if "res" in s:
        r = r + s["res"].float()
        got.append(r.to(s["x"].dtype))
    y = r * torch.rsqrt((r * r).mean(dim=1, keepdim=True) + 1e-5) * s["w"].float()
    if s["y"] is not None:
        return got + [y.to(s["x"].dtype)]
    q, scale = _to_e4m3(y, False)
    return got + [q.to(torch.float8_e4m3fn), scale]


def _quantize(s):
    q, scale = _to_e4m3(s["x"].float(), s["case"]["blocks"])
    return [q.to(torch.float8_e4m3fn), scale]


def _spread(scale, rows, cols, block_rows):
    return scale.repeat_interleave(block_rows, 0)[:rows].repeat_interleave(GROUP, 1)[:, :cols]


def _linear(s):
    a = s["a"].float() * _spread(s["sa"], *s["a"].shape, 1)
    b = s["b"].float() * _spread(s["sb"], *s["b"].shape, GROUP)
    return torch.matmul(a, b.t()).to(s["y"].dtype)


def _rotate(x, cos, sin, rd, interleaved):
    head, rest = x[..., :rd], x[..., rd:]
    if interleaved:
        u, v = head[..., 0::2], head[..., 1::2]
        head = torch.stack((u * cos - v * sin, u * sin + v * cos), dim=-1).flatten(-2)
    else:
        u, v = head[..., : rd // 2], head[..., rd // 2:]
        head = torch.cat((u * cos - v * sin, u * sin + v * cos), dim=-1)
    return torch.cat((head, rest), dim=-1)


def _rope(s):
    c = s["case"]
    hq, hk, dt = c["heads"], c["kv_heads"], s["qkv"].dtype
    angle = s["pos"].float()[:, None] * s["freq"].float()[None, :]
    cos, sin = angle.cos()[:, None] * s["factor"], angle.sin()[:, None] * s["factor"]
    qk = _rotate(s["qkv"][:, : hq + hk].float(), cos, sin, c["rotary_dim"], c["interleaved"]).to(dt)
    at = (s["slot"] // c["page_size"], s["slot"] % c["page_size"])
    s["k_cache"][at] = qk[:, hq:]
    s["v_cache"][at] = s["qkv"][:, hq + hk:]
    return [qk[:, :hq], s["k_cache"], s["v_cache"]]


def _padded(s, t, dtype):
    """Keys or values of every sequence, [batch][longest][kv_heads][head_dim]: zeros where a sequence holds none."""
    c, n = s["case"], s["max_kv_len"]
    at = torch.arange(n, device="cuda")
    page = s["page_table"][:, at // c["page_size"]].clamp(min=0).long()
    got = t[page, (at % c["page_size"])[None, :]].to(dtype)
    return got.masked_fill((at[None, :] >= s["kv_lens"][:, None])[:, :, None, None], 0.0)


def _attend(s, dtype):
    c = s["case"]
    b, hq, hk, d, nq, nk = c["batch"], c["heads"], c["kv_heads"], c["head_dim"], s["max_q_len"], s["max_kv_len"]
    row = torch.arange(s["q"].shape[0], device="cuda") - s["q_offsets"][s["seq"]].long()
    q = torch.zeros((b, nq, hq, d), dtype=dtype, device="cuda")
    q[s["seq"], row] = s["q"].to(dtype)
    k, v = _padded(s, s["k_cache"], dtype), _padded(s, s["v_cache"], dtype)
    q = q.view(b, nq, hk, hq // hk, d).permute(0, 2, 3, 1, 4).reshape(b, hk, (hq // hk) * nq, d)
    score = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(d ** -0.5).view(b, hk, hq // hk, nq, nk)
    pos = torch.arange(nq, device="cuda")[None, :] + (s["kv_lens"] - s["q_offsets"].diff())[:, None]
    key = torch.arange(nk, device="cuda")
    seen = key[None, None, :] < s["kv_lens"][:, None, None]
    if c["causal"]:
        seen = seen & (key[None, None, :] <= pos[:, :, None])
        if c["window"]:
            seen = seen & (key[None, None, :] > pos[:, :, None] - c["window"])
    score.masked_fill_(~seen[:, None, None].expand_as(score), -math.inf)
    top = score.amax(dim=-1, keepdim=True)
    safe = top.masked_fill(top == -math.inf, 0.0)
    score = score.sub_(safe).exp_()
    total = score.sum(dim=-1, keepdim=True)
    out = torch.matmul(score.view(b, hk, -1, nk), v.permute(0, 2, 1, 3)).view(b, hk, hq // hk, nq, d)
    out = out / total.masked_fill(total == 0, 1.0)
    lse = (safe + total.log())[..., 0]
    out = out.permute(0, 3, 1, 2, 4).reshape(b, nq, hq, d)[s["seq"], row]
    return out, lse.permute(0, 3, 1, 2).reshape(b, nq, hq)[s["seq"], row]


def _attention(s):
    out, lse = _attend(s, torch.float32)
    return [out.to(s["q"].dtype), lse]


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "quantize"):
        r, got = s["x"].double(), []
        if op == "norm":
            if "res" in s:
                r = r + s["res"].double()
                got.append(r)
            var = torch.einsum("ij,ij->i", r, r) / r.shape[1]
            r = r / torch.sqrt(var + 1e-5)[:, None] * s["w"].double()
            if s["y"] is not None:
                return got + [r]
        rows, cols = r.shape
        height = GROUP if case.get("blocks") else 1
        # largest of each group: every value falls into the group of its row and column
        group = (torch.arange(rows, device="cuda") // height)[:, None] * s["scale"].shape[1] + (torch.arange(cols, device="cuda") // GROUP)[None]
        top = torch.zeros(s["scale"].numel(), dtype=torch.float64, device="cuda")
        top.scatter_reduce_(0, group.reshape(-1), r.abs().reshape(-1), "amax")
        scale = torch.maximum(top / E4M3_MAX, torch.full_like(top, MIN_SCALE))
        # the values before they are rounded to 8 bits, so that an error says what the rounding costs
        return got + [r / scale[group], scale.view(s["scale"].shape)]
    if op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        group = torch.arange(k, device="cuda") // GROUP
        block = torch.arange(n, device="cuda") // GROUP
        a = s["a"].double() * s["sa"].double()[:, group]
        b = s["b"].double() * s["sb"].double()[block][:, group]
        return a @ b.t()
    if op == "rope":
        hq, hk, rd = case["heads"], case["kv_heads"], case["rotary_dim"]
        turn = torch.polar(torch.full((s["pos"].numel(), rd // 2), s["factor"], dtype=torch.float64, device="cuda"),
                           s["pos"].double()[:, None] * s["freq"][None, :])
        x = s["qkv"].double()
        i = torch.arange(rd // 2, device="cuda")
        first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rd // 2)
        z = torch.complex(x[..., first], x[..., second]) * turn[:, None]
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        k, v = s["k_cache"].double(), s["v_cache"].double()
        at = (s["slot"] // case["page_size"], s["slot"] % case["page_size"])
        k[at], v[at] = y[:, hq:hq + hk], x[:, hq + hk:]
        return [y[:, :hq], k, v]
    q_lens, kv_lens = _lens(case)
    hq, hk, d, ps = case["heads"], case["kv_heads"], case["head_dim"], case["page_size"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full((s["q"].shape[0], hq), -math.inf, dtype=torch.float64, device="cuda")
    at = 0
    for b, (nq, nk) in enumerate(zip(q_lens, kv_lens)):
        pages = s["page_table"][b, : -(-nk // ps)].long()
        k = s["k_cache"][pages].reshape(-1, hk, d)[:nk].double()
        v = s["v_cache"][pages].reshape(-1, hk, d)[:nk].double()
        pos = torch.arange(nk - nq, nk, device="cuda")[:, None]
        key = torch.arange(nk, device="cuda")[None]
        hidden = torch.zeros((nq, nk), dtype=torch.bool, device="cuda")
        if case["causal"]:
            hidden = key > pos
            if case["window"]:
                hidden = hidden | (key <= pos - case["window"])
        for h in range(hq):
            e = (s["q"][at:at + nq, h].double() @ k[:, h // (hq // hk)].t()) / math.sqrt(d)
            e = e.masked_fill(hidden, -math.inf)
            lse[at:at + nq, h] = torch.logsumexp(e, dim=1)
            out[at:at + nq, h] = torch.softmax(e, dim=1) @ v[:, h // (hq // hk)]
        at += nq
    return [out, lse]


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    if op in ("norm", "quantize"):
        n, cols = case["rows"] * case["cols"], case["cols"]
        scales = 4 * (-(-case["rows"] // GROUP) if case.get("blocks") else case["rows"]) * -(-cols // GROUP)
        if op == "quantize":
            return {"bytes": 3 * n + scales, "flops": 2 * n}
        return {"bytes": 2 * n * (3 if case["residual"] else 1) + 2 * cols + (n + scales if case["fp8"] else 2 * n), "flops": 5 * n}
    if op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        kb = -(-k // GROUP)
        return {"bytes": m * k + n * k + 2 * m * n + 4 * kb * (m + -(-n // GROUP)), "flops": 2 * m * n * k}
    q_lens, kv_lens = _lens(case)
    hq, hk, d = case["heads"], case["kv_heads"], case["head_dim"]
    tokens = sum(q_lens)
    if op == "rope":
        return {"bytes": 4 * tokens * (hq + 2 * hk) * d, "flops": 3 * tokens * (hq + hk) * case["rotary_dim"]}
    keys = pairs = 0
    for nq, nk in zip(q_lens, kv_lens):
        if not case["causal"]:
            keys, pairs = keys + nk, pairs + nq * nk
            continue
        w = case["window"] or nk
        keys += min(nk, w + nq - 1)
        first = nk - nq + 1  # keys before and with the first new token
        full = max(0, min(nk, w) - first)  # tokens that see all before them
        pairs += full * first + full * (full - 1) // 2 + (nq - full) * min(nk, w)
    return {"bytes": 2 * (2 * tokens * hq * d + 2 * keys * hk * d) + 4 * tokens * hq, "flops": 4 * d * hq * pairs}
