"""Cases of the operators around a decoder layer's attention half: the norms on both sides of a block, the dense gated
feed-forward block, attention that keeps a window and the first tokens, and the probabilities at the model's end.

  norms     norm after a block, its gate, the scaled residual, and the norm before the next block, in 16 bits or e4m3
  gated     both projections of a gated feed-forward block in e4m3, the activation and the product, in 16 bits or e4m3
  sinks     a chunk of new tokens of each sequence over the last keys of its paged cache and the first few
  logprobs  log probabilities of given tokens, entropy and the most probable alternatives, from a model's logits

Every operator has a plain form in elementary torch operations (32 bits, rounded once at the end) and `exact`, its
definition in 64 bits.  Sequence lengths and page orders of a case come from the case itself; values come from the seed.
"""
import math
import random

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
E4M3_MAX = 448.0
MIN_SCALE = 2.0 ** -100
GROUP = 128


def listed():
    return [
        # one token of the 8x7B-shaped layer: latency
        {"name": "norms_one_token", "op": "norms", "rows": 1, "cols": 4096, "dtype": "fp16", "post": True, "gate": "none",
         "fp8": False},
        # a ragged chunk of an odd width with a gate per channel
        {"name": "norms_chunk_odd", "op": "norms", "rows": 1531, "cols": 5121, "dtype": "bf16", "post": True, "gate": "row",
         "fp8": False},
        # a prefill batch of the 8x22B-shaped layer, before a projection in 8 bits
        {"name": "norms_fp8_prefill", "op": "norms", "rows": 8192, "cols": 6144, "dtype": "bf16", "post": True, "gate": "row",
         "fp8": True},
        # a small decode batch through a dense layer of the 8x7B shape: both projections stream from memory
        {"name": "gated_decode", "op": "gated", "m": 7, "n": 14336, "k": 4096, "dtype": "fp16", "fp8": True, "act": "silu"},
        # a ragged chunk through a small expert's width
        {"name": "gated_chunk_odd", "op": "gated", "m": 509, "n": 1408, "k": 2048, "dtype": "bf16", "fp8": False,
         "act": "gelu_tanh"},
        # a prefill batch through a dense layer of the 8x22B shape
        {"name": "gated_prefill", "op": "gated", "m": 8192, "n": 16384, "k": 6144, "dtype": "bf16", "fp8": True, "act": "silu"},
        # one token of one long conversation: latency
        {"name": "sinks_one_token", "op": "sinks", "batch": 1, "q_min": 1, "q_max": 1, "kv_min": 30001, "kv_max": 30001,
         "lens": 1, "heads": 32, "kv_heads": 8, "head_dim": 128, "page_size": 16, "heads_first": False, "window": 1024,
         "sinks": 4, "dtype": "fp16"},
        # a decode batch whose sequences run from a few tokens to far past the window
        {"name": "sinks_decode_ragged", "op": "sinks", "batch": 64, "q_min": 1, "q_max": 1, "kv_min": 17, "kv_max": 32768,
         "lens": 2, "heads": 48, "kv_heads": 8, "head_dim": 128, "page_size": 64, "heads_first": True, "window": 4096,
         "sinks": 67, "dtype": "bf16"},
        # chunks of prompts over what the cache holds already
        {"name": "sinks_prefill", "op": "sinks", "batch": 4, "q_min": 1500, "q_max": 2048, "kv_min": 4096, "kv_max": 16384,
         "lens": 3, "heads": 32, "kv_heads": 8, "head_dim": 128, "page_size": 32, "heads_first": False, "window": 4096,
         "sinks": 4, "dtype": "fp16"},
        # one sampled token, with the alternatives that a user asks for
        {"name": "logprobs_one_token", "op": "logprobs", "rows": 1, "vocab": 32000, "pad": 0, "given": 1, "top": 20,
         "dtype": "fp16", "masked": False},
        # a decode batch under a grammar that rules out half of an odd vocabulary
        {"name": "logprobs_decode_odd", "op": "logprobs", "rows": 61, "vocab": 151937, "pad": 0, "given": 3, "top": 5,
         "dtype": "fp32", "masked": True},
        # the quality of a model measured on a long text
        {"name": "logprobs_prompt", "op": "logprobs", "rows": 4096, "vocab": 131072, "pad": 0, "given": 1, "top": 1,
         "dtype": "bf16", "masked": False},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norms", "gated", "sinks", "sinks", "logprobs"])
    dtype = rng.choice(["fp16", "bf16"])
    if op == "norms":
        cols = rng.choice([_log(rng, 64, 8192), 8 * _log(rng, 8, 1024), rng.choice([2048, 4096, 6144])])
        return {"op": op, "rows": _log(rng, 1, 4096), "cols": cols, "dtype": dtype, "post": rng.random() < 0.8,
                "gate": rng.choice(["none", "row", "matrix"]), "fp8": rng.random() < 0.5}
    if op == "gated":
        n = rng.choice([_log(rng, 128, 16384), 128 * rng.randint(1, 128)])
        k = rng.choice([16 * _log(rng, 4, 384), 128 * rng.randint(1, 48)])
        return {"op": op, "m": _log(rng, 1, 8192), "n": n, "k": k, "dtype": dtype, "fp8": rng.random() < 0.6,
                "act": rng.choice(["silu", "silu", "gelu_tanh"])}
    if op == "logprobs":
        vocab, dtype = _log(rng, 512, 262144), rng.choice(["fp16", "bf16", "fp32"])
        most = ((1 << 29) if dtype != "fp32" else (1 << 28)) // vocab
        return {"op": op, "rows": _log(rng, 1, min(4096, most)), "vocab": vocab,
                "pad": rng.choice([0, 0, rng.randint(1, 128)]), "given": rng.choice([1, 1, rng.randint(0, 8)]),
                "top": rng.choice([0, 1, 5, 20, rng.randint(1, 32)]), "dtype": dtype,
                "masked": rng.random() < 0.3}
    heads, kv_heads = rng.choice([(32, 8), (48, 8), (16, 16), (16, 2), (8, 1), (12, 4)])
    c = {"op": op, "batch": _log(rng, 1, 32), "lens": rng.randint(10, 1 << 20), "heads": heads, "kv_heads": kv_heads,
         "head_dim": rng.choice([64, 128, 128]), "page_size": rng.choice([16, 32, 64, 128]),
         "heads_first": rng.random() < 0.5, "dtype": dtype}
    # new tokens a sequence: one, a few (drafted tokens), or a chunk
    c["q_max"] = rng.choice([1, 1, rng.randint(2, 8), _log(rng, 16, 1024)])
    c["q_min"] = rng.randint(1, c["q_max"]) if c["q_max"] > 1 else 1
    c["window"] = _log(rng, 8, 8192)
    c["sinks"] = rng.choice([1, 4, 16, _log(rng, 1, 512)])
    # the plain form pads every sequence to the longest visible part: at most 2^30 scores in all
    most = min(32768, (1 << 27) // (c["batch"] * kv_heads * c["head_dim"]) * 4, (1 << 30) // (c["batch"] * heads * c["q_max"]))
    c["kv_max"] = _log(rng, 64, max(65, most))
    c["kv_min"] = rng.randint(1, c["kv_max"])
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


def _cache(case, g, q_lens, kv_lens):
    """The paged cache, [pages][page_size][kv_heads][head_dim] in either order of storage, and the page table.  Only
    pages that some new token sees are held, handed out at random: the table says -1 for those between the first tokens
    and the window.  What no token sees of a held page is not even numbers."""
    dt, ps, hk, d = DTYPES[case["dtype"]], case["page_size"], case["kv_heads"], case["head_dim"]
    width = -(-max(kv_lens) // ps)
    key = torch.arange(width * ps, device="cuda")[None, :]
    kv = torch.tensor(kv_lens, device="cuda")[:, None]
    first = kv - torch.tensor(q_lens, device="cuda")[:, None] - case["window"] + 1
    seen = ((key < kv) & ((key >= first) | (key < case["sinks"]))).view(len(kv_lens), width, ps)
    held = seen.any(dim=2)
    pages = int(held.sum()) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(kv_lens), width), -1, dtype=torch.int32, device="cuda")
    table[held] = order[: pages - 3]
    rows, places = torch.nonzero(~seen[held], as_tuple=True)
    rows = table[held].long()[rows]

    def one():
        shape = (pages, hk, ps, d) if case["heads_first"] else (pages, ps, hk, d)
        t = torch.empty(shape, dtype=dt, device="cuda").normal_(generator=g)
        t = t.permute(0, 2, 1, 3) if case["heads_first"] else t
        t[rows, places] = float("nan")
        return t
    return one(), one(), table


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "norms":
        dt, rows, cols = DTYPES[case["dtype"]], case["rows"], case["cols"]
        normal = lambda *shape: torch.empty(shape, dtype=dt, device="cuda").normal_(generator=g)  # noqa: E731
        weight = lambda: (1 + 0.1 * torch.randn(cols, generator=g, device="cuda")).to(dt)  # noqa: E731
        st = {"case": case, "x": normal(rows, cols), "res": normal(rows, cols) * 4, "post": weight() if case["post"] else None,
              "w": weight(), "gate": None, "scales": (0.75, 1.25)}
        st["x"][:, ::61] *= 20   # a few outlier channels, as activations have them
        if case["gate"] != "none":
            st["gate"] = normal(*((cols,) if case["gate"] == "row" else (rows, cols)))
        st["res_out"] = torch.empty_like(st["x"])
        st["y"] = None if case["fp8"] else torch.empty_like(st["x"])
        st["q"] = st["scale"] = None
        if case["fp8"]:
            st["q"] = torch.empty((rows, cols), dtype=torch.float8_e4m3fn, device="cuda")
            st["scale"] = torch.empty((rows, -(-cols // GROUP)), dtype=torch.float32, device="cuda")
        return st
    if op == "gated":
        m, n, k = case["m"], case["n"], case["k"]
        kb, nb = -(-k // GROUP), -(-n // GROUP)

        def codes(rows):
            t = torch.empty((rows, k), dtype=torch.float16, device="cuda").normal_(generator=g)
            return (t * 120).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        spread = lambda r, s: s * torch.exp(0.4 * torch.randn((r, kb), generator=g, device="cuda"))  # noqa: E731
        s = 1 / 120 / math.sqrt(k)   # projections of about 1
        st = {"case": case, "a": codes(m), "sa": spread(m, 1e-2), "gate": codes(n), "sg": spread(nb, s), "up": codes(n),
              "su": spread(nb, s), "y": None, "q": None, "scale": None,
              "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
        if case["fp8"]:
            st["q"] = torch.empty((m, n + (-n % 16)), dtype=torch.float8_e4m3fn, device="cuda")[:, :n]
            st["scale"] = torch.empty((m, nb), dtype=torch.float32, device="cuda")
        else:
            st["y"] = torch.empty((m, n), dtype=DTYPES[case["dtype"]], device="cuda")
        return st
    if op == "logprobs":
        rows, vocab, given, top = case["rows"], case["vocab"], case["given"], case["top"]
        wide = torch.empty((rows, vocab + case["pad"]), dtype=DTYPES[case["dtype"]], device="cuda").normal_(generator=g)
        wide.mul_(2.5)
        logits = wide[:, :vocab]
        pick = lambda *shape: torch.randint(vocab, shape, generator=g, device="cuda")  # noqa: E731
        row = torch.arange(rows, device="cuda")[:, None]
        likely = pick(rows, 3)
        if case["masked"]:
            wide.masked_fill_(torch.rand(wide.shape, generator=g, device="cuda") < 0.5, -math.inf)
        high = (8 + 4 * torch.rand((rows, 3), generator=g, device="cuda")).to(logits.dtype)
        for i in range(3):  # a row may draw one position twice: the later value stays
            logits[row[:, 0], likely[:, i]] = high[:, i]
        targets = pick(rows, given)
        if given:
            targets[:, 0] = torch.where(torch.rand(rows, generator=g, device="cuda") < 0.7, likely[:, 0], targets[:, 0])
        f32 = lambda *shape: torch.empty(shape, dtype=torch.float32, device="cuda")  # noqa: E731
        return {"case": case, "logits": logits, "targets": targets.to(torch.int32) if given else None, "temperature": 0.8,
                "lp": f32(rows, given) if given else None, "lse": f32(rows), "entropy": f32(rows),
                "ids": torch.empty((rows, top), dtype=torch.int32, device="cuda") if top else None,
                "top": f32(rows, top) if top else None}
    q_lens, kv_lens = _lens(case)
    tokens, dt = sum(q_lens), DTYPES[case["dtype"]]
    off = [0]
    for n in q_lens:
        off.append(off[-1] + n)
    st = {"case": case, "q_offsets": torch.tensor(off, dtype=torch.int32, device="cuda"),
          "kv_lens": torch.tensor(kv_lens, dtype=torch.int32, device="cuda"),
          "status": torch.zeros(1, dtype=torch.int32, device="cuda"), "max_q_len": max(q_lens), "max_kv_len": max(kv_lens)}
    st["k_cache"], st["v_cache"], st["page_table"] = _cache(case, g, q_lens, kv_lens)
    st["seq"] = torch.repeat_interleave(torch.arange(len(q_lens), device="cuda"), torch.tensor(q_lens, device="cuda"))
    st["q"] = torch.empty((tokens, case["heads"], case["head_dim"]), dtype=dt, device="cuda").normal_(generator=g) * 1.5
    st["out"] = torch.empty_like(st["q"])
    st["lse"] = torch.empty((tokens, case["heads"]), dtype=torch.float32, device="cuda")
    return st


# ---------------------------------------------------------------- one pass
def run(state):
    if own:
        return _run_own(state)
    return {"norms": _norms, "gated": _gated, "sinks": _sinks, "logprobs": _logprobs}[state["case"]["op"]](state)


def _run_own(s):
    from any_precision_bit_pw_gb300 import pw
    c = s["case"]
    if c["op"] == "norms":
        pw.pw_norm_add_norm(s["x"], s["res"], 1e-5, post_weight=s["post"], weight=s["w"], gate=s["gate"],
                            residual_scale=s["scales"][0], block_scale=s["scales"][1], residual_out=s["res_out"], y=s["y"],
                            q=s["q"], scale=s["scale"])
        return [t for t in (s["res_out"], s["y"], s["q"], s["scale"]) if t is not None]
    if c["op"] == "gated":
        pw.pw_fp8_gated_linear(s["a"], s["sa"], s["gate"], s["sg"], s["up"], s["su"], s["status"], y=s["y"], q=s["q"],
                               scale=s["scale"], activation={"silu": pw.PW_ACT_SILU, "gelu_tanh": pw.PW_ACT_GELU_TANH}[c["act"]])
        return [t for t in (s["y"], s["q"], s["scale"]) if t is not None]
    if c["op"] == "logprobs":
        pw.pw_token_logprobs(s["logits"], targets=s["targets"], logprobs=s["lp"], lse=s["lse"], entropy=s["entropy"],
                             top_ids=s["ids"], top_logprobs=s["top"], scale=1 / s["temperature"])
        return [t for t in (s["lp"], s["lse"], s["entropy"], s["ids"], s["top"]) if t is not None]
    if "ws" not in s:  # kept by the caller beside its cache
        n = pw.pw_paged_attention_workspace(s["q"].shape[0], c["batch"], c["heads"], c["kv_heads"], c["head_dim"])
        s["ws"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
    pw.pw_paged_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["q_offsets"], s["kv_lens"], s["out"],
                          s["ws"], s["status"], scale=c["head_dim"] ** -0.5, window=c["window"], sinks=c["sinks"],
                          max_q_len=s["max_q_len"], max_kv_len=s["max_kv_len"], lse=s["lse"])
    return [s["out"], s["lse"]]


def _to_e4m3(y):
    """Codes and scales: s = max(largest of the group / 448, 2^-100), code = e4m3(y / s)."""
    rows, cols = y.shape
    t = torch.nn.functional.pad(y, (0, -cols % GROUP)).view(rows, -1, GROUP)
    scale = (t.abs().amax(dim=2) / E4M3_MAX).clamp(min=MIN_SCALE)
    return (t / scale[:, :, None]).view(rows, -1)[:, :cols].to(torch.float8_e4m3fn), scale


def _rms(t):
    return t * torch.rsqrt((t * t).mean(dim=1, keepdim=True) + 1e-5)


def _norms(s):
    u = s["x"].float()
    if s["post"] is not None:
        u = _rms(u) * s["post"].float()
    if s["gate"] is not None:
        u = u * s["gate"].float()
    r = s["scales"][0] * s["res"].float() + s["scales"][1] * u
    y = _rms(r) * s["w"].float()
    got = [r.to(s["x"].dtype)]
    if s["y"] is not None:
        return got + [y.to(s["x"].dtype)]
    return got + list(_to_e4m3(y))


def _spread(scale, rows, cols, block_rows):
    return scale.repeat_interleave(block_rows, 0)[:rows].repeat_interleave(GROUP, 1)[:, :cols]


def _gated(s):
    a = s["a"].float() * _spread(s["sa"], *s["a"].shape, 1)
    g = torch.matmul(a, (s["gate"].float() * _spread(s["sg"], *s["gate"].shape, GROUP)).t())
    u = torch.matmul(a, (s["up"].float() * _spread(s["su"], *s["up"].shape, GROUP)).t())
    if s["case"]["act"] == "silu":
        h = g / (1 + torch.exp(-g)) * u
    else:
        h = 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g))) * u
    return [h.to(s["y"].dtype)] if s["y"] is not None else list(_to_e4m3(h))


def _visible(s):
    """The keys that a sequence's new tokens see, first tokens and then the window: positions [batch][longest] and which
    of them there are."""
    c = s["case"]
    first = (s["kv_lens"] - s["q_offsets"].diff() - c["window"] + 1).clamp(min=0).long()[:, None]
    longest = min(s["max_kv_len"], c["sinks"] + c["window"] + s["max_q_len"] - 1)
    i = torch.arange(longest, device="cuda")[None, :]
    sinks = first.clamp(max=c["sinks"])
    key = torch.where(i < sinks, i, first + i - sinks)
    return key, key < s["kv_lens"][:, None]


def _sinks(s):
    c = s["case"]
    b, hq, hk, d, nq, ps = c["batch"], c["heads"], c["kv_heads"], c["head_dim"], s["max_q_len"], c["page_size"]
    group = hq // hk
    key, there = _visible(s)
    nk = key.shape[1]
    page = s["page_table"].gather(1, torch.where(there, key // ps, torch.zeros_like(key))).long().clamp(min=0)
    hidden = ~there[:, :, None, None]
    k = s["k_cache"][page, key % ps].float().masked_fill_(hidden, 0.0)
    v = s["v_cache"][page, key % ps].float().masked_fill_(hidden, 0.0)
    row = torch.arange(s["q"].shape[0], device="cuda") - s["q_offsets"][s["seq"]].long()
    q = torch.zeros((b, nq, hq, d), dtype=torch.float32, device="cuda")
    q[s["seq"], row] = s["q"].float()
    q = q.view(b, nq, hk, group, d).permute(0, 2, 3, 1, 4).reshape(b, hk, group * nq, d)
    score = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(d ** -0.5).view(b, hk, group, nq, nk)
    pos = (torch.arange(nq, device="cuda")[None, :] + (s["kv_lens"] - s["q_offsets"].diff())[:, None])[:, :, None]
    at = key[:, None, :]
    seen = there[:, None, :] & (at <= pos) & ((at > pos - c["window"]) | (at < c["sinks"]))
    score.masked_fill_(~seen[:, None, None].expand_as(score), -math.inf)
    top = score.amax(dim=-1, keepdim=True)
    safe = top.masked_fill(top == -math.inf, 0.0)
    score = score.sub_(safe).exp_()
    total = score.sum(dim=-1, keepdim=True)
    out = torch.matmul(score.view(b, hk, -1, nk), v.permute(0, 2, 1, 3)).view(b, hk, group, nq, d)
    out = out / total.masked_fill(total == 0, 1.0)
    lse = (safe + total.log())[..., 0]
    out = out.permute(0, 3, 1, 2, 4).reshape(b, nq, hq, d)[s["seq"], row]
    return [out.to(s["q"].dtype), lse.permute(0, 3, 1, 2).reshape(b, nq, hq)[s["seq"], row]]


def _logprobs(s):
    c, z = s["case"], s["logits"].float()
    got, order = [], None
    if c["top"]:
        # distinct whole numbers in the order of (value, lowest index first)
        bits = (z + 0.0).view(torch.int32).long()
        order = torch.where(bits < 0, -1 - (bits & 0x7FFFFFFF), bits) * c["vocab"]
        order -= torch.arange(c["vocab"], device="cuda")
        ids = c["vocab"] - 1 - (order.topk(c["top"], dim=1).values + (c["vocab"] - 1)) % c["vocab"]
    z = z * (1 / s["temperature"])
    top = z.amax(dim=1, keepdim=True)
    d = z - top
    e = d.exp()
    total = e.sum(dim=1, keepdim=True)
    d.masked_fill_(e == 0, 0.0)
    norm = total.log()
    if c["given"]:
        got.append(z.gather(1, s["targets"].long()) - top - norm)
    got += [(top + norm)[:, 0], (norm - (e * d).sum(dim=1, keepdim=True) / total)[:, 0]]
    if c["top"]:
        got += [ids.to(torch.int32), z.gather(1, ids) - top - norm]
    return got


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_codes(h):
    """The values before they are rounded to 8 bits, so that an error says what the rounding costs, and the scales."""
    rows, cols = h.shape
    groups = -(-cols // GROUP)
    group = (torch.arange(rows, device="cuda") * groups)[:, None] + (torch.arange(cols, device="cuda") // GROUP)[None]
    top = torch.zeros(rows * groups, dtype=torch.float64, device="cuda")
    top.scatter_reduce_(0, group.reshape(-1), h.abs().reshape(-1), "amax")
    scale = torch.maximum(top / E4M3_MAX, torch.full_like(top, MIN_SCALE))
    return [h / scale[group], scale.view(rows, groups)]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norms":
        block = s["x"].double()
        if case["post"]:
            block = block / torch.sqrt(torch.einsum("ij,ij->i", block, block) / case["cols"] + 1e-5)[:, None]
            block = torch.einsum("ij,j->ij", block, s["post"].double())
        if case["gate"] != "none":
            block = block * s["gate"].double().expand(case["rows"], case["cols"])
        alpha, beta = s["scales"]
        r = torch.add(s["res"].double() * alpha, block, alpha=beta)
        y = r / torch.sqrt(torch.einsum("ij,ij->i", r, r) / case["cols"] + 1e-5)[:, None] * s["w"].double()
        return [r] + (_exact_codes(y) if case["fp8"] else [y])
    if op == "gated":
        group = torch.arange(case["k"], device="cuda") // GROUP
        block = torch.arange(case["n"], device="cuda") // GROUP
        a = s["a"].double() * s["sa"].double()[:, group]
        g = a @ (s["gate"].double() * s["sg"].double()[block][:, group]).t()
        if case["act"] == "silu":
            h = g * torch.sigmoid(g)
        else:
            h = torch.nn.functional.gelu(g, approximate="tanh")
        h = h * (a @ (s["up"].double() * s["su"].double()[block][:, group]).t())
        return _exact_codes(h) if case["fp8"] else [h]
    if op == "logprobs":
        parts = []
        for i in range(0, case["rows"], 512):
            z = s["logits"][i:i + 512].double()
            lp = torch.log_softmax(z * (1 / s["temperature"]), dim=1)
            p = lp.exp()
            got = [lp.gather(1, s["targets"][i:i + 512].long())] if case["given"] else []
            got += [torch.logsumexp(z * (1 / s["temperature"]), dim=1), -torch.where(p > 0, p * lp, torch.zeros_like(p)).sum(dim=1)]
            if case["top"]:
                index, ids = torch.arange(case["vocab"], device="cuda")[None], []
                left = z.clone()
                done = torch.zeros_like(left, dtype=torch.bool)
                for _ in range(case["top"]):
                    best = left.masked_fill(done, -math.inf).amax(dim=1, keepdim=True)
                    at = torch.where((left == best) & ~done, index, case["vocab"]).amin(dim=1, keepdim=True)
                    done.scatter_(1, at, True)
                    ids.append(at)
                ids = torch.cat(ids, dim=1)
                got += [ids.to(torch.int32), lp.gather(1, ids)]
            parts.append(got)
        return [torch.cat(t) for t in zip(*parts)]
    q_lens, kv_lens = _lens(case)
    hq, hk, d, ps, w = case["heads"], case["kv_heads"], case["head_dim"], case["page_size"], case["window"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full((s["q"].shape[0], hq), -math.inf, dtype=torch.float64, device="cuda")
    at = 0
    for b, (nq, nk) in enumerate(zip(q_lens, kv_lens)):
        key = torch.arange(nk, device="cuda")
        key = key[(key < case["sinks"]) | (key > nk - nq - w)]
        page = s["page_table"][b, key // ps].long()
        k, v = s["k_cache"][page, key % ps].double(), s["v_cache"][page, key % ps].double()
        pos = torch.arange(nk - nq, nk, device="cuda")[:, None]
        hidden = (key[None] > pos) | ((key[None] <= pos - w) & (key[None] >= case["sinks"]))
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
    if op == "norms":
        n, cols = case["rows"] * case["cols"], case["cols"]
        read = 4 * n + 2 * cols * (1 + case["post"]) + {"none": 0, "row": 2 * cols, "matrix": 2 * n}[case["gate"]]
        write = 2 * n + (n + 4 * case["rows"] * -(-cols // GROUP) if case["fp8"] else 2 * n)
        return {"bytes": read + write, "flops": 10 * n}
    if op == "gated":
        m, n, k = case["m"], case["n"], case["k"]
        kb, nb = -(-k // GROUP), -(-n // GROUP)
        out = m * n + 4 * m * nb if case["fp8"] else 2 * m * n
        return {"bytes": m * k + 2 * n * k + 4 * kb * (m + 2 * nb) + out, "flops": 4 * m * n * k}
    if op == "logprobs":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * (4 if case["dtype"] == "fp32" else 2) + case["rows"] * (8 + 8 * case["given"] + 8 * case["top"]),
                "flops": 6 * n}
    q_lens, kv_lens = _lens(case)
    hq, hk, d, w, sinks = case["heads"], case["kv_heads"], case["head_dim"], case["window"], case["sinks"]
    keys = pairs = 0
    for nq, nk in zip(q_lens, kv_lens):
        first = max(0, nk - nq - w + 1)
        keys += nk - first + min(sinks, first)
        for pos in range(nk - nq, nk):
            gone = max(0, pos - w + 1)
            pairs += pos + 1 - gone + min(sinks, gone)
    return {"bytes": 2 * (2 * sum(q_lens) * hq * d + 2 * keys * hk * d) + 4 * sum(q_lens) * hq, "flops": 4 * d * hq * pairs}
