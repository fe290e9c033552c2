"""A decoder layer around the mixed-precision experts: residual norm, 8-bit
projections, rotary positions, attention over a paged cache, and the routed
expert layer of ``layer.py`` or a dense gated block, one stream, buffers allocated
once; and the model's end, the head's projection with the probabilities.

    cache = PagedCache(pages=4096, page_size=16, kv_heads=8, head_dim=128)
    layer = DecoderLayer(stack, 0, weights, heads=32, cache=cache, tokens=64)
    batch = cache.batch([3, 7], [1, 1])      # one new token of sequences 3 and 7
    x, residual = layer(x, residual, batch)  # both fp16 [T][H]
    head = Head(norm, Fp8Weight.quantize(w_head), tokens=64, top=5, after=layer)
    scores = head(x, residual, targets)      # log probabilities, entropy, alternatives

A layer's output is added to the residual by the layer (or the head) that comes
``after`` it, where the norms on both sides of a block are one kernel.

Every computation but the router's small product (a widening copy and cuBLAS) is
a libpw kernel (``pw.py``); the layer allocates and synchronises nothing in a
call, so a step can be captured in a CUDA graph once the batch's tensors are in
place.  ``layer.status`` holds the first failure of any of its kernels, the
experts' included; ``layer.experts.mass`` the experts' routing mass.
"""
from __future__ import annotations

from contextlib import nullcontext
from dataclasses import dataclass
from typing import Dict, List, Optional, Sequence

import torch

from . import pw
from .layer import APLMoEStack, MoECall


def _on(stream):
    """Makes ``stream`` (a torch stream or a raw handle; None: as it is) torch's
    current one, so that libpw's calls and torch's own work are in one order."""
    if stream is None:
        return nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(stream)   # 0 and 1: CUDA's names of the default stream
        stream = torch.cuda.ExternalStream(handle) if handle > 1 else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _settle(dev: torch.device) -> None:
    """Memory that was taken on the current stream is free (and zeroed, where it has to be) for calls on any stream."""
    if dev.type == "cuda":
        torch.cuda.current_stream(dev).synchronize()


@dataclass
class Batch:
    """New tokens of some sequences, as the kernels read them (pw.h)."""
    page_table: torch.Tensor   # int32 [batch][pages_per_seq]
    q_offsets: torch.Tensor    # int32 [batch + 1]
    kv_lens: torch.Tensor      # int32 [batch], the new tokens included
    tokens: int
    max_q_len: int
    max_kv_len: int


class PagedCache:
    """Key/value pages of one layer and, on the host, which sequence holds
    which.  Page states are plain Python; the device sees them through the
    tables that ``batch`` builds.  A table names pages and nothing of a layer: with
    one cache per layer, all of one shape, the first one's ``batch`` serves all
    layers of a step and the other caches are storage only."""

    def __init__(self, pages: int, page_size: int, kv_heads: int, head_dim: int, dtype=torch.float16, device="cuda"):
        shape = (pages, page_size, kv_heads, head_dim)
        self.k = torch.empty(shape, dtype=dtype, device=device)
        self.v = torch.empty(shape, dtype=dtype, device=device)
        self.page_size, self.device = page_size, torch.device(device)
        self.free_pages: List[int] = list(range(pages - 1, -1, -1))
        self.pages: Dict[int, List[int]] = {}
        self.lens: Dict[int, int] = {}
        _settle(self.device)

    def batch(self, seqs: Sequence[int], new_tokens: Sequence[int], width: Optional[int] = None) -> Batch:
        """Makes room for ``new_tokens`` more keys of each sequence and returns
        the tables of the call that will append them.  ``width`` fixes the page
        table's columns (for a captured graph)."""
        if len(set(seqs)) != len(seqs) or len(seqs) != len(new_tokens) or min(new_tokens, default=0) < 0:
            raise ValueError("batch: every sequence once, with its number of new tokens")
        total = [-(-(self.lens.get(s, 0) + n) // self.page_size) for s, n in zip(seqs, new_tokens)]   # pages of each
        more = [t - len(self.pages.get(s, ())) for s, t in zip(seqs, total)]
        if sum(more) > len(self.free_pages):
            raise RuntimeError(f"the cache is full: {sum(more)} pages wanted, {len(self.free_pages)} free")
        width = max(total + [1]) if width is None else width
        if max(total + [1]) > width:
            raise ValueError(f"batch: {max(total)} pages do not fit a table of {width}")
        for s, n, m in zip(seqs, new_tokens, more):
            self.pages.setdefault(s, []).extend(self.free_pages.pop() for _ in range(m))
            self.lens[s] = self.lens.get(s, 0) + n
        table = torch.full((max(len(seqs), 1), width), -1, dtype=torch.int32)
        for b, s in enumerate(seqs):
            table[b, : len(self.pages[s])] = torch.tensor(self.pages[s], dtype=torch.int32)
        offsets = torch.zeros(len(seqs) + 1, dtype=torch.int32)
        offsets[1:] = torch.tensor(list(new_tokens), dtype=torch.int32).cumsum(0)
        lens = torch.tensor([self.lens[s] for s in seqs], dtype=torch.int32)
        to = lambda t: t.to(self.device)  # noqa: E731
        return Batch(to(table), to(offsets), to(lens), int(offsets[-1]), max(new_tokens, default=0),
                     max([self.lens[s] for s in seqs], default=0))

    def release(self, seq: int) -> None:
        """Returns a sequence's pages (once the stream has passed the calls that read them)."""
        self.free_pages.extend(p for p in reversed(self.pages.pop(seq, [])) if p >= 0)
        self.lens.pop(seq, None)

    def trim(self, seq: int, window: int, sinks: int = 0) -> int:
        """Returns the pages of a sequence that no later token sees in attention
        over the last ``window`` keys and the first ``sinks`` (once the stream has
        passed the calls that read them), and how many they are.  Tables serve all
        layers of a step: ``window`` and ``sinks`` are the largest of any layer that reads
        them, and where one of them attends to every key there is nothing to return."""
        if window < 1 or sinks < 0:
            raise ValueError(f"trim: window {window}, sinks {sinks}")
        pages, n = self.pages.get(seq, []), self.page_size
        seen_from = self.lens.get(seq, 0) - window + 1            # by the next token
        gone = [j for j in range(-(-sinks // n), max(seen_from, 0) // n) if pages[j] >= 0]
        for j in gone:
            self.free_pages.append(pages[j])
            pages[j] = -1
        return len(gone)


@dataclass
class Fp8Weight:
    """e4m3 codes [N][K] with a scale per 128 x 128 block."""
    codes: torch.Tensor
    scale: torch.Tensor

    @staticmethod
    def quantize(w: torch.Tensor, stream=None) -> "Fp8Weight":
        n, k = w.shape
        pad = -k % 16                              # rows of the product are 16-byte aligned
        with _on(stream):   # memory that another stream has just freed may still be in use there
            codes = torch.empty((n, k + pad), dtype=torch.float8_e4m3fn, device=w.device)[:, :k]
            scale = torch.empty((-(-n // 128), -(-k // 128)), dtype=torch.float32, device=w.device)
            pw.pw_quantize_fp8(w, codes, scale, block_rows=128)
        return Fp8Weight(codes, scale)


@dataclass
class DecoderWeights:
    attn_norm: torch.Tensor    # [H]
    ffn_norm: torch.Tensor     # [H]
    qkv: Fp8Weight             # [(heads + 2 kv_heads) * head_dim][H]
    out: Fp8Weight             # [H][heads * head_dim]
    router: Optional[torch.Tensor] = None      # [experts][H] fp32; None: a dense block instead of the experts
    gate: Optional[Fp8Weight] = None           # the dense block: [I][H]
    up: Optional[Fp8Weight] = None             # [I][H]
    down: Optional[Fp8Weight] = None           # [H][I]
    # where a block's output is added: r = residual_scale * residual + gate * norm(output)
    post_attn_norm: Optional[torch.Tensor] = None   # [H]
    post_ffn_norm: Optional[torch.Tensor] = None    # [H]
    attn_gate: Optional[torch.Tensor] = None        # [H]
    ffn_gate: Optional[torch.Tensor] = None         # [H]
    residual_scale: float = 1.0


def _is_joined(w: DecoderWeights) -> bool:
    """Whether the feed-forward output joins the residual by more than an addition."""
    return w.post_ffn_norm is not None or w.ffn_gate is not None or w.residual_scale != 1.0


def _comes_after(after: Optional["DecoderLayer"], eps: float) -> None:
    """A layer or head that takes another one's output: the norm of that output and its own are one kernel with one eps."""
    if after is None:
        return
    if after.w.post_ffn_norm is not None and after.eps != eps:
        raise ValueError(f"the norm of the layer's output has eps {after.eps}, what comes after it {eps}")
    after.joined = True


def _take_output(after: Optional["DecoderLayer"], x, residual, eps, weight, **out) -> None:
    """The results of the layer that came before join, and the norm of what comes now."""
    if after is None or (residual is None and not _is_joined(after.w)):
        pw.pw_add_rmsnorm(x, weight, eps, residual=residual, **out)
    elif residual is None:
        raise ValueError("the output of the layer that came before goes with its residual")
    else:
        _add_norm(x, residual, eps, weight, after.w.post_ffn_norm, after.w.ffn_gate, after.w.residual_scale, **out)


def _add_norm(x, residual, eps, weight, post, gate, residual_scale, **out) -> None:
    """The block's output x joins the residual, and the norm before the next block."""
    if post is None and gate is None and residual_scale == 1.0:
        pw.pw_add_rmsnorm(x, weight, eps, residual=residual, **out)
    else:
        pw.pw_norm_add_norm(x, residual, eps, post_weight=post, weight=weight, gate=gate, residual_scale=residual_scale, **out)


class DecoderLayer:
    """One layer's calls, and buffers for up to ``tokens`` tokens.  Layers that
    run one after another on one stream can use the buffers of the first of them
    (``share``): each reads its inputs before it writes its results, so the
    results of one may be the inputs of the next.  ``max_batch`` goes to the
    attention's workspace query, whose answer holds for any number of sequences.
    ``after``: the layer whose results come in (None for the first, whose ``x`` is
    the embedding).  A layer whose weights have a norm, a gate or a scale for the
    feed-forward output needs a layer or a head ``after`` it (of the same ``eps``, if
    it is a norm); ``joined`` says that the caller adds its output to the residual
    instead.  With a ``window``, the first ``sinks`` keys of a sequence stay
    visible.  A layer with a dense block needs no ``stack``.
    """

    BUFFERS = ("x8", "x8_scale", "qkv", "q", "attn", "attn8", "attn8_scale", "o", "h", "residual", "h32", "logits", "status",
               "ws", "experts")
    DENSE_BUFFERS = ("ff8", "ff8_scale", "y")   # None without a dense block

    def __init__(self, stack: Optional[APLMoEStack], index: int, weights: DecoderWeights, heads: int, cache: PagedCache,
                 tokens: int, rotary_dim: Optional[int] = None, rope_base: float = 1e6,
                 rope_scaling: Optional[pw.pw_rope_scaling] = None, interleaved: bool = False, window: int = 0,
                 eps: float = 1e-5, max_batch: int = 256, share: Optional["DecoderLayer"] = None, sinks: int = 0,
                 after: Optional["DecoderLayer"] = None, activation: int = pw.PW_ACT_SILU, joined: bool = False):
        self.dense = weights.down is not None
        if self.dense == (weights.router is not None) or (stack is None and not self.dense):
            raise ValueError("decoder layer: a router and a stack of experts, or the gate, up and down of a dense block")
        H = weights.attn_norm.shape[0]
        dev = weights.attn_norm.device if stack is None else stack.device
        assert stack is None or stack.H == H
        self.sinks, self.after, self.activation, self.joined = sinks, after, activation, joined
        self.stack, self.index, self.w, self.cache = stack, index, weights, cache
        self.heads, self.kv_heads, self.head_dim = heads, cache.k.shape[2], cache.k.shape[3]
        self.eps, self.window, self.interleaved, self.tokens = eps, window, interleaved, tokens
        turns, self.rope_factor = pw.pw_rope_turns(self.head_dim if rotary_dim is None else rotary_dim, rope_base, rope_scaling)
        self.turns = turns.to(dev)   # (a copy from pageable memory: it is done when this returns)
        D, wide = self.head_dim, (heads + 2 * self.kv_heads) * self.head_dim
        assert tuple(weights.qkv.codes.shape) == (wide, H) and tuple(weights.out.codes.shape) == (H, heads * D)
        width = 0
        if self.dense:
            width = weights.down.codes.shape[1]
            assert tuple(weights.gate.codes.shape) == tuple(weights.up.codes.shape) == (width, H) == tuple(weights.down.codes.shape)[::-1]
        if share is not None and (
                (share.stack, share.heads, share.kv_heads, share.head_dim, share.tokens, share.h.shape[1], share.h.device)
                != (stack, heads, self.kv_heads, D, tokens, H, self.turns.device)):
            raise ValueError("decoder layer: buffers are shared between layers of one stack, on one device, with equal hidden "
                             "width, heads and tokens")
        _comes_after(after, eps)
        if share is not None:
            for name in self.BUFFERS + self.DENSE_BUFFERS:
                setattr(self, name, getattr(share, name))
            if self.dense and (self.ff8 is None or self.ff8.shape[1] != width):
                self._dense_buffers(tokens, H, width, dev)
                _settle(dev)
            return

        def empty(*shape, dtype=torch.float16):
            return torch.empty(shape, dtype=dtype, device=dev)
        self.x8, self.x8_scale = empty(tokens, H, dtype=torch.float8_e4m3fn), empty(tokens, -(-H // 128), dtype=torch.float32)
        self.qkv = empty(tokens, heads + 2 * self.kv_heads, D)
        self.q = empty(tokens, heads, D)
        self.attn = empty(tokens, heads, D)
        self.attn8 = empty(tokens, heads * D, dtype=torch.float8_e4m3fn)
        self.attn8_scale = empty(tokens, -(-heads * D // 128), dtype=torch.float32)
        self.o, self.h = empty(tokens, H), empty(tokens, H)
        self.residual = [empty(tokens, H), empty(tokens, H)]
        self.h32 = self.logits = self.experts = self.ff8 = self.ff8_scale = self.y = None
        if stack is not None:
            self.h32, self.logits = empty(tokens, H, dtype=torch.float32), empty(tokens, stack.routed, dtype=torch.float32)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)   # of every call, the experts' too
        n = pw.pw_paged_attention_workspace(tokens, max_batch, heads, self.kv_heads, D)
        self.ws = torch.zeros(n, dtype=torch.uint8, device=dev)
        # the experts' workspace grows with the tokens: one, for the most, serves every count
        if stack is not None:
            self.experts = MoECall(stack, tokens)
            self.experts.status = self.status
        if self.dense:
            self._dense_buffers(tokens, H, width, dev)
        _settle(dev)

    def _dense_buffers(self, tokens: int, H: int, width: int, dev) -> None:
        pad = -width % 16                          # rows of the product are 16-byte aligned
        self.ff8 = torch.empty((tokens, width + pad), dtype=torch.float8_e4m3fn, device=dev)[:, :width]
        self.ff8_scale = torch.empty((tokens, -(-width // 128)), dtype=torch.float32, device=dev)
        self.y = torch.empty((tokens, H), dtype=torch.float16, device=dev)

    def moe(self, tokens: int) -> MoECall:
        """The expert layer's buffers; a call of ``tokens`` tokens uses their first rows."""
        if tokens > self.tokens:
            raise ValueError(f"decoder layer: {tokens} tokens, at most {self.tokens}")
        return self.experts

    def __call__(self, x: torch.Tensor, residual: Optional[torch.Tensor], batch: Batch, stream=None):
        """x fp16 [T][H] (the previous layer's output) and the residual before
        it (None at the first layer) -> this layer's (output, residual).  The
        results are the layer's buffers, valid until the next call of a layer that
        has them.  All of it runs on ``stream`` (None: torch's current stream)."""
        with _on(stream):
            return self._run(x, residual, batch)

    def _run(self, x: torch.Tensor, residual: Optional[torch.Tensor], batch: Batch):
        T, w, c = batch.tokens, self.w, self.cache
        if x.shape[0] != T or T > self.tokens:
            raise ValueError(f"decoder layer: {x.shape[0]} rows for a batch of {T} tokens, at most {self.tokens}")
        if _is_joined(w) and not self.joined:
            raise ValueError("decoder layer: nothing comes `after` it that would take the norm, gate or scale of its output")
        if T == 0:
            return (self.y if self.dense else self.experts.y)[:0], self.residual[1][:0]
        x8, x8s, qkv, q, attn = self.x8[:T], self.x8_scale[:T], self.qkv[:T], self.q[:T], self.attn[:T]
        hq, hk = self.heads, self.kv_heads
        r1, r2 = self.residual[0][:T], self.residual[1][:T]
        _take_output(self.after, x, residual, self.eps, w.attn_norm, residual_out=r1, q=x8, scale=x8s)
        pw.pw_fp8_linear(x8, x8s, w.qkv.codes, w.qkv.scale, qkv.view(T, -1), self.status)
        pw.pw_rope_append(qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:], self.turns, c.k, c.v, batch.page_table,
                          batch.q_offsets, batch.kv_lens, q, self.status, interleaved=self.interleaved,
                          factor=self.rope_factor)
        pw.pw_paged_attention(q, c.k, c.v, batch.page_table, batch.q_offsets, batch.kv_lens, attn, self.ws, self.status,
                              scale=self.head_dim ** -0.5, window=self.window, max_q_len=batch.max_q_len,
                              max_kv_len=batch.max_kv_len, sinks=self.sinks)
        a8, a8s = self.attn8[:T], self.attn8_scale[:T]
        pw.pw_quantize_fp8(attn.view(T, -1), a8, a8s)
        pw.pw_fp8_linear(a8, a8s, w.out.codes, w.out.scale, self.o[:T], self.status)
        if self.dense:
            f8, f8s, y = self.ff8[:T], self.ff8_scale[:T], self.y[:T]
            _add_norm(self.o[:T], r1, self.eps, w.ffn_norm, w.post_attn_norm, w.attn_gate, w.residual_scale, residual_out=r2,
                      q=x8, scale=x8s)
            pw.pw_fp8_gated_linear(x8, x8s, w.gate.codes, w.gate.scale, w.up.codes, w.up.scale, self.status, q=f8, scale=f8s,
                                   activation=self.activation)
            pw.pw_fp8_linear(f8, f8s, w.down.codes, w.down.scale, y, self.status)
            return y, r2
        h = self.h[:T]
        _add_norm(self.o[:T], r1, self.eps, w.ffn_norm, w.post_attn_norm, w.attn_gate, w.residual_scale, residual_out=r2, y=h)
        logits = self.logits[:T]
        torch.mm(self.h32[:T].copy_(h), w.router.t(), out=logits)   # the router: a few columns in 32 bits
        y = self.moe(T)(self.index, h, logits)[:T]
        return y, r2


@dataclass
class Scores:
    """What a model says of next tokens, by rows of the call (the head's buffers)."""
    logits: torch.Tensor                    # fp16 [T][V]
    lse: torch.Tensor                       # fp32 [T]
    entropy: torch.Tensor                   # fp32 [T]
    logprobs: Optional[torch.Tensor]        # fp32 [T][n], of the targets
    top_ids: Optional[torch.Tensor]         # int32 [T][top]
    top_logprobs: Optional[torch.Tensor]    # fp32 [T][top]


class Head:
    """The model's end: the last layer's output joins the residual, the last norm,
    the projection to the vocabulary, and the probabilities of next tokens; buffers
    for up to ``tokens`` rows with ``given`` targets each.  ``after``: the last
    layer.  ``temperature`` divides the logits before the probabilities."""

    def __init__(self, norm: torch.Tensor, weight: Fp8Weight, tokens: int, top: int = 0, given: int = 1,
                 after: Optional[DecoderLayer] = None, eps: float = 1e-5, temperature: float = 1.0):
        V, H = weight.codes.shape
        dev = norm.device
        assert norm.shape == (H,)
        if not temperature > 0:
            raise ValueError(f"head: temperature {temperature}")
        self.norm, self.weight, self.after, self.eps, self.scale = norm, weight, after, eps, 1.0 / temperature
        self.tokens, self.given, self.top = tokens, given, top
        _comes_after(after, eps)

        def empty(*shape, dtype=torch.float32):
            return torch.empty(shape, dtype=dtype, device=dev)
        self.x8, self.x8_scale = empty(tokens, H + -H % 16, dtype=torch.float8_e4m3fn)[:, :H], empty(tokens, -(-H // 128))
        self.logits = empty(tokens, V + -V % 16, dtype=torch.float16)[:, :V]   # rows at 32-byte addresses
        self.lse, self.entropy, self.logprobs = empty(tokens), empty(tokens), empty(tokens, given)
        self.top_ids, self.top_logprobs = empty(tokens, top, dtype=torch.int32), empty(tokens, top)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        _settle(dev)

    def __call__(self, x: torch.Tensor, residual: Optional[torch.Tensor], targets: Optional[torch.Tensor] = None,
                 stream=None) -> Scores:
        """x, residual: the last layer's results, or some of their rows, fp16
        [T][H]; targets int32 [T][n] or None.  The results are the head's buffers,
        valid until its next call."""
        T, n = x.shape[0], 0 if targets is None else targets.shape[1]
        if T > self.tokens or n > self.given:
            raise ValueError(f"head: {T} rows of {n} targets, at most {self.tokens} of {self.given}")
        s = Scores(self.logits[:T], self.lse[:T], self.entropy[:T], self.logprobs[:T, :n] if n else None,
                   self.top_ids[:T] if self.top else None, self.top_logprobs[:T] if self.top else None)
        if T == 0:
            return s
        x8, x8s = self.x8[:T], self.x8_scale[:T]
        with _on(stream):
            _take_output(self.after, x, residual, self.eps, self.norm, q=x8, scale=x8s)
            pw.pw_fp8_linear(x8, x8s, self.weight.codes, self.weight.scale, s.logits, self.status)
            pw.pw_token_logprobs(s.logits, targets=targets if n else None, logprobs=s.logprobs, lse=s.lse, entropy=s.entropy,
                                 top_ids=s.top_ids, top_logprobs=s.top_logprobs, scale=self.scale)
        return s
