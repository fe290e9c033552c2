"""A decoder layer around the mixed-precision experts: residual norm, 8-bit
projections, rotary positions, attention over a paged cache, and the routed
expert layer of ``layer.py``, one stream, buffers allocated once.

    cache = PagedCache(pages=4096, page_size=16, kv_heads=8, head_dim=128)
    layer = DecoderLayer(stack, 0, weights, heads=32, cache=cache, tokens=64)
    batch = cache.batch([3, 7], [1, 1])      # one new token of sequences 3 and 7
    x, residual = layer(x, residual, batch)  # both fp16 [T][H]

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
        self.free_pages.extend(reversed(self.pages.pop(seq, [])))
        self.lens.pop(seq, None)


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
    router: torch.Tensor       # [experts][H] fp32


class DecoderLayer:
    """One layer's calls, and buffers for up to ``tokens`` tokens.  Layers that
    run one after another on one stream can use the buffers of the first of them
    (``share``): each reads its inputs before it writes its results, so the
    results of one may be the inputs of the next.  ``max_batch`` goes to the
    attention's workspace query, whose answer holds for any number of sequences.
    """

    BUFFERS = ("x8", "x8_scale", "qkv", "q", "attn", "attn8", "attn8_scale", "o", "h", "residual", "h32", "logits", "status",
               "ws", "experts")

    def __init__(self, stack: APLMoEStack, index: int, weights: DecoderWeights, heads: int, cache: PagedCache,
                 tokens: int, rotary_dim: Optional[int] = None, rope_base: float = 1e6,
                 rope_scaling: Optional[pw.pw_rope_scaling] = None, interleaved: bool = False, window: int = 0,
                 eps: float = 1e-5, max_batch: int = 256, share: Optional["DecoderLayer"] = None):
        dev, H = stack.device, stack.H
        self.stack, self.index, self.w, self.cache = stack, index, weights, cache
        self.heads, self.kv_heads, self.head_dim = heads, cache.k.shape[2], cache.k.shape[3]
        self.eps, self.window, self.interleaved, self.tokens = eps, window, interleaved, tokens
        turns, self.rope_factor = pw.pw_rope_turns(self.head_dim if rotary_dim is None else rotary_dim, rope_base, rope_scaling)
        self.turns = turns.to(dev)
        D, wide = self.head_dim, (heads + 2 * self.kv_heads) * self.head_dim
        assert tuple(weights.qkv.codes.shape) == (wide, H) and tuple(weights.out.codes.shape) == (H, heads * D)
        if share is not None:
            if (share.stack, share.heads, share.kv_heads, D, tokens) != (stack, heads, self.kv_heads, share.head_dim, share.tokens):
                raise ValueError("decoder layer: buffers are shared between layers of one stack with equal heads and tokens")
            for name in self.BUFFERS:
                setattr(self, name, getattr(share, name))
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
        self.h32, self.logits = empty(tokens, H, dtype=torch.float32), empty(tokens, stack.routed, dtype=torch.float32)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)   # of every call, the experts' too
        n = pw.pw_paged_attention_workspace(tokens, max_batch, heads, self.kv_heads, D)
        self.ws = torch.zeros(n, dtype=torch.uint8, device=dev)
        # the experts' workspace grows with the tokens: one, for the most, serves every count
        self.experts = MoECall(stack, tokens)
        self.experts.status = self.status
        if dev.type == "cuda":   # the layer may be called on any stream: its buffers are free and zeroed by then
            torch.cuda.current_stream(dev).synchronize()

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
        if T == 0:
            return self.experts.y[:0], self.residual[1][:0]
        x8, x8s, qkv, q, attn = self.x8[:T], self.x8_scale[:T], self.qkv[:T], self.q[:T], self.attn[:T]
        hq, hk = self.heads, self.kv_heads
        r1, r2 = self.residual[0][:T], self.residual[1][:T]
        pw.pw_add_rmsnorm(x, w.attn_norm, self.eps, residual=residual, residual_out=r1, q=x8, scale=x8s)
        pw.pw_fp8_linear(x8, x8s, w.qkv.codes, w.qkv.scale, qkv.view(T, -1), self.status)
        pw.pw_rope_append(qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:], self.turns, c.k, c.v, batch.page_table,
                          batch.q_offsets, batch.kv_lens, q, self.status, interleaved=self.interleaved,
                          factor=self.rope_factor)
        pw.pw_paged_attention(q, c.k, c.v, batch.page_table, batch.q_offsets, batch.kv_lens, attn, self.ws, self.status,
                              scale=self.head_dim ** -0.5, window=self.window, max_q_len=batch.max_q_len,
                              max_kv_len=batch.max_kv_len)
        a8, a8s = self.attn8[:T], self.attn8_scale[:T]
        pw.pw_quantize_fp8(attn.view(T, -1), a8, a8s)
        pw.pw_fp8_linear(a8, a8s, w.out.codes, w.out.scale, self.o[:T], self.status)
        h = self.h[:T]
        pw.pw_add_rmsnorm(self.o[:T], w.ffn_norm, self.eps, residual=r1, residual_out=r2, y=h)
        logits = self.logits[:T]
        torch.mm(self.h32[:T].copy_(h), w.router.t(), out=logits)   # the router: a few columns in 32 bits
        y = self.moe(T)(self.index, h, logits)[:T]
        return y, r2
