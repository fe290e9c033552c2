"""The decoder layer without a GPU: what it calls, in which order and on which
stream.  libpw's launches and torch's streams are recorded, not run."""
from contextlib import contextmanager
from types import SimpleNamespace

import pytest
import torch

pw = pytest.importorskip("any_precision_bit_pw_gb300.pw")
from any_precision_bit_pw_gb300 import decoder  # noqa: E402
from any_precision_bit_pw_gb300.decoder import DecoderLayer, DecoderWeights, Fp8Weight, PagedCache  # noqa: E402

HEADS, KV, D, H, EXPERTS = 4, 2, 64, 256, 8
LAUNCHES = ("pw_add_rmsnorm", "pw_quantize_fp8", "pw_fp8_linear", "pw_rope_append", "pw_paged_attention")


class FakeMoE:
    def __init__(self, stack, tokens, **kw):
        self.T, self.status = tokens, torch.zeros(1, dtype=torch.int32)
        self.y = torch.zeros(max(tokens, 1), H, dtype=torch.float16)
        self.log = stack.log
        self.log.append(("MoECall", stack.current()))

    def __call__(self, layer, x, logits, stream=None, **kw):
        self.log.append(("experts", self.log.stream if stream is None else stream))
        return self.y[: self.T]


class Log(list):
    stream = None      # torch's current stream; None: the default one


@pytest.fixture
def log(monkeypatch):
    log = Log()

    def record(name):
        def call(*args, stream=None, **kw):
            log.append((name, log.stream if stream is None else stream))
        return call
    for name in LAUNCHES:
        monkeypatch.setattr(pw, name, record(name))
    monkeypatch.setattr(decoder, "MoECall", FakeMoE)

    @contextmanager
    def on(stream):
        before, log.stream = log.stream, stream
        yield
        log.stream = before
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: ("external", handle))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda: "default")
    mm = torch.mm

    def product(*args, **kw):
        log.append(("router", log.stream))
        return mm(*args, **kw)
    monkeypatch.setattr(torch, "mm", product)
    return log


def weight(n, k):
    return Fp8Weight(torch.zeros(n, k, dtype=torch.float8_e4m3fn), torch.ones(-(-n // 128), -(-k // 128)))


def layer(log, tokens=8, **kw):
    stack = SimpleNamespace(device=torch.device("cpu"), H=H, routed=EXPERTS, log=log, current=lambda: log.stream)
    w = DecoderWeights(torch.ones(H).half(), torch.ones(H).half(), weight((HEADS + 2 * KV) * D, H), weight(H, HEADS * D),
                       torch.zeros(EXPERTS, H))
    return DecoderLayer(stack, 0, w, HEADS, PagedCache(8, 16, KV, D, device="cpu"), tokens, **kw)


ORDER = ["pw_add_rmsnorm", "pw_fp8_linear", "pw_rope_append", "pw_paged_attention", "pw_quantize_fp8", "pw_fp8_linear",
         "pw_add_rmsnorm", "router", "experts"]


@pytest.mark.parametrize("given,want", [(None, None), (0x5000, ("external", 0x5000)), (0, "default"), (1, "default")])
def test_one_stream_for_the_whole_layer(log, given, want):
    """The router's product is torch's: it has to follow the norm and precede
    the experts on the stream that they run on."""
    L = layer(log)
    log.clear()
    L(torch.zeros(3, H).half(), None, L.cache.batch([0, 1], [2, 1]), stream=given)
    calls = [c for c in log if c[0] != "MoECall"]
    assert [n for n, _ in calls] == ORDER
    where = {s for _, s in calls}
    assert where == {want}


def test_one_expert_workspace_for_every_token_count(log, monkeypatch):
    """Ragged chunks: the buffers are the constructor's, whatever the counts,
    and one status word takes the experts' failures too."""
    L = layer(log)
    assert [n for n, _ in log] == ["MoECall"] and L.experts.T == 8 and L.experts.status is L.status
    batches = [L.cache.batch([i], [n]) for i, n in enumerate((5, 8, 1, 3))]

    def allocate(*args, **kw):
        raise AssertionError("an allocation in a call")
    for name in ("empty", "zeros", "empty_like", "zeros_like"):
        monkeypatch.setattr(torch, name, allocate)
    monkeypatch.setattr(torch.Tensor, "float", allocate)
    x = torch.ones(8, H).half()
    for b in batches:
        y, r = L(x[: b.tokens], None, b)
        assert y.shape == r.shape == (b.tokens, H) and y.data_ptr() == L.experts.y.data_ptr()
    assert [n for n, _ in log].count("MoECall") == 1


def test_layers_share_buffers(log):
    first = layer(log)
    stack, w = first.stack, first.w
    log.clear()
    second = DecoderLayer(stack, 1, w, HEADS, PagedCache(8, 16, KV, D, device="cpu"), 8, share=first)
    assert not log and all(getattr(second, n) is getattr(first, n) for n in DecoderLayer.BUFFERS)
    mine = {n for n, v in vars(first).items() if isinstance(v, (torch.Tensor, list, FakeMoE)) and n != "turns"}
    assert mine == set(DecoderLayer.BUFFERS)          # no buffer is left out
    for kw in (dict(tokens=4), dict(stack=SimpleNamespace(**vars(stack), name="another"))):
        args = {**dict(stack=stack, tokens=8), **kw}
        with pytest.raises(ValueError):
            DecoderLayer(args["stack"], 1, w, HEADS, PagedCache(8, 16, KV, D, device="cpu"), args["tokens"], share=first)


@pytest.mark.parametrize("seqs", [[], [3], [3, 1]])
def test_a_step_without_tokens(log, seqs):
    """No sequences, or none with new tokens: empty results, no launch."""
    L = layer(log)
    L.cache.batch([3], [5])
    log.clear()
    batch = L.cache.batch(seqs, [0] * len(seqs))
    assert batch.tokens == 0 and batch.q_offsets.tolist() == [0] * (len(seqs) + 1)
    y, r = L(torch.zeros(0, H).half(), None, batch)
    assert y.shape == r.shape == (0, H) and y.dtype == r.dtype == torch.float16
    assert [n for n, _ in log if n != "MoECall"] == []
    with pytest.raises(ValueError):
        L(torch.zeros(1, H).half(), None, batch)


def test_a_weight_is_allocated_on_its_stream(log, monkeypatch):
    """What one stream has freed another may not write: the codes come from the
    memory of the stream that fills them."""
    empty = torch.empty

    def allocate(*args, **kw):
        log.append(("empty", log.stream))
        return empty(*args, **kw)
    monkeypatch.setattr(torch, "empty", allocate)
    w = Fp8Weight.quantize(torch.zeros(130, 200).half(), stream=0x5000)
    assert w.codes.shape == (130, 200) and w.scale.shape == (2, 2) and w.codes.stride(0) % 16 == 0
    assert log == [(n, ("external", 0x5000)) for n in ("empty", "empty", "pw_quantize_fp8")]
