"""Layers that follow one another, without a GPU: the buffers that they share, and how one
layer's output joins the residual in the next."""
import pytest
import torch

from test_decoder_dense_cpu import D, H, HEADS, KV, V, layer, log, weight, weights  # noqa: F401
from any_precision_bit_pw_gb300 import decoder
from any_precision_bit_pw_gb300.decoder import DecoderLayer, DecoderWeights, Fp8Weight, Head, PagedCache

W = 200   # another width of the dense block


def narrow():
    w = weights()
    w.gate, w.up, w.down = weight(W, H), weight(W, H), weight(H, W)
    return w


def test_memory_is_settled_where_it_is_taken(monkeypatch):
    """A constructor that takes memory waits for what the current stream has under way, since
    calls may run on another; one that takes none does not."""
    settled = []
    monkeypatch.setattr(decoder, "_settle", lambda dev: settled.append(dev))

    def count(f):
        settled.clear()
        return f(), len(settled)
    caches = [count(lambda: PagedCache(8, 16, KV, D, device="cpu")) for _ in range(4)]
    assert [n for _, n in caches] == [1] * 4
    make = lambda i, w, **kw: DecoderLayer(None, 0, w, HEADS, caches[i][0], 8, **kw)  # noqa: E731
    first, n = count(lambda: make(0, weights()))
    assert n == 1
    same, n = count(lambda: make(1, weights(), share=first))
    assert n == 0 and same.ff8 is first.ff8
    other, n = count(lambda: make(2, narrow(), share=first))
    assert n == 1 and other.ff8.shape == (8, W) and other.x8 is first.x8
    again, n = count(lambda: make(3, narrow(), share=other))
    assert n == 0 and again.ff8 is other.ff8 and again.y is other.y
    assert count(lambda: Head(torch.ones(H).half(), weight(V, H), 8))[1] == 1


def test_buffers_are_not_shared_across_widths_and_devices():
    """Dense layers have no stack that would tell: another hidden width, another device."""
    first = layer()

    def another(h, device="cpu"):
        def matrix(n, k):
            return Fp8Weight(torch.zeros(n, k, dtype=torch.float8_e4m3fn, device=device), torch.ones(-(-n // 128), -(-k // 128), device=device))
        one = torch.ones(h, device=device).half()
        w = DecoderWeights(one, one, matrix((HEADS + 2 * KV) * D, h), matrix(h, HEADS * D), gate=matrix(W, h), up=matrix(W, h),
                           down=matrix(h, W))
        return DecoderLayer(None, 0, w, HEADS, PagedCache(8, 16, KV, D, device=device), 8, share=first)
    assert another(H).x8 is first.x8
    for bad in ((2 * H, "cpu"), (H, "meta")):
        with pytest.raises(ValueError, match="shared"):
            another(*bad)


@pytest.mark.parametrize("kw", [dict(post_ffn_norm=torch.ones(H).half()), dict(ffn_gate=torch.ones(H).half()), dict(residual_scale=0.5)])
def test_an_output_that_nothing_joins_is_refused(log, kw):  # noqa: F811
    """A norm, gate or scale of a layer's output is taken by what was made `after` it: without that,
    the next layer would add the bare output."""
    first = layer(weights(**kw))
    second = layer(share=first)                     # (not told what comes in)
    x, b = torch.zeros(2, H).half(), first.cache.batch([0], [2])
    with pytest.raises(ValueError, match="after"):
        second(*first(x, None, b), b)
    assert not log
    second = layer(share=first, after=first)
    y, r = second(*first(x, None, b), b)
    assert [n for n, _, _ in log].count("pw_norm_add_norm") == 1 + ("residual_scale" in kw)
    # a head, or the caller
    for L, end in ((layer(weights(**kw)), True), (layer(weights(**kw), joined=True), False)):
        if end:
            Head(torch.ones(H).half(), weight(V, H), 8, after=L)
        assert L(x, None, L.cache.batch([0], [2]))[0].shape == (2, H)
    # plain layers need nobody
    plain = layer()
    assert plain(x, None, plain.cache.batch([0], [2]))[0].shape == (2, H)


def test_norms_in_one_kernel_have_one_eps():
    """The norm of a layer's output runs with that of what comes after it: another eps would be lost."""
    first = layer(weights(post_ffn_norm=torch.ones(H).half()), eps=1e-6)
    for make in (lambda **kw: layer(after=first, **kw), lambda **kw: Head(torch.ones(H).half(), weight(V, H), 8, after=first, **kw)):
        with pytest.raises(ValueError, match="eps"):
            make()
        assert not first.joined
    for make in (lambda **kw: layer(after=first, **kw), lambda **kw: Head(torch.ones(H).half(), weight(V, H), 8, after=first, **kw)):
        assert make(eps=1e-6).after is first and first.joined
    assert layer(after=layer(weights(ffn_gate=torch.ones(H).half()), eps=1e-6)).eps == 1e-5      # no norm of the output


def test_an_output_without_its_residual_is_refused(log):  # noqa: F811
    """What comes after a layer with a norm, gate or scale of its output takes both results of it."""
    first = layer(weights(ffn_gate=torch.ones(H).half()))
    x, b = torch.zeros(2, H).half(), first.cache.batch([0], [2])
    for then in (lambda x, r, L=layer(after=first): L(x, r, b), Head(torch.ones(H).half(), weight(V, H), 8, after=first)):
        with pytest.raises(ValueError, match="residual"):
            then(x, None)
        assert not log
        then(x, x)
        assert log[0][0] == "pw_norm_add_norm"
        log.clear()
    plain = layer()
    layer(after=plain)(x, None, b)
    assert log[0][0] == "pw_add_rmsnorm"
