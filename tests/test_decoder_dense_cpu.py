"""Dense layers, norms on both sides, windows with first keys and the model's end
without a GPU: what is called, in which order, with which weights, and the cache's pages."""
import pytest
import torch

pw = pytest.importorskip("any_precision_bit_pw_gb300.pw")
from any_precision_bit_pw_gb300 import decoder  # noqa: E402
from any_precision_bit_pw_gb300.decoder import DecoderLayer, DecoderWeights, Fp8Weight, Head, PagedCache  # noqa: E402

HEADS, KV, D, H, I, V = 4, 2, 64, 256, 300, 1000


@pytest.fixture
def log(monkeypatch):
    calls = []

    def record(name):
        def call(*args, **kw):
            calls.append((name, args, kw))
        return call
    for name in ("pw_add_rmsnorm", "pw_quantize_fp8", "pw_fp8_linear", "pw_rope_append", "pw_paged_attention",
                 "pw_norm_add_norm", "pw_fp8_gated_linear", "pw_token_logprobs"):
        monkeypatch.setattr(pw, name, record(name))
    return calls


def weight(n, k):
    return Fp8Weight(torch.zeros(n, k, dtype=torch.float8_e4m3fn), torch.ones(-(-n // 128), -(-k // 128)))


def weights(**kw):
    one = lambda: torch.ones(H).half()  # noqa: E731
    return DecoderWeights(one(), one(), weight((HEADS + 2 * KV) * D, H), weight(H, HEADS * D), gate=weight(I, H), up=weight(I, H),
                          down=weight(H, I), **kw)


def layer(w=None, **kw):
    return DecoderLayer(None, 0, w or weights(), HEADS, PagedCache(8, 16, KV, D, device="cpu"), 8, **kw)


def test_a_dense_layer(log):
    L = layer()
    assert L.experts is None and L.ff8.stride(0) % 16 == 0
    y, r = L(torch.zeros(3, H).half(), None, L.cache.batch([0, 1], [2, 1]))
    assert [n for n, _, _ in log] == ["pw_add_rmsnorm", "pw_fp8_linear", "pw_rope_append", "pw_paged_attention",
                                      "pw_quantize_fp8", "pw_fp8_linear", "pw_add_rmsnorm", "pw_fp8_gated_linear", "pw_fp8_linear"]
    assert y.data_ptr() == L.y.data_ptr() and y.shape == r.shape == (3, H)
    # the codes go from the norm to the gated block to the down projection
    assert log[6][2]["q"].data_ptr() == log[7][1][0].data_ptr() and log[7][2]["q"].data_ptr() == log[8][1][0].data_ptr()
    assert layer()(torch.zeros(0, H).half(), None, L.cache.batch([0], [0]))[0].shape == (0, H)


def test_norms_on_both_sides(log):
    """A layer's own norms join its attention's output; those of its feed-forward
    block are taken by the layer, or the head, that comes after it."""
    posts = [torch.full((H,), float(i)).half() for i in range(4)]
    first = layer(weights(post_attn_norm=posts[0], post_ffn_norm=posts[1], attn_gate=posts[2], ffn_gate=posts[3],
                          residual_scale=0.5))
    second = layer(after=first, share=first)
    head = Head(torch.ones(H).half(), weight(V, H), 8, top=3, after=second)
    x, b = torch.zeros(2, H).half(), first.cache.batch([0], [2])
    y, r = second(*first(x, None, b), b)
    head(y, r)
    joins = [(n, kw.get("post_weight"), kw.get("gate"), kw.get("residual_scale")) for n, _, kw in log if "norm" in n]
    assert joins == [("pw_add_rmsnorm", None, None, None), ("pw_norm_add_norm", posts[0], posts[2], 0.5),
                     ("pw_norm_add_norm", posts[1], posts[3], 0.5), ("pw_add_rmsnorm", None, None, None),
                     ("pw_add_rmsnorm", None, None, None)]
    assert second.y is first.y and second.ff8 is first.ff8


def test_window_and_first_keys_reach_the_attention(log):
    L = layer(window=32, sinks=4)
    L(torch.zeros(1, H).half(), None, L.cache.batch([0], [1]))
    kw = [k for n, _, k in log if n == "pw_paged_attention"][0]
    assert (kw["window"], kw["sinks"]) == (32, 4)


def test_weights_of_one_kind(log):
    w = weights()
    w.router = torch.zeros(8, H)
    with pytest.raises(ValueError):
        layer(w)
    w = weights()
    w.gate = w.up = w.down = None
    with pytest.raises(ValueError):
        layer(w)
    w.router = torch.zeros(8, H)
    with pytest.raises(ValueError):        # experts without their stack
        layer(w)


def test_head(log):
    head = Head(torch.ones(H).half(), weight(V, H), 8, top=5, given=2, temperature=0.5)
    s = head(torch.zeros(3, H).half(), None, torch.zeros(3, 1, dtype=torch.int32))
    assert [n for n, _, _ in log] == ["pw_add_rmsnorm", "pw_fp8_linear", "pw_token_logprobs"]
    assert log[2][2]["scale"] == 2.0 and s.logprobs.shape == (3, 1) and s.top_ids.shape == (3, 5) and s.logits.shape == (3, V)
    assert s.logits.stride(0) % 16 == 0
    log.clear()
    assert head(torch.zeros(3, H).half(), None).logprobs is None and log[2][2]["targets"] is None
    log.clear()
    assert head(torch.zeros(0, H).half(), None).lse.shape == (0,) and not log
    for bad in ((9, 1), (3, 3)):
        with pytest.raises(ValueError):
            head(torch.zeros(bad[0], H).half(), None, torch.zeros(bad, dtype=torch.int32))
    with pytest.raises(ValueError):
        Head(torch.ones(H).half(), weight(V, H), 8, temperature=0.0)


def test_trim_gives_back_what_no_later_token_sees():
    c = PagedCache(32, 4, 1, 8, device="cpu")
    c.batch([1], [30])
    held = list(c.pages[1])
    # the next token, at 30, sees keys 21 .. 30 and 0, 1: pages 1 .. 4 (keys 4 .. 19) are gone
    assert c.trim(1, 10, 2) == 4 and c.trim(1, 10, 2) == 0
    assert c.pages[1] == [held[0], -1, -1, -1, -1] + held[5:] and len(c.free_pages) == 32 - 8 + 4
    b = c.batch([1], [1])
    assert b.page_table.tolist() == [c.pages[1]] and b.kv_lens.tolist() == [31]
    assert c.trim(1, 10) == 1 and c.pages[1][0] == -1
    assert c.trim(7, 10) == 0 and c.trim(1, 1000) == 0
    # a window that begins with a page keeps it
    c.batch([2], [12])
    assert c.trim(2, 5) == 2 and c.pages[2][2] >= 0
    for bad in ((0, 0), (4, -1)):
        with pytest.raises(ValueError):
            c.trim(1, *bad)
    c.release(1)
    c.release(2)
    assert sorted(c.free_pages) == list(range(32))
