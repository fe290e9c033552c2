"""GPU: a call's tensors have to be on the GPU that its kernel runs on."""
import pytest
import torch

from test_gpu_attn_half import Batch, DEV, _gpu, pw  # noqa: F401

pytestmark = pytest.mark.gpu


def calls():
    """(call, its tensors by name) of the five operators; outputs hold 7."""
    half = lambda *s: torch.full(s, 7.0, dtype=torch.float16, device=DEV)  # noqa: E731
    f32 = lambda *s: torch.full(s, 7.0, device=DEV)  # noqa: E731
    code = lambda *s: torch.full(s, 7, dtype=torch.uint8, device=DEV)  # noqa: E731
    st = lambda: torch.full((1,), 7, dtype=torch.int32, device=DEV)  # noqa: E731
    yield pw.pw_add_rmsnorm, dict(x=half(3, 64), weight=half(64), residual=half(3, 64), residual_out=half(3, 64), y=half(3, 64),
                                  q=code(3, 64), scale=f32(3, 1)), dict(eps=1e-5)
    yield pw.pw_quantize_fp8, dict(x=half(3, 64), q=code(3, 64), scale=f32(3, 1)), {}
    yield pw.pw_fp8_linear, dict(a=code(3, 64), a_scale=f32(3, 1), b=code(5, 64), b_scale=f32(1, 1), y=half(3, 5), status=st()), {}
    b = Batch([2], [20], 2, 1, 64, 16, torch.float16, 1)
    cache = dict(k_cache=half(*b.k.shape), v_cache=half(*b.v.shape), page_table=b.table, q_offsets=b.offsets, kv_lens=b.lens)
    turns, _ = pw.pw_rope_turns(64)
    yield pw.pw_rope_append, dict(q=half(2, 2, 64), k=half(2, 1, 64), v=half(2, 1, 64), turns=turns.to(DEV), **cache,
                                  q_out=half(2, 2, 64), status=st(),
                                  positions=torch.zeros(2, dtype=torch.int32, device=DEV)), {}
    ws = torch.zeros(pw.pw_paged_attention_workspace(2, 1, 2, 1, 64), dtype=torch.uint8, device=DEV)
    yield pw.pw_paged_attention, dict(q=half(2, 2, 64), **cache, out=half(2, 2, 64), ws=ws, status=st(), lse=f32(2, 2)), dict(scale=0.1)


def test_another_gpus_tensors_are_refused(monkeypatch):
    """The current GPU is another than the tensors': no kernel is launched there."""
    before = torch._C._cuda_getDevice()
    for f, tensors, kw in calls():
        kept = {n: t.clone() for n, t in tensors.items()}
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: before + 1)
        with pytest.raises(ValueError, match="current device"):
            f(**tensors, **kw)
        monkeypatch.undo()
        torch.cuda.synchronize()
        assert all(torch.equal(t, kept[n]) for n, t in tensors.items())


def test_each_tensor_has_to_be_there():
    for f, tensors, kw in calls():
        for name in tensors:
            with pytest.raises(ValueError):
                f(**{**tensors, name: tensors[name].cpu()}, **kw)
        f(**tensors, **kw)
    torch.cuda.synchronize()
