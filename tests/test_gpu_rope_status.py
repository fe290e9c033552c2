"""GPU: what the rotary append says of tokens that have no place in the cache."""
import pytest
import torch

from test_gpu_attn_half import Batch, DEV, _gpu, pw, status  # noqa: F401

pytestmark = pytest.mark.gpu


def append(b, lens, table=None):
    turns, _ = pw.pw_rope_turns(64)
    kc, vc, st = b.k.clone(), b.v.clone(), status()
    qo = torch.full((b.T, 2, 64), 7.0, dtype=torch.float16, device=DEV)
    pw.pw_rope_append(b.qkv[:, :2], b.qkv[:, 2:3], b.qkv[:, 3:], turns.to(DEV), kc, vc, b.table if table is None else table,
                      b.offsets, torch.tensor(lens, dtype=torch.int32, device=DEV), qo, st)
    return qo, kc, vc, int(st.item())


@pytest.mark.parametrize("length", [1, 0, -4, 10 ** 9, 2 ** 31 - 1])
def test_lengths_that_cannot_be(length):
    """Below the new tokens, or past the table: an invalid length, not a missing
    page (a caller that reloads the page would ask for ever); the other
    sequence is appended, and no key or value is stored outside a place."""
    b = Batch([2, 2], [20, 17], 2, 1, 64, 16, torch.float16, 1)
    good, kg, vg, st = append(b, [20, 17])
    assert st == 0
    qo, kc, vc, st = append(b, [20, length])
    assert st == pw.PW_ERR_INVALID_ARG
    assert torch.equal(qo[:2], good[:2]) and not (qo[2:] == 7).all()
    last = int(b.table[1, 1]), int(b.table[1, 0])      # sequence 1's pages: keys 16 and 15 go there with length 17
    for got, want, before in ((kc, kg, b.k), (vc, vg, b.v)):
        for page in range(got.shape[0]):
            expect = before if page in last else want
            rows = slice(0, 1) if page == last[1] and length == 1 else slice(0, 0)   # length 1: one token has a place
            keep = torch.ones(16, dtype=torch.bool, device=DEV)
            keep[rows] = False
            assert torch.equal(got[page][keep].view(torch.int16), expect[page][keep].view(torch.int16))


def test_a_missing_page_is_not_resident():
    b = Batch([2], [20], 2, 1, 64, 16, torch.float16, 1)
    for bad in (-1, b.k.shape[0]):
        t = b.table.clone()
        t[0, 1] = bad
        assert append(b, [20], t)[3] == pw.PW_ERR_NOT_RESIDENT
