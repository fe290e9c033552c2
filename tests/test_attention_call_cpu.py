"""The attention's wrapper without a GPU: where positional arguments go."""
import struct

import pytest
import torch

pw = pytest.importorskip("any_precision_bit_pw_gb300.pw")


def test_a_stream_by_position(monkeypatch):
    """Options that were added later come behind the stream: the sixteenth argument is still that."""
    seen = []

    class Lib:
        def __getattr__(self, name):
            return lambda *args: seen.append((name, args)) or 0
    monkeypatch.setattr(pw, "lib", lambda: Lib())
    monkeypatch.setattr(pw, "_queue", lambda stream, dev: ("stream", stream))
    f16, i32 = dict(dtype=torch.float16), dict(dtype=torch.int32)
    q, out, cache = torch.zeros(1, 2, 64, **f16), torch.zeros(1, 2, 64, **f16), torch.zeros(4, 16, 1, 64, **f16)
    table, offsets, lens, status = (torch.zeros(n, **i32) for n in ((1, 4), 2, 1, 1))
    ws, lse = torch.zeros(64, dtype=torch.uint8), torch.zeros(1, 2)
    before = (q, cache, cache, table, offsets, lens, out, ws, status, 0.125, True, 8, 1, 64, lse)
    monkeypatch.setattr(pw, "_dtype16", lambda t, name: pw.PW_DTYPE_F16)
    pw.pw_paged_attention(*before, 0x5000)
    pw.pw_paged_attention(*before, 0x6000, sinks=3)
    assert [n for n, _ in seen] == ["pw_paged_attention", "pw_paged_attention_ex"]
    assert seen[0][1][-1] == ("stream", 0x5000) and seen[1][1][-1] == ("stream", 0x6000)
    assert struct.unpack("@8i", seen[1][1][1])[0] == 3
