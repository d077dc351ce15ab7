"""Tree attention's scratch is not allocated on a stream that is being captured, whichever stream is
the current one (CPU only, the library's calls and the streams replaced)."""
import contextlib

import pytest
import torch

from bit_mixed_precision_channel_b200 import binding as kb
from bit_mixed_precision_channel_b200 import cache as kc


def test_a_captured_stream_passed_as_an_argument(monkeypatch):
    cfg = kb.Config(num_q_heads=4, num_kv_heads=1, page_tokens=32, num_boost=16)
    c = kc.PagedKVCache(cfg, 1, max_pages=2, pool_pages=2, device="cpu")
    current = ["default"]

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    calls = []
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: current[-1] == "captured")
    monkeypatch.setattr(kc.kb, "tree_attention", lambda *a: calls.append(a))
    monkeypatch.setattr(kc.torch, "zeros", lambda *a, **k: torch.empty(0))
    c.device = torch.device("cuda")
    with pytest.raises(RuntimeError, match="before a capture"):
        c.verify(None, None, None, None, None, None, stream="captured")
    assert c.tree_workspace is None and not calls
    c.verify(None, None, None, None, None, None, stream="other")
    c.verify(None, None, None, None, None, None, stream="captured")  # the scratch is there
    assert len(calls) == 2
