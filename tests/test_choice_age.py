"""A choice of pages does not outlive a flush: the flushed window's tokens are in a page that it does
not list (CPU only, the library's calls replaced)."""
import pytest
import torch

from bit_mixed_precision_channel_b200 import binding as kb
from bit_mixed_precision_channel_b200 import cache as kc


@pytest.fixture
def cache(monkeypatch):
    for name in ("select_pages", "decode_attention_sparse", "decode_attention", "append_token", "append_flush", "append_path",
                 "flush_residual", "quantize_pages"):
        monkeypatch.setattr(kc.kb, name, lambda *a: None)
    cfg = kb.Config(num_q_heads=4, num_kv_heads=1, page_tokens=32, num_boost=16)
    c = kc.PagedKVCache(cfg, 2, max_pages=6, pool_pages=12, device="cpu")
    c.host_res_len = [29, 3]
    return c


def stale(c):
    try:
        c.attend_few(None, None)
        return False
    except RuntimeError as e:
        assert "call select again" in str(e)
        return True


def accept(c, *n):
    c.accept(None, None, torch.zeros(2, 64, dtype=torch.int32), n)


def test_a_step_that_flushes_ends_a_choice(cache):
    c = cache
    c.select(None, 2)
    for flushes in (False, False, True):  # 30, 31, 32 tokens in the window
        assert not stale(c)
        c.step(None, None, None, None)
        assert stale(c) is flushes
    c.select(None, 2)
    assert not stale(c)
    c.step(None, None, None, None)
    assert not stale(c)


def test_an_accepted_path_that_flushes_ends_a_choice(cache):
    c = cache
    c.select(None, 2)
    accept(c, 2, 20)
    assert not stale(c)
    accept(c, 1, 0)
    assert stale(c)
    c.select(None, 3)
    accept(c, 0, 8)  # not this choice's business that another one was made before
    assert not stale(c)
    accept(c, 0, 1)
    assert stale(c)


def test_append_and_flush_in_one_launch(cache):
    c = cache
    c.select(None, 2)
    for flushes in (False, False, True):
        assert not stale(c)
        flushing = c.reserve_flush_pages()
        c.append_flush(None, None)
        assert stale(c) is flushes  # before the host's mirror is brought up to date, too
        c.commit_host(flushing)
        assert stale(c) is flushes


def test_a_replayed_step_ends_a_choice_by_the_mirror(cache):
    c = cache
    c.host_res_len = [31, 31]
    c.select(None, 2)
    c.commit_host(c.reserve_flush_pages())
    assert stale(c)


def test_prefill_ends_a_choice(cache):
    c = cache
    for call in (lambda: c.prefill(0, torch.zeros(40, 1, 128).half(), torch.zeros(40, 1, 128).half()),
                 lambda: c.prefill_batch(torch.zeros(2, 32, 1, 128).half(), torch.zeros(2, 32, 1, 128).half())):
        c.select(None, 2)
        assert not stale(c)
        call()
        assert stale(c)


def test_a_refused_choice_does_not_renew_the_last(cache, monkeypatch):
    c = cache
    c.select(None, 2)
    accept(c, 3, 0)

    def refuse(*a):
        raise kb.KVQError("kvq_select_pages", 1)

    monkeypatch.setattr(kc.kb, "select_pages", refuse)
    with pytest.raises(kb.KVQError):
        c.select(None, 2)
    assert stale(c)
