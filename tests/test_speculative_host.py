"""Host side of PagedKVCache's speculative decoding (CPU only, the library's calls replaced): which
pages the accepted paths take, when a window is flushed, and what is refused before anything
changes."""
import pytest
import torch

from bit_mixed_precision_channel_b200 import binding as kb
from bit_mixed_precision_channel_b200 import cache as kc


@pytest.fixture
def calls(monkeypatch):
    log = []

    def append_path(cfg, k, v, path, n_path, taken, res_k, res_v, res_len, err, stream):
        room = cfg.page_tokens - res_len
        n = torch.minimum(n_path - taken, room)
        res_len += n
        taken += n
        log.append(("append", res_len.tolist()))

    def flush(cfg, res_k, res_v, res_len, new_page, table, num_pages, pool, err, stream):
        for b in range(len(res_len)):
            if res_len[b] == cfg.page_tokens:
                assert new_page[b] >= 0
                table[b, num_pages[b]] = new_page[b]
                num_pages[b] += 1
                res_len[b] = 0
        log.append(("flush", res_len.tolist()))

    monkeypatch.setattr(kc.kb, "append_path", append_path)
    monkeypatch.setattr(kc.kb, "flush_residual", flush)
    return log


def make(batch=3, pool_pages=12, max_pages=6):
    cfg = kb.Config(num_q_heads=4, num_kv_heads=1, page_tokens=32, num_boost=16)
    return kc.PagedKVCache(cfg, batch, max_pages=max_pages, pool_pages=pool_pages, device="cpu")


def accept(c, n_path, T=128):
    c.accept(None, None, torch.zeros(c.batch, T, dtype=torch.int32), n_path)


def test_paths_across_windows(calls):
    c = make()
    c.host_res_len = [5, 31, 0]
    c.res_len.copy_(torch.tensor([5, 31, 0]))
    accept(c, [3, 1, 100])
    assert c.host_res_len == [8, 0, 4] and c.res_len.tolist() == [8, 0, 4]
    assert [len(p) for p in c.host_pages] == [0, 1, 3] and c.num_pages.tolist() == [0, 1, 3]
    for b in range(3):
        n = len(c.host_pages[b])
        assert c.page_table[b, :n].tolist() == c.host_pages[b]
    assert len(set(sum(c.host_pages, []))) == 4 and len(c.free) == 8
    assert [x for x, _ in calls] == ["append", "flush"] * 3 + ["append"]


def test_short_paths_take_one_call_and_no_flush(calls):
    c = make()
    accept(c, [0, 4, 31])
    assert [x for x, _ in calls] == ["append"] and c.host_res_len == [0, 4, 31] and len(c.free) == 12


def test_a_step_after_an_accepted_path_reserves_its_own_page(calls):
    c = make(batch=1)
    accept(c, [32 + 31])
    assert c.host_new_page == [c.host_pages[0][0]]
    assert c.reserve_flush_pages() == [0]  # the window will fill: a fresh page, not the one already used
    assert c.new_page.tolist() == c.host_new_page and c.host_new_page[0] not in c.host_pages[0]


def test_refused_before_anything_changes(calls):
    c = make(pool_pages=2)
    for n in ([1, 1], [0, 0, 129], [0, -1, 0]):
        with pytest.raises(ValueError, match="n_path"):
            accept(c, n)
    with pytest.raises(RuntimeError, match="pool exhausted"):
        accept(c, [32, 32, 32])
    with pytest.raises(RuntimeError, match="page table full"):
        accept(make(max_pages=1), [64, 0, 0])
    assert calls == [] and c.host_res_len == [0, 0, 0] and len(c.free) == 2


def test_attend_few_needs_a_choice(calls):
    with pytest.raises(RuntimeError, match="select"):
        make().attend_few(None, None)


def test_buffers_a_captured_graph_may_hold_are_never_replaced(monkeypatch):
    seen = []
    monkeypatch.setattr(kc.kb, "tree_attention", lambda *a: seen.append(a[13]))
    monkeypatch.setattr(kc.kb, "select_pages", lambda *a: None)
    for gqa in (1, 2, 4, 8):
        cfg = kb.Config(num_q_heads=2 * gqa, num_kv_heads=2, page_tokens=32, num_boost=16)
        c = kc.PagedKVCache(cfg, 3, max_pages=6, pool_pages=12, device="cpu")
        del seen[:]
        for T in range(1, kb.MAX_DRAFT + 1):
            c.verify(torch.empty(3, T, 2 * gqa, 128), None, None, None, None, None)
            assert seen[-1] is seen[0] and seen[0].numel() >= kb.tree_workspace_bytes(cfg, 3, T), T
        first = c.select(None, 4)
        other = c.select(None, 5)
        assert other[0].shape == (3, 2, 5) and c.sel is other[0] and c.n_sel is other[1] is not first[1]
        again = c.select(None, 4)
        assert again[0] is first[0] is c.sel and again[1] is first[1] is c.n_sel


def test_scratch_is_not_allocated_in_a_capture(monkeypatch):
    c = make()
    c.device = torch.device("cuda")
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    with pytest.raises(RuntimeError, match="before a capture"):
        c.verify(torch.empty(3, 2, 4, 128), None, None, None, None, None)
    assert c.tree_workspace is None
    with pytest.raises(ValueError, match="at least one page"):
        c.select(None, 0)


def test_a_refused_choice_leaves_the_last_one(monkeypatch):
    def select_pages(cfg, pool, q, table, num, sel, n_sel, n_first, n_recent, err, stream):
        if n_first + n_recent > sel.shape[2]:
            raise kb.KVQError("kvq_select_pages", 1)

    monkeypatch.setattr(kc.kb, "select_pages", select_pages)
    c = make()
    first = c.select(None, 4)
    with pytest.raises(kb.KVQError):
        c.select(None, 1)
    assert c.sel is first[0] and c.n_sel is first[1]
