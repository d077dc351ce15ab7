"""Rounds of speculative decoding on one cache, as a user runs them: draft over few pages, verify the
tree over all, accept a path; the cache is then byte for byte the one that takes the same tokens
one at a time, and every attention is within the derived tolerance of 64 bits on the way."""
import numpy as np
import pytest
import torch

import oracle
from bit_mixed_precision_channel_b200 import binding as kb
from bit_mixed_precision_channel_b200 import synthetic as syn
from bit_mixed_precision_channel_b200.cache import PagedKVCache

from _kv import ocfg, to_dev
from _spec import D, assert_row, attend, pack_mask, tree_mask

pytestmark = pytest.mark.gpu


def rows_of(cache, b, h, dtype, slots=None):
    """Keys and values of sequence b, kv head h, read back from the cache, in 64 bits."""
    cfg, oc = cache.cfg, ocfg(cache.cfg)
    pool = cache.pool.view(-1, cfg.num_kv_heads, cache.record_bytes)
    ks, vs = [], []
    n, r = int(cache.num_pages[b]), int(cache.res_len[b])
    for s in range(n) if slots is None else slots:
        K, V = oracle.dequantize_page(pool[int(cache.page_table[b, s]), h].cpu().numpy(), oc)
        ks.append(K)
        vs.append(V)
    ks.append(cache.res_k[b, h, :r].double().cpu().numpy())
    vs.append(cache.res_v[b, h, :r].double().cpu().numpy())
    return np.concatenate(ks), np.concatenate(vs)


@pytest.mark.parametrize("dtype,gqa,P,k", [(kb.F16, 4, 32, 16), (kb.BF16, 8, 64, 32)])
def test_draft_verify_accept(dtype, gqa, P, k):
    rng = np.random.default_rng(P)
    H, B, T = 2, 3, 13
    cfg = kb.Config(num_q_heads=gqa * H, num_kv_heads=H, page_tokens=P, num_boost=k, dtype=dtype)
    a, ref = (PagedKVCache(cfg, B, max_pages=16, pool_pages=48) for _ in range(2))
    bits = lambda *s: to_dev(syn.to_bits(rng.standard_normal(s).astype(np.float32), dtype), dtype)  # noqa: E731
    for b, L in enumerate((5 * P + 7, P - 3, 3 * P)):
        K, V = bits(L, H, D), bits(L, H, D)
        a.prefill(b, K, V)
        ref.prefill(b, K, V)
    for rnd in range(6):
        # draft: attention over two pages and the window
        q1 = bits(B, gqa * H, D)
        sel, n_sel = a.select(q1, 2, n_first=1, n_recent=1)
        out1 = torch.full((B, gqa * H, D), float("nan"), device="cuda")
        a.attend_few(q1, out1)
        # verify a tree of 13 nodes (ragged), accept a path of it
        drafts = [T, int(rng.integers(1, T + 1)), T]
        q, kd, vd = bits(B, T, gqa * H, D), bits(B, T, H, D), bits(B, T, H, D)
        sees = tree_mask(rng, B, T)
        out = torch.zeros(B, T, gqa * H, D, device="cuda")
        a.verify(q, kd, vd, torch.from_numpy(pack_mask(sees)).cuda(), torch.tensor(drafts, dtype=torch.int32, device="cuda"), out)
        torch.cuda.synchronize()
        assert a.check_errors() == 0
        for b in range(B):
            h, g, i = int(rng.integers(H)), int(rng.integers(gqa)), int(rng.integers(drafts[b]))
            n = min(2, int(a.num_pages[b]))
            assert int(n_sel[b]) == n
            K, V = rows_of(a, b, h, dtype, sel[b, h, :n].tolist())
            want, tol = attend(q1[b, h * gqa + g].double().cpu().numpy(), K, V)
            assert_row(out1[b, h * gqa + g].cpu().numpy(), want, tol, f"round {rnd}: draft of sequence {b}")
            K, V = rows_of(a, b, h, dtype)
            L = len(K)
            K = np.concatenate([K, kd[b, :drafts[b], h].double().cpu().numpy()])
            V = np.concatenate([V, vd[b, :drafts[b], h].double().cpu().numpy()])
            seen = np.concatenate([np.ones(L, bool), sees[b, i, :drafts[b]]])
            want, tol = attend(q[b, i, h * gqa + g].double().cpu().numpy(), K, V, seen)
            assert_row(out[b, i, h * gqa + g].cpu().numpy(), want, tol, f"round {rnd}: node {i} of sequence {b}")
        leaf = [d - 1 for d in drafts]
        path = np.full((B, T), -1)
        n_path = []
        for b in range(B):
            nodes = np.nonzero(sees[b, leaf[b], :drafts[b]])[0][:int(rng.integers(0, T + 1))]
            path[b, :len(nodes)] = nodes
            n_path.append(len(nodes))
        a.accept(kd, vd, torch.as_tensor(path, dtype=torch.int32, device="cuda"), n_path)
        for b in range(B):  # the other cache: one sequence, one token at a time
            for i in range(n_path[b]):
                node = int(path[b, i])
                one = slice(b, b + 1)
                kb.append_token(cfg, kd[one, node].contiguous(), vd[one, node].contiguous(), ref.res_k[one], ref.res_v[one],
                                ref.res_len[one], ref.err)
                ref.host_res_len[b] += 1
                if ref.host_res_len[b] == P:
                    page = ref.take_pages(1)
                    kb.flush_residual(cfg, ref.res_k[one], ref.res_v[one], ref.res_len[one],
                                      torch.tensor(page, dtype=torch.int32, device="cuda"), ref.page_table[one],
                                      ref.num_pages[one], ref.pool, ref.err)
                    ref.host_pages[b] += page
                    ref.host_res_len[b] = 0
        torch.cuda.synchronize()
        assert a.check_errors() == 0 and ref.check_errors() == 0
        assert a.host_res_len == ref.host_res_len == a.res_len.tolist() == ref.res_len.tolist()
        assert torch.equal(a.num_pages, ref.num_pages) and [len(p) for p in a.host_pages] == a.num_pages.tolist()
    pools = [c.pool.view(-1, H, c.record_bytes) for c in (a, ref)]
    payload = kb.page_layout(cfg)["payload_bytes"]
    for b in range(B):
        assert a.page_table[b, :len(a.host_pages[b])].tolist() == a.host_pages[b]
        for x, y in zip(a.host_pages[b], ref.host_pages[b]):
            assert torch.equal(pools[0][x, :, :payload], pools[1][y, :, :payload])
        r = a.host_res_len[b]
        assert torch.equal(a.res_k[b, :, :r], ref.res_k[b, :, :r]) and torch.equal(a.res_v[b, :, :r], ref.res_v[b, :, :r])
    # an ordinary step goes on from there
    out = torch.empty(B, gqa * H, D, device="cuda")
    a.step(bits(B, gqa * H, D), bits(B, H, D), bits(B, H, D), out)
    torch.cuda.synchronize()
    assert a.check_errors() == 0 and torch.isfinite(out).all()


def test_calls_on_a_side_stream():
    cfg = kb.Config(num_q_heads=4, num_kv_heads=1, page_tokens=32, num_boost=16)
    c = PagedKVCache(cfg, 1, max_pages=8, pool_pages=8)
    x = torch.randn(100, 1, D, device="cuda").half()
    c.prefill(0, x, x)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    kd = torch.randn(1, 40, 1, D, device="cuda").half()
    path = torch.arange(40, dtype=torch.int32, device="cuda")[None]
    s.wait_stream(torch.cuda.current_stream())
    c.accept(kd, kd, path, [40], stream=s)
    s.synchronize()
    assert c.check_errors() == 0 and c.res_len.tolist() == [(100 + 40) % 32] and c.num_pages.tolist() == [4]
    assert torch.equal(c.res_k[0, 0, :12], kd[0, 28:40, 0])


def test_captured_steps_replay_after_larger_ones():
    """Select, sparse attention and verification captured once; calls of other sizes in between."""
    cfg = kb.Config(num_q_heads=8, num_kv_heads=2, page_tokens=32, num_boost=16)
    c = PagedKVCache(cfg, 2, max_pages=16, pool_pages=32)
    x = torch.randn(2, 12 * 32, 2, D, device="cuda").half()
    c.prefill_batch(x, x)
    q1 = torch.randn(2, 8, D, device="cuda").half()

    def tree(T):
        q, kd = torch.randn(2, T, 8, D, device="cuda").half(), torch.randn(2, T, 2, D, device="cuda").half()
        mask = torch.from_numpy(pack_mask(tree_mask(np.random.default_rng(T), 2, T))).cuda()
        return dict(q=q, k_draft=kd, v_draft=kd, mask=mask, draft_len=torch.full((2,), T, dtype=torch.int32, device="cuda"),
                    out=torch.zeros(2, T, 8, D, device="cuda"))

    t = tree(6)
    few = torch.zeros(2, 8, D, device="cuda")

    def step():
        c.select(q1, 3)
        c.attend_few(q1, few)
        c.verify(**t)

    step()
    torch.cuda.synchronize()
    want = few.clone(), t["out"].clone(), c.sel.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for T in (128, 1, 2, 40):
        c.select(q1, T % 16 + 1, 0, 1)
        c.attend_few(q1, torch.empty_like(few))
        c.verify(**tree(T))
        few.zero_()
        t["out"].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert c.check_errors() == 0
        assert torch.equal(few, want[0]) and torch.equal(t["out"], want[1]) and torch.equal(c.choices[3][0], want[2])


def test_a_captured_draft_step_keeps_its_choice():
    """A graph of attend_few alone goes on with the choice it was captured with, whatever is chosen after."""
    cfg = kb.Config(num_q_heads=8, num_kv_heads=2, page_tokens=32, num_boost=16)
    c = PagedKVCache(cfg, 2, max_pages=16, pool_pages=32)
    x = torch.randn(2, 12 * 32, 2, D, device="cuda").half()
    c.prefill_batch(x, x)
    q = torch.randn(2, 8, D, device="cuda").half()
    out = torch.zeros(2, 8, D, device="cuda")
    c.select(q, 3)
    c.attend_few(q, out)
    torch.cuda.synchronize()
    want = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.attend_few(q, out)
    c.select(-q, 9)
    c.attend_few(q, torch.empty_like(out))
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert c.check_errors() == 0 and torch.equal(out, want)
