"""Choice of pages and attention over the chosen ones: the choice equals a plain 64-bit ranking,
attention over it is within the derived tolerance of a 64-bit computation."""
import numpy as np
import pytest
import torch

import oracle
from bit_mixed_precision_channel_b200 import binding as kb
from bit_mixed_precision_channel_b200 import synthetic as syn

from _kv import to_dev
from _spec import Cache, D, assert_row, attend

pytestmark = pytest.mark.gpu


def bound(rec, q, oc):
    """Largest bound over the record's groups, from the record's sections (64 bits)."""
    L = oracle.layout(oc.P, oc.D, oc.k, oc.G)

    def part(name, n):
        return oracle.values(np.ascontiguousarray(rec[L[name]:L[name] + 2 * n]).view(np.uint16), oc.dtype).astype(np.float64)

    ng = oc.P // oc.G
    at = np.array([oracle.key_meta_pos(c) for c in range(D)])
    s, z = (part(n, ng * D).reshape(ng, D)[:, at] for n in ("k_scale", "k_zero"))
    hi = z + 3 * s
    if oc.k:
        idx = rec[L["boost_idx"]:L["boost_idx"] + oc.k].astype(int)
        sb = part("kb_scale", ng * oc.k).reshape(ng, oc.k)
        for j, c in enumerate(idx):
            hi[:, c] += 3 * sb[:, j]
    pos, neg = np.maximum(q, 0).sum(0), np.minimum(q, 0).sum(0)
    return (hi @ pos + z @ neg).max()


def choose(c, q, n_select, n_first, n_recent):
    """The choice of every (sequence, kv head), and the sequences' counts."""
    cfg = c.cfg
    sel = np.full((c.B, cfg.num_kv_heads, n_select), -1, np.int32)
    n_sel = np.minimum(c.pages, n_select)
    for b in range(c.B):
        n = c.pages[b]
        for h in range(cfg.num_kv_heads):
            qh = syn.from_bits(q[b, h * cfg.gqa:(h + 1) * cfg.gqa], cfg.dtype).astype(np.float64)
            memo = {}
            score = np.array([memo[p] if p in memo else memo.setdefault(p, bound(c.pool[p, h], qh, c.oc)) for p in c.table[b, :n]])
            for i in range(n):
                if i < n_first or i >= n - n_recent:
                    score[i] = np.inf
            best = np.sort(np.argsort(-score, kind="stable")[:n_select])
            sel[b, h, :len(best)] = best
    return sel, n_sel


def run_select(c, q, n_select, n_first, n_recent):
    sel = torch.full((c.B, c.cfg.num_kv_heads, n_select), 123, dtype=torch.int32, device="cuda")
    n_sel = torch.full((c.B,), 123, dtype=torch.int32, device="cuda")
    kb.select_pages(c.cfg, c.d["pool"], to_dev(q, c.cfg.dtype), c.d["page_table"], c.d["num_pages"], sel, n_sel,
                    n_first=n_first, n_recent=n_recent, err=c.err)
    return sel, n_sel


CASES = [
    # dtype, H, gqa, P, k, pages, select, first, recent, distinct
    (kb.F16, 2, 4, 128, 32, [40, 3, 0], 8, 1, 1, None),
    (kb.BF16, 2, 8, 64, 64, [30, 31, 8], 8, 0, 0, None),
    (kb.F16, 1, 1, 32, 16, [60], 1, 0, 0, None),
    (kb.F16, 1, 2, 32, 0, [25, 26], 25, 3, 4, None),
    (kb.BF16, 1, 4, 128, 128, [12], 5, 5, 0, None),     # nothing left to rank
    (kb.F16, 1, 4, 64, 16, [256, 257, 255], 64, 1, 2, 30),   # repeated pages: ties to the lower slot; both ways to select
    (kb.F16, 2, 4, 32, 16, [2000], 333, 0, 5, 500),
    (kb.BF16, 1, 1, 32, 32, [1025], 1024, 0, 0, 40),
    (kb.F16, 1, 1, 32, 16, [700], 10, 0, 0, 1),         # three different pages in all
]


@pytest.mark.parametrize("dtype,H,gqa,P,k,pages,select,first,recent,distinct", CASES)
def test_choice_equals_the_64_bit_ranking(dtype, H, gqa, P, k, pages, select, first, recent, distinct):
    cfg = kb.Config(num_q_heads=gqa * H, num_kv_heads=H, page_tokens=P, num_boost=k, dtype=dtype)
    c = Cache(cfg, pages, [0] * len(pages), seed=P + k + select, distinct=distinct)
    q = c.queries(c.B)
    sel, n_sel = run_select(c, q, select, first, recent)
    torch.cuda.synchronize()
    assert c.err.item() == 0
    want, counts = choose(c, q, select, first, recent)
    np.testing.assert_array_equal(n_sel.cpu().numpy(), counts)
    np.testing.assert_array_equal(sel.cpu().numpy(), want)


@pytest.mark.parametrize("k,boosts", [(128, [0, 100]), (16, [3, 16])])
def test_choice_among_heads_with_fewer_boosted_channels(k, boosts):
    cfg = kb.Config(num_q_heads=4, num_kv_heads=2, page_tokens=64, num_boost=k)
    c = Cache(cfg, [50, 7], [0, 0], seed=k, boosts=boosts)
    q = c.queries(2)
    sel, n_sel = run_select(c, q, 9, 0, 1)
    torch.cuda.synchronize()
    assert c.err.item() == 0
    want, counts = choose(c, q, 9, 0, 1)
    np.testing.assert_array_equal(n_sel.cpu().numpy(), counts)
    np.testing.assert_array_equal(sel.cpu().numpy(), want)


@pytest.mark.parametrize("B", [160, 330, 650])
def test_choice_with_more_sequences_than_clusters_of_eight(B):
    """Many sequences: fewer blocks share a sequence's pages, down to one; both ways to select."""
    cfg = kb.Config(num_q_heads=2, num_kv_heads=1, page_tokens=32, num_boost=16)
    rng = np.random.default_rng(B)
    c = Cache(cfg, rng.choice([0, 3, 7, 40, 255, 256, 257, 300], B).tolist(), [0] * B, seed=B, distinct=25)
    q = c.queries(B)
    sel, n_sel = run_select(c, q, 6, 1, 1)
    torch.cuda.synchronize()
    assert c.err.item() == 0
    want, counts = choose(c, q, 6, 1, 1)
    np.testing.assert_array_equal(n_sel.cpu().numpy(), counts)
    np.testing.assert_array_equal(sel.cpu().numpy(), want)


@pytest.mark.parametrize("n", [200, 5000, 204800])
def test_the_largest_page_table(n):
    """A table as long as the call allows, with few pages in it and with all."""
    cfg = kb.Config(num_q_heads=1, num_kv_heads=1, page_tokens=32, num_boost=0)
    c = Cache(cfg, [n, 12], [0, 0], seed=n, distinct=30)
    table = np.full((2, 204800), -1, np.int32)
    table[:, :min(c.max_pages, 204800)] = c.table[:, :204800]
    c.d["page_table"] = c.ints(table)
    q = c.queries(2)
    sel, n_sel = run_select(c, q, 50, 2, 3)
    torch.cuda.synchronize()
    assert c.err.item() == 0
    want, counts = choose(c, q, 50, 2, 3)
    np.testing.assert_array_equal(n_sel.cpu().numpy(), counts)
    np.testing.assert_array_equal(sel.cpu().numpy(), want)


def test_zero_query_ties_everywhere():
    """Every score is zero, of either sign: the lowest slots are chosen."""
    cfg = kb.Config(num_q_heads=2, num_kv_heads=1, page_tokens=32, num_boost=16)
    for n in (100, 900):
        c = Cache(cfg, [n], [0], seed=n, distinct=20)
        q = np.zeros((1, 2, D), np.uint16)
        q[0, 1] = 0x8000  # minus zero
        sel, _ = run_select(c, q, 7, 0, 0)
        assert sel.cpu().numpy().tolist() == [[list(range(7))]]


def test_a_bound_is_never_below_a_logit_sum():
    """What the score promises: no stored token gives the heads a larger sum of logits."""
    cfg = kb.Config(num_q_heads=4, num_kv_heads=1, page_tokens=64, num_boost=32)
    c = Cache(cfg, [6], [0], seed=77)
    q = syn.from_bits(c.queries(1)[0], cfg.dtype).astype(np.float64)
    for p in range(len(c.pool)):
        K, _ = oracle.dequantize_page(c.pool[p, 0], c.oc)
        assert (K @ q.sum(0)).max() <= bound(c.pool[p, 0], q, c.oc) * (1 + 1e-12)


def test_select_flags_bad_lengths_pages_and_queries():
    cfg = kb.Config(num_q_heads=4, num_kv_heads=2, page_tokens=32, num_boost=16)
    c = Cache(cfg, [20, 20, 20], [0] * 3, seed=5)
    q = c.queries(3)
    for bad in (-1, 10 ** 6):
        c.err.zero_()
        c.d["num_pages"][1] = bad
        sel, n_sel = run_select(c, q, 4, 0, 1)
        assert c.err.item() == kb.DEV_ERR_LENGTH and n_sel.tolist() == [4, 0, 4] and (sel[1] == -1).all()
    c.d["num_pages"][1] = 20
    want, _ = choose(c, q, 4, 0, 1)
    c.err.zero_()
    c.d["page_table"][2, 5] = len(c.pool)
    sel, _ = run_select(c, q, 4, 0, 1)
    assert c.err.item() == kb.DEV_ERR_PAGE_RANGE
    np.testing.assert_array_equal(sel[:2].cpu().numpy(), want[:2])
    c.d["page_table"][2, 5] = 0
    c.err.zero_()
    q[0, 1, 3] = 0x7e00
    sel, _ = run_select(c, q, 4, 0, 1)
    assert c.err.item() == kb.DEV_ERR_RANGE
    assert (sel >= 0).all() and (sel < 20).all()


def sparse(c, q, sel, n_sel, out=None, ws=None):
    cfg, d = c.cfg, c.d
    if ws is None:
        ws = torch.zeros(kb.decode_workspace_bytes(cfg, c.B, c.max_pages), dtype=torch.uint8, device="cuda")
    if out is None:
        out = torch.full((c.B, cfg.num_q_heads, D), float("nan"), device="cuda")
    kb.decode_attention_sparse(cfg, d["pool"], to_dev(q, cfg.dtype), d["page_table"], d["num_pages"], sel, n_sel,
                               d["res_k"], d["res_v"], d["res_len"], out, ws, err=c.err)
    return out


@pytest.mark.parametrize("dtype,H,gqa,P,k,pages,window,n", [
    (kb.F16, 2, 4, 128, 32, [20, 3, 0, 9], [50, 0, 0, 127], 7),
    (kb.BF16, 2, 8, 64, 64, [30, 1], [63, 64], 9),
    (kb.F16, 1, 1, 32, 16, [41], [1], 41),
    (kb.F16, 2, 2, 32, 0, [17, 40], [0, 0], 5),
    (kb.BF16, 1, 4, 32, 128, [6], [20], 1),
])
def test_sparse_attention_matches_64_bits(dtype, H, gqa, P, k, pages, window, n):
    """Random choices, a different one for each kv head, in any order; one head's list holds a slot twice."""
    cfg = kb.Config(num_q_heads=gqa * H, num_kv_heads=H, page_tokens=P, num_boost=k, dtype=dtype)
    c = Cache(cfg, pages, window, seed=P + k + n)
    q = c.queries(c.B)
    sel = np.full((c.B, H, n), -1, np.int32)
    counts = [min(n, p) for p in pages]
    for b in range(c.B):
        for h in range(H):
            sel[b, h, :counts[b]] = c.rng.permutation(pages[b])[:counts[b]]
    if counts[0] > 1:
        sel[0, 0, 1] = sel[0, 0, 0]
    out = sparse(c, q, c.ints(sel), c.ints(counts))
    torch.cuda.synchronize()
    assert c.err.item() == 0
    got = out.cpu().numpy()
    for b in range(c.B):
        for h in range(H):
            K, V = c.rows(b, h, sel[b, h, :counts[b]])
            for g in range(gqa):
                want, tol = attend(syn.from_bits(q[b, h * gqa + g], dtype).astype(np.float64), K, V)
                assert_row(got[b, h * gqa + g], want, tol, f"sequence {b}, head {h * gqa + g}")


def test_every_page_chosen_gives_what_the_dense_call_gives():
    cfg = kb.Config(num_q_heads=8, num_kv_heads=2, page_tokens=64, num_boost=16)
    c = Cache(cfg, [25, 4], [30, 0], seed=21)
    q = c.queries(2)
    sel, n_sel = run_select(c, q, 25, 0, 0)
    out = sparse(c, q, sel, n_sel)
    ws = torch.zeros(kb.decode_workspace_bytes(cfg, 2, c.max_pages), dtype=torch.uint8, device="cuda")
    want = torch.empty_like(out)
    d = c.d
    kb.decode_attention(cfg, d["pool"], to_dev(q, cfg.dtype), d["page_table"], d["num_pages"], d["res_k"], d["res_v"],
                        d["res_len"], want, ws, err=c.err)
    torch.cuda.synchronize()
    assert c.err.item() == 0
    out, want = out.cpu().numpy(), want.cpu().numpy()
    for b in range(2):
        for hq in range(8):
            K, V = c.rows(b, hq // 4)
            exact, tol = attend(syn.from_bits(q[b, hq], cfg.dtype).astype(np.float64), K, V)
            for got in (out, want):
                assert_row(got[b, hq], exact, tol, f"sequence {b}, head {hq}")


def test_sparse_flags_bad_slots_and_counts():
    cfg = kb.Config(num_q_heads=4, num_kv_heads=1, page_tokens=32, num_boost=16)
    c = Cache(cfg, [9, 9], [3, 3], seed=22)
    q = c.queries(2)
    sel = c.ints([[[0, 4, 8]], [[1, 2, 3]]])
    good = sparse(c, q, sel, c.ints([3, 3]))
    for slot in (9, -1, 2 ** 31 - 1):
        c.err.zero_()
        bad = sel.clone()
        bad[1, 0, 1] = slot
        out = sparse(c, q, bad, c.ints([3, 3]))
        assert c.err.item() == kb.DEV_ERR_PAGE_RANGE
        assert torch.equal(out[0], good[0])
    for count in (4, -1):
        c.err.zero_()
        sparse(c, q, sel, c.ints([3, count]))
        assert c.err.item() == kb.DEV_ERR_LENGTH
