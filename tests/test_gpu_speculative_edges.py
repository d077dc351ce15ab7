"""What a mask hides, values and queries at the ends of their ranges, and inputs that have to raise
a device flag, for the calls of speculative decoding."""
import numpy as np
import pytest
import torch

import oracle
from bit_mixed_precision_channel_b200 import binding as kb
from bit_mixed_precision_channel_b200 import synthetic as syn
from bit_mixed_precision_channel_b200.cache import PagedKVCache

from _kv import to_dev
from _spec import Cache, D, attend
from test_gpu_select import run_select, sparse
from test_gpu_tree import call, check, make

pytestmark = pytest.mark.gpu


def bits(x, dtype):
    return syn.to_bits(np.float32([x]), dtype)[0]


# ---------------------------------------------------------------- hidden and far values


@pytest.mark.parametrize("gqa", [1, 4, 8])
@pytest.mark.parametrize("dtype,value", [(kb.F16, 6e4), (kb.BF16, 1e4), (kb.BF16, 2.0 ** 60), (kb.BF16, 2.0 ** 120),
                                         (kb.BF16, 3.3e38)])
def test_a_token_no_row_sees_may_hold_any_number(dtype, value, gqa):
    """A hidden token of finite, large values is no part of any row, nor of the precision it is carried with."""
    cfg = kb.Config(num_q_heads=gqa, num_kv_heads=1, page_tokens=32, num_boost=16, dtype=dtype)
    sees = np.tril(np.ones((2, 6, 6), bool))
    sees[:, :, 3] = False
    c = make(cfg, [2, 1], [4, 0], 6, [6, 5], seed=2, sees=sees)
    sign = np.where(np.arange(D) % 3 == 0, -1.0, 1.0).astype(np.float32)
    c.k[:, 3] = c.v[:, 3] = syn.to_bits(np.float32(value) * sign, dtype)
    c.t["k_draft"], c.t["v_draft"] = to_dev(c.k, dtype), to_dev(c.v, dtype)
    call(c)
    torch.cuda.synchronize()
    assert c.err.item() == 0
    check(c)


@pytest.mark.parametrize("some", [0, 5])
def test_a_token_one_row_sees_does_not_reach_the_others(some):
    """Row `some` alone sees the token of large values: the others' results are as without it."""
    cfg = kb.Config(num_q_heads=8, num_kv_heads=1, page_tokens=32, num_boost=16, dtype=kb.BF16)
    sees = np.tril(np.ones((1, 6, 6), bool))
    sees[:, :, 3] = False
    sees[:, some, 3] = True
    c = make(cfg, [3], [9], 6, [6], seed=8, sees=sees)
    c.v[:, 3] = bits(2.0 ** 70, kb.BF16)
    c.t["v_draft"] = to_dev(c.v, kb.BF16)
    call(c)
    torch.cuda.synchronize()
    assert c.err.item() == 0
    check(c, rows=[i for i in range(6) if i != some])


def test_a_far_token_of_large_values_leaves_the_near_ones_their_bits():
    """A drafted token every row sees, of weight exp(-28) and values 2^30: 2^-10 of the result.

    Tolerance: a weight off by a factor within 1 +- e moves the mean by at most e sum p |v - o|, with e as in
    _spec.py; sums of products are off by 2^-17 sum p max|v|; a weight times its value scale is carried to 2^-31
    of the largest (a high and a low fp16 part, the largest above 2^6, an absolute step of 2^-25)."""
    cfg = kb.Config(num_q_heads=8, num_kv_heads=1, page_tokens=32, num_boost=16, dtype=kb.BF16)
    c = make(cfg, [0], [20], 4, [4], seed=30, chain=True)
    q0 = syn.from_bits(c.q[0, 0, 0], kb.BF16).astype(np.float64)
    c.q[:] = c.q[0, 0, 0]
    c.k[0, 0] = syn.to_bits((-28.0 * np.sqrt(D) / (q0 @ q0) * q0).astype(np.float32), kb.BF16)
    c.v[0, 0] = bits(2.0 ** 30, kb.BF16)
    c.t.update(q=to_dev(c.q, kb.BF16), k_draft=to_dev(c.k, kb.BF16), v_draft=to_dev(c.v, kb.BF16))
    call(c)
    torch.cuda.synchronize()
    assert c.err.item() == 0
    K, V = c.rows(0, 0)
    for i in range(4):
        Ki = np.concatenate([K, syn.from_bits(c.k[0, :i + 1, 0], kb.BF16).astype(np.float64)])
        Vi = np.concatenate([V, syn.from_bits(c.v[0, :i + 1, 0], kb.BF16).astype(np.float64)])
        z = Ki @ q0 / np.sqrt(D)
        p = np.exp(z - z.max())
        p /= p.sum()
        o, top = p @ Vi, np.abs(Vi).max(1)
        e = 2.0 ** -16 * (np.abs(Ki) @ np.abs(q0)).max() / np.sqrt(D) + 2.0 ** -20
        tol = 2 * e * (p[:, None] * np.abs(Vi - o)).sum(0).max() + 2.0 ** -17 * (p @ top) + 2.0 ** -30 * len(p) * (p * top).max()
        got = c.out[0, i].cpu().numpy()
        assert np.isfinite(got).all() and np.abs(got - o).max() <= tol < 0.01


# ---------------------------------------------------------------- values and keys that are no finite number


@pytest.mark.parametrize("T,gqa", [(2, 4), (6, 1), (3, 4)])
@pytest.mark.parametrize("dtype", [kb.F16, kb.BF16])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_values_that_are_no_number_are_flagged_if_a_row_sees_them(value, dtype, T, gqa):
    cfg = kb.Config(num_q_heads=gqa, num_kv_heads=1, page_tokens=32, num_boost=16, dtype=dtype)
    c = make(cfg, [2], [4], T, [T], seed=3, sees=np.eye(T, dtype=bool)[None])
    c.t["v_draft"][:, 1, :, 9] = value  # a sibling of token 0, which does not see it
    call(c)
    torch.cuda.synchronize()
    assert c.err.item() == kb.DEV_ERR_RANGE


@pytest.mark.parametrize("form", ["tree", "chosen pages"])
@pytest.mark.parametrize("dtype", [kb.F16, kb.BF16])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("pages", [0, 2])
def test_a_window_key_that_is_no_number_is_flagged(pages, value, dtype, form):
    """One token of a short window: the largest logit of its lane is another's, or there is none."""
    cfg = kb.Config(num_q_heads=4, num_kv_heads=1, page_tokens=32, num_boost=16, dtype=dtype)
    c = make(cfg, [pages], [3], 2, [2], seed=6)
    c.d["res_k"][:, :, 1, 40] = value
    if form == "tree":
        call(c)
    else:
        sparse(c, c.q[:, 0], c.ints(np.full((1, 1, 1), 0)), c.ints([min(pages, 1)]))
    torch.cuda.synchronize()
    assert c.err.item() == kb.DEV_ERR_RANGE


# ---------------------------------------------------------------- choices by queries that are no finite number


@pytest.mark.parametrize("pages", [20, 300])
@pytest.mark.parametrize("dtype", [kb.F16, kb.BF16])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_a_choice_by_a_query_that_is_no_number_is_flagged(value, dtype, pages):
    """Keys all above zero in the channel: every page's bound is the same infinity, not NaN."""
    cfg = kb.Config(num_q_heads=2, num_kv_heads=1, page_tokens=32, num_boost=16, dtype=dtype)
    c = Cache(cfg, [pages], [0], seed=5, distinct=12)
    for i in range(len(c.pool)):
        K = syn.from_bits(c.tokens(32), dtype)[:, 0]
        K[:, 7] = 1.0 + np.abs(K[:, 7])
        c.pool[i, 0] = oracle.quantize_page(syn.to_bits(K, dtype), c.values(32)[:, 0], c.oc)
    c.d["pool"] = torch.from_numpy(c.pool.reshape(-1)).cuda()
    q = c.queries(1)
    q[0, 1, 7] = bits(value, dtype)
    sel, n_sel = run_select(c, q, 4, 0, 0)
    torch.cuda.synchronize()
    assert c.err.item() == kb.DEV_ERR_RANGE
    assert n_sel.item() == 4 and (sel >= 0).all() and (sel < pages).all()


# ---------------------------------------------------------------- queries that are no finite number


@pytest.mark.parametrize("T,gqa", [(2, 4), (3, 4)])
@pytest.mark.parametrize("dtype", [kb.F16, kb.BF16])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_queries_that_are_no_number_are_flagged(value, dtype, T, gqa):
    """Without pages, and with keys of one sign: every logit may be minus infinity, which is no number that a
    softmax shows."""
    cfg = kb.Config(num_q_heads=gqa, num_kv_heads=1, page_tokens=32, num_boost=16, dtype=dtype)
    c = make(cfg, [0], [4], T, [T], seed=4)
    c.d["res_k"][:, :, :4, 7] = -1.0 if value > 0 else 1.0
    c.t["k_draft"][..., 7] = -1.0 if value > 0 else 1.0
    c.t["q"][0, 1, gqa - 1, 7] = value
    call(c)
    torch.cuda.synchronize()
    assert c.err.item() == kb.DEV_ERR_RANGE


# ---------------------------------------------------------------- keys at the end of their range


@pytest.mark.parametrize("lo,hi", [(-130560.0, -125000.0), (120000.0, 130560.0), (66000.0, 66000.0), (-130560.0, 300.0)])
def test_bf16_zero_points_up_to_the_documented_range(lo, hi):
    """Keys of a page up to 131008 in magnitude, met by a query that makes ordinary logits of them."""
    cfg = kb.Config(num_q_heads=8, num_kv_heads=1, page_tokens=32, num_boost=16, dtype=kb.BF16)
    c = make(cfg, [3], [4], 4, [4], seed=21)
    c.q[:] = 0
    c.q[..., 7] = bits(1e-4, kb.BF16)
    c.q[..., 8] = bits(0.5, kb.BF16)
    c.t["q"] = to_dev(c.q, kb.BF16)
    for s in range(3):
        K = c.tokens(32)[:, 0]
        K[:, 7] = syn.to_bits(c.rng.uniform(lo, hi, 32).astype(np.float32), kb.BF16)
        K[0, 7] = bits(lo, kb.BF16)
        c.pool[c.table[0, s], 0] = oracle.quantize_page(K, c.values(32)[:, 0], c.oc)
    c.d["pool"] = torch.from_numpy(c.pool.reshape(-1)).cuda()
    call(c)
    torch.cuda.synchronize()
    assert c.err.item() == 0
    check(c)


# ---------------------------------------------------------------- lengths


def test_chosen_pages_of_a_table_of_no_valid_length_are_flagged():
    cfg = kb.Config(num_q_heads=4, num_kv_heads=1, page_tokens=32, num_boost=16)
    c = Cache(cfg, [9, 9], [3, 3], seed=22)
    q = c.queries(2)
    sel = c.ints([[[0, 4, 8]], [[1, 2, 3]]])
    good = sparse(c, q, sel, c.ints([3, 3]))
    assert c.err.item() == 0
    for bad in (c.max_pages + 1, 2 ** 31 - 1, -1):
        c.err.zero_()
        c.d["num_pages"][1] = bad
        out = sparse(c, q, sel, c.ints([3, 3]))
        assert c.err.item() & kb.DEV_ERR_LENGTH
        assert torch.equal(out[0], good[0])


# ---------------------------------------------------------------- small queries


@pytest.mark.parametrize("form", ["many rows", "few rows", "chosen pages"])
def test_small_bf16_queries_on_large_keys(form):
    """Queries of 2^-17 on keys of 4e3 (4e3 times the largest, 14, and the widest channel, 21, are inside the
    documented range): logits from elements that fp16 holds as subnormals.

    Tolerance: that of _spec.py, and an element of the query off by at most 2^-25, which moves a logit by
    2^-25 sm_scale sum |k| and the mean by at most twice that times the distance of the values."""
    T = dict([("many rows", 5), ("few rows", 2), ("chosen pages", 1)])[form]
    cfg = kb.Config(num_q_heads=4, num_kv_heads=1, page_tokens=32, num_boost=16, dtype=kb.BF16)
    c = make(cfg, [5], [7], T, [T], seed=17)

    def grow(x):
        return syn.to_bits(4e3 * syn.from_bits(x, kb.BF16).astype(np.float32), kb.BF16)

    for s in range(5):
        c.pool[c.table[0, s], 0] = oracle.quantize_page(grow(c.tokens(32))[:, 0], c.values(32)[:, 0], c.oc)
    c.res_k[0, :, :7] = grow(c.res_k[0, :, :7])
    c.k = grow(c.k)
    c.q = c.queries(1, T, scale=2.0 ** -17)
    c.d.update(pool=torch.from_numpy(c.pool.reshape(-1)).cuda(), res_k=to_dev(c.res_k, kb.BF16))
    c.t.update(q=to_dev(c.q, kb.BF16), k_draft=to_dev(c.k, kb.BF16))
    if form == "chosen pages":
        out = sparse(c, c.q[:, 0], c.ints([[[0, 2, 3]]]), c.ints([3]))[:, None]
        K, V = c.rows(0, 0, [0, 2, 3])
    else:
        call(c)
        out = c.out
        K, V = c.rows(0, 0)
        K = np.concatenate([K, syn.from_bits(c.k[0, :, 0], kb.BF16).astype(np.float64)])
        V = np.concatenate([V, syn.from_bits(c.v[0, :, 0], kb.BF16).astype(np.float64)])
    torch.cuda.synchronize()
    assert c.err.item() == 0
    out = out.cpu().numpy()
    for i in range(T):
        sees = np.ones(len(K), bool)
        if form != "chosen pages":
            sees[len(K) - T:] = c.sees[0, i]
        for g in range(4):
            want, tol = attend(syn.from_bits(c.q[0, i, g], kb.BF16).astype(np.float64), K, V, sees)
            off = 2.0 ** -25 * np.abs(K).sum(1).max() / np.sqrt(D)
            tol += 2 * off * (V.max() - V.min() + np.abs(V).max())
            assert tol < 0.2 and np.abs(out[0, i, g] - want).max() <= tol


# ---------------------------------------------------------------- one scratch for two layers


@pytest.mark.parametrize("T", [2, 30])
def test_layers_share_the_scratch_of_the_first(T):
    cfg = kb.Config(num_q_heads=8, num_kv_heads=2, page_tokens=32, num_boost=16)
    layers = [PagedKVCache(cfg, 2, max_pages=16, pool_pages=32) for _ in range(2)]
    mask = torch.full((2, T, 1), -1, dtype=torch.int32, device="cuda")
    n = torch.full((2,), T, dtype=torch.int32, device="cuda")
    args, want = [], []
    for c in layers:
        x = torch.randn(2, 9 * 32, 2, D, device="cuda").half()
        c.prefill_batch(x, x)
        args.append([torch.randn(2, T, h, D, device="cuda").half() for h in (8, 2, 2)])
        want.append(torch.zeros(2, T, 8, D, device="cuda"))
        c.verify(*args[-1], mask, n, want[-1])
    layers[1].tree_workspace = layers[0].tree_workspace
    for _ in range(2):
        for c, a, w in zip(layers, args, want):
            out = torch.zeros_like(w)
            c.verify(*a, mask, n, out)
            torch.cuda.synchronize()
            assert c.check_errors() == 0 and torch.equal(out, w)
