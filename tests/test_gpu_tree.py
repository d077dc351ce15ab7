"""Attention of drafted trees over the 2-bit cache against a plain 64-bit computation, within
the tolerance _spec.py derives: head groupings, page sizes, boost counts, tree sizes from one
token to the largest, ragged lengths, masks that leave rows empty, and what must not be read
or written."""
import numpy as np
import pytest
import torch

from bit_mixed_precision_channel_b200 import binding as kb
from bit_mixed_precision_channel_b200 import synthetic as syn

from _kv import to_dev
from _spec import Cache, D, assert_row, attend, pack_mask, tree_mask

pytestmark = pytest.mark.gpu


def make(cfg, pages, window, T, drafts, seed, sees=None, chain=False, **more):
    c = Cache(cfg, pages, window, seed, **more)
    B, H = c.B, cfg.num_kv_heads
    c.T, c.drafts = T, list(drafts)
    c.k = np.stack([c.tokens(T) for _ in range(B)])
    c.v = np.stack([c.values(T) for _ in range(B)])
    c.q = c.queries(B, T)
    for b, n in enumerate(drafts):  # behind the drafted tokens: nothing that may be used
        c.k[b, n:] = 0x7fff
        c.v[b, n:] = 0x7fff
        c.q[b, n:] = 0x7fff
    c.sees = tree_mask(c.rng, B, T, chain) if sees is None else sees
    dt = cfg.dtype
    c.t = dict(q=to_dev(c.q, dt), k_draft=to_dev(c.k, dt), v_draft=to_dev(c.v, dt),
               mask=torch.from_numpy(pack_mask(c.sees)).cuda(), draft_len=c.ints(drafts))
    c.ws = torch.zeros(kb.tree_workspace_bytes(cfg, B, T), dtype=torch.uint8, device="cuda")
    c.ws[65536:] = 0xff  # behind the counters nothing has to be prepared
    c.out = torch.full((B, T, cfg.num_q_heads, D), 7.5, device="cuda")
    return c


def call(c, **over):
    d = c.d
    a = dict(pool=d["pool"], page_table=d["page_table"], num_pages=d["num_pages"], res_k=d["res_k"], res_v=d["res_v"],
             res_len=d["res_len"], out=c.out, workspace=c.ws, err=c.err, **c.t)
    a.update(over)
    kb.tree_attention(c.cfg, **a)


def check(c, out=None, rows=None, sm_scale=None):
    assert not c.ws[:65536].any(), "counters left behind"
    out = (c.out if out is None else out).cpu().numpy()
    cfg = c.cfg
    more = {} if sm_scale is None else dict(sm_scale=sm_scale)
    for b in range(c.B):
        n = c.drafts[b]
        assert (out[b, n:] == 7.5).all(), f"sequence {b}: rows behind its drafted tokens were written"
        for h in range(cfg.num_kv_heads):
            K, V = c.rows(b, h)
            L = len(K)
            K = np.concatenate([K, syn.from_bits(c.k[b, :n, h], cfg.dtype).astype(np.float64)])
            V = np.concatenate([V, syn.from_bits(c.v[b, :n, h], cfg.dtype).astype(np.float64)])
            for i in range(n) if rows is None else [i for i in rows if i < n]:
                sees = np.concatenate([np.ones(L, bool), c.sees[b, i, :n]])
                for g in range(cfg.gqa):
                    hq = h * cfg.gqa + g
                    q = syn.from_bits(c.q[b, i, hq], cfg.dtype).astype(np.float64)
                    want, tol = attend(q, K, V, sees, **more)
                    assert_row(out[b, i, hq], want, tol, f"sequence {b}, token {i}, head {hq}")


@pytest.mark.parametrize("dtype,H,gqa,P,k,T,pages,window,drafts", [
    (kb.F16, 2, 4, 128, 32, 16, [9, 3], [77, 0], [16, 11]),
    (kb.F16, 1, 1, 32, 16, 1, [8], [31], [1]),              # one head, one token
    (kb.F16, 2, 4, 128, 32, 1, [33, 0, 1, 5], [5, 0, 128, 64], [1, 1, 1, 1]),  # single-token step, a full window, no cache
    (kb.BF16, 2, 8, 64, 64, 33, [7, 1], [63, 1], [33, 32]),  # a mask of two words, more rows than a tile
    (kb.BF16, 1, 8, 128, 32, 128, [5, 2], [100, 3], [128, 65]),  # the largest tree
    (kb.F16, 2, 2, 64, 0, 7, [10, 0], [0, 40], [7, 3]),      # no boosted channels, odd tree
    (kb.F16, 1, 4, 32, 128, 9, [13, 2, 6], [0, 32, 17], [9, 0, 1]),  # every channel boosted; no drafted token at all
    (kb.BF16, 1, 1, 32, 0, 40, [1, 4], [0, 9], [40, 39]),
    (kb.BF16, 1, 2, 128, 128, 5, [3], [16], [5]),
    (kb.F16, 1, 8, 64, 16, 20, [0], [0], [20]),              # nothing but the drafted tokens
    # at most 8 rows of a kv head
    (kb.F16, 2, 4, 128, 32, 2, [9, 0, 40], [127, 128, 3], [2, 1, 2]),
    (kb.BF16, 2, 2, 64, 64, 4, [7, 1, 0], [64, 15, 0], [4, 3, 0]),
    (kb.F16, 1, 1, 32, 0, 8, [50, 2, 0], [31, 8, 0], [8, 5, 7]),
    (kb.BF16, 2, 8, 128, 16, 1, [33, 1, 0], [126, 0, 1], [1, 1, 0]),
    (kb.BF16, 1, 1, 32, 128, 3, [12], [32], [3]),
    (kb.F16, 3, 2, 64, 32, 3, [5, 6], [61, 62], [3, 2]),
    (kb.F16, 1, 1, 128, 32, 9, [3], [40], [9]),              # one row more
])
def test_matches_64_bits(dtype, H, gqa, P, k, T, pages, window, drafts):
    cfg = kb.Config(num_q_heads=gqa * H, num_kv_heads=H, page_tokens=P, num_boost=k, dtype=dtype)
    c = make(cfg, pages, window, T, drafts, seed=T + P + k)
    call(c)
    torch.cuda.synchronize()
    assert c.err.item() == 0
    check(c)


@pytest.mark.parametrize("T,gqa", [(9, 4), (2, 4)])
@pytest.mark.parametrize("dtype,P,k,boosts", [
    (kb.F16, 32, 128, [0, 5, 100, 128]),
    (kb.BF16, 128, 128, [127, 1, 64, 0]),
    (kb.F16, 64, 64, [63, 0, 64, 17]),
    (kb.BF16, 32, 16, [0, 1, 15, 16]),
])
def test_heads_with_fewer_boosted_channels(dtype, P, k, boosts, T, gqa):
    """Records with rows for more boosted channels than the head has: the rows in use name any channel."""
    cfg = kb.Config(num_q_heads=4 * gqa, num_kv_heads=4, page_tokens=P, num_boost=k, dtype=dtype)
    c = make(cfg, [11, 2], [9, 0], T, [T, T], seed=k + P, boosts=boosts)
    call(c)
    torch.cuda.synchronize()
    assert c.err.item() == 0
    check(c)


def test_long_sequences_beside_short_ones_are_split():
    cfg = kb.Config(num_q_heads=4, num_kv_heads=1, page_tokens=128, num_boost=32)
    c = make(cfg, [120, 0, 1, 64], [1, 3, 0, 127], 24, [24, 24, 5, 1], seed=3, distinct=12)
    call(c)
    torch.cuda.synchronize()
    assert c.err.item() == 0
    check(c, rows=[0, 4, 23])


def test_many_sequences():
    cfg = kb.Config(num_q_heads=2, num_kv_heads=1, page_tokens=32, num_boost=16)
    B = 300
    rng = np.random.default_rng(8)
    pages, window, drafts = rng.integers(0, 6, B), rng.integers(0, 33, B), rng.integers(0, 4, B)
    c = make(cfg, pages.tolist(), window.tolist(), 3, drafts.tolist(), seed=5, distinct=20)
    call(c)
    torch.cuda.synchronize()
    assert c.err.item() == 0
    check(c)


def test_more_sequences_than_threads():
    cfg = kb.Config(num_q_heads=1, num_kv_heads=1, page_tokens=32, num_boost=16)
    B = 2000
    rng = np.random.default_rng(9)
    pages, window, drafts = rng.integers(0, 4, B), rng.integers(0, 33, B), rng.integers(0, 10, B)
    pages[1100:1900] = window[1100:1900] = drafts[1100:1900] = 0
    c = make(cfg, pages.tolist(), window.tolist(), 9, drafts.tolist(), seed=5, distinct=20, chain=True)
    call(c)
    torch.cuda.synchronize()
    assert c.err.item() == 0
    check(c, rows=[0, 8])


@pytest.mark.parametrize("gqa", [1, 4])
def test_rows_whose_mask_leaves_nothing(gqa):
    """Without a cache, a token whose mask is empty has nothing to attend to: zero.  With one, it
    attends to the cache alone.  Bits at or behind draft_len name no token."""
    cfg = kb.Config(num_q_heads=gqa, num_kv_heads=1, page_tokens=32, num_boost=16)
    sees = np.zeros((2, 8, 8), bool)
    sees[:, 2, 1] = sees[:, 4, 4] = True
    sees[:, 5, 7] = True  # behind draft_len
    c = make(cfg, [0, 3], [0, 5], 8, [6, 6], seed=1, sees=sees)
    call(c)
    torch.cuda.synchronize()
    assert c.err.item() == 0
    check(c)
    assert (c.out[0, [0, 1, 3, 5]] == 0).all()


@pytest.mark.parametrize("dtype", [kb.F16, kb.BF16])
@pytest.mark.parametrize("gqa", [1, 4])
def test_a_token_no_row_sees_may_hold_anything(dtype, gqa):
    cfg = kb.Config(num_q_heads=gqa, num_kv_heads=1, page_tokens=32, num_boost=16, dtype=dtype)
    sees = np.tril(np.ones((1, 6, 6), bool))
    sees[:, :, 3] = False
    c = make(cfg, [2], [4], 6, [6], seed=2, sees=sees)
    for x in (c.t["k_draft"], c.t["v_draft"]):
        x[:, 3] = float("nan")
        x[:, 3, :, ::5] = float("inf")
    c.k[:, 3] = c.v[:, 3] = 0  # of no weight in the 64-bit result
    call(c)
    torch.cuda.synchronize()
    assert c.err.item() == 0
    check(c)


@pytest.mark.parametrize("gqa", [1, 4])
def test_large_values_and_queries(gqa):
    """Values of magnitude 3e3 and queries of 200: the softmax turns into the largest logit's value."""
    cfg = kb.Config(num_q_heads=gqa, num_kv_heads=1, page_tokens=32, num_boost=16)
    c = make(cfg, [4], [9], 4, [4], seed=4)
    c.q = c.queries(1, 4, scale=200.0)
    c.v = syn.to_bits(3e3 * c.rng.standard_normal((1, 4, 1, D)).astype(np.float32), cfg.dtype)
    c.res_v[0, :, :9] = syn.to_bits(3e3 * c.rng.standard_normal((1, 9, D)).astype(np.float32), cfg.dtype)
    c.t["q"], c.t["v_draft"] = to_dev(c.q, cfg.dtype), to_dev(c.v, cfg.dtype)
    c.d["res_v"] = to_dev(c.res_v, cfg.dtype)
    call(c)
    torch.cuda.synchronize()
    assert c.err.item() == 0
    check(c)


@pytest.mark.parametrize("dtype", [kb.F16, kb.BF16])
def test_pages_of_wide_value_ranges(dtype):
    """Pages whose value scales differ by a factor of a thousand, in both orders."""
    cfg = kb.Config(num_q_heads=8, num_kv_heads=1, page_tokens=64, num_boost=16, dtype=dtype)
    c = make(cfg, [4, 4], [3, 3], 3, [3, 3], seed=6)
    import oracle
    for b, order in ((0, (1.0, 1e3, 1e3, 1e-2)), (1, (1e3, 1e-2, 1.0, 1.0))):
        for s, f in enumerate(order):
            V = syn.to_bits((f * c.rng.standard_normal((64, D))).astype(np.float32), dtype)
            K = c.tokens(64)[:, 0]
            c.pool[c.table[b, s], 0] = oracle.quantize_page(K, V, c.oc)
    c.d["pool"] = torch.from_numpy(c.pool.reshape(-1)).cuda()
    call(c)
    torch.cuda.synchronize()
    assert c.err.item() == 0
    check(c)


@pytest.mark.parametrize("where", ["window", "drafted", "page", "nowhere"])
@pytest.mark.parametrize("dtype", [kb.F16, kb.BF16])
def test_keys_beyond_the_range_are_flagged_whatever_the_query(where, dtype):
    """A key no operand holds meets a query so small that its logit is ordinary: never a quiet weight of zero."""
    cfg = kb.Config(num_q_heads=8, num_kv_heads=1, page_tokens=32, num_boost=16, dtype=dtype)
    big = -2e5 if dtype == kb.BF16 else -6e4  # fp16: the largest keys are in range
    c = make(cfg, [2], [4], 4, [4], seed=21)
    import oracle
    c.q[:] = 0
    c.q[..., 7] = syn.to_bits(np.float32([1e-4]), dtype)[0]
    c.t["q"] = to_dev(c.q, dtype)
    one = syn.to_bits(np.float32([big]), dtype)[0]
    if where == "window":
        c.res_k[0, :, 2, 7] = one
        c.d["res_k"] = to_dev(c.res_k, dtype)
    elif where == "drafted":
        c.k[0, 0, :, 7] = one
        c.t["k_draft"] = to_dev(c.k, dtype)
    elif where == "page":
        K = c.tokens(32)[:, 0]
        K[:, 7] = one
        c.pool[c.table[0, 1], 0] = oracle.quantize_page(K, c.values(32)[:, 0], c.oc)
        c.d["pool"] = torch.from_numpy(c.pool.reshape(-1)).cuda()
    call(c)
    torch.cuda.synchronize()
    if dtype == kb.BF16 and where != "nowhere":
        assert c.err.item() == kb.DEV_ERR_RANGE
    else:
        assert c.err.item() == 0
        check(c)


@pytest.mark.parametrize("T", [2, 5])
def test_negative_and_zero_scale(T):
    cfg = kb.Config(num_q_heads=8, num_kv_heads=2, page_tokens=32, num_boost=16)
    for sm in (-0.05, 0.0, 1.0):
        c = make(cfg, [3], [7], T, [T], seed=9)
        call(c, sm_scale=sm)
        torch.cuda.synchronize()
        assert c.err.item() == 0
        check(c, sm_scale=sm)


def test_one_token_equals_the_step_after_its_append():
    """The single-token form against the decode call with the token already in the window."""
    cfg = kb.Config(num_q_heads=8, num_kv_heads=2, page_tokens=64, num_boost=32)
    c = make(cfg, [6, 1], [20, 0], 1, [1, 1], seed=12, garbage=False)
    call(c)
    d = c.d
    kb.append_token(cfg, c.t["k_draft"], c.t["v_draft"], d["res_k"], d["res_v"], d["res_len"], c.err)
    ws = torch.zeros(kb.decode_workspace_bytes(cfg, 2, c.max_pages), dtype=torch.uint8, device="cuda")
    out = torch.empty(2, 8, D, device="cuda")
    kb.decode_attention(cfg, d["pool"], c.t["q"], d["page_table"], d["num_pages"], d["res_k"], d["res_v"], d["res_len"],
                        out, ws, err=c.err)
    torch.cuda.synchronize()
    assert c.err.item() == 0
    # both are within the derived tolerance of the same 64-bit result; their difference is within its double
    check(c)
    assert (out - c.out[:, 0]).abs().max() <= 4e-3


@pytest.mark.parametrize("gqa", [1, 4])
def test_device_errors_are_flagged_and_leave_other_sequences_right(gqa):
    cfg = kb.Config(num_q_heads=gqa, num_kv_heads=1, page_tokens=32, num_boost=16)
    for name, value, flag in (("num_pages", 99, kb.DEV_ERR_LENGTH), ("num_pages", -1, kb.DEV_ERR_LENGTH),
                              ("res_len", 33, kb.DEV_ERR_LENGTH), ("res_len", -2, kb.DEV_ERR_LENGTH),
                              ("draft_len", 6, kb.DEV_ERR_LENGTH), ("draft_len", -1, kb.DEV_ERR_LENGTH),
                              ("page_table", 10 ** 6, kb.DEV_ERR_PAGE_RANGE), ("page_table", -7, kb.DEV_ERR_PAGE_RANGE)):
        c = make(cfg, [3, 2, 4], [4, 0, 9], 5, [5, 4, 3], seed=13)
        t = c.t[name] if name in c.t else c.d[name]
        t[(1, 0) if name == "page_table" else 1] = value
        call(c)
        torch.cuda.synchronize()
        assert c.err.item() == flag, name
        if name != "page_table":
            assert (c.out[1] == 7.5).all()  # the sequence is left out
        else:
            c.out[1, :4] = 0  # undefined
        keep = c.B, c.drafts
        got = c.out[[0, 2]]
        for i, b in enumerate((0, 2)):
            K, V = c.rows(b, 0)
            n = c.drafts[b]
            K = np.concatenate([K, syn.from_bits(c.k[b, :n, 0], cfg.dtype).astype(np.float64)])
            V = np.concatenate([V, syn.from_bits(c.v[b, :n, 0], cfg.dtype).astype(np.float64)])
            sees = np.concatenate([np.ones(len(K) - n, bool), c.sees[b, n - 1, :n]])
            want, tol = attend(syn.from_bits(c.q[b, n - 1, gqa - 1], cfg.dtype).astype(np.float64), K, V, sees)
            assert_row(got[i, n - 1, gqa - 1].cpu().numpy(), want, tol, f"{name}: sequence {b}")
        assert keep == (c.B, c.drafts)


@pytest.mark.parametrize("T,drafts", [(12, [12, 7]), (2, [2, 1])])
def test_same_bits_again_on_another_stream_and_replayed(T, drafts):
    """Nothing depends on the order of atomics, on the stream, or on what the workspace held."""
    cfg = kb.Config(num_q_heads=8, num_kv_heads=2, page_tokens=128, num_boost=32)
    c = make(cfg, [40, 3], [17, 90], T, drafts, seed=14, distinct=9)
    call(c)
    torch.cuda.synchronize()
    first = c.out.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = torch.full_like(c.out, 7.5)
    with torch.cuda.stream(s):
        c.ws[65536:] = 0x5a
        call(c, out=other)
    s.synchronize()
    assert torch.equal(first, other)
    g = torch.cuda.CUDAGraph()
    replayed = torch.full_like(c.out, 7.5)
    with torch.cuda.graph(g):
        call(c, out=replayed)
    for _ in range(3):
        replayed.fill_(7.5)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, replayed)
    # lengths are read at replay: a captured step goes on as the cache grows
    c.d["num_pages"].copy_(c.ints([39, 2]))
    c.pages = [39, 2]
    replayed.fill_(7.5)
    g.replay()
    torch.cuda.synchronize()
    assert c.err.item() == 0
    check(c, out=replayed, rows=[0, 6, 11])


def test_two_calls_at_once_with_a_workspace_each():
    cfg = kb.Config(num_q_heads=8, num_kv_heads=2, page_tokens=64, num_boost=16)
    c = make(cfg, [30, 12], [17, 40], 9, [9, 9], seed=15, distinct=9)
    call(c)
    torch.cuda.synchronize()
    outs, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            ws = torch.zeros_like(c.ws)
            for _ in range(4):
                out = torch.full_like(c.out, 7.5)
                call(c, out=out, workspace=ws)
                outs.append((out, ws))
    torch.cuda.synchronize()
    assert all(torch.equal(o, c.out) for o, _ in outs)


def test_shapes_take_turns_in_one_workspace():
    """Few rows (counters) and many (cut units), small and large batches, on the same scratch."""
    cs = []
    for B, gqa, T in ((2, 4, 2), (2, 4, 20), (40, 1, 3), (1, 8, 1), (3, 8, 60)):
        cfg = kb.Config(num_q_heads=2 * gqa, num_kv_heads=2, page_tokens=64, num_boost=16)
        cs.append(make(cfg, [(7 * b) % 30 for b in range(B)], [(5 * b) % 64 for b in range(B)], T, [T] * B, seed=B + T, distinct=12))
    ws = torch.zeros(max(c.ws.numel() for c in cs), dtype=torch.uint8, device="cuda")
    for _ in range(2):
        for c in cs:
            c.ws = ws
            c.out.fill_(7.5)
            call(c)
    torch.cuda.synchronize()
    for c in cs:
        assert c.err.item() == 0
        check(c, rows=[0])


def test_more_units_than_counters():
    """A batch whose arrival counters do not fit their place at the workspace's start."""
    cfg = kb.Config(num_q_heads=8, num_kv_heads=8, page_tokens=32, num_boost=0)
    B = 2100
    c = make(cfg, [2 if b % 700 == 0 else 0 for b in range(B)], [b % 3 for b in range(B)], 1, [1] * B, seed=3, distinct=4)
    call(c)
    call(c)
    torch.cuda.synchronize()
    assert c.err.item() == 0
    keep = [0, 1, 2, 700, 1400, 2099]
    got = c.out
    for b in keep:
        K, V = c.rows(b, 3)
        K = np.concatenate([K, syn.from_bits(c.k[b, :1, 3], cfg.dtype).astype(np.float64)])
        V = np.concatenate([V, syn.from_bits(c.v[b, :1, 3], cfg.dtype).astype(np.float64)])
        want, tol = attend(syn.from_bits(c.q[b, 0, 3], cfg.dtype).astype(np.float64), K, V)
        assert_row(got[b, 0, 3].cpu().numpy(), want, tol, f"sequence {b}")
