"""The accepted path of a drafted tree into the window: the same bytes as appending its tokens
one by one, across the flush of a window it fills."""
import numpy as np
import pytest
import torch

from bit_mixed_precision_channel_b200 import binding as kb
from bit_mixed_precision_channel_b200 import synthetic as syn

from _kv import to_dev
from _spec import D

pytestmark = pytest.mark.gpu


def setup(cfg, res_len, n_path, T, seed):
    rng = np.random.default_rng(seed)
    B, H, P = len(res_len), cfg.num_kv_heads, cfg.page_tokens
    bits = lambda *s: to_dev(syn.to_bits(rng.standard_normal(s).astype(np.float32), cfg.dtype), cfg.dtype)  # noqa: E731
    ints = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    path = np.full((B, T), -5)
    for b, n in enumerate(n_path):
        path[b, :n] = np.sort(rng.choice(T, n, replace=False))
    return dict(k_draft=bits(B, T, H, D), v_draft=bits(B, T, H, D), path=ints(path), n_path=ints(n_path),
                taken=ints([0] * B), res_k=bits(B, H, P, D), res_v=bits(B, H, P, D), res_len=ints(res_len),
                err=torch.zeros(1, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("dtype,H,P,T,res_len,n_path", [
    (kb.F16, 8, 128, 32, [0, 100, 127, 128, 60], [5, 9, 3, 4, 0]),
    (kb.BF16, 1, 32, 1, [0, 31, 32], [1, 1, 1]),
    (kb.F16, 3, 64, 128, [0, 63], [64, 100]),
])
def test_path_equals_single_appends_and_flushes(dtype, H, P, T, res_len, n_path):
    cfg = kb.Config(num_q_heads=H, num_kv_heads=H, page_tokens=P, num_boost=16, dtype=dtype)
    B = len(res_len)
    a = setup(cfg, res_len, n_path, T, seed=P + T)
    cache = [dict(res_k=a["res_k"].clone(), res_v=a["res_v"].clone(), res_len=a["res_len"].clone(),
                  table=torch.full((B, 4), -1, dtype=torch.int32, device="cuda"),
                  num_pages=torch.zeros(B, dtype=torch.int32, device="cuda"),
                  pool=torch.zeros(4 * B * H * kb.page_bytes(cfg), dtype=torch.uint8, device="cuda")) for _ in range(2)]
    page = [torch.arange(B, dtype=torch.int32, device="cuda") + i * B for i in range(4)]

    def flush(c, i):
        kb.flush_residual(cfg, c["res_k"], c["res_v"], c["res_len"], page[i], c["table"], c["num_pages"], c["pool"], a["err"])

    c = cache[0]
    for i in range(4):
        kb.append_path(cfg, a["k_draft"], a["v_draft"], a["path"], a["n_path"], a["taken"], c["res_k"], c["res_v"],
                       c["res_len"], a["err"])
        flush(c, i)
    torch.cuda.synchronize()
    assert a["err"].item() == 0 and torch.equal(a["taken"], a["n_path"])
    c = cache[1]  # one sequence at a time, one token at a time
    for b in range(B):
        one = {n: c[n][b:b + 1] for n in ("res_k", "res_v", "res_len", "table", "num_pages")} | dict(pool=c["pool"])
        flushes = 0

        def flush_one():
            nonlocal flushes
            kb.flush_residual(cfg, one["res_k"], one["res_v"], one["res_len"], page[flushes][b:b + 1], one["table"],
                              one["num_pages"], one["pool"], a["err"])
            flushes += 1

        if res_len[b] == P:
            flush_one()
        for s in range(n_path[b]):
            node = int(a["path"][b, s])
            kb.append_token(cfg, a["k_draft"][b:b + 1, node].contiguous(), a["v_draft"][b:b + 1, node].contiguous(),
                            one["res_k"], one["res_v"], one["res_len"], a["err"])
            if int(one["res_len"]) == P:
                flush_one()
    torch.cuda.synchronize()
    assert a["err"].item() == 0
    assert torch.equal(cache[0]["num_pages"], cache[1]["num_pages"])
    assert torch.equal(cache[0]["res_len"], cache[1]["res_len"])
    R = kb.page_bytes(cfg) * H
    for b in range(B):
        n = int(cache[0]["res_len"][b])
        for name in ("res_k", "res_v"):
            assert torch.equal(cache[0][name][b, :, :n], cache[1][name][b, :, :n])
        for i in range(int(cache[0]["num_pages"][b])):
            p, q = int(cache[0]["table"][b, i]), int(cache[1]["table"][b, i])
            assert torch.equal(cache[0]["pool"][p * R:(p + 1) * R], cache[1]["pool"][q * R:(q + 1) * R])


def test_rows_outside_the_path_are_left():
    cfg = kb.Config(num_q_heads=2, num_kv_heads=2, page_tokens=32, num_boost=16)
    a = setup(cfg, [10, 30], [4, 9], 16, seed=3)
    before = a["res_k"].clone()
    kb.append_path(cfg, **a)
    torch.cuda.synchronize()
    assert a["res_len"].tolist() == [14, 32] and a["taken"].tolist() == [4, 2] and a["err"].item() == 0
    assert torch.equal(a["res_k"][0, :, :10], before[0, :, :10]) and torch.equal(a["res_k"][0, :, 14:], before[0, :, 14:])
    for s in range(4):
        assert torch.equal(a["res_k"][0, :, 10 + s], a["k_draft"][0, int(a["path"][0, s])])


def test_bad_lengths_skip_the_sequence_and_bad_nodes_are_flagged():
    cfg = kb.Config(num_q_heads=2, num_kv_heads=2, page_tokens=32, num_boost=16)
    for name, value in (("res_len", 33), ("res_len", -1), ("n_path", 17), ("n_path", -1), ("taken", 5), ("taken", -1)):
        a = setup(cfg, [10, 10], [4, 4], 16, seed=3)
        a[name][1] = value
        before = a["res_k"].clone(), a["taken"].clone(), a["res_len"].clone()
        kb.append_path(cfg, **a)
        torch.cuda.synchronize()
        assert a["err"].item() == kb.DEV_ERR_LENGTH, name
        assert torch.equal(a["res_k"][1], before[0][1]) and a["res_len"][0].item() == 14
        assert a["taken"][1] == before[1][1] and a["res_len"][1] == before[2][1]
    for node in (-1, 16, 2 ** 31 - 1):
        a = setup(cfg, [10], [4], 16, seed=3)
        a["path"][0, 2] = node
        kb.append_path(cfg, **a)
        torch.cuda.synchronize()
        assert a["err"].item() == kb.DEV_ERR_LENGTH
        assert torch.equal(a["res_k"][0, :, 12], a["k_draft"][0, 0])
