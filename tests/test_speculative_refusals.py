"""Calls of speculative decoding that are refused on the host, through the C ABI and the binding
(CPU only: nothing is enqueued)."""
import ctypes

import pytest
import torch

from bit_mixed_precision_channel_b200 import binding as kb
from bit_mixed_precision_channel_b200 import build as kbuild

CFG = kb.Config(num_q_heads=8, num_kv_heads=2, page_tokens=32, num_boost=16)
B, MAXP, POOL, T = 3, 4, 6, 5
H, HQ, P, D = 2, 8, 32, 128
X = 0x10000  # an address that no check follows
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kb.load()


def c(cfg=CFG):
    return ctypes.byref(cfg.c())


SELECT = dict(cfg=CFG, pool=X, pool_pages=POOL, q=X, batch=B, page_table=X, max_pages=MAXP, num_pages=X, n_first=1,
              n_recent=1, n_select=3, sel=X, n_sel=X, err=None, stream=None)
SPARSE = dict(cfg=CFG, pool=X, pool_pages=POOL, q=X, batch=B, page_table=X, max_pages=MAXP, num_pages=X, sel=X, max_sel=3,
              n_sel=X, res_k=X, res_v=X, res_len=X, sm_scale=0.1, out=X, workspace=X, workspace_bytes=BIG, err=None,
              stream=None)
TREE = dict(cfg=CFG, pool=X, pool_pages=POOL, q=X, n_draft=T, batch=B, page_table=X, max_pages=MAXP, num_pages=X, res_k=X,
            res_v=X, res_len=X, k_draft=X, v_draft=X, mask=X, draft_len=X, sm_scale=0.1, out=X, workspace=X,
            workspace_bytes=BIG, err=None, stream=None)
PATH = dict(cfg=CFG, batch=B, n_draft=T, k_draft=X, v_draft=X, path=X, n_path=X, taken=X, res_k=X, res_v=X, res_len=X,
            err=None, stream=None)
CALLS = dict(kvq_select_pages=SELECT, kvq_decode_attention_sparse=SPARSE, kvq_tree_attention=TREE, kvq_append_path=PATH)


def status(lib, name, **over):
    a = {**CALLS[name], **over}
    return getattr(lib, name)(c(a.pop("cfg")), *a.values())


OPTIONAL = {"err", "stream", "cfg"}


@pytest.mark.parametrize("name", list(CALLS))
def test_null_pointers_and_negative_sizes(lib, name):
    for arg, v in CALLS[name].items():
        if v == X:
            assert status(lib, name, **{arg: None}) == 1, arg
    for arg in ("batch", "max_pages", "max_sel", "n_draft", "n_first", "n_recent"):
        if arg in CALLS[name]:
            assert status(lib, name, **{arg: -1}) == 1, arg
    if "pool_pages" in CALLS[name]:
        assert status(lib, name, pool_pages=0) == 1
    assert status(lib, name, cfg=kb.Config(head_dim=64)) == 2


@pytest.mark.parametrize("name,args", [
    ("kvq_select_pages", ("pool", "q")), ("kvq_decode_attention_sparse", ("pool", "q", "res_k", "res_v", "workspace")),
    ("kvq_tree_attention", ("pool", "q", "res_k", "res_v", "k_draft", "v_draft", "out", "workspace")),
    ("kvq_append_path", ("k_draft", "v_draft", "res_k", "res_v")),
])
def test_misaligned_buffers(lib, name, args):
    for arg in args:
        assert status(lib, name, **{arg: X + 8}) == 1, arg


def test_an_empty_batch_needs_no_buffers(lib):
    for name, a in CALLS.items():
        assert status(lib, name, batch=0, **{n: None for n, v in a.items() if v == X}) == 0, name


def test_limits(lib):
    assert status(lib, "kvq_select_pages", n_select=0) == 1
    assert status(lib, "kvq_select_pages", n_first=2, n_recent=2) == 1
    assert status(lib, "kvq_select_pages", n_first=2 ** 31 - 1, n_recent=2 ** 31 - 1, n_select=2 ** 31 - 1) == 1
    assert status(lib, "kvq_select_pages", max_pages=204801) == 2
    for name in ("kvq_tree_attention", "kvq_append_path"):
        assert status(lib, name, n_draft=0) == 1
        assert status(lib, name, n_draft=kb.MAX_DRAFT + 1) == 2
    assert status(lib, "kvq_decode_attention_sparse", batch=1 << 20, max_sel=1 << 20) == 1  # past the 32-bit work line
    assert status(lib, "kvq_tree_attention", batch=1 << 20, max_pages=1 << 20) == 1


def test_workspace_sizes(lib):
    need = kb.decode_workspace_bytes(CFG, B, MAXP)
    assert status(lib, "kvq_decode_attention_sparse", workspace_bytes=need - 1) == 4
    need = kb.tree_workspace_bytes(CFG, B, T)
    assert need > 0
    assert status(lib, "kvq_tree_attention", workspace_bytes=need - 1) == 4
    for batch, n in ((-1, 1), (1, 0), (1, kb.MAX_DRAFT + 1)):
        assert kb.tree_workspace_bytes(CFG, batch, n) == 0
    assert kb.tree_workspace_bytes(kb.Config(head_dim=64), 1, 1) == 0


def tensors(**over):
    i32, f16 = torch.int32, torch.float16
    t = dict(pool=torch.zeros(POOL * H * kb.page_bytes(CFG), dtype=torch.uint8),
             page_table=torch.zeros(B, MAXP, dtype=i32), num_pages=torch.zeros(B, dtype=i32),
             res_k=torch.zeros(B, H, P, D, dtype=f16), res_v=torch.zeros(B, H, P, D, dtype=f16),
             res_len=torch.zeros(B, dtype=i32))
    t.update(over)
    return t


def select_args(**over):
    t = tensors()
    a = dict(pool=t["pool"], q=torch.zeros(B, HQ, D, dtype=torch.float16), page_table=t["page_table"],
             num_pages=t["num_pages"], sel=torch.zeros(B, H, 3, dtype=torch.int32), n_sel=torch.zeros(B, dtype=torch.int32))
    a.update(over)
    return a


def tree_args(**over):
    a = tensors(q=torch.zeros(B, T, HQ, D, dtype=torch.float16), k_draft=torch.zeros(B, T, H, D, dtype=torch.float16),
                v_draft=torch.zeros(B, T, H, D, dtype=torch.float16), mask=torch.zeros(B, T, 1, dtype=torch.int32),
                draft_len=torch.zeros(B, dtype=torch.int32), out=torch.zeros(B, T, HQ, D),
                workspace=torch.zeros(kb.tree_workspace_bytes(CFG, B, T), dtype=torch.uint8))
    a.update(over)
    return a


def path_args(**over):
    t = tensors()
    a = dict(k_draft=torch.zeros(B, T, H, D, dtype=torch.float16), v_draft=torch.zeros(B, T, H, D, dtype=torch.float16),
             path=torch.zeros(B, T, dtype=torch.int32), n_path=torch.zeros(B, dtype=torch.int32),
             taken=torch.zeros(B, dtype=torch.int32), res_k=t["res_k"], res_v=t["res_v"], res_len=t["res_len"])
    a.update(over)
    return a


def sparse_args(**over):
    a = tensors(q=torch.zeros(B, HQ, D, dtype=torch.float16), sel=torch.zeros(B, H, 3, dtype=torch.int32),
                n_sel=torch.zeros(B, dtype=torch.int32), out=torch.zeros(B, HQ, D),
                workspace=torch.zeros(64, dtype=torch.uint8))
    a.update(over)
    return a


Z = torch.zeros
BAD = [
    (kb.select_pages, select_args, dict(sel=Z(B, H, 3, dtype=torch.int64)), "sel: dtype"),
    (kb.select_pages, select_args, dict(sel=Z(B, 3, dtype=torch.int32)), "sel must have 3"),
    (kb.select_pages, select_args, dict(sel=Z(B, H + 1, 3, dtype=torch.int32)), "sel: shape"),
    (kb.select_pages, select_args, dict(q=Z(B, HQ, D, dtype=torch.bfloat16)), "q: dtype"),
    (kb.select_pages, select_args, dict(n_sel=Z(B - 1, dtype=torch.int32)), "n_sel: 2 elements"),
    (kb.decode_attention_sparse, sparse_args, dict(sel=Z(B, H, 6, dtype=torch.int32)[:, :, ::2]), "sel must be contiguous"),
    (kb.decode_attention_sparse, sparse_args, dict(sel=Z(B - 1, H, 3, dtype=torch.int32)), "sel: shape"),
    (kb.decode_attention_sparse, sparse_args, dict(out=Z(B, HQ, D, dtype=torch.float16)), "out: dtype"),
    (kb.tree_attention, tree_args, dict(q=Z(B, HQ, D, dtype=torch.float16)), "q must have 4"),
    (kb.tree_attention, tree_args, dict(q=Z(B, T, HQ - 1, D, dtype=torch.float16)), "q: "),
    (kb.tree_attention, tree_args, dict(mask=Z(B, T, 1, dtype=torch.bool)), "mask: dtype"),
    (kb.tree_attention, tree_args, dict(mask=Z(B, T - 1, 1, dtype=torch.int32)), "mask: "),
    (kb.tree_attention, tree_args, dict(v_draft=Z(B, T, H, D - 1, dtype=torch.float16)), "v_draft: "),
    (kb.tree_attention, tree_args, dict(k_draft=Z(B, H, T, D, dtype=torch.float16).transpose(1, 2)), "k_draft must be contiguous"),
    (kb.tree_attention, tree_args, dict(draft_len=Z(B, dtype=torch.int64)), "draft_len: dtype"),
    (kb.tree_attention, tree_args, dict(out=Z(B, T - 1, HQ, D)), "out: "),
    (kb.append_path, path_args, dict(path=Z(B * T, dtype=torch.int32)), "path must have 2"),
    (kb.append_path, path_args, dict(taken=Z(B, dtype=torch.int64)), "taken: dtype"),
    (kb.append_path, path_args, dict(res_v=Z(B, H, P - 1, D, dtype=torch.float16)), "res_v: "),
]


@pytest.mark.parametrize("fn,make,over,msg", BAD)
def test_binding_refuses(fn, make, over, msg):
    with pytest.raises(ValueError, match=msg):
        fn(CFG, **make(**over))


@pytest.mark.parametrize("fn,make", [(kb.select_pages, select_args), (kb.decode_attention_sparse, sparse_args),
                                     (kb.tree_attention, tree_args), (kb.append_path, path_args)])
def test_well_formed_tensors_fail_only_on_the_device_check(fn, make):
    with pytest.raises(ValueError, match="CUDA tensors"):
        fn(CFG, **make())


def test_a_config_that_was_used_can_be_copied_and_pickled(lib):
    import copy
    import pickle
    cfg = kb.Config(num_q_heads=8, num_kv_heads=2, page_tokens=32, num_boost=16)
    cfg._marshalled()
    for other in (copy.copy(cfg), copy.deepcopy(cfg), pickle.loads(pickle.dumps(cfg))):
        assert other == cfg and hash(other) == hash(cfg)
        assert other._marshalled()[1:] == cfg._marshalled()[1:]


def test_a_config_the_library_does_not_take_is_named(lib):
    for cfg in (kb.Config(head_dim=64), kb.Config(num_boost=7), kb.Config(num_q_heads=7, num_kv_heads=2)):
        z = torch.zeros(1)
        for call in (lambda: kb.select_pages(cfg, z, z, z, z, z, z), lambda: kb.append_path(cfg, z, z, z, z, z, z, z, z)):
            with pytest.raises(kb.KVQError, match="kvq_check_config"):
                call()
