"""Drafted tensors whose rows are not those of the call: refused by the binding, because the library
would read them with the wrong stride (CPU only)."""
import pytest
import torch

from bit_mixed_precision_channel_b200 import binding as kb
from bit_mixed_precision_channel_b200 import cache as kc

from test_speculative_refusals import B, CFG, D, H, HQ, T, path_args, tree_args

Z = torch.zeros
F16, I32 = torch.float16, torch.int32


def kv(*shape):
    return Z(*shape, dtype=F16)


WRONG = [
    # an accepted path shorter than the tree: sequence 1 would be read at token `depth` of sequence 0
    (kb.append_path, path_args, dict(path=Z(B, T - 2, dtype=I32)), "k_draft: shape"),
    (kb.append_path, path_args, dict(k_draft=kv(B, T + 1, H, D)), "k_draft: shape"),
    (kb.append_path, path_args, dict(v_draft=kv(B, T + 1, H, D)), "v_draft: shape"),
    (kb.append_path, path_args, dict(v_draft=kv(B, T, 2 * H, D)), "v_draft: shape"),
    (kb.append_path, path_args, dict(k_draft=kv(B, H, T, D)), "k_draft: shape"),
    (kb.append_path, path_args, dict(k_draft=kv((B + 1) * T, H, D)), "k_draft: "),
    (kb.append_path, path_args, dict(k_draft=kv(B - 1, T, H, D)), "k_draft: shape"),
    (kb.tree_attention, tree_args, dict(q=kv(B, T - 1, HQ, D), out=Z(B, T - 1, HQ, D), mask=Z(B, T - 1, 1, dtype=I32)),
     "k_draft: shape"),
    (kb.tree_attention, tree_args, dict(q=kv(B, T, HQ + 1, D)), "q: shape"),
    (kb.tree_attention, tree_args, dict(k_draft=kv(B, T + 3, H, D)), "k_draft: shape"),
    (kb.tree_attention, tree_args, dict(v_draft=kv(B, T + 3, H, D)), "v_draft: shape"),
    (kb.tree_attention, tree_args, dict(v_draft=kv(B, H, T, D)), "v_draft: shape"),
    (kb.tree_attention, tree_args, dict(mask=Z(B, T, 2, dtype=I32)), "mask: shape"),
    (kb.tree_attention, tree_args, dict(mask=Z(B, T + 1, 1, dtype=I32)), "mask: shape"),
    (kb.tree_attention, tree_args, dict(mask=Z(B, T + 1, dtype=I32)), "mask: "),
    (kb.tree_attention, tree_args, dict(out=Z(B, T + 1, HQ, D)), "out: shape"),
    (kb.tree_attention, tree_args, dict(out=Z(B, HQ, T, D)), "out: shape"),
]


@pytest.mark.parametrize("fn,make,over,msg", WRONG)
def test_rows_of_another_length_are_refused(fn, make, over, msg):
    with pytest.raises(ValueError, match=msg):
        fn(CFG, **make(**over))


@pytest.mark.parametrize("fn,make,over", [
    # buffers of more sequences than the batch, flat ones, rows without the dimension of one mask word
    (kb.append_path, path_args, dict(k_draft=kv(B + 2, T, H, D), v_draft=kv(B * T, H, D))),
    (kb.append_path, path_args, dict(k_draft=kv(B * T * H * D))),
    (kb.tree_attention, tree_args, dict(mask=Z(B, T, dtype=I32), out=Z(B * T, HQ, D), q=kv(B + 1, T, HQ, D))),
    (kb.tree_attention, tree_args, dict(k_draft=kv(B, T, H * D), v_draft=kv(B * T * H, D))),
])
def test_other_shapes_of_the_same_rows_are_taken(fn, make, over):
    with pytest.raises(ValueError, match="CUDA tensors"):  # all that is left to refuse here
        fn(CFG, **make(**over))


def test_accept_refuses_a_path_narrower_than_the_tree_before_anything_changes():
    c = kc.PagedKVCache(CFG, B, max_pages=4, pool_pages=12, device="cpu")
    k = kv(B, T, H, D)
    with pytest.raises(ValueError, match="k_draft: shape"):
        c.accept(k, k, Z(B, 2, dtype=I32), [2, 1, 0])
    assert c.host_res_len == [0] * B and c.res_len.tolist() == [0] * B and len(c.free) == 12
