"""Window rows that are no finite number, in the plain decode step: the range flag, as documented, and
never a quiet row of zeros."""
import pytest
import torch

from bit_mixed_precision_channel_b200 import binding as kb

from _kv import to_dev
from _spec import Cache, D

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("where", ["key", "value"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dtype", [kb.F16, kb.BF16])
@pytest.mark.parametrize("pages,window", [(0, 3), (2, 3), (40, 20)])
@pytest.mark.parametrize("gqa", [1, 8])
def test_window_rows_that_are_no_number_are_flagged(gqa, pages, window, dtype, value, where):
    cfg = kb.Config(num_q_heads=gqa, num_kv_heads=1, page_tokens=32, num_boost=16, dtype=dtype)
    c = Cache(cfg, [pages], [window], seed=6)
    q = to_dev(c.queries(1), dtype)
    ws = torch.zeros(kb.decode_workspace_bytes(cfg, 1, c.max_pages), dtype=torch.uint8, device="cuda")
    out = torch.empty(1, gqa, D, device="cuda")
    for bad in (False, True):
        if bad:
            c.d["res_k" if where == "key" else "res_v"][:, :, 1, 40] = value
        kb.decode_attention(cfg, c.d["pool"], q, c.d["page_table"], c.d["num_pages"], c.d["res_k"], c.d["res_v"], c.d["res_len"],
                            out, ws, err=c.err)
        torch.cuda.synchronize()
        assert c.err.item() == (kb.DEV_ERR_RANGE if bad else 0)
