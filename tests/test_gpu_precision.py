"""How near attention over long caches stays to 64 bits: near enough that the loss of one part of the
split operands would show.

Bound, 1e-5 for keys and queries of about unit variance, unit values and 2000 to 4100 tokens.
* Logits: 16 accumulations (8 of 16 channels, a high and a low part), each truncated by at most 2^-23 of
  a partial sum, which stays below about 8: 1.5e-5 at the very most, all of one sign.  The output moves
  by sum p d (v - o); over n_eff = n / exp(var z) >= 380 effective tokens (var z = exp(1/2)) whose values
  are independent, and at 4.5 standard deviations (some thousand elements): 1.5e-5 * 4.5 / sqrt(380) = 3.5e-6.
* Output sums: centred codes leave |o| < 0.3; at most 64 truncated accumulations before a sum moves to fp32
  that rounds to nearest, 64 * 2^-23 * 0.3 = 2.3e-6.
* Operands carried to 22 bits: 2^-22 of the weights, below 1e-6.
Together 6.8e-6.  Without the keys' remainders a row is off by 1.3e-5 to 2.2e-4, without the low parts of
the probabilities by 1.4e-5 to 5.5e-5 (both computed in 64 bits on this data, every one of 48 rows above
1e-5); output sums left in tensor memory over 28 tiles were off by 3.6e-5.  The third part of a bf16
window's probabilities (2^-18 of them) and the centring of the sums over chosen pages (6e-6) are below
this bound."""
import numpy as np
import pytest
import torch

from bit_mixed_precision_channel_b200 import binding as kb
from bit_mixed_precision_channel_b200 import synthetic as syn

from _spec import Cache, D, attend
from test_gpu_select import sparse
from test_gpu_tree import call, make

pytestmark = pytest.mark.gpu

BOUND = 1e-5


def worst(c, out, seqs, heads):
    """Largest error over the drafted rows of some sequences and kv heads."""
    cfg, off = c.cfg, 0.0
    out = out.cpu().numpy().astype(np.float64)
    for b in seqs:
        n = c.drafts[b]
        for h in heads:
            K, V = c.rows(b, h)
            K = np.concatenate([K, syn.from_bits(c.k[b, :n, h], cfg.dtype).astype(np.float64)])
            V = np.concatenate([V, syn.from_bits(c.v[b, :n, h], cfg.dtype).astype(np.float64)])
            for i in range(n):
                sees = np.concatenate([np.ones(len(K) - n, bool), c.sees[b, i, :n]])
                for g in range(cfg.gqa):
                    hq = h * cfg.gqa + g
                    want, _ = attend(syn.from_bits(c.q[b, i, hq], cfg.dtype).astype(np.float64), K, V, sees)
                    off = max(off, np.abs(out[b, i, hq] - want).max())
    return off


@pytest.mark.parametrize("dtype", [kb.F16, kb.BF16])
@pytest.mark.parametrize("T,gqa", [(6, 4), (17, 8), (2, 4), (1, 8), (5, 1)])
@pytest.mark.parametrize("P,k", [(128, 32), (32, 0), (64, 128)])
def test_trees_over_thousands_of_tokens(dtype, T, gqa, P, k):
    cfg = kb.Config(num_q_heads=gqa, num_kv_heads=1, page_tokens=P, num_boost=k, dtype=dtype)
    c = make(cfg, [2048 // P, 4096 // P], [17, P - 1], T, [T, T], seed=T + P, distinct=40)
    call(c)
    torch.cuda.synchronize()
    assert c.err.item() == 0
    assert worst(c, c.out, range(2), [0]) <= BOUND


@pytest.mark.parametrize("dtype", [kb.F16, kb.BF16])
def test_units_that_one_block_walks_alone(dtype):
    """As many units of 32 tiles as the GPU has SMs: sums over whole sequences in one block."""
    cfg = kb.Config(num_q_heads=32, num_kv_heads=8, page_tokens=128, num_boost=32, dtype=dtype)
    c = make(cfg, [32] * 20, [(7 * b) % 128 for b in range(20)], 4, [4] * 20, seed=3, distinct=12)
    call(c)
    torch.cuda.synchronize()
    assert c.err.item() == 0
    assert worst(c, c.out, [0, 9, 19], [0, 3, 7]) <= BOUND


@pytest.mark.parametrize("dtype", [kb.F16, kb.BF16])
@pytest.mark.parametrize("P,k,gqa", [(128, 32, 4), (64, 16, 8), (32, 0, 1)])
def test_chosen_pages_of_thousands_of_tokens(dtype, P, k, gqa):
    cfg = kb.Config(num_q_heads=gqa, num_kv_heads=1, page_tokens=P, num_boost=k, dtype=dtype)
    n = 2048 // P
    c = Cache(cfg, [2 * n, n + 3], [9, P - 1], seed=P, distinct=40)
    q = c.queries(2)
    sel = np.stack([np.sort(c.rng.permutation(p)[:n])[None] for p in c.pages])
    out = sparse(c, q, c.ints(sel), c.ints([n, n])).cpu().numpy().astype(np.float64)
    assert c.err.item() == 0
    for b in range(2):
        K, V = c.rows(b, 0, sel[b, 0])
        for g in range(gqa):
            want, _ = attend(syn.from_bits(q[b, g], dtype).astype(np.float64), K, V)
            assert np.abs(out[b, g] - want).max() <= BOUND


@pytest.mark.parametrize("dtype", [kb.F16, kb.BF16])
def test_a_verified_token_is_the_decode_steps_token(dtype):
    """The single drafted token against the decode call after its append: each within the bound of 64 bits
    (the plain form's sums are not centred: 16 groups a warp, two truncations of 2^-23 of at most 1.5, 6e-6)."""
    cfg = kb.Config(num_q_heads=8, num_kv_heads=2, page_tokens=64, num_boost=32, dtype=dtype)
    c = make(cfg, [32, 30], [20, 0], 1, [1, 1], seed=12, garbage=False, distinct=40)
    call(c)
    d = c.d
    kb.append_token(cfg, c.t["k_draft"], c.t["v_draft"], d["res_k"], d["res_v"], d["res_len"], c.err)
    ws = torch.zeros(kb.decode_workspace_bytes(cfg, 2, c.max_pages), dtype=torch.uint8, device="cuda")
    out = torch.empty(2, 8, D, device="cuda")
    kb.decode_attention(cfg, d["pool"], c.t["q"], d["page_table"], d["num_pages"], d["res_k"], d["res_v"], d["res_len"],
                        out, ws, err=c.err)
    torch.cuda.synchronize()
    assert c.err.item() == 0
    assert (out - c.out[:, 0]).abs().max() <= 2 * BOUND
