"""Measured cases of the operators around speculative decoding over the 2-bit KV cache:

  select  choice of the pages a decode step reads, by the largest logits their stored key ranges allow
  sparse  decode attention over the chosen pages and the residual window
  tree    attention of a tree of drafted tokens over the whole cache, the residual window and the drafted tokens themselves
  append  the accepted path of a tree moved into the residual window

A step drafts with `select` and `sparse`, verifies the drafted tree with `tree`, and keeps what was accepted with `append`.
`run` computes them with elementary torch operations, or, with `own` set, through the package's calls on the same buffers."""
import math

import numpy as np
import torch

own = False

D = 128   # channels of a head
G = 32    # tokens that share a key scale
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- cases


def _case(name, op, dtype, batch, kv_heads, group, page, boost, pages, ragged, **more):
    return dict(name=name, op=op, dtype=dtype, batch=batch, kv_heads=kv_heads, group=group, page=page, boost=boost, pages=pages,
                ragged=ragged, **more)


def listed():
    return [
        # one user's chat of 4096 tokens: the smallest step, where launches and latency count
        _case("select one 4K", "select", "fp16", 1, 8, 4, 128, 32, 32, False, select=8, first=1, recent=1),
        # four documents of 32768 tokens, an eighth of the pages kept
        _case("select four 32K", "select", "fp16", 4, 8, 4, 128, 16, 256, False, select=32, first=1, recent=2),
        # a serving batch of ragged lengths in pages of 64 tokens, 8 query heads a kv head
        _case("select ragged 64", "select", "bf16", 64, 8, 8, 64, 32, 250, True, select=48, first=1, recent=4),
        # one head, pages of 32 tokens: the smallest attention over a choice of pages
        _case("sparse tiny", "sparse", "fp16", 1, 1, 1, 32, 16, 40, False, select=12),
        # the four documents' attention over the pages chosen above
        _case("sparse four 32K", "sparse", "fp16", 4, 8, 4, 128, 16, 256, False, select=32),
        # the ragged batch's attention
        _case("sparse ragged 64", "sparse", "bf16", 64, 8, 8, 64, 32, 250, True, select=48),
        # no draft to verify but the token itself: the single-token step of a batch of 16 x 4096 tokens
        _case("tree single 16x4K", "tree", "fp16", 16, 8, 4, 128, 32, 32, False, draft=1, chain=True),
        # a drafted chain of one user over some 1000 tokens, no grouped heads
        _case("tree chain one 1K", "tree", "fp16", 1, 8, 1, 64, 16, 15, False, draft=7, chain=True),
        # trees of 32 nodes for the batch of 16 x 4096 tokens
        _case("tree 32 16x4K", "tree", "fp16", 16, 8, 4, 128, 32, 32, False, draft=32, chain=False),
        # large batch, 8 query heads a kv head, ragged trees of up to 61 nodes over ragged lengths up to 8192
        _case("tree 61 ragged 32x8K", "tree", "bf16", 32, 8, 8, 128, 32, 64, True, draft=61, chain=False),
        # the accepted paths of 16 sequences' trees of 32 nodes
        _case("append 16", "append", "fp16", 16, 8, 4, 128, 32, 2, False, draft=32),
        # the large batch's accepted chains; some fill their window
        _case("append ragged 128", "append", "bf16", 128, 8, 8, 128, 32, 2, True, draft=48),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["select", "sparse", "tree", "append"])
    c = dict(op=op, dtype=rng.choice(["fp16", "bf16"]), kv_heads=rng.choice([1, 2, 4, 8]), group=rng.choice([1, 2, 4, 8]),
             page=rng.choice([32, 64, 128]), boost=rng.choice([0, 16, 32, 64, 128]), ragged=rng.random() < 0.5)
    if op in ("select", "sparse"):
        c["batch"] = _log(rng, 1, 64)
        c["pages"] = _log(rng, 4, 256)
        c["select"] = min(_log(rng, 3, 64), c["pages"])
        if op == "select":
            c["first"], c["recent"] = rng.randint(0, 1), rng.randint(0, 2)
    elif op == "tree":
        c["draft"] = _log(rng, 1, 64)
        c["chain"] = rng.random() < 0.3
        c["batch"] = _log(rng, 1, 32)
        c["pages"] = _log(rng, 1, 64 * 128 // c["page"])
    else:
        c["batch"], c["pages"], c["draft"] = _log(rng, 1, 128), 2, _log(rng, 1, 64)
    most = [work(x) for x in listed() if x["op"] == op]
    while c["batch"] > 1 and any(work(c)[m] > max(w[m] for w in most) for m in ("bytes", "flops")):
        c["batch"] = (c["batch"] + 1) // 2  # no more work than the largest listed case of the operator
    return c


# ---------------------------------------------------------------- sizes that follow from a case


def _lengths(c):
    """Pages, residual tokens, drafted tokens and accepted tokens of every sequence."""
    B, N, P, T = c["batch"], c["pages"], c["page"], c.get("draft", 1)
    i = np.arange(B)
    if c["ragged"]:
        pages = np.maximum(1, np.ceil(N * (0.12 + 0.88 * ((i * 0.6180339887 + 0.99) % 1.0)))).astype(np.int64)
        drafts = 1 + (T - 1 - 7 * i) % T
    else:
        pages, drafts = np.full(B, N), np.full(B, T)
    window = (P // 2 + 5 + 29 * i) % P
    if c["ragged"] and B >= 8:
        pages[3], window[3] = 0, 0  # a sequence without a cache
    depth = np.minimum(drafts, 1 + (3 + 5 * i) % 9)
    return pages, window, drafts, depth


def _layout(P, k):
    sizes = [("k_codes", P * D // 4), ("kb_codes", P * k // 4), ("v_codes", P * D // 4), ("k_scale", P // G * D * 2),
             ("k_zero", P // G * D * 2), ("kb_scale", P // G * k * 2), ("v_scale", P * 2), ("v_zero", P * 2), ("boost_idx", k)]
    at, off = {}, 0
    for name, n in sizes:
        at[name] = (off, off + n)
        off += n
    return at, off, (off + 127) // 128 * 128


def work(c):
    B, H, gq, P, k, N = c["batch"], c["kv_heads"], c["group"], c["page"], c["boost"], c["pages"]
    pages, window, drafts, depth = _lengths(c)
    _, payload, _ = _layout(P, k)
    q_bytes = B * H * gq * D * 2
    if c["op"] == "select":
        meta = P // G * (2 * D + k) * 2 + k  # scales, zeros and boosted channels
        n = int(pages.sum()) * H
        return {"bytes": n * meta + q_bytes + B * H * c["select"] * 4 + int(pages.sum()) * 4, "flops": 2 * n * P // G * (2 * D + k)}
    if c["op"] == "sparse":
        sel = np.minimum(pages, c["select"])
        tok = int((sel * P + window).sum()) * H
        return {"bytes": int(sel.sum()) * H * payload + int(window.sum()) * H * D * 4 + q_bytes + B * H * gq * D * 4 + B * H * c["select"] * 4,
                "flops": 4 * tok * gq * D}
    if c["op"] == "tree":
        rows = drafts * gq
        kv = int(pages.sum()) * H * payload + int((window + drafts).sum()) * H * D * 4
        return {"bytes": kv + int(rows.sum()) * H * D * 6, "flops": 4 * D * H * int((rows * (pages * P + window + drafts)).sum())}
    taken = np.minimum(depth, P - window)
    return {"bytes": int(taken.sum()) * H * D * 2 * 4 + B * c["draft"] * 4, "flops": 0}


# ---------------------------------------------------------------- inputs


def _make_pool(g, pages, H, P, k, dtype, dev):
    """Records as the quantizer leaves them for Gaussian keys of log-normal channel widths with a few wide channels: codes
    binomial over the range, ranges of about 4.1 widths a group, the widest channels at 4 bits."""
    at, payload, stride = _layout(P, k)
    pool = torch.zeros(pages, H, stride, dtype=torch.uint8, device=dev)

    def put(name, x):
        a, b = at[name]
        if b > a:
            pool[:, :, a:b] = x.contiguous().view(torch.uint8).reshape(pages, H, b - a)

    def bits(n):
        return torch.randint(-(1 << 31), 1 << 31, (pages, H, n), generator=g, device=dev, dtype=torch.int32)

    def codes(n):  # the sum of three random bits in each field of two
        m = 0x55555555
        return (bits(n) & m) + (bits(n) & m) + (bits(n) & m)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    width = torch.exp(normal(H, D))
    wide = torch.rand(H, D, generator=g, device=dev).argsort(-1)[:, :5]
    width.scatter_(1, wide, width.gather(1, wide) * (8 + 12 * torch.rand(H, 5, generator=g, device=dev)))
    score = width * (1 + 0.1 * normal(pages, H, D))
    idx = score.argsort(-1, descending=True)[..., :k].sort(-1).values  # [pages][H][k]
    lo = -width[:, None] * (2.05 + 0.35 * normal(pages, H, P // G, D)).clamp(0.5, 4)
    hi = width[:, None] * (2.05 + 0.35 * normal(pages, H, P // G, D)).clamp(0.5, 4)
    s2 = ((hi - lo) / 3).to(dtype)
    s4 = ((hi - lo) / 15).to(dtype)
    boosted = torch.zeros(pages, H, D, dtype=torch.bool, device=dev).scatter_(2, idx, True)
    scale = torch.where(boosted[:, :, None], s4 * 4, s2)
    c = np.arange(D)
    s, r, qd, f = c >> 4, (c >> 3) & 1, (c >> 1) & 3, c & 1
    pos = torch.from_numpy(32 * (s >> 1) + 8 * qd + 4 * (s & 1) + 2 * r + f).to(dev)
    meta = torch.empty_like(scale)
    meta[..., pos] = scale
    put("k_scale", meta)
    meta[..., pos] = lo.to(dtype)
    put("k_zero", meta)
    put("kb_scale", torch.gather(s4, 3, idx[:, :, None].expand(-1, -1, P // G, -1)))
    put("boost_idx", idx.to(torch.uint8))
    put("k_codes", codes(P * D // 16))
    put("kb_codes", bits(P * k // 16))
    put("v_codes", codes(P * D // 16))
    top, low = 2.6 + 0.3 * normal(pages, H, P), -2.6 + 0.3 * normal(pages, H, P)
    put("v_scale", ((top - low) / 3).to(dtype))
    put("v_zero", low.to(dtype))
    return pool, width


def prepare(c, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    B, H, gq, P, k, N, T = c["batch"], c["kv_heads"], c["group"], c["page"], c["boost"], c["pages"], c.get("draft", 1)
    dt = DTYPES[c["dtype"]]
    pages, window, drafts, depth = _lengths(c)

    def ints(x):
        return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=dev)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    s = dict(case=c, num_pages=ints(pages), res_len=ints(window))
    total = int(pages.sum()) + 3
    if c["op"] == "append":
        total, width = 0, torch.exp(normal(H, D))
    else:
        s["pool"], width = _make_pool(g, total, H, P, k, dt, dev)
        order = torch.rand(total, generator=g, device=dev).argsort().to(torch.int32)
        table = torch.full((B, N), -1, dtype=torch.int32, device=dev)
        used = torch.arange(N, device=dev)[None] < s["num_pages"][:, None]
        table[used] = order[: int(pages.sum())]
        s["page_table"] = table
    if c["op"] != "select":
        s["res_k"] = (normal(B, H, P, D) * width[:, None]).to(dt)
        s["res_v"] = normal(B, H, P, D).to(dt)
    if c["op"] in ("tree", "append"):
        s["k_draft"] = (normal(B, T, H, D) * width).to(dt)
        s["v_draft"] = normal(B, T, H, D).to(dt)
    r = np.random.RandomState(seed % (1 << 31))
    if c["op"] == "tree":
        s["q"] = normal(B, T, H * gq, D).to(dt)
        sees = np.zeros((B, T, T), bool)
        for i in range(T):  # a node sees itself and its ancestors
            parent = np.full(B, i - 1) if c["chain"] else r.randint(max(0, i - 6), max(1, i), B)
            if i:
                sees[:, i] = sees[np.arange(B), parent]
            sees[:, i, i] = True
        W = (T + 31) // 32
        packed = np.zeros((B, T, W), np.uint32)
        for j in range(T):
            packed[:, :, j // 32] |= sees[:, :, j].astype(np.uint32) << np.uint32(j % 32)
        s["mask"] = torch.from_numpy(packed.view(np.int32)).to(dev)
        s["draft_len"] = ints(drafts)
        s["out"] = torch.zeros(B, T, H * gq, D, device=dev)
    elif c["op"] == "append":
        path = np.full((B, T), -1)
        for b in range(B):
            path[b, : depth[b]] = np.sort(r.choice(drafts[b], depth[b], replace=False))
        s["path"], s["n_path"] = ints(path), ints(depth)
        s["taken"], s["start_len"] = ints(np.zeros(B)), ints(window)
    else:
        s["q"] = normal(B, H * gq, D).to(dt)
        if c["op"] == "sparse":
            n = np.minimum(pages, c["select"])
            sel = np.full((B, H, c["select"]), -1)
            for b in range(B):
                for h in range(H):
                    sel[b, h, : n[b]] = np.sort(r.choice(pages[b], n[b], replace=False)) if n[b] else 0
            s["sel"], s["n_sel"] = ints(sel), ints(n)
            s["out"] = torch.zeros(B, H * gq, D, device=dev)
        else:
            s["sel"] = torch.zeros(B, H, c["select"], dtype=torch.int32, device=dev)
            s["n_sel"] = torch.zeros(B, dtype=torch.int32, device=dev)
    if own:  # the handle and the scratch that a program keeps
        from bit_mixed_precision_channel_b200 import binding as kb

        cfg = kb.Config(num_q_heads=H * gq, num_kv_heads=H, page_tokens=P, num_boost=k, dtype=kb.BF16 if dt == torch.bfloat16 else kb.F16)
        size = kb.decode_workspace_bytes(cfg, B, N) if c["op"] == "sparse" else kb.tree_workspace_bytes(cfg, B, T) if c["op"] == "tree" else 0
        s["cfg"], s["workspace"] = cfg, torch.zeros(max(size, 256), dtype=torch.uint8, device=dev)
        s["err"] = torch.zeros(1, dtype=torch.int32, device=dev)
    return s


# ---------------------------------------------------------------- the plain forms


def _section(rec, c, name, as_type):
    a, b = _layout(c["page"], c["boost"])[0][name]
    return rec[..., a:b].contiguous().view(as_type)


def _fields(words):
    """The 16 codes of each word in element order: element 8a + 2b + f sits at bit 8b + 4f + 2a."""
    e = torch.arange(16, device=words.device, dtype=torch.int32)
    shift = 8 * ((e >> 1) & 3) + 4 * (e & 1) + 2 * (e >> 3)
    return (words[..., None] >> shift) & 3


def _key_rows(rec, c):
    """Dequantized keys [..., P, D] of records [..., bytes], in 32 bits."""
    P, k, dt, lead = c["page"], c["boost"], DTYPES[c["dtype"]], rec.shape[:-1]
    code = _fields(_section(rec, c, "k_codes", torch.int32)).reshape(*lead, P // G, G, 4, 8, 2, 2)  # qd, s, r, f
    sc = _section(rec, c, "k_scale", dt).reshape(*lead, P // G, 4, 4, 2, 2, 2).float()  # s >> 1, qd, s & 1, r, f
    ze = _section(rec, c, "k_zero", dt).reshape(*lead, P // G, 4, 4, 2, 2, 2).float()
    n = len(lead)
    order = list(range(n + 1)) + [n + 1, n + 3, n + 4, n + 2, n + 5]  # s >> 1, s & 1, r, qd, f: the natural order
    sc, ze = sc.permute(order).reshape(*lead, P // G, 1, D), ze.permute(order).reshape(*lead, P // G, 1, D)
    code = code.permute(*range(n + 2), n + 3, n + 4, n + 2, n + 5).reshape(*lead, P // G, G, D)
    x = code.float() * sc + ze
    if k:
        low = _fields(_section(rec, c, "kb_codes", torch.int32)).reshape(*lead, P // G, G, 4, k // 16, 2, 2)
        low = low.permute(*range(n + 2), n + 3, n + 4, n + 2, n + 5).reshape(*lead, P // G, G, k)
        sb = _section(rec, c, "kb_scale", dt).reshape(*lead, P // G, 1, k).float()
        idx = _section(rec, c, "boost_idx", torch.uint8).long().reshape(*lead, 1, 1, k).expand(low.shape)
        x.scatter_add_(-1, idx, low.float() * sb)
    return x.reshape(*lead, P, D)


def _value_rows(rec, c):
    """Dequantized values [..., P, D] of records [..., bytes], in 32 bits."""
    P, dt, lead = c["page"], DTYPES[c["dtype"]], rec.shape[:-1]
    n = len(lead)
    # word ((2g + (m >> 2)) * 32 + 4w + q) * 4 + (m & 3), element 8a + 2(2u + v) + f: token 32g + 16a + 8u + 2q + f, channel 16m + 8v + w
    code = _fields(_section(rec, c, "v_codes", torch.int32)).reshape(*lead, P // G, 2, 8, 4, 4, 2, 2, 2, 2)  # g, m>>2, w, q, m&3, a, u, v, f
    at = [n + i for i in (0, 5, 6, 3, 8, 1, 4, 7, 2)]  # g, a, u, q, f, m >> 2, m & 3, v, w
    code = code.permute(*range(n), *at).reshape(*lead, P, D)

    def per_token(name):  # token 32g + 8u + w at 32g + 4w + u
        x = _section(rec, c, name, dt).float().reshape(*lead, P // G, 8, 4)
        return x.transpose(-1, -2).reshape(*lead, P, 1)

    return code.float() * per_token("v_scale") + per_token("v_zero")


def _attend(q, K, V, sees):
    """softmax(q K^T / sqrt(D)) V over the keys that are seen; zero where none is. q [B][H][R][D], sees bool [B][1][R or 1][N]."""
    logit = torch.matmul(q.float(), K.transpose(-1, -2)) / math.sqrt(D)
    logit = logit.masked_fill_(~sees, float("-inf"))
    top = logit.amax(-1, keepdim=True)
    p = torch.exp(logit - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, V) / torch.where(total == 0, torch.ones_like(total), total)


def _select(s):
    c = s["case"]
    B, H, gq, P, k, N, n = c["batch"], c["kv_heads"], c["group"], c["page"], c["boost"], c["pages"], c["select"]
    dt = DTYPES[c["dtype"]]
    at = _layout(P, k)[0]
    rec = s["pool"][:, :, at["k_scale"][0]:]  # scales, zeros and boosted channels
    off = at["k_scale"][0]
    rec = rec[s["page_table"].clamp(min=0).long()].transpose(1, 2)  # [B][H][N][bytes]

    def part(name, as_type):
        a, b = at[name]
        return rec[..., a - off:b - off].contiguous().view(as_type)

    q = s["q"].double().reshape(B, H, gq, D)
    pos, neg = q.clamp(min=0).sum(2), q.clamp(max=0).sum(2)  # [B][H][D]
    ch = torch.arange(D, device=q.device)
    stored = (32 * (ch >> 5) + 8 * ((ch >> 1) & 3) + 4 * ((ch >> 4) & 1) + 2 * ((ch >> 3) & 1) + (ch & 1))
    sc = part("k_scale", dt).reshape(B, H, N, P // G, D)[..., stored].double()
    ze = part("k_zero", dt).reshape(B, H, N, P // G, D)[..., stored].double()
    score = (3 * sc * pos[:, :, None, None] + ze * (pos + neg)[:, :, None, None]).sum(-1)
    if k:
        idx = part("boost_idx", torch.uint8).long()  # [B][H][N][k]
        sb = part("kb_scale", dt).reshape(B, H, N, P // G, k).double()
        gathered = torch.gather(pos[:, :, None].expand(B, H, N, D), 3, idx)
        score = score + (3 * sb * gathered[:, :, :, None]).sum(-1)
    score = score.amax(-1)  # [B][H][N]
    slot = torch.arange(N, device=q.device)[None, None]
    have = s["num_pages"][:, None, None]
    score = torch.where((slot < c["first"]) | (slot >= have - c["recent"]), torch.full_like(score, float("inf")), score)
    score = torch.where(slot >= have, torch.full_like(score, float("-inf")), score)
    best = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :n]
    n_sel = s["num_pages"].clamp(max=n)
    taken = torch.arange(n, device=q.device)[None, None] < n_sel[:, None, None]
    best = torch.where(taken, best, torch.full_like(best, N)).sort(-1).values
    return {"sel": torch.where(taken, best, torch.full_like(best, -1)).to(torch.int32), "n_sel": n_sel}


def _sparse(s):
    c = s["case"]
    B, H, gq, P, n = c["batch"], c["kv_heads"], c["group"], c["page"], c["select"]
    have = torch.arange(n, device=s["q"].device) < s["n_sel"][:, None]
    page = torch.gather(s["page_table"][:, None].expand(B, H, -1), 2, s["sel"].clamp(min=0).long()).clamp(min=0).long()
    rec = s["pool"][page, torch.arange(H, device=page.device)[None, :, None]]
    K = torch.cat([_key_rows(rec, c).reshape(B, H, n * P, D), s["res_k"].float()], 2)
    V = torch.cat([_value_rows(rec, c).reshape(B, H, n * P, D), s["res_v"].float()], 2)
    window = torch.arange(P, device=page.device) < s["res_len"][:, None]
    sees = torch.cat([have.repeat_interleave(P, 1), window], 1)
    return _attend(s["q"].reshape(B, H, gq, D), K, V, sees[:, None, None]).reshape(B, H * gq, D)


def _tree(s):
    c = s["case"]
    B, H, gq, P, N, T = c["batch"], c["kv_heads"], c["group"], c["page"], c["pages"], c["draft"]
    dev = s["q"].device
    rec = s["pool"][s["page_table"].clamp(min=0).long()].transpose(1, 2)
    K = torch.cat([_key_rows(rec, c).reshape(B, H, N * P, D), s["res_k"].float(), s["k_draft"].transpose(1, 2).float()], 2)
    V = torch.cat([_value_rows(rec, c).reshape(B, H, N * P, D), s["res_v"].float(), s["v_draft"].transpose(1, 2).float()], 2)
    have = (torch.arange(N, device=dev) < s["num_pages"][:, None]).repeat_interleave(P, 1)
    window = torch.arange(P, device=dev) < s["res_len"][:, None]
    node = torch.arange(T, device=dev)
    there = node < s["draft_len"][:, None]
    seen = ((s["mask"][:, :, node >> 5] >> (node & 31).to(torch.int32)) & 1).bool() & there[:, None]
    sees = torch.cat([torch.cat([have, window], 1)[:, None].expand(B, T, -1), seen], 2)
    sees = sees.repeat_interleave(gq, 1)[:, None]
    q = s["q"].reshape(B, T, H, gq, D).transpose(1, 2).reshape(B, H, T * gq, D)
    o = _attend(q, K, V, sees).reshape(B, H, T, gq, D).transpose(1, 2).reshape(B, T, H * gq, D)
    s["out"].copy_(torch.where(there[:, :, None, None], o, s["out"]))
    return s["out"]


def _append(s):
    c = s["case"]
    P, T = c["page"], c["draft"]
    dev = s["res_k"].device
    todo = torch.minimum(s["n_path"] - s["taken"], P - s["res_len"])
    i = (torch.arange(P, device=dev) - s["res_len"][:, None])  # step of the path that lands on each row of the window
    step = i + s["taken"][:, None]
    fresh = (i >= 0) & (i < todo[:, None])
    node = torch.gather(s["path"], 1, step.clamp(0, T - 1).long()).clamp(0, T - 1).long()
    rows = torch.arange(node.shape[0], device=dev)[:, None]
    for_heads = fresh[:, None, :, None]
    s["res_k"].copy_(torch.where(for_heads, s["k_draft"][rows, node].transpose(1, 2), s["res_k"]))
    s["res_v"].copy_(torch.where(for_heads, s["v_draft"][rows, node].transpose(1, 2), s["res_v"]))
    s["res_len"] += todo
    s["taken"] += todo


def run(s):
    c = s["case"]
    if c["op"] == "append":
        s["res_len"].copy_(s["start_len"])
        s["taken"].zero_()
    if own:
        from bit_mixed_precision_channel_b200 import binding as kb

        if c["op"] == "select":
            kb.select_pages(s["cfg"], s["pool"], s["q"], s["page_table"], s["num_pages"], s["sel"], s["n_sel"],
                            n_first=c["first"], n_recent=c["recent"], err=s["err"])
        elif c["op"] == "sparse":
            kb.decode_attention_sparse(s["cfg"], s["pool"], s["q"], s["page_table"], s["num_pages"], s["sel"], s["n_sel"], s["res_k"],
                                       s["res_v"], s["res_len"], s["out"], s["workspace"], err=s["err"])
        elif c["op"] == "tree":
            kb.tree_attention(s["cfg"], s["pool"], s["q"], s["page_table"], s["num_pages"], s["res_k"], s["res_v"], s["res_len"],
                              s["k_draft"], s["v_draft"], s["mask"], s["draft_len"], s["out"], s["workspace"], err=s["err"])
        else:
            kb.append_path(s["cfg"], s["k_draft"], s["v_draft"], s["path"], s["n_path"], s["taken"], s["res_k"], s["res_v"],
                           s["res_len"], err=s["err"])
    elif c["op"] == "select":
        return _select(s)
    elif c["op"] == "sparse":
        return _sparse(s)
    elif c["op"] == "tree":
        return _tree(s)
    else:
        _append(s)
    if c["op"] == "select":
        return {"sel": s["sel"], "n_sel": s["n_sel"]}
    if c["op"] == "append":
        return {"res_k": s["res_k"], "res_v": s["res_v"], "res_len": s["res_len"], "taken": s["taken"]}
    return s["out"]


# ---------------------------------------------------------------- 64 bits


def _bit(e):
    return 8 * ((e >> 1) & 3) + 4 * (e & 1) + 2 * (e >> 3)


def _exact_rows(rec, c):
    """Keys and values [n][P][D] of records [n][bytes] in 64 bits, element by element from the places of its codes."""
    P, k, dt = c["page"], c["boost"], DTYPES[c["dtype"]]
    at, dev, n = _layout(P, k)[0], rec.device, rec.shape[0]

    def load(name, as_type):
        return rec[:, at[name][0]:at[name][1]].contiguous().view(as_type)

    def code(words, index, e):
        return ((words[:, torch.from_numpy(index).to(dev)] >> torch.from_numpy(_bit(e).astype(np.int32)).to(dev)) & 3).double()

    t, ch = np.meshgrid(np.arange(P), np.arange(D), indexing="ij")
    s, r, q, f = ch >> 4, (ch >> 3) & 1, (ch >> 1) & 3, ch & 1
    p = 32 * q + 4 * s + 2 * r + f
    group = t // G
    meta = torch.from_numpy(group * D + 32 * (s >> 1) + 8 * q + 4 * (s & 1) + 2 * r + f).to(dev)
    keys = code(load("k_codes", torch.int32), t * (D // 16) + p // 16, p % 16) * load("k_scale", dt).double()[:, meta]
    keys += load("k_zero", dt).double()[:, meta]
    if k:
        t, j = np.meshgrid(np.arange(P), np.arange(k), indexing="ij")
        s, r, q, f = j >> 4, (j >> 3) & 1, (j >> 1) & 3, j & 1
        p = 4 * (k // 16) * q + 4 * s + 2 * r + f
        low = code(load("kb_codes", torch.int32), t * (k // 16) + p // 16, p % 16)
        low = low * load("kb_scale", dt).double()[:, torch.from_numpy(t // G * k + j).to(dev)]
        keys.scatter_add_(2, load("boost_idx", torch.uint8).long()[:, None].expand(n, P, k), low)
    t, ch = np.meshgrid(np.arange(P), np.arange(D), indexing="ij")
    g, a, u, q, f = t >> 5, (t >> 4) & 1, (t >> 3) & 1, (t >> 1) & 3, t & 1
    m, v, w = ch >> 4, (ch >> 3) & 1, ch & 7
    vals = code(load("v_codes", torch.int32), ((2 * g + (m >> 2)) * 32 + 4 * w + q) * 4 + (m & 3), 8 * a + 2 * (2 * u + v) + f)
    tok = np.arange(P)
    place = torch.from_numpy((tok & ~31) + 4 * (tok & 7) + ((tok >> 3) & 3)).to(dev)
    vals = vals * load("v_scale", dt).double()[:, place, None] + load("v_zero", dt).double()[:, place, None]
    return keys, vals


def exact(c, seed):
    if c["op"] in ("select", "append"):
        return None  # places and copies: nothing is computed that could be rounded
    s = prepare(c, seed)
    B, H, gq, P = c["batch"], c["kv_heads"], c["group"], c["page"]
    T = c.get("draft", 1)
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    num, window = s["num_pages"].tolist(), s["res_len"].tolist()
    drafts = s["draft_len"].tolist() if c["op"] == "tree" else [1] * B
    table = s["page_table"].long()
    for b in range(B):
        for h in range(H):
            slots = s["sel"][b, h, : int(s["n_sel"][b])].long() if c["op"] == "sparse" else torch.arange(num[b], device="cuda")
            K, V = _exact_rows(s["pool"][table[b, slots], h], c)
            parts_k, parts_v = [K.reshape(-1, D), s["res_k"][b, h, : window[b]].double()], [V.reshape(-1, D), s["res_v"][b, h, : window[b]].double()]
            heads = slice(h * gq, (h + 1) * gq)
            t = drafts[b]
            if c["op"] == "tree":
                parts_k.append(s["k_draft"][b, :t, h].double())
                parts_v.append(s["v_draft"][b, :t, h].double())
                q = s["q"][b, :t, heads].double()
            else:
                q = s["q"][b, None, heads].double()
            K, V = torch.cat(parts_k), torch.cat(parts_v)
            if not K.shape[0]:
                continue
            z = torch.einsum("thd,nd->thn", q, K) / math.sqrt(D)
            if c["op"] == "tree":
                bits = s["mask"][b, :t].cpu().numpy().view(np.uint32)
                seen = np.stack([(bits[:, j // 32] >> np.uint32(j % 32)) & 1 for j in range(t)], 1).astype(bool)
                z[:, :, K.shape[0] - t:][~torch.from_numpy(seen).to("cuda")[:, None].expand(t, gq, t)] = float("-inf")
            o = torch.einsum("thn,nd->thd", torch.softmax(z, -1), V)
            if c["op"] == "tree":
                out[b, :t, heads] = o
            else:
                out[b, heads] = o[0]
    return out
