"""Device buffers and host bookkeeping of one layer's paged 2-bit KV cache.

PagedKVCache owns the caller-side state the C ABI expects (page pool, page table,
page counts, residual windows, decode workspace, device error word) plus a host free
list of physical pages.  Its methods only allocate, track page ids and call the
library; every transformation of the data happens in the library's kernels.

The decode step follows the pipeline of the KIVI article (section 3: recent tokens
kept in full precision, streaming append) with Kitty's paged layout: append the new
token to the residual window, flush the window into a fresh page when it holds a
whole page, then attend over pages + window.
"""
from __future__ import annotations

import contextlib

import torch

from . import binding as kb


class PagedKVCache:
    def __init__(self, cfg: kb.Config, batch: int, max_pages: int, pool_pages: int,
                 device: str | torch.device = "cuda", page_order=None):
        self.cfg = cfg
        self.batch = batch
        self.max_pages = max_pages
        self.pool_pages = pool_pages
        self.device = torch.device(device)
        H, P, D = cfg.num_kv_heads, cfg.page_tokens, cfg.head_dim
        dt = kb.torch_dtype(cfg.dtype)
        self.record_bytes = kb.page_bytes(cfg)
        self.pool = torch.zeros(pool_pages * H * self.record_bytes, dtype=torch.uint8, device=self.device)
        self.page_table = torch.full((batch, max_pages), -1, dtype=torch.int32, device=self.device)
        self.num_pages = torch.zeros(batch, dtype=torch.int32, device=self.device)
        self.res_len = torch.zeros(batch, dtype=torch.int32, device=self.device)
        self.res_k = torch.zeros(batch, H, P, D, dtype=dt, device=self.device)
        self.res_v = torch.zeros(batch, H, P, D, dtype=dt, device=self.device)
        ws = kb.decode_workspace_bytes(cfg, batch, max_pages)
        self.workspace = torch.zeros(max(ws, 256), dtype=torch.uint8, device=self.device)
        self.err = torch.zeros(1, dtype=torch.int32, device=self.device)
        self.new_page = torch.full((batch,), -1, dtype=torch.int32, device=self.device)
        self.counters = torch.zeros(batch, dtype=torch.int32, device=self.device)  # append_flush arrivals
        # speculative decoding: the last choice of pages and the buffers of every size asked for, the
        # accepted lengths, the tree's scratch.  Captured graphs may hold these buffers: none is replaced.
        self.sel = self.n_sel = None
        self.choices = {}
        self.grown = 0         # calls that may have appended pages
        self.grown_at_sel = 0  # ... when the last choice was made
        self.n_path = torch.zeros(batch, dtype=torch.int32, device=self.device)
        self.taken = torch.zeros(batch, dtype=torch.int32, device=self.device)
        self.tree_workspace = None
        # host mirrors used to hand out pages
        order = list(range(pool_pages)) if page_order is None else [int(x) for x in page_order]
        if sorted(order) != list(range(pool_pages)):
            raise ValueError("page_order must be a permutation of range(pool_pages)")
        self.free = order[::-1]  # pop() hands out order[0] first
        self.host_pages = [[] for _ in range(batch)]
        self.host_res_len = [0] * batch
        self.host_new_page = [-1] * batch  # what the device new_page buffer holds

    # ---------------------------------------------------------------- allocation
    def take_pages(self, n: int) -> list:
        if n > len(self.free):
            raise RuntimeError("page pool exhausted")
        return [self.free.pop() for _ in range(n)]

    # ---------------------------------------------------------------- prefill
    def prefill(self, b: int, k: torch.Tensor, v: torch.Tensor, stream=None):
        """k, v: [L][Hkv][D] on the device.  floor(L/P) pages are quantized, the
        remaining L mod P tokens are copied into the residual window."""
        P = self.cfg.page_tokens
        L = k.shape[0]
        n_full = L // P
        if len(self.host_pages[b]) + n_full > self.max_pages:
            raise RuntimeError("page table full")
        pages = self.take_pages(n_full)
        self.grown += bool(n_full)
        if n_full:
            dst = torch.tensor(pages, dtype=torch.int32, device=self.device)
            kb.quantize_pages(self.cfg, kb.Source.token_major(k, self.cfg), kb.Source.token_major(v, self.cfg),
                              dst, self.pool, self.err, stream)
            start = len(self.host_pages[b])
            self.page_table[b, start:start + n_full] = dst
        self.host_pages[b] += pages
        self.num_pages[b] = len(self.host_pages[b])
        r = L - n_full * P
        if r:
            self.res_k[b, :, :r] = k[n_full * P:].transpose(0, 1)
            self.res_v[b, :, :r] = v[n_full * P:].transpose(0, 1)
        self.res_len[b] = r
        self.host_res_len[b] = r

    def prefill_batch(self, k: torch.Tensor, v: torch.Tensor, stream=None):
        """All sequences at once with the same prompt length L (a multiple of P):
        k, v: [B][L][Hkv][D] contiguous.  One quantize launch for every page."""
        B, L = k.shape[0], k.shape[1]
        P = self.cfg.page_tokens
        assert B == self.batch and L % P == 0 and k.is_contiguous() and v.is_contiguous()
        n = L // P
        pages = self.take_pages(B * n)
        self.grown += 1
        dst = torch.tensor(pages, dtype=torch.int32, device=self.device)
        flat_k, flat_v = k.view(B * L, *k.shape[2:]), v.view(B * L, *v.shape[2:])
        kb.quantize_pages(self.cfg, kb.Source.token_major(flat_k, self.cfg), kb.Source.token_major(flat_v, self.cfg),
                          dst, self.pool, self.err, stream)
        self.page_table[:, :n] = dst.view(B, n)
        self.num_pages.fill_(n)
        self.res_len.zero_()
        for b in range(B):
            self.host_pages[b] += pages[b * n:(b + 1) * n]
            self.host_res_len[b] = 0
        return dst

    # ---------------------------------------------------------------- decode step
    def reserve_flush_pages(self) -> list:
        """Before a step: a fresh page for every sequence whose window will be full
        after this step's append; returns the sequences that will flush.  The device
        buffer is only written when its contents change."""
        P = self.cfg.page_tokens
        flushing = [b for b in range(self.batch) if self.host_res_len[b] + 1 == P]
        ids = [-1] * self.batch
        for b in flushing:
            ids[b] = self.take_pages(1)[0]
        if ids != self.host_new_page:
            self.new_page.copy_(torch.tensor(ids, dtype=torch.int32), non_blocking=False)
            self.host_new_page = ids
        return flushing

    def commit_host(self, flushing: list):
        P = self.cfg.page_tokens
        for b in range(self.batch):
            self.host_res_len[b] += 1
        self.grown += bool(flushing)
        for b in flushing:
            self.host_pages[b].append(self.host_new_page[b])
            self.host_res_len[b] = 0
        assert all(r < P for r in self.host_res_len)

    def append(self, k_new, v_new, stream=None):
        kb.append_token(self.cfg, k_new, v_new, self.res_k, self.res_v, self.res_len, self.err, stream)

    def flush(self, stream=None):
        self.grown += max(self.host_new_page, default=-1) >= 0
        kb.flush_residual(self.cfg, self.res_k, self.res_v, self.res_len, self.new_page, self.page_table,
                          self.num_pages, self.pool, self.err, stream)

    def append_flush(self, k_new, v_new, stream=None):
        """append then flush, in one launch."""
        self.grown += max(self.host_new_page, default=-1) >= 0
        kb.append_flush(self.cfg, k_new, v_new, self.res_k, self.res_v, self.res_len, self.new_page,
                        self.page_table, self.num_pages, self.pool, self.counters, self.err, stream)

    def attend(self, q, out, sm_scale=None, stream=None):
        kb.decode_attention(self.cfg, self.pool, q, self.page_table, self.num_pages, self.res_k, self.res_v,
                            self.res_len, out, self.workspace, sm_scale, self.err, stream)

    def step(self, q, k_new, v_new, out, sm_scale=None, stream=None):
        """One decode step: append, flush full windows, attend.  The host tracks every
        window's length, so the flush (quantize of the full windows and the page-table
        commit) is launched only on steps where some window fills: once every P steps
        per sequence.  Append, flush and commit stay separate launches: the single
        append_flush launch needs 41 KB of shared memory per CTA and, chained before the
        decode, delays the decode's CTAs more than it saves (measured on B200: 40.1 vs
        34.3 us per layer of the 8B-shaped 32-layer step)."""
        flushing = self.reserve_flush_pages()
        self.append(k_new, v_new, stream)
        if flushing:
            self.flush(stream)
        self.attend(q, out, sm_scale, stream)
        self.commit_host(flushing)

    # ---------------------------------------------------------------- speculative decoding
    # A round attends from a drafted tree to the whole cache with `verify` and keeps what was
    # accepted with `accept`; the drafted tokens' keys and values stay outside the cache until
    # then.  `select` and `attend_few` are a draft step's attention over few pages and the window:
    # they do not see tokens drafted before, which a drafter that needs them keeps itself.

    def select(self, q, n_select: int, n_first: int = 1, n_recent: int = 1, stream=None):
        """Chooses the n_select pages of every (sequence, KV head) whose stored key ranges
        allow q the largest logits (the first n_first and the last n_recent always): fills
        and returns self.sel [B][Hkv][n_select] and self.n_sel [B].  A choice holds until a
        window is flushed: the page then holds tokens that the choice does not list, so
        attend_few asks for a new one."""
        if n_select not in self.choices:
            if n_select < 1:
                raise ValueError(f"n_select is {n_select}: at least one page")
            with self._on(stream):
                self.choices[n_select] = (
                    torch.empty(self.batch, self.cfg.num_kv_heads, n_select, dtype=torch.int32, device=self.device),
                    torch.empty(self.batch, dtype=torch.int32, device=self.device))
        sel, n_sel = self.choices[n_select]
        kb.select_pages(self.cfg, self.pool, q, self.page_table, self.num_pages, sel, n_sel, n_first, n_recent, self.err,
                        stream)
        self.sel, self.n_sel = sel, n_sel
        self.grown_at_sel = self.grown
        return sel, n_sel

    def attend_few(self, q, out, sm_scale=None, stream=None):
        """Decode attention over the pages of the last `select` and the window.  Refused once
        pages were appended since (a graph that holds this call has to hold its `select` too,
        if it is replayed across a flush)."""
        if self.sel is None:
            raise RuntimeError("attend_few needs a choice of pages: call select first")
        if self.grown_at_sel != self.grown:
            raise RuntimeError("pages were appended since the last choice, which leaves their tokens out: call select again")
        kb.decode_attention_sparse(self.cfg, self.pool, q, self.page_table, self.num_pages, self.sel, self.n_sel,
                                   self.res_k, self.res_v, self.res_len, out, self.workspace, sm_scale, self.err, stream)

    def verify(self, q, k_draft, v_draft, mask, draft_len, out, sm_scale=None, stream=None):
        """Attention from the drafted tokens (q [B][T][Hq][D]) to the whole cache, the window and
        the drafted tokens their mask names; see tree_attention.  The cache is not changed.  The
        first call allocates the scratch (20 MB for every tree), so it cannot be one that is captured.
        Layers that are not verified at once can share one: set tree_workspace to the first one's."""
        if self.tree_workspace is None:
            need = max(kb.tree_workspace_bytes(self.cfg, self.batch, T) for T in (1, 2, 4, 8, kb.MAX_DRAFT))
            with self._on(stream):
                if self.device.type == "cuda" and torch.cuda.is_current_stream_capturing():
                    raise RuntimeError("verify allocates its scratch in its first call: call it once before a capture")
                self.tree_workspace = torch.zeros(need, dtype=torch.uint8, device=self.device)
        kb.tree_attention(self.cfg, self.pool, q, self.page_table, self.num_pages, self.res_k, self.res_v, self.res_len,
                          k_draft, v_draft, mask, draft_len, out, self.tree_workspace, sm_scale, self.err, stream)

    def accept(self, k_draft, v_draft, path, n_path, stream=None):
        """Appends the accepted tokens path[b][:n_path[b]] (path: int32 [B][T] on the device,
        n_path: integers on the host) of k_draft, v_draft [B][T][Hkv][D] to every sequence and
        flushes the windows they fill.  Nothing is changed if pages run out.  The lengths and the
        pages of a flush are copied from the host, which waits for them: not for a capture."""
        P, T = self.cfg.page_tokens, path.shape[1]
        left = [int(n) for n in n_path]
        if len(left) != self.batch or any(n < 0 or n > T for n in left):
            raise ValueError(f"n_path: {self.batch} lengths from 0 to {T}, not {left}")
        fills = [(r + n) // P for r, n in zip(self.host_res_len, left)]
        if any(len(h) + f > self.max_pages for h, f in zip(self.host_pages, fills)):
            raise RuntimeError("page table full")
        if sum(fills) > len(self.free):
            raise RuntimeError("page pool exhausted")
        with self._on(stream):
            self.n_path.copy_(torch.tensor(left, dtype=torch.int32))
            self.taken.zero_()
            while True:
                kb.append_path(self.cfg, k_draft, v_draft, path, self.n_path, self.taken, self.res_k, self.res_v,
                               self.res_len, self.err, stream)
                ids = [-1] * self.batch
                for b in range(self.batch):
                    t = min(left[b], P - self.host_res_len[b])
                    left[b] -= t
                    self.host_res_len[b] += t
                    if self.host_res_len[b] == P:
                        ids[b] = self.take_pages(1)[0]
                        self.host_pages[b].append(ids[b])
                        self.host_res_len[b] = 0
                if any(i >= 0 for i in ids):
                    self.new_page.copy_(torch.tensor(ids, dtype=torch.int32))
                    self.host_new_page = ids
                    self.flush(stream)
                if not any(left):
                    break

    def _on(self, stream):
        return torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext()

    def record(self, page: int, head: int) -> torch.Tensor:
        """Bytes of record (page, head) (a view into the pool)."""
        H, R = self.cfg.num_kv_heads, self.record_bytes
        off = (page * H + head) * R
        return self.pool[off:off + R]

    def check_errors(self) -> int:
        return int(self.err.item())
