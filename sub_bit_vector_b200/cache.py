"""Host-side plumbing for one layer's LoopVQ decode cache on the device.

Allocates the pools, windows, codebooks, queries, outputs and workspace of
a decode batch as torch device tensors, copies per-request host arrays into
them at the offsets the cache layout prescribes, and calls the library.  It
does no arithmetic of the method: codes, windows and codebooks are inputs, and
every step of encode and decode runs in libloopvq's kernels.
"""
from __future__ import annotations

import numpy as np
import torch

from . import loopvq as L


def _round_up(x: int, m: int) -> int:
    return (x + m - 1) // m * m


class DecodeCache:
    """Device buffers of one layer (K and V) for a batch of decode requests.

    ``ctx_lens`` are the per-request context lengths (current token
    included).  Bodies are laid out back to back in the index pools at
    32-token-aligned offsets; windows back to back in the window pools.
    """

    def __init__(self, *, n_loop, tc, n_heads_kv, head_dim, group_elems, ctx_lens, n_sink=64, n_recent=256,
                 page=8, n_codes=256, n_heads_q=None, cb_dtype=torch.bfloat16, q_dtype=torch.bfloat16,
                 out_dtype=torch.float32, device="cuda", max_ctx_len=None, pool_slack_tokens=0,
                 static_inputs=False):
        self.device = torch.device(device)
        self.T, self.Tc, self.H, self.D, self.G = n_loop, tc, n_heads_kv, head_dim, group_elems
        self.Hq = n_heads_q or n_heads_kv
        self.W = group_elems // tc
        self.J = head_dim // self.W
        self.NB = n_loop // tc
        self.C = n_codes
        self.n_sink, self.n_recent, self.page = n_sink, n_recent, page
        self.cb_dtype = cb_dtype
        self.desc = L.make_desc(n_loop, tc, n_heads_kv, head_dim, group_elems, n_codes, self.Hq,
                                L.LOOPVQ_BF16 if cb_dtype == torch.bfloat16 else L.LOOPVQ_F32)
        self.ctx_lens = [int(c) for c in ctx_lens]
        self.batch = len(self.ctx_lens)
        self.splits = [L.loopvq_ctx_split(c, n_sink, n_recent, page) for c in self.ctx_lens]
        body_off, win_off = [], []
        b = w = 0
        for (s, body, rec) in self.splits:
            body_off.append(b)
            win_off.append(w)
            b += _round_up(body, 32)
            w += s + rec
        self.body_off = body_off
        self.win_off = win_off
        self.body_pool_tokens = max(32, _round_up(b + pool_slack_tokens, 32))
        self.win_pool_tokens = max(1, w)
        self.max_ctx_len = max(self.ctx_lens) if max_ctx_len is None else max_ctx_len
        dev = self.device
        pool_bytes = L.loopvq_index_pool_bytes(self.desc, self.body_pool_tokens)
        self.idxK = torch.zeros(pool_bytes, dtype=torch.uint8, device=dev)
        self.idxV = torch.zeros(pool_bytes, dtype=torch.uint8, device=dev)
        self.winK = torch.zeros((self.T, self.H, self.win_pool_tokens, self.D), dtype=torch.bfloat16, device=dev)
        self.winV = torch.zeros_like(self.winK)
        pb = L.loopvq_codebook_packed_bytes(self.desc)
        self.cbK = torch.zeros(pb, dtype=torch.uint8, device=dev)
        self.cbV = torch.zeros(pb, dtype=torch.uint8, device=dev)
        self.q = torch.zeros((self.batch, self.Hq, self.D), dtype=q_dtype, device=dev)
        self.out = torch.zeros((self.batch, self.Hq, self.D), dtype=out_dtype, device=dev)
        self.lse = torch.zeros((self.batch, self.Hq), dtype=torch.float32, device=dev)
        self.ctx_dev = torch.tensor(self.ctx_lens, dtype=torch.int32, device=dev)
        self.body_off_dev = torch.tensor(body_off, dtype=torch.int64, device=dev)
        self.win_off_dev = torch.tensor(win_off, dtype=torch.int64, device=dev)
        # static_inputs: this cache's layout arrays, index pools and codebooks
        # are not written by kernels that may still run when a decode starts
        self.flags = L.LOOPVQ_LAYOUT_STATIC_INPUTS if static_inputs else 0
        self.layout = self._make_layout(None, None)
        ws = L.loopvq_decode_workspace_bytes(self.desc, self.layout)
        if ws == 0:
            raise ValueError("invalid cache layout")
        self.workspace = torch.zeros(_round_up(ws, 256), dtype=torch.uint8, device=dev)

    def _make_layout(self, new_k, new_v):
        return L.make_layout(self.batch, self.n_sink, self.n_recent, self.page, self.max_ctx_len, self.ctx_dev,
                             self.body_off_dev, self.win_off_dev, self.body_pool_tokens, self.win_pool_tokens,
                             self.flags, new_k=new_k, new_v=new_v)

    # ------------------------------------------------------------ inputs
    def set_codebooks(self, cb_k: np.ndarray, cb_v: np.ndarray) -> None:
        """Canonical codebooks [NB][H][J][C][Tc][W] (host arrays) -> packed."""
        for src, dst in ((cb_k, self.cbK), (cb_v, self.cbV)):
            t = torch.from_numpy(np.ascontiguousarray(src, dtype=np.float32)).to(self.cb_dtype).to(self.device)
            L.loopvq_codebook_pack(self.desc, t, dst)
        torch.cuda.current_stream().synchronize()

    def set_request_codes(self, r: int, codes_k: np.ndarray, codes_v: np.ndarray) -> None:
        """Body codes of request r, [NB][H][n_body][J] uint8 (token-major)."""
        n = self.splits[r][1]
        if codes_k.shape[2] != n or codes_v.shape[2] != n:
            raise ValueError(f"request {r}: expected {n} body tokens")
        if n == 0:
            return
        for kind, src, pool in ((L.LOOPVQ_KEYS, codes_k, self.idxK), (L.LOOPVQ_VALUES, codes_v, self.idxV)):
            t = torch.from_numpy(np.ascontiguousarray(src, dtype=np.uint8)).to(self.device)
            L.loopvq_index_pool_pack(self.desc, kind, t, n, pool, self.body_off[r], self.body_pool_tokens)
            torch.cuda.current_stream().synchronize()

    def set_request_window(self, r: int, win_k: np.ndarray, win_v: np.ndarray) -> None:
        """Window tokens (sink then recent) of request r, [T][H][n_win][D] values
        (rounded to bf16 on upload)."""
        s, _, rec = self.splits[r]
        n = s + rec
        if win_k.shape[2] != n:
            raise ValueError(f"request {r}: expected {n} window tokens")
        o = self.win_off[r]
        self.winK[:, :, o:o + n] = torch.from_numpy(np.ascontiguousarray(win_k, dtype=np.float32)).to(
            self.device, torch.bfloat16)
        self.winV[:, :, o:o + n] = torch.from_numpy(np.ascontiguousarray(win_v, dtype=np.float32)).to(
            self.device, torch.bfloat16)

    def set_queries(self, q: np.ndarray) -> None:
        """Queries [batch][Hq][D] of the loop step about to run."""
        self.q.copy_(torch.from_numpy(np.ascontiguousarray(q, dtype=np.float32)).to(self.device, self.q.dtype))

    # ------------------------------------------------------------ compute
    def decode(self, loop_step: int, softmax_scale: float | None = None, stream=None, new_k=None,
               new_v=None) -> None:
        """Decode attention at loop_step.  new_k/new_v ([batch][H][D] bf16
        device tensors) are the current token's K and V at this step: the
        kernel uses them and stores them in the token's window slot."""
        scale = self.D ** -0.5 if softmax_scale is None else softmax_scale
        layout = self.layout if new_k is None else self._make_layout(new_k, new_v)
        L.loopvq_decode_attn(self.desc, self.cbK, self.cbV, layout, self.idxK, self.idxV, self.winK,
                             self.winV, self.q, loop_step, scale, self.out, self.lse, self.workspace, stream)

    def device_status(self):
        return L.loopvq_read_device_status(self.workspace)

    def clear_status(self) -> None:
        L.loopvq_clear_device_status(self.workspace)

    def unpack_codes(self, r: int, kind: int) -> np.ndarray:
        n = self.splits[r][1]
        out = torch.empty((self.NB, self.H, n, self.J), dtype=torch.uint8, device=self.device)
        if n:
            L.loopvq_index_pool_unpack(self.desc, kind, self.idxK if kind == L.LOOPVQ_KEYS else self.idxV,
                                       self.body_off[r], self.body_pool_tokens, n, out)
        return out.cpu().numpy()

    def algorithmic_bytes(self) -> int:
        """Bytes one decode launch must move: index rows (K and V) of every body
        token, bf16 K and V of every window token, the query and the fp32
        output, summed over requests and query heads' KV streams."""
        idx = sum(b for (_, b, _) in self.splits) * self.H * 2 * self.J
        win = sum(s + r for (s, _, r) in self.splits) * self.H * 2 * self.D * 2
        qo = self.batch * self.Hq * self.D * (self.q.element_size() + self.out.element_size())
        return idx + win + qo


class PagedCache:
    """Incremental serving cache of one layer (K and V) for a batch of requests.

    LoopVQ project page, "Serving in SGLang": a new token's keys and values
    enter the cache in bf16; the ``n_sink`` sink tokens and the recent window
    are kept in bf16; for each ``page`` new tokens the page leaving the recent
    window is coded; decode reads the coded body from the indices.  Here the body lives in fixed-size pages
    of the index pools (``body_page_tokens`` tokens each, taken from a free
    list, listed per request in a page table) and the recent tokens in a ring
    of ``n_recent + page`` slots per request, so nothing is ever moved.

    Per generated token: ``begin_token(r)`` advances request r's length and,
    when its body grows, encodes the page leaving the recent window (one
    ``loopvq_encode`` per K and V, straight from the ring); then, for each
    loop step t, ``decode(t, new_k, new_v)`` attends with the new token's K/V
    written into its ring slot by the decode kernel itself.
    """

    def __init__(self, *, n_loop, tc, n_heads_kv, head_dim, group_elems, batch, max_ctx_len, n_sink=64,
                 n_recent=256, page=8, body_page_tokens=256, n_codes=256, n_heads_q=None,
                 cb_dtype=torch.bfloat16, q_dtype=torch.bfloat16, out_dtype=torch.float32, device="cuda",
                 spare_pages=0):
        if body_page_tokens % 32 or body_page_tokens % page:
            raise ValueError("body_page_tokens must be a multiple of 32 and of page")
        self.device = torch.device(device)
        self.T, self.Tc, self.H, self.D, self.G = n_loop, tc, n_heads_kv, head_dim, group_elems
        self.Hq = n_heads_q or n_heads_kv
        self.W = group_elems // tc
        self.J = head_dim // self.W
        self.NB = n_loop // tc
        self.n_sink, self.n_recent, self.page = n_sink, n_recent, page
        self.bpt = body_page_tokens
        self.ring = n_recent + page
        self.batch = batch
        self.max_ctx_len = max_ctx_len
        self.cb_dtype = cb_dtype
        self.desc = L.make_desc(n_loop, tc, n_heads_kv, head_dim, group_elems, n_codes, self.Hq,
                                L.LOOPVQ_BF16 if cb_dtype == torch.bfloat16 else L.LOOPVQ_F32)
        max_body = L.loopvq_ctx_split(max_ctx_len, n_sink, n_recent, page)[1]
        self.max_pages = max(1, -(-max_body // self.bpt))
        self.n_phys = batch * self.max_pages + spare_pages
        self.body_pool_tokens = self.n_phys * self.bpt
        self.win_stride = n_sink + self.ring
        self.win_pool_tokens = batch * self.win_stride
        dev = self.device
        pool_bytes = L.loopvq_index_pool_bytes(self.desc, self.body_pool_tokens)
        self.idxK = torch.zeros(pool_bytes, dtype=torch.uint8, device=dev)
        self.idxV = torch.zeros(pool_bytes, dtype=torch.uint8, device=dev)
        self.winK = torch.zeros((self.T, self.H, self.win_pool_tokens, self.D), dtype=torch.bfloat16, device=dev)
        self.winV = torch.zeros_like(self.winK)
        pb = L.loopvq_codebook_packed_bytes(self.desc)
        self.cbK = torch.zeros(pb, dtype=torch.uint8, device=dev)
        self.cbV = torch.zeros(pb, dtype=torch.uint8, device=dev)
        self.q = torch.zeros((batch, self.Hq, self.D), dtype=q_dtype, device=dev)
        self.out = torch.zeros((batch, self.Hq, self.D), dtype=out_dtype, device=dev)
        self.lse = torch.zeros((batch, self.Hq), dtype=torch.float32, device=dev)
        # host state
        self.ctx = [0] * batch
        self.head = [0] * batch
        self.pages = [[] for _ in range(batch)]
        self.free = list(range(self.n_phys))[::-1]
        # device copies of the host state
        self.ctx_dev = torch.zeros(batch, dtype=torch.int32, device=dev)
        self.head_dev = torch.zeros(batch, dtype=torch.int32, device=dev)
        self.pages_dev = torch.full((batch, self.max_pages), -1, dtype=torch.int32, device=dev)
        self.win_off_dev = torch.arange(batch, dtype=torch.int64, device=dev) * self.win_stride
        self.body_off_dev = torch.zeros(batch, dtype=torch.int64, device=dev)
        self._flags = L.LOOPVQ_LAYOUT_PAGED_BODY | L.LOOPVQ_LAYOUT_RING_WINDOW
        ws = L.loopvq_decode_workspace_bytes(self.desc, self._layout(None, None))
        if ws == 0:
            raise ValueError("invalid cache layout")
        self.workspace = torch.zeros(_round_up(ws, 256), dtype=torch.uint8, device=dev)

    def _layout(self, new_k, new_v):
        return L.make_layout(self.batch, self.n_sink, self.n_recent, self.page, self.max_ctx_len, self.ctx_dev,
                             self.body_off_dev, self.win_off_dev, self.body_pool_tokens, self.win_pool_tokens,
                             self._flags, self.pages_dev, self.bpt, self.max_pages, self.head_dev, self.ring,
                             new_k, new_v)

    def _sync_state(self, r):
        self.ctx_dev[r] = self.ctx[r]
        self.head_dev[r] = self.head[r]
        row = self.pages[r] + [-1] * (self.max_pages - len(self.pages[r]))
        self.pages_dev[r].copy_(torch.tensor(row, dtype=torch.int32))

    def split(self, r):
        """(sink, body, recent) of request r's current length."""
        return L.loopvq_ctx_split(self.ctx[r], self.n_sink, self.n_recent, self.page)

    # -------------------------------------------------------------- setup
    def set_codebooks(self, cb_k, cb_v) -> None:
        """Canonical codebooks [NB][H][J][C][Tc][W] (host arrays) -> packed."""
        for src, dst in ((cb_k, self.cbK), (cb_v, self.cbV)):
            t = torch.from_numpy(np.ascontiguousarray(src, dtype=np.float32)).to(self.cb_dtype).to(self.device)
            L.loopvq_codebook_pack(self.desc, t, dst)
        torch.cuda.current_stream().synchronize()

    def _slot_row(self, r, i):
        """Window-pool row of window token i of request r (sink, then ring)."""
        s = self.split(r)[0]
        base = r * self.win_stride
        return base + i if i < s else base + self.n_sink + (self.head[r] + i - s) % self.ring

    def _body_pos(self, r, p):
        """Index-pool position of body token p of request r (allocating its page)."""
        pi = p // self.bpt
        while len(self.pages[r]) <= pi:
            if not self.free:
                raise RuntimeError("index pool out of pages")
            self.pages[r].append(self.free.pop())
        return self.pages[r][pi] * self.bpt + p % self.bpt

    def prefill(self, r, K, V) -> None:
        """Prompt keys and values [T][N][H][D] (torch, any device, any float
        dtype): the window tokens are stored in bf16, the body is encoded into
        pages.  N is the request's new length."""
        N = K.shape[1]
        self.ctx[r], self.head[r] = N, 0
        s, body, rec = self.split(r)
        kb = K.to(self.device, torch.bfloat16)
        vb = V.to(self.device, torch.bfloat16)
        for i in list(range(s)) + list(range(s + body, N)):
            row = self._slot_row(r, i if i < s else i - body)
            self.winK[:, :, row] = kb[:, i]
            self.winV[:, :, row] = vb[:, i]
        H, D = self.H, self.D
        p = 0
        while p < body:
            n = min(body - p, self.bpt - p % self.bpt)
            pos = self._body_pos(r, p)
            for kind, x, pool in ((L.LOOPVQ_KEYS, kb, self.idxK), (L.LOOPVQ_VALUES, vb, self.idxV)):
                xs = x[:, s + p:s + p + n]
                L.loopvq_encode(self.desc, self.cbK if kind == L.LOOPVQ_KEYS else self.cbV, kind, xs, n,
                                xs.stride(0), xs.stride(1), xs.stride(2), pool, pos, self.body_pool_tokens)
            p += n
        self._sync_state(r)

    # -------------------------------------------------------------- per token
    def begin_token(self, r) -> None:
        """Request r grows by one token.  When its body grows, the oldest
        recent page is encoded from the ring into the body pages first."""
        s0, body0, rec0 = self.split(r)
        self.ctx[r] += 1
        s1, body1, rec1 = self.split(r)
        grown = body1 - body0
        if grown:
            if grown != self.page or self.head[r] % self.page:
                raise RuntimeError("unexpected window transition")
            pos = self._body_pos(r, body0)
            base = r * self.win_stride + self.n_sink + self.head[r]
            P = self.win_pool_tokens
            for kind, win, pool, cb in ((L.LOOPVQ_KEYS, self.winK, self.idxK, self.cbK),
                                        (L.LOOPVQ_VALUES, self.winV, self.idxV, self.cbV)):
                view = win[:, :, base:base + self.page]
                L.loopvq_encode(self.desc, cb, kind, view, self.page, self.H * P * self.D, self.D, P * self.D,
                                pool, pos, self.body_pool_tokens)
            self.head[r] = (self.head[r] + self.page) % self.ring
        self._sync_state(r)

    def set_queries(self, q) -> None:
        """Queries [batch][Hq][D] (host array or torch tensor) of the loop step about to run."""
        t = q if isinstance(q, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(q, dtype=np.float32))
        self.q.copy_(t.to(self.device, self.q.dtype))

    def decode(self, loop_step, new_k=None, new_v=None, softmax_scale=None, stream=None) -> None:
        """Decode attention at loop_step for every request.  new_k/new_v are
        the current token's bf16 K and V at this step ([batch][H][D] device
        tensors): the kernel stores them in the token's ring slot and uses
        them.  Without them the slot must already hold the token."""
        scale = self.D ** -0.5 if softmax_scale is None else softmax_scale
        layout = self._layout(new_k, new_v)
        L.loopvq_decode_attn(self.desc, self.cbK, self.cbV, layout, self.idxK, self.idxV, self.winK, self.winV,
                             self.q, loop_step, scale, self.out, self.lse, self.workspace, stream)

    def device_status(self):
        return L.loopvq_read_device_status(self.workspace)

    def body_codes(self, r, kind) -> np.ndarray:
        """Body codes of request r in logical order, [NB][H][n_body][J]."""
        body = self.split(r)[1]
        out = np.zeros((self.NB, self.H, body, self.J), dtype=np.uint8)
        pool = self.idxK if kind == L.LOOPVQ_KEYS else self.idxV
        p = 0
        while p < body:
            n = min(body - p, self.bpt - p % self.bpt)
            pos = self.pages[r][p // self.bpt] * self.bpt + p % self.bpt
            t = torch.empty((self.NB, self.H, n, self.J), dtype=torch.uint8, device=self.device)
            L.loopvq_index_pool_unpack(self.desc, kind, pool, pos, self.body_pool_tokens, n, t)
            out[:, :, p:p + n] = t.cpu().numpy()
            p += n
        return out


class MXCache:
    """Microscaled serving cache of one layer (K and V) for a batch of requests.

    Every token is coded the moment it is written (``loopvq_mx_write``): e4m3
    or e2m1 elements, one power-of-two scale per 32 channels, no codebook and
    no window.  Contexts live in pages of ``page_tokens`` tokens, taken from a
    free list.  A step:

        cache.extend([1, 0, 7, ...])          # new tokens of each request
        for t in range(n_loop):
            cache.write(k_t, v_t, t)          # [rows][H][D], packed by request
            out, lse = cache.attend(t, q_t, tree_mask)
        cache.keep([None, [], [0, 2, 5], ...])  # trees: the accepted nodes

    ``keep`` moves the accepted tokens behind the prefix and drops the rest;
    ``truncate`` drops tokens at the end, ``read`` gives a range's values back.
    Every request's lengths are host state; device arrays are made anew by each
    ``extend``, so calls that are still running on the GPU, on any stream, keep
    theirs.  All calls go to torch's current stream; a caller that changes streams
    orders them as for any tensor.  A CUDA graph captured from these calls has the
    lengths and pages of its step, at every replay (``loopvq.prepare_mx_*`` with
    the caller's own arrays serve graphs for many steps).
    """

    def __init__(self, *, n_loop, n_heads_kv, head_dim, batch, max_ctx_len, format="e4m3", page_tokens=256,
                 n_pages=None, n_heads_q=None, out_dtype=torch.bfloat16, device="cuda"):
        if format not in ("e4m3", "e2m1"):
            raise ValueError(f"unknown element format {format!r}")
        if page_tokens < 32 or page_tokens % 32:
            raise ValueError("page_tokens must be a positive multiple of 32")
        self.device = torch.device(device)
        self.T, self.H, self.D = n_loop, n_heads_kv, head_dim
        self.Hq = n_heads_q or n_heads_kv
        self.batch, self.max_ctx_len, self.page_tokens = batch, max_ctx_len, page_tokens
        self.out_dtype = out_dtype
        self.max_pages = max(1, -(-max_ctx_len // page_tokens))
        self.n_pages = batch * self.max_pages if n_pages is None else n_pages
        self.pool_tokens = self.n_pages * page_tokens
        self.desc = L.make_mx_desc(n_loop, n_heads_kv, head_dim,
                                   L.LOOPVQ_MX_E4M3 if format == "e4m3" else L.LOOPVQ_MX_E2M1, self.Hq)
        nbytes = L.loopvq_mx_pool_bytes(self.desc, self.pool_tokens)
        if nbytes == 0:
            raise ValueError("invalid cache geometry")
        self.poolK = torch.zeros(nbytes, dtype=torch.uint8, device=self.device)
        self.poolV = torch.zeros_like(self.poolK)
        self.fault_bits = torch.zeros(1, dtype=torch.int32, device=self.device)
        self.ctx = [0] * batch
        self.pages = [[] for _ in range(batch)]
        self.free = list(range(self.n_pages))[::-1]
        self.new = [0] * batch
        self.rows = 0
        self.layout = None
        self.captured = []       # layouts that CUDA graphs read

    def _layout(self, ctx, new, pages=None):
        off = [0]
        for n in new:
            off.append(off[-1] + n)
        dev = dict(dtype=torch.int32, device=self.device)
        table = [p + [-1] * (self.max_pages - len(p)) for p in pages or self.pages]
        return L.make_mx_layout(self.batch, self.page_tokens, self.max_pages, self.pool_tokens, self.max_ctx_len,
                                max(new), off[-1], torch.tensor(ctx, **dev), torch.tensor(off, **dev),
                                torch.tensor(table, **dev))

    # -------------------------------------------------------------- lengths
    def extend(self, n_new) -> None:
        """Contexts grow by n_new[r] tokens: the rows of the calls up to the
        next ``extend``, packed in the order of the requests."""
        n_new = [int(n) for n in n_new]
        if len(n_new) != self.batch or min(n_new) < 0:
            raise ValueError("one count of new tokens per request")
        grown = [c + n for c, n in zip(self.ctx, n_new)]
        if max(grown) > self.max_ctx_len:
            raise ValueError("a context would exceed max_ctx_len")
        need = [-(-c // self.page_tokens) - len(p) for c, p in zip(grown, self.pages)]
        if sum(need) > len(self.free):
            raise RuntimeError("cache out of pages")
        taken = reversed(self.free)
        pages = [p + [next(taken) for _ in range(n)] for p, n in zip(self.pages, need)]
        self.layout = self._layout(grown, n_new, pages)    # if that fails, nothing has changed
        del self.free[len(self.free) - sum(need):]
        self.pages, self.ctx, self.new, self.rows = pages, grown, n_new, sum(n_new)
        if self.device.type == "cuda":
            self.made_on = torch.cuda.current_stream(self.device).cuda_stream

    def truncate(self, r, ctx_len) -> None:
        """Request r's context ends at ctx_len; its pages behind that are free
        (0: the request is over).  Ends the present step."""
        r = range(self.batch)[r]
        if not 0 <= ctx_len <= self.ctx[r]:
            raise ValueError("truncate cannot grow a context")
        self.ctx[r] = ctx_len
        held = -(-ctx_len // self.page_tokens)
        self.free += self.pages[r][held:][::-1]
        self.pages[r] = self.pages[r][:held]
        self._end_step()

    def _end_step(self):
        self.new, self.rows, self.layout = [0] * self.batch, 0, None

    def _step(self):
        if self.layout is None:
            raise RuntimeError("extend() begins a step")
        if self.device.type == "cuda":
            # the arrays were made on another stream, maybe: their memory is not
            # for new ones before this stream's calls are done; a graph's stays
            stream = torch.cuda.current_stream(self.device)
            if torch.cuda.is_current_stream_capturing():
                if not any(lay is self.layout for lay in self.captured):
                    self.captured.append(self.layout)
            elif stream.cuda_stream != self.made_on:
                for a in self.layout._keep:
                    a.record_stream(stream)
        return self.layout

    # -------------------------------------------------------------- the step
    def _rows(self, x, heads, lead):
        if tuple(x.shape) != (*lead, self.rows, heads, self.D) or (x.numel() and x.stride(-1) != 1):
            raise ValueError(f"expected {[*lead, self.rows, heads, self.D]} with consecutive channels, "
                             f"got {list(x.shape)}")

    def write(self, k, v, loop_step=None) -> None:
        """Keys and values of the new tokens: [rows][H][D] at one loop step, or
        [T][rows][H][D] of all."""
        lay = self._step()
        lead = (self.T,) if loop_step is None else ()
        self._rows(k, self.H, lead)
        self._rows(v, self.H, lead)
        if k.stride() != v.stride():
            v = v.contiguous()
            k = k.contiguous()
        first, n = (0, self.T) if loop_step is None else (loop_step, 1)
        L.loopvq_mx_write(self.desc, lay, first, n, k, v, k.stride(0) if lead else 0, k.stride(-3), k.stride(-2),
                          self.poolK, self.poolV, self.fault_bits)

    def attend(self, loop_step, q, tree_mask=None, softmax_scale=None, softcap=0.0, slopes=None):
        """Attention of the new tokens at loop_step: q [rows][Hq][D] -> (out
        [rows][Hq][D], lse [rows][Hq]).  tree_mask: int64 [rows], bit j of a
        request's row i: its new token i sees its new token j (None: a chain).
        At most 64 new tokens per request: a longer prompt has a step of its own."""
        lay = self._step()
        self._rows(q, self.Hq, ())
        out = torch.empty((self.rows, self.Hq, self.D), dtype=self.out_dtype, device=self.device)
        lse = torch.empty((self.rows, self.Hq), dtype=torch.float32, device=self.device)
        ws = torch.empty(max(256, L.loopvq_mx_attn_workspace_bytes(self.desc, lay)), dtype=torch.uint8,
                         device=self.device)
        L.loopvq_mx_attn(self.desc, lay, self.poolK, self.poolV, q, q.stride(0), q.stride(1), tree_mask, loop_step,
                         self.D ** -0.5 if softmax_scale is None else softmax_scale, softcap, slopes, out, lse, ws,
                         self.fault_bits)
        return out, lse

    def keep(self, accepted) -> None:
        """accepted[r]: the new tokens of request r that stay, in the order
        that they take behind the prefix (None: all of them as they are).
        Of more than 64 new tokens of a request all stay, or the first ones.
        Ends the step."""
        lay = self._step()
        if len(accepted) != self.batch:
            raise ValueError("one list of accepted tokens per request")
        lists = [list(range(n)) if a is None else [int(i) for i in a] for a, n in zip(accepted, self.new)]
        for a, n in zip(lists, self.new):
            if len(a) > n or any(not 0 <= i < n for i in a):
                raise ValueError("accepted tokens are indices of the request's new tokens")
        moves = [a != list(range(len(a))) for a in lists]
        if any(moves):
            sent = lists
            if max(self.new) > 64:   # a prompt beside the trees: only the trees are sent
                if max(n for n, m in zip(self.new, moves) if m) > 64:
                    raise ValueError("of more than 64 new tokens only the first ones can be kept")
                lay = self._layout(self.ctx, [n if m else 0 for n, m in zip(self.new, moves)])
                sent = [a if m else [] for a, m in zip(lists, moves)]
            wide = max(len(a) for a in sent)
            dev = dict(dtype=torch.int32, device=self.device)
            L.loopvq_mx_keep(self.desc, lay, torch.tensor([a + [-1] * (wide - len(a)) for a in sent], **dev),
                             torch.tensor([len(a) for a in sent], **dev), wide, self.poolK, self.poolV,
                             self.fault_bits)
        ends = [c - n + len(a) for c, n, a in zip(self.ctx, self.new, lists)]
        for r, e in enumerate(ends):
            self.truncate(r, e)
        self._end_step()

    def read(self, r, begin=0, end=None, first_step=0, n_steps=None, dtype=None):
        """Values of tokens begin..end-1 of request r: (k, v), each [n_steps][tokens][H][D]."""
        r = range(self.batch)[r]
        end = self.ctx[r] if end is None else end
        n_steps = self.T - first_step if n_steps is None else n_steps
        if not 0 <= begin <= end <= self.ctx[r]:
            raise ValueError("the range is not in the context")
        n = end - begin
        lay = self._layout([end if i == r else 0 for i in range(self.batch)],
                           [n if i == r else 0 for i in range(self.batch)])
        k = torch.empty((n_steps, n, self.H, self.D), dtype=dtype or self.out_dtype, device=self.device)
        v = torch.empty_like(k)
        if n:
            L.loopvq_mx_read(self.desc, lay, first_step, n_steps, self.poolK, self.poolV, k, v, n * self.H * self.D,
                             self.H * self.D, self.D, self.fault_bits)
        return k, v

    def device_faults(self) -> int:
        """LOOPVQ_FAULT_* bits that the calls so far have set; waits for them."""
        return int(self.fault_bits.item())
