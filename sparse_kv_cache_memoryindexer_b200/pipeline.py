"""One trigger window of the LSA indexer path on one GPU: buffers plus the five C-ABI calls, and the
decode steps inside it.

Allocation and call order only (PyTorch holds the device memory); every stage is a kernel
of liblsa.so.  Order of the stages follows the hyper.ai summary ("Method") and the blog
review's sections 3-3.2: project -> score/threshold/OR/compact -> fetch -> Lightning Top-k; at each
decode step Top-k -> append to the window cache -> core attention over both.
"""
from __future__ import annotations

from contextlib import contextmanager

import torch

from . import lsa


@contextmanager
def _stage(name):
    """NVTX range around a stage's launches (ncu --nvtx / nsys show the stage boundaries)."""
    torch.cuda.nvtx.range_push(name)
    try:
        yield
    finally:
        torch.cuda.nvtx.range_pop()


class WindowCache:
    """The keys and values that stay on the GPU, in pages: the sliding window and the first tokens (the rest
    of the context is reached through the fetched entries).  Which pages a sequence has is the caller's:
    page_table [B][max_pages] holds a page number for every page_size tokens that some query can still see
    or that a new token falls on, and -1 elsewhere (a page behind the window may be given to others).

    cdtype float8_e4m3fn keeps the cache in 8 bits with one scale per page and head."""

    def __init__(self, B, H_kv, D, page_size, n_pages, max_pages, dtype, cdtype=None, window=0, n_sink=0, device="cuda"):
        dev = torch.device(device)
        cdtype = dtype if cdtype is None else cdtype
        # what the calls would refuse, before anything is allocated for it
        if D not in (32, 64, 128) or page_size not in (16, 32, 64, 128):
            raise ValueError(f"D must be 32, 64 or 128 and page_size 16, 32, 64 or 128, got {D} and {page_size}")
        if (dtype, cdtype) not in ((torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16),
                                   (torch.bfloat16, torch.float8_e4m3fn)):
            raise TypeError(f"dtype and cdtype must be fp32 and fp32, or bf16 and bf16 or float8_e4m3fn, got {dtype} and {cdtype}")
        self.B, self.H_kv, self.D, self.page_size = B, H_kv, D, page_size
        self.dtype, self.cdtype, self.window, self.n_sink = dtype, cdtype, window, n_sink
        shape = (n_pages, H_kv, page_size, D)
        self.k = torch.empty(shape, dtype=self.cdtype, device=dev)
        self.v = torch.empty(shape, dtype=self.cdtype, device=dev)
        fp8 = self.cdtype == torch.float8_e4m3fn
        self.k_scale = torch.empty((n_pages, H_kv), dtype=torch.float32, device=dev) if fp8 else None
        self.v_scale = torch.empty((n_pages, H_kv), dtype=torch.float32, device=dev) if fp8 else None
        self.page_table = torch.full((B, max_pages), -1, dtype=torch.int32, device=dev)
        self.len = torch.zeros(B, dtype=torch.int32, device=dev)  # tokens of each sequence so far

    def append(self, k, v, q_offsets, inv_freq=None, interleaved=False, q=None, q_out=None, stream=None):
        """Writes the new tokens' keys and values (rotated to their positions); `len` still counts the
        tokens before them, which is what attend() of the same tokens wants; advance() moves it on."""
        lsa.lsa_kv_append(k, v, q_offsets, self.len, self.page_table, self.k, self.v, k_scale=self.k_scale,
                          v_scale=self.v_scale, inv_freq=inv_freq, interleaved=interleaved, q=q, q_out=q_out,
                          stream=stream)

    def attend(self, q, q_offsets, out, workspace, softmax_scale=None, lse_out=None, stream=None):
        """Attention of the tokens last appended over the window and the first tokens."""
        lsa.lsa_window_attention(q, q_offsets, self.len, self.page_table, self.k, self.v, out, workspace,
                                 window=self.window, n_sink=self.n_sink, softmax_scale=softmax_scale,
                                 k_scale=self.k_scale, v_scale=self.v_scale, lse_out=lse_out, stream=stream)

    def advance(self, q_offsets):
        """Counts the appended tokens (on the current stream)."""
        self.len += (q_offsets[1:] - q_offsets[:-1]).to(torch.int32)


class IndexerPath:
    """Device buffers for one window of B sequences (ragged, total_S entries per layer)."""

    def __init__(self, L, B, d, r, n_h, d_I, tau, k, total_S, row_bytes, dtype, kdtype,
                 device="cuda", with_scores=False, with_mask=False, incremental=False):
        self.L, self.B, self.d, self.r, self.n_h, self.d_I = L, B, d, r, n_h, d_I
        self.tau, self.k, self.total_S, self.row_bytes = tau, k, int(total_S), row_bytes
        self.dtype, self.kdtype = dtype, kdtype
        dev = torch.device(device)
        T = self.total_S
        u8 = torch.uint8

        def ws(nbytes):
            return torch.empty(max(int(nbytes), 256), dtype=u8, device=dev)

        self.q = torch.empty((L, B, n_h, d_I), dtype=dtype, device=dev)
        self.w = torch.empty((L, B, n_h), dtype=torch.float32, device=dev)
        self.ws_proj = ws(lsa.lsa_project_workspace_size(L, B, d, r, n_h, d_I, dtype))
        self.idx = torch.empty(T, dtype=torch.int32, device=dev)
        self.count = torch.empty(B, dtype=torch.int32, device=dev)
        self.ws_score = ws(lsa.lsa_score_select_workspace_size(L, B, T))
        self.scores = torch.empty((L, T), dtype=torch.float32, device=dev) if with_scores else None
        self.mask = torch.empty(T, dtype=u8, device=dev) if with_mask else None
        self.hot_kv = torch.empty((T, row_bytes), dtype=u8, device=dev)
        # E4M3 keys are decoded to bf16 by the fetch (scales kept apart)
        hot_dt = torch.bfloat16 if kdtype == torch.float8_e4m3fn else kdtype
        self.hot_K = torch.empty((T, d_I), dtype=hot_dt, device=dev)
        self.hot_scale = torch.empty(T, dtype=torch.float32, device=dev) if kdtype == torch.float8_e4m3fn else None
        self.topk_idx = torch.empty((B, tau, k), dtype=torch.int32, device=dev)
        self.topk_score = torch.empty((B, tau, k), dtype=torch.float32, device=dev)
        self.ws_topk = ws(lsa.lsa_lightning_topk_workspace_size(B, tau, T, k))
        # the incremental row fetch of run(prev=...): workspace and the count of rows that crossed the link
        self.ws_incr = ws(lsa.lsa_fetch_incremental_workspace_size(B, T)) if incremental else None
        self.host_rows = torch.zeros(1, dtype=torch.int32, device=dev) if incremental else None
        # the host-link row gather of run(), at a higher priority than the caller's stream so that its
        # few fat CTAs are placed before the Top-k's persistent CTAs fill the SMs
        self._link = torch.cuda.Stream(device=dev, priority=-1)

    def project(self, h, W_dq, W_iuq, W_w, stream=None):
        lsa.lsa_project(h, W_dq, W_iuq, W_w, self.q, self.w, self.ws_proj, stream=stream)

    def select(self, K, k_scale, seq_offsets, threshold=0.5, q=None, w=None, stream=None):
        lsa.lsa_memindex_score_select(self.q if q is None else q, self.w if w is None else w, K, k_scale,
                                      seq_offsets, self.total_S, threshold, self.idx, self.count, self.ws_score,
                                      scores_out=self.scores, mask_out=self.mask, stream=stream)

    def fetch(self, seq_offsets, pool, K_sel, k_scale_sel, stream=None):
        """Rows and keys in one launch."""
        lsa.lsa_fetch_gather(self.idx, self.count, seq_offsets, self.total_S, pool, self.hot_kv, K_sel, k_scale_sel,
                             self.hot_K, self.hot_scale, stream=stream)

    def fetch_keys(self, seq_offsets, K_sel, k_scale_sel, stream=None):
        """The keys of the fetched entries only (device to device; the Top-k needs nothing else)."""
        lsa.lsa_fetch_gather(self.idx, self.count, seq_offsets, self.total_S, None, None, K_sel, k_scale_sel,
                             self.hot_K, self.hot_scale, stream=stream)

    def fetch_rows(self, seq_offsets, pool, stream=None):
        """The KV rows of the fetched entries only, over the host link."""
        lsa.lsa_fetch_gather(self.idx, self.count, seq_offsets, self.total_S, pool, self.hot_kv, stream=stream)

    def fetch_rows_incremental(self, seq_offsets, pool, prev, stream=None):
        """The KV rows of the fetched entries with the previous window's rows resident: rows that
        both windows fetched are copied on the device, only the others cross the host link.
        prev = (idx, count, seq_offsets, total_S, hot_kv) of the previous window."""
        p_idx, p_count, p_offs, p_T, p_hot = prev
        lsa.lsa_fetch_gather_incremental(self.idx, self.count, seq_offsets, self.total_S, p_idx, p_count, p_offs, p_T,
                                         p_hot, pool, self.hot_kv, self.ws_incr, host_rows_out=self.host_rows,
                                         stream=stream)

    def topk(self, q_dec, w_dec, seq_offsets, stream=None):
        lsa.lsa_lightning_topk(q_dec, w_dec, self.hot_K, self.hot_scale, self.idx, self.count, seq_offsets,
                               self.total_S, self.k, self.topk_idx, self.ws_topk, topk_score=self.topk_score,
                               stream=stream)

    def run(self, h, W_dq, W_iuq, W_w, K, k_scale, seq_offsets, pool, q_dec, w_dec, sel_layer=0,
            threshold=0.5, stream=None, events=None, prev=None):
        """The whole hot path for one trigger window.

        The KV rows cross the host link on a second stream while the keys are gathered and the
        Top-k runs on `stream` (the Top-k reads only the keys); `stream` waits for both before
        it returns, so work queued on it afterwards sees the whole window.  events: optional
        list of 7 timing events, recorded at the stage boundaries (start, after project, after
        select, after the keys, after the Top-k, after the rows (second stream), end).
        prev: the previous window's (idx, count, seq_offsets, total_S, hot_kv); the rows then come
        from the incremental fetch (the path must be built with incremental=True), and the
        previous hot buffer must stay untouched until `stream` has passed this window.
        """
        st = torch.cuda.current_stream() if stream is None else stream
        ev = events if events is not None else [None] * 7
        rec = lambda e, s: e.record(s) if e is not None else None
        rec(ev[0], st)
        with _stage("lsa.project"):
            self.project(h, W_dq, W_iuq, W_w, st)
        rec(ev[1], st)
        with _stage("lsa.score_select"):
            self.select(K, k_scale, seq_offsets, threshold, stream=st)
        rec(ev[2], st)
        selected = torch.cuda.Event()
        selected.record(st)
        self._link.wait_event(selected)
        with _stage("lsa.fetch_rows"):
            if prev is None:
                self.fetch_rows(seq_offsets, pool, self._link)
            else:
                self.fetch_rows_incremental(seq_offsets, pool, prev, self._link)
        rec(ev[5], self._link)
        rows_done = torch.cuda.Event()
        rows_done.record(self._link)
        with _stage("lsa.fetch_keys"):
            self.fetch_keys(seq_offsets, K[sel_layer], None if k_scale is None else k_scale[sel_layer], st)
        rec(ev[3], st)
        with _stage("lsa.lightning_topk"):
            self.topk(q_dec, w_dec, seq_offsets, st)
        rec(ev[4], st)
        st.wait_event(rows_done)
        rec(ev[6], st)

    def open_decode(self, cache, H_q, W=0):
        """Buffers for decode_step: one token per sequence, H_q query heads over `cache` (whose rows and the
        fetched rows must agree: row_bytes = 2 * H_kv * D elements), up to W entries compressed in the window."""
        dev = self.idx.device
        esize = torch.empty((), dtype=cache.dtype).element_size()
        if self.row_bytes != 2 * cache.H_kv * cache.D * esize or cache.cdtype != cache.dtype:
            raise ValueError(f"the fetched rows ({self.row_bytes} bytes) must be [2][H_kv][D] of the cache's type")
        if cache.B != self.B:
            raise ValueError(f"the cache holds {cache.B} sequences, the path {self.B}")
        if H_q <= 0 or H_q % cache.H_kv or not 1 <= self.k <= lsa.LSA_MAX_TOPK:
            raise ValueError(f"H_q must be a multiple of H_kv and k in [1, {lsa.LSA_MAX_TOPK}], got {H_q} of {cache.H_kv} and {self.k}")
        self.cache, self.H_q, self.W = cache, H_q, W
        u8 = torch.uint8
        self.step_idx = torch.empty((self.B, self.k), dtype=torch.int32, device=dev)
        self.step_score = torch.empty((self.B, self.k), dtype=torch.float32, device=dev)
        self.ws_step = torch.empty(max(lsa.lsa_lightning_topk_step_workspace_size(self.B, self.total_S, self.n_h, self.d_I, W), 256),
                                   dtype=u8, device=dev)
        self.ws_core = torch.empty(lsa.lsa_core_attention_workspace_size(self.B, self.B, H_q, cache.H_kv, cache.D, self.k),
                                   dtype=u8, device=dev)
        self.q_rot = torch.empty((self.B, H_q, cache.D), dtype=cache.dtype, device=dev)
        self.attn_out = torch.empty((self.B, H_q, cache.D), dtype=cache.dtype, device=dev)
        self.attn_lse = torch.empty((self.B, H_q), dtype=torch.float32, device=dev)
        self.one_each = torch.arange(self.B + 1, dtype=torch.int64, device=dev)

    def _check_window_entries(self, win_K, win_count, win_kv):
        """The Top-k picks among the entries compressed in the window; core attention then needs every one's row."""
        W = win_K.size(1)
        if W == 0:
            return
        if win_count is None or win_kv is None or win_kv.dim() < 2 or win_kv.size(1) < W:
            raise ValueError(f"win_K holds {W} entries a sequence: win_count and win_kv [B][{W}][row_bytes] go with it")
        if W > self.W:
            raise ValueError(f"win_K holds {W} entries a sequence, open_decode was told of {self.W}")

    def decode_step(self, q_step, w_step, q, k, v, seq_offsets, win_K=None, win_scale=None, win_count=None, win_kv=None,
                    inv_freq=None, interleaved=False, softmax_scale=None, stream=None):
        """One decode step of every sequence: the Lightning Top-k of its indexer query over the fetched entries
        (and the win_count entries compressed since the trigger: keys win_K, rows win_kv), the new token's q, k, v
        [B][heads][D] rotated and k, v appended to the window cache, and one softmax over the Top-k rows, the
        window and the first tokens.  Returns attn_out [B][H_q][D] (step_idx, attn_lse beside it); cache.advance
        follows once every layer is done.  Launches only kernels: a step can be recorded in a CUDA graph."""
        c = self.cache
        if win_K is not None:
            self._check_window_entries(win_K, win_count, win_kv)
        dev = c.k.get_device()
        if dev != lsa._current_device():  # (the Top-k runs on the current device)
            with torch.cuda.device(dev):
                return self.decode_step(q_step, w_step, q, k, v, seq_offsets, win_K, win_scale, win_count, win_kv,
                                        inv_freq, interleaved, softmax_scale, stream)
        with _stage("lsa.lightning_topk_step"):
            lsa.lsa_lightning_topk_step(q_step, w_step, self.hot_K, self.hot_scale, self.idx, self.count, seq_offsets,
                                        self.total_S, self.k, self.step_idx, self.ws_step, win_K=win_K,
                                        win_scale=win_scale, win_count=win_count, topk_score=self.step_score,
                                        stream=stream)
        with _stage("lsa.kv_append"):
            c.append(k, v, self.one_each, inv_freq=inv_freq, interleaved=interleaved, q=q, q_out=self.q_rot, stream=stream)
        with _stage("lsa.core_attention"):
            lsa.lsa_core_attention(self.q_rot, self.one_each, c.len, c.page_table, c.k, c.v, self.step_idx, self.idx,
                                   self.count, seq_offsets, self.total_S, self.hot_kv, self.attn_out, self.ws_core,
                                   win_kv=win_kv, window=c.window, n_sink=c.n_sink, softmax_scale=softmax_scale,
                                   lse_out=self.attn_lse, stream=stream)
        return self.attn_out
