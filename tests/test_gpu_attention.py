"""lsa_window_attention and lsa_core_attention against their definition in 64 bits (tests/attn_oracle.py)."""
import math

import pytest
import torch

import attn_oracle as ao

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sparse_kv_cache_memoryindexer_b200 as mod
    mod.lsa_check_device()
    return mod


class Case:
    def __init__(self, new, old, H, Hq, D, page, dt=BF16, cdt=None, window=0, sinks=0, seed=3, spare_rows=0, spread=1.0,
                 only_needed=True):
        g = torch.Generator().manual_seed(seed)
        self.new, self.old, self.H, self.Hq, self.D, self.page = new, old, H, Hq, D, page
        self.dt, self.cdt, self.window, self.sinks = dt, cdt or dt, window, sinks
        self.scale = D ** -0.5
        B, self.N = len(new), sum(new) + spare_rows
        self.offs = torch.tensor([0] + list(torch.tensor(new).cumsum(0)), dtype=torch.int64)
        self.len = torch.tensor(old, dtype=torch.int32)
        total = [max(1, -(-(o + n) // page)) for o, n in zip(old, new)]
        self.max_pages = max(total)
        need = []
        for o, n, t in zip(old, new, total):
            lo = max(0, o - window + 1) // page if window and only_needed else 0
            need.append(sorted(set(range(lo, t)) | set(range(min(t, -(-sinks // page))))))
        count = sum(len(p) for p in need)
        order = torch.randperm(count, generator=g)
        self.n_pages = count + 1
        self.table = torch.full((B, self.max_pages), -1, dtype=torch.int32)
        at = 0
        for b, pages in enumerate(need):
            for p in pages:
                self.table[b, p] = order[at]
                at += 1
        self.q = (torch.randn((self.N, Hq, D), generator=g) * spread).to(dt)
        shape = (self.n_pages, H, page, D)
        if self.cdt == ao.E4M3:
            self.kc = (torch.randn(shape, generator=g) * 60).clamp(-448, 448).to(ao.E4M3)
            self.vc = (torch.randn(shape, generator=g) * 60).clamp(-448, 448).to(ao.E4M3)
            # scales over four binades, not powers of two
            self.ks = 0.02 * torch.exp2(torch.randn((self.n_pages, H), generator=g))
            self.vs = 0.02 * torch.exp2(torch.randn((self.n_pages, H), generator=g))
        else:
            self.kc, self.vc = torch.randn(shape, generator=g).to(self.cdt), torch.randn(shape, generator=g).to(self.cdt)
            self.ks = self.vs = None
        self.k = 0

    def add_topk(self, k, entries, fetched, fresh, seed=11):
        """Per sequence: `fetched` of its entries in the hot buffer, `fresh` made since; Top-k in any order."""
        g = torch.Generator().manual_seed(seed)
        B = len(self.new)
        self.k, self.W = k, fresh
        self.so = torch.tensor([0] + list(torch.tensor(entries).cumsum(0)), dtype=torch.int64)
        self.T = int(self.so[-1])
        self.idx = torch.full((self.T,), -9, dtype=torch.int32)
        self.cnt = torch.tensor(fetched, dtype=torch.int32)
        self.hot = torch.randn((self.T, 2, self.H, self.D), generator=g).to(self.dt)
        self.win = torch.randn((B, fresh, 2, self.H, self.D), generator=g).to(self.dt) if fresh else None
        self.topk = torch.full((self.N, k), -1, dtype=torch.int32)
        for b in range(B):
            lst = torch.randperm(entries[b], generator=g)[:fetched[b]].sort().values.to(torch.int32)
            o = int(self.so[b])
            self.idx[o:o + fetched[b]] = lst
            pool = torch.cat([lst, entries[b] + torch.arange(fresh, dtype=torch.int32)])
            for i in range(self.new[b]):
                best = pool[torch.randperm(pool.numel(), generator=g)[:k]]
                self.topk[int(self.offs[b]) + i, :best.numel()] = best
        return self

    def cuda(self):
        up = lambda t: None if t is None else t.cuda()  # noqa: E731
        d = dict(q=up(self.q), q_offsets=up(self.offs), cache_len=up(self.len), page_table=up(self.table),
                 k_cache=up(self.kc), v_cache=up(self.vc), out=torch.full_like(self.q, 77.0).cuda(),
                 lse_out=torch.full((self.N, self.Hq), 77.0, device="cuda"), window=self.window, n_sink=self.sinks)
        if self.k:
            d.update(topk_idx=up(self.topk), idx=up(self.idx), count=up(self.cnt), seq_offsets=up(self.so),
                     total_S=self.T, hot_kv=up(self.hot), win_kv=None if self.win is None else up(self.win))
        else:
            d.update(k_scale=up(self.ks), v_scale=up(self.vs))
        return d

    def workspace(self, m):
        a = (self.N, len(self.new), self.Hq, self.H, self.D)
        n = m.lsa_core_attention_workspace_size(*a, self.k) if self.k else m.lsa_window_attention_workspace_size(*a)
        # whatever the workspace holds must not matter
        return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")


def call(m, case, d, ws=None, **kw):
    f = m.lsa_core_attention if case.k else m.lsa_window_attention
    f(workspace=case.workspace(m) if ws is None else ws, **{**d, **kw})


def check(case, d, rows=None, hidden=lambda b, j: False):
    """Outputs against the definition.  rows: the (sequence, token) pairs looked at (default: all);
    hidden(b, j): keys that the call must leave out."""
    out, lse = d["out"].cpu().double(), d["lse_out"].cpu().double()
    last = sum(case.new)
    assert (out[last:] == 77.0).all() and (lse[last:] == 77.0).all(), "rows behind the last sequence"
    G = case.Hq // case.H
    p_dtype = {BF16: BF16, F32: None, ao.E4M3: torch.float16}[case.cdt]
    for b, (n, old) in enumerate(zip(case.new, case.old)):
        for i in range(n):
            if rows is not None and (b, i) not in rows:
                continue
            keys = [j for j in ao.visible(old + i, old + n, case.window, case.sinks) if not hidden(b, j)]
            j = torch.tensor(keys, dtype=torch.int64)
            pg, sl = case.table[b].long()[j // case.page], j % case.page
            at = int(case.offs[b]) + i
            for h in range(case.H):
                K, V = case.kc[pg, :, sl][:, h].double(), case.vc[pg, :, sl][:, h].double()
                if case.ks is not None:
                    K, V = K * case.ks[pg, h].double()[:, None], V * case.vs[pg, h].double()[:, None]
                if case.k:
                    rows_ = []
                    S, o = int(case.so[b + 1] - case.so[b]), int(case.so[b])
                    held = case.idx[o:o + int(case.cnt[b])].tolist()
                    for e in case.topk[at].tolist():
                        if e >= S:
                            rows_.append(case.win[b, e - S])
                        elif e >= 0:
                            rows_.append(case.hot[o + held.index(e)])
                    if rows_:
                        r = torch.stack(rows_).double()
                        K, V = torch.cat([K, r[:, 0, h]]), torch.cat([V, r[:, 1, h]])
                for gq in range(G):
                    hq = h * G + gq
                    o_, l_, A, mag = ao.attend(case.q[at, hq].double(), K, V, case.scale)
                    bo, bl = ao.attend_bounds(o_, A, mag, K.shape[0], case.D, case.dt, p_dtype)
                    if K.shape[0] == 0:
                        assert (out[at, hq] == 0).all() and lse[at, hq] == -math.inf
                        continue
                    err = (out[at, hq] - o_).abs()
                    assert (err <= bo).all(), (b, i, hq, float((err / bo).max()))
                    assert abs(float(lse[at, hq]) - l_) <= bl, (b, i, hq, float(lse[at, hq]), l_, bl)


def run(m, case, rows=None):
    d = case.cuda()
    call(m, case, d)
    m.lsa_check_device()
    check(case, d, rows)
    return d


TYPES = [(BF16, BF16), (F32, F32), (BF16, ao.E4M3)]
HEADS = [(1, 1), (2, 2), (2, 14), (1, 16), (1, 64), (8, 64), (4, 12)]


@pytest.mark.parametrize("dt,cdt", TYPES)
@pytest.mark.parametrize("H,Hq", HEADS)
def test_one_token(m, dt, cdt, H, Hq):
    """Lengths around page and tile borders, one token, no history among them."""
    old = [0, 1, 15, 16, 62, 63, 64, 127, 300]
    for D, page in ((128, 64), (64, 16)):
        for window, sinks in ((0, 0), (1, 0), (50, 3), (64, 70), (1000, 4)):
            run(m, Case([1] * len(old), old, H, Hq, D, page, dt, cdt, window, sinks, seed=D + window))


@pytest.mark.parametrize("dt,cdt", TYPES)
@pytest.mark.parametrize("D,page", [(32, 16), (32, 128), (64, 32), (128, 16), (128, 32), (128, 128)])
def test_head_sizes_and_pages(m, dt, cdt, D, page):
    run(m, Case([1, 2, 0, 5], [200, 0, 3, 129], 2, 6, D, page, dt, cdt, 100, 2, spare_rows=2))


@pytest.mark.parametrize("dt,cdt", TYPES)
@pytest.mark.parametrize("H,Hq,D,page", [(1, 1, 64, 16), (2, 16, 128, 64), (1, 7, 128, 32), (2, 2, 32, 64), (2, 64, 64, 128)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (37, 4), (200, 130)])
def test_chunks(m, dt, cdt, H, Hq, D, page, window, sinks):
    """Several tokens at once: causal and window borders inside every tile."""
    run(m, Case([33, 1, 150, 16], [70, 500, 0, 129], H, Hq, D, page, dt, cdt, window, sinks, spare_rows=1))


@pytest.mark.parametrize("dt,cdt", TYPES)
@pytest.mark.parametrize("H,Hq", [(1, 8), (8, 64), (1, 1)])
def test_long_caches_of_unlike_lengths(m, dt, cdt, H, Hq):
    """Work split over the keys and joined again: every sequence's rows."""
    run(m, Case([1, 1, 1, 1, 1], [30001, 17, 4096, 9000, 0], H, Hq, 128, 64, dt, cdt))
    run(m, Case([1], [70000], H, Hq, 64, 128, dt, cdt, window=65000, sinks=5))


@pytest.mark.parametrize("cdt", [BF16, ao.E4M3])
def test_chunk_on_a_long_history(m, cdt):
    c = Case([300, 513], [5003, 1000], 2, 16, 128, 64, BF16, cdt, window=1500, sinks=4)
    run(m, c, rows={(b, i) for b, n in enumerate(c.new) for i in (0, 1, 15, 16, 17, 127, 128, 200, n - 2, n - 1)})


def test_strided_queries_and_no_lse(m):
    c = Case([3, 40], [100, 2], 2, 8, 64, 16)
    d = c.cuda()
    fused = torch.randn((c.N, 12, 64), device="cuda", dtype=BF16)
    fused[:, 2:10] = d["q"]
    d["q"] = fused[:, 2:10]
    call(m, c, d)
    check(c, d)
    e = c.cuda()
    e["lse_out"] = None
    call(m, c, e)
    m.lsa_check_device()
    assert torch.equal(e["out"], d["out"])


def test_large_scores_and_scale(m):
    """Scores of a hundred: the running maximum matters; softmax_scale is the caller's."""
    c = Case([1, 20], [700, 90], 2, 8, 64, 32, spread=8.0)
    d = c.cuda()
    c.scale = 0.5
    call(m, c, d, softmax_scale=0.5)
    m.lsa_check_device()
    check(c, d)


@pytest.mark.parametrize("cdt", [BF16, F32, ao.E4M3])
@pytest.mark.parametrize("n", [1, 3, 70])
def test_what_lies_in_unused_slots_does_not_matter(m, cdt, n):
    """Slots behind the last token, and outside the window on pages that are read, hold NaN and infinities."""
    dt = F32 if cdt == F32 else BF16
    for Hq, H, D in ((8, 2, 128), (2, 2, 64)):
        c = Case([n, n], [90, 333], H, Hq, D, 64, dt, cdt, window=75, sinks=3)
        want = run(m, c)
        d = c.cuda()
        for name in ("k_cache", "v_cache"):
            t = d[name].view(torch.uint8) if cdt == ao.E4M3 else d[name]
            bad = (0x7F, 0xFF) if cdt == ao.E4M3 else (math.nan, math.inf)
            keep = torch.zeros(t.shape[:1] + t.shape[2:3], dtype=torch.bool)
            for b in range(2):
                for i in range(n):
                    for j in ao.visible(c.old[b] + i, c.old[b] + n, c.window, c.sinks):
                        keep[int(c.table[b, j // 64]), j % 64] = True
            drop = (~keep).cuda()[:, None, :, None].expand(t.shape)
            t[drop] = bad[0]
            t[:, :, ::2][drop[:, :, ::2]] = bad[1]
        call(m, c, d)
        m.lsa_check_device()
        assert torch.equal(d["out"], want["out"]) and torch.equal(d["lse_out"], want["lse_out"])


@pytest.mark.parametrize("cdt", [BF16, F32, ao.E4M3])
def test_a_later_tokens_nan_stays_out_of_earlier_rows(m, cdt):
    """A token whose key and value are NaN (or infinite) is masked for the tokens before it, and for those whose
    window has moved past it: their results are as if it held anything else."""
    dt = F32 if cdt == F32 else BF16
    for n, Hq, H in ((9, 2, 1), (80, 16, 2), (2, 4, 2), (200, 4, 4)):
        c = Case([n], [40], H, Hq, 64, 32, dt, cdt, window=30, sinks=0)
        want = run(m, c)
        at = 40 + n // 2
        for bad in ((math.nan, math.inf) if cdt != ao.E4M3 else (0x7F,)):
            d = c.cuda()
            pg = int(c.table[0, at // 32])
            for name in ("k_cache", "v_cache"):
                t = d[name].view(torch.uint8) if cdt == ao.E4M3 else d[name]
                t[pg, :, at % 32] = bad
            call(m, c, d)
            m.lsa_check_device()
            for i in range(n):
                sees = at in ao.visible(40 + i, 40 + n, c.window, 0)
                if sees:
                    assert not torch.isfinite(d["out"][i].float()).all(), i
                    continue
                A = want["out"][i].double()
                # (a kernel may take another way through a tile with such values: its own rounding)
                tol = 3 * ao.half_step(BF16) if dt == BF16 else 1e-5
                assert torch.isfinite(d["out"][i].float()).all(), (n, i)
                assert (d["out"][i].double() - A).abs().max() <= tol * max(1.0, float(A.abs().max())), (n, i)
    # (1.0: values are standard normal and few keys are seen, so the largest |v| of a row is below 6 and the
    #  probabilities' rounding moves an output by well under 2^-8 of that)


def test_rows_with_nothing_to_see(m):
    """Every page that a query sees is unmapped: zeros and -inf, the other rows as ever; flagged."""
    from sparse_kv_cache_memoryindexer_b200 import LSAError
    for cdt in (BF16, F32, ao.E4M3):
        for n in (1, 40):
            c = Case([n, n], [100, 100], 2, 8, 64, 16, F32 if cdt == F32 else BF16, cdt)
            c.table[0] = -1
            d = c.cuda()
            call(m, c, d)
            with pytest.raises(LSAError, match="bad-page"):
                m.lsa_check_device()
            check(c, d, hidden=lambda b, j: b == 0)


def test_bad_data_is_left_out_and_flagged(m):
    from sparse_kv_cache_memoryindexer_b200 import LSAError
    for cdt in (BF16, F32, ao.E4M3):
        for n in (1, 30):
            for what, flag in (("page", "bad-page"), ("hole", "bad-page"), ("length", "count"), ("offsets", "offsets"),
                               ("scale", "scale")):
                if what == "scale" and cdt != ao.E4M3:
                    continue
                c = Case([n, n], [100, 61], 2, 8, 64, 16, F32 if cdt == F32 else BF16, cdt)
                d = c.cuda()
                pg = int(c.table[1, 2])
                if what == "page":
                    d["page_table"][1, 2] = c.n_pages
                elif what == "hole":
                    d["page_table"][1, 2] = -1
                elif what == "length":
                    d["cache_len"][1] = -5
                elif what == "offsets":
                    d["q_offsets"][2] = c.N + 7
                else:
                    d["k_scale"][pg] = math.nan
                    d["v_scale"][pg] = -1.0
                call(m, c, d)
                with pytest.raises(LSAError, match=flag):
                    m.lsa_check_device()
                if what in ("page", "hole", "scale"):
                    check(c, d, hidden=lambda b, j: b == 1 and j // 16 == 2)
                else:
                    check(c, d, rows={(0, i) for i in range(n)})
                m.lsa_check_device()


def test_zero_scales(m):
    """A page whose values are all zero by its scale still takes its share of the softmax."""
    for n in (1, 50):
        c = Case([n], [200], 2, 8, 128, 32, BF16, ao.E4M3)
        c.vs[c.table[0, 1].long()] = 0.0
        c.vs[c.table[0, 3].long()] = 2.0 ** -64
        c.ks[c.table[0, 2].long()] = 0.0
        run(m, c)
        c.vs[:] = 0.0
        d = c.cuda()
        call(m, c, d)
        m.lsa_check_device()
        assert (d["out"][:n] == 0).all() and torch.isfinite(d["lse_out"][:n]).all()


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("H,Hq,D", [(2, 32, 128), (1, 5, 64), (4, 4, 32), (1, 64, 128)])
def test_core_attention(m, dt, H, Hq, D):
    for k, entries, fetched, fresh in ((16, [100, 30, 64], [40, 0, 64], 0), (33, [500, 7, 90], [100, 7, 1], 5),
                                       (300, [2000, 900, 400], [800, 320, 10], 16)):
        run(m, Case([1, 1, 1], [20, 500, 0], H, Hq, D, 16, dt, window=40, sinks=2).add_topk(k, entries, fetched, fresh))


@pytest.mark.parametrize("dt", [BF16, F32])
def test_core_attention_several_tokens_and_none(m, dt):
    """Each token has its own list; a sequence without tokens; a list of nothing but -1; the same entry twice."""
    c = Case([3, 0, 2], [20, 500, 64], 2, 16, 128, 64, dt, window=10, spare_rows=2)
    c.add_topk(50, [300, 100, 64], [100, 100, 60], 4)
    c.topk[1] = -1
    c.topk[0, 1] = c.topk[0, 0]
    run(m, c)


@pytest.mark.parametrize("dt", [BF16, F32])
def test_core_attention_flags_entries_that_are_nowhere(m, dt):
    from sparse_kv_cache_memoryindexer_b200 import LSAError
    c = Case([1, 1], [20, 50], 2, 16, 128, 64, dt, window=10)
    c.add_topk(50, [300, 100], [100, 60], 4)
    d = c.cuda()
    missing = sorted(set(range(300)) - set(c.idx[:100].tolist()))[5]
    d["topk_idx"][0, 3], d["topk_idx"][1, 7] = missing, 104
    call(m, c, d)
    with pytest.raises(LSAError, match="index"):
        m.lsa_check_device()
    c.topk[0, 3] = c.topk[1, 7] = -1
    check(c, d)


def test_core_attention_window_nothing_but_selected(m):
    """With every window page given back, the selected entries alone carry the row (and the pages are flagged)."""
    from sparse_kv_cache_memoryindexer_b200 import LSAError
    c = Case([1], [20], 2, 16, 128, 64, BF16, window=10).add_topk(70, [300], [100], 0)
    c.table[:] = -1
    d = c.cuda()
    call(m, c, d)
    with pytest.raises(LSAError, match="bad-page"):
        m.lsa_check_device()
    check(c, d, hidden=lambda b, j: True)


def test_replayed_graph_follows_the_lengths(m):
    """A captured call reads lengths, pages and lists at every replay; the workspace needs no reset between."""
    for cdt in (BF16, ao.E4M3, F32):
        c = Case([1, 1], [4000, 90], 1, 8, 128, 64, F32 if cdt == F32 else BF16, cdt, window=0)
        d, ws = c.cuda(), c.workspace(m)
        call(m, c, d, ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(m, c, d, ws)
        for old in ([4000, 90], [17, 4000], [0, 63], [2500, 2501]):
            c.old = old
            c.len.copy_(torch.tensor(old))
            c.table = torch.cat([c.table[:1], c.table[:1]])  # both read the first sequence's pages
            d["page_table"].copy_(c.table)
            d["cache_len"].copy_(c.len)
            g.replay()
            m.lsa_check_device()
            check(c, d)


def test_two_streams_with_their_own_workspaces(m):
    cases = [Case([1], [20000], 2, 16, 128, 64, BF16, cdt, seed=s) for s, cdt in ((1, BF16), (2, ao.E4M3))]
    ds = [c.cuda() for c in cases]
    wss = [c.workspace(m) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, d, ws, s in zip(cases, ds, wss, streams):
            call(m, c, d, ws, stream=s)
    torch.cuda.synchronize()
    m.lsa_check_device()
    for c, d in zip(cases, ds):
        check(c, d)


def test_the_same_bits_every_time(m):
    for c in (Case([1, 1], [20000, 300], 2, 16, 128, 64), Case([200], [900], 2, 16, 128, 64, cdt=ao.E4M3),
              Case([1], [5], 2, 16, 128, 64, window=8).add_topk(200, [900], [300], 0)):
        a = run(m, c, rows={(0, 0)})
        for _ in range(3):
            b = c.cuda()
            call(m, c, b)
            assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse_out"], b["lse_out"])


def test_pages_past_32_bits(m):
    """Pages whose elements lie beyond 2^32."""
    H, page, D = 8, 128, 128
    n_pages = (1 << 32) // (H * page * D) + 3
    for cdt, n in ((BF16, 1), (ao.E4M3, 1), (BF16, 40), (ao.E4M3, 40)):
        c = Case([n], [150], H, 16, D, page, BF16, cdt)
        want = run(m, c, rows={(0, 0)})
        d = c.cuda()
        for name in ("k_cache", "v_cache"):
            t = torch.empty((n_pages, H, page, D), dtype=torch.uint8 if cdt == ao.E4M3 else cdt, device="cuda")
            for j in range(c.max_pages):
                t[n_pages - 2 + j] = d[name][int(c.table[0, j])].view(t.dtype)
            d[name] = t.view(cdt)
        d["page_table"] = torch.arange(n_pages - 2, n_pages - 2 + c.max_pages, dtype=torch.int32, device="cuda")[None]
        if cdt == ao.E4M3:
            for s in ("k_scale", "v_scale"):
                t = torch.ones((n_pages, H), device="cuda")
                t[n_pages - 2:n_pages - 2 + c.max_pages] = d[s][c.table[0].long().cuda()]
                d[s] = t
        call(m, c, d)
        m.lsa_check_device()
        assert torch.equal(d["out"], want["out"])
        del d
        torch.cuda.empty_cache()


def test_core_attention_long_fetch_lists(m):
    """Fetch lists longer than the shared memory that they are searched in: every 2^i-th entry of them."""
    for dt, D, fetched in ((BF16, 32, [15000, 6140, 6145]), (BF16, 64, [30000, 1, 0])):
        c = Case([1, 1, 1], [20, 500, 0], 2, 4, D, 16, dt, window=40, sinks=2)
        c.add_topk(100, [40000, 9000, 7000], fetched, 3)
        run(m, c)


def test_core_attention_of_many_users_and_full_lists(m):
    """Shared out over the CTAs instead of clusters (long lists, a long window), and 4096 entries a token."""
    c = Case([1] * 5, [9000, 0, 40, 5000, 100], 2, 16, 64, 64, BF16, window=5000, sinks=1)
    run(m, c.add_topk(4096, [6000] * 5, [5000, 4095, 10, 4100, 0], 4))


def test_many_sequences(m):
    """More sequences than a CTA has threads, empty ones among them, in both ways of sharing the work."""
    new = [(i * 7) % 3 for i in range(300)]
    old = [(i * 37) % 200 for i in range(300)]
    rows = {(b, i) for b in range(0, 300, 23) for i in range(new[b])} | {(299, i) for i in range(new[299])}
    for cdt, window in ((BF16, 0), (BF16, 60), (ao.E4M3, 0), (F32, 50)):
        run(m, Case(new, old, 1, 4, 64, 16, F32 if cdt == F32 else BF16, cdt, window=window), rows)
    old[17] = 20000
    run(m, Case(new, old, 1, 4, 64, 128, BF16, BF16), rows | {(17, i) for i in range(new[17])})


def test_negative_and_zero_scale(m):
    """softmax_scale may have any sign; zero weighs every visible key alike."""
    for n in (1, 50):
        for cdt in (BF16, ao.E4M3, F32):
            for scale in (-0.3, 0.0):
                c = Case([n, n], [100, 7], 2, 8, 64, 32, F32 if cdt == F32 else BF16, cdt, window=60, sinks=2)
                c.scale = scale
                d = c.cuda()
                call(m, c, d, softmax_scale=scale)
                m.lsa_check_device()
                out, lse = d["out"].cpu().double(), d["lse_out"].cpu().double()
                assert torch.isfinite(out).all() and torch.isfinite(lse).all()
                check_signed(c, out, lse)


def check_signed(case, out, lse):
    G = case.Hq // case.H
    p_dtype = {BF16: BF16, F32: None, ao.E4M3: torch.float16}[case.cdt]
    for b, (n, old) in enumerate(zip(case.new, case.old)):
        for i in {0, n // 2, n - 1}:
            j = torch.tensor(ao.visible(old + i, old + n, case.window, case.sinks))
            pg, sl = case.table[b].long()[j // case.page], j % case.page
            at = int(case.offs[b]) + i
            for hq in range(case.Hq):
                h = hq // G
                K, V = case.kc[pg, :, sl][:, h].double(), case.vc[pg, :, sl][:, h].double()
                if case.ks is not None:
                    K, V = K * case.ks[pg, h].double()[:, None], V * case.vs[pg, h].double()[:, None]
                o, l_, A, mag = ao.attend(case.q[at, hq].double(), K, V, case.scale)
                bo, bl = ao.attend_bounds(o, A, abs(mag), K.shape[0], case.D, case.dt, p_dtype)
                assert ((out[at, hq] - o).abs() <= bo).all(), (b, i, hq)
                assert abs(float(lse[at, hq]) - l_) <= bl, (b, i, hq)


def test_no_tokens_and_no_entries(m):
    """N = 0 (empty tensors) does nothing; without a single fetched entry the fresh ones still count."""
    c = Case([0, 0], [30, 4], 2, 4, 64, 16)
    d = c.cuda()
    call(m, c, d)
    c = Case([1, 1], [30, 4], 2, 16, 64, 16, window=20).add_topk(8, [0, 0], [0, 0], 5)
    run(m, c)
    m.lsa_check_device()


def test_bad_length_with_nan_ends(m):
    """A length far behind the page table, on rows that come out as NaN: flagged, and the way out for such rows
    does not walk positions that have no page."""
    from sparse_kv_cache_memoryindexer_b200 import LSAError
    for n in (3, 40):
        c = Case([n], [100], 1, 8, 64, 16)
        d = c.cuda()
        d["v_cache"][:] = math.nan
        d["cache_len"][0] = 2000000000
        call(m, c, d)
        with pytest.raises(LSAError, match="count"):
            m.lsa_check_device()


# The kernel for many rows is taken where it is the faster one, which the small cases above are not: here they
# run on it wherever it can take them (and the large ones on the other).

@pytest.fixture
def many_rows(monkeypatch):
    monkeypatch.setenv("LSA_ATTN_MANY", "1")


@pytest.fixture
def few_rows(monkeypatch):
    monkeypatch.setenv("LSA_ATTN_MANY", "0")


@pytest.mark.parametrize("cdt", [BF16, ao.E4M3])
@pytest.mark.parametrize("H,Hq,D,page", [(1, 1, 64, 16), (2, 16, 128, 64), (1, 7, 128, 32), (2, 64, 64, 128), (3, 12, 128, 128)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (37, 4), (200, 130), (1, 0)])
def test_many_rows_chunks(m, many_rows, cdt, H, Hq, D, page, window, sinks):
    test_chunks(m, BF16, cdt, H, Hq, D, page, window, sinks)


@pytest.mark.parametrize("cdt", [BF16, ao.E4M3])
@pytest.mark.parametrize("H,Hq", [(1, 1), (2, 14), (1, 64), (8, 64)])
def test_many_rows_one_token(m, many_rows, cdt, H, Hq):
    test_one_token(m, BF16, cdt, H, Hq)


@pytest.mark.parametrize("cdt", [BF16, ao.E4M3])
def test_many_rows_long_caches(m, many_rows, cdt):
    test_long_caches_of_unlike_lengths(m, BF16, cdt, 1, 8)
    test_chunk_on_a_long_history(m, cdt)


@pytest.mark.parametrize("cdt", [BF16, ao.E4M3])
def test_few_rows_kernel_takes_chunks(m, few_rows, cdt):
    test_chunk_on_a_long_history(m, cdt)


@pytest.mark.parametrize("cdt", [BF16, ao.E4M3])
@pytest.mark.parametrize("n", [1, 3, 70, 300])
def test_many_rows_unused_slots(m, many_rows, cdt, n):
    test_what_lies_in_unused_slots_does_not_matter(m, cdt, n)


@pytest.mark.parametrize("cdt", [BF16, ao.E4M3])
def test_many_rows_nan(m, many_rows, cdt):
    test_a_later_tokens_nan_stays_out_of_earlier_rows(m, cdt)


def test_many_rows_bad_data_and_the_rest(m, many_rows):
    test_strided_queries_and_no_lse(m)
    test_large_scores_and_scale(m)
    test_rows_with_nothing_to_see(m)
    test_bad_data_is_left_out_and_flagged(m)
    test_zero_scales(m)
    test_many_sequences(m)
    test_negative_and_zero_scale(m)
    test_replayed_graph_follows_the_lengths(m)
    test_two_streams_with_their_own_workspaces(m)
    test_the_same_bits_every_time(m)
    test_pages_past_32_bits(m)
    test_no_tokens_and_no_entries(m)
    test_bad_length_with_nan_ends(m)
