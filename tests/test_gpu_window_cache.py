"""lsa_kv_append against its definition in 64 bits (tests/attn_oracle.py)."""
import math

import pytest
import torch

import attn_oracle as ao

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sparse_kv_cache_memoryindexer_b200 as mod
    mod.lsa_check_device()
    return mod


class Case:
    """Inputs on the CPU, and the cache with pages in a shuffled order (spare pages at the end)."""

    def __init__(self, new, old, H, Hq, D, page, dt=torch.bfloat16, cdt=None, rot=None, interleaved=False, seed=1,
                 spare_rows=0, scale_exp=(-6, -3)):
        g = torch.Generator().manual_seed(seed)
        self.new, self.old, self.H, self.Hq, self.D, self.page = new, old, H, Hq, D, page
        self.dt, self.cdt, self.interleaved = dt, cdt or dt, interleaved
        B, self.N = len(new), sum(new) + spare_rows
        self.offs = torch.tensor([0] + list(torch.tensor(new).cumsum(0)), dtype=torch.int64)
        self.len = torch.tensor(old, dtype=torch.int32)
        need = [max(1, -(-(o + n) // page)) for o, n in zip(old, new)]
        self.max_pages = max(need)
        order = torch.randperm(sum(need), generator=g)
        self.n_pages = sum(need) + 2
        self.table = torch.full((B, self.max_pages), -1, dtype=torch.int32)
        at = 0
        for b, k in enumerate(need):
            self.table[b, :k] = order[at:at + k].to(torch.int32)
            at += k
        rot = D if rot is None else rot
        self.inv_freq = None if rot == 0 else (1e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float()
        self.fused = torch.randn((self.N, Hq + 2 * H, D), generator=g).to(dt)
        shape = (self.n_pages, H, page, D)
        if self.cdt == ao.E4M3:
            self.kc = (torch.randn(shape, generator=g) * 60).clamp(-448, 448).to(ao.E4M3)
            self.vc = (torch.randn(shape, generator=g) * 60).clamp(-448, 448).to(ao.E4M3)
            self.ks = torch.exp2(torch.randint(*scale_exp, (self.n_pages, H), generator=g).float())
            self.vs = torch.exp2(torch.randint(*scale_exp, (self.n_pages, H), generator=g).float())
        else:
            self.kc, self.vc = torch.randn(shape, generator=g).to(self.cdt), torch.randn(shape, generator=g).to(self.cdt)
            self.ks = self.vs = None

    def parts(self):
        f = self.fused
        return f[:, :self.Hq], f[:, self.Hq:self.Hq + self.H], f[:, self.Hq + self.H:]

    def cuda(self):
        up = lambda t: None if t is None else t.cuda()  # noqa: E731
        f = self.fused.cuda()
        d = dict(q=f[:, :self.Hq], k=f[:, self.Hq:self.Hq + self.H], v=f[:, self.Hq + self.H:], q_offsets=up(self.offs),
                 cache_len=up(self.len), page_table=up(self.table), k_cache=up(self.kc), v_cache=up(self.vc),
                 k_scale=up(self.ks), v_scale=up(self.vs), inv_freq=up(self.inv_freq), interleaved=self.interleaved,
                 q_out=torch.full((self.N, self.Hq, self.D), 77.0, dtype=self.dt, device="cuda"))
        return d


def check(case, d):
    """Every row of q_out, every slot of the caches and every scale."""
    q, k, v = case.parts()
    page, H = case.page, case.H
    got = {n: d[n + "_cache"].cpu() for n in ("k", "v")}
    want = {"k": case.kc.double(), "v": case.vc.double()}
    scales = {"k": case.ks, "v": case.vs}
    tol = {n: torch.zeros_like(want[n]) for n in ("k", "v")}
    exp_scale = {n: None if scales[n] is None else scales[n].double().clone() for n in ("k", "v")}
    qo = d["q_out"].cpu().double()
    step = ao.half_step(case.dt)
    assert (qo[sum(case.new):] == 77.0).all(), "rows behind the last sequence"
    for b, (n, old) in enumerate(zip(case.new, case.old)):
        at = int(case.offs[b])
        ys = {"k": [], "v": []}
        for i in range(n):
            y, mag = ao.rotate(q[at + i].double(), old + i, case.inv_freq, case.interleaved)
            err = (qo[at + i] - y).abs()
            bound = mag * ao.ROTATION
            assert (err <= bound + step * (y.abs() + bound)).all(), (b, i)
            ys["k"].append(ao.rotate(k[at + i].double(), old + i, case.inv_freq, case.interleaved))
            vd = v[at + i].double()
            ys["v"].append((vd, torch.zeros_like(vd)))
        for j in range(old // page, (old + n - 1) // page + 1 if n else 0):
            lo, hi = max(old, j * page), min(old + n, (j + 1) * page)
            pg, a, z = int(case.table[b, j]), lo - j * page, hi - j * page
            for t in ("k", "v"):
                y = torch.stack([ys[t][p - old][0] for p in range(lo, hi)], 1)      # [H][tokens][D]
                err = torch.stack([ys[t][p - old][1] for p in range(lo, hi)], 1) * ao.ROTATION
                if scales[t] is None:
                    want[t][pg, :, a:z], tol[t][pg, :, a:z] = y, err + ao.half_step(case.cdt) * (y.abs() + err)
                    continue
                for h in range(H):
                    finite = y[h][torch.isfinite(y[h])]
                    amax = float(finite.abs().max()) if finite.numel() else 0.0
                    # (a value that is not rotated is exact: it may stand on the border)
                    near = bool(err[h].any()) and ao.pow2_scale(amax * (1 + 2e-6)) != ao.pow2_scale(amax * (1 - 2e-6))
                    assert not near, "the case's amax must not stand on a power of two times 448"
                    before = float(scales[t][pg, h])
                    now = max(ao.pow2_scale(amax), before) if a else ao.pow2_scale(amax)
                    exp_scale[t][pg, h] = now
                    old_rows = want[t][pg, h, :a] * (before / now)
                    want[t][pg, h, :a] = old_rows
                    if now != before:  # rounded again to the larger scale
                        tol[t][pg, h, :a] = ao.e4m3_bound(old_rows, 1.0)
                    x = y[h] / now
                    want[t][pg, h, a:z] = x.clamp(-448, 448)
                    tol[t][pg, h, a:z] = torch.nan_to_num(ao.e4m3_bound(x, 1.0) + err[h] / now, nan=0.0, posinf=0.0)
    for t in ("k", "v"):
        if exp_scale[t] is not None:
            assert torch.equal(d[t + "_scale"].cpu().double(), exp_scale[t]), t
        g = got[t].double()
        same_nan = torch.isnan(g) == torch.isnan(want[t])
        assert same_nan.all(), t
        err = torch.nan_to_num(g - want[t]).abs()
        assert (err <= tol[t]).all(), (t, float((err - tol[t]).max()))


def run(m, case, **over):
    d = case.cuda()
    d.update(over)
    m.lsa_kv_append(**d)
    m.lsa_check_device()
    return d


TYPES = [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32), (torch.bfloat16, ao.E4M3)]


@pytest.mark.parametrize("dt,cdt", TYPES)
@pytest.mark.parametrize("page,D", [(16, 32), (64, 128), (128, 64), (32, 128), (128, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append(m, dt, cdt, page, D, interleaved):
    c = Case(new=[1, 0, 37, 130, 2], old=[0, 5, page - 1, 3 * page + 7, 2 * page], H=2, Hq=6, D=D, page=page, dt=dt,
             cdt=cdt, interleaved=interleaved, spare_rows=3, seed=page + D)
    check(c, run(m, c))


@pytest.mark.parametrize("dt,cdt", TYPES)
@pytest.mark.parametrize("rot", [0, 16, 64])
def test_append_partial_rotation(m, dt, cdt, rot):
    for interleaved in (False, True):
        c = Case(new=[3, 20], old=[77, 1], H=1, Hq=5, D=128, page=32, dt=dt, cdt=cdt, rot=rot, interleaved=interleaved)
        check(c, run(m, c))


@pytest.mark.parametrize("dt,cdt", TYPES)
def test_append_far_positions(m, dt, cdt):
    """A million tokens back: pages outside the table's used part are never looked at."""
    c = Case(new=[2], old=[3], H=2, Hq=2, D=128, page=64, dt=dt, cdt=cdt)
    far = 1048573
    c.old = [far]
    c.len = torch.tensor([far], dtype=torch.int32)
    c.max_pages = (far + 2) // 64 + 1
    table = torch.full((1, c.max_pages), -1, dtype=torch.int32)
    table[0, far // 64], table[0, (far + 1) // 64] = 0, 0
    c.table = table
    check(c, run(m, c))


def test_append_one_token_steps_many_users(m):
    c = Case(new=[1] * 70, old=[(37 * i) % 300 for i in range(70)], H=4, Hq=8, D=64, page=16)
    check(c, run(m, c))


def test_append_queries_in_place_and_without_queries(m):
    c = Case(new=[5, 9], old=[1, 60], H=2, Hq=4, D=64, page=16)
    d = c.cuda()
    q = d["q"].contiguous()
    d["q"] = d["q_out"] = q
    m.lsa_kv_append(**d)
    m.lsa_check_device()
    check(c, d)
    d2 = c.cuda()
    d2.update(q=None, q_out=None)
    m.lsa_kv_append(**d2)
    m.lsa_check_device()
    assert torch.equal(d2["k_cache"], d["k_cache"]) and torch.equal(d2["v_cache"], d["v_cache"])


def test_append_e4m3_scale_grows_over_calls(m):
    """The same page filled by four calls, each louder than the one before, then one that is quiet."""
    page, D = 32, 64
    c = Case(new=[3], old=[0], H=2, Hq=2, D=D, page=page, cdt=ao.E4M3)
    d = c.cuda()
    for i, loud in enumerate((0.01, 1.0, 30.0, 5000.0, 0.5)):
        c.old, c.len = [3 * i], torch.tensor([3 * i], dtype=torch.int32)
        c.max_pages = 1
        c.fused = (torch.randn((3, 6, D), generator=torch.Generator().manual_seed(i)) * loud).bfloat16()
        c.kc, c.vc, c.ks, c.vs = (d[n].cpu() for n in ("k_cache", "v_cache", "k_scale", "v_scale"))
        f = c.fused.cuda()
        d.update(q=f[:, :2], k=f[:, 2:4], v=f[:, 4:], cache_len=c.len.cuda(),
                 q_out=torch.full((3, 2, D), 77.0, dtype=torch.bfloat16, device="cuda"))
        m.lsa_kv_append(**d)
        m.lsa_check_device()
        check(c, d)


def test_append_e4m3_zeros_infinities_nan(m):
    c = Case(new=[4, 2], old=[0, 10], H=2, Hq=2, D=32, page=16, cdt=ao.E4M3, rot=0)
    _, k, v = c.parts()
    k[0:4, 0] = 0                       # a page of zeros: the least scale
    v[1, 1, 3], v[2, 1, 4] = math.inf, -math.inf
    v[0, 1, 5] = math.nan
    k[4, 1] = math.nan                  # a token of nothing but NaN sets no scale
    check(c, run(m, c))


def test_append_is_repeatable_and_replayable(m):
    """The same call twice gives the same bits; so does its capture in a graph, on another stream."""
    for cdt in (torch.bfloat16, ao.E4M3):
        c = Case(new=[1, 40, 3], old=[7, 100, 63], H=2, Hq=4, D=128, page=64, cdt=cdt)
        a, b = run(m, c), c.cuda()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                m.lsa_kv_append(**b)
        torch.cuda.synchronize()
        for _ in range(2):
            g.replay()
        torch.cuda.synchronize()
        m.lsa_check_device()
        for n in ("q_out", "k_cache", "v_cache"):
            assert torch.equal(a[n].view(torch.uint8), b[n].view(torch.uint8)), n


def test_append_flags_bad_data(m):
    """Bad pages, lengths and offsets are skipped: nothing is written for them."""
    from sparse_kv_cache_memoryindexer_b200 import LSAError
    for cdt in (torch.bfloat16, ao.E4M3):
        for what, flag in (("page", "bad-page"), ("unmapped", "bad-page"), ("length", "count"), ("behind", "count"),
                           ("offsets", "offsets")):
            c = Case(new=[2, 3], old=[4, 9], H=2, Hq=2, D=64, page=16, cdt=cdt)
            d = c.cuda()
            if what == "page":
                d["page_table"][1, 0] = c.n_pages
            elif what == "unmapped":
                d["page_table"][1, 0] = -1
            elif what == "length":
                d["cache_len"][1] = -4
            elif what == "behind":
                d["cache_len"][1] = 16 * c.max_pages
            else:
                d["q_offsets"][2] = c.N + 5
            m.lsa_kv_append(**d)
            with pytest.raises(LSAError, match=flag):
                m.lsa_check_device()
            pg = int(c.table[1, 0])
            assert torch.equal(d["k_cache"][pg].view(torch.uint8).cpu(), c.kc[pg].view(torch.uint8)), what
            m.lsa_check_device()


def test_append_past_32_bits(m):
    """Pages whose elements lie beyond 2^32."""
    H, page, D = 8, 128, 128
    n_pages = (1 << 32) // (H * page * D) + 3
    for cdt in (torch.bfloat16, ao.E4M3):
        c = Case(new=[3], old=[126], H=H, Hq=8, D=D, page=page, cdt=cdt)
        d = c.cuda()
        big = {}
        for n in ("k", "v"):
            t = torch.empty((n_pages, H, page, D), dtype=torch.uint8 if cdt == ao.E4M3 else cdt, device="cuda")
            big[n] = t.view(cdt) if cdt == ao.E4M3 else t
            for j in range(2):
                t[n_pages - 2 + j] = d[n + "_cache"][int(c.table[0, j])].view(t.dtype)
        d.update(k_cache=big["k"], v_cache=big["v"], page_table=torch.tensor([[n_pages - 2, n_pages - 1]], dtype=torch.int32,
                                                                             device="cuda"))
        if cdt == ao.E4M3:
            for n in ("k", "v"):
                s = torch.ones((n_pages, H), device="cuda")
                s[n_pages - 2:] = d[n + "_scale"][c.table[0].long().cuda()]
                d[n + "_scale"] = s
        m.lsa_kv_append(**d)
        m.lsa_check_device()
        e = run(m, c)
        for n in ("k", "v"):
            for j in range(2):
                assert torch.equal(d[n + "_cache"][n_pages - 2 + j].view(torch.uint8),
                                   e[n + "_cache"][int(c.table[0, j])].view(torch.uint8))
        del d, big
        torch.cuda.empty_cache()
