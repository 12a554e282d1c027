"""Every key counts, once: long caches whose work is split over CTAs, warps, pages and chunks and joined again, where a
lost or doubled chunk would hide below a bound that grows with the number of keys."""
import math

import pytest
import torch

import attn_oracle as ao
from test_gpu_attention import BF16, F32, Case, call

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sparse_kv_cache_memoryindexer_b200 as mod
    mod.lsa_check_device()
    return mod


@pytest.fixture(params=["0", "1"], ids=["few", "many"])
def kernel(request, monkeypatch):
    monkeypatch.setenv("LSA_ATTN_MANY", request.param)


def unit_scales(c):
    if c.cdt == ao.E4M3:
        c.ks.fill_(1.0)
        c.vs.fill_(1.0)
    return c


def seen(pos, window, sinks):
    j = torch.arange(pos + 1)
    return j[(j > pos - window) | (j < sinks)] if window else j


def place(c, b, cache, rows):
    """rows [n][H][D] into the slots of positions 0 .. n - 1 of sequence b."""
    j = torch.arange(rows.shape[0])
    pg, sl = c.table[b].long()[j // c.page], j % c.page
    view = torch.uint8 if c.cdt == ao.E4M3 else c.cdt
    cache.view(view)[pg, :, sl] = rows.to(c.cdt).view(view)


CASES = [([1, 1, 1], [30001, 17, 9000], 8, 8, 0, 0), ([1], [65004], 1, 8, 0, 0), ([1, 1], [20000, 5000], 2, 32, 7001, 37),
         ([40, 3], [11990, 30000], 1, 8, 0, 0), ([300], [8000], 2, 8, 3000, 100), ([700, 2], [0, 12000], 1, 4, 0, 0)]


@pytest.mark.parametrize("cdt", [BF16, F32, ao.E4M3])
@pytest.mark.parametrize("new,old,H,Hq,window,sinks", CASES)
@pytest.mark.parametrize("D,page", [(128, 64), (64, 16)])
def test_equal_weights_count_the_keys(m, kernel, cdt, new, old, H, Hq, window, sinks, D, page):
    """A query of zero weighs every visible key alike: lse is log n, and of one-hot values each dimension is the share of
    its class of keys.  Weights are one and their sums whole numbers (E4M3: times 2^15 or 2^7), so lse is off by log2's one
    ulp (2^-19 for a number up to 2^32) and two roundings of numbers up to 17 (2^-20 each), times log 2, which is below
    2^-18; a share by its division and the output's rounding."""
    c = unit_scales(Case(new, old, H, Hq, D, page, F32 if cdt == F32 else BF16, cdt, window=window, sinks=sinks, only_needed=False))
    c.q.zero_()
    classes = [(torch.arange(c.max_pages * page) * (2 * h + 1)) // (1, 16, 7)[h % 3] % D for h in range(H)]
    for b, (n, o) in enumerate(zip(new, old)):
        hot = torch.zeros((n + o, H, D))
        for h in range(H):
            hot[torch.arange(n + o), h, classes[h][:n + o]] = 1.0
        place(c, b, c.vc, hot)
    d = c.cuda()
    call(m, c, d)
    m.lsa_check_device()
    out, lse = d["out"].cpu().double(), d["lse_out"].cpu().double()
    step = ao.half_step(c.dt) + 2.0 ** -22
    for b, (n, o) in enumerate(zip(new, old)):
        for i in range(n):
            j = seen(o + i, window, sinks)
            at = int(c.offs[b]) + i
            assert (lse[at] - math.log(j.numel())).abs().max() <= 2.0 ** -18, (b, i)  # (a key more or less: 2^-16)
            for h in range(H):
                share = torch.bincount(classes[h][j], minlength=D).double() / j.numel()
                got = out[at, h * (Hq // H):(h + 1) * (Hq // H)]
                assert ((got - share).abs() <= step * share).all(), (b, i, h)


@pytest.mark.parametrize("cdt", [BF16, F32, ao.E4M3])
@pytest.mark.parametrize("n,old,window,sinks", [(1, 30000, 0, 0), (31, 29970, 0, 0), (9, 7990, 5003, 70)])
def test_each_chunk_has_its_key_found(m, kernel, cdt, n, old, window, sinks):
    """A key of every 16-key chunk in turn has a score so far above the others that the row is its value.  (Keys of +-1: the
    chosen one scores 3 * 128^0.5 = 34, the others 3 at one standard deviation: the 30,000 of them weigh
    30,000 e^(9/2 - 34) = 5e-9 together, and even at six deviations one weighs e^(18 - 34) = 1e-7.)"""
    Hq, D, page = 64, 128, 64
    g = torch.Generator().manual_seed(old + n)
    c = unit_scales(Case([n], [old], 1, Hq, D, page, F32 if cdt == F32 else BF16, cdt, window=window, sinks=sinks))
    total = old + n
    K = torch.randint(0, 2, (total, 1, D), generator=g).float() * 2 - 1
    V = (torch.randint(-7, 8, (total, 1, D), generator=g) / 4.0)
    mapped = c.table[0].long()[torch.arange(total) // page] >= 0
    j = torch.arange(total)[mapped]
    view = torch.uint8 if cdt == ao.E4M3 else c.cdt
    for cache, rows in ((c.kc, K), (c.vc, V)):
        cache.view(view)[c.table[0].long()[j // page], :, j % page] = rows[j].to(c.cdt).view(view)
    chunks = [x for x in range(-(-total // 16)) if not window or x * 16 < sinks or x * 16 + 16 > old - window]
    targets = [min(16 * x + (7 * x + 3) % 16, total - 1) for x in chunks]
    rows = n * Hq
    for at in range(0, len(targets), rows):
        some = targets[at:at + rows]
        q = torch.zeros((rows, D))
        q[:len(some)] = 3 * K[some, 0]
        c.q = q.view(n, Hq, D).to(c.dt)
        d = c.cuda()
        call(m, c, d)
        m.lsa_check_device()
        out = d["out"].cpu().float().view(rows, D)
        for r, p in enumerate(some):
            pos = old + r // Hq
            if p > pos or window and sinks <= p <= pos - window:
                continue  # (masked for this row)
            assert (out[r] - V[p, 0]).abs().max() <= 2.0 ** -7, (r, p)
