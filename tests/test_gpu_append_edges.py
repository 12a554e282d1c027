"""lsa_kv_append on bad data and at angles where a rounding would show.  Against the definition in 64 bits."""
import math

import pytest
import torch

import attn_oracle as ao
from test_gpu_window_cache import Case, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sparse_kv_cache_memoryindexer_b200 as mod
    mod.lsa_check_device()
    return mod


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf, -0.25])
@pytest.mark.parametrize("n", [1, 40])
def test_append_leaves_a_page_with_a_bad_scale(m, bad, n):
    """A page that holds tokens under a scale that is none: flagged, codes and scale as they were, for that head and
    tensor; the other heads, the other tensor and the pages after it are written."""
    from sparse_kv_cache_memoryindexer_b200 import LSAError
    c = Case(new=[n], old=[21], H=2, Hq=2, D=64, page=16, cdt=ao.E4M3)
    d = c.cuda()
    pg = int(c.table[0, 1])
    d["v_scale"][pg, 1] = bad
    m.lsa_kv_append(**d)
    with pytest.raises(LSAError, match="scale"):
        m.lsa_check_device()
    same = lambda a, b: torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8))  # noqa: E731
    assert same(d["v_cache"][pg, 1], c.vc[pg, 1])
    got = float(d["v_scale"][pg, 1])
    assert got == bad or math.isnan(got) and math.isnan(bad)
    # everything else, as where the scale was good
    e = c.cuda()
    m.lsa_kv_append(**e)
    m.lsa_check_device()
    check(c, e)
    for t in ("k_cache", "v_cache", "k_scale", "v_scale"):
        d[t][pg, 1] = e[t][pg, 1] if t.startswith("v") else d[t][pg, 1]
        assert torch.equal(d[t].view(torch.uint8), e[t].view(torch.uint8)), t
    assert torch.equal(d["q_out"], e["q_out"])


@pytest.mark.parametrize("B", [3, 400])
def test_append_with_offsets_that_decrease(m, B):
    """Offsets that go back are flagged; a token that two sequences then claim goes to the last one's place, whole, and no
    other slot is touched.  (400 sequences: more than a block has threads, the last ones empty.)"""
    from sparse_kv_cache_memoryindexer_b200 import LSAError
    old = [7, 3, 9] + [1] * (B - 3)
    c = Case(new=[5, 2, 5] + [0] * (B - 3), old=old, H=2, Hq=2, D=64, page=16)
    d = c.cuda()
    offs = torch.tensor([0, 5, 3, 8] + [8] * (B - 3))  # sequence 0: tokens 0 .. 4; 1: none, bad; 2: tokens 3 .. 7
    d["q_offsets"].copy_(offs)
    for _ in range(3):
        m.lsa_kv_append(**d)
        with pytest.raises(LSAError, match="offsets"):
            m.lsa_check_device()
        for t, cache in (("k", c.kc), ("v", c.vc)):
            want = cache.clone()
            src = c.parts()[1 if t == "k" else 2]
            for n in range(8):
                b = 0 if n < 3 else 2
                p = old[b] + n - int(offs[b])
                pg, sl = int(c.table[b, p // 16]), p % 16
                got = d[t + "_cache"][pg, :, sl].cpu()
                if t == "v":
                    assert torch.equal(got, src[n]), n
                else:
                    y, mag = ao.rotate(src[n].double(), p, c.inv_freq, False)
                    err = mag * ao.ROTATION
                    assert ((got.double() - y).abs() <= err + ao.half_step(c.dt) * (y.abs() + err)).all(), n
                want[pg, :, sl] = got
            assert torch.equal(d[t + "_cache"].cpu(), want)


def test_append_angles_are_not_rounded_to_fp32(m):
    """At angles next to a quarter turn the cosine is small, and its error shows how far off the angle is: a reduced angle
    rounded to fp32 (2^-25 of a half turn, 9e-8) would leave 1e-5 of a cosine of 0.01.  The cosine itself is within 2 ulp
    (2^-22), what puts the rounding back adds half an ulp, and the product in fp64 of a thousand positions leaves 1e-12."""
    H, D, page, n = 1, 128, 16, 200
    c = Case(new=[n], old=[900], H=H, Hq=1, D=D, page=page, dt=torch.float32)
    j = torch.arange(D // 2, dtype=torch.float64)
    c.inv_freq = ((math.pi * (150 + j) + math.pi / 2 + 0.002 + 0.008 * (j % 17) / 17) / 1000).float()
    for half, want in ((0, torch.cos), (1, torch.sin)):
        c.fused.zero_()
        c.fused[:, :, half * (D // 2):half * (D // 2) + D // 2] = 1.0
        d = c.cuda()
        m.lsa_kv_append(**d)
        m.lsa_check_device()
        a = (900 + torch.arange(n, dtype=torch.float64))[:, None] * c.inv_freq.double()[None]
        cos = torch.cos(a)
        got = d["q_out"][:, 0].cpu().double()
        # x = (1, 0): (cos, sin);  x = (0, 1): (-sin, cos)
        y = got[:, :D // 2] if half == 0 else got[:, D // 2:]
        p = torch.arange(900, 900 + n)
        k = d["k_cache"][c.table[0].long()[p // page], 0, p % page].cpu().double()
        yk = k[:, :D // 2] if half == 0 else k[:, D // 2:]
        near = (cos.abs() < 0.02) & (cos.abs() > 1e-3)
        assert near.sum() >= 64
        for v in (y, yk):
            assert ((v - cos).abs()[near] <= (2.0 ** -22 + 2.0 ** -24) * cos.abs()[near] + 1e-12).all()
            assert ((v - cos).abs() <= 2.0 ** -22).all()
