"""Core attention where a kernel leaves its common path: rows that are done again key by key, scales at the ends of
their range, infinities that a query may see, lengths behind the page table.  Against the definition in 64 bits, on
both kernels (LSA_ATTN_MANY) where both can take the call."""
import math

import pytest
import torch

import attn_oracle as ao
import test_gpu_attention
from test_gpu_attention import BF16, F32, Case, call, check

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


@pytest.mark.parametrize("n", [9, 60])
def test_bad_scale_on_rows_that_are_done_again(m, kernel, n):
    """A token of NaN behind the first rows sends them through the key-by-key way; a page with a NaN scale is left out
    there too."""
    from sparse_kv_cache_memoryindexer_b200 import LSAError
    c = Case([n], [100], 2, 8, 64, 16, BF16, ao.E4M3)
    d = c.cuda()
    pg, last = int(c.table[0, 2]), 100 + n - 1
    d["v_scale"][pg] = math.nan
    d["v_cache"].view(torch.uint8)[int(c.table[0, last // 16]), :, last % 16] = 0x7F
    call(m, c, d)
    with pytest.raises(LSAError, match="scale"):
        m.lsa_check_device()
    check(c, d, rows={(0, i) for i in range(n - 1)}, hidden=lambda b, j: j // 16 == 2)


@pytest.mark.parametrize("cdt", [BF16, ao.E4M3])
@pytest.mark.parametrize("old", [40, 9000])
def test_a_query_of_nan_gives_nan(m, kernel, cdt, old):
    """With its keys in one part or split over many; the rows beside it are as ever."""
    c = Case([3, 20], [old, 5], 2, 8, 64, 64, BF16, cdt)
    d = c.cuda()
    d["q"][1, 5] = math.nan
    d["q"][9] = math.nan
    call(m, c, d)
    m.lsa_check_device()
    for n, heads in ((1, [5]), (9, range(8))):
        for h in heads:
            assert torch.isnan(d["out"][n, h]).all() and torch.isnan(d["lse_out"][n, h]), (n, h)
    check(c, d, rows={(0, 0), (0, 2), (1, 0), (1, 5), (1, 7), (1, 19)})
    assert not torch.isnan(d["out"][1, :5]).any() and not torch.isnan(d["out"][1, 6:]).any()


@pytest.mark.parametrize("cdt", [BF16, F32, ao.E4M3])
@pytest.mark.parametrize("n", [1, 3, 20])
def test_length_behind_an_odd_number_of_pages(m, kernel, cdt, n):
    """A length that takes the tokens past the page table's end (an odd number of 16-key pages): flagged, and the rows see
    what the table holds, once."""
    from sparse_kv_cache_memoryindexer_b200 import LSAError
    c = Case([n], [112 - n], 2, 8, 64, 16, F32 if cdt == F32 else BF16, cdt)
    assert c.max_pages == 7
    d = c.cuda()
    d["cache_len"][0] = 115
    call(m, c, d)
    with pytest.raises(LSAError, match="count"):
        m.lsa_check_device()
    for i in range(n):  # (every row stands behind position 111)
        check_row(c, d, i, range(112))


def check_row(c, d, i, keys):
    """Row i of a case of one sequence, which sees `keys`."""
    j = torch.tensor(list(keys))
    pg, sl = c.table[0].long()[j // c.page], j % c.page
    for hq in range(c.Hq):
        h = hq // (c.Hq // c.H)
        K, V = c.kc[pg, :, sl][:, h].double(), c.vc[pg, :, sl][:, h].double()
        if c.ks is not None:
            K, V = K * c.ks[pg, h].double()[:, None], V * c.vs[pg, h].double()[:, None]
        o, l_, A, mag = ao.attend(c.q[i, hq].double(), K, V, c.scale)
        bo, bl = ao.attend_bounds(o, A, mag, j.numel(), c.D, c.dt, {BF16: BF16, F32: None, ao.E4M3: torch.float16}[c.cdt])
        assert ((d["out"][i, hq].cpu().double() - o).abs() <= bo).all(), (i, hq)
        assert abs(float(d["lse_out"][i, hq]) - l_) <= bl, (i, hq)


# value scales of pages beside one another
MIXED = [(0.0, 2.0 ** -20), (0.0, 2.0 ** -40), (0.0, 2.0 ** -100), (0.0, 2.0 ** 100), (2.0 ** -64, 2.0 ** 40),
         (2.0 ** -64, 2.0 ** 70), (2.0 ** -100, 2.0 ** 118), (2.0 ** -100, 2.0 ** -100), (2.0 ** 118, 2.0 ** 118),
         (0.0, 2.0 ** -64, 1.0), (0.0, 0.02), (2.0 ** -64, 0.02)]


def kind(j, values):
    """Which of the scales page j has: neighbours differ, and so do pages that are four apart."""
    return (j // 4 + j) % len(values)


def scales(c, values):
    for j in range(c.max_pages):
        c.vs[int(c.table[0, j])] = values[kind(j, values)]
    c.vc = c.vc.float().abs().clamp(min=2.0 ** -6).to(ao.E4M3)  # (so that what a page adds cannot cancel)
    return c


@pytest.mark.parametrize("values", MIXED)
@pytest.mark.parametrize("n,old", [(1, 300), (1, 6000), (50, 300), (300, 6000)])
def test_value_scales_far_apart(m, kernel, values, n, old):
    """Every scale that the call accepts, beside every other, in one part and in many."""
    c = scales(Case([n], [old], 2, 8, 128, 32, BF16, ao.E4M3), values)
    d = c.cuda()
    call(m, c, d)
    m.lsa_check_device()
    check(c, d, rows={(0, i) for i in {0, n // 2, n - 1}})


@pytest.mark.parametrize("loud", [8.0, 60.0])
@pytest.mark.parametrize("values", [(0.0, 0.02), (0.0, 2.0 ** -64), (0.0, 2.0 ** 60), (2.0 ** -64, 2.0 ** 40)])
@pytest.mark.parametrize("n,old", [(1, 300), (1, 6000), (3, 40), (50, 300), (300, 6000)])
def test_keys_of_zero_scale_with_the_largest_scores(m, kernel, loud, values, n, old):
    """The pages whose values are zero (or least) have the largest scores, by up to hundreds of binades: the others still
    carry the output."""
    c = scales(Case([n], [old], 2, 8, 128, 32, BF16, ao.E4M3), values)
    for j in range(c.max_pages):
        if kind(j, values) == 0:
            c.ks[int(c.table[0, j])] *= loud
    d = c.cuda()
    call(m, c, d)
    m.lsa_check_device()
    check(c, d, rows={(0, i) for i in {0, n // 2, n - 1}})


@pytest.mark.parametrize("value", [2.0 ** -100, 2.0 ** -64, 2.0 ** 120, 0.0])
def test_least_and_largest_scale_over_many_keys(m, kernel, value):
    """Tens of thousands of keys of nearly equal weight: the sum does not overflow."""
    c = scales(Case([2], [40000], 1, 4, 64, 64, BF16, ao.E4M3, spread=0.01), [value])
    d = c.cuda()
    call(m, c, d)
    m.lsa_check_device()
    check(c, d)


def test_unusual_scales_of_ragged_users(m, kernel):
    """Only the sequence that holds them is concerned; rows that see none of the pages are as ever."""
    c = Case([1, 4, 0, 30], [700, 90, 5, 129], 2, 16, 64, 16, BF16, ao.E4M3, window=200, sinks=3, spare_rows=2)
    c.vs[int(c.table[0, 40])] = 2.0 ** 90
    c.vs[int(c.table[1, 2])] = 0.0
    c.vs[int(c.table[3, 3])] = 2.0 ** -90
    d = c.cuda()
    call(m, c, d)
    m.lsa_check_device()
    check(c, d)


@pytest.mark.parametrize("n,old,window", [(1, 40, 0), (1, 5000, 0), (3, 40, 0), (1, 300, 20), (40, 30, 0)])
@pytest.mark.parametrize("listed", [0, 50])
def test_infinities_that_an_fp32_row_sees(m, n, old, window, listed):
    """A key of -inf weighs nothing, a value of infinity makes the output infinite, numbers next to the largest stay
    finite: as in the formula, for cached keys and listed ones."""
    c = Case([n], [old], 2, 8, 64, 16, F32, window=window)
    c.q = c.q.abs() + 0.1
    at = lambda p: (int(c.table[0, p // 16]), slice(None), p % 16)  # noqa: E731
    c.kc[at(old)][:, 5] = -math.inf      # (every row sees the first new token, and the one before it)
    c.vc[at(old - 1)][1, 7] = -3.4028e38
    if listed:
        c.add_topk(listed, [300], [100], 4)
        held, light = c.idx[:100].tolist(), c.topk[0, 3:6].tolist()
        row_of = lambda e: c.win[0, e - 300] if e >= 300 else c.hot[held.index(e)]  # noqa: E731
        for e in light:
            row_of(e)[0, :, 9] = -math.inf
        row_of(int(c.topk[0, 6]))[1, 0, 11] = 3.4028e38
    d = c.cuda()
    call(m, c, d)
    m.lsa_check_device()
    assert torch.isfinite(d["out"]).all() and torch.isfinite(d["lse_out"]).all()
    if listed:
        c.topk[torch.isin(c.topk, torch.tensor(light, dtype=torch.int32))] = -1
    check(c, d, rows={(0, i) for i in {0, n // 2, n - 1}}, hidden=lambda b, j: j == old)
    c.vc[at(old - 1)][1, 7] = math.inf
    e = c.cuda()
    call(m, c, e)
    m.lsa_check_device()
    assert (e["out"][:, 4:, 7] == math.inf).all()
    e["out"][:, 4:, 7] = d["out"][:, 4:, 7]
    assert torch.equal(e["out"], d["out"]) and torch.equal(e["lse_out"], d["lse_out"])


@pytest.mark.parametrize("cdt", [BF16, ao.E4M3])
def test_a_workspace_of_another_call_serves(m, kernel, cdt):
    """One made for a long prompt (or for one token) is enough for every call; nothing is written behind it."""
    H, Hq, D = 8, 64, 128
    small = m.lsa_window_attention_workspace_size(4096, 1, Hq, H, D)
    assert small < m.lsa_window_attention_workspace_size(64, 1, Hq, H, D)
    for n, old in ((1, 3000), (64, 3000), (40, 9000), (200, 3000)):  # (6, 2, 3 parts and one)
        c = Case([n], [old], H, Hq, D, 128, BF16, cdt)
        d = c.cuda()
        ws = torch.full((small + (8 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
        call(m, c, d, ws[:small])
        m.lsa_check_device()
        assert (ws[small:] == 0xA5).all()
        check(c, d, rows={(0, 0), (0, n - 1)})


def test_zero_scale_behind_a_half_that_is_not_there(m, kernel):
    """The window starts in the middle of a 32-key chunk, whose first 16 keys come in as zeros with their scales; the next
    page that the same warp reads (80 users: a CTA a tile, a chunk in four a warp) has a scale of zero itself, and the
    largest scores."""
    B, old = 80, 299 + 16 + 32 * 20  # the window's first key stands at 656 = 32 * 20 + 16
    c = Case([1] * B, [old] * B, 2, 8, 64, 16, BF16, ao.E4M3, window=300)
    c.vs[:] = 2.0 ** -30
    c.vc = c.vc.float().abs().clamp(min=2.0 ** -6).to(ao.E4M3)
    for b in range(B):
        pg = int(c.table[b, 48])  # chunk 24, the fifth of the window's
        c.vs[pg] = 0.0
        c.ks[pg] *= 20.0
    d = c.cuda()
    call(m, c, d)
    m.lsa_check_device()
    check(c, d, rows={(b, 0) for b in range(0, B, 7)})


@pytest.mark.parametrize("test", ["strided_queries_and_no_lse", "large_scores_and_scale", "rows_with_nothing_to_see",
                                  "bad_data_is_left_out_and_flagged", "zero_scales", "many_sequences", "negative_and_zero_scale",
                                  "replayed_graph_follows_the_lengths", "two_streams_with_their_own_workspaces",
                                  "the_same_bits_every_time", "pages_past_32_bits", "no_tokens_and_no_entries",
                                  "bad_length_with_nan_ends"])
def test_on_both_kernels(m, kernel, test):
    """Each by itself, so that one's failure does not hide the next."""
    getattr(test_gpu_attention, "test_" + test)(m)
