"""What lsa_kv_append, lsa_window_attention and lsa_core_attention refuse on the host, before any device
work: the C ABI with pointers that are never dereferenced, and the binding with CPU tensors."""
import ctypes as C
import math

import pytest
import torch

from sparse_kv_cache_memoryindexer_b200 import lsa

P = C.c_void_p(1 << 20)
F32, BF16, FP8 = lsa.LSA_F32, lsa.LSA_BF16, lsa.LSA_FP8_E4M3


def append(**kw):
    a = dict(q=P, qs=1024, k=C.c_void_p(1 << 21), ks=256, v=C.c_void_p(1 << 22), vs=256, dt=BF16, offs=P, N=4, B=2, len=P, table=P,
             mp=8, inv=P, rot=128, il=0, Hq=8, H=2, D=128, page=64, np=16, kc=P, vc=P, cdt=BF16, ksc=None, vsc=None,
             qo=C.c_void_p(1 << 30), st=None)
    a.update(kw)
    return lsa.library().lsa_kv_append(*a.values()), lsa.library().lsa_last_error().decode()


def window(**kw):
    a = dict(q=P, qs=1024, dt=BF16, offs=P, N=4, B=2, len=P, table=P, mp=8, Hq=8, H=2, D=128, page=64, np=16, kc=P, vc=P,
             cdt=BF16, ksc=None, vsc=None, window=0, sink=0, scale=0.1, out=C.c_void_p(1 << 30), lse=None, ws=P, wsb=1 << 40, st=None)
    a.update(kw)
    return lsa.library().lsa_window_attention(*a.values()), lsa.library().lsa_last_error().decode()


def core(**kw):
    a = dict(q=P, qs=1024, dt=BF16, offs=P, N=4, B=2, len=P, table=P, mp=8, Hq=8, H=2, D=128, page=64, np=16, kc=P, vc=P,
             window=0, sink=0, scale=0.1, topk=P, k=16, idx=P, cnt=P, so=P, T=100, hot=P, rb=1024, win=None, W=0, out=C.c_void_p(1 << 30),
             lse=None, ws=P, wsb=1 << 40, st=None)
    a.update(kw)
    return lsa.library().lsa_core_attention(*a.values()), lsa.library().lsa_last_error().decode()


@pytest.mark.parametrize("call", [append, window, core])
def test_shared_checks(call):
    INVALID, UNSUPPORTED = 1, 2
    odd = C.c_void_p((1 << 20) + 8)
    for kw, st, msg in ((dict(offs=None), INVALID, "null pointer"), (dict(len=None), INVALID, "null pointer"),
                        (dict(kc=None), INVALID, "null pointer"), (dict(B=0), INVALID, "positive"),
                        (dict(N=-1), INVALID, "positive"), (dict(mp=0), INVALID, "positive"), (dict(np=0), INVALID, "positive"),
                        (dict(H=0), INVALID, ""), (dict(Hq=0), INVALID, "positive"), (dict(D=96), None, ""),
                        (dict(page=48), UNSUPPORTED, "page_size"), (dict(page=8), UNSUPPORTED, "page_size"),
                        (dict(Hq=7), INVALID, "multiple of H_kv"), (dict(N=1 << 24), INVALID, "too large"),
                        (dict(mp=1 << 25), INVALID, "2^31"), (dict(np=1 << 31), INVALID, "too many pages"),
                        (dict(kc=odd), INVALID, "16-byte aligned"), (dict(dt=FP8), None, ""), (dict(dt=7), None, "")):
        got, text = call(**kw)
        assert (got == st if st is not None else got in (1, 2)), (kw, got, text)
        assert msg in text, (kw, text)


@pytest.mark.parametrize("call", [append, window])
def test_types_of_cache_and_scales(call):
    assert call(dt=F32, cdt=BF16)[0] == 2
    assert call(dt=F32, cdt=FP8, ksc=P, vsc=P)[0] == 2
    assert call(dt=BF16, cdt=F32)[0] == 2
    for kw in (dict(cdt=FP8), dict(cdt=FP8, ksc=P), dict(ksc=P, vsc=P), dict(vsc=P)):
        st, msg = call(**kw)
        assert st == 1 and "scale" in msg


def test_append_refuses():
    odd = C.c_void_p((1 << 21) + 2)
    for kw, st, msg in ((dict(q=None), 1, "together"), (dict(qo=None), 1, "together"), (dict(rot=160), 1, "rot_dim"),
                        (dict(rot=24), 2, "multiple of 16"), (dict(rot=0), 1, "inv_freq"), (dict(inv=None), 1, "inv_freq"),
                        (dict(ks=255), 1, "k_stride"), (dict(vs=260), 1, "16-byte"), (dict(k=odd), 1, "16-byte"),
                        (dict(qs=1023), 1, "q_stride"), (dict(qo=C.c_void_p((1 << 20) + 256)), 1, "overlap"),
                        (dict(qs=2048, qo=P), 1, "overlap")):
        got, text = append(**kw)
        assert got == st and msg in text, (kw, got, text)


@pytest.mark.parametrize("call", [window, core])
def test_attention_refuses(call):
    for kw, st, msg in ((dict(out=None), 1, "null pointer"), (dict(q=None), 1, "null pointer"), (dict(qs=1000), 1, "q_stride"),
                        (dict(window=-1), 1, "negative"), (dict(sink=-1), 1, "negative"), (dict(scale=math.nan), 1, "finite"),
                        (dict(scale=math.inf), 1, "finite"), (dict(ws=None), 5, "workspace needs"), (dict(wsb=16), 5, "workspace needs"),
                        (dict(ws=C.c_void_p((1 << 20) + 16)), 1, "256-byte"), (dict(out=C.c_void_p((1 << 20) + 4)), 1, "16-byte"),
                        (dict(out=P), 1, "overlap"), (dict(out=C.c_void_p((1 << 20) + 2048)), 1, "overlap")):
        got, text = call(**kw)
        assert got == st and msg in text, (kw, got, text)


def test_core_attention_refuses():
    for kw, st, msg in ((dict(topk=None), 1, "null pointer"), (dict(hot=None), 1, "null pointer"), (dict(k=0), 1, "k must be"),
                        (dict(k=5000), 1, "k must be"), (dict(T=1 << 31), 1, "total_S"), (dict(rb=512), 1, "row_bytes"),
                        (dict(W=3), 1, "win_kv"), (dict(win=P), 1, "win_kv"), (dict(win=P, W=1 << 30), 1, "B * W"),
                        (dict(hot=C.c_void_p((1 << 20) + 8)), 1, "16-byte"), (dict(dt=FP8), 1, "dt must be")):
        got, text = core(**kw)
        assert got == st and msg in text, (kw, got, text)


def test_no_tokens_is_no_work():
    assert append(N=0)[0] == 0 and window(N=0)[0] == 0 and core(N=0)[0] == 0


def test_workspace_sizes():
    w, c = lsa.lsa_window_attention_workspace_size, lsa.lsa_core_attention_workspace_size
    assert w(32, 32, 64, 8, 128) > 0 and c(32, 32, 64, 8, 128, 512) > 0
    # parts of a call whose few tiles are split: 256 rows of D + 2 floats each
    assert w(64, 1, 8, 1, 128) >= 2 * 256 * 130 * 4
    assert w(-1, 1, 8, 1, 128) == 0 and w(1, 0, 8, 1, 128) == 0 and c(1, 1, 0, 1, 128, 4) == 0
    # the size never depends on what the keys are, and stays bounded for long calls
    assert w(1 << 20, 16, 64, 8, 128) < 64 << 20 and w(64, 1, 64, 1, 128) < 64 << 20


def tensors(**over):
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    d = dict(q=bf(4, 8, 64), k=bf(4, 2, 64), v=bf(4, 2, 64), q_offsets=torch.zeros(3, dtype=torch.int64), cache_len=i32(2),
             page_table=i32(2, 5), k_cache=bf(9, 2, 16, 64), v_cache=bf(9, 2, 16, 64))
    d.update(over)
    return d


@pytest.mark.parametrize("over,error,match", [
    (dict(q_offsets=torch.zeros(3, dtype=torch.int32)), TypeError, "q_offsets must be torch.int64"),
    (dict(cache_len=torch.zeros(2, dtype=torch.int64)), TypeError, "cache_len must be torch.int32"),
    (dict(page_table=torch.zeros((2, 5))), TypeError, "page_table must be torch.int32"),
    (dict(page_table=torch.zeros((3, 5), dtype=torch.int32)), ValueError, "page_table"),
    (dict(q_offsets=torch.zeros(4, dtype=torch.int64)), ValueError, "B \\+ 1"),
    (dict(v_cache=torch.zeros((9, 2, 16, 64))), TypeError, "v_cache must be"),
    (dict(v_cache=torch.zeros((9, 2, 8, 64), dtype=torch.bfloat16)), ValueError, "k_cache and v_cache"),
    (dict(k_cache=torch.zeros((9, 2, 16, 64), dtype=torch.float16)), TypeError, "k_cache"),
    (dict(k_scale=torch.zeros(18), v_scale=torch.zeros(18)), ValueError, "E4M3"),
    (dict(q=torch.zeros((4, 8, 32), dtype=torch.bfloat16)), ValueError, "q must be"),
    (dict(q=torch.zeros((4, 8, 128), dtype=torch.bfloat16)[:, :, ::2]), ValueError, "contiguous in q"),
    (dict(q=torch.zeros((1, 8, 64), dtype=torch.bfloat16).expand(4, 8, 64)), ValueError, "overlap"),
    (dict(), ValueError, "device tensor expected"),
])
def test_binding_rejects(over, error, match):
    d = tensors(**over)
    out = torch.zeros((4, 8, 64), dtype=torch.bfloat16)
    ws = torch.zeros(256, dtype=torch.uint8)
    q = d.pop("q")
    k, v = d.pop("k"), d.pop("v")
    with pytest.raises(error, match=match):
        lsa.lsa_window_attention(q, out=out, workspace=ws, **d)
    with pytest.raises(error, match=match):
        lsa.lsa_kv_append(k, v, q=q, q_out=out, **d)


def test_binding_rejects_small_buffers_and_types():
    d = tensors()
    q, k, v = d.pop("q"), d.pop("k"), d.pop("v")
    out, ws = torch.zeros((4, 8, 64), dtype=torch.bfloat16), torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError, match="out holds"):
        lsa.lsa_window_attention(q, out=out[:3], workspace=ws, **d)
    with pytest.raises(TypeError, match="out must be"):
        lsa.lsa_window_attention(q, out=out.float(), workspace=ws, **d)
    with pytest.raises(TypeError, match="lse_out must be"):
        lsa.lsa_window_attention(q, out=out, workspace=ws, lse_out=out, **d)
    with pytest.raises(ValueError, match="lse_out holds"):
        lsa.lsa_window_attention(q, out=out, workspace=ws, lse_out=torch.zeros(31), **d)
    with pytest.raises(ValueError, match="k and v must be"):
        lsa.lsa_kv_append(k[:3], v, **d)
    with pytest.raises(ValueError, match="q_out"):
        lsa.lsa_kv_append(k, v, q=q, **d)
    with pytest.raises(TypeError, match="inv_freq must be"):
        lsa.lsa_kv_append(k, v, inv_freq=torch.zeros(8, dtype=torch.float64), **d)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    sel = dict(topk_idx=i32(4, 7), idx=i32(30), count=i32(2), seq_offsets=torch.zeros(3, dtype=torch.int64), total_S=30,
               hot_kv=torch.zeros((30, 512), dtype=torch.uint8))
    call = lambda **o: lsa.lsa_core_attention(q, out=out, workspace=ws, **d, **{**sel, **o})  # noqa: E731
    with pytest.raises(TypeError, match="topk_idx must be"):
        call(topk_idx=torch.zeros((4, 7), dtype=torch.int64))
    with pytest.raises(ValueError, match="topk_idx holds"):
        call(topk_idx=i32(3, 7))
    with pytest.raises(ValueError, match="idx holds"):
        call(idx=i32(29))
    with pytest.raises(ValueError, match="hot_kv holds"):
        call(hot_kv=torch.zeros((30, 511), dtype=torch.uint8))
    with pytest.raises(ValueError, match="win_kv"):
        call(win_kv=torch.zeros((3, 1, 512), dtype=torch.uint8))
    with pytest.raises(ValueError, match="win_kv holds"):
        call(win_kv=torch.zeros((2, 4, 500), dtype=torch.uint8))
    with pytest.raises(ValueError, match="seq_offsets"):
        call(seq_offsets=torch.zeros(2, dtype=torch.int64))


def test_empty_tensors_are_no_work():
    """An empty tensor has no pointer: with N = 0 none is asked for, and without entries no list or rows are."""
    assert append(N=0, q=None, k=None, v=None, qo=None)[0] == 0
    assert window(N=0, q=None, out=None)[0] == 0
    assert core(N=0, q=None, out=None, topk=None)[0] == 0
    assert core(N=0, T=0, idx=None, hot=None)[0] == 0
    assert core(T=5, idx=None)[0] == 1 and core(T=5, hot=None)[0] == 1
