"""What the window cache, the decode step and the binding refuse on the host, with CPU tensors; and that the binding
loads where torch lacks its private names."""
import os
import subprocess
import sys

import pytest
import torch

from sparse_kv_cache_memoryindexer_b200 import lsa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_binding_loads_without_torchs_private_names():
    code = """
import torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
from sparse_kv_cache_memoryindexer_b200 import lsa
assert lsa._current_device is torch.cuda.current_device
class S:
    cuda_stream = 1234
torch.cuda.current_stream = lambda dev: S if dev == 3 else None
assert lsa._raw_stream(3) == 1234
print("loaded")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "loaded" in r.stdout, r.stderr[-2000:]


def tensors():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    return dict(q=bf(4, 8, 64), q_offsets=torch.zeros(3, dtype=torch.int64), cache_len=i32(2), page_table=i32(2, 5),
                k_cache=bf(9, 2, 16, 64), v_cache=bf(9, 2, 16, 64), out=bf(4, 8, 64),
                workspace=torch.zeros(256, dtype=torch.uint8))


@pytest.mark.parametrize("over", [dict(window=1 << 31), dict(n_sink=1 << 31), dict(window=(1 << 32) + 5), dict(n_sink=-(1 << 32))])
def test_windows_that_do_not_fit_a_c_int(over):
    """They would be cut: a window of 2^32 + 5 to 5."""
    with pytest.raises(ValueError, match="below 2\\^31"):
        lsa.lsa_window_attention(**tensors(), **over)
    sel = dict(topk_idx=torch.zeros((4, 7), dtype=torch.int32), idx=torch.zeros(30, dtype=torch.int32),
               count=torch.zeros(2, dtype=torch.int32), seq_offsets=torch.zeros(3, dtype=torch.int64), total_S=30,
               hot_kv=torch.zeros((30, 512), dtype=torch.uint8))
    with pytest.raises(ValueError, match="below 2\\^31"):
        lsa.lsa_core_attention(**tensors(), **sel, **over)


def on_device(number):
    """Stands in for a WindowCache on a CUDA device."""
    class Cache:
        class k:
            get_device = staticmethod(lambda: number)
    return Cache


def test_decode_step_makes_the_caches_device_current(monkeypatch):
    """All three calls run there, whichever device is current; the one that was is so again."""
    from contextlib import contextmanager

    from sparse_kv_cache_memoryindexer_b200 import pipeline
    path = object.__new__(pipeline.IndexerPath)
    path.cache, now, seen = on_device(1), [0], []

    @contextmanager
    def device(d):
        before, now[0] = now[0], d
        yield
        now[0] = before

    class Reached(Exception):
        pass

    @contextmanager
    def stage(name):
        seen.append((name, now[0]))
        raise Reached
        yield

    monkeypatch.setattr(lsa, "_current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(pipeline, "_stage", stage)
    with pytest.raises(Reached):
        path.decode_step(*[None] * 6)
    assert seen == [("lsa.lightning_topk_step", 1)]


def test_decode_step_wants_the_rows_of_the_windows_entries(monkeypatch):
    """Keys of entries compressed in the window without their rows would be picked, and then left out of the softmax."""
    from sparse_kv_cache_memoryindexer_b200 import pipeline
    path = object.__new__(pipeline.IndexerPath)
    path.cache, path.W = on_device(0), 5
    monkeypatch.setattr(lsa, "_current_device", lambda: 0)
    K, n = torch.zeros((2, 5, 32)), torch.zeros(2, dtype=torch.int32)
    rows = lambda w: torch.zeros((2, w, 1024), dtype=torch.uint8)  # noqa: E731
    step = lambda **kw: path.decode_step(None, None, None, None, None, None, **kw)  # noqa: E731
    for kw in (dict(win_K=K, win_count=n), dict(win_K=K, win_count=n, win_kv=rows(4)), dict(win_K=K, win_kv=rows(5)),
               dict(win_K=K, win_count=n, win_kv=rows(0))):
        with pytest.raises(ValueError, match="go with it"):
            step(**kw)
    with pytest.raises(ValueError, match="was told of 5"):
        step(win_K=torch.zeros((2, 6, 32)), win_count=n, win_kv=rows(6))
    # what fits goes on to the calls (here: stopped at the first)
    class Reached(Exception):
        pass

    def reached(name):
        raise Reached
    monkeypatch.setattr(pipeline, "_stage", reached)
    for kw in (dict(), dict(win_K=K, win_count=n, win_kv=rows(5)), dict(win_K=K[:, :3], win_count=n, win_kv=rows(5)),
               dict(win_K=K[:, :0], win_count=n), dict(win_kv=rows(5))):
        with pytest.raises(Reached):
            step(**kw)


def test_window_cache_refuses_what_its_calls_would():
    from sparse_kv_cache_memoryindexer_b200 import WindowCache
    bf, f32, e4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
    make = lambda D=64, page=16, dt=bf, cdt=None: WindowCache(2, 2, D, page, 4, 4, dt, cdt, device="cpu")  # noqa: E731
    for kw in (dict(D=256), dict(D=96), dict(D=16), dict(page=8), dict(page=48), dict(page=256)):
        with pytest.raises(ValueError, match="D must be"):
            make(**kw)
    for kw in (dict(dt=torch.float16), dict(dt=f32, cdt=bf), dict(dt=f32, cdt=e4), dict(dt=bf, cdt=f32), dict(dt=e4)):
        with pytest.raises(TypeError, match="dtype and cdtype"):
            make(**kw)
    for kw in (dict(), dict(D=32), dict(D=128, page=128), dict(dt=f32), dict(cdt=e4)):
        make(**kw)


def test_open_decode_refuses_heads_and_lists_that_the_step_would():
    from sparse_kv_cache_memoryindexer_b200 import WindowCache, pipeline
    path = object.__new__(pipeline.IndexerPath)
    path.B, path.row_bytes, path.k, path.idx = 2, 2 * 2 * 64 * 2, 16, torch.zeros(4, dtype=torch.int32)
    cache = WindowCache(2, 2, 64, 16, 4, 4, torch.bfloat16, device="cpu")
    for H_q in (0, 3, -2):
        with pytest.raises(ValueError, match="multiple of H_kv"):
            path.open_decode(cache, H_q)
    path.k = 5000
    with pytest.raises(ValueError, match="k in"):
        path.open_decode(cache, 4)
