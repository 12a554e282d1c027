"""The attention side of a decode step allocates no device memory after its first call: neither from the driver nor from
torch's allocator.  Collected last (file name), beside the same test of the score entry points."""
import pytest
import torch

import attn_oracle as ao
import test_gpu_attention as ta
import test_gpu_window_cache as tw

pytestmark = pytest.mark.gpu


def test_append_and_attention_allocate_no_device_memory():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sparse_kv_cache_memoryindexer_b200 as m
    calls = []
    for dt, cdt in ((torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32), (torch.bfloat16, ao.E4M3)):
        d = tw.Case(new=[1, 40], old=[7, 100], H=2, Hq=4, D=128, page=64, dt=dt, cdt=cdt).cuda()
        calls.append(lambda d=d: m.lsa_kv_append(**d))
        for new, old in (([1, 1], [9000, 3]), ([300, 5], [2000, 100])):
            c = ta.Case(new, old, 2, 16, 128, 64, dt, cdt)
            d, ws = c.cuda(), c.workspace(m)
            calls.append(lambda c=c, d=d, ws=ws: ta.call(m, c, d, ws))
        if cdt == dt:
            c = ta.Case([1, 1], [50, 3], 2, 16, 128, 64, dt, window=40).add_topk(100, [500, 300], [200, 10], 4)
            d, ws = c.cuda(), c.workspace(m)
            calls.append(lambda c=c, d=d, ws=ws: ta.call(m, c, d, ws))
    for f in calls:
        f()
    torch.cuda.synchronize()
    free0, _ = torch.cuda.mem_get_info()
    alloc0, reserved0 = torch.cuda.memory_allocated(), torch.cuda.memory_reserved()
    for _ in range(3):
        for f in calls:
            f()
    torch.cuda.synchronize()
    m.lsa_check_device()
    free1, _ = torch.cuda.mem_get_info()
    assert free1 == free0, f"free device memory changed by {free0 - free1} bytes"
    assert torch.cuda.memory_allocated() == alloc0 and torch.cuda.memory_reserved() == reserved0
