"""A window and its decode steps as a user runs them: IndexerPath.run, then per step the Top-k, the append to
the window cache and core attention, eagerly and from a CUDA graph, against the definition in 64 bits; and
the window cache by itself in 8 bits, prompt and steps."""
import pytest
import torch

import attn_oracle as ao
import synth

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
H_KV, D, H_Q, PAGE, WINDOW, SINKS = 2, 128, 32, 16, 40, 3


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sparse_kv_cache_memoryindexer_b200 as mod
    mod.lsa_check_device()
    return mod


def check_row(out, lse, q, K, V, p_dtype):
    for h in range(q.shape[0]):
        g = h // (q.shape[0] // K.shape[1])
        o, l_, A, mag = ao.attend(q[h].double(), K[:, g].double(), V[:, g].double(), D ** -0.5)
        bo, bl = ao.attend_bounds(o, A, mag, K.shape[0], D, BF16, p_dtype)
        assert ((out[h].double() - o).abs() <= bo).all(), h
        assert abs(float(lse[h]) - l_) <= bl, h


def test_window_and_its_decode_steps(m):
    wl = synth.workload("ctx128k_bf16", B=2, S=(1500, 700), fetch=(0.135, 0.3), name="decode_path")
    inp = synth.make_inputs(wl)
    T, B = wl.total_S, wl.B
    k = 96
    path = m.IndexerPath(wl.L, B, wl.d, wl.r, wl.n_h, wl.d_I, wl.tau, k, T, wl.row_bytes, BF16, BF16)
    assert wl.row_bytes == 2 * H_KV * D * 2
    pool = m.MappedPool(T, wl.row_bytes)
    g = torch.Generator().manual_seed(5)
    try:
        rows = torch.randn((T, 2, H_KV, D), generator=g).to(BF16)
        pool.tensor.copy_(rows.view(torch.uint8).view(T, wl.row_bytes))
        up = lambda t: None if t is None else t.cuda()  # noqa: E731
        path.run(up(inp.h), up(inp.W_dq), up(inp.W_iuq), up(inp.W_w), up(inp.K), None, up(inp.seq_offsets), pool.tensor,
                 up(inp.q_dec), up(inp.w_dec))
        # the contexts behind the entries: 4 tokens an entry; the cache holds the last of them, and the first
        old = [4 * 1500, 4 * 700]
        steps, W = 20, 5
        n_pages = 40
        cache = m.WindowCache(B, H_KV, D, PAGE, n_pages, (max(old) + steps) // PAGE + 1, BF16, window=WINDOW, n_sink=SINKS)
        cache.k.copy_(torch.randn(cache.k.shape, generator=g))
        cache.v.copy_(torch.randn(cache.v.shape, generator=g))
        free = torch.randperm(n_pages, generator=g).tolist()
        table = torch.full(cache.page_table.shape, -1, dtype=torch.int32)
        for b in range(B):
            need = {0} | set(range((old[b] - WINDOW) // PAGE, (old[b] + steps) // PAGE + 1))
            for p in need:
                table[b, p] = free.pop()
        cache.page_table.copy_(table)
        cache.len.copy_(torch.tensor(old))
        path.open_decode(cache, H_Q, W)
        win_kv = torch.randn((B, W, 2, H_KV, D), generator=g).to(BF16)
        win_K = torch.randn((B, W, wl.d_I), generator=g).to(BF16)
        win_count = torch.zeros(B, dtype=torch.int32, device="cuda")
        inv_freq = (1e6 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float()
        q = torch.empty((B, H_Q + 2 * H_KV, D), dtype=BF16, device="cuda")
        qi, wi = torch.empty((B, wl.n_h, wl.d_I), dtype=BF16, device="cuda"), torch.empty((B, wl.n_h), device="cuda")
        args = dict(win_K=win_K.cuda(), win_count=win_count, win_kv=win_kv.cuda().view(torch.uint8).view(B, W, -1),
                    inv_freq=inv_freq.cuda())
        offs = up(inp.seq_offsets)

        def step():
            path.decode_step(qi, wi, q[:, :H_Q], q[:, H_Q:H_Q + H_KV], q[:, H_Q + H_KV:], offs, **args)
            cache.advance(path.one_each)

        graph = None
        pos0 = list(old)
        kc, vc = cache.k.cpu(), cache.v.cpu()
        for i in range(steps):
            qkv = torch.randn(q.shape, generator=g).to(BF16)
            q.copy_(qkv)
            qi.copy_(inp.q_dec[:, i])
            wi.copy_(inp.w_dec[:, i])
            win_count.fill_(min(i // 4, W))
            if i < 3:
                step()
            else:
                if graph is None:  # (the capture runs nothing)
                    torch.cuda.synchronize()
                    graph = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(graph):
                        step()
                graph.replay()
            m.lsa_check_device()
            # the append: the new token's key, rotated; its value as it is; nothing else changed
            k2, v2 = cache.k.cpu(), cache.v.cpu()
            for b in range(B):
                pos = pos0[b]
                pg, sl = int(table[b, pos // PAGE]), pos % PAGE
                for part, got, heads in (("q", path.q_rot[b].cpu(), slice(0, H_Q)), ("k", k2[pg, :, sl], slice(H_Q, H_Q + H_KV))):
                    y, mag = ao.rotate(qkv[b, heads].double(), pos, inv_freq, False)
                    err = mag * ao.ROTATION
                    assert ((got.double() - y).abs() <= err + ao.half_step(BF16) * (y.abs() + err)).all(), (i, part)
                assert torch.equal(v2[pg, :, sl], qkv[b, H_Q + H_KV:])
                kc[pg, :, sl], vc[pg, :, sl] = k2[pg, :, sl], v2[pg, :, sl]
            assert torch.equal(kc, k2) and torch.equal(vc, v2)
            # the attention: the step's own Top-k rows, taken from the pool itself, and the window
            sel = path.step_idx.cpu()
            for b in range(B):
                S, o = int(inp.seq_offsets[b + 1] - inp.seq_offsets[b]), int(inp.seq_offsets[b])
                mine = [e for e in sel[b].tolist() if e >= 0]
                assert len(mine) == min(k, int(path.count[b]) + int(win_count[b]))
                picked = torch.stack([rows[o + e] if e < S else win_kv[b, e - S] for e in mine])
                j = torch.tensor(ao.visible(pos0[b], pos0[b] + 1, WINDOW, SINKS))
                pg, sl = table[b].long()[j // PAGE], j % PAGE
                K = torch.cat([k2[pg, :, sl], picked[:, 0]])
                V = torch.cat([v2[pg, :, sl], picked[:, 1]])
                check_row(path.attn_out[b].cpu(), path.attn_lse[b].cpu(), path.q_rot[b].cpu(), K, V, BF16)
            pos0 = [p + 1 for p in pos0]
            assert cache.len.tolist() == pos0
    finally:
        torch.cuda.synchronize()
        pool.free()


def test_open_decode_refuses_rows_of_another_shape(m):
    path = m.IndexerPath(1, 2, 64, 64, 4, 32, 4, 16, 100, 1024, BF16, BF16)
    with pytest.raises(ValueError, match="fetched rows"):
        path.open_decode(m.WindowCache(2, 4, 128, 16, 8, 8, BF16), 8)
    with pytest.raises(ValueError, match="fetched rows"):
        path.open_decode(m.WindowCache(2, 2, 128, 16, 8, 8, BF16, torch.float8_e4m3fn), 8)
    with pytest.raises(ValueError, match="sequences"):
        path.open_decode(m.WindowCache(3, 2, 128, 16, 8, 8, BF16), 8)


@pytest.mark.parametrize("cdtype", [BF16, torch.float8_e4m3fn])
def test_prompt_then_steps_over_the_window_cache(m, cdtype):
    """A ragged prompt in two chunks, then single tokens; each call's rows against the cache as it then is, and
    the cache against the tokens that went into it."""
    g = torch.Generator().manual_seed(9)
    B, page, window, sinks = 3, 32, 150, 4
    chunks = [[200, 0, 37], [90, 300, 1], [1, 1, 1], [1, 1, 1]]
    total = [sum(c[b] for c in chunks) for b in range(B)]
    max_pages = max(total) // page + 1
    cache = m.WindowCache(B, H_KV, D, page, B * max_pages, max_pages, BF16, cdtype, window=window, n_sink=sinks)
    cache.k.view(torch.uint8).fill_(0x7F)  # NaN wherever nothing was written
    cache.v.view(torch.uint8).fill_(0x7F)
    table = torch.randperm(B * max_pages, generator=g).view(B, max_pages).to(torch.int32)
    cache.page_table.copy_(table)
    inv = (1e4 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)).float().cuda()
    given = [([], []) for _ in range(B)]
    fp8 = cdtype == torch.float8_e4m3fn
    for new in chunks:
        N = sum(new)
        offs = torch.tensor([0] + list(torch.tensor(new).cumsum(0)), dtype=torch.int64)
        old = cache.len.tolist()
        qkv = torch.randn((N, H_Q + 2 * H_KV, D), generator=g).to(BF16)
        x = qkv.cuda()
        q_rot, out = torch.empty((N, H_Q, D), dtype=BF16, device="cuda"), torch.empty((N, H_Q, D), dtype=BF16, device="cuda")
        lse = torch.empty((N, H_Q), device="cuda")
        ws = torch.empty(m.lsa_window_attention_workspace_size(N, B, H_Q, H_KV, D), dtype=torch.uint8, device="cuda")
        cache.append(x[:, H_Q:H_Q + H_KV], x[:, H_Q + H_KV:], offs.cuda(), inv_freq=inv, interleaved=True, q=x[:, :H_Q], q_out=q_rot)
        cache.attend(q_rot, offs.cuda(), out, ws, lse_out=lse)
        cache.advance(offs.cuda())
        m.lsa_check_device()
        kc, vc = cache.k.cpu(), cache.v.cpu()
        ks, vs = (cache.k_scale.cpu(), cache.v_scale.cpu()) if fp8 else (None, None)
        for b in range(B):
            assert int(cache.len[b]) == old[b] + new[b]
            for i in range(new[b]):
                y, _ = ao.rotate(qkv[int(offs[b]) + i, H_Q:H_Q + H_KV].double(), old[b] + i, inv.cpu(), True)
                given[b][0].append(y)
                given[b][1].append(qkv[int(offs[b]) + i, H_Q + H_KV:].double())
            if not given[b][0]:
                continue
            j = torch.arange(len(given[b][0]))
            pg, sl = table[b].long()[j // page], j % page
            K, V = kc[pg, :, sl].double(), vc[pg, :, sl].double()
            if fp8:
                K, V = K * ks[pg].double()[:, :, None], V * vs[pg].double()[:, :, None]
                # a code may have been rounded to a page's scale twice (it grew once or twice): a step each time
                for got, want, sc in ((K, torch.stack(given[b][0]), ks[pg]), (V, torch.stack(given[b][1]), vs[pg])):
                    step = torch.maximum(want.abs() * 2.0 ** -4, sc.double()[:, :, None] * 2.0 ** -10)
                    assert ((got - want).abs() <= 2 * step + 1e-5).all()
            else:
                assert torch.equal(V, torch.stack(given[b][1]))
            for i in sorted({0, 1, new[b] // 2, new[b] - 1} & set(range(new[b]))):
                vis = ao.visible(old[b] + i, old[b] + new[b], window, sinks)
                n = int(offs[b]) + i
                check_row(out[n].cpu(), lse[n].cpu(), q_rot[n].cpu(), K[vis], V[vis], torch.float16 if fp8 else BF16)
