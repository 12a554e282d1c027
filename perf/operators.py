"""What the attention side of a decode step costs: appending rotated keys and values to a paged cache
(bf16, or E4M3 with a scale per page and head), attention over that cache with a sliding window and
first tokens that stay visible, and attention over a query's Top-k entries together with the window.

run() computes a case in plain torch operations (fp32), or, where `own` is set, calls the
library's entry points; exact() computes the same outputs from the definition in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


# ------------------------------------------------------------------------------------- the cases
# Keys of a case.  op: append | attend | core.  B sequences; every sequence brings between n_lo and
# n_hi new tokens to a cache that holds between len_lo and len_hi tokens (spread evenly in the
# logarithm, the same for every seed).  Hq query heads share H key/value heads of D elements; pages
# of `page` tokens; `cache` is the type of the cached keys and values.

def listed():
    return [
        # one decode step of 32 users: the new token's q, k, v from one fused projection
        dict(name="append_step_bf16", op="append", cache="bf16", B=32, n_lo=1, n_hi=1, len_lo=900, len_hi=262143,
             Hq=64, H=8, D=128, page=64, rot=128, pairs="halves"),
        # four prompts' chunks at once, partial rotation of neighbouring pairs
        dict(name="append_chunk_bf16", op="append", cache="bf16", B=4, n_lo=2500, n_hi=6000, len_lo=1, len_hi=100001,
             Hq=64, H=8, D=128, page=64, rot=64, pairs="neighbours"),
        # chunks into an 8-bit cache, starting in the middle of pages whose scales may have to grow
        dict(name="append_chunk_e4m3", op="append", cache="e4m3", B=8, n_lo=300, n_hi=2047, len_lo=37, len_hi=70001,
             Hq=32, H=8, D=128, page=64, rot=128, pairs="halves"),
        # one user, one token, a short window: latency
        dict(name="step_one_user", op="attend", cache="bf16", B=1, n_lo=1, n_hi=1, len_lo=20011, len_hi=20011,
             Hq=64, H=8, D=128, page=64, window=512, sinks=4),
        # one decode step of 32 users with a window of 4096
        dict(name="step_bf16", op="attend", cache="bf16", B=32, n_lo=1, n_hi=1, len_lo=2000, len_hi=200000,
             Hq=64, H=8, D=128, page=64, window=4096, sinks=4),
        # fp32, small heads, odd sizes
        dict(name="step_f32", op="attend", cache="f32", B=5, n_lo=1, n_hi=3, len_lo=333, len_hi=9001,
             Hq=12, H=4, D=64, page=16, window=1000, sinks=1),
        # the 64 tokens of a decode window again in one call (a draft checked, a window recomputed)
        dict(name="window_of_64", op="attend", cache="bf16", B=8, n_lo=64, n_hi=64, len_lo=3000, len_hi=60000,
             Hq=64, H=8, D=128, page=64, window=4096, sinks=4),
        # two prompts' chunks, one of them odd
        dict(name="chunk_bf16", op="attend", cache="bf16", B=2, n_lo=1777, n_hi=4096, len_lo=5000, len_hi=30000,
             Hq=32, H=8, D=128, page=64, window=4096, sinks=4),
        # one decode step over whole histories in 8 bits, lengths 16 times apart in one batch
        dict(name="step_e4m3_history", op="attend", cache="e4m3", B=8, n_lo=1, n_hi=1, len_lo=8191, len_hi=131071,
             Hq=64, H=8, D=128, page=64, window=0, sinks=0),
        # a prompt's chunk over its whole history in 8 bits
        dict(name="chunk_e4m3_history", op="attend", cache="e4m3", B=1, n_lo=2048, n_hi=2048, len_lo=14001, len_hi=14001,
             Hq=32, H=8, D=128, page=64, window=0, sinks=0),
        # the decode step of sparse attention: Top-512 of the fetched entries, a window of 128, rows of 1 KB
        dict(name="core_step", op="core", cache="bf16", B=1, n_lo=1, n_hi=1, len_lo=131072, len_hi=131072,
             Hq=32, H=2, D=128, page=64, window=128, sinks=4, k=512, entries=32768, fetched=0.135, fresh=16),
        # the same for 32 users at 1M tokens of context: Top-2048, rows of 1 KB
        dict(name="core_step_32", op="core", cache="bf16", B=32, n_lo=1, n_hi=1, len_lo=260000, len_hi=1048575,
             Hq=64, H=2, D=128, page=64, window=512, sinks=4, k=2048, entries=65536, fetched=0.135, fresh=16),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append", "attend", "attend", "attend", "core"])
    H = rng.choice([1, 2, 4, 8])
    Hq = H * rng.choice([1, 2, 3, 4, 7, 8] if H > 2 else [4, 8, 16, 32])
    D = rng.choice([64, 128, 128])
    c = dict(op=op, Hq=Hq, H=H, D=D, page=rng.choice([16, 32, 64, 128]))
    step = rng.random() < 0.5  # single tokens, or chunks
    if op == "append":
        c["cache"] = rng.choice(["bf16", "bf16", "e4m3", "e4m3", "f32"])
        total = _log_int(rng, 1, 64) if step else _log_int(rng, 200, 8000)
        c["B"] = total if step else rng.randint(1, 9)
        c["n_hi"] = 1 if step else max(1, total // c["B"])
        c["n_lo"] = 1 if step else max(1, c["n_hi"] // rng.randint(1, 6))
        c["len_lo"] = _log_int(rng, 1, 3000)
        c["len_hi"] = c["len_lo"] + _log_int(rng, 1, 200000)
        c["rot"] = rng.choice([D, D, D // 2, 0])
        c["pairs"] = rng.choice(["halves", "neighbours"])
    elif op == "attend":
        c["cache"] = rng.choice(["bf16", "bf16", "e4m3", "e4m3", "f32"])
        few = step or c["cache"] == "f32"
        c["B"] = _log_int(rng, 1, 40) if few else rng.randint(1, 4)
        c["n_hi"] = rng.randint(1, 3) if few else _log_int(rng, 16, 2000)
        c["n_lo"] = max(1, c["n_hi"] // rng.randint(1, 4))
        c["len_lo"] = _log_int(rng, 1, 4000)
        c["len_hi"] = c["len_lo"] + _log_int(rng, 1, 20000 if few else 6000)
        c["window"] = rng.choice([0, _log_int(rng, 1, 5000), _log_int(rng, 64, 5000)])
        c["sinks"] = rng.choice([0, 1, 4, 20]) if c["window"] else 0
        seen = c["len_hi"] + c["n_hi"] if not c["window"] else min(c["len_hi"], c["window"]) + c["n_hi"]
        c["B"] = max(1, min(c["B"], int(1.5e9 / (Hq * c["n_hi"] * seen))))  # the plain form holds every score
    else:
        c["cache"] = "bf16"
        c["B"] = _log_int(rng, 1, 40)
        c["n_lo"] = c["n_hi"] = 1
        c["len_lo"] = _log_int(rng, 600, 100000)
        c["len_hi"] = c["len_lo"] + _log_int(rng, 1, 100000)
        c["window"] = _log_int(rng, 16, 1000)
        c["sinks"] = rng.choice([0, 1, 4])
        c["k"] = _log_int(rng, 16, 2048)
        c["entries"] = _log_int(rng, 1000, 40000)
        c["fetched"] = rng.choice([0.02, 0.135, 0.4])
        c["fresh"] = rng.choice([0, 7, 16])
    return c


def _sizes(case):
    """New tokens and cached tokens of each sequence, as the case alone says."""
    B = case["B"]
    r = random.Random(1000 * B + case["len_hi"] + case["n_hi"])
    new = [case["n_hi"]] + [r.randint(case["n_lo"], case["n_hi"]) for _ in range(B - 1)]
    old = [case["len_hi"]] + [_log_int(r, case["len_lo"], case["len_hi"]) for _ in range(B - 1)]
    return new, old


def _visible_pairs(case):
    """Per sequence: (query, key) pairs that are visible, and keys that some query sees."""
    new, old = _sizes(case)
    w, k = case["window"], case["sinks"]
    pairs, keys = [], []
    for n, c in zip(new, old):
        if w == 0:
            pairs.append(n * c + n * (n + 1) // 2)
            keys.append(c + n)
            continue
        total = 0
        for p in range(c, c + n):
            lo = max(0, p - w + 1)
            total += p + 1 - lo + min(k, lo)
        lo = max(0, c - w + 1)
        pairs.append(total)
        keys.append(c + n - lo + min(k, lo))
    return pairs, keys


def work(case):
    new, old = _sizes(case)
    N, H, Hq, D = sum(new), case["H"], case["Hq"], case["D"]
    cb = {"f32": 4, "bf16": 2, "e4m3": 1}[case["cache"]]
    ib = 4 if case["cache"] == "f32" else 2
    if case["op"] == "append":
        return {"bytes": 2 * N * Hq * D * ib + 2 * N * H * D * (ib + cb), "flops": 3 * N * (Hq + H) * case["rot"]}
    pairs, keys = _visible_pairs(case)
    bytes_ = 2 * sum(keys) * H * D * cb + 2 * N * Hq * D * ib + 4 * N * Hq
    flops = 4 * D * Hq * sum(pairs)
    if case["op"] == "core":
        k = min(case["k"], int(case["entries"] * case["fetched"]) + case["fresh"])
        bytes_ += N * k * (2 * H * D * ib + 4)
        flops += 4 * D * Hq * N * k
    return {"bytes": bytes_, "flops": flops}


# ------------------------------------------------------------------------------------- the inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dev = torch.device("cuda")
    op, B, H, Hq, D, ps = case["op"], case["B"], case["H"], case["Hq"], case["D"], case["page"]
    cdt = DTYPES[case["cache"]]
    dt = torch.float32 if cdt == torch.float32 else torch.bfloat16
    new, old = _sizes(case)
    N = sum(new)
    offs = [0]
    for n in new:
        offs.append(offs[-1] + n)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731

    # pages of the tokens that are still kept: all of them, or the window's and the first ones
    lists, used = [], 0
    for n, c in zip(new, old):
        last = (c + n - 1) // ps
        if op == "append":
            held = set(range(c // ps, last + 1))
        elif case["window"]:
            held = set(range(max(0, c - case["window"] + 1) // ps, last + 1)) | set(range((case["sinks"] + ps - 1) // ps))
        else:
            held = set(range(last + 1))
        lists.append(sorted(p for p in held if p <= last))
        used += len(lists[-1])
    max_pages = max((c + n - 1) // ps + 1 for n, c in zip(new, old))
    order = torch.randperm(used, generator=g, device=dev, dtype=torch.int64).to(torch.int32)
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, pages in enumerate(lists):
        table[b, torch.tensor(pages, device=dev)] = order[at:at + len(pages)]
        at += len(pages)

    s = dict(case=case, offs=torch.tensor(offs, dtype=torch.int64, device=dev), len=i32(old), table=table,
             n_max=max(new), len_max=max(c + n for n, c in zip(new, old)), N=N)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16 if dt == torch.bfloat16 else dt)

    shape = (used, H, ps, D)
    if cdt == torch.float8_e4m3fn:
        # codes as a cache holds them: each page's largest value near the top of the range
        make = lambda: (normal(*shape) * 70).clamp_(-448, 448).to(cdt)  # noqa: E731
        s["k_cache"], s["v_cache"] = make(), make()
        amp = lambda: torch.exp2(torch.randint(-9, -4, (used, H), generator=g, device=dev).float())  # noqa: E731
        s["k_scale"], s["v_scale"] = amp(), amp()
    else:
        s["k_cache"], s["v_cache"] = normal(*shape), normal(*shape)
        s["k_scale"] = s["v_scale"] = None

    if op == "append":
        qkv = normal(N, Hq + 2 * H, D)  # one fused projection's output: strided views
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
        s["q_out"] = torch.empty((N, Hq, D), dtype=dt, device=dev)
        R = case["rot"]
        s["inv_freq"] = None if R == 0 else (1e6 ** (-torch.arange(0, R, 2, device=dev, dtype=torch.float64) / R)).float()
        return s

    s["q"] = normal(N, Hq, D)
    s["out"] = torch.empty((N, Hq, D), dtype=dt, device=dev)
    s["lse"] = torch.empty((N, Hq), dtype=torch.float32, device=dev)
    if op == "core":
        S, k, fresh = case["entries"], case["k"], case["fresh"]
        T, F = B * S, int(S * case["fetched"])
        s["seq_offsets"] = torch.arange(0, T + 1, S, dtype=torch.int64, device=dev)
        s["idx"] = torch.zeros(T, dtype=torch.int32, device=dev)
        s["count"] = i32([F] * B)
        s["hot"] = torch.zeros((T, 2 * H * D), dtype=dt, device=dev)
        s["win"] = normal(B, fresh, 2 * H * D) if fresh else None
        s["topk"] = torch.full((N, k), -1, dtype=torch.int32, device=dev)
        for b in range(B):
            listed_ = torch.randperm(S, generator=g, device=dev)[:F].sort().values.to(torch.int32)
            s["idx"][b * S:b * S + F] = listed_
            s["hot"][b * S:b * S + F] = normal(F, 2 * H * D)
            # the best of the fetched and of the entries made since (numbered from S on), in score order
            pool = torch.cat([listed_, S + torch.arange(fresh, dtype=torch.int32, device=dev)])
            best = pool[torch.randperm(F + fresh, generator=g, device=dev)[:k]]
            s["topk"][b, :best.numel()] = best
        s["hot_bytes"] = s["hot"].view(torch.uint8)
        s["win_bytes"] = None if s["win"] is None else s["win"].view(torch.uint8)
        s["T"] = T
    return s


# ------------------------------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state)
    return _plain_append(state) if op == "append" else _plain_attend(state)


def _own(s):
    import sparse_kv_cache_memoryindexer_b200 as lsa
    c = s["case"]
    if c["op"] == "append":
        lsa.lsa_kv_append(s["k"], s["v"], s["offs"], s["len"], s["table"], s["k_cache"], s["v_cache"],
                          k_scale=s["k_scale"], v_scale=s["v_scale"], inv_freq=s["inv_freq"],
                          interleaved=c["pairs"] == "neighbours", q=s["q"], q_out=s["q_out"])
        return _append_outputs(s)
    if "ws" not in s:
        if c["op"] == "attend":
            n = lsa.lsa_window_attention_workspace_size(s["N"], c["B"], c["Hq"], c["H"], c["D"])
        else:
            n = lsa.lsa_core_attention_workspace_size(s["N"], c["B"], c["Hq"], c["H"], c["D"], c["k"])
        s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    if c["op"] == "attend":
        lsa.lsa_window_attention(s["q"], s["offs"], s["len"], s["table"], s["k_cache"], s["v_cache"], s["out"], s["ws"],
                                 window=c["window"], n_sink=c["sinks"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                                 lse_out=s["lse"])
    else:
        lsa.lsa_core_attention(s["q"], s["offs"], s["len"], s["table"], s["k_cache"], s["v_cache"], s["topk"], s["idx"],
                               s["count"], s["seq_offsets"], s["T"], s["hot_bytes"], s["out"], s["ws"],
                               win_kv=s["win_bytes"], window=c["window"], n_sink=c["sinks"], lse_out=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _append_outputs(s):
    out = {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if s["k_scale"] is not None:
        # the codes as float8 values and the power of two that each page and head multiplies them by
        out["k_scale"], out["v_scale"] = s["k_scale"], s["v_scale"]
    return out


def _tokens(s):
    """Sequence and position of every new token."""
    n = s["offs"][1:] - s["offs"][:-1]
    b = torch.repeat_interleave(torch.arange(n.numel(), device=n.device), n, output_size=s["N"])
    return b, s["len"].long()[b] + torch.arange(s["N"], device=n.device) - s["offs"][b]


def _rotate(x, pos, inv_freq, pairs):
    y = x.float()
    if inv_freq is None:
        return y
    R = 2 * inv_freq.numel()
    a = pos.double()[:, None] * inv_freq.double()  # far positions: the angle needs 64 bits
    cos, sin = torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]
    if pairs == "halves":
        x1, x2 = y[..., :R // 2], y[..., R // 2:R]
        return torch.cat([x1 * cos - x2 * sin, x2 * cos + x1 * sin, y[..., R:]], -1)
    x1, x2 = y[..., 0:R:2], y[..., 1:R:2]
    return torch.cat([torch.stack([x1 * cos - x2 * sin, x2 * cos + x1 * sin], -1).flatten(-2), y[..., R:]], -1)


def _plain_append(s):
    c = s["case"]
    b, pos = _tokens(s)
    page, slot = s["table"][b, pos // c["page"]].long(), pos % c["page"]
    s["q_out"].copy_(_rotate(s["q"], pos, s["inv_freq"], c["pairs"]))
    for name, y in (("k", _rotate(s["k"], pos, s["inv_freq"], c["pairs"])), ("v", s["v"].float())):
        cache, scale = s[name + "_cache"], s[name + "_scale"]
        if scale is None:
            cache[page, :, slot] = y.to(cache.dtype)
            continue
        amax = torch.zeros_like(scale).index_reduce_(0, page, y.abs().amax(-1), "amax")
        first = torch.full((scale.shape[0],), c["page"], dtype=torch.int64, device=scale.device)
        first = first.index_reduce_(0, page, slot, "amin")  # first new slot of a page; `page` where untouched
        m, e = torch.frexp(amax)  # amax = m 2^e, m in [1/2, 1): 448 2^x holds it from x = e - 9 (m <= 7/8) or e - 8 on
        need = torch.exp2((e - torch.where(m <= 0.875, 9, 8)).float()).clamp_min(2.0 ** -64)
        need = torch.where(amax > 0, need, 2.0 ** -64)
        kept = ((first > 0) & (first < c["page"]))[:, None]
        fresh = torch.where(kept, torch.maximum(need, scale), need)
        fresh = torch.where((first < c["page"])[:, None], fresh, scale)
        codes = (cache.float() * (scale / fresh)[:, :, None, None]).to(cache.dtype)
        earlier = torch.arange(c["page"], device=scale.device)[None, :] < first[:, None]
        moved = (fresh != scale)[:, :, None, None] & earlier[:, None, :, None]
        raw = cache.view(torch.uint8)
        raw.copy_(torch.where(moved, codes.view(torch.uint8), raw))
        raw[page, :, slot] = (y / fresh[page][:, :, None]).to(cache.dtype).view(torch.uint8)
        scale.copy_(fresh)
    return _append_outputs(s)


def _gather(cache, scale, page, slot):
    """[..., H, D] fp32 rows of the cache."""
    H = cache.shape[1]
    raw = cache.view(torch.uint8) if cache.element_size() == 1 else cache
    x = raw.permute(0, 2, 1, 3)[page, slot]
    if cache.element_size() == 1:
        return x.view(cache.dtype).float() * scale[page][..., :H, None]
    return x.float()


def _plain_attend(s):
    c = s["case"]
    H, G, D, ps, w, sinks = c["H"], c["Hq"] // c["H"], c["D"], c["page"], c["window"], c["sinks"]
    dev = s["q"].device
    b, pos = _tokens(s)
    i = pos - s["len"].long()[b]
    base = s["len"].long()
    end = base + (s["offs"][1:] - s["offs"][:-1])
    if w == 0:
        kp = torch.arange(s["len_max"], device=dev).expand(c["B"], -1)
        live = kp < end[:, None]
    else:
        lo = (base - w + 1).clamp_min(0)
        near = lo[:, None] + torch.arange(min(s["len_max"], w + s["n_max"] - 1), device=dev)
        far = torch.arange(sinks, device=dev).expand(c["B"], -1)
        kp = torch.cat([far, near], 1)
        live = torch.cat([far < torch.minimum(lo, end)[:, None], near < end[:, None]], 1)
    spot = torch.where(live, kp, base[:, None])  # any kept token stands in for a key that is not there
    page, slot = torch.gather(s["table"].long(), 1, spot // ps), spot % ps
    k, v = _gather(s["k_cache"], s["k_scale"], page, slot), _gather(s["v_cache"], s["v_scale"], page, slot)
    q = torch.zeros((c["B"], s["n_max"], c["Hq"], D), device=dev)
    q[b, i] = s["q"].float()
    q = q.view(c["B"], s["n_max"], H, G, D).permute(0, 2, 3, 1, 4).reshape(c["B"], H, G * s["n_max"], D)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) * D ** -0.5
    qp = base[:, None] + torch.arange(s["n_max"], device=dev)
    see = live[:, None, :] & (kp[:, None, :] <= qp[:, :, None])
    if w:
        see &= (kp[:, None, :] > qp[:, :, None] - w) | (kp < sinks)[:, None, :]
    x = x.view(c["B"], H, G, s["n_max"], -1).masked_fill_(~see[:, None, None], -math.inf)
    if c["op"] == "core":
        rows, there = _plain_selected(s)  # [B, k, 2, H, D]: one query token for each sequence
        xs = torch.matmul(q, rows[:, :, 0].permute(0, 2, 3, 1)) * D ** -0.5
        xs = xs.view(c["B"], H, G, 1, -1).masked_fill_(~there[:, None, None, None], -math.inf)
        x = torch.cat([x, xs], -1)
        v = torch.cat([v, rows[:, :, 1]], 1)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(c["B"], H, G * s["n_max"], -1), v.permute(0, 2, 1, 3)).view(c["B"], H, G, s["n_max"], D)
    o = o / torch.where(total > 0, total, 1.0)
    lse = (top + total.log()).squeeze(-1)
    out = o.permute(0, 3, 1, 2, 4).reshape(c["B"], s["n_max"], c["Hq"], D)[b, i]
    s["out"].copy_(out)
    s["lse"].copy_(lse.permute(0, 3, 1, 2).reshape(c["B"], s["n_max"], c["Hq"])[b, i])
    return {"out": s["out"], "lse": s["lse"]}


def _plain_selected(s):
    c = s["case"]
    S, H, D = c["entries"], c["H"], c["D"]
    top = s["topk"].long()
    F = s["count"].long()[:, None]
    held = s["idx"].view(c["B"], S)
    held = torch.where(torch.arange(S, device=held.device) < F, held, S).contiguous()
    slot = torch.searchsorted(held, top.clamp(0, S - 1).to(torch.int32)).clamp_max(S - 1)
    rows = s["hot"][slot + s["seq_offsets"][:-1, None]]
    if s["win"] is not None:
        made = torch.gather(s["win"], 1, (top - S).clamp(0, c["fresh"] - 1)[:, :, None].expand(-1, -1, 2 * H * D))
        rows = torch.where((top >= S)[:, :, None], made, rows)
    return rows.float().view(c["B"], top.shape[1], 2, H, D), top >= 0


# ------------------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attend(s)


def _exact_round_e4m3(x):
    """Nearest E4M3 value (3 mantissa bits, least exponent -6), ties to even; |x| <= 448."""
    _, e = torch.frexp(x)  # |x| in [2^(e-1), 2^e)
    step = torch.exp2((e - 4).clamp_min(-9).double())
    return torch.round(x / step) * step


def _exact_append(s):
    case = s["case"]
    new, old = _sizes(case)
    ps, R = case["page"], case["rot"]
    table = s["table"].cpu().tolist()
    q_out = torch.empty(s["q_out"].shape, dtype=torch.float64, device=s["q"].device)
    caches = {n: s[n + "_cache"].double() for n in ("k", "v")}
    scales = {n: None if s[n + "_scale"] is None else s[n + "_scale"].double() for n in ("k", "v")}
    at = 0
    for b in range(case["B"]):
        p = torch.arange(old[b], old[b] + new[b], device=q_out.device, dtype=torch.float64)
        part = slice(at, at + new[b])
        at += new[b]

        def turned(x):
            x = x.double().clone()
            if R:
                w = torch.exp(1j * p[:, None] * s["inv_freq"].double())[:, None]
                one, two = (slice(0, R // 2), slice(R // 2, R)) if case["pairs"] == "halves" else (slice(0, R, 2), slice(1, R, 2))
                z = torch.complex(x[..., one], x[..., two]) * w
                x[..., one], x[..., two] = z.real, z.imag
            return x
        q_out[part] = turned(s["q"][part])
        for n, y in (("k", turned(s["k"][part])), ("v", s["v"][part].double())):
            for j in range(old[b] // ps, (old[b] + new[b] - 1) // ps + 1):
                lo, hi = max(old[b], j * ps), min(old[b] + new[b], (j + 1) * ps)
                rows = y[lo - old[b]:hi - old[b]].transpose(0, 1)  # [H, tokens, D]
                pg, a, z = table[b][j], lo - j * ps, hi - j * ps
                if scales[n] is None:
                    caches[n][pg, :, a:z] = rows
                    continue
                need = torch.exp2(torch.ceil(torch.log2(rows.abs().amax((1, 2)) / 448))).clamp_min(2.0 ** -64)
                had = scales[n][pg].clone()
                now = torch.maximum(need, had) if a else need
                caches[n][pg, :, :a] = _exact_round_e4m3(caches[n][pg, :, :a] * (had / now)[:, None, None])
                caches[n][pg, :, a:z] = _exact_round_e4m3(rows / now[:, None, None])
                scales[n][pg] = now
    out = {"q": q_out, "k_cache": caches["k"], "v_cache": caches["v"]}
    if scales["k"] is not None:
        out["k_scale"], out["v_scale"] = scales["k"], scales["v"]
    return out


def _exact_attend(s):
    case = s["case"]
    new, old = _sizes(case)
    H, Hq, D, ps, w = case["H"], case["Hq"], case["D"], case["page"], case["window"]
    pairs, _ = _visible_pairs(case)
    if 4 * D * Hq * sum(n * (c + n) for n, c in zip(new, old)) > 4e12 and sum(pairs) > 1e8:
        return None
    dev = s["q"].device
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=dev)
    at = 0
    for b in range(case["B"]):
        end = old[b] + new[b]
        low = max(0, old[b] - w + 1) if w else 0
        keys = list(range(min(case["sinks"], low))) + list(range(low, end)) if w else list(range(end))
        j = torch.tensor(keys, device=dev)
        pg, sl = s["table"][b].long()[j // ps], j % ps
        for h in range(H):
            if s["k_scale"] is None:
                K, V = s["k_cache"][pg, h, sl].double(), s["v_cache"][pg, h, sl].double()
            else:
                K, V = (s[n + "_cache"].view(torch.uint8)[pg, h, sl].view(torch.float8_e4m3fn).double()
                        * s[n + "_scale"][pg, h].double()[:, None] for n in ("k", "v"))
            for first in range(0, new[b], 256):
                many = min(256, new[b] - first)
                me = torch.arange(old[b] + first, old[b] + first + many, device=dev)[:, None]
                hidden = j > me
                if w:
                    hidden |= (j <= me - w) & (j >= case["sinks"])
                heads = slice(h * (Hq // H), (h + 1) * (Hq // H))
                q = s["q"][at + first:at + first + many, heads].double().transpose(0, 1)
                KK, VV = K, V
                if case["op"] == "core":
                    mine = s["topk"][b][s["topk"][b] >= 0].long()
                    S = case["entries"]
                    F = int(case["entries"] * case["fetched"])
                    where = {e: n for n, e in enumerate(s["idx"][b * S:b * S + F].tolist())}
                    got = [s["hot"][b * S + where[e]] if e < S else s["win"][b, e - S] for e in mine.tolist()] if h == 0 else None
                    if h == 0:
                        chosen = torch.stack(got).double().view(-1, 2, H, D)
                    KK, VV = torch.cat([K, chosen[:, 0, h]]), torch.cat([V, chosen[:, 1, h]])
                    hidden = torch.cat([hidden, torch.zeros((many, chosen.shape[0]), dtype=torch.bool, device=dev)], 1)
                x = (q @ KK.T / math.sqrt(D)).masked_fill(hidden, -math.inf)
                lse[at + first:at + first + many, heads] = torch.logsumexp(x, -1).T
                out[at + first:at + first + many, heads] = (torch.softmax(x, -1) @ VV).transpose(0, 1)
        at += new[b]
    return {"out": out, "lse": lse}
