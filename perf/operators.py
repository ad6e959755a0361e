"""Operator benchmark cases: windowed causal attention with sink tokens, its
backward pass, the same attention over a paged key/value cache, and layer
norm's forward and backward pass.

Each case is run in one of two forms: ``own`` False computes the operator with
elementary torch operations in fp32 (one rounding at the end), ``own`` True
calls the library's entry points.  :func:`exact` evaluates the definition in
float64.

Definitions (head_dim 64, scale 1/8, G = Hq / Hkv query heads share a
key/value head): in a sequence, the query at position i sees the keys
{ j <= i : i - j <= w or j < sinks }.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ELEM = {"f32": 4, "f16": 2, "bf16": 2}
HD = 64
SCALE = 0.125
NO_WINDOW = 1 << 30


def _ints(text):
    return [int(t) for t in text.split(",")]


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # One short prompt of a small grouped-head model: a launch-latency call.
        dict(name="window_short_bf16", op="window", mode="forward", dtype="bf16", packed=True, lens="100", L=100,
             Hq=16, Hkv=4, w=64, sinks=4),
        # The fp32 test shape (H 2, L 512, w 64, 8 always-visible tokens), one training pass.
        dict(name="window_train_f32", op="window", mode="train", dtype="f32", packed=False, lens="512", L=512,
             Hq=2, Hkv=2, w=64, sinks=8),
        # A padded batch in the [B, H, L, 64] layout with Longformer-large's heads, inference.
        dict(name="window_batch_f16", op="window", mode="forward", dtype="f16", packed=False,
             lens="3642,3625,3149,3478", L=4096, Hq=16, Hkv=16, w=256, sinks=4),
        # Packed documents of ragged lengths, grouped heads: a training pass of one layer's attention.
        dict(name="window_train_bf16", op="window", mode="train", dtype="bf16", packed=True,
             lens="7001,1,4093,513,2900,127,1749", L=16384, Hq=16, Hkv=4, w=1024, sinks=4),
        # One long document, 12 heads, window 256, 32 always-visible tokens: training.
        dict(name="window_train_f16", op="window", mode="train", dtype="f16", packed=False, lens="16384", L=16384,
             Hq=12, Hkv=12, w=256, sinks=32),
        # One user's next token over a short context.
        dict(name="paged_token_f16", op="paged", dtype="f16", qlens="1", kvlens="1000", pages=64, page=16,
             Hq=16, Hkv=4, w=NO_WINDOW, sinks=0),
        # A serving batch of single tokens over ragged contexts, no window.
        dict(name="paged_decode_bf16", op="paged", dtype="bf16", qlens=",".join(["1"] * 48),
             kvlens=",".join(str(1 + (7919 * i * i + 613 * i) % 8192) for i in range(48)), pages=128, page=64,
             Hq=16, Hkv=4, w=NO_WINDOW, sinks=0),
        # Two prompts prefilled in chunks of 1024 over long contexts, window 4096 and sinks.
        dict(name="paged_chunk_f16", op="paged", dtype="f16", qlens="1024,1024", kvlens="15000,6144", pages=120,
             page=128, Hq=16, Hkv=4, w=4096, sinks=4),
        # A continuous batch: prompts' chunks next to single tokens, window 1024, pages behind the window freed.
        dict(name="paged_mixed_bf16", op="paged", dtype="bf16", qlens="1,256,1,1,77,1,200,1,1,1,3,1,1,1,1,1",
             kvlens="4097,256,33,7777,2077,1,5000,8000,1025,640,12,2222,6400,129,511,3071",
             pages=512, page=16, Hq=16, Hkv=4, w=1024, sinks=4),
        # A few tokens' layer norm while generating, hidden 1024.
        dict(name="norm_rows_f16", op="norm", mode="forward", dtype="f16", rows=8, N=1024),
        # The layer norm of one training step, 16384 tokens of hidden 1024.
        dict(name="norm_train_bf16", op="norm", mode="train", dtype="bf16", rows=16384, N=1024),
        # An odd width in fp32.
        dict(name="norm_train_f32", op="norm", mode="train", dtype="f32", rows=5001, N=1537),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_window(rng):
    dtype = rng.choice(["f16", "bf16", "f16", "bf16", "f32"])
    mode = rng.choice(["forward", "train"])
    top = 1024 if dtype == "f32" else 8192
    Hkv = rng.choice([1, 2, 3, 4])
    Hq = Hkv * rng.choice([1, 2, 3, 4])
    w = 0 if rng.random() < 0.05 else _log_int(rng, 1, 256 if dtype == "f32" else 768)
    sinks = rng.choice([0, 1, 4, 5, 16, 33, 64])
    packed = rng.random() < 0.5
    lens = [_log_int(rng, 1, top) for _ in range(rng.randint(1, 6))]
    while len(lens) > 1 and (sum(lens) if packed else len(lens) * max(lens)) > 2 * top:
        lens.pop()
    L = sum(lens) if packed else max(lens)
    return dict(op="window", mode=mode, dtype=dtype, packed=packed, lens=",".join(map(str, lens)), L=L, Hq=Hq,
                Hkv=Hkv, w=w, sinks=sinks)


def _draw_paged(rng):
    page = rng.choice([8, 16, 32, 64, 128, 256])
    Hkv = rng.choice([1, 2, 3, 4])
    kind = rng.choice(["decode", "chunk", "mixed"])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 8] if kind == "decode" else [1, 2, 3, 4])
    if kind == "decode":
        n = _log_int(rng, 1, 48)
        kv = [_log_int(rng, 1, 8192) for _ in range(n)]
        q = [1] * n
    else:
        n = rng.randint(1, 6)
        kv = [_log_int(rng, 1, 8192) for _ in range(n)]
        q = [1 if kind == "mixed" and rng.random() < 0.5 else _log_int(rng, 1, min(k, 512)) for k in kv]
    w = NO_WINDOW if rng.random() < 0.4 else _log_int(rng, 16, 4096)
    return dict(op="paged", dtype=rng.choice(["f16", "bf16"]), qlens=",".join(map(str, q)),
                kvlens=",".join(map(str, kv)), pages=-(-max(kv) // page), page=page, Hq=Hq, Hkv=Hkv, w=w,
                sinks=0 if w == NO_WINDOW else rng.choice([0, 1, 4, 16]))


def _draw_norm(rng):
    N = _log_int(rng, 33, 4096)
    if rng.random() < 0.6:
        N = max(64, N // 64 * 64)
    rows = _log_int(rng, 1, min(16384, (1 << 24) // N))
    return dict(op="norm", mode=rng.choice(["forward", "train"]), dtype=rng.choice(["f32", "f16", "bf16"]),
                rows=rows, N=N)


def draw(rng):
    return rng.choice([_draw_window, _draw_paged, _draw_norm])(rng)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def randn(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dt)

    if case["op"] == "norm":
        rows, N = case["rows"], case["N"]
        return dict(case=case, x=randn(rows, N) + randn(1, N, scale=0.5), dy=randn(rows, N),
                    gamma=1.0 + 0.1 * torch.randn(N, generator=g, device="cuda"),
                    beta=0.1 * torch.randn(N, generator=g, device="cuda"))
    if case["op"] == "window":
        lens, L, Hq, Hkv = _ints(case["lens"]), case["L"], case["Hq"], case["Hkv"]
        n = len(lens)
        st = dict(case=case)
        if case["packed"]:
            cu = torch.tensor([0] + lens).cumsum(0)
            st["cu"] = cu.to(torch.int32).cuda()
            # the projections' output for one packed batch: [T, heads, 64]
            st["q"], st["k"], st["v"] = randn(L, Hq, HD), randn(L, Hkv, HD), randn(L, Hkv, HD)
            st["dout"] = randn(L, Hq * HD)
            seq = torch.repeat_interleave(torch.arange(n), torch.tensor(lens))
            st["seq"], st["pos"] = seq.cuda(), (torch.arange(L) - cu[seq]).cuda()
        else:
            st["lens"] = torch.tensor(lens, dtype=torch.int32).cuda()
            st["q"], st["k"], st["v"] = (randn(n, h, L, HD) for h in (Hq, Hkv, Hkv))
            st["dout"] = randn(n, L, Hq * HD)
        return st
    # paged: a pool of pages handed out in random order
    ql, kl, P, MP, Hkv = _ints(case["qlens"]), _ints(case["kvlens"]), case["page"], case["pages"], case["Hkv"]
    n, T = len(ql), sum(ql)
    rng = random.Random(seed)
    need = [-(-k // P) for k in kl]
    pool = list(range(sum(need) + 3))
    rng.shuffle(pool)
    table = [[-1] * MP for _ in range(n)]
    for b in range(n):
        first = max(0, kl[b] - ql[b] - case["w"]) // P  # pages before this one hold no visible key but the sinks
        for j in range(need[b]):
            page = pool.pop()
            if j >= first or j * P < case["sinks"]:
                table[b][j] = page
    num_pages = sum(need) + 3
    st = dict(case=case, q=randn(T, case["Hq"], HD), k=randn(T, Hkv, HD), v=randn(T, Hkv, HD),
              k_cache=randn(num_pages, Hkv, P, HD), v_cache=randn(num_pages, Hkv, P, HD),
              table=torch.tensor(table, dtype=torch.int32).cuda(),
              cu=torch.tensor([0] + ql).cumsum(0).to(torch.int32).cuda(),
              kv_lens=torch.tensor(kl, dtype=torch.int32).cuda(), max_q=max(ql))
    seq = torch.repeat_interleave(torch.arange(n), torch.tensor(ql)).cuda()
    st["seq"], st["row"] = seq, torch.arange(T, device="cuda") - st["cu"].long()[seq]
    return st


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------
def _band(x, C):
    """[X, T, 64] -> [X, T / C, 2 C, 64]: each chunk's keys and the chunk's before it."""
    x = x.unflatten(1, (-1, C))
    return torch.cat([torch.nn.functional.pad(x, (0, 0, 0, 0, 1, 0))[:, :-1], x], 2)


def _unband(x, C):
    """The transpose of :func:`_band`."""
    return (x[:, :, C:] + torch.nn.functional.pad(x[:, 1:, :C], (0, 0, 0, 0, 0, 1))).flatten(1, 2)


def _plain_window(st):
    case = st["case"]
    Hq, Hkv, w, S, L = case["Hq"], case["Hkv"], case["w"], case["sinks"], case["L"]
    G, dt = Hq // Hkv, DTYPES[case["dtype"]]
    if case["packed"]:
        # one row per head over the packed tokens; other sequences' keys are masked
        q, k, v = (st[n].transpose(0, 1).float() for n in "qkv")
        X, do = 1, st["dout"].view(1, L, Hq, HD).transpose(1, 2).reshape(Hq, L, HD).float()
        seq, pos, first = st["seq"][None], st["pos"][None], (st["cu"].long()[st["seq"]])[None]
        n_tok = torch.diff(st["cu"]).long()[st["seq"]][None]
        real = torch.ones(1, L, dtype=torch.bool, device="cuda")
    else:
        X = st["q"].shape[0]
        q, k, v = (st[n].flatten(0, 1).float() for n in "qkv")
        do = st["dout"].view(X, L, Hq, HD).transpose(1, 2).reshape(X * Hq, L, HD).float()
        pos = torch.arange(L, device="cuda").expand(X, L)
        n_tok = st["lens"].long()[:, None].expand(X, L)
        real = pos < n_tok
        seq = torch.where(real, 0, -1)
        first = torch.zeros_like(pos)
    # chunks at least as wide as the window, so a query's window lies in its chunk and the one before
    C = max(1, min(max(w, 64), L))
    pad = -L % C
    padt = lambda t: torch.nn.functional.pad(t, (0, 0, 0, pad))  # noqa: E731
    q, k, v, do = padt(q), padt(k), padt(v), padt(do)
    padi = lambda t, x: torch.nn.functional.pad(t, (0, pad), value=x).unflatten(1, (-1, C))  # noqa: E731
    qs, qp, qr = padi(seq, -1), padi(pos, 0), padi(real, False)
    prev = lambda t, x: torch.cat([torch.nn.functional.pad(t, (0, 0, 1, 0), value=x)[:, :-1], t], 2)  # noqa: E731
    ks, kp, kr = prev(qs, -2), prev(qp, 0), prev(qr, False)
    d = qp[..., None] - kp[..., None, :]
    ok = (qs[..., None] == ks[..., None, :]) & qr[..., None] & kr[..., None, :] & (d >= 0) & (d <= w)
    nC = ok.shape[1]
    ok = ok[:, None, :, None]                                             # [X, 1, nC, 1, C, 2C]
    q6 = q.view(X, Hkv, G, nC, C, HD).transpose(2, 3)                     # [X, Hkv, nC, G, C, 64]
    k6, v6 = (_band(t, C).view(X, Hkv, nC, 1, 2 * C, HD) for t in (k, v))
    s_band = torch.where(ok, q6 @ k6.mT * SCALE, -torch.inf)
    # the sinks: the first S tokens of each query's sequence, outside its window
    o = torch.arange(S, device="cuda")
    sp = padi(first, 0)[..., None] + o                                    # [X, nC, C, S] token index
    oks = qr[..., None] & (qp[..., None] - o > w) & (o < padi(n_tok, 0)[..., None])
    sp = torch.where(oks, sp, 0)
    at = (torch.arange(X, device="cuda").view(X, 1, 1, 1, 1), torch.arange(Hkv, device="cuda").view(1, Hkv, 1, 1, 1),
          sp[:, None])
    oks = oks[:, None, :, None]
    k_s, v_s = (t.view(X, Hkv, -1, HD)[at] for t in (k, v))               # [X, Hkv, nC, C, S, 64]
    s_sink = torch.where(oks, torch.einsum("xhngcd,xhncsd->xhngcs", q6, k_s) * SCALE, -torch.inf)
    s = torch.cat([s_band, s_sink], -1)
    del s_band, s_sink
    m = s.amax(-1, keepdim=True).clamp(min=-1e30)
    s = torch.exp(s - m)
    p = s / s.sum(-1, keepdim=True).clamp(min=1e-30)
    del s
    pb, ps = p[..., :2 * C], p[..., 2 * C:]
    out = pb @ v6 + torch.einsum("xhngcs,xhncsd->xhngcd", ps, v_s)

    def tokens(t):  # [X, Hkv, nC, G, C, 64] -> [X, Hq, L, 64]
        return t.transpose(2, 3).reshape(X, Hq, nC * C, HD)[:, :, :L]

    def rows(t):  # -> [X, L, Hq * 64]
        t = tokens(t).transpose(1, 2).flatten(2).to(dt)
        return t[0] if case["packed"] else t

    if case["mode"] == "forward":
        return {"out": rows(out)}
    do6 = do.view(X, Hkv, G, nC, C, HD).transpose(2, 3)
    delta = (do6 * out).sum(-1, keepdim=True)
    dsb = pb * (do6 @ v6.mT - delta) * SCALE
    dss = ps * (torch.einsum("xhngcd,xhncsd->xhngcs", do6, v_s) - delta) * SCALE
    dq = dsb @ k6 + torch.einsum("xhngcs,xhncsd->xhngcd", dss, k_s)

    def keys(band, sink, rhs):
        t = _unband((band.mT @ rhs).sum(3).flatten(0, 1), C).view(X, Hkv, nC * C, HD)
        t = t.index_put(at, torch.einsum("xhngcs,xhngcd->xhncsd", sink, rhs), accumulate=True)[:, :, :L]
        return (t[0].transpose(0, 1) if case["packed"] else t).to(dt)

    dq_out = (tokens(dq)[0].transpose(0, 1) if case["packed"] else tokens(dq)).to(dt)
    return {"out": rows(out), "dq": dq_out, "dk": keys(dsb, dss, q6), "dv": keys(pb, ps, do6)}


def _plain_paged(st):
    case = st["case"]
    Hq, Hkv, P = case["Hq"], case["Hkv"], case["page"]
    G, B, MQ = Hq // Hkv, st["table"].shape[0], st["max_q"]
    seq, row = st["seq"], st["row"]
    cu, kv = st["cu"].long(), st["kv_lens"].long()
    first = kv - torch.diff(cu)                          # position of each sequence's first new token
    pos = first[seq] + row
    page = st["table"].long()[seq, pos // P]
    st["k_cache"][page, :, pos % P] = st["k"]
    st["v_cache"][page, :, pos % P] = st["v"]
    held = st["table"].clamp(min=0).long()
    k, v = (st[n][held].transpose(1, 2).reshape(B, Hkv, -1, HD).float() for n in ("k_cache", "v_cache"))
    q = torch.zeros(B, MQ, Hq, HD, device="cuda")
    q[seq, row] = st["q"].float()
    q = q.view(B, MQ, Hkv, G, HD).permute(0, 2, 1, 3, 4).reshape(B, Hkv, MQ * G, HD)
    s = q @ k.mT * SCALE
    i = (first[:, None] + torch.arange(MQ, device="cuda")).repeat_interleave(G, 1)[:, None, :, None]
    j = torch.arange(k.shape[2], device="cuda")
    ok = (j <= i) & ((i - j <= case["w"]) | (j < case["sinks"])) & (j < kv[:, None, None, None])
    s = torch.where(ok, s, -torch.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True).clamp(min=-1e30))
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = (p @ v).view(B, Hkv, MQ, G, HD).transpose(1, 2).reshape(B, MQ, Hq * HD)
    return {"out": o[seq, row].to(st["q"].dtype), "k_cache": st["k_cache"], "v_cache": st["v_cache"]}


def _plain_norm(st):
    x, dt = st["x"].float(), st["x"].dtype
    c = x - x.mean(-1, keepdim=True)
    rstd = torch.rsqrt((c * c).mean(-1, keepdim=True) + 1e-5)
    xh = c * rstd
    y = (xh * st["gamma"] + st["beta"]).to(dt)
    if st["case"]["mode"] == "forward":
        return {"y": y}
    dy = st["dy"].float()
    g = dy * st["gamma"]
    dx = rstd * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
    return {"y": y, "dx": dx.to(dt), "dgamma": (dy * xh).sum(0), "dbeta": dy.sum(0)}


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(st):
    case = st["case"]
    if not own:
        return {"window": _plain_window, "paged": _plain_paged, "norm": _plain_norm}[case["op"]](st)
    from sparse_attention_banded_b200 import lf
    if case["op"] == "window":
        at = dict(sinks=case["sinks"], cu_seqlens=st.get("cu"), seq_lens=st.get("lens"))
        out, lse = lf.lf_window_attention_forward(st["q"], st["k"], st["v"], case["w"], **at)
        if case["mode"] == "forward":
            return {"out": out}
        dq, dk, dv = lf.lf_window_attention_backward(st["q"], st["k"], st["v"], out, lse, st["dout"], case["w"], **at)
        return {"out": out, "dq": dq, "dk": dk, "dv": dv}
    if case["op"] == "paged":
        lf.lf_paged_cache_append(st["k"], st["v"], st["k_cache"], st["v_cache"], st["table"], st["cu"],
                                 st["kv_lens"])
        out = lf.lf_paged_attention_forward(st["q"], st["k_cache"], st["v_cache"], st["table"], st["cu"],
                                            st["kv_lens"], st["max_q"], w=case["w"], sinks=case["sinks"])
        return {"out": out, "k_cache": st["k_cache"], "v_cache": st["v_cache"]}
    if case["mode"] == "forward":
        return {"y": lf.lf_layer_norm_forward(st["x"], st["gamma"], st["beta"])[0]}
    y, mean, rstd = lf.lf_layer_norm_forward(st["x"], st["gamma"], st["beta"])
    dx, dgamma, dbeta = lf.lf_layer_norm_backward(st["dy"], st["x"], st["gamma"], mean, rstd)
    return {"y": y, "dx": dx, "dgamma": dgamma, "dbeta": dbeta}


# --------------------------------------------------------------------------
# work of one pass
# --------------------------------------------------------------------------
def _pairs(n, w, S, start=0):
    """Query-key pairs of the queries at positions start .. n-1."""
    total = 0
    for i in range(start, n):
        lo = max(0, i - w)
        total += i - lo + 1 + min(S, lo)
    return total


def work(case):
    e = ELEM[case["dtype"]]
    if case["op"] == "norm":
        n = case["rows"] * case["N"]
        if case["mode"] == "forward":
            return {"bytes": 2 * n * e + 8 * case["N"], "flops": 8 * n}
        return {"bytes": 4 * n * e + 16 * case["N"], "flops": 22 * n}
    Hq, Hkv, w, S = case["Hq"], case["Hkv"], case["w"], case["sinks"]
    if case["op"] == "window":
        lens = _ints(case["lens"])
        T, pairs = sum(lens), Hq * sum(_pairs(n, w, S) for n in lens)
        q, kv = T * Hq * HD * e, T * Hkv * HD * e
        if case["mode"] == "forward":
            return {"bytes": 2 * q + 2 * kv, "flops": 4 * HD * pairs}
        # forward: q, k, v read, out written; the gradient: dout read, dq, dk, dv written
        return {"bytes": 4 * q + 4 * kv, "flops": 14 * HD * pairs}
    nbytes = pairs = 0
    for ql, kl in zip(_ints(case["qlens"]), _ints(case["kvlens"])):
        lo = max(0, kl - ql - w)
        seen = kl - lo + min(S, lo)
        nbytes += 2 * ql * Hq * HD * e + 2 * seen * Hkv * HD * e + 2 * ql * Hkv * HD * e
        pairs += Hq * _pairs(kl, w, S, kl - ql)
    return {"bytes": nbytes, "flops": 4 * HD * pairs}


# --------------------------------------------------------------------------
# the definition in float64
# --------------------------------------------------------------------------
def _exact_rows(q, k, v, i0, w, S, do=None):
    """q [H, n, 64] at positions i0 .. i0+n-1 over k, v [H, m, 64] (float64):
    out, and with do the gradients (dq [H, n, 64], dk, dv [H, m, 64])."""
    H, n, m = q.shape[0], q.shape[1], k.shape[1]
    out, dq = torch.zeros_like(q), torch.zeros_like(q)
    dk, dv = torch.zeros_like(k), torch.zeros_like(v)
    step = 512
    for a in range(0, n, step):
        b = min(n, a + step)
        lo, hi = max(0, i0 + a - w), min(m, i0 + b)
        idx = torch.cat([torch.arange(min(S, lo)), torch.arange(lo, hi)]).cuda()
        i = torch.arange(i0 + a, i0 + b, device="cuda")[:, None]
        hidden = (idx > i) | ((i - idx > w) & (idx >= S))
        kk, vv = k[:, idx], v[:, idx]
        p = torch.softmax((torch.einsum("hnd,hmd->hnm", q[:, a:b], kk) / 8).masked_fill(hidden, float("-inf")), -1)
        out[:, a:b] = torch.einsum("hnm,hmd->hnd", p, vv)
        if do is not None:
            d = do[:, a:b]
            dp = torch.einsum("hnd,hmd->hnm", d, vv)
            ds = p * (dp - (p * dp).sum(-1, keepdim=True)) / 8
            dq[:, a:b] = torch.einsum("hnm,hmd->hnd", ds, kk)
            dk.index_add_(1, idx, torch.einsum("hnm,hnd->hmd", ds, q[:, a:b]))
            dv.index_add_(1, idx, torch.einsum("hnm,hnd->hmd", p, d))
    return out, dq, dk, dv


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        x = st["x"].double()
        gamma, beta = st["gamma"].double(), st["beta"].double()
        mu, var = x.mean(1, keepdim=True), x.var(1, unbiased=False, keepdim=True)
        sd = (var + 1e-5).sqrt()
        xh = (x - mu) / sd
        res = {"y": xh * gamma + beta}
        if case["mode"] == "train":
            dy = st["dy"].double()
            u = dy * gamma
            res["dx"] = (u - u.mean(1, keepdim=True) - xh * (u * xh).mean(1, keepdim=True)) / sd
            res["dgamma"], res["dbeta"] = (dy * xh).sum(0), dy.sum(0)
        return res
    Hq, Hkv, w, S = case["Hq"], case["Hkv"], case["w"], case["sinks"]
    G = Hq // Hkv
    if case["op"] == "window":
        lens, L, train = _ints(case["lens"]), case["L"], case["mode"] == "train"
        start = 0
        names = ("out", "dq", "dk", "dv") if train else ("out",)
        parts = {n: [] for n in names}
        for b, n in enumerate(lens):
            if case["packed"]:
                q, k, v = (st[t][start:start + n].transpose(0, 1).double() for t in "qkv")
                do = st["dout"][start:start + n]
                start += n
            else:
                q, k, v = (st[t][b, :, :n].double() for t in "qkv")
                do = st["dout"][b, :n]
            do = do.reshape(n, Hq, HD).transpose(0, 1).double()
            k, v = k.repeat_interleave(G, 0), v.repeat_interleave(G, 0)
            r = _exact_rows(q, k, v, 0, w, S, do if train else None)
            r = (r[0], r[1], r[2].view(Hkv, G, n, HD).sum(1), r[3].view(Hkv, G, n, HD).sum(1))
            for name, t in zip(names, r):
                if not case["packed"]:
                    t = torch.nn.functional.pad(t, (0, 0, 0, L - n))
                t = t.transpose(0, 1) if case["packed"] or name == "out" else t
                parts[name].append(t.flatten(1) if name == "out" else t)
        return {n: torch.cat(t) if case["packed"] else torch.stack(t) for n, t in parts.items()}
    ql, kl, P = _ints(case["qlens"]), _ints(case["kvlens"]), case["page"]
    kc, vc = st["k_cache"].double(), st["v_cache"].double()
    table, outs, at = st["table"].cpu().tolist(), [], 0
    for b in range(len(ql)):
        for t in range(ql[b]):
            j = kl[b] - ql[b] + t
            kc[table[b][j // P], :, j % P] = st["k"][at + t].double()
            vc[table[b][j // P], :, j % P] = st["v"][at + t].double()
        held = [max(0, t) for t in table[b][:-(-kl[b] // P)]]
        k, v = (c[held].transpose(0, 1).reshape(Hkv, -1, HD)[:, :kl[b]].repeat_interleave(G, 0) for c in (kc, vc))
        q = st["q"][at:at + ql[b]].transpose(0, 1).double()
        o = _exact_rows(q, k, v, kl[b] - ql[b], w, S)[0]
        outs.append(o.transpose(0, 1).flatten(1))
        at += ql[b]
    return {"out": torch.cat(outs), "k_cache": kc, "v_cache": vc}
