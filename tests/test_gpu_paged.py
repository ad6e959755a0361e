"""Attention of new tokens over a paged cache, and appending to it, against
the float64 definition: page sizes, chunk and context lengths, grouped heads,
windows and sinks, freed and missing pages, poisoned slots; and a run of the
serving steps against the attention over whole sequences."""
import random

import pytest
import torch

from sparse_attention_banded_b200 import build, lf
from tests._window_ref import check, reference

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
ALL = (1 << 31) - 1


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    lf.lib()
    lf.lf_device_status(reset=True)
    yield


@pytest.fixture(autouse=True)
def _status():
    yield
    assert lf.lf_device_status(reset=True) == 0


class Case:
    """Contexts in a shuffled pool of pages; every slot that holds no position
    is NaN, and so are the pages of no sequence."""

    def __init__(self, qlens, kvlens, Hq, Hkv, page, dtype="f16", seed=0, w=ALL, sinks=0, token_major=False, tail=2,
                 free=True, extra=3, stale=False):
        g = torch.Generator().manual_seed(seed)
        r = random.Random(seed)
        dt = DT[dtype]
        self.qlens, self.kvlens, self.Hq, self.Hkv, self.page, self.w, self.sinks = qlens, kvlens, Hq, Hkv, page, w, sinks
        n = len(qlens)
        need = [-(-m // page) for m in kvlens]
        self.num_pages = sum(need) + 2
        shape = (self.num_pages, page, Hkv, 64) if token_major else (self.num_pages, Hkv, page, 64)
        self.kc, self.vc = (torch.full(shape, float("nan"), dtype=dt, device="cuda") for _ in range(2))
        if token_major:
            self.kc, self.vc = self.kc.transpose(1, 2), self.vc.transpose(1, 2)
        pool = list(range(self.num_pages))
        r.shuffle(pool)
        self.k = [torch.randn(Hkv, m, 64, generator=g).to(dt).cuda() for m in kvlens]
        self.v = [torch.randn(Hkv, m, 64, generator=g).to(dt).cuda() for m in kvlens]
        table = torch.full((n, max(need + [1]) + extra), -1, dtype=torch.int32)
        for b in range(n):
            first = max(0, kvlens[b] - qlens[b] - w)
            for j in range(need[b]):
                p = pool.pop()
                lo, hi = j * page, min(kvlens[b], (j + 1) * page)
                if free and hi <= first and lo >= sinks:
                    if stale:
                        table[b, j] = p  # the entry still names a page, which holds NaN
                    continue  # wholly behind the window: freed
                table[b, j] = p
                old = kvlens[b] - qlens[b]  # the new tokens' slots are filled by the append
                if lo < old:
                    self.kc[p, :, :min(hi, old) - lo] = self.k[b][:, lo:min(hi, old)]
                    self.vc[p, :, :min(hi, old) - lo] = self.v[b][:, lo:min(hi, old)]
        self.table = table.cuda()
        T = sum(qlens) + tail
        self.q = torch.randn(T, Hq, 64, generator=g).to(dt).cuda()
        self.q[sum(qlens):] = float("nan")
        self.cu = torch.tensor([0] + qlens).cumsum(0).to(torch.int32).cuda()
        self.kv = torch.tensor(kvlens, dtype=torch.int32).cuda()
        self.out = torch.full((T, Hq * 64), 7.0, dtype=dt, device="cuda")
        news = [torch.cat([t[b][:, kvlens[b] - qlens[b]:].transpose(0, 1) for b in range(n)] +
                          [torch.full((tail, Hkv, 64), float("nan"), dtype=dt, device="cuda")]) for t in (self.k, self.v)]
        self.kn, self.vn = news

    def run(self):
        lf.lf_paged_cache_append(self.kn, self.vn, self.kc, self.vc, self.table, self.cu, self.kv)
        need = lf.lf_paged_attention_workspace_bytes(len(self.qlens), self.Hq, self.Hkv, self.q.shape[0],
                                                     max(self.qlens), self.table.shape[1], self.page, self.w, self.sinks)
        ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda") if need else None
        lf.lf_paged_attention_forward(self.q, self.kc, self.vc, self.table, self.cu, self.kv, max(self.qlens), self.w,
                                      self.sinks, out=self.out, workspace=ws)
        torch.cuda.synchronize()
        return self

    def check(self, skip=()):
        at = 0
        for b, (n, m) in enumerate(zip(self.qlens, self.kvlens)):
            if n and b not in skip:
                r = reference(self.q[at:at + n].transpose(0, 1), self.k[b], self.v[b], m - n, self.w, self.sinks)
                check("out of sequence %d" % b, self.out[at:at + n].view(n, self.Hq, 64).transpose(0, 1), r["out"], r["b_out"])
            at += n
        assert bool((self.out[at:] == 7.0).all()), "rows behind the last sequence were written"
        return self


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("page", [8, 16, 64, 128, 512])
def test_decode(dtype, page):
    Case([1] * 9, [1, 2, 63, 64, 65, 200, 777, 1025, 3000], 8, 2, page, dtype, seed=page).run().check()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("page", [8, 32, 256])
def test_chunks(dtype, page):
    Case([5, 64, 130, 0, 300, 33], [5, 64, 777, 0, 1300, 2222], 4, 2, page, dtype, seed=page).run().check()


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 2), (3, 1), (8, 1), (10, 2), (16, 2), (17, 1), (64, 1), (33, 1)])
@pytest.mark.parametrize("qlen", [1, 2, 40])
def test_grouped_heads(Hq, Hkv, qlen):
    Case([qlen, 1], [300, 90], Hq, Hkv, 16, seed=Hq + qlen).run().check()


@pytest.mark.parametrize("w,sinks", [(0, 0), (0, 4), (1, 1), (63, 0), (64, 4), (100, 70), (1000, 16), (ALL, 5)])
@pytest.mark.parametrize("qlens", [[1, 1, 1, 1], [70, 1, 3, 200]])
def test_windows_sinks_and_freed_pages(w, sinks, qlens):
    Case(qlens, [70, 400, 1111, 2500], 4, 1, 16, "bf16", seed=w % 97 + sinks, w=w, sinks=sinks).run().check()


@pytest.mark.parametrize("page", [8, 64])
def test_what_no_query_sees_may_be_anything(page):
    """Stale table entries behind the window, and the positions before the
    window (or past the sinks) in pages that are still held: NaN."""
    c = Case([1, 70, 3, 2], [700, 400, 1111, 90], 4, 2, page, "bf16", seed=page, w=100, sinks=3, stale=True)
    for b, (n, m) in enumerate(zip(c.qlens, c.kvlens)):
        for j in range(c.sinks, max(c.sinks, m - n - c.w)):
            p = int(c.table[b, j // page])
            if p >= 0:
                c.kc[p, :, j % page] = float("nan")
                c.vc[p, :, j % page] = float("nan")
    c.run().check()


def test_cache_with_heads_inside_pages():
    Case([1, 40], [500, 300], 4, 2, 32, seed=3, token_major=True).run().check()


def test_long_context_few_heads():
    """One sequence whose context is split over many CTAs."""
    Case([1], [20011], 2, 1, 64, "f16", seed=4).run().check()
    Case([17], [20011], 2, 1, 64, "bf16", seed=5).run().check()


def test_mixed_batch():
    q = [1, 256, 1, 1, 77, 1, 200, 1, 0, 1, 3]
    kv = [4097, 256, 33, 7777, 2077, 1, 5000, 8000, 9, 640, 12]
    Case(q, kv, 8, 2, 16, "bf16", seed=6, w=1024, sinks=4).run().check()


def test_wide_table():
    """The table may be far wider than any context."""
    Case([1, 2], [100, 5], 4, 2, 8, seed=7, extra=5000).run().check()


def test_append_writes_only_its_slots():
    c = Case([3, 0, 20], [40, 17, 20], 2, 2, 16, seed=8)
    before = c.kc.clone()
    c.run().check()
    changed = (c.kc.float().nan_to_num(123.0) != before.float().nan_to_num(123.0)).any(-1).any(1)  # [pages, slot]
    want = torch.zeros_like(changed)
    for b, (n, m) in enumerate(zip(c.qlens, c.kvlens)):
        for j in range(m - n, m):
            want[int(c.table[b, j // 16]), j % 16] = True
    assert torch.equal(changed, want)


def _page_case(edit, kv=None, qlens=(1, 40), kvlens=(200, 300), **kw):
    c = Case(list(qlens), list(kvlens), 4, 2, 16, seed=9, **kw)
    lf.lf_paged_cache_append(c.kn, c.vn, c.kc, c.vc, c.table, c.cu, c.kv)
    assert lf.lf_device_status(reset=True) == 0
    edit(c)
    lf.lf_paged_attention_forward(c.q, c.kc, c.vc, c.table, c.cu, c.kv, max(qlens), c.w, c.sinks, out=c.out)
    torch.cuda.synchronize()
    return c


@pytest.mark.parametrize("entry", [-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1])
@pytest.mark.parametrize("b", [0, 1])
def test_missing_pages_are_recorded_and_left_out(entry, b):
    def edit(c):
        c.table[b, 2] = entry
    c = _page_case(edit)
    assert lf.lf_device_status(reset=True) == 16
    c.check(skip=(b,))
    n, m, at = c.qlens[b], c.kvlens[b], sum(c.qlens[:b])
    vis = torch.ones(n, m, dtype=torch.bool).tril(m - n)
    vis[:, 32:48] = False
    r = reference(c.q[at:at + n].transpose(0, 1), c.k[b], c.v[b], m - n, c.w, c.sinks, visible=vis)
    check("out", c.out[at:at + n].view(n, 4, 64).transpose(0, 1), r["out"], r["b_out"])


def test_rows_with_no_page_left_are_zero():
    def edit(c):
        c.table[:] = -1
    c = _page_case(edit)
    assert lf.lf_device_status(reset=True) == 16
    assert bool((c.out[:41] == 0).all()) and bool((c.out[41:] == 7).all())


@pytest.mark.parametrize("kv,status", [([10 ** 9, 300], 15), ([200, 20], 15), ([-7, 300], 15), ([0, 300], 15)])
def test_lengths_that_do_not_fit(kv, status):
    def edit(c):
        c.kv.copy_(torch.tensor(kv, dtype=torch.int32))
    c = _page_case(edit)
    assert lf.lf_device_status(reset=True) == status
    assert bool((c.out[41:] == 7).all())
    if kv[1] == 300:
        c.check(skip=(0,))
        if kv[0] <= 0:
            assert bool((c.out[:1] == 0).all())
    else:  # its first 20 tokens stand at positions below 0
        c.check(skip=(1,))
        assert bool((c.out[1:21] == 0).all()) and bool(torch.isfinite(c.out[21:41]).all())


def test_longer_than_the_bound():
    c = Case([1, 40], [200, 300], 4, 2, 16, seed=10)
    lf.lf_paged_cache_append(c.kn, c.vn, c.kc, c.vc, c.table, c.cu, c.kv)
    for bound in (1, 39):
        c.out.fill_(7.0)
        lf.lf_paged_attention_forward(c.q, c.kc, c.vc, c.table, c.cu, c.kv, bound, out=c.out)
        assert lf.lf_device_status(reset=True) == 15
        assert bool((c.out[1:] == 7).all())
        c.check(skip=(1,))


def test_append_refuses_missing_pages():
    c = Case([3, 2], [40, 17], 2, 2, 16, seed=11)
    before = c.kc.clone()
    c.table[0, 2] = -1
    lf.lf_paged_cache_append(c.kn, c.vn, c.kc, c.vc, c.table, c.cu, c.kv)
    assert lf.lf_device_status(reset=True) == 16
    page = int(c.table[1, 0])
    same = torch.arange(c.num_pages, device="cuda") != page
    same[int(c.table[1, 1])] = False
    assert torch.equal(c.kc[same].nan_to_num(9.0), before[same].nan_to_num(9.0))
    c.kv.copy_(torch.tensor([2, 17], dtype=torch.int32))  # three new tokens, two positions
    lf.lf_paged_cache_append(c.kn, c.vn, c.kc, c.vc, c.table, c.cu, c.kv)
    assert lf.lf_device_status(reset=True) == 15


def test_captured_steps_follow_the_lengths():
    """One captured decode step, replayed while contexts grow; workspaces
    belong to the captured call."""
    w, sinks = 100, 2
    Hq, Hkv, page, n, steps = 4, 2, 16, 3, 40
    g = torch.Generator().manual_seed(12)
    full = [[torch.randn(steps, h, n, 64, generator=g).half().cuda() for h in (Hq, Hkv, Hkv)]][0]
    start = [0, 100, 700]
    old = [torch.randn(Hkv, s, 64, generator=g).half().cuda() for s in start]
    oldv = [torch.randn(Hkv, s, 64, generator=g).half().cuda() for s in start]
    pages = 64
    kc, vc = (torch.full((n * pages, Hkv, page, 64), float("nan"), dtype=torch.float16, device="cuda") for _ in range(2))
    table = torch.arange(n * pages, dtype=torch.int32).view(n, pages).cuda()
    kv = torch.tensor(start, dtype=torch.int32).cuda()
    for b in range(n):
        if start[b]:
            cu0 = torch.tensor([0, start[b]], dtype=torch.int32).cuda()
            lf.lf_paged_cache_append(old[b].transpose(0, 1), oldv[b].transpose(0, 1), kc, vc, table[b:b + 1].contiguous(),
                                     cu0, kv[b:b + 1].clone())
    cu = torch.arange(n + 1, dtype=torch.int32).cuda()
    q, k, v = (torch.empty(n, h, 64, dtype=torch.float16, device="cuda") for h in (Hq, Hkv, Hkv))

    def step():
        lf.lf_paged_cache_append(k, v, kc, vc, table, cu, kv)
        return lf.lf_paged_attention_forward(q, kc, vc, table, cu, kv, 1, w, sinks)

    for t, src in zip((q, k, v), full):
        t.copy_(src[0].transpose(0, 1))
    kv += 1
    step()
    kv -= 1
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    outs = []
    for t in range(steps):
        for x, src in zip((q, k, v), full):
            x.copy_(src[t].transpose(0, 1))
        kv += 1
        graph.replay()
        outs.append(out.clone())
    torch.cuda.synchronize()
    for b in range(n):
        kk = torch.cat([old[b], full[1][:, :, b].transpose(0, 1)], 1)
        vv = torch.cat([oldv[b], full[2][:, :, b].transpose(0, 1)], 1)
        r = reference(full[0][:, :, b].transpose(0, 1), kk, vv, start[b], w, sinks)
        got = torch.stack([o[b].view(Hq, 64) for o in outs], 1)
        check("sequence %d" % b, got, r["out"], r["b_out"])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_serving_equals_the_whole_sequence(dtype):
    """Prompts prefilled in chunks, then tokens one by one, through layer
    norm, the cache and the attention: each step's output equals (to the two
    calls' rounding bounds) the window attention over the whole sequence."""
    w, sinks, Hq, Hkv, page = 90, 3, 4, 2, 16
    lens = [230, 61]
    n = len(lens)
    g = torch.Generator().manual_seed(13)
    dt = DT[dtype]
    D = (Hq + 2 * Hkv) * 64
    x = [torch.randn(m, D, generator=g).to(dt).cuda() for m in lens]
    gamma = (1 + 0.1 * torch.randn(D, generator=g)).cuda()
    norm = lambda t: lf.lf_layer_norm_forward(t, gamma)[0]  # noqa: E731  (stands for norm + projection)
    cut = lambda t: (t[:, :Hq], t[:, Hq:Hq + Hkv], t[:, Hq + Hkv:])  # noqa: E731
    whole = [norm(t).view(-1, Hq + 2 * Hkv, 64) for t in x]
    cu_all = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    want, _ = lf.lf_window_attention_forward(*cut(torch.cat(whole)), w, sinks, cu_seqlens=cu_all)
    kc, vc = (torch.full((64, Hkv, page, 64), float("nan"), dtype=dt, device="cuda") for _ in range(2))
    table = torch.randperm(64, generator=g)[:n * 20].view(n, 20).to(torch.int32).cuda()
    done, got = [0, 0], [[], []]
    chunks = [[100, 90], [37, 3]]
    while any(done[b] < lens[b] for b in range(n)):
        take = [min(lens[b] - done[b], chunks[b].pop(0) if chunks[b] else 1) for b in range(n)]
        h = norm(torch.cat([x[b][done[b]:done[b] + take[b]] for b in range(n)])).view(-1, Hq + 2 * Hkv, 64)
        q, k, v = cut(h)
        done = [d + t for d, t in zip(done, take)]
        cu = torch.tensor([0] + take).cumsum(0).to(torch.int32).cuda()
        kv = torch.tensor(done, dtype=torch.int32).cuda()
        lf.lf_paged_cache_append(k, v, kc, vc, table, cu, kv)
        o = lf.lf_paged_attention_forward(q, kc, vc, table, cu, kv, max(take), w, sinks)
        for b in range(n):
            got[b].append(o[int(cu[b]):int(cu[b + 1])])
            for j in range(max(0, done[b] - w) // page):  # free what is behind the window
                if j * page >= sinks:
                    table[b, j] = -1
    got = torch.cat([torch.cat(t) for t in got])
    at = 0
    for b, m in enumerate(lens):
        q, k, v = (t.transpose(0, 1) for t in cut(whole[b]))
        r = reference(q, k, v, 0, w, sinks)
        for name, t in (("window", want), ("paged", got)):
            check(name, t[at:at + m].view(m, Hq, 64).transpose(0, 1), r["out"], r["b_out"])
        at += m


def test_training_block_gradients():
    """A decoder attention block trained as it would be used: layer norm,
    fused projection, windowed attention, output projection, residual; the
    library's gradients chained by hand against torch autograd in float64.
    fp32, so the bound is a relative 2^-24 times the lengths of the sums
    (largest 512 terms), eight of them in a row, on the largest value."""
    T, D, Hq, Hkv, w, s = 150, 128, 4, 2, 31, 2
    g = torch.Generator().manual_seed(14)
    f = lambda *sh, sc=1.0: (torch.randn(*sh, generator=g) * sc).cuda()  # noqa: E731
    x, gamma, beta = f(T, D), 1 + f(D, sc=0.1), f(D, sc=0.1)
    Wqkv, Wo, dy = f((Hq + 2 * Hkv) * 64, D, sc=D ** -0.5), f(D, Hq * 64, sc=0.05), f(T, D)
    cu = torch.tensor([0, 100, T], dtype=torch.int32).cuda()
    cut = lambda t: (t[:, :Hq], t[:, Hq:Hq + Hkv], t[:, Hq + Hkv:])  # noqa: E731
    h, mean, rstd = lf.lf_layer_norm_forward(x, gamma, beta)
    qkv = (h @ Wqkv.T).view(T, -1, 64)
    a, lse = lf.lf_window_attention_forward(*cut(qkv), w, s, cu_seqlens=cu)
    y = x + a @ Wo.T
    da = dy @ Wo
    dqkv = torch.empty_like(qkv)
    dq, dk, dv = cut(dqkv)
    lf.lf_window_attention_backward(*cut(qkv), a, lse, da, w, s, cu_seqlens=cu, dq=dq, dk=dk, dv=dv)
    d2 = dqkv.view(T, -1)
    dx, dgamma, dbeta = lf.lf_layer_norm_backward(d2 @ Wqkv, x, gamma, mean, rstd)
    got = dict(y=y, x=dx + dy, gamma=dgamma, beta=dbeta, Wqkv=d2.T @ h, Wo=dy.T @ a)
    L = {n: t.double().requires_grad_() for n, t in dict(x=x, gamma=gamma, beta=beta, Wqkv=Wqkv, Wo=Wo).items()}
    hh = torch.nn.functional.layer_norm(L["x"], (D,), L["gamma"], L["beta"], 1e-5)
    p = (hh @ L["Wqkv"].T).view(T, -1, 64).transpose(0, 1)
    i = torch.arange(T, device="cuda")
    start = torch.where(i < 100, 0, 100)
    rel = i[None] - start[:, None]
    ok = (i[None] <= i[:, None]) & (rel >= 0) & ((i[:, None] - i[None] <= w) | (rel < s))
    kk, vv = (t.repeat_interleave(Hq // Hkv, 0) for t in (p[Hq:Hq + Hkv], p[Hq + Hkv:]))
    sc = (p[:Hq] @ kk.mT / 8).masked_fill(~ok, float("-inf"))
    o = (torch.softmax(sc, -1) @ vv).transpose(0, 1).reshape(T, -1)
    yy = L["x"] + o @ L["Wo"].T
    yy.backward(dy.double())
    for n, t in got.items():
        want = yy.detach() if n == "y" else L[n].grad
        assert float((t.double() - want).abs().max()) <= 8 * 512 * 2.0 ** -24 * float(want.abs().max()), n


def test_sequences_share_pages():
    """Two sequences forked from one prompt: the same pages in both tables,
    each with a last page of its own."""
    c = Case([1, 5], [133, 140], 4, 2, 16, seed=20)
    c.k[1][:, :128], c.v[1][:, :128] = c.k[0][:, :128], c.v[0][:, :128]
    c.table[1, :8] = c.table[0, :8]
    c.run().check()


def test_two_calls_at_once():
    """Two batches on two streams, workspaces of their own."""
    cases = [Case([1, 30, 1], [900, 500, 3000], 8, 2, 16, seed=21 + i, w=700, sinks=2) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        for c, st in zip(cases, streams):
            lf.lf_paged_cache_append(c.kn, c.vn, c.kc, c.vc, c.table, c.cu, c.kv, stream=st)
            lf.lf_paged_attention_forward(c.q, c.kc, c.vc, c.table, c.cu, c.kv, 30, c.w, c.sinks, out=c.out, stream=st)
    torch.cuda.synchronize()
    for c in cases:
        c.check()


def test_cache_of_more_than_2_31_elements():
    """Pages whose offsets pass 32 bits (a pool of 2.6e9 elements a cache;
    only the pages in use are written)."""
    pages, Hkv, page = 80000, 8, 64
    kc, vc = (torch.empty(pages, Hkv, page, 64, dtype=torch.float16, device="cuda") for _ in range(2))
    g = torch.Generator().manual_seed(22)
    qlens, kvlens = [1, 40], [200, 100]
    table = torch.tensor([[79999, 3, 70001, 66000], [65537, 79998, 5, 6]], dtype=torch.int32).cuda()
    k, v = ([torch.randn(Hkv, m, 64, generator=g).half().cuda() for m in kvlens] for _ in range(2))
    kv = torch.tensor(kvlens, dtype=torch.int32).cuda()
    for b, m in enumerate(kvlens):
        lf.lf_paged_cache_append(k[b].transpose(0, 1), v[b].transpose(0, 1), kc, vc, table[b:b + 1].contiguous(),
                                 torch.tensor([0, m], dtype=torch.int32).cuda(), kv[b:b + 1].clone())
    q = torch.randn(41, 16, 64, generator=g).half().cuda()
    cu = torch.tensor([0, 1, 41], dtype=torch.int32).cuda()
    out = lf.lf_paged_attention_forward(q, kc, vc, table, cu, kv, 40)
    at = 0
    for b, (n, m) in enumerate(zip(qlens, kvlens)):
        r = reference(q[at:at + n].transpose(0, 1), k[b], v[b], m - n, 1 << 29, 0)
        check("sequence %d" % b, out[at:at + n].view(n, 16, 64).transpose(0, 1), r["out"], r["b_out"])
        at += n


def test_one_context_in_many_pieces():
    """A context cut into more pieces than one warp joins (a block per row),
    and a table whose pieces are mostly empty."""
    Case([1], [40000], 2, 1, 64, seed=23).run().check()
    Case([1, 1], [40000, 30], 4, 1, 64, seed=24, w=30000, sinks=3).run().check()
    Case([1], [100], 4, 1, 64, seed=25, extra=1000).run().check()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("w,sinks", [(ALL, 0), (100, 4)])
def test_more_chunks_than_the_gpu_holds(dtype, w, sinks):
    """Equal chunks of many sequences, more tiles than two per SM."""
    Case([17] * 90, [17 + (97 * i * i) % 700 for i in range(90)], 8, 4, 16, dtype, seed=w % 83, w=w, sinks=sinks).run().check()


def test_many_ragged_chunks_next_to_single_tokens():
    q = [1 + (7 * i * i) % 90 * (i % 2) for i in range(150)]
    kv = [n + (53 * i) % 400 for i, n in enumerate(q)]
    Case(q, kv, 10, 5, 32, "bf16", seed=9, w=300, sinks=2).run().check()
