"""Edges of the decoder operators on the GPU, against the float64 definition:
partial results of the two paged kernels side by side, rows that see few keys,
sink gradients of many sequences, streams."""
import pytest
import torch

from sparse_attention_banded_b200 import build, lf
from tests._window_ref import check, half_step, reference, subnormal_half_step
from tests.test_gpu_paged import Case

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


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


@pytest.mark.parametrize("q,kv,Hq,Hkv", [
    ([1, 150, 1, 3, 0, 1, 40, 2], [5000, 3000, 30, 7000, 9, 1, 2500, 4097], 8, 2),    # slots by sequence
    ([1, 17, 1], [6000, 5000, 100], 2, 2),                                            # slots by sequence, 16 each
    ([16, 17, 16, 15, 1], [3000, 2000, 40, 2500, 4000], 3, 3),                        # slots by token
    ([5, 6, 5, 1], [3000, 5000, 7, 2500], 3, 1)])                                     # the same, three heads a group
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_pieces_of_both_kernels_in_one_call(dtype, q, kv, Hq, Hkv):
    """Contexts cut by the decode kernel next to ones cut by the tensor-core
    kernel, in a table wide enough for several pieces of each."""
    c = Case(q, kv, Hq, Hkv, 16, dtype, seed=len(q) + Hq, extra=1000)
    n, T, wide = len(q), c.q.shape[0], c.table.shape[1]
    short = lf.lf_paged_attention_workspace_bytes(n, Hq, Hkv, T, 16 // (Hq // Hkv), wide, 16, c.w, 0)
    both = lf.lf_paged_attention_workspace_bytes(n, Hq, Hkv, T, max(q), wide, 16, c.w, 0)
    assert 0 < short < both
    c.run().check()


def _bound_without_out(q, k, v, w, sinks, do, scale=0.125):
    """dQ and dK and their bounds where delta is no sum with the rounded out.
    With e the relative error of a probability (fp32 scores of 64 products,
    at most S in size, against a log-sum-exp of as many; the exponential and
    the logarithm 2^-21), u half a step, z the subnormal half step:
        dP     2^-18 |dout|.|v|                  (64 fp32 products)
        delta  sum_j p_j (2 e + 2^-18) |dout|.|v_j|
        dS     E = p (both) + (u + 2 e + 2^-20) |dS| + z
        dq     scale sum_j E |k_j| + u |dq| + z;  dk likewise."""
    u, z = half_step(q.dtype), subnormal_half_step(q.dtype)
    r = reference(q, k, v, 0, w, sinks, scale, do)
    G = q.shape[0] // k.shape[0]
    q, k, v, do = q.double(), k.double().repeat_interleave(G, 0), v.double().repeat_interleave(G, 0), do.double()
    n = q.shape[1]
    i, j = torch.arange(n, device="cuda")[:, None], torch.arange(n, device="cuda")[None]
    ok = (j <= i) & ((i - j <= w) | (j < sinks))
    p = torch.softmax((q @ k.mT * scale).masked_fill(~ok, float("-inf")), -1)
    S = float((q.abs() @ k.abs().mT * scale).where(ok, 0.0).max())
    e = 2.0 ** -24 * (128 * S + n + 64) + 2.0 ** -21
    dp, dpa = do @ v.mT, do.abs() @ v.abs().mT
    ds = p * (dp - (p * dp).sum(-1, keepdim=True))
    E = p * (2.0 ** -18 * dpa + (2 * e + 2.0 ** -18) * (p * dpa).sum(-1, keepdim=True)) + (u + 2 * e + 2.0 ** -20) * ds.abs()
    E = E + z * ok
    b_dq = scale * E @ k.abs() + u * r["dq"].abs() + z
    b_dk = (scale * E.mT @ q.abs()).view(-1, G, n, 64).sum(1) + u * r["dk"].abs() + z
    return r["dq"], b_dq, r["dk"], b_dk


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("Hq,Hkv", [(3, 3), (4, 2), (10, 1)])
@pytest.mark.parametrize("w,sinks", [(1, 1), (1, 2), (1, 4), (0, 1), (0, 3), (5, 2), (1, 0), (27, 4), (0, 31)])
def test_gradients_of_rows_that_see_few_keys(dtype, Hq, Hkv, w, sinks):
    """Up to 32 keys a row, sinks among them, whatever the number of heads a
    group: dP and delta nearly cancel, and the rounding of out is no part of
    the error."""
    lens = [900, 1, 333]
    g = torch.Generator().manual_seed(w + 10 * sinks + Hq)
    q, k, v, do = (torch.randn(sum(lens), h, 64, generator=g).to(DT[dtype]).cuda() for h in (Hq, Hkv, Hkv, Hq))
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    do2 = do.view(sum(lens), Hq * 64)
    out, lse = lf.lf_window_attention_forward(q, k, v, w, sinks, cu_seqlens=cu)
    dq, dk, _ = lf.lf_window_attention_backward(q, k, v, out, lse, do2, w, sinks, cu_seqlens=cu)
    at = 0
    for n in lens:
        s = slice(at, at + n)
        rq, bq, rk, bk = _bound_without_out(*(t[s].transpose(0, 1) for t in (q, k, v)), w, sinks, do[s].transpose(0, 1))
        check("dq", dq[s].transpose(0, 1), rq, bq)
        check("dk", dk[s].transpose(0, 1), rk, bk)
        at += n


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("lens,w,sinks", [
    ([300, 20, 700, 7], 5, 4),                 # partials numbered by sequence
    ([30, 2, 1, 26, 27, 0] * 30 + [650], 25, 4),  # by start / (w + 2)
    ([20, 1, 0, 2, 3, 4, 5] * 20, 2, 33),      # by token
    ([150] * 5, 140, 130),                     # chunks that hold queries of the window only
    ([64, 64], 63, 2)])                        # no query outside the window
@pytest.mark.parametrize("Hq,Hkv", [(4, 2), (5, 5)])
def test_sink_gradients_of_many_sequences(dtype, lens, w, sinks, Hq, Hkv):
    """Every partial is written before it is read, and none past the
    workspace's end: it holds NaN before, and what follows it stays."""
    g = torch.Generator().manual_seed(len(lens) + w)
    T, tail = sum(lens), 3
    q, k, v, do = (torch.randn(T + tail, h, 64, generator=g).to(DT[dtype]).cuda() for h in (Hq, Hkv, Hkv, Hq))
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    need = lf.lf_window_attention_backward_workspace_bytes(True, len(lens), Hq, Hkv, T + tail, w, sinks)
    buf = torch.full((need + 65536,), 255, dtype=torch.uint8, device="cuda")
    out, lse = lf.lf_window_attention_forward(q, k, v, w, sinks, cu_seqlens=cu)
    got = lf.lf_window_attention_backward(q, k, v, out, lse, do.view(T + tail, -1), w, sinks, cu_seqlens=cu,
                                          workspace=buf[:need])
    assert bool((buf[need:] == 255).all())
    at = 0
    for n in lens:
        if n:
            s = slice(at, at + n)
            r = reference(*(t[s].transpose(0, 1) for t in (q, k, v)), 0, w, sinks, 0.125, do[s].transpose(0, 1))
            for name, t in zip(("dq", "dk", "dv"), got):
                check(name, t[s].transpose(0, 1), r[name], r["b_" + name])
        at += n


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("sinks", [298, 299, 300, 301, (1 << 31) - 1])
def test_sinks_up_to_every_key(dtype, sinks):
    """From L - 1 sinks on the attention is plainly causal: the same bits as
    a window of that length, forward and backward."""
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(2, h, 300, 64, generator=g).to(DT[dtype]).cuda() for h in (4, 2, 2))
    do = torch.randn(2, 300, 256, generator=g).to(DT[dtype]).cuda()
    out, lse = lf.lf_window_attention_forward(q, k, v, 3, sinks)
    got = lf.lf_window_attention_backward(q, k, v, out, lse, do, 3, sinks)
    for b in range(2):
        r = reference(q[b], k[b], v[b], 0, 3, sinks, 0.125, do[b].view(300, 4, 64).transpose(0, 1))
        check("out", out[b].view(300, 4, 64).transpose(0, 1), r["out"], r["b_out"])
        for name, t in zip(("dq", "dk", "dv"), got):
            check(name, t[b], r[name], r["b_" + name])
    if sinks >= 299:
        out2, lse2 = lf.lf_window_attention_forward(q, k, v, 300, 0)
        want = lf.lf_window_attention_backward(q, k, v, out2, lse2, do, 300, 0)
        assert torch.equal(out, out2) and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_sinks_far_wider_than_the_sequences(dtype):
    """4.2 million sinks, short sequences, most of the packed rows in none."""
    lens, T, w, sinks = [1000, 5, 130], 4300000, 2100000, 4200000
    g = torch.Generator().manual_seed(4)
    q, k, v, do = (torch.zeros(T, 1, 64, dtype=DT[dtype], device="cuda") for _ in range(4))
    for t in (q, k, v, do):
        t[:sum(lens)] = torch.randn(sum(lens), 1, 64, generator=g).to(DT[dtype]).cuda()
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    out, lse = lf.lf_window_attention_forward(q, k, v, w, sinks, cu_seqlens=cu)
    got = lf.lf_window_attention_backward(q, k, v, out, lse, do.view(T, 64), w, sinks, cu_seqlens=cu)
    at = 0
    for n in lens:
        s = slice(at, at + n)
        r = reference(*(t[s].transpose(0, 1) for t in (q, k, v)), 0, w, sinks, 0.125, do[s].transpose(0, 1))
        for name, t in zip(("dq", "dk", "dv"), got):
            check(name, t[s].transpose(0, 1), r[name], r["b_" + name])
        at += n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_more_sinks_than_keys_beyond_the_window(dtype):
    """Several blocks of sinks, of which short sequences have the first alone."""
    lens, w, sinks, Hq, Hkv = [700, 100, 60, 300, 129], 40, 400, 2, 1
    g = torch.Generator().manual_seed(5)
    q, k, v, do = (torch.randn(sum(lens), h, 64, generator=g).to(DT[dtype]).cuda() for h in (Hq, Hkv, Hkv, Hq))
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    out, lse = lf.lf_window_attention_forward(q, k, v, w, sinks, cu_seqlens=cu)
    got = lf.lf_window_attention_backward(q, k, v, out, lse, do.view(-1, Hq * 64), w, sinks, cu_seqlens=cu)
    at = 0
    for n in lens:
        s = slice(at, at + n)
        r = reference(*(t[s].transpose(0, 1) for t in (q, k, v)), 0, w, sinks, 0.125, do[s].transpose(0, 1))
        for name, t in zip(("dq", "dk", "dv"), got):
            check(name, t[s].transpose(0, 1), r[name], r["b_" + name])
        at += n


def _calls_on_a_stream():
    h = lambda *s: torch.randn(*s, device="cuda").half()  # noqa: E731
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731

    def window(st):
        q = h(2, 4, 300, 64)
        return [q], lambda: lf.lf_window_attention_forward(q, q, q, 20, 2, stream=st)[0]

    def backward(st):
        q, do = h(2, 4, 300, 64), h(2, 300, 256)
        out, lse = lf.lf_window_attention_forward(q, q, q, 20, 2)
        return [do], lambda: lf.lf_window_attention_backward(q, q, q, out, lse, do, 20, 2, stream=st)[0]

    def append(st):
        k, c, table, cu, kv = h(300, 4, 64), h(40, 4, 16, 64), torch.arange(40, dtype=torch.int32, device="cuda")[None], i32(0, 300), i32(300)
        return [k], lambda: (lf.lf_paged_cache_append(k, k, c, c, table, cu, kv, stream=st), c)[1]

    def paged(st):
        q, c, table, cu, kv = h(300, 4, 64), h(40, 4, 16, 64), torch.arange(40, dtype=torch.int32, device="cuda")[None], i32(0, 300), i32(300)
        return [q], lambda: lf.lf_paged_attention_forward(q, c, c, table, cu, kv, 300, stream=st)

    def norm(st):
        x = h(500, 512)
        return [x], lambda: lf.lf_layer_norm_forward(x, stream=st)[0]

    def norm_backward(st):
        x, dy = h(500, 512), h(500, 512)
        _, mean, rstd = lf.lf_layer_norm_forward(x)
        return [dy], lambda: lf.lf_layer_norm_backward(dy, x, None, mean, rstd, stream=st)[0]

    return dict(window=window, backward=backward, append=append, paged=paged, norm=norm, norm_backward=norm_backward)


@pytest.mark.parametrize("name", ["window", "backward", "append", "paged", "norm", "norm_backward"])
def test_an_input_freed_before_the_other_stream_has_read_it(name):
    """The caller lets go of an input while the call on another stream still
    waits: its memory is not handed out again."""
    side = torch.cuda.Stream()
    inputs, call = _calls_on_a_stream()[name](side)
    want = call().clone() if name != "append" else None
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)  # 0.1 s
    got = call()
    ptr, shape = inputs[0].data_ptr(), inputs[0].shape
    if name == "append":
        want = inputs[0].clone()
    del call, inputs
    new = [torch.full(shape, 7.0, dtype=torch.float16, device="cuda") for _ in range(4)]
    assert ptr not in [t.data_ptr() for t in new]
    torch.cuda.synchronize()
    if name == "append":
        got = got[:, :, :].transpose(1, 2).reshape(-1, 4, 64)[:300]
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("n", [33000, 48005, 65500])
def test_dv_of_late_keys_in_a_long_context(dtype, n):
    """q = 0: P is 1 / (i + 1), below fp16's 2^-14 in rows past 16384, and as
    exact as in other rows.  The log-sum-exp is ln(i + 1) from an exact sum:
    15.6 in log2, rounded three times at 2^-24 and off by 2^-22 from the
    logarithm, so P is off by e = 2^-18 and by its rounding, u; the last 64
    keys' sums have at most 64 terms (2^-18), and are rounded once:
        (u + 2^-17) sum p |dout| + u |dv| + z."""
    g = torch.Generator().manual_seed(n)
    q = torch.zeros(1, 1, n, 64, dtype=DT[dtype], device="cuda")
    k, v = (torch.randn(1, 1, n, 64, generator=g).to(DT[dtype]).cuda() for _ in range(2))
    do = (8 + 8 * torch.rand(1, n, 64, generator=g)).to(DT[dtype]).cuda()
    out, lse = lf.lf_window_attention_forward(q, k, v, n)
    _, _, dv = lf.lf_window_attention_backward(q, k, v, out, lse, do, n)
    p = 1 / torch.arange(n - 63, n + 1, dtype=torch.double, device="cuda")[:, None]
    want = (p * do[0, -64:].double()).flip(0).cumsum(0).flip(0)
    u, z = half_step(DT[dtype]), subnormal_half_step(DT[dtype])
    check("dv", dv[0, 0, -64:], want, (2 * u + 2.0 ** -17) * want + z)  # (all terms are positive)


@pytest.mark.parametrize("rows", [(1 << 31) - 1, (1 << 31) - 8])
def test_layer_norm_of_the_last_row_counts(rows):
    """One column: x is its own mean, y is beta, dx is 0."""
    x = torch.empty(rows, 1, dtype=torch.float16, device="cuda")
    x.view(-1)[:] = 1.0
    x[-5:, 0] = torch.arange(5, dtype=torch.float16, device="cuda")
    gamma, beta = torch.full((1,), 2.0, device="cuda"), torch.full((1,), 0.5, device="cuda")
    y, mean, rstd = lf.lf_layer_norm_forward(x, gamma, beta)
    for at in (slice(0, 10), slice(rows // 2, rows // 2 + 10), slice(rows - 10, rows)):
        assert torch.equal(mean[at], x[at, 0].float()) and bool((y[at] == 0.5).all())
    y.fill_(7.0)
    dx, dgamma, _ = lf.lf_layer_norm_backward(x, x, gamma, mean, rstd, dx=y)
    for at in (slice(0, 10), slice(rows // 2, rows // 2 + 10), slice(rows - 10, rows)):
        assert bool((dx[at] == 0).all())
    assert float(dgamma) == 0
    del x, y, mean, rstd, dx
    torch.cuda.empty_cache()  # 35 GB


@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_layer_norm_past_2_31_elements(dtype):
    rows, N = (1 << 21) + 5, 1030
    x = torch.empty(rows, N, dtype=DT[dtype], device="cuda")
    g = torch.Generator().manual_seed(9)
    few = torch.tensor([0, 1, rows // 2, rows - 2, rows - 1], device="cuda")
    x.fill_(1.0)
    x[:, ::2] = -1.0
    x[few] = torch.randn(5, N, generator=g).to(DT[dtype]).cuda()
    dy = x.clone()
    y, mean, rstd = lf.lf_layer_norm_forward(x)
    dx, _, dbeta = lf.lf_layer_norm_backward(dy, x, None, mean, rstd)
    small = x[few].clone()
    y2, mean2, rstd2 = lf.lf_layer_norm_forward(small)
    dx2, _, dbeta2 = lf.lf_layer_norm_backward(small, small, None, mean2, rstd2)
    assert torch.equal(y[few], y2) and torch.equal(mean[few], mean2) and torch.equal(dx[few], dx2)
    # the other rows are +-1 in turn: integers below 2^24 a block, exact; the
    # five others' sums are rounded on the way (2^-24 of 2^21, a few times)
    want = dbeta2.double() + torch.where(torch.arange(N, device="cuda") % 2 == 0, -1.0, 1.0).double() * (rows - 5)
    assert float((dbeta.double() - want).abs().max()) <= 8 * 2.0 ** -3
