"""Windowed causal attention with sinks and its gradients against the float64
definition, with element-wise bounds derived from the kernels' roundings:
layouts, grouped heads, windows and sinks around tile edges, empty and
one-token sequences, padding, poisoned storage outside the sequences, other
streams, captured graphs."""
import pytest
import torch

from sparse_attention_banded_b200 import build, lf
from tests._window_ref import check, reference

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


def _rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(DT[dtype]).cuda()


def _compare(got, seqs, w, sinks, scale=0.125):
    """got and seqs: per sequence the tensors [H, n, 64] (lse [H, n])."""
    for g, (q, k, v, do) in zip(got, seqs):
        if q.shape[1] == 0:
            continue
        r = reference(q, k, v, 0, w, sinks, scale, do)
        for name in g:
            check(name, g[name], r[name], r["b_" + name])


def _packed(lens, Hq, Hkv, w, sinks, dtype, seed=0, tail=3, fused=False, scale=0.125):
    """Run forward and backward on packed sequences with `tail` rows behind
    the last one, poisoned with NaN; fused: q, k, v and their gradients are
    slices of one [T, (Hq + 2 Hkv) * 64] buffer."""
    T = sum(lens) + tail
    dt = DT[dtype]
    nan = float("nan")
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    end = sum(lens)
    Hall = Hq + 2 * Hkv
    x = _rand((T, Hall, 64), dtype, seed)
    x[end:] = nan
    dx = torch.full((T, Hall, 64), 7.0, dtype=dt, device="cuda")
    cut = lambda t: (t[:, :Hq], t[:, Hq:Hq + Hkv], t[:, Hq + Hkv:])  # noqa: E731
    q, k, v = cut(x) if fused else (t.contiguous() for t in cut(x))
    dq, dk, dv = cut(dx) if fused else (t.contiguous() for t in cut(dx))
    do = _rand((T, Hq * 64), dtype, seed + 1)
    do[end:] = nan
    out = torch.full((T, Hq * 64), 7.0, dtype=dt, device="cuda")
    lse = torch.full((1, Hq, T), 7.0, device="cuda")
    ws = torch.full((lf.lf_window_attention_backward_workspace_bytes(True, len(lens), Hq, Hkv, T, w, sinks),), 255,
                    dtype=torch.uint8, device="cuda")  # NaN patterns
    lf.lf_window_attention_forward(q, k, v, w, sinks, scale, cu_seqlens=cu, out=out, lse=lse)
    lf.lf_window_attention_backward(q, k, v, out, lse, do, w, sinks, scale, cu_seqlens=cu, dq=dq, dk=dk, dv=dv,
                                    workspace=ws)
    torch.cuda.synchronize()
    for t in (out, dq, dk, dv):
        assert bool((t[end:] == 7.0).all()), "rows behind the last sequence were written"
    assert bool((lse[:, :, end:] == 7.0).all())
    got, seqs, at = [], [], 0
    for n in lens:
        s = slice(at, at + n)
        row = lambda t: t[s].view(n, t[0].numel() // 64, 64).transpose(0, 1)  # noqa: E731
        got.append(dict(out=row(out), lse=lse[0, :, s], dq=row(dq), dk=row(dk), dv=row(dv)))
        seqs.append((row(q), row(k), row(v), row(do)))
        at += n
    _compare(got, seqs, w, sinks, scale)
    return out, lse, dq, dk, dv


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("w,sinks", [(0, 0), (0, 3), (1, 1), (63, 4), (64, 0), (65, 70), (100, 130), (1 << 30, 4)])
def test_packed_windows_and_sinks(dtype, w, sinks):
    _packed([1, 0, 200, 64, 129, 333, 2], 4, 2, w, sinks, dtype, seed=w + sinks)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (6, 2), (8, 1), (10, 2), (64, 1), (14, 2), (33, 1)])
def test_grouped_heads(dtype, Hq, Hkv):
    _packed([150, 17], Hq, Hkv, 40, 3, dtype, seed=Hq, fused=True)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_longer_sequences(dtype):
    _packed([2300, 700], 4, 2, 500, 5, dtype, seed=5)
    _packed([1500], 2, 2, 1 << 30, 0, dtype, seed=6)


@pytest.mark.parametrize("Hq,Hkv,w", [(16, 16, 256), (16, 4, 700)])
def test_a_full_grid(Hq, Hkv, w):
    """More tiles than the GPU holds at once, several blocks each: every
    CTA's roles run at their own pace (the device status word stays clear)."""
    _packed([4096, 3001], Hq, Hkv, w, 4, "f16", seed=7)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_many_short_sequences(dtype):
    lens = [(7 * i * i + 3 * i) % 40 for i in range(70)]
    _packed(lens, 2, 1, 9, 2, dtype, seed=8, tail=0)


def test_scale_and_large_scores():
    """A peaked softmax: scores up to several hundred."""
    _packed([190, 70], 2, 1, 77, 2, "f16", seed=9, scale=1.5)
    _packed([190, 70], 2, 1, 77, 2, "f32", seed=9, scale=1.5)


def _padded(dtype, lens, L, Hq, Hkv, w, sinks, layout, seed=0, poison=True, with_lens=True):
    B = len(lens)
    dt = DT[dtype]

    def make(H, s):
        t = _rand((B, H, L, 64), dtype, s)
        for b, n in enumerate(lens):
            if poison:
                t[b, :, n:] = float("nan")
        if layout == "blhd":
            return t.transpose(1, 2).contiguous().transpose(1, 2)
        if layout == "gap":  # every row 72 elements apart
            big = torch.full((B, H, L, 72), float("nan"), dtype=dt, device="cuda")
            big[..., :64] = t
            return big[..., :64]
        return t

    q, k, v = make(Hq, seed), make(Hkv, seed + 1), make(Hkv, seed + 2)
    do = _rand((B, L, Hq * 64), dtype, seed + 3)
    for b, n in enumerate(lens):
        if poison:
            do[b, n:] = float("nan")
    sl = torch.tensor(lens, dtype=torch.int32).cuda() if with_lens else None
    out, lse = lf.lf_window_attention_forward(q, k, v, w, sinks, seq_lens=sl)
    g = [torch.full_like(t, 7.0) if layout == "bhld" else torch.empty_like(t) for t in (q, k, v)]
    lf.lf_window_attention_backward(q, k, v, out, lse, do, w, sinks, seq_lens=sl, dq=g[0], dk=g[1], dv=g[2])
    torch.cuda.synchronize()
    got, seqs = [], []
    for b, n in enumerate(lens):
        o, d = (t[b].view(L, Hq, 64).transpose(0, 1) for t in (out, do))
        got.append(dict(out=o[:, :n], lse=lse[b, :, :n], dq=g[0][b, :, :n], dk=g[1][b, :, :n], dv=g[2][b, :, :n]))
        seqs.append((q[b, :, :n], k[b, :, :n], v[b, :, :n], d[:, :n]))
        assert bool((o[:, n:] == 0).all()) and bool((lse[b, :, n:] == float("-inf")).all())
        assert all(bool((t[b, :, n:] == 0).all()) for t in g), "padded rows are zero"
    _compare(got, seqs, w, sinks)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("layout", ["bhld", "blhd", "gap"])
def test_padded_batch(dtype, layout):
    _padded(dtype, [0, 1, 131, 300], 300, 4, 2, 70, 5, layout)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_batch_without_lengths(dtype):
    _padded(dtype, [257, 257], 257, 3, 3, 128, 4, "bhld", with_lens=False)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_one_token(dtype):
    _padded(dtype, [1], 1, 4, 2, 5, 1, "bhld", with_lens=False)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_repeats_bit_for_bit(dtype):
    a = _packed([700, 45], 4, 2, 100, 4, dtype, seed=21)
    b = _packed([700, 45], 4, 2, 100, 4, dtype, seed=21)
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_gradients_against_differences():
    """Directional differences of <out, dout> in fp32 (central, step h): the
    difference's error is the fp32 rounding of the sums over 2h, and h^2 times
    the third derivative (a few units for scores of order one)."""
    T, Hq, Hkv, w, s = 90, 2, 1, 17, 3
    q, k, v, do = (_rand((T, h, 64), "f32", 30 + i, 0.5) for i, h in enumerate((Hq, Hkv, Hkv, Hq)))
    do = do.reshape(T, Hq * 64)
    cu = torch.tensor([0, 60, T], dtype=torch.int32).cuda()
    out, lse = lf.lf_window_attention_forward(q, k, v, w, s, cu_seqlens=cu)
    g = lf.lf_window_attention_backward(q, k, v, out, lse, do, w, s, cu_seqlens=cu)
    h = 2.0 ** -5
    for i in range(3):
        x = [q, k, v]
        d = _rand(x[i].shape, "f32", 40 + i)
        d = d / d.norm()
        vals = []
        for sgn in (1, -1):
            y = list(x)
            y[i] = x[i] + sgn * h * d
            o, _ = lf.lf_window_attention_forward(*y, w, s, cu_seqlens=cu)
            vals.append(float((o.double() * do.double()).sum()))
        want = (vals[0] - vals[1]) / (2 * h)
        # out to 2^-20 of its size (about 0.2 a value), 90*128 products of |dout| about 0.5, over 2h; plus h^2
        bound = 2.0 ** -20 * 0.25 * 0.5 * (T * Hq * 64) ** 0.5 * 8 / h + 4 * h * h
        assert abs(float((g[i] * d).sum()) - want) <= bound


def test_other_stream_and_overlap():
    """Two calls of different inputs on two streams at once: no shared state."""
    ref = [_packed([500, 300], 4, 2, 64, 4, "f16", seed=50 + i) for i in range(2)]
    ins = []
    for i in range(2):
        x = _rand((803, 8, 64), "f16", 50 + i)
        do = _rand((803, 256), "f16", 51 + i)
        ins.append((x[:, :4].contiguous(), x[:, 4:6].contiguous(), x[:, 6:].contiguous(), do))
    cu = torch.tensor([0, 500, 800], dtype=torch.int32).cuda()
    st = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    res = [None, None]
    for _ in range(3):
        for i in range(2):
            q, k, v, do = ins[i]
            out, lse = lf.lf_window_attention_forward(q, k, v, 64, 4, cu_seqlens=cu, stream=st[i])
            res[i] = (out,) + lf.lf_window_attention_backward(q, k, v, out, lse, do, 64, 4, cu_seqlens=cu, stream=st[i])
    torch.cuda.synchronize()
    for i in range(2):
        for got, want in zip(res[i], (ref[i][0],) + ref[i][2:]):
            assert torch.equal(got[:800], want[:800])


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_captured_graph_follows_new_inputs(dtype):
    lens2 = ([200, 56], [1, 255])
    q, k, v = (_rand((256, h, 64), dtype, 60 + h) for h in (4, 2, 2))
    do = _rand((256, 256), dtype, 61)
    cu = torch.tensor([0, 200, 256], dtype=torch.int32).cuda()

    def step():
        out, lse = lf.lf_window_attention_forward(q, k, v, 33, 2, cu_seqlens=cu)
        return (out, lse) + lf.lf_window_attention_backward(q, k, v, out, lse, do, 33, 2, cu_seqlens=cu)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        res = step()
    for i, lens in enumerate(lens2):
        q.copy_(_rand(q.shape, dtype, 70 + i))
        cu.copy_(torch.tensor([0, lens[0], 256], dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        for got, want in zip(res, step()):
            assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("bad", [[0, 300, 200, 400], [-5, 100, 200, 300], [0, 100, 200, 500], [400, 0, 400, 0]])
def test_offsets_that_do_not_fit_are_recorded(dtype, bad):
    """Reported in the status word; nothing outside the tensors is written."""
    T, buf = 400, 512
    base = torch.full((buf, 2, 64), 7.0, dtype=DT[dtype], device="cuda")
    q, k, v = (_rand((T, h, 64), dtype, 80 + h) for h in (2, 1, 1))
    out = base[:T].view(T, 128)
    cu = torch.tensor(bad, dtype=torch.int32).cuda()
    lse = torch.zeros(1, 2, T, device="cuda")
    lf.lf_window_attention_forward(q, k, v, 20, 2, cu_seqlens=cu, out=out, lse=lse)
    assert lf.lf_device_status(reset=True) == 15
    assert bool((base[T:] == 7.0).all())
    do = _rand((T, 128), dtype, 83)
    lf.lf_window_attention_backward(q, k, v, out, lse, do, 20, 2, cu_seqlens=cu)
    assert lf.lf_device_status(reset=True) == 15


def test_lengths_that_do_not_fit_are_recorded():
    q, k, v = (_rand((2, h, 100, 64), "f16", 90 + h) for h in (2, 1, 1))
    for bad in ([101, 5], [-1, 5]):
        lf.lf_window_attention_forward(q, k, v, 20, 2, seq_lens=torch.tensor(bad, dtype=torch.int32).cuda())
        assert lf.lf_device_status(reset=True) == 15


def test_values_outside_the_window_do_not_matter():
    """Keys and values in whole tiles outside a row's set change nothing."""
    T = 700
    q, k, v = (_rand((T, h, 64), "f16", 95 + h) for h in (2, 2, 2))
    cu = torch.tensor([0, T], dtype=torch.int32).cuda()
    a, _ = lf.lf_window_attention_forward(q, k, v, 50, 4, cu_seqlens=cu)
    k[128:300], v[128:300] = 5.0, -3.0
    b, _ = lf.lf_window_attention_forward(q, k, v, 50, 4, cu_seqlens=cu)
    assert torch.equal(a[:128], b[:128]) and torch.equal(a[350:], b[350:]) and not torch.equal(a[128:350], b[128:350])


def test_no_tokens():
    z = torch.empty(0, 2, 64, dtype=torch.float16, device="cuda")
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    out, lse = lf.lf_window_attention_forward(z, z, z, 4, cu_seqlens=cu)
    assert out.shape == (0, 128) and lse.shape == (1, 2, 0)
    g = lf.lf_window_attention_backward(z, z, z, out, lse, out, 4, cu_seqlens=cu)
    assert all(t.shape == (0, 2, 64) for t in g)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_rows_more_than_2_31_elements_apart(dtype):
    """Keys and values (and their gradients) in rows 2^25 elements apart: the
    last of 100 starts past 2^31."""
    T, step = 100, 1 << 25
    big = [torch.empty(T * step, dtype=DT[dtype], device="cuda").as_strided((T, 1, 64), (step, 64, 1)) for _ in range(2)]
    q, k, v = (_rand((T, 1, 64), dtype, 110 + i) for i in range(3))
    do = _rand((T, 64), dtype, 113)
    cu = torch.tensor([0, T], dtype=torch.int32).cuda()
    want_o, lse = lf.lf_window_attention_forward(q, k, v, 30, 2, cu_seqlens=cu)
    want = lf.lf_window_attention_backward(q, k, v, want_o, lse, do, 30, 2, cu_seqlens=cu)
    big[0].copy_(k)
    out, lse = lf.lf_window_attention_forward(q, big[0], v, 30, 2, cu_seqlens=cu)
    got = lf.lf_window_attention_backward(q, big[0], v, out, lse, do, 30, 2, cu_seqlens=cu, dk=big[1])
    assert torch.equal(out, want_o)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_heads_share_storage_with_the_output_of_a_projection():
    """q, k and v as interleaved slices of one [B, L, H, 3, 64] buffer, and
    gradients into slices of another."""
    B, L, H = 2, 150, 3
    x = _rand((B, L, H, 3, 64), "bf16", 120)
    q, k, v = (x[:, :, :, i].transpose(1, 2) for i in range(3))
    out, lse = lf.lf_window_attention_forward(q, k, v, 40, 4)
    do = _rand((B, L, H * 64), "bf16", 121)
    dx = torch.full_like(x, 7.0)
    g = [dx[:, :, :, i].transpose(1, 2) for i in range(3)]
    lf.lf_window_attention_backward(q, k, v, out, lse, do, 40, 4, dq=g[0], dk=g[1], dv=g[2])
    rows = lambda t: t.view(B, L, H, 64).transpose(1, 2)  # noqa: E731
    _compare([dict(out=rows(out)[b], lse=lse[b], dq=g[0][b], dk=g[1][b], dv=g[2][b]) for b in range(B)],
             [(q[b], k[b], v[b], rows(do)[b]) for b in range(B)], 40, 4)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,w,sinks", [(6, 6, 30, 0), (9, 3, 20, 7), (12, 3, 1 << 30, 4), (6, 6, 0, 130)])
def test_more_short_items_than_the_gpu_holds(dtype, Hq, Hkv, w, sinks):
    """Hundreds of short sequences, empty and one-token ones among them: a
    CTA takes several items, of which many hold nothing."""
    lens = [(11 * i * i + 5 * i) % 37 * (i % 3) for i in range(300)]
    _packed(lens[:100] + [290] + lens[100:], Hq, Hkv, w, sinks, dtype, seed=w % 89 + sinks)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_more_padded_items_than_the_gpu_holds(dtype):
    lens = [(13 * i * i + 7 * i) % 271 * (i % 2) for i in range(80)]
    _padded(dtype, lens, 270, 8, 8, 50, 3, "blhd", seed=31)


def test_a_captured_pass_of_many_items_repeats_bit_for_bit():
    q, k, v, do = (_rand((2, 10, 6000, 64), "f16", 40 + s) for s in range(4))
    do = do.transpose(1, 2).reshape(2, 6000, 640).contiguous()
    out, lse = lf.lf_window_attention_forward(q, k, v, 64, 4)
    want = lf.lf_window_attention_backward(q, k, v, out, lse, do, 64, 4)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, l = lf.lf_window_attention_forward(q, k, v, 64, 4)
        got = lf.lf_window_attention_backward(q, k, v, o, l, do, 64, 4)
    for _ in range(3):
        for t in (o, l, *got):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, out) and torch.equal(l, lse)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("lens,w", [([1] * 50, 9), ([200, 1, 65], 0)])
def test_rows_that_see_one_key_have_no_gradient_of_scores(dtype, lens, w):
    """P = 1, so dS = P (dP - delta) = 0: what is left is dP (1 - P) twice
    over, with |1 - P| off by the fp32 scores (64 products of |q k| scale, 10
    at most here, each rounding 2^-24 of that) and the approximate
    exponential and logarithm (2^-22): below 2^-13."""
    Hq, Hkv, T = 4, 2, sum(lens)
    q, k, v = (_rand((T, H, 64), dtype, 50 + H + i) for i, H in enumerate((Hq, Hkv, Hkv)))
    do = _rand((T, Hq * 64), dtype, 60)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    out, lse = lf.lf_window_attention_forward(q, k, v, w, 0, cu_seqlens=cu)
    dq, dk, dv = lf.lf_window_attention_backward(q, k, v, out, lse, do, w, 0, cu_seqlens=cu)
    G = Hq // Hkv
    kk, vv = (t.double().repeat_interleave(G, 1) for t in (k, v))
    dp = (do.double().view(T, Hq, 64).abs() * vv.abs()).sum(-1, keepdim=True)
    assert float((q.double() * kk).abs().sum(-1).max()) * 0.125 < 10
    off = 2.0 ** -13 * 0.125 * dp
    assert bool((dq.double().abs() <= off * kk.abs() + 2.0 ** -24).all())
    assert bool((dk.double().abs() <= (off * q.double().abs()).view(T, Hkv, G, 64).sum(2) + 2.0 ** -24).all())
    assert torch.equal(dv, do.float().view(T, Hkv, G, 64).sum(2).to(dv.dtype))  # P rounds to 1


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("n", [1, 3, 400])
def test_only_empty_sequences(dtype, n):
    """Rows of no sequence, or padding throughout."""
    _packed([0] * n, 3, 3, 10, 2, dtype, tail=5)
    _padded(dtype, [0] * n, 4, 3, 3, 1, 1, "bhld")
