"""Layer norm forward and backward against float64, bounds derived from the
roundings: fp32 statistics and one rounding of each output."""
import pytest
import torch

from sparse_attention_banded_b200 import build, lf
from tests._window_ref import check, half_step

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    lf.lib()
    yield


def _ref(x, gamma, beta, dy, eps, N):
    """Values and bounds.  With r = 2^-24 * (N / 32 + 64) the relative error
    of a row's fp32 sums (32 terms a thread, then a tree; N / 32 covers any
    order used), e_x = r * (|x| + max |x|) * rstd the error of xh (x - mean):
    y rounds once more."""
    dt = x.dtype
    u = half_step(dt)
    x, dy = x.double(), dy.double()
    g = torch.ones(N, dtype=torch.double, device=x.device) if gamma is None else gamma.double()
    b = torch.zeros(N, dtype=torch.double, device=x.device) if beta is None else beta.double()
    r = 2.0 ** -24 * (N / 32 + 64)
    mean = x.mean(1, keepdim=True)
    rstd = 1 / (x.var(1, unbiased=False, keepdim=True) + eps).sqrt()
    xh = (x - mean) * rstd
    big = x.abs().amax(1, keepdim=True)
    e_mean = r * x.abs().mean(1, keepdim=True) + 2.0 ** -24 * mean.abs()
    e_xh = rstd * (e_mean + 2.0 ** -23 * big) + xh.abs() * (r + rstd * e_mean)
    y = xh * g + b
    gg = dy * g
    m1, m2 = gg.mean(1, keepdim=True), (gg * xh).mean(1, keepdim=True)
    dx = rstd * (gg - m1 - xh * m2)
    e_m1 = r * gg.abs().mean(1, keepdim=True)
    e_m2 = (gg.abs() * e_xh).mean(1, keepdim=True) + r * (gg * xh).abs().mean(1, keepdim=True)
    e_dx = rstd * (e_m1 + e_xh * m2.abs() + xh.abs() * e_m2 + 2.0 ** -22 * (gg.abs() + m1.abs() + (xh * m2).abs()))
    R = x.shape[0]
    rr = 2.0 ** -24 * (R / 8 + 64)
    return dict(y=(y, u * y.abs() + g.abs() * e_xh + 2.0 ** -22 * (xh * g).abs() + 2.0 ** -24 * b.abs()),
                mean=(mean[:, 0], e_mean[:, 0]), rstd=(rstd[:, 0], (rstd * (r + rstd * e_mean + rstd ** 2 * e_mean ** 2))[:, 0]),
                dx=(dx, u * dx.abs() + e_dx + r * dx.abs()),
                dgamma=((dy * xh).sum(0), (dy.abs() * e_xh).sum(0) + rr * (dy * xh).abs().sum(0)),
                dbeta=(dy.sum(0), rr * dy.abs().sum(0)))


def _run(rows, N, dtype, affine=True, eps=1e-5, pad=0, offset=0.0, seed=0):
    g = torch.Generator().manual_seed(seed + rows * 131 + N)
    dt = DT[dtype]

    def rand(*s):
        return torch.randn(*s, generator=g)

    def rows_of(t):
        if not pad:
            return t.to(dt).cuda()
        big = torch.full((rows, N + pad), float("nan"), dtype=dt, device="cuda")
        big[:, :N] = t.to(dt)
        return big[:, :N]

    x, dy = rows_of(rand(rows, N) + offset), rows_of(rand(rows, N))
    gamma, beta = ((1 + 0.3 * rand(N)).cuda(), (0.3 * rand(N)).cuda()) if affine else (None, None)
    y, mean, rstd = lf.lf_layer_norm_forward(x, gamma, beta, eps)
    need = lf.lf_layer_norm_backward_workspace_bytes(rows, N)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    dx, dgamma, dbeta = lf.lf_layer_norm_backward(dy, x, gamma, mean, rstd, workspace=ws)
    torch.cuda.synchronize()
    for name, (want, bound) in _ref(x, gamma, beta, dy, eps, N).items():
        check(name, dict(y=y, mean=mean, rstd=rstd, dx=dx, dgamma=dgamma, dbeta=dbeta)[name], want, bound)
    return x, dy, gamma, beta, y, mean, rstd, dx, dgamma, dbeta


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,N", [(1, 1), (3, 2), (5, 31), (2, 33), (7, 64), (9, 257), (300, 768), (17, 1024),
                                    (33, 1025), (40, 1537), (3, 4096), (2, 4097), (5, 8192), (2, 16383), (3, 16384),
                                    (1000, 256), (4000, 65)])
def test_sizes(dtype, rows, N):
    _run(rows, N, dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_row_strides(dtype):
    _run(50, 512, dtype, pad=8)
    _run(50, 512, dtype, pad=3)
    _run(21, 515, dtype, pad=5)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_without_parameters_and_far_mean(dtype):
    _run(40, 640, dtype, affine=False)
    _run(40, 640, dtype, offset=30.0)  # the variance is centred, not a difference of squares


def test_constant_rows():
    """No variance: xh = 0, rstd = 1 / sqrt(eps); nothing overflows."""
    x = torch.full((4, 96), 3.0, dtype=torch.float16, device="cuda")
    y, mean, rstd = lf.lf_layer_norm_forward(x, None, None, 1e-5)
    assert bool((y == 0).all()) and bool((mean == 3).all())
    assert float((rstd - 1e5 ** 0.5).abs().max()) < 1e-3


def test_in_higher_dimensions_and_parts():
    x = torch.randn(3, 5, 128, device="cuda")
    y, mean, rstd = lf.lf_layer_norm_forward(x)
    y2, _, _ = lf.lf_layer_norm_forward(x.view(15, 128))
    assert y.shape == x.shape and torch.equal(y.view(15, 128), y2)
    dy = torch.randn_like(x)
    dx, dg, db = lf.lf_layer_norm_backward(dy, x, None, mean, rstd)
    only, none1, none2 = lf.lf_layer_norm_backward(dy, x, None, mean, rstd, param_grads=False)
    assert torch.equal(only, dx) and none1 is None and none2 is None
    buf = torch.full((128,), 9.0, device="cuda")
    _, _, got = lf.lf_layer_norm_backward(dy, x, None, mean, rstd, dbeta=buf, param_grads=False)
    assert got is buf and torch.equal(buf, db)


def test_no_rows():
    x = torch.empty(0, 64, device="cuda")
    y, mean, rstd = lf.lf_layer_norm_forward(x)
    dx, dg, db = lf.lf_layer_norm_backward(x, x, None, mean, rstd)
    assert y.shape == (0, 64) and dx.shape == (0, 64) and bool((dg == 0).all()) and bool((db == 0).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_graph_and_repeat(dtype):
    x, dy, gamma, beta, *first = _run(700, 384, dtype, seed=4)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, mean, rstd = lf.lf_layer_norm_forward(x, gamma, beta)
        res = (y, mean, rstd) + lf.lf_layer_norm_backward(dy, x, gamma, mean, rstd)
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(res, first):
        assert torch.equal(a, b)


def test_nan_stays_in_its_row():
    x = torch.randn(20, 200, device="cuda")
    x[7, 3] = float("nan")
    y, _, _ = lf.lf_layer_norm_forward(x)
    assert bool(torch.isnan(y[7]).all()) and not bool(torch.isnan(y[torch.arange(20) != 7]).any())
