"""Refusals of the windowed attention, its paged form and the layer norm:
argument checks on the host, before anything touches a device."""
import ctypes

import pytest

from sparse_attention_banded_b200 import build, lf

FAKE = 0x10000


@pytest.fixture(scope="module")
def L():
    build.build()
    return lf.lib()


def _h(p=FAKE, sb=1 << 20, sh=1 << 14, st=64):
    return ctypes.byref(lf.Heads(p, sb, sh, st))


def vp(x):
    return ctypes.c_void_p(x)


def _fwd(L, q=None, k=None, v=None, cu=0, lens=0, n=2, Hq=4, Hkv=2, Ln=256, w=64, sinks=4, scale=0.125, dtype=1,
         out=FAKE, lse=FAKE):
    return L.lf_window_attention_forward(q or _h(), k or _h(), v or _h(), vp(cu), vp(lens), n, Hq, Hkv, Ln, w, sinks,
                                         scale, dtype, None, vp(out), vp(lse))


def _bwd(L, cu=0, lens=0, n=2, Hq=4, Hkv=2, Ln=256, w=64, sinks=4, scale=0.125, dtype=1, out=FAKE, lse=FAKE,
         dout=FAKE, ws=FAKE, ws_bytes=1 << 40, dq=None, dk=None, dv=None, q=None):
    return L.lf_window_attention_backward(q or _h(), _h(), _h(), vp(out), vp(lse), vp(dout), vp(cu), vp(lens), n, Hq,
                                          Hkv, Ln, w, sinks, scale, dtype, vp(ws), ws_bytes, None, dq or _h(),
                                          dk or _h(), dv or _h())


SHARED = [
    (dict(q=_h(0)), 1), (dict(out=0), 1), (dict(lse=0), 1),
    (dict(n=0), 2), (dict(Hq=0), 2), (dict(Hkv=0), 2), (dict(Ln=-1), 2), (dict(w=-1), 2), (dict(sinks=-1), 2),
    (dict(Hq=3, Hkv=2), 2), (dict(Hq=130, Hkv=2), 2),        # ragged groups, groups wider than 64
    (dict(cu=FAKE, lens=FAKE), 2),
    (dict(scale=0.0), 2), (dict(scale=-1.0), 2), (dict(scale=float("inf")), 2), (dict(scale=float("nan")), 2),
    (dict(q=_h(st=0)), 2), (dict(q=_h(sh=-64)), 2),           # broadcast and reversed views
    (dict(dtype=7), 7),
    (dict(q=_h(FAKE + 8)), 8), (dict(q=_h(st=68)), 8), (dict(lse=FAKE + 4), 8), (dict(out=FAKE + 2), 8),
    (dict(cu=FAKE + 2), 8),
    (dict(n=1 << 16, Hq=64, Hkv=64, Ln=512), 13), (dict(n=1 << 23, Hq=1, Hkv=1, Ln=1), 13),
    (dict(q=_h(st=1 << 40)), 13),
]


@pytest.mark.parametrize("kw,status", SHARED + [(dict(k=_h(0)), 1), (dict(v=_h(st=4)), 8)])
def test_window_forward_refusals(L, kw, status):
    assert _fwd(L, **kw) == status


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(dout=0), 1), (dict(dq=_h(0)), 1), (dict(dk=_h(st=0)), 2), (dict(dv=_h(FAKE + 4)), 8), (dict(dout=FAKE + 8), 8),
    (dict(ws=0), 12), (dict(ws=FAKE + 16), 12), (dict(ws_bytes=100), 12)])
def test_window_backward_refusals(L, kw, status):
    assert _bwd(L, **kw) == status


def test_null_views_and_empty_calls(L):
    assert L.lf_window_attention_forward(None, _h(), _h(), None, None, 1, 1, 1, 64, 1, 0, 0.125, 1, None, vp(FAKE),
                                         vp(FAKE)) == 1
    assert _fwd(L, q=_h(0), k=_h(0), v=_h(0), Ln=0, out=0, lse=0) == 0  # no tokens: nothing to do
    assert _bwd(L, Ln=0, ws=0, ws_bytes=0) == 0


def test_backward_workspace_bytes(L):
    f = lf.lf_window_attention_backward_workspace_bytes
    assert f(False, 2, 4, 2, 256, 64, 0) == 2 * 4 * 256 * 4
    with_sinks = f(False, 2, 4, 2, 256, 64, 4)
    assert with_sinks > 2 * 4 * 256 * 4
    assert f(True, 2, 4, 2, 256, 64, 4) < with_sinks + 1
    assert f(False, 2, 4, 2, 256, 255, 4) == 2 * 4 * 256 * 4  # every window reaches the start
    assert f(False, 2, 3, 2, 256, 64, 4) == 0 and f(False, 2, 4, 2, 0, 64, 4) == 0


def _paged(L, q=None, kc=None, vc=None, table=FAKE, cu=FAKE, kv=FAKE, n=2, Hq=4, Hkv=2, T=8, max_q=4, mp=16, np_=64,
           ps=16, w=100, sinks=0, scale=0.125, dtype=1, ws=FAKE, ws_bytes=1 << 40, out=FAKE):
    return L.lf_paged_attention_forward(q or _h(), kc or _h(), vc or _h(), vp(table), vp(cu), vp(kv), n, Hq, Hkv, T,
                                        max_q, mp, np_, ps, w, sinks, scale, dtype, vp(ws), ws_bytes, None, vp(out))


@pytest.mark.parametrize("kw,status", [
    (dict(q=_h(0)), 1), (dict(kc=_h(0)), 1), (dict(table=0), 1), (dict(cu=0), 1), (dict(kv=0), 1), (dict(out=0), 1),
    (dict(n=0), 2), (dict(T=-1), 2), (dict(max_q=0), 2), (dict(mp=0), 2), (dict(np_=0), 2), (dict(w=-1), 2),
    (dict(sinks=-1), 2), (dict(ps=24), 2), (dict(ps=4), 2), (dict(ps=8192), 2), (dict(Hq=5), 2), (dict(Hq=256), 2),
    (dict(scale=0.0), 2), (dict(q=_h(st=0)), 2), (dict(kc=_h(sb=-64)), 2),
    (dict(dtype=0), 7), (dict(dtype=9), 7),
    (dict(kc=_h(st=68)), 8), (dict(out=FAKE + 8), 8), (dict(table=FAKE + 2), 8),
    (dict(T=1 << 30), 13), (dict(mp=(1 << 20) + 1), 13), (dict(n=1 << 21), 13),
])
def test_paged_forward_refusals(L, kw, status):
    assert _paged(L, **kw) == status


def _append(L, k=None, v=None, kc=None, vc=None, table=FAKE, cu=FAKE, kv=FAKE, n=2, Hkv=2, T=8, mp=16, np_=64, ps=16,
            dtype=1):
    return L.lf_paged_cache_append(k or _h(), v or _h(), kc or _h(), vc or _h(), vp(table), vp(cu), vp(kv), n, Hkv, T,
                                   mp, np_, ps, dtype, None)


@pytest.mark.parametrize("kw,status", [
    (dict(k=_h(0)), 1), (dict(vc=_h(0)), 1), (dict(table=0), 1), (dict(n=0), 2), (dict(Hkv=0), 2), (dict(ps=12), 2),
    (dict(kc=_h(sb=0)), 2), (dict(dtype=0), 7), (dict(v=_h(FAKE + 2)), 8), (dict(kc=_h(sh=4)), 8),
    (dict(mp=1 << 28), 13)])
def test_append_refusals(L, kw, status):
    assert _append(L, **kw) == status
    assert _append(L, T=0) == 0


def _norm(L, x=FAKE, xs=1024, g=FAKE, b=FAKE, rows=8, N=1024, eps=1e-5, dtype=1, y=FAKE, mean=FAKE, rstd=FAKE):
    return L.lf_layer_norm_forward(vp(x), xs, vp(g), vp(b), rows, N, eps, dtype, None, vp(y), vp(mean), vp(rstd))


def _norm_b(L, dy=FAKE, dys=1024, x=FAKE, xs=1024, g=FAKE, mean=FAKE, rstd=FAKE, rows=8, N=1024, dtype=1, ws=FAKE,
            ws_bytes=1 << 30, dx=FAKE, dg=FAKE, db=FAKE):
    return L.lf_layer_norm_backward(vp(dy), dys, vp(x), xs, vp(g), vp(mean), vp(rstd), rows, N, dtype, vp(ws),
                                    ws_bytes, None, vp(dx), vp(dg), vp(db))


@pytest.mark.parametrize("kw,status", [
    (dict(x=0), 1), (dict(y=0), 1), (dict(rows=-1), 2), (dict(N=0), 2), (dict(xs=1000), 2), (dict(eps=-1.0), 2),
    (dict(eps=float("nan")), 2), (dict(dtype=3), 7), (dict(x=FAKE + 2), 8), (dict(g=FAKE + 4), 8),
    (dict(mean=FAKE + 2), 8), (dict(N=16385, xs=16385), 13), (dict(rows=0, x=0, y=0), 0)])
def test_norm_forward_refusals(L, kw, status):
    assert _norm(L, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dy=0), 1), (dict(mean=0), 1), (dict(rstd=0), 1), (dict(dx=0), 1), (dict(rows=-1), 2), (dict(dys=1023), 2),
    (dict(dtype=-1), 7), (dict(dx=FAKE + 8), 8), (dict(dg=FAKE + 4), 8), (dict(N=20000, xs=20000, dys=20000), 13),
    (dict(ws=0), 12), (dict(ws=FAKE + 16), 12), (dict(ws_bytes=64), 12), (dict(rows=0, dg=0, db=0), 0)])
def test_norm_backward_refusals(L, kw, status):
    assert _norm_b(L, **kw) == status


def test_new_status_strings(L):
    assert lf.status_string(15).startswith("LF_ERR_BAD_LENGTHS") and lf.status_string(16).startswith("LF_ERR_BAD_PAGE")
    assert lf.status_string(17) == "unknown lf_status"


def test_binding_refuses_mismatched_tensors():
    """Shapes, types and devices are checked before the library is called
    (CPU tensors never reach it)."""
    import torch
    q = torch.zeros(1, 4, 8, 64, dtype=torch.float16)
    k = torch.zeros(1, 2, 8, 64, dtype=torch.float16)
    for bad in (dict(k=k.float()), dict(k=k[:, :, :4]), dict(cu_seqlens=torch.tensor([0, 8], dtype=torch.int32)),
                dict(seq_lens=torch.tensor([8])), dict(seq_lens=torch.tensor([8, 8], dtype=torch.int32)), dict()):
        a = dict(q=q, k=k, v=k, w=4)
        a.update(bad)
        with pytest.raises(ValueError):
            lf.lf_window_attention_forward(**a)
    with pytest.raises(ValueError):
        lf.lf_layer_norm_forward(torch.zeros(4, 64))
    for kw in (dict(w=1 << 31), dict(sinks=1 << 31)):
        with pytest.raises(ValueError, match="int32"):
            lf.lf_window_attention_forward(q, k, k, **{"w": 4, **kw})
