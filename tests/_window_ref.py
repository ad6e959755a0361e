"""float64 definition of the windowed causal attention with sinks, its
gradients, and element-wise error bounds derived from the roundings a
16-bit or fp32 kernel makes (u = half a step of the storage type)."""
import torch


def mask(n, m, first, w, sinks):
    """[n, m]: does the query at position first + r see key j?"""
    i = first + torch.arange(n)[:, None]
    j = torch.arange(m)[None, :]
    return (j <= i) & ((i - j <= w) | (j < sinks)) & (i >= 0)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def subnormal_half_step(dtype):
    """Below its smallest normal number a type's steps stop shrinking: they
    stay smallest_normal * eps, so a rounding there is off by up to half of
    that whatever the value (fp16: 2^-14 * 2^-10 / 2 = 2^-25)."""
    f = torch.finfo(dtype)
    return 0.5 * f.smallest_normal * f.eps


def reference(q, k, v, first, w, sinks, scale=0.125, dout=None, visible=None):
    """q [Hq, n, 64] at positions first.., k, v [Hkv, m, 64], any dtype; all
    returned float64 on q's device: a dict of out, lse, and with dout dq, dk,
    dv, each with its bound under "b_" + name.

    Bounds.  With u the half step of the storage type t (0 for the operands
    of fp32), e the relative error of a probability: the fp32 sum of a score's
    64 products (64 * 2^-24 * S, S the row's largest scale * |q|.|k|, twice:
    score and log-sum-exp), the n-term sums, the exponential (7.5e-5, the
    16-bit kernels' cubic; 2^-21 fp32):
      out   sum_j p_j v_j with p rounded, then out rounded:
            (2u + 2e) sum_j p_j |v_j|
      dv    (2u + 2e) sum_i p_ij |dout_i|
      dS    p (dP - delta): dP and delta from fp32 sums and the rounded out,
            then dS rounded:  E = p (|dout|.b_out + 2^-18 (|dout|.|v| + |dout|.|out|)) + (u + 2e) |dS|
      dq    scale sum_j (E + 2^-20 |dS|) |k_j|  + u |dq|;   dk likewise.
    Each rounding to the type adds its subnormal half step z: z per output,
    z |v_j|, z |dout_i|, z scale |k_j|, z scale |q_i| per visible pair.
    """
    dt = q.dtype
    u = half_step(dt)
    uo = 0.0 if dt == torch.float32 else u
    q, k, v = q.double(), k.double(), v.double()
    Hq, n, _ = q.shape
    Hkv, m, _ = k.shape
    G = Hq // Hkv
    ok = (mask(n, m, first, w, sinks) if visible is None else visible).to(q.device)
    k2, v2 = k.repeat_interleave(G, 0), v.repeat_interleave(G, 0)
    s = q @ k2.mT * scale
    S = (q.abs() @ k2.abs().mT * scale).where(ok, 0.0).amax() if m and n else torch.tensor(0.0)
    e = 2.0 ** -24 * (128 * float(S) + m + 64) + (2.0 ** -21 if dt == torch.float32 else 7.5e-5)
    s = s.masked_fill(~ok, float("-inf"))
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse.masked_fill(lse.isinf(), 0.0)[..., None])
    r = {"out": p @ v2, "lse": lse, "b_lse": torch.full_like(lse, 2 * e) + 2.0 ** -22 * lse.abs().nan_to_num(posinf=0.0)}
    z = subnormal_half_step(dt)
    zo = 0.0 if dt == torch.float32 else z
    okf = ok.double()
    r["b_out"] = (u + uo + 2 * e) * (p @ v2.abs()) + z + zo * (okf @ v2.abs())
    if dout is None:
        return r
    do = dout.double()
    dp = do @ v2.mT
    delta = (do * r["out"]).sum(-1, keepdim=True)
    ds = p * (dp - delta)
    E = p * ((do.abs() * r["b_out"]).sum(-1, keepdim=True)
             + 2.0 ** -18 * (do.abs() @ v2.abs().mT + (do.abs() * r["out"].abs()).sum(-1, keepdim=True)))
    E = E + (uo + 2 * e + 2.0 ** -20) * ds.abs()

    def group(t):
        return t.view(Hkv, G, m, 64).sum(1)

    r["dq"] = scale * ds @ k2
    r["dk"] = group(scale * ds.mT @ q)
    r["dv"] = group(p.mT @ do)
    E = E + zo * okf
    r["b_dq"] = scale * E @ k2.abs() + u * r["dq"].abs() + z
    r["b_dk"] = group(scale * E.mT @ q.abs()) + u * r["dk"].abs() + z
    r["b_dv"] = group(((uo + 2 * e) * p + zo * okf).mT @ do.abs()) + u * r["dv"].abs() + z
    return r


def check(name, got, ref, bound):
    got = got.double()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert torch.isfinite(got).all(), "%s: not finite" % name
    over = (got - ref).abs() - bound
    assert float(over.max() if over.numel() else 0.0) <= 0.0, "%s: off by up to %g over its bound (largest error %g)" % (
        name, float(over.max()), float((got - ref).abs().max()))
