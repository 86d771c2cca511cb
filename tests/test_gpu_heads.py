"""Norm and rotation of heads and their gradient against plain forms in 64 bits, and the gradient against differences.

Tolerances.  The kernel's inputs are exact.  A mean of d squares in fp32 is off by at most d 2^-24 relative, the reciprocal
root by half of that and 2^-22, two products by 2^-24 each: in all a = d 2^-25 + 2^-21 relative.  A turn's sine and cosine are
off by 2^-26 turns and two units in the last place, b = 4e-7 at most, and the two products and the sum by 2^-23 of the
pair's sizes.  So with P the sum of the pair's magnitudes (or the channel's own, unrotated) y is off by (a + b + 2^-22) P, and
half a step of the type.  The gradient's g = R^T dy is off by (b + 2^-22) P(dy); dx = r (w g - xn m), with m the mean of d terms
w g xn, by r (|w| (b + 2^-22) P + a |w g| + |xn| (mean |w xn| ((b + 2^-22) P + a |g|) + d 2^-24 mean |w g xn|) + a |xn m|),
twice that for the products' own roundings.  dw sums T Hq terms g xn, each off by (b + 2^-22) P |xn| + a |g xn|, in fp32
with no more than T Hq additions that round: T Hq 2^-24 of the terms' magnitudes at most.
"""
import math

import pytest
import torch

import long_context_sparse_dsa_gb300 as dsa
from test_gpu_decode import DEV, HALF, _built, _dt, _freq  # noqa: F401

pytestmark = pytest.mark.gpu
EPS = 1e-6
B = 4e-7


def _dims(T, Hq, d, dtype):
    return dsa.make_dims(max(4, (T + 3) // 4 * 4), Hq, d, 8, 64, 8, dtype=dtype)


def _pair_sum(x, rot, inter):
    """Of every channel the magnitudes of its pair, added; its own where it has none."""
    y, n = x.abs().clone(), rot
    if n:
        a, b = (x[..., 0:n:2].abs(), x[..., 1:n:2].abs()) if inter else (x[..., :n // 2].abs(), x[..., n // 2:n].abs())
        if inter:
            y[..., 0:n:2] = y[..., 1:n:2] = a + b
        else:
            y[..., :n // 2] = y[..., n // 2:n] = a + b
    return y


def _turned(x, pos, freq, inter, back=False):
    x = x.clone()
    if freq is None:
        return x
    ang = pos.double().view(-1, *[1] * (x.dim() - 1)) * freq.double()
    c, s = ang.cos(), (-ang if back else ang).sin()
    n = 2 * freq.numel()
    i = (slice(0, n, 2), slice(1, n, 2)) if inter else (slice(0, n // 2), slice(n // 2, n))
    a, b = x[..., i[0]].clone(), x[..., i[1]].clone()
    x[..., i[0]], x[..., i[1]] = a * c - b * s, a * s + b * c
    return x


def _inputs(T, Hq, d, dtype, seed, packed=False):
    g = torch.Generator().manual_seed(seed)
    if packed:
        x = torch.randn(T, Hq + 2, d, generator=g).to(_dt(dtype))
        q, k = x[:, :Hq], x[:, Hq]
    else:
        q, k = torch.randn(T, Hq, d, generator=g).to(_dt(dtype)), torch.randn(T, d, generator=g).to(_dt(dtype))
    qw, kw = 1 + 0.3 * torch.randn(d, generator=g), 1 + 0.3 * torch.randn(d, generator=g)
    return g, q, k, qw, kw


def _norm(x, w):
    x = x.double()
    r = (x.pow(2).mean(-1, keepdim=True) + EPS).rsqrt()
    return x * r, r, (x * r if w is None else x * r * w.double())


def _check_fwd(got, x, w, pos, freq, inter, dtype):
    d, rot = x.shape[-1], 0 if freq is None else 2 * freq.numel()
    _, _, n = _norm(x, w)
    want = _turned(n, pos, freq, inter)
    tol = (d * 2.0 ** -25 + 2.0 ** -21 + B + 2.0 ** -22) * _pair_sum(n, rot, inter) + HALF[dtype] * want.abs()
    err = (got.double().cpu() - want).abs()
    assert torch.all(err <= tol), (err / tol).max()


def _check_bwd(dx, dw, x, w, dy, pos, freq, inter):
    d, rot = x.shape[-1], 0 if freq is None else 2 * freq.numel()
    a, t = d * 2.0 ** -25 + 2.0 ** -21, B + 2.0 ** -22
    xn, r, _ = _norm(x, None)
    wd = torch.ones(d, dtype=torch.float64) if w is None else w.double()
    g, P = _turned(dy.double(), pos, freq, inter, back=True), _pair_sum(dy.double(), rot, inter)
    m = (wd * g * xn).mean(-1, keepdim=True)
    want = r * (wd * g - xn * m)
    slack = (wd.abs() * t * P + a * (wd * g).abs() + a * (xn * m).abs() + xn.abs() * (
        (wd * xn).abs() * (t * P + a * g.abs()) + d * 2.0 ** -24 * (wd * g * xn).abs()).mean(-1, keepdim=True))
    err = (dx.double().cpu() - want).abs()
    assert torch.all(err <= 2 * r * slack + 2.0 ** -24 * want.abs()), (err / (2 * r * slack)).max()
    if dw is not None:
        terms = (g * xn).flatten(0, -2)
        tol = 2 * (t * P * xn.abs() + a * (g * xn).abs()).flatten(0, -2).sum(0) + len(terms) * 2.0 ** -24 * terms.abs().sum(0)
        err = (dw.double().cpu() - terms.sum(0)).abs()
        assert torch.all(err <= tol + 1e-12), (err / tol).max()


CASES = [("bf16", 16, 128, 128, False, 300), ("bf16", 32, 64, 64, True, 77), ("bf16", 1, 128, 16, False, 1), ("bf16", 5, 64, 0, False, 9),
         ("bf16", 17, 128, 96, True, 33), ("fp32", 8, 64, 16, True, 130), ("fp32", 32, 128, 128, False, 19), ("fp32", 3, 128, 48, False, 2),
         ("bf16", 16, 128, 64, False, 20011)]


@pytest.mark.parametrize("dtype,Hq,d,rot,inter,T", CASES)
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("given", [False, True])   # positions
def test_forward_and_gradient(dtype, Hq, d, rot, inter, T, packed, given):
    g, q, k, qw, kw = _inputs(T, Hq, d, dtype, T + Hq, packed)
    dims = _dims(T, Hq, d, dtype)
    freq = _freq(rot) if rot else None
    rotation = dsa.make_rotation(freq, interleaved=inter) if rot else None
    pos = torch.randint(-1 << 20, 1 << 24, (T,), generator=g, dtype=torch.int32) if given else torch.arange(T)
    qd, kd = (torch.cat([q, k[:, None], k[:, None]], 1).to(DEV)[:, :Hq], torch.cat([q, k[:, None], k[:, None]], 1).to(DEV)[:, Hq]) \
        if packed else (q.to(DEV), k.to(DEV))
    qo, ko = torch.full((T, Hq, d), 7.0, dtype=_dt(dtype), device=DEV), torch.full((T, d), 7.0, dtype=_dt(dtype), device=DEV)
    kw_ = dict(q_weight=qw.to(DEV), k_weight=kw.to(DEV), rotation=rotation, positions=pos.to(DEV) if given else None)
    dsa.qk_norm_rotate(dims, qd, kd, qo, ko, EPS, **kw_)
    _check_fwd(qo, q, qw, pos, freq, inter, dtype)
    _check_fwd(ko, k, kw, pos, freq, inter, dtype)
    dyq, dyk = torch.randn(T, Hq, d, generator=g), torch.randn(T, d, generator=g)
    dq, dk = torch.full((T, Hq, d), 7.0, device=DEV), torch.full((T, d), 7.0, device=DEV)
    dqw, dkw = torch.full((d,), 7.0, device=DEV), torch.full((d,), 7.0, device=DEV)
    ws = torch.full((dsa.qk_norm_bwd_workspace_bytes(dims, T),), 0xFF, dtype=torch.uint8, device=DEV)
    dsa.qk_norm_rotate_bwd(dims, qd, kd, dyq.to(DEV), dyk.to(DEV), dq, dk, EPS, ws, dq_weight=dqw, dk_weight=dkw, **kw_)
    dsa.check_device_error()
    _check_bwd(dq, dqw, q, qw, dyq, pos, freq, inter)
    _check_bwd(dk, dkw, k, kw, dyk, pos, freq, inter)


@pytest.mark.parametrize("which", ["q", "k"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_one_of_the_two_without_weights(which, dtype):
    T, Hq, d = 50, 6, 128
    g, q, k, _, _ = _inputs(T, Hq, d, dtype, 5)
    dims, rotation = _dims(T, Hq, d, dtype), dsa.make_rotation(_freq(64))
    x = q if which == "q" else k
    xd, y, dy = x.to(DEV), torch.zeros_like(x).to(DEV), torch.randn(x.shape, generator=g)
    dx, dw = torch.zeros(x.shape, device=DEV), torch.zeros(d, device=DEV)
    pick = lambda a: (a, None) if which == "q" else (None, a)  # noqa: E731
    dsa.qk_norm_rotate(dims, *pick(xd), *pick(y), EPS, rotation=rotation)
    _check_fwd(y, x, None, torch.arange(T), _freq(64), False, dtype)
    ws = torch.full((dsa.qk_norm_bwd_workspace_bytes(dims, T),), 0xFF, dtype=torch.uint8, device=DEV)
    dsa.qk_norm_rotate_bwd(dims, *pick(xd), *pick(dy.to(DEV)), *pick(dx), EPS, ws, rotation=rotation,
                           **{f"d{which}_weight": dw})
    _check_bwd(dx, dw, x, None, dy, torch.arange(T), _freq(64), False)
    # without the weight's gradient
    dx2 = torch.zeros_like(dx)
    dsa.qk_norm_rotate_bwd(dims, *pick(xd), *pick(dy.to(DEV)), *pick(dx2), EPS, ws, rotation=rotation)
    assert torch.equal(dx, dx2)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_in_place(dtype):
    T, Hq, d = 301, 16, 128
    g, q, k, qw, kw = _inputs(T, Hq, d, dtype, 6)
    dims, rotation = _dims(T, Hq, d, dtype), dsa.make_rotation(_freq(128))
    kw_ = dict(q_weight=qw.to(DEV), k_weight=kw.to(DEV), rotation=rotation)
    qd, kd = q.to(DEV), k.to(DEV)
    qo, ko = torch.zeros_like(qd), torch.zeros_like(kd)
    dsa.qk_norm_rotate(dims, qd, kd, qo, ko, EPS, **kw_)
    dy = torch.randn(T, Hq, d, generator=g).to(DEV), torch.randn(T, d, generator=g).to(DEV)
    dx = torch.zeros_like(dy[0]), torch.zeros_like(dy[1])
    ws = torch.zeros(dsa.qk_norm_bwd_workspace_bytes(dims, T), dtype=torch.uint8, device=DEV)
    dsa.qk_norm_rotate_bwd(dims, qd, kd, *dy, *dx, EPS, ws, **kw_)
    dsa.qk_norm_rotate_bwd(dims, qd, kd, *dy, *dy, EPS, ws, **kw_)
    assert torch.equal(dy[0], dx[0]) and torch.equal(dy[1], dx[1])
    dsa.qk_norm_rotate(dims, qd, kd, qd, kd, EPS, **kw_)
    assert torch.equal(qd, qo) and torch.equal(kd, ko)


def test_zero_rows_infinities_and_no_tokens():
    """A head of zeros gives zeros and a finite gradient; an infinite value reaches its own head only."""
    T, Hq, d = 3, 4, 64
    g, q, k, qw, kw = _inputs(T, Hq, d, "bf16", 7)
    q[1, 2] = 0
    q[0, 1, 5] = math.inf
    dims = _dims(T, Hq, d, "bf16")
    qo, ko = torch.zeros(T, Hq, d, dtype=torch.bfloat16, device=DEV), torch.zeros(T, d, dtype=torch.bfloat16, device=DEV)
    kw_ = dict(q_weight=qw.to(DEV), k_weight=kw.to(DEV), rotation=dsa.make_rotation(_freq(16)))
    dsa.qk_norm_rotate(dims, q.to(DEV), k.to(DEV), qo, ko, EPS, **kw_)
    assert torch.all(qo[1, 2] == 0)
    bad = torch.zeros(T, Hq, dtype=torch.bool)
    bad[0, 1] = True
    assert torch.equal(torch.isfinite(qo.float()).all(-1).cpu(), ~bad)
    ws = torch.zeros(dsa.qk_norm_bwd_workspace_bytes(dims, T), dtype=torch.uint8, device=DEV)
    dy, dx = torch.ones(T, Hq, d, device=DEV), torch.zeros(T, Hq, d, device=DEV)
    q[0, 1, 5] = 0
    dsa.qk_norm_rotate_bwd(dims, q.to(DEV), None, dy, None, dx, None, EPS, ws, q_weight=kw_["q_weight"])
    assert torch.all(torch.isfinite(dx))
    _check_bwd(dx, None, q, qw, dy.cpu(), torch.arange(T), None, False)
    # no tokens: the weights' gradients are 0
    e = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device=DEV)  # noqa: E731
    f32 = torch.float32
    dqw, dkw = torch.full((d,), 7.0, device=DEV), torch.full((d,), 7.0, device=DEV)
    dsa.qk_norm_rotate(dims, e(0, Hq, d), e(0, d), e(0, Hq, d), e(0, d), EPS, **kw_)
    dsa.qk_norm_rotate_bwd(dims, e(0, Hq, d), e(0, d), e(0, Hq, d, dt=f32), e(0, d, dt=f32), e(0, Hq, d, dt=f32),
                           e(0, d, dt=f32), EPS, ws, dq_weight=dqw, dk_weight=dkw, **kw_)
    assert torch.all(dqw == 0) and torch.all(dkw == 0)


def test_gradient_against_differences():
    """Along a direction v, (f(x + h v) - f(x - h v)) / 2h of f = <dy, y> in 64 bits, from the fp32 kernel's own outputs at
    x + h v and x - h v: those are off by 1e-5 of P each, so h = 2^-4 leaves 2e-4 and the third derivative h^2."""
    T, Hq, d = 12, 8, 64
    g, q, k, qw, kw = _inputs(T, Hq, d, "fp32", 8)
    q = q * 3
    dims, rotation = _dims(T, Hq, d, "fp32"), dsa.make_rotation(_freq(64))
    dy = torch.randn(T, Hq, d, generator=g)
    v, vw = torch.randn(T, Hq, d, generator=g), torch.randn(d, generator=g)

    def f(x, w):
        y = torch.zeros(T, Hq, d, device=DEV)
        dsa.qk_norm_rotate(dims, x.to(DEV), None, y, None, EPS, q_weight=w.to(DEV), rotation=rotation)
        return (dy.double() * y.double().cpu()).sum()

    dx, dw = torch.zeros(T, Hq, d, device=DEV), torch.zeros(d, device=DEV)
    ws = torch.zeros(dsa.qk_norm_bwd_workspace_bytes(dims, T), dtype=torch.uint8, device=DEV)
    dsa.qk_norm_rotate_bwd(dims, q.to(DEV), None, dy.to(DEV), None, dx, None, EPS, ws, q_weight=qw.to(DEV), dq_weight=dw,
                           rotation=rotation)
    h = 2.0 ** -4
    size = math.sqrt(T * Hq * d)
    for num, ana in (((f(q + h * v, qw) - f(q - h * v, qw)) / (2 * h), (dx.double().cpu() * v).sum()),
                     ((f(q, qw + h * vw) - f(q, qw - h * vw)) / (2 * h), (dw.double().cpu() * vw).sum())):
        assert abs(num - ana) <= 2e-3 * size, (num, ana)


def test_gradient_is_reproducible_and_can_be_captured():
    T, Hq, d = 5000, 16, 128
    g, q, k, qw, kw = _inputs(T, Hq, d, "bf16", 9)
    dims, rotation = _dims(T, Hq, d, "bf16"), dsa.make_rotation(_freq(128))
    qd, kd, dy, dyk = q.to(DEV), k.to(DEV), torch.randn(T, Hq, d, generator=g).to(DEV), torch.randn(T, d, generator=g).to(DEV)
    out = [torch.zeros(T, Hq, d, device=DEV), torch.zeros(T, d, device=DEV), torch.zeros(d, device=DEV), torch.zeros(d, device=DEV)]
    ws = torch.zeros(dsa.qk_norm_bwd_workspace_bytes(dims, T), dtype=torch.uint8, device=DEV)
    call = lambda: dsa.qk_norm_rotate_bwd(dims, qd, kd, dy, dyk, out[0], out[1], EPS, ws, q_weight=qw.to(DEV),  # noqa: E731
                                          k_weight=kw.to(DEV), dq_weight=out[2], dk_weight=out[3], rotation=rotation)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    first = [x.clone() for x in out]
    qwd, kwd = qw.to(DEV), kw.to(DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsa.qk_norm_rotate_bwd(dims, qd, kd, dy, dyk, out[0], out[1], EPS, ws, q_weight=qwd, k_weight=kwd, dq_weight=out[2],
                               dk_weight=out[3], rotation=rotation)
    for x in out:
        x.fill_(7.0)
    ws.fill_(0xFF)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(first, out))
    dy.copy_(dy.flip(0))
    dyk.copy_(dyk.flip(0))
    qd.copy_(qd.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    _check_bwd(out[0], out[2], qd.cpu(), qw, dy.cpu(), torch.arange(T), _freq(128), False)


def test_layer_gradient_through_the_norm():
    """Forward: norm, then the layer; backward: the layer's dQ and dK through the norm.  The chain's two ends as they are used."""
    L, Hq, d, k = 256, 16, 128, 8
    g, q, kk, qw, kw = _inputs(L, Hq, d, "bf16", 10)
    dims = dsa.make_dims(L, Hq, d, 8, 64, k)
    rotation = dsa.make_rotation(_freq(64))
    qo, ko = torch.zeros_like(q).to(DEV), torch.zeros_like(kk).to(DEV)
    kw_ = dict(q_weight=qw.to(DEV), k_weight=kw.to(DEV), rotation=rotation)
    dsa.qk_norm_rotate(dims, q.to(DEV), kk.to(DEV), qo, ko, EPS, **kw_)
    V = torch.randn(L, d, generator=g).to(torch.bfloat16).to(DEV)
    q_I, k_I = (torch.randint(-3, 4, s, generator=g).to(torch.bfloat16).to(DEV) for s in ((L, 8, 64), (L, 64)))
    w = torch.randint(1, 5, (L, 8), generator=g).float().to(DEV)
    f = dsa.alloc_forward_buffers(dims, o_acc=True)
    dsa.layer_fwd(dims, qo, ko, V, q_I, k_I, w, f.o, f.lse, f.idx, f.kpool, f.ws, o_acc=f.o_acc)
    do = torch.randn(L, Hq, d, generator=g).to(torch.bfloat16).to(DEV)
    dq, dk, dv = torch.zeros(L, Hq, d, device=DEV), torch.zeros(L, d, device=DEV), torch.zeros(L, d, device=DEV)
    dsa.layer_bwd(dims, qo, ko, V, f.idx, f.o, f.lse, do, dq, dk, dv, None, o_acc=f.o_acc)
    ws = torch.zeros(dsa.qk_norm_bwd_workspace_bytes(dims, L), dtype=torch.uint8, device=DEV)
    dy = dq.clone(), dk.clone()
    dqw, dkw = torch.zeros(d, device=DEV), torch.zeros(d, device=DEV)
    dsa.qk_norm_rotate_bwd(dims, q.to(DEV), kk.to(DEV), dq, dk, dq, dk, EPS, ws, dq_weight=dqw, dk_weight=dkw, **kw_)
    dsa.check_device_error()
    _check_bwd(dq, dqw, q, qw, dy[0].cpu(), torch.arange(L), _freq(64), False)
    _check_bwd(dk, dkw, kk, kw, dy[1].cpu(), torch.arange(L), _freq(64), False)
