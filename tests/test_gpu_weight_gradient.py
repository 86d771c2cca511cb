"""The heads' weight gradients over many tokens, with a tolerance that a lost part of the sum cannot hide in.

Terms g xn are each off by t P |xn| + a |g xn| (test_gpu_heads), twice that for the products' own roundings.  They are added in fp32: by a
lane one after the other, at most K of them; then over a warp's groups (2 additions at most), over 8 warps (7), and over the CTAs
with the roundings carried along (2^-23 of the sum, and once more for the result): (K + 16) 2^-24 of the terms' magnitudes
in all.  K: a CTA has G = 256 / lanes groups, a block of G / s tokens by s shares of the heads, 304 CTAs at most go through the
blocks; so K = ceil(ceil(T s / G) / 304) ceil(H / s), which for s < 2 H is at most 2 T H / (304 G) + 4 H."""
import pytest
import torch

import long_context_sparse_dsa_gb300 as dsa
from test_gpu_decode import DEV, _built, _freq  # noqa: F401
from test_gpu_heads import B, EPS, _dims, _inputs, _norm, _pair_sum, _turned

pytestmark = pytest.mark.gpu


def _expect(x, dy, pos, freq, inter, dtype):
    """dw, its tolerance, and every token's part of it."""
    T, H, d = x.shape
    a, t = d * 2.0 ** -25 + 2.0 ** -21, B + 2.0 ** -22
    xn, _, _ = _norm(x, None)
    g, P = _turned(dy.double(), pos, freq, inter, back=True), _pair_sum(dy.double(), 0 if freq is None else 2 * freq.numel(), inter)
    lanes = d // (16 if dtype == "bf16" else 8)
    K = 2 * T * H / (304 * (256 // lanes)) + 4 * H
    terms = g * xn
    tol = 2 * (t * P * xn.abs() + a * terms.abs()).sum((0, 1)) + (K + 16) * 2.0 ** -24 * terms.abs().sum((0, 1))
    return terms.sum((0, 1)), tol, terms.sum(1)


@pytest.mark.parametrize("dtype,Hq,d,rot,inter,T", [
    ("bf16", 16, 128, 64, False, 20011), ("bf16", 16, 128, 128, False, 5000), ("bf16", 32, 64, 64, True, 9001), ("bf16", 3, 128, 0, False, 30001),
    ("bf16", 1, 64, 16, False, 100003), ("fp32", 8, 64, 16, True, 4093), ("fp32", 32, 128, 128, False, 3001), ("fp32", 5, 128, 96, True, 20000)])
def test_no_part_of_the_sum_is_lost(dtype, Hq, d, rot, inter, T):
    g, q, k, qw, kw = _inputs(T, Hq, d, dtype, T + Hq)
    freq = _freq(rot) if rot else None
    dims, rotation = _dims(T, Hq, d, dtype), dsa.make_rotation(freq, interleaved=inter) if rot else None
    dy, dyk = torch.randn(T, Hq, d, generator=g), torch.randn(T, d, generator=g)
    dq, dk = torch.zeros(T, Hq, d, device=DEV), torch.zeros(T, d, device=DEV)
    dqw, dkw = torch.full((d,), 7.0, device=DEV), torch.full((d,), 7.0, device=DEV)
    ws = torch.full((dsa.qk_norm_bwd_workspace_bytes(dims, T),), 0xFF, dtype=torch.uint8, device=DEV)
    dsa.qk_norm_rotate_bwd(dims, q.to(DEV), k.to(DEV), dy.to(DEV), dyk.to(DEV), dq, dk, EPS, ws, q_weight=qw.to(DEV),
                           k_weight=kw.to(DEV), dq_weight=dqw, dk_weight=dkw, rotation=rotation)
    dsa.check_device_error()
    pos, n = torch.arange(T), 256 // (d // (16 if dtype == "bf16" else 8))
    for got, x, y in ((dqw, q, dy), (dkw, k[:, None], dyk[:, None])):
        want, tol, parts = _expect(x, y, pos, freq, inter, dtype)
        # the tolerance is far below the sum, and most channels show a block of tokens, or one part in 304, that is missing
        assert tol.max() < 0.1 * want.abs().mean()
        for lost in (parts[-n:].sum(0), parts[::304].sum(0)):
            assert (lost.abs() > tol).double().mean() > 0.5
        err = (got.double().cpu() - want).abs()
        assert torch.all(err <= tol), (err / tol).max()
