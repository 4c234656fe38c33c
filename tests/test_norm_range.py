"""The root-mean-square norm and its backward pass at the far ends of their range, and with several rows a workgroup.

Reference and tolerances are those of `test_norm.py`, unless a case says otherwise."""

import pytest

from bit_quantized_finetuning_quant_amd import qlora
from helpers import announce, torch_mod
from test_norm import E, HALF, TINY, _close, _grads, _inputs, _y

gpu = pytest.mark.gpu
DIMS = [64, 1024, 2048, 4096, 8192, 16384, 20480]


@gpu
@pytest.mark.parametrize("D", DIMS)
def test_small_values_beside_huge_ones(D):
    """A value of 2^66 takes its row's squares past fp32.  The others, from 2^-50 to 2^0, keep their precision: y, and
    (one row) grad_weight = dy xhat, are near 2^-113 and up, far above bf16's smallest normal value."""
    torch = torch_mod()
    announce(f"norm, small values beside huge ones D={D}")
    eps = 1e-6
    p = _inputs(3, D, D, True)
    size = torch.randint(-50, 1, (3, D), device="cuda", generator=torch.Generator(device="cuda").manual_seed(D))
    s = torch.ldexp(p["dy"].float().sign() * (1 + p["x"].float().abs().clamp_max(0.9)), size).bfloat16()
    s[:, D // 3] = 2.0**66
    y = qlora.rms_norm_fwd(s, p["w"], eps)[0]
    want = _y(s, p["w"], eps)
    _close(y, want, (HALF + 68 * E) * want.abs() + TINY)
    for t in range(3):
        one = slice(t, t + 1)
        (gs, ts), (gw, tw) = _grads(p["dy"][one], s[one], p["w"], eps, None)
        got, gotw = qlora.rms_norm_bwd(p["dy"][one], s[one], p["w"], eps, need_grad_weight=True)
        _close(got, gs, ts)
        # (the bound of `_grads` ends in a constant that these values lie below)
        _close(gotw, gw, 141 * E * gw.abs())


@gpu
@pytest.mark.parametrize("D", DIMS)
def test_large_gradients_of_large_rows(D):
    """|w dy s| past fp32, where c = mean(w dy xhat) and the gradients are not: rows whose squares fit fp32 and rows whose
    squares do not."""
    torch = torch_mod()
    announce(f"norm backward, large gradients D={D}")
    eps = 1e-6
    p = _inputs(5, D, D + 5, True)
    s, dy = p["res"].double(), p["dy"].double()
    for row, (of_s, of_dy) in enumerate([(1e15, 1e25), (1e17, 1e34), (1e33, 1e34), (1.0, 1.0), (1e36, 1e34)]):
        s[row] *= of_s
        dy[row] *= of_dy
    s, dy = s.bfloat16(), dy.bfloat16()
    assert bool(s.isfinite().all()) and float((p["w"].double() * dy.double()).abs().max()) < 2.0**119
    for rows in ([0, 1, 2, 3, 4], [0], [1], [2], [4]):
        a, b = dy[rows], s[rows]
        (gs, ts), (gw, tw) = _grads(a, b, p["w"], eps, None)
        got, gotw = qlora.rms_norm_bwd(a, b, p["w"], eps, need_grad_weight=True)
        _close(got, gs, ts)
        _close(gotw, gw, tw)


@gpu
def test_the_largest_eps():
    """mean + eps past fp32, where the root is not."""
    torch = torch_mod()
    announce("norm, the largest eps")
    eps, D = float(torch.finfo(torch.float32).max), 64
    p = _inputs(4, D, 4, True)
    s = (1.7e18 * (1 + 0.01 * p["x"].double().clamp(-3, 3))).bfloat16()
    assert float(s.float().square().sum(1).max()) < eps  # the squares' sum fits
    y = qlora.rms_norm_fwd(s, p["w"], eps)[0]
    want = _y(s, p["w"], eps)
    _close(y, want, (HALF + 68 * E) * want.abs() + TINY)
    (gs, ts), (gw, tw) = _grads(p["dy"], s, p["w"], eps, None)
    got, gotw = qlora.rms_norm_bwd(p["dy"], s, p["w"], eps, need_grad_weight=True)
    _close(got, gs, ts)
    _close(gotw, gw, tw)


@gpu
@pytest.mark.parametrize("T,D", [(1300, 2048), (1100, 4096), (700, 8192), (520, 16384), (300, 20480), (2500, 1024),
                                 (4097, 8192)])
@pytest.mark.parametrize("fp32", [False, True])
def test_backward_of_several_rows_a_workgroup(T, D, fp32):
    """More rows than workgroups, some with one row more than others; 4097 x 8192 with dres reads 201 MB, past the
    caches.  (The rows' order does not change their own gradient: the launch without grad_weight has a workgroup a row.)"""
    torch = torch_mod()
    announce(f"norm backward, several rows a workgroup T={T} D={D} fp32={fp32}")
    p = _inputs(T, D, T + D, fp32)
    for dres in (p["dres"], None):
        (gs, ts), (gw, tw) = _grads(p["dy"], p["res"], p["w"], 1e-5, dres)
        got, gotw = qlora.rms_norm_bwd(p["dy"], p["res"], p["w"], 1e-5, dres=dres, need_grad_weight=True)
        _close(got, gs, ts)
        _close(gotw, gw, tw)
        assert torch.equal(qlora.rms_norm_bwd(p["dy"], p["res"], p["w"], 1e-5, dres=dres)[0], got)
        assert torch.equal(qlora.rms_norm_bwd(p["dy"], p["res"], p["w"], 1e-5, dres=dres, need_grad_weight=True)[1], gotw)


@pytest.mark.parametrize("D", [64, 1024, 1088, 4096, 4160, 8192, 65536])
def test_workspace_is_at_most_512_rows_of_sums(D):
    for T in (1, 3, 511, 512, 513, 2047, 2049, 1 << 20, (1 << 37) // D):
        assert 0 < qlora.rms_norm_bwd_workspace_bytes(T, D) <= 512 * D * 4
