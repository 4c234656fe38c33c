"""The root-mean-square norm with the residual's addition, and its backward pass.

The sum is compared bit for bit, the 8-bit result with act8_write of the same y.  The rest is compared with
the formula in 64 bits.  Tolerances of one value, e = 2^-24 (half a step of fp32) and 2^-8 for bf16:
  rstd      the sum of D squares takes at most 64 additions in a thread, 6 between lanes and 15 between waves,
            half of whose error reaches the root; with the division, root and reciprocal 64 e in all
  y         two products more and one rounding: (2^-8 + 68 e) |y|
  c         a sum as above of products rounded twice, and rstd: 160 e mean_d |w dy xhat|
  grad_s    (2^-8 + 2 e) |grad_s| + 2 e |dres| + rstd ((70 e) |w dy| + |xhat| (160 e mean |w dy xhat| + 140 e |c|))
  grad_w    T + 64 additions of products with xhat: (T + 140) e sum_t |dy xhat|
and bf16's smallest step, 2^-133, where values are subnormal.
"""

import ctypes

import pytest

from bit_quantized_finetuning_quant_amd import qlora
from helpers import announce, torch_mod

gpu = pytest.mark.gpu
E, HALF = 2.0**-24, 2.0**-8
TINY = 2.0**-133


def _inputs(T, D, seed, fp32=False, spread=1.0):
    torch = torch_mod()
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    big = torch.where(torch.rand(D, generator=g, device="cuda") < 0.02, 20.0, 1.0) * spread
    w = 1 + 0.3 * n(D)
    return {"x": (n(T, D) * spread).bfloat16(), "res": (n(T, D) * big).bfloat16(), "w": w if fp32 else w.bfloat16(),
            "dy": n(T, D).bfloat16(), "dres": n(T, D).bfloat16()}


def _y(s, w, eps):
    s, w = s.double(), w.double()
    return w * s / (s.square().mean(1, keepdim=True) + eps).sqrt()


def _grads(dy, s, w, eps, dres):
    """(value, tolerance) of grad_s and of grad_weight in 64 bits."""
    s, w, dy = s.double(), w.double(), dy.double()
    rstd = (s.square().mean(1, keepdim=True) + eps).rsqrt()
    xhat, wdy = s * rstd, w * dy
    c, ca = (wdy * xhat).mean(1, keepdim=True), (wdy * xhat).abs().mean(1, keepdim=True)
    gs = rstd * (wdy - xhat * c)
    tol = rstd * (70 * E * wdy.abs() + xhat.abs() * (160 * E * ca + 140 * E * c.abs()))
    if dres is not None:
        gs = gs + dres.double()
        tol = tol + 2 * E * dres.double().abs()
    gw = ((dy * xhat).sum(0), (s.shape[0] + 140) * E * (dy * xhat).abs().sum(0) + 1e-40)
    return (gs, tol + (HALF + 2 * E) * gs.abs() + TINY), gw


def _close(got, want, tol):
    off = (got.double() - want).abs() - tol
    assert bool((off <= 0).all()), float(off.max())


SIZES = [(1, 64), (1, 4096), (3, 128), (5, 576), (7, 1024), (66, 1088), (33, 2048), (2, 2112), (509, 4096), (31, 5120),
         (64, 8192), (9, 8256), (5, 16384), (3, 20480), (3, 33024), (2, 65536), (3000, 64)]


@gpu
@pytest.mark.parametrize("T,D", SIZES)
@pytest.mark.parametrize("fp32", [False, True])
def test_forward(T, D, fp32):
    torch = torch_mod()
    announce(f"norm forward T={T} D={D} fp32={fp32}")
    p = _inputs(T, D, T + D, fp32)
    y, s, a = qlora.rms_norm_fwd(p["x"], p["w"], 1e-5, residual=p["res"], need_act8=True)
    torch.cuda.synchronize()
    assert torch.equal(s, (p["x"].float() + p["res"].float()).bfloat16())
    want = _y(s, p["w"], 1e-5)
    _close(y, want, (HALF + 68 * E) * want.abs() + TINY)
    b = qlora.act8_write(y)
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scale, b.scale)
    # without a residual, and each result alone
    y1, s1, a1 = qlora.rms_norm_fwd(s, p["w"], 1e-5)
    assert s1 is s and a1 is None and torch.equal(y1, y)
    y2, _, a2 = qlora.rms_norm_fwd(s, p["w"], 1e-5, need_y=False, need_act8=True)
    assert y2 is None and torch.equal(a2.codes, a.codes) and torch.equal(a2.scale, a.scale)


@gpu
@pytest.mark.parametrize("T,D", SIZES)
@pytest.mark.parametrize("fp32", [False, True])
def test_backward(T, D, fp32):
    torch = torch_mod()
    announce(f"norm backward T={T} D={D} fp32={fp32}")
    p = _inputs(T, D, T + D + 1, fp32)
    for dres in (p["dres"], None):
        (gs, ts), (gw, tw) = _grads(p["dy"], p["res"], p["w"], 1e-5, dres)
        got, none = qlora.rms_norm_bwd(p["dy"], p["res"], p["w"], 1e-5, dres=dres)
        assert none is None
        _close(got, gs, ts)
        both, gotw = qlora.rms_norm_bwd(p["dy"], p["res"], p["w"], 1e-5, dres=dres, need_grad_weight=True)
        assert torch.equal(both, got)
        _close(gotw, gw, tw)
        again = qlora.rms_norm_bwd(p["dy"], p["res"], p["w"], 1e-5, dres=dres, need_grad_weight=True)[1]
        assert torch.equal(again, gotw)


@gpu
def test_gradients_are_those_of_differences():
    """Along random directions, the change of sum(dy y) over a step, in 64 bits, against the gradients."""
    torch = torch_mod()
    announce("norm gradients against differences")
    T, D, eps, step = 5, 192, 1e-5, 1e-5
    p = _inputs(T, D, 11, True)
    gs, gw = qlora.rms_norm_bwd(p["dy"], p["res"], p["w"], eps, need_grad_weight=True)
    s, w, dy = p["res"].double(), p["w"].double(), p["dy"].double()
    g = torch.Generator(device="cuda").manual_seed(5)
    (_, ts), (_, tw) = _grads(p["dy"], p["res"], p["w"], eps, None)
    for _ in range(4):
        v = torch.randn(T, D, generator=g, device="cuda", dtype=torch.float64)
        moved = [(dy * _y(s + k * step * v, w, eps)).sum() for k in (1, -1)]
        # the difference's own error: third derivatives times step^2, and rounding 2^-52 / step
        assert abs(float((moved[0] - moved[1]) / (2 * step) - (gs.double() * v).sum())) <= float((ts * v.abs()).sum()) + 1e-5
        v = torch.randn(D, generator=g, device="cuda", dtype=torch.float64)
        moved = [(dy * _y(s, w + k * step * v, eps)).sum() for k in (1, -1)]
        assert abs(float((moved[0] - moved[1]) / (2 * step) - (gw.double() * v).sum())) <= float((tw * v.abs()).sum()) + 1e-5


@gpu
@pytest.mark.parametrize("D", [64, 1024, 4096, 20480])
def test_rows_of_zeros_huge_tiny_and_not_finite_values(D):
    torch = torch_mod()
    announce(f"norm special rows D={D}")
    eps = 1e-6
    p = _inputs(9, D, D)
    s = p["res"].clone()
    s[1] = 0
    s[2] = (s[2].float() * 2.0**100).bfloat16()
    s[3] = (s[3].float() * 2.0**-100).bfloat16()
    s[4] = 3.3e38
    s[5, D // 2] = float("inf")
    s[6, 1] = float("nan")
    s[7, 0] = 2.0**120
    y, _, a = qlora.rms_norm_fwd(s, p["w"], eps, need_act8=True)
    gs, _ = qlora.rms_norm_bwd(p["dy"], s, p["w"], eps)
    gs2, gw = qlora.rms_norm_bwd(p["dy"][[0, 1, 2, 3, 4, 7, 8]], s[[0, 1, 2, 3, 4, 7, 8]], p["w"], eps,
                                 need_grad_weight=True)
    fine = [0, 1, 2, 3, 4, 7, 8]
    want = _y(s, p["w"], eps)
    _close(y[fine], want[fine], (HALF + 68 * E) * want[fine].abs() + 2 * TINY)
    (g, t), (w64, tw) = _grads(p["dy"][fine], s[fine], p["w"], eps, None)
    _close(gs[fine], g, t + 2 * TINY)
    assert torch.equal(gs2, gs[fine])
    _close(gw, w64, tw)
    assert bool((y[1] == 0).all()) and bool((a.codes[1] == 0).all())
    one = torch.zeros(D, dtype=torch.bool, device="cuda")
    one[D // 2] = True
    assert bool(y[5][one].isnan().all()) and bool((y[5][~one] == 0).all())
    assert bool(y[6].isnan().all()) and bool(gs[6].isnan().all())
    assert bool(gs[5][one].isnan().all())


@gpu
def test_in_place_on_a_stream_and_in_a_graph():
    """The sum replaces the residual, the gradient replaces dres; on a stream of its own, and captured."""
    torch = torch_mod()
    announce("norm in place, stream, graph")
    T, D = 77, 1152
    p = _inputs(T, D, 3)
    y, s, a = qlora.rms_norm_fwd(p["x"], p["w"], residual=p["res"], need_act8=True)
    gs, gw = qlora.rms_norm_bwd(p["dy"], s, p["w"], dres=p["dres"], need_grad_weight=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    res, dres, x = p["res"].clone(), p["dres"].clone(), p["x"].clone()
    side.wait_stream(torch.cuda.current_stream())
    y1, s1, a1 = qlora.rms_norm_fwd(p["x"], p["w"], residual=res, s=res, need_act8=True, stream=side)
    g1, w1 = qlora.rms_norm_bwd(p["dy"], s1, p["w"], dres=dres, grad_s=dres, need_grad_weight=True, stream=side)
    y2, s2, _ = qlora.rms_norm_fwd(x, p["w"], residual=p["res"], s=x, stream=side)
    dy = p["dy"].clone()
    side.wait_stream(torch.cuda.current_stream())
    g2, _ = qlora.rms_norm_bwd(dy, s, p["w"], dres=p["dres"], grad_s=dy, stream=side)
    side.synchronize()
    assert s1 is res and g1 is dres and s2 is x and g2 is dy
    for got, want in ((y1, y), (s1, s), (a1.codes, a.codes), (a1.scale, a.scale), (g1, gs), (w1, gw), (y2, y), (s2, s),
                      (g2, gs)):
        assert torch.equal(got, want)
    out = {"y": torch.empty_like(y), "s": torch.empty_like(s), "act8": qlora.Act8.empty(T, D)}
    back = {"grad_s": torch.empty_like(gs), "grad_weight": torch.empty_like(gw),
            "workspace": qlora.rms_norm_bwd_workspace(T, D)}

    def step():
        qlora.rms_norm_fwd(p["x"], p["w"], residual=p["res"], **out)
        qlora.rms_norm_bwd(p["dy"], out["s"], p["w"], dres=p["dres"], **back)

    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for t in (*out.values(), back["grad_s"], back["grad_weight"]):
            (t.codes if isinstance(t, qlora.Act8) else t).zero_()
        graph.replay()
        torch.cuda.synchronize()
        for got, want in ((out["y"], y), (out["s"], s), (out["act8"].codes, a.codes), (back["grad_s"], gs),
                          (back["grad_weight"], gw)):
            assert torch.equal(got, want)


@gpu
def test_rows_behind_the_last_stay_as_they_were():
    torch = torch_mod()
    announce("norm leaves what lies behind its rows")
    T, D = 5, 320
    p = _inputs(T, D, 8)
    big = {k: torch.full((T + 3, D), 7.0, dtype=torch.bfloat16, device="cuda") for k in ("y", "s", "g")}
    a = qlora.Act8(torch.full((T + 3, D), 7, dtype=torch.int8, device="cuda"),
                   torch.full((T + 3, D // 64), 7.0, device="cuda"))
    qlora.rms_norm_fwd(p["x"], p["w"], residual=p["res"], y=big["y"][:T], s=big["s"][:T],
                       act8=qlora.Act8(a.codes[:T], a.scale[:T]))
    qlora.rms_norm_bwd(p["dy"], p["res"], p["w"], grad_s=big["g"][:T])
    torch.cuda.synchronize()
    for t in (*big.values(), a.codes, a.scale):
        assert bool((t[T:] == 7).all()) and not bool((t[:T] == 7).all())


def test_refusals_of_the_binding():
    torch = torch_mod()
    x, w = torch.zeros(4, 128, dtype=torch.bfloat16), torch.zeros(128)
    f, b = qlora.rms_norm_fwd, qlora.rms_norm_bwd
    for call, says in (
            (lambda: f(x[0], w), "2-D"), (lambda: f(x[:, :100], w), "multiple of 64"),
            (lambda: f(x.float(), w), "x must be"), (lambda: f(x[:, :64], w[:64]), "contiguous"),
            (lambda: f(x, w[:64]), "weight must have shape"), (lambda: f(x, w.half()), "weight must be"),
            (lambda: f(x, w, residual=x[:2]), "residual must have shape"), (lambda: f(x, w, s=x), "without one it is x"),
            (lambda: f(x, w, need_y=False), "8-bit"), (lambda: f(x, w, y=x.float()), "y must be"),
            (lambda: f(x, w, act8=qlora.Act8.empty(4, 64, "cpu")), "act8 must hold 4 x 128"),
            (lambda: f(x, w), "on cpu"), (lambda: b(x, x[:, :100], w), "multiple of 64"),
            (lambda: b(x[:2], x, w), "dy must have shape"), (lambda: b(x, x, w, dres=x[:1]), "dres must have shape"),
            (lambda: b(x, x, w, grad_s=x.float()), "grad_s must be"),
            (lambda: b(x, x, w, grad_weight=w.bfloat16()), "grad_weight must be"), (lambda: b(x, x, w), "on cpu")):
        with pytest.raises(ValueError, match=says):
            call()


def test_refusals_of_the_c_abi():
    lib = qlora.lib()
    fake = 1 << 20  # 16-byte aligned, never dereferenced: every call is refused before a launch
    a8 = lambda T=4, K=128, c=fake, s=fake: ctypes.byref(qlora.Act8Struct(T, K, c, s))  # noqa: E731

    def fwd(x=fake, res=None, T=4, D=128, w=fake, dt=1, eps=1e-6, s=None, y=fake, y8=None):
        return lib.qlora_rms_norm_fwd(x, res, T, D, w, dt, eps, s, y, y8, None)

    def bwd(dy=fake, s=fake, dres=None, T=4, D=128, w=fake, dt=0, eps=1e-6, g=fake, gw=None, ws=None, n=0):
        return lib.qlora_rms_norm_bwd(dy, s, dres, T, D, w, dt, eps, g, gw, ws, n, None)

    for call in (fwd, bwd):
        for T, D in ((0, 128), (-1, 128), (4, 0), (4, 96), (4, 65536 + 64), (1 << 32, 64), (4, 1 << 40), (1 << 62, 1 << 62)):
            assert call(T=T, D=D) == 2
        for eps in (0.0, -1e-6, float("nan"), float("inf")):
            assert call(eps=eps) == 8
        assert call(dt=2) == 5 and call(dt=-1) == 5 and call(w=None) == 1 and call(w=fake + 4) == 3
    assert fwd(x=None) == 1 and fwd(y=None) == 1 and fwd(res=fake) == 1 and fwd(s=fake) == 1
    assert fwd(x=fake + 8) == 3 and fwd(res=fake + 2, s=fake) == 3 and fwd(res=fake, s=fake + 2) == 3 and fwd(y=fake + 2) == 3
    assert fwd(y8=a8(T=5)) == 2 and fwd(y8=a8(K=64)) == 2 and fwd(y8=a8(c=None)) == 1 and fwd(y8=a8(s=fake + 4)) == 3
    assert bwd(dy=None) == 1 and bwd(s=None) == 1 and bwd(g=None) == 1 and bwd(gw=fake) == 1
    assert bwd(dres=fake + 2) == 3 and bwd(g=fake + 2) == 3 and bwd(gw=fake + 4, ws=fake) == 3
    need = lib.qlora_rms_norm_bwd_workspace_bytes(4, 128)
    assert need > 0 and bwd(gw=fake, ws=fake, n=need - 1) == 4
    assert lib.qlora_rms_norm_bwd_workspace_bytes(1 << 20, 65536) <= 2048 * 65536 * 4
    assert lib.qlora_rms_norm_bwd_workspace_bytes(0, 128) == 0 and lib.qlora_rms_norm_bwd_workspace_bytes(4, 100) == 0
