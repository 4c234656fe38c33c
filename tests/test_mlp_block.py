"""The operators of a feed-forward block as a decoder layer runs them, forward and backward: the norm with the residual's
addition (its result also in 8 bits), the gated product behind its projections (in 8 bits for the down projection's
backward pass), the down projection, and back through the gated product into the projections' checkpointed backward pass
and the norm.

The forward results and gradients are compared, normwise within 1e-2 as those of the linear layers are, with the block
in 64 bits and its gradients by automatic differentiation there; the operators by themselves have tolerances of their
own elsewhere."""

import pytest

from bit_quantized_finetuning_quant_amd import qlora
from helpers import NORMWISE_TOL, announce, torch_mod

pytestmark = pytest.mark.gpu
EPS = 1e-5


def _layer(T, D, F, r, seed):
    torch = torch_mod()
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return {"x": n(T, D).bfloat16(), "res": (2 * n(T, D)).bfloat16(), "w": 1 + 0.2 * n(D), "dy": n(T, D).bfloat16(),
            "q": [qlora.quantize(n(F, D) * D**-0.5) for _ in range(2)], "qd": qlora.quantize(n(D, F) * F**-0.5),
            "A": (n(2 * r, D) * 0.05).bfloat16(), "B": [(n(F, r) * 0.1).bfloat16() for _ in range(2)],
            "Ad": (n(r, F) * 0.05).bfloat16(), "Bd": (n(D, r) * 0.1).bfloat16(), "scale": 2.0}


def _step(p, act, out=None):
    """Everything that the pass gives, by name; `out`: the buffers and workspaces to write into."""
    o = out or {}
    k = p["scale"]
    y, s, a = qlora.rms_norm_fwd(p["x"], p["w"], EPS, residual=p["res"], s=o.get("s"), y=o.get("y"), act8=o.get("a"),
                                 need_act8=True)
    g = qlora.linear_gated_fwd(y, p["q"], p["A"], p["B"], k, act, h=o.get("h"), act8=o.get("h8"), need_act8=True,
                               gate=o.get("gate"), up=o.get("up"), u_out=o.get("u"), workspace=o.get("wg"))
    z, ud = qlora.linear_fwd(g.h, p["qd"], p["Ad"], p["Bd"], k, y=o.get("z"), u_out=o.get("ud"), workspace=o.get("wd"))
    # the gradient that arrives at the layer's output reaches the down projection and, past it, the residual stream
    dh, gAd, gBd = qlora.linear_bwd_act8(p["dy"], g.act8, p["qd"], p["Ad"], p["Bd"], k, ud, grad_x=o.get("dh"),
                                         grad_A=o.get("gAd"), grad_B=o.get("gBd"), workspace=o.get("wdb"))
    dgate, dup = qlora.gated_act_bwd(dh, g.gate, g.up, act, dgate=o.get("dgate"), dup=o.get("dup"))
    dn, gA, gB = qlora.linear_set_bwd_act8([dgate, dup], a, p["q"], p["A"], p["B"], k, g.u, grad_x=o.get("dn"),
                                           grad_A_set=o.get("gA"), grad_Bs=o.get("gB"), workspace=o.get("wb"))
    ds, gw = qlora.rms_norm_bwd(dn, s, p["w"], EPS, dres=p["dy"], grad_s=o.get("ds"), need_grad_weight=True,
                                grad_weight=o.get("gw"), workspace=o.get("wn"))
    return {"s": s, "y": y, "a": a, "h": g.h, "h8": g.act8, "gate": g.gate, "up": g.up, "u": g.u, "z": z, "ud": ud, "dh": dh,
            "gAd": gAd, "gBd": gBd, "dgate": dgate, "dup": dup, "dn": dn, "gA": gA, "gB": gB, "ds": ds, "gw": gw}


def _reference(p, act):
    """The same in 64 bits: the layer's output is s + down(h), the loss dy . output."""
    torch = torch_mod()
    d = lambda t: t.detach().double().requires_grad_()  # noqa: E731
    k, r = p["scale"], p["Ad"].shape[0]
    s, w, A, Ad, Bd = d((p["x"].double() + p["res"].double()).bfloat16()), d(p["w"]), d(p["A"]), d(p["Ad"]), d(p["Bd"])
    B = [d(b) for b in p["B"]]
    W = [qlora.dequantize(q).double() for q in p["q"]]
    Wd = qlora.dequantize(p["qd"]).double()
    y = w * s / (s.square().mean(1, keepdim=True) + EPS).sqrt()
    gate, up = (y @ W[i].t() + k * (y @ A[i * r:(i + 1) * r].t()) @ B[i].t() for i in range(2))
    f = torch.nn.functional
    h = (f.silu(gate) if act == "silu" else f.gelu(gate, approximate="tanh")) * up
    z = h @ Wd.t() + k * (h @ Ad.t()) @ Bd.t()
    ((s + z) * p["dy"].double()).sum().backward()
    return {"y": y, "h": h, "z": z, "gAd": Ad.grad, "gBd": Bd.grad, "gA": A.grad, "gB": [b.grad for b in B], "ds": s.grad,
            "gw": w.grad}


@pytest.mark.parametrize("T,D,F,r,act", [(1, 128, 192, 8, "silu"), (7, 256, 704, 4, "gelu_tanh"), (64, 512, 1344, 16, "silu"),
                                         (100, 320, 512, 7, "silu"), (333, 512, 1408, 16, "gelu_tanh"),
                                         (2100, 1024, 2752, 64, "silu")])
def test_a_block_forward_and_backward(T, D, F, r, act):
    torch = torch_mod()
    announce(f"feed-forward block T={T} D={D} F={F} r={r} {act}")
    p = _layer(T, D, F, r, T)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _step(p, act)
    torch.cuda.current_stream().wait_stream(side)
    for name, want in _reference(p, act).items():
        for g, w in zip(*(([t] if not isinstance(t, list) else t) for t in (got[name], want))):
            off = float((g.double() - w.detach()).norm() / w.detach().norm())
            # what is read back in 8 bits is off by half a code, absmax / 254 of its 64 values
            assert off <= (NORMWISE_TOL if name not in ("gAd", "gA") else 2 * NORMWISE_TOL), (name, off)


def test_captured_passes_equal_eager_ones():
    """A pass into given buffers, captured once and replayed on three inputs, with eager work between the replays."""
    torch = torch_mod()
    announce("feed-forward block under graph capture")
    T, D, F, r = 300, 256, 704, 8
    p = _layer(T, D, F, r, 5)
    inputs = [_layer(T, D, F, r, s) for s in (5, 6, 7)]
    want = [_step(dict(p, x=i["x"], res=i["res"], dy=i["dy"]), "silu") for i in inputs]
    out = {k: (qlora.Act8(v.codes.clone(), v.scale.clone()) if isinstance(v, qlora.Act8) else [t.clone() for t in v]
               if isinstance(v, list) else v.clone()) for k, v in want[0].items()}
    out |= {"wg": qlora.linear_gated_workspace(T, F, D, r), "wd": qlora.linear_workspace(T, D, F, r),
            "wdb": qlora.linear_set_act8_workspace(T, [D], F, r), "wb": qlora.linear_set_act8_workspace(T, [F, F], D, r),
            "wn": qlora.rms_norm_bwd_workspace(T, D)}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(p, "silu", out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _step(p, "silu", out)
    for i, w in zip(inputs, want):
        for k in ("x", "res", "dy"):
            p[k].copy_(i[k])
        graph.replay()
        torch.cuda.synchronize()
        for k, v in w.items():
            for a, b in zip(*((t if isinstance(t, list) else [t.codes, t.scale] if isinstance(t, qlora.Act8) else [t])
                              for t in (out[k], v))):
                assert torch.equal(a, b), k
        torch.zeros(1000, device="cuda").add_(1.0)


def test_two_streams_at_once():
    """Two blocks on streams of their own, each with its own workspaces: the results of each alone."""
    torch = torch_mod()
    announce("feed-forward blocks on two streams")
    ps = [_layer(T, 512, 1344, 16, T) for T in (200, 40)]
    alone = [_step(p, "silu") for p in ps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    for _ in range(3):
        got = []
        for p, s in zip(ps, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(_step(p, "silu"))
        torch.cuda.synchronize()
        for g, a in zip(got, alone):
            for k in ("z", "ds", "gw", "gA", "gAd"):
                assert torch.equal(g[k], a[k]), k


def test_a_buffer_named_for_two_results_is_refused():
    torch = torch_mod()
    announce("feed-forward operators: a buffer named twice")
    p = _layer(4, 128, 128, 8, 1)
    x, r, q = p["x"], p["res"], p["q"]
    t = torch.zeros_like(x)
    for call in (lambda: qlora.rms_norm_fwd(x, p["w"], EPS, residual=r, s=t, y=t),
                 lambda: qlora.gated_act_bwd(x, r, r, dgate=t, dup=t),
                 lambda: qlora.linear_gated_fwd(x, q, p["A"], p["B"], 1.0, h=t, gate=t),
                 lambda: qlora.linear_gated_fwd(x, q, p["A"], p["B"], 1.0, gate=t, up=t),
                 lambda: qlora.linear_gated_fwd(x, q, p["A"], p["B"], 1.0, h=x)):
        with pytest.raises(qlora.QloraError, match="named for two results"):
            call()
    torch.cuda.synchronize()
    assert bool((t == 0).all())


def test_trusted_calls_give_the_same():
    torch = torch_mod()
    announce("feed-forward block, trusted calls")
    p = _layer(70, 256, 704, 8, 9)
    want = _step(p, "gelu_tanh")
    with qlora.trusted_calls():
        got = _step(p, "gelu_tanh")
    for k in ("z", "s", "h", "ds", "gw", "gA", "gAd"):
        assert torch.equal(got[k], want[k]), k
    assert torch.equal(got["a"].codes, want["a"].codes) and torch.equal(got["h8"].scale, want["h8"].scale)


def test_more_than_2_31_values():
    """Rows past 2^31 values: the last ones are those of a call on them alone (rows are independent of each other)."""
    torch = torch_mod()
    T, N = 200_001, 11008
    announce(f"feed-forward operators, {T} x {N}")
    g = torch.Generator(device="cuda").manual_seed(1)
    gate, up = (torch.empty(T, N, dtype=torch.bfloat16, device="cuda").normal_(generator=g) for _ in range(2))
    last = slice(T - 37, T)
    h, a = qlora.gated_act_fwd(gate, up, need_act8=True)
    h2, a2 = qlora.gated_act_fwd(gate[last], up[last], need_act8=True)
    assert torch.equal(h[last], h2) and torch.equal(a.codes[last], a2.codes) and torch.equal(a.scale[last], a2.scale)
    del a, a2
    for b, c in zip(qlora.gated_act_bwd(h, gate, up), qlora.gated_act_bwd(h[last], gate[last], up[last])):
        assert torch.equal(b[last], c)
    w = torch.randn(N, device="cuda")
    y, s, _ = qlora.rms_norm_fwd(gate, w, EPS, residual=up)
    y2, s2, _ = qlora.rms_norm_fwd(gate[last], w, EPS, residual=up[last])
    assert torch.equal(y[last], y2) and torch.equal(s[last], s2)
    ds = qlora.rms_norm_bwd(h, s, w, EPS, dres=up)[0]
    assert torch.equal(ds[last], qlora.rms_norm_bwd(h[last], s2, w, EPS, dres=up[last])[0])
    del y, s, ds, h, gate, up
    # behind the projections: 300 rows take the tiles that the whole takes, or tiles whose sums differ in their order
    K, r = 64, 8
    qs = [qlora.quantize(torch.randn(N, K, generator=g, device="cuda")) for _ in range(2)]
    x = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    A, Bs = torch.randn(2 * r, K, generator=g, device="cuda").bfloat16(), [torch.randn(N, r, generator=g, device="cuda").bfloat16()
                                                                        for _ in range(2)]
    out = qlora.linear_gated_fwd(x, qs, A, Bs, 0.25)
    few = qlora.linear_gated_fwd(x[-300:], qs, A, Bs, 0.25)
    for k in ("h", "gate", "up", "u"):
        a, b = getattr(out, k)[-300:].double(), getattr(few, k).double()
        assert float((a - b).norm() / b.norm()) <= NORMWISE_TOL, k
