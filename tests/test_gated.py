"""The gated product h = act(gate) up: alone, its backward pass, and behind its projections.

Everything is compared with the formula in 64 bits; the 8-bit results bit for bit with act8_write of h.
Tolerances of one value, e = 2^-24 (half a step of fp32) and 2^-8 for bf16.  sigma comes from exp2 of
|z| log2 e: z is off by up to 4 e of itself, the argument by one rounding more and the constant's, so sigma and
1 - sigma are off by (5 |z| + 16) e of themselves, `sg`; below 2^-126 they may be 0, which moves act by |g| 2^-126
and act' = s + g s t z' by (1 + |g| z') 2^-126 (z' grows with g^2 for gelu: 15 at g = -8, where sigma is 2^-127).
  act      sg + 2 e of itself
  act'     s + g s t z': (sg + 8 e) of s and twice that of |g s t z'|
  h        (2^-8 + sg + 4 e) |h|;   dup alike;   dgate 2^-8 of itself and |dh up| times the error of act'
Behind the projections gate and up are fp32 sums with u in bf16: with P = |x| |W| and U = |x| |A|,
  dg       (K + r + 8) e P + |scale| ((2^-8 + (K + r + 8) e) U) |B|          (du alike)
  gate     dg + 2^-8 |gate|
  h        1.13 dg (|up| + du) + |act| du + (2^-8 + sg + 4 e) of the largest |h| these leave,
           since |act'| <= 1.13 for both activations
"""

import ctypes
import math

import pytest

from bit_quantized_finetuning_quant_amd import qlora
from helpers import announce, torch_mod

gpu = pytest.mark.gpu
E, HALF = 2.0**-24, 2.0**-8
TINY = 2.0**-133
ACTS = ("silu", "gelu_tanh")
K2, C3 = 2 * math.sqrt(2 / math.pi), 0.044715


def _act(act, g):
    """(act, act', s, |g s t z'|, z', relative error of sigma) in 64 bits."""
    torch = torch_mod()
    z = g if act == "silu" else K2 * (g + C3 * g**3)
    dz = torch.ones_like(g) if act == "silu" else K2 * (1 + 3 * C3 * g * g)
    e = torch.exp(-z.abs())
    low, high = e / (1 + e), 1 / (1 + e)
    s, t = torch.where(z < 0, low, high), torch.where(z < 0, high, low)
    # past |g| = 128 the product is below 2^-180
    bend = torch.where(g.abs() > 128, torch.zeros_like(g), g * s * t * dz)
    sg = (5 * z.abs().clamp_max(110) + 16) * E
    value = torch.where(g == -math.inf, torch.zeros_like(g), g * s)
    return value, s + bend, s, bend.abs(), dz, sg


def _close(got, want, tol):
    off = (got.double() - want).abs() - tol
    assert bool((off <= 0).all()), float(off.max())


def _check_product(h, gate, up, act):
    value, _, _, _, _, sg = _act(act, gate.double())
    want = value * up.double()
    _close(h, want, (HALF + sg + 4 * E) * want.abs() + 2.0**-126 * (gate.double() * up.double()).abs().clamp_max(1e300) + TINY)


def _check_grads(dgate, dup, dh, gate, up, act):
    dh, gate, up = dh.double(), gate.double(), up.double()
    value, slope, s, bend, dz, sg = _act(act, gate)
    want = dh * up * slope
    small = gate.abs().clamp_max(128)  # past it sigma or 1 - sigma is 0 in either form
    flush = 2.0**-126 * (1 + small * dz.clamp_max(4000))
    tol = HALF * want.abs() + (1 + HALF) * (dh * up).abs() * ((sg + 8 * E) * (s + 2 * bend) + 2 * E * slope.abs() + flush)
    _close(dgate, want, tol + TINY)
    want = dh * value
    _close(dup, want, (HALF + sg + 4 * E) * want.abs() + dh.abs() * 2.0**-126 * gate.abs() + TINY)


@gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,N", [(1, 64), (3, 128), (2, 320), (7, 1088), (129, 704), (33, 11008), (1000, 2048)])
def test_product_and_gradients(T, N, act):
    torch = torch_mod()
    announce(f"gated product T={T} N={N} {act}")
    g = torch.Generator(device="cuda").manual_seed(T + N)
    n = lambda: torch.randn(T, N, generator=g, device="cuda")  # noqa: E731
    gate, up, dh = (n() * 3).bfloat16(), n().bfloat16(), n().bfloat16()
    h, a = qlora.gated_act_fwd(gate, up, act, need_act8=True)
    dgate, dup = qlora.gated_act_bwd(dh, gate, up, act)
    torch.cuda.synchronize()
    _check_product(h, gate, up, act)
    b = qlora.act8_write(h)
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scale, b.scale)
    none, a2 = qlora.gated_act_fwd(gate, up, act, need_h=False, need_act8=True)
    assert none is None and torch.equal(a2.codes, a.codes) and torch.equal(a2.scale, a.scale)
    _check_grads(dgate, dup, dh, gate, up, act)
    # in place, each place that is allowed
    for take in range(3):
        t = [dh.clone(), gate.clone(), up.clone()]
        out = qlora.gated_act_bwd(*t, act, dgate=t[take], dup=t[(take + 1) % 3])
        assert torch.equal(out[0], dgate) and torch.equal(out[1], dup)
    for take in range(2):
        t = [gate.clone(), up.clone()]
        assert torch.equal(qlora.gated_act_fwd(*t, act, h=t[take])[0], h)


@gpu
@pytest.mark.parametrize("act", ACTS)
def test_every_gate(act):
    """All finite bf16 gates, both infinities and NaN."""
    torch = torch_mod()
    announce(f"every gate {act}")
    gate = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).cuda().view(-1, 512)
    for size in (1.0, -0.75, 2.0**-20):
        up = torch.full_like(gate, size)
        dh = torch.full_like(gate, 0.5)
        h, _ = qlora.gated_act_fwd(gate, up, act)
        dgate, dup = qlora.gated_act_bwd(dh, gate, up, act)
        ok = gate.isfinite()
        f = lambda t: t[ok][None]  # noqa: E731
        _check_product(f(h), f(gate), f(up), act)
        _check_grads(f(dgate), f(dup), f(dh), f(gate), f(up), act)
        nan = gate.isnan()
        assert bool(h[nan].isnan().all()) and bool(dgate[nan].isnan().all()) and bool(dup[nan].isnan().all())
        low, high = gate == -math.inf, gate == math.inf
        assert bool((h[low] == 0).all()) and bool((dup[low] == 0).all()) and bool((dgate[low] == 0).all())
        assert bool((h[high] == math.copysign(math.inf, size)).all()) and bool((dup[high] == math.inf).all())
        assert bool((dgate[high].float() == 0.5 * size).all())


@gpu
@pytest.mark.parametrize("act", ACTS)
def test_gradients_are_those_of_differences(act):
    torch = torch_mod()
    announce(f"gated gradients against differences {act}")
    g = torch.Generator(device="cuda").manual_seed(2)
    gate, up, dh = (torch.randn(4, 128, generator=g, device="cuda").bfloat16() for _ in range(3))
    dgate, dup = qlora.gated_act_bwd(dh, gate, up, act)
    step = 1e-5
    a, b, d = gate.double(), up.double(), dh.double()
    slope = d * b * (_act(act, a + step)[0] - _act(act, a - step)[0]) / (2 * step)
    _close(dgate, slope, HALF * slope.abs() + (d * b).abs() * 1e-6 + 1e-9)
    value = d * (_act(act, a)[0] * ((b + step) - (b - step))) / (2 * step)
    _close(dup, value, HALF * value.abs() + (d * a).abs() * 1e-6 + 1e-9)


# ------------------------------------------------------------- behind the projections
def _block(T, K, N, r, seed, dq=True):
    torch = torch_mod()
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return {"x": n(T, K).bfloat16(), "qs": [qlora.quantize(n(N, K) * K**-0.5, double_quant=dq) for _ in range(2)],
            "A": (n(2 * r, K) * 0.05).bfloat16(), "Bs": [(n(N, r) * 0.1).bfloat16() for _ in range(2)], "scale": 16.0 / r}


def _expect(p, act):
    """{name: (value, tolerance)} of h, gate, up and u in 64 bits."""
    torch = torch_mod()
    mm = lambda a, b: torch.mm(a, b.t().contiguous())  # noqa: E731
    x, A, k = p["x"].double(), p["A"].double(), abs(p["scale"])
    r, K = A.shape[0] // 2, x.shape[1]
    many = (K + r + 8) * E
    out, v = {}, []
    u, U = mm(x, A), mm(x.abs(), A.abs())
    out["u"] = (u, HALF * u.abs() + (1 + HALF) * K * E * U)
    for i, (q, B) in enumerate(zip(p["qs"], p["Bs"])):
        W, B, cols = qlora.dequantize(q).double(), B.double(), slice(i * r, (i + 1) * r)
        y = mm(x, W) + p["scale"] * mm(u[:, cols].contiguous(), B)
        tol = many * mm(x.abs(), W.abs()) + k * (HALF + many) * mm(U[:, cols].contiguous(), B.abs())
        v.append((y, tol))
        out["gate" if i == 0 else "up"] = (y, tol * (1 + HALF) + HALF * y.abs())
    (g, dg), (up, du) = v
    value, _, _, _, _, sg = _act(act, g)
    move = 1.13 * dg * (up.abs() + du) + value.abs() * du
    out["h"] = (value * up, move + (HALF + sg + 4 * E) * ((value * up).abs() + move) + TINY)
    return out


def _check_block(p, out, act):
    for name, (want, tol) in _expect(p, act).items():
        got = getattr(out, name)
        if got is not None:
            _close(got, want, tol)


BLOCKS = [(1, 64, 64, 1), (1, 4096, 1024, 16), (2, 192, 320, 7), (3, 128, 192, 64), (4, 320, 64, 100), (5, 1024, 704, 8),
          (8, 256, 2112, 16), (16, 2048, 512, 8), (17, 512, 320, 8), (33, 4096, 704, 16), (48, 1088, 448, 16),
          (64, 704, 1024, 32), (65, 256, 320, 7), (100, 4096, 256, 128), (128, 512, 832, 256), (129, 320, 576, 8),
          (255, 192, 64, 1), (256, 128, 128, 16), (300, 4096, 320, 64), (511, 64, 1088, 8), (513, 2112, 192, 100),
          (1000, 256, 704, 64), (1024, 512, 1024, 8), (2049, 320, 448, 16), (4096, 128, 192, 200), (2, 262208, 64, 8),
          (40, 131136, 128, 16), (40, 65600, 832, 200), (23, 16448, 3264, 16), (64, 8192, 6208, 7),
          (3, 64, 4194240, 8), (70, 64, 1048640, 8), (1, 4194240, 64, 8), (200, 65600, 64, 1)]


@gpu
@pytest.mark.parametrize("T,K,N,r", BLOCKS)
def test_block(T, K, N, r):
    torch = torch_mod()
    act, dq = ACTS[(T + r) % 2], (T + K // 64) % 2 == 0
    announce(f"gated block T={T} K={K} N={N} r={r} {act} dq={dq}")
    p = _block(T, K, N, r, T + K + N + r, dq)
    a = (p["x"], p["qs"], p["A"], p["Bs"], p["scale"], act)
    out = qlora.linear_gated_fwd(*a, need_act8=True)
    torch.cuda.synchronize()
    _check_block(p, out, act)
    b = qlora.act8_write(out.h)
    assert torch.equal(out.act8.codes, b.codes) and torch.equal(out.act8.scale, b.scale)
    # what is not asked for is not written, and the rest stays the same
    lean = qlora.linear_gated_fwd(*a, keep=False)
    assert torch.equal(lean.h, out.h) and lean[1:] == (None,) * 4
    only8 = qlora.linear_gated_fwd(*a, keep=False, need_h=False, need_act8=True)
    assert only8.h is None and torch.equal(only8.act8.codes, b.codes) and torch.equal(only8.act8.scale, b.scale)
    again = qlora.linear_gated_fwd(*a)
    assert all(torch.equal(getattr(again, k), getattr(out, k)) for k in ("h", "gate", "up", "u"))


@gpu
@pytest.mark.parametrize("T,K,N,r", [(1, 4096, 11008, 16), (20, 4096, 11008, 16), (33, 4096, 11008, 64), (64, 8192, 2816, 16),
                                     (128, 4096, 11008, 8), (509, 4096, 11008, 64), (2048, 4096, 11008, 64),
                                     (2047, 4096, 11008, 16), (1500, 8192, 22016, 64)])
def test_block_of_the_7b_and_65b_mlp(T, K, N, r):
    torch = torch_mod()
    announce(f"gated block T={T} K={K} N={N} r={r}")
    p = _block(T, K, N, r, T, dq=T != 509)
    out = qlora.linear_gated_fwd(p["x"], p["qs"], p["A"], p["Bs"], p["scale"], need_act8=True)
    torch.cuda.synchronize()
    b = qlora.act8_write(out.h)
    assert torch.equal(out.act8.codes, b.codes) and torch.equal(out.act8.scale, b.scale)
    keep = slice(0, None, max(1, T // 64))  # rows are independent of each other
    few = dict(p, x=p["x"][keep].contiguous())
    _check_block(few, qlora.Gated(out.h[keep], None, out.gate[keep], out.up[keep], out.u[keep]), "silu")
    last = dict(p, x=p["x"][-40:].contiguous())
    _check_block(last, qlora.Gated(out.h[-40:], None, out.gate[-40:], out.up[-40:], out.u[-40:]), "silu")


# where the weights are decoded first: whole rounds of tiles, and a last one in ranges of K; ranks with and without
# padding, output tiles that end inside, one step of K
DECODED = [(4096, 64, 5568, 32), (1500, 256, 8256, 7), (2049, 320, 5568, 100), (5000, 256, 2752, 64),
           (3000, 1024, 5568, 31), (4096, 1024, 4160, 16), (2049, 2048, 4160, 200)]


@gpu
@pytest.mark.parametrize("T,K,N,r", DECODED)
def test_block_of_decoded_weights(T, K, N, r):
    announce(f"gated block of decoded weights T={T} K={K} N={N} r={r}")
    assert qlora.linear_gated_workspace_bytes(T, N, K, r) > 4 * N * K
    test_block(T, K, N, r)


@gpu
@pytest.mark.parametrize("T,K,N", [(5, 256, 320), (40, 256, 320), (100, 256, 320), (300, 256, 320), (4096, 64, 5568),
                                   (3000, 1024, 5568)])
def test_block_rows_and_members_do_not_mix(T, K, N):
    """A NaN or Inf in one token stays in its row, and a row of zeros is 0."""
    torch = torch_mod()
    announce(f"gated block special values T={T}")
    p = _block(T, K, N, 8, T)
    args = (p["qs"], p["A"], p["Bs"], p["scale"])
    base = qlora.linear_gated_fwd(p["x"], *args)
    x = p["x"].clone()
    x[1, 7], x[3] = float("nan"), 0
    out = qlora.linear_gated_fwd(x, *args, need_act8=True)
    rest = torch.ones(T, dtype=torch.bool)
    rest[[1, 3]] = False
    for k in ("h", "gate", "up", "u"):
        assert torch.equal(getattr(out, k)[rest], getattr(base, k)[rest])
        assert bool(getattr(out, k)[1].isnan().all()) and bool((getattr(out, k)[3] == 0).all())
    assert bool(out.act8.scale[1].isnan().all()) and bool((out.act8.codes[3] == 0).all())


@gpu
@pytest.mark.parametrize("T,K,N", [(1, 512, 704), (20, 512, 704), (64, 512, 704), (100, 512, 704), (300, 512, 704),
                                   (700, 512, 704), (4096, 64, 5568), (3000, 1024, 5568)])
def test_block_outputs_workspace_stream_and_graph(T, K, N):
    """Given outputs and workspace, rows behind the last one, a stream of its own, and a captured graph."""
    torch = torch_mod()
    announce(f"gated block graph T={T}")
    r = 16
    p = _block(T, K, N, r, T)
    args = (p["x"], p["qs"], p["A"], p["Bs"], p["scale"])
    want = qlora.linear_gated_fwd(*args, need_act8=True)
    torch.cuda.synchronize()
    bf = lambda n: torch.full((T + 2, n), 7.0, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    whole = {"h": bf(N), "gate": bf(N), "up": bf(N), "u_out": bf(2 * r)}
    codes, scale = torch.full((T + 2, N), 7, dtype=torch.int8, device="cuda"), torch.full((T + 2, N // 64), 7.0, device="cuda")
    out = {k: t[:T] for k, t in whole.items()}
    out["act8"] = qlora.Act8(codes[:T], scale[:T])
    need = qlora.linear_gated_workspace_bytes(T, N, K, r)
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN in every float
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    run = lambda **kw: qlora.linear_gated_fwd(*args, **out, workspace=ws[:need], **kw)  # noqa: E731

    def check():
        for k, t in whole.items():
            assert torch.equal(t[:T], getattr(want, k[0] if k == "u_out" else k)) and bool((t[T:] == 7).all())
        assert torch.equal(codes[:T], want.act8.codes) and bool((codes[T:] == 7).all())
        assert torch.equal(scale[:T], want.act8.scale) and bool((scale[T:] == 7).all())
        assert bool((ws[need:] == 0xFF).all())

    run(stream=side)
    side.synchronize()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(3):
        for t in out.values():
            (t.codes if isinstance(t, qlora.Act8) else t).zero_()
        ws[:need].fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        check()
        torch.zeros(1000, device="cuda").add_(1.0)


def test_refusals_of_the_binding():
    torch = torch_mod()
    t = torch.zeros(4, 128, dtype=torch.bfloat16)
    f, b = qlora.gated_act_fwd, qlora.gated_act_bwd
    for call, says in (
            (lambda: f(t, t, "relu"), "activation must be"), (lambda: f(t[0], t), "2-D"),
            (lambda: f(t[:, :100], t), "multiple of 64"), (lambda: f(t, t[:2]), "up must have shape"),
            (lambda: f(t.float(), t), "gate must be"), (lambda: f(t, t, need_h=False), "8-bit"),
            (lambda: f(t, t, h=t.float()), "h must be"), (lambda: f(t, t, act8=qlora.Act8.empty(2, 128, "cpu")), "act8 must hold"),
            (lambda: f(t, t), "on cpu"), (lambda: b(t, t, t, "swish"), "activation must be"),
            (lambda: b(t[:1], t, t), "dh must have shape"), (lambda: b(t, t, t, dgate=t[:2]), "dgate must have shape"),
            (lambda: b(t, t, t, dup=t.float()), "dup must be"), (lambda: b(t, t, t), "on cpu")):
        with pytest.raises(ValueError, match=says):
            call()

    class Dev:  # a packed weight that claims a CUDA device, so that each tensor check is reached
        type = "cuda"

        def __repr__(self):
            return "cuda:0"

    class Codes:
        device = Dev()

    weight = lambda n_out, n_in=64: qlora.NF4Weight(n_out, n_in, Codes(), None, None, None)  # noqa: E731
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    qs = [weight(128), weight(128)]

    def g(x=bf(5, 64), qs=qs, A=bf(16, 64), Bs=(bf(128, 8), bf(128, 8)), **kw):
        return qlora.linear_gated_fwd(x, qs, A, list(Bs), 0.5, **kw)

    for call, says in (
            (lambda: g(activation="gelu"), "activation must be"), (lambda: g(qs=qs[:1]), "the gate and the up weight"),
            (lambda: g(qs=[weight(128), weight(192)]), "up has n_out 192"), (lambda: g(qs=[weight(100), weight(100)]), "multiple of 64"),
            (lambda: g(qs=[weight(128), weight(128, 128)]), "member 1 has n_in"), (lambda: g(A=bf(15, 64)), "multiple of the 2"),
            (lambda: g(Bs=(bf(128, 8),)), "Bs must hold 2"), (lambda: g(Bs=(bf(128, 8), bf(128, 7))), r"Bs\[1\] must have shape"),
            (lambda: g(x=bf(5, 128)), "x must have shape"), (lambda: g(need_h=False), "8-bit"),
            (lambda: g(keep=False, gate=bf(5, 128)), "keep=True"), (lambda: g(gate=bf(5, 64)), "gate must have shape"),
            (lambda: g(up=bf(4, 128)), "up must have shape"), (lambda: g(u_out=bf(5, 8)), "u_out must have shape"),
            (lambda: g(h=bf(5, 64)), "h must have shape"), (lambda: g(act8=qlora.Act8.empty(5, 64, "cpu")), "act8 must hold 5 x 128"),
            (lambda: g(), "x must be on cuda:0, not cpu")):
        with pytest.raises(ValueError, match=says):
            call()


def test_refusals_of_the_c_abi():
    lib = qlora.lib()
    fake = 1 << 20  # 16-byte aligned, never dereferenced: every call is refused before a launch
    a8 = lambda T=4, K=128, c=fake, s=fake: ctypes.byref(qlora.Act8Struct(T, K, c, s))  # noqa: E731

    def fwd(g=fake, u=fake, T=4, N=128, act=0, h=fake, h8=None):
        return lib.qlora_gated_act_fwd(g, u, T, N, act, h, h8, None)

    def bwd(d=fake, g=fake, u=fake, T=4, N=128, act=1, dg=fake, du=fake):
        return lib.qlora_gated_act_bwd(d, g, u, T, N, act, dg, du, None)

    weight = lambda n=128, k=256, flags=0: qlora.NF4WeightStruct(n, k, fake, fake, fake, fake, flags)  # noqa: E731

    def block(x=fake, T=4, q=None, A=fake, B=(fake, fake), r=8, scale=1.0, act=0, h=fake, h8=None, gate=None, up=None, u=None,
              ws=fake, n=1 << 40):
        q = (qlora.NF4WeightStruct * 2)(*(q or (weight(), weight())))
        return lib.qlora_linear_gated_fwd(x, T, q, A, (ctypes.c_void_p * 2)(*B), r, scale, act, h, h8, gate, up, u, ws, n, None)

    for call in (fwd, bwd):
        for T, N in ((0, 128), (-1, 128), (4, 0), (4, 96), (1 << 32, 64), (1 << 62, 1 << 62)):
            assert call(T=T, N=N) == 2
        assert call(act=2) == 8 and call(act=-1) == 8 and call(g=None) == 1 and call(u=fake + 2) == 3
    assert fwd(h=None) == 1 and fwd(h=fake + 8) == 3 and fwd(h8=a8(T=3)) == 2 and fwd(h8=a8(c=None)) == 1
    assert fwd(h8=a8(s=fake + 4)) == 3 and bwd(d=None) == 1 and bwd(dg=None) == 1 and bwd(du=fake + 2) == 3
    for T in (0, -1, 1 << 38):
        assert block(T=T) == 2
    for r in (0, -1, 257):
        assert block(r=r) == 2
    for q in ((weight(128), weight(192)), (weight(96), weight(96)), (weight(k=96), weight(k=96)), (weight(k=256), weight(k=128)),
              (weight(n=1 << 22), weight(n=1 << 22)), (weight(k=1 << 22), weight(k=1 << 22)), (weight(0), weight(0))):
        assert block(q=q) == 2
    assert block(q=(weight(), weight(flags=1))) == 8 and block(q=(weight(flags=2), weight(flags=2))) == 8
    assert block(scale=float("nan")) == 8 and block(act=7) == 8
    assert block(x=None) == 1 and block(A=None) == 1 and block(B=(fake, None)) == 1 and block(h=None) == 1 and block(ws=None) == 1
    assert block(gate=fake) == 1 and block(up=fake) == 1 and block(h8=a8(c=None)) == 1
    assert block(h8=a8(K=64)) == 2 and block(h8=a8(s=fake + 8)) == 3
    for name in ("x", "A", "h", "u", "ws"):
        assert block(**{name: fake + 2}) == 3
    assert block(gate=fake, up=fake + 8) == 3 and block(gate=fake + 8, up=fake) == 3 and block(B=(fake, fake + 2)) == 3
    need = lib.qlora_linear_gated_workspace_bytes(4, 128, 256, 8)
    assert need > 0 and block(n=need - 1) == 4
    for bad in ((0, 128, 256, 8), (4, 96, 256, 8), (4, 128, 100, 8), (4, 128, 256, 0), (4, 1 << 22, 256, 8), (4, 128, 1 << 22, 8)):
        assert lib.qlora_linear_gated_workspace_bytes(*bad) == 0
