"""The loss of a frozen head over its vocabulary with the gradient of the hidden states, against the
formula in 64 bits.

Tolerances.  A logit is an fp32 sum of D exact products: it is off by at most
delta = (D + 2) 2^-24 max_tv sum_d |h W|.  With p_y the target's probability,
  d loss   = (1 - p_y) 2 delta                 through the logits (loss depends on l_v - l_y only)
           + 2^-20 loss                        exp2 / log1p / sums: a few fp32 roundings, relative
           + 2^-21 (|lse| + |l_y|)             where loss > log 2: it is then formed as N ln 2 - l_y + log S
  d grad   = c [ (2^-8 + V 2^-24) sum_{v != y} p_v |W_v|            e in bf16, fp32 sums
           + (4 delta + 2^-19) (sum_{v != y} p_v |W_v| + (1 - p_y) |W_y|) ]
           + 2^-8 |grad|                       the result in bf16
bf16 has 8 significant bits: in [1, 2) its values are 2^-7 apart, so a rounding moves a value by up to
2^-8 of it.
"""

import ctypes
import math

import pytest

from bit_quantized_finetuning_quant_amd import qlora
from helpers import announce, torch_mod

gpu = pytest.mark.gpu


def _inputs(T, D, V, seed, std=0.02, masked=0.3):
    torch = torch_mod()
    g = torch.Generator().manual_seed(seed)
    h = torch.randn(T, D, generator=g).bfloat16()
    w = (torch.randn(V, D, generator=g) * std).bfloat16()
    y = torch.randint(0, V, (T,), generator=g)
    y[torch.rand(T, generator=g) < masked] = -100
    return h, w, y


def _reference(h, w, y, scale=1.0, weight=None):
    """loss, lse, grad in fp64 on h's device, and the tolerances of loss and grad."""
    torch = torch_mod()
    T, V, D = h.shape[0], w.shape[0], h.shape[1]
    h, w = h.double(), w.double()
    live = y >= 0
    hz = torch.where(live[:, None], h, torch.zeros_like(h))
    ys = y.clamp_min(0)
    logits = torch.mm(hz, w.t())
    delta = (D + 2) * 2.0**-24 * float(torch.mm(hz.abs(), w.abs().t()).max())
    logp = torch.log_softmax(logits, 1)
    p = logp.exp()
    rows = torch.arange(T, device=h.device)
    ly = logits[rows, ys]
    lse = torch.logsumexp(logits, 1)
    others = p.clone()
    others[rows, ys] = 0
    rest = others.sum(1)
    loss = -logp[rows, ys]
    loss = torch.where(rest < 0.5, -torch.log1p(-rest), loss)  # exact for a token the model is sure of
    c = torch.full((T,), float(scale), dtype=torch.float64, device=h.device)
    if weight is not None:
        c = c * weight.double()
    pw = torch.mm(others, w)
    pa = torch.mm(others, w.abs())
    grad = c[:, None] * (pw - rest[:, None] * w[ys])
    tol_loss = rest * 2 * delta + 2.0**-20 * loss + 2.0**-21 * torch.where(loss > math.log(2), lse.abs() + ly.abs(), 0.0)
    tol_lse = 2 * delta + 2.0**-20 * (lse.abs() + 1)
    tol_grad = c.abs()[:, None] * ((2.0**-8 + V * 2.0**-24) * pa
                                   + (4 * delta + 2.0**-19) * (pa + rest[:, None] * w[ys].abs())) + 2.0**-8 * grad.abs()
    z = torch.zeros_like(loss)
    return (torch.where(live, loss, z), torch.where(live, lse, z), torch.where(live[:, None], grad, torch.zeros_like(grad)),
            torch.where(live, tol_loss, z), torch.where(live, tol_lse, z),
            torch.where(live[:, None], tol_grad, torch.zeros_like(grad)))


def _close(got, want, tol, name):
    over = ((got.double() - want).abs() - tol - 1e-37).max()
    assert not got.isnan().any(), f"{name} has NaN"
    assert float(over) <= 0, (name, float(over), float((got.double() - want).abs().max()))


def _check(h, head, w, y, scale=1.0, weight=None, **kw):
    """head: what the call takes; w: the bf16 values it stands for.  All on the GPU."""
    torch = torch_mod()
    loss, lse, grad = qlora.head_loss(h, head, y, scale=scale, weight=weight, **kw)
    score, lse2, none = qlora.head_loss(h, head, y, need_grad=False)
    torch.cuda.synchronize()
    assert none is None
    r = _reference(h, w, y, scale, weight)
    _close(loss, r[0], r[3], "loss")
    _close(lse, r[1], r[4], "lse")
    _close(grad, r[2], r[5], "grad_h")
    _close(score, r[0], r[3], "loss alone")
    _close(lse2, r[1], r[4], "lse alone")
    return loss, lse, grad


SHAPES = [(1, 64, 1), (1, 64, 2), (1, 128, 300), (2, 64, 255), (3, 192, 257), (16, 256, 1000), (37, 320, 129),
          (63, 128, 700), (64, 448, 2049), (65, 64, 511), (129, 256, 1025), (255, 512, 3001), (257, 192, 4100),
          (300, 1088, 777), (513, 2112, 1281), (1000, 256, 9001),
          # up to 64 tokens: one to four tiles of 16, one to many chunks of words, steps shared unevenly by the waves
          (1, 4096, 32003), (5, 8192, 3000), (16, 64, 16385), (17, 1024, 8193), (32, 2048, 641), (33, 64, 100001),
          (48, 576, 4097), (64, 1088, 20001), (2, 65536, 300),
          # the 256 x 256 tiles: lists of tokens and folds inside the products or in kernels of their own, the
          # last column tile of 64, one and many splits of the contraction
          (400, 4096, 8190), (512, 4096, 8192), (513, 4096, 8192), (520, 4032, 8193), (300, 1024, 33000),
          (257, 4096, 17001), (512, 704, 31999), (1100, 512, 9000), (2050, 192, 9001), (1300, 320, 12345),
          (2048, 256, 8192), (700, 128, 70000), (2300, 64, 16390),
          (511, 64, 8192), (512, 128, 8193), (513, 64, 8192), (514, 128, 8193), (512, 192, 100), (70, 4096, 419)]


@gpu
@pytest.mark.parametrize("T,D,V", SHAPES)
def test_loss_and_gradient(T, D, V):
    announce(f"head loss T={T} D={D} V={V}")
    h, w, y = (t.cuda() for t in _inputs(T, D, V, seed=T + V, std=3 / math.sqrt(D)))
    _check(h, w, w, y, scale=1 / T)


@gpu
@pytest.mark.parametrize("T,D,V", [(2050, 128, 20011), (300, 64, 70001), (700, 4096, 33000)])
def test_several_pieces_of_the_vocabulary(T, D, V):
    """More words than one piece holds, and (the first) a last piece shorter than its splits."""
    announce(f"head loss in pieces T={T} D={D} V={V}")
    h, w, y = (t.cuda() for t in _inputs(T, D, V, seed=7, std=2 / math.sqrt(D)))
    _check(h, w, w, y, scale=0.5)


@gpu
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("T,D,V", [(100, 64, 1 << 20), (256, 64, (1 << 20) - 3), (40, 64, (1 << 20) + 77), (1, 128, 1100000),
                                   (64, 65536, 65600)])
def test_few_tokens_of_a_very_large_vocabulary(T, D, V, packed):
    """The streams in several pieces, of exponentials or of chunks' sums, and the tiles for a few tokens of more words
    than the streams take."""
    torch = torch_mod()
    announce(f"head loss of a very large vocabulary T={T} D={D} V={V} packed={packed}")
    h, _, y = (t.cuda() for t in _inputs(T, D, V if D < 1000 else 4, seed=26))
    w = torch.empty(V, D, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(26)
    for at in range(0, V, 1 << 16):
        part = w[at:at + (1 << 16)]
        part.copy_(torch.randn(part.shape, generator=g, device="cuda") * (2 / math.sqrt(D)))
    y[y >= 0] = torch.randint(0, V, (int((y >= 0).sum()),), generator=g, device="cuda")
    y[0] = V - 1
    q = qlora.quantize(w) if packed else w
    _check(h, q, qlora.dequantize(q) if packed else w, y, scale=0.5)


@gpu
@pytest.mark.parametrize("T,D,V", [(64, 65536, 65600), (200, 64, 1 << 20), (1030, 8192, 9001)])
def test_packed_pieces_with_fp32_constants(T, D, V):
    """Pieces of a packed head without double quantization: streams that decode the rows themselves and that read
    decoded ones, and the tiles."""
    announce(f"head loss of pieces with fp32 constants T={T} D={D} V={V}")
    h, w, y = (t.cuda() for t in _inputs(T, D, V, seed=33, std=1 / math.sqrt(D)))
    q = qlora.quantize(w, double_quant=False)
    _check(h, q, qlora.dequantize(q), y)


@gpu
@pytest.mark.parametrize("order", ["rising", "falling"])
def test_exponents_of_the_streams_pieces(order):
    """Logits that rise or fall by 120 over four pieces of the streams: the sums of the pieces before and the piece's
    own are brought to one exponent."""
    torch = torch_mod()
    T, D, V = 256, 64, 1 << 20
    announce(f"head loss, {order} logits over the pieces of the streams")
    h, w, y = (t.cuda() for t in _inputs(T, D, V, seed=27, std=0.05, masked=0.1))
    ramp = torch.linspace(-60, 60, V, device="cuda")
    h[:, 0] = 1.0
    w[:, 0] = (ramp if order == "rising" else ramp.flip(0)).bfloat16()
    y[::3] = V - 1
    y[1::3] = 5
    _check(h, w, w, y)


@gpu
def test_several_chunks_of_tokens():
    T, D, V = 16384 + 700, 64, 515
    announce(f"head loss in chunks T={T} D={D} V={V}")
    h, w, y = (t.cuda() for t in _inputs(T, D, V, seed=8, std=0.3))
    y[16384:16400] = -1
    _check(h, w, w, y, weight=torch_mod().rand(T, device="cuda"))
    ws = qlora.head_loss_workspace(T, V, D)
    for at in (5, T - 5):  # a bad target in either chunk is reported
        bad = y.clone()
        bad[at] = V
        qlora.head_loss(h, w, bad, workspace=ws)
        assert qlora.status_read(ws) == 8
    T = 16384 + 300  # a last chunk short enough for another form
    _check(h[:T].contiguous(), w, w, y[:T].contiguous())


@gpu
@pytest.mark.parametrize("double_quant", [True, False])
@pytest.mark.parametrize("T,D,V", [(1, 64, 5), (33, 256, 1000), (300, 320, 777), (2050, 128, 20011)])
def test_packed_head(T, D, V, double_quant):
    announce(f"packed head T={T} D={D} V={V} double_quant={double_quant}")
    h, w, y = (t.cuda() for t in _inputs(T, D, V, seed=9, std=2 / math.sqrt(D)))
    q = qlora.quantize(w, double_quant=double_quant)
    _check(h, q, qlora.dequantize(q), y, scale=0.25)


@gpu
@pytest.mark.parametrize("double_quant", [True, False])
@pytest.mark.parametrize("T,D,V", [(1, 128, 1), (1, 4096, 32003), (2, 64, 63), (5, 192, 65), (16, 1024, 8193),
                                   (17, 320, 4100), (32, 448, 20001), (48, 64, 100001), (64, 1088, 2049), (65, 1088, 2049)])
def test_packed_head_decoded_in_the_streams(T, D, V, double_quant):
    """Up to 64 tokens the rows are decoded inside the products: one to four tiles of tokens, a tile with fewer
    than 64 rows, waves with none, one and many steps."""
    announce(f"packed head, few tokens, T={T} D={D} V={V} double_quant={double_quant}")
    h, w, y = (t.cuda() for t in _inputs(T, D, V, seed=23, std=2 / math.sqrt(D)))
    q = qlora.quantize(w, double_quant=double_quant)
    _check(h, q, qlora.dequantize(q), y, scale=0.25)


@gpu
@pytest.mark.parametrize("T", [40, 70, 1030])
def test_packed_head_in_pieces_by_size(T):
    """V D above a piece's decoded bytes: pieces also without the gradient."""
    D, V = 8192, 9001
    announce(f"packed head in pieces T={T} D={D} V={V}")
    h, w, y = (t.cuda() for t in _inputs(T, D, V, seed=10, std=0.02))
    q = qlora.quantize(w)
    _check(h, q, qlora.dequantize(q), y)


@gpu
@pytest.mark.parametrize("T", [15, 40, 260, 600])
@pytest.mark.parametrize("order", ["rising", "falling", "far"])
def test_exponents_of_tiles_and_pieces(order, T):
    """Logits whose largest value moves by hundreds between the tiles and the pieces: what a tile
    holds is rescaled by up to 2^-255 and below."""
    torch = torch_mod()
    D, V = 64, 140003
    announce(f"head loss, {order} logits T={T}")
    h, w, y = (t.cuda() for t in _inputs(T, D, V, seed=11, std=0.05, masked=0.1))
    ramp = torch.linspace(0, 60, V, device="cuda")
    if order == "falling":
        ramp = ramp.flip(0)
    if order == "far":
        ids = torch.arange(V, device="cuda")
        ramp = torch.where(ids % 128 == 5, 600.0, -600.0) * (ids > 70000)
    h[:, 0] = 1.0
    w[:, 0] = ramp.bfloat16()
    y[::3] = V - 1 if order == "rising" else 3  # also tokens the model is sure of, and sure against
    _check(h, w, w, y)


@gpu
@pytest.mark.parametrize("T", [64, 130, 600])
def test_sure_tokens_keep_relative_precision(T):
    """Losses down to about 1e-8 (3000 words 26 below the target, at 20003 words 1e-7): loss = log1p(others / e_y)
    and 1 - p_y are formed without a difference."""
    torch = torch_mod()
    D, V = 256, 3000 if T < 550 else 20003  # streams, tiles
    announce(f"head loss of sure tokens T={T}")
    h, w, y = (t.cuda() for t in _inputs(T, D, V, seed=12, std=0.02, masked=0.0))
    lean = torch.linspace(5, 28, T, device="cuda")[:, None] / w[y].float().square().sum(1, keepdim=True)
    h = (lean * w[y].float()).bfloat16()
    loss, _, _ = _check(h, w, w, y)
    assert float(loss.min()) < 1e-6 and float(loss.min()) > 0


@gpu
@pytest.mark.parametrize("T", [20, 64, 600])
def test_tokens_without_loss(T):
    """Negative targets: zeros, whatever the rows hold; a call without any loss; all rows but one."""
    torch = torch_mod()
    D, V = 128, 900 if T < 550 else 20003  # streams, tiles
    announce(f"head loss with masked tokens T={T}")
    h, w, y = (t.cuda() for t in _inputs(T, D, V, seed=13, std=0.3, masked=0.5))
    y[T // 2:T - 5] = -1
    dirty = h.clone()
    dirty[y < 0] = float("nan")
    dirty[T // 2 + 1] = float("inf")
    a, b = _check(h, w, w, y), qlora.head_loss(dirty, w, y)
    for x, z in zip(a, b):
        assert torch.equal(x, z)
    none = torch.full((T,), -100, device="cuda")
    loss, lse, grad = qlora.head_loss(dirty, w, none)
    assert not loss.any() and not lse.any() and not grad.any()
    loss, lse, _ = qlora.head_loss(dirty, w, none, need_grad=False)
    assert not loss.any() and not lse.any()
    one = none.clone()
    one[-1] = 17
    _check(h, w, w, one)


@gpu
@pytest.mark.parametrize("T", [40, 70, 600])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), 3e38])
def test_values_past_the_range(value, T):
    """NaN, Inf or an overflow in one token's row: NaN for that token, the others as they were."""
    torch = torch_mod()
    D, V = 128, 1000 if T < 550 else 20003  # streams, tiles
    announce(f"head loss with {value} in a row T={T}")
    h, w, y = (t.cuda() for t in _inputs(T, D, V, seed=14, std=0.3, masked=0.0))
    want = qlora.head_loss(h, w, y)
    bad = h.clone()
    bad[33] = value
    got = qlora.head_loss(bad, w, y)
    for a, b in zip(got, want):
        assert a[33].isnan().all()
        keep = torch.arange(T, device="cuda") != 33
        assert torch.equal(a[keep], b[keep])


@gpu
@pytest.mark.parametrize("T", [63, 70, 600])
def test_target_past_the_vocabulary(T):
    torch = torch_mod()
    D, V = 128, 1000 if T < 550 else 20003  # streams, tiles
    announce(f"head loss with a target past the vocabulary T={T}")
    h, w, y = (t.cuda() for t in _inputs(T, D, V, seed=15, masked=0.2))
    ws = qlora.head_loss_workspace(T, V, D)
    want = qlora.head_loss(h, w, y, workspace=ws)
    assert qlora.status_read(ws) == 0
    bad = y.clone()
    bad[7], bad[60] = V, 2**40
    bad[8] = -2**40
    got = qlora.head_loss(h, w, bad, workspace=ws)
    assert qlora.status_read(ws) == 8
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[7] = keep[60] = keep[8] = False
    for a, b in zip(got, want):
        assert not a[8].any()
        assert a[7].isnan().all() and a[60].isnan().all()
        assert torch.equal(a[keep], b[keep])
    qlora.head_loss(h, w, y, workspace=ws)
    assert qlora.status_read(ws) == 0


@gpu
def test_gradient_against_differences():
    """(L(h + eps d) - L(h - eps d)) / 2 eps of the call's own weighted loss, along directions in which
    the steps are exact in bf16.  L is a sum of T fp32 losses of about 7, each off by at most the
    tolerance above (2 delta < 2^-13 here); eps = 2^-3 on entries of h that are multiples of 2^-4."""
    torch = torch_mod()
    T, D, V = 12, 64, 500
    announce("head loss gradient against differences")
    h, w, y = (t.cuda() for t in _inputs(T, D, V, seed=16, std=0.05, masked=0.2))
    h = (torch.round(h.float() * 8) / 8).clamp(-3, 3).bfloat16()
    weight = torch.rand(T, device="cuda") + 0.5
    _, _, grad = qlora.head_loss(h, w, y, weight=weight)
    eps = 2.0**-3
    total = lambda x: float((qlora.head_loss(x, w, y, need_grad=False)[0].double() * weight.double()).sum())  # noqa: E731
    for seed in range(3):
        d = (torch.randint(0, 2, (T, D), generator=torch.Generator().manual_seed(seed)) * 2 - 1).cuda().float()
        up, down = (h.float() + eps * d).bfloat16(), (h.float() - eps * d).bfloat16()
        assert torch.equal(up.float() - h.float(), eps * d)
        slope = (total(up) - total(down)) / (2 * eps)
        want = float((grad.double() * d.double()).sum())
        # third-order term: eps^2 / 6 times the third derivative along d, at most max|W d|^3 per token
        third = eps**2 / 6 * 12 * 1.5 * float((w.double() @ d[0].double()).abs().max()) ** 3
        assert abs(slope - want) <= third + 2.0**-8 * float((grad.double() * d.double()).abs().sum()) + 2.0**-9


@gpu
@pytest.mark.parametrize("T", [10, 300, 600])
def test_captured_call_replays_equal_eager(T):
    """Two captured calls share a workspace; replays after eager work equal the eager results."""
    torch = torch_mod()
    D, V = 256, 2000 if T < 550 else 20003  # streams, tiles
    announce(f"head loss under graph capture T={T}")
    h, w, y = (t.cuda() for t in _inputs(T, D, V, seed=17, std=0.2))
    ws = qlora.head_loss_workspace(T, V, D)
    out = [torch.empty(T, device="cuda"), torch.empty(T, device="cuda"),
           torch.empty(T, D, device="cuda", dtype=torch.bfloat16)]
    score = torch.empty(T, device="cuda")

    def step():
        qlora.head_loss(h, w, y, loss=out[0], lse=out[1], grad_h=out[2], workspace=ws)
        qlora.head_loss(h, w, y, loss=score, lse=torch_lse, need_grad=False, workspace=ws)

    torch_lse = torch.empty(T, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for rep in range(3):
        h2, _, y2 = _inputs(T, D, V, seed=30 + rep, masked=0.1 + 0.3 * rep)
        h.copy_(h2.cuda())
        y.copy_(y2.cuda())
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (*out, score)]
        torch.zeros(1000, device="cuda").add_(1.0)
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, (*out, score)):
            assert torch.equal(a, b), rep


@gpu
@pytest.mark.parametrize("T", [9, 500, 600])
def test_two_streams_at_once_and_repeats_are_identical(T):
    torch = torch_mod()
    D, V = 512, 6000 if T < 550 else 20003  # streams, tiles
    announce(f"head loss on two streams T={T}")
    h, w, y = (t.cuda() for t in _inputs(T, D, V, seed=18, std=0.1))
    want = qlora.head_loss(h, w, y)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append([qlora.head_loss(h, w, y) for _ in range(3)])
    torch.cuda.synchronize()
    for calls in got:
        for r in calls:
            for a, b in zip(r, want):
                assert torch.equal(a, b)


@gpu
@pytest.mark.parametrize("T", [9, 64, 511, 700])
@pytest.mark.parametrize("side", [False, True])
def test_views_of_per_token_vectors(T, side):
    """Next-token targets are labels[1:], eight bytes off a 16-byte boundary; weights, losses and lse may be views of
    longer buffers too.  The results are the aligned call's, and what lies beside the views stays as it was."""
    torch = torch_mod()
    D, V = 128, 900 if T < 550 else 20003
    announce(f"head loss of views T={T} side={side}")
    h, w, labels = (t.cuda() for t in _inputs(T + 1, D, V, seed=28, std=0.2))
    h = h[:T]
    weights = torch.rand(T + 3, device="cuda")
    want = qlora.head_loss(h, w, labels[1:].clone(), weight=weights[3:].clone())
    held = [torch.full((T + 5,), 7.0, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    stream = torch.cuda.Stream() if side else None
    got = qlora.head_loss(h, w, labels[1:], weight=weights[3:], loss=held[0][1:T + 1], lse=held[1][2:T + 2], stream=stream)
    torch.cuda.synchronize()
    assert got[0].data_ptr() == held[0].data_ptr() + 4 and got[1].data_ptr() == held[1].data_ptr() + 8
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    for t, at in zip(held, (1, 2)):
        assert (t[:at] == 7).all() and (t[at + T:] == 7).all()


@gpu
def test_captured_call_with_views():
    """The copies of views are part of a captured call: replays read the targets of the day."""
    torch = torch_mod()
    T, D, V = 300, 128, 900
    announce("head loss of views under graph capture")
    h, w, labels = (t.cuda() for t in _inputs(T + 1, D, V, seed=29, std=0.2))
    h = h[:T]
    held = torch.zeros(T + 1, device="cuda")
    ws = qlora.head_loss_workspace(T, V, D)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        qlora.head_loss(h, w, labels[1:], loss=held[1:], workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _, lse, grad = qlora.head_loss(h, w, labels[1:], loss=held[1:], workspace=ws)
    for rep in range(3):
        labels.copy_(_inputs(T + 1, D, V, seed=40 + rep)[2].cuda())
        g.replay()
        torch.cuda.synchronize()
        got = [held[1:].clone(), lse.clone(), grad.clone()]
        torch.zeros(1000, device="cuda").add_(1.0)
        want = qlora.head_loss(h, w, labels[1:])
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), rep


@gpu
def test_a_given_streams_memory_is_its_own():
    """What a call on another stream than the current one allocates lies in that stream's memory pool: the
    workspace is given back when the call returns, before the kernels have run."""
    torch = torch_mod()
    announce("head loss on a given stream")
    h, w, y = (t.cuda() for t in _inputs(40, 256, 3000, seed=21, std=0.1))
    want = qlora.head_loss(h, w, y)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = qlora.head_loss(h, w, y, stream=side)
    pools = [(s["address"], s["address"] + s["total_size"], s["stream"]) for s in torch.cuda.memory_snapshot()]
    for t in got:
        assert [p[2] for p in pools if p[0] <= t.data_ptr() < p[1]] == [side.cuda_stream]
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def _exact_inputs(T, D, V, seed, similar):
    """h and W of multiples of 2^-3 and 2^-5 below 16 and 2: every partial sum of a logit is a multiple of 2^-8 below
    2^14, so the logits are exact in fp32.  Token t leans by 20 to 60 logits to a word that is not its target and
    whose row is `similar` to the target's row (the cosine between them)."""
    torch = torch_mod()
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    w = torch.round(n(V, D) * 8).clamp(-63, 63) / 32
    order = torch.randperm(V, generator=g)
    wrong, y = order[:T], order[T:2 * T]
    w[wrong] = torch.round((similar * w[y] + (1 - similar**2) ** 0.5 * 0.25 * n(T, D)) * 32).clamp(-63, 63) / 32
    lean = torch.linspace(20, 60, T)[:, None] / w[wrong].square().sum(1, keepdim=True)
    h = (torch.round(lean * w[wrong] * 8) / 8).clamp(-15, 15)
    assert float((h.abs() @ w.abs().t()).max()) < 2**14
    y[3::7] = -100
    return h.bfloat16(), w.bfloat16(), y


@gpu
@pytest.mark.parametrize("similar", [0.0, 0.9])
@pytest.mark.parametrize("T,D,V", [(1, 256, 300), (16, 512, 5000), (30, 256, 4000), (64, 256, 9000), (200, 256, 3000),
                                   (300, 1024, 7000), (512, 512, 8192), (512, 256, 17000), (700, 256, 9001),
                                   (2050, 256, 33000)])
def test_sure_of_a_wrong_word(T, D, V, similar):
    """The gradient of a token that is sure of a word other than its target is c p (W_word - W_target), however
    much of it cancels where the two rows are alike: the weights of the words sum to what the target's row is
    subtracted with.  With e_v (1 + d_v) in place of e_v, |d_v| <= 2^-8, in the product AND in the sum, and
    x the p-weighted sum of d over v != y, the gradient is off by
      sum_{v != y} p_v (d_v - x) (W_v - W_y) / (1 + x),   |d_v - x| <= 2^-8 min(2 (1 - p_v), 1 + (1 - p_y)),
    then V 2^-24 of the absolute terms of the product and of the sum, 2^-19 for exp2 and the factors, and 2^-8 of
    the result for its own rounding.  (No term for the logits: they are exact here.)"""
    torch = torch_mod()
    announce(f"head loss sure of a wrong word T={T} D={D} V={V} similar={similar}")
    h, w, y = (t.cuda() for t in _exact_inputs(T, D, V, seed=T + V, similar=similar))
    _, _, grad = qlora.head_loss(h, w, y, scale=0.5)
    torch.cuda.synchronize()
    hd, wd = h.double(), w.double()
    live = torch.nonzero(y >= 0)[:, 0]
    for t in live.tolist()[::max(1, live.numel() // 60)]:
        p = torch.softmax(torch.mv(wd, hd[t]), 0)
        diff = wd - wd[y[t]]
        p[y[t]] = 0  # its own term: (p_y - p_y - (1 - p_y)) W_y is in the difference
        rest = float(p.sum())
        want = 0.5 * torch.mv(diff.t(), p)
        spread = p * torch.minimum(2 * (1 - p), torch.full_like(p, 1 + rest))
        tol = 0.5 * (2.0**-8 / (1 - 2.0**-8) * torch.mv(diff.abs().t(), spread)
                     + (V * 2.0**-24 + 2.0**-19) * (torch.mv(wd.abs().t(), p) + rest * wd[y[t]].abs())) + 2.0**-8 * want.abs()
        _close(grad[t], want, tol, f"grad_h of token {t}")


# ------------------------------------------------------------------- refusals (no GPU)
def _call(h=0x10000, T=4, w=0x20000, V=100, D=128, y=0x30000, weight=None, scale=1.0, loss=0x40000, lse=None,
          grad=0x50000, ws=0x60000, ws_bytes=0):
    return qlora.lib().qlora_head_loss(h, T, w, V, D, y, weight, scale, loss, lse, grad, ws, ws_bytes, None)


def test_refusals_before_any_launch():
    assert _call(h=None) == 1 and _call(w=None) == 1 and _call(y=None) == 1 and _call(loss=None) == 1
    assert _call(ws=None) == 1
    for bad in (dict(T=0), dict(T=-1), dict(V=0), dict(D=0), dict(D=100), dict(D=65600), dict(V=1 << 40),
                dict(T=1 << 40), dict(D=-64)):
        assert _call(**bad) == 2, bad
    for bad in ("h", "w", "y", "weight", "loss", "lse", "grad", "ws"):
        assert _call(**{bad: 0x70008}) == 3, bad
    assert _call(scale=float("nan")) == 8 and _call(scale=float("inf")) == 8
    need = qlora.head_loss_workspace_bytes(4, 100, 128)
    assert need > 0 and _call(ws_bytes=need - 1) == 4
    st = qlora.NF4WeightStruct(100, 100, 0x10000, 0x20000, 0x30000, 0x40000)
    L = qlora.lib()
    args = (0x30000, None, 1.0, 0x40000, None, None, 0x60000, 1 << 40, None)
    assert L.qlora_head_loss_nf4(0x10000, 4, ctypes.byref(st), *args) == 2  # D % 64
    assert L.qlora_head_loss_nf4(0x10000, 4, None, *args) == 1


def test_workspace_sizes():
    b = qlora.head_loss_workspace_bytes
    assert b(0, 100, 128) == 0 and b(4, 0, 128) == 0 and b(4, 100, 100) == 0
    assert b(2048, 32000, 4096, grad=False) < b(2048, 32000, 4096) < b(2048, 32000, 4096, packed=True)
    # bounded in V: the pieces do not grow with the vocabulary
    assert b(4096, 1 << 20, 4096) <= b(4096, 1 << 16, 4096) + (8 << 20)
    # and far below the fp32 logits
    assert b(16384, 128000, 4096) < 16384 * 128000 * 4 / 8
    assert b(1 << 20, 32000, 4096) == b(16384, 32000, 4096)


def test_workspace_limits():
    """The limits that the header states, over both forms: 128 MB of exponentials, 64 MB of exponents and sums, 128 MB
    of partial sums or fp32 sums of the tokens taken at a time where these are more, 128 MB of decoded rows, and up to
    forty bytes a token."""
    MB = 1 << 20
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    for T in (1, 16, 33, 64, 65, 128, 256, 300, 512, 513, 1000, 4096, 16384, 100000):
        for D in (64, 1024, 4096, 8192, 65536):
            for V in (1, 300, 32000, 131072, (1 << 20) - 1, 1 << 20, (1 << 20) + 1, 1 << 22, 1 << 31):
                if V * D > 1 << 37:
                    continue
                tokens = min(T, 16384)
                for grad in (False, True):
                    for packed in (False, True):
                        limit = 64 * MB + 40 * up(tokens) + 4096
                        if grad:
                            limit += 128 * MB + max(128 * MB, up(tokens) * up(D) * 4)
                        if packed:
                            limit += 128 * MB
                        got = qlora.head_loss_workspace_bytes(T, V, D, grad, packed)
                        assert 0 < got <= limit, (T, V, D, grad, packed, got / MB, limit / MB)


def test_tensor_checks():
    torch = torch_mod()
    h, w, y = _inputs(4, 128, 100, seed=1)
    with pytest.raises(ValueError, match="must be on"):
        qlora.head_loss(h, w, y)
    with pytest.raises(ValueError, match="target must be"):
        qlora.head_loss(h, w, y.int())
    with pytest.raises(ValueError, match="target must have shape"):
        qlora.head_loss(h, w, y[:3])
    with pytest.raises(ValueError, match="h must be"):
        qlora.head_loss(h.float(), w, y)
    with pytest.raises(ValueError, match="head must have shape"):
        qlora.head_loss(h, w[:, :64].contiguous(), y)
    with pytest.raises(ValueError, match="contiguous"):
        qlora.head_loss(h, torch.randn(128, 100).bfloat16().t(), y)
    with pytest.raises(ValueError, match="weight must be"):
        qlora.head_loss(h, w, y, weight=torch.ones(4).double())
    with pytest.raises(ValueError, match="2-D"):
        qlora.head_loss(h[0], w, y)
