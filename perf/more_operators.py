"""Cases that measure what stands around the linears in the MLP half of a decoder layer: the root-mean-square
norm with the residual's addition, and the gated product of the gate and up projections, each with its backward
pass.  ``run`` computes them in elementary torch operations, or (``own``) by the calls of
``bit_quantized_finetuning_quant_amd.qlora``; ``exact`` computes them in 64 bits."""

import math
from statistics import NormalDist

import torch

own = False

BLOCK = 64    # elements per NF4 block and per block of an 8-bit checkpoint
GROUP = 256   # NF4 block constants per FP8 group
EPS = 1e-5


# ------------------------------------------------------------------- cases
def _norm(name, T, D, residual=True, act8=False, weight="bf16"):
    return {"name": name, "op": "norm", "T": T, "D": D, "residual": residual, "act8": act8, "weight": weight}


def _norm_bwd(name, T, D, residual=True, grad_weight=False, weight="bf16"):
    return {"name": name, "op": "norm_bwd", "T": T, "D": D, "residual": residual, "grad_weight": grad_weight,
            "weight": weight}


def _gated(name, T, K, N, r, keep=True, weight="dq", act="silu"):
    return {"name": name, "op": "gated", "T": T, "K": K, "N": N, "r": r, "keep": keep, "weight": weight, "act": act}


def _act(name, T, N, bwd, act8=False, act="silu"):
    return {"name": name, "op": "act_bwd" if bwd else "act", "T": T, "N": N, "act8": act8, "act": act}


def listed():
    return [
        # the norm before the MLP for one served token of the 7B width: latency
        _norm("norm 1x4096", 1, 4096),
        # a training batch of 4 x 512 tokens, 7B width
        _norm("norm 2048x4096", 2048, 4096),
        # the 65B workload of 8 x 512, the norm's result kept in 8 bits for the projections' backward pass
        _norm("norm 4096x8192 act8", 4096, 8192, act8=True),
        # a ragged batch's backward pass, 7B width, with the gradient of the residual path
        _norm_bwd("norm bwd 2047x4096", 2047, 4096),
        # the 65B workload's backward pass where the norm's weight is trained too
        _norm_bwd("norm bwd 4096x8192 gw", 4096, 8192, grad_weight=True, weight="fp32"),
        # gate, up and their product for one served token of the 7B MLP: nothing kept
        _gated("gated 1x4096x11008", 1, 4096, 11008, 16, keep=False),
        # 33 requests served together
        _gated("gated 33x4096x11008", 33, 4096, 11008, 16, keep=False),
        # a short ragged training batch on fp32 block constants, the gate by GELU
        _gated("gated 509x4096x11008", 509, 4096, 11008, 64, weight="fp32", act="gelu_tanh"),
        # a training batch of 4 x 512 tokens through the 7B MLP
        _gated("gated 2048x4096x11008", 2048, 4096, 11008, 64),
        # the 65B workload of 8 x 512
        _gated("gated 4096x8192x22016", 4096, 8192, 22016, 64),
        # the product formed again in the backward pass, in 8 bits, behind projections with dropout
        _act("act 2048x11008 act8", 2048, 11008, False, act8=True),
        # the gradients of gate and up, the 65B workload
        _act("act bwd 4096x22016", 4096, 22016, True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "gated", "gated", "act", "act_bwd"])
    T = _log_int(rng, 1, 4096)
    weight = rng.choice(["bf16", "fp32"])
    act = rng.choice(["silu", "silu", "gelu_tanh"])
    if op == "norm":
        c = _norm("", T, 64 * _log_int(rng, 1, 128), residual=rng.random() < 0.7, act8=rng.random() < 0.4, weight=weight)
    elif op == "norm_bwd":
        c = _norm_bwd("", T, 64 * _log_int(rng, 1, 128), residual=rng.random() < 0.7, grad_weight=rng.random() < 0.5,
                      weight=weight)
    elif op == "gated":
        while True:
            T, K, N = _log_int(rng, 1, 4096), 64 * _log_int(rng, 1, 128), 64 * _log_int(rng, 1, 344)
            if T * K * N <= 4096 * 8192 * 22016 // 2:
                break
        c = _gated("", T, K, N, rng.choice([1, 7, 8, 16, 32, 64, 100, 128]), keep=rng.random() < 0.6,
                   weight=rng.choice(["dq", "fp32"]), act=act)
    else:
        bwd = op == "act_bwd"
        c = _act("", T, 64 * _log_int(rng, 1, 344), bwd, act8=not bwd and rng.random() < 0.5, act=act)
    del c["name"]
    return c


def work(case):
    op, T = case["op"], case["T"]
    if op in ("norm", "norm_bwd"):
        n, wide = T * case["D"], 2 if case["weight"] == "bf16" else 4
        if op == "norm":
            # x in and y out; the residual in and the sum out; the codes out and read back, their values out
            moved = 4 + (4 if case["residual"] else 0) + (2 * (1 + 4 / BLOCK) + 2 if case["act8"] else 0)
            return {"bytes": n * moved + case["D"] * wide, "flops": n * (12 if case["act8"] else 6)}
        moved = 6 + (2 if case["residual"] else 0)
        return {"bytes": n * moved + case["D"] * (wide + (4 if case["grad_weight"] else 0)), "flops": n * 11}
    if op == "gated":
        K, N, r = case["K"], case["N"], case["r"]
        packed = 0.515869 if case["weight"] == "dq" else 0.5625
        moved = 2 * N * K * packed + T * K * 2 + 2 * r * (K + N) * 2 + T * N * 2
        moved += T * (N * 4 + 2 * r * 2) if case["keep"] else 0
        return {"bytes": moved, "flops": 4 * T * N * K + 4 * T * r * (K + N) + 8 * T * N}
    n = T * case["N"]
    if op == "act":
        return {"bytes": n * (6 + (2 * (1 + 4 / BLOCK) + 2 if case["act8"] else 0)), "flops": n * 12}
    return {"bytes": n * 10, "flops": n * 12}


# --------------------------------------------------------------- packed data
def _levels(device):
    """The 16 NF4 levels: normal quantiles at equal steps, 7 below an exact zero and 8 above."""
    q = NormalDist().inv_cdf
    delta = 1 - 0.5 * (1 / 32 + 1 / 30)
    top = q(delta)
    low = [-q(0.5 + j * (delta - 0.5) / 7) / top for j in range(7, 0, -1)]
    high = [q(0.5 + j * (delta - 0.5) / 8) / top for j in range(1, 9)]
    return torch.tensor([-1.0] + low[1:] + [0.0] + high[:7] + [1.0], dtype=torch.float64, device=device).float()


def _pack(w, double_quant=True):
    """[N x K] fp32 -> (codes, constants): NF4 in blocks of 64, the constants in FP8 groups of 256 or fp32."""
    lv = _levels(w.device)
    flat = w.reshape(-1, BLOCK)
    c1 = flat.abs().amax(1)
    code = torch.bucketize(flat / c1.clamp_min(1e-30)[:, None], (lv[1:] + lv[:-1]) / 2).to(torch.uint8).view(-1)
    codes = code[0::2] | (code[1::2] << 4)
    if not double_quant:
        return {"codes": codes, "fp8": None, "s2": c1, "mu": None}
    mu = c1.double().mean().float().view(1)
    d = torch.nn.functional.pad(c1 - mu, (0, -c1.numel() % GROUP)).view(-1, GROUP)
    s2 = d.abs().amax(1) / 448
    fp8 = (d / s2.clamp_min(1e-30)[:, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(-1)[: c1.numel()]
    return {"codes": codes, "fp8": fp8.contiguous(), "s2": s2, "mu": mu}


def _unpack(p, N, K):
    """The bf16 values that a packed weight stands for, as fp32 [N x K]."""
    code = torch.stack([p["codes"] & 15, p["codes"] >> 4], 1).view(-1).long()
    c1 = p["s2"]
    if p["fp8"] is not None:
        c1 = p["fp8"].view(torch.float8_e4m3fn).float() * p["s2"].repeat_interleave(GROUP)[: p["fp8"].numel()] + p["mu"]
    v = _levels(code.device)[code] * c1.repeat_interleave(BLOCK)
    return v.view(N, K).bfloat16().float()


def _kept8(y):
    """The bf16 values that an 8-bit checkpoint of bf16 y stands for: absmax / 127 per 64 columns, the code nearest to
    the exact quotient, ties to the even one (64 bits: the quotient of a tie is exact in them)."""
    b = y.double().view(y.shape[0], -1, BLOCK)
    top = b.abs().amax(2, keepdim=True)
    code = torch.round(127 * b / torch.where(top > 0, top, 1.0))
    return (code.float() * (top / 127).float()).view(y.shape).bfloat16()


# ----------------------------------------------------------------- prepare
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    s = {"case": case}
    op, T = case["op"], case["T"]
    if op in ("norm", "norm_bwd"):
        D = case["D"]
        # a residual stream: a few channels 20 times larger; the branch that is added to it is smaller
        big = torch.where(torch.rand(D, generator=gen, device=dev) < 0.005, 20.0, 1.0)
        s["w"] = 1 + 0.2 * normal(D)
        if case["weight"] == "bf16":
            s["w"] = s["w"].bfloat16()
        if op == "norm":
            s["x"] = (normal(T, D) * (0.5 if case["residual"] else big)).bfloat16()
            s["res"] = (normal(T, D) * big).bfloat16() if case["residual"] else None
        else:
            s["s"] = (normal(T, D) * big).bfloat16()
            s["dy"] = (normal(T, D) * 1e-3).bfloat16()
            s["dres"] = (normal(T, D) * 1e-3).bfloat16() if case["residual"] else None
    elif op == "gated":
        K, N, r = case["K"], case["N"], case["r"]
        s["x"] = normal(T, K).bfloat16()
        # weights that keep the projections near unit variance at every width
        s["w"] = [_pack(normal(N, K) * K**-0.5, case["weight"] == "dq") for _ in range(2)]
        s["A"] = (normal(2 * r, K) * 0.01).bfloat16()
        s["B"] = [(normal(N, r) * 0.01).bfloat16() for _ in range(2)]
        s["scale"] = 16.0 / r
    else:
        N = case["N"]
        s["gate"], s["up"] = (normal(T, N) * 1.5).bfloat16(), normal(T, N).bfloat16()
        if op == "act_bwd":
            s["dh"] = (normal(T, N) * 1e-3).bfloat16()
    return s


# --------------------------------------------------------------------- run
def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    from bit_quantized_finetuning_quant_amd import qlora

    c = s["case"]
    if c["op"] == "norm":
        y, total, a = qlora.rms_norm_fwd(s["x"], s["w"], EPS, residual=s["res"], need_act8=c["act8"])
        out = {"y": y, "s": total} if c["residual"] else {"y": y}
        if c["act8"]:
            out["kept"] = qlora.act8_read(a)
        return out
    if c["op"] == "norm_bwd":
        gs, gw = qlora.rms_norm_bwd(s["dy"], s["s"], s["w"], EPS, dres=s["dres"], need_grad_weight=c["grad_weight"])
        return {"grad_s": gs, "grad_weight": gw} if c["grad_weight"] else {"grad_s": gs}
    if c["op"] == "gated":
        ws = [qlora.NF4Weight(c["N"], c["K"], p["codes"], p["fp8"], p["s2"], p["mu"], p["fp8"] is not None)
              for p in s["w"]]
        g = qlora.linear_gated_fwd(s["x"], ws, s["A"], s["B"], s["scale"], activation=c["act"], keep=c["keep"])
        return {"h": g.h, "gate": g.gate, "up": g.up, "u": g.u} if c["keep"] else {"h": g.h}
    if c["op"] == "act":
        h, a = qlora.gated_act_fwd(s["gate"], s["up"], activation=c["act"], need_act8=c["act8"])
        return {"h": h, "kept": qlora.act8_read(a)} if c["act8"] else {"h": h}
    dgate, dup = qlora.gated_act_bwd(s["dh"], s["gate"], s["up"], activation=c["act"])
    return {"dgate": dgate, "dup": dup}


def _sigmoid_of(act, g):
    """sigma such that act(g) = g sigma, and the derivative of sigma's argument."""
    if act == "silu":
        return torch.sigmoid(g), torch.ones_like(g)
    c = 2 * math.sqrt(2 / math.pi)
    return torch.sigmoid(c * (g + 0.044715 * g * g * g)), c * (1 + 0.134145 * g * g)


def _plain(s):
    c = s["case"]
    if c["op"] == "norm":
        w, x = s["w"].float(), s["x"].float()
        out = {}
        if c["residual"]:  # the sum is the residual stream's next value, held in bf16
            out["s"] = (x + s["res"].float()).bfloat16()
            x = out["s"].float()
        out["y"] = (w * (x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS))).bfloat16()
        if c["act8"]:
            out["kept"] = _kept8(out["y"])
        return out
    if c["op"] == "norm_bwd":
        w, x, dy = s["w"].float(), s["s"].float(), s["dy"].float()
        rstd = torch.rsqrt(x.square().mean(1, keepdim=True) + EPS)
        xhat, wdy = x * rstd, w * dy
        grad = rstd * (wdy - xhat * (wdy * xhat).mean(1, keepdim=True))
        if c["residual"]:
            grad = s["dres"].float() + grad
        out = {"grad_s": grad.bfloat16()}
        if c["grad_weight"]:
            out["grad_weight"] = (dy * xhat).sum(0)
        return out
    if c["op"] == "gated":
        x, r, k = s["x"].float(), c["r"], s["scale"]
        u = x @ s["A"].float().t()
        gate, up = (x @ _unpack(p, c["N"], c["K"]).t() + k * (u[:, i * r:(i + 1) * r] @ b.float().t())
                    for i, (p, b) in enumerate(zip(s["w"], s["B"])))
        out = {"h": (gate * _sigmoid_of(c["act"], gate)[0] * up).bfloat16()}
        if c["keep"]:
            out |= {"gate": gate.bfloat16(), "up": up.bfloat16(), "u": u.bfloat16()}
        return out
    g, up = s["gate"].float(), s["up"].float()
    sig, slope = _sigmoid_of(c["act"], g)
    if c["op"] == "act":
        h = (g * sig * up).bfloat16()
        return {"h": h, "kept": _kept8(h)} if c["act8"] else {"h": h}
    dh = s["dh"].float()
    return {"dgate": (dh * up * (sig + g * sig * (1 - sig) * slope)).bfloat16(), "dup": (dh * (g * sig)).bfloat16()}


# ------------------------------------------------------------------- exact
def _act_exact(act, g):
    """act and its derivative from their definitions, in 64 bits."""
    if act == "silu":
        e = torch.exp(-g.abs())
        low, high = e / (1 + e), 1 / (1 + e)  # the smaller and the larger of sigma(g), sigma(-g)
        s, t = torch.where(g < 0, low, high), torch.where(g < 0, high, low)
        return g * s, s + g * s * t
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (g + 0.044715 * g**3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * 0.044715 * g**2)


def _kept8_exact(y):
    b = y.bfloat16().double().reshape(-1, BLOCK)
    top = b.abs().amax(1, keepdim=True)
    q = torch.where(top > 0, torch.round(b * 127 / top), 0.0)
    return (q * (top / 127).float().double()).float().reshape(y.shape).bfloat16()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        w, x, out = s["w"].double(), s["x"].double(), {}
        if case["residual"]:
            out["s"] = (s["x"].double() + s["res"].double()).bfloat16()
            x = out["s"].double()
        out["y"] = x / (x.pow(2).sum(1, keepdim=True) / case["D"] + EPS).sqrt() * w
        if case["act8"]:
            out["kept"] = _kept8_exact(out["y"])
        return out
    if op == "norm_bwd":
        w, x, dy, D = s["w"].double(), s["s"].double(), s["dy"].double(), case["D"]
        m = x.pow(2).sum(1, keepdim=True) / D + EPS
        g = dy * w / m.sqrt() - x * (dy * w * x).sum(1, keepdim=True) / (D * m**1.5)
        out = {"grad_s": g if s["dres"] is None else g + s["dres"].double()}
        if case["grad_weight"]:
            out["grad_weight"] = (dy * x / m.sqrt()).sum(0)
        return out
    if op == "gated":
        K, N, r = case["K"], case["N"], case["r"]
        x, A = s["x"].double(), s["A"].double()
        both, us = [], []
        for i in range(2):
            ui = torch.mm(x, A[i * r:(i + 1) * r].t())
            both.append(torch.mm(x, _unpack(s["w"][i], N, K).double().t()).add_(torch.mm(ui, s["B"][i].double().t()), alpha=s["scale"]))
            us.append(ui)
        out = {"h": _act_exact(case["act"], both[0])[0] * both[1]}
        if case["keep"]:
            out |= {"gate": both[0], "up": both[1], "u": torch.cat(us, 1)}
        return out
    g, up = s["gate"].double(), s["up"].double()
    value, slope = _act_exact(case["act"], g)
    if op == "act":
        h = value * up
        return {"h": h, "kept": _kept8_exact(h)} if case["act8"] else {"h": h}
    dh = s["dh"].double()
    return {"dgate": dh * up * slope, "dup": dh * value}
