"""Cases that measure the training-side operators around the QLoRA linear layer: the vocabulary loss
with the gradient of its hidden states, and the 8-bit activation checkpoint with the backward pass
that reads it.  ``run`` computes them in elementary torch operations, or (``own``) by the calls of
``bit_quantized_finetuning_quant_amd.qlora``; ``exact`` computes them in 64 bits."""

import math
from statistics import NormalDist

import torch

own = False

BLOCK = 64    # elements per NF4 block and per block of an 8-bit checkpoint
GROUP = 256   # NF4 block constants per FP8 group


# ------------------------------------------------------------------- cases
def _loss(name, T, D, V, head="bf16", train=True, masked="pad", weighted=False):
    return {"name": name, "op": "loss", "T": T, "D": D, "V": V, "head": head, "train": train, "masked": masked,
            "weighted": weighted}


def _act(name, T, K):
    return {"name": name, "op": "act", "T": T, "K": K}


def _bwd(name, T, N, K, members, r, head="dq"):
    return {"name": name, "op": "bwd", "T": T, "N": N, "K": K, "members": members, "r": r, "weight": head}


def listed():
    return [
        # the loss of a toy model's training step (the tests' width): launches and latency
        _loss("loss 16x256 V1000", 16, 256, 1000),
        # the log-probability of one served token under the 7B width's head
        _loss("score 1x4096 V32000", 1, 4096, 32000, train=False, masked="none"),
        # one training sequence with padding, 7B width
        _loss("loss 512x4096 V32000", 512, 4096, 32000),
        # a batch of 4 sequences whose prompts (two fifths) carry no loss, weighted per token
        _loss("loss 2048x4096 V32000 sft", 2048, 4096, 32000, masked="prompt", weighted=True),
        # a ragged batch on a packed 4-bit head with three added words
        _loss("loss 2047x4096 V32003 nf4", 2047, 4096, 32003, head="nf4", masked="none"),
        # held-out perplexity of the same batch over an odd, larger vocabulary
        _loss("score 2048x4096 V50001", 2048, 4096, 50001, train=False),
        # the 65B workload: 8 sequences of 512 with padding
        _loss("loss 4096x8192 V32000", 4096, 8192, 32000),
        # one token's activation, written and read back: latency
        _act("act 1x4096", 1, 4096),
        # one 7B projection's input at batch 4 x 512
        _act("act 2048x4096", 2048, 4096),
        # the 65B down projection's input at 8 x 512
        _act("act 4096x22016", 4096, 22016),
        # one 7B projection's backward pass from its checkpoint
        _bwd("bwd 2048x4096 r64", 2048, 4096, 4096, 1, 64),
        # q, k, v of a 7B layer from their shared checkpoint, a ragged short batch
        _bwd("bwd qkv 509x4096 r16", 509, 4096, 4096, 3, 16),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["loss", "loss", "loss", "act", "bwd", "bwd"])
    if op == "loss":
        while True:
            T, D, V = _log_int(rng, 1, 4096), 64 * _log_int(rng, 2, 128), _log_int(rng, 300, 60000)
            if T * D * V <= 4096 * 8192 * 32000 and V * D <= 32000 * 8192:
                break
        c = _loss("", T, D, V, head=rng.choice(["bf16", "bf16", "nf4"]), train=rng.random() < 0.75,
                  masked=rng.choice(["none", "pad", "prompt"]), weighted=rng.random() < 0.3)
    elif op == "act":
        c = _act("", _log_int(rng, 1, 4096), 64 * _log_int(rng, 1, 344))
    else:
        c = _bwd("", _log_int(rng, 1, 4096), _log_int(rng, 64, 11008), 64 * _log_int(rng, 1, 128), rng.randint(1, 4),
                 rng.choice([1, 7, 8, 16, 32, 64, 100, 128]), head=rng.choice(["dq", "fp32"]))
    del c["name"]
    return c


def _prompt(T):
    return 2 * min(T, 512) // 5


def _masked_count(case):
    T = case["T"]
    if case["masked"] == "pad":       # the last 26 tokens of every 512 carry no loss
        return sum(max(0, min(T, s + 512) - max(s + 486, s)) for s in range(0, T, 512))
    if case["masked"] == "prompt":    # the first two fifths of every 512 are prompt
        return sum(min(T, s + _prompt(T)) - s for s in range(0, T, 512))
    return 0


def work(case):
    if case["op"] == "loss":
        T, D, V = case["T"], case["D"], case["V"]
        live = T - _masked_count(case)
        head = V * D * 2 if case["head"] == "bf16" else V * D * 0.515869
        per_token = D * (4 if case["train"] else 2) + 16 + (4 if case["weighted"] else 0)
        return {"bytes": head + T * per_token, "flops": (4 if case["train"] else 2) * live * V * D}
    if case["op"] == "act":
        T, K = case["T"], case["K"]
        return {"bytes": T * K * (2 + 2 + 2 * (1 + 4 / BLOCK)), "flops": T * K * 6}
    T, N, K, m, r = case["T"], case["N"], case["K"], case["members"], case["r"]
    packed = 0.515869 if case["weight"] == "dq" else 0.5625
    moved = m * (N * K * packed + T * N * 2 + N * r * 2 + T * r * 2 + N * r * 4)
    moved += T * K * (1 + 4 / BLOCK) + T * K * 2 + m * r * K * (2 + 4)
    return {"bytes": moved, "flops": m * (2 * T * N * K + 4 * T * r * (N + K))}


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
    n, lv = w.numel(), _levels(w.device)
    flat = torch.nn.functional.pad(w.reshape(-1), (0, -n % BLOCK)).view(-1, BLOCK)
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
    return v[: N * K].view(N, K).bfloat16().float()


def _encode8(x):
    """bf16 [T x K] -> (int8 codes, fp32 scales [T x K/64]): absmax / 127 per 64 columns, the code nearest to the
    exact quotient, ties to the even one (64 bits: the quotient of a tie is exact in them)."""
    b = x.double().view(x.shape[0], -1, BLOCK)
    top = b.abs().amax(2)
    code = torch.round(127 * b / torch.where(top > 0, top, 1.0)[..., None])
    return code.to(torch.int8).view(x.shape), (top / 127).float()


def _decode8(code, scale):
    """The bf16 values that a checkpoint stands for."""
    v = code.float().view(code.shape[0], -1, BLOCK) * scale[..., None]
    return v.view(code.shape).bfloat16()


# ----------------------------------------------------------------- prepare
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    uniform = lambda *s: torch.rand(*s, generator=gen, device=dev)  # noqa: E731
    s = {"case": case}
    T = case["T"]
    if case["op"] == "loss":
        D, V = case["D"], case["V"]
        w = normal(V, D) * 0.02
        y = torch.randint(0, V, (T,), generator=gen, device=dev)
        # hidden states of a model that has learnt something: each leans to its target by 0 to 14 logits
        lean = uniform(T, 1) * 14 / w[y].square().sum(1, keepdim=True)
        s["h"] = (normal(T, D) + lean * w[y]).bfloat16()
        at = torch.arange(T, device=dev) % 512
        if case["masked"] == "pad":
            y = torch.where(at >= 486, -100, y)
        elif case["masked"] == "prompt":
            y = torch.where(at < _prompt(T), -100, y)
        s["y"], s["scale"] = y, 1.0 / max(1, T - _masked_count(case))
        s["weight"] = uniform(T) + 0.5 if case["weighted"] else None
        s["head"] = w.bfloat16() if case["head"] == "bf16" else _pack(w)
    elif case["op"] == "act":
        # a residual stream: mostly normal, a few channels 20 times larger
        big = torch.where(uniform(case["K"]) < 0.005, 20.0, 1.0)
        s["x"] = (normal(T, case["K"]) * big).bfloat16()
    else:
        N, K, m, r = case["N"], case["K"], case["members"], case["r"]
        x = normal(T, K).bfloat16()
        s["codes"], s["scales"] = _encode8(x)
        s["w"] = [_pack(normal(N, K) * 0.02, case["weight"] == "dq") for _ in range(m)]
        s["A"] = (normal(m * r, K) * 0.01).bfloat16()
        s["B"] = [(normal(N, r) * 0.01).bfloat16() for _ in range(m)]
        s["dy"] = [normal(T, N).bfloat16() for _ in range(m)]
        s["u"] = (x.float() @ s["A"].float().t()).bfloat16()
        s["scale"] = 16.0 / r
    return s


# --------------------------------------------------------------------- run
def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    from bit_quantized_finetuning_quant_amd import qlora

    c = s["case"]
    packed = lambda p, N, K: qlora.NF4Weight(N, K, p["codes"], p["fp8"], p["s2"], p["mu"],  # noqa: E731
                                             p["fp8"] is not None)
    if c["op"] == "loss":
        head = s["head"] if c["head"] == "bf16" else packed(s["head"], c["V"], c["D"])
        loss, lse, grad = qlora.head_loss(s["h"], head, s["y"], scale=s["scale"], weight=s["weight"],
                                          need_grad=c["train"])
        return {"loss": loss, "lse": lse, "grad_h": grad} if c["train"] else {"loss": loss, "lse": lse}
    if c["op"] == "act":
        return qlora.act8_read(qlora.act8_write(s["x"]))
    a = qlora.Act8(s["codes"], s["scales"])
    ws = [packed(p, c["N"], c["K"]) for p in s["w"]]
    if c["members"] == 1:
        gx, ga, gb = qlora.linear_bwd_act8(s["dy"][0], a, ws[0], s["A"], s["B"][0], s["scale"], u=s["u"])
        return {"grad_x": gx, "grad_A": ga, "grad_B": [gb]}
    gx, ga, gb = qlora.linear_set_bwd_act8(s["dy"], a, ws, s["A"], s["B"], s["scale"], u=s["u"])
    return {"grad_x": gx, "grad_A": ga, "grad_B": gb}


def _plain(s):
    c = s["case"]
    if c["op"] == "loss":
        w = s["head"].float() if c["head"] == "bf16" else _unpack(s["head"], c["V"], c["D"])
        live = s["y"] >= 0
        y = s["y"].clamp_min(0)[:, None]
        logits = s["h"].float() @ w.t()
        top = logits.amax(1, keepdim=True)
        e = torch.exp(logits - top)
        total = e.sum(1, keepdim=True)
        lse = (top + torch.log(total))[:, 0]
        out = {"loss": torch.where(live, lse - logits.gather(1, y)[:, 0], 0.0), "lse": torch.where(live, lse, 0.0)}
        if c["train"]:
            p = e / total
            p.scatter_add_(1, y, torch.full_like(total, -1.0))
            factor = live * s["scale"] if s["weight"] is None else live * s["scale"] * s["weight"]
            out["grad_h"] = ((p * factor[:, None]) @ w).bfloat16()
        return out
    if c["op"] == "act":
        return _decode8(*_encode8(s["x"]))
    x = _decode8(s["codes"], s["scales"]).float()
    r, m = c["r"], c["members"]
    dy = [d.float() for d in s["dy"]]
    v = torch.cat([d @ b.float() for d, b in zip(dy, s["B"])], 1)
    gx = s["scale"] * (v @ s["A"].float()) + sum(d @ _unpack(p, c["N"], c["K"]) for d, p in zip(dy, s["w"]))
    ga = s["scale"] * (v.t() @ x)
    gb = [s["scale"] * (dy[i].t() @ s["u"][:, i * r:(i + 1) * r].float()) for i in range(m)]
    return {"grad_x": gx.bfloat16(), "grad_A": ga, "grad_B": gb}


# ------------------------------------------------------------------- exact
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "loss":
        w = s["head"] if case["head"] == "bf16" else _unpack(s["head"], case["V"], case["D"])
        w, h, y, T = w.double(), s["h"].double(), s["y"], case["T"]
        logits = torch.mm(h, w.t())
        logp = torch.log_softmax(logits, 1)
        rows = torch.nonzero(y >= 0)[:, 0]
        loss, lse = logits.new_zeros(T), logits.new_zeros(T)
        loss[rows] = -logp[rows, y[rows]]
        lse[rows] = torch.logsumexp(logits[rows], 1)
        out = {"loss": loss, "lse": lse}
        if case["train"]:
            grad = h.new_zeros(T, case["D"])
            g = logp[rows].exp()
            g[torch.arange(rows.numel(), device=g.device), y[rows]] -= 1
            scale = s["scale"] * (s["weight"].double()[rows] if s["weight"] is not None else torch.ones_like(lse[rows]))
            grad[rows] = torch.mm(g, w) * scale[:, None]
            out["grad_h"] = grad
        return out
    if case["op"] == "act":
        # what is stored: the nearest of 255 multiples of absmax / 127, in bf16
        b = s["x"].double().reshape(-1, BLOCK)
        top = b.abs().amax(1, keepdim=True)
        q = torch.where(top > 0, torch.round(b * 127 / top), 0.0)
        return (q * (top / 127).float().double()).float().reshape(s["x"].shape).bfloat16()
    T, r, m = case["T"], case["r"], case["members"]
    x = s["codes"].double().reshape(-1, BLOCK) * s["scales"].double().reshape(-1, 1)
    x = x.float().bfloat16().double().reshape(T, case["K"])
    A, u, k = s["A"].double(), s["u"].double(), s["scale"]
    gx, ga, gb = torch.zeros_like(x), [], []
    for i in range(m):
        dy, B, Ai = s["dy"][i].double(), s["B"][i].double(), A[i * r:(i + 1) * r]
        v = torch.mm(dy, B)
        gx += torch.mm(dy, _unpack(s["w"][i], case["N"], case["K"]).double()) + k * torch.mm(v, Ai)
        ga.append(k * torch.mm(v.t(), x))
        gb.append(k * torch.mm(dy.t(), u[:, i * r:(i + 1) * r]))
    return {"grad_x": gx, "grad_A": torch.cat(ga), "grad_B": gb}
