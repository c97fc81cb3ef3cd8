"""Cases of the gated recurrence and of group normalisation, with their plain forms.

Gated recurrence ("scan"), per sequence and channel, with gate logits z and normaliser tau:
    a_t = sigmoid(z_t)^(1/tau),  u_t = x_t  (tied: (1 - a_t) x_t),  h_t = a_t h_{t-1} + u_t
A padded token leaves the state as it is, its output is zero and nothing of its row is read.

Group normalisation ("norm"), channels last, x [N, S, C] in G groups of channels:
    v = (x - mean) / sqrt(var + eps) * w + b   (center false: x / sqrt(mean(x^2) + eps) * w + b)
    y = act(v), or v * act(gate) with a gate;  statistics over the valid rows of one n and the
    channels of one group. Rows that are padding give zero.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # prompts of a 340M-shaped layer (8 x 2048 tokens, 4 heads x 512 channels); x and the gate
        # logits are halves of one projection
        {"name": "scan_prefill", "op": "scan", "dir": "fwd", "B": 8, "L": 2048, "D": 2048, "dtype": "bf16", "tau": 16.0,
         "bias": 0.0, "tied": False, "mask": "none", "state": False, "fused": True},
        # one long document read in parts, with long-memory gates and a state carried in and out
        {"name": "scan_long", "op": "scan", "dir": "fwd", "B": 1, "L": 32768, "D": 1024, "dtype": "bf16", "tau": 16.0,
         "bias": 3.0, "tied": True, "mask": "none", "state": True, "fused": False},
        # the smallest call: one short prompt of the tiny layer
        {"name": "scan_tiny", "op": "scan", "dir": "fwd", "B": 1, "L": 64, "D": 64, "dtype": "fp32", "tau": 16.0,
         "bias": 0.0, "tied": False, "mask": "none", "state": False, "fused": False},
        # a training step of the 340M-shaped layer on a right-padded batch
        {"name": "scan_train", "op": "scan", "dir": "train", "B": 8, "L": 2048, "D": 2048, "dtype": "bf16", "tau": 16.0,
         "bias": 0.0, "tied": False, "mask": "right", "state": False, "fused": True},
        # the wide layer (4 x 8192 tokens, 8 heads x 512 channels), plain sigmoid gates: the largest
        {"name": "scan_train_wide", "op": "scan", "dir": "train", "B": 4, "L": 8192, "D": 4096, "dtype": "fp16", "tau": 1.0,
         "bias": 3.0, "tied": True, "mask": "none", "state": False, "fused": False},
        # odd sizes in 32 bits, left padding, states with gradients
        {"name": "scan_train_odd", "op": "scan", "dir": "train", "B": 3, "L": 1001, "D": 333, "dtype": "fp32", "tau": 16.0,
         "bias": 1.0, "tied": True, "mask": "left", "state": True, "fused": False},
        # one token of one sequence, and of a full serving batch with finished sequences in it
        {"name": "step_one", "op": "scan", "dir": "step", "B": 1, "L": 1, "D": 2048, "dtype": "bf16", "tau": 16.0,
         "bias": 0.0, "tied": False, "mask": "none", "state": True, "fused": True},
        {"name": "step_batch", "op": "scan", "dir": "step", "B": 256, "L": 1, "D": 2048, "dtype": "bf16", "tau": 16.0,
         "bias": 3.0, "tied": True, "mask": "right", "state": True, "fused": True},
        # heads of 16384 tokens normalised one by one (4 heads x 512 channels) under an output gate
        {"name": "norm_heads", "op": "norm", "dir": "fwd", "N": 16384, "S": 1, "C": 2048, "G": 4, "dtype": "bf16",
         "act": "silu", "gate": True, "mask": "none", "center": False},
        {"name": "norm_heads_train", "op": "norm", "dir": "train", "N": 16384, "S": 1, "C": 2048, "G": 4, "dtype": "bf16",
         "act": "silu", "gate": True, "mask": "none", "center": True},
        # statistics over whole sequences of a padded batch, 32 groups of 32 channels
        {"name": "norm_rows_train", "op": "norm", "dir": "train", "N": 8, "S": 2048, "C": 1024, "G": 32, "dtype": "bf16",
         "act": "silu", "gate": False, "mask": "right", "center": True},
        # odd sizes in 32 bits
        {"name": "norm_odd", "op": "norm", "dir": "fwd", "N": 3, "S": 777, "C": 130, "G": 13, "dtype": "fp32",
         "act": "sigmoid", "gate": False, "mask": "none", "center": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    mask = rng.choice(["none", "none", "right", "left", "random"])
    if rng.random() < 0.55:
        way = rng.choice(["fwd", "train", "step"])
        D = _log(rng, 8, 4096)
        if rng.random() < 0.6:
            D = max(8, D // 8 * 8)
        c = {"op": "scan", "dir": way, "B": _log(rng, 1, 512 if way == "step" else 32), "L": 1, "D": D, "dtype": dtype,
             "tau": rng.choice([1.0, 8.0, 16.0]), "bias": rng.choice([0.0, 1.0, 3.0]), "tied": rng.random() < 0.5,
             "mask": mask, "state": way == "step" or rng.random() < 0.5, "fused": rng.random() < 0.5}
        if way != "step":
            c["L"] = _log(rng, 1, max(1, min(32768, 48_000_000 // (c["B"] * D))))
        return c
    G = _log(rng, 1, 32)
    if rng.random() < 0.5:  # one row a group
        S, width = 1, _log(rng, 8, max(8, 4096 // G))
        if rng.random() < 0.6:
            width = max(8, width // 8 * 8)
        N = _log(rng, 1, max(1, min(32768, 32_000_000 // (G * width))))
    else:
        width = _log(rng, 1, max(1, 2048 // G))
        N = _log(rng, 1, 16)
        few = max(2, -(-64 // width))  # fewer values in a group have no statistics worth the name
        S = _log(rng, few, max(few, min(16384, 24_000_000 // (N * G * width))))
    return {"op": "norm", "dir": rng.choice(["fwd", "train"]), "N": N, "S": S, "C": G * width, "G": G, "dtype": dtype,
            "act": rng.choice(["none", "silu", "sigmoid"]), "gate": rng.random() < 0.5, "mask": mask,
            "center": rng.random() < 0.7}


def _mask(kind, n, length, g, device):
    """Valid-token mask [n, length] (uint8, 1 = valid), or None."""
    if kind == "none":
        return None
    if length == 1:  # sequences that are done, rows that are padding
        return (torch.rand(n, 1, generator=g, device=device) < 0.8).to(torch.uint8)
    if kind == "random":
        return (torch.rand(n, length, generator=g, device=device) < 0.8).to(torch.uint8)
    pad = torch.randint(0, length // 2 + 1, (n, 1), generator=g, device=device)
    if n > 2:
        pad[n // 2] = length  # a sequence with nothing in it
    pos = torch.arange(length, device=device)[None, :]
    return (pos >= pad if kind == "left" else pos < length - pad).to(torch.uint8)


def prepare(case, seed):
    device = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=device).manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def normal(*shape, dtype=dt, mean=0.0, std=1.0):
        return (torch.randn(*shape, generator=g, device=device) * std + mean).to(dtype)

    s = dict(case)
    if case["op"] == "scan":
        B, L, D = case["B"], case["L"], case["D"]
        if case["fused"]:
            p = torch.randn(B, L, 2 * D, generator=g, device=device)
            p[..., D:] += case["bias"]
            p = p.to(dt)
            s["x"], s["z"] = p[..., :D], p[..., D:]
        else:
            s["x"], s["z"] = normal(B, L, D), normal(B, L, D, mean=case["bias"])
        s["h0"] = normal(B, D, dtype=torch.float32) if case["state"] else None
        s["M"] = _mask(case["mask"], B, L, g, device)
        if case["dir"] == "train":
            s["dh"] = normal(B, L, D)
            s["dlast"] = normal(B, D, dtype=torch.float32) if case["state"] else None
        if case["dir"] == "step":
            s["x"], s["z"], s["M"] = s["x"][:, 0], s["z"][:, 0], None if s["M"] is None else s["M"][:, 0].contiguous()
    else:
        N, S, C = case["N"], case["S"], case["C"]
        shape = (N, C) if S == 1 else (N, S, C)
        s["x"] = normal(*shape, mean=0.5, std=2.0)
        s["w"] = normal(C, dtype=torch.float32, mean=1.0, std=0.1)
        s["b"] = normal(C, dtype=torch.float32, std=0.1)
        s["g"] = normal(*shape) if case["gate"] else None
        M = _mask(case["mask"], N, S, g, device)
        s["M"] = None if M is None else M.view(shape[:-1])
        if case["dir"] == "train":
            s["dy"] = normal(*shape)
    return s


EPS = 1e-5


def run(s):
    if s["op"] == "scan":
        if s["dir"] == "step":
            return _step(s)
        return _scan(s)
    return _norm(s)


# ------------------------------------------------------------------ gated recurrence

def _gate(z, tau):
    """1 - a and (1 - sigmoid(z)) of a = sigmoid(z)^(1/tau), 32 bits."""
    z = z.float()
    e = torch.exp(-z.abs())
    y = -(torch.log1p(e) + (-z).clamp(min=0)) / tau
    return -torch.expm1(y), torch.where(z >= 0, e, torch.ones_like(e)) / (1 + e)


def _doubling(a, u):
    """All h_t = a_t h_{t-1} + u_t along dimension 1, from a zero state, in log2(L) passes."""
    step = 1
    while step < a.shape[1]:
        u = torch.cat([u[:, :step], torch.addcmul(u[:, step:], a[:, step:], u[:, :-step])], 1)
        a = torch.cat([a[:, :step], a[:, step:] * a[:, :-step]], 1)
        step *= 2
    return a, u


def _scan(s):
    if own:
        from scale_gated_linear_b200 import ops
        kw = dict(mask=s["M"], initial_state=s["h0"], gate_normalizer=s["tau"], tied=s["tied"])
        if s["dir"] == "fwd":
            return ops.gated_scan(s["x"], s["z"], **kw)
        h, last, saved = ops.gated_scan_forward(s["x"], s["z"], **kw)
        return h, last, ops.gated_scan_backward(s["dh"], s["dlast"], saved)
    x, z, M, h0, tied = s["x"].float(), s["z"], s["M"], s["h0"], s["tied"]
    c, down = _gate(z, s["tau"])
    u = c * x if tied else x
    if M is not None:
        valid = (M != 0)[..., None]
        c = torch.where(valid, c, torch.zeros_like(c))
        u = torch.where(valid, u, torch.zeros_like(u))
    a = 1 - c
    start = torch.zeros_like(u[:, 0]) if h0 is None else h0
    through, h = _doubling(a, u)
    h = torch.addcmul(h, through, start[:, None]) if h0 is not None else h
    del through
    last = h[:, -1].clone()
    out = (h if M is None else torch.where(valid, h, torch.zeros_like(h))).to(s["x"].dtype)
    if s["dir"] == "fwd":
        return out, last
    dh = s["dh"].float()
    if M is not None:
        dh = torch.where(valid, dh, torch.zeros_like(dh))
    if s["dlast"] is not None:
        dh = torch.cat([dh[:, :-1], (dh[:, -1] + s["dlast"])[:, None]], 1)
    # g_t = dh_t + a_{t+1} g_{t+1}, the same recurrence from the other end
    nxt = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1).flip(1)
    grad = _doubling(nxt, dh.flip(1))[1].flip(1)
    del nxt, dh
    dh0 = (a[:, 0] * grad[:, 0]) if h0 is not None else None
    before = torch.cat([start[:, None], h[:, :-1]], 1)
    if tied:
        before = before - x
    dz = grad * before * a * down / s["tau"]
    dx = c * grad if tied else grad
    if M is not None:
        dx = torch.where(valid, dx, torch.zeros_like(dx))
        dz = torch.where(valid, dz, torch.zeros_like(dz))
    return out, last, (dx.to(s["x"].dtype), dz.to(s["z"].dtype), dh0)


def _step(s):
    """One token: the state is updated in place, as a serving loop keeps it."""
    if own:
        from scale_gated_linear_b200 import ops
        return ops.gated_scan_step(s["x"], s["z"], s["h0"], mask=s["M"], gate_normalizer=s["tau"], tied=s["tied"]), s["h0"]
    x = s["x"].float()
    c, _ = _gate(s["z"], s["tau"])
    h = (1 - c) * s["h0"] + (c * x if s["tied"] else x)
    if s["M"] is None:
        return h.to(s["x"].dtype), s["h0"].copy_(h)
    valid = (s["M"] != 0)[:, None]
    new = torch.where(valid, h, s["h0"])
    return torch.where(valid, h, torch.zeros_like(h)).to(s["x"].dtype), s["h0"].copy_(new)


# ------------------------------------------------------------------ group normalisation

def _act(kind, v):
    """act(v) and its derivative."""
    if kind == "none":
        return v, torch.ones_like(v)
    sig = 1 / (1 + torch.exp(-v))
    if kind == "sigmoid":
        return sig, sig * (1 - sig)
    return v * sig, sig * (1 + v * (1 - sig))


def _norm(s):
    if own:
        from scale_gated_linear_b200 import ops
        kw = dict(weight=s["w"], bias=s["b"], gate=s["g"], mask=s["M"], activation=s["act"], center=s["center"], eps=EPS)
        if s["dir"] == "fwd":
            return ops.group_norm(s["x"], s["G"], **kw)
        y, saved = ops.group_norm_forward(s["x"], s["G"], **kw)
        return y, ops.group_norm_backward(s["dy"], saved)
    N, S, C, G = s["N"], s["S"], s["C"], s["G"]
    part = (N, S, G, C // G)
    x = s["x"].float().view(part)
    w, b = s["w"].view(G, -1), s["b"].view(G, -1)
    valid, count = None, float(S * (C // G))
    if s["M"] is not None:
        valid = (s["M"] != 0).view(N, S, 1, 1)
        x = torch.where(valid, x, torch.zeros_like(x))
        count = (valid.sum(1, keepdim=True) * (C // G)).clamp(min=1).float()

    def mean(t):
        return t.sum((1, 3), keepdim=True) / count

    if s["center"]:
        x = x - mean(x)
        if valid is not None:
            x = torch.where(valid, x, torch.zeros_like(x))
    rstd = 1 / torch.sqrt(mean(x * x) + EPS)
    xhat = x * rstd
    v = xhat * w + b
    gate = None if s["g"] is None else s["g"].float().view(part)
    f, df = _act(s["act"], v if gate is None else gate)
    y = f if gate is None else v * f

    def given(t, dtype):
        if valid is not None:
            t = torch.where(valid, t, torch.zeros_like(t))
        return t.to(dtype).view(s["x"].shape)

    y = given(y, s["x"].dtype)
    if s["dir"] == "fwd":
        return y
    dy = s["dy"].float().view(part)
    dv = dy * (df if gate is None else f)
    dgate = None if gate is None else given(dy * v * df, s["x"].dtype)
    if valid is not None:
        dv = torch.where(valid, dv, torch.zeros_like(dv))
    dw, db = (dv * xhat).sum((0, 1)).view(-1), dv.sum((0, 1)).view(-1)
    dxhat = dv * w
    dx = dxhat - xhat * mean(dxhat * xhat)
    if s["center"]:
        dx = dx - mean(dxhat)
    return y, (given(rstd * dx, s["x"].dtype), dw, db, dgate)


# ------------------------------------------------------------------ work and exact values

def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "scan":
        n, states = case["B"] * case["L"] * case["D"], case["B"] * case["D"] * 4
        tokens = 0 if case["mask"] == "none" else case["B"] * case["L"]
        carried = states * (2 if case["state"] else 1)
        if case["dir"] == "train":  # x, z, dh in; h, dx, dz out; states and their gradients
            return {"bytes": 6 * n * size + tokens + carried * (2 if case["state"] else 1), "flops": 30 * n}
        return {"bytes": 3 * n * size + tokens + carried, "flops": 12 * n}
    n = case["N"] * case["S"] * case["C"]
    tokens = 0 if case["mask"] == "none" else case["N"] * case["S"]
    gate = 1 if case["gate"] else 0
    if case["dir"] == "train":  # x, dy, gate in; y, dx, dgate out; weight, bias and their gradients
        return {"bytes": (4 + 2 * gate) * n * size + tokens + 16 * case["C"], "flops": 40 * n}
    return {"bytes": (2 + gate) * n * size + tokens + 8 * case["C"], "flops": 15 * n}


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_scan(s) if s["op"] == "scan" else _exact_norm(s)


def _exact_scan(s):
    """Token by token in 64 bits, and the adjoint recurrence token by token."""
    step = s["dir"] == "step"
    x, z = s["x"].double(), s["z"].double()
    if step:
        x, z = x[:, None], z[:, None]
    B, L, D = x.shape
    log_a = torch.where(z >= 0, -torch.log1p(torch.exp(-z.clamp(min=0))), z.clamp(max=0) - torch.log1p(torch.exp(z.clamp(max=0)))) / s["tau"]
    a = torch.exp(log_a)
    factor = -torch.expm1(log_a) if s["tied"] else torch.ones_like(a)
    slope = a / (s["tau"] * (1 + torch.exp(z)))  # da/dz
    keep = torch.ones(B, L, 1, dtype=torch.bool, device=x.device) if s["M"] is None else (s["M"] != 0).view(B, L, 1)
    a = torch.where(keep, a, 1.0)
    u = torch.where(keep, factor * x, 0.0)
    h = torch.zeros(B, D, dtype=torch.float64, device=x.device) if s["h0"] is None else s["h0"].double()
    states = torch.empty(L + 1, B, D, dtype=torch.float64, device=x.device)
    states[0] = h
    for t in range(L):
        torch.addcmul(u[:, t], a[:, t], states[t], out=states[t + 1])
    seen = states.transpose(0, 1)
    out, last = torch.where(keep, seen[:, 1:], 0.0), states[L].clone()
    if step:
        return out[:, 0], last
    if s["dir"] == "fwd":
        return out, last
    dh = torch.where(keep, s["dh"].double(), 0.0)
    grad = torch.empty(L, B, D, dtype=torch.float64, device=x.device)
    carry = torch.zeros_like(h) if s["dlast"] is None else s["dlast"].double()
    for t in range(L - 1, -1, -1):
        torch.add(dh[:, t], carry, out=grad[t])
        carry = a[:, t] * grad[t]
    grad = grad.transpose(0, 1)
    dx = torch.where(keep, grad * factor, 0.0)
    dz = torch.where(keep, grad * (seen[:, :-1] - (x if s["tied"] else 0.0)) * slope, 0.0)
    return out, last, (dx, dz, None if s["h0"] is None else carry)


def _exact_norm(s):
    """The definition in 64 bits; its gradients by automatic differentiation."""
    N, S, C, G = s["N"], s["S"], s["C"], s["G"]
    train = s["dir"] == "train"
    keep = torch.ones(N, S, dtype=torch.bool, device=s["x"].device) if s["M"] is None else (s["M"] != 0).view(N, S)
    w, b = (s[k].double().requires_grad_(train) for k in ("w", "b"))
    x = s["x"].double().requires_grad_(train)
    gate = None if s["g"] is None else s["g"].double().requires_grad_(train)
    rows = torch.where(keep[..., None], x.view(N, S, C), 0.0).view(N, S, G, C // G).permute(0, 2, 1, 3)
    inside = keep[:, None, :, None]
    n = (keep.sum(1).clamp(min=1) * (C // G)).view(N, 1, 1, 1)
    if s["center"]:
        rows = rows - rows.sum((2, 3), keepdim=True) / n
    var = torch.where(inside, rows * rows, 0.0).sum((2, 3), keepdim=True) / n
    v = (rows / torch.sqrt(var + EPS)).permute(0, 2, 1, 3).reshape(N, S, C) * w + b
    act = {"none": lambda t: t, "sigmoid": torch.sigmoid, "silu": lambda t: t * torch.sigmoid(t)}[s["act"]]
    y = act(v) if gate is None else v * act(gate.view(N, S, C))
    y = torch.where(keep[..., None], y, 0.0).view(s["x"].shape)
    if not train:
        return y
    wanted = [x, w, b] + ([] if gate is None else [gate])
    got = torch.autograd.grad(y, wanted, s["dy"].double())
    return y.detach(), (got[0], got[1], got[2], got[3] if gate is not None else None)
