"""Two operators around gated linear attention, as measured cases.

The gated linear recurrence (one state value per channel, for every sequence)

    h_t = exp(log_alpha_t) h_{t-1} + x_t

forward, over packed batches, backward, and as a single decode step; and the
per-head norm of queries and keys with the rotation by position in the same
pass, forward and backward, which takes q and k token-major, as a projection
leaves them, and gives them head-first, as the attention kernels take them.

`run` computes either the plain form, in elementary torch operations, or the
framework's kernels (`own`).
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp32": 4}

# The most elements of a drawn scan, and of the q and k of a drawn norm: those of the largest
# listed cases of each kind.
MOST_SCAN = 262144 * 1024
MOST_SCAN_TRAIN = 8 * 2048 * 2048
MOST_QK = 2 * 32768 * 32 * 128
MOST_QK_TRAIN = 4 * 4096 * 40 * 64


def listed():
    return [
        # one decode token of a recurrent layer for a few streams: latency
        {"name": "scan_step_small", "op": "scan_step", "B": 8, "D": 2048, "dtype": "bf16"},
        # one decode token for many streams
        {"name": "scan_step_many", "op": "scan_step", "B": 256, "D": 4096, "dtype": "bf16"},
        # the prefill of a batch, 16 heads of 128 channels
        {"name": "scan_fwd_medium", "op": "scan_fwd", "B": 8, "T": 2048, "D": 2048,
         "dtype": "bf16", "h0": False},
        # one very long sequence, few channels
        {"name": "scan_fwd_very_long", "op": "scan_fwd", "B": 1, "T": 262144, "D": 1024,
         "dtype": "bf16", "h0": True},
        # a packed batch of 24 ragged sequences, empty and one-token ones among them
        {"name": "scan_packed", "op": "scan_packed", "N": 24, "T": 65536, "D": 1000,
         "dtype": "bf16", "h0": True},
        # a training step's pass through the recurrence: forward, then all gradients
        {"name": "scan_train_medium", "op": "scan_train", "B": 8, "T": 2048, "D": 2048,
         "dtype": "bf16", "h0": True},
        # the same in fp32 with an odd number of channels and a ragged length
        {"name": "scan_train_odd", "op": "scan_train", "B": 3, "T": 4097, "D": 515,
         "dtype": "fp32", "h0": True},
        # the token before a decode step, for a batch of streams at far positions
        {"name": "qk_decode", "op": "qk_fwd", "B": 256, "T": 1, "Hq": 32, "Hk": 32, "d": 128,
         "rot": 128, "norm": "rms", "weights": True, "interleaved": False, "fused": True,
         "positions": "far", "dtype": "bf16"},
        # the prefill of a batch from one fused projection
        {"name": "qk_prefill", "op": "qk_fwd", "B": 8, "T": 2048, "Hq": 16, "Hk": 16, "d": 128,
         "rot": 128, "norm": "rms", "weights": True, "interleaved": False, "fused": True,
         "positions": "count", "dtype": "bf16"},
        # keys and queries of unit length for the gated delta rule, no rotation, long
        {"name": "qk_unit_long", "op": "qk_fwd", "B": 2, "T": 32768, "Hq": 16, "Hk": 16,
         "d": 128, "rot": 0, "norm": "l2", "weights": False, "interleaved": False,
         "fused": False, "positions": "count", "dtype": "bf16"},
        # training with fewer key heads than query heads, part of each head rotated in pairs
        {"name": "qk_train_shared", "op": "qk_train", "B": 4, "T": 4096, "Hq": 32, "Hk": 8,
         "d": 64, "rot": 32, "norm": "rms", "weights": True, "interleaved": True,
         "fused": True, "positions": "count", "dtype": "bf16"},
        # the same in fp32 with odd sizes
        {"name": "qk_train_odd", "op": "qk_train", "B": 3, "T": 777, "Hq": 5, "Hk": 3, "d": 96,
         "rot": 40, "norm": "rms", "weights": True, "interleaved": False, "fused": False,
         "positions": "far", "dtype": "fp32"},
    ]


def _spread(rng, low, high):
    """A whole number between `low` and `high`, even over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["scan_step", "scan_fwd", "scan_fwd", "scan_packed", "scan_train",
                     "scan_train", "qk_fwd", "qk_fwd", "qk_train", "qk_train"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "scan_step":
        return {"op": op, "B": _spread(rng, 1, 512), "D": _spread(rng, 16, 8192), "dtype": dtype}
    if op.startswith("scan"):
        D = _spread(rng, 16, 4096)
        if rng.random() < 0.6:
            D = max(16, D // 16 * 16)
        most = MOST_SCAN_TRAIN if op == "scan_train" else MOST_SCAN // 2
        T = _spread(rng, 1, min(32768 if op == "scan_train" else 262144, most // D))
        case = {"op": op, "T": T, "D": D, "dtype": dtype, "h0": rng.random() < 0.6}
        room = max(1, most // (D * T))
        if op == "scan_packed":
            case["N"] = _spread(rng, 1, 64)
        else:
            case["B"] = _spread(rng, 1, min(64, room))
        return case
    d = rng.choice([64, 128, 128, 256, 8 * rng.randint(2, 32)])
    Hk = rng.randint(1, 32)
    Hq = Hk if rng.random() < 0.6 else rng.randint(1, 32)
    most = (MOST_QK if op == "qk_fwd" else MOST_QK_TRAIN // 2) // ((Hq + Hk) * d)
    T = _spread(rng, 1, max(1, min(65536, most)))
    B = _spread(rng, 1, max(1, min(256, most // T)))
    return {"op": op, "B": B, "T": T, "Hq": Hq, "Hk": Hk, "d": d,
            "rot": rng.choice([0, d, d, 8 * rng.randint(1, d // 8)]),
            "norm": rng.choice(["rms", "rms", "l2"]), "weights": rng.random() < 0.7,
            "interleaved": rng.random() < 0.4, "fused": rng.random() < 0.5,
            "positions": rng.choice(["count", "far"]), "dtype": dtype}


# ---------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _gates(shape, g):
    """log alpha = logsigmoid(z) / tau, with a tau of its own for each channel: memories from one
    token to some hundreds."""
    tau = torch.exp2(torch.rand(shape[-1], generator=g, device="cuda") * 8)
    z = torch.randn(shape, generator=g, device="cuda")
    return torch.nn.functional.logsigmoid(z).div_(tau)


def _lengths(case, seed):
    """Bounds of N ragged sequences over T rows: an empty one and one of a single token where
    there is room."""
    N, T = case["N"], case["T"]
    g = torch.Generator().manual_seed(int(seed) * 104729 + 3)
    share = torch.rand(N, generator=g).pow(3) + 1e-3
    if N >= 4:
        share[1] = 0.0
        share[2] = 0.0
    lens = (share / share.sum() * T).floor().long()
    if N >= 4 and T > N:
        lens[2] = 1
    lens[0] += T - int(lens.sum())
    return [0] + torch.cumsum(lens, 0).tolist()


def _scan_inputs(case, seed):
    g = _generator(seed)
    dt, D = DTYPES[case["dtype"]], case["D"]
    if case["op"] == "scan_step":
        lead = (case["B"],)
        states = case["B"]
    elif case["op"] == "scan_packed":
        lead = (case["T"],)
        states = case["N"]
    else:
        lead = (case["B"], case["T"])
        states = case["B"]
    s = {"x": torch.randn(lead + (D,), generator=g, device="cuda").to(dt),
         "log_alpha": _gates(lead + (D,), g)}
    if case["op"] == "scan_step" or case.get("h0"):
        s["h0"] = torch.randn((states, D), generator=g, device="cuda")
    else:
        s["h0"] = None
    if case["op"] == "scan_packed":
        s["cu"] = _lengths(case, seed)
    if case["op"] == "scan_train":
        s["dh"] = torch.randn(lead + (D,), generator=g, device="cuda").to(dt)
        s["dhT"] = torch.randn((states, D), generator=g, device="cuda")
    return s


def _frequencies(rot):
    return 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)


def _qk_inputs(case, seed):
    g = _generator(seed)
    dt = DTYPES[case["dtype"]]
    B, T, Hq, Hk, d = (case[n] for n in ("B", "T", "Hq", "Hk", "d"))
    if case["fused"]:
        qkv = torch.randn((B, T, Hq + 2 * Hk, d), generator=g, device="cuda").to(dt)
        q, k = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk]
    else:
        q = torch.randn((B, T, Hq, d), generator=g, device="cuda").to(dt)
        k = torch.randn((B, T, Hk, d), generator=g, device="cuda").to(dt)
    s = {"q": q, "k": k, "norm": case["norm"], "eps": 1e-6, "interleaved": case["interleaved"]}
    s["wq"], s["wk"] = ((1 + 0.2 * torch.randn((2, d), generator=g, device="cuda")).unbind(0)
                        if case["weights"] else (None, None))
    s["inv_freq"] = _frequencies(case["rot"]) if case["rot"] else None
    s["positions"] = None
    if case["positions"] == "far":
        start = torch.randint(0, 1 << 20, (B, 1), generator=g, device="cuda")
        s["positions"] = start + torch.arange(T, device="cuda")
    if case["op"] == "qk_train":
        s["dq"] = torch.randn((B, Hq, T, d), generator=g, device="cuda").to(dt)
        s["dk"] = torch.randn((B, Hk, T, d), generator=g, device="cuda").to(dt)
    return s


def prepare(case, seed):
    scan = case["op"].startswith("scan")
    s = (_scan_inputs if scan else _qk_inputs)(case, seed)
    if case["op"] == "scan_step":
        s["h"] = s["h0"].clone()
    if case["op"].endswith("train"):
        for n in (("x", "log_alpha", "h0") if scan else ("q", "k", "wq", "wk")):
            if s[n] is not None:
                s[n] = s[n].detach().requires_grad_()
    s["op"] = case["op"]
    return s


# ---------------------------------------------------------------- the plain forms

def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t from zero along dimension -2, by pairs: the scan of half the length
    over neighbours joined in twos gives every second h, one more step the others."""
    T = a.shape[-2]
    if T == 1:
        return b
    even, odd = slice(0, T // 2 * 2, 2), slice(1, None, 2)
    joined = _scan(a[..., odd, :] * a[..., even, :], a[..., odd, :] * b[..., even, :]
                   + b[..., odd, :])
    h = torch.empty_like(b)
    h[..., odd, :] = joined
    h[..., 0, :] = b[..., 0, :]
    h[..., 2::2, :] = a[..., 2::2, :] * joined[..., :(T - 1) // 2, :] + b[..., 2::2, :]
    return h


def _scan_from(a, x, h0):
    """The scan of `x` from the state `h0` (None: zero), in 32 bits."""
    b = x.float()
    if h0 is not None:
        b = torch.cat([a[..., :1, :] * h0.unsqueeze(-2) + b[..., :1, :], b[..., 1:, :]], -2)
    return _scan(a, b)


def _plain_step(s):
    s["h"].copy_(torch.exp(s["log_alpha"]) * s["h"] + s["x"].float())
    return s["h"].to(s["x"].dtype), s["h"]


def _plain_fwd(s):
    h = _scan_from(torch.exp(s["log_alpha"]), s["x"], s["h0"])
    return h.to(s["x"].dtype), h[..., -1, :].contiguous()


def _plain_packed(s):
    # a zero gate at each first row cuts the sequences apart
    first = torch.tensor([p for p, e in zip(s["cu"], s["cu"][1:]) if e > p], device="cuda")
    which = torch.tensor([n for n in range(len(s["cu"]) - 1) if s["cu"][n + 1] > s["cu"][n]],
                         device="cuda")
    last = torch.tensor([e - 1 for p, e in zip(s["cu"], s["cu"][1:]) if e > p], device="cuda")
    a, b = torch.exp(s["log_alpha"]), s["x"].to(torch.float32, copy=True)
    hT = torch.zeros((len(s["cu"]) - 1, b.shape[-1]), device="cuda")
    if s["h0"] is not None:
        b[first] += a[first] * s["h0"][which]
        hT.copy_(s["h0"])
    a[first] = 0.0
    h = _scan(a, b)
    hT[which] = h[last]
    return h.to(s["x"].dtype), hT


def _plain_train(s):
    x, a = s["x"].detach(), torch.exp(s["log_alpha"].detach())
    h0 = None if s["h0"] is None else s["h0"].detach()
    h = _scan_from(a, x, h0)
    # g_t = dh_t + a_{t+1} g_{t+1}: the same scan from the last row to the first
    d = s["dh"].float()
    d = torch.cat([d[..., :-1, :], d[..., -1:, :] + s["dhT"].unsqueeze(-2)], -2)
    after = torch.cat([a[..., 1:, :], torch.zeros_like(a[..., :1, :])], -2)
    g = _scan(after.flip(-2), d.flip(-2)).flip(-2)
    begin = torch.zeros_like(h[..., 0, :]) if h0 is None else h0
    before = torch.cat([begin.unsqueeze(-2), h[..., :-1, :]], -2)
    u = a * g
    grads = [g.to(x.dtype), u * before]
    if h0 is not None:
        grads.append(u[..., 0, :].contiguous())
    return [h.to(x.dtype), h[..., -1, :].contiguous()] + grads


def _angles(s):
    """cos and sin of position times frequency, [B or 1, T, 1, rot / 2]; the angle in 64 bits."""
    p = s["positions"]
    if p is None:
        p = torch.arange(s["q"].shape[1], device="cuda")[None]
    angle = (p.double()[..., None] * s["inv_freq"])[:, :, None]
    return torch.cos(angle).float(), torch.sin(angle).float()


def _halves(z, rot, interleaved):
    """The two members of each rotated pair of the first `rot` values."""
    if interleaved:
        return z[..., 0:rot:2], z[..., 1:rot:2]
    return z[..., :rot // 2], z[..., rot // 2:rot]


def _rotated(z, cos, sin, rot, interleaved):
    u, v = _halves(z, rot, interleaved)
    r = z.clone()
    ru, rv = _halves(r, rot, interleaved)
    ru.copy_(u * cos - v * sin)
    rv.copy_(u * sin + v * cos)
    return r


def _qk_one(x, w, s, angles):
    """One of q and k: its rows over their norms, and the same with weight, rotated and
    head-first, in 32 bits."""
    z = x.detach().float()
    n = z.shape[-1] if s["norm"] == "rms" else 1
    r = torch.rsqrt(z.square().sum(-1, keepdim=True) / n + s["eps"])
    y = z * r if w is None else z * r * w.detach()
    if angles is not None:
        y = _rotated(y, *angles, 2 * angles[0].shape[-1], s["interleaved"])
    return z * r, r, n, y.transpose(1, 2).to(x.dtype).contiguous()


def _qk_one_backward(unit, r, n, w, d, s, angles):
    g = d.transpose(1, 2).float()
    if angles is not None:
        cos, sin = angles
        g = _rotated(g, cos, -sin, 2 * cos.shape[-1], s["interleaved"])
    dw = None
    if w is not None:
        dw = (g * unit).sum((0, 1, 2), dtype=torch.float64).float()
        g = g * w.detach()
    dx = r * (g - unit * ((g * unit).sum(-1, keepdim=True) / n))
    return dx.to(d.dtype).contiguous(), dw


def _plain_qk(s):
    angles = None if s["inv_freq"] is None else _angles(s)
    uq, rq, n, yq = _qk_one(s["q"], s["wq"], s, angles)
    uk, rk, n, yk = _qk_one(s["k"], s["wk"], s, angles)
    if s["op"] == "qk_fwd":
        return yq, yk
    dq, dwq = _qk_one_backward(uq, rq, n, s["wq"], s["dq"], s, angles)
    dk, dwk = _qk_one_backward(uk, rk, n, s["wk"], s["dk"], s, angles)
    return [yq, yk, dq, dk] + ([] if dwq is None else [dwq, dwk])


PLAIN = {"scan_step": _plain_step, "scan_fwd": _plain_fwd, "scan_packed": _plain_packed,
         "scan_train": _plain_train, "qk_fwd": _plain_qk, "qk_train": _plain_qk}


# ---------------------------------------------------------------- the framework's calls

def _own(s):
    import chunkwise_linear_rnn_gb300 as gla
    op = s["op"]
    if op == "scan_step":
        return gla.gla_scan_step(s["x"], s["log_alpha"], s["h"]), s["h"]
    if op == "scan_fwd":
        return gla.gla_scan_fwd(s["x"], s["log_alpha"], s["h0"])
    if op == "scan_packed":
        return gla.gla_scan_fwd_varlen(s["x"], s["log_alpha"], s["cu"], s["h0"])
    if op == "scan_train":
        h, hT = gla.gla_scan(s["x"], s["log_alpha"], s["h0"])
        leaves = [s[n] for n in ("x", "log_alpha", "h0") if s[n] is not None]
        grads = torch.autograd.grad((h, hT), leaves, (s["dh"], s["dhT"]))
        return [h.detach(), hT.detach()] + list(grads)
    kw = {"norm": s["norm"], "eps": s["eps"], "interleaved": s["interleaved"]}
    if op == "qk_fwd":
        return gla.gla_qk_norm_rope_fwd(s["q"], s["k"], s["wq"], s["wk"], s["positions"],
                                        s["inv_freq"], **kw)
    q, k = gla.gla_qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["positions"], s["inv_freq"],
                                **kw)
    leaves = [s[n] for n in ("q", "k", "wq", "wk") if s[n] is not None]
    grads = torch.autograd.grad((q, k), leaves, (s["dq"], s["dk"]))
    return [q.detach(), k.detach()] + list(grads)


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["op"]](state)


def work(case):
    e = SIZES[case["dtype"]]
    if case["op"].startswith("scan"):
        D = case["D"]
        rows = case["T"] if case["op"] == "scan_packed" else case["B"] * case.get("T", 1)
        states = 4 * D * (case["N"] if case["op"] == "scan_packed" else case["B"])
        n = rows * D
        begin = states if case["op"] == "scan_step" or case["h0"] else 0
        if case["op"] == "scan_train":
            # x, log_alpha, dh, h0, dhT in; h, hT, dx, dlog_alpha, dh0 out
            return {"bytes": n * (4 * e + 8) + 2 * begin + 2 * states, "flops": 8 * n}
        return {"bytes": n * (2 * e + 4) + begin + states, "flops": 3 * n}
    rows = case["B"] * case["T"]
    n = rows * (case["Hq"] + case["Hk"]) * case["d"]
    small = (8 * rows if case["positions"] == "far" and case["rot"] else 0) + 4 * case["rot"]
    weights = 8 * case["d"] if case["weights"] else 0
    if case["op"] == "qk_train":
        return {"bytes": 4 * e * n + small + 2 * weights, "flops": 20 * n}
    return {"bytes": 2 * e * n + small + weights, "flops": 8 * n}


# ---------------------------------------------------------------- the definitions in 64 bits

def _walk(x, log_alpha, h0):
    """Every h of one sequence, token after token: x [T, ...]."""
    a, h = torch.exp(log_alpha), torch.empty_like(x)
    before = torch.zeros_like(x[0]) if h0 is None else h0
    for at, xt, ht in zip(a.unbind(0), x.unbind(0), h.unbind(0)):
        torch.addcmul(xt, at, before, out=ht)
        before = ht
    return h


def _exact_scan(case, seed):
    s = _scan_inputs(case, seed)
    x, la = s["x"].double(), s["log_alpha"].double()
    h0 = None if s["h0"] is None else s["h0"].double()
    if case["op"] == "scan_step":
        h = torch.exp(la) * h0 + x
        return h, h
    if case["op"] == "scan_packed":
        out, hT = torch.empty_like(x), torch.zeros((case["N"], case["D"]), device="cuda",
                                                   dtype=torch.float64)
        for n, (p, e) in enumerate(zip(s["cu"], s["cu"][1:])):
            begin = None if h0 is None else h0[n]
            if e > p:
                out[p:e] = _walk(x[p:e], la[p:e], begin)
                hT[n] = out[e - 1]
            elif h0 is not None:
                hT[n] = begin
        return out, hT
    x, la = x.transpose(0, 1), la.transpose(0, 1)
    h = _walk(x, la, h0)
    answer = [h.transpose(0, 1).contiguous(), h[-1].clone()]
    if case["op"] == "scan_fwd":
        return tuple(answer)
    d = s["dh"].double().transpose(0, 1)
    a = torch.exp(la)
    dx, dla = torch.empty_like(x), torch.empty_like(x)
    carried = s["dhT"].double()
    for t in range(case["T"] - 1, -1, -1):
        g = d[t] + carried
        carried = g * a[t]
        dx[t] = g
        if t > 0:
            torch.mul(carried, h[t - 1], out=dla[t])
        else:
            dla[t] = 0.0 if h0 is None else carried * h0
    answer += [dx.transpose(0, 1).contiguous(), dla.transpose(0, 1).contiguous()]
    return answer + ([] if h0 is None else [carried])


def _exact_qk(case, seed):
    s = _qk_inputs(case, seed)
    rot, got, grads = case["rot"], [], []
    for x, w, d in ((s["q"], s["wq"], s.get("dq")), (s["k"], s["wk"], s.get("dk"))):
        x = x.double().requires_grad_(d is not None)
        w = None if w is None else w.double().requires_grad_(d is not None)
        square = (x * x).mean(-1, keepdim=True) if s["norm"] == "rms" else \
            (x * x).sum(-1, keepdim=True)
        y = x / torch.sqrt(square + s["eps"])
        if w is not None:
            y = y * w
        if rot:
            # each pair is a complex number, turned by its angle
            p = torch.arange(case["T"], device="cuda")[None] if s["positions"] is None \
                else s["positions"]
            turn = torch.exp(1j * (p.double()[:, :, None, None] * s["inv_freq"]))
            part = y[..., :rot]
            if s["interleaved"]:
                z = turn * torch.complex(part[..., ::2], part[..., 1::2])
                part = torch.stack([z.real, z.imag], -1).flatten(-2)
            else:
                z = turn * torch.complex(*part.chunk(2, -1))
                part = torch.cat([z.real, z.imag], -1)
            y = torch.cat([part, y[..., rot:]], -1)
        y = y.permute(0, 2, 1, 3)
        got.append(y.detach().contiguous())
        if d is not None:
            leaves = [x] if w is None else [x, w]
            grads.append(torch.autograd.grad(y, leaves, d.double()))
    if case["op"] == "qk_fwd":
        return tuple(got)
    return got + [g[i] for i in range(len(grads[0])) for g in grads]


def exact(case, seed):
    return (_exact_scan if case["op"].startswith("scan") else _exact_qk)(case, seed)
