"""Two operators of layers with one decay per head, as measured cases.

Linear attention with one gate per token and head,

    S_t = exp(log_alpha_t) S_{t-1} + k_t^T v_t,      o_t = scale q_t S_t

over packed prompts, token-major and with fewer key heads than value heads, and as
the single token of a decode step whose states lie in a pool; and the norm over each
head's channels with an activation that follows it (a group norm, channels last),
forward, for one token, and with its gradients.

`run` computes either the plain form, in elementary torch operations, or the
framework's kernels (`own`).
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp32": 4}

# The most state values of a drawn token, token-head-channel products of a drawn prompt, and
# values of a drawn norm: those of the largest listed cases of each kind.
MOST_TOKEN = 256 * 32 * 128 * 128
MOST_PROMPT = 65536 * 16 * (2 * 128 + 2 * 256)
MOST_NORM = 2 * 32768 * 16 * 256
MOST_NORM_TRAIN = 4 * 4096 * 16 * 128

# Tokens of a chunk of the plain form.
CHUNK = 128


def listed():
    return [
        # one decode token for a few streams: latency
        {"name": "token_few", "op": "token", "B": 4, "Hk": 16, "H": 16, "dk": 128, "dv": 128,
         "fixed": False, "padded": False, "dtype": "bf16"},
        # one decode token for many streams
        {"name": "token_many", "op": "token", "B": 256, "Hk": 32, "H": 32, "dk": 128, "dv": 128,
         "fixed": False, "padded": False, "dtype": "bf16"},
        # odd heads in fp32, three value heads to a key head, a batch padded for a captured step
        {"name": "token_odd", "op": "token", "B": 37, "Hk": 3, "H": 9, "dk": 96, "dv": 80,
         "fixed": True, "padded": True, "dtype": "fp32"},
        # a batch of short prompts, empty and one-token ones among them
        {"name": "prompt_short", "op": "prompt", "N": 32, "T": 1500, "Hk": 8, "H": 8, "dk": 64,
         "dv": 64, "even": False, "h0": False, "fixed": True},
        # the prefill of a batch of equal prompts
        {"name": "prompt_medium", "op": "prompt", "N": 8, "T": 16384, "Hk": 16, "H": 16,
         "dk": 128, "dv": 128, "even": True, "h0": False, "fixed": False},
        # long prompts that go on from a state, values twice as wide as keys
        {"name": "prompt_long", "op": "prompt", "N": 2, "T": 65536, "Hk": 16, "H": 16,
         "dk": 128, "dv": 256, "even": True, "h0": True, "fixed": False},
        # ragged prompts, two value heads to a key head
        {"name": "prompt_ragged", "op": "prompt", "N": 24, "T": 40000, "Hk": 8, "H": 16,
         "dk": 128, "dv": 128, "even": False, "h0": True, "fixed": False},
        # the norm behind a decode step
        {"name": "norm_token", "op": "norm", "B": 256, "T": 1, "H": 32, "d": 128,
         "norm": "rms", "act": "silu", "gate": True, "weight": "shared", "bias": False,
         "heads_first": False, "fused": True, "dtype": "bf16"},
        # the norm behind the attention of a batch of prompts, its gate in a fused projection
        {"name": "norm_prompts", "op": "norm", "B": 8, "T": 2048, "H": 16, "d": 128,
         "norm": "rms", "act": "silu", "gate": True, "weight": "shared", "bias": False,
         "heads_first": True, "fused": True, "dtype": "bf16"},
        # a group norm with weights and biases of every channel, long
        {"name": "norm_long", "op": "norm", "B": 2, "T": 32768, "H": 16, "d": 256,
         "norm": "layer", "act": "silu", "gate": True, "weight": "channel", "bias": True,
         "heads_first": False, "fused": False, "dtype": "bf16"},
        # a training step's pass through the norm: forward, then all gradients
        {"name": "norm_train", "op": "norm_train", "B": 4, "T": 4096, "H": 16, "d": 128,
         "norm": "rms", "act": "silu", "gate": True, "weight": "shared", "bias": False,
         "heads_first": True, "fused": True, "dtype": "bf16"},
        # odd sizes in fp32, the activation on the norm itself
        {"name": "norm_train_odd", "op": "norm_train", "B": 3, "T": 777, "H": 5, "d": 96,
         "norm": "layer", "act": "silu", "gate": False, "weight": "channel", "bias": True,
         "heads_first": False, "fused": False, "dtype": "fp32"},
    ]


def _spread(rng, low, high):
    """A whole number between `low` and `high`, even over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["token", "token", "prompt", "prompt", "prompt", "norm", "norm",
                     "norm_train", "norm_train"])
    if op.startswith("norm"):
        d = rng.choice([64, 128, 128, 256, 8 * rng.randint(2, 64)])
        H = rng.randint(1, 32)
        most = (MOST_NORM if op == "norm" else MOST_NORM_TRAIN) // (H * d)
        T = _spread(rng, 1, max(1, min(65536, most)))
        B = _spread(rng, 1, max(1, min(256, most // T)))
        weight = rng.choice(["none", "shared", "shared", "channel"])
        return {"op": op, "B": B, "T": T, "H": H, "d": d, "norm": rng.choice(["rms", "layer"]),
                "act": rng.choice(["silu", "silu", "sigmoid"]), "gate": rng.random() < 0.7,
                "weight": weight, "bias": weight != "none" and rng.random() < 0.4,
                "heads_first": rng.random() < 0.5, "fused": rng.random() < 0.5,
                "dtype": rng.choice(["bf16", "bf16", "fp32"])}
    Hk = rng.randint(1, 16)
    H = Hk * rng.choice([1, 1, 2, 3])
    dk = rng.choice([64, 128, 128, 8 * rng.randint(2, 16)])
    dv = rng.choice([64, 128, 128, 256, 8 * rng.randint(2, 32)])
    fixed = rng.random() < 0.3
    if op == "token":
        B = _spread(rng, 1, max(1, min(512, MOST_TOKEN // (H * dk * dv))))
        return {"op": op, "B": B, "Hk": Hk, "H": H, "dk": dk, "dv": dv, "fixed": fixed,
                "padded": rng.random() < 0.3, "dtype": rng.choice(["bf16", "bf16", "fp32"])}
    most = MOST_PROMPT // (2 * Hk * dk + 2 * H * dv)
    T = _spread(rng, 1, max(1, min(65536, most)))
    return {"op": op, "N": _spread(rng, 1, 64), "T": T, "Hk": Hk, "H": H, "dk": dk, "dv": dv,
            "even": rng.random() < 0.3, "h0": rng.random() < 0.5, "fixed": fixed}


# ---------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 6151 + 29)
    return g


def _gates(lead, case, g):
    """One log gate per token and head, with memories from two tokens to some thousands; or one
    per head, 1 - 2^-(5 + ...), the same for every token."""
    H = case["H"]
    if case["fixed"]:
        return torch.log1p(-torch.exp2(-5.0 - 6.0 * torch.rand(H, generator=g, device="cuda")))
    rate = torch.exp2(-12.0 * torch.rand(H, generator=g, device="cuda"))
    return -rate * torch.nn.functional.softplus(
        torch.randn(lead + (H,), generator=g, device="cuda"))


def _lengths(case, seed):
    """Bounds of N prompts over T rows: equal ones, or ragged ones with an empty one and one of a
    single token where there is room."""
    N, T = case["N"], case["T"]
    if case["even"]:
        return [T * n // N for n in range(N + 1)]
    g = torch.Generator().manual_seed(int(seed) * 104729 + 5)
    share = torch.rand(N, generator=g).pow(2) + 1e-3
    if N >= 4:
        share[1] = 0.0
        share[2] = 0.0
    lens = (share / share.sum() * T).floor().long()
    if N >= 4 and T > N:
        lens[2] = 1
    lens[0] += T - int(lens.sum())
    return [0] + torch.cumsum(lens, 0).tolist()


def _attention_inputs(case, seed):
    g = _generator(seed)
    Hk, H, dk, dv = (case[n] for n in ("Hk", "H", "dk", "dv"))
    dt = DTYPES[case.get("dtype", "bf16")]
    rows = case["B"] if case["op"] == "token" else case["T"]
    # one projection gives q, k and v of a token side by side
    qkv = torch.randn((rows, 2 * Hk * dk + H * dv), generator=g, device="cuda").to(dt)
    q, k, v = qkv.split([Hk * dk, Hk * dk, H * dv], -1)
    s = {"q": q.view(rows, Hk, dk), "k": k.view(rows, Hk, dk), "v": v.view(rows, H, dv),
         "log_alpha": _gates((rows,), case, g), "scale": dk ** -0.5}
    if case["op"] == "token":
        pool = rows + rows // 4 + 1
        s["h0"] = torch.randn((pool, H, dk, dv), generator=g, device="cuda")
        s["slots"] = torch.randperm(pool, generator=g, device="cuda")[:rows]
        if case["padded"]:
            s["slots"][rows - rows // 8:] = -1
        return s
    s["cu"] = _lengths(case, seed)
    s["h0"] = None
    if case["h0"]:
        s["h0"] = torch.randn((case["N"], H, dk, dv), generator=g, device="cuda")
    return s


def _norm_inputs(case, seed):
    g = _generator(seed)
    B, T, H, d = (case[n] for n in ("B", "T", "H", "d"))
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    if case["heads_first"]:
        x = (normal(B, H, T, d) + 0.3).to(dt).transpose(1, 2)
    else:
        x = (normal(B, T, H, d) + 0.3).to(dt)
    gate = None
    if case["gate"]:
        gate = normal(B, T, 2 * H if case["fused"] else H, d).to(dt)[:, :, -H:]
    shape = (H, d) if case["weight"] == "channel" else (d,)
    s = {"x": x, "gate": gate, "norm": case["norm"], "act": case["act"], "eps": 1e-5,
         "weight": None if case["weight"] == "none" else 1 + 0.2 * normal(*shape),
         "bias": 0.2 * normal(*shape) if case["bias"] else None}
    if case["op"] == "norm_train":
        s["dy"] = normal(B, T, H, d).to(dt)
    return s


LEAVES = ("x", "gate", "weight", "bias")


def prepare(case, seed):
    if case["op"].startswith("norm"):
        s = _norm_inputs(case, seed)
        if case["op"] == "norm_train":
            for n in LEAVES:
                if s[n] is not None:
                    s[n] = s[n].detach().requires_grad_()
    else:
        s = _attention_inputs(case, seed)
        if case["op"] == "token":
            s["h"] = s["h0"].clone()
    s["op"] = case["op"]
    return s


# ---------------------------------------------------------------- the plain forms

def _plain_token(s):
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    share = v.shape[1] // q.shape[1]
    q, k = q.repeat_interleave(share, 1), k.repeat_interleave(share, 1)
    used = s["slots"] >= 0
    at = s["slots"].clamp(min=0)
    # a padded row takes part with slot 0 and is dropped from what is written
    h = (torch.exp(s["log_alpha"])[..., None, None] * s["h"][at]
         + k[..., :, None] * v[..., None, :])
    o = s["scale"] * (q[..., :, None] * h).sum(-2)
    keep = used.nonzero()[:, 0]
    s["h"][at[keep]] = h[keep]
    return (o * used[:, None, None]).to(s["q"].dtype), s["h"]


def _chunks(cu):
    """First row, rows, and sequence of every chunk; and for every sequence the number of its
    first chunk and how many it has."""
    first, rows, begin, count = [], [], [], []
    for p, e in zip(cu, cu[1:]):
        begin.append(len(first))
        for t in range(p, e, CHUNK):
            first.append(t)
            rows.append(min(CHUNK, e - t))
        count.append(len(first) - begin[-1])
    return first, rows, begin, count


def _plain_prompt(s):
    q, k, v = s["q"], s["k"], s["v"]
    (T, H, dv), (Hk, dk) = v.shape, q.shape[1:]
    N = len(s["cu"]) - 1
    first, rows, begin, count = _chunks(s["cu"])
    o = torch.empty((T, H, dv), dtype=v.dtype, device="cuda")
    hT = torch.zeros((N, H, dk, dv), device="cuda")
    if s["h0"] is not None:
        hT.copy_(s["h0"])
    if not first:
        return o, hT
    step = torch.arange(CHUNK, device="cuda")
    first, rows = torch.tensor([first, rows], device="cuda")
    real = step < rows[:, None]                                     # [n, C]
    index = (first[:, None] + step).clamp(max=T - 1)

    def chunked(x, heads):
        """[T, heads, d] as [H, n, C, d] in 32 bits, zeros behind a chunk's rows."""
        x = (x[index] * real[..., None, None]).float().permute(2, 0, 1, 3)
        return x.repeat_interleave(H // heads, 0)

    q, k, v = chunked(q, Hk), chunked(k, Hk), chunked(v, H)
    gates = s["log_alpha"].double().expand(T, H)
    G = (gates[index] * real[..., None]).cumsum(1).permute(2, 0, 1)  # [H, n, C]
    toward = (G[..., :, None] - G[..., None, :]).float()
    toward = torch.exp(toward.masked_fill_(step[:, None] < step, -math.inf))
    inside = ((q @ k.transpose(-1, -2)) * toward) @ v
    total = G[..., -1]
    sums = k.transpose(-1, -2) @ (torch.exp((total[..., None] - G).float())[..., None] * v)
    decay = torch.exp(total.float())[..., None, None]
    # the state that enters each chunk: all sequences' j-th chunks at once
    enter = torch.empty_like(sums)
    for j in range(max(count)):
        live = [n for n in range(N) if count[n] > j]
        live, at = torch.tensor([live, [begin[n] + j for n in live]], device="cuda")
        h = hT[live].transpose(0, 1)
        enter[:, at] = h
        hT[live] = (decay[:, at] * h + sums[:, at]).transpose(0, 1)
    out = s["scale"] * (inside + torch.exp(G.float())[..., None] * (q @ enter))
    o[index[real]] = out.to(o.dtype).permute(1, 2, 0, 3)[real]
    return o, hT


def _act(z, kind):
    """The activation and its derivative."""
    g = 1 / (1 + torch.exp(-z))
    return (z * g, g * (1 + z * (1 - g))) if kind == "silu" else (g, g * (1 - g))


def _plain_norm(s):
    x = s["x"].detach().float()
    weight, bias = (None if s[n] is None else s[n].detach() for n in ("weight", "bias"))
    if s["norm"] == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"])
    unit = x * r
    n = unit if weight is None else unit * weight
    if bias is not None:
        n = n + bias
    a, slope = _act(n if s["gate"] is None else s["gate"].detach().float(), s["act"])
    y = (a if s["gate"] is None else n * a).to(s["x"].dtype)
    if s["op"] == "norm":
        return y
    dy = s["dy"].float()
    grads = []
    if s["gate"] is None:
        dn = dy * slope
    else:
        dn = dy * a
        grads.append((dy * n * slope).to(s["x"].dtype))
    for z, p in ((dn * unit, weight), (dn, bias)):
        if p is not None:
            z = z.sum((0, 1), dtype=torch.float64)
            grads.append((z if p.dim() == 2 else z.sum(0)).float())
    u = dn if weight is None else dn * weight
    dx = u - unit * (u * unit).mean(-1, keepdim=True)
    if s["norm"] == "layer":
        dx = dx - u.mean(-1, keepdim=True)
    return [y, (r * dx).to(s["x"].dtype)] + grads


PLAIN = {"token": _plain_token, "prompt": _plain_prompt, "norm": _plain_norm,
         "norm_train": _plain_norm}


# ---------------------------------------------------------------- the framework's calls

def _own(s):
    import chunkwise_linear_rnn_gb300 as gla
    op = s["op"]
    if op == "token":
        o = gla.gla_headgate_step(s["q"], s["k"], s["v"], s["log_alpha"], s["h"], s["scale"],
                                  slots=s["slots"])
        return o, s["h"]
    if op == "prompt":
        return gla.gla_headgate_fwd_varlen(s["q"], s["k"], s["v"], s["log_alpha"], s["cu"],
                                           s["scale"], s["h0"])
    kw = {"norm": s["norm"], "activation": s["act"], "eps": s["eps"]}
    if op == "norm":
        return gla.gla_group_norm_act_fwd(s["x"], s["gate"], s["weight"], s["bias"], **kw)
    y = gla.gla_group_norm_act(s["x"], s["gate"], s["weight"], s["bias"], **kw)
    leaves = [s[n] for n in LEAVES if s[n] is not None]
    return [y.detach()] + list(torch.autograd.grad(y, leaves, s["dy"]))


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["op"]](state)


def work(case):
    if case["op"].startswith("norm"):
        e = SIZES[case["dtype"]]
        n = case["B"] * case["T"] * case["H"] * case["d"]
        w = 0 if case["weight"] == "none" else case["d"]
        w = 4 * w * (case["H"] if case["weight"] == "channel" else 1) * (2 if case["bias"] else 1)
        if case["op"] == "norm":
            return {"bytes": (3 if case["gate"] else 2) * e * n + w, "flops": 12 * n}
        return {"bytes": (6 if case["gate"] else 4) * e * n + 2 * w, "flops": 30 * n}
    Hk, H, dk, dv = (case[n] for n in ("Hk", "H", "dk", "dv"))
    states = H * dk * dv
    if case["op"] == "token":
        B = case["B"] - (case["B"] // 8 if case["padded"] else 0)
        e = SIZES[case["dtype"]]
        gates = 4 * H if case["fixed"] else 4 * B * H
        return {"bytes": 8 * B * states + e * B * (2 * Hk * dk + 2 * H * dv) + gates + 8 * B,
                "flops": 5 * B * states}
    T = case["T"]
    gates = 4 * H if case["fixed"] else 4 * T * H
    return {"bytes": 2 * T * (2 * Hk * dk + 2 * H * dv) + gates
            + 4 * case["N"] * states * (2 if case["h0"] else 1), "flops": 5 * T * states}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_attention(case, seed):
    s = _attention_inputs(case, seed)
    share = case["H"] // case["Hk"]
    q, k = (s[n].double().repeat_interleave(share, 1) for n in ("q", "k"))
    v, a = s["v"].double(), torch.exp(s["log_alpha"].double()).expand(s["v"].shape[:2])

    def one(h, rows):
        """The rows' tokens, each on its own state of h; their outputs."""
        h.mul_(a[rows][..., None, None])
        h.add_(torch.einsum("bhi,bhj->bhij", k[rows], v[rows]))
        return s["scale"] * torch.einsum("bhi,bhij->bhj", q[rows], h)

    o = torch.zeros_like(v)
    if case["op"] == "token":
        pool = s["h0"].double()
        rows = torch.nonzero(s["slots"] >= 0)[:, 0]
        h = pool[s["slots"][rows]]
        o[rows] = one(h, rows)
        pool[s["slots"][rows]] = h
        return o, pool
    N, H, dk, dv = case["N"], case["H"], case["dk"], case["dv"]
    lens = [e - p for p, e in zip(s["cu"], s["cu"][1:])]
    if max(lens) > 70000:
        return None
    order = sorted(range(N), key=lambda n: -lens[n])
    h = torch.zeros((N, H, dk, dv), dtype=torch.float64, device="cuda")
    if s["h0"] is not None:
        h.copy_(s["h0"][order])
    begin = torch.tensor([s["cu"][n] for n in order], device="cuda")
    live = N
    for t in range(lens[order[0]]):
        # the sequences that still have a token stand first
        while lens[order[live - 1]] <= t:
            live -= 1
        rows = begin[:live] + t
        o[rows] = one(h[:live], rows)
    hT = torch.empty_like(h)
    hT[order] = h
    return o, hT


def _exact_norm(case, seed):
    s = _norm_inputs(case, seed)
    train = case["op"] == "norm_train"
    leaf = {n: s[n].double().requires_grad_(train) for n in LEAVES if s[n] is not None}
    x = leaf["x"]
    if case["norm"] == "layer":
        spread, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
        y = (x - mean) / torch.sqrt(spread + s["eps"])
    else:
        y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / case["d"] + s["eps"])
    y = y * leaf["weight"] if "weight" in leaf else y
    y = y + leaf["bias"] if "bias" in leaf else y
    z = leaf.get("gate", y)
    a = torch.sigmoid(z) if case["act"] == "sigmoid" else z * torch.sigmoid(z)
    y = a * y if "gate" in leaf else a
    if not train:
        return y
    return [y.detach()] + list(torch.autograd.grad(y, list(leaf.values()), s["dy"].double()))


def exact(case, seed):
    return (_exact_norm if case["op"].startswith("norm") else _exact_attention)(case, seed)
