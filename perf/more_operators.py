"""The cases by which more of the library's language-model operators are
measured: the gated linear recurrence (minGRU from its pre-activations, for
prompts, training and single tokens), the norm of queries and keys for each
head with the position's rotation, and the embedding with its gradient.

`own` false: the plain form, elementary torch operations in 32 bits.  `own`
true: the library's entry points.
"""
import math

import torch

own = False

BASE = 10000.0  # of the rotation's frequencies


def listed():
    return [
        # one long prompt of one user: one batch row, so the time axis has to be split
        {"name": "gated prompt long", "op": "gated_fwd", "B": 1, "T": 16384, "D": 2048, "dtype": "bf16",
         "positive": True, "state": True},
        # a training batch in bf16, forward and backward
        {"name": "gated train", "op": "gated_train", "B": 8, "T": 4096, "D": 2048, "dtype": "bf16", "positive": True,
         "state": False},
        # training a small model at the long-T shape in fp32, signed values, state carried over from the batch before
        {"name": "gated train few channels", "op": "gated_train", "B": 16, "T": 1024, "D": 64, "dtype": "fp32",
         "positive": False, "state": True},
        # one token of one user: latency
        {"name": "gated step one", "op": "gated_step", "B": 1, "slots": 4, "D": 2048, "dtype": "bf16", "positive": True},
        # one token of each of many users, states in a larger cache
        {"name": "gated step many", "op": "gated_step", "B": 384, "slots": 400, "D": 2048, "dtype": "bf16",
         "positive": True},
        # queries and keys of one token of one user
        {"name": "qk norm token", "op": "qk_fwd", "B": 1, "T": 1, "H": 16, "Hk": 16, "D": 128, "R": 128,
         "interleaved": False, "dtype": "bf16", "far": 32768},
        # a batch of ragged prompts continued at their own positions, few key heads, half of each head rotated
        {"name": "qk norm prompts", "op": "qk_fwd", "B": 5, "T": 1537, "H": 12, "Hk": 4, "D": 64, "R": 32,
         "interleaved": True, "dtype": "bf16", "far": 8192},
        # a training batch, forward and backward
        {"name": "qk norm train", "op": "qk_train", "B": 8, "T": 4096, "H": 16, "Hk": 16, "D": 128, "R": 128,
         "interleaved": False, "dtype": "bf16", "far": 0},
        # the same in fp32, heads of 64, keys shared by three heads
        {"name": "qk norm train fp32", "op": "qk_train", "B": 16, "T": 1000, "H": 12, "Hk": 4, "D": 64, "R": 64,
         "interleaved": False, "dtype": "fp32", "far": 0},
        # the next tokens of many users
        {"name": "embed tokens", "op": "embed_fwd", "N": 384, "V": 50000, "D": 2048, "dtype": "bf16", "kind": "int64"},
        # a training batch, forward and the table's gradient: few words are most of the text
        {"name": "embed train", "op": "embed_train", "N": 32768, "V": 50000, "D": 2048, "dtype": "bf16",
         "kind": "int64"},
        # a small vocabulary in fp32, odd sizes: every row of the table is met often
        {"name": "embed train small", "op": "embed_train", "N": 3071, "V": 977, "D": 257, "dtype": "fp32",
         "kind": "int32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gated_fwd", "gated_train", "gated_train", "gated_step", "qk_fwd", "qk_train", "embed_fwd",
                     "embed_train", "embed_train"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "gated_step":
        B, D = _log(rng, 1, 512), _log(rng, 64, 4096)
        return {"op": op, "B": B, "slots": B + _log(rng, 1, 32), "D": D, "dtype": dtype, "positive": rng.random() < 0.6}
    if op.startswith("gated"):
        B, D = _log(rng, 1, 16), _log(rng, 32, 4096)
        D = D if rng.random() < 0.3 else (D + 7) // 8 * 8
        T = max(2, min(_log(rng, 2, 32768), (1 << 25) // (B * D)))
        return {"op": op, "B": B, "T": T, "D": D, "dtype": dtype, "positive": rng.random() < 0.6,
                "state": rng.random() < 0.5}
    if op.startswith("qk"):
        D, Hk = rng.choice([32, 64, 64, 80, 128, 128, 256]), _log(rng, 1, 16)
        H, B = Hk * rng.choice([1, 1, 2, 3]), _log(rng, 1, 16)
        T = max(1, min(_log(rng, 1, 8192), (1 << 25) // (B * (H + Hk) * D)))
        return {"op": op, "B": B, "T": T, "H": H, "Hk": Hk, "D": D, "R": rng.choice([D, D, D // 2 // 8 * 8]),
                "interleaved": rng.random() < 0.3, "dtype": dtype, "far": rng.choice([0, 0, 4096, 100000])}
    V, D, N = _log(rng, 50, 60000), _log(rng, 16, 4096), _log(rng, 1, 32768)
    D = D if rng.random() < 0.3 else (D + 7) // 8 * 8
    V, N = min(V, (1 << 26) // D), min(N, (1 << 25) // D)
    return {"op": op, "N": N, "V": V, "D": D, "dtype": dtype, "kind": rng.choice(["int64", "int32"])}


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, op = _dtype(case), case["op"]

    def normal(*shape, scale=1.0, to=dt):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(to)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    if op.startswith("gated"):
        B, D = case["B"], case["D"]
        T = case.get("T", 1)
        # gates and values are the halves of one product; each channel has a memory of its own, of a step to some hundred
        both = normal(B, T, 2 * D, to=torch.float32)
        both[..., :D] += 1 - 6 * uniform(D)
        gate, value = both.to(dt).split(D, -1)
        s = {"op": op, "positive": case["positive"], "dtype": dt, "gate": gate, "value": value}
        if op == "gated_step":
            slots = torch.randperm(case["slots"], generator=gen, device="cuda")[:B].to(torch.int32)
            return dict(s, gate=gate[:, 0], value=value[:, 0], slots=slots, index=slots.long(),
                        state=uniform(case["slots"], D) if case["positive"] else normal(case["slots"], D, to=torch.float32))
        s["h0"] = (uniform(B, D) if case["positive"] else normal(B, D, to=torch.float32)) if case["state"] else None
        if op == "gated_train":
            s["grad_h"] = normal(B, T, D)
            s["grad_hT"] = normal(B, D, to=torch.float32) if case["state"] else None
        return s
    if op.startswith("qk"):
        B, T, H, Hk, D, R = (case[n] for n in ("B", "T", "H", "Hk", "D", "R"))
        # queries and keys are parts of one product with the values'
        q, k, _ = normal(B, T, (H + 2 * Hk) * D, scale=2.0).unflatten(-1, (-1, D)).split([H, Hk, Hk], 2)
        # each sequence goes on from a place of its own
        first = torch.randint(0, case["far"] + 1, (B, 1), generator=gen, device="cuda")
        at = (first + torch.arange(T, device="cuda")).to(torch.int32)
        # the rotations of all positions, which a program keeps: cosines, then sines
        angle = torch.arange(case["far"] + T, device="cuda", dtype=torch.float64)[:, None] * _frequencies(R)
        s = {"op": op, "q": q, "k": k, "wq": normal(D, scale=0.2) + 1, "wk": normal(D, scale=0.2) + 1, "at": at,
             "table": torch.cat([angle.cos(), angle.sin()], 1).float(), "eps": 1e-6, "R": R,
             "interleaved": case["interleaved"], "dtype": dt}
        if op == "qk_train":
            s["grad_q"], s["grad_k"] = normal(B, T, H, D), normal(B, T, Hk, D)
        return s
    N, V, D = case["N"], case["V"], case["D"]
    # words by their rank, the r-th about 1 / (r + 2) as often as text has them, in an order of their own
    often = (1 / (torch.arange(V, device="cuda", dtype=torch.float64) + 2)).cumsum(0)
    rank = torch.searchsorted(often, uniform(N).double() * often[-1]).clamp(max=V - 1)
    tokens = torch.randperm(V, generator=gen, device="cuda")[rank].to(getattr(torch, case["kind"]))
    s = {"op": op, "tokens": tokens, "index": tokens.long(), "W": normal(V, D, scale=0.02), "scale": math.sqrt(D),
         "dtype": dt}
    if op == "embed_train":
        s["grad"] = normal(N, D)
    return s


def _frequencies(R):
    return BASE ** (-2 * torch.arange(R // 2, device="cuda", dtype=torch.float64) / R)


# ---------------------------------------------------------------- plain forms
def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t over dimension 1, by doubling the span that each step covers."""
    T, d = a.shape[1], 1
    while d < T:
        b = torch.cat([b[:, :d], b[:, d:] + a[:, d:] * b[:, :-d]], 1)
        a = torch.cat([a[:, :d], a[:, d:] * a[:, :-d]], 1)
        d *= 2
    return b


def _gated_parts(s):
    k, v = s["gate"].float(), s["value"].float()
    z, a = torch.sigmoid(k), torch.sigmoid(-k)
    if not s["positive"]:
        return z, a, v, torch.ones_like(v)
    low = torch.sigmoid(v)
    return z, a, torch.where(v >= 0, v + 0.5, low), torch.where(v >= 0, torch.ones_like(v), low * (1 - low))


def _gated_plain(s):
    z, a, c, slope = _gated_parts(s)
    h0 = s["h0"] if s["h0"] is not None else torch.zeros_like(z[:, 0])
    b = z * c
    b[:, 0] += a[:, 0] * h0
    h = _scan(a, b)
    out = {"h": h.to(s["dtype"]), "h_T": h[:, -1].contiguous()}
    if s["op"] == "gated_fwd":
        return out
    g = s["grad_h"].float()
    if s["grad_hT"] is not None:
        g = torch.cat([g[:, :-1], g[:, -1:] + s["grad_hT"][:, None]], 1)
    nxt = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    lam = _scan(nxt.flip(1), g.flip(1)).flip(1)
    before = torch.cat([h0[:, None], h[:, :-1]], 1)
    out.update(dgate=(lam * (c - before) * z * a).to(s["dtype"]), dvalue=(lam * z * slope).to(s["dtype"]))
    return out if s["h0"] is None else dict(out, dh0=a[:, 0] * lam[:, 0])


def _gated_step_plain(s):
    z, a, c, _ = _gated_parts(s)
    h = a * s["state"][s["index"]] + z * c
    s["state"][s["index"]] = h
    return {"h": h.to(s["dtype"]), "state": s["state"]}


def _pairs(x, R, interleaved):
    """The two members of each rotated pair, and what is not rotated."""
    if interleaved:
        return x[..., 0:R:2], x[..., 1:R:2], x[..., R:]
    return x[..., :R // 2], x[..., R // 2:R], x[..., R:]


def _joined(x1, x2, rest, interleaved):
    turned = torch.stack([x1, x2], -1).flatten(-2) if interleaved else torch.cat([x1, x2], -1)
    return torch.cat([turned, rest], -1)


def _qk_plain(s):
    R, il, dt = s["R"], s["interleaved"], s["dtype"]
    cos, sin = s["table"][s["at"].long()][:, :, None].split(R // 2, -1)
    out = {}
    for n in ("q", "k"):
        x, w = s[n].float(), s["w" + n].float()
        rstd = (x.square().mean(-1, keepdim=True) + s["eps"]).rsqrt()
        hat = x * rstd
        x1, x2, rest = _pairs(hat * w, R, il)
        out[n] = _joined(x1 * cos - x2 * sin, x2 * cos + x1 * sin, rest, il).to(dt)
        if s["op"] == "qk_train":
            g1, g2, rest = _pairs(s["grad_" + n].float(), R, il)
            g = _joined(g1 * cos + g2 * sin, g2 * cos - g1 * sin, rest, il)
            wg = g * w
            out["d" + n] = (rstd * (wg - hat * (wg * hat).mean(-1, keepdim=True))).to(dt)
            out["dw" + n] = (g * hat).sum((0, 1, 2)).to(dt)
    return out


def _embed_plain(s):
    out = {"x": (s["W"][s["index"]].float() * s["scale"]).to(s["dtype"])}
    if s["op"] == "embed_train":
        # the sum of a word's rows, in the words' order, as a difference of running sums
        order = s["index"].argsort(stable=True)
        rows, counts = s["index"][order].unique_consecutive(return_counts=True)
        sums = torch.nn.functional.pad(s["grad"].double()[order].cumsum(0), (0, 0, 1, 0))
        ends = counts.cumsum(0)
        dW = torch.zeros(s["W"].shape, device="cuda")
        dW[rows] = ((sums[ends] - sums[ends - counts]) * s["scale"]).float()
        out["dW"] = dW.to(s["dtype"])
    return out


# ---------------------------------------------------------------- one pass
def run(s):
    op = s["op"]
    if not own:
        return {"gated_fwd": _gated_plain, "gated_train": _gated_plain, "gated_step": _gated_step_plain,
                "qk_fwd": _qk_plain, "qk_train": _qk_plain, "embed_fwd": _embed_plain, "embed_train": _embed_plain}[op](s)
    from scan_linear_recurrences_gb300 import api
    if op == "gated_step":
        h = api.gated_scan_step(s["gate"], s["value"], s["state"], slots=s["slots"], positive=s["positive"])
        return {"h": h, "state": s["state"]}
    if op == "gated_fwd":
        h, h_T = api.gated_scan_fwd(s["gate"], s["value"], s["h0"], positive=s["positive"])
        return {"h": h, "h_T": h_T}
    if op == "gated_train":
        h, h_T, carries = api.gated_scan_fwd(s["gate"], s["value"], s["h0"], positive=s["positive"], want_carries=True)
        dgate, dvalue, dh0 = api.gated_scan_bwd(s["gate"], s["value"], carries, s["grad_h"], s["grad_hT"],
                                                positive=s["positive"], need_dh0=s["h0"] is not None)
        out = {"h": h, "h_T": h_T, "dgate": dgate, "dvalue": dvalue}
        return out if dh0 is None else dict(out, dh0=dh0)
    if op.startswith("qk"):
        opts = {"table": s["table"], "positions": s["at"], "eps": s["eps"], "interleaved": s["interleaved"]}
        q, k = api.qk_norm_fwd(s["q"], s["k"], s["wq"], s["wk"], **opts)
        if op == "qk_fwd":
            return {"q": q, "k": k}
        dq, dk, dwq, dwk = api.qk_norm_bwd(s["q"], s["k"], s["wq"], s["wk"], s["grad_q"], s["grad_k"], **opts)
        return {"q": q, "dq": dq, "dwq": dwq, "k": k, "dk": dk, "dwk": dwk}
    out = {"x": api.embedding_fwd(s["tokens"], s["W"], scale=s["scale"])}
    if op == "embed_train":
        out["dW"] = api.embedding_bwd(s["tokens"], s["grad"], s["W"].shape[0], scale=s["scale"])
    return out


def work(case):
    es, op = (2 if case["dtype"] == "bf16" else 4), case["op"]
    if op.startswith("gated"):
        B, D = case["B"], case["D"]
        if op == "gated_step":  # gate, value read, h written, each state read and written
            return {"bytes": B * (D * (3 * es + 8) + 4), "flops": 15 * B * D}
        n, state = B * case["T"] * D, 4 * B * D
        fwd = 3 * n * es + state * (2 if case["state"] else 1)
        if op == "gated_fwd":
            return {"bytes": fwd, "flops": 15 * n}
        # gate, value, grad_h, dgate, dvalue; the last state's gradient and the first one's, and the first state
        return {"bytes": fwd + 5 * n * es + (3 * state if case["state"] else 0), "flops": 40 * n}
    if op.startswith("qk"):
        tokens, D = case["B"] * case["T"], case["D"]
        n = tokens * (case["H"] + case["Hk"]) * D
        # q and k read and written; the weights, the positions and a row of the table for each position that is met
        fwd = 2 * n * es + 2 * D * es + tokens * 4 + (tokens if case["far"] else case["T"]) * case["R"] * 4
        if op == "qk_fwd":
            return {"bytes": fwd, "flops": 9 * n}
        # q, k, their outputs' gradients, their gradients
        return {"bytes": fwd + 3 * n * es + 4 * D * es, "flops": 25 * n}
    N, V, D = case["N"], case["V"], case["D"]
    # about how many rows of the table N words meet
    often = [1 / (r + 2) for r in range(V)]
    total = sum(often)
    rows = sum(-math.expm1(N * math.log1p(-p / total)) for p in often)
    ids = N * (8 if case["kind"] == "int64" else 4)
    fwd = int(rows) * D * es + N * D * es + ids
    if op == "embed_fwd":
        return {"bytes": fwd, "flops": N * D}
    return {"bytes": fwd + N * D * es + V * D * es, "flops": 3 * N * D}


# ---------------------------------------------------------------- the definitions, in 64 bits
def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op.startswith("gated"):
        k, v = s["gate"].double(), s["value"].double()
        a = 1 / (1 + k.exp())
        z = k.exp() * a
        pos = v >= 0
        c = torch.where(pos, v + 0.5, 1 / (1 + (-v).exp())) if case["positive"] else v
        if op == "gated_step":
            state = s["state"].double()
            h = a * state[s["index"]] + z * c
            state[s["index"]] = h
            return {"h": h, "state": state}
        h0 = torch.zeros_like(z[:, 0]) if s["h0"] is None else s["h0"].double()
        hs, h = torch.empty_like(z), h0
        for t in range(case["T"]):
            h = h + z[:, t] * (c[:, t] - h)
            hs[:, t] = h
        out = {"h": hs, "h_T": h}
        if op == "gated_fwd":
            return out
        dgate, dvalue = torch.empty_like(z), torch.empty_like(z)
        flow = torch.zeros_like(h0) if s["grad_hT"] is None else s["grad_hT"].double()
        for t in range(case["T"] - 1, -1, -1):
            flow = flow + s["grad_h"][:, t].double()
            drop = hs[:, t - 1] if t else h0
            dvalue[:, t] = flow * z[:, t]
            dgate[:, t] = dvalue[:, t] * a[:, t] * (c[:, t] - drop)
            flow = flow * a[:, t]
        if case["positive"]:
            dvalue = torch.where(pos, dvalue, dvalue / (2 + v.exp() + (-v).exp()))
        out.update(dgate=dgate, dvalue=dvalue)
        return out if s["h0"] is None else dict(out, dh0=flow)
    if op.startswith("qk"):
        R, D = case["R"], case["D"]
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), s["at"].double()[..., None, None] * _frequencies(R))
        i = torch.arange(R // 2, device="cuda")
        first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + R // 2)

        def rotate(x, by):  # the pairs as complex numbers
            x = x.clone()
            y = torch.complex(x[..., first], x[..., second]) * by
            x[..., first], x[..., second] = y.real, y.imag
            return x

        out = {}
        for n in ("q", "k"):
            x, w = s[n].double(), s["w" + n].double()
            rms = torch.sqrt(torch.einsum("bthd,bthd->bth", x, x) / D + s["eps"])[..., None]
            out[n] = rotate(x / rms * w, turn)
            if op == "qk_train":
                g = rotate(s["grad_" + n].double(), turn.conj())
                along = torch.einsum("bthd,bthd->bth", g * w, x)[..., None] / (D * rms ** 3)
                out["d" + n] = g * w / rms - along * x
                out["dw" + n] = torch.einsum("bthd,bthd->d", g, x / rms)
        return out
    out = {"x": s["W"].double()[s["index"]] * s["scale"]}
    if op == "embed_train":
        dW = torch.zeros(case["V"], case["D"], dtype=torch.float64, device="cuda")
        out["dW"] = dW.index_add_(0, s["index"], s["grad"].double()) * s["scale"]
    return out
