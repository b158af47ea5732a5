"""The cases by which the library's language-model operators are measured:
linear attention with a decay for each head (prompts, training, single
tokens), the RMS norm with the residual's addition (training, and the fp8
output of serving) and the clipping of gradients by their global norm.

`own` false: the plain form, elementary torch operations in 32 bits.  `own`
true: the library's entry points.
"""
import math

import torch

own = False

CHUNK = 64       # chunk length of the plain form's linear attention
FP8_MAX = 448.0  # largest finite e4m3 value


def listed():
    return [
        # one long prompt of one user: few (batch, head) lanes, so the time axis has to be split
        {"name": "attn prompt long", "op": "attn_fwd", "B": 1, "T": 16384, "H": 16, "Hk": 16, "D": 128,
         "dtype": "bf16", "state": True, "fixed": False},
        # a batch of ragged prompts continued from cached states, query/key heads shared by three value heads
        {"name": "attn prompt shared heads", "op": "attn_fwd", "B": 5, "T": 1537, "H": 12, "Hk": 4, "D": 64,
         "dtype": "bf16", "state": True, "fixed": False},
        # a short prompt: a few sentences, latency counts
        {"name": "attn prompt short", "op": "attn_fwd", "B": 1, "T": 100, "H": 8, "Hk": 8, "D": 128,
         "dtype": "bf16", "state": True, "fixed": False},
        # a training batch in bf16, forward and backward
        {"name": "attn train", "op": "attn_train", "B": 8, "T": 4096, "H": 16, "Hk": 16, "D": 128,
         "dtype": "bf16", "state": False, "fixed": False},
        # training at the long-T shape with heads of 64 in fp32, one learned decay a head
        {"name": "attn train fp32", "op": "attn_train", "B": 16, "T": 1024, "H": 8, "Hk": 8, "D": 64,
         "dtype": "fp32", "state": True, "fixed": True},
        # one token of one user
        {"name": "attn step one", "op": "attn_step", "B": 1, "slots": 4, "H": 16, "Hk": 16, "D": 128, "dtype": "bf16"},
        # one token of each of many users, states in a larger cache
        {"name": "attn step many", "op": "attn_step", "B": 384, "slots": 400, "H": 16, "Hk": 16, "D": 128,
         "dtype": "bf16"},
        # the norm in front of an fp8 product, one token: latency
        {"name": "norm fp8 one token", "op": "norm_fp8", "rows": 1, "N": 4096, "dtype": "bf16", "group": 128},
        # the same over a prompt, a scale for each row
        {"name": "norm fp8 prompt", "op": "norm_fp8", "rows": 8191, "N": 5120, "dtype": "bf16", "group": 0},
        # a training batch's norm, forward and backward
        {"name": "norm train", "op": "norm_train", "rows": 32768, "N": 2048, "dtype": "bf16"},
        # a small model's gradients, in fp32
        {"name": "clip small", "op": "clip", "layers": 2, "width": 256, "dtype": "fp32", "max": 1.0},
        # gradients of a model of about a billion parameters, bf16 matrices and fp32 norm weights
        {"name": "clip large", "op": "clip", "layers": 22, "width": 2048, "dtype": "bf16", "max": 1.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn_fwd", "attn_fwd", "attn_train", "attn_train", "attn_step", "norm_fp8", "norm_train", "clip"])
    if op in ("attn_fwd", "attn_train"):
        D = rng.choice([64, 128])
        Hk = _log(rng, 1, 16)
        H = Hk * rng.choice([1, 1, 1, 2, 3])
        B = _log(rng, 1, 16)
        most = (1 << 19) * 64 // D if op == "attn_fwd" else (1 << 18) * 64 // D
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        T = max(2, min(_log(rng, 2, 16384), most // (B * H)))
        return {"op": op, "B": B, "T": T, "H": H, "Hk": Hk, "D": D, "dtype": dtype, "state": rng.random() < 0.5,
                "fixed": rng.random() < 0.25}
    if op == "attn_step":
        B, Hk, D = _log(rng, 1, 256), _log(rng, 2, 16), rng.choice([64, 128])
        return {"op": op, "B": B, "slots": B + _log(rng, 1, 32), "H": Hk * rng.choice([1, 1, 2]), "Hk": Hk, "D": D,
                "dtype": rng.choice(["bf16", "bf16", "fp32"])}
    if op == "clip":
        width = _log(rng, 100, 1536)
        return {"op": op, "layers": _log(rng, 1, 16), "width": width + (width == 768), "dtype": rng.choice(["bf16", "fp32"]),
                "max": rng.choice([1.0, 1.0, 1.0, 1e4])}
    N, group = _log(rng, 64, 8192), 0
    if rng.random() < 0.7:
        N = (N + 127) // 128 * 128
        group = rng.choice([0, 128])
    N = N + 128 if N == 3072 else N
    rows = min(_log(rng, 1, 32768), (1 << 26) // N)
    d = {"op": op, "rows": rows, "N": N, "dtype": rng.choice(["bf16", "bf16", "fp32"])}
    return dict(d, group=group) if op == "norm_fp8" else d


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _clip_shapes(case):
    w = case["width"]
    layer = [((w, w), False)] * 4 + [((4 * w, w), False), ((w, 4 * w), False), ((w,), True), ((w,), True)]
    return layer * case["layers"] + [((w,), True), ((977, w), False)]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, op = _dtype(case), case["op"]

    def normal(*shape, scale=1.0, to=dt):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(to)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    if op.startswith("attn"):
        B, H, Hk, D = (case[n] for n in ("B", "H", "Hk", "D"))
        # a head's decay a step between about 0.6 and 0.999, as gated linear attention learns them
        rate = torch.exp(-6.2 + 5.5 * uniform(H))
        if op == "attn_step":
            g = -rate * torch.nn.functional.softplus(normal(B, H, to=torch.float32) + 0.5)
            slots = torch.randperm(case["slots"], generator=gen, device="cuda")[:B].to(torch.int32)
            return {"op": op, "q": normal(B, Hk, D), "k": normal(B, Hk, D), "v": normal(B, H, D), "g": g,
                    "S": normal(case["slots"], H, D, D, scale=3.0, to=torch.float32), "slots": slots,
                    "index": slots.long(), "dtype": dt}
        T = case["T"]
        g = -rate if case["fixed"] else \
            -rate * torch.nn.functional.softplus(normal(B, T, H, to=torch.float32) + 0.5)
        s = {"op": op, "q": normal(B, T, Hk, D), "k": normal(B, T, Hk, D), "v": normal(B, T, H, D), "g": g,
             "S0": normal(B, H, D, D, scale=3.0, to=torch.float32) if case["state"] else None, "dtype": dt}
        if op == "attn_train":
            s["grad_o"] = normal(B, T, H, D)
            s["grad_ST"] = normal(B, H, D, D, scale=0.1, to=torch.float32) if case["state"] else None
        return s
    if op.startswith("norm"):
        rows, N = case["rows"], case["N"]
        s = {"op": op, "x": normal(rows, N), "res": normal(rows, N, scale=4.0), "w": normal(N, scale=0.2) + 1,
             "eps": 1e-6, "dtype": dt, "group": case.get("group")}
        if op == "norm_train":
            s["grad_y"], s["grad_r"] = normal(rows, N), normal(rows, N)
        return s
    # each matrix's gradient in `dtype`, the norm weights' in fp32; all of one type behind one another in
    # one buffer (as a framework's gradient buckets lie), each at a multiple of 64 elements
    shapes = _clip_shapes(case)
    s = {"op": op, "max_norm": case["max"], "grads": [], "out": [], "flat": []}
    kinds = [torch.float32 if vec else dt for _, vec in shapes]
    sizes = [math.prod(sh) for sh, _ in shapes]
    for kind in dict.fromkeys(kinds):
        n = sum((z + 63) // 64 * 64 for z, k in zip(sizes, kinds) if k == kind)
        s["flat"].append((kind, torch.zeros(n, device="cuda", dtype=kind), torch.zeros(n, device="cuda", dtype=kind)))
    at = {kind: 0 for kind, _, _ in s["flat"]}
    bufs = {kind: (a, b) for kind, a, b in s["flat"]}
    for (shape, _), kind, z in zip(shapes, kinds, sizes):
        a, b = bufs[kind]
        s["grads"].append(a[at[kind]:at[kind] + z].normal_(std=0.02, generator=gen).view(shape))
        s["out"].append(b[at[kind]:at[kind] + z].view(shape))
        at[kind] += (z + 63) // 64 * 64
    return s


# ---------------------------------------------------------------- plain forms
def _sums(x):
    """[..., n] -> [..., n, n]: entry (i, j) = x_{j+1} + ... + x_i for j <= i, -inf above the diagonal."""
    n = x.shape[-1]
    strict = torch.ones(n, n, dtype=torch.bool, device=x.device).tril(-1)
    s = x[..., :, None].expand(*x.shape, n).masked_fill(~strict, 0).cumsum(-2)
    return s.masked_fill(strict.T, -math.inf)


def _chunked(q, k, v, g, S0):
    """o_t = S_t^T q_t, S_t = e^{g_t} S_{t-1} + k_t v_t^T over [B,H,n,C,D] chunks, g [B,H,n,C], S0 [B,H,D,D];
    returns o, and the state after each chunk [B,H,n,D,D]."""
    G = g.cumsum(-1)
    o = ((q @ k.transpose(-1, -2)) * _sums(g).exp()) @ v
    rest = g.flip(-1).cumsum(-1).flip(-1) - g
    kv = (k * rest.exp()[..., None]).transpose(-1, -2) @ v
    total = G[..., -1]
    B, H, n, D = total.shape[0], total.shape[1], total.shape[2], q.shape[-1]
    ends = (_sums(total).exp() @ kv.reshape(B, H, n, -1)).reshape(kv.shape)
    ends = ends + total.cumsum(-1).exp()[..., None, None] * S0[:, :, None]
    starts = torch.cat([S0[:, :, None], ends[:, :, :-1]], 2)
    return o + G.exp()[..., None] * (q @ starts), ends


def _to_chunks(x, H):
    """[B,T,h,D] -> [B,H,n,C,D] in 32 bits, heads repeated to H, time padded with zeros."""
    x = x.float()
    x = x.repeat_interleave(H // x.shape[2], 2)
    x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, -x.shape[1] % CHUNK))
    return x.transpose(1, 2).reshape(x.shape[0], H, -1, CHUNK, x.shape[-1])


def _from_chunks(x, T, Hk):
    B, H, D = x.shape[0], x.shape[1], x.shape[-1]
    x = x.reshape(B, H, -1, D)[:, :, :T].transpose(1, 2)
    return x.reshape(B, T, Hk, H // Hk, D).sum(3)


def _attn_plain(s):
    q, k, v, g, dt = s["q"], s["k"], s["v"], s["g"], s["dtype"]
    (B, T, Hk, D), H = q.shape, v.shape[2]
    scale = D ** -0.5
    gc = _to_chunks((g if g.dim() == 3 else g.expand(B, T, H))[..., None], H)[..., 0]
    qc, kc, vc = _to_chunks(q, H) * scale, _to_chunks(k, H), _to_chunks(v, H)
    S0 = s["S0"] if s["S0"] is not None else q.new_zeros((B, H, D, D), dtype=torch.float32)
    o, ends = _chunked(qc, kc, vc, gc, S0)
    out = {"o": _from_chunks(o, T, H).to(dt), "S_T": ends[:, :, -1].contiguous()}
    if s["op"] == "attn_fwd":
        return out
    do = _to_chunks(s["grad_o"], H)
    R_T = s["grad_ST"] if s["grad_ST"] is not None else torch.zeros_like(S0)
    dq, _ = _chunked(do, vc, kc, gc, S0.transpose(-1, -2))
    # the reverse scans: the same map on flipped time, the decay of step t + 1 applied at step t
    back = lambda x: x.flatten(2, 3).flip(2).unflatten(2, (-1, CHUNK))  # noqa: E731
    gr = torch.nn.functional.pad(gc.flatten(2, 3).flip(2), (1, 0))[..., :-1].unflatten(2, (-1, CHUNK))
    dk, _ = _chunked(back(vc), back(do), back(qc), gr, R_T.transpose(-1, -2))
    dv, R = _chunked(back(kc), back(qc), back(do), gr, R_T)
    dk, dv, R = back(dk), back(dv), R.flip(2)
    R = R * gc[..., 0].exp()[..., None, None]             # dL/d(state before each chunk)
    after = torch.cat([R[:, :, 1:], R_T[:, :, None]], 2)  # dL/d(state after each chunk), of later steps
    part = (dq * qc).sum(-1) - (dk * kc).sum(-1)
    dg = part.flip(-1).cumsum(-1).flip(-1) + (after * ends).sum((-1, -2))[..., None]
    dg = dg.flatten(2, 3)[:, :, :T].transpose(1, 2).contiguous()
    out.update(dq=_from_chunks(dq * scale, T, Hk).to(dt), dk=_from_chunks(dk, T, Hk).to(dt),
               dv=_from_chunks(dv, T, H).to(dt), dg=dg if g.dim() == 3 else dg.sum((0, 1)))
    return out if s["S0"] is None else dict(out, dS0=R[:, :, 0].contiguous())


def _step_plain(s):
    S, v, D = s["S"], s["v"].float(), s["q"].shape[-1]
    group = v.shape[1] // s["q"].shape[1]
    q, k = (s[n].float().repeat_interleave(group, 1) for n in ("q", "k"))
    new = s["g"].exp()[..., None, None] * S[s["index"]] + k[..., :, None] * v[..., None, :]
    S[s["index"]] = new
    return {"o": (D ** -0.5 * (new * q[..., :, None]).sum(-2)).to(s["dtype"]), "S": S}


def _norm_plain(s):
    dt, w = s["dtype"], s["w"].float()
    r = (s["x"].float() + s["res"].float()).to(dt)  # the residual stream is kept in the model's type
    rstd = (r.float().square().mean(-1, keepdim=True) + s["eps"]).rsqrt()
    hat = r.float() * rstd
    y = hat * w
    if s["op"] == "norm_fp8":
        rows, N = y.shape
        yg = y.reshape(rows, -1, s["group"] or N)
        sc = yg.abs().amax(-1) * (1 / FP8_MAX)
        safe = torch.where(sc > 0, sc, torch.ones_like(sc))
        q8 = (yg / safe[..., None]).clamp(-FP8_MAX, FP8_MAX).reshape(rows, N).to(torch.float8_e4m3fn)
        return {"q": q8, "scales": sc, "r": r}
    dy = s["grad_y"].float()
    wdy = dy * w
    dx = rstd * (wdy - hat * (wdy * hat).mean(-1, keepdim=True)) + s["grad_r"].float()
    return {"y": y.to(dt), "r": r, "dx": dx.to(dt), "dw": (dy * hat).sum(0).to(dt)}


def _clip_plain(s):
    n = torch.stack([t.float().square().sum() for t in s["grads"]]).sum().sqrt()
    c = (s["max_norm"] / (n + 1e-6)).clamp(max=1.0)
    [o.copy_(t.float() * c) for o, t in zip(s["out"], s["grads"])]
    return {"norm": n, "clipped": [b for _, _, b in s["flat"]]}


# ---------------------------------------------------------------- one pass
def run(s):
    op = s["op"]
    if not own:
        return {"attn_fwd": _attn_plain, "attn_train": _attn_plain, "attn_step": _step_plain, "norm_fp8": _norm_plain,
                "norm_train": _norm_plain, "clip": _clip_plain}[op](s)
    from scan_linear_recurrences_gb300 import api
    if op in ("attn_fwd", "attn_train"):
        o, S_T = api.linear_attention_fwd(s["q"], s["k"], s["v"], s["g"], s["S0"], want_state=True)
        out = {"o": o, "S_T": S_T}
        if op == "attn_train":
            dq, dk, dv, dg, dS0 = api.linear_attention_bwd(s["q"], s["k"], s["v"], s["g"], s["grad_o"], s["S0"],
                                                           s["grad_ST"])
            out.update(dq=dq, dk=dk, dv=dv, dg=dg)
            if dS0 is not None:
                out["dS0"] = dS0
        return out
    if op == "attn_step":
        return {"o": api.linear_attention_step(s["q"], s["k"], s["v"], s["g"], s["S"], slots=s["slots"]), "S": s["S"]}
    if op == "norm_fp8":
        q8, scales, r = api.rms_norm_fp8_fwd(s["x"], s["w"], s["res"], eps=s["eps"], group=s["group"])
        return {"q": q8, "scales": scales, "r": r}
    if op == "norm_train":
        y, r, rstd = api.rms_norm_fwd(s["x"], s["w"], s["res"], eps=s["eps"])
        dx, dw = api.rms_norm_bwd(r, s["w"], rstd, s["grad_y"], s["grad_r"])
        return {"y": y, "r": r, "dx": dx, "dw": dw}
    n = api.clip_grad_norm(s["grads"], s["max_norm"], out=s["out"])
    return {"norm": n, "clipped": [b for _, _, b in s["flat"]]}


def work(case):
    es, op = (2 if case["dtype"] == "bf16" else 4), case["op"]
    if op.startswith("attn"):
        B, H, Hk, D = (case[n] for n in ("B", "H", "Hk", "D"))
        if op == "attn_step":  # q, k, v, g read, o written, each state read and written
            return {"bytes": B * ((2 * Hk + 2 * H) * D * es + 4 * H + 4) + 8 * B * H * D * D, "flops": 5 * B * H * D * D}
        T = case["T"]
        qk, v, g, S = B * T * Hk * D * es, B * T * H * D * es, 4 * (H if case["fixed"] else B * T * H), 4 * B * H * D * D
        fwd = 2 * qk + 2 * v + g + S * (2 if case["state"] else 1)
        if op == "attn_fwd":
            return {"bytes": fwd, "flops": 4 * B * T * H * D * D}
        # q, k, v, do, g, dq, dk, dv, dg; the initial state, its gradient and the final state's
        bwd = 4 * qk + 3 * v + 2 * g + (3 * S if case["state"] else 0)
        return {"bytes": fwd + bwd, "flops": 12 * B * T * H * D * D}
    if op.startswith("norm"):
        n = case["rows"] * case["N"]
        if op == "norm_fp8":  # x, res, w read; r, the fp8 values and the scales written
            return {"bytes": 3 * n * es + n + case["N"] * es + 4 * n // (case["group"] or case["N"]), "flops": 6 * n}
        # forward: x, res read, y, r written; backward: r, dy, dr read, dx written; w twice, dw
        return {"bytes": 8 * n * es + 3 * case["N"] * es, "flops": 16 * n}
    by = sum(math.prod(sh) * (4 if vec else es) for sh, vec in _clip_shapes(case))
    return {"bytes": 2 * by + 4, "flops": 3 * sum(math.prod(sh) for sh, _ in _clip_shapes(case))}


# ---------------------------------------------------------------- the definitions, in 64 bits
def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    d = lambda x: None if x is None else x.double()  # noqa: E731
    if op == "attn_step":
        S, group = d(s["S"]), case["H"] // case["Hk"]
        o = torch.empty(case["B"], case["H"], case["D"], dtype=torch.float64, device="cuda")
        for b, slot in enumerate(s["slots"].tolist()):
            for h in range(case["H"]):
                S[slot, h] *= math.exp(s["g"][b, h].item())
                S[slot, h] += torch.outer(d(s["k"][b, h // group]), d(s["v"][b, h]))
                o[b, h] = S[slot, h].T @ d(s["q"][b, h // group]) / math.sqrt(case["D"])
        return {"o": o, "S": S}
    if op.startswith("attn"):
        B, T, H, Hk, D = (case[n] for n in ("B", "T", "H", "Hk", "D"))
        group, sc = H // Hk, 1 / math.sqrt(D)
        heads = lambda x: d(x).unsqueeze(3).expand(B, T, Hk, group, D).reshape(B, T, H, D)  # noqa: E731
        q, k, v = heads(s["q"]) * sc, heads(s["k"]), d(s["v"])
        a = d(s["g"]).exp().expand(B, T, H)[..., None, None]
        S = torch.zeros(B, H, D, D, dtype=torch.float64, device="cuda") if s["S0"] is None else d(s["S0"])
        S0, o, dq, do = S, torch.empty_like(v), torch.empty_like(v), d(s.get("grad_o"))
        for t in range(T):
            S = a[:, t] * S + k[:, t, :, :, None] * v[:, t, :, None, :]
            o[:, t] = torch.einsum("bhij,bhi->bhj", S, q[:, t])
            if do is not None:
                dq[:, t] = torch.einsum("bhij,bhj->bhi", S, do[:, t])
        out = {"o": o, "S_T": S}
        if op == "attn_fwd":
            return out
        R = torch.zeros_like(S) if s["grad_ST"] is None else d(s["grad_ST"])
        dk, dv, dg = torch.empty_like(v), torch.empty_like(v), torch.empty(B, T, H, dtype=torch.float64, device="cuda")
        tail = (R * S).sum((-1, -2))  # <R_t, e^{g_t} S_{t-1}>, by its difference from step to step
        for t in range(T - 1, -1, -1):
            R = R + q[:, t, :, :, None] * do[:, t, :, None, :]
            dk[:, t] = torch.einsum("bhij,bhj->bhi", R, v[:, t])
            dv[:, t] = torch.einsum("bhij,bhi->bhj", R, k[:, t])
            tail = tail + (q[:, t] * dq[:, t]).sum(-1) - (k[:, t] * dk[:, t]).sum(-1)
            dg[:, t] = tail
            R = a[:, t] * R
        shared = lambda x: x.unflatten(2, (Hk, group)).sum(3)  # noqa: E731
        out.update(dq=shared(dq) * sc, dk=shared(dk), dv=dv, dg=dg.sum((0, 1)) if case["fixed"] else dg)
        return out if S0 is None or s["S0"] is None else dict(out, dS0=R)
    if op.startswith("norm"):
        r = (d(s["x"]) + d(s["res"])).to(s["dtype"]).double()  # the stream is held in the model's type
        n, w = case["N"], d(s["w"])
        rms = torch.sqrt(torch.einsum("rn,rn->r", r, r) / n + s["eps"])[:, None]
        if op == "norm_fp8":
            y = (r / rms * w).view(case["rows"], -1, case["group"] or n)
            sc = y.abs().max(-1).values / FP8_MAX
            return {"q": (y / sc[..., None]).view(case["rows"], n), "scales": sc, "r": r}
        dy = d(s["grad_y"])
        c = torch.einsum("rn,rn->r", dy * w, r)[:, None] / (n * rms ** 3)
        return {"y": r / rms * w, "r": r, "dx": dy * w / rms - c * r + d(s["grad_r"]),
                "dw": torch.einsum("rn,rn->n", dy, r / rms)}
    total = math.fsum(float(torch.linalg.vector_norm(b.double()) ** 2) for _, b, _ in s["flat"])
    n = math.sqrt(total)
    c = min(1.0, s["max_norm"] / (n + 1e-6))
    return {"norm": torch.tensor(n, dtype=torch.float64), "clipped": [b.double() * c for _, b, _ in s["flat"]]}
