"""Inputs and 64-bit references of the tests of the gated recurrence, the norm of
queries and keys, and the embedding."""
import torch

# Half a step of a type, relative to the value: what one rounding may be off by.
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def check_each(name, got, ref, err):
    """Every element within one rounding to its type of the reference, and `err` (a number or a tensor) beside it."""
    g, r = got.detach().double().cpu(), ref.detach().double().cpu()
    assert g.shape == r.shape, (name, g.shape, r.shape)
    off = (g - r).abs() - HALF[got.dtype] * r.abs() * (1 + 2.0 ** -8) - err
    assert torch.isfinite(g).all(), name
    if off.numel():
        i = int(off.argmax())
        assert off.max() <= 0, f"{name}: element {i}: {g.flatten()[i].item():.8g}, not {r.flatten()[i].item():.8g}"


# ---------------------------------------------------------------- gated recurrence
def gated_inputs(B, T, D, dtype=torch.float32, h0=True, positive=True, seed=0, shift=2.0, halves=True):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    both = n(B, T, 2 * D)
    both[..., :D] += 1 - shift * 2 * torch.rand(D, generator=gen)  # memories of a step to some
    both = both.to(dtype)
    gate, value = both[..., :D], both[..., D:]
    if not halves:
        gate, value = gate.contiguous(), value.contiguous()
    return {"gate": gate, "value": value, "h0": n(B, D) if h0 else None, "grad_h": n(B, T, D).to(dtype),
            "grad_hT": n(B, D) if h0 else None, "positive": positive}


def gated_ref(d, grads=True):
    """Step by step in 64 bits, the gradients by the formulas."""
    k, v = d["gate"].double(), d["value"].double()
    B, T, D = k.shape
    z, a = torch.sigmoid(k), torch.sigmoid(-k)
    low = torch.sigmoid(v)
    c = torch.where(v >= 0, v + 0.5, low) if d["positive"] else v
    slope = torch.where(v >= 0, 1.0, low * (1 - low)) if d["positive"] else torch.ones_like(v)
    masked = k == -torch.inf
    c, slope = c.masked_fill(masked, 0), slope.masked_fill(masked, 0)
    h = torch.zeros(B, D, dtype=torch.float64) if d["h0"] is None else d["h0"].double()
    before, hs = [], []
    for t in range(T):
        before.append(h)
        h = a[:, t] * h + z[:, t] * c[:, t]
        hs.append(h)
    stack = lambda x: torch.stack(x, 1) if T else torch.zeros(B, 0, D, dtype=torch.float64)  # noqa: E731
    out = {"h": stack(hs), "h_T": h}
    if grads:
        lam, flow = [None] * T, torch.zeros(B, D, dtype=torch.float64)
        if d["grad_hT"] is not None:
            flow = d["grad_hT"].double()
        for t in range(T - 1, -1, -1):
            lam[t] = flow + d["grad_h"][:, t].double()
            flow = a[:, t] * lam[t]
        lam = out["lam"] = stack(lam)
        out["dvalue"], out["dgate"], out["dh0"] = lam * z * slope, lam * (c - stack(before)) * z * a, flow
    return out


# ---------------------------------------------------------------- norm of queries and keys
def qk_inputs(B, T, Hq, Hk, D, R, dtype=torch.float32, interleaved=False, rows=None, positions=True, seed=0):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    q, k, _ = (2 * n(B, T, (Hq + 2 * Hk) * D)).to(dtype).unflatten(-1, (Hq + 2 * Hk, D)).split([Hq, Hk, Hk], 2)
    rows = rows or 3 * T + 5
    at = torch.randint(0, rows, (B, T), generator=gen, dtype=torch.int32) if positions and R else None
    return {"q": q, "k": k, "wq": (1 + 0.3 * n(D)).to(dtype), "wk": (1 + 0.3 * n(D)).to(dtype), "at": at, "rows": rows,
            "R": R, "interleaved": interleaved, "grad_q": n(B, T, Hq, D).to(dtype), "grad_k": n(B, T, Hk, D).to(dtype)}


def angles(rows, R, base=10000.0):
    i = torch.arange(R // 2, dtype=torch.float64)
    return torch.arange(rows, dtype=torch.float64)[:, None] * base ** (-2 * i / R)


def qk_forward64(x, w, at, d, eps):
    """One of the two, in 64 bits; `at` [B,T] long."""
    R, D = d["R"], x.shape[-1]
    n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    if w is not None:
        n = n * w
    if R == 0:
        return n
    live = (at >= 0) & (at < d["rows"])
    ang = angles(d["rows"], R)[at.clamp(0, d["rows"] - 1)][:, :, None]
    c, s = ang.cos(), ang.sin()
    i = torch.arange(R // 2)
    e1, e2 = (2 * i, 2 * i + 1) if d["interleaved"] else (i, i + R // 2)
    y = n.clone()
    y[..., e1] = n[..., e1] * c - n[..., e2] * s
    y[..., e2] = n[..., e2] * c + n[..., e1] * s
    return y * live[:, :, None, None]


def qk_ref(d, eps=1e-6, grads=True):
    B, T = d["q"].shape[:2]
    at = torch.arange(T).expand(B, T) if d["at"] is None else d["at"].long()
    out = {}
    for n in ("q", "k"):
        x = d[n].double().requires_grad_(grads)
        w = None if d["w" + n] is None else d["w" + n].double().requires_grad_(grads)
        y = qk_forward64(x, w, at, d, eps)
        out[n] = y
        if grads:
            g = torch.autograd.grad((y * d["grad_" + n].double()).sum(), [x] + ([] if w is None else [w]),
                                    allow_unused=True, materialize_grads=True)
            out["d" + n] = g[0]
            out["dw" + n] = None if w is None else g[1]
    return out


# ---------------------------------------------------------------- embedding
def embed_inputs(N, V, D, dtype=torch.float32, kind=torch.int64, seed=0, few=False):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    # text: the r-th word about 1 / (r + 1) as often; few: all of a handful of words
    p = 1 / (torch.arange(V) + 1.0) if not few else (torch.arange(V) < 3).float() + 1e-12
    tokens = torch.multinomial(p, N, replacement=True, generator=gen) if N else torch.zeros(0, dtype=torch.int64)
    tokens = torch.randperm(V, generator=gen)[tokens].to(kind)
    return {"tokens": tokens, "W": n(V, D).to(dtype), "grad": n(N, D).to(dtype)}


def embed_grad_ref(tokens, grad, V, scale):
    """dW in 64 bits, the sums of the terms' magnitudes, and the terms' count."""
    t, g = tokens.flatten().long(), grad.reshape(-1, grad.shape[-1]).double()
    ok = (t >= 0) & (t < V)
    t, g = t[ok], g[ok]
    zero = torch.zeros(V, g.shape[-1], dtype=torch.float64)
    return (zero.index_add(0, t, g) * scale, zero.index_add(0, t, g.abs()) * abs(scale),
            torch.zeros(V).index_add(0, t, torch.ones(len(t)))[:, None])
