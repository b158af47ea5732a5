"""Inputs and 64-bit references of the language-model operators' tests."""
import math

import torch

# Tolerances (relative L2 of a whole output against the 64-bit reference).
# fp32 outputs: the library's own bound.  bf16 outputs: rounding to bf16 errs by
# 1.66e-3 in the root mean square and is granted 2^-9 = 1.95e-3; attention
# rounds an operand of its products too, and the two at worst add.
FP32 = 1e-5
U = 2.0 ** -9
BF16_ONE, BF16_TWO = 1.01 * U, 2.02 * U


def rel(got, ref):
    g, r = got.detach().double().cpu(), ref.detach().double().cpu()
    assert g.shape == r.shape, (g.shape, r.shape)
    if r.numel() == 0:
        return 0.0
    assert torch.isfinite(g).all()
    n = r.norm().item()
    d = (g - r).norm().item()
    return d / n if n > 0 else d


def check(name, got, ref, tol):
    e = rel(got, ref)
    assert e <= tol, f"{name}: rel_l2={e:.3e} (<= {tol:.1e})"


def check_rounded(name, got, ref, tol):
    """An output that is computed in fp32 and rounded once: compared with the reference rounded to its type."""
    check(name, got, ref.to(got.dtype), tol)


def attn_inputs(B, T, H, Hk, D, dtype=torch.float32, S0=True, fixed=False, seed=0, decay=0.1):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    rate = torch.exp(-torch.rand(H, generator=gen) * 4) * decay
    g = -rate if fixed else -rate * torch.nn.functional.softplus(n(B, T, H))
    return {"q": n(B, T, Hk, D).to(dtype), "k": n(B, T, Hk, D).to(dtype), "v": n(B, T, H, D).to(dtype), "g": g,
            "S0": n(B, H, D, D) if S0 else None, "grad_o": n(B, T, H, D).to(dtype),
            "grad_ST": n(B, H, D, D) * 0.3 if S0 else None}


def attn_forward64(q, k, v, g, S0, scale):
    """The recurrence, step by step."""
    (B, T, Hk, D), H = q.shape, v.shape[2]
    q, k = (x.repeat_interleave(H // Hk, 2) for x in (q, k))
    a = g.exp().expand(B, T, H)
    S = S0 if S0 is not None else torch.zeros(B, H, D, D, dtype=torch.float64)
    o = []
    for t in range(T):
        S = a[:, t, :, None, None] * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        o.append(scale * (S * q[:, t, :, :, None]).sum(2))
    return (torch.stack(o, 1) if T else torch.zeros(B, 0, H, D, dtype=torch.float64)), S


def attn_ref(d, scale=None, grads=True):
    """Outputs and gradients in 64 bits (the gradients by automatic differentiation of the recurrence)."""
    scale = d["q"].shape[-1] ** -0.5 if scale is None else scale
    x = {n: d[n].double().requires_grad_(grads) for n in ("q", "k", "v", "g", "S0") if d[n] is not None}
    o, ST = attn_forward64(x["q"], x["k"], x["v"], x["g"], x.get("S0"), scale)
    out = {"o": o, "S_T": ST}
    if grads:
        L = (o * d["grad_o"].double()).sum()
        if d["grad_ST"] is not None:
            L = L + (ST * d["grad_ST"].double()).sum()
        names = list(x)
        for n, gr in zip(names, torch.autograd.grad(L, [x[n] for n in names])):
            out["d" + n] = gr
    return out


def cuda(d):
    return {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in d.items()}


def norm_ref(x, w, res, eps, dtype, gy=None, gr=None):
    """y, r, rstd (and dx, dw) in 64 bits, r rounded to the type."""
    r = x.double() if res is None else (x.float() + res.float()).to(dtype).double()
    rstd = 1 / torch.sqrt((r * r).mean(-1, keepdim=True) + eps)
    hat = r * rstd
    out = {"y": hat * w.double(), "r": r, "rstd": rstd[..., 0]}
    if gy is not None:
        gy = gy.double()
        wg = gy * w.double()
        out["dx"] = rstd * (wg - hat * (wg * hat).mean(-1, keepdim=True)) + (gr.double() if gr is not None else 0)
        out["dw"] = (gy * hat).reshape(-1, x.shape[-1]).sum(0)
    return out


def fp8_values():
    """All finite non-negative e4m3 values, ascending."""
    v = [math.ldexp(m, -9) for m in range(8)]
    v += [math.ldexp(8 + m, e - 10) for e in range(1, 16) for m in range(8) if not (e == 15 and m == 7)]
    return torch.tensor(v, dtype=torch.float64)
