"""The example's serving on the CPU, with plain forms in the place of the library's
operators: batches with empty rows, sequences longer than the model was made for."""
import pytest
import torch

from examples import linear_attention_lm as ex
from scan_linear_recurrences_gb300 import api


def _norm(x, w, res=None):
    r = x if res is None else x + res
    return r * torch.rsqrt(r.square().mean(-1, keepdim=True) + 1e-6) * w, r, None


def _qk_norm(q, k, wq, wk, table, positions=None):
    if positions is None:
        assert len(table) >= q.shape[1]
        positions = torch.arange(q.shape[1]).expand(q.shape[:2])
    assert positions.dtype in (torch.int32, torch.int64) and positions.shape == q.shape[:-2]
    R, live = table.shape[1], (positions >= 0) & (positions < len(table))
    c, s = table[positions.long().clamp(0, len(table) - 1)][..., None, :].split(R // 2, -1)

    def one(x, w):
        n, _, _ = _norm(x, w)
        n1, n2, rest = n.split([R // 2, R // 2, x.shape[-1] - R], -1)
        return torch.cat([n1 * c - n2 * s, n2 * c + n1 * s, rest], -1) * live[..., None, None]

    return one(q, wq), one(k, wk)


def _step(q, k, v, g, S, slots, scale):
    """One token of each sequence on the cache S; an empty row's output is zero."""
    out, n = torch.zeros_like(v), v.shape[1] // q.shape[1]
    for b, slot in enumerate(slots.tolist()):
        if 0 <= slot < len(S):
            S[slot] = g[b].exp()[:, None, None] * S[slot] + k[b].repeat_interleave(n, 0)[:, :, None] * v[b][:, None]
            out[b] = scale * (S[slot] * q[b].repeat_interleave(n, 0)[:, :, None]).sum(1)
    return out


def _attention(q, k, v, g, scale, want_state):
    B, T, H, D = v.shape
    S, o = torch.zeros(B, H, D, D), []
    for t in range(T):
        o.append(_step(q[:, t], k[:, t], v[:, t], g[:, t], S, torch.arange(B), scale))
    return torch.stack(o, 1), S


@pytest.fixture
def model(monkeypatch):
    table = api.rotary_table
    for name, fn in (("rotary_table", lambda n, R, base=10000.0, device=None: table(n, R, base, "cpu")),
                     ("rms_norm_fwd", _norm), ("qk_norm_fwd", _qk_norm), ("linear_attention_fwd", _attention),
                     ("linear_attention_step", _step), ("embedding_fwd", lambda t, w: w[t]),
                     ("rms_norm_fp8_fwd", lambda x, w, res: (_norm(x, w, res)[0], 1.0, x + res))):
        monkeypatch.setattr(api, name, fn)
    torch.manual_seed(0)

    def make(length):
        m = ex.Model(vocab=16, width=32, layers=2, heads=2, kv_heads=1, D=16, length=length)
        for layer in m.layers:
            layer.freeze()
        return m.requires_grad_(False)

    return make


def _same(a, b):
    # sums of some dozen terms of about one in fp32, in other orders
    assert (a - b).abs().max() <= 1e-4, (a - b).abs().max()


def test_empty_rows_leave_every_user_as_it_was(model):
    m, gen = model(64), torch.Generator().manual_seed(1)
    text = torch.randint(16, (3, 9), generator=gen)
    users = torch.tensor([1, 2, 0], dtype=torch.int32)
    cache, padded = m.cache(3), m.cache(3)
    m.serve(text[:, :6], cache, users)
    # the same prompts, one batch of them with a row that is nobody's
    m.serve(torch.cat([text[:1, :6], text[2:, :6] * 0]), padded, torch.tensor([1, -1], dtype=torch.int32))
    m.serve(text[1:, :6], padded, users[1:])
    for t in range(6, 9):
        want = m.serve(text[:, t], cache, users)
        # user 1 beside empty rows of both kinds, then the others beside one
        a = m.serve(torch.stack([text[2, 0], text[0, t], text[1, 0]]), padded, torch.tensor([-1, 1, 3], dtype=torch.int32))
        b = m.serve(torch.cat([text[1:, t], text[:1, 0]]), padded, torch.tensor([2, 0, -5], dtype=torch.int32))
        _same(a[1], want[0]), _same(b[:2], want[1:])


def test_sequences_longer_than_the_model_was_made_for(model):
    long, short = model(64), model(8)
    short.load_state_dict(long.state_dict())
    for layer in short.layers:
        layer.freeze()
    text, users = torch.randint(16, (2, 20), generator=torch.Generator().manual_seed(2)), torch.tensor([1, 0], dtype=torch.int32)
    want = long.serve(text, long.cache(2), users)
    _same(short.serve(text, short.cache(2), users), want)
    cache = short.cache(2)
    got = [short.serve(text[:, :5], cache, users)[:, -1]] + [short.serve(text[:, t], cache, users) for t in range(5, 20)]
    _same(torch.stack(got, 1), want[:, 4:])
