"""A small language model on linear attention: trained, then used token by token.

Tokens are looked up by embedding, whose gradient is summed by sorted tokens; every
layer is  r += attention(norm(r)),  r += mlp(norm(r))  with
  * rms_norm, which adds the residual and normalises in one pass,
  * qk_norm, which normalises each head of the queries and keys (to unit length to
    begin with, so that the state stays bounded) and turns half of it by its position,
  * linear_attention with a learned decay for each head and step,
  * clip_grad_norm over all gradients before the optimiser's step,
and answers with
  * linear_attention_fwd over the prompt, which leaves each layer's state in a cache,
  * linear_attention_step for each new token, on the cache's rows of its users,
  * rms_norm_fp8_fwd in front of the mlp, whose weights are kept in 8 bits.

The text is synthetic: each sequence is written in a few words of its own, drawn
from the vocabulary, so that what is likely next has to be remembered.

    python -m examples.linear_attention_lm [--steps 200]
"""
import argparse
import math

import torch
from torch.nn import functional as F

from scan_linear_recurrences_gb300 import api

FP8_MAX = 448.0


class Layer(torch.nn.Module):
    def __init__(self, width, heads, kv_heads, D):
        super().__init__()
        self.q_norm = torch.nn.Parameter(torch.full((D,), D ** -0.5))
        self.k_norm = torch.nn.Parameter(torch.full((D,), D ** -0.5))
        self.H, self.Hk, self.D = heads, kv_heads, D
        self.norm1 = torch.nn.Parameter(torch.ones(width))
        self.norm2 = torch.nn.Parameter(torch.ones(width))
        self.qkv = torch.nn.Linear(width, (2 * kv_heads + heads) * D, bias=False)
        self.gate = torch.nn.Linear(width, heads)
        self.out = torch.nn.Linear(heads * D, width, bias=False)
        self.up = torch.nn.Linear(width, 4 * width, bias=False)
        self.down = torch.nn.Linear(4 * width, width, bias=False)
        with torch.no_grad():  # decays a step between about 0.9 and 0.999 to begin with
            self.gate.weight.mul_(0.1)
            self.gate.bias.copy_(torch.linspace(-2.3, -7.0, heads))

    def project(self, y, norm, table, at=None):
        """q, k (normed and turned), v as a view of one product, and the decay's logarithm."""
        q, k, v = self.qkv(y).unflatten(-1, (-1, self.D)).split([self.Hk, self.Hk, self.H], -2)
        q, k = norm(q, k, self.q_norm, self.k_norm, table, at)
        return q, k, v, -F.softplus(self.gate(y).float())

    def forward(self, x, res, table):
        """x: what the layer before adds to the residual stream res (None: x is the stream)."""
        if res is None:
            y, res = api.rms_norm(x, self.norm1), x
        else:
            y, res = api.rms_norm(x, self.norm1, res)
        o, _ = api.linear_attention(*self.project(y, api.qk_norm, table), scale=1.0)
        y, res = api.rms_norm(self.out(o.flatten(-2)), self.norm2, res)
        return self.down(F.gelu(self.up(y))), res

    @torch.no_grad()
    def freeze(self):
        """The up projection in 8 bits, a scale for each of its rows."""
        w = self.up.weight.float()
        self.up_scale = w.abs().amax(1) / FP8_MAX
        self.up8 = (w / self.up_scale[:, None]).to(torch.float8_e4m3fn)

    @torch.no_grad()
    def serve(self, x, res, states, slots, place, table, at):
        """A prompt (x [B,T,width]: the states are left in their places) or one token of each sequence ([B,width])."""
        if res is None:
            y, res = api.rms_norm_fwd(x, self.norm1)[0], x
        else:
            y, res, _ = api.rms_norm_fwd(x, self.norm1, res)
        q, k, v, g = self.project(y, api.qk_norm_fwd, table, at)
        if x.dim() == 3:
            o, S = api.linear_attention_fwd(q, k, v, g, scale=1.0, want_state=True)
            states[place] = S
        else:
            o = api.linear_attention_step(q, k, v, g, states[:-1], slots, scale=1.0)
        y8, scale, res = api.rms_norm_fp8_fwd(self.out(o.flatten(-2)), self.norm2, res)
        # the product of 8-bit operands, scaled by rows and columns (here in 32 bits)
        up = (y8.float() @ self.up8.float().T) * scale * self.up_scale
        return self.down(F.gelu(up.to(x.dtype))), res


class Model(torch.nn.Module):
    def __init__(self, vocab=64, width=256, layers=2, heads=4, kv_heads=2, D=64, length=4096):
        super().__init__()
        self.length, self.turned, self.table = length, D // 2, None  # (the table stays in fp32, beside the parameters)
        self.embed = torch.nn.Embedding(vocab, width)
        self.layers = torch.nn.ModuleList(Layer(width, heads, kv_heads, D) for _ in range(layers))
        self.norm = torch.nn.Parameter(torch.ones(width))
        self.head = torch.nn.Linear(width, vocab, bias=False)
        torch.nn.init.normal_(self.embed.weight, std=0.5)

    def places(self, n):
        """The rotations of the places 0 .. n - 1: of `length` of them, until a longer sequence needs more."""
        if self.table is None or len(self.table) < n or self.table.device != self.norm.device:
            self.table = api.rotary_table(max(n, self.length), self.turned, device=self.norm.device)
        return self.table

    def places_of(self, at):
        """The rotations of these places, a row each: a sequence goes on for as long as it likes."""
        i = torch.arange(self.turned // 2, dtype=torch.float64, device=at.device)
        angle = at.double()[:, None] * 10000.0 ** (-2 * i / self.turned)
        return torch.cat([angle.cos(), angle.sin()], 1).float()

    def forward(self, tokens):
        x, res, table = api.embedding(tokens, self.embed.weight), None, self.places(tokens.shape[1])
        for layer in self.layers:
            x, res = layer(x, res, table)
        return self.head(api.rms_norm(x, self.norm, res)[0])

    def cache(self, users):
        """A state for each layer, user and head, and how many tokens each user's have seen; behind the users' a spare
        place, for what empty rows leave."""
        L = self.layers[0]
        states = [torch.zeros(users + 1, L.H, L.D, L.D, device=self.norm.device) for _ in self.layers]
        return [*states, torch.zeros(users + 1, dtype=torch.int32, device=self.norm.device)]

    @torch.no_grad()
    def serve(self, tokens, cache, slots):
        """Logits after the prompts [B,T], or after one more token [B], of the users in `slots` (int32 [B]).  A slot that
        is no user's, such as -1, marks an empty row of the batch: its logits mean nothing."""
        *states, seen = cache
        users = len(seen) - 1
        live = (slots >= 0) & (slots < users)
        place = torch.where(live, slots, users).long()
        if tokens.dim() == 2:  # a prompt begins at the first place
            table, at = self.places(tokens.shape[1]), None
            seen[place] = tokens.shape[1]
        else:
            table, at = self.places_of(seen[place]), torch.arange(len(slots), dtype=torch.int32, device=slots.device)
            seen[place] += 1
        x, res = api.embedding_fwd(tokens.contiguous(), self.embed.weight), None
        for layer, S in zip(self.layers, states):
            x, res = layer.serve(x, res, S, slots, place, table, at)
        return self.head(api.rms_norm_fwd(x, self.norm, res)[0])


def texts(B, T, vocab, gen, words=4):
    """Sequences of `words` tokens each, and those tokens."""
    own = torch.rand(B, vocab, generator=gen).argsort(1)[:, :words]
    return own.gather(1, torch.randint(words, (B, T), generator=gen)).cuda(), own.cuda()


def train(model, steps, B=16, T=192, lr=2e-3, max_norm=1.0, seed=0):
    """Returns the loss of each step."""
    gen = torch.Generator().manual_seed(seed)
    vocab = model.embed.num_embeddings
    opt = torch.optim.AdamW(model.parameters(), lr=lr, weight_decay=0.0)
    losses = []
    for _ in range(steps):
        text, _ = texts(B, T + 1, vocab, gen)
        loss = F.cross_entropy(model(text[:, :-1]).float().flatten(0, 1), text[:, 1:].flatten())
        opt.zero_grad()
        loss.backward()
        api.clip_grad_norm([p.grad for p in model.parameters()], max_norm)
        opt.step()
        losses.append(loss.detach())
    return torch.stack(losses).tolist()


def answer(model, prompts, tokens, slots, cache):
    """The `tokens` most likely tokens after each prompt, one step a token."""
    for layer in model.layers:
        layer.freeze()
    logits = model.serve(prompts, cache, slots)[:, -1]
    out = []
    for _ in range(tokens):
        out.append(logits.argmax(-1))
        logits = model.serve(out[-1], cache, slots)
    return torch.stack(out, 1)


def main(steps=200):
    torch.manual_seed(0)
    model = Model().to("cuda", torch.bfloat16)
    losses = train(model, steps)
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f} in {steps} steps ({math.log(64):.3f}: no memory, {math.log(4):.3f}: the best)")
    text, own = texts(6, 100, 64, torch.Generator().manual_seed(1))
    slots = torch.tensor([5, 0, 7, 2, 6, 3], dtype=torch.int32, device="cuda")  # six users of a cache for eight
    got = answer(model, text, 60, slots, model.cache(8))
    kept = (got[..., None] == own[:, None]).any(-1).float().mean().item()
    print(f"{kept:.0%} of the next 60 tokens in the prompt's words")
    return losses, kept


if __name__ == "__main__":
    args = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    args.add_argument("--steps", type=int, default=200)
    main(args.parse_args().steps)
