"""Long generation in a bounded context: a two-layer hybrid model with random weights, on the
library's calls.

Layer 1 is linear attention with one decay per head (fp32 states in a slot pool), layer 2 softmax
attention over a paged 8-bit cache. Ragged prompts run in one pass; then tokens are decoded one at
a time. The cache keeps a weight per token and head: what attention has given it so far. When a
row's cache reaches its limit it is cut down to a budget of the tokens with the largest weights,
beside the first and the latest ones, moved into fresh pages; the old pages are free again.

    python examples/bounded_context.py

`check()` compares the run without a limit with one token at a time, and with a run that moves
every token it has, which must not change anything.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from linear_attention_state_kda_gb300 import kda  # noqa: E402

H, HK = 4, 2                       # linear attention: value heads, heads of queries and keys
HQ, HKV, D = 8, 2, 128             # softmax attention; the head width of both
HID, VOCAB, ROT, N_POS = 512, 1003, 64, 4096
LATEST, SINKS, RECENT = 16, 4, 32  # prompt tokens that weigh the cache; tokens kept at both ends


class Model:
    def __init__(self, device, seed=0):
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)

        def w(*shape, std):
            return (torch.randn(*shape, generator=gen, device=device) * std).bfloat16()

        self.emb = w(VOCAB, HID, std=1.0)
        self.lin_in = w(HID, (2 * HK + H) * D, std=HID ** -0.5)
        self.lin_gate = w(HID, H, std=HID ** -0.5)
        self.lin_out = w(H * D, HID, std=(H * D) ** -0.5)
        self.attn_in = w(HID, (HQ + 2 * HKV) * D, std=HID ** -0.5)
        self.attn_out = w(HQ * D, HID, std=(HQ * D) ** -0.5)
        self.norm = [1 + 0.1 * torch.randn(D, generator=gen, device=device) for _ in range(2)]
        self.head = w(HID, VOCAB, std=2.0 * HID ** -0.5)
        ang = torch.arange(N_POS, device=device)[:, None] * \
            10000.0 ** (-torch.arange(0, ROT, 2, device=device) / ROT)
        self.cos_sin = torch.cat([ang.cos(), ang.sin()], 1).float()

    def linear_inputs(self, x):
        """q, k, v (views of one projection) and log-decays of layer 1."""
        qkv = (x @ self.lin_in).reshape(-1, 2 * HK + H, D)
        q, k = kda.head_norm_rope(qkv[:, :HK], qkv[:, HK:2 * HK], l2=True)
        g = -torch.nn.functional.softplus((x @ self.lin_gate).float() - 2)
        return q, k, qkv[:, 2 * HK:], g

    def attention_inputs(self, x, pos):
        qkv = (x @ self.attn_in).reshape(-1, HQ + 2 * HKV, D)
        q, k = kda.head_norm_rope(qkv[:, :HQ], qkv[:, HQ:HQ + HKV], *self.norm,
                                  cos_sin=self.cos_sin, positions=pos)
        return q, k, qkv[:, HQ + HKV:]


class Context:
    """What a batch keeps: a state slot per row; pages, of which a row has two sets in turn, and a
    weight per cached token and head; cached tokens and the position of the next one."""

    def __init__(self, batch, max_len, device):
        cols = -(-max_len // kda.PAGE)
        n = 2 * batch * cols
        self.pool = torch.zeros(batch, H, D, D, device=device)
        self.slots = torch.arange(batch, dtype=torch.int32, device=device)
        self.tables = torch.randperm(n, device=device).to(torch.int32).reshape(2, batch, cols)
        code = torch.zeros(n, HKV, kda.PAGE, D, dtype=torch.float8_e4m3fn, device=device)
        scale = torch.zeros(n, HKV, device=device)
        self.k, self.kv = (code, scale), (code, scale, code.clone(), scale.clone())
        self.weights = torch.zeros(n, HKV, kda.PAGE, device=device)
        self.length = torch.zeros(batch, dtype=torch.int32, device=device)
        self.position = torch.zeros(batch, dtype=torch.int32, device=device)

    def evict(self, budget):
        new = self.tables[1].contiguous()
        self.length, kept = kda.cache_evict(
            self.length, self.tables[0].contiguous(), new, *self.kv, self.weights, budget,
            sinks=min(SINKS, budget), recent=min(RECENT, budget - min(SINKS, budget)))
        self.tables = self.tables.flip(0)
        return kept


def prompt(m, c, tokens, lens):
    """Runs ragged prompts (tokens [B, W] padded, lens [B]) into an empty context; the logits of
    each row's last token."""
    B, W = tokens.shape
    real = torch.arange(W, device=tokens.device)[None] < lens[:, None]
    cu = torch.nn.functional.pad(lens.cumsum(0), (1, 0)).to(torch.int32)
    pos = torch.arange(W, device=tokens.device).expand(B, W)[real].to(torch.int32)
    x = m.emb[tokens[real].long()]
    o, c.pool = kda.decay_prefill(*m.linear_inputs(x), cu_seqlens=cu, scale=D ** -0.5)
    x = x + o.reshape(-1, H * D) @ m.lin_out
    q, k, v = m.attention_inputs(x, pos)
    table = c.tables[0].contiguous()
    kda.cache_write(k, v, c.length, table, *c.kv, cu_seqlens=cu)
    padded = q.new_zeros(B, W, HQ, D)
    padded[real] = q
    o = kda.cache_attention(padded, c.length, table, *c.kv, scale=D ** -0.5, lens=lens)
    x = x + o[real].reshape(-1, HQ * D) @ m.attn_out
    # the latest tokens weigh the prompt
    n = lens.clamp(max=LATEST)
    at = (lens - n)[:, None] + torch.arange(LATEST, device=lens.device)
    last = padded.gather(1, at.clamp(max=W - 1)[:, :, None, None].expand(-1, -1, HQ, D).long())
    kda.cache_weigh(last, (lens - n).to(torch.int32), table, *c.k, c.weights, scale=D ** -0.5, lens=n,
                    keep=0.0)
    c.length, c.position = lens.clone(), lens.clone()
    return (x[cu[1:].long() - 1] @ m.head).float()


def step(m, c, tokens):
    """Decodes one token of each row (tokens [B]); its logits."""
    x = m.emb[tokens.long()]
    o = kda.decay_window(*m.linear_inputs(x), c.slots, c.slots[:, None], c.pool, scale=D ** -0.5)
    x = x + o.reshape(-1, H * D) @ m.lin_out
    q, k, v = m.attention_inputs(x, c.position)
    table = c.tables[0].contiguous()
    cu = torch.arange(len(tokens) + 1, dtype=torch.int32, device=tokens.device)
    kda.cache_write(k, v, c.length, table, *c.kv, cu_seqlens=cu)
    o = kda.cache_attention(q, c.length, table, *c.kv, scale=D ** -0.5)
    kda.cache_weigh(q, c.length, table, *c.k, c.weights, scale=D ** -0.5)
    c.length, c.position = c.length + 1, c.position + 1
    return ((x + o.reshape(-1, HQ * D) @ m.attn_out) @ m.head).float()


def generate(m, tokens, lens, follow, limit=None, budget=None, device="cuda"):
    """Logits of the prompts' last tokens and of the tokens `follow` [B, steps] after them. A cache
    of `limit` tokens is cut down to `budget`."""
    c = Context(len(lens), tokens.shape[1] + follow.shape[1], device)
    out, cuts = [prompt(m, c, tokens, lens)], 0
    for i in range(follow.shape[1]):
        if limit is not None and int(c.length.max()) >= limit:
            c.evict(budget)
            cuts += 1
        out.append(step(m, c, follow[:, i]))
    return torch.stack(out, 1), c, cuts


def draw(lens, steps, device, seed=1):
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    tokens = torch.randint(0, VOCAB, (len(lens), max(lens)), generator=gen, device=device)
    follow = torch.randint(0, VOCAB, (len(lens), steps), generator=gen, device=device)
    return tokens.int(), torch.tensor(lens, dtype=torch.int32, device=device), follow.int()


def check(device="cuda"):
    """(prompts against single tokens, moved against unmoved: largest relative differences of the
    logits; cached tokens of a bounded run, its cuts)."""
    m = Model(device)
    tokens, lens, follow = draw([150, 1, 70, 40], 24, device)
    whole, _, _ = generate(m, tokens, lens, follow, device=device)
    moved, _, cuts = generate(m, tokens, lens, follow, limit=0, budget=192, device=device)
    assert cuts == follow.shape[1]
    # one token at a time, rows that begin later waiting
    alone = 0.0
    for b, n in enumerate(lens.tolist()):
        c = Context(1, n + follow.shape[1], device)
        row = torch.cat([tokens[b, :n], follow[b]])
        got = torch.stack([step(m, c, row[i:i + 1])[0] for i in range(len(row))])[n - 1:]
        alone = max(alone, float((got - whole[b]).abs().max() / whole[b].abs().max()))
    bound, c, cuts = generate(m, tokens, lens, follow, limit=100, budget=64, device=device)
    assert bool(torch.isfinite(bound).all())
    return alone, float((moved - whole).abs().max()), c.length.tolist(), cuts


if __name__ == "__main__":
    alone, moved, length, cuts = check()
    print("prompts against single tokens: largest relative difference of logits %.3g" % alone)
    print("all tokens moved before each step: difference %.3g" % moved)
    print("bounded to 100 cached tokens: %d cuts, lengths %s" % (cuts, length))
