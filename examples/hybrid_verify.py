"""Speculative decoding of a two-layer hybrid model with random weights, on the library's calls.

Layer 1 is a KDA layer (fp32 state in a slot pool, one snapshot per token of the window), layer 2
softmax attention over a paged 8-bit cache. Each step runs a window of the last token and the
drafts through both layers, verifies the drafts, and goes on from the accepted tokens: the state
from the slot that the verification names, the cache by its length alone (rejected tokens are
overwritten by the next window).

    python examples/hybrid_verify.py

`check()` also runs the tokens that came out one at a time and compares the logits.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from linear_attention_state_kda_gb300 import kda  # noqa: E402

H, HQ, HKV, D = 4, 8, 2, 128       # KDA heads; query and key/value heads of the attention layer
HID, VOCAB, ROT, N_POS = 512, 1003, 64, 4096


class Model:
    def __init__(self, device, seed=0):
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)

        def w(*shape, std):
            return (torch.randn(*shape, generator=gen, device=device) * std).bfloat16()

        self.emb = w(VOCAB, HID, std=1.0)
        self.kda_in = w(HID, 3 * H * D, std=HID ** -0.5)
        self.kda_gate = w(HID, H * D, std=HID ** -0.5)
        self.kda_beta = w(HID, H, std=HID ** -0.5)
        self.kda_out = w(H * D, HID, std=(H * D) ** -0.5)
        self.attn_in = w(HID, (HQ + 2 * HKV) * D, std=HID ** -0.5)
        self.attn_out = w(HQ * D, HID, std=(HQ * D) ** -0.5)
        self.q_norm = 1 + 0.1 * torch.randn(D, generator=gen, device=device)
        self.k_norm = 1 + 0.1 * torch.randn(D, generator=gen, device=device)
        self.head = w(HID, VOCAB, std=2.0 * HID ** -0.5)
        ang = torch.arange(N_POS, device=device)[:, None] * \
            10000.0 ** (-torch.arange(0, ROT, 2, device=device) / ROT)
        self.cos_sin = torch.cat([ang.cos(), ang.sin()], 1).float()


class Cache:
    """What a batch keeps between steps: KDA states in slots, pages of keys and values, lengths."""

    def __init__(self, batch, window, max_len, device):
        pages = -(-(max_len + window) // kda.PAGE)
        self.window = window
        # per row: two sets of window slots, used in turn (a window reads a slot of the last set)
        self.pool = torch.zeros(batch * 2 * window, H, D, D, device=device)
        self.slots = torch.arange(batch * 2 * window, dtype=torch.int32, device=device) \
            .reshape(batch, 2, window)
        self.turn = 0
        self.read = self.slots[:, 1, 0].contiguous()  # zeros: the state before the first token
        n = batch * pages
        self.table = torch.randperm(n, device=device).to(torch.int32).reshape(batch, pages)
        code = torch.zeros(n, HKV, kda.PAGE, D, dtype=torch.float8_e4m3fn, device=device)
        scale = torch.zeros(n, HKV, device=device)
        self.kv = (code, scale, code.clone(), scale.clone())
        self.length = torch.zeros(batch, dtype=torch.int32, device=device)
        self.cu = torch.arange(batch + 1, dtype=torch.int32, device=device) * window

    def write_slots(self):
        return self.slots[:, self.turn].contiguous()


def forward(m, c, tokens):
    """Logits [B, W, V] of windows `tokens` [B, W] after what the cache holds."""
    B, W = tokens.shape
    x = m.emb[tokens.long()].reshape(B * W, HID)
    # KDA layer: 2-norm of q and k, then the window over the slot pool
    qkv = (x @ m.kda_in).reshape(B * W, 3 * H, D)
    q, k = kda.head_norm_rope(qkv[:, :H], qkv[:, H:2 * H], l2=True)
    g = -torch.nn.functional.softplus((x @ m.kda_gate).float()).reshape(B * W, H, D)
    o = kda.decode_window(q, k, qkv[:, 2 * H:].contiguous(), g, (x @ m.kda_beta).float(), c.read,
                          c.write_slots(), c.pool, scale=D ** -0.5, beta_is_logit=True)
    x = x + o.reshape(B * W, H * D) @ m.kda_out
    # attention layer: norm and rotation, append to the cache, attend
    qkv = (x @ m.attn_in).reshape(B * W, HQ + 2 * HKV, D)
    pos = (c.length[:, None] + torch.arange(W, dtype=torch.int32, device=x.device)).reshape(-1)
    q, k = kda.head_norm_rope(qkv[:, :HQ], qkv[:, HQ:HQ + HKV], m.q_norm, m.k_norm,
                              cos_sin=m.cos_sin, positions=pos)
    kda.cache_write(k, qkv[:, HQ + HKV:], c.length, c.table, *c.kv, cu_seqlens=c.cu)
    o = kda.cache_attention(q, c.length, c.table, *c.kv, scale=D ** -0.5)
    x = x + o.reshape(B * W, HQ * D) @ m.attn_out
    return (x @ m.head).float().reshape(B, W, VOCAB)


def generate(m, batch=5, drafts=3, steps=6, device="cuda", seed=1):
    """Runs `steps` windows. Returns per row the tokens (the first one included) and the target's
    logits at each of them but the last."""
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    c = Cache(batch, drafts + 1, (drafts + 1) * (steps + 1), device)
    bigram = torch.softmax(2 * torch.randn(VOCAB, VOCAB, generator=gen, device=device), -1)
    last = torch.randint(0, VOCAB, (batch,), generator=gen, device=device)
    out = [[int(t)] for t in last]
    logits_out = [[] for _ in out]
    for _ in range(steps):
        # drafts from a bigram table: a stand-in for a draft model
        window, probs = [last], []
        for _ in range(drafts):
            probs.append(bigram[window[-1]])
            window.append(torch.multinomial(probs[-1], 1, generator=gen)[:, 0])
        tokens = torch.stack(window, 1).to(torch.int32)
        logits = forward(m, c, tokens)
        n, new, resume = kda.draft_verify(
            torch.softmax(logits, -1), tokens[:, 1:].contiguous(),
            torch.rand(batch, drafts, generator=gen, device=device),
            torch.rand(batch, generator=gen, device=device),
            draft_probs=torch.stack(probs, 1), write_slots=c.write_slots())
        c.read, c.turn = resume, 1 - c.turn
        c.length = c.length + n + 1
        last = new.gather(1, n[:, None].long())[:, 0].long()
        for b, k in enumerate(n.tolist()):
            out[b] += new[b, :k + 1].tolist()
            logits_out[b] += list(logits[b, :k + 1])
    return out, logits_out


def check(device="cuda"):
    """The largest difference between the logits of the verified windows and those of the same
    tokens run one at a time, over the largest logit."""
    m = Model(device)
    out, logits = generate(m, device=device)
    worst = 0.0
    for tokens, want in zip(out, logits):
        c = Cache(1, 1, len(tokens) + 1, device)
        for t, y in zip(tokens[:-1], want):
            got = forward(m, c, torch.tensor([[t]], dtype=torch.int32, device=device))[0, 0]
            worst = max(worst, float((got - y).abs().max() / y.abs().max()))
            c.read, c.turn = c.write_slots()[:, 0].contiguous(), 1 - c.turn
            c.length = c.length + 1
    return out, worst


if __name__ == "__main__":
    rows, diff = check()
    for r in rows:
        print(len(r) - 1, "tokens:", r)
    print("windows against single tokens: largest relative difference of logits %.3g" % diff)
