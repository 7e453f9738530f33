"""Cases of the operators that serve contexts of any length in bounded memory: linear attention with
one decay per head (prompts in chunks, tokens and verify windows over a slot pool), and eviction
from the paged 8-bit cache by accumulated attention weight (weighing, then compaction).

``run`` computes an operator in its plain form (elementary torch operations in 32 bits), or, with
``own`` set, through the library's binding. ``exact`` is the definition in 64 bits.
"""
import math
import random

import torch

own = False

BLOCK = 64      # tokens of a cache page: one scale for each (page, head)
FP8_MAX = 448.0
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


def listed():
    return [
        # a short prompt of a small model: latency only
        dict(name="prefill_77", op="prefill", n=1, len=77, H=4, Hk=4, d=64, const=False, init=True,
             dtype="bf16"),
        # a 16k-token prompt, decay per token and head
        dict(name="prefill_16k", op="prefill", n=1, len=16384, H=32, Hk=32, d=128, const=False,
             init=True, dtype="bf16"),
        # a batch of ragged prompts, constant decay per head, queries and keys shared by four heads
        dict(name="prefill_ragged_40", op="prefill", n=40, len=1000, H=16, Hk=4, d=128, const=True,
             init=False, dtype="bf16"),
        # fp32, a few ragged sequences of odd lengths
        dict(name="prefill_f32_5", op="prefill", n=5, len=1301, H=6, Hk=3, d=64, const=False,
             init=True, dtype="f32"),
        # one token of three requests: latency only
        dict(name="window_3x1", op="window", n=3, W=1, H=8, Hk=8, d=128, const=False, dtype="bf16"),
        # one decode step of a serving batch
        dict(name="window_256x1", op="window", n=256, W=1, H=32, Hk=32, d=128, const=False,
             dtype="bf16"),
        # verify windows of four tokens, every column's state kept, keys shared by two heads
        dict(name="window_96x4", op="window", n=96, W=4, H=32, Hk=16, d=128, const=True,
             dtype="bf16"),
        # two requests with short contexts, one token each
        dict(name="weigh_2x100", op="weigh", n=2, W=1, ctx=100, Hq=32, Hkv=8, d=128, dtype="bf16"),
        # a serving batch, one token each, contexts of any length up to 16k
        dict(name="weigh_128x16k", op="weigh", n=128, W=1, ctx=16384, Hq=32, Hkv=8, d=128,
             dtype="bf16"),
        # the last 64 tokens of a 32k-token prompt weigh all of it, once, before it is cut down
        dict(name="weigh_prompt_32k", op="weigh", n=1, W=64, ctx=32768, Hq=32, Hkv=8, d=128,
             dtype="bf16"),
        # three short contexts cut to two pages
        dict(name="evict_3x500", op="evict", n=3, ctx=500, budget=128, sinks=4, recent=32, Hkv=8,
             d=64),
        # a serving batch, contexts up to 16k cut to 4k tokens each
        dict(name="evict_32x16k", op="evict", n=32, ctx=16384, budget=4096, sinks=4, recent=64,
             Hkv=8, d=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "window", "weigh", "evict"])
    d = rng.choice([64, 128, 128])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op in ("prefill", "window"):
        Hk = rng.choice([1, 2, 3, 4, 8, 16])
        H = Hk * rng.choice([1, 1, 2, 3])
        const = rng.random() < 0.4
    if op == "prefill":
        n = _log(rng, 1, 64)
        top = 16384 * 32 * 128 // (H * d * (4 if dtype == "f32" else 1))
        return dict(op=op, n=n, len=_log(rng, 1, max(1, min(16384, top // n))), H=H, Hk=Hk, d=d,
                    const=const, init=rng.random() < 0.5, dtype=dtype)
    if op == "window":
        W = rng.choice([1, 1, 1, 2, 3, 5, 8])
        return dict(op=op, n=_log(rng, 1, max(1, min(256, 256 * 32 * 2 // (H * (W + 1))))), W=W, H=H,
                    Hk=Hk, d=d, const=const, dtype=dtype)
    Hkv = rng.choice([1, 2, 3, 4, 8])
    n = _log(rng, 1, 128)
    if op == "weigh":
        W = rng.choice([1, 1, 1, 2, 4, 7, 16, 33, 64])
        G = rng.choice([1, 2, 3, 4, 5, 8])
        return dict(op=op, n=n, W=W, ctx=_log(rng, 1, min(131072, 2097152 // (n * W))), Hq=Hkv * G,
                    Hkv=Hkv, d=d, dtype=dtype)
    ctx = _log(rng, 1, min(131072, 32 * 16384 // n))
    budget = _log(rng, 1, min(8192, 32 * 4096 // n))
    return dict(op=op, n=n, ctx=ctx, budget=budget, sinks=min(budget // 4, rng.randint(0, 8)),
                recent=rng.randint(0, budget // 2), Hkv=Hkv, d=d)


# ---------------------------------------------------------------- inputs

def _gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed))
    return g


def _pages(gen, need, more=0):
    """A page table of `need` [n, max_pages] used entries: distinct pages in a shuffled order, -1
    where a row has none. Returns it, `more` further pages, and the number of pages of the pool."""
    used = int(need.sum())
    n_pages = used + more + 3
    perm = torch.randperm(n_pages, generator=gen, device="cuda")[:used + more].to(torch.int32)
    table = torch.full(need.shape, -1, dtype=torch.int32, device="cuda")
    table[need] = perm[:used]
    return table, perm[used:], n_pages


def _pow2_scale(amax):
    """Smallest power of two s with amax <= 448 s, at least 2^-100."""
    m, e = torch.frexp(amax)
    e = (e - 9 + (m > 0.875).to(e.dtype)).clamp(min=-100)
    e = torch.where(amax > 0, e, torch.full_like(e, -100))
    return ((e + 127) << 23).view(torch.float32)  # 2^e by its bits: exact


def _random_cache(gen, n_pages, H, d, spread):
    """Codes and scales of pages of ~N(0, spread) values, a few channels eight times larger, some
    pages larger than others."""
    codes = torch.empty(n_pages, H, BLOCK, d, dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty(n_pages, H, device="cuda")
    chan = 1.0 + 7.0 * (torch.rand(H, 1, d, generator=gen, device="cuda") < 0.02)
    step = max(1, (1 << 28) // (H * BLOCK * d))
    for i in range(0, n_pages, step):
        n = min(step, n_pages - i)
        size = torch.exp(0.3 * torch.randn(n, H, 1, 1, generator=gen, device="cuda"))
        x = torch.randn(n, H, BLOCK, d, generator=gen, device="cuda") * (spread * chan * size)
        s = _pow2_scale(x.abs().amax((2, 3)))
        codes[i:i + n] = (x / s[:, :, None, None]).to(torch.float8_e4m3fn)
        scale[i:i + n] = s
    return codes, scale


def _lengths(c):
    """Length of each row: by the case alone, so that every seed's outputs have the same shape.
    Ragged, the first of full length."""
    top = c["len"] if c["op"] == "prefill" else c["ctx"]
    rng = random.Random("%d %d" % (c["n"], top))
    return [top] + [rng.randint(1, top) for _ in range(c["n"] - 1)]


def prepare(case, seed):
    gen = _gen(seed)
    c = dict(case)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    uni = lambda *s: torch.rand(*s, generator=gen, device="cuda")  # noqa: E731
    st = {"case": c}
    if c["op"] in ("prefill", "window"):
        n, H, Hk, d = c["n"], c["H"], c["Hk"], c["d"]
        T = sum(_lengths(c)) if c["op"] == "prefill" else n * c["W"]
        dt = DT[c["dtype"]]
        qkv = torch.empty(T, 2 * Hk + H, d, dtype=dt, device="cuda")
        for i in range(0, T, 4096):
            x = rnd(min(4096, T - i), 2 * Hk + H, d)
            x[:, :2 * Hk] *= torch.sigmoid(x[:, :2 * Hk])  # queries and keys behind a SiLU
            qkv[i:i + 4096] = x.to(dt)
        # rows of the fused projection
        st["q"], st["k"], st["v"] = qkv[:, :Hk], qkv[:, Hk:2 * Hk], qkv[:, 2 * Hk:]
        # heads forget over 2 .. 1000 tokens
        rate = torch.exp2(-1.0 - 9.0 * torch.arange(H, device="cuda") / max(1, H - 1))
        st["g"] = -rate * (0.7 + 0.6 * uni(H)) if c["const"] else \
            -rate * torch.nn.functional.softplus(rnd(T, H))
        st["scale"] = d ** -0.5
        if c["op"] == "prefill":
            lens = torch.tensor([0] + _lengths(c), device="cuda")
            st["cu"] = lens.cumsum(0).to(torch.int32)
            st["init"] = rnd(n, H, d, d) if c["init"] else None
        else:
            W = c["W"]
            n_slots = n * (W + 1) + 5
            st["pool"] = rnd(n_slots, H, d, d)
            slots = torch.randperm(n_slots, generator=gen, device="cuda").to(torch.int32)
            st["read"] = slots[:n].contiguous()
            # a single token updates its state in place; a window keeps the state after each token
            st["write"] = st["read"][:, None].contiguous() if W == 1 else \
                slots[n:n * (W + 1)].reshape(n, W).contiguous()
        return st
    n, Hkv, d = c["n"], c["Hkv"], c["d"]
    ctx = torch.tensor(_lengths(c), dtype=torch.int32, device="cuda")
    new = c["W"] if c["op"] == "weigh" else 0
    top = -(-(c["ctx"] + new) // BLOCK)
    need = torch.arange(top, device="cuda")[None] * BLOCK < (ctx + new)[:, None]
    width = -(-c["budget"] // BLOCK) if c["op"] == "evict" else 0
    st["pages"], more, n_pages = _pages(gen, need, n * width)
    st["kc"], st["ks"] = _random_cache(gen, n_pages, Hkv, d, 0.9)
    st["start"] = ctx
    # weights so far: a few tokens hold most of them, many hold none that differ
    st["weights"] = torch.exp(2.0 * rnd(n_pages, Hkv, BLOCK) - 3.0)
    if c["op"] == "weigh":
        Hq = c["Hq"]
        st["q"] = (rnd(n * c["W"], Hq, d) * (0.5 + 1.5 * uni(1, Hq, 1))).to(DT[c["dtype"]])
        st["scale"], st["keep"] = d ** -0.5, 0.98
    else:
        st["weights"] *= (uni(n_pages, Hkv, BLOCK) < 0.8)
        st["vc"], st["vs"] = _random_cache(gen, n_pages, Hkv, d, 0.4)
        st["new_pages"] = more.reshape(n, width)
        zero = torch.zeros(1, dtype=torch.int32, device="cuda")
        kept = ctx.clamp(max=c["budget"])
        st["zeros"] = torch.zeros_like(ctx)
        st["read_cu"] = torch.cat([zero, kept.cumsum(0).to(torch.int32)])
        st["read_tokens"] = int(kept.sum())
    return st


# ---------------------------------------------------------------- plain forms

def _shared(x, H):
    """[.., Hk, d] queries or keys of their groups' heads: [.., H, d] in 32 bits."""
    return x.float().repeat_interleave(H // x.shape[-2], -2)


def _prefill(st, c):
    """Chunks of 128 tokens: products inside a chunk under the decays' lower triangle, the state
    before each chunk as a decayed sum of the chunks before it in its sequence."""
    H, d, C = c["H"], c["d"], 128
    lens = st["cu"].long().diff()
    chunks = (lens + C - 1) // C
    seq = torch.repeat_interleave(torch.arange(c["n"], device="cuda"), chunks)
    nth = torch.arange(seq.numel(), device="cuda") - (chunks.cumsum(0) - chunks)[seq]
    tok = (nth * C)[:, None] + torch.arange(C, device="cuda")
    real = tok < lens[seq][:, None]
    tok = torch.where(real, tok + st["cu"].long()[seq][:, None], 0)
    g = st["g"].double().expand(st["v"].shape[0], H)
    pick = lambda x: (x[tok] * real[..., None, None]).transpose(1, 2)  # noqa: E731  [N, H, C, d]
    q, k, v = pick(_shared(st["q"], H)), pick(_shared(st["k"], H)), pick(st["v"].float())
    dec = (g[tok] * real[..., None]).transpose(1, 2).cumsum(2)  # [N, H, C], 64 bits
    total = dec[..., -1]
    low = torch.ones(C, C, dtype=torch.bool, device="cuda").tril()
    w = torch.exp((dec[..., :, None] - dec[..., None, :]).masked_fill(~low, -math.inf).float())
    o = (q @ k.transpose(2, 3) * w) @ v
    own_state = (k * torch.exp((total[..., None] - dec).float())[..., None]).transpose(2, 3) @ v
    # decay from the end of chunk b to the start of chunk a of the same sequence
    upto = total.cumsum(0)
    reach = (upto - total)[:, None] - upto[None]
    order = torch.arange(seq.numel(), device="cuda")
    before = (seq[:, None] == seq) & (order[:, None] > order)
    m = torch.exp(reach.masked_fill(~before[..., None], -math.inf).float()).permute(2, 0, 1)
    s = (m @ own_state.transpose(0, 1).reshape(H, seq.numel(), d * d)).reshape(H, -1, d, d) \
        .transpose(0, 1)
    first = chunks.cumsum(0) - chunks
    if st["init"] is not None:
        since = (upto - total) - (upto - total)[first][seq]
        s = s + st["init"][seq] * torch.exp(since.float())[..., None, None]
    o = o + (q @ s) * torch.exp(dec.float())[..., None]
    last = first + chunks - 1
    final = s[last] * torch.exp(total[last].float())[..., None, None] + own_state[last]
    o = (o * st["scale"]).transpose(1, 2)[real]
    return o.to(st["v"].dtype), final


def _window(st, c):
    n, W, H, d = c["n"], c["W"], c["H"], c["d"]
    q, k = _shared(st["q"], H).reshape(n, W, H, d), _shared(st["k"], H).reshape(n, W, H, d)
    v = st["v"].float().reshape(n, W, H, d)
    dec = st["g"].expand(n * W, H).reshape(n, W, H).cumsum(1)
    s = st["pool"][st["read"].long()][:, None] * torch.exp(dec)[..., None, None]
    kv = k[..., :, None] * v[..., None, :]  # [n, W, H, d, d]
    low = torch.ones(W, W, dtype=torch.bool, device="cuda").tril()[None, :, :, None]
    w = torch.exp((dec[:, :, None] - dec[:, None]).masked_fill(~low, -math.inf))
    s = s + torch.einsum("nwuh,nuhk->nwhk", w, kv.flatten(-2)).unflatten(-1, (d, d))
    st["pool"][st["write"].long()] = s
    o = (q[..., None, :] @ s)[..., 0, :] * st["scale"]
    return o.reshape(n * W, H, d).to(st["v"].dtype), st["pool"]


def _weigh(st, c):
    n, W, Hq, Hkv, d = c["n"], c["W"], c["Hq"], c["Hkv"], c["d"]
    page = st["pages"].clamp(min=0).long()
    L = page.shape[1] * BLOCK
    k = st["kc"].view(torch.uint8)[page].view(torch.float8_e4m3fn).float()
    k = (k * st["ks"][page][..., None, None]).transpose(1, 2).reshape(n, Hkv, L, d)
    q = st["q"].float().reshape(n, W, Hkv, Hq // Hkv, d).permute(0, 2, 1, 3, 4)
    s = q.reshape(n, Hkv, -1, d) @ k.transpose(2, 3) * st["scale"]
    t = torch.arange(L, device="cuda")
    seen = t <= st["start"][:, None, None] + torch.arange(W, device="cuda")[:, None]
    s = s.reshape(n, Hkv, W, -1, L).masked_fill(~seen[:, None, :, None], -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    add = (p / p.sum(-1, keepdim=True)).sum((2, 3))  # [n, Hkv, L]
    row = torch.arange(n, device="cuda")[:, None]
    old = st["weights"][page].transpose(1, 2).reshape(n, Hkv, L)
    old = torch.where((t < st["start"][:, None])[:, None], old * st["keep"], 0.0)
    there = t < st["start"][:, None] + W
    row, at = there.nonzero(as_tuple=True)
    st["weights"][page[row, at // BLOCK], :, at % BLOCK] = (old + add)[row, :, at]
    return st["weights"]


def _evict(st, c):
    n, Hkv, d, m = c["n"], c["Hkv"], c["d"], c["budget"]
    page = st["pages"].clamp(min=0).long()
    L = page.shape[1] * BLOCK
    t = torch.arange(L, device="cuda")
    length = st["start"].long()[:, None]
    w = st["weights"][page].transpose(1, 2).reshape(n, Hkv, L)
    always = (t < c["sinks"]) | (t >= length - c["recent"])
    w = torch.where(always[:, None], math.inf, w)
    w = torch.where((t < length)[:, None], w, -math.inf)
    order = torch.sort(w, dim=-1, descending=True, stable=True)[1][..., :m]
    count = length.clamp(max=m)
    there = torch.arange(order.shape[-1], device="cuda") < count
    kept = torch.where(there[:, None], order, L).sort(-1)[0]
    kept = torch.nn.functional.pad(kept, (0, st["new_pages"].shape[1] * BLOCK - kept.shape[-1]),
                                   value=L)
    real = kept < L
    at = torch.where(real, kept, 0)
    src = page[torch.arange(n, device="cuda")[:, None, None], at // BLOCK]
    head = torch.arange(Hkv, device="cuda")[:, None]
    dst = st["new_pages"].long()
    out = []
    for codes, scale in ((st["kc"], st["ks"]), (st["vc"], st["vs"])):
        s0 = torch.where(real, scale[src, head], 0.0).reshape(n, Hkv, -1, BLOCK)
        s = s0.amax(-1)
        x = codes.view(torch.uint8)[src, head, at % BLOCK].view(torch.float8_e4m3fn).float()
        x = x.reshape(n, Hkv, -1, BLOCK, d) * (s0 / s.clamp(min=2.0 ** -100)[..., None])[..., None]
        x = x.to(torch.float8_e4m3fn)
        used = (torch.arange(dst.shape[1], device="cuda") * BLOCK < count).nonzero(as_tuple=True)
        codes.view(torch.uint8)[dst[used]] = x.view(torch.uint8).transpose(1, 2)[used]
        scale[dst[used]] = s.transpose(1, 2)[used]
        value = x.float() * s[..., None, None]
        value = value.reshape(n, Hkv, -1, d).transpose(1, 2).bfloat16()  # exact: 4 bits and a power
        out.append(value[torch.arange(value.shape[1], device="cuda") < count])
    moved = torch.where(real, st["weights"][src, head, at % BLOCK], 0.0)
    moved = moved.reshape(n, Hkv, -1, BLOCK).transpose(1, 2)
    st["weights"][dst[used]] = moved[used]
    kept = torch.where(real, kept, -1)[..., :m]
    return out[0], out[1], st["weights"], kept.to(torch.int32), count[:, 0].to(torch.int32)


def run(state):
    c, st = state["case"], state
    if own:
        from linear_attention_state_kda_gb300 import kda
    if c["op"] == "prefill":
        if own:
            return kda.decay_prefill(st["q"], st["k"], st["v"], st["g"], cu_seqlens=st["cu"],
                                     init_state=st["init"], scale=st["scale"])
        return _prefill(st, c)
    if c["op"] == "window":
        if own:
            o = kda.decay_window(st["q"], st["k"], st["v"], st["g"], st["read"], st["write"],
                                 st["pool"], scale=st["scale"])
            return o, st["pool"]
        return _window(st, c)
    if c["op"] == "weigh":
        if own:
            return kda.cache_weigh(st["q"], st["start"], st["pages"], st["kc"], st["ks"],
                                   st["weights"], scale=st["scale"], keep=st["keep"])
        return _weigh(st, c)
    if own:
        count, kept = kda.cache_evict(st["start"], st["pages"], st["new_pages"], st["kc"], st["ks"],
                                      st["vc"], st["vs"], st["weights"], c["budget"],
                                      sinks=c["sinks"], recent=c["recent"])
        k, v = kda.cache_read(st["zeros"], st["new_pages"], st["kc"], st["ks"], st["vc"], st["vs"],
                              st["read_tokens"], cu_seqlens=st["read_cu"])
        return k, v, st["weights"], kept, count
    return _evict(st, c)


# ---------------------------------------------------------------- definitions in 64 bits

def _exact_recurrence(q, k, v, g, init, lens, scale):
    """Token by token, all sequences side by side: q, k, v [n, L, H, d], g [n, L, H]. Yields each
    token's outputs and the states after it."""
    s = init.double().clone()
    for t in range(q.shape[1]):
        live = (t < lens)[:, None, None, None]
        new = s * torch.exp(g[:, t])[..., None, None] + k[:, t, :, :, None] * v[:, t, :, None, :]
        s = torch.where(live, new, s)
        yield torch.einsum("nhk,nhkv->nhv", q[:, t], s) * scale, s


def exact(case, seed):
    st = prepare(case, seed)
    c = st["case"]
    if c["op"] in ("prefill", "window"):
        n, H, d = c["n"], c["H"], c["d"]
        if c["op"] == "prefill":
            cu = st["cu"].tolist()
            lens = [b - a for a, b in zip(cu, cu[1:])]
            if max(lens) * (1.5e-4 + n * H * d * d * 2.0e-11) > 15:
                return None
        else:
            lens = [c["W"]] * n
            cu = [i * c["W"] for i in range(n + 1)]
        top = max(lens)

        def padded(x):
            x = x.double()
            rows = [torch.nn.functional.pad(x[a:b], [0, 0] * (x.dim() - 1) + [0, top - (b - a)])
                    for a, b in zip(cu, cu[1:])]
            return torch.stack(rows)

        T = st["v"].shape[0]
        heads = torch.arange(H, device="cuda") // (H // c["Hk"])
        q, k = padded(st["q"][:, heads]), padded(st["k"][:, heads])
        v, g = padded(st["v"]), padded(st["g"].expand(T, H))
        at = torch.tensor(lens, device="cuda")
        if c["op"] == "window":
            init = st["pool"][st["read"].long()]
            pool = st["pool"].double()
        else:
            init = torch.zeros(n, H, d, d, device="cuda") if st["init"] is None else st["init"]
        outs = torch.empty(n, top, H, d, dtype=torch.float64, device="cuda")
        s = init.double()
        for t, (o, s) in enumerate(_exact_recurrence(q, k, v, g, init, at, st["scale"])):
            outs[:, t] = o
            if c["op"] == "window":
                pool[st["write"][:, t].long()] = s
        o = torch.cat([outs[i, :m] for i, m in enumerate(lens)])
        return o, (pool if c["op"] == "window" else s)
    lens = _lengths(c)
    Hkv, d = c["Hkv"], c["d"]
    weights = st["weights"].double()

    def cached(codes, scale, b, length):
        page = st["pages"][b, :-(-length // BLOCK)].long()
        x = codes.view(torch.uint8)[page].view(torch.float8_e4m3fn).double()
        x = x * scale[page].double()[..., None, None]
        return page, x.transpose(0, 1).reshape(Hkv, -1, d)[:, :length]

    if c["op"] == "weigh":
        W, G = c["W"], c["Hq"] // Hkv
        if sum(lens) * Hkv * (G * W + 8) * d * 2.0e-12 > 15:
            return None
        for b, past in enumerate(lens):
            length = past + W
            page, k = cached(st["kc"], st["ks"], b, length)
            q = st["q"][b * W:(b + 1) * W].double().reshape(W, Hkv, G, d)
            s = torch.einsum("whgd,htd->hwgt", q, k) * st["scale"]
            later = torch.ones(W, length, dtype=torch.bool, device="cuda").triu(past + 1)
            p = torch.softmax(s.masked_fill(later[:, None], -math.inf), -1).sum((1, 2))
            t = torch.arange(length, device="cuda")
            old = weights[page[t // BLOCK], :, t % BLOCK]
            old[past:] = 0
            weights[page[t // BLOCK], :, t % BLOCK] = st["keep"] * old + p.T
        return weights
    out = [[], []]
    kept_all = torch.full((c["n"], Hkv, c["budget"]), -1, dtype=torch.int32, device="cuda")
    table = st["new_pages"].tolist()
    for b, length in enumerate(lens):
        count = min(length, c["budget"])
        page, _ = cached(st["kc"], st["ks"], b, length)
        w = weights[page].transpose(0, 1).reshape(Hkv, -1)[:, :length]
        fixed = set(range(min(c["sinks"], length))) | set(range(max(0, length - c["recent"]), length))
        free = torch.tensor([t for t in range(length) if t not in fixed], dtype=torch.long,
                            device="cuda")
        fixed = torch.tensor(sorted(fixed), dtype=torch.long, device="cuda")
        want = count - fixed.numel()
        sides = []
        for h in range(Hkv):
            # the heaviest first, of equal ones the earliest
            rank = torch.argsort(-w[h, free], stable=True)[:max(0, want)]
            keep = torch.cat([fixed, free[rank]]).sort()[0]
            kept_all[b, h, :count] = keep.to(torch.int32)
            sides.append(keep)
        for side, (codes, scale) in enumerate(((st["kc"], st["ks"]), (st["vc"], st["vs"]))):
            page, x = cached(codes, scale, b, length)
            value = torch.empty(count, Hkv, d, dtype=torch.float64, device="cuda")
            for h, keep in enumerate(sides):
                for i in range(0, count, BLOCK):
                    at = keep[i:i + BLOCK]
                    s = scale[page[at // BLOCK], h].max().double()
                    code = (x[h, at] / s).float().to(torch.float8_e4m3fn)  # exact up to the code
                    value[i:i + BLOCK, h] = code.double() * s
            out[side].append(value)
        for h, keep in enumerate(sides):
            for i in range(0, count, BLOCK):
                at = keep[i:i + BLOCK]
                weights[table[b][i // BLOCK], h] = 0
                weights[table[b][i // BLOCK], h, :at.numel()] = w[h, at]
    count = torch.tensor([min(x, c["budget"]) for x in lens], dtype=torch.int32, device="cuda")
    return torch.cat(out[0]), torch.cat(out[1]), weights, kept_all, count


def work(case):
    c = case
    if c["op"] == "prefill":
        T, n, size = sum(_lengths(c)), c["n"], SIZE[c["dtype"]]
        states = n * c["H"] * c["d"] ** 2 * 4 * (2 if c["init"] else 1)
        g = c["H"] * 4 if c["const"] else T * c["H"] * 4
        return {"bytes": T * 2 * (c["Hk"] + c["H"]) * c["d"] * size + g + states + 4 * (n + 1),
                "flops": T * c["H"] * 4 * c["d"] ** 2}
    if c["op"] == "window":
        n, W, H, d, size = c["n"], c["W"], c["H"], c["d"], SIZE[c["dtype"]]
        g = H * 4 if c["const"] else n * W * H * 4
        return {"bytes": n * (W + 1) * (H * d * d * 4 + 4) + n * W * 2 * (c["Hk"] + H) * d * size + g,
                "flops": n * W * H * 5 * d * d}
    lens = _lengths(c)
    if c["op"] == "weigh":
        W, keys = c["W"], sum(lens) + c["n"] * c["W"]
        pages = sum(-(-(x + W) // BLOCK) for x in lens)
        return {"bytes": keys * c["Hkv"] * (c["d"] + 8) + pages * 4 * (c["Hkv"] + 1)
                + c["n"] * (W * c["Hq"] * c["d"] * SIZE[c["dtype"]] + 4),
                "flops": keys * W * c["Hq"] * 2 * c["d"]}
    kept, pages = sum(min(x, c["budget"]) for x in lens), sum(-(-x // BLOCK) for x in lens)
    # the weights once, the kept tokens' codes moved and read back, their weights and places
    return {"bytes": c["Hkv"] * (sum(lens) * 4 + kept * (2 * 3 * c["d"] + 2 * 2 * c["d"] + 8)
                                 + pages * 8) + pages * 4,
            "flops": c["Hkv"] * sum(lens)}
