"""Cases of the serving operators next to the recurrence: per-head norm with rotation, the paged
8-bit cache (write and read back), attention over it, and the verification of drafted tokens.

``run`` computes an operator in its plain form (elementary torch operations in 32 bits), or, with
``own`` set, through the library's binding.
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
        # one decode step of two requests: q and k heads of one attention layer, latency only
        dict(name="norm_rope_2", op="norm_rope", tokens=2, Hq=32, Hk=8, d=128, rot=128, l2=False,
             interleaved=False, dtype="bf16"),
        # a 16k-token prompt, q and k taken from the fused projection's rows
        dict(name="norm_rope_16k", op="norm_rope", tokens=16384, Hq=32, Hk=8, d=128, rot=128,
             l2=False, interleaved=False, dtype="bf16"),
        # one verify window of a few requests: 4 tokens each, most into pages that hold earlier tokens
        dict(name="cache_window_16x4", op="cache", n=16, new=4, past=1500, H=8, d=128, dtype="bf16"),
        # a 16k-token prompt written into an empty cache and read back
        dict(name="cache_prompt_16k", op="cache", n=1, new=16384, past=0, H=32, d=128, dtype="bf16"),
        # ragged fp32 chunks at head size 64, pages continued in the middle
        dict(name="cache_chunks_f32", op="cache", n=7, new=777, past=301, H=6, d=64, dtype="f32"),
        # two requests with short contexts, one token each
        dict(name="attn_2x100", op="attn", n=2, W=1, ctx=100, Hq=32, Hkv=8, d=128, dtype="bf16"),
        # one long context, one token: the cache's length is the only axis to split over
        dict(name="attn_1x128k", op="attn", n=1, W=1, ctx=131072, Hq=32, Hkv=8, d=128, dtype="bf16"),
        # a serving batch, one token each, contexts of any length up to 16k
        dict(name="attn_128x16k", op="attn", n=128, W=1, ctx=16384, Hq=32, Hkv=8, d=128,
             dtype="bf16"),
        # verify windows of four tokens, eight query heads to a cached head
        dict(name="attn_window_64x4", op="attn", n=64, W=4, ctx=8192, Hq=64, Hkv=8, d=128,
             dtype="bf16"),
        # fp32 queries at head size 64, odd group and window
        dict(name="attn_f32_5x3", op="attn", n=5, W=3, ctx=3001, Hq=15, Hkv=3, d=64, dtype="f32"),
        # three drafted tokens of four requests over a small vocabulary of odd size
        dict(name="verify_4x3", op="verify", n=4, W=3, V=32003, onehot=False, dtype="f32"),
        # a serving batch: seven drafted tokens each over a large vocabulary
        dict(name="verify_256x7", op="verify", n=256, W=7, V=131072, onehot=False, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "cache", "attn", "attn", "verify"])
    d = rng.choice([64, 128, 128])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "norm_rope":
        Hk = rng.choice([1, 2, 3, 4, 8, 16])
        Hq = Hk * rng.choice([1, 2, 3, 4])
        top = 16384 * 40 * 256 // ((Hq + Hk) * d * SIZE[dtype])
        return dict(op=op, tokens=_log(rng, 1, min(16384, top)), Hq=Hq, Hk=Hk, d=d,
                    rot=rng.choice([0, 32, d // 2, d, d]), l2=rng.random() < 0.3,
                    interleaved=rng.random() < 0.4, dtype=dtype)
    if op == "cache":
        n = _log(rng, 1, 256)
        return dict(op=op, n=n, new=_log(rng, 1, max(1, 32768 // n)), past=_log(rng, 1, 4096) - 1,
                    H=rng.choice([1, 2, 3, 4, 8]), d=d, dtype=dtype)
    if op == "attn":
        n = _log(rng, 1, 128)
        Hkv = rng.choice([1, 2, 3, 4, 8])
        G = rng.choice([1, 2, 3, 4, 5, 8]) if Hkv > 1 else rng.choice([1, 4, 8, 16])
        W = rng.choice([1, 1, 1, 2, 3, 4, 7])
        return dict(op=op, n=n, W=W, ctx=_log(rng, 1, min(131072, 1048576 // (n * W))),
                    Hq=Hkv * G, Hkv=Hkv, d=d, dtype=dtype)
    return dict(op=op, n=_log(rng, 1, 200), W=rng.randint(1, 7), V=_log(rng, 1000, 131072),
                onehot=rng.random() < 0.25, dtype="f32" if rng.random() < 0.7 else "bf16")


# ---------------------------------------------------------------- inputs

def _gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed))
    return g


def _pages(gen, need):
    """A page table of `need` [n, max_pages] used entries: distinct pages in a shuffled order, -1
    where a row has none. Returns it and the number of pages of the pool (a few more than used)."""
    used = int(need.sum())
    n_pages = used + 3
    perm = torch.randperm(n_pages, generator=gen, device="cuda")[:used].to(torch.int32)
    table = torch.full(need.shape, -1, dtype=torch.int32, device="cuda")
    table[need] = perm
    return table, n_pages


def _pow2_scale(amax):
    """Smallest power of two s with amax <= 448 s, at least 2^-100."""
    m, e = torch.frexp(amax)
    e = (e - 9 + (m > 0.875).to(e.dtype)).clamp(min=-100)
    e = torch.where(amax > 0, e, torch.full_like(e, -100))
    return ((e + 127) << 23).view(torch.float32)  # 2^e by its bits: exact


def _random_cache(gen, n_pages, H, d, spread):
    """Codes and scales of pages of ~N(0, spread) values, a few channels eight times larger."""
    codes = torch.empty(n_pages, H, BLOCK, d, dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty(n_pages, H, device="cuda")
    chan = 1.0 + 7.0 * (torch.rand(H, 1, d, generator=gen, device="cuda") < 0.02)
    step = max(1, (1 << 28) // (H * BLOCK * d))
    for i in range(0, n_pages, step):
        n = min(step, n_pages - i)
        x = torch.randn(n, H, BLOCK, d, generator=gen, device="cuda") * (spread * chan)
        s = _pow2_scale(x.abs().amax((2, 3)))
        codes[i:i + n] = (x / s[:, :, None, None]).to(torch.float8_e4m3fn)
        scale[i:i + n] = s
    return codes, scale


def _lengths(c):
    """Tokens already cached and new tokens of each row: by the case alone, so that every seed's
    outputs have the same shape. Contexts and long chunks are ragged, the first of full length."""
    rng = random.Random("%d %d" % (c["n"], c["ctx"] if c["op"] == "attn" else c["new"]))
    ragged = lambda top: [top] + [rng.randint(1, top) for _ in range(c["n"] - 1)]  # noqa: E731
    if c["op"] == "attn":
        return ragged(c["ctx"]), [c["W"]] * c["n"]
    new = ragged(c["new"]) if c["new"] > 16 else [c["new"]] * c["n"]
    return [rng.randint(0, c["past"]) for _ in new], new


def prepare(case, seed):
    gen = _gen(seed)
    c = dict(case)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    uni = lambda *s: torch.rand(*s, generator=gen, device="cuda")  # noqa: E731
    st = {"case": c}
    if c["op"] == "norm_rope":
        T, Hq, Hk, d, rot = c["tokens"], c["Hq"], c["Hk"], c["d"], c["rot"]
        qkv = (rnd(T, Hq + 2 * Hk, d) * (0.2 + 2.0 * uni(T, 1, 1))).to(DT[c["dtype"]])
        st["q"], st["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]  # rows of the fused projection
        st["qw"], st["kw"] = (None, None) if c["l2"] else (1.0 + 0.3 * rnd(d), 1.0 + 0.3 * rnd(d))
        st["table"], st["pos"] = None, None
        if rot:
            n_pos = 2 * T + 64
            inv = torch.pow(10000.0, -torch.arange(0, rot, 2, device="cuda").double() / rot)
            ang = torch.arange(n_pos, device="cuda").double()[:, None] * inv
            st["table"] = torch.cat([ang.cos(), ang.sin()], 1).float()
            st["pos"] = torch.randint(0, n_pos, (T,), generator=gen, device="cuda",
                                      dtype=torch.int32)
    elif c["op"] == "cache":
        n, H, d = c["n"], c["H"], c["d"]
        past, new = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in _lengths(c))
        top = -(-(c["new"] + c["past"]) // BLOCK)
        need = torch.arange(top, device="cuda")[None] * BLOCK < (past + new)[:, None]
        st["pages"], n_pages = _pages(gen, need)
        T = int(new.sum())
        st["kc"], st["ks"] = _random_cache(gen, n_pages, H, d, 0.5)
        st["vc"], st["vs"] = _random_cache(gen, n_pages, H, d, 0.2)
        grow = torch.exp(rnd(T, 1, 1))  # some tokens are larger than what their page holds
        st["k"], st["v"] = (rnd(T, H, d) * 0.5 * grow).to(DT[c["dtype"]]), \
            (rnd(T, H, d) * 0.2 * grow).to(DT[c["dtype"]])
        zero = torch.zeros(1, dtype=torch.int32, device="cuda")
        st["cu"] = torch.cat([zero, new.cumsum(0).to(torch.int32)])
        st["start"] = past
        st["read_start"] = past // BLOCK * BLOCK  # from the start of the first page written
        back = new + past - st["read_start"]
        st["read_cu"] = torch.cat([zero, back.cumsum(0).to(torch.int32)])
        st["read_tokens"] = int(back.sum())
    elif c["op"] == "attn":
        n, W, Hq, Hkv, d = c["n"], c["W"], c["Hq"], c["Hkv"], c["d"]
        ctx = torch.tensor(_lengths(c)[0], dtype=torch.int32, device="cuda")
        top = -(-(c["ctx"] + W) // BLOCK)
        need = torch.arange(top, device="cuda")[None] * BLOCK < (ctx + W)[:, None]
        st["pages"], n_pages = _pages(gen, need)
        st["kc"], st["ks"] = _random_cache(gen, n_pages, Hkv, d, 0.9)
        st["vc"], st["vs"] = _random_cache(gen, n_pages, Hkv, d, 0.4)
        st["start"] = ctx
        st["q"] = (rnd(n * W, Hq, d) * (0.5 + 1.5 * uni(1, Hq, 1))).to(DT[c["dtype"]])
    else:
        n, W, V = c["n"], c["W"], c["V"]
        dt = DT[c["dtype"]]
        logits = rnd(n, W + 1, V) * 3.0
        st["target"] = torch.softmax(logits, -1).to(dt)
        logits = logits[:, :W] + 0.7 * rnd(n, W, V)
        if c["onehot"]:  # drafted without probabilities: the most likely token of the draft
            st["draft"], st["tokens"] = None, logits.argmax(-1).to(torch.int32)
        else:
            noise = -torch.log(-torch.log(uni(n, W, V).clamp(1e-30, 1 - 1e-7)))
            st["tokens"] = (logits + noise).argmax(-1).to(torch.int32)
            st["draft"] = torch.softmax(logits, -1).to(dt)
        st["ua"], st["us"] = uni(n, W), uni(n)
        st["slots"] = torch.randperm(4096, generator=gen, device="cuda")[:n * (W + 1)] \
            .to(torch.int32).reshape(n, W + 1)
    return st


# ---------------------------------------------------------------- plain forms

def _norm_rope(x, w, st, c):
    x32 = x.float()
    s = x32.square().sum(-1, keepdim=True)
    y = x32 * torch.rsqrt((s if c["l2"] else s / c["d"]) + 1e-6)
    if w is not None:
        y = y * w
    h = c["rot"] // 2
    if h:
        cos, sin = st["table"][st["pos"].long()][:, None].split(h, -1)
        if c["interleaved"]:
            a, b = y[..., 0:2 * h:2], y[..., 1:2 * h:2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = y[..., :h], y[..., h:2 * h]
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        y = torch.cat([r, y[..., 2 * h:]], -1)
    return y.to(x.dtype)


def _e4m3(x):
    return x.clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)


def _rows(cu, start, table, total):
    """Per packed token: its sequence, its page and its place in the page."""
    t = torch.arange(total, device="cuda")
    seq = torch.searchsorted(cu[1:].long(), t, right=True)
    pos = start.long()[seq] + t - cu.long()[seq]
    return seq, table[seq, pos // BLOCK].long(), pos % BLOCK


def _cache_write(x, codes, scale, st):
    n_pages, H, _, d = codes.shape
    x = x.float()
    _, page, at = _rows(st["cu"], st["start"], st["pages"], x.shape[0])
    amax = torch.zeros(n_pages, H, device="cuda")
    amax = amax.scatter_reduce(0, page[:, None].expand(-1, H), x.abs().amax(-1), "amax")
    new = _pow2_scale(amax)
    # the first page of each sequence keeps the tokens that it held before
    first = st["start"].long() // BLOCK
    p0 = st["pages"][torch.arange(first.numel(), device="cuda"), first].long()
    keep = torch.arange(BLOCK, device="cuda")[None, :, None] < (st["start"] % BLOCK)[:, None, None]
    partial = (st["start"] % BLOCK > 0)[:, None]
    s0 = torch.where(partial, torch.maximum(scale[p0], new[p0]), new[p0])
    raw = codes.view(torch.uint8)
    held = _e4m3(raw[p0].view(torch.float8_e4m3fn).float() * (scale[p0] / s0)[:, :, None, None])
    raw[p0] = torch.where(keep[:, None], held.view(torch.uint8), raw[p0])
    touched = torch.zeros(n_pages, dtype=torch.bool, device="cuda")
    touched[page] = True
    new[p0] = s0
    scale.copy_(torch.where(touched[:, None], new, scale))
    raw[page, :, at] = _e4m3(x / scale[page][:, :, None]).view(torch.uint8)


def _cache_read(codes, scale, st, dtype):
    _, page, at = _rows(st["read_cu"], st["read_start"], st["pages"], st["read_tokens"])
    x = codes.view(torch.uint8)[page, :, at].view(torch.float8_e4m3fn).float()
    return (x * scale[page][:, :, None]).to(dtype)


def _attend(st, c):
    n, W, Hq, Hkv, d = c["n"], c["W"], c["Hq"], c["Hkv"], c["d"]
    page = st["pages"].clamp(min=0).long()
    L = page.shape[1] * BLOCK

    def whole(codes, scale):
        x = codes.view(torch.uint8)[page].view(torch.float8_e4m3fn).float()
        x *= scale[page][..., None, None]
        return x.transpose(1, 2).reshape(n, Hkv, L, d)

    q = st["q"].float().reshape(n, W, Hkv, Hq // Hkv, d).permute(0, 2, 1, 3, 4)
    s = q.reshape(n, Hkv, -1, d) @ whole(st["kc"], st["ks"]).transpose(2, 3) * d ** -0.5
    t = torch.arange(L, device="cuda")
    seen = t <= st["start"][:, None, None] + torch.arange(W, device="cuda")[:, None]
    seen = seen[:, None, :, None].expand(n, 1, W, Hq // Hkv, L).reshape(n, 1, -1, L)
    s = s.masked_fill(~seen, float("-inf"))
    p = torch.exp(s - s.amax(-1, keepdim=True))
    o = p @ whole(st["vc"], st["vs"]) / p.sum(-1, keepdim=True)
    o = o.reshape(n, Hkv, W, Hq // Hkv, d).permute(0, 2, 1, 3, 4)
    return o.reshape(n * W, Hq, d).to(st["q"].dtype)


def _verify(st, c):
    n, W, V = c["n"], c["W"], c["V"]
    x = st["tokens"].long()
    p = st["target"][:, :W].gather(2, x[..., None])[..., 0].float()
    q = torch.ones_like(p) if c["onehot"] else st["draft"].gather(2, x[..., None])[..., 0].float()
    taken = (st["ua"] * q < p).long().cumprod(1)
    acc = taken.sum(1)
    row = torch.arange(n, device="cuda")
    pr = st["target"][row, acc].float()
    at = acc.clamp(max=W - 1)
    if c["onehot"]:
        qr = torch.zeros_like(pr).scatter_(1, x[row, at][:, None], 2.0)
    else:
        qr = st["draft"][row, at].float()
    qr = torch.where((acc < W)[:, None], qr, torch.zeros_like(qr))
    whole = lambda y: (y.clamp(0, 1) * 2.0 ** 40).floor().to(torch.int64)  # noqa: E731
    w = whole(pr - qr)
    w = torch.where((w.sum(1) > 0)[:, None], w, whole(pr))
    cum = w.cumsum(1)
    total = cum[:, -1]
    u = (st["us"] * 2.0 ** 24).floor().to(torch.int64)
    limit = (total >> 24) * u + ((total & 0xFFFFFF) * u >> 24)
    last = (cum <= limit[:, None]).sum(1)
    col = torch.arange(W + 1, device="cuda")
    out = torch.cat([x, torch.zeros_like(x[:, :1])], 1)
    out = torch.where(col == acc[:, None], last[:, None], out)
    out = torch.where(col > acc[:, None], torch.full_like(out, -1), out)
    return acc.to(torch.int32), out.to(torch.int32), st["slots"][row, acc]


def run(state):
    c, st = state["case"], state
    if own:
        from linear_attention_state_kda_gb300 import kda
    if c["op"] == "norm_rope":
        if own:
            return kda.head_norm_rope(st["q"], st["k"], st["qw"], st["kw"], eps=1e-6, l2=c["l2"],
                                      cos_sin=st["table"], positions=st["pos"],
                                      interleaved=c["interleaved"])
        return _norm_rope(st["q"], st["qw"], st, c), _norm_rope(st["k"], st["kw"], st, c)
    if c["op"] == "cache":
        if own:
            kda.cache_write(st["k"], st["v"], st["start"], st["pages"], st["kc"], st["ks"],
                            st["vc"], st["vs"], cu_seqlens=st["cu"])
            k, v = kda.cache_read(st["read_start"], st["pages"], st["kc"], st["ks"], st["vc"],
                                  st["vs"], st["read_tokens"], cu_seqlens=st["read_cu"],
                                  dtype=st["k"].dtype)
        else:
            _cache_write(st["k"], st["kc"], st["ks"], st)
            _cache_write(st["v"], st["vc"], st["vs"], st)
            k = _cache_read(st["kc"], st["ks"], st, st["k"].dtype)
            v = _cache_read(st["vc"], st["vs"], st, st["v"].dtype)
        return {"k": k, "v": v, "k_scale": st["ks"], "v_scale": st["vs"]}
    if c["op"] == "attn":
        if own:
            return kda.cache_attention(st["q"], st["start"], st["pages"], st["kc"], st["ks"],
                                       st["vc"], st["vs"], scale=c["d"] ** -0.5)
        return _attend(st, c)
    if own:
        return kda.draft_verify(st["target"], st["tokens"], st["ua"], st["us"],
                                draft_probs=st["draft"], write_slots=st["slots"])
    return _verify(st, c)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    z = SIZE[c["dtype"]]
    if c["op"] == "norm_rope":
        el = c["tokens"] * (c["Hq"] + c["Hk"]) * c["d"]
        return {"bytes": 2 * el * z + c["tokens"] * (c["rot"] * 4 + 4), "flops": 10 * el}
    if c["op"] == "cache":
        past, new = _lengths(c)
        keep, new = sum(x % BLOCK for x in past), sum(new)
        el = 2 * c["H"] * c["d"]
        return {"bytes": el * (new * (z + 1) + (new + keep) * (1 + z)), "flops": 4 * el * new}
    if c["op"] == "attn":
        ctx = sum(_lengths(c)[0]) + c["n"] * c["W"]
        qo = 2 * c["n"] * c["W"] * c["Hq"] * c["d"] * z
        return {"bytes": 2 * ctx * c["Hkv"] * c["d"] + qo,
                "flops": 4 * ctx * c["W"] * c["Hq"] * c["d"]}
    rows = 1 if c["onehot"] else 2
    return {"bytes": c["n"] * rows * c["V"] * z, "flops": 3 * c["n"] * c["V"]}


# ---------------------------------------------------------------- definitions in 64 bits

def _exact_e4m3(x):
    """x (float64) rounded to the nearest value of the 8-bit format (ties to even), saturated."""
    _, e = torch.frexp(x)
    step = (((e - 1).clamp(min=-6) - 3 + 1023).to(torch.int64) << 52).view(torch.float64)
    return (torch.round(x / step) * step).clamp(-FP8_MAX, FP8_MAX)


def _exact_scale(m):
    s = 2.0 ** -100
    if m > 0:
        s = max(s, 2.0 ** math.ceil(math.log2(m / FP8_MAX)))
        s = s * 2 if m > FP8_MAX * s else s
        s = s / 2 if s > 2.0 ** -100 and m <= FP8_MAX * s / 2 else s
    return s


def _exact_cache(st, c):
    out = {}
    cu, start, rcu = st["cu"].tolist(), st["start"].tolist(), st["read_cu"].tolist()
    table = st["pages"].tolist()
    for name, dt in (("k", c["dtype"]), ("v", c["dtype"])):
        x = st[name].double()
        val = st[name + "c"].double()
        scale = st[name + "s"].double()
        back = torch.empty(rcu[-1], c["H"], c["d"], dtype=torch.float64, device="cuda")
        for s in range(c["n"]):
            done = 0
            while done < cu[s + 1] - cu[s]:
                pos = start[s] + done
                page, off = table[s][pos // BLOCK], pos % BLOCK
                n = min(BLOCK - off, cu[s + 1] - cu[s] - done)
                new = x[cu[s] + done:cu[s] + done + n].transpose(0, 1)
                sc = torch.tensor([_exact_scale(m) for m in new.abs().amax((1, 2)).tolist()],
                                  dtype=torch.float64, device="cuda")
                if off:
                    sc = torch.maximum(sc, scale[page])
                    ratio = (scale[page] / sc)[:, None, None]
                    val[page, :, :off] = _exact_e4m3(val[page, :, :off] * ratio)
                scale[page] = sc
                val[page, :, off:off + n] = _exact_e4m3(new / sc[:, None, None])
                to = rcu[s] + done + start[s] % BLOCK - off
                back[to:to + off + n] = \
                    (val[page, :, :off + n] * sc[:, None, None]).transpose(0, 1)
                done += n
        out[name], out[name + "_scale"] = back, scale
    return out


def exact(case, seed):
    st = prepare(case, seed)
    c = st["case"]
    if c["op"] == "norm_rope":
        got = []
        for x, w in ((st["q"], st["qw"]), (st["k"], st["kw"])):
            x = x.double()
            ss = torch.einsum("thd,thd->th", x, x)
            y = x / torch.sqrt((ss if c["l2"] else ss / c["d"]) + 1e-6)[..., None]
            y = y if w is None else y * w.double()
            if c["rot"]:
                h = c["rot"] // 2
                tab = st["table"].double()[st["pos"].long()]
                turn = torch.complex(tab[:, :h], tab[:, h:])[:, None]
                r = y[..., :c["rot"]]
                if c["interleaved"]:
                    z = torch.view_as_complex(r.unflatten(-1, (h, 2)).contiguous()) * turn
                    r = torch.view_as_real(z).flatten(-2)
                else:
                    z = torch.complex(r[..., :h].contiguous(), r[..., h:].contiguous()) * turn
                    r = torch.cat([z.real, z.imag], -1)
                y = torch.cat([r, y[..., c["rot"]:]], -1)
            got.append(y)
        return tuple(got)
    if c["op"] == "cache":
        return _exact_cache(st, c)
    if c["op"] == "attn":
        n, W, G, d = c["n"], c["W"], c["Hq"] // c["Hkv"], c["d"]
        o = torch.empty(n, W, c["Hkv"], G, d, dtype=torch.float64, device="cuda")
        q = st["q"].double().reshape(n, W, c["Hkv"], G, d)
        for b, ctx in enumerate(st["start"].tolist()):
            L = ctx + W
            pg = st["pages"][b, :-(-L // BLOCK)].long()

            def side(codes, scale):
                raw = codes.view(torch.uint8)[pg].view(torch.float8_e4m3fn).double()
                x = raw * scale[pg].double()[..., None, None]
                return x.permute(1, 0, 2, 3).reshape(c["Hkv"], -1, d)[:, :L]

            s = torch.einsum("whgd,htd->hwgt", q[b], side(st["kc"], st["ks"])) / math.sqrt(d)
            for j in range(W):
                s[:, j, :, ctx + j + 1:] = -math.inf
            o[b] = torch.einsum("hwgt,htd->whgd", torch.softmax(s, -1), side(st["vc"], st["vs"]))
        return o.reshape(n * W, c["Hq"], d)
    return None  # whole numbers: the plain form's are the definition's
