"""The serving operators on a stream of their own, and batches larger than the attention's search
handles in one step."""
import numpy as np
import pytest
import torch

import serving_ref as ref
from kda_testutil import f64
from linear_attention_state_kda_gb300 import kda
from test_gpu_cache_attention import DEV, _check, _i32, _make

pytestmark = pytest.mark.gpu


def test_memory_made_for_another_stream_is_not_reused_early():
    """The workspace and outputs that a call allocates stay untouched until its stream has run,
    though the caller drops them at once and the current stream allocates the same sizes."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1)
    start = [4000, 17, 900]
    q, table, pool = _make(gen, start, 2, 8, 2, 128, "bf16")
    st = _i32(start)
    want = kda.cache_attention(q, st, table, *pool, scale=0.05)
    norm, _ = kda.head_norm_rope(q, None)
    need = kda.cache_attention_workspace(3, 2, 8, 2, 128)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got_o, got_n = torch.empty_like(q), torch.empty_like(q)
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)  # about a tenth of a second: the calls queue behind it
    o = kda.cache_attention(q, st, table, *pool, scale=0.05, stream=side)
    n, _ = kda.head_norm_rope(q, None, stream=side)
    with torch.cuda.stream(side):
        got_o.copy_(o)
        got_n.copy_(n)
    del o, n
    junk = [torch.full((need,), 0xff, dtype=torch.uint8, device=DEV) for _ in range(3)]
    junk += [torch.full_like(q, float("nan")) for _ in range(6)]
    torch.cuda.synchronize()
    assert torch.equal(got_o, want) and torch.equal(got_n, norm)
    assert len(junk) == 9


@pytest.mark.parametrize("batch,Hq,d,dtype", [(33, 4, 64, "bf16"), (257, 2, 128, "f32"),
                                              (20000, 2, 64, "bf16")])
def test_large_batches_mostly_padding(batch, Hq, d, dtype):
    """Rows without keys between a few rows with some: every row's result, and zeros elsewhere."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(batch)
    rng = np.random.default_rng(batch)
    live = rng.choice(batch, size=min(batch, 90), replace=False)
    start = np.full(batch, -1)
    start[live] = rng.integers(0, 150, live.size)
    start[live[0]] = 1500
    cols = 24
    table = torch.full((batch, cols), -1, dtype=torch.int32, device=DEV)
    n_pages = live.size * cols
    perm = torch.randperm(n_pages, generator=gen, device=DEV).to(torch.int32)
    table[torch.from_numpy(live).to(DEV)] = perm.reshape(live.size, cols)
    q, _, pool = _make(gen, [1500], 1, Hq, 1, d, dtype, spare=n_pages)
    q = torch.randn(batch, Hq, d, generator=gen, device=DEV).to(q.dtype)
    got = kda.cache_attention(q, _i32(start.tolist()), table, *pool, scale=0.05)
    idx = torch.from_numpy(live).to(DEV)
    _check(q[idx].contiguous(), start[live].tolist(), None, table[idx], pool, 0.05, dtype, got[idx])
    rest = torch.ones(batch, dtype=torch.bool, device=DEV)
    rest[idx] = False
    assert (got[rest] == 0).all()


def test_cache_of_many_short_sequences():
    """One or two tokens each for a thousand sequences, some of them empty or skipped, through
    cu_seqlens; read back whole."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(2)
    rng = np.random.default_rng(3)
    n, H, d = 1000, 2, 64
    lens = rng.integers(0, 3, n)
    start = rng.integers(-1, 64, n)
    cu = np.concatenate([[0], np.cumsum(lens)])
    T = int(cu[-1])
    table = torch.randperm(2 * n, generator=gen, device=DEV).to(torch.int32).reshape(n, 2)
    shape = (2 * n, H, 64, d)
    kc = torch.randint(0, 0x60, shape, generator=gen, device=DEV).to(torch.uint8)
    ks = torch.exp2(torch.randint(-9, -4, shape[:2], generator=gen, device=DEV).double()).float()
    vc, vs = kc.clone(), ks.clone()
    k = torch.randn(T, H, d, generator=gen, device=DEV, dtype=torch.bfloat16)
    v = 5 * torch.randn(T, H, d, generator=gen, device=DEV, dtype=torch.bfloat16)
    host = table.cpu().numpy()
    want = []
    for x, c, s in ((k, kc, ks), (v, vc, vs)):
        val, sc = ref.values(c), f64(s)
        ref.cache_write(f64(x), val, sc, cu, start, None, host, 2 * n)
        want.append((val, sc))
    kda.cache_write(k, v, _i32(start.tolist()), table, kc, ks, vc, vs, cu_seqlens=_i32(cu.tolist()))
    back = np.where(start >= 0, start + lens, 0)
    rcu = np.concatenate([[0], np.cumsum(back)])
    k2, v2 = kda.cache_read(_i32([0] * n), table, kc, ks, vc, vs, int(rcu[-1]),
                            cu_seqlens=_i32(rcu.tolist()))
    for (val, sc), x in zip(want, (f64(k2), f64(v2))):
        for s in range(n):
            a, _ = ref.gather(val, sc, host[s], int(back[s]), 2 * n)
            assert np.array_equal(x[rcu[s]:rcu[s + 1]], a), s


def test_workspace_elsewhere_is_refused():
    """A workspace in host memory is refused by the binding: nothing is launched with its pointer."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(4)
    start = [300, 17]
    q, table, pool = _make(gen, start, 2, 8, 2, 128, "bf16")
    st = _i32(start)
    ws = torch.zeros(kda.cache_attention_workspace(2, 2, 8, 2, 128) + 256, dtype=torch.uint8)
    before = kda.launch_count()
    with pytest.raises(ValueError, match="device"):
        kda.cache_attention(q, st, table, *pool, scale=0.05, workspace=ws)
    assert kda.launch_count() == before
    kda.cache_attention(q, st, table, *pool, scale=0.05, workspace=ws.to(DEV))
    assert kda.launch_count() > before


def _held_back(shape_bytes, call):
    """Runs `call` on a stream of its own while the current stream still has to read a block of
    `shape_bytes` bytes that was dropped just before; returns whether the reader got its data."""
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    blocks = [torch.full((n,), 37, dtype=torch.uint8, device=DEV) for n in shape_bytes]
    copies = [torch.empty_like(b) for b in blocks]
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # about a tenth of a second
    for c, b in zip(copies, blocks):
        c.copy_(b)
    del blocks, b
    out = call(side)
    side.synchronize()
    done = torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    assert not done  # the reader was still waiting when the call had run
    return out, all(bool((c == 37).all()) for c in copies)


def test_memory_made_for_another_stream_is_not_taken_from_pending_work():
    """Outputs and workspace of a call on another stream do not lie in memory that the current stream
    has yet to read, though it is free for the current stream's next tensors."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(6)
    start = [4000, 17, 900]
    q, table, pool = _make(gen, start, 2, 8, 2, 128, "bf16")
    st, zero, cu = _i32(start), _i32([0, 0, 0]), _i32([0, 100, 150, 500])
    p = torch.softmax(torch.randn(300, 4, 50, generator=gen, device=DEV), -1)
    toks = p[:, :3].argmax(-1).to(torch.int32).contiguous()
    ua, us = torch.rand(300, 3, generator=gen, device=DEV), torch.zeros(300, device=DEV)
    n = q.numel() * 2
    need = kda.cache_attention_workspace(3, 2, 8, 2, 128)
    for sizes, call in (
            ([n], lambda s: kda.head_norm_rope(q, None, stream=s)[0]),
            ([n, need], lambda s: kda.cache_attention(q, st, table, *pool, scale=0.05, stream=s)),
            ([500 * 2 * 128 * 2] * 2,
             lambda s: kda.cache_read(zero, table, *pool, 500, cu_seqlens=cu, stream=s)),
            ([300 * 4 * 4, 300 * 4], lambda s: kda.draft_verify(p, toks, ua, us, stream=s)[1])):
        want = call(None)
        got, kept = _held_back(sizes, call)
        assert kept
        for x, y in zip(*((z,) if torch.is_tensor(z) else z for z in (got, want))):
            assert torch.equal(x, y)
