"""kda_cache_attention where one SM goes from a unit's short last row group (1 .. 128 rows, some
tiles of keys) on to a unit of 256 rows: only one of the kernel's two row tiles has rows in the
first, and the other one must not look at the second's pages early.

Key and value scales differ strongly from page to page and from head to head, and values are
positive, so that a tile whose weights are of another page's scales shows in the result: its share
of the keys (128 of at most 4200, 3%) is off by a factor, against a tolerance of 2^-10 of the
largest value and 2^-8 of the result. Tolerances as derived in test_gpu_cache_attention."""
import pytest
import torch

import serving_ref as ref
from linear_attention_state_kda_gb300 import kda
from test_gpu_cache_attention import DEV, _i32, _make

pytestmark = pytest.mark.gpu


def _want(q, start, table, pool, scale, batch):
    """The definition in 64 bits with torch operations, row by row and head by head."""
    code = torch.from_numpy(ref.code_values()).to(DEV)
    W, Hq, d = q.shape[0] // batch, q.shape[1], q.shape[2]
    Hkv = pool[0].shape[1]
    G = Hq // Hkv
    out = torch.zeros(batch, W, Hq, d, dtype=torch.float64, device=DEV)
    x = q.double().reshape(batch, W, Hq, d)
    for b in range(batch):
        n = start[b] + W
        page = table[b, :(n + 63) // 64].long()
        at = page.clamp(min=0)
        there = (page >= 0).repeat_interleave(64)[:n]
        t = torch.arange(n, device=DEV)
        seen = there & (t <= start[b] + torch.arange(W, device=DEV)[:, None])
        for h in range(Hkv):
            k, v = ((code[pool[i][at, h].long()] * pool[i + 1][at, h].double()[:, None, None])
                    .reshape(-1, d)[:n] for i in (0, 2))
            for u in range(h * G, h * G + G):
                s = (scale * (x[b, :, u] @ k.T)).masked_fill(~seen, float("-inf"))
                out[b, :, u] = torch.softmax(s, -1) @ v
    return out.reshape(q.shape)


@pytest.mark.parametrize("start,W,Hq,Hkv,d,absent", [
    ([4096] * 4, 80, 32, 8, 128, False), ([2048] * 16, 66, 32, 8, 128, False),
    ([0] * 4, 1100, 32, 8, 128, False), ([4096] * 4, 70, 32, 8, 64, False),
    ([1500] * 20, 140, 16, 8, 128, True), ([2048] * 12, 70, 32, 8, 64, True)])
def test_from_a_short_row_group_into_the_next_unit(start, W, Hq, Hkv, d, absent):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(len(start) + W + d)
    q, table, pool = _make(gen, start, W, Hq, Hkv, d, "bf16")
    for i in (1, 3):
        shape = pool[i].shape
        pool[i] = torch.exp2(-3.0 - 6.0 * torch.randint(0, 2, shape, generator=gen, device=DEV))
    pool[2] &= 0x7f
    if absent:
        table[1::2, 0] = -1  # the first tile of every other row lacks a page
        table[2::4, 1] = -1
    scale = 0.3 * d ** -0.5
    got = kda.cache_attention(q, _i32(start), table, *pool, scale=scale)
    want = _want(q, start, table, pool, scale, len(start))
    top = 30 * float(pool[3].max())
    err = (got.double() - want).abs() / (2.0 ** -10 * top + 2.0 ** -8 * want.abs())
    assert float(err.max()) <= 1, float(err.max())
    for _ in range(3):
        assert torch.equal(kda.cache_attention(q, _i32(start), table, *pool, scale=scale), got)


def test_pieces_that_take_long():
    """Contexts of 3.8 million tokens (two pages in turn), two heads on each SM: a row tile waits 30
    thousand tiles for the other one's piece. No wait gives up, and the result is right.

    Each of a row's sums is 30 thousand tiles of at most 8 additions in fp32, each of which may lose
    2^-23 of the sum so far: 0.03 of the largest result, besides the usual 2^-10 of the largest value
    and 2^-8 of the result."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(9)
    B, W, Hq, Hkv, d, tiles = 76, 75, 16, 4, 64, 30000
    start = [tiles * 128 - W] * B
    q, _, pool = _make(gen, [100], 1, Hq, Hkv, d, "bf16", spare=0)
    pool[2] &= 0x7f
    q = torch.randn(B * W, Hq, d, generator=gen, device=DEV).bfloat16()
    table = _i32([0, 1]).repeat(tiles).expand(B, -1).contiguous()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    scale = 0.3 * d ** -0.5
    got = kda.cache_attention(q, _i32(start), table, *pool, scale=scale, status=status)
    assert int(status) == 0
    code = torch.from_numpy(ref.code_values()).to(DEV)
    t = torch.arange(128, device=DEV)
    seen = start[0] + 1 + torch.arange(W, device=DEV)  # keys of the window's tokens
    times = ((seen[:, None] - 1 - t) // 128 + 1).double()  # of each of the two pages' rows
    x = q.double().reshape(B, W, Hkv, Hq // Hkv, d)
    k, v = ((code[pool[i].long()] * pool[i + 1].double()[:, :, None, None])
            .transpose(0, 1).reshape(Hkv, 128, d) for i in (0, 2))
    s = scale * torch.einsum("bwhgd,htd->bwhgt", x, k) + times.log()[None, :, None, None]
    want = torch.einsum("bwhgt,htd->bwhgd", torch.softmax(s, -1), v).reshape(q.shape)
    top = 30 * float(pool[3].max())
    tol = 0.03 * want.abs().max() + 2.0 ** -10 * top + 2.0 ** -8 * want.abs()
    assert bool(((got.double() - want).abs() <= tol).all())
