"""kda_cache_attention with many query rows per key/value head (windows times grouped heads), where
the keys and channels, not the rows, fill the tensor cores' tiles. Tolerances as in
test_gpu_cache_attention: 2^-10 max|v| + 2^-8 |o| for bf16."""
import numpy as np
import pytest
import torch

from linear_attention_state_kda_gb300 import kda
from test_gpu_cache_attention import DEV, _check, _i32, _make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("start,W,Hq,Hkv,d", [
    ([0], 16, 4, 2, 128), ([127, 128, 129, 0], 6, 12, 4, 128), ([300, 5], 16, 8, 2, 128),
    ([1500, 63, 255], 9, 21, 3, 128), ([700], 13, 10, 2, 128), ([40, 2000], 16, 24, 1, 128),
    ([90, 31], 5, 20, 4, 64), ([400, 7], 16, 8, 2, 64)])
def test_parity(start, W, Hq, Hkv, d):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(sum(start) + 5 * W + Hq)
    q, table, pool = _make(gen, start, W, Hq, Hkv, d, "bf16")
    scale = 0.3 * d ** -0.5
    got = kda.cache_attention(q, _i32(start), table, *pool, scale=scale)
    _check(q, start, None, table, pool, scale, "bf16", got)
    again = kda.cache_attention(q, _i32(start), table, *pool, scale=scale)
    assert torch.equal(again, got)


@pytest.mark.parametrize("G", [6, 12])
def test_many_rows_of_ragged_length(G):
    """More units than SMs, so that most are cut and several share an SM."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(78)
    start = [0, 1, 2, 1500, 5, 64, 700, 100, 1, 0, 900, 63, 64, 65, 127, 128] * 3 + [2500, -1]
    lens = [4, 4, 1, 2, 3, 4, 0, 4, 4, 4, 4, 3, 2, 4, 4, 4] * 3 + [4, 4]
    q, table, pool = _make(gen, start, 4, 4 * G, 4, 128, "bf16")
    got = kda.cache_attention(q, _i32(start), table, *pool, scale=0.04, lens=_i32(lens))
    _check(q, start, lens, table, pool, 0.04, "bf16", got)


def test_growing_scores():
    """Keys whose scores grow along the context: the rows' maximum is raised again and again."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(6)
    start, W, G = [1200, 300], 4, 8
    q, table, pool = _make(gen, start, W, 2 * G, 2, 128, "bf16")
    host = table.cpu().numpy()
    q[:] = q.abs()
    for b in range(2):
        for blk, page in enumerate(host[b]):
            pool[0][page] &= 0x7f                      # positive keys
            pool[1][page] = 2.0 ** (-9 + blk // 2)     # larger page by page
    got = kda.cache_attention(q, _i32(start), table, *pool, scale=0.05)
    _check(q, start, None, table, pool, 0.05, "bf16", got)


def test_pages_of_very_different_scales():
    """Value pages from 2^-60 to 2^20: a page whose values are tiny still counts in the sum of
    weights, and one with huge values but no weight stays out."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(7)
    start, W, G = [500], 4, 8
    q, table, pool = _make(gen, start, W, 2 * G, 2, 128, "bf16")
    page = table.cpu().numpy()[0]
    pool[3][page[0]] = 2.0 ** -60
    pool[3][page[2]] = 2.0 ** 20
    got = kda.cache_attention(q, _i32(start), table, *pool, scale=0.05)
    _check(q, start, None, table, pool, 0.05, "bf16", got)


@pytest.mark.parametrize("W,G,d", [(4, 8, 128), (8, 8, 128), (16, 5, 128), (8, 4, 64)])
def test_masked_rows_absent_pages_and_stale_codes(W, G, d):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(5)
    start, lens = [200, -1, 70, 100, 64, 40], [W, W, 2, 0, W, W]
    q, table, pool = _make(gen, start, W, 2 * G, 2, d, "bf16")
    host = table.cpu().numpy()
    table[0, 1] = -1
    table[4] = _i32([-1] * table.shape[1])
    table[5, 0] = 10 ** 6
    used = {int(p) for b in (0, 2) for p in host[b]}
    for i in (0, 2):
        for page in range(pool[i].shape[0]):
            if page not in used:
                pool[i][page] = 0x7f
        for b in (0, 2):
            end = start[b] + lens[b]
            pool[i][host[b][end // 64], :, end % 64:] = 0xff
            for blk in range(end // 64 + 1, host.shape[1]):
                pool[i][host[b][blk]] = 0x7f
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = kda.cache_attention(q, _i32(start), table, *pool, scale=0.05, lens=_i32(lens),
                              status=status)
    assert int(status) == kda.STATUS_BAD_PAGE
    assert torch.isfinite(got.float()).all()
    for b in (1, 3, 4, 5):
        assert (got[b * W:(b + 1) * W] == 0).all()
    _check(q, start, lens, table, pool, 0.05, "bf16", got)
    # NaN in the window's third token
    at = start[0] + 2
    for i, nan in ((0, 0x7f), (2, 0xff)):
        keep = pool[i].clone()
        pool[i][host[0][at // 64], 0, at % 64, 7] = nan
        one = kda.cache_attention(q, _i32(start), table, *pool, scale=0.05, lens=_i32(lens))
        assert torch.equal(one[:2], got[:2]) and torch.equal(one[W:], got[W:])
        assert torch.equal(one[:W, G:], got[:W, G:])
        bad = torch.isnan(one[2:W, :G].float())
        if i == 0:
            assert bad.all()
        else:
            assert bad[..., 7].all() and int(bad.sum()) == bad[..., 7].numel()
        pool[i].copy_(keep)
    # infinity and NaN in a query row stay in that row
    q2 = q.clone()
    q2[0, 0, 3], q2[1, 1, 4] = float("inf"), float("nan")
    one = kda.cache_attention(q2, _i32(start), table, *pool, scale=0.05, lens=_i32(lens))
    assert torch.isnan(one[0, 0].float()).all() and torch.isnan(one[1, 1].float()).all()
    same = np.ones((q.shape[0], q.shape[1]), dtype=bool)
    same[0, 0] = same[1, 1] = False
    assert torch.equal(one[torch.from_numpy(same)], got[torch.from_numpy(same)])


def test_table_entries_past_the_context_are_not_looked_at():
    """Only pages that a query sees are looked up: what the table holds after them is not."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(8)
    start = [190, 60]
    for W, G in ((1, 4), (4, 8)):
        q, table, pool = _make(gen, start, W, 2 * G, 2, 128, "bf16")
        want = kda.cache_attention(q, _i32(start), table, *pool, scale=0.05)
        wide = torch.full((2, 9), 2 ** 31 - 1, dtype=torch.int32, device=DEV)
        for b in range(2):
            n = (start[b] + W + 63) // 64
            wide[b, :n] = table[b, :n]
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        got = kda.cache_attention(q, _i32(start), wide, *pool, scale=0.05, status=status)
        assert torch.equal(got, want) and int(status) == 0


@pytest.mark.parametrize("start,W,Hq,Hkv,d,dtype", [
    ([0], 200, 4, 2, 128, "bf16"), ([37, 0], 130, 6, 2, 64, "bf16"), ([500], 333, 2, 1, 128, "bf16"),
    ([0, 90], 65, 3, 3, 64, "f32"), ([64], 17, 2, 2, 128, "f32")])
def test_chunks_of_a_prompt(start, W, Hq, Hkv, d, dtype):
    """Windows longer than a verify window: many row groups, whose first rows see few keys; with a
    ragged length, and a NaN value that only the last tokens see."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(W + d)
    q, table, pool = _make(gen, start, W, Hq, Hkv, d, dtype)
    lens = [W] + [W - 9] * (len(start) - 1)
    scale = 0.3 * d ** -0.5
    got = kda.cache_attention(q, _i32(start), table, *pool, scale=scale, lens=_i32(lens))
    _check(q, start, lens, table, pool, scale, dtype, got)
    at = start[0] + W - 3
    pool[2][int(table[0, at // 64]), :, at % 64, 5] = 0x7f
    one = kda.cache_attention(q, _i32(start), table, *pool, scale=scale, lens=_i32(lens))
    assert torch.equal(one[:W - 3], got[:W - 3]) and torch.equal(one[W:], got[W:])
    assert torch.isnan(one[W - 3:W, :, 5].float()).all()
    rest = torch.arange(d, device=DEV) != 5
    assert torch.equal(one[W - 3:W][..., rest], got[W - 3:W][..., rest])
