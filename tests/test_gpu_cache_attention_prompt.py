"""kda_cache_attention over chunks of a prompt: more than 64 bf16 query rows per key/value head, which
run in units of 256 rows on their own kernel. Tolerances as in test_gpu_cache_attention: 2^-10 max|v|
+ 2^-8 |o|."""
import numpy as np
import pytest
import torch

from linear_attention_state_kda_gb300 import kda
from test_gpu_cache_attention import DEV, _check, _i32, _make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("start,W,Hq,Hkv,d", [
    ([0], 65, 1, 1, 128), ([127, 128, 0], 16, 8, 1, 128), ([63, 64], 43, 6, 2, 128),
    ([255, 1], 64, 8, 2, 128), ([900], 257, 2, 2, 128), ([0, 129], 100, 14, 2, 128),
    ([0], 128, 1, 1, 64), ([300, 5], 40, 10, 2, 64), ([1000], 86, 3, 1, 64), ([0], 520, 1, 1, 64)])
def test_parity(start, W, Hq, Hkv, d):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(sum(start) + 3 * W + Hq + d)
    q, table, pool = _make(gen, start, W, Hq, Hkv, d, "bf16")
    scale = 0.3 * d ** -0.5
    got = kda.cache_attention(q, _i32(start), table, *pool, scale=scale)
    _check(q, start, None, table, pool, scale, "bf16", got)
    again = kda.cache_attention(q, _i32(start), table, *pool, scale=scale)
    assert torch.equal(again, got)


@pytest.mark.parametrize("d", [64, 128])
def test_ragged_chunks_of_many_rows(d):
    """Units that are cut, several on an SM, row groups without a token, and more than 32 rows."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(d)
    start = [0, 1, 130, 700, 5, 64, -1, 100, 1, 0, 300] * 3 + [400, -1]
    lens = [90, 3, 64, 65, 1, 90, 9, 0, 33, 64, 2] * 3 + [90, 0]
    q, table, pool = _make(gen, start, 90, 8, 2, d, "bf16")
    got = kda.cache_attention(q, _i32(start), table, *pool, scale=0.05, lens=_i32(lens))
    _check(q, start, lens, table, pool, 0.05, "bf16", got)
    for b, n in enumerate(lens):
        if start[b] < 0 or n == 0:
            assert (got[b * 90:(b + 1) * 90] == 0).all()
        assert (got[b * 90 + n:(b + 1) * 90] == 0).all()


def test_one_long_row_is_cut_over_all_sms():
    gen = torch.Generator(device=DEV)
    gen.manual_seed(3)
    q, table, pool = _make(gen, [9000], 20, 4, 1, 128, "bf16")
    got = kda.cache_attention(q, _i32([9000]), table, *pool, scale=0.04)
    _check(q, [9000], None, table, pool, 0.04, "bf16", got)


@pytest.mark.parametrize("d", [64, 128])
def test_growing_scores_and_different_scales(d):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(6)
    start, W = [1200, 300], 70
    q, table, pool = _make(gen, start, W, 4, 2, d, "bf16")
    host = table.cpu().numpy()
    grow = [p.clone() for p in pool]
    q2 = q.abs()
    for b in range(2):
        for blk, page in enumerate(host[b]):
            grow[0][page] &= 0x7f                      # positive keys
            grow[1][page] = 2.0 ** (-9 + blk // 2)     # larger page by page
    got = kda.cache_attention(q2, _i32(start), table, *grow, scale=0.05)
    _check(q2, start, None, table, grow, 0.05, "bf16", got)
    # tiny values count in the sum of weights, huge ones without weight stay out; a negative scale
    pool[3][host[0][0]] = 2.0 ** -60
    pool[3][host[0][3]] = 2.0 ** 20
    got = kda.cache_attention(q, _i32(start), table, *pool, scale=-0.05)
    _check(q, start, None, table, pool, -0.05, "bf16", got)


@pytest.mark.parametrize("W,G,d", [(96, 4, 128), (70, 1, 128), (130, 3, 64)])
def test_absent_pages_stale_codes_and_nan(W, G, d):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(5)
    start, lens = [200, -1, 70, 100, 64, 40], [W, W, 2, 0, W, W]
    q, table, pool = _make(gen, start, W, 2 * G, 2, d, "bf16")
    host = table.cpu().numpy()
    table[0, 1] = -1
    table[4] = _i32([-1] * table.shape[1])
    table[5, 0] = 10 ** 6
    used = {int(p) for b in (0, 2, 5) for p in host[b]}
    for i in (0, 2):
        for page in range(pool[i].shape[0]):
            if page not in used:
                pool[i][page] = 0x7f
        for b in (0, 2, 5):
            end = start[b] + lens[b]
            pool[i][host[b][end // 64], :, end % 64:] = 0xff
            for blk in range(end // 64 + 1, host.shape[1]):
                pool[i][host[b][blk]] = 0x7f
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = kda.cache_attention(q, _i32(start), table, *pool, scale=0.05, lens=_i32(lens),
                              status=status)
    assert int(status) == kda.STATUS_BAD_PAGE
    assert torch.isfinite(got.float()).all()
    _check(q, start, lens, table, pool, 0.05, "bf16", got)
    # NaN in a token of the window reaches the tokens from there on: a key the whole row, a value
    # its channel
    j = W - 30
    at = start[0] + j
    for i, nan in ((0, 0x7f), (2, 0xff)):
        keep = pool[i].clone()
        pool[i][host[0][at // 64], 1, at % 64, d - 2] = nan
        one = kda.cache_attention(q, _i32(start), table, *pool, scale=0.05, lens=_i32(lens))
        assert torch.equal(one[:j], got[:j]) and torch.equal(one[W:], got[W:])
        assert torch.equal(one[:, :G], got[:, :G])
        bad = torch.isnan(one[j:W, G:].float())
        if i == 0:
            assert bad.all()
        else:
            assert bad[..., d - 2].all() and int(bad.sum()) == bad[..., d - 2].numel()
        pool[i].copy_(keep)
    # infinity and NaN in a query row stay in that row
    q2 = q.clone()
    q2[0, 0, 3], q2[1, 1, 4] = float("inf"), float("nan")
    one = kda.cache_attention(q2, _i32(start), table, *pool, scale=0.05, lens=_i32(lens))
    assert torch.isnan(one[0, 0].float()).all() and torch.isnan(one[1, 1].float()).all()
    same = np.ones((q.shape[0], q.shape[1]), dtype=bool)
    same[0, 0] = same[1, 1] = False
    same = torch.from_numpy(same)
    assert torch.equal(one[same], got[same])


def test_large_and_tiny_queries():
    """Rows of very different size in one unit: each is scaled by its own power of two."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(11)
    q, table, pool = _make(gen, [150], 80, 2, 2, 128, "bf16")
    q *= (2.0 ** torch.arange(-40, 40, device=DEV).float()).to(q.dtype)[:, None, None]
    got = kda.cache_attention(q, _i32([150]), table, *pool, scale=2.0 ** -44)
    _check(q, [150], None, table, pool, 2.0 ** -44, "bf16", got)
