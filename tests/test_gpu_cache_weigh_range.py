"""kda_cache_weigh where scores are far apart, key by key, and at the ends of the ranges of queries and
key scales; and windows of many query rows over wide tables.

A score is off by at most ds = 2^-16 of its sum of absolute products (3/2 of that with more than 64
query rows; their largest over the row's keys is taken for all), so a weight p = exp(s - lse) lies
between p e^-2ds and p e^2ds, and, as a query's weights add up to 1, is at least 1 minus the most that
the others can be. Scores and the logarithm of their sum are fp32 numbers: the rounding of either, 2^-24
of the largest score each, moves a weight by e to that, 2^-22 of it with the products' own roundings, and
a query's sum with it. The exponentials and sums are off by 2^-18 of the result."""
import numpy as np
import pytest
import torch

import serving_ref as ref
from kda_testutil import f64
from linear_attention_state_kda_gb300 import kda
from test_gpu_cache_attention import DEV, _i32, _make
from test_gpu_cache_weigh import _weights, check

pytestmark = pytest.mark.gpu


def bounds(q, start, table, pool, before, scale, W):
    """Smallest and largest weights, [n_pages, Hkv, 64], and by how much the best key of each query
    leads at least: the share that it must hold."""
    lo, hi = f64(before).copy(), f64(before).copy()
    Hkv, G = pool[0].shape[1], q.shape[1] // pool[0].shape[1]
    ds = 2.0 ** -16 * (1.5 if W * G > 64 else 1.0)
    qq, table, shares = f64(q), table.cpu().numpy(), []
    for b, s0 in enumerate(start):
        k, there = ref.gather(ref.values(pool[0]), f64(pool[1]), table[b], s0 + W, pool[0].shape[0])
        t = np.arange(s0 + W)
        assert there.all()
        for x in (lo, hi):
            x[table[b][t[s0:] // 64], :, t[s0:] % 64] = 0.0
        for j in range(W):
            n = s0 + j + 1
            page, at = table[b][t[:n] // 64], t[:n] % 64
            for h in range(q.shape[1]):
                kh, x = k[:n, h // G], qq[b * W + j, h]
                s = scale * (kh @ x)
                off = 2 * ds * scale * (np.abs(kh) @ np.abs(x)).max()
                z = s - s.max()
                lse = np.log(np.exp(z).sum())
                fp32 = np.exp(2.0 ** -22 * np.abs(s).max())
                most = np.exp(np.minimum(z - lse + off, 0.0)) * fp32
                rest = most.sum() - most
                least = np.maximum(np.exp(z - lse - off), 1.0 - rest) / fp32
                lo[page, h // G, at] += least
                hi[page, h // G, at] += most
                shares.append(least.max())
    return lo, hi, np.array(shares)


@pytest.mark.parametrize("W,d,dtype", [(2, 128, "bf16"), (40, 128, "bf16"), (3, 64, "bf16"),
                                       (2, 128, "f32")])
def test_one_key_takes_all(W, d, dtype):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(41)
    start = [700, 65]
    q, table, pool = _make(gen, start, W, 8, 2, d, dtype)
    q = (q.float() * 1e4).to(q.dtype)
    before = _weights(pool[0].shape[0], 2)
    got = before.clone()
    scale = 0.3 * d ** -0.5
    kda.cache_weigh(q, _i32(start), table, pool[0], pool[1], got, scale=scale)
    lo, hi, shares = bounds(q, start, table, pool, before, scale, W)
    assert (shares > 0.99).mean() > 0.8  # the bounds say which key it is
    got = f64(got)
    off = 2.0 ** -18 * hi + 1e-37
    assert (got >= lo - off).all() and (got <= hi + off).all()


@pytest.mark.parametrize("down,up", [(-126, 122), (-126, 110), (-120, 100), (-95, 60), (100, -90)])
@pytest.mark.parametrize("W,d,dtype", [(2, 128, "bf16"), (40, 128, "bf16"), (5, 64, "bf16"),
                                       (2, 128, "f32")])
def test_small_queries_and_large_scales(W, d, dtype, down, up):
    """Queries near the ends of fp32's range (bf16 entries below the normal range among them) and key
    scales that bring the scores back."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(42)
    start = [300, 65]
    q, table, pool = _make(gen, start, W, 8, 2, d, dtype)
    q = (q.double() * 2.0 ** down).to(q.dtype)
    ks = (pool[1].double() * 2.0 ** up).float()
    before = _weights(pool[0].shape[0], 2)
    got = before.clone()
    scale = 0.3 * d ** -0.5 * 2.0 ** (-down - up)
    kda.cache_weigh(q, _i32(start), table, pool[0], ks, got, scale=scale)
    check(q, start, None, table, [pool[0], ks], before, got, scale, 1.0)


@pytest.mark.parametrize("W,Hq", [(150, 16), (21, 400)])
def test_many_rows_in_two_launches(W, Hq):
    """Wide tables, and more query rows than the statistics are kept of at a time."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(43)
    start, lens = [130, -1, 64, 3], [W, 4, W - 1, 1]
    q, table, pool = _make(gen, start, W, Hq, 2, 64, "f32")
    wide = torch.full((4, 600), -1, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = table
    assert kda.cache_weigh_workspace(q.dtype, 4, W, Hq, 2, 64, 600) > 0
    before = _weights(pool[0].shape[0], 2)
    got = before.clone()
    kda.cache_weigh(q, _i32(start), wide, pool[0], pool[1], got, scale=0.04, lens=_i32(lens), keep=0.5)
    check(q, start, lens, wide, pool, before, got, 0.04, 0.5)
