"""kda_cache_weigh against the softmax in 64 bits.

Tolerance, element by element. A score is an fp32 sum of at most 128 exact products (fp32 queries:
known to 2^-22; windows of more than 64 query rows: to 2^-20 of the query's largest entry, 2^-17 of
that sum for the queries here): |ds| <= 2^-16 of the sum of absolute products (3/2 of it in such
windows), whose largest over the row's keys is top; a weight p = exp(s - lse) moves by at most
2 |ds| p, the exponentials, the sums of at most 2^13 weights and of the old weight by 2^-18 of the
result together."""
import numpy as np
import pytest
import torch

import bounded_ref as bref
import serving_ref as ref
from kda_testutil import f64
from linear_attention_state_kda_gb300 import kda
from test_gpu_cache_attention import DEV, _i32, _make

pytestmark = pytest.mark.gpu


def _weights(n_pages, H, seed=0):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return torch.rand(n_pages, H, 64, generator=gen, device=DEV)


def check(q, start, lens, table, pool, before, got, scale, keep):
    want = f64(before)
    size, written = bref.weigh(f64(q), start, lens, table.cpu().numpy(), ref.values(pool[0]),
                               f64(pool[1]), want, scale, keep, len(start))
    got = f64(got)
    err = np.abs(got - want)
    many = q.shape[0] // len(start) * (q.shape[1] // pool[0].shape[1]) > 64
    tol = 2.0 ** -15 * (1.5 if many else 1) * size + 2.0 ** -18 * np.abs(want) + 1e-37
    ok = np.where(written, err <= tol, got == f64(before))
    assert ok.all(), float(np.where(written, err / tol, 0).max())


@pytest.mark.parametrize("start,W,Hq,Hkv,d,dtype", [
    ([0], 1, 1, 1, 128, "bf16"), ([0, 1, 62, 63, 64, 65], 1, 8, 2, 128, "bf16"),
    ([127, 700, 5], 1, 32, 8, 128, "bf16"), ([1000, 3, 129, 64], 4, 16, 2, 128, "bf16"),
    ([90, 31], 16, 8, 8, 128, "bf16"), ([333, 60], 3, 48, 3, 128, "bf16"),
    ([2000, 15], 1, 16, 1, 64, "bf16"), ([70, 400, 0], 5, 15, 3, 64, "bf16"),
    ([300, 2], 70, 4, 2, 128, "bf16"), ([500, 64], 33, 6, 2, 64, "bf16"),
    ([1000, 0, 191], 64, 16, 2, 128, "bf16"), ([130], 300, 2, 1, 128, "bf16"),
    ([2500, 63], 17, 8, 2, 128, "bf16"), ([5, 700], 65, 3, 3, 128, "bf16"),
    ([129, 40], 1, 12, 4, 128, "f32"), ([500, 7], 3, 15, 3, 64, "f32"),
    ([300], 7, 16, 1, 128, "f32"), ([0, 63], 40, 8, 2, 64, "f32"), ([5000], 1, 4, 2, 128, "f32")])
def test_parity(start, W, Hq, Hkv, d, dtype):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(sum(start) + 17 * W + d)
    q, table, pool = _make(gen, start, W, Hq, Hkv, d, dtype)
    scale = 0.3 * d ** -0.5
    before = _weights(pool[0].shape[0], Hkv)
    got = before.clone()
    r = kda.cache_weigh(q, _i32(start), table, pool[0], pool[1], got, scale=scale, keep=0.75)
    assert r is got
    check(q, start, None, table, pool, before, got, scale, 0.75)
    again = before.clone()
    kda.cache_weigh(q.reshape(len(start), W, Hq, d), _i32(start), table, pool[0], pool[1], again,
                    scale=scale, keep=0.75)
    assert torch.equal(again, got)


@pytest.mark.parametrize("dtype,wide", [("bf16", 1), ("f32", 1), ("bf16", 20)])
def test_ragged_padded_and_absent(dtype, wide):
    """Padding rows, windows of no token, absent and bad pages, positions past the table, unseen
    NaN codes, and entries that hold NaN where nothing of the old value counts."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(4)
    # (wide: 80 query heads a key/value head, more than 64 query rows)
    start, lens, W = [200, -1, 70, 30, 100, 0], [2, 4, 0, 9, 4, 1], 4
    q, table, pool = _make(gen, start, W, 8 * wide, 2, 128, dtype)
    table[0, 1] = -1
    table[4, :] = -3
    n_pages = pool[0].shape[0]
    table[3, 0] = n_pages + 5
    codes = pool[0]
    codes[table[0, 3].item(), :, 10:] = 0x7f  # after position 201, the last one seen
    before = _weights(n_pages, 2)
    before[table[0, 3].item(), :, 8:] = float("nan")  # the window's own tokens and later ones
    got = before.clone()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    kda.cache_weigh(q, _i32(start), table, pool[0], pool[1], got, scale=0.03, lens=_i32(lens),
                    status=status)
    assert int(status) == kda.STATUS_BAD_PAGE
    table[3, 0] = -1
    clean, got2 = torch.nan_to_num(before), torch.nan_to_num(got)
    check(q, start, lens, table, pool, clean, got2, 0.03, 1.0)
    assert not torch.isnan(got[table[0, 3].item(), :, :10]).any()
    assert torch.isnan(got[table[0, 3].item(), :, 10:]).all()
    # keep = 0: what was there does not count, NaN included
    got = torch.full_like(before, float("nan"))
    kda.cache_weigh(q, _i32(start), table, pool[0], pool[1], got, scale=0.03, lens=_i32(lens), keep=0)
    check(q, start, lens, table, pool, torch.zeros_like(before), torch.nan_to_num(got), 0.03, 0.0)
    assert torch.isnan(got[table[1, 0].item()]).all()


def test_past_the_table():
    gen = torch.Generator(device=DEV)
    gen.manual_seed(5)
    q, table, pool = _make(gen, [100, 20], 3, 4, 2, 64, "bf16")
    before = _weights(pool[0].shape[0], 2)
    got = before.clone()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    kda.cache_weigh(q, _i32([500, 20]), table, pool[0], pool[1], got, scale=0.05, status=status)
    assert int(status) == kda.STATUS_BAD_PAGE
    # every position of the table is seen and older than the window
    cut = q.clone()
    want = before.clone()
    big = torch.cat([table, torch.full((2, 8), -1, dtype=torch.int32, device=DEV)], 1).contiguous()
    kda.cache_weigh(cut, _i32([500, 20]), big, pool[0], pool[1], want, scale=0.05)
    assert torch.allclose(got, want, rtol=1e-5, atol=1e-9)


@pytest.mark.parametrize("W", [2, 40])
@pytest.mark.parametrize("spread", [1.0, 1e4, 1e-20])
def test_extreme_scores(spread, W):
    """Scores far apart (one key takes all), and queries near the ends of the range."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(6)
    start = [700, 65]
    q, table, pool = _make(gen, start, W, 8, 2, 128, "bf16")
    q = (q.float() * spread).bfloat16()
    before = _weights(pool[0].shape[0], 2)
    got = before.clone()
    scale = 0.3 * 128 ** -0.5 / (spread if spread < 1 else 1)
    kda.cache_weigh(q, _i32(start), table, pool[0], pool[1], got, scale=scale)
    assert torch.isfinite(got).all()
    want = f64(before)
    bref.weigh(f64(q), start, None, table.cpu().numpy(), ref.values(pool[0]), f64(pool[1]), want,
               scale, 1.0, 2)
    # the sums of a row's weights are its queries, whatever the scores
    assert abs(f64(got).sum() - want.sum()) < 1e-3 * W
    if spread <= 1:
        check(q, start, None, table, pool, before, got, scale, 1.0)


@pytest.mark.parametrize("dtype,d,W,Hq", [("bf16", 128, 1, 8), ("f32", 64, 1, 8), ("bf16", 64, 48, 4),
                                          ("f32", 128, 20, 4), ("bf16", 128, 64, 8),
                                          ("bf16", 128, 150, 4)])
def test_long_context(dtype, d, W, Hq):
    """More keys than the scores have room for, against float64 on the GPU."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(7)
    n, Hkv = 150001, 2
    q, table, pool = _make(gen, [n], W, Hq, Hkv, d, dtype)
    before = _weights(pool[0].shape[0], Hkv)
    got = before.clone()
    scale = 0.3 * d ** -0.5
    kda.cache_weigh(q, _i32([n]), table, pool[0], pool[1], got, scale=scale)
    val = torch.tensor(ref.code_values(), device=DEV)
    page = table[0].long()
    k = val[pool[0][page].long()] * pool[1][page].double()[..., None, None]
    k = k.transpose(0, 1).reshape(Hkv, -1, d)[:, :n + W]
    qq = q.double().reshape(W, Hkv, Hq // Hkv, d)
    s = torch.einsum("whgd,htd->hwgt", qq, k) * scale
    later = torch.ones(W, n + W, dtype=torch.bool, device=DEV).triu(n + 1)
    p = torch.softmax(s.masked_fill(later[:, None], -float("inf")), -1).sum((1, 2))
    old = before[page].transpose(0, 1).reshape(Hkv, -1)[:, :n + W].double().clone()
    old[:, n:] = 0
    now = got[page].transpose(0, 1).reshape(Hkv, -1)[:, :n + W].double()
    # scores below 16, sums of absolute products below 64 here: 2 * 2^-16 * 64 in the worst case
    top = (qq.abs().amax() * k.abs().amax() * d * scale).item()
    assert ((now - old - p).abs() <= 2.0 ** -15 * top * p + 2.0 ** -18 * (p + old)).all()


def test_many_rows_graph_and_stream():
    gen = torch.Generator(device=DEV)
    gen.manual_seed(8)
    start = torch.randint(0, 150, (300,), generator=gen, device=DEV).tolist()
    q, table, pool = _make(gen, start, 1, 4, 2, 64, "bf16")
    before = _weights(pool[0].shape[0], 2)
    got = before.clone()
    st = _i32(start)
    kda.cache_weigh(q, st, table, pool[0], pool[1], got, scale=0.05)
    check(q, start, None, table, pool, before, got, 0.05, 1.0)
    w = before.clone()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        kda.cache_weigh(q, st, table, pool[0], pool[1], w, scale=0.05)
    w.copy_(before)
    gr.replay()
    assert torch.equal(w, got)
    w.copy_(before)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    kda.cache_weigh(q, st, table, pool[0], pool[1], w, scale=0.05, stream=side)
    side.synchronize()
    assert torch.equal(w, got)


def test_infinite_and_nan_queries():
    """A query with an infinity or NaN makes its own row's weights NaN where it sees, nothing else."""
    for W in (2, 40):
        gen = torch.Generator(device=DEV)
        gen.manual_seed(9)
        q, table, pool = _make(gen, [100, 70], W, 8, 2, 128, "bf16")
        clean = torch.zeros(pool[0].shape[0], 2, 64, device=DEV)
        kda.cache_weigh(q, _i32([100, 70]), table, pool[0], pool[1], clean, scale=0.03)
        for x in (float("nan"), float("inf")):
            bad = q.clone()
            bad[W - 1, 5, 17] = x  # the last token of row 0, head 1's group
            got = torch.zeros_like(clean)
            kda.cache_weigh(bad, _i32([100, 70]), table, pool[0], pool[1], got, scale=0.03)
            page = table[0].long()
            mine = got[page, 1].reshape(-1)[:100 + W]
            assert torch.isnan(mine).all()
            got[page, 1] = clean[page, 1]
            assert torch.equal(got, clean)


@pytest.mark.parametrize("dtype,d,W,Hq", [("bf16", 128, 4, 8), ("bf16", 64, 4, 24), ("f32", 128, 4, 8),
                                          ("f32", 64, 9, 16)])
def test_wide_tables(dtype, d, W, Hq):
    """Few rows with wide page tables: statistics and weights in a launch each, most ranges of keys
    empty. Padding rows, windows of no token, absent pages, several groups of query rows; and two
    captured graphs that share a workspace."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(10)
    start, lens = [200, -1, 70, 30, 1000, 0], [2, 4, 0, W, W - 1, 1]
    q, table, pool = _make(gen, start, W, Hq, 2, d, dtype)
    table[0, 1] = -1
    table[4, 3] = -7
    wide = torch.full((6, 700), -1, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = table
    wide[5, 690] = 0  # far behind what row 5 sees
    need = kda.cache_weigh_workspace(q.dtype, 6, W, Hq, 2, d, 700)
    assert need > 0
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device=DEV)
    before = _weights(pool[0].shape[0], 2)
    got = before.clone()
    args = (_i32(start), wide, pool[0], pool[1])
    kda.cache_weigh(q, *args, got, scale=0.04, lens=_i32(lens), keep=0.5, workspace=ws)
    check(q, start, lens, table, pool, before, got, 0.04, 0.5)
    q2, ln = q.flip(0).contiguous(), _i32(lens)
    want = before.clone()
    kda.cache_weigh(q2, *args, want, scale=0.04, lens=ln, keep=0.5)
    a, b = before.clone(), before.clone()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for gr, x, w in zip(graphs, (q, q2), (a, b)):
        with torch.cuda.graph(gr):
            kda.cache_weigh(x, *args, w, scale=0.04, lens=ln, keep=0.5, workspace=ws)
    for _ in range(2):
        a.copy_(before)
        b.copy_(before)
        graphs[0].replay()
        graphs[1].replay()
    assert torch.equal(a, got) and torch.equal(b, want)


@pytest.mark.parametrize("dtype,d,W", [("bf16", 128, 1), ("f32", 64, 3)])
def test_more_keys_than_a_cluster_has_room_for(dtype, d, W):
    """Many rows (clusters), one of them longer than the scores have room for."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(11)
    start = [40000] + [3 * i for i in range(19)]
    q, table, pool = _make(gen, start, W, 16, 2, d, dtype)
    before = _weights(pool[0].shape[0], 2)
    got = before.clone()
    scale = 0.3 * d ** -0.5
    assert kda.cache_weigh_workspace(q.dtype, 20, W, 16, 2, d, table.shape[1]) == 0
    kda.cache_weigh(q, _i32(start), table, pool[0], pool[1], got, scale=scale)
    check(q, start, None, table, pool, before, got, scale, 1.0)


def test_many_queries_in_two_graphs():
    """Windows of more than 64 query rows, captured: two graphs that share a workspace."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(12)
    start, W = [700, 3], 40
    q, table, pool = _make(gen, start, W, 8, 2, 128, "bf16")
    ws = torch.empty(kda.cache_weigh_workspace(q.dtype, 2, W, 8, 2, 128, table.shape[1]),
                     dtype=torch.uint8, device=DEV)
    qs, st = (q, q.flip(0).contiguous()), _i32(start)
    before = _weights(pool[0].shape[0], 2)
    want = [before.clone() for _ in qs]
    for x, w in zip(qs, want):
        kda.cache_weigh(x, st, table, pool[0], pool[1], w, scale=0.04)
    got, graphs = [before.clone() for _ in qs], [torch.cuda.CUDAGraph() for _ in qs]
    for gr, x, w in zip(graphs, qs, got):
        with torch.cuda.graph(gr):
            kda.cache_weigh(x, st, table, pool[0], pool[1], w, scale=0.04, workspace=ws)
    for w in got:
        w.copy_(before)
    for gr in graphs:
        gr.replay()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
