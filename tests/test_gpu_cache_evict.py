"""kda_cache_evict against a plain implementation: positions, codes, scales and weights are equal."""
import numpy as np
import pytest
import torch

import bounded_ref as bref
import serving_ref as ref
from kda_testutil import f64
from linear_attention_state_kda_gb300 import kda
from test_gpu_cache_attention import DEV, _i32, _make

pytestmark = pytest.mark.gpu


def _setup(length, Hkv, d, budget, seed=0, zeros=True):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    width = -(-budget // 64)
    q, table, pool = _make(gen, [max(x - 1, 0) for x in length], 1, Hkv, Hkv, d, "bf16",
                           spare=len(length) * width + 2)
    n_pages = pool[0].shape[0]
    used = set(table.flatten().tolist())
    free = [p for p in range(n_pages) if p not in used][:len(length) * width]
    new = _i32(free).reshape(len(length), width) if free else \
        torch.empty(len(length), 0, dtype=torch.int32, device=DEV)
    w = torch.rand(n_pages, Hkv, 64, generator=gen, device=DEV)
    w = torch.round(w * 50) / 50 if zeros else w  # many equal ones
    return table, new, [p.contiguous() for p in pool], w


def _run(length, table, new, pool, w, budget, sinks, recent):
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    pool2, w2 = [p.clone() for p in pool], w.clone()
    count, kept = kda.cache_evict(_i32(length), table, new, *pool2, w2, budget, sinks=sinks,
                                  recent=recent, status=status)
    sides = [(ref.values(pool[0]).copy(), f64(pool[1])), (ref.values(pool[2]).copy(), f64(pool[3]))]
    ww = f64(w)
    c, k = bref.evict(length, table.cpu().numpy(), new.cpu().numpy(), sides, ww, budget, sinks, recent)
    assert count.tolist() == c.tolist()
    assert np.array_equal(kept.cpu().numpy(), k)
    assert np.array_equal(f64(w2), ww, equal_nan=True)
    dst = new.cpu().numpy()
    for b, n in enumerate(c):
        for i in range(0, max(int(n), 0), 64):
            page, m = dst[b][i // 64], min(64, int(n) - i)
            if not 0 <= page < w.shape[0]:
                continue
            for (val, scale), code, s in ((sides[0], pool2[0], pool2[1]), (sides[1], pool2[2], pool2[3])):
                assert np.array_equal(f64(s[page]), scale[page])
                got = ref.values(code[page])[:, :m]
                assert np.array_equal(got, val[page, :, :m], equal_nan=True)
    # the old pages are as they were
    old = table.flatten().long()
    old = old[(old >= 0) & (old < w.shape[0])]
    assert all(torch.equal(a[old], b[old]) for a, b in zip(pool, pool2))
    return int(status), count, kept, pool2, w2


@pytest.mark.parametrize("length,Hkv,d,budget,sinks,recent", [
    ([1], 1, 64, 1, 0, 0), ([200], 2, 128, 64, 0, 0), ([200, 0, 63, 64, 65, 130], 2, 128, 65, 3, 10),
    ([500, 70, 129], 3, 64, 128, 4, 32), ([300, 90], 1, 128, 100, 0, 100), ([300], 2, 64, 100, 100, 0),
    ([1000, 5], 2, 128, 999, 1, 1), ([100, 300], 1, 64, 500, 7, 90), ([64, 64], 4, 64, 63, 0, 1),
    ([3000, 1], 1, 64, 700, 5, 64), ([20], 2, 64, 0, 0, 0)])
def test_parity(length, Hkv, d, budget, sinks, recent):
    x = _setup(length, Hkv, d, budget, seed=sum(length) + budget)
    assert _run(length, *x, budget, sinks, recent)[0] == 0


def test_special_weights():
    """NaN, infinities, zeros of both signs, subnormals, negative weights."""
    length, budget = [400, 190], 96
    table, new, pool, w = _setup(length, 2, 64, budget, seed=2)
    pick = torch.rand(w.shape, device=DEV)
    for i, x in enumerate((float("nan"), float("inf"), -float("inf"), 0.0, -0.0, 1e-42, -1e-42, -3.0)):
        w[(pick > i * 0.1) & (pick < i * 0.1 + 0.07)] = x
    for b in (96, 350, 5):
        _run(length, table, new, pool, w, min(b, 96), 2, 2)
    w.fill_(float("nan"))
    _run(length, table, new, pool, w, budget, 0, 0)
    w.zero_()
    _run(length, table, new, pool, w, budget, 0, 7)


def test_padding_absent_and_bad_pages():
    length, budget = [300, -1, 200, 260, 130, -7], 100
    table, new, pool, w = _setup(length, 2, 128, budget, seed=3)
    n_pages = w.shape[0]
    table[0, 1] = -1
    table[0, 4] = -2
    table[2, :] = -1          # nothing present
    assert _run(length, table, new, pool, w, budget, 70, 20)[0] == 0
    new[3, 1] = -1            # dropped
    assert _run(length, table, new, pool, w, budget, 0, 0)[0] == 0
    table[3, 2] = n_pages
    assert _run(length, table, new, pool, w, budget, 5, 5)[0] == kda.STATUS_BAD_PAGE
    table[3, 2] = -1
    new[4, 0] = n_pages + 3
    assert _run(length, table, new, pool, w, budget, 5, 5)[0] == kda.STATUS_BAD_PAGE


def test_length_past_the_table():
    length = [500, 90]
    table, new, pool, w = _setup([300, 90], 1, 64, 128, seed=4)
    assert _run(length, table, new, pool, w, 128, 3, 40)[0] == kda.STATUS_BAD_PAGE


def test_scales_far_apart():
    """Tokens of pages whose scales differ by more than the format's range meet in one page."""
    length, budget = [640], 128
    table, new, pool, w = _setup(length, 2, 64, budget, seed=5, zeros=False)
    for s in (pool[1], pool[3]):
        e = torch.tensor([-100, -20, 0, 3, 120, -99, -9, -10, -11, 60], device=DEV, dtype=torch.float64)
        s[table[0].long()] = torch.exp2(e)[:, None].float().expand(-1, 2)
    _run(length, table, new, pool, w, budget, 2, 2)


@pytest.mark.parametrize("length,budget,Hkv", [([70000], 5000, 2), ([430000, 17], 2000, 1)])
def test_long(length, budget, Hkv):
    """More positions than a cluster of CTAs holds keys of; few distinct weights."""
    table, new, pool, w = _setup(length, Hkv, 64, budget, seed=6)
    st = _i32(length)
    pool2, w2 = [p.clone() for p in pool], w.clone()
    count, kept = kda.cache_evict(st, table, new, *pool2, w2, budget, sinks=3, recent=50)
    assert count.tolist() == [min(x, budget) for x in length]
    for b, n in enumerate(length):
        flat = w[table[b].long()].transpose(0, 1).reshape(Hkv, -1)[:, :n].clone()
        flat[:, :3] = 9
        flat[:, max(0, n - 50):] = 9
        m = min(n, budget)
        want = torch.sort(flat, dim=-1, descending=True, stable=True)[1][:, :m].sort(-1)[0]
        assert torch.equal(kept[b, :, :m].long(), want)
        assert (kept[b, :, m:] == -1).all()
        moved = w2[new[b].long()].transpose(0, 1).reshape(Hkv, -1)[:, :m]
        old = w[table[b].long()].transpose(0, 1).reshape(Hkv, -1)
        assert torch.equal(moved, old.gather(1, want))


def test_graph_stream_and_given_outputs():
    length, budget = [300, 80], 100
    table, new, pool, w = _setup(length, 2, 128, budget, seed=7)
    st = _i32(length)
    a = [p.clone() for p in pool] + [w.clone()]
    want = kda.cache_evict(st, table, new, *a, budget, sinks=1, recent=9)
    b = [p.clone() for p in pool] + [w.clone()]
    out = [torch.full_like(x, 77) for x in want]
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        r = kda.cache_evict(st, table, new, *b, budget, sinks=1, recent=9, new_length=out[0],
                            kept=out[1])
    assert r[0] is out[0] and r[1] is out[1]
    for x, y in zip(b, pool + [w]):
        x.copy_(y)
    gr.replay()
    live = torch.cat([table.flatten(), new.flatten()]).long()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    read = lambda c: kda.cache_read(_i32([0, 0]), new, *c[:4], 180, cu_seqlens=_i32([0, 100, 180]))  # noqa: E731,E501
    assert all(torch.equal(x, y) for x, y in zip(read(a), read(b)))
    assert torch.equal(a[4][live], b[4][live])
    c = [p.clone() for p in pool] + [w.clone()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = kda.cache_evict(st, table, new, *c, budget, sinks=1, recent=9, stream=side)
    side.synchronize()
    assert torch.equal(got[1], want[1]) and all(torch.equal(x, y) for x, y in zip(read(a), read(c)))
