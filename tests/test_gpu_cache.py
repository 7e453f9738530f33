"""kda_cache_write and kda_cache_read against the definition in 64 bits: the scales are powers of
two, so codes and values have to be equal, not near."""
import numpy as np
import pytest
import torch

import serving_ref as ref
from kda_testutil import f64
from linear_attention_state_kda_gb300 import kda

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _pool(gen, n_pages, H, d):
    """Random codes (no NaN) and power-of-two scales."""
    codes = torch.randint(0, 255, (n_pages, H, 64, d), generator=gen, device=DEV).to(torch.uint8)
    codes[(codes & 127) == 127] = 3
    e = torch.randint(-9, -4, (n_pages, H), generator=gen, device=DEV)
    return codes, torch.exp2(e.double()).float()


def _written(start, lens, n_pages, table):
    """Mask [n_pages, 64] of the rows that hold a defined value after the write."""
    m = np.ones((n_pages, 64), dtype=bool)
    for s, st in enumerate(start):
        if st < 0 or lens[s] <= 0:
            continue
        end = st + lens[s]
        blk = (end - 1) // 64
        page = table[s][blk] if blk < len(table[s]) else -1
        if 0 <= page < n_pages and end % 64:
            m[page, end % 64:] = False
    return m


@pytest.mark.parametrize("lens,start,H,d,dtype,cut", [
    ([1], [0], 1, 128, "bf16", None), ([64, 65, 63], [0, 0, 0], 2, 128, "bf16", None),
    ([1, 1, 1, 1], [63, 64, 1, 130], 3, 64, "bf16", None),
    ([4, 4, 4], [61, 62, 100], 2, 128, "f32", [4, 1, 0]),
    ([200, 0, 7, 129], [37, 5, 0, 63], 5, 64, "f32", None),
    ([70, 3], [-1, 10], 2, 128, "bf16", None),
    ([300], [1], 1, 128, "f32", None)])
def test_write_and_read_back(lens, start, H, d, dtype, cut):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(sum(lens) * 7 + d)
    n, T = len(lens), sum(lens)
    cols = max(1, max((max(s, 0) + m + 63) // 64 for s, m in zip(start, lens)))
    n_pages = n * cols + 2
    table = torch.randperm(n_pages, generator=gen, device=DEV)[:n * cols].to(torch.int32) \
        .reshape(n, cols).contiguous()
    kc, ks = _pool(gen, n_pages, H, d)
    vc, vs = _pool(gen, n_pages, H, d)
    grow = torch.exp(2 * torch.randn(T, 1, 1, generator=gen, device=DEV))
    fused = torch.randn(T, 2 * H + 1, d, generator=gen, device=DEV) * grow
    fused[T // 2, 0, 3] = 0.0
    fused = fused.to(DT[dtype])
    k, v = fused[:, :H], fused[:, H:2 * H]
    cu = np.concatenate([[0], np.cumsum(lens)])
    want = []
    for x, c, s in ((k, kc, ks), (v, vc, vs)):
        val, sc = ref.values(c), f64(s)
        ref.cache_write(f64(x), val, sc, cu, start, cut, table.cpu().numpy(), n_pages)
        want.append((val, sc))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    kda.cache_write(k, v, _i32(start), table, kc, ks, vc, vs, cu_seqlens=_i32(cu.tolist()),
                    lens=None if cut is None else _i32(cut), status=status)
    assert int(status) == 0
    keep = _written(start, lens if cut is None else cut, n_pages, table.cpu().numpy())
    for (val, sc), c, s in zip(want, (kc, vc), (ks, vs)):
        assert np.array_equal(f64(s), sc)
        got = ref.values(c)
        assert np.array_equal(got.transpose(0, 2, 1, 3)[keep], val.transpose(0, 2, 1, 3)[keep])
    # read the whole of every sequence back
    back = [max(s, 0) + m for s, m in zip(start, lens if cut is None else cut)]
    rcu = np.concatenate([[0], np.cumsum(back)])
    rstart = [0 if s >= 0 else -1 for s in start]
    k2, v2 = kda.cache_read(_i32(rstart), table, kc, ks, vc, vs, int(rcu[-1]),
                            cu_seqlens=_i32(rcu.tolist()), dtype=DT[dtype])
    for (val, sc), x in zip(want, (k2, v2)):
        for s in range(n):
            a, there = ref.gather(val, sc, table.cpu().numpy()[s], back[s], n_pages)
            if start[s] < 0:
                a = np.zeros_like(a)
            assert np.array_equal(f64(x[rcu[s]:rcu[s + 1]]), a)


def test_scale_at_its_bounds():
    """Largest values at and next to 448 * 2^k, tiny and huge ones, zeros, NaN and infinities."""
    tops = [448.0, float(np.nextafter(np.float32(448), np.float32(1e9))), 1.75 * 2.0 ** -120,
            3.0e38, 0.0, 1e-44, float("nan"), float("inf"), 7.0 * 2.0 ** 40]
    n = len(tops)
    x = torch.zeros(n, 1, 64, device=DEV)
    x[:, 0, 5] = torch.tensor(tops, device=DEV)
    x[:, 0, 9] = -0.25 * torch.tensor(tops, device=DEV)
    kc = torch.zeros(n, 1, 64, 64, dtype=torch.float8_e4m3fn, device=DEV)
    ks = torch.ones(n, 1, device=DEV)
    vc, vs = kc.clone(), ks.clone()
    table = torch.arange(n, dtype=torch.int32, device=DEV).reshape(n, 1)
    zero = torch.zeros(n, dtype=torch.int32, device=DEV)
    cu = torch.arange(n + 1, dtype=torch.int32, device=DEV)
    kda.cache_write(x, -x, zero, table, kc, ks, vc, vs, cu_seqlens=cu)
    val, sc = np.zeros((n, 1, 64, 64)), np.ones((n, 1))
    with np.errstate(invalid="ignore", over="ignore"):
        ref.cache_write(f64(x), val, sc, np.arange(n + 1), [0] * n, None, np.arange(n)[:, None], n)
    assert np.array_equal(f64(ks), sc) and np.array_equal(f64(vs), sc)
    got = ref.values(kc)[:, :, :1]
    assert np.array_equal(got, val[:, :, :1], equal_nan=True)
    assert np.array_equal(ref.values(vc)[:, :, :1], -val[:, :, :1], equal_nan=True)


def test_pages_absent_out_of_range_and_past_the_table():
    H, d, n_pages = 2, 64, 3
    kc = torch.full((n_pages, H, 64, d), 9, dtype=torch.uint8, device=DEV)
    ks = torch.ones(n_pages, H, device=DEV)
    vc, vs = kc.clone(), ks.clone()
    x = torch.randn(130, H, d, device=DEV)
    table = _i32([[-1, 7]])
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    kda.cache_write(x, x, _i32([0]), table, kc, ks, vc, vs, status=status)
    assert int(status) == kda.STATUS_BAD_PAGE
    assert (kc == 9).all() and (vs == 1).all()
    status.zero_()
    k, v = kda.cache_read(_i32([0]), table, kc, ks, vc, vs, 130, status=status)
    assert int(status) == kda.STATUS_BAD_PAGE and (k == 0).all() and (v == 0).all()
    status.zero_()
    cu = _i32([0, 40, 20])  # decreasing: the second sequence is malformed
    kda.cache_write(x, x, _i32([0, 0]), _i32([[0], [1]]), kc, ks, vc, vs, cu_seqlens=cu,
                    status=status)
    assert int(status) == kda.STATUS_BAD_OFFSETS and (kc[1:] == 9).all()


def test_cache_beyond_4_gib():
    """Pages on both sides of the 32-bit byte offset."""
    H, d = 8, 128
    n_pages = (1 << 32) // (H * 64 * d) + 40
    kc = torch.empty(n_pages, H, 64, d, dtype=torch.uint8, device=DEV)
    ks = torch.ones(n_pages, H, device=DEV)
    vc, vs = torch.empty_like(kc), torch.ones_like(ks)
    kc[:40] = 5
    x = torch.randn(100, H, d, device=DEV, dtype=torch.bfloat16)
    y = torch.randn(100, H, d, device=DEV, dtype=torch.bfloat16)
    high = _i32([[n_pages - 1, n_pages - 2]])
    kda.cache_write(x, y, _i32([0]), high, kc, ks, vc, vs)
    k1, v1 = kda.cache_read(_i32([0]), high, kc, ks, vc, vs, 100)
    q = torch.randn(1, 2 * H, d, device=DEV, dtype=torch.bfloat16)
    o1 = kda.cache_attention(q, _i32([99]), high, kc, ks, vc, vs, scale=d ** -0.5)
    assert (kc[:40] == 5).all()
    low = _i32([[1, 0]])
    kda.cache_write(x, y, _i32([0]), low, kc, ks, vc, vs)
    k2, v2 = kda.cache_read(_i32([0]), low, kc, ks, vc, vs, 100)
    o2 = kda.cache_attention(q, _i32([99]), low, kc, ks, vc, vs, scale=d ** -0.5)
    assert torch.equal(k1, k2) and torch.equal(v1, v2) and torch.equal(o1, o2)
