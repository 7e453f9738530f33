"""kda_cache_attention against the softmax in 64 bits over the values that the codes stand for.

Tolerances. Scores are fp32 sums of at most 128 products of a query known to 22 bits (fp32) or
exactly (bf16) with an exact key: |ds| <= 128 * 2^-24 * sum|q k| scale, below 2^-14 for the
scores here (sum|q k| scale < 8), and the exponential and the sums add a few 2^-22. A weight that
is off by a factor 1 + e moves the result by at most 2 e max|v|: 2^-12 max|v| for fp32 inputs,
whose probabilities carry 22 bits. bf16 inputs: probabilities rounded to 11 significant bits (half
an ulp is 2^-11, so 2^-10 max|v|) and the result once to 8 (2^-8 of it)."""
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


def _make(gen, start, W, Hq, Hkv, d, dtype, spare=3):
    B = len(start)
    cols = max(1, max((max(s, 0) + W + 63) // 64 for s in start))
    n_pages = B * cols + spare
    table = torch.randperm(n_pages, generator=gen, device=DEV)[:B * cols].to(torch.int32) \
        .reshape(B, cols).contiguous()
    pool = []
    for _ in range(2):
        c = torch.randint(0, 256, (n_pages, Hkv, 64, d), generator=gen, device=DEV).to(torch.uint8)
        c = (c & 0x80) | (c & 0x7f) % 0x60  # |values| <= 30
        s = torch.exp2(torch.randint(-6, -2, (n_pages, Hkv), generator=gen, device=DEV).double())
        pool += [c.to(torch.uint8).contiguous(), s.float()]
    q = torch.randn(B * W, Hq, d, generator=gen, device=DEV).to(DT[dtype])
    return q, table, pool


def _check(q, start, lens, table, pool, scale, dtype, got):
    B = len(start)
    kv, vv = ref.values(pool[0]), ref.values(pool[2])
    want = ref.attention(f64(q), start, lens, table.cpu().numpy(), kv, f64(pool[1]), vv,
                         f64(pool[3]), scale, B)
    top = np.abs(vv * f64(pool[3])[:, :, None, None])
    top = np.nanmax(top)
    tol = 2.0 ** -12 * top if dtype == "f32" else 2.0 ** -10 * top + 2.0 ** -8 * np.abs(want)
    err = np.abs(f64(got) - want)
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("start,W,Hq,Hkv,d,dtype", [
    ([0], 1, 1, 1, 128, "bf16"), ([0, 1, 62, 63, 64, 65], 1, 8, 2, 128, "bf16"),
    ([127, 700, 5], 1, 32, 8, 128, "bf16"), ([1000, 3, 129, 64], 4, 16, 2, 128, "bf16"),
    ([90, 31], 16, 8, 8, 128, "bf16"), ([333, 60], 3, 48, 3, 128, "bf16"),
    ([250], 16, 32, 2, 128, "bf16"), ([2000, 15], 1, 16, 1, 64, "bf16"),
    ([70, 400, 0], 5, 15, 3, 64, "bf16"), ([63, 64, 1], 2, 5, 5, 64, "bf16"),
    ([129, 40], 1, 12, 4, 128, "f32"), ([500, 7], 3, 15, 3, 64, "f32"),
    ([300], 7, 16, 1, 128, "f32"), ([0, 63], 16, 20, 1, 64, "f32"), ([5000], 1, 4, 2, 128, "f32")])
def test_parity(start, W, Hq, Hkv, d, dtype):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(sum(start) + 17 * W + d)
    q, table, pool = _make(gen, start, W, Hq, Hkv, d, dtype)
    scale = 0.3 * d ** -0.5
    got = kda.cache_attention(q, _i32(start), table, *pool, scale=scale)
    _check(q, start, None, table, pool, scale, dtype, got)
    again = kda.cache_attention(q.reshape(len(start), W, Hq, d), _i32(start), table, *pool,
                                scale=scale)
    assert torch.equal(again.reshape(q.shape), got)  # the same bits every time


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_rows_of_ragged_length(dtype):
    """Enough rows and heads that work is split unevenly over the SMs."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(77)
    start = [0, 1, 2, 3000, 5, 64, 700, 100, 1, 0, 2500, 63, 64, 65, 127, 128] * 3 + [4000]
    q, table, pool = _make(gen, start, 2, 12, 6, 64, dtype)
    got = kda.cache_attention(q, _i32(start), table, *pool, scale=0.04)
    _check(q, start, None, table, pool, 0.04, dtype, got)


@pytest.mark.parametrize("dtype,d,W,G", [("bf16", 128, 4, 4), ("f32", 64, 4, 3),
                                         ("bf16", 64, 16, 4), ("f32", 128, 16, 2)])
def test_masked_rows_absent_pages_and_stale_codes(dtype, d, W, G):
    """Padding rows, ragged windows, absent pages, ids past the pool, and NaN codes wherever no
    query may look: rows past the context, other pages, and later tokens of the window."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(5)
    start, lens = [200, -1, 70, 100, 64, 40], [W, W, 2, 0, W, W]
    q, table, pool = _make(gen, start, W, 2 * G, 2, d, dtype)
    host = table.cpu().numpy()
    table[0, 1] = -1                      # a hole in the context
    table[4] = _i32([-1] * table.shape[1])  # nothing at all
    table[5, 0] = 10 ** 6                 # past the pool
    used = {int(p) for b in (0, 2) for p in host[b]}
    for i in (0, 2):
        for page in range(pool[i].shape[0]):
            if page not in used:
                pool[i][page] = 0x7f
        for b in (0, 2):                  # past the last token that row b has
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
    assert (got[2 * W + 2:3 * W] == 0).all()
    _check(q, start, lens, table, pool, 0.05, dtype, got)
    if W < 4:
        return
    # NaN in the window's third token: the first two tokens of the window do not see it
    at = start[0] + 2
    for i, nan in ((0, 0x7f), (2, 0xff)):
        keep = pool[i].clone()
        pool[i][host[0][at // 64], 0, at % 64, 7] = nan
        one = kda.cache_attention(q, _i32(start), table, *pool, scale=0.05, lens=_i32(lens))
        assert torch.equal(one[:2], got[:2]) and torch.equal(one[W:], got[W:])
        assert torch.equal(one[:W, G:], got[:W, G:])  # the other head's cache is clean
        bad = torch.isnan(one[2:W, :G].float())
        if i == 0:
            assert bad.all()
        else:
            assert bad[..., 7].all() and int(bad.sum()) == bad[..., 7].numel()
        pool[i].copy_(keep)


def test_large_scores_and_positions_past_the_table():
    """Scores of several hundreds: the running maximum keeps the exponentials in range. A start
    past the page table sees the table's pages only and says so."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(9)
    start = [600, 130]
    q, table, pool = _make(gen, start, 1, 4, 2, 128, "f32")
    got = kda.cache_attention(q, _i32(start), table, *pool, scale=3.0)
    kv = ref.values(pool[0])
    want = ref.attention(f64(q), start, None, table.cpu().numpy(), kv, f64(pool[1]),
                         ref.values(pool[2]), f64(pool[3]), 3.0, 2)
    # ds grows with the score: sum|q k| scale < 1500 here, so |ds| < 128 * 2^-24 * 1500
    assert np.abs(f64(got) - want).max() < 2 * 128 * 2.0 ** -24 * 1500 * np.abs(want).max() * 2
    cols = table.shape[1]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    a = kda.cache_attention(q, _i32([cols * 64 + 5] * 2), table, *pool, scale=0.1, status=status)
    assert int(status) == kda.STATUS_BAD_PAGE
    status.zero_()
    b = kda.cache_attention(q, _i32([cols * 64 - 1] * 2), table, *pool, scale=0.1, status=status)
    assert int(status) == 0 and torch.equal(a, b)


def test_own_workspace_and_other_stream():
    gen = torch.Generator(device=DEV)
    gen.manual_seed(3)
    start = [900, 17]
    q, table, pool = _make(gen, start, 2, 8, 2, 128, "bf16")
    want = kda.cache_attention(q, _i32(start), table, *pool, scale=0.05)
    need = kda.cache_attention_workspace(2, 2, 8, 2, 128)
    ws = torch.full((need + 512,), 0xff, dtype=torch.uint8, device=DEV)
    st = _i32(start)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    o = torch.empty_like(q)
    kda.cache_attention(q, st, table, *pool, scale=0.05, o=o, workspace=ws, stream=s)
    s.synchronize()
    assert torch.equal(o, want)
    assert (ws[need:] == 0xff).all()


def test_graph_replay():
    """Captured in a CUDA graph: lengths are read on the device, so a replay follows them."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(4)
    start = [900, 17, 300]
    q, table, pool = _make(gen, start, 1, 8, 2, 128, "bf16")
    st = _i32(start)
    o = torch.empty_like(q)
    ws = torch.empty(max(1, kda.cache_attention_workspace(3, 1, 8, 2, 128)), dtype=torch.uint8,
                     device=DEV)
    kda.cache_attention(q, st, table, *pool, scale=0.05, o=o, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kda.cache_attention(q, st, table, *pool, scale=0.05, o=o, workspace=ws)
    for new in ([5, 600, 0], [900, 17, 300]):
        st.copy_(_i32(new))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, kda.cache_attention(q, _i32(new), table, *pool, scale=0.05))
