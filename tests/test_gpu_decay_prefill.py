"""kda_decay_prefill against the recurrence in 64 bits.

Tolerances, element by element, relative to the same sums with every term's absolute value (A for
outputs, B for states). bf16: the state and the weighted products q.k enter the outputs rounded to
bf16, each term by at most 2^-8 of itself: 2^-8 A; the fp32 sums of at most 2^9 terms in a chunk, or of
that many chunks, are off by 2^-15 A in the worst case, exponentials by a few 2^-22: 2^-14 A in all;
and the output's own rounding, 2^-8 of it. Over a whole tensor these roundings are independent, each
at most 2^-8 and 2^-8 / sqrt(3) in the root mean square, and the terms of random inputs add up like
the outputs: the two together stay below 2^-8 sqrt(2 / 3) of the outputs in the 2-norm, 2^-8 of them
with the rest. fp32: 2^-14 A covers the sums. States: parts of 24 bits and sums of at most 64 terms a
chunk and a few hundred chunks: 2^-15 B."""
import numpy as np
import pytest
import torch

import bounded_ref as ref
from kda_testutil import f64
from linear_attention_state_kda_gb300 import kda

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def make(lens, H, Hk, d, dtype, seed=0, const=False, init=True, rate=None, extra=0):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    T = sum(lens) + extra
    qkv = rnd(T, 2 * Hk + H, d).to(DT[dtype])
    if rate is None:
        rate = torch.exp2(-1.0 - 8.0 * torch.arange(H, device=DEV) / max(1, H - 1))
    g = -rate * (torch.ones(H, device=DEV) if const else
                 torch.nn.functional.softplus(rnd(T, H)))
    s0 = rnd(len(lens), H, d, d) if init else None
    cu = _i32(np.concatenate([[0], np.cumsum(lens)]).tolist())
    return qkv[:, :Hk], qkv[:, Hk:2 * Hk], qkv[:, 2 * Hk:], g, cu, s0


def check(q, k, v, g, cu, s0, scale, o, fin, dtype):
    T, H, d = v.shape
    init = np.zeros((cu.numel() - 1, H, d, d)) if s0 is None else f64(s0)
    gg = np.broadcast_to(f64(g), (T, H))
    want, st, a, b = ref.decay_prefill(f64(q), f64(k), f64(v), gg, cu.tolist(), init, scale)
    n = int(cu[-1])
    tol = 2.0 ** -14 * a
    if dtype == "bf16":
        tol = tol + 2.0 ** -8 * (a + np.abs(want))
        off = np.linalg.norm((f64(o) - want)[:n])
        assert off <= 2.0 ** -8 * np.linalg.norm(want[:n]), off / np.linalg.norm(want[:n])
    err = np.abs(f64(o) - want)[:n]
    assert (err <= tol[:n] + 1e-30).all(), float((err / (tol[:n] + 1e-30)).max())
    err = np.abs(f64(fin) - st)
    assert (err <= 2.0 ** -15 * b + 1e-30).all(), float((err / (2.0 ** -15 * b + 1e-30)).max())


@pytest.mark.parametrize("lens,H,Hk,d,dtype,const,init", [
    ([1], 1, 1, 128, "bf16", False, True), ([63], 2, 1, 128, "bf16", True, False),
    ([64], 3, 3, 128, "bf16", False, True), ([65], 2, 2, 64, "bf16", False, True),
    ([128], 1, 1, 64, "bf16", False, False), ([129, 127], 2, 2, 128, "bf16", True, True),
    ([0, 1, 0, 130, 5, 0], 4, 2, 128, "bf16", False, True),
    ([300, 2, 64, 63, 200], 6, 2, 64, "bf16", False, True),
    ([1500], 2, 2, 128, "bf16", False, True), ([700, 1, 1300, 0, 257], 3, 1, 128, "bf16", True, True),
    ([1100, 900], 2, 1, 64, "bf16", False, False),
    ([1], 1, 1, 64, "f32", False, True), ([31, 33, 0, 32], 4, 2, 64, "f32", False, True),
    ([129, 7], 3, 3, 128, "f32", True, False), ([1300, 1, 600], 2, 1, 128, "f32", False, True),
    ([777, 0, 600], 3, 3, 64, "f32", True, True)])
def test_parity(lens, H, Hk, d, dtype, const, init):
    x = make(lens, H, Hk, d, dtype, seed=sum(lens) + H + d, const=const, init=init)
    q, k, v, g, cu, s0 = x
    scale = d ** -0.5
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    o, fin = kda.decay_prefill(q, k, v, g, cu_seqlens=cu, init_state=s0, scale=scale, status=status)
    check(*x, scale, o, fin, dtype)
    assert int(status) == 0
    again, fin2 = kda.decay_prefill(q.contiguous(), k.contiguous(), v.contiguous(), g, cu_seqlens=cu,
                                    init_state=s0, scale=scale)
    assert torch.equal(o, again) and torch.equal(fin, fin2)


def test_one_sequence_without_offsets_and_without_final():
    q, k, v, g, cu, s0 = make([333], 2, 2, 128, "bf16")
    a, fin = kda.decay_prefill(q, k, v, g, cu_seqlens=cu, init_state=s0)
    b, none = kda.decay_prefill(q, k, v, g, init_state=s0, want_final=False)
    assert torch.equal(a, b) and none is None and fin.shape == s0.shape


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["strong", "drop", "reset", "none", "mixed"])
def test_decays(dtype, kind):
    """Any g <= 0: strong decay throughout, one drop between slow tokens, resets, no decay."""
    q, k, v, g, cu, s0 = make([400, 150], 2, 2, 128, dtype, seed=3)
    g = g.clone()
    if kind == "strong":
        g *= 400
    elif kind == "drop":
        g *= 0.01
        g[70] = -300.0
        g[431] = -1e30
    elif kind == "reset":
        g[::37] = -float("inf")
    elif kind == "none":
        g.zero_()
    else:
        g[torch.arange(550, device=DEV) % 5 == 0, 1] = -90.0
    o, fin = kda.decay_prefill(q, k, v, g, cu_seqlens=cu, init_state=s0, scale=0.1)
    check(q, k, v, g, cu, s0, 0.1, o, fin, dtype)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_rows_outside_the_sequences_are_left(dtype, d):
    """Offsets that begin after row 0 and end before the last row."""
    q, k, v, g, cu, s0 = make([90, 700], 2, 1, d, dtype, seed=5, extra=30)
    cu = cu + 11
    full = torch.full_like(v, 7.0).contiguous()
    for x in (q, k, v):  # NaN around the sequences does not reach them
        x[:11] = float("nan")
        x[801:] = float("nan")
    o, fin = kda.decay_prefill(q, k, v, g, cu_seqlens=cu, init_state=s0, scale=0.1, o=full)
    assert o is full and (o[:11] == 7).all() and (o[801:] == 7).all()
    sl = slice(11, 801)
    check(q[sl], k[sl], v[sl], g[sl], cu - 11, s0, 0.1, o[sl], fin, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nan_stays_in_its_sequence_and_after_its_chunk_begins(dtype):
    q, k, v, g, cu, s0 = make([200, 150, 300], 2, 2, 128, dtype, seed=6)
    want, fin0 = kda.decay_prefill(q, k, v, g, cu_seqlens=cu, init_state=s0)
    for x, bad in ((q, float("nan")), (k, float("inf")), (v, float("nan"))):
        y = [t.clone() for t in (q, k, v)]
        y[[q is x, k is x, v is x].index(True)][200 + 100, 0] = bad
        o, fin = kda.decay_prefill(*y, g, cu_seqlens=cu, init_state=s0)
        assert torch.equal(o[:264], want[:264]) and torch.equal(o[350:], want[350:])
        assert torch.equal(o[:, 1], want[:, 1])
        assert torch.equal(fin[[0, 2]], fin0[[0, 2]])
    g2 = g.clone()
    g2[300, 0] = float("nan")
    o, fin = kda.decay_prefill(q, k, v, g2, cu_seqlens=cu, init_state=s0)
    assert torch.equal(o[:264], want[:264]) and torch.isnan(o[301:350, 0]).all()
    assert torch.equal(o[350:], want[350:]) and torch.isnan(fin[1, 0]).all()


def test_large_values():
    """Entries near the ends of bf16's range: products stay in fp32's."""
    q, k, v, g, cu, s0 = make([130, 64], 2, 2, 128, "bf16", seed=7, init=False)
    q, k, v = (q.float() * 2.0 ** 40).bfloat16(), (k.float() * 2.0 ** -60).bfloat16(), \
        (v.float() * 2.0 ** 70).bfloat16()
    o, fin = kda.decay_prefill(q, k, v, g, cu_seqlens=cu, scale=2.0 ** -30)
    check(q, k, v, g, cu, s0, 2.0 ** -30, o, fin, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_offsets(dtype):
    q, k, v, g, cu, s0 = make([100, 100, 100], 2, 2, 64, dtype, seed=8)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    bad = _i32([0, 100, 700, 300])  # past the end, then decreasing
    o = torch.full_like(v, 3.0).contiguous()
    _, fin = kda.decay_prefill(q, k, v, g, cu_seqlens=bad, init_state=s0, o=o, status=status)
    want, fin0 = kda.decay_prefill(q[:100], k[:100], v[:100], g[:100], init_state=s0[:1])
    assert int(status) == kda.STATUS_BAD_OFFSETS
    assert torch.equal(o[:100], want) and (o[100:] == 3).all() and torch.equal(fin[0], fin0[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_split_over_two_calls(dtype):
    """A prompt in two calls, the second from the first one's exit states: as close to the
    recurrence as in one."""
    lens = [500, 130]
    q, k, v, g, cu, s0 = make(lens, 2, 1, 128, dtype, seed=9)
    cut = [200, 64]
    rows = [np.r_[0:200, 500:564], np.r_[200:500, 564:630]]
    o = torch.empty_like(v).contiguous()
    s = s0
    for r, n in zip(rows, (cut, [300, 66])):
        r = torch.from_numpy(r).to(DEV)
        part, s = kda.decay_prefill(q[r], k[r], v[r], g[r],
                                    cu_seqlens=_i32([0, n[0], n[0] + n[1]]), init_state=s, scale=0.1)
        o[r] = part
    check(q, k, v, g, cu, s0, 0.1, o, s, dtype)


def test_many_sequences_and_heads():
    rng = np.random.default_rng(1)
    lens = rng.integers(0, 40, 300).tolist()
    for dtype, H, Hk, d in (("bf16", 5, 5, 128), ("bf16", 4, 1, 64), ("f32", 2, 1, 64)):
        x = make(lens, H, Hk, d, dtype, seed=10)
        o, fin = kda.decay_prefill(*x[:4], cu_seqlens=x[4], init_state=x[5], scale=0.1)
        check(*x, 0.1, o, fin, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_graph_stream_and_workspace(dtype):
    """Captured and replayed on new inputs, with a caller's workspace that two graphs share, and on
    a stream other than the current one."""
    q, k, v, g, cu, s0 = make([900, 300], 2, 2, 128, dtype, seed=11)
    need = kda.decay_prefill_workspace(DT[dtype], 2, 1200, 2, 128)
    ws = torch.full((need + 64,), 0xff, dtype=torch.uint8, device=DEV)
    want = kda.decay_prefill(q, k, v, g, cu_seqlens=cu, init_state=s0, workspace=ws)
    q2 = (q.float() * 0.5 + k.float()).to(q.dtype)
    want2 = kda.decay_prefill(q2, k, v, g, cu_seqlens=cu, init_state=s0)
    qq, outs, graphs = q.clone(), [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(kda.decay_prefill(qq, k, v, g, cu_seqlens=cu, init_state=s0, workspace=ws))
        graphs.append(gr)
    for x, y in ((q, want), (q2, want2)):
        qq.copy_(x)
        for gr, (o, fin) in zip(graphs, outs):
            gr.replay()
            assert torch.equal(o, y[0]) and torch.equal(fin, y[1])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    o, fin = kda.decay_prefill(q, k, v, g, cu_seqlens=cu, init_state=s0, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, want[0]) and torch.equal(fin, want[1])


def test_long_prompt_many_segments():
    """A prompt that is cut into many segments, beside short ones, on sampled heads."""
    lens = [6000, 3, 1000]
    for dtype, d in (("bf16", 128), ("bf16", 64), ("f32", 64)):
        x = make(lens, 40, 20, d, dtype, seed=12)
        q, k, v, g, cu, s0 = x
        o, fin = kda.decay_prefill(q, k, v, g, cu_seqlens=cu, init_state=s0, scale=0.1)
        for h in (0, 17, 39):
            check(q[:, h // 2:h // 2 + 1], k[:, h // 2:h // 2 + 1], v[:, h:h + 1], g[:, h:h + 1], cu,
                  s0[:, h:h + 1], 0.1, o[:, h:h + 1], fin[:, h:h + 1], dtype)


@pytest.mark.parametrize("dtype,d,H,T", [("bf16", 128, 4, 12160 + 13), ("bf16", 64, 3, 20160),
                                         ("f32", 64, 2, 64 * 19 + 1)])
def test_segments_of_an_odd_number_of_chunks(dtype, d, H, T):
    """Segments of 5, 7 and (fp32) 2 chunks, several a block or one: the last one's end, too."""
    x = make([T], H, 1, d, dtype, seed=13)
    q, k, v, g, cu, s0 = x
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    o, fin = kda.decay_prefill(q, k, v, g, cu_seqlens=cu, init_state=s0, scale=0.1, status=status)
    assert int(status) == 0
    check(q, k, v[:, :1], g[:, :1], cu, s0[:, :1], 0.1, o[:, :1], fin[:, :1], dtype)
    check(q, k, v[:, -1:], g[:, -1:], cu, s0[:, -1:], 0.1, o[:, -1:], fin[:, -1:], dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_two_calls_at_once(dtype):
    """Two streams, a workspace each: the answers of one call after the other."""
    xs = [make([1500, 70], 3, 3, 128, dtype, seed=20 + i) for i in range(2)]
    want = [kda.decay_prefill(*x[:4], cu_seqlens=x[4], init_state=x[5]) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(3):
        got = []
        for x, s in zip(xs, streams):
            with torch.cuda.stream(s):
                got.append(kda.decay_prefill(*x[:4], cu_seqlens=x[4], init_state=x[5]))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
