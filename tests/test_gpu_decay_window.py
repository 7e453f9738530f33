"""kda_decay_window against the recurrence in 64 bits.

Tolerances, relative to the sums of absolute terms: fp32 arithmetic over at most 128 channels and 16
tokens, 2^-16 of them for outputs and 2^-18 for states (two roundings of 2^-24 and an exponential's
few 2^-23 per token), plus the rounding of bf16 outputs, 2^-8."""
import numpy as np
import pytest
import torch

import bounded_ref as ref
from kda_testutil import f64
from linear_attention_state_kda_gb300 import kda
from test_gpu_decay_prefill import DEV, _i32, make

pytestmark = pytest.mark.gpu


def _setup(B, W, H, Hk, d, dtype, const=False, seed=0):
    q, k, v, g, _, _ = make([B * W], H, Hk, d, dtype, seed=seed, const=const, init=False)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed + 1)
    n = B * (W + 1) + 3
    pool = torch.randn(n, H, d, d, generator=gen, device=DEV)
    slots = torch.randperm(n, generator=gen, device=DEV).to(torch.int32)
    return q, k, v, g, pool, slots[:B].contiguous(), \
        slots[B:B * (W + 1)].reshape(B, W).contiguous()


def _check(q, k, v, g, before, read, write, scale, o, after, dtype):
    B, W = write.shape
    H, d = v.shape[1:]
    want = before.copy()
    rep = lambda x: np.repeat(f64(x), H // x.shape[1], 1)  # noqa: E731
    q, k, v = rep(q), rep(k), rep(v)
    g = np.broadcast_to(f64(g), (B * W, H))
    for b in range(B):
        r = slice(b * W, (b + 1) * W)
        if not 0 <= read[b] < len(before):
            assert (o[r] == 0).all()
            continue
        x, st = ref.decay_steps(q[r], k[r], v[r], g[r], before[read[b]])
        xa, sa = ref.decay_steps(np.abs(q[r]), np.abs(k[r]), np.abs(v[r]), g[r],
                                 np.abs(before[read[b]]))
        tol = 2.0 ** -16 * xa * scale + (2.0 ** -8 * np.abs(x) * scale if dtype == "bf16" else 0)
        assert (np.abs(o[r] - x * scale) <= tol).all()
        for j in range(W):
            if 0 <= write[b, j] < len(before):
                assert (np.abs(after[write[b, j]] - st[j]) <= 2.0 ** -18 * sa[j]).all()
                want[write[b, j]] = after[write[b, j]]
    assert np.array_equal(after, want)  # nothing else was written


@pytest.mark.parametrize("B,W,H,Hk,d,dtype,const", [
    (1, 1, 1, 1, 128, "bf16", False), (3, 1, 4, 2, 128, "bf16", True), (2, 4, 3, 1, 64, "bf16", False),
    (5, 16, 2, 2, 128, "bf16", False), (4, 7, 2, 2, 128, "f32", True), (3, 1, 5, 5, 64, "f32", False)])
def test_parity(B, W, H, Hk, d, dtype, const):
    q, k, v, g, pool, read, write = _setup(B, W, H, Hk, d, dtype, const, seed=B + W + H)
    before = f64(pool)
    o = kda.decay_window(q, k, v, g, read, write, pool, scale=0.3)
    _check(q, k, v, g, before, read.tolist(), write.cpu().numpy(), 0.3, f64(o), f64(pool), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place_steps_equal_a_window_and_a_prompt(dtype):
    """Tokens one at a time in place, as one window, and as a prompt end in the same state."""
    B, W, H, d = 3, 6, 2, 128
    q, k, v, g, pool, read, write = _setup(B, W, H, H, d, dtype, seed=9)
    entry = pool[read.long()].clone()
    step = pool.clone()
    idx = torch.arange(B, device=DEV) * W
    for j in range(W):
        r = idx + j
        kda.decay_window(q[r], k[r], v[r], g[r].contiguous(), read, read[:, None].contiguous(), step)
    kda.decay_window(q, k, v, g, read, write, pool)
    last = pool[write[:, -1].long()]
    assert torch.equal(step[read.long()], last)
    _, fin = kda.decay_prefill(q, k, v, g, cu_seqlens=_i32([0, W, 2 * W, 3 * W]), init_state=entry)
    assert (fin - last).abs().max() <= 2.0 ** -15 * (last.abs().max() + 20)


def test_padding_and_bad_slots():
    q, k, v, g, pool, read, write = _setup(5, 3, 2, 1, 128, "bf16", seed=4)
    n = pool.shape[0]
    read[1], read[3] = -1, n
    write[0, 1], write[2, 2], write[4, 0] = -5, n + 7, -1
    before = f64(pool)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    o = kda.decay_window(q, k, v, g, read, write, pool, scale=0.3, status=status)
    assert int(status) == kda.STATUS_BAD_SLOT
    _check(q, k, v, g, before, read.tolist(), write.cpu().numpy(), 0.3, f64(o), f64(pool), "bf16")


def test_graph_and_stream():
    q, k, v, g, pool, read, _ = _setup(4, 1, 2, 2, 128, "bf16", seed=5)
    write = read[:, None].contiguous()
    a, b, c = pool.clone(), pool.clone(), pool.clone()
    want = [kda.decay_window(q, k, v, g, read, write, a) for _ in range(3)]
    kda.decay_window(q, k, v, g, read, write, b.clone())  # warm
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        o = kda.decay_window(q, k, v, g, read, write, b)
    for w in want:
        gr.replay()
        assert torch.equal(o, w)
    assert torch.equal(a, b)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for w in want:
        x = kda.decay_window(q, k, v, g, read, write, c, stream=side)
        side.synchronize()
        assert torch.equal(x, w)


def test_pool_beyond_32_bits():
    """Slots whose byte and element offsets pass 2^32."""
    H, d, n = 64, 128, 4200  # 4.4e9 elements
    pool = torch.zeros(n, H, d, d, device=DEV)
    q, k, v, g, _, _ = make([2], H, H, d, "bf16", seed=6, init=False)
    read, write = _i32([n - 1, 1]), _i32([[n - 2], [2]])
    pool[n - 1] = 0.25
    pool[1] = 0.5
    o = kda.decay_window(q, k, v, g, read, write, pool)
    for row, (r, s) in enumerate(((0.25, n - 2), (0.5, 2))):
        x, st = ref.decay_steps(f64(q)[row:row + 1], f64(k)[row:row + 1], f64(v)[row:row + 1],
                                f64(g)[row:row + 1], np.full((H, d, d), r))
        assert np.abs(f64(pool[s]) - st[0]).max() <= 2.0 ** -18 * np.abs(st[0]).max()
        assert np.abs(f64(o[row]) - x[0]).max() <= 2.0 ** -7 * np.abs(x[0]).max()
    assert (pool[3:n - 2:97] == 0).all()
