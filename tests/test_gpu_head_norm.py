"""kda_head_norm_rope against the formula in 64 bits.

Tolerance: the sum of squares, the square root, the product and the rotation are some ten fp32
roundings of values no larger than the row's largest result, so 16 * 2^-24 of that; bf16 rounds
the result once more: half an ulp of 8 significant bits, 2^-8 of the value."""
import numpy as np
import pytest
import torch

import serving_ref as ref
from kda_testutil import f64
from linear_attention_state_kda_gb300 import kda

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _near(got, want, dtype):
    tol = 16 * 2.0 ** -24 * np.abs(want).max(-1, keepdims=True) + 1e-30
    if dtype == "bf16":
        tol = tol + 2.0 ** -8 * np.abs(want)
    assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) / tol).max())


def _table(n_pos, rot):
    ang = np.arange(n_pos)[:, None] * 10000.0 ** (-np.arange(rot // 2) * 2.0 / max(rot, 1))
    return torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1)).float().to(DEV)


@pytest.mark.parametrize("T,Hq,Hk,d,rot,l2,inter,dtype", [
    (1, 1, 1, 128, 128, False, False, "bf16"), (5, 32, 8, 128, 128, False, False, "bf16"),
    (33, 7, 3, 128, 64, False, True, "bf16"), (17, 9, 1, 64, 64, False, False, "bf16"),
    (9, 5, 2, 64, 16, True, False, "bf16"), (130, 6, 6, 128, 0, True, False, "bf16"),
    (3, 4, 4, 128, 48, False, False, "f32"), (21, 3, 2, 64, 32, False, True, "f32"),
    (2, 1, 1, 64, 64, False, False, "f32"), (40, 17, 0, 128, 96, False, True, "f32"),
    (6, 0, 5, 128, 32, False, False, "bf16")])
def test_parity(T, Hq, Hk, d, rot, l2, inter, dtype):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(T * 131 + d)
    qkv = (torch.randn(T, Hq + 2 * Hk + 1, d, generator=gen, device=DEV) * 3).to(DT[dtype])
    q = qkv[:, :Hq] if Hq else None
    k = qkv[:, Hq:Hq + Hk] if Hk else None
    before = qkv.clone()
    w = [1 + 0.5 * torch.randn(d, generator=gen, device=DEV) for _ in range(2)]
    if l2:
        w = [None, None]
    n_pos = 3 * T + 5
    tab = _table(n_pos, rot) if rot else None
    pos = torch.randint(0, n_pos, (T,), generator=gen, device=DEV, dtype=torch.int32)
    got = kda.head_norm_rope(q, k, w[0], w[1], eps=1e-5, l2=l2, cos_sin=tab, positions=pos,
                             interleaved=inter)
    for x, y, wt in zip((q, k), got, w):
        if x is None:
            assert y is None
            continue
        want = ref.head_norm(f64(x), None if wt is None else f64(wt), 1e-5, l2,
                             None if tab is None else f64(tab), pos.cpu().numpy(), inter)
        _near(f64(y), want, dtype)
    # in place on the fused rows gives the same bits and touches nothing else
    kda.head_norm_rope(q, k, w[0], w[1], eps=1e-5, l2=l2, cos_sin=tab, positions=pos,
                       interleaved=inter, q_out=q, k_out=k)
    for x, y in zip((q, k), got):
        assert x is None or torch.equal(x, y)
    assert torch.equal(qkv[:, Hq + Hk:], before[:, Hq + Hk:])


def test_default_positions_and_bad_position():
    x = torch.randn(4, 2, 64, device=DEV)
    tab = _table(4, 64)
    a, _ = kda.head_norm_rope(x, None, cos_sin=tab)
    b, _ = kda.head_norm_rope(x, None, cos_sin=tab,
                              positions=torch.arange(4, dtype=torch.int32, device=DEV))
    assert torch.equal(a, b)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    pos = torch.tensor([0, 4, -1, 3], dtype=torch.int32, device=DEV)
    c, _ = kda.head_norm_rope(x, None, cos_sin=tab, positions=pos, status=status)
    assert int(status) == kda.STATUS_BAD_POSITION
    plain, _ = kda.head_norm_rope(x, None)
    assert torch.equal(c[1:3], plain[1:3]) and torch.equal(c[3], a[3])


def test_non_finite_rows_stay_their_own():
    """A row with NaN or infinity, and an all-zero row, do not reach other rows."""
    x = torch.randn(6, 4, 128, device=DEV, dtype=torch.bfloat16)
    clean, _ = kda.head_norm_rope(x, None)
    y = x.clone()
    y[1, 2, 5] = float("nan")
    y[3, 0, 7] = float("inf")
    y[4, 1] = 0
    got, _ = kda.head_norm_rope(y, None, eps=1e-6)
    assert torch.isnan(got[1, 2]).all() and torch.isnan(got[3, 0, 7])
    assert (got[4, 1] == 0).all()
    same = torch.ones(6, 4, dtype=torch.bool, device=DEV)
    same[1, 2] = same[3, 0] = same[4, 1] = False
    assert torch.equal(got[same], clean[same])


def test_other_stream():
    x = torch.randn(64, 8, 128, device=DEV, dtype=torch.bfloat16)
    want, _ = kda.head_norm_rope(x, None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got, _ = kda.head_norm_rope(x, None, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
