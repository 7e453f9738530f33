"""kda_decay_prefill in bf16 is as exact as fp32 arithmetic with one rounding at the end.

Tolerance, element by element, with A the output's sum with every term's absolute value. The output's
own rounding is off by at most 2^-8 of it. The state and the weighted products q.k, which are no inputs,
enter their products in two bf16 parts: the first is cut after 8 bits (a rest below 2^-7), the second
rounded (2^-8 of that): 2^-15 of a term, and the two cover different terms. States are known to 2^-15
(as the tests of states hold them to), which scales the terms that they enter; the fp32 sums of at
most 2^9 terms lose at most 2^-15 A, the exponentials a few 2^-22. In all below 2^-13 A + 2^-8 |o|.
A single bf16 rounding of either operand is off by up to 2^-8 of a term: where an output's terms
cancel, that is far more than the output's own rounding."""
import numpy as np
import pytest
import torch

import bounded_ref as ref
from kda_testutil import f64
from linear_attention_state_kda_gb300 import kda
from test_gpu_decay_prefill import make

pytestmark = pytest.mark.gpu


def check(q, k, v, g, cu, s0, scale, o):
    T, H, d = v.shape
    init = np.zeros((cu.numel() - 1, H, d, d)) if s0 is None else f64(s0)
    want, _, a, _ = ref.decay_prefill(f64(q), f64(k), f64(v), np.broadcast_to(f64(g), (T, H)),
                                      cu.tolist(), init, scale)
    tol = 2.0 ** -13 * a + 2.0 ** -8 * np.abs(want) + 1e-30
    err = np.abs(f64(o) - want)
    assert (err <= tol).all(), (float((err / tol).max()), float((err > tol).mean()))


@pytest.mark.parametrize("lens,H,Hk,d,const,init", [
    ([64], 2, 2, 128, False, True), ([65, 1], 2, 1, 64, True, True),
    ([77], 4, 4, 64, False, True), ([200, 0, 63, 130], 4, 2, 128, True, False),
    ([1500], 2, 2, 128, False, True), ([1100, 900], 2, 1, 64, False, False)])
def test_one_rounding(lens, H, Hk, d, const, init):
    x = make(lens, H, Hk, d, "bf16", seed=31 + d, const=const, init=init)
    q, k, v, g, cu, s0 = x
    o, _ = kda.decay_prefill(q, k, v, g, cu_seqlens=cu, init_state=s0, scale=d ** -0.5)
    check(*x, d ** -0.5, o)


@pytest.mark.parametrize("what", ["state", "tokens"])
@pytest.mark.parametrize("d", [64, 128])
def test_terms_that_cancel(what, d):
    """Either operand alone: a state that outweighs the tokens, and no state and hardly any decay."""
    q, k, v, g, cu, s0 = make([150], 3, 3, d, "bf16", seed=33, init=what == "state")
    if what == "state":
        s0 = s0 * 1000
    else:
        g = g * 1e-3
    o, _ = kda.decay_prefill(q, k, v, g, cu_seqlens=cu, init_state=s0, scale=0.1)
    check(q, k, v, g, cu, s0, 0.1, o)


@pytest.mark.parametrize("d", [64, 128])
def test_largest_entries(d):
    """States and weighted products next to the end of bf16's range: no part overflows."""
    q, k, v, g, cu, s0 = make([130], 2, 2, d, "bf16", seed=34)
    # (the largest entry of these is past the largest bf16 by more than half a step)
    s0 = s0 * (torch.arange(d, device=s0.device) % 7 == 0)[:, None]
    s0 = s0 / s0.abs().amax() * 3.4e38
    assert torch.isinf(s0.bfloat16()).any() and torch.isfinite(s0).all()
    q = (q.float() * 2.0 ** -40).bfloat16()
    g = g.clone()
    g[:, :] = -0.7
    o, fin = kda.decay_prefill(q, k, v, g, cu_seqlens=cu, init_state=s0, scale=2.0 ** -20)
    assert torch.isfinite(o).all() and torch.isfinite(fin).all()
    check(q, k, v, g, cu, s0, 2.0 ** -20, o)
