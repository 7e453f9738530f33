"""Decay prompts and tokens, weighing and eviction together, as the example runs them."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import bounded_ref as bref
import serving_ref as ref
from kda_testutil import f64
from linear_attention_state_kda_gb300 import kda

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "bounded_context.py")


def _example():
    spec = importlib.util.spec_from_file_location("bounded_context", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    return example


def test_the_example_runs():
    """Prompts in one pass against single tokens: the same sums in another order, activations rounded
    to bf16 (2^-8) a few times a layer, and keys and values whose page scales may have grown in
    other steps (a code off by one step of the 8-bit format, 2^-4, in what attention averages): the
    logits stay within 2^-4 of the largest. Moving every cached token before each step changes no
    code, no scale and no order: the logits are equal. A bounded run keeps to its limit."""
    alone, moved, length, cuts = _example().check()
    assert alone < 2.0 ** -4, alone
    assert moved == 0.0
    # 150 tokens at the start: one cut, then one at every 36 more
    assert cuts == 1 and length[0] == 64 + 24
    assert length[1:] == [25, 64 + 24, 40 + 24]


def test_a_cut_of_a_generation_against_plain_forms():
    """Weights of a prompt and of tokens after it, what a cut keeps of them, and the next token's
    attention over what was kept, each against the plain implementation in 64 bits."""
    ex = _example()
    m = ex.Model("cuda")
    tokens, lens, follow = ex.draw([200, 90], 3, "cuda", seed=4)
    _, c, _ = ex.generate(m, tokens, lens, follow)
    table = c.tables[0].contiguous()
    length, budget = c.length.clone(), 70
    w0, kv0 = c.weights.clone(), [x.clone() for x in c.kv]
    # every weight given so far: LATEST prompt tokens and three more, HQ / HKV query heads each
    for b, n in enumerate(length.tolist()):
        flat = w0[table[b].long()].transpose(0, 1).reshape(ex.HKV, -1)[:, :n].double().sum(1)
        want = (min(ex.LATEST, int(lens[b])) + 3) * (ex.HQ // ex.HKV)
        # n sums of fp32 numbers of at most 20 additions each, statistics off by 2^-20 at most
        assert torch.allclose(flat, torch.full_like(flat, want), rtol=2.0 ** -16)
    sides = [(ref.values(kv0[0]).copy(), f64(kv0[1])), (ref.values(kv0[2]).copy(), f64(kv0[3]))]
    ww, new = f64(w0), c.tables[1].contiguous()
    cnt, kept = bref.evict(length.tolist(), table.cpu().numpy(), new.cpu().numpy(), sides, ww, budget,
                           ex.SINKS, ex.RECENT)
    got = c.evict(budget)
    assert np.array_equal(got.cpu().numpy(), kept) and c.length.tolist() == cnt.tolist()
    # the next query over the cut cache, against softmax over the kept old tokens
    gen = torch.Generator(device="cuda")
    gen.manual_seed(7)
    q = torch.randn(2, ex.HQ, ex.D, generator=gen, device="cuda").bfloat16()
    new = c.tables[0].contiguous()
    o = kda.cache_attention(q, c.length - 1, new, *c.kv, scale=ex.D ** -0.5)
    val = [ref.values(kv0[i]) * f64(kv0[i + 1])[:, :, None, None] for i in (0, 2)]
    for b in range(2):
        for h in range(ex.HQ):
            pos, hk = kept[b, h * ex.HKV // ex.HQ, :cnt[b]], h * ex.HKV // ex.HQ
            page = table[b].cpu().numpy()[pos // 64]
            kk, vv = (x[page, hk, pos % 64] for x in val)
            s = kk @ f64(q[b, h]) * ex.D ** -0.5
            p = np.exp(s - s.max())
            want = p @ vv / p.sum()
            # bf16 weights and outputs (2^-8 each), codes moved to a larger scale rounded only below
            # the format's normal range
            err = np.abs(f64(o[b, h]) - want).max()
            assert err <= 2.0 ** -6 * np.abs(vv).max(), err
