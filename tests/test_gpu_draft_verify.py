"""kda_draft_verify against the definition: whole numbers, equal."""
import numpy as np
import pytest
import torch

import serving_ref as ref
from linear_attention_state_kda_gb300 import kda

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _make(seed, B, W, V, dtype, flat=False):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    logits = torch.randn(B, W + 1, V, generator=gen, device=DEV) * (0.01 if flat else 3.0)
    target = torch.softmax(logits, -1).to(DT[dtype])
    near = logits[:, :W] + 0.5 * torch.randn(B, W, V, generator=gen, device=DEV)
    draft = torch.softmax(near, -1).to(DT[dtype])
    toks = torch.multinomial(draft.float().reshape(B * W, V) + 1e-20, 1, generator=gen) \
        .to(torch.int32).reshape(B, W) if W else torch.empty(B, 0, dtype=torch.int32, device=DEV)
    ua = torch.rand(B, W, generator=gen, device=DEV)
    us = torch.rand(B, generator=gen, device=DEV)
    slots = torch.randperm(10 * B * (W + 1), generator=gen, device=DEV)[:B * (W + 1)] \
        .to(torch.int32).reshape(B, W + 1)
    return target, draft, toks.contiguous(), ua, us, slots


def _host(t):
    return None if t is None else t.float().cpu().numpy()


def _check(target, draft, toks, ua, us, slots, lens=None, status=None):
    n, out, resume = kda.draft_verify(target, toks, ua, us, draft_probs=draft, write_slots=slots,
                                      lens=lens, status=status)
    want = ref.verify(_host(target), _host(draft), toks.cpu().numpy(),
                      None if lens is None else lens.cpu().numpy(), _host(ua), _host(us),
                      slots.cpu().numpy())
    for got, w in zip((n, out, resume), want):
        assert np.array_equal(got.cpu().numpy(), w), (got.cpu().numpy(), w)
    return n


@pytest.mark.parametrize("B,W,V,dtype", [
    (1, 0, 1, "f32"), (1, 1, 1, "f32"), (3, 1, 2, "bf16"), (5, 3, 37, "f32"),
    (9, 16, 1000, "bf16"), (33, 4, 4097, "f32"), (2, 2, 50001, "f32"), (1, 3, 131072, "f32"),
    (4, 5, 32003, "bf16"), (2, 1, 270001, "f32"), (300, 2, 515, "f32")])
@pytest.mark.parametrize("onehot", [False, True])
def test_parity(B, W, V, dtype, onehot):
    target, draft, toks, ua, us, slots = _make(B * 31 + V, B, W, V, dtype)
    _check(target, None if onehot else draft, toks, ua, us, slots)


def test_flat_distribution_and_ends_of_the_random_numbers():
    """u at 0 and just below 1 sample the first and the last token with weight."""
    target, draft, toks, ua, us, slots = _make(3, 6, 2, 20011, "f32", flat=True)
    us[:3] = torch.tensor([0.0, 1.0 - 2.0 ** -24, 0.5], device=DEV)
    ua[0], ua[1] = 0.0, 1.0 - 2.0 ** -24
    target[0, 2, :7] = 0.0
    _check(target, draft, toks, ua, us, slots)


def test_every_count_is_reached():
    target, draft, toks, ua, us, slots = _make(8, 64, 3, 100, "f32")
    n = _check(target, draft, toks, ua, us, slots)
    assert set(n.tolist()) == {0, 1, 2, 3}


def test_ragged_rows_padding_and_bad_tokens():
    target, draft, toks, ua, us, slots = _make(11, 6, 4, 999, "f32")
    lens = torch.tensor([4, 0, 2, -1, 9, 4], dtype=torch.int32, device=DEV)
    toks[0, 1], toks[2, 0] = -3, 999
    ua[0, 0] = 0.0
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    _check(target, draft, toks, ua, us, slots, lens=lens, status=status)
    assert int(status) == kda.STATUS_BAD_TOKEN


def test_no_weight_left():
    """p <= q everywhere: p is sampled instead; p without weight: no token. NaN has no weight."""
    target, draft, toks, ua, us, slots = _make(12, 4, 1, 777, "f32")
    ua[:] = 1.0 - 2.0 ** -24
    draft[0] = target[0, :1]
    draft[0, 0, toks[0, 0]] += 0.5
    target[1, 0] = 0.0
    target[2, 0] = float("nan")
    target[3, 0, ::2] = float("nan")
    draft[3, 0, 1::4] = float("nan")
    draft[3, 0, toks[3, 0]] = 1.0
    _check(target, draft, toks, ua, us, slots)


def test_rows_with_a_stride():
    """Rows of padded buffers, at odd offsets."""
    B, W, V = 3, 2, 1001
    target, draft, toks, ua, us, slots = _make(13, B, W, V, "f32")
    wide_t = torch.full((B, W + 1, V + 7), 0.9, device=DEV)
    wide_d = torch.full((B, W, V + 3), 0.9, device=DEV)
    wide_t[..., 1:V + 1], wide_d[..., 2:V + 2] = target, draft
    a = kda.draft_verify(target, toks, ua, us, draft_probs=draft, write_slots=slots)
    b = kda.draft_verify(wide_t[..., 1:V + 1], toks, ua, us, draft_probs=wide_d[..., 2:V + 2],
                         write_slots=slots)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_samples_follow_the_target():
    """Drafts from q verified against p give tokens distributed as p, whatever q is. With n
    independent rows the count of a token of probability p has deviation sqrt(n p (1-p)); six of
    them bound all 16 counts."""
    n, V = 65536, 16
    gen = torch.Generator(device=DEV)
    gen.manual_seed(21)
    p = torch.softmax(torch.randn(V, generator=gen, device=DEV), 0)
    q = torch.softmax(torch.randn(V, generator=gen, device=DEV), 0)
    toks = torch.multinomial(q, n, replacement=True, generator=gen).to(torch.int32).reshape(n, 1)
    ua = torch.rand(n, 1, generator=gen, device=DEV)
    us = torch.rand(n, generator=gen, device=DEV)
    _, out, _ = kda.draft_verify(p.expand(n, 2, V).contiguous(), toks, ua, us,
                                 draft_probs=q.expand(n, 1, V).contiguous())
    count = torch.bincount(out[:, 0].long(), minlength=V).double()
    pd = p.double()
    assert ((count - n * pd).abs() < 6 * (n * pd * (1 - pd)).sqrt()).all()
