"""kda_cache_attention at the ends of the ranges of its inputs: value pages of very small scales,
and queries of very large entries."""
import pytest
import torch

from linear_attention_state_kda_gb300 import kda
from test_gpu_cache_attention import DEV, _check, _i32, _make

pytestmark = pytest.mark.gpu

# one query row a unit, two and four warps a team, units of 256 rows
SHAPES = [(1, 4, 2, 128), (4, 16, 2, 64), (6, 8, 1, 128), (70, 4, 2, 128), (90, 6, 2, 64)]


@pytest.mark.parametrize("exps", [(-70,), (-80,), (-90,), (-100,), (-100, -95), (-79, -83, -75)])
@pytest.mark.parametrize("W,Hq,Hkv,d", SHAPES)
def test_small_value_scales(W, Hq, Hkv, d, exps):
    """Every value page has a scale of 2^-70 .. 2^-100. Tolerance as for other scales (2^-10 of the
    largest value + 2^-8 of the result): scores differ by at most 1.5 in units of log2 here, the
    largest weight of the smallest scale is at least 2^-13 as f16 whose steps are 2^-24, so a weight
    is off by at most 2^-25 of 2^-14.5 or more: 2^-10.5 of the mean value."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(W + d)
    start = [700, 90]
    q, table, pool = _make(gen, start, W, Hq, Hkv, d, "bf16")
    pick = torch.randint(0, len(exps), pool[3].shape, generator=gen, device=DEV)
    pool[3] = torch.exp2(torch.tensor(exps, device=DEV).double())[pick].float()
    pool[2] &= 0x7f  # (positive: a result near the largest value, not near zero)
    scale = 0.01 * (128 / d) ** 0.5
    got = kda.cache_attention(q, _i32(start), table, *pool, scale=scale)
    _check(q, start, None, table, pool, scale, "bf16", got)


@pytest.mark.parametrize("e", [-70, -80, -90])
def test_small_value_scales_fp32(e):
    """Weights in two f16 parts, off by at most 2^-25 of 2^-4.5 or more: within the 2^-12."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(-e)
    start = [700, 90]
    q, table, pool = _make(gen, start, 3, 6, 2, 128, "f32")
    pool[3].fill_(2.0 ** e)
    pool[2] &= 0x7f
    got = kda.cache_attention(q, _i32(start), table, *pool, scale=0.01)
    _check(q, start, None, table, pool, 0.01, "f32", got)


@pytest.mark.parametrize("W,Hq,Hkv,d,dtype", [s + ("bf16",) for s in SHAPES] +
                         [(3, 6, 2, 128, "f32"), (2, 3, 3, 64, "f32")])
def test_large_queries(W, Hq, Hkv, d, dtype):
    """Query entries from 1 to 2^126, with a scale that leaves scores of a usual size."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(W + d)
    start = [300, 40]
    q, table, pool = _make(gen, start, W, Hq, Hkv, d, dtype)
    q = q.clamp(-3.9, 3.9)
    for up in (2.0 ** 112, 2.0 ** 118, 2.0 ** 124):
        got = kda.cache_attention(q * up, _i32(start), table, *pool, scale=0.02 / up)
        _check(q, start, None, table, pool, 0.02, dtype, got)
