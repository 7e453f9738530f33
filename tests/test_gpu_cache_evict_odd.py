"""kda_cache_evict where a CTA has an odd number of pages: its last tile of 128 keys is half empty."""
import pytest

from test_gpu_cache_evict import _run, _setup, pytestmark  # noqa: F401


@pytest.mark.parametrize("length,Hkv,d,budget,sinks,recent", [
    ([64], 2, 64, 33, 1, 2), ([60, 1, 64, 30], 3, 128, 40, 4, 8), ([190, 64, 129], 2, 64, 64, 0, 7),
    # two and four CTAs of 67 pages
    ([8500, 4288, 4289], 1, 64, 1000, 4, 64), ([17100], 2, 64, 4200, 4, 64)])
def test_parity(length, Hkv, d, budget, sinks, recent):
    x = _setup(length, Hkv, d, budget, seed=3 * sum(length) + budget)
    pages = x[0].shape[1]
    ctas = 1
    while ctas < 8 and pages * 64 > ctas * 8192:
        ctas *= 2
    assert (pages + ctas - 1) // ctas % 2 == 1
    assert _run(length, *x, budget, sinks, recent)[0] == 0
