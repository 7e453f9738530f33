"""Scratch bytes of kda_cache_weigh: they do not grow with the window without end."""
import pytest
import torch


@pytest.mark.parametrize("dtype,d", [(torch.float32, 128), (torch.float32, 64), (torch.bfloat16, 64),
                                     (torch.bfloat16, 128)])
def test_bounded(dtype, d):
    from linear_attention_state_kda_gb300 import build as libbuild
    libbuild.build()
    from linear_attention_state_kda_gb300 import kda
    for batch, Hq, Hkv in ((1, 64, 8), (1, 8, 8), (3, 32, 2), (31, 16, 1)):
        top = 65536 if batch * 65536 * Hq <= 1 << 30 else (1 << 30) // (batch * Hq)
        for window in (1, 7, 64, 700, 4096, top):
            need = kda.cache_weigh_workspace(dtype, batch, window, Hq, Hkv, d, 4096)
            # queries of the window, where they are more, as their values
            size = 4 if dtype == torch.float32 else 2
            assert 0 < need <= max(8 << 20, batch * window * Hq * d * size), (window, need)
