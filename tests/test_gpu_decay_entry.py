"""kda_decay_prefill of prompts in several segments: the entry states, which a kernel of the same call
writes while the next one has begun, are this call's and no other's."""
import pytest
import torch

from linear_attention_state_kda_gb300 import kda
from test_gpu_decay_prefill import DEV, DT, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_calls_through_one_workspace(dtype, d):
    """Calls on end with one workspace and other inputs each, and twice in a graph: the answers of
    calls with workspaces of their own."""
    lens, H = [2600, 700], 3
    xs = [make(lens, H, H, d, dtype, seed=50 + i) for i in range(4)]
    need = kda.decay_prefill_workspace(DT[dtype], len(lens), sum(lens), H, d)
    assert need > 0
    want = []
    for q, k, v, g, cu, s0 in xs:
        want.append(kda.decay_prefill(q, k, v, g, cu_seqlens=cu, init_state=s0))
        torch.cuda.synchronize()
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device=DEV)
    call = lambda x: kda.decay_prefill(*x[:4], cu_seqlens=x[4], init_state=x[5],  # noqa: E731
                                       workspace=ws)
    for _ in range(5):
        got = [call(x) for x in xs]
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [call(x) for x in xs]
    for _ in range(3):
        graph.replay()
    for a, b in zip(got, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
