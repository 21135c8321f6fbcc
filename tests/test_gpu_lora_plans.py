"""The adapters' ways of splitting their work: what the choice between them costs."""
import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def moe():
    from mxfp4_weight_streaming_amd import binding
    return binding


def _time(moe, M, r, K, N):
    """Microseconds of a call in a graph, an adapter a token."""
    g = torch.Generator(device="cuda").manual_seed(M)
    draw = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)  # noqa: E731
    lp = moe.lora(draw(M, r, K), draw(M, N, r))
    x, y, ids = draw(M, K), draw(M, N), torch.arange(M, dtype=torch.int32, device="cuda")
    out, ws = torch.empty(M, N, dtype=BF, device="cuda"), moe.lora_workspace(lp, M)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for _ in range(40):
            moe.moe_lora_add(lp, x, ids, y, out, ws)
    best = float("inf")
    for _ in range(6):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        graph.replay()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) * 25)
    return best


@pytest.mark.parametrize("K,M", [(8192, 24), (2560, 48)])
def test_a_few_tokens_more_cost_little(moe, K, M):
    """No step in time from a number of tokens that the XCDs share evenly to one that they do not."""
    even, odd = _time(moe, M, 16, K, 2560), _time(moe, M + 1 if K > 2560 else M + 3, 16, K, 2560)
    print(f"K={K}: {M} tokens {even:.2f} us, the odd number {odd:.2f} us", flush=True)
    assert odd < 1.3 * even
