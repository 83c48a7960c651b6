"""The largest batches that the routing calls take."""
import pytest
import torch

from gpu_helpers import say
from test_gpu_route import _call, _check, _m

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [(1 << 25) + 5, 1 << 26])
def test_the_largest_batch(tokens):
    """As many tokens as a call may have, over the lane layout with the fewest
    rows a workgroup (64 groups): both sides of the place where one launch ends, and
    the last rows, are as in small calls."""
    m = _m()
    E, G, k = 64, 64, 2
    z = torch.zeros(tokens, E, dtype=torch.bfloat16, device="cuda")
    ends = [slice(0, 300), slice((1 << 25) - 300, min(tokens, (1 << 25) + 300)), slice(tokens - 300, tokens)]
    gen = torch.Generator(device="cuda").manual_seed(26)
    for e in ends:
        z[e] = torch.randn(e.stop - e.start, E, generator=gen, device="cuda").to(torch.bfloat16)
    kw = dict(kind="sigmoid", renorm=True, n_group=G, topk_group=8)
    say(f"[route] {tokens} tokens")
    ids, w = _call(z, k, **kw)
    g = torch.ones(tokens, k, device="cuda")
    g[:, 1] = -1
    d = torch.full_like(z, 3.0)
    m.moe_route_backward(z, ids, w, g, d, score=m.SCORE_SIGMOID, renorm=True)
    torch.cuda.synchronize()
    assert bool((ids >= 0).all()) and bool((w > 0).all()) and not bool((d == 3.0).any())
    for e in ends:
        few, fw = _check(z[e].contiguous(), k, **kw)
        assert torch.equal(ids[e], few) and torch.equal(w[e], fw)
        small = torch.empty(e.stop - e.start, E, dtype=torch.bfloat16, device="cuda")
        m.moe_route_backward(z[e].contiguous(), few, fw, g[e].contiguous(), small, score=m.SCORE_SIGMOID, renorm=True)
        assert torch.equal(d[e], small)
