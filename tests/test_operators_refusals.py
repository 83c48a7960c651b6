"""More refusals of the operators' binding, without a GPU: what a tensor's
shape, type, layout or place shows to be wrong is an error before any call."""
import os

import pytest
import torch

LIB = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_expert_tile_amd", "libmoe.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libmoe.so not built")


def _m():
    import moe_expert_tile_amd as m
    return m


def _scale_args(m, T=6, k=2, d=256):
    s = m.Shape(1, 0, 4, k, d, 128, 32, [T], T * k)
    plan = torch.zeros(m.moe_query_sizes(s)["plan_bytes"] // 4, dtype=torch.int32)
    bf = torch.bfloat16
    return s, dict(plan_ws=plan, recv_self=torch.zeros(T * k, d, dtype=bf), topk_w=torch.zeros(T, k),
                   d_out=torch.zeros(T, d, dtype=bf), d_recv=torch.zeros(T * k, d, dtype=bf),
                   d_topk_w=torch.zeros(T, k))


@pytest.mark.parametrize("name,bad", [
    ("d_out", lambda t: t[:1].expand(6, 256)),           # the gradient of a sum
    ("d_out", lambda t: t.t().contiguous().t()), ("d_out", lambda t: t.float()), ("d_out", lambda t: t.half()),
    ("d_out", lambda t: t[:5]), ("d_out", lambda t: t[:, :128].contiguous()), ("d_out", lambda t: t.view(-1)),
    ("recv_self", lambda t: t[:11]), ("recv_self", lambda t: t[:, ::2]), ("recv_self", lambda t: t.float()),
    ("topk_w", lambda t: t.double()), ("topk_w", lambda t: t.bfloat16()), ("topk_w", lambda t: t.t().contiguous().t()),
    ("topk_w", lambda t: t[:5]), ("topk_w", lambda t: t[:, :1].contiguous()),
    ("d_recv", lambda t: t[:11]), ("d_recv", lambda t: t.float()), ("d_recv", lambda t: t.view(6, 512)),
    ("d_recv", lambda t: t[:1].expand(12, 256)),
    ("d_topk_w", lambda t: t.bfloat16()), ("d_topk_w", lambda t: t[:5]), ("d_topk_w", lambda t: t[:1].expand(6, 2)),
    ("plan_ws", lambda t: t[::2]),
])
def test_bad_scale_backward_tensors_are_rejected(name, bad):
    m = _m()
    s, a = _scale_args(m)
    a[name] = bad(a[name])
    with pytest.raises(m.MoEError, match=name) as ei:
        m.moe_scale_backward(s, **a)
    assert ei.value.status == m.MOE_EINVAL


def test_scale_backward_on_the_cpu_is_rejected():
    """Sound tensors but for their place; more rows than needed are sound."""
    m = _m()
    s, a = _scale_args(m)
    a["d_out"] = torch.zeros(7, 256, dtype=torch.bfloat16)
    a["d_recv"] = torch.zeros(20, 256, dtype=torch.int16)
    with pytest.raises(m.MoEError, match="not on a GPU"):
        m.moe_scale_backward(s, **a)
    bad = m.Shape(1, 3, 4, 2, 256, 128, 32, [6], 12)
    with pytest.raises(m.MoEError):
        m.moe_scale_backward(bad, **a)


def test_empty_gradients_of_the_scale_step_are_no_refusal():
    """A rank without tokens: either gradient, asked for alone, has no address; with tokens a call for neither is refused."""
    m = _m()
    some = 1 << 20   # an address, never read
    for tokens in (0, 6):
        s, a = _scale_args(m, T=tokens)
        rc = m._lib.moe_scale_backward(s.ptr, some, None, some, some, None, None, 0)
        assert (rc == m.MOE_EINVAL) == (tokens > 0) and rc in (m.MOE_OK, m.MOE_EINVAL, m.MOE_EHIP, m.MOE_EUNSUPPORTED)
        a["d_recv"] = a["d_topk_w"] = None
        with pytest.raises(m.MoEError, match="neither d_recv nor d_topk_w is given") as ei:
            m.moe_scale_backward(s, **a)
        assert ei.value.status == m.MOE_EINVAL


def test_an_empty_gradient_of_the_product_is_no_refusal():
    """Without rows dx, asked for alone, has no address; with rows a call for no gradient is refused."""
    import ctypes
    m = _m()
    some = 1 << 20   # an address, never read

    def call(rows, d_out):
        d = m.moe_linear_desc(rows, 32, 64, 0, 0, m.ACT_NONE, 0)
        return m._lib.moe_linear_backward(ctypes.byref(d), None, some, None, d_out, None, None, None, some, 0)

    assert call(0, None) in (m.MOE_OK, m.MOE_EHIP, m.MOE_EUNSUPPORTED)   # no launch; without a GPU no device
    assert call(4, some) == m.MOE_EINVAL
    x, w, g = (torch.zeros(s, dtype=torch.bfloat16) for s in ((0, 64), (32, 64), (0, 32)))
    with pytest.raises(m.MoEError, match="none of dx, dw and dbias is given") as ei:
        m.moe_linear_backward(x, w, g)
    assert ei.value.status == m.MOE_EINVAL


@pytest.mark.parametrize("stream", [None, 0, 1 << 20])
def test_tensors_on_the_cpu_are_rejected_whatever_the_stream(stream):
    m = _m()
    bf = torch.bfloat16
    x, w, out = torch.zeros(128, 8192, dtype=bf), torch.zeros(64, 8192, dtype=bf), torch.zeros(128, 64, dtype=bf)
    z, ids, wt = torch.zeros(4, 16), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    for call in (lambda: m.moe_linear(x, w, out, stream=stream),        # (a size that needs a workspace)
                 lambda: m.moe_linear_backward(x, w, out, dx=torch.zeros_like(x), stream=stream),
                 lambda: m.moe_route(z, ids, wt, stream=stream),
                 lambda: m.moe_route_backward(z, ids, wt, wt, torch.zeros_like(z), stream=stream)):
        with pytest.raises(m.MoEError, match="not on a GPU") as ei:
            call()
        assert ei.value.status == m.MOE_EINVAL


@pytest.mark.gpu
def test_a_stream_of_another_gpu_is_rejected():
    import types
    m = _m()
    bf = torch.bfloat16
    other = types.SimpleNamespace(cuda_stream=torch.cuda.current_stream().cuda_stream, device_index=1)
    s, a = _scale_args(m)
    a = {k: v.cuda() for k, v in a.items()}
    x, w, out = (torch.zeros(*n, dtype=bf, device="cuda") for n in ((128, 8192), (64, 8192), (128, 64)))
    z, wt = torch.zeros(4, 16, device="cuda"), torch.zeros(4, 2, device="cuda")
    ids = torch.full((4, 2), 3, dtype=torch.int32, device="cuda")
    for call in (lambda: m.moe_linear(x, w, out, stream=other),
                 lambda: m.moe_linear_backward(x, w, out, dx=torch.zeros_like(x), stream=other),
                 lambda: m.moe_route(z, ids, wt, stream=other),
                 lambda: m.moe_route_backward(z, ids, wt, wt, torch.zeros_like(z), stream=other),
                 lambda: m.moe_scale_backward(s, **a, stream=other)):
        with pytest.raises(m.MoEError, match="GPU 1") as ei:
            call()
        assert ei.value.status == m.MOE_EINVAL
    torch.cuda.synchronize()
    assert bool((ids == 3).all())


def test_a_scale_of_zero_is_rejected():
    """In the C options 0 stands for 1; a number given to the binding is meant."""
    m = _m()
    z, ids, w = torch.zeros(4, 16), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    for scale in (0, 0.0, -0.0):
        with pytest.raises(m.MoEError, match="scale is 0") as ei:
            m.moe_route(z, ids, w, scale=scale)
        assert ei.value.status == m.MOE_EINVAL
        with pytest.raises(m.MoEError, match="scale is 0"):
            m.moe_route_backward(z, ids, w, w, torch.zeros_like(z), scale=scale)


def test_a_scale_below_the_smallest_float_is_rejected():
    m = _m()
    z, ids, w = torch.zeros(4, 16), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    with pytest.raises(m.MoEError, match="scale is 0"):
        m.moe_route(z, ids, w, scale=1e-50)


@pytest.mark.gpu
def test_a_scale_held_in_a_tensor_is_read_at_every_call():
    m = _m()
    z = torch.randn(64, 16, device="cuda")
    ids, w = torch.empty(64, 2, dtype=torch.int32, device="cuda"), torch.empty(64, 2, device="cuda")
    scale = torch.tensor(1.0)
    m.moe_route(z, ids, w, scale=scale)
    once = w.clone()
    scale.fill_(2.0)
    m.moe_route(z, ids, w, scale=scale)
    assert torch.equal(w, 2 * once)
    d, twice = torch.empty_like(z), torch.empty_like(z)
    m.moe_route_backward(z, ids, w, torch.ones_like(w), d, scale=2.0)
    m.moe_route_backward(z, ids, w, torch.ones_like(w), twice, scale=scale)
    assert torch.equal(d, twice)
    with pytest.raises(TypeError):
        m.moe_route(z, ids, w, n_group=2.0)
