"""The differentiable operations of the linear attention allocate and compute
what a gradient needs only where one is asked for."""
import pytest
import torch

from test_linear_attn_gpu import both, inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"


def peak(f):
    """Result, and bytes allocated at the most on the way."""
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    out = f()
    return out, torch.cuda.max_memory_allocated() - before


def test_a_prompt_saves_no_states(gpu):
    s, _, _ = inputs(2, 4096, 8, 1, 128, 64, "bf16", True, True, seed=50)
    states = gpu.linear_attn_states_bytes(2, 4096, 8, 128, 64, 1)
    assert states > 30 << 20
    rest = s["v"].numel() * 2 + s["h0"].numel() * 4 + \
        gpu.linear_attn_workspace_bytes(2, 4096, 8, 1, 128, 64, 1) + (4 << 20)
    args = [s[n] for n in ("q", "k", "v", "g", "h0")]
    kw = {"scale": 0.1, "reset": s["reset"]}
    (want, h), with_states = peak(lambda: both_of(gpu, [x.clone().requires_grad_() for x in args], kw))
    assert with_states > states
    (o, last), plain = peak(lambda: gpu.linear_attn(*args, **kw, return_last=True))
    assert plain < rest
    assert torch.equal(o, want) and torch.equal(last, h) and not o.requires_grad
    leaves = [x.clone().requires_grad_() for x in args]
    with torch.no_grad():
        o, plain = peak(lambda: gpu.linear_attn(*leaves, **kw))
    assert plain < rest and torch.equal(o, want) and not o.requires_grad
    with torch.inference_mode():
        assert torch.equal(gpu.linear_attn(*leaves, **kw), want)


def both_of(gpu, leaves, kw):
    o, h = gpu.linear_attn(*leaves, **kw, return_last=True)
    assert o.requires_grad and h.requires_grad
    return o.detach(), h.detach()


def test_gradients_of_some(gpu):
    """Each input's gradient by itself, with and without the last state."""
    s, do, dh = inputs(2, 70, 4, 2, 16, 24, "f32", True, True, seed=51)
    _, _, d = both(gpu, s, do, dh)
    _, _, only = both(gpu, s, do, None)
    for n in ("q", "k", "v", "g", "h0"):
        t = {m: s[m].clone().requires_grad_(m == n) for m in ("q", "k", "v", "g", "h0")}
        o, h = gpu.linear_attn(*t.values(), scale=0.3, reset=s["reset"], return_last=True)
        ((o * do).sum() + (h * dh).sum()).backward()
        assert torch.equal(t[n].grad, d["d" + n]), n
        assert all(x.grad is None for m, x in t.items() if m != n)
        t[n].grad = None
        (gpu.linear_attn(*t.values(), scale=0.3, reset=s["reset"]) * do).sum().backward()
        assert torch.equal(t[n].grad, only["d" + n]), n
    h0 = s["h0"].clone().requires_grad_()
    o, h = gpu.linear_attn(s["q"], s["k"], s["v"], s["g"], h0, scale=0.3, return_last=True)
    h.sum().backward()  # o is not used
    assert torch.isfinite(h0.grad).all() and h0.grad.any()


def test_refusals_without_a_gradient(gpu):
    s, _, _ = inputs(2, 40, 4, 2, 16, 24, "bf16", seed=52)
    q, k, v, g = (s[n] for n in "qkvg")
    for bad in ((q, k[0], v, g), (q, k, v[0], g), (q, k, v[..., 0], g), (q, k, v, g[:, 1:]),
                (None, k, v, g), (q.float(), k, v, g)):
        for last in (False, True):
            with pytest.raises((ValueError, TypeError)):
                gpu.linear_attn(*bad, return_last=last)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_group_norm_gradients_of_some(gpu, io):
    """dweight and dbias are made (and their workspace is taken) only where they
    are wanted; all else is the same."""
    from test_group_norm_gpu import inputs as norm_inputs
    rows, groups, size = 9000, 2, 256
    s = norm_inputs(rows, groups, size, io, True, True, True, seed=60)
    args = (groups, s["weight"], s["bias"], s["z"])
    want, with_weights = peak(lambda: gpu.group_norm_bwd(s["x"], s["dy"], *args))
    need = gpu.group_norm_bwd_workspace_bytes(rows, groups, size, int(io == "bf16"))
    assert need > 1 << 20
    for w in (False, True):
        for b in (False, True):
            d, used = peak(lambda: gpu.group_norm_bwd(s["x"], s["dy"], *args, want_dweight=w,
                                                      want_dbias=b))
            assert (d["dweight"] is not None) == w and (d["dbias"] is not None) == b
            for n, x in d.items():
                assert x is None or torch.equal(x, want[n]), n
            assert w or b or used <= with_weights - need
    for only in ("x", "weight", "bias", "z"):
        t = {n: s[n].clone().requires_grad_(n == only) for n in ("x", "weight", "bias", "z")}
        gpu.group_norm(t["x"], groups, t["weight"], t["bias"], t["z"]).backward(s["dy"])
        assert torch.equal(t[only].grad, want["d" + only]), only
        assert all(x.grad is None for n, x in t.items() if n != only)
