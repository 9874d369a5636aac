"""The tensor layer of the 128-element operators on a host without a GPU, with
plain torch in the kernels' place."""

import sys

import pytest
import torch


@pytest.fixture
def layers(mx, monkeypatch):
    """ops128 with its operators in plain arithmetic, without FP8."""
    from fp8_quantization_mx_b200 import ops128

    def quantize128(x, *args, direction="rows", **kw):
        return {"rows": (x, None), "cols": (x.t(), None), "both": (x, None, x.t(), None)}[direction]

    def norm(x, weight, residual=None, eps=1e-6, return_y=False):
        h = x if residual is None else x + residual
        y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + eps) * weight
        return y, None, None if residual is None else h, y if return_y else None

    def norm_bwd(gy, h, weight, eps, grad_residual=None):
        r = torch.rsqrt(h.square().mean(1, keepdim=True) + eps)
        n, g = h * r, gy * weight
        gh = r * (g - n * (g * n).mean(1, keepdim=True))
        return gh if grad_residual is None else gh + grad_residual, (gy * n).sum(0)

    monkeypatch.setattr(ops128, "quantize128", quantize128)
    monkeypatch.setattr(ops128, "rms_norm_quantize", norm)
    monkeypatch.setattr(ops128, "rms_norm_bwd", norm_bwd)
    monkeypatch.setattr(ops128, "gemm128", lambda a, sa, b, sb, **kw: a @ b.t())
    monkeypatch.setattr(ops128, "_layer_inputs", lambda **kw: None)
    return ops128


def plain_layer(x, nw, w, r, eps=1e-6):
    h = x if r is None else x + r
    return h * torch.rsqrt(h.square().mean(-1, keepdim=True) + eps) * nw @ w.t(), h


@pytest.mark.parametrize("shape", [(6, 8), (2, 3, 8)], ids=str)
@pytest.mark.parametrize("asked", ["x residual", "x", "residual", "norm_weight", "weight",
                                   "x residual norm_weight weight"])
def test_gradients_of_x_and_residual_accumulate_apart(layers, shape, asked):
    """Two backward passes into the same leaves: each gradient is the sum of
    both, in memory of its own, and exists where it was asked for."""
    g = torch.Generator().manual_seed(0)
    names = ("x", "residual", "norm_weight", "weight")
    sizes = (shape, shape, (8,), (4, 8))
    made = [torch.randn(s, generator=g, dtype=torch.float64) for s in sizes]
    mine, plain = ({n: t.clone().requires_grad_(n in asked.split()) for n, t in zip(names, made)}
                   for _ in range(2))
    for seed in (1, 2):
        g.manual_seed(seed)
        gy, gh = (torch.randn(*shape[:-1], n, generator=g, dtype=torch.float64) for n in (4, 8))
        for t, out in ((mine, layers.rms_norm_linear128(mine["x"], mine["norm_weight"], mine["weight"],
                                                        residual=mine["residual"])),
                       (plain, plain_layer(plain["x"], plain["norm_weight"], plain["weight"],
                                           plain["residual"]))):
            both = [(o, d) for o, d in zip(out, (gy, gh)) if o.requires_grad]
            torch.autograd.backward(*zip(*both))
    for n in names:
        a, b = mine[n].grad, plain[n].grad
        assert (a is None) == (n not in asked.split()) == (b is None)
        if a is not None:   # some 50 roundings of 2^-53 each, of values up to about 10
            assert torch.allclose(a, b, rtol=0, atol=1e-12)
    if mine["x"].grad is not None and mine["residual"].grad is not None:
        assert mine["x"].grad.untyped_storage().data_ptr() != \
            mine["residual"].grad.untyped_storage().data_ptr()


def test_layers_refuse_a_gradient_format_before_the_forward_pass(layers):
    x, nw, w = torch.ones(3, 8, requires_grad=True), torch.ones(8), torch.ones(4, 8)
    for fmt in (0, 3, -1, None):
        with pytest.raises(ValueError, match="grad_format"):
            layers.linear128(x, w, grad_format=fmt)
        with pytest.raises(ValueError, match="grad_format"):
            layers.rms_norm_linear128(x, nw, w, grad_format=fmt)
    for fmt in (layers.E4M3, layers.E5M2):
        layers.linear128(x, w, grad_format=fmt).sum().backward()


@pytest.mark.parametrize("there", [False, True], ids=["missing", "unloadable"])
def test_calls_without_the_extension_module_are_left_to_python(mx, monkeypatch, tmp_path, there):
    """The C++ module may not have been built, or for another torch."""
    from fp8_quantization_mx_b200 import ops128
    if there:
        (tmp_path / "_fast128.so").write_bytes(b"not a library")
    monkeypatch.setattr(mx, "__path__", [str(tmp_path)])
    monkeypatch.delattr(mx, "_fast128", raising=False)
    monkeypatch.delitem(sys.modules, "fp8_quantization_mx_b200._fast128", raising=False)
    monkeypatch.setattr(ops128, "_fast", None)
    assert ops128._bind_fast() is False and ops128._fast is False
    with pytest.raises(ValueError, match="CUDA"):   # Python's own check
        ops128.quantize128(torch.zeros(4, 256))


@pytest.mark.parametrize("why", ["no torch", "no compiler", "does not compile"])
def test_the_library_builds_without_the_extension_module(mx, monkeypatch, tmp_path, why):
    """The C library needs neither torch's headers nor a host compiler for them:
    without the module, or with one that is out of date, there is a warning."""
    from fp8_quantization_mx_b200 import build as b
    fast = tmp_path / "_fast128.so"
    fast.write_bytes(b"of another source")
    monkeypatch.setattr(b, "FAST", str(fast))
    if why == "no torch":
        monkeypatch.setitem(sys.modules, "torch", None)
    elif why == "no compiler":
        monkeypatch.setenv("PATH", str(tmp_path))
    else:
        (tmp_path / "broken.cpp").write_text("#error no such torch\n")
        monkeypatch.setattr(b, "FAST_SRC", str(tmp_path / "broken.cpp"))
    with pytest.warns(UserWarning, match="_fast128"):
        assert b.build() == b.LIB
    # what is out of date is not loaded (nothing is known of it without torch)
    assert fast.exists() == (why == "no torch")
