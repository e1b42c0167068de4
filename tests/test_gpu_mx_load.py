"""What DenoiseModel.load() and the MX calls take beside contiguous bf16 tensors and Python floats: whatever the bf16
forms take."""

import numpy as np
import pytest
import torch

import diffusion_transformer_joint_axial_b200 as qi
from diffusion_transformer_joint_axial_b200 import workloads as W

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
SEGS = [W.text(16), W.image(4, 4, 1), W.image(4, 6, 0)]
HEADS, CH, BLOCKS, STEPS = 1, 16, 2, 2


def _loaded(dev, precision, change):
    params, draw = W.denoise_model(HEADS, CH, BLOCKS, STEPS, seed=5)
    T = W.seg_tokens(SEGS[-1])
    x0, ph = draw(1, sum(W.seg_tokens(s) for s in SEGS) - T, T, 6)
    m = qi.denoise.DenoiseModel(SEGS, HEADS, CH, BLOCKS, STEPS, W.denoise_sigmas(STEPS), device=dev,
                                precision=precision)
    m.load(change(params), x0, ph)
    torch.cuda.synchronize()
    return m


def _bytes(t):
    if isinstance(t, qi.MXTensor):
        return torch.cat([t.q.view(torch.uint8).reshape(-1), t.scale.view(torch.uint8).reshape(-1)])
    return t.view(torch.uint8)


def _assert_same_parameters(a, b):
    for name in ("w_in", "b_in", "norm_out", "w_v", "b_v", "x", "prefix_h"):
        assert torch.equal(getattr(a, name), getattr(b, name)), name
    for i, (p, q) in enumerate(zip(a.blocks, b.blocks)):
        for k in p:
            assert torch.equal(_bytes(p[k]), _bytes(q[k])), (i, k)


def _each(f):
    def change(params):
        out = {k: f(v) for k, v in params.items() if k != "blocks"}
        out["blocks"] = [{k: f(v) for k, v in b.items()} for b in params["blocks"]]
        return out
    return change


CHANGES = {
    "float32": _each(lambda t: t.float()),
    "float64": _each(lambda t: t.double()),
    "transposed": _each(lambda t: t.t().contiguous().t() if t.dim() == 2 else t),
    "strided": _each(lambda t: torch.stack([t, t], -1)[..., 0]),
    "on the device": _each(lambda t: t.cuda()),
}


@pytest.mark.parametrize("change", CHANGES)
@pytest.mark.parametrize("precision", ["bf16", "mx"])
def test_load_takes_types_and_strides(cuda_device, precision, change):
    """bf16 values in another type or layout load as the values themselves."""
    _assert_same_parameters(_loaded(cuda_device, precision, CHANGES[change]), _loaded(cuda_device, precision, lambda p: p))


@pytest.mark.parametrize("precision", ["bf16", "mx"])
def test_load_takes_blocks_from_an_iterator(cuda_device, precision):
    """Parameters that a program produces block by block."""
    _assert_same_parameters(_loaded(cuda_device, precision, lambda p: dict(p, blocks=iter(p["blocks"]))),
                            _loaded(cuda_device, precision, lambda p: p))


def test_rows_longer_than_an_int_are_refused(cuda_device):
    """A row of 2^32 + 32 values, not of 32."""
    x = torch.empty(1, 2 ** 32 + 32, dtype=BF, device=cuda_device)
    for call in (lambda: qi.rmsnorm_mx(x, x[0], 1e-6), lambda: qi.mx_quantize(x)):
        with pytest.raises(qi.QI21Error):
            call()


def test_results_in_place_of_operands(cuda_device):
    """Through the binding: an 8-bit result in its own operand is refused, neighbours in one buffer are not."""
    dev = cuda_device
    gen = torch.Generator(device=dev).manual_seed(3)
    a = qi.mx_quantize(torch.randn(300, 256, generator=gen, device=dev).to(BF))
    w = qi.mx_quantize(torch.randn(512, 256, generator=gen, device=dev).to(BF))
    want = qi.linear_swiglu_mx(a, w)
    for out in (a, qi.MXTensor(want.q, a.scale), qi.MXTensor(a.q, want.scale)):
        with pytest.raises(qi.QI21Error):
            qi.linear_swiglu_mx(a, w, out=out)
    y = torch.empty(2, 300, 256, dtype=BF, device=dev)
    with pytest.raises(qi.QI21Error):
        qi.linear_mx(a, w, n_out=2, out=[y[0], y[0]])
    qi.linear_mx(a, w, n_out=2, out=[y[0], y[1]])
    assert torch.equal(torch.cat([y[0], y[1]], 1), qi.linear_mx(a, w)[0])
    both = torch.empty(2, 300, 256, dtype=torch.uint8, device=dev)
    both[0] = a.q.view(torch.uint8)
    x = qi.MXTensor(both[0].view(torch.float8_e4m3fn), a.scale)
    got = qi.linear_swiglu_mx(x, w, out=qi.MXTensor(both[1].view(torch.float8_e4m3fn), want.scale.clone()))
    assert torch.equal(got.q.view(torch.uint8), want.q.view(torch.uint8))
