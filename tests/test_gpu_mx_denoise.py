"""The denoising loop with its blocks' projections and feed-forward layers in MX (8-bit) form."""

import numpy as np
import pytest
import torch

import diffusion_transformer_joint_axial_b200 as qi
import oracle as O
from diffusion_transformer_joint_axial_b200 import workloads as W

pytestmark = pytest.mark.gpu

SEGS = [W.text(40), W.image(6, 6, 1), W.image(8, 8, 0)]
HEADS, CH, BLOCKS, STEPS = 2, 16, 2, 3


def _model(dev, cached=True, segs=SEGS, precision="mx", seed=31):
    sig = W.denoise_sigmas(STEPS)
    params, draw = W.denoise_model(HEADS, CH, BLOCKS, STEPS, seed=seed)
    L, T = sum(W.seg_tokens(s) for s in segs), W.seg_tokens(segs[-1])
    x0, ph = draw(1, L - T, T, seed + 1)
    m = qi.denoise.DenoiseModel(segs, HEADS, CH, BLOCKS, STEPS, sig, device=dev, cached=cached, precision=precision)
    m.load(params, x0, ph)
    return m, params, x0, ph, sig


def _f64(params):
    conv = lambda v: W.as_f64(v) if isinstance(v, torch.Tensor) else v
    out = {k: conv(v) for k, v in params.items() if k != "blocks"}
    out["blocks"] = [{k: conv(v) for k, v in b.items()} for b in params["blocks"]]
    return out


# What 8 bits cost, from the format alone.  Rounding to e4m3 is off by step / sqrt(12) rms, 2.6 % of
# a value; a product of two quantised operands by sqrt(2) times that, 3.7 %.  The attention's branch:
# V 3.7 %, the weights about 5 % (scores of order 1 from Q and K, 3.7 % each), the quantised output and
# its projection 3.7 %: 7.3 %.  The feed-forward branch: gate and up 3.7 % each, the second product
# 3.7 %: 6.6 %.  Two blocks of two branches, added to a residual stream of the same size: at most
# 10.6 % of the velocity's rms in every step, and over the steps (their errors alike in the worst case, and
# felt again by the next step) less than twice that.
LOSS = 0.2


@pytest.mark.parametrize("segs,seed", [(SEGS, 31), ([W.text(200), W.image(24, 24, 1), W.image(40, 40, 0)], 45)])
def test_against_oracle(cuda_device, segs, seed):
    m, params, x0, ph, sig = _model(cuda_device, segs=segs, seed=seed)
    m.run()
    m.check()
    ref = O.denoise(W.as_f64(x0), W.as_f64(ph), _f64(params), segs, sig, cached=True)
    got, start = W.as_f64(m.x.cpu()), W.as_f64(x0)
    rms = lambda a: float(np.sqrt(np.mean(a * a)))
    assert np.isfinite(got).all()
    assert rms(got - ref) <= LOSS * rms(ref - start), (rms(got - ref), rms(ref - start))
    # a replay of the captured loop, from the same latents, gives the same bits
    eager = m.x.clone()
    m.x.copy_(x0)
    m.capture()
    m.x.copy_(x0)
    m.replay()
    m.check()
    assert torch.equal(m.x, eager)


def test_cached_is_the_recomputation(cuda_device):
    """The Prefix never sees the step, and every MX row is quantised by itself: the two loops differ by where
    they round to bf16, which moves some values across an e4m3 border, so by less than quantising does."""
    out = []
    for cached in (True, False):
        m, _, x0, *_ = _model(cuda_device, cached=cached)
        m.run()
        m.check()
        out.append(W.as_f64(m.x.cpu()))
    rms = lambda a: float(np.sqrt(np.mean(a * a)))
    assert rms(out[0] - out[1]) <= LOSS * rms(out[1] - W.as_f64(x0))


def test_default_precision_is_unchanged(cuda_device):
    a, *_ = _model(cuda_device, precision="bf16")
    assert isinstance(a.blocks[0]["w_qkv"], torch.Tensor) and "a8" not in a.act[a.L]
    with pytest.raises(qi.QI21Error):
        _model(cuda_device, precision="int8")
