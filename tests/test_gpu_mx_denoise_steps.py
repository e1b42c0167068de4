"""The 8-bit denoising loop call by call: what every call of a block reads is what the one before it wrote, with the right
parameters, and every result is the float64 oracle's on those inputs; and the cached loop against the recomputed one."""

import numpy as np
import pytest
import torch

import diffusion_transformer_joint_axial_b200 as qi
from diffusion_transformer_joint_axial_b200 import _binding as qb
from diffusion_transformer_joint_axial_b200 import workloads as W
from oracle import mx_oracle as X

import test_gpu_mx as mx

pytestmark = pytest.mark.gpu

SEGS = [W.text(40), W.image(6, 6, 1), W.image(8, 8, 0)]
HEADS, CH, BLOCKS, STEPS = 2, 16, 2, 3


def _model(dev, segs, heads, blocks, steps, seed, cached=True):
    params, draw = W.denoise_model(heads, CH, blocks, steps, seed=seed)
    T = W.seg_tokens(segs[-1])
    x0, ph = draw(1, sum(W.seg_tokens(s) for s in segs) - T, T, seed + 1)
    m = qi.denoise.DenoiseModel(segs, heads, CH, blocks, steps, W.denoise_sigmas(steps), device=dev, cached=cached,
                                precision="mx")
    m.load(params, x0, ph)
    return m, params, x0, ph


def _copy(v):
    if isinstance(v, qi.MXTensor):
        return qi.MXTensor(v.q.clone(), v.scale.clone())
    if isinstance(v, torch.Tensor):
        return v.clone()
    return [_copy(e) for e in v] if isinstance(v, list) else v


def _record(monkeypatch):
    """Every call of the loop: (name, inputs as they were, keyword inputs, results)."""
    calls = []
    for name in ("rmsnorm", "linear", "linear_residual", "rmsnorm_mx", "linear_mx", "linear_swiglu_mx", "mx_quantize",
                 "attn_full", "attn_cached"):
        def wrapped(*args, _name=name, _real=getattr(qb, name), **kw):
            before = [_copy(a) for a in args], {k: _copy(v) for k, v in kw.items() if k not in ("out", "workspace")}
            out = _real(*args, **kw)
            calls.append((_name, *before, _copy(out)))
            return out
        monkeypatch.setattr(qb, name, wrapped)
    return calls


def _same(a, b):
    if isinstance(a, qi.MXTensor):
        return np.array_equal(*(X.values(*mx._read(t)) for t in (a, b)))
    return torch.equal(a.reshape(-1), b.reshape(-1))


def _quantized(w):
    """The 8-bit form of a parameter, by the oracle."""
    q, byte = X.quantize(W.as_f64(w))
    return X.values(q, byte)


def _check_block(calls, h, blk, attend):
    """Eight calls of one block on hidden states h; returns the hidden states that they leave."""
    names = [c[0] for c in calls]
    assert names == ["rmsnorm_mx", "linear_mx", attend, "mx_quantize", "linear_mx", "rmsnorm_mx", "linear_swiglu_mx",
                     "linear_mx"]
    f = W.as_f64
    D = h.shape[-1]
    flat = lambda t: f(t).reshape(-1, t.shape[-1])
    norm1, qkv, att, quant, proj, norm2, gated, down = calls

    def check_norm(c, x, w):
        assert _same(c[1][0], x) and _same(c[1][1].cpu(), w) and c[1][2] == 1e-6 and not c[2]
        mx._check_rounded(c[3], X.rms_norm(flat(x), f(w), 1e-6), (D / 64 + 10) * 2.0 ** -24)

    def check_linear(c, x, w, b, n_out, residual):
        args, kw, outs = c[1], c[2], c[3]
        assert len(args) == 3 and _same(args[0], x) and _same(args[2].cpu(), b)
        wv = _quantized(w)
        assert np.array_equal(X.values(*mx._read(args[1])), wv)
        assert kw.pop("n_out", 1) == n_out
        r = kw.pop("residual", None)
        assert (r is None) == (residual is None) and (r is None or _same(r, residual)) and not kw
        mx._check_linear(outs, X.values(*mx._read(x)), wv, f(b), "none", None if r is None else flat(r), 1.0, wv.shape[1])

    check_norm(norm1, h, blk["norm1"])
    check_linear(qkv, norm1[3], blk["w_qkv"], blk["b_qkv"], 3, None)
    assert all(_same(a, b) for a, b in zip(att[1][:3], qkv[3]))
    assert _same(quant[1][0], att[3]) and np.array_equal(X.values(*mx._read(quant[3])), _quantized(att[3].reshape(-1, D)))
    check_linear(proj, quant[3], blk["w_o"], blk["b_o"], 1, h)
    mid = proj[3][0]
    check_norm(norm2, mid, blk["norm2"])
    # the gated projection: slack as in its own test
    assert _same(gated[1][0], norm2[3]) and not gated[2]
    w, b = qi.interleave_gate_up(blk["w_gu"]), qi.interleave_gate_up(blk["b_gu"])
    assert np.array_equal(X.values(*mx._read(gated[1][1])), _quantized(w)) and _same(gated[1][2].cpu(), b)
    xv, wv, bv = X.values(*mx._read(norm2[3])), _quantized(w), f(b)
    M = xv.shape[0]
    y = X.linear_mx(xv, wv, bv)
    acc = (mx._acc_bound(xv, wv, D) + 2.0 ** -23 * np.abs(y)).reshape(M, -1, 2, 128)
    y = y.reshape(M, -1, 2, 128)
    g, u = np.abs(y[:, :, 0]), np.abs(y[:, :, 1])
    s = np.abs(y[:, :, 0] / (1 + np.exp(-y[:, :, 0])))
    slack = (1.11 * u * acc[:, :, 0] + s * acc[:, :, 1] + acc[:, :, 0] * acc[:, :, 1]
             + s * u * (8 + 4 * g) * 2.0 ** -23 + 1e-30).reshape(M, -1)
    mx._check_rounded(gated[3], X.swiglu(xv, wv, bv), 0.0, slack)
    check_linear(down, gated[3], blk["w_down"], blk["b_down"], 1, mid)
    return down[3][0]


@pytest.mark.parametrize("cached", [True, False])
def test_every_call_of_the_loop(cuda_device, monkeypatch, cached):
    m, params, x0, ph = _model(cuda_device, SEGS, HEADS, BLOCKS, STEPS, 31, cached)
    calls = _record(monkeypatch)
    m.run()
    m.check()
    P, sig = m.P, W.denoise_sigmas(STEPS)
    x, at = x0, 0
    for step in range(STEPS):
        full = step == 0 or not cached
        name, args, _, out = calls[at]
        assert name == "linear" and _same(args[0].cpu(), x) and _same(args[1].cpu(), params["w_in"])
        assert _same(args[2].cpu(), params["b_in"][step])
        h = torch.cat([ph.to(cuda_device), out[0]], 1) if full else out[0]
        at += 1
        for blk in params["blocks"]:
            h = _check_block(calls[at:at + 8], h, blk, "attn_full" if full else "attn_cached")
            at += 8
        h_t = h.reshape(1, -1, h.shape[-1])[:, P:] if full else h
        (n1, a1, _, o1), (n2, a2, kw2, o2) = calls[at:at + 2]
        assert (n1, n2) == ("rmsnorm", "linear_residual")
        assert _same(a1[0], h_t.contiguous()) and _same(a1[1].cpu(), params["norm_out"]) and _same(a2[0], o1)
        assert _same(a2[1].cpu(), params["w_v"]) and _same(a2[2].cpu(), params["b_v"]) and _same(a2[3].cpu(), x)
        assert kw2["alpha"] == sig[step + 1] - sig[step]
        x = o2.cpu()
        at += 2
    assert at == len(calls) and _same(m.x.cpu(), x)


@pytest.mark.parametrize("segs,heads,blocks", [
    ([W.text(64), W.image(8, 8, 1), W.image(8, 12, 0)], 2, 2),
    ([W.text(128), W.image(16, 16, 1), W.image(40, 40, 0)], 2, 2),
    (W.WORKLOADS["t2i"]["segments"], W.WORKLOADS["t2i"]["H"], 1)])
def test_cached_loop_is_the_recomputed_one_bit_for_bit(cuda_device, segs, heads, blocks):
    """A Prefix of whole 128-key tiles, products that sum K in one part for both numbers of tokens, and an attention that
    sums its keys in one part (the cached step's workspace has no room for pieces; the second layout's
    step would be cut into some): the Prefix never sees the step and every row is computed by itself, so reuse of its
    keys and values changes nothing."""
    D = 128 * heads
    for M in (sum(W.seg_tokens(s) for s in segs), W.seg_tokens(segs[-1])):
        for N, K, kw in ((3 * D, D, {}), (D, D, dict(residual=True)), (6 * D, D, dict(gated=True)),
                         (D, 3 * D, dict(residual=True))):
            assert qi.mx_plan(M, N, K, **kw)[1] == 1
    out = []
    for cached in (True, False):
        m, _, x0, _ = _model(cuda_device, segs, heads, blocks, 3, 33, cached)
        up = lambda n: (n + 255) // 256 * 256
        m.ws_cached = qi.new_workspace(up(up(256 + m.T * 64 * 8) + heads * m.T * 128 * 2), cuda_device)
        m.run()
        m.check()
        out.append(m.x.cpu())
    assert torch.equal(out[0], out[1])
    assert (out[0].float() - x0.float()).abs().mean() > 0.1
