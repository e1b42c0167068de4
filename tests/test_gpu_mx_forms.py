"""Each kernel behind the MX products against the float64 oracle: few tokens with K in parts, CTA pairs with one and with
several tiles each, pairs with K split.  Every case first asserts that its sizes reach the kernel that it is about."""

import numpy as np
import pytest
import torch

import diffusion_transformer_joint_axial_b200 as qi
from diffusion_transformer_joint_axial_b200 import workloads as W
from oracle import mx_oracle as X

import mx_forms as forms
import test_gpu_mx as mx
from parity import check_status

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _plan(M, N, K, want, **kw):
    assert qi.mx_plan(M, N, K, **kw) == want


@pytest.mark.parametrize("M,N,K,n_out,act,residual,want", forms.LINEAR)
def test_linear(cuda_device, M, N, K, n_out, act, residual, want):
    """Bias, activation, alpha and residual, into new tensors and, with a residual, in place."""
    _plan(M, N, K, want, act=act, residual=residual)
    rng = np.random.default_rng(M + 3 * N + K)
    dev = cuda_device
    x, xv = mx._mx_operand(rng, M, K, 1.0, dev)
    w, wv = mx._mx_operand(rng, N, K, K ** -0.5, dev)
    b = mx._bf(0.1 * rng.standard_normal(N))
    r = mx._bf(rng.standard_normal((M, N))) if residual else None
    alpha = -0.625 if residual else 1.75
    ws = qi.new_workspace(256, dev)
    args = dict(n_out=n_out, act=act, alpha=alpha, workspace=ws)
    outs = qi.linear_mx(x, w, b.to(dev), residual=None if r is None else r.to(dev), **args)
    check_status(ws)
    mx._check_linear(outs, xv, wv, W.as_f64(b), act, None if r is None else W.as_f64(r), alpha, K, str(want))
    if residual:
        h = r.to(dev)
        (got,) = qi.linear_mx(x, w, b.to(dev), residual=h, out=[h], **args)
        check_status(ws)
        assert got is h and torch.equal(h, outs[0])


def _powers(rng, R, K):
    """(float64 values, bf16 tensor) of +-2^e with another e in -3 .. 3 for every (row, block)."""
    e = rng.integers(-3, 4, (R, K // 32))
    v = np.ldexp(rng.choice([-1.0, 1.0], (R, K)), np.repeat(e, 32, 1))
    return v, mx._bf(v)


EXACT = [(M, N, K, want) for M, N, K, want in (
    (128, 264, 7456, ("few", 4)),
    (385, 1032, 4128, ("few", 2)),
    (2600, 4104, 1184, ("pairs", 1)),           # K ends with one block
    (5000, 2056, 1056, ("pairs", 1)),           # several tiles a pair: slots and accumulators in turn
    (4700, 4104, 1024, ("pairs", 1)),
    (700, 2056, 3104, ("pairs_split", 2)),
    (300, 3976, 4096, ("pairs_split", 2)))]


@pytest.mark.parametrize("M,N,K,want", EXACT)
def test_exact_products_read_every_scale(cuda_device, M, N, K, want):
    """The partial sums are whole multiples of 2^-6 below 2^24 of them, so fp32 holds them in any order and a scale
    from a wrong row, block, tile or step shows."""
    _plan(M, N, K, want)
    rng = np.random.default_rng(M + N)
    xv, xb = _powers(rng, M, K)
    wv, wb = _powers(rng, N, K)
    assert 64 * (np.abs(xv) @ np.abs(wv).T).max() < 2 ** 24
    (got,) = qi.linear_mx(qi.mx_quantize(xb.to(cuda_device)), qi.mx_quantize(wb.to(cuda_device)))
    assert torch.equal(got.cpu(), torch.from_numpy(xv @ wv.T).to(torch.float32).to(BF))


@pytest.mark.parametrize("M,F,K,want", forms.GATED)
def test_gated_exact_sums_read_every_scale(cuda_device, M, F, K, want):
    """The same sums through the gate: exact up to silu's exponential, off by (8 + 4 |g|) 2^-23 of a value."""
    _plan(M, 2 * F, K, want, gated=True)
    rng = np.random.default_rng(M + F)
    xv, xb = _powers(rng, M, K)
    wv, wb = _powers(rng, 2 * F, K)
    assert 64 * (np.abs(xv) @ np.abs(wv).T).max() < 2 ** 24
    # gates of about +-1: a power of two on top of every row of W scales its sums exactly
    down = 2.0 ** -np.rint(np.log2(np.sqrt(K) * 5))
    got = qi.linear_swiglu_mx(qi.mx_quantize(xb.to(cuda_device)), qi.mx_quantize((wb.double() * down).to(BF).to(cuda_device)))
    y = (xv @ wv.T * down).reshape(M, -1, 2, 128)
    g, u = y[:, :, 0], y[:, :, 1]
    ref = (g / (1 + np.exp(-g)) * u).reshape(M, F)
    # (a gate below -87 is a value below 2^-120; see the last term)
    slack = np.abs(ref) * ((8 + 4 * np.abs(g)) * 2.0 ** -23).reshape(M, F) + 1e-30
    mx._check_rounded(got, ref, 0.0, slack)


SOME = [(2600, 4104, 1184, ("pairs", 1)), (700, 2056, 3104, ("pairs_split", 2)), (385, 1032, 4128, ("few", 2))]


@pytest.mark.parametrize("M,N,K,want", SOME)
def test_non_finite_blocks_reach_their_rows_and_columns_only(cuda_device, M, N, K, want):
    """NaN and infinity in blocks of X and W, in the first and the last step of K: whole rows and columns of NaN, and
    everything else as it is without them."""
    _plan(M, N, K, want)
    rng = np.random.default_rng(M)
    dev = cuda_device
    xb, wb = mx._act(rng, M, K), mx._bf(rng.standard_normal((N, K)) * K ** -0.5)
    (clean,) = qi.linear_mx(qi.mx_quantize(xb.to(dev)), qi.mx_quantize(wb.to(dev)))
    rows, cols = {2: 5, 257: K - 1, M - 1: K // 2}, {0: K - 3, 130: 7, N - 1: 40}
    for r, k in rows.items():
        xb[r, k] = float("nan")
    for c, k in cols.items():
        wb[c, k] = float("-inf")
    (got,) = qi.linear_mx(qi.mx_quantize(xb.to(dev)), qi.mx_quantize(wb.to(dev)))
    bad = torch.zeros(M, N, dtype=torch.bool, device=dev)
    bad[list(rows)] = True
    bad[:, list(cols)] = True
    assert torch.equal(torch.isnan(got), bad)
    assert torch.equal(got[~bad], clean[~bad])


@pytest.mark.parametrize("M,N,K,residual,want", [
    (2601, 4104, 1184, False, ("pairs", 1)), (5003, 2056, 1056, True, ("pairs", 1)),
    (701, 2056, 3104, False, ("pairs_split", 2)), (509, 4096, 3104, True, ("pairs_split", 2)),
    (387, 1032, 4128, False, ("few", 2))])
def test_rows_behind_the_last_stay(cuda_device, M, N, K, residual, want):
    """bf16 results: what lies behind row M in the same storage is not written, all of the M rows are."""
    _plan(M, N, K, want, residual=residual)
    rng = np.random.default_rng(M)
    dev = cuda_device
    x, _ = mx._mx_operand(rng, M, K, 1.0, dev)
    w, _ = mx._mx_operand(rng, N, K, K ** -0.5, dev)
    out = torch.full((M + 40, N), 7.0, dtype=BF, device=dev)
    r = torch.zeros(M, N, dtype=BF, device=dev) if residual else None
    qi.linear_mx(x, w, residual=r, out=[out[:M]])
    assert bool((out[M:] == 7).all()) and float((out[:M] == 7).double().mean()) < 1e-3


@pytest.mark.parametrize("M,F,K,want", [(905, 1152, 1056, ("pairs", 1)), (2503, 3200, 512, ("pairs", 1)),
                                        (301, 2048, 4096, ("pairs_split", 2))])
def test_gated_rows_behind_the_last_stay(cuda_device, M, F, K, want):
    """8-bit values and scales of the rows behind the last one."""
    _plan(M, 2 * F, K, want, gated=True)
    rng = np.random.default_rng(M)
    dev = cuda_device
    x, _ = mx._mx_operand(rng, M, K, 1.0, dev)
    w, _ = mx._mx_operand(rng, 2 * F, K, K ** -0.5, dev)
    q = torch.full((M + 40, F), 9, dtype=torch.uint8, device=dev)
    groups = (M + 127) // 128
    scale = torch.full((groups, F // 128, 32, 4, 4), 0xAB, dtype=torch.uint8, device=dev)
    qi.linear_swiglu_mx(x, w, out=qi.MXTensor(q[:M].view(torch.float8_e4m3fn), scale.view(torch.float8_e8m0fnu)))
    assert bool((q[M:] == 9).all()) and float((q[:M] == 9).double().mean()) < 0.1
    full = X.untile(scale.cpu().numpy(), groups * 128, F)
    assert (full[M:] == 0xAB).all() and (full[:M] != 0xAB).all()


PADDED = [(1, 136, 96, False, ("few", 1)), (128, 264, 7456, False, ("few", 4)), (385, 1032, 4128, False, ("few", 2)),
          (2601, 4104, 1184, False, ("pairs", 1)), (701, 2056, 3104, False, ("pairs_split", 2)),
          (77, 512, 160, True, ("few", 1)), (905, 2304, 1056, True, ("pairs", 1)), (701, 2304, 3104, True, ("pairs_split", 2))]


@pytest.mark.parametrize("M,N,K,gated,want", PADDED)
def test_padding_of_scales_is_ignored(cuda_device, M, N, K, gated, want):
    """Scale bytes of the rows and blocks that pad the last tiles may be anything, NaN among it."""
    _plan(M, N, K, want, gated=gated)
    rng = np.random.default_rng(M + N)
    dev = cuda_device
    x, _ = mx._mx_operand(rng, M, K, 1.0, dev)
    w, _ = mx._mx_operand(rng, N, K, K ** -0.5, dev)

    def run():
        if gated:
            t = qi.linear_swiglu_mx(x, w)
            return t.q.view(torch.uint8)
        return qi.linear_mx(x, w)[0]

    want = run()
    for t in (x, w):
        s = t.scale.view(torch.uint8)
        rows, cols = s.shape[0] * 128, s.shape[1] * 4
        flat = s.permute(0, 3, 2, 1, 4).reshape(rows, cols)      # a copy: bytes by row and block
        pad = torch.ones_like(flat, dtype=torch.bool)
        pad[: t.q.shape[0], : K // 32] = False
        assert bool(pad.any())
        flat[pad] = 255
        s.copy_(flat.view(s.shape[0], 4, 32, s.shape[1], 4).permute(0, 3, 2, 1, 4))
        assert np.array_equal(X.untile(s.cpu().numpy(), *t.q.shape) == 255, np.zeros((t.q.shape[0], K // 32), dtype=bool))
    assert torch.equal(run(), want)
