"""The MX (block-scaled 8-bit) operators on the GPU against the float64 oracle."""

import numpy as np
import pytest
import torch

import diffusion_transformer_joint_axial_b200 as qi
from diffusion_transformer_joint_axial_b200 import _binding as qb
from diffusion_transformer_joint_axial_b200 import workloads as W
from oracle import mx_oracle as X

from parity import check_status

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _bf(a):
    return torch.from_numpy(np.asarray(a, dtype=np.float32)).to(BF)


def _act(rng, M, K):
    """Rows of normal values whose channels differ in size."""
    return _bf(rng.standard_normal((M, K)) * np.exp(0.5 * rng.standard_normal(K)))


def _read(mx):
    """(values over 2^e [R, K], scale bytes [R, K / 32]) of an MX tensor, float64 and integers."""
    K = mx.q.shape[-1]
    q = mx.q.reshape(-1, K).view(torch.uint8).cpu().numpy()
    return X.e4m3_decode(q), X.untile(mx.scale.view(torch.uint8).cpu().numpy(), q.shape[0], K)


def _check_rounded(mx, y, rel, slack=0.0):
    """(q, byte) is a right rounding of some y' with |y' - y| <= rel |y| + slack: the exponent is the rule's for
    the largest |y'| of the block, and each value is within half a step of y': 2^-4 relative (three
    mantissa bits), or 2^-10 in units of 2^e below the smallest normal value."""
    q, byte = _read(mx)
    assert np.isfinite(q).all() and byte.max() < 255
    R, K = y.shape
    slack = np.broadcast_to(slack, y.shape)
    dev = rel * np.abs(y) + slack
    hi = (np.abs(y) + dev).reshape(R, -1, 32).max(-1)
    lo = np.maximum(np.abs(y) - dev, 0).reshape(R, -1, 32).max(-1)
    e = byte - 127
    assert np.all(lo <= np.ldexp(448.0, e)), "exponent too small"
    assert np.all((hi > np.ldexp(448.0, e - 1)) | (e == -127)), "exponent too large"
    step = np.repeat(np.ldexp(1.0, e), 32, axis=1)
    err = np.abs(q * step - y)
    bound = np.maximum(2.0 ** -4 * (np.abs(y) + dev), 2.0 ** -10 * step) + dev
    assert np.all(err <= bound), float((err - bound).max())


# ------------------------------------------------------------------ quantise

@pytest.mark.parametrize("M,K", [(1, 32), (1, 4096), (5, 96), (31, 160), (127, 128), (128, 256), (129, 2080), (300, 4064),
                                 (1000, 12288)])
def test_quantize_is_the_rule(cuda_device, M, K):
    """bf16 inputs are exact, so values and scales are the oracle's bit for bit."""
    rng = np.random.default_rng(M + K)
    x = _act(rng, M, K)
    x[0, : K // 2] *= 2.0 ** -120                       # subnormal after scaling, clamped exponents
    x[M - 1, K - 32:] = 0
    got = qi.mx_quantize(x.to(cuda_device))
    q, byte = _read(got)
    rq, rb = X.quantize(W.as_f64(x))
    assert np.array_equal(byte, rb)
    assert np.array_equal(q, rq)


def test_quantize_thresholds_extremes_and_non_finite(cuda_device):
    tops = [1.75, 1.7578125, 448.0, 450.0, 3.3895313892515355e38, 2.0 ** -126, 2.0 ** -133, 2.0 ** -118 * 1.75, 0.0]
    x = torch.zeros(len(tops) + 3, 64, dtype=BF)
    for i, t in enumerate(tops):
        x[i, 5] = t
        x[i, 40] = -t / 2
    n = len(tops)
    x[n], x[n + 1], x[n + 2] = 1.0, 2.0, 3.0
    x[n, 31], x[n + 1, 32], x[n + 2, 63] = float("nan"), float("inf"), float("-inf")
    got = qi.mx_quantize(x.to(cuda_device))
    q, byte = _read(got)
    rq, rb = X.quantize(W.as_f64(x))
    assert np.array_equal(byte, rb)
    assert np.array_equal(q, rq, equal_nan=True)


def test_padding_rows_are_left_alone(cuda_device):
    """Scale bytes of rows past M stay as they were; blocks past K in a written row read zero; values past the
    last row are not touched."""
    M, K = 130, 160
    rng = np.random.default_rng(3)
    x = _act(rng, M, K).to(cuda_device)
    q = torch.full((M + 2, K), 7, dtype=torch.uint8, device=cuda_device)
    scale = torch.full((2, 2, 32, 4, 4), 0xAB, dtype=torch.uint8, device=cuda_device)
    out = qi.MXTensor(q[:M].view(torch.float8_e4m3fn), scale.view(torch.float8_e8m0fnu))
    w = torch.ones(K, dtype=BF, device=cuda_device)
    for call in (lambda: qi.mx_quantize(x, out=out), lambda: qi.rmsnorm_mx(x, w, 1e-6, out=out)):
        scale.fill_(0xAB)
        call()
        s = scale.cpu().numpy()
        r = np.arange(256)[:, None]
        b = np.arange(8)[None, :]
        full = s[r // 128, b // 4, r % 32, r % 128 // 32, b % 4]
        assert (full[M:] == 0xAB).all() and (full[:M, 5:] == 0).all() and (full[:M, :5] != 0xAB).any()
        assert (q[M:] == 7).all()


# ---------------------------------------------------------------------- norm

@pytest.mark.parametrize("M,D,delta", [(1, 32, False), (1, 4096, True), (3, 96, True), (37, 4096, True), (130, 2080, True),
                                       (64, 4096, False), (257, 8224, True), (20, 12288, False), (9, 20480, True),
                                       (2, 65536, True), (4000, 512, True), (3000, 1056, False)])
def test_rmsnorm_mx(cuda_device, M, D, delta):
    rng = np.random.default_rng(M + D)
    x, w = _act(rng, M, D), _bf(1 + 0.1 * rng.standard_normal(D))
    d = _bf(0.3 * rng.standard_normal((M, D))) if delta else None
    dev, eps = cuda_device, 1e-6
    if delta:
        h, got = qi.rmsnorm_mx(x.to(dev), w.to(dev), eps, delta=d.to(dev))
        want = (x.float() + d.float()).to(BF)           # one rounding of the exact sum
        assert torch.equal(h.cpu(), want)
        x = want
    else:
        got = qi.rmsnorm_mx(x.to(dev), w.to(dev), eps)
    y = X.rms_norm(W.as_f64(x), W.as_f64(w), eps)
    # fp32 sum of D squares over at least 32 partial sums: D / 32 + 8 roundings of 2^-24 at
    # most, and two for the mean, all halved by the root; four for the reciprocal root (two units
    # in the last place), one for the product with it (h * w is exact)
    _check_rounded(got, y, (D / 64 + 10) * 2.0 ** -24)


@pytest.mark.parametrize("alias", ["x", "delta"])
def test_rmsnorm_mx_sum_in_place(cuda_device, alias):
    rng = np.random.default_rng(8)
    M, D = 70, 4096
    x, d, w = _act(rng, M, D).to(cuda_device), _act(rng, M, D).to(cuda_device), torch.ones(D, dtype=BF, device=cuda_device)
    h, want = qi.rmsnorm_mx(x, w, 1e-6, delta=d)
    dst = x if alias == "x" else d
    h2, got = qi.rmsnorm_mx(x, w, 1e-6, delta=d, sum_out=dst)
    assert h2 is dst and torch.equal(dst, h)
    assert torch.equal(got.q.view(torch.uint8), want.q.view(torch.uint8))
    assert torch.equal(got.scale.view(torch.uint8), want.scale.view(torch.uint8))


def test_rmsnorm_mx_zero_and_non_finite_rows(cuda_device):
    M, D = 4, 256
    x = torch.ones(M, D, dtype=BF)
    x[0] = 0
    x[1, 3] = float("nan")
    x[2, 200] = float("inf")
    w = torch.ones(D, dtype=BF, device=cuda_device)
    q, byte = _read(qi.rmsnorm_mx(x.to(cuda_device), w, 1e-6))
    assert (q[0] == 0).all() and (byte[0] == 0).all()
    assert (byte[1] == 255).all() and np.isnan(q[1]).all()
    # an infinite sum of squares: every finite value becomes 0, inf * 0 is NaN
    assert np.isnan(q[2, 192:224]).all() and (q[2, :192] == 0).all() and byte[2, 6] == 255
    assert (X.values(q, byte)[3] == 1.0).all()


# ------------------------------------------------------------------ products

def _mx_operand(rng, R, K, scale, dev):
    t = qi.mx_quantize(_bf(rng.standard_normal((R, K)) * scale * np.exp(rng.standard_normal((1, K)) * 0.5)).to(dev))
    q, byte = _read(t)
    return t, X.values(q, byte)


def _acc_bound(xv, wv, K):
    """fp32 accumulation: K / 32 steps, each adding 32 exact products with an error of at most 2^-22 of the
    sum of magnitudes so far."""
    return (K / 32 + 4) * 2.0 ** -22 * (np.abs(xv) @ np.abs(wv).T)


def _check_linear(outs, xv, wv, b, act, res, alpha, K, what=""):
    got = torch.cat([o.reshape(-1, o.shape[-1]) for o in outs], dim=-1).double().cpu().numpy()
    ref = X.linear_mx(xv, wv, b, act, res, alpha)
    y = X.linear_mx(xv, wv, b)
    a = X.linear_mx(xv, wv, b, act)
    # the activations' slope is below 1.14; exp of magnitude t is off by (3 + 1.2 t) 2^-23 relative,
    # and gelu's exponent u by 2^-22 |u|
    u = np.abs(y) if act == "silu" else 1.6 * np.abs(y + 0.044715 * y ** 3)
    rel = 0.0 if act == "none" else (8 + 4 * np.minimum(u, 90)) * 2.0 ** -23
    err = 1.14 * _acc_bound(xv, wv, K) + 2.0 ** -23 * np.abs(y) + rel * np.abs(a) + 1e-30
    bound = 2.0 ** -8 * np.abs(ref) + 1.01 * abs(alpha) * err
    if res is not None:
        bound += 2.0 ** -23 * (np.abs(res) + np.abs(alpha * a))
    assert np.isfinite(got).all(), what
    assert np.all(np.abs(got - ref) <= bound), "%s: worst excess %.3g" % (what, float((np.abs(got - ref) - bound).max()))


SHAPES = [
    # M, N, K, n_out, bias, act, residual
    (1, 8, 32, 1, False, "none", False),            # the smallest
    (1, 4096, 256, 1, True, "silu", False),         # a time embedding's first layer
    (1, 1024, 4096, 1, True, "none", False),        # one row, long K
    (3, 264, 96, 3, True, "none", False),           # ragged everywhere
    (16, 136, 160, 1, True, "gelu_tanh", True),
    (17, 512, 1056, 1, False, "none", True),
    (32, 2048, 2048, 1, True, "none", False),
    (33, 520, 544, 1, True, "silu", True),
    (64, 768, 768, 3, False, "none", False),
    (65, 1000, 4064, 1, True, "gelu_tanh", False),
    (128, 128, 128, 1, False, "none", False),       # exact tiles
    (129, 256, 320, 2, True, "none", False),        # one row past a tile
    (256, 512, 512, 1, True, "none", True),
    (333, 1024, 2048, 1, True, "gelu_tanh", False),
    (700, 1032, 672, 3, True, "silu", False),
    (1000, 20480, 160, 4, True, "none", False),     # many column tiles
    (2049, 2056, 96, 1, True, "none", True),        # ragged in M, N and K past the large tiles
    (4352, 1536, 1024, 1, True, "silu", True),
    (333, 4096, 4096, 1, True, "gelu_tanh", False),  # few large tiles: K in two halves
    (1000, 2056, 4128, 1, True, "none", True),       # the same, ragged everywhere
    (513, 3 * 808, 3968, 3, True, "silu", False),    # segments that end inside of a box
]


@pytest.mark.parametrize("M,N,K,n_out,bias,act,residual", SHAPES)
def test_linear_mx(cuda_device, M, N, K, n_out, bias, act, residual):
    rng = np.random.default_rng(M + 3 * N + K)
    x, xv = _mx_operand(rng, M, K, 1.0, cuda_device)
    w, wv = _mx_operand(rng, N, K, K ** -0.5, cuda_device)
    b = _bf(0.1 * rng.standard_normal(N)) if bias else None
    r = _bf(rng.standard_normal((M, N))) if residual else None
    alpha = -0.625 if residual else 1.0
    ws = qi.new_workspace(256, cuda_device)
    outs = qi.linear_mx(x, w, None if b is None else b.to(cuda_device), n_out=n_out, act=act,
                        residual=None if r is None else r.to(cuda_device), alpha=alpha, workspace=ws)
    check_status(ws)
    _check_linear(outs, xv, wv, None if b is None else W.as_f64(b), act, None if r is None else W.as_f64(r), alpha, K,
                  "linear_mx %dx%dx%d" % (M, N, K))


@pytest.mark.parametrize("M,F,K", [(1, 128, 32), (1, 1536, 4096), (5, 256, 96), (16, 384, 160), (33, 640, 1056), (77, 1024, 512),
                                   (129, 256, 320), (300, 1152, 1024), (1000, 2304, 672), (2500, 3200, 512),
                                   (300, 2048, 4096), (700, 1152, 3104)])
def test_linear_swiglu_mx(cuda_device, M, F, K):
    rng = np.random.default_rng(M + F + K)
    x, xv = _mx_operand(rng, M, K, 1.0, cuda_device)
    w, wv = _mx_operand(rng, 2 * F, K, K ** -0.5, cuda_device)
    b = _bf(0.1 * rng.standard_normal(2 * F))
    ws = qi.new_workspace(256, cuda_device)
    got = qi.linear_swiglu_mx(x, w, b.to(cuda_device), workspace=ws)
    check_status(ws)
    bv = W.as_f64(b)
    y = X.linear_mx(xv, wv, bv).reshape(M, -1, 2, 128)
    acc = (_acc_bound(xv, wv, K) + 2.0 ** -23 * np.abs(y.reshape(M, -1))).reshape(M, -1, 2, 128)
    g, u = y[:, :, 0], y[:, :, 1]
    ref = X.swiglu(xv, wv, bv)
    s = np.abs(g / (1 + np.exp(-g)))
    # accumulation of g and u carried through silu(g) * u, and the exponential as above
    slack = (1.11 * np.abs(u) * acc[:, :, 0] + s * acc[:, :, 1] + acc[:, :, 0] * acc[:, :, 1]
             + s * np.abs(u) * (8 + 4 * np.abs(g)) * 2.0 ** -23 + 1e-30).reshape(M, F)
    _check_rounded(got, ref, 0.0, slack)


def test_exact_products_read_every_scale(cuda_device):
    """Operands of powers of two with a different scale in every (row, block): the sums are exact, so any
    scale taken from a wrong row, block or tile shows."""
    rng = np.random.default_rng(11)
    for M, N, K in ((200, 264, 416), (300, 520, 1024), (2100, 1032, 288), (9, 392, 672)):
        ex, ew = rng.integers(-3, 4, (M, K // 32)), rng.integers(-3, 4, (N, K // 32))
        xv = np.ldexp(rng.choice([-1.0, 1.0], (M, K)), np.repeat(ex, 32, 1))
        wv = np.ldexp(rng.choice([-1.0, 1.0], (N, K)), np.repeat(ew, 32, 1))
        # exactly representable fp32 sums: K <= 1024 terms of 2^-6 .. 2^6
        x, w = qi.mx_quantize(_bf(xv).to(cuda_device)), qi.mx_quantize(_bf(wv).to(cuda_device))
        (got,) = qi.linear_mx(x, w)
        want = torch.from_numpy(xv @ wv.T).to(torch.float32).to(BF)
        assert torch.equal(got.cpu(), want), (M, N, K)


def test_more_token_tiles_than_a_grid_axis(cuda_device):
    """Eight million rows into four segments of eight columns: one 64-byte box holds them all.  The rows repeat, so
    the result of the first 1024, checked on their own, must repeat too."""
    rng = np.random.default_rng(14)
    M, K, N = 128 * 65535 + 1, 32, 32
    x, xv = _mx_operand(rng, 1024, K, 1.0, cuda_device)
    w, wv = _mx_operand(rng, N, K, K ** -0.5, cuda_device)
    few = qi.linear_mx(x, w, n_out=4)
    _check_linear(few, xv, wv, None, "none", None, 1.0, K)
    q = x.q.view(torch.uint8).repeat(8193, 1)[:M].contiguous().view(torch.float8_e4m3fn)
    scale = x.scale.view(torch.uint8).repeat(8192, 1, 1, 1, 1).view(torch.float8_e8m0fnu)
    outs = qi.linear_mx(qi.MXTensor(q, scale), w, n_out=4)
    for o, f in zip(outs, few):
        whole = (M // 1024) * 1024
        assert bool((o[:whole].view(-1, 1024, 8) == f).all()) and torch.equal(o[whole:], f[: M - whole])


@pytest.mark.parametrize("M", [40, 300, 1100])
def test_products_leave_what_lies_behind_alone(cuda_device, M):
    """Rows behind the last token, in values and scales, stay as they were."""
    rng = np.random.default_rng(M)
    dev, K, N = cuda_device, 512, 4096
    x, _ = _mx_operand(rng, M, K, 1.0, dev)
    w, _ = _mx_operand(rng, N, K, K ** -0.5, dev)
    out = torch.full((M + 5, N), 7.0, dtype=BF, device=dev)
    qi.linear_mx(x, w, out=[out[:M]])
    assert bool((out[M:] == 7).all()) and not bool((out[:M] == 7).all(1).any())
    q = torch.full((M + 5, N // 2), 9, dtype=torch.uint8, device=dev)
    groups = (M + 127) // 128
    scale = torch.full((groups, N // 256, 32, 4, 4), 0xAB, dtype=torch.uint8, device=dev)
    qi.linear_swiglu_mx(x, w, out=qi.MXTensor(q[:M].view(torch.float8_e4m3fn), scale.view(torch.float8_e8m0fnu)))
    assert bool((q[M:] == 9).all())
    s = scale.cpu().numpy()
    r, b = np.arange(groups * 128)[:, None], np.arange(N // 64)[None, :]
    full = s[r // 128, b // 4, r % 32, r % 128 // 32, b % 4]
    assert (full[M:] == 0xAB).all() and (full[:M] != 0xAB).all()


def test_linear_mx_residual_in_place(cuda_device):
    rng = np.random.default_rng(12)
    for M, N, K in ((40, 264, 256), (900, 512, 256), (400, 4104, 4096), (3000, 2056, 512), (5000, 4096, 320)):
        x, _ = _mx_operand(rng, M, K, 1.0, cuda_device)
        w, _ = _mx_operand(rng, N, K, K ** -0.5, cuda_device)
        r = _bf(rng.standard_normal((M, N))).to(cuda_device)
        (want,) = qi.linear_mx(x, w, residual=r, alpha=0.5)
        (got,) = qi.linear_mx(x, w, residual=r, alpha=0.5, out=[r])
        assert got is r and torch.equal(r, want)


def test_non_finite_scales_reach_their_rows_only(cuda_device):
    rng = np.random.default_rng(13)
    for M in (6, 600):
        xb = _act(rng, M, 256)
        xb[2, 100] = float("nan")
        x = qi.mx_quantize(xb.to(cuda_device))
        w, _ = _mx_operand(rng, 264, 256, 0.06, cuda_device)
        (y,) = qi.linear_mx(x, w)
        bad = torch.isnan(y).all(1).cpu()
        assert bool(bad[2]) and int(torch.isnan(y).any(1).sum()) == 1
        (g,) = qi.linear_mx(x, w, act="gelu")
        assert bool(torch.isnan(g[2]).all()) and bool(torch.isfinite(g[3:]).all())


def test_activation_tails(cuda_device):
    """Large products: silu and gelu go to y or to 0 without a NaN."""
    x = torch.zeros(4, 32, dtype=BF)
    x[0, 0], x[1, 0], x[2, 0], x[3, 0] = 100.0, -100.0, 1e6, -1e6
    w = torch.zeros(8, 32, dtype=BF)
    w[:, 0] = 1.0
    xm, wm = qi.mx_quantize(x.to(cuda_device)), qi.mx_quantize(w.to(cuda_device))
    v = X.values(*_read(xm))[:, 0]
    for act in ("silu", "gelu_tanh"):
        (y,) = qi.linear_mx(xm, wm, act=act)
        y = y.double().cpu().numpy()
        assert np.allclose(y[0], v[0], rtol=2 ** -8) and np.allclose(y[2], v[2], rtol=2 ** -8)
        assert (np.abs(y[1]) <= 1e-30).all() and (np.abs(y[3]) <= 1e-30).all()


# ---------------------------------------------------- as a user calls them

def _layer(dev, rng, M, D, F):
    """One feed-forward half of a block in MX form: add + norm -> gated projection -> down projection."""
    bf = lambda a: _bf(a).to(dev)
    h, d, nw = bf(rng.standard_normal((M, D))), bf(0.3 * rng.standard_normal((M, D))), bf(1 + 0.1 * rng.standard_normal(D))
    w_gu = qi.mx_quantize(qi.interleave_gate_up(bf(rng.standard_normal((2 * F, D)) * D ** -0.5)))
    b_gu, b_d = bf(0.02 * rng.standard_normal(2 * F)), bf(0.02 * rng.standard_normal(D))
    w_d = qi.mx_quantize(bf(rng.standard_normal((D, F)) * F ** -0.5))
    ws = qi.new_workspace(256, dev)
    a, m = qi.mx_empty((M, D), dev), qi.mx_empty((M, F), dev)
    s, out = torch.empty_like(h), torch.empty_like(h)

    def run():
        qi.rmsnorm_mx(h, nw, 1e-6, delta=d, sum_out=s, out=a)
        qi.linear_swiglu_mx(a, w_gu, b_gu, out=m, workspace=ws)
        qi.linear_mx(m, w_d, b_d, residual=s, out=[out], workspace=ws)

    return dict(h=h, d=d, nw=nw, w_gu=w_gu, b_gu=b_gu, w_d=w_d, b_d=b_d, ws=ws, a=a, m=m, s=s, out=out, run=run)


@pytest.mark.parametrize("M", [1, 50, 600, 1300])
def test_feed_forward_chain(cuda_device, M):
    """Every step against the oracle on what the step before it wrote, then the captured chain bit for bit."""
    rng = np.random.default_rng(M)
    D, F = 512, 768
    L = _layer(cuda_device, rng, M, D, F)
    L["run"]()
    check_status(L["ws"])
    f = W.as_f64
    assert torch.equal(L["s"], (L["h"].float() + L["d"].float()).to(BF))
    _check_rounded(L["a"], X.rms_norm(f(L["s"]), f(L["nw"]), 1e-6), (D / 64 + 10) * 2.0 ** -24)
    a, w, m, wd = (X.values(*_read(L[k])) for k in ("a", "w_gu", "m", "w_d"))
    ref = X.swiglu(a, w, f(L["b_gu"]))
    _check_rounded(L["m"], ref, 2.0 ** -16, 1e-5)
    _check_linear([L["out"]], m, wd, f(L["b_d"]), "none", f(L["s"]), 1.0, F)

    eager = [L["out"].clone(), L["m"].q.view(torch.uint8).clone(), L["s"].clone()]
    side = torch.cuda.Stream(cuda_device)
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        L["run"]()
    L["out"].zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(L["out"], eager[0]) and torch.equal(L["m"].q.view(torch.uint8), eager[1])
    L["d"].mul_(0.5)                                     # a replay reads the current contents
    graph.replay()
    torch.cuda.synchronize()
    replayed = L["out"].clone()
    L["run"]()
    assert torch.equal(L["out"], replayed) and not torch.equal(replayed, eager[0])


def test_two_streams_one_workspace_header(cuda_device):
    """Calls on two streams at once with workspaces of their own, and repeated calls: the same bits."""
    rng = np.random.default_rng(21)
    layers = [_layer(cuda_device, rng, M, 512, 640) for M in (48, 1100)]
    want = []
    for L in layers:
        L["run"]()
        want.append(L["out"].clone())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(cuda_device) for _ in layers]
    for _ in range(20):
        for L, st in zip(layers, streams):
            with torch.cuda.stream(st):
                L["run"]()
    torch.cuda.synchronize()
    for L, w in zip(layers, want):
        assert torch.equal(L["out"], w)
        check_status(L["ws"])


def test_every_kernel_at_once(cuda_device):
    """Few and many tokens, whole and split over clusters, on four streams at a time: CTAs that hold tensor memory and
    wait for others of their cluster share SMs with one another, and every call gives the same bits."""
    rng = np.random.default_rng(23)
    layers = [_layer(cuda_device, rng, M, 1024, 2048) for M in (1, 48, 400, 2300)]
    want = []
    for L in layers:
        L["run"]()
        want.append((L["out"].clone(), L["m"].q.view(torch.uint8).clone()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(cuda_device) for _ in layers]
    for i in range(60):
        for k in range(len(layers)):
            with torch.cuda.stream(streams[k]):
                for _ in range(1 + (i + k) % 3):
                    layers[k]["run"]()
    torch.cuda.synchronize()
    for L, (out, q) in zip(layers, want):
        assert torch.equal(L["out"], out) and torch.equal(L["m"].q.view(torch.uint8), q)
        check_status(L["ws"])


def test_captured_across_streams(cuda_device):
    """A capture that forks to a second stream and joins again, with copies and other kernels between the calls;
    two graphs of it share one workspace."""
    rng = np.random.default_rng(24)
    dev, M, D = cuda_device, 300, 512
    x, d = _act(rng, M, D).to(dev), _act(rng, M, D).to(dev)
    nw = torch.ones(D, dtype=BF, device=dev)
    w = qi.mx_quantize((_act(rng, 1024, D).float() * 0.05).to(BF).to(dev))
    ws = qi.new_workspace(256, dev)
    a, b, copy = qi.mx_empty((M, D), dev), qi.mx_empty((M, D), dev), torch.empty_like(x)
    h, ya, yb = torch.empty_like(x), torch.empty(M, 1024, dtype=BF, device=dev), torch.empty(M, 1024, dtype=BF, device=dev)
    other = torch.cuda.Stream(dev)

    def run():
        here = torch.cuda.current_stream()
        copy.copy_(x)
        qi.mx_quantize(copy, out=a)
        other.wait_stream(here)
        with torch.cuda.stream(other):
            qi.rmsnorm_mx(copy, nw, 1e-6, delta=d, sum_out=h, out=b)
            qi.linear_mx(b, w, out=[yb], workspace=ws)
            h.mul_(2)
        qi.linear_mx(a, w, act="silu", out=[ya], workspace=ws)
        here.wait_stream(other)
        qi.linear_mx(b, w, residual=ya, out=[ya], workspace=ws)

    run()
    torch.cuda.synchronize()
    want = [t.clone() for t in (ya, yb, h)]
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        graphs.append(g)
    for g in graphs * 3:
        for t in (ya, yb, h):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(t, v) for t, v in zip((ya, yb, h), want))
    check_status(ws)


def test_leading_dimensions_and_defaults(cuda_device):
    rng = np.random.default_rng(22)
    x = _act(rng, 6 * 50, 256).reshape(6, 50, 256).to(cuda_device)
    w = qi.mx_quantize(_act(rng, 384, 256).to(cuda_device))
    mx = qi.mx_quantize(x)
    flat = qi.mx_quantize(x.reshape(300, 256))
    assert torch.equal(mx.scale.view(torch.uint8), flat.scale.view(torch.uint8))
    outs = qi.linear_mx(mx, w, n_out=3)
    assert [tuple(o.shape) for o in outs] == [(6, 50, 128)] * 3
    (one,) = qi.linear_mx(flat, w)
    assert torch.equal(torch.cat(outs, -1).reshape(300, 384), one)
    empty = qi.linear_mx(qi.mx_empty((0, 256), cuda_device), w)
    assert empty[0].shape == (0, 384)


def test_binding_refuses(cuda_device):
    dev = cuda_device
    x = torch.zeros(4, 64, dtype=BF, device=dev)
    mx = qi.mx_quantize(x)
    w = qi.mx_quantize(torch.zeros(256, 64, dtype=BF, device=dev))
    bad = [lambda: qi.mx_quantize(x.float()), lambda: qi.mx_quantize(x.t()), lambda: qi.mx_quantize(x[:, :48].contiguous()),
           lambda: qi.mx_quantize(x, out=qi.mx_empty((5, 64), dev)), lambda: qi.mx_quantize(x, out=(mx.q, mx.scale)),
           lambda: qi.rmsnorm_mx(x, x[0], 1e-6, sum_out=x), lambda: qi.rmsnorm_mx(x, x[0].float(), 1e-6),
           lambda: qi.rmsnorm_mx(x, x[0], -1.0), lambda: qi.rmsnorm_mx(x, x[0], 1e-6, delta=x[:2]),
           lambda: qi.linear_mx(x, w), lambda: qi.linear_mx(mx, w, act="relu"), lambda: qi.linear_mx(mx, w, n_out=3),
           lambda: qi.linear_mx(mx, w, n_out=2, residual=torch.zeros(4, 256, dtype=BF, device=dev)),
           lambda: qi.linear_mx(mx, qi.mx_empty((256, 96), dev)), lambda: qi.linear_mx(mx, w, bias=x[0]),
           lambda: qi.linear_mx(mx, w, alpha=float("nan")),
           lambda: qi.linear_mx(qi.MXTensor(mx.q, mx.scale.view(torch.uint8)), w),
           lambda: qi.linear_mx(mx, w, workspace=torch.zeros(100, dtype=torch.uint8, device=dev)),
           lambda: qi.linear_mx(mx, w, workspace=torch.zeros(256, dtype=torch.uint8)),
           lambda: qi.linear_swiglu_mx(mx, w, workspace=torch.zeros(256, dtype=torch.uint8)),
           lambda: qi.mx_quantize(x.cpu()), lambda: qi.linear_mx(qi.mx_empty((4, 64), "cpu"), w),
           lambda: qi.linear_mx(mx, qi.mx_empty((256, 64), "cpu")),
           lambda: qi.linear_swiglu_mx(mx, qi.mx_empty((128, 64), dev)),
           lambda: qi.linear_swiglu_mx(mx, w, out=qi.mx_empty((4, 256), dev))]
    for i, call in enumerate(bad):
        with pytest.raises(qb.QI21Error):
            call()
            pytest.fail("case %d was accepted" % i)
