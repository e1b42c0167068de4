"""The MX oracle against facts that do not come from its own formulas, and the MX entry
points' argument checks (no GPU)."""

import ctypes
import os

import numpy as np
import pytest
import torch

from diffusion_transformer_joint_axial_b200 import _binding as qb
from oracle import mx_oracle as X


def test_e4m3_codes_are_torchs():
    codes = np.arange(256, dtype=np.uint8)
    theirs = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(X.e4m3_decode(codes), theirs, equal_nan=True)


def test_e4m3_round_is_nearest_even_on_the_grid():
    grid = np.sort(X.e4m3_decode(np.array([c for c in range(128) if c != 127])))
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.uniform(-448, 448, 2000), np.exp(rng.uniform(-9, 6, 2000)), grid, (grid[1:] + grid[:-1]) / 2])
    got = X.e4m3_round(v)
    full = np.concatenate([-grid, grid])
    near = np.abs(v[:, None] - full[None, :]).min(1)
    assert np.array_equal(np.abs(got - v), near)
    mid = (grid[1:] + grid[:-1]) / 2                     # ties go to the even code
    code = np.searchsorted(grid, X.e4m3_round(mid))
    assert np.all(code % 2 == 0)
    t = torch.from_numpy(v).float()
    assert np.array_equal(X.e4m3_round(t.double().numpy()), t.to(torch.float8_e4m3fn).double().numpy())


@pytest.mark.parametrize("top,e", [(448.0, 0), (np.nextafter(448.0, 1e9), 1), (224.0, -1), (1.0, -8), (1.75, -8), (1.76, -7),
                                   (0.0, -127), (2.0 ** -133, -127), (3e38, 120)])
def test_block_exponents(top, e):
    x = np.zeros((1, 32))
    x[0, 7] = -top
    assert X.block_exponents(x)[0, 0] == e
    q, byte = X.quantize(x)
    assert byte[0, 0] == e + 127 and np.abs(q).max() <= 448


def test_non_finite_blocks():
    x = np.ones((1, 96))
    x[0, 3], x[0, 70] = np.nan, -np.inf
    q, byte = X.quantize(x)
    assert list(byte[0] == 255) == [True, False, True]
    v = X.values(q, byte)
    assert np.isnan(v[0, :32]).all() and (v[0, 32:64] == 1).all() and np.isnan(v[0, 64:]).all()


def test_untile_follows_the_byte_rule():
    R, K = 300, 288
    flat = np.random.default_rng(1).integers(0, 255, qb.load_library().qi21_mx_scale_size(R, K)).astype(np.uint8)
    got = X.untile(flat.reshape(3, 3, 32, 4, 4), R, K)
    for r, b in ((0, 0), (31, 3), (32, 0), (127, 8), (128, 4), (299, 8), (200, 7)):
        tile = (r // 128) * 3 + b // 4
        assert got[r, b] == flat[tile * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4]


def test_gelu_and_swiglu_pins():
    y = np.linspace(-9, 9, 181)
    theirs = torch.nn.functional.gelu(torch.from_numpy(y), approximate="tanh").numpy()
    assert np.allclose(X.gelu_tanh(y), theirs, atol=1e-15)
    rng = np.random.default_rng(2)
    wg, wu, x = rng.standard_normal((256, 32)), rng.standard_normal((256, 32)), rng.standard_normal((3, 32))
    il = qb.interleave_gate_up(torch.from_numpy(np.concatenate([wg, wu]))).numpy()
    g = x @ wg.T
    assert np.allclose(X.swiglu(x, il), g / (1 + np.exp(-g)) * (x @ wu.T), atol=1e-12)


# ---------------------------------------------------------------- refusals

@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(qb.LIB_PATH):
        pytest.skip("libqi21.so not built")
    return qb.load_library()


BAD = qb.QI21_ERR_INVALID_ARG
p = ctypes.c_void_p


def test_scale_size(lib):
    assert lib.qi21_mx_scale_size(1, 32) == 512
    assert lib.qi21_mx_scale_size(128, 128) == 512
    assert lib.qi21_mx_scale_size(129, 160) == 4 * 512
    assert lib.qi21_mx_scale_size(0, 32) == 0 and lib.qi21_mx_scale_size(-1, 32) == 0


def test_quantize_rejects(lib):
    f = lambda M=4, K=64, x=16, q=16, s=16: lib.qi21_mx_quantize(M, K, p(x), p(q), p(s), None)
    assert f(K=48) == BAD and f(K=0) == BAD and f(M=-1) == BAD and f(M=1 << 31) == BAD and f(K=(1 << 24) + 32) == BAD
    assert f(x=0) == BAD and f(q=24) == BAD and f(s=20) == BAD
    assert f(M=0, x=0) == qb.QI21_OK


def test_rmsnorm_mx_rejects(lib):
    f = lambda M=4, D=64, x=16, d=0, w=16, eps=1e-6, h=0, q=16, s=16: lib.qi21_rmsnorm_mx(
        M, D, p(x), p(d), p(w), ctypes.c_float(eps), p(h), p(q), p(s), None)
    assert f(D=40) == BAD and f(D=0) == BAD and f(M=-1) == BAD
    assert f(eps=-1.0) == BAD and f(eps=float("nan")) == BAD and f(eps=float("inf")) == BAD
    assert f(d=16) == BAD and f(h=16) == BAD                     # delta and sum come together
    assert f(d=24, h=16) == BAD and f(d=16, h=24) == BAD
    assert f(x=0) == BAD and f(w=0) == BAD and f(q=0) == BAD and f(s=8) == BAD
    assert f(M=0, x=0) == qb.QI21_OK


def _outs(*v):
    return (p * len(v))(*v)


def test_linear_mx_rejects(lib):
    def f(M=4, N=96, K=64, x=16, xs=16, w=16, ws=16, b=0, act=0, r=0, alpha=1.0, out=_outs(16, 16, 16, 16), n=1, wk=256,
          wb=256):
        return lib.qi21_linear_mx(M, N, K, p(x), p(xs), p(w), p(ws), p(b), act, p(r), ctypes.c_float(alpha), out, n,
                                  p(wk), wb, None)
    assert f(n=0) == BAD and f(n=5) == BAD and f(N=36, n=3) == BAD and f(N=100) == BAD
    assert f(K=48) == BAD and f(K=0) == BAD and f(M=-1) == BAD and f(N=-8) == BAD
    assert f(act=3) == BAD and f(act=-1) == BAD
    assert f(r=16, n=2) == BAD and f(r=24) == BAD
    assert f(alpha=float("nan")) == BAD and f(alpha=float("inf")) == BAD
    for k in ("x", "xs", "w", "ws", "wk"):
        assert f(**{k: 0}) == BAD and f(**{k: 20}) == BAD, k
    assert f(b=40) == BAD and f(out=None) == BAD and f(out=_outs(16, 20), n=2) == BAD and f(wb=100) == BAD
    assert f(M=0, x=0) == qb.QI21_OK and f(N=0, w=0) == qb.QI21_OK


def test_linear_swiglu_mx_rejects(lib):
    def f(M=4, N=256, K=64, x=16, xs=16, w=16, ws=16, b=0, q=16, s=16, wk=256, wb=256):
        return lib.qi21_linear_swiglu_mx(M, N, K, p(x), p(xs), p(w), p(ws), p(b), p(q), p(s), p(wk), wb, None)
    assert f(N=128) == BAD and f(N=384) == BAD and f(K=16) == BAD and f(M=-1) == BAD
    for k in ("x", "xs", "w", "ws", "q", "s", "wk"):
        assert f(**{k: 0}) == BAD and f(**{k: 20}) == BAD, k
    assert f(b=40) == BAD and f(wb=255) == BAD
    assert f(M=0, x=0) == qb.QI21_OK


def test_binding_needs_a_device_or_checks_first():
    if torch.cuda.is_available():
        pytest.skip("covered by the GPU tests")
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(qb.QI21Error):
        qb.mx_quantize(x)
    with pytest.raises(qb.QI21Error):
        qb.mx_empty((4, 40), "cpu")
    t = qb.mx_empty((2, 3, 160), "cpu")
    assert t.q.shape == (2, 3, 160) and t.scale.shape == (1, 2, 32, 4, 4)
    assert int(t.scale.view(torch.uint8).sum()) == 0
