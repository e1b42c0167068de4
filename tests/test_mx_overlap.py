"""MX calls whose results would overwrite what they read (other tiles read it again), or one another, are refused; a
norm's sum in x or delta and a product in its residual are not."""

import ctypes
import os

import pytest
import torch

from diffusion_transformer_joint_axial_b200 import _binding as qb

if not os.path.exists(qb.LIB_PATH) or torch.cuda.is_available():
    pytest.skip("needs libqi21.so, and no GPU: the addresses are not real", allow_module_level=True)

p = ctypes.c_void_p
M, N, K = 300, 512, 256                     # x and q: 76 800 bytes and 6 scale tiles; out: 307 200 bytes
X, XS, W_, WS, B, Q, QS, R, WK = (0x100000 * i for i in range(1, 10))
MX = M * K


def _gated(q=Q, s=QS):
    return qb.load_library().qi21_linear_swiglu_mx(M, N, K, p(X), p(XS), p(W_), p(WS), p(B), p(q), p(s), p(WK), 256, None)


def _linear(*out, r=None):
    ptrs = (p * len(out))(*out)
    return qb.load_library().qi21_linear_mx(M, N, K, p(X), p(XS), p(W_), p(WS), p(B), 0, p(r), ctypes.c_float(1), ptrs,
                                            len(out), p(WK), 256, None)


def _norm(x=X, d=None, h=None, q=Q, s=QS):
    return qb.load_library().qi21_rmsnorm_mx(M, K, p(x), p(d), p(W_), ctypes.c_float(1e-6), p(h), p(q), p(s), None)


def _quantize(q=Q, s=QS):
    return qb.load_library().qi21_mx_quantize(M, K, p(X), p(q), p(s), None)


REFUSED = {
    "gated q": [lambda a=a: _gated(q=a) for a in (X, X + 16, X + MX - 16, X - MX + 16, W_ + 512, XS, B + 16, QS + 16)],
    "gated scale": [lambda a=a: _gated(s=a) for a in (XS, XS + 3056, XS - 3056, WS + 1024, X, Q + 32)],
    "linear": [lambda a=a: _linear(a) for a in (X, X + MX - 16, X - 16, W_, XS + 16, WS, B)],
    "segments": [lambda: _linear(Q, Q), lambda: _linear(Q, Q + 16), lambda: _linear(Q, R, Q + 76800 - 16, QS)],
    "beside the residual": [lambda: _linear(R + 16, r=R), lambda: _linear(R - 16, r=R)],
    "norm": [lambda: _norm(q=X), lambda: _norm(s=X + 16), lambda: _norm(q=W_), lambda: _norm(q=QS - 16),
             lambda: _norm(d=B, h=X + 16), lambda: _norm(d=B, h=B - 16), lambda: _norm(d=B, h=R, q=R + 16),
             lambda: _norm(d=B, h=W_)],
    "quantize": [lambda: _quantize(q=X), lambda: _quantize(q=X + 2 * MX - 16), lambda: _quantize(s=X + 16),
                 lambda: _quantize(q=QS - 16)],
}


@pytest.mark.parametrize("what", REFUSED)
def test_overlap_is_refused(what):
    for i, call in enumerate(REFUSED[what]):
        assert call() == qb.QI21_ERR_INVALID_ARG, i
        assert b"overlap" in qb.load_library().qi21_last_error(), i


def test_neighbours_and_places_are_not_refused():
    """Accepted by the checks: without a device the launch itself fails then."""
    for call in (lambda: _gated(q=X + MX), lambda: _gated(q=X - MX), lambda: _gated(s=XS + 3072), lambda: _linear(R, r=R),
                 lambda: _linear(Q, Q + 153600), lambda: _norm(d=B, h=X), lambda: _norm(d=B, h=B), lambda: _norm(x=B, d=B, h=B),
                 lambda: _quantize(q=X + 2 * MX)):
        assert call() == qb.QI21_ERR_CUDA
