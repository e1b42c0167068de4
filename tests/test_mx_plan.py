"""Which kernel an MX product runs (a host-only query): the sizes that the GPU tests use for each, and its refusals."""

import ctypes
import os

import pytest

import mx_forms as forms
from diffusion_transformer_joint_axial_b200 import _binding as qb

if not os.path.exists(qb.LIB_PATH):
    pytest.skip("libqi21.so not built", allow_module_level=True)


@pytest.mark.parametrize("M,N,K,n_out,act,residual,want", forms.LINEAR)
def test_linear_sizes_reach_their_kernel(M, N, K, n_out, act, residual, want):
    assert qb.mx_plan(M, N, K, act=act, residual=residual, num_sms=forms.SMS) == want


@pytest.mark.parametrize("M,F,K,want", forms.GATED)
def test_gated_sizes_reach_their_kernel(M, F, K, want):
    assert qb.mx_plan(M, 2 * F, K, gated=True, num_sms=forms.SMS) == want


def test_the_ends_of_the_range():
    assert qb.mx_plan(1, 8, 32, num_sms=148) == ("few", 1)
    assert qb.mx_plan(128 * 65535 + 1, 8, 32, num_sms=148) == ("pairs", 1)  # more token tiles than a grid axis
    assert qb.mx_plan(16384, 24576, 4096, gated=True, num_sms=148) == ("pairs", 1)
    for sms in (2, 20, 148):                        # no cluster that does not fit
        kernel, parts = qb.mx_plan(300, 4096, 4096, num_sms=sms)
        assert kernel in qb.MX_KERNELS and parts <= sms


def test_plan_refuses():
    bad = [dict(M=0), dict(N=0), dict(M=-1), dict(K=48), dict(N=100), dict(N=128, gated=True), dict(act="relu"),
           dict(gated=True, act="silu"), dict(gated=True, residual=True), dict(num_sms=-1), dict(num_sms=1)]
    for b in bad:
        with pytest.raises(qb.QI21Error):
            qb.mx_plan(**dict(dict(M=4, N=256, K=64, num_sms=148), **b))
    i = ctypes.c_int32()
    lib = qb.load_library()
    assert lib.qi21_mx_plan(4, 256, 64, 0, 0, 0, 148, None, ctypes.byref(i)) == qb.QI21_ERR_INVALID_ARG
    assert lib.qi21_mx_plan(4, 256, 64, 0, 0, 0, 148, ctypes.byref(i), None) == qb.QI21_ERR_INVALID_ARG
    assert lib.qi21_mx_plan(4, 256, 64, 0, 3, 0, 148, ctypes.byref(i), ctypes.byref(i)) == qb.QI21_ERR_INVALID_ARG
