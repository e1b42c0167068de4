"""The MX products whose CTAs read or signal one another (K split over a cluster, CTA pairs): calls in which some rows
and features do not exist, so that some warps of a cluster have nothing to store and leave early."""

import pytest
import torch

import diffusion_transformer_joint_axial_b200 as qi

from parity import check_status

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _operand(gen, R, K, dev):
    return qi.mx_quantize(torch.randn(R, K, generator=gen, device=dev).to(BF))


@pytest.mark.parametrize("M,N,K,gated", [
    # few tokens, K in four parts
    (1, 136, 4096, False),     # eight live features in the second tile
    (33, 264, 7456, False),    # ragged tokens and features
    (16, 512, 4096, True),
    # two CTA pairs, each with half of K
    (257, 4096, 4096, False),  # one live row in the second token tile: a CTA without any
    (300, 4040, 4096, False),  # a chunk of columns that ends inside
    (300, 3976, 4096, False),  # chunks that do not exist
    (300, 4096, 4096, True),
    (385, 2560, 4096, True)])
def test_nobody_leaves_while_its_sums_are_read(cuda_device, M, N, K, gated):
    assert qi.mx_plan(M, N, K, gated=gated) == (("few", 4) if M < 100 else ("pairs_split", 2))
    _same_bits_in_many_calls(cuda_device, M, N, K, gated)


@pytest.mark.parametrize("M,N,K,gated", [
    (300, 512, 160, True),     # pairs of one tile each, two stages of K
    (900, 512, 96, True),
    (300, 1024, 672, True),    # one stage more than there are slots for
    (700, 1024, 416, True),
    (2500, 6400, 160, True),   # several tiles a pair, one pair fewer tiles than another
    (5000, 2056, 1056, False)])
def test_pairs_leave_behind_every_signal(cuda_device, M, N, K, gated):
    """Pairs whose last signals to the other CTA (a stage or an accumulator that is free) nothing waits for in turn."""
    assert qi.mx_plan(M, N, K, gated=gated) == ("pairs", 1)
    _same_bits_in_many_calls(cuda_device, M, N, K, gated)


def _same_bits_in_many_calls(cuda_device, M, N, K, gated):
    """The same bits in every one of many calls, on two streams at a time, so that the shared memory of a CTA that
    left is written by another at once."""
    dev = cuda_device
    gen = torch.Generator(device=dev).manual_seed(M + N)
    x, w = _operand(gen, M, K, dev), _operand(gen, N, K, dev)
    bits = lambda t: (t.q if gated else t[0]).view(torch.uint8)

    def call(ws, out=None):
        if gated:
            return qi.linear_swiglu_mx(x, w, out=out, workspace=ws)
        return qi.linear_mx(x, w, out=out, workspace=ws)

    ws = [qi.new_workspace(256, dev) for _ in range(2)]
    want = bits(call(ws[0])).clone()
    outs = [call(w_) for w_ in ws]
    streams = [torch.cuda.Stream(dev) for _ in ws]
    torch.cuda.synchronize()
    bad = torch.zeros(2, dtype=torch.int64, device=dev)
    for _ in range(50):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                call(ws[i], outs[i])
                call(ws[i], outs[i])
                bad[i] += (bits(outs[i]) != want).sum()
    torch.cuda.synchronize()
    assert bad.tolist() == [0, 0]
    for w_ in ws:
        check_status(w_)
