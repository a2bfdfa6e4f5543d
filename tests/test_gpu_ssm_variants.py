"""The kernels that the causal convolution's and the scan's calls choose between (long
runs, types, taps, numbers of states, token steps with and without each option), and
how parameters' gradients are added up over workgroups."""
import pytest
import torch

from state_passing_amd import linrec

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32 = torch.float32


def whole(g, most, *shape):
    """Whole numbers 0 .. most in fp32 on the GPU."""
    return torch.randint(0, most + 1, shape, generator=g).float().to(DEV)


def test_convolution_sums_over_workgroups_are_exact():
    """dw and dbias of whole numbers: a workgroup's 1024 tokens add up to less than 2^24, exactly, so what
    comes is the exact sum over the 128 workgroups, rounded once (added in fp32 they would round at 2^24)."""
    g, T, C, K = torch.Generator().manual_seed(1), 131072, 8, 4
    d = linrec._CONV(1, T, C, K, 0, linrec.F32, linrec.F32)
    assert linrec._lib().linrec_conv_bwd_workspace_bytes(d) == 4 * ((K - 1) * C + 128 * (K + 1) * C)
    x, dy, w = whole(g, 1, 1, T, C), whole(g, 2 ** 14 - 1, 1, T, C), torch.randn(C, K, generator=g).to(DEV)
    _, dw, dbias, _ = linrec.conv_bwd(x, w, torch.zeros(C, device=DEV), None, dy, act=None)
    x, dy = x[0].cpu().double(), dy[0].cpu().double()
    want = torch.stack([(dy[K - 1 - k:] * x[:T - (K - 1 - k)]).sum(0) for k in range(K)], 1)
    assert want.min() > 2 ** 25
    assert torch.equal(dw.cpu(), want.float()) and torch.equal(dbias.cpu(), dy.sum(0).float())


def test_scan_sums_over_segments_are_exact():
    """dD and ddt_bias likewise: gates of exp(-1000) = 0 leave ddt = x dy (c and b pick one state), whole numbers
    whose sum over a segment's 128 tokens is exact; 256 segments."""
    g, T, C, N = torch.Generator().manual_seed(2), 32768, 64, 16
    d = linrec._SCAN(1, T, C, N, 1, 0, linrec.F32, linrec.F32)
    assert linrec._lib().linrec_scan_fwd_workspace_bytes(d) == 4 * 256 * C * (N + 1)
    x, dy = whole(g, 1, 1, T, C), whole(g, 2 ** 17 - 1, 1, T, C)
    one = torch.zeros(1, 1, T, N, device=DEV)
    one[..., 3] = 1
    A, ones = torch.full((C, N), -1000.0, device=DEV), torch.ones(C, device=DEV)
    first = (x, torch.zeros_like(x), A, one, one)
    rest = dict(D=ones, dt_bias=ones, softplus=False)
    r = linrec.scan_bwd(*first, linrec.scan_fwd(*first, save=True, **rest)[2], dy, **rest)
    want = (x[0].cpu().double() * dy[0].cpu().double()).sum(0)
    assert want.min() > 2 ** 29
    assert torch.equal(r.dD.cpu(), want.float()) and torch.equal(r.ddt_bias.cpu(), want.float())
    assert (r.dA == 0).all()
