"""Base products of few rows a matrix: of up to 8, x is held in fixed point of 256 values each.

Bounds: with m the largest magnitude of x in a block of 256 values and 2^E <= m < 2^(E+1), a value of the block is off by
at most half a unit, 2^(E-22) <= 2^-22 m, and not at all if its magnitude is 2^(E-14) or more.  So an output is off by
at most sum over blocks of 2^-22 m_block sum |s (q - z)| beside the fp32 sums' 2 d_in 2^-23 S (S = sum |s (q - z) x|)."""
import numpy as np
import pytest
import torch

import segmented_rank_gemm_sgmv_b200 as sg
from expert_cases import dense64, f64, rounded, weights4

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


def allowed(w, x, d_in):
    big = np.abs(x) @ np.abs(w).T
    slack = 2 * d_in * 2.0 ** -23 * big
    for a in range(0, d_in, 256):
        slack += 2.0 ** -22 * np.abs(x[:, a:a + 256]).max(1)[:, None] * np.abs(w[:, a:a + 256]).sum(1)[None, :]
    return slack


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 8, 9, 12, 16])
@pytest.mark.parametrize("spread", [0, 10, 40])
def test_values_of_many_binades(T, spread):
    """x over 2 * spread binades, one block of zeros, outliers: within the bound of each block's largest value."""
    g = torch.Generator("cuda").manual_seed(T + spread)
    d_in, d_out = 1120, 150
    codes, scales, z = weights4(g, (), d_out, d_in, 32, T % 2 == 0, F, False)
    x = torch.randn(T, d_in, generator=g, device="cuda") * torch.exp2(spread * (2 * torch.rand(T, d_in, generator=g, device="cuda") - 1))
    x[:, 256:512] = 0
    x[:, 700] *= 1000
    x = x.to(BF)
    w = dense64(codes, scales, z)
    ref, slack = f64(x) @ w.T, allowed(w, f64(x), d_in)
    y = torch.empty(T, d_out, device="cuda")
    sg.base_product(x, codes, scales, y, zeros=z)
    assert (np.abs(f64(y) - ref) <= slack + 2.0 ** -24 * (np.abs(ref) + slack)).all()


@pytest.mark.parametrize("T", [1, 7, 16])
def test_values_within_fourteen_binades_are_exact(T):
    """Powers of two over 14 binades in a block, scales of 1: every product and sum is exact, and so is y."""
    g = torch.Generator("cuda").manual_seed(T)
    d_in, d_out = 512, 70
    codes = torch.randint(0, 256, (d_out, d_in // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.ones(d_out, d_in // 128, device="cuda")
    x = torch.zeros(T, d_in, dtype=BF, device="cuda")
    for t in range(T):                     # one value of each binade 2^0 .. 2^-14 in each block
        for block in range(2):
            at = block * 256 + torch.randperm(256, generator=g, device="cuda")[:15]
            x[t, at] = torch.exp2(-torch.arange(15, device="cuda").float()).to(BF)
    y = torch.empty(T, d_out, device="cuda")
    sg.base_product(x, codes, scales, y)
    assert torch.equal(y.cpu(), rounded(f64(x) @ dense64(codes, scales, None).T, F))


@pytest.mark.parametrize("scale", [2.0 ** -126, 2.0 ** -133, 1e30, 3e38])
def test_extreme_magnitudes(scale):
    """The smallest normal and subnormal values of bf16 and the largest ones; weights of 1, one value a row."""
    codes = torch.full((8, 32), 0x11, dtype=torch.uint8, device="cuda")
    scales = torch.ones(8, 1, device="cuda")
    x = torch.zeros(2, 64, dtype=BF, device="cuda")
    x[0, 3] = scale
    x[1, 60] = -scale
    y = torch.empty(2, 8, device="cuda")
    sg.base_product(x, codes, scales, y)
    assert torch.equal(y, torch.stack([x[0, 3].float().expand(8), x[1, 60].float().expand(8)]))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("T", [1, 3, 16])
def test_rows_that_are_not_finite_follow_the_formula(T, bad):
    """An infinity times a weight of 0 is NaN, others keep its sign; rows without it keep their bits."""
    g = torch.Generator("cuda").manual_seed(T)
    codes, scales, z = weights4(g, (), 40, 640, 64, True, BF, True)
    x = torch.randint(-2, 3, (T, 640), generator=g, device="cuda").to(BF)
    clean = torch.empty(T, 40, device="cuda")
    sg.base_product(x, codes, scales, clean, zeros=z)
    x[T - 1, 300] = bad
    y = torch.empty(T, 40, device="cuda")
    sg.base_product(x, codes, scales, y, zeros=z)
    want = torch.from_numpy(dense64(codes, scales, z)[:, 300]).float().cuda() * bad
    assert torch.equal(y[:-1], clean[:-1]) and torch.equal(torch.nan_to_num(y[-1], nan=7.0), torch.nan_to_num(want, nan=7.0))


@pytest.mark.parametrize("T", [1, 16])
def test_two_streams_at_once(T):
    """Calls that overlap on two streams: each has its own workspace from torch's allocator."""
    g = torch.Generator("cuda").manual_seed(9)
    codes, scales, _ = weights4(g, (), 4096, 2048, 128, False, BF, True)
    xs = [torch.randint(-2, 3, (T, 2048), generator=g, device="cuda").to(BF) for _ in range(2)]
    want = []
    for x in xs:
        y = torch.empty(T, 4096, device="cuda")
        sg.base_product(x, codes, scales, y)
        want.append(y)
    streams = [torch.cuda.Stream() for _ in xs]
    got = [torch.empty_like(w) for w in want]
    torch.cuda.synchronize()
    for _ in range(20):
        for x, y, s in zip(xs, got, streams):
            sg.base_product(x, codes, scales, y, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert sg.check_errors() == 0
