"""4-bit base products against a plain 64-bit form.

Exact cases: x of small integers and scales that are powers of two make every partial sum a multiple of 2^-3
below 2^20, so that fp32 sums in any order are exact and y has to be the rounded 64-bit value bit for bit.
Real-valued cases (of up to 8 rows also tests/test_base_product_few_rows_gpu.py): with S = sum |s (q - z) x| of an output, each of fewer than 2 d_in additions and scalings in
fp32 is off by at most 2^-23 of a partial result no larger than S (a tensor core may truncate where an fma
rounds), so |y - y64| <= 2 d_in 2^-23 S, plus half a step of y's type."""
import numpy as np
import pytest
import torch

import segmented_rank_gemm_sgmv_b200 as sg
from expert_cases import dense64, f64, order_ref, padded, rounded, weights4

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


def ints(g, rows, d, top, extra=0):
    x = padded(rows, d, BF, extra)
    x.copy_(torch.randint(-top, top + 1, (rows, d), generator=g, device="cuda"))
    return x


def same(y, ref, dtype):
    want = rounded(ref, dtype)
    assert torch.equal(y.cpu(), want), f"{(y.cpu() != want).sum().item()} of {want.numel()} values differ"


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 17, 33, 64, 65, 130])
def test_exact_small(T, zeros, group):
    g = torch.Generator("cuda").manual_seed(T * 7 + group + zeros)
    d_in, d_out = group * 9, 77
    codes, scales, z = weights4(g, (), d_out, d_in, group, zeros, BF if T % 2 else F, True)
    x = ints(g, T, d_in, 2, 8)
    for dt, extra in ((BF, 0), (F, 3)):
        y = padded(T, d_out, dt, extra)
        sg.base_product(x, codes, scales, y, zeros=z)
        same(y, f64(x) @ dense64(codes, scales, z).T, dt)
    sg.check_errors()


@pytest.mark.parametrize("T,d_in,d_out,group", [
    (1, 32, 1, 32), (1, 64, 3, 64), (1, 128, 16, 128), (1, 96, 17, 32), (1, 8192, 1024, 128), (2, 28672, 129, 128),
    (5, 8192, 8192, 64), (3, 160, 1000, 32), (40, 4096, 513, 128), (200, 1024, 255, 32), (257, 2048, 384, 128),
    (300, 640, 130, 128), (129, 224, 127, 32), (1025, 512, 128, 64), (64, 28672, 128, 128),
])
@pytest.mark.parametrize("zeros", [False, True])
def test_exact_shapes(T, d_in, d_out, group, zeros):
    g = torch.Generator("cuda").manual_seed(T + d_in + d_out)
    codes, scales, z = weights4(g, (), d_out, d_in, group, zeros, BF, True)
    x = ints(g, T, d_in, 1)
    ref = f64(x) @ dense64(codes, scales, z).T
    for dt in (BF, F):
        y = torch.empty(T, d_out, dtype=dt, device="cuda")
        sg.base_product(x, codes, scales, y, zeros=z)
        same(y, ref, dt)


@pytest.mark.parametrize("T,d_in,d_out,group,zeros,sdt", [
    (1, 4096, 1000, 128, False, BF), (4, 1024, 321, 64, True, F), (31, 992, 200, 32, True, BF), (150, 1024, 300, 128, False, F),
    (520, 768, 257, 64, True, BF)])
def test_real_values(T, d_in, d_out, group, zeros, sdt):
    g = torch.Generator("cuda").manual_seed(T)
    codes, scales, z = weights4(g, (), d_out, d_in, group, zeros, sdt, False)
    x = torch.randn(T, d_in, generator=g, device="cuda").to(BF)
    w = dense64(codes, scales, z)
    ref, big = f64(x) @ w.T, np.abs(f64(x)) @ np.abs(w).T
    for dt, half in ((BF, 2.0 ** -8), (F, 2.0 ** -24)):
        y = torch.empty(T, d_out, dtype=dt, device="cuda")
        sg.base_product(x, codes, scales, y, zeros=z)
        tol = 2 * d_in * 2.0 ** -23 * big
        assert (np.abs(f64(y) - ref) <= tol + half * (np.abs(ref) + tol)).all()
    y2 = torch.empty_like(y)
    sg.base_product(x, codes, scales, y2, zeros=z)
    assert torch.equal(y, y2)


def test_every_code_and_zero_point():
    """One column of W at a time: x is a unit vector, so y is (code - zero) * scale itself."""
    d_in, d_out = 32, 256
    n = torch.arange(256, device="cuda", dtype=torch.int64)
    codes = torch.zeros(d_out, 16, dtype=torch.uint8, device="cuda")
    codes[:, 5] = n.to(torch.uint8)
    scales = torch.full((d_out, 1), 3.0, device="cuda")
    x = torch.zeros(2, d_in, dtype=BF, device="cuda")
    x[0, 10] = 1
    x[1, 11] = 1
    y = torch.empty(2, d_out, device="cuda")
    sg.base_product(x, codes, scales, y)
    lo, hi = n % 16, n // 16
    assert torch.equal(y[0], 3.0 * (lo - 16 * (lo > 7)).float()) and torch.equal(y[1], 3.0 * (hi - 16 * (hi > 7)).float())
    for zp in range(16):
        z = torch.full((d_out, 1), zp, dtype=torch.uint8, device="cuda")
        sg.base_product(x, codes, scales, y, zeros=z)
        assert torch.equal(y[0], 3.0 * (lo - zp).float()) and torch.equal(y[1], 3.0 * (hi - zp).float())


@pytest.mark.parametrize("T", [2, 40, 300])
def test_infinities_and_nan_stay_in_their_rows(T):
    g = torch.Generator("cuda").manual_seed(3)
    codes, scales, _ = weights4(g, (), 100, 256, 64, False, BF, True)
    codes = codes & 0x77 | 0x11   # no code is 0, all positive
    x = ints(g, T, 256, 1)
    clean = torch.empty(T, 100, device="cuda")
    sg.base_product(x, codes, scales, clean)
    x[0, 17], x[1, 200] = float("nan"), float("inf")
    y = torch.empty(T, 100, device="cuda")
    sg.base_product(x, codes, scales, y)
    assert y[0].isnan().all() and (y[1] == float("inf")).all() and torch.equal(y[2:], clean[2:])


@pytest.mark.parametrize("T", [1, 20, 140])
def test_neighbours_of_y_are_left_alone(T):
    g = torch.Generator("cuda").manual_seed(4)
    codes, scales, _ = weights4(g, (), 67, 128, 32, False, F, True)
    x = ints(g, T, 128, 2)
    for dt in (BF, F):
        full = torch.full((T + 2, 75), 7.0, dtype=dt, device="cuda")
        sg.base_product(x, codes, scales, full[1:-1, 1:68])
        same(full[1:-1, 1:68], f64(x) @ dense64(codes, scales, None).T, dt)
        full[1:-1, 1:68] = 7.0
        assert (full == 7.0).all()


def routed(g, T, k, E, drop=0.0, only=None):
    ids = torch.rand(T, E, generator=g, device="cuda").topk(min(k, E), 1).indices.int()
    if only is not None:
        ids.fill_(only)
    if drop:
        ids = torch.where(torch.rand(ids.shape, generator=g, device="cuda") < drop, -1, ids)
    return ids.contiguous()


@pytest.mark.parametrize("T,k,E,drop,only", [
    (1, 1, 1, 0, None), (1, 2, 8, 0, None), (5, 3, 16, 0.3, None), (16, 2, 4, 0, None), (37, 4, 9, 0.1, None),
    (200, 2, 3, 0.05, None), (300, 1, 5, 0, 2), (64, 2, 100, 0, None), (150, 3, 2048, 0, None), (9, 2, 4, 1.0, None),
    (600, 2, 4, 0.02, None), (2, 1, 4096, 0, None)])
@pytest.mark.parametrize("gathered", [False, True])
def test_experts_exact(T, k, E, drop, only, gathered):
    g = torch.Generator("cuda").manual_seed(T * 100 + E)
    d_in, d_out, group = 160, 45, 32
    codes, scales, z = weights4(g, (E,), d_out, d_in, group, T % 2 == 1, BF, True)
    ids = routed(g, T, k, E, drop, only)
    k = ids.shape[1]
    offsets, row_of, slot_of = sg.expert_order(ids, E)
    x = ints(g, T, d_in, 2, 8)
    w = dense64(codes, scales, z)
    off, _, slots = order_ref(ids.cpu().numpy(), E)
    for dt in (BF, F):
        y = padded(T * k, d_out, dt, 2, fill=5.0)
        if gathered:
            xs = torch.full((T * k, d_in), float("nan"), dtype=BF, device="cuda")
            sg.expert_gather(x, row_of, xs)
            sg.base_product_experts(xs, codes, scales, offsets, y, zeros=z)
        else:
            sg.base_product_experts(x, codes, scales, offsets, y, zeros=z, slot_of=slot_of)
        ref = np.full((T * k, d_out), 5.0)
        for e in range(E):
            if off[e + 1] > off[e]:
                ref[off[e]:off[e + 1]] = f64(x)[slots[off[e]:off[e + 1]] // k] @ w[e].T
        same(y, ref, dt)
    assert sg.check_errors() == 0


def test_experts_more_rows_than_slots_used_and_wide_matrices():
    """A capacity buffer: y has more rows than the experts fill; d_out over several tiles."""
    g = torch.Generator("cuda").manual_seed(8)
    E, d_in, d_out = 3, 512, 1030
    codes, scales, z = weights4(g, (E,), d_out, d_in, 128, True, F, True)
    for counts in ([40, 0, 25], [0, 0, 1], [130, 200, 3]):
        offsets = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
        n = sum(counts)
        x = ints(g, n + 30, d_in, 1)
        y = torch.full((n + 30, d_out), 5.0, device="cuda")
        sg.base_product_experts(x, codes, scales, offsets, y, zeros=z)
        w = dense64(codes, scales, z)
        off = offsets.tolist()
        for e in range(E):
            same(y[off[e]:off[e + 1]], f64(x[off[e]:off[e + 1]]) @ w[e].T, F)
        assert (y[n:] == 5.0).all()
    assert sg.check_errors() == 0


def test_bad_offsets_and_slots_are_reported():
    """Values that the kernels check themselves: the rows concerned are not written, nothing is read out of range."""
    g = torch.Generator("cuda").manual_seed(9)
    codes, scales, _ = weights4(g, (2,), 40, 64, 32, False, BF, True)
    x = ints(g, 6, 64, 1)
    good = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    y = torch.full((6, 40), 5.0, device="cuda")
    sg.base_product_experts(x, codes, scales, good, y)
    clean = y.clone()
    for bad in ([0, 2, 9], [0, 7, 6], [-3, 2, 6], [0, 4, 2]):
        y.fill_(5.0)
        sg.base_product_experts(x, codes, scales, torch.tensor(bad, dtype=torch.int32, device="cuda"), y)
        with pytest.raises(sg.SgmvError) as e:
            sg.check_errors()
        assert e.value.status == 6
    slots = torch.tensor([0, 1, 2, 99, -1, 5], dtype=torch.int32, device="cuda")
    y.fill_(5.0)
    sg.base_product_experts(x, codes, scales, good, y, slot_of=slots)
    with pytest.raises(sg.SgmvError):
        sg.check_errors()
    assert (y[3:5] == 5.0).all() and torch.equal(y[[0, 1, 2, 5]], clean[[0, 1, 2, 5]])
    sg.check_errors()


def test_codes_past_two_gigabytes():
    """Offsets into the codes pass 32 bits; only the last rows are compared."""
    g = torch.Generator("cuda").manual_seed(10)
    E, d_out, d_in = 33, 16384, 8192       # 2.2 GB of codes
    codes = torch.randint(0, 256, (E, d_out, d_in // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.ones(E, d_out, d_in // 128, dtype=BF, device="cuda")
    offsets = torch.tensor([0] * E + [3], dtype=torch.int32, device="cuda")
    x = ints(g, 3, d_in, 1)
    y = torch.empty(3, d_out, device="cuda")
    sg.base_product_experts(x, codes, scales, offsets, y)
    same(y[:, -500:], f64(x) @ dense64(codes[-1, -500:], scales[-1, -500:], None).T, F)


@pytest.mark.parametrize("T", [3, 100])
def test_captured_and_on_another_stream(T):
    g = torch.Generator("cuda").manual_seed(11)
    codes, scales, z = weights4(g, (), 300, 512, 64, True, BF, False)
    x = torch.randn(T, 512, generator=g, device="cuda").to(BF)
    eager = torch.empty(T, 300, dtype=BF, device="cuda")
    sg.base_product(x, codes, scales, eager, zeros=z)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = torch.empty_like(eager)
    sg.base_product(x, codes, scales, other, zeros=z, stream=s)
    s.synchronize()
    assert torch.equal(eager, other)
    graph = torch.cuda.CUDAGraph()
    y = torch.empty_like(eager)
    with torch.cuda.graph(graph):
        sg.base_product(x, codes, scales, y, zeros=z)
    for _ in range(2):
        y.zero_()
        graph.replay()
        assert torch.equal(y, eager)
    x.neg_()
    graph.replay()
    assert torch.equal(y, -eager)
