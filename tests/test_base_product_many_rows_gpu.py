"""Base products of 17 rows a matrix and more: every tile of rows and its edges, K from one stage on.

Exact: x of -1, 0, 1 and scales of 1/8 .. 1 make every partial sum a multiple of 2^-3 below 15 d_in < 2^20, so that fp32
sums in any order are exact and y has to be the rounded 64-bit value bit for bit."""
import numpy as np
import pytest
import torch

import segmented_rank_gemm_sgmv_b200 as sg
from expert_cases import dense64, f64, padded, rounded, weights4

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


def units(g, rows, d_in):
    return torch.randint(-1, 2, (rows, d_in), generator=g, device="cuda").to(BF)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T", [17, 32, 33, 64, 65, 128, 129, 145, 240, 256, 257, 511])
def test_edges_of_the_row_tiles(T, group):
    g = torch.Generator("cuda").manual_seed(T + group)
    for n, d_out, extra in ((1, 134, 2), (2, 7, 0), (11, 260, 1), (34, 129, 3)):
        d_in = n * group
        codes, scales, z = weights4(g, (), d_out, d_in, group, n % 2 == 0, (BF, F)[T % 2], True)
        x = units(g, T, d_in)
        ref = f64(x) @ dense64(codes, scales, z).T
        for dt in (BF, F):
            y = padded(T, d_out, dt, extra, fill=5.0)
            sg.base_product(x, codes, scales, y, zeros=z)
            assert torch.equal(y.cpu(), rounded(ref, dt)), (n, d_out, dt)
            if extra:
                assert (y.as_strided((T, extra), y.stride(), d_out) == 5.0).all()
    assert sg.check_errors() == 0


@pytest.mark.parametrize("group", [32, 64, 128])
def test_experts_of_uneven_size(group):
    """Averages that choose each tile of rows, with experts far above and below them."""
    g = torch.Generator("cuda").manual_seed(group)
    d_in, d_out = group * 6, 140
    for counts in ([20, 100, 0, 1], [700, 3, 40], [0, 50, 300, 17, 90], [16, 17, 18], [1000, 0, 0, 0, 0, 0, 0, 0]):
        E, rows = len(counts), sum(counts)
        codes, scales, z = weights4(g, (E,), d_out, d_in, group, True, BF, True)
        x = units(g, rows, d_in)
        offsets = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
        slots = torch.randperm(rows, generator=g, device="cuda").int()
        w, off = dense64(codes, scales, z), offsets.tolist()
        for slot_of in (None, slots):
            y = torch.empty(rows, d_out, device="cuda")
            sg.base_product_experts(x, codes, scales, offsets, y, zeros=z, slot_of=slot_of)
            xs = f64(x if slot_of is None else x[slots.long()])
            for e in range(E):
                assert torch.equal(y[off[e]:off[e + 1]].cpu(), rounded(xs[off[e]:off[e + 1]] @ w[e].T, F)), (counts, e)
    assert sg.check_errors() == 0


@pytest.mark.parametrize("rows,E", [(6, 4), (90, 4)])
def test_experts_captured_then_replayed_with_other_routes(rows, E):
    g = torch.Generator("cuda").manual_seed(rows)
    d_in, d_out = 256, 70
    codes, scales, z = weights4(g, (E,), d_out, d_in, 64, True, BF, True)
    w = dense64(codes, scales, z)
    x, ids = units(g, rows, d_in), torch.zeros(rows, 1, dtype=torch.int32, device="cuda")
    offsets, row_of, slot_of = sg.expert_order(ids, E)
    y = torch.empty(rows, d_out, device="cuda")

    def step():
        sg.expert_order(ids, E, offsets, row_of, slot_of)
        sg.base_product_experts(x, codes, scales, offsets, y, zeros=z, slot_of=slot_of)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        x.copy_(units(g, rows, d_in))
        ids.copy_(torch.randint(0, E, (rows, 1), generator=g, device="cuda"))
        y.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        at = row_of[:, 0].long().cpu()
        for t in range(rows):
            assert torch.equal(y[at[t]].cpu(), rounded(f64(x[t]) @ w[int(ids[t])].T, F))
    assert sg.check_errors() == 0


def test_two_streams_at_once_through_slots():
    """Calls that overlap on two streams gather x into a workspace each."""
    g = torch.Generator("cuda").manual_seed(1)
    E, rows, d_in, d_out = 3, 900, 1024, 512
    codes, scales, _ = weights4(g, (E,), d_out, d_in, 128, False, BF, True)
    offsets = torch.tensor([0, 200, 500, 900], dtype=torch.int32, device="cuda")
    inputs = [(units(g, rows, d_in), torch.randperm(rows, generator=g, device="cuda").int()) for _ in range(2)]
    want = []
    for x, slots in inputs:
        y = torch.empty(rows, d_out, device="cuda")
        sg.base_product_experts(x, codes, scales, offsets, y, slot_of=slots)
        want.append(y)
    streams, got = [torch.cuda.Stream() for _ in inputs], [torch.empty_like(y) for y in want]
    torch.cuda.synchronize()
    for _ in range(20):
        for (x, slots), y, s in zip(inputs, got, streams):
            sg.base_product_experts(x, codes, scales, offsets, y, slot_of=slots, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and sg.check_errors() == 0
