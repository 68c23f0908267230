"""Tokens sorted by expert and back, against plain 64-bit forms.

The order, the gather and every slot without a row are exact.  A sum of k products w * v in fp32 (an fma each) is
off by at most k half steps of partial sums no larger than S = |add| + sum |w v|: k 2^-24 S; a dot product of d
terms by d 2^-24 S; then half a step of the type (2^-8 bf16, 2^-24 fp32) on top."""
import numpy as np
import pytest
import torch

import segmented_rank_gemm_sgmv_b200 as sg
from expert_cases import dense64, f64, order_ref, padded, weights4

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F: 2.0 ** -24}


def near(got, want, slack, dtype):
    err = np.abs(f64(got) - want)
    tol = slack + HALF[dtype] * (np.abs(want) + slack)
    assert (err <= tol).all(), f"{(err > tol).sum()} values off, worst {np.max(err - tol):.3g}"


def choices(rng, T, k, E, drop):
    ids = rng.integers(0, E, size=(T, k)).astype(np.int32)
    ids[rng.random((T, k)) < drop] = -1
    return ids


@pytest.mark.parametrize("T,k,E,drop", [
    (0, 1, 1, 0), (0, 3, 7, 0), (1, 1, 1, 0), (1, 1, 4096, 0), (1, 64, 8, 0), (31, 1, 2, 0.5), (33, 3, 5, 1.0), (100, 8, 256, 0),
    (512, 8, 64, 0.1), (1024, 4, 128, 0), (1025, 4, 33, 0.2), (4097, 1, 4096, 0.1), (5000, 7, 1, 0.3), (8192, 8, 256, 0.05),
    (20000, 3, 2049, 0), (70001, 2, 300, 0.01)])
def test_order(T, k, E, drop):
    rng = np.random.default_rng(T + 10 * k + E)
    ids = choices(rng, T, k, E, drop)
    want = order_ref(ids, E)
    got = sg.expert_order(torch.from_numpy(ids).cuda(), E)
    for a, b in zip(got, want):
        assert a.dtype == torch.int32 and np.array_equal(a.cpu().numpy(), b)
    assert sg.check_errors() == 0


@pytest.mark.parametrize("T", [50, 6000])
def test_order_reports_ids_out_of_range(T):
    rng = np.random.default_rng(T)
    ids = choices(rng, T, 2, 6, 0.1)
    bad = ids.copy()
    for v in (6, 7, 1 << 30, -2, -(1 << 31)):
        bad[rng.integers(0, T), rng.integers(0, 2)] = v
    got = sg.expert_order(torch.from_numpy(bad).cuda(), 6)
    with pytest.raises(sg.SgmvError) as e:
        sg.check_errors()
    assert e.value.status == 6
    for a, b in zip(got, order_ref(bad, 6)):
        assert np.array_equal(a.cpu().numpy(), b)
    sg.check_errors()


def test_order_into_given_tensors_and_two_calls_at_once():
    rng = np.random.default_rng(5)
    a, b = choices(rng, 30000, 2, 128, 0.1), choices(rng, 30000, 2, 128, 0.0)
    need = sg.expert_order_workspace(30000, 2, 128)
    assert need > 0 and sg.expert_order_workspace(10, 2, 128) == 0 and sg.expert_order_workspace(1, 65, 4) == -1
    dev = [torch.from_numpy(v).cuda() for v in (a, b)]
    streams = [torch.cuda.Stream() for _ in dev]
    outs = [(torch.empty(129, dtype=torch.int32, device="cuda"), torch.empty_like(v), torch.empty(60000, dtype=torch.int32, device="cuda"),
             torch.empty(need // 4, dtype=torch.int32, device="cuda")) for v in dev]
    torch.cuda.synchronize()
    for _ in range(5):
        for v, s, o in zip(dev, streams, outs):
            sg.expert_order(v, 128, *o, stream=s)
    torch.cuda.synchronize()
    for v, o in zip((a, b), outs):
        for x, y in zip(o, order_ref(v, 128)):
            assert np.array_equal(x.cpu().numpy(), y)
    with pytest.raises(sg.SgmvError) as e:
        sg.expert_order(dev[0], 128, *outs[0][:3], workspace=outs[0][3][:-1])
    assert e.value.status == 8


SIZES = [(1, 1, 1, 1, 0), (1, 2, 4, 8, 0), (3, 4, 8, 5, 0.3), (33, 2, 8, 1000, 0.1), (40, 3, 16, 4097, 0.2), (7, 8, 64, 8192, 0.0),
         (64, 1, 4, 520, 1.0), (500, 5, 10, 96, 0.05), (2, 64, 64, 264, 0.1)]


@pytest.mark.parametrize("T,k,E,d,drop", SIZES)
@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("extra", [0, 8, 3])
def test_gather_and_its_gradient(T, k, E, d, drop, dt, extra):
    g = torch.Generator("cuda").manual_seed(T + d)
    ids = torch.from_numpy(choices(np.random.default_rng(T), T, k, E, drop)).cuda()
    _, row_of, _ = sg.expert_order(ids, E)
    row = row_of.cpu().numpy()
    x = padded(T, d, dt, extra, g=g)
    xs = padded(T * k, d, dt, extra, fill=5.0)
    sg.expert_gather(x, row_of, xs)
    want = torch.full((T * k, d), 5.0, dtype=dt)
    for t in range(T):
        for j in range(k):
            if row[t, j] >= 0:
                want[row[t, j]] = x[t].cpu()
    assert torch.equal(xs.cpu(), want)
    dxs = padded(T * k, d, dt, extra, g=g)
    n = int((row >= 0).sum())
    dxs[n:] = float("nan")               # rows that no slot has are not read
    dx = padded(T, d, dt, extra)
    sg.expert_gather_backward(dxs, row_of, dx)
    v = np.where((row >= 0)[..., None], f64(dxs)[np.clip(row, 0, None)], 0)
    near(dx, v.sum(1), k * 2.0 ** -24 * np.abs(v).sum(1), dt)
    assert sg.check_errors() == 0


@pytest.mark.parametrize("T,k,E,d,drop", SIZES)
@pytest.mark.parametrize("ti,to", [(BF, BF), (BF, F), (F, BF), (F, F)])
@pytest.mark.parametrize("extra", [0, 1])
def test_combine_and_its_gradient(T, k, E, d, drop, ti, to, extra):
    g = torch.Generator("cuda").manual_seed(T + d + k)
    ids = torch.from_numpy(choices(np.random.default_rng(T), T, k, E, drop)).cuda()
    _, row_of, _ = sg.expert_order(ids, E)
    row, kept = row_of.cpu().numpy(), (row_of >= 0).cpu().numpy()
    n = int(kept.sum())
    ys = padded(T * k, d, ti, extra, g=g)
    ys[n:] = float("nan")
    w = torch.randn(T, k, generator=g, device="cuda")
    w[row_of < 0] = float("nan")         # weights of slots without a row are not read
    add = padded(T, d, to, extra, g=g)
    picked = np.where(kept[..., None], f64(ys)[np.clip(row, 0, None)], 0)
    w64 = np.where(kept, f64(w), 0)
    for weights, base in ((w, add), (w, None), (None, add), (None, None)):
        terms = picked * (w64 if weights is not None else kept.astype(np.float64))[..., None]
        b = f64(base) if base is not None else np.zeros((T, d))
        y = padded(T, d, to, extra)
        sg.expert_combine(ys, row_of, y, weights=weights, add=base)
        near(y, b + terms.sum(1), k * 2.0 ** -24 * (np.abs(b) + np.abs(terms).sum(1)), to)
    y2 = add.clone()
    sg.expert_combine(ys, row_of, y2, weights=w, add=y2)      # in place
    y3 = torch.empty_like(y2)
    sg.expert_combine(ys, row_of, y3, weights=w, add=add)
    assert torch.equal(y2, y3)

    dy = padded(T, d, to, extra, g=g)
    dys = padded(T * k, d, ti, extra, fill=5.0)
    dw = torch.empty(T, k, device="cuda")
    sg.expert_combine_backward(dy, ys, row_of, w, dys, dw)
    want = np.full((T * k, d), 5.0)
    prod = w64[..., None] * f64(dy)[:, None, :]
    want[row[kept]] = prod[kept]
    near(dys, want, 2.0 ** -24 * np.abs(want), ti)            # one product in fp32, then the type's rounding
    dots = f64(dy)[:, None, :] * picked
    near(dw, dots.sum(2), d * 2.0 ** -24 * np.abs(dots).sum(2), F)
    assert (dw.cpu().numpy()[~kept] == 0).all() and (f64(dys)[n:] == 5.0).all()
    # each alone gives the same bits
    a, b = padded(T * k, d, ti, extra, fill=5.0), torch.empty_like(dw)
    sg.expert_combine_backward(dy, ys, row_of, w, dys=a)
    sg.expert_combine_backward(dy, ys, row_of, w, dweights=b)
    assert torch.equal(a, dys) and torch.equal(b, dw)
    assert sg.check_errors() == 0


def test_combine_gradient_against_differences():
    """Central differences of the scalar <combine(ys, w), dy>, which is linear in ys and in w: with a step of 1 on
    values of a few bits the differences are exact in fp32."""
    g = torch.Generator("cuda").manual_seed(1)
    T, k, E, d = 4, 2, 3, 16
    ids = torch.tensor([[0, 2], [1, -1], [2, 2], [0, 1]], dtype=torch.int32, device="cuda")
    _, row_of, _ = sg.expert_order(ids, E)
    small = lambda *s: torch.randint(-3, 4, s, generator=g, device="cuda").float()  # noqa: E731
    ys, w, dy = small(T * k, d), small(T, k), small(T, d)

    def value(ys, w):
        y = torch.empty(T, d, device="cuda")
        sg.expert_combine(ys, row_of, y, weights=w)
        return (y * dy).sum().item()

    dys, dw = torch.zeros_like(ys), torch.empty_like(w)
    sg.expert_combine_backward(dy, ys, row_of, w, dys, dw)
    for i in range(T * k):
        for c in (0, 5, 15):
            step = torch.zeros_like(ys)
            step[i, c] = 1
            assert (value(ys + step, w) - value(ys - step, w)) / 2 == dys[i, c].item()
    for t in range(T):
        for j in range(k):
            step = torch.zeros_like(w)
            step[t, j] = 1
            assert (value(ys, w + step) - value(ys, w - step)) / 2 == dw[t, j].item()


def test_infinities_follow_the_formula():
    ids = torch.tensor([[0, 1], [1, -1]], dtype=torch.int32, device="cuda")
    _, row_of, _ = sg.expert_order(ids, 2)
    ys = torch.ones(4, 8, device="cuda")
    ys[1, 0], ys[1, 1] = float("inf"), float("nan")           # expert 1's row of token 0
    w = torch.tensor([[1.0, 0.0], [2.0, float("inf")]], device="cuda")
    y = torch.empty(2, 8, device="cuda")
    sg.expert_combine(ys, row_of, y, weights=w)
    assert y[0, :2].isnan().all() and (y[0, 2:] == 1).all() and (y[1] == 2).all()


def test_rows_outside_the_buffer_are_skipped_and_reported():
    """A row_of longer than the buffer: the kernels check every row before the access."""
    x = torch.randn(3, 40, device="cuda")
    row_of = torch.tensor([[0, 9], [1, -7], [2, 3]], dtype=torch.int32, device="cuda")
    xs = torch.full((4, 40), 5.0, device="cuda")
    calls = [lambda: sg.expert_gather(x, row_of, xs), lambda: sg.expert_gather_backward(xs, row_of, torch.empty_like(x)),
             lambda: sg.expert_combine(xs, row_of, torch.empty_like(x)),
             lambda: sg.expert_combine_backward(x, xs, row_of, None, torch.empty_like(xs), torch.empty(3, 2, device="cuda"))]
    for call in calls:
        call()
        with pytest.raises(sg.SgmvError) as e:
            sg.check_errors()
        assert e.value.status == 6
    assert torch.equal(xs, x[[0, 1, 2, 2]])


def test_buffers_past_four_gigabytes():
    """Byte offsets of rows pass 32 bits."""
    T, k, d = 40000, 2, 32768
    ids = torch.arange(T * k, device="cuda", dtype=torch.int32).reshape(T, k) % 3
    _, row_of, _ = sg.expert_order(ids, 3)
    x = torch.empty(T, d, dtype=BF, device="cuda")
    x[:, :] = (torch.arange(T, device="cuda") % 251).to(BF)[:, None]
    xs = torch.zeros(T * k, d, dtype=BF, device="cuda")
    sg.expert_gather(x, row_of, xs)
    slots = torch.empty(T * k, dtype=torch.int64, device="cuda")
    slots[row_of.reshape(-1).long()] = torch.arange(T * k, device="cuda")
    for c in (0, d // 2, d - 1):
        assert torch.equal(xs[:, c], x[slots // k, c])
    y = torch.empty_like(x)
    sg.expert_combine(xs, row_of, y, weights=torch.full((T, k), 0.5, device="cuda"))
    assert torch.equal(y, x)
    del x, y
    sg.check_errors()


def expert_layer(x, ids, weights, w4, pool, plan, E, k, y):
    """An adapted expert projection: sorted rows, base products, each expert's adapter, the weighted sum onto y."""
    offsets, row_of, slot_of = sg.expert_order(ids, E)
    xs = torch.zeros(ids.numel(), x.shape[1], dtype=BF, device="cuda")
    ys = torch.zeros(ids.numel(), y.shape[1], dtype=F, device="cuda")
    sg.expert_gather(x, row_of, xs)
    sg.base_product_experts(xs, w4[0], w4[1], offsets, ys, zeros=w4[2])
    sg.lora_delta(xs, plan, pool, ys, 0, 1.0)
    sg.expert_combine(ys, row_of, y, weights=weights, add=y)
    return row_of


@pytest.mark.parametrize("T,k,E", [(3, 2, 4), (40, 2, 5), (200, 3, 6)])
def test_adapted_expert_layer_and_its_replay(T, k, E):
    """The operators as they are used together: a mixture-of-experts projection whose experts carry adapters.  ys is
    kept in fp32, x is of small integers: base and delta are bounded as in their own tests, the whole by the sum."""
    rng = np.random.default_rng(T)
    g = torch.Generator("cuda").manual_seed(T)
    d_in, d_out, r = 512, 1024, 8
    host_ids = np.argsort(rng.random((T, E)), 1)[:, :k].astype(np.int32)
    ids = torch.from_numpy(host_ids).cuda()
    weights = torch.softmax(torch.randn(T, k, generator=g, device="cuda"), 1)
    w4 = weights4(g, (E,), d_out, d_in, 64, True, BF, False)
    x = torch.randn(T, d_in, generator=g, device="cuda").to(BF)
    y0 = torch.randn(T, d_out, generator=g, device="cuda")
    A = [(torch.randn(r, d_in, generator=g, device="cuda") / d_in ** 0.5).to(BF) for _ in range(E)]
    B = [(torch.randn(d_out, r, generator=g, device="cuda") / r ** 0.5).to(BF) for _ in range(E)]
    pool = sg.AdapterPool([(d_in, d_out)], num_pages=256, page_elems=512, max_rank=r, device=0)
    for e in range(E):
        pool.load(e, r, [A[e]], [B[e]])
    plan = pool.plan(np.sort(host_ids.reshape(-1), kind="stable"))      # the sorted rows' adapters
    plan.upload()
    y = y0.clone()
    row = expert_layer(x, ids, weights, w4, pool, plan, E, k, y).cpu().numpy()
    assert np.array_equal(row, order_ref(host_ids, E)[1])
    sg.check_errors()
    w, x64 = dense64(*w4), f64(x)
    want, slack = f64(y0), np.abs(f64(y0)) * 2.0 ** -24 * k
    for t in range(T):
        for j in range(k):
            e, wt = host_ids[t, j], f64(weights)[t, j]
            v = f64(A[e]) @ x64[t]
            v_abs = np.abs(f64(A[e])) @ np.abs(x64[t])
            want[t] += wt * (w[e] @ x64[t] + f64(B[e]) @ v)
            big = np.abs(w[e]) @ np.abs(x64[t])
            # base: 2 d_in steps of 2^-23; delta: d_in + r fp32 steps, and v as a bf16 pair (2^-16) on tensor cores
            slack[t] += wt * ((2 * d_in + k + 4) * 2.0 ** -23 * big + (2.0 ** -16 + 2 * (d_in + r) * 2.0 ** -23) * (np.abs(f64(B[e])) @ v_abs))
    near(y, want, slack, F)

    graph = torch.cuda.CUDAGraph()
    z = y0.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        expert_layer(x, ids, weights, w4, pool, plan, E, k, z)
    torch.cuda.current_stream().wait_stream(s)
    for _ in range(2):
        z.copy_(y0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(z, y)
    del graph
    pool.close()
