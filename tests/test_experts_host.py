"""Refusals of the expert operators and the base products: a status before any CUDA call (C ABI, no GPU needed),
and the binding's own checks."""
import pytest
import torch

import segmented_rank_gemm_sgmv_b200 as sg

P = 1 << 20   # an aligned address that is never touched


def product(**kw):
    a = dict(x=P, ldx=256, T=2, d_in=256, d_out=8, codes=P, scales=P, sdt=0, zeros=None, group=64, y=P, ldy=8, ydt=0, ws=P, nws=1 << 30)
    a.update(kw)
    return sg.load_library().sgmv_base_product(a["x"], a["ldx"], a["T"], a["d_in"], a["d_out"], a["codes"], a["scales"], a["sdt"],
                                               a["zeros"], a["group"], a["y"], a["ldy"], a["ydt"], a["ws"], a["nws"], None)


def test_base_product_workspace():
    lib = sg.load_library()
    # three digits a value and 16 bytes a group for each row
    assert lib.sgmv_base_product_workspace(1, 32, 32) == 96 + 16
    assert lib.sgmv_base_product_workspace(3, 8192, 128) == 3 * 3 * 8192 + 3 * 64 * 16
    assert lib.sgmv_base_product_workspace(0, 64, 64) == 0 and lib.sgmv_base_product_workspace(17, 8192, 128) == 0
    for bad in ((-1, 64, 64), (1, 0, 64), (1, 64, 128), (1, 96, 64), (1, 1 << 21, 64), (1 << 24, 64, 64)):
        assert lib.sgmv_base_product_workspace(*bad) == -1
    assert product(ws=None) == 1 and product(ws=P + 8) == 1 and product(nws=10) == 8 and product(T=1 << 24) == 2


@pytest.mark.parametrize("kw,why", [
    (dict(T=-1), b"rows"), (dict(d_in=0), b"d_in"), (dict(d_out=0), b"d_out"), (dict(group=16), b"group"), (dict(group=0), b"group"),
    (dict(d_in=224, group=64), b"multiple"), (dict(sdt=2), b"scale_dtype"), (dict(ydt=-1), b"y_dtype"), (dict(x=None), b"required"),
    (dict(codes=None), b"required"), (dict(scales=None), b"required"), (dict(y=None), b"required"), (dict(x=P + 8), b"aligned"),
    (dict(ldx=255), b"aligned"), (dict(ldx=248), b"ldx"), (dict(codes=P + 4), b"codes"), (dict(scales=P + 2, sdt=1), b"scales"),
    (dict(scales=P + 1), b"scales"), (dict(y=P + 1), b"y must"), (dict(y=P + 2, ydt=1), b"y must"), (dict(ldy=7), b"ldy")])
def test_base_product_refuses(kw, why):
    assert product(**kw) == 1 and why in sg.load_library().sgmv_last_error()


def test_base_product_of_nothing():
    assert product(T=0, x=None, y=None) == 0


def experts(**kw):
    a = dict(x_rows=4, E=3, offsets=P, slot_of=None, k=1, rows=4)
    a.update(kw)
    return sg.load_library().sgmv_base_product_experts(P, 64, a["x_rows"], 64, 8, a["E"], P, P, 0, None, 64, a["offsets"], a["slot_of"],
                                                       a["k"], a["rows"], P, 8, 0, a.get("ws"), a.get("nws", 0), None)


def test_base_product_experts_workspace():
    lib = sg.load_library()
    f = lib.sgmv_base_product_experts_workspace
    assert f(8, 64, 64, 1, 0) == f(8, 64, 64, 1, 1) == lib.sgmv_base_product_workspace(8, 64, 64) > 0 and f(0, 64, 64, 3, 1) == 0
    assert f(17, 64, 64, 1, 0) == 0 and f(17, 64, 64, 1, 1) == 17 * 128
    assert f(-1, 64, 64, 1, 0) == f(1, 64, 64, 4097, 0) == f(1, 64, 64, 0, 0) == f(1, 64, 16, 1, 0) == -1
    many = dict(rows=400, x_rows=400, slot_of=P)
    assert experts(**many) == 1 and b"workspace" in lib.sgmv_last_error()
    assert experts(**many, ws=P + 8, nws=1 << 20) == 1 and experts(**many, ws=P, nws=400 * 128 - 1) == 8


@pytest.mark.parametrize("kw", [dict(E=0), dict(E=4097), dict(offsets=None), dict(offsets=P + 2), dict(x_rows=3), dict(slot_of=P, k=0),
                                dict(slot_of=P, k=65), dict(slot_of=P, x_rows=0), dict(slot_of=P + 1), dict(rows=-1), dict(x_rows=-1)])
def test_base_product_experts_refuses(kw):
    assert experts(**kw) == 1 and b"base_product_experts" in sg.load_library().sgmv_last_error()


def order(**kw):
    a = dict(ids=P, T=5, k=2, E=4, offsets=P, row_of=P, slot_of=P, ws=None, nws=0)
    a.update(kw)
    return sg.load_library().sgmv_expert_order(a["ids"], a["T"], a["k"], a["E"], a["offsets"], a["row_of"], a["slot_of"], a["ws"], a["nws"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(k=0), 1), (dict(k=65), 1), (dict(E=0), 1), (dict(E=4097), 1), (dict(T=1 << 30), 2), (dict(ids=None), 1),
    (dict(offsets=None), 1), (dict(row_of=None), 1), (dict(slot_of=None), 1), (dict(ids=P + 2), 1), (dict(offsets=P + 1), 1),
    (dict(T=100000), 1), (dict(T=100000, ws=P, nws=16), 8), (dict(T=100000, ws=P + 2, nws=1 << 30), 1)])
def test_expert_order_refuses(kw, status):
    assert order(**kw) == status and b"expert_order" in sg.load_library().sgmv_last_error()


def test_expert_order_workspace():
    lib = sg.load_library()
    assert lib.sgmv_expert_order_workspace(0, 1, 1) == 0 and lib.sgmv_expert_order_workspace(16, 8, 4096) == 0
    for bad in ((-1, 1, 1), (1, 0, 1), (1, 65, 1), (1, 1, 0), (1, 1, 4097), (1 << 30, 2, 1)):
        assert lib.sgmv_expert_order_workspace(*bad) == -1
    for T, k, E in ((1 << 20, 8, 4096), (1 << 24, 64, 1), (100000, 2, 64)):
        n = lib.sgmv_expert_order_workspace(T, k, E)
        assert n > 0 and n % (4 * E) == 0 and n <= 4 * 65536


@pytest.mark.parametrize("kw", [dict(T=-1), dict(d=0), dict(rows=-1), dict(k=0), dict(k=65), dict(dt=2), dict(x=None), dict(xs=None),
                                dict(row_of=None), dict(ldx=7), dict(ldxs=7), dict(x=P + 1), dict(row_of=P + 2)])
def test_row_operators_refuse(kw):
    a = dict(x=P, ldx=8, T=2, d=8, dt=0, row_of=P, k=2, xs=P, ldxs=8, rows=4)
    a.update(kw)
    lib = sg.load_library()
    assert lib.sgmv_expert_gather(a["x"], a["ldx"], a["T"], a["d"], a["dt"], a["row_of"], a["k"], a["xs"], a["ldxs"], a["rows"], None) == 1
    assert lib.sgmv_expert_gather_backward(a["xs"], a["ldxs"], a["rows"], a["T"], a["d"], a["dt"], a["row_of"], a["k"], a["x"], a["ldx"],
                                           None) == 1
    assert lib.sgmv_expert_combine(a["xs"], a["ldxs"], a["rows"], a["dt"], a["row_of"], None, a["T"], a["k"], a["d"], None, 0, a["x"],
                                   a["ldx"], 0, None) == 1
    assert lib.sgmv_expert_combine_backward(a["x"], a["ldx"], a["dt"], a["xs"], a["ldxs"], a["rows"], 0, a["row_of"], None, a["T"], a["k"],
                                            a["d"], a["xs"], a["ldxs"], P, None) == 1


def test_row_operators_of_nothing():
    lib = sg.load_library()
    assert lib.sgmv_expert_gather(None, 8, 0, 8, 0, None, 2, None, 8, 0, None) == 0
    assert lib.sgmv_expert_combine(None, 8, 0, 0, None, None, 0, 2, 8, None, 0, None, 8, 0, None) == 0
    assert lib.sgmv_expert_combine_backward(P, 8, 0, P, 8, 4, 0, P, None, 2, 2, 8, None, 0, None, None) == 0
    assert lib.sgmv_expert_combine(P, 8, 4, 0, P, P + 2, 2, 2, 8, None, 0, P, 8, 0, None) == 1
    assert lib.sgmv_expert_combine(P, 8, 4, 0, P, P, 2, 2, 8, P, 7, P, 8, 0, None) == 1


def test_binding_refuses_host_tensors():
    x, codes = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(8, 32, dtype=torch.uint8)
    row_of = torch.zeros(2, 2, dtype=torch.int32)
    for call in (lambda: sg.base_product(x, codes, torch.ones(8, 1), torch.empty(2, 8)),
                 lambda: sg.base_product_experts(x, codes[None], torch.ones(1, 8, 1), torch.zeros(2, dtype=torch.int32), torch.empty(2, 8)),
                 lambda: sg.expert_order(row_of, 4), lambda: sg.expert_gather(x, row_of, x), lambda: sg.expert_gather_backward(x, row_of, x),
                 lambda: sg.expert_combine(x, row_of, x), lambda: sg.expert_combine_backward(x, x, row_of, None)):
        with pytest.raises(ValueError, match="current CUDA device"):
            call()


@pytest.mark.gpu
def test_binding_refuses_shapes_and_types():
    bf = dict(dtype=torch.bfloat16, device="cuda")
    x, y = torch.zeros(2, 64, **bf), torch.zeros(2, 8, **bf)
    codes, scales = torch.zeros(8, 32, dtype=torch.uint8, device="cuda"), torch.ones(8, 2, device="cuda")
    row_of = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    w = torch.ones(2, 2, device="cuda")
    bad = [lambda: sg.base_product(x.float(), codes, scales, y), lambda: sg.base_product(x[:, :32], codes, scales, y),
           lambda: sg.base_product(x, codes, scales, y[:, :7]), lambda: sg.base_product(x, codes, scales, y[:1]),
           lambda: sg.base_product(x, codes.to(torch.int8), scales, y), lambda: sg.base_product(x, codes, scales.half(), y),
           lambda: sg.base_product(x, codes, scales[:, :1], y), lambda: sg.base_product(x, codes, scales[:7], y),
           lambda: sg.base_product(x, codes, scales, y, zeros=scales), lambda: sg.base_product(x, codes, scales, y.t().contiguous().t()),
           lambda: sg.base_product(x, codes, scales, y.half()), lambda: sg.base_product(x, codes, scales, y.cpu()),
           lambda: sg.base_product_experts(x, codes, scales, row_of[0], y),
           lambda: sg.base_product_experts(x, codes[None], scales[None], row_of, y),
           lambda: sg.base_product_experts(x, codes[None], scales[None], row_of[0], y[:1]),
           lambda: sg.base_product_experts(x, codes[None], scales[None], row_of[0], y, slot_of=row_of),
           lambda: sg.expert_order(row_of.long(), 4), lambda: sg.expert_order(row_of[0], 4), lambda: sg.expert_order(row_of, 4, offsets=row_of),
           lambda: sg.expert_gather(x, row_of, y), lambda: sg.expert_gather(x, row_of, x.float()), lambda: sg.expert_gather(x[:1], row_of, x),
           lambda: sg.expert_combine(x, row_of, y), lambda: sg.expert_combine(x, row_of, x, weights=w.to(torch.bfloat16)),
           lambda: sg.expert_combine(x, row_of, x, weights=w[:1]), lambda: sg.expert_combine(x, row_of, x, add=x.float()),
           lambda: sg.expert_combine_backward(x, x, row_of, w, dys=x.float()),
           lambda: sg.expert_combine_backward(x, x, row_of, w, dweights=w.double())]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, sg.SgmvError)):
            call()
            pytest.fail(f"call {i} was not refused")
    with pytest.raises(sg.SgmvError):
        sg.expert_order(row_of, 0)
    sg.check_errors()


def test_row_operators_refuse_rows_past_2_30_values():
    """Column numbers are 32 bits wide."""
    lib, d = sg.load_library(), (1 << 30) + 8
    assert lib.sgmv_expert_gather(P, d, 1, d, 0, P, 1, P, d, 1, None) == 2
    assert lib.sgmv_expert_gather_backward(P, d, 1, 1, d, 0, P, 1, P, d, None) == 2
    assert lib.sgmv_expert_combine(P, d, 1, 0, P, None, 1, 1, d, None, 0, P, d, 0, None) == 2
    assert lib.sgmv_expert_combine_backward(P, d, 0, P, d, 1, 0, P, None, 1, 1, d, P, d, P, None) == 2
