"""Plain 64-bit forms of the expert operators and the 4-bit base products, and their inputs."""
import numpy as np
import torch


def weights4(g, lead, d_out, d_in, group, zeros, scale_dtype, exact):
    """(codes, scales, zeros) on the GPU.  `exact`: scales are powers of two in [1/8, 1]."""
    shape = (*lead, d_out, d_in // group)
    codes = torch.randint(0, 256, (*lead, d_out, d_in // 2), generator=g, device="cuda", dtype=torch.uint8)
    if exact:
        scales = torch.exp2(-torch.randint(0, 4, shape, generator=g, device="cuda").float())
    else:
        scales = (0.25 + torch.rand(shape, generator=g, device="cuda")) * torch.where(
            torch.rand(shape, generator=g, device="cuda") < 0.5, -1.0, 1.0)
    z = torch.randint(0, 16, shape, generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    return codes, scales.to(scale_dtype), z


def dense64(codes, scales, zeros):
    """The matrix the codes stand for, fp64 [.., d_out, d_in]."""
    q = np.empty((*codes.shape[:-1], codes.shape[-1] * 2), dtype=np.float64)
    c = codes.cpu().numpy()
    q[..., 0::2], q[..., 1::2] = c & 15, c >> 4
    s = scales.double().cpu().numpy()
    group = q.shape[-1] // s.shape[-1]
    if zeros is None:
        q = np.where(q >= 8, q - 16, q)
    else:
        q = q - np.repeat(zeros.cpu().numpy().astype(np.float64), group, -1)
    return q * np.repeat(s, group, -1)


def f64(t):
    return t.detach().double().cpu().numpy()


def rounded(a, dtype):
    """fp64 values rounded to the type (through fp32 only where that is exact: fp32 itself)."""
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype)


def order_ref(ids, n_experts):
    """(offsets, row_of, slot_of) by a plain loop."""
    ids = np.asarray(ids)
    flat = ids.reshape(-1)
    rows = [[] for _ in range(n_experts)]
    for s, e in enumerate(flat.tolist()):
        if 0 <= e < n_experts:
            rows[e].append(s)
    offsets = np.concatenate([[0], np.cumsum([len(r) for r in rows])]).astype(np.int32)
    slots = [s for r in rows for s in r]
    row_of = np.full(flat.shape, -1, np.int32)
    slot_of = np.full(flat.shape, -1, np.int32)
    for i, s in enumerate(slots):
        row_of[s] = i
        slot_of[i] = s
    return offsets, row_of.reshape(ids.shape), slot_of


def padded(rows, cols, dtype, extra, fill=None, g=None):
    """A [rows, cols] view of a buffer with `extra` more columns a row, all of it `fill` or random."""
    full = torch.full((rows, cols + extra), float("nan") if fill is None else fill, dtype=dtype, device="cuda")
    if g is not None:
        full.copy_(torch.randn(rows, cols + extra, generator=g, device="cuda"))
    return full[:, :cols]
