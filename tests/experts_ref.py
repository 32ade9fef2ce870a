"""Plain fp64 forms of the operators on the components' lists (numpy), and
the assignments the tests feed them."""
import numpy as np
import torch

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
# largest relative error of one rounding to the storage type
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
# half the spacing of the subnormals: an absolute error of the same rounding
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -25}


def assignment(n, m, k, rng, holes=0.1, repeats=False):
    """idx [n, m] as gmm_assign writes it (distinct components; -1 behind a
    row's last), with some rows empty; with repeats the same component may come twice."""
    if repeats or m > k:
        idx = rng.integers(0, k, size=(n, m))
    else:
        idx = np.argsort(rng.random((n, k)), axis=1)[:, :m] if n * k < 4_000_000 else \
            (rng.integers(0, k, size=(n, 1)) + np.arange(m) * max(1, k // m)) % k
    last = np.where(rng.random(n) < holes, rng.integers(0, m + 1, size=n), m)
    idx[np.arange(m)[None, :] >= last[:, None]] = -1
    return idx.astype(np.int32)


def lists(idx, k):
    flat = idx.reshape(-1)
    ok = (flat >= 0) & (flat < k)
    order = np.concatenate([np.nonzero(flat == kk)[0] for kk in range(k)]) if k <= 64 else \
        np.argsort(np.where(ok, flat, k), kind="stable")[:ok.sum()]
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[ok], minlength=k))])
    entry = np.full(flat.size, -1)
    slot = np.full(flat.size, -1)
    entry[:order.size] = order
    slot[order] = np.arange(order.size)
    return offsets, entry, slot.reshape(idx.shape)


def f64(t):
    return t.detach().double().cpu().numpy()


def gathered(z, slot):
    """[n, m, d] rows of every entry, zero where it is not listed."""
    return np.where((slot >= 0)[..., None], z[np.maximum(slot, 0)], 0.0)


def decode4(codes, scales, group, d_in):
    q = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)[..., :d_in].astype(np.float64) - 8
    return q * np.repeat(scales, group, -1)[..., :d_in]


def quantize4(w, group):
    """(codes, scales as fp32 numpy) of fp32 weights [rows, d_in], in fp32
    arithmetic: one division for the scale, one rounding to bf16, one division and
    one rounding for the code."""
    rows, d = w.shape
    groups = -(-d // group)
    pad = np.zeros((rows, groups * group), np.float32)
    pad[:, :d] = w
    g = pad.reshape(rows, groups, group)
    top = np.abs(g).max(-1) / np.float32(7)
    s = torch.from_numpy(top).to(torch.bfloat16).float().numpy()
    with np.errstate(all="ignore"):
        q = np.rint(g / s[..., None])
    q = np.where((s[..., None] == 0) | ~np.isfinite(s[..., None]), 0, np.clip(q, -8, 7))
    q = (q.reshape(rows, -1)[:, :d] + 8).astype(np.uint8)
    if d % 2:
        q = np.concatenate([q, np.full((rows, 1), 8, np.uint8)], 1)
    return q[:, 0::2] | (q[:, 1::2] << 4), s


def close(got, ref, bound, what):
    """Element by element |got - ref| <= bound; both finite."""
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.isfinite(got).all(), what
    over = np.abs(got - ref) - bound
    worst = float(over.max()) if over.size else -1.0
    assert worst <= 0.0, f"{what}: {int((over > 0).sum())} of {over.size} values off by up to {worst:.3e} over the bound"
