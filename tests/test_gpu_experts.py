"""The operators on the components' lists (include/gmm_experts.h) against their
plain fp64 forms.

Bounds, element by element.  A sum of L fp32 terms t_i, in any order, is off by
at most (L + 1) 2^-23 sum |t_i| (each product and each addition rounds or truncates once,
2^-23 relative at most), and the store rounds once more, half a step of its type (U) or of its
subnormals (TINY).  Where inputs are small whole numbers every product and sum
is exact, so the outputs equal the fp64 result rounded once to the storage type.
"""
import numpy as np
import pytest
import torch

from soft_clustering_amd import experts
from tests import experts_ref as R

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -23
CASES = [   # n, m, k
    (1, 1, 1), (1, 2, 16), (1, 16, 4096), (7, 3, 5), (64, 1, 64), (100, 2, 65), (300, 4, 3), (1000, 2, 16),
    (2731, 3, 300),
]


def dev(a, dtype=None):
    t = torch.as_tensor(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


def routes_of(idx, k):
    return experts.Routes(*(dev(a.astype(np.int32)) for a in R.lists(idx, k)))


def padded(rows, width, dtype, pad, fill=float("nan")):
    """A [rows, width] view of a wider buffer, and the buffer."""
    buf = torch.full((rows, width + pad), fill, dtype=dtype, device="cuda")
    return buf[:, :width], buf


def rows_tensor(rng, rows, width, dtype, pad, whole):
    a = rng.integers(-3, 4, size=(rows, width)).astype(np.float32) if whole else \
        rng.standard_normal((rows, width)).astype(np.float32)
    v, buf = padded(rows, width, dtype, pad)
    v.copy_(torch.from_numpy(a))
    return v


def untouched(buf, width, first_row, fill):
    """The padding columns and the rows from first_row on still hold `fill`."""
    b = buf.float()
    want = torch.full_like(b, fill)
    assert torch.equal(b[:, width:], want[:, width:])
    assert torch.equal(b[first_row:], want[first_row:])


# --- lists ---------------------------------------------------------------------
@pytest.mark.parametrize("n,m,k", CASES + [
    (4096, 2, 16), (4097, 2, 16), (8192, 1, 4096), (20_000, 7, 1), (50_001, 3, 4095), (100_000, 2, 4096),
    (400_000, 16, 33)])
def test_route(n, m, k):
    rng = np.random.default_rng(n + 31 * k)
    idx = R.assignment(n, m, k, rng, repeats=k < m)
    r = experts.route(dev(idx), k)
    for got, want in zip(r, R.lists(idx, k)):
        assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("n,k", [(1000, 5), (30_000, 700)])
def test_route_foreign_values(n, k):
    """Entries outside [0, k), the extremes of int32 among them, are in no list;
    one component twice in a row counts twice; one list takes everything."""
    rng = np.random.default_rng(7)
    idx = rng.integers(0, k, size=(n, 4)).astype(np.int32)
    idx[::3, 1] = idx[::3, 0]
    idx[::5, 2] = [2 ** 31 - 1, -2 ** 31, k, -1][k % 4]
    idx[1::5, 3] = -2 ** 31
    for a in (idx, np.full_like(idx, k - 1), np.full_like(idx, -1)):
        r = experts.route(dev(a), k)
        for got, want in zip(r, R.lists(a, k)):
            assert np.array_equal(got.cpu().numpy(), want)


def test_route_no_points():
    r = experts.route(torch.empty((0, 2), dtype=torch.int32, device="cuda"), 5)
    assert r.offsets.tolist() == [0] * 6 and r.entry.numel() == 0 and tuple(r.slot.shape) == (0, 2)


# --- rows there and back -----------------------------------------------------------
ROWS = [(n, m, k, d, dt, pad) for i, (n, m, k) in enumerate(CASES) for d, dt, pad in [
    [(64, "f32", 0), (128, "bf16", 8), (93, "f16", 0)], [(1, "bf16", 0), (77, "f32", 3), (1000, "f16", 0)],
    [(8, "f16", 0), (513, "bf16", 1), (260, "f32", 4)]][i % 3]]


@pytest.mark.parametrize("n,m,k,d,dt,pad", ROWS)
def test_rows(n, m, k, d, dt, pad):
    """dispatch and its gradient, combine and its gradients."""
    rng = np.random.default_rng(n * 1009 + d)
    idx = R.assignment(n, m, k, rng, repeats=k < m)
    off, entry, slot = R.lists(idx, k)
    total, rows = off[-1], n * m
    r, t = routes_of(idx, k), R.DT[dt]
    x = rows_tensor(rng, n, d, t, pad, False)
    y, ybuf = padded(rows, d, t, pad, 9.0)
    experts.dispatch(x, r, out=y)
    assert torch.equal(y[:total], x[torch.from_numpy(entry[:total] // m).cuda()])
    untouched(ybuf, d, total, 9.0)

    z = rows_tensor(rng, rows, d, t, pad, False)
    gamma = rng.random((n, m)).astype(np.float32)
    gamma[idx < 0] = np.nan          # the weight of an unlisted column is not used
    g = dev(gamma)
    terms = R.gathered(R.f64(z), slot)
    g0 = np.where(idx >= 0, gamma.astype(np.float64), 0.0)[..., None]
    for name, got, t3 in [("dispatch_backward", experts.dispatch_backward(z, r), terms),
                          ("combine", experts.combine(z, g, r), terms * g0)]:
        ref = t3.sum(1)
        R.close(R.f64(got), ref, R.U[dt] * np.abs(ref) + R.TINY[dt] + (m + 1) * 2 * EPS * np.abs(t3).sum(1), name)

    dout = rows_tensor(rng, n, d, t, pad, False)
    dz, dzbuf = padded(rows, d, t, pad, 5.0)
    _, dg = experts.combine_backward(dout, z, g, r, dz=dz)
    do = R.f64(dout)
    ref = do[entry[:total] // m] * gamma.reshape(-1)[entry[:total]].astype(np.float64)[:, None]
    R.close(R.f64(dz[:total]), ref, (R.U[dt] * 1.01 + EPS) * np.abs(ref) + R.TINY[dt], "dz")
    untouched(dzbuf, d, total, 5.0)
    prod = terms * do[:, None, :]
    R.close(R.f64(dg), prod.sum(-1), (d + 1) * EPS * np.abs(prod).sum(-1), "dgamma")
    only_z = experts.combine_backward(dout, None, g, r, need=(True, False))
    only_g = experts.combine_backward(dout, z, g, r, need=(False, True))
    assert only_z[1] is None and only_g[0] is None
    assert torch.equal(only_z[0][:total], dz[:total]) and torch.equal(only_g[1], dg)


def test_rows_nonfinite():
    """Infinities and NaN travel with their own rows only; a point in no list gets zero."""
    idx = np.array([[0, 1], [1, -1], [-1, -1], [0, 1]], dtype=np.int32)
    r = routes_of(idx, 2)
    z = torch.ones((8, 16), device="cuda")
    slot = R.lists(idx, 2)[2]
    z[slot[0, 1], 3] = float("inf")
    z[slot[3, 0], 5] = float("nan")
    z[5:] = float("nan")              # rows in no list
    out = experts.combine(z, torch.ones((4, 2), device="cuda"), r).cpu()
    want = torch.tensor([2.0, 1.0, 0.0, 2.0])[:, None].expand(4, 16).clone()
    want[0, 3], want[3, 5] = float("inf"), float("nan")
    assert torch.equal(torch.nan_to_num(out, nan=-7.0), torch.nan_to_num(want, nan=-7.0))
    back = experts.dispatch_backward(z, r).cpu()
    assert torch.equal(back[2], torch.zeros(16)) and back[0, 3] == float("inf")


# --- linear models --------------------------------------------------------------
LINEAR = [   # n, m, k, d_in, d_out, dtype, pad
    (1, 1, 1, 1, 1, "f32", 0), (1, 2, 16, 64, 64, "bf16", 0), (1, 2, 16, 1024, 512, "f16", 0),
    (1, 16, 4096, 8, 8, "f16", 0), (3, 2, 4, 128, 130, "f32", 0), (16, 2, 3, 200, 72, "bf16", 8),
    (33, 1, 2, 77, 130, "f32", 3), (100, 2, 65, 16, 24, "f16", 0), (129, 1, 1, 128, 128, "bf16", 0),
    (500, 3, 7, 77, 93, "f16", 1), (1000, 2, 16, 64, 64, "f32", 0), (1000, 2, 5, 264, 136, "bf16", 0),
    (2731, 3, 300, 40, 56, "f16", 0), (4000, 1, 2, 31, 257, "bf16", 0), (6000, 2, 3, 136, 72, "f32", 4),
    (3, 1, 3, 25, 1557, "f32", 0), (2, 8, 17, 72, 1030, "bf16", 0), (5, 2, 40, 264, 1024, "f16", 3),
    (60, 4, 9, 77, 600, "f32", 0), (150, 2, 90, 200, 640, "f32", 0), (1200, 1, 70, 64, 131, "f32", 1),
    (900, 3, 6, 131, 128, "bf16", 0), (900, 3, 6, 136, 77, "f16", 0),
    (700, 2, 3, 3, 130, "f32", 0), (700, 2, 3, 130, 2, "f32", 1), (900, 1, 2, 5, 7, "bf16", 0),
    (900, 3, 4, 200, 3, "f16", 0), (4, 2, 3, 3, 50, "f16", 5), (10, 2, 3, 2, 33, "f32", 0),
]


@pytest.mark.parametrize("whole", [True, False], ids=["whole", "normal"])
@pytest.mark.parametrize("n,m,k,di,do,dt,pad", LINEAR)
def test_linear(n, m, k, di, do, dt, pad, whole):
    rng = np.random.default_rng(n * 7 + di)
    idx = R.assignment(n, m, k, rng, repeats=k < m)
    off, entry, slot = R.lists(idx, k)
    total, rows = off[-1], n * m
    r, t = routes_of(idx, k), R.DT[dt]
    x = rows_tensor(rng, n, di, t, pad, whole)
    w = rows_tensor(rng, k * do, di, t, 0, whole).reshape(k, do, di).contiguous()
    b = dev((rng.integers(-3, 4, size=(k, do)) if whole else rng.standard_normal((k, do))).astype(np.float32))
    dy = rows_tensor(rng, rows, do, t, pad, whole)
    y, ybuf = padded(rows, do, t, pad, 9.0)
    experts.linear(x, w, b, r, out=y)
    dx, dxbuf = padded(rows, di, t, pad, 5.0)
    _, dw, db = experts.linear_backward(dy, x, w, r, dx=dx)
    # rows by slot instead of the points' rows: the same numbers, bit for bit
    xs = experts.dispatch(x, r)
    assert torch.equal(experts.linear(xs, w, b, r, sorted_rows=True)[:total], y[:total])
    _, dws, dbs = experts.linear_backward(dy, xs, w, r, sorted_rows=True, need=(False, True, True))
    assert torch.equal(dws, dw) and torch.equal(dbs, db)
    no_bias = experts.linear(x, w, None, r)
    untouched(ybuf, do, total, 9.0)
    untouched(dxbuf, di, total, 5.0)
    X, W, B, DY = R.f64(x), R.f64(w), R.f64(b), R.f64(dy)
    once = lambda a: R.f64(torch.from_numpy(a).to(t))   # noqa: E731
    for kk in range(k):
        s = slice(off[kk], off[kk + 1])
        xk, dyk = X[entry[s] // m], DY[s]
        prod = xk @ W[kk].T
        ref, ref_x = prod + B[kk], dyk @ W[kk]
        ref_w, ref_b = dyk.T @ xk, dyk.sum(0)
        if whole:
            # sums stay below 2^24: exact in fp32, one rounding in the store
            assert np.array_equal(R.f64(y[s]), once(ref)) and np.array_equal(R.f64(no_bias[s]), once(prod))
            assert np.array_equal(R.f64(dx[s]), once(ref_x))
            assert np.array_equal(R.f64(dw[kk]), ref_w) and np.array_equal(R.f64(db[kk]), ref_b)
            continue
        at = np.abs(xk) @ np.abs(W[kk]).T
        R.close(R.f64(y[s]), ref, R.U[dt] * np.abs(ref) * 1.01 + R.TINY[dt] + (di + 2) * EPS * (at + np.abs(B[kk])), "y")
        R.close(R.f64(dx[s]), ref_x, R.U[dt] * np.abs(ref_x) * 1.01 + R.TINY[dt] +
                (do + 1) * EPS * (np.abs(dyk) @ np.abs(W[kk])), "dx")
        c = xk.shape[0]
        R.close(R.f64(dw[kk]), ref_w, (c + 1) * EPS * (np.abs(dyk).T @ np.abs(xk)), "dw")
        R.close(R.f64(db[kk]), ref_b, (c + 1) * EPS * np.abs(dyk).sum(0), "db")


@pytest.mark.parametrize("n,m,k,di,do,dt", [
    (33_000, 2, 5, 520, 264, "bf16"), (70_000, 1, 3, 264, 776, "f16"), (20_000, 2, 40, 1032, 512, "bf16"),
    (9_000, 2, 2, 512, 512, "f32"), (50_000, 2, 7, 77, 130, "f32"), (30_000, 1, 4, 300, 258, "bf16")])
def test_linear_large(n, m, k, di, do, dt):
    """Sizes whose tiles fill the GPU, lists of several chunks: whole numbers, exact sums, against
    fp64 products on the GPU."""
    rng = np.random.default_rng(di)
    idx = R.assignment(n, m, k, rng, repeats=k < m)
    idx[: n // 3, 0] = k - 1          # one long list
    off, entry, slot = R.lists(idx, k)
    r, t = routes_of(idx, k), R.DT[dt]
    gen = torch.Generator(device="cuda").manual_seed(di)
    whole = lambda *s: torch.randint(-2, 3, s, generator=gen, device="cuda")   # noqa: E731
    x, w, dy, b = whole(n, di).to(t), whole(k, do, di).to(t), whole(n * m, do).to(t), whole(k, do).float()
    y = experts.linear(x, w, b, r)
    dx, dw, db = experts.linear_backward(dy, x, w, r)
    point = torch.from_numpy(np.maximum(entry, 0) // m).cuda()
    for kk in range(k):
        s = slice(off[kk], off[kk + 1])
        xk, dyk, wk = x[point[s]].double(), dy[s].double(), w[kk].double()
        assert torch.equal(y[s], (xk @ wk.t().contiguous() + b[kk].double()).to(t)), (kk, "y")
        assert torch.equal(dx[s], (dyk @ wk).to(t)), (kk, "dx")
        assert torch.equal(dw[kk].double(), dyk.t().contiguous() @ xk), (kk, "dw")
        assert torch.equal(db[kk].double(), dyk.sum(0)), (kk, "db")


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_linear_nonfinite_rows(dt):
    """A non-finite row touches its own outputs and its own list's gradient
    only; the rows behind the last list are never read."""
    n, m, k, d = 300, 2, 3, 64
    rng = np.random.default_rng(3)
    idx = R.assignment(n, m, k, rng, holes=0.3)
    off, entry, slot = R.lists(idx, k)
    r, t = routes_of(idx, k), R.DT[dt]
    x = rows_tensor(rng, n, d, t, 0, True)
    w = rows_tensor(rng, k * d, d, t, 0, True).reshape(k, d, d).contiguous()
    dy = rows_tensor(rng, n * m, d, t, 0, True)
    clean = experts.linear(x, w, None, r), *experts.linear_backward(dy, x, w, r)
    s = off[1] - 1                    # the last row of list 0, beside list 1's first
    dy[off[-1]:] = float("nan")
    dy[s, 5] = float("inf")
    x[entry[s] // m, 7] = float("nan")
    y, dx, dw, db = experts.linear(x, w, None, r), *experts.linear_backward(dy, x, w, r)
    assert db[0, 5] == float("inf")
    db[0, 5] = clean[3][0, 5]
    assert torch.equal(db, clean[3])
    hit = np.unique(slot[entry[s] // m])
    same = np.setdiff1d(np.arange(off[-1]), hit)
    assert torch.equal(y[same], clean[0][same]) and torch.isnan(y[hit[hit >= 0]]).all()
    same = np.setdiff1d(np.arange(off[-1]), [s])
    assert torch.equal(dx[same], clean[1][same]) and not torch.isfinite(dx[s]).any()
    lists_hit = np.unique(np.searchsorted(off, hit[hit >= 0], side="right") - 1)
    for kk in np.setdiff1d(np.arange(k), lists_hit):
        assert torch.equal(dw[kk], clean[2][kk])


def test_gradients_against_differences():
    """<dout, combine(linear(x))> is linear in each of x, w, b and gamma, so a
    central difference over any step is its derivative up to rounding; whole
    numbers make both sides exact."""
    n, m, k, di, do = 40, 3, 5, 12, 20
    rng = np.random.default_rng(11)
    idx = R.assignment(n, m, k, rng)
    r = routes_of(idx, k)
    whole = lambda *s: dev(rng.integers(-2, 3, size=s).astype(np.float32))   # noqa: E731
    x, w, b, gamma, dout = whole(n, di), whole(k, do, di), whole(k, do), whole(n, m), whole(n, do)

    def value(x, w, b, gamma):
        return (experts.combine(experts.linear(x, w, b, r), gamma, r).double() * dout.double()).sum().item()

    y = experts.linear(x, w, b, r)
    dy, dgamma = experts.combine_backward(dout, y, gamma, r)
    dxs, dw, db = experts.linear_backward(dy, x, w, r)
    grads = {"x": experts.dispatch_backward(dxs, r), "w": dw, "b": db, "gamma": dgamma}
    args = {"x": x, "w": w, "b": b, "gamma": gamma}
    for name, grad in grads.items():
        for _ in range(6):
            step = whole(*args[name].shape)
            up = value(**{**args, name: args[name] + step})
            down = value(**{**args, name: args[name] - step})
            live = grad if name != "gamma" else torch.where(r.slot >= 0, grad, 0.0)
            assert (up - down) / 2 == (live.double() * step.double()).sum().item(), name


# --- 4-bit models -----------------------------------------------------------------
@pytest.mark.parametrize("rows,d,group,dt", [(1, 1, 32, "f32"), (5, 128, 128, "bf16"), (33, 77, 32, "f16"),
                                             (100, 1024, 64, "f32"), (64, 130, 128, "bf16"), (7, 4095, 32, "f16")])
def test_quantize4(rows, d, group, dt):
    rng = np.random.default_rng(d)
    w = rng.standard_normal((rows, d)).astype(np.float32) * 10.0 ** rng.integers(-3, 2, size=(rows, 1))
    w[0] = 0.0
    if rows > 4:
        w[3, :group] = 1e-30 if dt != "f16" else 6e-8
    wt = torch.from_numpy(w.astype(np.float32)).to(R.DT[dt])
    codes, scales = experts.quantize4(wt.cuda(), group)
    rc, rs = R.quantize4(wt.float().numpy(), group)
    assert np.array_equal(scales.float().cpu().numpy(), rs)
    assert np.array_equal(codes.cpu().numpy(), rc)
    # every weight is within half a code step of its decoded value (one step where it is clamped)
    back = R.decode4(rc, rs.astype(np.float64), group, d)
    s = np.repeat(rs, group, -1)[:, :d]
    assert (np.abs(back - wt.double().numpy()) <= s * 0.5001 + 1e-45).all()


def test_quantize4_nonfinite():
    w = torch.ones((3, 64), device="cuda")
    w[0, 3], w[1, 40] = float("nan"), float("inf")
    codes, scales = experts.quantize4(w, 32)
    assert torch.isnan(scales.float()).cpu().tolist() == [[True, False], [False, True], [False, False]]
    assert (codes[0, :16] == 0x88).all() and (codes[1, 16:] == 0x88).all()


LINEAR4 = [   # n, m, k, d_in, d_out, group, dtype
    (1, 1, 1, 1, 1, 32, "f32"), (1, 2, 16, 256, 100, 128, "bf16"), (1, 8, 8, 4096, 64, 128, "f16"),
    (5, 3, 7, 77, 93, 32, "f16"), (24, 4, 64, 128, 256, 64, "bf16"), (32, 2, 3, 130, 31, 64, "f32"),
    (33, 16, 20, 96, 48, 32, "bf16"), (100, 2, 4, 512, 40, 32, "f16"), (3, 2, 4, 1056, 17, 128, "f32"),
    (1024, 1, 2, 32, 8, 32, "bf16"), (16, 16, 100, 1024, 32, 32, "f16"), (9, 2, 5, 4128, 20, 64, "bf16"),
    (2, 1, 3, 8192, 17, 64, "f16"), (1, 1, 2, 40_000, 5, 32, "bf16"), (1, 2, 3, 2050, 33, 128, "f32"),
]


@pytest.mark.parametrize("with_bias", [True, False], ids=["bias", "plain"])
@pytest.mark.parametrize("n,m,k,di,do,group,dt", LINEAR4)
def test_linear4(n, m, k, di, do, group, dt, with_bias):
    rng = np.random.default_rng(n + di)
    idx = R.assignment(n, m, k, rng, holes=0.2, repeats=k < m)
    x = rows_tensor(rng, n, di, R.DT[dt], 0, False)
    gamma = rng.random((n, m)).astype(np.float32)
    gamma[idx < 0] = np.nan
    codes = rng.integers(0, 256, size=(k, do, (di + 1) // 2)).astype(np.uint8)
    scales = torch.from_numpy(rng.uniform(0.01, 0.1, size=(k, do, -(-di // group)))).to(torch.bfloat16)
    bias = rng.standard_normal((k, do)).astype(np.float32) if with_bias else None
    got = experts.linear4(x, dev(idx), dev(gamma), dev(codes), scales.cuda(), group,
                          bias=dev(bias) if with_bias else None)
    W = R.decode4(codes, scales.double().numpy(), group, di)
    X = R.f64(x)
    ref, size = np.zeros((n, do)), np.zeros((n, do))
    for i in range(m):
        on = idx[:, i] >= 0
        wk, g = W[idx[on, i]], gamma[on, i].astype(np.float64)[:, None]
        bk = bias[idx[on, i]].astype(np.float64) if with_bias else 0.0
        ref[on] += g * (np.einsum("noj,nj->no", wk, X[on]) + bk)
        size[on] += g * (np.einsum("noj,nj->no", np.abs(wk), np.abs(X[on])) + np.abs(bk))
    # the codes' products run before the offset of 8 is taken off or after: up to 136 / 8 = 17 times the terms
    R.close(R.f64(got), ref, R.U[dt] * np.abs(ref) * 1.01 + R.TINY[dt] + 18 * (di + 4) * EPS * size, "linear4")


def test_linear4_foreign_components():
    """Components outside [0, k) are skipped; a point without any gets zero;
    one component twice counts twice."""
    k, di, do = 4, 64, 32
    rng = np.random.default_rng(5)
    x = rows_tensor(rng, 4, di, torch.float32, 0, True)
    idx = np.array([[0, k], [-1, -2 ** 31], [2, 2], [2 ** 31 - 1, 3]], dtype=np.int32)
    gamma = torch.ones((4, 2), device="cuda")
    codes = dev(rng.integers(0, 256, size=(k, do, di // 2)).astype(np.uint8))
    scales = torch.ones((k, do, 2), dtype=torch.bfloat16, device="cuda")
    got = R.f64(experts.linear4(x, dev(idx), gamma, codes, scales, 32))
    y = np.einsum("koj,nj->kno", R.decode4(codes.cpu().numpy(), np.ones((k, do, 2)), 32, di), R.f64(x))
    assert np.array_equal(got, np.stack([y[0, 0], np.zeros(do), 2 * y[2, 2], y[3, 3]]))


def test_linear4_nonfinite():
    """A component with a NaN scale and a point with a NaN or an infinity touch only
    the points that list the one and the rows of the other."""
    n, m, k, di, do = 12, 2, 5, 256, 40
    rng = np.random.default_rng(1)
    for dt in ("f32", "bf16", "f16"):
        idx = R.assignment(n, m, k, rng)
        idx[0], idx[1], idx[2] = (3, 4), (0, 1), (2, 0)
        x = rows_tensor(rng, n, di, R.DT[dt], 0, True)
        gamma = torch.ones((n, m), device="cuda")
        codes = dev(rng.integers(0, 256, size=(k, do, di // 2)).astype(np.uint8))
        scales = torch.ones((k, do, di // 32), dtype=torch.bfloat16, device="cuda")
        clean = experts.linear4(x, dev(idx), gamma, codes, scales, 32)
        scales[3, 7, 1] = float("nan")
        x[1, 5], x[2, 9] = float("nan"), float("inf")
        got = experts.linear4(x, dev(idx), gamma, codes, scales, 32)
        hit = (idx == 3).any(1)
        rows = [p for p in range(n) if p not in (1, 2)]
        cols = [c for c in range(do) if c != 7]
        assert torch.equal(got[rows][:, cols], clean[rows][:, cols])
        assert torch.equal(torch.isnan(got[rows, 7]).cpu(), torch.from_numpy(hit[rows]))
        assert not torch.isfinite(got[1]).any() and not torch.isfinite(got[2]).any()


# --- together -----------------------------------------------------------------------
@pytest.mark.parametrize("cov,dt", [("diag", "f32"), ("iso", "bf16"), ("full", "f16")])
def test_mixture_then_models(cov, dt):
    """Fit a mixture, assign, route, apply the components' models and combine; the
    gradients of the models and of the responsibilities; then the same points on 4-bit models."""
    from soft_clustering_amd import gmm
    n, d, k, m, do = 3000, 32, 12, 2, 48
    rng = np.random.default_rng(2)
    mu = rng.uniform(-4, 4, size=(k, d))
    x = dev((mu[rng.integers(0, k, n)] + rng.standard_normal((n, d))).astype(np.float32), R.DT[dt])
    g = gmm.Gmm(n, d, k, cov, dt)
    pi, mean = torch.empty(k, device="cuda"), torch.empty((k, d), device="cuda")
    var = torch.empty(g.cov_shape, device="cuda")
    g.fit(x, pi, mean, var, max_iter=5, init="random_points", seed=4, use_graph=False)
    idx, gamma = g.assign(x, m)
    routes = experts.route(idx, k)
    w = dev(rng.standard_normal((k, do, d)).astype(np.float32) / 6, R.DT[dt])
    b = dev(rng.standard_normal((k, do)).astype(np.float32))
    y = experts.linear(x, w, b, routes)
    out = experts.combine(y, gamma, routes)
    I, G, X, W, B = idx.cpu().numpy(), R.f64(gamma), R.f64(x), R.f64(w), R.f64(b)
    off, entry, slot = R.lists(I, k)
    assert np.array_equal(routes.entry.cpu().numpy(), entry) and (I[:, 0] >= 0).all()
    terms = np.where((I >= 0)[..., None], np.einsum("nmoj,nj->nmo", W[I], X) + B[I], 0.0)
    size = np.where((I >= 0)[..., None], np.einsum("nmoj,nj->nmo", np.abs(W)[I], np.abs(X)) + np.abs(B)[I], 0.0)
    ref, top = (G[..., None] * terms).sum(1), (G[..., None] * size).sum(1)
    # y is stored once, out once more
    R.close(R.f64(out), ref, 2.1 * R.U[dt] * top + (d + 6) * EPS * top + 3 * R.TINY[dt], "out")
    dout = dev(rng.standard_normal((n, do)).astype(np.float32), R.DT[dt])
    dy, dgamma = experts.combine_backward(dout, y, gamma, routes)
    dxs, dw, db = experts.linear_backward(dy, x, w, routes)
    dx = experts.dispatch_backward(dxs, routes)
    DO = R.f64(dout)
    R.close(R.f64(dgamma), np.einsum("nmo,no->nm", terms, DO),
            (1.01 * R.U[dt] + (do + d + 6) * EPS) * np.einsum("nmo,no->nm", size, np.abs(DO)) + do * R.TINY[dt] * 10, "dgamma")
    DY = G[..., None] * DO[:, None, :]
    ref_x, top_x = np.einsum("nmo,nmoj->nj", DY, W[I]), np.einsum("nmo,nmoj->nj", np.abs(DY), np.abs(W)[I])
    R.close(R.f64(dx), ref_x, 3.1 * R.U[dt] * top_x + (do + 6) * EPS * top_x + 40 * R.TINY[dt], "dx")
    for kk in range(k):
        e = entry[off[kk]:off[kk + 1]]
        dyk, xk = DY.reshape(-1, do)[e], X[e // m]
        top_w = np.abs(dyk).T @ np.abs(xk)
        R.close(R.f64(dw[kk]), dyk.T @ xk, (1.01 * R.U[dt] + (len(e) + 3) * EPS) * top_w +
                R.TINY[dt] * np.abs(xk).sum(0), "dw")
        R.close(R.f64(db[kk]), dyk.sum(0), (1.01 * R.U[dt] + (len(e) + 3) * EPS) * np.abs(dyk).sum(0) +
                R.TINY[dt] * len(e), "db")
    codes, scales = experts.quantize4(w, 32)
    few = slice(0, 20)
    got = experts.linear4(x[few], idx[few].contiguous(), gamma[few].contiguous(), codes, scales, 32, bias=b)
    W4 = R.decode4(codes.cpu().numpy(), R.f64(scales), 32, d)
    ref = (G[few, :, None] * (np.einsum("nmoj,nj->nmo", W4[I[few]], X[few]) + B[I[few]])).sum(1)
    R.close(R.f64(got), ref, 1.01 * R.U[dt] * np.abs(ref) + 18 * (d + 4) * EPS * top[few] * 1.2 + R.TINY[dt], "linear4")


def _all_outputs(x, idx, gamma, w, b, dout, codes, scales, k, stream=None):
    r = experts.route(idx, k, stream=stream)
    y = experts.linear(x, w, b, r, stream=stream)
    out = experts.combine(y, gamma, r, stream=stream)
    dy, dg = experts.combine_backward(dout, y, gamma, r, stream=stream)
    dxs, dw, db = experts.linear_backward(dy, x, w, r, stream=stream)
    dx = experts.dispatch_backward(dxs, r, stream=stream)
    o4 = experts.linear4(x[:30], idx[:30], gamma[:30], codes, scales, 32, bias=b, stream=stream)
    return [r.offsets, r.entry, r.slot, out, dg, dw, db, dx, o4]


def _inputs(n, m, k, di, do, dt, seed):
    rng = np.random.default_rng(seed)
    t = R.DT[dt]
    idx = dev(R.assignment(n, m, k, rng))
    w = dev(rng.standard_normal((k, do, di)).astype(np.float32), t)
    return (dev(rng.standard_normal((n, di)).astype(np.float32), t), idx, dev(rng.random((n, m)).astype(np.float32)), w,
            dev(rng.standard_normal((k, do)).astype(np.float32)), dev(rng.standard_normal((n, do)).astype(np.float32), t),
            *experts.quantize4(w, 32), k)


@pytest.mark.parametrize("n", [200, 9000])
def test_other_stream_and_graph(n):
    """On a stream of its own, and captured and replayed with new inputs
    between the replays: the eager results, bit for bit."""
    a, b = (_inputs(n, 2, 9, 64, 96, "bf16", s) for s in (1, 2))
    want = {0: _all_outputs(*a), 1: _all_outputs(*b)}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = _all_outputs(*a, stream=side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want[0]))
    held = [t.clone() if torch.is_tensor(t) else t for t in a]
    graphs = []
    for _ in range(2):                    # two graphs of the same calls
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = _all_outputs(*held)
        graphs.append((graph, outs))
    for turn in (1, 0, 1, 1, 0):
        for t, new in zip(held, (a, b)[turn]):
            if torch.is_tensor(t):
                t.copy_(new)
        for graph, outs in graphs:
            graph.replay()
        eager = _all_outputs(*(a, b)[1 - turn])     # the program's own work between
        torch.cuda.synchronize()
        total = int(want[turn][0][-1])
        for graph, outs in graphs:
            assert all(torch.equal(p, q) for p, q in zip(outs, want[turn])), (turn, total)
        assert all(torch.equal(p, q) for p, q in zip(eager, want[1 - turn]))


def test_no_points():
    """n = 0: empty rows, zero gradients of the weights."""
    r = experts.route(torch.empty((0, 2), dtype=torch.int32, device="cuda"), 3)
    x, z = torch.empty((0, 16), device="cuda"), torch.empty((0, 24), device="cuda")
    w, g = torch.ones((3, 24, 16), device="cuda"), torch.empty((0, 2), device="cuda")
    assert experts.dispatch(x, r).shape == (0, 16) and experts.combine(z, g, r).shape == (0, 24)
    assert experts.linear(x, w, None, r).shape == (0, 24)
    dx, dw, db = experts.linear_backward(z, x, w, r)
    assert dx.shape == (0, 16) and not dw.any() and not db.any()
    idx = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    codes, scales = experts.quantize4(w, 32)
    assert experts.linear4(x, idx, g, codes, scales, 32).shape == (0, 24)


def test_offsets_past_32_bits():
    """Rows whose bytes pass 4 GiB, there and back; every 997th point against its own rows."""
    n, m, k, d = 9_000_000, 2, 7, 128
    gen = torch.Generator(device="cuda").manual_seed(1)
    idx = torch.randint(0, k, (n, m), generator=gen, device="cuda", dtype=torch.int32)
    x = torch.randint(-3, 4, (n, d), generator=gen, device="cuda").to(torch.bfloat16)
    gamma = torch.ones((n, m), device="cuda")
    r = experts.route(idx, k)
    y = experts.dispatch(x, r)
    assert y.numel() * y.element_size() > 1 << 32
    some = torch.cat([torch.arange(0, n, 997, device="cuda"), torch.arange(n - 50, n, device="cuda")])
    at = r.slot[some].long()
    assert torch.equal(y[at[:, 0]], x[some]) and torch.equal(y[at[:, 1]], x[some])
    assert torch.equal(experts.combine(y, gamma, r)[some], 2 * x[some])
    w = torch.randint(-2, 3, (k, d, d), generator=gen, device="cuda").to(torch.bfloat16)
    z = experts.linear(x, w, None, r, out=y)
    ref = torch.stack([x[some].double() @ w[kk].double().t().contiguous() for kk in range(k)])
    for i in range(m):
        want = ref[idx[some, i].long(), torch.arange(len(some), device="cuda")]
        assert torch.equal(z[at[:, i]], want.to(torch.bfloat16))
    dx = experts.linear_backward(z, None, w, r, need=(True, False, False))[0]
    want = torch.stack([z[at[:, 0]].double() @ w[kk].double() for kk in range(k)])
    want = want[idx[some, 0].long(), torch.arange(len(some), device="cuda")]
    # 128 products of whole numbers, at most 768 x 2 each: exact in fp32
    assert torch.equal(dx[at[:, 0]], want.to(torch.bfloat16))


def test_refused_tensors():
    """Wrong types, shapes, strides and devices are refused before anything runs."""
    x, idx, gamma, w, b, dout, codes, scales, k = _inputs(10, 2, 3, 16, 24, "f32", 1)
    r = experts.route(idx, k)
    y = experts.linear(x, w, b, r)
    bad = [
        lambda: experts.route(idx.long(), k), lambda: experts.route(idx.cpu(), k), lambda: experts.route(idx.t(), k),
        lambda: experts.dispatch(x[:9], r), lambda: experts.dispatch(x.double(), r), lambda: experts.dispatch(x.cpu(), r),
        lambda: experts.dispatch(x.t().contiguous().t(), r), lambda: experts.dispatch(x[:1].expand(10, 16), r),
        lambda: experts.combine(y, gamma.half(), r), lambda: experts.combine(y, None, r),
        lambda: experts.combine(y, gamma, r, out=torch.empty((10, 23), device="cuda")),
        lambda: experts.linear(x, w.half(), b, r), lambda: experts.linear(x, w[:2], b, r),
        lambda: experts.linear(x, w, b.half(), r), lambda: experts.linear(x, w.transpose(1, 2), b, r),
        lambda: experts.linear_backward(y, x, w, r, need=(True, False, True)),
        lambda: experts.linear_backward(y[:5], x, w, r),
        lambda: experts.combine_backward(dout, None, gamma, r),
        lambda: experts.combine_backward(dout, y, gamma, r, dz=y), lambda: experts.linear(x, w, b, r, out=x),
        lambda: experts.linear4(x, idx, gamma, codes, scales, 48), lambda: experts.linear4(x, idx, gamma, codes, scales, 16),
        lambda: experts.linear4(x, idx, gamma, codes[:, :, :3], scales, 32),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was not refused")
    for f in (lambda: experts.route(idx, 0), lambda: experts.route(idx, 4097),
              lambda: experts.route(torch.zeros((2, 17), dtype=torch.int32, device="cuda"), 3),
              lambda: experts.quantize4(w, 48)):
        with pytest.raises(experts.GmmError):
            f()
