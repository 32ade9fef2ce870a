"""What the operators behind the soft assignment are measured on.

A mixture whose components each own a linear model: `gmm.Gmm.assign` lists the
m most responsible components of every point and their responsibilities, and
the operators of `soft_clustering_amd.experts` take the points from there:

  route     the lists of the components: the points that list each of them
  dispatch  the rows of the lists, and the gradient of that gather
  combine   the rows back at their points, weighted and summed, with gradients
  linear    y = W_k x + b_k on every row of list k, with gradients
  linear4   the same on 4-bit weights with group scales, weighted and summed,
            for one point or a few

`run` computes them in plain torch operations, or (`own`) through the library.
The layouts are the library's: entry e = point * m + column; offsets[k] ..
offsets[k + 1] are the slots of list k, entry[s] the entry in slot s (lists
keep the order of the entries), slot[e] its place or -1.
"""
import math

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
DEV = "cuda"


def listed():
    return [
        # one serving batch sent to the 16 components of the small mixtures: latency
        {"name": "route-batch", "op": "route", "n": 48, "m": 2, "k": 16},
        # the inverted lists of 1e7 points in two of 256 clusters each
        {"name": "route-lists-1e7", "op": "route", "n": 10_000_000, "m": 2, "k": 256},
        # the rows of a million fp32 points laid out by list, each in two lists
        {"name": "dispatch-1e6-d64-f32", "op": "dispatch", "dir": "fwd", "n": 1_000_000, "m": 2, "k": 16,
         "d": 64, "dtype": "f32"},
        # its gradient, at an odd width (rows of 186 bytes, no vector loads)
        {"name": "dispatch-back-odd", "op": "dispatch", "dir": "bwd", "n": 50_021, "m": 3, "k": 100,
         "d": 93, "dtype": "f16"},
        # one serving batch put together again: latency
        {"name": "combine-batch-bf16", "op": "combine", "dir": "fwd", "n": 48, "m": 2, "k": 16,
         "d": 128, "dtype": "bf16"},
        # a training step's way back over a million points, gradients of rows and weights
        {"name": "combine-back-1e6-bf16", "op": "combine", "dir": "bwd", "n": 1_000_000, "m": 2, "k": 256,
         "d": 128, "dtype": "bf16"},
        # one point through two of 16 wide linear models: the weights' bytes and latency
        {"name": "linear-point-bf16", "op": "linear", "dir": "fwd", "n": 1, "m": 2, "k": 16,
         "d_in": 1024, "d_out": 1024, "dtype": "bf16"},
        # a local map of every cluster applied to a million points, each in two lists: bandwidth
        {"name": "linear-1e6-d128-f16", "op": "linear", "dir": "fwd", "n": 1_000_000, "m": 2, "k": 256,
         "d_in": 128, "d_out": 128, "dtype": "f16"},
        # the gradients of a training batch through wide models: matrix rate
        {"name": "linear-back-bf16", "op": "linear", "dir": "bwd", "n": 16_384, "m": 2, "k": 64,
         "d_in": 1024, "d_out": 2048, "dtype": "bf16"},
        # ragged lists, odd widths, fp32 storage
        {"name": "linear-back-odd-f32", "op": "linear", "dir": "bwd", "n": 20_011, "m": 3, "k": 37,
         "d_in": 77, "d_out": 130, "dtype": "f32"},
        # one point through two wide models in 4 bits: the codes' bytes and latency
        {"name": "linear4-point-bf16", "op": "linear4", "n": 1, "m": 2, "k": 16, "d_in": 4096, "d_out": 4096,
         "group": 128, "dtype": "bf16"},
        # a few points whose lists overlap
        {"name": "linear4-batch-f16", "op": "linear4", "n": 24, "m": 4, "k": 64, "d_in": 1024, "d_out": 2048,
         "group": 64, "dtype": "f16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["route", "dispatch", "combine", "linear", "linear4"])
    c = {"op": op}
    k = _log_int(rng, 1, 1024)
    m = min(k, rng.choice([1, 2, 2, 3, 4, 7, 8, 16]))
    if op == "route":
        c |= {"n": _log_int(rng, 1, 20_000_000 // m), "m": m, "k": min(4096, k * rng.choice([1, 1, 4]))}
    elif op in ("dispatch", "combine"):
        d = rng.choice([_log_int(rng, 1, 1024), 8 * _log_int(rng, 1, 128)])
        c |= {"dir": rng.choice(["fwd", "bwd"]), "n": _log_int(rng, 1, max(1, 100_000_000 // (m * d))), "m": m, "k": k,
              "d": d, "dtype": rng.choice(["f32", "bf16", "f16"])}
    elif op == "linear":
        k = min(k, 256)
        m = min(m, k)
        d_in, d_out = (rng.choice([_log_int(rng, 1, 2048), 8 * _log_int(rng, 1, 256)]) for _ in range(2))
        k = max(m, min(k, 100_000_000 // (d_in * d_out)))
        dtype = rng.choice(["f32", "bf16", "f16"])
        way = rng.choice(["fwd", "bwd"])
        # fp32 products run at a sixteenth of the 16-bit rate
        most = 2.5e11 / (16 if dtype == "f32" else 1) / (2.0 * d_in * d_out * m * (2 if way == "bwd" else 1))
        c |= {"dir": way, "n": _log_int(rng, 1, max(1, min(int(most), 200_000_000 // (m * max(d_in, d_out))))),
              "m": m, "k": k, "d_in": d_in, "d_out": d_out, "dtype": dtype}
    else:
        group = rng.choice([32, 64, 128])
        d_in = rng.choice([_log_int(rng, 16, 4096), 32 * _log_int(rng, 1, 128)])
        d_out = _log_int(rng, 1, 4096)
        k = max(1, min(k, 64, 130_000_000 // (d_in * d_out)))
        m = min(m, k, 8)
        c |= {"n": _log_int(rng, 1, 32), "m": m, "k": k, "d_in": d_in, "d_out": d_out, "group": group,
              "dtype": rng.choice(["f32", "bf16", "f16"])}
    return c


# --- inputs -------------------------------------------------------------------
def _assignment(n, m, k, gen, rng):
    """Top-m lists as gmm_assign writes them: distinct components per point, by popularity; unlisted
    columns (-1, weight 0) at the end of a few rows; a few rows with none."""
    pop = torch.tensor(rng.dirichlet(np.ones(k)), dtype=torch.float64, device=DEV).cumsum(0)
    u = torch.rand(n, generator=gen, device=DEV, dtype=torch.float64) * pop[-1]
    first = torch.searchsorted(pop, u).clamp_(max=k - 1)
    cols = [first]
    step = max(1, (k - 1) // max(1, m - 1))
    for i in range(1, m):   # m - 1 further components, distinct: steps of 1 .. step around the circle
        cols.append(cols[-1] + torch.randint(1, step + 1, (n,), generator=gen, device=DEV))
    idx = torch.stack(cols, 1).remainder_(k).to(torch.int32)
    e = torch.empty((n, m), device=DEV).exponential_(1.0, generator=gen).sort(1, descending=True).values
    gamma = e / (e.sum(1, keepdim=True) + 0.05)
    cut = torch.rand((n, m), generator=gen, device=DEV)
    gone = torch.cat([cut[:, :1] < 0.002, cut[:, 1:] < 0.02], 1).cummax(1).values if m > 1 else cut < 0.002
    return idx.masked_fill_(gone, -1).contiguous(), gamma.masked_fill_(gone, 0.0).contiguous()


def _lists(idx, k):
    """The lists of an assignment, in plain torch."""
    flat = idx.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < k), flat, torch.full_like(flat, k))
    key, entry = torch.sort(key, stable=True)
    offsets = torch.searchsorted(key, torch.arange(k + 1, device=key.device)).to(torch.int32)
    listed_ = key < k
    places = torch.arange(key.numel(), device=key.device)
    slot = torch.empty_like(key).scatter_(0, entry, torch.where(listed_, places, -1))
    entry = torch.where(listed_, entry, -1)
    return offsets, entry.to(torch.int32), slot.to(torch.int32).reshape(idx.shape)


def _points(n, d, idx, k, gen, dtype):
    """Points around the mean of their first component."""
    mu = 2.0 * torch.randn((k, d), generator=gen, device=DEV)
    x = torch.randn((n, d), generator=gen, device=DEV)
    return x.add_(mu[idx[:, 0].long().clamp_(min=0)]).to(DT[dtype])


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    rng = np.random.default_rng(seed)
    c, op = case, case["op"]
    n, m, k = c["n"], c["m"], c["k"]
    idx, gamma = _assignment(n, m, k, gen, rng)
    s = {"case": c, "idx": idx, "gamma": gamma}
    if op == "route":
        s |= {"offsets": torch.empty(k + 1, dtype=torch.int32, device=DEV), "entry": torch.empty_like(idx).view(-1),
              "slot": torch.empty_like(idx)}
        return s
    rows = n * m
    normal = lambda *shape: torch.randn(shape, generator=gen, device=DEV)   # noqa: E731
    if op != "linear4":
        s["offsets"], s["entry"], s["slot"] = _lists(idx, k)
    if op in ("dispatch", "combine"):
        d, t = c["d"], DT[c["dtype"]]
        if (op, c["dir"]) == ("dispatch", "fwd"):
            s |= {"x": _points(n, d, idx, k, gen, c["dtype"]), "out": torch.zeros((rows, d), dtype=t, device=DEV)}
        elif op == "dispatch":
            s |= {"dy": normal(rows, d).to(t), "out": torch.empty((n, d), dtype=t, device=DEV)}
        else:
            s |= {"z": normal(rows, d).to(t), "out": torch.zeros((rows if c["dir"] == "bwd" else n, d), dtype=t, device=DEV)}
            if c["dir"] == "bwd":
                s |= {"dout": normal(n, d).to(t), "dgamma": torch.empty_like(gamma)}
        return s
    di, do, t = c["d_in"], c["d_out"], DT[c["dtype"]]
    s |= {"x": _points(n, di, idx, k, gen, c["dtype"]), "bias": 0.1 * normal(k, do)}
    if op == "linear":
        s["w"] = normal(k, do, di).mul_(di ** -0.5).to(t)
        s["out"] = torch.zeros((rows, do if c["dir"] == "fwd" else di), dtype=t, device=DEV)
        if c["dir"] == "bwd":
            s |= {"dy": normal(rows, do).to(t), "dw": torch.empty((k, do, di), device=DEV), "db": torch.empty((k, do), device=DEV)}
        return s
    groups = -(-di // c["group"])
    s["codes"] = torch.randint(0, 256, (k, do, (di + 1) // 2), generator=gen, device=DEV, dtype=torch.uint8)
    s["scales"] = (normal(k, do, groups).abs_().add_(0.5) * (0.2 * di ** -0.5)).to(torch.bfloat16)
    s["out"] = torch.empty((n, do), dtype=t, device=DEV)
    return s


# --- the plain forms ----------------------------------------------------------
def _row_of(s):
    """Point of every slot (0 where there is none) and whether there is one."""
    there = s["entry"] >= 0
    return s["entry"].clamp(min=0).long() // s["case"]["m"], there[:, None]


def _plain_dispatch(s):
    point, there = _row_of(s)
    return (s["x"][point] * there)


def _plain_gather(z, slot):
    """The rows of every point, [n, m, d] in 32 bits, zero where a column is not listed."""
    return z.float()[slot.clamp(min=0).long()] * (slot >= 0)[..., None]


def _plain_combine_backward(s):
    dout, c = s["dout"].float(), s["case"]
    dgamma = (_plain_gather(s["z"], s["slot"]) * dout[:, None, :]).sum(-1)
    point, there = _row_of(s)
    weight = s["gamma"].view(-1)[s["entry"].clamp(min=0).long()]
    return (dout[point] * weight[:, None] * there).to(DT[c["dtype"]]), dgamma


def _list_of(s):
    """List of every slot (0 where there is none), its place in the list."""
    places = torch.arange(s["entry"].numel(), device=DEV)
    lst = torch.searchsorted(s["offsets"][1:].contiguous().long(), places, right=True)
    lst = torch.where(places < s["offsets"][-1], lst, 0)
    return lst, places - s["offsets"][lst]


def _padded(rows, lst, place, there, k, longest):
    """Rows laid out [k, longest, d] in 32 bits; the last row of the buffer takes what is in no list."""
    at = torch.where(there[:, 0], lst * longest + place, k * longest)
    buf = torch.zeros((k * longest + 1, rows.shape[1]), device=DEV)
    buf[at] = rows.float()
    return buf[:-1].view(k, longest, -1), at


def _unpadded(y, at, there):
    return torch.cat([y.reshape(-1, y.shape[-1]), y.new_zeros((1, y.shape[-1]))])[at] * there


def _plain_linear(s):
    c, t = s["case"], DT[s["case"]["dtype"]]
    point, there = _row_of(s)
    lst, place = _list_of(s)
    x = s["x"][point]
    if s["entry"].numel() < c["k"]:   # fewer rows than lists: each row's own weights
        y = torch.bmm(s["w"][lst].float(), x.float()[:, :, None])[:, :, 0] + s["bias"][lst]
        return (y * there).to(t)
    longest = int((s["offsets"][1:] - s["offsets"][:-1]).max())
    buf, at = _padded(x, lst, place, there, c["k"], longest)
    y = torch.bmm(buf, s["w"].float().transpose(1, 2)) + s["bias"][:, None, :]
    return _unpadded(y, at, there).to(t)


def _plain_linear_backward(s):
    c, t = s["case"], DT[s["case"]["dtype"]]
    point, there = _row_of(s)
    lst, place = _list_of(s)
    longest = int((s["offsets"][1:] - s["offsets"][:-1]).max())
    xs, at = _padded(s["x"][point], lst, place, there, c["k"], longest)
    dy, _ = _padded(s["dy"], lst, place, there, c["k"], longest)
    dx = torch.bmm(dy, s["w"].float())
    dw = torch.bmm(dy.transpose(1, 2).contiguous(), xs)
    return _unpadded(dx, at, there).to(t), dw, dy.sum(1)


def _plain_weights(codes, scales, group, d_in):
    """(code - 8) * scale, [..., d_out, d_in] in 32 bits; even columns in the low halves of the bytes."""
    q = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)[..., :d_in].float() - 8.0
    return q * scales.float().repeat_interleave(group, -1)[..., :d_in]


def _plain_linear4(s):
    c, t = s["case"], DT[s["case"]["dtype"]]
    n, m, k = c["n"], c["m"], c["k"]
    there = (s["idx"] >= 0)[..., None]
    at = s["idx"].clamp(min=0).long()
    x = s["x"].float()
    if n * m < k:   # fewer rows than lists: each row's own weights
        w = _plain_weights(s["codes"][at], s["scales"][at], c["group"], c["d_in"])
        y = (w.view(n, m * c["d_out"], -1) @ x[:, :, None]).view(n, m, -1)
    else:
        w = _plain_weights(s["codes"], s["scales"], c["group"], c["d_in"])
        y = (x @ w.view(k * c["d_out"], -1).t()).view(n, k, -1).gather(1, at[..., None].expand(-1, -1, c["d_out"]))
    return ((y + s["bias"][at]) * s["gamma"][..., None] * there).sum(1).to(t)


def run(s):
    c, op = s["case"], s["case"]["op"]
    back = c.get("dir") == "bwd"
    if own:
        return _own(s, op, back)
    if op == "route":
        return dict(zip(("offsets", "entry", "slot"), _lists(s["idx"], c["k"])))
    if op == "dispatch":
        return {"dx": _plain_gather(s["dy"], s["slot"]).sum(1).to(DT[c["dtype"]])} if back else {"y": _plain_dispatch(s)}
    if op == "combine":
        if back:
            return dict(zip(("dz", "dgamma"), _plain_combine_backward(s)))
        return {"out": (_plain_gather(s["z"], s["slot"]) * s["gamma"][..., None]).sum(1).to(DT[c["dtype"]])}
    if op == "linear":
        return dict(zip(("dx", "dw", "db"), _plain_linear_backward(s))) if back else {"y": _plain_linear(s)}
    return {"out": _plain_linear4(s)}


def _own(s, op, back):
    from soft_clustering_amd import experts
    if op == "route":
        r = experts.route(s["idx"], s["case"]["k"], out=experts.Routes(s["offsets"], s["entry"], s["slot"]))
        return {"offsets": r.offsets, "entry": r.entry, "slot": r.slot}
    if op == "linear4":
        return {"out": experts.linear4(s["x"], s["idx"], s["gamma"], s["codes"], s["scales"], s["case"]["group"],
                                       bias=s["bias"], out=s["out"])}
    routes = experts.Routes(s["offsets"], s["entry"], s["slot"])
    if op == "dispatch":
        if back:
            return {"dx": experts.dispatch_backward(s["dy"], routes, out=s["out"])}
        return {"y": experts.dispatch(s["x"], routes, out=s["out"])}
    if op == "combine":
        if back:
            return dict(zip(("dz", "dgamma"), experts.combine_backward(s["dout"], s["z"], s["gamma"], routes,
                                                                       dz=s["out"], dgamma=s["dgamma"])))
        return {"out": experts.combine(s["z"], s["gamma"], routes, out=s["out"])}
    if back:
        return dict(zip(("dx", "dw", "db"), experts.linear_backward(s["dy"], s["x"], s["w"], routes, dx=s["out"],
                                                                    dw=s["dw"], db=s["db"])))
    return {"y": experts.linear(s["x"], s["w"], s["bias"], routes, out=s["out"])}


# --- what a pass cannot do without ---------------------------------------------
def work(case):
    c, op = case, case["op"]
    n, m, k = c["n"], c["m"], c["k"]
    rows = n * m
    lists = 4 * (2 * rows + k + 1)   # offsets, entry, slot
    if op == "route":
        return {"bytes": 4 * rows + lists, "flops": 0}
    e = SIZE[c["dtype"]]
    if op == "dispatch":
        return {"bytes": e * c["d"] * (n + rows) + 4 * rows, "flops": rows * c["d"] if c["dir"] == "bwd" else 0}
    if op == "combine":
        if c["dir"] == "fwd":
            return {"bytes": e * c["d"] * (n + rows) + 8 * rows, "flops": 2 * rows * c["d"]}
        return {"bytes": e * c["d"] * (n + 2 * rows) + 12 * rows, "flops": 3 * rows * c["d"]}
    di, do = c["d_in"], c["d_out"]
    hit = min(k, rows)   # lists with rows
    if op == "linear":
        if c["dir"] == "fwd":
            return {"bytes": e * (n * di + rows * do + hit * di * do) + 4 * (hit * do + rows), "flops": 2 * rows * di * do}
        return {"bytes": e * (n * di + rows * (do + di) + hit * di * do) + 4 * (k * do * (di + 1) + rows),
                "flops": 4 * rows * di * do}
    return {"bytes": hit * do * ((di + 1) // 2 + 2 * -(-di // c["group"]) + 4) + e * n * (di + do) + 8 * rows,
            "flops": 2 * rows * di * do}


# --- the same in 64 bits ---------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    n, m, k = c["n"], c["m"], c["k"]
    if op == "route":
        flat = s["idx"].reshape(-1).cpu().numpy()
        offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[flat >= 0], minlength=k))])
        order = np.argsort(np.where(flat < 0, k, flat).astype(np.int16), kind="stable")[:offsets[-1]]
        entry, slot = np.full(n * m, -1), np.full(n * m, -1)
        entry[:order.size] = order
        slot[order] = np.arange(order.size)
        return {"offsets": offsets, "entry": entry, "slot": slot.reshape(n, m)}
    idx, gamma = s["idx"].long(), s["gamma"].double()
    if op == "linear4":
        out = torch.zeros((n, c["d_out"]), dtype=torch.float64, device=DEV)
        wide = torch.empty((c["d_out"], 2 * s["codes"].shape[2]), dtype=torch.float64, device=DEV)
        for kk in idx[idx >= 0].unique().tolist():
            wide[:, 0::2] = (s["codes"][kk] % 16).double() - 8
            wide[:, 1::2] = torch.div(s["codes"][kk], 16, rounding_mode="floor").double() - 8
            group_of = torch.arange(c["d_in"], device=DEV) // c["group"]
            w = wide[:, :c["d_in"]] * s["scales"][kk].double()[:, group_of]
            weight = torch.where(idx == kk, gamma, 0.0).sum(1)
            out += weight[:, None] * (s["x"].double() @ w.T + s["bias"][kk].double())
        return {"out": out}
    off, entry = s["offsets"].tolist(), s["entry"].long()
    total = off[-1]
    e = entry[:total]
    if op == "dispatch":
        if c["dir"] == "fwd":
            y = torch.zeros((n * m, c["d"]), dtype=torch.float64, device=DEV)
            y[:total] = s["x"].double()[e // m]
            return {"y": y}
        dx = torch.zeros((n, c["d"]), dtype=torch.float64, device=DEV)
        return {"dx": dx.index_add_(0, e // m, s["dy"][:total].double())}
    if op == "combine":
        w = gamma.reshape(-1)[e]
        if c["dir"] == "fwd":
            out = torch.zeros((n, c["d"]), dtype=torch.float64, device=DEV)
            return {"out": out.index_add_(0, e // m, s["z"][:total].double() * w[:, None])}
        rows = s["dout"].double()[e // m]
        dgamma = torch.zeros(n * m, dtype=torch.float64, device=DEV)
        dgamma[e] = (rows * s["z"][:total].double()).sum(1)
        dz = torch.zeros((n * m, c["d"]), dtype=torch.float64, device=DEV)
        dz[:total] = rows * w[:, None]
        return {"dz": dz, "dgamma": dgamma.view(n, m)}
    di, do = c["d_in"], c["d_out"]
    back = c["dir"] == "bwd"
    f64 = dict(dtype=torch.float64, device=DEV)
    y = torch.zeros((n * m, di if back else do), **f64)
    dw, db = (torch.zeros((k, do, di), **f64), torch.zeros((k, do), **f64)) if back else (None, None)
    for kk in range(k):
        a, b = off[kk], off[kk + 1]
        if a == b:
            continue
        xk, wk = s["x"][entry[a:b] // m].double(), s["w"][kk].double()
        if back:
            dyk = s["dy"][a:b].double()
            y[a:b] = dyk @ wk
            dw[kk] = dyk.T @ xk
            db[kk] = dyk.sum(0)
        else:
            y[a:b] = xk @ wk.T + s["bias"][kk].double()
    return {"dx": y, "dw": dw, "db": db} if back else {"y": y}
