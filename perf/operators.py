"""The gated linear recurrence (forward, backward, one-token step) and the state cache's page
operations: the cases they are measured on, their plain forms and their values in 64 bits.

For every batch row b and channel d (r, i: the pre-activations of the two gates)

    rho_t = sigmoid(r_t + r_bias)            iota_t = sigmoid(i_t + i_bias)
    v_t   = c softplus(lam) rho_t            a_t = exp(-v_t)        m_t = sqrt(1 - a_t^2)
    h_t   = a_t h_{t-1} + m_t iota_t x_t     y_t = h_t silu(z_t)    (y_t = h_t without z)

A reset at step t starts a new document of a packed row: a_t = 0 and m_t = 1.  A batch row of
`lengths[b]` steps ends there: its last state is the state after that step, what lies behind in y
is left as it was, and the gradients there are zero.

A cache is a set of pools (layers, slots, ...); a page is one slot of every layer and pool.
"""
import math

import torch

own = False

C = 8.0  # decay constant of the recurrence
IO = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------------- the cases
def listed():
    return [
        # one sequence, one token, Mamba-130M's inner width: the latency of a decode step
        dict(name="step one", op="step", batch=1, dim=1536, slots=1, io="bf16", gate=True),
        # a serving batch decoding from the slots of a larger pool, some rows of it padding
        dict(name="step batch", op="step", batch=256, dim=5120, slots=320, io="bf16", gate=True),
        # the smallest scan: a few channels, fp32
        dict(name="scan tiny", op="scan", batch=1, dim=64, seqlen=256, io="f32", gate=False, fused=False, ragged=False,
             packed=False, carry=False),
        # prefill of a padded batch of prompts, x, r and i slices of one projection's output
        dict(name="scan prefill", op="scan", batch=4, dim=5120, seqlen=2048, io="bf16", gate=True, fused=True,
             ragged=True, packed=False, carry=False),
        # one long document, continued from a carried state
        dict(name="scan long", op="scan", batch=1, dim=5120, seqlen=32768, io="bf16", gate=True, fused=False,
             ragged=False, packed=False, carry=True),
        # a training step (forward and backward) at Mamba-130M's layer shape, packed documents
        dict(name="train packed", op="train", batch=8, dim=1536, seqlen=2048, io="bf16", gate=True, fused=False,
             ragged=False, packed=True, carry=False),
        # odd sizes in fp32, padded rows, states carried in and gradients reaching the last ones
        dict(name="train odd", op="train", batch=3, dim=1001, seqlen=2047, io="f32", gate=True, fused=False, ragged=True,
             packed=False, carry=True),
        # few channels and a long row: the sequence is the only axis with work to share
        dict(name="train long", op="train", batch=1, dim=384, seqlen=32768, io="bf16", gate=False, fused=False,
             ragged=False, packed=False, carry=False),
        # admission: prefix snapshots are copied into slots, running sequences forked
        dict(name="admit small", op="admit", layers=4, slots=24, dim=385, copies=2, forks=3),
        dict(name="admit large", op="admit", layers=64, slots=64, dim=5120, copies=8, forks=12),
        # retirement: ended sequences are freed and the live pages moved to the front
        dict(name="retire small", op="retire", layers=4, slots=24, dim=385, ended=7),
        dict(name="retire large", op="retire", layers=24, slots=256, dim=1536, ended=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["step", "step", "scan", "scan", "scan", "train", "train", "train", "admit", "retire"])
    io = rng.choice(["bf16", "bf16", "f32"])
    coin = lambda: rng.random() < 0.5  # noqa: E731
    if op == "step":
        batch = _log(rng, 1, 512)
        return dict(op=op, batch=batch, dim=_log(rng, 16, 8192), slots=batch + rng.randrange(1 + batch), io=io, gate=coin())
    if op in ("scan", "train"):
        most = 4e7 if op == "scan" else 1.5e7
        while True:
            batch, dim, seqlen = _log(rng, 1, 16), _log(rng, 16, 8192), _log(rng, 1, 40000)
            if batch * dim * seqlen <= most:
                break
        return dict(op=op, batch=batch, dim=dim, seqlen=seqlen, io=io, gate=coin(), fused=coin(), ragged=coin(),
                    packed=coin(), carry=coin())
    layers, slots, dim = rng.randrange(1, 33), _log(rng, 4, 256), _log(rng, 16, 2048)
    if op == "admit":
        free = slots // 3
        return dict(op=op, layers=layers, slots=slots, dim=dim, copies=rng.randrange(max(1, slots // 4)),
                    forks=1 + rng.randrange(free + 1))
    return dict(op=op, layers=layers, slots=slots, dim=dim, ended=1 + rng.randrange(slots))


# --------------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    f32 = dict(device="cuda", dtype=torch.float32)
    randn = lambda *s: torch.randn(*s, generator=g, **f32)  # noqa: E731
    s = dict(case)
    if case["op"] in ("admit", "retire"):
        layers, slots, dim = case["layers"], case["slots"], case["dim"]
        # what this library's decode carries for a sequence: the scan's state and the conv's inputs
        s["states"], s["conv"] = randn(layers, slots, dim, 16), randn(layers, slots, dim, 3)
        order = torch.randperm(slots, generator=g, device="cuda").to(torch.int32)
        used = torch.ones(slots, dtype=torch.int32, device="cuda")
        if case["op"] == "admit":
            k, n = case["copies"], case["forks"]
            free = max(n - 1, slots // 3)  # the last fork can find no free slot
            used[order[:free].long()] = 0
            live = order[free:]
            s["src"], s["dst"] = live[:k].contiguous(), live[k:2 * k].contiguous()  # snapshots into admitted slots
            s["src"] = s["src"][: s["dst"].numel()]
            parents = live[torch.randint(live.numel(), (n,), generator=g, device="cuda")]
            parents[::4] = -1  # a new sequence: a page of zeros
            s["parents"], s["children"] = parents, torch.empty_like(parents)
        else:
            s["ended_slots"] = order[: case["ended"]].contiguous()
            s["table0"] = order.flip(0).contiguous()  # the sequences' slots, in batch order
            s["table"], s["remap"] = torch.empty_like(s["table0"]), torch.empty_like(s["table0"])
            s["count"] = torch.empty(1, dtype=torch.int32, device="cuda")
        s["used0"], s["used"] = used, used.clone()
        return s
    io, batch, dim = IO[case["io"]], case["batch"], case["dim"]
    # channel decays a^c between 0.9 and 0.999 at an open gate
    s["lam"] = torch.log(torch.expm1(-torch.log(0.9 + 0.099 * torch.rand(dim, generator=g, **f32)) / C))
    s["rb"], s["ib"] = 0.1 * randn(dim), 0.1 * randn(dim)
    if case["op"] == "step":
        s["x"], s["r"], s["i"] = randn(batch, 3 * dim).to(io).split(dim, 1)
        s["z"] = randn(batch, dim).to(io) if case["gate"] else None
        s["y"] = torch.zeros(batch, dim, dtype=io, device="cuda")
        s["state"] = randn(case["slots"], dim)
        s["at"] = torch.randperm(case["slots"], generator=g, device="cuda")[:batch].to(torch.int32)
        s["at"][5::17] = -1  # rows that pad the batch
        return s
    L = case["seqlen"]
    data = lambda *shape: torch.randn(*shape, generator=g, device="cuda", dtype=io)  # noqa: E731
    if case["fused"]:
        s["x"], s["r"], s["i"] = data(batch, 3 * dim, L).split(dim, 1)
    else:
        s["x"], s["r"], s["i"] = data(batch, dim, L), data(batch, dim, L), data(batch, dim, L)
    s["z"] = data(batch, dim, L) if case["gate"] else None
    s["h0"] = randn(batch, dim) if case["carry"] else None
    s["lengths"] = s["reset"] = None
    if case["ragged"]:
        s["lengths"] = torch.randint(L // 2, L + 1, (batch,), generator=g, device="cuda").to(torch.int32)
        s["lengths"][0] = L
    if case["packed"]:
        s["reset"] = (torch.rand(batch, L, generator=g, device="cuda") < 1 / 256).to(torch.uint8)
        s["reset"][:, 0] = 1
    s["y"], s["last"] = torch.zeros(batch, dim, L, dtype=io, device="cuda"), torch.empty(batch, dim, **f32)
    if case["op"] == "train":
        s["dy"] = data(batch, dim, L)
        s["dlast"] = randn(batch, dim) if case["carry"] else None
        s["dx"], s["dr"], s["di"] = (torch.empty(batch, 3 * dim, L, dtype=io, device="cuda").split(dim, 1) if case["fused"]
                                     else [torch.empty(batch, dim, L, dtype=io, device="cuda") for _ in range(3)])
        s["dz"] = torch.empty_like(s["z"]) if case["gate"] else None
        s["dlam"], s["drb"], s["dib"] = (torch.empty(dim, **f32) for _ in range(3))
        s["dh0"] = torch.empty(batch, dim, **f32)
    return s


# --------------------------------------------------------------------------- one pass
def run(s):
    if own:
        return {"step": _own_step, "scan": _own_scan, "train": _own_train, "admit": _own_admit, "retire": _own_retire}[s["op"]](s)
    return {"step": _step, "scan": _scan, "train": _train, "admit": _admit, "retire": _retire}[s["op"]](s)


def _own_step(s):
    import selective_state_space_16_b200 as ssm
    ssm.ssm_gated_state_update(s["state"], s["x"], s["r"], s["i"], s["lam"], s["rb"], s["ib"], s["z"], s["y"],
                               slots=s["at"], c=C)
    return {"y": s["y"], "state": s["state"]}


def _own_scan(s):
    import selective_state_space_16_b200 as ssm
    ssm.ssm_gated_scan_fwd(s["x"], s["r"], s["i"], s["lam"], s["rb"], s["ib"], s["z"], s["y"], s["last"],
                           initial_state=s["h0"], lengths=s["lengths"], reset=s["reset"], c=C)
    return {"y": s["y"], "last": s["last"]}


def _own_train(s):
    import selective_state_space_16_b200 as ssm
    if "workspace" not in s:  # kept by the program from step to step
        b, d, L = s["x"].shape
        s["checkpoints"] = ssm.new_gated_checkpoints(b, d, L, device="cuda")
        s["workspace"] = ssm.new_gated_workspace(b, d, L, device="cuda")
    ssm.ssm_gated_scan_fwd(s["x"], s["r"], s["i"], s["lam"], s["rb"], s["ib"], s["z"], s["y"], s["last"],
                           initial_state=s["h0"], lengths=s["lengths"], reset=s["reset"], checkpoints=s["checkpoints"], c=C)
    ssm.ssm_gated_scan_bwd(s["x"], s["r"], s["i"], s["lam"], s["rb"], s["ib"], s["z"], s["dy"], s["dx"], s["dr"],
                           s["di"], s["dlam"], s["drb"], s["dib"], s["dz"], s["workspace"], initial_state=s["h0"],
                           dlast_state=s["dlast"], dinitial_state=s["dh0"], lengths=s["lengths"], reset=s["reset"],
                           checkpoints=s["checkpoints"], c=C)
    return {k: s[k] for k in ("y", "last", "dx", "dr", "di", "dz", "dlam", "drb", "dib", "dh0")}


def _own_cache(s, n):
    import selective_state_space_16_b200 as ssm
    if "pools" not in s:  # the program's handle and workspace
        s["pools"] = ssm.CachePools([s["states"], s["conv"]])
        s["workspace"] = ssm.new_cache_workspace(s["pools"], n, device="cuda")
    return ssm


def _own_admit(s):
    ssm = _own_cache(s, max(s["copies"], s["forks"]))
    s["used"].copy_(s["used0"])
    ssm.ssm_cache_copy(s["pools"], s["src"], s["dst"], s["workspace"])
    ssm.ssm_cache_fork(s["pools"], s["used"], s["parents"], s["children"], s["workspace"])
    return {k: s[k] for k in ("states", "conv", "used", "children")}


def _own_retire(s):
    ssm = _own_cache(s, s["slots"])
    s["used"].copy_(s["used0"])
    s["table"].copy_(s["table0"])
    ssm.ssm_cache_free(s["pools"], s["used"], s["ended_slots"])
    ssm.ssm_cache_compact(s["pools"], s["used"], s["table"], s["remap"], s["count"], s["workspace"])
    return {k: s[k] for k in ("states", "conv", "used", "table", "remap", "count")}


# --------------------------------------------------------------------------- plain forms
def _linear_scan(a, b):
    """h_t = a_t h_{t-1} + b_t along the last axis, by doubling."""
    k = 1
    while k < a.shape[-1]:
        b = torch.cat((b[..., :k], b[..., k:] + a[..., k:] * b[..., :-k]), -1)
        a = torch.cat((a[..., :k], a[..., k:] * a[..., :-k]), -1)
        k *= 2
    return b


def _coefficients(s, x, r, i, column):
    """rho, iota, v, a, m in 32 bits; `column` spreads a channel's parameter over its steps."""
    rho = 1 / (1 + torch.exp(-(r.float() + column(s["rb"]))))
    iota = 1 / (1 + torch.exp(-(i.float() + column(s["ib"]))))
    v = column(C * torch.log1p(torch.exp(s["lam"]))) * rho
    return rho, iota, v, torch.exp(-v), torch.sqrt(-torch.expm1(-2 * v))


def _silu(z):
    return z / (1 + torch.exp(-z))


def _step(s):
    rho, iota, v, a, m = _coefficients(s, s["x"], s["r"], s["i"], lambda p: p)
    rows = s["at"] >= 0
    at = s["at"].clamp(min=0).long()
    h = a * s["state"][at] + m * iota * s["x"].float()
    s["state"][at[rows]] = h[rows]
    y = h if s["z"] is None else h * _silu(s["z"].float())
    s["y"].copy_(torch.where(rows[:, None], y.to(s["y"].dtype), s["y"]))
    return {"y": s["y"], "state": s["state"]}


def _forward(s):
    x = s["x"].float()
    rho, iota, v, a, m = _coefficients(s, s["x"], s["r"], s["i"], lambda p: p[:, None])
    valid = None
    if s["reset"] is not None:
        at = s["reset"][:, None, :] != 0
        a, m = a.masked_fill(at, 0), m.masked_fill(at, 1)
    b = m * iota * x
    if s["lengths"] is not None:
        valid = torch.arange(x.shape[2], device=x.device) < s["lengths"][:, None, None]
        a, b = torch.where(valid, a, 1), torch.where(valid, b, 0)
    if s["h0"] is not None:
        b[..., 0] += a[..., 0] * s["h0"]
    h = _linear_scan(a, b)
    y = h if s["z"] is None else h * _silu(s["z"].float())
    if valid is not None:
        y = torch.where(valid, y, 0)  # the buffer's own zeros
    return x, rho, iota, v, a, m, h, valid, y.to(s["x"].dtype)


def _scan(s):
    *_, h, valid, y = _forward(s)
    return {"y": y, "last": h[..., -1].contiguous()}


def _train(s):
    x, rho, iota, v, a, m, h, valid, y = _forward(s)
    io, dh = s["x"].dtype, s["dy"].float()
    zero = torch.zeros_like(h[..., :1]) if s["h0"] is None else s["h0"][..., None]
    before = torch.cat((zero, h[..., :-1]), -1)
    dz = None
    if s["z"] is not None:
        z = s["z"].float()
        sig = 1 / (1 + torch.exp(-z))
        dz = dh * h * sig * (1 + z * (1 - sig))
        dh = dh * z * sig
    if valid is not None:
        dh = torch.where(valid, dh, 0)
    if s["dlast"] is not None:
        dh = torch.cat((dh[..., :-1], dh[..., -1:] + s["dlast"][..., None]), -1)
    after = torch.cat((a[..., 1:], torch.ones_like(a[..., :1])), -1)
    g = _linear_scan(after.flip(-1), dh.flip(-1)).flip(-1)
    # dm/dv = a^2 / m: v/m is finite for v -> 0
    decay = g * (iota * x * a * a * torch.where(m > 0, v / m, 0) - before * a * v)
    if s["reset"] is not None:
        decay = decay.masked_fill(s["reset"][:, None, :] != 0, 0)
    dr = decay * (1 / (1 + torch.exp(s["r"].float() + s["rb"][:, None])))
    di = g * m * x * iota * (1 / (1 + torch.exp(s["i"].float() + s["ib"][:, None])))
    dx = g * m * iota
    if valid is not None:
        decay, dr, di, dx = (torch.where(valid, t, 0) for t in (decay, dr, di, dx))
        dz = None if dz is None else torch.where(valid, dz, 0)
    lam = s["lam"]
    dlam = decay.sum((0, 2)) / (1 + torch.exp(-lam)) / torch.log1p(torch.exp(lam))
    return {"y": y, "last": h[..., -1].contiguous(), "dx": dx.to(io), "dr": dr.to(io), "di": di.to(io),
            "dz": None if dz is None else dz.to(io), "dlam": dlam, "drb": dr.sum((0, 2)), "dib": di.sum((0, 2)),
            "dh0": a[..., 0] * g[..., 0]}


def _admit(s):
    s["used"].copy_(s["used0"])
    src, dst = s["src"].long(), s["dst"].long()
    s["states"][:, dst], s["conv"][:, dst] = s["states"][:, src], s["conv"][:, src]
    # each fork takes the lowest free slot that is left
    free = torch.sort((s["used"] != 0).to(torch.int32), stable=True).indices
    n = s["parents"].numel()
    room = torch.arange(n, device="cuda") < (s["used"] == 0).sum()
    child = torch.where(room, torch.cat((free, free.new_zeros(n)))[:n], -1)
    took, parent = child[room], s["parents"].long()[room]
    fresh = parent < 0
    for pool in (s["states"], s["conv"]):
        pool[:, took] = torch.where(fresh[:, None, None], 0, pool[:, parent.clamp(min=0)])
    s["used"][took] = 1
    s["children"].copy_(child)
    return {k: s[k] for k in ("states", "conv", "used", "children")}


def _retire(s):
    s["used"].copy_(s["used0"])
    s["used"][s["ended_slots"].long()] = 0
    live = s["used"] != 0
    count = live.sum()
    slot = torch.arange(live.numel(), device="cuda")
    to, fro = slot[~live & (slot < count)], slot[live & (slot >= count)]
    s["states"][:, to], s["conv"][:, to] = s["states"][:, fro], s["conv"][:, fro]
    remap = torch.where(live & (slot < count), slot, -1)
    remap[fro] = to
    s["remap"].copy_(remap)
    s["used"].copy_(slot < count)
    s["count"].copy_(count[None])
    s["table"].copy_(remap[s["table0"].long()])
    return {k: s[k] for k in ("states", "conv", "used", "table", "remap", "count")}


# --------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    if op in ("admit", "retire"):
        page = case["layers"] * case["dim"] * (16 + 3) * 4
        if op == "admit":
            n = case["forks"]
            new = -(-n // 4)
            return {"bytes": page * (2 * case["copies"] + 2 * (n - new) + new), "flops": 0}
        live = case["slots"] - case["ended"]
        return {"bytes": page * 2 * case["ended"] * live / case["slots"] + 16 * case["slots"], "flops": 0}
    size = IO[case["io"]].itemsize
    if op == "step":
        n = (case["batch"] - len(range(5, case["batch"], 17))) * case["dim"]  # without the padding rows
        return {"bytes": n * (8 + size * (5 if case["gate"] else 4)) + 12 * case["dim"], "flops": 30 * n}
    batch = case["batch"]
    share = (1 + 0.75 * (batch - 1)) / batch if case["ragged"] else 1  # of a batch's steps that are not padding
    n = batch * case["dim"] * case["seqlen"]
    arrays, flops = 5 if case["gate"] else 4, 30
    if op == "train":  # forward, and backward: the inputs and dy again; the gradients, zero over the padding
        arrays, flops = arrays * 2 + (4 if case["gate"] else 3) / share, 100
    return {"bytes": n * share * size * arrays + 4 * batch * case["dim"] * (4 if op == "train" else 2), "flops": flops * n * share}


# --------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    """The recurrence one step after another in 64 bits; the cache's pages are copies and have no such value."""
    if case["op"] in ("admit", "retire"):
        return None
    s = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in prepare(case, seed).items()}
    sig, flat = torch.sigmoid, (lambda t: t.permute(2, 0, 1).contiguous())  # time first
    rate = C * torch.nn.functional.softplus(s["lam"])
    if case["op"] == "step":
        log_a = -rate * sig(s["r"] + s["rb"])
        x = torch.sqrt(-torch.expm1(2 * log_a)) * sig(s["i"] + s["ib"]) * s["x"]
        at, y, state = s["at"].tolist(), torch.zeros_like(s["y"]), s["state"].clone()
        rows = [b for b in range(len(at)) if at[b] >= 0]
        to = [at[b] for b in rows]
        state[to] = torch.exp(log_a[rows]) * state[to] + x[rows]
        y[rows] = state[to] if s["z"] is None else state[to] * s["z"][rows] * sig(s["z"][rows])
        return {"y": y, "state": state}
    x, r, i = flat(s["x"]), flat(s["r"]) + s["rb"], flat(s["i"]) + s["ib"]
    L, batch, dim = x.shape
    inside = torch.ones(L, batch, 1, dtype=torch.bool, device="cuda")
    if s["lengths"] is not None:
        inside = torch.arange(L, device="cuda")[:, None, None] < s["lengths"][None, :, None]
    start = torch.zeros_like(inside) if s["reset"] is None else (s["reset"].t()[..., None] != 0) & inside
    log_a = -rate * sig(r)
    a = torch.exp(log_a).masked_fill(start, 0).masked_fill(~inside, 1)
    m = torch.sqrt(-torch.expm1(2 * log_a)).masked_fill(start, 1).masked_fill(~inside, 0)
    u = sig(i) * x
    h = torch.empty(L + 1, batch, dim, dtype=torch.float64, device="cuda")
    h[0] = 0 if s["h0"] is None else s["h0"]
    b = m * u
    for t in range(L):
        torch.addcmul(b[t], a[t], h[t], out=h[t + 1])
    del b
    z = None if s["z"] is None else flat(s["z"])
    back = lambda t: t.permute(1, 2, 0)  # noqa: E731
    out = {"y": back((h[1:] if z is None else h[1:] * z * sig(z)) * inside), "last": h[L].clone()}
    if case["op"] == "scan":
        return out
    dy = flat(s["dy"])
    gh = torch.empty(L + 1, batch, dim, dtype=torch.float64, device="cuda")  # gradient of the state after step t - 1
    gh[1:] = (dy if z is None else dy * z * sig(z)) * inside
    if s["dlast"] is not None:
        gh[L] += s["dlast"]
    for t in range(L - 1, 0, -1):
        gh[t].addcmul_(a[t], gh[t + 1])
    torch.mul(a[0], gh[1], out=gh[0])
    g = gh[1:]
    moves = inside & ~start
    dlog = (g * (a * h[:-1] - torch.where(moves, u * a * a / m, 0))) * moves  # d/d log a of both uses of a
    dr = dlog * log_a * sig(-r)
    di = g * m * x * sig(i) * sig(-i) * inside
    out.update(dx=back(g * m * sig(i) * inside), dr=back(dr), di=back(di), dz=None,
               dlam=(dlog * -sig(r)).sum((0, 1)) * C * sig(s["lam"]), drb=dr.sum((0, 1)), dib=di.sum((0, 1)), dh0=gh[0].clone())
    if z is not None:
        out["dz"] = back(dy * h[1:] * sig(z) * (1 + z * sig(-z)) * inside)
    return out
