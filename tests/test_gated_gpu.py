"""The gated linear recurrence on the GPU against the 64-bit reference (-m gpu): forward, backward,
one-token step, and the three together."""
import numpy as np
import pytest
import torch

import selective_state_space_16_b200 as ssm
from gated_reference import U, check, f64, reference, sigmoid
from selective_state_space_16_b200 import binding

pytestmark = pytest.mark.gpu
IO = {"bf16": torch.bfloat16, "f32": torch.float32}
GRADS = ("dx", "dr", "di", "dz", "dlam", "dr_bias", "di_bias", "dinitial_state")


def inputs(B, D, L, io, gate=True, biases=True, state=True, lengths=None, reset=None, fused=False, seed=0):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    if fused:  # slices of one projection's output
        x, r, i = rnd(B, 3 * D, L).to(IO[io]).cuda().split(D, 1)
    else:
        x, r, i = (rnd(B, D, L).to(IO[io]).cuda() for _ in range(3))
    # decays between nearly 1 and nearly 0 at an open gate
    lam = torch.linspace(-9.0, 2.0, D) if D > 1 else torch.tensor([-4.0])
    t = dict(x=x, r=r, i=i, lam=lam.cuda(), z=rnd(B, D, L).to(IO[io]).cuda() if gate else None,
             r_bias=(0.3 * rnd(D)).cuda() if biases else None, i_bias=(0.3 * rnd(D)).cuda() if biases else None,
             initial_state=rnd(B, D).cuda() if state else None)
    t["lengths"] = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    if reset is not None:
        reset = (torch.rand(B, L, generator=g) < reset).to(torch.uint8).cuda()
    t["reset"] = reset
    return t, rnd(B, D, L).to(IO[io]).cuda(), rnd(B, D).cuda()


def run_all(t, dy, dlast, checkpoints):
    B, D, L = t["x"].shape
    ck = ssm.new_gated_checkpoints(B, D, L) if checkpoints else None
    y, last = ssm.gated_scan_fwd(**t, checkpoints=ck)
    grads = ssm.gated_scan_bwd(**t, dy=dy, dlast_state=dlast, checkpoints=ck)
    return dict(grads, y=y, last=last)


def compare(got, t, dy, dlast, what):
    want = reference(**t, dy=dy, dlast=dlast, bf16=t["x"].dtype == torch.bfloat16)
    for k, w in want.items():
        check(got[k], w, f"{what} {k}")
    assert (got["dz"] is None) == (t["z"] is None)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("L", [1, 2, 7, 8, 9, 16, 31, 64, 255, 256, 257, 511, 512, 513, 1000, 2061])
def test_lengths(cuda_device, io, L):
    t, dy, dlast = inputs(2, 5, L, io, seed=L)
    compare(run_all(t, dy, dlast, True), t, dy, dlast, f"L={L} {io}")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("gate,biases,state", [(False, False, False), (True, False, True), (False, True, False)])
@pytest.mark.parametrize("checkpoints", [False, True])
def test_optional_inputs(cuda_device, io, gate, biases, state, checkpoints):
    t, dy, dlast = inputs(3, 33, 300, io, gate, biases, state, seed=5)
    dlast = dlast if state else None
    compare(run_all(t, dy, dlast, checkpoints), t, dy, dlast, "optional")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("reset", [None, 0.03, 1.0])
def test_padded_and_packed_rows(cuda_device, io, fused, reset):
    L = 531
    t, dy, dlast = inputs(6, 9, L, io, lengths=[L, 0, 1, 257, 10 ** 6, -4], reset=reset, fused=fused, seed=7)
    compare(run_all(t, dy, dlast, True), t, dy, dlast, "padded")
    compare(run_all(t, dy, dlast, False), t, dy, dlast, "padded, no checkpoints")


def test_rows_behind_the_lengths_are_left(cuda_device):
    t, dy, dlast = inputs(3, 4, 300, "bf16", lengths=[300, 0, 140])
    for k in ("x", "r", "i", "z"):  # what lies behind reaches nothing
        t[k][2, :, 140:] = float("nan")
        t[k][1] = float("inf")
    dy[2, :, 140:] = float("nan")
    y = torch.full_like(t["x"], 7.0)
    last = torch.empty(3, 4, device="cuda")
    ssm.ssm_gated_scan_fwd(t["x"], t["r"], t["i"], t["lam"], t["r_bias"], t["i_bias"], t["z"], y, last,
                           initial_state=t["initial_state"], lengths=t["lengths"])
    assert bool((y[1] == 7).all()) and bool((y[2, :, 140:] == 7).all()) and bool(torch.isfinite(y).all())
    assert torch.equal(last[1], t["initial_state"][1])
    for ck in (False, True):
        got = run_all(t, dy, dlast, ck)
        for k in ("dx", "dr", "di", "dz"):
            assert bool((got[k][1] == 0).all()) and bool((got[k][2, :, 140:] == 0).all()), k
        assert all(bool(torch.isfinite(got[k]).all()) for k in GRADS)
        assert torch.equal(got["dinitial_state"][1], dlast[1])
    clean = {k: (v.clone() if v is not None else None) for k, v in t.items()}
    for k in ("x", "r", "i", "z"):
        clean[k][2, :, 140:] = clean[k][1] = 0
    dy[2, :, 140:] = 0
    compare(got, clean, dy, dlast, "padding")


def test_nothing_passes_a_reset(cuda_device):
    """A document's NaN or infinity reaches neither the documents after it nor, backwards, those before."""
    t, dy, dlast = inputs(2, 3, 700, "f32", reset=0.0)
    for at in (0, 100, 300, 555):
        t["reset"][:, at] = 1
    t["initial_state"][0] = float("nan")
    t["x"][0, :, 120] = float("inf")
    t["x"][1, 1, 299] = float("nan")
    dy[1, 2, 310] = float("nan")
    dlast[0] = float("nan")
    got = run_all(t, dy, dlast, True)
    for k in ("y", "dx", "dr", "di", "dz"):
        bad = ~torch.isfinite(got[k])
        assert not bool(bad[:, :, :100].any()) and not bool(bad[0, :, 300:555].any()) and not bool(bad[1, :, 555:].any()), k
    assert not bool(torch.isfinite(got["y"][0, :, 120:300]).any()) and bool(torch.isfinite(got["y"][0, :, 300:]).all())
    assert not bool(torch.isfinite(got["dx"][1, 2, 300:311]).any()) and bool(torch.isfinite(got["dx"][1, 2, :300]).all())


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_saturated_gates(cuda_device, io):
    """Gates shut and wide open, decays of nearly 1 and of 0: finite gradients throughout."""
    t, dy, dlast = inputs(2, 6, 130, io, seed=11)
    t["r"][0, :, ::3], t["r"][1, :, ::4] = -40.0, 60.0
    t["i"][0, :, 1::3], t["i"][1, :, 1::4] = -60.0, 45.0
    t["lam"] = torch.tensor([-30.0, -12.0, -3.0, 0.0, 3.0, 25.0], device="cuda")
    got = run_all(t, dy, dlast, True)
    assert all(bool(torch.isfinite(got[k]).all()) for k in GRADS + ("y", "last"))
    compare(got, t, dy, dlast, "saturated")


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_shut_gates_leave_the_state_alone(cuda_device, io):
    """A recurrence gate of the type's lowest value or -inf (a masked step) keeps the state, and its step has no
    gradient; an input gate so shut lets nothing in; lam = -inf freezes a channel.  From group to group of 8 steps
    the state is composed anew, of at most 6 products and sums of magnitudes up to the largest state: it may move
    by 12 half steps of that, and is the same bit for bit inside a group."""
    t, dy, dlast = inputs(2, 4, 90, io, gate=False, seed=43)
    low = torch.finfo(IO[io]).min
    t["r"][0, :, 20:60], t["r"][1, :, 20:60] = low, float("-inf")
    t["x"][:, :, 30:40] = 1e30
    t["i"][0, :, 70:], t["i"][1, :, 70:] = low, float("-inf")
    t["lam"][0] = float("-inf")
    got = run_all(t, dy, dlast, True)
    y = got["y"].float()
    for a in range(24, 56, 8):
        assert torch.equal(y[:, :, a:a + 8], y[:, :, a:a + 1].expand(-1, -1, 8))
    most = y.abs().amax(2, keepdim=True) + t["initial_state"].abs()[..., None]
    moved = (y[:, :, 20:60] - y[:, :, 19:20]).abs()
    assert bool((moved <= (12 * U / 2 * most if io == "f32" else 2.0 ** -7 * y[:, :, 19:20].abs())).all())
    for k in ("dx", "dr", "di"):
        assert not bool(got[k][:, :, 20:60].any()), k
    assert not bool(got["dx"][:, :, 70:].any()) and not bool(got["di"][:, :, 70:].any())
    assert torch.equal(got["last"][:, 0], t["initial_state"][:, 0])
    assert all(bool(torch.isfinite(got[k]).all()) for k in GRADS if got[k] is not None)


@pytest.mark.parametrize("io,D,L", [("f32", 2600, 4100), ("bf16", 3000, 8192)])
def test_many_long_rows(cuda_device, io, D, L):
    """Shapes whose last wave is filled by splitting rows: every 97th channel against the reference."""
    g = torch.Generator("cuda").manual_seed(47)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    t = {k: rnd(1, D, L).to(IO[io]) for k in ("x", "r", "i", "z")}
    t.update(lam=torch.linspace(-9, 2, D, device="cuda"), r_bias=0.3 * rnd(D), i_bias=0.3 * rnd(D), initial_state=rnd(1, D),
             lengths=torch.tensor([L - 5], dtype=torch.int32, device="cuda"), reset=None)
    dy, dlast = rnd(1, D, L).to(IO[io]), rnd(1, D)
    got = run_all(t, dy, dlast, True)
    pick = slice(3, None, 97)
    some = {k: v if v is None or k == "lengths" else v[pick] if v.dim() == 1 else v[:, pick] for k, v in t.items()}
    want = reference(**some, dy=dy[:, pick], dlast=dlast[:, pick], bf16=io == "bf16")
    for k, w in want.items():
        check(got[k][pick] if got[k].dim() == 1 else got[k][:, pick], w, f"{io} {k}")
    assert all(bool(torch.isfinite(got[k]).all()) for k in GRADS)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("B,D,L", [(1, 1, 40000), (1, 3, 9001), (2, 700, 129), (1, 2500, 77), (40, 130, 60), (2, 75, 2500), (1, 170, 5003),
                                   (1, 90, 4100), (4, 150, 1030)])
def test_shapes(cuda_device, io, B, D, L):
    t, dy, dlast = inputs(B, D, L, io, seed=B + D + L)
    compare(run_all(t, dy, dlast, True), t, dy, dlast, f"{B}x{D}x{L}")


def test_rows_split_over_blocks_with_resets_and_lengths(cuda_device):
    """Few rows, each shared by the warps of several blocks: documents, padding and non-finite values across them."""
    B, D, L = 3, 5, 21000
    t, dy, dlast = inputs(B, D, L, "bf16", lengths=[L, 9, 13001], reset=0.0003, seed=41)
    compare(run_all(t, dy, dlast, True), t, dy, dlast, "split")
    compare(run_all(t, dy, dlast, False), t, dy, dlast, "split, no checkpoints")
    t["reset"][0, :] = 0
    t["reset"][0, 4000] = t["reset"][0, 9000] = 1
    t["x"][0, :, 100] = float("nan")
    dy[0, :, 20000] = float("inf")
    got = run_all(t, dy, dlast, True)
    assert bool(torch.isfinite(got["y"][0, :, 4000:]).all()) and not bool(torch.isfinite(got["y"][0, 0, 101]))
    for k in ("dx", "dr", "di", "dz"):
        assert bool(torch.isfinite(got[k][0, :, 4000:9000]).all()) and bool(torch.isfinite(got[k][0, :, 20001:]).all()), k
    assert not bool(torch.isfinite(got["dx"][0, 0, 19999]))


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_operands_of_every_alignment(cuda_device, io):
    """Each operand starts at its own offset and has its own strides."""
    B, D, L = 2, 4, 541
    t, dy, dlast = inputs(B, D, L, io, lengths=[L, 400], seed=13)

    def shifted(v, by, pad):
        wide = torch.full((B, D, L + pad), 3.0, dtype=v.dtype, device="cuda")
        flat = torch.empty(wide.numel() + by + 64, dtype=v.dtype, device="cuda")
        at = flat[by:by + wide.numel()].view(wide.shape)[..., :L]
        at.copy_(v)
        return at

    for k, by, pad in (("x", 1, 3), ("r", 5, 0), ("i", 8, 16), ("z", 0, 1)):
        t[k] = shifted(t[k], by, pad)
    dy = shifted(dy, 3, 2)
    ck, ws = ssm.new_gated_checkpoints(B, D, L), ssm.new_gated_workspace(B, D, L)
    out = {k: shifted(torch.zeros_like(dy), by, pad) for k, by, pad in (("y", 2, 5), ("dx", 7, 1), ("dr", 1, 0), ("di", 0, 8), ("dz", 9, 7))}
    last, dh0 = torch.empty(B, D, device="cuda"), torch.empty(B, D, device="cuda")
    dlam, drb, dib = (torch.empty(D, device="cuda") for _ in range(3))
    more = dict(initial_state=t["initial_state"], lengths=t["lengths"])
    a = [t[k] for k in ("x", "r", "i", "lam", "r_bias", "i_bias", "z")]
    for given in (ck, None):
        ssm.ssm_gated_scan_fwd(*a, out["y"], last, checkpoints=ck, **more)
        ssm.ssm_gated_scan_bwd(*a, dy, out["dx"], out["dr"], out["di"], dlam, drb, dib, out["dz"], ws, dlast_state=dlast,
                               dinitial_state=dh0, checkpoints=given, **more)
        compare(dict(out, last=last, dinitial_state=dh0, dlam=dlam, dr_bias=drb, di_bias=dib), t, dy, dlast, "shifted")
        # the checkpoints go by position: copies of the operands at other addresses may read them
        a = [v if v is None else v.clone() for v in a]
        for v in out.values():
            base = v._base if v._base is not None else v
            assert bool(torch.isfinite(v).all()) and base.shape[0] > 0


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("L", [37, 100, 250, 700])
@pytest.mark.parametrize("one", [None, "i", "z", "dy", "dr", "dz"])
def test_operands_that_lie_alike(cuda_device, io, L, one):
    """All inputs alike and all gradients alike, each at an odd place, but for `one` of them; what lies beside their
    rows stays."""
    B, D = 3, 7
    t, dy, dlast = inputs(B, D, L, io, seed=L)
    inp = dict(t, dy=dy)
    names = ("x", "r", "i", "z", "dy"), ("dx", "dr", "di", "dz")
    wide = {}

    def placed(k, by, pad):
        by, pad = (by + 1, pad + 2) if k == one else (by, pad)
        flat = torch.full((B * D * (L + pad) + by + 16,), 7.0, dtype=dy.dtype, device="cuda")
        wide[k] = flat
        return flat[by:by + B * D * (L + pad)].view(B, D, L + pad)[..., :L]

    for k in names[0]:
        v = placed(k, 3, 1)
        v.copy_(inp[k])
        inp[k] = v
    out = {k: placed(k, 5, 3) for k in names[1]}
    dy = inp.pop("dy")
    ck, ws = ssm.new_gated_checkpoints(B, D, L), ssm.new_gated_workspace(B, D, L)
    a = [inp[k] for k in ("x", "r", "i", "lam", "r_bias", "i_bias", "z")]
    y, last, dh0 = torch.empty(B, D, L, dtype=dy.dtype, device="cuda"), torch.empty(B, D, device="cuda"), torch.empty(B, D, device="cuda")
    sums = [torch.empty(D, device="cuda") for _ in range(3)]
    ssm.ssm_gated_scan_fwd(*a, y, last, initial_state=inp["initial_state"], checkpoints=ck)
    ssm.ssm_gated_scan_bwd(*a, dy, out["dx"], out["dr"], out["di"], *sums, out["dz"], ws, initial_state=inp["initial_state"],
                           dlast_state=dlast, dinitial_state=dh0, checkpoints=ck)
    got = dict(out, y=y, last=last, dinitial_state=dh0, **dict(zip(("dlam", "dr_bias", "di_bias"), sums)))
    compare(got, t, dy, dlast, f"alike but {one}")
    for k, v in wide.items():
        view = inp[k] if k in inp else out.get(k, dy)
        view.fill_(7.0)
        assert bool((v == 7).all()), f"{k}: written beside its rows"


@pytest.mark.parametrize("B,D,L", [(1, 70001, 2), (9001, 1, 3), (1500, 2, 5), (5, 4099, 1), (3, 4097, 17), (129, 127, 9)])
def test_many_short_rows(cuda_device, B, D, L):
    t, dy, dlast = inputs(B, D, L, "bf16", lengths=[1 + k % L for k in range(B)], seed=B)
    compare(run_all(t, dy, dlast, True), t, dy, dlast, f"{B}x{D}x{L}")


def test_transposed_batch_and_channels(cuda_device):
    """Strides of (dim, batch, seqlen) tensors."""
    t, dy, dlast = inputs(3, 5, 290, "bf16", seed=17)
    for k in ("x", "r", "i", "z"):
        t[k] = t[k].transpose(0, 1).contiguous().transpose(0, 1)
    compare(run_all(t, dy, dlast, True), t, dy, dlast, "transposed")


def test_broadcast_inputs(cuda_device):
    """Operands shared by the batch rows or by the channels (stride 0); flags as bool."""
    t, dy, dlast = inputs(3, 6, 333, "bf16", reset=0.02, seed=67)
    t["r"], t["i"], t["z"] = t["r"][:1].expand(3, 6, 333), t["i"][:, :1].expand(3, 6, 333), t["z"][:1, :1].expand(3, 6, 333)
    t["reset"] = t["reset"].bool()
    dy = dy[:1].expand(3, 6, 333)
    compare(run_all(t, dy, dlast, True), t, dy, dlast, "broadcast")


def test_far_offsets(cuda_device):
    """Rows and slots more than 2^32 bytes apart."""
    far, L = (1 << 31) + 16, 100
    buf = torch.empty(far + 12000, dtype=torch.bfloat16, device="cuda")
    at = lambda k, v=None: (lambda w: w if v is None else w.copy_(v))(buf.as_strided((2, 3, L), (far, 128, 1), 1000 * k))  # noqa: E731
    t, dy, dlast = inputs(2, 3, L, "bf16", seed=71)
    for k, name in enumerate(("x", "r", "i", "z")):
        t[name] = at(k, t[name])
    dy = at(4, dy)
    out = {k: at(5 + n) for n, k in enumerate(("y", "dx", "dr", "di", "dz"))}
    last, dh0, ck, ws = torch.empty(2, 3, device="cuda"), torch.empty(2, 3, device="cuda"), ssm.new_gated_checkpoints(2, 3, L), ssm.new_gated_workspace(2, 3, L)
    dlam, drb, dib = (torch.empty(3, device="cuda") for _ in range(3))
    a = [t[k] for k in ("x", "r", "i", "lam", "r_bias", "i_bias", "z")]
    ssm.ssm_gated_scan_fwd(*a, out["y"], last, initial_state=t["initial_state"], checkpoints=ck)
    ssm.ssm_gated_scan_bwd(*a, dy, out["dx"], out["dr"], out["di"], dlam, drb, dib, out["dz"], ws, initial_state=t["initial_state"],
                           dlast_state=dlast, dinitial_state=dh0, checkpoints=ck)
    compare(dict(out, last=last, dinitial_state=dh0, dlam=dlam, dr_bias=drb, di_bias=dib), t, dy, dlast, "far")
    state = buf.view(torch.float32).as_strided((2, 3), (far // 2, 1), 5500)
    state.copy_(torch.randn(2, 3))
    y0, ey, st, est = step_reference(t, state, [1, 0], 0, True)
    cols = [v[..., 0].contiguous() for v in (t["x"], t["r"], t["i"], t["z"])]
    y = torch.empty(2, 3, dtype=torch.bfloat16, device="cuda")
    ssm.ssm_gated_state_update(state, *cols[:3], t["lam"], t["r_bias"], t["i_bias"], cols[3], y,
                               slots=torch.tensor([1, 0], dtype=torch.int32, device="cuda"))
    check(y, (y0, ey), "far y")
    check(state, (st, est), "far state")
    del buf, t, a, out, dy, state
    torch.cuda.empty_cache()


def test_wanted_gradients_only(cuda_device):
    t, dy, dlast = inputs(2, 7, 300, "f32", gate=False, seed=19)
    full = run_all(t, dy, dlast, True)
    dx, dr, di = (torch.empty_like(t["x"]) for _ in range(3))
    dlam = torch.empty(7, device="cuda")
    ws = ssm.new_gated_workspace(2, 7, 300)
    for wanted in (None, dlam):
        ssm.ssm_gated_scan_bwd(t["x"], t["r"], t["i"], t["lam"], t["r_bias"], t["i_bias"], None, dy, dx, dr, di, wanted, None, None,
                               None, ws, initial_state=t["initial_state"], dlast_state=dlast)
        for k, v in (("dx", dx), ("dr", dr), ("di", di)):
            assert torch.equal(v, full[k])
    assert torch.equal(dlam, full["dlam"])


def test_empty(cuda_device):
    lam = torch.zeros(4, device="cuda")
    wide = torch.randn(2, 4, 13, device="cuda")[..., 5:5]  # (an empty slice has no address, but its strides)
    y, last = ssm.gated_scan_fwd(wide, wide, wide, lam, z=wide)
    assert y.shape == (2, 4, 0) and not bool(last.any())
    for B, L in ((2, 0), (0, 5)):
        x = torch.empty(B, 4, L, device="cuda", dtype=torch.bfloat16)
        h0 = torch.randn(B, 4, device="cuda")
        y, last = ssm.gated_scan_fwd(x, x, x, lam, initial_state=h0)
        assert y.shape == x.shape and torch.equal(last, h0)
        g = ssm.gated_scan_bwd(x, x, x, lam, dy=x, dlast_state=h0)
        assert torch.equal(g["dinitial_state"], h0) and not bool(g["dlam"].any()) and not bool(g["di_bias"].any())


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_same_results_every_time(cuda_device, io):
    t, dy, dlast = inputs(5, 70, 1300, io, lengths=[1300, 5, 0, 1299, 700], reset=0.01, seed=23)
    first, again = (run_all(t, dy, dlast, True) for _ in range(2))
    assert all(torch.equal(first[k], again[k]) for k in first)


def test_state_carried_from_block_to_block(cuda_device):
    """Scanning [0, 300) and then the rest from its last state, in place, gives the whole scan."""
    t, dy, dlast = inputs(2, 40, 1001, "f32", seed=29)
    want = reference(**t)
    state, ys = t["initial_state"].clone(), []
    for a, b in ((0, 300), (300, 301), (301, 301), (301, 1001)):
        part = {k: t[k][..., a:b] for k in ("x", "r", "i", "z")}
        y = torch.empty(2, 40, b - a, device="cuda")
        ssm.ssm_gated_scan_fwd(part["x"], part["r"], part["i"], t["lam"], t["r_bias"], t["i_bias"], part["z"], y, state,
                               initial_state=state)
        ys.append(y)
    check(torch.cat(ys, -1), want["y"], "blocks y")
    check(state, want["last"], "blocks last")


# ------------------------------------------------------------------------------- one-token step
def step_reference(t, state, slots, k, bf16):
    """The step on column k of the inputs, one row after another; returns y and its bound, the state and its bound."""
    col = {n: None if t[n] is None else t[n][..., k:k + 1] for n in ("x", "r", "i", "z")}
    st, est = f64(state), np.zeros(state.shape)
    y, ey = np.full(col["x"].shape[:2], np.nan), np.ones(col["x"].shape[:2])
    for b, s in enumerate(slots):
        if 0 <= s < st.shape[0]:
            one = {n: None if v is None else v[b:b + 1] for n, v in col.items()}
            o = reference(**one, lam=t["lam"], r_bias=t["r_bias"], i_bias=t["i_bias"], initial_state=torch.from_numpy(st[s:s + 1]), bf16=bf16)
            y[b], e = o["y"][0][0, :, 0], est[s]
            gate = 1 if t["z"] is None else np.abs(f64(one["z"])[0, :, 0]) * sigmoid(f64(one["z"])[0, :, 0])
            ey[b] = o["y"][1][0, :, 0] + e * gate * 1.01
            st[s], est[s] = o["last"][0][0], o["last"][1][0] + e
    return y, ey, st, est + U * np.abs(st) + 1e-30


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("B,D,slots", [(1, 1, None), (4, 33, None), (5, 129, [3, 0, -1, 7, 6]), (6, 1000, [2, 2, 9, 2, 0, 10]),
                                       (3, 1537, [1, 1, 1]), (300, 24, "all")])
@pytest.mark.parametrize("gate", [True, False])
def test_step(cuda_device, io, B, D, slots, gate):
    n = 10 if slots != "all" else 311
    at = list(range(B)) if slots is None else [int(v) for v in torch.randperm(n)[:B]] if slots == "all" else slots
    n = B if slots is None else n
    t, _, _ = inputs(B, D, 3, io, gate=gate, seed=B + D)
    state = torch.randn(n, D, device="cuda")
    dev = None if slots is None else torch.tensor(at, dtype=torch.int32, device="cuda")
    for k in range(3):
        y0, ey, st, est = step_reference(t, state, at, k, io == "bf16")
        y = torch.full((B, D), 5.0, dtype=IO[io], device="cuda")
        cols = [None if t[v] is None else t[v][..., k].contiguous() for v in ("x", "r", "i", "z")]
        ssm.ssm_gated_state_update(state, *cols[:3], t["lam"], t["r_bias"], t["i_bias"], cols[3], y, slots=dev)
        skipped = np.isnan(y0[:, 0])
        assert bool((y[torch.from_numpy(skipped).cuda()] == 5).all())
        check(y[torch.from_numpy(~skipped).cuda()], (y0[~skipped], ey[~skipped]), f"step {k} y")
        check(state, (st, est), f"step {k} state")


def test_step_of_more_slots_than_a_bitmap_holds(cuda_device):
    n, D, at = 400_000, 8, [399_999, 5, 399_999, -1, 400_000, 5, 7]
    t, _, _ = inputs(7, D, 1, "f32", seed=53)
    state = torch.randn(n, D, device="cuda")
    y0, ey, st, est = step_reference(t, state, at, 0, False)
    y = torch.full((7, D), 5.0, device="cuda")
    cols = [t[v][..., 0].contiguous() for v in ("x", "r", "i", "z")]
    ssm.ssm_gated_state_update(state, *cols[:3], t["lam"], t["r_bias"], t["i_bias"], cols[3], y,
                               slots=torch.tensor(at, dtype=torch.int32, device="cuda"))
    rows = [0, 1, 2, 5, 6]
    check(y[rows], (y0[rows], ey[rows]), "many slots y")
    check(state, (st, est), "many slots state")
    assert bool((y[[3, 4]] == 5).all())


def test_step_strided_rows(cuda_device):
    """Rows sliced from wider tensors, at odd offsets; the slots of a pool that holds more per slot."""
    for io in IO.values():
        wide = torch.randn(4, 200, device="cuda").to(io)
        x, r, i, z = wide[:, 1:38], wide[:, 38:75], wide[:, 76:113], wide[:, 120:157]
        pool = torch.randn(6, 50, device="cuda")
        keep, state = pool.clone(), pool[:, 3:40]
        lam = torch.linspace(-6, 1, 37, device="cuda")
        y = torch.zeros(4, 90, dtype=io, device="cuda")
        slots = torch.tensor([5, 0, 2, 3], dtype=torch.int32, device="cuda")
        t = dict(x=x[..., None], r=r[..., None], i=i[..., None], z=z[..., None], lam=lam, r_bias=None, i_bias=None)
        y0, ey, st, est = step_reference(t, state, slots.tolist(), 0, io == torch.bfloat16)
        ssm.ssm_gated_state_update(state, x, r, i, lam, None, None, z, y[:, 5:42], slots=slots)
        check(y[:, 5:42], (y0, ey), "strided y")
        check(state, (st, est), "strided state")
        assert torch.equal(pool[:, :3], keep[:, :3]) and torch.equal(pool[:, 40:], keep[:, 40:])
        assert not bool(y[:, :5].any()) and not bool(y[:, 42:].any())


def test_prefill_then_decode_is_the_scan(cuda_device):
    """A prompt through the scan and the rest token by token on the slots of a pool: the whole scan."""
    B, D, L, cut = 3, 60, 40, 29
    t, _, _ = inputs(B, D, L, "f32", seed=31, state=False)
    want = reference(**t)
    head = {k: t[k][..., :cut] for k in ("x", "r", "i", "z")}
    y, last = ssm.gated_scan_fwd(**dict(t, **head))
    pool = torch.full((8, D), float("nan"), device="cuda")
    slots = torch.tensor([6, 1, 4], dtype=torch.int32, device="cuda")
    pool[slots.long()] = last
    ys = [y]
    for k in range(cut, L):
        c = [t[n][..., k].contiguous() for n in ("x", "r", "i", "z")]
        yk = torch.empty(B, D, device="cuda")
        ssm.ssm_gated_state_update(pool, *c[:3], t["lam"], t["r_bias"], t["i_bias"], c[3], yk, slots=slots)
        ys.append(yk[..., None])
    check(torch.cat(ys, -1), want["y"], "prefill and decode y")
    check(pool[slots.long()], want["last"], "prefill and decode state")
    assert bool(torch.isnan(pool[[0, 2, 3, 5, 7]]).all())


# ------------------------------------------------------------------------------- streams, graphs, refusals
def test_captured_and_replayed_on_another_stream(cuda_device):
    t, dy, dlast = inputs(2, 50, 700, "bf16", seed=37)
    eager = run_all(t, dy, dlast, True)
    a = [t[k] for k in ("x", "r", "i", "lam", "r_bias", "i_bias", "z")]
    y, last, out = torch.zeros_like(t["x"]), torch.zeros(2, 50, device="cuda"), {k: torch.zeros_like(eager[k]) for k in GRADS}
    ck, ws = ssm.new_gated_checkpoints(2, 50, 700), ssm.new_gated_workspace(2, 50, 700, True)

    def step():
        ssm.ssm_gated_scan_fwd(*a, y, last, initial_state=t["initial_state"], checkpoints=ck)
        ssm.ssm_gated_scan_bwd(*a, dy, out["dx"], out["dr"], out["di"], out["dlam"], out["dr_bias"], out["di_bias"], out["dz"], ws,
                               initial_state=t["initial_state"], dlast_state=dlast, dinitial_state=out["dinitial_state"], checkpoints=ck)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for k in range(2):
        for v in (y, last, *out.values()):
            v.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager["y"]) and torch.equal(last, eager["last"])
        assert all(torch.equal(out[n], eager[n]) for n in GRADS)
    got = {}
    side.wait_stream(torch.cuda.current_stream())
    got["y"], got["last"] = ssm.gated_scan_fwd(**t, stream=side)
    got.update(ssm.gated_scan_bwd(**t, dy=dy, dlast_state=dlast, stream=side.cuda_stream))
    side.synchronize()
    assert all(torch.equal(got[n], eager[n]) for n in ("y", "last"))
    assert all(torch.equal(got[n], eager[n]) for n in ("dx", "dr", "di", "dz"))


def test_two_streams_at_once(cuda_device):
    """Calls that overlap, each with its own buffers, give what they give alone."""
    jobs = [inputs(2, 300, 1500, "bf16", seed=s) for s in (59, 61)]
    alone = [run_all(t, dy, dlast, True) for t, dy, dlast in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = [None, None]
    for _ in range(3):
        for k, ((t, dy, dlast), stream) in enumerate(zip(jobs, streams)):
            with torch.cuda.stream(stream):
                got[k] = run_all(t, dy, dlast, True)
    torch.cuda.synchronize()
    for a, b in zip(alone, got):
        assert all(torch.equal(a[n], b[n]) for n in a)


def test_refusals(cuda_device):
    t, dy, dlast = inputs(2, 5, 16, "bf16")
    good = dict(t)

    def refused(exc, **kw):
        with pytest.raises(exc):
            ssm.gated_scan_fwd(**dict(good, **kw))

    refused(TypeError, r=t["r"].float())
    refused(TypeError, lam=t["lam"].double())
    refused(TypeError, lengths=torch.tensor([3, 4], device="cuda"))
    refused(ValueError, r=t["r"][..., :8])
    refused(ValueError, x=t["x"].transpose(1, 2).contiguous().transpose(1, 2))
    refused(ValueError, lam=t["lam"][:4])
    refused(ValueError, lam=t["lam"].cpu())
    refused(ValueError, initial_state=torch.zeros(2, 10, device="cuda")[:, ::2])
    refused(ValueError, reset=torch.zeros(2, 17, dtype=torch.uint8, device="cuda"))
    refused(binding.SsmError, checkpoints=torch.empty(16, dtype=torch.uint8, device="cuda"))
    refused(ValueError, checkpoints=torch.empty(1 << 16, dtype=torch.uint8))
    refused(binding.SsmError, c=-1.0)
    a = [t[k] for k in ("x", "r", "i", "lam", "r_bias", "i_bias", "z")]
    last = torch.empty(2, 5, device="cuda")
    with pytest.raises(binding.SsmError):
        ssm.ssm_gated_scan_fwd(*a, t["x"], last)  # y is an input
    with pytest.raises(binding.SsmError):
        ssm.ssm_gated_scan_fwd(*a, torch.empty(2, 1, 16, dtype=torch.bfloat16, device="cuda").expand(2, 5, 16), last)
    with pytest.raises(binding.SsmError):
        ssm.gated_scan_bwd(**t, dy=dy, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert ssm.ssm_gated_scan_fwd(*a, t["x"], last, check=False) == binding.SSM_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        ssm.ssm_gated_state_update(torch.zeros(2, 6, device="cuda"), *(v[..., 0].contiguous() for v in (t["x"], t["r"], t["i"])), t["lam"],
                                   None, None, None, torch.empty(2, 5, dtype=torch.bfloat16, device="cuda"))
