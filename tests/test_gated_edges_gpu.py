"""The gated linear recurrence at its edges (-m gpu): what lies behind the buffers it is given, steps outside a row
beside infinities and NaNs, the output gate, the ends of the parameters' range."""
import numpy as np
import pytest
import torch

import selective_state_space_16_b200 as ssm
import test_gated_gpu
from gated_reference import check, reference
from selective_state_space_16_b200 import binding, gated
from test_gated_gpu import IO, compare, inputs, step_reference

pytestmark = pytest.mark.gpu


def off_vectors(v, by):
    """The same values, `by` elements behind a 16-byte boundary."""
    flat = torch.empty(v.numel() + by + 16, dtype=v.dtype, device=v.device)
    at = flat[by:by + v.numel()].view(v.shape)
    return at.copy_(v)


def guarded(nbytes):
    """A buffer of that many bytes, and the sentinels behind it."""
    whole = torch.full((nbytes + 65536,), 0x5a, dtype=torch.uint8, device="cuda")
    return whole[:nbytes], whole[nbytes:]


def forward_backward(t, dy, dlast, ck, ws, ck_bwd):
    B, D, L = t["x"].shape
    a = [t[k] for k in ("x", "r", "i", "lam", "r_bias", "i_bias", "z")]
    more = dict(initial_state=t["initial_state"], lengths=t["lengths"], reset=t["reset"])
    y, last, dh0 = torch.zeros(B, D, L, dtype=dy.dtype, device="cuda"), torch.empty(B, D, device="cuda"), torch.empty(B, D, device="cuda")
    out = {k: torch.empty(B, D, L, dtype=dy.dtype, device="cuda") for k in ("dx", "dr", "di")}
    out["dz"] = None if t["z"] is None else torch.empty_like(out["dx"])
    sums = [torch.empty(D, device="cuda") for _ in range(3)]
    ssm.ssm_gated_scan_fwd(*a, y, last, checkpoints=ck, **more)
    ssm.ssm_gated_scan_bwd(*a, dy, out["dx"], out["dr"], out["di"], *sums, out["dz"], ws, dlast_state=dlast, dinitial_state=dh0,
                           checkpoints=ck_bwd, **more)
    return dict(out, y=y, last=last, dinitial_state=dh0, **dict(zip(("dlam", "dr_bias", "di_bias"), sums)))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("by", [1, 3])
@pytest.mark.parametrize("B,D", [(1, 1), (1, 5), (3, 7)])
@pytest.mark.parametrize("L", [1, 5, 37, 100])
def test_nothing_behind_the_buffers_is_written(cuda_device, io, by, B, D, L):
    """Short rows that do not fill a block, off the 16-byte boundaries: checkpoints and workspace of exactly the sizes
    that the library asks for."""
    t, dy, dlast = inputs(B, D, L, io, seed=L + by)
    for k in ("x", "r", "i", "z"):
        t[k] = off_vectors(t[k], by)
    dy = off_vectors(dy, by)
    ck, behind_ck = guarded(ssm.ssm_gated_checkpoint_size(B, D, L))
    for given in (True, False):
        ws, behind_ws = guarded(ssm.ssm_gated_bwd_workspace_size(B, D, L, given))
        got = forward_backward(t, dy, dlast, ck, ws, ck if given else None)
        assert bool((behind_ck == 0x5a).all()) and bool((behind_ws == 0x5a).all())
        compare(got, t, dy, dlast, f"{B}x{D}x{L} off by {by}")


def with_and_without_checkpoints(t, dy, dlast):
    """The results, which are the same bit for bit whether the backward has the forward's checkpoints or makes its own."""
    sizes = t["x"].shape
    ck = ssm.new_gated_checkpoints(*sizes)
    got, own = (forward_backward(t, dy, dlast, ck, ssm.new_gated_workspace(*sizes, g is not None), g) for g in (ck, None))
    for k, v in got.items():
        assert v is own[k] or torch.equal(v.view(torch.uint8), own[k].view(torch.uint8)), k
    return got


EDGES = [(2, 3, 701), (2, 3, 37), (3, 7, 101), (2, 600, 301), (2, 3, 9001)]  # rows split, shared warps, a warp each, clusters


def set_rows(v, rows):
    for b, value in enumerate(rows):
        if value is not None:
            v[b] = value


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("B,D,L", EDGES)
@pytest.mark.parametrize("before", [float("nan"), float("inf")])
def test_what_came_before_a_first_reset_reaches_no_gradient(cuda_device, io, B, D, L, before):
    """A reset at step 0 drops the initial state, wherever the rows lie: the parameters' sums too."""
    t, dy, dlast = inputs(B, D, L, io, reset=0.01, seed=L)
    t["reset"][:, 0] = 1
    t["initial_state"][:] = before
    got = with_and_without_checkpoints(t, dy, dlast)
    compare(got, t, dy, dlast, f"{B}x{D}x{L}")
    assert all(bool(torch.isfinite(v).all()) for v in got.values())


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("B,D,L", EDGES)
@pytest.mark.parametrize("state,dstate", [(float("nan"), None), (float("inf"), None), (None, float("inf")), (None, float("nan"))])
def test_rows_without_steps_reach_no_sum(cuda_device, io, B, D, L, state, dstate):
    """A batch row of length 0 hands its state and the state's gradient on and has no part in anything else."""
    t, dy, dlast = inputs(B, D, L, io, lengths=[L - 2, 0] + [7] * (B - 2), seed=L)
    set_rows(t["initial_state"], [None, state])
    set_rows(dlast, [None, dstate])
    got = with_and_without_checkpoints(t, dy, dlast)
    compare(got, t, dy, dlast, f"{B}x{D}x{L}")
    assert all(bool(torch.isfinite(got[k]).all()) for k in ("dlam", "dr_bias", "di_bias"))
    for k in ("dx", "dr", "di", "dz"):
        assert not bool(got[k][1].any()), k


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("B,D,L", EDGES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_gradients_behind_a_row_are_zeros_beside_any_state(cuda_device, io, B, D, L, bad):
    """A row whose last step, a reset, leaves a state that is not finite: behind it are zeros, and the sums that
    this step does not enter stay finite."""
    n = L - 3
    t, dy, dlast = inputs(B, D, L, io, lengths=[n] * B, reset=0.0, seed=L)
    t["reset"][:, n - 1] = 1
    t["x"][0, :, n - 1] = bad
    got = with_and_without_checkpoints(t, dy, dlast)
    for k in ("dx", "dr", "di", "dz"):
        assert not bool(got[k][:, :, n:].any()), k
    compare(got, t, dy, dlast, f"{B}x{D}x{L}")
    assert all(bool(torch.isfinite(got[k]).all()) for k in ("dlam", "dr_bias"))


@pytest.mark.parametrize("low,high", [(-1.0, 1.0), (-20.0, -1.0), (1.0, 20.0), (-90.0, -60.0)])
def test_the_output_gate_is_right_to_the_rounding_of_bf16(cuda_device, low, high):
    """y of bf16 is the value in 32 bits rounded once: within that value's bound and half a step, 2^-8 of it, far on
    the gate's shut side too (the rounding is of a value that may be off by the bound: hence the product)."""
    t, _, _ = inputs(2, 24, 500, "bf16", seed=73)
    t["z"] = torch.linspace(low, high, 2 * 24 * 500, device="cuda").view(2, 24, 500).to(torch.bfloat16)
    val, err = reference(**t)["y"]
    tol = err * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(val)
    y, _ = ssm.gated_scan_fwd(**t)
    check(y, (val, tol), f"gate {low} .. {high}")
    state = torch.zeros(1, 24, device="cuda").expand(2, 24).clone()
    cols = [t[k][..., 3].contiguous() for k in ("x", "r", "i", "z")]
    y = torch.empty(2, 24, dtype=torch.bfloat16, device="cuda")
    ssm.ssm_gated_state_update(state, *cols[:3], t["lam"], t["r_bias"], t["i_bias"], cols[3], y)
    one = {k: t[k][..., 3:4] for k in ("x", "r", "i", "z")}
    val, err = reference(**dict(t, **one, initial_state=None))["y"]
    check(y[..., None], (val, err * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(val)), "gate of a step")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("B,D,L", EDGES)
def test_decay_exponents_beyond_fp32(cuda_device, io, B, D, L):
    """c softplus(lam) past the largest fp32 forgets at once (a = 0, m = 1), and steps outside a row, whose gate is
    shut, still pass the state on."""
    t, dy, dlast = inputs(B, D, L, io, lengths=[L - 3] * B, seed=L)
    y, last = ssm.gated_scan_fwd(**t, c=3e38)
    grads = ssm.gated_scan_bwd(**t, dy=dy, dlast_state=dlast, c=3e38)
    want = reference(**t, dy=dy, dlast=dlast, c=3e38, bf16=io == "bf16")
    for k, w in want.items():
        check(dict(grads, y=y, last=last)[k], w, f"c=3e38 {k}")
    some, all_ = (dict(t, lam=torch.full((D,), v, device="cuda")) for v in (1e30, float("inf")))
    for a, b in zip(ssm.gated_scan_fwd(**some), ssm.gated_scan_fwd(**all_)):
        assert torch.equal(a, b) and bool(torch.isfinite(a).all())
    some, all_ = (ssm.gated_scan_bwd(**w, dy=dy, dlast_state=dlast) for w in (some, all_))
    for k, v in some.items():
        assert torch.equal(v, all_[k]) and bool(torch.isfinite(v).all()), k
    frozen = ssm.gated_scan_fwd(**dict(t, lam=torch.full((D,), -200.0, device="cuda")), c=3e38)[1]  # c softplus(lam) is 0
    assert torch.equal(frozen, t["initial_state"])


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_a_shut_gate_keeps_the_state_of_any_channel_in_a_step(cuda_device, io):
    x = torch.randn(3, 40, device="cuda").to(IO[io])
    shut = torch.full_like(x, float("-inf"))
    lam = torch.linspace(-9, 3, 40, device="cuda")
    lam[:20] = 1e38
    state = torch.randn(3, 40, device="cuda")
    keep, y = state.clone(), torch.empty_like(x)
    ssm.ssm_gated_state_update(state, x, shut, x, lam, None, None, None, y)
    assert torch.equal(state, keep)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("L", [37, 100, 301])
def test_rows_that_go_backwards_in_memory(cuda_device, io, L):
    """Inputs of negative strides, which the C ABI takes.  (A row is composed in groups that lie on 16 bytes, so the same row
    elsewhere is the same to the bound, not to the bit.)"""
    B, D = 3, 7
    t, _, _ = inputs(B, D, L, io, seed=L)
    want = reference(**t, bf16=io == "bf16")
    y, last = torch.empty_like(t["x"]), torch.empty(B, D, device="cuda")
    packed, kept = [], []
    for k in ("x", "r", "i", "z"):
        kept.append(t[k].flip(0, 1).contiguous())
        packed += [kept[-1].data_ptr() + ((B - 1) * D + D - 1) * L * kept[-1].element_size(), -D * L, -L]
    args = gated._ARGS.pack(*packed, *(t[k].data_ptr() for k in ("lam", "r_bias", "i_bias", "initial_state")), 0, 0, L, B, D,
                            binding.SSM_BF16 if io == "bf16" else binding.SSM_F32, 8.0)
    code = ssm.load().ssm_gated_scan_fwd(args, gated._OUT.pack(y.data_ptr(), D * L, L), last.data_ptr(), None, 0,
                                         torch.cuda.current_stream().cuda_stream)
    assert code == binding.SSM_OK
    check(y, want["y"], "y")
    check(last, want["last"], "last")


@pytest.mark.parametrize("B,D,L", EDGES + [(2, 3, 0)])
def test_the_states_gradient_may_stay_in_its_buffer(cuda_device, B, D, L):
    """dinitial_state over dlast_state, as a backward taken block by block carries it."""
    t, dy, dlast = inputs(B, D, L, "bf16", lengths=[L, 0] + [L // 2] * (B - 2), seed=79)
    want = ssm.gated_scan_bwd(**t, dy=dy, dlast_state=dlast)["dinitial_state"]
    a = [t[k] for k in ("x", "r", "i", "lam", "r_bias", "i_bias", "z")]
    out = [torch.empty_like(dy) for _ in range(4)]
    ssm.ssm_gated_scan_bwd(*a, dy, *out[:3], None, None, None, out[3], ssm.new_gated_workspace(B, D, L), initial_state=t["initial_state"],
                           lengths=t["lengths"], dlast_state=dlast, dinitial_state=dlast)
    assert torch.equal(dlast, want)


def beside(v):
    """The elements of v's buffer that are not v's, as a copy with v's filled in."""
    keep = v.clone()
    v.fill_(7.0)
    whole = v._base.clone()
    v.copy_(keep)
    return whole


def placed(shape, dtype, by, pad):
    """A tensor that starts `by` elements into a buffer of sevens and has `pad` of them between its rows."""
    flat = torch.full((shape[0] * shape[1] * (shape[2] + pad) + by + 64,), 7.0, dtype=dtype, device="cuda")
    return flat.as_strided(shape, (shape[1] * (shape[2] + pad), shape[2] + pad, 1), by)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("L", [5, 37, 100, 250, 541])
@pytest.mark.parametrize("first,second", [((3, 1), (0, 0)), ((0, 0), (5, 2)), ((1, 8), (6, 1))])
def test_checkpoints_go_by_position(cuda_device, io, L, first, second):
    """The checkpoints of a forward are read by a backward whose operands lie at other addresses and strides; what lies
    beside the outputs' rows stays."""
    B, D = 3, 7
    t, dy, dlast = inputs(B, D, L, io, lengths=[L, L // 2, 1], seed=L)
    ck, ws = ssm.new_gated_checkpoints(B, D, L), ssm.new_gated_workspace(B, D, L, True)
    y, last, dh0 = placed(dy.shape, dy.dtype, *first), torch.empty(B, D, device="cuda"), torch.empty(B, D, device="cuda")
    y.zero_()
    a = {k: placed(dy.shape, dy.dtype, *first).copy_(t[k]) for k in ("x", "r", "i", "z")}
    more = dict(initial_state=t["initial_state"], lengths=t["lengths"])
    ssm.ssm_gated_scan_fwd(a["x"], a["r"], a["i"], t["lam"], t["r_bias"], t["i_bias"], a["z"], y, last, checkpoints=ck, **more)
    a = {k: placed(dy.shape, dy.dtype, *second).copy_(t[k]) for k in ("x", "r", "i", "z")}
    out = {k: placed(dy.shape, dy.dtype, by, pad) for k, by, pad in (("dx", 7, 1), ("dr", 1, 0), ("di", 0, 8), ("dz", 9, 7))}
    sums = [torch.empty(D, device="cuda") for _ in range(3)]
    ssm.ssm_gated_scan_bwd(a["x"], a["r"], a["i"], t["lam"], t["r_bias"], t["i_bias"], a["z"], dy, out["dx"], out["dr"], out["di"], *sums,
                           out["dz"], ws, dlast_state=dlast, dinitial_state=dh0, checkpoints=ck, **more)
    got = dict(out, y=y, last=last, dinitial_state=dh0, **dict(zip(("dlam", "dr_bias", "di_bias"), sums)))
    compare(got, t, dy, dlast, f"L={L}")
    for k in ("y", *out):
        assert bool((beside(got[k]) == 7).all()), f"{k}: written beside its rows"


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("B,D", [(200, 8192), (2000, 600), (3000, 37)])
@pytest.mark.parametrize("kind", ["distinct", "repeated", "none"])
def test_steps_of_many_rows_per_block(cuda_device, io, B, D, kind):
    """More rows than a launch has blocks for, so that each block walks several: slots in any order with padding
    rows among them, slots named again by rows of the same block and of others, and rows without slots."""
    t, _, _ = inputs(B, D, 1, io, seed=B + D)
    g = torch.Generator().manual_seed(B)
    n = {"distinct": B + 50, "repeated": B // 8, "none": B - 9}[kind]  # (none: the last rows have no state)
    at = list(range(B)) if kind == "none" else torch.randperm(n, generator=g)[:B].tolist() if kind == "distinct" else \
        torch.randint(0, n, (B,), generator=g).tolist()
    if kind != "none":
        at[3::11] = [-1] * len(at[3::11])
        at[-1], at[7] = n, -(2 ** 31)
    state = torch.randn(n, D, generator=g).cuda()
    y0, ey, st, est = step_reference(t, state, at, 0, io == "bf16")
    y = torch.full((B, D), 5.0, dtype=IO[io], device="cuda")
    cols = [t[k][..., 0].contiguous() for k in ("x", "r", "i", "z")]
    ssm.ssm_gated_state_update(state, *cols[:3], t["lam"], t["r_bias"], t["i_bias"], cols[3], y,
                               slots=None if kind == "none" else torch.tensor(at, dtype=torch.int32, device="cuda"))
    skipped = np.isnan(y0[:, 0])
    assert bool((y[torch.from_numpy(skipped).cuda()] == 5).all())
    check(y[torch.from_numpy(~skipped).cuda()], (y0[~skipped], ey[~skipped]), "y")
    check(state, (st, est), "state")


@pytest.mark.parametrize("io,D", [("f32", 1800), ("f32", 2368), ("bf16", 1800), ("bf16", 2400)])
def test_rows_around_a_wave(cuda_device, io, D):
    """As many long rows as the GPU holds warps of a kernel, and a few more or less: a warp each or two."""
    test_gated_gpu.test_many_long_rows(cuda_device, io, D, 4100)
