"""The gated recurrence's C ABI without a device: sizes, refusals, struct layouts; and the 64-bit
reference of the GPU tests against central differences."""
import numpy as np
import pytest
import torch

import selective_state_space_16_b200 as ssm
from gated_reference import reference
from selective_state_space_16_b200 import binding, gated

IV, UN, WS, OK = binding.SSM_ERR_INVALID_ARG, binding.SSM_ERR_UNSUPPORTED, binding.SSM_ERR_WORKSPACE, binding.SSM_OK
P = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from selective_state_space_16_b200 import build as b
    b.build()
    return ssm.load()


def args(x=P, r=P, i=P, z=0, lam=P, r_bias=0, i_bias=0, h0=0, lengths=0, reset=0, L=8, b=2, d=3, io=binding.SSM_BF16, c=8.0):
    st = (d * L, L)
    return gated._ARGS.pack(x, *st, r, *st, i, *st, z, *st, lam, r_bias, i_bias, h0, lengths, reset, L, b, d, io, c)


def fwd(lib, y=2 * P, ys=(24, 8), last=None, ck=None, ckb=1 << 20, **kw):
    return lib.ssm_gated_scan_fwd(args(**kw), gated._OUT.pack(y, *ys), last, ck, ckb, None)


def bwd(lib, dy=2 * P, dx=3 * P, dr=4 * P, di=5 * P, dz=0, dlam=0, ws=P, wsb=1 << 20, ds=(24, 8), ck=None, ckb=1 << 20, **kw):
    st = (24, 8)
    g = gated._GRADS.pack(dy, *st, 0, dx, *ds, dr, *st, di, *st, dz, *st, dlam, 0, 0, 0)
    return lib.ssm_gated_scan_bwd(args(**kw), g, ck, ckb, ws, wsb, None)


def test_forward_refusals(lib):
    for bad in (dict(x=0), dict(r=0), dict(i=0), dict(lam=0), dict(y=0), dict(b=-1), dict(d=-1), dict(L=-1), dict(io=7),
                dict(c=0.0), dict(c=-1.0), dict(c=float("inf")), dict(c=float("nan")), dict(x=P + 1), dict(z=P + 1), dict(lam=P + 2),
                dict(h0=P + 2), dict(lengths=P + 1), dict(y=2 * P + 1), dict(y=P), dict(y=6 * P, z=6 * P), dict(ck=P + 8),
                dict(ys=(0, 8)), dict(ys=(24, 0)), dict(ys=(16, 8)), dict(ys=(24, 7)), dict(io=binding.SSM_F32, x=P + 2)):
        assert fwd(lib, **bad) == IV, bad
    assert fwd(lib, b=65536, d=32768) == UN
    assert fwd(lib, L=(1 << 31) - 1024) == UN
    assert lib.ssm_gated_scan_fwd(None, gated._OUT.pack(P, 24, 8), None, None, 0, None) == IV
    assert lib.ssm_gated_scan_fwd(args(), None, None, None, 0, None) == IV
    assert fwd(lib, ck=P, ckb=16) == WS
    assert fwd(lib, b=0, x=0, r=0, i=0, y=0) == OK
    assert fwd(lib, d=0) == OK


def test_backward_refusals(lib):
    for bad in (dict(dy=0), dict(dx=0), dict(dr=0), dict(di=0), dict(z=6 * P), dict(dx=P), dict(dr=2 * P), dict(dx=3 * P + 1),
                dict(dy=2 * P + 1), dict(dlam=P + 1), dict(ck=P + 4), dict(ds=(8, 8)), dict(x=0), dict(c=0.0), dict(io=2)):
        assert bwd(lib, **bad) == IV, bad
    assert bwd(lib, ws=None) == WS
    assert bwd(lib, ws=P + 16) == WS
    assert bwd(lib, wsb=16) == WS
    assert bwd(lib, d=0) == OK
    assert lib.ssm_gated_scan_bwd(args(), None, None, 0, P, 1 << 20, None) == IV
    assert bwd(lib, ck=P, ckb=16) == WS


def test_step_refusals(lib):
    def step(state=P, ss=8, slots=0, x=2 * P, r=2 * P, i=2 * P, z=0, y=3 * P, xs=8, ys=8, lam=P, b=2, d=8, n=2, io=binding.SSM_BF16,
             c=8.0):
        return lib.ssm_gated_state_update(gated._STEP.pack(state, ss, slots, x, r, i, z, y, xs, xs, xs, xs, ys, lam, 0, 0, b, d, n, io,
                                                           c), None)
    for bad in (dict(state=0), dict(x=0), dict(r=0), dict(i=0), dict(y=0), dict(lam=0), dict(b=-1), dict(d=-1), dict(n=-1), dict(io=5),
                dict(c=0.0), dict(ss=7), dict(ys=7), dict(y=2 * P), dict(state=P + 2), dict(x=2 * P + 1), dict(slots=P + 2)):
        assert step(**bad) == IV, bad
    assert step(b=65536) == UN
    assert step(b=0) == OK and step(d=0) == OK
    assert lib.ssm_gated_state_update(None, None) == IV


def test_sizes(lib):
    assert ssm.ssm_gated_checkpoint_size(2, 3, 100) >= 2 * 3 * (100 + 15) // 8 * 4
    assert ssm.ssm_gated_checkpoint_size(2, 3, 100) % 16 == 0
    assert ssm.ssm_gated_checkpoint_size(-1, 3, 100) == 0
    assert ssm.ssm_gated_checkpoint_size(1 << 16, 1 << 15, 1) == 0
    with_, without = (ssm.ssm_gated_bwd_workspace_size(2, 300, 1000, k) for k in (True, False))
    assert with_ % 256 == 0 and with_ >= 3 * 600 * 4 and without >= with_ + ssm.ssm_gated_checkpoint_size(2, 300, 1000)
    assert ssm.ssm_gated_bwd_workspace_size(2, -3, 4) == 0


def test_packed_structs_have_the_headers_layout(tmp_path):
    import os
    import subprocess
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "ssm_gated.h"\nint main(void) { printf("%zu %zu %zu %zu %zu %zu\\n",'
                   "sizeof(ssm_gated_args_t), sizeof(ssm_gated_grads_t), sizeof(ssm_gated_step_t), sizeof(ssm_gated_out_t),"
                   "offsetof(ssm_gated_args_t, c), offsetof(ssm_gated_step_t, c)); return 0; }\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.check_call(["gcc", "-I", os.path.join(root, "include"), "-o", str(tmp_path / "s"), str(src)])
    got = [int(v) for v in subprocess.check_output([str(tmp_path / "s")]).split()]
    assert got == [gated._ARGS.size, gated._GRADS.size, gated._STEP.size, gated._OUT.size, gated._ARGS.size - 4,
                   gated._STEP.size - 8]


def test_binding_refuses_what_it_can_see():
    x = torch.zeros(2, 3, 8)
    with pytest.raises(ValueError, match="CUDA"):
        ssm.gated_scan_fwd(x, x, x, torch.zeros(3))
    a = (x, x, x, torch.zeros(3), None, None, None, x, None)
    with pytest.raises(ValueError, match="CUDA"):
        ssm.ssm_gated_scan_fwd(*a)
    with pytest.raises(TypeError):
        ssm.ssm_gated_scan_fwd(x.half(), *a[1:])


@pytest.mark.parametrize("gate,lengths,reset", [(True, None, None), (False, [5, 0], None), (True, [6, 3], [[0, 0, 1, 0, 0, 0], [1, 0, 0, 0, 0, 0]])])
def test_reference_gradients_are_the_derivatives(gate, lengths, reset):
    g = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    B, D, L = 2, 2, 6
    t = dict(x=rnd(B, D, L), r=rnd(B, D, L), i=rnd(B, D, L), lam=rnd(D) - 2, r_bias=rnd(D), i_bias=rnd(D), initial_state=rnd(B, D))
    if gate:
        t["z"] = rnd(B, D, L)
    more = dict(lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32),
                reset=None if reset is None else torch.tensor(reset, dtype=torch.uint8))
    dy, dlast = rnd(B, D, L), rnd(B, D)
    out = reference(**t, **more, dy=dy, dlast=dlast)
    inside = torch.arange(L) < (torch.full((B,), L) if lengths is None else torch.tensor(lengths))[:, None]

    def loss():
        o = reference(**t, **more)
        return float((o["y"][0] * (dy * inside[:, None]).numpy()).sum() + (o["last"][0] * dlast.numpy()).sum())

    names = dict(x="dx", r="dr", i="di", z="dz", lam="dlam", r_bias="dr_bias", i_bias="di_bias", initial_state="dinitial_state")
    for k, v in t.items():
        want = np.zeros(v.shape)
        for at in np.ndindex(*v.shape):
            keep, step = float(v[at]), 1e-6
            v[at] = keep + step
            up = loss()
            v[at] = keep - step
            want[at] = (up - loss()) / (2 * step)
            v[at] = keep
        # central differences: step^2 f''' / 6 and 2^-52 |loss| / step
        np.testing.assert_allclose(out[names[k]][0], want, rtol=1e-6, atol=1e-8, err_msg=k)
