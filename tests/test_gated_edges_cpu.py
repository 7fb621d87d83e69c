"""The gated recurrence without a device, at its edges: the kernels' own arithmetic compiled for the host."""
import os
import subprocess

import pytest
import torch

import selective_state_space_16_b200 as ssm
from selective_state_space_16_b200 import binding, build, gated

CSRC = build.CSRC


@pytest.fixture(autouse=True, scope="module")
def built():
    build.build()

REACH = r"""
#include <cstdio>
#include "gated_math.cuh"
int main() {
    long long bs, ds, most, at;
    int before;
    while (scanf("%lld %lld %lld %d %lld", &bs, &ds, &most, &before, &at) == 5) {
        ssm::GatedTensor t{};
        t.bs = bs, t.ds = ds, t.most = most, t.before = before;
        ssm::Reach r{-15, 15};
        ssm::narrow(r, t, at);
        printf("%d %d\n", r.low, r.high);
    }
}
"""


@pytest.fixture(scope="module")
def reach(tmp_path_factory):
    at = tmp_path_factory.mktemp("reach")
    (at / "reach.cu").write_text(REACH)
    subprocess.check_call([build.NVCC, *build.ARCH, "-std=c++17", "-I", CSRC, "-o", str(at / "reach"), str(at / "reach.cu")])

    def run(rows):
        text = "\n".join(" ".join(str(v) for v in r) for r in rows)
        out = subprocess.run([str(at / "reach")], input=text, capture_output=True, text=True, check=True).stdout
        return [tuple(int(v) for v in line.split()) for line in out.splitlines()]
    return run


def test_no_row_reaches_outside_its_operand(reach):
    """Whole vectors may reach up to 15 steps beside a row as far as the operand goes, from its first row's begin to its
    last one's end, at any distance of the rows; nowhere with rows that go backwards in memory."""
    rows, want = [], []
    for bs, ds in ((3000, 1000), (1000, 5000), (0, 7), (7, 0), (0, 0), (1, 3), ((1 << 31) + 16, 128), (5, 1 << 33), (-3000, 1000),
                   (3000, -1000), (-5, -20), (-((1 << 31) + 16), 128), (128, -((1 << 31) + 16)), (-(1 << 33), -7), (-(1 << 32), 0),
                   (-((1 << 32) + 3), 5), (1 << 31, -(1 << 31))):
        B, D = 3, 4
        up = bs >= 0 and ds >= 0
        for b in range(B):
            for d in range(D):
                at, most = b * bs + d * ds, (B - 1) * bs + (D - 1) * ds
                rows.append((bs, ds, most, 15 if up else 0, at))
                want.append((-min(at, 15), min(most - at, 15)) if up else (0, 0))
    got = reach(rows)
    assert len(got) == len(want)
    for r, g, w in zip(rows, got, want):
        assert w[0] <= g[0] and g[1] <= w[1], (r, g, w)  # not outside
        assert g == w or not r[3], (r, g, w)                       # and as far as it may


def test_an_output_may_be_no_input():
    """As the header says: not even a parameter, a state or a list.  (initial_state and last_state may be one buffer, and
    dlast_state and dinitial_state.)"""
    lib, ok = ssm.load(), binding.SSM_ERR_LAUNCH  # (accepted arguments get as far as the device, which is not here)
    P = 1 << 20
    ins = {k: P * (j + 1) for j, k in enumerate(("x", "r", "i", "z", "lam", "r_bias", "i_bias", "h0", "lengths", "reset"))}
    B, D, L = 2, 3, 8
    st = (D * L, L)

    def args():
        return gated._ARGS.pack(ins["x"], *st, ins["r"], *st, ins["i"], *st, ins["z"], *st, *(ins[k] for k in (
            "lam", "r_bias", "i_bias", "h0", "lengths", "reset")), L, B, D, binding.SSM_F32, 8.0)

    def fwd(y=50 * P, last=51 * P):
        return lib.ssm_gated_scan_fwd(args(), gated._OUT.pack(y, *st), last, None, 0, None)

    def bwd(dy=60 * P, dlast=61 * P, **out):
        o = dict({k: P * (70 + j) for j, k in enumerate(("dx", "dr", "di", "dz", "dlam", "drb", "dib", "dh0"))}, **out)
        g = gated._GRADS.pack(dy, *st, dlast, o["dx"], *st, o["dr"], *st, o["di"], *st, o["dz"], *st, o["dlam"], o["drb"], o["dib"], o["dh0"])
        return lib.ssm_gated_scan_bwd(args(), g, None, 0, 90 * P, 1 << 20, None)

    if torch.cuda.is_available():
        pytest.skip("accepted calls would run on these addresses")
    assert fwd() == ok and fwd(last=ins["h0"]) == ok and fwd(last=0) == ok
    assert bwd() == ok and bwd(dh0=61 * P) == ok and bwd(dh0=0, dlam=0, drb=0, dib=0) == ok
    for k, p in ins.items():
        assert fwd(y=p) == binding.SSM_ERR_INVALID_ARG, k
        assert fwd(last=p) == (ok if k == "h0" else binding.SSM_ERR_INVALID_ARG), k
        for out in ("dx", "dr", "di", "dz", "dlam", "drb", "dib", "dh0"):
            assert bwd(**{out: p}) == binding.SSM_ERR_INVALID_ARG, (out, k)
    for out in ("dx", "dr", "di", "dz", "dlam", "drb", "dib", "dh0"):
        assert bwd(**{out: 60 * P}) == binding.SSM_ERR_INVALID_ARG, out
        assert bwd(**{out: 61 * P}) == (ok if out == "dh0" else binding.SSM_ERR_INVALID_ARG), out


def test_limits_of_a_step():
    """batch at most 65535, dim below 2^31 - 65536: refused before any device is asked for."""
    def step(b, d):
        P = 1 << 20
        return ssm.load().ssm_gated_state_update(gated._STEP.pack(P, d, 0, 2 * P, 2 * P, 2 * P, 0, 3 * P, d, d, d, d, d, P, 0, 0, b, d, b,
                                                                  binding.SSM_BF16, 8.0), None)
    if torch.cuda.is_available():
        pytest.skip("accepted calls would run on these addresses")
    assert step(65535, 8) == step(1, (1 << 31) - 65537) == binding.SSM_ERR_LAUNCH  # (accepted: no device)
    for b, d in ((65536, 8), (1, (1 << 31) - 65536), (1, (1 << 31) - 1)):
        assert step(b, d) == binding.SSM_ERR_UNSUPPORTED, (b, d)
