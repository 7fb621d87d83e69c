"""The gated recurrence without a device, at its edges: the kernels' own arithmetic compiled for the host."""
import os
import subprocess

import pytest

from selective_state_space_16_b200 import build

CSRC = build.CSRC

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
