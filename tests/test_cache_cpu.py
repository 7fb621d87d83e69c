"""The state cache's C ABI without a device: sizes and refusals."""
import pytest
import torch

import selective_state_space_16_b200 as ssm
from selective_state_space_16_b200 import binding, cache

IV, UN, WS, OK = binding.SSM_ERR_INVALID_ARG, binding.SSM_ERR_UNSUPPORTED, binding.SSM_ERR_WORKSPACE, binding.SSM_OK
P = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from selective_state_space_16_b200 import build as b
    b.build()
    return ssm.load()


def pool(data=P, page=64, slot=64, layer=64 * 8, layers=3):
    return cache._POOL.pack(data, page, slot, layer, layers)


def test_pool_refusals(lib):
    def call(p=None, k=1, slots=8):
        return lib.ssm_cache_free(pool() if p is None else p, k, slots, P, P, 0, 0, None)
    assert call() == OK  # an empty list
    for bad in (pool(data=0), pool(page=-1), pool(layers=-1), pool(slot=63), pool(slot=0), pool(layer=64 * 8 - 1), pool(layer=0)):
        assert call(bad) == IV
    assert call(pool(slot=64 * 3, layer=64)) == OK  # slots outside, layers inside
    assert call(pool(slot=64 * 3 - 1, layer=64)) == IV
    assert call(pool(layers=1, layer=0)) == OK and call(pool(slot=0, layer=64), slots=1) == OK
    assert call(k=0) == IV and call(k=9) == IV and call(slots=-1) == IV
    assert call(slots=(1 << 20) + 1, p=pool(layers=1)) == UN
    assert call(pool(page=1 << 46, slot=1 << 46, layers=1)) == UN  # 2^32 units of 16 KB
    assert lib.ssm_cache_free(None, 1, 8, P, P, 0, 0, None) == IV


def test_list_and_workspace_refusals(lib):
    p, big = pool(), 1 << 16
    copy = lambda src=P, dst=P, n=4, ws=P, b=big: lib.ssm_cache_copy(p, 1, 8, src, dst, n, ws, b, None)  # noqa: E731
    assert copy(n=0, src=None, ws=None) == OK
    assert copy(src=None) == IV and copy(dst=None) == IV and copy(n=-1) == IV and copy(src=P + 2) == IV
    assert copy(ws=None) == WS and copy(ws=P + 64) == WS and copy(b=256) == WS
    fork = lambda used=P, par=2 * P, ch=3 * P, n=4, ws=P, b=big: lib.ssm_cache_fork(p, 1, 8, used, par, ch, n, ws, b, None)  # noqa: E731
    assert fork(n=0) == OK
    assert fork(used=None) == IV and fork(par=None) == IV and fork(ch=None) == IV and fork(n=-1) == IV and fork(ch=3 * P + 1) == IV
    assert fork(ch=2 * P) == IV and fork(ch=2 * P + 12) == IV and fork(par=3 * P + 12) == IV
    assert fork(ws=None) == WS and fork(b=256) == WS
    free = lambda used=P, lst=2 * P, n=4: lib.ssm_cache_free(p, 1, 8, used, lst, n, 0, None)  # noqa: E731
    assert free(used=None) == IV and free(lst=None) == IV and free(n=-1) == IV and free(lst=P + 1) == IV
    compact = lambda used=P, t=2 * P, nt=4, ws=P, b=big: lib.ssm_cache_compact(p, 1, 8, used, t, nt, None, None, ws, b, None)  # noqa: E731
    assert compact(used=None) == IV and compact(nt=-1) == IV and compact(t=P + 1) == IV
    assert compact(ws=None) == WS and compact(b=256) == WS


def test_workspace_size(lib):
    f = ssm.ssm_cache_workspace_size
    assert f(8, 4) % 256 == 0 and f(8, 4) >= 256 + 3 * 8 * 4 and f(8, 1000) >= 256 + 3 * 4000
    assert f(-1, 4) == 0 and f(4, -1) == 0 and f((1 << 20) + 1, 4) == 0


def test_packed_pool_has_the_headers_layout(tmp_path):
    import os
    import subprocess
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "ssm_cache.h"\nint main(void) { printf("%zu %zu\\n",'
                   "sizeof(ssm_cache_pool_t), offsetof(ssm_cache_pool_t, layers)); return 0; }\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.check_call(["gcc", "-I", os.path.join(root, "include"), "-o", str(tmp_path / "s"), str(src)])
    assert [int(v) for v in subprocess.check_output([str(tmp_path / "s")]).split()] == [cache._POOL.size, 32]
    assert cache.SSM_CACHE_NEW == -1


def test_pools_refuse_what_they_can_see():
    with pytest.raises(ValueError, match="CUDA"):
        ssm.CachePools([torch.zeros(2, 3, 4)])
    with pytest.raises(ValueError, match="pools"):
        ssm.CachePools([])
