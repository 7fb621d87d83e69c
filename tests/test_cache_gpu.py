"""The state cache's page operations on the GPU against the same steps taken one by one (-m gpu)."""
import pytest
import torch

import selective_state_space_16_b200 as ssm
import workloads
from selective_state_space_16_b200 import binding

pytestmark = pytest.mark.gpu
i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731


def make(layers=3, slots=12, shapes=((40, 16), (40, 3)), dtypes=(torch.float32, torch.bfloat16), seed=0):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(layers, slots, *s, generator=g).to(d).cuda() for s, d in zip(shapes, dtypes)]


def copied(pools, pairs):
    """The pools after the copies, one after another."""
    out = [p.clone() for p in pools]
    n = pools[0].shape[1]
    for s, d in pairs:
        if 0 <= s < n and 0 <= d < n:
            for p in out:
                p[:, d] = p[:, s].clone()
    return out


def same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


PAIRS = [
    [(0, 5)], [(0, 5), (0, 6), (3, 1)], [(4, 4), (2, 7)], [(-1, 3), (2, 12), (2, 99), (-7, -7), (1, 0)],
    [(0, 1), (1, 2), (2, 3)],             # a chain: each pair reads what the one before wrote
    [(2, 3), (1, 2), (0, 1)],             # a shift: each page is read before it is written
    [(0, 11), (1, 0), (11, 1)],           # a swap through a third page
    [(0, 5), (1, 5), (2, 5)],             # the later copy stays
    [(3, 8), (8, 3), (3, 8)], [],
]


@pytest.mark.parametrize("pairs", PAIRS)
def test_copy(cuda_device, pairs):
    pools = make()
    want = copied(pools, pairs)
    h = ssm.CachePools(pools)
    ws = ssm.new_cache_workspace(h, max(1, len(pairs)))
    ssm.ssm_cache_copy(h, i32(*[p[0] for p in pairs]), i32(*[p[1] for p in pairs]), ws)
    assert same(pools, want)


def test_copy_many_pairs(cuda_device):
    g = torch.Generator().manual_seed(3)
    pools = make(layers=2, slots=4000, shapes=((5, 3),), dtypes=(torch.float32,))
    for clash in (False, True):
        perm = torch.randperm(4000, generator=g)
        src = perm[:1900] if not clash else torch.randint(4000, (1900,), generator=g)
        dst = perm[2000:3900] if not clash else torch.randint(4000, (1900,), generator=g)
        want = copied(pools, list(zip(src.tolist(), dst.tolist())))
        h = ssm.CachePools(pools)
        ssm.ssm_cache_copy(h, i32(*src.tolist()), i32(*dst.tolist()), ssm.new_cache_workspace(h, 1900))
        assert same(pools, want)


@pytest.mark.parametrize("page", [1, 2, 3, 7, 8, 12, 16, 24, 1000, 4096, 16384, 16385, 16386, 16388, 16392, 16400, 70001])
def test_page_sizes(cuda_device, page):
    """Pages of any number of bytes, dense pools: every slot starts at its own alignment."""
    pool = torch.randint(0, 256, (2, 7, page), dtype=torch.uint8, device="cuda")
    want = copied([pool], [(0, 6), (5, 1)])
    h = ssm.CachePools([pool])
    ssm.ssm_cache_copy(h, i32(0, 5), i32(6, 1), ssm.new_cache_workspace(h, 2))
    assert same([pool], want)
    used = torch.ones(7, dtype=torch.int32, device="cuda")
    ssm.ssm_cache_free(h, used, i32(3, 6, 3, -1, 9), zero_pages=True)
    want[0][:, 3] = want[0][:, 6] = 0
    assert same([pool], want) and used.tolist() == [1, 1, 1, 0, 1, 1, 0]


@pytest.mark.parametrize("by", [0, 1, 3, 8])
def test_strided_pools(cuda_device, by):
    """Slots of a wider tensor, layers inside slots, a base off the 16-byte grid; what lies between stays."""
    wide = torch.randn(2, 9, 70, device="cuda")
    inside = torch.randn(9, 5, 33, device="cuda").transpose(0, 1)  # (layers, slots): layers inside slots
    raw = torch.randint(0, 256, (4 * 9 * 50 + 16,), dtype=torch.uint8, device="cuda")
    odd = raw[by:by + 4 * 9 * 50].view(4, 9, 50)
    pools = [wide[:, :, by:by + 40], inside, odd]
    want, keep, keep_raw = copied(pools, [(8, 0), (2, 3)]), wide.clone(), raw.clone()
    h = ssm.CachePools(pools)
    ssm.ssm_cache_copy(h, i32(8, 2), i32(0, 3), ssm.new_cache_workspace(h, 2))
    assert same([p.contiguous() for p in pools], want)
    assert torch.equal(wide[:, :, :by], keep[:, :, :by]) and torch.equal(wide[:, :, by + 40:], keep[:, :, by + 40:])
    assert torch.equal(raw[:by], keep_raw[:by]) and torch.equal(raw[by + 1800:], keep_raw[by + 1800:])


def forked(pools, used, parents):
    out, used, kids = [p.clone() for p in pools], list(used), []
    before = list(used)
    n = len(used)
    for p in parents:
        ok = p == -1 or (0 <= p < n and before[p] != 0)
        kid = next((s for s in range(n) if used[s] == 0), -1) if ok else -1
        kids.append(kid)
        if kid >= 0:
            used[kid] = 1
            for t in out:
                t[:, kid] = 0 if p == -1 else t[:, p].clone()
    return out, used, kids


@pytest.mark.parametrize("used,parents", [
    ([1, 0, 1, 0, 0, 7, 0, 0, 1, 0, 0, 0], [2, 2, 5, -1, 0]),
    ([1, 0, 1, 0, 0, 1, 0, 0, 1, 0, 0, 0], [1, 3, 0, -2, 12, 400, -1]),  # free, outside: no child, no slot taken
    ([1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 0, 0], [4, -1, 6, 7]),               # two slots left for four
    ([1] * 12, [0, -1]), ([0] * 12, [-1] * 14), ([1, 0] * 6, []),
])
def test_fork(cuda_device, used, parents):
    pools = make(seed=1)
    pools[0][:, 2] = float("nan")
    want, used1, kids = forked(pools, used, parents)
    h = ssm.CachePools(pools)
    du, dc = i32(*used), torch.full((len(parents),), 77, dtype=torch.int32, device="cuda")
    ssm.ssm_cache_fork(h, du, i32(*parents), dc, ssm.new_cache_workspace(h, max(1, len(parents))))
    assert same(pools, want) and dc.tolist() == kids
    assert [bool(u) for u in du.tolist()] == [bool(u) for u in used1]


def test_fork_many(cuda_device):
    g = torch.Generator().manual_seed(4)
    pools = make(layers=1, slots=5000, shapes=((3,),), dtypes=(torch.float32,))
    used = (torch.rand(5000, generator=g) < 0.6).to(torch.int32)
    parents = torch.randint(-3, 5010, (2600,), generator=g, dtype=torch.int32)
    want, used1, kids = forked(pools, used.tolist(), parents.tolist())
    h = ssm.CachePools(pools)
    du, dc = used.cuda(), torch.empty(2600, dtype=torch.int32, device="cuda")
    ssm.ssm_cache_fork(h, du, parents.cuda(), dc, ssm.new_cache_workspace(h, 2600))
    assert same(pools, want) and dc.tolist() == kids and du.tolist() == used1


def compacted(pools, used, table):
    out, n = [p.clone() for p in pools], len(used)
    live = sum(1 for u in used if u)
    holes = [s for s in range(live) if not used[s]]
    movers = [s for s in range(live, n) if used[s]]
    remap = [s if used[s] else -1 for s in range(n)]
    for s, d in zip(movers, holes):
        remap[s] = d
        for t in out:
            t[:, d] = t[:, s].clone()
    return out, [1] * live + [0] * (n - live), [remap[t] if 0 <= t < n else -1 for t in table], remap, live


@pytest.mark.parametrize("used", [[1, 0, 1, 0, 0, 1, 0, 0, 1, 0, 1, 1], [0] * 12, [1] * 12, [0] * 11 + [3], [1] * 5 + [0] * 7,
                                  [0] * 6 + [1] * 6, [5, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 9]])
def test_compact(cuda_device, used):
    pools = make(seed=2)
    table = [11, 0, 2, -1, 5, 12, 8, 10, 11]
    want, used1, table1, remap1, live = compacted(pools, used, table)
    h = ssm.CachePools(pools)
    du, dt, dr, dc = i32(*used), i32(*table), torch.empty(12, dtype=torch.int32, device="cuda"), i32(-5)
    ssm.ssm_cache_compact(h, du, dt, dr, dc, ssm.new_cache_workspace(h))
    assert same(pools, want) and du.tolist() == used1 and dt.tolist() == table1 and dr.tolist() == remap1 and dc.tolist() == [live]
    again = [p.clone() for p in pools]  # nothing is left to move
    ssm.ssm_cache_compact(h, du, None, None, None, ssm.new_cache_workspace(h))
    assert same(pools, again) and du.tolist() == used1


def test_compact_many(cuda_device):
    g = torch.Generator().manual_seed(5)
    pools = make(layers=2, slots=7003, shapes=((4,),), dtypes=(torch.bfloat16,))
    used = (torch.rand(7003, generator=g) < 0.4).to(torch.int32)
    table = torch.randint(-2, 7005, (9000,), generator=g, dtype=torch.int32)
    want, used1, table1, remap1, live = compacted(pools, used.tolist(), table.tolist())
    h = ssm.CachePools(pools)
    du, dt = used.cuda(), table.cuda()
    ssm.ssm_cache_compact(h, du, dt, None, None, ssm.new_cache_workspace(h))
    assert same(pools, want) and du.tolist() == used1 and dt.tolist() == table1


def test_empty(cuda_device):
    """No slots, no layers, empty pages, empty lists."""
    none = ssm.CachePools([torch.empty(3, 0, 5, device="cuda")])
    used, kids, count = torch.empty(0, dtype=torch.int32, device="cuda"), i32(7, 7), i32(7)
    ws = ssm.new_cache_workspace(none, 2)
    ssm.ssm_cache_fork(none, used, i32(-1, 0), kids, ws)
    table = i32(0, 3)
    ssm.ssm_cache_compact(none, used, table, None, count, ws)
    ssm.ssm_cache_copy(none, i32(0), i32(1), ws)
    ssm.ssm_cache_free(none, used, i32(0, 2), zero_pages=True)
    assert kids.tolist() == [-1, -1] and count.tolist() == [0] and table.tolist() == [-1, -1]
    thin = [torch.empty(0, 6, 4, device="cuda"), torch.empty(2, 6, 0, device="cuda")]  # only the bookkeeping is left
    h = ssm.CachePools(thin)
    used, kids = i32(1, 0, 0, 1, 0, 1), i32(7, 7)
    ws = ssm.new_cache_workspace(h, 2)
    ssm.ssm_cache_fork(h, used, i32(3, -1), kids, ws)
    ssm.ssm_cache_free(h, used, i32(0))
    ssm.ssm_cache_compact(h, used, kids, None, None, ws)
    assert used.tolist() == [1, 1, 1, 1, 0, 0] and kids.tolist() == [1, 2]


@pytest.mark.parametrize("slots", [2048, 2049])
def test_calls_on_either_side_of_the_small_ones(cuda_device, slots):
    """The largest pool of a small call and the next one: every operation, on pages of odd sizes and strides."""
    g = torch.Generator().manual_seed(slots)
    wide = torch.randn(2, slots, 9, generator=g).cuda()
    pools = [wide[:, :, 2:7], torch.randint(0, 256, (1, slots, 3), generator=g, dtype=torch.uint8).cuda(),
             torch.randn(slots, 3, 4, generator=g).bfloat16().cuda().transpose(0, 1)]
    keep = wide.clone()
    h = ssm.CachePools(pools)
    ws = ssm.new_cache_workspace(h, 40)
    dense = lambda: [p.contiguous() for p in pools]  # noqa: E731
    for pairs in ([(0, slots - 1), (slots - 2, 7), (5, 9)], [(0, 1), (1, slots - 1), (slots - 1, 2), (3, 2)]):
        want = copied(dense(), pairs)
        ssm.ssm_cache_copy(h, i32(*[p[0] for p in pairs]), i32(*[p[1] for p in pairs]), ws)
        assert same(dense(), want)
    used = (torch.rand(slots, generator=g) < 0.99).to(torch.int32)
    parents = torch.randint(-1, slots, (30,), generator=g, dtype=torch.int32)
    want, used1, kids = forked(dense(), used.tolist(), parents.tolist())
    du, dc = used.cuda(), torch.empty(30, dtype=torch.int32, device="cuda")
    ssm.ssm_cache_fork(h, du, parents.cuda(), dc, ws)
    assert same(dense(), want) and dc.tolist() == kids and du.tolist() == used1
    ended = torch.randperm(slots, generator=g)[:25].to(torch.int32)
    ssm.ssm_cache_free(h, du, ended.cuda())
    assert du.sum() == sum(used1) - sum(used1[e] for e in ended.tolist())
    want, used2, table, remap, live = compacted(dense(), du.tolist(), list(range(slots)))
    dt, dr, n = torch.arange(slots, dtype=torch.int32, device="cuda"), torch.empty(slots, dtype=torch.int32, device="cuda"), i32(0)
    ssm.ssm_cache_compact(h, du, dt, dr, n, ws)
    assert same(dense(), want) and du.tolist() == used2 and dt.tolist() == table and dr.tolist() == remap and n.tolist() == [live]
    assert torch.equal(wide[:, :, :2], keep[:, :, :2]) and torch.equal(wide[:, :, 7:], keep[:, :, 7:])


def test_far_offsets(cuda_device):
    """A pool of more than 2^32 bytes: slots and layers beyond 32-bit offsets."""
    pool = torch.empty(2, 3, (1 << 30) + 16, dtype=torch.uint8, device="cuda")
    pool[1, 2, -100:] = 9
    pool[1, 2, :100] = 8
    pool[1, 0, :100], pool[1, 0, -100:] = 1, 1
    h = ssm.CachePools([pool])
    ssm.ssm_cache_copy(h, i32(2), i32(0), ssm.new_cache_workspace(h, 1))
    assert bool((pool[1, 0, -100:] == 9).all()) and bool((pool[1, 0, :100] == 8).all())
    del pool, h
    torch.cuda.empty_cache()


def test_captured_and_replayed(cuda_device):
    """Admission, retirement and compaction in one graph; the lists are read at replay."""
    pools = make(seed=6)
    h = ssm.CachePools(pools)
    used, parents, kids = i32(*[1, 1, 0, 0, 1, 0, 0, 0, 1, 0, 0, 0]), i32(0, -1), i32(0, 0)
    ended, table, count = i32(1), i32(0, 8, 4), i32(0)
    ws = ssm.new_cache_workspace(h, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ssm.ssm_cache_fork(h, used, parents, kids, ws)
        ssm.ssm_cache_free(h, used, ended)
        ssm.ssm_cache_compact(h, used, table, None, count, ws)
    state, u, t = [p.clone() for p in pools], used.tolist(), table.tolist()
    for par, end in (([0, -1], [1]), ([4, 8], [0]), ([-1, 5], [2])):
        parents.copy_(i32(*par))
        ended.copy_(i32(*end))
        graph.replay()
        state, u, k = forked(state, u, par)
        u[end[0]] = 0
        state, u, t, _, live = compacted(state, u, t)
        torch.cuda.synchronize()
        assert same(pools, state) and used.tolist() == u and kids.tolist() == k and table.tolist() == t and count.tolist() == [live]


def test_decode_over_the_cache(cuda_device):
    """Sequences are admitted, forked, decoded, retired and compacted; those that remain decode on, from the
    front of the pool, as if they had been alone: the selective scan's states and the gated recurrence's."""
    D, slots, steps = 24, 10, 6
    dec = workloads.decode_inputs(slots, D, seed=3, io="f32", pool=steps)
    A, Dp, bias = dec["A"].cuda(), dec["D"].cuda(), dec["delta_bias"].cuda()
    lam = torch.linspace(-6, 0, D, device="cuda")
    token = [{k: v.cuda() for k, v in s.items()} for s in dec["sets"]]

    def step(scan, gated, k, rows):
        """Row j of the batch is sequence rows[j]; the states are the first slots."""
        n = len(rows)
        a = {key: v[rows].contiguous() for key, v in token[k].items()}
        y = [torch.empty(n, D, device="cuda") for _ in range(2)]
        ssm.ssm_state_update(scan[:n], a["u"], a["delta"], A, a["B"], a["C"], Dp, a["z"], bias, True, y[0])
        ssm.ssm_gated_state_update(gated[:n], a["u"], a["delta"], a["z"], lam, None, None, None, y[1])
        return y

    # each sequence alone: 0, 1, 2 new; 3 and 4 forks of 1 after two steps; 0 and 3 end after four
    def alone(seq, fork_of=None):
        scan, gated = torch.zeros(1, D, 16, device="cuda"), torch.zeros(1, D, device="cuda")
        for k in range(steps):
            y = step(scan, gated, k, [fork_of if fork_of is not None and k < 2 else seq])
        return torch.cat([y[0], y[1]])

    pools = [torch.randn(1, slots, D, 16, device="cuda"), torch.randn(1, slots, D, device="cuda")]
    h, used = ssm.CachePools(pools), torch.zeros(slots, dtype=torch.int32, device="cuda")
    ws = ssm.new_cache_workspace(h, 4)
    table = i32(-1, -1, -1)
    ssm.ssm_cache_fork(h, used, i32(-1, -1, -1), table, ws)
    assert table.tolist() == [0, 1, 2]
    rows = [0, 1, 2]
    for k in range(steps):
        if k == 2:
            kids = i32(0, 0)
            ssm.ssm_cache_fork(h, used, table[[1, 1]], kids, ws)
            table, rows = torch.cat([table, kids]), [0, 1, 2, 3, 4]
        if k == 4:
            ssm.ssm_cache_free(h, used, table[[0, 3]], zero_pages=True)
            count = i32(0)
            ssm.ssm_cache_compact(h, used, table, None, count, ws)
            assert count.tolist() == [3] and table.tolist() == [-1, 1, 2, -1, 0]
            rows = [4, 1, 2]  # in the order of their slots
        y = step(pools[0][0], pools[1][0], k, rows)
    for j, (seq, fork_of) in enumerate(((4, 1), (1, None), (2, None))):
        assert torch.equal(torch.cat([y[0][j:j + 1], y[1][j:j + 1]]), alone(seq, fork_of))


def test_refusals(cuda_device):
    pools = make()
    h = ssm.CachePools(pools)
    ws = ssm.new_cache_workspace(h, 4)
    used, lst = torch.ones(12, dtype=torch.int32, device="cuda"), i32(1, 2)
    for call in (lambda: ssm.ssm_cache_copy(h, lst, i32(3), ws), lambda: ssm.ssm_cache_fork(h, used[:5], lst, i32(0, 0), ws),
                 lambda: ssm.ssm_cache_fork(h, used, lst, i32(0), ws), lambda: ssm.ssm_cache_free(h, used, lst.cpu()),
                 lambda: ssm.ssm_cache_free(h, used, i32(0, 1, 2, 3)[::2]), lambda: ssm.ssm_cache_compact(h, used, lst, used[:3], None, ws),
                 lambda: ssm.CachePools([pools[0], pools[1][:, :5]]), lambda: ssm.CachePools([pools[0].transpose(2, 3)])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        ssm.ssm_cache_free(h, used, lst.long())
    with pytest.raises(binding.SsmError):
        ssm.ssm_cache_fork(h, used, lst, lst, ws)
    with pytest.raises(binding.SsmError):
        ssm.ssm_cache_compact(h, used, None, None, None, ws[:256])
    assert ssm.ssm_cache_copy(h, lst, lst, ws[:256], check=False) == binding.SSM_ERR_WORKSPACE
    overlapping = torch.zeros(200, device="cuda").as_strided((2, 12, 10), (0, 10, 1))
    assert ssm.ssm_cache_copy(ssm.CachePools([overlapping]), lst, lst, ws, check=False) == binding.SSM_ERR_INVALID_ARG
