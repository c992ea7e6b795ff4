"""Pages of the 4-bit cache that a broken table, a full stack or a short slot map would lose or hand out twice."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import dynamic_sparse_attention_head_b200 as msa  # noqa: E402

I32, BOUNDS = torch.int32, 8


def _ints(x, dtype=I32):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


@pytest.mark.parametrize("entry", [-1, 12, 1 << 30])
def test_release_drops_a_table_entry_that_names_no_page(entry):
    cache = msa.KV4Cache.alloc(12, 1, 16, 64)
    table = _ints([[3, entry, 4], [5, -1, -1], [6, 7, -1]])
    kv, free, nf = _ints([40, 16, 20]), _ints([0, 1] + [-9] * 10), _ints([2])
    cache.release(_ints([2, 0, 2]), kv, table, free, nf)
    assert cache.device_status() == BOUNDS and cache.device_status() == 0
    assert nf.tolist() == [6] and free[:6].tolist() == [0, 1, 6, 7, 3, 4]
    assert kv.tolist() == [0, 16, 0] and table.tolist() == [[-1, -1, -1], [5, -1, -1], [-1, -1, -1]]
    # what is handed out next are pages
    sl, pos, cu = _ints([0] * 96, torch.int64), _ints([0] * 96), _ints([0] * 4)
    cache.slots(kv, _ints([48, 0, 48]), table, free, nf, sl, pos, cu)
    assert cache.device_status() == 0 and nf.tolist() == [0] and kv.tolist() == [48, 16, 48]
    assert sorted(table[[0, 2]].flatten().tolist()) == [0, 1, 3, 4, 6, 7]
    assert sl.tolist() == [int(table[b, j // 16]) * 16 + j % 16 for b in (0, 2) for j in range(48)]


def test_release_leaves_requests_that_the_stack_has_no_room_for():
    cache = msa.KV4Cache.alloc(6, 1, 16, 64)
    table = _ints([[0, 1, -1], [2, 3, 4], [5, -1, -1], [1, -1, -1]])
    kv, free, nf = _ints([32, 33, 16, 5]), _ints([1, -9, -9, -9, -9, -9]), _ints([1])
    before = table.clone()
    cache.release(_ints([0, 1, 2, 3]), kv, table, free, nf)  # room for five of the seven named: the first two
    assert cache.device_status() == BOUNDS
    assert nf.tolist() == [6] and free.tolist() == [1, 0, 1, 2, 3, 4]
    assert kv.tolist() == [0, 0, 16, 5] and torch.equal(table[2:], before[2:]) and (table[:2] == -1).all()
    # a broken entry takes no room: both requests fit
    table, kv, free, nf = _ints([[0, -1, 1], [2, -1, -1]]), _ints([48, 7]), _ints([-9] * 6), _ints([3])
    cache.release(_ints([0, 1]), kv, table, free, nf)
    assert cache.device_status() == BOUNDS and nf.tolist() == [6] and free.tolist() == [-9] * 3 + [0, 1, 2] and kv.tolist() == [0, 0]


def test_release_of_many_pages_with_and_without_broken_entries():
    """Requests of more entries than the block has threads, in the order of the list."""
    rng = np.random.default_rng(5)
    B, blocks, page = 40, 90, 16
    n_pages = B * blocks
    lens = rng.integers(0, blocks * page + 1, B)
    lens[3], lens[4] = 0, blocks * page
    for share in (0.0, 0.05, 1.0):
        table = rng.permutation(n_pages).reshape(B, blocks)
        table[rng.random(table.shape) < share] = n_pages + 5
        ids = np.concatenate((rng.permutation(B)[:30], [4, 4, 17]))
        cache = msa.KV4Cache.alloc(n_pages, 1, page, 128)
        t, kv, free, nf = _ints(table), _ints(lens), _ints([-9] * n_pages), _ints([0])
        cache.release(_ints(ids), kv, t, free, nf)
        want, seen = [], []
        for i in ids:
            if i not in seen:
                seen.append(i)
                want += [int(p) for p in table[i, :-(-lens[i] // page)] if p < n_pages]
        named = {i for i in seen}
        assert cache.device_status() == (BOUNDS if share and len(want) < sum(-(-lens[i] // page) for i in seen) else 0)
        assert int(nf) == len(want) and free[:len(want)].tolist() == want
        assert kv.tolist() == [0 if b in named else int(lens[b]) for b in range(B)]
        left = table.copy()
        for b in named:
            left[b, :-(-lens[b] // page)] = -1
        assert t.tolist() == left.tolist()


@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("kv,new,cap,kept", [
    ([0, 4, 5], [20, 30, 2], 25, 1),          # the second passes the map's end
    ([0, 4, 5], [20, 30, 2], 50, 2),          # the third is behind it
    ([0, 4, 5], [20, 30, 2], 52, 3),          # all just fit
    ([7, 0], [3, 1], 0, 0),
    ([7, 0, 9], [0, 0, 4], 0, 2),             # requests without tokens need no entry
    ([15] * 300, [3] * 300, 620, 206),
    ([0, 17, 0, 400], [30000, 1, 0, 20011], 30001, 3),  # over several blocks
])
def test_whole_requests_are_refused_where_the_map_ends(kv, new, cap, kept, alias):
    page, B = 16, len(kv)
    blocks = max(-(-(k + n) // page) for k, n in zip(kv, new))
    held = [-(-k // page) for k in kv]
    n_pages = sum(held) + sum(-(-n // page) + 1 for n in new)
    cache = msa.KV4Cache.alloc(n_pages, 1, page, 128, whole_requests=True)
    table, at = np.full((B, blocks), -1), 0
    for b, h in enumerate(held):
        table[b, :h] = np.arange(at, at + h)
        at += h
    t, free, nf = _ints(table), _ints(list(range(at, n_pages)) + [0] * at), _ints([n_pages - at])
    k, n = _ints(kv), _ints(new)
    ko, nfo = (k, nf) if alias else (torch.zeros_like(k), torch.zeros_like(nf))
    sl, pos, cu = _ints([-77] * cap, torch.int64), _ints([-77] * cap), _ints([0] * (B + 1))
    cache.slots(k, n, t, free, nf, sl, pos, cu, kv_lens_out=None if alias else ko, n_free_out=None if alias else nfo)
    assert cache.device_status() == (BOUNDS if kept < B else 0)
    assert ko.tolist() == [a + m if b < kept else a for b, (a, m) in enumerate(zip(kv, new))]
    assert cu.tolist() == np.concatenate(([0], np.cumsum(new))).tolist()
    taken = sum(-(-(a + m) // page) - -(-a // page) for a, m in list(zip(kv, new))[:kept])
    assert nfo.tolist() == [n_pages - at - taken]
    t = t.cpu().numpy()
    assert (t[kept:] == table[kept:]).all()
    want = [int(t[b, p // page]) * page + p % page if b < kept else -1 for b in range(B) for p in range(kv[b], kv[b] + new[b])]
    assert sl.tolist() == (want + [-77] * cap)[:cap]
    assert pos.tolist() == ([p for b in range(B) for p in range(kv[b], kv[b] + new[b])] + [-77] * cap)[:cap]
    assert len(set(want[:int(cu[kept])])) == int(cu[kept])


def test_a_captured_step_reads_no_other_requests_rows_where_the_map_is_too_short():
    """Slot map, write and attention of a step in one graph, two new tokens where the map has room for one: the pages of the
    second request, released by one whose values were 100, are not read."""
    page, group = 16, 64
    cache = msa.KV4Cache.alloc(4, 1, page, group, whole_requests=True)
    x = torch.full((1, 32, 128), 100.0, dtype=torch.bfloat16, device="cuda")
    table, kv = _ints([[0], [1]]), _ints([16, 16])
    cache.append(x, x, torch.arange(32, device="cuda"))
    free, nf = _ints([2, 3, -1, -1]), _ints([0])
    cache.release(_ints([0, 1]), kv, table, free, nf)
    x = torch.ones(1, 1, 128, dtype=torch.bfloat16, device="cuda")
    sl, pos, cu, one = _ints([0], torch.int64), _ints([0]), _ints([0, 0, 0]), _ints([1, 1])
    q, ws = torch.ones(1, 2, 128, dtype=torch.bfloat16, device="cuda"), cache.alloc_workspace()
    o = torch.full_like(q, 7.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.slots(kv, one, table, free, nf, sl, pos, cu)
        cache.append(x, x, sl)
        cache.attend(q, o, table, kv, cu, 1, 0.1, ws)
    graph.replay()
    assert kv.tolist() == [1, 0] and nf.tolist() == [1] and cache.device_status() == BOUNDS
    assert (o[0, 0] == 1).all() and (o[0, 1] == 0).all()
