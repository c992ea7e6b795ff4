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
