"""The paged 4-bit cache on the GPU against its 64-bit forms (kv4_oracle): slot maps and release, the
write (whole pages, bit for bit), the read back, attention over it, and a run of them together."""
import numpy as np
import pytest

import kv4_oracle as ko

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import dynamic_sparse_attention_head_b200 as msa  # noqa: E402

I32 = torch.int32


def _dev(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16).cuda()


def _host(t):
    return t.float().cpu().numpy().astype(np.float64)


def _ints(x, dtype=I32):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


def _cache(n_pages, Hkv, page, group, fill=0xFF):
    c = msa.KV4Cache.alloc(n_pages, Hkv, page, group)
    c.pages.fill_(fill)  # 0xFF: every scale a NaN until it is written
    return c


# ---- slot maps -----------------------------------------------------------------------------------
def _slots(kv, new, page, blocks, n_pages, n_free, alias, cap=None, seed=0):
    rng = np.random.default_rng(seed)
    B = len(kv)
    cache = msa.KV4Cache(torch.zeros(n_pages, 1, page * 136, dtype=torch.uint8, device="cuda"), page=page, group=128)
    perm = rng.permutation(n_pages)
    table, at = np.full((B, blocks), -1, np.int64), 0
    for b, k in enumerate(kv):
        h = min(-(-max(k, 0) // page), blocks)
        table[b, :h] = perm[at:at + h]
        at += h
    assert at <= n_pages - n_free or n_free == 0
    free = np.concatenate((perm[n_pages - n_free:], np.zeros(n_pages - n_free, np.int64)))
    ref = ko.slots(kv, new, table, free, n_free, page, blocks)
    total = ref[3][-1]
    cap = total + 5 if cap is None else cap
    tab = torch.full((B, blocks + 3), -7, dtype=I32, device="cuda")
    tab[:, :blocks] = _ints(table)
    d = dict(kv=_ints(kv), new=_ints(new), free=_ints(free), nf=_ints([n_free]), cu=_ints([99] * (B + 1)),
             sl=_ints([-77] * cap, torch.int64), pos=_ints([-77] * cap))
    kvo, nfo = (d["kv"], d["nf"]) if alias else (torch.zeros_like(d["kv"]), torch.zeros_like(d["nf"]))
    cache.slots(d["kv"], d["new"], tab[:, :blocks], d["free"], d["nf"], d["sl"], d["pos"], d["cu"],
                kv_lens_out=None if alias else kvo, n_free_out=None if alias else nfo)
    st = cache.device_status()
    t, k, nf, cu, sl, pos, ok = ref
    n = min(cap, total)
    assert tab[:, :blocks].cpu().numpy().tolist() == t.tolist() and (tab[:, blocks:] == -7).all()
    assert kvo.tolist() == k and nfo.tolist() == [nf] and d["cu"].tolist() == cu
    assert d["sl"][:n].tolist() == sl[:n] and (d["sl"][n:] == -77).all()
    want = [p for p in pos[:n]]
    assert d["pos"][:n].tolist() == want and (d["pos"][n:] == -77).all()
    assert (st == 0) == (ok and total <= cap)
    assert cache.device_status() == 0  # read and cleared
    assert int(cache.state[4]) == 0


@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_slots_decode_batch(page, alias):
    rng = np.random.default_rng(page)
    kv = rng.integers(0, 5 * page, 700).tolist()
    kv[:4] = [0, page - 1, page, page + 1]
    need = sum(-(-k // page) for k in kv)
    _slots(kv, [1] * 700, page, 7, need + 800, 750, alias)


@pytest.mark.parametrize("B,cap", [(1, None), (511, None), (512, None), (513, None), (300, 40), (64, 0)])
@pytest.mark.parametrize("most", [1, 4, 5])
def test_slots_of_a_few_tokens_each(B, cap, most):
    rng = np.random.default_rng(B + most)
    kv, new = rng.integers(0, 70, B).tolist(), rng.integers(0, most + 1, B).tolist()
    new[-1] = most
    _slots(kv, new, 16, 6, 4 * 600 + 600, 590, True, cap=cap)
    _slots(kv, new, 16, 6, 4 * 600 + 600, 7, False, cap=cap)  # the free pages end somewhere in the batch


@pytest.mark.parametrize("alias", [False, True])
def test_slots_prompts_over_several_blocks(alias):
    _slots([0, 17, 0, 400], [30000, 1, 0, 20011], 16, 2000, 6000, 5000, alias)


def test_slots_empty_batch_and_empty_requests():
    _slots([5, 0], [0, 0], 16, 2, 8, 4, True)
    cache = msa.KV4Cache.alloc(4, 1, 16, 64)
    cu, nf = _ints([3]), _ints([4])
    cache.slots(_ints([]), _ints([]), torch.zeros(0, 2, dtype=I32, device="cuda"), _ints([0, 1, 2, 3]), nf,
                _ints([], torch.int64), _ints([]), cu)
    assert cu.tolist() == [0] and nf.tolist() == [4] and cache.device_status() == 0


def test_slots_most_requests():
    rng = np.random.default_rng(1)
    kv = rng.integers(0, 40, 2048).tolist()
    _slots(kv, rng.integers(0, 4, 2048).tolist(), 16, 4, 8000, 2048, True)


def test_slots_out_of_pages_and_rows():
    _slots([0, 0, 3, 0], [20, 40, 1, 0], 16, 4, 30, 4, False)   # the second does not fit the free pages: none after it
    _slots([0, 60, 0], [20, 10, 5], 16, 4, 30, 10, True)        # the second does not fit its row: the others do
    _slots([0, 5], [20, 1], 16, 4, 10, 0, True)                 # no page at all
    _slots([0, 4, 5], [20, -3, 2], 16, 4, 30, 10, False)        # a negative length counts as none
    _slots([0, 4, 5], [20, 30, 2], 16, 4, 30, 10, True, cap=25)  # the map is too short: the rest is left out


def test_slots_negative_lengths():
    _slots([5, -3, 7], [2, 4, -6], 16, 4, 30, 10, True)
    _slots([-1], [3], 16, 4, 30, 10, False)


def test_slots_refuses_broken_free_count_on_the_device():
    cache = msa.KV4Cache.alloc(4, 1, 16, 64)
    nf, kv = _ints([9]), _ints([0])
    sl, pos, cu = _ints([0], torch.int64), _ints([0]), _ints([0, 0])
    cache.slots(kv, _ints([1]), torch.full((1, 2), -1, dtype=I32, device="cuda"), _ints([0, 1, 2, 3]), nf, sl, pos, cu)
    assert cache.device_status() == 8
    assert sl.tolist() == [3 * 16] and nf.tolist() == [3]  # cut to the stack's room


def test_release_returns_pages_once():
    cache = msa.KV4Cache.alloc(12, 1, 16, 64)
    table = _ints([[3, 4, -1], [5, -1, -1], [6, 7, 8], [9, -1, -1]])
    kv, free, nf = _ints([20, 16, 33, 0]), _ints([0, 1] + [-1] * 10), _ints([2])
    cache.release(_ints([2, 0, 2, 3]), kv, table, free, nf)  # request 2 twice, request 3 empty
    assert cache.device_status() == 0
    assert nf.tolist() == [7] and free[:7].tolist() == [0, 1, 6, 7, 8, 3, 4]
    assert kv.tolist() == [0, 16, 0, 0]
    assert table.tolist() == [[-1, -1, -1], [5, -1, -1], [-1, -1, -1], [9, -1, -1]]
    cache.release(_ints([1, 4, -1]), kv, table, free, nf)  # two ids that there are not
    assert cache.device_status() == 8 and nf.tolist() == [8] and kv.tolist() == [0, 0, 0, 0]
    cache.release(_ints([]), kv, table, free, nf)
    assert nf.tolist() == [8]


def test_slots_and_release_in_turn_keep_every_page():
    """Continuous batching: pages in the table and on the stack are always all pages, each once."""
    rng = np.random.default_rng(4)
    page, B, n_pages = 16, 9, 60
    cache = msa.KV4Cache.alloc(n_pages, 1, page, 64)
    table, kv = torch.full((B, 6), -1, dtype=I32, device="cuda"), _ints([0] * B)
    free, nf = _ints(rng.permutation(n_pages)), _ints([n_pages])
    sl, pos, cu = _ints([0] * 500, torch.int64), _ints([0] * 500), _ints([0] * (B + 1))
    for step in range(25):
        lens = kv.cpu().numpy()
        new = np.minimum(rng.integers(0, 30, B), 96 - lens)
        cache.slots(kv, _ints(new), table, free, nf, sl, pos, cu)
        done = np.nonzero(rng.random(B) < 0.25)[0]
        cache.release(_ints(done), kv, table, free, nf)
        assert cache.device_status() == 0
        t, k = table.cpu().numpy(), kv.cpu().numpy()
        held = [p for b in range(B) for p in t[b, :-(-k[b] // page)]]
        assert sorted(held + free[:int(nf)].tolist()) == list(range(n_pages)), step


# ---- write and read ------------------------------------------------------------------------------
def _rows_of(rng, H, T):
    x = rng.standard_normal((2, H, T, 128)) * np.exp(rng.uniform(-3, 3, (2, H, T, 1)))
    x[0, :, :, 5] += 20.0
    return ko.bf16(x)


@pytest.mark.parametrize("page,group", [(16, 32), (16, 128), (32, 64), (64, 32), (128, 64), (256, 128)])
@pytest.mark.parametrize("T,H", [(1, 1), (37, 3), (300, 2)])
def test_append_writes_the_format_and_read_gives_its_values(page, group, T, H):
    rng = np.random.default_rng(page + group + T)
    n_pages = -(-T // page) + 3
    K, V = _rows_of(rng, H, T)
    slots = rng.permutation(n_pages * page)[:T]
    slots[T // 3] = -1 if T > 1 else slots[0]
    cache = _cache(n_pages, H, page, group, fill=0x5A)
    ref = cache.pages.cpu().numpy()
    k = _dev(K.transpose(1, 0, 2)).transpose(0, 1)  # [H, T, 128] as a view of [T, H, 128]
    v = torch.zeros(H, T + 2, 128, dtype=torch.bfloat16, device="cuda")[:, 1:T + 1]
    v.copy_(_dev(V))
    sl = _ints(slots, torch.int64)
    cache.append(k, v, sl)
    for t, s in enumerate(slots):
        for h in range(H):
            if s >= 0:
                ko.write(ref, page, group, s, h, K[h, t], V[h, t])
    got = cache.pages.cpu().numpy()
    assert (got == ref).all(), f"{int((got != ref).sum())} bytes differ"
    ok, ov = torch.full_like(k, 3.0), torch.full((T, H, 128), 3.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    cache.read(sl, ok, ov)
    assert cache.device_status() == 0
    for t, s in enumerate(slots):
        for h in range(H):
            for got_row, part in zip((ok[h, t], ov[h, t]), ko.parts(ref, page, group, s, h) if s >= 0 else (None, None)):
                if part is None:
                    assert (got_row == 3.0).all()
                    continue
                c, st, lo = part
                want = lo + c * st
                # one fp32 fused operation, then bf16
                assert (np.abs(_host(got_row) - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -23)).all()


def test_append_edges_flat_tiny_infinite_and_nan_groups():
    x = np.zeros((1, 8, 128))
    x[0, 1] = -3.5
    x[0, 2, 7] = np.inf
    x[0, 3, 100] = np.nan
    x[0, 4, 0], x[0, 4, 1] = 3e38, -3e38
    x[0, 5, 3] = 2.0 ** -130
    x[0, 6, :64] = 2.0 ** -120 * np.arange(64)
    x[0, 7] = np.linspace(-1, 1, 128)
    x = np.where(np.isnan(x), np.nan, ko.bf16(np.nan_to_num(x, nan=0.0, posinf=np.inf, neginf=-np.inf)))
    for group in (32, 64, 128):
        cache = _cache(1, 1, 16, group)
        d, sl = _dev(x), torch.arange(8, device="cuda")
        cache.append(d, d, sl)
        ref = np.full((1, 1, 16 * ko.row_bytes(group)), 0xFF, np.uint8)
        for t in range(8):
            ko.write(ref, 16, group, t, 0, x[0, t], x[0, t])
        assert (cache.pages.cpu().numpy() == ref).all()
        k, v = torch.empty_like(d), torch.empty_like(d)
        cache.read(sl, k, v)
        bad = np.isnan(_host(k))
        want = (~np.isfinite(x)).reshape(1, 8, -1, group).any(-1)
        want[0, 4, 0] = True  # its range overflows fp32
        assert (bad == np.repeat(want, group, -1)).all()
        assert torch.equal(k[:, 5:6], torch.zeros_like(k[:, 5:6])) and torch.equal(k[:, 1], d[:, 1])


def test_append_and_read_skip_slots_behind_the_cache():
    cache = _cache(2, 1, 16, 64, fill=0)
    x = _dev(np.ones((1, 4, 128)))
    sl = _ints([5, 32, -4, 1 << 40], torch.int64)
    cache.append(x, x, sl)
    assert cache.device_status() == 8 and cache.device_status() == 0
    k, v = torch.full_like(x, 4.0), torch.full_like(x, 4.0)
    cache.read(sl, k, v)
    assert cache.device_status() == 8
    assert (k[0, 0] == 1).all() and (v[0, 0] == 1).all() and (k[0, 1:] == 4).all() and (v[0, 1:] == 4).all()


# ---- attention -----------------------------------------------------------------------------------
def _filled(rng, kv_lens, Hkv, page, group, extra_blocks=2, scale_v=1.0):
    """A cache whose requests' tokens are written by the library; everything else is 0xFF (NaN)."""
    need = [-(-k // page) for k in kv_lens]
    n_pages = sum(need) + 2
    cache = _cache(n_pages, Hkv, page, group)
    perm = rng.permutation(n_pages)
    table = np.full((len(kv_lens), max(need, default=0) + extra_blocks), -1, np.int64)
    at = 0
    for b, k in enumerate(kv_lens):
        table[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
        if k:
            K, V = _rows_of(rng, Hkv, k)
            sl = [table[b, j // page] * page + j % page for j in range(k)]
            cache.append(_dev(K), _dev(V * scale_v), _ints(sl, torch.int64))
    table[:, -1] = 1 << 30  # entries that no length reaches
    return cache, table


def _attend(cache, Q, table, kv_lens, cu, scale, max_q=None, ws=None, pad=0, lse=True):
    Hq, T = Q.shape[0], Q.shape[1]
    q = torch.empty(T + pad, Hq, 128, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    q[:, :T] = _dev(Q)
    q[:, T:] = float("nan")
    o = torch.full((Hq, T + pad + 3, 128), 5.0, dtype=torch.bfloat16, device="cuda")[:, 2:T + pad + 2]
    L = torch.full((Hq, T + pad), 5.0, device="cuda") if lse else None
    n = [b - a for a, b in zip(cu, cu[1:])]
    cache.attend(q, o, _ints(table), _ints(kv_lens), _ints(cu), max(n, default=0) if max_q is None else max_q, scale,
                 cache.alloc_workspace() if ws is None else ws, lse=L)
    return o, L


def _compare(o, L, ref):
    O, lse, tO, tL = ref
    T = O.shape[1]
    got, gl = _host(o)[:, :T], L.cpu().numpy().astype(np.float64)[:, :T]
    rows = ~np.isnan(lse)
    assert np.isfinite(got).all()
    ratio = np.abs(got - O)[rows] / np.maximum(tO[rows], 1e-300)
    assert (np.abs(got - O)[rows] <= tO[rows]).all(), f"O: {ratio.max():.2f} of the bound"
    empty = np.isneginf(lse)
    assert (np.isneginf(gl) == empty).all()
    fin = rows & ~empty
    assert (np.abs(gl[fin] - lse[fin]) <= tL[fin]).all(), "lse"
    assert (got[~rows] == 5.0).all() and (gl[~rows] == 5.0).all()  # rows of no request
    assert (_host(o)[:, T:] == 5.0).all() and (L[:, T:] == 5.0).all()


SHAPES = [  # Hq, Hkv, page, group, kv lens, new tokens
    (4, 4, 16, 32, [1], [1]),
    (7, 1, 16, 64, [15, 16, 17, 0, 31, 32, 33], [1, 1, 1, 1, 1, 1, 1]),
    (8, 2, 64, 128, [63, 64, 65, 1, 128, 200], [1] * 6),
    (28, 4, 64, 64, [300, 5], [1, 1]),
    (8, 1, 128, 32, [700], [1]),
    (16, 1, 32, 64, [100, 40], [1, 1]),              # 16 rows a token
    (12, 1, 256, 128, [300], [1]),
    (40, 1, 16, 64, [50], [1]),                      # three row tiles a token
    (4, 2, 64, 64, [90, 7, 33, 1], [3, 7, 0, 1]),    # drafts; a prompt from its start; a request without tokens
    (7, 1, 64, 32, [120, 64], [5, 64]),              # tiles that end inside a token's heads
    (6, 2, 16, 128, [70, 3], [40, 6]),               # more new tokens than cached ones: rows without keys
    (2, 1, 32, 64, [260], [131]),
    (7, 1, 64, 64, [300, 70, 0, 33], [37, 70, 0, 9]),  # the kernel for many rows from here on: pairs of 256 rows
    (4, 2, 16, 32, [150, 200], [150, 64]),             # a prompt from its start
    (8, 1, 32, 128, [129, 128, 127, 1], [100, 1, 33, 1]),
    (3, 1, 256, 64, [300], [290]),
    (28, 4, 128, 32, [140], [19]),                     # three pairs, the last one of 20 rows
    (16, 2, 64, 128, [5, 400], [40, 20]),              # more new tokens than cached ones
]

MANY = 1 << 20  # a hint that takes the kernel for many rows; 1: never does


@pytest.mark.parametrize("max_q", [1, None, MANY])
@pytest.mark.parametrize("Hq,Hkv,page,group,kv,new", SHAPES)
def test_attention_against_64_bits(Hq, Hkv, page, group, kv, new, max_q):
    rng = np.random.default_rng(sum(kv) + Hq)
    cache, table = _filled(rng, kv, Hkv, page, group)
    cu = np.concatenate(([0], np.cumsum(new))).tolist()
    Q = ko.bf16(rng.standard_normal((Hq, cu[-1], 128)) * 1.5)
    ref = ko.attend(cache.pages.cpu().numpy(), page, group, Q, table, kv, cu, 0.1, wide=max_q == MANY)
    o, L = _attend(cache, Q, table, kv, cu, 0.1, pad=3, max_q=max_q)
    assert cache.device_status() == 0
    _compare(o, L, ref)


@pytest.mark.parametrize("max_q", [0, 1, 5, MANY])
def test_attention_hint_only_picks_the_tile(max_q):
    rng = np.random.default_rng(2)
    cache, table = _filled(rng, [130, 50], 2, 64, 64)
    Q = ko.bf16(rng.standard_normal((8, 8, 128)))
    ref = ko.attend(cache.pages.cpu().numpy(), 64, 64, Q, table, [130, 50], [0, 5, 8], 0.2, wide=max_q == MANY)
    o, L = _attend(cache, Q, table, [130, 50], [0, 5, 8], 0.2, max_q=max_q)
    _compare(o, L, ref)


def _torch_attend(cache, Q, table, kv, cu, scale):
    """fp64 on the GPU for long contexts, from the library's own read back in fp64 via the format."""
    page, group, Hkv = cache.page, cache.group, cache.Hkv
    ng = 128 // group
    G = Q.shape[0] // Hkv
    O, L = torch.zeros(Q.shape, dtype=torch.float64, device="cuda"), torch.zeros(Q.shape[:2], dtype=torch.float64, device="cuda")
    x = torch.arange(128, device="cuda")
    for b in range(len(kv)):
        j = torch.arange(kv[b], device="cuda")
        pg, r = _ints(table)[b].long()[j // page], j % page
        blk = cache.pages.view(cache.n_pages, Hkv, page // 16, -1)[pg, :, r // 16]  # [kv, Hkv, bytes]
        i = (r % 16)[:, None]
        at = {"k": 64 * i + 16 * (x % 32 // 8) + 4 * (x // 32) + x % 8 // 2,
              "v": 1024 + 64 * i + 8 * ((x % 32 // 4) ^ (4 * (i // 2 % 2))) + 2 * (x // 32) + x % 4 // 2}
        val = {}
        for n, base in (("k", 2048), ("v", 2048 + 64 * ng)):
            byte = blk.gather(2, at[n][:, None].expand(-1, Hkv, -1)).int()
            code = torch.where(x % 2 == 1, byte >> 4, byte & 15).double()
            sm = blk.gather(2, (base + 4 * ng * i + torch.arange(4 * ng, device="cuda"))[:, None].expand(-1, Hkv, -1))
            sm = sm.contiguous().view(torch.bfloat16).double().view(kv[b], Hkv, ng, 2)
            val[n] = (sm[..., 1].repeat_interleave(group, -1) + code * sm[..., 0].repeat_interleave(group, -1)).transpose(0, 1)
        for h in range(Q.shape[0]):
            q = Q[h, cu[b]:cu[b + 1]].double()
            s = q @ val["k"][h // G].T * scale
            n = cu[b + 1] - cu[b]
            s = s.masked_fill(j[None] > (kv[b] - n + torch.arange(n, device="cuda"))[:, None], float("-inf"))
            L[h, cu[b]:cu[b + 1]] = torch.logsumexp(s, -1)
            O[h, cu[b]:cu[b + 1]] = torch.softmax(s, -1) @ val["v"][h // G]
    return O, L


@pytest.mark.parametrize("Hq,Hkv,page,group,kv,new", [
    (28, 4, 64, 64, [40000], [1]),
    (32, 8, 64, 128, [9000, 33, 15000, 1, 4097], [1] * 5),
    (8, 2, 16, 32, [20001, 77], [2, 2]),
    (28, 4, 128, 64, [3001, 1500], [130, 257]),
    (4, 4, 32, 32, [5000] * 3, [33, 1, 64]),
    (8, 1, 64, 128, [50000], [8]),                    # one pair of 64 rows, cut over every CTA
    (4, 1, 16, 64, [2100, 900], [2100, 800]),         # prompts from their start: folds
    (28, 4, 256, 32, [20000, 300, 7000], [300, 300, 1]),
])
def test_attention_over_long_contexts_split_over_the_gpu(Hq, Hkv, page, group, kv, new):
    """Contexts cut over many CTAs and joined.  Inputs of unit size: the weighted magnitudes behind an
    output are at most 2 max |v| <= 16, so the bound of kv4_oracle.tolerance is below
    |O| 2^-8 + A 2^-10, with A the weighted mean of |v| + 2 |lo| <= 8 here (8 * 2^-10 < 8e-3).  Scores
    are below 16 in the sum of their magnitudes: lse is off by less than 16 * 2^-16 < 2.5e-4."""
    rng = np.random.default_rng(7)
    need = [-(-k // page) for k in kv]
    cache = _cache(sum(need) + 1, Hkv, page, group)
    perm, at = rng.permutation(sum(need) + 1), 0
    table = np.full((len(kv), max(need)), -1, np.int64)
    torch.manual_seed(3)
    for b, k in enumerate(kv):
        table[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
        j = torch.arange(k, device="cuda")
        x = torch.randn(2, Hkv, k, 128, device="cuda", dtype=torch.bfloat16)
        cache.append(x[0], x[1], _ints(table)[b].long()[j // page] * page + j % page)
    cu = np.concatenate(([0], np.cumsum(new))).tolist()
    Q = torch.randn(Hq, cu[-1], 128, device="cuda", dtype=torch.bfloat16)
    O, L = _torch_attend(cache, Q, table, kv, cu, 0.088)
    o, lse = torch.zeros_like(Q), torch.zeros(Hq, cu[-1], device="cuda")
    ws = cache.alloc_workspace()
    args = (_ints(table), _ints(kv), _ints(cu), max(new), 0.088, ws)
    cache.attend(Q, o, *args, lse=lse)
    assert cache.device_status() == 0
    assert ((o.double() - O).abs() <= O.abs() * 2.0 ** -8 + 8 * 2.0 ** -10).all()
    # of the norm: bf16's rounding is below 2^-8 of it, the probabilities' below 2^-10 of the magnitudes
    assert float((o.double() - O).norm() / O.norm()) < 2.0 ** -8 + 2.0 ** -10
    assert float((lse.double() - L).abs().max()) < 2.5e-4
    again, lse2 = torch.zeros_like(Q), torch.zeros_like(lse)
    cache.attend(Q, again, *args, lse=lse2)
    assert torch.equal(o, again) and torch.equal(lse, lse2)  # the same bits
    assert int(ws[:1024].max()) == 0  # ready for the next call


@pytest.mark.parametrize("n,max_q", [(2, 2), (20, MANY)])
@pytest.mark.parametrize("scale_v", [2.0 ** 60, 2.0 ** -60])
def test_attention_scales_far_from_one(scale_v, n, max_q):
    rng = np.random.default_rng(11)
    cache, table = _filled(rng, [150], 1, 16, 64, scale_v=scale_v)
    Q = ko.bf16(rng.standard_normal((4, n, 128)) * 1e-3)
    ref = ko.attend(cache.pages.cpu().numpy(), 16, 64, Q, table, [150], [0, n], 0.1, wide=max_q == MANY)
    _compare(*_attend(cache, Q, table, [150], [0, n], 0.1, max_q=max_q), ref)


@pytest.mark.parametrize("max_q", [1, MANY])
def test_attention_sharp_rows_and_rising_scores(max_q):
    """Scores that rise along the keys move the running maximum again and again; the largest weigh all."""
    rng = np.random.default_rng(12)
    page, group, n = 16, 128, 600
    cache = _cache(40, 1, page, group)
    K = ko.bf16(rng.standard_normal((1, n, 128)) * 0.1)
    K[0, :, 0] = ko.bf16(np.linspace(-100, 100, n))
    V = ko.bf16(rng.standard_normal((1, n, 128)) * np.exp(np.linspace(-6, 6, n))[None, :, None])
    table = np.arange(40)[None]
    cache.append(_dev(K), _dev(V), _ints(np.arange(n), torch.int64))
    Q = np.zeros((3, 1, 128))
    Q[0, 0, 0], Q[1, 0, 0], Q[2, 0, 0] = 4.0, -4.0, 1e-3
    ref = ko.attend(cache.pages.cpu().numpy(), page, group, Q, table, [n], [0, 1], 1.0, wide=max_q == MANY)
    _compare(*_attend(cache, Q, table, [n], [0, 1], 1.0, max_q=max_q), ref)


@pytest.mark.parametrize("max_q", [4, MANY])
def test_attention_nan_keys_reach_only_the_rows_that_see_them(max_q):
    rng = np.random.default_rng(13)
    K, V = _rows_of(rng, 1, 40)
    K, V = K.copy(), V.copy()
    K[0, 38, 3] = np.nan   # seen by the last two of four new tokens
    V[0, 39, 70] = np.inf  # by the last one, in its second group
    cache = _cache(3, 1, 16, 64)
    cache.append(_dev(K), _dev(V), torch.arange(40, device="cuda"))
    Q = ko.bf16(rng.standard_normal((2, 4, 128)))
    ref = ko.attend(cache.pages.cpu().numpy(), 16, 64, Q[:, :2], np.arange(3)[None], [38], [0, 2], 0.1, wide=max_q == MANY)
    o, L = _attend(cache, Q, np.arange(3)[None], [40], [0, 4], 0.1, max_q=max_q)
    _compare(o[:, :2], L[:, :2], ref)
    assert torch.isnan(o[:, 2:]).all() and torch.isnan(L[:, 2:]).all()
    K[0, 38, 3] = 1.0
    cache.append(_dev(K), _dev(V), torch.arange(40, device="cuda"))
    o, L = _attend(cache, Q, np.arange(3)[None], [40], [0, 4], 0.1, max_q=max_q)
    assert torch.isfinite(o[:, :3]).all() and torch.isfinite(L).all()
    assert torch.isfinite(o[:, 3, :64]).all() and torch.isnan(o[:, 3, 64:]).all()


@pytest.mark.parametrize("max_q", [1, MANY])
def test_attention_records_and_hides_what_is_out_of_bounds(max_q):
    rng = np.random.default_rng(14)
    cache, table = _filled(rng, [100, 60], 1, 16, 64, extra_blocks=1)
    Q = ko.bf16(rng.standard_normal((2, 2, 128)))
    host = cache.pages.cpu().numpy()
    broken = table.copy()
    broken[0, 3] = cache.n_pages      # behind the cache
    broken[0, 5] = -1
    ref = ko.attend(host, 16, 64, Q, table, [100, 60], [0, 1, 2], 0.1, wide=max_q == MANY, hidden=lambda b, j: b == 0 and j // 16 in (3, 5))
    o, L = _attend(cache, Q, broken, [100, 60], [0, 1, 2], 0.1, max_q=max_q)
    assert cache.device_status() == 8 and cache.device_status() == 0
    _compare(o, L, ref)
    # lengths behind the table row are cut to it (its last entry names no page)
    o, L = _attend(cache, Q, table, [10 ** 9, 60], [0, 1, 2], 0.1, max_q=max_q)
    assert cache.device_status() == 8
    # rows 100 .. of request 0's last page were never written: NaN, so only request 1 can be compared
    assert torch.isnan(o[:, 0]).all()
    one = ko.attend(host, 16, 64, Q[:, 1:], table[1:], [60], [0, 1], 0.1, wide=max_q == MANY)
    _compare(o[:, 1:], L[:, 1:], one)
    # query offsets that run backwards or out of Q: those requests are left out
    o, L = _attend(cache, Q, table, [100, 60], [5, 1, 2], 0.1, max_q=max_q)
    assert cache.device_status() == 8
    _compare(o[:, 1:], L[:, 1:], one)
    assert (o[:, 0] == 5.0).all()
    o, L = _attend(cache, Q, table, [-5, 60], [0, 1, 2], 0.1, max_q=max_q)
    assert cache.device_status() == 8 and (o[:, 0] == 0).all() and torch.isneginf(L[:, 0]).all()
    _compare(o[:, 1:], L[:, 1:], one)


def test_attention_one_workspace_for_calls_of_different_shapes_and_graphs():
    rng = np.random.default_rng(15)
    cache, table = _filled(rng, [900, 333], 2, 64, 64)
    ws = cache.alloc_workspace()
    small, large = ko.bf16(rng.standard_normal((4, 2, 128))), ko.bf16(rng.standard_normal((4, 70, 128)))
    host = cache.pages.cpu().numpy()
    ref_s = ko.attend(host, 64, 64, small, table, [900, 333], [0, 1, 2], 0.1)
    qs, ql = _dev(small), _dev(large)
    tab, kv, cs, cl = _ints(table), _ints([900, 333]), _ints([0, 1, 2]), _ints([0, 40, 70])
    o_s, o_l = torch.zeros_like(qs), torch.zeros_like(ql)
    cache.attend(ql, o_l, tab, kv, cl, MANY, 0.1, ws)
    first = o_l.clone()
    graphs = []
    for q, o, cu, n in ((qs, o_s, cs, 1), (ql, o_l, cl, MANY)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            cache.attend(q, o, tab, kv, cu, n, 0.1, ws)
        graphs.append(g)
    o_s.zero_(), o_l.zero_()
    for _ in range(3):
        for g in graphs:
            g.replay()
    assert torch.equal(o_l, first)
    L = torch.zeros(4, 2, device="cuda")
    o = torch.zeros_like(qs)
    cache.attend(qs, o, tab, kv, cs, 1, 0.1, ws, lse=L)
    assert torch.equal(o, o_s)
    _compare(o, L, ref_s)
    # lengths are read on the device: a replay follows them
    kv[0] = 800
    graphs[0].replay()
    ref = ko.attend(host, 64, 64, small, table, [800, 333], [0, 1, 2], 0.1)
    assert (np.abs(_host(o_s) - ref[0]) <= ref[2]).all() and not torch.equal(o, o_s)


@pytest.mark.parametrize("B,max_q,wide", [(2048, 1, False), (1025, MANY, False), (1024, MANY, True)])
def test_attention_most_requests(B, max_q, wide):
    """The most requests of a call, and of the kernel for many rows (above it the other one serves)."""
    rng = np.random.default_rng(B)
    kv = rng.integers(0, 12, B)
    K, V = _rows_of(rng, 1, int(kv.sum()))
    cache = _cache(B, 1, 16, 128)
    table = rng.permutation(B)[:, None]
    sl = np.concatenate([table[b, 0] * 16 + np.arange(k) for b, k in enumerate(kv)])
    cache.append(_dev(K), _dev(V), _ints(sl, torch.int64))
    new = rng.integers(0, 3, B)
    cu = np.concatenate(([0], np.cumsum(new))).tolist()
    Q = ko.bf16(rng.standard_normal((2, cu[-1], 128)))
    ref = ko.attend(cache.pages.cpu().numpy(), 16, 128, Q, table, kv.tolist(), cu, 0.1, wide=wide)
    o, L = _attend(cache, Q, table, kv, cu, 0.1, max_q=max_q, pad=2)
    assert cache.device_status() == 0
    _compare(o, L, ref)


@pytest.mark.parametrize("max_q", [3, MANY])
def test_attention_rows_of_any_size_side_by_side(max_q):
    """Rows of one tile whose queries are 2^60 times the others', infinite or NaN: every finite row is its own."""
    rng = np.random.default_rng(19)
    cache, table = _filled(rng, [200], 1, 16, 64)
    Q = ko.bf16(rng.standard_normal((4, 3, 128)))
    Q[0, 1] *= 2.0 ** -60
    ref = ko.attend(cache.pages.cpu().numpy(), 16, 64, Q, table, [200], [0, 3], 0.1, wide=max_q == MANY)
    broken = Q.copy()
    broken[1, 0, 5], broken[2, 1, 100], broken[3, 2, 0] = np.inf, np.nan, -np.inf
    broken[0, 2] = ko.bf16(Q[0, 2] * 2.0 ** 60)
    o, L = _attend(cache, broken, table, [200], [0, 3], 0.1, max_q=max_q)
    for h, t in ((1, 0), (2, 1), (3, 2)):
        assert torch.isnan(o[h, t]).all() and torch.isnan(L[h, t])
        o[h, t], L[h, t] = 0.0, 0.0
        ref[0][h, t] = ref[1][h, t] = 0.0
    big = ko.attend(cache.pages.cpu().numpy(), 16, 64, broken[:1], table, [200], [0, 3], 0.1, wide=max_q == MANY)
    for x, y in zip(ref, big):  # scores of 2^60 too
        x[0, 2] = y[0, 2]
    _compare(o, L, ref)


@pytest.mark.parametrize("max_q", [1, MANY])
def test_attention_in_place(max_q):
    rng = np.random.default_rng(20)
    cache, table = _filled(rng, [700, 90, 33], 2, 16, 64)
    q = _dev(rng.standard_normal((8, 60, 128)))
    args = (_ints(table), _ints([700, 90, 33]), _ints([0, 37, 59, 60]), max_q, 0.1, cache.alloc_workspace())
    o = torch.zeros_like(q)
    cache.attend(q, o, *args)
    cache.attend(q, q, *args)
    assert torch.equal(o, q)


def test_two_attention_calls_at_once_with_a_workspace_each():
    rng = np.random.default_rng(16)
    cache, table = _filled(rng, [2000, 1000], 2, 64, 128)
    q = _dev(rng.standard_normal((8, 2, 128)))
    tab, kv, cu = _ints(table), _ints([2000, 1000]), _ints([0, 1, 2])
    ref = torch.zeros_like(q)
    cache.attend(q, ref, tab, kv, cu, 1, 0.1, cache.alloc_workspace())
    outs, streams = [torch.zeros_like(q) for _ in range(2)], [torch.cuda.Stream() for _ in range(2)]
    wss = [cache.alloc_workspace() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for o, s, w in zip(outs, streams, wss):
            cache.attend(q, o, tab, kv, cu, 1, 0.1, w, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], ref) and torch.equal(outs[1], ref)


def test_offsets_behind_32_bits():
    """Pages whose bytes lie behind 2^32 in the cache."""
    page, group, Hkv = 256, 128, 8
    per = Hkv * msa.kv4_page_bytes(page, group)
    n_pages = (1 << 32) // per + 40
    cache = msa.KV4Cache(torch.empty(n_pages, Hkv, per // Hkv, dtype=torch.uint8, device="cuda"), page, group)
    rng = np.random.default_rng(17)
    K, V = _rows_of(rng, Hkv, 300)
    table = np.array([[n_pages - 1, n_pages - 30]])
    sl = [table[0, j // page] * page + j % page for j in range(300)]
    cache.append(_dev(K), _dev(V), _ints(sl, torch.int64))
    k, v = torch.zeros(Hkv, 300, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(Hkv, 300, 128, dtype=torch.bfloat16, device="cuda")
    cache.read(_ints(sl, torch.int64), k, v)
    code, step, lo = ko.quantise(V, group)
    want = np.repeat(lo, group, -1) + code * np.repeat(step, group, -1)
    assert (np.abs(_host(v) - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -23)).all()
    Q = ko.bf16(rng.standard_normal((Hkv, 1, 128)))
    # the same tokens in a small cache give the same bits
    small = _cache(2, Hkv, page, group)
    small.append(_dev(K), _dev(V), torch.arange(300, device="cuda"))
    o1, l1 = _attend(cache, Q, table, [300], [0, 1], 0.1)
    o2, l2 = _attend(small, Q, np.array([[0, 1]]), [300], [0, 1], 0.1)
    assert torch.equal(o1, o2) and torch.equal(l1, l2)


# ---- a run of them together ----------------------------------------------------------------------
def test_prompt_then_decoding_through_the_layer():
    """norm + rotation -> sparse prefill (dense heads) -> the cache, then three single-token steps:
    every step's attention against 64 bits over the values the cache stands for, and the first step
    against the unquantised layer within what 4 bits leave."""
    from workload import TEXT, Head, Problem
    L, Hq, Hkv, page, group = 1088, 4, 2, 64, 32
    p = Problem(L=L, Hq=Hq, Hkv=Hkv, segments=[(0, L, TEXT)], heads=[Head("dense")] * Hq)
    torch.manual_seed(1)
    proj = torch.randn(L + 3, Hq + 2 * Hkv, 128, device="cuda", dtype=torch.bfloat16)
    w = [(1 + 0.1 * torch.randn(128, device="cuda")).to(torch.bfloat16) for _ in range(2)]
    rope = msa.Rope(base=1e6)
    cache = _cache(24, Hkv, page, group)
    table, kv = torch.full((1, 20), -1, dtype=I32, device="cuda"), _ints([0])
    free, nf = _ints(np.random.default_rng(0).permutation(24)), _ints([24])
    sl, pos, cu = torch.zeros(L, dtype=torch.int64, device="cuda"), torch.zeros(L, dtype=I32, device="cuda"), _ints([0, 0])

    def project(t0, t1):
        x = proj[t0:t1]
        Q, K = (torch.empty(h, t1 - t0, 128, dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv))
        msa.qk_norm_rope(x[:, :Hq].transpose(0, 1), x[:, Hq:Hq + Hkv].transpose(0, 1), Q, K, pos[:t1 - t0], rope, *w)
        return Q, K, x[:, Hq + Hkv:].transpose(0, 1)

    cache.slots(kv, _ints([L]), table, free, nf, sl, pos, cu)
    Q, K, V = project(0, L)
    plan = msa.Plan(p)
    ws, O = plan.alloc_workspace(indexed=True), torch.empty_like(Q)
    plan.forward(Q, K, V, ws, O, indexed=True, cache=cache, slots=sl)
    assert plan.device_status(ws) == 0 and cache.device_status() == 0
    O2 = torch.empty_like(Q)
    plan.forward(Q, K, V, ws, O2, indexed=True)
    assert torch.equal(O, O2)  # the cache changes nothing in the layer
    aws = cache.alloc_workspace()
    Ks, Vs = [K], [V]
    for step in range(3):
        cache.slots(kv, _ints([1]), table, free, nf, sl, pos, cu)
        q, k, v = project(L + step, L + step + 1)
        cache.append(k, v, sl[:1])
        o, lse = torch.empty_like(q), torch.empty(Hq, 1, device="cuda")
        cache.attend(q, o, table, kv, cu, 1, p.scale, aws, lse=lse)
        assert cache.device_status() == 0 and kv.tolist() == [L + step + 1] and pos[0] == L + step
        ref = ko.attend(cache.pages.cpu().numpy(), page, group, _host(q), table.cpu().numpy(), kv.tolist(), [0, 1], p.scale)
        _compare_exact(o, lse, ref)
        Ks.append(k), Vs.append(v)
        kk, vv = torch.cat(Ks, 1).double().repeat_interleave(2, 0), torch.cat(Vs, 1).double().repeat_interleave(2, 0)
        full = torch.softmax(q.double() @ kk.transpose(1, 2) * p.scale, -1) @ vv
        # steps of at most 7 / 15 per group of 32: a value is off by 0.14 rms; over ~1000 keys the errors average out
        assert float((o.double() - full).norm() / full.norm()) < 0.25
    # the cached prefix, read back, is the layer's K and V within a step
    kb, vb = torch.empty_like(K), torch.empty(Hkv, L, 128, dtype=torch.bfloat16, device="cuda")
    t = torch.arange(L, device="cuda")
    cache.read(table[0].long()[t // page] * page + t % page, kb, vb)
    rng_ = K.float().view(Hkv, L, -1, group)
    step = ((rng_.amax(-1) - rng_.amin(-1)) / 15).repeat_interleave(group, -1)
    # half a step, the step's rounding over 15 codes, and the value's
    assert ((kb.float() - K.float()).abs() <= step * (0.5 + 15 * 2.0 ** -8) + kb.float().abs() * 2.0 ** -8).all()


def _compare_exact(o, lse, ref):
    O, L, tO, tL = ref
    assert (np.abs(_host(o) - O) <= tO).all() and (np.abs(lse.cpu().numpy() - L) <= tL).all()


def test_step_of_a_decoding_batch_in_one_graph():
    """Slot map, norm + rotation, write and attention of one token per request captured once and
    replayed: the lengths advance on the device."""
    rng = np.random.default_rng(18)
    B, Hq, Hkv, page, group = 5, 8, 2, 16, 64
    cache = _cache(60, Hkv, page, group)
    lens = [3, 15, 16, 31, 40]
    table, kv = torch.full((B, 8), -1, dtype=I32, device="cuda"), _ints([0] * B)
    free, nf = _ints(rng.permutation(60)), _ints([60])
    n0 = sum(lens)
    sl, pos, cu = torch.zeros(n0, dtype=torch.int64, device="cuda"), torch.zeros(n0, dtype=I32, device="cuda"), _ints([0] * (B + 1))
    cache.slots(kv, _ints(lens), table, free, nf, sl, pos, cu)
    K, V = _rows_of(rng, Hkv, n0)
    cache.append(_dev(K), _dev(V), sl)
    x = torch.zeros(B, Hq + 2 * Hkv, 128, dtype=torch.bfloat16, device="cuda")
    one, rope, ws = _ints([1] * B), msa.Rope(base=1e4), cache.alloc_workspace()
    q, k = torch.zeros(Hq, B, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(Hkv, B, 128, dtype=torch.bfloat16, device="cuda")
    o, lse = torch.zeros_like(q), torch.zeros(Hq, B, device="cuda")

    def step():
        cache.slots(kv, one, table, free, nf, sl[:B], pos[:B], cu)
        msa.qk_norm_rope(x[:, :Hq].transpose(0, 1), x[:, Hq:Hq + Hkv].transpose(0, 1), q, k, pos[:B], rope)
        cache.append(k, x[:, Hq + Hkv:].transpose(0, 1), sl[:B])
        cache.attend(q, o, table, kv, cu, 1, 0.1, ws, lse=lse)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(4):
        x.copy_(torch.from_numpy(rng.standard_normal((B, Hq + 2 * Hkv, 128)).astype(np.float32)))
        g.replay()
        assert cache.device_status() == 0
        assert kv.tolist() == [n + i + 1 for n in lens] and pos[:B].tolist() == [n + i for n in lens]
        ref = ko.attend(cache.pages.cpu().numpy(), page, group, _host(q), table.cpu().numpy(), kv.tolist(), cu.tolist(), 0.1)
        _compare_exact(o, lse, ref)
