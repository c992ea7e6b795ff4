"""Host side of the operators around the layer: sizes, argument checks and refusals of the calls (made
before any device access, so placeholder addresses do), and the tests' own 64-bit forms."""
import copy
import ctypes
import pickle

import numpy as np
import pytest

import kv4_oracle as ko
import dynamic_sparse_attention_head_b200 as msa
from dynamic_sparse_attention_head_b200 import KV4CacheC, RopeC, Strides, _lib

INVALID, SHAPE, ALIGN, WORKSPACE, UNSUPPORTED = 1, 2, 3, 4, 5
FAKE = 1 << 20  # 16- and 256-byte aligned, never touched


def _strides(row=128, head=4096 * 128):
    return Strides(**{f"{n}_{k}": v for n in "qkvo" for k, v in (("head", head), ("row", row))})


def _cache(**kw):
    f = dict(pages=FAKE, n_pages=100, page_tokens=64, Hkv=4, group=64, state=FAKE)
    f.update(kw)
    return ctypes.byref(KV4CacheC(**f))


def test_page_bytes():
    for page in (16, 32, 64, 128, 256):
        for group in (32, 64, 128):
            n = msa.kv4_page_bytes(page, group)
            assert n == page * ko.row_bytes(group) and n % 16 == 0
    for page, group in ((8, 64), (48, 64), (512, 64), (0, 64), (-16, 64), (64, 16), (64, 0), (64, 256)):
        assert _lib.msa_kv4_page_bytes(page, group) == 0
        with pytest.raises(ValueError):
            msa.kv4_page_bytes(page, group)


def _rope(**kw):
    c = RopeC(dim=128, n_axes=1, scale=1.0)
    for k, v in kw.items():
        if k == "sections":
            for i, x in enumerate(v):
                c.sections[i] = x
        elif k == "inv_freq":
            for i, x in enumerate(v):
                c.inv_freq[i] = x
        else:
            setattr(c, k, v)
    return ctypes.byref(c)


def test_norm_rope_argument_checks():
    def call(Q=FAKE, K=FAKE, i=_strides(), Qo=FAKE, Ko=FAKE, o=_strides(), T=5, Hq=4, Hkv=2, wq=FAKE, wk=None, eps=1e-6,
             rope=None, pos=FAKE, ps=5):
        return _lib.msa_qk_norm_rope(Q, K, ctypes.byref(i) if i else None, Qo, Ko, ctypes.byref(o) if o else None, T, Hq,
                                     Hkv, wq, wk, eps, rope or _rope(), pos, ps, None)
    for kw in (dict(Q=None), dict(K=None), dict(Qo=None), dict(Ko=None), dict(i=None), dict(o=None), dict(T=-1),
               dict(Hq=-1), dict(Hkv=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(pos=None),
               dict(rope=_rope(n_axes=0)), dict(rope=_rope(n_axes=5)), dict(rope=_rope(scale=float("nan"))),
               dict(rope=_rope(inv_freq=[float("inf")])), dict(rope=_rope(n_axes=2, sections=[-1, 65]))):
        assert call(**kw) == INVALID, kw
    for kw in (dict(rope=_rope(dim=130)), dict(rope=_rope(dim=24)), dict(rope=_rope(dim=-16)),
               dict(rope=_rope(n_axes=2, sections=[10, 10])), dict(rope=_rope(n_axes=2, sections=[32, 32]), ps=4)):
        assert call(**kw) == SHAPE, kw
    for kw in (dict(Q=FAKE + 8), dict(Ko=FAKE + 2), dict(wq=FAKE + 8), dict(wk=FAKE + 4), dict(i=_strides(row=100)),
               dict(o=_strides(head=129)), dict(pos=FAKE + 2)):
        assert call(**kw) == ALIGN, kw
    assert call(Hq=70000) == UNSUPPORTED and call(T=1 << 32, ps=1 << 32) == UNSUPPORTED
    assert call(T=0, Q=None, K=None, Qo=None, Ko=None, pos=None) == 0  # nothing to do, no launch
    assert call(Hq=0, Hkv=0) == 0


def test_rope_description_checks():
    assert msa.Rope(dim=64).n_axes == 1 and msa.Rope(sections=(16, 24, 24)).n_axes == 3
    for kw in (dict(dim=8), dict(dim=144), dict(dim=64, inv_freq=[1.0]), dict(sections=(1, 2, 3)), dict(sections=()),
               dict(sections=(-1, 65)), dict(sections=(10, 10, 10, 10, 24))):
        with pytest.raises(ValueError):
            msa.Rope(**kw)


def test_rope_copies_stand_alone():
    rope = msa.Rope(sections=(16, 24, 24), scale=0.5)
    for twin in (copy.deepcopy(rope), pickle.loads(pickle.dumps(rope))):
        assert ctypes.addressof(twin._c) != ctypes.addressof(rope._c)
        assert bytes(twin._c) == bytes(rope._c) and twin.n_axes == 3
        assert not any(v == ctypes.addressof(rope._c) for v in vars(twin).values() if isinstance(v, int))


def test_cache_argument_checks():
    bad = [(dict(pages=None), INVALID), (dict(state=None), INVALID), (dict(n_pages=0), INVALID),
           (dict(n_pages=1 << 31), INVALID), (dict(page_tokens=48), SHAPE), (dict(group=16), SHAPE), (dict(Hkv=0), SHAPE),
           (dict(Hkv=2000), SHAPE), (dict(pages=FAKE + 8), ALIGN), (dict(state=FAKE + 4), ALIGN)]
    s = ctypes.byref(_strides())
    ws = int(_lib.msa_kv4_attend_workspace_bytes())
    for kw, code in bad:
        c = _cache(**kw)
        assert _lib.msa_kv4_append(c, FAKE, FAKE, s, FAKE, 1, None) == code, kw
        assert _lib.msa_kv4_read(c, FAKE, FAKE, s, FAKE, 1, None) == code, kw
        assert _lib.msa_kv4_slots(c, FAKE, FAKE, 1, FAKE, 8, 8, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1, None) == code
        assert _lib.msa_kv4_release(c, FAKE, 1, FAKE, 1, FAKE, 8, 8, FAKE, FAKE, None) == code, kw
        assert _lib.msa_kv4_attend(c, FAKE, FAKE, s, 1, 4, 0.1, FAKE, 8, 8, FAKE, FAKE, 1, 1, None, FAKE, ws, None) == code
        assert _lib.msa_kv4_status(c, None) == code, kw
    assert _lib.msa_kv4_append(None, FAKE, FAKE, s, FAKE, 1, None) == INVALID


def test_append_read_argument_checks():
    for fn in (_lib.msa_kv4_append, _lib.msa_kv4_read):
        def call(K=FAKE, V=FAKE, s=_strides(), slots=FAKE, T=3):
            return fn(_cache(), K, V, ctypes.byref(s) if s else None, slots, T, None)
        for kw in (dict(K=None), dict(V=None), dict(s=None), dict(slots=None), dict(T=-1)):
            assert call(**kw) == INVALID, kw
        for kw in (dict(K=FAKE + 8), dict(V=FAKE + 4), dict(slots=FAKE + 4), dict(s=_strides(row=12))):
            assert call(**kw) == ALIGN, kw
        assert call(T=1 << 33) == UNSUPPORTED
        assert call(T=0, K=None, V=None, slots=None) == 0


def test_slots_release_argument_checks():
    def slots(kv=FAKE, new=FAKE, B=2, table=FAKE, stride=8, blocks=8, free=FAKE, nf=FAKE, kvo=FAKE, nfo=FAKE, cu=FAKE,
              sl=FAKE, pos=FAKE, cap=4):
        return _lib.msa_kv4_slots(_cache(), kv, new, B, table, stride, blocks, free, nf, kvo, nfo, cu, sl, pos, cap, None)
    for kw in (dict(kv=None), dict(new=None), dict(B=-1), dict(table=None), dict(free=None), dict(nf=None), dict(kvo=None),
               dict(nfo=None), dict(cu=None), dict(sl=None), dict(pos=None), dict(cap=-1), dict(blocks=-1)):
        assert slots(**kw) == INVALID, kw
    assert slots(stride=7) == SHAPE and slots(sl=FAKE + 4) == ALIGN
    assert slots(B=2049) == UNSUPPORTED and slots(blocks=1 << 26, stride=1 << 26) == UNSUPPORTED

    def release(ids=FAKE, n=2, kv=FAKE, B=2, table=FAKE, stride=8, blocks=8, free=FAKE, nf=FAKE):
        return _lib.msa_kv4_release(_cache(), ids, n, kv, B, table, stride, blocks, free, nf, None)
    for kw in (dict(ids=None), dict(n=-1), dict(kv=None), dict(B=-1), dict(table=None), dict(free=None), dict(nf=None)):
        assert release(**kw) == INVALID, kw
    assert release(stride=7) == SHAPE and release(n=2049) == UNSUPPORTED
    assert release(n=0, ids=None) == 0
    for kw in (dict(kv=FAKE + 2), dict(new=FAKE + 2), dict(table=FAKE + 1), dict(free=FAKE + 2), dict(nf=FAKE + 2),
               dict(kvo=FAKE + 2), dict(nfo=FAKE + 2), dict(cu=FAKE + 2), dict(pos=FAKE + 2)):
        assert slots(**kw) == ALIGN, kw
    for kw in (dict(ids=FAKE + 2), dict(kv=FAKE + 2), dict(table=FAKE + 2), dict(free=FAKE + 2), dict(nf=FAKE + 2)):
        assert release(**kw) == ALIGN, kw


def test_attend_argument_checks():
    ws = int(_lib.msa_kv4_attend_workspace_bytes())

    def call(c=None, Q=FAKE, O=FAKE, s=_strides(), T=3, Hq=8, scale=0.1, table=FAKE, stride=8, blocks=8, kv=FAKE, cu=FAKE,
             B=2, max_q=2, lse=None, w=FAKE, wb=ws):
        return _lib.msa_kv4_attend(c or _cache(), Q, O, ctypes.byref(s) if s else None, T, Hq, scale, table, stride, blocks,
                                   kv, cu, B, max_q, lse, w, wb, None)
    for kw in (dict(Q=None), dict(O=None), dict(s=None), dict(T=-1), dict(scale=0.0), dict(scale=-1.0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(table=None), dict(kv=None), dict(cu=None),
               dict(B=-1), dict(max_q=-1), dict(w=None), dict(blocks=-1)):
        assert call(**kw) == INVALID, kw
    assert call(Hq=6) == SHAPE and call(Hq=0) == SHAPE and call(stride=7) == SHAPE
    for kw in (dict(Q=FAKE + 8), dict(O=FAKE + 2), dict(w=FAKE + 128), dict(s=_strides(row=4))):
        assert call(**kw) == ALIGN, kw
    assert call(wb=ws - 1) == WORKSPACE
    assert call(B=2049) == UNSUPPORTED and call(blocks=1 << 26, stride=1 << 26) == UNSUPPORTED
    assert call(T=1 << 30, Hq=16) == UNSUPPORTED
    # 2^31 - 2^15 tokens a row: numbers that a warp looks ahead to would pass 32 bits
    assert call(blocks=(1 << 31) - (1 << 15) >> 6, stride=1 << 26) == UNSUPPORTED
    for kw in (dict(table=FAKE + 2), dict(kv=FAKE + 1), dict(cu=FAKE + 2), dict(lse=FAKE + 2)):
        assert call(**kw) == ALIGN, kw
    assert call(scale=3e38) == INVALID  # log2(e) of it is infinite
    assert call(T=0, Q=None, O=None) == 0 and call(B=0, kv=None, cu=None, table=None) == 0


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    torch = pytest.importorskip("torch")
    pages = torch.zeros(4, 2, msa.kv4_page_bytes(16, 64), dtype=torch.uint8)
    with pytest.raises(ValueError):
        msa.KV4Cache(pages, page=16, group=64)  # not on a GPU
    with pytest.raises(ValueError):
        msa.KV4Cache(pages, page=32, group=64)  # another page's bytes
    with pytest.raises(ValueError):
        msa.KV4Cache(pages.float(), page=16, group=64)
    Q, K = torch.zeros(4, 3, 128, dtype=torch.bfloat16), torch.zeros(2, 3, 128, dtype=torch.bfloat16)
    pos, rope = torch.zeros(3, dtype=torch.int32), msa.Rope()
    with pytest.raises(ValueError):
        msa.qk_norm_rope(Q, K, Q, K, pos, rope)  # not on a GPU
    for bad in (dict(K=K[:, :2]), dict(K=K.float()), dict(pos=pos[:2]), dict(pos=pos.long()), dict(Qo=K),
                dict(wq=torch.ones(64, dtype=torch.bfloat16)), dict(rope=msa.Rope(sections=(32, 32)))):
        a = dict(Q=Q, K=K, Qo=Q, Ko=K, pos=pos, rope=rope, wq=None)
        a.update(bad)
        with pytest.raises(ValueError):
            msa.qk_norm_rope(a["Q"], a["K"], a["Qo"], a["Ko"], a["pos"], a["rope"], wq=a["wq"])


def test_forward_takes_cache_and_slots_together():
    from workload import llama3_8b_text
    plan = msa.Plan(llama3_8b_text(L=4096))
    with pytest.raises(ValueError):
        plan.forward(None, None, None, None, None, slots=1)


# ---- the 64-bit forms themselves -----------------------------------------------------------------
def test_oracle_format_round_trip_and_error():
    """Every value comes back within half a step (the codes' borders) plus the step's own rounding
    (15 * 2^-9 of a step) and the clamp of the last code; a page's bytes are all used once."""
    rng = np.random.default_rng(0)
    for group in (32, 64, 128):
        x = ko.bf16(rng.standard_normal((6, 128)) * 3)
        code, step, lo = ko.quantise(x, group)
        back = np.repeat(lo, group, -1) + code * np.repeat(step, group, -1)
        assert (np.abs(back - x) <= np.repeat(step, group, -1) * (0.5 + 15 * 2.0 ** -8)).all()
        pages = np.full((2, 1, 16 * ko.row_bytes(group)), 0xAA, np.uint8)
        touched = np.zeros_like(pages)
        for slot in range(16, 32):
            before = pages.copy()
            pages[1] ^= 0xFF  # every byte changes unless the write sets it
            after_flip = pages.copy()
            ko.write(pages, 16, group, slot, 0, x[slot % 6], x[(slot + 1) % 6])
            k, v, ks, vs = ko._offsets(slot % 16, group)
            own = np.zeros(pages.shape[-1], bool)
            own[np.unique(k)] = own[np.unique(v)] = True
            own[ks:ks + 4 * (128 // group)] = own[vs:vs + 4 * (128 // group)] = True
            assert (pages[1, 0][~own] == after_flip[1, 0][~own]).all()
            touched[1, 0] += own
            pages[1] ^= 0xFF * (~own).astype(np.uint8)
            assert (pages[0] == before[0]).all()
            (kc, kst, klo), (vc, vst, vlo) = ko.parts(pages, 16, group, slot, 0)
            assert (kc == code[slot % 6]).all() and (vc == code[(slot + 1) % 6]).all()
            assert (klo == np.repeat(lo[slot % 6], group)).all() and (vst == np.repeat(step[(slot + 1) % 6], group)).all()
        assert (touched[1] == 1).all()


def test_oracle_quantise_edges():
    x = np.zeros((5, 128))
    x[1] = 7.0                      # one value
    x[2, 3] = np.inf
    x[3, 3], x[3, 4] = 3.3e38, -3.3e38
    x[3] = ko.bf16(x[3])
    x[4, 0] = 2.0 ** -127           # below the smallest step
    code, step, lo = ko.quantise(x, 128)
    assert (code[:2] == 0).all() and (step[:2] == 0).all() and lo[1, 0] == 7.0
    assert np.isnan(step[2:4]).all() and np.isnan(lo[2:4]).all()
    assert step[4, 0] == 0 and (code[4] == 0).all()


def test_oracle_attention_against_direct_form():
    rng = np.random.default_rng(3)
    page, group = 16, 64
    pages = np.zeros((4, 1, page * ko.row_bytes(group)), np.uint8)
    for s in range(64):
        ko.write(pages, page, group, s, 0, ko.bf16(rng.standard_normal(128)), ko.bf16(rng.standard_normal(128)))
    Q = ko.bf16(rng.standard_normal((2, 5, 128)))
    table = np.array([[2, 0, 1, -1], [3, -1, -1, -1]])
    O, L, tO, tL = ko.attend(pages, page, group, Q, table, [37, 2], [0, 1, 4], 0.1)
    K = np.stack([np.add(*(lambda c, s, l: (l, c * s))(*ko.parts(pages, page, group, table[0, j // 16] * 16 + j % 16, 0)[0]))
                  for j in range(37)])
    s = K @ Q[1, 0] * 0.1
    assert abs(L[1, 0] - np.log(np.exp(s).sum())) < 1e-12
    assert np.isneginf(L[0, 1]) and (O[0, 1] == 0).all()  # first of three new tokens on two cached ones
    assert np.isfinite(L[0, 2]) and np.isnan(L[0, 4])
    assert (tO[0, 0] > 0).all() and (tO[0, 0] < 0.05).all() and 0 < tL[0, 0] < 1e-2


def test_oracle_slots():
    table = np.full((3, 4), -1)
    table[1, 0] = 9
    free = np.array([5, 6, 7, 8, 0, 0])
    t, kv, nf, cu, sl, pos, ok = ko.slots([0, 15, 0], [3, 2, 16], table, free, 4, 16, 4)
    assert ok and kv == [3, 17, 16] and nf == 1 and cu == [0, 3, 5, 21]
    assert t[0, 0] == 8 and t[1].tolist() == [9, 7, -1, -1] and t[2, 0] == 6
    assert sl[:5] == [128, 129, 130, 9 * 16 + 15, 7 * 16] and pos[3:5] == [15, 16]
    t, kv, nf, cu, sl, pos, ok = ko.slots([0, 0, 0], [3, 33, 1], np.full((3, 4), -1), free, 3, 16, 4)
    assert not ok and kv == [3, 0, 0] and nf == 2 and sl[3:] == [-1] * 34
