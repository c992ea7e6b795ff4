"""msa_qk_norm_rope against the formula in 64 bits.  The kernel works in fp32 and rounds once: a
result is off by at most half a bf16 step (2^-8 of it) and by 2^-18 of the magnitudes behind it (the
norm's sum of 128 squares in a tree of 8 + 4 levels, rsqrt and two products: below 2^-20 together;
the angle held to 2^-25 of half a turn, pi 2^-25 < 2^-23, and sine and cosine to 2^-22)."""
import numpy as np
import pytest

import kv4_oracle as ko

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import dynamic_sparse_attention_head_b200 as msa  # noqa: E402


def _dev(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16).cuda()


def _host(t):
    return t.float().cpu().numpy().astype(np.float64)


def _check(got, x, pos, rope_args, w, eps=1e-6):
    dim, inv, axis, inter, scale = rope_args
    ref, mag = ko.norm_rope(x, pos, inv, axis, dim, inter, w, eps, scale)
    err = np.abs(got - ref)
    tol = np.abs(ref) * 2.0 ** -8 + mag * 2.0 ** -18 + 2.0 ** -133
    assert np.isfinite(got).all()
    assert (err <= tol).all(), float((err / tol).max())


def _axis(sections):
    return [a for a, n in enumerate(sections) for _ in range(n)]


CASES = [  # T, Hq, Hkv, dim, interleaved, sections, norm
    (1, 28, 4, 128, False, None, True),
    (1, 1, 1, 128, True, None, False),
    (7, 12, 1, 64, False, None, True),
    (33, 5, 3, 96, True, (12, 18, 18), True),
    (65, 32, 8, 128, False, (16, 24, 24), True),
    (129, 2, 1, 32, False, (0, 16), False),
    (3, 4, 4, 16, True, (2, 2, 2, 2), True),
    (5, 4, 2, 0, False, None, True),
    (1000, 28, 4, 128, False, None, True),
    (2, 0, 3, 128, False, None, True),
    (2, 3, 0, 128, True, None, True),
]


@pytest.mark.parametrize("T,Hq,Hkv,dim,inter,sections,norm", CASES)
def test_against_formula(T, Hq, Hkv, dim, inter, sections, norm):
    rng = np.random.default_rng(T * 131 + dim)
    qk = ko.bf16(rng.standard_normal((T, Hq + Hkv, 128)) * np.exp(rng.uniform(-4, 4, (T, Hq + Hkv, 1))))
    axes = len(sections) if sections else 1
    pos = rng.integers(0, 1 << 20, (axes, T)).astype(np.int32)
    pos[:, 0] = [0, 2 ** 31 - 1, -5, 12345][:axes]
    w = [ko.bf16(1 + 0.3 * rng.standard_normal(128)) if norm else None for _ in range(2)]
    rope = msa.Rope(dim=dim, base=1e6, interleaved=inter, sections=sections, scale=1.25 if inter else 1.0)
    inv = [1e6 ** (-2 * i / dim) for i in range(dim // 2)]
    d = _dev(qk)
    Q, K = d[:, :Hq].transpose(0, 1), d[:, Hq:].transpose(0, 1)  # the projection's layout
    Qo = torch.full((Hq, T, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    Ko = torch.full((T, Hkv, 128), 9.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    p = torch.from_numpy(pos).cuda()
    msa.qk_norm_rope(Q, K, Qo, Ko, p if sections else p[0], rope, *(None if x is None else _dev(x) for x in w))
    args = (dim, inv, _axis(sections or (dim // 2,)), inter, 1.25 if inter else 1.0)
    _check(_host(Qo), qk[:, :Hq].transpose(1, 0, 2), pos, args, w[0])
    _check(_host(Ko), qk[:, Hq:].transpose(1, 0, 2), pos, args, w[1])


def test_in_place_and_padded_strides():
    rng = np.random.default_rng(5)
    x = ko.bf16(rng.standard_normal((3, 50, 128)))
    pos = rng.integers(0, 1 << 17, (1, 50)).astype(np.int32)
    buf = torch.full((3, 64, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    view = buf[:, 5:55, 128:]
    view.copy_(_dev(x))
    kbuf = view[:1].clone()
    msa.qk_norm_rope(view, kbuf, view, kbuf, torch.from_numpy(pos[0]).cuda(), msa.Rope())
    inv = [1e6 ** (-2 * i / 128) for i in range(64)]
    _check(_host(view), x, pos, (128, inv, [0] * 64, False, 1.0), None)
    buf[:, 5:55, 128:] = 7.0
    assert (buf == 7.0).all()  # nothing around the rows was written


def test_given_frequencies_and_far_positions():
    """Scaled frequencies (one of zero, one negative, one above a turn per position) at the ends of
    the position range."""
    rng = np.random.default_rng(6)
    inv = [0.0, -0.3, 7.5, 1e-7] + [0.01 * i for i in range(60)]
    pos = np.array([[0, 1, -1, 2 ** 31 - 1, -2 ** 31, 10 ** 9]], np.int32)
    x = ko.bf16(rng.standard_normal((2, 6, 128)))
    q = _dev(x)
    o, ko_ = torch.empty_like(q), torch.empty_like(q[:1])
    msa.qk_norm_rope(q, q[:1], o, ko_, torch.from_numpy(pos).cuda(), msa.Rope(inv_freq=inv))
    # 2^31 positions on a frequency held to 2^-64 turns: 2^-33 turns
    _check(_host(o), x, pos, (128, inv, [0] * 64, False, 1.0), None)


def test_frequencies_of_any_size():
    """Above 2^10 a frequency is held to 2^-53 turns (long double), below 2^-75 it is no turn at all."""
    rng = np.random.default_rng(9)
    inv = [1023.99, 1024.0, -1024.5, 2e5, -6.5, 6.283185307179586, 1e-22, -1e-30, 5e-324, 2.0 ** -1022] + [0.1 * i for i in range(54)]
    pos = np.array([[0, 1, -1, 7, -100, 100]], np.int32)
    q = _dev(ko.bf16(rng.standard_normal((2, 6, 128))))
    o, k = torch.empty_like(q), torch.empty_like(q[:1])
    msa.qk_norm_rope(q, q[:1], o, k, torch.from_numpy(pos).cuda(), msa.Rope(inv_freq=inv))
    _check(_host(o), _host(q), pos, (128, inv, [0] * 64, False, 1.0), None)


def test_positions_of_text_shared_by_the_axes():
    x = torch.randn(3, 17, 128, device="cuda").to(torch.bfloat16)
    pos, rope = torch.arange(100, 117, dtype=torch.int32, device="cuda"), msa.Rope(sections=(16, 24, 24))
    one, three = torch.empty_like(x), torch.empty_like(x)
    msa.qk_norm_rope(x[:2], x[2:], one[:2], one[2:], pos.expand(3, 17), rope)
    msa.qk_norm_rope(x[:2], x[2:], three[:2], three[2:], pos.repeat(3, 1), rope)
    assert torch.equal(one, three)


def test_zero_rows_and_large_values():
    q = torch.zeros(1, 3, 128, dtype=torch.bfloat16, device="cuda")
    q[0, 1] = 2.0 ** 50
    q[0, 2, 0] = float("inf")
    o = torch.empty_like(q)
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    msa.qk_norm_rope(q, q[:0], o, o[:0], pos, msa.Rope(dim=64), w)
    assert (o[0, 0] == 0).all() and (o[0, 1] == 1).all()
    msa.qk_norm_rope(q, q[:0], o, o[:0], pos, msa.Rope(dim=64, interleaved=True))
    assert (o[0, 1] == q[0, 1]).all() and (o[0, 2, 64:] == 0).all()


def test_graph_replay_and_side_stream():
    rng = np.random.default_rng(8)
    x = _dev(rng.standard_normal((6, 40, 128)))
    pos = torch.arange(40, dtype=torch.int32, device="cuda")
    rope, ref, out = msa.Rope(), torch.empty_like(x), torch.empty_like(x)
    msa.qk_norm_rope(x[:4], x[4:], ref[:4], ref[4:], pos, rope)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        msa.qk_norm_rope(x[:4], x[4:], out[:4], out[4:], pos, rope)
    pos += 3
    g.replay()
    moved = torch.empty_like(x)
    msa.qk_norm_rope(x[:4], x[4:], moved[:4], moved[4:], pos, rope)
    assert torch.equal(out, moved) and not torch.equal(out, ref)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    msa.qk_norm_rope(x[:4], x[4:], ref[:4], ref[4:], pos, rope, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(ref, moved)
