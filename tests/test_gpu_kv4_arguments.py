"""Tensors of unusual strides at the calls around the layer."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import dynamic_sparse_attention_head_b200 as msa  # noqa: E402

I32, BF16 = torch.int32, torch.bfloat16


def _odd(x):
    """The same tensor with a stride of 1 along its axes of one, as DLPack hands it over."""
    return x.as_strided(x.shape, [s if n > 1 else 1 for n, s in zip(x.shape, x.stride())], x.storage_offset())


@pytest.mark.parametrize("H,T", [(1, 1), (4, 1), (1, 5), (4, 5)])
def test_strides_of_axes_of_one_are_not_looked_at(H, T):
    g = torch.Generator(device="cuda").manual_seed(H + T)
    q, k, v = (torch.randn(H, T, 128, generator=g, device="cuda").to(BF16) for _ in range(3))
    pos, rope = torch.arange(T, dtype=I32, device="cuda"), msa.Rope()
    cache, slots = msa.KV4Cache.alloc(2, H, 16, 64), torch.arange(T, device="cuda")
    table, lens = torch.zeros(1, 1, dtype=I32, device="cuda"), torch.tensor([T], dtype=I32, device="cuda")
    cu, ws, outs = torch.tensor([0, T], dtype=I32, device="cuda"), cache.alloc_workspace(), []
    for f in (lambda x: x, _odd):
        qo, ko, o, kr, vr = (torch.zeros_like(q) for _ in range(5))
        msa.qk_norm_rope(f(q), f(k), f(qo), f(ko), pos, rope)
        cache.append(f(ko), f(v), slots)
        cache.read(slots, f(kr), f(vr))
        cache.attend(f(qo), f(o), f(table), lens, cu, T, 0.1, ws)
        outs.append((qo, ko, kr, vr, o))
    assert cache.device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(*outs)) and outs[1][4].abs().amin(-1).gt(0).any()


def test_outputs_whose_rows_overlap_are_refused():
    H, T = 3, 4
    x = torch.ones(H, T, 128, dtype=BF16, device="cuda")
    one_head, one_row = x[:1].expand(H, T, 128), x[:, :1].expand(H, T, 128)
    shifted = torch.ones(1000, dtype=BF16, device="cuda").as_strided((H, T, 128), (200, 64, 1))
    pos, rope = torch.arange(T, dtype=I32, device="cuda"), msa.Rope()
    cache, slots = msa.KV4Cache.alloc(2, H, 16, 64), torch.arange(T, device="cuda")
    table, lens = torch.zeros(1, 1, dtype=I32, device="cuda"), torch.tensor([T], dtype=I32, device="cuda")
    cu, ws = torch.tensor([0, T], dtype=I32, device="cuda"), cache.alloc_workspace()
    for y in (one_head, one_row, shifted):
        for call in (lambda: msa.qk_norm_rope(x, x, y, x.clone(), pos, rope), lambda: msa.qk_norm_rope(x, x, x.clone(), y, pos, rope),
                     lambda: cache.read(slots, y, x), lambda: cache.read(slots, x, y),
                     lambda: cache.attend(x, y, table, lens, cu, T, 0.1, ws)):
            with pytest.raises(ValueError, match="overlap"):
                call()
    assert (x == 1).all() and (shifted == 1).all()
    # as inputs they are as good as any other
    out = [torch.empty_like(x) for _ in range(2)]
    cache.append(one_head, one_row, slots)
    cache.attend(one_row, out[0], table, lens, cu, T, 0.1, ws)
    cache.append(x, x, slots)
    cache.attend(x, out[1], table, lens, cu, T, 0.1, ws)
    assert torch.equal(*out) and cache.device_status() == 0


def test_a_norm_alone_needs_no_positions():
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k = (torch.randn(h, 9, 128, generator=g, device="cuda").to(BF16) for h in (3, 2))
    w = [torch.randn(128, generator=g, device="cuda").to(BF16) for _ in range(2)]
    outs = []
    for pos in (torch.arange(9, dtype=I32, device="cuda"), None):
        qo, ko = torch.empty_like(q), torch.empty_like(k)
        msa.qk_norm_rope(q, k, qo, ko, pos, msa.Rope(dim=0), *w)
        outs.append((qo, ko))
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    x = q.double() * torch.rsqrt(q.double().square().mean(-1, keepdim=True) + 1e-6) * w[0].double()
    # one rounding to bf16, and fp32's before it (a sum of 128 squares, rsqrt, two products: below 2^-20)
    assert ((outs[1][0].double() - x).abs() <= x.abs() * (2.0 ** -8 + 2.0 ** -18)).all()
    with pytest.raises(TypeError):
        msa.qk_norm_rope(q, k, *outs[0], None, msa.Rope(dim=16))
