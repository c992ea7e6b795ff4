"""Attention over the 4-bit cache where few of the keys, or few of the values, outweigh the others: both kernels
against 64 bits, with bounds relative to the magnitudes that a row itself weighs."""
import numpy as np
import pytest

import kv4_oracle as ko

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import dynamic_sparse_attention_head_b200 as msa  # noqa: E402

I32 = torch.int32
MANY = 1 << 20  # a hint that takes the kernel for many rows; 1: the one for few


def _bf16(x):
    return torch.as_tensor(x, dtype=torch.float32).to(torch.bfloat16).cuda()


def _filled(K, V, page, group):
    """A cache of one request whose pages lie in another order, and its table."""
    Hkv, n = K.shape[:2]
    pages = -(-n // page)
    cache = msa.KV4Cache.alloc(pages + 2, Hkv, page, group)
    cache.pages.fill_(0xFF)  # NaN scales until a row is written
    table = torch.randperm(pages + 2, generator=torch.Generator().manual_seed(n))[:pages].cuda()
    j = torch.arange(n, device="cuda")
    cache.append(K, V, table[j // page] * page + j % page)
    return cache, table.to(I32)[None]


def _values(x, group):
    """What the cache stands for, in 64 bits, from the format's definition: values, minima and steps a channel."""
    code, step, lo = ko.quantise(x.double().cpu().numpy(), group)
    step, lo = (np.repeat(a, group, -1) for a in (step, lo))
    return [torch.from_numpy(a).cuda() for a in (lo + code * step, lo, step)]


def _compare(cache, table, K, V, Q, scale, max_q, v_error, lost, B=200):
    """K, V [1, kv, 128], Q [H, n, 128]; the last n keys are the queries' own.  B requests hold the same keys and ask the
    same: with more of them than SMs a CTA walks over whole contexts, and what it sums up is not cut into short pieces.  What a kernel may be off by, with p the
    weights and m the largest of them (the sums are over a row's keys):
      scores: ko.tolerance's bound of fp32 sums (136 of them, 2^-24 each) times the largest sum of magnitudes behind a key
        that weighs anything: a relative error of every weight, twice (numerator and denominator), with the exponential's
        2^-21 and the sums' n / 2 * 2^-24.  The many-row kernel's key operands are exact: a key's steps are within 2^4 of
        one another here;
      weights: in fp16, 2^-11 relative; what all of them lose absolutely, times their values, is `lost` of m;
      values: v_error[j], of every value of key j, and 2^-11 relative;
      O: rounded to bf16, 2^-8."""
    kv, n = K.shape[1], Q.shape[1]
    (k, kl, ks), (v, vl, vs) = (_values(x, cache.group) for x in (K, V))
    q = Q.double()
    s = q @ k[0].T * scale
    see = torch.arange(kv, device="cuda")[None] <= kv - n + torch.arange(n, device="cuda")[:, None]
    s = s.masked_fill(~see, float("-inf"))
    p = torch.softmax(s, -1)
    assert ((ks == 0) | (ks * 16 >= ks.amax(-1, keepdim=True))).all()
    reach = (q.abs() @ (kl.abs() + 15 * ks)[0].T).masked_fill(p == 0, 0).amax(-1, keepdim=True) * scale
    ds = reach * 2.0 ** -16 + 2.0 ** -21 + (kv / 2 + 32) * 2.0 ** -24
    mag = v.abs()[0] if max_q == MANY else ((vl + 8 * vs).abs() + 8 * vs)[0]  # few rows: codes less 8 beside lo + 8 step
    O = p @ v[0]
    # the largest weight is at least 1 / (weights' sum): p's own scale
    bound = O.abs() * 2.0 ** -8 + (p @ mag) * (2.0 ** -10 + 2 * ds) + (p @ v_error)[..., None] + \
        lost * p.amax(-1, keepdim=True)
    qs = Q.repeat(1, B, 1)
    o, lse = torch.zeros_like(qs), torch.zeros(qs.shape[:2], device="cuda")
    cache.attend(qs, o, table.repeat(B, 1), torch.full((B,), kv, dtype=I32, device="cuda"),
                 torch.arange(0, B * n + 1, n, dtype=I32, device="cuda"), max_q, scale, cache.alloc_workspace(), lse=lse)
    assert cache.device_status() == 0
    O, bound, ds = O.repeat(1, B, 1), bound.repeat(1, B, 1), ds.repeat(1, B, 1)
    err = (o.double() - O).abs()
    assert (err <= bound).all(), f"{float((err / bound).max()):.2f} of the bound, off by {float(err.norm() / O.norm()):.2e}"
    ref = torch.logsumexp(s, -1).repeat(1, B)
    assert ((lse.double() - ref).abs() <= ds[..., 0] + 2.0 ** -21 * ref.abs().clamp(min=1)).all()
    return o, O


@pytest.mark.parametrize("max_q", [1, MANY])
@pytest.mark.parametrize("kv,gap,at", [(32768, 17.0, 0), (32768, 18.0, 0), (100003, 18.0, 0), (40000, 17.5, 30011)])
def test_keys_far_below_a_sink_still_weigh(kv, gap, at, max_q):
    """One key whose value is zero lies `gap` above the scores of all others, which are N(0, 1): what they add up to is
    the whole of O, though each of them weighs 2^-25 of the largest and less.  Weights keep 2^-32 of the largest: fp16's
    smallest step is 2^-24, half of it is lost, and the largest weight is 2^7 (in the few-row kernel the factor is the
    values' step, within 2 of its power of two).  The values are of one size, 2^-18 of the largest at most lost."""
    g = torch.Generator(device="cuda").manual_seed(kv)
    q = torch.randn(128, generator=g, device="cuda")
    Q = q[None, None].expand(2, 5, 128).to(torch.bfloat16).contiguous()
    K = torch.randn(1, kv, 128, generator=g, device="cuda")
    V = 1 + 0.5 * torch.randn(1, kv, 128, generator=g, device="cuda")
    scale = float(1 / q.norm())
    K[0, at] = Q[0, 0].float() * (gap / (scale * float((Q[0, 0].float() * q).sum())))
    V[0, at] = 0
    K, V = K.to(torch.bfloat16), V.to(torch.bfloat16)
    cache, table = _filled(K, V, 64, 64)
    size = float(V.abs().max())
    own = torch.full((kv,), 2.0 ** -18 * size, dtype=torch.float64, device="cuda")
    own[at] = 0  # zero is exact
    # few rows: codes less 8 beside lo + 8 step, whose magnitudes add up to less than three of the values'
    o, O = _compare(cache, table, K, V, Q, scale, max_q, own, kv * 2.0 ** -32 * size * (1 if max_q == MANY else 6))
    # the roundings of 32768 weights and more average out: of the norm, O's own is left
    assert float((o.double() - O).norm() / O.norm()) < 2.0 ** -8 + 2.0 ** -10


def _losses(V, max_q):
    size = V.double().abs()[0].amax(-1)
    usual, kv = float(size.median() * 2), size.numel()
    lost = kv * 2.0 ** -28 * usual + 128 * 2.0 ** -32 * float(size.max()) if max_q == MANY else kv * 2.0 ** -31 * float(size.max())
    return size * 2.0 ** -12, lost


@pytest.mark.parametrize("max_q", [1, MANY])
@pytest.mark.parametrize("far", [2.0 ** 12, 2.0 ** 20, 2.0 ** -20])
@pytest.mark.parametrize("at,group", [(0, 64), (777, 128), (1000, 32), (2999, 64)])
def test_a_value_of_another_size_leaves_the_others_as_they_are(at, group, far, max_q):
    """One token's values are `far` times the others'; no row weighs it (its score is 28 nats below zero, or it is the
    last key, which only the last row sees), or nearly.  Values keep their own precision: fp16's 11 bits of each, or half
    a subnormal step, 2^-25; a key's largest value is scaled to 2^-13 at least, so 2^-12 of that (few rows: fp32).  The
    weights of the 128 keys in the outlier's own tile are scaled down with it and lose 2^-32 of it, all others 2^-32 of the
    power of two in force, at most 2^4 above their own values (few rows: all lose it of the outlier, and twice)."""
    kv = 3000
    g = torch.Generator(device="cuda").manual_seed(at)
    Q = torch.randn(2, 5, 128, generator=g, device="cuda")
    K = torch.randn(1, kv, 128, generator=g, device="cuda")
    V = torch.randn(1, kv, 128, generator=g, device="cuda")
    Q[..., 0], K[..., 0] = 4.0, 0.0
    K[0, at], V[0, at] = 0.0, far * (1 + torch.rand(128, generator=g, device="cuda"))
    K[0, at, 0] = -20.0
    Q, K, V = (x.to(torch.bfloat16) for x in (Q, K, V))
    cache, table = _filled(K, V, 64, group)
    _compare(cache, table, K, V, Q, 0.35, max_q, *_losses(V, max_q))


@pytest.mark.parametrize("max_q", [1, MANY])
@pytest.mark.parametrize("far", [2.0 ** 12, 2.0 ** 20, 2.0 ** -20])
@pytest.mark.parametrize("at,group", [(0, 64), (777, 128), (1000, 32), (2999, 64)])
def test_a_key_of_another_size_leaves_the_others_as_they_are(at, group, far, max_q):
    """One key is `far` times the others and weighs nothing (its score is below -28 far; the last key is seen by the last
    row alone), or it is as small and weighs as much as a key of zeros.  The others' scores keep fp32's precision."""
    kv = 3000
    g = torch.Generator(device="cuda").manual_seed(at + 1)
    Q = torch.randn(2, 5, 128, generator=g, device="cuda")
    K = torch.randn(1, kv, 128, generator=g, device="cuda")
    V = torch.randn(1, kv, 128, generator=g, device="cuda")
    Q[..., 0], K[0, at, 0] = 4.0, -40.0
    K[0, at] *= far
    Q, K, V = (x.to(torch.bfloat16) for x in (Q, K, V))
    cache, table = _filled(K, V, 64, group)
    _compare(cache, table, K, V, Q, 0.35, max_q, *_losses(V, max_q))


def test_nan_values_reach_the_second_stream_before_pairs_without_one():
    """Pairs of more than 128 rows, whose last keys hold a NaN value group, followed by many of at most 128 rows, which
    leave the second stream of rows without work: what the first pair's rows still read is not reused."""
    kv, group, page, B = 300, 64, 64, 1000
    K, V = (torch.randn(1, kv, 128, generator=torch.Generator().manual_seed(i)).to(torch.bfloat16).cuda() for i in (1, 2))
    V[0, kv - 60, 70] = float("nan")
    cache, table = _filled(K, V, page, group)
    new = torch.tensor(([200] + [100] * 5 + [129] + [1] * 4) * 100, dtype=I32)[:B]
    cu = torch.cat((torch.zeros(1, dtype=I32), new.cumsum(0).int())).cuda()
    T = int(cu[-1])
    Q = torch.randn(1, T, 128, device="cuda").to(torch.bfloat16)
    O, lse = torch.zeros_like(Q), torch.zeros(1, T, device="cuda")
    cache.attend(Q, O, table.repeat(B, 1), torch.full((B,), kv, dtype=I32, device="cuda"), cu, MANY, 0.1, cache.alloc_workspace(), lse=lse)
    assert cache.device_status() == 0
    b = torch.repeat_interleave(torch.arange(B), new.long()).cuda()
    pos = kv - new.cuda()[b] + torch.arange(T, device="cuda") - cu[b]  # a row's own key
    sees = pos >= kv - 60
    assert torch.equal(torch.isnan(O[0, :, 64:]), sees[:, None].expand(T, 64))
    assert torch.isfinite(O[0, :, :64]).all() and torch.isfinite(lse).all()
