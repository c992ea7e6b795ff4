"""A batch of single tokens, drafts and a long prompt in one call of the attention over the 4-bit cache, against 64 bits
and against a call for each kind."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import dynamic_sparse_attention_head_b200 as msa  # noqa: E402
from test_gpu_kv4 import _torch_attend  # noqa: E402

I32 = torch.int32


@pytest.mark.parametrize("Hq,Hkv,page,group", [(8, 2, 64, 64), (28, 4, 16, 128), (4, 4, 256, 32)])
def test_single_tokens_drafts_and_a_prompt_in_one_call(Hq, Hkv, page, group):
    """Inputs of unit size; the bounds are those of test_attention_over_long_contexts_split_over_the_gpu, twice where two
    calls are compared."""
    rng = np.random.default_rng(Hq)
    kv = rng.integers(1, 9000, 24)
    new = rng.choice([1, 1, 1, 3, 8], 24)
    kv[7], new[7] = 5001, 301  # the prompt, among the others
    kv[3], new[11] = 20, 0
    kv = np.maximum(kv, new)
    need = -(-kv // page)
    g = torch.Generator(device="cuda").manual_seed(Hq)
    cache = msa.KV4Cache.alloc(int(need.sum()) + 1, Hkv, page, group)
    cache.pages.fill_(0xFF)
    perm, at = rng.permutation(int(need.sum()) + 1), 0
    table = np.full((24, int(need.max())), -1)
    for b in range(24):
        table[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
        j = torch.arange(int(kv[b]), device="cuda")
        x = torch.randn(2, Hkv, int(kv[b]), 128, generator=g, device="cuda").to(torch.bfloat16)
        cache.append(x[0], x[1], torch.tensor(table[b], device="cuda")[j // page] * page + j % page)
    cu = np.concatenate(([0], np.cumsum(new)))
    Q = torch.randn(Hq, int(cu[-1]), 128, generator=g, device="cuda").to(torch.bfloat16)
    ws = cache.alloc_workspace()

    def attend(rows, most):
        """The requests `rows` in a call of their own, their outputs where they belong."""
        cols = np.concatenate([np.arange(cu[b], cu[b + 1]) for b in rows])
        q = Q[:, cols].contiguous()
        o, lse = torch.zeros_like(q), torch.zeros(Hq, len(cols), device="cuda")
        own = torch.tensor(np.concatenate(([0], np.cumsum(new[rows]))), dtype=I32, device="cuda")
        cache.attend(q, o, torch.tensor(table[rows], dtype=I32, device="cuda"), torch.tensor(kv[rows], dtype=I32, device="cuda"), own,
                     most, 0.088, ws, lse=lse)
        return cols, o, lse

    O, L = _torch_attend(cache, Q, table, kv.tolist(), cu.tolist(), 0.088)
    _, o, lse = attend(np.arange(24), 301)
    assert cache.device_status() == 0
    bound = O.abs() * 2.0 ** -8 + 8 * 2.0 ** -10
    assert ((o.double() - O).abs() <= bound).all() and float((lse.double() - L).abs().max()) < 2.5e-4
    for rows, most in ((np.array([7]), 301), (np.delete(np.arange(24), 7), 8)):
        cols, part, plse = attend(rows, most)
        assert ((part.double() - o[:, cols].double()).abs() <= 2 * bound[:, cols]).all()
        assert float((plse - lse[:, cols]).abs().max()) < 5e-4
    assert cache.device_status() == 0
