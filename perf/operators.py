"""Workloads of the operators around the sparse prefill of a layer: what makes its queries and keys
(per-head norm and position rotation), and what holds and reads its keys and values afterwards (a paged
4-bit cache: block tables and slot maps, the write, the read back, attention over it).

`run` computes each operator in its plain form (elementary torch operations), or, with `own` true, by the
library's calls.  Tensors follow the library's layout: Q and O [Hq, T, 128], K and V [Hkv, T, 128], bf16.

Cache layout (uint8 [n_pages, Hkv, page_bytes], page_bytes = page * (128 + 8 * NG), NG = 128 / group): blocks of
16 tokens; in a block, for token i:
  K codes   64 * i                     channel x in byte 16 * (x % 32 // 8) + 4 * (x // 32) + x % 8 // 2, low nibble first
  V codes   1024 + 64 * i              channel x in byte 8 * ((x % 32 // 4) ^ (4 * (i // 2 % 2))) + 2 * (x // 32) + x % 4 // 2
  K scales  2048 + 4 * NG * i          per group: bf16 step, bf16 minimum
  V scales  2048 + 64 * NG + 4 * NG * i
The value of a code is minimum + code * step.
"""
import math
import random

import torch

own = False

D = 128
EPS = 1e-6


# ---------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------
def listed():
    return [
        # a decode step's queries and keys, a few dozen requests, one token each: launch latency
        {"name": "norm-rope-decode", "op": "norm_rope", "T": 48, "Hq": 28, "Hkv": 4, "norm": True, "rot": 128, "inter": False,
         "axes": 1, "far": 32768},
        # the 128K video prompt's layer (28 q / 4 kv heads), three position axes (time, height, width)
        {"name": "norm-rope-128k", "op": "norm_rope", "T": 131072, "Hq": 28, "Hkv": 4, "norm": True, "rot": 128, "inter": False,
         "axes": 3, "far": 131072},
        # a decode batch: one token per request, most of them inside their last page
        {"name": "slots-decode", "op": "slots", "B": 256, "kv": 16384, "new": 1, "page": 64},
        # prompts of odd lengths arriving together, some on top of a cached prefix
        {"name": "slots-prompts", "op": "slots", "B": 7, "kv": 5000, "new": 131071, "page": 64},
        # one new token per request of a decode batch, written and read back
        {"name": "append-decode", "op": "append", "T": 64, "Hkv": 4, "page": 64, "group": 64, "runs": 64},
        # the 128K prompt's keys and values, after its prefill
        {"name": "append-128k", "op": "append", "T": 131072, "Hkv": 4, "page": 64, "group": 64, "runs": 1},
        # a cached prefix brought back to bf16 for the prefill of a longer prompt; odd length
        {"name": "read-prefix", "op": "read", "T": 4999, "Hkv": 8, "page": 16, "group": 32, "runs": 3},
        # the largest prefix
        {"name": "read-256k", "op": "read", "T": 262144, "Hkv": 4, "page": 128, "group": 128, "runs": 1},
        # a handful of short contexts, one token each: launch latency
        {"name": "attend-short", "op": "attend", "B": 4, "kv": 700, "q": 1, "Hq": 32, "Hkv": 8, "page": 16, "group": 32},
        # a ragged decode batch (32 q / 8 kv heads)
        {"name": "attend-batch", "op": "attend", "B": 64, "kv": 16384, "q": 1, "Hq": 32, "Hkv": 8, "page": 64, "group": 128},
        # one token over the 1M-token cache (28 q / 4 kv heads)
        {"name": "attend-1m", "op": "attend", "B": 1, "kv": 1048576, "q": 1, "Hq": 28, "Hkv": 4, "page": 64, "group": 64},
        # follow-up prompts over cached contexts, causal among their own tokens
        {"name": "attend-chunk", "op": "attend", "B": 2, "kv": 32768, "q": 601, "Hq": 28, "Hkv": 4, "page": 64, "group": 64},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "slots", "append", "read", "attend", "attend"])
    heads = rng.choice([(28, 4), (32, 8), (16, 16), (12, 1), (8, 2)])
    page, group = rng.choice([16, 32, 64, 128, 256]), rng.choice([32, 64, 128])
    if op == "norm_rope":
        T = _log(rng, 1, 100000)
        rot = rng.choice([128, 128, 64, 32, 96])
        return {"op": op, "T": T, "Hq": heads[0], "Hkv": heads[1], "norm": rng.random() < 0.7, "rot": rot,
                "inter": rng.random() < 0.3, "axes": rng.choice([1, 1, 3]), "far": max(T, rng.choice([4096, 131072, 1048576]))}
    if op == "slots":
        if rng.random() < 0.5:
            return {"op": op, "B": _log(rng, 1, 1024), "kv": _log(rng, 16, 32768), "new": rng.randint(1, 5), "page": page}
        return {"op": op, "B": rng.randint(1, 12), "kv": _log(rng, 16, 8192), "new": _log(rng, 100, 70000), "page": page}
    if op in ("append", "read"):
        T = _log(rng, 1, 60000)
        return {"op": op, "T": T, "Hkv": heads[1], "page": page, "group": group, "runs": rng.randint(1, max(1, min(64, T)))}
    base = {"op": op, "Hq": heads[0], "Hkv": heads[1], "page": page, "group": group}
    if rng.random() < 0.5:  # decode and draft verification
        B = _log(rng, 1, 64)
        return {**base, "B": B, "kv": _log(rng, 16, max(32, min(400000, 1600000 // (B * heads[1])))), "q": rng.choice([1, 1, 1, 2, 5])}
    B = rng.randint(1, 3)  # prompts over a cache, or from its start
    q = _log(rng, 2, 500)
    return {**base, "B": B, "kv": max(q, _log(rng, 64, 24000)), "q": q}


def _lengths(case):
    """(cached + new, new) tokens of each request, from the case alone: the first is the longest."""
    r = random.Random(case["B"] * 1000003 + case["kv"])
    kv, new = [], []
    for b in range(case["B"]):
        n = case["q"] if b == 0 else r.randint(max(1, case["q"] // 2), case["q"])
        new.append(n)
        kv.append(case["kv"] if b == 0 else max(n, int(case["kv"] * r.uniform(0.02, 1.0))))
    return kv, new


def _requests(case):
    """(cached, new) tokens of each request of a slot-map case."""
    r = random.Random(case["B"] * 1000003 + case["kv"])
    have = [r.randint(0, case["kv"]) for _ in range(case["B"])]
    new = [case["new"]] + [r.randint((case["new"] + 1) // 2, case["new"]) for _ in range(case["B"] - 1)]
    return have, new


def _rows(case):
    """Rows of a slot map: `runs` requests that share the tokens."""
    n, k = case["T"], case["runs"]
    return [n // k + (1 if i < n % k else 0) for i in range(k)]


def _page_bytes(case):
    return case["page"] * (128 + 8 * (D // case["group"]))


def _sections(case):
    """Frequencies of each position axis: a quarter for the first, the rest shared."""
    n = case["rot"] // 2
    if case["axes"] == 1:
        return [n]
    a = n // 4
    return [a, (n - a) // 2, n - a - (n - a) // 2]


def work(case):
    op = case["op"]
    if op == "norm_rope":
        n = case["T"] * (case["Hq"] + case["Hkv"]) * D
        return {"bytes": 4 * n + 4 * case["axes"] * case["T"], "flops": 8 * n}
    if op == "slots":
        have, new = _requests(case)
        P = case["page"]
        pages = sum(-(-(h + n) // P) - -(-h // P) for h, n in zip(have, new))
        return {"bytes": 12 * sum(new) + 8 * pages + 16 * case["B"], "flops": 0}
    if op in ("append", "read"):
        row = 2 * (64 + 4 * (D // case["group"]))
        n = case["T"] * case["Hkv"]
        # values in, codes out (append: and back to values, as its result is compared)
        full = n * (512 + row) * (2 if op == "append" else 1)
        return {"bytes": full + 8 * case["T"] * (2 if op == "append" else 1), "flops": 6 * n * D}
    kv, new = _lengths(case)
    row = 2 * (64 + 4 * (D // case["group"]))
    seen = sum(n * (m - n) + n * (n + 1) // 2 for m, n in zip(kv, new))
    t = sum(new) * case["Hq"]
    return {"bytes": sum(kv) * case["Hkv"] * row + t * (4 * D + 4) + 4 * sum(-(-m // case["page"]) for m in kv),
            "flops": 4 * D * case["Hq"] * seen}


# ---------------------------------------------------------------------------------------------------
# the cache's format, in torch
# ---------------------------------------------------------------------------------------------------
def _quantise(x, group):
    """Codes (int64), step and minimum of each group of channels, x bf16 [..., 128]."""
    y = x.float().view(*x.shape[:-1], D // group, group)
    lo, hi = y.amin(-1, keepdim=True), y.amax(-1, keepdim=True)
    step = ((hi - lo) / 15).to(torch.bfloat16).float()
    step = torch.where(step < 2.0 ** -126, torch.zeros_like(step), step)
    r = torch.where(step > 0, 1 / step, torch.zeros_like(step))
    # the product in 64 bits: a value next to a border falls on its own side
    code = torch.round((y - lo).double() * r.double()).clamp(0, 15).long()
    return code.view(x.shape), step.squeeze(-1).to(torch.bfloat16), lo.squeeze(-1).to(torch.bfloat16)


def _places(i, device):
    """Byte of each channel among a token's K and V codes, [..., 128]; i: the token's place in its block of 16."""
    x = torch.arange(D, device=device)
    k = 16 * (x % 32 // 8) + 4 * (x // 32) + x % 8 // 2
    v = 8 * ((x % 32 // 4) ^ (4 * (i[..., None] // 2 % 2))) + 2 * (x // 32) + x % 4 // 2
    return k.expand_as(v), v


def _nibbles(code, place):
    """64 bytes of a token from its 128 codes: the even channel of a pair is the low nibble."""
    both = (code[..., 0::2] | (code[..., 1::2] << 4)).to(torch.uint8)
    return torch.zeros_like(both).scatter(-1, place[..., 0::2], both)


def _store(pages, case, slots, K, V):
    """Quantises K and V [Hkv, T, 128] into the pages (in place)."""
    P, ng = case["page"], D // case["group"]
    page, r = slots // P, slots % P
    at, i = (r // 16) * (16 * (128 + 8 * ng)), r % 16
    kp, vp = _places(i, slots.device)
    cols = torch.arange(64, device=slots.device)
    sm = torch.arange(4 * ng, device=slots.device)
    for base, stride, x, place, scale_base in ((0, 64, K, kp, 2048), (1024, 64, V, vp, 2048 + 64 * ng)):
        code, step, lo = _quantise(x.transpose(0, 1), case["group"])  # [T, Hkv, ...]
        data = _nibbles(code, place[:, None, :].expand_as(code))
        h = torch.arange(x.shape[0], device=slots.device)
        pages[page[:, None, None], h[None, :, None], (at + base + stride * i)[:, None, None] + cols] = data
        scales = torch.stack((step, lo), -1).contiguous().view(torch.uint8).view(*step.shape[:-1], 4 * ng)
        pages[page[:, None, None], h[None, :, None], (at + scale_base + 4 * ng * i)[:, None, None] + sm] = scales


def _load(pages, case, slots):
    """K and V in 32 bits, [T, Hkv, 128], of the tokens at `slots`."""
    P, group = case["page"], case["group"]
    ng = D // group
    blocks = pages.view(pages.shape[0], pages.shape[1], P // 16, 16 * (128 + 8 * ng))
    page, r = slots // P, slots % P
    got = blocks[page, :, r // 16]  # [T, Hkv, block]
    i = (r % 16)[:, None, None]
    kp, vp = _places(r % 16, slots.device)
    odd = (torch.arange(D, device=slots.device) % 2 * 4).to(torch.uint8)
    out = []
    for base, place, scale_base in ((0, kp, 2048), (1024, vp, 2048 + 64 * ng)):
        byte = got.gather(-1, (base + 64 * i + place[:, None, :]).expand(got.shape[0], got.shape[1], D))
        code = ((byte >> odd) & 15).float()
        sm = got.gather(-1, (scale_base + 4 * ng * i + torch.arange(4 * ng, device=slots.device)).expand(got.shape[0], got.shape[1], 4 * ng))
        sm = sm.contiguous().view(torch.bfloat16).view(got.shape[0], got.shape[1], ng, 2).float()
        step, lo = (sm[..., k].repeat_interleave(group, -1) for k in (0, 1))
        out.append(lo + code * step)
    return out


def _unpacked(pages, case):
    """K and V in 32 bits of every token of the given pages [..., Hkv, page_bytes] -> [..., Hkv, page, 128]."""
    P, group = case["page"], case["group"]
    ng = D // group
    b = pages.unflatten(-1, (P // 16, 16 * (128 + 8 * ng)))
    i = torch.arange(16, device=pages.device)
    kp, vp = _places(i, pages.device)
    odd = (torch.arange(D, device=pages.device) % 2 * 4).to(torch.uint8)
    out = []
    for base, place, scale_base in ((0, kp, 2048), (1024, vp, 2048 + 64 * ng)):
        byte = b[..., (base + 64 * i[:, None] + place).flatten()].unflatten(-1, (16, D))
        code = ((byte >> odd) & 15).float()
        sm = b[..., scale_base:scale_base + 64 * ng].contiguous().view(torch.bfloat16).unflatten(-1, (16, ng, 2)).float()
        code = code.unflatten(-1, (ng, group))
        out.append((sm[..., 1:2] + code * sm[..., 0:1]).flatten(-2).flatten(-3, -2))
    return out


# ---------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------
def _normal(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def _keys(g, H, T):
    """Keys and values as a model has them: a few key channels carry an offset, rows differ in size."""
    off = torch.randn(H, 1, D, generator=g, device="cuda") * (torch.rand(H, 1, D, generator=g, device="cuda") < 0.05) * 4
    K = (torch.randn(H, T, D, generator=g, device="cuda") + off).to(torch.bfloat16)
    V = (torch.randn(H, T, D, generator=g, device="cuda") * torch.empty(H, T, 1, device="cuda").uniform_(0.5, 2.0, generator=g)).to(torch.bfloat16)
    return K, V


def _rope_tables(case):
    n = case["rot"] // 2
    return [1e6 ** (-i / n) for i in range(n)]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    s = {"case": case}
    if own:
        import dynamic_sparse_attention_head_b200 as msa
        s["msa"] = msa
    if op == "norm_rope":
        T, Hq, Hkv = case["T"], case["Hq"], case["Hkv"]
        # the projection's output, token by token: [T, Hq + Hkv, 128]
        qk = _normal(g, T, Hq + Hkv, D, scale=3.0)
        s["Q"], s["K"] = qk[:, :Hq].transpose(0, 1), qk[:, Hq:].transpose(0, 1)
        s["pos"] = torch.randint(0, case["far"], (case["axes"], T), generator=g, device="cuda", dtype=torch.int32)
        s["wq"], s["wk"] = ((1 + _normal(g, D, scale=0.2).float()).to(torch.bfloat16) if case["norm"] else None for _ in range(2))
        s["Qo"], s["Ko"] = (torch.zeros(h, T, D, dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv))
        s["inv_freq"] = torch.tensor(_rope_tables(case), dtype=torch.float64, device="cuda")
        s["axis"] = torch.tensor([a for a, n in enumerate(_sections(case)) for _ in range(n)], device="cuda")
        if own:
            s["rope"] = s["msa"].Rope(dim=case["rot"], inv_freq=_rope_tables(case), interleaved=case["inter"],
                                      sections=_sections(case) if case["axes"] > 1 else None)
        return s
    if op == "slots":
        have, new = _requests(case)
        P, B = case["page"], case["B"]
        blocks = max(-(-(h + n) // P) for h, n in zip(have, new)) + 3
        used = sum(-(-h // P) for h in have)
        pages = used + sum(-(-n // P) + 1 for n in new) + 17
        perm = torch.randperm(pages, generator=g, device="cuda", dtype=torch.int32)
        table = torch.full((B, blocks), -1, dtype=torch.int32)
        order, at = perm.cpu(), 0
        for b, h in enumerate(have):
            n = -(-h // P)
            table[b, :n] = order[at:at + n]
            at += n
        s["kv"], s["new"] = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (have, new))
        s["table"], s["free"] = table.cuda(), torch.cat((perm[used:], perm.new_zeros(used)))
        s["n_free"] = torch.tensor([pages - used], dtype=torch.int32, device="cuda")
        s["kv_out"], s["n_free_out"] = torch.zeros_like(s["kv"]), torch.zeros_like(s["n_free"])
        s["cu"] = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
        s["slots"] = torch.zeros(sum(new), dtype=torch.int64, device="cuda")
        s["pos"] = torch.zeros(sum(new), dtype=torch.int32, device="cuda")
        if own:
            s["cache"] = s["msa"].KV4Cache(torch.zeros(pages, 1, P * 136, dtype=torch.uint8, device="cuda"), page=P, group=128)
        return s
    P, H = case["page"], case["Hkv"]
    if op in ("append", "read"):
        T = case["T"]
        rows = _rows(case)
        per = [-(-n // P) + 1 for n in rows]
        pages = sum(per) + 3
        perm = torch.randperm(pages, generator=g, device="cuda")
        r = random.Random(seed)
        slots, at = [], 0
        for n, p in zip(rows, per):
            t = torch.arange(n, device="cuda") + r.randint(0, P - 1)  # a request goes on inside a page
            slots.append(perm[at + t // P] * P + t % P)
            at += p
        s["slots"] = torch.cat(slots)
        s["pages"] = torch.zeros(pages, H, _page_bytes(case), dtype=torch.uint8, device="cuda")
        s["K"], s["V"] = _keys(g, H, T)
        if op == "read":
            _store(s["pages"], case, s["slots"], s["K"], s["V"])
        s["Ko"], s["Vo"] = torch.zeros_like(s["K"]), torch.zeros_like(s["V"])
    else:
        kv, new = _lengths(case)
        per = [-(-m // P) for m in kv]
        pages = sum(per) + 3
        perm = torch.randperm(pages, generator=g, device="cuda")
        table = torch.full((case["B"], max(per) + 1), -1, dtype=torch.int32, device="cuda")
        s["pages"] = torch.zeros(pages, H, _page_bytes(case), dtype=torch.uint8, device="cuda")
        at = 0
        for b, m in enumerate(kv):
            mine = perm[at:at + per[b]]
            table[b, :per[b]] = mine.int()
            at += per[b]
            for t0 in range(0, m, 131072):
                t = torch.arange(t0, min(m, t0 + 131072), device="cuda")
                K, V = _keys(g, H, t.numel())
                _store(s["pages"], case, mine[t // P] * P + t % P, K, V)
        s["table"] = table
        s["kv"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        s["max_q"], s["scale"] = max(new), 1 / math.sqrt(D)
        s["Q"] = _normal(g, case["Hq"], cu[-1], D)
        s["O"] = torch.zeros_like(s["Q"])
        s["lse"] = torch.zeros(case["Hq"], cu[-1], dtype=torch.float32, device="cuda")
    if own:
        s["cache"] = s["msa"].KV4Cache(s["pages"], page=P, group=case["group"])
        if op == "attend":
            s["ws"] = s["cache"].alloc_workspace(case["Hq"])
    return s


# ---------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        return {"norm_rope": _own_norm_rope, "slots": _own_slots, "append": _own_append, "read": _own_read, "attend": _own_attend}[op](s)
    return {"norm_rope": _norm_rope, "slots": _slots, "append": _append, "read": _read, "attend": _attend}[op](s)


def _own_norm_rope(s):
    s["msa"].qk_norm_rope(s["Q"], s["K"], s["Qo"], s["Ko"], s["pos"], s["rope"], wq=s["wq"], wk=s["wk"], eps=EPS)
    return {"Q": s["Qo"], "K": s["Ko"]}


def _own_slots(s):
    s["cache"].slots(s["kv"], s["new"], s["table"], s["free"], s["n_free"], s["slots"], s["pos"], s["cu"], kv_lens_out=s["kv_out"],
                     n_free_out=s["n_free_out"])
    return {"table": s["table"], "kv": s["kv_out"], "n_free": s["n_free_out"], "cu": s["cu"], "slots": s["slots"], "pos": s["pos"]}


def _own_append(s):
    s["cache"].append(s["K"], s["V"], s["slots"])
    s["cache"].read(s["slots"], s["Ko"], s["Vo"])
    return {"K": s["Ko"], "V": s["Vo"]}


def _own_read(s):
    s["cache"].read(s["slots"], s["Ko"], s["Vo"])
    return {"K": s["Ko"], "V": s["Vo"]}


def _own_attend(s):
    s["cache"].attend(s["Q"], s["O"], s["table"], s["kv"], s["cu"], s["max_q"], s["scale"], s["ws"], lse=s["lse"])
    return {"O": s["O"], "lse": s["lse"]}


def _norm_rope(s):
    case = s["case"]
    rot = case["rot"]
    angle = s["pos"].double()[s["axis"]].transpose(0, 1) * s["inv_freq"]  # [T, rot / 2]
    c, n = angle.cos().float(), angle.sin().float()

    def one(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
        r = x[..., :rot]
        if case["inter"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack((a * c - b * n, b * c + a * n), -1).flatten(-2)
        else:
            a, b = r[..., :rot // 2], r[..., rot // 2:]
            r = torch.cat((a * c - b * n, b * c + a * n), -1)
        return torch.cat((r, x[..., rot:]), -1).to(torch.bfloat16)

    return {"Q": one(s["Q"], s["wq"]), "K": one(s["K"], s["wk"])}


def _slots(s):
    P = s["case"]["page"]
    kv, new, table, free = s["kv"].long(), s["new"].long(), s["table"].clone(), s["free"]
    after = kv + new
    have, need = (kv + P - 1) // P, (after + P - 1) // P
    cu = torch.nn.functional.pad(new.cumsum(0), (1, 0))
    taken = (need - have).cumsum(0)
    first = taken - (need - have)
    # every block of the table: an old page, or the next one from the top of the stack
    block = torch.arange(table.shape[1], device=kv.device)[None, :]
    fresh = (block >= have[:, None]) & (block < need[:, None])
    at = s["n_free"].long() - 1 - (first[:, None] + block - have[:, None])
    table = torch.where(fresh, free[at.clamp(0, free.numel() - 1)], table)
    token = torch.arange(s["slots"].numel(), device=kv.device)
    b = torch.searchsorted(cu, token, right=True) - 1
    pos = kv[b] + token - cu[b]
    slots = table[b, pos // P].long() * P + pos % P
    return {"table": table, "kv": after.int(), "n_free": s["n_free"] - taken[-1:].int(), "cu": cu.int(), "slots": slots, "pos": pos.int()}


def _append(s):
    _store(s["pages"], s["case"], s["slots"], s["K"], s["V"])
    return _read(s)


def _read(s):
    K, V = _load(s["pages"], s["case"], s["slots"])
    return {"K": K.transpose(0, 1).to(torch.bfloat16).contiguous(), "V": V.transpose(0, 1).to(torch.bfloat16).contiguous()}


def _attend(s):
    case = s["case"]
    B, Hq, Hkv, P = case["B"], case["Hq"], case["Hkv"], case["page"]
    G, q = Hq // Hkv, s["max_q"]
    cu, kv = s["cu"].long(), s["kv"].long()
    new = cu[1:] - cu[:-1]
    K, V = _unpacked(s["pages"][s["table"].long().clamp(min=0)], case)  # [B, blocks, Hkv, P, 128]
    K, V = (x.transpose(1, 2).flatten(2, 3) for x in (K, V))  # [B, Hkv, blocks * P, 128]
    i = torch.arange(q, device=cu.device)
    row = (cu[:-1, None] + i).clamp(max=s["Q"].shape[1] - 1)  # [B, q]
    Q = s["Q"].float()[:, row].view(Hkv, G, B, q, D).permute(2, 0, 1, 3, 4).reshape(B, Hkv, G * q, D)
    S = (Q @ K.transpose(-1, -2)).view(B, Hkv, G, q, -1) * s["scale"]
    j = torch.arange(K.shape[2], device=cu.device)
    seen = (j <= (kv - new)[:, None, None] + i[:, None]) & (j < kv[:, None, None])  # [B, q, keys]
    S = S.masked_fill(~seen[:, None, None], -math.inf)
    m = S.amax(-1, keepdim=True)
    S = (S - m).exp()
    l = S.sum(-1, keepdim=True)
    O = (S.view(B, Hkv, G * q, -1) @ V).view(B, Hkv, G, q, D) / l
    lse = (m + l.log()).squeeze(-1)
    at = torch.arange(s["Q"].shape[1], device=cu.device)
    b = torch.searchsorted(cu, at, right=True) - 1
    i = at - cu[b]
    O = O.permute(0, 3, 1, 2, 4)[b, i].flatten(1, 2)  # [T, Hq, 128]
    lse = lse.permute(0, 3, 1, 2)[b, i].flatten(1, 2)
    return {"O": O.transpose(0, 1).to(torch.bfloat16).contiguous(), "lse": lse.transpose(0, 1).contiguous()}


# ---------------------------------------------------------------------------------------------------
# the operators' definitions in 64 bits
# ---------------------------------------------------------------------------------------------------
def _decode64(pages, case, slots):
    """K and V [Hkv, T, 128] in 64 bits, byte by byte from the format's definition."""
    P, group = case["page"], case["group"]
    ng = D // group
    flat = pages.transpose(0, 1).flatten(1)  # [Hkv, n_pages * page_bytes]
    start = slots // P * pages.shape[2] + slots % P // 16 * (2048 + 128 * ng)
    i = slots % 16
    x = torch.arange(D, device=slots.device)
    k_at = start[:, None] + 64 * i[:, None] + (x % 32 // 8) * 16 + (x // 32) * 4 + (x % 8) // 2
    v_at = start[:, None] + 1024 + 64 * i[:, None] + ((x % 32 // 4)[None, :] ^ ((i // 2 % 2) * 4)[:, None]) * 8 + (x // 32) * 2 + (x % 4) // 2
    res = []
    for at, sb in ((k_at, 2048), (v_at, 2048 + 64 * ng)):
        c = flat[:, at]
        c = torch.where(x % 2 == 1, c // 16, c % 16).double()
        sat = (start + sb + 4 * ng * i)[:, None] + (x // group) * 4
        half = lambda a: ((flat[:, a].int() | (flat[:, a + 1].int() << 8)) << 16).view(torch.float32).double()  # noqa: E731
        res.append(half(sat + 2) + c * half(sat))
    return res


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op == "norm_rope":
        rot, n = case["rot"], case["rot"] // 2
        dev = s["pos"].device
        x = torch.arange(rot, device=dev)
        freq = x // 2 if case["inter"] else x % n
        other = x ^ 1 if case["inter"] else (x + n) % rot
        sign = torch.where((x % 2 == 0) if case["inter"] else (x < n), -1.0, 1.0).double()
        ang = s["pos"].double().gather(0, s["axis"][:, None].expand(n, case["T"])).T * s["inv_freq"]
        out = {}
        for name in ("Q", "K"):
            v, w = s[name].double(), s["w" + name.lower()]
            if w is not None:
                v = v / torch.sqrt(v.square().sum(-1, keepdim=True) / D + EPS) * w.double()
            r = v[..., :rot] * torch.cos(ang)[:, freq] + sign * v[..., other] * torch.sin(ang)[:, freq]
            out[name] = torch.cat((r, v[..., rot:]), -1)
        return out
    if op == "slots":
        return None  # whole numbers
    if op == "read":
        K, V = _decode64(s["pages"], case, s["slots"])
        return {"K": K, "V": V}
    if op == "append":
        out = {}
        for name in ("K", "V"):
            x = s[name].double().unflatten(-1, (D // case["group"], case["group"]))
            lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
            step = ((hi - lo).float() / 15).bfloat16().double()  # the step and its reciprocal are stored and used rounded
            r = (1 / step.float()).double()
            c = torch.where(step > 0, torch.round((x - lo).float().double() * r), 0.0).clamp(max=15)
            out[name] = (lo + c * step).flatten(-2)
        return out
    kv, new = _lengths(case)
    G = case["Hq"] // case["Hkv"]
    O = torch.empty(s["Q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["lse"].shape, dtype=torch.float64, device="cuda")
    for b in range(case["B"]):
        t = torch.arange(kv[b], device="cuda")
        K, V = _decode64(s["pages"], case, s["table"][b].long()[t // case["page"]] * case["page"] + t % case["page"])
        q0 = int(s["cu"][b])
        for h in range(case["Hq"]):
            for i0 in range(0, new[b], 512):
                i = torch.arange(i0, min(new[b], i0 + 512), device="cuda")
                S = s["Q"][h, q0 + i].double() @ K[h // G].T * s["scale"]
                S = torch.where(t[None, :] <= (kv[b] - new[b] + i)[:, None], S, -math.inf)
                lse[h, q0 + i] = torch.logsumexp(S, -1)
                O[h, q0 + i] = torch.softmax(S, -1) @ V[h // G]
    return {"O": O, "lse": lse}
