"""Plain 64-bit forms of the operators around the layer (per-head norm and rotation, slot maps, the 4-bit
cache's format, attention over it), in numpy, for the tests.  bf16 arrays are float64 arrays whose
values bf16 holds; `bf16` rounds to them."""
import numpy as np

D = 128


def bf16(x):
    """Rounds to bf16 (nearest even), as float64; the argument is rounded to float32 first, as the
    format's definition does."""
    u = np.ascontiguousarray(np.asarray(x, np.float32)).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7fff + ((u >> 16) & 1)) >> 16).astype(np.uint32)
    r = np.where((u & 0x7fffffff) > 0x7f800000, 0x7fc0, r).astype(np.uint32)
    return (r << 16).view(np.float32).astype(np.float64)


def bits(x):
    """bf16 bit patterns (uint16) of float64 values that bf16 holds."""
    return (np.asarray(x, np.float32).view(np.uint32) >> 16).astype(np.uint16)


# ---- norm and rotation ---------------------------------------------------------------------------
def norm_rope(x, pos, inv_freq, axis, dim, interleaved, w, eps, scale):
    """x [H, T, 128]; pos [axes, T]; returns the values and the sum of magnitudes behind each."""
    x = np.asarray(x, np.float64)
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    out, mag = x.copy(), np.abs(x)
    for i in range(dim // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + dim // 2)
        # the angle modulo one turn in long double: positions reach 2^31
        f = np.fmod(pos[axis[i]].astype(np.longdouble) * np.longdouble(inv_freq[i]), 2 * np.longdouble(
            "3.14159265358979323846264338327950288"))
        c, s = np.cos(f).astype(np.float64) * scale, np.sin(f).astype(np.float64) * scale
        out[..., a] = x[..., a] * c - x[..., b] * s
        out[..., b] = x[..., b] * c + x[..., a] * s
        mag[..., a] = mag[..., b] = (np.abs(x[..., a]) + np.abs(x[..., b])) * max(1.0, abs(scale))
    return out, mag


# ---- slot maps -----------------------------------------------------------------------------------
def slots(kv, new, table, free, n_free, page, max_blocks):
    """(table, kv_out, n_free, cu, slots, positions, all served)."""
    table, kv_out, cu = table.copy(), [], [0]
    sl, pos, ok, want = [], [], True, 0
    for b, (k, n) in enumerate(zip(kv, new)):
        n = max(n, 0)
        have, need = -(-k // page), -(-(k + n) // page)
        fits = k >= 0 and new[b] >= 0 and need <= max_blocks
        if k >= 0 and need <= max_blocks:
            want += need - have
        served = k >= 0 and need <= max_blocks and want <= n_free
        ok &= fits and served
        if served:
            for i in range(have, need):
                table[b, i] = free[n_free - 1 - (want - (need - have) + i - have)]
        for i in range(n):
            sl.append(int(table[b, (k + i) // page]) * page + (k + i) % page if served else -1)
            pos.append(k + i)
        kv_out.append(k + n if served else k)
        cu.append(cu[-1] + n)
    taken, run = 0, 0
    for k, n in zip(kv, new):
        n = max(n, 0)
        if k >= 0 and -(-(k + n) // page) <= max_blocks:
            run += -(-(k + n) // page) - -(-k // page)
        if run <= n_free:
            taken = run
    return table, kv_out, n_free - taken, cu, sl, pos, ok


# ---- the format ----------------------------------------------------------------------------------
def quantise(x, group):
    """x [..., 128] -> codes (int), step, lo of each group (float64; NaN groups: code 0)."""
    y = np.asarray(x, np.float64).reshape(*x.shape[:-1], D // group, group)
    with np.errstate(all="ignore"):
        lo, hi = y.min(-1), y.max(-1)
        rng = (hi.astype(np.float32) - lo.astype(np.float32)).astype(np.float32)
        step = bf16(rng / np.float32(15))
        step = np.where(step < 2.0 ** -126, 0.0, step)
        bad = ~np.isfinite(y).all(-1) | ~np.isfinite(rng)
        r = np.where(step > 0, np.float32(1) / step.astype(np.float32), np.float32(0)).astype(np.float64)
        d = (y.astype(np.float32) - lo.astype(np.float32)[..., None]).astype(np.float64)
        code = np.clip(np.rint(d * r[..., None]), 0, 15)
    code = np.where(bad[..., None], 0, code).astype(np.int64)
    return code.reshape(x.shape), np.where(bad, np.nan, step), np.where(bad, np.nan, lo)


def row_bytes(group):
    return 128 + 8 * (D // group)


def _offsets(r, group):
    ng = D // group
    base, i = (r // 16) * 16 * row_bytes(group), r % 16
    ch = np.arange(D)
    k = base + 64 * i + 16 * (ch % 32 // 8) + 4 * (ch // 32) + ch % 8 // 2
    v = base + 1024 + 64 * i + 8 * ((ch % 32 // 4) ^ (4 * (i // 2 % 2))) + 2 * (ch // 32) + ch % 4 // 2
    return k, v, base + 2048 + 4 * ng * i, base + 2048 + 64 * ng + 4 * ng * i


def write(pages, page, group, slot, h, krow, vrow):
    """Quantises one token's rows of KV head h into pages (uint8 [n, Hkv, bytes])."""
    p, r = divmod(int(slot), page)
    k_at, v_at, ks, vs = _offsets(r, group)
    for at, sat, x in ((k_at, ks, krow), (v_at, vs, vrow)):
        code, step, lo = quantise(x, group)
        dst = pages[p, h]
        dst[at[0::2]] = (code[0::2] | (code[1::2] << 4)).astype(np.uint8)
        sm = np.stack((bits(step), bits(lo)), -1)
        sm[np.isnan(step)] = 0x7fc0
        dst[sat:sat + 4 * (D // group)] = np.ascontiguousarray(sm).view(np.uint8).reshape(-1)


def parts(pages, page, group, slot, h):
    """(codes, steps, minima) per channel of K and of V at a slot."""
    p, r = divmod(int(slot), page)
    k_at, v_at, ks, vs = _offsets(r, group)
    src, out = pages[p, h], []
    for at, sat in ((k_at, ks), (v_at, vs)):
        b = src[at].astype(np.int64)
        code = np.where(np.arange(D) % 2 == 1, b >> 4, b & 15)
        sm = src[sat:sat + 4 * (D // group)].copy().view(np.uint16).astype(np.uint32) << 16
        sm = sm.view(np.float32).astype(np.float64).reshape(-1, 2)
        out.append((code, np.repeat(sm[:, 0], group), np.repeat(sm[:, 1], group)))
    return out


# ---- attention -----------------------------------------------------------------------------------
def attend(pages, page, group, Q, table, kv_lens, cu_q, scale, hidden=lambda b, j: False, wide=False):
    """Q [Hq, T, 128] -> O, lse and the error bound of each element (see `tolerance`), float64; rows behind
    cu_q[-1] are NaN in all three.  hidden(b, j): keys on no page; wide: the bound of the kernel for
    many query rows."""
    Hq, T, _ = Q.shape
    Hkv = pages.shape[1]
    G = Hq // Hkv
    O, L = np.full(Q.shape, np.nan), np.full((Hq, T), np.nan)
    tolO, tolL = np.full(Q.shape, np.nan), np.full((Hq, T), np.nan)
    for b in range(len(kv_lens)):
        n, kv = cu_q[b + 1] - cu_q[b], int(kv_lens[b])
        if n <= 0:
            continue
        for h in range(Hkv):
            ps = [parts(pages, page, group, int(table[b, j // page]) * page + j % page, h)
                  if not hidden(b, j) else [(np.zeros(D, int), np.zeros(D), np.zeros(D))] * 2 for j in range(kv)]
            shown = np.array([not hidden(b, j) for j in range(kv)], bool)
            K, V, Ka, Va, St, Ks = np.zeros((kv, D)), np.zeros((kv, D)), np.zeros((kv, D)), np.zeros((kv, D)), 0.0, 0.0
            for j, ((kc, ks, kl), (vc, vs, vl)) in enumerate(ps):
                K[j], V[j] = kl + kc * ks, vl + vc * vs
                Ka[j], Va[j] = np.abs(kl) + kc * ks, np.abs(vl + 8 * vs) + 8 * vs
                Ks = max(Ks, float(np.nanmax(ks)) if not np.isnan(ks).all() else 0.0)
                St = max(St, float(np.nanmax(vs)) if not np.isnan(vs).all() else 0.0)
            for g in range(G):
                for i in range(n):
                    q = Q[h * G + g, cu_q[b] + i]
                    see = (np.arange(kv) <= kv - n + i) & shown
                    at = (h * G + g, cu_q[b] + i)
                    if not see.any():
                        O[at], L[at], tolO[at], tolL[at] = 0, -np.inf, 0, 0
                        continue
                    s = (K[see] @ q) * scale
                    m = s.max()
                    p = np.exp(s - m)
                    l = p.sum()
                    O[at], L[at] = p @ V[see] / l, m + np.log(l)
                    tolO[at], tolL[at] = tolerance(O[at], L[at], p / l, Va[see], (Ka[see] @ np.abs(q)).max() * scale,
                                                   int(see.sum()), St)
                    if wide:
                        tolO[at], tolL[at] = tolerance_wide(O[at], L[at], p / l, V[see], Va[see], (Ka[see] @ np.abs(q)).max() * scale,
                                                            int(see.sum()), np.nanmax(np.abs(V)), Ks * np.abs(q).sum() * scale)
    return O, L, tolO, tolL


def tolerance(O, lse, p, Va, reach, n, step):
    """Bound of the kernel's error for one row.
    Scores: exact products of codes, summed in fp32 with up to 136 additions and scalings: within
    `reach` (the largest sum of magnitudes behind a score) * 136 * 2^-24 <= reach * 2^-16.
    Probabilities enter the second product in fp16 after the running maximum and the largest step are
    taken out: 2^-11 relative, or 2^-32 of the largest step (fp16's subnormals, at most 15 codes).
    The second product runs on codes less 8, beside sums of lo + 8 step: their magnitudes are Va.
    A relative error of every weight moves O by at most twice its weighted magnitudes (numerator and
    denominator); sums over n weights in fp32 add n / 8 * 2^-24 (a thread sums every eighth key or
    fewer) and the exponential 2^-21.  O is rounded to bf16: 2^-8."""
    ds = reach * 2.0 ** -16 + 2.0 ** -21 + (n / 8 + 32) * 2.0 ** -24
    A = p @ Va
    return np.abs(O) * 2.0 ** -8 + A * (2.0 ** -11 + 2 * ds) + n * 15 * step * 2.0 ** -32 + 2.0 ** -130, \
        ds + 2.0 ** -21 * max(1.0, abs(lse))


def tolerance_wide(O, lse, p, V, Va, reach, n, v_max, step_reach):
    """The same for the kernel that takes many rows.  Scores: exact products, 17 sums of 16 in fp32, a
    step of the tensor core's within 2^-22 (reach * 17 * 2^-22 < reach * 2^-17), and fp16's subnormals
    below the tile's largest step: 2^-16 of it per channel (step_reach: largest step times sum |q|).
    Values are rounded to fp16, 2^-11 relative and 2^-18 of the tile's largest value; probabilities
    2^-11 relative and 2^-25 each.  Sums over n in fp32: n / 2 * 2^-24 (two running sums)."""
    ds = (reach + step_reach) * 2.0 ** -16 + 2.0 ** -21 + (n / 2 + 32) * 2.0 ** -24
    A = p @ np.abs(V)
    return np.abs(O) * 2.0 ** -8 + A * (2.0 ** -10 + 2 * ds) + v_max * (2.0 ** -18 + n * 2.0 ** -25) + 2.0 ** -130, \
        ds + 2.0 ** -21 * max(1.0, abs(lse))
