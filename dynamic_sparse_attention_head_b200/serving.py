"""What stands around the layer calls: the per-head norm and rotation that make its queries and keys
(msa_qk_norm_rope), and the paged 4-bit cache that holds its keys and values for the tokens that
follow (msa_kv4_*).  Argument checks and marshalling only; the checks are written to cost little, as
a decode step calls these once per layer and token.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import torch

from . import KV4CacheC, RopeC, Strides, _check, _lib

_BF16, _I32, _I64, _U8, _F32 = torch.bfloat16, torch.int32, torch.int64, torch.uint8, torch.float32
_byref = ctypes.byref
_device_now, _stream_now = torch.cuda.current_device, torch._C._cuda_getCurrentRawStream


def _bad(name, t, want):
    """The error of an argument that is not `want`."""
    if not isinstance(t, torch.Tensor):
        return TypeError(f"{name}: {want} is wanted, got {type(t).__name__}")
    return ValueError(f"{name}: {want} is wanted, got {tuple(t.shape)} {t.dtype} with strides {t.stride()} on {t.device}")


def _vector(name, t, dtype, index, n=None):
    """A contiguous vector of `n` entries (None: any) on GPU `index`; its length."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.dim() != 1 or t.get_device() != index or \
            not t.is_contiguous() or (n is not None and t.numel() != n):
        raise _bad(name, t, f"a contiguous {dtype} vector{'' if n is None else f' of {n}'} on cuda:{index}")
    return t.numel()


def _rows(name, t, heads, tokens, index):
    """[heads, tokens, 128] bf16 rows on GPU `index`: their head and token strides."""
    if not isinstance(t, torch.Tensor) or t.dtype is not _BF16 or t.dim() != 3 or t.get_device() != index:
        raise _bad(name, t, f"a bf16 [H, T, 128] tensor on cuda:{index}")
    h, n, d = t.shape
    sh, st, sd = t.stride()
    if d != 128 or (sd != 1 and t.numel()) or (heads is not None and h != heads) or (tokens is not None and n != tokens):
        raise _bad(name, t, f"[{'H' if heads is None else heads}, {'T' if tokens is None else tokens}, 128] with "
                            "contiguous rows")
    return sh, st


def _index(name, t):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise _bad(name, t, "a CUDA tensor")
    return t.get_device()


def _launch(fn, index, stream, *args):
    """One call on GPU `index` (made current around it where it is not), on the given stream or the
    device's current one."""
    st = _stream_now(index) if stream is None else stream.cuda_stream
    if _device_now() == index:
        code = fn(*args, st)
    else:
        with torch.cuda.device(index):
            code = fn(*args, st)
    if code:
        _check(fn.__name__, code)


class Rope:
    """Rotary position embedding of qk_norm_rope: `dim` rotated channels (a multiple of 16), the
    frequencies from `base` (inv_freq[i] = base ** (-2 i / dim)) or given (dim / 2 of them: scaled
    variants), pairs (i, i + dim / 2) or, interleaved, (2 i, 2 i + 1).  `sections`: frequencies of each
    position axis (video tokens: time, height, width), summing to dim / 2; None: one axis.  `scale`
    multiplies the rotated channels."""

    def __init__(self, dim: int = 128, base: float = 1e6, inv_freq: Optional[Sequence[float]] = None,
                 interleaved: bool = False, sections: Optional[Sequence[int]] = None, scale: float = 1.0):
        if dim < 0 or dim > 128 or dim % 16:
            raise ValueError("dim: a multiple of 16 up to 128 is wanted")
        freq = [float(base) ** (-2.0 * i / dim) for i in range(dim // 2)] if inv_freq is None else \
            [float(f) for f in inv_freq]
        if len(freq) != dim // 2:
            raise ValueError(f"inv_freq: {dim // 2} frequencies are wanted, got {len(freq)}")
        sec = [dim // 2] if sections is None else [int(x) for x in sections]
        if not 1 <= len(sec) <= 4 or min(sec) < 0 or sum(sec) != dim // 2:
            raise ValueError(f"sections: up to 4 counts that sum to {dim // 2} are wanted, got {sec}")
        self.n_axes = len(sec)
        self._c = RopeC(dim=dim, interleaved=int(bool(interleaved)), n_axes=len(sec), scale=float(scale))
        for i, f in enumerate(freq):
            self._c.inv_freq[i] = f
        for i, x in enumerate(sec):
            self._c.sections[i] = x


def qk_norm_rope(Q, K, Qo, Ko, positions, rope: Rope, wq=None, wk=None, eps: float = 1e-6, stream=None):
    """msa_qk_norm_rope: RMS norm of every head's rows (weights wq / wk bf16 [128]; None: no norm) and
    the rotation at `positions`, in one pass.  Q, Qo [Hq, T, 128], K, Ko [Hkv, T, 128]: bf16 CUDA
    tensors, any head and token strides that are multiples of 8 (the projection's [T, H, 128]
    transposed); Qo / Ko may be Q / K.  positions: int32 [T], or [axes, T] for a rope with sections."""
    dev = _index("Q", Q)
    qh, qr = _rows("Q", Q, None, None, dev)
    Hq, T = Q.shape[:2]
    kh, kr = _rows("K", K, None, T, dev)
    Hkv = K.shape[0]
    qoh, qor = _rows("Qo", Qo, Hq, T, dev)
    koh, kor = _rows("Ko", Ko, Hkv, T, dev)
    axes = rope.n_axes
    if not isinstance(positions, torch.Tensor) or positions.dtype is not _I32 or positions.get_device() != dev or \
            positions.shape != ((axes, T) if positions.dim() == 2 else (T,)) or (positions.dim() == 1 and axes != 1) or \
            (T > 1 and positions.stride(-1) != 1):
        raise _bad("positions", positions, f"int32 [{axes}, {T}] with contiguous rows on cuda:{dev}")
    if wq is not None:
        _vector("wq", wq, _BF16, dev, 128)
    if wk is not None:
        _vector("wk", wk, _BF16, dev, 128)
    _launch(_lib.msa_qk_norm_rope, dev, stream, Q.data_ptr(), K.data_ptr(), _byref(Strides(qh, qr, kh, kr)), Qo.data_ptr(),
            Ko.data_ptr(), _byref(Strides(qoh, qor, koh, kor)), T, Hq, Hkv, None if wq is None else wq.data_ptr(),
            None if wk is None else wk.data_ptr(), eps, _byref(rope._c), positions.data_ptr(),
            positions.stride(0) if positions.dim() == 2 else T)


def kv4_page_bytes(page: int, group: int) -> int:
    """Bytes of one page of one KV head: page * (128 + 8 * 128 / group)."""
    n = int(_lib.msa_kv4_page_bytes(int(page), int(group)))
    if not n:
        raise ValueError(f"page: 16, 32, 64, 128 or 256 tokens, group: 32, 64 or 128 channels; got {page}, {group}")
    return n


class KV4Cache:
    """One layer's paged 4-bit K/V cache (msa_kv4_cache): `pages` uint8 [n_pages, Hkv, kv4_page_bytes(page,
    group)] on the GPU, `page` tokens a page, `group` channels a scale.  `KV4Cache.alloc` makes the
    pages too.  Calls on one cache run in stream order (`read` and `attend` may overlap); a CUDA graph
    may hold any of them."""

    def __init__(self, pages, page: int = 64, group: int = 64):
        want = kv4_page_bytes(page, group)
        if not isinstance(pages, torch.Tensor) or pages.dtype is not _U8 or pages.dim() != 3 or \
                pages.shape[2] != want or not pages.is_contiguous() or not pages.is_cuda:
            raise _bad("pages", pages, f"a contiguous uint8 [n_pages, Hkv, {want}] CUDA tensor")
        self.pages, self.page, self.group = pages, int(page), int(group)
        self.n_pages, self.Hkv = int(pages.shape[0]), int(pages.shape[1])
        self.device, self._dev = pages.device, pages.get_device()
        self.state = torch.zeros(64, dtype=_U8, device=pages.device)
        self._c = KV4CacheC(pages=pages.data_ptr(), n_pages=self.n_pages, page_tokens=self.page, Hkv=self.Hkv,
                            group=self.group, state=self.state.data_ptr())
        self._ref = _byref(self._c)

    @classmethod
    def alloc(cls, n_pages: int, Hkv: int, page: int = 64, group: int = 64, device="cuda") -> "KV4Cache":
        return cls(torch.zeros(n_pages, Hkv, kv4_page_bytes(page, group), dtype=_U8, device=device), page, group)

    def alloc_workspace(self, Hq: int = 0):
        """Zero-filled workspace of `attend` (its size does not depend on the shapes)."""
        return torch.zeros(int(_lib.msa_kv4_attend_workspace_bytes()), dtype=_U8, device=self.device)

    def _table(self, t, B):
        """Row stride and blocks of a block table [B, blocks]."""
        if not isinstance(t, torch.Tensor) or t.dtype is not _I32 or t.dim() != 2 or t.get_device() != self._dev:
            raise _bad("block_table", t, f"an int32 [{B}, blocks] tensor on cuda:{self._dev}")
        n, blocks = t.shape
        row, one = t.stride()
        if n != B or (blocks > 1 and one != 1) or (B > 1 and row < blocks):
            raise _bad("block_table", t, f"[{B}, blocks] with contiguous rows")
        return (row if row > blocks else blocks), blocks

    def slots(self, kv_lens, new_lens, block_table, free_pages, n_free, slots, positions, cu_new, kv_lens_out=None,
              n_free_out=None, stream=None):
        """msa_kv4_slots: pages for new_lens[b] more tokens per request, from the top of the free stack
        free_pages[: n_free]; fills block_table's new entries, cu_new [B + 1], slots (int64) and
        positions (int32) of the new tokens (entries behind the last are left), and kv_lens / n_free
        (in place, or in the *_out tensors)."""
        dev = self._dev
        B = _vector("kv_lens", kv_lens, _I32, dev)
        _vector("new_lens", new_lens, _I32, dev, B)
        row, blocks = self._table(block_table, B)
        _vector("free_pages", free_pages, _I32, dev, self.n_pages)
        _vector("n_free", n_free, _I32, dev, 1)
        _vector("cu_new", cu_new, _I32, dev, B + 1)
        if kv_lens_out is None:
            kv_lens_out = kv_lens
        else:
            _vector("kv_lens_out", kv_lens_out, _I32, dev, B)
        if n_free_out is None:
            n_free_out = n_free
        else:
            _vector("n_free_out", n_free_out, _I32, dev, 1)
        cap = _vector("slots", slots, _I64, dev)
        _vector("positions", positions, _I32, dev, cap)
        _launch(_lib.msa_kv4_slots, dev, stream, self._ref, kv_lens.data_ptr(), new_lens.data_ptr(), B,
                block_table.data_ptr(), row, blocks, free_pages.data_ptr(), n_free.data_ptr(), kv_lens_out.data_ptr(),
                n_free_out.data_ptr(), cu_new.data_ptr(), slots.data_ptr(), positions.data_ptr(), cap)

    def release(self, ids, kv_lens, block_table, free_pages, n_free, stream=None):
        """msa_kv4_release: the pages of requests `ids` (int32) go back on the free stack."""
        dev = self._dev
        n = _vector("ids", ids, _I32, dev)
        B = _vector("kv_lens", kv_lens, _I32, dev)
        row, blocks = self._table(block_table, B)
        _vector("free_pages", free_pages, _I32, dev, self.n_pages)
        _vector("n_free", n_free, _I32, dev, 1)
        _launch(_lib.msa_kv4_release, dev, stream, self._ref, ids.data_ptr(), n, kv_lens.data_ptr(), B,
                block_table.data_ptr(), row, blocks, free_pages.data_ptr(), n_free.data_ptr())

    def append(self, K, V, slots, stream=None):
        """msa_kv4_append: quantises K, V [Hkv, T, 128] (bf16) into the cache at `slots` (int64 [T];
        negative: skipped; each at most once)."""
        dev = self._dev
        T = _vector("slots", slots, _I64, dev)
        kh, kr = _rows("K", K, self.Hkv, T, dev)
        vh, vr = _rows("V", V, self.Hkv, T, dev)
        _launch(_lib.msa_kv4_append, dev, stream, self._ref, K.data_ptr(), V.data_ptr(),
                _byref(Strides(0, 0, kh, kr, vh, vr)), slots.data_ptr(), T)

    def read(self, slots, K, V, stream=None):
        """msa_kv4_read: the values at `slots` into K, V [Hkv, T, 128] (bf16)."""
        dev = self._dev
        T = _vector("slots", slots, _I64, dev)
        kh, kr = _rows("K", K, self.Hkv, T, dev)
        vh, vr = _rows("V", V, self.Hkv, T, dev)
        _launch(_lib.msa_kv4_read, dev, stream, self._ref, K.data_ptr(), V.data_ptr(),
                _byref(Strides(0, 0, kh, kr, vh, vr)), slots.data_ptr(), T)

    def attend(self, Q, O, block_table, kv_lens, cu_q, max_q: int, scale: float, ws, lse=None, stream=None):
        """msa_kv4_attend: Q, O [Hq, T, 128] (bf16); request b's query tokens are columns cu_q[b] ..
        cu_q[b + 1) and the last of its kv_lens[b] cached tokens.  max_q: the most query tokens of any
        request (picks the kernel's tile).  lse: fp32 [Hq, T] or None.  ws: alloc_workspace()."""
        dev = self._dev
        qh, qr = _rows("Q", Q, None, None, dev)
        Hq, T = Q.shape[:2]
        oh, orow = _rows("O", O, Hq, T, dev)
        B = _vector("kv_lens", kv_lens, _I32, dev)
        _vector("cu_q", cu_q, _I32, dev, B + 1)
        row, blocks = self._table(block_table, B)
        if lse is not None and (not isinstance(lse, torch.Tensor) or lse.dtype is not _F32 or lse.shape != (Hq, T) or
                                lse.get_device() != dev or not lse.is_contiguous()):
            raise _bad("lse", lse, f"a contiguous float32 [{Hq}, {T}] tensor on cuda:{dev}")
        n = _vector("ws", ws, _U8, dev)
        _launch(_lib.msa_kv4_attend, dev, stream, self._ref, Q.data_ptr(), O.data_ptr(),
                _byref(Strides(qh, qr, 0, 0, 0, 0, oh, orow)), T, Hq, scale, block_table.data_ptr(), row, blocks,
                kv_lens.data_ptr(), cu_q.data_ptr(), B, max_q, None if lse is None else lse.data_ptr(), ws.data_ptr(), n)

    def device_status(self, stream=None) -> int:
        """msa_kv4_status (synchronises): 0, or the first error recorded on the device, which it clears."""
        st = _stream_now(self._dev) if stream is None else stream.cuda_stream
        with torch.cuda.device(self._dev):
            return int(_lib.msa_kv4_status(self._ref, st))
