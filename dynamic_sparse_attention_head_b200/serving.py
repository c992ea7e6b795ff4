"""What stands around the layer calls: the per-head norm and rotation that make its queries and keys
(msa_qk_norm_rope), and the paged 4-bit cache that holds its keys and values for the tokens that
follow (msa_kv4_*).  Marshalling only; a decode step calls these once per layer and token, so the
checks of their tensors are in C++ (csrc/binding.cpp).
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import torch

from . import KV4_WHOLE_REQUESTS, KV4CacheC, RopeC, _check, _lib

try:
    from . import _binding as _native  # checks the tensors and calls the library (csrc/binding.cpp)
except ImportError as e:
    raise ImportError(f"_binding.so is not built or does not load ({e}); run dynamic_sparse_attention_head_b200/build.py") from e


def _stream(stream):
    return None if stream is None else stream.cuda_stream


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
    transposed); Qo / Ko may be Q / K.  positions: int32 [T], or [axes, T] for a rope with sections
    (expanded from one row where the axes agree); None for a norm alone (dim = 0)."""
    code = _native.norm_rope(Q, K, Qo, Ko, positions, ctypes.addressof(rope._c), rope.n_axes, wq, wk, eps,
                             None if stream is None else stream.cuda_stream)
    if code:
        _check("msa_qk_norm_rope", code)


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
    may hold any of them.  `whole_requests`: `slots` refuses a request whose new tokens do not all have an entry in its map,
    and all after it, as it does where the pages run out (otherwise the map alone is cut, and the lengths go on over
    tokens that cannot be written)."""

    def __init__(self, pages, page: int = 64, group: int = 64, whole_requests: bool = False):
        want = kv4_page_bytes(page, group)
        if not isinstance(pages, torch.Tensor) or pages.dtype is not torch.uint8 or pages.dim() != 3 or \
                pages.shape[2] != want or not pages.is_contiguous() or not pages.is_cuda:
            got = f"{tuple(pages.shape)} {pages.dtype} on {pages.device}" if isinstance(pages, torch.Tensor) else type(pages)
            raise ValueError(f"pages: a contiguous uint8 [n_pages, Hkv, {want}] CUDA tensor is wanted, got {got}")
        self.pages, self.page, self.group = pages, int(page), int(group)
        self.n_pages, self.Hkv = int(pages.shape[0]), int(pages.shape[1])
        self.device, self._dev = pages.device, pages.get_device()
        self.state = torch.zeros(64, dtype=torch.uint8, device=pages.device)
        self._c = KV4CacheC(pages=pages.data_ptr(), n_pages=self.n_pages, page_tokens=self.page, Hkv=self.Hkv,
                            group=self.group, flags=KV4_WHOLE_REQUESTS if whole_requests else 0, state=self.state.data_ptr())
        self._addr = ctypes.addressof(self._c)

    @classmethod
    def alloc(cls, n_pages: int, Hkv: int, page: int = 64, group: int = 64, device="cuda",
              whole_requests: bool = False) -> "KV4Cache":
        return cls(torch.zeros(n_pages, Hkv, kv4_page_bytes(page, group), dtype=torch.uint8, device=device), page, group,
                   whole_requests)

    def alloc_workspace(self, Hq: int = 0):
        """Zero-filled workspace of `attend` (its size does not depend on the shapes)."""
        return torch.zeros(int(_lib.msa_kv4_attend_workspace_bytes()), dtype=torch.uint8, device=self.device)

    def slots(self, kv_lens, new_lens, block_table, free_pages, n_free, slots, positions, cu_new, kv_lens_out=None,
              n_free_out=None, stream=None):
        """msa_kv4_slots: pages for new_lens[b] more tokens per request, from the top of the free stack
        free_pages[: n_free]; fills block_table's new entries, cu_new [B + 1], slots (int64) and
        positions (int32) of the new tokens (entries behind the last are left), and kv_lens / n_free
        (in place, or in the *_out tensors).  More new tokens than `slots` holds are an error of device_status(); see
        `whole_requests`."""
        code = _native.slots(self._addr, self._dev, kv_lens, new_lens, block_table, free_pages, n_free, slots, positions,
                             cu_new, kv_lens_out, n_free_out, None if stream is None else stream.cuda_stream)
        if code:
            _check("msa_kv4_slots", code)

    def release(self, ids, kv_lens, block_table, free_pages, n_free, stream=None):
        """msa_kv4_release: the pages of requests `ids` (int32) go back on the free stack."""
        code = _native.release(self._addr, self._dev, ids, kv_lens, block_table, free_pages, n_free, _stream(stream))
        if code:
            _check("msa_kv4_release", code)

    def append(self, K, V, slots, stream=None):
        """msa_kv4_append: quantises K, V [Hkv, T, 128] (bf16) into the cache at `slots` (int64 [T];
        negative: skipped; each at most once)."""
        code = _native.append(self._addr, self._dev, K, V, slots, None if stream is None else stream.cuda_stream)
        if code:
            _check("msa_kv4_append", code)

    def read(self, slots, K, V, stream=None):
        """msa_kv4_read: the values at `slots` into K, V [Hkv, T, 128] (bf16)."""
        code = _native.read(self._addr, self._dev, K, V, slots, None if stream is None else stream.cuda_stream)
        if code:
            _check("msa_kv4_read", code)

    def attend(self, Q, O, block_table, kv_lens, cu_q, max_q: int, scale: float, ws, lse=None, stream=None):
        """msa_kv4_attend: Q, O [Hq, T, 128] (bf16); request b's query tokens are columns cu_q[b] ..
        cu_q[b + 1) and the last of its kv_lens[b] cached tokens.  max_q: the most query tokens of any
        request (picks the kernel for all requests of the call: long prompts and single tokens are better served
        by a call each).  lse: fp32 [Hq, T] or None.  ws: alloc_workspace()."""
        code = _native.attend(self._addr, self._dev, Q, O, block_table, kv_lens, cu_q, max_q, scale, ws, lse,
                              None if stream is None else stream.cuda_stream)
        if code:
            _check("msa_kv4_attend", code)

    def device_status(self, stream=None) -> int:
        """msa_kv4_status (synchronises): 0, or the first error recorded on the device, which it clears."""
        return int(_native.status(self._addr, self._dev, _stream(stream)))
