"""Python binding of libmsa (modality-aware permutation sparse attention, sm_100a).

Argument marshalling only: every step of the path runs in the library's CUDA kernels.
The binding takes torch CUDA tensors (bf16, last dimension 128 contiguous) and passes
their device pointers, strides and the current CUDA stream through the C ABI declared
in include/msa.h.  Importing it without the built library raises ImportError.
"""
from __future__ import annotations

import ctypes
import os
from typing import Dict, List, Optional, Sequence

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmsa.so")

KINDS = {"dense": 0, "ashape": 1, "vslash": 2, "block": 3, "grid": 4, "qbound": 5, "bound2d": 6}
KIND_NAMES = {v: k for k, v in KINDS.items()}
MAX_STRIDES = 8
HEAD_PER_SEGMENT = 1  # msa_head_cfg.flags: Q-boundary index per modality segment
STATUS = {0: "ok", 1: "invalid argument", 2: "shape", 3: "alignment", 4: "workspace", 5: "unsupported",
          6: "cuda", 7: "device timeout", 8: "device bounds", 9: "state"}

_I32, _I64, _F32, _F64, _P = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_double, ctypes.c_void_p


class HeadCfg(ctypes.Structure):
    _fields_ = [("kind", _I32), ("sink", _I32), ("local", _I32), ("k_v", _I32), ("k_s", _I32),
                ("topk_blocks", _I32), ("block_budget", _F64), ("n_strides", _I32), ("strides", _I32 * MAX_STRIDES),
                ("n_phases", _I32), ("flags", _I32), ("grid_budget", _F64)]


class Segment(ctypes.Structure):
    _fields_ = [("start", _I64), ("len", _I64), ("modality", _I32), ("_pad", _I32)]


class ProblemC(ctypes.Structure):
    _fields_ = [("L", _I64), ("Hq", _I32), ("Hkv", _I32), ("d", _I32), ("scale", _F32), ("n_segments", _I32),
                ("segments", _P), ("heads", _P)]


class Strides(ctypes.Structure):
    _fields_ = [("q_head", _I64), ("q_row", _I64), ("k_head", _I64), ("k_row", _I64), ("v_head", _I64),
                ("v_row", _I64), ("o_head", _I64), ("o_row", _I64)]


class HeadIndices(ctypes.Structure):
    _fields_ = [("stride", _I32), ("n_phases", _I32), ("phases", _P), ("n_v", (_I32 * 2) * 2),
                ("v", (_P * 2) * 2), ("n_s", _I32 * 2), ("s", _P * 2), ("blk_ptr", _P), ("blk_idx", _P),
                ("n_seg", _I32), ("seg_nv", _P), ("seg_v", _P), ("seg_ns", _P), ("seg_s", _P)]


class RopeC(ctypes.Structure):
    _fields_ = [("dim", _I32), ("interleaved", _I32), ("n_axes", _I32), ("sections", _I32 * 4), ("scale", _F32),
                ("inv_freq", _F64 * 64)]


class KV4CacheC(ctypes.Structure):
    _fields_ = [("pages", _P), ("n_pages", _I64), ("page_tokens", _I32), ("Hkv", _I32), ("group", _I32), ("_pad", _I32),
                ("state", _P)]


class MsaError(RuntimeError):
    def __init__(self, fn: str, code: int, msg: str = ""):
        super().__init__(f"{fn} failed: {STATUS.get(code, code)} ({msg})")
        self.code = code


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libmsa.so is not built ({LIB_PATH}); run dynamic_sparse_attention_head_b200/build.py")
    lib = ctypes.CDLL(LIB_PATH)
    sig = {
        "msa_plan_create": ([ctypes.POINTER(ProblemC), ctypes.POINTER(_P)], _I32),
        "msa_plan_destroy": ([_P], None),
        "msa_workspace_bytes": ([_P], ctypes.c_size_t),
        "msa_workspace_bytes_indexed": ([_P], ctypes.c_size_t),
        "msa_sparse_prefill_indexed": ([_P, _P, _P, _P, _P, ctypes.POINTER(Strides), _P, ctypes.c_size_t, _P, _P],
                                       _I32),
        "msa_estimate": ([_P, _P, _P, ctypes.POINTER(Strides), _P, ctypes.c_size_t, _P], _I32),
        "msa_set_indices": ([_P, _P, _P, ctypes.c_size_t, _P], _I32),
        "msa_permute": ([_P, _P, _P, _P, ctypes.POINTER(Strides), _P, ctypes.c_size_t, _P], _I32),
        "msa_sparse_prefill": ([_P, _P, _P, _P, ctypes.POINTER(Strides), _P, ctypes.c_size_t, _P, _P], _I32),
        "msa_unpermute": ([_P, _P, ctypes.c_size_t, _P, ctypes.POINTER(Strides), _P], _I32),
        "msa_read_indices": ([_P, _P, _I32, _P, ctypes.POINTER(_I64), _P], _I32),
        "msa_read_tiles": ([_P, _P, _I32, _P, ctypes.POINTER(_I64), _P], _I32),
        "msa_tile_stats": ([_P, _P, _P, _P], _I32),
        "msa_tile_stats_heads": ([_P, _P, _P, _P], _I32),
        "msa_attention_units": ([_P, _P], _I32),
        "msa_mask_pairs": ([_P, _P, _P, _P], _I32),
        "msa_selftest_timeout": ([_P, _P, ctypes.c_uint32, _P], _I32),
        "msa_device_status": ([_P, _P, _P], _I32),
        "msa_status_string": ([_I32], ctypes.c_char_p),
        "msa_kernel_launches": ([], ctypes.c_uint64),
        "msa_vslash_estimate_static": ([_P, _P, _I64, _I64, _I64, _F32, _I32, _I32, _P, _P, _P, _P], _I32),
        "msa_weight_share": ([_P, _P, _I64, _I32, _I32, ctypes.POINTER(Strides), _F32, _P, _P, _I32, ctypes.c_double,
                              _P, _P], _I32),
        "msa_qk_norm_rope": ([_P, _P, ctypes.POINTER(Strides), _P, _P, ctypes.POINTER(Strides), _I64, _I32, _I32, _P,
                              _P, _F32, ctypes.POINTER(RopeC), _P, _I64, _P], _I32),
        "msa_kv4_page_bytes": ([_I32, _I32], ctypes.c_size_t),
        "msa_kv4_slots": ([ctypes.POINTER(KV4CacheC), _P, _P, _I32, _P, _I64, _I32, _P, _P, _P, _P, _P, _P, _P, _I64,
                           _P], _I32),
        "msa_kv4_release": ([ctypes.POINTER(KV4CacheC), _P, _I32, _P, _I32, _P, _I64, _I32, _P, _P, _P], _I32),
        "msa_kv4_append": ([ctypes.POINTER(KV4CacheC), _P, _P, ctypes.POINTER(Strides), _P, _I64, _P], _I32),
        "msa_kv4_read": ([ctypes.POINTER(KV4CacheC), _P, _P, ctypes.POINTER(Strides), _P, _I64, _P], _I32),
        "msa_kv4_attend_workspace_bytes": ([], ctypes.c_size_t),
        "msa_kv4_attend": ([ctypes.POINTER(KV4CacheC), _P, _P, ctypes.POINTER(Strides), _I32, _I32, _F32, _P, _I64,
                            _I32, _P, _P, _I32, _I32, _P, _P, ctypes.c_size_t, _P], _I32),
        "msa_kv4_status": ([ctypes.POINTER(KV4CacheC), _P], _I32),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    return lib


_lib = _load()
EXPORTS = ("msa_plan_create", "msa_plan_destroy", "msa_workspace_bytes", "msa_workspace_bytes_indexed",
           "msa_sparse_prefill_indexed", "msa_estimate", "msa_set_indices",
           "msa_permute", "msa_sparse_prefill", "msa_unpermute", "msa_read_indices", "msa_read_tiles",
           "msa_tile_stats", "msa_tile_stats_heads", "msa_attention_units", "msa_mask_pairs", "msa_selftest_timeout", "msa_device_status", "msa_status_string",
           "msa_kernel_launches", "msa_vslash_estimate_static", "msa_weight_share", "msa_qk_norm_rope",
           "msa_kv4_page_bytes", "msa_kv4_slots", "msa_kv4_release", "msa_kv4_append", "msa_kv4_read",
           "msa_kv4_attend_workspace_bytes", "msa_kv4_attend", "msa_kv4_status")


def kernel_launches() -> int:
    """Kernels launched by libmsa since it was loaded."""
    return int(_lib.msa_kernel_launches())


def _check(fn: str, code: int):
    if code != 0:
        raise MsaError(fn, code, _lib.msa_status_string(code).decode())


def _stream_ptr(stream=None) -> Optional[int]:
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _head_cfg(h) -> HeadCfg:
    c = HeadCfg()
    c.kind = KINDS[h.kind] if isinstance(h.kind, str) else int(h.kind)
    c.sink, c.local, c.k_v, c.k_s = int(h.sink), int(h.local), int(h.k_v), int(h.k_s)
    c.topk_blocks, c.block_budget = int(h.topk_blocks), float(h.block_budget)
    st = list(getattr(h, "strides", ()) or ())
    c.n_strides = len(st)
    for i, s in enumerate(st[:MAX_STRIDES]):
        c.strides[i] = int(s)
    c.n_phases, c.grid_budget = int(h.n_phases), float(h.grid_budget)
    c.flags = HEAD_PER_SEGMENT if getattr(h, "per_segment", False) else 0
    return c


def _strides(Q=None, K=None, V=None, O=None) -> Strides:
    s = Strides()
    for name, t in (("q", Q), ("k", K), ("v", V), ("o", O)):
        if t is None:
            continue
        assert t.dim() == 3 and t.shape[-1] == 128 and t.stride(-1) == 1, f"{name}: [H, L, 128] with d contiguous"
        setattr(s, f"{name}_head", t.stride(0))
        setattr(s, f"{name}_row", t.stride(1))
    return s


class Plan:
    """A validated problem (layout, head patterns, budgets) and its workspace size.

    `problem` needs attributes L, Hq, Hkv, d, scale, segments [(start, len, modality)]
    and heads (each with kind, sink, local, k_v, k_s, topk_blocks, block_budget, strides,
    n_phases, grid_budget).
    """

    def __init__(self, problem):
        self.problem = problem
        segs = (Segment * len(problem.segments))()
        for i, (s0, n, m) in enumerate(problem.segments):
            segs[i].start, segs[i].len, segs[i].modality = int(s0), int(n), int(m)
        heads = (HeadCfg * problem.Hq)()
        for i, h in enumerate(problem.heads):
            heads[i] = _head_cfg(h)
        pc = ProblemC(L=int(problem.L), Hq=int(problem.Hq), Hkv=int(problem.Hkv), d=int(problem.d),
                      scale=float(problem.scale), n_segments=len(problem.segments),
                      segments=ctypes.cast(segs, _P), heads=ctypes.cast(heads, _P))
        self._keep = (segs, heads)
        h = _P()
        _check("msa_plan_create", _lib.msa_plan_create(ctypes.byref(pc), ctypes.byref(h)))
        self._h = h
        self.workspace_bytes = int(_lib.msa_workspace_bytes(h))
        self.workspace_bytes_indexed = int(_lib.msa_workspace_bytes_indexed(h))

    def __del__(self):
        if getattr(self, "_h", None):
            _lib.msa_plan_destroy(self._h)
            self._h = None

    def alloc_workspace(self, indexed: bool = False):
        """Device workspace for the three-call path, or (indexed) the smaller one of the
        index-based path."""
        import torch
        n = self.workspace_bytes_indexed if indexed else self.workspace_bytes
        return torch.empty(n, dtype=torch.uint8, device="cuda")

    # ---- the four steps --------------------------------------------------------------
    def estimate(self, Q, K, ws, stream=None):
        s = _strides(Q=Q, K=K)
        _check("msa_estimate", _lib.msa_estimate(self._h, Q.data_ptr(), K.data_ptr(), ctypes.byref(s), ws.data_ptr(),
                                                 ws.numel(), _stream_ptr(stream)))

    def set_indices(self, idx: List[Dict], ws, stream=None):
        """idx[h]: dict with 'V'/'S' (vertical-slash), {'V': {a: ...}, 'S': {a: ...}} (Q-boundary),
        {'V': {(a, b): ...}, 'S': {a: ...}} (2D-boundary), 'stride'/'phases' (grid), 'T' (block)."""
        arr = (HeadIndices * self.problem.Hq)()
        keep = []

        def ptr(a):
            a = np.ascontiguousarray(np.asarray(a, np.int32))
            keep.append(a)
            return a.ctypes.data, len(a)

        for h, x in enumerate(idx):
            kind = self.problem.heads[h].kind
            hi = arr[h]
            if kind == "vslash":
                hi.v[0][0], hi.n_v[0][0] = ptr(x["V"])
                hi.s[0], hi.n_s[0] = ptr(x["S"])
            elif kind == "qbound" and getattr(self.problem.heads[h], "per_segment", False):
                nseg = len(self.problem.segments)
                vp, sp = (_P * nseg)(), (_P * nseg)()
                nv, ns = np.zeros(nseg, np.int32), np.zeros(nseg, np.int32)
                for k in range(nseg):
                    vp[k], nv[k] = ptr(x["V"][k])
                    sp[k], ns[k] = ptr(x["S"][k])
                keep += [vp, sp, nv, ns]
                hi.n_seg = nseg
                hi.seg_nv, hi.seg_ns = nv.ctypes.data, ns.ctypes.data
                hi.seg_v, hi.seg_s = ctypes.cast(vp, _P), ctypes.cast(sp, _P)
            elif kind == "qbound":
                for a, v in x["V"].items():
                    hi.v[a][0], hi.n_v[a][0] = ptr(v)
                for a, v in x["S"].items():
                    hi.s[a], hi.n_s[a] = ptr(v)
            elif kind == "bound2d":
                for (a, b), v in x["V"].items():
                    hi.v[a][b], hi.n_v[a][b] = ptr(v)
                for a, v in x["S"].items():
                    hi.s[a], hi.n_s[a] = ptr(v)
            elif kind == "grid":
                hi.stride = int(x["stride"])
                hi.phases, hi.n_phases = ptr(x["phases"])
            elif kind == "block":
                T = x["T"]
                bp = np.zeros(len(T) + 1, np.int32)
                bp[1:] = np.cumsum([len(t) for t in T])
                hi.blk_ptr, _ = ptr(bp)
                hi.blk_idx, _ = ptr(np.concatenate([np.asarray(t, np.int32) for t in T]) if len(T) else [0])
        _check("msa_set_indices", _lib.msa_set_indices(self._h, ctypes.cast(arr, _P), ws.data_ptr(), ws.numel(),
                                                       _stream_ptr(stream)))

    def permute(self, Q, K, V, ws, stream=None):
        s = _strides(Q=Q, K=K, V=V)
        _check("msa_permute", _lib.msa_permute(self._h, Q.data_ptr(), K.data_ptr(), V.data_ptr(), ctypes.byref(s),
                                               ws.data_ptr(), ws.numel(), _stream_ptr(stream)))

    def sparse_prefill(self, Q, K, V, ws, lse=None, stream=None):
        s = _strides(Q=Q, K=K, V=V)
        _check("msa_sparse_prefill",
               _lib.msa_sparse_prefill(self._h, Q.data_ptr(), K.data_ptr(), V.data_ptr(), ctypes.byref(s),
                                       ws.data_ptr(), ws.numel(), lse.data_ptr() if lse is not None else None,
                                       _stream_ptr(stream)))

    def unpermute(self, ws, O, stream=None):
        s = _strides(O=O)
        _check("msa_unpermute", _lib.msa_unpermute(self._h, ws.data_ptr(), ws.numel(), O.data_ptr(), ctypes.byref(s),
                                                   _stream_ptr(stream)))

    def sparse_prefill_indexed(self, Q, K, V, ws, O, lse=None, stream=None):
        """Permute + sparse prefill + unpermute in one call: Q rows gathered by index in the
        kernel, O written at original positions."""
        s = _strides(Q=Q, K=K, V=V, O=O)
        _check("msa_sparse_prefill_indexed",
               _lib.msa_sparse_prefill_indexed(self._h, Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(),
                                               ctypes.byref(s), ws.data_ptr(), ws.numel(),
                                               lse.data_ptr() if lse is not None else None, _stream_ptr(stream)))

    def forward(self, Q, K, V, ws, O, lse=None, stream=None, indexed: bool = False, cache: Optional["KV4Cache"] = None,
                slots=None):
        """The whole path: estimate -> permute -> sparse prefill -> unpermute, or (indexed)
        estimate -> index-based sparse prefill.  With `cache` (and `slots`, int64 [L]) the layer's
        keys and values are then also written to the 4-bit cache, for the tokens that follow."""
        if (cache is None) != (slots is None):
            raise ValueError("cache and slots go together")
        self.estimate(Q, K, ws, stream)
        if indexed:
            self.sparse_prefill_indexed(Q, K, V, ws, O, lse, stream)
        else:
            self.permute(Q, K, V, ws, stream)
            self.sparse_prefill(Q, K, V, ws, lse, stream)
            self.unpermute(ws, O, stream)
        if cache is not None:
            cache.append(K, V, slots, stream)

    # ---- inspection (synchronising) --------------------------------------------------
    def _record(self, fn, head, ws, stream=None) -> np.ndarray:
        n = _I64(0)
        code = fn(self._h, ws.data_ptr(), int(head), None, ctypes.byref(n), _stream_ptr(stream))
        if code not in (0, 1):
            _check(fn.__name__, code)
        buf = np.zeros(max(1, n.value), np.int32)
        _check(fn.__name__, fn(self._h, ws.data_ptr(), int(head), buf.ctypes.data, ctypes.byref(n),
                               _stream_ptr(stream)))
        return buf[:n.value]

    def read_indices(self, head: int, ws, stream=None) -> Dict:
        r = self._record(_lib.msa_read_indices, head, ws, stream).tolist()
        i = 0

        def take(n):
            nonlocal i
            out = np.asarray(r[i:i + n], np.int64)
            i += n
            return out

        kind = KIND_NAMES[r[0]]
        stride, nph = r[1], r[2]
        i = 3
        phases = take(nph)
        v = {}
        for a in (0, 1):
            for b in (0, 1):
                n = r[i]
                i += 1
                v[(a, b)] = take(n)
        s = {}
        for a in (0, 1):
            n = r[i]
            i += 1
            s[a] = take(n)
        nb = r[i]
        i += 1
        T = None
        if kind == "block":
            ptrs = take(nb + 1)
            flat = take(int(ptrs[-1]))
            T = [flat[ptrs[b]:ptrs[b + 1]] for b in range(nb)]
        nseg = r[i]
        i += 1
        segv, segs = {}, {}
        for k in range(nseg):  # per-segment Q-boundary: each segment's vertical and slash lines
            n = r[i]
            i += 1
            segv[k] = take(n)
            n = r[i]
            i += 1
            segs[k] = take(n)
        out = {"kind": kind}
        if kind == "grid":
            out.update(stride=stride, phases=phases)
        elif kind == "vslash":
            out.update(V=v[(0, 0)], S=s[0])
        elif kind == "qbound" and nseg > 0:
            out.update(per_segment=True, V=segv, S=segs)
        elif kind == "qbound":
            out.update(V={a: v[(a, 0)] for a in (0, 1)}, S=s)
        elif kind == "bound2d":
            out.update(V=v, S=s)
        elif kind == "block":
            out["T"] = T
        return out

    def read_tiles(self, head: int, ws, stream=None) -> List[Dict]:
        """Work list of one head: per item its class, rows and tiles (source, the 128 key
        positions, and whether the tile is flagged fully allowed for every row)."""
        r = self._record(_lib.msa_read_tiles, head, ws, stream)
        n_items, i = int(r[0]), 1
        items = []
        for _ in range(n_items):
            cls, nrows = int(r[i]), int(r[i + 1])
            rows = r[i + 2:i + 2 + 128].astype(np.int64)
            i += 2 + 128
            nt = int(r[i])
            i += 1
            tiles = []
            for _ in range(nt):
                src = int(r[i])
                keys = r[i + 1:i + 1 + 128].astype(np.int64)
                i += 129
                tiles.append((src & 7, keys, bool(src & 8)))
            items.append({"cls": cls, "nrows": nrows, "rows": rows, "tiles": tiles})
        return items

    def tile_stats(self, ws, stream=None):
        t = (_I64 * 2)()
        _check("msa_tile_stats", _lib.msa_tile_stats(self._h, ws.data_ptr(), ctypes.cast(t, _P), _stream_ptr(stream)))
        return int(t[0]), int(t[1])

    def tile_stats_heads(self, ws, stream=None):
        """Executed tiles of each query head (int64 [Hq])."""
        import numpy as np
        c = np.zeros(self.problem.Hq, np.int64)
        _check("msa_tile_stats_heads", _lib.msa_tile_stats_heads(self._h, ws.data_ptr(), c.ctypes.data_as(_P),
                                                                 _stream_ptr(stream)))
        return c

    def mask_pairs(self, ws, stream=None):
        """Allowed (query, key) pairs per query head under the current masks (int64 [Hq]);
        useful FLOPs = 4 * d * sum."""
        import numpy as np
        c = np.zeros(self.problem.Hq, np.int64)
        _check("msa_mask_pairs", _lib.msa_mask_pairs(self._h, ws.data_ptr(), c.ctypes.data_as(_P), _stream_ptr(stream)))
        return c

    def attention_units(self):
        """(work units, key chunks) of msa_sparse_prefill for this plan."""
        return self.attention_work()[:2]

    def attention_work(self):
        """(work units, key chunks, unit bands) of msa_sparse_prefill for this plan."""
        t = (_I64 * 3)()
        _check("msa_attention_units", _lib.msa_attention_units(self._h, ctypes.cast(t, _P)))
        return int(t[0]), int(t[1]), int(t[2])

    def selftest_timeout(self, ws, limit_us: int = 10000, stream=None):
        """Launch a bounded wait that runs out after limit_us; device_status then reports
        MSA_ERR_TIMEOUT (7)."""
        _check("msa_selftest_timeout", _lib.msa_selftest_timeout(self._h, ws.data_ptr(), int(limit_us),
                                                                 _stream_ptr(stream)))

    def device_status(self, ws, stream=None) -> int:
        return int(_lib.msa_device_status(self._h, ws.data_ptr(), _stream_ptr(stream)))


def vslash_estimate_static(Qh, Kh, scale: float, k_v: int, k_s: int, v_out, s_out, counts_out, stream=None):
    """msa_vslash_estimate_static: vertical/slash lines of one head without any workspace.
    Qh, Kh: [L, 128] bf16 CUDA tensors; v_out [k_v], s_out [k_s], counts_out [2]: int32 CUDA
    tensors the caller allocated beforehand."""
    assert Qh.dim() == 2 and Kh.dim() == 2 and Qh.stride(1) == 1 and Kh.stride(1) == 1
    _check("msa_vslash_estimate_static",
           _lib.msa_vslash_estimate_static(Qh.data_ptr(), Kh.data_ptr(), Qh.shape[0], Qh.stride(0), Kh.stride(0),
                                           float(scale), int(k_v), int(k_s), v_out.data_ptr(), s_out.data_ptr(),
                                           counts_out.data_ptr(), _stream_ptr(stream)))


def weight_share(Q, K, scale: float, heads, rows, recall: float = 0.95, stream=None):
    """msa_weight_share: for each sample s, the fewest dense causal attention weights of query
    row rows[s] of head heads[s] whose sum reaches `recall` of the row's softmax mass.
    Q [Hq, L, 128], K [Hkv, L, 128]: bf16 CUDA tensors; heads, rows: int32 CUDA tensors [n].
    Returns an int64 CUDA tensor [n] (the share of row i is count / (i + 1))."""
    import torch
    assert Q.dim() == 3 and K.dim() == 3 and Q.stride(2) == 1 and K.stride(2) == 1
    n = int(rows.numel())
    out = torch.empty(n, dtype=torch.int64, device=Q.device)
    _check("msa_weight_share",
           _lib.msa_weight_share(Q.data_ptr(), K.data_ptr(), Q.shape[1], Q.shape[0], K.shape[0],
                                 ctypes.byref(_strides(Q, K)), float(scale), heads.data_ptr(), rows.data_ptr(), n,
                                 float(recall), out.data_ptr(), _stream_ptr(stream)))
    return out


# ---- queries and keys before the layer; keys and values after it --------------------------
def _tensor(name, t, dtype, dim, device, contiguous=True):
    """Checks one argument tensor: type, dimensions, device and layout."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: a tensor is wanted")
    if t.dtype != dtype or t.dim() != dim:
        raise ValueError(f"{name}: a {dim}-dimensional tensor of {dtype} is wanted, got {tuple(t.shape)} {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the others on {device}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} has to be contiguous")
    return t


def _rows(name, t, heads, tokens, device):
    """Checks a [heads, tokens, 128] bf16 tensor whose rows are contiguous."""
    import torch
    _tensor(name, t, torch.bfloat16, 3, device, contiguous=False)
    if t.shape[2] != 128 or (t.stride(2) != 1 and t.numel()) or (heads is not None and t.shape[0] != heads) or \
            (tokens is not None and t.shape[1] != tokens):
        raise ValueError(f"{name}: [{'H' if heads is None else heads}, {'T' if tokens is None else tokens}, 128] with "
                         f"contiguous rows is wanted, got {tuple(t.shape)} with strides {t.stride()}")
    return t


def _on(device, stream):
    """Device guard of a call on `device`, and its stream there."""
    import torch
    if device.type != "cuda":
        raise ValueError(f"CUDA tensors are wanted, got {device}")
    return torch.cuda.device(device), (stream if stream is not None else torch.cuda.current_stream(device)).cuda_stream


class Rope:
    """Rotary position embedding of msa_qk_norm_rope: `dim` rotated channels (a multiple of 16), the
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
    import torch
    dev = _rows("Q", Q, None, None, None).device
    T = Q.shape[1]
    _rows("K", K, None, T, dev)
    _rows("Qo", Qo, Q.shape[0], T, dev)
    _rows("Ko", Ko, K.shape[0], T, dev)
    pos = _tensor("positions", positions, torch.int32, positions.dim(), dev, contiguous=False)
    if pos.dim() == 1:
        pos = pos.unsqueeze(0)
    if pos.dim() != 2 or tuple(pos.shape) != (rope.n_axes, T) or (T > 1 and pos.stride(1) != 1):
        raise ValueError(f"positions: int32 [{rope.n_axes}, {T}] with contiguous rows is wanted, got "
                         f"{tuple(positions.shape)}")
    for name, w in (("wq", wq), ("wk", wk)):
        if w is not None and _tensor(name, w, torch.bfloat16, 1, dev).numel() != 128:
            raise ValueError(f"{name}: 128 weights are wanted")
    guard, st = _on(dev, stream)
    with guard:
        _check("msa_qk_norm_rope",
               _lib.msa_qk_norm_rope(Q.data_ptr(), K.data_ptr(), ctypes.byref(_strides(Q=Q, K=K)), Qo.data_ptr(),
                                     Ko.data_ptr(), ctypes.byref(_strides(Q=Qo, K=Ko)), T, Q.shape[0], K.shape[0],
                                     wq.data_ptr() if wq is not None else None,
                                     wk.data_ptr() if wk is not None else None, float(eps), ctypes.byref(rope._c),
                                     pos.data_ptr(), pos.stride(0), st))


def kv4_page_bytes(page: int, group: int) -> int:
    """Bytes of one page of one KV head: page * (128 + 8 * 128 / group)."""
    n = int(_lib.msa_kv4_page_bytes(int(page), int(group)))
    if not n:
        raise ValueError(f"page: 16, 32, 64, 128 or 256 tokens, group: 32, 64 or 128 channels; got {page}, {group}")
    return n


class KV4Cache:
    """One layer's paged 4-bit K/V cache (msa_kv4_cache): `pages` uint8 [n_pages, Hkv, kv4_page_bytes(page,
    group)] on the GPU, `page` tokens a page, `group` channels a scale.  `KV4Cache.alloc` makes the
    pages too.  Calls on one cache run in stream order; a CUDA graph may hold any of them."""

    def __init__(self, pages, page: int = 64, group: int = 64):
        import torch
        want = kv4_page_bytes(page, group)
        _tensor("pages", pages, torch.uint8, 3, None)
        if pages.shape[2] != want:
            raise ValueError(f"pages: [n_pages, Hkv, {want}] is wanted, got {tuple(pages.shape)}")
        if pages.device.type != "cuda":
            raise ValueError(f"pages: a CUDA tensor is wanted, got {pages.device}")
        self.pages, self.page, self.group = pages, int(page), int(group)
        self.n_pages, self.Hkv = int(pages.shape[0]), int(pages.shape[1])
        self.device = pages.device
        self.state = torch.zeros(64, dtype=torch.uint8, device=pages.device)
        self._c = KV4CacheC(pages=pages.data_ptr(), n_pages=self.n_pages, page_tokens=self.page, Hkv=self.Hkv,
                            group=self.group, state=self.state.data_ptr())

    @classmethod
    def alloc(cls, n_pages: int, Hkv: int, page: int = 64, group: int = 64, device="cuda") -> "KV4Cache":
        import torch
        return cls(torch.zeros(n_pages, Hkv, kv4_page_bytes(page, group), dtype=torch.uint8, device=device), page, group)

    def alloc_workspace(self, Hq: int = 0):
        """Zero-filled workspace of `attend` (its size does not depend on the shapes)."""
        import torch
        return torch.zeros(int(_lib.msa_kv4_attend_workspace_bytes()), dtype=torch.uint8, device=self.device)

    def _ints(self, name, t, n=None):
        import torch
        _tensor(name, t, torch.int32, 1, self.device)
        if n is not None and t.numel() != n:
            raise ValueError(f"{name}: {n} entries are wanted, got {t.numel()}")
        return t

    def _table(self, t, B):
        import torch
        _tensor("block_table", t, torch.int32, 2, self.device, contiguous=False)
        if t.shape[0] != B or (t.shape[1] > 1 and t.stride(1) != 1) or (B > 1 and t.stride(0) < t.shape[1]):
            raise ValueError(f"block_table: [{B}, blocks] with contiguous rows is wanted, got {tuple(t.shape)}")
        return t, max(int(t.stride(0)), int(t.shape[1]))

    def slots(self, kv_lens, new_lens, block_table, free_pages, n_free, slots, positions, cu_new, kv_lens_out=None,
              n_free_out=None, stream=None):
        """msa_kv4_slots: pages for new_lens[b] more tokens per request, from the top of the free stack
        free_pages[: n_free]; fills block_table's new entries, cu_new [B + 1], slots (int64) and
        positions (int32) of the new tokens (entries behind the last are left), and kv_lens / n_free
        (in place, or in the *_out tensors)."""
        import torch
        B = self._ints("kv_lens", kv_lens).numel()
        self._ints("new_lens", new_lens, B)
        tab, stride = self._table(block_table, B)
        self._ints("free_pages", free_pages, self.n_pages)
        self._ints("n_free", n_free, 1)
        self._ints("cu_new", cu_new, B + 1)
        kv_out = self._ints("kv_lens_out", kv_lens if kv_lens_out is None else kv_lens_out, B)
        nf_out = self._ints("n_free_out", n_free if n_free_out is None else n_free_out, 1)
        cap = _tensor("slots", slots, torch.int64, 1, self.device).numel()
        self._ints("positions", positions, cap)
        guard, st = _on(self.device, stream)
        with guard:
            _check("msa_kv4_slots",
                   _lib.msa_kv4_slots(ctypes.byref(self._c), kv_lens.data_ptr(), new_lens.data_ptr(), B, tab.data_ptr(),
                                      stride, tab.shape[1], free_pages.data_ptr(), n_free.data_ptr(), kv_out.data_ptr(),
                                      nf_out.data_ptr(), cu_new.data_ptr(), slots.data_ptr(), positions.data_ptr(), cap,
                                      st))

    def release(self, ids, kv_lens, block_table, free_pages, n_free, stream=None):
        """msa_kv4_release: the pages of requests `ids` (int32) go back on the free stack."""
        n = self._ints("ids", ids).numel()
        B = self._ints("kv_lens", kv_lens).numel()
        tab, stride = self._table(block_table, B)
        self._ints("free_pages", free_pages, self.n_pages)
        self._ints("n_free", n_free, 1)
        guard, st = _on(self.device, stream)
        with guard:
            _check("msa_kv4_release",
                   _lib.msa_kv4_release(ctypes.byref(self._c), ids.data_ptr(), n, kv_lens.data_ptr(), B, tab.data_ptr(),
                                        stride, tab.shape[1], free_pages.data_ptr(), n_free.data_ptr(), st))

    def _kv(self, K, V, slots):
        import torch
        T = _tensor("slots", slots, torch.int64, 1, self.device).numel()
        _rows("K", K, self.Hkv, T, self.device)
        _rows("V", V, self.Hkv, T, self.device)
        return T, ctypes.byref(_strides(K=K, V=V))

    def append(self, K, V, slots, stream=None):
        """msa_kv4_append: quantises K, V [Hkv, T, 128] (bf16) into the cache at `slots` (int64 [T];
        negative: skipped; each at most once)."""
        T, s = self._kv(K, V, slots)
        guard, st = _on(self.device, stream)
        with guard:
            _check("msa_kv4_append", _lib.msa_kv4_append(ctypes.byref(self._c), K.data_ptr(), V.data_ptr(), s,
                                                         slots.data_ptr(), T, st))

    def read(self, slots, K, V, stream=None):
        """msa_kv4_read: the values at `slots` into K, V [Hkv, T, 128] (bf16)."""
        T, s = self._kv(K, V, slots)
        guard, st = _on(self.device, stream)
        with guard:
            _check("msa_kv4_read", _lib.msa_kv4_read(ctypes.byref(self._c), K.data_ptr(), V.data_ptr(), s,
                                                     slots.data_ptr(), T, st))

    def attend(self, Q, O, block_table, kv_lens, cu_q, max_q: int, scale: float, ws, lse=None, stream=None):
        """msa_kv4_attend: Q, O [Hq, T, 128] (bf16); request b's query tokens are columns cu_q[b] ..
        cu_q[b + 1) and the last of its kv_lens[b] cached tokens.  max_q: the most query tokens of any
        request (picks the kernel's tile).  lse: fp32 [Hq, T] or None.  ws: alloc_workspace()."""
        import torch
        _rows("Q", Q, None, None, self.device)
        Hq, T = int(Q.shape[0]), int(Q.shape[1])
        _rows("O", O, Hq, T, self.device)
        B = self._ints("kv_lens", kv_lens).numel()
        self._ints("cu_q", cu_q, B + 1)
        tab, stride = self._table(block_table, B)
        if lse is not None and tuple(_tensor("lse", lse, torch.float32, 2, self.device).shape) != (Hq, T):
            raise ValueError(f"lse: [{Hq}, {T}] is wanted, got {tuple(lse.shape)}")
        _tensor("ws", ws, torch.uint8, 1, self.device)
        guard, st = _on(self.device, stream)
        with guard:
            _check("msa_kv4_attend",
                   _lib.msa_kv4_attend(ctypes.byref(self._c), Q.data_ptr(), O.data_ptr(), ctypes.byref(_strides(Q=Q, O=O)),
                                       T, Hq, float(scale), tab.data_ptr(), stride, tab.shape[1], kv_lens.data_ptr(),
                                       cu_q.data_ptr(), B, int(max_q), lse.data_ptr() if lse is not None else None,
                                       ws.data_ptr(), ws.numel(), st))

    def device_status(self, stream=None) -> int:
        """msa_kv4_status (synchronises): 0, or the first error recorded on the device, which it clears."""
        guard, st = _on(self.device, stream)
        with guard:
            return int(_lib.msa_kv4_status(ctypes.byref(self._c), st))


def executed_flops(tiles: int) -> int:
    """FLOPs of the executed 128x128 tiles (QK^T and PV, d = 128)."""
    return 4 * 128 * 128 * 128 * int(tiles)
