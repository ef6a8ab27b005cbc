"""ctypes binding of libprhs.so: argument marshalling only.

Every function here has the name of the C entry point it calls (without the
``prhs_`` prefix) and does no arithmetic of the method: it turns torch CUDA
tensors into device pointers, fills the ``prhs_kv`` descriptor, calls the C
function and raises ``PrhsError`` on a non-OK status. Torch only provides
device memory and streams.
"""
from __future__ import annotations

import ctypes
import os

import torch

from .build import LIB

PRHS_OK, PRHS_EINVAL, PRHS_EUNSUPPORTED, PRHS_EWORKSPACE, PRHS_ECUDA, PRHS_EDEVICE = range(6)
PRHS_F32, PRHS_BF16 = 0, 1
DEV_TIMEOUT, DEV_BAD_INDEX, DEV_BAD_LEN, DEV_BAD_BLOCK, DEV_CAPACITY = 1, 2, 4, 8, 16

# Entry points declared in include/prhs.h, in declaration order.
EXPORTS = ["prhs_workspace_size", "prhs_workspace_init", "prhs_score_select", "prhs_retrieve",
           "prhs_score",
           "prhs_select", "prhs_cis_dilate",
           "prhs_sparse_attn", "prhs_sparse_attn_noalloc", "prhs_set_mass", "prhs_dense_attn",
           "prhs_decode_step", "prhs_append_kv", "prhs_plan_tokens", "prhs_rope_turns",
           "prhs_rope_append", "prhs_tree_workspace_size", "prhs_tree_attn",
           "prhs_commit_tokens", "prhs_commit_planned", "prhs_selftest_wait_timeout", "prhs_last_error",
           "prhs_device_error_bits", "prhs_status_str", "prhs_last_message", "prhs_num_sms",
           "prhs_launch_count"]


# Drafted tokens of one sequence's tree, and the 32-bit words of a token's mask.
TREE_MAX = 128
TREE_WORDS = TREE_MAX // 32
ROPE_KINDS = {"plain": 0, "linear": 1, "ntk": 2, "bands": 3, "ramp": 4}


class PrhsError(RuntimeError):
    def __init__(self, status: int, where: str, message: str):
        super().__init__(f"{where}: status {status}: {message}")
        self.status = status


class prhs_kv(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("B", ctypes.c_int), ("Hq", ctypes.c_int),
                ("Hkv", ctypes.c_int), ("d", ctypes.c_int), ("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("t_max", ctypes.c_int), ("seq_lens", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("block_size", ctypes.c_int),
                ("max_blocks", ctypes.c_int), ("num_blocks", ctypes.c_int)]


class prhs_rope(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("turns", ctypes.c_void_p), ("mscale", ctypes.c_float)]


_lib = None


def load(path: str | None = None) -> ctypes.CDLL:
    """Load libprhs.so (fails loudly when it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or LIB
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with python -m sparse_kv_selection_gb300.build")
    lib = ctypes.CDLL(path)
    P, I, F, D, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_double, ctypes.c_size_t
    KV = ctypes.POINTER(prhs_kv)
    ROPE, L = ctypes.POINTER(prhs_rope), ctypes.c_longlong
    sig = {
        "prhs_workspace_size": (Z, [KV, I]),
        "prhs_workspace_init": (I, [P, Z, P]),
        "prhs_score_select": (I, [KV, P, F, I, P, I, I, P, P, P, I, P, P, P, I, P, P, Z, P]),
        "prhs_retrieve": (I, [KV, P, F, I, P, I, I, P, P, P, I, P, P, P, I, P, P, P, P, Z, P]),
        "prhs_score": (I, [KV, P, F, P, P, Z, P]),
        "prhs_select": (I, [KV, P, I, P, I, I, P, P, P, I, P, P, P, I, P, P, Z, P]),
        "prhs_cis_dilate": (I, [KV, P, P, I, P, P, I, I, I, I, D, I, P, P, P, I, P, P]),
        "prhs_sparse_attn": (I, [KV, P, F, P, P, I, P, P, P, Z, P]),
        "prhs_sparse_attn_noalloc": (I, [KV, P, F, P, P, I, P, P, P]),
        "prhs_set_mass": (I, [KV, P, F, P, P, I, P, P, Z, P]),
        "prhs_dense_attn": (I, [KV, P, F, P, P, P, Z, P]),
        "prhs_decode_step": (I, [KV, P, P, F, I, P, I, I, I, I, D, I, P, P, P, I, P, P, P, I, P, P, P, P,
                                 P, Z, P]),
        "prhs_append_kv": (I, [KV, P, P, P]),
        "prhs_plan_tokens": (I, [KV, P, I, P, P, I, P, P, P, P, P, P, P, P, P]),
        "prhs_rope_turns": (I, [I, I, D, D, D, D, D, P, ctypes.POINTER(F)]),
        "prhs_rope_append": (I, [KV, ROPE, I, P, P, P, L, P, L, P, L, P, P, P]),
        "prhs_tree_workspace_size": (Z, [KV, I]),
        "prhs_tree_attn": (I, [KV, P, P, L, P, L, F, I, P, I, P, P, P, P, Z, P]),
        "prhs_commit_tokens": (I, [KV, I, P, P, I, P, P, L, P, L, P, P]),
        "prhs_commit_planned": (I, [KV, I, P, P, P, I, P, P, L, P, L, P, P]),
        "prhs_selftest_wait_timeout": (I, [ctypes.c_uint, P]),
        "prhs_last_error": (I, []),
        "prhs_device_error_bits": (ctypes.c_uint, []),
        "prhs_launch_count": (ctypes.c_ulonglong, []),
        "prhs_status_str": (ctypes.c_char_p, [I]),
        "prhs_last_message": (ctypes.c_char_p, []),
        "prhs_num_sms": (I, []),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError("tensor arguments must be contiguous")
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(status: int, where: str) -> None:
    if status != PRHS_OK:
        raise PrhsError(status, where, load().prhs_last_message().decode())


class KVCache:
    """Device-resident KV cache plus the descriptor the C ABI takes.

    ``k``/``v`` are contiguous [B][Hkv][t_max][d] or paged
    [num_blocks][Hkv][block_size][d] tensors of dtype float32 or bfloat16;
    ``seq_lens`` int32 [B]; ``block_table`` int32 [B][max_blocks] or None.
    """

    def __init__(self, k, v, seq_lens, Hq, block_table=None, block_size=16):
        assert k.is_cuda and v.is_cuda and k.shape == v.shape
        self.k, self.v = k.contiguous(), v.contiguous()
        self.seq_lens = seq_lens.to(torch.int32).contiguous()
        self.block_table = None if block_table is None else block_table.to(torch.int32).contiguous()
        self.device, self.dtype = self.k.device, self.k.dtype
        self.index = 0 if self.device.index is None else self.device.index
        self.desc = prhs_kv()
        d = self.desc
        d.dtype = PRHS_BF16 if k.dtype == torch.bfloat16 else PRHS_F32
        if k.dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("cache dtype must be float32 or bfloat16")
        d.Hq = Hq
        d.d = k.shape[-1]
        d.Hkv = k.shape[1]
        d.k, d.v = _ptr(self.k), _ptr(self.v)
        d.seq_lens = _ptr(self.seq_lens)
        if self.block_table is None:
            d.B, d.t_max = k.shape[0], k.shape[2]
            d.block_table, d.block_size, d.max_blocks, d.num_blocks = None, 0, 0, 0
        else:
            d.B = self.block_table.shape[0]
            d.t_max = 0
            d.block_table = _ptr(self.block_table)
            d.block_size = k.shape[2]
            d.max_blocks = self.block_table.shape[1]
            d.num_blocks = k.shape[0]

    @property
    def B(self):
        return self.desc.B

    @property
    def Hq(self):
        return self.desc.Hq

    @property
    def t_max(self):
        d = self.desc
        return d.t_max if self.block_table is None else d.max_blocks * d.block_size

    def ref(self):
        return ctypes.byref(self.desc)


def workspace_size(kv: KVCache, cap: int = 0) -> int:
    n = load().prhs_workspace_size(kv.ref(), cap)
    if n == 0:
        raise PrhsError(PRHS_EINVAL, "workspace_size", load().prhs_last_message().decode())
    return n


def workspace_init(ws, stream=None) -> None:
    _check(load().prhs_workspace_init(_ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "workspace_init")


def make_workspace(kv: KVCache, cap: int = 0, stream=None):
    """Allocate (through torch) and zero a workspace for this cache."""
    n = workspace_size(kv, cap)
    ws = torch.empty(n, dtype=torch.uint8, device=kv.k.device)
    workspace_init(ws, stream)
    return ws


def score_select(kv, q, scale, N, idx, n_sel, delta, ws, *, n_budget=None, head_skip=None,
                 anchor_idx=None, anchor_n=None, q_anchor=None, n_sink=0, window=0,
                 stream=None) -> None:
    cap = idx.shape[-1]
    acap = anchor_idx.shape[-1] if anchor_idx is not None else 0
    _check(load().prhs_score_select(kv.ref(), _ptr(q), float(scale), int(N), _ptr(n_budget),
                                    int(n_sink), int(window),
                                    _ptr(head_skip), _ptr(idx), _ptr(n_sel), cap, _ptr(delta),
                                    _ptr(anchor_idx), _ptr(anchor_n), acap, _ptr(q_anchor),
                                    _ptr(ws), ws.numel(), _stream(stream)), "score_select")


def retrieve(kv, q, scale, N, idx, n_sel, delta, out, lse, ws, *, n_budget=None, head_skip=None,
             anchor_idx=None, anchor_n=None, q_anchor=None, n_sink=0, window=0,
             stream=None) -> None:
    """Top-N set, delta and the attention over the set for the heads not
    flagged in head_skip (prhs_retrieve); out [B][Hq][d] and lse [B][Hq] fp32."""
    cap = idx.shape[-1]
    acap = anchor_idx.shape[-1] if anchor_idx is not None else 0
    _check(load().prhs_retrieve(kv.ref(), _ptr(q), float(scale), int(N), _ptr(n_budget),
                                int(n_sink), int(window),
                                _ptr(head_skip), _ptr(idx), _ptr(n_sel), cap, _ptr(delta),
                                _ptr(anchor_idx), _ptr(anchor_n), acap, _ptr(q_anchor),
                                _ptr(out), _ptr(lse), _ptr(ws), ws.numel(), _stream(stream)),
           "retrieve")


def score(kv, q, scale, ws, *, head_skip=None, stream=None) -> None:
    _check(load().prhs_score(kv.ref(), _ptr(q), float(scale), _ptr(head_skip), _ptr(ws),
                             ws.numel(), _stream(stream)), "score")


def select(kv, q, N, idx, n_sel, delta, ws, *, n_budget=None, head_skip=None, anchor_idx=None,
           anchor_n=None, q_anchor=None, n_sink=0, window=0, stream=None) -> None:
    cap = idx.shape[-1]
    acap = anchor_idx.shape[-1] if anchor_idx is not None else 0
    _check(load().prhs_select(kv.ref(), _ptr(q), int(N), _ptr(n_budget), int(n_sink), int(window),
                              _ptr(head_skip),
                              _ptr(idx), _ptr(n_sel), cap, _ptr(delta), _ptr(anchor_idx),
                              _ptr(anchor_n), acap, _ptr(q_anchor), _ptr(ws), ws.numel(),
                              _stream(stream)), "select")


def cis_dilate(kv, anchor_idx, anchor_n, q, q_anchor, w, tau, idx, n_sel, reuse, *, max_run=0,
               anchor_age=None, n_sink=0, window=0, n_den=0, stream=None) -> None:
    _check(load().prhs_cis_dilate(kv.ref(), _ptr(anchor_idx), _ptr(anchor_n), anchor_idx.shape[-1],
                                  _ptr(q), _ptr(q_anchor), int(w), int(n_den), int(n_sink),
                                  int(window), float(tau), int(max_run),
                                  _ptr(anchor_age), _ptr(idx), _ptr(n_sel), idx.shape[-1],
                                  _ptr(reuse), _stream(stream)), "cis_dilate")


def set_mass(kv, q, scale, idx, n_sel, delta, ws, stream=None) -> None:
    """Dropped attention mass of the given sets under q (prhs_set_mass)."""
    _check(load().prhs_set_mass(kv.ref(), _ptr(q), float(scale), _ptr(idx), _ptr(n_sel),
                                idx.shape[-1], _ptr(delta), _ptr(ws), ws.numel(), _stream(stream)),
           "set_mass")


def sparse_attn(kv, q, scale, idx, n_sel, out, lse, ws, stream=None) -> None:
    _check(load().prhs_sparse_attn(kv.ref(), _ptr(q), float(scale), _ptr(idx), _ptr(n_sel),
                                   idx.shape[-1], _ptr(out), _ptr(lse), _ptr(ws), ws.numel(),
                                   _stream(stream)), "sparse_attn")


def sparse_attn_noalloc(kv, q, scale, idx, n_sel, out, lse, stream=None) -> None:
    """prhs_sparse_attn without a workspace (fixed in-library scratch)."""
    _check(load().prhs_sparse_attn_noalloc(kv.ref(), _ptr(q), float(scale), _ptr(idx),
                                           _ptr(n_sel), idx.shape[-1], _ptr(out), _ptr(lse),
                                           _stream(stream)), "sparse_attn_noalloc")


def dense_attn(kv, q, scale, out, lse, ws, stream=None) -> None:
    _check(load().prhs_dense_attn(kv.ref(), _ptr(q), float(scale), _ptr(out), _ptr(lse),
                                  _ptr(ws), ws.numel(), _stream(stream)), "dense_attn")


def decode_step(kv, q, scale, N, w, tau, anchor_idx, anchor_n, q_anchor, idx, n_sel, reuse, delta,
                out, lse, ws, *, n_budget=None, max_run=0, anchor_age=None, n_sink=0, window=0,
                n_den=0, gate=None, stream=None) -> None:
    _check(load().prhs_decode_step(kv.ref(), _ptr(q), _ptr(gate), float(scale), int(N),
                                   _ptr(n_budget), int(n_sink), int(window), int(w), int(n_den),
                                   float(tau), int(max_run), _ptr(anchor_age), _ptr(anchor_idx),
                                   _ptr(anchor_n),
                                   anchor_idx.shape[-1], _ptr(q_anchor), _ptr(idx), _ptr(n_sel),
                                   idx.shape[-1], _ptr(reuse), _ptr(delta), _ptr(out), _ptr(lse),
                                   _ptr(ws), ws.numel(), _stream(stream)), "decode_step")


def append_kv(kv, k_new, v_new, stream=None) -> None:
    """Write one key and value row per (sequence, KV head) at each
    sequence's current length and advance kv.seq_lens (prhs_append_kv)."""
    _check(load().prhs_append_kv(kv.ref(), _ptr(k_new), _ptr(v_new), _stream(stream)), "append_kv")


# --------------------------------------------------------------------------- #
# token batches: several new tokens per sequence in one step
# --------------------------------------------------------------------------- #
def _array(t, name, shape, dtype, device, optional=False):
    """Pointer of a packed array argument after checking what it is."""
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return t.data_ptr()
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the cache on {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return _ptr(t)


def _rows(t, name, T, heads, d, dtype, device):
    """Pointer and token stride of [T][heads][d] rows that may be a view of a
    wider buffer (a fused projection's output): packed within a token."""
    if t is None:
        return None, heads * d
    if t.dtype is dtype and t.shape == (T, heads, d) and t.device == device and t.is_contiguous():
        return t.data_ptr(), heads * d
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the cache on {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != (T, heads, d):
        raise ValueError(f"{name} must have shape {(T, heads, d)}, got {tuple(t.shape)}")
    s0, s1, s2 = t.stride()
    if T and ((heads > 1 and s1 != d) or s2 != 1):
        raise ValueError(f"{name}: the rows of one token must be packed")
    return t.data_ptr(), (s0 if T > 1 else heads * d)


# The current device, and a device's current stream as a handle: torch's own
# shortcuts past the objects that the public functions build at every call (1.3 us
# of about 10), where this torch has them.
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = (getattr(torch._C, "_cuda_getCurrentRawStream", None)
               or (lambda index: torch.cuda.current_stream(index).cuda_stream))


def _call(kv, where, fn, stream, *args) -> None:
    """fn(*args, stream) with the cache's device current (torch's current
    stream of that device when none is given); raises on a non-OK status."""
    if _device() != kv.index:
        with torch.cuda.device(kv.index):
            return _call(kv, where, fn, stream, *args)
    st = _raw_stream(kv.index) if stream is None else _stream(stream)
    status = fn(*args, st)
    if status != PRHS_OK:
        _check(status, where)


def rope_turns(rot_dim, base=10000.0, kind="plain", factor=1.0, original=0.0, low=0.0, high=0.0):
    """The fixed-point turns a position of each rotated pair (a list of Python
    integers below 2**64) and the factor on cos and sin (prhs_rope_turns)."""
    if kind not in ROPE_KINDS:
        raise ValueError(f"scaling must be one of {sorted(ROPE_KINDS)}, got {kind!r}")
    out = (ctypes.c_uint64 * max(1, int(rot_dim) // 2))()
    mscale = ctypes.c_float()
    _check(load().prhs_rope_turns(ROPE_KINDS[kind], int(rot_dim), float(base), float(factor),
                                  float(original), float(low), float(high), out,
                                  ctypes.byref(mscale)), "rope_turns")
    return list(out), float(mscale.value)


class RopeTable:
    """Rotary frequencies on the device, for rope_append.

    rot_dim elements of each head are rotated (a multiple of 16 up to d),
    pairs (i, i + rot_dim / 2) or, interleaved, (2i, 2i + 1). scaling: None,
    "linear", "ntk", "bands" or "ramp" with factor (and original, low, high
    for the last two), as prhs_rope_kind defines them.
    """

    def __init__(self, rot_dim, base=10000.0, *, interleaved=False, scaling=None, factor=1.0,
                 original=0.0, low=0.0, high=0.0, device="cuda"):
        turns, mscale = rope_turns(rot_dim, base, scaling or "plain", factor, original, low, high)
        signed = [x - (1 << 64) if x >= 1 << 63 else x for x in turns]
        self.turns = torch.tensor(signed, dtype=torch.int64, device=device)
        self.mscale = mscale
        self.desc = prhs_rope(int(rot_dim), int(bool(interleaved)), self.turns.data_ptr(), mscale)

    def ref(self):
        return ctypes.byref(self.desc)


def plan_tokens(kv, n_new, cu_new, positions, slots, *, parents=None, tree_mask=None,
                free_pages=None, free_head=None, n_pages=None, free_head_out=None,
                n_pages_out=None, stream=None) -> None:
    """Pages, slots, positions and tree masks of positions.numel() packed
    tokens (prhs_plan_tokens). On a paged cache kv.block_table gets the new
    pages; free_head and n_pages are updated in place unless their _out arrays
    are given."""
    dev, i32, T, B = kv.device, torch.int32, positions.numel(), kv.desc.B
    if kv.block_table is not None:
        free_head_out = free_head if free_head_out is None else free_head_out
        n_pages_out = n_pages if n_pages_out is None else n_pages_out
        n_free = 0 if free_pages is None else free_pages.numel()
        pages = (_array(free_pages, "free_pages", (n_free,), i32, dev, True), n_free,
                 _array(free_head, "free_head", (1,), i32, dev), _array(n_pages, "n_pages", (B,), i32, dev))
        pages_out = (_array(free_head_out, "free_head_out", (1,), i32, dev),
                     _array(n_pages_out, "n_pages_out", (B,), i32, dev))
    else:
        pages, pages_out = (None, 0, None, None), (None, None)
    _call(kv, "plan_tokens", load().prhs_plan_tokens, stream, kv.ref(),
          _array(n_new, "n_new", (B,), i32, dev), T, _array(parents, "parents", (T,), i32, dev, True), *pages,
          _array(cu_new, "cu_new", (B + 1,), i32, dev), _array(positions, "positions", (T,), i32, dev),
          _array(slots, "slots", (T,), i32, dev),
          _array(tree_mask, "tree_mask", (T, TREE_WORDS), i32, dev, True), *pages_out)


def rope_append(kv, rope, positions, q, k, v, q_out, *, slots=None, k_out=None, stream=None) -> None:
    """Rotate q [T][Hq][d] and k [T][Hkv][d] at positions [T] into q_out and,
    where given, k_out; with slots, rotated k and v go to those rows of the
    cache (prhs_rope_append). q, k and v may be views with a token stride."""
    dev, dt, T, desc = kv.device, kv.dtype, positions.numel(), kv.desc
    Hq, Hkv, d = desc.Hq, desc.Hkv, desc.d
    if rope.turns.device != dev:
        raise ValueError(f"rope is on {rope.turns.device}, the cache on {dev}")
    if v is None and slots is not None:
        raise ValueError("v is required with slots")
    qp, qs = _rows(q, "q", T, Hq, d, dt, dev)
    kp, ks = _rows(k, "k", T, Hkv, d, dt, dev)
    vp, vs = _rows(v, "v", T, Hkv, d, dt, dev)
    _call(kv, "rope_append", load().prhs_rope_append, stream, kv.ref(), rope.ref(), T,
          _array(positions, "positions", (T,), torch.int32, dev),
          _array(slots, "slots", (T,), torch.int32, dev, True), qp, qs, kp, ks, vp, vs,
          _array(q_out, "q_out", (T, Hq, d), dt, dev), _array(k_out, "k_out", (T, Hkv, d), dt, dev, True))


def tree_workspace_size(kv: KVCache, max_new: int) -> int:
    with torch.cuda.device(kv.index):
        n = load().prhs_tree_workspace_size(kv.ref(), int(max_new))
    if n == 0:
        raise PrhsError(PRHS_EINVAL, "tree_workspace_size", load().prhs_last_message().decode())
    return n


def make_tree_workspace(kv: KVCache, max_new: int):
    """Allocate (through torch) the workspace of tree_attn for this cache and
    at most max_new tokens a sequence."""
    return torch.empty(tree_workspace_size(kv, max_new), dtype=torch.uint8, device=kv.device)


def tree_attn(kv, q, k_new, v_new, scale, cu_new, max_new, out, lse, ws, *, tree_mask=None,
              stream=None) -> None:
    """Attention of packed new tokens over their caches and each other: by
    tree_mask [T][4] int32, or causal (prhs_tree_attn). out [T][Hq][d] has the
    cache's element type, lse [T][Hq] is float32. On a bfloat16 cache the weights
    are rounded to bfloat16 before they meet v (dense_attn keeps them in float32)."""
    dev, dt, T, desc = kv.device, kv.dtype, q.shape[0], kv.desc
    Hq, Hkv, d = desc.Hq, desc.Hkv, desc.d
    kp, ks = _rows(k_new, "k_new", T, Hkv, d, dt, dev)
    vp, vs = _rows(v_new, "v_new", T, Hkv, d, dt, dev)
    if ws.device != dev:
        raise ValueError(f"ws is on {ws.device}, the cache on {dev}")
    _call(kv, "tree_attn", load().prhs_tree_attn, stream, kv.ref(), _array(q, "q", (T, Hq, d), dt, dev), kp, ks,
          vp, vs, float(scale), T, _array(cu_new, "cu_new", (desc.B + 1,), torch.int32, dev), int(max_new),
          _array(tree_mask, "tree_mask", (T, TREE_WORDS), torch.int32, dev, True),
          _array(out, "out", (T, Hq, d), dt, dev), _array(lse, "lse", (T, Hq), torch.float32, dev),
          _ptr(ws), ws.numel() * ws.element_size())


def commit_tokens(kv, cu_new, accept_n, new_lens=None, *, slots=None, accept_idx=None, k_new=None,
                  v_new=None, T=None, stream=None) -> None:
    """Write the accepted tokens' packed rows behind each cached prefix and
    advance the lengths, in place unless new_lens is given. With the slots that
    plan_tokens gave, sequences that it refused are left as they are
    (prhs_commit_planned); without, the block table alone says where the rows go
    (prhs_commit_tokens). Without k_new and v_new only the lengths advance; T
    then bounds the packed tokens (default: those of slots, or B * t_max)."""
    dev, dt, i32, desc = kv.device, kv.dtype, torch.int32, kv.desc
    B, Hkv, d = desc.B, desc.Hkv, desc.d
    if (k_new is None) != (v_new is None):
        raise ValueError("k_new and v_new must be both given or both left out")
    if T is None:
        T = (k_new.shape[0] if k_new is not None else slots.numel() if slots is not None
             else min(B * kv.t_max, ((1 << 31) - 1) // (kv.Hq + 2 * Hkv)))
    kp, ks = _rows(k_new, "k_new", T, Hkv, d, dt, dev)
    vp, vs = _rows(v_new, "v_new", T, Hkv, d, dt, dev)
    cap = 0 if accept_idx is None else accept_idx.shape[-1]
    fn, planned = load().prhs_commit_tokens, ()
    if slots is not None:
        fn, planned = load().prhs_commit_planned, (_array(slots, "slots", (T,), i32, dev),)
    _call(kv, "commit_tokens", fn, stream, kv.ref(), int(T),
          _array(cu_new, "cu_new", (B + 1,), i32, dev), *planned,
          _array(accept_idx, "accept_idx", (B, cap), i32, dev, True), cap,
          _array(accept_n, "accept_n", (B,), i32, dev), kp, ks, vp, vs,
          _array(kv.seq_lens if new_lens is None else new_lens, "new_lens", (B,), i32, dev))


def selftest_wait_timeout(limit_us: int, stream=None) -> None:
    """Run the bounded-wait self-test kernel (prhs_selftest_wait_timeout): its
    wait runs out after limit_us and sets DEV_TIMEOUT in the error word."""
    _check(load().prhs_selftest_wait_timeout(int(limit_us), _stream(stream)),
           "selftest_wait_timeout")


def last_error() -> int:
    """Synchronise, read and clear the device error word; return its bits."""
    lib = load()
    s = lib.prhs_last_error()
    if s == PRHS_EDEVICE:
        return int(lib.prhs_device_error_bits())
    _check(s, "last_error")
    return 0


def num_sms() -> int:
    return int(load().prhs_num_sms())


def launch_count() -> int:
    """Kernels the library has issued since it was loaded (prhs_launch_count)."""
    return int(load().prhs_launch_count())


def status_str(s: int) -> str:
    return load().prhs_status_str(s).decode()
