"""Binding of the paged KV cache operators (include/pred.h, "the paged KV cache").

As in the package's other calls, the functions carry the C names and only
marshal arguments.  ``KVCache`` and ``Rope`` describe a cache and a rotation once,
for all the calls of a program that keeps them.
"""

import ctypes

import numpy as np

from . import _lib
from ._lib import PredKvCache, PredRope, PredRopeScaling

_KINDS = {"none": _lib.PRED_ROPE_NONE, "linear": _lib.PRED_ROPE_LINEAR, "ntk": _lib.PRED_ROPE_NTK,
          "llama3": _lib.PRED_ROPE_LLAMA3, "yarn": _lib.PRED_ROPE_YARN}

# torch and the dtypes a tensor may have, from the first call that takes tensors on (the package itself needs none)
torch = _BF16 = _FP8 = _WORD = _I32 = _F32 = _current_raw = None


def _load_torch():
    global torch, _BF16, _FP8, _WORD, _I32, _F32, _current_raw
    import torch as t
    _BF16 = (t.bfloat16, t.int16, t.uint16)
    _FP8 = (t.float8_e4m3fn, t.uint8)
    _WORD = (t.int64, t.uint64)
    _I32, _F32 = (t.int32,), (t.float32,)
    _current_raw = getattr(t._C, "_cuda_getCurrentRawStream", None)
    torch = t


def _pkg():
    import rank_kv_block_amd
    return rank_kv_block_amd


def _check(rc):
    if rc:
        rk = _pkg()
        raise rk.PredError(rc, rk.pred_last_error())
    return rc


def _dims(h):
    d = getattr(h, "dims", None)
    return _pkg().pred_get_dims(h) if d is None else d


def _raw_stream(stream, device):
    """The stream's handle (the current one's without making a Stream object of it, 2.5 us of a 10 us call)."""
    if stream is None:
        return _current_raw(device) if _current_raw else torch.cuda.current_stream(device).cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


class _Args:
    """Pointer checks of one call: every tensor on the current device."""

    __slots__ = ("device",)

    def __init__(self):
        if torch is None:
            _load_torch()
        self.device = torch.cuda.current_device()

    def _place(self, t, what, dtypes):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{what}: expected a torch.Tensor")
        if t.dtype not in dtypes:
            raise TypeError(f"{what}: dtype {t.dtype} not in {dtypes}")
        if t.get_device() != self.device:
            raise ValueError(f"{what}: tensor must live on the current GPU ({self.device}), not on {t.device}")

    def ptr(self, t, what, dtypes, shape):
        """Device pointer of a contiguous tensor of this shape (None -> NULL)."""
        if t is None:
            return None
        self._place(t, what, dtypes)
        if t.shape != shape:
            raise ValueError(f"{what} must be {list(shape)}, not {list(t.shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{what}: tensor must be contiguous")
        return t.data_ptr()

    def rows(self, t, what, n, heads, dim):
        """(pointer, token stride) of [n, heads, dim] bf16 whose tokens may lie apart."""
        self._place(t, what, _BF16)
        if t.shape != (n, heads, dim):
            raise ValueError(f"{what} must be [{n}, {heads}, {dim}], not {list(t.shape)}")
        if n and heads and ((dim > 1 and t.stride(2) != 1) or (heads > 1 and t.stride(1) != dim)):
            raise ValueError(f"{what}: a token's heads must be contiguous")
        return t.data_ptr(), t.stride(0) if n > 1 else heads * dim

    def buffer(self, t, what):
        """(pointer, bytes) of a workspace."""
        if t is None:
            return None, 0
        if not isinstance(t, torch.Tensor) or t.get_device() != self.device or not t.is_contiguous():
            raise ValueError(f"{what} must be a contiguous tensor on the current GPU")
        return t.data_ptr(), t.numel() * t.element_size()


class KVCache:
    """One layer's paged cache: ``k`` and ``v`` [max_blocks, block_size, num_kv_heads, head_dim], bf16 or e4m3
    (float8_e4m3fn or uint8), views with equal strides whose last dimension is contiguous.  An element stands for
    ``k_scale`` (``v_scale``) times what is stored; a bf16 cache has scales of 1.  Keeps the tensors alive."""

    __slots__ = ("k", "v", "shape", "device", "_struct", "_ref")

    def __init__(self, k, v, k_scale=1.0, v_scale=1.0):
        if torch is None:
            _load_torch()
        for t, what in ((k, "k"), (v, "v")):
            if not isinstance(t, torch.Tensor) or t.dim() != 4:
                raise TypeError(f"{what}: expected a tensor [max_blocks, block_size, num_kv_heads, head_dim]")
            if t.device.type != "cuda":
                raise ValueError(f"{what}: tensor must live on the GPU")
            if t.dtype not in _BF16 + _FP8:
                raise TypeError(f"{what}: dtype {t.dtype} not in {_BF16 + _FP8}")
        if k.shape != v.shape or k.stride() != v.stride() or k.dtype != v.dtype or k.device != v.device:
            raise ValueError("k and v must have one shape, one dtype, one device and the same strides")
        if k.shape[3] > 1 and k.stride(3) != 1:
            raise ValueError("the last dimension must be contiguous")
        self.k, self.v, self.shape, self.device = k, v, tuple(k.shape), k.get_device()
        n, block, heads, dim = self.shape
        # a dimension of one element is never stepped over, whatever its stride says
        token = k.stride(1) if block > 1 else max(dim, heads * k.stride(2) if heads > 1 else dim)
        head = k.stride(2) if heads > 1 else max(dim, dim if block == 1 else block * token)
        extent = (block - 1) * token + (heads - 1) * head + dim
        stride = k.stride(0) if n > 1 else -(-extent // 16) * 16
        self._struct = PredKvCache(k.data_ptr(), v.data_ptr(), stride, token, head,
                                   _lib.PRED_KV_FP8 if k.dtype in _FP8 else _lib.PRED_KV_BF16, k_scale, v_scale)
        self._ref = ctypes.byref(self._struct)

    def _of(self, d, args):
        if self.shape != (d.max_blocks, d.block_size, d.num_kv_heads, d.head_dim):
            raise ValueError(f"the cache must be [{d.max_blocks}, {d.block_size}, {d.num_kv_heads}, {d.head_dim}], "
                             f"not {list(self.shape)}")
        if self.device != args.device:
            raise ValueError(f"the cache must live on the current GPU ({args.device}), not on {self.device}")
        return self._ref


class Rope:
    """A rotation: ``turns`` is the GPU copy ([rot_dim / 2] int64 or uint64) of pred_rope_turns's output."""

    __slots__ = ("turns", "rot_dim", "device", "_struct", "_ref")

    def __init__(self, turns, rot_dim, interleaved=False, mscale=1.0, backward=False):
        if torch is None:
            _load_torch()
        if not isinstance(turns, torch.Tensor) or turns.dtype not in _WORD or turns.device.type != "cuda":
            raise TypeError("turns: expected an int64 or uint64 tensor on the GPU")
        if turns.shape != (rot_dim // 2,) or not turns.is_contiguous():
            raise ValueError(f"turns must be contiguous [{rot_dim // 2}], not {list(turns.shape)}")
        self.turns, self.rot_dim, self.device = turns, rot_dim, turns.get_device()
        self._struct = PredRope(turns.data_ptr(), rot_dim, bool(interleaved), bool(backward), mscale)
        self._ref = ctypes.byref(self._struct)

    def _on(self, args):
        if self.device != args.device:
            raise ValueError(f"turns must live on the current GPU ({args.device}), not on {self.device}")
        return self._ref


def pred_rope_turns(rot_dim, theta, kind="none", factor=1.0, low=0.0, high=0.0, original_length=0.0):
    """(turns, mscale): a rotation's frequencies as uint64 fractions of a turn a position [rot_dim / 2], and the factor
    on its cosines and sines.  ``kind``: "none", "linear", "ntk", "llama3", "yarn" or a PRED_ROPE_* value."""
    if isinstance(kind, str):
        if kind not in _KINDS:
            raise ValueError(f"kind {kind!r} is not one of {sorted(_KINDS)}")
        kind = _KINDS[kind]
    out = np.zeros(max(rot_dim // 2, 1), np.uint64)
    mscale = ctypes.c_float()
    _check(_lib.load().pred_rope_turns(rot_dim, theta, ctypes.byref(PredRopeScaling(kind, factor, low, high,
                                                                                    original_length)),
                                       out.ctypes.data_as(ctypes.c_void_p), ctypes.byref(mscale)))
    return out, mscale.value


def pred_rotate(h, rope, x, positions, out, stream=None):
    """x [n_tokens, n_heads, head_dim] bf16 (tokens may lie apart) rotated to its positions [n_tokens] int32 into out
    (x itself for in place)."""
    d, a = _dims(h), _Args()
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise TypeError("x: expected a tensor [n_tokens, n_heads, head_dim]")
    n, heads = x.shape[0], x.shape[1]
    xp, xs = a.rows(x, "x", n, heads, d.head_dim)
    op, os_ = a.rows(out, "out", n, heads, d.head_dim)
    _check(_lib.load().pred_rotate(h, rope._on(a), xp, xs, n, heads, a.ptr(positions, "positions", _I32, (n,)),
                                   op, os_, _raw_stream(stream, a.device)))


def pred_rotate_store(h, rope, q, k, v, positions, slots, cache, q_out, stream=None):
    """q, k, v [n_tokens, heads, head_dim] bf16 (tokens may lie apart): q and k rotated to positions [n_tokens] int32,
    q into q_out, k and v into the cache at slots [n_tokens] int64 (block * block_size + offset, -1: none)."""
    d, a = _dims(h), _Args()
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise TypeError("q: expected a tensor [n_tokens, num_q_heads, head_dim]")
    n = q.shape[0]
    qp, qs = a.rows(q, "q", n, d.num_q_heads, d.head_dim)
    kp, ks = a.rows(k, "k", n, d.num_kv_heads, d.head_dim)
    vp, vs = a.rows(v, "v", n, d.num_kv_heads, d.head_dim)
    _check(_lib.load().pred_rotate_store(
        h, rope._on(a), qp, qs, kp, ks, vp, vs, n, a.ptr(positions, "positions", _I32, (n,)),
        a.ptr(slots, "slots", _WORD[:1], (n,)), cache._of(d, a),
        a.ptr(q_out, "q_out", _BF16, (n, d.num_q_heads, d.head_dim)), _raw_stream(stream, a.device)))


def pred_attend_workspace_bytes(h, n_seqs, n_rows, n_blocks):
    return _lib.load().pred_attend_workspace_bytes(h, n_seqs, n_rows, n_blocks)


def pred_attend_kernel_name(h, cache, n_rows=1, with_block_lse=False):
    """The kernel pred_attend runs for this handle, cache and rows per sequence."""
    name = _lib.load().pred_attend_kernel_name(h, cache._ref, n_rows, bool(with_block_lse))
    if name is None:
        rk = _pkg()
        raise rk.PredError(rk.PRED_ERR_NULL_ARG if not h else rk.PRED_ERR_OUT_OF_RANGE, rk.pred_last_error())
    return name.decode()


def pred_attend(h, cache, q, tree, block_tables, kv_len, draft_len, scale, out, lse=None, block_lse=None,
                workspace=None, n_blocks=None, stream=None):
    """Attention of each sequence's newest tokens: q [n_seqs, n_rows, num_q_heads, head_dim] bf16 -> out alike.
    tree [n_seqs, n_rows] int64 words or None (a chain); block_tables [n_seqs, n_blocks] int32, or None for the identity
    over n_blocks blocks (default: all of the cache's); kv_len, draft_len [n_seqs] int32 or None; lse [n_seqs, n_rows,
    num_q_heads] and block_lse [n_seqs, n_blocks, n_rows, num_q_heads] float32 outputs or None."""
    d, a = _dims(h), _Args()
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise TypeError("q: expected a tensor [n_seqs, n_rows, num_q_heads, head_dim]")
    S, M = q.shape[0], q.shape[1]
    if block_tables is not None:
        if not isinstance(block_tables, torch.Tensor):
            raise TypeError("block_tables: expected a torch.Tensor")
        if block_tables.dim() != 2:
            raise ValueError("block_tables must be [n_seqs, n_blocks]")
        n_blocks = block_tables.shape[1]
    elif n_blocks is None:
        n_blocks = d.max_blocks
    shape = (S, M, d.num_q_heads, d.head_dim)
    ws, ws_bytes = a.buffer(workspace, "workspace")
    _check(_lib.load().pred_attend(
        h, cache._of(d, a), a.ptr(q, "q", _BF16, shape), M, a.ptr(tree, "tree", _WORD, (S, M)),
        a.ptr(block_tables, "block_tables", _I32, (S, n_blocks)), n_blocks, S, a.ptr(kv_len, "kv_len", _I32, (S,)),
        a.ptr(draft_len, "draft_len", _I32, (S,)), scale, a.ptr(out, "out", _BF16, shape),
        a.ptr(lse, "lse", _F32, shape[:3]), a.ptr(block_lse, "block_lse", _F32, (S, n_blocks, M, d.num_q_heads)),
        ws, ws_bytes, _raw_stream(stream, a.device)))


def pred_accumulate_weight(h, lse, block_lse, accepted, kv_len, decay, mass, mass_out=None, stream=None):
    """mass_out = decay * mass + each block's share of the accepted rows' attention: lse [n_seqs, n_rows, num_q_heads],
    block_lse [n_seqs, n_blocks, n_rows, num_q_heads] from pred_attend; accepted [n_seqs] int64 row bits or None;
    kv_len [n_seqs] int32 or None; mass, mass_out [n_seqs, n_blocks] float32 (mass_out None: in place)."""
    d, a = _dims(h), _Args()
    if not isinstance(block_lse, torch.Tensor) or block_lse.dim() != 4:
        raise TypeError("block_lse: expected a tensor [n_seqs, n_blocks, n_rows, num_q_heads]")
    S, n, M = block_lse.shape[:3]
    mass_ptr = a.ptr(mass, "mass", _F32, (S, n))
    _check(_lib.load().pred_accumulate_weight(
        h, a.ptr(lse, "lse", _F32, (S, M, d.num_q_heads)), a.ptr(block_lse, "block_lse", _F32, (S, n, M, d.num_q_heads)),
        M, a.ptr(accepted, "accepted", _WORD, (S,)), a.ptr(kv_len, "kv_len", _I32, (S,)), n, S, decay,
        mass_ptr, mass_ptr if mass_out is None else a.ptr(mass_out, "mass_out", _F32, (S, n)), _raw_stream(stream, a.device)))


def pred_evict_workspace_bytes(n_blocks, n_seqs):
    return _lib.load().pred_evict_workspace_bytes(n_blocks, n_seqs)


def pred_evict_blocks(h, block_tables, mass, kv_len, budget, protect_first, protect_last, tables_out, mass_out,
                      kv_len_out, evicted, workspace=None, stream=None):
    """Each sequence trimmed to `budget` blocks: the lowest-mass blocks outside the first protect_first and last
    protect_last moved behind the kept ones.  block_tables, tables_out [n_seqs, n_blocks] int32, mass, mass_out alike
    float32, kv_len, kv_len_out, evicted [n_seqs] int32; an output may be its input."""
    a = _Args()
    if not isinstance(block_tables, torch.Tensor) or block_tables.dim() != 2:
        raise TypeError("block_tables: expected a tensor [n_seqs, n_blocks]")
    shape = tuple(block_tables.shape)
    S, n = shape
    ws, ws_bytes = a.buffer(workspace, "workspace")
    _check(_lib.load().pred_evict_blocks(
        h, a.ptr(block_tables, "block_tables", _I32, shape), a.ptr(mass, "mass", _F32, shape),
        a.ptr(kv_len, "kv_len", _I32, (S,)), n, S, budget, protect_first, protect_last,
        a.ptr(tables_out, "tables_out", _I32, shape), a.ptr(mass_out, "mass_out", _F32, shape),
        a.ptr(kv_len_out, "kv_len_out", _I32, (S,)), a.ptr(evicted, "evicted", _I32, (S,)), ws, ws_bytes,
        _raw_stream(stream, a.device)))
