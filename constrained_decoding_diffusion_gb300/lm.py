"""The model-side operators of libfa.so (include/fa.h) on torch tensors: rotary positions, a
paged and quantised key/value cache, attention of drafted tokens over it, and beam selection
under an automaton.

Like `native`, this module only checks and marshals tensors; every operator runs in the
library's CUDA kernels on torch's current stream (or the one given).  Tensors must live on the
current device and stay alive and unchanged until the stream has passed the call; results that a call
makes on a given stream belong to that stream's memory, like tensors made under torch.cuda.stream.
"""
from __future__ import annotations

import ctypes
import math
from typing import NamedTuple, Optional

import torch

from . import native

FA_DTYPE_F32, FA_DTYPE_F16, FA_DTYPE_BF16 = 0, 1, 2
FA_CACHE_F16, FA_CACHE_BF16, FA_CACHE_E4M3 = 1, 2, 3
FA_MAX_DRAFT = 1024
FA_MAX_BEAM_TOP = 256

_DTYPE = {torch.float32: FA_DTYPE_F32, torch.float16: FA_DTYPE_F16, torch.bfloat16: FA_DTYPE_BF16}
_FORMAT = {torch.float16: FA_CACHE_F16, torch.bfloat16: FA_CACHE_BF16, torch.float8_e4m3fn: FA_CACHE_E4M3}


class _Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("format", ctypes.c_int32), ("n_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


def _lib():
    return native._lib or native.load()


_raw_stream = torch._C._cuda_getCurrentRawStream   # the current stream's handle without a Stream object


def _stream(stream, t) -> int:
    return _raw_stream(t.device.index) if stream is None else stream.cuda_stream


def _new(shape, dtype, device, stream):
    """A result of a call on a stream, from that stream's memory: the current one's may hold a freed tensor
    that its earlier kernels have yet to read or write."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _check(rc: int):
    if rc:
        native._check(rc)


# The checks below run on every call of a decoding loop, so each takes one pass over the few
# attributes it needs and leaves the wording of a refusal to _refuse.

def _refuse(t, dtype, name, shape):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    raise ValueError("%s must be contiguous" % name)


def _dtype(t, name) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    got = _DTYPE.get(t.dtype)
    if got is None:
        raise TypeError("%s must be float32, float16 or bfloat16, got %s" % (name, t.dtype))
    return got


def _ptr(t, dtype, name, shape):
    """A contiguous tensor's address after checking it; None for None."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or not t.is_cuda or not t.is_contiguous():
        _refuse(t, dtype, name, shape)
    return t.data_ptr()


def _rows(t, name, shape):
    """The strides of a tensor whose innermost dimension is contiguous."""
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    st = t.stride()
    if st[-1] != 1 and shape[-1] > 1:
        raise ValueError("%s: the innermost dimension must be contiguous" % name)
    return st


# ------------------------------------------------------------------ rotary positions

def rope_phases(rot_dim: int, base: float = 10000.0, scaling: Optional[str] = None, factor: float = 1.0,
                original_length: int = 4096, fast_turns: float = 32.0, slow_turns: float = 1.0, device="cuda"):
    """The phase table of fa_rope and the mscale that goes with it: (int64 [rot_dim / 2], float).

    Pair i turns by base^(-2i / rot_dim) radians per position.  For contexts `factor` times the
    original length, scaling is
      None      as trained
      "linear"  every angle divided by factor (interpolated positions)
      "base"    the base stretched to base * factor^(rot_dim / (rot_dim - 2)): the slowest pair is
                divided by factor, the fastest unchanged
      "blend"   pairs that make more than fast_turns turns over original_length unchanged, fewer
                than slow_turns divided by factor, linear in the number of turns between;
                mscale = 0.1 ln(factor) + 1
    A phase is the turn per position as a 64-bit fraction, its bits in an int64."""
    if rot_dim < 0 or rot_dim % 2:
        raise ValueError("rot_dim must be even")
    if scaling not in (None, "linear", "base", "blend"):
        raise ValueError("scaling must be None, 'linear', 'base' or 'blend'")
    if not (1.0 <= factor < math.inf and 0.0 < base < math.inf):
        raise ValueError("factor must be at least 1, base positive, and both finite")
    if scaling == "blend" and not fast_turns > slow_turns:
        raise ValueError("fast_turns must be above slow_turns")
    if scaling == "base" and rot_dim > 2:
        base = base * factor ** (rot_dim / (rot_dim - 2))
    got = []
    for i in range(rot_dim // 2):
        turns = base ** (-2.0 * i / rot_dim) / (2 * math.pi)
        if scaling == "linear":
            turns /= factor
        elif scaling == "blend":
            keep = (turns * original_length - slow_turns) / (fast_turns - slow_turns)
            keep = min(1.0, max(0.0, keep))
            turns = keep * turns + (1.0 - keep) * turns / factor
        bits = int(turns * 2.0 ** 64) % (1 << 64)
        got.append(bits - (1 << 64) if bits >> 63 else bits)
    mscale = 0.1 * math.log(factor) + 1.0 if scaling == "blend" else 1.0
    return torch.tensor(got, dtype=torch.int64, device=device), mscale


def fa_rope(x, positions, phase, out=None, interleaved: bool = False, mscale: float = 1.0, inverse: bool = False,
            stream=None):
    """Rotate the first 2 * len(phase) elements of every head of x [N, H, D] at positions [N];
    inverse gives the gradient of the forward call.  out defaults to a new tensor and may be x."""
    dt = _dtype(x, "x")
    if x.dim() != 3:
        raise ValueError("x must have shape [tokens, heads, dim]")
    N, H, D = x.shape
    if out is None:
        out = _new((N, H, D), x.dtype, x.device, stream)
    elif _dtype(out, "out") != dt:
        raise TypeError("out must have the type of x")
    xs, os = _rows(x, "x", x.shape), _rows(out, "out", x.shape)
    _check(_lib().fa_rope(dt, N, H, D, 2 * phase.numel(), int(interleaved), int(inverse), x.data_ptr(), xs[0], xs[1],
                                 _ptr(positions, torch.int32, "positions", (N,)),
                                 _ptr(phase, torch.int64, "phase", phase.shape), mscale, out.data_ptr(), os[0], os[1],
                                 _stream(stream, x)))
    return out


class Rope(torch.autograd.Function):
    """fa_rope with its gradient: Rope.apply(x, positions, phase, interleaved, mscale, inverse).  The map
    is linear and its transpose the inverse rotation, so the gradient is the same function and
    has derivatives of any order."""

    @staticmethod
    def forward(ctx, x, positions, phase, interleaved=False, mscale=1.0, inverse=False):
        ctx.save_for_backward(positions, phase)
        ctx.how = (interleaved, mscale, not inverse)
        return fa_rope(x, positions, phase, interleaved=interleaved, mscale=mscale, inverse=inverse)

    @staticmethod
    def backward(ctx, grad):
        positions, phase = ctx.saved_tensors
        if grad.stride(-1) != 1:   # a broadcast gradient, as of a sum
            grad = grad.contiguous()
        return Rope.apply(grad, positions, phase, *ctx.how), None, None, None, None, None


# ------------------------------------------------------------------ the cache

class KVCache(NamedTuple):
    """Paged keys and values [n_pages, kv_heads, page_size, head_dim] in float16, bfloat16 or
    float8_e4m3fn, the latter with float32 scales [n_pages, kv_heads, page_size]."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: Optional[torch.Tensor] = None
    v_scale: Optional[torch.Tensor] = None

    @classmethod
    def empty(cls, n_pages: int, kv_heads: int, page_size: int, head_dim: int, dtype=torch.float8_e4m3fn, device="cuda"):
        if dtype not in _FORMAT:
            raise TypeError("a cache is float16, bfloat16 or float8_e4m3fn, not %s" % dtype)
        shape = (n_pages, kv_heads, page_size, head_dim)
        k, v = (torch.empty(shape, dtype=dtype, device=device) for _ in range(2))
        if dtype != torch.float8_e4m3fn:
            return cls(k, v)
        return cls(k, v, *(torch.empty(shape[:3], dtype=torch.float32, device=device) for _ in range(2)))

    def describe(self) -> _Cache:
        k, v, ks, vs = self
        dtype, shape = k.dtype, k.shape
        form = _FORMAT.get(dtype)
        if form is None or len(shape) != 4:
            raise TypeError("cache pages must be float16, bfloat16 or float8_e4m3fn of shape "
                            "[n_pages, kv_heads, page_size, head_dim]")
        n, h, g, d = shape
        if form != FA_CACHE_E4M3:
            if ks is not None or vs is not None:
                raise ValueError("a 16-bit cache has no scales")
            return _Cache(_ptr(k, dtype, "cache.k", shape), _ptr(v, dtype, "cache.v", shape), None, None, form, n, g, h, d)
        if ks is None or vs is None:
            raise ValueError("an 8-bit cache has scales")
        rows = (n, h, g)
        return _Cache(_ptr(k, dtype, "cache.k", shape), _ptr(v, dtype, "cache.v", shape),
                      _ptr(ks, torch.float32, "cache.k_scale", rows), _ptr(vs, torch.float32, "cache.v_scale", rows), form, n, g, h, d)


def fa_cache_write(cache: KVCache, k, v, page_table, start, count=None, positions=None, phase=None,
                   interleaved: bool = False, mscale: float = 1.0, stream=None):
    """Store k, v [B, T, kv_heads, head_dim] in the slots start[b] + j, j < count[b], the keys
    rotated at positions [B, T] first when given with a phase table."""
    c = cache.describe()
    dt = _dtype(k, "k")
    if k.dim() != 4 or _dtype(v, "v") != dt:
        raise ValueError("k and v must have shape [batch, tokens, heads, dim] and one type")
    B, T = k.shape[:2]
    shape = (B, T, c.kv_heads, c.head_dim)
    ks, vs = _rows(k, "k", shape), _rows(v, "v", shape)
    P = page_table.shape[1]
    _check(_lib().fa_cache_write(
        ctypes.byref(c), dt, B, T, k.data_ptr(), ks[0], ks[1], ks[2], v.data_ptr(), vs[0], vs[1], vs[2],
        _ptr(page_table, torch.int32, "page_table", (B, P)), P, _ptr(start, torch.int32, "start", (B,)),
        _ptr(count, torch.int32, "count", (B,)), _ptr(positions, torch.int32, "positions", (B, T)),
        None if phase is None else _ptr(phase, torch.int64, "phase", phase.shape), 0 if phase is None else 2 * phase.numel(),
        int(interleaved), mscale, _stream(stream, k)))


def fa_cache_read(cache: KVCache, page_table, length, k_out, v_out, stream=None):
    """Slots [0, length[b]) back into k_out, v_out [B, N, kv_heads, head_dim]; zeros past them."""
    c = cache.describe()
    dt = _dtype(k_out, "k_out")
    B, N = k_out.shape[:2]
    shape = (B, N, c.kv_heads, c.head_dim)
    P = page_table.shape[1]
    _check(_lib().fa_cache_read(
        ctypes.byref(c), dt, B, N, _ptr(page_table, torch.int32, "page_table", (B, P)), P,
        _ptr(length, torch.int32, "length", (B,)), _ptr(k_out, k_out.dtype, "k_out", shape),
        _ptr(v_out, k_out.dtype, "v_out", shape), _stream(stream, k_out)))
    return k_out, v_out


def fa_cache_keep(cache: KVCache, page_table, length, path, stream=None):
    """Move the slots length[b] + path[b, i] of an accepted path (ascending, ended by -1) to
    length[b] + i."""
    c = cache.describe()
    B, P = page_table.shape
    n = path.shape[1]
    _check(_lib().fa_cache_keep(ctypes.byref(c), B, n, _ptr(page_table, torch.int32, "page_table", (B, P)), P,
                                       _ptr(length, torch.int32, "length", (B,)), _ptr(path, torch.int32, "path", (B, n)),
                                       _stream(stream, path)))


# ------------------------------------------------------------------ attention of drafted tokens

def fa_tree_mask(parents, mask=None, depth=None, stream=None):
    """The mask words [B, T, ceil(T / 64)] int64 and depths [B, T] of the trees parents [B, T]."""
    B, T = parents.shape
    if mask is None:
        mask = _new((B, T, (T + 63) // 64), torch.int64, parents.device, stream)
    if depth is None:
        depth = _new((B, T), torch.int32, parents.device, stream)
    _check(_lib().fa_tree_mask(B, T, _ptr(parents, torch.int32, "parents", (B, T)),
                                      _ptr(mask, torch.int64, "mask", (B, T, (T + 63) // 64)),
                                      _ptr(depth, torch.int32, "depth", (B, T)), _stream(stream, parents)))
    return mask, depth


class TreeAttention:
    """Owner of the workspace and outputs of fa_tree_attention for a fixed (B, T, heads, dim).  A call
    returns the owner's own tensors, which the next one overwrites."""

    def __init__(self, B: int, T: int, q_heads: int, kv_heads: int, head_dim: int, dtype=torch.bfloat16, device="cuda"):
        n = ctypes.c_size_t()
        native.load()
        _check(_lib().fa_tree_attention_workspace_bytes(B, T, q_heads, kv_heads, head_dim, ctypes.byref(n)))
        self.shape = (B, T, q_heads, head_dim)
        self.ws_bytes = n.value
        self.workspace = torch.empty(max(n.value, 256), dtype=torch.uint8, device=device)
        self.out = torch.empty(self.shape, dtype=dtype, device=device)
        self.lse = torch.empty((B, T, q_heads), dtype=torch.float32, device=device)

    def __call__(self, q, cache: KVCache, page_table, length, mask=None, count=None, scale: Optional[float] = None,
                 stream=None):
        """Attention of q [B, T, q_heads, head_dim] over the cache: (out, lse).  length [B] slots
        come before the draft, count [B] of the T drafted tokens are in use, mask as made by
        fa_tree_mask (None: every drafted token sees all of them); scale defaults to
        head_dim ** -0.5."""
        B, T, H, D = self.shape
        c = cache.describe()
        dt = _dtype(q, "q")
        if q.dtype != self.out.dtype:
            raise TypeError("q must be %s, got %s" % (self.out.dtype, q.dtype))
        if c.head_dim != D:
            raise ValueError("the cache's head_dim is %d, not %d" % (c.head_dim, D))
        sb, st, sh = _rows(q, "q", self.shape)[:3]
        if B == 1 or T == 1 or H == 1:   # the stride of a single element means nothing, and torch makes any
            sb, st, sh = sb if B > 1 else 0, st if T > 1 else 0, sh if H > 1 else 0
        P = page_table.shape[1]
        _check(_lib().fa_tree_attention(
            ctypes.byref(c), dt, B, T, H, q.data_ptr(), sb, st, sh,
            _ptr(page_table, torch.int32, "page_table", (B, P)), P, _ptr(length, torch.int32, "length", (B,)),
            _ptr(count, torch.int32, "count", (B,)), _ptr(mask, torch.int64, "mask", (B, T, (T + 63) // 64)),
            D ** -0.5 if scale is None else scale, self.out.data_ptr(), self.lse.data_ptr(), self.workspace.data_ptr(),
            self.ws_bytes, _stream(stream, q)))
        return self.out, self.lse


# ------------------------------------------------------------------ beams

def fa_beam_tables(aut: native.CompiledAutomaton, stream=None):
    """The next-state table [S, V] int16 and the live bits [S, ceil(V / 32)] int32 of a DFA,
    without the moves from which no accepting state can be reached."""
    S, V = aut.n_states, aut.vocab
    nxt = _new((S, V), torch.int16, "cuda", stream)
    live = _new((S, (V + 31) // 32), torch.int32, "cuda", stream)
    _check(_lib().fa_beam_tables(aut.handle, nxt.data_ptr(), live.data_ptr(), _stream(stream, nxt)))
    return nxt, live


class BeamSelect:
    """Owner of the workspace and outputs of fa_beam_select for a fixed (N, K, V, top).  A call
    returns the owner's own tensors, which the next one overwrites; with K == top they may be its
    scores and states."""

    def __init__(self, N: int, K: int, V: int, top: int, dtype=torch.float32, device="cuda"):
        n = ctypes.c_size_t()
        native.load()
        _check(_lib().fa_beam_select_workspace_bytes(N, K, V, top, ctypes.byref(n)))
        self.N, self.K, self.V, self.top, self.dtype = N, K, V, top, dtype
        self.workspace = torch.empty(max(n.value, 256), dtype=torch.uint8, device=device)
        self.score = torch.empty((N, top), dtype=torch.float32, device=device)
        self.parent, self.token, self.state = (torch.empty((N, top), dtype=torch.int32, device=device) for _ in range(3))

    def __call__(self, logp, scores, states=None, next=None, live=None, stream=None):
        """The best cells of scores [N, K] + logp [N, K, V]: (score, parent, token, state), state
        None without an automaton (states [N, K], next and live as from fa_beam_tables)."""
        N, K, V = self.N, self.K, self.V
        dt = _dtype(logp, "logp")
        if logp.dtype != self.dtype:
            raise TypeError("logp must be %s, got %s" % (self.dtype, logp.dtype))
        st = _rows(logp, "logp", (N, K, V))
        S = 0 if next is None else next.shape[0]
        _check(_lib().fa_beam_select(
            dt, N, K, V, self.top, logp.data_ptr(), st[0], st[1], _ptr(scores, torch.float32, "scores", (N, K)),
            _ptr(states, torch.int32, "states", (N, K)), S, _ptr(next, torch.int16, "next", (S, V)),
            _ptr(live, torch.int32, "live", (S, (V + 31) // 32)), self.score.data_ptr(), self.parent.data_ptr(),
            self.token.data_ptr(), self.state.data_ptr() if S else None, self.workspace.data_ptr(), self.workspace.numel(),
            _stream(stream, logp)))
        return self.score, self.parent, self.token, self.state if S else None


def fa_beam_reorder(src, parent, dst=None, token=None, at: int = 0, stream=None):
    """Row parent[n, k] of src [N, K, W] int32 as row k of dst [N, top, W] (-1 where there is no
    parent); with token [N, top] word `at` of each row becomes its token."""
    N, K, W = src.shape
    top = parent.shape[1]
    if dst is None:
        dst = _new((N, top, W), torch.int32, src.device, stream)
    _check(_lib().fa_beam_reorder(N, K, top, W, _ptr(src, torch.int32, "src", (N, K, W)),
                                         _ptr(parent, torch.int32, "parent", (N, top)),
                                         _ptr(token, torch.int32, "token", (N, top)), int(at),
                                         _ptr(dst, torch.int32, "dst", (N, top, W)), _stream(stream, src)))
    return dst
