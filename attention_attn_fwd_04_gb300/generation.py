"""Generation next to the fused attention: rotary positions, a paged
key/value cache and the attention of one new token per request over it.

Argument marshalling only, like the rest of the binding: every step runs in
``libattn_gb300.so`` (``include/attn.h`` has the formulas and the rules).
The calls of a decode step take a few microseconds on the GPU, so tensors are
read and made by a small compiled module (``csrc/generation_binding.cpp``)
instead of from Python.
All calls are asynchronous on ``stream`` (default: the current stream of the
tensors' device).  With ``stream`` given, the tensors a call creates belong to
that stream.  No call records autograd history: the gradient of :func:`rope`
is :func:`rope_bwd`, to be called from the caller's own backward pass.  Tensors
that a call writes into get a new version, as by torch's in-place operations.

A step of a server, with caches seen as ``[num_pages, H_kv, page_size, D]``
(any strides whose rows are contiguous):

    plan = rope_plan(128, base=500000.0)
    m = cache_slots(ctx, new, table, free_pages, n_free, page_size=64,
                    num_pages=num_pages, max_tokens=max_tokens)
    q = cache_append(k, v, k_cache, v_cache, m.slots, q=q, plan=plan,
                     positions=m.positions)
    o, lse = attn_decode(q, k_cache, v_cache, table, m.seq_lens)

That is a step in which every request adds one token, so token b is request
b's.  Where some pause (``new`` 0) or the step is padded to ``max_tokens``, the
tokens stand closer together than the requests, and the attention takes each
token's request's row:

    r = m.token_req.clamp(min=0).long()
    o, lse = attn_decode(q, k_cache, v_cache, table[r],
                         torch.where(m.token_req >= 0, m.seq_lens[r], 0))
"""
from __future__ import annotations

import ctypes
import math
from typing import NamedTuple, Optional, Sequence

import torch

from . import _check, _lib

ROPE_MAX_DIM = 256
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {None: 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4, "custom": 5}


class RopeConfig(ctypes.Structure):
    """Mirror of ``attn_rope_config``."""

    _fields_ = [("version", ctypes.c_uint32), ("rot_dim", ctypes.c_int32),
                ("layout", ctypes.c_int32), ("scaling", ctypes.c_int32)] + \
        [(n, ctypes.c_double) for n in ("base", "factor", "original_len", "beta_fast",
                                        "beta_slow", "low_factor", "high_factor", "mscale")] + \
        [("inv_freq", ctypes.c_void_p)]


class RopePlanStruct(ctypes.Structure):
    """Mirror of ``attn_rope_plan``."""

    _fields_ = [("version", ctypes.c_uint32), ("rot_dim", ctypes.c_int32),
                ("layout", ctypes.c_int32), ("mscale", ctypes.c_float),
                ("turns", ctypes.c_uint64 * (ROPE_MAX_DIM // 2))]


class CacheDesc(ctypes.Structure):
    """Mirror of ``attn_cache_desc``."""

    _fields_ = [("version", ctypes.c_uint32), ("dtype", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("H_kv", ctypes.c_int32), ("D", ctypes.c_int32),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_strides", ctypes.c_int64 * 3), ("v_strides", ctypes.c_int64 * 3),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)]


class RopePlan:
    """A rotation plan (host memory; make it once per model)."""

    def __init__(self, struct: RopePlanStruct):
        self._struct = struct
        self._ref = ctypes.byref(struct)
        self._at = ctypes.addressof(struct)

    @property
    def rot_dim(self) -> int:
        return self._struct.rot_dim

    @property
    def layout(self) -> str:
        return "interleaved" if self._struct.layout else "half"

    @property
    def mscale(self) -> float:
        return self._struct.mscale

    def inv_freq(self) -> list:
        """Radians per position of every pair, as the kernels use them
        (modulo one turn)."""
        return [self._struct.turns[i] * (2.0 * math.pi / 2.0 ** 64)
                for i in range(self.rot_dim // 2)]


class CacheSlots(NamedTuple):
    """What :func:`cache_slots` returns."""

    seq_lens: torch.Tensor   # int32 [B]: tokens of each request after the step
    cu_new: torch.Tensor     # int32 [B + 1]: new tokens before each request
    token_req: torch.Tensor  # int32 [max_tokens]: request of each new token, -1 behind the last
    positions: torch.Tensor  # int32 [max_tokens]
    slots: torch.Tensor      # int64 [max_tokens], -1 behind the last
    n_free: Optional[torch.Tensor]  # int32 [1]: free pages left


def rope_plan(rot_dim: int, *, base: float = 10000.0, layout: str = "half",
              scaling: Optional[str] = None, factor: float = 1.0, original_len: float = 0.0,
              beta_fast: float = 32.0, beta_slow: float = 1.0, low_factor: float = 1.0,
              high_factor: float = 4.0, mscale: Optional[float] = None,
              inv_freq: Optional[Sequence[float]] = None) -> RopePlan:
    """Plan of a rotation of the first ``rot_dim`` elements of each head.
    ``layout``: ``"half"`` pairs (i, i + rot_dim / 2), ``"interleaved"``
    (2 i, 2 i + 1).  ``scaling``: None, ``"linear"``, ``"ntk"``, ``"yarn"``,
    ``"bands"`` (with ``factor``, and ``original_len`` for the last two) or
    own frequencies in ``inv_freq``.  ``mscale`` multiplies cos and sin."""
    if layout not in ROPE_LAYOUTS:
        raise ValueError("layout must be one of %s" % sorted(ROPE_LAYOUTS))
    if inv_freq is not None:
        if scaling not in (None, "custom"):
            raise ValueError("inv_freq takes no other scaling")
        scaling = "custom"
    if scaling not in ROPE_SCALINGS:
        raise ValueError("scaling must be one of %s" % sorted(map(str, ROPE_SCALINGS)))
    if mscale is not None and not mscale > 0:
        raise ValueError("mscale must be > 0")
    # a 0 means the default in the C structure; here it was given
    read = dict(custom=(), yarn=("base", "beta_fast", "beta_slow"),
                bands=("base", "low_factor", "high_factor")).get(scaling, ("base",))
    given = dict(base=base, beta_fast=beta_fast, beta_slow=beta_slow, low_factor=low_factor,
                 high_factor=high_factor)
    for name in read:
        if given[name] == 0:
            raise ValueError("%s must not be 0" % name)
    c = RopeConfig(version=1, rot_dim=int(rot_dim), layout=ROPE_LAYOUTS[layout],
                   scaling=ROPE_SCALINGS[scaling], base=float(base), factor=float(factor),
                   original_len=float(original_len), beta_fast=float(beta_fast),
                   beta_slow=float(beta_slow), low_factor=float(low_factor),
                   high_factor=float(high_factor), mscale=0.0 if mscale is None else float(mscale))
    if inv_freq is not None:
        f = [float(x) for x in inv_freq]
        if len(f) != int(rot_dim) // 2:
            raise ValueError("inv_freq must hold rot_dim / 2 frequencies")
        arr = (ctypes.c_double * max(1, len(f)))(*f)
        c.inv_freq = ctypes.addressof(arr)
    p = RopePlanStruct()
    _check(_lib.attn_rope_plan_init(ctypes.byref(c), ctypes.byref(p)), "attn_rope_plan_init")
    return RopePlan(p)


# ---------------------------------------------------------------- helpers ----

class _LazyNative:
    """The compiled module, imported on first use (after ``_lib``'s library,
    which it links against).  A missing module raises."""

    def __getattr__(self, name):
        _lib.attn_abi_version  # raises when the library is missing
        try:
            from . import _generation
        except ImportError as e:
            raise ImportError("the generation binding is not built (%s). Build it with `python -m "
                              "attention_attn_fwd_04_gb300.build`." % e) from e
        for f in ("rope", "slots", "append", "decode"):  # found directly from now on
            setattr(self, f, getattr(_generation, f))
        return getattr(_generation, name)


_native = _LazyNative()


def _on(stream, t: torch.Tensor):
    """``stream`` as the current one, for the allocations and the call."""
    if stream.device != t.device:
        raise ValueError("stream and tensors must be on one device")
    return torch.cuda.stream(stream)


# ------------------------------------------------------------------- rope ----

def rope(x: torch.Tensor, plan: RopePlan, positions: Optional[torch.Tensor] = None, *,
         offset: int = 0, out: Optional[torch.Tensor] = None,
         stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Rotary positions of ``x`` [B, H, S, D] (bf16, any strides with
    contiguous rows): token s of batch b is at ``positions[b, s] + offset``
    (int32 [S] or [B, S]; default s).  ``out`` may be ``x``.  The result has no
    autograd history; :func:`rope_bwd` is the gradient."""
    if stream is not None:
        with _on(stream, x):
            return rope(x, plan, positions, offset=offset, out=out)
    r = _native.rope(False, x, plan._at, positions, offset, out)
    if type(r) is int:
        _check(r, "attn_rope")
    return r


def rope_bwd(dout: torch.Tensor, plan: RopePlan, positions: Optional[torch.Tensor] = None, *,
             offset: int = 0, out: Optional[torch.Tensor] = None,
             stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Gradient of :func:`rope` with respect to ``x`` for the upstream
    gradient ``dout``; arguments as there.  ``out`` may be ``dout``."""
    if stream is not None:
        with _on(stream, dout):
            return rope_bwd(dout, plan, positions, offset=offset, out=out)
    r = _native.rope(True, dout, plan._at, positions, offset, out)
    if type(r) is int:
        _check(r, "attn_rope_bwd")
    return r


# ------------------------------------------------------------------ cache ----

def cache_slots(ctx_lens: torch.Tensor, new_lens: torch.Tensor, block_table: torch.Tensor,
                free_pages: Optional[torch.Tensor] = None,
                n_free: Optional[torch.Tensor] = None, *, page_size: int, num_pages: int,
                max_tokens: int, out: Optional[CacheSlots] = None,
                stream: Optional[torch.cuda.Stream] = None) -> CacheSlots:
    """Slot map of a step in which request b, holding ``ctx_lens[b]`` tokens,
    adds ``new_lens[b]`` (int32 [B]).  Pages that the new tokens need come off
    the end of ``free_pages[:n_free]`` (int32; ``n_free`` int32 [1]) and are
    written into ``block_table`` (int32 [B, max_pages]); without
    ``free_pages`` the table must name them already.  ``out``: tensors of an
    earlier call to write into; its ``seq_lens`` may be ``ctx_lens`` and its
    ``n_free`` may be ``n_free``.  Without it the outputs are parts of one
    allocation: keeping (or saving) one keeps all.  A step that cannot be
    served adds nothing and is reported by :func:`get_device_status`."""
    if stream is not None:
        with _on(stream, block_table):
            return cache_slots(ctx_lens, new_lens, block_table, free_pages, n_free,
                               page_size=page_size, num_pages=num_pages, max_tokens=max_tokens,
                               out=out)
    r = _native.slots(ctx_lens, new_lens, block_table, free_pages, n_free, page_size, num_pages,
                      max_tokens, out)
    if type(r) is int:
        _check(r, "attn_cache_slots")
    return r if out is not None else CacheSlots._make(r)


def cache_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                 slots: torch.Tensor, *, q: Optional[torch.Tensor] = None,
                 q_out: Optional[torch.Tensor] = None, plan: Optional[RopePlan] = None,
                 positions: Optional[torch.Tensor] = None,
                 k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None) -> Optional[torch.Tensor]:
    """Write new keys and values ``k``, ``v`` [T, H_kv, D] (bf16, any strides
    with contiguous rows, such as parts of one projection's output) into the
    slots (int64 [T], below 0: nowhere) of caches [num_pages, H_kv, page_size,
    D] (bf16, or float8_e4m3fn with float32 [H_kv] scales, stored value =
    value / scale).  With ``plan`` the keys, and the queries ``q`` [T, H, D]
    if given, are rotated to ``positions`` (int32 [T]) on the way; the
    queries go to ``q_out`` (may be ``q``; default: a new tensor), which is
    returned."""
    if stream is not None:
        with _on(stream, k):
            return cache_append(k, v, k_cache, v_cache, slots, q=q, q_out=q_out, plan=plan,
                                positions=positions, k_scale=k_scale, v_scale=v_scale)
    r = _native.append(k, v, k_cache, v_cache, slots, q, q_out, None if plan is None else plan._at,
                       positions, k_scale, v_scale)
    if type(r) is int:
        _check(r, "attn_cache_append")
    return r


# ----------------------------------------------------------------- decode ----

def decode_workspace_bytes(H: int, H_kv: int, D: int) -> int:
    """Size of the scratch of :func:`attn_decode`."""
    return int(_lib.attn_decode_workspace_bytes(H, H_kv, D))


def attn_decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                block_table: torch.Tensor, seq_lens: torch.Tensor, *,
                scale: Optional[float] = None, window: Optional[int] = None, alibi: bool = False,
                alibi_slopes: Optional[torch.Tensor] = None, softcap: Optional[float] = None,
                rel_bias: Optional[torch.Tensor] = None, k_scale: Optional[torch.Tensor] = None,
                v_scale: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                lse: Optional[torch.Tensor] = None, return_lse: bool = True,
                workspace: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None):
    """Attention of the newest token of every request over the paged cache:
    ``q`` [B, H, D] (bf16, contiguous rows on 4-byte boundaries), caches as
    for :func:`cache_append` (pages of a multiple of 16 tokens are fastest),
    ``block_table`` int32 [B, max_pages], ``seq_lens`` int32 [B] (the newest
    token among them; 0 gives O = 0, LSE = -inf).
    Returns ``(O, LSE)`` (or ``O``), bf16 [B, H, D] and float32 [B, H],
    written into ``out`` / ``lse`` when given, else parts of one allocation
    (keeping or saving one keeps both).  Short rows are fastest where the table
    shows that they are: pass the columns of the step's longest request,
    ``block_table[:, :columns]`` (a view will do).  Score mods and ``window`` as
    for :func:`attn_fwd`; without ``softcap`` a ``rel_bias`` of
    -inf hides its keys.  ``workspace``: uint8 scratch of
    :func:`decode_workspace_bytes` bytes for callers that place it
    themselves; it belongs to the call until the call has finished."""
    if stream is not None:
        with _on(stream, q):
            return attn_decode(q, k_cache, v_cache, block_table, seq_lens, scale=scale,
                               window=window, alibi=alibi, alibi_slopes=alibi_slopes,
                               softcap=softcap, rel_bias=rel_bias, k_scale=k_scale,
                               v_scale=v_scale, out=out, lse=lse, return_lse=return_lse,
                               workspace=workspace)
    r = _native.decode(q, k_cache, v_cache, block_table, seq_lens, scale, window, alibi,
                       alibi_slopes, softcap, rel_bias, k_scale, v_scale, out, lse, return_lse,
                       workspace)
    if type(r) is int:
        _check(r, "attn_decode")
    return r
