"""Token operators over paged pools: rotary positions, appending tokens,
attention of one new token, the decode step. Python wraps the C entry points
of include/kv.h under their names, as the rest of the package does, and offers
two objects that check tensors before the call:

    rope = Rope(head_dim, base=10000.0, scaling="yarn", factor=4.0, original_context=32768)
    seqs = PagedTokens(pool, tables, lens)            # borrowed tensors, one batch of sequences
    seqs.append(k, v, cu_new=cu, rope=rope)           # prompts: keys rotated on the way
    ...
    lens += 1                                         # on the device; pages entered in `tables`
    out = seqs.decode_append(k, v, q, rope=rope)      # one new token of each sequence

The same steps apart are rope.rotate(q, positions), seqs.append(k, v, rope=rope)
and seqs.decode(q). PagedTokens.of_plan makes the pages that a frame plan shows
readable by decode().
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os

from . import capi
from .capi import KV_ROPE_HALF, KV_ROPE_INTERLEAVED, KV_ROPE_LINEAR, KV_ROPE_NONE, KV_ROPE_NTK, KV_ROPE_YARN

LAYOUTS = {"half": KV_ROPE_HALF, "interleaved": KV_ROPE_INTERLEAVED}
SCALINGS = {"none": KV_ROPE_NONE, "linear": KV_ROPE_LINEAR, "ntk": KV_ROPE_NTK, "yarn": KV_ROPE_YARN}


# ---------------------------------------------------------------- C names
def kv_rope_init(rot_dim, layout=KV_ROPE_HALF, scaling=KV_ROPE_NONE, base=10000.0, factor=1.0, original_context=0.0,
                 low_turns=1.0, high_turns=32.0, amplitude=0.0) -> int:
    h = ctypes.c_void_p()
    capi.check(capi.lib().kv_rope_init(ctypes.byref(h), rot_dim, layout, scaling, base, factor, original_context,
                                       low_turns, high_turns, amplitude), "kv_rope_init")
    return h.value


def kv_rope_init_frequencies(rot_dim, layout, theta, amplitude=1.0) -> int:
    h = ctypes.c_void_p()
    buf = (ctypes.c_double * len(theta))(*theta)
    if 2 * len(theta) != rot_dim:
        raise ValueError(f"theta: {len(theta)} frequencies, expected {rot_dim // 2}")
    capi.check(capi.lib().kv_rope_init_frequencies(ctypes.byref(h), rot_dim, layout, buf, amplitude),
               "kv_rope_init_frequencies")
    return h.value


def kv_rope_free(rope) -> None:
    capi.lib().kv_rope_free(rope)


def kv_rope_get(rope) -> dict:
    rot, layout, amp = ctypes.c_int(), ctypes.c_int(), ctypes.c_double()
    theta = (ctypes.c_double * 128)()
    capi.check(capi.lib().kv_rope_get(rope, ctypes.byref(rot), ctypes.byref(layout), ctypes.byref(amp), theta, 128),
               "kv_rope_get")
    return {"rot_dim": rot.value, "layout": layout.value, "amplitude": amp.value,
            "theta": list(theta[: rot.value // 2])}


def _by_address(rows):
    return ctypes.byref(rows) if isinstance(rows, capi.kv_rows) else rows


def kv_rotate(rope, x, out, positions, n_tokens, n_heads, head_dim, dtype, inverse=False, stream=None) -> None:
    """x and out: capi.kv_rows; positions: a device address."""
    capi.check(capi.lib().kv_rotate(rope, _by_address(x), _by_address(out), positions, n_tokens, n_heads, head_dim, dtype,
                                    int(bool(inverse)), stream), "kv_rotate")


def kv_append_tokens(tokens, k, v, n_tokens, cu_new=None, rope=None, positions=None, stream=None) -> None:
    """tokens: capi.kv_tokens; k and v: capi.kv_rows; cu_new and positions: device addresses."""
    capi.check(capi.lib().kv_append_tokens(tokens, _by_address(k), _by_address(v), n_tokens, cu_new, rope, positions,
                                           stream), "kv_append_tokens")


def kv_decode_workspace_bytes(tokens, q_heads) -> int:
    return capi.lib().kv_decode_workspace_bytes(tokens, q_heads)


def kv_decode_workspace_init(tokens, q_heads, workspace, workspace_bytes, stream=None) -> None:
    capi.check(capi.lib().kv_decode_workspace_init(tokens, q_heads, workspace, workspace_bytes, stream),
               "kv_decode_workspace_init")


def kv_decode(tokens, q, q_heads, scale, window, out, workspace, workspace_bytes, stream=None) -> None:
    capi.check(capi.lib().kv_decode(tokens, _by_address(q), q_heads, scale, window, out, workspace, workspace_bytes, stream),
               "kv_decode")


def kv_decode_append(tokens, k, v, q, q_heads, rope, positions, scale, window, out, workspace, workspace_bytes,
                     stream=None) -> None:
    capi.check(capi.lib().kv_decode_append(tokens, _by_address(k), _by_address(v), _by_address(q), q_heads, rope,
                                           positions, scale, window, out, workspace, workspace_bytes, stream),
               "kv_decode_append")


def kv_tokens_check(tokens, stream=None) -> None:
    capi.check(capi.lib().kv_tokens_check(tokens, stream), "kv_tokens_check")


# ---------------------------------------------------------------- objects
# The objects' calls go through a native binding (binding/tokens.cpp), which
# checks the tensors. It and torch are loaded with the first object: importing
# this package does neither.
torch = None
_native = None


def _bind():
    global torch, _native
    if _native is not None:
        return
    import torch as t
    path = os.path.join(os.path.dirname(capi.LIB_PATH), "_tokens.so")
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m paged_kv_cache_frame_b200.build`")
    capi.lib()
    name = __package__ + "._tokens"
    spec = importlib.util.spec_from_file_location(name, path, loader=importlib.machinery.ExtensionFileLoader(name, path))
    native = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(native)
    native.init(capi.check)
    torch, _native = t, native


def _on(device, stream):
    """Context of a call on a given stream (torch's, or a raw handle): made
    torch's current one, with its device."""
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    if stream.device != device:
        raise ValueError(f"stream on {stream.device}, expected {device}")
    return torch.cuda.stream(stream)


class Rope:
    """Rotary positions for the first rot_dim values of a head.

    layout: "half" (pairs (i, i + rot_dim / 2)) or "interleaved" (neighbours).
    scaling: "none", "linear", "ntk" or "yarn" (with original_context,
    low_turns, high_turns; the ramp is linear in a pair's turns over
    original_context, so a checkpoint whose ramp is linear in the pair's index
    needs inv_freq). inv_freq: rot_dim / 2 frequencies in radians a position
    in place of base and scaling. amplitude: factor on the rotated
    values (default: the scaling's own)."""

    def __init__(self, rot_dim, layout="half", base=10000.0, scaling="none", factor=1.0, original_context=0,
                 low_turns=1.0, high_turns=32.0, amplitude=None, inv_freq=None):
        if layout not in LAYOUTS:
            raise ValueError(f"layout: {layout!r}, expected one of {sorted(LAYOUTS)}")
        if scaling not in SCALINGS:
            raise ValueError(f"scaling: {scaling!r}, expected one of {sorted(SCALINGS)}")
        if amplitude is not None and not amplitude > 0:
            raise ValueError("amplitude: must be positive")
        _bind()
        if inv_freq is not None:
            if scaling != "none":
                raise ValueError("inv_freq: given frequencies are not scaled again")
            self.handle = kv_rope_init_frequencies(rot_dim, LAYOUTS[layout], [float(f) for f in inv_freq],
                                                   1.0 if amplitude is None else amplitude)
        else:
            self.handle = kv_rope_init(rot_dim, LAYOUTS[layout], SCALINGS[scaling], base, factor, original_context,
                                       low_turns, high_turns, amplitude or 0.0)
        self._native = _native.rope(self.handle)   # owns the handle, with the autograd nodes made of it
        got = kv_rope_get(self.handle)
        self.rot_dim, self.layout, self.amplitude, self.inv_freq = rot_dim, layout, got["amplitude"], got["theta"]

    def rotate(self, x, positions, out=None, inverse=False, stream=None):
        """x [tokens, heads, head_dim] (bfloat16, float16 or float32; the
        last dimension dense) rotated at positions [tokens] (int32), into
        `out` if given (x itself, or apart from it). Differentiable in x, the
        gradient too, in reverse mode (tangents are refused). A captured backward pass belongs in one capture with its
        forward, through torch.autograd.grad: a captured .backward() meets the
        streams of any eager graph of the same leaves that is still alive."""
        if stream is None:
            return _native.rotate(self._native, x, positions, out, inverse)
        if x.requires_grad and torch.is_grad_enabled():
            raise ValueError("rotate: stream is not for a call that records a gradient (use torch.cuda.stream)")
        with _on(x.device, stream):
            return _native.rotate(self._native, x, positions, out, inverse)


class PagedTokens:
    """A batch of sequences in a paged pool (borrowed tensors).

    pool: [max_pages, 2, page_size, heads, head_dim], bfloat16 or float16,
    head_dim 64 or 128. tables: [n_seqs, width] int32 page ids. lens:
    [n_seqs] int32, tokens of each sequence, the new ones included; 0 marks an
    unused row. Both may be changed in place between calls, and replayed
    captures read them anew. The object holds the device's error word: keep it
    as long as a captured call may be replayed, and order its use on another
    stream behind its construction, as for any tensor."""

    def __init__(self, pool, tables, lens, _read_only=False):
        _bind()
        self._native = _native.tokens(pool, tables, lens, _read_only)
        self._pool, self._tables, self._lens = pool, tables, lens
        self._c = capi.kv_tokens.from_address(_native.address(self._native))   # for the C names
        self.n_seqs = tables.shape[0]
        self.max_pages, _, self.page_size, self.H, self.D = pool.shape

    # The library holds their addresses: other tensors need another object.
    pool = property(lambda self: self._pool)
    tables = property(lambda self: self._tables)
    lens = property(lambda self: self._lens)

    @classmethod
    def of_plan(cls, plan, block, streams=None):
        """The tokens that a frame plan shows, as sequences: what kv_run
        attends to, for decode(). Read only: append() and decode_append() are
        refused, as the pages and their free slots are the caches'. streams: indices into the plan's caches
        (default all), whose pools must be one (a group's, or one cache's).
        Tables and lengths are copies: they hold until a cache's page state
        changes. Refused where a cache changed after the plan, where the open
        step's block is not written yet, and where pages hold tokens that the
        plan hides."""
        _bind()
        streams = list(range(len(plan.caches))) if streams is None else list(streams)
        if not streams:
            raise ValueError("streams: none given")
        from . import _torch_dtype, kv_get_kv_tiles, kv_plan_check
        pool = plan.caches[streams[0]].pools[block]
        if pool is None or isinstance(pool, int):
            raise ValueError("of_plan: the block's pool must be bound as a tensor")
        tables, lens = [], []
        for i in streams:
            c = plan.caches[i]
            if c.pools[block] is not pool:
                raise ValueError("streams: their caches do not share one pool")
            kv_plan_check(plan.handle, i, block)
            pages, last = plan.page_table(i)
            n = (len(pages) - 1) * c.page_size + last
            if sum(-(-(hi - lo) // step) for _, lo, hi, _, step in kv_get_kv_tiles(plan.handle, i, True)) != n:
                raise ValueError(f"streams: stream {i}'s pages hold tokens that the plan hides")
            tables.append(pages)
            lens.append(n)
        width = max(len(t) for t in tables)
        c = plan.caches[streams[0]]
        shape = (c.max_pages, 2, c.page_size, c.H, c.D)
        # the cache's bytes in the cache's type: bind_pool takes any tensor that is large enough
        return cls(pool.view(-1).view(torch.uint8)[:c.pool_bytes()].view(_torch_dtype(c.fp16)).view(shape),
                   torch.tensor([t + [0] * (width - len(t)) for t in tables], dtype=torch.int32, device=pool.device),
                   torch.tensor(lens, dtype=torch.int32, device=pool.device), _read_only=True)

    def append(self, k, v, cu_new=None, rope=None, positions=None, stream=None):
        """Write new tokens' k and v [tokens, heads, head_dim], the keys
        rotated by `rope` at `positions` [tokens] (default: their index in the
        sequence). cu_new [n_seqs + 1]: tokens cu_new[s] .. cu_new[s + 1] - 1
        are the last of sequence s (None: one each)."""
        rope = None if rope is None else rope._native
        if stream is None:
            return _native.append(self._native, k, v, cu_new, rope, positions)
        with _on(self._pool.device, stream):
            return _native.append(self._native, k, v, cu_new, rope, positions)

    def workspace_bytes(self, q_heads) -> int:
        """Bytes of a workspace for decode and decode_append."""
        return _native.workspace_bytes(self._native, q_heads)

    def workspace(self, q_heads, stream=None):
        """A prepared workspace for decode and decode_append with that many
        query heads. Calls that may overlap on the GPU need one each; those
        without a given one share one per stream."""
        if stream is None:
            return _native.workspace(self._native, q_heads)
        with _on(self._pool.device, stream):
            return _native.workspace(self._native, q_heads)

    def decode(self, q, out=None, scale=None, window=0, workspace=None, stream=None):
        """Attention of one new token per sequence: q [n_seqs, q heads,
        head_dim] against the sequence's last `window` tokens (0: all). scale:
        default 1/sqrt(head_dim). out: q itself, or apart from q and the pool.
        workspace: of workspace() (default: one per stream, in a capture one
        per call, prepared by the graph)."""
        if stream is None:
            return _native.decode(self._native, None, None, q, None, None, out, scale, window, workspace)
        with _on(self._pool.device, stream):
            return _native.decode(self._native, None, None, q, None, None, out, scale, window, workspace)

    def decode_append(self, k, v, q, rope=None, positions=None, out=None, scale=None, window=0, workspace=None,
                      stream=None):
        """A decode step: append(k, v, rope=rope), rotate q at the same
        positions [n_seqs] (default lens - 1) and decode(q), in one launch."""
        rope = None if rope is None else rope._native
        if stream is None:
            return _native.decode(self._native, k, v, q, rope, positions, out, scale, window, workspace)
        with _on(self._pool.device, stream):
            return _native.decode(self._native, k, v, q, rope, positions, out, scale, window, workspace)

    def check_device(self, stream=None):
        """Synchronise and raise KVError if a kernel met a page id or length
        out of range since the last check."""
        if stream is None:
            return _native.check(self._native)
        with _on(self._pool.device, stream):
            return _native.check(self._native)
