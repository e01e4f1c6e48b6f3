"""Token operators over paged pools: rotary positions, appending tokens,
attention of one new token, the decode step. Python wraps the C entry points
of include/kv.h under their names, as the rest of the package does, and two
objects check tensors before the call:

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
import functools
import struct

from . import capi
from .capi import (KV_BF16, KV_FP16, KV_FP32, KV_ROPE_HALF, KV_ROPE_INTERLEAVED, KV_ROPE_LINEAR, KV_ROPE_NONE,
                   KV_ROPE_NTK, KV_ROPE_YARN)

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


# ---------------------------------------------------------------- tensors
torch = None    # bound by the first object: importing this package does not import torch
_codes = {}


def _bind_torch():
    global torch
    if torch is None:
        import torch as t
        _codes.update({t.bfloat16: KV_BF16, t.float16: KV_FP16, t.float32: KV_FP32})
        torch = t


def _check(x, name, shape, dtype, device, contiguous=True):
    """Shape, dtype, layout and device of a tensor, before its address goes to
    the library. Not contiguous: the last dimension only has to be dense."""
    if (x.dtype is dtype and x.shape == shape and x.device == device
            and (x.is_contiguous() or (not contiguous and x.stride(-1) == 1))):
        return
    if tuple(x.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(x.shape)}, expected {tuple(shape)}")
    if x.dtype != dtype:
        raise ValueError(f"{name}: dtype {x.dtype}, expected {dtype}")
    if x.device != device:
        raise ValueError(f"{name}: on {x.device}, expected {device}")
    if contiguous:
        raise ValueError(f"{name}: must be contiguous")
    if x.shape[-1] > 1 and x.numel():
        raise ValueError(f"{name}: the last dimension must be contiguous")


def _no_gradient(*named):
    for name, x in named:
        if x.requires_grad:
            raise ValueError(f"{name}: requires a gradient, which this operator does not have "
                             "(detach it or call under torch.no_grad)")


_pack_rows = struct.Struct("@Pqq").pack    # a kv_rows


def _rows(x):
    """The kv_rows of a [n, heads, head_dim] tensor, packed; the stride of a
    dimension of one element says nothing and is 0."""
    n, h, _ = x.shape
    t, s, _ = x.stride()
    return _pack_rows(x.data_ptr(), t if n > 1 else 0, s if h > 1 else 0)


class _On:
    """The device and stream of a call: its tensors' device made current for
    the call, its outputs and workspace allocated for the stream that uses
    them (torch's current one on that device unless given)."""

    __slots__ = ("stream", "guard")

    def __init__(self, device, stream):
        if device.type != "cuda":
            raise ValueError(f"tensors must be on a CUDA device, not on {device}")
        if stream is None:
            self.guard = torch.cuda.device(device)
            self.stream = torch.cuda.current_stream(device).cuda_stream
            return
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=device)
        if stream.device != device:
            raise ValueError(f"stream on {stream.device}, expected {device}")
        self.guard = torch.cuda.stream(stream)   # makes the device current as well
        self.stream = stream.cuda_stream

    def __enter__(self):
        self.guard.__enter__()
        return self.stream

    def __exit__(self, *exc):
        self.guard.__exit__(*exc)
        return False


def _here(device, stream):
    """The current stream's handle where a call needs no switch of device or
    stream, else None (_On makes it)."""
    if stream is None and device.type == "cuda":
        i = device.index
        if torch._C._cuda_getDevice() == i:
            return torch._C._cuda_getCurrentRawStream(i)
    return None


def _like(x):
    """An uninitialised contiguous tensor of x's shape."""
    return torch.empty_like(x) if x.is_contiguous() else torch.empty_like(x, memory_format=torch.contiguous_format)


@functools.lru_cache(maxsize=None)
def _rotation_with_gradient():
    class Rotation(torch.autograd.Function):
        """y = rotation of x; dx = the inverse rotation of dy, itself
        differentiable."""

        @staticmethod
        def forward(ctx, x, positions, rope, inverse):
            ctx.save_for_backward(positions)
            ctx.rope = rope
            ctx.inverse = inverse
            return rope._rotate(x, positions, None, inverse, None)

        @staticmethod
        def backward(ctx, dy):
            positions, = ctx.saved_tensors
            if dy.stride(-1) != 1:
                dy = dy.contiguous()
            if not torch.is_grad_enabled():
                return ctx.rope._rotate(dy, positions, None, not ctx.inverse, None), None, None, None
            return Rotation.apply(dy, positions, ctx.rope, not ctx.inverse), None, None, None

    return Rotation


class Rope:
    """Rotary positions for the first rot_dim values of a head.

    layout: "half" (pairs (i, i + rot_dim / 2)) or "interleaved" (neighbours).
    scaling: "none", "linear", "ntk" or "yarn" (with original_context,
    low_turns, high_turns). inv_freq: rot_dim / 2 frequencies in radians a
    position in place of base and scaling. amplitude: factor on the rotated
    values (default: the scaling's own)."""

    def __init__(self, rot_dim, layout="half", base=10000.0, scaling="none", factor=1.0, original_context=0,
                 low_turns=1.0, high_turns=32.0, amplitude=None, inv_freq=None):
        self.handle = None
        _bind_torch()
        if layout not in LAYOUTS:
            raise ValueError(f"layout: {layout!r}, expected one of {sorted(LAYOUTS)}")
        if scaling not in SCALINGS:
            raise ValueError(f"scaling: {scaling!r}, expected one of {sorted(SCALINGS)}")
        if amplitude is not None and not amplitude > 0:
            raise ValueError("amplitude: must be positive")
        if inv_freq is not None:
            if scaling != "none":
                raise ValueError("inv_freq: given frequencies are not scaled again")
            self.handle = kv_rope_init_frequencies(rot_dim, LAYOUTS[layout], [float(f) for f in inv_freq],
                                                   1.0 if amplitude is None else amplitude)
        else:
            self.handle = kv_rope_init(rot_dim, LAYOUTS[layout], SCALINGS[scaling], base, factor, original_context,
                                       low_turns, high_turns, amplitude or 0.0)
        self._lib = capi.lib()
        got = kv_rope_get(self.handle)
        self.rot_dim, self.layout, self.amplitude, self.inv_freq = rot_dim, layout, got["amplitude"], got["theta"]

    def __del__(self):
        h = getattr(self, "handle", None)
        if h:
            self.handle = None
            try:
                kv_rope_free(h)
            except Exception:   # interpreter shutdown: the library may already be gone
                pass

    def _rotate(self, x, positions, out, inverse, stream):
        code = _codes.get(x.dtype)
        if code is None:
            raise ValueError(f"x: dtype {x.dtype}, expected bfloat16, float16 or float32")
        if x.dim() != 3:
            raise ValueError(f"x: shape {tuple(x.shape)}, expected [tokens, heads, head_dim]")
        shape, device = x.shape, x.device
        _check(x, "x", shape, x.dtype, device, contiguous=False)
        _check(positions, "positions", shape[:1], torch.int32, device)
        if out is not None:
            _check(out, "out", shape, x.dtype, device, contiguous=False)
        s = _here(device, stream)
        if s is not None:
            return self._launch(x, positions, out, inverse, code, s)
        with _On(device, stream) as s:
            return self._launch(x, positions, out, inverse, code, s)

    def _launch(self, x, positions, out, inverse, code, s):
        n, h, d = x.shape
        if out is None:
            out = _like(x)
        rc = self._lib.kv_rotate(self.handle, _rows(x), _rows(out), positions.data_ptr(), n, h, d, code, inverse, s)
        if rc:
            capi.check(rc, "kv_rotate")
        return out

    def rotate(self, x, positions, out=None, inverse=False, stream=None):
        """x [tokens, heads, head_dim] (bfloat16, float16 or float32; the
        last dimension dense) rotated at positions [tokens] (int32), into
        `out` if given (x itself, or apart from it). Differentiable in x, the
        gradient too. A captured backward pass belongs in one capture with its
        forward, through torch.autograd.grad: a captured .backward() meets the
        streams of any eager graph of the same leaves that is still alive."""
        if (x.requires_grad or (out is not None and out.requires_grad)) and torch.is_grad_enabled():
            if out is not None or stream is not None:
                raise ValueError("rotate: out and stream are not for a call that records a gradient "
                                 "(use torch.cuda.stream for the latter)")
            return _rotation_with_gradient().apply(x, positions, self, bool(inverse))
        return self._rotate(x, positions, out, bool(inverse), stream)


class PagedTokens:
    """A batch of sequences in a paged pool (borrowed tensors).

    pool: [max_pages, 2, page_size, heads, head_dim], bfloat16 or float16,
    head_dim 64 or 128. tables: [n_seqs, width] int32 page ids. lens:
    [n_seqs] int32, tokens of each sequence, the new ones included; 0 marks an
    unused row. Both may be changed in place between calls, and replayed
    captures read them anew. The object holds the device's error word: keep it
    as long as a captured call may be replayed, and order its use on another
    stream behind its construction, as for any tensor."""

    def __init__(self, pool, tables, lens):
        _bind_torch()
        if pool.dim() != 5 or pool.shape[1] != 2:
            raise ValueError(f"pool: shape {tuple(pool.shape)}, expected [max_pages, 2, page_size, heads, head_dim]")
        if pool.dtype not in (torch.bfloat16, torch.float16):
            raise ValueError(f"pool: dtype {pool.dtype}, expected bfloat16 or float16")
        if pool.device.type != "cuda":
            raise ValueError(f"pool: must be a CUDA tensor, not on {pool.device}")
        _check(pool, "pool", pool.shape, pool.dtype, pool.device)
        if tables.dim() != 2:
            raise ValueError(f"tables: shape {tuple(tables.shape)}, expected [n_seqs, width]")
        self.n_seqs, width = tables.shape
        _check(tables, "tables", (self.n_seqs, width), torch.int32, pool.device, contiguous=False)
        _check(lens, "lens", (self.n_seqs,), torch.int32, pool.device)
        self._pool, self._tables, self._lens = pool, tables, lens
        self.max_pages, _, self.page_size, self.H, self.D = pool.shape
        self._dtype, self._device = pool.dtype, pool.device
        self.error = torch.zeros(1, dtype=torch.int32, device=pool.device)
        self._c = capi.kv_tokens(
            pool.data_ptr(), tables.data_ptr(), lens.data_ptr(), self.error.data_ptr(),
            tables.stride(0) if self.n_seqs > 1 else width, self.max_pages, self.page_size, self.H, self.D,
            _codes[pool.dtype], width, self.n_seqs)
        self._lib = capi.lib()
        self._bytes = {}        # query heads -> workspace bytes
        self._workspaces = {}   # (stream, query heads) -> the workspace of eager calls there

    # The library holds their addresses: other tensors need another object.
    pool = property(lambda self: self._pool)
    tables = property(lambda self: self._tables)
    lens = property(lambda self: self._lens)

    @classmethod
    def of_plan(cls, plan, block, streams=None):
        """The tokens that a frame plan shows, as sequences: what kv_run
        attends to, for decode(). streams: indices into the plan's caches
        (default all), whose pools must be one (a group's, or one cache's).
        Tables and lengths are copies: they hold until a cache's page state
        changes. Refused where pages hold tokens that the plan hides."""
        _bind_torch()
        streams = list(range(len(plan.caches))) if streams is None else list(streams)
        if not streams:
            raise ValueError("streams: none given")
        pool = plan.caches[streams[0]].pools[block]
        if pool is None or isinstance(pool, int):
            raise ValueError("of_plan: the block's pool must be bound as a tensor")
        tables, lens = [], []
        for i in streams:
            c = plan.caches[i]
            if c.pools[block] is not pool:
                raise ValueError("streams: their caches do not share one pool")
            pages, last = plan.page_table(i)
            n = (len(pages) - 1) * c.page_size + last
            from . import kv_get_kv_tiles
            if sum(-(-(hi - lo) // step) for _, lo, hi, _, step in kv_get_kv_tiles(plan.handle, i, True)) != n:
                raise ValueError(f"streams: stream {i}'s pages hold tokens that the plan hides")
            tables.append(pages)
            lens.append(n)
        width = max(len(t) for t in tables)
        c = plan.caches[streams[0]]
        shape = (c.max_pages, 2, c.page_size, c.H, c.D)
        return cls(pool.view(-1)[:c.max_pages * 2 * c.page_size * c.H * c.D].view(shape),
                   torch.tensor([t + [0] * (width - len(t)) for t in tables], dtype=torch.int32, device=pool.device),
                   torch.tensor(lens, dtype=torch.int32, device=pool.device))

    def _index(self, x, name, n):
        if x is None:
            return None
        _check(x, name, (n,), torch.int32, self._device)
        return x.data_ptr()

    def append(self, k, v, cu_new=None, rope=None, positions=None, stream=None):
        """Write new tokens' k and v [tokens, heads, head_dim], the keys
        rotated by `rope` at `positions` [tokens] (default: their index in the
        sequence). cu_new [n_seqs + 1]: tokens cu_new[s] .. cu_new[s + 1] - 1
        are the last of sequence s (None: one each)."""
        n = self.n_seqs if cu_new is None or k.dim() != 3 else k.shape[0]
        shape = (n, self.H, self.D)
        _check(k, "k", shape, self._dtype, self._device, contiguous=False)
        _check(v, "v", shape, self._dtype, self._device, contiguous=False)
        if (k.requires_grad or v.requires_grad) and torch.is_grad_enabled():
            _no_gradient(("k", k), ("v", v))
        cu = self._index(cu_new, "cu_new", self.n_seqs + 1)
        pos = self._index(positions, "positions", n)
        s = _here(self._device, stream)
        if s is not None:
            return self._append(k, v, n, cu, rope, pos, s)
        with _On(self._device, stream) as s:
            return self._append(k, v, n, cu, rope, pos, s)

    def _append(self, k, v, n, cu, rope, pos, s):
        rc = self._lib.kv_append_tokens(self._c, _rows(k), _rows(v), n, cu, rope.handle if rope is not None else None,
                                         pos, s)
        if rc:
            capi.check(rc, "kv_append_tokens")

    def workspace_bytes(self, q_heads) -> int:
        """Bytes of a workspace for decode and decode_append."""
        if q_heads not in self._bytes:
            with torch.cuda.device(self._device):
                self._bytes[q_heads] = kv_decode_workspace_bytes(self._c, q_heads)
        return self._bytes[q_heads]

    def workspace(self, q_heads, stream=None):
        """A prepared workspace for decode and decode_append with that many
        query heads. Calls that may overlap on the GPU need one each; those
        without a given one share one per stream."""
        with _On(self._device, stream) as s:
            return self._new_workspace(q_heads, s)

    def _new_workspace(self, q_heads, s):
        ws = torch.empty(self.workspace_bytes(q_heads), dtype=torch.uint8, device=self._device)
        kv_decode_workspace_init(self._c, q_heads, ws.data_ptr(), ws.numel(), s)
        return ws

    def _check_call(self, q, out, scale, workspace):
        if q.dim() != 3:
            raise ValueError(f"q: shape {tuple(q.shape)}, expected [n_seqs, q heads, head_dim]")
        heads = q.shape[1]
        shape = (self.n_seqs, heads, self.D)
        _check(q, "q", shape, self._dtype, self._device, contiguous=False)
        if heads < 1 or heads % self.H:
            raise ValueError(f"q: {heads} heads, expected a multiple of the pool's {self.H}")
        if out is not None:
            _check(out, "out", shape, self._dtype, self._device)
        if scale is not None and not scale:
            raise ValueError("scale: 0 would weigh all tokens alike")
        if workspace is not None and (workspace.device != self._device or not workspace.is_contiguous()):
            raise ValueError("workspace: must be contiguous, on the pool's device")

    def _buffers(self, q, out, workspace, s):
        if out is None:
            out = _like(q)
        if workspace is None:
            heads = q.shape[1]
            if torch._C._cuda_isCurrentStreamCapturing():
                workspace = self._new_workspace(heads, s)   # the graph's own, prepared by each replay
            else:
                workspace = self._workspaces.get((s, heads))
                if workspace is None:
                    workspace = self._workspaces[s, heads] = self._new_workspace(heads, s)
        return out, workspace

    def decode(self, q, out=None, scale=None, window=0, workspace=None, stream=None):
        """Attention of one new token per sequence: q [n_seqs, q heads,
        head_dim] against the sequence's last `window` tokens (0: all). scale:
        default 1/sqrt(head_dim). workspace: of workspace() (default: one per
        stream, in a capture one per call, prepared by the graph)."""
        self._check_call(q, out, scale, workspace)
        if q.requires_grad and torch.is_grad_enabled():
            _no_gradient(("q", q))
        s = _here(self._device, stream)
        if s is not None:
            return self._decode(q, out, scale, window, workspace, s)
        with _On(self._device, stream) as s:
            return self._decode(q, out, scale, window, workspace, s)

    def _decode(self, q, out, scale, window, workspace, s):
        out, ws = self._buffers(q, out, workspace, s)
        rc = self._lib.kv_decode(self._c, _rows(q), q.shape[1], scale or 0.0, window, out.data_ptr(), ws.data_ptr(),
                                  ws.nbytes, s)
        if rc:
            capi.check(rc, "kv_decode")
        return out

    def decode_append(self, k, v, q, rope=None, positions=None, out=None, scale=None, window=0, workspace=None,
                      stream=None):
        """A decode step: append(k, v, rope=rope), rotate q at the same
        positions [n_seqs] (default lens - 1) and decode(q), in one launch."""
        shape = (self.n_seqs, self.H, self.D)
        _check(k, "k", shape, self._dtype, self._device, contiguous=False)
        _check(v, "v", shape, self._dtype, self._device, contiguous=False)
        self._check_call(q, out, scale, workspace)
        if (q.requires_grad or k.requires_grad or v.requires_grad) and torch.is_grad_enabled():
            _no_gradient(("k", k), ("v", v), ("q", q))
        pos = self._index(positions, "positions", self.n_seqs)
        s = _here(self._device, stream)
        if s is not None:
            return self._decode_append(k, v, q, rope, pos, out, scale, window, workspace, s)
        with _On(self._device, stream) as s:
            return self._decode_append(k, v, q, rope, pos, out, scale, window, workspace, s)

    def _decode_append(self, k, v, q, rope, pos, out, scale, window, workspace, s):
        out, ws = self._buffers(q, out, workspace, s)
        rc = self._lib.kv_decode_append(self._c, _rows(k), _rows(v), _rows(q), q.shape[1],
                                         rope.handle if rope is not None else None, pos, scale or 0.0, window,
                                         out.data_ptr(), ws.data_ptr(), ws.nbytes, s)
        if rc:
            capi.check(rc, "kv_decode_append")
        return out

    def check_device(self, stream=None):
        """Synchronise and raise KVError if a kernel met a page id or length
        out of range since the last check."""
        with _On(self._device, stream) as s:
            kv_tokens_check(self._c, s)
