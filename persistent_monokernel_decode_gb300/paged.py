"""A paged K/V cache for a batch of sequences: the ``kie_paged_*`` operators of include/kie.h on CUDA tensors.

``paged_extend``, ``paged_append``, ``paged_attention`` and ``paged_release`` marshal arguments like the rest of the
binding: they check types, shapes and devices, allocate their outputs with PyTorch and launch on the current stream
of the tensors' device, without synchronising. ``PagedCache`` holds the pages and tables that such a program keeps.
"""
from __future__ import annotations

import struct
from typing import NamedTuple

from . import KIE_OK, KieError, _torch, lib

KIE_F16, KIE_BF16, KIE_F32, KIE_E4M3 = 0, 1, 2, 3

# The argument structs of include/kie.h, packed in one go (a call packs some forty fields).
_PAGES = "4P12q5i4x"
_EXTEND = struct.Struct("@5Pq7P5i4x")
_RELEASE = struct.Struct("@4Pq3P4i")
_APPEND = struct.Struct("@" + _PAGES + "4P8q3P5i4x")
_ATTENTION = struct.Struct("@" + _PAGES + "3P4q2PqPNf5i")


class PagedStep(NamedTuple):
    """What paged_extend computed (CUDA tensors): lens, n_free, admitted, row_start per request; slots, positions,
    seqs per packed row."""
    lens: object
    n_free: object
    admitted: object
    row_start: object
    slots: object
    positions: object
    seqs: object


class _Ready:
    """What the calls need of torch and the library, looked up once."""

    def __init__(self):
        torch = self.torch = _torch()
        L = lib()
        self.extend, self.release = L.kie_paged_extend, L.kie_paged_release
        self.append, self.attention = L.kie_paged_append, L.kie_paged_attention
        self.kinds = {torch.float16: KIE_F16, torch.bfloat16: KIE_BF16, torch.float32: KIE_F32,
                      torch.float8_e4m3fn: KIE_E4M3}
        # the handle alone: making a torch.cuda.Stream of it takes 3 us a call
        self.current_device, self.raw_stream = torch.cuda.current_device, torch._C._cuda_getCurrentRawStream
        self.workspace = {}  # bytes by (device, heads, kv heads, head_dim)

    def workspace_bytes(self, device, n_heads, n_kv_heads, head_dim):
        key = (device.index, n_heads, n_kv_heads, head_dim)
        if key not in self.workspace:
            with self.torch.cuda.device(device):
                self.workspace[key] = lib().kie_paged_attention_workspace(n_heads, n_kv_heads, head_dim)
        return self.workspace[key]

    def launch(self, fn, packed, device):
        """Call fn on the current stream of `device`, which is made the current device for the call."""
        index = device.index
        if index != self.current_device():
            with self.torch.cuda.device(device):
                rc = fn(packed, self.raw_stream(index))
        else:
            rc = fn(packed, self.raw_stream(index))
        if rc != KIE_OK:
            raise KieError(rc, (lib().kie_paged_last_error() or b"").decode())


_ready = None


def _setup() -> _Ready:
    global _ready
    if _ready is None:
        _ready = _Ready()
    return _ready


def _ints(torch, device, t, name, n=None):
    """Address of a contiguous int32 tensor on `device` (of n values)."""
    if t.dtype != torch.int32 or not t.is_contiguous() or t.device != device or (n is not None and t.numel() != n):
        raise ValueError(f"{name} must be a contiguous int32 tensor{'' if n is None else f' of {n}'} on {device}")
    return t.data_ptr()


def _table(torch, device, t, n_seqs):
    """(address, row stride, max_blocks) of a block table."""
    shape, stride = t.shape, t.stride()
    if t.dtype != torch.int32 or len(shape) != 2 or shape[0] != n_seqs or shape[1] < 1 or stride[1] != 1 or \
            t.device != device:
        raise ValueError(f"block_table must be an int32 [{n_seqs}, max_blocks] tensor on {device} with contiguous rows")
    return t.data_ptr(), stride[0], shape[1]


def _rows(t, name, shape, dtype, device):
    """(address, first two strides) of a tensor of rows."""
    stride = t.stride()
    if t.shape != shape or t.dtype != dtype or t.device != device or stride[2] != 1:
        raise ValueError(f"{name} must be a {dtype} {list(shape)} tensor on {device} with contiguous rows")
    return t.data_ptr(), stride[0], stride[1]


def _pages(r, device, k, v, k_scale, v_scale):
    """The packed fields of a kie_pages from page tensors [n_blocks, n_kv_heads, block_size, head_dim] (any outer
    strides)."""
    shape, ks, vs, kind = k.shape, k.stride(), v.stride(), r.kinds.get(k.dtype, KIE_F32)
    if len(shape) != 4 or v.shape != shape or v.dtype != k.dtype or ks[3] != 1 or vs[3] != 1:
        raise ValueError("the pages are two tensors [n_blocks, n_kv_heads, block_size, head_dim] of one type whose "
                         "last dimension is contiguous")
    if kind == KIE_F32:
        raise ValueError(f"pages are float16, bfloat16 or float8_e4m3fn, not {k.dtype}")
    if k.device != device or v.device != device or device.type != "cuda":
        raise ValueError(f"the pages and the rows must be on one CUDA device, not {k.device}, {v.device} and {device}")
    if kind != KIE_E4M3:
        if k_scale is not None or v_scale is not None:
            raise ValueError("only float8_e4m3fn pages have scales")
        return (k.data_ptr(), v.data_ptr(), 0, 0, ks[0], ks[1], ks[2], vs[0], vs[1], vs[2], 0, 0, 0, 0, 0, 0,
                shape[0], shape[1], shape[2], shape[3], kind)
    for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
        if t is None or t.dtype != r.torch.float32 or t.shape != shape[:3] or t.device != device:
            raise ValueError(f"{name} must be a float32 {list(shape[:3])} tensor on {device}")
    return (k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), *ks[:3], *vs[:3], *k_scale.stride(),
            *v_scale.stride(), *shape, kind)


def paged_extend(new_lens, lens, block_table, free_blocks, n_free, block_size: int, n_rows: int) -> PagedStep:
    """Pages and slots for new_lens[r] more tokens of each request r (kie_paged_extend): new entries go into
    block_table [R, max_blocks] in place, everything else into new tensors. lens, new_lens int32 [R]; free_blocks
    int32 (a stack whose first n_free[0] entries are free pages); n_rows >= sum(new_lens) rows are listed."""
    r = _ready or _setup()
    torch, dev, R = r.torch, lens.device, lens.numel()
    if dev.type != "cuda" or n_rows < 0:
        raise ValueError("lens must be a CUDA tensor and n_rows >= 0")
    table, stride, width = _table(torch, dev, block_table, R)
    inputs = (_ints(torch, dev, lens, "lens"), _ints(torch, dev, new_lens, "new_lens", R),
              _ints(torch, dev, free_blocks, "free_blocks"), _ints(torch, dev, n_free, "n_free", 1))
    ints = torch.empty(2 * R + 2 + 3 * n_rows, dtype=torch.int32, device=dev)
    admitted = torch.empty(R, dtype=torch.bool, device=dev)
    at, rows = ints.data_ptr(), 4 * n_rows
    first = at + 8 * R + 8
    r.launch(r.extend, _EXTEND.pack(*inputs, table, stride, at, at + 4 * R, at + 4 * R + 4, first, first + rows,
                                    first + 2 * rows, admitted.data_ptr(), R, width, block_size, n_rows,
                                    free_blocks.numel()), dev)
    lens_out, n_free_out, row_start, slots, positions, seqs = ints.split((R, 1, R + 1, n_rows, n_rows, n_rows))
    return PagedStep(lens_out, n_free_out, admitted, row_start, slots, positions, seqs)


def paged_release(done, lens, block_table, free_blocks, n_free, block_size: int):
    """Pages of the requests with done[r] (bool [R]) back onto free_blocks, in place (kie_paged_release). Returns
    (lens, n_free): 0 for the finished requests, and the new number of free pages."""
    r = _ready or _setup()
    torch, dev, R = r.torch, lens.device, lens.numel()
    if dev.type != "cuda":
        raise ValueError("lens must be a CUDA tensor")
    if done.dtype != torch.bool or done.numel() != R or not done.is_contiguous() or done.device != dev:
        raise ValueError(f"done must be a contiguous bool tensor of {R} on {dev}")
    table, stride, width = _table(torch, dev, block_table, R)
    inputs = (done.data_ptr(), _ints(torch, dev, lens, "lens"), _ints(torch, dev, n_free, "n_free", 1), table, stride,
              _ints(torch, dev, free_blocks, "free_blocks"))
    out = torch.empty(R + 1, dtype=torch.int32, device=dev)
    at = out.data_ptr()
    r.launch(r.release, _RELEASE.pack(*inputs, at, at + 4 * R, R, width, block_size, free_blocks.numel()), dev)
    return out.split((R, 1))


def paged_append(k, v, k_cache, v_cache, slots, *, positions=None, rope=None, q=None, q_out=None, k_scale=None,
                 v_scale=None, k_pairs: bool = False):
    """K/V rows [T, n_kv_heads, head_dim] into their slots (int32 [T]) of the pages, rotated at `positions` by the
    table `rope` (fp32 [n_pos, head_dim / 2, 2], see rope_table) if it is given, and rounded to the pages' type
    (kie_paged_append). q [T, n_heads, head_dim], if given, is rotated into q_out, which is returned (new if None;
    rows whose slot is out of range are left as they were). Slots must not repeat."""
    r = _ready or _setup()
    torch, dev, dtype, shape = r.torch, k.device, k.dtype, k.shape
    pages = _pages(r, dev, k_cache, v_cache, k_scale, v_scale)
    if len(shape) != 3 or shape[1] != pages[17] or shape[2] != pages[19]:
        raise ValueError(f"k must be [rows, {pages[17]}, {pages[19]}] like the pages")
    T, _, dh = shape
    k_at, k0, k1 = _rows(k, "k", shape, dtype, dev)
    v_at, v0, v1 = _rows(v, "v", shape, dtype, dev)
    slots_at = _ints(torch, dev, slots, "slots", T)
    q_at = out_at = q0 = q1 = o0 = o1 = n_heads = rope_at = positions_at = n_pos = 0
    if q is not None:
        if q.dim() != 3 or q.shape[0] != T or q.shape[2] != dh:
            raise ValueError(f"q must be [{T}, n_heads, {dh}]")
        n_heads = q.shape[1]
        q_at, q0, q1 = _rows(q, "q", q.shape, dtype, dev)
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=dtype, device=dev)
        out_at, o0, o1 = _rows(q_out, "q_out", q.shape, dtype, dev)
    if rope is not None:
        if positions is None:
            raise ValueError("a rope table needs positions")
        positions_at = _ints(torch, dev, positions, "positions", T)
        if rope.dtype != torch.float32 or rope.shape[1:] != (dh // 2, 2) or not rope.is_contiguous() or \
                rope.device != dev:
            raise ValueError(f"rope must be a contiguous float32 [n_pos, {dh // 2}, 2] tensor on {dev}")
        rope_at, n_pos = rope.data_ptr(), rope.shape[0]
    r.launch(r.append, _APPEND.pack(*pages, k_at, v_at, q_at, out_at, k0, k1, v0, v1, q0, q1, o0, o1, slots_at,
                                    positions_at, rope_at, T, n_heads, n_pos, r.kinds.get(dtype, -1), bool(k_pairs)),
             dev)
    return q_out


def paged_attention(q, k_cache, v_cache, block_table, lens, *, scale=None, window: int = 0, k_scale=None, v_scale=None,
                    out=None, return_lse: bool = False):
    """Attention of one new token per sequence over the pages (kie_paged_attention): q [B, n_heads, head_dim], lens
    int32 [B] positions cached (the new token's among them), block_table int32 [B, max_blocks]. scale: 1 /
    sqrt(head_dim) by default; window: only the last `window` positions (0: all). Returns out, or (out, lse) with
    lse fp32 [B, n_heads]. The workspace is allocated by the call, so calls on several streams and captured graphs
    share none."""
    r = _ready or _setup()
    torch, dev, dtype, shape = r.torch, q.device, q.dtype, q.shape
    pages = _pages(r, dev, k_cache, v_cache, k_scale, v_scale)
    if len(shape) != 3 or shape[2] != pages[19]:
        raise ValueError(f"q must be [sequences, n_heads, {pages[19]}] like the pages")
    B, H, dh = shape
    q_at, q0, q1 = _rows(q, "q", shape, dtype, dev)
    table, stride, width = _table(torch, dev, block_table, B)
    lens_at = _ints(torch, dev, lens, "lens", B)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=dev)
    out_at, o0, o1 = _rows(out, "out", shape, dtype, dev)
    lse = torch.empty((B, H), dtype=torch.float32, device=dev) if return_lse else None
    size = r.workspace_bytes(dev, H, pages[17], dh)
    workspace = torch.empty(size, dtype=torch.uint8, device=dev)
    r.launch(r.attention, _ATTENTION.pack(*pages, q_at, out_at, lse.data_ptr() if return_lse else 0, q0, q1, o0, o1,
                                          table, lens_at, stride, workspace.data_ptr(), size,
                                          dh ** -0.5 if scale is None else scale, B, H, width, window,
                                          r.kinds.get(dtype, -1)), dev)
    return (out, lse) if return_lse else out


def rope_table(theta: float, head_dim: int, n_pos: int, device=None):
    """(cos, sin) of p * theta^(-2i / head_dim) for positions p < n_pos, in fp64 rounded to fp32 [n_pos, head_dim/2, 2]:
    the table that the decoder builds for itself."""
    torch = _torch()
    i = torch.arange(0, head_dim, 2, dtype=torch.float64)
    angle = torch.arange(n_pos, dtype=torch.float64)[:, None] * theta ** (-i / head_dim)
    return torch.stack([angle.cos(), angle.sin()], -1).float().to(device or torch.device("cuda"))


class PagedCache:
    """K/V pages of every layer of a model for up to max_seqs sequences, with their block table, lengths and free
    list, all on the GPU. A step: ``extend`` (pages and slots for the new tokens), then per layer ``append`` and
    ``attention``; ``release`` takes finished sequences' pages back; ``load`` copies a prompt that a Decoder has
    prefilled."""

    def __init__(self, model, n_blocks: int, block_size: int, max_seqs: int, max_blocks: int, dtype=None):
        torch = _torch()
        self.model, self.block_size = model, block_size
        self.device = torch.device("cuda", torch.cuda.current_device())
        shape = (model.n_layers, n_blocks, model.n_kv_heads, block_size, model.head_dim)
        dtype = dtype or torch.float16
        self.k, self.v = (torch.zeros(shape, dtype=dtype, device=self.device) for _ in range(2))
        fp8 = dtype == torch.float8_e4m3fn
        self.k_scale, self.v_scale = (torch.ones(shape[:4], device=self.device) if fp8 else None for _ in range(2))
        self.rope = rope_table(model.rope_theta, model.head_dim, max_blocks * block_size, self.device)
        ints = dict(dtype=torch.int32, device=self.device)
        self.block_table = torch.full((max_seqs, max_blocks), -1, **ints)
        self.lens = torch.zeros(max_seqs, **ints)
        self.free_blocks = torch.arange(n_blocks - 1, -1, -1, **ints)  # page 0 is given first
        self.n_free = torch.full((1,), n_blocks, **ints)

    def _layer(self, l: int) -> dict:
        scales = {} if self.k_scale is None else {"k_scale": self.k_scale[l], "v_scale": self.v_scale[l]}
        return {"k_cache": self.k[l], "v_cache": self.v[l], **scales}

    def extend(self, new_lens, n_rows: int) -> PagedStep:
        """Pages and slots for new_lens (int32 [max_seqs]) more tokens per sequence; updates lens and the free list."""
        step = paged_extend(new_lens, self.lens, self.block_table, self.free_blocks, self.n_free, self.block_size, n_rows)
        self.lens, self.n_free = step.lens, step.n_free
        return step

    def release(self, done) -> None:
        """Take back the pages of the sequences with done (bool [max_seqs])."""
        self.lens, self.n_free = paged_release(done, self.lens, self.block_table, self.free_blocks, self.n_free,
                                               self.block_size)

    def append(self, l: int, k, v, step: PagedStep, q=None, q_out=None):
        """Rotate and store layer l's K/V rows of a step; returns the rotated q."""
        return paged_append(k, v, slots=step.slots, positions=step.positions, rope=self.rope, q=q, q_out=q_out,
                            **self._layer(l))

    def attention(self, l: int, q, **kw):
        """Layer l's attention of one new token per sequence: q [max_seqs, n_heads, head_dim] (see paged_attention)."""
        return paged_attention(q, block_table=self.block_table, lens=self.lens, **self._layer(l), **kw)

    def load(self, decoder, step: PagedStep, first_row: int = 0) -> None:
        """Copy the prompt that `decoder` (a Decoder of this model) has prefilled, positions 0 .. position - 1 of
        every layer, to the slots of rows first_row .. of a step that extended a sequence by that many tokens. Waits
        for the decoder's stream."""
        torch = _torch()
        n, m, d = decoder.position, self.model, decoder
        decoder.sync()
        kv = d._kvbuf.view(torch.float16)[:2 * m.n_layers * m.n_kv_heads * d.max_seq * m.head_dim]
        kv = kv.view(m.n_layers, 2, m.n_kv_heads, d.max_seq, m.head_dim)[:, :, :, :n].transpose(2, 3)
        slots = step.slots[first_row:first_row + n]
        if slots.numel() != n:
            raise ValueError("the step has too few rows for the decoder's prompt")
        for l in range(m.n_layers):
            paged_append(kv[l, 0], kv[l, 1], slots=slots, k_pairs=True, **self._layer(l))
