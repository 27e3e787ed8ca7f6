"""A paged K/V cache for a batch of sequences: the ``kie_paged_*`` operators of include/kie.h on CUDA tensors.

``paged_extend``, ``paged_append``, ``paged_attention`` and ``paged_release`` marshal arguments like the rest of the
binding: they check types, shapes and devices, allocate their outputs with PyTorch and launch on the current stream
of the tensors' device, without synchronising. ``PagedCache`` holds the pages and tables that such a program keeps.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

from . import (KIE_OK, KieError, KiePagedAppendArgs, KiePagedAttentionArgs, KiePagedExtendArgs, KiePagedReleaseArgs,
               _torch, lib)

KIE_F16, KIE_BF16, KIE_F32, KIE_E4M3 = 0, 1, 2, 3


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


def _dtypes(torch):
    return {torch.float16: KIE_F16, torch.bfloat16: KIE_BF16, torch.float32: KIE_F32, torch.float8_e4m3fn: KIE_E4M3}


def _check(rc):
    if rc != KIE_OK:
        raise KieError(rc, (lib().kie_paged_last_error() or b"").decode())


def _need(ok, msg):
    if not ok:
        raise ValueError(msg)


def _ints(torch, device, **tensors):
    """Contiguous int32 tensors on one device."""
    for name, t in tensors.items():
        _need(t.dtype == torch.int32 and t.is_contiguous() and t.device == device,
              f"{name} must be a contiguous int32 tensor on {device}")


def _table(torch, device, block_table, n_seqs):
    _need(block_table.dtype == torch.int32 and block_table.dim() == 2 and block_table.device == device and
          block_table.shape[0] == n_seqs and block_table.shape[1] >= 1 and block_table.stride(1) == 1,
          f"block_table must be an int32 [{n_seqs}, max_blocks] tensor on {device} with contiguous rows")


def _launch(torch, fn, args, device):
    """Call fn on the current stream of `device`, which is made the current device for the call."""
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            _check(fn(ctypes.byref(args), torch.cuda.current_stream().cuda_stream))
    else:
        _check(fn(ctypes.byref(args), torch.cuda.current_stream().cuda_stream))


def _pages(torch, p, k, v, k_scale, v_scale, device):
    """Fill a KiePages from page tensors [n_blocks, n_kv_heads, block_size, head_dim] (any outer strides)."""
    _need(k.dim() == 4 and k.shape == v.shape and k.dtype == v.dtype,
          "the pages are two tensors [n_blocks, n_kv_heads, block_size, head_dim] of one type")
    kind = _dtypes(torch).get(k.dtype)
    _need(kind is not None and kind != KIE_F32, f"pages are float16, bfloat16 or float8_e4m3fn, not {k.dtype}")
    _need(k.device == device and v.device == device and k.is_cuda, f"the pages must be on {device}")
    ks, vs = k.stride(), v.stride()
    _need(ks[3] == 1 and vs[3] == 1, "the pages' last dimension must be contiguous")
    p.k, p.v = k.data_ptr(), v.data_ptr()
    p.k_stride[:], p.v_stride[:] = ks[:3], vs[:3]
    p.n_blocks, p.n_kv_heads, p.block_size, p.head_dim = k.shape
    p.dtype = kind
    if kind == KIE_E4M3:
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            _need(t is not None and t.dtype == torch.float32 and t.shape == k.shape[:3] and t.device == device,
                  f"{name} must be a float32 [n_blocks, n_kv_heads, block_size] tensor on {device}")
        p.k_scale, p.v_scale = k_scale.data_ptr(), v_scale.data_ptr()
        p.k_scale_stride[:], p.v_scale_stride[:] = k_scale.stride(), v_scale.stride()
    else:
        _need(k_scale is None and v_scale is None, "only float8_e4m3fn pages have scales")
    return kind


def paged_extend(new_lens, lens, block_table, free_blocks, n_free, block_size: int, n_rows: int) -> PagedStep:
    """Pages and slots for new_lens[r] more tokens of each request r (kie_paged_extend): new entries go into
    block_table [R, max_blocks] in place, everything else into new tensors. lens, new_lens int32 [R]; free_blocks
    int32 (a stack whose first n_free[0] entries are free pages); n_rows >= sum(new_lens) rows are listed."""
    torch = _torch()
    dev, R = lens.device, lens.numel()
    _need(lens.is_cuda, "lens must be a CUDA tensor")
    _ints(torch, dev, lens=lens, new_lens=new_lens, free_blocks=free_blocks, n_free=n_free)
    _need(new_lens.numel() == R and n_free.numel() == 1, "new_lens must have a value per request, and n_free one")
    _table(torch, dev, block_table, R)
    _need(n_rows >= 0, "n_rows must be >= 0")
    ints = torch.empty(2 * R + 2 + 3 * n_rows, dtype=torch.int32, device=dev)
    lens_out, n_free_out, row_start, slots, positions, seqs = ints.split((R, 1, R + 1, n_rows, n_rows, n_rows))
    admitted = torch.empty(R, dtype=torch.bool, device=dev)
    at = ints.data_ptr()
    a = KiePagedExtendArgs(lens.data_ptr(), new_lens.data_ptr(), free_blocks.data_ptr(), n_free.data_ptr(),
                           block_table.data_ptr(), block_table.stride(0), at, at + 4 * R, at + 4 * (R + 1),
                           at + 4 * (2 * R + 2), at + 4 * (2 * R + 2 + n_rows), at + 4 * (2 * R + 2 + 2 * n_rows),
                           admitted.data_ptr(), R, block_table.shape[1], block_size, n_rows, free_blocks.numel())
    _launch(torch, lib().kie_paged_extend, a, dev)
    return PagedStep(lens_out, n_free_out, admitted, row_start, slots, positions, seqs)


def paged_release(done, lens, block_table, free_blocks, n_free, block_size: int):
    """Pages of the requests with done[r] (bool [R]) back onto free_blocks, in place (kie_paged_release). Returns
    (lens, n_free): 0 for the finished requests, and the new number of free pages."""
    torch = _torch()
    dev, R = lens.device, lens.numel()
    _need(lens.is_cuda, "lens must be a CUDA tensor")
    _ints(torch, dev, lens=lens, free_blocks=free_blocks, n_free=n_free)
    _need(done.dtype == torch.bool and done.numel() == R and done.is_contiguous() and done.device == dev,
          f"done must be a contiguous bool tensor of {R} on {dev}")
    _need(n_free.numel() == 1, "n_free must have one value")
    _table(torch, dev, block_table, R)
    lens_out, n_free_out = torch.empty(R + 1, dtype=torch.int32, device=dev).split((R, 1))
    at = lens_out.data_ptr()
    a = KiePagedReleaseArgs(done.data_ptr(), lens.data_ptr(), n_free.data_ptr(), block_table.data_ptr(),
                            block_table.stride(0), free_blocks.data_ptr(), at, at + 4 * R, R, block_table.shape[1],
                            block_size, free_blocks.numel())
    _launch(torch, lib().kie_paged_release, a, dev)
    return lens_out, n_free_out


def _rows(t, name, shape, dtype, device):
    _need(t.shape == shape and t.dtype == dtype and t.device == device and (t.stride(2) == 1),
          f"{name} must be a {dtype} {list(shape)} tensor on {device} with contiguous rows")


def paged_append(k, v, k_cache, v_cache, slots, *, positions=None, rope=None, q=None, q_out=None, k_scale=None,
                 v_scale=None, k_pairs: bool = False):
    """K/V rows [T, n_kv_heads, head_dim] into their slots (int32 [T]) of the pages, rotated at `positions` by the
    table `rope` (fp32 [n_pos, head_dim / 2, 2], see rope_table) if it is given, and rounded to the pages' type
    (kie_paged_append). q [T, n_heads, head_dim], if given, is rotated into q_out, which is returned (new if None;
    rows whose slot is out of range are left as they were). Slots must not repeat."""
    torch = _torch()
    dev = k.device
    a = KiePagedAppendArgs()
    _need(k.dim() == 3, "k must be [rows, n_kv_heads, head_dim]")
    _pages(torch, a.pages, k_cache, v_cache, k_scale, v_scale, dev)
    T, hkv, dh = k.shape
    _need(hkv == k_cache.shape[1] and dh == k_cache.shape[3], "k's heads or head_dim are not the pages'")
    a.x_dtype = _dtypes(torch).get(k.dtype, -1)
    _rows(k, "k", (T, hkv, dh), k.dtype, dev)
    _rows(v, "v", (T, hkv, dh), k.dtype, dev)
    _ints(torch, dev, slots=slots)
    _need(slots.numel() == T, "slots must have a value per row")
    a.k, a.v, a.slots = k.data_ptr(), v.data_ptr(), slots.data_ptr()
    a.k_stride[:], a.v_stride[:] = k.stride()[:2], v.stride()[:2]
    if rope is not None:
        _need(positions is not None, "a rope table needs positions")
        _ints(torch, dev, positions=positions)
        _need(positions.numel() == T, "positions must have a value per row")
        _need(rope.dtype == torch.float32 and rope.dim() == 3 and rope.shape[1:] == (dh // 2, 2) and
              rope.is_contiguous() and rope.device == dev,
              f"rope must be a contiguous float32 [n_pos, {dh // 2}, 2] tensor on {dev}")
        a.rope, a.positions, a.n_pos = rope.data_ptr(), positions.data_ptr(), rope.shape[0]
    if q is not None:
        _need(q.dim() == 3, "q must be [rows, n_heads, head_dim]")
        _rows(q, "q", (T, q.shape[1], dh), k.dtype, dev)
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=dev)
        _rows(q_out, "q_out", q.shape, k.dtype, dev)
        a.q, a.q_out, a.n_heads = q.data_ptr(), q_out.data_ptr(), q.shape[1]
        a.q_stride[:], a.q_out_stride[:] = q.stride()[:2], q_out.stride()[:2]
    a.n_rows, a.k_pairs = T, bool(k_pairs)
    _launch(torch, lib().kie_paged_append, a, dev)
    return q_out


_workspace = {}  # bytes by (device, heads, kv heads, head_dim)


def _workspace_bytes(torch, device, n_heads, n_kv_heads, head_dim):
    key = (device.index, n_heads, n_kv_heads, head_dim)
    if key not in _workspace:
        with torch.cuda.device(device):
            _workspace[key] = lib().kie_paged_attention_workspace(n_heads, n_kv_heads, head_dim)
    return _workspace[key]


def paged_attention(q, k_cache, v_cache, block_table, lens, *, scale=None, window: int = 0, k_scale=None, v_scale=None,
                    out=None, return_lse: bool = False):
    """Attention of one new token per sequence over the pages (kie_paged_attention): q [B, n_heads, head_dim], lens
    int32 [B] positions cached (the new token's among them), block_table int32 [B, max_blocks]. scale: 1 /
    sqrt(head_dim) by default; window: only the last `window` positions (0: all). Returns out, or (out, lse) with
    lse fp32 [B, n_heads]. The workspace is allocated by the call, so calls on several streams and captured graphs
    share none."""
    torch = _torch()
    dev = q.device
    a = KiePagedAttentionArgs()
    _need(q.dim() == 3 and q.is_cuda, "q must be a CUDA tensor [sequences, n_heads, head_dim]")
    _pages(torch, a.pages, k_cache, v_cache, k_scale, v_scale, dev)
    B, H, dh = q.shape
    _need(dh == k_cache.shape[3], "q's head_dim is not the pages'")
    _rows(q, "q", (B, H, dh), q.dtype, dev)
    _ints(torch, dev, lens=lens)
    _need(lens.numel() == B, "lens must have a value per sequence")
    _table(torch, dev, block_table, B)
    if out is None:
        out = torch.empty((B, H, dh), dtype=q.dtype, device=dev)
    else:
        _rows(out, "out", (B, H, dh), q.dtype, dev)
    a.q, a.out, a.q_dtype = q.data_ptr(), out.data_ptr(), _dtypes(torch).get(q.dtype, -1)
    a.q_stride[:], a.out_stride[:] = q.stride()[:2], out.stride()[:2]
    lse = None
    if return_lse:
        lse = torch.empty((B, H), dtype=torch.float32, device=dev)
        a.lse = lse.data_ptr()
    size = _workspace_bytes(torch, dev, H, k_cache.shape[1], dh)
    workspace = torch.empty(max(size, 1), dtype=torch.uint8, device=dev)
    a.workspace, a.workspace_bytes = workspace.data_ptr(), size
    a.block_table, a.table_stride, a.lens = block_table.data_ptr(), block_table.stride(0), lens.data_ptr()
    a.scale = dh ** -0.5 if scale is None else scale
    a.n_seqs, a.n_heads, a.max_blocks, a.window = B, H, block_table.shape[1], window
    _launch(torch, lib().kie_paged_attention, a, dev)
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
        _need(slots.numel() == n, "the step has too few rows for the decoder's prompt")
        for l in range(m.n_layers):
            paged_append(kv[l, 0], kv[l, 1], slots=slots, k_pairs=True, **self._layer(l))
