"""A paged K/V cache for a batch of sequences: the ``kie_paged_*`` operators of include/kie.h on CUDA tensors.

``paged_extend``, ``paged_append``, ``paged_attention`` and ``paged_release``, and for sequences that share pages
``paged_fork``, ``paged_copy``, ``paged_compact`` and ``paged_prefix_attention``, with ``token_logprobs`` beside them,
check types, shapes and devices, allocate their outputs with PyTorch and launch on the current stream of the tensors'
device, without synchronising. What they marshal per call is done in native code (csrc/kie_paged_py.cpp). They are for
inference: no gradients pass through them.
``PagedCache`` holds the pages and tables that such a program keeps.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

from . import KieError, _torch, lib


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


class PagedFork(NamedTuple):
    """What paged_fork computed (CUDA tensors): lens per request, n_free, ok (bool [1]), and the rows to copy for each
    request, as paged_copy takes them."""
    lens: object
    n_free: object
    ok: object
    copy_src: object
    copy_dst: object
    copy_rows: object


class PagedMoves(NamedTuple):
    """What paged_compact computed (CUDA tensors): n_free; the moves src -> dst (-1 behind the last); page_map, the new id
    of each page (-1: free)."""
    n_free: object
    src: object
    dst: object
    page_map: object


class TokenLogprobs(NamedTuple):
    """What token_logprobs computed: logprob, entropy [N]; top_ids, top_logprobs [N, top]."""
    logprob: object
    entropy: object
    top_ids: object
    top_logprobs: object


_ready = None


def _native():
    """The marshalling module (csrc/kie_paged_py.cpp), bound to libkie.so. Raises without a GPU or before the build."""
    global _ready
    if _ready is None:
        _torch()
        L = lib()
        try:
            from . import _paged
        except ImportError as e:
            raise RuntimeError(f"the paged operators' binding cannot be loaded ({e}): run __graft_entry__.build() (or "
                               "persistent_monokernel_decode_gb300.build()) first") from e
        names = ("paged_extend", "paged_release", "paged_append", "paged_attention", "paged_attention_workspace",
                 "paged_last_error", "paged_prefix_attention", "paged_prefix_attention_workspace", "paged_fork", "paged_copy",
                 "paged_compact", "token_logprobs")
        _paged.bind(*[ctypes.cast(getattr(L, "kie_" + n), ctypes.c_void_p).value for n in names], KieError)
        _ready = _paged
    return _ready


def paged_extend(new_lens, lens, block_table, free_blocks, n_free, block_size: int, n_rows: int) -> PagedStep:
    """Pages and slots for new_lens[r] more tokens of each request r (kie_paged_extend): new entries go into
    block_table [R, max_blocks] in place, everything else into new tensors. lens, new_lens int32 [R]; free_blocks
    int32 (a stack whose first n_free[0] entries are free pages); n_rows >= sum(new_lens) rows are listed."""
    return PagedStep(*(_ready or _native()).extend(new_lens, lens, block_table, free_blocks, n_free, block_size, n_rows))


def paged_release(done, lens, block_table, free_blocks, n_free, block_size: int, shares=None):
    """Pages of the requests with done[r] (bool [R]) back onto free_blocks, in place (kie_paged_release). Returns
    (lens, n_free): 0 for the finished requests, and the new number of free pages. With shares (int32 [n_blocks], as
    paged_fork keeps it) a page goes back when its last holder is done."""
    return (_ready or _native()).release(done, lens, block_table, free_blocks, n_free, block_size, shares)


def paged_fork(parents, lens, block_table, shares, free_blocks, n_free, block_size: int) -> PagedFork:
    """Request r continues what request parents[r] (int32 [R]) held before the call, sharing its full pages; one of its own
    number, or one from R on, leaves it as it is, a negative one ends it (kie_paged_fork). block_table, free_blocks and
    shares (int32 [n_blocks]: the holders of each page beyond the first, zeros at first) are updated in place; the rows of
    half-filled pages have to be copied by paged_copy(f.copy_src, f.copy_dst, ..., rows=f.copy_rows) before the next
    append. If the free pages do not suffice, ok is False and nothing has changed."""
    return PagedFork(*(_ready or _native()).fork(parents, lens, block_table, shares, free_blocks, n_free, block_size))


def paged_copy(src, dst, k_cache, v_cache, *, rows=None, k_scale=None, v_scale=None) -> None:
    """Pages src[i] to dst[i] (int32) inside a cache: k_cache and v_cache of all layers [n_layers, n_blocks, n_kv_heads,
    block_size, head_dim], or of one, and their scales; rows (int32): only the first positions of each (kie_paged_copy).
    Pairs with a page that is none, such as -1, are left out."""
    (_ready or _native()).copy(src, dst, k_cache, v_cache, rows, k_scale, v_scale)


def paged_compact(lens, block_table, shares, free_blocks, n_free, block_size: int) -> PagedMoves:
    """The pages in use renumbered to lie at the cache's beginning (kie_paged_compact): block_table, shares and free_blocks
    are updated in place, and paged_copy(m.src, m.dst, ...) has to move what they hold before the next append or attention."""
    return PagedMoves(*(_ready or _native()).compact(lens, block_table, shares, free_blocks, n_free, block_size))


def token_logprobs(logits, tokens, *, top: int = 0) -> TokenLogprobs:
    """Log probabilities of tokens (int32 [N]; 0.0 where a token is none, such as -1) under softmax(logits), logits
    float16, bfloat16 or float32 [N, vocab] with contiguous rows; the entropy of each row; and its `top` (32 at most) most
    probable tokens in descending order, the lowest id first among equal ones (kie_token_logprobs)."""
    return TokenLogprobs(*(_ready or _native()).logprobs(logits, tokens, top))


def paged_append(k, v, k_cache, v_cache, slots, *, positions=None, rope=None, q=None, q_out=None, k_scale=None,
                 v_scale=None, k_pairs: bool = False):
    """K/V rows [T, n_kv_heads, head_dim] into their slots (int32 [T]) of the pages, rotated at `positions` by the
    table `rope` (fp32 [n_pos, head_dim / 2, 2], see rope_table) if it is given, and rounded to the pages' type
    (kie_paged_append). q [T, n_heads, head_dim], if given, is rotated into q_out, which is returned (new if None;
    rows whose slot is out of range are left as they were). Slots must not repeat."""
    return (_ready or _native()).append(k, v, k_cache, v_cache, slots, positions, rope, q, q_out, k_scale, v_scale, k_pairs)


def paged_attention(q, k_cache, v_cache, block_table, lens, *, scale=None, window: int = 0, k_scale=None, v_scale=None,
                    out=None, return_lse: bool = False, seqs=None, positions=None):
    """Attention of one new token per sequence over the pages (kie_paged_attention): q [B, n_heads, head_dim], lens
    int32 [B] positions cached (the new token's among them), block_table int32 [B, max_blocks]. scale: 1 /
    sqrt(head_dim) by default; window: only the last `window` positions (0: all). Returns out, or (out, lse) with
    lse fp32 [B, n_heads]. The workspace is allocated by the call, so calls on several streams and captured graphs
    share none.

    With seqs and positions (int32 [B], as a PagedStep lists them) and lens None, row t of q is the token at positions[t]
    of the sequence in row seqs[t] of block_table [R, max_blocks], and attends to the positions up to its own; rows of
    no sequence (-1) get zeros."""
    return (_ready or _native()).attention(q, k_cache, v_cache, block_table, lens, scale, window, k_scale, v_scale, out,
                                           return_lse, seqs, positions)


def paged_prefix_attention(q, k_cache, v_cache, block_table, lens, group_start, prefix_lens, *, scale=None, k_scale=None,
                           v_scale=None, out=None, return_lse: bool = False, seqs=None, positions=None):
    """paged_attention (without a window) for rows that share beginnings, which are read once for all of them
    (kie_paged_prefix_attention): rows group_start[g] .. group_start[g + 1] - 1 of q (int32 [G + 1]) have the same first
    prefix_lens[g] positions (int32 [G]), read through the block table row of the group's longest row. Rows outside the
    groups attend as in paged_attention."""
    return (_ready or _native()).prefix_attention(q, k_cache, v_cache, block_table, lens, scale, 0, k_scale, v_scale, out,
                                                  return_lse, seqs, positions, group_start, prefix_lens)


def paged_set_timeout_ns(ns: int) -> None:
    """How long a wait inside paged_prefix_attention may take (2 seconds at first), for all later calls of the process: what
    a wait that runs out concerns is NaN (kie_paged_set_timeout_ns)."""
    if not 0 < ns < 1 << 64:
        raise ValueError("ns must be above 0 and fit 64 bits")
    lib().kie_paged_set_timeout_ns(ns)


def rope_table(theta: float, head_dim: int, n_pos: int, device=None):
    """(cos, sin) of p * theta^(-2i / head_dim) for positions p < n_pos, in fp64 rounded to fp32 [n_pos, head_dim/2, 2]:
    the table that the decoder builds for itself."""
    torch = _torch()
    i = torch.arange(0, head_dim, 2, dtype=torch.float64)
    angle = torch.arange(n_pos, dtype=torch.float64)[:, None] * theta ** (-i / head_dim)
    return torch.stack([angle.cos(), angle.sin()], -1).float().to(device or torch.device("cuda"))


class PagedCache:
    """K/V pages of every layer of a model for up to max_seqs sequences, with their block table, lengths and free
    list, all on the GPU at fixed addresses. A step: ``extend`` (pages and slots for the new tokens), then per layer ``append`` and
    ``attention``; ``release`` takes finished sequences' pages back; ``load`` copies a prompt that a Decoder has
    prefilled. With shared=True sequences may share pages: ``fork`` lets sequences continue others."""

    def __init__(self, model, n_blocks: int, block_size: int, max_seqs: int, max_blocks: int, dtype=None,
                 shared: bool = False):
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
        self.shares = torch.zeros(n_blocks, **ints) if shared else None  # holders of each page beyond the first

    def _layer(self, l: int) -> dict:
        scales = {} if self.k_scale is None else {"k_scale": self.k_scale[l], "v_scale": self.v_scale[l]}
        return {"k_cache": self.k[l], "v_cache": self.v[l], **scales}

    def extend(self, new_lens, n_rows: int) -> PagedStep:
        """Pages and slots for new_lens (int32 [max_seqs]) more tokens per sequence. lens, the table and the free list
        are updated in place, so that a captured step goes on from where its last replay ended."""
        step = paged_extend(new_lens, self.lens, self.block_table, self.free_blocks, self.n_free, self.block_size, n_rows)
        self._update(step.lens, step.n_free)
        return step

    def _update(self, lens, n_free) -> None:
        _torch()._foreach_copy_([self.lens, self.n_free], [lens, n_free])

    def release(self, done) -> None:
        """Take back the pages of the sequences with done (bool [max_seqs])."""
        self._update(*paged_release(done, self.lens, self.block_table, self.free_blocks, self.n_free, self.block_size,
                                    self.shares))

    def _copy(self, src, dst, rows=None) -> None:
        paged_copy(src, dst, self.k, self.v, rows=rows, k_scale=self.k_scale, v_scale=self.v_scale)

    def fork(self, parents) -> PagedFork:
        """Let sequence r go on from what sequence parents[r] (int32 [max_seqs]) holds; r itself leaves it as it is, -1 ends
        it. See paged_fork; where ok is False in the result, pages did not suffice and nothing has changed."""
        if self.shares is None:
            raise ValueError("sequences can be forked in a PagedCache of shared=True only")
        f = paged_fork(parents, self.lens, self.block_table, self.shares, self.free_blocks, self.n_free, self.block_size)
        self._copy(f.copy_src, f.copy_dst, f.copy_rows)
        self._update(f.lens, f.n_free)
        return f

    def compact(self) -> PagedMoves:
        """Move the pages in use to the beginning of the cache: afterwards they are pages 0 .. n_blocks - n_free - 1. See
        paged_compact; page_map in the result gives the new id of each page."""
        torch = _torch()
        shares = self.shares if self.shares is not None else torch.zeros(self.k.shape[1], dtype=torch.int32, device=self.device)
        m = paged_compact(self.lens, self.block_table, shares, self.free_blocks, self.n_free, self.block_size)
        self._copy(m.src, m.dst)
        self.n_free.copy_(m.n_free)
        return m

    def append(self, l: int, k, v, step: PagedStep, q=None, q_out=None):
        """Rotate and store layer l's K/V rows of a step (packed in its order); returns the rotated q, packed likewise."""
        return paged_append(k, v, slots=step.slots, positions=step.positions, rope=self.rope, q=q, q_out=q_out,
                            **self._layer(l))

    def attention(self, l: int, q, step: PagedStep | None = None, *, groups=None, **kw):
        """Layer l's attention of a step's rows, q [n_rows, n_heads, head_dim] as `append` returned it, each over its own
        sequence up to its own position (rows that were not admitted get zeros). Without a step, q [max_seqs, n_heads,
        head_dim] holds one row per sequence, sequence b's newest token in row b: a step's rows lie like that only if it
        brought exactly one token for every sequence. See paged_attention. groups = (group_start, prefix_lens): neighbouring
        rows of q share beginnings, which are read once; see paged_prefix_attention."""
        rows = {"lens": self.lens} if step is None else {"lens": None, "seqs": step.seqs, "positions": step.positions}
        if groups is None:
            return paged_attention(q, block_table=self.block_table, **rows, **self._layer(l), **kw)
        return paged_prefix_attention(q, block_table=self.block_table, group_start=groups[0], prefix_lens=groups[1], **rows,
                                      **self._layer(l), **kw)

    def load(self, decoder, step: PagedStep, first_row: int = 0) -> None:
        """Copy the prompt that `decoder` (a Decoder of this model) has prefilled, positions 0 .. position - 1 of
        every layer, to the slots of rows first_row .. of a step that extended a sequence by that many tokens.
        Synchronous, like the prefill. Raises ValueError, and copies nothing, unless those rows are positions 0 .. position - 1
        of one admitted sequence and the decoder's cache has this model's layers and heads."""
        torch = _torch()
        n, m, d = decoder.position, self.model, decoder
        if any(getattr(d.model, x) != getattr(m, x) for x in ("n_layers", "n_kv_heads", "head_dim")):
            raise ValueError("the decoder's model has other layers or K/V heads")
        if first_row < 0:
            raise ValueError("first_row must be >= 0")
        decoder.sync()
        kv = d._kvbuf.view(torch.float16)[:2 * m.n_layers * m.n_kv_heads * d.max_seq * m.head_dim]
        kv = kv.view(m.n_layers, 2, m.n_kv_heads, d.max_seq, m.head_dim)[:, :, :, :n].transpose(2, 3)
        slots = step.slots[first_row:first_row + n]
        if slots.numel() != n:
            raise ValueError("the step has too few rows for the decoder's prompt")
        seqs, positions = (x[first_row:first_row + n].tolist() for x in (step.seqs, step.positions))
        if n and (seqs[0] < 0 or seqs != seqs[:1] * n or positions != list(range(n))):
            raise ValueError("the step's rows are not positions 0 .. position - 1 of one admitted sequence")
        for l in range(m.n_layers):
            paged_append(kv[l, 0], kv[l, 1], slots=slots, k_pairs=True, **self._layer(l))
        torch.cuda.current_stream(self.device).synchronize()  # the decoder may go on, on whatever stream it has
