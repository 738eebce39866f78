"""The paged 8-bit key / value cache for generation with a ragged batch.

``PagedCache`` holds the cache's tensors and calls the library on them:
``append`` puts tokens into it (rotating queries and keys on the way),
``advance`` moves the positions by what it took, ``decode`` lets one query per sequence attend it.  Which page a chunk gets is
the caller's choice, written into ``table``; ``PagedDecodeState`` hands pages
out in order and generates token by token, as ``DecodeState`` does on a dense
cache.  Positions and tables live on the device, so a captured step serves
every position.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import binding as B
from .binding import HGA_ALL, HGA_BF16, HGA_E4M3, HGA_INT8

_HELD = {HGA_INT8: torch.int8, HGA_E4M3: torch.float8_e4m3fn}


@dataclass(frozen=True)
class PagedParams:
    """Mirror of hga_paged_params.  k_c / k_g may be HGA_ALL (-1)."""
    B: int
    Hq: int
    Hkv: int
    d: int
    n_pages: int             # pages in the pool
    max_chunks: int          # chunks per sequence, at most (width of the table)
    k_c: int = HGA_ALL
    k_g: int = HGA_ALL
    dtype: int = HGA_BF16
    cache_dtype: int = HGA_INT8
    scale: float = 0.0

    @property
    def torch_dtype(self):
        return torch.bfloat16 if self.dtype == HGA_BF16 else torch.float32

    def c(self):
        return B._PagedParams(self.B, self.Hq, self.Hkv, self.d, self.max_chunks, self.n_pages, self.k_c, self.k_g,
                              float(self.scale), self.dtype, self.cache_dtype)


def paged_widths(p: PagedParams) -> tuple[int, int]:
    wc, wg = ctypes.c_int(), ctypes.c_int()
    B._check(B.load().hga_paged_widths(ctypes.byref(p.c()), ctypes.byref(wc), ctypes.byref(wg)))
    return wc.value, wg.value


def paged_workspace_size(p: PagedParams) -> int:
    """Bytes of device scratch that a dense decode call needs."""
    return int(B.load().hga_paged_workspace_size(ctypes.byref(p.c())))


def _dense(t, name, shape, dtype, dev):
    """Data pointer of a contiguous tensor on device `dev`, the current one."""
    if t.shape != shape or t.dtype is not dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {list(shape)}")
    if t.get_device() != dev:
        B._here(t, name, dev)                        # raises
    return t.data_ptr()


class PagedCache:
    """The tensors of a paged cache (include/hga.h, hga_paged_cache).  Tensors
    that are not given are allocated: the pool and the open rows zeroed, the
    table filled with -1 (no page).  Decode calls only read the cache; dense
    ones share its ``workspace``, so those that may overlap on the GPU are
    given others."""

    def __init__(self, p: PagedParams, device="cuda", **tensors):
        paged_widths(p)                              # the parameters are valid
        self.p = p
        f32, i32 = torch.float32, torch.int32
        held = _HELD[p.cache_dtype]
        shapes = dict(k_pages=((p.n_pages, p.Hkv, 64, p.d), held), v_pages=((p.n_pages, p.Hkv, 64, p.d), held),
                      k_scale=((p.n_pages, p.Hkv, 8), f32), v_scale=((p.n_pages, p.Hkv, 8), f32),
                      csum=((p.n_pages, p.Hkv, p.d), f32), gsum=((p.n_pages, p.Hkv, 8, p.d), f32),
                      k_tail=((p.B, p.Hkv, 64, p.d), f32), v_tail=((p.B, p.Hkv, 64, p.d), p.torch_dtype),
                      table=((p.B, p.max_chunks), i32))
        for name in tensors:
            if name not in shapes:
                raise ValueError(f"a paged cache has no tensor {name!r}")
        ptrs = []
        for name, (shape, dtype) in shapes.items():
            t = tensors.get(name)
            if t is None:
                t = (torch.full(shape, -1, dtype=dtype, device=device) if name == "table"
                     else torch.zeros(shape, dtype=dtype, device=device))
            elif t.shape != shape or t.dtype != dtype or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {list(shape)}")
            setattr(self, name, t)
            ptrs.append(B._here(t, name))
        self._p, self._c = p.c(), B._PagedCache(*ptrs)
        self._pp, self._pc = ctypes.byref(self._p), ctypes.byref(self._c)
        self._widths = paged_widths(p)
        n = paged_workspace_size(p)
        self.workspace = torch.empty(n, dtype=torch.uint8, device=self.table.device) if n else None
        lib = B.load()
        self._append, self._advance, self._decode = lib.hga_paged_append, lib.hga_paged_advance, lib.hga_paged_decode
        self._dtype = p.torch_dtype

    def _rows(self, t, name, N, H, dev):
        st, sh, sd = t.stride()
        if t.shape != (N, H, self.p.d) or t.dtype is not self._dtype or sd != 1:
            raise ValueError(f"{name} must be {self._dtype} rows [{N}][{H}][{self.p.d}] with unit stride along d")
        if t.get_device() != dev:
            B._here(t, name, dev)                    # raises
        return t.data_ptr(), st, sh

    def append(self, pos, k, v, cu=None, q=None, q_out=None, rope=None, interleaved: bool = False, stream=None):
        """Tokens cu[b] .. cu[b + 1] - 1 of k, v [N][Hkv][d] (and q [N][Hq][d])
        join sequence b at positions pos[b], pos[b] + 1, ... (int32, device;
        cu None: one token each).  q_out [N][Hq][d] gets the rotated queries;
        ``rope`` as of ``rope_table`` (None: k and q are taken as they are)."""
        p, dev = self.p, torch.cuda.current_device()
        N = k.shape[0]
        kp, kt, kh = self._rows(k, "k", N, p.Hkv, dev)
        vp, vt, vh = self._rows(v, "v", N, p.Hkv, dev)
        qp, qt, qh = (None, 0, 0) if q is None else self._rows(q, "q", N, p.Hq, dev)
        out = None if q_out is None else _dense(q_out, "q_out", (N, p.Hq, p.d), self._dtype, dev)
        table, rows, rot = None, 0, 0
        if rope is not None:
            rows, rot = rope.shape
            table = _dense(rope, "rope", (rows, rot), torch.float32, dev)
        code = self._append(
            self._pp, self._pc, _dense(pos, "pos", (p.B,), torch.int32, dev),
            None if cu is None else _dense(cu, "cu", (p.B + 1,), torch.int32, dev), N, qp, qt, qh, kp, kt, kh, vp, vt, vh,
            out, table, rows, rot, interleaved, B._raw_stream(stream, dev))
        if code:
            B._check(code)

    def advance(self, pos, cu=None, N=None, rope=None, last=None, stream=None):
        """pos[b] (int32, device) grows by the tokens that ``append`` took for
        sequence b from the same pos, cu and rope, N tokens in all (B without
        cu); none for an empty slot or past the cache's or the rotation
        table's end.  last [B] (int32) gets the position of the last one, or
        -1 where there was none."""
        p, dev = self.p, torch.cuda.current_device()
        if N is None:
            if cu is not None:
                raise ValueError("advance with offsets needs N, the tokens of the append")
            N = p.B
        rows, rot = (0, 0) if rope is None else rope.shape
        code = self._advance(
            self._pp, _dense(pos, "pos", (p.B,), torch.int32, dev),
            None if cu is None else _dense(cu, "cu", (p.B + 1,), torch.int32, dev), N, rows, rot,
            None if last is None else _dense(last, "last", (p.B,), torch.int32, dev), B._raw_stream(stream, dev))
        if code:
            B._check(code)

    def decode(self, pos, q, O, lse, cidx=None, gidx=None, workspace=None, stream=None):
        """The query q [B][Hq][d] of each sequence, at position pos[b] (int32,
        device; negative: empty), attends its cache: O [B][Hq][d] and lse
        [B][Hq] (float32), routing rows cidx [B][Hkv][wc], gidx [B][Hkv][wg]
        (int32; may be None when k_c = k_g = HGA_ALL: dense attention, with
        ``workspace`` of paged_workspace_size bytes, the cache's by default)."""
        p, dev = self.p, torch.cuda.current_device()
        wc, wg = self._widths
        ws = self.workspace if workspace is None else workspace
        if ws is not None and not ws.is_contiguous():          # (its bytes would not be its own)
            raise ValueError("workspace must be a contiguous tensor")
        code = self._decode(
            self._pp, self._pc, _dense(pos, "pos", (p.B,), torch.int32, dev),
            _dense(q, "q", (p.B, p.Hq, p.d), self._dtype, dev),
            _dense(O, "O", (p.B, p.Hq, p.d), torch.float32, dev), _dense(lse, "lse", (p.B, p.Hq), torch.float32, dev),
            None if cidx is None else _dense(cidx, "cidx", (p.B, p.Hkv, wc), torch.int32, dev),
            None if gidx is None else _dense(gidx, "gidx", (p.B, p.Hkv, wg), torch.int32, dev),
            None if ws is None else B._here(ws, "workspace", dev), 0 if ws is None else ws.numel() * ws.element_size(),
            B._raw_stream(stream, dev))
        if code:
            B._check(code)


class PagedDecodeState:
    """Generation with HGA from a paged 8-bit cache, a batch of sequences at
    positions of their own.

    Pages are handed out in order: sequence b's chunk c gets page
    b * max_chunks + c.  ``prefill`` appends prompts, each ``step`` appends one
    token per sequence and attends; both rotate by ``rope`` (``rope_table``)
    when it is given.  ``pos`` counts the tokens in the cache; ``step``
    advances it on the device, so a step can be captured and replayed.  A
    negative ``pos[b]`` is an empty slot: its tokens are passed over, its O is
    0, and it stays as it is until the program writes another position there
    (the old one, to go on with a sequence that was held).

    ``capacity`` is the most that a sequence can hold: the pages (``max_tokens``
    rounded up to whole chunks) or the rotation table's rows, which must not be
    fewer than ``max_tokens``.  What goes past it is not taken: ``pos`` stays,
    O is 0, and the fault is recorded on the device (``device_check``), since
    only the device knows the positions."""

    def __init__(self, B_: int, Hq: int, Hkv: int, d: int, max_tokens: int, k_c: int, k_g: int, dtype: int = HGA_BF16,
                 cache_dtype: int = HGA_INT8, scale: float = 0.0, rope=None, interleaved: bool = False,
                 device="cuda"):
        if max_tokens < 1:
            raise ValueError(f"max_tokens must be >= 1 (got {max_tokens})")
        chunks = -(-max_tokens // 64)
        self.capacity = 64 * chunks
        if rope is not None:
            B._check_table(rope, "rope")
            if rope.shape[0] < max_tokens:
                raise ValueError(f"a rotation table of {rope.shape[0]} rows is shorter than max_tokens={max_tokens}")
            self.capacity = min(self.capacity, rope.shape[0])
        self.p = p = PagedParams(B_, Hq, Hkv, d, B_ * chunks, chunks, k_c, k_g, dtype, cache_dtype, scale)
        i32 = dict(device=device, dtype=torch.int32)
        self.cache = PagedCache(p, table=torch.arange(B_ * chunks, **i32).view(B_, chunks))
        wc, wg = paged_widths(p)
        dense = k_c == HGA_ALL and k_g == HGA_ALL
        self.cidx = None if dense else torch.empty(B_, Hkv, wc, **i32)
        self.gidx = None if dense else torch.empty(B_, Hkv, wg, **i32)
        self.O = torch.empty(B_, Hq, d, device=device, dtype=torch.float32)
        self.lse = torch.empty(B_, Hq, device=device, dtype=torch.float32)
        self.q = torch.empty(B_, Hq, d, device=device, dtype=p.torch_dtype)
        self.pos = torch.zeros(B_, **i32)            # tokens in the cache; negative: an empty slot
        self.last = torch.full((B_,), -1, **i32)     # position of each sequence's newest token in a step, -1: it got none
        self.rope, self.interleaved = rope, interleaved

    def prefill(self, k, v, cu, stream=None):
        """Prompts k, v [N][Hkv][d] (unrotated), sequence b's tokens at
        cu[b] .. cu[b + 1] - 1 (int32, device)."""
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            self.cache.append(self.pos, k, v, cu=cu, rope=self.rope, interleaved=self.interleaved)
            self.cache.advance(self.pos, cu=cu, N=k.shape[0], rope=self.rope)

    def step(self, q, k, v, stream=None):
        """The next token of every sequence: q [B][Hq][d], k, v [B][Hkv][d];
        returns O [B][Hq][d] (float32, the state's buffer)."""
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            self.cache.append(self.pos, k, v, q=q, q_out=self.q, rope=self.rope, interleaved=self.interleaved)
            self.cache.advance(self.pos, rope=self.rope, last=self.last)
            self.cache.decode(self.last, self.q, self.O, self.lse, self.cidx, self.gidx)
        return self.O
