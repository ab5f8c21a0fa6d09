"""The paged serving calls for torch CUDA tensors.

A context decoded into a paged pool (``torch_api.decode_into_paged``) is
continued here: ``PagedTables`` makes the block tables and slot maps of a
batch, ``PagedAppend`` norms, rotates and stores the batch's new tokens, and
``PagedAttention`` attends over the pool, with a sliding window and sinks or
behind a shared prefix.  Each object holds what a program keeps between calls
(argument block, workspace, status word) for one geometry and one device; the
math runs in libcachegen's kernels.  Nothing here synchronises: data errors go
to ``status``, which the caller reads after synchronising
(``torch_api.status_of``).  Work is queued on ``stream``, or on the current
stream of the object's device; an object is used by one stream at a time, and
buffers that belong to another stream are the caller's to order, as everywhere
in this package.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import (CG_DTYPE_BF16, CG_DTYPE_F16, AppendArgs, AttentionArgs, ExtendArgs, Shape,
               cg_attention_workspace_bytes, check, library)

# torch.int16 holds fp16 bits, as everywhere in this package
_DTYPES = {torch.float16: CG_DTYPE_F16, torch.int16: CG_DTYPE_F16,
           torch.bfloat16: CG_DTYPE_BF16}


def _code(dtype: torch.dtype) -> int:
    if dtype not in _DTYPES:
        raise ValueError(f"dtype must be float16 (or int16 bits) or bfloat16, not {dtype}")
    return _DTYPES[dtype]


class _Call:
    """Device, status word and launch of one object's calls."""

    def __init__(self, device, status):
        self.device = torch.device(device)
        if self.device.type != "cuda":
            raise ValueError("the paged calls run on CUDA devices")
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.status = (torch.zeros(1, dtype=torch.int32, device=self.device)
                       if status is None else status)

    def _vector(self, t: torch.Tensor, name: str, dtype, count: int | None = None) -> int:
        if t.dtype != dtype or t.device != self.device or not t.is_contiguous() or \
                (count is not None and t.numel() < count):
            raise ValueError(f"{name} must be a contiguous {dtype} tensor on {self.device}"
                             + (f" with at least {count} entries" if count is not None else ""))
        return t.data_ptr()

    def _rows(self, t: torch.Tensor, name: str, heads: int, dim: int, code: int) -> int:
        """Token stride of [N, heads, dim] rows whose heads are contiguous."""
        if t.device != self.device or _DTYPES.get(t.dtype) != code or t.dim() != 3 or \
                t.shape[1] != heads or t.shape[2] != dim:
            raise ValueError(f"{name} must be [N, {heads}, {dim}] of the object's type on "
                             f"{self.device}")
        s0, s1, s2 = t.stride()
        if (s2 != 1 and dim > 1) or (s1 != dim and heads > 1):
            raise ValueError(f"{name}'s heads must be contiguous within a token")
        return s0 if t.shape[0] > 1 else max(s0, heads * dim)

    def _pool(self, pool: torch.Tensor, shape: Shape, code: int) -> tuple[int, int]:
        if pool.device != self.device or _DTYPES.get(pool.dtype) != code or pool.dim() != 6 or \
                not pool.is_contiguous() or pool.shape[0] != shape.num_layers or \
                pool.shape[1] != 2 or pool.shape[4] != shape.num_kv_heads or \
                pool.shape[5] != shape.head_dim:
            raise ValueError("pool must be a contiguous [L, 2, num_pages, page_tokens, H, D] "
                             f"tensor of the object's type on {self.device}")
        return pool.shape[2], pool.shape[3]

    def _launch(self, fn, stream, *args) -> None:
        """fn(*args, stream) with this object's device current."""
        if stream is None:
            handle = torch.cuda.current_stream(self.device).cuda_stream
        else:
            handle = stream if isinstance(stream, int) else stream.cuda_stream
        if torch.cuda.current_device() == self.device.index:
            rc = fn(*args, handle)
        else:
            with torch.cuda.device(self.device):
                rc = fn(*args, handle)
        if rc:
            check(rc, fn.__name__)


class PagedTables(_Call):
    """Block tables and slot maps of a batch of ``num_requests`` requests that
    adds at most ``max_tokens`` tokens a call (cg_extend_tables).  The outputs
    are this object's buffers: kv_lens, q_starts, slots, positions, taken."""

    def __init__(self, num_requests: int, max_tokens: int, page_tokens: int, num_pages: int,
                 device, status: torch.Tensor | None = None):
        super().__init__(device, status)
        self.num_requests, self.max_tokens = num_requests, max_tokens
        dev = self.device
        self.kv_lens = torch.zeros(num_requests, dtype=torch.int32, device=dev)
        self.q_starts = torch.zeros(num_requests + 1, dtype=torch.int32, device=dev)
        self.slots = torch.full((max_tokens,), -1, dtype=torch.int64, device=dev)
        self.positions = torch.full((max_tokens,), -1, dtype=torch.int32, device=dev)
        self.taken = torch.zeros(1, dtype=torch.int32, device=dev)
        a = self._args = ExtendArgs()
        a.num_requests, a.max_tokens = num_requests, max_tokens
        a.page_tokens, a.num_pages = page_tokens, num_pages
        a.kv_lens, a.q_starts = self.kv_lens.data_ptr(), self.q_starts.data_ptr()
        a.slots, a.positions = self.slots.data_ptr(), self.positions.data_ptr()
        a.taken_out, a.status = self.taken.data_ptr(), self.status.data_ptr()
        self._ref = ctypes.byref(a)
        self._fn = library().cg_extend_tables

    def extend(self, held: torch.Tensor, added: torch.Tensor, block_tables: torch.Tensor,
               free_pages: torch.Tensor, taken: torch.Tensor | None = None,
               position_base: int = 0, stream=None) -> None:
        """held and added: int32 [num_requests] (held may be ``kv_lens``);
        block_tables: int32 [num_requests, max_pages], extended in place;
        free_pages: int32 page ids; taken: how many of them are handed out
        already (default: this object's own count)."""
        a = self._args
        if block_tables.dim() != 2 or block_tables.shape[0] != self.num_requests:
            raise ValueError("block_tables must be [num_requests, max_pages]")
        a.held = self._vector(held, "held", torch.int32, self.num_requests)
        a.added = self._vector(added, "added", torch.int32, self.num_requests)
        a.block_tables = self._vector(block_tables, "block_tables", torch.int32)
        a.max_pages = block_tables.shape[1]
        a.free_pages = self._vector(free_pages, "free_pages", torch.int32)
        a.num_free = free_pages.numel()
        a.taken = self._vector(self.taken if taken is None else taken, "taken", torch.int32, 1)
        a.position_base = position_base
        self._launch(self._fn, stream, self._ref)


def rope_table(max_positions: int, rot_dim: int, device, theta: float = 10000.0,
               stream=None) -> torch.Tensor:
    """The [max_positions, rot_dim] table of PagedAppend: cosines, then sines."""
    call = _Call(device, None)
    out = torch.empty((max_positions, rot_dim), dtype=torch.float32, device=call.device)
    call._launch(library().cg_rope_table, stream, max_positions, rot_dim, theta, out.data_ptr())
    return out


class PagedAppend(_Call):
    """Norm, rotate and store new tokens (cg_append_qkv)."""

    def __init__(self, shape, num_q_heads: int, dtype: torch.dtype, device,
                 status: torch.Tensor | None = None):
        super().__init__(device, status)
        self.shape = shape if isinstance(shape, Shape) else Shape(*shape)
        self.num_q_heads, self._type = num_q_heads, _code(dtype)
        a = self._args = AppendArgs()
        a.num_q_heads, a.dtype, a.status = num_q_heads, self._type, self.status.data_ptr()
        self._refs = ctypes.byref(self.shape), ctypes.byref(a)
        self._fn = library().cg_append_qkv

    def append(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_out: torch.Tensor,
               pool: torch.Tensor, layer: int, positions: torch.Tensor | None,
               slots: torch.Tensor, rope: torch.Tensor | None, q_weight=None, k_weight=None,
               eps: float = 1e-6, interleaved: bool = False, stream=None) -> None:
        """q [N, Hq, D], k and v [N, H, D] (views of one packed tensor will do),
        q_out like q (or q itself); positions int32 [N] and slots int64 [N] as
        PagedTables makes them; rope: rope_table's, or None for no rotation;
        weights [D], or None for no norm."""
        a, s, code = self._args, self.shape, self._type
        n, h, d = q.shape[0], s.num_kv_heads, s.head_dim
        a.q_stride = self._rows(q, "q", self.num_q_heads, d, code)
        a.k_stride = self._rows(k, "k", h, d, code)
        a.v_stride = self._rows(v, "v", h, d, code)
        a.q_out_stride = self._rows(q_out, "q_out", self.num_q_heads, d, code)
        if k.shape[0] != n or v.shape[0] != n or q_out.shape[0] != n:
            raise ValueError("q, k, v and q_out must have the same number of tokens")
        a.q, a.k, a.v, a.q_out = q.data_ptr(), k.data_ptr(), v.data_ptr(), q_out.data_ptr()
        a.num_tokens, a.layer = n, layer
        a.num_pages, a.page_tokens = self._pool(pool, s, code)
        a.pool = pool.data_ptr()
        a.slots = self._vector(slots, "slots", torch.int64, n)
        a.rot_dim = a.max_positions = 0
        a.rope = a.positions = None
        if rope is not None:
            if rope.dim() != 2:
                raise ValueError("rope must be [max_positions, rot_dim]")
            a.rope = self._vector(rope, "rope", torch.float32)
            a.max_positions, a.rot_dim = rope.shape
            a.positions = self._vector(positions, "positions", torch.int32, n)
        for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
            if w is not None:
                if _DTYPES.get(w.dtype) != code:
                    raise ValueError(f"{name} must be of the object's type")
                self._vector(w, name, w.dtype, d)
            setattr(a, name, None if w is None else w.data_ptr())
        a.eps, a.interleaved = eps, int(interleaved)
        self._launch(self._fn, stream, *self._refs)


class PagedAttention(_Call):
    """Attention over the paged pool (cg_attention_paged, cg_attention_shared)
    for at most max_tokens query rows of max_requests requests; holds the
    workspace."""

    def __init__(self, shape, num_q_heads: int, dtype: torch.dtype, max_tokens: int,
                 max_requests: int, device, status: torch.Tensor | None = None):
        super().__init__(device, status)
        self.shape = shape if isinstance(shape, Shape) else Shape(*shape)
        self.num_q_heads, self._type = num_q_heads, _code(dtype)
        self.max_tokens, self.max_requests = max_tokens, max_requests
        a = self._args = AttentionArgs()
        a.num_q_heads, a.dtype, a.status = num_q_heads, self._type, self.status.data_ptr()
        self._refs = ctypes.byref(self.shape), ctypes.byref(a)
        self._fn, self._shared_fn = library().cg_attention_paged, library().cg_attention_shared
        self._scale = 1.0 / math.sqrt(self.shape.head_dim)
        self.workspace = None
        self._reserve(False)

    def _reserve(self, shared: bool) -> None:
        need = cg_attention_workspace_bytes(self.shape, self.num_q_heads, self.max_tokens,
                                            self.max_requests, shared)
        if self.workspace is None or self.workspace.numel() < need:
            self.workspace = torch.empty(need, dtype=torch.uint8, device=self.device)
            self._args.workspace = self.workspace.data_ptr()
            self._args.workspace_bytes = need
        self._has_shared = shared

    def reserve_shared(self) -> None:
        """Size the workspace for run_shared now (its first call does so
        otherwise), for a program that captures its first call."""
        if not self._has_shared:
            self._reserve(True)

    def _set(self, q, pool, layer, q_starts, kv_lens, block_tables, max_q, out, scale, lse):
        a, s, code = self._args, self.shape, self._type
        n, requests = q.shape[0], kv_lens.numel()
        if n > self.max_tokens or requests > self.max_requests:
            raise ValueError("more rows or requests than this object was made for")
        a.q_stride = self._rows(q, "q", self.num_q_heads, s.head_dim, code)
        a.out_stride = self._rows(out, "out", self.num_q_heads, s.head_dim, code)
        if out.shape[0] != n:
            raise ValueError("out must have as many rows as q")
        if block_tables.dim() != 2 or block_tables.shape[0] != requests:
            raise ValueError("block_tables must be [num_requests, max_pages]")
        a.q, a.out, a.num_tokens, a.num_requests = q.data_ptr(), out.data_ptr(), n, requests
        a.max_q, a.layer = max_q, layer
        a.num_pages, a.page_tokens = self._pool(pool, s, code)
        a.pool = pool.data_ptr()
        a.q_starts = self._vector(q_starts, "q_starts", torch.int32, requests + 1)
        a.kv_lens = self._vector(kv_lens, "kv_lens", torch.int32)
        a.block_tables = self._vector(block_tables, "block_tables", torch.int32)
        a.max_pages = block_tables.shape[1]
        a.scale = self._scale if scale is None else scale
        a.lse = None if lse is None else self._vector(lse, "lse", torch.float32,
                                                      n * self.num_q_heads)

    def run(self, q: torch.Tensor, pool: torch.Tensor, layer: int, q_starts: torch.Tensor,
            kv_lens: torch.Tensor, block_tables: torch.Tensor, max_q: int, out: torch.Tensor,
            window: int = 0, sinks: int = 0, scale: float | None = None,
            lse: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """q and out: [N, Hq, D]; q_starts int32 [B + 1], kv_lens int32 [B] and
        block_tables int32 [B, max_pages] as PagedTables makes them; max_q: no
        request has more new tokens; window 0: no window; scale: 1 / sqrt(D)
        by default; lse: fp32 [N, Hq] that receives the log-sums."""
        self._set(q, pool, layer, q_starts, kv_lens, block_tables, max_q, out, scale, lse)
        self._args.window, self._args.sinks = window, sinks
        self._launch(self._fn, stream, *self._refs)
        return out

    def run_shared(self, q: torch.Tensor, pool: torch.Tensor, layer: int,
                   prefix_table: torch.Tensor, prefix_tokens: int, q_starts: torch.Tensor,
                   kv_lens: torch.Tensor, block_tables: torch.Tensor, max_q: int,
                   out: torch.Tensor, scale: float | None = None,
                   lse: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """As run without a window, behind a prefix of prefix_tokens tokens in
        the pages of prefix_table (int32) that every request shares."""
        self.reserve_shared()
        self._set(q, pool, layer, q_starts, kv_lens, block_tables, max_q, out, scale, lse)
        a = self._args
        pages = -(-prefix_tokens // a.page_tokens)
        table = self._vector(prefix_table, "prefix_table", torch.int32, pages)
        a.window = a.sinks = 0
        self._launch(self._shared_fn, stream, *self._refs, table, prefix_tokens)
        return out
