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
stream of the object's device; an object is used by one stream, and one host
thread, at a time.  Its own buffers may be used on any stream: one that is new
to the object waits until they are made.  (A captured call does not wait:
``torch.cuda.graph`` has waited for the device before it captures, and a
program that begins a capture otherwise synchronises after making the object.)
A graph that captured an object's calls uses its buffers: keep the object as
long as the graph, and replay both in order as calls of one object are.
The caller's tensors are the caller's to order and to keep, as everywhere in
this package.
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

from . import (CG_DTYPE_BF16, CG_DTYPE_F16, AppendArgs, AttentionArgs, ExtendArgs, Shape,
               cg_attention_workspace_bytes, check, library)

# torch.int16 holds fp16 bits, as everywhere in this package
_DTYPES = {torch.float16: (CG_DTYPE_F16, (torch.float16, torch.int16)),
           torch.int16: (CG_DTYPE_F16, (torch.float16, torch.int16)),
           torch.bfloat16: (CG_DTYPE_BF16, (torch.bfloat16,))}

# The argument blocks are filled in one go: a single-token step costs a few
# microseconds on the GPU, and setting 25 fields one by one as many here.
_EXTEND = struct.Struct("@7i11P")
_APPEND = struct.Struct("@9if3P3qPq7P")
_ATTENTION = struct.Struct("@11if2P2q7PQ")
assert (_EXTEND.size, _APPEND.size, _ATTENTION.size) == tuple(
    map(ctypes.sizeof, (ExtendArgs, AppendArgs, AttentionArgs)))

# The current stream's handle and device of a call: a microsecond cheaper by
# torch's private names, where it has them.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)
_get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _capturing(stream: torch.cuda.Stream) -> bool:
    with torch.cuda.stream(stream):
        return torch.cuda.is_current_stream_capturing()


class _Call:
    """Device, value type, status word and launch of one object's calls."""

    def __init__(self, device, status, dtype: torch.dtype = torch.float16):
        self.device = torch.device(device)
        if self.device.type != "cuda":
            raise ValueError("the paged calls run on CUDA devices")
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        if dtype not in _DTYPES:
            raise ValueError(f"dtype must be float16 (or int16 bits) or bfloat16, not {dtype}")
        self._index = self.device.index
        self._code, self._dtypes = _DTYPES[dtype]
        self.status = (torch.zeros(1, dtype=torch.int32, device=self.device)
                       if status is None else status)
        self._status = self._vector(self.status, "status", torch.int32, 1)
        self._ready = None
        self._buffers = ()
        self._made(self.status)

    def _vector(self, t: torch.Tensor, name: str, dtype, count: int = 0) -> int:
        if t.dtype is not dtype or t.get_device() != self._index or not t.is_contiguous() or \
                t.numel() < count:
            raise ValueError(f"{name} must be a contiguous {dtype} tensor on {self.device}"
                             + (f" with at least {count} entries" if count else ""))
        return t.data_ptr()

    def _rows(self, t: torch.Tensor, name: str, tokens: int, heads: int, dim: int) -> int:
        """Token stride of [tokens, heads, dim] rows whose heads are contiguous."""
        if t.dim() != 3 or t.shape != (tokens, heads, dim) or t.dtype not in self._dtypes or \
                t.get_device() != self._index:
            raise ValueError(f"{name} must be [{tokens}, {heads}, {dim}] of the object's type on "
                             f"{self.device}")
        s0, s1, s2 = t.stride()
        if s2 != 1 or (s1 != dim and heads > 1):
            raise ValueError(f"{name}'s heads must be contiguous within a token")
        return s0 if tokens > 1 else max(s0, heads * dim)

    def _pool(self, pool: torch.Tensor, shape: Shape) -> tuple[int, int]:
        if pool.dim() == 6:
            layers, two, pages, page_tokens, heads, dim = pool.shape
            if layers == shape.num_layers and two == 2 and heads == shape.num_kv_heads and \
                    dim == shape.head_dim and pool.dtype in self._dtypes and \
                    pool.get_device() == self._index and pool.is_contiguous():
                return pages, page_tokens
        raise ValueError("pool must be a contiguous [L, 2, num_pages, page_tokens, H, D] "
                         f"tensor of the object's type on {self.device}")

    def _made(self, *buffers: torch.Tensor) -> None:
        """Add buffers that have been made on the current stream to the object's."""
        self._buffers += buffers
        here = torch.cuda.current_stream(self.device)
        self._seen = set()  # streams that know the buffers
        if not _capturing(here):  # a capture has memory of its own, which nothing still uses
            self._ready = torch.cuda.Event()
            self._ready.record(here)
            self._seen.add(here.cuda_stream)

    def _meet(self, handle: int) -> None:
        """Have a stream that is new to the buffers wait until they are made
        (their memory may come from work that is still queued), and tell the
        caching allocator that it uses them, so that their memory is not handed
        out again before that stream is done with them."""
        s = (torch.cuda.ExternalStream(handle, device=self.device) if handle
             else torch.cuda.default_stream(self.device))
        for t in self._buffers:
            t.record_stream(s)
        if _capturing(s):
            return  # cannot wait for what is outside of its capture; met again later
        if self._ready is not None:
            s.wait_event(self._ready)
        self._seen.add(handle)

    def _launch(self, fn, stream, *args) -> None:
        """fn(*args, stream) with this object's device current."""
        if stream is None:
            handle = _raw_stream(self._index)
        else:
            handle = stream if isinstance(stream, int) else stream.cuda_stream
        if handle not in self._seen:
            self._meet(handle)
        if _get_device() == self._index:
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
        self.page_tokens, self.num_pages = page_tokens, num_pages
        dev = self.device
        self.kv_lens = torch.zeros(num_requests, dtype=torch.int32, device=dev)
        self.q_starts = torch.zeros(num_requests + 1, dtype=torch.int32, device=dev)
        self.slots = torch.full((max_tokens,), -1, dtype=torch.int64, device=dev)
        self.positions = torch.full((max_tokens,), -1, dtype=torch.int32, device=dev)
        self.taken = torch.zeros(1, dtype=torch.int32, device=dev)
        self._made(self.kv_lens, self.q_starts, self.slots, self.positions, self.taken)
        self._args = ExtendArgs()
        self._ref = ctypes.byref(self._args)
        self._fn = library().cg_extend_tables

    def extend(self, held: torch.Tensor, added: torch.Tensor, block_tables: torch.Tensor,
               free_pages: torch.Tensor, taken: torch.Tensor | None = None,
               position_base: int = 0, stream=None) -> None:
        """held and added: int32 [num_requests] (held may be ``kv_lens``);
        block_tables: int32 [num_requests, max_pages], extended in place;
        free_pages: int32 page ids; taken: how many of them are handed out
        already (default: this object's own count)."""
        n = self.num_requests
        if block_tables.dim() != 2 or block_tables.size(0) != n:
            raise ValueError("block_tables must be [num_requests, max_pages]")
        i32, vector = torch.int32, self._vector
        _EXTEND.pack_into(
            self._args, 0, n, self.page_tokens, self.num_pages, block_tables.size(1),
            free_pages.numel(), self.max_tokens, position_base, vector(held, "held", i32, n),
            vector(added, "added", i32, n), vector(free_pages, "free_pages", i32),
            vector(self.taken if taken is None else taken, "taken", i32, 1),
            self.taken.data_ptr(), vector(block_tables, "block_tables", i32),
            self.kv_lens.data_ptr(), self.q_starts.data_ptr(), self.slots.data_ptr(),
            self.positions.data_ptr(), self._status)
        self._launch(self._fn, stream, self._ref)


def rope_table(max_positions: int, rot_dim: int, device, theta: float = 10000.0,
               stream=None) -> torch.Tensor:
    """The [max_positions, rot_dim] table of PagedAppend: cosines, then sines."""
    call = _Call(device, None)
    out = torch.empty((max_positions, rot_dim), dtype=torch.float32, device=call.device)
    call._made(out)
    call._launch(library().cg_rope_table, stream, max_positions, rot_dim, theta, out.data_ptr())
    return out


class PagedAppend(_Call):
    """Norm, rotate and store new tokens (cg_append_qkv)."""

    def __init__(self, shape, num_q_heads: int, dtype: torch.dtype, device,
                 status: torch.Tensor | None = None):
        super().__init__(device, status, dtype)
        self.shape = shape if isinstance(shape, Shape) else Shape(*shape)
        self.num_q_heads = num_q_heads
        self._args = AppendArgs()
        self._refs = ctypes.byref(self.shape), ctypes.byref(self._args)
        self._fn = library().cg_append_qkv

    def _weight(self, w, name: str) -> int:
        if w is None:
            return 0
        if w.dtype not in self._dtypes:
            raise ValueError(f"{name} must be of the object's type")
        return self._vector(w, name, w.dtype, self.shape.head_dim)

    def append(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_out: torch.Tensor,
               pool: torch.Tensor, layer: int, positions: torch.Tensor | None,
               slots: torch.Tensor, rope: torch.Tensor | None, q_weight=None, k_weight=None,
               eps: float = 1e-6, interleaved: bool = False, stream=None) -> None:
        """q [N, Hq, D], k and v [N, H, D] (views of one packed tensor will do),
        q_out like q (or q itself); positions int32 [N] and slots int64 [N] as
        PagedTables makes them; rope: rope_table's, or None for no rotation;
        weights [D], or None for no norm."""
        s, hq, rows = self.shape, self.num_q_heads, self._rows
        n, h, d = q.size(0), s.num_kv_heads, s.head_dim
        pages, page_tokens = self._pool(pool, s)
        far = rot = table = where = 0
        if rope is not None:
            if rope.dim() != 2 or positions is None:
                raise ValueError("rope must be [max_positions, rot_dim], with positions")
            far, rot = rope.shape
            table = self._vector(rope, "rope", torch.float32)
            where = self._vector(positions, "positions", torch.int32, n)
        _APPEND.pack_into(
            self._args, 0, n, hq, layer, pages, page_tokens, far, rot, int(interleaved),
            self._code, eps, q.data_ptr(), k.data_ptr(), v.data_ptr(), rows(q, "q", n, hq, d),
            rows(k, "k", n, h, d), rows(v, "v", n, h, d), q_out.data_ptr(),
            rows(q_out, "q_out", n, hq, d), self._weight(q_weight, "q_weight"),
            self._weight(k_weight, "k_weight"), table, where,
            self._vector(slots, "slots", torch.int64, n), pool.data_ptr(), self._status)
        self._launch(self._fn, stream, *self._refs)


class PagedAttention(_Call):
    """Attention over the paged pool (cg_attention_paged, cg_attention_shared)
    for at most max_tokens query rows of max_requests requests; holds the
    workspace."""

    def __init__(self, shape, num_q_heads: int, dtype: torch.dtype, max_tokens: int,
                 max_requests: int, device, status: torch.Tensor | None = None):
        super().__init__(device, status, dtype)
        self.shape = shape if isinstance(shape, Shape) else Shape(*shape)
        self.num_q_heads = num_q_heads
        self.max_tokens, self.max_requests = max_tokens, max_requests
        self._args = AttentionArgs()
        self._refs = ctypes.byref(self.shape), ctypes.byref(self._args)
        self._fn, self._shared_fn = library().cg_attention_paged, library().cg_attention_shared
        self._scale = 1.0 / math.sqrt(self.shape.head_dim)
        self.workspace = self._replaced = None
        self._ran = False
        self._reserve(False)

    def _reserve(self, shared: bool) -> None:
        need = cg_attention_workspace_bytes(self.shape, self.num_q_heads, self.max_tokens,
                                            self.max_requests, shared)
        if self.workspace is None or self.workspace.numel() < need:
            here = _raw_stream(self._index)
            if here not in self._seen:
                self._meet(here)
            if self._ran:
                self._replaced = self.workspace  # a captured call goes on using it
            self.workspace = torch.empty(need, dtype=torch.uint8, device=self.device)
            self._buffers = (self.status,)
            self._made(self.workspace)
        self._has_shared = shared

    def reserve_shared(self) -> None:
        """Size the workspace for run_shared now (its first call does so
        otherwise), for a program that captures its first call, and before the
        first run(), whose workspace would be kept beside the new one."""
        if not self._has_shared:
            self._reserve(True)

    def _set(self, q, pool, layer, q_starts, kv_lens, block_tables, max_q, out, window, sinks,
             scale, lse):
        s, hq = self.shape, self.num_q_heads
        n, requests, d = q.size(0), kv_lens.numel(), s.head_dim
        if n > self.max_tokens or requests > self.max_requests:
            raise ValueError("more rows or requests than this object was made for")
        if block_tables.dim() != 2 or block_tables.size(0) != requests:
            raise ValueError("block_tables must be [num_requests, max_pages]")
        pages, page_tokens = self._pool(pool, s)
        i32, vector = torch.int32, self._vector
        _ATTENTION.pack_into(
            self._args, 0, requests, n, max_q, hq, layer, pages, page_tokens,
            block_tables.size(1), window, sinks, self._code,
            self._scale if scale is None else scale, q.data_ptr(), out.data_ptr(),
            self._rows(q, "q", n, hq, d), self._rows(out, "out", n, hq, d),
            0 if lse is None else vector(lse, "lse", torch.float32, n * hq),
            vector(q_starts, "q_starts", i32, requests + 1), vector(kv_lens, "kv_lens", i32),
            vector(block_tables, "block_tables", i32), pool.data_ptr(), self._status,
            self.workspace.data_ptr(), self.workspace.numel())
        return page_tokens

    def run(self, q: torch.Tensor, pool: torch.Tensor, layer: int, q_starts: torch.Tensor,
            kv_lens: torch.Tensor, block_tables: torch.Tensor, max_q: int, out: torch.Tensor,
            window: int = 0, sinks: int = 0, scale: float | None = None,
            lse: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """q and out: [N, Hq, D]; q_starts int32 [B + 1], kv_lens int32 [B] and
        block_tables int32 [B, max_pages] as PagedTables makes them; max_q: no
        request has more new tokens; window 0: no window; scale: 1 / sqrt(D)
        by default; lse: fp32 [N, Hq] that receives the log-sums."""
        self._set(q, pool, layer, q_starts, kv_lens, block_tables, max_q, out, window, sinks,
                  scale, lse)
        self._ran = True
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
        page_tokens = self._set(q, pool, layer, q_starts, kv_lens, block_tables, max_q, out, 0, 0,
                                scale, lse)
        table = self._vector(prefix_table, "prefix_table", torch.int32,
                             -(-prefix_tokens // page_tokens))
        self._launch(self._shared_fn, stream, *self._refs, table, prefix_tokens)
        return out
