"""Serving from decoded pages: block tables, row writes and tree attention over
a paged KV cache (skv_page_map, skv_cache_append, skv_tree_attention).

As in api.py, PyTorch only provides device memory and streams. The `_into`
calls enqueue on the current (or given) stream and return without
synchronising; check_status() waits and raises what the device reported. The
calls of one object share its status word and workspace, so they must not run
at once on different streams. A call that makes its result itself (step, attend)
comes after what the current stream has been given, and the result is the
current stream's.
"""
from __future__ import annotations

import ctypes as C
import math

import torch

from . import _binding as B
from .api import _after_current, _check_dev, _ptr


def _stream_of(stream, device: int) -> int:
    """The handle of `stream`, or of the current stream of the tensors' device (the
    raw query: a Stream object costs several microseconds of a short step). Kernels are
    launched on the current device, so that has to be the tensors'."""
    if torch._C._cuda_getDevice() != device or (stream is not None and stream.device_index != device):
        raise ValueError(f"the pools are on cuda:{device}: make it the current device and give a stream of it")
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(device)


_BF16, _I32, _I64, _F32 = torch.bfloat16, torch.int32, torch.int64, torch.float32
# what a pool may be kept as: the format's own type, or its bits
_CODES = {torch.bfloat16: B.SKV_BF16, torch.int16: B.SKV_BF16, torch.uint16: B.SKV_BF16,
          torch.float8_e4m3fn: B.SKV_E4M3, torch.uint8: B.SKV_E4M3, torch.int8: B.SKV_E4M3}


def _check_words(what: str, dtype, numel: int, device: int, *ts):
    """Contiguous tensors of one type and size on that device (a step makes a dozen of these
    checks, each of a few tenths of a microsecond: no calls that are not needed)."""
    for t in ts:
        if t.dtype is not dtype or t.numel() != numel or t.get_device() != device or not t.is_contiguous():
            raise ValueError(f"{what} must be contiguous {dtype} tensors of {numel} entries on cuda:{device}")


def _table_rows(t):
    if not t.is_cuda or t.dtype != torch.int32 or t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1) \
            or (t.shape[0] > 1 and t.stride(0) < t.shape[1]):
        raise ValueError("block_table must be an int32 CUDA tensor [n_requests][max_pages] with whole rows")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _capturing(stream) -> bool:
    """Whether `stream` (None: the current one) or the current stream is being captured."""
    if torch.cuda.is_current_stream_capturing():
        return True
    with torch.cuda.stream(stream):
        return torch.cuda.is_current_stream_capturing()


class _Status:
    def _new_status(self, device):
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self._status, self._device = self.status.data_ptr(), self.status.device.index

    def _settle(self):
        """End of a constructor: what it filled is filled, whatever stream calls first (in a capture
        the fills are part of the graph)."""
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream(self._device).synchronize()

    def check_status(self, where: str, stream=None):
        (stream or torch.cuda.current_stream()).synchronize()
        st = int(self.status.item())
        if st:
            raise B.SKVError(where, st)


class PageTable(_Status):
    """A block table [n_requests][max_pages] (int32) over a pool of `pool_pages`
    pages of `page_tokens` tokens, kept on the GPU (skv_page_map). workspace=True makes the
    workspace of fork and compact (a first call makes it otherwise, which a capture cannot)."""

    _ended = False      # whether the last call was a step in two parts (PagePool)

    def __init__(self, block_table: torch.Tensor, page_tokens: int, pool_pages: int, workspace: bool = False):
        self._stride = _table_rows(block_table)
        self.block_table, self._table = block_table, block_table.data_ptr()
        self.page_tokens, self.pool_pages = int(page_tokens), int(pool_pages)
        self._shape = block_table.shape
        self.n_requests, self.max_pages = self._shape
        self._new_status(block_table.device)
        self.workspace = None
        if workspace:
            self._make_workspace()
        self._settle()

    def _make_workspace(self, stream=None):
        """The workspace, which any content suits; it stays as long as the object: a captured graph holds
        its address."""
        v = C.c_uint64()
        B.check("skv_page_workspace_bytes", B.lib().skv_page_workspace_bytes(self.n_requests, self.pool_pages, C.byref(v)))
        self.workspace = torch.empty(v.value, dtype=torch.uint8, device=self.block_table.device)
        _after_current(stream)
        self._workspace, self._workspace_bytes = self.workspace.data_ptr(), v.value

    def _ready(self, table_out, stream):
        """What fork and compact need beside their arrays; table_out's row stride."""
        rows, cols = self._shape
        if table_out.dtype is not _I32 or table_out.shape != self._shape or table_out.get_device() != self._device:
            raise ValueError("table_out must be an int32 tensor of the block_table's shape and device")
        down, across = table_out.stride()
        if (cols > 1 and across != 1) or (rows > 1 and down < cols) or table_out.data_ptr() == self._table:
            raise ValueError("table_out must have whole rows and be another tensor than the block_table")
        if self.workspace is None:
            if _capturing(stream):
                raise ValueError("give PageTable workspace=True before a capture")
            self._make_workspace(stream)
        return down if rows > 1 else cols

    def map_into(self, ctx_len, new_len, n_pages, free_pages, free_state, cu_new, slots, n_pages_out,
                 free_state_out, stream=None):
        """Enqueue skv_page_map: pages for each request's new tokens off the ring
        (free_pages, free_state = [head, count]), their table entries, cu_new and the
        slot map; a request of ctx_len < 0 gives its pages back. The new page counts and
        ring state go to n_pages_out and free_state_out (other tensors than the inputs)."""
        n, size, room, dev = self.n_requests, free_pages.numel(), slots.numel(), self._device
        _check_words("ctx_len, new_len, n_pages and n_pages_out", _I32, n, dev, ctx_len, new_len, n_pages, n_pages_out)
        _check_words("free_state and free_state_out", _I32, 2, dev, free_state, free_state_out)
        _check_words("cu_new", _I32, n + 1, dev, cu_new)
        _check_words("free_pages", _I32, size, dev, free_pages)
        _check_words("slots", _I64, room, dev, slots)
        rc = B.lib().skv_page_map(self.page_tokens, self.pool_pages, n, ctx_len.data_ptr(), new_len.data_ptr(),
                                  self._table, self._stride, self.max_pages, n_pages.data_ptr(), n_pages_out.data_ptr(),
                                  free_pages.data_ptr(), size, free_state.data_ptr(), free_state_out.data_ptr(),
                                  cu_new.data_ptr(), slots.data_ptr(), room, self._status, _stream_of(stream, self._device))
        B.check("skv_page_map", rc)
        self._ended = False

    def fork_into(self, parents, ctx_len, n_pages, free_pages, free_state, table_out, n_pages_out, ctx_out, free_state_out,
                  copy_src, copy_dst, copy_tokens, trim: bool = False, stream=None):
        """Enqueue skv_page_fork: row s of table_out goes on from row parents[s] (None: from
        itself; -1, or a row of ctx_len < 0: empty), sharing its full pages; pages that no row holds any
        more go back to the ring. copy_src, copy_dst and copy_tokens are for PagedKV.copy_into, once for
        each layer's pools. Outputs are other tensors than the inputs."""
        n, size, dev = self.n_requests, free_pages.numel(), self._device
        _check_words("ctx_len, n_pages, n_pages_out, ctx_out and the copies", _I32, n, dev, ctx_len, n_pages, n_pages_out, ctx_out,
                     copy_src, copy_dst, copy_tokens)
        _check_words("free_state and free_state_out", _I32, 2, dev, free_state, free_state_out)
        _check_words("free_pages", _I32, size, dev, free_pages)
        if parents is not None:
            _check_words("parents", _I32, n, dev, parents)
            parents = parents.data_ptr()
        out = self._ready(table_out, stream)
        rc = B.lib().skv_page_fork(self.page_tokens, self.pool_pages, n, parents, ctx_len.data_ptr(), self._table, self._stride,
                                   self.max_pages, n_pages.data_ptr(), trim, table_out.data_ptr(), out, n_pages_out.data_ptr(),
                                   ctx_out.data_ptr(), free_pages.data_ptr(), size, free_state.data_ptr(), free_state_out.data_ptr(),
                                   copy_src.data_ptr(), copy_dst.data_ptr(), copy_tokens.data_ptr(), self._status, self._workspace,
                                   self._workspace_bytes, _stream_of(stream, dev))
        B.check("skv_page_fork", rc)
        self._ended = False

    def compact_into(self, n_pages, free_pages, free_state, table_out, free_state_out, copy_src, copy_dst, stream=None):
        """Enqueue skv_page_compact: the held pages move to the front of the pool; table_out has their new
        numbers and the ring the pages behind them. copy_src and copy_dst (room for the moves: as many as
        pages are held is always enough) are for PagedKV.copy_into, once for each layer's pools."""
        size, room, dev = free_pages.numel(), copy_src.numel(), self._device
        _check_words("n_pages", _I32, self.n_requests, dev, n_pages)
        _check_words("free_state and free_state_out", _I32, 2, dev, free_state, free_state_out)
        _check_words("free_pages", _I32, size, dev, free_pages)
        _check_words("copy_src and copy_dst", _I32, room, dev, copy_src, copy_dst)
        out = self._ready(table_out, stream)
        rc = B.lib().skv_page_compact(self.pool_pages, self.n_requests, self._table, self._stride, self.max_pages, n_pages.data_ptr(),
                                      table_out.data_ptr(), out, free_pages.data_ptr(), size, free_state.data_ptr(),
                                      free_state_out.data_ptr(), copy_src.data_ptr(), copy_dst.data_ptr(), room, self._status,
                                      self._workspace, self._workspace_bytes, _stream_of(stream, dev))
        B.check("skv_page_compact", rc)
        self._ended = False


class PagePool(PageTable):
    """A PageTable with its page counts and its ring of free pages: all pages free
    at first, counts swapped by every step. Rows that share pages (fork) give them back when the last of
    them has ended. A row's ctx_len may go back to any page's border (to 0: its request has ended and
    another one takes the row), but not into the middle of a page that it shares: its new tokens would be
    written over the other rows'. Of a pool that shares pages a step keeps no more of a row's pages
    than its ctx_len tokens need, and takes a second launch; every 16th one that is checked looks whether pages are shared
    still."""

    def __init__(self, n_requests: int, max_pages: int, page_tokens: int, pool_pages: int, device="cuda"):
        super().__init__(torch.full((n_requests, max_pages), -1, dtype=torch.int32, device=device), page_tokens,
                         pool_pages)
        self.n_pages = torch.zeros(n_requests, dtype=torch.int32, device=device)
        self.free_pages = torch.arange(pool_pages, dtype=torch.int32, device=device)
        self.free_state = torch.tensor([0, pool_pages], dtype=torch.int32, device=device)
        self._next = (torch.empty_like(self.n_pages), torch.empty_like(self.free_state))
        self._shared, self._steps, self._mid = False, 0, None
        self._ends = PageTable(self.block_table, page_tokens, pool_pages)      # what ends rows in a step, with a status of its own
        self._settle()

    def step(self, ctx_len, new_len, max_new: int, check: bool = True, stream=None):
        """Map one step's new tokens (max_new: room for so many slots). Returns
        (cu_new, slots), slots past the step's tokens -1. Not for a capture, whose replays would
        all start from the same counts: capture map_into, and copy its counts back behind it. A step
        that is refused leaves everything as it was; with check=False, where rows share pages, rows that ended
        have given theirs back all the same."""
        dev = self.block_table.device
        if _capturing(stream):
            raise ValueError("PagePool.step swaps its counts on the host; capture map_into")
        cu = torch.empty(self.n_requests + 1, dtype=torch.int32, device=dev)
        slots = torch.empty(max_new, dtype=torch.int64, device=dev)
        counts = (self.n_pages, self.free_state)
        if self._shared:
            counts = self._end(ctx_len, stream)
        _after_current(stream)
        self.map_into(ctx_len, new_len, counts[0], self.free_pages, counts[1], cu, slots, *self._next, stream=stream)
        self._ended = self._shared
        before, (self.n_pages, self.free_state) = (self.n_pages, self.free_state), self._next
        self._next = before
        if check:
            try:
                self.check_status("skv_page_map", stream)
            except B.SKVError as e:
                if e.name != "CORRUPT":                  # nothing was mapped, and nothing has ended
                    self._next, (self.n_pages, self.free_state) = (self.n_pages, self.free_state), before
                raise
            if self._shared:
                self._steps += 1
                if self._steps % 16 == 0:
                    self._shared = self._sharing(stream)
        elif stream is not None:                         # given up early, they are not handed out early
            cu.record_stream(stream)
            slots.record_stream(stream)
        return cu, slots

    def _end(self, ctx_len, stream):
        """The page counts and the ring state of a step's rows without those that have ended, for its map. A page of
        an ended request may be another one's: the map would give it back all the same. And a row that goes
        back, or starts again, would get its new tokens on pages that it shares: trimmed, it gives those
        up. (Every row is its own heir: entries of the table stay where they are, and of the ring those behind
        its end are written.)"""
        if self._mid is None:
            words = torch.empty((5, self.n_requests), dtype=torch.int32, device=self.block_table.device)
            self._mid = (torch.empty_like(self.block_table), *words.unbind(), torch.empty_like(self.free_state))
        _after_current(stream)
        table, n_pages, ctx_out, src, dst, tokens, state = self._mid
        self._ends.fork_into(None, ctx_len, self.n_pages, self.free_pages, self.free_state, table, n_pages, ctx_out, state, src, dst, tokens,
                             trim=True, stream=stream)
        return n_pages, state

    def _sharing(self, stream):
        """Whether rows share a page: they have more entries than there are different pages in them (a compaction whose
        results are dropped counts those)."""
        with torch.cuda.stream(stream):
            ring, src, dst = torch.empty((3, self.pool_pages), dtype=torch.int32, device=self.block_table.device).unbind()
            state = torch.empty_like(self.free_state)
            self._ends.compact_into(self.n_pages, ring, self.free_state, self._mid[0], state, src, dst)
            return int(self.n_pages.sum() + state[1]) != self.pool_pages

    def check_status(self, where: str, stream=None):
        super().check_status(where, stream)
        if self._ended:                                  # the last call was a step in two parts
            self._ends.check_status("skv_page_fork", stream)

    def fork(self, parents, ctx_len, trim: bool = False, check: bool = True, stream=None):
        """Row s goes on from row parents[s] (None: from itself; -1 or ctx_len < 0: it ends) and shares its
        full pages. Returns (ctx_len of the new rows, copy_src, copy_dst, copy_tokens): give the
        last three to copy of every layer's PagedKV before the rows are used. The block_table is
        rewritten in place. Not for a capture: capture fork_into."""
        if _capturing(stream):
            raise ValueError("PagePool.fork swaps its counts on the host; capture fork_into")
        ctx, src, dst, tokens = torch.empty((4, self.n_requests), dtype=torch.int32, device=self.block_table.device).unbind()
        table = self._other_table(stream)
        self.fork_into(parents, ctx_len, self.n_pages, self.free_pages, self.free_state, table, self._next[0], ctx, self._next[1], src, dst,
                       tokens, trim=trim, stream=stream)
        self._take(table, self._next[0], stream)
        if parents is not None:
            self._shared, self._steps = True, 0
        if check:
            self.check_status("skv_page_fork", stream)
        elif stream is not None:                         # given up early, they are not handed out early
            for t in (ctx, src, dst, tokens):
                t.record_stream(stream)
        return ctx, src, dst, tokens

    def compact(self, check: bool = True, stream=None):
        """The held pages move to the front of the pool. Returns (copy_src, copy_dst): give them to
        copy of every layer's PagedKV before the pages are used. Not for a capture."""
        if _capturing(stream):
            raise ValueError("PagePool.compact swaps its counts on the host; capture compact_into")
        src, dst = torch.empty((2, self.pool_pages), dtype=torch.int32, device=self.block_table.device).unbind()
        table = self._other_table(stream)
        self.compact_into(self.n_pages, self.free_pages, self.free_state, table, self._next[1], src, dst, stream=stream)
        self._take(table, self.n_pages, stream)
        if check:
            self.check_status("skv_page_compact", stream)
        elif stream is not None:
            for t in (src, dst):
                t.record_stream(stream)
        return src, dst

    def _other_table(self, stream):
        """A second table for a call on `stream`, in that stream's memory and order: earlier calls on it
        may still be writing the first."""
        if self.workspace is None:
            self._make_workspace(stream)
        _after_current(stream)
        with torch.cuda.stream(stream):
            return self.block_table.clone()

    def _take(self, table, n_pages, stream):
        """The rows of `table`, n_pages (self.n_pages, or what the call left in _next) and the ring state
        that the call left become the pool's."""
        with torch.cuda.stream(stream):
            self.block_table.copy_(table)
        spare = self._next[0] if n_pages is self.n_pages else self.n_pages
        now = (spare, self.free_state)
        self.n_pages, self.free_state = n_pages, self._next[1]
        self._next = now


class PagedKV(_Status):
    """K and V pools [n_pages][page_tokens][n_heads][head_dim] of codes (bf16, or int16 and
    uint16 of its bits; float8_e4m3fn, or uint8 and int8), of any strides that are multiples of
    16 bytes and the same for both (pages as decode_chunks returns them, viewed in four
    dimensions, are such pools).

    block_table: int32 [n_requests][max_pages], needed by attend; k_scale, v_scale:
    float32 [n_heads] of an e4m3 cache. q_heads > 0 makes the workspace of attend, for any
    number of query heads (a first call makes it otherwise, which a capture cannot)."""

    def __init__(self, k_pages: torch.Tensor, v_pages: torch.Tensor, block_table: torch.Tensor | None = None,
                 k_scale: torch.Tensor | None = None, v_scale: torch.Tensor | None = None, q_heads: int = 0):
        for t, what in ((k_pages, "k_pages"), (v_pages, "v_pages")):
            if not t.is_cuda or t.dim() != 4 or t.dtype not in _CODES or (t.shape[3] > 1 and t.stride(3) != 1):
                raise ValueError(f"{what} must be a CUDA tensor [n_pages][page_tokens][n_heads][head_dim] of codes "
                                 "(bfloat16, int16 or uint16; float8_e4m3fn, uint8 or int8)")
        if k_pages.shape != v_pages.shape or k_pages.stride() != v_pages.stride() \
                or _CODES[k_pages.dtype] != _CODES[v_pages.dtype] or k_pages.device != v_pages.device:
            raise ValueError("k_pages and v_pages must have the same shape, strides, format and device")
        n_pages, page_tokens, n_heads, head_dim = k_pages.shape
        for s in (k_scale, v_scale):
            if s is not None:
                _check_dev(s, "k_scale and v_scale", torch.float32, numel=n_heads)
        for t in (k_scale, v_scale, block_table):
            if t is not None and t.device != k_pages.device:
                raise ValueError("the scales and the block_table must be on the pools' device")
        self.k_pages, self.v_pages, self.k_scale, self.v_scale = k_pages, v_pages, k_scale, v_scale
        self.block_table, self.n_heads, self.head_dim = block_table, n_heads, head_dim
        self._row_shape, self._scale = torch.Size((n_heads, head_dim)), 1.0 / math.sqrt(head_dim)
        stride, n_requests, max_pages = 0, 0, 0
        if block_table is not None:
            stride = _table_rows(block_table)
            n_requests, max_pages = block_table.shape
        self.n_requests = n_requests
        ps, ts, hs = k_pages.stride()[:3]
        self._c = B.skv_paged(B.SKV_FORMAT_VERSION, _CODES[k_pages.dtype], n_heads, head_dim, page_tokens, n_pages, k_pages.data_ptr(), v_pages.data_ptr(),
                              ps if n_pages > 1 else 0, ts if page_tokens > 1 else 0, hs if n_heads > 1 else 0,
                              _ptr(k_scale), _ptr(v_scale), _ptr(block_table), stride, n_requests, max_pages)
        self._ref = C.byref(self._c)
        B.check("skv_paged_check", B.lib().skv_paged_check(self._ref))
        self._new_status(k_pages.device)
        self.q_heads, self.workspace = q_heads, None
        if q_heads:
            self._make_workspace(q_heads)
        self._settle()

    def _make_workspace(self, q_heads: int, stream=None):
        """The workspace, its counters 0 before what `stream` (None: the current one) does next. Its
        size is the same for every number of query heads, and it stays as long as the object: a
        captured graph holds its address."""
        v = C.c_uint64()
        B.check("skv_tree_attention_workspace_bytes",
                B.lib().skv_tree_attention_workspace_bytes(self._ref, q_heads, C.byref(v)))
        self.workspace = torch.empty(v.value, dtype=torch.uint8, device=self.k_pages.device)
        self.workspace[:B.SKV_ATTENTION_ZERO_BYTES].zero_()
        _after_current(stream)
        self._workspace, self._workspace_bytes = self.workspace.data_ptr(), v.value

    def append_into(self, k, v, slots, rows=None, stream=None):
        """Enqueue skv_cache_append: rows of k and v (bf16 [n_src][n_heads][head_dim], any
        row and head strides that are multiples of 8) into the slots (int64, -1 skips)."""
        shape, stride, dev = k.shape, k.stride(), self._device
        if v.shape != shape or v.stride() != stride or k.dtype is not _BF16 or v.dtype is not _BF16 or k.get_device() != dev \
                or v.get_device() != dev or len(shape) != 3 or shape[1:] != self._row_shape or stride[2] != 1:
            raise ValueError("k and v must be bf16 tensors [n_src][%d][%d] on the pools' device, of the same strides, the last 1"
                             % tuple(self._row_shape))
        n = slots.numel()
        _check_words("slots", _I64, n, dev, slots)
        if rows is not None:
            _check_words("rows", _I32, n, dev, rows)
            rows = rows.data_ptr()
        rc = B.lib().skv_cache_append(self._ref, k.data_ptr(), v.data_ptr(), stride[0], stride[1], shape[0], rows,
                                      slots.data_ptr(), n, self._status, _stream_of(stream, self._device))
        B.check("skv_cache_append", rc)

    def append(self, k, v, slots, rows=None, stream=None):
        """append_into, waited for and checked."""
        self.append_into(k, v, slots, rows, stream)
        self.check_status("skv_cache_append", stream)

    def rotate_append_into(self, rotary, q, k, v, positions, slots, q_out, stream=None):
        """Enqueue skv_rotate_append: the heads of q and k normalised and rotated (`rotary`, a Rotary),
        q into q_out (contiguous, of q's shape; None with q None: no queries), k and v into the slots as
        append_into writes them. positions: int32 [n], or [n_axes][n] (None where nothing is rotated); -1 in
        slots: queries only."""
        shape, stride, dev = k.shape, k.stride(), self._device
        if v.shape != shape or v.stride() != stride or k.dtype is not _BF16 or v.dtype is not _BF16 or k.get_device() != dev \
                or v.get_device() != dev or len(shape) != 3 or shape[1:] != self._row_shape or stride[2] != 1:
            raise ValueError("k and v must be bf16 tensors [n][%d][%d] on the pools' device, of the same strides, the last 1"
                             % tuple(self._row_shape))
        n = shape[0]
        if rotary._device != dev or rotary.head_dim != self.head_dim:
            raise ValueError("the Rotary must be on the pools' device and of their head_dim")
        q_ptr = out_ptr = None
        heads = q_row = q_head = 0
        if q is not None:
            q_shape, q_stride = q.shape, q.stride()
            if len(q_shape) != 3 or q.dtype is not _BF16 or q.get_device() != dev or q_shape[0] != n or q_shape[2] != self.head_dim \
                    or q_stride[2] != 1:
                raise ValueError(f"q must be a bf16 tensor [{n}][q_heads][{self.head_dim}] on cuda:{dev}")
            if q_out is None or q_out.shape != q_shape or q_out.dtype is not _BF16 or q_out.get_device() != dev or not q_out.is_contiguous():
                raise ValueError("q_out must be a contiguous bf16 tensor of q's shape and device")
            q_ptr, out_ptr, heads, q_row, q_head = q.data_ptr(), q_out.data_ptr(), q_shape[1], q_stride[0], q_stride[1]
        elif q_out is not None:
            raise ValueError("q_out without q")
        at = None
        if positions is not None:
            if rotary.n_axes > 1 and positions.shape != (rotary.n_axes, n):
                raise ValueError(f"positions must be an int32 tensor [{rotary.n_axes}][{n}]")
            _check_words("positions", _I32, rotary.n_axes * n, dev, positions)
            at = positions.data_ptr()
        elif rotary.rot_dim:
            raise ValueError(f"the Rotary turns {rotary.rot_dim} channels: positions are needed")
        _check_words("slots", _I64, n, dev, slots)
        rc = B.lib().skv_rotate_append(self._ref, rotary._ref, q_ptr, q_row, q_head, heads, k.data_ptr(), v.data_ptr(), stride[0], stride[1],
                                       at, slots.data_ptr(), n, out_ptr, self._status, _stream_of(stream, dev))
        B.check("skv_rotate_append", rc)

    def rotate_append(self, rotary, q, k, v, positions, slots, stream=None):
        """rotate_append_into a new tensor, waited for and checked; returns the queries."""
        out = None if q is None else torch.empty(q.shape, dtype=_BF16, device=q.device)
        _after_current(stream)
        self.rotate_append_into(rotary, q, k, v, positions, slots, out, stream)
        self.check_status("skv_rotate_append", stream)
        return out

    def move_into(self, cu_new, rows, slots, kept, stream=None):
        """Enqueue skv_cache_move: the accepted tokens' K and V to the places that `kept` names (rows and
        kept as Verifier.verify_into leaves them, slots those of the new tokens)."""
        n, dev = rows.numel(), self._device
        _check_words("rows", _I32, n, dev, rows)
        _check_words("slots and kept", _I64, n, dev, slots, kept)
        requests = cu_new.numel() - 1
        if requests < 0:
            raise ValueError("cu_new needs an entry")
        _check_words("cu_new", _I32, requests + 1, dev, cu_new)
        rc = B.lib().skv_cache_move(self._ref, requests, cu_new.data_ptr(), n, rows.data_ptr(), slots.data_ptr(), kept.data_ptr(),
                                    self._status, _stream_of(stream, dev))
        B.check("skv_cache_move", rc)

    def move(self, cu_new, rows, slots, kept, stream=None):
        """move_into, waited for and checked."""
        self.move_into(cu_new, rows, slots, kept, stream)
        self.check_status("skv_cache_move", stream)

    def copy_into(self, src, dst, tokens=None, stream=None):
        """Enqueue skv_cache_copy: K and V pages src (int32, -1 skips) to pages dst, the first tokens[i]
        tokens of each (None: whole pages)."""
        n, dev = src.numel(), self._device
        _check_words("src and dst", _I32, n, dev, src, dst)
        if tokens is not None:
            _check_words("tokens", _I32, n, dev, tokens)
            tokens = tokens.data_ptr()
        rc = B.lib().skv_cache_copy(self._ref, src.data_ptr(), dst.data_ptr(), tokens, n, self._status, _stream_of(stream, dev))
        B.check("skv_cache_copy", rc)

    def copy(self, src, dst, tokens=None, stream=None):
        """copy_into, waited for and checked."""
        self.copy_into(src, dst, tokens, stream)
        self.check_status("skv_cache_copy", stream)

    def attend_into(self, q, ctx_len, cu_new, out, mask=None, max_nodes: int | None = None,
                    scale: float | None = None, lse=None, stream=None):
        """Enqueue skv_tree_attention. q: bf16 [n_rows][q_heads][head_dim] (row and head
        strides multiples of 8); out: the same shape, contiguous; mask: int64 [n_rows][words]
        of visibility bits among a request's new tokens, None: each sees the ones before it;
        max_nodes: about the most new tokens of a request (default: the mean over the requests,
        rounded up, so that a batch of single tokens is taken for one); scale defaults
        to 1 / sqrt(head_dim); lse: float32 [n_rows][q_heads] or None."""
        if self.block_table is None:
            raise ValueError("attend needs a block_table")
        shape, stride, dev = q.shape, q.stride(), self._device
        if len(shape) != 3 or q.dtype is not _BF16 or q.get_device() != dev or stride[2] != 1 or shape[2] != self.head_dim \
                or shape[1] == 0 or shape[1] % self.n_heads:
            raise ValueError(f"q must be a bf16 tensor [n_rows][a multiple of {self.n_heads}][{self.head_dim}] on cuda:{dev}")
        n, heads = shape[0], shape[1]
        if out.shape != shape or out.dtype is not _BF16 or out.get_device() != dev or not out.is_contiguous():
            raise ValueError("out must be a contiguous bf16 tensor of q's shape and device")
        _check_words("ctx_len", _I32, self.n_requests, dev, ctx_len)
        _check_words("cu_new", _I32, self.n_requests + 1, dev, cu_new)
        words = 0
        if mask is not None:
            if mask.dim() != 2 or mask.shape[0] != n or mask.shape[1] == 0:
                raise ValueError("mask must be an int64 CUDA tensor [n_rows][words]")
            words = mask.shape[1]
            _check_words("mask", _I64, n * words, dev, mask)
            mask = mask.data_ptr()
        if lse is not None:
            _check_words("lse", _F32, n * heads, dev, lse)
            lse = lse.data_ptr()
        if self.workspace is None:
            if _capturing(stream):
                raise ValueError("give PagedKV its q_heads before a capture")
            self._make_workspace(heads, stream)
        rc = B.lib().skv_tree_attention(
            self._ref, q.data_ptr(), stride[0], stride[1], heads, n, ctx_len.data_ptr(), cu_new.data_ptr(), mask, words,
            -(-n // max(self.n_requests, 1)) if max_nodes is None else max_nodes, self._scale if scale is None else scale, out.data_ptr(), lse,
            self._status, self._workspace, self._workspace_bytes, _stream_of(stream, self._device))
        B.check("skv_tree_attention", rc)

    def attend(self, q, ctx_len, cu_new, mask=None, max_nodes: int | None = None, scale: float | None = None,
               stream=None):
        """attend_into a new tensor (rows outside every request 0), waited for and checked."""
        out = torch.zeros(q.shape, dtype=torch.bfloat16, device=q.device)
        _after_current(stream)
        self.attend_into(q, ctx_len, cu_new, out, mask, max_nodes, scale, stream=stream)
        self.check_status("skv_tree_attention", stream)
        return out
