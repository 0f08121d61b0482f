"""A paged K / V cache for several video streams at once.

Long-video survey (atlascloud.ai), section "Route 3 · Self Forcing": video is
generated chunk after chunk, each chunk attending to the earlier ones through
a KV cache that may be capped at a number of frames.  ``PagedCache`` keeps
what the streams of a server share -- block tables, lengths, the ring of free
pages -- on the device and runs the three calls of a step on it::

    cache.plan(new_lens)                      # once a step
    for layer in layers:                      # and denoising pass
        cache.write(q, k, v, wq, wk, table, k_pages[layer], v_pages[layer])
        cache.attn(q, k_pages[layer], v_pages[layer], o)

The page pools belong to the caller, one pair per layer (``new_pools``); all
layers share the tables.  The layouts and rules are those of include/wan.h.
No call synchronises; everything a step needs is on the device, so a step can
be captured into a CUDA graph (after a first one outside the capture) and
replayed after new_lens was overwritten.
"""

import math

import torch

from . import wan


_SCALE = 1.0 / math.sqrt(128)
_BF16 = torch.bfloat16


def _pad4(n):
    """int32 counts padded to whole 16-byte pieces."""
    return -(-int(n) // 4) * 4


class PagedCache:
    """State and plan of a paged cache on one device.

    streams: int32 CUDA tensor [R, 4] of (H, W, chunk_tokens, window_tokens)
    per stream (it may be rewritten between steps when a stream is reused).
    grid: the grid of the RoPE table, which every position must lie in.
    max_pages: block table entries a stream can use, evicted ones included.
    token_cap: packed rows of q, k, v and o.  max_new: most new tokens of
    one stream in a step (default token_cap); together with heads / kv_heads
    it picks the attention kernel (max_new may be set anew before a plan).

    The cache's tensors are allocated and filled on the stream that is
    current here; calls on another one are ordered behind it by the caller,
    as for any tensor.

    state holds everything that a plan carries from step to step in one
    int32 tensor, with the views kv_lens, first_pages, block_table, free_ring
    and ring_state: saving and restoring it takes a step back (pages must
    not have been written in between).  q_start, q_lens, status and tokens
    are the plan's results.
    """

    def __init__(self, streams, grid, *, n_pages, page_size, max_pages,
                 heads, kv_heads=None, token_cap, max_new=None):
        kv_heads = heads if kv_heads is None else kv_heads
        if streams.dtype != torch.int32 or streams.dim() != 2 \
                or streams.shape[1] != 4 or not streams.is_contiguous():
            raise ValueError("streams must be a contiguous int32 [R, 4] "
                             "tensor")
        R = streams.shape[0]
        sizes = dict(n_pages=n_pages, page_size=page_size,
                     max_pages=max_pages, heads=heads, kv_heads=kv_heads,
                     token_cap=token_cap)
        for name, v in sizes.items():
            if int(v) < 1:
                raise ValueError("%s must be at least 1" % name)
        if page_size not in (16, 32, 64, 128):
            raise ValueError("page_size must be 16, 32, 64 or 128")
        if heads % kv_heads:
            raise ValueError("heads (%d) must divide by kv_heads (%d)"
                             % (heads, kv_heads))
        if not 1 <= R <= 1024:
            raise ValueError("1 to 1024 streams, not %d" % R)
        max_new = token_cap if max_new is None else max_new
        if max_new < 1:
            raise ValueError("max_new must be at least 1")
        wan._on_cuda(("streams", streams))
        dev = streams.device
        self.streams, self.grid, self.device = streams, grid, dev
        self.n_streams, self.n_pages = R, int(n_pages)
        self.page_size, self.max_pages = int(page_size), int(max_pages)
        self.heads, self.kv_heads = int(heads), int(kv_heads)
        self.token_cap, self.max_new = int(token_cap), int(max_new)

        def parts(buf, counts):
            out, at = [], 0
            for n in counts:
                out.append(buf[at:at + n])
                at += _pad4(n)
            return out

        counts = (R, R, R * self.max_pages, self.n_pages, 2)
        self.state = torch.zeros(sum(map(_pad4, counts)), dtype=torch.int32,
                                 device=dev)
        (self.kv_lens, self.first_pages, table, self.free_ring,
         self.ring_state) = parts(self.state, counts)
        self.block_table = table.view(R, self.max_pages)
        n_work = wan.paged_work_bytes(R) // 4
        counts = (R + 1, R, R, 4 * self.token_cap, n_work)
        buf = torch.zeros(sum(map(_pad4, counts)), dtype=torch.int32,
                          device=dev)
        (self.q_start, self.q_lens, self.status, tokens,
         self._work) = parts(buf, counts)
        self.tokens = tokens.view(self.token_cap, 4)
        self.tokens.fill_(-1)
        self._index = streams.get_device()
        self._table_bytes = wan.rope3d_table_bytes(grid)
        if self._table_bytes == 0:
            raise ValueError("grid %r has no RoPE table" % (grid,))
        self._desc = None
        self._need_for = self._planned = None
        self._q_shape = torch.Size((self.token_cap, self.heads, 128))
        self._kv_shape = torch.Size((self.token_cap, self.kv_heads, 128))
        self._pool_shape = torch.Size((self.n_pages, self.kv_heads,
                                       self.page_size, 128))
        self.reset()
        # Scratch of both sizes that a max_new can need, now: allocated inside
        # a call it would belong to the current stream while the call may run
        # on another, or to the graph that is being captured.
        self._workspaces = {}
        d = self.descriptor()
        for d.max_new in (1, 2 ** 31 - 1):
            need = wan.paged_workspace_bytes(d, dev)
            if need not in self._workspaces:
                self._workspaces[need] = torch.empty(need, dtype=torch.uint8,
                                                     device=dev)

    def reset(self):
        """All streams empty, all pages free."""
        self.state.zero_()
        self.block_table.fill_(-1)
        self.free_ring.copy_(torch.arange(self.n_pages, dtype=torch.int32,
                                          device=self.device))
        self.ring_state[1].fill_(self.n_pages)

    def new_pools(self, layers=None):
        """Zeroed K and V pools of one layer, or [layers, ...] of several."""
        shape = tuple(self._pool_shape)
        if layers is not None:
            shape = (int(layers),) + shape
        return (torch.zeros(shape, dtype=torch.bfloat16, device=self.device),
                torch.zeros(shape, dtype=torch.bfloat16, device=self.device))

    def descriptor(self):
        """The wan_paged_t of the cache (its arrays stay where they are for
        the cache's life, so it is built once)."""
        d = self._desc
        if d is None:
            d = self._desc = wan.PagedDesc(
                self.n_streams, self.max_pages, self.n_pages, self.page_size,
                self.token_cap, self.max_new, self.heads, self.kv_heads,
                self.grid, *(t.data_ptr() for t in (
                    self.streams, self.kv_lens, self.first_pages,
                    self.block_table, self.free_ring, self.ring_state,
                    self.q_start, self.q_lens, self.status, self.tokens,
                    self._work)))
        # (ctypes would cut off what passes 32 bits)
        d.max_new = min(self.max_new, 2 ** 31 - 1)
        return d

    def _check(self, shape, name, t):
        """t is a contiguous bf16 tensor of the shape, on the cache's
        device."""
        if t.dtype != _BF16 or not t.is_contiguous():
            raise ValueError("%s must be a contiguous bf16 tensor" % name)
        if t.shape != shape:
            wan._shape_is(t, shape, name)
        if t.get_device() != self._index:
            wan._on_cuda(("streams", self.streams), (name, t))

    def _weights(self, n, name, t):
        if t.dtype != torch.float32 or not t.is_contiguous() \
                or t.numel() != n:
            wan._f32_n(t, n, name)
        if t.get_device() != self._index:
            wan._on_cuda(("streams", self.streams), (name, t))

    def _bytes(self, need, name, t):
        if not t.is_contiguous():
            raise ValueError("%s must be a contiguous tensor" % name)
        if t.numel() * t.element_size() < need:
            raise ValueError("%s holds %d bytes, %d are needed"
                             % (name, t.numel() * t.element_size(), need))
        if t.get_device() != self._index:
            wan._on_cuda(("streams", self.streams), (name, t))

    def plan(self, new_lens, stream=None):
        """Plans a step: new_lens int32 CUDA tensor [R], > 0 new tokens of
        the stream, 0 none, < 0 the stream has ended (wan_paged_plan)."""
        if new_lens.dtype != torch.int32 or not new_lens.is_contiguous():
            raise ValueError("new_lens must be a contiguous int32 tensor")
        wan._shape_is(new_lens, (self.n_streams,), "new_lens")
        if new_lens.get_device() != self._index:
            wan._on_cuda(("streams", self.streams), ("new_lens", new_lens))
        wan.paged_plan(self.descriptor(), new_lens, stream=stream)
        self._planned = self.max_new

    def write(self, q, k, v, wq, wk, table, k_pages, v_pages, q_out=None,
              eps=1e-6, stream=None):
        """QK-Norm and RoPE of the planned rows: q into q_out (default: in
        place), k into its slots of k_pages; v into v_pages
        (wan_paged_write)."""
        self._check(self._q_shape, "q", q)
        if q_out is None:
            q_out = q
        else:
            self._check(self._q_shape, "q_out", q_out)
        self._check(self._kv_shape, "k", k)
        self._check(self._kv_shape, "v", v)
        self._check(self._pool_shape, "k_pages", k_pages)
        self._check(self._pool_shape, "v_pages", v_pages)
        self._weights(self.heads * 128, "wq", wq)
        self._weights(self.kv_heads * 128, "wk", wk)
        if table is None:
            raise ValueError("write needs a RoPE table")
        self._bytes(self._table_bytes, "table", table)
        wan.paged_write(self.descriptor(), q, q_out, k, v, wq, wk, k_pages,
                        v_pages, table, eps, stream=stream)

    def workspace_bytes(self):
        """Scratch an attention call needs."""
        if self._need_for != self.max_new:
            self._need = wan.paged_workspace_bytes(self.descriptor(),
                                                   self.device)
            self._need_for = self.max_new
        return self._need

    def workspace(self):
        """The cache's own scratch: one for each of the two sizes that a
        max_new can need, allocated with the cache and kept for its life,
        since captured graphs go on using the one they were captured with.
        Calls that overlap on the device need one each (``attn``'s workspace
        argument)."""
        return self._workspaces[self.workspace_bytes()]

    def attn(self, q, k_pages, v_pages, o, softmax_scale=None, stream=None,
             workspace=None):
        """o = softmax(q K^T scale) V over the pages for the planned rows
        (wan_paged_attn).  The last plan on the device must have been made
        with this max_new: a plan() call with another one is refused here, a
        graph replayed since leaves o as it was and shows in
        wan.device_status()."""
        self._check(self._q_shape, "q", q)
        self._check(self._q_shape, "o", o)
        self._check(self._pool_shape, "k_pages", k_pages)
        self._check(self._pool_shape, "v_pages", v_pages)
        if self._planned != self.max_new:
            # the plan divided the work for the kernel max_new picks
            raise ValueError("attn needs a plan made with the same max_new")
        if softmax_scale is None:
            softmax_scale = _SCALE
        if workspace is None:
            workspace = self.workspace()
        else:
            self._bytes(self.workspace_bytes(), "workspace", workspace)
        wan.paged_attn(self.descriptor(), q, k_pages, v_pages, o,
                       softmax_scale, workspace, stream=stream)
