"""The attention step around the linears: rotary positions with several axes, a paged FP8
key / value cache and the attention over it, and low-rank adapters beside a projection.

As in ``ops``, every call marshals arguments and launches the library's HIP kernels on the
current stream (include/fp8w8a8.h states each definition and layout). Batches are ragged:
request i owns the rows ``starts[i] .. starts[i + 1] - 1`` of a [tokens, ...] tensor, with
``starts`` int32 [requests + 1] on the GPU. Lengths, offsets, page and adapter numbers are
read by the kernels only, so no call waits for the GPU and all of them can be captured.
"""

import ctypes

import torch

from ._lib import ROPE_HALVES, ROPE_INTERLEAVED, check, lib, pack_rows
from .ops import _on_device, _ptr, _require

# The calls that serve single tokens take a few microseconds on the GPU, so the way there is
# kept short: tensors are looked at once, addresses go as integers, structures as packed words,
# the device is only changed where it is another one.
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_int32, _bf16 = torch.int32, torch.bfloat16


def _launch(device, name, fn, *args):
    """fn(*args, stream) on `device` and its current stream; raises if the library refuses."""
    index = device.index
    if index == torch.cuda.current_device():
        status = fn(*args, _current_stream(index))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _current_stream(index))
    if status:
        check(status, name)


def _dense(t, dtype, name, dims, device):
    """Require a contiguous tensor of this type and number of dims on the handle's device."""
    if not (isinstance(t, torch.Tensor) and t.get_device() == device.index and t.dtype is dtype and t.dim() == dims
            and t.is_contiguous()):
        _require(t, (dtype,), name, dims)
        _on_device(device, **{name: t})


def _rows(t, name, device=None, heads=None, dim=None):
    """Require a bf16 [tokens, heads, dim] tensor on a GPU (this one, if given), of any strides; returns its shape."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor (the HIP library is the only implementation)")
    if device is not None and t.get_device() != device.index:
        _on_device(device, **{name: t})
    if t.dtype is not _bf16:
        raise TypeError(f"{name} has dtype {t.dtype}, expected torch.bfloat16")
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{name} must be [tokens, heads, dim], got shape {tuple(shape)}")
    if heads is not None and shape[1] != heads:
        raise ValueError(f"{name} has {shape[1]} heads, expected {heads}")
    if dim is not None and shape[2] != dim:
        raise ValueError(f"{name} has head dimension {shape[2]}, expected {dim}")
    return shape


def _words(t):
    """A tensor's fp8_rows, or None if the library cannot take it in place (dense 16-byte aligned rows)."""
    tokens, heads, dim = t.shape
    token, head, column = t.stride()
    if tokens == 1:  # a stride that is never stepped may be anything
        token = dim
    if heads == 1:
        head = dim
    at = t.data_ptr()
    if column == 1 and token % 8 == 0 and head % 8 == 0 and at % 16 == 0:
        return pack_rows(at, heads, token, head)
    return None


def _packed(t):
    """(tensor, its fp8_rows): a dense copy where it cannot be taken in place. The caller holds it until the launch."""
    words = _words(t)
    if words is None:
        # not .contiguous(): a dense tensor at an odd address would come back as it is
        t = t.clone(memory_format=torch.contiguous_format)
        words = pack_rows(t.data_ptr(), t.shape[1], t.shape[1] * t.shape[2], t.shape[2])
    return t, words


def _new_like(t):
    return torch.empty_like(t) if t.is_contiguous() else torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _out_rows(out, like, name):
    """(output, its fp8_rows): the caller's, written in place, so it has to fit as it is, or a new dense one."""
    if out is None:
        out = _new_like(like)
    elif _rows(out, name, like.device, like.shape[1], like.shape[2])[0] != like.shape[0]:
        raise ValueError(f"{name} must have shape {tuple(like.shape)}, got {tuple(out.shape)}")
    words = _words(out)
    if words is None:
        raise ValueError(f"{name} must have dense 16-byte aligned rows")
    return out, words


class RopeAxes:
    """Rotary positions with several axes: ``widths[i]`` columns of every head turn with axis i.

    ``interleaved`` pairs neighbouring columns; otherwise column j of an axis pairs with
    column j + width / 2. Columns past the widths' sum pass through.
    """

    def __init__(self, head_dim, widths, base=10000.0, interleaved=True):
        self.head_dim, self.widths = int(head_dim), tuple(int(w) for w in widths)
        self._lib = lib()
        plan = ctypes.c_void_p()
        check(self._lib.fp8_rope_create(self.head_dim, len(self.widths), (ctypes.c_int64 * len(self.widths))(*self.widths),
                                        float(base), ROPE_INTERLEAVED if interleaved else ROPE_HALVES,
                                        ctypes.byref(plan)), "fp8_rope_create")
        self._plan = plan

    def __del__(self):
        plan = getattr(self, "_plan", None)
        if plan is not None and plan.value:
            self._lib.fp8_rope_destroy(plan)
            self._plan = None

    def forward(self, q, k, positions, q_out=None, k_out=None):
        """(rotated q, rotated k) of q [tokens, heads, head_dim] and k [tokens, any heads, head_dim] or None.

        ``positions`` is int32 [tokens, axes]. ``q_out`` / ``k_out`` may be q / k themselves.
        """
        tokens = _rows(q, "q", dim=self.head_dim)[0]
        device = q.device
        _dense(positions, _int32, "positions", 2, device)
        if positions.shape != (tokens, len(self.widths)):
            raise ValueError(f"positions must be [{tokens}, {len(self.widths)}], got {tuple(positions.shape)}")
        q, q_words = _packed(q)
        q_out, q_out_words = _out_rows(q_out, q, "q_out")
        k_words = k_out_words = None
        if k is None:
            if k_out is not None:
                raise ValueError("k_out without k")
        else:
            if _rows(k, "k", device, dim=self.head_dim)[0] != tokens:
                raise ValueError("q and k must have the same tokens")
            k, k_words = _packed(k)
            k_out, k_out_words = _out_rows(k_out, k, "k_out")
        if tokens:  # an empty tensor has no device address to pass
            _launch(device, "fp8_rope_run", self._lib.fp8_rope_run, self._plan, tokens, positions.data_ptr(), q_words,
                    q_out_words, k_words, k_out_words)
        return q_out, k_out

    __call__ = forward


class Fp8KVCache:
    """A pool of FP8 key / value pages, one scale for each page and head.

    ``Fp8KVCache(pages, heads, head_dim, page_tokens)`` allocates the pool;
    ``k_codes`` u8 [pages, heads, page_tokens, head_dim], ``v_codes`` u8 [pages, heads,
    head_dim, page_tokens], ``k_scale`` / ``v_scale`` fp32 [pages, heads] adopt one.
    """

    def __init__(self, pages=None, heads=None, head_dim=128, page_tokens=64, device=None, *, k_codes=None,
                 v_codes=None, k_scale=None, v_scale=None):
        given = [t is not None for t in (k_codes, v_codes, k_scale, v_scale)]
        if any(given) and not all(given):
            raise ValueError("pass k_codes, v_codes, k_scale and v_scale together")
        if all(given):
            if pages is not None or heads is not None:
                raise ValueError("pass either sizes or the pool's tensors, not both")
            _require(k_codes, (torch.uint8,), "k_codes", 4)
            _require(v_codes, (torch.uint8,), "v_codes", 4)
            _require(k_scale, (torch.float32,), "k_scale", 2)
            _require(v_scale, (torch.float32,), "v_scale", 2)
            pages, heads, page_tokens, head_dim = k_codes.shape
            if tuple(v_codes.shape) != (pages, heads, head_dim, page_tokens):
                raise ValueError(f"v_codes must be {(pages, heads, head_dim, page_tokens)}, got {tuple(v_codes.shape)}")
            for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
                if tuple(t.shape) != (pages, heads):
                    raise ValueError(f"{name} must be {(pages, heads)}, got {tuple(t.shape)}")
            device = k_codes.device
            _on_device(device, v_codes=v_codes, k_scale=k_scale, v_scale=v_scale)
        else:
            if pages is None or heads is None:
                raise ValueError("Fp8KVCache needs pages and heads, or a pool's tensors")
            device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
            if device.type != "cuda":
                raise ValueError(f"the pool must be on a GPU (the HIP library is the only implementation), not {device}")
            k_codes = torch.empty((pages, heads, page_tokens, head_dim), dtype=torch.uint8, device=device)
            v_codes = torch.empty((pages, heads, head_dim, page_tokens), dtype=torch.uint8, device=device)
            k_scale = torch.empty((pages, heads), dtype=torch.float32, device=device)
            v_scale = torch.empty((pages, heads), dtype=torch.float32, device=device)
        self.k_codes, self.v_codes, self.k_scale, self.v_scale = k_codes, v_codes, k_scale, v_scale
        self.pages, self.heads, self.page_tokens, self.head_dim = pages, heads, page_tokens, head_dim
        self.device = k_codes.device
        self._lib = lib()
        cache = ctypes.c_void_p()
        check(self._lib.fp8_kv_cache_create(self.device.index or 0, pages, page_tokens, heads, head_dim, _ptr(k_codes),
                                            _ptr(v_codes), _ptr(k_scale), _ptr(v_scale), ctypes.byref(cache)),
              "fp8_kv_cache_create")
        self._cache = cache

    def __del__(self):
        cache = getattr(self, "_cache", None)
        if cache is not None and cache.value:
            self._lib.fp8_kv_cache_destroy(cache)
            self._cache = None

    def _batch(self, table, lengths, starts):
        device = self.device
        _dense(table, _int32, "table", 2, device)
        _dense(lengths, _int32, "lengths", 1, device)
        _dense(starts, _int32, "starts", 1, device)
        requests = lengths.shape[0]
        rows, table_pages = table.shape
        if rows != requests or starts.shape[0] != requests + 1:
            raise ValueError(f"{requests} lengths need a table of {requests} rows and {requests + 1} starts, got "
                             f"{rows} and {starts.shape[0]}")
        return requests, table_pages

    def append(self, k, v, table, lengths, starts):
        """Quantise the step's k and v [tokens, heads, head_dim] into their pages.

        ``table`` int32 [requests, table_pages] names the pages, ``lengths`` int32 [requests]
        counts each request's tokens with the step's, which are the last.
        """
        requests, table_pages = self._batch(table, lengths, starts)
        tokens = _rows(k, "k", self.device, self.heads, self.head_dim)[0]
        if _rows(v, "v", self.device, self.heads, self.head_dim)[0] != tokens:
            raise ValueError("k and v must have the same tokens")
        if requests == 0 or tokens == 0 or table_pages == 0:  # nothing to store, or nowhere
            return
        k, k_words = _packed(k)
        v, v_words = _packed(v)
        _launch(self.device, "fp8_kv_append", self._lib.fp8_kv_append, self._cache, requests, tokens, k_words, v_words,
                table.data_ptr(), table_pages, lengths.data_ptr(), starts.data_ptr())

    def workspace_bytes(self, requests, tokens, heads, table_pages):
        """Bytes of workspace ``attend`` takes at these sizes."""
        return self._lib.fp8_kv_attend_workspace_bytes(self._cache, requests, tokens, heads, table_pages)

    def attend(self, q, table, lengths, starts, scale=None, causal=False, out=None, workspace=None):
        """Attention of the step's q [tokens, heads, head_dim] over each request's cached tokens.

        ``heads`` is a multiple of the cache's. ``scale`` defaults to head_dim ** -0.5.
        ``causal`` lets a token see the places up to its own. A token that sees nothing
        gives zeros.
        """
        requests, table_pages = self._batch(table, lengths, starts)
        tokens, heads, _ = _rows(q, "q", self.device, dim=self.head_dim)
        if heads == 0 or heads % self.heads != 0:
            raise ValueError(f"q has {heads} heads, not a multiple of the cache's {self.heads}")
        if out is None:
            out = _new_like(q)
        else:
            _dense(out, _bf16, "out", 3, self.device)
            if out.shape != q.shape:
                raise ValueError(f"out must have shape {tuple(q.shape)}, got {tuple(out.shape)}")
        if workspace is not None:
            _on_device(self.device, workspace=workspace)
            if not workspace.is_contiguous():  # its bytes are counted from its elements
                raise ValueError("workspace must be contiguous")
        if requests == 0 or tokens == 0:
            return out
        if table_pages == 0:  # no places at all: one page that is not named, so that rows of no request are left
            table, table_pages = torch.full((requests, 1), -1, dtype=_int32, device=self.device), 1
        q, q_words = _packed(q)
        if workspace is None:
            need = self.workspace_bytes(requests, tokens, heads, table_pages)
            if need:
                workspace = torch.empty((need,), dtype=torch.uint8, device=q.device)
        at, size = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())
        _launch(self.device, "fp8_kv_attend", self._lib.fp8_kv_attend, self._cache, requests, tokens, q_words,
                table.data_ptr(), table_pages, lengths.data_ptr(), starts.data_ptr(),
                self.head_dim ** -0.5 if scale is None else scale, 1 if causal else 0, out.data_ptr(), at, size)
        return out


class LoraAdapters:
    """Low-rank adapters of many requests beside a projection they share.

    ``a`` bf16 [adapters, rank, k], ``b`` bf16 [adapters, n, rank], ``scale`` fp32 [adapters]
    (ones if not given). ``forward(base, x, starts, adapter)`` adds
    scale[a] * B[a] (A[a] x) to the rows of each request whose adapter a is one of them.
    """

    def __init__(self, a, b, scale=None):
        _require(a, (torch.bfloat16,), "a", 3)
        _require(b, (torch.bfloat16,), "b", 3)
        adapters, rank, k = a.shape
        n = b.shape[1]
        if b.shape[0] != adapters or b.shape[2] != rank:
            raise ValueError(f"b must be [{adapters}, n, {rank}], got {tuple(b.shape)}")
        if scale is None:
            scale = torch.ones((adapters,), dtype=torch.float32, device=a.device)
        _require(scale, (torch.float32,), "scale", 1)
        if scale.shape[0] != adapters:
            raise ValueError("scale must have one entry per adapter")
        _on_device(a.device, b=b, scale=scale)
        self.a, self.b, self.scale = a, b, scale  # the plan borrows these
        self.adapters, self.rank, self.n, self.k = adapters, rank, n, k
        self.device = a.device
        self._lib = lib()
        plan = ctypes.c_void_p()
        check(self._lib.fp8_lora_create(self.device.index or 0, adapters, rank, n, k, _ptr(a), _ptr(b), _ptr(scale),
                                        ctypes.byref(plan)), "fp8_lora_create")
        self._plan = plan

    def __del__(self):
        plan = getattr(self, "_plan", None)
        if plan is not None and plan.value:
            self._lib.fp8_lora_destroy(plan)
            self._plan = None

    def forward(self, base, x, starts, adapter, out=None):
        """base [tokens, n] plus each request's adapter of x [tokens, k]; ``out`` may be ``base`` itself.

        ``adapter`` is int32 [requests]; a number outside 0 .. adapters - 1 means none. Rows
        outside every request are not written.
        """
        device = self.device
        _dense(base, _bf16, "base", 2, device)
        _dense(x, _bf16, "x", 2, device)
        _dense(starts, _int32, "starts", 1, device)
        _dense(adapter, _int32, "adapter", 1, device)
        tokens, requests = x.shape[0], adapter.shape[0]
        if x.shape[1] != self.k or base.shape != (tokens, self.n):
            raise ValueError(f"x must be [{tokens}, {self.k}] and base [{tokens}, {self.n}], got {tuple(x.shape)} "
                             f"and {tuple(base.shape)}")
        if starts.shape[0] != requests + 1:
            raise ValueError(f"{requests} adapter numbers need {requests + 1} starts, got {starts.shape[0]}")
        if out is None:
            out = torch.empty_like(base)
        else:
            _dense(out, _bf16, "out", 2, device)
            if out.shape != base.shape:
                raise ValueError(f"out must have shape {tuple(base.shape)}, got {tuple(out.shape)}")
        if tokens and requests:
            _launch(device, "fp8_lora_run", self._lib.fp8_lora_run, self._plan, requests, tokens, x.data_ptr(),
                    base.data_ptr(), starts.data_ptr(), adapter.data_ptr(), out.data_ptr())
        return out

    __call__ = forward


__all__ = ["RopeAxes", "Fp8KVCache", "LoraAdapters"]
