"""Binding of the softmax-attention operators of include/lq.h: per-head norm
and rotation of q and k, the paged key-value cache and attention over it.

Like the rest of the package this module only checks and marshals arguments.
A tensor's device decides where a call runs: the current device is switched
for the call when it is another one, and without an explicit ``stream`` the
current stream of the tensors' device is used.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

import linear_attention_recurrent_int8_b200 as _lq

_Tensor, _f32, _i32 = torch.Tensor, torch.float32, torch.int32
_current_device = torch.cuda.current_device
_raw_stream = torch._C._cuda_getCurrentRawStream


def _check_i32(value, name: str):
    """ctypes would cut the value off to 32 bits."""
    if not -(1 << 31) <= value < 1 << 31:
        raise ValueError(f"{name}: {value} is not a 32-bit integer")


@dataclass(frozen=True)
class AttnConfig:
    """lq_attn_config.  ``scale`` defaults to head_dim ** -0.5."""
    q_heads: int
    kv_heads: int
    head_dim: int = 128
    io_dtype: int = _lq.LQ_BF16
    norm: int = _lq.LQ_NORM_NONE
    eps: float = 1e-6
    rot_dim: int = 0
    rot_pairs: int = _lq.LQ_ROT_HALVES
    scale: float | None = None
    softcap: float = 0.0
    window: int = 0

    def __post_init__(self):
        for name in ("q_heads", "kv_heads", "head_dim", "io_dtype", "norm", "rot_dim", "rot_pairs", "window"):
            _check_i32(getattr(self, name), name)
        scale = self.head_dim ** -0.5 if self.scale is None and self.head_dim > 0 else self.scale
        c = _lq.LqAttnConfig(self.q_heads, self.kv_heads, self.head_dim, self.io_dtype, self.norm,
                             self.rot_dim, self.rot_pairs, self.window, self.eps, scale or 0.0,
                             self.softcap)
        if c.softcap == 0.0 and self.softcap != 0.0:  # (0 would mean no cap)
            raise ValueError(f"softcap: {self.softcap} is below the range of float")
        object.__setattr__(self, "_c", c)
        object.__setattr__(self, "_ref", ctypes.byref(c))
        object.__setattr__(self, "_layout", (self.kv_heads, self.head_dim, self.io_dtype))
        object.__setattr__(self, "io_torch_dtype",
                           torch.bfloat16 if self.io_dtype == _lq.LQ_BF16 else torch.float32)

    def c(self):
        """The C struct (its values are those given at construction)."""
        return self._c


class KvCache:
    """A paged key-value cache (lq_kv_cache): k_pages and v_pages [num_pages,
    kv_heads, page_size, head_dim] of the io dtype and block_table int32
    [batch, max_pages], torch tensors that the caller allocates.  Their
    contents may change between calls; the tensors are fixed."""

    def __init__(self, cfg: AttnConfig, k_pages, v_pages, block_table):
        for t, name in ((k_pages, "k_pages"), (v_pages, "v_pages")):
            _check_dense(t, name, cfg.io_torch_dtype)
            if t.dim() != 4 or t.shape[1] != cfg.kv_heads or t.shape[3] != cfg.head_dim:
                raise ValueError(f"{name}: shape {tuple(t.shape)}, expected [num_pages, {cfg.kv_heads}, "
                                 f"page_size, {cfg.head_dim}]")
        if k_pages.shape != v_pages.shape:
            raise ValueError(f"v_pages: shape {tuple(v_pages.shape)}, k_pages has {tuple(k_pages.shape)}")
        _check_dense(block_table, "block_table", torch.int32)
        if block_table.dim() != 2:
            raise ValueError(f"block_table: shape {tuple(block_table.shape)}, expected [batch, max_pages]")
        if v_pages.device != k_pages.device or block_table.device != k_pages.device:
            raise ValueError("k_pages, v_pages and block_table: on different devices")
        self._tensors = (k_pages, v_pages, block_table)
        self.layout = cfg._layout
        self.device = k_pages.device
        self.batch, self.max_pages = block_table.shape
        self.num_pages, _, self.page_size, _ = k_pages.shape
        for name in ("batch", "max_pages", "num_pages", "page_size"):
            _check_i32(getattr(self, name), name)
        self._c = _lq.LqKvCache(k_pages.data_ptr(), v_pages.data_ptr(), block_table.data_ptr(),
                                self.batch, self.num_pages, self.page_size, self.max_pages)
        self._ref = ctypes.byref(self._c)

    @property
    def k_pages(self):
        return self._tensors[0]

    @property
    def v_pages(self):
        return self._tensors[1]

    @property
    def block_table(self):
        return self._tensors[2]

    def c(self):
        return self._c


# --------------------------------------------------------------------------
# Argument checks
# --------------------------------------------------------------------------
#
# These run on every call of a decode step, whose kernels take a few
# microseconds: each check asks a tensor for as little as it needs, and the
# devices are compared by index.

def _check_dense(t, name: str, dtype):
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: not contiguous")


def _check_vector(t, name: str, dtype, numel: int):
    _check_dense(t, name, dtype)
    if t.numel() != numel:
        raise ValueError(f"{name}: {t.numel()} elements, expected {numel} (shape {tuple(t.shape)})")


def _rows(t, name: str, cfg: AttnConfig, heads: int):
    """(tokens, token stride) of a [..., heads, head_dim] tensor whose heads
    are contiguous and whose tokens lie at one stride."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dtype is not cfg.io_torch_dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {cfg.io_torch_dtype}")
    shape = t.shape
    d = cfg.head_dim
    if len(shape) < 3 or shape[-2] != heads or shape[-1] != d:
        raise ValueError(f"{name}: shape {tuple(shape)}, expected [..., tokens, {heads}, {d}]")
    if t.is_contiguous():
        return t.numel() // (heads * d), heads * d
    strides = t.stride()
    if strides[-1] != 1 or (heads > 1 and strides[-2] != d):
        raise ValueError(f"{name}: the heads of a token are not contiguous (strides {strides})")
    if len(shape) == 3 and shape[0] > 1:
        return shape[0], strides[0]
    tokens, stride = 1, None  # leading dimensions, innermost first, as one
    for n, s in zip(reversed(shape[:-2]), reversed(strides[:-2])):
        if n == 1:
            continue
        if stride is None:
            stride = s
        elif s != stride * tokens:
            raise ValueError(f"{name}: the tokens do not lie at one stride (strides {strides})")
        tokens *= n
    return tokens, heads * d if stride is None else stride


def _check_out(t, name: str, cfg: AttnConfig, tokens: int, heads: int):
    _check_dense(t, name, cfg.io_torch_dtype)
    shape = t.shape
    if t.numel() != tokens * heads * cfg.head_dim or len(shape) < 2 or shape[-1] != cfg.head_dim or \
            shape[-2] != heads:
        raise ValueError(f"{name}: shape {tuple(shape)}, expected {tokens} rows of [{heads}, {cfg.head_dim}]")


def _check_weights(cfg: AttnConfig, q_weight, k_weight):
    if q_weight is not None:
        _check_vector(q_weight, "q_weight", _f32, cfg.head_dim)
    if k_weight is not None:
        _check_vector(k_weight, "k_weight", _f32, cfg.head_dim)


def _table_len(cfg: AttnConfig, cos_sin) -> int:
    if cos_sin is None:
        return 0
    _check_dense(cos_sin, "cos_sin", _f32)
    shape = cos_sin.shape
    if len(shape) != 2 or shape[1] != cfg.rot_dim:
        raise ValueError(f"cos_sin: shape {tuple(shape)}, expected [positions, {cfg.rot_dim}]")
    return shape[0]


def _check_devices(*tensors) -> int:
    """Index of the CUDA device that all of the tensors (None aside) are on."""
    first = None
    for t in tensors:
        if t is not None:
            i = t.get_device()  # -1 on the host
            if i < 0:
                raise ValueError(f"expected CUDA tensors, one {tuple(t.shape)} is on {t.device}")
            if first is None:
                first = i
            elif i != first:
                raise ValueError(f"a tensor {tuple(t.shape)} is on {t.device}, others are on cuda:{first}")
    return first


def _check_cache(cfg: AttnConfig, cache: KvCache):
    if not isinstance(cache, KvCache):
        raise TypeError(f"cache: expected a KvCache, got {type(cache).__name__}")
    if cache.layout != cfg._layout:
        raise ValueError(f"cache: made for (kv_heads, head_dim, io_dtype) {cache.layout}, not {cfg._layout}")


def _check_places(cache: KvCache, pos, cu_tokens, tokens: int):
    _check_vector(pos, "pos", _i32, cache.batch)
    if cu_tokens is not None:
        _check_vector(cu_tokens, "cu_tokens", _i32, cache.batch + 1)
    elif cache.batch < 1 or tokens % cache.batch != 0:
        raise ValueError(f"{tokens} tokens for {cache.batch} sequences need cu_tokens")


def _stream_on(index: int, stream) -> int:
    """cudaStream_t of a call on device `index`."""
    if stream is None:
        return _raw_stream(index)
    if stream.device.index != index:
        raise ValueError(f"stream: on {stream.device}, expected cuda:{index}")
    return stream.cuda_stream


def _call(index: int, name: str, *args):
    """The C function with device `index` current."""
    f = getattr(_lq.load_library(), name)
    if _current_device() == index:
        status = f(*args)
    else:
        with torch.cuda.device(index):
            status = f(*args)
    if status != _lq.LQ_OK:
        _lq._check(status, name)


def _p(t):
    return None if t is None else t.data_ptr()


# --------------------------------------------------------------------------
# The C entry points, same names
# --------------------------------------------------------------------------

def lq_qk_norm_rotate(cfg: AttnConfig, q, k, q_weight, k_weight, positions, cos_sin, q_out, k_out,
                      stream=None) -> None:
    """Norm and rotation of q [..., tokens, q_heads, head_dim] and k [...,
    tokens, kv_heads, head_dim] (k and k_out may be None) into q_out and
    k_out; q and k may be token-strided slices of one projection's output."""
    n, q_stride = _rows(q, "q", cfg, cfg.q_heads)
    k_stride = 0
    _check_out(q_out, "q_out", cfg, n, cfg.q_heads)
    if (k is None) != (k_out is None):
        raise ValueError("k and k_out: give both or neither")
    if k is not None:
        nk, k_stride = _rows(k, "k", cfg, cfg.kv_heads)
        if nk != n:
            raise ValueError(f"k: {nk} tokens, q has {n}")
        _check_out(k_out, "k_out", cfg, n, cfg.kv_heads)
    _check_weights(cfg, q_weight, k_weight)
    table_len = _table_len(cfg, cos_sin)
    if positions is not None:
        _check_vector(positions, "positions", _i32, n)
    dev = _check_devices(q, k, q_weight, k_weight, positions, cos_sin, q_out, k_out)
    _call(dev, "lq_qk_norm_rotate", cfg._ref, _p(q), q_stride, _p(k), k_stride, _p(q_weight),
          _p(k_weight), _p(positions), _p(cos_sin), table_len, n, _p(q_out), _p(k_out),
          _stream_on(dev, stream))


def lq_kv_append(cfg: AttnConfig, cache: KvCache, pos, cu_tokens, q, k, v, q_weight, k_weight, cos_sin,
                 q_out, stream=None) -> None:
    """Appends the keys (normalised and rotated) and values of new tokens to
    the cache and writes the normalised and rotated q to q_out (q and q_out
    may be None).  pos: int32 [batch], tokens already cached (negative: idle
    slot); cu_tokens: int32 [batch + 1], or None for equally many new tokens
    per sequence."""
    _check_cache(cfg, cache)
    n, k_stride = _rows(k, "k", cfg, cfg.kv_heads)
    nv, v_stride = _rows(v, "v", cfg, cfg.kv_heads)
    if nv != n:
        raise ValueError(f"v: {nv} tokens, k has {n}")
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out: give both or neither")
    q_stride = 0
    if q is not None:
        nq, q_stride = _rows(q, "q", cfg, cfg.q_heads)
        if nq != n:
            raise ValueError(f"q: {nq} tokens, k has {n}")
        _check_out(q_out, "q_out", cfg, n, cfg.q_heads)
    _check_weights(cfg, q_weight, k_weight)
    table_len = _table_len(cfg, cos_sin)
    _check_places(cache, pos, cu_tokens, n)
    dev = _check_devices(cache.k_pages, q, k, v, q_weight, k_weight, pos, cu_tokens, cos_sin, q_out)
    _call(dev, "lq_kv_append", cfg._ref, cache._ref, _p(pos), _p(cu_tokens), n, _p(q), q_stride, _p(k),
          k_stride, _p(v), v_stride, _p(q_weight), _p(k_weight), _p(cos_sin), table_len, _p(q_out),
          _stream_on(dev, stream))


def lq_attn_workspace_bytes(cfg: AttnConfig, batch: int) -> int:
    """Bytes of lq_attn_decode's workspace on the current device; -1 for an
    invalid configuration or batch."""
    _check_i32(batch, "batch")
    return _lq.load_library().lq_attn_workspace_bytes(cfg._ref, int(batch))


def lq_attn_decode(cfg: AttnConfig, cache: KvCache, pos, q, o, workspace="auto", stream=None) -> None:
    """Attention of one new token per sequence (appended before) over its
    cached tokens: q and o [batch, q_heads, head_dim].  workspace: "auto"
    allocates (torch) what lq_attn_workspace_bytes gives; a CUDA tensor is
    used as it is and must not serve two calls at once."""
    _check_cache(cfg, cache)
    _check_out(q, "q", cfg, cache.batch, cfg.q_heads)
    _check_out(o, "o", cfg, cache.batch, cfg.q_heads)
    _check_vector(pos, "pos", _i32, cache.batch)
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError(f"workspace: {workspace!r}")
        dev = _check_devices(cache.k_pages, pos, q, o)
        # allocated on the call's own stream: the memory is that stream's
        with torch.cuda.device(dev), torch.cuda.stream(stream):
            workspace = torch.empty(max(lq_attn_workspace_bytes(cfg, cache.batch), 0),
                                    dtype=torch.uint8, device="cuda")
    elif not isinstance(workspace, torch.Tensor) or not workspace.is_contiguous():
        raise ValueError("workspace: expected a contiguous tensor")
    else:
        dev = _check_devices(cache.k_pages, pos, q, o, workspace)
    _call(dev, "lq_attn_decode", cfg._ref, cache._ref, _p(pos), _p(q), _p(o), _p(workspace),
          workspace.numel() * workspace.element_size(), _stream_on(dev, stream))


def lq_attn_prefill(cfg: AttnConfig, cache: KvCache, pos, cu_tokens, q, o, stream=None) -> None:
    """Attention of runs of new tokens (appended before) over the cached
    tokens up to each one's own position: q and o [tokens, q_heads,
    head_dim]; pos and cu_tokens as for lq_kv_append."""
    _check_cache(cfg, cache)
    _check_dense(q, "q", cfg.io_torch_dtype)
    n = q.numel() // max(cfg.q_heads * cfg.head_dim, 1)  # (the library refuses heads of none)
    _check_out(q, "q", cfg, n, cfg.q_heads)
    _check_out(o, "o", cfg, n, cfg.q_heads)
    _check_places(cache, pos, cu_tokens, n)
    dev = _check_devices(cache.k_pages, pos, cu_tokens, q, o)
    _call(dev, "lq_attn_prefill", cfg._ref, cache._ref, _p(pos), _p(cu_tokens), n, _p(q), _p(o),
          _stream_on(dev, stream))
