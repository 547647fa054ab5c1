"""GB300 (sm_103a) submanifold sparse 3x3x3 convolution.

A thin Python binding over the C ABI of ``libspconv.so`` (include/spconv.h):
the functions below only check and marshal arguments; every step of the path
(mapper, masks, sort, compaction, GEMM) runs in the library's CUDA kernels.
PyTorch supplies device memory and streams.

    m = build_map(coords)                       # int32 [N, 4] (b, x, y, z), CUDA
    out = subm_forward(m, feats, weights)       # bf16 [N, C_in] x [27, C_in, C_out]

One map serves every layer on the same sites; weights can be packed once, and
a layer's batch norm (inference form), bias, residual and ReLU are applied to
the fp32 sum before its single rounding:

    wp = wpack_create(weights)                  # [27 or 125, C_in, C_out]
    y = subm_forward_packed(m, x, wp, scale=s, bias=b, residual=x, relu=True)
    y32 = subm_forward(m, x.float(), weights.float())   # exact fp32 mode

Kernel size 5 and offset groups: ``build_map(coords, kernel_size=5)`` (125
taps, always five groups), ``build_map(coords, groups=3)``.  Downsampling and
its inverse, on the output sites of a stride-2 grid:

    d = build_map_strided(coords)               # sites o with a site in {2o + d}
    y = subm_forward(d, x, w)                   # [d.n, C_out] at map_out_coords(d)
    u = build_map_inverse(d)                    # back onto the input sites
    z = subm_forward(u, y, w2)                  # [N, C_out2]

Between two convolutions on the same sites, on rows of features alone:

    y, x = rms_norm(y, w_norm, residual=x)      # norm of y + x, and the new residual
    h = gated_ffn(y, w_gate, w_up)              # silu(y W_gate) * (y W_up)
    x = linear(h, w_down, residual=x)           # act(h W + bias) + residual

with 8-bit forms (``rms_norm(..., quantize=True)``, ``quantize_weight``) and
gradients (``rms_norm_backward``, ``linear_backward``, ``gated_ffn_backward``).

The tensors, maps and packs of a call lie on the current GPU (``ValueError``
otherwise).  A ``stream`` argument belongs to it too; for a row-wise operator it
makes its own GPU current during the call.

Errors raise ``SpconvError`` with the library's status code; errors found on
the device (duplicate or out-of-range coordinates) surface through
``map_status`` or the next call on the map.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import torch

from . import _native

__all__ = ["SpconvError", "Map", "WPack", "build_map", "subm_forward", "wpack_create",
           "subm_forward_packed", "map_status", "map_info", "map_export", "map_destroy",
           "rms_norm", "rms_norm_backward", "linear", "linear_backward", "gated_ffn", "gated_ffn_backward",
           "quantize_weight", "rows_status", "trim_pool", "last_launch_count", "status_string", "ACTIVATIONS", "MAPPERS",
           "BIT_ORDERS", "PIPELINES", "GEMMS", "library"]

MAPPERS = {"auto": 0, "dense": 1, "sorted": 2, "hash": 3}
PIPELINES = {"auto": 0, "fused": 1, "multi": 2, "wide": 3}
GEMMS = {"auto": 0, "tile_union": 1, "tap_major": 2}
BIT_ORDERS = {"calibrated": 0, "plain": 1}
ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
_E4M3 = torch.float8_e4m3fn
_DTYPES = {torch.bfloat16: 0, torch.float32: 1}
_current_device = torch._C._cuda_getDevice   # (without a Device object)


def library():
    """The loaded ctypes library (raises if it has not been built)."""
    return _native.load()


def status_string(code: int) -> str:
    """The library's message for a status code (``spconv_status_string``)."""
    return library().spconv_status_string(int(code)).decode()


class SpconvError(RuntimeError):
    """A call into the library returned a status other than SPCONV_OK; ``code`` holds it."""

    def __init__(self, code: int, where: str = ""):
        super().__init__(f"{where}: {status_string(code)} ({code})" if where else status_string(code))
        self.code = code


def _check(code: int, where: str):
    if code != 0:
        raise SpconvError(code, where)


def _require_current(dev: int, name: str):
    """The library launches and allocates on the current device, so everything of a call belongs to it."""
    if dev != _current_device():
        raise ValueError(f"{name} is on cuda:{dev}, the current device is cuda:{_current_device()}")


def _stream_ptr(stream: Optional[torch.cuda.Stream]) -> ctypes.c_void_p:
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    _require_current(stream.device.index, "stream")
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t: Optional[torch.Tensor]) -> ctypes.c_void_p:
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _require_cuda(t: torch.Tensor, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    _require_current(t.get_device(), name)


class Map:
    """A kernel map (handle ``spconv_map_t``); shared by every layer on these sites."""

    def __init__(self, handle: ctypes.c_void_p, n: int, coords: torch.Tensor, kernel_size: int = 3,
                 n_in: Optional[int] = None, keep=None):
        self._h = handle
        self.n = n                 # rows: the sites the output lives on
        self.n_in = n if n_in is None else n_in   # rows of the features a forward reads
        self.kernel_size = kernel_size
        self.taps = kernel_size ** 3
        self._coords = coords      # kept alive while the build may still read it
        self._keep = keep          # (an inverse map: the strided map it reads)

    @property
    def handle(self) -> ctypes.c_void_p:
        if self._h is None:
            raise ValueError("map has been destroyed")
        return self._h

    def require_current(self):
        """Raises ``ValueError`` where the map is not on the current GPU."""
        _require_current(self._coords.get_device(), "map")

    def destroy(self):
        if getattr(self, "_h", None) is not None:
            library().spconv_map_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


class WPack:
    """Pre-packed weights (handle ``spconv_wpack_t``)."""

    def __init__(self, handle, c_in, c_out, dtype, src, taps=27):
        self._h = handle
        self.c_in, self.c_out, self.dtype, self.taps = c_in, c_out, dtype, taps
        self._src = src

    @property
    def handle(self):
        if self._h is None:
            raise ValueError("weight pack has been destroyed")
        return self._h

    def require_current(self):
        """Raises ``ValueError`` where the pack is not on the current GPU."""
        _require_current(self._src.get_device(), "weight pack")

    def destroy(self):
        if getattr(self, "_h", None) is not None:
            library().spconv_wpack_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def build_map(coords: torch.Tensor, spatial_shape: Optional[Sequence[int]] = None,
              batch_size: int = 0, kernel_size: int = 3, mapper: str = "auto",
              bit_order: str = "calibrated", dense_max_cells: int = 0, pipeline: str = "auto",
              gemm: str = "auto", stream: Optional[torch.cuda.Stream] = None, groups: int = 0) -> Map:
    """``spconv_build_map``: kernel map of ``coords`` (int32 [N, 4] (b, x, y, z) on the GPU).

    ``spatial_shape`` None and ``batch_size`` 0 derive them on the device
    (this synchronises the stream).  ``gemm`` picks the bf16 forward's work
    decomposition on this map (``GEMMS``).  ``kernel_size`` 3 or 5;
    ``groups`` the offset groups (0: 1 for K = 3, 5 for K = 5; or K).
    """
    st = _stream_ptr(stream)
    lib = library()
    _require_cuda(coords, "coords")
    if coords.dtype != torch.int32 or coords.dim() != 2 or coords.shape[1] != 4:
        raise ValueError("coords must be int32 [N, 4]")
    shape_arr = None
    if spatial_shape is not None:
        shape_arr = (ctypes.c_int32 * 3)(*[int(v) for v in spatial_shape])
    opt = _native.Options(MAPPERS[mapper], BIT_ORDERS[bit_order], int(dense_max_cells),
                          PIPELINES[pipeline], GEMMS[gemm], int(groups))
    h = ctypes.c_void_p()
    rc = lib.spconv_build_map(_ptr(coords), int(coords.shape[0]),
                              ctypes.cast(shape_arr, _native.c_int32_p) if shape_arr is not None else None,
                              int(batch_size), int(kernel_size), ctypes.byref(opt), st,
                              ctypes.byref(h))
    _check(rc, "spconv_build_map")
    return Map(h, int(coords.shape[0]), coords, int(kernel_size))


def _epilogue(n: int, c_out: int, dtype: torch.dtype, device, scale, bias, residual, relu):
    """The ``spconv_epilogue_t`` of a forward, or None when it is the identity.

    Returns (struct or None, tensors to keep alive until the call returns)."""
    if scale is None and bias is None and residual is None and not relu:
        return None, ()
    keep = []

    def vec(t, name):
        if t is None:
            return None
        _require_cuda(t, name)
        if t.dtype != torch.float32 or t.dim() != 1 or t.shape[0] != c_out or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous fp32 [{c_out}] tensor")
        keep.append(t)
        return t.data_ptr()

    e = _native.Epilogue()
    e.scale_dev = vec(scale, "scale")
    e.bias_dev = vec(bias, "bias")
    if residual is not None:
        _require_cuda(residual, "residual")
        if residual.dtype != dtype or tuple(residual.shape) != (n, c_out):
            raise ValueError(f"residual must be {dtype} [{n}, {c_out}]")
        keep.append(residual)
        e.residual_dev = residual.data_ptr()
    e.relu = 1 if relu else 0
    return e, tuple(keep)


def build_map_strided(coords: torch.Tensor, spatial_shape: Optional[Sequence[int]] = None,
                      batch_size: int = 0, kernel_size: int = 3, stride: int = 2, bit_order: str = "calibrated",
                      stream: Optional[torch.cuda.Stream] = None) -> Map:
    """``spconv_build_map_strided``: the map of a strided convolution (kernel 3, stride 2,
    padding 1) from the input sites ``coords``; its rows are the output sites
    (``map_out_coords``).  Synchronises the stream once."""
    st = _stream_ptr(stream)
    lib = library()
    _require_cuda(coords, "coords")
    if coords.dtype != torch.int32 or coords.dim() != 2 or coords.shape[1] != 4:
        raise ValueError("coords must be int32 [N, 4]")
    shape_arr = None
    if spatial_shape is not None:
        shape_arr = (ctypes.c_int32 * 3)(*[int(v) for v in spatial_shape])
    opt = _native.Options(0, BIT_ORDERS[bit_order], 0, 0, 0, 0)
    h = ctypes.c_void_p()
    rc = lib.spconv_build_map_strided(_ptr(coords), int(coords.shape[0]),
                                      ctypes.cast(shape_arr, _native.c_int32_p) if shape_arr is not None else None,
                                      int(batch_size), int(kernel_size), int(stride), ctypes.byref(opt),
                                      st, ctypes.byref(h))
    _check(rc, "spconv_build_map_strided")
    rows = ctypes.c_int64(0)
    _check(lib.spconv_map_rows(h, ctypes.byref(rows), None), "spconv_map_rows")   # (no second synchronisation)
    return Map(h, int(rows.value), coords, 3, n_in=int(coords.shape[0]))


def build_map_inverse(m: Map, bit_order: str = "calibrated") -> Map:
    """``spconv_build_map_inverse``: the map of the transposed convolution of strided map
    ``m``, from its output sites back onto its input sites."""
    m.require_current()
    opt = _native.Options(0, BIT_ORDERS[bit_order], 0, 0, 0, 0)
    h = ctypes.c_void_p()
    _check(library().spconv_build_map_inverse(m.handle, ctypes.byref(opt), ctypes.byref(h)),
           "spconv_build_map_inverse")
    return Map(h, m.n_in, m._coords, 3, n_in=m.n, keep=m)


def map_out_coords(m: Map, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """``spconv_map_out_coords``: a strided map's output sites, int32 [n, 4]."""
    m.require_current()
    st = _stream_ptr(stream)
    out = torch.empty((m.n, 4), dtype=torch.int32, device=torch.device("cuda", torch.cuda.current_device()))
    _check(library().spconv_map_out_coords(m.handle, _ptr(out), st), "spconv_map_out_coords")
    return out


def subm_forward(m: Map, feats: torch.Tensor, weights: torch.Tensor,
                 out: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None, *,
                 scale: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                 residual: Optional[torch.Tensor] = None, relu: bool = False) -> torch.Tensor:
    """``spconv_subm_forward``: feats [N, C_in] x weights [V, C_in, C_out] -> [N, C_out], V = K^3.

    bf16 inputs use fp32 accumulation and one rounding at the store; fp32
    inputs take the exact fp32 path.  ``scale``/``bias`` (fp32 [C_out]),
    ``residual`` ([N, C_out], the output dtype; may be ``out``) and ``relu``
    are applied to each fp32 sum before that rounding
    (``spconv_subm_forward_ex``): y = sum*scale + bias + residual, then max(y, 0).
    """
    m.require_current()
    st = _stream_ptr(stream)
    lib = library()
    _require_cuda(feats, "feats")
    _require_cuda(weights, "weights")
    if feats.dtype not in _DTYPES or weights.dtype != feats.dtype:
        raise ValueError("feats and weights must both be bf16 or both fp32")
    if feats.dim() != 2 or feats.shape[0] != m.n_in:
        raise ValueError(f"feats must be [{m.n_in}, C_in]")
    if weights.dim() != 3 or weights.shape[0] != m.taps or weights.shape[1] != feats.shape[1]:
        raise ValueError(f"weights must be [{m.taps}, C_in, C_out]")
    c_in, c_out = int(weights.shape[1]), int(weights.shape[2])
    if out is None:
        out = torch.empty((m.n, c_out), dtype=feats.dtype, device=feats.device)
    else:
        _require_cuda(out, "out")
        if out.dtype != feats.dtype or tuple(out.shape) != (m.n, c_out):
            raise ValueError(f"out must be {feats.dtype} [{m.n}, {c_out}]")
    epi, _keep = _epilogue(m.n, c_out, feats.dtype, feats.device, scale, bias, residual, relu)
    if epi is None:
        rc = lib.spconv_subm_forward(m.handle, _ptr(feats), _ptr(weights), _ptr(out), c_in, c_out,
                                     _DTYPES[feats.dtype], st)
        _check(rc, "spconv_subm_forward")
    else:
        rc = lib.spconv_subm_forward_ex(m.handle, _ptr(feats), _ptr(weights), _ptr(out), c_in, c_out,
                                        _DTYPES[feats.dtype], ctypes.byref(epi), st)
        _check(rc, "spconv_subm_forward_ex")
    return out


def wpack_create(weights: torch.Tensor, stream: Optional[torch.cuda.Stream] = None) -> WPack:
    """``spconv_wpack_create_ex``: pack [K^3, C_in, C_out] weights (K = 3 or 5,
    from the first dimension) once for many forwards."""
    st = _stream_ptr(stream)
    lib = library()
    _require_cuda(weights, "weights")
    sizes = {27: 3, 125: 5}
    if weights.dtype not in _DTYPES or weights.dim() != 3 or int(weights.shape[0]) not in sizes:
        raise ValueError("weights must be bf16 or fp32 [27 or 125, C_in, C_out]")
    c_in, c_out = int(weights.shape[1]), int(weights.shape[2])
    h = ctypes.c_void_p()
    rc = lib.spconv_wpack_create_ex(_ptr(weights), sizes[int(weights.shape[0])], c_in, c_out,
                                    _DTYPES[weights.dtype], st, ctypes.byref(h))
    _check(rc, "spconv_wpack_create_ex")
    return WPack(h, c_in, c_out, weights.dtype, weights, int(weights.shape[0]))


def subm_forward_packed(m: Map, feats: torch.Tensor, wp: WPack, out: Optional[torch.Tensor] = None,
                        stream: Optional[torch.cuda.Stream] = None, *,
                        scale: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                        residual: Optional[torch.Tensor] = None, relu: bool = False) -> torch.Tensor:
    """``spconv_subm_forward_packed``: forward with weights from ``wpack_create``;
    the epilogue arguments are those of ``subm_forward``."""
    m.require_current()
    wp.require_current()
    st = _stream_ptr(stream)
    lib = library()
    _require_cuda(feats, "feats")
    if feats.dtype != wp.dtype or feats.dim() != 2 or feats.shape != (m.n_in, wp.c_in):
        raise ValueError(f"feats must be {wp.dtype} [{m.n_in}, {wp.c_in}]")
    if wp.taps != m.taps:
        raise ValueError(f"weights pack has {wp.taps} taps, the map {m.taps}")
    if out is None:
        out = torch.empty((m.n, wp.c_out), dtype=feats.dtype, device=feats.device)
    else:
        _require_cuda(out, "out")
        if out.dtype != feats.dtype or tuple(out.shape) != (m.n, wp.c_out):
            raise ValueError(f"out must be {feats.dtype} [{m.n}, {wp.c_out}]")
    epi, _keep = _epilogue(m.n, wp.c_out, feats.dtype, feats.device, scale, bias, residual, relu)
    if epi is None:
        rc = lib.spconv_subm_forward_packed(m.handle, _ptr(feats), wp.handle, _ptr(out), st)
        _check(rc, "spconv_subm_forward_packed")
    else:
        rc = lib.spconv_subm_forward_packed_ex(m.handle, _ptr(feats), wp.handle, _ptr(out), ctypes.byref(epi), st)
        _check(rc, "spconv_subm_forward_packed_ex")
    return out


def subm_forward_layers(m: Map, feats: torch.Tensor, wps: Sequence[WPack], relu: Sequence[bool] = (),
                        outs: Optional[Sequence[torch.Tensor]] = None,
                        stream: Optional[torch.cuda.Stream] = None) -> list:
    """``spconv_subm_forward_layers``: ``len(wps)`` layers over map ``m`` in one launch;
    layer l reads layer l - 1's output (layer 0: ``feats``) and applies a ReLU
    when ``relu[l]``.  ``outs`` gives one output per layer (consecutive ones may
    not overlap; two buffers may alternate); by default two buffers alternate.
    Returns the list of per-layer outputs (views of ``outs``)."""
    m.require_current()
    for w in wps:
        w.require_current()
    st = _stream_ptr(stream)
    lib = library()
    _require_cuda(feats, "feats")
    L = len(wps)
    if L < 1:
        raise ValueError("at least one layer")
    wp0 = wps[0]
    if feats.dtype != torch.bfloat16 or tuple(feats.shape) != (m.n_in, wp0.c_in):
        raise ValueError(f"feats must be bf16 [{m.n_in}, {wp0.c_in}]")
    relu = list(relu) + [False] * (L - len(relu))
    if outs is None:
        bufs = [torch.empty((m.n, wp0.c_out), dtype=feats.dtype, device=feats.device) for _ in range(min(L, 2))]
        outs = [bufs[l % 2] for l in range(L)]
    else:
        outs = list(outs)
        if len(outs) != L:
            raise ValueError(f"{L} outputs expected")
        for o in outs:
            _require_cuda(o, "out")
            if o.dtype != feats.dtype or tuple(o.shape) != (m.n, wp0.c_out):
                raise ValueError(f"outputs must be bf16 [{m.n}, {wp0.c_out}]")
    wh = (ctypes.c_void_p * L)(*[w.handle for w in wps])
    oh = (ctypes.c_void_p * L)(*[_ptr(o) for o in outs])
    epis = (_native.Epilogue * L)()
    for l in range(L):
        epis[l].relu = 1 if relu[l] else 0
    rc = lib.spconv_subm_forward_layers(m.handle, _ptr(feats), ctypes.cast(wh, ctypes.POINTER(ctypes.c_void_p)),
                                        ctypes.cast(oh, ctypes.POINTER(ctypes.c_void_p)), L, epis, st)
    _check(rc, "spconv_subm_forward_layers")
    return outs


def map_status(m: Map) -> int:
    """``spconv_map_status``: 0, or the first device-detected error code (synchronises)."""
    return int(library().spconv_map_status(m.handle))


def map_info(m: Map) -> dict:
    """``spconv_map_info`` as a dict (synchronises)."""
    info = _native.MapInfo()
    _check(library().spconv_map_info(m.handle, ctypes.byref(info)), "spconv_map_info")
    return dict(n=info.n, pairs=info.pairs, n_tiles=info.n_tiles, tile_taps=info.tile_taps,
                mapper={1: "dense", 2: "sorted", 3: "hash"}.get(info.mapper, str(info.mapper)),
                pipeline={1: "fused", 2: "multi", 3: "wide"}.get(info.pipeline, str(info.pipeline)),
                key_bits=info.key_bits, shape=tuple(info.shape), batch_size=info.batch_size,
                gemm={1: "tile_union", 2: "tap_major"}.get(info.gemm, str(info.gemm)),
                kernel_size=info.kernel_size, groups=info.groups, n_in=info.n_in,
                conv={0: "submanifold", 1: "strided", 2: "inverse"}.get(info.conv, str(info.conv)),
                out_shape=tuple(info.out_shape))


def map_export(m: Map, stream: Optional[torch.cuda.Stream] = None) -> dict:
    """``spconv_map_export``: nbr [N, V], tap_off [V+1], in_rows/out_rows [P];
    mask and perm [N] with one offset group, [G, N] with G > 1."""
    m.require_current()
    st = _stream_ptr(stream)
    info = map_info(m)
    n, p = info["n"], info["pairs"]
    V, G = info["kernel_size"] ** 3, info["groups"]
    dev = torch.device("cuda", torch.cuda.current_device())
    nbr = torch.empty((n, V), dtype=torch.int32, device=dev)
    gshape = (n,) if G == 1 else (G, n)
    mask = torch.empty(gshape, dtype=torch.int32, device=dev)
    perm = torch.empty(gshape, dtype=torch.int32, device=dev)
    tap_off = torch.empty((V + 1,), dtype=torch.int32, device=dev)
    ins = torch.empty((max(p, 1),), dtype=torch.int32, device=dev)
    outs = torch.empty((max(p, 1),), dtype=torch.int32, device=dev)
    rc = library().spconv_map_export(m.handle, _ptr(nbr), _ptr(mask), _ptr(perm), _ptr(tap_off),
                                     _ptr(ins), _ptr(outs), st)
    _check(rc, "spconv_map_export")
    return dict(nbr=nbr, mask=mask, perm=perm, tap_off=tap_off, in_rows=ins[:p], out_rows=outs[:p],
                info=info)


def map_destroy(m: Map):
    """``spconv_map_destroy``."""
    m.destroy()


# ---- row-wise operators --------------------------------------------------------
# A call on a few rows costs what the host does for it, so these functions look
# at each tensor once and allocate only outputs.
_BF16 = torch.bfloat16
_raw_stream = torch._C._cuda_getCurrentRawStream   # of a device, without making a Stream object
_c = None


def _lib():
    global _c
    if _c is None:
        _c = library()
    return _c


def _rows(t: torch.Tensor, name: str, shape, dtype, dev: int) -> int:
    """Row stride of ``t``, checked to be ``shape`` rows of ``dtype`` on GPU ``dev``."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        raise ValueError(f"{name} must be a {dtype} {list(shape)} tensor on cuda:{dev}")
    ld, step = t.stride()
    n, c = shape
    if step != 1 and c > 1:
        raise ValueError(f"{name} must have contiguous rows")
    if ld < c:
        if n > 1:
            raise ValueError(f"{name} must not have overlapping rows")
        return c
    return ld


def _vector(t: torch.Tensor, name: str, c: int, dev: int) -> int:
    """Address of an fp32 [c] vector on GPU ``dev``."""
    if t.dtype is not torch.float32 or t.shape != (c,) or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous fp32 [{c}] tensor on cuda:{dev}")
    return t.data_ptr()


def _weight(t: torch.Tensor, name: str, shape, dtype, dev: int) -> int:
    """Address of a dense weight on GPU ``dev``."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} {list(shape)} tensor on cuda:{dev}")
    return t.data_ptr()


def _activation(name: str) -> int:
    code = ACTIVATIONS.get(name)
    if code is None:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}")
    return code


def _matrix(t: torch.Tensor, name: str):
    """The shape of a 2-D CUDA tensor and its GPU, which has to be the current one: the library takes
    its stream, its memory and its kernels there."""
    if t.dim() != 2 or not t.is_cuda:
        raise ValueError(f"{name} must be a 2-D CUDA tensor")
    dev = t.get_device()
    _require_current(dev, name)
    return t.shape, dev


def _on_stream(stream: torch.cuda.Stream, tensors, call):
    """``call()`` on ``stream``: what it allocates belongs to that stream, and what it reads is kept
    from reuse until the stream is past it."""
    if stream.cuda_stream != torch.cuda.current_stream(stream.device).cuda_stream:
        for t in tensors:
            if t is not None and t.is_cuda:
                t.record_stream(stream)
    with torch.cuda.stream(stream):
        return call()


def rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None, *, eps: float = 1e-6,
             quantize: bool = False, sum_out: Optional[torch.Tensor] = None,
             stream: Optional[torch.cuda.Stream] = None):
    """``spconv_rms_norm``: y = h / sqrt(mean(h^2) + eps) * weight over the rows of h = x + residual.

    ``x`` and ``residual`` bf16 or fp32 [N, C] (rows may be strided), ``weight`` fp32 [C].
    Returns y, or with ``quantize`` (q, scale): e4m3 values and one fp32 scale per row, y = q * scale.
    With a ``residual`` the sum h follows as the last value, in x's dtype: (y, h) or (q, scale, h).
    ``sum_out`` takes h ([N, C], contiguous; may be ``residual`` or ``x``)."""
    if stream is not None:
        return _on_stream(stream, (x, weight, residual, sum_out),
                          lambda: rms_norm(x, weight, residual, eps=eps, quantize=quantize, sum_out=sum_out))
    shape, dev = _matrix(x, "x")
    n, c = shape
    dtype = x.dtype
    dt = _DTYPES.get(dtype)
    if dt is None:
        raise ValueError("x must be bf16 or fp32")
    if weight is None:
        raise ValueError("weight is required")
    ldx, r, ldr = _rows(x, "x", shape, dtype, dev), None, 0
    w = _vector(weight, "weight", c, dev)
    h = sum_out
    if h is not None:
        _weight(h, "sum_out", shape, dtype, dev)
    device = x.device
    if residual is not None:
        r, ldr = residual.data_ptr(), _rows(residual, "residual", shape, dtype, dev)
        if h is None:
            h = torch.empty(shape, dtype=dtype, device=device)
    if quantize:
        out = torch.empty(shape, dtype=_E4M3, device=device)
        scale = torch.empty((n,), dtype=torch.float32, device=device)
    else:
        out, scale = torch.empty(shape, dtype=dtype, device=device), None
    rc = _lib().spconv_rms_norm(x.data_ptr(), ldx, r, ldr, w, n, c, dt, eps, None if h is None else h.data_ptr(),
                                out.data_ptr(), 2 if quantize else dt, None if scale is None else scale.data_ptr(),
                                _raw_stream(dev))
    if rc:
        raise SpconvError(rc, "spconv_rms_norm")
    if residual is None:
        return (out, scale) if quantize else out
    return (out, scale, h) if quantize else (out, h)


def rms_norm_backward(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, dres: Optional[torch.Tensor] = None, *,
                      eps: float = 1e-6, stream: Optional[torch.cuda.Stream] = None):
    """``spconv_rms_norm_backward``: (dx, dweight) of the norm of ``x`` (the sum ``rms_norm`` returned,
    where there was a residual), for the gradient ``dy`` of y and ``dres`` of the sum.  dx is the gradient
    of x and of the residual alike; dweight fp32 [C]."""
    if stream is not None:
        return _on_stream(stream, (dy, x, weight, dres), lambda: rms_norm_backward(dy, x, weight, dres, eps=eps))
    shape, dev = _matrix(x, "x")
    n, c = shape
    dtype = x.dtype
    dt = _DTYPES.get(dtype)
    if dt is None:
        raise ValueError("x must be bf16 or fp32")
    if weight is None:
        raise ValueError("weight is required")
    ldx, ldy, r, ldr = _rows(x, "x", shape, dtype, dev), _rows(dy, "dy", shape, dtype, dev), None, 0
    if dres is not None:
        r, ldr = dres.data_ptr(), _rows(dres, "dres", shape, dtype, dev)
    w = _vector(weight, "weight", c, dev)
    device = x.device
    dx = torch.empty(shape, dtype=dtype, device=device)
    dw = torch.empty((c,), dtype=torch.float32, device=device)
    rc = _lib().spconv_rms_norm_backward(dy.data_ptr(), ldy, x.data_ptr(), ldx, w, r, ldr, n, c, dt, eps, dx.data_ptr(),
                                         dw.data_ptr(), _raw_stream(dev))
    if rc:
        raise SpconvError(rc, "spconv_rms_norm_backward")
    return dx, dw


def _operands(x: torch.Tensor, w: torch.Tensor, name: str):
    """Checks x [N, C_in] against a weight, bf16 [C_in, C_out] or e4m3 [C_out, C_in].

    Returns (n, c_in, c_out, whether e4m3, row stride of x, shape of the weight, the GPU)."""
    shape, dev = _matrix(x, "x")
    n, c_in = shape
    dtype = x.dtype
    if w.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    if dtype is _BF16:
        eight, c_out = False, w.shape[1]
        wshape = (c_in, c_out)
    elif dtype is _E4M3:
        eight, c_out = True, w.shape[0]
        wshape = (c_out, c_in)
    else:
        raise ValueError("x must be bf16 or float8_e4m3fn")
    _weight(w, name, wshape, dtype, dev)
    return n, c_in, c_out, eight, _rows(x, "x", shape, dtype, dev), wshape, dev


def _scale(t: Optional[torch.Tensor], name: str, c: int, eight: bool, dev: int) -> Optional[int]:
    if (t is not None) != eight:
        raise ValueError(f"{name}: e4m3 operands need their scales, bf16 ones have none")
    return _vector(t, name, c, dev) if eight else None


def linear(x: torch.Tensor, weight: torch.Tensor, *, bias: Optional[torch.Tensor] = None, activation: str = "none",
           residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
           x_scale: Optional[torch.Tensor] = None, w_scale: Optional[torch.Tensor] = None,
           stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """``spconv_linear``: act(x W + bias) + residual, bf16 [N, C_out].

    bf16: ``x`` [N, C_in], ``weight`` [C_in, C_out].  8 bits: ``x`` float8_e4m3fn with ``x_scale`` fp32 [N],
    ``weight`` float8_e4m3fn [C_out, C_in] with ``w_scale`` fp32 [C_out] (``quantize_weight``).  ``bias`` fp32
    [C_out], ``residual`` bf16 [N, C_out] (may be ``out``); rows of x, residual and out may be strided."""
    if stream is not None:
        return _on_stream(stream, (x, weight, bias, residual, out, x_scale, w_scale),
                          lambda: linear(x, weight, bias=bias, activation=activation, residual=residual, out=out,
                                         x_scale=x_scale, w_scale=w_scale))
    n, c_in, c_out, eight, ldx, _, dev = _operands(x, weight, "weight")
    xs, ws = _scale(x_scale, "x_scale", n, eight, dev), _scale(w_scale, "w_scale", c_out, eight, dev)
    b, r, ldr = None, None, 0
    if bias is not None:
        b = _vector(bias, "bias", c_out, dev)
    if residual is not None:
        r, ldr = residual.data_ptr(), _rows(residual, "residual", (n, c_out), _BF16, dev)
    device = x.device
    if out is None:
        out, ldo = torch.empty((n, c_out), dtype=_BF16, device=device), c_out
    else:
        ldo = _rows(out, "out", (n, c_out), _BF16, dev)
    rc = _lib().spconv_linear(x.data_ptr(), ldx, xs, weight.data_ptr(), ws, n, c_in, c_out, 2 if eight else 0, b,
                              _activation(activation), r, ldr, out.data_ptr(), ldo, _raw_stream(dev))
    if rc:
        raise SpconvError(rc, "spconv_linear")
    return out


def linear_backward(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, *, bias: Optional[torch.Tensor] = None,
                    activation: str = "none", stream: Optional[torch.cuda.Stream] = None):
    """``spconv_linear_backward``: (dx, dweight, dbias) of act(x W + bias) for the gradient ``dy``; bf16,
    dbias fp32 (None without a bias).  The residual's gradient is ``dy`` itself."""
    if stream is not None:
        return _on_stream(stream, (dy, x, weight, bias),
                          lambda: linear_backward(dy, x, weight, bias=bias, activation=activation))
    n, c_in, c_out, eight, ldx, wshape, dev = _operands(x, weight, "weight")
    if eight:
        raise ValueError("gradients are of bf16 operands")
    ldy, b = _rows(dy, "dy", (n, c_out), _BF16, dev), None if bias is None else _vector(bias, "bias", c_out, dev)
    device = x.device
    dx = torch.empty((n, c_in), dtype=_BF16, device=device)
    dw = torch.empty(wshape, dtype=_BF16, device=device)
    db = None if bias is None else torch.empty((c_out,), dtype=torch.float32, device=device)
    rc = _lib().spconv_linear_backward(dy.data_ptr(), ldy, x.data_ptr(), ldx, weight.data_ptr(), n, c_in, c_out, 0,
                                       b, _activation(activation), dx.data_ptr(), dw.data_ptr(),
                                       None if db is None else db.data_ptr(), _raw_stream(dev))
    if rc:
        raise SpconvError(rc, "spconv_linear_backward")
    return dx, dw, db


def gated_ffn(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, *, activation: str = "silu",
              out: Optional[torch.Tensor] = None, x_scale: Optional[torch.Tensor] = None,
              gate_scale: Optional[torch.Tensor] = None, up_scale: Optional[torch.Tensor] = None,
              stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """``spconv_gated_ffn``: act(x W_gate) * (x W_up), bf16 [N, C_hidden].

    Operands as for ``linear``: bf16 [C_in, C_hidden] weights, or e4m3 [C_hidden, C_in] with scales."""
    if stream is not None:
        return _on_stream(stream, (x, w_gate, w_up, out, x_scale, gate_scale, up_scale),
                          lambda: gated_ffn(x, w_gate, w_up, activation=activation, out=out, x_scale=x_scale,
                                            gate_scale=gate_scale, up_scale=up_scale))
    n, c_in, c_h, eight, ldx, wshape, dev = _operands(x, w_gate, "w_gate")
    up = _weight(w_up, "w_up", wshape, x.dtype, dev)
    xs = _scale(x_scale, "x_scale", n, eight, dev)
    gs, us = _scale(gate_scale, "gate_scale", c_h, eight, dev), _scale(up_scale, "up_scale", c_h, eight, dev)
    device = x.device
    if out is None:
        out, ldo = torch.empty((n, c_h), dtype=_BF16, device=device), c_h
    else:
        ldo = _rows(out, "out", (n, c_h), _BF16, dev)
    rc = _lib().spconv_gated_ffn(x.data_ptr(), ldx, xs, w_gate.data_ptr(), gs, up, us, n, c_in, c_h, 2 if eight else 0,
                                 _activation(activation), out.data_ptr(), ldo, _raw_stream(dev))
    if rc:
        raise SpconvError(rc, "spconv_gated_ffn")
    return out


def gated_ffn_backward(dh: torch.Tensor, x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, *,
                       activation: str = "silu", stream: Optional[torch.cuda.Stream] = None):
    """``spconv_gated_ffn_backward``: (dx, dw_gate, dw_up) for the gradient ``dh`` of ``gated_ffn``; bf16."""
    if stream is not None:
        return _on_stream(stream, (dh, x, w_gate, w_up),
                          lambda: gated_ffn_backward(dh, x, w_gate, w_up, activation=activation))
    n, c_in, c_h, eight, ldx, wshape, dev = _operands(x, w_gate, "w_gate")
    if eight:
        raise ValueError("gradients are of bf16 operands")
    up = _weight(w_up, "w_up", wshape, x.dtype, dev)
    ldh = _rows(dh, "dh", (n, c_h), _BF16, dev)
    device = x.device
    dx = torch.empty((n, c_in), dtype=_BF16, device=device)
    dwg, dwu = torch.empty(wshape, dtype=_BF16, device=device), torch.empty(wshape, dtype=_BF16, device=device)
    rc = _lib().spconv_gated_ffn_backward(dh.data_ptr(), ldh, x.data_ptr(), ldx, w_gate.data_ptr(), up, n, c_in, c_h, 0,
                                          _activation(activation), dx.data_ptr(), dwg.data_ptr(), dwu.data_ptr(),
                                          _raw_stream(dev))
    if rc:
        raise SpconvError(rc, "spconv_gated_ffn_backward")
    return dx, dwg, dwu


def quantize_weight(weight: torch.Tensor, *, stream: Optional[torch.cuda.Stream] = None):
    """``spconv_quantize_weight``: bf16 [C_in, C_out] to (e4m3 [C_out, C_in], fp32 scale [C_out]), once per weight."""
    if stream is not None:
        return _on_stream(stream, (weight,), lambda: quantize_weight(weight))
    (c_in, c_out), dev = _matrix(weight, "weight")
    w = _weight(weight, "weight", (c_in, c_out), _BF16, dev)
    device = weight.device
    q = torch.empty((c_out, c_in), dtype=_E4M3, device=device)
    scale = torch.empty((c_out,), dtype=torch.float32, device=device)
    rc = _lib().spconv_quantize_weight(w, c_in, c_out, q.data_ptr(), scale.data_ptr(), _raw_stream(dev))
    if rc:
        raise SpconvError(rc, "spconv_quantize_weight")
    return q, scale


def rows_status(stream: Optional[torch.cuda.Stream] = None) -> int:
    """``spconv_rows_status``: 0, or the first error the row-wise operators recorded on the device since
    the last call (synchronises): on the current GPU, or on the stream's."""
    if stream is not None:
        return _on_stream(stream, (), rows_status)
    return int(library().spconv_rows_status(_stream_ptr(None)))


def trim_pool(keep_bytes: int = 0):
    """``spconv_trim_pool``: gives the memory that the library's pool holds on the current GPU without using it
    (scratch of the row-wise operators, destroyed maps and packs) back to the device (synchronises)."""
    _check(library().spconv_trim_pool(int(keep_bytes)), "spconv_trim_pool")


def last_launch_count() -> int:
    """Kernels the library launched in its last call on this thread."""
    return int(library().spconv_last_launch_count())
