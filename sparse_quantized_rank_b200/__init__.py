"""Python binding of libcql, the B200 compressed linear layer.

    y = deq(Q (.) M) x + S_csr x + deq(L_q) (deq(R_q) x)

Argument marshalling only: every function below calls the C ABI declared in
``include/cql.h`` with the same name, passing device pointers taken from torch
tensors (torch supplies device memory and streams, nothing else).  There is no
CPU fallback: if ``libcql.so`` is missing or cannot be loaded, the first call
raises.

``CompressedLinear`` is a small convenience owner of the packed buffer and
workspace for one layer.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libcql.so")
LIB_CHECKED_PATH = os.path.join(HERE, "libcql_checked.so")   # the range-checked build

# enums (include/cql.h)
CQL_OK, CQL_ERR_ARG, CQL_ERR_ALIGN, CQL_ERR_FORMAT, CQL_ERR_SIZE, CQL_ERR_UNSUPPORTED, \
    CQL_ERR_CUDA, CQL_ERR_TIMEOUT, CQL_ERR_RANGE = range(9)
CQL_MASK_NONE, CQL_MASK_2_4, CQL_MASK_BITMAP50 = 0, 1, 2
CQL_CODEC_INT4_SYM, CQL_CODEC_INT3_SYM, CQL_CODEC_LUT3_ROW, CQL_CODEC_LUT4_ROW = 0, 1, 2, 3
CQL_DT_F32, CQL_DT_F16, CQL_DT_BF16, CQL_DT_FP8_BLOCK = 0, 1, 2, 3
CQL_FLAG_NO_MAIN, CQL_FLAG_NO_CSR, CQL_FLAG_NO_LOWRANK = 1, 2, 4
CQL_FLAG_DEBUG_SKIP_X = 0x100
CQL_FLAG_CUDA_CORE = 0x200
CQL_NPLANES = 13
CQL_MAX_DECODE_BATCH = 16
CQL_FP8_MAX_ROWS, CQL_FP8_MAX_COLS, CQL_FP8_MAX_OUT, CQL_FP8_MAX_TOKENS, CQL_FP8_MAX_EXPERTS = \
    1 << 24, 65536, 1 << 20, 1 << 20, 1024

EXPORTED = (
    "cql_status_string", "cql_version", "cql_packed_layout", "cql_pack_workspace_size",
    "pack_compressed_weight", "cql_workspace_size", "cql_workspace_init",
    "compressed_linear_forward", "cql_get_device_status", "compressed_linear_forward_noalloc",
    "cql_adapter_workspace_size", "cql_build_adapters", "cql_read_header", "cql_plane_checksums",
    "cql_fp8_matrix_layout", "cql_fp8_quantize", "cql_fp8_dequantize", "cql_fp8_workspace_size",
    "cql_fp8_linear_forward", "cql_fp8_grouped_forward",
)


class cql_desc(ctypes.Structure):
    _fields_ = [
        ("n_out", ctypes.c_int32), ("k_in", ctypes.c_int32), ("mask", ctypes.c_int32),
        ("codec", ctypes.c_int32), ("group", ctypes.c_int32), ("clip_alpha", ctypes.c_float),
        ("outlier_frac", ctypes.c_float), ("rank", ctypes.c_int32), ("adapter_bits", ctypes.c_int32),
        ("adapter_group", ctypes.c_int32), ("flags", ctypes.c_uint32), ("salient_channels", ctypes.c_int32),
        ("salient_log2", ctypes.c_int32), ("reserved", ctypes.c_int32 * 3),
    ]


class cql_layout(ctypes.Structure):
    _fields_ = [
        ("total_bytes", ctypes.c_uint64), ("nnz", ctypes.c_uint64),
        ("off", ctypes.c_uint64 * CQL_NPLANES), ("len", ctypes.c_uint64 * CQL_NPLANES),
    ]


class cql_fp8_layout(ctypes.Structure):
    _fields_ = [(f, ctypes.c_uint64) for f in ("total_bytes", "codes_off", "codes_len", "scales_off", "scales_len")]


class CqlError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {cql_status_string(status)} ({status})")
        self.status = status


_libs = {}
_active = LIB_PATH


def use_library(checked: bool) -> None:
    """Route every call of this module to the range-checked library
    (libcql_checked.so, built with -DCQL_CHECKED) or back to libcql.so.
    Objects keep the buffers they made with either; both libraries share the
    packed format and the workspace layout."""
    global _active
    _active = LIB_CHECKED_PATH if checked else LIB_PATH


def lib():
    """The loaded library (raises if it is missing: there is no fallback)."""
    if _active not in _libs:
        if not os.path.exists(_active):
            raise RuntimeError(f"{_active} is missing: build it with "
                               "`python -m sparse_quantized_rank_b200.build`"
                               + (" --checked" if _active == LIB_CHECKED_PATH else ""))
        L = ctypes.CDLL(_active)
        P, U64, I32 = ctypes.c_void_p, ctypes.c_uint64, ctypes.c_int32
        L.cql_status_string.restype = ctypes.c_char_p
        L.cql_status_string.argtypes = [ctypes.c_int]
        L.cql_version.restype = I32
        L.cql_packed_layout.argtypes = [ctypes.POINTER(cql_desc), ctypes.POINTER(cql_layout)]
        L.cql_pack_workspace_size.argtypes = [ctypes.POINTER(cql_desc), ctypes.POINTER(U64)]
        L.pack_compressed_weight.argtypes = [ctypes.POINTER(cql_desc), P, ctypes.c_int, P, P, P, P, P, U64, P,
                                             U64, P]
        L.cql_workspace_size.argtypes = [ctypes.POINTER(cql_desc), I32, ctypes.POINTER(U64)]
        L.cql_workspace_init.argtypes = [P, U64, P]
        L.compressed_linear_forward.argtypes = [ctypes.POINTER(cql_desc), P, P, ctypes.c_int, P, ctypes.c_int,
                                                I32, P, U64, P]
        L.cql_get_device_status.argtypes = [P, P, ctypes.POINTER(ctypes.c_int)]
        L.compressed_linear_forward_noalloc.argtypes = [ctypes.POINTER(cql_desc), P, P, ctypes.c_int, P,
                                                        ctypes.c_int, I32, P]
        L.cql_adapter_workspace_size.argtypes = [ctypes.POINTER(cql_desc), ctypes.POINTER(U64)]
        L.cql_build_adapters.argtypes = [ctypes.POINTER(cql_desc), P, ctypes.c_int, P, P, P, P, P, U64, P]
        L.cql_read_header.argtypes = [P, U64, ctypes.POINTER(cql_desc), ctypes.POINTER(cql_layout)]
        L.cql_plane_checksums.argtypes = [P, U64, ctypes.POINTER(ctypes.c_uint32 * CQL_NPLANES)]
        I64, DT = ctypes.c_int64, ctypes.c_int
        L.cql_fp8_matrix_layout.argtypes = [I64, I32, ctypes.POINTER(cql_fp8_layout)]
        L.cql_fp8_quantize.argtypes = [P, DT, I64, I32, I64, P, U64, P]
        L.cql_fp8_dequantize.argtypes = [P, U64, I64, I32, P, DT, I64, P]
        L.cql_fp8_workspace_size.argtypes = [I32, I32, I32, ctypes.POINTER(U64)]
        L.cql_fp8_linear_forward.argtypes = [I32, I32, P, P, DT, I64, P, DT, I64, I32, P, U64, P, P]
        L.cql_fp8_grouped_forward.argtypes = [I32, I32, I32, P, P, DT, I64, P, P, DT, I64, I32, P, U64, P, P]
        for fn in EXPORTED[2:]:
            getattr(L, fn).restype = ctypes.c_int
        _libs[_active] = L
    return _libs[_active]


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(s) -> Optional[int]:
    if s is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(st: int, where: str):
    if st != CQL_OK:
        raise CqlError(st, where)


def make_desc(n_out: int, k_in: int, mask: int = CQL_MASK_2_4, codec: int = CQL_CODEC_INT4_SYM,
              clip_alpha: float = 0.9, outlier_frac: float = 0.0, rank: int = 0, flags: int = 0,
              salient_channels: int = 0, salient_log2: int = 0) -> cql_desc:
    d = cql_desc()
    d.n_out, d.k_in, d.mask, d.codec, d.group = n_out, k_in, mask, codec, 128
    d.clip_alpha, d.outlier_frac, d.rank = clip_alpha, outlier_frac, rank
    d.adapter_bits, d.adapter_group, d.flags = 4, 128, flags
    d.salient_channels, d.salient_log2 = salient_channels, salient_log2
    return d


# ---------------------------------------------------------------------------
# the C ABI, same names
# ---------------------------------------------------------------------------

def cql_status_string(s: int) -> str:
    return lib().cql_status_string(int(s)).decode()


def cql_version() -> int:
    return int(lib().cql_version())


def cql_packed_layout(desc: cql_desc) -> cql_layout:
    out = cql_layout()
    _check(lib().cql_packed_layout(ctypes.byref(desc), ctypes.byref(out)), "cql_packed_layout")
    return out


def cql_pack_workspace_size(desc: cql_desc) -> int:
    v = ctypes.c_uint64()
    _check(lib().cql_pack_workspace_size(ctypes.byref(desc), ctypes.byref(v)), "cql_pack_workspace_size")
    return int(v.value)


def pack_compressed_weight(desc, W, w_dt, L, R, act_absmean, fisher, packed, packed_bytes, workspace, ws_bytes,
                           stream=None):
    _check(lib().pack_compressed_weight(ctypes.byref(desc), _ptr(W), int(w_dt), _ptr(L), _ptr(R), _ptr(act_absmean),
                                        _ptr(fisher), _ptr(packed), int(packed_bytes), _ptr(workspace),
                                        int(ws_bytes), _stream(stream)),
           "pack_compressed_weight")


def cql_workspace_size(desc: cql_desc, batch: int) -> int:
    v = ctypes.c_uint64()
    _check(lib().cql_workspace_size(ctypes.byref(desc), int(batch), ctypes.byref(v)), "cql_workspace_size")
    return int(v.value)


def cql_workspace_init(workspace, ws_bytes, stream=None):
    _check(lib().cql_workspace_init(_ptr(workspace), int(ws_bytes), _stream(stream)), "cql_workspace_init")


def compressed_linear_forward(desc, packed, x, x_dt, y, y_dt, batch, workspace, ws_bytes, stream=None):
    _check(lib().compressed_linear_forward(ctypes.byref(desc), _ptr(packed), _ptr(x), int(x_dt), _ptr(y), int(y_dt),
                                           int(batch), _ptr(workspace), int(ws_bytes), _stream(stream)),
           "compressed_linear_forward")


def compressed_linear_forward_noalloc(desc, packed, x, x_dt, y, y_dt, batch, stream=None):
    """Forward without a workspace (the library's fixed 4 MiB scratch array is
    used instead); for callers that cannot allocate device memory."""
    _check(lib().compressed_linear_forward_noalloc(ctypes.byref(desc), _ptr(packed), _ptr(x), int(x_dt), _ptr(y),
                                                   int(y_dt), int(batch), _stream(stream)),
           "compressed_linear_forward_noalloc")


def cql_adapter_workspace_size(desc: cql_desc) -> int:
    v = ctypes.c_uint64()
    _check(lib().cql_adapter_workspace_size(ctypes.byref(desc), ctypes.byref(v)), "cql_adapter_workspace_size")
    return int(v.value)


def cql_build_adapters(desc, W, w_dt, packed, act_absmean, L, R, workspace, ws_bytes, stream=None):
    _check(lib().cql_build_adapters(ctypes.byref(desc), _ptr(W), int(w_dt), _ptr(packed), _ptr(act_absmean), _ptr(L),
                                    _ptr(R), _ptr(workspace), int(ws_bytes), _stream(stream)),
           "cql_build_adapters")


def cql_read_header(packed_host: bytes):
    """(cql_desc, cql_layout) stored in a host copy of a packed buffer."""
    buf = ctypes.create_string_buffer(bytes(packed_host), len(packed_host))
    d, lay = cql_desc(), cql_layout()
    _check(lib().cql_read_header(ctypes.cast(buf, ctypes.c_void_p), len(packed_host), ctypes.byref(d),
                                 ctypes.byref(lay)), "cql_read_header")
    return d, lay


def cql_plane_checksums(packed_host: bytes):
    """CRC-32 of every plane of a host copy of a packed buffer."""
    buf = ctypes.create_string_buffer(bytes(packed_host), len(packed_host))
    out = (ctypes.c_uint32 * CQL_NPLANES)()
    _check(lib().cql_plane_checksums(ctypes.cast(buf, ctypes.c_void_p), len(packed_host), ctypes.byref(out)),
           "cql_plane_checksums")
    return list(out)


def cql_get_device_status(workspace, stream=None) -> int:
    """Device error word of a workspace (None: the fixed scratch of the
    no-workspace entry point on the current device)."""
    v = ctypes.c_int()
    _check(lib().cql_get_device_status(_ptr(workspace), _stream(stream), ctypes.byref(v)), "cql_get_device_status")
    return int(v.value)


def cql_fp8_matrix_layout(rows: int, cols: int) -> cql_fp8_layout:
    out = cql_fp8_layout()
    _check(lib().cql_fp8_matrix_layout(int(rows), int(cols), ctypes.byref(out)), "cql_fp8_matrix_layout")
    return out


def cql_fp8_quantize(src, dt, rows, cols, ld, matrix, matrix_bytes, stream=None):
    _check(lib().cql_fp8_quantize(_ptr(src), int(dt), int(rows), int(cols), int(ld), _ptr(matrix), int(matrix_bytes),
                                  _stream(stream)), "cql_fp8_quantize")


def cql_fp8_dequantize(matrix, matrix_bytes, rows, cols, out, dt, ld, stream=None):
    _check(lib().cql_fp8_dequantize(_ptr(matrix), int(matrix_bytes), int(rows), int(cols), _ptr(out), int(dt), int(ld),
                                    _stream(stream)), "cql_fp8_dequantize")


def cql_fp8_workspace_size(k_in: int, experts: int, tokens: int) -> int:
    v = ctypes.c_uint64()
    _check(lib().cql_fp8_workspace_size(int(k_in), int(experts), int(tokens), ctypes.byref(v)),
           "cql_fp8_workspace_size")
    return int(v.value)


def cql_fp8_linear_forward(n_out, k_in, weight, x, x_dt, ldx, y, y_dt, ldy, tokens, workspace, ws_bytes, status,
                           stream=None):
    _check(lib().cql_fp8_linear_forward(n_out, k_in, _ptr(weight), _ptr(x), x_dt, ldx, _ptr(y), y_dt, ldy, tokens,
                                        _ptr(workspace), ws_bytes, _ptr(status), _stream(stream)),
           "cql_fp8_linear_forward")


def cql_fp8_grouped_forward(n_out, k_in, experts, weight, x, x_dt, ldx, offsets, y, y_dt, ldy, tokens, workspace,
                            ws_bytes, status, stream=None):
    _check(lib().cql_fp8_grouped_forward(n_out, k_in, experts, _ptr(weight), _ptr(x), x_dt, ldx, _ptr(offsets),
                                         _ptr(y), y_dt, ldy, tokens, _ptr(workspace), ws_bytes, _ptr(status),
                                         _stream(stream)),
           "cql_fp8_grouped_forward")


# ---------------------------------------------------------------------------
# convenience owner of one packed layer
# ---------------------------------------------------------------------------

def check_forward_args(desc: cql_desc, x, out=None, device=None) -> None:
    """Raise ValueError unless x is a contiguous [B][K] fp16/bf16 tensor and
    out (if given) a contiguous [B][N] fp32/fp16/bf16 tensor, both on
    ``device`` (the packed layer's).  The C entry point receives raw
    pointers and cannot see a tensor's size, so a wrong shape would make the
    kernels read or write past its end: it is refused here."""
    import torch
    if x.dim() != 2 or x.shape[1] != desc.k_in or not x.is_contiguous():
        raise ValueError(f"x must be a contiguous [batch][{desc.k_in}] tensor, got {tuple(x.shape)}")
    if x.dtype not in (torch.float16, torch.bfloat16):
        raise ValueError(f"x must be float16 or bfloat16, got {x.dtype}")
    if device is not None and x.device != device:
        raise ValueError(f"x is on {x.device}, the packed layer on {device}")
    if out is not None:
        if tuple(out.shape) != (x.shape[0], desc.n_out) or not out.is_contiguous():
            raise ValueError(f"out must be a contiguous [{x.shape[0]}][{desc.n_out}] tensor, got {tuple(out.shape)}")
        if out.dtype not in (torch.float32, torch.float16, torch.bfloat16):
            raise ValueError(f"out must be float32, float16 or bfloat16, got {out.dtype}")
        if out.device != x.device:
            raise ValueError(f"out is on {out.device}, x on {x.device}")


def check_pack_args(desc: cql_desc, W, L=None, R=None, act_absmean=None, fisher=None) -> None:
    """Raise ValueError unless the packer's inputs have the shapes and dtypes
    the descriptor implies (W [N][K] fp32/bf16; L [N][r], R [r][K],
    act_absmean [K], fisher [N][K] fp32) and share W's device.  The C entry
    point reads them through raw pointers and cannot check their sizes."""
    import torch
    n, k, r = desc.n_out, desc.k_in, desc.rank
    want = [("W", W, (n, k), (torch.float32, torch.bfloat16))]
    if r > 0:
        if L is None or R is None:
            raise ValueError(f"rank {r} needs L [{n}][{r}] and R [{r}][{k}]")
        want += [("L", L, (n, r), (torch.float32,)), ("R", R, (r, k), (torch.float32,))]
    if act_absmean is not None:
        want.append(("act_absmean", act_absmean, (k,), (torch.float32,)))
    elif desc.salient_channels > 0:
        raise ValueError("salient_channels > 0 needs act_absmean [K]")
    if fisher is not None:
        want.append(("fisher", fisher, (n, k), (torch.float32,)))
    for name, t, shape, dts in want:
        if tuple(t.shape) != shape:
            raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
        if t.dtype not in dts:
            raise ValueError(f"{name} must be one of {dts}, got {t.dtype}")
        if t.device != W.device:
            raise ValueError(f"{name} is on {t.device}, W on {W.device}")


def _dt_of(t) -> int:
    import torch
    return {torch.float32: CQL_DT_F32, torch.float16: CQL_DT_F16, torch.bfloat16: CQL_DT_BF16}[t.dtype]


class CompressedLinear:
    """Packs one layer on the GPU and runs its forward pass.

    ``W`` is a CUDA tensor [N][K] (fp32 or bf16), ``L`` [N][r] and ``R`` [r][K]
    fp32 CUDA tensors (or None when rank is 0), ``act_absmean`` a fp32 CUDA
    tensor [K] of per-channel mean |x| (SLiM^O layers only), ``fisher`` a
    fp32 CUDA tensor [N][K] Fisher diagonal (LUT codecs: weighted k-means).
    A descriptor with clip_alpha 0 has the packer search alpha; the chosen
    value is in ``clip_alpha()``.  Buffers are torch tensors: the packed
    layer once, and one forward workspace per distinct batch size, on the
    first call at that size (its layout depends on the batch, and the
    kernels leave it ready for the next call at the same size); later calls
    allocate only the output tensor (or none, given ``out``)."""

    def __init__(self, desc: cql_desc, W, L=None, R=None, stream=None, act_absmean=None, fisher=None):
        import torch
        check_pack_args(desc, W, L, R, act_absmean, fisher)
        self.desc = desc
        self.layout = cql_packed_layout(desc)
        dev = W.device
        self.packed = torch.empty(self.layout.total_bytes, dtype=torch.uint8, device=dev)
        pw = cql_pack_workspace_size(desc)
        pws = torch.empty(max(pw, 256), dtype=torch.uint8, device=dev)
        args = [None if t is None else t.contiguous() for t in (W, L, R, act_absmean, fisher)]
        if isinstance(stream, torch.cuda.Stream):
            # the pack runs on a side stream: keep the allocator from reusing
            # the inputs' memory (the caller may drop W right away, and the
            # contiguous copies are temporaries) before that stream is done
            for t in args:
                if t is not None:
                    t.record_stream(stream)
        Wc, Lc, Rc, ac, fc = args
        pack_compressed_weight(desc, Wc, _dt_of(Wc), Lc, Rc, ac, fc, self.packed, self.layout.total_bytes, pws, pw,
                               stream)
        self._pack_ws = pws            # kept alive until the pack kernels ran
        self._ws = {}

    def clip_alpha(self) -> float:
        """The clip threshold the layer was encoded with (read from the packed
        header: the searched value when the descriptor asked for a search)."""
        return float(self.packed[28:32].cpu().view(__import__("torch").float32).item())

    @classmethod
    def with_adapters(cls, desc: cql_desc, W, act_absmean=None, naive: bool = False, stream=None, fisher=None):
        """Pack W with adapters built on the GPU from its own compression
        error: SLiM-LoRA weighted by ``act_absmean`` (Naive-LoRA when
        ``naive`` or when no statistic is given).  Packs with zero adapters,
        builds L and R (cql_build_adapters), packs again with them.  The
        built factors are kept as ``.L`` and ``.R``."""
        import torch
        dev = W.device
        r = desc.rank
        zL = torch.zeros(desc.n_out, r, dtype=torch.float32, device=dev)
        zR = torch.zeros(r, desc.k_in, dtype=torch.float32, device=dev)
        first = cls(desc, W, zL, zR, stream=stream, act_absmean=act_absmean, fisher=fisher)
        nb = cql_adapter_workspace_size(desc)
        ws = torch.empty(max(nb, 256), dtype=torch.uint8, device=dev)
        stat = None if (naive or act_absmean is None) else act_absmean.contiguous()
        cql_build_adapters(desc, W.contiguous(), _dt_of(W), first.packed, stat, zL, zR, ws, nb, stream)
        layer = cls(desc, W, zL, zR, stream=stream, act_absmean=act_absmean, fisher=fisher)
        layer.L, layer.R = zL, zR
        layer._build_ws = (ws, first)            # alive until the queued kernels ran
        return layer

    def workspace(self, batch: int, stream=None):
        import torch
        nbytes = cql_workspace_size(self.desc, batch)
        ws = self._ws.get(batch)
        if ws is None:
            ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=self.packed.device)
            cql_workspace_init(ws, nbytes, stream)
            self._ws[batch] = ws
        return ws, nbytes

    def forward(self, x, out_dtype=None, out=None, flags: Optional[int] = None, stream=None):
        import torch
        check_forward_args(self.desc, x, out, self.packed.device)
        batch = x.shape[0]
        if out is None:
            out = torch.empty(batch, self.desc.n_out, dtype=out_dtype or x.dtype, device=x.device)
        ws, nbytes = self.workspace(batch, stream)
        d = self.desc
        if flags is not None:
            d = cql_desc.from_buffer_copy(self.desc)
            d.flags = flags
        compressed_linear_forward(d, self.packed, x, _dt_of(x), out, _dt_of(out), batch, ws, nbytes, stream)
        return out

    def device_status(self, batch: int, stream=None) -> int:
        ws, _ = self.workspace(batch, stream)
        return cql_get_device_status(ws, stream)

    def pack_status(self, stream=None) -> int:
        """Device error word of the pack that built this layer: CQL_OK, or
        CQL_ERR_RANGE when the range-checked library saw a pack kernel index
        outside its plane."""
        return cql_get_device_status(self._pack_ws, stream)


# ---------------------------------------------------------------------------
# block-scaled FP8 matrices and layers
# ---------------------------------------------------------------------------
# These calls are short next to a decode step, so their path through Python is
# kept short too: sizes are looked up once for each shape, the device and stream
# are only switched where they differ from the current ones, and the library is
# called with plain numbers (1.5 us less than through the functions above).

@functools.lru_cache(maxsize=4096)
def _fp8_bytes(rows: int, cols: int) -> int:
    return int(cql_fp8_matrix_layout(rows, cols).total_bytes)


@functools.lru_cache(maxsize=4096)
def _fp8_scratch(k_in: int, experts: int, tokens: int) -> int:
    return cql_fp8_workspace_size(k_in, experts, tokens)


def _rows_of(name: str, t, cols: Optional[int] = None) -> int:
    """Raise ValueError unless t is a 2-D fp32/fp16/bf16 tensor whose rows do
    not overlap and whose columns are adjacent (and number ``cols``, if
    given); return the distance between its rows in elements."""
    shape = t.shape
    if len(shape) != 2 or (cols is not None and shape[1] != cols):
        raise ValueError(f"{name} must be a [rows][{'cols' if cols is None else cols}] tensor, got {tuple(shape)}")
    if t.dtype not in (_FP8_TYPES or _fp8_types()):
        raise ValueError(f"{name} must be float32, float16 or bfloat16, got {t.dtype}")
    rows, width = shape
    r, c = t.stride()
    if width > 1 and c != 1:
        raise ValueError(f"{name}: the columns of a row must be adjacent, got strides {tuple(t.stride())}")
    if rows <= 1:
        return width
    if r < width:
        raise ValueError(f"{name}: rows must not overlap, got strides {tuple(t.stride())}")
    return r


def _no_gradient(name: str) -> None:
    """Raise ValueError if autograd would have to see the call: there is no
    backward pass, and an output without history would drop the gradient."""
    import torch
    if torch.is_grad_enabled():
        raise ValueError(f"{name} requires grad, and the block-scaled FP8 layers have no backward pass: call under "
                         f"torch.no_grad() or detach {name}")


_FP8_TYPES = {}


def _fp8_types():
    if not _FP8_TYPES:
        import torch
        _FP8_TYPES.update({torch.float32: CQL_DT_F32, torch.float16: CQL_DT_F16, torch.bfloat16: CQL_DT_BF16})
    return _FP8_TYPES


def _stream_of(device, stream):
    """A caller's stream as torch knows it: a raw handle too becomes a stream
    that torch's allocator can keep memory for."""
    import torch
    if stream is None or isinstance(stream, torch.cuda.Stream):
        return stream
    if device.type != "cuda":
        raise ValueError(f"block-scaled FP8 runs on CUDA tensors, got {device}")
    return torch.cuda.ExternalStream(int(stream), device=device)


def _on(device, stream, call):
    """call(raw stream) with the tensors' device (and the caller's stream, if
    one is given) current, so that what it allocates belongs to that stream."""
    import torch
    index = device.index
    if index is None or device.type != "cuda":
        raise ValueError(f"block-scaled FP8 runs on CUDA tensors, got {device}")
    if stream is None:
        if index == torch._C._cuda_getDevice():
            return call(torch._C._cuda_getCurrentRawStream(index))
        with torch.cuda.device(device):
            return call(torch._C._cuda_getCurrentRawStream(index))
    if stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
    with torch.cuda.device(device), torch.cuda.stream(stream):
        return call(stream.cuda_stream)


class Fp8Matrix:
    """A block-scaled FP8 matrix [rows][cols] in the memory layout of
    ``include/cql.h``: ``buffer`` is a contiguous uint8 CUDA tensor of at least
    ``cql_fp8_matrix_layout(rows, cols).total_bytes`` bytes, 256-byte aligned.
    The buffer is all there is to save and load."""

    def __init__(self, rows: int, cols: int, buffer):
        import torch
        self.nbytes = _fp8_bytes(rows, cols)
        if buffer.dtype != torch.uint8 or not buffer.is_contiguous():
            raise ValueError("buffer must be a contiguous uint8 tensor")
        if buffer.numel() < self.nbytes:
            raise ValueError(f"buffer has {buffer.numel()} bytes, [{rows}][{cols}] needs {self.nbytes}")
        if buffer.data_ptr() % 256:
            raise ValueError("buffer must be 256-byte aligned")
        self.rows, self.cols, self.buffer = int(rows), int(cols), buffer
        self.device = buffer.device

    @property
    def layout(self) -> cql_fp8_layout:
        return cql_fp8_matrix_layout(self.rows, self.cols)

    @classmethod
    def quantize(cls, src, stream=None):
        """The block-scaled form of a [rows][cols] fp32/fp16/bf16 CUDA tensor
        (any distance between rows, adjacent columns).  The codes are frozen: no
        gradient reaches a parameter that they were made from."""
        import torch
        ld = _rows_of("src", src)
        rows, cols = src.shape

        n, device = _fp8_bytes(rows, cols), src.device

        def call(s):
            buffer = torch.empty(n, dtype=torch.uint8, device=device)
            st = lib().cql_fp8_quantize(src.data_ptr(), _FP8_TYPES[src.dtype], rows, cols, ld, buffer.data_ptr(), n, s)
            if st != CQL_OK:
                raise CqlError(st, "cql_fp8_quantize")
            return buffer

        if stream is not None:
            stream = _stream_of(device, stream)
        m = cls.__new__(cls)
        m.rows, m.cols, m.nbytes, m.device = rows, cols, n, device
        m.buffer = _on(device, stream, call)
        if stream is not None:
            src.record_stream(stream)
        return m

    def dequantize(self, dtype=None, out=None, stream=None):
        """The matrix's values as a [rows][cols] tensor of ``dtype`` (float32,
        exact, unless given), or into ``out``."""
        import torch
        if out is None:
            dtype = dtype or torch.float32
            if dtype not in _fp8_types():
                raise ValueError(f"dtype must be float32, float16 or bfloat16, got {dtype}")
        else:
            if tuple(out.shape) != (self.rows, self.cols) or (dtype is not None and dtype != out.dtype):
                raise ValueError(f"out must be [{self.rows}][{self.cols}] of the asked dtype, got {tuple(out.shape)} "
                                 f"{out.dtype}")
            if out.device != self.device:
                raise ValueError(f"out is on {out.device}, the matrix on {self.device}")

        def call(s):
            y = out if out is not None else torch.empty(self.rows, self.cols, dtype=dtype, device=self.device)
            ld = self.cols if out is None else _rows_of("out", out)
            st = lib().cql_fp8_dequantize(self.buffer.data_ptr(), self.nbytes, self.rows, self.cols, y.data_ptr(),
                                          _FP8_TYPES[y.dtype], ld, s)
            if st != CQL_OK:
                raise CqlError(st, "cql_fp8_dequantize")
            return y

        if stream is not None:
            stream = _stream_of(self.device, stream)
        y = _on(self.device, stream, call)
        if stream is not None:
            self.buffer.record_stream(stream)
            y.record_stream(stream)
        return y


class _Fp8Layer:
    """What ``Fp8Linear`` and ``Fp8Experts`` share: the weight, the device
    error word, and the checks and memory of a call.  Scratch and (unless
    ``out`` is given) output memory comes from torch's allocator on the call's
    stream, so calls may overlap on several streams and be captured.

    A forward reads the weight before the kernels in front of it are complete:
    after a kernel that writes the layer's weight buffer (other than
    ``cql_fp8_quantize``), some operation that is not a forward has to come first
    on the stream (``include/cql.h``).  Making the layer contains one.

    The layers have no backward pass; a forward refuses an x that requires grad
    while gradients are enabled."""

    def __init__(self, weight, n_experts: int, n_out: int, stream=None):
        import torch
        if n_out < 1:
            raise ValueError("the layer has no outputs")
        if not isinstance(weight, Fp8Matrix):
            weight = Fp8Matrix.quantize(weight, stream)
        self.weight, self.n_experts, self.n_out, self.k_in = weight, n_experts, n_out, weight.cols
        self.device = weight.device
        self._index = self.device.index
        _fp8_types()
        self.status = _on(self.device, _stream_of(self.device, stream), lambda s: torch.zeros(2, dtype=torch.int32, device=self.device))

    def _call(self, x, offsets, out_dtype, out, stream):
        import torch
        if isinstance(x, Fp8Matrix):
            if x.cols != self.k_in:
                raise ValueError(f"x has {x.cols} columns, the layer reads {self.k_in}")
            tokens, ldx, x_dt, src, scratch = x.rows, 0, CQL_DT_FP8_BLOCK, x.buffer, 0
        else:
            ldx, src = _rows_of("x", x, self.k_in), x
            if x.requires_grad:
                _no_gradient("x")
            tokens, x_dt = x.shape[0], _FP8_TYPES[x.dtype]
            scratch = _fp8_scratch(self.k_in, self.n_experts, tokens)
        if src.device != self.device:
            raise ValueError(f"x is on {src.device}, the layer on {self.device}")
        if out is None:
            dtype = out_dtype or (torch.bfloat16 if ldx == 0 else x.dtype)
            ldy, y_dt = self.n_out, _FP8_TYPES.get(dtype)
            if y_dt is None:
                raise ValueError(f"out_dtype must be float32, float16 or bfloat16, got {dtype}")
        else:
            if tuple(out.shape) != (tokens, self.n_out) or (out_dtype is not None and out_dtype != out.dtype):
                raise ValueError(f"out must be [{tokens}][{self.n_out}] of the asked dtype, got {tuple(out.shape)} "
                                 f"{out.dtype}")
            if out.device != self.device:
                raise ValueError(f"out is on {out.device}, the layer on {self.device}")
            if out.requires_grad:
                _no_gradient("out")
            dtype, ldy, y_dt = out.dtype, _rows_of("out", out), _FP8_TYPES[out.dtype]

        if stream is None and torch._C._cuda_getDevice() == self._index:          # the common case, straight on
            return self._launch(src, x_dt, ldx, offsets, out, dtype, y_dt, ldy, tokens, scratch,
                                torch._C._cuda_getCurrentRawStream(self._index))
        if stream is not None:
            stream = _stream_of(self.device, stream)
        y = _on(self.device, stream, lambda s: self._launch(src, x_dt, ldx, offsets, out, dtype, y_dt, ldy, tokens,
                                                            scratch, s))
        if stream is not None:
            for t in (src, y, offsets, self.weight.buffer, self.status):
                if t is not None:
                    t.record_stream(stream)
        return y

    def _launch(self, src, x_dt, ldx, offsets, y, dtype, y_dt, ldy, tokens, scratch, s):
        """The call itself, on the current stream (s: its handle)."""
        import torch
        empty, device = torch.empty, self.device
        if y is None:
            y = empty(tokens, self.n_out, dtype=dtype, device=device)
        ws = empty(scratch, dtype=torch.uint8, device=device) if scratch else None
        at = ws.data_ptr() if scratch else None
        if offsets is None:
            st = lib().cql_fp8_linear_forward(
                self.n_out, self.k_in, self.weight.buffer.data_ptr(), src.data_ptr(), x_dt, ldx, y.data_ptr(), y_dt,
                ldy, tokens, at, scratch, self.status.data_ptr(), s)
        else:
            st = lib().cql_fp8_grouped_forward(
                self.n_out, self.k_in, self.n_experts, self.weight.buffer.data_ptr(), src.data_ptr(), x_dt, ldx,
                offsets.data_ptr(), y.data_ptr(), y_dt, ldy, tokens, at, scratch, self.status.data_ptr(), s)
        if st != CQL_OK:
            raise CqlError(st, "cql_fp8_linear_forward" if offsets is None else "cql_fp8_grouped_forward")
        return y

    def device_status(self, stream=None) -> int:
        """The first error that a call of this layer recorded on the device
        (CQL_OK if none), read after the stream's work and cleared."""
        return _on(self.device, _stream_of(self.device, stream), lambda s: cql_get_device_status(self.status, s))


class Fp8Linear(_Fp8Layer):
    """y = Xq Wq^T with block-scaled FP8 operands.  ``weight``: an Fp8Matrix
    [n_out][k_in], or a fp32/fp16/bf16 CUDA tensor that is quantised here."""

    def __init__(self, weight, stream=None):
        super().__init__(weight, 1, weight.rows if isinstance(weight, Fp8Matrix) else weight.shape[0], stream)

    def forward(self, x, out_dtype=None, out=None, stream=None):
        """x: [tokens][k_in] fp32/fp16/bf16 (any distance between rows),
        quantised here, or an Fp8Matrix.  Returns [tokens][n_out] in
        ``out_dtype`` (x's dtype unless given; bfloat16 for an Fp8Matrix), or
        writes ``out`` (any distance between rows)."""
        return self._call(x, None, out_dtype, out, stream)


class Fp8Experts(_Fp8Layer):
    """The linear layer of each expert over its own tokens.  ``weight``: an
    Fp8Matrix of experts * n_out rows (expert e's rows from e * n_out on), or a
    [experts][n_out][k_in] CUDA tensor that is quantised here."""

    def __init__(self, weight, n_experts: Optional[int] = None, stream=None):
        if isinstance(weight, Fp8Matrix):
            if n_experts is None or n_experts < 1 or weight.rows % n_experts:
                raise ValueError(f"{weight.rows} rows do not divide into {n_experts} experts")
        else:
            if weight.dim() != 3 or (n_experts is not None and n_experts != weight.shape[0]):
                raise ValueError(f"weight must be [experts][n_out][k_in], got {tuple(weight.shape)}")
            n_experts = weight.shape[0]
            if weight.numel() == 0:
                raise ValueError(f"weight must not be empty, got {tuple(weight.shape)}")
            stream = _stream_of(weight.device, stream)
            # a copy of rows at several distances is made on the stream too
            rows = _on(weight.device, stream, lambda s: weight.reshape(-1, weight.shape[2]))
            if stream is not None:
                weight.record_stream(stream)
            weight = Fp8Matrix.quantize(rows, stream)
        super().__init__(weight, int(n_experts), weight.rows // int(n_experts), stream)

    def forward(self, x, offsets, out_dtype=None, out=None, stream=None):
        """x: [tokens][k_in] (or an Fp8Matrix) with the tokens of expert e in
        rows offsets[e] to offsets[e+1]; ``offsets`` an int32 CUDA tensor
        [experts + 1].  Rows that belong to no expert are left as they were in
        ``out`` (undefined without ``out``)."""
        import torch
        if offsets.dtype != torch.int32 or offsets.shape != (self.n_experts + 1,) or not offsets.is_contiguous():
            raise ValueError(f"offsets must be a contiguous int32 tensor of {self.n_experts + 1} entries")
        if offsets.device != self.device:
            raise ValueError(f"offsets are on {offsets.device}, the layer on {self.device}")
        return self._call(x, offsets, out_dtype, out, stream)
