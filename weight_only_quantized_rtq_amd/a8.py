"""8-bit activations: row operators that write codes with a scale per row, and
the product of such rows with the int8 and FP8 weights.

    rows, h = rms_norm(x, weight, residual=res, fmt="q8")   # A8Rows, x + res
    y = gemm_a8(rows, w)                                    # w: Q8Weight (or F8Weight with fmt="f8")

Argument marshalling only, as the rest of the binding. Activations are
float32, float16 or bfloat16 [M, K] tensors whose rows may lie in a wider
buffer (stride(1) == 1). Where `out`, `sum_out` or `y` is not given it is
allocated on the call's stream. `stream` runs the call on another stream than
the current one; ordering the inputs before it, and what uses the outputs
after it, is the caller's part, as everywhere in torch. Nothing here records
gradients.
"""
from __future__ import annotations

import contextlib
import struct
from dataclasses import dataclass

import torch

from . import FMT_F8, FMT_NONE, FMT_Q8, MAX_BLOCKS, F8Weight, Projection, Q8Weight, _check, _need, _stream, load_library

A8_MAX_K = 131071
_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_FMTS = {None: FMT_NONE, "q8": FMT_Q8, "f8": FMT_F8}
_Tensor = torch.Tensor
# what torch.cuda.current_device() and current_stream().cuda_stream come down to, where torch has a GPU
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_CODES = {FMT_Q8: torch.int8, FMT_F8: torch.uint8}


# rtq_proj_a8: fmt, N, K, y_dtype, x, x_scale, payload, scale, y, ldy, bias
_PROJ_A8 = struct.Struct("@iiiiPPPPPqP")


@dataclass
class A8Rows:
    """Rows of activations in 8 bits: row m holds scale[m] * codes[m]."""
    codes: torch.Tensor      # int8 [M, K], or uint8 [M, K]: E4M3 codes
    scale: torch.Tensor      # float32 [M]

    @property
    def M(self) -> int:
        return self.codes.shape[0]

    @property
    def K(self) -> int:
        return self.codes.shape[1]

    @property
    def fmt(self) -> int:
        return FMT_Q8 if self.codes.dtype == torch.int8 else FMT_F8

    def validate(self) -> None:
        codes, scale = self.codes, self.scale
        dev = _device_of(codes)
        _plain(codes, torch.int8 if codes.dtype == torch.int8 else torch.uint8, "codes", dev)
        _plain(scale, torch.float32, "scale", dev)
        shape = codes.shape
        if len(shape) != 2 or scale.shape != shape[:1]:
            raise ValueError(f"8-bit row shapes disagree: codes {tuple(shape)}, scale {tuple(scale.shape)}")

    def dequant(self) -> torch.Tensor:
        """The float32 values [M, K] the rows stand for."""
        codes = self.codes if self.codes.dtype == torch.int8 else self.codes.view(torch.float8_e4m3fn)
        return codes.to(torch.float32) * self.scale[:, None]


def _device_of(t) -> int:
    """The device of a call: the current one, which every tensor has to be on.
    What is no device tensor is refused by its own check, without asking for one."""
    return _current_device() if isinstance(t, _Tensor) and t.is_cuda else -2


def _plain(t, dtype, name: str, dev: int) -> int:
    """The pointer of a contiguous device tensor of a type (_need words the refusals)."""
    try:
        if t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _need(t, dtype, name)
    return t.data_ptr()


def _rows(t, name: str, dev: int, shape=None, dtype=None) -> int:
    """Checks a [M, K] tensor whose rows may be strided; returns the row stride."""
    try:
        have, kind = t.shape, t.dtype
        if t.is_contiguous() and t.get_device() == dev and \
                (kind in _DTYPES if dtype is None else kind is dtype) and \
                (len(have) == 2 if shape is None else have == shape):
            return have[1]
    except AttributeError:
        raise TypeError(f"{name} must be a torch.Tensor") from None
    if kind not in _DTYPES if dtype is None else kind != dtype:
        raise TypeError(f"{name} must be {dtype or 'float32, float16 or bfloat16'}, got {kind}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{dev}")
    if len(have) != 2 or (shape is not None and have != shape):
        raise ValueError(f"{name} must be {'[M, K]' if shape is None else list(shape)}, got {list(have)}")
    M, K = have
    ld, step = t.stride()
    if step != 1 and K > 1:
        raise ValueError(f"{name}: the elements of a row must be adjacent, stride {t.stride()}")
    if M <= 1:
        return K
    if ld < K:
        raise ValueError(f"{name}: rows overlap, stride {t.stride()}")
    return ld


def _launch_stream(stream, dev: int) -> int:
    """The raw stream of the call: the device's current one, or the given one."""
    return _current_stream(dev) if stream is None else _stream(stream)


def _on(stream):
    """The context new outputs are allocated in: the stream the call runs on."""
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream)))


def _fmt(fmt) -> int:
    try:
        return _FMTS[fmt]
    except KeyError:
        raise ValueError(f"unknown format {fmt!r}") from None


def _row_out(out, M: int, K: int, x, fmt: int, out_dtype, stream, dev: int):
    """The output of a row operator, checked or new: (object to return, its
    pointer, the scale's pointer, its dtype code)."""
    if fmt == FMT_NONE:
        if out is None:
            out_dtype = x.dtype if out_dtype is None else out_dtype
            if out_dtype not in (x.dtype, torch.float32):
                raise TypeError(f"out_dtype must be {x.dtype} or float32, got {out_dtype}")
            with _on(stream):
                out = torch.empty((M, K), dtype=out_dtype, device=x.device)
        elif not isinstance(out, torch.Tensor) or out.dtype not in (x.dtype, torch.float32) \
                or out_dtype not in (None, out.dtype):
            raise TypeError(f"out must be a {x.dtype} or float32 tensor (of out_dtype, where that is given)")
        p = _plain(out, out.dtype, "out", dev)
        if out.shape != (M, K):
            raise ValueError(f"out must be [{M}, {K}], got {list(out.shape)}")
        return out, p, None, _DTYPES[out.dtype]
    if out_dtype is not None:
        raise TypeError("out_dtype is for dense output (fmt None)")
    if out is None:
        with _on(stream):
            out = A8Rows(torch.empty((M, K), dtype=_CODES[fmt], device=x.device),
                         torch.empty((M,), dtype=torch.float32, device=x.device))
    elif not isinstance(out, A8Rows):
        raise TypeError("out must be an A8Rows")
    codes, scale = out.codes, out.scale
    p, s = _plain(codes, _CODES[fmt], "out.codes", dev), _plain(scale, torch.float32, "out.scale", dev)
    if codes.shape != (M, K) or scale.shape != (M,):
        raise ValueError(f"out must hold [{M}, {K}] codes and [{M}] scales, got {list(codes.shape)} and "
                         f"{list(scale.shape)}")
    return out, p, s, 0


def quantize_rows(x: torch.Tensor, fmt: str = "q8", out: A8Rows | None = None, stream=None) -> A8Rows:
    """Rows of x in 8 bits (rtq_quantize_rows): "q8" int8, "f8" E4M3."""
    lib = load_library()
    code = _fmt(fmt)
    if code == FMT_NONE:
        raise ValueError('quantize_rows writes "q8" or "f8"')
    dev = _device_of(x)
    ld = _rows(x, "x", dev)
    M, K = x.shape
    out, p, s, _ = _row_out(out, M, K, x, code, None, stream, dev)
    _check(lib.rtq_quantize_rows(x.data_ptr(), ld, _DTYPES[x.dtype], code, p, s, M, K, _launch_stream(stream, dev)))
    return out


def rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, residual: torch.Tensor | None = None,
             fmt: str | None = None, out=None, sum_out: torch.Tensor | None = None, out_dtype=None, stream=None):
    """Root-mean-square norm of x (or of h = x + residual) times the float32
    weight [K] (rtq_rms_norm). fmt "q8" / "f8" returns A8Rows, None a dense
    tensor of out_dtype (x's dtype, the default, or float32). With a residual
    the result is (output, h); sum_out holds h and may be x or residual itself."""
    lib = load_library()
    code = _fmt(fmt)
    dev = _device_of(x)
    ld = _rows(x, "x", dev)
    shape = x.shape
    M, K = shape
    wp = _plain(weight, torch.float32, "weight", dev)
    if weight.shape != (K,):
        raise ValueError(f"weight must be [{K}], got {list(weight.shape)}")
    rp = sp = None
    ldr = lds = 0
    if residual is not None:
        ldr = _rows(residual, "residual", dev, shape, x.dtype)
        if sum_out is None:
            with _on(stream):
                sum_out = torch.empty(shape, dtype=x.dtype, device=x.device)
        lds = _rows(sum_out, "sum_out", dev, shape, x.dtype)
        rp, sp = residual.data_ptr(), sum_out.data_ptr()
    elif sum_out is not None:
        raise ValueError("sum_out needs a residual")
    out, p, s, out_code = _row_out(out, M, K, x, code, out_dtype, stream, dev)
    _check(lib.rtq_rms_norm(x.data_ptr(), ld, rp, ldr, sp, lds, wp, eps, _DTYPES[x.dtype], code, out_code, p, s, M, K,
                            _launch_stream(stream, dev)))
    return out if residual is None else (out, sum_out)


def silu_mul(a: torch.Tensor, b: torch.Tensor, fmt: str | None = None, out=None, out_dtype=None, stream=None):
    """silu(a) * b (rtq_silu_mul): A8Rows for fmt "q8" / "f8", else dense."""
    lib = load_library()
    code = _fmt(fmt)
    dev = _device_of(a)
    lda = _rows(a, "a", dev)
    ldb = _rows(b, "b", dev, a.shape, a.dtype)
    M, K = a.shape
    out, p, s, out_code = _row_out(out, M, K, a, code, out_dtype, stream, dev)
    _check(lib.rtq_silu_mul(a.data_ptr(), lda, b.data_ptr(), ldb, _DTYPES[a.dtype], code, out_code, p, s, M, K,
                            _launch_stream(stream, dev)))
    return out


def _not_a_weight(w) -> TypeError:
    return TypeError(f"8-bit rows multiply a Q8Weight or an F8Weight, got {type(w).__name__}")


def _checked(x: A8Rows):
    """Rows of a call, checked: (fmt, M, K, the codes' pointer, the scales')."""
    if not isinstance(x, A8Rows):
        raise TypeError("x must be an A8Rows (quantize_rows, rms_norm or silu_mul with a format)")
    x.validate()
    codes = x.codes
    M, K = codes.shape
    return x.fmt, M, K, codes.data_ptr(), x.scale.data_ptr()


def _pack(rows, w, y: torch.Tensor, bias, dev: int) -> bytes:
    """One descriptor; `rows` is what _checked() gave."""
    if not isinstance(w, (Q8Weight, F8Weight)):
        raise _not_a_weight(w)
    x_fmt, M, K, xp, xsp = rows
    payload, fmt = w.payload, w.fmt
    if fmt != x_fmt:
        raise TypeError(f"{_CODES[x_fmt]} rows do not multiply a {type(w).__name__}")
    wp = _plain(payload, _CODES[fmt], "payload", dev)
    shape = payload.shape
    if len(shape) != 2 or shape[1] != K:
        raise ValueError(f"x is [{M}, {K}], the weight {list(shape)}")
    N = shape[0]
    sp = bp = 0
    if fmt == FMT_Q8:
        scale = w.scale
        sp = _plain(scale, torch.float32, "scale", dev)
        if scale.shape != (N,):
            raise ValueError(f"int8 weight shapes disagree: payload {list(shape)}, scale {list(scale.shape)}")
    ldy = _rows(y, "y", dev, (M, N))
    if bias is not None:
        bp = _plain(bias, torch.float32, "bias", dev)
        if bias.shape != (N,):
            raise ValueError(f"bias {list(bias.shape)} does not match N={N}")
    return _PROJ_A8.pack(fmt, N, K, _DTYPES[y.dtype], xp, xsp, wp, sp, y.data_ptr(), ldy, bp)


def gemm_a8(x: A8Rows, w, y: torch.Tensor | None = None, bias: torch.Tensor | None = None, out_dtype=None,
            stream=None) -> torch.Tensor:
    """y = x . W^T (+ bias) for 8-bit rows and a Q8Weight or F8Weight of the same
    format (rtq_gemm_a8). y is float32 unless out_dtype (or y itself) says otherwise."""
    lib = load_library()
    if not isinstance(w, (Q8Weight, F8Weight)):
        raise _not_a_weight(w)
    if y is None:
        out_dtype = torch.float32 if out_dtype is None else out_dtype
        if out_dtype not in _DTYPES:
            raise TypeError(f"out_dtype must be float32, float16 or bfloat16, got {out_dtype}")
    rows = _checked(x)
    if y is None:
        with _on(stream):
            y = torch.empty((rows[1], w.N), dtype=out_dtype, device=x.codes.device)
    elif out_dtype not in (None, y.dtype):
        raise TypeError(f"y is {y.dtype}, out_dtype {out_dtype}")
    dev = _device_of(y)
    d = _pack(rows, w, y, bias, dev)
    _check(lib.rtq_gemm_a8(d, rows[1], _launch_stream(stream, dev)))
    return y


def project_a8(projections: list[Projection], stream=None) -> None:
    """Several projections of 8-bit rows in one call (rtq_project_a8): each
    Projection's x is an A8Rows, all of them with the same number of rows, and
    its y a float32, float16 or bfloat16 tensor that may be columns of a wider one."""
    lib = load_library()
    if not 1 <= len(projections) <= MAX_BLOCKS * 8:
        raise ValueError(f"1..{MAX_BLOCKS * 8} projections per call, got {len(projections)}")
    dev, known, M, packed = _device_of(projections[0].y), None, None, []
    for p in projections:
        if p.x is not known:
            known, rows = p.x, _checked(p.x)
            if M not in (None, rows[1]):
                raise ValueError(f"the projections of one call share M: {rows[1]} and {M}")
            M = rows[1]
        packed.append(_pack(rows, p.weight, p.y, p.bias, dev))
    _check(lib.rtq_project_a8(b"".join(packed), len(packed), M, _launch_stream(stream, dev)))


def ffn_a8(x: torch.Tensor, weight: torch.Tensor, w1, w3, w2, eps: float = 1e-6,
           residual: torch.Tensor | None = None, stream=None):
    """A gated FFN on 8-bit rows: with n = rms_norm(x (+ residual), weight),
    (silu(n . W1^T) * (n . W3^T)) . W2^T, every product on 8-bit rows of the
    weights' format. Returns y [M, w2.N] in x's dtype, or (y, x + residual)."""
    for w in (w1, w3, w2):
        if not isinstance(w, (Q8Weight, F8Weight)):
            raise _not_a_weight(w)
        if w.fmt != w1.fmt:
            raise TypeError("the weights of one FFN share a format")
    if (w3.N, w3.K, w2.K) != (w1.N, w1.K, w1.N):
        raise ValueError(f"FFN weight shapes disagree: w1 [{w1.N}, {w1.K}], w3 [{w3.N}, {w3.K}], w2 [{w2.N}, {w2.K}]")
    fmt = "q8" if w1.fmt == FMT_Q8 else "f8"
    rows = rms_norm(x, weight, eps, residual=residual, fmt=fmt, stream=stream)
    h = None
    if residual is not None:
        rows, h = rows
    with _on(stream):
        ab = torch.empty((x.shape[0], w1.N + w3.N), dtype=x.dtype, device=x.device)
    a, b = ab[:, :w1.N], ab[:, w1.N:]
    project_a8([Projection(w1, rows, a), Projection(w3, rows, b)], stream)
    y = gemm_a8(silu_mul(a, b, fmt=fmt, stream=stream), w2, out_dtype=x.dtype, stream=stream)
    return y if h is None else (y, h)
