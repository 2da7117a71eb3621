"""The operators on 8-bit activations refuse bad arguments on the host, before
any HIP call: nothing here launches a kernel or needs a GPU."""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")

import weight_only_quantized_rtq_amd as rtq  # noqa: E402

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_FORMAT, ERR_HIP, ERR_OVERLAP = range(7)
A, B, C, D, E = (0x7f0000000000 + (i << 36) for i in range(5))      # device addresses, never dereferenced


@pytest.fixture(scope="module")
def lib():
    return rtq.load_library()


def quant(lib, x=A, ldx=512, dtype=0, fmt=2, codes=B, scale=C, M=4, K=512):
    return lib.rtq_quantize_rows(x, ldx, dtype, fmt, codes, scale, M, K, None)


def norm(lib, x=A, ldx=512, r=None, ldr=0, s=None, lds=0, w=D, eps=1e-6, dtype=0, fmt=2, out_dtype=0, out=B, scale=C,
         M=4, K=512):
    return lib.rtq_rms_norm(x, ldx, r, ldr, s, lds, w, eps, dtype, fmt, out_dtype, out, scale, M, K, None)


def silu(lib, a=A, lda=512, b=D, ldb=512, dtype=0, fmt=2, out_dtype=0, out=B, scale=C, M=4, K=512):
    return lib.rtq_silu_mul(a, lda, b, ldb, dtype, fmt, out_dtype, out, scale, M, K, None)


@pytest.mark.parametrize("call", [quant, norm, silu])
def test_row_operators_share_their_refusals(lib, call):
    assert call(lib, M=0) == OK
    assert call(lib, M=-1) == ERR_SHAPE and call(lib, M=2 ** 30) == ERR_SHAPE
    assert call(lib, K=0) == ERR_SHAPE and call(lib, K=2 ** 30) == ERR_SHAPE
    assert call(lib, M=2 ** 29, K=2 ** 29) == ERR_SHAPE
    assert call(lib, dtype=3) == ERR_FORMAT and call(lib, dtype=-1) == ERR_FORMAT
    assert call(lib, fmt=1) == ERR_FORMAT and call(lib, fmt=9) == ERR_FORMAT
    assert call(lib, scale=None) == ERR_NULL
    assert call(lib, scale=C + 2) == ERR_ALIGN
    out = "codes" if call is quant else "out"
    assert call(lib, **{out: None}) == ERR_NULL
    assert call(lib, **{out: C - 16}) == ERR_OVERLAP            # codes run into the scales
    assert call(lib, **{out: A + 4}) == ERR_OVERLAP
    assert call(lib, scale=A) == ERR_OVERLAP
    first = "a" if call is silu else "x"
    ld = "lda" if call is silu else "ldx"
    assert call(lib, **{first: None}) == ERR_NULL
    assert call(lib, **{first: A + 2}) == ERR_ALIGN
    assert call(lib, **{first: A + 1, "dtype": 2}) == ERR_ALIGN
    assert call(lib, **{ld: 511}) == ERR_SHAPE
    assert call(lib, **{ld: 2 ** 62}) == ERR_SHAPE
    # an output between an input's rows
    assert call(lib, **{ld: 4096, out: A + 4 * 600}) == ERR_OVERLAP


def test_quantizer_takes_no_dense_output(lib):
    assert quant(lib, fmt=0) == ERR_FORMAT


def test_norm_refusals(lib):
    for eps in (0.0, -1e-6, math.inf, math.nan):
        assert norm(lib, eps=eps) == ERR_SHAPE, eps
    assert norm(lib, w=None) == ERR_NULL
    assert norm(lib, w=D + 2) == ERR_ALIGN
    assert norm(lib, r=E, ldr=512) == ERR_NULL and norm(lib, s=E, lds=512) == ERR_NULL
    assert b"come together" in lib.rtq_last_error()
    both = dict(r=E, ldr=512, s=E + (1 << 30), lds=512)
    assert norm(lib, **{**both, "ldr": 100}) == ERR_SHAPE
    assert norm(lib, **{**both, "lds": 100}) == ERR_SHAPE
    assert norm(lib, **{**both, "s": E + 4}) == ERR_OVERLAP         # shifted against the residual
    assert norm(lib, **{**both, "s": E, "lds": 1024}) == ERR_OVERLAP
    assert norm(lib, **{**both, "s": A + 2048}) == ERR_OVERLAP
    assert norm(lib, **{**both, "s": D}) == ERR_OVERLAP
    assert norm(lib, **{**both, "out": E + (1 << 30) + 64}) == ERR_OVERLAP
    assert norm(lib, fmt=0, scale=C) == ERR_FORMAT                  # dense takes no scale
    assert norm(lib, fmt=0, scale=None, dtype=2, out_dtype=1) == ERR_FORMAT
    assert norm(lib, fmt=0, scale=None, out=B + 2) == ERR_ALIGN


def test_silu_refusals(lib):
    assert silu(lib, b=None) == ERR_NULL
    assert silu(lib, ldb=7) == ERR_SHAPE
    assert silu(lib, out=D) == ERR_OVERLAP
    assert silu(lib, fmt=0, scale=None, dtype=1, out_dtype=2) == ERR_FORMAT


class ProjA8(ctypes.Structure):
    """rtq_proj_a8 as the header lays it out."""
    _fields_ = [("fmt", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32), ("y_dtype", ctypes.c_int32),
                ("x", ctypes.c_void_p), ("x_scale", ctypes.c_void_p), ("payload", ctypes.c_void_p),
                ("scale", ctypes.c_void_p), ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64),
                ("bias", ctypes.c_void_p)]


def proj(fmt=2, N=64, K=128, y_dtype=0, x=A, sx=B, w=C, sw=B + (1 << 20), y=D, ldy=None, bias=None):
    return ProjA8(fmt, N, K, y_dtype, x, sx, w, sw, y, N if ldy is None else ldy, bias)


def test_binding_packs_the_descriptor():
    from weight_only_quantized_rtq_amd.a8 import _PROJ_A8
    d = ProjA8.from_buffer_copy(_PROJ_A8.pack(2, 64, 128, 1, A, B, C, 0, D, 70, E))
    assert _PROJ_A8.size == ctypes.sizeof(ProjA8)
    assert (d.fmt, d.N, d.K, d.y_dtype, d.x, d.x_scale, d.payload, d.scale, d.y, d.ldy, d.bias) == (
        2, 64, 128, 1, A, B, C, None, D, 70, E)


def project(lib, *projs, M=4, n=None):
    arr = (ProjA8 * len(projs))(*projs)
    return lib.rtq_project_a8(arr, len(projs) if n is None else n, M, None)


def test_projection_refusals(lib):
    assert lib.rtq_project_a8(None, 1, 4, None) == ERR_NULL
    assert lib.rtq_gemm_a8(None, 4, None) == ERR_NULL
    assert project(lib, proj(), n=0) == ERR_SHAPE and project(lib, proj(), n=513) == ERR_SHAPE
    assert project(lib, proj(), M=-1) == ERR_SHAPE and project(lib, proj(), M=2 ** 30) == ERR_SHAPE
    assert project(lib, proj(), M=0) == OK
    assert lib.rtq_gemm_a8(ctypes.byref(proj()), 0, None) == OK
    for fmt in (0, 1, 4):
        assert project(lib, proj(fmt=fmt)) == ERR_FORMAT
    assert project(lib, proj(y_dtype=3)) == ERR_FORMAT
    for bad in (dict(N=0), dict(K=0), dict(K=131072), dict(N=2 ** 30), dict(ldy=63), dict(ldy=2 ** 60)):
        assert project(lib, proj(**bad)) == ERR_SHAPE, bad
    assert project(lib, proj(N=2 ** 29), M=2 ** 20) == ERR_SHAPE
    for name in ("x", "sx", "w", "sw", "y"):
        assert project(lib, proj(**{name: None})) == ERR_NULL, name
    for bad in (dict(sx=B + 2), dict(sw=B + 1), dict(bias=E + 2), dict(y=D + 2), dict(y=D + 1, y_dtype=2)):
        assert project(lib, proj(**bad)) == ERR_ALIGN, bad
    for bad in (dict(y=A), dict(y=B), dict(y=C + 4), dict(bias=D + 8)):
        assert project(lib, proj(**bad)) == ERR_OVERLAP, bad
    # the second of two
    assert project(lib, proj(), proj(y=D + (1 << 20), K=0)) == ERR_SHAPE
    assert b"projection 1" in lib.rtq_last_error()


def test_outputs_side_by_side(lib):
    """Columns of one buffer are disjoint; anything else that shares bytes is refused. The last
    projection is refused for its format, so nothing is launched where the outputs are fine."""
    row = 256
    a = proj(N=64, ldy=row)

    def status(y, N=64, ldy=row, M=4):
        return project(lib, a, proj(y=y, N=N, ldy=ldy), M=M)

    assert status(D + 63 * 4) == ERR_OVERLAP                         # one column shared
    assert status(D + 200 * 4) == ERR_OVERLAP                        # runs into the next row's first columns
    assert status(D + 64 * 4, ldy=row + 64) == ERR_OVERLAP           # other strides
    assert status(D) == ERR_OVERLAP
    # an input in the buffer of the outputs
    assert project(lib, a, proj(y=D + 64 * 4, ldy=row, bias=D + 4 * row * 3)) == ERR_OVERLAP


def rows(M=4, K=128, dtype=torch.int8):
    return rtq.A8Rows(torch.zeros(M, K, dtype=dtype), torch.zeros(M))


def test_binding_refuses_host_tensors_and_types():
    x, w = torch.zeros(4, 128), torch.ones(128)
    q8 = rtq.Q8Weight(torch.zeros(64, 128, dtype=torch.int8), torch.zeros(64))
    for call in (lambda: rtq.quantize_rows(x), lambda: rtq.rms_norm(x, w), lambda: rtq.silu_mul(x, x),
                 lambda: rtq.gemm_a8(rows(), q8),
                 lambda: rtq.ffn_a8(x, w, q8, q8, rtq.Q8Weight(torch.zeros(128, 64, dtype=torch.int8), torch.zeros(128)))):
        with pytest.raises(ValueError, match="device tensor"):
            call()
    with pytest.raises(TypeError):
        rtq.quantize_rows(x.double())
    with pytest.raises(TypeError):
        rtq.quantize_rows([1.0])
    with pytest.raises(ValueError, match="unknown format"):
        rtq.quantize_rows(x, "q4")
    with pytest.raises(ValueError):
        rtq.quantize_rows(x, None)
    with pytest.raises(TypeError, match="A8Rows"):
        rtq.gemm_a8(x, q8)
    with pytest.raises(TypeError, match="Q4Weight"):
        rtq.gemm_a8(rows(), rtq.Q4Weight(torch.zeros(64, 64, dtype=torch.uint8), torch.zeros(64, 4, 2).half()))
    with pytest.raises(TypeError, match="Q4Weight"):
        rtq.ffn_a8(x, w, rtq.Q4Weight(torch.zeros(64, 64, dtype=torch.uint8), torch.zeros(64, 4, 2).half()), q8, q8)
    with pytest.raises(ValueError, match="disagree"):
        rtq.ffn_a8(x, w, q8, q8, rtq.Q8Weight(torch.zeros(128, 60, dtype=torch.int8), torch.zeros(128)))
    f8 = rtq.F8Weight(torch.zeros(64, 128, dtype=torch.uint8))
    with pytest.raises(TypeError, match="share a format"):
        rtq.ffn_a8(x, w, q8, f8, q8)
    with pytest.raises(ValueError):
        rtq.project_a8([])
    with pytest.raises(TypeError, match="out_dtype"):
        rtq.gemm_a8(rows(), q8, out_dtype=torch.float64)
