"""GPU tests of the product of 8-bit rows with 8-bit weights, of the grouped
call, and of the operators in a chain, against the fp64 oracle."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
import weight_only_quantized_rtq_amd as rtq  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def codes(shape, fmt, g):
    """int8 codes over the whole range; E4M3 codes without NaN, of every exponent."""
    if fmt == "q8":
        return torch.randint(-127, 128, shape, generator=g, dtype=torch.int8)
    c = torch.randint(0, 127, shape, generator=g, dtype=torch.uint8)
    return c | (torch.randint(0, 2, shape, generator=g, dtype=torch.uint8) << 7)


def make(M, N, K, fmt, seed, bias=True):
    g = torch.Generator().manual_seed(seed)
    x = rtq.A8Rows(codes((M, K), fmt, g), torch.rand(M, generator=g) + 0.01)
    w = codes((N, K), fmt, g)
    w = rtq.Q8Weight(w, torch.rand(N, generator=g) + 0.01) if fmt == "q8" else rtq.F8Weight(w)
    return x, w, torch.randn(N, generator=g) * 100 if bias else None


def dev(x, w, bias):
    x = rtq.A8Rows(x.codes.to(DEV), x.scale.to(DEV))
    w = rtq.Q8Weight(w.payload.to(DEV), w.scale.to(DEV)) if w.fmt == rtq.FMT_Q8 else rtq.F8Weight(w.payload.to(DEV))
    return x, w, None if bias is None else bias.to(DEV)


def check(y, x, w, bias, rows=None):
    torch.cuda.synchronize()
    fmt = "q8" if w.fmt == rtq.FMT_Q8 else "f8"
    pick = slice(None) if rows is None else rows
    sw = w.scale.cpu().numpy() if fmt == "q8" else None
    want, size = oracle.a8.gemm_a8(x.codes.cpu().numpy()[pick], x.scale.cpu().numpy()[pick], w.payload.cpu().numpy(), sw,
                                   None if bias is None else bias.cpu().numpy(), fmt)
    got = y.double().cpu().numpy()[pick]
    info = torch.finfo(y.dtype)
    u = 2.0 ** -24
    product = want if bias is None else want - bias.cpu().numpy().astype(np.float64)
    # int8: the exact sum to fp32, the scales' product, their product; E4M3: K - 1 additions of exact
    # products in any order, each off by a whole step where the matrix unit truncates, and the scale;
    # for a 16-bit y also 7 * 2^-13 of sum|x w|, the fixed-point groups of the FP8 instructions.
    # Then the bias and y's own rounding.
    tol = np.abs(product) * 3 * u if fmt == "q8" else size * (x.K + 1) * 2 * u
    if fmt == "f8" and y.dtype != torch.float32:
        tol = tol + size * 7 * 2.0 ** -13
    if bias is not None:
        tol = tol + np.abs(want) * u
    tol = tol * 1.01 + np.abs(want) * info.eps / 2 + float(info.tiny) * info.eps
    with np.errstate(all="ignore"):
        fits = np.abs(want) <= float(info.max)
        assert np.array_equal(np.isnan(got), np.isnan(want))
        assert np.all((np.abs(got - want) <= tol)[fits & ~np.isnan(want)])
    if fmt == "f8" and not np.isnan(want).any() and fits.all():
        # As a whole: K / 32 additions to a sum that grows as the root of its length, each truncating
        # at most 2^-23 of it, come to (2/3) (K / 32) 2^-23 of the result even if all point one way;
        # 2^-22 for the rest. The FP8 groups' truncation on codes of every exponent: 5e-5 measured.
        whole = (x.K / 48 * 2 + 4) * u
        assert oracle.rel_fro(got, want) <= (whole if y.dtype == torch.float32 else whole + 1e-4 + info.eps)


SHAPES = [
    (1, 1, 1), (1, 16, 16), (1, 512, 512), (1, 2048, 512), (1, 1000, 4096), (2, 17, 33), (3, 512, 2048), (4, 100, 15),
    (7, 65, 127), (8, 512, 512), (15, 130, 129), (16, 2048, 512), (17, 64, 256), (31, 31, 31), (32, 512, 2048),
    (33, 256, 1024), (40, 1000, 1008), (64, 64, 64), (65, 65, 65), (80, 512, 512), (80, 2048, 512), (80, 512, 2048),
    (96, 257, 2051), (128, 128, 128), (129, 300, 144), (200, 513, 4112), (255, 255, 255), (256, 256, 256),
    (257, 259, 512), (300, 2000, 640), (500, 384, 16), (512, 512, 8), (1000, 1024, 1024), (1025, 130, 272),
    (2048, 768, 512), (4100, 500, 192),
]


@pytest.mark.parametrize("fmt", ["q8", "f8"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm(M, N, K, fmt):
    for dtype, bias in ((torch.float32, True), (torch.bfloat16, False), (torch.float16, True)):
        x, w, b = dev(*make(M, N, K, fmt, M + N + K, bias))
        if dtype == torch.float16:
            x.scale.mul_(1e-4)
        y = rtq.gemm_a8(x, w, bias=b, out_dtype=dtype)
        assert y.dtype == dtype
        check(y, x, w, b)


# K in every remainder of stages over teams, with whole and partial last stages; few tiles and many
TEAM_SHAPES = [(150, 2000, 1040), (300, 520, 1152), (77, 1999, 1280), (150, 2000, 1300), (300, 520, 1153), (77, 1999, 1535),
               (300, 520, 1663), (500, 2040, 1040), (500, 2040, 1280), (490, 2030, 1026), (500, 2040, 1285), (490, 2030, 1409),
               (500, 2040, 1551), (1400, 2000, 1025), (1400, 2000, 1283), (1400, 1990, 2049)]


@pytest.mark.parametrize("fmt", ["q8", "f8"])
@pytest.mark.parametrize("M,N,K", TEAM_SHAPES)
def test_sums_of_several_teams(M, N, K, fmt):
    for dtype, bias in ((torch.float32, True), (torch.bfloat16, False)):
        x, w, b = dev(*make(M, N, K, fmt, M + N + K, bias))
        y = rtq.gemm_a8(x, w, bias=b, out_dtype=dtype)
        check(y, x, w, b)
        assert torch.equal(y, rtq.gemm_a8(x, w, bias=b, out_dtype=dtype))


@pytest.mark.parametrize("M", [60, 150, 300, 700])
def test_teams_of_long_and_short_sums_in_one_call(M):
    """A launch that splits a long K has projections of one stage, fewer than its teams, beside it."""
    for fmt in ("q8", "f8"):
        for Ks in ((65, 2049, 130), (64, 2048, 128, 512)):
            projs = []
            for i, K in enumerate(Ks):
                x, w, b = dev(*make(M, 200 + 8 * i, K, fmt, M + K, i % 2 == 0))
                projs.append(rtq.Projection(w, x, torch.empty(M, w.N, device=DEV), b))
            rtq.project_a8(projs)
            for p in projs:
                check(p.y, p.x, p.weight, p.bias)


@pytest.mark.parametrize("M,N,K", [(1, 64, 131071), (20, 40, 131056), (130, 70, 131071), (300, 300, 100000)])
def test_longest_sums(M, N, K):
    """The largest codes over the longest K: int32 holds the sum."""
    for code in (-128, 127):
        x = rtq.A8Rows(torch.full((M, K), -128, dtype=torch.int8, device=DEV), torch.ones(M, device=DEV))
        w = rtq.Q8Weight(torch.full((N, K), code, dtype=torch.int8, device=DEV), torch.ones(N, device=DEV))
        want = np.float32(-128 * code * K)
        assert (rtq.gemm_a8(x, w).cpu().numpy() == want).all()
    x, w, b = dev(*make(M, N, K, "f8", K))
    check(rtq.gemm_a8(x, w, bias=b), x, w, b)


@pytest.mark.parametrize("fmt", ["q8", "f8"])
@pytest.mark.parametrize("M", [1, 5, 16, 48, 80, 260, 700])
def test_strided_and_misaligned(M, fmt):
    """y as columns of a wider buffer, codes at odd addresses; what lies around y stays."""
    N, K = 200, 528
    x, w, b = dev(*make(M, N, K, fmt, M))
    for off in (0, 1, 4, 8):
        store = torch.zeros(M * K + 64, dtype=x.codes.dtype, device=DEV)
        xc = store[off:off + M * K].view(M, K).copy_(x.codes)
        wstore = torch.zeros(N * K + 64, dtype=w.payload.dtype, device=DEV)
        wc = wstore[off:off + N * K].view(N, K).copy_(w.payload)
        w2 = rtq.Q8Weight(wc, w.scale) if fmt == "q8" else rtq.F8Weight(wc)
        for dtype in (torch.float32, torch.bfloat16):
            buf = torch.full((M + 2, N + 9), 7.0, dtype=dtype, device=DEV)
            y = buf[1:M + 1, 3:3 + N]
            rtq.gemm_a8(rtq.A8Rows(xc, x.scale), w2, y=y, bias=b)
            check(y, x, w, b)
            buf[1:M + 1, 3:3 + N] = 7
            assert (buf == 7).all()


@pytest.mark.parametrize("M", [1, 16, 80, 333])
def test_nan_rows_and_zero_rows(M):
    for fmt in ("q8", "f8"):
        v = torch.randn(M, 512, device=DEV)
        v[M // 2, 3] = float("nan")
        v[0] = 0
        if M == 1:
            v[0, 0] = float("inf")
        x = rtq.quantize_rows(v, fmt)
        _, w, b = dev(*make(1, 96, 512, fmt, 1))
        y = rtq.gemm_a8(x, w, bias=b).cpu()
        bad = torch.isnan(y).all(1)
        assert bad.nonzero().flatten().tolist() == [M // 2] and torch.isfinite(y[~bad]).all()
        if M > 1:
            assert torch.equal(y[0], b.cpu())
    # a NaN weight code reaches its own column alone
    x, w, _ = dev(*make(M, 96, 520, "f8", 2))
    w.payload[5, 519] = 0x7F
    y = rtq.gemm_a8(x, w).cpu()
    assert torch.isnan(y[:, 5]).all() and torch.isfinite(y[:, :5]).all() and torch.isfinite(y[:, 6:]).all()


@pytest.mark.parametrize("M", [1, 8, 80, 600])
def test_project_equals_single_calls(M):
    """Both formats, shared and separate rows, several widths, more projections than one launch holds."""
    projs, singles = [], []
    for i in range(21):
        fmt = "q8" if i % 3 else "f8"
        N, K = [(512, 512), (70, 512), (512, 2048), (33, 65), (2048, 512)][i % 5]
        x, w, b = dev(*make(M, N, K, fmt, 100 + i, i % 2 == 0))
        y = torch.full((M, N), float("nan"), dtype=[torch.float32, torch.bfloat16, torch.float16][i % 3], device=DEV)
        projs.append(rtq.Projection(w, x, y, b))
        singles.append(rtq.gemm_a8(x, w, bias=b, out_dtype=y.dtype))
    rtq.project_a8(projs)
    torch.cuda.synchronize()
    for p, s in zip(projs, singles):
        # the grouped call may take another tile; int8 sums are the same in every order
        if p.weight.fmt == rtq.FMT_Q8:
            assert torch.equal(p.y, s)
        check(p.y, p.x, p.weight, p.bias)


def test_outputs_in_one_buffer():
    M, K = 80, 512
    buf = torch.full((M, 4 * 512 + 3), 9.0, device=DEV)
    x, w0, _ = dev(*make(M, 512, K, "q8", 1))
    projs = []
    for i in range(4):
        _, w, b = dev(*make(1, 512, K, "q8", 10 + i))
        projs.append(rtq.Projection(w, x, buf[:, 512 * i:512 * (i + 1)], b))
    rtq.project_a8(projs)
    for p in projs:
        check(p.y, x, p.weight, p.bias)
    assert (buf[:, 2048:] == 9).all()


def test_empty_batch_and_repeat():
    x, w, b = dev(*make(3, 64, 128, "q8", 1))
    empty = rtq.A8Rows(x.codes[:0], x.scale[:0])
    assert rtq.gemm_a8(empty, w, bias=b).shape == (0, 64)
    for M, N, K in ((1, 1000, 4096), (80, 512, 2048), (512, 512, 512), (3000, 1000, 1000)):
        for fmt in ("q8", "f8"):
            x, w, b = dev(*make(M, N, K, fmt, 2))
            first = rtq.gemm_a8(x, w, bias=b)
            for _ in range(3):
                assert torch.equal(first, rtq.gemm_a8(x, w, bias=b))


def test_offsets_past_32_bits():
    """x, weight and y each past 2^32 bytes, checked on rows at the far ends."""
    K = 512
    M = (1 << 32) // K + 300
    g = torch.Generator(device=DEV).manual_seed(3)
    x = rtq.A8Rows(torch.randint(-127, 128, (M, K), generator=g, device=DEV, dtype=torch.int8), torch.rand(M, device=DEV))
    _, w, b = dev(*make(1, 160, K, "q8", 4))
    y = rtq.gemm_a8(x, w, bias=b)
    rows = torch.tensor([0, 1, M // 2, (1 << 32) // K - 1, (1 << 32) // K, M - 1], device=DEV)
    part = rtq.A8Rows(x.codes[rows].contiguous(), x.scale[rows].contiguous())
    check(y[rows], part, w, b)
    assert torch.equal(y[-200:], rtq.gemm_a8(rtq.A8Rows(x.codes[-200:], x.scale[-200:]), w, bias=b))
    del y
    wide = rtq.Q8Weight(x.codes, x.scale)                   # [M, K] as a weight of M outputs
    few, _, _ = dev(*make(130, 1, K, "q8", 5))
    for m in (130, 3):
        rows_x = rtq.A8Rows(few.codes[:m], few.scale[:m])
        y = rtq.gemm_a8(rows_x, wide)
        tail = rtq.Q8Weight(x.codes[-77:], x.scale[-77:])
        assert torch.equal(y[:, -77:].contiguous(), rtq.gemm_a8(rows_x, tail))
        check(y[:, -77:], rows_x, tail, None)


def oracle_ffn(x, res, nw, ws, fmt, dtype):
    """The chain with each stage's own rounding, stage by stage in fp64."""
    h, p, r = oracle.a8.rms_norm_parts(x, res, nw, 1e-6, dtype)
    c, s = oracle.a8.codes_and_scale(p, r, fmt)
    pay = [w.payload.cpu().numpy() for w in ws]
    sc = [w.scale.cpu().numpy() if fmt == "q8" else None for w in ws]
    a, _ = oracle.a8.gemm_a8(c, s, pay[0], sc[0], None, fmt)
    b, _ = oracle.a8.gemm_a8(c, s, pay[1], sc[1], None, fmt)
    a, b = (oracle.a8.round_to(v, dtype) for v in (a, b))
    c, s = oracle.a8.codes_and_scale(oracle.a8.silu_mul(a, b), 1.0, fmt)
    y, _ = oracle.a8.gemm_a8(c, s, pay[2], sc[2], None, fmt)
    return h, y


@pytest.mark.parametrize("fmt", ["q8", "f8"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("M", [1, 16, 80, 500])
def test_ffn_chain(M, dtype, fmt):
    T = torch.float32 if dtype == "fp32" else torch.bfloat16
    g = torch.Generator().manual_seed(M)
    x, res = (torch.randn(M, 512, generator=g).to(T).to(DEV) for _ in range(2))
    nw = (1 + 0.1 * torch.randn(512, generator=g)).to(DEV)
    ws = [rtq.quantize((torch.randn(n, k, generator=g) * 0.02).to(DEV), fmt) for n, k in ((2048, 512), (2048, 512), (512, 2048))]
    y, h = rtq.ffn_a8(x, nw, *ws, residual=res)
    assert y.dtype == T
    want_h, want = oracle_ffn(x.float().cpu().numpy(), res.float().cpu().numpy(), nw.cpu().numpy(), ws, fmt, dtype)
    assert np.array_equal(h.float().cpu().numpy(), want_h)
    # One difference is possible between the stages: a stage's fp32 roundings move a value of a or b
    # across a rounding border of its type or of the codes. A code is off by one step of about
    # 1 / 127 (2^-4 for E4M3) then, in few of the 2048 terms; dense arithmetic is far closer.
    err = oracle.rel_fro(y.float().cpu().numpy(), want)
    assert err <= 2e-3 + torch.finfo(T).eps
    assert torch.equal(rtq.ffn_a8(x, nw, *ws, residual=res)[0], y)
    no_res = rtq.ffn_a8(h, nw, *ws)
    assert torch.equal(no_res, y)


def test_other_stream_and_graph():
    """The chain on a stream of its own, two chains at once, and captured: replays with new
    inputs, eager work and synchronizations between them, each equal to the eager result."""
    M = 80
    g = torch.Generator().manual_seed(7)
    nw = torch.ones(512, device=DEV)
    ws = [rtq.quantize((torch.randn(n, k, generator=g) * 0.02).to(DEV), "q8") for n, k in ((2048, 512), (2048, 512), (512, 2048))]
    inputs = [torch.randn(M, 512, generator=g).to(DEV) for _ in range(4)]
    res = torch.randn(M, 512, generator=g).to(DEV)
    want = [rtq.ffn_a8(x, nw, *ws, residual=res) for x in inputs]
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(2)]
    got = [rtq.ffn_a8(x, nw, *ws, residual=res, stream=side[i % 2]) for i, x in enumerate(inputs)]
    torch.cuda.synchronize()
    for (y, h), (wy, wh) in zip(got, want):
        assert torch.equal(y, wy) and torch.equal(h, wh)
    x = inputs[0].clone()
    with torch.cuda.stream(side[0]):
        rtq.ffn_a8(x, nw, *ws, residual=res)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, h = rtq.ffn_a8(x, nw, *ws, residual=res)
    for i in (1, 2, 3, 0, 2):
        x.copy_(inputs[i])
        graph.replay()
        eager = rtq.ffn_a8(inputs[(i + 1) % 4], nw, *ws, residual=res)
        torch.cuda.synchronize()
        assert torch.equal(y, want[i][0]) and torch.equal(h, want[i][1])
        assert torch.equal(eager[0], want[(i + 1) % 4][0])


def test_refusals_on_the_device():
    x, w, b = dev(*make(4, 64, 128, "q8", 1))
    xf, wf, _ = dev(*make(4, 64, 128, "f8", 1))
    for call in (lambda: rtq.gemm_a8(x, wf), lambda: rtq.gemm_a8(xf, w), lambda: rtq.gemm_a8(x.codes, w)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError):
        rtq.gemm_a8(rtq.A8Rows(x.codes[:, :64].contiguous(), x.scale), w)
    with pytest.raises(ValueError):
        rtq.gemm_a8(rtq.A8Rows(x.codes[:, ::2], x.scale), w)
    with pytest.raises(ValueError):
        rtq.gemm_a8(rtq.A8Rows(x.codes, x.scale[:3]), w)
    with pytest.raises(ValueError):
        rtq.gemm_a8(x, w, y=torch.empty(4, 63, device=DEV))
    with pytest.raises(TypeError):
        rtq.gemm_a8(x, w, y=torch.empty(4, 64, device=DEV), out_dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        rtq.gemm_a8(x, w, bias=b[:63])
    y = torch.empty(4, 64, device=DEV)
    with pytest.raises(rtq.RtqError) as e:
        rtq.project_a8([rtq.Projection(w, x, y), rtq.Projection(w, x, y)])
    assert e.value.status == 6
    other, _, _ = dev(*make(5, 64, 128, "q8", 1))
    with pytest.raises(ValueError, match="share M"):
        rtq.project_a8([rtq.Projection(w, x, y), rtq.Projection(w, other, torch.empty(5, 64, device=DEV))])


def test_more_columns_than_one_launch_holds():
    """N past the columns of one launch, alone and beside a small task; the pieces meet at column 2^23."""
    N, K = (1 << 23) + 37, 16
    g = torch.Generator(device=DEV).manual_seed(8)
    w = rtq.Q8Weight(torch.randint(-127, 128, (N, K), generator=g, device=DEV, dtype=torch.int8),
                     torch.rand(N, generator=g, device=DEV))
    bias = torch.rand(N, generator=g, device=DEV)
    x, small, _ = dev(*make(2, 50, K, "q8", 9))
    y, y2 = torch.full((2, N), float("nan"), device=DEV), torch.empty(2, 50, device=DEV)
    rtq.project_a8([rtq.Projection(w, x, y, bias), rtq.Projection(small, x, y2)])
    check(y2, x, small, None)
    for at in (0, (1 << 23) - 40, N - 64):
        part = slice(at, min(N, at + 77))
        check(y[:, part], x, rtq.Q8Weight(w.payload[part], w.scale[part]), bias[part])
    assert not torch.isnan(y).any()


def test_timing_marks_cover_the_product():
    x, w, _ = dev(*make(80, 64, 128, "q8", 1))
    rtq.timing_enable(True)
    try:
        rtq.gemm_a8(x, w)
        ms, launches = rtq.timing_read()
    finally:
        rtq.timing_enable(False)
    assert launches == 1 and ms > 0
