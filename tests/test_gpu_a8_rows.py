"""GPU tests of the row operators (quantizer, norm, gated product) against the
fp64 oracle: codes equal, scales and dense rows within counted roundings."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
import weight_only_quantized_rtq_amd as rtq  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6


def host(t):
    return t.float().cpu().numpy()


def make(M, K, dtype, seed, pad=0, scale=1.0):
    """[M, K] rows inside [M, K + pad]; a few columns far larger than the rest."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K + pad, generator=g) * scale
    x[:, torch.rand(K + pad, generator=g) > 0.98] *= 20
    return x.to(DTYPES[dtype]).to(DEV)[:, :K]


def check_codes(out, p, r, fmt):
    torch.cuda.synchronize()
    codes, scale = oracle.a8.codes_and_scale(p, r, fmt)
    got = out.codes.cpu().numpy()
    assert got.dtype == codes.dtype
    assert np.array_equal(got, codes), f"{np.sum(got != codes)} of {codes.size} codes differ"
    s = out.scale.cpu().numpy()
    assert np.array_equal(np.isnan(s), np.isnan(scale))
    # the fp64 value (good to 2^-45) rounded once on either side: one fp32 step at most
    fine = ~np.isnan(scale)
    assert np.all(np.abs(s[fine] - scale[fine]) <= np.spacing(np.abs(scale[fine])))


def check_dense(got, want, roundings):
    """|got - want| within `roundings` fp32 ones and the output's own, of half a step each; results
    below the type's normal range are off by half a step of its smallest numbers."""
    torch.cuda.synchronize()
    info = torch.finfo(got.dtype)
    g = got.double().cpu().numpy()
    with np.errstate(all="ignore"):
        inside = np.abs(want) <= info.max
        assert np.array_equal(np.isnan(g), np.isnan(want))
        tol = np.abs(want) * (roundings * 2.0 ** -24 * 1.01 + info.eps / 2) + float(info.tiny) * info.eps + 2.0 ** -148
        assert np.all((np.abs(g - want) <= tol)[inside & ~np.isnan(want)])


LENGTHS = [1, 7, 8, 9, 64, 511, 512, 513, 1000, 1024, 1030, 2048, 2049, 4096, 4100, 8192, 8200, 16384, 16390, 40001]


@pytest.mark.parametrize("K", LENGTHS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize_rows(dtype, K):
    for fmt, M, pad in (("q8", 5, 0), ("f8", 6, 3)):
        x = make(M, K, dtype, K, pad)
        check_codes(rtq.quantize_rows(x, fmt), host(x).astype(np.float64), 1.0, fmt)


@pytest.mark.parametrize("K", LENGTHS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_rms_norm(dtype, K):
    w = 1 + 0.3 * torch.randn(K, generator=torch.Generator().manual_seed(K)).to(DEV)
    for fmt, M, residual, pad in (("q8", 5, True, 0), ("f8", 3, False, 5), ("q8", 2, False, 0), ("f8", 6, True, 8)):
        x = make(M, K, dtype, K + 1, pad)
        res = make(M, K, dtype, K + 2, pad) if residual else None
        out = rtq.rms_norm(x, w, EPS, residual=res, fmt=fmt)
        h, p, r = oracle.a8.rms_norm_parts(host(x), None if res is None else host(res), host(w), EPS, dtype)
        if residual:
            out, s = out
            assert s.dtype == x.dtype and np.array_equal(host(s), h)
        check_codes(out, p, r, fmt)
        for out_dtype in {x.dtype, torch.float32}:
            y = rtq.rms_norm(x, w, EPS, residual=res, out_dtype=out_dtype)
            y = y[0] if residual else y
            assert y.dtype == out_dtype
            check_dense(y, p * r[:, None], 3)          # r, h r, times w


@pytest.mark.parametrize("K", LENGTHS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_silu_mul(dtype, K):
    for fmt, M, fused in (("q8", 5, False), ("f8", 4, True)):
        if fused:
            ab = make(M, 2 * K, dtype, K + 3, scale=2.0)
            a, b = ab[:, :K], ab[:, K:]
        else:
            a, b = make(M, K, dtype, K + 4, 3), make(M, K, dtype, K + 5)
        p = oracle.a8.silu_mul(host(a), host(b))
        check_codes(rtq.silu_mul(a, b, fmt=fmt), p, 1.0, fmt)
        for out_dtype in {a.dtype, torch.float32}:
            # 2^hi and 1 / (1 + e) to one step (two halves) each; the correction of e, 1 + e, a u, u b: four more
            check_dense(rtq.silu_mul(a, b, out_dtype=out_dtype), p, 8)


def special_rows(K, dtype):
    """Rows that reach every branch, as fp32 values that the type holds."""
    rng = np.random.default_rng(K)
    top = {"fp32": 3e38, "bf16": 3e38, "fp16": 6e4}[dtype]
    tiny = {"fp32": 1e-44, "bf16": 9.2e-41, "fp16": 6e-8}[dtype]
    n = rng.standard_normal(K)
    ties = rng.integers(-254, 255, K) / 2.0
    ties[0] = 127.0
    rows = [np.zeros(K), n * 1e-20, n * 1e-30, np.full(K, tiny), np.full(K, top), n * top / 8, ties, -ties / 64,
            np.where(np.arange(K) == K // 2, 1.0, 0.0), np.full(K, -2.5), np.where(np.arange(K) == K - 1, top, n),
            np.where(np.arange(K) == 0, tiny, 0.0), n * 2.0 ** 61, n * 2.0 ** -59]
    for bad in (np.nan, np.inf, -np.inf):
        rows += [np.where(np.arange(K) == K // 3, bad, n), np.full(K, bad)]
    v = np.array(rows)
    with np.errstate(over="ignore"):
        return torch.from_numpy(np.clip(v, -top, top) if dtype == "fp16" else v).float().to(DTYPES[dtype]).to(DEV) \
            if dtype != "fp16" else torch.from_numpy(np.where(np.isfinite(v), np.clip(v, -top, top), v)).half().to(DEV)


@pytest.mark.parametrize("fmt", ["q8", "f8"])
@pytest.mark.parametrize("K", [9, 512, 1000, 2048, 8192, 20000])
@pytest.mark.parametrize("dtype", DTYPES)
def test_special_rows(dtype, K, fmt):
    x = special_rows(K, dtype)
    check_codes(rtq.quantize_rows(x, fmt), host(x).astype(np.float64), 1.0, fmt)
    # weights of one keep the ties ties; others push products past fp32 and below it
    for w in (torch.ones(K), torch.full((K,), 1e-30), torch.full((K,), 3e30),
              torch.randn(K, generator=torch.Generator().manual_seed(1))):
        w = w.float().to(DEV)
        h, p, r = oracle.a8.rms_norm_parts(host(x), None, host(w), EPS, dtype)
        check_codes(rtq.rms_norm(x, w, EPS, fmt=fmt), p, r, fmt)
    flipped = x.flip(0)
    for a, b in ((x, flipped), (x, torch.ones_like(x)), (-x.abs(), flipped), (x / 16, x)):
        check_codes(rtq.silu_mul(a, b.contiguous(), fmt=fmt), oracle.a8.silu_mul(host(a), host(b)), 1.0, fmt)


@pytest.mark.parametrize("fmt", ["q8", "f8"])
def test_gated_product_of_far_negative_gates(fmt):
    """exp(-a) past fp32, with factors that bring the product back into it."""
    K = 640
    g = torch.Generator().manual_seed(4)
    a = -70 - 60 * torch.rand(6, K, generator=g)
    b = torch.randn(6, K, generator=g) * torch.tensor([1.0, 1e10, 1e25, 1e36, 1e38, 1e-5])[:, None]
    a[3] = torch.where(torch.arange(K) % 2 == 0, a[3], torch.full((K,), -1e-41))
    check_codes(rtq.silu_mul(a.to(DEV), b.to(DEV), fmt=fmt), oracle.a8.silu_mul(a.numpy(), b.numpy()), 1.0, fmt)
    check_dense(rtq.silu_mul(a.to(DEV), b.to(DEV)), oracle.a8.silu_mul(a.numpy(), b.numpy()), 8)


def test_quotients_next_to_a_border():
    """Values placed one fp32 step to either side of every border of a row, by the hundred."""
    for fmt, R in (("q8", 127.0), ("f8", 448.0)):
        rng = np.random.default_rng(5)
        rows = []
        for _ in range(40):
            P = np.float32(rng.uniform(0.5, 2.0))
            if fmt == "q8":
                border = np.arange(-126.5, 127.0)
            else:
                v = oracle.decode_f8(np.arange(0x7F, dtype=np.uint8))
                border = (v[1:] + v[:-1]) / 2
            at = (border * float(P) / R).astype(np.float32)
            rows.append(np.concatenate([[P], at, np.nextafter(at, np.float32(9)), np.nextafter(at, np.float32(-9))]))
        x = torch.from_numpy(np.array(rows, np.float32)).to(DEV)
        check_codes(rtq.quantize_rows(x, fmt), host(x).astype(np.float64), 1.0, fmt)
        # and through a norm whose products are inexact in fp32
        w = torch.from_numpy((1 + rng.uniform(0, 1, x.shape[1])).astype(np.float32)).to(DEV)
        y = (x.double() / w.double()).float()
        h, p, r = oracle.a8.rms_norm_parts(host(y), None, host(w), EPS, "fp32")
        check_codes(rtq.rms_norm(y, w, EPS, fmt=fmt), p, r, fmt)


@pytest.mark.parametrize("fmt", ["q8", "f8"])
@pytest.mark.parametrize("dtype", DTYPES)
def test_true_ties_of_rounded_products(dtype, fmt):
    """Rows of one gate, and norms with weights of one value: R p / P is b / max b or x / max x exactly."""
    if fmt == "q8":
        b = np.arange(-127.0, 127.5, 0.5)
    else:
        v = oracle.decode_f8(np.arange(0x7F, dtype=np.uint8)).astype(np.float64)
        b = np.concatenate([v, (v[1:] + v[:-1]) / 2])
    code = (lambda t: np.rint(t).astype(np.int8)) if fmt == "q8" else oracle.a8.nearest_e4m3
    g = torch.Generator().manual_seed(8)
    a = (torch.randn(200, 1, generator=g) * 4).to(DTYPES[dtype])
    rows = torch.from_numpy(b)[None].repeat(200, 1).to(DTYPES[dtype]).to(DEV)
    assert np.array_equal(host(rows[0]), b)
    out = rtq.silu_mul(a.repeat(1, b.size).to(DEV), rows, fmt=fmt)
    want = np.stack([code(np.copysign(1.0, s) * b) for s in a[:, 0].tolist()])
    assert np.array_equal(out.codes.cpu().numpy(), want)
    for value in (1.1, 0.3, 2 / 3):
        out = rtq.rms_norm(rows, torch.full((b.size,), value, device=DEV), EPS, fmt=fmt)
        assert np.array_equal(out.codes.cpu().numpy(), np.stack([code(b)] * 200))


@pytest.mark.parametrize("dtype", DTYPES)
def test_sum_in_place_and_what_lies_around_it(dtype):
    """sum_out may be the residual or x; rows of wider buffers and guards stay as they were."""
    M, K = 7, 777
    w = torch.rand(K, device=DEV)
    for which in ("residual", "x"):
        wide = make(M + 2, K + 40, dtype, 9).contiguous()
        other = make(M, K, dtype, 10)
        inner = wide[1:M + 1, 8:K + 8]
        before = wide.clone()
        args = (other, inner) if which == "residual" else (inner, other)
        h, p, r = oracle.a8.rms_norm_parts(host(args[0]), host(args[1]), host(w), EPS, dtype)
        out, s = rtq.rms_norm(args[0], w, EPS, residual=args[1], fmt="q8", sum_out=inner)
        assert s is inner
        check_codes(out, p, r, "q8")
        assert np.array_equal(host(inner), h)
        before[1:M + 1, 8:K + 8] = inner
        assert torch.equal(before, wide)
    codes = torch.full((M + 2, K), 77, dtype=torch.int8, device=DEV)
    scale = torch.full((M + 2,), 5.0, device=DEV)
    x = make(M, K, dtype, 11)
    rtq.quantize_rows(x, "q8", out=rtq.A8Rows(codes[1:M + 1], scale[1:M + 1]))
    check_codes(rtq.A8Rows(codes[1:M + 1], scale[1:M + 1]), host(x).astype(np.float64), 1.0, "q8")
    assert (codes[0] == 77).all() and (codes[-1] == 77).all() and scale[0] == 5 and scale[-1] == 5


@pytest.mark.parametrize("K", [3, *range(9, 17), *range(513, 520), 1021, 4094, 9003, 16391])
@pytest.mark.parametrize("dtype", DTYPES)
def test_partial_chunks_in_place_and_their_neighbours(dtype, K):
    """Every remainder of K by eight: codes, the sum in place and dense rows, with guards on both sides."""
    M = 5
    w = 1 + 0.1 * torch.randn(K, generator=torch.Generator().manual_seed(K)).to(DEV)
    wide, other = make(M + 2, K + 3, dtype, K).contiguous(), make(M, K, dtype, K + 1)
    inner, before = wide[1:M + 1, 2:K + 2], wide.clone()
    h, p, r = oracle.a8.rms_norm_parts(host(inner), host(other), host(w), EPS, dtype)
    codes = torch.full((M + 2, K), 77, dtype=torch.uint8, device=DEV)
    scale = torch.full((M + 2,), 5.0, device=DEV)
    out = rtq.A8Rows(codes[1:M + 1], scale[1:M + 1])
    rtq.rms_norm(inner, w, EPS, residual=other, fmt="f8", sum_out=inner, out=out)
    check_codes(out, p, r, "f8")
    assert np.array_equal(host(inner), h)
    before[1:M + 1, 2:K + 2] = inner
    assert torch.equal(before, wide)
    assert (codes[0] == 77).all() and (codes[-1] == 77).all() and scale[0] == 5 and scale[-1] == 5
    dense = torch.full((M + 2, K), 3.0, dtype=DTYPES[dtype], device=DEV)
    rtq.rms_norm(inner, w, EPS, out=dense[1:M + 1])
    h, p, r = oracle.a8.rms_norm_parts(host(inner), None, host(w), EPS, dtype)
    check_dense(dense[1:M + 1], p * r[:, None], 3)
    rtq.silu_mul(inner, other, out=dense[1:M + 1])
    check_dense(dense[1:M + 1], oracle.a8.silu_mul(host(inner), host(other)), 8)
    assert (dense[0] == 3).all() and (dense[-1] == 3).all()


def test_empty_and_many_rows():
    w = torch.ones(8, device=DEV)
    x = torch.empty(0, 8, device=DEV)
    assert rtq.quantize_rows(x).codes.shape == (0, 8)
    out, s = rtq.rms_norm(x, w, residual=x, fmt="f8")
    assert out.scale.shape == (0,) and s.shape == (0, 8)
    assert rtq.silu_mul(x, x).shape == (0, 8)
    # more rows than the largest grid holds: four rows a workgroup, and one
    for M, K in ((5_000_003, 3), (1_050_000, 1025)):
        x = torch.arange(M, device=DEV, dtype=torch.float32)[:, None].expand(M, K).to(torch.bfloat16).contiguous()
        q = rtq.quantize_rows(x, "q8")
        # (a quotient by a number in fp32 is torch's product with its rounded reciprocal)
        assert torch.equal(q.scale, (x[:, 0].double() / 127).float())
        assert (q.codes[1:] == 127).all() and (q.codes[0] == 0).all()
        del x, q


def test_dense_rows_with_infinities_follow_the_formula():
    x = torch.randn(4, 100, device=DEV)
    x[1, 5], x[2, 7], x[3, 0] = float("inf"), float("nan"), 3e38
    w = torch.rand(100, device=DEV)
    y = rtq.rms_norm(x, w).cpu()
    assert torch.isfinite(y[0]).all() and torch.isfinite(y[3]).all() and torch.isnan(y[2]).all()
    assert torch.isnan(y[1, 5]) and (y[1, :5] == 0).all()


def test_refusals_on_the_device():
    x, w = torch.zeros(4, 64, device=DEV), torch.ones(64, device=DEV)
    with pytest.raises(ValueError, match="adjacent"):
        rtq.quantize_rows(x.t())
    with pytest.raises(ValueError, match="overlap"):
        rtq.quantize_rows(x[:1].expand(4, 64))
    with pytest.raises(ValueError, match="weight"):
        rtq.rms_norm(x, w[:63])
    with pytest.raises(TypeError):
        rtq.rms_norm(x, w.half())
    with pytest.raises(TypeError):
        rtq.rms_norm(x, w, residual=x.half())
    with pytest.raises(ValueError):
        rtq.rms_norm(x, w, residual=x[:3])
    with pytest.raises(ValueError, match="residual"):
        rtq.rms_norm(x, w, sum_out=torch.zeros_like(x))
    with pytest.raises(TypeError):
        rtq.rms_norm(x, w, fmt="q8", out_dtype=torch.float32)
    with pytest.raises(TypeError):
        rtq.rms_norm(x.half(), w, out_dtype=torch.bfloat16)
    with pytest.raises(rtq.RtqError) as e:
        rtq.rms_norm(x, w, 0.0)
    assert e.value.status == 2
    with pytest.raises(rtq.RtqError) as e:
        rtq.silu_mul(x, x, out=x)
    assert e.value.status == 6
    with pytest.raises(TypeError):
        rtq.quantize_rows(x, "f8", out=rtq.A8Rows(torch.empty(4, 64, dtype=torch.int8, device=DEV), w[:4]))
    with pytest.raises(ValueError):
        rtq.quantize_rows(x, "q8", out=rtq.A8Rows(torch.empty(4, 63, dtype=torch.int8, device=DEV), w[:4]))


def test_offsets_past_32_bits():
    """More than 2^32 elements: rows at the far ends against the same rows on their own."""
    M, K = (1 << 20) + 700, 4104
    x = torch.zeros(M, K, dtype=torch.bfloat16, device=DEV)
    ends = torch.tensor([0, 1, (1 << 32) // K - 1, (1 << 32) // K, (1 << 32) // K + 1, M - 1], device=DEV)
    x[ends] = torch.randn(len(ends), K, device=DEV).to(torch.bfloat16)
    w = torch.rand(K, device=DEV)
    few = x[ends].contiguous()
    for fmt in ("q8", "f8"):
        for call in (lambda v: rtq.quantize_rows(v, fmt), lambda v: rtq.rms_norm(v, w, fmt=fmt),
                     lambda v: rtq.silu_mul(v, v, fmt=fmt)):
            big, want = call(x), call(few)
            assert torch.equal(big.codes[ends], want.codes) and torch.equal(big.scale[ends], want.scale)
            assert big.scale.count_nonzero() == len(ends)
            del big


@pytest.mark.parametrize("fmt", ["q8", "f8", None])
def test_captured_and_on_other_streams(fmt):
    """Two streams at once, and a graph replayed with new inputs and eager work in between."""
    g = torch.Generator().manual_seed(3)
    xs = [torch.randn(33, 1000, generator=g).to(DEV) for _ in range(4)]
    res, w = torch.randn(33, 1000, generator=g).to(DEV), torch.rand(1000, generator=g).to(DEV)

    def values(r):
        out, h = r
        return [h] + ([out] if fmt is None else [out.codes, out.scale])

    want = [values(rtq.rms_norm(x, w, residual=res, fmt=fmt)) for x in xs]
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(2)]
    got = [values(rtq.rms_norm(x, w, residual=res, fmt=fmt, stream=side[i % 2])) for i, x in enumerate(xs)]
    raw = values(rtq.rms_norm(xs[0], w, residual=res, fmt=fmt, stream=side[0].cuda_stream))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for r, s in zip(got, want) for a, b in zip(r, s))
    assert all(torch.equal(a, b) for a, b in zip(raw, want[0]))
    x = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = values(rtq.rms_norm(x, w, residual=res, fmt=fmt))
    for i in (2, 1, 3, 0):
        x.copy_(xs[i])
        graph.replay()
        eager = values(rtq.rms_norm(xs[(i + 1) % 4], w, residual=res, fmt=fmt))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[i]))
        assert all(torch.equal(a, b) for a, b in zip(eager, want[(i + 1) % 4]))
