"""Pins of the fp64 oracle of the operators on 8-bit activations: hand-made
rows, PyTorch's own casts, and the exact-rational quotient."""
from fractions import Fraction

import numpy as np
import pytest

import oracle

torch = pytest.importorskip("torch")


def test_codes_of_hand_made_rows():
    p = np.array([[127.0, -127.0, 63.5, 64.5, -0.5, 0.4, 1.5, 0.0]])
    codes, scale = oracle.a8.codes_and_scale(p, 1.0, "q8")
    assert codes.tolist() == [[127, -127, 64, 64, 0, 0, 2, 0]]          # ties to even
    assert scale.tolist() == [1.0]
    codes, scale = oracle.a8.codes_and_scale(p * 2.0 ** -20, 3.0, "q8")
    assert codes.tolist() == [[127, -127, 64, 64, 0, 0, 2, 0]]
    assert scale.tolist() == [np.float32(3 * 2.0 ** -20)]
    p = np.array([[448.0, -448.0, 1.0, 17.0, 19.0, -2.0 ** -10, 3 * 2.0 ** -10, 0.0]])
    codes, scale = oracle.a8.codes_and_scale(p, 1.0, "f8")
    assert oracle.decode_f8(codes).tolist() == [[448, -448, 1, 16, 20, 0, 2 * 2.0 ** -9, 0]]
    assert codes[0, 5] == 0x80 and scale.tolist() == [1.0]


def test_rows_without_a_finite_scale():
    p = np.array([[0.0, 0.0], [np.nan, 1.0], [np.inf, 1.0], [1e300, 1.0], [1e-300, -1e-300]])
    for fmt in ("q8", "f8"):
        codes, scale = oracle.a8.codes_and_scale(p, 1.0, fmt)
        assert scale[0] == 0 and np.isnan(scale[1:4]).all() and scale[4] == 0
        assert not codes[:4].any() and codes[4, 0] != 0


def test_int8_codes_against_exact_quotients():
    rng = np.random.default_rng(1)
    p = rng.standard_normal((3, 200))
    p[2] = rng.integers(-254, 255, 200) / 2.0
    p[2, 0] = 127.0
    codes, _ = oracle.a8.codes_and_scale(p, 1.0, "q8")
    for row, c in zip(p, codes):
        P = max(abs(Fraction(float(v))) for v in row)
        assert [round(127 * Fraction(float(v)) / P) for v in row] == c.tolist()


def test_e4m3_rounding_against_the_cast():
    v = np.concatenate([oracle.decode_f8(np.arange(0x7F, dtype=np.uint8)), np.linspace(0, 448, 10007),
                        np.exp2(np.linspace(-12, 8.8, 5003))])
    v = np.concatenate([v, -v]).astype(np.float32)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(oracle.a8.nearest_e4m3(v.astype(np.float64)), want)
    # next to a tie by less than fp32 can tell
    t = np.array([17.0 * (1 + 2.0 ** -40), 17.0 * (1 - 2.0 ** -40), 17.0])
    assert oracle.decode_f8(oracle.a8.nearest_e4m3(t)).tolist() == [18.0, 16.0, 16.0]


def test_rounding_to_bf16_and_fp16():
    v = np.random.default_rng(2).standard_normal(5000).astype(np.float32)
    for name, t in (("bf16", torch.bfloat16), ("fp16", torch.float16)):
        want = torch.from_numpy(v).to(t).to(torch.float32).numpy()
        assert np.array_equal(oracle.a8.round_to(v, name), want)


def test_norm_and_product_on_small_cases():
    h, p, r = oracle.a8.rms_norm_parts(np.array([[3.0, 4.0]]), np.array([[0.0, 0.0]]), np.array([2.0, 1.0]), 1e-30, "fp32")
    assert h.tolist() == [[3.0, 4.0]] and p.tolist() == [[6.0, 4.0]] and np.allclose(r, 1 / np.sqrt(12.5), rtol=1e-15)
    assert np.allclose(oracle.a8.silu_mul([[0.0, 2.0]], [[5.0, 3.0]]), [[0.0, 6.0 / (1 + np.exp(-2.0))]], rtol=1e-15)
    y, size = oracle.a8.gemm_a8(np.array([[1, -2]]), [0.5], np.array([[3, 4]]), [2.0], [10.0], "q8")
    assert y.tolist() == [[5.0]] and size.tolist() == [[11.0]]


@pytest.mark.parametrize("fmt", ["q8", "f8"])
def test_ties_of_rounded_products(fmt):
    """Rows of one gate: the codes are those of b / max b, whichever way the gate's fp64 value rounds."""
    if fmt == "q8":
        b = np.arange(-127.0, 127.5, 0.5)
    else:
        v = oracle.decode_f8(np.arange(0x7F, dtype=np.uint8)).astype(np.float64)
        b = np.concatenate([v, (v[1:] + v[:-1]) / 2])
    for a in np.random.default_rng(3).standard_normal(200).astype(np.float32) * 4:
        codes, _ = oracle.a8.codes_and_scale(oracle.a8.silu_mul(np.full((1, b.size), a), b[None]), 1.0, fmt)
        t = np.copysign(1.0, a) * b                        # max |b| is R, so this is R b / max |b|
        want = np.rint(t).astype(np.int8) if fmt == "q8" else oracle.a8.nearest_e4m3(t)
        assert np.array_equal(codes[0], want)
