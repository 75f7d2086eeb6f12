"""The arithmetic identities of the dequantization by one fma on the subnormal code, proven
exhaustively on the host for every code and zero point (numpy, binary64, where every
intermediate is exact):

* A code q alone in a 16-bit half is the bf16 number q·2^-133, subnormal below 128 and in the
  first normal binade, which continues the same steps, from 128 on; a nibble at bits 4..7
  is 16·q·2^-133.
* fma(q·2^-133, 2^127, −z·2^-6), or with 16·q and 2^123, is (q − z)·2^-6, a bf16 number:
  its one rounding changes nothing.
* The product with s·2^6, rounded once to bf16, is bf16_rn((q − z)·s) for every bf16 s below
  2^122 (s·2^6 is a bf16 number then, subnormal s included).

The pair and decode kernels take 8-bit codes so, the pair kernel and the gated decode form 4-bit codes."""
import numpy as np
import pytest

import oracle


def f64(bits):
    return (np.asarray(bits, np.uint32) << 16).view(np.float32).astype(np.float64)


def is_bf16(x):
    x = np.atleast_1d(np.asarray(x, np.float64))
    return np.array_equal(f64(oracle.bf16_from_f64(x)), x)


def test_codes_are_bf16_numbers():
    q = np.arange(256, dtype=np.uint16)
    assert np.array_equal(f64(q), q * 2.0 ** -133)
    n = np.arange(16, dtype=np.uint16)
    assert np.array_equal(f64(n << 4), 16 * n * 2.0 ** -133)


@pytest.mark.parametrize("bits", [4, 8])
def test_fma_is_exact(bits):
    q = np.arange(1 << bits, dtype=np.float64)
    for z in range((1 << bits) + 1):             # (symmetric codes: z = 8 or 128)
        nz = -z * 2.0 ** -6
        assert is_bf16(nz)
        for m, shift in ((2.0 ** 127, 1.0), *(((2.0 ** 123, 16.0),) if bits == 4 else ())):
            assert is_bf16(m)
            got = (shift * q * 2.0 ** -133) * m + nz
            assert np.array_equal(got, (q - z) * 2.0 ** -6)
            assert is_bf16(got)


def scales():
    """Every bf16 significand at exponents over the range, all subnormals, the largest below 2^122."""
    sig = np.arange(128, dtype=np.uint32)
    exps = np.array([1, 2, 7, 8, 60, 127, 180, 247, 248], dtype=np.uint32)
    return np.concatenate([((exps[:, None] << 7) | sig).ravel(), np.arange(1, 128, dtype=np.uint32)])


def test_scaled_scales_are_bf16_numbers():
    s = f64(scales())
    assert s.max() < 2.0 ** 122 and is_bf16(s * 64)
    assert s.max() * 64 < 2.0 ** 128 and 2.0 ** 122 * 64 == 2.0 ** 128


@pytest.mark.parametrize("bits", [4, 8])
def test_product_rounds_once(bits):
    s = f64(scales())
    for d in range(-(1 << bits), 1 << bits):
        # (a product of two bf16 numbers has 16 significant bits: exact in binary64)
        got = oracle.bf16_from_f64((d * 2.0 ** -6) * (s * 64))
        assert np.array_equal(got, oracle.bf16_from_f64(d * s)), d


@pytest.mark.parametrize("bits", [4, 8])
def test_symmetric_codes_are_flipped_to_offset_form(bits):
    half = 1 << bits - 1
    for c in range(1 << bits):
        signed = c - (1 << bits) if c >= half else c
        assert (c ^ half) - half == signed
