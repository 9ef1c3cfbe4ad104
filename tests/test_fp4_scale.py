"""The steps that csa2_fp4_quant's group scales are computed by, on the CPU over every mantissa: amax / 6 in
E4M3 without a division (csa2_fp4.cu has the proof; every step here is exact but for the roundings named)."""
import numpy as np

SIXTH = np.float32(1) / np.float32(6)


def _e4m3(v):
    """Nearest E4M3 value, ties to even, saturating; v float64 >= 0."""
    e = np.maximum(np.floor(np.log2(np.where(v > 0, v, 1.0))), -6)
    step = np.exp2(e - 3)
    return np.minimum(np.rint(v / step) * step, 448.0)


def test_fp32_product_and_remainder_is_the_rounded_quotient():
    a = (np.arange(1 << 23, dtype=np.uint32) + 0x3F800000).view(np.float32)
    y = a * SIXTH
    rest = a.astype(np.float64) - 6.0 * y.astype(np.float64)
    assert (rest.astype(np.float32) == rest).all()  # the remainder needs no rounding
    z = y.astype(np.float64) + rest * np.float64(SIXTH)
    # z, itself rounded to 53 bits, lies on no border between two fp32 values: rounding it is the fused step's rounding
    assert ((z.view(np.uint64) & 0x1FFFFFFF) != 0x10000000).all()
    assert (z.astype(np.float32) == (a.astype(np.float64) / 6.0).astype(np.float32)).all()


def test_the_rounded_quotient_gives_the_scale():
    """E4M3 of the fp32 quotient is E4M3 of the quotient, in the subnormal scales' binades and among the others."""
    for e in (-10, -9, -8, -7, 0, 7):
        a = (np.arange(1 << 23, dtype=np.uint32) + ((127 + e + 2) << 23)).view(np.float32)
        q = a.astype(np.float64) / 6.0
        assert (_e4m3(q) == _e4m3(q.astype(np.float32).astype(np.float64))).all()


def test_bf16_product_rounded_to_13_bits_gives_the_scale():
    a = ((np.arange((127 - 10) << 7, (127 + 12) << 7, dtype=np.uint32)) << 16).view(np.float32)
    y = (((a * SIXTH).view(np.uint32) + 0x400) & np.uint32(0xFFFFF800)).view(np.float32)
    assert (_e4m3(y.astype(np.float64)) == _e4m3(a.astype(np.float64) / 6.0)).all()
