"""The tests' own MX4 reference against worked values."""
import numpy as np

from tests import mx4_ref as ref


def _block(*head):
    v = np.zeros((1, 32))
    v[0, :len(head)] = head
    return v


def test_encode_worked_values():
    # largest 6 -> floor(log2 6) = 2, scale 2^0: ties go to the even code
    code, e = ref.encode(_block(6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -5, -0.0, 0.26, 5.01))
    assert e[0, 0] == 127
    assert code[0, :12].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 14, 8, 1, 7]
    # largest 7.9: same scale, saturates; largest 8: scale 2^1
    assert ref.rounded(_block(7.9, 3.9))[0, :2].tolist() == [6.0, 4.0]
    code, e = ref.encode(_block(8, 1))
    assert e[0, 0] == 128 and code[0, :2].tolist() == [6, 1]
    # zeros, and the smallest subnormal
    assert ref.encode(_block(0))[1][0, 0] == 0
    code, e = ref.encode(_block(2.0 ** -127, 2.0 ** -149))
    assert e[0, 0] == 0 and code[0, :2].tolist() == [2, 0]
    # the largest finite BF16
    code, e = ref.encode(_block(ref.bf16_to_f64(np.array([0x7F7F], np.uint16))[0]))
    assert e[0, 0] == 252 and code[0, 0] == 7
    for bad in (np.inf, -np.inf, np.nan):
        code, e = ref.encode(_block(1, bad))
        assert e[0, 0] == 255 and not code.any()
        assert np.isnan(ref.rounded(_block(1, bad))).all()


def test_container_places():
    R, K = 17, 160
    code = np.zeros((1, R, K), np.uint8)
    e = np.full((1, R, K // 32), 100, np.uint8)
    code[0, 16, 133] = 5            # tile 1, group 1, piece 0, code 5 -> byte 2, high half
    code[0, 3, 64] = 9              # tile 0, group 0, piece 16*2 + 3, byte 0, low half
    e[0, 16, 4] = 77                # tile 1, quad 0, piece 0, byte 1
    codes, scales = ref.container(code, e)
    assert codes.size == 2 * 2 * 1024 and scales.size == 2 * 256
    assert codes[(1 * 2 + 1) * 1024 + 2] == 5 << 4
    assert codes[(16 * 2 + 3) * 16] == 9
    assert np.count_nonzero(codes) == 2
    assert scales[256 + 1] == 77
    assert scales[256 + 4] == 127   # row 17 is padding
    assert scales[2] == 127         # group 2 does not exist


def test_bf16_rounding():
    bits = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    v = ref.bf16_to_f64(bits)
    fin = np.isfinite(v)
    assert np.array_equal(ref.f64_to_bf16_bits(v[fin]), bits[fin])
