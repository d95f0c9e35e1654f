"""Pins for oracle.fp4: the e2m1 grid and its ties, hand-computed blocks of both
formats, the scale tiles' order and a brute-force product."""

import numpy as np

from oracle import fp4


def test_e2m1_grid_ties_and_saturation():
    v = [0, .25, .26, .5, .75, 1, 1.25, 1.26, 1.75, 2, 2.5, 2.51, 3.5, 4, 5, 5.01, 6, 100, -0.75, -5]
    want = [0, 0, .5, .5, 1, 1, 1, 1.5, 2, 2, 2, 3, 4, 4, 4, 6, 6, 6, -1, -4]
    assert fp4.decode_e2m1(fp4.encode_e2m1(v)).tolist() == want
    codes = np.arange(16)
    assert np.array_equal(fp4.encode_e2m1(fp4.decode_e2m1(codes)) & 7, codes & 7)


def test_hand_block_mxfp4():
    x = np.zeros((1, 32))
    x[0, :4] = [3.0, -1.0, 0.5, 0.1]  # amax 3: 6 / 3 = 2 -> s = 2
    codes, byte, row = fp4.quant_rows(x, "mxfp4")
    assert byte.tolist() == [[126]] and row is None
    assert fp4.decode_e2m1(codes)[0, :4].tolist() == [6, -2, 1, 0]
    assert fp4.values(codes, byte, row, "mxfp4")[0, :4].tolist() == [3, -1, .5, 0]


def test_hand_block_nvfp4():
    x = np.zeros((1, 32))
    x[0, 0], x[0, 1], x[0, 16] = 6.0, 3.0, 0.75  # R = 2^8 (2688 / 6 = 448); blocks: 256, 32
    codes, byte, row = fp4.quant_rows(x, "nvfp4")
    assert row.tolist() == [256.0]
    assert fp4.decode_e4m3(byte).tolist() == [[256.0, 32.0]]
    assert fp4.values(codes, byte, row, "nvfp4")[0, [0, 1, 16]].tolist() == [6, 3, .75]
    z = fp4.quant_rows(np.zeros((2, 16)), "nvfp4")
    assert not z[0].any() and not z[1].any()


def test_error_is_within_half_a_step():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((20, 128)).astype(np.float32).view(np.uint32) & 0xFFFF0000
    x = x.view(np.float32).astype(np.float64)
    for fmt in ("mxfp4", "nvfp4"):
        v = fp4.values(*fp4.quant_rows(x, fmt), fmt)
        amax = np.abs(x.reshape(20, -1, fp4.BLOCK[fmt])).max(2).repeat(fp4.BLOCK[fmt], 1)
        # the widest step is 2 of 6 (s within a factor 2 of amax for mxfp4, 1/16 for nvfp4)
        assert np.all(np.abs(v - x) <= amax * (1 / 3 if fmt == "mxfp4" else 1 / 6 * 1.07 + 1 / 16))


def test_pack_and_tiles():
    c = np.array([[1, 2, 15, 0]], dtype=np.uint8)
    assert fp4.pack(c).tolist() == [[0x21, 0x0F]] and np.array_equal(fp4.unpack(fp4.pack(c)), c)
    byte = np.zeros((130, 5), dtype=np.uint8)
    byte[33, 4] = 7       # tile 0, word 1, lane 1, quarter 1
    byte[129, 2] = 9      # tile 1, word 0, lane 1, quarter 0
    t = fp4.tile_scales(byte)
    assert t.size == 2 * 2 * 512 and t.sum() == 16
    assert t[(0 * 2 + 1) * 512 + 1 * 16 + 1 * 4 + 0] == 7 and t[(1 * 2 + 0) * 512 + 1 * 16 + 0 * 4 + 2] == 9


def test_gmm_is_the_sum_over_the_contraction():
    rng = np.random.default_rng(1)
    x, w = rng.standard_normal((5, 4)), rng.standard_normal((3, 2, 4))
    got = fp4.gmm(x, w, [2, 0, 3])
    for r, e in enumerate([0, 0, 2, 2, 2]):
        for n in range(2):
            assert abs(got[r, n] - sum(x[r, k] * w[e, n, k] for k in range(4))) < 1e-12
