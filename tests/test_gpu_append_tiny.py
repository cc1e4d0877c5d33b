"""mla_append_kv of columns so small that absmax / 448 rounds to 0 in fp32: the
656-byte format's scale is then the least float, not 0, and no code is NaN."""
import numpy as np
import pytest
import torch

import oracle
from mla_decode_attention_gb300 import binding
from tests._util import f64_np
from tests.test_gpu_append import BF16, DEV, FP8_528, FP8_656, case, library, run  # noqa: F401

pytestmark = pytest.mark.gpu

LEAST = 2.0 ** -149


@pytest.mark.parametrize("fmt", [BF16, FP8_656, FP8_528])
def test_columns_near_the_least_float(fmt):
    """Weights of 40 and 0 times the least float on normalised rows: columns are
    up to 224 times it (checked), so each is a whole multiple that the quotient by
    the least float gives back."""
    c = case(fmt, [70, 3], 3, seed=51)
    c["weight"] = torch.where(torch.arange(512) % 7 == 3, 0.0, 40 * LEAST).float()
    rows = run(c, rope=False)
    x = f64_np(c["x"])
    want = oracle.rms_norm(x[..., :512], f64_np(c["weight"]), 1e-6)
    assert 40 * LEAST <= np.abs(want).max() <= 224 * LEAST
    pos = oracle.token_positions(c["lens"].tolist(), None, 3)
    for b in range(2):
        for j in range(3):
            row = rows[int(c["table"][b, pos[b, j] // 64]), pos[b, j] % 64]
            if fmt == BF16:
                assert torch.equal(row[:512].float(), torch.zeros(512))     # below half of bf16's least
                continue
            raw = row.numpy()
            codes = oracle.e4m3_to_f64(raw[:512])
            assert np.all(np.isfinite(codes))
            if fmt == FP8_528:
                assert np.all(codes == 0)                                    # below 2^-10 of the least scale, 2^-127
                continue
            scale = np.ascontiguousarray(raw[512:528]).view(np.float32).astype(np.float64)
            assert np.all(scale == LEAST)
            # the fp32 product is a whole multiple, off by half of one; then half a step of e4m3, 2^-4 of the value
            assert np.all(np.abs(codes * LEAST - want[b, j]) <= 2.0 ** -4 * (np.abs(want[b, j]) + 0.5 * LEAST) + 0.5 * LEAST * 1.001)


def test_zero_columns_keep_the_scale_one():
    c = case(FP8_656, [70, 3], 3, seed=52)
    c["weight"] = torch.zeros(512)
    rows = run(c, rope=False)
    raw = rows[int(c["table"][0, 1]), 5].numpy()
    assert np.all((raw[:512] & 0x7F) == 0)                                   # zeros of either sign
    assert np.all(np.ascontiguousarray(raw[512:528]).view(np.float32) == 1.0)
