"""mla_window_decode where a page that only some of a block's tokens need is
missing: the others' outputs do not depend on it, whatever the pool holds."""
import numpy as np
import pytest
import torch

import oracle
from mla_decode_attention_gb300 import binding
from tests._util import assert_parity, f64_np
from tests.test_gpu_append import DEV, library  # noqa: F401
from tests.test_gpu_window import BF16, FP8_528, FP8_656, SCALE, case, keys_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,h", [(FP8_656, 16), (FP8_656, 32), (FP8_528, 16), (FP8_528, 32), (BF16, 16), (BF16, 32), (BF16, 48)])
@pytest.mark.parametrize("entry", [-1, 10 ** 6])
def test_a_bad_page_of_the_oldest_token_alone(fmt, h, entry):
    """Windows of 64 that end at 126 .. 129: the first token alone has a key on
    the request's first page, whose entry is bad.  Page 0 of the pool, which no
    request names, is NaN."""
    c = case(fmt, [130, 70], 4, h, 64, 0, seed=31)
    n = c["cache"].shape[0]
    pool = torch.cat([torch.full_like(c["cache"][:1], float("nan") if fmt == BF16 else 0xFF), c["cache"]])
    table = torch.where(c["table"] >= 0, c["table"] + 1, c["table"])
    keys, good = keys_of(pool, fmt), table.clone()
    assert good[0, 0] > 0 and n + 1 == pool.shape[0]
    table[0, 0] = entry
    buf = binding.WindowBuffers(2, 4, h, 64, 0, DEV)
    binding.mla_window_decode(c["q"].to(DEV), pool.to(DEV), fmt, table.to(DEV), c["lens"].to(DEV), SCALE, 64, 0, buf.num_sm_parts,
                              buf.workspace, buf.out, buf.lse, buf.err)
    torch.cuda.synchronize()
    assert int(buf.err.item()) == binding.MLA_DEVERR_BAD_PAGE
    ro, rl = oracle.window_decode(f64_np(c["q"]), keys, good.numpy().clip(0), c["lens"].tolist(), None, SCALE, 64, 0)
    out, lse = f64_np(buf.out), f64_np(buf.lse)
    for b, j in [(0, 1), (0, 2), (0, 3), (1, 0), (1, 1), (1, 2), (1, 3)]:
        assert_parity(out[b, j], ro[b, j], lse[b, :, j], rl[b, :, j], f"token ({b}, {j})")
    assert np.all(np.isfinite(out))
