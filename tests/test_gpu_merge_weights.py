"""Values that are not finite in parts of little weight: only a part without keys leaves no trace."""
import pytest
import torch

from mla_decode_attention_gb300 import binding
from tests.test_gpu_append import DEV, library  # noqa: F401
from tests.test_gpu_merge import case as states, run as merge
from tests.test_gpu_prefill import case, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,d", [(2, 512), (3, 128), (9, 128), (40, 64)])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_a_part_far_below_the_others(dtype, n, d, bad):
    """Its lse is finite: it has seen keys, and a sum with what is not finite is not finite."""
    parts, lses = states(n, 20, 3, d, dtype, empty=0.0)
    lses[n - 1] = -300.0
    clean = merge(parts, lses)
    parts[n - 1, 7, 1, 5] = bad
    out, lse = merge(parts, lses)
    assert not bool(out[7, 1, 5].isfinite())
    rest = torch.ones(20, 3, d, dtype=torch.bool)
    rest[7, 1, 5] = False
    assert torch.equal(out[rest], clean[0][rest]) and torch.equal(lse, clean[1])
    lses[n - 1] = -float("inf")                        # without keys it leaves none
    out, _ = merge(parts, lses)
    assert bool(out.isfinite().all())


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_a_piece_far_below_the_others(bad):
    """The same call in one piece and in several: keys 0 .. 1999 score about 200 less than the rest."""
    c = case([8], [4000], 2, rope="none", causal=False)
    c["q"].fill_(1.0)
    c["k"].normal_(0, 0.05, generator=torch.Generator().manual_seed(4))
    c["k"][:2000] -= 20.0                              # 20 * 128 / 128^0.5 = 226
    clean = run(c)
    c["v"][100, 1, 5] = bad
    assert binding.mla_prefill_workspace_size(8, 4000, 1, 2, 2, 152) > 0
    for parts in (1, 152, 37):
        out, lse = run(c, parts=parts)
        assert not bool(out[:, 1, 5].isfinite().any()), f"{parts} parts"
        rest = torch.ones_like(out, dtype=torch.bool)
        rest[:, 1, 5] = False
        assert bool(out[rest].isfinite().all())
        if parts == 152:
            assert torch.equal(out[rest], clean[0][rest]) and torch.equal(lse, clean[1])
