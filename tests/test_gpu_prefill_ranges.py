"""Packed sequences that leave no item of work are reported as any others that do not follow each other."""
import pytest
import torch

from mla_decode_attention_gb300 import binding
from tests.test_gpu_append import DEV, library  # noqa: F401

pytestmark = pytest.mark.gpu


def call(cu_q, cu_k, rows, h):
    x = torch.zeros(rows, h, 128, dtype=torch.bfloat16, device=DEV)
    buf = binding.PrefillBuffers(rows, rows, len(cu_q) - 1, h, h, DEV)
    buf.out.fill_(9.0)
    cu = [torch.tensor(c, dtype=torch.int32, device=DEV) for c in (cu_q, cu_k)]
    binding.mla_prefill(x, x, x, cu[0], cu[1], 1.0, True, buf.num_sm_parts, buf.workspace, buf.out, buf.lse, err=buf.err)
    torch.cuda.synchronize()
    return int(buf.err.item()), buf.out


@pytest.mark.parametrize("cu_q", [[300, 200, 100], [400, 0, 0], [2**31 - 1, 500, 450], [400, 399, -7]])
@pytest.mark.parametrize("h", [2, 128])
def test_lengths_that_leave_nothing(cu_q, h):
    """More blocks than SMs (128 heads), so that every block that runs takes on others."""
    err, _ = call(cu_q, [0, 200, 400], 400, h)
    assert err == binding.MLA_DEVERR_BAD_RANGE


@pytest.mark.parametrize("cu_k", [[0, 200, 100], [-1, 200, 400], [0, 200, 401]])
@pytest.mark.parametrize("h", [2, 128])
def test_keys_alone(cu_k, h):
    err, _ = call([100, 100, 100], cu_k, 400, h)       # (no query at all)
    assert err == binding.MLA_DEVERR_BAD_RANGE


@pytest.mark.parametrize("h", [2, 128])
def test_empty_sequences_are_no_fault(h):
    err, out = call([100, 100, 100], [0, 200, 400], 400, h)
    assert err == 0 and bool((out == 9.0).all())
