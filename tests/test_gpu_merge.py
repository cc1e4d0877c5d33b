"""mla_merge_states against the fp64 definition.

Tolerances.  Exponentials, sum, quotient and n products and sums in fp32: an error below (n + 8) 2^-22 of sum w |part|
(expf's argument is off by half a step of at most 2^6, 2^-18 relative at most in a weight, for log-sum-exps up to 64), then one
rounding to bf16, 2^-8 relative.  lse: 2^-22 of its size and of the sum's logarithm's error, below 2^-18 here."""
import numpy as np
import pytest
import torch

import oracle
from mla_decode_attention_gb300 import binding
from tests._util import f64_np
from tests.test_gpu_append import DEV, library  # noqa: F401

pytestmark = pytest.mark.gpu


def case(n, tokens, h, d, dtype=torch.bfloat16, seed=0, empty=0.2):
    g = torch.Generator().manual_seed(seed)
    lses = 8 * torch.randn(n, h, tokens, generator=g)
    lses[torch.rand(n, h, tokens, generator=g) < empty] = -float("inf")
    parts = torch.randn(n, tokens, h, d, generator=g).to(dtype)
    parts[torch.isinf(lses).permute(0, 2, 1)] = float("nan")     # not read
    return parts, lses


def check(parts, lses, out, lse):
    p, l = f64_np(parts), f64_np(lses)
    want, want_lse = oracle.merge_states(p, l)
    size, _ = oracle.merge_states(np.abs(p), l)
    o, got = f64_np(out), f64_np(lse)
    assert np.array_equal(np.isneginf(got), np.isneginf(want_lse))
    ok = ~np.isneginf(want_lse)
    assert np.max(np.abs(got[ok] - want_lse[ok]), initial=0.0) <= 2.0 ** -18 * 64
    assert np.all(np.abs(o - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -18 + (len(p) + 8) * 2.0 ** -22) * size * 1.01 + 1e-38)


def run(parts, lses):
    _, t, h, d = parts.shape
    out, lse = torch.full((t, h, d), 9.0, dtype=torch.bfloat16, device=DEV), torch.full((h, t), 9.0, device=DEV)
    binding.mla_merge_states(parts.to(DEV), lses.to(DEV), out, lse)
    torch.cuda.synchronize()
    return out.cpu(), lse.cpu()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,tokens,h,d", [(1, 1, 1, 8), (2, 1, 128, 512), (2, 300, 3, 128), (3, 7, 5, 64), (5, 33, 2, 72), (7, 9, 16, 128),
                                          (8, 5, 3, 256), (9, 40, 1, 264), (16, 3, 4, 504), (33, 11, 2, 128), (40, 2, 3, 40), (2, 1000, 1, 512)])
def test_shapes(n, tokens, h, d, dtype):
    parts, lses = case(n, tokens, h, d, dtype, seed=n + tokens)
    check(parts, lses, *run(parts, lses))


def test_rows_without_keys():
    parts, lses = case(3, 20, 4, 128, empty=1.0)
    out, lse = run(parts, lses)
    assert bool((out == 0).all()) and bool((lse == -float("inf")).all())


def test_one_state_is_copied():
    parts, lses = case(4, 50, 3, 128, empty=0.0)
    lses[[0, 1, 3]] = -float("inf")
    parts[[0, 1, 3]] = float("nan")
    out, lse = run(parts, lses)
    assert torch.equal(out, parts[2]) and torch.allclose(lse, lses[2], rtol=2e-7)


def test_nan_stays_in_its_row():
    parts, lses = case(3, 9, 4, 128, empty=0.0)
    clean = run(parts, lses)
    lses[1, 2, 5] = float("nan")
    parts[2, 7, 1, 30] = float("nan")
    parts[2, 7, 1, 31] = float("inf")
    out, lse = run(parts, lses)
    assert bool(out[5, 2].isnan().all()) and bool(lse[2, 5].isnan())
    assert bool(out[7, 1, 30].isnan()) and float(out[7, 1, 31]) == float("inf")
    bad = torch.zeros(9, 4, 128, dtype=torch.bool)
    bad[5, 2] = bad[7, 1, 30:32] = True
    assert torch.equal(out[~bad], clean[0][~bad])
    assert int((lse != clean[1]).sum()) == 1


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strides_and_in_place(dtype):
    parts, lses = case(3, 60, 5, 128, dtype)
    wide = torch.zeros(60, 3, 5, 200, dtype=dtype)
    wide[..., 8:136] = parts.permute(1, 0, 2, 3)
    out, lse = torch.zeros(60, 9, 128, dtype=torch.bfloat16, device=DEV), torch.zeros(60, 5, 2, device=DEV)
    binding.mla_merge_states(wide.to(DEV)[..., 8:136].permute(1, 0, 2, 3), lses.permute(0, 2, 1).contiguous().to(DEV).permute(0, 2, 1),
                             out[:, 2:7], lse[..., 1].T)
    check(parts, lses, out[:, 2:7].cpu(), lse[..., 1].T.cpu())
    assert bool((out[:, :2] == 0).all()) and bool((out[:, 7:] == 0).all()) and bool((lse[..., 0] == 0).all())
    if dtype == torch.bfloat16:
        p, l = parts.to(DEV), lses.to(DEV)
        for i in (0, 2):
            a, b = p.clone(), l.clone()
            binding.mla_merge_states(a, b, a[i], b[i])
            check(parts, lses, a[i].cpu(), b[i].cpu())


def test_decode_states():
    """mla_decode's log-sum-exps [batch, h, 1] as they are."""
    parts, lses = case(2, 64, 128, 512)
    stacked = lses.permute(0, 2, 1).contiguous().view(2, 64, 128, 1).to(DEV)
    out, lse = torch.zeros(64, 128, 512, dtype=torch.bfloat16, device=DEV), torch.zeros(64, 128, 1, device=DEV)
    binding.mla_merge_states(parts.to(DEV), stacked[..., 0].transpose(1, 2), out, lse[..., 0].T)
    check(parts, lses, out.cpu(), lse[..., 0].T.cpu())
