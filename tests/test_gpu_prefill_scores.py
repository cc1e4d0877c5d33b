"""mla_prefill where scores are large: q and k are finite, q . k up to 2^110.

Only column 0 of q and k is not zero and q there is a power of two, so that every score is one exact product
in fp32 and the differences between a row's scores are exact too.  Tolerances: outputs as in test_gpu_prefill
(the exponent's rounding, 2^-24 of a size below 150 wherever a weight is left, is below the share of the scores'
arithmetic there).  lse: softmax_scale and log2 e rounded to fp32, their product, its product with
ln 2 and with the score, each 2^-24 of it: 2^-21 covers them; and 1e-3."""
import numpy as np
import pytest
import torch

import oracle
from mla_decode_attention_gb300 import binding
from tests._util import LSE_ABS, f64_np
from tests.test_gpu_append import DEV, library  # noqa: F401
from tests.test_gpu_prefill import case, definition, run

pytestmark = pytest.mark.gpu

EXPONENTS = (0, 10, 16, 20, 24, 26, 27, 28, 29, 30, 31, 32, 33, 36, 50, 110)


def check(c, out, lse, what):
    assert c["err"] == 0
    want, want_lse, size = definition(c)
    o, l = f64_np(out), f64_np(lse)
    none = np.isneginf(want_lse)
    assert np.array_equal(none, np.isneginf(l)), f"{what}: rows without keys"
    bad = ~(np.abs(np.where(none, 0.0, l) - np.where(none, 0.0, want_lse)) <= LSE_ABS + 2.0 ** -21 * np.abs(np.where(none, 0.0, want_lse)))
    assert not bad.any(), f"{what}: lse at {np.argwhere(bad)[:5].tolist()}"
    bad = ~(np.abs(o - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2.0 ** -10) * size)
    assert not bad.any(), f"{what}: {int(bad.any((1, 2)).sum())} tokens, out at {np.argwhere(bad)[:5].tolist()}"


def large(n, m, h, causal, rope, order, sign, seed=0):
    """Token t's query is sign * 2^e, e by turns; keys by `order` along the sequence."""
    c = case([n], [m], h, rope=rope, causal=causal, seed=seed)
    c["q"].zero_()
    e = torch.tensor([EXPONENTS[t % len(EXPONENTS)] for t in range(n)], dtype=torch.float64)
    c["q"][..., 0] = (sign * torch.exp2(e)).to(torch.bfloat16)[:, None]
    keys = torch.randn(m, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)
    if order != "any":
        keys = keys.sort(descending=order == "falling").values
    if order == "ties":                       # the two largest at both ends
        keys[0] = keys[-1] = 4.0
    c["k"].zero_()
    c["k"][..., 0] = keys[:, None]
    if c["rope"] is not None:
        c["rope"].zero_()
    return c


@pytest.mark.parametrize("order", ["any", "rising", "falling", "ties"])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("n,m,h,causal,rope", [(300, 300, 2, True, "shared"), (40, 700, 1, False, "none"), (200, 1300, 1, True, "none")])
def test_large_scores(order, sign, n, m, h, causal, rope):
    c = large(n, m, h, causal, rope, order, sign, seed=m)
    for parts in (1, 152):
        check(c, *run(c, parts=parts), f"{order} {sign} {parts} parts")


def test_large_scores_in_pieces():
    """Cut along the keys: one piece's scores far above the others', and below."""
    for order in ("rising", "falling", "any"):
        c = large(16, 4000, 2, False, "shared", order, 1.0)
        assert binding.mla_prefill_workspace_size(16, 4000, 1, 2, 2, 152) > 0
        check(c, *run(c, parts=152), order)


def test_rows_beside_large_scores_keep_their_bits():
    """Rows of ordinary scores beside rows of large ones of the same warp."""
    c = case([256], [700], 2, causal=False)
    clean = run(c)
    rows = torch.arange(0, 256, 7)
    c["q"][rows] = (c["q"][rows].float() * 2.0 ** 40).to(torch.bfloat16)
    out, lse = run(c)
    others = torch.ones(256, dtype=torch.bool)
    others[rows] = False
    assert torch.equal(out[others], clean[0][others]) and torch.equal(lse[:, others], clean[1][:, others])
    assert bool(out.isfinite().all()) and bool(lse.isfinite().all())


@pytest.mark.parametrize("ninf", [1, 128, 130])
def test_first_keys_of_minus_infinity(ninf):
    """Scores of -inf before keys whose scores are large and negative."""
    c = large(64, 400, 1, False, "none", "any", 1.0)
    c["k"][..., 0].abs_().add_(1.0).neg_()
    c["k"][:ninf, :, 0] = -float("inf")
    check(c, *run(c), f"{ninf}")
