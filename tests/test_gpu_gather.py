"""mla_gather_kv against the formats' definitions: exact for the bf16 and the 528-byte cache; for the 656-byte cache
the fp32 product rounded once, which the definition (code * scale exactly, rounded once) equals but where the fp32
product falls on a tie (then one bf16 step off)."""
import numpy as np
import pytest
import torch

import oracle
from mla_decode_attention_gb300 import binding, workloads
from tests._util import f64_np
from tests.test_gpu_append import DEV, FORMATS, library, width  # noqa: F401
from tests.test_gpu_window import keys_of

pytestmark = pytest.mark.gpu


def case(fmt, lens, first=None, seed=0, spare=2, before=0, behind=0, pages=None):
    g = torch.Generator().manual_seed(seed)
    b = len(lens)
    begin = [0] * b if first is None else first
    slots = max(1, max((s + n + 63) // 64 for s, n in zip(begin, lens)))
    n = pages or b * slots + spare
    table = torch.randperm(n, generator=g)[:b * slots].view(b, slots).int()
    x = torch.randn(n, 64, width(fmt), generator=g)
    cache = x.to(torch.bfloat16) if fmt == FORMATS[0] else (workloads.quantize_fp8_tokens(x) if fmt == FORMATS[1] else workloads.quantize_fp8_v41_tokens(x))
    cu = [before] + (before + np.cumsum(lens)).tolist()
    for i, (s, m) in enumerate(zip(begin, lens)):          # entries of pages without a token of the call
        at = torch.arange(slots)
        table[i, (at < s // 64) | (at * 64 >= s + m)] = -9
    return dict(fmt=fmt, cache=cache, table=table, cu=cu, first=first, rows=cu[-1] + behind)


def run(c, gap=0, stream=None):
    out = torch.full((c["rows"], width(c["fmt"]) + gap), 9.0, dtype=torch.bfloat16, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    first = None if c["first"] is None else torch.tensor(c["first"], dtype=torch.int32, device=DEV)
    binding.mla_gather_kv(c["cache"].to(DEV), c["fmt"], c["table"].to(DEV), torch.tensor(c["cu"], dtype=torch.int32, device=DEV), out[:, gap:],
                          first, err, stream)
    torch.cuda.synchronize()
    c["err"] = int(err.item())
    assert bool((out[:, :gap] == 9.0).all())
    return out[:, gap:].cpu()


def check(c, out):
    assert c["err"] == 0
    a, z = c["cu"][0], c["cu"][-1]
    assert bool((out[:a] == 9.0).all()) and bool((out[z:] == 9.0).all())
    want = oracle.gather_rows(keys_of(c["cache"], c["fmt"]), c["table"].numpy(), c["cu"], c["first"])
    got = f64_np(out[a:z])
    if c["fmt"] == FORMATS[1]:
        other = np.abs(got - want)
        assert np.mean(other > 0) < 1e-3
        assert np.all(other <= 2.0 ** -7 * np.abs(want))     # one step of 8 significant bits at most
        assert np.array_equal(got[:, 512:], want[:, 512:])
    else:
        assert np.array_equal(got, want)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("lens,first", [([1], None), ([64], None), ([65, 1, 0, 63], None), ([0, 0, 7, 0], [3, 0, 60, 1]),
                                        ([200, 17, 300], [1, 63, 1000]), ([1] * 100, list(range(100))), ([5, 0], [0, 5000])])
def test_rows(fmt, lens, first):
    c = case(fmt, lens, first, seed=len(lens))
    check(c, run(c))
    check(c, run(c, gap=8))


@pytest.mark.parametrize("fmt", FORMATS)
def test_rows_of_no_request_are_left(fmt):
    c = case(fmt, [30, 0, 41], [5, 5, 5], before=9, behind=70)
    check(c, run(c))


@pytest.mark.parametrize("fmt", FORMATS)
def test_many_requests(fmt):
    g = np.random.default_rng(1)
    c = case(fmt, g.integers(0, 50, 1000).tolist(), g.integers(0, 100, 1000).tolist())
    check(c, run(c))


@pytest.mark.parametrize("fmt", FORMATS)
def test_what_is_not_finite_is_read_as_it_is(fmt):
    c = case(fmt, [70])
    if fmt == FORMATS[0]:
        c["cache"][c["table"][0, 0], 3, 9] = float("nan")
        c["cache"][c["table"][0, 1], 1, 575] = -float("inf")
    else:
        c["cache"][c["table"][0, 0], 3, 9] = 0x7F            # the NaN code
    out = run(c)
    assert out[3].isnan().sum() == 1 and bool(out[3, 9].isnan())
    if fmt == FORMATS[0]:
        assert float(out[65, 575]) == -float("inf")


@pytest.mark.parametrize("fmt", FORMATS)
def test_pages_that_are_not_there_read_as_zeros(fmt):
    for entry, first in ((-1, 0), (40, 0), (2**31 - 1, 0), (None, 64 * 2 - 10), (None, -5), (None, 2**31 - 1), (None, -2**31)):
        c = case(fmt, [100], pages=40)
        if entry is not None:
            c["table"][0, 1] = entry
            lost = slice(64, 100)
        else:
            c["table"] = torch.tensor([[4, 5]], dtype=torch.int32)
            c["first"] = [first]
            lost = slice(10, 100) if first == 118 else (slice(0, 5) if first == -5 else slice(0, 100))
        out = run(c)
        assert c["err"] == binding.MLA_DEVERR_BAD_PAGE
        assert bool((out[lost] == 0).all())
        kept = torch.ones(100, dtype=torch.bool)
        kept[lost] = False
        assert bool((out[kept].float().abs().amax(1) > 0).all())


def test_pages_past_32_bits():
    """2^31 elements into a bf16 pool, 2^32 bytes into an FP8 one, and a start whose position needs no such pool."""
    for fmt in FORMATS[:2]:
        pages = (1 << 32) // (64 * (1152 if fmt == FORMATS[0] else 656)) + 40
        shape = (pages, 64, 576 if fmt == FORMATS[0] else 656)
        cache = torch.zeros(shape, dtype=torch.bfloat16 if fmt == FORMATS[0] else torch.uint8, device=DEV)
        row = torch.randn(1, 64, 576)
        part = row.to(torch.bfloat16) if fmt == FORMATS[0] else workloads.quantize_fp8_tokens(row)
        cache[-1:] = part.to(DEV)
        table = torch.tensor([[0, pages - 1]], dtype=torch.int32, device=DEV)
        out = torch.zeros(64, 576, dtype=torch.bfloat16, device=DEV)
        binding.mla_gather_kv(cache, fmt, table, torch.tensor([0, 64], dtype=torch.int32, device=DEV), out,
                              torch.tensor([64], dtype=torch.int32, device=DEV))
        c = dict(fmt=fmt, cache=part, table=torch.zeros(1, 1, dtype=torch.int32), cu=[0, 64], first=None, err=0)
        check(c, out.cpu())
        del cache
