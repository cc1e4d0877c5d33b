"""GPU parity of mla_prefill against the fp64 definition.

Tolerances.  A weight is rounded to bf16 once (half a step, 2^-8 relative) and the sum that
divides is fp32, of the unrounded ones, so an output is off by at most
2^-8 sum w |v|, by its own rounding, 2^-8 |out|, and by what the scores' fp32 arithmetic
leaves: 192 products and their sum, 192 * 2^-23 of sum |q k| * scale, here below 20 * 192 * 2^-23 =
5e-4 in a score and a weight; 2^-10 of sum w |v| covers it.  The rounding errors are
independent, so over a whole call their root mean square is far lower: rel-L2
3e-3, and LSE 1e-3, as for every attention here."""
import numpy as np
import pytest
import torch

import oracle
from mla_decode_attention_gb300 import binding
from tests._util import LSE_ABS, OUT_REL_L2, f64_np
from tests.test_gpu_append import DEV, library  # noqa: F401

pytestmark = pytest.mark.gpu


def starts(lens, at=0):
    return [at] + (at + np.cumsum(lens)).tolist()


def case(q_lens, k_lens, h, h_k=None, rope="shared", causal=True, seed=0, gap=0, scale=1.5, before=0, behind=0):
    """``before``, ``behind``: rows of no sequence, NaN in every input."""
    g = torch.Generator().manual_seed(seed)
    h_k = h_k or h
    cu_q, cu_k = starts(q_lens, before), starts(k_lens, before)
    nq, nk = cu_q[-1] + behind, cu_k[-1] + behind
    make = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)  # noqa: E731
    d = 128 if rope == "none" else 192
    q, both = scale * make(nq, h, d + gap), make(nk, h_k, 256 + gap)
    turned = None if rope == "none" else (make(nk, 64 + 8 * (gap > 0)) if rope == "shared" else make(nk, h_k, 64 + gap))
    for t, cu in ((q, cu_q), (both, cu_k), (turned, cu_k)):
        if t is not None:
            t[:cu[0]] = float("nan")
            t[cu[-1]:] = float("nan")
    return dict(q=q[..., gap:], k=both[..., :128], v=both[..., 128:256], rope=None if turned is None else turned[..., turned.shape[-1] - 64:],
                cu_q=cu_q, cu_k=cu_k, scale=d ** -0.5, causal=causal)


def run(c, parts=None, out=None, stream=None):
    gpu = lambda t: None if t is None else t.to(DEV)  # noqa: E731

    def on_gpu(t):
        """The same strides there."""
        if t is None:
            return None
        whole = torch.empty(t.untyped_storage().nbytes() // 2, dtype=t.dtype, device=DEV)
        whole.copy_(torch.empty(0, dtype=t.dtype).set_(t.untyped_storage()))
        return whole.as_strided(t.shape, t.stride(), t.storage_offset())
    nq, h, _ = c["q"].shape
    buf = binding.PrefillBuffers(nq, c["k"].shape[0], len(c["cu_q"]) - 1, h, c["k"].shape[1], DEV, parts)
    dst = buf.out if out is None else out
    dst.fill_(9.0)
    buf.lse.fill_(9.0)
    if buf.workspace is not None:
        buf.workspace.fill_(float("nan"))
    cu = [torch.tensor(x, dtype=torch.int32) for x in (c["cu_q"], c["cu_k"])]
    binding.mla_prefill(on_gpu(c["q"]), on_gpu(c["k"]), on_gpu(c["v"]), gpu(cu[0]), gpu(cu[1]), c["scale"], c["causal"], buf.num_sm_parts,
                        buf.workspace, dst, buf.lse, on_gpu(c["rope"]), buf.err, stream)
    torch.cuda.synchronize()
    c["err"] = int(buf.err.item())
    return dst.cpu(), buf.lse.cpu()


def definition(c):
    f = lambda t: None if t is None else f64_np(t)  # noqa: E731
    return oracle.packed_attention(f(c["q"]), f(c["k"]), f(c["v"]), c["cu_q"], c["cu_k"], c["scale"], c["causal"], f(c["rope"]))


def check(c, out, lse, what="", rel=OUT_REL_L2):
    assert c["err"] == 0
    want, want_lse, size = definition(c)
    live = slice(c["cu_q"][0], c["cu_q"][-1])
    o, l = f64_np(out), f64_np(lse)
    for part in (slice(0, live.start), slice(live.stop, None)):
        assert np.all(o[part] == 9.0) and np.all(l[:, part] == 9.0), f"{what}: rows of no sequence"
    o, l, want, want_lse, size = o[live], l[:, live], want[live], want_lse[:, live], size[live]
    none = np.isneginf(want_lse)
    assert np.array_equal(none, np.isneginf(l)), what
    assert np.all(np.isfinite(o)), what
    assert np.all(o.transpose(1, 0, 2)[none] == 0.0), what
    assert not none.size or np.max(np.abs(np.where(none, 0.0, l) - np.where(none, 0.0, want_lse)), initial=0.0) <= LSE_ABS, what
    off = np.abs(o - want) - (2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2.0 ** -10) * size)
    assert np.max(off, initial=-1.0) <= 0.0, f"{what}: {np.max(off)} at {np.unravel_index(np.argmax(off), off.shape)}"
    norm = np.linalg.norm(want)
    if norm > 0:
        assert np.linalg.norm(o - want) <= rel * norm, f"{what}: {np.linalg.norm(o - want) / norm}"


@pytest.mark.parametrize("q_lens", [[1], [2], [127], [128], [129], [255], [256], [257], [384], [511, 1, 300]])
@pytest.mark.parametrize("rope", ["shared", "none"])
@pytest.mark.parametrize("causal", [True, False])
def test_lengths(q_lens, rope, causal):
    c = case(q_lens, q_lens, 3, rope=rope, causal=causal, seed=sum(q_lens))
    check(c, *run(c))


@pytest.mark.parametrize("q_lens,k_lens", [
    ([0, 5, 0, 0, 130, 0], [0, 5, 3, 0, 130, 0]), ([7], [0]), ([300, 5], [20, 0]), ([200, 300, 1], [500, 1000, 77]),
    ([129], [128]), ([260], [3]), ([1] * 70, list(range(70))), ([5], [1400]), ([256] * 3, [1290, 256, 640])])
@pytest.mark.parametrize("causal", [True, False])
def test_queries_and_keys_of_different_number(q_lens, k_lens, causal):
    """Empty sequences and sets of keys, more queries than keys (the first see none), chunks over a context."""
    c = case(q_lens, k_lens, 2, causal=causal, seed=len(q_lens) + sum(k_lens))
    check(c, *run(c))


@pytest.mark.parametrize("h,h_k", [(1, 1), (5, 1), (6, 2), (24, 3), (16, 1), (48, 1), (96, 1), (128, 1), (64, 8), (130, 10)])
@pytest.mark.parametrize("rope", ["shared", "own", "none"])
def test_grouped_heads(h, h_k, rope):
    c = case([37, 150, 1], [37, 200, 90], h, h_k, rope, seed=h + h_k)
    check(c, *run(c))


@pytest.mark.parametrize("q_lens,k_lens,h,h_k", [([300, 7], [300, 7], 320, 40), ([2900], [2900], 2, 2), ([500, 1000], [1500, 1000], 44, 11)])
def test_blocks_beside_each_other(q_lens, k_lens, h, h_k):
    """More blocks of a head's rows than run side by side, heads in more than one group, both with a remainder."""
    c = case(q_lens, k_lens, h, h_k, seed=h)
    check(c, *run(c))


def test_rows_of_no_sequence_are_left_and_leave_no_trace():
    for before, behind in ((0, 50), (17, 0), (200, 300)):
        c = case([100, 33], [130, 64], 4, before=before, behind=behind)
        check(c, *run(c), f"{before} before, {behind} behind")


@pytest.mark.parametrize("gap", [8, 64])
def test_strides(gap):
    """Queries, keys and position columns that lie among others; heads outside tokens; one token, one head."""
    for q_lens, h, h_k, rope in (([70, 200], 4, 2, "shared"), ([70, 200], 4, 2, "own"), ([1], 3, 3, "shared"), ([65], 1, 1, "none")):
        c = case(q_lens, q_lens, h, h_k, rope, gap=gap)
        check(c, *run(c), f"{h}")
        for name in ("q", "k", "v"):
            c[name] = c[name].transpose(0, 1).contiguous().transpose(0, 1)
        n = c["q"].shape[0]
        out = torch.empty(h, n, 128, dtype=torch.bfloat16, device=DEV).transpose(0, 1)
        check(c, *run(c, out=out), f"{h} head by head")
        wide = torch.empty(n, h, 128 + gap, dtype=torch.bfloat16, device=DEV)
        wide.fill_(5.0)
        check(c, *run(c, out=wide[..., gap:]), f"{h} wide")
        assert bool((wide[..., :gap] == 5.0).all())


@pytest.mark.parametrize("q_lens,k_lens,h,causal", [([3], [4000], 2, False), ([16, 1], [2600, 2100], 4, True), ([200], [1300], 1, True),
                                                    ([40, 0, 9], [40, 7000, 9], 2, True)])
@pytest.mark.parametrize("rope", ["shared", "none"])
def test_few_rows_are_split_over_their_keys(q_lens, k_lens, h, causal, rope):
    c = case(q_lens, k_lens, h, rope=rope, causal=causal, before=5, behind=40)
    nq, nk = c["q"].shape[0], c["k"].shape[0]
    assert binding.mla_prefill_workspace_size(nq, nk, len(q_lens), h, h, 152) > 0
    split = run(c)
    check(c, *split)
    whole = run(c, parts=1)
    check(c, *whole, "in one piece")
    for parts in (2, 37, 1000):
        check(c, *run(c, parts=parts), f"{parts} parts")


@pytest.mark.parametrize("q_lens,k_lens,h,parts", [([40], [2000], 5, 4), ([40, 3], [4000, 3800], 5, 8), ([300], [4300], 3, 4)])
@pytest.mark.parametrize("causal", [True, False])
def test_more_blocks_than_parts_are_cut_where_rounds_would_stay_part_full(q_lens, k_lens, h, parts, causal):
    c = case(q_lens, k_lens, h, causal=causal, seed=parts)
    assert binding.mla_prefill_workspace_size(sum(q_lens), sum(k_lens), len(q_lens), h, h, parts) > 0
    check(c, *run(c, parts=parts))


def test_results_do_not_depend_on_timing():
    c = case([700, 90, 333], [900, 90, 1000], 6, 2)
    first = run(c)
    for _ in range(5):
        again = run(c)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_one_key_is_copied():
    """Its weight is 1: the output is the value itself, bit for bit."""
    c = case([1, 1], [1, 1], 7)
    out, lse = run(c)
    assert torch.equal(out, c["v"])
    check(c, out, lse)


@pytest.mark.parametrize("scale", [0.0, 30.0])
def test_flat_and_peaked_weights(scale):
    c = case([300], [900], 3, scale=scale)
    if scale:  # (scores in the hundreds: their fp32 error, 192 * 2^-23 of sum |q k| * scale, reaches 1e-2 in a weight)
        out, lse = run(c)
        want, want_lse, _ = definition(c)
        assert np.linalg.norm(f64_np(out) - want) <= 6e-3 * np.linalg.norm(want)
        assert np.max(np.abs(f64_np(lse) - want_lse)) <= 1e-2
    else:
        check(c, *run(c))


def test_rising_scores_move_the_reference():
    """Keys whose scores grow along the sequence: every tile raises the rows' maximum by more than 2^8."""
    c = case([256], [1500], 2, rope="none", causal=False)
    c["q"].fill_(1.0)
    c["k"].copy_((torch.arange(1500) // 100 * 2.0).to(torch.bfloat16)[:, None, None].expand_as(c["k"]))
    check(c, *run(c))
    c["k"].copy_((-(torch.arange(1500) // 100) * 2.0).to(torch.bfloat16)[:, None, None].expand_as(c["k"]))
    check(c, *run(c), "falling")


@pytest.mark.parametrize("others", [0.0, -40.0, 40.0])
def test_first_keys_that_have_no_weight(others):
    """The first key's score is -inf, or far below the others', or far above: 40 * 2^0.5 * 128 / 128^0.5 = 640 in the exponent."""
    for first in (-float("inf"), -3000.0, 0.0, 60.0):
        c = case([70], [400], 2, rope="none", causal=False)
        c["q"].fill_(2.0 ** 0.5)
        c["k"].normal_(0, 0.05, generator=torch.Generator().manual_seed(4)).add_(others)
        c["k"][0] = first
        check(c, *run(c), f"{first}")


def test_lowest_values_in_unseen_places():
    c = case([50, 200], [90, 300], 3, before=40, behind=40)
    clean = run(c)
    low = torch.finfo(torch.bfloat16).min
    for name in ("q", "k", "v", "rope"):
        cu = c["cu_q"] if name == "q" else c["cu_k"]
        c[name][:cu[0]] = low
        c[name][cu[-1]:] = low
    out, lse = run(c)
    assert torch.equal(out, clean[0]) and torch.equal(lse, clean[1])
    for name in ("k", "v", "rope"):
        c[name][c["cu_k"][1] + 250:c["cu_k"][2]] = low       # seen by the last 50 queries only
    out, lse = run(c)
    seen = slice(0, c["cu_q"][2] - 50)
    assert torch.equal(out[seen], clean[0][seen]) and torch.equal(lse[:, seen], clean[1][:, seen])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("h,h_k", [(2, 2), (6, 2)])
def test_values_that_are_not_finite_reach_only_those_who_see_them(bad, h, h_k):
    n, m = 390, 500
    for key in (110, 130, 300, 499):  # keys 0 .. 110 are seen by all queries
        c = case([20, n, 33], [20, m, 40], h, h_k)
        clean = run(c)
        c["v"][20 + key, 1, 5] = bad
        out, lse = run(c)
        assert torch.equal(lse, clean[1])
        rows = torch.zeros(c["q"].shape[0], h, 128, dtype=torch.bool)
        first = max(0, key - (m - n))
        rows[20 + first:20 + n, (h // h_k):, 5] = True
        assert torch.equal(out[~rows], clean[0][~rows])
        assert bool((out[rows].isnan() if bad != bad else out[rows] == bad).all())


def test_what_is_not_finite_adds_up():
    """inf and -inf in one column, one seen by all and one by some; a NaN key and an infinite value."""
    c = case([20, 390, 33], [20, 390, 33], 2)
    c["v"][20 + 3, 1, 5] = float("inf")           # in the first tile: seen by queries 3 .. of the sequence
    c["v"][20 + 200, 1, 5] = -float("inf")
    c["k"][20 + 300, 1, 9] = float("nan")
    c["v"][20 + 310, 1, 7] = float("inf")
    out, lse = run(c)
    o = out[20:410, 1]
    assert bool(o[:3].isfinite().all()) and bool((o[3:200, 5] == float("inf")).all()) and bool(o[200:, 5].isnan().all())
    assert bool(o[300:].isnan().all()) and bool(o[:300, 7].isfinite().all()) and bool(lse[1, 320:410].isnan().all())


def test_keys_that_are_not_finite_reach_only_those_who_see_them():
    for key in (0, 150, 389):
        for name in ("k", "rope"):
            c = case([20, 390, 33], [20, 390, 33], 3)
            clean = run(c)
            if name == "k":
                c["k"][20 + key, 1, 100] = float("nan")
                heads = [1]
            else:
                c["rope"][20 + key, 7] = float("nan")
                heads = [0, 1, 2]
            out, lse = run(c)
            rows = torch.zeros(c["q"].shape[0], 3, dtype=torch.bool)
            rows[20 + key:410, heads] = True
            assert bool(out[rows].isnan().all()) and bool(lse.T[rows].isnan().all())
            assert torch.equal(out[~rows], clean[0][~rows]) and torch.equal(lse.T[~rows], clean[1].T[~rows])


def test_a_query_that_is_not_finite_stays_alone():
    c = case([300], [300], 2)
    clean = run(c)
    c["q"][77, 1, 3] = float("nan")
    out, lse = run(c)
    rows = torch.zeros(300, 2, dtype=torch.bool)
    rows[77, 1] = True
    assert bool(out[rows].isnan().all()) and bool(lse.T[rows].isnan().all())
    assert torch.equal(out[~rows], clean[0][~rows]) and torch.equal(lse.T[~rows], clean[1].T[~rows])


def test_ranges_that_do_not_fit_are_reported():
    c = case([100, 50], [100, 50], 2)
    for cu_q, cu_k in (([0, 100, 90], [0, 100, 150]), ([0, 100, 151], [0, 100, 150]), ([0, 100, 150], [0, 170, 150]),
                       ([-5, 100, 150], [0, 100, 150]), ([0, 100, 150], [0, 100, 2**31 - 1]), ([0, 2**31 - 1, -2**31], [0, 100, 150])):
        c["cu_q"], c["cu_k"] = cu_q, cu_k
        run(c)
        assert c["err"] == binding.MLA_DEVERR_BAD_RANGE


def test_many_sequences():
    g = np.random.default_rng(3)
    q_lens = g.integers(0, 40, 900).tolist()
    c = case(q_lens, [n + int(e) for n, e in zip(q_lens, g.integers(0, 9, 900))], 2)
    check(c, *run(c))


def test_larger_prompts():
    c = case([1500, 700], [1500, 2300], 16, 4)
    check(c, *run(c))
