"""mla_prefill cut along the keys with inputs that are not finite, sequences by falling length past the first 32, and
strides past 2^31 elements."""
import numpy as np
import pytest
import torch

from mla_decode_attention_gb300 import binding
from tests.test_gpu_append import DEV, library  # noqa: F401
from tests.test_gpu_prefill import case, check, run

pytestmark = pytest.mark.gpu

N, M = 200, 1300     # queries and keys of the cut calls: query j sees keys 0 .. j + 1100


def cut(h=1, rope="shared"):
    c = case([N], [M], h, rope=rope)
    assert binding.mla_prefill_workspace_size(N, M, 1, h, h, 152) > 0
    return c


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("rope", ["shared", "none"])
def test_values_that_are_not_finite(bad, rope):
    for key in (0, 5, 127, 128, 255, 256, 640, 1099, 1100, 1101, 1151, 1152, 1279, 1280, 1299):
        c = cut(rope=rope)
        clean = run(c)
        c["v"][key, 0, 77] = bad
        out, lse = run(c)
        rows = torch.zeros(N, 1, 128, dtype=torch.bool)
        rows[max(0, key - (M - N)):, :, 77] = True
        assert torch.equal(lse, clean[1]) and torch.equal(out[~rows], clean[0][~rows]), key
        assert bool((out[rows].isnan() if bad != bad else out[rows] == bad).all()), key


def test_what_is_not_finite_adds_up():
    """inf in the first piece, -inf in an edge tile of the last, both in one column; a NaN key behind."""
    c = cut()
    c["v"][3, 0, 5] = float("inf")
    c["v"][1200, 0, 5] = -float("inf")
    c["k"][1290, 0, 9] = float("nan")
    c["v"][1250, 0, 7] = float("inf")
    out, lse = run(c)
    assert bool((out[:100, 0, 5] == float("inf")).all()) and bool(out[100:, 0, 5].isnan().all())
    assert bool(out[:150, 0, 7].isfinite().all()) and bool((out[150:190, 0, 7] == float("inf")).all())
    assert bool(out[190:].isnan().all()) and bool(lse[:, 190:].isnan().all()) and bool(lse[:, :190].isfinite().all())


@pytest.mark.parametrize("name", ["k", "rope"])
def test_keys_that_are_not_finite(name):
    for key in (0, 127, 128, 700, 1100, 1152, 1299):
        c = cut(2)
        clean = run(c)
        heads = [1] if name == "k" else [0, 1]
        if name == "k":
            c["k"][key, 1, 100] = float("nan")
        else:
            c["rope"][key, 7] = float("nan")
        out, lse = run(c)
        rows = torch.zeros(N, 2, dtype=torch.bool)
        rows[max(0, key - (M - N)):, heads] = True
        assert bool(out[rows].isnan().all()) and bool(lse.T[rows].isnan().all()), key
        assert torch.equal(out[~rows], clean[0][~rows]) and torch.equal(lse.T[~rows], clean[1].T[~rows]), key


def test_a_query_that_is_not_finite_stays_alone():
    c = cut(2)
    clean = run(c)
    c["q"][77, 1, 3] = float("nan")
    out, lse = run(c)
    rows = torch.zeros(N, 2, dtype=torch.bool)
    rows[77, 1] = True
    assert bool(out[rows].isnan().all()) and bool(lse.T[rows].isnan().all())
    assert torch.equal(out[~rows], clean[0][~rows]) and torch.equal(lse.T[~rows], clean[1].T[~rows])


@pytest.mark.parametrize("h,h_k", [(6, 6), (40, 5)])
def test_more_sequences_than_are_sorted_at_once(h, h_k):
    """70 sequences of 1 to 900 keys, some empty, some of one length, more items than SMs."""
    g = np.random.default_rng(7)
    k_lens = g.integers(1, 900, 70).tolist()
    k_lens[5] = k_lens[40] = 0
    k_lens[10:14] = [640] * 4
    q_lens = [int(g.integers(0, n + 1)) for n in k_lens]
    q_lens[20] = 0
    c = case(q_lens, k_lens, h, h_k)
    assert sum(-(-n // (256 // (h // h_k))) for n in q_lens) * h_k > 152
    check(c, *run(c))


def test_strides_past_2_31_elements():
    """Queries, keys, values and outputs whose rows lie far apart: the last ones begin past 2^31 elements."""
    n, m, h = 300, 300, 2
    c = case([n], [m], h)
    apart = 1 << 23                                    # 300 rows of 16 MB: 2^31.2 elements
    dev = {}
    for name in ("q", "k", "v", "rope"):
        t = c[name]
        far = torch.empty((n - 1) * apart + 1024, dtype=torch.bfloat16, device=DEV)
        dev[name] = far.as_strided(t.shape, (apart,) + ((192, 1) if t.dim() == 3 else (1,)))
        dev[name].copy_(t.to(DEV))
    out = torch.empty((n - 1) * apart + 1024, dtype=torch.bfloat16, device=DEV).as_strided((n, h, 128), (apart, 128, 1))
    buf = binding.PrefillBuffers(n, m, 1, h, h, DEV)
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    dev["v"][170, 1, 5] = float("inf")                 # (read again from its place in memory)
    c["v"][170, 1, 5] = 0.0
    binding.mla_prefill(dev["q"], dev["k"], dev["v"], cu, cu, c["scale"], True, buf.num_sm_parts, buf.workspace, out, buf.lse,
                        dev["rope"], buf.err)
    torch.cuda.synchronize()
    c["err"] = int(buf.err.item())
    got = out.cpu()
    assert bool((got[170:, 1, 5] == float("inf")).all()) and bool(got[:170].isfinite().all())
    plain = dev["v"].clone()
    plain[170, 1, 5] = 0.0
    binding.mla_prefill(dev["q"], dev["k"], plain, cu, cu, c["scale"], True, buf.num_sm_parts, buf.workspace, out, buf.lse,
                        dev["rope"], buf.err)
    check(c, out.cpu(), buf.lse.cpu())
