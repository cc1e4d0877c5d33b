"""mla_window_decode where keys that are not finite are seen: a token that sees a
NaN gets what its formula gives, NaN in every column and in lse, and is not taken
for a token that sees no key (0 and -inf); a token that does not see it is as if
it were not there, whichever tokens share its block of query rows."""
import numpy as np
import pytest
import torch

import oracle
from mla_decode_attention_gb300 import binding
from tests._util import assert_parity, f64_np
from tests.test_gpu_append import DEV, library  # noqa: F401
from tests.test_gpu_window import BF16, FP8_528, FP8_656, SCALE, case, keys_of

pytestmark = pytest.mark.gpu

KINDS = [(BF16, 128), (BF16, 64), (BF16, 16), (FP8_656, 128), (FP8_656, 48), (FP8_528, 32)]
NAN, INF = float("nan"), float("inf")


def spoil(c, b, t, value, column=5):
    """A value that is not finite in one column of request b's key t."""
    page, slot = int(c["table"][b, t // 64]), t % 64
    assert page >= 0
    if c["fmt"] == BF16:
        c["cache"][page, slot, column] = value
    elif column < 512:
        assert np.isnan(value)
        c["cache"][page, slot, column] = 0x7F                       # the e4m3 NaN
    else:
        c["cache"][page, slot, 528:].view(torch.bfloat16)[column - 512] = value


def run(c, parts=None):
    """As it is called, whatever it answers."""
    b, s, h, _ = c["q"].shape
    buf = binding.WindowBuffers(b, s, h, c["window"], c["sinks"], DEV, parts)
    gpu = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    binding.mla_window_decode(gpu(c["q"]), gpu(c["cache"]), c["fmt"], gpu(c["table"]), gpu(c["lens"]), SCALE, c["window"], c["sinks"],
                              buf.num_sm_parts, buf.workspace, buf.out, buf.lse, buf.err, None, gpu(c["logits"]), gpu(c["new"]))
    torch.cuda.synchronize()
    assert int(buf.err.item()) == 0
    return f64_np(buf.out), f64_np(buf.lse)


def check(c, bad, out, lse):
    """Tokens that see one of the keys `bad` [(request, position)] are NaN; the
    others as if those keys were any finite row."""
    new = None if c["new"] is None else c["new"].tolist()
    pos = oracle.token_positions(c["lens"].tolist(), new, c["q"].shape[1])
    keys = keys_of(c["cache"], c["fmt"])
    table = c["table"].numpy().clip(0)
    clean = np.array(keys)
    for b, t in bad:
        clean[table[b, t // 64], t % 64] = 0.0
    ro, rl = oracle.window_decode(f64_np(c["q"]), clean, table, c["lens"].tolist(), new, SCALE, c["window"], c["sinks"],
                                  None if c["logits"] is None else c["logits"].numpy())
    hit = 0
    for b in range(pos.shape[0]):
        for j in range(pos.shape[1]):
            p = int(pos[b, j])
            if p < 0:
                assert np.all(out[b, j] == 0) and np.all(np.isneginf(lse[b, :, j]))
            elif set(oracle.window_keys(p, c["window"], c["sinks"]).tolist()) & {t for r, t in bad if r == b}:
                hit += 1
                assert np.all(np.isnan(out[b, j])) and np.all(np.isnan(lse[b, :, j])), f"token ({b}, {j})"
            else:
                assert_parity(out[b, j], ro[b, j], lse[b, :, j], rl[b, :, j], f"token ({b}, {j})")
    assert hit


@pytest.mark.parametrize("fmt,h", KINDS)
@pytest.mark.parametrize("logits", [False, True])
def test_a_token_that_sees_nan_is_nan(fmt, h, logits):
    """In the first tile, at tile and page borders, in the newest key, in a first
    token; one request all of whose keys are NaN, others untouched."""
    c = case(fmt, [1, 63, 129, 300, 300, 700, 700, 0, 4], 1, h, 260, 3, seed=41, logits=logits)
    bad = [(0, 0), (2, 128), (3, 127), (4, 40), (5, 1), (6, 600), (8, 0), (8, 1), (8, 2), (8, 3)]
    for b, t in bad:
        spoil(c, b, t, NAN)
    check(c, bad, *run(c))


@pytest.mark.parametrize("fmt,h", KINDS)
@pytest.mark.parametrize("parts", [None, 3, 10])
def test_in_one_piece_of_a_token_that_is_cut(fmt, h, parts):
    c = case(fmt, [2200, 1700, 1999], 1, h, 1500, 200, seed=42, logits=True)
    assert parts or binding.mla_window_workspace_size(3, 1, h, 1500, 200, binding.mla_num_sm_parts(0, h)) > 0
    bad = [(0, 2199), (2, 7)]
    for b, t in bad:
        spoil(c, b, t, NAN)
    check(c, bad, *run(c, parts))


@pytest.mark.parametrize("fmt,h", [k for k in KINDS if k[0] != FP8_528])
def test_nan_in_the_rotated_columns_alone(fmt, h):
    c = case(fmt, [200, 130, 64], 1, h, 100, 0, seed=43)
    spoil(c, 1, 129, NAN, 530)
    check(c, [(1, 129)], *run(c))


@pytest.mark.parametrize("h", [128, 64, 16])
def test_infinite_scores(h):
    """An infinite key: heads with score +inf are NaN (inf - inf), heads with
    score -inf give it no weight: their other columns are as without it."""
    c = case(BF16, [300, 200], 1, h, 260, 0, seed=44)
    spoil(c, 0, 150, INF, 7)
    out, lse = run(c)
    up = f64_np(c["q"])[0, 0, :, 7] > 0
    assert up.any() and not up.all()
    assert np.all(np.isnan(out[0, 0, up])) and np.all(np.isnan(lse[0, up, 0]))
    table = c["table"].numpy().clip(0)
    q = f64_np(c["q"])[0, 0, ~up]
    t = np.array([t for t in oracle.window_keys(299, 260, 0) if t != 150])
    ro, rl = oracle.attend(q, keys_of(c["cache"], BF16)[table[0, t // 64], t % 64], SCALE)
    rest = np.arange(512) != 7
    assert_parity(out[0, 0][~up][:, rest], ro[:, rest], lse[0, ~up, 0], rl)


BLOCKS = [(BF16, 128), (BF16, 64), (BF16, 48), (BF16, 32), (BF16, 16), (FP8_656, 64), (FP8_656, 32), (FP8_656, 16), (FP8_528, 32), (FP8_528, 16)]


@pytest.mark.parametrize("fmt,h", BLOCKS)
@pytest.mark.parametrize("s", [2, 3, 8, 11])
def test_keys_that_some_tokens_of_a_block_see(fmt, h, s):
    """NaN in a request's newest key, in an older new one, in the oldest that its
    first tokens see, in a first token, at page and tile borders."""
    lens = [300, 129, 200, 64 + s, 500, 257, 700]
    c = case(fmt, lens, s, h, 60, 3, seed=45, logits=True)
    bad = [(0, 299), (1, 129 - s + 1), (2, 200 - s - 59), (3, 63 + s), (4, 500 - 60), (5, 256), (5, 255 - s // 2)]
    for b, t in bad:
        spoil(c, b, t, NAN)
    out, lse = run(c)
    check(c, bad, out, lse)
    assert not np.any(np.isnan(out[6])) and not np.any(np.isnan(out[:6, 0][[0, 1, 3]]))


@pytest.mark.parametrize("fmt,h", BLOCKS)
def test_a_chunk_with_padding_and_many_bad_keys(fmt, h):
    c = case(fmt, [170, 150, 131], 40, h, 30, 5, new=[40, 33, 9], seed=46)
    g = torch.Generator().manual_seed(47)
    bad = sorted({(b, int(t)) for b, (L, n) in enumerate([(170, 40), (150, 33), (131, 9)])
                  for t in torch.randint(L - n - 29, L, (6,), generator=g)})
    for i, (b, t) in enumerate(bad):
        spoil(c, b, t, NAN, 83 * i % 512)
    check(c, bad, *run(c))
    check(c, bad, *run(c, 3))


@pytest.mark.parametrize("fmt,h", [k for k in BLOCKS if k[1] < 64])
def test_blocks_of_tokens_that_are_cut(fmt, h):
    """Long windows: the keys that some tokens see are in the first and last of
    many pieces."""
    c = case(fmt, [1900, 1500, 64], 11, h, 1200, 3, seed=48, logits=True)
    bad = [(0, 1899), (0, 1895), (1, 1500 - 1200 - 5), (2, 60)]
    for b, t in bad:
        spoil(c, b, t, NAN)
    check(c, bad, *run(c))


@pytest.mark.parametrize("h", [16, 48, 64])
@pytest.mark.parametrize("value", [INF, -INF])
def test_infinite_keys_stay_with_the_tokens_that_see_them(h, value):
    c = case(BF16, [300, 200], 4, h, 90, 0, seed=49)
    ref = run(c)
    for b, t in [(0, 298), (1, 200 - 4 - 89)]:
        for column in range(0, 512, 37):
            spoil(c, b, t, value, column)
    out, lse = run(c)
    for b, j in [(0, 0), (0, 1), (1, 1), (1, 2), (1, 3)]:
        assert np.array_equal(out[b, j], ref[0][b, j]) and np.array_equal(lse[b, :, j], ref[1][b, :, j])
