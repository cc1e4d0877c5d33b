"""GPU parity of mla_window_decode against the fp64 oracle, with the bounds of
every other decode (out rel-L2 3e-3, max-abs 2e-2 of the token's RMS beyond one
bf16 rounding, LSE 1e-3), applied to every query token; tokens that see no key
exactly 0 and -inf; single-key rows exact copies.  Every cache slot and page
that no token of the call sees holds NaN."""
import numpy as np
import pytest
import torch

import oracle
from mla_decode_attention_gb300 import binding, workloads
from tests._util import LSE_ABS, OUT_REL_L2, assert_parity, f64_np
from tests.test_gpu_append import DEV, library  # noqa: F401

pytestmark = pytest.mark.gpu

BF16, FP8_656, FP8_528 = binding.MLA_KV_BF16, binding.MLA_KV_FP8_656, binding.MLA_KV_FP8_528
SCALE = workloads.SOFTMAX_SCALE


def keys_of(cache, fmt):
    """Cache pool -> keys in float64."""
    if fmt == BF16:
        return f64_np(cache)
    if fmt == FP8_656:
        return oracle.fp8_tokens_to_keys(cache.numpy())
    return oracle.fp8_v41_tokens_to_f64(cache.numpy())


def case(fmt, lens, s, h, window, sinks, new=None, seed=0, logits=False, spare=2):
    g = torch.Generator().manual_seed(seed)
    b, d = len(lens), 512 if fmt == FP8_528 else 576
    slots = max(1, (max(lens) + 63) // 64)
    n = b * slots + spare
    table = torch.randperm(n, generator=g)[:b * slots].view(b, slots).int()
    x = torch.randn(n, 64, d, generator=g)
    cache = x.to(torch.bfloat16) if fmt == BF16 else (workloads.quantize_fp8_tokens(x) if fmt == FP8_656 else workloads.quantize_fp8_v41_tokens(x))
    pos = oracle.token_positions(lens, new, s)
    live = torch.zeros(n, 64, dtype=torch.bool)
    for bi in range(b):
        seen = set()
        for p in pos[bi]:
            seen.update(oracle.window_keys(int(p), window, sinks).tolist() if p >= 0 else [])
        at = torch.tensor(sorted(seen), dtype=torch.long)
        live[table[bi, at // 64].long(), at % 64] = True
        gone = sorted(set(range(slots)) - set((at // 64).tolist()))
        table[bi, gone] = -7                      # pages given away: never looked at
    if fmt == BF16:
        cache[~live] = float("nan")
    else:
        cache[~live] = 0xFF                        # NaN codes, scales and columns
    return dict(fmt=fmt, live=live, lens=torch.tensor(lens, dtype=torch.int32), new=None if new is None else torch.tensor(new, dtype=torch.int32),
                cache=cache, table=table, q=torch.randn(b, s, h, d, generator=g).to(torch.bfloat16), window=window, sinks=sinks,
                logits=torch.randn(h, generator=g) if logits else None)


def run(c, parts=None):
    b, s, h, _ = c["q"].shape
    buf = binding.WindowBuffers(b, s, h, c["window"], c["sinks"], DEV, parts)
    buf.out.fill_(9.0)
    buf.lse.fill_(9.0)
    gpu = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    binding.mla_window_decode(gpu(c["q"]), gpu(c["cache"]), c["fmt"], gpu(c["table"]), gpu(c["lens"]), SCALE, c["window"], c["sinks"],
                              buf.num_sm_parts, buf.workspace, buf.out, buf.lse, buf.err, None, gpu(c["logits"]), gpu(c["new"]))
    torch.cuda.synchronize()
    assert int(buf.err.item()) == 0
    return buf.out.cpu(), buf.lse.cpu()


def check(c, out, lse):
    keys = keys_of(c["cache"], c["fmt"])
    table = c["table"].numpy().clip(0)
    new = None if c["new"] is None else c["new"].tolist()
    ro, rl = oracle.window_decode(f64_np(c["q"]), keys, table, c["lens"].tolist(), new, SCALE, c["window"], c["sinks"],
                                  None if c["logits"] is None else c["logits"].numpy())
    out, lse = f64_np(out), f64_np(lse)
    empty = oracle.token_positions(c["lens"].tolist(), new, c["q"].shape[1]) < 0
    assert np.all(out[empty] == 0) and np.all(np.isneginf(lse.transpose(0, 2, 1)[empty]))
    for b, j in zip(*np.nonzero(~empty)):
        assert_parity(out[b, j], ro[b, j], lse[b, :, j], rl[b, :, j], f"token ({b}, {j})")


def parity(*a, parts=None, **kw):
    c = case(*a, **kw)
    check(c, *run(c, parts))


LENS = [1, 63, 64, 65, 127, 128, 129, 200, 1000]
KINDS = [(BF16, 128), (BF16, 64), (BF16, 16), (FP8_656, 128), (FP8_656, 48), (FP8_528, 128), (FP8_528, 32)]


@pytest.mark.parametrize("fmt,h", KINDS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (64, 1), (65, 0), (128, 4), (129, 65), (200, 130), (2**31 - 1, 0), (100, 2**31 - 1)])
def test_single_tokens(fmt, h, window, sinks):
    parity(fmt, LENS, 1, h, window, sinks, seed=window % 1000 + sinks % 7)


@pytest.mark.parametrize("fmt,h", KINDS)
@pytest.mark.parametrize("s,new", [(2, None), (5, [5, 0, 3, 1, 5, 2, 4, 9, -1])])
def test_several_tokens_padding_and_sink_logits(fmt, h, s, new):
    parity(fmt, [3, 64, 66, 0, 130, 700, 258, 64, 90], s, h, 100, 3, new=new, seed=s, logits=True)


@pytest.mark.parametrize("fmt,h", KINDS)
def test_few_tokens_are_cut_into_pieces(fmt, h):
    """Long windows of few tokens: pieces, workspace, combine; lengths far below
    the window leave pieces empty."""
    c = case(fmt, [2200, 70, 1], 1, h, 1500, 200, seed=5, logits=True)
    assert binding.mla_window_workspace_size(3, 1, h, 1500, 200, binding.mla_num_sm_parts(0, h)) > 0
    check(c, *run(c))
    for parts in (1, 3, 10):
        check(c, *run(c, parts))


@pytest.mark.parametrize("fmt,h", [(BF16, 128), (BF16, 64), (FP8_656, 64), (FP8_528, 128)])
@pytest.mark.parametrize("parts", [1, 2, 5])
def test_long_windows_one_after_the_other(fmt, h, parts):
    """Every part walks several tokens with many tiles all of whose keys are
    seen between the tiles at the window's ends, which have keys that are not."""
    parity(fmt, [1100, 1900, 1333, 1500, 1920], 2, h, 1000, 70, seed=12, parts=parts)


@pytest.mark.parametrize("fmt,h", [(BF16, 128), (BF16, 16), (BF16, 48), (BF16, 32), (BF16, 64), (FP8_656, 64), (FP8_656, 16),
                                   (FP8_528, 128), (FP8_528, 32)])
@pytest.mark.parametrize("window,sinks", [(70, 5), (3, 0)])
def test_a_chunk_of_a_prompt(fmt, h, window, sinks):
    """Many tokens a request, several of them in a block of query rows with few
    heads: every part walks several pieces, blocks begin and end with padding."""
    parity(fmt, [170, 150, 131], 133, h, window, sinks, new=[133, 121, 9], seed=6, parts=20)


@pytest.mark.parametrize("fmt,h", [(BF16, 128), (BF16, 64), (FP8_656, 64)])
def test_parts_that_begin_with_padding(fmt, h):
    """The first item of a part, or of every part, has no token; some parts have
    nothing to do at all."""
    parity(fmt, [100, 90, 0, 0, 0, 300], 6, h, 50, 2, new=[0, 6, 6, 6, 0, 1], seed=14, parts=4)
    parity(fmt, [0, 0, 70], 2, h, 50, 0, new=[0, 1, 2], seed=15)
    parity(fmt, [0], 1, h, 50, 0, seed=16)
    parity(fmt, [0, 2000], 1, h, 1500, 1, seed=17)


@pytest.mark.parametrize("fmt,h,s", [(BF16, 128, 75), (BF16, 16, 290), (BF16, 48, 150), (BF16, 64, 1), (FP8_656, 128, 75), (FP8_528, 32, 150)])
@pytest.mark.parametrize("parts", [1, 2])
def test_parts_that_walk_many_items(fmt, h, s, parts):
    """More items a part than are planned at a time, a good part of them without
    a token."""
    if s > 1:
        parity(fmt, [s + 40, s - 7], s, h, 70, 5, new=[s, s - 20], seed=21, parts=parts)
    else:
        parity(fmt, [(37 * i) % 260 for i in range(150)], 1, h, 70, 5, new=[i % 3 for i in range(150)], seed=22, parts=parts)


@pytest.mark.parametrize("fmt,h", [(BF16, 128), (FP8_656, 64)])
def test_parts_that_walk_many_items_and_cut_the_last(fmt, h):
    assert binding.mla_window_workspace_size(52, 3, h, 1000, 3, 5) > 0
    parity(fmt, [300 + 16 * i for i in range(52)], 3, h, 1000, 3, seed=23, parts=5)


@pytest.mark.parametrize("fmt,h,first", [(BF16, 128, 58250), (BF16, 16, 58250), (FP8_656, 64, 102295), (FP8_528, 32, 127095)])
def test_pages_past_32_bits(fmt, h, first):
    """The request's pages lie on either side of 2^32 bytes."""
    c = case(fmt, [300, 500], 2, h, 200, 70, seed=24)
    ref = run(c)
    n = c["cache"].shape[0]
    big = torch.empty(first + n, *c["cache"].shape[1:], dtype=c["cache"].dtype, device=DEV)
    assert big.numel() * big.element_size() > 2 ** 32 > first * big[0].numel() * big.element_size()
    big[first:] = c["cache"].to(DEV)
    c["table"] = torch.where(c["table"] < 0, c["table"], c["table"] + first)
    c["cache"] = big
    out, lse = run(c)
    assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])


@pytest.mark.parametrize("fmt,h", [(BF16, 128), (BF16, 32), (FP8_528, 64)])
def test_more_parts_than_the_device_has(fmt, h):
    parity(fmt, [1500, 70, 900], 3, h, 1100, 40, seed=26, logits=True, parts=300)


@pytest.mark.parametrize("h,value", [(128, float("inf")), (64, float("-inf")), (16, torch.finfo(torch.bfloat16).min)])
def test_infinities_and_lowest_values_in_unseen_slots(h, value):
    c = case(BF16, [200, 64, 700, 131], 2, h, 100, 3, new=[2, 1, 2, 2], seed=27)
    c["cache"][~c["live"]] = value
    check(c, *run(c))


def test_queries_of_padding_may_hold_anything():
    for fmt, h in ((BF16, 128), (BF16, 16), (FP8_656, 48)):
        c = case(fmt, [200, 64, 700], 5, h, 100, 3, new=[2, 0, 5], seed=28)
        ref = run(c)
        for b, n in enumerate(c["new"].tolist()):
            c["q"][b, n:] = float("nan")
        out, lse = run(c)
        assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])


@pytest.mark.parametrize("fmt,h", [(BF16, 128), (FP8_656, 16)])
def test_two_captured_calls_with_cut_items_run_side_by_side(fmt, h):
    """Two graphs, a workspace each, replayed at once on two streams; the
    lengths are written between replays."""
    cases = [case(fmt, [2200, 70, 900], 1, h, 1500, 200, seed=25 + i) for i in range(2)]
    sides = []
    for c in cases:
        buf = binding.WindowBuffers(3, 1, h, 1500, 200, DEV)
        assert buf.workspace is not None
        gpu = [c[k].to(DEV) for k in ("q", "cache", "table", "lens")]
        call = lambda buf=buf, a=gpu: binding.mla_window_decode(  # noqa: E731
            a[0], a[1], fmt, a[2], a[3], SCALE, 1500, 200, buf.num_sm_parts, buf.workspace, buf.out, buf.lse, buf.err)
        call()
        stream = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            call()
            call()
        sides.append((buf, gpu[3], stream, graph))
    for lens in ([2200, 70, 900], [0, 70, 900], [2200, 1, 0]):
        for buf, sl, _, _ in sides:
            sl.copy_(torch.tensor(lens, dtype=torch.int32))
            buf.out.fill_(9.0)
        torch.cuda.synchronize()
        for _ in range(5):
            for _, _, stream, graph in sides:
                with torch.cuda.stream(stream):
                    graph.replay()
        torch.cuda.synchronize()
        for c, (buf, _, _, _) in zip(cases, sides):
            c["lens"] = torch.tensor(lens, dtype=torch.int32)
            assert int(buf.err.item()) == 0
            check(c, buf.out.cpu(), buf.lse.cpu())


@pytest.mark.parametrize("h", [16, 32, 48, 64])
@pytest.mark.parametrize("fmt", [BF16, FP8_528])
def test_long_windows_of_blocks_of_tokens(fmt, h):
    """Blocks of several tokens that are cut into pieces and merged."""
    parity(fmt, [1900, 700, 64, 12], 11, h, 1200, 3, new=None, seed=13, logits=True)


@pytest.mark.parametrize("fmt,h", [(BF16, 128), (BF16, 32), (FP8_656, 128), (FP8_528, 64)])
def test_window_of_one_copies_its_row(fmt, h):
    c = case(fmt, [1, 5, 64, 65, 700], 1, h, 1, 0, seed=7)
    out, lse = run(c)
    keys = keys_of(c["cache"], fmt)
    for b, L in enumerate(c["lens"].tolist()):
        row = keys[int(c["table"][b, (L - 1) // 64]), (L - 1) % 64, :512]
        assert np.array_equal(f64_np(out)[b, 0], np.broadcast_to(row, (h, 512)))


@pytest.mark.parametrize("h", [128, 64])
def test_large_scores_move_the_reference(h):
    """Scores that grow along the window (the softmax's reference moves at every
    tile) and lie far apart."""
    c = case(BF16, [900, 900], 1, h, 700, 10, seed=8)
    c["q"] = (c["q"].float() * 6).to(torch.bfloat16)
    for b in range(2):
        for p in range(900):
            page = int(c["table"][b, p // 64])
            if page >= 0:
                c["cache"][page, p % 64] = (c["cache"][page, p % 64].float() * (0.2 + p / 300)).to(torch.bfloat16)
    check(c, *run(c))


@pytest.mark.parametrize("fmt,h", [(BF16, 128), (BF16, 48), (FP8_656, 64)])
def test_same_result_as_dense_decode_when_everything_is_visible(fmt, h):
    c = case(fmt, [500, 64, 333], 2, h, 4096, 0, seed=9)
    out, lse = run(c)
    c["cache"][~c["live"]] = 0
    buf = binding.DecodeBuffers(3, 2, h, DEV)
    q, cache, bt, sl = (c[k].to(DEV) for k in ("q", "cache", "table", "lens"))
    binding.mla_get_metadata(sl, 3, 2, True, 0, buf.num_sm_parts, buf.metadata)
    binding.mla_decode(q, cache, fmt, bt, sl, SCALE, True, buf.metadata, buf.num_sm_parts, buf.workspace, buf.out, buf.lse, buf.err)
    # both are within the parity bounds of the definition, so within twice those of each other
    a, d = f64_np(out), f64_np(buf.out)
    assert np.linalg.norm(a - d) <= 2 * OUT_REL_L2 * np.linalg.norm(d)
    assert np.abs(f64_np(lse) - f64_np(buf.lse)).max() <= 2 * LSE_ABS


def test_bad_pages_are_flagged():
    for fmt, h in ((BF16, 128), (BF16, 16), (FP8_656, 64)):
        c = case(fmt, [100, 300], 1, h, 128, 4, seed=10)
        c["cache"] = torch.zeros_like(c["cache"])
        good = run(c)
        c["table"][1, 4] = 10 ** 6
        b, s = 2, 1
        buf = binding.WindowBuffers(b, s, h, 128, 4, DEV)
        args = lambda bt: (c["q"].to(DEV), c["cache"].to(DEV), fmt, bt, c["lens"].to(DEV), SCALE, 128, 4,  # noqa: E731
                           buf.num_sm_parts, buf.workspace, buf.out, buf.lse, buf.err)
        binding.mla_window_decode(*args(c["table"].to(DEV)))
        assert int(buf.err.item()) == binding.MLA_DEVERR_BAD_PAGE
        assert torch.equal(buf.out[0].cpu(), good[0][0])
        buf.err.zero_()
        binding.mla_window_decode(*args(c["table"].to(DEV)[:, :3]))       # the row ends before the window
        assert int(buf.err.item()) == binding.MLA_DEVERR_BAD_PAGE


def test_binding_refusals():
    c = case(BF16, [100, 300], 1, 64, 4096, 4, seed=11)
    q, cache, bt, sl = (c[k].to(DEV) for k in ("q", "cache", "table", "lens"))
    buf = binding.WindowBuffers(2, 1, 64, 4096, 4, DEV)
    ok = [q, cache, BF16, bt, sl, SCALE, 4096, 4, buf.num_sm_parts, buf.workspace, buf.out, buf.lse]

    def but(i, v):
        return ok[:i] + [v] + ok[i + 1:]
    for bad in (but(0, q.float()), but(0, q[0]), but(0, q[..., :512]), but(0, torch.cat([q, q], 3)[..., :576]), but(1, cache.float()),
                but(2, 5), but(3, bt.long()), but(3, bt[:1]), but(4, sl.long()), but(9, buf.workspace.cpu()),
                but(10, buf.out.float()), but(10, buf.out[:, :, :32]), but(11, buf.lse[:1]), but(11, buf.lse.cpu())):
        with pytest.raises(ValueError):
            binding.mla_window_decode(*bad)
    for kw in (dict(attn_sink=torch.zeros(63, device=DEV)), dict(new_lens=sl.long()), dict(err=sl)):
        with pytest.raises(ValueError):
            binding.mla_window_decode(*ok, **kw)
    for bad in (but(6, 0), but(7, -1), but(5, 0.0), but(8, 0), but(9, None), but(9, buf.workspace[:-1])):
        with pytest.raises(binding.MlaError):
            binding.mla_window_decode(*bad)
