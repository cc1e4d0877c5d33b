"""GPU parity of mla_append_kv against the fp64 oracle.

Tolerances.  The kernel's inputs are exact (bf16, fp32 tables) and its fp32
arithmetic leaves a relative error below 2^-16 on a normalised value (a sum of
512 squares, 64 in a row on a lane and three joins: < 67 * 2^-24, halved by the
square root; a root, a quotient and two products: 4 * 2^-24) and below 2^-16 of
the pair's length on a rotated one.  On top of it comes the one rounding of the
format, half a step: bf16 2^-8 relative; e4m3 2^-4 relative, or 2^-10 of the
scale among its subnormals.  A bf16 value next to a rounding border may also
land on its other side; that error is again at most the half step plus what the
fp32 value was off.
"""
import numpy as np
import pytest
import torch

import oracle
from mla_decode_attention_gb300 import binding, workloads
from tests._util import bf16_np, f64_np

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
FP32 = 2.0 ** -16
BF16, FP8_528, FP8_656 = binding.MLA_KV_BF16, binding.MLA_KV_FP8_528, binding.MLA_KV_FP8_656
FORMATS = [BF16, FP8_656, FP8_528]


@pytest.fixture(scope="module", autouse=True)
def library():
    from mla_decode_attention_gb300 import build
    import os
    if not os.path.exists(binding.LIB_PATH):
        build.build()
    return binding.lib()


def width(fmt):
    return 512 if fmt == FP8_528 else 576


def rope_table(rows):
    a = torch.arange(rows, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)
    return torch.cat([a.cos(), a.sin()], 1).float()


def case(fmt, lens, s, new=None, seed=0, gap=0, pages_more=3):
    g = torch.Generator().manual_seed(seed)
    b, d = len(lens), width(fmt)
    slots = max(1, (max(lens) + 63) // 64)
    perm = torch.randperm(b * slots + pages_more, generator=g)
    table = perm[:b * slots].view(b, slots).int()
    x = torch.randn(b, s, d + gap, generator=g).to(torch.bfloat16)[..., gap:]
    n = b * slots + pages_more
    if fmt == BF16:
        cache = torch.randn(n, 64, 576, generator=g).to(torch.bfloat16)
    else:
        cache = torch.randint(0, 256, (n, 64, 656 if fmt == FP8_656 else 528), generator=g, dtype=torch.uint8)
    return dict(fmt=fmt, lens=torch.tensor(lens, dtype=torch.int32), new=None if new is None else torch.tensor(new, dtype=torch.int32),
                x=x, table=table, cache=cache, rope=rope_table(max(lens) + 1), weight=1 + 0.3 * torch.randn(512, generator=g))


def on_gpu(x):  # keeps a view's strides
    if x is None or x.is_contiguous():
        return None if x is None else x.to(DEV)
    base = x._base.to(DEV)
    return base.as_strided(x.shape, x.stride(), x.storage_offset())


def run(c, style=0, eps=1e-6, rope=True, norm=True, err=None):
    cache = c["cache"].to(DEV)
    binding.mla_append_kv(on_gpu(c["x"]), cache, c["fmt"], c["table"].to(DEV), c["lens"].to(DEV),
                          c["rope"].to(DEV) if rope else None, style, c["weight"].to(DEV) if norm else None,
                          eps if norm else 0.0, on_gpu(c["new"]), err)
    torch.cuda.synchronize()
    return cache.cpu()


def check(c, got, style=0, eps=1e-6, rope=True, norm=True, dropped=()):
    b, s, d = c["x"].shape
    pos = oracle.token_positions(c["lens"].tolist(), None if c["new"] is None else c["new"].tolist(), s)
    for bi, j in dropped:
        pos[bi, j] = -1
    bi, j = np.nonzero(pos >= 0)
    p = pos[bi, j]
    want = oracle.latent_rows(f64_np(c["x"])[bi, j], p, f64_np(c["rope"]) if rope else None, style == 1,
                              f64_np(c["weight"]) if norm else None, eps if norm else 0.0, c["fmt"] == FP8_528)
    page, slot = c["table"].numpy()[bi, p // 64], p % 64
    rows = got[page, slot]
    rest = got.clone()
    rest[page, slot] = c["cache"][page, slot]
    assert torch.equal(rest.view(torch.uint8), c["cache"].view(torch.uint8)), "a slot of no new token was written"
    # length of the rotated pairs, for the error of their fp32 arithmetic
    length = np.abs(want)
    tail = want[:, -64:]
    half = np.roll(tail, 32, 1) if style == 1 else tail.reshape(-1, 32, 2)[..., ::-1].reshape(-1, 64)
    length[:, -64:] = np.hypot(tail, half)

    def near(x, cols, step, more=0.0):
        w, l = want[:, cols], length[:, cols]
        assert np.all(np.abs(x - w) <= step * (np.abs(w) + FP32 * l) + FP32 * l + more)

    if c["fmt"] == BF16:
        near(oracle.bf16_bits_to_f64(bf16_np(rows)), slice(0, d), 2.0 ** -8)
        return
    raw = rows.numpy()
    codes = oracle.e4m3_to_f64(raw[:, :512])
    tiles = np.abs(want[:, :512]).reshape(len(want), -1, 128 if c["fmt"] == FP8_656 else 32).max(-1) / 448
    if c["fmt"] == FP8_656:
        scale = np.ascontiguousarray(raw[:, 512:528]).view(np.float32).astype(np.float64)
        assert np.all(np.abs(scale - np.where(tiles > 0, tiles, 1.0)) <= 2 * FP32 * tiles)
        near(oracle.bf16_bits_to_f64(np.ascontiguousarray(raw[:, 528:]).view(np.uint16)), slice(512, 576), 2.0 ** -8)
        each = np.repeat(scale, 128, 1)
    else:
        scale = oracle.e8m0_to_f64(raw[:, 512:])
        # the smallest power of two at or above tiles, up to the fp32 error of tiles
        up = np.where(tiles > 0, tiles, 1.0)
        assert np.all((scale >= up * (1 - 2 * FP32)) & (scale < 2 * up * (1 + 2 * FP32)))
        each = np.repeat(scale, 32, 1)
    near(codes * each, slice(0, 512), 2.0 ** -4, 2.0 ** -10 * each * (1 + FP32))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("style", [0, 1])
@pytest.mark.parametrize("lens,s,new", [
    ([1], 1, None), ([200, 333], 1, None), ([64, 65, 128, 1, 0], 1, None), ([5, 700, 64, 130], 3, None),
    ([2, 1], 4, None),                          # padded at the start
    ([90, 64, 7, 0, 300], 33, [33, 0, 5, 1, 32]),  # padded at the end, nothing new, an empty request
    ([1021], 1021, None),
])
def test_parity(fmt, style, lens, s, new):
    c = case(fmt, lens, s, new, seed=len(lens) + s)
    check(c, run(c, style), style)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rope,norm", [(False, True), (True, False), (False, False)])
def test_without_rotation_or_norm(fmt, rope, norm):
    c = case(fmt, [77, 130], 20, seed=3)
    check(c, run(c, 0, rope=rope, norm=norm), 0, rope=rope, norm=norm)


@pytest.mark.parametrize("fmt", FORMATS)
def test_strided_rows(fmt):
    c = case(fmt, [100, 101, 40], 7, [7, 3, 5], seed=4, gap=64)
    assert not c["x"].is_contiguous()
    check(c, run(c))


@pytest.mark.parametrize("fmt", FORMATS)
def test_plain_rows_are_the_formats_own_bits(fmt):
    """No norm, no rotation: the bytes of the reference encoders, bit for bit."""
    c = case(fmt, [640], 640, seed=5)
    x = c["x"].float()
    x[0, 0] = 0.0                       # all zero: scale 1
    x[0, 1, :32] = torch.ldexp(torch.rand(32) + 0.5, torch.tensor(-120))   # tiny values
    x[0, 2] *= 1e30                      # large ones
    x[0, 3, :] = 448.0                   # absmax / 448 = 1 exactly
    x[0, 4, :] = torch.finfo(torch.bfloat16).max
    x[0, 5, :] = 2.0 ** -133             # bf16 subnormals: the scale's ratio underflows or is subnormal
    x[0, 6, :] = 448.0 * 2.0 ** -127     # ratio 2^-127
    x[0, 7, :] = 1.25 * 448.0 * 2.0 ** -127
    c["x"] = x.to(torch.bfloat16)
    got = run(c, rope=False, norm=False)
    pos = torch.arange(640)
    rows = got[c["table"][0, pos // 64].long(), pos % 64]
    xf = c["x"][0].float()
    want = {BF16: lambda: c["x"][0], FP8_656: lambda: workloads.quantize_fp8_tokens(xf),
            FP8_528: lambda: workloads.quantize_fp8_v41_tokens(xf)}[fmt]()
    assert torch.equal(rows.view(torch.uint8), want.view(torch.uint8))


def test_bad_pages_and_positions_are_flagged_and_left_out():
    for fmt in FORMATS:
        c = case(fmt, [70, 130, 64, 10], 2, seed=6)
        good = c["table"].clone()
        c["table"][0, 1] = 10 ** 6               # token 69 and 68: bad page
        c["table"][1, 2] = -1                    # tokens 128, 129
        c["rope"] = c["rope"][:64]               # positions 64 .. have no row
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        got = run(c, err=err)
        assert int(err.item()) == binding.MLA_DEVERR_BAD_PAGE | binding.MLA_DEVERR_BAD_INDEX
        c["table"] = good
        check(c, got, dropped=[(0, 0), (0, 1), (1, 0), (1, 1)])
    c = case(BF16, [70, 10], 1, seed=7)          # the table's row ends before the token's page
    wide = c["table"]
    c["table"] = wide[:, :1]
    cache, err = c["cache"].to(DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    binding.mla_append_kv(c["x"].to(DEV), cache, BF16, wide.to(DEV)[:, :1], c["lens"].to(DEV), c["rope"].to(DEV), 0,
                          c["weight"].to(DEV), 1e-6, None, err)
    assert int(err.item()) == binding.MLA_DEVERR_BAD_PAGE
    c["table"] = wide
    check(c, cache.cpu(), dropped=[(0, 0)])


def test_non_finite_rows_stay_their_own():
    for fmt in FORMATS:
        c = case(fmt, [40], 4, seed=8)
        clean = run(c)
        c["x"][0, 1, 5], c["x"][0, 2, 511] = float("nan"), float("inf")
        got = run(c)
        at = [(int(c["table"][0, 0]), 36 + i) for i in (0, 3)]
        for p, s in at:
            assert torch.equal(got[p, s], clean[p, s])


def test_many_pages_reach_past_32_bits():
    """A token of a page whose byte offset in the cache passes 2^32."""
    pages = (1 << 32) // (64 * 1152) + 40
    cache = torch.zeros(pages, 64, 576, dtype=torch.bfloat16, device=DEV)
    c = case(BF16, [64, 10], 2, seed=9)
    c["table"][0, 0], c["table"][1, 0] = pages - 1, pages - 30
    binding.mla_append_kv(c["x"].to(DEV), cache, BF16, c["table"].to(DEV), c["lens"].to(DEV), c["rope"].to(DEV), 0,
                          c["weight"].to(DEV), 1e-6)
    torch.cuda.synchronize()
    written = cache.view(-1, 576).abs().sum(1).nonzero()[:, 0].tolist()
    assert written == [(pages - 30) * 64 + 8, (pages - 30) * 64 + 9, (pages - 1) * 64 + 62, (pages - 1) * 64 + 63]


def test_binding_refusals():
    c = case(BF16, [10, 10], 2, seed=10)
    x, cache, bt, sl = c["x"].to(DEV), c["cache"].to(DEV), c["table"].to(DEV), c["lens"].to(DEV)
    ok = (x, cache, BF16, bt, sl)
    for bad in ((x.float(), *ok[1:]), (x[..., :512], *ok[1:]), (x, cache.float(), *ok[2:]), (x, cache[:, :32], *ok[2:]),
                (x, cache, FP8_656, bt, sl), (x, cache, 7, bt, sl), (x, cache, BF16, bt.long(), sl), (x, cache, BF16, bt[:1], sl),
                (x, cache, BF16, bt, sl.long()), (x, cache, BF16, bt, sl[:1]), (x.transpose(0, 1), *ok[1:]),
                (x, cache, BF16, bt, sl.cpu())):
        with pytest.raises(ValueError):
            binding.mla_append_kv(*bad)
    for kw in (dict(rope_table=c["rope"].to(DEV).double()), dict(rope_table=c["rope"].to(DEV)[:, :32]),
               dict(norm_weight=c["weight"].to(DEV)[:100], norm_eps=1.0), dict(new_lens=sl[:1]),
               dict(err=torch.zeros(2, dtype=torch.int32, device=DEV))):
        with pytest.raises(ValueError):
            binding.mla_append_kv(*ok, **kw)
    with pytest.raises(binding.MlaError):
        binding.mla_append_kv(*ok, norm_weight=c["weight"].to(DEV))      # a weight without a norm
    with pytest.raises(binding.MlaError):
        binding.mla_append_kv(*ok, rope_table=c["rope"].to(DEV), rope_style=5)
