"""GPU parity of mla_query_norm_rope against the fp64 oracle.

Tolerance, as for mla_append_kv: the fp32 arithmetic is off by less than 2^-16
of a value (a rotated one: of its pair's length), and the one rounding to bf16
by half a step, 2^-8 relative.
"""
import numpy as np
import pytest
import torch

import oracle
from mla_decode_attention_gb300 import binding
from tests._util import f64_np
from tests.test_gpu_append import DEV, FP32, library, on_gpu, rope_table  # noqa: F401

pytestmark = pytest.mark.gpu


def case(lens, s, h, d, new=None, seed=0, gaps=(0, 0), norm=True):
    """q [b, s, h, d]; gaps: unused columns between heads and between tokens."""
    g = torch.Generator().manual_seed(seed)
    b = len(lens)
    base = (3 * torch.randn(b * s, h * (d + gaps[0]) + gaps[1], generator=g)).to(torch.bfloat16)
    row = base.shape[1]
    q = base.as_strided((b, s, h, d), (s * row, row, d + gaps[0], 1), gaps[1])
    return dict(lens=torch.tensor(lens, dtype=torch.int32), new=None if new is None else torch.tensor(new, dtype=torch.int32),
                q=q, rope=rope_table(max(max(lens), 1)), weight=1 + 0.3 * torch.randn(d, generator=g) if norm else None)


def run(c, style=0, eps=1e-6, rope=True, out=None, err=None):
    q = on_gpu(c["q"])
    out = q if out == "q" else out if out is not None else torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
    binding.mla_query_norm_rope(q, out, c["lens"].to(DEV), c["rope"].to(DEV) if rope else None, style,
                                None if c["weight"] is None else c["weight"].to(DEV), eps, on_gpu(c["new"]), err)
    torch.cuda.synchronize()
    return out.cpu()


def check(c, got, before, style=0, eps=1e-6, rope=True, dropped=()):
    b, s, h, d = c["q"].shape
    pos = oracle.token_positions(c["lens"].tolist(), None if c["new"] is None else c["new"].tolist(), s)
    for at in dropped:
        pos[at] = -1
    ok = pos >= 0
    assert torch.equal(got[torch.from_numpy(~ok)], before[torch.from_numpy(~ok)]), "a padding slot was written"
    x = f64_np(c["q"])[ok]
    want = oracle.query_rows(x, pos[ok], f64_np(c["rope"]) if rope else None, style == 1,
                             None if c["weight"] is None else f64_np(c["weight"]), eps)
    if not rope and eps == 0:
        assert np.array_equal(f64_np(got)[ok], x)
        return
    length = np.abs(want)
    tail = want[..., -64:]
    half = np.roll(tail, 32, -1) if style == 1 else tail.reshape(*tail.shape[:-1], 32, 2)[..., ::-1].reshape(tail.shape)
    length[..., -64:] = np.hypot(tail, half)
    assert np.all(np.abs(f64_np(got)[ok] - want) <= 2.0 ** -8 * (np.abs(want) + FP32 * length) + FP32 * length)
    if eps == 0:  # what is not rotated is copied
        assert np.array_equal(f64_np(got)[ok][..., :-64], x[..., :-64])


@pytest.mark.parametrize("d", [64, 128, 192, 256, 320, 384, 448, 512, 576])
@pytest.mark.parametrize("h", [1, 5, 128])
@pytest.mark.parametrize("style", [0, 1])
def test_parity(d, h, style):
    c = case([9, 300, 64], 3, h, d, seed=d + h)
    got = run(c, style)
    check(c, got, torch.full_like(got, 7.0), style)


@pytest.mark.parametrize("lens,s,new", [([1], 1, None), ([0, 5], 1, None), ([2, 1, 90], 4, None),
                                        ([90, 64, 7, 0, 300], 33, [33, 0, 5, 1, 32])])
@pytest.mark.parametrize("d,norm", [(192, True), (576, False)])
def test_padding_is_left_alone(lens, s, new, d, norm):
    c = case(lens, s, 16, d, new, seed=s, norm=norm)
    eps = 1e-6 if norm else 0.0
    got = run(c, 0, eps)
    check(c, got, torch.full_like(got, 7.0), 0, eps)


@pytest.mark.parametrize("style", [0, 1])
@pytest.mark.parametrize("rope,eps,weighted", [(True, 0.0, False), (False, 1e-5, True), (True, 1e-5, False), (False, 0.0, False)])
def test_in_place_and_parts_left_out(style, rope, eps, weighted):
    for d in (64, 192, 576):
        c = case([70, 5, 3], 4, 48, d, [4, 0, 3], seed=d, norm=weighted)
        check(c, run(c, style, eps, rope, out="q"), c["q"], style, eps, rope)
        got = run(c, style, eps, rope)
        check(c, got, torch.full_like(got, 7.0), style, eps, rope)


@pytest.mark.parametrize("gaps", [(64, 0), (0, 24), (8, 16)])
def test_strides(gaps):
    c = case([30, 200], 5, 6, 192, [5, 2], seed=1, gaps=gaps)
    wide = torch.full((2, 5, 6, 576), 3.0, dtype=torch.bfloat16, device=DEV)
    got = run(c, out=wide[..., 128:320])                 # columns of a wider output
    check(c, got, torch.full_like(got, 3.0))
    assert torch.all(wide[..., :128] == 3) and torch.all(wide[..., 320:] == 3)
    q = on_gpu(c["q"])                                   # in place: the columns between the heads stay
    before = q._base.cpu()
    binding.mla_query_norm_rope(q, q, c["lens"].to(DEV), c["rope"].to(DEV), 0, c["weight"].to(DEV), 1e-6, on_gpu(c["new"]))
    check(c, q.cpu(), c["q"])
    gone = torch.ones_like(before)
    gone.as_strided(q.shape, q.stride(), q.storage_offset()).zero_()
    assert torch.equal(q._base.cpu() * gone, before * gone)


def test_positions_without_a_row_are_flagged_and_left_out():
    c = case([70, 10], 2, 8, 512, seed=2)
    c["rope"] = c["rope"][:69]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = run(c, err=err)
    assert int(err.item()) == binding.MLA_DEVERR_BAD_INDEX
    check(c, got, torch.full_like(got, 7.0), dropped=[(0, 1)])


def test_non_finite_heads_stay_their_own():
    c = case([70], 1, 9, 192, seed=3)
    clean = run(c)
    c["q"][0, 0, 4, 7], c["q"][0, 0, 5, 190] = float("nan"), float("inf")
    got = run(c)
    keep = [0, 1, 2, 3, 6, 7, 8]
    assert torch.equal(got[0, 0, keep], clean[0, 0, keep])


def test_zero_and_extreme_heads():
    c = case([70], 1, 4, 512, seed=4)
    c["q"][0, 0, 0] = 0.0
    c["q"][0, 0, 1] *= 2.0 ** 50
    c["q"][0, 0, 2] *= 2.0 ** -50
    got = run(c)
    check(c, got, torch.full_like(got, 7.0))


def test_offsets_past_32_bits():
    """Rows whose element offset in q and out passes 2^31."""
    h, d, tokens = 128, 576, 30000
    q = torch.zeros(tokens, 1, h, d, dtype=torch.bfloat16, device=DEV)
    assert q.numel() > 1 << 31
    g = torch.Generator(device=DEV).manual_seed(5)
    q[-1] = torch.randn(1, h, d, generator=g, device=DEV).to(torch.bfloat16)
    q[0] = q[-1]
    lens = torch.full((tokens,), 33, dtype=torch.int32, device=DEV)
    binding.mla_query_norm_rope(q, q, lens, rope_table(40).to(DEV), 0, None, 1e-6)
    torch.cuda.synchronize()
    assert torch.equal(q[0], q[-1]) and float(q[0].float().abs().sum()) > 0
    assert float(q[1:-1].float().abs().sum()) == 0


def test_more_requests_than_one_launch_takes():
    b = 65535 + 700
    lens = [1 + i % 90 for i in range(b)]
    c = case(lens, 1, 2, 64, new=[0 if i % 5 == 0 else 1 for i in range(b)], seed=9)
    check(c, run(c), torch.full(c["q"].shape, 7.0, dtype=torch.bfloat16))


def test_binding_refusals():
    c = case([10, 10], 2, 4, 192, seed=6)
    q, sl = c["q"].to(DEV), c["lens"].to(DEV)
    out = torch.empty_like(q)
    for bad in ((q.float(), out, sl), (q, out.float(), sl), (q, out[:1], sl), (q[0], out[0], sl), (q, out, sl.long()),
                (q, out, sl[:1]), (q.transpose(0, 1), out, sl), (q.transpose(2, 3), out.transpose(2, 3), sl),
                (q, out.cpu(), sl), (q, out, sl.cpu())):
        with pytest.raises(ValueError):
            binding.mla_query_norm_rope(*bad)
    with pytest.raises(ValueError):
        binding.mla_query_norm_rope(q, out, sl, norm_weight=torch.ones(64, device=DEV), norm_eps=1e-6)
    for bad in (dict(norm_eps=-1.0), dict(norm_weight=torch.ones(192, device=DEV)), dict(rope_style=2)):
        with pytest.raises(binding.MlaError):
            binding.mla_query_norm_rope(q, out, sl, c["rope"].to(DEV), **bad)
    with pytest.raises(binding.MlaError):
        binding.mla_query_norm_rope(q[..., :96], out[..., :96], sl)     # not a multiple of 64
    with pytest.raises(binding.MlaError):
        binding.mla_query_norm_rope(q[..., 1:65], out[..., :64], sl)    # not on 16 bytes
    e = q.expand(2, 2, 4, 192)[:, :, :1].expand(2, 2, 4, 192)
    with pytest.raises(binding.MlaError):
        binding.mla_query_norm_rope(q, e, sl)                           # heads of out overlap
