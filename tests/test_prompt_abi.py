"""Refusals of the prompt entry points before any launch (no GPU): the C ABI with pointers that are never followed, the
binding's own checks, and the size of the workspace."""
import os

import pytest
import torch

from mla_decode_attention_gb300 import binding, build


@pytest.fixture(scope="session", autouse=True)
def built_library():
    if not os.path.exists(binding.LIB_PATH):
        build.build()
    return binding.lib()


GATHER = dict(cache=0x10000, fmt=0, pages=8, bt=0x20000, bts=4, width=4, cu=0x30000, starts=None, b=2, rows=100, out=0x40000, stride=576,
              err=None, stream=None)
PREFILL = dict(q=0x10000, qt=384, qh=192, k=0x20000, kt=512, kh=256, r=0x30000, rt=64, rh=0, v=0x40000, vt=512, vh=256, cuq=0x50000,
               cuk=0x60000, b=2, nq=1000, nk=1000, h=2, hk=2, scale=0.07, causal=1, parts=1, ws=0x70000, wsb=1 << 40, out=0x80000,
               ot=256, oh=128, lse=0x90000, err=None, stream=None)
MERGE = dict(parts=0x10000, f32=0, ps=25600, ts=256, hs=128, lses=0x20000, lp=200, lh=100, lt=1, n=2, t=100, h=2, d=128, out=0x30000,
             ot=256, oh=128, lse=0x40000, olh=100, olt=1, stream=None)
NAN = float("nan")


def call(name, base, over):
    a = dict(base)
    assert set(over) <= set(a)
    a.update(over)
    return getattr(binding.lib(), name)(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(cache=None), -1), (dict(bt=None), -1), (dict(cu=None), -1), (dict(out=None), -1), (dict(b=0), -2), (dict(rows=-1), -2),
    (dict(rows=(1 << 25) + 1), -2), (dict(b=(1 << 16) + 1), -2), (dict(pages=0), -2), (dict(pages=(1 << 25) + 1), -2), (dict(width=0), -2), (dict(bts=3), -2),
    (dict(stride=568), -2), (dict(stride=1 << 40), -2), (dict(fmt=2, stride=504), -2), (dict(stride=580), -3), (dict(cache=0x10008), -3),
    (dict(out=0x40002), -3), (dict(fmt=3), -6), (dict(fmt=-1), -6), (dict(rows=0, out=None, cache=None, cu=None), 0),
])
def test_gather_refuses(over, code):
    assert call("mla_gather_kv", GATHER, over) == code


@pytest.mark.parametrize("over,code", [
    (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(cuq=None), -1), (dict(cuk=None), -1), (dict(out=None), -1),
    (dict(lse=None), -1), (dict(nq=1, nk=100000, parts=152, b=1, ws=None), -1), (dict(nq=1, nk=100000, parts=152, b=1, wsb=1000), -2),
    (dict(b=0), -2), (dict(b=(1 << 16) + 1), -2), (dict(nq=-1), -2), (dict(nk=-1), -2), (dict(nq=(1 << 25) + 1), -2), (dict(nk=1 << 26), -2),
    (dict(h=0), -2), (dict(hk=0), -2), (dict(h=3), -2), (dict(h=130, hk=1), -2), (dict(parts=0), -2), (dict(scale=0.0), -2),
    (dict(scale=-1.0), -2), (dict(scale=NAN), -2), (dict(scale=float("inf")), -2), (dict(qh=184), -2), (dict(qt=184), -2),
    (dict(kh=120), -2), (dict(kt=0), -2), (dict(vh=0), -2), (dict(vt=120), -2), (dict(rt=56), -2), (dict(rh=56), -2), (dict(ot=128), -2),
    (dict(oh=64), -2), (dict(oh=0), -2), (dict(ot=1 << 39), -2), (dict(kt=1 << 39), -2), (dict(q=0x10008), -3), (dict(k=0x20002), -3),
    (dict(r=0x30008), -3), (dict(v=0x40004), -3), (dict(out=0x80008), -3), (dict(ws=0x70004), -3), (dict(qh=196, qt=392), -3),
    (dict(kt=516), -3), (dict(vh=132), -3), (dict(rt=68), -3), (dict(rh=68), -3), (dict(oh=132, ot=264), -3), (dict(r=None, qh=120), -2),
    (dict(nq=0, q=None, out=None, lse=None), 0),
])
def test_prefill_refuses(over, code):
    assert call("mla_prefill", PREFILL, over) == code


@pytest.mark.parametrize("over,code", [
    (dict(parts=None), -1), (dict(lses=None), -1), (dict(out=None), -1), (dict(lse=None), -1), (dict(n=0), -2), (dict(h=0), -2),
    (dict(t=-1), -2), (dict(d=0), -2), (dict(d=12), -2), (dict(d=520), -2), (dict(t=(1 << 30) + 1), -2), (dict(ps=-8), -2),
    (dict(ot=248), -2), (dict(oh=0), -2), (dict(olh=0), -2), (dict(olh=50), -2), (dict(ts=1 << 40), -2), (dict(parts=0x10008), -3),
    (dict(out=0x30008), -3), (dict(ps=25604), -3), (dict(ts=260), -3), (dict(hs=132), -3), (dict(oh=132, ot=264), -3),
    (dict(f32=1, hs=130), -3), (dict(t=0, parts=None), 0),
])
def test_merge_refuses(over, code):
    assert call("mla_merge_states", MERGE, over) == code


def test_prefill_workspace():
    size = binding.mla_prefill_workspace_size
    assert size(4096, 4096, 1, 128, 128, 152) == 0                 # blocks of query rows enough
    assert size(1, 100, 1, 1, 1, 152) == 0                         # too few keys to cut
    assert size(16, 16384, 1, 16, 16, 152) == 9 * 16 * 16 * 129 * 4
    assert size(16, 1 << 20, 1, 1, 1, 152) == 32 * 16 * 129 * 4    # at most 32 pieces
    assert size(16, 1 << 20, 1, 1, 1, 1) == 0
    assert size(0, 0, 1, 1, 1, 152) == 0
    for bad in ((-1, 1, 1, 1, 1, 1), (1, -1, 1, 1, 1, 1), (1, 1, 0, 1, 1, 1), (1, 1, 1, 0, 1, 1), (1, 1, 1, 3, 2, 1), (1, 1, 1, 1, 1, 0)):
        with pytest.raises(binding.MlaError):
            size(*bad)
    assert binding.lib().mla_prefill_workspace_size(1, 1, 1, 1, 1, 1, None) == -1


def test_binding_refuses_host_tensors():
    x, i = torch.zeros(2, 1, 128, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        binding.mla_gather_kv(torch.zeros(1, 64, 576, dtype=torch.bfloat16), 0, i.view(1, 2), i, x.view(1, 256))
    with pytest.raises(ValueError):
        binding.mla_prefill(x, x, x, i, i, 1.0, True, 1, None, x, torch.zeros(1, 2))
    with pytest.raises(ValueError):
        binding.mla_merge_states(x[None], torch.zeros(1, 1, 2), x, torch.zeros(1, 2))
