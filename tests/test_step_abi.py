"""Refusals of the new-token entry points before any launch (no GPU): the C ABI
with pointers that are never followed, and the binding's own checks."""
import ctypes
import os

import pytest
import torch

from mla_decode_attention_gb300 import binding, build


@pytest.fixture(scope="session", autouse=True)
def built_library():
    if not os.path.exists(binding.LIB_PATH):
        build.build()
    return binding.lib()


APPEND = dict(x=0x10000, stride=576, sl=0x20000, new=None, b=2, s=1, table=0x30000, rows=100, style=0, w=0x40000, eps=1e-6,
              cache=0x50000, fmt=0, pages=8, bt=0x60000, bts=4, width=4, err=None, stream=None)
QUERY = dict(q=0x10000, qt=1024, qh=512, sl=0x20000, new=None, b=2, s=1, h=2, d=512, table=0x30000, rows=100, style=0,
             w=0x40000, eps=1e-6, out=0x50000, ot=1024, oh=512, err=None, stream=None)
WINDOW = dict(q=0x10000, cache=0x20000, fmt=0, pages=8, bt=0x30000, bts=4, width=4, sl=0x40000, new=None, b=2, s=1, h=16,
              window=128, sinks=4, scale=0.07, sink=None, parts=152, ws=0x50000, wsb=1 << 40, out=0x60000, lse=0x70000, err=None,
              stream=None)
NAN = float("nan")


def call(name, base, over):
    a = dict(base)
    assert set(over) <= set(a)
    a.update(over)
    return getattr(binding.lib(), name)(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(x=None), -1), (dict(sl=None), -1), (dict(cache=None), -1), (dict(bt=None), -1),
    (dict(b=0), -2), (dict(s=0), -2), (dict(b=1 << 13, s=(1 << 11) + 1), -2), (dict(rows=0), -2),
    (dict(table=None), -2), (dict(rows=-1), -2), (dict(eps=0.0), -2), (dict(eps=-1.0), -2), (dict(eps=NAN), -2),
    (dict(eps=float("inf")), -2), (dict(pages=0), -2), (dict(pages=(1 << 25) + 1), -2), (dict(width=0), -2),
    (dict(bts=3), -2), (dict(stride=568), -2), (dict(stride=580), -3), (dict(x=0x10008), -3), (dict(cache=0x50004), -3),
    (dict(table=0x30004), -3), (dict(w=0x40008), -3), (dict(style=2), -6), (dict(fmt=3), -6), (dict(stride=1 << 40), -2),
])
def test_append_refuses(over, code):
    assert call("mla_append_kv", APPEND, over) == code


@pytest.mark.parametrize("over,code", [
    (dict(q=None), -1), (dict(out=None), -1), (dict(sl=None), -1), (dict(b=0), -2), (dict(s=-1), -2), (dict(h=0), -2),
    (dict(d=32), -2), (dict(d=96), -2), (dict(d=640, qh=640, oh=640, qt=1280, ot=1280), -2), (dict(b=1 << 20, s=16, h=128), -2),
    (dict(qh=504), -2), (dict(oh=0), -2), (dict(qt=1016), -2), (dict(ot=512), -2), (dict(eps=0.0), -2),
    (dict(rows=0), -2), (dict(q=0x10002), -3), (dict(out=0x50008), -3), (dict(qt=1028), -3), (dict(oh=516, ot=1032), -3),
    (dict(style=-1), -6), (dict(out=0x10000, ot=2048), -2), (dict(out=0x10000, oh=520, ot=1040, qt=1040), -2),
    (dict(qt=1 << 62), -2), (dict(qh=1 << 62), -2), (dict(h=1 << 20, oh=1 << 44, ot=1 << 38), -2),
])
def test_query_refuses(over, code):
    assert call("mla_query_norm_rope", QUERY, over) == code


@pytest.mark.parametrize("over,code", [
    (dict(q=None), -1), (dict(cache=None), -1), (dict(bt=None), -1), (dict(sl=None), -1), (dict(out=None), -1),
    (dict(lse=None), -1), (dict(b=1, window=8192, ws=None), -1), (dict(b=1, window=8192, wsb=1000), -2), (dict(b=0), -2), (dict(s=0), -2),
    (dict(b=1 << 20, s=17), -2), (dict(h=100), -2), (dict(h=256), -2), (dict(window=0), -2), (dict(window=-5), -2),
    (dict(sinks=-1), -2), (dict(parts=0), -2), (dict(pages=0), -2), (dict(width=0), -2), (dict(bts=2), -2),
    (dict(scale=0.0), -2), (dict(scale=NAN), -2), (dict(q=0x10008), -3), (dict(cache=0x20001), -3), (dict(out=0x60002), -3),
    (dict(ws=0x50004), -3), (dict(fmt=9), -6),
])
def test_window_refuses(over, code):
    assert call("mla_window_decode", WINDOW, over) == code


def test_window_workspace():
    size = binding.mla_window_workspace_size
    assert size(64, 1, 128, 128, 4, 76) == 0            # nothing is cut
    one = 2 * 152 * 64 * 513 * 4                        # two blocks of rows per part
    assert size(1, 1, 64, 8192, 0, 152) == one
    assert size(1, 1, 128, 8192, 0, 76) == one          # 76 parts of two SMs
    assert size(1, 9, 16, 8192, 0, 152) == one          # several tokens a block, either kernel
    assert size(1, 1, 64, 2**31 - 1, 2**31 - 1, 152) == one
    assert size(1 << 20, 16, 128, 4096, 0, 76) == 0
    for bad in ((0, 1, 64, 1, 0, 1), (1, 1, 63, 1, 0, 1), (1, 1, 64, 0, 0, 1), (1, 1, 64, 1, -1, 1), (1, 1, 64, 1, 0, 0)):
        with pytest.raises(binding.MlaError):
            size(*bad)
    assert binding.lib().mla_window_workspace_size(1, 1, 64, 1, 0, 1, None) == -1


def test_binding_refuses_host_tensors():
    x = torch.zeros(1, 1, 576, dtype=torch.bfloat16)
    i = torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        binding.mla_append_kv(x, torch.zeros(1, 64, 576, dtype=torch.bfloat16), 0, i.view(1, 1), i)
    with pytest.raises(ValueError):
        binding.mla_query_norm_rope(x.view(1, 1, 1, 576), x.view(1, 1, 1, 576), i)
    with pytest.raises(ValueError):
        binding.mla_window_decode(x.view(1, 1, 1, 576), torch.zeros(1, 64, 576, dtype=torch.bfloat16), 0, i.view(1, 1), i,
                                  1.0, 1, 0, 1, None, x, x)
