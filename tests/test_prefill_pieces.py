"""Which calls mla_prefill cuts along their keys, seen by its workspace (no GPU)."""
import os

import pytest

from mla_decode_attention_gb300 import binding, build


@pytest.fixture(scope="session", autouse=True)
def built_library():
    if not os.path.exists(binding.LIB_PATH):
        build.build()
    return binding.lib()


def pieces(total_q, total_k, batch, h_q, h_k=None, parts=152):
    n = binding.mla_prefill_workspace_size(total_q, total_k, batch, h_q, h_k or h_q, parts)
    assert n % (total_q * h_q * 129 * 4) == 0
    return n // (total_q * h_q * 129 * 4) or 1


@pytest.mark.parametrize("tokens,keys,batch,h", [(2048, 2048, 2, 8), (1024, 1024, 2, 16), (1024, 1024, 4, 8), (512, 512, 4, 16),
                                                 (1024, 2048, 2, 16), (512, 512, 2, 8)])
def test_sequences_whose_blocks_are_full_of_rows_stay_whole(tokens, keys, batch, h):
    """A piece of full blocks costs more than idle SMs at the end (2 x 2048 tokens of 8 heads: 41 us whole, 47 in three)."""
    assert pieces(batch * tokens, batch * keys, batch, h) == 1


@pytest.mark.parametrize("total_q,total_k,batch,h,h_k", [(26, 36576, 3, 16, 16), (16, 16000, 16, 4, 4), (16, 132000, 16, 4, 4), (200, 3000, 2, 8, 8),
                                                         (256, 8000, 4, 8, 8), (600, 4600, 2, 16, 16), (8192, 8192, 2, 4, 4), (128, 8000, 2, 64, 8)])
def test_few_rows_or_long_keys_are_cut(total_q, total_k, batch, h, h_k):
    assert pieces(total_q, total_k, batch, h, h_k) > 1


@pytest.mark.parametrize("parts", [1, 100, 152])
def test_the_workspace_is_bounded(parts):
    """2048 partial rows of 516 bytes for each SM at most, whatever the sizes."""
    most = 0
    for batch in (1, 2, 3, 17, 300):
        for h, h_k in ((1, 1), (8, 8), (16, 16), (128, 128), (64, 8), (128, 1), (200, 200)):
            for total_q in (0, 1, 16, 300, 2048, 8192, 16384, 65536, 1 << 20, 1 << 25):
                for total_k in (0, 1000, 16384, 262144, 1 << 21, 1 << 22, 1 << 25):
                    try:
                        n = binding.mla_prefill_workspace_size(total_q, total_k, batch, h, h_k, parts)
                    except binding.MlaError:  # (more blocks of rows than a call may have)
                        continue
                    assert n <= 2048 * 516 * parts, (total_q, total_k, batch, h, h_k)
                    most = max(most, n)
    assert most > 0 or parts == 1


@pytest.mark.parametrize("total_q,total_k,batch", [(8192, 262144, 2), (16384, 1 << 21, 2), (65536, 1 << 22, 2), (4096, 65536, 1)])
def test_long_contexts_are_not_cut_for_little(total_q, total_k, batch):
    """Thousands of blocks on 152 SMs: cutting them could save a percent or two and take gigabytes."""
    assert pieces(total_q, total_k, batch, 128) == 1


@pytest.mark.parametrize("total_q,total_k,batch,h,want", [(1024, 9024, 1, 40, 4), (100, 12100, 1, 200, 3), (600, 32600, 2, 40, 5), (1, 16000, 1, 128, 7)])
def test_calls_that_gain_are_cut(total_q, total_k, batch, h, want):
    assert pieces(total_q, total_k, batch, h) == want
