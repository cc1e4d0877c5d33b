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
