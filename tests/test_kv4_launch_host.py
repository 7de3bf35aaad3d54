"""CPU tests of what the 4-bit KV cache's calls launch, and of what they refuse because no launch holds it.  No call
here reaches the GPU."""
from __future__ import annotations

import pytest

import lossless_bf16_kv_amd as sz
from lossless_bf16_kv_amd import kv4
from test_kv4_host import batch, cache, call

MOST = (1 << 31) - 1


def refused(name, word, **kw):
    assert call(name, **kw) == sz.E_INVALID
    text = sz.lib().splitzip_last_error().decode()
    assert word in text, text


# The kernels count up to 1024 tokens past a budget in 32 bits.
@pytest.mark.parametrize("budget", [MOST, MOST - 127, MOST - 1023, MOST - 65535])
def test_evict_budget_of_nearly_2_31(budget):
    refused("evict", "too many tokens to keep", c=cache(kv_heads=1), b=batch(n_seqs=1, total=1), budget=budget, lens=1 << 21)


@pytest.mark.parametrize("budget", [MOST, 1 << 32, (1 << 32) + 5])
def test_evict_budget_past_32_bits_is_not_cut(budget):
    # before anything of the cache is looked at
    with pytest.raises(ValueError, match="budget"):
        kv4.KV4Cache.evict(None, None, None, None, budget)
