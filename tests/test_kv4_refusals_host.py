"""CPU tests: an eviction's new lengths must not lie over the old ones, which its kernels still read."""
from __future__ import annotations

import ctypes

import pytest

import lossless_bf16_kv_amd as sz
from lossless_bf16_kv_amd import kv4

P = 1 << 20          # stands for a device pointer; no call below reaches the GPU with it


def evict(lens, out_lens, seqs=3):
    c = kv4.splitzip_kv4_cache(P, P, P, P, P, P, 10, 64, 8, 128, 0)
    b = kv4.splitzip_kv4_batch(P, lens, None, 5, seqs, 5, seqs, 1, 320)
    # too many tokens to keep: a call whose lengths are apart is refused for that, and nothing is launched
    status = kv4._lib().splitzip_kv4_evict(ctypes.byref(c), ctypes.byref(b), P, 5, 5, (1 << 31) - 1, 0, 0, out_lens, P, None)
    assert status == sz.E_INVALID
    return sz.lib().splitzip_last_error().decode()


@pytest.mark.parametrize("apart", [0, 4, 8, -4, -8])
def test_evict_lengths_over_each_other(apart):
    assert "overlap" in evict(P + 64, P + 64 + apart)


@pytest.mark.parametrize("apart", [12, -12, 4096])
def test_evict_lengths_apart(apart):
    assert "too many" in evict(P + 64, P + 64 + apart)
