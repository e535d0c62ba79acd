"""The host side of the 4-bit cache's calls without a GPU: which caches go with
which call."""
import pytest
import torch

from paged_kv_cache_162_gb300 import _lib as L
from paged_kv_cache_162_gb300 import engine as E

F16 = torch.float16


@pytest.fixture
def called(monkeypatch):
    """Names of the library's calls made, none of which runs."""
    names = []
    for name in ("pkv_paged_attention_decode", "pkv_decode_step", "pkv_paged_attention_decode_shared_prefix",
                 "pkv_reshape_and_cache", "pkv_copy_blocks", "pkv_copy_blocks_q4", "pkv_swap_blocks", "pkv_swap_blocks_q4"):
        monkeypatch.setattr(L, name, lambda *args, name=name, **kw: names.append(name))
    return names


def caches(q4):
    return [torch.zeros(4, 2, 16, 36, dtype=torch.uint8) if q4 else torch.zeros(4, 16, 2, 64, dtype=F16) for _ in range(2)]


CALLS = {
    "paged_attention_decode": lambda k, v, t: E.paged_attention_decode(t["q"], t["q"], k, v, t["bt"], t["n"]),
    "decode_step": lambda k, v, t: E.decode_step(t["q"], t["q"], t["q"], t["q"], k, v, t["bt"], t["n"], t["n"], t["n"], t["slots"]),
    "paged_attention_decode_shared_prefix":
        lambda k, v, t: E.paged_attention_decode_shared_prefix(t["q"], t["q"], k, v, t["bt"], t["n"], t["groups"]),
    "reshape_and_cache": lambda k, v, t: E.reshape_and_cache(t["q"], t["q"], k, v, t["slots"]),
}


@pytest.mark.parametrize("name", CALLS)
def test_calls_on_16_bit_caches_refuse_4_bit_ones(called, name):
    """A 4-bit block is smaller than the 16-bit one that the call would read or write there."""
    t = dict(q=torch.zeros(3, 2, 64, dtype=F16), bt=torch.zeros(3, 2, dtype=torch.int32), n=torch.ones(3, dtype=torch.int32),
             slots=torch.zeros(3, dtype=torch.int64), groups=torch.zeros(1, 3, dtype=torch.int32))
    (k, v), (k4, v4) = caches(False), caches(True)
    for pair in ((k4, v4), (k4, v), (k, v4)):
        with pytest.raises(L.PkvError, match=f"{name}: takes 16-bit caches"):
            CALLS[name](*pair, t)
    assert not called
    CALLS[name](k, v, t)
    assert called == ["pkv_" + name]


def test_copies_and_swaps_of_16_bit_blocks_refuse_4_bit_pools(called):
    (k, v), (k4, v4) = caches(False), caches(True)
    pairs = torch.zeros(1, 2, dtype=torch.int64)
    with pytest.raises(L.PkvError, match="copy_blocks"):
        E.copy_blocks(k, v4, pairs)
    for args in ((k, v, k4, v4), (k, v4, k, v), (k, v, k4, v), (k, v, k, v4)):
        with pytest.raises(L.PkvError, match="swap_blocks"):
            E.swap_blocks(*args, pairs, L.PKV_SWAP_OUT)
    assert not called
    E.copy_blocks(k, v, pairs), E.swap_blocks(k, v, k, v, pairs, L.PKV_SWAP_IN)
    E.copy_blocks(k4, v4, pairs), E.swap_blocks(k4, v4, k4, v4, pairs, L.PKV_SWAP_IN)
    assert called == ["pkv_copy_blocks", "pkv_swap_blocks", "pkv_copy_blocks_q4", "pkv_swap_blocks_q4"]


def test_copies_of_4_bit_blocks_refuse_pools_with_gaps(called):
    """K and V interleaved in one tensor: the blocks do not follow one another."""
    both = torch.zeros(4, 2, 2, 16, 36, dtype=torch.uint8)
    k, v = both[:, 0], both[:, 1]
    whole, pairs = caches(True), torch.zeros(1, 2, dtype=torch.int64)
    for args in ((k, v), (whole[0], v)):
        with pytest.raises(L.PkvError, match="copy_blocks.*contiguous"):
            E.copy_blocks(*args, pairs)
    for i in range(4):
        args = [*whole, *whole]
        args[i] = k
        with pytest.raises(L.PkvError, match="swap_blocks.*contiguous"):
            E.swap_blocks(*args, pairs, L.PKV_SWAP_OUT)
    assert not called
