"""Attention over a 4-bit cache in CTAs that fill half of an SM (the bound:
q4_cases.attend_reference)."""
import numpy as np
import pytest
import torch

import q4_cases as C
from oracle import q4 as Q
from paged_kv_cache_162_gb300 import _lib as L
from paged_kv_cache_162_gb300 import engine as E

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("S,Hkv,G,D,dtype,hi", [
    (20, 8, 8, 128, "bf16", 1024), (38, 8, 5, 64, "f16", 2048), (100, 3, 7, 128, "f16", 1500), (25, 8, 6, 64, "bf16", 5600),
    (160, 1, 8, 128, "bf16", 4000), (19, 9, 4, 128, "bf16", 1100), (33, 9, 12, 64, "f16", 1200), (20, 8, 10, 128, "bf16", 2000),
])
def test_two_units_per_sm(S, Hkv, G, D, dtype, hi):
    """Between one and two units for every SM: a CTA each that fills half of one."""
    rng = np.random.default_rng(hi)
    lens = rng.integers(1, hi + 1, S)
    lens[:3] = [hi, 0, 1]
    assert 152 < S * Hkv <= 304
    c = C.attend_case(43, S, Hkv * G, Hkv, D, 16, dtype, lens)
    out = run(c, C.on_gpu(c))
    ref, bound = C.attend_reference(c)
    assert (np.abs(Q.widen(C.bits_of(out), dtype) - ref) <= bound).all()
    assert L.pkv_get_device_errors() == 0
