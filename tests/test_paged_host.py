"""The paged cache on the CPU: what its Python form refuses and decides before
it reaches the library, with CPU tensors and a fake pool of another device, and
the oracle at the ends of its range."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import paged as ref


@pytest.fixture(scope="module")
def dsa():
    from __graft_entry__ import build
    build()
    from ar_image_gen_gb300 import dsa as mod
    return mod


class FakePool:
    """Shape, type and place of a CUDA tensor."""

    def __init__(self, shape, dtype, device):
        self.shape, self.dtype, self.device_index, self.is_cuda = torch.Size(shape), dtype, device, True

    def get_device(self):
        return self.device_index

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20


@pytest.mark.parametrize("pages,scales", [(1, 1), (1, 0), (0, 1)])
def test_a_pool_of_another_device_is_refused(dsa, monkeypatch, pages, scales):
    """Before anything is made on the current device, 0."""
    monkeypatch.setattr(dsa, "_current_device", lambda: 0)

    def never(*a):
        raise AssertionError("reached the library")

    monkeypatch.setattr(dsa, "dsa_paged_create", never)
    with pytest.raises(ValueError):
        dsa.PagedKV(2, 2, 64, 16, 3, "fp8e4m3", pages=FakePool((3, 2, 16, 2, 64), torch.float8_e4m3fn, pages),
                    scales=FakePool((3, 2, 2), torch.float32, scales))


@pytest.fixture
def cache(dsa, monkeypatch):
    """A cache object over CPU tensors whose library calls are recorded, not made."""
    calls = []

    class Library:
        def dsa_paged_attend(self, *a):
            calls.append(a)
            return dsa.DSA_OK

        dsa_paged_append = dsa_paged_attend

    monkeypatch.setattr(dsa, "_L", Library())
    kv = dsa.PagedKV.__new__(dsa.PagedKV)
    kv.h, kv.device, kv._bf16, kv._int32 = ctypes.c_void_p(), -1, torch.bfloat16, torch.int32
    kv.q_heads, kv.kv_heads, kv.head_dim, kv.page_size = 4, 2, 64, 16
    yield kv, calls
    kv.h = None


def batch(n_seqs, n):
    return (torch.zeros(n_seqs + 1, dtype=torch.int32), torch.zeros(n_seqs, dtype=torch.int32),
            torch.zeros((n_seqs, 3), dtype=torch.int32)), torch.zeros((n, 4, 64), dtype=torch.bfloat16)


@pytest.mark.parametrize("n_seqs,n,hint", [(96, 96, 1), (3, 3, 1), (4, 2, 1), (1, 500, 500), (2, 1025, 513), (32, 160, 5), (0, 0, 1),
                                           (3, 0, 1), (0, 5, 5)])
def test_attend_without_a_hint_takes_the_mean(dsa, cache, n_seqs, n, hint):
    kv, calls = cache
    (cu, lens, table), q = batch(n_seqs, n)
    kv.attend(q, cu, lens, table, torch.zeros_like(q), stream=0)
    assert calls[-1][3] == hint
    kv.attend(q, cu, lens, table, torch.zeros_like(q), max_new=7, stream=0)
    assert calls[-1][3] == 7


def test_append_refuses_half_a_pair(dsa, cache):
    """Positions without a plan, and an output for queries that are not given, would be ignored in silence."""
    kv, calls = cache
    (cu, lens, table), q = batch(2, 5)
    k = torch.zeros((5, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        kv.append(None, k, k, cu, lens, table, pos=torch.zeros((5, 1), dtype=torch.int32), stream=0)
    with pytest.raises(ValueError):
        kv.append(None, k, k, cu, lens, table, q, stream=0)
    assert not calls
    kv.append(None, k, k, cu, lens, table, stream=0)
    assert len(calls) == 1


def test_the_oracle_takes_keys_of_any_size():
    """The exponent of the K scale by rational arithmetic: the smallest e with x^2 + z^2 <= (448 2^e)^2."""
    def smallest(x, z):
        top = Fraction(x) ** 2 + Fraction(z) ** 2
        return next(e for e in range(-72, 121) if e == 120 or top <= (448 * Fraction(2) ** e) ** 2)

    g = np.random.default_rng(0)
    sizes = [(1.75 * 2.0 ** e, 0.0) for e in (-64, -63, 0, 63, 64, 90, 127)] + [(1.7578125 * 2.0 ** e, 0.0) for e in (-64, -63, 60, 64, 90)]
    sizes += [(m * 2.0 ** e, n * 2.0 ** e) for e in (-80, -66, -64, -63, -1, 30, 62, 64, 66, 99, 126)
              for m, n in np.round(g.uniform(1, 2, (20, 2)) * 128) / 128]
    for x, z in sizes:
        k = np.zeros((1, 64))
        k[0, 3], k[0, 35] = x, z
        assert ref._smallest(ref.k_reach(k, 32)[0]) == smallest(x, z), (x, z)
