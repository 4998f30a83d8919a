"""The paged cache at the ends of its range, against the 64-bit oracle: keys
of any size.  Tolerances: tests/test_gpu_paged.py.
"""
import pytest
import torch

from tests.paged_case import Case
from tests.test_gpu_paged import append_and_check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dsa():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from __graft_entry__ import build
    build()
    from ar_image_gen_gb300 import dsa as mod
    return mod


# ---- the K scale -----------------------------------------------------------

@pytest.mark.parametrize("pairs", [(), (20,), (64,)])
@pytest.mark.parametrize("new", [1, 3, 16, 40])
def test_keys_of_any_size_set_their_scale(dsa, new, pairs):
    """Norms from 2^-80 to nearly 2^128, far beyond where their squares leave fp32; chunks that stay in registers and
    chunks that do not."""
    sizes = [2.0 ** -80, 2.0 ** -64.5, 1.5 * 2.0 ** -64, 1.75 * 2.0 ** -64, 1.8125 * 2.0 ** -64, 2.0 ** -63, 2.0 ** -40, 1.0,
             2.0 ** 62, 2.0 ** 63.9, 2.0 ** 64, 1e20, 2.0 ** 66, 1e30, 2.0 ** 100, 2.0 ** 126]
    c = Case("fp8e4m3", 2, 2, 128, 64, [new] * len(sizes), [new] * len(sizes), seed=7)
    for s, size in enumerate(sizes):
        k = c.k[s * new:(s + 1) * new].double()
        # the largest pair or element has that size, in one element; the rest up to a quarter of it
        k *= size / 4 / k.abs().max()
        k[new // 2, :, 5] = size
        k[new // 2, :, 5 + 64] = 0
        c.k[s * new:(s + 1) * new] = k.to(torch.bfloat16)
    c.q[:] = 0
    append_and_check(dsa, c, pairs)


def test_a_scale_grows_to_a_large_key(dsa):
    """Codes that are there already move to the larger scale."""
    c = Case("fp8e4m3", 1, 1, 64, 16, [9, 12], [2, 1], seed=8)
    c.k[0], c.k[1], c.k[2] = 1e25, 1e21, 3e37
    append_and_check(dsa, c, ())
