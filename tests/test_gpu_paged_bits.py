"""The paged attention's bits, against the 64-bit oracle: what its weights and
queries may lose on the way into a product, whatever the number of keys and
whichever block of rows takes them.

bf16 caches: a weight is the sum of two bf16 numbers, each rounded: 2^-16 of
it; with more than 16 rows of a sequence and KV head one number: 2^-8.  E4M3
caches: a weight is rounded to fp16 and to 9 bits, half a step of which is
2^-9, and moved by half a step of the cut, 2^-11 at the most: 2^-9 + 2^-10 with
fp16's own; it keeps half a step of 2^-28 (2^-25 with more than 32 rows) of the
reference that weight x V scale refers to, twice that of the largest weight
times the largest |v| where the pages' scales are alike.  An element of q over
an E4M3 cache is held to 2^-21 of its row's largest.  fp32 logits, exponentials
and sums: 2^-15 for logits up to some tens.  The result is rounded once: 2^-8.
"""
import numpy as np
import pytest
import torch

from oracle import paged as ref
from tests.paged_case import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dsa():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from __graft_entry__ import build
    build()
    from ar_image_gen_gb300 import dsa as mod
    return mod


def stored(kv, c):
    if c.kv == "bf16":
        return kv.pages.double().cpu().numpy()
    codes = kv.pages.contiguous().view(torch.uint8).cpu().numpy().reshape(c.codes.shape)
    return ref.e4m3_decode(codes) * kv.scales.double().cpu().numpy()[:, :, None, :, None]


def attend_and_check(c, max_new=None, k=None, v=None, logits=0.0):
    """Appends the new tokens (or k and v), attends and compares; `logits`: what the logits may be off by beside fp32."""
    kv = c.cache()
    cu, lens, table = c.batch()
    if k is None:
        kv.append(None, c.k.cuda(), c.v.cuda(), cu, lens, table)
    else:  # every token of the one sequence
        kv.append(None, k.cuda(), v.cuda(), torch.tensor([0, k.shape[0]], dtype=torch.int32, device="cuda"), lens, table)
    out = torch.empty_like(c.q, device="cuda")
    kv.attend(c.q.cuda(), cu, lens, table, out, max_new=max_new or int(max(c.new)))
    assert kv.sync_status() == 0
    compare(c, out, stored(kv, c), logits, (max_new or max(c.new)) * c.Hq // c.Hk)


def compare(c, out, values, logits=0.0, rows=1):
    want, reach, floor = ref.attend(c.q.double().numpy(), values, c.cu, c.lens, c.table)
    weights = 2.0 ** -9 + 2.0 ** -10 if c.kv != "bf16" else 2.0 ** -8 if rows > 16 else 2.0 ** -16
    tol = (weights + 2.0 ** -15 + np.expm1(2 * logits)) * reach + 2.0 ** -8 * np.abs(want)
    if c.kv != "bf16":
        tol += 2.0 ** (-25 if rows > 32 else -28) * floor
    err = np.abs(out.double().cpu().numpy() - want)
    assert (err <= tol).all(), (float((err > tol).mean()), float(np.nanmax(err / tol)), np.argwhere(~(err <= tol))[:3])


# query and KV heads, new tokens: blocks of 2, 8, 16, 32 and 128 rows
BLOCKS = [(3, 3, 1), (8, 2, 1), (16, 1, 1), (32, 1, 1), (8, 2, 40), (3, 3, 150)]


@pytest.mark.parametrize("kv", ["bf16", "fp8e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hk,new", BLOCKS)
def test_weights_keep_their_bits(dsa, kv, d, Hq, Hk, new):
    """Rows of a few keys, whose weights do not average each other's errors, and of some hundreds."""
    lens = [max(n, new) for n in (2, 3, 3, 4, 5, 6, 9, 14, 40, 130, 500)]
    attend_and_check(Case(kv, Hq, Hk, d, 16, lens, [new] * len(lens), seed=Hq + d))


@pytest.mark.parametrize("kv", ["bf16", "fp8e4m3"])
def test_every_hint_gives_the_same_result(dsa, kv):
    c = Case(kv, 8, 2, 128, 32, [200, 50, 7], [9, 1, 7], seed=4)
    for hint in (1, 2, 4, 9, 10000):
        attend_and_check(c, max_new=hint)


@pytest.mark.parametrize("kv", ["bf16", "fp8e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hk,new", BLOCKS[:5])
def test_many_small_weights_beside_a_large_one(dsa, kv, d, Hq, Hk, new):
    """A first key that takes nearly all of the weight and has next to no V: the output is the sum of thousands of
    weights of 2^-19 to 2^-22.  320 sequences of the same pages, so that rows are cut into few pieces."""
    n, S = 8200, 320
    c = Case(kv, Hq, Hk, d, 16, [n], [new], seed=3)
    g = torch.Generator().manual_seed(new + Hq)
    c.q[:] = 0
    c.q[:, :, 0] = 16
    k, v = torch.zeros((n, Hk, d)), 0.5 + torch.randn((n, Hk, d), generator=g).abs()
    unit = np.sqrt(d) / 16  # of one in the logit
    k[:, :, 0] = unit * 2 * torch.rand((n, Hk), generator=g)
    k[0, :, 0] = unit * 15
    v[0] = 2.0 ** -12
    cache = c.cache()
    cu, lens, table = c.batch()
    cache.append(None, k.to(torch.bfloat16).cuda(), v.to(torch.bfloat16).cuda(),
                 torch.tensor([0, n], dtype=torch.int32, device="cuda"), lens, table)
    q = c.q.cuda().repeat(S, 1, 1)
    out = torch.empty_like(q)
    cache.attend(q, torch.arange(S + 1, dtype=torch.int32, device="cuda") * new, lens.repeat(S), table.repeat(S, 1), out, max_new=new)
    assert cache.sync_status() == 0
    for got in out.reshape(S, new, Hq, d).unique(dim=0):
        compare(c, got, stored(cache, c), rows=new * Hq // Hk)


@pytest.mark.parametrize("Hq,Hk,new", BLOCKS[:5])
def test_queries_with_an_outlier(dsa, Hq, Hk, new):
    """Elements 2^-12 of their row's largest, alike, over keys of one sign: their errors add up in the logit."""
    d = 64
    n = max(new, 4)
    c = Case("fp8e4m3", Hq, Hk, d, 16, [n], [new], seed=5)
    c.q[:] = 49 / 1024
    c.q[:, :, 0] = 240
    k = (torch.arange(n) % 4 * 4 / 3)[:, None, None].expand(n, Hk, d).clone()
    k[:, :, 0] = 0
    v = torch.randn((n, Hk, d), generator=torch.Generator().manual_seed(1))
    # 63 elements, each off by 2^-21 of 240, with keys of 4
    attend_and_check(c, k=k.to(torch.bfloat16), v=v.to(torch.bfloat16), logits=63 * 240 * 2.0 ** -21 * 4 / 8)
