"""The paged cache at the ends of its range, against the 64-bit oracle: keys
and V scales of any size, pages that are missing for whole tiles, tiles whose
logits leave nothing, calls after one that gave up and beside a reading of the status,
pools that are no device memory or pass 32 bits, appends side by side.  Tolerances: tests/test_gpu_paged.py, and
tests/paged_case.py for the attention.
"""
import numpy as np
import pytest
import torch

from oracle import paged as ref
from tests.paged_case import Case, check_attend
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


def attended(c, kv, values, table=None, status=0, max_new=None):
    """Attends the case over what kv holds and compares with the oracle over `values`."""
    cu, lens, dev_table = c.batch()
    out = torch.empty_like(c.q, device="cuda")
    kv.attend(c.q.cuda(), cu, lens, dev_table, out, max_new=max_new or int(max(c.new)))
    assert kv.sync_status() == status
    check_attend(out, ref.attend(c.q.double().numpy(), values, c.cu, c.lens, c.table if table is None else table), c.kv)


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


# ---- pages that are missing, and scales of 0 --------------------------------

@pytest.mark.parametrize("kv_type,zero", [("bf16", False), ("fp8e4m3", False), ("fp8e4m3", True)])
@pytest.mark.parametrize("lens,new,gone", [
    ([700], [1], 16), ([700], [3], 24), ([700], [12], 24), ([700], [40], 16), ([1500, 400], [40, 1], 24), ([20000], [1], 900),
    ([20000], [40], 900), ([20000], [1], 1248),
])
def test_tiles_of_missing_pages(dsa, kv_type, zero, lens, new, gone):
    """A dropped prefix: the first `gone` pages are no pages of the pool (or have scales of 0), tiles of nothing else
    among them; they hold zeros, whose weights count."""
    c = Case(kv_type, 4, 2, 64, 16, lens, new, seed=2)
    values = np.concatenate([c.values, np.zeros((1,) + c.values.shape[1:])])
    table = c.table.copy()
    for s in range(len(lens)):
        m = min(gone, (lens[s] - new[s]) // 16 - 1)
        table[s, :m] = c.n_pages
        if zero:
            c.scales[c.table[s, :m]] = 0
        else:
            c.table[s, :m] = -1
    kv = c.cache()
    cu, lens_d, t = c.batch()
    kv.append(None, c.k.cuda(), c.v.cuda(), cu, lens_d, t)
    assert kv.sync_status() == dsa.DSA_OK
    n = c.n_pages
    if kv_type == "bf16":
        values[:n] = kv.pages.double().cpu().numpy()
    else:
        codes = kv.pages.contiguous().view(torch.uint8).cpu().numpy().reshape(c.codes.shape)
        values[:n] = ref.e4m3_decode(codes) * kv.scales.double().cpu().numpy()[:, :, None, :, None]
    attended(c, kv, values, table, dsa.DSA_OK if zero else dsa.DSA_ERR_DEVICE_CHECK)


# ---- V scales ---------------------------------------------------------------

@pytest.mark.parametrize("e", [-72, 100, 119])
@pytest.mark.parametrize("new", [1, 6, 40])
def test_weights_beside_v_scales_of_any_size(dsa, e, new):
    """V scales at both ends: the sum of the weights keeps the small ones."""
    c = Case("fp8e4m3", 8, 2, 64, 16, [900, 300], [new, new], seed=4)
    c.codes = np.where(c.codes & 0x7f > 0x70, 0x30, c.codes).astype(np.uint8)  # up to 128; every slot a value
    c.scales[:, :, 1] = 2.0 ** e
    c.q *= 3
    attended(c, c.cache(), ref.e4m3_decode(c.codes) * c.scales[:, :, None, :, None])


# ---- logits that leave nothing ----------------------------------------------

@pytest.mark.parametrize("Hq,Hk,new", [(3, 3, 1), (8, 2, 1), (12, 1, 1), (8, 2, 40)])
@pytest.mark.parametrize("n,hidden", [(600, 128), (600, 300), (20000, 9000), (700, 0)])
def test_tiles_whose_logits_are_minus_infinity(dsa, Hq, Hk, new, n, hidden):
    """Keys of minus infinity weigh nothing, also where they fill the first tiles of a row or all of a piece."""
    c = Case("bf16", Hq, Hk, 64, 16, [n], [new], seed=6)
    kv = c.cache()
    cu, lens, table = c.batch()
    kv.append(None, c.k.cuda(), c.v.cuda(), cu, lens, table)
    c.q[:, :, 0] = 1
    values = kv.pages.double().cpu().numpy()
    for t in range(hidden):
        kv.pages[c.table[0, t // 16], :, t % 16, 0, 0] = float("-inf")
    values = kv.pages.double().cpu().numpy()
    attended(c, kv, values)


@pytest.mark.parametrize("kv_type", ["bf16", "fp8e4m3"])
@pytest.mark.parametrize("Hq,Hk,new", [(3, 3, 1), (8, 2, 1), (8, 2, 40)])
def test_logits_far_below_zero(dsa, kv_type, Hq, Hk, new):
    """Finite logits of -1e33 and less: the largest takes the row."""
    n = 300
    c = Case(kv_type, Hq, Hk, 64, 16, [n], [new], seed=6)
    c.q[:] = 0
    c.q[:, :, 0] = 2
    kv = c.cache()
    cu, lens, table = c.batch()
    k = torch.zeros((n, Hk, 64))
    k[:, :, 0] = -(1e34 * 2.0 ** torch.linspace(0, 8, n))[:, None]
    v = torch.randn((n, Hk, 64), generator=torch.Generator().manual_seed(0))
    kv.append(None, k.to(torch.bfloat16).cuda(), v.to(torch.bfloat16).cuda(), torch.tensor([0, n], dtype=torch.int32, device="cuda"),
              lens, table)
    if kv_type == "bf16":
        values = kv.pages.double().cpu().numpy()
    else:
        codes = kv.pages.contiguous().view(torch.uint8).cpu().numpy().reshape(c.codes.shape)
        values = ref.e4m3_decode(codes) * kv.scales.double().cpu().numpy()[:, :, None, :, None]
    attended(c, kv, values)


@pytest.mark.parametrize("Hq,Hk,new", [(3, 3, 1), (8, 2, 1), (12, 1, 1), (8, 2, 40)])
@pytest.mark.parametrize("n", [300, 20000])
def test_infinities_of_attended_values(dsa, Hq, Hk, new, n):
    """They reach the rows that attend them, as infinities, and no other element."""
    c = Case("bf16", Hq, Hk, 64, 16, [n], [new], seed=6)
    kv = c.cache()
    cu, lens, table = c.batch()
    kv.append(None, c.k.cuda(), c.v.cuda(), cu, lens, table)
    for t, e, x in ((7, 3, "inf"), (n // 2, 9, "-inf"), (n - 45, 20, "inf"), (5, 30, "nan")):
        kv.pages[c.table[0, t // 16], :, t % 16, 1, e] = float(x)
    out = torch.empty_like(c.q, device="cuda")
    kv.attend(c.q.cuda(), cu, lens, table, out, max_new=new)
    assert kv.sync_status() == dsa.DSA_OK
    got = out.float().cpu().numpy()
    assert (got[:, :, [3, 20]] == np.inf).all() and (got[:, :, 9] == -np.inf).all() and np.isnan(got[:, :, 30]).all()
    rest = [e for e in range(64) if e not in (3, 9, 20, 30)]
    assert np.isfinite(got[:, :, rest]).all()


# ---- after a call that gave up ----------------------------------------------

@pytest.mark.parametrize("kv_type,Hq,new,n_seqs", [("bf16", 1, 1, 800), ("fp8e4m3", 1, 1, 800), ("fp8e4m3", 4, 8, 400),
                                                   ("bf16", 8, 16, 300), ("fp8e4m3", 8, 16, 300)])
def test_a_call_after_one_that_gave_up(dsa, kv_type, Hq, new, n_seqs):
    """Several items a CTA, some of whose waits give up: the next call is whole, whether or not the status was read."""
    c = Case(kv_type, Hq, 1, 128, 16, [1500], [new], seed=2)
    kv = c.cache()
    _, lens, table = c.batch()
    kv.append(None, c.k.cuda(), c.v.cuda(), *c.batch())
    batch = torch.arange(n_seqs + 1, dtype=torch.int32, device="cuda") * new, lens.repeat(n_seqs), table.repeat(n_seqs, 1)
    q = c.q.cuda().repeat(n_seqs, 1, 1)
    first, out = torch.empty_like(q), torch.empty_like(q)
    kv.attend(q, *batch, first, max_new=new)
    assert kv.sync_status() == dsa.DSA_OK
    for limit in (0, 1, 2, 3, 4, 6) * 3:
        kv.attend(-q, *batch, out, max_new=new)  # what the workspace holds is of other queries
        kv.set_wait_limit(limit)
        kv.attend(-q, *batch, out, max_new=new)
        kv.set_wait_limit(0xffffffff)
        kv.attend(q, *batch, out, max_new=new)
        assert torch.equal(out, first), limit
    assert kv.sync_status() == dsa.DSA_ERR_TIMEOUT
    assert kv.sync_status() == dsa.DSA_OK


def test_reading_the_status_leaves_a_running_call_alone(dsa):
    """A bad append on one stream, an attention on another: what the first did is read while the second runs."""
    n_seqs = 800
    c = Case("bf16", 1, 1, 128, 16, [6000], [1], seed=2)
    kv = c.cache()
    _, lens, table = c.batch()
    k, v = c.k.cuda(), c.v.cuda()
    kv.append(None, k, v, *c.batch())
    batch = torch.arange(n_seqs + 1, dtype=torch.int32, device="cuda"), lens.repeat(n_seqs), table.repeat(n_seqs, 1)
    q = c.q.cuda().repeat(n_seqs, 1, 1)
    first, out = torch.empty_like(q), torch.empty_like(q)
    kv.attend(q, *batch, first, max_new=1)
    assert kv.sync_status() == dsa.DSA_OK
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    bad = torch.tensor([0, 1], dtype=torch.int32, device="cuda"), torch.tensor([-1], dtype=torch.int32, device="cuda"), table
    torch.cuda.synchronize()
    for _ in range(20):
        out.fill_(7.0)
        torch.cuda.synchronize()
        kv.append(None, k, v, *bad, stream=a)
        a.synchronize()
        kv.attend(q, *batch, out, max_new=1, stream=b)
        assert kv.sync_status(a) == dsa.DSA_ERR_DEVICE_CHECK
        torch.cuda.synchronize()
        assert torch.equal(out, first)
    assert kv.sync_status() == dsa.DSA_OK


def test_two_errors_are_read_one_after_the_other(dsa):
    c = Case("fp8e4m3", 2, 2, 64, 16, [20, 300], [1, 1], seed=2)
    kv = c.cache()
    cu, lens, table = c.batch()
    q = c.q.cuda()
    lens[0] = -1
    kv.set_wait_limit(0)
    kv.attend(q, cu, lens, table, torch.empty_like(q))
    kv.set_wait_limit(0xffffffff)
    assert [kv.sync_status() for _ in range(3)] == [dsa.DSA_ERR_TIMEOUT, dsa.DSA_ERR_DEVICE_CHECK, dsa.DSA_OK]


# ---- whose memory a pool is --------------------------------------------------

def test_a_pool_is_memory_of_the_current_device(dsa):
    """Host memory is refused where it can be told; memory of another device likewise (two devices at least)."""
    host = np.zeros(1 << 16, dtype=np.uint8)
    at = (host.ctypes.data + 127) // 128 * 128
    scales = torch.ones((1, 1, 2), device="cuda")
    pages = torch.zeros(1 << 13, dtype=torch.uint8, device="cuda")
    for p, s in ((at, scales), (pages, at)):
        code, h = dsa.dsa_paged_create(1, 1, 64, 16, 1, dsa.DSA_FP8_E4M3, p, s)
        assert code == dsa.DSA_ERR_ARG and not h.value and dsa.dsa_last_error()
    code, h = dsa.dsa_paged_create(1, 1, 64, 16, 1, dsa.DSA_FP8_E4M3, pages, scales)
    assert code == dsa.DSA_OK and dsa.dsa_paged_destroy(h) == dsa.DSA_OK


# ---- large pools, calls side by side -----------------------------------------

@pytest.mark.parametrize("kv_type,n_pages", [("bf16", 700000), ("fp8e4m3", 1200000)])
@pytest.mark.parametrize("new", [1, 40])
def test_pages_beyond_32_bits_of_bytes(dsa, kv_type, n_pages, new):
    """A pool of 5 GB: what its last pages hold and give equals what a small pool does, bit for bit."""
    c = Case(kv_type, 4, 1, 128, 16, [200, 77], [new, new], seed=3)
    small = c.cache()
    large = dsa.PagedKV(4, 1, 128, 16, n_pages, kv_type)
    assert large.pages.numel() * large.pages.element_size() > 2 ** 32
    large.pages[-c.n_pages:].view(torch.uint8).copy_(small.pages.view(torch.uint8))
    if kv_type != "bf16":
        large.scales[-c.n_pages:] = small.scales
    cu, lens, table = c.batch()
    far = torch.where(table >= 0, table + n_pages - c.n_pages, table)
    outs = []
    for kv, t in ((small, table), (large, far)):
        kv.append(None, c.k.cuda(), c.v.cuda(), cu, lens, t)
        outs.append(torch.empty_like(c.q, device="cuda"))
        kv.attend(c.q.cuda(), cu, lens, t, outs[-1], max_new=new)
        assert kv.sync_status() == dsa.DSA_OK
    assert torch.equal(large.pages[-c.n_pages:].view(torch.uint8), small.pages.view(torch.uint8))
    assert torch.equal(outs[0], outs[1]) and torch.isfinite(outs[0]).all()


def test_appends_side_by_side(dsa):
    """Two streams append to other pages of one pool through one handle."""
    c = Case("fp8e4m3", 2, 2, 128, 16, [900, 800], [900, 800], seed=9)
    together, apart = c.cache(), c.cache()
    _, lens, table = c.batch()
    k, v = c.k.cuda(), c.v.cuda()
    together.append(None, k, v, *c.batch())
    streams = [torch.cuda.Stream() for _ in range(2)]
    parts = []
    for s in range(2):
        a, b = int(c.cu[s]), int(c.cu[s + 1])
        parts.append((k[a:b], v[a:b], torch.tensor([0, b - a], dtype=torch.int32, device="cuda"), lens[s:s + 1].contiguous(),
                      table[s:s + 1].contiguous()))
    torch.cuda.synchronize()
    for _ in range(10):
        for st, part in zip(streams, parts):
            apart.append(None, *part, stream=st)
    torch.cuda.synchronize()
    assert together.sync_status() == dsa.DSA_OK and apart.sync_status() == dsa.DSA_OK
    assert torch.equal(apart.pages.view(torch.uint8), together.pages.view(torch.uint8))
    assert torch.equal(apart.scales, together.scales)
