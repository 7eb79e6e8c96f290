"""Calls of the tables on the device and of the attention over selected blocks at the ends of
what their documentation allows: the most lists, batches in which some sequences gain nothing,
outputs without rows, tensors of other kinds of device."""
import numpy as np
import pytest


@pytest.fixture(scope="module")
def pk():
    from paged_kv_cache_92_gb300 import build

    build.build()
    import paged_kv_cache_92_gb300 as pk

    pk.load()
    return pk


def dev(x):
    import torch

    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("B,H", [(65535, 257), (32768, 1024)])
def test_decode_of_more_lists_than_24_bits(pk, B, H):
    """From 2^24 lists on (a CTA of 128 threads each) a thread's number passes 32 bits; at 2^25
    the threads of the grid do so to the last bit. Sequences of one token: the output is its row
    of V, to the bit (a weight of 2^7 over a sum of 2^7)."""
    import torch

    D, BS = 64, 8
    k, v = (torch.randn(3, H, BS, D, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(1024, H, D, device="cuda").bfloat16().repeat(-(-B // 1024), 1, 1)[:B]
    tables = (torch.arange(B, dtype=torch.int32, device="cuda") % 3).view(B, 1).contiguous()
    sel = torch.zeros(B, H, 1, dtype=torch.int32, device="cuda")
    lens = torch.ones(B, dtype=torch.int32, device="cuda")
    out = pk.pa_decode_selected(q, k, v, tables, lens, BS, sel)
    assert pk.pa_device_errors() == 0
    for b in range(3):
        assert (out[b::3] == v[b, :, 0]).all()
    # a length past the table row is reported wherever its sequence is, and counts as a full row
    for b in (0, B // 2, B - 1):
        bad = lens.clone()
        bad[b] = BS + 1
        full = lens.clone()
        full[b] = BS
        got = pk.pa_decode_selected(q, k, v, tables, bad, BS, sel, out=out)[b].clone()
        assert pk.pa_device_errors() == pk.DEVERR_CONTEXT_LEN
        pk.pa_decode_selected(q, k, v, tables, full, BS, sel, out=out)
        assert pk.pa_device_errors() == 0 and torch.equal(out[b], got)


@pytest.mark.gpu
@pytest.mark.parametrize("B,Q,G,H", [(1, 1, 8, 2), (70, 3, 8, 2), (5, 9, 1, 3)])
def test_decode_reports_each_sequence(pk, B, Q, G, H):
    """One bad length in the batch, too long or shorter than the new tokens, is reported whatever
    the lists, column groups and CTAs of a list."""
    import torch

    k, v = (torch.randn(4, H, 16, 64, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(B, Q, G * H, 64, device="cuda").bfloat16()
    tables = torch.zeros(B, 40, dtype=torch.int32, device="cuda")
    sel = torch.zeros(B, H, 40, dtype=torch.int32, device="cuda")
    for b in {0, B // 2, B - 1}:
        for n, bit in ((641, True), (640, False), (0, False), (-7, False), (Q - 1, Q > 1)):
            lens = torch.full((B,), 500, dtype=torch.int32, device="cuda")
            lens[b] = n
            pk.pa_decode_selected(q, k, v, tables, lens, 640, sel)
            assert pk.pa_device_errors() == (pk.DEVERR_CONTEXT_LEN if bit else 0), (b, n)
