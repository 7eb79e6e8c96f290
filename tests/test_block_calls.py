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


# ------------------------------------------------------------------ bounds: whose blocks


def token_bounds(codes, bounds, tables, old, lens, BS):
    """`bounds` (float64) with those of the blocks that hold a token old <= t < lens, over the
    block's tokens t < lens."""
    out = bounds.copy()
    for b, n in enumerate(lens):
        for j in sorted({t // BS for t in range(max(old[b], 0), n)}):
            x = codes[tables[b, j], :, :min(BS, n - j * BS)]
            out[tables[b, j], :, 0], out[tables[b, j], :, 1] = x.min(1), x.max(1)
    return out


def cache_of(fmt, NB, H, BS, D, seed):
    """A K cache on the host, and its values without the head's scale."""
    import torch

    import oracle

    rng = np.random.default_rng(seed)
    if fmt == "bf16":
        k = torch.from_numpy(rng.standard_normal((NB, H, BS, D)).astype(np.float32)).bfloat16()
        return k, k.double().numpy()
    if fmt == "fp8":
        k = rng.integers(0, 256, (NB, H, BS, D), dtype=np.uint8)
        k[(k & 0x7F) == 0x7F] = 0
        return torch.from_numpy(k), oracle.e4m3_to_f64(k)
    k = rng.integers(0, 256, (NB, H, BS, D * 9 // 16), dtype=np.uint8)
    f = k.reshape(NB, H, -1)[..., BS * D // 2:]
    f[:] = rng.integers(0x28, 0x48, f.shape)
    return torch.from_numpy(k), oracle.fp4_values(k, np.ones(H, np.float32), D)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("D,BS,H", [(64, 8, 3), (128, 16, 8), (64, 32, 1), (128, 32, 2)])
def test_bounds_of_blocks_with_new_tokens_alone(pk, fmt, D, BS, H):
    """Sequences that gain tokens, none, or fewer than they had (in the same block, in another):
    blocks without a new token are left as they were."""
    import torch

    lens = [0, 1, BS, BS + 1, 7 * BS - 1, 100, 333, 3 * BS + 2, 2 * BS, 50]
    blocks = [-(-n // BS) + 1 for n in lens]
    NB = sum(blocks) + 2
    ids = np.random.default_rng(BS).permutation(NB).astype(np.int32)
    tables, at = np.full((len(lens), max(blocks)), -1, np.int32), 0
    for b, n in enumerate(blocks):
        tables[b, :n], at = ids[at:at + n], at + n
    k, codes = cache_of(fmt, NB, H, BS, D, 7)
    olds = {"all new": ([0] * 10, 333), "none new": (list(lens), 1),
            "some": ([0, 0, BS - 1, BS, 6 * BS, 100, 333, 3 * BS, 2 * BS - 1, 49], BS),
            "fewer": ([3, 2, BS + 1, BS + 2, 7 * BS, 101, 336, 3 * BS + 4, 2 * BS + 1, 64], 1),
            "some idle": ([0, 1, BS, BS, 7 * BS - 1, 99, 333, 3 * BS + 1, 2 * BS, 0], 50)}
    for name, (old, most) in olds.items():
        start = torch.randn(NB, H, 2, D).bfloat16()
        got = start.cuda()
        pk.pa_block_bounds(k.cuda(), got, dev(tables), dev(np.array(lens, np.int32)), most,
                           old_lens=dev(np.array(old, np.int32)))
        want = token_bounds(codes, start.double().numpy(), tables, old, lens, BS)
        assert np.array_equal(got.double().cpu().numpy(), want), name
        assert pk.pa_device_errors() == 0, name


@pytest.mark.gpu
def test_bounds_of_a_block_that_an_idle_sequence_shares(pk):
    """300 sequences of 20 tokens that gain none share the second block of one that grew to 32:
    the block's bounds are the grown one's, whoever comes last."""
    import torch

    k, codes = cache_of("bf16", 303, 2, 16, 128, 5)
    B = 301
    tables = np.stack([np.arange(B), np.full(B, 302)], 1).astype(np.int32)
    lens, old = np.full(B, 20, np.int32), np.full(B, 20, np.int32)
    for at in (0, 150, 300):  # the one that grew
        n = lens.copy()
        n[at] = 32
        start = torch.randn(303, 2, 2, 128).bfloat16()
        want = token_bounds(codes, start.double().numpy(), tables, old, n, 16)
        for _ in range(5):
            got = start.cuda()
            pk.pa_block_bounds(k.cuda(), got, dev(tables), dev(n), 12, old_lens=dev(old))
            assert np.array_equal(got.double().cpu().numpy(), want)
    assert pk.pa_device_errors() == 0


@pytest.mark.gpu
def test_bounds_still_report_lengths(pk):
    """A length past the table row is reported, with new tokens and without."""
    import torch

    k, _ = cache_of("bf16", 4, 1, 16, 64, 5)
    tables = dev(np.array([[0, 1], [2, 3]], np.int32))
    for lens, old, most, bit in (([40, 20], [40, 20], 1, True), ([20, 33], [20, 20], 13, True),
                                 ([2**31 - 1, 1], [2**31 - 1, 1], 1, True),
                                 ([32, 32], [32, 32], 1, False), ([32, 32], [0, 32], 1, True),
                                 ([-4, 3], [7, -2], 3, False)):
        got = torch.zeros(4, 1, 2, 64, dtype=torch.bfloat16, device="cuda")
        pk.pa_block_bounds(k.cuda(), got, tables, dev(np.array(lens, np.int32)), most,
                           old_lens=dev(np.array(old, np.int32)))
        assert pk.pa_device_errors() == (pk.DEVERR_CONTEXT_LEN if bit else 0), (lens, old)


# ------------------------------------------------------------------ tables: outputs without rows


@pytest.mark.gpu
@pytest.mark.parametrize("slots,positions", [(True, False), (False, True), (True, True)])
def test_tables_without_rows_for_new_tokens(pk, slots, positions):
    """An output that is given and has no rows has no room for a new token: the step is refused
    and changes nothing, as with any other number of rows. A step that gains none is done."""
    import torch

    def go(old, new):
        tables = torch.tensor([[3, -1, -1], [1, 2, -1]], dtype=torch.int32, device="cuda")
        ring, state = pk.make_free_ring([0, 4, 5], 6)
        out = torch.full((4,), 9, dtype=torch.int32, device="cuda")
        before = tables.tolist(), ring.tolist()
        rows = dict(slot_mapping=torch.empty(0, dtype=torch.int64, device="cuda") if slots else None,
                    positions=torch.empty(0, dtype=torch.int32, device="cuda") if positions else None)
        pk.pa_update_tables(tables, dev(np.array(old, np.int32)), dev(np.array(new, np.int32)), ring,
                            state, out, 6, 16, **rows)
        return out.tolist(), before == (tables.tolist(), ring.tolist()), pk.pa_device_errors()

    assert go([16, 20], [17, 20]) == ([0, 3, -1, 0], True, pk.DEVERR_CONTEXT_LEN)
    assert go([16, 20], [16, 21]) == ([0, 3, -1, 0], True, pk.DEVERR_CONTEXT_LEN)
    assert go([16, 20], [16, 20]) == ([0, 3, 0, 0], True, 0)
    assert go([16, 20], [16, 3]) == ([0, 4, 0, 0], False, 0)


@pytest.mark.gpu
def test_tables_without_rows_or_outputs_grow(pk):
    """Without slots and positions (None) any number of new tokens is taken."""
    import torch

    tables = torch.tensor([[3, -1, -1]], dtype=torch.int32, device="cuda")
    ring, state = pk.make_free_ring([0, 4, 5], 6)
    out = torch.full((4,), 9, dtype=torch.int32, device="cuda")
    pk.pa_update_tables(tables, dev(np.array([16], np.int32)), dev(np.array([40], np.int32)), ring,
                        state, out, 6, 16)
    assert tables.tolist() == [[3, 0, 4]] and out.tolist() == [2, 1, 0, 0]
    assert pk.pa_device_errors() == 0


@pytest.mark.gpu
def test_tables_arrays_of_no_bytes_overlap_nothing(pk):
    """No sequences and no rows: arrays of no bytes may point anywhere, into an output too."""
    import ctypes

    import torch

    ring, state = pk.make_free_ring([0, 4, 5], 6)
    out = torch.full((4,), 9, dtype=torch.int32, device="cuda")
    p = pk.UpdateTablesParams(
        ring.data_ptr(), ring.data_ptr() + 4, ring.data_ptr() + 8, ring.data_ptr(),
        state.data_ptr(), out.data_ptr(), state.data_ptr() + 8, state.data_ptr() + 4, None, 3, 0, 16,
        6, 6, 0)
    assert pk.load().pa_update_tables(ctypes.byref(p), pk._stream_handle(None)) == 0
    assert out.tolist() == [0, 3, 0, 0] and pk.pa_device_errors() == 0


# ------------------------------------------------------------------ the binding


def test_another_kind_of_device_is_refused(pk, monkeypatch):
    """A tensor of another accelerator whose index is the current CUDA device's."""
    import torch

    class Elsewhere(torch.Tensor):
        def get_device(self):
            return 0

    pk._current()  # (binds torch's calls)
    monkeypatch.setattr(pk, "_device", lambda: 0)
    x = torch.zeros(4, dtype=torch.int32).as_subclass(Elsewhere)
    assert x.get_device() == 0 and x.data_ptr() != 0
    for call in (lambda: pk._ptr(x, torch.int32, "x", 0), lambda: pk._dev_ptr(x, torch.int32, "x")):
        with pytest.raises(ValueError, match="x must live on a CUDA device"):
            call()


@pytest.mark.gpu
def test_device_errors_of_several_kernels_at_once(pk):
    """The bits of all kernels since the last call, once; what none has set stays clear."""
    import torch

    i = lambda *x: dev(np.array(x, np.int32))  # noqa: E731
    ring, state = pk.make_free_ring([0], 4)
    k = torch.zeros(4, 1, 8, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    bounds = torch.zeros(pk.block_bounds_shape(4, 1, 64), dtype=torch.bfloat16, device="cuda")
    calls = [  # more blocks than there are; a table entry; a list past the blocks; a short row
        (lambda: pk.pa_update_tables(i([-1, -1]), i(0), i(16), ring, state, i(0, 0, 0, 0), 4, 8),
         pk.DEVERR_POOL),
        (lambda: pk.pa_block_bounds(k, bounds, i([9, 1]), i(16), 16), pk.DEVERR_TABLE_ENTRY),
        (lambda: pk.pa_decode_selected(q, k, k, i([0, 1]), i(8), 16, i([[1]])), pk.DEVERR_KEEP),
        (lambda: pk.pa_block_select(torch.zeros(1, 1, 2, device="cuda"), i(99), 8, 1, 0, 0),
         pk.DEVERR_CONTEXT_LEN)]
    torch.cuda.synchronize()
    assert pk.pa_device_errors() == 0
    for chosen in range(1 << len(calls)):
        want = 0
        for n, (call, bit) in enumerate(calls):
            if chosen >> n & 1:
                call()
                want |= bit
        assert pk.pa_device_errors() == want and pk.pa_device_errors() == 0
