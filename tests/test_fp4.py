"""The 4-bit KV cache: the quantising write, its read-back, the block copy and
the decode, against the oracle in float64.

Bit-exact: the write (whole caches compared: rounding ties, saturation, zeros,
NaN groups) and the copy. The read-back: the exact product rounded once to
float and once to bf16. The decode: the exact attention over the dequantised
cache; what the kernel rounds is the softmax weights, to f16, and the output,
to bf16. Half a step relative to the value is torch.finfo(t).eps / 2: 2^-11 in
f16 (2^-25 absolute below 2^-14, of weights whose largest is at least one) and
2^-8 in bf16 (eps is the step at one, and a value just above a power of two
has half of that as its largest relative error). Weights sum to one, so with
`a` the row's sum of weight times |V| an element is off by at most
  2^-11 a + 2^-25 L max|V|   for the weights,
  2^-8 |out|                 for the output, and
  2^-12 a                    for fp32: 20 roundings of 2^-24 in a score of
magnitude up to 64 are 2^-14 of a weight, the sums of up to 2^12 terms less.
Padding slots hold NaN scales, so a masked slot
that leaks into a result shows.
"""
import ctypes

import numpy as np
import pytest

import oracle
import workloads


@pytest.fixture(scope="module")
def pk():
    from paged_kv_cache_92_gb300 import build

    build.build()
    import paged_kv_cache_92_gb300 as pk

    pk.load()
    return pk


def _scales(Hkv, seed, base):
    rng = np.random.default_rng(seed)
    return (base * np.exp(rng.uniform(-0.5, 0.5, size=Hkv))).astype(np.float32)


def _tile(BS, D):
    return BS * D * 9 // 16


def _poison(cache, tables, lens, BS, D):
    """NaN scales and random codes in the slots past each sequence's end."""
    NB, Hkv = cache.shape[:2]
    flat = cache.reshape(NB, Hkv, -1)
    for b, L in enumerate(lens):
        if L % BS:
            blk, off = int(tables[b, (L - 1) // BS]), L % BS
            flat[blk, :, BS * D // 2 + off * D // 16:] = 0x7F
            flat[blk, :, off * D // 2:BS * D // 2] = 0xA5


class Case:
    """A batch on the 4-bit cache: random tables, rows with a few wide channels."""

    def __init__(self, lens, Hq, Hkv, D=128, BS=16, Q=1, seed=0, wide=4.0):
        import torch

        self.lens = np.asarray(lens, dtype=np.int32)
        self.Hq, self.Hkv, self.D, self.BS, self.Q = Hq, Hkv, D, BS, Q
        need = int(((self.lens + BS - 1) // BS).sum())
        self.NB = need + 3
        order = np.random.default_rng(seed).permutation(self.NB).astype(np.int32)
        self.tables = workloads.sequential_tables(self.lens.astype(np.int64), order, BS,
                                                  max(1, int(-(-self.lens.max() // BS))))
        self.ks, self.vs = _scales(Hkv, seed + 4, 0.05), _scales(Hkv, seed + 5, 0.03)
        spread = torch.ones(D)
        spread[5::16] = wide
        rows = [(workloads.bf16_normal((self.NB * BS, Hkv, D), seed + i).float() * spread
                 ).to(torch.bfloat16) for i in (2, 3)]
        slots = np.arange(self.NB * BS)
        zero = np.zeros((self.NB, Hkv, BS, D * 9 // 16), np.uint8)
        self.k, self.v = (oracle.fp4_write(oracle.bf16_to_f64(r), zero, slots, s, D)
                          for r, s in zip(rows, (self.ks, self.vs)))
        for c in (self.k, self.v):
            _poison(c, self.tables, self.lens, BS, D)
        self.q = workloads.bf16_normal((len(lens), Q, Hq, D), seed + 1)

    def cuda(self):
        import torch

        q = self.q if self.Q > 1 else self.q[:, 0].contiguous()
        return (q.cuda(), torch.from_numpy(self.k).cuda(), torch.from_numpy(self.v).cuda(),
                torch.from_numpy(self.tables).cuda(), torch.from_numpy(self.lens).cuda(),
                max(1, int(self.lens.max()))), dict(k_scale=torch.from_numpy(self.ks).cuda(),
                                                    v_scale=torch.from_numpy(self.vs).cuda())

    def cuda_cut(self):
        """The same batch with room for 4,096 tokens a sequence: the work is dealt out
        as a stream that cuts the sequences' keys into pieces of a few steps."""
        import torch

        a, sc = self.cuda()
        room = -(-4096 // self.BS)
        tab = torch.full((len(self.lens), room), -1, dtype=torch.int32, device="cuda")
        tab[:, :a[3].shape[1]] = a[3]
        return a[:3] + (tab, a[4], 4096), sc

    def want(self, scale=None):
        kr, vr = (oracle.fp4_values(c, s, self.D) for c, s in ((self.k, self.ks), (self.v, self.vs)))
        q = oracle.bf16_to_f64(self.q)
        out, w = oracle.attention_rows(q, kr, vr, self.tables, self.lens, scale)
        mag, _ = oracle.attention_rows(q, kr, np.abs(vr), self.tables, self.lens, scale)
        # the subnormal weights' share, as a part of `mag`
        flush = 2.0 ** -25 * int(self.lens.max()) * np.nanmax(np.abs(vr))
        return out, mag + flush / (2.0 ** -11 + 2.0 ** -12)


def _bound(out, mag):
    return 2.0 ** -8 * np.abs(out) + (2.0 ** -11 + 2.0 ** -12) * mag + 1e-30


def _check(pk, got, case, scale=None):
    got = oracle.bf16_to_f64(got.cpu()).reshape(len(case.lens), case.Q, case.Hq, case.D)
    want, mag = case.want(scale)
    assert np.isfinite(got).all()
    over = np.abs(got - want) / _bound(want, mag)
    assert over.max() <= 1.0, (over.max(), np.unravel_index(over.argmax(), over.shape))
    assert pk.pa_device_errors() == 0


# ------------------------------------------------------------------ the oracle


def test_oracle_grids_and_rounding():
    """The E4M3 grid equals the C oracle's table; nearest_code against brute force."""
    table = oracle.e4m3_to_f64(np.arange(127))
    assert np.array_equal(table, oracle._e4m3_grid())
    mids = (oracle.E2M1_GRID[1:] + oracle.E2M1_GRID[:-1]) / 2
    assert oracle.nearest_code(mids, oracle.E2M1_GRID).tolist() == [0, 2, 2, 4, 4, 6, 6]
    rng = np.random.default_rng(0)
    for grid in (oracle.E2M1_GRID, table):
        x = rng.uniform(0, grid[-1] * 1.2, 400)
        brute = np.array([int(np.argmin(np.abs(grid - v))) for v in x])
        assert np.array_equal(oracle.nearest_code(x, grid), brute)


def test_oracle_write_then_values_is_within_half_a_step():
    """Every element is within half the widest step (one group scale) of its row's value."""
    rng = np.random.default_rng(3)
    x = rng.standard_normal((6, 2, 64)).astype(np.float32)
    s = np.array([0.05, 0.4], np.float32)
    cache = oracle.fp4_write(x, np.zeros((1, 2, 8, 36), np.uint8), np.arange(6), s, 64)
    back = oracle.fp4_values(cache, s, 64)[0].transpose(1, 0, 2)[:6]
    group = np.abs(x).reshape(6, 2, 4, 16).max(-1, keepdims=True)
    # the group scale is within 2^-4 of max / 6, the grid's widest half step is one scale
    assert (np.abs(back - x).reshape(6, 2, 4, 16) <= group / 6 * (1 + 2 ** -4) + 1e-6).all()


def test_oracle_attention_rows_matches_decode_numpy():
    B, Hq, Hkv, D, NB = 3, 4, 2, 64, 8
    kc, vc = (oracle.bf16_bits(workloads.bf16_normal((NB, Hkv, 16, D), i)) for i in (1, 2))
    q = workloads.bf16_normal((B, Hq, D), 5)
    tables = np.array([[3, 1], [0, 7], [2, 6]], np.int32)
    lens = np.array([17, 32, 1], np.int32)
    want = oracle.paged_decode_numpy(q, kc, vc, tables, lens)
    got, w = oracle.attention_rows(oracle.bf16_to_f64(q)[:, None], oracle.bf16_to_f64(kc),
                                   oracle.bf16_to_f64(vc), tables, lens)
    assert np.allclose(got[:, 0], want, atol=1e-12)
    assert all(np.allclose(x.sum(-1), 1.0) for x in w)


# ------------------------------------------------------------------ refusals (CPU)


def _lib_params(pk, **kw):
    p = pk.DecodeParams()
    base = dict(max_blocks_per_seq=4, num_seqs=2, num_q_heads=8, num_kv_heads=2, head_dim=128,
                block_size=16, num_blocks=8, max_context_len=64, scale=0.088, kv_dtype=2)
    base.update(kw)
    for k, v in base.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("kw,status", [
    (dict(), 1),  # valid shapes, NULL pointers
    (dict(head_dim=96), 2), (dict(block_size=64), 2), (dict(num_q_heads=12, num_kv_heads=1), 2),
    (dict(kv_dtype=3), 1), (dict(partition_tokens=24), 1),
    (dict(partition_tokens=48, block_size=32), 1),  # partitions are whole blocks
    (dict(query_len=1025), 1), (dict(query_len=1024, num_seqs=64), 2),
    (dict(num_seqs=512, num_kv_heads=16, num_q_heads=16, max_blocks_per_seq=1 << 20,
          max_context_len=1 << 24), 2),  # more stream positions than 32 bits count
    (dict(max_context_len=0), 1), (dict(scale=0.0), 1),
])
def test_decode_refusals(pk, kw, status):
    p = _lib_params(pk, **kw)
    assert pk.load().pa_decode(ctypes.byref(p), None, 0, None) == status
    assert pk.load().pa_last_error()


@pytest.mark.parametrize("kw,words", [
    (dict(partition_tokens=48, block_size=32), b"partition_tokens must be a multiple of block_size"),
    (dict(query_len=1024, num_seqs=64), b"num_seqs * query_len <= 65535"),
    (dict(num_seqs=512, num_kv_heads=16, num_q_heads=16, max_blocks_per_seq=1 << 20,
          max_context_len=1 << 24), b"below 2^31")])
def test_decode_refusals_name_this_cache(pk, kw, words):
    """What a refusal says is about the 4-bit cache, not about a kernel that it never takes."""
    for variant in (0, 1):
        p = _lib_params(pk, variant=variant, **kw)
        assert pk.load().pa_decode(ctypes.byref(p), None, 0, None) in (1, 2)
        got = pk.load().pa_last_error()
        assert words in got and b"4-bit cache" in got and b"CUDA-core" not in got


def test_decode_longest_sequence(pk):
    """A sequence's steps are counted by rounding its length up in 32 bits."""
    for blocks, status in ((2 ** 26 - 1, 2), (2 ** 26 - 2, 1)):  # 2^31 - 32 and - 64 tokens
        p = _lib_params(pk, num_seqs=1, num_kv_heads=1, num_q_heads=1, block_size=32,
                        max_blocks_per_seq=blocks, max_context_len=2 ** 31 - 1)
        assert pk.load().pa_decode(ctypes.byref(p), None, 0, None) == status
        assert (b"2^31 - 64" in pk.load().pa_last_error()) == (status == 2)
        assert (pk.load().pa_decode_workspace_size(ctypes.byref(p)) > 0) == (status == 1)
        p.max_context_len = 4096  # the bound on the lengths, whatever the tables hold
        assert pk.load().pa_decode(ctypes.byref(p), None, 0, None) == 1


@pytest.mark.parametrize("name", ["pa_reshape_and_cache_fp4", "pa_gather_fp4"])
@pytest.mark.parametrize("dims,status", [
    ((-1, 2, 64, 16, 4), 1), ((2, 0, 64, 16, 4), 1), ((2, 2, 96, 16, 4), 2),
    ((2, 2, 64, 12, 4), 2), ((2, 2, 64, 16, 0), 1), ((2, 2, 64, 16, 4), 1), ((0, 2, 64, 16, 4), 0)])
def test_row_call_refusals(pk, name, dims, status):
    lib = pk.load()
    assert getattr(lib, name)(*([None] * 7), *dims, None) == status
    # misaligned rows (never dereferenced: refused on the host)
    if status == 1 and dims[0] == 2 and dims[1] and dims[4]:
        assert getattr(lib, name)(8, 16, 16, 16, 16, 16, 16, *dims, None) == 1
        assert b"misaligned" in lib.pa_last_error()


@pytest.mark.parametrize("dims,status", [
    ((-1, 2, 64, 16, 4), 1), ((70000, 2, 64, 16, 4), 1), ((2, 2, 32, 16, 4), 2),
    ((2, 2, 64, 4, 4), 2), ((2, 2, 64, 16, 4), 1), ((0, 2, 64, 16, 4), 0)])
def test_copy_refusals(pk, dims, status):
    assert pk.load().pa_copy_blocks_fp4(None, None, None, *dims, None) == status


def test_binding_refuses_mixed_shapes(pk):
    import torch

    k = torch.zeros(pk.fp4_cache_shape(4, 2, 16, 128), dtype=torch.uint8)
    assert tuple(k.shape) == (4, 2, 16, 72)
    assert pk.kv_cache_format(k) == (pk.KV_FP4_E2M1, 128)
    assert pk.kv_cache_format(k[..., :36]) == (pk.KV_FP4_E2M1, 64)
    assert pk.kv_cache_format(torch.zeros(1, 1, 16, 64, dtype=torch.uint8)) == (1, 64)
    rows = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    slots, s = torch.zeros(3, dtype=torch.int64), torch.ones(2)
    with pytest.raises(ValueError):
        pk.pa_reshape_and_cache_fp4(rows[..., :64], rows[..., :64], k, k, slots, s, s)
    with pytest.raises(ValueError):
        pk.pa_reshape_and_cache_fp4(rows, rows, k, k, slots, s[:1], s)
    with pytest.raises(ValueError):
        pk.pa_gather_fp4(k.view(4, 2, 36, 32), k, slots, s, s)
    with pytest.raises(ValueError):
        pk.fp4_cache_shape(4, 2, 16, 96)
    q = torch.zeros(1, 4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # the caches differ in shape
        pk.make_decode_params(q, q, k, k[:3], torch.zeros(1, 1, dtype=torch.int32),
                              torch.zeros(1, dtype=torch.int32), 16)


def test_workspace_holds_two_partials_per_cta(pk):
    """The header alone where contexts are short (at most 1,024 tokens); else the plan (a
    cost per sequence and column group, and the total) and two partials a CTA:
    four CTAs an SM, or one per 16 steps and starts."""
    def size(**kw):
        return pk.load().pa_decode_workspace_size(ctypes.byref(_lib_params(pk, **kw)))

    def ru(x):
        return (x + 255) // 256 * 256

    assert size() == size(max_blocks_per_seq=64, max_context_len=1024) == 256
    assert size(max_blocks_per_seq=64, max_context_len=4096) == 256  # the table holds 1,024
    kw = dict(max_blocks_per_seq=128, max_context_len=1056)
    grid = 2 * 2 * (33 + 8) // 16          # items x (steps + start), 16 a CTA
    rows = 2 * grid * 8
    assert size(**kw) == 256 + ru(3 * 4) + ru(rows * 8) + ru(rows * 128 * 4)
    kw["query_len"] = 9                    # groups of two tokens (G 4): five
    grid = 2 * 5 * 2 * (33 + 8) // 16
    rows = 2 * grid * 8
    assert size(**kw) == 256 + ru(11 * 4) + ru(rows * 8) + ru(rows * 128 * 4)


# ------------------------------------------------------------------ GPU: rows


def _special_rows(T, Hkv, D, rng):
    """Rows with ties on every grid midpoint, saturation, zeros, tiny and huge values."""
    x = rng.standard_normal((T, Hkv, D)) * 8
    g = x.reshape(-1, 16)
    mids = (oracle.E2M1_GRID[1:] + oracle.E2M1_GRID[:-1]) / 2
    for i in range(0, min(8, len(g))):  # group maximum 6 * 2^k: with scale 1 the step is 2^k
        g[i, :8] = np.append(mids, 6.0) * 2.0 ** (i - 4)
        g[i, 8:] = -g[i, :8]
    g[8] = 0.0
    g[9] = -0.0
    g[10, 3] = 3e4      # beyond 448 * 6: the group scale saturates
    g[11] = 1e-6        # below the smallest scale
    g[12, 5] = np.inf
    g[13, 2] = np.nan
    g[14] = 2.0 ** -9 * 6 * np.linspace(-1, 1, 16)  # the smallest scale (subnormal E4M3)
    return x


@pytest.mark.gpu
@pytest.mark.parametrize("D,BS", [(64, 8), (128, 16), (64, 32), (128, 8)])
def test_write_bit_exact_and_read_back(pk, D, BS):
    import torch

    T, Hkv, NB = 37, 3, 12
    rng = np.random.default_rng(D + BS)
    rows = [torch.from_numpy(_special_rows(T, Hkv, D, rng)).to(torch.bfloat16) for _ in range(2)]
    ks, vs = np.array([1.0, 0.37, 2.0 ** -20], np.float32), np.array([1.0, 3.0, 1e3], np.float32)
    slots = rng.permutation(NB * BS)[:T].astype(np.int64)
    slots[[3, 17]] = -1
    shape = pk.fp4_cache_shape(NB, Hkv, BS, D)
    old = [rng.integers(0, 256, size=shape, dtype=np.uint8) for _ in range(2)]
    kc, vc = (torch.from_numpy(c).cuda() for c in old)
    s_gpu = [torch.from_numpy(s).cuda() for s in (ks, vs)]
    pk.pa_reshape_and_cache_fp4(rows[0].cuda(), rows[1].cuda(), kc, vc,
                                torch.from_numpy(slots).cuda(), *s_gpu)
    torch.cuda.synchronize()
    for got, o, r, s in zip((kc, vc), old, rows, (ks, vs)):
        want = oracle.fp4_write(oracle.bf16_to_f64(r), o, slots, s, D)
        assert np.array_equal(got.cpu().numpy(), want)
    # the read-back, a slot twice and negative slots among them
    pick = np.concatenate([slots, slots[:2], [-1]]).astype(np.int64)
    out = pk.pa_gather_fp4(kc, vc, torch.from_numpy(pick).cuda(), *s_gpu)
    torch.cuda.synchronize()
    for got, c, s in zip(out, (kc, vc), (ks, vs)):
        val = oracle.fp4_values(c.cpu().numpy(), np.ones(Hkv), D)  # exact in float32
        val = val.transpose(0, 2, 1, 3).reshape(NB * BS, Hkv, D)
        with np.errstate(over="ignore", invalid="ignore"):
            f = val[np.maximum(pick, 0)].astype(np.float32) * s[:, None]
        f[pick < 0] = 0
        want = torch.from_numpy(f).to(torch.bfloat16)
        assert torch.equal(got.cpu().view(torch.int16), want.view(torch.int16)) or torch.equal(
            torch.nan_to_num(got.cpu().float()), torch.nan_to_num(want.float()))
        assert torch.equal(torch.isnan(got.cpu()), torch.isnan(want))
    assert pk.pa_device_errors() == 0


@pytest.mark.gpu
def test_write_covers_every_bf16_value(pk):
    """All 65,536 bf16 patterns, 16 to a group, under several head scales."""
    import torch

    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    perm = torch.from_numpy(np.random.default_rng(1).permutation(65536))
    # neighbours in magnitude share a group, and a second copy mixes magnitudes
    rows = torch.cat([bits, bits[perm]]).view(torch.bfloat16).view(-1, 1, 128)
    T = rows.shape[0]
    for s in (1.0, 2.0 ** -30, 0.037, 2.0 ** 40):
        sc = np.array([s], np.float32)
        kc = torch.zeros(pk.fp4_cache_shape(T // 16, 1, 16, 128), dtype=torch.uint8, device="cuda")
        vc = kc.clone()
        g = torch.from_numpy(sc).cuda()
        r = rows.cuda()
        pk.pa_reshape_and_cache_fp4(r, r, kc, vc, torch.arange(T, device="cuda"), g, g)
        torch.cuda.synchronize()
        want = oracle.fp4_write(oracle.bf16_to_f64(rows), np.zeros(tuple(kc.shape), np.uint8),
                                np.arange(T), sc, 128)
        assert np.array_equal(kc.cpu().numpy(), want)
        assert torch.equal(kc, vc)


@pytest.mark.gpu
@pytest.mark.parametrize("D,BS,Hkv", [(64, 8, 1), (128, 16, 8), (64, 32, 3)])
def test_copy_blocks_bit_exact(pk, D, BS, Hkv):
    import torch

    rng = np.random.default_rng(2)
    old = [rng.integers(0, 256, size=pk.fp4_cache_shape(9, Hkv, BS, D), dtype=np.uint8)
           for _ in range(2)]
    kc, vc = (torch.from_numpy(c).cuda() for c in old)
    pairs = np.array([[0, 5], [3, 8], [0, 1]], np.int32)
    pk.pa_copy_blocks_fp4(kc, vc, torch.from_numpy(pairs).cuda())
    torch.cuda.synchronize()
    for got, o in zip((kc, vc), old):
        want = o.copy()
        want[pairs[:, 1]] = o[pairs[:, 0]]
        assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.gpu
def test_bad_device_values_set_bits(pk):
    import torch

    c = Case([20, 40], 8, 2, seed=3)
    args, sc = c.cuda()
    rows = torch.ones(2, 2, 128, dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([c.NB * 16, -5], device="cuda")
    before = args[1].clone()
    pk.pa_reshape_and_cache_fp4(rows, rows, args[1], args[2], slots, sc["k_scale"], sc["v_scale"])
    assert pk.pa_device_errors() == pk.DEVERR_SLOT
    assert torch.equal(args[1], before)
    out = pk.pa_gather_fp4(args[1], args[2], slots, sc["k_scale"], sc["v_scale"], rows, rows.clone())
    assert pk.pa_device_errors() == pk.DEVERR_SLOT
    assert not out[0].any()
    bad = list(args)
    bad[3] = args[3].clone()
    bad[3][1, 0] = c.NB
    pk.pa_decode(*bad, **sc)
    assert pk.pa_device_errors() == pk.DEVERR_TABLE_ENTRY
    bad = list(args)
    bad[4] = torch.tensor([20, 49], dtype=torch.int32, device="cuda")
    pk.pa_decode(*bad, **sc)
    assert pk.pa_device_errors() == pk.DEVERR_CONTEXT_LEN


# ------------------------------------------------------------------ GPU: decode

EDGE = [1, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257]


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D,BS", [
    (8, 8, 128, 16), (4, 2, 64, 8), (8, 2, 128, 8), (16, 2, 128, 32), (8, 1, 64, 16),
    (6, 3, 128, 16), (1, 1, 64, 32)])
def test_decode_edge_lengths(pk, Hq, Hkv, D, BS):
    c = Case(EDGE, Hq, Hkv, D, BS, seed=Hq + D + BS)
    args, sc = c.cuda()
    _check(pk, pk.pa_decode(*args, **sc), c)
    args, sc = c.cuda_cut()
    _check(pk, pk.pa_decode(*args, **sc), c)


@pytest.mark.gpu
@pytest.mark.parametrize("Q,Hq,Hkv,D,BS", [
    (2, 8, 2, 128, 16), (3, 4, 4, 64, 8), (5, 8, 1, 128, 32), (4, 16, 2, 64, 16), (17, 2, 2, 128, 16),
    (33, 4, 1, 128, 8)])
def test_decode_several_new_tokens(pk, Q, Hq, Hkv, D, BS):
    lens = [Q, Q + 1, Q + 14, Q + 15, Q + 16, Q + 31, Q + 97, 200]
    c = Case(lens, Hq, Hkv, D, BS, Q=Q, seed=Q)
    args, sc = c.cuda()
    _check(pk, pk.pa_decode(*args, **sc), c)
    args, sc = c.cuda_cut()
    _check(pk, pk.pa_decode(*args, **sc), c)


@pytest.mark.gpu
@pytest.mark.parametrize("B", [1, 300])
def test_decode_many_and_few_sequences(pk, B):
    """One long sequence over every CTA, and more sequences than threads of a CTA."""
    rng = np.random.default_rng(B)
    lens = [3001] if B == 1 else rng.integers(1, 60, B)
    c = Case(lens, 4, 1, 64, 16, seed=B)
    args, sc = c.cuda()
    _check(pk, pk.pa_decode(*args, **sc), c)
    args, sc = c.cuda_cut()
    _check(pk, pk.pa_decode(*args, **sc), c)


@pytest.mark.gpu
def test_decode_long_and_ragged(pk):
    c = Case([5000, 1, 2049, 700, 4097], 8, 2, seed=11)
    args, sc = c.cuda()
    _check(pk, pk.pa_decode(*args, **sc), c)
    _check(pk, pk.pa_decode(*args, scale=0.3, **sc), c, 0.3)


@pytest.mark.gpu
def test_decode_extreme_queries(pk):
    """Queries far from one, and one row of zeros: the power-of-two scaling is exact."""
    import torch

    c = Case([33, 65, 90], 4, 2, 64, seed=5)
    c.q[0] *= 2.0 ** 60
    c.q[1] *= 2.0 ** -60
    c.q[2, 0, 1] = 0
    args, sc = c.cuda()
    # the scale undoes the factor, so that the scores are ordinary
    for b, s in ((0, 2.0 ** -63), (1, 2.0 ** 57), (2, 0.125)):
        one = [args[0][b:b + 1].contiguous(), args[1], args[2], args[3][b:b + 1].contiguous(),
               args[4][b:b + 1].contiguous(), args[5]]
        got = oracle.bf16_to_f64(pk.pa_decode(*one, scale=s, **sc).cpu())
        want, mag = c.want(s)
        assert (np.abs(got[0] - want[b, 0]) <= _bound(want[b, 0], mag[b, 0])).all(), b
    assert pk.pa_device_errors() == 0
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_decode_empty_and_short_sequences(pk):
    import torch

    c = Case([40, 3, 17], 4, 2, Q=4, seed=6)
    args, sc = c.cuda()
    lens = torch.tensor([0, 3, 17], dtype=torch.int32, device="cuda")
    want, mag = c.want()
    for a, mx in ((args, 40), (c.cuda_cut()[0], 4096)):
        out = pk.pa_decode(*a[:4], lens, mx, **sc)
        assert pk.pa_device_errors() == pk.DEVERR_CONTEXT_LEN  # 3 keys cannot hold 4 new tokens
        assert not out[:2].any()
        got = oracle.bf16_to_f64(out[2].cpu())
        assert (np.abs(got - want[2]) <= _bound(want[2], mag[2])).all()
    none = torch.zeros(3, dtype=torch.int32, device="cuda")  # nothing cached at all
    assert not pk.pa_decode(*c.cuda_cut()[0][:4], none, 4096, **sc).any()
    assert pk.pa_device_errors() == 0


@pytest.mark.gpu
def test_decode_nan_rows_stay_with_those_who_see_them(pk):
    """A NaN in the K or V of a new token reaches that token and later ones only,
    and a NaN V group only its 16 elements."""
    import torch

    Q, L, BS, D = 5, 53, 16, 128
    for which in (0, 1):
        c = Case([L], 4, 2, D, BS, Q=Q, seed=8)
        cache = (c.k, c.v)[which]
        clean = c.want()
        pos = L - Q + 2  # new token 2
        blk, off = int(c.tables[0, pos // BS]), pos % BS
        cache.reshape(c.NB, 2, -1)[blk, 1, BS * D // 2 + off * D // 16 + 3] = 0x7F
        args, sc = c.cuda()
        for a in (args, c.cuda_cut()[0]):
            got = oracle.bf16_to_f64(pk.pa_decode(*a, **sc).cpu())
            nan = np.isnan(got)
            want = np.zeros_like(nan)
            if which == 0:
                want[0, 2:, 2:] = True          # K: the whole rows of KV head 1
            else:
                want[0, 2:, 2:, 48:64] = True   # V: group 3
            assert np.array_equal(nan, want), which
            ok = ~want
            assert (np.abs(got - clean[0])[ok] <= _bound(*clean)[ok]).all()
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_decode_bits_do_not_depend_on_placement_or_variant(pk):
    import torch

    c = Case([300, 47, 1290], 8, 2, seed=12)
    args, sc = c.cuda()
    base = pk.pa_decode(*args, **sc)
    assert torch.equal(base, pk.pa_decode(*args, variant=1, **sc))
    assert torch.equal(base, pk.pa_decode(*args, partition_tokens=128, **sc))
    perm = torch.from_numpy(np.random.default_rng(4).permutation(c.NB)).cuda()
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(c.NB, device="cuda")
    tab = torch.where(args[3] >= 0, inv[args[3].clamp(min=0).long()].int(), args[3])
    moved = pk.pa_decode(args[0], args[1][perm].contiguous(), args[2][perm].contiguous(), tab,
                         args[4], args[5], **sc)
    assert torch.equal(base, moved)


@pytest.mark.gpu
def test_decode_length_one_returns_v0(pk):
    import torch

    c = Case([1, 1], 8, 2, seed=13)
    args, sc = c.cuda()
    out = pk.pa_decode(*args, **sc)
    slots = args[3][:, 0].long() * 16
    _, v = pk.pa_gather_fp4(args[1], args[2], slots, **sc)
    assert torch.equal(out, v.repeat_interleave(4, dim=1))


@pytest.mark.gpu
def test_step_calls_agree(pk):
    """pa_append_decode, pa_decode_noalloc and pa_step_host give the bits of the
    write followed by pa_decode; a wrong slot is flagged and not written."""
    import torch

    for Q in (1, 3):
        c = Case([40, 17, 65], 8, 2, Q=Q, seed=20 + Q)
        args, sc = c.cuda()
        B = 3
        kn, vn = (workloads.bf16_normal((B * Q, 2, 128), 30 + i).cuda() for i in range(2))
        pos = np.array([[L - Q + i for i in range(Q)] for L in c.lens])
        slots = np.take_along_axis(c.tables, pos // 16, 1).astype(np.int64) * 16 + pos % 16
        slots = torch.from_numpy(slots.reshape(-1)).cuda()
        pair = torch.tensor([[int(c.tables[0, 0]), c.NB - 1]], dtype=torch.int32, device="cuda")
        free = set(range(c.NB)) - set(c.tables.reshape(-1).tolist())
        pair[0, 1] = min(free)

        k1, v1 = args[1].clone(), args[2].clone()
        pk.pa_copy_blocks_fp4(k1, v1, pair)
        pk.pa_reshape_and_cache_fp4(kn, vn, k1, v1, slots, **sc)
        want = pk.pa_decode(args[0], k1, v1, *args[3:], **sc)

        k2, v2 = args[1].clone(), args[2].clone()
        pk.pa_copy_blocks_fp4(k2, v2, pair)
        got = pk.pa_append_decode(args[0], k2, v2, *args[3:], kn, vn, slots, **sc)
        assert torch.equal(got, want) and torch.equal(k1, k2) and torch.equal(v1, v2)
        assert torch.equal(pk.pa_decode_noalloc(args[0], k2, v2, *args[3:], **sc), want)

        for pin in (True, False):
            k3, v3 = args[1].clone(), args[2].clone()
            p = pk.make_step_host_params(k3, v3, B, 8, args[3].shape[1], args[5], 1, query_len=Q,
                                         **sc)
            host = pk.pack_step_inputs(p, args[0], kn, vn, slots, args[3], args[4], pair, pin=pin)
            out = torch.empty(args[0].shape, dtype=torch.bfloat16, pin_memory=pin)
            ws = torch.empty(pk.pa_step_host_workspace_size(p), dtype=torch.uint8, device="cuda")
            pk.pa_step_host(p, host, out, ws)
            assert torch.equal(out, want.cpu()) and torch.equal(k3, k1) and torch.equal(v3, v1)
        assert pk.pa_device_errors() == 0

        wrong = slots.clone()
        wrong[0] += 1 if int(wrong[0]) % 16 < 15 else -1
        k4, v4 = args[1].clone(), args[2].clone()
        pk.pa_append_decode(args[0], k4, v4, *args[3:], kn, vn, wrong, **sc)
        assert pk.pa_device_errors() == pk.DEVERR_APPEND_SLOT


@pytest.mark.gpu
def test_decode_on_a_stream_and_in_a_graph(pk):
    """Another stream than the current one, and a captured step replayed on new inputs."""
    import torch

    c = Case([300, 47], 8, 2, seed=14)
    args, sc = c.cuda()
    want = pk.pa_decode(*args, **sc)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    p = pk.make_decode_params(args[0], torch.empty_like(args[0]), *args[1:], **sc)
    ws = torch.empty(pk.pa_decode_workspace_size(p), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(args[0])
    torch.cuda.synchronize()
    pk.pa_decode(*args, out=out, workspace=ws, stream=side, **sc)
    side.synchronize()
    assert torch.equal(out, want)
    q = args[0].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pk.pa_decode(q, *args[1:], out=out, workspace=ws, **sc)
    q.copy_(args[0].flip(0))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, pk.pa_decode(q, *args[1:], **sc))


@pytest.mark.gpu
def test_decode_negative_and_zero_scales(pk):
    """A head scale is a factor like any other: its sign turns the scores, zero makes them equal."""
    c = Case([300, 47, 17], 8, 4, seed=16)
    c.ks *= np.array([1, -1, 0, -40], np.float32)
    c.vs *= np.array([-1, 1, 0, 1], np.float32)
    args, sc = c.cuda()
    _check(pk, pk.pa_decode(*args, **sc), c)
    args, sc = c.cuda_cut()
    _check(pk, pk.pa_decode(*args, **sc), c)


@pytest.mark.gpu
def test_tensors_of_another_device_are_refused(pk, monkeypatch):
    c = Case([40], 8, 2, seed=20)
    args, sc = c.cuda()
    pk.pa_decode(*args, **sc)
    monkeypatch.setattr(pk, "_device", lambda: 1)  # as under torch.cuda.device(1)
    with pytest.raises(ValueError, match="current CUDA device"):
        pk.pa_decode(*args, **sc)


@pytest.mark.gpu
def test_decode_nan_keys_of_a_whole_piece(pk):
    """NaN scales in all of a long run of K rows: their head's outputs are NaN, however the
    run falls to the CTAs, and the others' are not."""
    import torch

    c = Case([6000, 6000], 8, 2, seed=21)
    args, sc = c.cuda()
    k = args[1].view(c.NB, 2, -1)
    k[args[3][0, :300].long(), 1, 16 * 64:] = 0x7F      # keys 0 to 4799 of sequence 0, KV head 1
    out = pk.pa_decode(*args, **sc).float()
    assert out[0, 4:].isnan().all()
    assert out[0, :4].isfinite().all() and out[1].isfinite().all()


@pytest.mark.gpu
def test_two_calls_at_once(pk):
    """Two batches on two streams, each with its workspace."""
    import torch

    cases = [Case([3000, 700, 40], 8, 2, seed=17), Case([2500, 1, 1200, 90], 8, 2, seed=18)]
    calls = [c.cuda() for c in cases]
    want = [pk.pa_decode(*a, **sc) for a, sc in calls]
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [torch.empty_like(w) for w in want]
    spaces = [torch.empty(8 << 20, dtype=torch.uint8, device="cuda") for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for (a, sc), s, o, ws in zip(calls, streams, outs, spaces):
            pk.pa_decode(*a, out=o, workspace=ws, stream=s, **sc)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


@pytest.mark.gpu
def test_offsets_beyond_32_bits(pk):
    """A cache of more than 2^32 bytes: rows in its last blocks decode, copy, read back and
    weigh as the same rows in a small one."""
    import torch

    c = Case([200, 77], 8, 2, seed=19)
    args, sc = c.cuda()
    shift = (1 << 32) // (2 * _tile(16, 128)) + 1000     # blocks before the small cache's copy
    big = [torch.zeros(pk.fp4_cache_shape(shift + c.NB, 2, 16, 128), dtype=torch.uint8,
                       device="cuda") for _ in range(2)]
    for b, small in zip(big, args[1:3]):
        b[shift:] = small
    tab = torch.where(args[3] >= 0, args[3] + shift, args[3])
    far = (args[0], big[0], big[1], tab, *args[4:])
    assert torch.equal(pk.pa_decode(*far, **sc), pk.pa_decode(*args, **sc))
    w = [torch.zeros(2, 200, device="cuda") for _ in range(2)]
    for a, x in ((far, w[0]), (args, w[1])):
        pk.pa_token_weights(a[0], a[1], a[3], a[4], 200, x, k_scale=sc["k_scale"])
    assert torch.equal(*w)
    slots = torch.arange(c.NB * 16, device="cuda")
    for x, y in zip(pk.pa_gather_fp4(*big, slots + shift * 16, **sc),
                    pk.pa_gather_fp4(args[1], args[2], slots, **sc)):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))
    keep, n = pk.pa_evict_select(w[0], args[4], 50, 3)
    for a in (far, args):
        pk.pa_evict_compact(a[1], a[2], a[3], a[3], keep, n)
    pair = torch.tensor([[int(args[3][0, 0]), c.NB - 1]], dtype=torch.int32, device="cuda")
    pk.pa_copy_blocks_fp4(big[0], big[1], pair + shift)
    pk.pa_copy_blocks_fp4(args[1], args[2], pair)
    for b, small in zip(big, args[1:3]):
        assert torch.equal(b[shift:], small) and not b[:64].any()
    assert pk.pa_device_errors() == 0


@pytest.mark.gpu
def test_empty_batch(pk):
    import torch

    c = Case([16], 8, 2, seed=15)
    args, sc = c.cuda()
    out = pk.pa_decode(args[0][:0], args[1], args[2], args[3][:0], args[4][:0], 16, **sc)
    assert out.shape[0] == 0
    e = torch.empty(0, 2, 128, dtype=torch.bfloat16, device="cuda")
    pk.pa_reshape_and_cache_fp4(e, e, args[1], args[2],
                                torch.empty(0, dtype=torch.int64, device="cuda"), **sc)
    assert pk.pa_device_errors() == 0


# ------------------------------------------------------------------ GPU: the softmax weights' range
#
# Weights are held in f16 with the largest that a reference was taken from at 2^7 (and at most
# 2^15): those down to 2^-14 are rounded by at most 2^-11 of their value, lesser ones by at most
# half the subnormal step, 2^-25, which is 2^-32 of the row's largest weight. So beside the terms of
# `_bound` an element is off by at most 2^-32 L max|V|.


def _ones_case(pk, keys, values):
    """One sequence, one KV head, d 64, block 16, head scales and group scales of one: K codes
    `keys` [L][64], V codes `values` [L][64] (E2M1, the sign in bit 3)."""
    import torch

    L, D, BS = len(keys), 64, 16
    nb = -(-L // BS)
    caches = []
    for codes in (keys, values):
        full = np.zeros((nb * BS, D), np.uint8)
        full[:L] = codes
        flat = np.full((nb, 1, BS * D * 9 // 16), 0x38, np.uint8)
        flat[:, 0, :BS * D // 2] = (full[:, 0::2] | full[:, 1::2] << 4).reshape(nb, -1)
        caches.append(flat.reshape(nb, 1, BS, D * 9 // 16))
    tab = np.random.default_rng(L).permutation(nb).astype(np.int32)[None]
    for c in caches:
        c[tab[0]] = c.copy()
    return caches, tab


def _check_weights_range(pk, caches, tab, L, q, scale):
    import torch

    one = np.ones(1, np.float32)
    kr, vr = (oracle.fp4_values(c, one, 64) for c in caches)
    qd = oracle.bf16_to_f64(q)
    lens = np.array([L], np.int32)
    want, _ = oracle.attention_rows(qd, kr, vr, tab, lens, scale)
    mag, _ = oracle.attention_rows(qd, kr, np.abs(vr), tab, lens, scale)
    bound = _bound(want, mag) + 2.0 ** -32 * L * np.abs(vr).max()
    s = torch.ones(1, device="cuda")
    dev = [torch.from_numpy(c).cuda() for c in caches]
    for room in (tab.shape[1], 256):  # as it is, and with room for 4,096 tokens (the stream)
        wide = np.full((1, max(room, tab.shape[1])), -1, np.int32)
        wide[:, :tab.shape[1]] = tab
        got = pk.pa_decode(q[:, 0].cuda(), *dev, torch.from_numpy(wide).cuda(),
                           torch.from_numpy(lens).cuda(), max(L, room * 16), scale,
                           k_scale=s, v_scale=s)
        got = oracle.bf16_to_f64(got.cpu())[:, None]
        assert np.isfinite(got).all()
        over = np.abs(got - want) / bound
        assert over.max() <= 1.0, (room, over.max())
    assert pk.pa_device_errors() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("gap", [12.0, 20.0, 24.5, 25.5, 27.0, 30.0])
@pytest.mark.parametrize("L", [300, 1000, 2000])
def test_decode_flat_tail_behind_large_weights(pk, gap, L):
    """A few keys whose weights are 2^gap times those of all others, with values of zero, so
    that the output is the tail's alone. One of them in each warp's first step."""
    import torch

    rng = np.random.default_rng(L)
    keys = np.zeros((L, 64), np.uint8)
    values = rng.integers(0, 8, (L, 64)).astype(np.uint8)
    keys[[0, 32, 64, 96]] = 2          # elements of one: a product of 64
    values[[0, 32, 64, 96]] = 0
    caches, tab = _ones_case(pk, keys, values)
    q = torch.ones(1, 1, 2, 64, dtype=torch.bfloat16)
    q[:, :, 1] = 0.5                   # the second head's gap is half as wide
    scale = float(np.float32(gap * np.log(2.0) / 64))
    _check_weights_range(pk, caches, tab, L, q, scale)


@pytest.mark.gpu
@pytest.mark.parametrize("big", [2.0 ** -2, 2.0 ** 6, 2.0 ** 8])
def test_decode_scores_of_millions(pk, big):
    """Scores far beyond the softmax's range that differ by a few units, rising from step to
    step of a warp by just under and just over what moves the reference. All products are exact
    (21 bits), and so are the scores' differences up to the scale's last places."""
    import torch

    L = 1000
    keys = np.zeros((L, 64), np.uint8)
    keys[:, 0] = 7                                            # 6 * big
    keys[:, 1] = np.minimum(np.arange(L) // 128, 7)           # 0 to 6, times big * 2^-17
    values = np.random.default_rng(1).integers(0, 16, (L, 64)).astype(np.uint8)
    caches, tab = _ones_case(pk, keys, values)
    q = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16)
    q[..., 0], q[..., 1] = big, big * 2.0 ** -17
    for unit in np.linspace(2.4, 3.3, 19):  # of half a code in the log2 domain; 3 units are a jump
        scale = float(np.float32(unit * np.log(2.0) / (big * 2.0 ** -18)))
        _check_weights_range(pk, caches, tab, L, q, scale)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D,BS,Q,lens", [(8, 2, 128, 16, 130, [130, 131, 200, 333]),
                                                (8, 1, 64, 32, 65, [65, 66, 96, 97, 700]),
                                                (1, 1, 64, 16, 1024, [1024, 1100])])
def test_decode_prompt_chunks(pk, Hq, Hkv, D, BS, Q, lens):
    """Chunks of many new tokens: groups of columns in their dozens, up to the longest chunk."""
    c = Case(lens, Hq, Hkv, D, BS, Q=Q, seed=Q)
    args, sc = c.cuda()
    _check(pk, pk.pa_decode(*args, **sc), c)
    args, sc = c.cuda_cut()
    _check(pk, pk.pa_decode(*args, **sc), c)


@pytest.mark.gpu
@pytest.mark.parametrize("power", [20, 27, 28, 29, 31, 34, 40, 60])
@pytest.mark.parametrize("low,high", [(6, 7), (15, 14)])  # codes: 4 and 6, or -6 and -4
def test_decode_scores_of_any_size(pk, power, low, high):
    """Scores of 2^power in the log2 domain, where a unit is far below their last place: the
    largest share the weight and the others get none, as in exact arithmetic."""
    import torch

    L = 500
    rng = np.random.default_rng(power)
    keys = np.zeros((L, 64), np.uint8)
    keys[:, 0] = low
    keys[[70, 71, 300, 467], 0] = high
    values = rng.integers(0, 16, (L, 64)).astype(np.uint8)
    caches, tab = _ones_case(pk, keys, values)
    q = torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16)
    q[..., 0] = 1.0
    for m in rng.uniform(1, 2, 12):
        _check_weights_range(pk, caches, tab, L, q, float(np.float32(m * 2.0 ** power / 6)))
