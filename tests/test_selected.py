"""Attention over selected blocks: bounds, scores, the choice and the decode, against
plain numpy in 64 bits.

Bounds and the choice are exact. A score is a sum of 2 d exact products in fp32: with A the
sum of their magnitudes times the factor, the matrix unit's d / 8 accumulations each round
by at most 2^-22 of a running value within A, the factor and its product by 3 * 2^-24: less
than (d / 8 + 1) 2^-22 A, at most 2^-17 A.

An output is sum w_t v_t with w = p / sum p. With A the largest scale * log2(e) * sum |q k| of
a row, a score in the log2 domain is off by at most 2^-18 A (d / 16 accumulations and three
roundings), its exponential by that times ln 2 and 2^-22, a weight in the product by E more
(2^-17 in two bf16 terms, 2^-11 in f16); numerator and denominator take n / 16
accumulations of 2^-22. In f16 a weight is off by up to 2^-32 of the row's largest besides
(f16 ends at 2^-24, the largest is held at 2^7 or above, and a rounding there takes half of
2^-24): as the largest is at most the sum, that is 2^-32 V in the output, V = sum |v|. In
fp32 weights below 2^-126 of the largest are lost: 2^-120 V. With W = sum w |v| an output is
within W (2^-16 A + E + 2^-19 + n 2^-25) + (2^-32 or 2^-120) V + 2^-8 |out| of its value, the
last for bf16.
"""
import ctypes
import math

import numpy as np
import pytest

import oracle
import workloads

FMTS = ["bf16", "fp8", "fp4"]


@pytest.fixture(scope="module")
def pk():
    from paged_kv_cache_92_gb300 import build

    build.build()
    import paged_kv_cache_92_gb300 as pk

    pk.load()
    return pk


# ------------------------------------------------------------------ plain forms


class Cache:
    """One K and one V cache on the host: their bytes, and their values [NB][Hkv][BS][D]
    (K also with the head's scale left out)."""

    def __init__(self, fmt, NB, Hkv, BS, D, seed, poison=()):
        import torch

        rng = np.random.default_rng(seed)
        self.fmt, self.BS, self.D = fmt, BS, D
        self.ks = self.vs = None
        if fmt == "bf16":
            raw = [rng.standard_normal((NB, Hkv, BS, D)).astype(np.float32) for _ in range(2)]
            for b, o in poison:
                raw[0][b, :, o] = raw[1][b, :, o] = np.nan
            self.k, self.v = (torch.from_numpy(x).to(torch.bfloat16) for x in raw)
            self.k_values, self.v_values = (x.double().numpy() for x in (self.k, self.v))
            self.k_codes = self.k_values
            return
        self.ks = (0.05 * np.exp(rng.uniform(-0.5, 0.5, Hkv))).astype(np.float32)
        self.vs = (0.03 * np.exp(rng.uniform(-0.5, 0.5, Hkv))).astype(np.float32)
        if Hkv > 1:
            self.ks[1] *= -1.0  # scales of either sign
        if fmt == "fp8":
            k, v = (rng.integers(0, 256, (NB, Hkv, BS, D), dtype=np.uint8) for _ in range(2))
            for c in (k, v):
                c[(c & 0x7F) >= 0x60] &= 0x9F  # up to 30: neither NaN nor all of the weight
            for b, o in poison:
                k[b, :, o] = v[b, :, o] = 0x7F
            W = min(BS, 16)
            self.k, self.v = torch.from_numpy(k), torch.from_numpy(
                np.ascontiguousarray(v.reshape(NB, Hkv, BS // W, W, D).swapaxes(-1, -2)))
            self.k_codes, v_codes = oracle.e4m3_to_f64(k), oracle.e4m3_to_f64(v)
        else:
            def tiles(s):
                x = rng.integers(0, 256, (NB, Hkv, BS, D * 9 // 16), dtype=np.uint8)
                f = x.reshape(NB, Hkv, -1)[..., BS * D // 2:].reshape(NB, Hkv, BS, D // 16)
                f[:] = rng.integers(0x28, 0x48, f.shape)  # group scales of 0.25 to 4
                for b, o in poison:
                    f[b, :, o] = 0x7F
                return x
            k, v = tiles(self.ks), tiles(self.vs)
            self.k, self.v = torch.from_numpy(k), torch.from_numpy(v)
            one = np.ones(Hkv, np.float32)
            self.k_codes, v_codes = oracle.fp4_values(k, one, D), oracle.fp4_values(v, one, D)
        s = lambda a: a.astype(np.float64)[:, None, None]  # noqa: E731
        self.k_values, self.v_values = self.k_codes * s(self.ks), v_codes * s(self.vs)

    def scales(self, device="cuda"):
        import torch

        if self.ks is None:
            return dict(k_scale=None, v_scale=None)
        return dict(k_scale=torch.from_numpy(self.ks).to(device),
                    v_scale=torch.from_numpy(self.vs).to(device))


def plain_bounds(cache, bounds, tables, old, lens):
    """`bounds` (float64) with the touched blocks' least and largest codes."""
    out = bounds.copy()
    for b, n in enumerate(lens):
        for j in range(old[b] // cache.BS, -(-n // cache.BS)):
            x = cache.k_codes[tables[b, j], :, : max(0, min(cache.BS, n - j * cache.BS))]
            bad = np.isnan(x).any(1)
            lo, hi = x.min(1), x.max(1)
            lo[bad] = hi[bad] = np.nan
            out[tables[b, j], :, 0], out[tables[b, j], :, 1] = lo, hi
    return out


def plain_scores(q, bounds, ks, tables, lens, BS, scale):
    """[B][Hkv][blocks] scores and, for the tolerance, the sums of magnitudes. q [B][Q][Hq][D]."""
    B, Q, Hq, D = q.shape
    Hkv = bounds.shape[1]
    out, mag = {}, {}
    for b, n in enumerate(lens):
        if n < Q:
            continue
        for g in range(Hkv):
            f = np.float64(np.float32(scale)) * (1.0 if ks is None else np.float64(ks[g]))
            rows = q[b, :, g * (Hq // Hkv):(g + 1) * (Hq // Hkv)] * f
            for j in range(-(-n // BS)):
                lo, hi = bounds[tables[b, j], g]
                first = max(0, j * BS - (n - Q))  # the first new token that sees the block
                with np.errstate(invalid="ignore"):
                    s = np.maximum(rows[first:], 0) * hi + np.minimum(rows[first:], 0) * lo
                    t = s.sum(-1)
                t[np.isnan(t)] = np.inf
                out[b, g, j] = t.max()
                mag[b, g, j] = np.abs(s).sum(-1).max()
    return out, mag


def plain_select(scores, lens, BS, budget, sink, recent):
    B, H, stride = scores.shape
    out = np.full((B, H, budget), -1, np.int32)
    for b, L in enumerate(lens):
        n = min(-(-max(L, 0) // BS), stride)
        for h in range(H):
            got = list(range(n))
            if n > budget:
                w = [(np.isnan(x), 0.0 if np.isnan(x) else -x) for x in scores[b, h, :n].tolist()]
                mid = sorted(range(sink, n - recent), key=lambda j: (*w[j], j))
                got = sorted(list(range(sink)) + list(range(n - recent, n))
                             + mid[:budget - sink - recent])
            out[b, h, :len(got)] = got
    return out


def plain_attend(cache, q, tables, lens, selected, scale):
    """out [B][Q][Hq][D], and W, A and V of the tolerance."""
    B, Q, Hq, D = q.shape
    Hkv, BS = cache.k_values.shape[1], cache.BS
    out, W, V = np.zeros_like(q), np.zeros_like(q), np.zeros_like(q)
    A = np.zeros(q.shape[:3] + (1,))
    G = Hq // Hkv
    for b, n in enumerate(lens):
        nblk = -(-n // BS)
        for g in range(Hkv):
            listed = [int(j) for j in selected[b, g, :max(nblk, 0)] if 0 <= j < nblk]
            t = np.array([j * BS + o for j in listed for o in range(BS)], np.int64)
            if n < Q or not len(t):
                continue
            blk = tables[b, t // BS]
            k, v = cache.k_values[blk, g, t % BS], cache.v_values[blk, g, t % BS]
            for i in range(Q):
                on = t <= n - Q + i
                if not on.any():
                    continue
                for h in range(g * G, (g + 1) * G):
                    s = k[on] @ q[b, i, h] * scale
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    out[b, i, h], W[b, i, h] = p @ v[on], p @ np.abs(v[on])
                    V[b, i, h] = np.abs(v[on]).sum(0)
                    A[b, i, h] = (np.abs(k[on]) @ np.abs(q[b, i, h])).max() * scale * 1.4427
    return out, W, A, V


def close(got, want, W, A, V, fmt, n):
    E, least = (2.0 ** -17, 2.0 ** -120) if fmt == "bf16" else (2.0 ** -11, 2.0 ** -32)
    tol = W * (2.0 ** -16 * A + E + 2.0 ** -19 + n * 2.0 ** -25) + least * V \
        + 2.0 ** -8 * np.abs(want)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    bad = np.abs(got - want) > tol * (1 + 2.0 ** -8)
    assert not (bad & ~np.isnan(want)).any(), np.nanmax(np.abs(got - want) / (tol + 1e-300))


def layout(lens, BS, seed, extra=3, width=1):
    blocks = [-(-max(n, 0) // BS) for n in lens]
    order = np.random.default_rng(seed).permutation(sum(blocks) + extra).astype(np.int32)
    tables = np.full((len(lens), max(blocks + [1]) + width), -1, np.int32)
    at = 0
    for b, k in enumerate(blocks):
        tables[b, :k] = order[at:at + k]
        at += k
    poison = [(int(tables[b, n // BS]), o) for b, n in enumerate(lens) if n > 0 and n % BS
              for o in range(n % BS, BS)]  # rows behind the sequences hold NaN
    return tables, len(order), poison


def dev(x):
    import torch

    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


# ------------------------------------------------------------------ refusals (CPU)


def _fill(p, base, kw):
    for k, v in {**base, **kw}.items():
        setattr(p, k, v)
    return p


BOUNDS = dict(k_cache=256, bounds=256, block_tables=256, context_lens=256, max_blocks_per_seq=4,
              num_seqs=2, num_kv_heads=2, head_dim=128, block_size=16, num_blocks=8,
              max_new_tokens=1)


@pytest.mark.parametrize("kw,status", [
    (dict(num_seqs=-1), 1), (dict(num_seqs=65536), 1), (dict(num_kv_heads=0), 1),
    (dict(num_kv_heads=65536), 1), (dict(num_blocks=0), 1), (dict(max_blocks_per_seq=0), 1),
    (dict(max_new_tokens=0), 1), (dict(block_size=12), 2), (dict(head_dim=96), 2),
    (dict(kv_dtype=3), 1), (dict(max_blocks_per_seq=1 << 27), 1), (dict(k_cache=None), 1),
    (dict(bounds=None), 1), (dict(block_tables=None), 1), (dict(context_lens=None), 1),
    (dict(k_cache=264), 1), (dict(bounds=264), 1), (dict(old_lens=2), 1),
    (dict(num_seqs=0, bounds=None), 0)])
def test_bounds_refusals(pk, kw, status):
    p = _fill(pk.BlockBoundsParams(), BOUNDS, kw)
    assert pk.load().pa_block_bounds(ctypes.byref(p), None) == status
    assert pk.load().pa_block_bounds(None, None) == 1


SCORES = dict(q=256, bounds=256, block_tables=256, context_lens=256, scores=256, scores_stride=4,
              max_blocks_per_seq=4, num_seqs=2, num_q_heads=8, num_kv_heads=2, head_dim=128,
              block_size=16, num_blocks=8, max_context_len=64, scale=0.088)


@pytest.mark.parametrize("kw,status", [
    (dict(num_seqs=65536), 1), (dict(num_q_heads=7), 1), (dict(num_q_heads=6), 2),
    (dict(num_q_heads=32), 2), (dict(num_kv_heads=0), 1), (dict(head_dim=80), 2),
    (dict(block_size=64), 2), (dict(query_len=-1), 1), (dict(query_len=1025), 1),
    (dict(scale=0.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(scores_stride=3), 1), (dict(max_context_len=0), 1), (dict(num_blocks=0), 1),
    (dict(max_blocks_per_seq=1 << 27, scores_stride=1 << 27), 1), (dict(q=None), 1),
    (dict(scores=None), 1), (dict(q=260), 1), (dict(scores=258), 1), (dict(k_scale=1), 1),
    (dict(num_seqs=0, q=None), 0)])
def test_scores_refusals(pk, kw, status):
    p = _fill(pk.BlockScoresParams(), SCORES, kw)
    assert pk.load().pa_block_scores(ctypes.byref(p), None) == status
    assert pk.load().pa_block_scores(None, None) == 1


@pytest.mark.parametrize("dims,status", [
    ((-1, 2, 8, 16, 4, 1, 1), 1), ((65536, 2, 8, 16, 4, 1, 1), 1), ((2, 0, 8, 16, 4, 1, 1), 1),
    ((2, 2, 0, 16, 4, 1, 1), 1), ((2, 2, 8, 4, 4, 1, 1), 2), ((2, 2, 8, 16, 0, 0, 0), 1),
    ((2, 2, 8, 16, 4, 3, 2), 1), ((2, 2, 8, 16, 4, -1, 2), 1), ((2, 2, 8, 16, 4, 1, -1), 1),
    ((2, 2, 8, 16, 2**31 - 1, 2**31 - 1, 2**31 - 1), 1), ((2, 2, (1 << 30) + 1, 16, 4, 1, 1), 1),
    ((65535, 32769, 8, 16, 4, 1, 1), 1), ((0, 2, 8, 16, 4, 1, 1), 0)])
def test_select_refusals(pk, dims, status):
    lib = pk.load()
    assert lib.pa_block_select(256, 256, 256, *dims, None) == status
    if status == 0:
        assert lib.pa_block_select(None, 256, 256, 2, *dims[1:], None) == 1
        assert lib.pa_block_select(258, 256, 256, 2, *dims[1:], None) == 1


DECODE = dict(q=256, out=256, k_cache=256, v_cache=256, block_tables=256, context_lens=256,
              max_blocks_per_seq=4, num_seqs=2, num_q_heads=8, num_kv_heads=2, head_dim=128,
              block_size=16, num_blocks=8, max_context_len=64, scale=0.088)


@pytest.mark.parametrize("kw,n,status", [
    (dict(), 0, 1), (dict(), -3, 1), (dict(num_seqs=65536), 4, 1), (dict(num_q_heads=12), 4, 2),
    (dict(num_q_heads=9), 4, 1), (dict(head_dim=32), 4, 2), (dict(block_size=4), 4, 2),
    (dict(kv_dtype=5), 4, 1), (dict(kv_dtype=1), 4, 1), (dict(kv_dtype=2, k_scale=4), 4, 1),
    (dict(query_len=1025), 4, 1), (dict(scale=float("inf")), 4, 1), (dict(variant=2), 4, 1),
    (dict(partition_tokens=8), 4, 1), (dict(wait_timeout_us=-1), 4, 1),
    (dict(num_seqs=65535, num_kv_heads=2049, num_q_heads=2049), 4, 2),
    (dict(max_blocks_per_seq=1 << 27), 4, 1), (dict(q=None), 4, 1), (dict(out=264), 4, 1),
    (dict(max_context_len=0), 4, 1), (dict(num_seqs=0, q=None), 4, 0)])
def test_decode_refusals(pk, kw, n, status):
    p = _fill(pk.DecodeParams(), DECODE, kw)
    lib = pk.load()
    assert lib.pa_decode_selected(ctypes.byref(p), 256, n, None, 0, None) == status
    if status == 0:
        p.num_seqs, p.q = 2, 256
        assert lib.pa_decode_selected(ctypes.byref(p), None, n, None, 0, None) == 1
        assert lib.pa_decode_selected(ctypes.byref(p), 258, n, None, 0, None) == 1
    assert lib.pa_decode_selected(None, 256, 4, None, 0, None) == 1


def test_binding_refuses_mixed_shapes(pk):
    import torch

    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    k = torch.zeros(6, 2, 16, 64, dtype=torch.bfloat16)
    bounds = torch.zeros(pk.block_bounds_shape(6, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        pk.pa_block_bounds(k, bounds[:5], i(2, 3), i(2), 1)
    with pytest.raises(ValueError):
        pk.pa_block_bounds(k, bounds, i(2, 3), i(3), 1)
    with pytest.raises(ValueError):
        pk.pa_block_bounds(k, bounds, i(2, 3), i(2), 1, old_lens=i(1))
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    for bad in (dict(q=q[..., :32]), dict(context_lens=i(1)), dict(block_tables=i(3, 3)),
                dict(scores=torch.zeros(2, 3, 3)), dict(k_scale=torch.ones(3))):
        with pytest.raises(ValueError):
            pk.pa_block_scores(**{**dict(q=q, bounds=bounds, block_tables=i(2, 3),
                                         context_lens=i(2), max_context_len=48, block_size=16),
                                  **bad})
    with pytest.raises(ValueError):
        pk.pa_block_select(torch.zeros(2, 2, 3), i(3), 16, 2)
    with pytest.raises(ValueError):
        pk.pa_block_select(torch.zeros(2, 2, 3), i(2), 16, 2, selected=i(2, 2, 3))
    for bad in (i(2, 1, 2), i(1, 2, 2), i(2, 2)):
        with pytest.raises(ValueError):
            pk.pa_decode_selected(q, k, k, i(2, 3), i(2), 48, bad)
    with pytest.raises(ValueError):  # a host tensor
        pk.pa_decode_selected(q, k, k, i(2, 3), i(2), 48, i(2, 2, 2))


def test_plain_attention_over_all_blocks_is_the_decode():
    c = Cache("bf16", 8, 2, 16, 64, 1)
    tables, lens = np.array([[3, 1, 5], [0, 7, -1]], np.int32), [40, 17]
    q = workloads.bf16_normal((2, 4, 64), 5)
    want = oracle.paged_decode_numpy(q, oracle.bf16_bits(c.k), oracle.bf16_bits(c.v), tables,
                                     np.array(lens, np.int32))
    sel = np.tile(np.array([2, 0, 1], np.int32), (2, 2, 1))
    sel[1] = [1, 0, -1]
    got, _, _, _ = plain_attend(c, q.double().numpy()[:, None], tables, lens, sel, 1 / 8)
    assert np.allclose(got[:, 0], want, atol=1e-12)


def test_plain_score_bounds_every_logit():
    c = Cache("fp8", 6, 2, 16, 64, 2)
    tables, lens = np.array([[3, 1, 5]], np.int32), [41]
    q = np.random.default_rng(3).standard_normal((1, 2, 4, 64))
    b = plain_bounds(c, np.zeros((6, 2, 2, 64)), tables, [0], lens)
    got, _ = plain_scores(q, b, c.ks, tables, lens, 16, 0.25)
    for (_, g, j), s in got.items():
        k = c.k_values[tables[0, j], g, : min(16, 41 - 16 * j)]
        assert (k @ q[0, :, 2 * g:2 * g + 2].reshape(-1, 64).T * 0.25).max() <= s + 1e-9


# ------------------------------------------------------------------ GPU: bounds


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,BS,Hkv", [(64, 8, 3), (128, 16, 8), (64, 32, 1), (128, 8, 2),
                                      (64, 16, 5), (128, 32, 2)])
def test_bounds(pk, fmt, D, BS, Hkv):
    import torch

    lens = [0, 1, BS, BS + 1, 7 * BS - 1, 100, 333]
    tables, NB, poison = layout(lens, BS, D + BS)
    c = Cache(fmt, NB, Hkv, BS, D, 7, poison)
    for old, most in (([0] * 7, 333), ([0, 0, BS - 1, BS, 6 * BS, 99, 200], 133),
                      ([0, 1, BS, BS + 1, 7 * BS - 1, 100, 333], 1)):
        start = torch.randn(NB, Hkv, 2, D).bfloat16()
        want = plain_bounds(c, start.double().numpy(), tables, old, lens)
        got = start.cuda()
        args = (c.k.cuda(), got, dev(tables), dev(np.array(lens, np.int32)), most)
        pk.pa_block_bounds(*args, old_lens=dev(np.array(old, np.int32)))
        torch.cuda.synchronize()
        assert np.array_equal(got.double().cpu().numpy(), want)
        assert pk.pa_device_errors() == 0
        if sum(old) == 0:
            again = pk.pa_block_bounds(c.k.cuda(), start.cuda(), *args[2:])
            assert torch.equal(again, got)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FMTS)
def test_bounds_of_nan_infinity_and_extremes(pk, fmt):
    import torch

    c = Cache(fmt, 3, 1, 16, 64, 3, poison=[(1, 4)])
    if fmt == "bf16":
        c.k[2, 0, 3, 5], c.k[2, 0, 9, 5], c.k[2, 0, 1, 6] = math.inf, -math.inf, -0.0
    elif fmt == "fp8":
        c.k[2, 0, 3, 5], c.k[2, 0, 9, 5], c.k[2, 0, :, 6] = 0x7E, 0xFE, 0x01  # +-448, 2^-9
    else:
        c.k.view(3, 1, -1)[2, 0, 16 * 32:] = 0x7E  # scales of 448: up to 2688
    c2 = Cache.__new__(Cache)
    c2.BS = 16
    c2.k_codes = (c.k.double().numpy() if fmt == "bf16" else oracle.e4m3_to_f64(c.k.numpy())
                  if fmt == "fp8" else oracle.fp4_values(c.k.numpy(), np.ones(1, np.float32), 64))
    tables = np.array([[0, 1, 2]], np.int32)
    want = plain_bounds(c2, np.zeros((3, 1, 2, 64)), tables, [0], [48])
    got = torch.zeros(3, 1, 2, 64, dtype=torch.bfloat16, device="cuda")
    pk.pa_block_bounds(c.k.cuda(), got, dev(tables), dev(np.array([48], np.int32)), 48)
    assert np.array_equal(got.double().cpu().numpy(), want, equal_nan=True)
    assert np.isnan(want[1]).all() and not np.isnan(want[2]).any()


@pytest.mark.gpu
def test_bounds_bad_lengths_and_entries(pk):
    import torch

    c = Cache("bf16", 6, 2, 16, 64, 3)
    start = torch.zeros(6, 2, 2, 64, dtype=torch.bfloat16)

    def go(tables, lens, old, most):
        got = start.cuda()
        pk.pa_block_bounds(c.k.cuda(), got, dev(np.array(tables, np.int32)),
                           dev(np.array(lens, np.int32)), most, old_lens=dev(np.array(old, np.int32)))
        return got.double().cpu().numpy(), pk.pa_device_errors()

    def want(tables, lens, old):
        return plain_bounds(c, start.double().numpy(), np.array(tables), old, lens)

    got, err = go([[1, 99, 2], [-5, 3, 0]], [48, 32], [0, 0], 48)
    assert err == pk.DEVERR_TABLE_ENTRY
    ok = want([[1, 1, 2], [3, 3, 0]], [48, 32], [0, 0])
    assert np.array_equal(got, ok)
    got, err = go([[1, 4]], [2**31 - 1], [0], 48)  # past the table row
    assert err == pk.DEVERR_CONTEXT_LEN and np.array_equal(got, want([[1, 4]], [32], [0]))
    # more tokens than announced: the blocks that n can touch are (n + 2 BS - 2) / BS
    got, err = go([[1, 4, 5]], [48], [0], 1)
    assert err == pk.DEVERR_CONTEXT_LEN and np.array_equal(got, want([[1]], [16], [0]))
    got, err = go([[1, 4, 5]], [48], [0], 2)
    assert err == pk.DEVERR_CONTEXT_LEN and np.array_equal(got, want([[1, 4]], [32], [0]))
    got, err = go([[1, 4, 5]], [16], [40], 1)  # a sequence that shrank
    assert err == 0 and (got == 0).all()
    got, err = go([[1, 4, 5]], [-3], [-9], 1)
    assert err == 0 and (got == 0).all()


# ------------------------------------------------------------------ GPU: scores


@pytest.mark.gpu
@pytest.mark.parametrize("D,BS,G,Hkv,Q", [
    (64, 8, 1, 3, 1), (128, 16, 4, 8, 1), (64, 32, 8, 1, 1), (128, 8, 8, 2, 3), (64, 16, 2, 5, 4),
    (128, 32, 4, 2, 17), (128, 16, 1, 1, 9)])
@pytest.mark.parametrize("scaled", [False, True])
def test_scores(pk, D, BS, G, Hkv, Q, scaled):
    import torch

    lens = [0, Q, BS + Q, 7 * BS, 16 * BS + 1, 1000, 2345]
    tables, NB, _ = layout(lens, BS, D + BS)
    rng = np.random.default_rng(Q + G)
    x = rng.standard_normal((NB, Hkv, 2, D)) * np.where(np.arange(D) % 16 == 5, 4.0, 1.0)
    bounds = torch.from_numpy(np.sort(x, 2)).bfloat16()
    ks = (rng.uniform(0.5, 2, Hkv) * np.where(np.arange(Hkv) % 2, -1, 1)).astype(np.float32)
    q = workloads.bf16_normal((len(lens), Q, G * Hkv, D), 3)
    want, mag = plain_scores(q.double().numpy(), bounds.double().numpy(), ks if scaled else None,
                             tables, lens, BS, D ** -0.5)
    start = torch.randn(len(lens), Hkv, tables.shape[1] + 2)
    got = pk.pa_block_scores((q if Q > 1 else q[:, 0]).contiguous().cuda(), bounds.cuda(),
                             dev(tables), dev(np.array(lens, np.int32)), 2345, BS,
                             scores=start.cuda(), k_scale=dev(ks) if scaled else None).cpu().numpy()
    assert pk.pa_device_errors() == 0
    left = start.numpy().copy()
    for at, s in want.items():
        assert abs(got[at] - s) <= 2.0 ** -17 * mag[at], (at, got[at], s)
        left[at] = got[at]
    assert np.array_equal(left, got)  # nothing else was written


@pytest.mark.gpu
def test_scores_that_are_no_numbers(pk):
    """Infinite and NaN bounds and queries: +infinity wherever the bound is no number."""
    import torch

    tables = np.array([[0, 1, 2, 3, 4, 5]], np.int32)
    bounds = torch.zeros(6, 1, 2, 64, dtype=torch.bfloat16)
    bounds[:, :, 1] = 1.0
    bounds[1, 0, 1, 7] = math.inf    # a finite query element below 0: 0 * inf
    bounds[2, 0, 0, 7] = -math.inf
    bounds[3, 0, 0, 9] = math.nan
    bounds[4, 0, :, 9] = math.nan
    bounds[5, 0, :, 7] = math.inf    # least and largest: q < 0 makes it -inf
    q = torch.ones(1, 1, 1, 64, dtype=torch.bfloat16)
    q[..., 7] = -2.0
    want, _ = plain_scores(q.double().numpy(), bounds.double().numpy(), None, tables, [96], 16, 0.5)
    got = pk.pa_block_scores(q[:, 0].cuda(), bounds.cuda(), dev(tables),
                             dev(np.array([96], np.int32)), 96, 16, scale=0.5).cpu().numpy()
    for at, s in want.items():
        assert got[at] == s, at
    assert np.isinf(got[0, 0, 1:]).all() and got[0, 0, 0] == 31.5


@pytest.mark.gpu
def test_scores_bad_lengths_and_entries(pk):
    import torch

    bounds = torch.randn(4, 2, 2, 64).sort(2)[0].bfloat16().cuda()
    q = workloads.bf16_normal((3, 2, 4, 64), 3).cuda()
    start = torch.full((3, 2, 5), 7.0, device="cuda")
    tables = np.array([[0, 1, 2, 3], [0, 99, -1, 3], [1, 2, 3, 0]], np.int32)
    got = pk.pa_block_scores(q, bounds, dev(tables), dev(np.array([1, 64, 9999], np.int32)), 64, 16,
                             scores=start.clone())
    assert pk.pa_device_errors() == pk.DEVERR_CONTEXT_LEN | pk.DEVERR_TABLE_ENTRY
    assert (got[0] == 7).all() and (got[:, :, 4] == 7).all()
    ok = pk.pa_block_scores(q, bounds, dev(tables.clip(0, 3)), dev(np.array([0, 64, 64], np.int32)),
                            64, 16, scores=start.clone())
    assert torch.equal(ok[2], got[2]) and torch.equal(ok[1, :, [0, 3]], got[1, :, [0, 3]])
    assert pk.pa_device_errors() == 0


# ------------------------------------------------------------------ GPU: choice


def _scores(rng, B, H, n, kind):
    x = rng.standard_normal((B, H, n)).astype(np.float32) * 3
    if kind == "ties":
        x = np.round(x)
    elif kind == "equal":
        x[:] = -2.5
    elif kind == "special":
        for v in (np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-45, 3.4e38, -3.4e38):
            x[rng.random(x.shape) < 0.06] = v
    elif kind == "nan":
        x[:] = np.nan
        x[..., ::7] = 1.0
    elif kind == "close":  # neighbours in the last place
        x = np.nextafter(np.float32(8), np.float32(9)) * np.ones_like(x)
        x[rng.random(x.shape) < 0.5] = 8.0
    return x


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["normal", "ties", "equal", "special", "nan", "close"])
@pytest.mark.parametrize("budget,sink,recent", [(1, 0, 0), (1, 0, 1), (1, 1, 0), (5, 1, 2),
                                                (64, 2, 4), (64, 32, 32), (200, 0, 0),
                                                (700, 1, 1)])
@pytest.mark.parametrize("BS", [8, 32])
def test_select(pk, kind, budget, sink, recent, BS):
    import torch

    rng = np.random.default_rng(budget)
    lens = [0, 1, BS, BS * budget, BS * budget + 1, 64 * BS + 3, 201 * BS, 777 * BS - 5]
    x = _scores(rng, len(lens), 3, max(-(-n // BS) for n in lens) + 3, kind)
    got = pk.pa_block_select(dev(x), dev(np.array(lens, np.int32)), BS, budget, sink, recent)
    assert np.array_equal(got.cpu().numpy(), plain_select(x, lens, BS, budget, sink, recent))
    assert pk.pa_device_errors() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("stride,n", [(2047, 2047), (2048, 2048), (2049, 2049), (16384, 16384),
                                      (16385, 9000), (40000, 40000), (131072, 100001)])
@pytest.mark.parametrize("kind", ["normal", "ties", "special"])
def test_select_of_long_rows(pk, stride, n, kind):
    """Rows on either side of what registers hold, and of many spans."""
    x = _scores(np.random.default_rng(stride), 2, 2, stride, kind)
    lens = [8 * n, 8 * (n // 2) - 3]
    for budget, sink, recent in ((n // 2, 1, 3), (33, 0, 1), (n - 1, 0, 0)):
        got = pk.pa_block_select(dev(x), dev(np.array(lens, np.int32)), 8, budget, sink, recent)
        assert np.array_equal(got.cpu().numpy(), plain_select(x, lens, 8, budget, sink, recent))


def _spread(rng, B, H, n, kind):
    """Scores that no one width of bin suits."""
    x = rng.standard_normal((B, H, n)).astype(np.float32)
    if kind == "outlier":  # all but one in a bin of equal widths
        x[..., n // 3] = 1e30
    elif kind == "outliers":
        x[..., n // 3], x[..., n // 2] = 1e30, -1e30
    elif kind == "exponents":
        x = np.ldexp(np.sign(x), rng.integers(-149, 128, x.shape)).astype(np.float32)
    elif kind == "subnormal":
        x = (x * 1e-42).astype(np.float32)
    elif kind == "ends":  # a difference that overflows
        x[..., n // 3], x[..., n // 2] = 3.4e38, -3.4e38
    elif kind == "halves":  # a difference near the largest number
        x[..., n // 3], x[..., n // 2] = 1.5e38, -1.5e38
    elif kind == "clusters":  # runs of 31 to 34 neighbours in the last place, far apart
        at = np.cumsum(rng.integers(31, 35, n))
        which = np.searchsorted(at, np.arange(n), side="right")
        step = np.arange(n) - np.concatenate([[0], at])[which]
        base = (which + 1).astype(np.float32)
        x = np.broadcast_to((base.view(np.int32) + step.astype(np.int32)).view(np.float32), x.shape)
        x = rng.permuted(x, axis=-1)
    return np.ascontiguousarray(x, np.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["outlier", "outliers", "exponents", "subnormal", "ends", "halves",
                                  "clusters"])
@pytest.mark.parametrize("n", [70, 1027, 2048, 4095, 8000, 16384, 20001])
def test_select_of_scores_of_all_sizes(pk, kind, n):
    x = _spread(np.random.default_rng(n), 2, 3, n, kind)
    lens = [16 * n, 16 * (n - 1) - 5]
    for budget, sink, recent in ((1, 0, 0), (33, 1, 1), (64, 0, 4), (n // 2, 1, 0), (n - 1, 0, 0)):
        got = pk.pa_block_select(dev(x), dev(np.array(lens, np.int32)), 16, budget, sink, recent)
        assert np.array_equal(got.cpu().numpy(), plain_select(x, lens, 16, budget, sink, recent))


@pytest.mark.gpu
def test_select_of_a_row_that_is_too_short(pk):
    x = np.arange(20, dtype=np.float32).reshape(1, 2, 10)
    lens = dev(np.array([2**31 - 1], np.int32))
    got = pk.pa_block_select(dev(x), lens, 16, 4, 1, 1)
    assert pk.pa_device_errors() == pk.DEVERR_CONTEXT_LEN
    assert got.cpu().tolist() == [[[0, 7, 8, 9]] * 2]
    got = pk.pa_block_select(dev(x), dev(np.array([-5], np.int32)), 16, 4, 1, 1)
    assert got.cpu().tolist() == [[[-1] * 4] * 2] and pk.pa_device_errors() == 0


# ------------------------------------------------------------------ GPU: decode


def lists(rng, lens, Hkv, BS, S, how):
    """Selected blocks: `some` as the choice gives them, `any` in any order, with holes."""
    out = np.full((len(lens), Hkv, S), -1, np.int32)
    for b, n in enumerate(lens):
        blocks = -(-max(n, 0) // BS)
        for h in range(Hkv):
            k = min(S, blocks)
            x = np.sort(rng.permutation(blocks)[:k])
            if how == "some" and k:
                x[-1] = blocks - 1
            if how == "any":
                rng.shuffle(x)
                x[rng.random(k) < 0.3] = -rng.integers(1, 5)
            out[b, h, :k] = x
    return out


SHAPES = [(64, 8, 1, 3, 1), (128, 16, 4, 8, 1), (64, 32, 8, 1, 1), (128, 8, 8, 2, 1),
          (64, 16, 2, 2, 2), (128, 32, 4, 2, 3), (128, 16, 2, 1, 5), (64, 8, 4, 2, 2),
          (128, 32, 1, 1, 8), (64, 16, 8, 1, 11), (128, 8, 1, 2, 4), (64, 32, 4, 3, 1)]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,BS,G,Hkv,Q", SHAPES)
@pytest.mark.parametrize("S,how", [(1, "some"), (7, "any"), (40, "some"), (300, "any")])
def test_decode(pk, fmt, D, BS, G, Hkv, Q, S, how):
    import torch

    lens = [0, Q, BS + Q, 5 * BS, 640, 641 + Q, 1999]
    tables, NB, poison = layout(lens, BS, D + BS + Q)
    c = Cache(fmt, NB, Hkv, BS, D, 11 + Q, poison)
    rng = np.random.default_rng(S)
    q = workloads.bf16_normal((len(lens), Q, G * Hkv, D), S)
    sel = lists(rng, lens, Hkv, BS, S, how)
    want, W, A, V = plain_attend(c, q.double().numpy(), tables, lens, sel, D ** -0.5)
    got = pk.pa_decode_selected((q if Q > 1 else q[:, 0]).contiguous().cuda(), c.k.cuda(),
                                c.v.cuda(), dev(tables), dev(np.array(lens, np.int32)), 1999,
                                dev(sel), **c.scales())
    assert pk.pa_device_errors() == 0
    close(got.double().cpu().numpy().reshape(want.shape), want, W, A, V, fmt, S * BS)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("B,S", [(1, 512), (1, 64), (3, 200), (40, 100), (200, 30)])
def test_decode_splits(pk, fmt, B, S):
    """One CTA a list and clusters of two, four and eight."""
    import torch

    rng = np.random.default_rng(B)
    lens = rng.integers(1, 9000 if B < 10 else 2000, B).tolist()
    lens[0] = 8192 if B < 10 else 1600
    tables, NB, poison = layout(lens, 16, B)
    c = Cache(fmt, NB, 2, 16, 128, B, poison)
    q = workloads.bf16_normal((B, 8, 128), S)
    sel = lists(rng, lens, 2, 16, S, "some")
    want, W, A, V = plain_attend(c, q.double().numpy()[:, None], tables, lens, sel, 128 ** -0.5)
    args = (q.cuda(), c.k.cuda(), c.v.cuda(), dev(tables), dev(np.array(lens, np.int32)), max(lens),
            dev(sel))
    got = pk.pa_decode_selected(*args, **c.scales())
    close(got.double().cpu().numpy()[:, None], want, W, A, V, fmt, S * 16)
    assert torch.equal(got, pk.pa_decode_selected(*args, **c.scales()))  # the same bits
    assert pk.pa_device_errors() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FMTS)
def test_decode_large_and_flat_scores(pk, fmt):
    """Scores of thousands, which one key takes, and of zero, which all share."""
    import torch

    lens = [777, 500]
    tables, NB, poison = layout(lens, 16, 3)
    c = Cache(fmt, NB, 2, 16, 128, 5, poison)
    for factor in (300.0, 0.0, 1e-30):
        q = workloads.bf16_normal((2, 8, 128), 5) * factor
        sel = lists(np.random.default_rng(1), lens, 2, 16, 30, "some")
        want, W, A, V = plain_attend(c, q.double().numpy()[:, None], tables, lens, sel, 128 ** -0.5)
        got = pk.pa_decode_selected(q.cuda(), c.k.cuda(), c.v.cuda(), dev(tables),
                                    dev(np.array(lens, np.int32)), 777, dev(sel), **c.scales())
        close(got.double().cpu().numpy()[:, None], want, W, A, V, fmt, 480)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("BS", [8, 16, 32])
@pytest.mark.parametrize("G,Q", [(4, 2), (2, 4), (8, 3), (1, 6)])
def test_decode_nan_of_later_tokens_stays_there(pk, fmt, BS, G, Q):
    """A token whose rows are NaN reaches the new tokens that see it and no other one."""
    import torch

    L = 5 * BS + 3 + Q
    tables, NB, poison = layout([L], BS, 2)
    t = L - Q + 1  # the second new token's own row
    c = Cache(fmt, NB, 1, BS, 64, 5, poison + [(int(tables[0, t // BS]), t % BS)])
    q = workloads.bf16_normal((1, Q, G, 64), 5)
    sel = np.arange(-(-L // BS), dtype=np.int32)[None, None]
    got = pk.pa_decode_selected(q.cuda(), c.k.cuda(), c.v.cuda(), dev(tables),
                                dev(np.array([L], np.int32)), L, dev(sel), **c.scales())
    got = got.double().cpu().numpy()
    assert np.isnan(got[0, 1:]).all() and not np.isnan(got[0, 0]).any()
    clean = Cache(fmt, NB, 1, BS, 64, 5, poison)
    want, W, A, V = plain_attend(clean, q.double().numpy(), tables, [L], sel, 0.125)
    close(got[:, :1], want[:, :1], W[:, :1], A[:, :1], V[:, :1], fmt, L)


@pytest.mark.gpu
def test_decode_bad_lengths_lists_and_tables(pk):
    import torch

    c = Cache("bf16", 8, 2, 16, 64, 5)
    q = workloads.bf16_normal((4, 2, 4, 64), 5).cuda()
    tables = np.array([[0, 1, 2], [3, 4, 5], [6, 99, 7], [1, -3, 2]], np.int32)
    lens = np.array([1, 9999, 48, -4], np.int32)
    sel = np.full((4, 2, 3), -1, np.int32)
    sel[1] = [0, 2, 7]
    sel[2] = [1, 0, 2]
    out = pk.pa_decode_selected(q, c.k.cuda(), c.v.cuda(), dev(tables), dev(lens), 48, dev(sel))
    assert pk.pa_device_errors() == pk.DEVERR_CONTEXT_LEN | pk.DEVERR_KEEP | pk.DEVERR_TABLE_ENTRY
    assert (out[0] == 0).all() and (out[3] == 0).all()
    ok = np.array([0, 48, 48, 0], np.int32)
    sel[1], sel[2] = [0, 2, -1], [0, 2, -1]
    again = pk.pa_decode_selected(q, c.k.cuda(), c.v.cuda(), dev(tables.clip(0, 7)), dev(ok), 48,
                                  dev(sel))
    assert torch.equal(out[1:3], again[1:3]) and pk.pa_device_errors() == 0


@pytest.mark.gpu
def test_decode_offsets_past_32_bits(pk):
    """Blocks at the end of caches of more than 4 GiB (2^31 elements)."""
    import torch

    NB, Hkv, BS, D = 140000, 8, 16, 128
    k = torch.zeros(NB, Hkv, BS, D, dtype=torch.bfloat16, device="cuda")
    small = Cache("bf16", 4, Hkv, BS, D, 1)
    at = [NB - 1, 5, NB - 2, NB - 7]
    k[at] = small.k.cuda()
    v = torch.zeros_like(k)
    v[at] = small.v.cuda()
    q = workloads.bf16_normal((1, 32, D), 5)
    sel = np.tile(np.array([0, 2, 3], np.int32), (1, Hkv, 1))
    want, W, A, V = plain_attend(small, q.double().numpy()[:, None], np.array([[0, 1, 2, 3]]), [60],
                              sel, D ** -0.5)
    lens, tables = dev(np.array([60], np.int32)), dev(np.array([at], np.int32))
    got = pk.pa_decode_selected(q.cuda(), k, v, tables, lens, 60, dev(sel))
    close(got.double().cpu().numpy()[:, None], want, W, A, V, "bf16", 48)
    bounds = torch.zeros(pk.block_bounds_shape(NB, Hkv, D), dtype=torch.bfloat16, device="cuda")
    pk.pa_block_bounds(k, bounds, tables, lens, 60)
    plain = plain_bounds(small, np.zeros((4, Hkv, 2, D)), np.array([[0, 1, 2, 3]]), [0], [60])
    assert np.array_equal(bounds[at].double().cpu().numpy(), plain)
    s = pk.pa_block_scores(q.cuda(), bounds, tables, lens, 60, BS).cpu().numpy()
    want, mag = plain_scores(q.double().numpy()[:, None], plain, None, np.array([[0, 1, 2, 3]]),
                             [60], BS, D ** -0.5)
    assert all(abs(s[i] - x) <= 2.0 ** -17 * mag[i] for i, x in want.items())


# ------------------------------------------------------------------ GPU: a run of them


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,D,BS", [("bf16", 128, 16), ("fp8", 128, 16), ("fp4", 64, 32),
                                      ("fp8", 64, 8)])
def test_steps_together(pk, fmt, D, BS):
    """Prompts, then decode steps: tables on the device, write, bounds, scores, choice,
    attention, all in one captured step that is replayed. While the budget covers the
    context the result is the whole decode's; then it is that over the listed blocks."""
    import torch

    B, Hkv, G, budget = 3, 2, 4, 6
    lens = [5 * BS - 2, 3 * BS + 5, 1]
    steps, NB, mb = 2 * BS + 3, 40, 12
    rng = np.random.default_rng(8)
    ring, state = pk.make_free_ring(rng.permutation(NB), NB)
    nstate = torch.empty_like(state)
    tables = torch.full((B, mb), -1, dtype=torch.int32, device="cuda")
    old = torch.zeros(B, dtype=torch.int32, device="cuda")
    new = torch.tensor(lens, dtype=torch.int32, device="cuda")
    like = Cache(fmt, NB, Hkv, BS, D, 1)
    sc = like.scales()
    k, v = like.k.cuda(), like.v.cuda()
    bounds = torch.zeros(pk.block_bounds_shape(NB, Hkv, D), dtype=torch.bfloat16, device="cuda")
    write = {"bf16": pk.pa_reshape_and_cache, "fp8": pk.pa_reshape_and_cache_fp8,
             "fp4": pk.pa_reshape_and_cache_fp4}[fmt]
    extra = () if fmt == "bf16" else (sc["k_scale"].abs(), sc["v_scale"].abs())
    scales = {} if fmt == "bf16" else dict(k_scale=extra[0], v_scale=extra[1])
    rows = [torch.randn(64 * 8, Hkv, D, device="cuda").bfloat16() for _ in range(2)]

    def grow(n, slots):
        pk.pa_update_tables(tables, old, new, ring, state, nstate, NB, BS, slot_mapping=slots)
        write(rows[0][:n], rows[1][:n], k, v, slots, *extra)
        pk.pa_block_bounds(k, bounds, tables, new, max(lens) + 1, old_lens=old)
        state.copy_(nstate)

    grow(sum(lens) + 2, torch.empty(sum(lens) + 2, dtype=torch.int64, device="cuda"))
    q = torch.randn(B, Hkv * G, D, device="cuda").bfloat16()
    slots = torch.empty(B, dtype=torch.int64, device="cuda")
    scores = torch.zeros(B, Hkv, mb, device="cuda")
    out = torch.empty_like(q)
    most = max(lens) + steps
    sel = torch.empty(B, Hkv, budget, dtype=torch.int32, device="cuda")

    def step():
        old.copy_(new)
        new.add_(1)
        grow(B, slots)
        pk.pa_block_scores(q, bounds, tables, new, most, BS, scores=scores,
                           k_scale=scales.get("k_scale"))
        pk.pa_block_select(scores, new, BS, budget, 1, 1, selected=sel)
        pk.pa_decode_selected(q, k, v, tables, new, most, sel, out=out, **scales)

    step()  # once before the capture: lazy set-up
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    torch.cuda.synchronize()
    short = 0
    for _ in range(steps - 1):
        for x in rows:
            x.normal_()
        q.normal_()
        graph.replay()
        torch.cuda.synchronize()
        now, t = new.cpu().tolist(), tables.cpu().numpy()
        if fmt == "bf16":
            like.k_values, like.v_values = (x.double().cpu().numpy() for x in (k, v))
        else:
            every = torch.arange(NB * BS, device="cuda")
            if fmt == "fp4":
                got = [x.double().cpu().numpy() for x in (
                    oracle_values(k, extra[0], D), oracle_values(v, extra[1], D))]
            else:
                W = min(BS, 16)
                got = [oracle.e4m3_to_f64(x.cpu().numpy()) * e.double().cpu().numpy()[:, None, None]
                       for x, e in ((k, extra[0]),
                                    (v.transpose(-1, -2).reshape(NB, Hkv, BS, D), extra[1]))]
            like.k_values, like.v_values = got
        chosen = sel.cpu().numpy()
        assert np.array_equal(chosen, plain_select(scores.cpu().numpy(), now, BS, budget, 1, 1))
        want, W, A, V = plain_attend(like, q.double().cpu().numpy()[:, None], t, now, chosen,
                                  D ** -0.5)
        close(out.double().cpu().numpy()[:, None], want, W, A, V, fmt, budget * BS)
        whole = pk.pa_decode(q, k, v, tables, new, most, **scales).double().cpu().numpy()
        for b in range(B):
            if -(-now[b] // BS) <= budget:
                short += 1
                assert np.abs(whole[b] - out[b].double().cpu().numpy()).max() <= 2e-2
    assert short and pk.pa_device_errors() == 0


def oracle_values(cache, scale, D):
    import torch

    return torch.from_numpy(oracle.fp4_values(cache.cpu().numpy(), scale.cpu().numpy(), D))


@pytest.mark.gpu
def test_two_streams_at_once(pk):
    """Two calls in flight on streams of their own share nothing."""
    import torch

    sets = []
    for seed in (1, 2):
        lens = [3000, 2000, 1500, 4000]
        tables, NB, poison = layout(lens, 16, seed)
        c = Cache("bf16", NB, 4, 16, 128, seed, poison)
        q = workloads.bf16_normal((4, 16, 128), seed)
        sel = lists(np.random.default_rng(seed), lens, 4, 16, 90, "some")
        want = plain_attend(c, q.double().numpy()[:, None], tables, lens, sel, 128 ** -0.5)
        sets.append(((q.cuda(), c.k.cuda(), c.v.cuda(), dev(tables), dev(np.array(lens, np.int32)),
                      4000, dev(sel)), want, torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = [[pk.pa_decode_selected(*a, stream=s) for a, _, s in sets] for _ in range(20)]
    torch.cuda.synchronize()
    for pair in outs:
        for got, (_, (want, W, A, V), _) in zip(pair, sets):
            close(got.double().cpu().numpy()[:, None], want, W, A, V, "bf16", 90 * 16)


@pytest.mark.gpu
def test_decode_block_listed_twice_counts_twice(pk):
    lens = [90]
    tables, NB, poison = layout(lens, 16, 6)
    c = Cache("bf16", NB, 1, 16, 128, 6, poison)
    q = workloads.bf16_normal((1, 4, 128), 6)
    sel = np.array([[[5, 2, 5, 5, 0, 2]]], np.int32)
    want, W, A, V = plain_attend(c, q.double().numpy()[:, None], tables, lens, sel, 128 ** -0.5)
    got = pk.pa_decode_selected(q.cuda(), c.k.cuda(), c.v.cuda(), dev(tables),
                                dev(np.array(lens, np.int32)), 90, dev(sel))
    close(got.double().cpu().numpy()[:, None], want, W, A, V, "bf16", 96)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FMTS)
def test_decode_many_new_tokens(pk, fmt):
    """1,024 of them, a column group each at eight query heads a KV head."""
    import torch

    L, Q, G = 1100, 1024, 8
    tables, NB, poison = layout([L], 32, 4)
    c = Cache(fmt, NB, 1, 32, 64, 4, poison)
    q = workloads.bf16_normal((1, Q, G, 64), 4)
    sel = np.arange(35, dtype=np.int32)[None, None].copy()
    sel[0, 0, 3:9] = -1
    got = pk.pa_decode_selected(q.cuda(), c.k.cuda(), c.v.cuda(), dev(tables),
                                dev(np.array([L], np.int32)), L, dev(sel), **c.scales())
    got = got.double().cpu().numpy()
    some = [0, 1, 19, 20, 211, 212, 700, 1023]
    for i in some:  # token i as the only new one of a shorter sequence
        n = L - Q + i + 1
        want, W, A, V = plain_attend(c, q.double().numpy()[:, i:i + 1], tables, [n], sel, 0.125)
        close(got[:, i:i + 1], want, W, A, V, fmt, L)
    assert torch.isfinite(torch.from_numpy(got)).all() and pk.pa_device_errors() == 0


@pytest.mark.gpu
def test_most_sequences(pk):
    """65,535 sequences that read one block."""
    import torch

    B, BS, D = 65535, 8, 64
    c = Cache("bf16", 2, 1, BS, D, 1, poison=[(1, o) for o in range(5, 8)])
    q = workloads.bf16_normal((B, 1, D), 2).cuda()
    tables = torch.ones(B, 1, dtype=torch.int32, device="cuda")
    lens = torch.full((B,), 5, dtype=torch.int32, device="cuda")
    bounds = torch.zeros(pk.block_bounds_shape(2, 1, D), dtype=torch.bfloat16, device="cuda")
    pk.pa_block_bounds(c.k.cuda(), bounds, tables, lens, 5)
    x = c.k_codes[1, 0, :5]
    assert np.array_equal(bounds[1, 0].double().cpu().numpy(), np.stack([x.min(0), x.max(0)]))
    scores = pk.pa_block_scores(q, bounds, tables, lens, 5, BS)
    qd = q.double().cpu().numpy()
    want, mag = plain_scores(qd[-3:, None], bounds.double().cpu().numpy(), None,
                             np.ones((3, 1), np.int32), [5] * 3, BS, D ** -0.5)
    assert all(abs(scores[B - 3 + i[0], 0, 0].item() - s) <= 2.0 ** -17 * mag[i]
               for i, s in want.items())
    sel = pk.pa_block_select(scores, lens, BS, 3, 1, 1)
    assert (sel == torch.tensor([0, -1, -1], dtype=torch.int32, device="cuda")).all()
    out = pk.pa_decode_selected(q, c.k.cuda(), c.v.cuda(), tables, lens, 5, sel)
    for b in (0, 1, 40000, B - 1):
        want, W, A, V = plain_attend(c, qd[b:b + 1, None], np.ones((1, 1), np.int32), [5],
                                     np.zeros((1, 1, 1), np.int32), D ** -0.5)
        close(out[b:b + 1].double().cpu().numpy()[:, None], want, W, A, V, "bf16", 8)
    assert torch.isfinite(out).all() and pk.pa_device_errors() == 0


@pytest.mark.parametrize("source", ["pa_tables.cu", "pa_blocks.cu", "pa_decode_selected.cu"])
def test_kernels_do_not_spill(source, tmp_path):
    """Launch bounds were chosen so that ptxas keeps every kernel in registers."""
    import os
    import re
    import subprocess

    from paged_kv_cache_92_gb300 import build

    got = subprocess.run([build._nvcc(), *build.ARCH, "-O3", "-std=c++17", f"-I{build.INCLUDE}",
                          "-lineinfo", "-Xptxas", "-v", "-cubin", "-o", str(tmp_path / "k.cubin"),
                          os.path.join(build.CSRC, source)], capture_output=True, text=True,
                         check=True)
    lines = re.findall(r"function '(\w+)'.*?(\d+) bytes spill stores, (\d+) bytes spill loads",
                       got.stderr, flags=re.S)
    assert lines and [x for x in lines if x[1:] != ("0", "0")] == []
