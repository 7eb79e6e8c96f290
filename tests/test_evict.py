"""Eviction: token weights, the choice under a budget, the move, and the pool's
half, against float64 and plain Python.

The choice and the move are integers and copies: equal. A token weight is a
sum of softmax weights in fp32. With A the largest scale * sum |q_i k_i| *
log2(e) of a row, a score takes 8 accumulations of 16 exact products (each
rounds by at most 2^-22 of a running value within A) and three roundings of
2^-24 A: 2^-18 A. Its exponential is off by that times ln 2, the
approximation's 2^-22 and, through the row's sum, as much again; sums of up
to 2^12 terms add 2^-12 * 2^-24 * 2^12. So a weight is within 2^-17 (1 + A) of
its value. The accumulated form adds one rounding of the total.
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


# ------------------------------------------------------------------ plain forms


def select(weights, lens, budget, recent):
    keep = np.full((len(lens), budget), -1, np.int32)
    for b, L in enumerate(lens):
        if L <= budget:
            got = range(L)
        else:
            old = L - recent
            w = [(-np.inf if np.isnan(x) else x, np.isnan(x)) for x in weights[b, :old].tolist()]
            order = sorted(range(old), key=lambda t: (w[t][1], -w[t][0], t))[:budget - recent]
            got = sorted(order) + list(range(old, L))
        keep[b, :len(got)] = list(got)
    return keep, np.minimum(lens, budget).astype(np.int32)


def rows_of(cache, fmt, which, D):
    """A view of a cache's rows [NB][Hkv][BS][...] per element kind (list of arrays)."""
    NB, Hkv = cache.shape[:2]
    if fmt == "bf16":
        return [cache]
    if fmt == "fp8":
        assert which == "k"
        return [cache]
    BS = cache.shape[2]
    flat = cache.reshape(NB, Hkv, -1)
    return [flat[..., :BS * D // 2].reshape(NB, Hkv, BS, D // 2),
            flat[..., BS * D // 2:].reshape(NB, Hkv, BS, D // 16)]


def compact(cache, fmt, which, D, BS, src, dst, keep, n):
    """The move on a copy, row by row from the old contents."""
    new, old = cache.copy(), cache.copy()
    if fmt == "fp8" and which == "v":
        W = min(BS, 16)
        def row(c, blk, off):
            return c.reshape(c.shape[0], c.shape[1], BS // W, D, W)[blk, :, off // W, :, off % W]
        for b in range(len(n)):
            for j in range(n[b]):
                t = keep[b, j]
                row(new, dst[b, j // BS], j % BS)[:] = row(old, src[b, t // BS], t % BS)
        return new
    for x, y in zip(rows_of(new, fmt, which, D), rows_of(old, fmt, which, D)):
        assert np.shares_memory(x, new)
        for b in range(len(n)):
            for j in range(n[b]):
                t = keep[b, j]
                x[dst[b, j // BS], :, j % BS] = y[src[b, t // BS], :, t % BS]
    return new


# ------------------------------------------------------------------ refusals (CPU)


def _tw(pk, **kw):
    p = pk.TokenWeightsParams()
    base = dict(weights_stride=64, max_blocks_per_seq=4, num_seqs=2, num_q_heads=8, num_kv_heads=2,
                head_dim=128, block_size=16, num_blocks=8, max_context_len=64, scale=0.088)
    base.update(kw)
    for k, v in base.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("kw,status", [
    (dict(), 1), (dict(head_dim=96), 2), (dict(block_size=4), 2), (dict(num_q_heads=6), 2),
    (dict(num_q_heads=7), 1), (dict(kv_dtype=3), 1), (dict(query_len=1025), 1),
    (dict(query_len=1024, num_seqs=300), 2), (dict(weights_stride=63), 1), (dict(scale=0.0), 1),
    (dict(scale=float("nan")), 1), (dict(max_context_len=0), 1), (dict(num_seqs=-1), 1),
    (dict(num_seqs=65536), 1), (dict(num_seqs=0), 0)])
def test_token_weights_refusals(pk, kw, status):
    p = _tw(pk, **kw)
    lib = pk.load()
    assert lib.pa_token_weights(ctypes.byref(p), None, 0, None) == status
    size = lib.pa_token_weights_workspace_size(ctypes.byref(p))
    assert (size > 0) == (status == 0 or not kw)
    assert lib.pa_token_weights(None, None, 0, None) == 1


@pytest.mark.parametrize("kw", [
    dict(max_blocks_per_seq=1 << 26, block_size=32), dict(scale=float("inf")),
    dict(num_seqs=512, max_blocks_per_seq=1 << 25, max_context_len=1 << 27, weights_stride=1 << 27),
    dict(num_seqs=32768, query_len=2, num_q_heads=32768, num_kv_heads=32768)])  # 2^31 rows
def test_token_weights_sizes_beyond_the_index_range(pk, kw):
    p = _tw(pk, **kw)
    assert pk.load().pa_token_weights(ctypes.byref(p), None, 0, None) == 1
    assert pk.load().pa_token_weights_workspace_size(ctypes.byref(p)) == 0


@pytest.mark.parametrize("stride,budget", [((1 << 30) + 1, 8), (64, (1 << 30) + 1),
                                           (2**31 - 1, 2**31 - 1)])
def test_select_sizes_beyond_the_index_range(pk, stride, budget):
    lib = pk.load()
    assert lib.pa_evict_select(256, 256, 256, 256, 1, stride, budget, 0, None) == 1
    assert b"2^30" in lib.pa_last_error()


@pytest.mark.parametrize("at", [0, 4, -4])
def test_select_refuses_lengths_in_place(pk, at):
    """The kept lengths over the lengths that other CTAs may still have to read."""
    lib = pk.load()
    assert lib.pa_evict_select(256, 1024, 256, 1024 + at, 2, 64, 8, 0, None) == 1
    assert b"overlap" in lib.pa_last_error()


@pytest.mark.parametrize("kw", [dict(max_blocks_per_seq=1 << 26), dict(max_dst_blocks_per_seq=1 << 26)])
def test_compact_sizes_beyond_the_index_range(pk, kw):
    p = pk.EvictCompactParams()
    base = dict(num_seqs=1, num_kv_heads=1, num_blocks=1, max_blocks_per_seq=1,
                max_dst_blocks_per_seq=1, keep_stride=1, head_dim=64, block_size=32)
    base.update(kw)
    for k, v in base.items():
        setattr(p, k, v)
    lib = pk.load()
    assert lib.pa_evict_compact(ctypes.byref(p), None) == 1 and b"2^30" in lib.pa_last_error()


def test_token_weights_workspace(pk):
    """The header, a (max, sum) per row and partition, and every score."""
    p = _tw(pk, query_len=3)
    rows = 2 * 3 * 8
    want = 256 + -(-rows * 8 // 256) * 256 + -(-rows * 64 * 4 // 256) * 256
    assert pk.load().pa_token_weights_workspace_size(ctypes.byref(p)) == want
    for f in ("q", "k_cache", "block_tables", "context_lens", "token_weights"):
        setattr(p, f, 256)
    lib = pk.load()
    assert lib.pa_token_weights(ctypes.byref(p), 256, want - 1, None) == 1
    assert lib.pa_token_weights(ctypes.byref(p), 128, want, None) == 1
    p.q = 264
    assert lib.pa_token_weights(ctypes.byref(p), 256, want, None) == 1


@pytest.mark.parametrize("args,status", [
    ((2, 64, 0, 0), 1), ((2, 64, 8, -1), 1), ((2, 64, 8, 9), 1), ((-1, 64, 8, 0), 1),
    ((2, 0, 8, 0), 1), ((65536, 64, 8, 0), 1), ((2, 64, 8, 8), 1), ((0, 64, 8, 8), 0)])
def test_select_refusals(pk, args, status):
    assert pk.load().pa_evict_select(None, None, None, None, *args, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(), 1), (dict(head_dim=96), 2), (dict(block_size=12), 2), (dict(kv_dtype=5), 1),
    (dict(keep_stride=0), 1), (dict(num_seqs=70000), 1), (dict(max_dst_blocks_per_seq=0), 1),
    (dict(token_weights=256, weights_stride=0), 1), (dict(num_seqs=0), 0)])
def test_compact_refusals(pk, kw, status):
    p = pk.EvictCompactParams()
    base = dict(max_blocks_per_seq=4, max_dst_blocks_per_seq=2, keep_stride=8, num_seqs=2,
                num_kv_heads=2, head_dim=64, block_size=16, num_blocks=8)
    base.update(kw)
    for k, v in base.items():
        setattr(p, k, v)
    assert pk.load().pa_evict_compact(ctypes.byref(p), None) == status
    if not kw:
        for f in ("k_cache", "v_cache", "block_tables", "dst_tables", "keep", "new_lens"):
            setattr(p, f, 256)
        p.v_cache = 257
        assert pk.load().pa_evict_compact(ctypes.byref(p), None) == 1


def test_binding_refusals(pk):
    import torch

    q = torch.zeros(2, 8, 64, dtype=torch.bfloat16)
    k = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16)
    t = torch.zeros(2, 2, dtype=torch.int32)
    n = torch.zeros(2, dtype=torch.int32)
    w = torch.zeros(2, 32)
    with pytest.raises(ValueError):
        pk.pa_token_weights(q, k, t, n, 32, w)
    with pytest.raises(ValueError):
        pk.pa_evict_select(w, n[:1], 4)
    with pytest.raises(ValueError):
        pk.pa_evict_select(w, n, 4, keep=torch.zeros(2, 5, dtype=torch.int32))
    with pytest.raises(ValueError):
        pk.pa_evict_compact(k, k[:3], t, t, t, n)
    with pytest.raises(ValueError):
        pk.pa_evict_compact(k, k, t[:1], t, t, n)


# ------------------------------------------------------------------ the pool (CPU)


def test_pool_compact_keeps_own_blocks_and_replaces_shared_ones(pk):
    pool = pk.Pool(16, 4)
    a = pool.seq_create()
    pool.append_tokens(a, 18)                  # 5 blocks: 0..4
    b = pool.seq_fork(a, 8)                    # shares blocks 0, 1
    pool.append_tokens(b, 9)                   # 17 tokens, blocks 0, 1, 5, 6, 7
    c = pool.seq_create()
    pool.append_tokens(c, 3)                   # block 8
    ta, tb = pool.table(a), pool.table(b)
    pool.compact([a, b, c], [10, 17, 3])       # b and c keep their lengths
    assert pool.table(b) == tb and pool.length(b) == 17
    got = pool.table(a)
    assert pool.length(a) == 10 and got[2] == ta[2] and len(got) == 3
    assert not set(got[:2]) & set(ta + tb)     # the shared blocks are replaced by fresh ones
    assert pool.refcount(ta[0]) == 1 and pool.refcount(ta[3]) == 0 and pool.refcount(ta[4]) == 0
    # both of a batch that share a block get fresh ones, although the first gives its share up
    d = pool.seq_fork(b, 8)
    td, tb = pool.table(d), pool.table(b)
    pool.compact([d, b], [6, 9])
    assert not set(pool.table(d)) & set(td + tb)
    assert not set(pool.table(b)[:2]) & set(td + tb) and pool.table(b)[2] == tb[2]
    assert not set(pool.table(b)) & set(pool.table(d))
    pool.compact([b], [0])
    assert pool.table(b) == [] and pool.length(b) == 0
    for s in (a, b, c, d):
        pool.seq_free(s)
    assert pool.stats()["free_blocks"] == 16


def test_pool_compact_never_writes_prefix_cache_blocks(pk):
    pool = pk.Pool(8, 4)
    seq, cached, _ = pool.create_prompt(list(range(10)))
    t = pool.table(seq)
    pool.compact([seq], [6])
    assert not set(pool.table(seq)) & set(t[:2])   # two full prompt blocks are cached
    again, cached, _ = pool.create_prompt(list(range(10)))
    assert cached == 8 and pool.table(again)[:2] == t[:2]


def test_pool_compact_is_all_or_nothing(pk):
    pool = pk.Pool(6, 4)
    a = pool.seq_create()
    pool.append_tokens(a, 16)
    b = pool.seq_fork(a, 16)                   # four shared blocks, two free
    before = pool.stats()
    with pytest.raises(pk.PoolOOM):
        pool.compact([a], [12])
    assert pool.stats() == before and pool.length(a) == 16
    for seqs, lens in (([a, a], [4, 4]), ([a], [17]), ([a], [-1])):
        with pytest.raises(pk.PagedKVError) as e:
            pool.compact(seqs, lens)
        assert e.value.status == 1
    with pytest.raises(pk.PagedKVError) as e:
        pool.compact([99], [0])
    assert e.value.status == 5
    assert pool.stats() == before
    pool.compact([], [])
    pool.compact([a, b], [4, 16])
    assert pool.refcount(pool.table(b)[1]) == 1


# ------------------------------------------------------------------ GPU


class Case:
    def __init__(self, fmt, lens, Hq, Hkv, D=128, BS=16, Q=1, seed=0, spare=0):
        import torch

        self.fmt, self.Hq, self.Hkv, self.D, self.BS, self.Q = fmt, Hq, Hkv, D, BS, Q
        self.lens = np.asarray(lens, np.int32)
        need = int(((self.lens + BS - 1) // BS).sum())
        self.NB = NB = need + 3 + spare
        order = np.random.default_rng(seed).permutation(NB).astype(np.int32)
        self.tables = workloads.sequential_tables(self.lens.astype(np.int64), order, BS,
                                                  max(1, int(-(-self.lens.max() // BS))))
        self.spare = order[need:]
        self.q = workloads.bf16_normal((len(lens), Q, Hq, D), seed + 1)
        rng = np.random.default_rng(seed + 2)
        self.s = (0.05 * np.exp(rng.uniform(-0.5, 0.5, Hkv))).astype(np.float32)
        rows = workloads.bf16_normal((NB, Hkv, BS, D), seed + 3)
        if fmt == "bf16":
            self.k = rows
            self.v = workloads.bf16_normal((NB, Hkv, BS, D), seed + 4)
            self.kval = oracle.bf16_to_f64(rows)
        elif fmt == "fp8":
            x = (rows.float() / torch.from_numpy(self.s)[:, None, None]).clamp(-448, 448)
            self.k = x.to(torch.float8_e4m3fn).view(torch.uint8)
            W = min(BS, 16)
            self.v = torch.from_numpy(rng.integers(0, 256, (NB, Hkv, BS // W, D, W), np.uint8))
            self.kval = oracle.e4m3_to_f64(self.k.numpy()) * self.s[:, None, None]
        else:
            flat = oracle.bf16_to_f64(rows).transpose(0, 2, 1, 3).reshape(NB * BS, Hkv, D)
            zero = np.zeros((NB, Hkv, BS, D * 9 // 16), np.uint8)
            k = oracle.fp4_write(flat, zero, np.arange(NB * BS), self.s, D)
            self.kval = oracle.fp4_values(k, self.s, D)
            self.k = torch.from_numpy(k)
            self.v = torch.from_numpy(oracle.fp4_write(flat[::-1], zero, np.arange(NB * BS), self.s, D))
        # slots behind a sequence's end hold NaN
        for b, L in enumerate(self.lens):
            if L % BS:
                blk, off = int(self.tables[b, (L - 1) // BS]), int(L % BS)
                if fmt == "fp4":
                    self.k.view(NB, Hkv, -1)[blk, :, BS * D // 2 + off * D // 16:] = 0x7F
                elif fmt == "fp8":
                    self.k[blk, :, off:] = 0x7F
                else:
                    self.k[blk, :, off:] = float("nan")

    def args(self):
        import torch

        q = self.q if self.Q > 1 else self.q[:, 0].contiguous()
        a = (q.cuda(), self.k.cuda(), torch.from_numpy(self.tables).cuda(),
             torch.from_numpy(self.lens).cuda(), max(1, int(self.lens.max())))
        return a, ({} if self.fmt == "bf16" else dict(k_scale=torch.from_numpy(self.s).cuda()))

    def want(self, stride, scale=None):
        q = oracle.bf16_to_f64(self.q)
        _, w = oracle.attention_rows(q, self.kval, None, self.tables, self.lens, scale)
        out = np.zeros((len(self.lens), stride))
        for b, x in enumerate(w):
            out[b, :x.shape[-1]] = x.sum((0, 1))
        A, sc = 0.0, (1 / np.sqrt(self.D)) if scale is None else scale
        for b, L in enumerate(self.lens):
            for h in range(self.Hq if L else 0):
                K = self.kval[self.tables[b][:-(-L // self.BS)], h // (self.Hq // self.Hkv)]
                K = np.abs(K.reshape(-1, self.D)[:L])
                A = max(A, float((K @ np.abs(q[b, :, h]).T).max()) * sc * 1.4427)
        return out, A


SHAPES = [(8, 8, 128, 16, 1), (4, 2, 64, 8, 3), (8, 1, 128, 32, 1), (16, 2, 64, 16, 5),
          (6, 3, 128, 8, 2), (2, 2, 64, 32, 17)]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("Hq,Hkv,D,BS,Q", SHAPES)
def test_token_weights(pk, fmt, Hq, Hkv, D, BS, Q):
    import torch

    lens = [Q, Q + 1, Q + 7, Q + 15, Q + 16, Q + 31, Q + 32, 129 + Q, 300]
    c = Case(fmt, lens, Hq, Hkv, D, BS, Q, seed=Hq + D + BS + Q)
    args, sc = c.args()
    stride = 307
    want, A = c.want(stride)
    tol = 2.0 ** -17 * (1 + A) * want
    base = torch.rand(len(lens), stride, device="cuda")
    w = pk.pa_token_weights(*args, base.clone(), accumulate=False, **sc)
    got = w.cpu().double().numpy()
    for b, L in enumerate(lens):
        assert (np.abs(got[b, :L] - want[b, :L]) <= tol[b, :L] + 1e-37).all(), (b, A)
        assert torch.equal(w[b, L:], base[b, L:])  # behind the sequence: as it was
    acc = pk.pa_token_weights(*args, base.clone(), **sc)
    x = base.cpu().double().numpy() + want
    inside = np.arange(stride) < np.asarray(lens)[:, None]
    err = np.abs(acc.cpu().double().numpy() - np.where(inside, x, base.cpu().double().numpy()))
    assert (err <= np.where(inside, tol + 2.0 ** -23 * x, 0)).all()
    # the same bits again
    assert torch.equal(acc, pk.pa_token_weights(*args, base.clone(), **sc))
    assert pk.pa_device_errors() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp4"])
def test_token_weights_long_ragged_scale(pk, fmt):
    import torch

    c = Case(fmt, [5001, 1, 2048, 130], 8, 2, seed=9)
    args, sc = c.args()
    for scale in (None, 0.5):
        want, A = c.want(5001, scale)
        w = torch.zeros(4, 5001, device="cuda")
        pk.pa_token_weights(*args, w, scale=scale, **sc)
        got = w.cpu().double().numpy()
        assert (np.abs(got - want) <= 2.0 ** -17 * (1 + A) * want + 1e-37).all()
        assert np.allclose(got.sum(1), 8, rtol=1e-4)  # one per query head


@pytest.mark.gpu
def test_token_weights_empty_short_and_bad(pk):
    import torch

    c = Case("bf16", [40, 40, 40, 40], 4, 2, 64, Q=4, seed=3)
    args, _ = c.args()
    base = torch.rand(4, 50, device="cuda")
    lens = torch.tensor([0, 3, 40, 49], dtype=torch.int32, device="cuda")
    w = pk.pa_token_weights(args[0], args[1], args[2], lens, 48, base.clone(), accumulate=False)
    assert pk.pa_device_errors() == pk.DEVERR_CONTEXT_LEN
    assert torch.equal(w[:2], base[:2]) and torch.equal(w[2, 40:], base[2, 40:])
    want, A = c.want(50)
    assert (np.abs(w[2].cpu().double().numpy() - want[2])[:40] <= 2.0 ** -17 * (1 + A) * want[2, :40]).all()
    bad = args[2].clone()
    bad[0, 1] = -7
    pk.pa_token_weights(args[0], args[1], bad, args[3], 40, base.clone())
    assert pk.pa_device_errors() == pk.DEVERR_TABLE_ENTRY


def _weights_with_ties(rng, B, stride):
    w = rng.random((B, stride)).astype(np.float32) ** 4
    w = np.where(rng.random((B, stride)) < 0.5, np.round(w * 8) / 8, w).astype(np.float32)
    w[0, :7] = [np.nan, np.inf, -np.inf, -0.0, 0.0, -1.0, np.nan]
    return w


@pytest.mark.gpu
@pytest.mark.parametrize("budget,recent", [(1, 0), (1, 1), (7, 3), (64, 0), (64, 64), (100, 13),
                                           (1000, 1)])
def test_select(pk, budget, recent):
    import torch

    rng = np.random.default_rng(budget + recent)
    lens = np.array([400, 0, 1, 63, 64, 65, 100, 101, 399, 1023, 1024, 1025, 2600], np.int32)
    w = _weights_with_ties(rng, len(lens), 2600)
    w[5] = 0.0                       # all equal: the lowest indices
    w[8, :] = np.nan                 # NaN everywhere: likewise
    w[9] = -np.abs(w[9])
    want = select(w, lens, budget, recent)
    keep, n = pk.pa_evict_select(torch.from_numpy(w).cuda(), torch.from_numpy(lens).cuda(), budget,
                                 recent)
    assert np.array_equal(keep.cpu().numpy(), want[0]) and np.array_equal(n.cpu().numpy(), want[1])
    assert pk.pa_device_errors() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("budget,recent", [(33000, 100), (9, 2), (69000, 0), (12, 12)])
def test_select_beyond_one_span(pk, budget, recent):
    """Clusters of CTAs: sequences of a few tokens for each, of as many as one round of
    registers holds (8,192 a CTA), and of more."""
    import torch

    rng = np.random.default_rng(5)
    lens = np.array([70001, 32768, 32769 + recent, 40000, 65536 + recent, 13, 1, 9000], np.int32)
    w = _weights_with_ties(rng, 8, 70001)
    w[3, ::2] = 0.25                 # ties over every CTA of the cluster
    want = select(w, lens, budget, recent)
    keep, n = pk.pa_evict_select(torch.from_numpy(w).cuda(), torch.from_numpy(lens).cuda(), budget,
                                 recent)
    assert np.array_equal(keep.cpu().numpy(), want[0]) and np.array_equal(n.cpu().numpy(), want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("stride", [8192 + 5, 8193 + 5, 4 * 8192 + 5, 4 * 8192 + 6])
def test_select_at_the_change_of_ctas(pk, stride):
    """Rows of candidates that one CTA, four and eight hold: the last of each and the first."""
    import torch

    rng = np.random.default_rng(stride)
    lens = np.array([stride, stride - 1, 2048 * 4 + 5, 2049, 700, 600, 0], np.int32)
    w = _weights_with_ties(rng, 7, stride)
    w[1, 1::3] = 0.5
    want = select(w, lens, 600, 5)
    keep, n = pk.pa_evict_select(torch.from_numpy(w).cuda(), torch.from_numpy(lens).cuda(), 600, 5)
    assert np.array_equal(keep.cpu().numpy(), want[0]) and np.array_equal(n.cpu().numpy(), want[1])


@pytest.mark.gpu
def test_select_cuts_lengths_beyond_the_weights(pk):
    import torch

    w = torch.arange(20, dtype=torch.float32, device="cuda").view(1, 20)
    keep, n = pk.pa_evict_select(w, torch.tensor([21], dtype=torch.int32, device="cuda"), 4, 1)
    assert keep.tolist() == [[16, 17, 18, 19]] and n.tolist() == [4]
    assert pk.pa_device_errors() == pk.DEVERR_CONTEXT_LEN


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("D,BS,Hkv", [(128, 16, 2), (64, 8, 3), (128, 32, 1), (64, 32, 2),
                                      (128, 8, 8)])
@pytest.mark.parametrize("place", ["in place", "elsewhere", "mixed"])
def test_compact(pk, fmt, D, BS, Hkv, place):
    import torch

    lens = [1, 40, 77, 200, 613]
    budget = 65
    rng = np.random.default_rng(D + BS + Hkv)
    nb = -(-budget // BS)
    c = Case(fmt, lens, Hkv, Hkv, D, BS, seed=BS + Hkv, spare=nb * len(lens))
    w = rng.random((5, 620)).astype(np.float32)
    w[3, :30] = 2.0                        # a long run of rows that stay where they are
    keep, n = select(w, c.lens, budget, 9)
    src = c.tables
    dst = np.full((5, max(nb, 1)), -1, np.int32)
    spare = list(c.spare)
    for b in range(5):
        for j in range(-(-int(n[b]) // BS)):
            own = place == "in place" or (place == "mixed" and (b + j) % 2)
            dst[b, j] = src[b, j] if own else spare.pop()
    k0, v0 = c.k.cuda(), c.v.cuda()
    k, v, tw = k0.clone(), v0.clone(), torch.from_numpy(w).cuda()
    pk.pa_evict_compact(k, v, torch.from_numpy(src).cuda(), torch.from_numpy(dst).cuda(),
                        torch.from_numpy(keep).cuda(), torch.from_numpy(n).cuda(), tw)
    torch.cuda.synchronize()

    def raw(t):
        return (t.view(torch.int16) if t.dtype == torch.bfloat16 else t).cpu().numpy()

    for got, old, which in ((k, k0, "k"), (v, v0, "v")):
        want = compact(raw(old), fmt, which, D, BS, src, dst, keep, n)
        assert np.array_equal(raw(got), want), which
    want = np.zeros_like(w)
    for b in range(5):
        want[b, :n[b]] = w[b, keep[b, :n[b]]]
    assert np.array_equal(tw.cpu().numpy(), want)
    assert pk.pa_device_errors() == 0


@pytest.mark.gpu
def test_compact_long_in_place(pk):
    """Many tiles: the order of reads and writes within a sequence."""
    import torch

    for fmt in ("bf16", "fp8", "fp4"):
        c = Case(fmt, [6000, 5000], 2, 2, seed=4)
        rng = np.random.default_rng(0)
        w = rng.random((2, 6000)).astype(np.float32)
        w[1, :2500] = 3.0  # the second sequence's first half stays
        keep, n = select(w, c.lens, 4000, 17)
        k0, v0 = c.k.cuda(), c.v.cuda()
        k, v = k0.clone(), v0.clone()
        tab = torch.from_numpy(c.tables).cuda()
        pk.pa_evict_compact(k, v, tab, tab, torch.from_numpy(keep).cuda(),
                            torch.from_numpy(n).cuda())
        torch.cuda.synchronize()
        for got, old, which in ((k, k0, "k"), (v, v0, "v")):
            o = (old.view(torch.int16) if fmt == "bf16" else old).cpu().numpy()
            x = (got.view(torch.int16) if fmt == "bf16" else got).cpu().numpy()
            assert np.array_equal(x, compact(o, fmt, which, 128, 16, c.tables, c.tables, keep, n))


@pytest.mark.gpu
def test_compact_bad_device_values(pk):
    import torch

    c = Case("bf16", [64, 64], 2, 2, 64, seed=6)
    tab = torch.from_numpy(c.tables).cuda()
    keep = torch.tensor([[5, 3, 1, 64], [1, 2, 3, 4]], dtype=torch.int32, device="cuda")
    n = torch.tensor([4, 0], dtype=torch.int32, device="cuda")
    k0, v0 = c.k.cuda(), c.v.cuda()
    k, v = k0.clone(), v0.clone()
    pk.pa_evict_compact(k, v, tab, tab, keep, n)
    assert pk.pa_device_errors() == pk.DEVERR_KEEP
    blk = c.tables[0, 0]
    assert torch.equal(k[blk, :, 0], k0[blk, :, 5]) and torch.equal(k[blk, :, 1], k0[blk, :, 3])
    assert torch.equal(k[blk, :, 2:5], k0[blk, :, 2:5])  # entries 1 < 2 and 64: not moved
    bad = tab.clone()
    bad[1, 0] = c.NB
    pk.pa_evict_compact(k, v, tab, bad, keep, torch.tensor([0, 2], dtype=torch.int32, device="cuda"))
    assert pk.pa_device_errors() == pk.DEVERR_TABLE_ENTRY
    k1 = k.clone()
    pk.pa_evict_compact(k, v, tab, tab[:, :1].contiguous(), keep,
                        torch.tensor([0, 5], dtype=torch.int32, device="cuda"))
    assert pk.pa_device_errors() == pk.DEVERR_CONTEXT_LEN  # cut to the four that keep holds
    blk = c.tables[1, 0]
    assert torch.equal(k[blk, :, :4], k1[blk, :, 1:5])
    pk.pa_evict_compact(k, v, tab, tab, keep, torch.tensor([-3, 0], dtype=torch.int32, device="cuda"))
    assert pk.pa_device_errors() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
def test_a_run_together(pk, fmt):
    """Steps of a generation with a budget: append, weights accumulated, and now and
    then the choice, the pool's half and the move; a model of the tokens' rows in
    float64 follows. Shared prefix blocks survive for the sequence that keeps them."""
    import torch

    D, Hq, Hkv, BS, budget, recent = 128, 8, 2, 16, 40, 8
    pool = pk.Pool(64, BS)
    a = pool.seq_create()
    pool.append_tokens(a, 37)
    other = pool.seq_fork(a, 32)               # keeps two blocks of the prefix
    seqs = [a, pool.seq_create()]
    pool.append_tokens(seqs[1], 25)
    NB = 64
    s = torch.full((Hkv,), 0.05, device="cuda")
    sc = {} if fmt == "bf16" else dict(k_scale=s, v_scale=s)
    if fmt == "bf16":
        kc = torch.zeros(NB, Hkv, BS, D, dtype=torch.bfloat16, device="cuda")
        vc = kc.clone()
    elif fmt == "fp8":
        kc = torch.zeros(NB, Hkv, BS, D, dtype=torch.uint8, device="cuda")
        vc = torch.zeros(NB, Hkv, 1, D, BS, dtype=torch.uint8, device="cuda")
    else:
        kc = torch.zeros(pk.fp4_cache_shape(NB, Hkv, BS, D), dtype=torch.uint8, device="cuda")
        vc = kc.clone()

    def write(kn, vn, slots):
        slots = torch.tensor(slots, dtype=torch.int64, device="cuda")
        if fmt == "bf16":
            pk.pa_reshape_and_cache(kn, vn, kc, vc, slots)
        elif fmt == "fp8":
            pk.pa_reshape_and_cache_fp8(kn, vn, kc, vc, slots, s, s)
        else:
            pk.pa_reshape_and_cache_fp4(kn, vn, kc, vc, slots, s, s)

    def values(cache, which):
        x = cache.cpu()
        if fmt == "bf16":
            return oracle.bf16_to_f64(x)
        sv = s.cpu().numpy().astype(np.float64)[:, None, None]
        if fmt == "fp8":
            y = oracle.e4m3_to_f64(x.numpy())
            y = y if which == "k" else y[:, :, 0].transpose(0, 1, 3, 2)
            return y * sv
        return oracle.fp4_values(x.numpy(), s.cpu().numpy(), D)

    # the prompts
    for i, q in enumerate(seqs):
        n = pool.length(q)
        slots = [pool.table(q)[t // BS] * BS + t % BS for t in range(n)]
        rows = [workloads.bf16_normal((n, Hkv, D), 50 + 2 * i + j).cuda() for j in range(2)]
        write(*rows, slots)
    kept_prefix = [x.clone() for x in (kc[pool.table(other)], vc[pool.table(other)])]
    weights = torch.zeros(2, 96, device="cuda")
    model = np.zeros((2, 96))
    rows_model = [[(kv[pool.table(q)[t // BS], :, t % BS]) for t in range(pool.length(q))]
                  for q in seqs for kv in [values(kc, "k")]]
    evictions = 0
    for step in range(30):
        slots, cows = [], []
        for q in seqs:
            slot, cow = pool.append_slot(q)
            slots.append(slot)
            if cow:
                cows.append(cow)
        if cows:
            pair = torch.tensor(cows, dtype=torch.int32, device="cuda")
            {"bf16": pk.pa_copy_blocks, "fp8": pk.pa_copy_blocks_fp8,
             "fp4": pk.pa_copy_blocks_fp4}[fmt](kc, vc, pair)
        kn, vn = (workloads.bf16_normal((2, Hkv, D), 100 + 2 * step + j).cuda() for j in range(2))
        q = workloads.bf16_normal((2, Hq, D), 300 + step)
        tables, lens = pool.export(seqs, 16)
        tg, lg = torch.from_numpy(tables).cuda(), torch.from_numpy(lens).cuda()
        out = pk.pa_append_decode(q.cuda(), kc, vc, tg, lg, int(lens.max()), kn, vn,
                                  torch.tensor(slots, device="cuda"), **sc)
        kw = {} if fmt == "bf16" else dict(k_scale=s)
        pk.pa_token_weights(q.cuda(), kc, tg, lg, int(lens.max()), weights, **kw)
        kv, vv = values(kc, "k"), values(vc, "v")
        for b, sq in enumerate(seqs):
            rows_model[b].append(kv[tables[b, (lens[b] - 1) // BS], :, (lens[b] - 1) % BS])
            for t in range(lens[b]):  # every row is where the model has it
                assert np.array_equal(kv[tables[b, t // BS], :, t % BS], rows_model[b][t])
        want, w = oracle.attention_rows(oracle.bf16_to_f64(q)[:, None], kv, vv, tables, lens)
        assert np.abs(oracle.bf16_to_f64(out.cpu()) - want[:, 0]).max() <= 2e-2
        for b in range(2):
            model[b, :lens[b]] += w[b].sum((0, 1))
        got = weights.cpu().double().numpy()
        assert np.abs(got - model).max() <= 1e-4 * max(1.0, model.max())
        if step % 10 == 9:
            keep, n = pk.pa_evict_select(weights, lg, budget, recent)
            new = [min(int(x), budget) for x in lens]
            pool.compact(seqs, new)
            dst = torch.from_numpy(pool.export(seqs, 16)[0]).cuda()
            pk.pa_evict_compact(kc, vc, tg, dst, keep, n, weights)
            keep = keep.cpu().numpy()
            assert n.tolist() == new
            for b in range(2):
                at = keep[b, :new[b]]
                assert at[-recent:].tolist() == list(range(lens[b] - recent, lens[b])) or \
                    lens[b] <= budget
                rows_model[b] = [rows_model[b][t] for t in at]
                model[b] = np.append(model[b, at], np.zeros(96 - new[b]))
                evictions += lens[b] > budget
    assert evictions >= 3
    for x, y in zip(kept_prefix, (kc[pool.table(other)], vc[pool.table(other)])):
        assert torch.equal(x, y)
    assert pk.pa_device_errors() == 0
    pool.close()


@pytest.mark.gpu
def test_captured_and_on_another_stream(pk):
    """The three calls in one graph, replayed on new inputs, and on a side stream."""
    import torch

    c = Case("bf16", [300, 47, 129], 8, 2, seed=2, spare=20)
    args, _ = c.args()
    B, budget = 3, 50
    dst = torch.from_numpy(c.spare[:3 * 4].reshape(3, 4).copy()).cuda()
    w = torch.zeros(B, 300, device="cuda")
    v = c.v.cuda()
    ws = torch.empty(pk.pa_token_weights_workspace_size(*args, w), dtype=torch.uint8, device="cuda")
    keep = torch.empty(B, budget, dtype=torch.int32, device="cuda")
    n = torch.empty(B, dtype=torch.int32, device="cuda")
    q = args[0].clone()

    def step(stream=None):
        pk.pa_token_weights(q, *args[1:], w, accumulate=False, workspace=ws, stream=stream)
        pk.pa_evict_select(w, args[3], budget, 5, keep=keep, new_lens=n, stream=stream)
        pk.pa_evict_compact(args[1], v, args[2], dst, keep, n, stream=stream)

    def state():
        return [x.clone() for x in (w, keep, n, args[1], v)]

    step()
    want = state()
    for x in (w, keep, n):
        x.zero_()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    step(side)
    side.synchronize()
    got = state()
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(want, got))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    q.copy_(q.flip(1))
    g.replay()
    torch.cuda.synchronize()
    got = state()
    assert not torch.equal(got[1], want[1])
    step()
    want = state()
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(want, got))


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [False, True])
def test_a_call_allocates_on_its_own_stream(pk, handle):
    """Memory that a call on another stream borrows is not handed to the current one
    while the call still waits there, and the result does not come from memory that
    the current stream still writes."""
    import torch

    B, L, Hq, Hkv, D, BS = 2, 4000, 8, 2, 128, 16
    torch.manual_seed(3)
    nb = -(-L // BS)
    q = torch.randn(B, Hq, D, device="cuda").bfloat16()
    kc, vc = (torch.randn(B * nb, Hkv, BS, D, device="cuda").bfloat16() for _ in range(2))
    tab = torch.arange(B * nb, dtype=torch.int32, device="cuda").reshape(B, nb)
    lens = torch.tensor([L, 1234], dtype=torch.int32, device="cuda")
    w = torch.zeros(B, L, device="cuda")
    pk.pa_token_weights(q, kc, tab, lens, L, w)
    out = pk.pa_decode(q, kc, vc, tab, lens, L)
    keep, n = pk.pa_evict_select(w, lens, 300, 20)
    side = torch.cuda.Stream()
    on = side.cuda_stream if handle else side
    w2 = torch.zeros_like(w)
    size = pk.pa_token_weights_workspace_size(q, kc, tab, lens, L, w)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)           # some 10 ms
    pk.pa_token_weights(q, kc, tab, lens, L, w2, stream=on)
    out2 = pk.pa_decode(q, kc, vc, tab, lens, L, stream=on)
    keep2, n2 = pk.pa_evict_select(w2, lens, 300, 20, stream=on)
    mine = [torch.zeros(s, dtype=torch.uint8, device="cuda") for s in (size, size // 2, 4096, 512)]
    torch.cuda.synchronize()
    assert not any(m.any() for m in mine)
    assert torch.equal(w, w2) and torch.equal(out, out2)
    assert torch.equal(keep, keep2) and torch.equal(n, n2)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp4"])
def test_kernels_wait_for_the_one_before(pk, fmt):
    """A kernel's CTAs may be dispatched while the preceding kernel runs, one that lets its
    dependents start at its entry among them: what it writes is seen all the same. Every call
    follows at once a kernel that changes what it reads."""
    import torch

    B, L, Hq, Hkv, D, BS = 16, 1200, 8, 8, 128, 16
    torch.manual_seed(4)
    nb = -(-L // BS)
    T = B * nb * BS
    shape = pk.fp4_cache_shape(B * nb, Hkv, BS, D) if fmt == "fp4" else (B * nb, Hkv, BS, D)
    kc = torch.zeros(shape, dtype=torch.uint8 if fmt == "fp4" else torch.bfloat16, device="cuda")
    vc = kc.clone()
    sc = dict(k_scale=torch.full((Hkv,), .05, device="cuda"),
              v_scale=torch.full((Hkv,), .03, device="cuda")) if fmt == "fp4" else {}
    tab = torch.arange(B * nb, dtype=torch.int32, device="cuda").reshape(B, nb)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    slots = torch.arange(T, device="cuda")
    rows = [[torch.randn(T, Hkv, D, device="cuda").bfloat16() for _ in range(2)] for _ in range(2)]
    qs = [torch.randn(B, Hq, D, device="cuda").bfloat16() for _ in range(2)]
    ls = [torch.randint(600, L + 1, (B,), dtype=torch.int32, device="cuda") for _ in range(2)]
    q, w = qs[0].clone(), torch.zeros(B, L, device="cuda")
    ks = dict(k_scale=sc["k_scale"]) if sc else {}

    def step(i, settle):
        wait = torch.cuda.synchronize if settle else (lambda: None)
        lens.copy_(ls[i])
        wait()
        if fmt == "fp4":
            pk.pa_reshape_and_cache_fp4(*rows[i], kc, vc, slots, **sc)
        else:
            pk.pa_reshape_and_cache(*rows[i], kc, vc, slots)
        wait()
        pk.pa_token_weights(q, kc, tab, lens, L, w, accumulate=False, **ks)
        wait()
        q.copy_(qs[i])
        wait()
        out = pk.pa_decode(q, kc, vc, tab, lens, L, **sc)
        w.mul_(1 + i)
        wait()
        keep, n = pk.pa_evict_select(w, lens, 500, 30)
        wait()
        pk.pa_evict_compact(kc, vc, tab, tab, keep, n, w)
        wait()
        after = pk.pa_decode(q, kc, vc, tab, n, 500, **sc)
        got = [out, w.clone(), keep, n, after, kc.clone(), vc.clone()]
        if fmt == "fp4":
            got += pk.pa_gather_fp4(kc, vc, slots[:5000], **sc)
        return got

    step(0, True)
    want = [step(i, True) for i in (1, 0)]
    for _ in range(8):
        for i, ref in zip((1, 0), want):
            torch.cuda._sleep(200_000)
            for x, y in zip(step(i, False), ref):
                assert torch.equal(x, y)


@pytest.mark.gpu
def test_captured_behind_copies_fills_and_joined_streams(pk):
    """Capture where a call does not follow one kernel on its stream: behind a copy, a fill, a
    host-to-device copy, and behind two streams' work; and two branches of calls that join."""
    import torch

    B, L, Hq, Hkv, D, BS = 4, 3000, 8, 2, 128, 16
    torch.manual_seed(6)
    nb = -(-L // BS)
    k, v = (torch.randint(0, 256, pk.fp4_cache_shape(B * nb, Hkv, BS, D), dtype=torch.uint8,
                          device="cuda") for _ in range(2))
    for c in (k, v):
        c.view(B * nb, Hkv, -1)[..., BS * D // 2:] = 0x38        # group scales of one
    sc = dict(k_scale=torch.full((Hkv,), .05, device="cuda"),
              v_scale=torch.full((Hkv,), .03, device="cuda"))
    tab = torch.arange(B * nb, dtype=torch.int32, device="cuda").reshape(B, nb)
    host = torch.tensor([3000, 1, 1700, 2999], dtype=torch.int32).pin_memory()
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    q0 = torch.randn(B, Hq, D, device="cuda").bfloat16()
    q, out, out2 = torch.zeros_like(q0), torch.zeros_like(q0), torch.zeros_like(q0)
    w, junk = torch.ones(B, L, device="cuda"), torch.zeros(1 << 20, device="cuda")
    ws = [torch.empty(32 << 20, dtype=torch.uint8, device="cuda") for _ in range(2)]
    slots = torch.arange(100, device="cuda")
    main, side = torch.cuda.Stream(), torch.cuda.Stream()

    def body():
        lens.copy_(host, non_blocking=True)
        q.copy_(q0)
        pk.pa_decode(q, k, v, tab, lens, L, out=out, workspace=ws[0], **sc)
        w.zero_()
        pk.pa_token_weights(q, k, tab, lens, L, w, workspace=ws[0], k_scale=sc["k_scale"])
        side.wait_stream(main)
        with torch.cuda.stream(side):
            junk.add_(1)
            pk.pa_decode(q, k, v, tab, lens, L, out=out2, workspace=ws[1], **sc)
        keep, n = pk.pa_evict_select(w, lens, 200, 9)
        rows = pk.pa_gather_fp4(k, v, slots, **sc)
        main.wait_stream(side)
        pk.pa_evict_compact(k, v, tab, tab, keep, n)
        after = pk.pa_decode(q, k, v, tab, n, 200, workspace=ws[0], **sc)
        return keep, n, *rows, after

    k0, v0 = k.clone(), v.clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(main):
        want = body()
    torch.cuda.synchronize()
    want = [t.clone() for t in (*want, out, out2, w, k, v)]
    k.copy_(k0)
    v.copy_(v0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=main):
        got = body()
    for _ in range(3):
        k.copy_(k0)
        v.copy_(v0)
        lens.zero_()
        g.replay()
        torch.cuda.synchronize()
        for x, y in zip((*got, out, out2, w, k, v), want):
            assert torch.equal(x, y)
    assert pk.pa_device_errors() == 0


@pytest.mark.gpu
def test_compacted_weights_follow_their_rows(pk):
    """Where a row is not moved its weight stays too; a weight that the row of weights does
    not reach becomes zero and is flagged."""
    import torch

    c = Case("bf16", [64, 64], 2, 2, 64, seed=7)
    tab = torch.from_numpy(c.tables).cuda()
    w = torch.rand(2, 80, generator=torch.Generator().manual_seed(1)) + 0.5
    keep = torch.tensor([[2, 0, 5, 64, 70], [1, 2, 3, 4, 20]], dtype=torch.int32, device="cuda")
    n = torch.tensor([5, 5], dtype=torch.int32, device="cuda")
    dst = tab.clone()
    dst[1, 0] = c.NB                                   # no such block: nothing of sequence 1 moves
    k0, got = c.k.cuda(), w.cuda()
    k = k0.clone()
    pk.pa_evict_compact(k, c.v.cuda(), tab, dst, keep, n, got)
    assert pk.pa_device_errors() == pk.DEVERR_KEEP | pk.DEVERR_TABLE_ENTRY
    want = torch.zeros(2, 80)
    want[0, :5] = w[0, [2, 1, 5, 3, 4]]                # entries 0 < 1, 64 and 70: not moved
    want[1, :5] = w[1, :5]
    assert torch.equal(got.cpu(), want)
    old = [k0[c.tables[0, t // 16], :, t % 16] for t in (2, 1, 5, 3, 4)]
    assert all(torch.equal(k[c.tables[0, 0], :, j], x) for j, x in enumerate(old))

    short = w[:, :40].contiguous().cuda()              # weights of 40 tokens, tables of 64
    keep = torch.tensor([[3, 39, 40, 63], [0, 1, 2, 3]], dtype=torch.int32, device="cuda")
    pk.pa_evict_compact(k0, c.v.cuda(), tab, tab, keep, n - 1, short)
    assert pk.pa_device_errors() == pk.DEVERR_KEEP
    want = torch.zeros(2, 40)
    want[0, :2], want[1, :4] = w[0, [3, 39]], w[1, :4]
    assert torch.equal(short.cpu(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("budget", [513, 1200, 4000])
def test_compacted_weights_of_long_rows(pk, budget):
    """Many tiles of weights in place, of sequences cut a little, much and not at all."""
    import torch

    c = Case("bf16", [5000, 1201, 700, budget, 0], 1, 1, 64, seed=8)
    rng = np.random.default_rng(budget)
    w = rng.random((5, 5001)).astype(np.float32)
    w[1, :600] = 2.0
    keep, n = select(w, c.lens, budget, 11)
    tab, got = torch.from_numpy(c.tables).cuda(), torch.from_numpy(w).cuda()
    pk.pa_evict_compact(c.k.cuda(), c.v.cuda(), tab, tab, torch.from_numpy(keep).cuda(),
                        torch.from_numpy(n).cuda(), got)
    want = np.zeros_like(w)
    for b in range(5):
        want[b, :n[b]] = w[b, keep[b, :n[b]]]
    assert np.array_equal(got.cpu().numpy(), want)
    assert pk.pa_device_errors() == 0


def _check_weights(pk, c, stride, scale=None):
    import torch

    args, sc = c.args()
    want, A = c.want(stride, scale)
    tol = 2.0 ** -17 * (1 + A) * want + 1e-37
    base = torch.rand(len(c.lens), stride, device="cuda")
    w = pk.pa_token_weights(*args, base.clone(), accumulate=False, scale=scale, **sc)
    got = w.cpu().double().numpy()
    for b, L in enumerate(c.lens):
        assert (np.abs(got[b, :L] - want[b, :L]) <= tol[b, :L]).all(), (b, A)
        assert torch.equal(w[b, L:], base[b, L:])
    assert pk.pa_device_errors() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("Hq,Hkv,D,BS,Q", [(16, 4, 128, 16, 4), (8, 1, 128, 32, 2), (4, 4, 128, 8, 17),
                                           (32, 8, 128, 16, 3), (2, 2, 64, 8, 9)])
def test_token_weights_over_two_column_tiles(pk, fmt, Hq, Hkv, D, BS, Q):
    """More than eight query rows a KV head, and partitions (128 tokens here) that end
    among the new tokens, so that rows of one column group span different numbers of them."""
    lens = [Q, 128, 128 + Q // 2, 127 + Q, 128 + Q, 255, 256 + Q // 2, 255 + Q, 300]
    _check_weights(pk, Case(fmt, lens, Hq, Hkv, D, BS, Q, seed=Hq + BS + Q), 301)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D,Q,lens", [(8, 2, 128, 130, [130, 131, 200, 333]),
                                             (1, 1, 64, 1024, [1024, 1100])])
def test_token_weights_of_prompt_chunks(pk, Hq, Hkv, D, Q, lens):
    for fmt in ("bf16", "fp4"):
        _check_weights(pk, Case(fmt, lens, Hq, Hkv, D, 16, Q, seed=Q), max(lens))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("Q", [1, 5])
def test_token_weights_negative_and_zero_scales(pk, fmt, Q):
    """A head scale's sign turns the scores, zero makes them equal."""
    c = Case(fmt, [300, 47, 17], 8, 4, Q=Q, seed=11)
    f = np.array([1, -1, 0, -8], np.float32)
    c.s *= f
    c.kval *= f[:, None, None]
    _check_weights(pk, c, 300)
