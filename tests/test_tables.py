"""Block tables, slots and positions made on the device, against a plain walk over the
sequences. Everything is an integer: equal."""
import ctypes

import numpy as np
import pytest

import oracle


@pytest.fixture(scope="module")
def pk():
    from paged_kv_cache_92_gb300 import build

    build.build()
    import paged_kv_cache_92_gb300 as pk

    pk.load()
    return pk


def walk(tables, old, new, ring, head, count, bs, num_blocks, cap):
    """The step on copies, sequence after sequence: (tables, ring, state, slots, positions,
    starts), or None where it is not possible."""
    have, want = [-(-n // bs) for n in old], [-(-n // bs) for n in new]
    pops = sum(max(w - h, 0) for h, w in zip(have, want))
    pushes = sum(max(h - w, 0) for h, w in zip(have, want))
    tokens = sum(max(n - o, 0) for o, n in zip(old, new))
    if min(old, default=0) < 0 or min(new, default=0) < 0 or tokens > cap \
            or max(have + want, default=0) > tables.shape[1] or pops > count \
            or count + pushes > len(ring):
        return None
    tables, ring, size = tables.copy(), ring.copy(), len(ring)
    fix = lambda e: int(e) if 0 <= e < num_blocks else -1  # noqa: E731
    h, tail = head, head + count
    slots, positions, starts = [], [], []
    for b, (o, n) in enumerate(zip(old, new)):
        starts.append(len(slots))
        for j in range(want[b], have[b]):
            ring[tail % size] = fix(tables[b, j])
            tail += 1
        for j in range(have[b], want[b]):
            tables[b, j] = fix(ring[h % size])
            h += 1
        for t in range(o, n):
            e = fix(tables[b, t // bs])
            slots.append(-1 if e < 0 else e * bs + t % bs)
            positions.append(t)
    starts.append(len(slots))
    pad = [-1] * (cap - len(slots))
    return (tables, ring, np.array([h % size, tail - h, 0, 0], np.int32),
            np.array(slots + pad, np.int64), np.array(positions + pad, np.int32),
            np.array(starts, np.int32))


def layout(old, bs, max_blocks, num_blocks, head, seed, ring_size=None):
    """Tables that hold the old lengths, and a ring of the other blocks from `head` on."""
    order = np.random.default_rng(seed).permutation(num_blocks).astype(np.int32)
    tables = np.full((len(old), max_blocks), -1, np.int32)
    at = 0
    for b, n in enumerate(old):
        k = max(0, min(-(-n // bs), max_blocks))
        tables[b, :k] = order[at:at + k]
        at += k
    size = ring_size or num_blocks
    ring = np.full(size, -7, np.int32)  # what is free, and stale ids elsewhere
    free = order[at:]
    ring[(head + np.arange(len(free))) % size] = free
    return tables, ring, len(free)


def run(pk, tables, old, new, ring, head, count, bs, num_blocks, cap, stream=None, **drop):
    import torch

    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    t, r = dev(tables), dev(ring)
    state = dev(np.array([head, count, 5, 6], np.int32))
    out = torch.full((4,), 9, dtype=torch.int32, device="cuda")
    slots = torch.full((cap,), 77, dtype=torch.int64, device="cuda")
    pos = torch.full((cap,), 77, dtype=torch.int32, device="cuda")
    starts = torch.full((len(old) + 1,), 77, dtype=torch.int32, device="cuda")
    o, n = dev(np.array(old, np.int32)), dev(np.array(new, np.int32))
    outs = dict(slot_mapping=slots, positions=pos, token_starts=starts)
    for k in drop.get("drop", ()):
        outs[k] = None
    torch.cuda.synchronize()
    for _ in range(2):  # the same call again gives the same result
        pk.pa_update_tables(t, o, n, r, state, out, num_blocks, bs, stream=stream, **outs)
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in (t, r, out, slots, pos, starts)]


def check(got, want):
    for name, x, y in zip(("tables", "ring", "state", "slots", "positions", "starts"), got, want):
        assert np.array_equal(x, y), name


# ------------------------------------------------------------------ refusals (CPU)


def _params(pk, **kw):
    p = pk.UpdateTablesParams()
    base = dict(block_tables=4096, old_lens=256, new_lens=512, free_ring=8192, ring_state=768,
                new_ring_state=1024, slot_mapping=16384, positions=32768, token_starts=65536,
                max_blocks_per_seq=4, num_seqs=2, block_size=16, num_blocks=8, ring_size=8,
                max_new_tokens=8)
    base.update(kw)
    for k, v in base.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("kw,status,words", [
    (dict(num_seqs=-1), 1, b"num_seqs"), (dict(num_seqs=65536), 1, b"num_seqs"),
    (dict(max_blocks_per_seq=0), 1, b"positive"), (dict(num_blocks=0), 1, b"positive"),
    (dict(ring_size=0), 1, b"positive"), (dict(max_new_tokens=-1), 1, b"max_new_tokens"),
    (dict(block_size=4), 2, b"block_size"), (dict(block_size=64), 2, b"block_size"),
    (dict(max_blocks_per_seq=1 << 26), 1, b"2^30"), (dict(ring_size=1 << 30), 1, b"2^30"),
    (dict(max_new_tokens=1 << 30), 1, b"2^30"), (dict(block_tables=None), 1, b"NULL"),
    (dict(old_lens=None), 1, b"NULL"), (dict(new_lens=None), 1, b"NULL"),
    (dict(free_ring=None), 1, b"NULL"), (dict(ring_state=None), 1, b"NULL"),
    (dict(new_ring_state=None), 1, b"NULL"),
    (dict(slot_mapping=None, positions=None), 1, b"without slot_mapping"),
    (dict(slot_mapping=16388), 1, b"misaligned"), (dict(positions=32770), 1, b"misaligned"),
    (dict(free_ring=8193), 1, b"misaligned"), (dict(new_ring_state=768), 1, b"overlaps"),
    (dict(new_ring_state=780), 1, b"overlaps"), (dict(token_starts=508), 1, b"overlaps"),
    (dict(slot_mapping=200), 1, b"overlaps"), (dict(positions=516), 1, b"overlaps"),
    (dict(block_tables=256), 1, b"overlaps"), (dict(free_ring=740), 1, b"overlaps")])
def test_refusals(pk, kw, status, words):
    p = _params(pk, **kw)
    assert pk.load().pa_update_tables(ctypes.byref(p), None) == status
    assert words in pk.load().pa_last_error()
    assert pk.load().pa_update_tables(None, None) == 1


def test_binding_refuses_mixed_shapes(pk):
    import torch

    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    good = dict(block_tables=i(2, 4), old_lens=i(2), new_lens=i(2), free_ring=i(8),
                ring_state=i(4), new_ring_state=i(4), num_blocks=8, block_size=16)
    for k, v in dict(block_tables=i(3, 4), new_lens=i(3), free_ring=i(2, 4), ring_state=i(3),
                     new_ring_state=i(5), token_starts=i(2)).items():
        with pytest.raises(ValueError):
            pk.pa_update_tables(**{**good, k: v})
    with pytest.raises(ValueError):  # rows of different counts
        pk.pa_update_tables(**good, slot_mapping=torch.zeros(3, dtype=torch.int64), positions=i(4))
    with pytest.raises(ValueError):  # a host tensor
        pk.pa_update_tables(**good)
    for bad in ([0, 0], [8], [-1]):
        with pytest.raises(ValueError):
            pk.make_free_ring(bad, 8, device="cpu")
    ring, state = pk.make_free_ring([5, 2], 8, device="cpu")
    assert ring.tolist()[:2] == [5, 2] and state.tolist() == [0, 2, 0, 0]


def test_plain_walk_agrees_with_the_pool_model():
    """Growing sequences take the ring's blocks in the order in which the host pool hands
    out its free list."""
    order = np.array([5, 2, 7, 0, 3, 1, 6, 4], np.int32)
    model = oracle.PoolModel(8, 16, free_order=order)
    seqs = [model.seq_create() for _ in range(3)]
    slots = [s for i, n in zip(seqs, (17, 0, 33)) for s in model.append_tokens(i, n)[0]]
    tables = np.full((3, 3), -1, np.int32)
    got = walk(tables, [0, 0, 0], [17, 0, 33], order, 0, 8, 16, 8, 50)
    assert got[3].tolist() == slots
    assert got[0][0, :2].tolist() == model.table(seqs[0]) and got[2].tolist() == [5, 3, 0, 0]


# ------------------------------------------------------------------ GPU


@pytest.mark.gpu
@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("seed,B,hi", [(1, 1, 40), (2, 7, 200), (3, 64, 300), (4, 513, 90),
                                       (5, 1500, 40)])
def test_steps(pk, bs, seed, B, hi):
    """Sequences that begin, end, grow, shrink and stay; rings that wrap around."""
    rng = np.random.default_rng(seed * 100 + bs)
    old = [int(x) for x in rng.integers(0, hi, B)]
    new = [int(rng.choice([0, o, o + 1, rng.integers(0, hi), rng.integers(0, o + 1)]))
           for o in old]
    mb = -(-max(old + new + [1]) // bs) + 1
    need = sum(max(-(-o // bs), -(-n // bs)) for o, n in zip(old, new))
    nb = sum(-(-o // bs) for o in old) + need + 3
    head = int(rng.integers(0, nb))
    tables, ring, count = layout(old, bs, mb, nb, head, seed)
    cap = sum(max(n - o, 0) for o, n in zip(old, new)) + 5
    want = walk(tables, old, new, ring, head, count, bs, nb, cap)
    assert want is not None
    check(run(pk, tables, old, new, ring, head, count, bs, nb, cap), want)
    assert pk.pa_device_errors() == 0


@pytest.mark.gpu
def test_most_sequences(pk):
    """65,535 of them: 128 a thread, and many CTAs."""
    rng = np.random.default_rng(0)
    old = rng.integers(0, 20, 65535).tolist()
    new = [int(n) for n in rng.integers(0, 20, 65535)]
    nb = 65535 * 3 * 2
    tables, ring, count = layout(old, 8, 3, nb, nb - 5, 1)
    cap = sum(max(n - o, 0) for o, n in zip(old, new))
    want = walk(tables, old, new, ring, nb - 5, count, 8, nb, cap)
    check(run(pk, tables, old, new, ring, nb - 5, count, 8, nb, cap), want)
    assert pk.pa_device_errors() == 0


@pytest.mark.gpu
def test_long_prompt_and_exact_fit(pk):
    """One prompt over many CTAs; the ring is emptied, then filled to its last entry."""
    old, new = [0, 3], [100001, 3]
    nb = -(-100001 // 16) + 1
    tables, ring, count = layout(old, 16, nb, nb, 11, 2)
    want = walk(tables, old, new, ring, 11, count, 16, nb, 100001)
    assert want[2].tolist()[1] == 0
    got = run(pk, tables, old, new, ring, 11, count, 16, nb, 100001)
    check(got, want)
    back = walk(want[0], new, [0, 0], want[1], want[2][0], 0, 16, nb, 4)
    check(run(pk, got[0], new, [0, 0], got[1], int(got[2][0]), 0, 16, nb, 4), back)
    assert back[2].tolist()[1] == nb and pk.pa_device_errors() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("old,new,count,cap,size,short,bit", [
    ([5, 20], [40, 20], 1, 99, 8, 1, "POOL"),       # two blocks needed, one free
    ([5, 20], [90, 90], 3, 999, 8, 6, "POOL"),
    ([5, 20], [0, 0], 6, 9, 8, -1, "POOL"),         # no room for three released ones
    ([5, 20], [8, 26], 2, 8, 8, -1, "CONTEXT_LEN"),  # nine tokens, eight rows
    ([5, -1], [8, 3], 2, 99, 8, -1, "CONTEXT_LEN"),
    ([5, 20], [8, -3], 2, 99, 8, -1, "CONTEXT_LEN"),
    ([5, 20], [97, 20], 6, 99, 8, -1, "CONTEXT_LEN"),  # past the table row
    ([5, 20], [2**31 - 1, 20], 6, 99, 8, -1, "CONTEXT_LEN"),
    ([2**31 - 1, 2**31 - 1], [0, 0], 6, 99, 8, -1, "CONTEXT_LEN"),
    ([5, 20], [6, 21], 9, 99, 8, -1, "POOL"),       # a count that the ring cannot have
    ([5, 20], [6, 21], -1, 99, 8, -1, "POOL")])
def test_impossible_steps_change_nothing(pk, old, new, count, cap, size, short, bit):
    tables = np.array([[3, 1, 0, 0, 0, 0], [0, 2, 0, 0, 0, 0]], np.int32)
    ring = np.arange(size, dtype=np.int32) % 8
    got = run(pk, tables, old, new, ring, 3, count, 16, 8, cap)
    check(got, (tables, ring, [3, count, short, 0], np.full(cap, -1), np.full(cap, -1),
                np.zeros(3)))
    assert pk.pa_device_errors() == getattr(pk, "DEVERR_" + bit)


@pytest.mark.gpu
def test_bad_entries_are_passed_on_as_none(pk):
    """Ids outside the pool in the ring and in the tables: never an index."""
    tables = np.array([[3, 99, 5], [-4, 2, 6], [7, 8, 1]], np.int32)
    ring = np.array([40, -3, 4, 0, 0, 0, 0, 0, 0], np.int32)
    old, new = [20, 5, 48], [20, 40, 16]
    want = walk(tables, old, new, ring, 0, 3, 16, 8, 40)
    got = run(pk, tables, old, new, ring, 0, 3, 16, 8, 40)
    check(got, want)
    assert (got[3][:11] == -1).all() and got[1][3:5].tolist() == [-1, 1]
    assert pk.pa_device_errors() == pk.DEVERR_TABLE_ENTRY


@pytest.mark.gpu
@pytest.mark.parametrize("drop", [("slot_mapping",), ("positions",), ("token_starts",),
                                  ("slot_mapping", "positions", "token_starts")])
def test_optional_outputs(pk, drop):
    old, new = [5, 20, 0], [37, 3, 16]
    tables, ring, count = layout(old, 16, 4, 12, 9, 3)
    want = walk(tables, old, new, ring, 9, count, 16, 12, 60)
    got = run(pk, tables, old, new, ring, 9, count, 16, 12, 60, drop=drop)
    names = ("tables", "ring", "state", "slot_mapping", "positions", "token_starts")
    for n, x, y in zip(names, got, want):
        assert np.array_equal(x, y) or (n in drop and (x == 77).all()), n


@pytest.mark.gpu
def test_no_sequences(pk):
    import torch

    z = torch.zeros(0, dtype=torch.int32, device="cuda")
    ring, state = pk.make_free_ring([1, 0], 2)
    out = torch.full((4,), 9, dtype=torch.int32, device="cuda")
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    starts = torch.ones(1, dtype=torch.int32, device="cuda")
    pk.pa_update_tables(torch.zeros(0, 4, dtype=torch.int32, device="cuda"), z, z, ring, state, out,
                        2, 16, slot_mapping=slots, token_starts=starts)
    assert out.tolist() == [0, 2, 0, 0] and slots.tolist() == [-1] * 3 and starts.tolist() == [0]


@pytest.mark.gpu
def test_decode_loop_in_a_graph(pk):
    """A captured step, replayed: lengths and ring states swap places on the device, and
    the tables are those of the walk."""
    import torch

    rng = np.random.default_rng(9)
    B, bs, steps = 70, 16, 40
    lens = rng.integers(1, 50, B).tolist()
    nb = sum(-(-(n + steps) // bs) for n in lens)
    tables, ring, count = layout(lens, bs, 8, nb, 4, 9)
    t, r = torch.from_numpy(tables).cuda(), torch.from_numpy(ring).cuda()
    old = torch.tensor(lens, dtype=torch.int32, device="cuda")
    new, state = torch.empty_like(old), torch.tensor([4, count, 0, 0], dtype=torch.int32, device="cuda")
    nstate = torch.empty_like(state)
    slots = torch.empty(B, dtype=torch.int64, device="cuda")

    def step():
        torch.add(old, 1, out=new)
        pk.pa_update_tables(t, old, new, r, state, nstate, nb, bs, slot_mapping=slots)
        old.copy_(new)
        state.copy_(nstate)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    head = 4
    for _ in range(steps):
        graph.replay()
        torch.cuda.synchronize()
        nxt = [n + 1 for n in lens]
        want = walk(tables, lens, nxt, ring, head, count, bs, nb, B)
        tables, ring, (head, count, _, _) = want[0], want[1], want[2].tolist()
        lens = nxt
        assert np.array_equal(t.cpu().numpy(), tables)
        assert np.array_equal(slots.cpu().numpy(), want[3])
        assert state.tolist() == [head, count, 0, 0]
    assert pk.pa_device_errors() == 0


@pytest.mark.gpu
def test_own_stream(pk):
    import torch

    old, new = [0] * 30, [100] * 30
    tables, ring, count = layout(old, 16, 8, 220, 0, 1)
    want = walk(tables, old, new, ring, 0, count, 16, 220, 3000)
    s = torch.cuda.Stream()
    check(run(pk, tables, old, new, ring, 0, count, 16, 220, 3000, stream=s), want)


@pytest.mark.gpu
def test_release_after_eviction(pk):
    """The kept lengths of an eviction are on the device: the blocks behind them go back
    without a copy to the host, and the next tokens take them."""
    import torch

    rng = np.random.default_rng(4)
    B, bs, budget, nb = 5, 16, 64, 80
    old = [200, 64, 65, 7, 150]
    tables, ring, count = layout(old, bs, 13, nb, 3, 4)
    t, r = torch.from_numpy(tables).cuda(), torch.from_numpy(ring).cuda()
    lens = torch.tensor(old, dtype=torch.int32, device="cuda")
    w = torch.from_numpy(rng.random((B, 208), np.float32)).cuda()
    kc, vc = (torch.randn(nb, 2, bs, 64, device="cuda").bfloat16() for _ in range(2))
    keep, kept = pk.pa_evict_select(w, lens, budget, 8)
    pk.pa_evict_compact(kc, vc, t, t, keep, kept)
    a = torch.tensor([3, count, 0, 0], dtype=torch.int32, device="cuda")
    b, c = torch.empty_like(a), torch.empty_like(a)
    pk.pa_update_tables(t, lens, kept, r, a, b, nb, bs)
    slots = torch.empty(B, dtype=torch.int64, device="cuda")
    pk.pa_update_tables(t, kept, kept + 1, r, b, c, nb, bs, slot_mapping=slots)
    now = [min(n, budget) for n in old]
    one = walk(tables, old, now, ring, 3, count, bs, nb, 0)
    two = walk(one[0], now, [n + 1 for n in now], one[1], *one[2][:2].tolist(), bs, nb, B)
    assert np.array_equal(t.cpu().numpy(), two[0]) and slots.cpu().tolist() == two[3].tolist()
    assert c.tolist() == two[2].tolist() and pk.pa_device_errors() == 0
