"""Block tables made on the GPU and attention over selected blocks, as cases that can be timed
and compared.

Five operators, each in a plain form (elementary torch operations in 32 bits, rounded once) and
through the library's entry points (``own``):

* ``tables``   a step's new lengths turned into block tables, slots and positions: fresh blocks
               taken from the head of a ring of free ones, released blocks put at its tail;
* ``bounds``   the least and the largest key of a block, element by element;
* ``scores``   an upper bound of the attention score that any key of a block can reach;
* ``select``   the blocks to attend to under a budget: the first, the last, the best of the rest;
* ``attend``   attention of one or several new tokens over the selected blocks alone.

Caches are bf16, 8-bit (E4M3, V in sub-tiles of transposed rows) or 4-bit (E2M1 codes, then an
E4M3 scale per 16 elements, in every (block, KV head) tile); the latter two have a scale per head.
"""
import math
import random

import torch

own = False

KV_BYTES = {"bf16": 2.0, "fp8": 1.0, "fp4": 9.0 / 16.0}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _case(name, op, batch, hq, hkv, dim, bs, lo, hi, kv="bf16", q=1, budget=0, sink=0, recent=0,
          new=1, turnover=0.0):
    """``new``: tokens that a sequence gains, at most (0: all of its tokens are new);
    ``turnover``: the share of sequences that end, and of those that begin, in the step."""
    c = dict(op=op, batch=batch, hq=hq, hkv=hkv, dim=dim, bs=bs, lo=lo, hi=hi, kv=kv, q=q,
             budget=budget, sink=sink, recent=recent, new=new, turnover=turnover)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decode step of 64 sequences: one new token each, now and then a fresh block: latency
        _case("tables_step_b64", "tables", 64, 32, 8, 128, 16, 128, 2047),
        # a scheduler's step with prompts: of 256 sequences a quarter ends and a quarter begins
        _case("tables_prompts_b256", "tables", 256, 32, 8, 128, 16, 1, 4095, turnover=0.25, new=3),
        # the last blocks' bounds after one decode step of an 8B-class layer: latency
        _case("bounds_step_b64", "bounds", 64, 32, 8, 128, 16, 128, 2047),
        # bounds of long prompts after their prefill, odd lengths
        _case("bounds_prompts_b16", "bounds", 16, 32, 8, 128, 16, 8191, 32767, new=0),
        # the same for the 4-bit cache, larger blocks, after an eviction has moved everything
        _case("bounds_fp4_b32", "bounds", 32, 32, 8, 128, 32, 4097, 16383, kv="fp4", new=0),
        # scores of an 8B-class layer's decode batch over long contexts
        _case("scores_8b_b64", "scores", 64, 32, 8, 128, 16, 8192, 32768),
        # two very long contexts with four new tokens each (verification of a draft), 8-bit cache
        _case("scores_long_q4", "scores", 2, 64, 8, 128, 16, 65537, 131072, kv="fp8", q=4),
        # the choice for that batch: 2,048 tokens of each context
        _case("select_8b_b64", "select", 64, 32, 8, 128, 16, 8192, 32768, budget=128, sink=1,
              recent=4),
        # the choice for a few very long contexts in small blocks
        _case("select_long_b4", "select", 4, 64, 8, 128, 8, 65537, 131072, budget=512, sink=1,
              recent=8),
        # attention of the 8B-class batch over 128 blocks of each context
        _case("attend_8b_b64", "attend", 64, 32, 8, 128, 16, 8192, 32768, budget=128, sink=1,
              recent=4),
        # 70B-class layer, very long contexts in 8 bits, 256 blocks of each
        _case("attend_70b_fp8_b32", "attend", 32, 64, 8, 128, 16, 32768, 131072, kv="fp8",
              budget=256, sink=1, recent=4),
        # one sequence, two new tokens, 4-bit cache of head dim 64: latency
        _case("attend_one_fp4_q2", "attend", 1, 32, 8, 64, 16, 20001, 20001, kv="fp4", q=2,
              budget=64, sink=1, recent=3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "bounds", "scores", "select", "attend", "attend"])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 8])
    dim, bs = rng.choice([64, 128]), rng.choice([8, 16, 32])
    kv = rng.choice(["bf16", "fp8", "fp4"])
    if op == "tables":
        hi = _log(rng, 2, 16384)
        batch = max(1, min(_log(rng, 1, 1024), 400000 // hi))
        return _case(None, op, batch, hq, hkv, dim, bs, rng.randint(1, hi), hi,
                     new=_log(rng, 1, 64), turnover=rng.choice([0.0, 0.1, 0.4]))
    hi = _log(rng, 4, 131072)
    batch = max(1, min(_log(rng, 1, 256), 300000 // hi))
    lo = rng.randint(4, hi)
    q = rng.randint(1, 4) if op in ("scores", "attend") else 1
    budget = min(_log(rng, 1, 512), max(1, 32768 // batch // bs))
    sink = rng.randint(0, min(2, budget))
    return _case(None, op, batch, hq, hkv, dim, bs, lo, hi, kv=kv, q=q, budget=budget, sink=sink,
                 recent=rng.randint(0, min(4, budget - sink)), new=rng.choice([0, 1, 5]))


def _lens(c):
    """(lengths before, lengths after) of the step, from the case's sizes alone."""
    r = random.Random("%(op)s %(batch)d %(bs)d %(lo)d %(hi)d %(new)d %(turnover).2f" % c)
    old, new = [], []
    for _ in range(c["batch"]):
        n, kind = r.randint(c["lo"], c["hi"]), r.random()
        gain = min(r.randint(1, max(1, c["new"])), n) if c["new"] else n
        if kind < c["turnover"]:  # ends
            n, gain = 0, -n
        elif kind < 2 * c["turnover"]:  # begins
            gain = n
        old.append(n - gain)
        new.append(n)
    return old, new


def work(c):
    old, new = _lens(c)
    bs, hkv, dim, b, q = c["bs"], c["hkv"], c["dim"], c["batch"], c["q"]
    have, want = [-(-n // bs) for n in old], [-(-n // bs) for n in new]
    blocks = sum(want)
    if c["op"] == "tables":
        moved = sum(abs(w - h) for h, w in zip(have, want))
        tokens = sum(max(n - o, 0) for o, n in zip(old, new))
        return {"bytes": 8 * b + 8 * moved + 12 * tokens + 4 * (b + 1), "flops": 0}
    if c["op"] == "bounds":
        first = [o // bs for o in old]
        rows = sum(n - f * bs for f, n in zip(first, new))
        units = sum(w - f for f, w in zip(first, want))
        return {"bytes": rows * hkv * dim * KV_BYTES[c["kv"]] + units * (hkv * dim * 4 + 4) + 8 * b,
                "flops": 2 * rows * hkv * dim}
    if c["op"] == "scores":
        return {"bytes": blocks * (hkv * (4 * dim + 4) + 4) + 2 * b * q * c["hq"] * dim,
                "flops": 4 * dim * c["hq"] * q * blocks}
    if c["op"] == "select":
        return {"bytes": 4 * hkv * (blocks + b * c["budget"]) + 4 * b, "flops": 0}
    taken = sum(min(w, c["budget"]) for w in want)
    return {"bytes": taken * hkv * (2 * bs * dim * KV_BYTES[c["kv"]] + 8) + 4 * b * q * c["hq"] * dim,
            "flops": 4 * taken * bs * c["hq"] * dim * q}


# ---------------------------------------------------------------- inputs


def _spread(dim, dev, wide):
    """Keys and values of real layers have a few large channels."""
    s = torch.ones(dim, device=dev)
    s[5::16] = wide
    return s


def _pack4(x, s, nb, hkv, bs, dim):
    """Rows [nb, hkv, bs, dim] in float32 as 4-bit tiles: nearest codes under the group scale."""
    g = (x / s.view(-1, 1, 1)).unflatten(-1, (-1, 16))
    sf = (g.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    a = g.abs() / sf.float().clamp(min=2.0 ** -9).unsqueeze(-1)
    edges = torch.tensor([(E2M1[i] + E2M1[i + 1]) / 2 for i in range(7)], device=x.device)
    code = torch.bucketize(a, edges).to(torch.uint8) | (torch.signbit(g).to(torch.uint8) << 3)
    code = code.flatten(-2).unflatten(-1, (-1, 2))
    code = (code[..., 0] | (code[..., 1] << 4)).reshape(nb, hkv, -1)
    return torch.cat([code, sf.view(torch.uint8).reshape(nb, hkv, -1)], -1).view(nb, hkv, bs, -1)


def _cache(c, nb, s, which, g, dev):
    """One cache of nb blocks in the case's type."""
    hkv, bs, dim = c["hkv"], c["bs"], c["dim"]
    wide = _spread(dim, dev, 3.0)
    out = []
    per = max(1, (1 << 26) // (bs * hkv * dim))
    for at in range(0, nb, per):
        n = min(per, nb - at)
        x = torch.randn((n, hkv, bs, dim), generator=g, device=dev) * wide
        if c["kv"] == "bf16":
            x = x.to(torch.bfloat16)
        elif c["kv"] == "fp8":
            x = (x / s.view(-1, 1, 1)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            if which == "v":
                w = min(bs, 16)
                x = x.view(n, hkv, bs // w, w, dim).transpose(-1, -2).contiguous()
        else:
            x = _pack4(x, s, n, hkv, bs, dim)
        out.append(x)
    return torch.cat(out)


def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    old, new = _lens(c)
    op, b, hq, hkv, dim, bs, q = (c[k] for k in ("op", "batch", "hq", "hkv", "dim", "bs", "q"))
    most = max(1, max(-(-n // bs) for n in old + new))
    s = dict(c, most=most, hi_len=max(new + [1]), scale=1.0 / math.sqrt(dim),
             old=torch.tensor(old, dtype=torch.int32, device=dev),
             lens=torch.tensor(new, dtype=torch.int32, device=dev))
    if own:
        import paged_kv_cache_92_gb300 as pk
        pk.load()
        s["pk"] = pk
    # every sequence's blocks, scattered over a pool that is four fifths full
    held = old if op == "tables" else new
    count = torch.tensor([-(-n // bs) for n in held], device=dev)
    used = int(count.sum())
    fresh = sum(max(-(-n // bs) + -(-o // bs) * -1, 0) for o, n in zip(old, new))
    nb = max(used + fresh, int(math.ceil(1.25 * used))) + 3
    order = torch.randperm(nb, generator=g, device=dev).to(torch.int32)
    j = torch.arange(most, device=dev).view(1, -1)
    first = (torch.cumsum(count, 0) - count).view(-1, 1)
    at = (first + j).clamp(max=nb - 1)
    s["tables"] = torch.where(j < count.view(-1, 1), order[at], torch.full_like(order[at], -1))
    s["nb"] = nb
    if op == "tables":
        head = int(torch.randint(0, nb, (1,), generator=g, device=dev))
        s["ring"] = torch.roll(torch.roll(order, -used), head)
        s["state"] = torch.tensor([head, nb - used, 0, 0], dtype=torch.int32, device=dev)
        cap = sum(max(n - o, 0) for o, n in zip(old, new)) + b // 4  # a padded batch
        s["new_state"] = torch.zeros_like(s["state"])
        s["slots"] = torch.zeros(max(cap, 1), dtype=torch.int64, device=dev)
        s["positions"] = torch.zeros(max(cap, 1), dtype=torch.int32, device=dev)
        s["starts"] = torch.zeros(b + 1, dtype=torch.int32, device=dev)
        return s
    coded = c["kv"] != "bf16"
    s["ks"], s["vs"] = (base * torch.exp(torch.rand(hkv, generator=g, device=dev) - 0.5)
                        if coded else None for base in (0.05, 0.03))
    if op in ("scores", "attend"):
        shape = (b, q, hq, dim) if q > 1 else (b, hq, dim)
        s["q_rows"] = torch.randn(shape, generator=g, device=dev).to(torch.bfloat16)
    if op in ("bounds", "attend"):
        s["k_cache"] = _cache(c, nb, s["ks"], "k", g, dev)
    if op in ("bounds", "scores"):
        # what lies there from earlier steps: about what blocks of normal keys have
        mid = torch.randn((nb, hkv, 2, dim), generator=g, device=dev)
        mid = torch.stack([mid.amin(2) - 1.0, mid.amax(2) + 1.0], 2) * _spread(dim, dev, 3.0)
        s["bounds"] = (mid / (s["ks"].view(-1, 1, 1) if coded else 1.0)).to(torch.bfloat16)
    if op in ("scores", "select"):
        # what lies there from the step before; as many distinct values as scores have
        s["scores"] = 8.0 + 3.0 * torch.randn((b, hkv, most + 3), generator=g, device=dev)
    if op == "select":
        s["selected"] = torch.zeros((b, hkv, c["budget"]), dtype=torch.int32, device=dev)
    if op == "attend":
        s["v_cache"] = _cache(c, nb, s["vs"], "v", g, dev)
        s["selected"] = _plain_select(torch.rand((b, hkv, most), generator=g, device=dev), s["lens"],
                                      bs, c["budget"], c["sink"], c["recent"])
        s["out"] = torch.empty_like(s["q_rows"])
        if own:
            n = pk.pa_decode_selected_workspace_size(
                s["q_rows"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["hi_len"],
                s["selected"], k_scale=s["ks"], v_scale=s["vs"])
            s["workspace"] = torch.empty(max(n, 256), dtype=torch.uint8, device=dev)
    return s


# ---------------------------------------------------------------- plain forms


def _plain_tables(s):
    bs, ring, size = s["bs"], s["ring"], s["ring"].numel()
    tables, dev = s["tables"], s["ring"].device
    old, new = s["old"].long().view(-1, 1), s["lens"].long().view(-1, 1)
    have, want = (old + bs - 1) // bs, (new + bs - 1) // bs
    pop, push, gain = (want - have).clamp(min=0), (have - want).clamp(min=0), (new - old).clamp(min=0)
    head, count = s["state"][0].long(), s["state"][1].long()
    j = torch.arange(tables.shape[1], device=dev).view(1, -1)
    src = (head + torch.cumsum(pop, 0) - pop + j - have) % size
    dst = (head + count + torch.cumsum(push, 0) - push + j - want) % size
    gone = (j >= want) & (j < have)
    taken = ring[src]
    ring[dst[gone]] = tables[gone]
    tables.copy_(torch.where((j >= have) & (j < want), taken, tables))
    popped, pushed = pop.sum(), push.sum()
    zero = torch.zeros_like(head)
    s["new_state"].copy_(torch.stack([(head + popped) % size, count - popped + pushed, zero, zero]))
    ends = torch.cumsum(gain.flatten(), 0)
    s["starts"][0].zero_()
    s["starts"][1:].copy_(ends)
    i = torch.arange(s["slots"].numel(), device=dev)
    b = torch.searchsorted(ends, i, right=True).clamp(max=tables.shape[0] - 1)
    pos = (old.flatten()[b] + i - (ends - gain.flatten())[b]).clamp(min=0)
    slot = tables[b, (pos // bs).clamp(max=tables.shape[1] - 1)].long() * bs + pos % bs
    real = i < ends[-1]
    s["slots"].copy_(torch.where(real, slot, torch.full_like(slot, -1)))
    s["positions"].copy_(torch.where(real, pos, torch.full_like(pos, -1)))
    return tables, ring, s["new_state"], s["slots"], s["positions"], s["starts"]


def _codes(tiles, kv, which, bs, dim):
    """Tiles [..., bs, row] of K or V -> float32 rows [..., bs, dim], head scale left out."""
    if kv == "bf16":
        return tiles.float()
    if kv == "fp8":
        x = tiles.view(torch.float8_e4m3fn).float()
        return x.transpose(-1, -2).flatten(-3, -2) if which == "v" else x
    codes, f = tiles.flatten(-2).split([bs * dim // 2, bs * dim // 16], -1)
    codes = codes.unflatten(-1, (bs, dim // 2))
    f = f.contiguous().view(torch.float8_e4m3fn).float().unflatten(-1, (bs, dim // 16, 1))
    v = torch.tensor(E2M1, device=tiles.device)
    v = torch.cat([v, -v])[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()]
    return (v.unflatten(-1, (-1, 16)) * f).flatten(-2)


def _plain_bounds(s):
    bs, dim, tables = s["bs"], s["dim"], s["tables"]
    old, new = s["old"].long().view(-1, 1), s["lens"].long().view(-1, 1)
    j = torch.arange(tables.shape[1], device=tables.device).view(1, -1)
    b, at = ((j >= old // bs) & (j * bs < new)).nonzero(as_tuple=True)
    block = tables[b, at].long()
    x = _codes(s["k_cache"][block], s["kv"], "k", bs, dim)  # [blocks, heads, bs, dim]
    t = at.view(-1, 1) * bs + torch.arange(bs, device=tables.device)
    inside = (t < new.flatten()[b].view(-1, 1)).view(-1, 1, bs, 1)
    lo = torch.where(inside, x, torch.full_like(x, math.inf)).amin(2)
    hi = torch.where(inside, x, torch.full_like(x, -math.inf)).amax(2)
    s["bounds"][block] = torch.stack([lo, hi], 2).to(torch.bfloat16)
    return s["bounds"]


def _plain_scores(s):
    b, q, hq, hkv, dim, bs = (s[k] for k in ("batch", "q", "hq", "hkv", "dim", "bs"))
    dev = s["bounds"].device
    most = s["tables"].shape[1]
    x = s["bounds"][s["tables"].clamp(min=0).long()].float().transpose(1, 2)  # [b, hkv, most, 2, dim]
    rows = s["q_rows"].float().view(b, q, hkv, hq // hkv, dim).permute(0, 2, 1, 3, 4).flatten(2, 3)
    f = torch.full((hkv, 1, 1), s["scale"], device=dev)
    if s["ks"] is not None:
        f = f * s["ks"].view(-1, 1, 1)
    up, down = rows.clamp(min=0), rows.clamp(max=0)
    # (a negative factor turns the bound around)
    up, down = torch.where(f > 0, up, down), torch.where(f > 0, down, up)
    bound = up @ x[:, :, :, 1].transpose(-1, -2) + down @ x[:, :, :, 0].transpose(-1, -2)
    bound = bound * f
    bound = torch.where(bound.isnan(), torch.full_like(bound, math.inf), bound)
    j = torch.arange(most, device=dev)
    last = s["lens"].long().view(-1, 1, 1) - q + torch.arange(q, device=dev).view(1, -1, 1)
    seen = (j * bs <= last).repeat_interleave(hq // hkv, 1).unsqueeze(1)
    bound = torch.where(seen, bound, torch.full_like(bound, -math.inf)).amax(2)
    part = s["scores"][:, :, :most]
    inside = (j * bs < s["lens"].view(-1, 1)).unsqueeze(1)
    part.copy_(torch.where(inside, bound, part))
    return s["scores"]


def _plain_select(scores, lens, bs, budget, sink, recent):
    n = ((lens.long() + bs - 1) // bs).view(-1, 1, 1)
    j = torch.arange(scores.shape[2], device=scores.device).view(1, 1, -1)
    key = torch.where(scores.isnan() | (j >= n), torch.full_like(scores, -math.inf), scores)
    order = torch.sort(key, dim=2, descending=True, stable=True)[1]
    # what always stays comes first, what is not a number behind the numbers, the padding last
    rank = torch.where((j < sink) | (j >= n - recent), 0, torch.where(scores.isnan(), 2, 1))
    rank = torch.where(j < n, rank, 3).expand_as(scores).gather(2, order)
    order = order.gather(2, torch.sort(rank, dim=2, stable=True)[1])
    room = min(budget, scores.shape[2])
    kept = torch.where(j[..., :room] < n, order[..., :room], torch.full_like(order[..., :room], 1 << 30))
    kept = torch.sort(kept, dim=2)[0]
    out = torch.full(scores.shape[:2] + (budget,), -1, dtype=torch.int32, device=scores.device)
    out[..., :room] = torch.where(kept < (1 << 30), kept, torch.full_like(kept, -1)).int()
    return out


def _plain_attend(s):
    b, q, hq, hkv, dim, bs = (s[k] for k in ("batch", "q", "hq", "hkv", "dim", "bs"))
    sel, dev = s["selected"].long(), s["selected"].device
    block = s["tables"].gather(1, sel.clamp(min=0).flatten(1)).long().view_as(sel)
    head = torch.arange(hkv, device=dev).view(1, -1, 1)
    k = _codes(s["k_cache"][block, head], s["kv"], "k", bs, dim).flatten(2, 3)
    rows = s["q_rows"].float().view(b, q, hkv, hq // hkv, dim).permute(0, 2, 3, 1, 4).flatten(2, 3)
    if s["ks"] is not None:
        k = k * s["ks"].view(-1, 1, 1)
    sc = (rows * s["scale"]) @ k.transpose(-1, -2)
    t = (sel.unsqueeze(-1) * bs + torch.arange(bs, device=dev)).flatten(2)
    t = torch.where((sel >= 0).repeat_interleave(bs, 2), t, torch.full_like(t, 1 << 40))
    last = s["lens"].long().view(-1, 1) - q + torch.arange(q, device=dev)
    seen = t.unsqueeze(2) <= last.repeat(1, hq // hkv).view(b, 1, -1, 1)
    sc = torch.where(seen, sc, torch.full_like(sc, -math.inf))
    p = torch.exp(sc - sc.amax(-1, keepdim=True).clamp(min=-1e30))
    v = _codes(s["v_cache"][block, head], s["kv"], "v", bs, dim).flatten(2, 3)
    if s["vs"] is not None:
        v = v * s["vs"].view(-1, 1, 1)
    v = torch.where((t < s["lens"].view(-1, 1, 1)).unsqueeze(-1), v, torch.zeros_like(v))
    o = (p @ v) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = o.unflatten(2, (-1, q)).permute(0, 3, 1, 2, 4)
    return o.reshape(s["q_rows"].shape).to(torch.bfloat16)


def run(s):
    op = s["op"]
    if own:
        pk = s["pk"]
        if op == "tables":
            pk.pa_update_tables(s["tables"], s["old"], s["lens"], s["ring"], s["state"],
                                s["new_state"], s["nb"], s["bs"], slot_mapping=s["slots"],
                                positions=s["positions"], token_starts=s["starts"])
            return s["tables"], s["ring"], s["new_state"], s["slots"], s["positions"], s["starts"]
        if op == "bounds":
            return pk.pa_block_bounds(s["k_cache"], s["bounds"], s["tables"], s["lens"],
                                      s["new"] or s["hi_len"], old_lens=s["old"])
        if op == "scores":
            return pk.pa_block_scores(s["q_rows"], s["bounds"], s["tables"], s["lens"],
                                      s["hi_len"], s["bs"], scores=s["scores"], scale=s["scale"],
                                      k_scale=s["ks"])
        if op == "select":
            return pk.pa_block_select(s["scores"], s["lens"], s["bs"], s["budget"], s["sink"],
                                      s["recent"], selected=s["selected"])
        return pk.pa_decode_selected(s["q_rows"], s["k_cache"], s["v_cache"], s["tables"],
                                     s["lens"], s["hi_len"], s["selected"], s["scale"],
                                     out=s["out"], workspace=s["workspace"], k_scale=s["ks"],
                                     v_scale=s["vs"])
    if op == "tables":
        return _plain_tables(s)
    if op == "bounds":
        return _plain_bounds(s)
    if op == "scores":
        return _plain_scores(s)
    if op == "select":
        return _plain_select(s["scores"], s["lens"], s["bs"], s["budget"], s["sink"], s["recent"])
    return _plain_attend(s)


# ---------------------------------------------------------------- 64 bits


def _exact_rows(s, which, blocks, h):
    """The rows of some blocks and one KV head in 64 bits, block by block, with the head's scale."""
    bs, dim, n = s["bs"], s["dim"], len(blocks)
    x = s[which + "_cache"][blocks, h]
    if s["kv"] == "bf16":
        return x.double().reshape(n * bs, dim)
    sc = s["ks" if which == "k" else "vs"][h].double()
    if s["kv"] == "fp8":
        x = x.view(torch.float8_e4m3fn).double()
        if which == "v":
            x = torch.einsum("nsdw->nswd", x)
        return x.reshape(n * bs, dim) * sc
    raw = x.reshape(n, -1)
    nib = raw[:, : bs * dim // 2].reshape(-1, 1)
    nib = torch.cat([nib % 16, torch.div(nib, 16, rounding_mode="floor")], 1).long().flatten()
    ex, man = torch.div(nib % 8, 2, rounding_mode="floor"), (nib % 2).double()
    val = torch.where(ex == 0, man / 2, (1 + man / 2) * torch.pow(2.0, (ex - 1).double()))
    val = torch.where(nib >= 8, -val, val).reshape(n * bs, dim // 16, 16)
    f = raw[:, bs * dim // 2:].contiguous().view(torch.float8_e4m3fn).double()
    return (val * f.reshape(n * bs, dim // 16, 1)).reshape(n * bs, dim) * sc


def exact(c, seed):
    s = prepare(c, seed)
    op, dev, bs = c["op"], torch.device("cuda"), c["bs"]
    old, new = _lens(c)
    if op == "tables":
        tables, ring = s["tables"].tolist(), s["ring"].tolist()
        head, free = s["state"].tolist()[:2]
        size, tail = len(ring), head + free
        slots, positions, starts = [], [], [0]
        for row, was, now in zip(tables, old, new):
            for j in range(-(-now // bs), -(-was // bs)):
                ring[tail % size], tail = row[j], tail + 1
            for j in range(-(-was // bs), -(-now // bs)):
                row[j], head = ring[head % size], head + 1
            for t in range(was, now):
                slots.append(row[t // bs] * bs + t % bs)
                positions.append(t)
            starts.append(len(slots))
        pad = [-1] * (s["slots"].numel() - len(slots))
        return (torch.tensor(tables, dtype=torch.int32, device=dev),
                torch.tensor(ring, dtype=torch.int32, device=dev),
                torch.tensor([head % size, tail - head, 0, 0], dtype=torch.int32, device=dev),
                torch.tensor(slots + pad, dtype=torch.int64, device=dev),
                torch.tensor(positions + pad, dtype=torch.int32, device=dev),
                torch.tensor(starts, dtype=torch.int32, device=dev))
    b, hkv, hq, dim, q = c["batch"], c["hkv"], c["hq"], c["dim"], c["q"]
    if b * hkv > 4096:
        return None
    if op == "select":
        rows = s["scores"].tolist()
        out = []
        for row, n in zip(rows, new):
            n = -(-n // bs)
            for w in row:
                stay = [j for j in range(n) if j < c["sink"] or j >= n - c["recent"]]
                rest = sorted(range(c["sink"], max(c["sink"], n - c["recent"])),
                              key=lambda j: (-w[j], j))
                got = sorted((stay + rest)[: c["budget"]])
                out.append(got + [-1] * (c["budget"] - len(got)))
        return torch.tensor(out, dtype=torch.int32, device=dev).view(b, hkv, c["budget"])
    if op == "bounds":
        s["ks"] = torch.ones(hkv, device=dev)  # bounds leave the head's scale out
        out = s["bounds"].double()
        for i in range(b):
            j0, j1 = old[i] // bs, -(-new[i] // bs)
            if j0 >= j1:
                continue
            at = s["tables"][i, j0:j1].long()
            for h in range(hkv):
                x = _exact_rows(s, "k", at, h).reshape(-1, bs, dim)
                tail = x[-1:, : new[i] - (j1 - 1) * bs]
                lo = torch.cat([x[:-1].min(1)[0], tail.min(1)[0]])
                hi = torch.cat([x[:-1].max(1)[0], tail.max(1)[0]])
                out[at, h, 0], out[at, h, 1] = lo, hi
        return out
    rows = s["q_rows"].double().reshape(b, q, hkv, hq // hkv, dim)
    if op == "scores":
        out = s["scores"].double()
        for i in range(b):
            n = -(-new[i] // bs)
            x = s["bounds"][s["tables"][i, :n].long()].double()  # [n, hkv, 2, dim]
            for h in range(hkv):
                f = s["scale"] * (1.0 if s["ks"] is None else float(s["ks"][h]))
                best = torch.full((n,), -math.inf, dtype=torch.float64, device=dev)
                for k in range(q):
                    seen = (new[i] - q + k) // bs + 1
                    for r in rows[i, k, h]:
                        ends = torch.maximum(f * r * x[:seen, h, 0], f * r * x[:seen, h, 1]).sum(1)
                        best[:seen] = torch.maximum(best[:seen], ends)
                out[i, h, :n] = best
        return out
    out = torch.zeros_like(rows)
    chosen = s["selected"].tolist()
    for i in range(b):
        for h in range(hkv):
            at = [j for j in chosen[i][h] if j >= 0]
            blocks = s["tables"][i, at].long()
            k, v = (_exact_rows(s, w, blocks, h) for w in "kv")
            t = (torch.tensor(at, device=dev).view(-1, 1) * bs + torch.arange(bs, device=dev)).flatten()
            for n in range(q):
                on = t <= new[i] - q + n
                if bool(on.any()):
                    p = torch.softmax(rows[i, n, h] @ k[on].T * s["scale"], -1)
                    out[i, n, h] = p @ v[on]
    return out.reshape(s["q_rows"].shape)
