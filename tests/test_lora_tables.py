"""How the adapters' gradient cuts row tables into items and slots
(csrc/lora.hip), followed on the CPU: every row of a well-formed table is in one
item, and no table at all, however malformed, leads outside rows or slots."""
import random

CUS = 256


def plan(rows, E, r, K, N):
    passes = -(-r // 64)
    slabs = (-(-K // 128) + -(-N // 128)) * passes
    wanted = max(1, 2 * CUS // slabs)
    chunk = max(256, -(-(-(-rows // wanted)) // 128) * 128)
    items = rows // chunk + E
    return chunk, items, min(2 * rows // chunk, items)


def adapters(offsets, E, rows, chunk):
    """(rows from, to, items) of every adapter"""
    for e in range(E):
        lo = min(max(offsets[e], 0), rows)
        hi = max(min(max(offsets[e + 1], 0), rows), lo)
        lo, hi = lo & ~31, hi & ~31
        yield lo, hi, -(-(hi - lo) // chunk) if hi > lo else 1


def walk(offsets, E, rows, chunk, items, slots):
    """What the launched blocks do: (adapter, row0, row1, slot) of each, and the slots that the joining blocks read."""
    found, read = [], []
    item = slot = many = 0
    for e, (lo, hi, m) in enumerate(adapters(offsets, E, rows, chunk)):
        for part in range(m):
            if item + part < items:
                s = slot + part if m > 1 else -1
                if s < slots:
                    found.append((e, lo + part * chunk, min(hi, lo + (part + 1) * chunk), s))
        if m > 1:
            if slot < slots and many < min(E, slots // 2):
                read.append((e, [slot] + [slot + n for n in range(1, m) if slot + n < slots]))
            slot += m
            many += 1
        item += m
    return found, read


def _well_formed(rng, E, rows):
    blocks = rows // 32
    cuts = sorted(rng.randint(0, blocks) for _ in range(E))
    if rng.random() < 0.3:
        cuts = sorted(rng.choice(cuts) for _ in range(E))
    return [0 if rng.random() < 0.5 else cuts[0] * 32] + [c * 32 for c in cuts]


def test_well_formed_tables():
    rng = random.Random(1)
    split = 0
    for _ in range(3000):
        E, rows = rng.randint(1, 70), 32 * rng.randint(0, 300)
        r, K, N = 8 * rng.randint(1, 16), 8 * rng.randint(1, 800), 8 * rng.randint(1, 800)
        chunk, items, slots = plan(rows, E, r, K, N)
        off = _well_formed(rng, E, rows)
        found, read = walk(off, E, rows, chunk, items, slots)
        seen, used = set(), {}
        for e, row0, row1, slot in found:
            for block in range(row0, row1, 32):
                assert off[e] <= block < off[e + 1] and block not in seen
                seen.add(block)
            if slot >= 0:
                assert slot not in used and slot < slots
                used[slot] = e
        assert seen == set(range(off[0], off[E], 32))
        assert {e for e, _, _, _ in found} == set(range(E))                 # the others' zeros too
        assert sorted(s for _, ss in read for s in ss) == sorted(used) and all(used[s] == e for e, ss in read for s in ss)
        split += len(read)
    assert split > 300


def test_malformed_tables():
    rng = random.Random(2)
    for _ in range(5000):
        E, rows = rng.randint(1, 40), 32 * rng.randint(0, 200)
        chunk, items, slots = plan(rows, E, 8, 64 * rng.randint(1, 60), 64)
        off = [rng.choice([0, rows, -5, 1 << 30, -(1 << 31), rng.randint(-40, rows + 40)]) for _ in range(E + 1)]
        found, read = walk(off, E, rows, chunk, items, slots)
        for e, row0, row1, slot in found:
            assert 0 <= row0 <= row1 <= rows or row0 >= row1
            assert row0 >= row1 or (row0 % 32 == 0 and row1 % 32 == 0)
            assert -1 <= slot < max(slots, 0) or slot == -1
        for e, ss in read:
            assert all(0 <= s < slots for s in ss)
