"""The barriers of the tensor-core tree attention, run as a model with random delays.

The model has the kernel's warps (two that copy, those that widen or look through tiles, two
that issue products, two softmaxes), its barriers (counts, transactions, waits by parity, which
an older phase of the same parity passes too) and its rings.  Ring sizes, groups and how long
descriptions are kept are read from the kernel's source.  Every part checks that what it reads
is the tile that it means: a wait that passes a phase early, a copy into a slot in use or a
description that is overwritten shows as another tile's number.
"""
import os
import random
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
with open(os.path.join(ROOT, "streaming_sinkhorn_solver_gb300", "csrc", "fs_tree_tc.cu")) as _f:
    SOURCE = _f.read()
MODES = {"ROWS": 0, "KEYS": 1, "HALF": 2}


def constants(hd, eight, mode):
    """kRing, kRaw, kGroups, kScales and kBits of a kernel, from its source's expressions."""
    names = {"HD": hd, "Q8": eight, "MODE": MODES[mode], "kAlternate": mode != "ROWS", **MODES}

    def value(text):
        """A C expression of these names: a ? b : c, and what python has alike."""
        while "(" in text:
            inner = re.search(r"\(([^()]*)\)", text)
            text = text[:inner.start()] + str(value(inner[1])) + text[inner.end():]
        if "?" in text:
            cond, rest = text.split("?", 1)
            depth = 1
            for at, ch in enumerate(rest):
                depth += {"?": 1, ":": -1}.get(ch, 0)
                if depth == 0:
                    return value(rest[:at]) if value(cond) else value(rest[at + 1:])
        text = re.sub(r"!(?!=)", " not ", text).replace("&&", " and ").replace("||", " or ")
        return int(eval(text.strip().replace("/", "//"), {}, names))

    for name in ("kFitWarps", "kGroups", "kRing", "kRaw", "kScales", "kBits"):
        expr = re.search(rf"static constexpr int [^;]*?\b{name} = ([^;,]+)[;,]", SOURCE)[1]
        names[name] = value(expr)
    return {k: names[k] for k in ("kGroups", "kRing", "kRaw", "kScales", "kBits")}


def own_barriers():
    """Whether the softmax waits for looked-through values at a barrier of the tile's own."""
    waits = re.findall(r"warp_wait\(([^;]*?)ERR_TIMEOUT_EPILOGUE", SOURCE)
    return not any("ready" in w for w in waits) and any("looked[tile - mixed_from], 0" in w for w in waits)


class Bar:
    def __init__(self, count):
        self.count = self.pending = count
        self.bytes = self.phase = 0

    def _turn(self):
        if self.pending == 0 and self.bytes == 0:
            self.phase += 1
            self.pending = self.count

    def arrive(self, expect=0):
        assert self.pending > 0, "an arrival too many"
        self.bytes += expect
        self.pending -= 1
        self._turn()

    def land(self, n):
        self.bytes -= n
        assert self.bytes >= 0 or self.pending > 0, "bytes too many"
        self._turn()

    def passed(self, parity):
        return (self.phase & 1) != parity


def run(c, eight, mode, nt, mixed_from, seed, two=True, own=True, slow=None):
    """What went wrong, a list; `slow`: a part that is held back for most of the time."""
    rnd = random.Random(seed)
    alternate = mode != "ROWS"
    ring, raws, groups = c["kRing"], c["kRaw"], c["kGroups"]
    both = not alternate and two
    bars = {n: [[Bar(k) for _ in range(16)] for _ in range(2)]
            for n, k in (("full", 1), ("free", 2), ("ready", 2), ("empty", 2 if both else 1))}
    full, free, ready, empty = (bars[n] for n in ("full", "free", "ready", "empty"))
    last, looked = [Bar(1) for _ in range(8)], [Bar(2) for _ in range(8)]
    sfull, sfree = [Bar(1), Bar(1)], [Bar(1), Bar(1)]
    pfull, pfree = ([[Bar(1), Bar(1)] for _ in range(2)] for _ in range(2))
    tile, raw = ([[None] * 16 for _ in range(2)] for _ in range(2))
    counted, flags, scales = [None] * c["kBits"], [None] * c["kBits"], [None] * max(c["kScales"], 1)
    wrong, coming, pipe, now = [], [], [], [0]

    def expect(what, got, want):
        if got != want:
            wrong.append((what, want, got))

    def wait(bar, parity):
        while not bar.passed(parity):
            yield

    def copier(kv):
        slots, to = (raws, raw) if eight else (ring, tile)
        for y in range(nt):
            s = y % slots
            if y >= slots:
                yield from wait((free if eight else empty)[kv][s], (y // slots & 1) ^ 1)
            bar = last[y - mixed_from] if not eight and kv == 1 and y >= mixed_from else full[kv][s]
            if kv == 0:
                counted[y % c["kBits"]] = y
            bar.arrive(1)
            to[kv][s] = None

            def land(y=y, s=s, bar=bar):
                to[kv][s] = y
                bar.land(1)
            coming.append((now[0] + rnd.randint(5, 400 if slow == f"copy{kv}" else 60), land))
            yield

    def fitter(kv, half, group):
        first, step = (group, groups) if eight else (mixed_from, 1)
        if not eight and kv == 0:
            return
        for j in range(first, nt, step):
            s = j % ring
            if eight:
                yield from wait(full[kv][j % raws], j // raws & 1)
                expect("copied", raw[kv][j % raws], j)
                yield
                if kv == 0:
                    expect("counted, widening", counted[j % c["kBits"]], j)
                elif j >= mixed_from and half == 0:
                    flags[j % c["kBits"]] = j
                free[kv][j % raws].arrive()
                if j >= ring:
                    yield from wait(empty[kv][s], (j // ring & 1) ^ 1)
                if half == 0:
                    tile[kv][s] = j
                    if kv == 0:
                        scales[j % c["kScales"]] = j
                yield
                if groups > 1 and j > 0:
                    yield from wait(ready[kv][(j - 1) % ring], (j - 1) // ring & 1)
                ready[kv][s].arrive()
                if own and kv == 1 and j >= mixed_from:
                    looked[j - mixed_from].arrive()
            else:
                yield from wait(last[j - mixed_from], 0)
                expect("copied", tile[1][s], j)
                if half == 0:
                    flags[j % c["kBits"]] = j
                yield
                looked[j - mixed_from].arrive()

    def mine(t):
        return list(range(t, nt, 2)) if alternate else list(range(nt))

    def products(t):
        my = mine(t)
        for j in range(-1, len(my)):
            if j + 1 < len(my):
                y = my[j + 1]
                yield from wait((ready if eight else full)[0][y % ring], y // ring & 1)
                if j >= 0:
                    yield from wait(sfree[t], j & 1)

                def scored(y=y):
                    expect("keys", tile[0][y % ring], y)
                    sfull[t].arrive()
                    empty[0][y % ring].arrive()
                pipe.append(scored)
                yield
            if j < 0:
                continue
            y = my[j]
            if not eight and y >= mixed_from:
                yield from wait(looked[y - mixed_from], 0)
            else:
                yield from wait((ready if eight else full)[1][y % ring], y // ring & 1)
            yield from wait(pfull[t][j & 1], j >> 1 & 1)

            def summed(y=y, j=j):
                expect("values", tile[1][y % ring], y)
                pfree[t][j & 1].arrive()
                empty[1][y % ring].arrive()
            pipe.append(summed)
            yield

    def softmax(t):
        for j, y in enumerate(mine(t)):
            yield from wait(sfull[t], j & 1)
            yield
            sfree[t].arrive()
            if y >= mixed_from:
                if own or not eight:
                    yield from wait(looked[y - mixed_from], 0)
                else:
                    yield from wait(ready[1][y % ring], y // ring & 1)
                expect("looked through", flags[y % c["kBits"]], y)
            for _ in range(rnd.randint(1, 25)):
                expect("counted", counted[y % c["kBits"]], y)
                if y >= mixed_from:
                    expect("flags", flags[y % c["kBits"]], y)
                if eight:
                    expect("scales", scales[y % c["kScales"]], y)
                yield
            if j > 0 and rnd.random() < 0.3:            # O is moved to another reference
                yield from wait(pfree[t][j & 1 ^ 1], (j - 1) >> 1 & 1)
            pfull[t][j & 1].arrive()

    parts = {"copy0": copier(0), "copy1": copier(1)}
    for kv in range(2):
        for g in range(groups):
            for half in range(2):
                parts[f"fit{kv}{g}{half}"] = fitter(kv, half, g)
    for t in range(2 if alternate or two else 1):
        parts[f"products{t}"], parts[f"softmax{t}"] = products(t), softmax(t)
    pace = {n: 9 if slow and n.startswith(slow) else rnd.choice([1, 1, 2, 5, 9]) for n in parts}
    busy = 0
    while parts or coming or pipe:
        now[0] += 1
        if now[0] > 60000:
            return wrong + [("stuck", sorted(parts), nt)]
        for e in [e for e in coming if e[0] <= now[0]]:
            coming.remove(e)
            e[1]()
        if pipe and now[0] >= busy:
            pipe.pop(0)()
            busy = now[0] + rnd.randint(1, 4)
        for n in list(parts):
            if now[0] % pace[n] == 0:
                try:
                    next(parts[n])
                except StopIteration:
                    del parts[n]
    return wrong


def many(c, eight, mode, seeds, own=True):
    found = []
    for seed in range(seeds):
        r = random.Random(seed)
        nt = r.choice([1, 2, 3, 4, 5, 7, 9, 13, 17, 40])
        mixed_from = max(0, nt - r.choice([1, 1, 2, 5]))
        slow = r.choice([None, None, "copy0", "copy1", "fit1", "fit0", "softmax0"])
        try:
            bad = run(c, eight, mode, nt, mixed_from, seed, two=bool(seed % 3), own=own, slow=slow)
        except AssertionError as e:
            bad = [(str(e), nt, seed)]
        found += bad[:1]
    return found


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("hd", [64, 128])
def test_no_wait_passes_early(hd, eight, mode):
    c = constants(hd, eight, mode)
    assert c["kRing"] >= 3 and c["kScales"] > c["kRing"]
    assert not many(c, eight, mode, 150, own=not eight or own_barriers())


def test_the_model_finds_what_it_is_for():
    c = constants(128, False, "KEYS")
    assert many(dict(c, kRing=5, kScales=10, kBits=10), False, "KEYS", 300)      # slots of both streams
    c = constants(128, True, "HALF")
    assert c["kGroups"] == 2 and c["kRing"] == 3
    assert many(c, True, "HALF", 300, own=False)         # flags that are waited for with their tile
    assert many(dict(c, kBits=c["kRing"] + 2), True, "HALF", 300)                # overwritten descriptions
    assert many(dict(c, kScales=c["kRing"] + 1), True, "HALF", 300)
