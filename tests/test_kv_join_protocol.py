"""CPU model of how the paged attention (csrc/kv_attn.cu) hands out the parts of units and has them joined: every
finding warp's loop, the queue they share, the counts of parts.  A finished unit's join waits in one variable of the
warp that counted its last part until the next description takes it along; the model fails where it is overwritten,
left over, or done before a part is there."""
import os
import random
import re

import pytest

import tiled_exact_attention_fa2_gb300._build as build

DESCS, AHEAD, JOIN = 4, 32, 32
MIN_ITEMS = (48, 64, 128)  # kMinItem's values


def cut_into_items(slots, ctas, least):
    """Items (unit, part, parts, first slot, slots) of units of `slots` each, by layout()'s rule for many units."""
    total = sum(slots)
    share = -(-total // ctas)
    items, before = [], 0
    for u, n in enumerate(slots):
        tail = before >= total - total // 4
        cut = max((share + 15) // 16 if tail else (share + 3) // 4, least)
        parts = max((n + cut // 2) // cut, 1)
        items += [(u, i, parts, n * i // parts, n * (i + 1) // parts - n * i // parts) for i in range(parts)]
        before += n
    return items


class Run:
    def __init__(self, seed, items, ctas):
        self.rng, self.items, self.ctas = random.Random(seed), items, ctas
        self.taken, self.counts, self.finished, self.joined, self.groups = 0, {}, set(), [], {}
        self.error = None

    def item(self, i):
        return self.items[i]

    def group(self, unit, part, parts):
        """What a part is counted for, and of how many."""
        if parts <= JOIN:
            return (unit, 0), parts
        return (unit, part // JOIN), min(JOIN, parts - part // JOIN * JOIN)

    def finder(self, me, descs, processed):
        """One warp's find_items(); yields until the scheduler has let the described items be worked on."""
        total = len(self.items)
        at, there, done, open_, ahead, join = me, me < total, 0, 0, 0, None
        while True:
            if there and (open_ < 2 or (len(descs) - done < DESCS and ahead < AHEAD)):
                if at is None:
                    left = max(total - 2 * self.ctas, 0)
                    n, self.taken = self.taken, self.taken + 1
                    at = 2 * self.ctas + n if n < left else total
                    there = at < total
                    if not there:
                        continue
                descs.append((at, join))
                join = None
                open_, ahead = open_ + 1, ahead + self.items[at][4]
                at = at + self.ctas if len(descs) == 1 else None
                there = at is None or at < total
            elif not there and open_ == 0:
                descs.append(("end", join))
                return
            elif not there and join:
                descs.append((None, join))
                join = None
            else:
                while processed[0] <= done:
                    yield
                at_done = descs[done][0]
                done += 1
                if at_done is None:
                    continue
                unit, part, parts, _, length = self.items[at_done]
                open_, ahead = open_ - 1, ahead - length
                if parts > 1:
                    key, size = self.group(unit, part, parts)
                    self.counts[key] = self.counts.get(key, 0) + 1
                    if self.counts[key] == size:
                        if join is not None:
                            self.error = self.error or f"the join of {join} is lost"
                        join = key

    def work(self, what, join):
        """The computing warps: the join that a description carries, then its item."""
        if join is not None:
            parts = {i[1] for i in self.items if i[0] == join[0]}
            mine = [(join[0], p) for p in parts if self.group(join[0], p, len(parts))[0] == join]
            if not all(p in self.finished for p in mine):
                self.error = self.error or f"{join} is joined before its parts are there"
            self.joined.append(join)
        if isinstance(what, int):
            self.finished.add(self.items[what][:2])

    def run(self):
        state = []
        for me in range(self.ctas):
            descs, processed = [], [0]
            state.append((self.finder(me, descs, processed), descs, processed))
        running = set(range(self.ctas))
        while running and not self.error:
            me = self.rng.choice(sorted(running))
            find, descs, processed = state[me]
            if self.rng.random() < 0.5 and processed[0] < len(descs):
                self.work(*descs[processed[0]])
                processed[0] += 1
            elif next(find, "ended") == "ended" and processed[0] == len(descs):
                running.discard(me)
        if self.error:
            return self.error
        cut = {self.group(u, p, n)[0] for u, p, n, _, _ in self.items if n > 1}
        if sorted(self.joined) != sorted(cut):
            return f"{len(cut)} to be joined, {len(self.joined)} were"
        if len(self.finished) != len(self.items):
            return "items left out"
        total = len(self.items)
        if total > self.ctas and self.taken != max(total - 2 * self.ctas, 0) + min(self.ctas, total - self.ctas):
            return f"{self.taken} asked the queue"  # (whoever asks last sets it back)
        return None


def units(seed):
    r = random.Random(seed)
    short = lambda: r.randint(1, 40)  # noqa: E731
    long = lambda: int(2 ** r.uniform(4, 12))  # noqa: E731
    return [long() if r.random() < r.choice([0.1, 0.5, 0.9]) else short() for _ in range(r.randint(1, 120))]


@pytest.mark.parametrize("least", MIN_ITEMS)
def test_every_cut_unit_is_joined_once(least):
    cut = 0
    for seed in range(150):
        ctas = random.Random(seed).choice([2, 3, 5, 8])
        run = Run(seed, cut_into_items(units(seed), ctas, least), ctas)
        result = run.run()
        assert result is None, f"seed {seed}: {result}"
        cut += len(run.joined)
    assert cut > 500


def test_model_catches_parts_that_are_too_short():
    """Units of 6 to 60 slots in two or three parts, whatever their length."""
    found = []
    for seed in range(150):
        r = random.Random(seed)
        items = []
        for u in range(60):
            n, parts = r.randint(6, 60), r.randint(2, 3)
            items += [(u, i, parts, n * i // parts, n * (i + 1) // parts - n * i // parts) for i in range(parts)]
        found.append(Run(seed, items, 3).run())
    assert any(f and "lost" in f for f in found)


def test_model_has_the_kernels_numbers():
    text = open(os.path.join(build.CSRC, "kv_attn.cu")).read()
    for name, value in (("kDescs", DESCS), ("kAhead", AHEAD), ("kJoin", JOIN)):
        assert int(re.search(rf"constexpr int {name} = (\d+);", text).group(1)) == value
    rule = re.search(r"constexpr int kMinItem = (.*?);", text).group(1)
    assert sorted({int(x) for x in re.findall(r"[?:(] *(\d+)", rule)}) == sorted(MIN_ITEMS)
