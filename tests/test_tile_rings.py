"""The rings of the int8 tile kernel, walked on the CPU: three sets of converters share
rings of four stages, copies land in any order, and a barrier tells only the parity
of its phase.  Whatever comes first, a set finds its own block's rows and weights."""
import os
import random
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "combine_route_count_prefix_gb300", "csrc", "gemm_int8_tiles.cu")


def source():
    """Stages of the kernel for int8 rows, and the order of a set's waits, as the source has them."""
    text = open(SOURCE).read()
    stages = {n: int(re.search(rf"constexpr int {n} = (?:TB == 64 \? )?(\d+)", text).group(1)) for n in ("SA", "S8", "SR")}
    stages["sets"] = int(re.search(r"constexpr int kSets = (\d+)", text).group(1))
    widen = text[text.index("auto widen ="):text.index("auto widen =") + 4000]
    waits = re.findall(r"wait_bounded_inline\(&(\w+)\[", re.sub(r"//[^\n]*", "", widen))[:3]
    return stages, waits


class Barrier:
    """An mbarrier as a wait sees it: a phase's parity, nothing more."""

    def __init__(self):
        self.phase = 0

    def passed(self, parity):
        return self.phase & 1 != parity


def walk(stages, waits, blocks, rng):
    """One random order of everything that may happen.  Returns the first wrong block, or None."""
    n = dict(r8=stages["SR"], w8=stages["S8"], ab=stages["SA"])
    full = {r: [Barrier() for _ in range(k)] for r, k in n.items()}
    empty = {r: [Barrier() for _ in range(k)] for r, k in n.items()}
    held = {r: [None] * k for r, k in n.items()}     # the block whose bytes lie in a stage
    asked = dict(r8=0, w8=0)                         # blocks whose copies have been started
    flying = []                                      # (ring, block)
    at = list(range(stages["sets"]))                 # each set's block
    step = [0] * stages["sets"]
    multiplied = 0

    def parity(ring, b):
        return b // n[ring] & 1

    def convert(i):
        """The set's next step, or False while it has to wait."""
        b = at[i]
        if step[i] < 3:
            ring, kind = waits[step[i]].split("_")
            bar = (full if kind == "full" else empty)[ring][b % n[ring]]
            if not bar.passed(parity(ring, b) ^ (kind == "empty")):
                return False
        elif step[i] == 3:                           # both operands have been read and the block is there
            for ring in ("r8", "w8"):
                if held[ring][b % n[ring]] != b:
                    return b
                empty[ring][b % n[ring]].phase += 1
            full["ab"][b % n["ab"]].phase += 1
        step[i] += 1
        if step[i] == 4:
            at[i], step[i] = b + stages["sets"], 0
        return True

    weight = [rng.random() ** 2 + 0.03 for _ in range(5)]     # some agents far slower than others
    while multiplied < blocks:
        what = rng.choices(range(5), weight)[0]
        if what < 2:
            ring = ("r8", "w8")[what]
            b = asked[ring]
            if b < blocks and empty[ring][b % n[ring]].passed(parity(ring, b) ^ 1):
                asked[ring] += 1
                held[ring][b % n[ring]] = None       # being written
                flying.append((ring, b))
        elif what == 2 and flying:
            ring, b = flying.pop(rng.randrange(len(flying)))
            held[ring][b % n[ring]] = b
            full[ring][b % n[ring]].phase += 1
        elif what == 3:
            i = rng.randrange(stages["sets"])
            if at[i] < blocks:
                wrong = convert(i)
                if wrong is not True and wrong is not False:
                    return wrong
        elif what == 4 and full["ab"][multiplied % n["ab"]].passed(parity("ab", multiplied)):
            empty["ab"][multiplied % n["ab"]].phase += 1
            multiplied += 1
    return None


def first_wrong(stages, waits, orders):
    for seed in range(orders):
        wrong = walk(stages, waits, 14, random.Random(seed))
        if wrong is not None:
            return wrong
    return None


def test_every_set_finds_its_own_block():
    stages, waits = source()
    assert sorted(waits) == ["ab_empty", "r8_full", "w8_full"]
    assert first_wrong(stages, waits, 400) is None


@pytest.mark.parametrize("waits", [["r8_full", "ab_empty", "w8_full"], ["w8_full", "ab_empty", "r8_full"]], ids=str)
def test_a_copy_awaited_before_the_stage_is_free_can_be_the_one_before(waits):
    """The walk sees the fault: a copy's parity passes one phase early."""
    assert first_wrong(source()[0], waits, 400) is not None
