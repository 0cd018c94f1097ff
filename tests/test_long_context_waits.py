"""What the kernels for long contexts and few rows may have in flight, and wait
for: read from their sources, or worked through on the CPU (a missing wait is
nothing to try on a GPU)."""
import glob
import os
import re

import pytest

import mla_attention_nvfp4_gb300 as mla

CSRC = os.path.join(os.path.dirname(mla.__file__), "csrc")


def code_of(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_no_copy_or_commit_reaches_another_ctas_shared_memory():
    # the library is every rank's, whatever memory a cache lies in; and a commit that arrives in another CTA may find it ended
    names = [os.path.basename(p) for p in glob.glob(os.path.join(CSRC, "*.c*")) + glob.glob(os.path.join(CSRC, "*.h"))]
    assert "fp8_weights.cu" in names
    for name in names:
        assert "multi" + "cast" not in code_of(name), name


@pytest.mark.parametrize("tiles", [1, 2])
@pytest.mark.parametrize("n", [1, 2, 3, 4, 7, 100])
def test_key_weights_wait_for_all_copies_in_flight(tiles, n):
    """drain_copies looks at the last `stages` copies before `issued`: copy i in slot i % stages, of phase i / stages.
    Chunk c of tile n is in slot 5 (n % tiles) + c, of phase n / tiles, and those of the last `tiles` tiles may be in
    flight; of the last tile any lane may be missing."""
    code = code_of("fp8_weights.cu")
    assert re.search(r"drain_copies\(ms\.full, C::slots, ms\.copies\)", code)
    assert re.search(r"i = n % C::tiles \* 5 \+ c;\s*ok = mbar_wait\(&ms\.empty\[i\]", code)
    counted = re.search(r"(copies = __reduce_max_sync\(0xffffffffu, copies\);\s*)?if \(lane == 0\) ms\.copies = ([^;]+);", code)
    for missing in (set(), {0}, {1, 4}, {0, 1, 2, 3}):
        issued = [n - (lane in missing) for lane in range(5)]  # chunks a lane
        count = eval(counted.group(2), {}, {"copies": max(issued) if counted.group(1) else issued[0]})
        stages = 5 * tiles
        waited = {(i % stages, i // stages % 2) for i in range(max(0, count - stages), count)}
        flying = {(5 * (t % tiles) + c, t // tiles % 2) for c in range(5) for t in range(max(0, n - tiles), issued[c])}
        assert flying <= waited, (missing, flying - waited)


@pytest.mark.parametrize("heads", [16, 32, 64, 128])
def test_key_weights_groups_wait_for_every_phase_of_their_barriers(heads):
    """A wait for a phase's parity passes while the barrier is in the phase after it, so that a waiter who leaves one out may
    take the phase before it for its own: each group of sum warps has to wait for every phase of what it waits for."""
    code = code_of("fp8_weights.cu")
    groups = 4 if heads >= 64 else 2
    assert re.search(r"constexpr int kGroups = kH >= 64 \? 4 : 2;", code)
    assert re.search(r"if \(n % kGroups<kH> != group\) continue;", code)
    env = {"kGroups": groups, "kInfo": int(re.search(r"constexpr int kInfo = (\d+);", code).group(1))}

    def value(text, **kw):
        text = re.sub(r"kGroups<kH>", "kGroups", text).replace("/", "//")
        return eval(text, {}, {**env, **kw, "half": kw["n"] & 1})

    waits = dict((m.group(1), m.groups()[1:]) for m in
                 re.finditer(r"mbar_wait\(&ms\.(s_full|info_full)\[([^]]+)\], ([^,]+), err", code))
    done = re.search(r"mma_commit\(&ms\.s_full\[([^]]+)\]\)", code).group(1), "info", re.search(
        r"mbar_arrive\(&ms\.info_full\[([^]]+)\]\)", code).group(1)
    for name, arrives in (("s_full", done[0]), ("info_full", done[2])):
        which, parity = waits[name]
        phases = {}  # of each barrier: how many are done
        seen = {}    # of each group and barrier: phases it has waited for
        for n in range(48):
            g = n % groups
            bar = value(arrives, n=n)
            assert bar == value(which, n=n, group=g)
            assert value(parity, n=n, group=g) == phases.get(bar, 0) % 2, (name, n)
            assert seen.get((g, bar), 0) == phases.get(bar, 0), (name, n, "a phase left out")
            phases[bar] = phases.get(bar, 0) + 1
            seen[g, bar] = seen.get((g, bar), 0) + 1
