"""weight_kernel's two warps of a row wait for one another at a named barrier,
which has no time limit of its own: it stays bounded only if both come to it
equally often, on a timeout too.  Host-side checks: of the source (one place
where they meet; what is decided behind it is the barrier's own answer, the
same for both, never another look at the abort flag, which may have changed
for one of them; every way out of the walk ends with a meeting), and of that
rule in all combinations of give-ups."""

import itertools
import os
import re

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_sparse_attention_psa_b200",
                   "csrc", "weight.cu")


def _code():
    with open(SRC) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_the_pair_parts_at_one_meeting():
    src = _code()
    assert "named_barrier_sync(" not in src, "a barrier that does not say who gave up"
    assert src.count("named_barrier_or(") == 1, "the warps of a row meet in one place"
    body = re.search(r"auto meet = \[&\]\(bool gone\) -> bool \{(.*?)\};", src, re.S)
    assert body and re.sub(r"\s", "", body.group(1)) == "returnnamed_barrier_or(pair_bar,64,gone||*abort_flag);"
    sums = src[body.end():]
    sums = sums[:sums.index("tmem_dealloc")]
    assert "*abort_flag" not in sums, "the flag is looked at before the barrier only"
    assert sums.count("meet(") == 2 and "if ((met = meet(false))) break;" in sums
    # behind the walk over the units: a last meeting, whatever ended it
    assert re.search(r"if \(!ok \|\| met\) break;\s*\}\s*__syncwarp\(\);\s*if \(!met\) meet\(true\);", sums)


def test_the_rule_in_all_combinations():
    """Two warps with `n` meetings and a last one; each may give up before any of
    them (its next meeting is then its last) and sees the flag from any on.
    They part at the answer both get: none is left waiting."""
    n = 3
    when = [*range(n + 1), None]
    for give_up in itertools.product(when, when):
        for sees in itertools.product(range(n + 2), repeat=2):
            left = [False, False]
            for j in range(n + 1):
                assert left[0] == left[1], "one waits for a partner that has left"
                if left[0]:
                    break
                last = [j == n or (g is not None and j >= g) for g in give_up]
                answer = any(last[w] or j >= sees[w] for w in (0, 1))
                left = [answer or x for x in last]
            assert left == [True, True]


def test_a_warp_uses_a_unit_only_if_every_lane_has_it():
    """Lanes of the lse and the MMA warp wait for the next unit one by one; after
    a timeout one may come back without a unit while lane 0 has one, and its
    fields are then not to be used (the lse warp makes addresses of them)."""
    parts = _code().split("next_unit(x, false);")
    assert len(parts) == 3
    for after in parts[1:]:
        assert re.match(r"\s*__syncwarp\(\);\s*if \(!__all_sync\(0xffffffffu, x\.nt >= 0\)\) break;", after)
