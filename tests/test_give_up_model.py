"""A wait that runs out in amk_linear's walking kernels (csrc/amk_op_linear.cuh): whichever of a
draining warpgroup's warps give up, at whichever tile, all of them reach the kernel's end.

The barriers of a warpgroup's four warps are walked as the source orders them: a tile's sums are
waited for (a wait of each warp's own, which may run out in any of them), the warps agree on going
on, and the gated halves are handed over under a barrier a round."""
import itertools
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
WARPS, TILES, ROUNDS = 4, 2, 2


def warp(gives_up_at, agree):
    """A warp's barriers in turn: yields (barrier, vote), is sent the votes' conjunction."""
    for tile in range(TILES):
        ok = tile != gives_up_at
        if agree:
            ok = yield "group", ok
        if not ok:
            break
        for _ in range(ROUNDS):
            yield "group", True
        if not agree:  # both buffers are read before the next tile writes them
            yield "group", True
    yield "end", True


def ends(gives_up, agree):
    warps = [warp(g, agree) for g in gives_up]
    at = [next(w) for w in warps]
    while any(a is not None for a in at):
        here = {a[0] for a in at if a is not None}
        if len(here) > 1 or any(a is None for a in at):
            return False  # some at one barrier, the others at another for good
        vote = all(a[1] for a in at)
        for i, w in enumerate(warps):
            try:
                at[i] = w.send(vote)
            except StopIteration:
                at[i] = None
    return True


def cases():
    return itertools.product([None, *range(TILES)], repeat=WARPS)


def test_without_an_agreement_some_warps_wait_for_good():
    assert any(not ends(c, agree=False) for c in cases())


def test_every_warp_reaches_the_end():
    assert all(ends(c, agree=True) for c in cases())


def test_the_source_agrees_before_its_barriers():
    src = open(os.path.join(ROOT, "persistent_megakernel_decode_cta_b200", "csrc",
                            "amk_op_linear.cuh")).read()
    drain = src[src.index("const int wg = (warp - 4) >> 2"):src.index("} else if constexpr (CODES) {")]
    agree = re.search(r"ok = named_bar_and\(1 \+ wg, 128, ok\);\s*if \(!ok\)\s*break;", drain)
    assert agree, "no agreement"
    # no way out of a tile between it and the last of the group's barriers
    barriers = [m.start() for m in re.finditer(r"named_bar\(1 \+ wg, 128\)", drain)]
    assert barriers and all(b > agree.end() for b in barriers)
    assert "break" not in drain[agree.end():barriers[-1]]


def test_clusters_hear_of_it_before_they_add_up():
    """In the kernels that wait: the barrier before a cluster's sums are read tells every rank."""
    csrc = os.path.join(ROOT, "persistent_megakernel_decode_cta_b200", "csrc")
    for name, merges in (("amk_op_linear.cuh", 1), ("amk_op_attention.cu", 2)):
        src = open(os.path.join(csrc, name)).read()
        assert len(re.findall(r"cluster_sync_failed\(fail, split\);", src)) == merges
        # what is read behind it is read only where no rank failed
        for part in src.split("cluster_sync_failed(fail, split);")[1:]:
            assert "!*fail" in part[:part.index("cluster_sync();")]
