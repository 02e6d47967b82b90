"""The ring of amk_linear's converting kernels (csrc/amk_op_linear.cuh): two groups of warps take
its stages by turns, each waiting for its own stages alone by the parity of a barrier's phase.

Every interleaving of a small run is walked: copies that land in any order, the two groups, the
products (in order).  A group may start on a stage only when its copy has landed, and the run must
never stop short.  The rings looked at are those of the compiled variants."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "persistent_megakernel_decode_cta_b200")

PROBE = r"""
#include <atomic>
#include <cstdio>
#include "amk_op_linear.cuh"
using namespace amk::linear;
template <int Q, int NT, bool SPLIT, bool PROMOTE> void show()
{
    using C = Cfg<Q, NT, SPLIT, PROMOTE>;
    printf("%d %d %d %d %d %d\n", Q, NT, (int)SPLIT, (int)PROMOTE, (int)C::STAGES, (int)C::FULLS);
}
template <int Q> void all()
{
    show<Q, 16, true, true>();
    show<Q, 32, true, true>();
    show<Q, 64, true, true>();
    show<Q, 128, true, true>();
    show<Q, 128, false, true>();
}
int main()
{
    all<AMK_QUANT_W8A16>();
    all<AMK_QUANT_W4A16>();
    show<AMK_QUANT_W8A16, 192, false, false>();
}
"""


def walk(stages, fulls, uses=13):
    """None, or what went wrong: "early" (a group took a stage whose copy had not landed) or
    "stuck"."""
    index = [0] * uses                 # a use's number among those of its barrier
    for u in range(uses):
        index[u] = u // fulls
    # issued copies, landed ones, each group's next use, whether it has passed the wait, products
    start = (0, 0, (0, 1), (False, False), 0)
    seen, todo = {start}, [start]
    while todo:
        issued, landed, nxt, inside, done = todo.pop()
        after = []
        if issued < uses:
            old = issued - stages      # the stage's last use: multiplied, and so converted
            if old < 0 or done > old:
                after.append((issued + 1, landed, nxt, inside, done))
        for u in range(issued):
            if not landed >> u & 1:
                after.append((issued, landed | 1 << u, nxt, inside, done))
        for g in (0, 1):
            u = nxt[g]
            if u >= uses:
                continue
            if not inside[g]:
                phases = sum(landed >> v & 1 for v in range(u % fulls, uses, fulls))
                if (phases & 1) != (index[u] & 1):
                    if phases <= index[u]:
                        return "early"
                    after.append((issued, landed, nxt,
                                  tuple(True if i == g else x for i, x in enumerate(inside)), done))
            elif done > u - 2:         # its TMEM buffer has been multiplied
                after.append((issued, landed,
                              tuple(x + 2 if i == g else x for i, x in enumerate(nxt)),
                              tuple(False if i == g else x for i, x in enumerate(inside)), done))
        if done < uses and nxt[done & 1] > done:
            after.append((issued, landed, nxt, inside, done + 1))
        if not after and done < uses:
            return "stuck"
        for s in after:
            if s not in seen:
                seen.add(s)
                todo.append(s)
    return None


def test_three_stages_need_two_barriers_each():
    assert walk(3, 3) == "early"
    assert walk(3, 6) is None


@pytest.mark.parametrize("stages", [2, 4, 6])
def test_even_rings(stages):
    assert walk(stages, stages, uses=2 * stages + 5) is None


def test_every_compiled_ring(tmp_path):
    src, exe = tmp_path / "rings.cu", tmp_path / "rings"
    src.write_text(PROBE)
    subprocess.run([os.environ.get("NVCC", "nvcc"), "-gencode", "arch=compute_100a,code=sm_100a",
                    "-std=c++17", "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(PKG, "csrc"), str(src), "-o", str(exe)], check=True)
    rows = [tuple(map(int, line.split())) for line in
            subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines()]
    assert len(rows) == 11
    for *variant, stages, fulls in rows:
        # a barrier's uses are one group's, whatever the copies' order
        assert fulls in (stages, 2 * stages) and fulls % 2 == 0, (variant, stages, fulls)
        if stages <= 4:
            assert walk(stages, fulls) is None, (variant, stages, fulls)
