"""Static checks on the sources of the attention over trees of drafted tokens (no
GPU, no compiler)."""
import re

import pytest

from test_kernel_sources import _kernel_body, _sources


def test_no_cta_exits_ahead_of_its_copies():
    """The tcgen05 kernel's loading warps wait for the last copies of each ring
    whichever warp gave up on a wait: one that had issued all of its copies saw
    nothing of that."""
    body = _kernel_body(_sources()["attention_tree_tc.cu"], "tree_tc05_kernel")
    loads = body[body.index("-- loads"):]
    loads = loads[loads.index("if (k + 1 < part.n) lookup(t + 1);"):]
    end = loads[:loads.index("__syncwarp();")]
    assert "mbar_wait(full + stage, phase);" in end and "mbar_wait(q_full + i, " in end
    assert not re.search(r"\bok\b", end)


@pytest.mark.parametrize("stages", [4, 5])
def test_the_parity_of_a_rings_last_fills(stages):
    """What the loading warps wait for, for every number of fills: the phase of each
    stage's last one, or for a stage without one the parity that a new barrier lets
    through."""
    body = _kernel_body(_sources()["attention_tree_tc.cu"], "tree_tc05_kernel")
    assert "mbar_wait(q_full + i, ((part.f + 1 - i) / 2 - 1) & 1);" in body
    for n in range(4 * stages):
        stage, phase = n % stages, 1 ^ (n // stages & 1)
        for _ in range(stages):
            fills = len(range(stage, n, stages))
            assert phase == (fills - 1) % 2, (n, stage)
            stage += 1
            if stage == stages:
                stage, phase = 0, phase ^ 1
        for i in range(2):
            assert ((n + 1 - i) // 2 - 1) & 1 == (len(range(i, n, 2)) - 1) % 2


def test_the_rules_for_pairs_go_by_the_devices_sms():
    """As the grids do: a pair to an SM is as many pairs as the device has SMs.  The
    one literal is the bound on shares, which the workspace's size goes by."""
    srcs = {f: t for f, t in _sources().items() if f.startswith(("attention_tree", "tree_share"))}
    code = {f: re.sub(r"//[^\n]*", "", t) for f, t in srcs.items()}
    assert {f: len(re.findall(r"\b15[0-9]\b", t)) for f, t in code.items() if re.search(r"\b15[0-9]\b", t)} == {"tree_share.cuh": 1}
    assert "return 152 * ctas_per_sm(N);" in code["tree_share.cuh"]
    assert sum(t.count("few_pairs(a)") for t in code.values()) == 3
