"""The loop that drafts and verifies, on a pool that runs out of blocks: who waits
keeps its place, its text and its cache, the others go on with the tokens that the
model chooses."""
import numpy as np
import pytest
import torch

import oracle
from gpt_transformer_forward_gb300 import binding as ab

from gpu_helpers import assert_close, host, need_gpu, no_device_error
from test_gpu_draft_step import ALL, LOGIT_TOL, NAMES, Loop

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("precision", ALL, ids=[NAMES[p] for p in ALL])
def test_a_sequence_that_waits_keeps_everything(precision):
    B, N = 4, 8
    loop = Loop(precision, B, N, 11, seed=2, rules=False)  # one block less than three each
    cfg, tol = loop.cfg, LOGIT_TOL[precision]
    seen = {}

    def decode_step_tree(kv, tok, pos, *args, **kw):
        seen.update(pos=pos.clone(), pool=loop.pool.clone())
        return step(kv, tok, pos, *args, **kw)

    step, loop.m.decode_step_tree = loop.m.decode_step_tree, decode_step_tree
    memo = {}

    def guess(b, told):
        key = tuple(told)
        if key not in memo:
            memo[key] = int(oracle.forward(cfg, loop.params, np.array([told], np.int32))[0][0, -1, :cfg.vocab_size].argmax())
        return memo[key]

    both = 0  # steps in which some waited and some went on
    for _ in range(6):
        texts, places = [list(t) for t in loop.text], loop.pos.tolist()
        count = loop.step(guess)
        no_device_error()
        pos, L = seen["pos"].tolist(), loop.last
        waits = [p == -1 for p in pos]
        both += any(waits) and not all(waits)
        table = loop.table.cpu().numpy()
        shape = (cfg.num_layers, 2, loop.num_blocks, cfg.num_heads, loop.bs, -1)
        changed = (seen["pool"].view(shape) != loop.pool.view(shape)).any(-1).any(0).any(0).any(1).cpu().numpy()
        for b in range(B):
            if waits[b]:
                assert count[b] == 0 and loop.pos[b] == places[b] and loop.text[b] == texts[b]
                assert (L["path"][b] == -1).all()
                continue
            assert pos[b] == places[b] and 1 <= count[b] <= N and loop.pos[b] == places[b] + count[b]
            assert L["path"][b, 0] == 0 and len(loop.text[b]) == len(texts[b]) + count[b]
            ref = oracle.forward(cfg, loop.params, np.array([loop.text[b]], np.int32))[0][0, :, :cfg.vocab_size]
            for k in range(count[b]):
                node, at = int(L["path"][b, k]), len(texts[b]) - 1 + k
                assert_close(L["plain"][b, node, :cfg.vocab_size], ref[at], atol=tol, what=f"sequence {b}, {k} accepted")
                assert ref[at, loop.text[b][at + 1]] >= ref[at].max() - 2 * tol
            # its new rows, the tree's and those that were moved, are its own
            for j in range(pos[b], pos[b] + N):
                changed[table[b, j // loop.bs], j % loop.bs] = False
        assert not changed.any(), "rows of no tree of this step"
    assert both > 0 and loop.waited > 0
    assert loop.pos.tolist() == [len(t) - 1 for t in loop.text]
    # the cache of each sequence, waiting or not, is its text's: one more step of each
    room = loop.held[0] > loop.pos  # a block for one more position
    one, _ = loop.m.new_outputs(B, 1, probs=False)
    last = torch.tensor([[t[-1]] for t in loop.text], dtype=torch.int32, device="cuda")
    step(loop.kv, last, torch.where(room, loop.pos, torch.full_like(loop.pos, -1)), one, loop.m.new_tree_workspace(B, 1))
    got = host(one)[:, 0]
    for b in range(B):
        if room[b]:
            ref = oracle.forward(cfg, loop.params, np.array([loop.text[b]], np.int32))[0][0, -1, :cfg.vocab_size]
            assert_close(got[b, :cfg.vocab_size], ref, atol=tol, what=f"sequence {b}")
    no_device_error()
