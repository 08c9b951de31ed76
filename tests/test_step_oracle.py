"""The definitions of oracle/step.py, pinned by hand and against torch."""
import numpy as np
import torch

from oracle import step


def test_tables_by_hand():
    # row 0 holds page 7 and its 15 tokens grow by 3; row 1 has ended; row 2 is new, 17 tokens
    got = step.build_tables([3, -1, 17, 0], [15, 20, 0, 0], [0, 1, 2, -1], 16, [[7, -1, -1], [4, 9, -1], [-1, -1, -1]], [1, 2, 0],
                            [5, 6, -1, -1], 2, 3, 21)
    assert got["free"] == [5, 6, 4, 9] and got["num_free"] == [1]
    assert got["table"] == [[7, 9, -1], [-1] * 3, [4, 6, -1], [-1] * 3]
    assert got["lens"] == [18, 0, 17, 0] and got["qsl"] == [0, 3, 3, 20, 20] and got["counts"] == [2, 0, 2]
    assert got["slots"] == [7 * 16 + 15, 9 * 16, 9 * 16 + 1] + [4 * 16 + i for i in range(16)] + [6 * 16] + [-1]
    assert not got["bad"]


def test_tables_without_enough_pages():
    got = step.build_tables([1, 40, 1, 2], [16, 0, 3, 0], [0, 1, 2, 3], 16, [[3, -1, -1]] + [[8, -1, -1] for _ in range(3)], [1, 0, 1, 0],
                            [1, 2], 2, 3, 44)
    # the second needs three and gets none, nor does the fourth; the third has its page
    assert got["lens"] == [17, 0, 4, 0] and got["bad"] and got["num_free"] == [1] and got["counts"] == [2, 0, 1, 0]


def test_masks_by_hand():
    masks, pos = step.tree_masks([-1, 0, 0, 2, -1], [12], [0, 5], 2)
    assert masks == [[1, 0], [3, 0], [5, 0], [13, 0], [16, 0]] and pos == [7, 8, 8, 9, 7]
    masks, _ = step.tree_masks(list(range(-1, 39)), [40], [0, 40], 2)
    assert masks[31] == [-1, 0] and masks[39] == [-1, 255]


def test_attention_against_torch():
    rng = np.random.default_rng(0)
    q, k, v = (rng.standard_normal((n, 256)) for n in (9, 30, 30))
    seen = rng.random((9, 30)) < 0.5
    seen[4] = False
    out, _, lse, _ = step.attention(q, k, v, seen, 1 / 16)
    x = torch.tensor(q @ k.T / 16).masked_fill(~torch.tensor(seen), -torch.inf)
    want = torch.softmax(x, -1) @ torch.tensor(v)
    want[4] = 0
    assert np.abs(out - want.numpy()).max() < 1e-12
    ref = torch.logsumexp(x, -1).numpy()
    assert lse[4] == -np.inf and np.abs(np.delete(lse - ref, 4)).max() < 1e-12


def test_seen_of_a_chain_is_causal():
    masks, _ = step.tree_masks(list(range(-1, 6)), [20], [0, 7], 1)
    assert (step.tree_seen(masks, 7, 20) == (np.arange(20) <= 13 + np.arange(7)[:, None])).all()
