"""Hand-worked pins of the plan's, the trees' and the candidates' oracle."""
import numpy as np

from oracle import tree_oracle as T


def test_plan_by_hand():
    # pages of 16; sequence 0 grows inside its page, 1 takes two, 2 gives one back, 3 finds too few, 4 needs none
    table = np.array([[5, -9], [6, -9], [7, 8], [9, -9], [4, -9]])
    table = np.concatenate([table, np.full((5, 1), -9)], 1)
    got = T.plan([3, 16, 20, 16, 0], [2, 20, -10, 1, 0], table, [0, 11, 12, 0, 0, 0], (1, 2), 16, 20, rows=24)
    assert got["ctx"].tolist() == [5, 36, 10, 16, 0] and got["state"].tolist() == [3, 1]
    assert got["offsets"].tolist() == [0, 2, 22, 22, 22, 22]
    assert got["table"][1].tolist() == [6, 11, 12] and got["queue"].tolist() == [0, 11, 12, 8, 0, 0]
    assert got["slots"][:4].tolist() == [83, 84, 11 * 16, 11 * 16 + 1] and got["slots"][18:].tolist() == [
        12 * 16, 12 * 16 + 1, 12 * 16 + 2, 12 * 16 + 3, -1, -1]
    assert got["positions"][2] == 16 and not got["bad"]


def test_plan_places_and_errors():
    table = np.zeros((2, 1), int)
    got = T.plan([0, 17], [3, 1], table, [7, 30], (0, 2), 16, 30, place=np.array([[2, -1, 0, 5], [0, 0, 0, 0]]))
    assert got["slots"].tolist() == [[7 * 16 + 2, -1, 7 * 16, -1], [-1] * 4] and got["bad"] == {-1}
    got = T.plan([0, 0], [1, 1], table, [7, 30], (0, 2), 16, 30, rows=2)
    assert got["slots"].tolist() == [7 * 16, -1] and got["bad"] == {-6} and got["positions"].tolist() == [0, 0]


def test_trees_by_hand():
    assert T.lines([-1, 0, 0, 2, -2, 4, 6, -1, 1]) == [[0], [0, 1], [0, 2], [0, 2, 3], [], [], [], [7], [0, 1, 8]]
    see = T.tree_seen([-1, 0, 1, -2], 3, window=2)
    assert see.astype(int).tolist() == [[0, 0, 1, 1, 0, 0, 0], [0, 0, 0, 1, 1, 0, 0], [0, 0, 0, 0, 1, 1, 0], [0] * 7]


def test_candidates_by_hand():
    x = np.array([2.0, -2.0, 4.0, 1.0, 4.0, np.nan], np.float32)
    y = T.adjust(x, np.array([1, 2, 0, 0, 0, 0]), np.array([0, 0, 1, 0, 0, 0], bool), 2.0, 0.25, 0.5, {3: 1.0},
                 np.array([1, 1, 1, 1, 0, 1], bool))
    assert y[:5].tolist() == [0.25, -5.0, 2.0, 2.0, -np.inf]
    assert T.best(y, 6).tolist() == [5, 2, 3, 0, 1, 4]
