"""The serving oracle against closed forms and worked examples."""
import numpy as np

from oracle import serving_oracle as so


def test_plan_worked_example():
    # pages of 16; request 0: 16 cached (one full page), 2 new -> one page; request 1: 3 cached, 13 new -> none;
    # request 2: nothing cached, 17 new -> two pages.  Pages come off the end of [5, 6, 7, 8].
    table = [[1, -1, -1], [2, -1, -1], [-1, -1, -1]]
    q, kv, slots, req, pos, tab, left, st = so.paged_plan([16, 3, 0], [2, 13, 17], table, [5, 6, 7, 8], 4, 16, 34)
    assert st == 0 and left == 1 and q == [0, 2, 15, 32] and kv == [18, 16, 17]
    assert tab.tolist() == [[1, 8, -1], [2, -1, -1], [7, 6, -1]]
    assert slots[:2] == [128, 129] and slots[2:15] == list(range(35, 48))
    assert slots[15:32] == list(range(112, 128)) + [96] and slots[32:] == [-1, -1]
    assert req[:3] == [0, 0, 1] and pos[2] == 3 and pos[31] == 16 and req[32] == -1


def test_plan_is_all_or_nothing():
    for args, bit in ((([0], [17], [[-1, -1]], [3], 1, 16, 17), 4), (([0], [17], [[-1]], [3, 4], 2, 16, 17), 2),
                      (([-1], [1], [[-1]], [3], 1, 16, 1), 1), (([0], [2], [[-1]], [3], 1, 16, 1), 8)):
        q, kv, slots, _, _, tab, left, st = so.paged_plan(*args)
        assert st == bit and set(q) == {0} and set(slots) == {-1} and left == args[4]
        assert tab.tolist() == args[2]


def test_attention_closed_forms():
    rng = np.random.default_rng(0)
    K, V = rng.normal(size=(3, 2, 16, 8)), rng.normal(size=(3, 2, 16, 8))
    table = np.array([[2, 0]])
    # q = 0: the mean of the visible values
    Q = np.zeros((2, 4, 8))
    O, _, rows = so.attention(Q, K, V, [0, 2], [20], table, 1.0)
    seq = np.concatenate([V[2], V[0]], 1)
    for i in range(2):
        for h in range(4):
            assert np.allclose(O[i, h], seq[h // 2, :19 + i].mean(0))
    assert rows.all()
    O, _, _ = so.attention(Q, K, V, [0, 2], [20], table, 1.0, window=3)
    assert np.allclose(O[1, 3], seq[1, 17:20].mean(0))
    O, _, _ = so.attention(Q, K, V, [0, 2], [20], table, 1.0, causal=False)
    assert np.allclose(O[0, 3], seq[1, :20].mean(0))
    # a very peaked softmax picks one key; fewer keys than tokens leave the first rows empty
    Q = 1e4 * K[2, 0, 5] * np.ones((2, 2, 1))
    O, _, _ = so.attention(Q[:1], K[:, :1], V[:, :1], [0, 1], [9], table, 1.0)
    best = int(np.argmax(K[2, 0, :9] @ K[2, 0, 5]))
    assert np.allclose(O[0, 0], V[2, 0, best])
    O, _, _ = so.attention(Q, K[:, :1], V[:, :1], [0, 2], [1], table, 1.0)
    assert (O[0] == 0).all() and np.allclose(O[1, 0], V[2, 0, 0])


def test_norm_closed_forms():
    v = np.array([[3.0, -3.0, 3.0, -3.0]])
    assert np.allclose(so.norm(v, "rms", eps=0.0), np.sign(v))
    assert np.allclose(so.norm(v + 5, "layer", eps=0.0), np.sign(v))
    h, x = so.norm_residual(v, np.ones((1, 4)), 0.5, ("none",), np.array([[2.0, 2, 2, 2]]), [0], None)
    assert np.allclose(h, 0.5 * v + 2) and np.allclose(x, h)
    h, _ = so.norm_residual(v, np.ones((1, 4)), 1.0, None, np.ones((1, 4)), [7], None)
    assert np.allclose(h, v)
