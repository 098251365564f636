"""The window oracle itself, without a GPU: against torch's masked softmax and
autograd in fp64, against differences, and the tables against a hand-made case."""
import numpy as np
import pytest
import torch

from oracle import window_oracle as wo


def _case(seed, T, Hq, Hkv, d=8):
    rng = np.random.default_rng(seed)
    return [rng.standard_normal((T, h, d)) for h in (Hq, Hkv, Hkv, Hq)]


@pytest.mark.parametrize("window,n_sink", [(0, 0), (1, 0), (5, 2), (40, 1), (3, 100)])
def test_attention_and_gradients_match_masked_autograd(window, n_sink):
    T, Hq, Hkv = 23, 4, 2
    q, K, V, dO = _case(1, T, Hq, Hkv)
    tq, tk, tv = (torch.tensor(x, requires_grad=True) for x in (q, K, V))
    t = torch.arange(T)
    see = (t[None] <= t[:, None]) & ((t[None] > t[:, None] - (window or T)) | (t[None] < n_sink))
    kk, vv = (x.repeat_interleave(Hq // Hkv, 1) for x in (tk, tv))
    s = torch.einsum("thd,chd->htc", tq, kk) / np.sqrt(q.shape[-1])
    s = s.masked_fill(~see, float("-inf"))
    o = torch.einsum("htc,chd->thd", s.softmax(-1), vv)
    (o * torch.tensor(dO)).sum().backward()
    O, lse, spread, reach = wo.attention(q, K, V, np.arange(T), window, n_sink)
    np.testing.assert_allclose(O, o.detach().numpy(), atol=1e-12)
    np.testing.assert_allclose(lse, s.logsumexp(-1).detach().numpy().T, atol=1e-12)
    assert (spread >= np.abs(O) - 1e-12).all() and (reach > 0).all()
    g, e = wo.backward(q, K, V, dO, window, n_sink)
    for got, ref, amp in zip(g, (tq.grad, tk.grad, tv.grad), e):
        np.testing.assert_allclose(got, ref.numpy(), atol=1e-11)
        assert (amp >= np.abs(got) - 1e-12).all()


def test_gradients_match_differences():
    T, w, ns = 12, 4, 1
    q, K, V, dO = _case(2, T, 2, 1)
    f = lambda a, b, c: (wo.attention(a, b, c, np.arange(T), w, ns)[0] * dO).sum()  # noqa: E731
    g, _ = wo.backward(q, K, V, dO, w, ns)
    rng, args, h = np.random.default_rng(3), [q, K, V], 1e-6
    for i in range(3):
        for _ in range(6):
            at = tuple(rng.integers(0, n) for n in args[i].shape)
            up, dn = [x.copy() for x in args], [x.copy() for x in args]
            up[i][at] += h
            dn[i][at] -= h
            assert abs((f(*up) - f(*dn)) / (2 * h) - g[i][at]) < 1e-7


def test_rows_without_a_visible_key_are_zero():
    q, K, V, _ = _case(4, 3, 2, 1)
    O, lse, _, _ = wo.attention(q, K[:0], V[:0], [-3, -2, -1], 0, 0)
    assert (O == 0).all() and np.isneginf(lse).all()
    O, lse, _, _ = wo.attention(q, K, V, [-1, 0, 1], 1, 0)
    assert (O[0] == 0).all() and np.isneginf(lse[0]).all()
    np.testing.assert_allclose(O[1], np.repeat(V[0], 2, 0))   # only itself


def test_tables_by_hand():
    # pages of 4: request 0 holds page 7 with 3 tokens and adds 3 (fills it, then
    # takes one page); request 1 is new with 1 token; request 2 adds nothing
    table, cu, lens, slots, pos, left, fine = wo.paged_tables(
        [3, 0, 4], [3, 1, 0], [10, 11, 12], [[7, -1], [-1, -1], [9, -1]], 4, 6)
    assert table == [[7, 12], [11, -1], [9, -1]] and left == 1 and fine
    assert cu == [0, 3, 4, 4] and lens == [6, 1, 4]
    assert slots == [7 * 4 + 3, 12 * 4, 12 * 4 + 1, 11 * 4, -1, -1]
    assert pos == [3, 4, 5, 0, -1, -1]


def test_tables_take_no_page_for_a_column_that_the_table_lacks():
    # pages of 4, two columns: request 0 takes one page for 9 tokens past its
    # first 3, request 1 gets the next
    table, cu, lens, slots, pos, left, fine = wo.paged_tables(
        [3, 0], [9, 1], [10, 11, 12], [[7, -1], [-1, -1]], 4, 10)
    assert table == [[7, 12], [11, -1]] and left == 1 and not fine
    assert slots == [31, 48, 49, 50, 51, -1, -1, -1, -1, 44] and lens == [12, 1]
