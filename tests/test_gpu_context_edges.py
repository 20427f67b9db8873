"""Serving operators for long contexts and drafted tokens at the edges of what
their arguments allow.
"""
import numpy as np
import pytest
import torch

from oracle import context_oracle as co
from test_gpu_context import BF, F, f64, gsi, i32, verify_case  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ drafts
@pytest.mark.parametrize("V", [2**18 - 1, 2**18, 2**18 + 1, 300_001])
@pytest.mark.parametrize("tdt,ddt", [(F, F), (BF, BF), (BF, None)])
def test_verify_rows_of_more_mass_than_64_bits_hold(gsi, V, tdt, ddt):  # noqa: F811
    # tokens of 1 each: 2^18 of them are 2^64 of the sums' units, of 2^-46
    def ones(target, draft, tokens, u, v):
        target[:] = 1.0
        u[:] = 1.0  # the certain draft, and the one of 1, do not stand
        if draft is not None:
            draft[:] = 0.0
            draft[:-1].scatter_(1, tokens[1:, None].long(), 1.0)
    got = verify_case(gsi, [0, 1, 2], V, tdt, ddt, seed=V % 7, edit=ones)
    assert got.accepted.tolist() == [0, 0, 0] and got.out[0] >= 0


@pytest.mark.parametrize("R", [1, 400])  # one row over eight CTAs, and in one
def test_verify_the_widest_row(gsi, R):  # noqa: F811
    V, skip = 2**24, 2**20 + 77
    target = torch.ones(1, V, dtype=BF, device="cuda")
    target[0, :skip] = 0.0
    q_start = np.full(R + 1, 0)
    q_start[R:] = 1
    for v in (0.0, 0.3, 0.75, 0.9999, 1 - 2.0**-24):
        samples = torch.full((R,), v, device="cuda")
        got = gsi.verify_drafts(target, None, i32([0]), torch.zeros(1, device="cuda"), samples, i32(q_start))
        # the k-th of equal tokens is the first whose running sum, k + 1, is above v times their number
        assert got.out.tolist() == [skip + int(float(samples[0]) * (V - skip))], v


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("p,q,u,stands", [
    (0.5, NAN, 0.9, True), (0.0, NAN, 0.9, False),     # NaN counts as 0: 0 < p
    (0.5, -0.1, 1.0, True), (0.0, -0.1, 0.5, False),   # so does what is negative
    (-0.1, -0.5, 0.5, False), (NAN, 0.5, 0.0, False), (-0.2, 0.5, 0.0, False),
    (0.95, 2.0, 0.9, True), (0.85, 2.0, 0.9, False),   # above 1 counts as 1
    (INF, 2.0, 0.9, True), (3.0, 2.0, 1.0, False), (3.0, INF, 0.99, True), (1.0, INF, 1.0, False)])
@pytest.mark.parametrize("dt", [F, BF])
def test_verify_takes_a_draft_by_what_its_probabilities_count_as(gsi, p, q, u, stands, dt):  # noqa: F811
    target = torch.tensor([[0.25, p, 0.25, 0.25], [1.0, 0.0, 0.0, 0.0]], device="cuda").to(dt)
    draft = torch.tensor([[0.0, q, 0.0, 0.0], [0.0] * 4], device="cuda").to(dt)
    us, v = torch.tensor([u, 0.0], device="cuda"), torch.tensor([0.999], device="cuda")
    got = gsi.verify_drafts(target, draft, i32([0, 1]), us, v, i32([0, 2]))
    assert got.accepted.tolist() == [int(stands)]
    want = co.verify(f64(target), f64(draft), [0, 1], us.tolist(), v.tolist(), [0, 2])
    assert got.out.tolist() == want[0] and want[1] == [int(stands)]
    if dt is F:  # a certain draft: its 1 against what the target's probability counts as
        got = gsi.verify_drafts(target, None, i32([0, 1]), us, v, i32([0, 2]))
        count = min(max(p, 0.0), 1.0) if p == p else 0.0
        assert got.accepted.tolist() == [int(float(us[0]) < count)]
