"""What the bounds of the differential-attention tests reject, without a GPU: outputs that
are wrong, and weights that were rounded to fewer bits than the kernels keep.  The kernels'
arithmetic is modelled in float64 with the weights' rounding alone."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from tests.diff import DT, PAGE, Case, check_sink, exact_case, exact_want, f64, sink


def rounded(x, dtype, factor, parts):
    """x kept in `parts` numbers of the element type, times a factor."""
    x, y = x * factor, np.zeros_like(x)
    for _ in range(parts):
        y = y + f64(torch.from_numpy(x - y).to(DT[dtype]))
    return y / factor


def model(c, factor, parts, joint=False):
    """Outputs [T][H][2D] in the element type, weights kept in `parts` parts of `factor` times their
    size: each map's relative to its maximum (one token), or the difference of both
    (`joint`, several tokens)."""
    out, lam = np.zeros((c.T, c.heads, 2 * c.dim)), f64(c.lam)
    q, k, v, row = f64(c.q), f64(c.k_pages), f64(c.v_pages), 0
    for b, (n, new) in enumerate(zip(c.lens, c.qs)):
        t = np.arange(n)
        page = c.table.numpy()[b, t // PAGE]
        for i in range(new):
            seen = t <= n - new + i
            for h in range(c.heads):
                p = h // c.group
                values = np.concatenate([v[page, 2 * p + m, t % PAGE] for m in (0, 1)], 1)[seen]
                ws = []
                for m in (0, 1):
                    s = k[page, 2 * p + m, t % PAGE][seen] @ q[row, 2 * h + m] * c.scale
                    w = np.exp(s - s.max())
                    if not joint:
                        w = rounded(w, c.dtype, factor, parts) / w.sum()
                    else:
                        w = w / w.sum()
                    ws.append(w)
                d = ws[0] - lam[h] * ws[1]
                out[row, h] = (rounded(d, c.dtype, factor, parts) if joint else d) @ values
            row += 1
    if c.eps > 0:
        out /= np.sqrt(np.mean(out * out, -1, keepdims=True) + c.eps)
    w = 1.0 if c.weight is None else f64(c.weight)
    return torch.from_numpy(c.factor * w * out).to(DT[c.dtype])


def accepted(check):
    try:
        check()
    except AssertionError:
        return False
    return True


@pytest.mark.parametrize("scale", [1e-3, 0.5, 1e4, 1e6])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_exact_scores_reject_wrong_outputs(scale, dtype):
    c = exact_case(scale, dtype, [90, 3, 17])
    want = exact_want(c)
    got = model(c, 1.0, 2)
    c.check(got, want, True)
    wrong = [torch.zeros_like(got), -got, got.flip(1), got.flip(0), got.roll(1, -1), 1.01 * got]
    for i, x in enumerate(wrong):
        assert not accepted(lambda: c.check(x, want, True)), i


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_exact_scores_reject_a_missing_second_part(dtype):
    c = exact_case(0.5, dtype, [90, 3, 17])
    assert not accepted(lambda: c.check(model(c, 1.0, 1), exact_want(c), True))


@pytest.mark.parametrize("n", [1040, 2500])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_equal_weights_reject_a_missing_second_part(dtype, n):
    from tests.diff import HALF_STEP
    c = Case([n], [2], pairs=1, dtype=dtype, seed=5, eps=0.0, factor=1.0, weight=False, lam=-0.98 * HALF_STEP[dtype])
    c.q.zero_()
    c.v_pages.copy_((1 + c.v_pages.float() / 8).to(DT[dtype]))
    want = c.want()
    c.check(model(c, 2.0**14 if dtype == "fp16" else 1.0, 2, joint=True), want, True)
    # relative to the row's largest coefficient a weight is 1 - lambda
    assert not accepted(lambda: c.check(model(c, n, 1, joint=True), want, True))


@pytest.mark.parametrize("gap", [16, 20, 24, 28])
def test_a_sink_rejects_weights_without_room_below_them(gap):
    """fp16 weights of a largest 1 have their smallest step 24 log2 units below it; with 2^15 of it
    (one token), or 2^14 of a whole row's weight (several), they pass."""
    one, several = sink(gap, "fp16", 64, 1, [300, 40], [1, 1]), sink(gap, "fp16", 64, 1, [300, 40], [3, 5])
    check_sink(one, model(one, 2.0**15, 2))
    check_sink(several, model(several, 2.0**14, 2, joint=True))
    assert not accepted(lambda: check_sink(one, model(one, 1.0, 2)))
    assert not accepted(lambda: check_sink(one, torch.zeros(2, 1, 128)))
    b = sink(gap, "bf16", 64, 1, [300, 40], [1, 1])
    check_sink(b, model(b, 1.0, 2))
    assert not accepted(lambda: check_sink(b, model(b, 1.0, 2).flip(0) * 1.1))
