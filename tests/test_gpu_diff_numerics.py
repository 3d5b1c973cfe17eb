"""GPU tests of differential attention where small weights, lost rows and long waits
show: through the binding, against the float64 oracle.  Tolerances: tests/diff.py,
and beside the cases that have exact scores."""

from __future__ import annotations

import pytest

from paged_kv_decode_24_gb300 import binding

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from tests.diff import DT, HALF_STEP, Case, Device, check_sink, exact_case, exact_want, sink  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib(lib):
    return lib


# --------------------------------------------------------------------------
# both parts of the weights

@pytest.mark.parametrize("lens,qs", [([1040], [16]), ([2500], [70]), ([1024, 1025, 1026], [130, 130, 130])],
                         ids=lambda x: "_".join(map(str, x)))
@pytest.mark.parametrize("dim,group", [(64, 1), (64, 4), (128, 2), (128, 8)])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_prefill_keeps_two_parts_of_the_weights_at_every_length(lens, qs, dim, group, dtype):
    """Queries of zero: every weight of a row is (1 - lambda) / n, with lambda such that
    rounding 1 - lambda to the element type is off by nearly half a step.  All weights of a row
    are off alike then, so nothing averages, and values around 1 leave that error whole."""
    u = HALF_STEP[dtype]
    c = Case(lens, qs, pairs=1, group=group, dim=dim, dtype=dtype, seed=5, eps=0.0, factor=1.0, weight=False,
             lam=-0.98 * u)
    c.q.zero_()
    c.v_pages.copy_((1 + c.v_pages.float() / 8).to(DT[dtype]))
    rows = sorted({0, 1, qs[0] - 1, sum(qs) // 2, sum(qs) - 1})
    d = Device(c).make_prefill_plan()
    got = d.prefill()
    assert d.done() == 0
    c.check(got, c.want(rows), True, rows=rows)
    assert bool(torch.isfinite(got).all())


@pytest.mark.parametrize("gap", [16, 20, 24, 28])
@pytest.mark.parametrize("dim,group", [(64, 1), (64, 8), (128, 4)])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_decode_of_small_weights_beside_a_sink(gap, dim, group, dtype):
    c = sink(gap, dtype, dim, group, [300, 40], [1, 1])
    for splits in (1, 3, 12):
        d = Device(c).make_plan(forced_splits=splits)
        got = d.decode()
        assert d.done() == 0
        check_sink(c, got)


@pytest.mark.parametrize("gap", [16, 20, 24, 28])
@pytest.mark.parametrize("dim,group", [(64, 1), (64, 8), (128, 4)])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_prefill_of_small_weights_beside_a_sink(gap, dim, group, dtype):
    c = sink(gap, dtype, dim, group, [300, 40], [3, 30])
    d = Device(c).make_prefill_plan()
    got = d.prefill()
    assert d.done() == 0
    check_sink(c, got)


# --------------------------------------------------------------------------
# exact scores: bounds that a wrong weight does not pass (tests/test_diff_bounds.py)

@pytest.mark.parametrize("scale", [1e-3, 0.5, 1e4, 1e6])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("dim,group", [(64, 2), (128, 8)])
def test_decode_of_exact_scores(scale, dtype, dim, group):
    c = exact_case(scale, dtype, [90, 3, 17], dim, group)
    for splits in (1, 2, 12):
        d = Device(c).make_plan(forced_splits=splits)
        got = d.decode()
        assert d.done() == 0
        c.check(got, exact_want(c), True, f"splits {splits}")
