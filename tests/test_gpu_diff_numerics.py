"""GPU tests of differential attention where small weights, lost rows and long waits
show: through the binding, against the float64 oracle.  Tolerances: tests/diff.py,
and beside the cases that have exact scores."""

from __future__ import annotations

import numpy as np
import pytest

from paged_kv_decode_24_gb300 import binding

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from tests.diff import DT, HALF_STEP, PAGE, Case, Device, check_sink, exact_case, exact_want, f64, sink  # noqa: E402


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
# queries that are not numbers

def poisoned(c, marks):
    """The case's outputs with NaN in queries of map m of head h of row r, marks = (r, h, m)."""
    want = c.want()
    for r, h, m in marks:
        c.q[r, 2 * h + m, 5] = float("nan")
    return want


def check_poisoned(c, got, want, marks):
    g = f64(got)
    lost = np.zeros(g.shape[:2], bool)
    for r, h, _ in marks:
        lost[r, h] = True
    assert np.isnan(g[lost]).all()
    out, o, base, size = want
    keep = np.where(lost[..., None], out, g)     # the others are as they would be
    c.check(torch.from_numpy(keep), (out, o, base, size), True)


@pytest.mark.parametrize("group,dim", [(1, 64), (4, 128), (8, 64)])
@pytest.mark.parametrize("splits", [1, 3, 12])
def test_decode_shows_queries_that_are_not_numbers(group, dim, splits):
    c = Case([300, 40, 1, 77], pairs=2, group=group, dim=dim, seed=3, poison=True)
    marks = [(0, 0, 0), (1, c.heads - 1, 1), (2, c.heads // 2, 0)]
    want = poisoned(c, marks)
    d = Device(c).make_plan(forced_splits=splits)
    got = d.decode()
    assert d.done() == 0
    check_poisoned(c, got, want, marks)


@pytest.mark.parametrize("group,dim", [(1, 64), (4, 128), (8, 64)])
@pytest.mark.parametrize("splits", [1, 2])
def test_decode_of_many_short_sequences_shows_queries_that_are_not_numbers(group, dim, splits):
    """Tasks of one warp each."""
    c = Case([20 + i % 60 for i in range(900)], pairs=3, group=group, dim=dim, seed=4)
    marks = [(0, 0, 1), (500, c.heads - 1, 0)]
    for r, h, m in marks:
        c.q[r, 2 * h + m, 5] = float("nan")
    d = Device(c).make_plan(forced_splits=splits)
    assert d.plan.c.num_shared_ctas < d.plan.c.num_ctas
    got = d.decode()
    assert d.done() == 0
    lost = torch.isnan(got).all(-1)
    assert torch.equal(lost, torch.isnan(got).any(-1)) and int(lost.sum()) == 2
    assert all(bool(lost[r, h]) for r, h, _ in marks)


@pytest.mark.parametrize("group,dim", [(1, 64), (4, 128)])
def test_prefill_shows_queries_that_are_not_numbers(group, dim):
    c = Case([300, 40], [70, 40], pairs=2, group=group, dim=dim, seed=3, poison=True)
    marks = [(0, 0, 0), (75, c.heads - 1, 1), (109, 1, 0)]
    want = poisoned(c, marks)
    d = Device(c).make_prefill_plan()
    got = d.prefill()
    assert d.done() == 0
    check_poisoned(c, got, want, marks)


# --------------------------------------------------------------------------
# another plan's partials

def test_decode_joins_no_partials_of_another_plan():
    """Two plans with as many tasks, groups and partials, dealt to other CTAs: a call with the
    one, over a workspace that holds the other and its partials, writes nothing."""
    short, long = Case([160] * 20, pairs=2, group=2, dim=64, seed=1), Case([1920] * 20, pairs=2, group=2, dim=64, seed=1)
    shape = binding.make_shape(20, 8, 4, 64, PAGE, long.max_pages, long.num_pages, "fp16")
    d = Device(long).make_plan(sms=8, forced_splits=10)
    other = binding.DiffPlan(shape, short.lens, 8, forced_splits=10)
    for name in ("num_work_items", "num_groups", "num_split_items", "workspace_bytes"):
        assert getattr(other.c, name) == getattr(d.plan.c, name)
    assert other.c.num_ctas != d.plan.c.num_ctas and other.c.max_splits > 8
    d.decode()                                    # its partials stay in the workspace
    assert d.done() == 0
    d.plan = other
    got = d.decode()
    assert d.done() == binding.PA_DEV_PLAN_MISMATCH
    assert bool(torch.isnan(got).all())


def test_decode_joins_nothing_where_a_split_does_not_fit():
    """The workspace holds a plan of longer sequences, otherwise alike: their last splits lie past
    the call's block table.  What an earlier call left of those splits is not joined."""
    long, short = Case([1920] * 3, pairs=2, group=2, dim=64, seed=1), Case([1600] * 3, pairs=2, group=2, dim=64, seed=1)
    d, e = Device(long).make_plan(forced_splits=10), Device(short).make_plan(forced_splits=10)
    for name in ("num_work_items", "num_groups", "num_split_items", "num_ctas", "num_shared_ctas", "workspace_bytes"):
        assert getattr(e.plan.c, name) == getattr(d.plan.c, name)
    assert long.max_pages > 120 > short.max_pages
    d.decode()
    assert d.done() == 0
    e.ws = d.ws
    got = e.decode()
    assert e.done() == binding.PA_DEV_PLAN_MISMATCH
    assert bool(torch.isnan(got).all())


# --------------------------------------------------------------------------
# waits

@pytest.mark.parametrize("dim,group", [(64, 1), (128, 4)])
def test_prefill_limits_one_wait_and_not_a_pass(dim, group):
    """A context whose first pass alone takes milliseconds, with a limit far below that and far
    above any single copy or product: no wait runs out while stages keep moving."""
    n = 1 << 18
    c = Case([n], [2], pairs=1, group=group, dim=dim, seed=2)
    d = Device(c).make_prefill_plan()
    want = d.prefill()
    assert d.done() == 0
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    d.prefill()
    end.record()
    assert d.done() == 0
    limit = 300_000
    assert start.elapsed_time(end) * 1e6 > 4 * limit
    d.make_prefill_plan(wait_limit_ns=limit)
    got = d.prefill()
    assert d.done() == 0
    assert torch.equal(got, want)


def cold():
    """Nothing of what a call reads is left in L2."""
    torch.empty(512 << 20, dtype=torch.uint8, device="cuda").fill_(1)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("splits", [0, 3])
def test_decode_gives_up_at_a_limit_below_any_copy(dim, splits):
    """As many pages as keep memory busy, so that copies are waited for."""
    c = Case([3000] * 40, pairs=2, group=4, dim=dim, dtype="bf16", seed=7)
    d = Device(c).make_plan(forced_splits=splits)
    want = d.decode()
    assert d.done() == 0
    plan, ws = d.plan, d.ws
    d.make_plan(forced_splits=splits, wait_limit_ns=1)
    cold()
    got = d.decode()
    assert d.done() == binding.PA_DEV_TIMEOUT
    written = ~torch.isnan(got).all(-1)
    assert not bool(written.all()) and torch.equal(got[written], want[written])
    d.status.zero_()
    d.plan, d.ws = plan, ws
    assert torch.equal(d.decode(), want) and d.done() == 0


@pytest.mark.parametrize("dim", [64, 128])
def test_prefill_gives_up_at_a_limit_below_any_copy(dim):
    c = Case([1500, 40, 700], [400, 40, 1], pairs=2, group=2, dim=dim, dtype="bf16", seed=7)
    d = Device(c).make_prefill_plan()
    want = d.prefill()
    assert d.done() == 0
    plan = d.plan
    d.make_prefill_plan(wait_limit_ns=1)
    cold()
    got = d.prefill()
    assert d.done() == binding.PA_DEV_TIMEOUT
    missing = torch.isnan(got)
    assert bool(missing.any()) and torch.equal(missing.any(-1), missing.all(-1))
    assert torch.equal(got[~missing], want[~missing])
    d.status.zero_()
    d.plan = plan
    binding.prefill_upload(plan, d.ws)
    assert torch.equal(d.prefill(), want) and d.done() == 0


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
