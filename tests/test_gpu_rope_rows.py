"""GPU tests of the rotary append for packed rows with positions of their own, and of queries
rotated in place, against the float64 oracle.  Tolerances: tests/test_gpu_rope.py."""

from __future__ import annotations

import numpy as np
import pytest

import oracle
from paged_kv_decode_24_gb300 import binding

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from tests.diff import DT, Case, Device, f64, rope_table  # noqa: E402
from tests.test_gpu_rope import close16, run  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib(lib):
    return lib


def check(c, d, q, rows, interleaved):
    places = oracle.row_places(c.lens, c.qs, c.table.numpy())
    close16(f64(q), f64(c.q), rows, interleaved, c.dtype)
    close16(f64(d.k_pages)[places[:, 0], :, places[:, 1]], f64(c.k_new), rows, interleaved, c.dtype)
    assert np.array_equal(f64(d.v_pages)[places[:, 0], :, places[:, 1]], f64(c.v_new))


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dim,rot,interleaved", [(128, 128, False), (64, 32, True)])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_packed_rows_with_positions_of_their_own(dtype, dim, rot, interleaved, in_place):
    """Positions in any order, equal ones among them, the table's first and last; the cache's places
    stay those of the tokens."""
    c = Case([40, 0, 33, 129, 7], [7, 0, 33, 1, 7], pairs=2, group=2, dim=dim, dtype=dtype, seed=rot)
    table = rope_table(301, rot)
    positions = np.random.default_rng(1).integers(0, 301, c.T)
    positions[[0, 1, -1]] = 300, 0, 0
    d = Device(c).make_prefill_plan()
    q = run(d, binding.Rope(table.cuda(), interleaved), True, positions=positions.tolist(),
            q_out=d.q if in_place else None)
    assert d.done() == 0 and (q.data_ptr() == d.q.data_ptr()) == in_place
    check(c, d, q, table.double().numpy()[positions], interleaved)


def test_packed_rows_whose_position_is_not_in_the_table():
    c = Case([40, 33], [7, 33], pairs=1, group=2, dim=64, seed=1)
    table = rope_table(50, 64)
    positions = np.arange(40)
    positions[3], positions[20] = -1, 50
    d = Device(c).make_prefill_plan()
    q = run(d, binding.Rope(table.cuda()), True, positions=positions.tolist())
    assert d.done() == binding.PA_DEV_BAD_POSITION
    lost = np.isin(np.arange(40), [3, 20])
    assert bool(torch.isnan(q[torch.from_numpy(lost)]).all())
    places = oracle.row_places(c.lens, c.qs, c.table.numpy())
    close16(f64(q)[~lost], f64(c.q)[~lost], table.double().numpy()[positions[~lost]], False, "fp16")
    for pool, old, new in ((d.k_pages, c.k_pages, None), (d.v_pages, c.v_pages, c.v_new)):
        at = places[lost]
        assert np.array_equal(f64(pool)[at[:, 0], :, at[:, 1]], f64(old)[at[:, 0], :, at[:, 1]])   # as it was
        if new is not None:
            at = places[~lost]
            assert np.array_equal(f64(pool)[at[:, 0], :, at[:, 1]], f64(new)[~lost])


@pytest.mark.parametrize("tokens", [False, True])
def test_a_single_row_in_place_inside_a_wider_one(tokens):
    """One token's queries, keys and values side by side in one row, the queries rotated where they are."""
    c = Case([77], [1], pairs=2, group=4, dim=128, dtype="bf16", seed=2)
    d = Device(c)
    if tokens:
        d.make_prefill_plan()
    wq, wk = c.hq * c.dim, c.kv * c.dim
    row = torch.cat([d.q.flatten(1), d.k_new.flatten(1), d.v_new.flatten(1)], 1)
    before = row.clone()
    q, k, v = (x.unflatten(1, (-1, c.dim)) for x in row.split([wq, wk, wk], 1))
    table = rope_table(80, 128)
    args = (binding.Rope(table.cuda()), q, k, v, q, d.k_pages, d.v_pages, d.table, d.seq_lens)
    if tokens:
        binding.rope_append_tokens(d.shape, d.plan, *args, d.ws, d.status)
    else:
        binding.rope_append(d.shape, *args, d.status)
    assert d.done() == 0
    check(c, d, q, table.double().numpy()[[76]], False)
    assert torch.equal(row[:, wq:], before[:, wq:])       # keys and values stay


def test_several_rows_in_place_inside_wider_ones_are_refused():
    c = Case([77, 5], pairs=2, group=4, dim=128, dtype="bf16", seed=2)
    d = Device(c)
    row = torch.zeros(2, (c.hq + 2 * c.kv) * c.dim, dtype=DT["bf16"], device="cuda")
    q, k, v = (x.unflatten(1, (-1, c.dim)) for x in row.split([c.hq * c.dim, c.kv * c.dim, c.kv * c.dim], 1))
    with pytest.raises((ValueError, binding.PagedAttnError)):
        binding.rope_append(d.shape, binding.Rope(rope_table(80, 128).cuda()), q, k, v, q, d.k_pages, d.v_pages,
                            d.table, d.seq_lens, d.status)
