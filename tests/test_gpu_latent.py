"""Latent attention on the GPU against the float64 oracle: append and gather
bit for bit, the absorbed and the expanded attention within the tolerance
derived in tests/latent.py, and the four as one run."""

from __future__ import annotations

import zlib

import numpy as np
import pytest

import oracle
from paged_kv_decode_24_gb300 import binding

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from tests.latent import DT, LATENT, ROW, Case, Device, assert_latent_close, f64  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib(lib):
    return lib


def seed_of(*x):
    return zlib.crc32(str(x).encode())


def bits(t):
    return t.cpu().view(torch.int16)


# ---- append and gather

ROWS_CASES = [([1], [1]), ([16, 17, 1, 300], [16, 3, 1, 0]), ([0, 5, 0, 129, 64], [0, 5, 0, 64, 1]),
              ([33] * 70, [1] * 70), ([1000, 2049], [1000, 1025])]


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("case", ROWS_CASES, ids=lambda c: f"B{len(c[0])}_T{sum(c[1])}")
def test_append_and_gather_are_bit_exact(case, page):
    c = Case(*case, heads=1, page=page, dtype="bf16", seed=seed_of(case, page))
    d = Device(c)
    d.append()
    rows = d.gather()
    assert d.done() == 0
    table = c.table.numpy()
    want = oracle.latent_append(c.pages.view(torch.int16).numpy(), c.c_new.view(torch.int16).numpy(),
                                c.r_new.view(torch.int16).numpy(), table, c.lens, c.qs)
    assert np.array_equal(bits(d.pages).numpy(), want)     # every other row as it was
    assert np.array_equal(bits(rows).numpy(), oracle.latent_gather(want, table, c.lens))


def test_append_takes_slices_of_a_wider_projection():
    c = Case([40, 9], [7, 9], heads=1, seed=3)
    d = Device(c)
    wide = torch.randn(c.T, 1000, device="cuda").half()
    d.c_new, d.r_new = wide[:, 8:8 + LATENT], wide[:, 904:904 + 64]
    d.append()
    assert d.done() == 0
    want = oracle.latent_append(f64(c.pages), f64(d.c_new.cpu()), f64(d.r_new.cpu()),
                                c.table.numpy(), c.lens, c.qs)
    assert np.array_equal(f64(d.pages.cpu()), want)


def test_rows_of_a_bad_page_are_skipped_and_flagged():
    c = Case([50, 20], [50, 4], heads=1, seed=4)
    c.table[0, 1] = c.num_pages
    d = Device(c)
    d.append()
    assert d.done() == binding.PA_DEV_BAD_PAGE
    d.status.zero_()
    rows = d.gather().cpu()
    assert d.done() == binding.PA_DEV_BAD_PAGE
    assert torch.all(rows[16:32] == 0) and torch.equal(rows[:16, :LATENT], c.c_new[:16])
    assert torch.equal(rows[32:50, :LATENT], c.c_new[32:50])


# ---- absorbed attention

ABSORBED = [
    # lens, q_lens, heads, page
    ([1], [1], 1, 16),
    ([1, 2, 15, 16, 17, 63, 64, 65], [1] * 8, 16, 16),
    ([300, 0, 129, 1000], [1, 0, 1, 1], 16, 32),
    ([100, 64], [5, 3], 3, 64),                   # rows of several tokens in a tile, 9 and 15 rows
    ([70, 513], [7, 2], 20, 128),                 # tiles that begin inside a token
    ([257, 31], [1, 31], 128, 64),
    ([2000, 333], [1, 4], 40, 16),
    ([129, 128, 127, 192], [1, 2, 1, 1], 64, 32),  # ends at and around a stage of 128
]


# the kernels: 16-row tiles (mma.sync), 64-row tiles (tcgen05), 128-row tiles on SM pairs (tcgen05)
all_kernels = pytest.mark.parametrize("rows", [16, 64, 128], ids=["mma_sync", "tcgen05", "tcgen05_pair"])


@all_kernels
@pytest.mark.parametrize("splits", [0, 3])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("case", ABSORBED, ids=lambda c: f"L{c[0][:3]}_q{c[1][:2]}_H{c[2]}_S{c[3]}")
def test_absorbed_parity(case, dtype, splits, rows):
    lens, qs, heads, page = case
    c = Case(lens, qs, heads=heads, page=page, dtype=dtype, seed=seed_of(case), poison=True)
    d = Device(c, forced_splits=splits, rows_per_tile=rows)
    assert d.plan.c.rows_per_tile == rows
    out = d.attention()
    assert d.done() == 0
    want = oracle.latent_attention(f64(c.q), f64(c.pages), c.table.numpy(), lens, qs, c.scale)
    assert_latent_close(out.double().cpu().numpy(), want, max(lens), dtype, str(case))


@all_kernels
def test_absorbed_planner_splits_and_reruns_give_the_same_bits(rows):
    c = Case([20000, 777], [1, 1], heads=16, page=64, dtype="bf16", seed=8)
    d = Device(c, rows_per_tile=rows)
    assert d.plan.c.num_merges >= 1
    a, b = d.attention(), d.attention()
    assert d.done() == 0
    assert torch.equal(bits(a), bits(b))
    want = oracle.latent_attention(f64(c.q), f64(c.pages), c.table.numpy(), c.lens, c.qs, c.scale)
    assert_latent_close(a.double().cpu().numpy(), want, 20000, "bf16")


@all_kernels
@pytest.mark.parametrize("splits", [0, 2])
def test_absorbed_bad_pages_are_left_out(splits, rows):
    """One page of a sequence, every page of another (its rows get zeros)."""
    c = Case([200, 40, 90], [2, 1, 1], heads=5, page=16, seed=9)
    c.table[0, 3] = -1
    c.table[1, :3] = c.num_pages + 9
    d = Device(c, forced_splits=splits, rows_per_tile=rows)
    out = d.attention()
    assert d.done() == binding.PA_DEV_BAD_PAGE
    want = oracle.latent_attention(f64(c.q), f64(c.pages), c.table.numpy(), c.lens, c.qs, c.scale,
                                   bad_pages=[(0, 3), (1, 0), (1, 1), (1, 2)])
    assert_latent_close(out.double().cpu().numpy(), want, 200, "fp16")
    assert torch.all(out[2] == 0)


@all_kernels
@pytest.mark.parametrize("scale", [1e-4, 1.0])
def test_absorbed_scale_extremes(scale, rows):
    """Near-uniform weights, and weights that are almost one-hot with scores of
    hundreds (the running maximum moves)."""
    c = Case([1200], [1], heads=16, page=16, seed=10, scale=scale)
    d = Device(c, rows_per_tile=rows)
    out = d.attention()
    assert d.done() == 0
    want = oracle.latent_attention(f64(c.q), f64(c.pages), c.table.numpy(), c.lens, c.qs, scale)
    assert_latent_close(out.double().cpu().numpy(), want, 1200, "fp16")


@all_kernels
def test_absorbed_offsets_past_32_bits(rows):
    """Pages beyond 2^31 elements (and 4 GB) of the pool."""
    pages = 2**32 // (16 * ROW * 2) + 40000       # 5 GB
    c = Case([100, 300], [3, 1], heads=16, seed=11)
    base = pages - c.num_pages
    d = Device(c, rows_per_tile=rows)
    big = torch.empty(pages, 16, ROW, dtype=torch.float16, device="cuda")
    big[base:] = d.pages
    assert base * 16 * ROW > 2**31
    d.pages, d.shape.num_pages = big, pages
    d.table = torch.where(d.table >= 0, d.table + base, d.table)
    d.append()
    rows, out = d.gather(), d.attention()
    assert d.done() == 0
    after = oracle.latent_append(f64(c.pages), f64(c.c_new), f64(c.r_new), c.table.numpy(), c.lens,
                                 c.qs)
    assert np.array_equal(f64(rows.cpu()), oracle.latent_gather(after, c.table.numpy(), c.lens))
    want = oracle.latent_attention(f64(c.q), after, c.table.numpy(), c.lens, c.qs, c.scale)
    assert_latent_close(out.double().cpu().numpy(), want, 300, "fp16")


@all_kernels
@pytest.mark.parametrize("splits", [1, 2])
def test_absorbed_buffers_aligned_to_16_bytes_only(splits, rows):
    c = Case([300, 70], [2, 1], heads=12, page=16, seed=23)
    d = Device(c, forced_splits=splits, rows_per_tile=rows)

    def shifted(t):   # the same contents 16 bytes off a 256-byte boundary
        n = 16 // t.element_size()
        big = torch.empty(t.numel() + n, dtype=t.dtype, device="cuda")
        big[n:] = t.flatten()
        return big[n:].view(t.shape)

    d.q, d.pages, d.ws = shifted(d.q), shifted(d.pages), shifted(d.ws)
    assert all(t.data_ptr() % 32 == 16 for t in (d.q, d.pages, d.ws))
    torch.cuda.synchronize()   # calls may read the plan before the kernel ahead has ended
    out = shifted(torch.full((c.T, 12, LATENT), float("nan"), dtype=DT["fp16"], device="cuda"))
    d.attention(out)
    assert d.done() == 0
    want = oracle.latent_attention(f64(c.q), f64(c.pages), c.table.numpy(), c.lens, c.qs, c.scale)
    assert_latent_close(out.double().cpu().numpy(), want, 300, "fp16")


# ---- expanded attention

EXPANDED = [
    # lens, q_lens, heads, head_dim
    ([1], [1], 1, 64),
    ([1, 2, 63, 64, 65, 0, 130], [1, 2, 63, 64, 65, 0, 130], 3, 128),
    ([300, 129, 1000], [64, 129, 1], 5, 64),
    ([513, 700], [513, 257], 2, 128),
    ([260, 300], [255, 256], 4, 128),
    ([1500], [511], 3, 64),
]


@pytest.mark.parametrize("rows", [128, 256])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("case", EXPANDED, ids=lambda c: f"L{c[0][:3]}_q{c[1][:2]}_H{c[2]}_D{c[3]}")
def test_expanded_parity(case, dtype, rows):
    lens, qs, heads, hd = case
    c = Case(lens, qs, heads=heads, head_dim=hd, dtype=dtype, seed=seed_of(case))
    d = Device(c, form="expanded", rows_per_tile=rows)
    out = d.prefill()
    assert d.done() == 0
    want = oracle.latent_prefill(f64(c.qx), f64(c.k), f64(c.rows[:, LATENT:]), f64(c.v), lens, qs,
                                 c.scale)
    assert_latent_close(out.double().cpu().numpy(), want, max(lens), dtype, str(case))


def test_expanded_takes_other_strides():
    """Head-major keys, dense values, a dense rotary key."""
    c = Case([90, 200], [90, 33], heads=3, head_dim=64, seed=12)
    d = Device(c, form="expanded")
    d.k = d.k.transpose(0, 1).contiguous().transpose(0, 1)
    d.v = d.v.contiguous()
    d.k_rope = d.k_rope.contiguous()
    out = d.prefill()
    assert d.done() == 0
    want = oracle.latent_prefill(f64(c.qx), f64(c.k), f64(c.rows[:, LATENT:]), f64(c.v), c.lens,
                                 c.qs, c.scale)
    assert_latent_close(out.double().cpu().numpy(), want, 200, "fp16")


@pytest.mark.parametrize("rows", [128, 256])
def test_expanded_other_sequences_never_leak(rows):
    """The neighbours of a sequence in the packed rows hold NaN and infinity:
    its own output stays finite and right."""
    c = Case([100, 77, 100], [100, 50, 100], heads=2, head_dim=128, seed=13)
    for x in (c.kv, c.rows):
        x[:100] = float("nan")
        x[177:] = float("inf")
    d = Device(c, form="expanded", rows_per_tile=rows)
    out = d.prefill()[100:150]
    assert d.done() == 0
    s = slice(100, 177)
    want = oracle.latent_prefill(f64(c.qx[100:150]), f64(c.k[s]), f64(c.rows[s, LATENT:]),
                                 f64(c.v[s]), [77], [50], c.scale)
    assert_latent_close(out.double().cpu().numpy(), want, 77, "fp16")


@pytest.mark.parametrize("rows", [128, 256])
@pytest.mark.parametrize("scale", [1e-4, 2.0])
def test_expanded_scale_extremes(scale, rows):
    c = Case([700], [700], heads=2, seed=14, scale=scale)
    d = Device(c, form="expanded", rows_per_tile=rows)
    out = d.prefill()
    assert d.done() == 0
    want = oracle.latent_prefill(f64(c.qx), f64(c.k), f64(c.rows[:, LATENT:]), f64(c.v), c.lens, c.qs,
                                 scale)
    assert_latent_close(out.double().cpu().numpy(), want, 700, "fp16")


# ---- together

def test_the_two_forms_agree_over_one_cache():
    """append -> gather -> expand -> prefill against absorbed queries over the
    same cache, with W (keys) and U (values) of each head: the two forms are the
    same attention."""
    lens, qs, H, D = [150, 75, 300], [150, 20, 64], 4, 128
    c = Case(lens, qs, heads=H, head_dim=D, page=32, seed=15)
    g = torch.Generator(device="cuda").manual_seed(1)
    W = torch.randn(H, D, LATENT, generator=g, device="cuda") * LATENT**-0.5
    U = torch.randn(H, D, LATENT, generator=g, device="cuda") * LATENT**-0.5
    e = Device(c, form="expanded")
    e.append()
    rows = e.gather()
    c64 = rows[:, :LATENT].double()
    e.k = torch.einsum("tc,hdc->thd", c64, W.double()).half()
    e.v = torch.einsum("tc,hdc->thd", c64, U.double()).half()
    e.k_rope = rows[:, LATENT:]
    x = e.prefill()
    assert e.done() == 0
    a = Device(c)
    a.pages = e.pages
    a.q = torch.cat([torch.einsum("thd,hdc->thc", e.qx[..., :D].double(), W.double()).half(),
                     e.qx[..., D:]], 2)
    lat = a.attention()
    assert a.done() == 0
    y = torch.einsum("thc,hdc->thd", lat.double(), U.double())
    # each form against its own 64-bit result above; here both against the other:
    # k, v, q' and the latent output are each rounded once to fp16 (2^-11), which
    # moves a score of size ~6 by a few 2^-11 of it
    rel = float((x.double() - y).norm() / y.norm())
    assert rel < 8 * 2.0**-11, rel


def test_decode_steps_over_a_growing_cache():
    """Prompt by the expanded form, then three decode steps: append one token,
    attend; each step's plan goes into the same workspace."""
    H, page = 16, 16
    final = [40, 131]
    c = Case(final, [1, 1], heads=H, page=page, seed=16, dtype="bf16")
    pool = c.pages.clone()
    ws = torch.empty(8 << 20, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dev_pages, table = pool.cuda(), c.table.cuda()
    for step in range(3):
        lens = [n - 2 + step for n in final]
        s = Case(final, [1, 1], heads=H, page=page, seed=100 + step, dtype="bf16")
        plan = binding.LatentPlan(c.shape(), lens, [1, 1], 152)
        binding.latent_upload(plan, ws)
        cn, rn, q = s.c_new.cuda(), s.r_new.cuda(), s.q.cuda()
        out = torch.empty(2, H, LATENT, dtype=DT["bf16"], device="cuda")
        binding.latent_append(c.shape(), plan, cn, rn, dev_pages, table, ws, status)
        binding.latent_attention(c.shape(), plan, q, dev_pages, table, c.scale, out, ws, status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        pool = oracle.latent_append(f64(pool) if step == 0 else pool, f64(s.c_new), f64(s.r_new),
                                    c.table.numpy(), lens, [1, 1])
        want = oracle.latent_attention(f64(s.q), pool, c.table.numpy(), lens, [1, 1], c.scale)
        assert_latent_close(out.double().cpu().numpy(), want, 131, "bf16", f"step {step}")


@all_kernels
def test_captured_step_replays_and_follows_a_new_upload(rows):
    """append + attention in a CUDA graph; between replays a plan of the same
    structure is uploaded (longer sequences), two graphs on workspaces of their
    own run on two streams at once."""
    lens0, lens1 = [120, 333], [125, 340]
    c = Case([128, 352], [1, 1], heads=16, page=16, seed=17)
    graphs = []
    for _ in range(2):
        d = Device(c, forced_splits=2)
        plans = [binding.LatentPlan(d.shape, x, [1, 1], 152, forced_splits=2, rows_per_tile=rows)
                 for x in (lens0, lens1)]
        d.ws = binding.alloc_workspace(plans[0])
        assert plans[0].c.blob_bytes == plans[1].c.blob_bytes
        d.plan = plans[0]
        d.out = torch.empty(2, 16, LATENT, dtype=DT["fp16"], device="cuda")
        binding.latent_upload(plans[0], d.ws)
        d.append()
        d.attention(d.out)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            d.append()
            d.attention(d.out)
        graphs.append((g, d, plans, torch.cuda.Stream()))
    pool = f64(c.pages)
    pool = oracle.latent_append(pool, f64(c.c_new), f64(c.r_new), c.table.numpy(), lens0, [1, 1])
    for i, lens in enumerate((lens0, lens1)):
        pool = oracle.latent_append(pool, f64(c.c_new), f64(c.r_new), c.table.numpy(), lens, [1, 1])
        want = oracle.latent_attention(f64(c.q), pool, c.table.numpy(), lens, [1, 1], c.scale)
        for g, d, plans, st in graphs:
            binding.latent_upload(plans[i], d.ws)
        torch.cuda.synchronize()
        for g, d, plans, st in graphs:
            with torch.cuda.stream(st):
                for _ in range(4):
                    g.replay()
        for g, d, plans, st in graphs:
            assert d.done() == 0
            assert_latent_close(d.out.double().cpu().numpy(), want, 352, "fp16")


def test_calls_on_another_stream():
    c = Case([500, 90], [1, 1], heads=16, seed=18)
    d = Device(c)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        a = d.attention()
    b = d.attention(stream=s)
    assert d.done() == 0
    assert torch.equal(bits(a), bits(b))


def test_workspace_of_another_plan_is_flagged():
    c = Case([100, 50], [1, 1], heads=16, seed=19)
    d = Device(c)
    other = Device(Case([100, 50, 60], [1, 1, 1], heads=16, seed=20))
    d.ws = torch.cat([other.ws, other.ws])
    torch.cuda.synchronize()   # calls may read the plan before the kernel ahead has ended
    out = d.attention()
    assert d.done() == binding.PA_DEV_PLAN_MISMATCH
    assert torch.all(torch.isnan(out))
    d.status.zero_()
    d.append()
    assert d.done() == binding.PA_DEV_PLAN_MISMATCH
    assert torch.equal(d.pages.cpu(), c.pages)


@all_kernels
@pytest.mark.parametrize("splits", [1, 4])
def test_waits_that_run_out_are_reported(splits, rows):
    """One nanosecond per wait: rows are left as they were or right, the status
    says so, and the next call with the default limit is right."""
    c = Case([900, 1500, 30], [1, 1, 1], heads=16, seed=21)
    d = Device(c, forced_splits=splits, rows_per_tile=rows, wait_limit_ns=1)
    out = d.attention()
    assert d.done() == binding.PA_DEV_TIMEOUT
    got = out.double().cpu().numpy()
    left = np.isnan(got).all(axis=-1)
    assert np.array_equal(left, np.isnan(got).any(axis=-1)) and left.any()
    want = oracle.latent_attention(f64(c.q), f64(c.pages), c.table.numpy(), c.lens, c.qs, c.scale)
    keep = tuple(x[~left] for x in want)
    assert_latent_close(got[~left], keep, 1500, "fp16")
    d2 = Device(c, forced_splits=splits, rows_per_tile=rows)
    out = d2.attention()
    assert d2.done() == 0
    assert_latent_close(out.double().cpu().numpy(), want, 1500, "fp16")


@pytest.mark.parametrize("rows", [128, 256])
def test_expanded_waits_that_run_out_are_reported(rows):
    c = Case([900, 300], [900, 40], heads=3, seed=22)
    d = Device(c, form="expanded", rows_per_tile=rows, wait_limit_ns=1)
    out = d.prefill()
    assert d.done() == binding.PA_DEV_TIMEOUT
    got = out.double().cpu().numpy()
    rows = np.isnan(got).all(axis=-1)
    assert np.array_equal(rows, np.isnan(got).any(axis=-1)) and rows.any()
    want = oracle.latent_prefill(f64(c.qx), f64(c.k), f64(c.rows[:, LATENT:]), f64(c.v), c.lens, c.qs,
                                 c.scale)
    assert_latent_close(got[~rows], tuple(x[~rows] for x in want), 900, "fp16")
    d2 = Device(c, form="expanded")
    out = d2.prefill()
    assert d2.done() == 0
    assert_latent_close(out.double().cpu().numpy(), want, 900, "fp16")


@pytest.mark.parametrize("seed", range(16))
def test_random_batches_against_the_oracle(seed):
    """Random lengths, new tokens, heads, pages, types, tile rows, splits and
    scales: append, rows read back, absorbed and expanded attention."""
    rng = np.random.default_rng(1000 + seed)
    B = int(rng.integers(1, 9))
    lens = [int(x) for x in np.exp(rng.uniform(0, np.log(900), B))]
    if rng.random() < 0.3:
        lens[int(rng.integers(B))] = 0
    qs = [int(min(n, rng.choice([0, 1, 1, 2, rng.integers(1, 300)]))) for n in lens]
    heads = int(rng.choice([1, 2, 7, 16, 33, 64, 100, 128]))
    qs = [q if q * heads < 3000 else 1 for q in qs]
    page, hd = int(rng.choice([16, 32, 64, 128])), int(rng.choice([64, 128]))
    dtype = str(rng.choice(["fp16", "bf16"]))
    c = Case(lens, qs, heads=heads, head_dim=hd, page=page, dtype=dtype, seed=seed, poison=True,
             scale=float(rng.uniform(0.01, 0.2)))
    what = f"{lens} {qs} H{heads} S{page} D{hd} {dtype}"
    after = oracle.latent_append(f64(c.pages), f64(c.c_new), f64(c.r_new), c.table.numpy(), lens, qs)
    want = oracle.latent_attention(f64(c.q), after, c.table.numpy(), lens, qs, c.scale)
    for rows in (0, 16, 64, 128):
        d = Device(c, rows_per_tile=rows, forced_splits=int(rng.choice([0, 0, 2, 5])))
        d.append()
        out = d.attention()
        assert d.done() == 0
        assert_latent_close(out.double().cpu().numpy(), want, max(lens), dtype, f"{what} rows {rows}")
    assert np.array_equal(np.nan_to_num(f64(d.gather().cpu())),
                          np.nan_to_num(oracle.latent_gather(after, c.table.numpy(), lens)))
    want = oracle.latent_prefill(f64(c.qx), f64(c.k), f64(c.rows[:, LATENT:]), f64(c.v), lens, qs, c.scale)
    for rows in (0, 128, 256):
        e = Device(c, form="expanded", rows_per_tile=rows)
        out = e.prefill()
        assert e.done() == 0
        assert_latent_close(out.double().cpu().numpy(), want, max(lens), dtype, f"{what} tiles {rows}")


def test_rows_behind_the_last_sequence_stay():
    """Buffers with room behind the batch's rows: the rest keeps its contents."""
    c = Case([70, 33], [3, 33], heads=5, head_dim=64, seed=24)
    for form in ("absorbed", "expanded"):
        d = Device(c, form=form)
        width = LATENT if form == "absorbed" else 64
        big = torch.full((c.T + 9, 5, width), 3.0, dtype=DT["fp16"], device="cuda")
        (d.attention if form == "absorbed" else d.prefill)(big[:c.T])
        rows = torch.full((c.Tk + 9, ROW), 3.0, dtype=DT["fp16"], device="cuda")
        binding.latent_gather(d.shape, d.plan, d.pages, d.table, rows[:c.Tk], d.ws, d.status)
        assert d.done() == 0
        assert torch.all(big[c.T:] == 3) and torch.all(rows[c.Tk:] == 3)
        assert not torch.any(torch.all(big[:c.T] == 3, dim=-1))


def test_expanded_captured_and_replayed_with_new_inputs():
    c = Case([500, 90], [500, 33], heads=2, seed=25)
    d = Device(c, form="expanded")
    out = d.prefill()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        d.prefill(out)
    other = Case([500, 90], [500, 33], heads=2, seed=26)
    for src, dst in ((other.qx, d.qx), (other.kv, d.kv), (other.rows, d.rows)):
        dst.copy_(src)
    out.fill_(float("nan"))
    for _ in range(3):
        g.replay()
    assert d.done() == 0
    want = oracle.latent_prefill(f64(other.qx), f64(other.k), f64(other.rows[:, LATENT:]), f64(other.v),
                                 c.lens, c.qs, c.scale)
    assert_latent_close(out.double().cpu().numpy(), want, 500, "fp16")


@all_kernels
def test_one_sequence_of_many_pieces(rows):
    """A sequence cut into more pieces than a warp has lanes."""
    c = Case([3000], [1], heads=16, page=64, dtype="bf16", seed=27)
    d = Device(c, rows_per_tile=rows, forced_splits=47)   # 64-token stages: 47, 128: 24
    out = d.attention()
    assert d.done() == 0
    assert d.plan.c.num_slots == min(47, -(-3000 // (128 if rows == 128 else 64)))
    want = oracle.latent_attention(f64(c.q), f64(c.pages), c.table.numpy(), c.lens, c.qs, c.scale)
    assert_latent_close(out.double().cpu().numpy(), want, 3000, "bf16")


@all_kernels
@pytest.mark.parametrize("batch,splits", [(1, 40), (8, 16), (20, 7), (40, 2), (9, 3)])
def test_merge_by_every_number_of_warps(batch, splits, rows):
    """Few and many rows, few and many pieces: 1, 2, 4 and 8 warps a row."""
    heads = {16: 16, 64: 48, 128: 100}[rows]
    c = Case([splits * 128] * batch, [1] * batch, heads=heads, page=32, seed=29 + splits)
    d = Device(c, rows_per_tile=rows, forced_splits=splits)
    out = d.attention()
    assert d.done() == 0 and d.plan.c.num_slots == batch * splits
    want = oracle.latent_attention(f64(c.q), f64(c.pages), c.table.numpy(), c.lens, c.qs, c.scale)
    assert_latent_close(out.double().cpu().numpy(), want, splits * 128, "fp16")
    assert torch.equal(d.attention(), out)


@pytest.mark.parametrize("rows", [128, 256])
def test_expanded_rows_to_clear_under_any_wait_limit(rows):
    """Neighbours that hold NaN behind the last visible token, and wait limits
    from none to longer than the call: every row of the sequence between is as it
    was or right, and a row that was left has its status."""
    c = Case([100, 333, 100], [100, 300, 100], heads=3, head_dim=128, seed=31)
    for x in (c.kv, c.rows):
        x[:100] = float("nan")
        x[433:] = float("nan")
    s = slice(100, 433)
    want = oracle.latent_prefill(f64(c.qx[100:400]), f64(c.k[s]), f64(c.rows[s, LATENT:]),
                                 f64(c.v[s]), [333], [300], c.scale)
    for limit in (1, 300, 1000, 2000, 3000, 5000, 8000, 20000, 10**9):
        d = Device(c, form="expanded", rows_per_tile=rows, wait_limit_ns=limit)
        out = torch.full((c.T, 3, 128), 7.0, dtype=DT["fp16"], device="cuda")
        d.prefill(out)
        status = d.done()
        got = out[100:400].double().cpu().numpy()
        left = (got == 7).all(axis=-1)
        assert status == (binding.PA_DEV_TIMEOUT if left.any() else status) and status in (0, 8)
        assert limit < 10**9 or (status == 0 and not left.any())
        if not left.all():
            assert_latent_close(got[~left], tuple(x[~left] for x in want), 333, "fp16", f"{limit} ns")


def test_pair_call_that_takes_longer_than_a_drain():
    """One pair of SMs works through eight long sequences, well over the 10 ms of
    the waits at a kernel's end: the call is right, and so is the next one."""
    lens, heads, page = [131072 - 77 * b for b in range(8)], 128, 128
    counts = [-(-n // page) for n in lens]
    g = torch.Generator(device="cuda").manual_seed(32)
    shape = binding.make_latent_shape(8, heads, 128, page, max(counts), sum(counts), "bf16")
    pages = torch.randn(sum(counts), page, ROW, generator=g, device="cuda").bfloat16()
    order = torch.randperm(sum(counts), generator=g, device="cuda").int()
    table = torch.full((8, max(counts)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = order[at:at + n]
        at += n
    q = torch.randn(8, heads, ROW, generator=g, device="cuda").bfloat16()
    plan = binding.LatentPlan(shape, lens, [1] * 8, 2)
    assert plan.c.num_ranges == 1 and plan.c.num_segments == 8
    ws = binding.alloc_workspace(plan)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.latent_upload(plan, ws)
    outs = []
    for _ in range(2):
        out = torch.full((8, heads, LATENT), float("nan"), dtype=torch.bfloat16, device="cuda")
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        binding.latent_attention(shape, plan, q, pages, table, 0.07, out, ws, status)
        end.record()
        torch.cuda.synchronize()
        assert int(status.item()) == 0 and start.elapsed_time(end) > 10
        outs.append(out)
    assert torch.equal(bits(outs[0]), bits(outs[1]))
    for b, n in enumerate(lens):
        z = pages[table[b, :counts[b]].long()].reshape(-1, ROW)[:n].double()
        x = q[b].double()
        w = torch.softmax(x @ z.T * 0.07, 1)
        want = [w @ z[:, :LATENT], w @ z[:, :LATENT].abs(), (x.abs() @ z.abs().T * 0.07).amax(1)]
        assert_latent_close(outs[0][b].double().cpu().numpy(), [y.cpu().numpy() for y in want], n,
                            "bf16", f"sequence {b}")


@all_kernels
def test_absorbed_under_any_wait_limit(rows):
    """Wait limits from none to longer than the call, ranges of several pieces with
    rows to clear: every row is as it was or right, a row that was left has its
    status, and the next call with the default limit is right."""
    lens, qs = [900, 77, 1500, 30, 333], [1, 2, 1, 1, 3]
    c = Case(lens, qs, heads=16, seed=33, poison=True)
    want = oracle.latent_attention(f64(c.q), f64(c.pages), c.table.numpy(), lens, qs, c.scale)
    for limit in (1, 300, 1000, 2000, 3000, 5000, 8000, 20000, 0):
        d = Device(c, rows_per_tile=rows, num_sms=4, wait_limit_ns=limit)
        out = torch.full((c.T, 16, LATENT), 7.0, dtype=DT["fp16"], device="cuda")
        d.attention(out)
        status = d.done()
        got = out.double().cpu().numpy()
        left = (got == 7).all(axis=-1)
        assert status == (binding.PA_DEV_TIMEOUT if left.any() else status) and status in (0, 8)
        assert limit or (status == 0 and not left.any())
        if not left.all():
            assert_latent_close(got[~left], tuple(x[~left] for x in want), 1500, "fp16", f"{limit} ns")


def test_captured_upload_outlives_its_plan_object():
    """A graph of upload, append and attention, replayed after the program has
    dropped the plan and made others: the workspace holds the plan again."""
    c = Case([500, 90], [1, 1], heads=16, seed=34)
    d = Device(c)
    out = d.attention()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.latent_upload(d.plan, d.ws)
        d.append()
        d.attention(out)
    kept = d.plan
    d.plan = None
    del kept
    others = [binding.LatentPlan(d.shape, [9 + i, 400], [1, 1], 152) for i in range(50)]
    for _ in range(2):
        out.fill_(float("nan"))
        d.ws.zero_()
        torch.cuda.synchronize()   # calls may read the plan before the kernel ahead has ended
        g.replay()
        assert d.done() == 0
        pool = oracle.latent_append(f64(c.pages), f64(c.c_new), f64(c.r_new), c.table.numpy(), c.lens, c.qs)
        want = oracle.latent_attention(f64(c.q), pool, c.table.numpy(), c.lens, c.qs, c.scale)
        assert_latent_close(out.double().cpu().numpy(), want, 500, "fp16")
    assert len(others) == 50


@pytest.mark.parametrize("dtype,power", [("bf16", 8), ("bf16", 15), ("bf16", 23), ("fp16", 12)])
@pytest.mark.parametrize("splits", [0, 2])
def test_scores_far_beyond_the_exponential(dtype, power, splits):
    """Scores of 10^8 to 10^18.  Inputs are whole numbers up to 7 times a power of
    two, so that scores are exact in fp32 and differ by at least 2^16 x 1.7: where
    one token has the largest, it has all the weight.  Weight and result are
    each rounded at most once (half a step each, 2 u in all), and nothing is lost to
    infinity or zero."""
    c = Case([300, 70, 520], [3, 1, 20], heads=7, dtype=dtype, seed=40, scale=1.7)
    g = torch.Generator().manual_seed(41)
    for name in ("q", "pages", "qx", "kv", "rows"):
        t = getattr(c, name)
        setattr(c, name, (torch.randint(-7, 8, t.shape, generator=g) * 2.0**power).to(t.dtype))
    u = 2 * torch.finfo(DT[dtype]).eps / 2

    def check(out, want, what):
        one = (want[1] == np.abs(want[0])).all(axis=-1)
        assert one.mean() > 0.8
        got = out.double().cpu().numpy()
        assert np.all(np.isfinite(got)), what
        assert np.all(np.abs(got - want[0])[one] <= u * (1 + u) * np.abs(want[0])[one]), what
    want = oracle.latent_attention(f64(c.q), f64(c.pages), c.table.numpy(), c.lens, c.qs, c.scale)
    for rows in (16, 64, 128):
        d = Device(c, rows_per_tile=rows, forced_splits=splits)
        out = d.attention()
        assert d.done() == 0
        check(out, want, f"rows {rows}")
    want = oracle.latent_prefill(f64(c.qx), f64(c.k), f64(c.rows[:, LATENT:]), f64(c.v), c.lens, c.qs, c.scale)
    for rows in (128, 256):
        d = Device(c, form="expanded", rows_per_tile=rows)
        out = d.prefill()
        assert d.done() == 0
        check(out, want, f"tiles {rows}")


# batches whose ranges hold several pieces of several tiles, on few SMs
MANY_PIECES = [
    # lens, q_lens, heads, page, num_sms
    ([500, 77, 0, 1300, 64, 257, 30, 900], [1] * 2 + [0] + [1] * 5, 16, 16, 4),
    ([700, 128, 65, 1029], [3, 1, 2, 5], 20, 32, 2),              # tiles that begin inside a token
    ([129, 1000, 15, 513, 384, 2000], [1, 2, 1, 1, 3, 1], 128, 64, 8),
    ([63, 1, 190, 2, 64, 333, 128, 16, 127], [1] * 9, 48, 128, 2),   # one range, tails of every kind
]


@all_kernels
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("case", MANY_PIECES, ids=lambda c: f"B{len(c[0])}_H{c[2]}_S{c[3]}_sm{c[4]}")
def test_ranges_of_many_pieces(case, dtype, rows):
    """A CTA (or pair) works through pieces of several tiles in turn: queries,
    accumulators, statistics and barriers are used again."""
    lens, qs, heads, page, sms = case
    c = Case(lens, qs, heads=heads, page=page, dtype=dtype, seed=seed_of(case), poison=True)
    d = Device(c, num_sms=sms, rows_per_tile=rows)
    assert d.plan.c.num_ranges <= sms and d.plan.c.num_segments >= 2 * d.plan.c.num_ranges
    out = d.attention()
    assert d.done() == 0
    want = oracle.latent_attention(f64(c.q), f64(c.pages), c.table.numpy(), lens, qs, c.scale)
    assert_latent_close(out.double().cpu().numpy(), want, max(lens), dtype, str(case))
    assert torch.equal(bits(d.attention()), bits(out))


@all_kernels
def test_ranges_of_many_pieces_with_bad_pages(rows):
    """Rows to clear in some pieces of a range and not in others."""
    lens, qs = [200, 70, 333, 48, 500, 90], [1, 2, 1, 1, 1, 1]
    c = Case(lens, qs, heads=16, page=16, seed=35, poison=True)
    bad = [(0, 3), (1, 0), (3, 0), (3, 1), (3, 2), (4, 31)]
    for b, j in bad:
        c.table[b, j] = -1 if j % 2 else c.num_pages
    d = Device(c, num_sms=2, rows_per_tile=rows)
    assert d.plan.c.num_segments >= 3 * d.plan.c.num_ranges
    out = d.attention()
    assert d.done() == binding.PA_DEV_BAD_PAGE
    want = oracle.latent_attention(f64(c.q), f64(c.pages), c.table.numpy(), lens, qs, c.scale, bad_pages=bad)
    assert_latent_close(out.double().cpu().numpy(), want, 500, "fp16")
    assert torch.all(out[4] == 0)


def test_a_long_prompt_and_a_long_context():
    """Expanded attention over many stages: the rings turn often."""
    c = Case([4100, 6001], [300, 129], heads=2, seed=36, dtype="bf16")
    for rows in (128, 256):
        d = Device(c, form="expanded", rows_per_tile=rows)
        out = d.prefill()
        assert d.done() == 0
        want = oracle.latent_prefill(f64(c.qx), f64(c.k), f64(c.rows[:, LATENT:]), f64(c.v), c.lens, c.qs,
                                     c.scale)
        assert_latent_close(out.double().cpu().numpy(), want, 6001, "bf16")


def test_binding_refuses_wrong_sizes_and_devices():
    """Sizes, dense last dimensions and element types are checked for each tensor
    before the library is called; nothing is written."""
    c = Case([40, 9], [7, 9], heads=2, head_dim=64, seed=37)
    a, e = Device(c), Device(c, form="expanded")
    out, outx = torch.zeros(16, 2, LATENT, device="cuda").half(), torch.zeros(16, 2, 64, device="cuda").half()
    rows = torch.zeros(49, ROW, device="cuda").half()
    before = a.pages.clone()

    def append(**kw):
        x = {"c": a.c_new, "r": a.r_new, "pages": a.pages, "table": a.table, **kw}
        binding.latent_append(a.shape, a.plan, x["c"], x["r"], x["pages"], x["table"], a.ws, a.status)

    def attention(**kw):
        x = {"q": a.q, "pages": a.pages, "table": a.table, "out": out, "ws": a.ws, **kw}
        binding.latent_attention(a.shape, a.plan, x["q"], x["pages"], x["table"], 0.1, x["out"], x["ws"], a.status)

    def prefill(**kw):
        x = {"q": e.qx, "k": e.k, "r": e.k_rope, "v": e.v, "out": outx, **kw}
        binding.latent_prefill(e.shape, e.plan, x["q"], x["k"], x["r"], x["v"], 0.1, x["out"], e.ws, e.status)

    def gather(**kw):
        x = {"rows": rows, **kw}
        binding.latent_gather(a.shape, a.plan, a.pages, a.table, x["rows"], a.ws, a.status)

    size, dense, element = "must have shape", "dense in its last|contiguous", "must be"
    for call, kw, kind, what in [
            (append, {"c": a.c_new[:-1]}, ValueError, size), (append, {"c": a.c_new[:, :-8]}, ValueError, size),
            (append, {"r": a.r_new.float()}, TypeError, element),
            (append, {"r": a.r_new.t().contiguous().t()}, ValueError, dense),
            (append, {"table": a.table[:, :-1].contiguous()}, ValueError, size),
            (append, {"table": a.table.long()}, TypeError, element),
            (append, {"pages": a.pages[:-1]}, ValueError, size), (append, {"c": c.c_new}, TypeError, element),
            (attention, {"q": a.q[:, :1].contiguous()}, ValueError, size),
            (attention, {"q": a.q.transpose(0, 1).contiguous().transpose(0, 1)}, ValueError, dense),
            (attention, {"out": out[:-1]}, ValueError, size), (attention, {"out": out.float()}, TypeError, element),
            (attention, {"pages": a.pages[:, :, ::2]}, ValueError, dense),
            (attention, {"ws": a.ws[:, None]}, ValueError, "one-dimensional"),
            (gather, {"rows": rows[1:]}, ValueError, size), (gather, {"rows": rows.bfloat16()}, TypeError, element),
            (prefill, {"k": e.k[:, :, :32]}, ValueError, size), (prefill, {"k": e.k[1:]}, ValueError, size),
            (prefill, {"v": e.v[:, :1]}, ValueError, size),
            (prefill, {"v": torch.cat([e.v, e.v], 2)[..., ::2]}, ValueError, dense),
            (prefill, {"r": e.k_rope[:, :56]}, ValueError, size),
            (prefill, {"q": e.qx[..., :-8]}, ValueError, dense), (prefill, {"out": outx[:, 0]}, ValueError, dense)]:
        with pytest.raises(kind, match=what):
            call(**kw)
    for call, kw in [(append, {"c": a.c_new[:1].expand(16, -1)}), (prefill, {"k": e.k[:, :1].expand(-1, 2, -1)}),
                     (attention, {"ws": a.ws[:-1]})]:
        with pytest.raises(binding.PagedAttnError):    # broadcast strides, a workspace too small
            call(**kw)
    assert a.done() == 0 and e.done() == 0
    assert torch.equal(bits(a.pages), bits(before)) and not out.any() and not outx.any() and not rows.any()
