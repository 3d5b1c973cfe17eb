"""Host-side checks of the latent attention calls that need no GPU: the
planner's work lists, the oracle against its own definition, and every refusal
(each before any CUDA call)."""

from __future__ import annotations

import ctypes
import gc
import os
import re
import shutil
import subprocess
import weakref

import numpy as np
import pytest

import oracle
from paged_kv_decode_24_gb300 import binding

PTR = ctypes.c_void_p(0x10000)   # 16-byte aligned, never touched
ODD = ctypes.c_void_p(0x10008)


def shape(batch=3, heads=16, head_dim=128, page=16, max_pages=64, num_pages=100, dtype="bf16"):
    return binding.make_latent_shape(batch, heads, head_dim, page, max_pages, num_pages, dtype)


def parts(plan):
    """header, cu_q, cu_k, ranges, segments, merges (absorbed) or tiles (expanded)."""
    b = plan.blob()
    B, form, rows, nr, ns, nm = b[1], b[6], b[7], b[8], b[9], b[10]
    at = 16
    cu_q, cu_k = b[at:at + B + 1], b[at + B + 1:at + 2 * (B + 1)]
    at = (at + 2 * (B + 1) + 3) // 4 * 4
    if form == 1:
        return b[:16], cu_q, cu_k, b[at:at + 8 * nr].reshape(nr, 8)
    ranges = b[at:at + nr + 1]
    at = (at + nr + 1 + 3) // 4 * 4
    segments = b[at:at + 8 * ns].reshape(ns, 8)
    merges = b[at + 8 * ns:at + 8 * ns + 4 * nm].reshape(nm, 4)
    return b[:16], cu_q, cu_k, ranges, segments, merges


BATCHES = [
    ([1], [1], 1), ([5, 0, 77], [1, 0, 1], 16), ([1000, 33, 2000], [1, 1, 1], 16),
    ([100, 64, 500], [5, 3, 7], 3), ([40000, 10, 3], [1, 1, 1], 128), ([300] * 40, [1] * 40, 128),
    ([64, 65, 63, 128, 129], [64, 1, 2, 128, 5], 20), ([2000] * 200, [1] * 200, 16),
    ([0, 0], [0, 0], 4),
]


@pytest.mark.parametrize("rows", [0, 16, 64, 128])
@pytest.mark.parametrize("splits", [0, 1, 3])
@pytest.mark.parametrize("case", BATCHES, ids=lambda c: f"B{len(c[0])}_H{c[2]}_L{max(c[0])}")
def test_absorbed_plan_covers_every_row_and_token_once(lib, case, splits, rows):
    lens, qs, heads = case
    s = shape(len(lens), heads, max_pages=3000)
    p = binding.LatentPlan(s, lens, qs, 152, rows_per_tile=rows, forced_splits=splits)
    head, cu_q, cu_k, ranges, seg, merges = parts(p)
    most = max(q * heads for q in qs)
    R = head[7]
    assert R == (rows or (16 if most <= 16 else 64 if most <= 64 else 128)) == p.c.rows_per_tile
    assert list(cu_q) == [0, *np.cumsum(qs)] and list(cu_k) == [0, *np.cumsum(lens)]
    stage = 128 if R == 128 else 64
    # ranges split the list of pieces, none is empty
    assert ranges[0] == 0 and ranges[-1] == len(seg) and np.all(np.diff(ranges) > 0)
    workers = 76 if R == 128 else 152
    if splits == 0:
        assert len(ranges) - 1 <= workers
    tiles = {}
    for b, row0, nrows, t0, t1, slot, packed0, pos0 in seg.tolist():
        assert 1 <= nrows <= R and row0 % R == 0
        assert packed0 == cu_q[b] * heads + row0 and pos0 == lens[b] - qs[b]
        assert t0 % stage == 0 and t0 < t1
        tiles.setdefault((b, row0), []).append((t0, t1, slot, nrows))
    want = {(b, r) for b in range(len(lens)) for r in range(0, qs[b] * heads, R)}
    assert set(tiles) == want
    slots, cut = [], []
    for (b, row0), pieces in tiles.items():
        n = pieces[0][3]
        assert n == min(R, qs[b] * heads - row0) and all(x[3] == n for x in pieces)
        span = lens[b] - qs[b] + (row0 + n - 1) // heads + 1     # tokens its last row sees
        assert [x[0] for x in pieces] == [0, *[x[1] for x in pieces[:-1]]] and pieces[-1][1] == span
        if len(pieces) == 1:
            assert pieces[0][2] == -1
        else:
            ids = [x[2] for x in pieces]
            assert ids == list(range(ids[0], ids[0] + len(ids)))
            slots += ids
            cut.append((ids[0], len(ids), cu_q[b] * heads + row0, n))
        if splits:
            assert len(pieces) == min(splits, -(-span // stage))
    assert sorted(slots) == list(range(head[11])) and sorted(cut) == sorted(map(tuple, merges.tolist()))


def test_absorbed_ranges_have_equal_work(lib):
    """No range has more than a stage, a piece's fixed cost and the shortest
    piece above the mean, whatever the lengths."""
    rng = np.random.default_rng(5)
    for heads, unit, fixed in ((16, 64, 1), (128, 128, 2)):
        lens = rng.integers(3000, 9000, 64).tolist()
        s = shape(64, heads, max_pages=1000)
        _, _, _, ranges, seg, _ = parts(binding.LatentPlan(s, lens, [1] * 64, 152))
        cost = -(-(seg[:, 4] - seg[:, 3]) // unit) + fixed
        per = np.add.reduceat(cost, ranges[:-1])
        assert per.max() <= per.mean() + 2 + fixed + 2, (heads, per.max(), per.mean())


def test_few_expanded_tiles_are_halves(lib):
    def longest_tile(lens, qs, heads):
        p = binding.LatentPlan(shape(len(lens), heads, max_pages=3000), lens, qs, 152, form="expanded")
        tiles = parts(p)[3]
        return len(tiles), int(tiles[:, 1].max())
    assert longest_tile([8192], [256], 32) == (64, 128)
    assert longest_tile([2048], [2048], 8) == (128, 128)
    assert longest_tile([8192] * 2, [256] * 2, 76) == (152, 256)   # halves would need two turns
    assert longest_tile([8192], [8192], 32) == (1024, 256)
    assert longest_tile([130, 5], [130, 5], 3)[1] <= 256


def test_few_tiles_are_cut_one_by_one(lib):
    def counts(lens, heads):
        p = binding.LatentPlan(shape(len(lens), heads, max_pages=3000), lens, [1] * len(lens), 152)
        _, _, _, ranges, seg, _ = parts(p)
        return len(ranges) - 1, len(seg), p.c.num_merges, seg
    # short tiles stay whole
    assert counts([128] * 8, 16)[:3] == (8, 8, 0) and counts([256] * 8, 64)[:3] == (8, 8, 0)
    assert counts([384, 3, 100], 128)[:3] == (3, 3, 0) and counts([100] * 152, 16)[:3] == (152, 152, 0)
    # longer ones become pieces of about one length, one for each SM (or pair) at most
    for lens, heads, most in (([1024] * 8, 16, 152), ([3000, 500, 64], 64, 152), ([4000, 9000], 128, 76),
                              ([30000], 16, 152)):
        n, pieces, merges, seg = counts(lens, heads)
        assert n == pieces <= most and merges > 0
        unit = 128 if heads == 128 else 64
        size = -(-(seg[:, 4] - seg[:, 3]) // unit)
        for b, length in enumerate(lens):
            mine = size[seg[:, 0] == b]
            assert mine.max() - mine.min() <= 1 and mine.sum() == -(-length // unit)
        assert size.max() <= size[seg[:, 0] == int(np.argmax(lens))].max()
    # more tiles than SMs: ranges of equal work
    n, pieces, _, _ = counts([500] * 200, 16)
    assert n == 152 and pieces > 200


@pytest.mark.parametrize("rows", [0, 128, 256])
@pytest.mark.parametrize("case", BATCHES, ids=lambda c: f"B{len(c[0])}_H{c[2]}_L{max(c[0])}")
def test_expanded_plan_covers_every_token_and_head_once(lib, case, rows):
    lens, qs, heads = case
    p = binding.LatentPlan(shape(len(lens), heads, max_pages=3000), lens, qs, 152, form="expanded",
                           rows_per_tile=rows)
    head, cu_q, cu_k, tiles = parts(p)
    assert p.c.num_ranges == len(tiles) and p.c.workspace_bytes >= p.c.blob_bytes
    seen = set()
    for h, n, q0, pos0, k0 in tiles[:, :5].tolist():
        b = int(np.searchsorted(cu_q, q0, side="right")) - 1
        while qs[b] == 0:
            b -= 1
        assert 1 <= n <= (rows or 256) and k0 == cu_k[b] and pos0 == lens[b] - qs[b] + q0 - cu_q[b]
        assert q0 + n <= cu_q[b + 1]
        seen |= {(q0 + i, h) for i in range(n)}
    assert len(seen) == sum(qs) * heads == int(tiles[:, 1].sum())
    stages = -(-(tiles[:, 3] + tiles[:, 1]) // 128)
    assert np.all(np.diff(stages) <= 0)          # the longest first


def plan_code(s, lens, qs, sms=152, form=0, **opts):
    o = binding.PaLatentOptions(opts.get("rows", 0), opts.get("splits", 0), 0)
    out = binding.PaLatentPlan()
    a, b = np.asarray(lens, np.int32), np.asarray(qs, np.int32)
    code = binding.load().pa_latent_plan(ctypes.byref(s), a.ctypes.data if a.size else None,
                                         b.ctypes.data if b.size else None, sms, form,
                                         ctypes.byref(o), ctypes.byref(out))
    if code == 0:
        binding.load().pa_latent_plan_free(ctypes.byref(out))
    return code


INVALID, UNSUPPORTED, WORKSPACE, PLAN = 1, 2, 3, 8


def test_plan_refusals(lib):
    good = shape(2)
    assert plan_code(good, [5, 3], [1, 3]) == 0
    for lens, qs in (([5, -1], [1, 0]), ([5, 3], [1, 4]), ([5, 3], [-1, 0]), ([64 * 16 + 1, 3], [1, 1])):
        assert plan_code(good, lens, qs) == INVALID
    assert plan_code(good, [5, 3], [1, 1], sms=0) == INVALID
    assert plan_code(good, [5, 3], [1, 1], form=2) == INVALID
    assert plan_code(good, [5, 3], [1, 1], rows=32) == INVALID
    assert plan_code(good, [5, 3], [1, 1], splits=-1) == INVALID
    assert plan_code(good, [5, 3], [1, 1], form=1, rows=64) == INVALID
    assert plan_code(good, [5, 3], [1, 1], form=1, rows=128) == 0
    assert plan_code(good, [5, 3], [1, 1], rows=256) == INVALID
    assert plan_code(good, [5, 3], [1, 1], form=1, splits=2) == INVALID
    for k, v, want in (("num_heads", 129, UNSUPPORTED), ("num_heads", 0, INVALID),
                       ("head_dim", 96, UNSUPPORTED), ("latent_dim", 256, UNSUPPORTED),
                       ("rope_dim", 32, UNSUPPORTED), ("page_size", 8, UNSUPPORTED),
                       ("page_size", 48, UNSUPPORTED), ("page_size", 0, INVALID),
                       ("dtype", 2, UNSUPPORTED), ("batch", -1, INVALID), ("num_pages", 0, INVALID),
                       ("max_pages_per_seq", 0, INVALID), ("max_pages_per_seq", 2**30, INVALID)):
        s = shape(2)
        setattr(s, k, v)
        assert plan_code(s, [5, 3], [1, 1]) == want, (k, v)
    big = shape(1, max_pages=2**27 - 1)       # packed rows times heads past 32 bits
    assert plan_code(big, [2**31 - 32], [2**31 - 32]) == INVALID
    assert lib.pa_latent_plan(ctypes.byref(good), None, None, 152, 0, None,
                              ctypes.byref(binding.PaLatentPlan())) == INVALID
    lib.pa_latent_plan_free(None)


class Call:
    """The four device calls with fake pointers: every refusal comes before a
    CUDA call, so these run without a GPU."""

    def __init__(self, lib, form="absorbed", **sh):
        self.lib, self.s = lib, shape(2, **sh)
        self.p = binding.LatentPlan(self.s, [500, 3], [1, 3], 152, form=form)

    def args(self, **kw):
        return kw.get("s", self.s), kw.get("plan", self.p.c), kw.get("n", self.p.workspace_bytes)

    def append(self, **kw):
        s, plan, n = self.args(**kw)
        return self.lib.pa_latent_append(
            ctypes.byref(s), ctypes.byref(plan), kw.get("c", PTR), kw.get("cs", 512),
            kw.get("r", PTR), kw.get("rs", 64), kw.get("pages", PTR), kw.get("table", PTR),
            kw.get("ws", PTR), n, kw.get("status", PTR), None)

    def gather(self, **kw):
        s, plan, n = self.args(**kw)
        return self.lib.pa_latent_gather(
            ctypes.byref(s), ctypes.byref(plan), kw.get("pages", PTR), kw.get("table", PTR),
            kw.get("rows", PTR), kw.get("ws", PTR), n, kw.get("status", PTR), None)

    def attention(self, **kw):
        s, plan, n = self.args(**kw)
        return self.lib.pa_latent_attention(
            ctypes.byref(s), ctypes.byref(plan), kw.get("q", PTR), kw.get("pages", PTR),
            kw.get("table", PTR), ctypes.c_float(kw.get("scale", 0.1)), kw.get("out", PTR),
            kw.get("ws", PTR), n, kw.get("status", PTR), None)

    def prefill(self, **kw):
        s, plan, n = self.args(**kw)
        return self.lib.pa_latent_prefill(
            ctypes.byref(s), ctypes.byref(plan), kw.get("q", PTR), kw.get("k", PTR),
            kw.get("kt", 2048), kw.get("kh", 128), kw.get("kr", PTR), kw.get("krs", 576),
            kw.get("v", PTR), kw.get("vt", 2048), kw.get("vh", 128),
            ctypes.c_float(kw.get("scale", 0.1)), kw.get("out", PTR), kw.get("ws", PTR), n,
            kw.get("status", PTR), None)


NAMES = {"append": ["c", "r", "pages"], "gather": ["pages", "rows"],
         "attention": ["q", "pages", "out"], "prefill": ["q", "k", "kr", "v", "out"]}


@pytest.mark.parametrize("op", list(NAMES))
def test_call_refusals(lib, op):
    c = Call(lib, "expanded" if op == "prefill" else "absorbed")
    call = getattr(c, op)
    for name in NAMES[op] + ["ws"]:
        assert call(**{name: None}) == INVALID and call(**{name: ODD}) == INVALID, name
    for name in ["status"] + (["table"] if op != "prefill" else []):
        assert call(**{name: None}) == INVALID
        assert call(**{name: ctypes.c_void_p(0x10002)}) == INVALID
    assert call(n=c.p.workspace_bytes - 1) == WORKSPACE
    for k, v in (("batch", 3), ("num_heads", 8), ("head_dim", 64), ("page_size", 32),
                 ("max_pages_per_seq", 65)):
        s = shape(2)
        setattr(s, k, v)
        assert call(s=s) == PLAN, k
    s = shape(2)
    s.num_heads = 200
    assert call(s=s) == UNSUPPORTED
    for k, v in (("num_segments", 99), ("num_slots", -1), ("rows_per_tile", 32), ("form", 9),
                 ("workspace_bytes", 0)):
        plan = binding.PaLatentPlan.from_buffer_copy(c.p.c)
        setattr(plan, k, v)
        if op == "prefill" and k == "num_segments":
            continue    # the expanded plan has none: the field is not read
        assert call(plan=plan) == PLAN, k


def test_scale_stride_and_form_refusals(lib):
    a, e = Call(lib), Call(lib, "expanded")
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert a.attention(scale=scale) == INVALID and e.prefill(scale=scale) == INVALID
    assert a.attention(plan=e.p.c, n=10**6) == PLAN and e.prefill(plan=a.p.c, n=10**6) == PLAN
    for kw in ({"cs": 511}, {"cs": 504}, {"cs": 516}, {"rs": 63}, {"rs": 0}, {"cs": -512}):
        assert a.append(**kw) == INVALID, kw
    for kw in ({"kt": 0}, {"kh": 0}, {"vt": 7}, {"vh": 4}, {"krs": -64}, {"krs": 56},
               {"kt": 1 << 40}, {"kt": 128, "kh": 128}, {"kh": 120}, {"vt": 2040}):
        assert e.prefill(**kw) == INVALID, kw


def test_empty_batches_launch_nothing(lib):
    s = shape(0)
    for form in ("absorbed", "expanded"):
        p = binding.LatentPlan(s, [], [], 152, form=form)
        none = ctypes.c_void_p(None)
        f = ctypes.c_float(1.0)
        if form == "absorbed":
            assert lib.pa_latent_append(ctypes.byref(s), ctypes.byref(p.c), none, 512, none, 64, none,
                                        none, none, 0, none, None) == 0
            assert lib.pa_latent_gather(ctypes.byref(s), ctypes.byref(p.c), none, none, none, none, 0,
                                        none, None) == 0
            assert lib.pa_latent_attention(ctypes.byref(s), ctypes.byref(p.c), none, none, none, f,
                                           none, none, 0, none, None) == 0
        else:
            assert lib.pa_latent_prefill(ctypes.byref(s), ctypes.byref(p.c), none, none, 8, 8, none,
                                         64, none, 8, 8, f, none, none, 0, none, None) == 0


def test_binding_checks_sizes_before_the_call(lib):
    torch = pytest.importorskip("torch")
    s = shape(2)
    p = binding.LatentPlan(s, [5, 3], [1, 3], 152)
    cpu = torch.zeros(4, 512, dtype=torch.bfloat16)
    with pytest.raises((TypeError, ValueError)):
        binding._latent_rows(cpu, torch.bfloat16, (4, 512), "c_new")
    with pytest.raises(ValueError):
        binding.LatentPlan(s, [5, 3, 2], [1, 3], 152)
    with pytest.raises(KeyError):
        binding.LatentPlan(s, [5, 3], [1, 3], 152, form="other")
    with pytest.raises(binding.PagedAttnError):
        binding.LatentPlan(s, [5, 3], [1, 4], 152)
    del p


# ---- the oracle

def test_oracle_forms_agree_in_64_bits():
    """Absorbed and expanded attention of the same cache and maps are equal."""
    rng = np.random.default_rng(0)
    lens, qs, H, D, S = [21, 40], [21, 3], 3, 64, 16
    table = np.array([[4, 1, 0], [2, 5, 3]])
    pages = rng.standard_normal((6, S, 576))
    W, U = rng.standard_normal((2, H, D, 512)) * 0.05
    q = rng.standard_normal((24, H, D + 64))
    rows = oracle.latent_gather(pages, table, lens)
    k = np.einsum("tc,hdc->thd", rows[:, :512], W)
    v = np.einsum("tc,hdc->thd", rows[:, :512], U)
    x = oracle.latent_prefill(q, k, rows[:, 512:], v, lens, qs, 0.09)[0]
    qa = np.concatenate([np.einsum("thd,hdc->thc", q[..., :D], W), q[..., D:]], 2)
    y = oracle.latent_attention(qa, pages, table, lens, qs, 0.09)[0]
    assert np.abs(x - np.einsum("thc,hdc->thd", y, U)).max() < 1e-12


def test_oracle_closed_forms():
    """One visible token: its own latent; equal scores: the mean; a sequence
    whose pages are all bad: zeros."""
    rng = np.random.default_rng(1)
    pages = rng.standard_normal((3, 16, 576))
    table = np.array([[1, 2]])
    q = rng.standard_normal((1, 2, 576))
    out = oracle.latent_attention(q, pages, table, [1], [1], 1.0)[0]
    assert np.allclose(out, pages[1, 0, :512][None, None], atol=0)
    out = oracle.latent_attention(q * 0, pages, table, [20], [1], 1.0)[0]
    mean = np.concatenate([pages[1], pages[2, :4]])[:, :512].mean(0)
    assert np.allclose(out[0], mean[None], atol=1e-14)
    out = oracle.latent_attention(q, pages, table, [20], [1], 1.0, bad_pages=[(0, 0), (0, 1)])[0]
    assert np.all(out == 0)


C_STRUCTS = {"pa_latent_shape_t": "PaLatentShape", "pa_latent_plan_t": "PaLatentPlan",
             "pa_latent_options_t": "PaLatentOptions"}


def test_structs_and_plans_from_c(lib, tmp_path):
    """The binding's structures have the C structs' sizes and offsets, and a C
    program makes a plan of either form."""
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    lines = []
    for c, py in C_STRUCTS.items():
        lines.append(f'printf("{c} - %zu\\n", sizeof({c}));')
        lines += [f'printf("{c} {f[0]} %zu\\n", offsetof({c}, {f[0]}));'
                  for f in getattr(binding, py)._fields_]
    code = """#include <stddef.h>
#include <stdio.h>
#include "pagedattn.h"
int main(void) {
  pa_latent_shape_t s = {2, 16, 128, 512, 64, 16, 64, 100, PA_DTYPE_BF16};
  const int32_t lens[2] = {700, 33}, qs[2] = {1, 33};
  pa_latent_options_t o = {0, 2, 0};
  pa_latent_plan_t p;
  if (pa_latent_plan(&s, lens, qs, 152, PA_LATENT_ABSORBED, &o, &p) != PA_OK) return 1;
  if (p.total_q != 34 || p.total_k != 733 || p.num_slots < 2) return 2;
  pa_latent_plan_free(&p);
  if (pa_latent_plan(&s, lens, qs, 152, PA_LATENT_EXPANDED, NULL, &p) != PA_OK) return 3;
  pa_latent_plan_free(&p);
  if (p.host_blob != NULL) return 4;
  %s
  return 0;
}
""" % "\n  ".join(lines)
    src, exe = tmp_path / "latent.c", str(tmp_path / "latent")
    src.write_text(code)
    root, libdir = os.path.dirname(os.path.dirname(os.path.abspath(__file__))), os.path.dirname(binding.LIB_PATH)
    r = subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I",
                        os.path.join(root, "include"), str(src), "-o", exe, "-L", libdir, "-lpagedattn",
                        "-Wl,-rpath," + libdir], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0
    n = 0
    for line in r.stdout.split("\n")[:-1]:
        c, field, value = line.split()
        cls = getattr(binding, C_STRUCTS[c])
        assert (ctypes.sizeof(cls) if field == "-" else getattr(cls, field).offset) == int(value), line
        n += 1
    assert n == sum(1 + len(getattr(binding, py)._fields_) for py in C_STRUCTS.values())


# ---- hand-overs, by reading: what a wait that gave up may still let happen
# cannot be brought about on a GPU without stalling it

def kernel_source(name):
    """A kernel's source without comments, white space as single blanks."""
    path = os.path.join(os.path.dirname(binding.LIB_PATH), os.pardir, "csrc", name)
    with open(path, encoding="utf-8") as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    return re.sub(r"\s+", " ", text)


def test_value_rows_are_cleared_only_after_a_wait_whose_answer_counts():
    """Expanded form: the zeros behind the last visible token may be written
    only once the last stage's copies have landed.  That wait has the plan's
    limit, and its failure sets the status and the flag that keeps the rows from
    being cleared and handed over; the short drain waits, whose answers are not
    used, come after it."""
    src = kernel_source("latent_prefill.cu")
    copies = src[src.index("warp == 9 || warp == 10"):src.index("} else if (warp == 8)")]
    landed = copies.find("good = mbar_wait_bounded_sleep(full + 8 * ((n - 1) & 1), "
                         "(uint32_t)(((n - 1) >> 1) & 1), p.wait_ns)")
    assert landed >= 0, "no wait with the plan's limit before the rows are cleared"
    gave_up = copies.index("if (!good) { set_status(p.status, PA_DEV_TIMEOUT); *flag = 1; }")
    clears = copies.index("make_uint4(0u, 0u, 0u, 0u)")
    assert landed < gave_up < copies.index("kDrainWaitNs") < clears < copies.index("L::V_CLEAR")
    assert "*flag == 0" in copies[gave_up:clears]


def test_second_cta_waits_for_the_drain_after_the_first_has_committed_it():
    """Pairs: the last commit arrives in both CTAs.  The second one, which issues
    no products, starts its limited wait only behind the cluster barrier that the
    first CTA reaches after the commit, whatever the call takes, and neither frees
    tensor memory or ends before."""
    src = kernel_source("latent_pair.cu")
    src = src[src.index("latent_pair_kernel("):src.index("cudaError_t launch_t(")]
    commit = src.index("commit2(sb + L::DRAIN)")
    waits = [m.start() for m in re.finditer(r"L::DRAIN, 0u, kDrainWaitNs\)", src)]
    meet = src.index("cluster_sync();", commit)
    free = src.index("tcgen05.dealloc")
    assert len(waits) == 2 and commit < waits[0] < meet < waits[1] < free, (commit, waits, meet, free)
    first, second = (src[src.rindex("if (", 0, w):w] for w in waits)
    assert first.startswith("if (rank == 0)") and second.startswith("if (rank != 0)")
    assert src.index("cluster_sync();", meet + 1) > free


@pytest.mark.parametrize("name", ["latent_prefill.cu", "latent_solo.cu", "latent_pair.cu"])
def test_aligned_instructions_follow_a_reconvergence(name):
    """Tensor-memory accesses and hand-written barriers are for a whole converged
    warp.  Between a branch, a vote or a wait and the next of them stands a
    __syncwarp: nothing relies on where the compiler lets a warp's lanes meet."""
    src = kernel_source(name)
    src = src[src.index("__launch_bounds__"):src.index("cudaError_t launch_t(")]
    access = r"tc5::(?:ld16|ld32|st16|st16u|wait_ld|wait_st)\(|tcgen05\.(?:alloc|dealloc|relinquish)"
    branch = r"\bif \(|__any_sync|__all_sync|warp_wait\(|\bwait\(|mbar_\w+\("
    last, checked = "", 0
    for m in re.finditer(f"(?P<sync>__syncwarp\\(\\))|(?P<access>{access})|(?P<branch>{branch})", src):
        if m.lastgroup == "access":
            assert last != "branch", src[max(0, m.start() - 160):m.end() + 40]
            checked += 1
        last = m.lastgroup
    assert checked >= 10
    for path, func in (("latent_tc5.cuh", "void row_pair_barrier("), ("latent_pair.cu", "void cluster_sync("),
                       ("latent_mma.cu", "void work_barrier(")):
        text = kernel_source(path)
        body = text[text.index(func):]
        assert 0 < body.index("__syncwarp()") < body.index("asm volatile"), path


def test_a_flag_that_others_may_set_is_read_by_a_vote():
    """Expanded form: the lanes that clear rows meet in __syncwarp, so all of them
    or none take that branch, also when another warp gives up meanwhile."""
    src = kernel_source("latent_prefill.cu")
    reads = [src[max(0, m.start() - 20):m.end()] for m in re.finditer(r"\*flag == 0", src)]
    assert reads and all("__all_sync(kFull, *flag == 0" in r for r in reads), reads


def drains_cover_what_is_under_way(full, first, ring, seed):
    """Model of a copy warp that gives up: `full` barriers hold a count of finished
    phases and answer a parity test as an mbarrier does, copies land at random
    times.  first(issued, stages) names the stages the warp's last waits go
    through, in order.  True if nothing is under way after them."""
    rng = np.random.default_rng(seed)
    stages = int(rng.integers(1, 9))
    land = rng.exponential(1.0, stages) + np.arange(stages) * rng.choice([0.0, 0.5])
    freed, issued = 0, 0
    for j in range(stages):
        while freed < j - ring + 1:
            if rng.random() < 0.3 or not (land[freed] <= rng.uniform(0, 3)):
                break          # the wait gave up, wherever that stage stands
            freed += 1
        if freed < j - ring + 1:
            break
        issued += 1
    now = 0.0
    done = [land[i] if i < issued else np.inf for i in range(stages + 2)]
    for i in range(freed):
        done[i] = 0.0          # known to be read

    def phases(bar, t):        # finished phases of a barrier, in the order of its uses
        n = 0
        for i in range(bar, stages + 2, full):
            if done[i] > t:
                break
            n += 1
        return n
    for i in first(freed, issued):
        bar, use = i % full, i // full
        times = [now, *sorted(x for x in done if now < x < np.inf)]
        t = next((t for t in times if (phases(bar, t) & 1) != (use & 1)), now)
        now = max(now, t)
    return all(x <= now for x in done[:issued])


def test_last_waits_of_the_copy_warps():
    """A barrier's parity cannot tell a use from the one two before it, so a warp
    that gave up waits for the uses that are under way in order, from the first one
    not known to be read; waiting for the last two stages only may wait for
    nothing."""
    assert all(drains_cover_what_is_under_way(2, lambda freed, issued: range(freed, issued), 2, s)
               for s in range(3000))
    assert not all(drains_cover_what_is_under_way(
        2, lambda freed, issued: range(max(0, issued - 1), issued + 1), 2, s) for s in range(3000))
    prefill, solo, pair = (kernel_source(f"latent_{x}.cu") for x in ("prefill", "solo", "pair"))
    assert "for (int i = freed; i < j; ++i) mbar_wait_bounded_sleep(full + 8 * (i & 1)" in prefill
    assert "for (; freed * per < u - ring + 1; ++freed) { good = " in prefill     # exact when it gave up
    assert "const int u = c - (g < issued ? 0 : 2);" in solo and "if (!good) { issued = g; break; }" in solo
    assert "const int issued = g + (begun ? 1 : 0);" in pair and "c - 1 - (x < issued ? 0 : 1);" in pair


def test_a_captured_upload_keeps_its_plan(lib, monkeypatch):
    """A graph's replays read the plan's host copy, so the binding keeps a plan
    whose upload was captured, until free(); others go with their last
    reference."""
    torch = pytest.importorskip("torch")
    seen = []

    class Lib:
        def __getattr__(self, name):
            return getattr(lib, name)

        def pa_latent_plan_upload(self, plan, workspace, n, stream):
            seen.append(n)
            return 0
    monkeypatch.setattr(binding, "load", lambda: Lib())
    monkeypatch.setattr(binding, "_latent_ptr", lambda t, dtype, size, name: PTR)
    monkeypatch.setattr(binding, "_stream", lambda stream=None: None)
    ws = torch.zeros(64, dtype=torch.uint8)
    for capturing in (False, True):
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing)
        plan = binding.LatentPlan(shape(2), [5, 3], [1, 3], 152)
        ref = weakref.ref(plan)
        binding.latent_upload(plan, ws)
        binding.latent_upload(plan, ws)
        del plan
        gc.collect()
        assert (ref() is not None) == capturing
    ref().free()
    gc.collect()
    assert ref() is None and seen == [64] * 4


def test_a_scale_that_leaves_fp32_in_log2_units_is_refused(lib):
    """The kernels hold scale x log2(e): from 3.4028e38 / 1.4427 on that is
    infinite, and 0 times infinity would turn scores of zero into NaN."""
    a, e = Call(lib), Call(lib, "expanded")
    for scale in (2.36e38, 3e38, 3.4e38, float("-inf")):
        assert a.attention(scale=scale) == INVALID and e.prefill(scale=scale) == INVALID


@pytest.mark.parametrize("rows", [0, 128, 256])
@pytest.mark.parametrize("case", BATCHES, ids=lambda c: f"B{len(c[0])}_H{c[2]}_L{max(c[0])}")
def test_expanded_tiles_are_whole_but_for_the_last(lib, case, rows):
    """Each sequence's tiles have exactly the plan's tile size, the last one the
    rest; the planner's own choice is one of the two sizes for the whole call."""
    lens, qs, heads = case
    p = binding.LatentPlan(shape(len(lens), heads, max_pages=3000), lens, qs, 152, form="expanded",
                           rows_per_tile=rows)
    tiles = parts(p)[3]
    got = sorted((int(q0), int(h), int(n)) for h, n, q0 in tiles[:, :3].tolist())

    def cut(size):
        cu = [0, *np.cumsum(qs)]
        return sorted((cu[b] + t, h, min(size, qs[b] - t)) for b in range(len(qs)) for t in range(0, qs[b], size)
                      for h in range(heads))
    assert got in ([cut(rows)] if rows else [cut(256), cut(128)])


def test_absorbed_ranges_stay_within_two_stages_of_the_mean(lib):
    """The bound of equal work, exactly: a range ends in a cut at most one stage, the
    piece's fixed cost and the shortest piece (one stage) behind its share."""
    rng = np.random.default_rng(7)
    for heads, unit, fixed in ((16, 64, 1), (48, 64, 1), (128, 128, 2)):
        for _ in range(20):
            n = int(rng.integers(160, 400))
            lens = rng.integers(200, 9000, n).tolist()
            s = shape(n, heads, max_pages=1000)
            _, _, _, ranges, seg, _ = parts(binding.LatentPlan(s, lens, [1] * n, 152))
            cost = -(-(seg[:, 4] - seg[:, 3]) // unit) + fixed
            per = np.add.reduceat(cost, ranges[:-1])
            assert per.max() <= per.mean() + fixed + 2, (heads, per.max(), per.mean())
