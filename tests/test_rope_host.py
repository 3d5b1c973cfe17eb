"""Host-side checks of the rotary append that need no GPU: what q_out may not share.
Every call here is refused before anything is launched."""

from __future__ import annotations

import ctypes

import pytest

from paged_kv_decode_24_gb300 import binding

INVALID = 1
MB = 1 << 20


def at(address):
    return ctypes.c_void_p(address)


def call(lib, tokens, q_out, dtype="bf16", kind=0, dim=128, **places):
    """The call with every array in a megabyte range of its own (pools: 64), and q_out as given:
    sequences of 100 and 300 tokens, 16 / 8 heads, 100 positions."""
    s = binding.make_shape(2, 16, 8, dim, 16, 64, 100, dtype)
    a = dict(table=1, q=2, k=3, v=4, pos=5, bt=6, lens=7, status=8, ws=9, ksc=10, vsc=11, kp=100, vp=200)
    a = {n: at(i * 64 * MB) for n, i in a.items()}
    if not kind:
        a["ksc"] = a["vsc"] = at(None)
    a.update(places)
    r = binding.PaRope(dim, 0, 100, kind, a["table"])
    args = [a["q"], 16 * dim, a["k"], 8 * dim, a["v"], 8 * dim, a["pos"], q_out, a["kp"], a["vp"], a["ksc"], a["vsc"],
            a["bt"], a["lens"]]
    if tokens:
        p = binding.PrefillPlan(s, [100, 300], [7, 30])
        return lib.pa_rope_append_tokens(ctypes.byref(s), ctypes.byref(p.c), ctypes.byref(r), *args, a["ws"],
                                         p.workspace_bytes, a["status"], None)
    return lib.pa_rope_append(ctypes.byref(s), ctypes.byref(r), *args, a["status"], None)


@pytest.mark.parametrize("tokens", [False, True])
def test_q_out_shares_nothing_that_the_call_reads_or_writes(lib, tokens):
    rows = 37 if tokens else 2
    size = rows * 16 * 128 * 2
    pool = 100 * 8 * 16 * 128 * 2
    arrays = {"table": (1, 100 * 128 * 4), "k": (3, rows * 8 * 128 * 2), "v": (4, rows * 8 * 128 * 2),
              "pos": (5, rows * 4), "bt": (6, 2 * 64 * 4), "lens": (7, 8), "status": (8, 4), "kp": (100, pool),
              "vp": (200, pool)}
    if tokens:
        arrays["ws"] = (9, 64)
    for name, (i, n) in arrays.items():
        first = i * 64 * MB
        for q_out in (first, first - size + 16, first + (n - 1) // 16 * 16):    # its first and last bytes too
            assert call(lib, tokens, at(q_out)) == INVALID, (name, q_out - first)


@pytest.mark.parametrize("kind", [1, 2])
def test_q_out_shares_nothing_with_8_bit_pools_and_scales(lib, kind):
    size, pool, scales = 2 * 16 * 128 * 2, 100 * 8 * 16 * 128, 100 * 8 * 16 * 4
    for i, n in ((100, pool), (200, pool), (10, scales), (11, scales)):
        first = i * 64 * MB
        for q_out in (first, first - size + 16, first + n - 16):
            assert call(lib, False, at(q_out), "fp16", kind) == INVALID, (i, q_out - first)
