"""Shared helpers of the rotary-append and differential-attention tests:
inputs on the host and the device, the calls, and the tolerances.

Tolerance of an attention output.  u is half a step of the element type
relative to the value (fp16 2^-11, bf16 2^-8).  A value before the norm,
o = sum_t (P1[t] - lambda P2[t]) V[t], differs from the float64 one on the same
16-bit inputs by
  - the rounding of the weights, uw of each: kept in two parts, the second part
    leaves u^2 of each (both calls); kept in the element type alone, it would be u;
  - fp32 arithmetic: a score is a sum of D products, each addition off by at most
    2^-23 of the sum A of their absolute values, so a weight is off by at most
    2 D 2^-23 A, relatively; a sum over L tokens adds L 2^-23; exponentials, their
    arguments' rounding and merges stay below 2^-18.
All of these are relative to the absolute terms, whose sum is `base`:
    d = (uw + 2 D 2^-23 A + L 2^-23 + 2^-18) base.
Without a norm the output is off by factor |w| d + u |out|.  With it, out =
factor w o / r, r = sqrt(mean(o^2) + eps): by the triangle inequality r is off
by at most e = sqrt(mean(d^2)), so with r' = max(r - e, sqrt(eps)) the output is
off by at most factor |w| (d + |o| e / r) / r', plus its own rounding u |out|, plus
the norm's arithmetic, 2^-20 |out| (a sum of at most 256 squares in fp32 in 8
terms a lane and 5 steps, a root).  fp16 outputs below the normal range are
off by half of 2^-24 instead.
"""

from __future__ import annotations

import math

import numpy as np
import torch

import oracle
from paged_kv_decode_24_gb300 import binding

PAGE = 16
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
HALF_STEP = {k: torch.finfo(v).eps / 2 for k, v in DT.items()}


def f64(t):
    return t.double().cpu().numpy()


def rope_table(positions, rot, base=10000.0, dtype=torch.float32):
    half = rot // 2
    a = torch.outer(torch.arange(positions, dtype=torch.float64),
                    base ** (-torch.arange(half, dtype=torch.float64) / half))
    return torch.cat([a.cos(), a.sin()], 1).to(dtype)


class Case:
    """Inputs of one ragged batch, from a seed, as torch CPU tensors.

    bad: {(sequence, page of the sequence): entry} of the block table that name
    pages which do not exist.  poison: rows that no sequence owns hold NaN."""

    def __init__(self, lens, qs=None, pairs=2, group=1, dim=64, dtype="fp16", seed=0, extra=5,
                 poison=False, scale=None, eps=1e-5, factor=0.5, weight=True, lam=None, bad=(),
                 amplitude=1.0):
        g = torch.Generator().manual_seed(seed)
        dt = DT[dtype]

        def n(*s):
            return (torch.randn(s, generator=g) * amplitude).to(dt)

        self.lens = list(lens)
        self.qs = [1] * len(lens) if qs is None else list(qs)
        self.kv, self.group, self.dim, self.dtype = 2 * pairs, group, dim, dtype
        self.hq = self.kv * group
        self.heads = self.hq // 2
        counts = [-(-x // PAGE) for x in lens]
        used = sum(counts)
        self.num_pages = used + extra
        self.max_pages = max(max(counts, default=0), 1) + 1
        perm = torch.randperm(self.num_pages, generator=g)[:used].to(torch.int32)
        self.table = torch.full((len(lens), self.max_pages), -7, dtype=torch.int32)
        self.k_pages = n(self.num_pages, self.kv, PAGE, dim)
        self.v_pages = n(self.num_pages, self.kv, PAGE, dim)
        owned = torch.zeros(self.num_pages, PAGE, dtype=torch.bool)
        at = 0
        for b, c in enumerate(counts):
            self.table[b, :c] = perm[at:at + c]
            for j in range(c):
                owned[perm[at + j], :min(PAGE, lens[b] - j * PAGE)] = True
            at += c
        for (b, j), entry in dict(bad).items():
            owned[self.table[b, j].long()] = False
            self.table[b, j] = entry
        if poison:
            for pool in (self.k_pages, self.v_pages):
                pool.transpose(1, 2)[~owned] = float("nan")
        self.T = sum(self.qs)
        self.q = n(self.T, self.hq, dim)
        self.k_new, self.v_new = n(self.T, self.kv, dim), n(self.T, self.kv, dim)
        self.lam = torch.rand(self.heads, generator=g) if lam is None else torch.full((self.heads,), lam)
        self.weight = 1 + 0.2 * torch.randn(2 * dim, generator=g) if weight else None
        self.eps, self.factor = eps, factor
        self.scale = dim ** -0.5 if scale is None else scale

    def shape(self):
        return binding.make_shape(len(self.lens), self.hq, self.kv, self.dim, PAGE, self.max_pages,
                                  self.num_pages, self.dtype)

    def want(self, rows=None, q=None, k_pages=None, v_pages=None, qs=None):
        return oracle.diff_attention(
            f64(self.q if q is None else q), f64(self.k_pages if k_pages is None else k_pages),
            f64(self.v_pages if v_pages is None else v_pages), self.table.numpy(), self.lens,
            self.qs if qs is None else qs, self.scale, f64(self.lam),
            None if self.weight is None else f64(self.weight), self.eps, self.factor, rows)

    def check(self, got, want, two_parts, what="", rows=None):
        """got [T][H][2D] against the oracle's tuple."""
        out, o, base, size = want
        g = f64(got)
        assert g.shape == out.shape
        if rows is not None:
            g, out, o, base, size = g[rows], out[rows], o[rows], base[rows], size[rows]
        assert np.all(np.isfinite(g)), f"{what}: non-finite output"
        u, longest = HALF_STEP[self.dtype], max(self.lens, default=0)
        uw = u * u if two_parts else u
        d = (uw + 2 * self.dim * 2.0**-23 * size[..., None] + longest * 2.0**-23 + 2.0**-18) * base
        w = np.ones(2 * self.dim) if self.weight is None else np.abs(f64(self.weight))
        f = abs(self.factor) * w
        if self.eps > 0:
            r = np.sqrt(np.mean(o * o, -1, keepdims=True) + self.eps)
            e = np.sqrt(np.mean(d * d, -1, keepdims=True))
            low = np.maximum(r - e, np.sqrt(self.eps))
            tol = f * (d + np.abs(o) * e / r) / low
        else:
            tol = f * d
        tol = tol + (u + 2.0**-20) * np.abs(out) + 2.0**-25
        err = np.abs(g - out)
        worst = float((err / tol).max(initial=0.0))
        assert worst <= 1.0, f"{what}: error {worst:.3g} of the bound"
        return worst


# --------------------------------------------------------------------------
# cases with exact scores

def sink(gap, dtype, dim, group, lens, qs):
    """A first token with values of zero stands `gap` log2 units above all others in both maps.
    Scores are exact: one product of a query's 1 with a multiple of 1/8 below 32."""
    c = Case(lens, qs, pairs=1, group=group, dim=dim, dtype=dtype, seed=gap, eps=0.0, factor=2.0**gap / 256,
             weight=False, lam=0.25, scale=float(np.float32(math.log(2))))
    g = torch.Generator().manual_seed(gap + 1)
    c.q.zero_()
    c.q[..., 0] = 1
    c.k_pages[..., 0] = -torch.randint(0, 8, c.k_pages.shape[:-1], generator=g).to(DT[dtype]) / 8
    c.v_pages.copy_((1 + c.v_pages.float() / 4).to(DT[dtype]))
    for b in range(len(lens)):
        c.k_pages[c.table[b, 0].long(), :, 0, 0] = gap
        c.v_pages[c.table[b, 0].long(), :, 0] = 0
    return c


def check_sink(c, got):
    """Beside the terms of tests/diff.py: exact scores leave the roundings of score x scale, of
    the difference to the reference and of the exponent's offset, each at most half a step of
    numbers up to 64 in log2 units, 3 x 2^-19 x ln 2 of a weight, and a scale off by 2^-24 of
    32 units.  A weight in two parts of fp16 is off by at most 2^-25, half of the smallest
    step, times the factor that weights are kept with: 2^-39 where a weight of 1 is 2^14."""
    out, o, base, _ = c.want()
    u, longest = HALF_STEP[c.dtype], max(c.lens)
    absolute = 0.0
    if c.dtype == "fp16":
        absolute = 2.0**-39 * (1 + abs(float(c.lam[0]))) * longest * float(c.v_pages.float().abs().max())
    rel = u * u + 3 * 2.0**-19 * 0.7 + 2.0**-19 + longest * 2.0**-23 + 2.0**-18
    tol = c.factor * (rel * base + absolute) + (u + 2.0**-20) * np.abs(out) + 2.0**-25
    err = np.abs(f64(got) - out)
    worst = float((err / tol).max())
    assert worst <= 1.0, f"error {worst:.3g} of the bound"


def exact_case(scale, dtype, lens, dim=64, group=2):
    """Whole scores of at most 32, so that they are exact, and of a few sizes, so that large
    scales leave several equal tokens on top."""
    c = Case(lens, pairs=1, group=group, dim=dim, dtype=dtype, seed=5, scale=scale, eps=0.0, factor=1.0, weight=False)
    for name in ("q", "k_pages"):
        x = torch.clamp((getattr(c, name).float() * 0.7).round(), -2, 2)
        x[..., 8:] = 0
        getattr(c, name).copy_(x.to(DT[dtype]))
    return c


def exact_want(c):
    """The oracle's tuple with the size that exact scores leave: score x scale and its difference
    to the maximum are each off by half a step of at most 32 x scale x log2(e) log2 units; from
    scale 10 on scores that differ do so by 14 units and more, whose weights, 2^-14 and below, are
    off by that much of 2^-14 of the row."""
    out, o, base, _ = c.want()
    units = 32 * min(c.scale, 1.0) * 1.45 * 2 * 2.0**-24 if c.scale < 10 else 2.0**-24
    return out, o, base, np.full(out.shape[:2], units / (2 * c.dim * 2.0**-23))


class Device:
    """A Case on the GPU."""

    def __init__(self, c: Case):
        self.c = c
        for name in ("table", "k_pages", "v_pages", "q", "k_new", "v_new", "lam"):
            setattr(self, name, getattr(c, name).cuda())
        self.shape = c.shape()
        self.seq_lens = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        weight = None if c.weight is None else c.weight.cuda()
        self.weights = binding.DiffWeights(self.lam, weight, c.eps, c.factor)
        self.plan = self.ws = None

    def make_plan(self, sms=152, **kw):
        self.plan = binding.DiffPlan(self.shape, self.c.lens, sms, **kw)
        self.ws = binding.alloc_workspace(self.plan)
        self.ws.fill_(0xFF)   # NaN partials: a row merged from an unwritten slot would show
        binding.diff_upload(self.plan, self.ws)
        return self

    def make_prefill_plan(self, **kw):
        self.plan = binding.PrefillPlan(self.shape, self.c.lens, self.c.qs, **kw)
        self.ws = binding.alloc_workspace(self.plan)
        binding.prefill_upload(self.plan, self.ws)
        return self

    def empty_out(self):
        return torch.full((self.c.T, self.c.heads, 2 * self.c.dim), float("nan"),
                          dtype=DT[self.c.dtype], device="cuda")

    def decode(self, out=None, q=None, stream=None):
        out = self.empty_out() if out is None else out
        binding.diff_attention(self.shape, self.plan, self.weights, self.q if q is None else q,
                               self.k_pages, self.v_pages, self.table, self.seq_lens, self.c.scale,
                               out, self.ws, self.status, stream=stream)
        return out

    def prefill(self, out=None, q=None, stream=None):
        out = self.empty_out() if out is None else out
        binding.diff_prefill(self.shape, self.plan, self.weights, self.q if q is None else q,
                             self.k_pages, self.v_pages, self.table, self.seq_lens, self.c.scale,
                             out, self.ws, self.status, stream=stream)
        return out

    def done(self):
        torch.cuda.synchronize()
        return int(self.status.item())
