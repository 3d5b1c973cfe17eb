"""Shared helpers of the latent attention tests: inputs on the host and the
device, the calls, and the tolerance.

Tolerance.  With u half a step of the element type relative to the value
(fp16 2^-11, bf16 2^-8), an output value o = sum_t w_t v_t differs from the
float64 one, on the same 16-bit inputs, by
  - the rounding of the result:                          u |o|
  - the rounding of each weight, where a kernel keeps the
    weights in the element type:                         u sum_t w_t |v_t|
  - fp32 arithmetic: a score is a sum of at most 576 products, each addition
    off by at most 2^-23 of the sum of absolute products A (an accumulator that
    drops bits instead of rounding them included), so a score is off by at most
    576 x 2^-23 A and a weight by twice that, relatively (the weight's own and
    the normaliser's); the output sum over L tokens adds L x 2^-23, and the
    exponential, its argument's rounding and the merge of pieces less than
    2^-18.
The sum of the three is the bound on each value.  Roundings do not all take
their largest size with the same sign, so the 2-norm of the difference is also
held to 2u of the output's norm: the two roundings have at most u / sqrt(3)
each as root mean square, the fp32 part is below u.
"""

from __future__ import annotations

import numpy as np
import torch

from paged_kv_decode_24_gb300 import binding

LATENT, ROPE, ROW = 512, 64, 576
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
HALF_STEP = {k: torch.finfo(v).eps / 2 for k, v in DT.items()}


def assert_latent_close(got, want, longest, dtype, what=""):
    """want: (out, base, size) of the oracle."""
    out, base, size = want
    g = np.asarray(got, np.float64)
    assert g.shape == out.shape
    assert np.all(np.isfinite(g)), f"{what}: non-finite output"
    u = HALF_STEP[dtype]
    fp32 = 2 * 576 * 2.0**-23 * size[..., None] + longest * 2.0**-23 + 2.0**-18
    tol = u * np.abs(out) + (u + fp32) * base + np.finfo(np.float16).tiny
    err = np.abs(g - out)
    worst = float((err / tol).max(initial=0.0))
    assert worst <= 1.0, f"{what}: error {worst:.3g} of the bound"
    norm = np.linalg.norm(out)
    rel = float(np.linalg.norm(err) / norm) if norm else 0.0
    assert rel <= 2 * u, f"{what}: 2-norm {rel:.3g} over {2 * u:.3g}"
    return worst, rel


class Case:
    """Inputs of one ragged batch, from a seed, as torch CPU tensors."""

    def __init__(self, lens, qs, heads=4, head_dim=128, page=16, dtype="fp16", seed=0, extra=5,
                 poison=False, scale=None):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.qs = list(lens), list(qs)
        self.heads, self.head_dim, self.page, self.dtype = heads, head_dim, page, dtype
        dt = DT[dtype]

        def n(*s):
            return torch.randn(s, generator=g).to(dt)

        counts = [-(-x // page) for x in lens]
        used = sum(counts)
        self.num_pages = used + extra
        self.max_pages = max(max(counts, default=0), 1) + 1
        perm = torch.randperm(self.num_pages, generator=g)[:used].to(torch.int32)
        self.table = torch.full((len(lens), self.max_pages), -7, dtype=torch.int32)
        self.pages = n(self.num_pages, page, ROW)
        if poison:   # rows that no sequence owns hold NaN
            owned = torch.zeros(self.num_pages, page, dtype=torch.bool)
        at = 0
        for b, c in enumerate(counts):
            self.table[b, :c] = perm[at:at + c]
            if poison:
                for j in range(c):
                    owned[perm[at + j], :min(page, lens[b] - j * page)] = True
            at += c
        if poison:
            self.pages[~owned] = float("nan")
        self.T, self.Tk = sum(qs), sum(lens)
        self.c_new, self.r_new = n(self.T, LATENT), n(self.T, ROPE)
        self.q = n(self.T, heads, ROW)
        self.qx = n(self.T, heads, head_dim + ROPE)
        self.kv = n(self.Tk, heads, 2 * head_dim)
        self.rows = n(self.Tk, ROW)
        self.scale = scale if scale is not None else (head_dim + ROPE) ** -0.5

    @property
    def k(self):
        return self.kv[:, :, :self.head_dim]

    @property
    def v(self):
        return self.kv[:, :, self.head_dim:]

    def shape(self):
        return binding.make_latent_shape(len(self.lens), self.heads, self.head_dim, self.page,
                                         self.max_pages, self.num_pages, self.dtype)


def f64(t):
    return t.double().numpy()


class Device:
    """A Case on the GPU, with a plan and its workspace."""

    def __init__(self, c, form="absorbed", num_sms=None, **plan):
        self.c = c
        for name in ("table", "pages", "c_new", "r_new", "q", "qx", "kv", "rows"):
            setattr(self, name, getattr(c, name).cuda())
        self.k, self.v = self.kv[:, :, :c.head_dim], self.kv[:, :, c.head_dim:]
        self.k_rope = self.rows[:, LATENT:]
        self.shape = c.shape()
        sms = num_sms or torch.cuda.get_device_properties("cuda").multi_processor_count
        self.plan = binding.LatentPlan(self.shape, c.lens, c.qs, sms, form=form, **plan)
        self.ws = binding.alloc_workspace(self.plan)
        self.ws.fill_(0xFF)   # NaN partials: a row merged from an unwritten slot would show
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        binding.latent_upload(self.plan, self.ws)

    def append(self):
        binding.latent_append(self.shape, self.plan, self.c_new, self.r_new, self.pages, self.table,
                              self.ws, self.status)

    def gather(self):
        rows = torch.full((self.c.Tk, ROW), float("nan"), dtype=DT[self.c.dtype], device="cuda")
        binding.latent_gather(self.shape, self.plan, self.pages, self.table, rows, self.ws,
                              self.status)
        return rows

    def attention(self, out=None, stream=None):
        if out is None:
            out = torch.full((self.c.T, self.c.heads, LATENT), float("nan"), dtype=DT[self.c.dtype],
                             device="cuda")
        binding.latent_attention(self.shape, self.plan, self.q, self.pages, self.table,
                                 self.c.scale, out, self.ws, self.status, stream=stream)
        return out

    def prefill(self, out=None, stream=None):
        if out is None:
            out = torch.full((self.c.T, self.c.heads, self.c.head_dim), float("nan"),
                             dtype=DT[self.c.dtype], device="cuda")
        binding.latent_prefill(self.shape, self.plan, self.qx, self.k, self.k_rope, self.v,
                               self.c.scale, out, self.ws, self.status, stream=stream)
        return out

    def done(self):
        torch.cuda.synchronize()
        return int(self.status.item())
