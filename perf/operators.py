"""Latent attention over a paged cache: the measured operators and their cases.

A layer with latent attention caches one vector a token, shared by all heads:
the latent (512 values) and the rotary key (64 values).  Four operators work
on that cache:

* ``append``    writes a step's new rows into their pages;
* ``gather``    reads whole sequences back as dense rows (to expand them into
                keys and values of each head);
* ``absorbed``  attention of queries that already hold the key projection,
                over the cached rows themselves: scores over all 576 values,
                output the weighted mean of the 512 latent values;
* ``expanded``  causal attention of a prompt over keys and values that were
                expanded for each head, the rotary key shared by the heads.

``own`` False: the plain form in elementary torch operations, fp32 inside.
``own`` True: the calls of paged_kv_decode_24_gb300.binding.
"""

import math

import torch

own = False

LATENT, ROPE = 512, 64
ROW = LATENT + ROPE
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# --------------------------------------------------------------------------
# cases

def listed():
    return [
        # one new token of one conversation: pure latency
        _case("append_one_token", "append", batch=1, lo=1000, hi=1000, q=1, page=16, dtype="bf16"),
        # the prompts of a few requests, written at once (odd counts, rows sliced
        # out of a wider projection)
        _case("append_prompts", "append", batch=24, lo=301, hi=4099, q=4099, page=64, dtype="bf16"),
        # two short contexts read back ahead of a chunk of a prompt
        _case("gather_short", "gather", batch=2, lo=33, hi=500, q=1, page=16, dtype="fp16"),
        # the contexts of a batch of long documents read back
        _case("gather_contexts", "gather", batch=20, lo=900, hi=12007, q=1, page=16, dtype="bf16"),
        # the first tokens of one conversation, few heads: pure latency
        _case("absorbed_first_tokens", "absorbed", batch=1, lo=77, hi=77, q=1, heads=16, page=16,
              dtype="fp16"),
        # a decode batch where the heads are spread over several GPUs: bound by the
        # cache's bytes
        _case("absorbed_batch_16_heads", "absorbed", batch=64, lo=500, hi=8001, q=1, heads=16,
              page=64, dtype="bf16"),
        # a decode batch with all heads on one GPU: bytes and products near balance
        _case("absorbed_batch_128_heads", "absorbed", batch=32, lo=700, hi=8191, q=1, heads=128,
              page=64, dtype="bf16"),
        # two very long contexts, all heads: work split over the tokens
        _case("absorbed_long_128_heads", "absorbed", batch=2, lo=40001, hi=65537, q=1, heads=128,
              page=16, dtype="bf16"),
        # checking three drafted tokens a sequence
        _case("absorbed_drafts", "absorbed", batch=21, lo=200, hi=6003, q=3, heads=20, page=32,
              dtype="fp16"),
        # short prompts of a few heads, ragged
        _case("expanded_short", "expanded", batch=3, lo=1, hi=130, q=130, heads=5, head_dim=64,
              dtype="fp16"),
        # one long prompt
        _case("expanded_prompt", "expanded", batch=1, lo=8192, hi=8192, q=8192, heads=32,
              head_dim=128, dtype="bf16"),
        # chunks of long prompts behind their cached contexts, ragged
        _case("expanded_chunks", "expanded", batch=6, lo=1500, hi=7001, q=513, heads=16,
              head_dim=128, dtype="fp16"),
    ]


def _case(name, op, batch, lo, hi, q, dtype, page=16, heads=1, head_dim=128):
    c = {"op": op, "batch": batch, "lo": lo, "hi": hi, "q": q, "page": page, "heads": heads,
         "head_dim": head_dim, "dtype": dtype}
    return {"name": name, **c} if name else c


def _log(rng, lo, hi):
    """A whole number of [lo, hi], its logarithm uniform."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["append", "gather", "absorbed", "absorbed", "absorbed", "expanded", "expanded"])
    dtype = rng.choice(["fp16", "bf16"])
    page = rng.choice([16, 32, 64])
    if op in ("append", "gather"):
        batch = _log(rng, 1, 40)
        hi = _log(rng, 1, max(1, min(12000, 240000 // batch)))
        lo = rng.randint(1, hi)
        q = rng.choice([1, _log(rng, 1, hi)]) if op == "append" else 1
        return _case(None, op, batch, lo, hi, q, dtype, page)
    if op == "absorbed":
        heads = rng.choice([_log(rng, 1, 128), 16, 128])
        q = rng.choice([1, 1, rng.randint(2, 8)])
        batch = _log(rng, 1, 64)
        hi = _log(rng, 1, max(1, min(65537, 260000 // batch)))
        lo = rng.randint(max(1, hi // 8), hi)
        return _case(None, op, batch, lo, hi, q, dtype, page, heads)
    heads, batch = _log(rng, 1, 64), _log(rng, 1, 8)
    hi = _log(rng, 1, max(1, min(8192, int((8192 * 8192 * 32 / (batch * heads)) ** 0.5))))
    lo = rng.randint(max(1, hi // 8), hi)
    q = rng.choice([hi, _log(rng, 1, hi)])
    return _case(None, op, batch, lo, hi, q, dtype, page, heads, rng.choice([64, 128]))


def _lens(case):
    """The lengths of a ragged batch and its new tokens, from the case alone."""
    lo, hi = case["lo"], case["hi"]
    lens = [lo + ((i + 1) * 2654435761 % (1 << 32)) * (hi - lo + 1) // (1 << 32)
            for i in range(case["batch"])]
    return lens, [min(case["q"], n) for n in lens]


def work(case):
    lens, qs = _lens(case)
    n_q, n_k, h = sum(qs), sum(lens), case["heads"]
    pairs = sum(q * (n - q) + q * (q + 1) // 2 for n, q in zip(lens, qs))
    if case["op"] == "append":
        return {"bytes": 2 * n_q * ROW * 2, "flops": 0}
    if case["op"] == "gather":
        return {"bytes": 2 * n_k * ROW * 2, "flops": 0}
    if case["op"] == "absorbed":
        return {"bytes": 2 * (n_k * ROW + n_q * h * (ROW + LATENT)),
                "flops": 2 * pairs * h * (ROW + LATENT)}
    d = case["head_dim"]
    return {"bytes": 2 * (n_q * h * (d + ROPE + d) + n_k * (h * 2 * d + ROPE)),
            "flops": 2 * pairs * h * (d + ROPE + d)}


# --------------------------------------------------------------------------
# inputs

def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dt)

    lens, qs = _lens(case)
    n_q, n_k, h, d, page = sum(qs), sum(lens), case["heads"], case["head_dim"], case["page"]
    s = {"case": case, "lens": lens, "qs": qs, "scale": 1.0 / math.sqrt(d + ROPE), "dtype": dt}
    cu_q, cu_k = [0], [0]
    for n, q in zip(lens, qs):
        cu_q.append(cu_q[-1] + q)
        cu_k.append(cu_k[-1] + n)
    dev = {"cu_q": cu_q, "cu_k": cu_k, "lens_d": lens, "qs_d": qs}
    s.update({k: torch.tensor(v, dtype=torch.int64, device="cuda") for k, v in dev.items()})
    if case["op"] != "expanded":
        pages_of = [-(-n // page) for n in lens]
        used = sum(pages_of)
        pool = used + 7
        s["pages"] = normal(pool, page, ROW)
        order = torch.randperm(pool, generator=g, device="cuda")[:used].to(torch.int32)
        table = torch.zeros(len(lens), max(pages_of), dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(pages_of):
            table[b, :n] = order[at:at + n]
            at += n
        s["table"] = table
    if case["op"] == "append":
        # the projection that makes the latent and the rotary key also makes other values
        s["projected"] = normal(n_q, ROW + 160)
        s["c_new"], s["r_new"] = s["projected"][:, :LATENT], s["projected"][:, LATENT:ROW]
    elif case["op"] == "gather":
        s["rows"] = torch.empty(n_k, ROW, dtype=dt, device="cuda")
    elif case["op"] == "absorbed":
        s["q"] = normal(n_q, h, ROW)
        s["out"] = torch.empty(n_q, h, LATENT, dtype=dt, device="cuda")
    else:
        s["q"] = normal(n_q, h, d + ROPE)
        s["rows"] = normal(n_k, ROW)              # as read back from the cache
        s["kv"] = normal(n_k, h, 2 * d)           # as the expanding projection writes them
        s["k"], s["v"] = s["kv"][:, :, :d], s["kv"][:, :, d:]
        s["k_rope"] = s["rows"][:, LATENT:]
        s["out"] = torch.empty(n_q, h, d, dtype=dt, device="cuda")
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        from paged_kv_decode_24_gb300 import binding
        sms = torch.cuda.get_device_properties("cuda").multi_processor_count
        paged = "pages" in s
        shape = binding.make_latent_shape(
            case["batch"], case["heads"], case["head_dim"], case["page"],
            s["table"].shape[1] if paged else -(-max(s["lens"]) // case["page"]),
            s["pages"].shape[0] if paged else 1, case["dtype"])
        plan = binding.LatentPlan(shape, s["lens"], s["qs"], sms,
                                  form="expanded" if case["op"] == "expanded" else "absorbed")
        ws = binding.alloc_workspace(plan)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        binding.latent_upload(plan, ws)
        if case["op"] == "append":
            s["call"] = binding.prepare_latent_append(shape, plan, s["c_new"], s["r_new"], s["pages"],
                                                      s["table"], ws, status)
        elif case["op"] == "gather":
            s["call"] = binding.prepare_latent_gather(shape, plan, s["pages"], s["table"], s["rows"],
                                                      ws, status)
        elif case["op"] == "absorbed":
            s["call"] = binding.prepare_latent_attention(shape, plan, s["q"], s["pages"], s["table"],
                                                         s["scale"], s["out"], ws, status)
        else:
            s["call"] = binding.prepare_latent_prefill(shape, plan, s["q"], s["k"], s["k_rope"],
                                                       s["v"], s["scale"], s["out"], ws, status)
    return s


# --------------------------------------------------------------------------
# one pass

def run(s):
    op = s["case"]["op"]
    if own:
        s["call"]()
        return s["pages"] if op == "append" else s["rows"] if op == "gather" else s["out"]
    return {"append": _append, "gather": _gather, "absorbed": _absorbed, "expanded": _expanded}[op](s)


def _of_row(cu, n):
    """The sequence of each packed row, and the row's place within it."""
    at = torch.arange(n, device="cuda")
    b = torch.searchsorted(cu, at, right=True) - 1
    return b, at - cu[b]


def _append(s):
    page, pages = s["case"]["page"], s["pages"]
    b, i = _of_row(s["cu_q"], s["c_new"].shape[0])
    pos = s["lens_d"][b] - s["qs_d"][b] + i
    pages[s["table"][b, pos // page].long(), pos % page] = torch.cat([s["c_new"], s["r_new"]], 1)
    return pages


def _gather(s):
    page = s["case"]["page"]
    b, t = _of_row(s["cu_k"], s["rows"].shape[0])
    return s["pages"][s["table"][b, t // page].long(), t % page]


def _attend(q, k, v, pos, s):
    """q [B, heads, rows, .], k and v [B, heads, L, .] in fp32, padded; pos [B, rows]: the last
    token that each row sees of its own sequence."""
    j = torch.arange(k.shape[2], device="cuda")
    seen = (j <= pos[:, :, None]) & (j < s["lens_d"][:, None, None])
    x = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    x = x.masked_fill_(~seen[:, None], -math.inf)
    x = x.sub_(x.amax(-1, keepdim=True)).exp_()
    x = x.div_(x.sum(-1, keepdim=True))
    return torch.matmul(x, v)


def _padded(s):
    """Indices that pad packed query rows [T] to [B, longest], each row's last visible token,
    and indices back."""
    i = torch.arange(max(s["qs"]), device="cuda")
    at = torch.minimum(s["cu_q"][:-1, None] + i, s["cu_q"][1:, None] - 1)
    pos = (s["lens_d"] - s["qs_d"])[:, None] + i
    b, i = _of_row(s["cu_q"], sum(s["qs"]))
    return at, pos, b, i


def _absorbed(s):
    page, h = s["case"]["page"], s["case"]["heads"]
    t = torch.arange(max(s["lens"]), device="cuda")
    kv = s["pages"][s["table"][:, t // page].long(), t % page].float()[:, None]
    at, pos, b, i = _padded(s)
    q = s["q"][at].float().flatten(1, 2)[:, None]     # the heads share the keys: one product
    x = _attend(q, kv, kv[..., :LATENT], pos.repeat_interleave(h, 1), s)
    return x.unflatten(2, (-1, h))[b, 0, i].to(s["dtype"])


def _expanded(s):
    t = torch.arange(max(s["lens"]), device="cuda")
    rows = torch.minimum(s["cu_k"][:-1, None] + t, s["cu_k"][1:, None] - 1)
    k = s["k"][rows].float().transpose(1, 2)
    v = s["v"][rows].float().transpose(1, 2)
    r = s["k_rope"][rows].float()[:, None].expand(-1, k.shape[1], -1, -1)
    at, pos, b, i = _padded(s)
    q = s["q"][at].float().transpose(1, 2)
    x = _attend(q, torch.cat([k, r], 3), v, pos, s)
    return x[b, :, i].to(s["dtype"])


# --------------------------------------------------------------------------
# the definition in 64 bits, sequence by sequence

def exact(case, seed):
    s = _inputs(case, seed)
    page = case["page"]
    if case["op"] == "append":
        pool = s["pages"].double()
        at = 0
        for b, (n, q) in enumerate(zip(s["lens"], s["qs"])):
            for j in range((n - q) // page, -(-n // page)):       # pages that get rows
                first, last = max(n - q, j * page), min(n, (j + 1) * page)
                new = s["projected"][at + first - (n - q):at + last - (n - q), :ROW]
                pool[int(s["table"][b, j]), first - j * page:last - j * page] = new.double()
            at += q
        return pool
    if case["op"] == "expanded":
        out, at_q, at_k = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda"), 0, 0
        for n, q in zip(s["lens"], s["qs"]):
            later = torch.triu(torch.ones(q, n, dtype=torch.bool, device="cuda"), n - q + 1)
            for h in range(case["heads"]):
                k = torch.cat([s["k"][at_k:at_k + n, h], s["k_rope"][at_k:at_k + n]], 1).double()
                x = s["q"][at_q:at_q + q, h].double() @ k.T * s["scale"]
                w = torch.softmax(x.masked_fill(later, -math.inf), 1)
                out[at_q:at_q + q, h] = w @ s["v"][at_k:at_k + n, h].double()
            at_q, at_k = at_q + q, at_k + n
        return out
    seqs = []
    for b, n in enumerate(s["lens"]):
        own_pages = s["table"][b, :-(-n // page)].long()
        seqs.append(s["pages"][own_pages].reshape(-1, ROW)[:n])
    if case["op"] == "gather":
        return torch.cat(seqs).double()
    out, at = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda"), 0
    for n, q, rows in zip(s["lens"], s["qs"], seqs):
        rows = rows.double()
        for i in range(q):
            seen = rows[:n - q + i + 1]
            w = torch.softmax(s["q"][at + i].double() @ seen.T * s["scale"], 1)
            out[at + i] = w @ seen[:, :LATENT]
        at += q
    return out
