"""Timed cases of the operators that serve ragged batches of requests.

Three operators, used one after the other by a serving loop:

- ``tables``: row offsets, blocks of 64 rows, positions and pool slots of a
  batch, from the requests' lengths;
- ``norm``: the norm of queries and keys for each head, with the position
  rotation in the same pass;
- ``gdr``: the gated delta rule over a ragged batch (prompts, continued
  prompts and single tokens) with the states in the pool's slots.

``own`` False computes each in its plain form with elementary torch
operations; True calls the framework. ``exact`` gives the results from the
definitions in 64 bits.
"""
import math

import torch

own = False

BLOCK = 64          # rows of one block of the block tables
HALF = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ the cases
def listed():
    gdn = dict(op="gdr", hv=32, hk=16, d=128, gate="head", dtype="bf16", pool="fp32")
    kda = dict(gdn, hk=32, gate="channel")
    return [
        # one token of each running request of a full serving batch
        dict(name="tables step", op="tables", b=512, lo=1, hi=1, slots=2561, rows=512, fresh=0.02),
        # a thousand prompts admitted at once, the longest 500 rows
        dict(name="tables prompts", op="tables", b=1000, lo=0, hi=500, slots=4096, rows=262144, fresh=0.9),
        # the decode step's queries and keys: normalised in fp32, no rotation
        dict(name="norm step", op="norm", rows=256, hq=16, hk=16, d=128, mode="l2", rot=0, inter=False,
             din="bf16", dout="fp32", weight=False, far=0, pad=0),
        # a prompt's queries and keys out of a fused projection, half rotated
        dict(name="norm prompts", op="norm", rows=16384, hq=16, hk=16, d=128, mode="rms", rot=64, inter=False,
             din="bf16", dout="bf16", weight=True, far=0, pad=4096),
        # odd row count, shared key heads, adjacent pairs, positions far out
        dict(name="norm far odd", op="norm", rows=5003, hq=12, hk=4, d=64, mode="rms", rot=64, inter=True,
             din="fp16", dout="fp16", weight=False, far=1000000, pad=0),
        # one token for every request of the serving batch
        dict(gdn, name="gdr step", b=512, lo=1, hi=1, resume=1.0),
        # a few tokens for each request (drafted tokens), gates by key channel
        dict(kda, name="gdr few channel", b=128, lo=1, hi=6, resume=1.0),
        # one short prompt alone: latency
        dict(gdn, name="gdr one prompt", b=1, lo=1000, hi=1000, resume=0.0),
        # prompts of every length, empty ones and single tokens among them
        dict(gdn, name="gdr ragged", b=24, lo=0, hi=1900, resume=0.4),
        # one long document
        dict(gdn, name="gdr long", b=1, lo=32768, hi=32768, resume=0.0),
        # a full admission batch
        dict(gdn, name="gdr batch", b=32, lo=2048, hi=2048, resume=0.0),
        # prompts handed over into 8-bit states
        dict(gdn, name="gdr packed", pool="packed", b=48, lo=1, hi=420, resume=0.3),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "norm", "gdr", "gdr", "gdr"])
    if op == "tables":
        b, hi = _log_int(rng, 1, 3000), _log_int(rng, 1, 400)
        return dict(op=op, b=b, lo=rng.choice([0, 1, hi]), hi=hi, slots=b + _log_int(rng, 1, 2000),
                    rows=min(262144, b * hi), fresh=rng.random())
    if op == "norm":
        d = rng.choice([32, 64, 128])
        hk = rng.choice([1, 2, 3, 4, 8, 16])
        return dict(op=op, rows=_log_int(rng, 1, 12000), hq=hk * rng.choice([1, 2, 4]), hk=hk, d=d,
                    mode=rng.choice(["l2", "rms"]), rot=rng.choice([0, d // 2, d]), inter=rng.random() < 0.5,
                    din=rng.choice(["bf16", "fp16", "fp32"]), dout=rng.choice(["bf16", "fp16", "fp32"]),
                    weight=rng.random() < 0.5, far=rng.choice([0, 100000, 1000000]), pad=rng.choice([0, 64, 1024]))
    hk = rng.choice([1, 2, 4, 8, 16])
    d = rng.choice([64, 128, 128, 128])
    gate = rng.choice(["head", "head", "channel"])
    b = _log_int(rng, 1, 48)
    hi = _log_int(rng, 1, 2500 if gate == "head" and d == 128 else 300)
    return dict(op=op, hv=hk * rng.choice([1, 2]), hk=hk, d=d, gate=gate, dtype=rng.choice(["bf16", "bf16", "fp32"])
                if hi <= 300 else "bf16", pool=rng.choice(["fp32", "fp32", "packed"]), b=b, lo=rng.choice([0, 1, hi]),
                hi=hi, resume=rng.choice([0.0, 0.5, 1.0]))


def _lengths(case):
    """Lengths of the requests, the case's own: lo..hi, spread over their logarithm, host side."""
    b, lo, hi = case["b"], case["lo"], case["hi"]
    gen = torch.Generator().manual_seed(100003 * b + hi)
    if lo == hi:
        return torch.full((b,), hi, dtype=torch.int64)
    u = torch.rand(b, generator=gen)
    n = torch.exp(u * math.log(hi + 1.0)).to(torch.int64)
    return n.clamp(max(lo, 0), hi) if lo else (n - (u < 0.1).to(torch.int64)).clamp(0, hi)


# ----------------------------------------------------------------- the inputs
def prepare(case, seed):
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return {"tables": _prepare_tables, "norm": _prepare_norm, "gdr": _prepare_gdr}[case["op"]](case, host, gen)


def _prepare_tables(case, host, gen):
    b, slots, rows = case["b"], case["slots"], case["rows"]
    lengths = _lengths(case)
    past = torch.randint(1, 4000, (b,), generator=host)
    perm = torch.randperm(slots, generator=host)[:b]
    fresh = torch.rand(b, generator=host) < case["fresh"]
    used = torch.rand(slots, generator=host) < 0.3      # slots of requests outside this batch
    used[perm] = ~fresh
    i32 = lambda x: x.to(torch.int32).cuda()  # noqa: E731
    z = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    s = dict(case=case, lengths=i32(lengths), past=i32(torch.where(fresh, 0, past)),
             slot_ids=i32(torch.where(fresh, -1, perm)), used=used.to(torch.uint8).cuda(),
             cu_seqlens=z(b + 1), cu_blocks=z(b + 1), positions=z(rows), block_req=z(rows // BLOCK + b),
             slot_out=z(b), used_out=torch.zeros(slots, dtype=torch.uint8, device="cuda"))
    return s


def _prepare_norm(case, host, gen):
    rows, hq, hk, d, pad = (case[x] for x in ("rows", "hq", "hk", "d", "pad"))
    # one projection holds q, k and `pad` further columns of each row
    x = torch.randn((rows, (hq + hk) * d + pad), device="cuda", generator=gen)
    x = (x * torch.exp(0.5 * torch.randn((rows, 1), device="cuda", generator=gen))).to(HALF[case["din"]])
    s = dict(case=case, q=x[:, :hq * d].unflatten(1, (hq, d)), k=x[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d)),
             wq=None, wk=None, positions=None)
    if case["weight"]:
        s["wq"], s["wk"] = (1 + 0.2 * torch.randn((2, d), device="cuda", generator=gen)).unbind(0)
    if case["rot"]:
        start = torch.randint(0, case["far"] + 1, (1,), generator=host).item()
        s["positions"] = (start + torch.arange(rows, device="cuda")).to(torch.int32)
    out = HALF[case["dout"]]
    s["q_out"] = torch.zeros((rows, hq, d), dtype=out, device="cuda")
    s["k_out"] = torch.zeros((rows, hk, d), dtype=out, device="cuda")
    return s


def _unit(x):
    return x / x.square().sum(-1, keepdim=True).sqrt()


def _prepare_gdr(case, host, gen):
    b, hv, hk, d = case["b"], case["hv"], case["hk"], case["d"]
    n = _lengths(case)
    rows = max(1, int(n.sum()))
    dt = HALF[case["dtype"]]
    rnd = lambda *shape: torch.randn(shape, device="cuda", generator=gen)  # noqa: E731
    # keys share a direction, as the outputs of an activation do
    k = _unit(rnd(rows, hk, d) + 0.5 * rnd(1, hk, d)).to(dt)
    q = _unit(rnd(rows, hk, d) + 0.5 * rnd(1, hk, d)).to(dt)
    half_life = 2.0 ** (10 * torch.rand((hv, d) if case["gate"] == "channel" else (hv,), device="cuda", generator=gen))
    g = torch.exp2(-torch.exp(0.2 * rnd(rows, *half_life.shape)) / half_life)
    resume = torch.rand(b, generator=host) < case["resume"]
    past = torch.where(resume, torch.randint(1, 4000, (b,), generator=host), 0)
    n_slots = b + 3
    slot_ids = torch.randperm(n_slots, generator=host)[:b]
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)])
    blocks = torch.cat([torch.zeros(1, dtype=torch.int64), ((n + BLOCK - 1) // BLOCK).cumsum(0)])
    req = torch.repeat_interleave(torch.arange(b), (n + BLOCK - 1) // BLOCK)
    block_req = torch.zeros(rows // BLOCK + b, dtype=torch.int64)
    block_req[:req.numel()] = req
    i32 = lambda x: x.to(torch.int32).cuda()  # noqa: E731
    s = dict(case=case, q=q, k=k, v=rnd(rows, hv, d).to(dt), beta=torch.sigmoid(rnd(rows, hv)), g=g,
             o=torch.zeros((rows, hv, d), dtype=dt, device="cuda"), past=i32(past), slot_ids=i32(slot_ids),
             cu_seqlens=i32(cu), cu_blocks=i32(blocks), block_req=i32(block_req), lengths=i32(n),
             max_len=int(n.max()), longest=int(n.max()))
    if case["pool"] == "packed":
        # 8-bit states, stored as codes, a scale for each row and fixed
        # column scales: one head record is d fp16 row scales, then d rows of d bytes
        s["col"] = torch.exp(0.3 * rnd(hv, d))
        codes = torch.randint(1, 256, (n_slots, hv, d, d), device="cuda", generator=gen, dtype=torch.uint8)
        r = (0.002 * torch.exp(0.3 * rnd(n_slots, hv, d))).to(torch.float16)
        s["pool"] = torch.cat([r.view(torch.uint8).reshape(n_slots, hv, 2 * d), codes.reshape(n_slots, hv, d * d)],
                              -1).reshape(-1)
        s["values"] = torch.zeros((n_slots, hv, d, d), device="cuda")
    else:
        s["pool"] = 0.1 * rnd(n_slots, hv, d, d)
    if own:  # the handle and the workspace that a serving loop keeps
        import numpy as np
        from quantized_linear_attention_sq_b200 import SQ_FMT_FP32, SQ_FMT_PACKED, SQ_GATE_HEAD, SQ_GATE_KEY_CHANNEL
        from quantized_linear_attention_sq_b200.ragged import BatchTables
        from quantized_linear_attention_sq_b200.state import StatePool
        channel = case["gate"] == "channel"
        kind = SQ_GATE_KEY_CHANNEL if channel else SQ_GATE_HEAD
        if case["pool"] == "packed":
            unit = (hv, d) if channel else (hv,)
            s["handle"] = StatePool(n_slots, hv, hk, d, kind, SQ_FMT_PACKED, np.full(unit, 8, np.int8),
                                    np.zeros(unit, np.uint8), s["col"].cpu().numpy(), np.ones((hv, d), np.float32))
        else:
            s["handle"] = StatePool(n_slots, hv, hk, d, kind, SQ_FMT_FP32)
        s["tables"] = BatchTables(cu_seqlens=s["cu_seqlens"], cu_blocks=s["cu_blocks"], block_req=s["block_req"],
                                  past=s["past"])
        s["workspace"] = s["handle"].new_ragged_workspace(b, rows, s["max_len"], dt)
    return s


# ---------------------------------------------------------------- one pass
def run(state):
    return {"tables": _run_tables, "norm": _run_norm, "gdr": _run_gdr}[state["case"]["op"]](state)


def _run_tables(s):
    if own:
        from quantized_linear_attention_sq_b200.ragged import batch_tables
        batch_tables(s["lengths"], s["past"], s["cu_seqlens"], s["cu_blocks"], s["positions"], s["block_req"],
                     slot_ids=s["slot_ids"], slot_used=s["used"], slot_out=s["slot_out"], used_out=s["used_out"])
    else:
        rows, b = s["positions"].numel(), s["lengths"].numel()
        cu = torch.cat([s["lengths"].new_zeros(1), s["lengths"].clamp(min=0).cumsum(0)]).clamp(max=rows)
        n = cu[1:] - cu[:-1]
        blocks = torch.cat([cu.new_zeros(1), ((n + BLOCK - 1) // BLOCK).cumsum(0)])

        def owner(ends, size):  # the request that each of `size` entries belongs to
            starts = torch.zeros(size + 1, dtype=torch.int64, device="cuda").index_add_(
                0, ends[1:-1].long(), torch.ones(b - 1, dtype=torch.int64, device="cuda"))
            return starts[:size].cumsum(0)

        row = torch.arange(rows, device="cuda")
        req = owner(cu, rows)
        at = torch.arange(s["block_req"].numel(), device="cuda")
        s["cu_seqlens"].copy_(cu)
        s["cu_blocks"].copy_(blocks)
        s["positions"].copy_(torch.where(row < cu[-1], row - cu[req] + s["past"][req], s["positions"]))
        s["block_req"].copy_(torch.where(at < blocks[-1], owner(blocks, at.numel()), s["block_req"]))
        # the r-th request without a slot takes the r-th free slot
        free, need = s["used"] == 0, s["slot_ids"] < 0
        slot_rank, rank = free.cumsum(0) - 1, need.cumsum(0) - 1
        size = free.numel()
        of_rank = torch.full((size + 1,), -1, dtype=torch.int64, device="cuda")
        of_rank.scatter_(0, torch.where(free, slot_rank, size), torch.arange(size, device="cuda"))
        of_rank[size] = -1
        s["slot_out"].copy_(torch.where(need, of_rank[rank.clamp(0, size)], s["slot_ids"]))
        s["used_out"].copy_(torch.where(free & (slot_rank < need.sum()), 1, s["used"]))
    return {k: s[k] for k in ("cu_seqlens", "cu_blocks", "positions", "block_req", "slot_out", "used_out")}


NORM_EPS = 1e-6
ROT_BASE = 10000.0


def _run_norm(s):
    c = s["case"]
    scale = c["d"] ** -0.5
    if own:
        from quantized_linear_attention_sq_b200.ragged import qk_norm
        qk_norm(s["q"], s["k"], s["q_out"], s["k_out"], mode=c["mode"], eps=NORM_EPS, q_weight=s["wq"],
                k_weight=s["wk"], q_scale=scale, positions=s["positions"], rot_dim=c["rot"], base=ROT_BASE,
                interleaved=c["inter"])
        return s["q_out"], s["k_out"]
    rot = c["rot"]
    if rot:
        freq = ROT_BASE ** (-torch.arange(rot // 2, device="cuda", dtype=torch.float64) * 2 / rot)
        angle = s["positions"].double()[:, None] * freq
        cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    for x, w, f, out in ((s["q"], s["wq"], scale, s["q_out"]), (s["k"], s["wk"], 1.0, s["k_out"])):
        x = x.float()
        sq = x.square()
        x = x / ((sq.sum(-1, keepdim=True) if c["mode"] == "l2" else sq.mean(-1, keepdim=True)) + NORM_EPS).sqrt()
        if w is not None:
            x = x * w
        x = x * f
        if rot:
            a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if c["inter"] else (x[..., :rot // 2], x[..., rot // 2:rot])
            a, b = a * cos - b * sin, b * cos + a * sin
            turned = torch.stack([a, b], -1).flatten(-2) if c["inter"] else torch.cat([a, b], -1)
            x = torch.cat([turned, x[..., rot:]], -1)
        out.copy_(x)
    return s["q_out"], s["k_out"]


def _unpack(s):
    """fp32 states of an 8-bit pool: code x row scale x column scale."""
    c = s["case"]
    hv, d = c["hv"], c["d"]
    rec = s["pool"].view(-1, hv, 2 * d + d * d)
    r = rec[..., :2 * d].contiguous().view(torch.float16)
    q = rec[..., 2 * d:].reshape(-1, hv, d, d)
    return (q.float() - 128) * r.float()[..., None] * s["col"][:, None, :], rec


def _scale_up(x):
    """fp32 to fp16, rounded toward plus infinity."""
    h = x.to(torch.float16)
    return torch.where(h.float() < x, (h.view(torch.int16) + 1).view(torch.float16), h)


def _pack(s, rec, S, slots):
    t = S * (1 / s["col"])[:, None, :]
    r = _scale_up(t.abs().amax(-1) / 127)
    q = torch.where(r[..., None] > 0, (t / r.float()[..., None]), 0.0).round().clamp(-127, 127)
    n, hv, d = r.shape
    rec[slots] = torch.cat([r.view(torch.uint8).reshape(n, hv, 2 * d),
                            (q + 128).to(torch.uint8).reshape(n, hv, d * d)], -1)


def _run_gdr(s):
    c = s["case"]
    packed = c["pool"] == "packed"
    if own:
        s["handle"].prefill_ragged(s["pool"], s["q"], s["k"], s["v"], s["beta"], s["g"], s["o"], s["tables"],
                                   slot_ids=s["slot_ids"], max_len=s["max_len"], workspace=s["workspace"])
        if packed:
            s["handle"].dequantize_state(s["pool"], s["values"])
            return s["o"], s["values"].to(torch.bfloat16)
        return s["o"], s["pool"]
    b, hv, d = c["b"], c["hv"], c["d"]
    share = hv // c["hk"]
    slots = s["slot_ids"].long()
    if packed:
        every, rec = _unpack(s)
    else:
        every = s["pool"]
    S = torch.where((s["past"] > 0)[:, None, None, None], every[slots], 0.0)
    start, n = s["cu_seqlens"][:-1].long(), s["lengths"].long()
    width = BLOCK if s["longest"] > 8 and c["gate"] == "head" else 1
    last = s["q"].shape[0] - 1
    one = torch.eye(width, device="cuda")
    i, j = torch.arange(width, device="cuda")[:, None], torch.arange(width, device="cuda")
    for t0 in range(0, s["longest"], width):
        # rows [b, width] of this block of every request; `live` the ones that exist
        t = t0 + torch.arange(width, device="cuda")
        live = t < n[:, None]
        row = (start[:, None] + t).clamp(max=last)
        heads = lambda x: x[row].float().transpose(1, 2)  # noqa: E731  [b, heads, width, ...]
        q, k = (heads(s[x]).repeat_interleave(share, 1) for x in ("q", "k"))
        v, beta = heads(s["v"]), torch.where(live[:, None], heads(s["beta"]), 0.0)
        alive = live.view(b, 1, width, *([1] * (s["g"].dim() - 2)))
        g = torch.where(alive, s["g"][row].transpose(1, 2), 1.0)
        if width == 1:  # token by token
            S = (g[:, :, 0, :, None] if c["gate"] == "channel" else g[:, :, 0, None, None]) * S
            u = beta * (v[:, :, 0] - (S * k[:, :, 0, :, None]).sum(-2))
            S = S + k[:, :, 0, :, None] * u[:, :, None]
            o = (S * q[:, :, 0, :, None]).sum(-2)[:, :, None]
        else:
            # decay from the end of token j to the end of token i: exp(G_i - G_j)
            G = g.double().log().cumsum(-1)
            decay = torch.where(i >= j, (G[..., :, None] - G[..., None, :]).exp(), 0.0).float()
            kk = k @ k.transpose(-1, -2)
            A = torch.where(i > j, beta[..., None] * decay * kk, 0.0)
            # inverse of 1 + A, blocks of doubling size along the diagonal
            T = one.expand_as(A)
            for level in range(6):
                pair = (i >> (level + 1) == j >> (level + 1)) & (i >> level != j >> level)
                T = T - T @ (torch.where(pair, A, 0.0) @ T)
            EG = G.exp().float()[..., None]
            u = T @ (beta[..., None] * (v - EG * (k @ S)))
            o = EG * (q @ S) + torch.where(i >= j, decay * (q @ k.transpose(-1, -2)), 0.0) @ u
            S = EG[..., -1:, :] * S + ((G[..., -1:] - G).exp().float()[..., None] * k).transpose(-1, -2) @ u
        at = torch.where(live, row, last + 1).flatten()
        o = o.transpose(1, 2).flatten(0, 1).to(s["o"].dtype)
        grown = torch.cat([s["o"], s["o"][:1]])
        grown[at] = o
        s["o"].copy_(grown[:-1])
    if packed:
        _pack(s, rec, S, slots)
        return s["o"], _unpack(s)[0].to(torch.bfloat16)
    s["pool"][slots] = S
    return s["o"], s["pool"]


# ------------------------------------------------------------ work of one pass
def work(case):
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    if case["op"] == "tables":
        rows = min(case["rows"], int(_lengths(case).sum()))
        return {"bytes": 4.0 * (5 * case["b"] + rows + rows / BLOCK) + 2.0 * case["slots"], "flops": float(rows)}
    if case["op"] == "norm":
        n = float(case["rows"] * (case["hq"] + case["hk"]) * case["d"])
        return {"bytes": n * (size[case["din"]] + size[case["dout"]]), "flops": 8 * n}
    b, hv, hk, d = (case[x] for x in ("b", "hv", "hk", "d"))
    rows = int(_lengths(case).sum())
    act = rows * (size[case["dtype"]] * d * (2 * hk + 2 * hv) + 4 * hv * (1 + (d if case["gate"] == "channel" else 1)))
    state = b * hv * d * (d * 4 if case["pool"] == "fp32" else d + 2)
    return {"bytes": float(act + state * (1 + case["resume"])), "flops": 6.0 * d * d * hv * rows}


# --------------------------------------------------------- results in 64 bits
def exact(case, seed):
    if case["op"] == "tables":
        return None
    s = prepare(case, seed)
    return _exact_norm(s) if case["op"] == "norm" else _exact_gdr(s)


def _exact_norm(s):
    c, rot = s["case"], s["case"]["rot"]
    out = []
    for x, w, f in ((s["q"], s["wq"], c["d"] ** -0.5), (s["k"], s["wk"], 1.0)):
        y = x.double()
        total = torch.einsum("rhc,rhc->rh", y, y)[..., None]
        y = y * torch.rsqrt((total if c["mode"] == "l2" else total / c["d"]) + NORM_EPS) * f
        y = y if w is None else y * w.double()
        if rot:
            first, second = (slice(0, rot, 2), slice(1, rot, 2)) if c["inter"] else (slice(0, rot // 2), slice(rot // 2, rot))
            power = torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot
            turn = torch.polar(torch.ones((), device="cuda", dtype=torch.float64),
                               s["positions"].double()[:, None, None] / ROT_BASE ** power)
            z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * turn
            y[..., first], y[..., second] = z.real, z.imag
        out.append(y)
    return tuple(out)


def _exact_gdr(s):
    """Token by token over all requests at once; a request that has ended keeps its state."""
    c = s["case"]
    b, hv, hk, d = c["b"], c["hv"], c["hk"], c["d"]
    pool = s["pool"]
    if c["pool"] == "packed":
        raw = s["pool"].reshape(-1, hv, (d + 2) * d)
        r = raw[:, :, :2 * d].contiguous().view(torch.float16).double()
        col = s["col"].double()
        pool = torch.einsum("shij,shi,hj->shij", raw[:, :, 2 * d:].reshape(-1, hv, d, d).double() - 128, r, col)
    pool = pool.double()
    if b * s["longest"] * hv * d * d > 1.2e12:
        return None
    S = pool[s["slot_ids"].long()]
    S[s["past"] <= 0] = 0
    o = s["o"].double()
    first, n = s["cu_seqlens"].tolist()[:-1], s["lengths"].tolist()
    order = sorted(range(b), key=lambda x: -n[x])           # longest first: the live ones stay in front
    S = S[order]
    first = torch.tensor([first[x] for x in order], device="cuda")
    sizes = [n[x] for x in order]
    group = torch.arange(hv, device="cuda") // (hv // hk)
    live = b
    for t in range(s["longest"]):
        while sizes[live - 1] <= t:
            live -= 1
        row, X = first[:live] + t, S[:live]
        k, q = s["k"][row][:, group].double(), s["q"][row][:, group].double()
        gate = s["g"][row].double()
        X.mul_(gate[..., None] if gate.dim() == 3 else gate[..., None, None])
        u = s["v"][row].double() - (k[..., None, :] @ X)[..., 0, :]
        X.add_(k[..., :, None] * (s["beta"][row].double()[..., None] * u)[..., None, :])
        o[row] = (q[..., None, :] @ X)[..., 0, :]
    if c["pool"] == "packed":
        T = S / s["col"].double()[:, None, :]
        top = T.abs().amax(-1) / 127
        r = top.to(torch.float16)
        r = torch.where(r.double() < top, torch.nextafter(r, torch.full_like(r, float("inf"))), r).double()[..., None]
        S = torch.where(r > 0, torch.round(T / r).clamp(-127, 127) * r, 0.0) * s["col"].double()[:, None, :]
    pool[s["slot_ids"].long()[order]] = S
    return o, pool
