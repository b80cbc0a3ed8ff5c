"""Plain 64-bit definitions of the ragged-batch operators, for their tests."""
import torch

from quantized_linear_attention_sq_b200 import _abi


def tables(lengths, past, max_rows, slot_ids=None, used=None):
    """Every table of sq_batch_tables as Python lists (written entries only)."""
    cu, cb, pos, req, status = [0], [0], [], [], 0
    for b, n in enumerate(lengths):
        n = max(n, 0)
        if cu[-1] + n > max_rows:
            n, status = max_rows - cu[-1], _abi.SQ_STATUS_TRUNCATED
        p = past[b] if past is not None else 0
        pos += [p + t for t in range(n)]
        blocks = -(-n // _abi.SQ_RAGGED_BLOCK)
        req += [b] * blocks
        cu.append(cu[-1] + n)
        cb.append(cb[-1] + blocks)
    out = dict(cu_seqlens=cu, cu_blocks=cb, positions=pos, block_req=req)
    if slot_ids is not None:
        slot_out, used_out = list(slot_ids), list(used)
        for b, s in enumerate(slot_ids):
            if s < 0:
                free = [x for x, u in enumerate(used_out) if not u]
                slot_out[b] = free[0] if free else -1
                if free:
                    used_out[free[0]] = 1
                else:
                    status |= _abi.SQ_STATUS_NO_SLOT
        out.update(slot_out=slot_out, used_out=used_out)
    out["status"] = status
    return out


def norm(x, mode, eps, weight, scale, positions, rot, base, interleaved):
    """x [rows, heads, d] -> fp64."""
    x = x.double()
    sq = x.square()
    x = x / ((sq.sum(-1, keepdim=True) if mode == "l2" else sq.mean(-1, keepdim=True)) + eps).sqrt()
    if weight is not None:
        x = x * weight.double()
    x = x * scale
    if rot:
        i = torch.arange(rot // 2, dtype=torch.float64, device=x.device)
        angle = positions.double()[:, None] * base ** (-2 * i / rot)
        c, s = angle.cos()[:, None], angle.sin()[:, None]
        first = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
        second = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
        a, b = x[..., first].clone(), x[..., second].clone()
        x[..., first], x[..., second] = a * c - b * s, b * c + a * s
    return x


def recurrence(q, k, v, beta, g, S):
    """The gated delta rule over the rows of one request in fp64: q, k [n, h_k,
    d], v [n, h_v, d], beta [n, h_v], g [n, h_v(, d)], S [h_v, d, d].
    Returns (o [n, h_v, d], S after the last row)."""
    S = S.double().clone()
    n, hv, d = v.shape
    rep = hv // q.shape[1]
    o = torch.zeros((n, hv, d), dtype=torch.float64, device=v.device)
    for t in range(n):
        kt, qt = (x[t].double().repeat_interleave(rep, 0) for x in (k, q))
        gt = g[t].double().clamp(0, 1)
        S = (gt[:, :, None] if gt.dim() == 2 else gt[:, None, None]) * S
        u = beta[t].double()[:, None] * (v[t].double() - torch.einsum("hij,hi->hj", S, kt))
        S = S + kt[:, :, None] * u[:, None, :]
        o[t] = torch.einsum("hij,hi->hj", S, qt)
    return o, S
