"""The block-boundary operators in 64 bits on the CPU, from their formulas, with bounds for what fp32 arithmetic and one
rounding into the storage type may add. u = 2^-24 is half a step of fp32 relative to the value."""
import math

import torch

U = 2.0 ** -24
HALF = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # fp32 results: counted in u below
TINY = {torch.float32: 0.0, torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}        # half of fp16's smallest step
BLOCK = 128
DEPTH = 64  # additions behind one another in a row's sum: 8 per slot, 4 slots, 6 lane steps, 16 waves, and to spare


def f64(t):
    return None if t is None else t.detach().cpu().double()


def blocks(hidden):
    return -(-hidden // BLOCK)


def spread(scales, hidden):
    """One scale per block -> one per element."""
    return scales.repeat_interleave(BLOCK, -1)[..., :hidden]


def codes_f64(codes):
    return codes.cpu().view(torch.float8_e4m3fn).double()


def norm(ins, residual, gamma, eps):
    """h, rstd, y and the bounds on the kernel's fp32 h, rstd (relative) and y, before any rounding into the type."""
    n = len(ins)
    h = sum(f64(x) for x in ins)
    mag = sum(f64(x).abs() for x in ins)
    if residual is not None:
        h, mag, n = h + f64(residual), mag + f64(residual).abs(), n + 1
    g = f64(gamma)
    ms = (h * h).mean(1, keepdim=True)
    rstd = (ms + eps) ** -0.5
    y = h * rstd * g
    dh = (n - 1) * U * mag
    rel = 0.5 * (DEPTH * U + 2 * (dh * h.abs()).mean(1, keepdim=True) / (ms + eps)) + 4 * U
    dy = dh * rstd * g.abs() + y.abs() * (rel + 3 * U)
    return h, rstd, y, dh, rel, dy


def norm_bwd(ins, h, gamma, rstd, residual_grad, rows_deep):
    """dx, dgamma and their bounds; h in fp32 or exact, as the kernel reads it (one rounding where it is code x scale)."""
    n = len(ins)
    dy, mag = sum(f64(x) for x in ins), sum(f64(x).abs() for x in ins)
    g, r = f64(gamma), f64(rstd)[:, None]
    ddy = (n - 1) * U * mag
    xh = h * r
    gd = dy * g
    dgd = ddy * g.abs() + U * gd.abs()
    dxh = 2 * U * xh.abs()
    m = (gd * xh).mean(1, keepdim=True)
    dm = (dgd * xh.abs() + gd.abs() * dxh).mean(1, keepdim=True) + (DEPTH + 2) * U * (gd * xh).abs().mean(1, keepdim=True)
    dx = r * (gd - xh * m)
    ddx = r * (dgd + dxh * m.abs() + xh.abs() * dm + U * (xh * m).abs() + 2 * U * (gd.abs() + (xh * m).abs()))
    if residual_grad is not None:
        dx = dx + f64(residual_grad)
        ddx = ddx + U * (f64(residual_grad).abs() + dx.abs())
    term = dy * xh
    dgamma = term.sum(0)
    ddgamma = (ddy * xh.abs() + dy.abs() * dxh).sum(0) + (rows_deep + 2) * U * term.abs().sum(0)
    return dx, dgamma, ddx, ddgamma


def close(got, want, bound, what):
    """|got - want| <= bound + half a step of the type; NaN where want is NaN and nowhere else."""
    g = f64(got)
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(g), nan), f"{what}: NaN in other places"
    limit = bound + HALF[got.dtype] * (want.abs() + bound) + TINY[got.dtype]
    bad = ((g - want).abs() > limit) & ~nan & ~(g == want)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}: "
                           f"{g[bad][0].item()} for {want[bad][0].item()}, allowed {limit.expand_as(g)[bad][0].item()}")


def close_codes(codes, scales, want, bound, what):
    """The value code x scale within half a step of E4M3 of `want` (relative 2^-4; 2^-10 of the scale below the
    smallest normal), the scale within its own bound of the block's largest magnitude over 448."""
    rows, hidden = want.shape
    s = f64(scales)
    pad = blocks(hidden) * BLOCK - hidden
    amax = torch.nn.functional.pad(want.abs(), (0, pad)).view(rows, -1, BLOCK).amax(2)
    off = torch.nn.functional.pad(bound.expand_as(want), (0, pad)).view(rows, -1, BLOCK).amax(2)
    unit = amax == 0
    assert ((s - torch.where(unit, 1.0, amax / 448)).abs() <= off / 448 + 2 * U * amax / 448).all(), f"{what}: scales"
    v = codes_f64(codes) * spread(s, hidden)
    # codes are rounded from v * (448 / amax), two fp32 operations, instead of v / scale
    limit = (want.abs() + bound) * (2.0 ** -4 + 4 * U) + 2.0 ** -10 * spread(s, hidden) + bound
    bad = (v - want).abs() > limit
    assert not bad.any(), f"{what}: {int(bad.sum())} codes off, first at {bad.nonzero()[0].tolist()}"


def sort(ids, experts, align):
    """offsets, counts, pos, {row: slot} by going through the slots one after another."""
    members = [[] for _ in range(experts)]
    flat = ids.reshape(-1).tolist()
    for q, e in enumerate(flat):
        if 0 <= e < experts:
            members[e].append(q)
    offsets, pos, src = [0], [-1] * len(flat), {}
    for m in members:
        for i, q in enumerate(m):
            pos[q] = offsets[-1] + i
            src[offsets[-1] + i] = q
        offsets.append(offsets[-1] + -(-len(m) // align) * align)
    return offsets, [len(m) for m in members], pos, src


def combine(ys, pos, weights, addend):
    there = (pos >= 0)
    rows = torch.where(there[:, :, None], f64(ys)[pos.clamp(min=0).long()], 0.0)
    if weights is not None:
        rows = rows * torch.where(there, f64(weights), 0.0)[:, :, None]
    out, mag = rows.sum(1), rows.abs().sum(1)
    if addend is not None:
        out, mag = out + f64(addend), mag + f64(addend).abs()
    return out, (pos.shape[1] + 1) * U * mag


def combine_bwd(dout, ys, pos, weights, rows):
    """dys (zeros where no slot is), dweights and the bound of the latter."""
    tokens, k = pos.shape
    d, hidden = f64(dout), dout.shape[1]
    dys = torch.zeros(rows, hidden, dtype=torch.float64)
    there = pos >= 0
    t = torch.arange(tokens)[:, None].expand(tokens, k)
    dys[pos[there].long()] = d[t[there]] * f64(weights)[there][:, None]
    prod = f64(ys)[pos.clamp(min=0).long()] * d[:, None, :]
    dw = torch.where(there, prod.sum(2), 0.0)
    deep = math.ceil(hidden / 64) + 24  # a lane's own terms, then the lanes and the waves
    return dys, dw, torch.where(there, prod.abs().sum(2), 0.0) * deep * U
