"""Plain 64-bit forms of the row formats and of attention over listed rows,
and random inputs for them (shared by the GPU tests of packing, attention and
pages).  Nothing here uses the library."""
from __future__ import annotations

import numpy as np
import torch

GROUP = 128
TYPE = {"bf16": torch.bfloat16, "f16": torch.float16, "fp8": torch.bfloat16}
INVALID = -1  # KVR_LOC_INVALID as int32


def row_bytes(fmt, d_v, d_rope):
    if fmt == "fp8":
        return d_v + (d_v // GROUP * 4 + 15) // 16 * 16 + 2 * d_rope
    return 2 * (d_v + d_rope)


def unpack(rows, fmt, d_v, d_rope):
    """Keys (float64, [..., d_v + d_rope]) of uint8 rows on the CPU."""
    rows = rows.cpu().contiguous()
    if fmt != "fp8":
        return rows.view(TYPE[fmt]).double()
    groups = d_v // GROUP
    code = rows[..., :d_v].contiguous().view(torch.float8_e4m3fn).double()
    scale = rows[..., d_v:d_v + 4 * groups].contiguous().view(torch.float32).double()
    rope = rows[..., rows.shape[-1] - 2 * d_rope:].contiguous().view(torch.bfloat16).double()
    return torch.cat([code * scale.repeat_interleave(GROUP, dim=-1), rope], -1)


def random_rows(rng, count, fmt, d_v, d_rope, size=1.0):
    """uint8 [count][row_bytes] on the CPU: normal latents (each row of its own
    size, so fp8 scales differ) and rope parts."""
    x = torch.from_numpy(rng.standard_normal((count, d_v))) * size
    x = x * torch.from_numpy(np.exp(0.5 * rng.standard_normal((count, 1))))
    rope = torch.zeros(count, d_rope, dtype=torch.float64)
    if d_rope:
        rope = torch.from_numpy(rng.standard_normal((count, d_rope)))
    if fmt != "fp8":
        return torch.cat([x, rope], 1).to(TYPE[fmt]).view(torch.uint8)
    x = x.view(count, d_v // GROUP, GROUP).float()
    scale = x.abs().amax(2) / 448
    code = (x / scale[..., None]).to(torch.float8_e4m3fn).view(count, d_v).view(torch.uint8)
    pad = torch.zeros(count, row_bytes(fmt, d_v, 0) - d_v - scale.shape[1] * 4, dtype=torch.uint8)
    return torch.cat([code, scale.contiguous().view(torch.uint8), pad,
                      rope.to(torch.bfloat16).contiguous().view(torch.uint8).view(count, -1)], 1)


def attend(q, keys, d_v, scale):
    """(out [heads, d_v], lse [heads], spread [heads, d_v]) in 64 bits of one
    query's heads over the listed keys; spread = sum_j p_j |v_j|, the size that
    rounding errors of the probabilities are measured against."""
    heads = q.shape[0]
    if keys.shape[0] == 0:
        z = torch.zeros(heads, d_v, dtype=torch.float64)
        return z, torch.full((heads,), -np.inf, dtype=torch.float64), z
    s = (q.double() @ keys.T) * scale
    lse = torch.logsumexp(s, 1)
    p = torch.exp(s - lse[:, None])
    v = keys[:, :d_v]
    return p @ v, lse, p @ v.abs()


def score_size(q, keys, scale):
    """max over rows of scale * sum_d |q_d k_d| for each head: what the
    rounding of 32-bit sums is measured against."""
    if keys.shape[0] == 0:
        return torch.zeros(q.shape[0], dtype=torch.float64)
    return (q.double().abs() @ keys.abs().T).amax(1) * abs(scale)
