"""Rotary positions, by the bounds of test_gpu_rotate.py: workgroups of several tokens;
outputs whose heads overlap are refused, those that only look as if they did are not."""
from __future__ import annotations

import pytest
import torch

from tests.test_gpu_rotate import DEV, TYPE, check, context, frequencies

pytestmark = pytest.mark.gpu


def overlap(n, heads, token, head, d):
    """Whether two heads share a value, from the definition."""
    at = sorted(t * token + h * head for t in range(n) for h in range(heads))
    return any(b - a < d for a, b in zip(at, at[1:]))


def test_outputs_that_overlap():
    """Every layout of a few heads by small strides."""
    from hierarchical_sparse_kv_resolve_amd import KvrError
    c, d, freq = context(), 4, frequencies(4)
    kinds = set()
    for n, heads in ((1, 1), (1, 3), (2, 2), (3, 4), (4, 3), (2, 7), (9, 2)):
        pos = torch.arange(n, dtype=torch.int32, device=DEV)
        x = torch.randn(n, heads, d, device=DEV)
        for token in (1, 3, 4, 5, 8, 10, 16, 20, 28, 33):
            for head in (2, 4, 6, 8, 9, 12, 20, 37):
                flat = torch.full((n * token + heads * head + d,), 7.0, device=DEV)
                out = flat.as_strided((n, heads, d), (token, head, 1))
                kw = dict(d_rot=4, layout="half")
                bad = overlap(n, heads, token, head, d)
                kinds.add((bad, token >= (heads - 1) * head + d or head >= (n - 1) * token + d))
                if bad:
                    for args in ((x, out), (out, None), (None, None, x, out)):
                        with pytest.raises(KvrError, match="heads of the output overlap"):
                            c.rotate_rows(n, pos, freq, *args, **kw)
                    assert (flat == 7).all()
                else:
                    c.rotate_rows(n, pos, freq, x, out, **kw)
                    check(out, x, pos, freq, 4, 0, "half", 1.0, False, "f32")
                    assert (flat == 7).sum() == flat.numel() - n * heads * d
    assert (False, False) in kinds and (True, False) in kinds  # interleaved ones of both kinds
    # with many heads, nothing but strides is looked at before the refusal
    flat = torch.zeros(1 << 20, device=DEV)
    out = flat.as_strided((30000, 1000, 4), (5, 7, 1))
    pos = torch.zeros(30000, dtype=torch.int32, device=DEV)
    with pytest.raises(KvrError, match="heads of the output overlap"):
        c.rotate_rows(30000, pos, freq, out, d_rot=4, layout="half")


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("n,heads,d_head,d_rot,kheads,typ", [
    (2049, 1, 16, 16, 0, "bf16"), (2047, 1, 16, 16, 0, "bf16"), (5001, 20, 16, 16, 2, "f16"),
    (32767, 1, 16, 16, 1, "bf16"), (32768, 3, 32, 16, 0, "f32"), (2049, 3, 128, 128, 1, "f32"),
    (5001, 1, 128, 128, 2, "bf16"), (32767, 2, 128, 128, 1, "bf16"), (8191, 5, 80, 20, 3, "bf16"),
    (2049, 1, 1024, 1024, 0, "bf16"), (5001, 1, 1024, 1024, 1, "f32"),
    (4097, 1, 1024, 1024, 1, "f16")])
def test_several_tokens_a_workgroup(n, heads, d_head, d_rot, kheads, typ, layout):
    """Enough tokens of few units for a workgroup to take several, the last one fewer;
    addresses aligned or not; each token at its own position."""
    g = torch.Generator(device=DEV).manual_seed(n + heads + d_rot)
    pos = torch.randint(0, 1 << 20, (n,), generator=g, device=DEV, dtype=torch.int32)
    freq, c, at = frequencies(d_rot), context(), d_head - d_rot
    for first in (0, 3):
        def make(h, d):
            wide = torch.randn(n, h, d + first, generator=g, device=DEV).to(TYPE[typ])
            return wide[..., first:]

        x, k = make(heads, d_head), make(kheads, d_rot) if kheads else None
        out = torch.full((n, heads, d_head), 7.0, device=DEV, dtype=TYPE[typ])
        kout = torch.full((n, kheads, d_rot), 7.0, device=DEV, dtype=TYPE[typ]) if kheads else None
        c.rotate_rows(n, pos, freq, x, out, k, kout, d_rot=d_rot, layout=layout, at=at)
        check(out, x, pos, freq, d_rot, at, layout, 1.0, False, typ)
        if kheads:
            check(kout, k, pos, freq, d_rot, 0, layout, 1.0, False, typ)
        c.rotate_rows(n, pos, freq, x, key=k, d_rot=d_rot, layout=layout, at=at)  # in place
        assert torch.equal(x, out) and (k is None or torch.equal(k, kout))
