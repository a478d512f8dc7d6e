"""Dense attention backward on the GPU against the gradients' formulas in fp64, against differences of
the forward pass, and in the ways a training program calls it.

Tolerance. The reference takes the kernel's own inputs (bf16 tensors, the fp32 log-sum-exps) to the
formulas in fp64. The kernel adds, per element of a gradient, the rounding of P or dS to bf16 (each
factor off by at most u = 2^-8 relative, so the sum by at most u times the sum of the terms'
magnitudes), the rounding of the result (at most u relative), and fp32 arithmetic. In fp32 the
exponent x = scale log2(e) s - LSE log2(e) is off by at most
2^-24 (4 |s scale log2 e| + 4 |LSE log2 e| + 2 d scale log2(e) sum|q k|-like terms); with the inputs
here (|s scale| and |LSE| below 40) P is off by less than 2^-14 relative, the base-2 exponential by
2^-21, and dP - delta by 2^-24 (d + 8) times its terms' magnitudes A_ij = |dO_i|.|v_j| + |dO_i|.|O_i|
+ |dLSE_i|: less than 2^-15 A_ij. So, with M the sums of magnitudes taken in fp64:
  |error(dV_jc)| <= u sum_i P |dO| + 2^-13 sum_i P |dO| + u |dV_jc|
  |error(dQ_ic)| <= scale ((u + 2^-13) sum_j |dS| |k| + 2^-14 sum_j P A |k|) + u |dQ_ic|
and likewise for dK. fp32 accumulation over n terms adds at most n 2^-24 of the magnitudes (below
2^-11 for the lengths here); 2^-10 of the magnitudes covers it together with the terms above.
"""
import math

import pytest
import torch

U = 2.0 ** -8
SMALL = 2.0 ** -10


def reference(q, k, v, o, lse, do, dlse, causal, scale):
    """Gradients in fp64 and, for each, the bound on the kernel's error stated above."""
    q, k, v, o, lse, do = (t.double() for t in (q, k, v, o, lse, do))
    B, S, Hq, d = q.shape
    G = Hq // k.shape[2]
    ke, ve = k.repeat_interleave(G, 2), v.repeat_interleave(G, 2)
    s = torch.einsum("bihd,bjhd->bhij", q, ke) * scale
    p = torch.exp(s - lse.permute(0, 2, 1)[..., None])
    p = torch.where(torch.isneginf(lse).permute(0, 2, 1)[..., None], 0.0, p)
    if causal:
        p = p.masked_fill(torch.ones(S, S, dtype=torch.bool, device=q.device).triu(1), 0.0)
    delta = (do * o).sum(-1).permute(0, 2, 1)[..., None]
    dl = torch.zeros_like(delta) if dlse is None else dlse.double().permute(0, 2, 1)[..., None]
    ds = p * (torch.einsum("bihd,bjhd->bhij", do, ve) - (delta - dl))
    mag = p * (torch.einsum("bihd,bjhd->bhij", do.abs(), ve.abs())
               + (do * o).abs().sum(-1).permute(0, 2, 1)[..., None] + dl.abs())

    def to_kv(t):
        return t.unflatten(2, (k.shape[2], G)).sum(3)

    def dqk(w):
        return torch.einsum("bhij,bjhd->bihd", w, ke) * scale, to_kv(torch.einsum("bhij,bihd->bjhd", w, q)) * scale

    dv = to_kv(torch.einsum("bhij,bihd->bjhd", p, do))
    dq, dk = dqk(ds)
    ka, qa = ke.abs(), q.abs()
    w = U * ds.abs() + SMALL * (ds.abs() + mag / 16)
    tq = torch.einsum("bhij,bjhd->bihd", w, ka) * scale
    tk = to_kv(torch.einsum("bhij,bihd->bjhd", w, qa)) * scale
    tv = (U + SMALL) * to_kv(torch.einsum("bhij,bihd->bjhd", p, do.abs()))
    return (dq, dk, dv), (tq + U * dq.abs(), tk + U * dk.abs(), tv + U * dv.abs())


def inputs(B, S, Hq, Hkv, d, seed=0, gain=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed + 13 * S + Hq + d)
    r = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    q, k, v = (r(B, S, h, d).mul_(gain).bfloat16() for h in (Hq, Hkv, Hkv))
    return q, k, v, r(B, S, Hq, d).bfloat16(), r(B, S, Hq)


def check(grads, q, k, v, o, lse, do, dlse, causal, scale, what):
    want, tol = reference(q, k, v, o, lse, do, dlse, causal, scale)
    for name, got, ref, t in zip(("dq", "dk", "dv"), grads, want, tol):
        err = (got.double() - ref).abs()
        assert torch.isfinite(got).all(), f"{what}: non-finite {name}"
        assert (err <= t + 1e-30).all(), f"{what}: {name} off by {float((err / (t + 1e-30)).max()):.2f} of its bound"
        if float(ref.norm()) > 0:
            # errors of both signs: the whole tensor is far closer than the bound on each element
            rel = float(err.norm() / ref.norm())
            assert rel <= 2 * U, f"{what}: {name} relative error {rel}"


CASES = [
    # (B, S, Hq, Hkv, d, causal, dlse)
    (1, 1, 1, 1, 64, True, False),      # one token
    (2, 1, 4, 2, 128, False, True),
    (1, 2, 2, 1, 128, True, False),
    (1, 63, 2, 2, 64, True, True),
    (1, 64, 2, 2, 128, False, False),   # half a tile: the second warpgroup's columns are all padding
    (1, 65, 2, 1, 128, True, False),
    (1, 127, 3, 3, 64, False, False),
    (1, 128, 1, 1, 64, False, False),   # exactly one tile
    (1, 128, 1, 1, 128, True, False),
    (3, 129, 2, 2, 128, True, True),    # one row into the second tile
    (1, 129, 2, 2, 64, False, False),
    (1, 256, 2, 1, 64, True, False),
    (2, 300, 6, 2, 128, True, False),   # GQA 3
    (2, 300, 6, 2, 64, False, True),
    (1, 517, 8, 1, 128, False, False),  # one key/value head
    (1, 517, 8, 1, 64, True, False),
    (1, 900, 4, 4, 128, True, False),   # the ring of slots wraps several times
    (1, 900, 4, 2, 64, True, False),
    (1, 1200, 2, 2, 128, False, False),
    (1, 384, 64, 64, 64, True, False),  # more units than SMs, several chunks of heads
    (5, 260, 40, 8, 128, True, False),  # a last chunk with fewer heads
]


@pytest.mark.gpu
@pytest.mark.parametrize("B,S,Hq,Hkv,d,causal,with_dlse", CASES)
def test_bwd_matches_fp64(B, S, Hq, Hkv, d, causal, with_dlse):
    import io_aware_exact_flash_gb300 as fa

    q, k, v, do, dl = inputs(B, S, Hq, Hkv, d)
    dlse = dl if with_dlse else None
    scale = 1.0 / math.sqrt(d)
    o, lse = fa.fa_fwd(q, k, v, causal=causal, scale=scale)
    grads = fa.fa_bwd(q, k, v, o, lse, do, causal=causal, scale=scale, dlse=dlse)
    assert fa.fa_get_device_status() == (0, 0)
    check(grads, q, k, v, o, lse, do, dlse, causal, scale, f"bwd {B, S, Hq, Hkv, d, causal}")
