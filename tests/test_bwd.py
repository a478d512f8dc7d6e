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


def reference(q, k, v, o, lse, do, dlse, causal, scale, u=U, small=SMALL):
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
    w = (u + small) * ds.abs() + 2.0 ** -14 * mag
    tq = torch.einsum("bhij,bjhd->bihd", w, ka) * scale
    tk = to_kv(torch.einsum("bhij,bihd->bjhd", w, qa)) * scale
    tv = (u + small) * to_kv(torch.einsum("bhij,bihd->bjhd", p, do.abs()))
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


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("B,S,Hq,Hkv", [(3, 1, 4, 2), (5, 2, 6, 2), (1, 3, 8, 1), (150, 4, 4, 2), (2, 9, 4, 4),
                                        (20, 16, 12, 6)])
def test_bwd_of_few_tokens_rounds_once(B, S, Hq, Hkv, d, causal):
    """Up to 16 tokens P and dS are two bf16 operands each, off by at most u^2 = 2^-16 together. In the
    bounds above that takes the place of u, and with at most 16 terms per head and 8 heads the fp32 sums add
    less than 2^-17 of the magnitudes, so that 2^-13 covers them with the 2^-14 of P. (150 and 20 entries: more
    units than SMs.)"""
    import io_aware_exact_flash_gb300 as fa

    q, k, v, do, dlse = inputs(B, S, Hq, Hkv, d, seed=3)
    scale = 1.0 / math.sqrt(d)
    o, lse = fa.fa_fwd(q, k, v, causal=causal, scale=scale)
    grads = fa.fa_bwd(q, k, v, o, lse, do, causal=causal, scale=scale, dlse=dlse)
    assert fa.fa_get_device_status() == (0, 0)
    want, tol = reference(q, k, v, o, lse, do, dlse, causal, scale, u=2.0 ** -16, small=2.0 ** -13)
    for name, got, ref, t in zip(("dq", "dk", "dv"), grads, want, tol):
        worst = float(((got.double() - ref).abs() / (t + 1e-30)).max())
        assert worst <= 1, f"{name} off by {worst:.2f} of its bound"


@pytest.mark.gpu
@pytest.mark.parametrize("B,S,Hq,Hkv,d,causal", [
    (1, 384, 64, 64, 64, True),     # a CTA's second unit has one to three steps
    (1, 384, 64, 64, 128, True),
    (1, 100, 400, 400, 64, False),  # one step each, several units per CTA
    (1, 100, 400, 200, 128, True),
    (2, 130, 120, 120, 128, False), # two steps
    (2, 300, 96, 32, 64, False),
])
def test_bwd_short_units_one_after_the_other(B, S, Hq, Hkv, d, causal):
    """CTAs that run many short units of both kinds: the loads of the next units start while the last ones
    are still computed. Every one of several runs has the same bits."""
    import io_aware_exact_flash_gb300 as fa

    q, k, v, do, _ = inputs(B, S, Hq, Hkv, d)
    scale = 1.0 / math.sqrt(d)
    o, lse = fa.fa_fwd(q, k, v, causal=causal, scale=scale)
    runs = [fa.fa_bwd(q, k, v, o, lse, do, causal=causal, scale=scale) for _ in range(10)]
    check(runs[0], q, k, v, o, lse, do, None, causal, scale, f"short units {B, S, Hq, Hkv, d, causal}")
    for g in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(g, runs[0]))
    assert fa.fa_get_device_status() == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("d,causal", [(64, False), (128, True)])
def test_bwd_long_rows(d, causal):
    """Many tiles per unit (the rings and barrier phases wrap many times), an odd length."""
    import io_aware_exact_flash_gb300 as fa

    q, k, v, do, _ = inputs(1, 2501, 2, 1, d)
    scale = 1.0 / math.sqrt(d)
    o, lse = fa.fa_fwd(q, k, v, causal=causal, scale=scale)
    grads = fa.fa_bwd(q, k, v, o, lse, do, causal=causal, scale=scale)
    check(grads, q, k, v, o, lse, do, None, causal, scale, "long rows")


@pytest.mark.gpu
def test_bwd_matches_differences():
    """<gradient, direction> against central differences of the forward pass in fp64. Each gradient is
    within 2 u of the formula's (asserted above); o is given to the backward rounded to bf16, which moves
    delta, and so each gradient, by at most another u of its terms: 4 u of the norms bounds both."""
    import io_aware_exact_flash_gb300 as fa

    B, S, Hq, Hkv, d = 1, 200, 4, 2, 64
    q, k, v, do, dlse = inputs(B, S, Hq, Hkv, d, seed=5)
    scale = 1.0 / math.sqrt(d)
    o, lse = fa.fa_fwd(q, k, v, causal=True, scale=scale)
    grads = fa.fa_bwd(q, k, v, o, lse, do, causal=True, scale=scale, dlse=dlse)

    def loss(q, k, v):
        s = torch.einsum("bihd,bjhd->bhij", q, k.repeat_interleave(Hq // Hkv, 2)) * scale
        s = s.masked_fill(torch.ones(S, S, dtype=torch.bool, device=q.device).triu(1), float("-inf"))
        out = torch.einsum("bhij,bjhd->bihd", s.softmax(-1), v.repeat_interleave(Hq // Hkv, 2))
        return (out * do.double()).sum() + (s.logsumexp(-1).permute(0, 2, 1) * dlse.double()).sum()

    x = [t.double() for t in (q, k, v)]
    g = torch.Generator(device="cuda").manual_seed(9)
    for i in range(3):
        grad = grads[i].double()
        way = grad / grad.norm() + torch.randn(grad.shape, generator=g, device="cuda").double() / grad.numel() ** 0.5
        eps = 1e-4
        up, down = list(x), list(x)
        up[i], down[i] = x[i] + eps * way, x[i] - eps * way
        fd = float((loss(*up) - loss(*down)) / (2 * eps))
        assert abs(float((grad * way).sum()) - fd) <= 4 * U * float(grad.norm() * way.norm())


@pytest.mark.gpu
def test_bwd_large_scores():
    """Sharp softmax rows (scores of tens): most P are 0, LSE and scores cancel. The exponent's fp32 error
    is at most 2^-24 (|s| + |LSE|) log2(e) 4 < 2^-13 for magnitudes below 300: inside the bound's 2^-10."""
    import io_aware_exact_flash_gb300 as fa

    q, k, v, do, _ = inputs(1, 300, 2, 2, 64, gain=4.0)
    o, lse = fa.fa_fwd(q, k, v, causal=True)
    assert float(lse.abs().max()) < 300
    grads = fa.fa_bwd(q, k, v, o, lse, do, causal=True)
    check(grads, q, k, v, o, lse, do, None, True, 1 / 8.0, "large scores")


@pytest.mark.gpu
def test_bwd_rows_without_keys_and_far_lse():
    """LSE = -inf marks a row without keys: no gradient from it or to it. Checked against the formulas."""
    import io_aware_exact_flash_gb300 as fa

    q, k, v, do, dlse = inputs(2, 150, 2, 1, 128)
    o, lse = fa.fa_fwd(q, k, v, causal=False)
    lse[0, 7, 0] = lse[1, 149, 1] = lse[0, 64, 1] = float("-inf")
    grads = fa.fa_bwd(q, k, v, o, lse, do, causal=False, dlse=dlse)
    assert not grads[0][0, 7, 0].any() and not grads[0][1, 149, 1].any()
    dl = dlse.masked_fill(torch.isneginf(lse), 0.0)
    check(grads, q, k, v, o, lse, do, dl, False, 1 / math.sqrt(128), "rows without keys")


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_bwd_non_finite_stays_in_its_head(d):
    """A NaN reaches gradients of its own batch entry and kv head only; a masked dO of infinity does not
    reach the keys of other tiles."""
    import io_aware_exact_flash_gb300 as fa

    q, k, v, do, _ = inputs(2, 260, 4, 2, d)
    o, lse = fa.fa_fwd(q, k, v, causal=True)
    clean = fa.fa_bwd(q, k, v, o, lse, do, causal=True)
    bad = do.clone()
    bad[1, 3, 2, 5] = float("nan")   # kv head 1 of batch entry 1
    grads = fa.fa_bwd(q, k, v, o, lse, bad, causal=True)
    for got, ref, heads in zip(grads, clean, (slice(2, 4), slice(1, 2), slice(1, 2))):
        keep = torch.ones(got.shape[:3], dtype=torch.bool, device="cuda")
        keep[1, :, heads] = False
        assert torch.equal(got[keep], ref[keep])
    assert torch.isnan(grads[0][1, 3, 2]).any()
    # row 3 is in the first tile: keys of later tiles never see it
    assert torch.equal(grads[1][1, 128:], clean[1][1, 128:]) and torch.equal(grads[2][1, 128:], clean[2][1, 128:])


@pytest.mark.gpu
def test_bwd_is_deterministic_and_leaves_the_rest_alone():
    import io_aware_exact_flash_gb300 as fa

    q, k, v, do, _ = inputs(2, 333, 6, 3, 128)
    keep = [t.clone() for t in (q, k, v, do)]
    o, lse = fa.fa_fwd(q, k, v, causal=True)
    first = fa.fa_bwd(q, k, v, o, lse, do, causal=True)
    # outputs inside larger buffers, 16-byte but not 32-byte aligned, with sentinels around them
    outs, bufs = [], []
    for t in (q, k, v):
        buf = torch.full((t.numel() + 64,), 7.0, device="cuda", dtype=torch.bfloat16)
        outs.append(buf[8:8 + t.numel()].view(t.shape))
        bufs.append(buf)
    need = fa.fa_bwd_workspace_bytes(2, 6, 3, 333, 128, True)
    ws = torch.full((need + 512,), 255, device="cuda", dtype=torch.uint8)  # garbage (NaN) inside
    off = -ws.data_ptr() % 256
    again = fa.fa_bwd(q, k, v, o, lse, do, causal=True, dq=outs[0], dk=outs[1], dv=outs[2],
                      workspace=ws[off:off + need])
    for a, b, out, buf in zip(first, again, outs, bufs):
        assert b is out and torch.equal(a, b)
        assert (buf[:8] == 7).all() and (buf[8 + out.numel():] == 7).all()
    assert (ws[off + need:] == 255).all()
    assert all(torch.equal(a, b) for a, b in zip(keep, (q, k, v, do)))


@pytest.mark.gpu
def test_bwd_in_graphs_that_share_a_workspace():
    """Two captured backward passes of different shapes, one workspace, replayed in turn with new inputs."""
    import io_aware_exact_flash_gb300 as fa

    shapes = [(1, 200, 4, 2, 64, True), (2, 130, 2, 2, 128, False)]
    need = max(fa.fa_bwd_workspace_bytes(B, Hq, Hkv, S, d, c) for B, S, Hq, Hkv, d, c in shapes)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    graphs, states = [], []
    for B, S, Hq, Hkv, d, c in shapes:
        q, k, v, do, _ = inputs(B, S, Hq, Hkv, d)
        o, lse = fa.fa_fwd(q, k, v, causal=c)
        out = tuple(torch.zeros_like(t) for t in (q, k, v))
        st = (q, k, v, o, lse, do)
        run = lambda st=st, c=c, out=out: fa.fa_bwd(*st, causal=c, dq=out[0], dk=out[1], dv=out[2], workspace=ws)  # noqa: E731
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            run()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        graphs.append(graph)
        states.append((st, out, c))
    for turn in range(2):
        for graph, (st, out, c) in zip(graphs, states):
            st[5].copy_(torch.randn_like(st[5].float()).bfloat16())  # another dO
            for t in out:
                t.zero_()
            graph.replay()
        for st, out, c in states:
            want = fa.fa_bwd(*st, causal=c)
            assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.gpu
def test_bwd_on_two_streams_at_once():
    import io_aware_exact_flash_gb300 as fa

    cases = [inputs(1, 700, 8, 4, 128, seed=s)[:4] for s in (1, 2)]
    fwd = [fa.fa_fwd(q, k, v, causal=True) for q, k, v, _ in cases]
    want = [fa.fa_bwd(q, k, v, o, l, do, causal=True) for (q, k, v, do), (o, l) in zip(cases, fwd)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            (q, k, v, do), (o, l) = cases[i], fwd[i]
            got[i].append(fa.fa_bwd(q, k, v, o, l, do, causal=True, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))


@pytest.mark.gpu
def test_bwd_python_refusals():
    import io_aware_exact_flash_gb300 as fa

    q, k, v, do, dlse = inputs(1, 64, 2, 2, 64)
    o, lse = fa.fa_fwd(q, k, v)
    good = dict(q=q, k=k, v=v, out=o, lse=lse, dout=do)
    for kw in (dict(q=q.half()), dict(dout=do.cpu())):
        with pytest.raises(TypeError):
            fa.fa_bwd(**{**good, **kw})
    wide = torch.cat([do, do], 3)
    for kw in (dict(dout=wide[..., :64]), dict(out=o[:, :32].contiguous()), dict(lse=lse.double()),
               dict(lse=lse[..., :1].contiguous()), dict(k=k[:, :, :1].contiguous()), dict(dlse=dlse[:, :3]),
               dict(dq=torch.empty_like(q)[:, :32]), dict(dk=torch.empty_like(k).float()),
               dict(workspace=torch.empty(4096, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            fa.fa_bwd(**{**good, **kw})
    with pytest.raises(fa.FaError) as e:
        fa.fa_bwd(**good, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.code == 4  # FA_ERR_WORKSPACE
    for kw in (dict(dq=q), dict(dk=v), dict(dv=torch.empty_like(v), dk=None, dq=do)):  # outputs over inputs
        with pytest.raises(fa.FaError) as e:
            fa.fa_bwd(**{**good, **kw})
        assert e.value.code == 1


@pytest.mark.gpu
def test_bwd_long_sequence_sampled():
    """20011 tokens: gradients of sampled queries and keys against the formulas in fp64, row by row and
    column by column, within the bounds above (the sums are longer: n 2^-24 with n = 20011 is 2^-9.7 of the
    magnitudes, so SMALL counts twice here)."""
    import io_aware_exact_flash_gb300 as fa

    S, Hq, d = 20011, 2, 128
    q, k, v, do, _ = inputs(1, S, Hq, 1, d)
    scale = 1.0 / math.sqrt(d)
    o, lse = fa.fa_fwd(q, k, v, causal=True, scale=scale)
    dq, dk, dv = fa.fa_bwd(q, k, v, o, lse, do, causal=True, scale=scale)
    Q, O, DO = (t[0].double() for t in (q, o, do))
    K, V, L = k[0, :, 0].double(), v[0, :, 0].double(), lse[0].double()
    delta, dabs = (DO * O).sum(-1), (DO * O).abs().sum(-1)
    idx = torch.arange(S, device="cuda")
    for i in (0, 1, 127, 128, 5000, 12800, S - 1):
        for h in range(Hq):
            p = torch.exp(K[:i + 1] @ Q[i, h] * scale - L[i, h])
            ds = p * (V[:i + 1] @ DO[i, h] - delta[i, h])
            mag = p * (V[:i + 1].abs() @ DO[i, h].abs() + dabs[i, h])
            want = ds @ K[:i + 1] * scale
            w = U * ds.abs() + 2 * SMALL * (ds.abs() + mag / 16)
            tol = w @ K[:i + 1].abs() * scale + U * want.abs()
            assert ((dq[0, i, h].double() - want).abs() <= tol + 1e-30).all(), f"dq row {i}"
    for j in (0, 1, 126, 129, 5001, 12799, S - 2, S - 1):
        want_k = torch.zeros(d, dtype=torch.float64, device="cuda")
        want_v, tol_k, tol_v = want_k.clone(), want_k.clone(), want_k.clone()
        for h in range(Hq):
            p = torch.where(idx >= j, torch.exp(Q[:, h] @ K[j] * scale - L[:, h]), 0.0)
            ds = p * (DO[:, h] @ V[j] - delta[:, h])
            mag = p * (DO[:, h].abs() @ V[j].abs() + dabs[:, h])
            want_v += p @ DO[:, h]
            want_k += ds @ Q[:, h] * scale
            tol_v += (U + 2 * SMALL) * (p @ DO[:, h].abs())
            tol_k += (U * ds.abs() + 2 * SMALL * (ds.abs() + mag / 16)) @ Q[:, h].abs() * scale
        assert ((dk[0, j, 0].double() - want_k).abs() <= tol_k + U * want_k.abs() + 1e-30).all(), f"dk row {j}"
        assert ((dv[0, j, 0].double() - want_v).abs() <= tol_v + U * want_v.abs() + 1e-30).all(), f"dv row {j}"


@pytest.mark.gpu
def test_bwd_offsets_past_32_bits():
    """A batch whose tensors have more than 2^31 elements (4.3 GB each): the first and the last entries."""
    import io_aware_exact_flash_gb300 as fa

    B, S, H, d = 8200, 128, 16, 128
    assert B * S * H * d > 1 << 31
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    big = [torch.zeros(B, S, H, d, device="cuda", dtype=torch.bfloat16) for _ in range(5)]
    lse = torch.zeros(B, S, H, device="cuda")
    scale = 1.0 / math.sqrt(d)
    ends = {}
    for b in (0, B - 1):
        q, k, v, do, _ = inputs(1, S, H, H, d, seed=b)
        o, l = fa.fa_fwd(q, k, v, causal=True, scale=scale)
        ends[b] = (q, k, v, o, l, do)
        for t, x in zip(big, (q, k, v, o, do)):
            t[b] = x[0]
        lse[b] = l[0]
    grads = fa.fa_bwd(big[0], big[1], big[2], big[3], lse, big[4], causal=True, scale=scale)
    for b, (q, k, v, o, l, do) in ends.items():
        check([g[b:b + 1] for g in grads], q, k, v, o, l, do, None, True, scale, f"entry {b}")
    assert not any(g[1:B - 1].any() for g in grads)
