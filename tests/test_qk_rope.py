"""Per-head RMS norm and rotary positions, forward and backward, on the GPU against the definition in
fp64, and the backward pass against differences of the definition.

Tolerance. A result is rounded to bf16 once: at most u = 2^-8 of its value. Before that, in fp32
(u32 = 2^-24): the sum of d <= 128 squares and its root err by less than 2^-18 relative, each product by
u32; cos and sin of an angle reduced to a fraction of a turn in 32 bits err by at most 2^-22 absolute.
So a rotated element is off by at most u |y| + 2^-16 (|z_a| + |z_b|), and a gradient dx by at most
u |dx| + 2^-14 of its terms' magnitudes r (|g w| + |xhat| mean|g w xhat|) of its pair or head. A weight's
gradient sums n = T heads terms in fp32: a lane's chain, then a tree; each term is off by 2^-15 of its
magnitude and the chain (at most n terms) by n u32 of the sum of magnitudes; with n below 2^11 here,
2^-12 of the sum of magnitudes bounds both.
"""
import pytest
import torch

U = 2.0 ** -8


def make(T, Hq, Hkv, d, rot, axes, norm, fused=False, seed=0, far=False):
    g = torch.Generator(device="cuda").manual_seed(seed + 7 * T + Hq + d + rot)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    if fused:  # views of one projection, with the values between them
        qkv = r(T, (Hq + 2 * Hkv) * d).mul_(1.5).bfloat16()
        q = qkv[:, :Hq * d].unflatten(1, (Hq, d))
        k = qkv[:, Hq * d:(Hq + Hkv) * d].unflatten(1, (Hkv, d))
    else:
        q, k = r(T, Hq, d).mul_(1.5).bfloat16(), r(T, Hkv, d).mul_(1.5).bfloat16()
    a = dict(positions=None, inv_freq=None, q_weight=None, k_weight=None, eps=1e-5, sections=None)
    if rot:
        lim = 2 ** 31 - 1 if far else 4096
        pos = torch.randint(-lim if far else 0, lim, (axes, T), generator=g, device="cuda", dtype=torch.int64)
        a["positions"] = (pos.int() if axes > 1 else pos[0].int()).contiguous()
        a["inv_freq"] = (10000.0 ** -(torch.arange(rot // 2, device="cuda").double() * 2 / rot)).float()
        if axes > 1:
            base = rot // 2 // axes
            a["sections"] = [rot // 2 - base * (axes - 1)] + [base] * (axes - 1)
    if norm:
        a["q_weight"], a["k_weight"] = ((1 + 0.3 * r(d)).bfloat16() for _ in range(2))
    return q, k, a, r(T, Hq, d).bfloat16(), r(T, Hkv, d).bfloat16()


def pairs_of(rot, interleaved, device):
    i = torch.arange(rot // 2, device=device)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def cos_sin(a, T, device):
    if a["positions"] is None:
        z = torch.zeros(T, 1, 0, dtype=torch.float64, device=device)
        return z, z
    pos = a["positions"].double().reshape(-1, T)
    sections = a["sections"] or [a["inv_freq"].numel()]
    axis = torch.tensor([x for x, n in enumerate(sections) for _ in range(n)], device=device)
    phi = (pos[axis].t() * a["inv_freq"].double()).unsqueeze(1)
    return phi.cos(), phi.sin()


def define(x, w, eps, c, s, ia, ib):
    """The definition in fp64, differentiable: y, and z before the rotation."""
    z = x
    if w is not None:
        z = x * w / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    y = z.clone()
    y[..., ia] = z[..., ia] * c - z[..., ib] * s
    y[..., ib] = z[..., ib] * c + z[..., ia] * s
    return y, z


CASES = [
    # (T, Hq, Hkv, d, rot, axes, norm, interleaved, fused)
    (1, 32, 8, 128, 128, 1, True, False, False),    # one token
    (1, 1, 1, 64, 64, 1, True, True, True),
    (3, 5, 3, 128, 128, 1, True, False, True),      # heads that do not fill a warp step
    (7, 9, 1, 64, 32, 1, True, False, False),       # partly rotated
    (7, 9, 2, 64, 16, 1, False, True, True),        # the smallest rotation, no norm
    (33, 4, 4, 128, 96, 3, True, True, False),      # rotated part not a power of two, three axes
    (33, 8, 2, 128, 64, 4, True, False, True),      # four axes
    (50, 6, 2, 64, 64, 2, False, False, False),
    (5, 3, 2, 128, 0, 1, True, False, True),        # norm only
    (257, 32, 8, 128, 128, 1, True, False, True),
    (1000, 8, 2, 64, 64, 3, True, True, True),
    (1500, 1, 1, 128, 128, 1, True, False, False),  # more tokens than warps of a small grid
]


@pytest.mark.gpu
@pytest.mark.parametrize("T,Hq,Hkv,d,rot,axes,norm,interleaved,fused", CASES)
def test_forward_and_backward_match_fp64(T, Hq, Hkv, d, rot, axes, norm, interleaved, fused):
    import io_aware_exact_flash_gb300 as fa

    q, k, a, dyq, dyk = make(T, Hq, Hkv, d, rot, axes, norm, fused)
    q0, k0 = q.clone(), k.clone()
    out = fa.fa_qk_norm_rope(q, k, interleaved=interleaved, **a)
    dq, dk, dwq, dwk = fa.fa_qk_norm_rope_bwd(dyq, dyk, q, k, interleaved=interleaved, **a)
    assert torch.equal(q, q0) and torch.equal(k, k0)
    assert (dwq is None) == (not norm) and (dwk is None) == (not norm)
    c, s = cos_sin(a, T, q.device)
    ia, ib = pairs_of(rot, interleaved, q.device)
    for y, x, wname, dy, dx, dw in ((out[0], q, "q_weight", dyq, dq, dwq), (out[1], k, "k_weight", dyk, dk, dwk)):
        xd = x.double().requires_grad_(True)
        w = None if a[wname] is None else a[wname].double().requires_grad_(True)
        want, z = define(xd, w, a["eps"], c, s, ia, ib)
        want.backward(dy.double())
        pair = z.detach().abs()
        pair[..., ia], pair[..., ib] = pair[..., ia] + pair[..., ib], pair[..., ia] + pair[..., ib]
        err = (y.double() - want.detach()).abs()
        assert (err <= U * want.detach().abs() + 2.0 ** -16 * pair).all(), f"forward {wname}: {float(err.max())}"
        # magnitudes of the backward's terms
        back = dy.double().abs()
        both = back.clone()
        both[..., ia] = both[..., ib] = back[..., ia] + back[..., ib]
        if w is None:
            mag = both
        else:
            r = 1 / torch.sqrt((xd.detach() ** 2).mean(-1, keepdim=True) + a["eps"])
            xhat = (xd.detach() * r).abs()
            gw = both * w.detach().abs()
            mag = r * (gw + xhat * (gw * xhat).mean(-1, keepdim=True))
            sums = (both * xhat).sum((0, 1))
            assert ((dw.double() - w.grad).abs() <= 2.0 ** -12 * sums + 1e-30).all(), f"gradient of {wname}"
            assert float((dw.double() - w.grad).norm()) <= 2.0 ** -15 * float(sums.norm())
        err = (dx.double() - xd.grad).abs()
        assert (err <= U * xd.grad.abs() + 2.0 ** -14 * mag).all(), f"backward {wname}: {float(err.max())}"


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_positions_over_the_whole_int32_range(interleaved):
    """An fp32 angle would be off by whole turns here; the reference reduces the angle with integers:
    inv_freq = m 2^-e exactly, so position * inv_freq is exact in Python integers."""
    import math
    from fractions import Fraction

    import io_aware_exact_flash_gb300 as fa

    T, d = 6, 64
    q = torch.ones(T, 1, d, device="cuda", dtype=torch.bfloat16)
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 1234567891], device="cuda", dtype=torch.int32)
    inv = torch.logspace(0, -6, d // 2, dtype=torch.float64).float().cuda()
    y, _ = fa.fa_qk_norm_rope(q, q, positions=pos, inv_freq=inv, interleaved=interleaved)
    # pi to 150 bits (Machin's formula in rationals)
    atan = lambda n: sum(Fraction((-1) ** i, (2 * i + 1) * n ** (2 * i + 1)) for i in range(40))  # noqa: E731
    two_pi = 2 * (16 * atan(5) - 4 * atan(239))
    for t in range(T):
        for i in range(d // 2):
            turn = Fraction(int(pos[t])) * Fraction(float(inv[i])) / two_pi
            phi = 2 * math.pi * float(turn - (turn.numerator // turn.denominator))
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + d // 2)
            # fp64 rounding of inv_freq / 2 pi moves the turn by at most 2^31 2^-53 2, i.e. 3e-6 of an angle
            for got, want in ((y[t, 0, a], math.cos(phi) - math.sin(phi)), (y[t, 0, b], math.cos(phi) + math.sin(phi))):
                assert abs(float(got) - want) <= U * abs(want) + 1e-5


@pytest.mark.gpu
def test_in_place_and_strided_outputs():
    import io_aware_exact_flash_gb300 as fa

    T, Hq, Hkv, d = 37, 6, 2, 128
    q, k, a, dyq, dyk = make(T, Hq, Hkv, d, d, 1, True, fused=True)
    want = fa.fa_qk_norm_rope(q, k, **a)
    wgrad = fa.fa_qk_norm_rope_bwd(dyq, dyk, q, k, **a)
    qkv = q._base.clone()
    values = qkv[:, (Hq + Hkv) * d:].clone()
    q2 = qkv[:, :Hq * d].unflatten(1, (Hq, d))
    k2 = qkv[:, Hq * d:(Hq + Hkv) * d].unflatten(1, (Hkv, d))
    got = fa.fa_qk_norm_rope(q2, k2, q_out=q2, k_out=k2, **a)  # in place, inside the projection
    assert got[0] is q2 and torch.equal(q2, want[0]) and torch.equal(k2, want[1])
    assert torch.equal(qkv[:, (Hq + Hkv) * d:], values)
    # gradients written into the projection's gradient; then in place over the incoming ones
    dqkv = torch.full_like(qkv, float("nan"))
    dq2 = dqkv[:, :Hq * d].unflatten(1, (Hq, d))
    dk2 = dqkv[:, Hq * d:(Hq + Hkv) * d].unflatten(1, (Hkv, d))
    fa.fa_qk_norm_rope_bwd(dyq, dyk, q, k, dq=dq2, dk=dk2, **a)
    assert torch.equal(dq2, wgrad[0]) and torch.equal(dk2, wgrad[1])
    assert torch.isnan(dqkv[:, (Hq + Hkv) * d:]).all()
    g1, g2 = dyq.clone(), dyk.clone()
    res = fa.fa_qk_norm_rope_bwd(g1, g2, q, k, dq=g1, dk=g2, **a)
    assert all(torch.equal(x, y) for x, y in zip(res, wgrad))


@pytest.mark.gpu
def test_no_tokens():
    import io_aware_exact_flash_gb300 as fa

    q, k, a, dyq, dyk = make(0, 4, 2, 64, 64, 1, True)
    out = fa.fa_qk_norm_rope(q, k, **a)
    assert out[0].shape == (0, 4, 64) and out[1].shape == (0, 2, 64)
    nan = torch.full((64,), float("nan"), device="cuda")
    dq, dk, dwq, dwk = fa.fa_qk_norm_rope_bwd(dyq, dyk, q, k, dq_weight=nan, dk_weight=nan.clone(), **a)
    assert dq.shape == q.shape and not dwq.any() and not dwk.any()


@pytest.mark.gpu
def test_zero_and_non_finite_heads_stay_apart():
    """A head of zeros normalises to zeros (eps > 0), and a non-finite element reaches no other head."""
    import io_aware_exact_flash_gb300 as fa

    q, k, a, _, _ = make(9, 8, 2, 128, 128, 1, True)
    clean = fa.fa_qk_norm_rope(q, k, **a)[0]
    q = q.clone()
    q[4, 3] = 0
    q[5, 2, 7] = float("inf")
    q[6, 1, 100] = float("nan")
    y = fa.fa_qk_norm_rope(q, k, **a)[0]
    assert not y[4, 3].any()
    touched = torch.zeros(9, 8, dtype=torch.bool, device="cuda")
    touched[4, 3] = touched[5, 2] = touched[6, 1] = True
    assert torch.equal(y[~touched], clean[~touched])
    assert torch.isnan(y[6, 1]).all()


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """More than 2^31 elements of queries: the last tokens give the bits of a call on them alone."""
    import io_aware_exact_flash_gb300 as fa

    T, Hq, d = 525000, 32, 128
    assert T * Hq * d > 1 << 31
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    q = torch.zeros(T, Hq, d, device="cuda", dtype=torch.bfloat16)
    k = torch.zeros(T, 1, d, device="cuda", dtype=torch.bfloat16)
    qs, ks, a, dyq, dyk = make(700, Hq, 1, d, d, 1, True)
    q[-700:], k[-700:] = qs, ks
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")
    pos[-700:] = a["positions"]
    want = fa.fa_qk_norm_rope(qs, ks, **a)
    got = fa.fa_qk_norm_rope(q, k, **{**a, "positions": pos})
    assert torch.equal(got[0][-700:], want[0]) and torch.equal(got[1][-700:], want[1])
    assert not got[0][:-700].any()
    del got
    dq = torch.zeros_like(q)
    dq[-700:] = dyq
    dk = torch.zeros_like(k)
    dk[-700:] = dyk
    wantb = fa.fa_qk_norm_rope_bwd(dyq, dyk, qs, ks, **a)
    res = fa.fa_qk_norm_rope_bwd(dq, dk, q, k, dq=dq, dk=dk, **{**a, "positions": pos})
    assert torch.equal(res[0][-700:], wantb[0]) and torch.equal(res[1][-700:], wantb[1])
    assert not res[0][:-700].any()


@pytest.mark.gpu
def test_python_refusals():
    import io_aware_exact_flash_gb300 as fa

    q, k, a, dq_out, dk_out = make(9, 4, 2, 64, 64, 2, True)
    forward = dict(q=q, k=k, **a)
    backward = dict(dq_out=dq_out, dk_out=dk_out, **forward)
    types = (dict(q=q.half()), dict(k=k.cpu()), dict(q=[1]))
    values = (dict(k=k[:5]), dict(k=k[0]), dict(q=q.transpose(0, 1).contiguous().transpose(0, 1)), dict(q_weight=None),
              dict(k_weight=[1.0] * 64), dict(q_weight=a["q_weight"].float()), dict(q_weight=a["q_weight"][:32]),
              dict(positions=None), dict(inv_freq=None), dict(positions=a["positions"].long()),
              dict(positions=a["positions"][:, :5]), dict(positions=[1, 2]), dict(inv_freq=a["inv_freq"].double()),
              dict(inv_freq=0.5), dict(inv_freq=a["inv_freq"].cpu()), dict(sections=None), dict(sections=[32]),
              dict(sections=[16, 17]), dict(sections=[33, -1]),
              dict(q_weight=None, k_weight=None, positions=None, inv_freq=None, sections=None))
    for call, good in ((fa.fa_qk_norm_rope, forward), (fa.fa_qk_norm_rope_bwd, backward)):
        for kw in types:
            with pytest.raises(TypeError):
                call(**{**good, **kw})
        for kw in values:
            with pytest.raises(ValueError):
                call(**{**good, **kw})
        for kw in (dict(eps=0.0), dict(eps=float("nan"))):
            with pytest.raises(fa.FaError) as e:
                call(**{**good, **kw})
            assert e.value.code == 1
    for kw in (dict(q_out=k), dict(q_out=q[:, :2]), dict(k_out=q)):
        with pytest.raises(ValueError):
            fa.fa_qk_norm_rope(**{**forward, **kw})
    for kw in (dict(dq=dk_out), dict(dq_weight=torch.empty(64, device="cuda").double()), dict(dk_out=dk_out[:5]),
               dict(workspace=torch.empty(4096, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            fa.fa_qk_norm_rope_bwd(**{**backward, **kw})
    with pytest.raises(fa.FaError) as e:
        fa.fa_qk_norm_rope_bwd(**backward, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.code == 4  # FA_ERR_WORKSPACE


@pytest.mark.gpu
def test_two_streams_and_a_graph_agree_with_one_call():
    import io_aware_exact_flash_gb300 as fa

    cases = [make(T, 8, 2, 64, 32, 1, True, seed=T) for T in (301, 77)]
    run = lambda c, **kw: (fa.fa_qk_norm_rope(c[0], c[1], **c[2], **kw)  # noqa: E731
                           + fa.fa_qk_norm_rope_bwd(c[3], c[4], c[0], c[1], **c[2], **kw))
    want = [run(c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[run(c, stream=s) for c, s in zip(cases, streams)] for _ in range(5)]
    graphs, results = [], []
    for c in cases:  # each graph has its own memory
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            results.append(run(c))
    for _ in range(2):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for turn in got + [results]:
        for have, expected in zip(turn, want):
            assert all(torch.equal(x, y) for x, y in zip(have, expected))
