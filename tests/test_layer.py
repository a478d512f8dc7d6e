"""The operators of an attention layer run together, as a model uses them: query/key norm with rotary
positions, attention, and both backward passes (training); the same norm before the paged append and
decode (serving)."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -8


def layer_inputs(B, S, Hq, Hkv, d, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    qkv = r(B * S, (Hq + 2 * Hkv) * d).bfloat16()
    wq, wk = ((1 + 0.2 * r(d)).bfloat16() for _ in range(2))
    pos = torch.arange(S, device="cuda", dtype=torch.int32).repeat(B)
    inv = (10000.0 ** -(torch.arange(d // 2, device="cuda").double() * 2 / d)).float()
    return qkv, wq, wk, pos, inv, r(B, S, Hq, d).bfloat16()


def split(qkv, Hq, Hkv, d):
    parts = qkv.split([Hq * d, Hkv * d, Hkv * d], 1)
    return [p.unflatten(1, (-1, d)) for p in parts]


def train_step(fa, qkv, wq, wk, pos, inv, dout, B, S, Hq, Hkv, d):
    """One layer's forward and backward: (out, dqkv, dwq, dwk)."""
    q, k, v = split(qkv, Hq, Hkv, d)
    qr, kr = fa.fa_qk_norm_rope(q, k, pos, inv, wq, wk)
    q4, k4, v4 = qr.view(B, S, Hq, d), kr.view(B, S, Hkv, d), v.contiguous().view(B, S, Hkv, d)
    out, lse = fa.fa_fwd(q4, k4, v4, causal=True)
    dq, dk, dv = fa.fa_bwd(q4, k4, v4, out, lse, dout, causal=True)
    dqkv = torch.empty_like(qkv)
    gq, gk, gv = split(dqkv, Hq, Hkv, d)
    _, _, dwq, dwk = fa.fa_qk_norm_rope_bwd(dq.view(-1, Hq, d), dk.view(-1, Hkv, d), q, k, pos, inv, wq, wk, dq=gq,
                                            dk=gk)
    gv.copy_(dv.view(-1, Hkv, d))
    return out, dqkv, dwq, dwk


def exact_step(qkv, wq, wk, pos, inv, dout, B, S, Hq, Hkv, d):
    x = qkv.double().requires_grad_(True)
    a, b = (w.double().requires_grad_(True) for w in (wq, wk))
    phi = (pos.double()[:, None] * inv.double())[:, None]
    c, s = phi.cos(), phi.sin()

    def turn(t, w):
        t = t * w / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6)
        lo, hi = t.chunk(2, -1)
        return torch.cat([lo * c - hi * s, hi * c + lo * s], -1)

    q, k, v = split(x, Hq, Hkv, d)
    q, k, v = turn(q, a).view(B, S, Hq, d), turn(k, b).view(B, S, Hkv, d), v.view(B, S, Hkv, d)
    k, v = k.repeat_interleave(Hq // Hkv, 2), v.repeat_interleave(Hq // Hkv, 2)
    sc = torch.einsum("bihd,bjhd->bhij", q, k) / math.sqrt(d)
    sc = sc.masked_fill(torch.ones(S, S, dtype=torch.bool, device=x.device).triu(1), float("-inf"))
    out = torch.einsum("bhij,bjhd->bihd", sc.softmax(-1), v)
    out.backward(dout.double())
    return out.detach(), x.grad, a.grad, b.grad


# Against the exact layer every result carries at most six roundings to bf16 on its way (rotated q and k,
# P or dS, o in delta, the gradients between the two backward passes, the result), each at most u of what is
# rounded. A rounding of q and k moves a score by at most u sqrt(2) |q||k| scale, about 1.4 u sqrt(d) / sqrt(d)
# times their unit-rms norms, i.e. the others' order. 8 u of the norm (a third more than six) bounds the sum.
TOL = 8 * U


@pytest.mark.parametrize("B,S,Hq,Hkv,d", [(2, 190, 4, 2, 128), (1, 333, 6, 6, 64)])
def test_training_step_of_a_layer(B, S, Hq, Hkv, d):
    import io_aware_exact_flash_gb300 as fa

    args = layer_inputs(B, S, Hq, Hkv, d, 3)
    got = train_step(fa, *args, B, S, Hq, Hkv, d)
    want = exact_step(*args, B, S, Hq, Hkv, d)
    for name, a, b in zip(("out", "dqkv", "dq_weight", "dk_weight"), got, want):
        rel = float((a.double() - b).norm() / b.norm())
        assert rel <= TOL, f"{name}: relative error {rel}"
    assert fa.fa_get_device_status() == (0, 0)


def test_training_step_captured_in_a_graph():
    """The whole step replayed with other inputs gives the bits of the eager calls; an eager step of the
    same tensors is alive when the graph is captured."""
    import io_aware_exact_flash_gb300 as fa

    B, S, Hq, Hkv, d = 2, 150, 4, 1, 64
    args = list(layer_inputs(B, S, Hq, Hkv, d, 4))
    alive = train_step(fa, *args, B, S, Hq, Hkv, d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        train_step(fa, *args, B, S, Hq, Hkv, d)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = train_step(fa, *args, B, S, Hq, Hkv, d)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(res, alive))
    other = layer_inputs(B, S, Hq, Hkv, d, 5)
    for t, o in zip(args, other):
        t.copy_(o)
    graph.replay()
    want = train_step(fa, *other, B, S, Hq, Hkv, d)
    assert all(torch.equal(a, b) for a, b in zip(res, want))


def test_decode_step_with_norm_append_and_attention():
    """New tokens of several sequences: norm and rotation at their own positions, append, paged attention,
    against the forward pass over the whole sequences at once (the same bf16 rows, so the same bound as the
    paged kernels have against the oracle: 2 u of the values' norm)."""
    import io_aware_exact_flash_gb300 as fa

    Hq, Hkv, d, page = 8, 2, 128, 16
    lens = [40, 1, 17]  # tokens before the new one
    g = torch.Generator(device="cuda").manual_seed(8)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    wq, wk = ((1 + 0.2 * r(d)).bfloat16() for _ in range(2))
    inv = (10000.0 ** -(torch.arange(d // 2, device="cuda").double() * 2 / d)).float()
    tables = torch.full((3, 4), -1, dtype=torch.int32)
    free = 0
    for i, n in enumerate(lens):
        for p in range((n + 1 + page - 1) // page):
            tables[i, p] = free
            free += 1
    tables = tables.cuda()
    kp = torch.full((free, page, Hkv, d), float("nan"), device="cuda", dtype=torch.bfloat16)
    vp = kp.clone()
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    rows = [r(n + 1, (Hq + 2 * Hkv) * d).bfloat16() for n in lens]

    def norm(x, pos):
        q, k, v = split(x, Hq, Hkv, d)
        return (*fa.fa_qk_norm_rope(q, k, pos, inv, wq, wk), v.contiguous())

    # prompts
    past = torch.cat([x[:-1] for x in rows])
    _, k, v = norm(past, torch.cat([torch.arange(n, device="cuda", dtype=torch.int32) for n in lens]))
    cu = i32([0, 40, 41, 58])
    fa.fa_paged_append(k, v, cu, i32([0, 0, 0]), tables, kp, vp)
    # one decode step
    q, k, v = norm(torch.cat([x[-1:] for x in rows]), i32(lens))
    fa.fa_paged_append(k, v, i32([0, 1, 2, 3]), i32(lens), tables, kp, vp)
    out, _ = fa.fa_paged_fwd(q, kp, vp, tables, i32([0, 1, 2, 3]), i32([n + 1 for n in lens]), 1)
    for i, x in enumerate(rows):
        n = x.shape[0]
        q1, k1, v1 = norm(x, torch.arange(n, device="cuda", dtype=torch.int32))
        want, _ = fa.fa_fwd(q1[None], k1[None], v1[None], causal=True)
        err = (out[i].double() - want[0, -1].double()).norm() / want[0, -1].double().norm()
        assert float(err) <= 2 * U
    assert fa.fa_get_device_status() == (0, 0)
