"""Operators of an attention layer in training and serving, as cases to measure.

Two operators: the backward pass of dense attention, and the per-head RMS norm of queries and keys
with the rotary position embedding in the same pass (one or several position axes; forward and
backward). Every case can be run in its plain form (elementary torch operations in 32 bits) or, with
``own`` set, through the package's entry points on the same inputs.
"""
import math

import torch

own = False  # False: the plain forms; True: the package's kernels

DEVICE = "cuda"


# ------------------------------------------------------------------------------------------ cases
def _bwd(B, S, Hq, Hkv, d, causal, dlse=False):
    return {"op": "attn_bwd", "B": B, "S": S, "Hq": Hq, "Hkv": Hkv, "d": d, "causal": causal, "dlse": dlse}


def _rope(op, T, Hq, Hkv, d, rot, axes, norm, interleaved, fused):
    return {"op": op, "T": T, "Hq": Hq, "Hkv": Hkv, "d": d, "rot": rot, "axes": axes, "norm": norm,
            "interleaved": interleaved, "fused": fused}


def listed():
    cases = [
        # one short odd-length sequence of a small model: the latency of a backward call
        ("bwd_s77_d64_causal", _bwd(1, 77, 4, 2, 64, True)),
        # bidirectional encoder fine-tuning: a batch of short full-attention sequences
        ("bwd_b8_s512_d64_full", _bwd(8, 512, 16, 16, 64, False)),
        # grouped-query training on an odd length, with a loss that also uses the log-sum-exp
        ("bwd_b2_s1000_gqa_dlse", _bwd(2, 1000, 32, 8, 128, True, True)),
        # grouped queries without a mask (a prefix or an image encoder)
        ("bwd_b1_s2048_gqa_full", _bwd(1, 2048, 32, 8, 128, False)),
        # the shape of the causal prefill benchmark, now trained
        ("bwd_b4_s4096_causal", _bwd(4, 4096, 32, 32, 128, True)),
        # long-context grouped-query training, one sequence
        ("bwd_b1_s8192_gqa_causal", _bwd(1, 8192, 32, 8, 128, True)),
        # serving: one token of one sequence (launch latency)
        ("rope_t1_decode", _rope("rope_fwd", 1, 32, 8, 128, 128, 1, True, False, True)),
        # serving: a decode batch, one token per sequence
        ("rope_t128_decode", _rope("rope_fwd", 128, 32, 8, 128, 128, 1, True, False, True)),
        # prefill or training: queries and keys as views of one fused projection
        ("rope_t16384_prefill", _rope("rope_fwd", 16384, 32, 8, 128, 128, 1, True, False, True)),
        # images and video: positions in time, height and width, no norm, adjacent pairs
        ("rope_t8192_three_axes", _rope("rope_fwd", 8192, 16, 16, 128, 128, 3, False, True, False)),
        # training a small model with a partly rotated head on an odd token count
        ("rope_bwd_t1001_d64_partial", _rope("rope_bwd", 1001, 8, 2, 64, 32, 1, True, True, False)),
        # training: the backward pass of the prefill shape, with three axes
        ("rope_bwd_t16384_three_axes", _rope("rope_bwd", 16384, 32, 8, 128, 128, 3, True, False, True)),
    ]
    return [dict(c, name=n) for n, c in cases]


def _log_int(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    if rng.random() < 0.5:
        limit = max(work(c)["flops"] for c in listed() if c["op"] == "attn_bwd")
        while True:
            Hkv = rng.choice([1, 2, 3, 4, 8, 16, 32])
            case = _bwd(_log_int(rng, 1, 16), _log_int(rng, 1, 8192), Hkv * rng.choice([1, 2, 3, 4, 8]), Hkv,
                        rng.choice([64, 128]), rng.random() < 0.6, rng.random() < 0.3)
            full = dict(case, causal=False)  # what the plain form computes
            if case["Hq"] <= 64 and work(full)["flops"] <= 2 * limit:
                return case
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8, 16])
    Hq = Hkv * rng.choice([1, 2, 4, 5, 8])
    T = _log_int(rng, 1, 16384)
    while T * (Hq + Hkv) * d > 16384 * 40 * 128:
        T = _log_int(rng, 1, 16384)
    rot = rng.choice([32, 64, d])
    return _rope(rng.choice(["rope_fwd", "rope_bwd"]), T, Hq, Hkv, d, rot, rng.choice([1, 1, 2, 3]),
                 rng.random() < 0.7, rng.random() < 0.4, rng.random() < 0.5)


def work(case):
    d, Hq, Hkv = case["d"], case["Hq"], case["Hkv"]
    if case["op"] == "attn_bwd":
        rows = case["B"] * case["S"]
        # read q, o, dout, k, v and the log-sum-exps (and their gradients); write dq, dk, dv
        nbytes = rows * d * 2 * (4 * Hq + 4 * Hkv) + rows * Hq * 4 * (2 if case["dlse"] else 1)
        scores = case["B"] * Hq * (case["S"] * (case["S"] + 1) // 2 if case["causal"] else case["S"] * case["S"])
        return {"bytes": nbytes, "flops": 5 * 2 * d * scores}  # S, dP, dV, dQ and dK
    elems = case["T"] * (Hq + Hkv) * d
    streams = 2 if case["op"] == "rope_fwd" else 3
    small = case["T"] * case["axes"] * 4 + case["rot"] * 2 + (4 * d if case["norm"] else 0)
    if case["op"] == "rope_bwd" and case["norm"]:
        small += 2 * d * 4
    return {"bytes": elems * 2 * streams + small, "flops": elems * (7 if case["op"] == "rope_fwd" else 14)}


# ----------------------------------------------------------------------------------------- inputs
def _sections(case):
    """Rotation pairs per position axis: an even share each, the first axis taking the rest."""
    pairs, n = case["rot"] // 2, case["axes"]
    each = pairs // (n + 1) if n > 1 else 0
    return [pairs - each * (n - 1)] + [each] * (n - 1)


def _attn_inputs(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    B, S, Hq, Hkv, d = (case[n] for n in ("B", "S", "Hq", "Hkv", "d"))

    def normal(*shape, gain=1.0):
        return (torch.randn(shape, generator=g, device=DEVICE) * gain).to(torch.bfloat16)

    q, k, v = normal(B, S, Hq, d), normal(B, S, Hkv, d), normal(B, S, Hkv, d)
    dout = normal(B, S, Hq, d, gain=0.05)
    dlse = torch.randn((B, S, Hq), generator=g, device=DEVICE) * 0.01 if case["dlse"] else None
    scale = 1.0 / math.sqrt(d)
    # the forward pass that the gradients belong to: its output and log-sum-exps
    out = torch.empty_like(q)
    lse = torch.empty((B, S, Hq), device=DEVICE)
    mask = torch.ones((S, S), dtype=torch.bool, device=DEVICE).triu(1) if case["causal"] else None
    G = Hq // Hkv
    for b in range(B):
        for h in range(Hkv):
            qs = q[b, :, h * G:(h + 1) * G].float().transpose(0, 1)
            s = torch.matmul(qs, k[b, :, h].float().t()).mul_(scale)
            if mask is not None:
                s.masked_fill_(mask, float("-inf"))
            m = s.amax(-1, keepdim=True)
            p = s.sub_(m).exp_()
            total = p.sum(-1, keepdim=True)
            out[b, :, h * G:(h + 1) * G] = (torch.matmul(p, v[b, :, h].float()) / total).transpose(0, 1)
            lse[b, :, h * G:(h + 1) * G] = (m + total.log()).squeeze(-1).t()
    return {"q": q, "k": k, "v": v, "out": out, "lse": lse, "dout": dout, "dlse": dlse, "scale": scale, "mask": mask}


def _rope_inputs(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    T, Hq, Hkv, d, rot, axes = (case[n] for n in ("T", "Hq", "Hkv", "d", "rot", "axes"))

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEVICE).mul_(1.5).to(torch.bfloat16)

    if case["fused"]:  # one projection's output: queries, keys and values of a token side by side
        qkv = normal(T, (Hq + 2 * Hkv) * d)
        q = qkv[:, :Hq * d].unflatten(1, (Hq, d))
        k = qkv[:, Hq * d:(Hq + Hkv) * d].unflatten(1, (Hkv, d))
    else:
        q, k = normal(T, Hq, d), normal(T, Hkv, d)
    if axes == 1:  # tokens of several sequences, some of them deep in a long context
        start = torch.randint(0, 1 << 20, (T // 512 + 1,), generator=g, device=DEVICE)
        positions = (start.repeat_interleave(512)[:T] + torch.arange(T, device=DEVICE) % 512).to(torch.int32)
    else:          # time, height and width on a grid of patches
        positions = torch.randint(0, 512, (axes, T), generator=g, device=DEVICE, dtype=torch.int32)
    exponent = torch.arange(rot // 2, device=DEVICE, dtype=torch.float64) * (2.0 / rot)
    inv_freq = (1000000.0 ** -exponent).float()
    state = {"q": q, "k": k, "positions": positions, "inv_freq": inv_freq, "q_weight": None, "k_weight": None,
             "eps": 1e-6, "sections": _sections(case), "interleaved": case["interleaved"]}
    if case["norm"]:
        for name in ("q_weight", "k_weight"):
            state[name] = (1.0 + 0.2 * torch.randn((d,), generator=g, device=DEVICE)).to(torch.bfloat16)
    if case["op"] == "rope_bwd":
        state["dq_out"], state["dk_out"] = normal(T, Hq, d), normal(T, Hkv, d)
    return state


def _inputs(case, seed):
    return _attn_inputs(case, seed) if case["op"] == "attn_bwd" else _rope_inputs(case, seed)


def prepare(case, seed):
    state = _inputs(case, seed)
    state["op"], state["case"] = case["op"], dict(case)
    if own:
        import io_aware_exact_flash_gb300 as fa

        state["fa"] = fa
        q, k = state["q"], state["k"]
        if case["op"] == "attn_bwd":
            state["grads"] = tuple(torch.empty_like(t) for t in (q, k, state["v"]))
            need = fa.fa_bwd_workspace_bytes(case["B"], case["Hq"], case["Hkv"], case["S"], case["d"], case["causal"])
            state["workspace"] = torch.empty(need, dtype=torch.uint8, device=DEVICE)
        else:
            state["q_res"] = torch.empty(q.shape, dtype=q.dtype, device=DEVICE)
            state["k_res"] = torch.empty(k.shape, dtype=k.dtype, device=DEVICE)
            if case["op"] == "rope_bwd":
                need = fa.fa_qk_norm_rope_bwd_workspace_bytes(case["T"], case["Hq"], case["Hkv"], case["d"])
                state["workspace"] = torch.empty(need, dtype=torch.uint8, device=DEVICE)
    return state


# --------------------------------------------------------------------------------------- plain forms
def _plain_attn_bwd(st):
    q, k, v, out, lse, dout = (st[n] for n in ("q", "k", "v", "out", "lse", "dout"))
    B, S, Hq, d = q.shape
    Hkv = k.shape[2]
    G = Hq // Hkv
    scale, mask = st["scale"], st["mask"]
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    for b in range(B):
        for h in range(Hkv):
            hs = slice(h * G, (h + 1) * G)
            qf, dof = q[b, :, hs].float().transpose(0, 1), dout[b, :, hs].float().transpose(0, 1)  # [G, S, d]
            kf, vf = k[b, :, h].float(), v[b, :, h].float()                                       # [S, d]
            delta = (dof * out[b, :, hs].float().transpose(0, 1)).sum(-1)                         # [G, S]
            if st["dlse"] is not None:
                delta = delta - st["dlse"][b, :, hs].t()
            p = torch.matmul(qf, kf.t()).mul_(scale).sub_(lse[b, :, hs].t().unsqueeze(-1)).exp_()
            if mask is not None:
                p.masked_fill_(mask, 0.0)
            dv[b, :, h] = torch.matmul(p.transpose(1, 2), dof).sum(0)
            ds = torch.matmul(dof, vf.t()).sub_(delta.unsqueeze(-1)).mul_(p)
            dq[b, :, hs] = torch.matmul(ds, kf).mul_(scale).transpose(0, 1)
            dk[b, :, h] = torch.matmul(ds.transpose(1, 2), qf).sum(0).mul_(scale)
    return dq, dk, dv


def _plain_angles(st):
    """cos and sin [T, pairs] of each token's rotation; the angles are formed in 64 bits."""
    pos = st["positions"].double().reshape(-1, st["positions"].shape[-1])  # [axes, T]
    axis = torch.cat([torch.full((n,), a, device=pos.device) for a, n in enumerate(st["sections"])])
    angle = pos[axis].t() * st["inv_freq"].double()
    return angle.cos().float(), angle.sin().float()


def _plain_split(x, pairs, interleaved):
    """First and second members of each rotated pair, and what stays unrotated."""
    if interleaved:
        return x[..., 0:2 * pairs:2], x[..., 1:2 * pairs:2], x[..., 2 * pairs:]
    return x[..., :pairs], x[..., pairs:2 * pairs], x[..., 2 * pairs:]


def _plain_rotate(x, cos, sin, interleaved):
    a, b, rest = _plain_split(x, cos.shape[-1], interleaved)
    c, s = cos.unsqueeze(1), sin.unsqueeze(1)
    first, second = a * c - b * s, b * c + a * s
    turned = torch.stack((first, second), -1).flatten(-2) if interleaved else torch.cat((first, second), -1)
    return torch.cat((turned, rest), -1)


def _plain_rope_fwd(st):
    cos, sin = _plain_angles(st)
    res = []
    for x, w in ((st["q"], st["q_weight"]), (st["k"], st["k_weight"])):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + st["eps"]) * w.float()
        res.append(_plain_rotate(x, cos, sin, st["interleaved"]).to(torch.bfloat16))
    return tuple(res)


def _plain_rope_bwd(st):
    cos, sin = _plain_angles(st)
    dx, dw = [], []
    for x, w, dy in ((st["q"], st["q_weight"], st["dq_out"]), (st["k"], st["k_weight"], st["dk_out"])):
        g = _plain_rotate(dy.float(), cos, -sin, st["interleaved"])  # the inverse rotation
        if w is not None:
            x = x.float()
            r = torch.rsqrt((x * x).mean(-1, keepdim=True) + st["eps"])
            xhat = x * r
            dw.append((g * xhat).sum(0, dtype=torch.float64).sum(0).float())
            g = g * w.float()
            g = (g - xhat * (g * xhat).mean(-1, keepdim=True)) * r
        dx.append(g.to(torch.bfloat16))
    return tuple(dx + dw)


# ----------------------------------------------------------------------------------------- one pass
def run(state):
    op = state["op"]
    if not own:
        return {"attn_bwd": _plain_attn_bwd, "rope_fwd": _plain_rope_fwd, "rope_bwd": _plain_rope_bwd}[op](state)
    fa = state["fa"]
    if op == "attn_bwd":
        dq, dk, dv = state["grads"]
        return fa.fa_bwd(state["q"], state["k"], state["v"], state["out"], state["lse"], state["dout"],
                         causal=state["mask"] is not None, scale=state["scale"], dlse=state["dlse"], dq=dq, dk=dk,
                         dv=dv, workspace=state["workspace"])
    common = dict(positions=state["positions"], inv_freq=state["inv_freq"], q_weight=state["q_weight"],
                  k_weight=state["k_weight"], eps=state["eps"], sections=state["sections"],
                  interleaved=state["interleaved"])
    if op == "rope_fwd":
        return fa.fa_qk_norm_rope(state["q"], state["k"], q_out=state["q_res"], k_out=state["k_res"], **common)
    dq, dk, dq_weight, dk_weight = fa.fa_qk_norm_rope_bwd(
        state["dq_out"], state["dk_out"], state["q"], state["k"], dq=state["q_res"], dk=state["k_res"],
        workspace=state["workspace"], **common)
    return (dq, dk) if dq_weight is None else (dq, dk, dq_weight, dk_weight)


# ---------------------------------------------------------------------------------- 64-bit definition
def _exact_attn_bwd(st, case):
    B, S, Hq, Hkv, d = (case[n] for n in ("B", "S", "Hq", "Hkv", "d"))
    grads = [torch.zeros(t.shape, dtype=torch.float64, device=DEVICE) for t in (st["q"], st["k"], st["v"])]
    rows = 2048  # query rows at a time
    col = torch.arange(S, device=DEVICE)
    for b in range(B):
        for hq in range(Hq):
            hk = hq // (Hq // Hkv)
            K, V = st["k"][b, :, hk].double(), st["v"][b, :, hk].double()
            for r0 in range(0, S, rows):
                r = slice(r0, min(S, r0 + rows))
                n = r.stop if case["causal"] else S  # keys that these rows can see
                Q, dO, O = (st[x][b, r, hq].double() for x in ("q", "dout", "out"))
                logp = st["scale"] * torch.einsum("id,jd->ij", Q, K[:n]) - st["lse"][b, r, hq].double()[:, None]
                if case["causal"]:
                    logp = torch.where(col[None, :n] <= col[r, None], logp, float("-inf"))
                P = torch.exp(logp)
                dP = torch.einsum("id,jd->ij", dO, V[:n])
                shift = torch.einsum("id,id->i", dO, O)
                if st["dlse"] is not None:
                    shift = shift - st["dlse"][b, r, hq].double()
                dS = st["scale"] * P * (dP - shift[:, None])
                grads[0][b, r, hq] = torch.einsum("ij,jd->id", dS, K[:n])
                grads[1][b, :n, hk] += torch.einsum("ij,id->jd", dS, Q)
                grads[2][b, :n, hk] += torch.einsum("ij,id->jd", P, dO)
    return tuple(grads)


def _exact_rope(st, case):
    pairs = case["rot"] // 2
    pos = st["positions"].reshape(case["axes"], -1).double()
    owner = [a for a, n in enumerate(_sections(case)) for _ in range(n)]
    phase = torch.stack([pos[owner[i]] * float(st["inv_freq"][i]) for i in range(pairs)], 1)
    turn = torch.complex(torch.cos(phase), torch.sin(phase))[:, None, :]  # a pair as a complex number
    first = [2 * i if case["interleaved"] else i for i in range(pairs)]
    second = [2 * i + 1 if case["interleaved"] else i + pairs for i in range(pairs)]

    def rotate(x, by):
        z = torch.complex(x[..., first], x[..., second]) * by
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    main, sums = [], []
    for name in ("q", "k"):
        x = st[name].double()
        w = None if st[name + "_weight"] is None else st[name + "_weight"].double()
        size = x.shape[-1]
        rms = None if w is None else ((x ** 2).sum(-1, keepdim=True) / size + st["eps"]) ** 0.5
        if case["op"] == "rope_fwd":
            main.append(rotate(x if w is None else x / rms * w, turn))
            continue
        back = rotate(st["d" + name + "_out"].double(), turn.conj())
        if w is None:
            main.append(back)
            continue
        sums.append((back * x / rms).sum((0, 1)))
        inner = (back * w * x).sum(-1, keepdim=True)
        main.append(back * w / rms - x * inner / (size * rms ** 3))
    return tuple(main + sums)


def exact(case, seed):
    if case["op"] == "attn_bwd":
        if work(case)["flops"] > 6e12:
            return None  # too long in 64 bits
        return _exact_attn_bwd(_inputs(case, seed), case)
    return _exact_rope(_inputs(case, seed), case)
