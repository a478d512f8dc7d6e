"""Host-side refusals of the backward pass and of the query/key norm with rotary positions: bad arguments
return their status before anything touches a device (no GPU needed; addresses are never dereferenced)."""
import ctypes

import pytest

from tests.test_abi import lib  # noqa: F401  (the library fixture)

try:
    import torch

    HAS_GPU = torch.cuda.is_available()
except Exception:  # pragma: no cover
    HAS_GPU = False
# Calls whose arguments are all fine end at the missing device. Where there is one they would launch
# kernels on addresses that are not memory, so they are made only without one.
without_a_gpu = pytest.mark.skipif(HAS_GPU, reason="the calls would run: their addresses are made up")

MB = 1 << 20
BASE = 1 << 40  # 16-byte aligned addresses, 64 MB apart, never dereferenced


def at(i, off=0):
    return BASE + 64 * MB * i + off


def vp(x):
    return ctypes.c_void_p(x) if x else None


def _bwd(lib, **kw):  # noqa: F811
    a = dict(q=at(0), k=at(1), v=at(2), o=at(3), lse=at(4), do=at(5), dlse=None, dq=at(6), dk=at(7), dv=at(8), B=1,
             Hq=4, Hkv=2, S=128, d=128, causal=1, scale=0.1, ws=at(9), wsb=MB)
    a.update(kw)
    return lib.fa_bwd(vp(a["q"]), vp(a["k"]), vp(a["v"]), vp(a["o"]), vp(a["lse"]), vp(a["do"]), vp(a["dlse"]),
                      vp(a["dq"]), vp(a["dk"]), vp(a["dv"]), a["B"], a["Hq"], a["Hkv"], a["S"], a["d"], a["causal"],
                      a["scale"], vp(a["ws"]), a["wsb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=0), 1), (dict(o=0), 1), (dict(lse=0), 1), (dict(do=0), 1), (dict(dq=0), 1), (dict(dv=0), 1),
    (dict(B=0), 1), (dict(S=0), 1), (dict(S=-3), 1), (dict(Hq=3), 1), (dict(Hkv=0), 1), (dict(Hq=0), 1),
    (dict(scale=0.0), 1), (dict(scale=float("inf")), 1), (dict(scale=float("nan")), 1),
    (dict(dq=at(0)), 1), (dict(dk=at(1, 1024)), 1), (dict(dv=at(7, 128)), 1), (dict(dq=at(5)), 1),
    (dict(ws=at(6)), 1), (dict(dk=at(9, 2048)), 1), (dict(dlse=at(8)), 1),
    (dict(d=96), 2), (dict(d=32), 2), (dict(B=1 << 12, S=1 << 20), 2), (dict(Hq=1 << 14, Hkv=1 << 14, S=1 << 24), 2),
    (dict(q=at(0, 8)), 3), (dict(dk=at(7, 2)), 3), (dict(lse=at(4, 2)), 3), (dict(dlse=at(10, 1)), 3),
    (dict(ws=at(9, 16)), 3),
    (dict(ws=0), 4), (dict(wsb=4095), 4),
])
def test_bwd_host_validation(lib, kw, code):  # noqa: F811
    assert _bwd(lib, **kw) == code


def test_bwd_workspace(lib):  # noqa: F811
    from io_aware_exact_flash_gb300 import binding as b

    # 256 floats per query tile and head
    assert b.fa_bwd_workspace_bytes(1, 4, 2, 128, 128) == 4 * 1024
    assert b.fa_bwd_workspace_bytes(3, 4, 2, 129, 64, True) == 3 * 4 * 2 * 1024
    for bad in ((0, 4, 2, 128, 128), (1, 3, 2, 128, 128), (1, 4, 2, 0, 64), (1, 4, 2, 128, 80)):
        assert b.fa_bwd_workspace_bytes(*bad) == 0


@without_a_gpu
def test_bwd_workspace_is_just_enough(lib):  # noqa: F811
    assert _bwd(lib, wsb=4096) not in (1, 2, 3, 4)  # past the checks


def _rope(lib, bwd=False, **kw):  # noqa: F811
    a = dict(q=at(0), qs=512, k=at(1), ks=256, wq=at(2), wk=at(3), eps=1e-6, pos=at(4), inv=at(5), axes=1, sec=None,
             rot=128, inter=0, T=10, Hq=4, Hkv=2, d=128, qo=at(6), qos=512, ko=at(7), kos=256, gq=at(8), gqs=512,
             gk=at(9), gks=256, dwq=at(10), dwk=at(11), ws=at(12), wsb=MB)
    a.update(kw)
    sec = (ctypes.c_int32 * len(a["sec"]))(*a["sec"]) if a["sec"] else None
    shared = (vp(a["wq"]), vp(a["wk"]), a["eps"], vp(a["pos"]), vp(a["inv"]), a["axes"], sec, a["rot"], a["inter"],
              a["T"], a["Hq"], a["Hkv"], a["d"])
    if not bwd:
        return lib.fa_qk_norm_rope(vp(a["q"]), a["qs"], vp(a["k"]), a["ks"], *shared, vp(a["qo"]), a["qos"],
                                   vp(a["ko"]), a["kos"], None)
    return lib.fa_qk_norm_rope_bwd(vp(a["gq"]), a["gqs"], vp(a["gk"]), a["gks"], vp(a["q"]), a["qs"], vp(a["k"]),
                                   a["ks"], *shared, vp(a["qo"]), a["qos"], vp(a["ko"]), a["kos"], vp(a["dwq"]),
                                   vp(a["dwk"]), vp(a["ws"]), a["wsb"], None)


SHARED = [
    (dict(q=0), 1), (dict(qo=0), 1), (dict(k=0), 1), (dict(ko=0), 1), (dict(wk=0), 1), (dict(wq=0), 1),
    (dict(T=-1), 1), (dict(Hq=0), 1), (dict(Hkv=-2), 1), (dict(eps=0.0), 1), (dict(eps=float("nan")), 1),
    (dict(rot=-16), 1), (dict(rot=144), 1), (dict(pos=0), 1), (dict(inv=0), 1), (dict(axes=0), 1),
    (dict(axes=2), 1), (dict(axes=2, sec=[32, 31]), 1), (dict(axes=2, sec=[65, -1]), 1),
    (dict(wq=0, wk=0, rot=0), 1),                    # nothing to do
    (dict(qs=511), 1), (dict(qs=0), 1), (dict(kos=-256), 1),
    (dict(qo=at(1)), 1), (dict(ko=at(6, 512)), 1),   # an output over the other tensors
    (dict(qo=at(4)), 1), (dict(ko=at(3)), 1), (dict(qo=at(5)), 1),
    (dict(qo=at(0, 16)), 1), (dict(qo=at(0), qos=520), 1),  # over its own input, but not in place
    (dict(d=96), 2), (dict(rot=24), 2), (dict(axes=5, sec=[16, 16, 16, 8, 8]), 2), (dict(T=1 << 31), 2),
    (dict(q=at(0, 8)), 3), (dict(qs=516), 3), (dict(kos=257), 3), (dict(wq=at(2, 2)), 3), (dict(pos=at(4, 2)), 3),
    (dict(inv=at(5, 1)), 3),
]


@pytest.mark.parametrize("kw,code", SHARED)
@pytest.mark.parametrize("bwd", [False, True])
def test_rope_host_validation(lib, bwd, kw, code):  # noqa: F811
    assert _rope(lib, bwd, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(gq=0), 1), (dict(gks=128), 1), (dict(dwq=0), 1), (dict(dwk=0), 1), (dict(qo=at(9)), 1),
    (dict(dwk=at(10, 256)), 1), (dict(dwq=at(12, 4096)), 1), (dict(ws=at(7)), 1), (dict(dwq=at(8, 64)), 1),
    (dict(dwk=at(2)), 1), (dict(ws=at(4)), 1),
    (dict(gk=at(9, 8)), 3), (dict(dwq=at(10, 2)), 3),
])
def test_rope_bwd_host_validation(lib, kw, code):  # noqa: F811
    assert _rope(lib, True, **kw) == code


@without_a_gpu
def test_rope_calls_that_pass_validation(lib):  # noqa: F811
    """In place, interleaved rows of one projection, and tensors that are not needed: past the checks (the
    calls then need a device, so here they fail with another status)."""
    fine = (1, 2, 3, 4)
    assert _rope(lib, qo=at(0), ko=at(1)) not in fine
    fused = dict(q=at(0), qs=1024, k=at(0, 1024), ks=1024)  # 4 + 2 + 2 heads of 128 side by side
    assert _rope(lib, **fused) not in fine
    assert _rope(lib, **fused, qo=at(0), qos=1024, ko=at(0, 1024), kos=1024) not in fine
    assert _rope(lib, **fused, qo=at(0, 1024), qos=1024) == 1  # queries written over the keys
    assert _rope(lib, q=0, k=0, qo=0, ko=0, pos=0, T=0) not in fine
    assert _rope(lib, rot=0, pos=0, inv=0) not in fine
    assert _rope(lib, True, wq=0, wk=0, q=0, k=0, dwq=0, dwk=0, ws=0, wsb=0) not in fine
    assert _rope(lib, True, qo=at(8), ko=at(9)) not in fine
    assert _rope(lib, axes=3, sec=[16, 24, 24]) not in fine
    assert _rope(lib, axes=2, sec=[64, 0]) not in fine


def test_rope_bwd_workspace(lib):  # noqa: F811
    from io_aware_exact_flash_gb300 import binding as b

    one = b.fa_qk_norm_rope_bwd_workspace_bytes(1, 4, 2, 128)
    many = b.fa_qk_norm_rope_bwd_workspace_bytes(100000, 4, 2, 128)
    assert 0 < one <= many and one % (2 * 128 * 4) == 0
    assert b.fa_qk_norm_rope_bwd_workspace_bytes(0, 4, 2, 64) == 0
    assert b.fa_qk_norm_rope_bwd_workspace_bytes(-1, 4, 2, 64) == 0
    assert b.fa_qk_norm_rope_bwd_workspace_bytes(8, 4, 2, 96) == 0
