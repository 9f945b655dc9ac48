"""Scored attention on the CPU: the 64-bit definition against differences, the bucket rule, and
what the calls refuse before they touch a GPU."""
import ctypes
import math

import numpy as np
import pytest

import scored_ref as S


@pytest.fixture(scope="module")
def F():
    from microscaled_precision_causal_gb300 import build
    build.build()
    import microscaled_precision_causal_gb300 as F
    return F


CASES = {
    "cap": dict(softcap=1.5), "slopes": dict(slopes=np.array([0.5, 0.1])), "prefix": dict(prefix=[3, 0]),
    "window": dict(window=(2, 1)), "rel": dict(rel=True), "all": dict(softcap=2.0, slopes=np.array([0.2, 0.05]), rel=True,
                                                                     prefix=[2, 5], window=(1, 0)),
}


@pytest.mark.parametrize("name", CASES)
def test_gradients_equal_central_differences(name):
    rng = np.random.default_rng(3)
    kw = dict(CASES[name])
    lengths, hq, hkv, d = [6, 4], 2, 1, 3
    if kw.get("rel"):
        kw["rel"] = rng.standard_normal((hq, 5))
    x = {n: rng.standard_normal((10, h, d)) for n, h in (("q", hq), ("k", hkv), ("v", hkv))}
    if kw.get("rel") is not None:
        x["rel"] = kw.pop("rel")
    dout = rng.standard_normal((10, hq, d))

    def loss(y):
        return (S.run(lengths=lengths, **y, **kw)["o"] * dout).sum()
    got = S.run(lengths=lengths, dout=dout, **x, **kw)
    for n in x:
        want = np.zeros_like(x[n])
        for at in np.ndindex(*x[n].shape):
            hi, lo = (dict(x, **{n: x[n].copy()}) for _ in range(2))
            hi[n][at] += 1e-5
            lo[n][at] -= 1e-5
            want[at] = (loss(hi) - loss(lo)) / 2e-5
        # central differences: h^2 times the third derivative (order 10) and 1e-15 / h
        assert np.abs(got["d" + n] - want).max() <= 1e-8, n


@pytest.mark.parametrize("nb,md,both", [(32, 128, True), (32, 128, False), (16, 96, True), (4, 2, True), (2, 5, False),
                                        (3, 7, False), (64, 1024, False)])
def test_bucket_rule(nb, md, both):
    side = nb // 2 if both else nb
    ids = [S.bucket(-n, nb, md, both) for n in range(1100)]
    assert ids == sorted(ids) and ids[0] == 0 and max(ids) == side - 1
    assert all(ids[n] == n for n in range(side // 2)) and all(i == side - 1 for i in ids[md:])
    ups = [S.bucket(n, nb, md, both) for n in range(1, 1100)]
    assert ups == ([i + side for i in ids[1:]] if both else [0] * 1099)


def _opts(F, **kw):
    o = F.default_score_options()
    for n, x in kw.items():
        setattr(o, n, x)
    return o


def test_default_score_options(F):
    o = F.default_score_options()
    assert (o.softcap, o.slopes, o.rel_bias, o.rel_max, o.prefix_lens, o.window_left, o.window_right) == (
        0.0, None, None, 0, None, -1, -1)


FWD = [
    (dict(d=96), {}, -2), (dict(hq=3), {}, -2), (dict(hq=0), {}, -1), (dict(hq=2048, hkv=2048), {}, -2),
    (dict(causal=2), {}, -1), (dict(T=-1), {}, -1), (dict(T=1 << 27), {}, -2), (dict(N=-1), {}, -1),
    (dict(q=0), {}, -1), (dict(k=0), {}, -1), (dict(v=0), {}, -1), (dict(cu=0), {}, -1), (dict(plan=0), {}, -1),
    (dict(out=0), {}, -1), (dict(lse=0), {}, -1), (dict(q=264), {}, -3), (dict(v=257), {}, -3), (dict(out=258), {}, -3),
    (dict(lse=258), {}, -3), (dict(plan=260), {}, -3),
    ({}, dict(softcap=-1.0), -1), ({}, dict(softcap=math.inf), -1), ({}, dict(softcap=math.nan), -1),
    ({}, dict(softcap=1e-32), -2), ({}, dict(softcap=1e32), -2),
    ({}, dict(rel_bias=256, rel_max=0), -1), ({}, dict(rel_bias=256, rel_max=1025), -2),
    ({}, dict(rel_bias=257, rel_max=4), -3), ({}, dict(slopes=258), -3), ({}, dict(prefix_lens=258), -3),
]


@pytest.mark.parametrize("i", range(len(FWD)))
def test_forward_refusals(F, i):
    args, opts, want = FWD[i]
    a = dict(dict(q=256, k=256, v=256, cu=256, N=1, T=100, hq=4, hkv=2, d=128, causal=1, plan=256, out=256, lse=256), **args)
    o = _opts(F, **opts)
    assert F.lib().flamia_scored_fwd(a["q"], a["k"], a["v"], a["cu"], a["N"], a["T"], a["hq"], a["hkv"], a["d"], a["causal"],
                                     0.0, ctypes.byref(o), a["plan"], a["out"], a["lse"], None) == want


@pytest.mark.parametrize("softcap,scale,d,want", [
    (1e-3, 1.2e30, 128, -2), (0.75, 1e30, 64, -2), (1e-30, 1.3, 64, -2), (0.8, 1e30, 64, -3), (1e-30, 0.9, 64, -3),
    (1e-30, 0.0, 64, -3), (1e30, 8e-31, 128, -3), (0.0, 1.2e30, 128, -3), (0.0, 1.3e30, 128, -2), (0.0, 7e-31, 128, -2)])
def test_cap_and_scale_ranges(F, softcap, scale, d, want):
    """-3: the checks went on to the misaligned output."""
    o = _opts(F, softcap=softcap)
    assert F.lib().flamia_scored_fwd(256, 256, 256, 256, 1, 100, 4, 2, d, 1, scale, ctypes.byref(o), 256, 258, 256,
                                     None) == want
    assert F.lib().flamia_scored_bwd(256, 256, 256, 258, 256, 256, 256, 1, 100, 4, 2, d, 1, scale, ctypes.byref(o), 256, 256,
                                     256, 256, None, 256, 1 << 30, None) == want


BWD = FWD[:20] + [
    (dict(dout=0), {}, -1), (dict(dq=0), {}, -1), (dict(dk=0), {}, -1), (dict(dv=0), {}, -1), (dict(ws=0), {}, -1),
    (dict(dout=264), {}, -3), (dict(dq=264), {}, -3), (dict(dk=264), {}, -3), (dict(dv=264), {}, -3), (dict(ws=128), {}, -3),
    (dict(drel=256), {}, -1), (dict(drel=258), dict(rel_bias=256, rel_max=4), -3), (dict(bytes=1000), {}, -4),
    (dict(drel=256, bytes=100 * 4 * 4 + 256), dict(rel_bias=256, rel_max=64), -4), ({}, dict(softcap=-2.0), -1),
]


@pytest.mark.parametrize("i", range(len(BWD)))
def test_backward_refusals(F, i):
    args, opts, want = BWD[i]
    a = dict(dict(q=256, k=256, v=256, cu=256, N=1, T=100, hq=4, hkv=2, d=128, causal=1, plan=256, out=256, lse=256, dout=256,
                  dq=256, dk=256, dv=256, drel=0, ws=256, bytes=1 << 30), **args)
    o = _opts(F, **opts)
    assert F.lib().flamia_scored_bwd(a["q"], a["k"], a["v"], a["out"], a["lse"], a["dout"], a["cu"], a["N"], a["T"], a["hq"],
                                     a["hkv"], a["d"], a["causal"], 0.0, ctypes.byref(o), a["plan"], a["dq"], a["dk"],
                                     a["dv"], a["drel"], a["ws"], a["bytes"], None) == want


def test_workspace_bytes(F):
    f = F.flamia_scored_bwd_workspace_bytes
    assert f(-1, 1, 4, 2, 128) == 0 and f(100, 1, 4, 2, 128, -1) == 0
    assert 0 < f(1000, 2, 4, 2, 128) < f(1000, 2, 4, 2, 128, 64) < f(1000, 2, 4, 2, 128, 128)
    assert f(0, 0, 4, 2, 128) > 0


@pytest.mark.parametrize("nb,hq,md,both,R,table,want", [
    (1, 4, 8, 0, 8, 256, -1), (32, 0, 128, 0, 128, 256, -1), (32, 4, 0, 0, 128, 256, -1), (32, 4, 16, 0, 128, 256, -1),
    (31, 4, 128, 1, 128, 256, -1), (2, 4, 128, 1, 128, 256, -1), (32, 4, 128, 2, 128, 256, -1), (32, 4, 128, 0, 127, 256, -1),
    (32, 4, 128, 0, 1025, 256, -2), (2048, 4, 1024, 1, 1024, 256, -2), (32, 2000, 128, 0, 128, 256, -2),
    (32, 4, 128, 0, 128, 0, -1), (32, 4, 128, 0, 128, 258, -3)])
def test_bucket_refusals(F, nb, hq, md, both, R, table, want):
    assert F.lib().flamia_relbias_expand(table, nb, hq, md, both, 256, R, None) == want
    assert F.lib().flamia_relbias_reduce(table, R, nb, hq, md, both, 256, None) == want


@pytest.mark.parametrize("window,want", [((-1, -1), (-1, -1)), ((2**32 + 5, 2**31), (2**31 - 1, 2**31 - 1)), ((3, -7), (3, -1)),
                                         ((-2**33, 0), (-1, 0))])
def test_windows_past_32_bits(F, window, want):
    """As bounds that no document reaches, or none: ctypes would keep the low 32 bits."""
    pytest.importorskip("torch")
    att = F.FlamiaScoredAttention(10, 1, 1, 1, 64, device="cpu", window=window)
    assert (att.opts.window_left, att.opts.window_right) == want == att.window


@pytest.mark.parametrize("shape", [(4, 16), (3, 17), (5, 17), (68,), (1, 4, 17)])
def test_relative_bias_shapes(F, shape):
    """An even width would be written past its end, and so would too few rows."""
    torch = pytest.importorskip("torch")
    table, rel = torch.zeros(8, 4), torch.zeros(shape)
    with pytest.raises(F.FlamiaError, match="rel_max"):
        F.flamia_relbias_expand(table, 8, False, rel, stream=0)
    with pytest.raises(F.FlamiaError, match="rel_max"):
        F.flamia_relbias_reduce(rel, 8, False, table, stream=0)


def test_object_refusals(F):
    """What FlamiaScoredAttention refuses, on CPU tensors: nothing is launched."""
    torch = pytest.importorskip("torch")
    new = lambda **kw: F.FlamiaScoredAttention(**dict(dict(total_tokens=10, num_seqs=2, hq=4, hkv=2, head_dim=64,
                                                           device="cpu"), **kw))
    for bad in (dict(head_dim=96), dict(hq=3), dict(total_tokens=-1), dict(buckets=(31, 128, True)),
                dict(buckets=(32, 16, False)), dict(buckets=(32, 2000, False)), dict(buckets=(1, 8, False))):
        with pytest.raises(F.FlamiaError):
            new(**bad)
    att = new()
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)
    q, k, cu = z(10, 4, 64), z(10, 2, 64), z(3, dtype=torch.int32)
    ok = dict(q=q, k=k, v=k, cu_seqlens=cu)
    with pytest.raises(F.FlamiaError, match="CUDA device"):
        att.forward(**ok)
    for bad in (dict(q=q.float()), dict(q=z(9, 4, 64)), dict(k=z(10, 4, 64)), dict(v=z(2, 10, 64).transpose(0, 1)),
                dict(cu_seqlens=cu.long()), dict(cu_seqlens=z(4, dtype=torch.int32)), dict(slopes=z(4)),
                dict(slopes=z(2, dtype=torch.float32)), dict(prefix_lens=z(3, dtype=torch.int32)),
                dict(table=z(32, 4, dtype=torch.float32))):
        with pytest.raises(F.FlamiaError, match="want|table"):
            att.forward(**dict(ok, **bad))
    bwd = dict(ok, out=q, lse=z(4, 10, dtype=torch.float32), dout=q)
    for bad in (dict(out=q.float()), dict(lse=z(10, 4, dtype=torch.float32)), dict(dout=z(10, 2, 64))):
        with pytest.raises(F.FlamiaError, match="want"):
            att.backward(**dict(bwd, **bad))
    with pytest.raises(F.FlamiaError, match="needs one"):
        new(buckets=(32, 128, True)).forward(**ok)
