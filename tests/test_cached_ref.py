"""The paged cache on the CPU: the 64-bit definition by small cases, and what the calls refuse
before they touch a GPU."""
import ctypes

import numpy as np
import pytest

import cached_ref as C
import oracle as O


@pytest.fixture(scope="module")
def F():
    from microscaled_precision_causal_gb300 import build
    build.build()
    import microscaled_precision_causal_gb300 as F
    return F


def test_rows_are_quantized_by_themselves():
    """448 2^e at least the largest value, 224 2^e below it; every value within half a step; a row alone the same."""
    rng = np.random.default_rng(1)
    x = rng.standard_normal((40, 3, 64)) * np.exp2(rng.integers(-60, 60, (40, 3, 1)))
    x[5] = 0
    x[6, 1] = np.nan
    codes, scales = C.quantize(x)
    y = C.dequantize(codes, scales)
    assert (scales[5] == 127).all() and (y[5] == 0).all() and scales[6, 1] == 255 and np.isnan(y[6, 1]).all()
    fine = np.ones((40, 3), bool)
    fine[5], fine[6, 1] = False, False
    top, s = np.abs(x[fine]).max(-1), np.exp2(scales[fine].astype(float) - 127)
    assert (top <= 448 * s).all() and (top > 224 * s).all()
    step = np.maximum(2.0 ** -4 * np.abs(x[fine]), 2.0 ** -10 * s[:, None])       # half a step, or half a subnormal one
    assert (np.abs(y[fine] - x[fine]) <= step).all()
    assert np.array_equal(C.quantize(x[7, 2])[0], codes[7, 2])


@pytest.mark.parametrize("left,softcap", [(-1, 0.0), (3, 0.0), (0, 2.0), (-1, 1.5)])
def test_definition_by_rows(left, softcap):
    rng = np.random.default_rng(2)
    c, L, group, d = 4, 11, 2, 5
    q, k, v = rng.standard_normal((c, 4, d)), rng.standard_normal((L, 2, d)), rng.standard_normal((L, 2, d))
    r = C.attend(q, k, v, group, left=left, softcap=softcap)
    for t in range(c):
        i = L - c + t
        seen = range(max(0, i - left) if left >= 0 else 0, i + 1)
        for h in range(4):
            s = np.array([q[t, h] @ k[j, h // group] / np.sqrt(d) for j in seen])
            s = softcap * np.tanh(s / softcap) if softcap else s
            w = np.exp(s)
            assert abs(r["lse"][h, t] - np.log(w.sum())) < 1e-12
            assert np.abs(r["o"][t, h] - sum(w[x] / w.sum() * v[j, h // group] for x, j in enumerate(seen))).max() < 1e-12


def test_definition_against_the_oracle():
    """A whole sequence as one chunk is causal attention."""
    rng = np.random.default_rng(3)
    q, k, v = (rng.standard_normal((20, h, 8)) for h in (4, 2, 2))
    o, lse = O.dense_attention(q, k, v, [0, 20], 4, 2)[:2]
    r = C.attend(q, k, v, 2)
    assert np.abs(r["o"] - o).max() < 1e-12 and np.abs(r["lse"] - lse).max() < 1e-12


def cache(F, **kw):
    return F.KVCache(**dict(dict(k=256, v=256, k_scales=256, v_scales=256, num_pages=10, page_size=16, hkv=2, head_dim=128,
                                 format=1), **kw))


CACHES = [
    (dict(k=None), -1), (dict(v=None), -1), (dict(k_scales=None), -1), (dict(v_scales=None), -1), (dict(num_pages=0), -1),
    (dict(hkv=0), -1), (dict(format=2), -1), (dict(format=-1), -1), (dict(page_size=0), -2), (dict(page_size=48), -2),
    (dict(page_size=256), -2), (dict(head_dim=96), -2), (dict(hkv=2048), -2), (dict(num_pages=1 << 30, hkv=4), -2),
    (dict(k=264), -3), (dict(v=264), -3), (dict(k_scales=264), -3), (dict(v_scales=257), -3),
]
CALLS = [
    (dict(table=None), -1), (dict(max_pages=0), -1), (dict(max_pages=1 << 27), -2), (dict(N=-1), -1), (dict(T=-1), -1),
    (dict(T=1 << 27), -2), (dict(plan=None), -1), (dict(plan=264), -3), (dict(table=258), -3),
]


def _refusals(call):
    base = dict(table=256, max_pages=4, N=2, T=100, plan=256)
    for args, want in CACHES:
        assert call(args, base) == want, args
    for args, want in CALLS:
        assert call({}, dict(base, **args)) == want, args


@pytest.mark.parametrize("what", ["write", "read"])
def test_write_and_read_refusals(F, what):
    f = getattr(F.lib(), f"flamia_cache_{what}")

    def call(kw, a, k=256, v=256):
        return f(ctypes.byref(cache(F, **kw)), a["table"], a["max_pages"], a["N"], a["T"], a["plan"], k, v, None)
    _refusals(call)
    ok = dict(table=256, max_pages=4, N=2, T=100, plan=256)
    assert call({}, ok, k=None) == -1 and call({}, ok, v=None) == -1
    assert call({}, ok, k=264) == -3 and call({}, ok, v=264) == -3
    assert f(None, 256, 4, 2, 100, 256, 256, 256, None) == -1
    assert call({}, dict(ok, T=0), k=None, v=None) == 0                              # no tokens: nothing is launched
    assert call(dict(format=0, k_scales=None, v_scales=None), ok, k=None) == -1      # (bf16 needs no scales)


def test_forward_refusals(F):
    L = F.lib()

    def call(kw, a):
        a = dict(dict(q=256, hq=4, chunk=3, left=-1, cap=0.0, scale=0.0, out=256, lse=256, ws=256, bytes=1 << 30), **a)
        return L.flamia_cached_fwd(a["q"], ctypes.byref(cache(F, **kw)), a["table"], a["max_pages"], a["N"], a["T"], a["hq"],
                                   a["chunk"], a["left"], a["cap"], a["scale"], a["plan"], a["out"], a["lse"], a["ws"],
                                   a["bytes"], None)
    _refusals(call)
    ok = dict(table=256, max_pages=4, N=2, T=100, plan=256)
    for args, want in [(dict(q=None), -1), (dict(out=None), -1), (dict(lse=None), -1), (dict(ws=None), -1), (dict(hq=0), -1),
                       (dict(hq=3), -2), (dict(hq=2048), -2), (dict(chunk=0), -1), (dict(chunk=1 << 30), -2),
                       (dict(cap=-1.0), -1), (dict(cap=float("nan")), -1), (dict(cap=1e-32), -2), (dict(cap=1e32), -2),
                       (dict(scale=1.3e30), -2), (dict(scale=7e-31), -2), (dict(scale=1e30, cap=0.5), -2), (dict(q=264), -3),
                       (dict(out=264), -3), (dict(lse=258), -3), (dict(ws=128), -3), (dict(bytes=1000), -4)]:
        assert call({}, dict(ok, **args)) == want, args
    need = F.flamia_cached_fwd_workspace_bytes(4, 2, 128, 100)
    assert call({}, dict(ok, chunk=100, bytes=need - 1)) == -4
    assert call({}, dict(ok, T=0, q=None, out=None, lse=None, ws=None)) == 0


def test_plan_refusals(F):
    L = F.lib()
    assert F.flamia_cache_plan_bytes(-1, 1, 4, 2) == 0 and F.flamia_cache_plan_bytes(10, 1, 0, 2) == 0
    assert F.flamia_cache_plan_bytes(1000, 3, 8, 2) >= 3 * 32
    ok = dict(cu=256, kv=256, N=2, T=100, hq=4, hkv=2, chunk=10, keys=64, left=-1, plan=256, bytes=1 << 20)

    def call(**kw):
        a = dict(ok, **kw)
        return L.flamia_cache_plan_build(a["cu"], a["kv"], a["N"], a["T"], a["hq"], a["hkv"], a["chunk"], a["keys"], a["left"],
                                         a["plan"], a["bytes"], None)
    for args, want in [(dict(cu=None), -1), (dict(kv=None), -1), (dict(plan=None), -1), (dict(N=-1), -1), (dict(T=-1), -1),
                       (dict(hq=0), -1), (dict(hkv=0), -1), (dict(hq=3), -2), (dict(hq=2048), -2), (dict(chunk=0), -1),
                       (dict(keys=0), -1), (dict(keys=1 << 31), -2), (dict(chunk=1 << 30), -2), (dict(T=1 << 27), -2),
                       (dict(plan=264), -3), (dict(cu=258), -3), (dict(kv=257), -3), (dict(bytes=64), -4)]:
        assert call(**args) == want, args


def test_object_refusals(F):
    """What the objects refuse, on CPU tensors: nothing is launched."""
    torch = pytest.importorskip("torch")
    for bad in (dict(num_pages=0), dict(page_size=24), dict(hkv=0), dict(head_dim=80), dict(fmt="fp8")):
        with pytest.raises(F.FlamiaError):
            F.FlamiaPagedCache(**dict(dict(num_pages=4, page_size=16, hkv=2, head_dim=64, device="cpu"), **bad))
    new = lambda **kw: F.FlamiaCachedAttention(**dict(dict(total_tokens=10, num_seqs=2, hq=4, hkv=2, head_dim=64, max_chunk=8,
                                                           max_pages=3, page_size=16, device="cpu"), **kw))
    for bad in (dict(head_dim=96), dict(hq=3), dict(total_tokens=-1), dict(max_chunk=0), dict(max_pages=0), dict(page_size=20),
                dict(max_pages=1 << 27)):
        with pytest.raises(F.FlamiaError):
            new(**bad)
    att, kv = new(), F.FlamiaPagedCache(4, 16, 2, 64, device="cpu")
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)
    i32 = torch.int32
    cu, lens, table, q, k = z(3, dtype=i32), z(2, dtype=i32), z(2, 3, dtype=i32), z(10, 4, 64), z(10, 2, 64)
    with pytest.raises(F.FlamiaError, match="plan_build"):
        att.forward(kv, q, table)
    with pytest.raises(F.FlamiaError, match="FlamiaCachedAttention runs on a CUDA device"):
        att.plan_build(cu, lens)
    for bad in ((z(2, dtype=i32), lens), (cu.long(), lens), (cu, z(3, dtype=i32)), (cu, lens.long())):
        with pytest.raises(F.FlamiaError, match="want"):
            att.plan_build(*bad)
    att._planned = True
    for bad in (F.FlamiaPagedCache(4, 32, 2, 64, device="cpu"), F.FlamiaPagedCache(4, 16, 1, 64, device="cpu"),
                F.FlamiaPagedCache(4, 16, 2, 128, device="cpu")):
        with pytest.raises(F.FlamiaError, match="cache: want"):
            att.forward(bad, q, table)
    for t in (z(2, 4, dtype=i32), table.long(), z(3, 2, dtype=i32).t()):
        with pytest.raises(F.FlamiaError, match="page_table: want"):
            att.forward(kv, q, t)
    for x in (q.float(), z(9, 4, 64), z(10, 2, 64), z(4, 10, 64).transpose(0, 1)):
        with pytest.raises(F.FlamiaError, match="q: want"):
            att.forward(kv, x, table)
    for f in (lambda a, b: att.write(kv, a, b, table), lambda a, b: att.read(kv, table, a, b)):
        for a, b in ((k.float(), k), (k, z(10, 4, 64)), (k, z(2, 10, 64).transpose(0, 1))):
            with pytest.raises(F.FlamiaError, match="want"):
                f(a, b)


def test_pages_are_replaced_by_tensors_of_their_kind_only(F):
    """The calls' addresses follow an assignment; what does not fit is refused and changes nothing."""
    torch = pytest.importorskip("torch")
    for fmt, dtype, names in (("e4m3", torch.uint8, ("k", "v", "k_scales", "v_scales")), ("bf16", torch.bfloat16, ("k", "v"))):
        c = F.FlamiaPagedCache(4, 16, 2, 64, fmt, device="cpu")
        shapes = {"k": (4, 2, 16, 64), "v": (4, 2, 16, 64), "k_scales": (4, 2, 16), "v_scales": (4, 2, 16)}
        for n in names:
            old = getattr(c, n)
            odd = torch.zeros(old.numel() + 1, dtype=dtype)[1:].view(old.shape)
            for bad in (torch.zeros(shapes[n], dtype=torch.float32), torch.zeros(5, *shapes[n][1:], dtype=dtype), odd, None,
                        torch.zeros(shapes[n], dtype=dtype).transpose(0, 1).contiguous().transpose(0, 1),
                        torch.zeros(shapes[n], dtype=dtype, device="meta")):
                with pytest.raises(F.FlamiaError, match=n + ": want"):
                    setattr(c, n, bad)
                assert getattr(c, n) is old and getattr(c.view, n) == old.data_ptr()
            new = torch.ones_like(old)
            setattr(c, n, new)
            assert getattr(c, n) is new and getattr(c.view, n) == new.data_ptr() == getattr(c.ref.contents, n)
            c.k += 1                                                  # (in place: the same tensor assigned)
            assert c.view.k == c.k.data_ptr()
        if fmt == "bf16":
            c.k_scales = None
            assert c.view.k_scales is None
            with pytest.raises(F.FlamiaError, match="k_scales: there is none"):
                c.k_scales = torch.zeros(4, 2, 16, dtype=torch.uint8)


def test_a_steps_buffers_are_replaced_by_their_kind_only(F):
    torch = pytest.importorskip("torch")
    att = F.FlamiaCachedAttention(10, 2, 4, 2, 64, max_chunk=8, max_pages=3, page_size=16, device="cpu")
    for n, align in (("plan", 16), ("out", 16), ("lse", 4), ("workspace", 256)):
        old = getattr(att, n)
        bads = [old[1:].clone(), torch.zeros(old.shape, dtype=torch.float64), None]
        if old.dtype == torch.uint8:
            room = torch.zeros(old.numel() + 2 * align, dtype=torch.uint8)
            off = -room.data_ptr() % align + align // 2
            bads.append(room[off:off + old.numel()])                  # (half of the alignment that it wants)
        for bad in bads:
            with pytest.raises(F.FlamiaError, match=n + ": want"):
                setattr(att, n, bad)
            assert getattr(att, n) is old
        room = torch.zeros(old.numel() * old.element_size() + 256, dtype=torch.uint8)
        new = room[-room.data_ptr() % 256:][:old.numel() * old.element_size()].view(old.dtype).view(old.shape)
        setattr(att, n, new)
        assert getattr(att, n) is new
