"""The 8-bit prefix operators: row quantiser, int8 product, int8 K/V cache and
attention over it, against their definitions in float64.

A rounding to a type t is off by at most eps(t) / 2 relative to the value
(bf16 2^-8, fp32 2^-24); the tolerances below count those.
"""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

import flow_matching_action_pi0_b200 as fm
from flow_matching_action_pi0_b200 import build as fbuild

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
HALF_ULP = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


# ------------------------------------------------------------------ references
def quant_ref(x):
    """Rows of float64 values -> (codes, scale): the definition in include/pae.h."""
    x = np.asarray(x, np.float64)
    amax = np.abs(x).max(-1)
    s = (amax / 127.0).astype(np.float32)
    bad = ~np.isfinite(amax)
    s[~bad & (s < np.float32(2.0 ** -120))] = 0
    s[bad] = np.nan
    with np.errstate(all="ignore"):
        q = np.rint(x / s[..., None].astype(np.float64))
    q[~(s > 0)] = 0
    return q.astype(np.int8), s


def attention_ref(q, k, v, lens, causal, k_new, v_new, scale):
    """float64, one sequence and head at a time; k, v are the values the cache
    stands for.  Returns (o, weight): weight = sum p |v| / sum p, the size that
    a relative error of the probabilities acts on."""
    B, nq, Hq, d = q.shape
    G = Hq // k.shape[1]
    o, a = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    for b in range(B):
        n = max(0, min(int(lens[b]), k.shape[2]))
        for h in range(Hq):
            kk, vv = k[b, h // G, :n], v[b, h // G, :n]
            if k_new is not None:
                kk, vv = torch.cat([kk, k_new[b, :, h // G]]), torch.cat([vv, v_new[b, :, h // G]])
            for i in range(nq):
                m = n - nq + 1 + i if causal else kk.shape[0]
                if m <= 0:
                    continue
                p = torch.softmax(kk[:m] @ q[b, i, h] * scale, 0)
                o[b, i, h], a[b, i, h] = p @ vv[:m], p @ vv[:m].abs()
    return o, a


def assert_attention(got, o, a, more=0.0):
    """A probability (times the value scale) is rounded once, to fp16 or bf16,
    the output once; the scores' fp32 sums (|q k| adds to some tens over d <=
    256 terms), 16-bit query digits and the 2^-22 of exp2 move a probability by
    less than 2^-10."""
    tol = a * (2.0 ** -8 + 2.0 ** -10) + o.abs() * 2.0 ** -8 + more
    over = ((got.cpu().double() - o).abs() - tol).max()
    assert over <= 0, f"beyond the bound by {over:.3e}"


# ------------------------------------------------------------- refusals (CPU)
@pytest.fixture(scope="module")
def lib():
    fbuild.build()
    return fm.lib()


P16 = 1 << 20  # a 16-byte aligned stand-in: refused calls never follow it


def _cache(**kw):
    c = dict(k=P16, v=P16, k_scale=P16, v_scale=P16, n_slots=2, n_kv_heads=1, capacity=64, head_dim=64)
    c.update(kw)
    return fm.pae_kv8(**c)


def _query(**kw):
    q = dict(lens=P16, q=P16, out=P16, n_seq=2, n_q=1, n_q_heads=4, n_new=0, causal=0, scale=0.0)
    q.update(kw)
    s = fm.pae_kv8_query(**q)
    for name in ("q_strides", "out_strides", "k_new_strides", "v_new_strides"):
        if name not in kw:
            setattr(s, name, (256, 256, 64))
    return s


def test_quantize_rows_refusals(lib):
    ok = dict(x=P16, ldx=64, rows=2, width=64, dtype=fm.PAE_BF16, eps=0.0, codes=P16, scale=P16)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.pae_quantize_rows(a["x"], a["ldx"], a["rows"], a["width"], a["dtype"], a["eps"], a["codes"], a["scale"], None)

    for kw in (dict(x=None), dict(codes=None), dict(scale=None), dict(ldx=63), dict(rows=-1), dict(width=0),
               dict(dtype=fm.PAE_W4A16), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(x=P16 + 1)):
        assert call(**kw) == fm.PAE_ERR_ARG, kw
    assert call(rows=(1 << 30) + 1) == fm.PAE_ERR_UNSUPPORTED
    assert call(width=(1 << 30) + 1, ldx=1 << 31) == fm.PAE_ERR_UNSUPPORTED
    assert call(rows=0, x=None) == fm.PAE_OK


def test_linear_i8_refusals(lib):
    ok = dict(x=P16, xs=P16, w=P16, ws=P16, tokens=4, n=8, k=32, y=P16, ldy=8, dtype=fm.PAE_BF16)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.pae_linear_i8(a["x"], a["xs"], a["w"], a["ws"], a["tokens"], a["n"], a["k"], a["y"], a["ldy"], a["dtype"], None)

    for kw in (dict(x=None), dict(xs=None), dict(w=None), dict(ws=None), dict(y=None), dict(tokens=-1), dict(n=0),
               dict(k=0), dict(ldy=7), dict(dtype=9), dict(x=P16 + 8), dict(w=P16 + 8), dict(y=P16 + 1)):
        assert call(**kw) == fm.PAE_ERR_ARG, kw
    for kw in (dict(k=24), dict(k=131072), dict(tokens=1 << 25), dict(n=1 << 25)):
        assert call(**kw) == fm.PAE_ERR_UNSUPPORTED, kw
    assert call(tokens=0) == fm.PAE_OK


def test_kv8_refusals(lib):
    ll = ctypes.c_longlong * 2

    def io(f, cache=None, k=P16, v=P16, ks=None, vs=None, cu=P16, n_seq=2, rows=3, dtype=fm.PAE_BF16):
        return f(ctypes.byref(cache or _cache()), k, v, ks and ll(*ks), vs and ll(*vs), cu, None, n_seq, rows, dtype, None)

    for f in (lib.pae_kv8_write, lib.pae_kv8_read):
        for kw in (dict(cache=_cache(k=None)), dict(cache=_cache(n_slots=0)), dict(cache=_cache(capacity=0)),
                   dict(cache=_cache(capacity=(1 << 30) + 1)), dict(cache=_cache(v=P16 + 4)), dict(k=None), dict(k=P16 + 8),
                   dict(ks=(12, 64)), dict(vs=(-64, 64)), dict(cu=None), dict(n_seq=3), dict(n_seq=-1), dict(rows=-1),
                   dict(dtype=fm.PAE_W4A16)):
            assert io(f, **kw) == fm.PAE_ERR_ARG, kw
        assert io(f, cache=_cache(head_dim=96)) == fm.PAE_ERR_UNSUPPORTED
        assert io(f, rows=0) == fm.PAE_OK
        assert f(None, P16, P16, None, None, None, None, 1, 1, fm.PAE_BF16, None) == fm.PAE_ERR_ARG
    assert io(lib.pae_kv8_read, ks=(0, 64)) == fm.PAE_ERR_ARG  # rows that are written share a place


def test_kv8_attention_refusals(lib):
    big = 1 << 30

    def call(cache=None, ws=P16, wb=big, **kw):
        q = _query(**kw)
        return lib.pae_kv8_attention(ctypes.byref(cache or _cache()), ctypes.byref(q), ws, wb, None)

    for kw in (dict(lens=None), dict(q=None), dict(out=None), dict(n_seq=3), dict(n_seq=-1), dict(n_q=-1),
               dict(n_q_heads=0), dict(n_new=-1), dict(n_new=2), dict(scale=math.nan), dict(q=P16 + 8),
               dict(q_strides=(4, 64, 64)), dict(out_strides=(256, 256, 0)), dict(out_strides=(0, 256, 64)),
               dict(n_new=2, k_new=P16, v_new=P16, causal=1), dict(n_new=2, k_new=P16, v_new=P16 + 8)):
        assert call(**kw) == fm.PAE_ERR_ARG, kw
    assert call(cache=_cache(n_kv_heads=3), n_q_heads=4) == fm.PAE_ERR_ARG
    assert call(cache=_cache(n_slots=70000), n_seq=70000) == fm.PAE_ERR_UNSUPPORTED
    split = _cache(capacity=4096)
    need = fm.pae_kv8_workspace(split, 2, 1, 4)
    assert need > 0
    assert call(cache=split, ws=None, wb=need) == fm.PAE_ERR_ARG
    assert call(cache=split, wb=need - 1) == fm.PAE_ERR_ARG
    assert call(n_seq=0) == fm.PAE_OK and call(n_q=0) == fm.PAE_OK
    assert fm.pae_kv8_workspace(split, 0, 1, 4) == 0
    with pytest.raises(fm.PaeError):
        fm.pae_kv8_workspace(split, 3, 1, 4)


def test_wrappers_refuse_cpu_tensors_and_bad_shapes():
    x = torch.zeros(2, 32)
    with pytest.raises(ValueError):
        fm.quantize_rows(x)
    with pytest.raises(ValueError):
        fm.quantize_rows(x.to(torch.float16))
    with pytest.raises(ValueError):
        fm.quantize_rows(x[0])
    with pytest.raises(ValueError):
        fm.linear_i8(x.to(torch.int8), torch.ones(2), x.to(torch.int8), torch.ones(2))
    with pytest.raises(ValueError):
        fm.linear_i8(x.to(torch.int8), torch.ones(2), torch.zeros(4, 16, dtype=torch.int8), torch.ones(4))
    # sizes that do not fit the library's integers (views of one element)
    huge = torch.zeros(1, 1).expand((1 << 32) + 2, 1)
    with pytest.raises(ValueError, match="2\\^30"):
        fm.quantize_rows(huge)
    with pytest.raises(ValueError, match="2\\^30"):
        fm.quantize_rows(huge.t())
    codes = torch.zeros(1, 1, dtype=torch.int8).expand((1 << 32) + 2, 16)
    with pytest.raises(ValueError, match="2\\^30"):
        fm.linear_i8(codes, torch.ones(1), codes[:4], torch.ones(4))
    with pytest.raises(ValueError):
        fm.quantize_rows(x, 1e-60)  # 0 as a float


def test_a_cache_in_host_memory_is_refused():
    c = fm.KvCacheInt8(1, 1, 8, 64, device="cpu")
    row = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    n = torch.zeros(1, dtype=torch.int32)
    for call in (lambda: c.write(row, row), lambda: c.read(None, None, 1), lambda: c.attend(row[None], n),
                 lambda: c.write(row, row, start=n)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


@pytest.mark.gpu
def test_wrappers_refuse_what_does_not_fit():
    """Wrong types, shapes, layouts, devices and plans, each named by its error
    and leaving the operators usable."""
    bf = dict(device="cuda", dtype=torch.bfloat16)
    x, w = torch.ones(4, 64, **bf), torch.ones(8, 64, device="cuda", dtype=torch.int8)
    q, s = fm.quantize_rows(x)
    ws = torch.ones(8, device="cuda")
    c = fm.KvCacheInt8(2, 2, 64, 64)
    rows = torch.ones(3, 2, 64, **bf)
    n = torch.full((2,), 3, dtype=torch.int32, device="cuda")
    qs, new = torch.ones(2, 20, 4, 64, **bf), torch.ones(2, 5, 2, 64, **bf)
    plan = c.plan(2, 20, 4)
    cu = torch.tensor([0, 1, 3], dtype=torch.int32, device="cuda")
    bad = [lambda: fm.quantize_rows(x.half()), lambda: fm.quantize_rows(x[0]), lambda: fm.quantize_rows(x.t()[:, :2]),
           lambda: fm.quantize_rows(x[:, :0]), lambda: fm.quantize_rows(x, 0.0), lambda: fm.quantize_rows(x, -1.0),
           lambda: fm.linear_i8(x, s, w, ws), lambda: fm.linear_i8(q, s[:3], w, ws), lambda: fm.linear_i8(q, s, w, ws.double()),
           lambda: fm.linear_i8(q, s, w.t(), ws), lambda: fm.linear_i8(q.cpu(), s, w, ws), lambda: fm.linear_i8(q, s, w, ws, torch.float16),
           lambda: fm.linear_i8(q, s, w, ws, out=torch.empty(4, 9, **bf)), lambda: fm.linear_i8(q, s, w, ws, out=torch.empty(8, 4, **bf).t()),
           lambda: c.write(rows, rows[:2]), lambda: c.write(rows, rows.float()), lambda: c.write(rows[0], rows[0]),
           lambda: c.write(rows[:, :1], rows[:, :1]), lambda: c.write(rows, rows, cu.long()), lambda: c.write(rows, rows, cu[:0]),
           lambda: c.write(rows, rows, cu.cpu()), lambda: c.write(rows, rows, cu, n[:1]), lambda: c.read(cu, None, -1),
           lambda: c.read(cu, None, 3, torch.float16), lambda: c.attend(qs[0], n), lambda: c.attend(qs.float(), n),
           lambda: c.attend(qs, n[:1]), lambda: c.attend(qs, n.cpu()), lambda: c.attend(qs, n, scale=0.0),
           lambda: c.attend(qs, n, k_new=new), lambda: c.attend(qs, n, k_new=new, v_new=new[:, :4]),
           lambda: c.attend(qs, n, k_new=new[:1], v_new=new[:1]), lambda: c.attend(qs, n, out=qs[:, :1]),
           lambda: c.attend(qs, n, out=qs.float()), lambda: c.attend(qs, n, k_new=new, v_new=new, plan=plan),
           lambda: c.attend(qs[:, :, :, :32], n), lambda: c.attend(qs[:, :19], n, plan=plan)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was accepted")
    for call in (lambda: fm.quantize_rows([1.0]), lambda: fm.linear_i8(q, s, w, None), lambda: c.write(rows, None),
                 lambda: fm.quantize_rows(x, "eps"), lambda: c.read(cu, None, "rows"), lambda: c.read(cu, None, 3, "bf16")):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: c.attend(qs, n, causal=True, k_new=new, v_new=new), lambda: c.attend(qs, n, scale=float("nan")),
                 lambda: fm.linear_i8(q[:, :24].contiguous(), s, w[:, :24].contiguous(), ws)):
        with pytest.raises(fm.PaeError):
            call()
    c.write(rows, rows, cu)
    assert bool((c.attend(qs, torch.tensor([1, 2], dtype=torch.int32, device="cuda"), plan=plan) == 1).all())
    fm.pae_int8_sync()


@pytest.mark.gpu
def test_cache_refuses_sizes_past_its_integers():
    c = fm.KvCacheInt8(2, 1, 64, 64)
    row = torch.zeros(1, 1, 64, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="2\\^30"):
        c.write(row.expand((1 << 32) + 2, 1, 64), row.expand((1 << 32) + 2, 1, 64))
    with pytest.raises(ValueError, match="2\\^30"):
        c.read(None, None, (1 << 32) + 2)
    with pytest.raises(ValueError, match="slots"):
        c.write(row, row, torch.zeros(4, dtype=torch.int32, device="cuda"))
    many = row[None].expand(2, (1 << 32) + 2, 1, 64)
    with pytest.raises(ValueError, match="2\\^30"):
        c.attend(row[None].expand(2, 1, 1, 64), torch.zeros(2, dtype=torch.int32, device="cuda"), k_new=many, v_new=many)


# -------------------------------------------------------------- row quantiser
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,width", [(1, 1), (3, 7), (2, 1024), (5, 2047), (1, 4096), (1300, 512), (1201, 1024), (8200, 512), (4100, 1000), (2100, 2048), (300, 256), (300, 496),
                                        (1190, 2048), (7, 16384), (3, 20000), (1500, 40)])
def test_quantize_rows(rows, width, dtype):
    g = torch.Generator().manual_seed(rows * 31 + width)
    x = (torch.randn(rows, width, generator=g) * torch.exp(torch.randn(rows, 1, generator=g) * 3)).to(DT[dtype])
    q, s = fm.quantize_rows(x.cuda())
    rq, rs = quant_ref(x.double().numpy())
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(q.cpu().numpy(), rq)
    q2, s2 = fm.quantize_rows(x.cuda(), rms_eps=1e-6)
    assert torch.equal(q2, q)
    want = rs.astype(np.float64) / np.sqrt((x.double().numpy() ** 2).mean(-1) + 1e-6)
    # at most 80 squares added in a row per thread, a tree over the threads and
    # rsqrt: under 128 roundings of 2^-24, halved by the root
    assert np.all(np.abs(s2.cpu().numpy() - want) <= want * 2.0 ** -17)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("width", [24, 1024, 1023])
def test_quantize_rows_edges(width, dtype):
    """Zeros, tiny and huge rows, NaN, infinities, halves, a row stride."""
    t = DT[dtype]
    rows = torch.zeros(10, width, dtype=torch.float64)
    g = torch.Generator().manual_seed(width)
    base = torch.randn(width, generator=g).double()
    rows[1] = base * 2.0 ** -125
    rows[2] = base * 2.0 ** -110
    rows[3] = base / base.abs().max() * 3e38
    rows[4] = base
    rows[4, 3] = math.nan
    rows[5] = base
    rows[5, 5] = -math.inf
    rows[6] = torch.arange(width).double() % 128 - 0.5  # scale 1 when the maximum is 127: exact halves
    rows[6, 0] = 127.0
    rows[6] = rows[6].clamp(-127, 127)
    rows[7] = (torch.arange(width).double() % 255 - 127) * 0.5
    rows[7, 0] = 127.0
    rows[8, 0] = -1.0
    rows[9] = base.abs()
    x = rows.to(t)
    wide = torch.full((10, width + 8), math.nan, dtype=t, device="cuda")
    wide[:, :width] = x.cuda()
    q, s = fm.quantize_rows(wide[:, :width])
    rq, rs = quant_ref(x.double().numpy())
    assert np.array_equal(s.cpu().numpy(), rs, equal_nan=True)
    assert np.array_equal(q.cpu().numpy(), rq)
    assert np.isnan(rs[4]) and np.isnan(rs[5]) and rs[0] == 0 and rs[1] == 0 and rs[2] > 0
    q2, s2 = fm.quantize_rows(wide[:, :width], rms_eps=1e-6)
    assert torch.equal(q2, q)
    fin = [0, 1, 2, 3, 6, 7, 8, 9]
    want = rs[fin].astype(np.float64) / np.sqrt((x.double().numpy()[fin] ** 2).mean(-1) + 1e-6)
    assert np.all(np.abs(s2.cpu().numpy()[fin] - want) <= want * 2.0 ** -17)
    assert bool(torch.isnan(s2[4])) and bool(torch.isnan(s2[5]))


# ---------------------------------------------------------------- int8 product
def _linear_ref(x, xs, w, ws):
    return (x.double() @ w.double().t()) * xs.double()[:, None] * ws.double()[None, :]


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("tokens,n,k", [(1, 1, 16), (1, 2560, 1024), (2, 130, 144), (16, 129, 2048), (17, 512, 4096),
                                        (50, 8192, 1024), (64, 1000, 80), (65, 7, 32), (128, 128, 128), (129, 513, 1040),
                                        (968, 512, 2048), (300, 2300, 272), (1601, 1024, 512), (4000, 40, 64),
                                        (33, 96, 16384), (100, 33, 16400)])
def test_linear_i8(tokens, n, k, out):
    g = torch.Generator(device="cuda").manual_seed(tokens + 7 * n + 13 * k)
    x = torch.randint(-128, 128, (tokens, k), generator=g, device="cuda", dtype=torch.int8)
    w = torch.randint(-128, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
    xs = torch.rand(tokens, generator=g, device="cuda") + 0.01
    ws = torch.rand(n, generator=g, device="cuda") + 0.01
    y = fm.linear_i8(x, xs, w, ws, out_dtype=DT[out])
    ref = _linear_ref(x, xs, w, ws)
    # the sum is exact; its conversion, two products and the output round
    tol = ref.abs() * (3 * 2.0 ** -24 + HALF_ULP[out])
    assert bool(((y.double() - ref).abs() <= tol).all())
    # a strided output: columns and rows around it stay as they were
    big = torch.full((tokens + 2, n + 5), 7.0, dtype=DT[out], device="cuda")
    fm.linear_i8(x, xs, w, ws, out=big[1:-1, 2:2 + n])
    assert torch.equal(big[1:-1, 2:2 + n], y)
    big[1:-1, 2:2 + n] = 7.0
    assert bool((big == 7.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("tokens", [3, 200])
def test_linear_i8_sums_reach_32_bits(tokens):
    """All codes at their extremes at the largest k: |sum| = 2^14 k < 2^31."""
    k = 131056
    x = torch.full((tokens, k), -128, dtype=torch.int8, device="cuda")
    w = torch.full((5, k), -128, dtype=torch.int8, device="cuda")
    w[1] = 127
    w[2, ::2] = 0
    y = fm.linear_i8(x, torch.ones(tokens, device="cuda"), w, torch.ones(5, device="cuda"), out_dtype=torch.float32)
    want = torch.tensor([128 * 128 * k, -128 * 127 * k, 128 * 64 * k, 128 * 128 * k, 128 * 128 * k], dtype=torch.float64)
    assert torch.equal(y.cpu(), want.float().expand(tokens, 5))


@pytest.mark.gpu
@pytest.mark.parametrize("tokens", [3, 200, 600])
def test_linear_i8_small_scales(tokens):
    """Scales whose product is subnormal (1.37 2^-80, 1.61 2^-60) and sums that
    bring the result back: two fp32 products of a whole number below 2^24 with
    normal results are off by half a step each, 2^-23 in all (and 2^-47)."""
    k, n = 512, 300
    g = torch.Generator().manual_seed(tokens)
    x, w = torch.randint(100, 128, (tokens, k), generator=g), torch.randint(100, 128, (n, k), generator=g)
    sx, sw = torch.full((tokens,), 1.37 * 2.0 ** -80), torch.full((n,), 1.61 * 2.0 ** -60)
    want = (x.double() @ w.double().t()) * sx.double()[:, None] * sw.double()
    assert float((x.double() @ w.double().t()).max()) < 2 ** 24
    got = fm.linear_i8(x.to(torch.int8).cuda(), sx.cuda(), w.to(torch.int8).cuda(), sw.cuda(), out_dtype=torch.float32)
    assert bool(((got.cpu().double() - want).abs() <= want * (2.0 ** -23 + 2.0 ** -46)).all())


# ------------------------------------------------------------------- K/V cache
def _cu(lens):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("hk,d", [(1, 256), (3, 128), (2, 64)])
@pytest.mark.parametrize("lens,start", [([1], [0]), ([0, 5, 0, 130, 1], [3, 0, 9, 70, 199]), ([1] * 33, list(range(33))),
                                        ([40, 260], [180, 0]), ([3, 2], [-2, 10])])
def test_kv8_write_and_read(lens, start, hk, d, dtype):
    cap, T, pad = 200, sum(lens), 3
    g = torch.Generator().manual_seed(T + d)
    # K and V are slices of one projection, with rows of no sequence behind
    qkv = torch.randn(T + pad, 4 * hk, d, generator=g).to(DT[dtype]).cuda()
    k, v = qkv[:, hk:2 * hk], qkv[:, 3 * hk:]
    c = fm.KvCacheInt8(len(lens) + 1, hk, cap, d)
    for t in (c.k, c.v, c.k_scale, c.v_scale):
        t.fill_(77)
    st = torch.tensor(start, dtype=torch.int32, device="cuda")
    c.write(k, v, _cu(lens), st)
    rk, rv = c.read(_cu(lens), st, T + pad, dtype=DT[dtype])
    for rows, codes, scales, back in ((k, c.k, c.k_scale, rk), (v, c.v, c.v_scale, rv)):
        wq, ws = np.full(c.shape, 77, np.int8), np.full(c.shape[:3], 77, np.float32)
        q, s = quant_ref(rows.double().cpu().numpy())
        want = np.zeros((T + pad, hk, d))
        t = 0
        for b, n in enumerate(lens):
            for i in range(n):
                at = start[b] + i
                if 0 <= at < cap:
                    wq[b, :, at], ws[b, :, at] = q[t], s[t]
                    want[t] = q[t].astype(np.float64) * s[t][:, None]
                t += 1
        assert np.array_equal(codes.cpu().numpy(), wq)
        assert np.array_equal(scales.cpu().numpy(), ws)
        # code x scale rounds once in fp32, once to the output type
        tol = np.abs(want) * (2.0 ** -24 + HALF_ULP[dtype])
        assert np.all(np.abs(back.double().cpu().numpy() - want) <= tol)


@pytest.mark.gpu
def test_kv8_rows_with_nan_and_without_sequences():
    c = fm.KvCacheInt8(1, 1, 8, 64)
    k = torch.randn(3, 1, 64, device="cuda")
    k[1, 0, 5] = math.nan
    c.write(k, k)
    rk, _ = c.read(None, None, 3, dtype=torch.float32)
    assert bool(torch.isnan(rk[1]).all()) and bool(torch.isfinite(rk[[0, 2]]).all())
    c.write(k[:0], k[:0])
    before = c.k.clone()
    c.write(k, k, torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert torch.equal(before, c.k)


# ------------------------------------------------------------------- attention
def _filled(slots, hk, cap, d, g):
    """A cache written over all of its positions, and the values it stands for."""
    c = fm.KvCacheInt8(slots, hk, cap, d)
    rows = [torch.randn(slots * cap, hk, d, generator=g).to(torch.bfloat16).cuda() for _ in range(2)]
    c.write(*rows, torch.arange(0, slots * cap + 1, cap, dtype=torch.int32, device="cuda"))
    vals = [(q.double() * s.double().unsqueeze(-1)).cpu() for q, s in ((c.k, c.k_scale), (c.v, c.v_scale))]
    return c, vals


CASES = [  # lens, capacity, kv heads, group, queries, fresh, causal, d
    ([968], 968, 1, 8, 1, 0, False, 256), ([1, 0, 130], 130, 1, 8, 1, 0, False, 256), ([700, 64], 1000, 2, 1, 1, 0, False, 64),
    ([333, 17, 1024], 1024, 2, 4, 2, 0, False, 128), ([5, 300], 300, 1, 16, 1, 0, True, 64), ([1, 2, 9], 300, 1, 3, 4, 0, True, 256),
    ([260, 0, 64], 260, 1, 8, 50, 50, False, 256), ([100], 100, 1, 8, 16, 0, False, 64), ([130, 1], 130, 2, 4, 33, 7, False, 128),
    ([0, 0], 64, 1, 2, 20, 0, False, 64), ([0, 5], 64, 1, 1, 1, 1, False, 256), ([64, 63, 65], 70, 1, 4, 1, 64, False, 64),
    ([200, 100, 20], 200, 1, 8, 40, 0, True, 256), ([300], 300, 3, 5, 31, 0, True, 128), ([129], 4096, 1, 8, 30, 0, True, 64),
    ([4096, 1000], 4096, 1, 2, 1, 0, False, 64), ([600], 600, 1, 8, 20, 130, False, 256), ([17], 64, 1, 17, 1, 0, False, 128),
    ([1500], 1500, 1, 1, 9, 0, True, 256), ([65, 1], 66, 4, 1, 130, 0, True, 64),
    # on both sides of the choice between row groups and tiles
    ([0, 64, 3] * 20, 64, 1, 2, 20, 0, False, 64), ([100, 1, 0] * 8, 100, 1, 8, 16, 0, False, 64), ([0, 40] * 12, 66, 4, 1, 130, 0, True, 64),
    ([4096], 4096, 1, 8, 20, 0, False, 128), ([4096], 4096, 1, 8, 25, 0, True, 128), ([968] * 12, 968, 1, 8, 2, 0, False, 256),
    ([968] * 12, 968, 1, 8, 3, 0, True, 256), ([20000, 1], 20000, 1, 8, 1, 0, False, 128),
]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,cap,hk,group,nq,fresh,causal,d", CASES)
def test_kv8_attention(lens, cap, hk, group, nq, fresh, causal, d):
    g = torch.Generator().manual_seed(sum(lens) + cap + nq)
    B, hq = len(lens), hk * group
    c, (k, v) = _filled(B + 1, hk, cap, d, g)
    q = torch.randn(B, nq, hq, d, generator=g).to(torch.bfloat16)
    new = [torch.randn(B, fresh, hk, d, generator=g).to(torch.bfloat16) for _ in range(2)] if fresh else [None, None]
    o, a = attention_ref(q.double(), k, v, lens, causal, *[None if t is None else t.double() for t in new], d ** -0.5)
    dev = [None if t is None else t.cuda() for t in new]
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = c.attend(q.cuda(), n, causal=causal, k_new=dev[0], v_new=dev[1])
    assert_attention(got, o, a)
    empty = (a == 0).all(-1)
    assert bool((got.cpu()[empty] == 0).all())
    # positions no query may see: NaN scales there change nothing
    for b in range(B + 1):
        for t in (c.k_scale, c.v_scale):
            t[b, :, (lens[b] if b < B else 0):] = math.nan
    assert torch.equal(c.attend(q.cuda(), n, causal=causal, k_new=dev[0], v_new=dev[1]), got)


@pytest.mark.gpu
@pytest.mark.parametrize("nq,group", [(4, 2), (40, 4), (130, 8)])
def test_kv8_attention_causal_masks_nan_rows(nq, group):
    """A NaN row at position p reaches exactly the queries that may see p."""
    g = torch.Generator().manual_seed(nq)
    c, _ = _filled(1, 1, 300, 128, g)
    n = torch.tensor([300], dtype=torch.int32, device="cuda")
    q = torch.randn(1, nq, group, 128, generator=g).to(torch.bfloat16).cuda()
    clean = c.attend(q, n, causal=True)
    at = 300 - nq + 2  # seen by queries 2 and later
    for t in (c.k_scale, c.v_scale):
        keep = t[0, 0, at].clone()
        t[0, 0, at] = math.nan
        got = c.attend(q, n, causal=True)
        assert bool(torch.isnan(got[:, 2:]).all())
        assert torch.equal(got[:, :2], clean[:, :2])
        t[0, 0, at] = keep


@pytest.mark.gpu
@pytest.mark.parametrize("nq,fresh,causal", [(1, 0, False), (4, 0, True), (40, 0, False), (40, 33, False), (60, 0, True), (160, 0, False)])
def test_kv8_attention_rows_of_very_different_size(nq, fresh, causal):
    """Value rows from 2^-60 to 2^60 side by side (a row's weight decides, not
    its neighbours' size), zero rows, and huge rows where a query may not look."""
    g = torch.Generator().manual_seed(nq + fresh)
    B, cap, d, group = 2, 400, 128, 4
    c = fm.KvCacheInt8(B, 1, cap, d)
    k = torch.randn(B * cap, 1, d, generator=g)
    size = torch.exp2(torch.randint(-60, 61, (B * cap, 1, 1), generator=g).float())
    size[torch.rand(B * cap, 1, 1, generator=g) < 0.1] = 0.0
    v = torch.randn(B * cap, 1, d, generator=g) * size
    v[cap:] = torch.randn(cap, 1, d, generator=g)   # the second sequence: unit rows,
    lens = [cap, 300]
    v[cap + 300 - 3:cap + 300] *= 1e30               # huge ones at its last positions
    c.write(k.to(torch.bfloat16).cuda(), v.to(torch.bfloat16).cuda(), torch.tensor([0, cap, 2 * cap], dtype=torch.int32, device="cuda"))
    vals = [(t.double() * s.double().unsqueeze(-1)).cpu() for t, s in ((c.k, c.k_scale), (c.v, c.v_scale))]
    q = torch.randn(B, nq, group, d, generator=g).to(torch.bfloat16)
    new = [torch.randn(B, fresh, 1, d, generator=g).to(torch.bfloat16) for _ in range(2)] if fresh else [None, None]
    o, a = attention_ref(q.double(), *vals, lens, causal, *[None if t is None else t.double() for t in new], d ** -0.5)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = c.attend(q.cuda(), n, causal=causal, k_new=None if not fresh else new[0].cuda(), v_new=None if not fresh else new[1].cuda())
    # fp16 holds c = p vs / 2^ref in steps of 2^-24 at the bottom, an error of 2^-25
    # at most, against a largest c of 1 at least; a channel adds cap + fresh of
    # them, times codes up to 127.  In units of the output that is (cap + fresh)
    # 2^-25 (127 max p vs), and 127 p vs is the largest |p v| of a key's channels,
    # which is not above the row's largest a.
    assert_attention(got, o, a, (cap + fresh) * 2.0 ** -25 * a.amax(-1, keepdim=True))
    if causal:  # the queries before the huge rows see unit rows alone
        assert float(got[1, :nq - 3].abs().max()) < 10


@pytest.mark.gpu
@pytest.mark.parametrize("nq,fresh", [(1, 0), (4, 0), (40, 0), (40, 33), (160, 0)])
def test_kv8_attention_weight_on_empty_values(nq, fresh):
    """A key that takes nearly all the weight and has no value, or values of
    2^-90: what the others contribute keeps its precision."""
    g = torch.Generator().manual_seed(nq + fresh)
    B, cap, d, group = 2, 300, 64, 4
    c = fm.KvCacheInt8(B, 1, cap, d)
    k = torch.randn(B * cap, 1, d, generator=g)
    v = torch.randn(B * cap, 1, d, generator=g)
    q = torch.randn(B, nq, group, d, generator=g)
    q[..., 0] = 8.0
    for b in range(B):
        for at in (5, 130):  # score about 8 * 20 / 8 = 20 above the others'
            k[b * cap + at] = 0.0
            k[b * cap + at, 0, 0] = 20.0
            v[b * cap + at] *= 0.0 if b == 0 else 2.0 ** -90
    c.write(k.to(torch.bfloat16).cuda(), v.to(torch.bfloat16).cuda(), torch.tensor([0, cap, 2 * cap], dtype=torch.int32, device="cuda"))
    vals = [(t.double() * s.double().unsqueeze(-1)).cpu() for t, s in ((c.k, c.k_scale), (c.v, c.v_scale))]
    q = q.to(torch.bfloat16)
    new = [torch.randn(B, fresh, 1, d, generator=g).to(torch.bfloat16) for _ in range(2)] if fresh else [None, None]
    o, a = attention_ref(q.double(), *vals, [cap] * B, False, *[None if t is None else t.double() for t in new], d ** -0.5)
    n = torch.full((B,), cap, dtype=torch.int32, device="cuda")
    got = c.attend(q.cuda(), n, k_new=None if not fresh else new[0].cuda(), v_new=None if not fresh else new[1].cuda())
    assert_attention(got, o, a)


@pytest.mark.gpu
@pytest.mark.parametrize("nq,fresh,cap", [(1, 0, 128), (1, 0, 4000), (50, 50, 200), (50, 50, 968)])
def test_kv8_attention_strides_scale_in_place_and_plan(nq, fresh, cap):
    g = torch.Generator().manual_seed(cap)
    B, hk, group, d = 2, 2, 4, 128
    c, (k, v) = _filled(B, hk, cap, d, g)
    lens = [cap, cap // 3]
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    # q, k_new, v_new out of one fused projection; out head-major
    fused = torch.randn(B, max(nq, fresh, 1), hk * group + 2 * hk, d, generator=g).to(torch.bfloat16).cuda()
    q, kn, vn = fused[:, :nq, :hk * group], fused[:, :fresh, hk * group:hk * group + hk], fused[:, :fresh, hk * group + hk:]
    if not fresh:
        kn = vn = None
    o, a = attention_ref(q.cpu().double(), k, v, lens, False, *[None if t is None else t.cpu().double() for t in (kn, vn)], 0.3)
    out = torch.full((B, hk * group, nq + 1, d), 5.0, dtype=torch.bfloat16, device="cuda")
    plan = c.plan(B, nq, hk * group, fresh=fresh)
    if plan.workspace is not None:
        plan.workspace.fill_(0xFF)  # NaN patterns: its contents carry nothing
    c.attend(q, n, k_new=kn, v_new=vn, scale=0.3, out=out[:, :, :nq].transpose(1, 2), plan=plan)
    got = out[:, :, :nq].transpose(1, 2)
    assert_attention(got, o, a)
    assert bool((out[:, :, nq] == 5.0).all())
    inplace = q.clone()
    c.attend(inplace, n, k_new=kn, v_new=vn, scale=0.3, out=inplace, plan=plan)
    assert torch.equal(inplace, got)
    with pytest.raises(ValueError):
        c.attend(q[:1], n[:1], plan=plan)


@pytest.mark.gpu
def test_kv8_offsets_past_32_bits():
    """A cache of more than 2^32 bytes per operand: its last slot is exact."""
    slots, cap, d = 17, 1 << 20, 256
    c = fm.KvCacheInt8(slots, 1, cap, d)
    assert c.k.numel() > 2 ** 32
    g = torch.Generator().manual_seed(5)
    rows = [torch.randn(96, 1, d, generator=g).to(torch.bfloat16).cuda() for _ in range(2)]
    cu = torch.zeros(slots + 1, dtype=torch.int32, device="cuda")
    cu[-1] = 96
    st = torch.full((slots,), cap - 96, dtype=torch.int32, device="cuda")
    c.write(*rows, cu, st)
    rk, rv = c.read(cu, st, 96, dtype=torch.float32)
    for r, x, s in ((rk, rows[0], c.k_scale), (rv, rows[1], c.v_scale)):
        q, sc = quant_ref(x.double().cpu().numpy())
        assert np.array_equal(s[-1, :, cap - 96:].cpu().numpy().T, sc)
        assert np.all(np.abs(r.double().cpu().numpy() - q * sc[..., None].astype(np.float64)) <= np.abs(q * sc[..., None]) * 2.0 ** -24)
    # zero keys and values elsewhere: 96 rows among 2^20 with logit 0
    lens = torch.zeros(slots, dtype=torch.int32, device="cuda")
    lens[-1] = cap
    for nq in (1, 20):
        q = torch.randn(slots, nq, 8, d, generator=g).to(torch.bfloat16).cuda()
        got = c.attend(q, lens)
        kk, vv = [t.double() for t in (rk[:, 0], rv[:, 0])]
        e = torch.exp(torch.einsum("qhd,kd->qhk", q[-1].double(), kk) / 16)
        want = torch.einsum("qhk,kd->qhd", e, vv) / (e.sum(-1, keepdim=True) + cap - 96)
        weight = torch.einsum("qhk,kd->qhd", e, vv.abs()) / (e.sum(-1, keepdim=True) + cap - 96)
        assert_attention(got[-1], want.cpu(), weight.cpu())
        assert bool((got[:-1] == 0).all())


# -------------------------------------------------------------------- together
def _pipeline(h, wq, ws, c, cu, q, lens):
    x, s = fm.quantize_rows(h, rms_eps=1e-6)
    kv = fm.linear_i8(x, s, wq, ws)
    d = c.shape[3]
    c.write(kv[:, :d].unflatten(1, (1, d)), kv[:, d:].unflatten(1, (1, d)), cu)
    return c.attend(q, lens), kv


@pytest.mark.gpu
def test_prefix_in_8_bits_end_to_end():
    """Hidden states -> RMSNorm and product -> cache -> attention, as a prefix
    goes through them: eagerly, on a side stream, captured and replayed."""
    g = torch.Generator().manual_seed(1)
    lens, width, d, nq = [300, 129], 512, 256, 8
    h = torch.randn(sum(lens), width, generator=g).to(torch.bfloat16).cuda()
    wq, ws = fm.quantize_rows((0.02 * torch.randn(2 * d, width, generator=g)).cuda())
    q = torch.randn(2, nq, 8, d, generator=g).to(torch.bfloat16).cuda()
    n, cu = torch.tensor(lens, dtype=torch.int32, device="cuda"), _cu(lens)
    c = fm.KvCacheInt8(2, 1, 400, d)
    got, kv = _pipeline(h, wq, ws, c, cu, q, n)
    x = h.double().cpu()
    xq, xs = quant_ref(x.numpy())
    # whole-number sums first (a sum may be exactly zero), then the scales
    sums = torch.from_numpy(xq.astype(np.float64)) @ wq.double().cpu().t()
    norm = torch.from_numpy(xs.astype(np.float64)) / torch.sqrt((x ** 2).mean(-1) + 1e-6)
    ref = sums * norm[:, None] * ws.double().cpu()[None, :]
    # 2^-17 of the norm's scale, the product's roundings, bf16
    assert bool(((kv.cpu().double() - ref).abs() <= ref.abs() * (2.0 ** -17 + 2.0 ** -22 + 2.0 ** -8)).all())
    vals = [(t.double() * s.double().unsqueeze(-1)).cpu() for t, s in ((c.k, c.k_scale), (c.v, c.v_scale))]
    assert_attention(got, *attention_ref(q.cpu().double(), *vals, lens, False, None, None, d ** -0.5))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again, _ = _pipeline(h, wq, ws, c, cu, q, n)
    side.synchronize()
    assert torch.equal(again, got)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured, _ = _pipeline(h, wq, ws, c, cu, q, n)
    h2 = torch.randn(sum(lens), width, generator=g).to(torch.bfloat16).cuda()
    h.copy_(h2)
    for t in (c.k, c.v, c.k_scale, c.v_scale):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    fresh = fm.KvCacheInt8(2, 1, 400, d)
    want, _ = _pipeline(h2, wq, ws, fresh, cu, q, n)
    assert torch.equal(captured, want)
    fm.pae_int8_sync()


@pytest.mark.gpu
def test_two_streams_with_their_own_plans():
    g = torch.Generator().manual_seed(3)
    c, _ = _filled(2, 1, 3000, 256, g)
    n = torch.tensor([3000, 1500], dtype=torch.int32, device="cuda")
    qs = [torch.randn(2, m, 8, 256, generator=g).to(torch.bfloat16).cuda() for m in (1, 30)]
    want = [c.attend(q, n) for q in qs]
    streams, plans = [torch.cuda.Stream() for _ in qs], [c.plan(2, q.shape[1], 8) for q in qs]
    outs = [torch.empty_like(q) for q in qs]
    torch.cuda.synchronize()
    for _ in range(20):
        for q, s, p, o in zip(qs, streams, plans, outs):
            with torch.cuda.stream(s):
                c.attend(q, n, plan=p, out=o)
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert torch.equal(w, o)


CAPTURE_FIRST = """
import torch
import flow_matching_action_pi0_b200 as fm
torch.cuda.set_device(0)
fm.pae_int8_init()
x = torch.linspace(-1, 1, 70 * 128, device="cuda").view(70, 128).bfloat16()
w, ws = torch.ones(256, 128, dtype=torch.int8, device="cuda"), torch.ones(256, device="cuda")
cache = fm.KvCacheInt8(1, 1, 100, 128)
n = torch.tensor([70], dtype=torch.int32, device="cuda")
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    q, s = fm.quantize_rows(x, 1e-6)
    y = fm.linear_i8(q, s, w, ws)
    cache.write(y[:, None, :128], y[:, None, 128:])
    one, many = cache.attend(x[None, :1, None], n), cache.attend(x[None, :, None], n)
    back = cache.read(None, None, 70)
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in (q, s, y, one, many, *back)]
q, s = fm.quantize_rows(x, 1e-6)
y = fm.linear_i8(q, s, w, ws)
cache.write(y[:, None, :128], y[:, None, 128:])
want = [q, s, y, cache.attend(x[None, :1, None], n), cache.attend(x[None, :, None], n), *cache.read(None, None, 70)]
assert all(torch.equal(a, b) for a, b in zip(got, want))
fm.pae_int8_sync()
print("captured")
"""


@pytest.mark.gpu
def test_a_capture_may_hold_the_first_calls():
    """After pae_int8_init every operator may run for the first time inside a capture."""
    import subprocess
    import sys
    r = subprocess.run([sys.executable, "-c", CAPTURE_FIRST], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
