"""The 8-bit prefix operators where they are easily wrong: values of zero, long
tails of small weights, queries of wide range, scales at the end of fp32, wide
rows, products of several tiles per SM, errors that were left pending.

Tolerances count roundings: one to a type t is off by at most eps(t) / 2 relative
to the value (bf16 2^-8, fp16 2^-11, fp32 2^-24).
"""
import ctypes
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import flow_matching_action_pi0_b200 as fm
from flow_matching_action_pi0_b200 import build as fbuild
from tests.test_abi import _cfg, _create_status
from tests.test_int8_ops import DT, HALF_ULP, assert_attention, attention_ref, quant_ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _put(c, k_codes, k_scale, v_codes, v_scale):
    """Fill a cache with codes [slots, heads, cap, d] and scales; the values it stands for, float64."""
    for t, x in ((c.k, k_codes), (c.v, v_codes), (c.k_scale, k_scale), (c.v_scale, v_scale)):
        t.copy_(x)
    return [(q.double() * s.double().unsqueeze(-1)).cpu() for q, s in ((c.k, c.k_scale), (c.v, c.v_scale))]


def _lens(*n):
    return torch.tensor(n, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------ values of zero
@pytest.mark.gpu
@pytest.mark.parametrize("nq,cap,zeros,causal", [
    (1, 100, 100, False), (1, 3000, 3000, False), (600, 100, 100, False), (600, 100, 100, True),  # row groups; tiles, one part
    (200, 600, 600, False), (200, 600, 600, True),                                                # tiles, several parts
    (200, 600, 75, False), (200, 600, 525, False), (1, 3000, 640, False),                         # a part of zeros beside others
    (40, 100, 70, True), (600, 700, 150, True)])                                                  # the first queries see zeros alone
def test_values_of_zero_under_low_scores(nq, cap, zeros, causal):
    """All scores near -163 in log2: keys whose values are zero contribute zero,
    however small the row's weight is in absolute terms."""
    d, group = 128, 4
    g = torch.Generator().manual_seed(nq + cap + zeros)
    c = fm.KvCacheInt8(1, 1, cap, d)
    vs = torch.rand(1, 1, cap, generator=g) * 0.01 + 0.01
    vs[..., :zeros] = 0.0
    vc = torch.randint(-127, 128, (1, 1, cap, d), generator=g, dtype=torch.int8)
    vc[..., :zeros, :] = 0
    kc = torch.randint(90, 110, (1, 1, cap, d), generator=g, dtype=torch.int8)
    k, v = _put(c, kc, torch.full((1, 1, cap), 0.1), vc, vs)
    q = -torch.ones(1, nq, group, d, dtype=torch.bfloat16)
    o, a = attention_ref(q.double(), k, v, [cap], causal, None, None, d ** -0.5)
    got = c.attend(q.cuda(), _lens(cap), causal=causal)
    assert bool(torch.isfinite(got).all())
    assert_attention(got, o, a)
    assert bool((got.cpu()[a == 0] == 0).all())
    # a NaN value scale still shows
    c.v_scale[0, 0, 0] = math.nan
    sees = slice(max(0, nq - cap) if causal else 0, nq)
    assert bool(torch.isnan(c.attend(q.cuda(), _lens(cap), causal=causal)[:, sees]).all())


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [2.0 ** 127, 2.0 ** 126, 2.0 ** 100, 2.0 ** -100, 2.0 ** -110, 1.5 * 2.0 ** -120])
@pytest.mark.parametrize("nq,cap,fresh", [(1, 200, 0), (1, 3000, 0), (600, 100, 0), (200, 600, 0), (3, 100, 1)])
def test_values_at_the_ends_of_fp32(nq, cap, fresh, scale):
    """Value scales up to 2^127 (codes up to 1: results stay finite) and down to
    the smallest the quantiser gives; results are normal numbers throughout."""
    d, group = 64, 4
    g = torch.Generator().manual_seed(nq + cap)
    c = fm.KvCacheInt8(1, 1, cap, d)
    kc = torch.randint(-127, 128, (1, 1, cap, d), generator=g, dtype=torch.int8)
    most = 1 if scale >= 2.0 ** 120 else 127
    vc = torch.randint(0, most + 1, (1, 1, cap, d), generator=g, dtype=torch.int8)
    k, v = _put(c, kc, torch.full((1, 1, cap), 1.0 / 64), vc, torch.full((1, 1, cap), scale))
    q = torch.randn(1, nq, group, d, generator=g).to(torch.bfloat16)
    new = [torch.zeros(1, fresh, 1, d, dtype=torch.bfloat16)] * 2 if fresh else [None, None]
    o, a = attention_ref(q.double(), k, v, [cap], False, *[None if t is None else t.double() for t in new], d ** -0.5)
    got = c.attend(q.cuda(), _lens(cap), k_new=new[0] if not fresh else new[0].cuda(), v_new=new[1] if not fresh else new[1].cuda())
    assert_attention(got, o, a)


# ------------------------------------------------------------------ long tails
@pytest.mark.gpu
@pytest.mark.parametrize("below", [25.4, 27.5])
@pytest.mark.parametrize("nq,cap", [(600, 1 << 20), (1, 1 << 20)])
def test_a_long_tail_of_small_weights(nq, cap, below):
    """One key takes nearly all the weight, 2^20 others 2^-25.4 or 2^-27.5 of it
    each: together 2.4 % or 0.6 %, with values of the other sign.

    A contribution is held in steps of 2^-27 of the row's largest at worst, an
    error of 2^-28 each, and at most 2^17 keys share a reference; the parts of
    others are in units of their own largest: 2^-11 of sum p |v| in all."""
    d, group = 64, 16
    c = fm.KvCacheInt8(1, 1, cap, d)
    c.v.fill_(127)
    c.v[0, 0, 0] = -127
    c.v_scale.fill_(2.0 ** -7)
    c.k_scale.fill_(2.0 ** -5)
    q = torch.full((1, nq, group, d), 1.0, dtype=torch.bfloat16, device="cuda")
    scale = below * math.log(2.0) / (64 * 64 * 2.0 ** -5)
    c.k[0, 0, 0] = 64  # its score: 64 channels x 64 codes
    got = c.attend(q, _lens(cap), scale=scale).double()
    s = float(np.float32(scale)) * 64 * 64 * 2.0 ** -5  # log of the first key's weight
    tail = (cap - 1) * math.exp(-s)
    value = 127 * 2.0 ** -7
    want = value * (tail - 1) / (tail + 1)
    # (assert_attention's bound with the fp16 rounding of a probability, not bf16's)
    tol = value * (2.0 ** -11 + 2.0 ** -11 + 2.0 ** -12) + abs(want) * 2.0 ** -8
    assert float((got - want).abs().max()) <= tol, (float(got.min()), float(got.max()), want)


# ------------------------------------------------------------ query precision
@pytest.mark.gpu
@pytest.mark.parametrize("nq", [1, 40])
@pytest.mark.parametrize("size", [30.0, 1000.0])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_queries_of_wide_range(d, size, nq):
    """One channel of a query is far above the others and its key codes are zero:
    the others decide.  Two keys with values +-1 share the weight, so an error
    of a score shows undivided.

    A probability rounds to fp16 (2^-11).  The query counts as a 24-bit integer of
    its row's range: a channel is off by at most 2^-22 of the power of two below
    the row's largest, which moves a score by at most 2^-22 size sum|k| scale and
    a probability by as much (two keys: a quarter of the sum of both).  fp32
    scores and exp2: their sums over |q k| up to about 40 are off by less than 2^-12."""
    B, group = 8, 8
    g = torch.Generator().manual_seed(nq + d)
    c = fm.KvCacheInt8(B, 1, 2, d)
    kc = torch.randint(-127, 128, (B, 1, 2, d), generator=g, dtype=torch.int8)
    kc[..., 0] = 0
    vc = torch.full((B, 1, 2, d), 127, dtype=torch.int8)
    vc[:, :, 1] = -127
    k, v = _put(c, kc, torch.full((B, 1, 2), 2.0 / 127), vc, torch.full((B, 1, 2), 1.0 / 127))
    q = torch.randn(B, nq, group, d, generator=g)
    q[..., 0] = size
    q = q.to(torch.bfloat16)
    o, a = attention_ref(q.double(), k, v, [2] * B, False, None, None, d ** -0.5)
    got = c.attend(q.cuda(), _lens(*[2] * B))
    score = 2.0 ** -22 * size * float(k.abs().sum(-1).max()) * d ** -0.5
    tol = a * (2.0 ** -11 + 2.0 ** -12 + score) + o.abs() * 2.0 ** -8
    over = ((got.cpu().double() - o).abs() - tol).max()
    assert over <= 0, f"beyond the bound by {over:.3e}"


@pytest.mark.gpu
@pytest.mark.parametrize("tokens", [3, 200, 600])
@pytest.mark.parametrize("sx,sw", [(1.37 * 2.0 ** 110, 1.61 * 2.0 ** -40), (1.61 * 2.0 ** -40, 1.37 * 2.0 ** 110)])
def test_linear_i8_large_scales(tokens, sx, sw):
    """A sum times the larger scale alone is past fp32 (2^22 2^110), the result
    is not.  Two roundings of 2^-24 as for the small scales."""
    k, n = 512, 300
    g = torch.Generator().manual_seed(tokens)
    x, w = torch.randint(100, 128, (tokens, k), generator=g), torch.randint(100, 128, (n, k), generator=g)
    xs, ws = torch.full((tokens,), sx), torch.full((n,), sw)
    want = (x.double() @ w.double().t()) * xs.double()[:, None] * ws.double()
    got = fm.linear_i8(x.to(torch.int8).cuda(), xs.cuda(), w.to(torch.int8).cuda(), ws.cuda(), out_dtype=torch.float32)
    assert bool(((got.cpu().double() - want).abs() <= want * (2.0 ** -23 + 2.0 ** -46)).all())


# -------------------------------------------------------------- int8 product
def _product(tokens, n, k, sx=None, sw=None):
    g = torch.Generator(device="cuda").manual_seed(tokens + 7 * n + 13 * k)
    x = torch.randint(-128, 128, (tokens, k), generator=g, device="cuda", dtype=torch.int8)
    w = torch.randint(-128, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
    xs = torch.rand(tokens, generator=g, device="cuda") + 0.01
    ws = torch.rand(n, generator=g, device="cuda") + 0.01
    return x, xs, w, ws


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("tokens,n,k", [(2500, 6008, 96), (2501, 6001, 96), (3997, 10000, 1024), (3997, 9999, 1024),
                                        (7743, 4112, 512)])
def test_linear_i8_of_several_tiles_per_sm(tokens, n, k, out):
    """A CTA (the first two shapes) or a pair of CTAs (the others) walks three to
    eight tiles, the last ones ragged: accumulators, scales and output boxes in
    turn.  Whatever the plan, tiles are at most 256 x 256 (pairs) or 128 x 256, so
    every shape is more than three rounds over the SMs.  Rows that start on 16
    bytes leave as tensor stores, the others along the rows."""
    assert -(-tokens // 256) * -(-n // 256) >= 3 * 74
    x, xs, w, ws = _product(tokens, n, k)
    ref = (x.double() @ w.double().t()) * xs.double()[:, None] * ws.double()
    y = fm.linear_i8(x, xs, w, ws, out_dtype=DT[out])
    # the sum is exact; its conversion, two products and the output round
    assert bool(((y.double() - ref).abs() <= ref.abs() * (3 * 2.0 ** -24 + HALF_ULP[out])).all())
    big = torch.full((tokens + 2, n + 8), 7.0, dtype=DT[out], device="cuda")
    fm.linear_i8(x, xs, w, ws, out=big[1:-1, :n])
    assert torch.equal(big[1:-1, :n], y)
    big[1:-1, :n] = 7.0
    assert bool((big == 7.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("tokens,n,ld", [(129, 543, 544), (300, 11, 12), (700, 715, 728), (2500, 6003, 6008), (65, 1, 8)])
def test_linear_i8_rows_that_end_inside_16_bytes(tokens, n, ld, out):
    """Rows start on 16 bytes, but hold no whole number of them: the columns
    behind them stay as they were."""
    x, xs, w, ws = _product(tokens, n, 160)
    ref = (x.double() @ w.double().t()) * xs.double()[:, None] * ws.double()
    big = torch.full((tokens + 1, ld), 7.0, dtype=DT[out], device="cuda")
    y = fm.linear_i8(x, xs, w, ws, out=big[:tokens, :n])
    assert bool(((y.double() - ref).abs() <= ref.abs() * (3 * 2.0 ** -24 + HALF_ULP[out])).all())
    y.fill_(7.0)
    assert bool((big == 7.0).all())


# -------------------------------------------------------------------- wide rows
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("width", [1 << 22, (1 << 22) + 3])
def test_norms_of_very_wide_rows(width, dtype):
    """Equal elements, whose squares round the same way every time they are
    added: 2^14 per thread.  Groups of 64 sums, and their sums: under 400
    roundings of 2^-24, halved by the root, and those of the scale's formula."""
    x = torch.full((2, width), 0.1, dtype=DT[dtype], device="cuda")
    x[1] = torch.linspace(-1, 1, width, device="cuda").to(DT[dtype])
    _, s = fm.quantize_rows(x, rms_eps=1e-6)
    want = (x.double().abs().amax(-1) / 127).float().double() / torch.sqrt((x.double() ** 2).mean(-1) + 1e-6)
    assert bool(((s.double() - want).abs() <= want * 2.0 ** -16).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("width", [512, 100])
@pytest.mark.parametrize("eps", [1e-44, 1e-40, 1e-30, 1e-6, 1e20])
def test_norms_of_small_and_large_rows(width, dtype, eps):
    """Rows whose squares are below fp32 or above it, with an eps on either side.
    (The bound is test_quantize_rows'; a result below 2^-126 rounds to a step of
    2^-149, half of which is 2^-150.)"""
    g = torch.Generator().manual_seed(width)
    x = torch.randn(12, width, generator=g).double()
    for i, e in enumerate((-100, -80, -74, -70, -66, -50, -1, 0, 30, 60, 90, 120)):
        x[i] *= 2.0 ** e
    x = x.to(DT[dtype])
    _, s = fm.quantize_rows(x.cuda(), rms_eps=eps)
    want = quant_ref(x.double().numpy())[1].astype(np.float64) / np.sqrt((x.double().numpy() ** 2).mean(-1) + float(np.float32(eps)))
    assert np.all(np.abs(s.cpu().numpy() - want) <= want * 2.0 ** -17 + 2.0 ** -150)


# ------------------------------------------------------------ pending errors
PENDING = """
import torch
import flow_matching_action_pi0_b200 as fm
x = torch.linspace(-1, 1, 256, device="cuda").view(2, 128)
codes, scale = torch.empty(2, 128, dtype=torch.int8, device="cuda"), torch.empty(2, device="cuda")
def quantize():
    fm.pae_quantize_rows(x.data_ptr(), 128, 2, 128, fm.PAE_FP32, 0.0, codes.data_ptr(), scale.data_ptr(), 0)
quantize()
torch.cuda.synchronize()
side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
status = None
try:
    with torch.cuda.graph(graph, stream=side):
        x.add_(0)
        try:
            fm.pae_int8_sync(side.cuda_stream)  # not allowed in a capture, which it ends
        except fm.PaeError as e:
            status = e.status
except RuntimeError:
    pass
assert status == fm.PAE_ERR_CUDA, status
scale.zero_()
quantize()
fm.pae_int8_sync()
assert bool((scale > 0).all())
print("usable")
"""


@pytest.mark.gpu
def test_a_refused_call_leaves_the_operators_usable():
    """A failure that is over (a synchronisation inside a capture) is reported
    once, by the call that met it."""
    r = subprocess.run([sys.executable, "-c", PENDING], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0 and "usable" in r.stdout, r.stderr[-2000:]



# -------------------------------------------------------------------- contexts
def test_a_prefix_too_wide_for_32_bit_sums_is_refused():
    def create(width):
        return _create_status(_cfg(kv_int8=True, prefix_w8a8=True, prefix_width=width))[::2]

    st, msg = create(131072)  # the next multiple of 64 past the product's 131056
    assert st == fm.PAE_ERR_UNSUPPORTED and "prefix_width" in msg
    st, msg = create(131008)  # the last one within: the next check is reached, the missing weights
    assert st == fm.PAE_ERR_ARG and "NULL" in msg


@pytest.mark.gpu
@pytest.mark.parametrize("opt,how", [("FUSED_NORM", 1), ("FACTORED_NORM", 2)])
@pytest.mark.parametrize("rope", [0.0, 10000.0])
@pytest.mark.parametrize("batch", [1, 3])
def test_norms_in_the_projections_over_an_int8_prefix(opt, how, rope, batch):
    """The other placements of the norm project q, k and v through epilogues of
    their own, which put the action keys into the int8 prefix's buffer too."""
    import oracle  # noqa: F401
    import workloads as wl
    from tests.helpers import assert_parity, oracle_rows, run_gpu, set_prefixes
    from workloads import device as wd
    cfg = wl.TINY_FP32.replace(name="kv8_norms", dtype=wl.BF16, batch=batch, rope_base=rope)
    W = wl.make_weights(cfg)
    ex = fm.ActionExpert(fm.make_config(kv_int8=True, **wd.abi_config(cfg)), wd.upload_weights(cfg, W))
    try:
        lengths = [64, 17, 0][:batch]
        ks, vs = wl.make_prefix(cfg, lengths=lengths)
        set_prefixes(ex, cfg, ks, vs)
        ex.set_option(getattr(fm, "PAE_OPT_" + opt), 1)
        assert ex.query(fm.PAE_Q_FUSED_NORM, batch) == how
        ex.precompute_tables(wl.uniform_grid(cfg.steps))
        noise = wl.make_noise(cfg)
        out = run_gpu(ex, noise)
        shp = (cfg.layers, batch, cfg.n_kv_heads, cfg.prefix)
        vals = [np.frombuffer(ex.debug_copy(n + "codes").tobytes(), np.int8).reshape(shp + (cfg.head_dim,)).astype(np.float64) *
                np.frombuffer(ex.debug_copy(n + "scales").tobytes(), np.float32).reshape(shp)[..., None] for n in "kv"]
        k8, v8 = [[[t[l, b, :, :n].transpose(1, 0, 2) for l in range(cfg.layers)] for b, n in enumerate(lengths)] for t in vals]
        assert_parity(out, oracle_rows(cfg, W, k8, v8, noise, wl.uniform_grid(cfg.steps)), cfg.dtype, cfg.name)
    finally:
        ex.close()


# ----------------------------------------------------------------------- build
@pytest.fixture
def small_tree(tmp_path, monkeypatch):
    """The build on one small source in a folder of its own."""
    (tmp_path / "csrc").mkdir()
    (tmp_path / "csrc" / "one.cu").write_text('extern "C" int pae_one(void) { return 1; }\n')
    (tmp_path / "csrc" / "int8_tensors.cpp").write_text("this is not C++\n")
    for name, path in dict(HERE=".", CSRC="csrc", LIB="libpae.so", TENSORS="_int8_tensors.so",
                           _TENSORS_SRC="csrc/int8_tensors.cpp").items():
        monkeypatch.setattr(fbuild, name, str(tmp_path / path))
    return tmp_path


def test_the_library_builds_without_pytorch(small_tree, monkeypatch):
    def nothing():
        raise AssertionError("the tensor module was compiled")

    monkeypatch.setattr(fbuild, "_torch_version", lambda: None)
    monkeypatch.setattr(fbuild, "_tensors_command", nothing)
    assert fbuild.build() == fbuild.LIB
    assert ctypes.CDLL(fbuild.LIB).pae_one() == 1


def test_a_tensor_module_that_fails_leaves_the_library(small_tree, capsys):
    with pytest.raises(RuntimeError, match="int8_tensors"):
        fbuild.build()
    assert ctypes.CDLL(fbuild.LIB).pae_one() == 1
    assert not os.path.exists(fbuild.TENSORS)


def test_a_tensor_module_for_another_pytorch_is_built_again(small_tree, monkeypatch):
    (small_tree / "csrc" / "int8_tensors.cpp").write_text('extern "C" int two(void) { return 2; }\n')
    built = []

    def command():
        built.append(1)
        return ["g++", "-shared", "-fPIC", fbuild._TENSORS_SRC, "-o", fbuild.TENSORS + ".tmp"]

    monkeypatch.setattr(fbuild, "_tensors_command", command)
    for version, times in (("1.0", 1), ("1.0", 1), ("1.1", 2), ("1.1", 2)):
        monkeypatch.setattr(fbuild, "_torch_version", lambda v=version: v)
        fbuild.build()
        assert len(built) == times


# ----------------------------------------------------------------------- cache
def test_the_tensors_of_a_cache_cannot_be_exchanged():
    """The cache's calls hold their addresses."""
    c = fm.KvCacheInt8(1, 1, 8, 64, device="cpu")
    for name in ("k", "v", "k_scale", "v_scale"):
        with pytest.raises(AttributeError):
            setattr(c, name, getattr(c, name).clone())
        getattr(c, name).fill_(1)
        assert bool((getattr(c, name) == 1).all())
    assert c.shape == (1, 1, 8, 64) and c.k.shape == c.shape
