"""The action expert with its prefix in 8 bits (PAE_KV_INT8, PAE_PREFIX_W8A8):
prefix slots against the quantiser's definition, final actions against the
float64 oracle on the keys and values that the slots stand for.
"""
import numpy as np
import pytest

import flow_matching_action_pi0_b200 as fm
import oracle
import workloads as wl
from tests.helpers import assert_bf16_slot_close, assert_parity, max_abs, oracle_rows, run_gpu, set_prefixes
from tests.test_abi import _cfg, _create_status
from tests.test_int8_ops import quant_ref
from workloads import device as wd

ROPE = 10000.0


# ------------------------------------------------------------------------- CPU
def test_flags_are_checked():
    def status(**kw):
        return _create_status(_cfg(**kw))[::2]

    st, msg = status(dtype="fp32", kv_int8=True)
    assert st == fm.PAE_ERR_UNSUPPORTED and "8-bit" in msg
    st, msg = status(prefix_w8a8=True, prefix_width=128)
    assert st == fm.PAE_ERR_ARG and "PAE_KV_INT8" in msg
    st, msg = status(kv_int8=True, prefix_w8a8=True)
    assert st == fm.PAE_ERR_ARG and "prefix_width" in msg
    assert status(dtype=fm.PAE_BF16 | 0x400)[0] == fm.PAE_ERR_ARG
    # valid flags reach the next check, the missing weights
    st, msg = status(kv_int8=True, prefix_w8a8=True, prefix_width=128)
    assert st == fm.PAE_ERR_ARG and "NULL" in msg
    st, msg = status(dtype="w4a16", kv_int8=True)
    assert st == fm.PAE_ERR_ARG and "NULL" in msg


def test_plan_queries():
    kw = dict(layers=18, width=1024, n_q_heads=8, n_kv_heads=1, head_dim=256, mlp_dim=4096, action_dim=32, chunk=50,
              max_batch=32, max_prefix=968)
    c8, c16 = fm.make_config(dtype="bf16", kv_int8=True, **kw), fm.make_config(dtype="bf16", **kw)
    assert fm.pae_plan_query(c8, fm.PAE_Q_ATTN_CHUNK, 1) == 64
    assert fm.pae_plan_query(c8, fm.PAE_Q_ATTN_SPLITS, 1) == 8
    assert fm.pae_plan_query(c8, fm.PAE_Q_ATTN_SPLITS, 32) == 1
    for what in (fm.PAE_Q_SPLITS, fm.PAE_Q_TOKEN_TILE, fm.PAE_Q_FUSED_NORM):
        assert fm.pae_plan_query(c8, what, 4) == fm.pae_plan_query(c16, what, 4)


# ------------------------------------------------------------------------- GPU
def _expert(cfg, W=None, w8a8=False):
    W = wl.make_weights(cfg) if W is None else W
    dev = wd.upload_weights(cfg, W)
    return fm.ActionExpert(fm.make_config(kv_int8=True, prefix_w8a8=w8a8, **wd.abi_config(cfg)), dev), W


def _slots(ex, cfg):
    """(codes, scales) of K and of V, [L][B][Hkv][P][d]."""
    shp = (cfg.layers, cfg.batch, cfg.n_kv_heads, max(cfg.prefix, 1))
    return [(np.frombuffer(ex.debug_copy(n + "codes").tobytes(), np.int8).reshape(shp + (cfg.head_dim,)),
             np.frombuffer(ex.debug_copy(n + "scales").tobytes(), np.float32).reshape(shp)) for n in "kv"]


def _values(ex, cfg, lengths):
    """What the slots stand for, as the oracle takes prefixes: [row][layer] [n][Hkv][d]."""
    out = []
    for codes, scales in _slots(ex, cfg):
        val = codes.astype(np.float64) * scales[..., None]
        out.append([[val[l, b, :, :n].transpose(1, 0, 2) for l in range(cfg.layers)] for b, n in enumerate(lengths)])
    return out


def _denoise(ex, cfg):
    ex.precompute_tables(wl.uniform_grid(cfg.steps))
    noise = wl.make_noise(cfg)
    return noise, run_gpu(ex, noise)


TINY = wl.TINY_FP32.replace(dtype=wl.BF16)
CASES = [
    (TINY.replace(name="kv8_b1"), [64]),
    (TINY.replace(name="kv8_ragged", batch=5, rope_base=ROPE), [64, 0, 17, 63, 1]),
    (TINY.replace(name="kv8_gqa2", n_kv_heads=2, batch=20, chunk=15, rope_base=ROPE), [(7 * b) % 65 for b in range(20)]),
    (TINY.replace(name="kv8_d256", n_q_heads=2, head_dim=256, batch=2), [64, 9]),
    (TINY.replace(name="kv8_w4a16", dtype=wl.W4A16, rope_base=ROPE, batch=3), [64, 7, 0]),
    (TINY.replace(name="kv8_splits", prefix=600, batch=2, chunk=50), [600, 65]),
    (TINY.replace(name="kv8_one_token", chunk=1, batch=2), [64, 3]),
    (TINY.replace(name="kv8_no_prefix", prefix=0, batch=1), [0]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("cfg,lengths", CASES, ids=[c.name for c, _ in CASES])
def test_actions_over_an_int8_prefix(cfg, lengths):
    ex, W = _expert(cfg)
    try:
        ks, vs = wl.make_prefix(cfg, lengths=lengths)
        set_prefixes(ex, cfg, ks, vs)
        noise, out = _denoise(ex, cfg)
        for rows, (codes, scales) in zip((ks, vs), _slots(ex, cfg)):
            for b, n in enumerate(lengths):
                for l in range(cfg.layers if n else 0):
                    q, s = quant_ref(np.asarray(rows[b][l], np.float64).reshape(n, cfg.n_kv_heads, cfg.head_dim))
                    assert np.array_equal(codes[l, b, :, :n].transpose(1, 0, 2), q)
                    assert np.array_equal(scales[l, b, :, :n].T, s)
        k8, v8 = _values(ex, cfg, lengths)
        grid = wl.uniform_grid(cfg.steps)
        assert_parity(out, oracle_rows(cfg, W, k8, v8, noise, grid), cfg.dtype, cfg.name)
        # the other ways to run the loop: direct launches, no PDL, norms in the
        # projections, step ranges; loops without an int8 path fall back to the graph
        for opt in (fm.PAE_OPT_PERSISTENT, fm.PAE_OPT_DATAFLOW):
            ex.set_option(opt, 1)
            assert np.array_equal(run_gpu(ex, noise), out)
            ex.set_option(opt, 0)
        ex.set_option(fm.PAE_OPT_PDL, 0)
        assert np.array_equal(run_gpu(ex, noise), out)
        ex.set_option(fm.PAE_OPT_USE_GRAPH, 0)
        assert np.array_equal(run_gpu(ex, noise), out)
        import torch
        x = torch.from_numpy(noise).cuda()
        y = ex.denoise_steps(x, torch.empty_like(x), 0, 1)
        y = ex.denoise_steps(y, torch.empty_like(x), 1, cfg.steps)
        ex.sync()
        assert np.array_equal(y.cpu().numpy(), out)
    finally:
        ex.close()


@pytest.mark.gpu
def test_a_new_observation_replaces_the_int8_prefix():
    cfg = TINY.replace(name="kv8_swap", batch=2, prefix_width=128)
    W = dict(wl.make_weights(cfg))
    W["w_prefix_kv"] = wl.make_prefix_model(cfg, prefix_len=40)["w_prefix_kv"]
    ex, _ = _expert(cfg, W)
    try:
        ks, vs = wl.make_prefix(cfg, lengths=[64, 30])
        set_prefixes(ex, cfg, ks, vs)
        noise, first = _denoise(ex, cfg)
        hs = [wl.round_bf16(np.random.default_rng(l).standard_normal((40, 128))) for l in range(cfg.layers)]
        ex.set_prefix_hidden(0, [wd.to_dev(h, wd.act_dtype(cfg)) for h in hs], 40)
        second = run_gpu(ex, noise)
        assert max_abs(first[0], second[0]) > 1e-3 and np.array_equal(first[1], second[1])
        set_prefixes(ex, cfg, ks[:1], vs[:1], rows=[0])
        assert np.array_equal(run_gpu(ex, noise), first)
    finally:
        ex.close()


def _hidden(cfg, lengths):
    return [[wl.round_bf16(np.random.default_rng(100 * b + l).standard_normal((n, cfg.prefix_width)) * (1 + l))
             for l in range(cfg.layers)] for b, n in enumerate(lengths)]


@pytest.mark.gpu
@pytest.mark.parametrize("w8a8", [False, True], ids=["bf16_product", "int8_product"])
@pytest.mark.parametrize("rope", [0.0, ROPE])
@pytest.mark.parametrize("hk,d,lengths", [(1, 64, [64, 0, 37]), (2, 64, [130, 1, 65]), (1, 256, [200, 16, 3])])
def test_prefix_production_in_8_bits(hk, d, lengths, rope, w8a8):
    cfg = TINY.replace(name="kv8_hidden", n_kv_heads=hk, head_dim=d, batch=3, prefix=max(lengths), prefix_width=384,
                       rope_base=rope)
    W = dict(wl.make_weights(cfg))
    W["w_prefix_kv"] = wl.make_prefix_model(cfg, prefix_len=4)["w_prefix_kv"]
    p = oracle.params_from_weights(cfg, W)
    ex, _ = _expert(cfg, W, w8a8)
    try:
        hs = _hidden(cfg, lengths)
        for b, n in enumerate(lengths):
            ex.set_prefix_hidden(b, [wd.to_dev(h, wd.act_dtype(cfg)) for h in hs[b]], n)
        noise, out = _denoise(ex, cfg)
        slots = _slots(ex, cfg)
        k8, v8 = _values(ex, cfg, lengths)
        for b, n in enumerate(lengths):
            if n == 0:
                continue
            ref = oracle.prefix_kv_from_hidden([np.float64(h) for h in hs[b]], [np.float64(w) for w in W["w_prefix_kv"]], p)
            for l in range(cfg.layers):
                for i, got in enumerate((k8[b][l], v8[b][l])):
                    half = slots[i][1][l, b, :, :n].T[..., None] / 2.0  # half a quantisation step
                    if not w8a8:
                        # within the bf16 slot's bound of the oracle, plus that half step
                        nearest = np.clip(ref[i][l], got - half, got + half)
                        assert_bf16_slot_close(nearest, ref[i][l], f"row {b} layer {l}")
                        continue
                    # the product's definition: whole-number sums, the three scales, rotation
                    q, s = quant_ref(np.float64(hs[b][l]))
                    wq, ws = quant_ref(np.float64(W["w_prefix_kv"][l]))
                    norm = s / np.sqrt((np.float64(hs[b][l]) ** 2).mean(-1) + cfg.rms_eps)
                    y = (q.astype(np.float64) @ wq.astype(np.float64).T) * norm[:, None] * ws
                    y = y[:, i * hk * d:(i + 1) * hk * d].reshape(n, hk, d)
                    size = np.abs(y).max(-1, keepdims=True)
                    if i == 0 and rope:
                        y = oracle.expert.rope(y, np.arange(n), rope)
                    # 2^-17 of the norm's scale and a few fp32 roundings of values up to
                    # 1.5 times the row's largest; the scale itself one more
                    assert np.all(np.abs(got - y) <= half + size * 2.0 ** -15)
        assert_parity(out, oracle_rows(cfg, W, k8, v8, noise, wl.uniform_grid(cfg.steps)), cfg.dtype, cfg.name)
    finally:
        ex.close()


@pytest.mark.gpu
@pytest.mark.slow
def test_pi05_int8_prefix_batch_1():
    cfg = wl.PI05_BF16_BS1.replace(name="pi05_kv8")
    ex, W = _expert(cfg)
    try:
        ks, vs = wl.make_prefix(cfg)
        set_prefixes(ex, cfg, ks, vs)
        noise, out = _denoise(ex, cfg)
        k8, v8 = _values(ex, cfg, [cfg.prefix])
        assert_parity(out, oracle_rows(cfg, W, k8, v8, noise, wl.uniform_grid(cfg.steps)), cfg.dtype, cfg.name)
    finally:
        ex.close()


@pytest.mark.gpu
def test_unaligned_rows_are_refused():
    cfg = TINY.replace(name="kv8_unaligned")
    ex, _ = _expert(cfg)
    try:
        with pytest.raises(fm.PaeError) as e:
            fm.pae_set_prefix(ex.ctx, 0, [(1 << 20) + 8] * cfg.layers, [1 << 20] * cfg.layers, 4)
        assert e.value.status == fm.PAE_ERR_ARG
    finally:
        ex.close()
