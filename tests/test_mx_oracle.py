"""The microscaled oracle against hand values and torch's own e4m3 conversion, and the refusals of the microscaled
entry points (CPU: every call here fails its checks, so nothing is enqueued)."""
import numpy as np
import pytest
import torch

import oracle.mx_oracle as ox
import sparse_mixture_experts_04_amd as moe


def test_e4m3_codes_are_torchs():
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.standard_normal(20000) * np.exp(3 * rng.standard_normal(20000)), ox.element_values(ox.FP8),
                        (ox.element_values(ox.FP8)[1:] + ox.element_values(ox.FP8)[:-1]) / 2]).astype(np.float32)
    ref = torch.from_numpy(np.clip(v, -448, 448)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ox.round_codes(v.astype(np.float64), ox.FP8), ref)


def test_e2m1_ties_and_saturation():
    v = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.9, -0.25, -5.0, -0.0, 0.26])
    assert ox.round_codes(v, ox.FP4).tolist() == [0, 2, 2, 4, 4, 6, 6, 7, 7, 8, 14, 8, 1]


@pytest.mark.parametrize("fmt", [ox.FP4, ox.FP8])
def test_scale_bytes(fmt):
    x = np.zeros((6, 32))
    x[1, 3] = 1.0                      # 2^0
    x[2, :] = -np.nextafter(2.0, 0)    # just below 2^1
    x[3, 5] = 2.0
    x[4, 0] = np.inf
    x[5, 31] = 1e-45
    e = ox.EMAX[fmt]
    assert ox.scale_bytes(x, fmt)[:, 0].tolist() == [0, 127 - e, 127 - e, 128 - e, 255, 0]


@pytest.mark.parametrize("fmt", [ox.FP4, ox.FP8])
def test_values_are_quantised_to_themselves(fmt):
    rng = np.random.default_rng(1)
    c, s = ox.quantize(rng.standard_normal((7, 96)), fmt)
    v = ox.values(c, s, fmt)
    c2, s2 = ox.quantize(v, fmt)
    assert np.array_equal(ox.values(c2, s2, fmt), v)
    assert np.array_equal(ox.unpack(ox.pack(c, fmt), fmt), c)


def _refused(status, fn, *a, **kw):
    with pytest.raises(moe.MoeError) as ei:
        fn(*a, **kw, stream=0)
    assert ei.value.status == status, ei.value


INVALID, UNSUPPORTED, SMALL = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE_TOO_SMALL


@pytest.mark.parametrize("fn", [moe.moe_mx_quantize, moe.moe_mx_dequantize])
def test_quantise_refusals(fn):
    _refused(INVALID, fn, 7, moe.MOE_MXFP4, 4, 64, 16, 16, 16)
    _refused(INVALID, fn, moe.MOE_BF16, 2, 4, 64, 16, 16, 16)
    _refused(INVALID, fn, moe.MOE_BF16, moe.MOE_MXFP8, -1, 64, 16, 16, 16)
    _refused(INVALID, fn, moe.MOE_BF16, moe.MOE_MXFP8, 4, -32, 16, 16, 16)
    _refused(UNSUPPORTED, fn, moe.MOE_BF16, moe.MOE_MXFP8, 4, 48, 16, 16, 16)
    _refused(UNSUPPORTED, fn, moe.MOE_BF16, moe.MOE_MXFP8, 1 << 40, 1 << 40, 16, 16, 16)
    for bad in range(3):
        for value in (None, 8):  # missing, not 16-byte aligned
            _refused(INVALID, fn, moe.MOE_BF16, moe.MOE_MXFP8, 4, 64, *[value if i == bad else 16 for i in range(3)])
    fn(moe.MOE_BF16, moe.MOE_MXFP8, 0, 64, None, None, None, stream=0)  # nothing to do


def test_norm_refusals():
    cfg = moe.config(4, 128, 64, 2, 1, -1, "bf16")
    f = moe.moe_add_rmsnorm
    ok = dict(X=16, residual=16, gamma=16, eps=1e-5, sum=16, y=32, fmt=moe.MOE_MXFP8, codes=16, scales=16)
    for change in (dict(X=None), dict(gamma=None), dict(codes=None), dict(scales=None), dict(fmt=5), dict(eps=-1.0),
                   dict(eps=float("nan")), dict(eps=float("inf")), dict(X=24), dict(residual=8), dict(y=4), dict(codes=8),
                   dict(sum=None, y=None, codes=None, scales=None), dict(y=16)):
        _refused(INVALID, f, cfg, **{**ok, **change})
    _refused(UNSUPPORTED, f, moe.config(4, 32768 + 64, 64, 2, 1, -1, "bf16"), **ok)
    _refused(UNSUPPORTED, f, moe.config(4, 96, 64, 2, 1, -1, "bf16"), **ok)
    f(moe.config(0, 128, 64, 2, 1, -1, "bf16"), **{**ok, "X": None}, stream=0)  # no tokens


def test_product_refusals():
    cfg = moe.config(4, 128, 64, 2, 1, -1, "bf16")
    for fn, n in ((moe.moe_expert_up_mx, 8), (moe.moe_expert_down_mx, 6)):
        _refused(INVALID, fn, cfg, 3, *[16] * n)
        for bad in range(n):
            _refused(INVALID, fn, cfg, moe.MOE_MXFP4, *[None if i == bad else 16 for i in range(n)])
        _refused(INVALID, fn, cfg, moe.MOE_MXFP4, 8, *[16] * (n - 1))
        _refused(UNSUPPORTED, fn, moe.config(4, 96, 64, 2, 1, -1, "bf16"), moe.MOE_MXFP4, *[16] * n)
        fn(moe.config(0, 128, 64, 2, 1, -1, "bf16"), moe.MOE_MXFP4, *[None] * n, stream=0)
    need = moe.moe_workspace_size(cfg, moe.MOE_OP_EXPERT_FFN_MX)
    assert need >= 4 * 64 + 4 * 2
    ffn = moe.moe_expert_ffn_mx
    _refused(SMALL, ffn, cfg, moe.MOE_MXFP4, *[16] * 9, 16, need - 1)
    _refused(INVALID, ffn, cfg, moe.MOE_MXFP4, *[16] * 9, None, need)
    _refused(INVALID, ffn, cfg, moe.MOE_MXFP4, *[16] * 9, 8, need)
    for bad in range(9):
        _refused(INVALID, ffn, cfg, moe.MOE_MXFP4, *[None if i == bad else 16 for i in range(9)], 16, need)


def test_forward_refusals():
    cfg = moe.config(4, 128, 64, 2, 1, -1, "bf16")
    need = moe.moe_workspace_size(cfg, moe.MOE_OP_FORWARD_MX)
    names = ("X residual gamma eps Wg gate_bias W1q W1s W2q W2s sum out topk_ids topk_w expert_counts expert_offsets perm "
             "inv_perm ws").split()
    ok = {n: 16 for n in names}
    ok |= {"eps": 1e-5, "ws_bytes": need}
    f = moe.moe_forward_mx
    for n in names:
        if n not in ("residual", "gate_bias", "sum", "eps"):
            _refused(INVALID, f, cfg, moe.MOE_MXFP8, **{**ok, n: None})
    _refused(SMALL, f, cfg, moe.MOE_MXFP8, **{**ok, "ws_bytes": need - 1})
    _refused(INVALID, f, cfg, moe.MOE_MXFP8, **{**ok, "eps": float("nan")})
    _refused(INVALID, f, cfg, 9, **ok)
    _refused(INVALID, f, cfg, moe.MOE_MXFP8, **{**ok, "X": 8})


def test_tensors_are_checked():
    cfg = moe.config(4, 128, 64, 2, 1, -1, "bf16")
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU tensor"):
        moe.moe_add_rmsnorm(cfg, x, None, x, 1e-5, x, None)
    with pytest.raises(TypeError):
        moe.mx_quantize(torch.zeros(4, 64, dtype=torch.float16))
    with pytest.raises(ValueError):
        moe.mx_quantize(x, fmt=4)


@pytest.mark.parametrize("fn,order", [(moe.moe_mx_quantize, (0, 1, 2)), (moe.moe_mx_dequantize, (1, 2, 0))])
@pytest.mark.parametrize("dtype,es", [(moe.MOE_BF16, 2), (moe.MOE_F32, 4)])
@pytest.mark.parametrize("fmt", [moe.MOE_MXFP4, moe.MOE_MXFP8])
def test_overlapping_arrays_are_refused(fn, order, dtype, es, fmt):
    # 4 x 64 elements; each pair of (array, codes, scales) in turn shares its last or first 16 bytes
    sizes = (256 * es, 256 // (2 if fmt == moe.MOE_MXFP4 else 1), 256 // 32)
    apart = (1 << 20, 2 << 20, 3 << 20)
    for a in range(3):
        for b in range(3):
            if a != b:
                at = list(apart)
                at[b] = apart[a] + (sizes[a] - 1) // 16 * 16
                _refused(INVALID, fn, dtype, fmt, 4, 64, *[at[i] for i in order])


def test_forward_refuses_one_buffer_for_sum_and_out():
    cfg = moe.config(4, 128, 64, 2, 1, -1, "bf16")
    need = moe.moe_workspace_size(cfg, moe.MOE_OP_FORWARD_MX)
    at = [(i + 1) << 20 for i in range(17)]
    _refused(INVALID, moe.moe_forward_mx, cfg, moe.MOE_MXFP8, *at[:3], 1e-5, *at[3:9], at[9], at[9], *at[10:], need)


def test_codes_of_another_format_are_refused():
    codes, scales = torch.zeros(3, 64, dtype=torch.uint8), torch.zeros(3, 2, dtype=torch.uint8)
    for c, s, fmt in ((codes, scales, moe.MOE_MXFP4), (codes[:, :32], scales, moe.MOE_MXFP8),
                      (codes[:2], scales, moe.MOE_MXFP8)):
        with pytest.raises(ValueError, match="do not go with"):
            moe.mx_dequantize(c, s, fmt)
    with pytest.raises(ValueError, match="fmt must be"):
        moe.mx_dequantize(codes, scales, 2)


def test_layer_refuses_other_shapes():
    cfg = moe.config(4, 128, 64, 2, 1, -1, "bf16")
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    ok = dict(gamma=z(128), Wg=z(128, 2), W1=z(2, 64, 128), W2=z(2, 128, 64))
    for name, t in (("gamma", z(64)), ("W1", z(2, 128, 64)), ("W2", z(2, 64, 128)), ("W1", z(3, 64, 128))):
        with pytest.raises(ValueError, match=f"{name} must have shape"):
            moe.MxMoELayer(cfg, **{**ok, name: t})
    with pytest.raises(ValueError, match="fmt must be"):
        moe.MxMoELayer(cfg, **ok, fmt=3)
