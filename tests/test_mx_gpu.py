"""The microscaled (MX) operators on the GPU against the float64 oracle: quantisation and back, the residual's addition
with the norm, the experts' products at the sizes and dispatches where they can go wrong, and the layer made of them."""
import numpy as np
import pytest
import torch

import oracle.mx_oracle as ox
from oracle import gelu_tanh
import sparse_mixture_experts_04_amd as moe
from mx_util import FMT, HALF, KIND, as_dtype, check_codes, code_buffers, dispatch, f64, product_error, random_mx, read, to_dev

pytestmark = pytest.mark.gpu
EPS = 1e-5


def values_for(rng, rows, cols, dtype):
    """Rows of very different sizes, with the blocks where a quantisation can go wrong among them."""
    x = rng.standard_normal((rows, cols)) * np.exp(2 * rng.standard_normal((rows, 1)))
    tiny, top = (2.0 ** -133, 3.38953139e38) if dtype == "bf16" else (2.0 ** -149, 3.4028234e38)
    special = [np.zeros(32), np.full(32, -0.0), np.linspace(-8, 8, 32), np.linspace(0, 480, 32), np.full(32, tiny),
               np.full(32, top), np.where(np.arange(32) == 7, np.nan, 1.0), np.where(np.arange(32) == 31, -np.inf, 2.0),
               2.0 ** -np.arange(32.0), np.arange(32) * 0.25, np.full(32, np.nextafter(np.float32(2), 0)),
               np.where(np.arange(32) == 0, 2.0 ** -126, 2.0 ** -130)]
    flat = x.reshape(-1, 32)
    for i, s in enumerate(special[:flat.shape[0]]):
        flat[(i * 5 + i // 7) % flat.shape[0]] = s
    return as_dtype(flat.reshape(rows, cols), dtype)


@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 64), (3, 96), (257, 160), (8, 3584), (1000, 1408), (4097, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("form", ["fp4", "fp8"])
def test_quantise_bits(rows, cols, dtype, form):
    fmt = FMT[form]
    x = values_for(np.random.default_rng(rows + cols), rows, cols, dtype)
    codes, scales = code_buffers(rows + 1, cols, fmt)
    moe.moe_mx_quantize(KIND[dtype], fmt, rows, cols, x.cuda(), codes, scales)
    c, s, _ = read(codes[:rows], scales[:rows], fmt)
    ref_c, ref_s = ox.quantize(f64(x), fmt)
    assert np.array_equal(s, ref_s)
    assert np.array_equal(c, ref_c)
    assert (codes[rows:] == 0xA5).all() and (scales[rows:] == 0xA5).all()  # nothing past the end
    # and back, exact in fp32, rounded once in bf16
    for kind, out in ((moe.MOE_F32, torch.float32), (moe.MOE_BF16, torch.bfloat16)):
        back = torch.full((rows + 1, cols), 7.0, dtype=out, device="cuda")
        moe.moe_mx_dequantize(kind, fmt, rows, cols, codes, scales, back)
        ref = torch.from_numpy(ox.values(ref_c, ref_s, fmt)).to(out)
        assert torch.equal(back[:rows].cpu().nan_to_num(nan=1.5), ref.nan_to_num(nan=1.5))
        assert (back[rows:] == 7).all()


@pytest.mark.parametrize("form", ["fp4", "fp8"])
def test_every_code_and_scale_reads_back(form):
    fmt = FMT[form]
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1)
    per = 32 if fmt == moe.MOE_MXFP8 else 16
    scales = torch.arange(256, dtype=torch.uint8).view(256, 1).repeat(1, 256 // per)
    cols = scales.shape[1] * 32
    out = torch.empty((256, cols), device="cuda")
    moe.moe_mx_dequantize(moe.MOE_F32, fmt, 256, cols, codes.cuda(), scales.cuda(), out)
    ref = torch.from_numpy(ox.values(ox.unpack(codes.numpy(), fmt), scales.numpy(), fmt)).float()
    got = out.cpu()
    assert torch.equal(got.isnan(), ref.isnan())
    assert torch.equal(got.nan_to_num(nan=0.0), ref.nan_to_num(nan=0.0))


@pytest.mark.parametrize("T,d", [(1, 64), (1, 3584), (5, 192), (300, 448), (33, 2048), (130, 4096), (3, 5632), (2, 8192),
                                 (2, 8256), (2, 32768)])
@pytest.mark.parametrize("dtype,form,with_r", [("bf16", "fp8", True), ("bf16", "fp4", False), ("f32", "fp8", False),
                                               ("f32", "fp4", True)])
def test_add_rmsnorm(T, d, dtype, form, with_r):
    rng = np.random.default_rng(T * 7 + d)
    fmt = FMT[form]
    size = np.exp(3 * rng.standard_normal((T, 1)))
    x, r, g = (as_dtype(a, dtype) for a in (size * rng.standard_normal((T, d)), 2 * size * rng.standard_normal((T, d)),
                                            1 + 0.2 * rng.standard_normal(d)))
    if T > 2:
        x[1], r[1] = 0, 0  # a row of zeros
    cfg = moe.config(T, d, 64, 1, 1, -1, dtype)
    X, R, G = x.cuda(), r.cuda() if with_r else None, g.cuda()
    s, y = torch.full_like(X, 7), torch.full_like(X, 7)
    codes, scales = code_buffers(T, d, fmt)
    moe.moe_add_rmsnorm(cfg, X, R, G, EPS, s, y, fmt, codes, scales)
    ref_s, ref_n = ox.add_rmsnorm(f64(x), f64(r) if with_r else None, f64(g), EPS)
    h = HALF[dtype]
    # s: the fp32 addition and the store; n: see mx_util
    assert (np.abs(f64(s) - ref_s) <= (h + 2.0 ** -24) * 1.01 * np.abs(ref_s)).all()
    # the addition's rounding is relative to the sum, so cancellation costs nothing more
    d_n = 2.0 ** -21 * np.abs(ref_n)
    assert (np.abs(f64(y) - ref_n) <= h * 1.01 * np.abs(ref_n) + d_n).all()
    c, sc, _ = read(codes, scales, fmt)
    check_codes(c, sc, ref_n, d_n, fmt)
    # each output alone, in place, gives the same bits
    only = torch.empty_like(X)
    moe.moe_add_rmsnorm(cfg, X, R, G, EPS, None, only)
    assert torch.equal(only, y)
    c2, s2 = code_buffers(T, d, fmt)
    moe.moe_add_rmsnorm(cfg, X, R, G, EPS, None, None, fmt, c2, s2)
    assert torch.equal(c2, codes) and torch.equal(s2, scales)
    stream = R.clone() if with_r else X.clone()
    moe.moe_add_rmsnorm(cfg, X, stream if with_r else None, G, EPS, stream, only)  # sum over the residual
    assert torch.equal(stream, s) and torch.equal(only, y)
    over = X.clone()
    moe.moe_add_rmsnorm(cfg, over, R, G, EPS, None, over)  # y over x
    assert torch.equal(over, y)


def test_add_rmsnorm_extremes():
    """Sizes whose squares leave fp32's range, and rows with NaN and infinities among ordinary ones."""
    d = 256
    x = torch.randn(8, d, generator=torch.Generator().manual_seed(0)).bfloat16()
    x[1] *= 2.0 ** 100
    x[2] *= 2.0 ** -90
    x[3, 5] = float("nan")
    x[4, 200] = float("inf")
    g = torch.ones(d).bfloat16()
    cfg = moe.config(8, d, 64, 1, 1, -1, "bf16")
    y = torch.empty_like(x, device="cuda")
    codes, scales = code_buffers(8, d, moe.MOE_MXFP8)
    moe.moe_add_rmsnorm(cfg, x.cuda(), None, g.cuda(), 0.0, None, y, moe.MOE_MXFP8, codes, scales)
    _, n = ox.add_rmsnorm(f64(x), None, f64(g), 0.0)
    fine = [0, 1, 2, 5, 6, 7]
    got = f64(y)
    assert (np.abs(got[fine] - n[fine]) <= 2.0 ** -7.9 * np.abs(n[fine])).all()
    assert np.isnan(got[3]).all() and np.isnan(got[4, 200]) and (scales[3] == 255).all() and scales[4, 200 // 32] == 255


# T, d, F, E, k, capacity, only: small and odd sizes, K tails of 64 and 128 at both products, one expert, empty experts,
# many rows on one expert, batches on both sides of each kernel's rule
SHAPES = [(1, 64, 64, 1, 1, -1, None), (1, 256, 128, 8, 2, -1, None), (8, 512, 256, 64, 2, -1, None),
          (5, 192, 320, 3, 3, -1, None), (17, 320, 192, 16, 2, -1, None), (33, 448, 704, 2, 1, -1, None),
          (40, 1024, 512, 5, 2, 7, None), (64, 256, 1408, 4, 4, -1, None), (65, 1408, 256, 4, 2, -1, None),
          (130, 256, 576, 64, 4, -1, None), (200, 512, 512, 1, 1, -1, None), (300, 128, 64, 2, 2, -1, None),
          (333, 640, 448, 8, 4, 100, None), (520, 384, 832, 3, 1, -1, 1), (777, 256, 320, 6, 2, 0, None),
          (1100, 320, 256, 2, 2, -1, None), (400, 2688, 1408, 3, 2, -1, None), (700, 1152, 640, 2, 2, 300, None),
          (261, 768, 2304, 2, 2, -1, None), (3, 4672, 192, 2, 1, -1, None), (20, 128, 4736, 2, 2, -1, None),
          (50, 8256, 64, 3, 1, -1, 0), (150, 2688, 1408, 4, 2, -1, None), (90, 1152, 1536, 2, 2, -1, None),
          (70, 2304, 1280, 3, 1, 40, None), (300, 1344, 1088, 2, 1, -1, None), (450, 448, 1344, 64, 2, -1, None),
          (450, 1344, 704, 64, 2, -1, 5), (700, 640, 1408, 64, 2, -1, 3), (300, 1408, 640, 64, 4, -1, None)]


def run_products(shape, form, dtype, seed=0):
    T, d, F, E, k, cap, only = shape
    rng = np.random.default_rng(seed)
    fmt = FMT[form]
    cfg = moe.config(T, d, F, E, k, cap, dtype)
    perm, offsets = dispatch(rng, T, E, k, cap, 0.5, only)
    X = random_mx(rng, T, d, fmt)
    W1 = random_mx(rng, E * F, d, moe.MOE_MXFP4)
    W1 = (W1[0], W1[1], (W1[2] / np.sqrt(d)).reshape(E, F, d))
    # the same scaling in the stored scales: a power of two near 1 / sqrt(d)
    shift = int(round(0.5 * np.log2(d)))
    w1s = W1[1] - shift
    w1v = W1[2] * np.sqrt(d) * 2.0 ** -shift
    W2 = random_mx(rng, E * d, F, moe.MOE_MXFP4)
    xq, xs, w1q, w1sd, w2q, w2s, p, o = to_dev(X[0], X[1], W1[0], w1s, W2[0], W2[1], perm, offsets)
    N = int(offsets[-1])
    hq, hs = code_buffers(T * k, F, fmt)
    moe.moe_expert_up_mx(cfg, fmt, xq, xs, p, o, w1q, w1sd, hq, hs)
    y = torch.full((T * k, d), 7.0, dtype=torch.bfloat16 if dtype == "bf16" else torch.float32, device="cuda")
    moe.moe_expert_down_mx(cfg, fmt, hq, hs, o, w2q, w2s, y)
    torch.cuda.synchronize()
    # up against the oracle
    u, total, peak = ox.expert_up(X[2], perm, offsets, w1v, k)
    h = gelu_tanh(u)
    e = 1.13 * product_error(total, peak, d, fmt) + 2.0 ** -20 * np.abs(u)
    hc, hsc, hv = read(hq, hs, fmt)
    check_codes(hc[:N], hsc[:N], h, e, fmt, f"H of {shape}")
    assert (hq[N:] == 0xA5).all() and (hs[N:] == 0xA5).all()  # rows past the last pair stay
    # down against the oracle on the computed H
    yr, total, peak = ox.expert_down(hv[:N], offsets, W2[2].reshape(E, d, F))
    e = product_error(total, peak, F, fmt) + HALF[dtype] * 1.01 * np.abs(yr)
    got = f64(y)
    bad = np.abs(got[:N] - yr) > e
    assert not bad.any(), f"Y of {shape}: {int(bad.sum())} off, first {np.argwhere(bad)[:4]}"
    assert (got[N:] == 7).all()
    # both in one call: the same bits
    y2 = torch.full_like(y, 7.0)
    ws = torch.full((moe.moe_workspace_size(cfg, moe.MOE_OP_EXPERT_FFN_MX),), 0xFF, dtype=torch.uint8, device="cuda")
    moe.moe_expert_ffn_mx(cfg, fmt, xq, xs, p, o, w1q, w1sd, w2q, w2s, y2, ws)
    assert torch.equal(y, y2)


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s[:5])))
@pytest.mark.parametrize("form", ["fp4", "fp8"])
def test_products(shape, form):
    run_products(shape, form, "bf16")


@pytest.mark.parametrize("shape", [SHAPES[4], SHAPES[8], SHAPES[12]], ids=lambda s: "x".join(map(str, s[:5])))
@pytest.mark.parametrize("form", ["fp4", "fp8"])
def test_products_fp32_output(shape, form):
    run_products(shape, form, "f32", seed=1)


@pytest.mark.parametrize("T", [6, 300])
@pytest.mark.parametrize("form", ["fp4", "fp8"])
def test_bad_rows_stay_their_own(T, form):
    """Permutation entries that name no token give zero rows; a token with a NaN scale spoils its own row alone."""
    fmt = FMT[form]
    d, F, E, k = 256, 192, 2, 1
    rng = np.random.default_rng(3)
    cfg = moe.config(T, d, F, E, k, -1, "bf16")
    perm, offsets = dispatch(rng, T, E, k)
    X, W1, W2 = random_mx(rng, T, d, fmt), random_mx(rng, E * F, d, 0), random_mx(rng, E * d, F, 0)
    def out(xs, perm):
        a = to_dev(X[0], xs, perm, offsets, W1[0], W1[1], W2[0], W2[1])
        y = torch.empty((T, d), dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(moe.moe_workspace_size(cfg, moe.MOE_OP_EXPERT_FFN_MX), dtype=torch.uint8, device="cuda")
        moe.moe_expert_ffn_mx(cfg, fmt, *a, y, ws)
        return y.cpu()
    good = out(X[1], perm)
    assert good.isfinite().all()
    broken = perm.copy()
    broken[2], broken[4] = -1, T + 5
    y = out(X[1], broken)
    same = [r for r in range(T) if r not in (2, 4)]
    assert torch.equal(y[same], good[same]) and (y[[2, 4]] == 0).all()
    xs = X[1].copy()
    xs[perm[1], 1] = 255
    y = out(xs, perm)
    same = [r for r in range(T) if r != 1]
    assert torch.equal(y[same], good[same]) and y[1].isnan().all()


def make_layer(T, d, F, E, k, form, cap=-1, dtype="bf16", seed=0):
    g = torch.Generator().manual_seed(seed)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    n = lambda *s, scale=1.0: (scale * torch.randn(*s, generator=g)).to(t).cuda()  # noqa: E731
    cfg = moe.config(T, d, F, E, k, cap, dtype)
    layer = moe.MxMoELayer(cfg, 1 + n(d, scale=0.1), n(d, E, scale=d ** -0.5), n(E, F, d, scale=d ** -0.5),
                           n(E, d, F, scale=F ** -0.5), gate_bias=n(E, scale=0.2).float(), fmt=FMT[form])
    return layer, n(T, d), n(T, d)


@pytest.mark.parametrize("T,d,F,E,k,form,cap,dtype", [(1, 256, 128, 8, 2, "fp8", -1, "bf16"),
                                                      (8, 512, 256, 64, 2, "fp4", -1, "bf16"),
                                                      (90, 320, 192, 8, 2, "fp8", 20, "bf16"),
                                                      (700, 256, 320, 8, 3, "fp4", -1, "bf16"),
                                                      (150, 128, 128, 4, 2, "fp8", -1, "f32")])
def test_layer_is_its_parts(T, d, F, E, k, form, cap, dtype):
    """moe_forward_mx gives the bits of the calls it is made of, and the oracle's layer within its roundings."""
    layer, x, r = make_layer(T, d, F, E, k, form, cap, dtype)
    cfg, fmt, b = layer.cfg, layer.fmt, layer.buf
    out = layer.forward(x, r).clone()
    s, y, yp, o2 = (torch.empty_like(x) for _ in range(4))
    codes, scales = code_buffers(T, d, fmt)
    moe.moe_add_rmsnorm(cfg, x, r, layer.gamma, layer.eps, s, y, fmt, codes, scales)
    plain = moe.ForwardBuffers.allocate(cfg)
    moe.moe_route(cfg, y, layer.Wg, layer.gate_bias, plain.topk_ids, plain.topk_w, plain.ws)
    moe.moe_dispatch(cfg, plain.topk_ids, y, plain.expert_counts, plain.expert_offsets, plain.perm, plain.inv_perm, None,
                     plain.ws)
    yp = torch.zeros((T * k, d), dtype=x.dtype, device="cuda")
    ws = torch.empty(moe.moe_workspace_size(cfg, moe.MOE_OP_EXPERT_FFN_MX), dtype=torch.uint8, device="cuda")
    moe.moe_expert_ffn_mx(cfg, fmt, codes, scales, plain.perm, plain.expert_offsets, *layer.W1, *layer.W2, yp, ws)
    moe.moe_combine(cfg, yp, plain.inv_perm, plain.topk_w, o2)
    assert torch.equal(layer.sum, s)
    for name in ("topk_ids", "topk_w", "expert_counts", "expert_offsets", "perm", "inv_perm"):
        assert torch.equal(getattr(b, name), getattr(plain, name)), name
    assert torch.equal(out, o2)
    # the oracle, from the codes the norm gave: products within their bounds, the combine in fp32
    N = int(plain.expert_offsets[-1])
    w1 = ox.values(ox.unpack(layer.W1[0].cpu().numpy(), 0), layer.W1[1].cpu().numpy(), 0)
    w2 = ox.values(ox.unpack(layer.W2[0].cpu().numpy(), 0), layer.W2[1].cpu().numpy(), 0)
    offsets, perm = plain.expert_offsets.cpu().numpy(), plain.perm.cpu().numpy()
    u, _, _ = ox.expert_up(read(codes, scales, fmt)[2], perm, offsets, w1, k)
    hc, hs = ox.quantize(gelu_tanh(u), fmt)
    yr, _, _ = ox.expert_down(ox.values(hc, hs, fmt), offsets, w2)
    w, inv = plain.topk_w.cpu().double().numpy(), plain.inv_perm.cpu().numpy().reshape(T, k)
    ref = np.zeros((T, d))
    for slot in range(k):
        kept = inv[:, slot] >= 0
        ref[kept] += w[kept, slot, None] * yr[inv[kept, slot]]
    # Roundings: Yp and out (2^-8 each in bf16); an H code on the other side of a rounding border moves by one step,
    # rarely: 4% of a row's size bounds a row in which one H code in a hundred moved by an eighth (fp8: fewer).
    got = f64(out)
    size = np.sqrt((ref ** 2).mean(1, keepdims=True)) + 1e-30
    assert (np.abs(got - ref) / size).max() <= 0.1 and N <= T * k
    assert (np.linalg.norm(got - ref, axis=1) <= 0.04 * np.linalg.norm(ref, axis=1) + 1e-30).all()


def test_forward_without_residual_and_tokens():
    layer, x, _ = make_layer(40, 256, 128, 4, 2, "fp8")
    out = layer.forward(x)
    assert torch.equal(layer.sum, x) and out.isfinite().all()
    cfg = moe.config(0, 256, 128, 4, 2, -1, "bf16")
    empty = moe.MxMoELayer(cfg, layer.gamma, layer.Wg, torch.zeros(4, 128, 256, dtype=torch.bfloat16, device="cuda"),
                           torch.zeros(4, 256, 128, dtype=torch.bfloat16, device="cuda"))
    assert empty.forward(x[:0]).shape == (0, 256)
    assert (empty.buf.expert_offsets == 0).all()


@pytest.mark.parametrize("T,form", [(8, "fp8"), (300, "fp4")])
def test_graph_replay(T, form):
    """Captured and replayed, with the program's own work between, the layer gives the eager bits."""
    layer, x, r = make_layer(T, 256, 192, 8, 2, form)
    ref, ref_s = layer.forward(x, r).clone(), layer.sum.clone()
    x2 = torch.randn_like(x)
    ref2 = layer.forward(x2, r).clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward(x, r)
    for _ in range(4):
        layer.buf.out.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(layer.buf.out, ref) and torch.equal(layer.sum, ref_s)
        assert torch.equal(layer.forward(x2, r), ref2)
        torch.cuda.synchronize()


def test_other_stream():
    """Work goes to the stream that is given, in its order."""
    layer, x, r = make_layer(300, 256, 192, 8, 2, "fp8")
    ref = layer.forward(x, r).clone()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        late = x * 2
        late.mul_(0.5)
        out = layer.forward(late, r)
        got = out.clone()
    s.synchronize()
    assert torch.equal(got, ref)
    layer.buf.out.zero_()
    torch.cuda.synchronize()
    layer.forward(x, r, stream=s)
    s.synchronize()
    assert torch.equal(layer.buf.out, ref)


def test_refused_tensors():
    x = torch.randn(8, 128, device="cuda").bfloat16()
    with pytest.raises(ValueError, match="contiguous"):
        moe.mx_quantize(x.t())
    c, s = moe.mx_quantize(x, moe.MOE_MXFP8)
    with pytest.raises(ValueError, match="holds"):
        moe.moe_mx_dequantize(moe.MOE_BF16, moe.MOE_MXFP8, 9, 128, c, s, x)
    with pytest.raises(TypeError):
        moe.moe_mx_dequantize(moe.MOE_F32, moe.MOE_MXFP8, 8, 128, c, s, x)
    with pytest.raises(moe.MoeError):  # rows that do not start on 16 bytes
        moe.moe_mx_quantize(moe.MOE_BF16, moe.MOE_MXFP8, 1, 64, x.view(-1)[1:65], c, s)
    layer, y, _ = make_layer(4, 128, 64, 2, 1, "fp8")
    with pytest.raises(ValueError, match="no such view"):
        layer.buf.workspace_view(layer.cfg, "H")


def test_values_through_torch_types():
    """Codes and scales may be held in torch's own 8-bit types."""
    x = torch.randn(16, 256, device="cuda")
    c, s = moe.mx_quantize(x, moe.MOE_MXFP8)
    v = moe.mx_dequantize(c, s, moe.MOE_MXFP8, torch.float32)
    w = moe.mx_dequantize(c.view(torch.float8_e4m3fn), s.view(torch.float8_e8m0fnu), moe.MOE_MXFP8, torch.float32)
    ref = c.view(torch.float8_e4m3fn).float().view(16, 8, 32) * s.view(torch.float8_e8m0fnu).float().unsqueeze(-1)
    assert torch.equal(v, w) and torch.equal(v, ref.view(16, 256))


# Sizes whose byte or element offsets pass 32 bits.  Only sampled rows and columns are compared, the last ones among
# them: an offset that wrapped would read or write elsewhere.

def random_codes(rows, cols, fmt):
    """Random finite codes and moderate scales, made on the GPU."""
    c, s = code_buffers(rows, cols, fmt)
    c.random_(0, 256) if fmt == moe.MOE_MXFP4 else c.random_(0, 120)
    return c, s.random_(118, 125)


@pytest.mark.parametrize("T", [4, 700])
@pytest.mark.parametrize("form", ["fp4", "fp8"])
def test_weights_past_32_bit_offsets(T, form):
    d, F, E, k, fmt = 8192, 16384, 64, 2, FMT[form]
    cfg = moe.config(T, d, F, E, k, -1, "bf16")
    xq, xs = random_codes(T, d, fmt)
    w1, w2 = random_codes(E * F, d, moe.MOE_MXFP4), random_codes(E * d, F, moe.MOE_MXFP4)
    for w, K in ((w1, d), (w2, F)):  # results of order 1
        w[1].sub_(int(0.5 * np.log2(K)))
    assert w1[0].numel() > 2 ** 31 and w2[0].numel() > 2 ** 31
    perm = np.concatenate([np.arange(T) * 2, np.arange(T) * 2 + 1]).astype(np.int32)  # every token: experts 1 and 63
    offsets = np.array([0, 0] + [T] * 62 + [2 * T], dtype=np.int32)
    p, o = to_dev(perm, offsets)
    hq, hs = code_buffers(T * k, F, fmt)
    moe.moe_expert_up_mx(cfg, fmt, xq, xs, p, o, *w1, hq, hs)
    y = torch.full((T * k, d), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_expert_down_mx(cfg, fmt, hq, hs, o, *w2, y)
    torch.cuda.synchronize()
    rows = {1: [0, T - 1], 63: [T, 2 * T - 1]}
    for e in (1, 63):
        r = rows[e]
        for n0 in (0, F - 64):
            at = slice(e * F + n0, e * F + n0 + 64)
            xv = read(xq, xs, fmt)[2][perm[r] // 2]
            u, total, peak = ox.product(xv, read(w1[0][at], w1[1][at], 0)[2])
            bound = 1.13 * product_error(total, peak, d, fmt) + 2.0 ** -20 * np.abs(u)
            c, s, _ = read(hq[r], hs[r], fmt)
            check_codes(c[:, n0:n0 + 64], s[:, n0 // 32:n0 // 32 + 2], gelu_tanh(u), bound, fmt, f"expert {e} from {n0}")
        for n0 in (0, d - 64):
            at = slice(e * d + n0, e * d + n0 + 64)
            yr, total, peak = ox.product(read(hq[r], hs[r], fmt)[2], read(w2[0][at], w2[1][at], 0)[2])
            bound = product_error(total, peak, F, fmt) + HALF["bf16"] * 1.01 * np.abs(yr)
            assert (np.abs(f64(y[r, n0:n0 + 64]) - yr) <= bound).all(), (e, n0)


def test_gathered_rows_past_32_bit_offsets():
    T, d, F, fmt = 262147, 8192, 64, moe.MOE_MXFP8
    cfg = moe.config(T, d, F, 2, 1, -1, "bf16")
    xq, xs = random_codes(T, d, fmt)
    assert xq.numel() > 2 ** 31
    w1 = random_codes(2 * F, d, moe.MOE_MXFP4)
    w1[1].sub_(6)
    half = T // 2
    perm = np.concatenate([np.arange(half, T), np.arange(half)]).astype(np.int32)  # the late tokens: expert 0
    p, o = to_dev(perm, np.array([0, T - half, T], dtype=np.int32))
    hq, hs = code_buffers(T, F, fmt)
    moe.moe_expert_up_mx(cfg, fmt, xq, xs, p, o, *w1, hq, hs)
    torch.cuda.synchronize()
    for e, r in ((0, [0, T - half - 2, T - half - 1]), (1, [T - half, T - 1])):
        tokens = torch.from_numpy(perm[r]).long().cuda()
        u, total, peak = ox.product(read(xq[tokens], xs[tokens], fmt)[2],
                                    read(w1[0][e * F:(e + 1) * F], w1[1][e * F:(e + 1) * F], 0)[2])
        bound = 1.13 * product_error(total, peak, d, fmt) + 2.0 ** -20 * np.abs(u)
        c, s, _ = read(hq[r], hs[r], fmt)
        check_codes(c, s, gelu_tanh(u), bound, fmt, f"expert {e}")


def test_rows_past_32_bit_offsets():
    """The last rows of arrays of more than 2^31 elements have the bits of the same rows alone."""
    rows, d = 131075, 16384
    x = torch.zeros(rows, d, dtype=torch.bfloat16, device="cuda")
    x[-5:] = torch.randn(5, d, device="cuda").bfloat16()
    last = x[-5:].clone()
    for fmt in (moe.MOE_MXFP4, moe.MOE_MXFP8):
        c, s = moe.mx_quantize(x, fmt)
        c2, s2 = moe.mx_quantize(last, fmt)
        assert torch.equal(c[-5:], c2) and torch.equal(s[-5:], s2)
        assert torch.equal(moe.mx_dequantize(c, s, fmt)[-5:], moe.mx_dequantize(c2, s2, fmt))
    g = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    results = []
    for t in (x, last):
        total, y = torch.empty_like(t), torch.empty_like(t)
        c, s = code_buffers(t.shape[0], d, moe.MOE_MXFP8)
        moe.moe_add_rmsnorm(moe.config(t.shape[0], d, 64, 1, 1, -1, "bf16"), t, t, g, EPS, total, y, moe.MOE_MXFP8, c, s)
        results.append([v[-5:].clone() for v in (total, y, c, s)])
        del total, y, c, s
    assert all(torch.equal(a, b) for a, b in zip(*results))


@pytest.mark.parametrize("T,form", [(6, "fp4"), (300, "fp8")])
@pytest.mark.parametrize("sum_is,out_is", [("x", None), ("r", None), (None, "x"), (None, "r"), ("x", "r"), ("r", "x")])
def test_layer_in_place(T, form, sum_is, out_is):
    """sum and out may be the buffers of X and the residual: the same bits."""
    layer, x, r = make_layer(T, 256, 192, 8, 2, form)
    out, total = layer.forward(x, r).clone(), layer.sum.clone()
    b, own = layer.buf, {"x": x.clone(), "r": r.clone()}
    s, o = own.get(sum_is, layer.sum), own.get(out_is, b.out)
    moe.moe_forward_mx(layer.cfg, layer.fmt, own["x"], own["r"], layer.gamma, layer.eps, layer.Wg, layer.gate_bias,
                       *layer.W1, *layer.W2, s, o, b.topk_ids, b.topk_w, b.expert_counts, b.expert_offsets, b.perm,
                       b.inv_perm, b.ws)
    assert torch.equal(s, total) and torch.equal(o, out)


def test_two_layers_on_two_streams():
    """Calls with buffers of their own may run at the same time."""
    (a, xa, ra), (c, xc, rc) = (make_layer(T, 512, 320, 8, 2, f) for T, f in ((300, "fp8"), (9, "fp4")))
    ref = a.forward(xa, ra).clone(), c.forward(xc, rc).clone()
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        a.buf.out.zero_(), c.buf.out.zero_()
        torch.cuda.synchronize()
        for s, layer, x, r in ((streams[0], a, xa, ra), (streams[1], c, xc, rc)):
            for _ in range(4):
                layer.forward(x, r, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(a.buf.out, ref[0]) and torch.equal(c.buf.out, ref[1])


# Batches whose tiles fill more than two and at most three blocks per CU (short rings): K an odd multiple of 64 in
# either product, K of two stages, several chunks of scales, fp32 results
SHORT = [(700, 1408, 1344, 64, 2, -1, None), (700, 192, 1408, 64, 2, -1, None), (700, 576, 1408, 64, 2, 30, None)]


@pytest.mark.parametrize("shape", SHORT, ids=lambda s: "x".join(map(str, s[:5])))
@pytest.mark.parametrize("form", ["fp4", "fp8"])
def test_products_short_rings(shape, form):
    run_products(shape, form, "bf16", seed=2)


def test_products_short_rings_fp32_output():
    run_products((300, 1408, 640, 64, 4, -1, None), "fp8", "f32", seed=3)


def test_products_short_rings_long_k():
    run_products((260, 2240, 5504, 4, 1, -1, None), "fp4", "bf16", seed=4)
