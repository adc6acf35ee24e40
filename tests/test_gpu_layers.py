"""GPU parity of the layer norm and the linear layer against their fp64
definitions, every output within the oracle's error bound, the same bits on a
second run; streams, graphs, in-place forms, special values and refusals."""
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

import numpy as np
import pytest
import torch

import microscaling_quantized_convolution_b200 as mqv
from oracle import layers_oracle as L
from tests.conftest import ROOT
from tests.layers_cases import (LIN_FEW, LIN_LONG, LIN_PAIR, LIN_PIXELS, LIN_THIN, LIN_TOKENS, LIN_WIDE, LN_ROWS,
                                LN_TILES, LN_WIDE_TILES, activations, shape_id, stored)

pytestmark = pytest.mark.gpu

KIND = {torch.float32: "f32", torch.bfloat16: "bf16"}
F32, BF16 = torch.float32, torch.bfloat16
FWD, WGRAD, DGRAD = mqv.OP_FWD, mqv.OP_WGRAD, mqv.OP_DGRAD
EPS = float(np.float32(1e-5))          # the descriptor holds fp32


def dev(a, dtype=F32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()


def check(got, ref, what):
    value, err = ref
    lim = L.rounding(value, err, KIND[got.dtype])
    g = got.double().cpu().numpy().reshape(value.shape)
    off = np.abs(g - value)
    bad = ~(off <= lim)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}, "
                           f"worst {np.max(off / lim):.3g} of the bound")


def poison(shape, dtype):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


# -------------------------------------------------------------- layer norm

TYPES = [(F32, F32), (F32, BF16), (BF16, BF16), (BF16, F32)]


def ln_inputs(shape, seed=0):
    rng = np.random.default_rng(sum(shape) + seed)
    P, C, N = shape
    return (activations(rng, shape), rng.standard_normal(C) * 0.3 + 1, rng.standard_normal(C) * 0.3,
            rng.standard_normal(shape) * 1e-2)


@pytest.mark.parametrize("xt,yt", TYPES, ids=["f32-f32", "f32-bf16", "bf16-bf16", "bf16-f32"])
@pytest.mark.parametrize("shape", LN_ROWS + LN_TILES, ids=shape_id)
def test_layer_norm(shape, xt, yt):
    P, C, N = shape
    x, gamma, beta, gy = ln_inputs(shape)
    x, gy = stored(x, KIND[xt]), stored(gy, KIND[yt])
    gamma, beta = stored(gamma, "f32"), stored(beta, "f32")
    d = mqv.ln_desc(P, C, N)
    xd, gyd, gd, bd = dev(x, xt), dev(gy, yt), dev(gamma), dev(beta)
    y, mean, rstd = mqv.ln_fwd(d, xd, gd, bd, y=poison(shape, yt), mean=poison((P, N), F32), rstd=poison((P, N), F32))
    ref = L.ln_fwd(x, gamma, beta, EPS)
    for got, name in ((y, "y"), (mean, "mean"), (rstd, "rstd")):
        check(got, ref[name], name)
    for gxt in (F32, BF16):
        gx, gg, gb = mqv.ln_bwd(d, gyd, xd, mean, rstd, gd, gx=poison(shape, gxt), ggamma=poison((C,), F32),
                                gbeta=poison((C,), F32))
        bref = L.ln_bwd(gy, x, mean.double().cpu().numpy(), rstd.double().cpu().numpy(), gamma)
        for got, name in ((gx, "gx"), (gg, "ggamma"), (gb, "gbeta")):
            check(got, bref[name], name)
    y2, mean2, rstd2 = mqv.ln_fwd(d, xd, gd, bd, y_dtype=yt)
    gx2, gg2, gb2 = mqv.ln_bwd(d, gyd, xd, mean2, rstd2, gd, gx_dtype=gxt)
    for a, b in ((y, y2), (mean, mean2), (rstd, rstd2), (gx, gx2), (gg, gg2), (gb, gb2)):
        assert torch.equal(a, b.view(a.shape))


@pytest.mark.parametrize("xt,yt", TYPES, ids=["f32-f32", "f32-bf16", "bf16-bf16", "bf16-f32"])
@pytest.mark.parametrize("shape", LN_WIDE_TILES, ids=shape_id)
def test_layer_norm_on_wide_tiles(shape, xt, yt):
    test_layer_norm(shape, xt, yt)


@pytest.mark.parametrize("shape", [(9, 264, 1), (9, 33, 1), (5, 24, 16), (3, 20, 12)], ids=shape_id)
def test_layer_norm_without_parameters_or_statistics(shape):
    x, _, _, gy = ln_inputs(shape)
    x, gy = stored(x, "f32"), stored(gy, "f32")
    d = mqv.ln_desc(*shape)
    y, mean, rstd = mqv.ln_fwd(d, dev(x), stats=False)
    assert mean is None and rstd is None
    ref = L.ln_fwd(x, None, None, EPS)
    check(y, ref["y"], "y")
    y1, _, _ = mqv.ln_fwd(d, dev(x), gamma=dev(np.full(shape[1], 2.0)), stats=False)       # gamma without beta
    check(y1, L.ln_fwd(x, np.full(shape[1], 2.0), None, EPS)["y"], "y")
    _, mean, rstd = mqv.ln_fwd(d, dev(x))
    gx, gg, gb = mqv.ln_bwd(d, dev(gy), dev(x), mean, rstd, param_grads=False)
    assert gg is None and gb is None
    bref = L.ln_bwd(gy, x, mean.double().cpu().numpy(), rstd.double().cpu().numpy(), None)
    check(gx, bref["gx"], "gx")
    _, gg, gb = mqv.ln_bwd(d, dev(gy), dev(x), mean, rstd)
    check(gg, bref["ggamma"], "ggamma")
    check(gb, bref["gbeta"], "gbeta")


@pytest.mark.parametrize("shape", [(4, 512, 1), (4, 100, 1), (3, 64, 16)], ids=shape_id)
def test_layer_norm_in_place(shape):
    x, gamma, beta, gy = ln_inputs(shape)
    d = mqv.ln_desc(*shape)
    xd, gyd = dev(x), dev(gy)
    y, mean, rstd = mqv.ln_fwd(d, xd, dev(gamma), dev(beta))
    gx, _, _ = mqv.ln_bwd(d, gyd, xd, mean, rstd, dev(gamma))
    g2 = gyd.clone()
    assert torch.equal(mqv.ln_bwd(d, g2, xd, mean, rstd, dev(gamma), gx=g2)[0], gx)
    x2 = xd.clone()
    assert torch.equal(mqv.ln_fwd(d, x2, dev(gamma), dev(beta), y=x2)[0], y)


@pytest.mark.parametrize("shape", [(6, 320, 1), (6, 33, 1), (6, 48, 16)], ids=shape_id)
def test_layer_norm_special_columns(shape):
    """A NaN or infinity spoils its own column only; a constant column gives
    beta; a large common offset keeps its precision."""
    P, C, N = shape
    x, gamma, beta, _ = ln_inputs(shape)
    x = stored(x, "f32")
    x[0, 3, 0] = np.nan
    x[1, C - 1, 0] = np.inf
    x[2, 0, 0] = -np.inf
    x[3, :, 0] = 7.25
    x[4, :, 0] = stored(4096.0 + x[4, :, 0], "f32")
    d = mqv.ln_desc(*shape)
    y, mean, rstd = mqv.ln_fwd(d, dev(x), dev(gamma), dev(beta))
    bad = torch.isnan(y)
    assert bad[:3, :, 0].all() and bad.sum() == 3 * C
    ref = L.ln_fwd(x[3:], stored(gamma, "f32"), stored(beta, "f32"), EPS)
    check(y[3:], ref["y"], "y")
    assert torch.equal(y[3, :, 0], dev(beta))
    if N > 1:
        ref = L.ln_fwd(x[:, :, 1:], stored(gamma, "f32"), stored(beta, "f32"), EPS)
        check(y[:, :, 1:].contiguous(), ref["y"], "y")


@pytest.mark.parametrize("shape", [(6, 320, 1), (6, 33, 1), (700, 264, 1), (6, 48, 16), (5, 20, 12), (4, 1500, 16),
                                   (4, 5000, 3), (4, 700, 63), (4, 128, 64)], ids=shape_id)
def test_layer_norm_gradients_of_special_columns(shape):
    """Infinities and NaN in gy, x or the statistics of a column spoil that
    column's gx and no other, bit for bit, and reach ggamma and gbeta only in
    the channels that have them (x and the statistics: ggamma)."""
    P, C, N = shape
    x, gamma, beta, gy = ln_inputs(shape)
    d, gam = mqv.ln_desc(*shape), dev(gamma)
    xd, gyd = dev(x), dev(gy)
    _, mean, rstd = mqv.ln_fwd(d, xd, gam, dev(beta))
    want, wg, wb = mqv.ln_bwd(d, gyd, xd, mean, rstd, gam)
    n = N - 1
    gyd[1, 2, n], gyd[2, C - 1, 0] = float("nan"), float("inf")
    gx, gg, gb = mqv.ln_bwd(d, gyd, xd, mean, rstd, gam)
    bad = torch.zeros((P, N), dtype=torch.bool, device="cuda")
    bad[1, n] = bad[2, 0] = True
    assert not torch.isfinite(gx).all(1)[bad].any()
    assert torch.equal(gx.transpose(1, 2)[~bad], want.transpose(1, 2)[~bad])
    odd = torch.zeros(C, dtype=torch.bool, device="cuda")
    odd[2] = odd[C - 1] = True
    for got, ref in ((gg, wg), (gb, wb)):
        assert not torch.isfinite(got[odd]).any() and torch.equal(got[~odd], ref[~odd])
    gyd = dev(gy)
    xd[1, 2, n] = float("nan")
    mean[2, 0], rstd[2, 0] = float("nan"), float("inf")
    gx, gg, gb = mqv.ln_bwd(d, gyd, xd, mean, rstd, gam)
    assert torch.equal(gx.transpose(1, 2)[~bad], want.transpose(1, 2)[~bad]) and torch.equal(gb, wb)
    assert torch.isnan(gx[1, :, n]).all() and torch.isnan(gg).all()


@pytest.mark.parametrize("shape,rows,per_warp", [((1, 16384, 4), 1024, 32), ((1, 4096, 8), 512, 16)])
def test_layer_norm_sums_take_no_more_additions_than_bounded(shape, rows, per_warp):
    """A one, and in every place where a partial sum that holds it takes
    another addend 2^-24, which a sum of 1 loses whole: a thread's channels
    are `rows` apart, a warp holds `per_warp` neighbouring rows.  The mean is
    off by as many of them as a term goes through additions, which the
    oracle's bound counts."""
    P, C, N = shape
    x = np.zeros(shape)
    x[:, 0] = 1.0
    x[:, rows::rows] = 2.0 ** -24                              # within a thread
    x[:, [1 << i for i in range(per_warp.bit_length() - 1)]] = 2.0 ** -24      # across the warp
    x[:, per_warp:rows:per_warp] = 2.0 ** -24                  # across the warps
    y, mean, rstd = mqv.ln_fwd(mqv.ln_desc(*shape), dev(x))
    ref = L.ln_fwd(x, None, None, EPS)
    for got, name in ((mean, "mean"), (rstd, "rstd"), (y, "y")):
        check(got, ref[name], name)


def test_layer_norm_of_nothing():
    for N in (1, 16):
        d = mqv.ln_desc(0, 64, N)
        x = torch.empty((0, 64, N), device="cuda")
        y, mean, rstd = mqv.ln_fwd(d, x)
        gx, gg, gb = mqv.ln_bwd(d, x, x, mean, rstd, ggamma=poison((64,), F32), gbeta=poison((64,), F32))
        assert y.shape == gx.shape == x.shape and not gg.any() and not gb.any()


# ------------------------------------------------------------ linear layer

def lin_inputs(shape, seed=0):
    P, Cin, Cout, N = shape
    rng = np.random.default_rng(sum(shape) + seed)
    return (stored(rng.standard_normal((Cout, Cin)) * (2.0 / Cin) ** 0.5, "bf16"),
            stored(activations(rng, (P, Cin, N)), "bf16"), stored(rng.standard_normal(Cout) * 0.1, "f32"),
            rng.standard_normal((P, Cout, N)), rng.standard_normal((P, Cout, N)) * 1e-2)


@pytest.mark.parametrize("shape", LIN_TOKENS + LIN_PIXELS + LIN_WIDE + LIN_LONG, ids=shape_id)
def test_linear_layer(shape):
    P, Cin, Cout, N = shape
    w, x, bias, res, gy = lin_inputs(shape)
    out = (P, Cout, N)
    wd, xd, bd = dev(w, BF16), dev(x, BF16), dev(bias)
    for act, yt, use_bias, use_res in (("none", F32, False, False), ("gelu", BF16, True, True),
                                       ("silu", F32, True, False), ("relu", BF16, False, True)):
        r = stored(res, KIND[yt])
        d = mqv.lin_desc(P, Cin, Cout, N, act)
        args = dict(bias=bd if use_bias else None, residual=dev(r, yt) if use_res else None)
        y, z = mqv.lin_fwd(d, wd, xd, **args, y=poison(out, yt), z=poison(out, BF16))
        ref = L.lin_fwd(w, x, bias if use_bias else None, r if use_res else None, act)
        check(y, ref["y"], f"y ({act})")
        check(z, ref["z"], f"z ({act})")
        y2, none = mqv.lin_fwd(d, wd, xd, **args, y_dtype=yt)
        assert none is None and torch.equal(y, y2)
    gz = stored(gy, "bf16")
    gzd = dev(gz, BF16)
    for gxt in (F32, BF16):
        gx = mqv.lin_dgrad(d, wd, gzd, gx=poison((P, Cin, N), gxt))
        check(gx, L.lin_dgrad(w, gz)["gx"], "gx")
    gw = mqv.lin_wgrad(d, gzd, xd, gw=poison((Cout, Cin), F32))
    check(gw, L.lin_wgrad(gz, x)["gw"], "gw")
    assert torch.equal(gx, mqv.lin_dgrad(d, wd, gzd)) and torch.equal(gw, mqv.lin_wgrad(d, gzd, xd))
    assert mqv.device_errors() == 0


@pytest.mark.parametrize("shape", LIN_PAIR + LIN_FEW, ids=shape_id)
def test_linear_layer_in_pairs_and_of_few_tokens(shape):
    test_linear_layer(shape)


def _integers(shape, limit, g):
    return torch.randint(-limit, limit + 1, shape, generator=g, device="cuda").to(BF16)


@pytest.mark.parametrize("shape", LIN_TOKENS + LIN_PIXELS + LIN_WIDE + LIN_LONG + LIN_PAIR + LIN_FEW + LIN_THIN,
                         ids=shape_id)
def test_products_of_integers_are_exact(shape):
    """Small integers: every sum of products, in any order, is an integer below
    2^24 that fp32 holds (9 times at most 12500 terms), so the results have one
    value, and a product left out or taken twice shows."""
    P, Cin, Cout, N = shape
    assert 9 * max(Cin, Cout, P * N) + 100 < 1 << 24
    g = torch.Generator(device="cuda").manual_seed(sum(shape))
    w, x, gz = _integers((Cout, Cin), 3, g), _integers((P, Cin, N), 3, g), _integers((P, Cout, N), 3, g)
    bias, res = _integers((Cout,), 50, g).float(), _integers((P, Cout, N), 50, g)
    d = mqv.lin_desc(*shape)
    # columns as rows: plain matrices, fp64
    xm, gm = (t.double().transpose(1, 2).reshape(P * N, -1) for t in (x, gz))
    rows = lambda t: t.double().transpose(1, 2).reshape(P * N, -1)  # noqa: E731
    zr = xm @ w.double().t()
    for dtype in (F32, BF16):
        y, z = mqv.lin_fwd(d, w, x, y=poison((P, Cout, N), dtype), save_z=True)
        assert torch.equal(rows(y), zr.to(dtype).double()) and torch.equal(rows(z), zr.to(BF16).double())
        y, _ = mqv.lin_fwd(d, w, x, bias=bias, residual=res.to(dtype))
        assert torch.equal(rows(y), (zr + bias.double() + rows(res)).to(dtype).double())
        gx = mqv.lin_dgrad(d, w, gz, gx=poison((P, Cin, N), dtype))
        assert torch.equal(rows(gx), (gm @ w.double()).to(dtype).double())
    gw = mqv.lin_wgrad(d, gz, x, gw=poison((Cout, Cin), F32))
    assert torch.equal(gw.double(), gm.t() @ xm)
    assert mqv.device_errors() == 0


@pytest.mark.parametrize("shape", [
    (596, 531, 3752, 1), (513, 3778, 546, 1), (134, 2456, 3168, 1), (245, 520, 1248, 4), (300, 585, 739, 8),
    (332, 152, 2040, 8), (1280, 1100, 1000, 1), (65, 1992, 2500, 1), (130, 72, 136, 1), (300, 264, 520, 32),
    (7, 16, 8, 4), (10, 24, 24, 8), (9, 48, 72, 20), (6, 65, 63, 16), (64, 4096, 256, 1), (33, 3001, 257, 1),
    (1, 2056, 40, 1), (3, 4099, 33, 1), (4, 136, 72, 1)], ids=shape_id)
def test_every_epilogue_of_integers_is_exact(shape):
    """Each of bias, residual and kept pre-activation with and without the
    others, without an activation and with ReLU, in fp32 and bfloat16: all
    integers that fp32 holds, so each result has one value."""
    P, Cin, Cout, N = shape
    g = torch.Generator(device="cuda").manual_seed(sum(shape))
    w, x = _integers((Cout, Cin), 3, g), _integers((P, Cin, N), 3, g)
    bias, res = _integers((Cout,), 50, g).float(), _integers((P, Cout, N), 50, g)
    sums = torch.einsum("oi,pin->pon", w.double(), x.double())
    for act in ("none", "relu"):
        d = mqv.lin_desc(*shape, act)
        for with_bias in (False, True):
            z = sums + bias.double()[:, None] if with_bias else sums
            a = z.clamp(min=0) if act == "relu" else z
            for with_res in (False, True):
                for dtype in (F32, BF16):
                    for keep in (False, True):
                        y, kept = mqv.lin_fwd(d, w, x, bias=bias if with_bias else None,
                                              residual=res.to(dtype) if with_res else None, y_dtype=dtype,
                                              y=poison((P, Cout, N), dtype), z=poison((P, Cout, N), BF16) if keep else None)
                        what = (act, with_bias, with_res, dtype, keep)
                        want = a + res.double() if with_res else a
                        assert torch.equal(y.double(), want.to(dtype).double()), what
                        assert not keep or torch.equal(kept.double(), z.to(BF16).double()), what
    assert mqv.device_errors() == 0


def _long_sums(op, M, K, N, dtype):
    """(result [M][N] of positive products over K, its value, both fp64): the
    case in which every step of a running sum that truncates loses."""
    g = torch.Generator(device="cuda").manual_seed(K + M)
    a, b = ((torch.rand((n, K), generator=g, device="cuda") * 0.5 + 0.5).to(BF16) for n in (M, N))
    ref = torch.zeros((M, N), dtype=torch.float64, device="cuda")
    for k in range(0, K, 8192):
        ref += a[:, k:k + 8192].double() @ b[:, k:k + 8192].double().t()
    d = {FWD: mqv.lin_desc(M, K, N), DGRAD: mqv.lin_desc(M, N, K), WGRAD: mqv.lin_desc(K, N, M)}[op]
    # the whole of K in one tile's accumulator, or in its runs
    assert "split" not in mqv.selftest_lin_instance(d, op, dtype)
    if op == FWD:
        y, _ = mqv.lin_fwd(d, b, a, y_dtype=dtype)
    elif op == DGRAD:
        y = mqv.lin_dgrad(d, b.t().contiguous(), a, gx_dtype=dtype)
    else:
        y = mqv.lin_wgrad(d, a.t().contiguous(), b.t().contiguous())
    assert mqv.device_errors() == 0
    return y.view(M, N).double(), ref


@pytest.mark.parametrize("op", [FWD, DGRAD, WGRAD])
@pytest.mark.parametrize("M,N", [(2048, 1280), (1999, 1283)])
def test_long_sums_in_fp32(op, M, N):
    """Within (64 + K / 512)·2^-24 of the sum: an accumulator takes 32 steps of
    16 products and loses at most a step of the sum, 2·2^-24, at each; the
    runs are added to nearest, a rounding of 2^-24 each."""
    K = 8192
    y, ref = _long_sums(op, M, K, N, F32)
    worst = float(((y - ref).abs() / ref).max())
    assert worst <= (64 + K / 512) * 2.0 ** -24


def test_long_sums_in_bfloat16():
    """Half a step of bfloat16, and what the fp32 sum may be off by: runs of
    32768 products, 2048 steps of at most 2·2^-24 of a sum that grows evenly,
    2048·2^-24 of it, and a rounding for each run."""
    K = 1 << 18
    y, ref = _long_sums(FWD, 2048, K, 1280, BF16)
    err = (2048 + K / 32768) * 2.0 ** -24 * ref
    half = torch.exp2(torch.floor(torch.log2(ref + err)) - 8)
    worst = float(((y - ref).abs() / (half + err)).max())
    assert worst <= 1


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("shape", [(1, 1, 1), (1, 9, 1), (5, 1003, 1), (300, 64, 1), (2100, 520, 1), (3, 5, 2),
                                   (49, 64, 16), (40, 33, 12), (600, 24, 64), (5, 3, 84), (2, 2, 5000), (3, 7, 2056)],
                         ids=shape_id)
def test_activation_gradient(shape, act):
    P, C, N = shape
    rng = np.random.default_rng(sum(shape))
    z = stored(rng.standard_normal(shape) * 3, "bf16")
    d = mqv.lin_desc(P, 8, C, N, act)
    for gt in (F32, BF16):
        gy = stored(rng.standard_normal(shape) * 1e-2, KIND[gt])
        gz, gb = mqv.lin_act_grad(d, dev(gy, gt), dev(z, BF16), gz=poison(shape, BF16), gbias=poison((C,), F32))
        ref = L.lin_act_grad(gy, z, act)
        check(gz, ref["gz"], "gz")
        check(gb, ref["gbias"], "gbias")
        gz2, gb2 = mqv.lin_act_grad(d, dev(gy, gt), dev(z, BF16))
        assert torch.equal(gz, gz2) and torch.equal(gb, gb2)
        gz3, none = mqv.lin_act_grad(d, dev(gy, gt), dev(z, BF16), bias_grad=False)
        assert none is None and torch.equal(gz, gz3)
    g = dev(gy, BF16)
    assert torch.equal(mqv.lin_act_grad(d, g, dev(z, BF16), gz=g)[0], gz)          # in place


def test_activation_extremes():
    """Far arguments: the activations and slopes reach their limits without
    a NaN, and a NaN passes through."""
    z = torch.tensor([0.0, -0.0, 80.0, -80.0, 1e30, -1e30, float("nan")], device="cuda").to(BF16).view(7, 1, 1)
    one = torch.ones((1, 1), dtype=BF16, device="cuda")
    gy = torch.ones((7, 1, 1), device="cuda")
    for act in ("relu", "gelu", "silu"):
        d = mqv.lin_desc(7, 1, 1, 1, act)
        y, _ = mqv.lin_fwd(d, one, z, y_dtype=F32)
        s, _ = mqv.lin_act_grad(d, gy, z)
        zf = z.double().cpu().numpy()[:6]
        # below -60 only exp(z) is left of the value: its argument z·log2(e), rounded
        # by U relative, is off by U·|z|·log2(e) absolute, so exp2 of it by U·|z|
        # relative (ln 2·log2 e = 1), plus at most 8 U for exp2, sum and division
        v = L.act_value(zf, act)
        check(y[:6], (v, 24 * L.U * np.abs(zf) * (zf > -60) + (np.abs(zf) + 8) * L.U * np.abs(v) * (zf > -1e9)), act)
        check(s[:6], (L.act_slope(zf, act), np.full_like(zf, 16 * L.U)), act)
        assert torch.isnan(y[6, 0, 0]) and (act == "relu" or torch.isnan(s[6, 0, 0]))


@pytest.mark.parametrize("shape", [(9, 8, 64, 1), (5, 8, 33, 1), (3, 8, 24, 16), (3, 8, 5, 3)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_relu_drops_gradients_where_it_is_off(shape, dtype):
    """An infinity or NaN in gy under an inactive unit reaches neither gz nor
    gbias; under an active one it does, in its own channel only."""
    P, _, C, N = shape
    d = mqv.lin_desc(*shape, "relu")
    rng = np.random.default_rng(11)
    z, gy = rng.standard_normal((2, P, C, N)).astype(np.float32)
    z[0, 0, 0], z[1, 1, 0], z[2, 2, 0], z[0, 3, 0] = -1.0, 0.0, -0.0, 1.0
    plain = gy.copy()
    gy[0, 0, 0], gy[1, 1, 0], gy[2, 2, 0] = np.inf, np.nan, -np.inf
    plain[0, 0, 0] = plain[1, 1, 0] = plain[2, 2, 0] = 5.0
    gz, gb = mqv.lin_act_grad(d, dev(gy, dtype), dev(z, BF16))
    pz, pb = mqv.lin_act_grad(d, dev(plain, dtype), dev(z, BF16))
    assert torch.isfinite(gz).all() and torch.equal(gz, pz) and torch.equal(gb, pb)
    gy[0, 3, 0] = np.inf
    gz, gb = mqv.lin_act_grad(d, dev(gy, dtype), dev(z, BF16))
    assert torch.isinf(gz[0, 3, 0]) and (~torch.isfinite(gz)).sum() == 1
    assert torch.isinf(gb[3]) and (~torch.isfinite(gb)).sum() == 1


def test_linear_layer_of_nothing():
    for N in (1, 16):
        d = mqv.lin_desc(0, 24, 40, N, "gelu")
        w = torch.ones((40, 24), dtype=BF16, device="cuda")
        x = torch.empty((0, 24, N), dtype=BF16, device="cuda")
        y, z = mqv.lin_fwd(d, w, x, save_z=True)
        gz, gb = mqv.lin_act_grad(d, y, z, gbias=poison((40,), F32))
        gx, gw = mqv.lin_dgrad(d, w, gz), mqv.lin_wgrad(d, gz, x, gw=poison((40, 24), F32))
        assert y.shape == (0, 40, N) and gx.shape == (0, 24, N) and not gb.any() and not gw.any()


@pytest.mark.parametrize("act", ["none", "silu"])
def test_activation_gradient_of_nothing_alone(act):
    g = torch.empty((0, 40, 16), device="cuda")
    z = g.to(BF16)
    gz, gb = mqv.lin_act_grad(mqv.lin_desc(0, 24, 40, 16, act), g, z, bias_grad=False)
    assert gz.shape == g.shape and gz.dtype == BF16 and gb is None


def test_linear_layer_residual_in_place():
    for shape in ((70, 128, 136, 1), (5, 64, 48, 16), (1, 64, 200, 1)):
        w, x, bias, res, _ = lin_inputs(shape)
        P, Cin, Cout, N = shape
        d = mqv.lin_desc(*shape)
        for t in (F32, BF16):
            r = dev(res, t)
            y, _ = mqv.lin_fwd(d, dev(w, BF16), dev(x, BF16), dev(bias), residual=r)
            assert y.dtype == t
            assert torch.equal(mqv.lin_fwd(d, dev(w, BF16), dev(x, BF16), dev(bias), residual=r, y=r)[0], y)


def test_infinite_inputs_stay_in_their_outputs():
    """An infinity or NaN in one token reaches that token's outputs only."""
    for shape in ((70, 128, 136, 1), (3, 64, 48, 16), (4, 64, 64, 1)):
        P, Cin, Cout, N = shape
        w, x, bias, _, _ = lin_inputs(shape)
        d = mqv.lin_desc(*shape)
        y, _ = mqv.lin_fwd(d, dev(w, BF16), dev(x, BF16), dev(bias))
        x[1, 5, 0], x[2, 0, 0] = np.nan, np.inf
        b, _ = mqv.lin_fwd(d, dev(w, BF16), dev(x, BF16), dev(bias))
        fine = torch.isfinite(b)
        assert not fine[1, :, 0].any() and not fine[2, :, 0].any() and (~fine).sum() == 2 * Cout
        assert torch.equal(b[fine], y[fine])


@pytest.mark.parametrize("shape", [(70, 128, 136, 1), (90, 73, 41, 1), (3, 64, 48, 16), (5, 33, 40, 12), (4, 31, 37, 7),
                                   (3, 4099, 33, 1), (4, 136, 72, 1), (596, 531, 3752, 1), (300, 585, 739, 8),
                                   (1280, 1100, 1000, 1), (65, 1992, 2500, 1)], ids=shape_id)
def test_special_values_stay_in_their_sums(shape):
    """A NaN or infinity in w, x or gz reaches the results whose sums have it,
    whatever lies beside it in memory, and no other, bit for bit."""
    P, Cin, Cout, N = shape
    w, x, bias, _, gy = lin_inputs(shape)
    wd, xd, bd, gd = dev(w, BF16), dev(x, BF16), dev(bias), dev(gy, BF16)
    d = mqv.lin_desc(*shape)
    y, gx, gw = mqv.lin_fwd(d, wd, xd, bd)[0], mqv.lin_dgrad(d, wd, gd), mqv.lin_wgrad(d, gd, xd)
    # the last values of a row, and the first of the next
    w2, x2, g2 = wd.clone(), xd.clone(), gd.clone()
    w2[1, Cin - 1], w2[2, 0] = float("nan"), float("inf")
    x2[P // 2, Cin - 1, N - 1], x2[P - 1, 0, 0] = float("inf"), float("nan")
    g2[P // 2, Cout - 1, N - 1], g2[P - 1, 0, 0] = float("nan"), float("-inf")
    cols = torch.zeros((P, N), dtype=torch.bool, device="cuda")
    cols[P // 2, N - 1] = cols[P - 1, 0] = True

    def spoiled(got, want, where):
        """where: of got's shape, true where a value has to be spoiled."""
        where = where.expand(got.shape)
        assert not torch.isfinite(got[where]).any() and torch.equal(got[~where], want[~where])

    def channels(n, *which):
        m = torch.zeros(n, dtype=torch.bool, device="cuda")
        m[list(which)] = True
        return m

    spoiled(mqv.lin_fwd(d, w2, xd, bd)[0], y, channels(Cout, 1, 2)[:, None])
    spoiled(mqv.lin_dgrad(d, w2, gd), gx, channels(Cin, 0, Cin - 1)[:, None])
    spoiled(mqv.lin_fwd(d, wd, x2, bd)[0], y, cols[:, None])
    spoiled(mqv.lin_dgrad(d, wd, g2), gx, cols[:, None])
    spoiled(mqv.lin_wgrad(d, gd, x2), gw, channels(Cin, 0, Cin - 1))
    spoiled(mqv.lin_wgrad(d, g2, xd), gw, channels(Cout, 0, Cout - 1)[:, None])
    assert mqv.device_errors() == 0


# ----------------------------------- streams, graphs, workspaces, refusals

def _block(d1, d2, ln, t, x, **kw):
    """Pre-norm MLP with residual, forward and backward, every pass of it."""
    h, mean, rstd = mqv.ln_fwd(ln, x, t["gamma"], t["beta"], y_dtype=BF16, **kw)
    a, z = mqv.lin_fwd(d1, t["w1"], h, bias=t["b1"], save_z=True, **kw)
    y, _ = mqv.lin_fwd(d2, t["w2"], a, bias=t["b2"], residual=x, **kw)
    gy = t["gy"]
    g2, gb2 = mqv.lin_act_grad(d2, gy, **kw)
    ga, gw2 = mqv.lin_dgrad(d2, t["w2"], g2, **kw), mqv.lin_wgrad(d2, g2, a, **kw)
    g1, gb1 = mqv.lin_act_grad(d1, ga, z, **kw)
    gh, gw1 = mqv.lin_dgrad(d1, t["w1"], g1, **kw), mqv.lin_wgrad(d1, g1, h, **kw)
    gx, gg, gb = mqv.ln_bwd(ln, gh, x, mean, rstd, t["gamma"], **kw)
    return {"y": y, "gb2": gb2, "gw2": gw2, "gb1": gb1, "gw1": gw1, "gx": gx, "ggamma": gg, "gbeta": gb}


def _block_inputs(P, C, H, N, seed=0):
    rng = np.random.default_rng(seed)
    t = {"w1": dev(rng.standard_normal((H, C)) * (2 / C) ** 0.5, BF16), "b1": dev(rng.standard_normal(H) * 0.1),
         "w2": dev(rng.standard_normal((C, H)) * (1 / H) ** 0.5, BF16), "b2": dev(rng.standard_normal(C) * 0.1),
         "gamma": dev(rng.standard_normal(C) * 0.2 + 1), "beta": dev(rng.standard_normal(C) * 0.2),
         "gy": dev(rng.standard_normal((P, C, N)) * 1e-2, BF16)}
    x = dev(rng.standard_normal((P, C, N)), BF16)
    return t, x, mqv.lin_desc(P, C, H, N, "gelu"), mqv.lin_desc(P, H, C, N), mqv.ln_desc(P, C, N)


def _block_fp64(t, x):
    p = {k: v.double().requires_grad_() for k, v in t.items() if k != "gy"}
    xx = x.double()
    xx.requires_grad_()
    m = xx.mean(1, keepdim=True)
    v = (xx - m).square().mean(1, keepdim=True)
    h = (xx - m) / (v + 1e-5).sqrt() * p["gamma"][:, None] + p["beta"][:, None]
    z = torch.einsum("oi,pin->pon", p["w1"], h) + p["b1"][:, None]
    y = torch.einsum("oi,pin->pon", p["w2"], torch.nn.functional.gelu(z)) + p["b2"][:, None]
    (y * t["gy"].double()).sum().backward()
    return {"y": y.detach() + x.double(), "gb2": p["b2"].grad, "gw2": p["w2"].grad, "gb1": p["b1"].grad,
            "gw1": p["w1"].grad, "gx": xx.grad, "ggamma": p["gamma"].grad, "gbeta": p["beta"].grad}


BLOCKS = [(200, 96, 264, 1), (1, 64, 128, 1), (37, 33, 70, 1), (25, 64, 128, 16), (9, 24, 56, 12)]


@pytest.mark.parametrize("shape", BLOCKS, ids=shape_id)
def test_block_of_norm_and_linear_layers(shape):
    """The passes chained as a block uses them.  bfloat16 intermediates (h, a,
    z, ga, g1, gh: at most six roundings of 2^-8 on any path, each entering a
    sum of random signs) leave the outputs within 6·2^-8 of the fp64 block in
    the 2-norm."""
    t, x, d1, d2, ln = _block_inputs(*shape)
    got, ref = _block(d1, d2, ln, t, x), _block_fp64(t, x)
    for k, v in got.items():
        off = (v.double() - ref[k]).norm() / ref[k].norm()
        assert off < 6 * 2 ** -8, f"{k}: {off:.3g}"
    assert mqv.device_errors() == 0


@pytest.mark.parametrize("shape", BLOCKS, ids=shape_id)
def test_block_on_another_stream_and_in_a_graph(shape):
    t, x, d1, d2, ln = _block_inputs(*shape)
    want = {k: v.clone() for k, v in _block(d1, d2, ln, t, x).items()}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = _block(d1, d2, ln, t, x, stream=s)
    s.synchronize()
    for k in want:
        assert torch.equal(got[k], want[k]), k
    # two graphs, replayed side by side on two streams, each several times
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = _block(d1, d2, ln, t, x)
        graphs.append((g, out, torch.cuda.Stream()))
    for g, out, st in graphs:
        for v in out.values():
            v.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for g, out, st in graphs:
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for g, out, st in graphs:
        for k in want:
            assert torch.equal(out[k], want[k]), k
    # new inputs reach a replay
    x.mul_(-1.5)
    graphs[0][0].replay()
    torch.cuda.synchronize()
    fresh = _block(d1, d2, ln, t, x)
    for k in want:
        assert torch.equal(graphs[0][1][k], fresh[k]), k


_FIRST = """
import torch, microscaling_quantized_convolution_b200 as mqv
P, C, H, N = {shape}
x, w = torch.ones((P, C, N), device="cuda"), torch.ones((H, C), dtype=torch.bfloat16, device="cuda")
ln, d = mqv.ln_desc(P, C, N), mqv.lin_desc(P, C, H, N, "gelu")
x[:, 0] = 3.0
torch.cuda.synchronize()
def passes():
    h, mean, rstd = mqv.ln_fwd(ln, x, y_dtype=torch.bfloat16)
    y, z = mqv.lin_fwd(d, w, h, save_z=True)
    gz, gb = mqv.lin_act_grad(d, y, z)
    gx = mqv.lin_dgrad(d, w, gz)
    return (h, y, z, gz, gb, gx, mqv.lin_wgrad(d, gz, h)) + mqv.ln_bwd(ln, gx, x, mean, rstd)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = passes()
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, passes(), strict=True))
assert mqv.device_errors() == 0
"""


@pytest.mark.parametrize("shape", [(300, 72, 136, 1), (9, 24, 56, 12), (2048, 1024, 2048, 1)], ids=shape_id)
def test_first_calls_of_a_process_are_captured(shape):
    """Nothing that a first call sets up (kernel attributes, the error word, the
    tensor map encoder) is refused under capture."""
    run = subprocess.run([sys.executable, "-c", _FIRST.format(shape=shape)], cwd=ROOT, capture_output=True, text=True,
                         timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]


def test_block_from_several_host_threads():
    """Threads with a stream each, calling at once, get what one alone gets."""
    jobs = [_block_inputs(*shape, seed=i) for i, shape in enumerate(BLOCKS)]
    want = [{k: v.clone() for k, v in _block(d1, d2, ln, t, x).items()} for t, x, d1, d2, ln in jobs]
    torch.cuda.synchronize()

    def work(i):
        t, x, d1, d2, ln = jobs[i]
        s = torch.cuda.Stream()
        outs = [_block(d1, d2, ln, t, x, stream=s) for _ in range(8)]
        s.synchronize()
        return outs

    with ThreadPoolExecutor(len(jobs)) as pool:
        for ref, outs in zip(want, pool.map(work, range(len(jobs)))):
            for out in outs:
                for k in ref:
                    assert torch.equal(out[k], ref[k]), k
    assert mqv.device_errors() == 0


# ------------------------------------------------- offsets past 32 bits
#
# Tensors of more than 2^31 elements, zero but for their last positions: those
# are checked against the definition, what lies before them against zero.

def _tail(shape, k, rng, scale=1.0):
    """(device tensor of zeros but for its last k positions, those as stored)."""
    v = stored(rng.standard_normal((k, *shape[1:])) * scale, "bf16")
    t = torch.zeros(shape, dtype=BF16, device="cuda")
    t[-k:] = dev(v, BF16)
    return t, v


def _zero_before(t, k):
    return not any(c.any() for c in t[:-k].split(1 << max(0, 28 - (t[0].numel() - 1).bit_length())))


@pytest.mark.parametrize("shape", [(525000, 4096, 1), (2150000, 1001, 1), (33600, 1000, 64), (240000, 1001, 9)], ids=shape_id)
def test_layer_norm_past_32_bits(shape):
    P, C, N = shape
    assert P * C * N > 1 << 31
    rng, k = np.random.default_rng(5), 2
    (x, xv), (gy, gyv) = _tail(shape, k, rng), _tail(shape, k, rng, 1e-2)
    gamma = stored(rng.standard_normal(C) * 0.3 + 1, "f32")
    d = mqv.ln_desc(P, C, N)
    y, mean, rstd = mqv.ln_fwd(d, x, dev(gamma))
    ref = L.ln_fwd(xv, gamma, None, EPS)
    for got, name in ((y, "y"), (mean, "mean"), (rstd, "rstd")):
        check(got[-k:], ref[name], name)
    assert _zero_before(y, k) and _zero_before(mean, k)
    gx, gg, gb = mqv.ln_bwd(d, gy, x, mean, rstd, dev(gamma), gx=y)
    ref = L.ln_bwd(gyv, xv, mean[-k:].double().cpu().numpy(), rstd[-k:].double().cpu().numpy(), gamma)
    check(gx[-k:], ref["gx"], "gx")
    check(gg, ref["ggamma"], "ggamma")
    check(gb, ref["gbeta"], "gbeta")
    assert _zero_before(gx, k)


@pytest.mark.parametrize("shape", [(2100000, 1024, 16, 1), (2150000, 1001, 24, 1), (33600, 1000, 8, 64),
                                   (240000, 1001, 5, 9)], ids=shape_id)
def test_linear_layer_past_32_bits(shape):
    """Many inputs to few outputs, and the same few back to many."""
    P, big, small, N = shape
    assert P * big * N > 1 << 31
    rng, k = np.random.default_rng(6), 2
    x, xv = _tail((P, big, N), k, rng)
    g, gv = _tail((P, small, N), k, rng)
    w = stored(rng.standard_normal((small, big)) * 0.03, "bf16")
    d = mqv.lin_desc(P, big, small, N)
    y, _ = mqv.lin_fwd(d, dev(w, BF16), x, y_dtype=F32)
    check(y[-k:], L.lin_fwd(w, xv, None, None, "none")["y"], "y")
    assert _zero_before(y, k)
    check(mqv.lin_wgrad(d, g, x), L.lin_wgrad(gv, xv)["gw"], "gw")
    out = mqv.lin_dgrad(d, dev(w, BF16), g)
    check(out[-k:], L.lin_dgrad(w, gv)["gx"], "gx")
    assert _zero_before(out, k)
    # the other way: x is the output side
    d, wt = mqv.lin_desc(P, small, big, N, "relu"), np.ascontiguousarray(w.T)
    out, _ = mqv.lin_fwd(d, dev(wt, BF16), g, residual=x, y=out)
    check(out[-k:], L.lin_fwd(wt, gv, None, xv, "relu")["y"], "y")
    assert _zero_before(out, k)
    check(mqv.lin_wgrad(d, x, g), L.lin_wgrad(xv, gv)["gw"], "gw")
    z = out
    zv = z[-k:].double().cpu().numpy()
    gz, gb = mqv.lin_act_grad(d, x, z, gz=x)
    ref = L.lin_act_grad(xv, zv, "relu")
    check(gz[-k:], ref["gz"], "gz")
    check(gb, ref["gbias"], "gbias")
    assert _zero_before(gz, k) and mqv.device_errors() == 0


def test_given_workspaces_and_ragged_pointers():
    shape = (90, 72, 136, 1)
    w, x, bias, _, gy = lin_inputs(shape)
    d = mqv.lin_desc(*shape, "silu")
    wd, xd, gd = dev(w, BF16), dev(x, BF16), dev(gy, BF16)
    for op, call in ((mqv.OP_FWD, lambda ws: mqv.lin_fwd(d, wd, xd, ws=ws)[0]),
                     (mqv.OP_DGRAD, lambda ws: mqv.lin_dgrad(d, wd, gd, ws=ws)),
                     (mqv.OP_WGRAD, lambda ws: mqv.lin_wgrad(d, gd, xd, ws=ws)),
                     (mqv.OP_ACT_GRAD, lambda ws: mqv.lin_act_grad(d, gd, gd, ws=ws)[1])):
        need = mqv.lin_workspace_bytes(d, op)
        want = call(None)
        ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
        assert torch.equal(call(ws[:need]), want)
        assert (ws[need:] == 255).all()
        if need:
            with pytest.raises(mqv.MqvError):
                call(ws[:need - 1])
            with pytest.raises(mqv.MqvError):
                call(ws[8:])
    big = torch.zeros(90 * 72 + 4, dtype=BF16, device="cuda")
    with pytest.raises(mqv.MqvError):                              # 8 bytes off a 16-byte boundary
        mqv.lin_fwd(d, wd, big[4:])


def _guarded(call, need, kind):
    """call(ws) with a workspace of exactly `need` bytes between guard bytes,
    all of them NaN patterns: the same result as with the call's own, twice
    (the second time over what the first left), the guards untouched; a
    shorter and a misaligned one are refused."""
    assert need > 0 and need % 256 == 0, kind
    want = [t.clone() for t in call(None)]
    buf = torch.full((need + 2048,), 255, dtype=torch.uint8, device="cuda")
    ws = buf[1024:1024 + need]
    for _ in range(2):
        got = call(ws)
        assert all(torch.equal(a, b) for a, b in zip(got, want, strict=True)), kind
        assert (buf[:1024] == 255).all() and (buf[1024 + need:] == 255).all(), kind
    for bad in (buf[1024:1024 + need - 1], buf[1032:1032 + need]):
        with pytest.raises(mqv.MqvError):
            call(bad)


@pytest.mark.parametrize("shape,ops", [
    # K split, whole vectors
    ((64, 4096, 256, 1), (FWD,)), ((4100, 136, 72, 1), (WGRAD,)), ((500, 520, 136, 16), (WGRAD,)),
    # copies of operands with unaligned rows
    ((129, 257, 255, 1), (FWD, WGRAD, DGRAD)), ((90, 1003, 1001, 1), (FWD, WGRAD, DGRAD)),
    # both, in one tile or another
    ((33, 3001, 257, 1), (FWD, WGRAD, DGRAD)), ((2570, 3076, 161, 1), (FWD, WGRAD, DGRAD)),
    ((70, 2000, 136, 7), (FWD, WGRAD, DGRAD)), ((200, 1992, 72, 12), (FWD, WGRAD, DGRAD)),
    ((600, 128, 136, 20), (FWD, WGRAD, DGRAD))], ids=str)
def test_product_workspaces_of_their_exact_size(shape, ops):
    P, Cin, Cout, N = shape
    w, x, bias, res, gy = lin_inputs(shape)
    wd, xd, bd, rd, gd = dev(w, BF16), dev(x, BF16), dev(bias), dev(res), dev(gy, BF16)
    d = mqv.lin_desc(*shape, "silu")
    calls = {FWD: lambda ws: mqv.lin_fwd(d, wd, xd, bias=bd, residual=rd, save_z=True, ws=ws),
             DGRAD: lambda ws: (mqv.lin_dgrad(d, wd, gd, ws=ws),), WGRAD: lambda ws: (mqv.lin_wgrad(d, gd, xd, ws=ws),)}
    for op in ops:
        _guarded(calls[op], mqv.lin_workspace_bytes(d, op), (shape, op))
    assert mqv.device_errors() == 0


@pytest.mark.parametrize("shape", [(5, 1023, 1), (700, 136, 1), (3, 20, 12), (4, 128, 64), (2, 2048, 16), (1, 1, 1)],
                         ids=shape_id)
def test_gradient_workspaces_of_their_exact_size(shape):
    P, C, N = shape
    x, gamma, _, gy = ln_inputs(shape)
    xd, gd, gyd = dev(x), dev(gamma), dev(gy)
    ln, lin = mqv.ln_desc(*shape), mqv.lin_desc(P, 8, C, N, "gelu")
    _, mean, rstd = mqv.ln_fwd(ln, xd, gd)
    _guarded(lambda ws: mqv.ln_bwd(ln, gyd, xd, mean, rstd, gd, ws=ws), mqv.ln_bwd_workspace_bytes(ln), shape)
    z = xd.to(BF16)
    _guarded(lambda ws: mqv.lin_act_grad(lin, gyd, z, ws=ws), mqv.lin_workspace_bytes(lin, mqv.OP_ACT_GRAD), shape)


def test_binding_refusals():
    d, ln = mqv.lin_desc(4, 16, 24, 1, "gelu"), mqv.ln_desc(4, 16)
    w = torch.zeros((24, 16), dtype=BF16, device="cuda")
    x, y = torch.zeros((4, 16), dtype=BF16, device="cuda"), torch.zeros((4, 24), dtype=BF16, device="cuda")
    s, f = torch.zeros(4, device="cuda"), torch.zeros((4, 16), device="cuda")
    short = torch.zeros(5, dtype=BF16, device="cuda")
    bad = [
        lambda: mqv.lin_fwd(d, w, short), lambda: mqv.lin_fwd(d, short, x), lambda: mqv.lin_fwd(d, w, f),
        lambda: mqv.lin_fwd(d, w, x.t()), lambda: mqv.lin_fwd(d, w, x, bias=s), lambda: mqv.lin_fwd(d, w, x, bias=y),
        lambda: mqv.lin_fwd(d, w, x, residual=y, y_dtype=F32), lambda: mqv.lin_fwd(d, w, x, y=short),
        lambda: mqv.lin_fwd(d, w, x, z=short), lambda: mqv.lin_fwd(d, w, x, y_dtype=torch.float16),
        lambda: mqv.lin_fwd(d, w.cpu(), x), lambda: mqv.lin_fwd(d, w, x, y=y, y_dtype=F32),
        lambda: mqv.lin_act_grad(d, y), lambda: mqv.lin_act_grad(d, y, short), lambda: mqv.lin_act_grad(d, short, y),
        lambda: mqv.lin_act_grad(d, y, y, gbias=s), lambda: mqv.lin_dgrad(d, w, short),
        lambda: mqv.lin_dgrad(d, w, y, gx=short), lambda: mqv.lin_wgrad(d, short, x), lambda: mqv.lin_wgrad(d, y, short),
        lambda: mqv.lin_wgrad(d, y, x, gw=w), lambda: mqv.ln_fwd(ln, short), lambda: mqv.ln_fwd(ln, x.half()),
        lambda: mqv.ln_fwd(ln, x, gamma=s), lambda: mqv.ln_fwd(ln, x, mean=short),
        lambda: mqv.ln_bwd(ln, x, x, s, short), lambda: mqv.ln_bwd(ln, short, x, s, s),
        lambda: mqv.ln_bwd(ln, x, x, s, s, ws=torch.zeros(4096)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    with pytest.raises(mqv.MqvError):                              # two outputs in one buffer
        mqv.ln_fwd(ln, x, mean=s, rstd=s)
    assert mqv.device_errors() == 0
