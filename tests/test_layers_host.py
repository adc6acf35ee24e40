"""Layer norm and linear layer without a GPU: the oracle's gradients against
central differences and against torch's fp64 autograd, workspace sizes, and
every refusal of the C ABI and the binding, which come before any launch."""
import ctypes
import os
import re
import subprocess
import sys

import numpy as np
import pytest
import torch

import microscaling_quantized_convolution_b200 as mqv
from microscaling_quantized_convolution_b200 import build as mqv_build
from oracle import layers_oracle as L
from tests.conftest import ROOT
from tests.layers_cases import (LIN_FEW, LIN_LONG, LIN_PAIR, LIN_PIXELS, LIN_TOKENS, LIN_WIDE, LN_ROWS, LN_TILES,
                                LN_WIDE_TILES)


@pytest.fixture(scope="module", autouse=True)
def lib():
    mqv_build.build()
    return mqv.lib()


# ------------------------------------------------------- the oracle itself

def _difference(f, x, i, h=1e-5):
    a, b = x.copy(), x.copy()
    a.flat[i] += h
    b.flat[i] -= h
    return (f(a) - f(b)) / (2 * h)


@pytest.mark.parametrize("shape", [(3, 6, 1), (2, 5, 4)])
def test_ln_gradients_against_differences(shape):
    rng = np.random.default_rng(1)
    x, gy = rng.standard_normal(shape), rng.standard_normal(shape)
    gamma, beta = rng.standard_normal(shape[1]), rng.standard_normal(shape[1])

    def loss(x=x, gamma=gamma, beta=beta):
        return float((L.ln_fwd(x, gamma, beta, 1e-3)["y"][0] * gy).sum())

    f = L.ln_fwd(x, gamma, beta, 1e-3)
    b = L.ln_bwd(gy, x, f["mean"][0], f["rstd"][0], gamma)
    for i in range(x.size):
        assert abs(_difference(lambda t: loss(x=t), x, i) - b["gx"][0].flat[i]) < 1e-7
    for i in range(shape[1]):
        assert abs(_difference(lambda t: loss(gamma=t), gamma, i) - b["ggamma"][0][i]) < 1e-7
        assert abs(_difference(lambda t: loss(beta=t), beta, i) - b["gbeta"][0][i]) < 1e-7


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("N", [1, 3])
def test_lin_gradients_against_differences(act, N):
    rng = np.random.default_rng(2)
    w, x = rng.standard_normal((4, 5)), rng.standard_normal((3, 5, N))
    bias, gy, res = rng.standard_normal(4), rng.standard_normal((3, 4, N)), rng.standard_normal((3, 4, N))

    def loss(w=w, x=x, bias=bias):
        return float((L.lin_fwd(w, x, bias, res, act)["y"][0] * gy).sum())

    z = L.lin_fwd(w, x, bias, res, act)["z"][0]
    a = L.lin_act_grad(gy, z, act)
    gx, gw = L.lin_dgrad(w, a["gz"][0])["gx"][0], L.lin_wgrad(a["gz"][0], x)["gw"][0]
    for i in range(x.size):
        assert abs(_difference(lambda t: loss(x=t), x, i) - gx.flat[i]) < 1e-7
    for i in range(w.size):
        assert abs(_difference(lambda t: loss(w=t), w, i) - gw.flat[i]) < 1e-7
    for i in range(4):
        assert abs(_difference(lambda t: loss(bias=t), bias, i) - a["gbias"][0][i]) < 1e-7


def test_oracle_matches_torch_autograd():
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.standard_normal((6, 10))).requires_grad_()
    gamma = torch.from_numpy(rng.standard_normal(10)).requires_grad_()
    beta = torch.from_numpy(rng.standard_normal(10)).requires_grad_()
    gy = torch.from_numpy(rng.standard_normal((6, 10)))
    y = torch.nn.functional.layer_norm(x, (10,), gamma, beta, 1e-5)
    y.backward(gy)
    f = L.ln_fwd(x.detach().numpy()[:, :, None], gamma.detach().numpy(), beta.detach().numpy(), 1e-5)
    b = L.ln_bwd(gy.numpy()[:, :, None], x.detach().numpy()[:, :, None], f["mean"][0], f["rstd"][0],
                 gamma.detach().numpy())
    assert np.allclose(f["y"][0][:, :, 0], y.detach().numpy(), atol=1e-12)
    assert np.allclose(b["gx"][0][:, :, 0], x.grad.numpy(), atol=1e-12)
    assert np.allclose(b["ggamma"][0], gamma.grad.numpy(), atol=1e-12)
    z = torch.from_numpy(rng.standard_normal(1000) * 4)
    for act, f in (("gelu", torch.nn.functional.gelu), ("silu", torch.nn.functional.silu), ("relu", torch.relu)):
        assert np.allclose(L.act_value(z.numpy(), act), f(z).numpy(), atol=1e-14)


# --------------------------------------------------------- sizes, refusals

@pytest.mark.parametrize("shape", LN_ROWS + LN_TILES + [(0, 5, 1), (0, 64, 16)])
def test_ln_accepts_every_test_shape(shape):
    b = mqv.ln_bwd_workspace_bytes(mqv.ln_desc(*shape))
    assert b % 256 == 0 and (b > 0 or shape[0] == 0)


@pytest.mark.parametrize("shape", LIN_TOKENS + LIN_PIXELS + LIN_WIDE + LIN_LONG + [(0, 5, 6, 1), (0, 64, 32, 16)])
def test_lin_accepts_every_test_shape(shape):
    d = mqv.lin_desc(*shape)
    for op in (mqv.OP_FWD, mqv.OP_WGRAD, mqv.OP_DGRAD, mqv.OP_ACT_GRAD):
        assert mqv.lin_workspace_bytes(d, op) >= 0


@pytest.mark.parametrize("kw", [dict(P=-1), dict(C=0), dict(N=0), dict(C=-4), dict(eps=-1.0), dict(eps=float("nan")),
                                dict(eps=float("inf")), dict(C=16385), dict(P=1 << 31), dict(P=1 << 20, N=1 << 12),
                                dict(P=(1 << 31) - 1, C=1024)])
def test_bad_ln_descriptors(kw):
    with pytest.raises(mqv.MqvError) as e:
        mqv.ln_bwd_workspace_bytes(mqv.ln_desc(**{**dict(P=4, C=8, N=1), **kw}))
    assert e.value.status in (1, 2)


@pytest.mark.parametrize("kw", [dict(P=-1), dict(Cin=0), dict(Cout=0), dict(N=0), dict(act=9), dict(P=1 << 31),
                                dict(Cin=1 << 25), dict(P=1 << 30, Cout=2048), dict(N=1 << 31)])
def test_bad_lin_descriptors(kw):
    with pytest.raises(mqv.MqvError) as e:
        mqv.lin_workspace_bytes(mqv.lin_desc(**{**dict(P=4, Cin=8, Cout=8, N=1), **kw}), mqv.OP_FWD)
    assert e.value.status in (1, 2)


@pytest.mark.parametrize("op", [mqv.OP_FWD, mqv.OP_WGRAD, mqv.OP_DGRAD, mqv.OP_ACT_GRAD])
def test_weights_whose_tiles_pass_32_bits(op):
    """More weights than an int counts tiles of are refused, whatever P is."""
    for P, N in ((0, 1), (1, 1), (2, 4)):
        with pytest.raises(mqv.MqvError) as e:
            mqv.lin_workspace_bytes(mqv.lin_desc(P, 1 << 24, 1 << 24, N), op)
        assert e.value.status in (1, 2)
        assert mqv.lin_workspace_bytes(mqv.lin_desc(P, 1 << 20, 1 << 16, N), op) >= 0


def test_reserved_fields_and_unknown_ops():
    d = mqv.lin_desc(4, 8, 8)
    with pytest.raises(mqv.MqvError):
        mqv.lin_workspace_bytes(d, mqv.OP_FWD_BLOCKSCALED)
    d.reserved = 1
    with pytest.raises(mqv.MqvError):
        mqv.lin_workspace_bytes(d, mqv.OP_FWD)
    n = mqv.ln_desc(4, 8)
    n.reserved = 1
    with pytest.raises(mqv.MqvError):
        mqv.ln_bwd_workspace_bytes(n)
    assert mqv.lib().mqv_lin_workspace_size(None, mqv.OP_FWD, None) == 1
    assert mqv.lib().mqv_lin_workspace_size(ctypes.byref(mqv.lin_desc(4, 8, 8)), mqv.OP_FWD, None) == 1
    assert mqv.lib().mqv_ln_bwd_workspace_size(ctypes.byref(mqv.ln_desc(4, 8)), None) == 1


# ------------------------------------------------------- kernel instances

def _ln_instances():
    """The instances that the dispatch can launch, from its source, as the test
    hook names them (the last parameter, EXACT, is false where not given)."""
    params = {"launch_ln_fwd_rows": 6, "launch_ln_bwd_rows": 6, "launch_ln_fwd_tiles": 4, "launch_ln_bwd_tiles": 5}
    with open(os.path.join(mqv_build.CSRC, "mqv_layers_api.cu")) as f:
        calls = re.findall(r"(launch_ln_\w+)<([\w, ]+)>\(a, pl, to\)", f.read())
    out = set()
    for name, args in calls:
        args = [{"true": "1", "false": "0"}.get(a, a) for a in args.split(", ")]
        out.add(f"{name}<{', '.join(args + ['0'] * (params[name] - len(args)))}>")
    assert len(out) > 20
    return out


def test_every_layer_norm_instance_is_for_some_shape():
    reached = set()
    for N in (1, 2, 3, 4, 8, 12, 16, 64):
        for C in range(1, 16385, 1 if N == 1 else 61 if N > 4 else 97):
            reached |= {mqv.selftest_ln_instance(mqv.ln_desc(2, c, N), bwd) for c in {C, min(16384, -(-C // 64) * 64)}
                        for bwd in (False, True)}
    assert reached == _ln_instances()


def test_gpu_shapes_reach_every_layer_norm_instance():
    reached = {mqv.selftest_ln_instance(mqv.ln_desc(*s), bwd) for s in LN_ROWS + LN_TILES + LN_WIDE_TILES
               for bwd in (False, True)}
    assert reached == _ln_instances()


def test_gpu_shapes_reach_every_product_instance():
    """Every tile, with outputs by TMA and without, in one run of K and in
    several, whole and split; the pair's tile in each pass, for tokens and for
    pixels.  A change of the tile model that moves them fails here."""
    reached, passes = set(), set()
    for s in LIN_TOKENS + LIN_PIXELS + LIN_WIDE + LIN_LONG + LIN_PAIR + LIN_FEW:
        for op in (mqv.OP_FWD, mqv.OP_WGRAD, mqv.OP_DGRAD):
            for t in (torch.float32, torch.bfloat16):
                name = mqv.selftest_lin_instance(mqv.lin_desc(*s), op, t)
                reached.add(name.replace(" copy a", "").replace(" copy b", ""))
                if "gemm_tc_kernel<256" in name:
                    passes.add((name.split(">")[0], "split" in name, op, s[3] > 1))
    for p, r in ((1, 1), (2, 1), (3, 2), (4, 2)):
        assert {f"few_tokens_kernel<{p}, {r}, {odd}>" for odd in (0, 1)} <= reached
    for tile in ("64, 0", "128, 0", "256, 1"):
        for fast in (0, 1):
            for runs in (0, 1):
                assert f"gemm_tc_kernel<{tile}, {fast}, {runs}>" in reached, (tile, fast, runs)
                assert any(f"gemm_tc_kernel<{tile}, {fast}, {runs}> split_sum_kernel<{v}>" in reached for v in (1, 4))
    for op in (mqv.OP_FWD, mqv.OP_WGRAD, mqv.OP_DGRAD):
        for pixels in (False, True):
            for fast in (0, 1):
                for runs in (0, 1):
                    assert any((f"gemm_tc_kernel<256, 1, {fast}, {runs}", split, op, pixels) in passes
                               for split in (False, True)), (op, pixels, fast, runs)


def test_instance_hooks_refuse_what_the_calls_refuse():
    assert mqv.selftest_ln_instance(mqv.ln_desc(0, 64)) == "" == mqv.selftest_lin_instance(mqv.lin_desc(0, 8, 8), mqv.OP_FWD)
    with pytest.raises(mqv.MqvError):
        mqv.selftest_ln_instance(mqv.ln_desc(1, 16385))
    with pytest.raises(mqv.MqvError):
        mqv.selftest_lin_instance(mqv.lin_desc(1, 0, 8), mqv.OP_FWD)
    with pytest.raises(mqv.MqvError):
        mqv.selftest_lin_instance(mqv.lin_desc(1, 8, 8), mqv.OP_ACT_GRAD)
    text = ctypes.create_string_buffer(b"untouched", 12)
    assert mqv.lib().mqv_selftest_ln_instance(ctypes.byref(mqv.ln_desc(1, 8)), 0, text, 0) == 1
    assert mqv.lib().mqv_selftest_ln_instance(ctypes.byref(mqv.ln_desc(1, 8)), 0, None, 12) == 1
    assert text.value == b"untouched"
    assert mqv.lib().mqv_selftest_ln_instance(ctypes.byref(mqv.ln_desc(1, 8)), 0, text, 4) == 0
    assert text.value == b"lau"                                   # cut off within its size


@pytest.mark.parametrize("bad", [0, -1, (1 << 32) + 1])
def test_warp_wait_limit_is_validated(bad):
    assert mqv.lib().mqv_selftest_warp_wait_timeout(bad, None) == 1


# addresses of pretend buffers, far enough apart for the shapes used here;
# each call below is refused before anything is launched
A = [1 << 20 << i for i in range(10)]


def _ln_fwd(d, x=A[0], xt=1, gamma=A[1], beta=A[2], y=A[3], yt=1, mean=A[4], rstd=A[5]):
    return mqv.lib().mqv_ln_fwd(ctypes.byref(d), x, xt, gamma, beta, y, yt, mean, rstd, None)


def _ln_bwd(d, gy=A[0], gyt=1, x=A[1], xt=1, mean=A[2], rstd=A[3], gamma=A[4], gx=A[5], gxt=1, gg=A[6], gb=A[7],
            ws=A[8], wsn=1 << 20):
    return mqv.lib().mqv_ln_bwd(ctypes.byref(d), gy, gyt, x, xt, mean, rstd, gamma, gx, gxt, gg, gb, ws, wsn, None)


def _lin_fwd(d, w=A[0], x=A[1], bias=A[2], res=A[3], z=A[4], y=A[5], yt=1, ws=A[6], wsn=1 << 20):
    return mqv.lib().mqv_lin_fwd(ctypes.byref(d), w, x, bias, res, z, y, yt, ws, wsn, None)


def _lin_act_grad(d, gy=A[0], gyt=1, z=A[1], gz=A[2], gb=A[3], ws=A[4], wsn=1 << 20):
    return mqv.lib().mqv_lin_act_grad(ctypes.byref(d), gy, gyt, z, gz, gb, ws, wsn, None)


def _lin_dgrad(d, w=A[0], gz=A[1], gx=A[2], gxt=1, ws=A[3], wsn=1 << 20):
    return mqv.lib().mqv_lin_dgrad(ctypes.byref(d), w, gz, gx, gxt, ws, wsn, None)


def _lin_wgrad(d, gz=A[0], x=A[1], gw=A[2], ws=A[3], wsn=1 << 20):
    return mqv.lib().mqv_lin_wgrad(ctypes.byref(d), gz, x, gw, ws, wsn, None)


LN = mqv.ln_desc(4, 64, 1)
LIN = mqv.lin_desc(4, 64, 64, 1, "gelu")
INVALID, WORKSPACE = 1, 3


@pytest.mark.parametrize("call,d,kw,status", [
    (_ln_fwd, LN, dict(x=None), INVALID),
    (_ln_fwd, LN, dict(y=None), INVALID),
    (_ln_fwd, LN, dict(x=A[0] + 8), INVALID),                     # misaligned
    (_ln_fwd, LN, dict(gamma=A[1] + 4), INVALID),
    (_ln_fwd, LN, dict(xt=2), INVALID),
    (_ln_fwd, LN, dict(yt=-1), INVALID),
    (_ln_fwd, LN, dict(mean=None), INVALID),                      # one of the pair
    (_ln_fwd, LN, dict(y=A[0] + 256), INVALID),                   # y inside x
    (_ln_fwd, LN, dict(y=A[0], yt=0), INVALID),                   # in place, other type
    (_ln_fwd, LN, dict(mean=A[3]), INVALID),                      # two outputs
    (_ln_fwd, LN, dict(rstd=A[1]), INVALID),
    (_ln_bwd, LN, dict(gy=None), INVALID),
    (_ln_bwd, LN, dict(mean=None), INVALID),
    (_ln_bwd, LN, dict(gb=None), INVALID),
    (_ln_bwd, LN, dict(ws=None), WORKSPACE),
    (_ln_bwd, LN, dict(wsn=16), WORKSPACE),
    (_ln_bwd, LN, dict(ws=A[8] + 8), WORKSPACE),
    (_ln_bwd, LN, dict(gx=A[1]), INVALID),                        # gx over x
    (_ln_bwd, LN, dict(gxt=7), INVALID),
    (_ln_bwd, LN, dict(ws=A[1]), INVALID),                        # workspace over an input
    (_lin_fwd, LIN, dict(w=None), INVALID),
    (_lin_fwd, LIN, dict(x=None), INVALID),
    (_lin_fwd, LIN, dict(y=None), INVALID),
    (_lin_fwd, LIN, dict(x=A[1] + 2), INVALID),
    (_lin_fwd, LIN, dict(y=A[1]), INVALID),
    (_lin_fwd, LIN, dict(z=A[5]), INVALID),
    (_lin_fwd, LIN, dict(y=A[3] + 16), INVALID),                  # shifted against the residual
    (_lin_fwd, LIN, dict(yt=3), INVALID),
    (_lin_act_grad, LIN, dict(z=None), INVALID),
    (_lin_act_grad, LIN, dict(gy=None), INVALID),
    (_lin_act_grad, LIN, dict(gz=None, gb=None), INVALID),
    (_lin_act_grad, LIN, dict(wsn=0), WORKSPACE),
    (_lin_act_grad, LIN, dict(gz=A[1]), INVALID),
    (_lin_act_grad, LIN, dict(gz=A[0], gyt=0), INVALID),
    (_lin_dgrad, LIN, dict(gz=None), INVALID),
    (_lin_dgrad, LIN, dict(gx=A[1]), INVALID),
    (_lin_dgrad, LIN, dict(gxt=2), INVALID),
    (_lin_wgrad, LIN, dict(x=None), INVALID),
    (_lin_wgrad, LIN, dict(gw=A[0]), INVALID),
    (_lin_wgrad, LIN, dict(gw=A[2] + 4), INVALID),
])
def test_bad_arguments_are_refused(call, d, kw, status):
    assert call(d, **kw) == status
    assert mqv.lib().mqv_last_error() != b""


def test_empty_calls_launch_nothing():
    """P = 0 and no parameter gradients: valid, and no CUDA call is made."""
    d = mqv.ln_desc(0, 64, 1)
    assert _ln_fwd(d, x=None, y=None, mean=None, rstd=None) == 0
    assert _lin_fwd(mqv.lin_desc(0, 8, 8), x=None, res=None, z=None, y=None) == 0


@pytest.mark.parametrize("N", [1, 2048, 1 << 20, 1 << 28])
def test_activation_gradient_of_nothing_needs_no_plan(N):
    """P = 0 has no element limit, so C and N together may pass any grid's:
    the workspace query answers 0 (asked in a process of its own, which an
    arithmetic trap would end)."""
    code = ("import microscaling_quantized_convolution_b200 as m; "
            f"print(m.lin_workspace_bytes(m.lin_desc(0, 1, 1 << 24, {N}, 'gelu'), m.OP_ACT_GRAD))")
    run = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT)
    assert run.returncode == 0 and run.stdout.strip() == "0", (run.returncode, run.stdout, run.stderr[-500:])


@pytest.mark.parametrize("act", ["none", "gelu"])
def test_activation_gradient_of_nothing_without_a_bias_gradient(act):
    """An empty tensor has a null pointer, so with P = 0 neither gz nor gbias
    need be there; nothing is launched.  With positions, one is needed."""
    assert _lin_act_grad(mqv.lin_desc(0, 8, 8, 1, act), gy=None, z=None, gz=None, gb=None, ws=None, wsn=0) == 0
    assert _lin_act_grad(mqv.lin_desc(1, 8, 8, 1, act), gz=None, gb=None) == INVALID


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(4, 64)
    h = x.to(torch.bfloat16)
    w = torch.zeros(64, 64, dtype=torch.bfloat16)
    s = torch.zeros(4)
    for f in (lambda: mqv.ln_fwd(LN, x), lambda: mqv.ln_bwd(LN, x, x, s, s), lambda: mqv.lin_fwd(LIN, w, h),
              lambda: mqv.lin_act_grad(LIN, h, h), lambda: mqv.lin_dgrad(LIN, w, h), lambda: mqv.lin_wgrad(LIN, h, h)):
        with pytest.raises(ValueError, match="CUDA"):
            f()
