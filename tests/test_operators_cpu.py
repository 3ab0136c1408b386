"""The MXFP4, experts' product and balance loss calls without a GPU: their
refusals (validated before any HIP call, so fake device addresses are safe),
the binding's checks, and the plain 64-bit forms the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

import combine_group_limited_amd as ep
import plain64 as P
from combine_group_limited_amd import _lib as L

FAKE = 0x7F0000000000
FP8, BF16, MX, FP32 = L.EP_TYPE_FP8_E4M3, L.EP_TYPE_BF16, L.EP_TYPE_MXFP4, L.EP_TYPE_FP32
BAD, ALIGN, UNSUP, WS = L.EP_ERR_INVALID_ARG, L.EP_ERR_ALIGNMENT, L.EP_ERR_UNSUPPORTED, L.EP_ERR_WORKSPACE


def _cfg(**kw):
    base = dict(T=64, H=256, E=16, G=1, TG=1, k=4, R=1)
    base.update(kw)
    return ep.Config(**base)


def _with(args, over):
    a = list(args)
    for i, v in over.items():
        a[i] = v
    return a


@pytest.mark.parametrize("over,code", [
    ({0: -1}, BAD), ({1: 0}, BAD), ({1: 48}, BAD), ({1: -32}, BAD), ({2: FP8}, BAD), ({2: MX}, BAD), ({2: 9}, BAD),
    ({1: (1 << 20) + 32}, UNSUP), ({0: (1 << 40) + 1}, UNSUP),
    ({3: None}, BAD), ({4: None}, BAD), ({5: None}, BAD), ({3: FAKE + 8}, ALIGN), ({4: FAKE + 4}, ALIGN),
])
def test_quantize_refusals(over, code):
    lib = ep.lib()
    a = _with([4, 64, BF16, FAKE, FAKE, FAKE, None], over)
    assert lib.ep_mxfp4_quantize(*a) == code
    # dequantize(rows, cols, codes, scales, type, out)
    assert lib.ep_mxfp4_dequantize(a[0], a[1], a[4], a[5], a[2], a[3], None) == code


def test_quantize_of_nothing():
    lib = ep.lib()
    assert lib.ep_mxfp4_quantize(0, 64, BF16, None, None, None, None) == L.EP_OK
    assert lib.ep_mxfp4_dequantize(0, 64, None, None, FP32, None, None) == L.EP_OK


# arguments after the configuration (and the capacity): x_type, K, N, x, xs,
# list, w, ws, then [y_type,] y [, y_scales]
PRODUCT = [FP8, 256, 64, FAKE, FAKE, FAKE, FAKE, FAKE]
COMMON = [
    ({0: BF16}, BAD), ({0: FP32}, BAD), ({0: 7}, BAD),
    ({1: 0}, BAD), ({1: 192}, BAD), ({1: -128}, BAD), ({1: 32768 + 128}, UNSUP),
    ({2: 0}, BAD), ({2: 48}, BAD), ({2: -32}, BAD), ({2: 32768 + 32}, UNSUP),
    ({3: None}, BAD), ({4: None}, BAD), ({5: None}, BAD), ({6: None}, BAD), ({7: None}, BAD),
    ({3: FAKE + 8}, ALIGN), ({4: FAKE + 2}, ALIGN), ({5: FAKE + 2}, ALIGN), ({6: FAKE + 8}, ALIGN), ({7: FAKE + 2}, ALIGN),
    ({0: MX, 1: 16}, BAD), ({0: MX, 1: 100}, BAD), ({0: MX, 1: 32768 + 32}, UNSUP),
]


@pytest.mark.parametrize("over,code", COMMON)
def test_expert_refusals(over, code):
    lib, c = ep.lib(), _cfg().c()
    r, a = ctypes.byref(c), _with(PRODUCT, over)
    assert lib.ep_expert_product(r, *a, FAKE, None) == code
    assert lib.ep_expert_product_ll(r, 8, *a, FAKE, None) == code
    for out in ([BF16, FAKE, None], [MX, FAKE, FAKE]):
        assert lib.ep_expert_swiglu(r, *a, *out, None) == code
        assert lib.ep_expert_swiglu_ll(r, 8, *a, *out, None) == code


def test_expert_output_and_capacity_refusals():
    lib, c = ep.lib(), _cfg().c()
    r = ctypes.byref(c)
    assert lib.ep_expert_product(r, *PRODUCT, None, None) == BAD
    assert lib.ep_expert_product(r, *PRODUCT, FAKE + 8, None) == ALIGN
    for call, first in ((lib.ep_expert_swiglu, []), (lib.ep_expert_swiglu_ll, [8])):
        assert call(r, *first, *PRODUCT, FP8, FAKE, None, None) == BAD         # no such output
        assert call(r, *first, *PRODUCT, FP32, FAKE, None, None) == BAD
        assert call(r, *first, *PRODUCT, BF16, FAKE, FAKE, None) == BAD        # bf16 has no scales
        assert call(r, *first, *PRODUCT, MX, FAKE, None, None) == BAD          # MXFP4 has
        assert call(r, *first, *PRODUCT, MX, None, FAKE, None) == BAD
        assert call(r, *first, *PRODUCT, MX, FAKE + 4, FAKE, None) == ALIGN
        wide = _with(PRODUCT, {2: 16384 + 32})                                   # 2 N weight rows
        assert call(r, *first, *wide, BF16, FAKE, None, None) == UNSUP
    for cap in (0, -1, 1 << 28):
        assert lib.ep_expert_product_ll(r, cap, *PRODUCT, FAKE, None) == BAD
        assert lib.ep_expert_swiglu_ll(r, cap, *PRODUCT, BF16, FAKE, None, None) == BAD
    bad = _cfg(H=100).c()
    assert lib.ep_expert_product(ctypes.byref(bad), *PRODUCT, FAKE, None) == BAD
    assert lib.ep_expert_product(None, *PRODUCT, FAKE, None) == BAD
    assert lib.ep_expert_swiglu_ll(None, 8, *PRODUCT, BF16, FAKE, None, None) == BAD
    z = _cfg(T=0).c()  # no tokens: nothing to do
    none = [FP8, 256, 64, None, None, FAKE, FAKE, FAKE]
    assert lib.ep_expert_product(ctypes.byref(z), *none, None, None) == L.EP_OK
    assert lib.ep_expert_swiglu(ctypes.byref(z), *none, MX, None, None, None) == L.EP_OK


def test_balance_refusals():
    lib, c = ep.lib(), _cfg().c()
    r = ctypes.byref(c)
    need = lib.ep_balance_workspace_bytes(r, 3)
    assert need > 0 and need % 256 == 0
    assert lib.ep_balance_workspace_bytes(r, 4000) > need
    for s in (0, -1, 65537):
        assert lib.ep_balance_workspace_bytes(r, s) == 0
    assert lib.ep_balance_workspace_bytes(None, 1) == 0
    # logits, idx, S, seq, mask, loss, count, ntok, prob, workspace, bytes
    ok = [FAKE, FAKE, 3, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, need]
    for over, code in (({0: None}, BAD), ({1: None}, BAD), ({2: 0}, BAD), ({3: None}, BAD), ({2: 65537}, UNSUP),
                       ({5: None}, BAD), ({6: None}, BAD), ({7: None}, BAD), ({8: None}, BAD), ({9: None}, WS),
                       ({10: need - 1}, WS), ({9: FAKE + 128}, ALIGN), ({0: FAKE + 2}, ALIGN), ({3: FAKE + 1}, ALIGN),
                       ({8: FAKE + 2}, ALIGN)):
        assert lib.ep_balance_loss(r, *_with(ok, over), None) == code, over
    # logits, count, ntok, S, seq, mask, grad_loss, grad
    ok = [FAKE, FAKE, FAKE, 3, FAKE, FAKE, FAKE, FAKE]
    for over, code in (({0: None}, BAD), ({1: None}, BAD), ({2: None}, BAD), ({3: 0}, BAD), ({4: None}, BAD),
                       ({3: 65537}, UNSUP), ({6: None}, BAD), ({7: None}, BAD), ({7: FAKE + 2}, ALIGN),
                       ({6: FAKE + 1}, ALIGN)):
        assert lib.ep_balance_loss_backward(r, *_with(ok, over), None) == code, over
    z = _cfg(T=0).c()
    assert lib.ep_balance_loss_backward(ctypes.byref(z), None, FAKE, FAKE, 1, None, None, FAKE, None, None) == L.EP_OK


def test_binding_refuses_wrong_tensors():
    cfg = _cfg()
    with pytest.raises(ValueError):
        ep.mxfp4_quantize(torch.zeros(4, 64, dtype=torch.bfloat16))   # not on a GPU
    with pytest.raises(TypeError):
        ep.mxfp4_quantize(torch.zeros(4, 64, dtype=torch.float16))
    with pytest.raises(ValueError):
        ep.mxfp4_quantize(torch.zeros(4, 48))
    with pytest.raises(ValueError):
        ep.mxfp4_dequantize(torch.zeros(4, 24, dtype=torch.uint8), torch.zeros(4, 1, dtype=torch.uint8))
    with pytest.raises(TypeError):
        ep.mxfp4_dequantize(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8), torch.float16)
    with pytest.raises(ValueError):
        ep.balance_loss(cfg, torch.zeros(cfg.T, cfg.E), torch.zeros(cfg.T, cfg.k, dtype=torch.int32))
    with pytest.raises(ValueError):
        ep.expert_product(cfg, torch.zeros(256, 256, dtype=torch.uint8), torch.zeros(256, 2),
                          torch.zeros(16, 64, 128, dtype=torch.uint8), torch.zeros(16, 64, 8, dtype=torch.uint8),
                          torch.zeros(17, dtype=torch.int32))


def test_plain_e2m1_ties_and_saturation():
    v = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 100.0, -0.25, -5.0, 0.2500001, 0.0, -0.0]
    assert P.E2M1[P.e2m1_codes(v)].tolist() == [0, 1, 1, 2, 2, 4, 4, 6, 6, 0, -4, 0.5, 0, 0]
    assert P.e2m1_codes([-0.0, -0.25]).tolist() == [8, 8]


def test_plain_quantiser_round_trip():
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((5, 128)) * np.exp2(rng.integers(-40, 40, (5, 128)))).astype(np.float32)
    x[0, :32] = 0
    codes, scales = P.mx_quantize(x)
    v = P.mx_values(codes, scales)
    assert np.all(v[0, :32] == 0) and np.all(scales[0, 0] == 0)
    step = np.repeat(np.exp2(scales.astype(float) - 127), 32, axis=-1)
    a = np.abs(x) / step
    assert a.max() < 8
    # half a step of E2M1 at the value, or saturation from up to 8 down to 6
    half = np.where(a < 2, 0.25, np.where(a < 4, 0.5, np.where(a <= 6, 1.0, 2.0)))
    assert np.all(np.abs(x - v) <= half * step)
    again = P.mx_quantize(v)
    assert np.array_equal(P.mx_values(*again), v)


def test_plain_gradient_against_differences():
    rng = np.random.default_rng(11)
    T, E, k = 13, 10, 3
    logits = rng.standard_normal((T, E)) * 2
    idx = np.argsort(-logits, 1)[:, :k]
    seq, mask = [0, 5, 5, 13], np.ones(T, bool)
    mask[[1, 7]] = False
    gl = np.array([0.7, 3.0, -1.3])
    _, count, ntok, _ = P.balance(logits, idx, seq, mask, k)
    g, _ = P.balance_grad(logits, count, ntok, seq, mask, k, gl)

    def total(x):  # picks, and so the counts, stay as they are
        return (gl * P.balance(x, idx, seq, mask, k)[0]).sum()
    h = 1e-5
    for t in range(T):
        for e in range(E):
            d = np.zeros((T, E))
            d[t, e] = h
            diff = (total(logits + d) - total(logits - d)) / (2 * h)
            # third derivatives are below 10 here: h^2 of them, and rounding / h
            assert abs(diff - g[t, e]) < 1e-9 + 2e-16 * 10 / h, (t, e)
