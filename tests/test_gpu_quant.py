"""MXFP4 quantisation and its inverse against the plain 64-bit form, bit for
bit: random rows, ragged sizes, every scale, ties, zeros, NaN and infinities,
guard bytes after every output, another stream, and a captured graph."""
import numpy as np
import pytest
import torch

import combine_group_limited_amd as ep
import plain64 as P
from pipeline import to_dev, to_host

pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, flush=True)


def bf16(x):
    """x rounded to bf16 (to nearest), as bits and as values."""
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16)
    return t, t.float().numpy()


def rows_of(rng, rows, cols):
    """Values over every binade, with blocks of zeros, ties, and specials."""
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-3, 3, (rows, cols)))
    x = x * np.exp2(rng.integers(-149, 120, (rows, cols // 32)).astype(float)).repeat(32, 1)
    b = x.reshape(-1, 32)
    n = b.shape[0]
    b[0] = 0
    if n > 3:
        b[1] = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 4.0] * 4) * np.where(np.arange(32) % 2, 1, -1)
        b[2, 5] = np.nan
        b[3, 31] = -np.inf
    return np.ascontiguousarray(x, dtype=np.float32)


SIZES = [(1, 32), (1, 64), (3, 96), (63, 32), (64, 32), (65, 32), (7, 7168), (129, 2048), (1000, 160)]


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_quantize_bit_exact(rows, cols, wide):
    say("quantize", rows, cols, wide)
    rng = np.random.default_rng(rows * 10007 + cols)
    with np.errstate(over="ignore"):
        x = rows_of(rng, rows, cols)
    t = torch.from_numpy(x)
    if not wide:
        t, x = bf16(x)
    codes = torch.full((rows * cols // 2 + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows * cols // 32 + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    ep.mxfp4_quantize(t.cuda(), codes[:rows * cols // 2].view(rows, cols // 2),
                      scales[:rows * cols // 32].view(rows, cols // 32))
    rc, rs = P.mx_quantize(x)
    assert np.array_equal(to_host(scales[:rows * cols // 32]), rs.ravel())
    assert np.array_equal(to_host(codes[:rows * cols // 2]), rc.ravel())
    assert bool((codes[rows * cols // 2:] == 0xA5).all()) and bool((scales[rows * cols // 32:] == 0xA5).all())


@pytest.mark.parametrize("wide", [False, True])
def test_dequantize_every_code_and_scale(wide):
    codes = np.tile(P.pack(np.arange(32) % 16), (256, 1))
    scales = np.arange(256, dtype=np.uint8)[:, None]
    say("dequantize", wide)
    out = ep.mxfp4_dequantize(to_dev(codes), to_dev(scales), torch.float32 if wide else torch.bfloat16).float()
    with np.errstate(over="ignore"):
        ref = P.mx_values(codes, scales).astype(np.float32)
    got = to_host(out)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    ok = ~np.isnan(ref)
    assert np.array_equal(got[ok].view(np.uint32), ref[ok].view(np.uint32))


@pytest.mark.parametrize("rows,cols", SIZES)
def test_dequantize_sizes(rows, cols):
    rng = np.random.default_rng(rows + cols)
    codes = rng.integers(0, 256, (rows, cols // 2), dtype=np.uint8)
    scales = rng.integers(60, 200, (rows, cols // 32), dtype=np.uint8)
    for dt in (torch.bfloat16, torch.float32):
        buf = torch.full((rows * cols + 32,), 7.0, dtype=dt, device="cuda")
        say("dequantize", rows, cols, dt)
        ep.mxfp4_dequantize(to_dev(codes), to_dev(scales), dt, buf[:rows * cols].view(rows, cols))
        assert np.array_equal(to_host(buf[:rows * cols].float()).reshape(rows, cols),
                              P.mx_values(codes, scales).astype(np.float32))
        assert bool((buf[rows * cols:] == 7.0).all())


def test_weights_of_three_dimensions_and_nothing():
    rng = np.random.default_rng(5)
    t, x = bf16(rng.standard_normal((3, 40, 128)))
    c, s = ep.mxfp4_quantize(t.cuda())
    rc, rs = P.mx_quantize(x)
    assert np.array_equal(to_host(c), rc) and np.array_equal(to_host(s), rs)
    c, s = ep.mxfp4_quantize(torch.empty(0, 64, device="cuda"))
    assert c.shape == (0, 32) and s.shape == (0, 2)
    assert ep.mxfp4_dequantize(c, s).shape == (0, 64)


def test_another_stream_and_a_graph():
    rng = np.random.default_rng(6)
    t, x = bf16(rng.standard_normal((200, 256)))
    d = t.cuda()
    rc, rs = P.mx_quantize(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c, s = ep.mxfp4_quantize(d, stream=side)
    side.synchronize()
    assert np.array_equal(to_host(c), rc) and np.array_equal(to_host(s), rs)
    out = torch.empty(200, 256, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ep.mxfp4_quantize(d, c, s)
        ep.mxfp4_dequantize(c, s, out=out)
    ref = P.mx_values(rc, rs).astype(np.float32)
    for rep in range(3):
        c.fill_(rep), s.fill_(rep), out.fill_(rep)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(to_host(c), rc) and np.array_equal(to_host(out.float()), ref), rep
