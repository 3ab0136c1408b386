"""The experts' products against the plain 64-bit form: both row types, both
receive layouts, both epilogues, experts without rows and with one, ragged
widths, NaN in rows no token took, bad offset lists, and whole paths.

Tolerance of a bf16 result v of K products whose magnitudes add up to m:
half a bf16 step of v (2^-8 |v|), and one fp32 unit (2^-23) of m for each of
the K sums and of the K / 128 scalings.  The gated result adds, by its
derivatives, those errors of gate and up, and the exponential's and the
reciprocal's: (|gate| + 4) 2^-22 of the result."""
import numpy as np
import pytest
import torch

import combine_group_limited_amd as ep
import plain64 as P
from pipeline import to_dev, to_host

pytestmark = pytest.mark.gpu

BF16 = 2.0 ** -8


def say(*a):
    print(*a, flush=True)


class Case:
    """Seeded rows, weights and counts; `lists` of rows per expert."""

    def __init__(self, seed, counts, K, N, act, gate=False, cap=None, spare=0):
        rng = np.random.default_rng(seed)
        E = len(counts)
        self.E, self.K, self.N, self.act, self.cap, self.gate = E, K, N, act, cap, gate
        counts = np.asarray(counts)
        if cap is None:
            self.rows = int(counts.sum()) + spare
            self.owner = np.concatenate([np.repeat(np.arange(E), counts), np.full(spare, -1)])
            self.list = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        else:
            self.rows = E * cap
            self.owner = np.full((E, cap), -1)
            for e, c in enumerate(counts):
                self.owner[e, :min(c, cap)] = e
            self.owner = self.owner.ravel()
            self.list = counts.astype(np.int32)
        # T tokens of one pick each
        self.cfg = ep.Config(T=max(int(counts.sum()) + spare if cap is None else int(counts.sum()), 1), H=128, E=E,
                             G=1, TG=1, k=1, R=1)
        self.rows = self.cfg.T if cap is None else self.rows
        if act == "fp8":
            self.x = rng.integers(0, 256, (self.rows, K), dtype=np.uint8)
            self.x[(self.x & 0x7F) == 0x7F] = 0x11  # no NaN
            self.xs = (rng.random((self.rows, K // 128)) * 0.02 + 0.001).astype(np.float32)
            unused = self.owner < 0
            self.x[unused], self.xs[unused] = 0x7F, np.nan
            self.xv = P.fp8_values(self.x, self.xs)
        else:
            self.x = rng.integers(0, 256, (self.rows, K // 2), dtype=np.uint8)
            self.xs = rng.integers(120, 130, (self.rows, K // 32), dtype=np.uint8)
            self.xs[self.owner < 0] = 255
            self.xv = P.mx_values(self.x, self.xs)
        wn = 2 * N if gate else N
        self.w = rng.integers(0, 256, (E, wn, K // 2), dtype=np.uint8)
        self.ws = rng.integers(114, 121, (E, wn, K // 32), dtype=np.uint8)
        self.wv = P.mx_values(self.w, self.ws)

    def expected(self):
        """(values, tolerance before rounding) of the product or gated form."""
        x = np.where((self.owner >= 0)[:, None], self.xv, 0.0)
        y, mag = P.product(x, self.wv, self.owner)
        tol = (self.K + self.K // 128) * 2.0 ** -23 * mag
        if not self.gate:
            return y, tol
        a, b = y[:, :self.N], y[:, self.N:]
        ta, tb = tol[:, :self.N], tol[:, self.N:]
        s = a * P.sigmoid(a)
        # |d silu| <= 1.1; second order in the tolerances is within the factor 2
        return s * b, 2 * (1.1 * np.abs(b) * ta + np.abs(s) * tb) + np.abs(s * b) * (np.abs(a) + 4) * 2.0 ** -22

    def call(self, **kw):
        x, xs, w, ws, li = (to_dev(v) for v in (self.x, self.xs, self.w, self.ws, self.list))
        name = "expert_swiglu" if self.gate else "expert_product"
        if self.cap is None:
            return getattr(ep, name)(self.cfg, x, xs, w, ws, li, **kw)
        return getattr(ep, name + "_ll")(self.cfg, self.cap, x, xs, w, ws, li, **kw)

    def check(self, what):
        out = torch.full((self.rows + 1, self.N), 7.0, dtype=torch.bfloat16, device="cuda")
        say("experts", what, self.rows, "x", self.K, "->", self.N, self.act, "gate" if self.gate else "")
        self.call(out=out[:self.rows])
        got = to_host(out.float())
        v, tol = self.expected()
        used = self.owner >= 0
        assert np.all(got[:-1][~used] == 7.0) and np.all(got[-1] == 7.0), "rows of no expert were written"
        d = np.abs(got[:-1][used] - v[used])
        lim = tol[used] + BF16 * (np.abs(v[used]) + tol[used])
        bad = ~(d <= lim)
        assert not bad.any(), "%d of %d off, worst %g of its tolerance" % (bad.sum(), bad.size, np.nanmax(d / lim))


FEW = [3, 0, 1, 16, 17, 5, 0, 33]
MANY = [300, 0, 1, 256, 129, 64, 15, 513]
SOME = [16, 33, 0, 1, 20, 31, 32, 17]
LOTS = [300, 513, 0, 257, 400]


@pytest.mark.parametrize("act", ["fp8", "mxfp4"])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("counts,K,N,cap", [
    (FEW, 128, 32, None), (FEW, 384, 96, None), (FEW, 1280, 160, 40), (FEW, 256, 64, 8), ([1], 2944, 64, None),
    ([0, 1, 0], 512, 32, 1), ([1] + [0] * 1023, 128, 32, None), ([2, 0, 1] * 33, 256, 64, None),
    (MANY, 128, 32, None), (MANY, 640, 288, None), (MANY, 1152, 352, 520), (MANY, 256, 512, 256),
    ([77], 384, 1024, None),
    ([40] * 12, 512, 96, None),
    (LOTS, 128, 32, None), (LOTS, 640, 288, None), (LOTS, 1152, 352, 600), ([256] * 8, 1024, 512, None),
    ([1000, 200], 2048, 416, None), ([222], 896, 64, None),
    (SOME, 128, 32, None), (SOME, 640, 288, None), (SOME, 1152, 352, 40), ([20] * 65, 256, 1056, None),
    ([100, 0, 31, 64] * 16, 384, 1312, None), ([40] * 130, 384, 608, None),
    ([2, 0, 1] * 33, 2176, 160, None), ([20] * 65, 2176, 160, None), ([1, 0, 1, 2] * 24, 640, 1056, None),
    ([20, 9, 31] * 16, 896, 1120, None),
    (MANY, 128, 1824, None), (MANY, 640, 1824, None), (MANY, 384, 1824, 520),
    (LOTS, 128, 1568, None), (LOTS, 640, 1632, None), (LOTS, 1152, 1568, 600), ([256] * 8, 1024, 1152, None),
    ([1000, 200], 2048, 1824, None),
])
def test_products(act, gate, counts, K, N, cap):
    Case(len(counts) * 1000 + K + N, counts, K, N, act, gate, cap, spare=0 if cap else 3).check("%s" % (counts[:8],))


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("counts", [FEW, MANY])
@pytest.mark.parametrize("K,N", [(32, 32), (64, 64), (96, 32), (160, 288), (544, 64), (672, 96), (1440, 160)])
def test_mxfp4_rows_of_any_blocks(counts, K, N, gate):
    Case(K * 3 + N, counts, K, N, "mxfp4", gate, None, spare=1).check("%d columns" % K)


@pytest.mark.parametrize("act", ["fp8", "mxfp4"])
@pytest.mark.parametrize("counts,K,N,cap", [(FEW, 384, 96, None), (MANY, 640, 288, None), (FEW, 256, 64, 40),
                                            (SOME, 640, 288, None), ([100, 0, 31, 64] * 16, 384, 1312, None),
                                            (MANY, 640, 928, None), (LOTS, 384, 928, 600),
                                            ([40] * 12, 512, 96, 64), (LOTS, 640, 288, None),
                                            (LOTS, 1408, 64, 600)])
def test_gated_to_mxfp4(act, counts, K, N, cap):
    c = Case(K + N, counts, K, N, act, True, cap, spare=0 if cap else 2)
    codes = torch.full((c.rows, N // 2), 0x5A, dtype=torch.uint8, device="cuda")
    scales = torch.full((c.rows, N // 32), 0x5A, dtype=torch.uint8, device="cuda")
    say("gated to mxfp4", c.rows, K, N, act)
    c.call(out_dtype="mxfp4", out=codes, out_scales=scales)
    codes, scales = to_host(codes), to_host(scales)
    v, tol = c.expected()
    used = c.owner >= 0
    assert np.all(codes[~used] == 0x5A) and np.all(scales[~used] == 0x5A)
    v, tol, s = v[used], tol[used], scales[used]
    hi = (np.abs(v) + tol).reshape(len(v), -1, 32).max(-1)
    lo = np.maximum(np.abs(v) - tol, 0).reshape(len(v), -1, 32).max(-1)
    assert np.all((s >= P.mx_scale(lo)) & (s <= P.mx_scale(hi)))
    # rounding is monotone: the codes' values lie between those of v - tol and v + tol
    unit = np.exp2(s.astype(float) - 127).repeat(32, 1)
    got = P.E2M1[P.unpack(codes[used])]
    assert np.all(got >= P.E2M1[P.e2m1_codes((v - tol) / unit)])
    assert np.all(got <= P.E2M1[P.e2m1_codes((v + tol) / unit)])


@pytest.mark.parametrize("act", ["fp8", "mxfp4"])
@pytest.mark.parametrize("per,N", [(4, 64), (20, 64), (200, 64), (200, 5152)])
def test_a_nan_row_stays_alone(act, per, N):
    c = Case(9, [per, per], 256, N, act)
    if act == "fp8":
        c.x[1, 3] = 0x7F
    else:
        c.xs[1, 2] = 255
    got = to_host(c.call().float())
    assert np.isnan(got[1]).all() and np.isfinite(np.delete(got, 1, 0)).all()
    c.ws[1, 5, 1] = 255  # a weight block without a scale: one column of one expert
    got = to_host(c.call().float())
    bad = np.zeros(got.shape, bool)
    bad[1], bad[per:, 5] = True, True
    assert np.array_equal(np.isnan(got), bad)


@pytest.mark.parametrize("per,N", [(3, 64), (120, 64), (120, 4512)])
def test_offset_lists_that_lead_outside_are_clamped(per, N):
    c = Case(10, [per] * 4, 256, N, "mxfp4")
    good = c.list.copy()
    for at, v in ((4, 1 << 30), (0, -5)):
        c.list = good.copy()
        c.list[at] = v
        c.check("clamped list %d" % v)  # the clamped list is the right one
    c = Case(11, [per] * 4, 256, N, "fp8", cap=per)
    c.list[2] = 1 << 30                  # a count beyond the capacity
    c.check("clamped count")


@pytest.mark.parametrize("act", ["fp8", "mxfp4"])
@pytest.mark.parametrize("per,N", [(2, 128), (100, 128), (100, 2080)])
def test_two_runs_another_stream_and_a_graph(per, N, act):
    c = Case(12, [per] * 6, 768, N, act, True)
    x, xs, w, ws, li = (to_dev(v) for v in (c.x, c.xs, c.w, c.ws, c.list))
    first = ep.expert_swiglu(c.cfg, x, xs, w, ws, li)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(first)
    torch.cuda.synchronize()
    ep.expert_swiglu(c.cfg, x, xs, w, ws, li, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ep.expert_swiglu(c.cfg, x, xs, w, ws, li, out=out)
    for rep in range(3):
        out.fill_(float(rep))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first), rep


def test_rows_past_four_gigabytes():
    # 600000 rows of 8192 bytes: the last expert's rows lie past 4 GiB
    T, K, N, E = 600000, 8192, 32, 4
    cfg = ep.Config(T=T, H=128, E=E, G=1, TG=1, k=1, R=1)
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.full((T, K), 0x38, dtype=torch.uint8, device="cuda")       # 1.0
    tail = torch.randint(0, 0x70, (50, K), generator=g, device="cuda", dtype=torch.uint8)
    x[-50:] = tail
    xs = torch.full((T, K // 128), 0.5, device="cuda")
    w = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    ws = torch.full((E, N, K // 32), 118, dtype=torch.uint8, device="cuda")
    off = torch.tensor([0, 1000, 1000, T - 50, T], dtype=torch.int32, device="cuda")
    say("rows past 4 GiB")
    y = ep.expert_product(cfg, x, xs, w, ws, off)
    got = to_host(y[-50:].float())
    xv = P.e4m3_values(to_host(tail)) * 0.5
    wv = P.mx_values(to_host(w[3]), to_host(ws[3]))
    ref, mag = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    tol = (K + K // 128) * 2.0 ** -23 * mag
    assert np.all(np.abs(got - ref) <= tol + BF16 * (np.abs(ref) + tol))


@pytest.mark.parametrize("ll", [False, True])
def test_whole_path(ll):
    """Route, FP8 dispatch, both products with the MXFP4 rows between them,
    combine: against the oracle-checked steps' own outputs in 64 bits."""
    T, H, E, F, k = 48, 256, 16, 96, 4
    cfg = ep.Config(T=T, H=H, E=E, G=4, TG=2, k=k, R=4)
    rng = np.random.default_rng(77)
    lg = to_dev(rng.standard_normal((T, E)).astype(np.float32))
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16).cuda()
    w1 = torch.from_numpy((rng.standard_normal((E, 2 * F, H)) / 16).astype(np.float32)).cuda()
    # K = 96 is no multiple of 128: the second product has 128 columns, the last 32 of them zero
    w2 = torch.from_numpy((rng.standard_normal((E, H, 128)) / 11).astype(np.float32)).cuda()
    w1 = torch.cat([w1[:, :F], w1.new_zeros(E, 32, H), w1[:, F:], w1.new_zeros(E, 32, H)], 1).contiguous()
    w1q, w1s = ep.mxfp4_quantize(w1)
    w2q, w2s = ep.mxfp4_quantize(w2)
    idx, wt = ep.route(cfg, lg)
    if ll:
        d = ep.dispatch_ll(cfg, x, idx, T)
        h, hs = ep.expert_swiglu_ll(cfg, T, d["recv"], d["scales"], w1q, w1s, d["count"], out_dtype="mxfp4")
        y = ep.expert_product_ll(cfg, T, h, hs, w2q, w2s, d["count"])
        slot, recv, sc = d["slot"], d["recv"], d["scales"]
        out = ep.combine_ll(cfg, T, y, slot, wt)
    else:
        lay = ep.get_layout(cfg, idx)
        slot = lay["slot"]
        recv, sc = ep.dispatch(cfg, x, slot)
        h, hs = ep.expert_swiglu(cfg, recv, sc, w1q, w1s, lay["off"], out_dtype="mxfp4")
        y = ep.expert_product(cfg, h, hs, w2q, w2s, lay["off"])
        out = ep.combine(cfg, y, slot, wt)
    torch.cuda.synchronize()
    slot, idx, wt = to_host(slot), to_host(idx), to_host(wt).astype(np.float64)
    xv = P.fp8_values(to_host(recv), to_host(sc))
    hv = P.mx_values(to_host(h), to_host(hs))
    w1v, w2v = P.mx_values(to_host(w1q), to_host(w1s)), P.mx_values(to_host(w2q), to_host(w2s))
    got = to_host(out.float())
    ref, tol = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            r, e = slot[t, j], idx[t, j]
            g = w1v[e] @ xv[r]
            a, b = g[:128], g[128:]
            v = a * P.sigmoid(a) * b
            # the kernel's own 4-bit rows are within their rounding of the plain ones
            unit = np.exp2(to_host(hs)[r].astype(float) - 127).repeat(32)
            assert np.all(np.abs(hv[r] - v) <= 2 * unit + 1e-3 * np.abs(v))
            y1 = w2v[e] @ hv[r]
            mag = np.abs(w2v[e]) @ np.abs(hv[r])
            ref[t] += wt[t, j] * y1
            tol[t] += wt[t, j] * (BF16 * np.abs(y1) + 130 * 2.0 ** -23 * mag * 2) + 8 * 2.0 ** -24 * np.abs(wt[t, j] * y1)
    assert np.all(np.abs(got - ref) <= tol + BF16 * (np.abs(ref) + tol))
