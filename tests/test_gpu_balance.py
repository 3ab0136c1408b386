"""The balance loss, its counts and its gradient against the plain 64-bit
form: expert counts for every lane layout, ragged and empty sequences, masks
that leave nothing, padding that holds NaN and infinities, saturated logits,
unrouted and repeated picks, unaligned rows, streams and graphs.

Tolerances: probabilities are sums of positive terms, so their relative error
is at most 2^-24 for every rounding on the way: up to 8 in a score, E / 4 + 8
in a token's sum, 4 in the quotient and the mean, and 32 + n / 32 + 32 in the
sums over tokens.  The gradient's terms carry the same errors before they
cancel."""
import numpy as np
import pytest
import torch

import combine_group_limited_amd as ep
import plain64 as P
from pipeline import to_dev, to_host

pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, flush=True)


def rel(E, n):
    return (8 + E / 4 + 8 + 4 + 64 + n / 32) * 2.0 ** -24


def check(T, E, k, seq, mask=None, logits=None, idx=None, seed=0, misalign=False, note=""):
    rng = np.random.default_rng(seed + T * 31 + E)
    if logits is None:
        logits = (rng.standard_normal((T, E)) * 2).astype(np.float32)
    if idx is None:
        idx = np.argsort(-np.nan_to_num(logits), 1, kind="stable")[:, :k].astype(np.int32)
    S = len(seq) - 1
    gl = (rng.standard_normal(S) + 0.1).astype(np.float32)
    cfg = ep.Config(T=T, H=128, E=E, G=1, TG=1, k=k, R=1, m=1)
    say("balance", T, E, k, "S", S, note)
    if misalign:
        buf = torch.empty(T * E + 1, dtype=torch.float32, device="cuda")
        dl = buf[1:].view(T, E)
        dl.copy_(torch.from_numpy(logits))
    else:
        dl = to_dev(logits)
    ds = to_dev(np.asarray(seq, np.int32))
    dm = None if mask is None else to_dev(np.asarray(mask, np.uint8))
    r = ep.balance_loss(cfg, dl, to_dev(idx), ds, dm)
    grad = torch.full((T + 1, E), 7.0, device="cuda")
    ep.balance_loss_backward(cfg, dl, r["count"], r["ntok"], to_dev(gl), ds, dm, grad[:T])
    torch.cuda.synchronize()
    m = np.ones(T, bool) if mask is None else np.asarray(mask).astype(bool)
    loss, count, ntok, prob = P.balance(logits.astype(np.float64), idx, seq, m, k)
    assert np.array_equal(to_host(r["count"]), count)
    assert np.array_equal(to_host(r["ntok"]), ntok)
    n = max(1, int(ntok.max()))
    for name, ref in (("prob", prob), ("loss", loss)):
        got = to_host(r[name]).astype(np.float64)
        assert np.all(np.abs(got - ref) <= rel(E, n) * np.abs(ref) + 1e-44), name
    g, size = P.balance_grad(logits.astype(np.float64), count, ntok, seq, m, k, gl.astype(np.float64))
    got = to_host(grad)
    assert np.all(got[T] == 7.0)
    assert np.all(np.abs(got[:T] - g) <= rel(E, 0) * size + 1e-44)
    return got[:T], g


@pytest.mark.parametrize("E,k", [(1, 1), (2, 1), (8, 2), (16, 4), (17, 3), (60, 8), (64, 6), (65, 2), (99, 8), (128, 8),
                                 (160, 6), (250, 8), (256, 8), (384, 8), (510, 4), (512, 8), (777, 3), (1024, 32)])
def test_expert_counts(E, k):
    for T in (1, 3, 70):
        check(T, E, k, [0, T])
    check(70, E, k, [0, 9, 9, 40, 70], misalign=True, note="unaligned rows")


@pytest.mark.parametrize("T", [1, 15, 16, 17, 4096, 9001])
def test_sequences(T):
    rng = np.random.default_rng(T)
    check(T, 32, 4, [0, T])
    cuts = np.sort(rng.integers(0, T + 1, 6))
    check(T, 32, 4, [0, *cuts.tolist(), T], mask=rng.random(T) < 0.7, note="ragged, masked")
    check(T, 32, 4, [0] * 70 + [T] * 71, note="mostly empty")
    if T < 100:
        check(T, 32, 4, list(range(T + 1)), note="one token each")


def test_many_sequences():
    T = 5000
    rng = np.random.default_rng(8)
    seq = np.sort(rng.integers(0, T + 1, 4499)).tolist()
    check(T, 16, 2, [0, *seq, T], mask=rng.random(T) < 0.9)


def test_masked_tokens_take_no_part():
    T, E, k = 200, 64, 4
    rng = np.random.default_rng(9)
    lg = rng.standard_normal((T, E)).astype(np.float32)
    mask = rng.random(T) < 0.5
    mask[100:150] = False  # a whole sequence
    off = np.flatnonzero(~mask)
    idx = np.argsort(-lg, 1)[:, :k].astype(np.int32)
    lg[off[0::3]] = np.nan
    lg[off[1::3]] = np.inf
    lg[off[2::3]] = np.finfo(np.float32).min
    seq = [0, 30, 100, 150, 200]
    got, _ = check(T, E, k, seq, mask, lg, idx)
    assert np.all(got[~mask] == 0)
    check(T, E, k, seq, np.zeros(T, bool), lg, idx, note="nothing left")


@pytest.mark.parametrize("E", [48, 256])
def test_saturated_logits(E):
    T, k = 64, 2
    rng = np.random.default_rng(10)
    lg = (rng.standard_normal((T, E)) * 40).astype(np.float32)
    lg[0] = 200.0                  # every score 1
    lg[1] = -200.0                 # every score 0: no probabilities
    lg[2] = -np.inf
    lg[3, ::2], lg[3, 1::2] = np.inf, -np.inf
    lg[4] = -85.0
    lg[5, :] = np.finfo(np.float32).min
    lg[5, 3] = 1.0                 # all but one expert closed
    lg[6] = 15.0 + rng.random(E)   # 1 - s needs its own digits
    lg = np.clip(lg, -np.inf, np.inf)
    # scores below the smallest normal number are cut to it or to 0: keep logits out of that sliver
    lg[(lg < -80) & (lg > -90) & (lg != -85.0)] = -80
    lg[(lg <= -90)] = np.where(np.isinf(lg[lg <= -90]), -np.inf, -1000.0)
    check(T, E, k, [0, 7, T], logits=lg)


def test_picks_unrouted_and_repeated():
    T, E, k = 300, 40, 6
    rng = np.random.default_rng(12)
    idx = rng.integers(0, E, (T, k)).astype(np.int32)
    idx[rng.random(idx.shape) < 0.1] = -1
    idx[rng.random(idx.shape) < 0.1] = E + 3
    idx[5] = 7
    check(T, E, k, [0, 100, 300], idx=idx)


def test_gradient_against_differences():
    """The kernel's gradient against central differences of the 64-bit loss,
    the picks held."""
    T, E, k = 12, 20, 3
    rng = np.random.default_rng(13)
    lg = rng.standard_normal((T, E)).astype(np.float32)
    idx = np.argsort(-lg, 1)[:, :k].astype(np.int32)
    seq, m = [0, 4, 12], np.ones(T, bool)
    cfg = ep.Config(T=T, H=128, E=E, G=1, TG=1, k=k, R=1, m=1)
    ds, gl = to_dev(np.asarray(seq, np.int32)), np.array([1.5, -0.75], np.float32)
    r = ep.balance_loss(cfg, to_dev(lg), to_dev(idx), ds)
    g = to_host(ep.balance_loss_backward(cfg, to_dev(lg), r["count"], r["ntok"], to_dev(gl), ds))
    x, h = lg.astype(np.float64), 1e-5
    for t in range(T):
        for e in range(0, E, 3):
            d = np.zeros((T, E))
            d[t, e] = h
            diff = ((P.balance(x + d, idx, seq, m, k)[0] - P.balance(x - d, idx, seq, m, k)[0]) * gl).sum() / (2 * h)
            assert abs(g[t, e] - diff) < 1e-9 + rel(E, 0) * 4 * abs(gl).max() * E / k, (t, e)


def test_offset_lists_that_lead_outside_are_clamped():
    T, E, k = 50, 32, 2
    rng = np.random.default_rng(14)
    lg = rng.standard_normal((T, E)).astype(np.float32)
    idx = np.argsort(-lg, 1)[:, :k].astype(np.int32)
    cfg = ep.Config(T=T, H=128, E=E, G=1, TG=1, k=k, R=1, m=1)
    a = ep.balance_loss(cfg, to_dev(lg), to_dev(idx), to_dev(np.array([-9, 20, 1 << 30], np.int32)))
    b = ep.balance_loss(cfg, to_dev(lg), to_dev(idx), to_dev(np.array([0, 20, T], np.int32)))
    for name in ("loss", "count", "ntok", "prob"):
        assert torch.equal(a[name], b[name]), name
    # tokens in no sequence: gradient 0
    seq = to_dev(np.array([10, 20, 40], np.int32))
    c = ep.balance_loss(cfg, to_dev(lg), to_dev(idx), seq)
    one = torch.ones(2, device="cuda")
    g = to_host(ep.balance_loss_backward(cfg, to_dev(lg), c["count"], c["ntok"], one, seq))
    assert np.all(g[:10] == 0) and np.all(g[40:] == 0) and np.all(np.any(g[10:40] != 0, 1))
    assert to_host(c["ntok"]).tolist() == [10, 20]


def test_no_tokens_default_arguments_in_place_and_bool_mask():
    cfg = ep.Config(T=0, H=128, E=24, G=1, TG=1, k=2, R=1)
    r = ep.balance_loss(cfg, torch.empty(0, 24, device="cuda"), torch.empty(0, 2, dtype=torch.int32, device="cuda"))
    for name in ("loss", "count", "ntok", "prob"):
        assert bool((r[name] == 0).all()), name
    T, E, k = 333, 24, 2
    cfg = ep.Config(T=T, H=128, E=E, G=1, TG=1, k=k, R=1, m=1)
    lg = torch.randn(T, E, device="cuda")
    idx = lg.topk(k, 1).indices.to(torch.int32)
    mask = torch.rand(T, device="cuda") < 0.8
    one = torch.ones(1, device="cuda")
    a = ep.balance_loss(cfg, lg, idx, token_mask=mask)
    b = ep.balance_loss(cfg, lg, idx, torch.tensor([0, T], dtype=torch.int32, device="cuda"), mask.to(torch.uint8))
    for name in ("loss", "count", "ntok", "prob"):
        assert torch.equal(a[name], b[name]), name
    g = ep.balance_loss_backward(cfg, lg, a["count"], a["ntok"], one, token_mask=mask)
    same = lg.clone()
    ep.balance_loss_backward(cfg, same, a["count"], a["ntok"], one, token_mask=mask, grad_logits=same)
    assert torch.equal(same, g)


def test_two_runs_another_stream_and_a_graph():
    T, E, k = 3000, 256, 8
    cfg = ep.Config(T=T, H=128, E=E, G=1, TG=1, k=k, R=1, m=1)
    lg = torch.randn(T, E, device="cuda")
    idx = lg.topk(k, 1).indices.to(torch.int32)
    seq = torch.tensor([0, 700, 700, 3000], dtype=torch.int32, device="cuda")
    gl = torch.rand(3, device="cuda")

    def run(out, ws, grad, **kw):
        r = ep.balance_loss(cfg, lg, idx, seq, out=out, workspace=ws, **kw)
        ep.balance_loss_backward(cfg, lg, r["count"], r["ntok"], gl, seq, grad_logits=grad, **kw)
        return [r["loss"], r["count"], r["ntok"], r["prob"], grad]

    def buffers():
        return (dict(loss=torch.empty(3, device="cuda"), count=torch.empty(3, E, dtype=torch.int32, device="cuda"),
                     ntok=torch.empty(3, dtype=torch.int32, device="cuda"), prob=torch.empty(3, E, device="cuda")),
                torch.full((ep.balance_workspace_bytes(cfg, 3),), 0xEE, dtype=torch.uint8, device="cuda"),
                torch.empty(T, E, device="cuda"))
    first = [t.clone() for t in run(*buffers())]
    side = torch.cuda.Stream()
    b = buffers()
    torch.cuda.synchronize()
    got = run(*b, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, first))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = run(*b)
    for rep in range(3):
        for t in got:
            t.view(torch.uint8).fill_(0x5A + rep)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, first)), rep
