"""The operators this package adds between routing and combine, as cases that
can be measured: the router's balance loss with its gradient, the MXFP4
quantiser, and the experts' products over MXFP4 weights.

`own` selects what `run` does: the plain form (elementary torch operations in
32 bits or more) or the package's entry points, on the same prepared inputs.

Number formats: MXFP4 is the OCP Microscaling format with E2M1 elements (0,
0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), two to a byte (the even column
in the low half), and one E8M0 scale 2^(b - 127) for every 32 columns.  FP8
rows are dispatch's payload: E4M3 codes and a 32-bit scale for every 128
columns.
"""
import functools
import math

import torch

own = False

HIDDEN = 7168  # the hidden size of every workload but the small one


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # balance loss and its gradient, one training micro-batch of one step
        # a decode-sized batch: three small launches, latency is all there is
        dict(name="balance 128 tokens", op="balance", T=128, E=256, k=8, S=1, pad=0.0),
        # the prefill batch as four packed sequences with padding inside
        dict(name="balance 4096 tokens", op="balance", T=4096, E=256, k=8, S=4, pad=0.05),
        # a long packed batch: 37 ragged sequences, bandwidth counts
        dict(name="balance 65536 tokens", op="balance", T=65536, E=256, k=8, S=37, pad=0.02),
        # the quantiser: the hidden rows of a decode batch
        dict(name="quantize 128 rows", op="quantize", rows=128, cols=HIDDEN, wide=False),
        # as many rows as the largest workload routes
        dict(name="quantize 131072 rows", op="quantize", rows=131072, cols=HIDDEN, wide=False),
        # one token's eight experts: the weights of eight experts are read once
        dict(name="product one token", op="product", act="fp8", slots="rows", T=1, E=256, k=8, K=HIDDEN, N=2048,
             skew=0.0, lost=0.0),
        # the decode batch on the low-latency rows, second product of the experts
        dict(name="product decode rows", op="product", act="mxfp4", slots="capacity", T=128, E=256, k=8, K=2048,
             N=HIDDEN, skew=0.0, lost=0.0),
        # one rank's eight experts with the tokens of every rank: matrix rate counts
        dict(name="product one rank", op="product", act="mxfp4", slots="rows", T=16384, E=8, k=2, K=HIDDEN, N=4096,
             skew=0.0, lost=0.0),
        # prefill, every expert, straight from the FP8 dispatch, gated activation fused
        dict(name="swiglu prefill", op="swiglu", act="fp8", slots="rows", T=4096, E=256, k=8, K=HIDDEN, N=1024,
             skew=0.0, lost=0.0),
        # one rank's experts under skewed routing, odd widths, some picks unrouted
        dict(name="swiglu odd and skewed", op="swiglu", act="fp8", slots="rows", T=3001, E=12, k=3, K=2944, N=1440,
             skew=1.0, lost=0.02),
        # both products of the experts, the 4-bit rows between them: decode
        dict(name="experts decode", op="experts", act="fp8", slots="capacity", T=128, E=256, k=8, K=HIDDEN, N=1024,
             skew=0.0, lost=0.0),
        # the same for one rank's share of a prefill batch
        dict(name="experts one rank", op="experts", act="fp8", slots="rows", T=16384, E=8, k=2, K=HIDDEN, N=2048,
             skew=0.5, lost=0.0),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("balance", "quantize", "product", "swiglu", "experts"))
    if op == "balance":
        E = rng.choice((8, 16, 64, 96, 99, 128, 160, 256))
        T = _spread(rng, 100, 65000)
        return dict(op=op, T=T, E=E, k=rng.randint(1, min(8, E)), S=min(T, _spread(rng, 1, 64)),
                    pad=rng.choice((0.0, 0.03, 0.3)))
    if op == "quantize":
        return dict(op=op, rows=_spread(rng, 65, 40000), cols=128 * _spread(rng, 2, 56), wide=rng.random() < 0.3)
    slots = rng.choice(("rows", "rows", "capacity"))
    E = rng.choice((8, 12, 16, 32, 64, 96, 128, 256))
    k = rng.randint(1, min(8, E))
    K = 128 * _spread(rng, 3, 56)
    N = 32 * _spread(rng, 8, 128 if op == "product" else 64)
    T = _spread(rng, 1, 500 if slots == "capacity" else 16000)
    # no more work than the largest listed case
    wide = 2 * N if op != "product" else N
    while E * wide * K > 256 * 2048 * HIDDEN:
        E //= 2
    k = min(k, E)
    while T > 1 and T * k * wide * K > 16384 * 2 * 4096 * HIDDEN // 2:
        T //= 2
    return dict(op=op, act=rng.choice(("fp8", "mxfp4")), slots=slots, T=T, E=E, k=k, K=K, N=N,
                skew=rng.choice((0.0, 0.0, 0.7)), lost=rng.choice((0.0, 0.03)))


# ------------------------------------------------------------ the inputs

def _device():
    return torch.device("cuda", torch.cuda.current_device())


def _picks(g, T, E, k, skew, lost, dev):
    """The experts of each token, best first, int32 [T, k]; a share `lost` of
    them is -1 (unrouted).  `skew` lifts the logits of a few experts."""
    logits = torch.randn(T, E, generator=g, device=dev)
    if skew:
        lift = torch.randperm(E, generator=g, device=dev).float().add_(1).pow_(-1.2).mul_(3 * skew)
        logits += lift
    idx = logits.topk(k, dim=1).indices.to(torch.int32)
    if lost:
        idx[torch.rand(T, k, generator=g, device=dev) < lost] = -1
    return logits, idx


def _pool(g, n, dev):
    """n bytes of E2M1 code pairs as quantised normal values have them."""
    m = min(n, 1 << 24)
    v = torch.randn(2 * m, generator=g, device=dev).mul_(2.0)
    a = _round_e2m1(v).abs()
    # 0, .5, 1, 1.5, 2, 3, 4, 6 are codes 0 .. 7, the sign is bit 3
    codes = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    codes |= torch.signbit(v).to(torch.uint8) << 3
    pool = codes[0::2] | (codes[1::2] << 4)
    if n <= m:
        return pool[:n].clone()
    out = torch.empty(n, dtype=torch.uint8, device=dev)
    at = 0
    shifts = torch.randint(0, m, (n // (m // 2) + 2,), generator=g, device=dev).tolist()
    for s in shifts:
        take = min(m - s, n - at)
        out[at:at + take] = pool[s:s + take]
        at += take
        if at == n:
            return out
    while at < n:
        take = min(m, n - at)
        out[at:at + take] = pool[:take]
        at += take
    return out


def _weights(g, E, N, K, dev):
    """E experts' weights [N, K] in MXFP4: values of about 1 / sqrt(K)."""
    w = _pool(g, E * N * K // 2, dev).view(E, N, K // 2)
    base = 127 - 1 - int(round(0.5 * math.log2(K)))
    s = torch.randint(base - 1, base + 2, (E, N, K // 32), generator=g, device=dev, dtype=torch.uint8)
    return w, s


def _rows(g, act, rows, K, dev):
    """Activation rows with their scales, as dispatch or the quantiser leaves
    them."""
    if act == "fp8":
        q = torch.empty(rows, K, dtype=torch.uint8, device=dev)
        for at in range(0, rows, 16384):
            v = torch.randn(min(16384, rows - at), K, generator=g, device=dev).mul_(150.0).clamp_(-448.0, 448.0)
            q[at:at + v.shape[0]] = v.to(torch.float8_e4m3fn).view(torch.uint8)
        return q, torch.rand(rows, K // 128, generator=g, device=dev).add_(2.5).div_(448.0)
    q = _pool(g, rows * K // 2, dev).view(rows, K // 2)
    return q, torch.randint(125, 128, (rows, K // 32), generator=g, device=dev, dtype=torch.uint8)


def prepare(case, seed):
    dev = _device()
    g = torch.Generator(device=dev)
    g.manual_seed(seed * 7919 + 13)
    c = dict(case)
    if c["op"] == "quantize":
        dt = torch.float32 if c["wide"] else torch.bfloat16
        x = torch.empty(c["rows"], c["cols"], dtype=dt, device=dev)
        for at in range(0, c["rows"], 16384):
            x[at:at + 16384] = torch.randn(min(16384, c["rows"] - at), c["cols"], generator=g, device=dev)
        x[:, torch.randint(0, c["cols"], (max(1, c["cols"] // 100),), generator=g, device=dev)] *= 100  # outlier channels
        x[0, :64] = 0
        return dict(case=c, x=x)
    T, E, k = c["T"], c["E"], c["k"]
    if c["op"] == "balance":
        logits, idx = _picks(g, T, E, k, 0.5, 0.0, dev)
        cuts = torch.randint(0, T + 1, (c["S"] - 1,), generator=g, device=dev).sort().values
        seq = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), cuts,
                         torch.full((1,), T, dtype=torch.int64, device=dev)]).to(torch.int32)
        mask = None
        if c["pad"]:
            mask = (torch.rand(T, generator=g, device=dev) >= c["pad"]).to(torch.uint8)
            # padding rows hold whatever was there: every other one NaN
            logits[(mask == 0) & (torch.arange(T, device=dev) % 2 == 0)] = float("nan")
            idx[mask == 0] = -1
        gl = torch.rand(c["S"], generator=g, device=dev).mul_(1e-2).add_(1e-3)
        return dict(case=c, logits=logits, idx=idx, seq=seq, mask=mask, grad_loss=gl)
    K, N = c["K"], c["N"]
    _, idx = _picks(g, T, E, k, c["skew"], c["lost"], dev)
    flat = idx[idx >= 0].long()
    count = torch.zeros(E, dtype=torch.int64, device=dev).index_add_(0, flat, torch.ones_like(flat))
    off = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), count.cumsum(0)]).to(torch.int32)
    count = count.to(torch.int32)
    rows = E * T if c["slots"] == "capacity" else T * k
    st = dict(case=c, count=count, off=off, most=int(count.max()))
    st["x"], st["xs"] = _rows(g, c["act"], rows, K, dev)
    if c["slots"] == "capacity":  # rows no token took hold NaN
        unused = (torch.arange(T, device=dev)[None] >= count[:, None]).view(-1)
        if c["act"] == "fp8":
            st["x"][unused] = 0x7F
            st["xs"][unused] = float("nan")
        else:
            st["xs"][unused] = 255
    st["w"], st["ws"] = _weights(g, E, N if c["op"] == "product" else 2 * N, K, dev)
    width = N
    if c["op"] == "experts":
        width = K
        st["w2"], st["w2s"] = _weights(g, E, K, N, dev)
    st["out"] = torch.zeros(rows, width, dtype=torch.bfloat16, device=dev)  # rows of no token stay as they are
    return st


# ------------------------------------------------------------- plain forms

def _round_e2m1(v):
    """The nearest E2M1 value of each of v's values, ties to the even code,
    saturated to 6 (0, .5, 1, 1.5 and 2 lie half a unit apart, 2, 3 and 4 one,
    4 and 6 two)."""
    a = v.clamp(-6.0, 6.0)
    step = torch.where(a.abs() < 2, 0.5, torch.where(a.abs() < 4, 1.0, 2.0))
    return torch.round(a / step) * step


@functools.lru_cache(None)
def _tables(dev):
    """Values of the 256 E2M1 code pairs, and of the 256 E8M0 scales."""
    one = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    one = one + [-v for v in one]
    pair = torch.tensor([[one[b & 15], one[b >> 4]] for b in range(256)], dtype=torch.float32, device=dev)
    scale = torch.tensor([2.0 ** (b - 127) for b in range(255)] + [float("nan")], dtype=torch.float64).float()
    return pair, scale.to(dev)


def _from_mxfp4(codes, scales):
    pair, scale = _tables(codes.device)
    v = pair[codes.int()].view(*codes.shape[:-1], -1, 32)
    v *= scale[scales.int()].unsqueeze(-1)
    return v.view(*codes.shape[:-1], -1)


def _from_fp8(codes, scales):
    v = codes.view(torch.float8_e4m3fn).float().view(*codes.shape[:-1], -1, 128)
    v *= scales.unsqueeze(-1)
    return v.view(*codes.shape[:-1], -1)


def _to_mxfp4(x):
    """Values and E8M0 scales of x [rows, cols] in MXFP4."""
    b = x.float().view(x.shape[0], -1, 32)
    amax = b.abs().amax(-1)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 3, -127).clamp_(-127, 127)
    v = _round_e2m1(torch.ldexp(b, -e.unsqueeze(-1)))
    return torch.ldexp(v, e.unsqueeze(-1)).view(x.shape), (e + 127).to(torch.uint8)


def _plain_balance(st):
    c, x, idx, seq = st["case"], st["logits"], st["idx"], st["seq"]
    T, E, k, S = c["T"], c["E"], c["k"], c["S"]
    sid = torch.searchsorted(seq[1:-1], torch.arange(T, dtype=torch.int32, device=x.device), right=True)
    keep = st["mask"] != 0 if st["mask"] is not None else torch.ones(T, dtype=torch.bool, device=x.device)
    x = x.masked_fill(~keep[:, None], 0.0)
    s, rest = 1 / (1 + torch.exp(-x)), 1 / (1 + torch.exp(x))
    p = s / s.sum(1, keepdim=True)
    member = ((sid[None] == torch.arange(S, device=x.device)[:, None]) & keep[None]).double()
    n = member.sum(1)
    on = (idx >= 0) & keep[:, None]
    at = sid[:, None] * E + idx
    count = torch.zeros(S * E + 1, dtype=torch.int32, device=x.device)
    count.index_add_(0, torch.where(on, at, S * E).view(-1), torch.ones(T * k, dtype=torch.int32, device=x.device))
    count = count[:-1].view(S, E)
    some = n.clamp(min=1)[:, None]
    prob = member @ p.double() / some
    share = count.double() * E / (k * some)
    loss = (share * prob).sum(1)
    d = (share / some).float()[sid]
    lift = d - (d * p).sum(1, keepdim=True)
    grad = st["grad_loss"][sid][:, None] * lift * p * rest * keep[:, None]
    return dict(loss=loss.float(), count=count, ntok=n.to(torch.int32), prob=prob.float(), grad=grad)


def _plain_product(st, x, w, ws):
    """x [rows, K] in 32 bits times the rows' experts' weights, 32 bits."""
    c, off, count = st["case"], st["off"], st["count"]
    E, rows = c["E"], x.shape[0]
    if c["slots"] == "capacity":
        used = (torch.arange(c["T"], device=x.device)[None] < count[:, None])[..., None]
        x = torch.where(used, x.view(E, c["T"], -1), 0.0)
        return torch.bmm(x, _from_mxfp4(w, ws).transpose(1, 2)).view(rows, -1)
    r = torch.arange(rows, dtype=torch.int32, device=x.device)
    owner = torch.searchsorted(off[1:], r, right=True)
    used = (owner < E)[:, None]
    owner = owner.clamp(max=E - 1)
    if rows <= E:  # few rows: the weights of each row's expert
        return torch.bmm(_from_mxfp4(w[owner], ws[owner]), x[..., None])[..., 0] * used
    most = st["most"]
    at = torch.where(used[:, 0], owner * most + r - off[owner], E * most)
    full = torch.zeros(E * most + 1, x.shape[1], device=x.device)
    full[at] = x
    y = torch.bmm(full[:-1].view(E, most, -1), _from_mxfp4(w, ws).transpose(1, 2)).view(E * most, -1)
    return y[at.clamp(max=E * most - 1)] * used


def _plain_experts(st):
    c = st["case"]
    y = _plain_product(st, (_from_fp8 if c["act"] == "fp8" else _from_mxfp4)(st["x"], st["xs"]), st["w"], st["ws"])
    if c["op"] != "product":
        gate, up = y.chunk(2, dim=1)
        y = gate / (1 + torch.exp(-gate)) * up
        if c["op"] == "experts":
            y = _plain_product(st, _to_mxfp4(y)[0], st["w2"], st["w2s"])
    return y.to(torch.bfloat16)


# ------------------------------------------------------ the package's calls

@functools.lru_cache(None)
def _config(T, H, E, k):
    import combine_group_limited_amd as ep
    return ep.Config(T=T, H=H, E=E, G=1, TG=1, k=k, R=1)


def _own(st):
    import combine_group_limited_amd as ep
    c = st["case"]
    if c["op"] == "quantize":
        codes, scales = ep.mxfp4_quantize(st["x"])
        return dict(values=ep.mxfp4_dequantize(codes, scales), scales=scales)
    if c["op"] == "balance":
        cfg = _config(c["T"], 128, c["E"], c["k"])
        r = ep.balance_loss(cfg, st["logits"], st["idx"], st["seq"], st["mask"])
        grad = ep.balance_loss_backward(cfg, st["logits"], r["count"], r["ntok"], st["grad_loss"], st["seq"],
                                        st["mask"])
        return dict(loss=r["loss"], count=r["count"], ntok=r["ntok"], prob=r["prob"], grad=grad)
    cfg, packed = _config(c["T"], 128, c["E"], c["k"]), c["slots"] == "rows"
    x, xs = st["x"], st["xs"]
    if c["op"] != "product":
        last = dict(out_dtype="mxfp4") if c["op"] == "experts" else dict(out=st["out"])
        if packed:
            y = ep.expert_swiglu(cfg, x, xs, st["w"], st["ws"], st["off"], **last)
        else:
            y = ep.expert_swiglu_ll(cfg, c["T"], x, xs, st["w"], st["ws"], st["count"], **last)
        if c["op"] == "swiglu":
            return y
        x, xs = y
    w, ws = (st["w2"], st["w2s"]) if c["op"] == "experts" else (st["w"], st["ws"])
    if packed:
        return ep.expert_product(cfg, x, xs, w, ws, st["off"], out=st["out"])
    return ep.expert_product_ll(cfg, c["T"], x, xs, w, ws, st["count"], out=st["out"])


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "quantize":
        values, scales = _to_mxfp4(state["x"])
        return dict(values=values.to(torch.bfloat16), scales=scales)
    return _plain_balance(state) if op == "balance" else _plain_experts(state)


def work(case):
    c = case
    if c["op"] == "quantize":
        n = c["rows"] * c["cols"]
        # the rows in, codes and scales out; and back to 16-bit values
        return dict(bytes=n * (4 if c["wide"] else 2) + 2 * (n // 2 + n // 32) + 2 * n, flops=4 * n)
    T, E, k = c["T"], c["E"], c["k"]
    if c["op"] == "balance":
        # logits in twice (the gradient needs the whole batch's counts), picks in, gradient out
        return dict(bytes=T * (12 * E + 4 * k) + 8 * c["S"] * E, flops=40 * T * E)
    K, N = c["K"], c["N"]
    picks = T * k * (1 - c["lost"])
    active = E * (1 - (1 - k / E) ** T)  # experts that some token picks, under even routing
    width = N if c["op"] == "product" else 2 * N
    row = K + K / 32 if c["act"] == "fp8" else K / 2 + K / 32
    moved, flops = active * width * K * 17 / 32 + picks * row, 2.0 * picks * width * K
    if c["op"] == "experts":
        moved += active * N * K * 17 / 32 + 2 * picks * N * 17 / 32 + 2 * picks * K
        flops += 2.0 * picks * N * K
    else:
        moved += 2 * picks * N
    return dict(bytes=moved, flops=flops)


# ------------------------------------------- the definition, in 64 bits

def _value64(codes):
    """E2M1 codes (one to a byte) from sign, exponent and fraction bits."""
    e, m = ((codes >> 1) & 3).double(), (codes & 1).double()
    v = torch.where(e == 0, m / 2, (1 + m / 2) * 2.0 ** (e - 1))
    return torch.where(codes >= 8, -v, v)


def _mxfp4_64(codes, scales):
    v = torch.stack((_value64(codes & 15), _value64(codes >> 4)), dim=-1).flatten(-2)
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, dim=-1)


def _quantize64(x):
    """MXFP4 values and scales by search over the eight magnitudes."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=x.device)
    mid = (grid[1:] + grid[:-1]) / 2
    b = x.double().reshape(x.shape[0], -1, 32)
    big = b.abs().amax(-1, keepdim=True)
    # the power of two at or below the largest magnitude, two binades down (E2M1's largest is 1.5 * 2^2)
    e = torch.floor(torch.log2(big.clamp(min=2.0 ** -200)))
    e = torch.where(torch.exp2(e) > big, e - 1, e)
    e = (torch.where(torch.exp2(e + 1) <= big, e + 1, e) - 2).clamp(-127, 127)
    a = b.abs() * torch.exp2(-e)
    low = torch.bucketize(a, mid)                # a tie goes to the lower neighbour here,
    high = torch.bucketize(a, mid, right=True)   # to the upper one here: take the even code
    q = grid[torch.where(low % 2 == 0, low, high)] * torch.exp2(e)
    return torch.where(b < 0, -q, q).reshape(x.shape), (e.squeeze(-1) + 127).to(torch.uint8)


def exact(case, seed):
    st = prepare(case, seed)
    c = st["case"]
    if c["op"] == "quantize":
        values = torch.empty(st["x"].shape, dtype=torch.float64, device=st["x"].device)
        scales = []
        for at in range(0, c["rows"], 8192):
            v, s = _quantize64(st["x"][at:at + 8192])
            values[at:at + 8192] = v
            scales.append(s)
        return dict(values=values, scales=torch.cat(scales))
    T, E, k = c["T"], c["E"], c["k"]
    if c["op"] == "balance":
        S, seq = c["S"], st["seq"].tolist()
        x = st["logits"].double()
        keep = st["mask"].bool() if st["mask"] is not None else torch.ones(T, dtype=torch.bool, device=x.device)
        loss, count, prob = [], [], []
        grad = torch.zeros_like(x)
        for s in range(S):
            rows = torch.nonzero(keep[seq[s]:seq[s + 1]]).squeeze(1) + seq[s]
            n = rows.numel()
            sc = torch.sigmoid(x[rows])
            p = sc / sc.sum(1, keepdim=True)
            picks = st["idx"][rows]
            cnt = torch.bincount(picks[picks >= 0].long(), minlength=E)
            f = cnt.double() * E / (k * max(n, 1))
            mean = p.sum(0) / max(n, 1)
            loss.append((f * mean).sum())
            count.append(cnt)
            prob.append(mean)
            if n:  # p_i = s_i / sum s, ds/dx = s (1 - s)
                dp = f / n
                ds = (dp - (p * dp).sum(1, keepdim=True)) / sc.sum(1, keepdim=True)
                grad[rows] = st["grad_loss"][s].double() * ds * sc * torch.sigmoid(-x[rows])
        return dict(loss=torch.stack(loss), count=torch.stack(count).to(torch.int32), ntok=None,
                    prob=torch.stack(prob), grad=grad)
    count = st["count"].tolist()
    width = c["K"] if c["op"] == "experts" else c["N"]
    y = torch.zeros(st["x"].shape[0], width, dtype=torch.float64, device=st["x"].device)
    start = 0
    for e in range(E):
        if c["slots"] == "capacity":
            start = e * T
        rows = slice(start, start + count[e])
        start += count[e]
        if not count[e]:
            continue
        if c["act"] == "fp8":
            x = st["x"][rows].view(torch.float8_e4m3fn).double() * st["xs"][rows].double().repeat_interleave(128, dim=1)
        else:
            x = _mxfp4_64(st["x"][rows], st["xs"][rows])
        v = x @ _mxfp4_64(st["w"][e], st["ws"][e]).t()
        if c["op"] != "product":
            gate, up = v[:, :c["N"]], v[:, c["N"]:]
            v = gate * torch.sigmoid(gate) * up
            if c["op"] == "experts":
                v = _quantize64(v)[0] @ _mxfp4_64(st["w2"][e], st["w2s"][e]).t()
        y[rows] = v
    return y
