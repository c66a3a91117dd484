"""The operators of an expert layer's training and serving, as they are measured.

Three operators that a program runs next to the quantile-balanced bias:

* ``route``: the K experts of every token by biased score, their normalised
  gates, the per-expert counts of every sequence, the sequence-wise balance
  loss and the gradient of both through the sigmoid;
* ``linear`` and ``experts``: the matrix product in 8-bit floating point with
  a power-of-two scale for each block of 128, for one weight matrix and for
  one matrix per expert, forward and backward, its inputs quantised on the way;
* ``exchange``: the order that puts each expert's tokens side by side, the
  gate-weighted sum of what the experts return, and its gradients.

``run`` computes them in plain torch operations, or with the library's entry
points where ``own`` is set.
"""
import math
import random

import torch

own = False

BLOCK = 128          # values along the summed dimension that share a scale
TOP = 448.0          # the largest value of the 8-bit type (e4m3)
EXPERTS = (16, 32, 64, 128, 256)


# --------------------------------------------------------------------------
# the cases
# --------------------------------------------------------------------------

def listed():
    return [
        # a decoding step's router: the experts and gates of 16 tokens, no loss
        dict(name="route_step", op="route", N=16, E=256, K=8, seqs=0, masked=False, train=False),
        # a small packed batch: sequences of all lengths (none and one among them), a tenth of it padding
        dict(name="route_ragged", op="route", N=5003, E=64, K=6, seqs=41, masked=True, train=True),
        # a training microbatch at the bias update's own shape (256 experts, 6 a token): 32 packed sequences
        dict(name="route_train", op="route", N=131072, E=256, K=6, seqs=32, masked=False, train=True),
        # one token through a projection: bound by the weight's bytes
        dict(name="linear_token", op="linear", M=1, N=4096, C=4096, train=False),
        # sizes that are no multiple of a tile or of a block, forward and backward
        dict(name="linear_odd", op="linear", M=777, N=2005, C=1001, train=True),
        # a projection's training step: three large products
        dict(name="linear_train", op="linear", M=8192, N=8192, C=4096, train=True),
        # a decoding step's experts: 16 tokens, 8 experts each of 256, most experts without a row or with one
        dict(name="experts_step", op="experts", rows=128, E=256, N=1024, C=2048, align=1, skew=0.3, train=False),
        # few, unequal experts with odd sizes, some of them empty
        dict(name="experts_odd", op="experts", rows=1999, E=16, N=730, C=1163, align=128, skew=2.0, train=True),
        # a microbatch's experts: 16,384 tokens, 8 experts each
        dict(name="experts_train", op="experts", rows=131072, E=64, N=1024, C=2048, align=128, skew=0.2, train=True),
        # a decoding step's exchange: order and weighted sum
        dict(name="exchange_step", op="exchange", N=16, K=8, E=256, H=2048, align=1, drop=0.0, train=False),
        # odd sizes, a seventh of the tokens routed nowhere
        dict(name="exchange_ragged", op="exchange", N=3001, K=6, E=64, H=1101, align=128, drop=0.14, train=True),
        # a microbatch's exchange with its gradients
        dict(name="exchange_train", op="exchange", N=32768, K=8, E=256, H=2048, align=128, drop=0.0, train=True),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over its logarithm; about half of them odd."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["route", "linear", "experts", "exchange"])
    train = rng.random() < 0.6
    if op == "route":
        E = rng.choice(EXPERTS)
        N = _spread(rng, 1, 131072)
        seqs = _spread(rng, 1, max(1, min(256, N))) if train else 0
        return dict(op=op, N=N, E=E, K=rng.randint(1, min(15, E - 1)), seqs=seqs,
                    masked=train and rng.random() < 0.5, train=train)
    if op == "linear":
        return dict(op=op, M=_spread(rng, 1, 8192), N=_spread(rng, 16, 8192), C=_spread(rng, 16, 4096), train=train)
    if op == "experts":
        return dict(op=op, rows=_spread(rng, 1, 65536), E=rng.choice(EXPERTS[:3]) if train else rng.choice(EXPERTS),
                    N=_spread(rng, 64, 1024), C=_spread(rng, 64, 2048),
                    align=128 if train else rng.choice([1, 16, 128]), skew=round(rng.uniform(0.0, 2.0), 2), train=train)
    E = rng.choice(EXPERTS)
    return dict(op=op, N=_spread(rng, 1, 32768), K=rng.randint(1, min(8, E - 1)), E=E, H=_spread(rng, 64, 2048),
                align=rng.choice([1, 16, 128]), drop=rng.choice([0.0, 0.1, 0.5]), train=train)


def _off(case):
    """The experts' row offsets of an `experts` case (E + 1 whole numbers): its
    rows dealt out by unequal weights, every expert's start rounded up."""
    rng = random.Random("%(rows)d %(E)d %(N)d %(C)d %(align)d %(skew)s" % case)
    weight = [math.exp(case["skew"] * rng.gauss(0.0, 1.0)) for _ in range(case["E"])]
    count = [0] * case["E"]
    for e in rng.choices(range(case["E"]), weight, k=case["rows"]):
        count[e] += 1
    off, a = [0], case["align"]
    for c in count:
        off.append(off[-1] + -(-c // a) * a)
    return off, count


def _capacity(case):
    """Rows that hold any dispatch of an `exchange` case."""
    pairs, a = case["N"] * case["K"], case["align"]
    return -(-(pairs + min(case["E"], pairs) * (a - 1)) // a) * a


def _ld(n):
    return -(-n // BLOCK) * BLOCK


def _sld(n):
    return -(-n // (4 * BLOCK)) * 4


def work(case):
    op = case["op"]
    if op == "route":
        N, E, K, B = case["N"], case["E"], case["K"], max(1, case["seqs"])
        scores, picks = 4 * N * E, 8 * N * K
        if not case["train"]:
            return dict(bytes=scores + 4 * E + picks, flops=N * E * 2)
        # the gradient follows the whole batch's counts, yet the scores are one input, read once;
        # in: scores, bias, gate gradients; out: experts, gates, counts, loss, gradient
        return dict(bytes=2 * scores + picks + 4 * N * K + 4 * B * E + N * case["masked"], flops=N * E * 10)
    if op == "exchange":
        N, K, H, E = case["N"], case["K"], case["H"], case["E"]
        R = N * K * (1.0 - case["drop"])
        fwd = 8 * N * K + 4 * _capacity(case) + 4 * E + 2 * R * H + 4 * N * K + 2 * N * H
        bwd = 2 * N * H + 2 * _capacity(case) * H + 4 * N * K if case["train"] else 0
        return dict(bytes=int(fwd + bwd), flops=int(2 * R * H + (3 * R * H if case["train"] else 0)))
    if op == "linear":
        M, G = case["M"], 1
        N, C, real, held = case["N"], case["C"], M, 1
    else:
        off, count = _off(case)
        M, real, held = off[-1], case["rows"], sum(c > 0 for c in count)
        N, C, G = case["N"], case["C"], case["E"]
    b = 2 * real * C + held * N * C + 2 * M * N
    if case["train"]:
        b += 2 * real * N + 2 * M * C + 4 * G * N * C
    return dict(bytes=int(b), flops=2 * real * N * C * (3 if case["train"] else 1))


# --------------------------------------------------------------------------
# the inputs
# --------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _empty(shape, dtype):
    return torch.empty(shape, device="cuda", dtype=dtype)


def _sequences(case, seed):
    """Offsets of a packed batch: unequal lengths, every seventh sequence empty
    where there are many, and a short tail of tokens that belong to none."""
    rng = random.Random(seed)
    N, B = case["N"], case["seqs"]
    part = [0.0 if B > 8 and q % 7 == 3 else rng.expovariate(1.0) + 0.05 for q in range(B)]
    end = N - (N // 50 if case["masked"] else 0)
    total, run, off = sum(part), 0.0, [0]
    for p in part:
        run += p
        off.append(int(round(end * run / total)))
    off[-1] = end
    return off


def prepare(case, seed):
    g = _gen(seed)
    op, st = case["op"], dict(case=case)
    if op == "route":
        N, E, K, B = case["N"], case["E"], case["K"], case["seqs"]
        logits = _randn(g, N, E) + 0.5 * _randn(g, 1, E)
        st["s"] = torch.sigmoid(logits)
        st["b"] = (torch.rand((E,), generator=g, device="cuda") - 0.5) * 0.2
        st["topk"], st["gate"] = _empty((N, K), torch.int32), _empty((N, K), torch.float32)
        if case["train"]:
            st["seq_off"] = torch.tensor(_sequences(case, seed), dtype=torch.int32, device="cuda")
            st["valid"] = (torch.rand((N,), generator=g, device="cuda") > 0.1).to(torch.uint8) if case["masked"] else None
            st["coef"] = 1e-2
            # the loss is one term of a scaled sum; the gates' gradient comes from the weighted sum
            st["dloss"] = torch.full((1,), 512.0, device="cuda")
            st["dgate"] = 1e-3 * _randn(g, N, K)
            st["count"], st["weight"] = _empty((B, E), torch.int32), _empty((B, E), torch.float32)
            st["loss"], st["dlogits"] = _empty((1,), torch.float32), _empty((N, E), torch.float32)
            # room for the library's partial sums, for every sequence and every block of tokens
            st["ws"] = _empty((16 * E * (B + N // 32 + 2),), torch.uint8)
        return st
    if op == "exchange":
        N, K, E, H, a, R = case["N"], case["K"], case["E"], case["H"], case["align"], _capacity(case)
        bias = 0.7 * _randn(g, 1, E)
        ids = torch.topk(_randn(g, N, E) + bias, K, dim=1).indices.to(torch.int32)
        keep = torch.rand((N, 1), generator=g, device="cuda") >= case["drop"]
        st["topk"] = torch.where(keep, ids, torch.full_like(ids, -1)).contiguous()
        gate = torch.rand((N, K), generator=g, device="cuda") + 0.1
        st["gate"] = (gate / gate.sum(1, keepdim=True)) * keep
        st["rows"] = _randn(g, R, H).to(torch.bfloat16)
        st["off"], st["row_src"] = _empty((E + 1,), torch.int32), _empty((R,), torch.int32)
        st["pos"], st["out"] = _empty((N, K), torch.int32), _empty((N, H), torch.bfloat16)
        st["ws"] = _empty((8 * E * (N * K // 512 + 2),), torch.uint8)
        if case["train"]:
            st["dout"] = _randn(g, N, H).to(torch.bfloat16)
            st["drows"], st["dgate"] = _empty((R, H), torch.bfloat16), _empty((N, K), torch.float32)
        return st
    N, C = case["N"], case["C"]
    if op == "linear":
        M, G = case["M"], 1
        live = torch.ones((M, 1), dtype=torch.bool, device="cuda")
    else:
        off, count = _off(case)
        M, G = off[-1], case["E"]
        st["off"] = torch.tensor(off, dtype=torch.int32, device="cuda")
        st["largest"] = max(b - a for a, b in zip(off, off[1:]))
        start = st["off"].long()
        owner = torch.searchsorted(start[1:], torch.arange(M, device="cuda"), right=True)
        slot = torch.arange(M, device="cuda") - start[owner]
        live = (slot < torch.tensor(count, device="cuda")[owner]).unsqueeze(1)
    # activations whose channels differ in size, as normalised hidden states have them;
    # an expert's unused rows are zero
    st["x"] = (_randn(g, M, C) * torch.exp(0.5 * _randn(g, 1, C)) * live).to(torch.bfloat16)
    w = _randn(g, G, N, C) / math.sqrt(C)
    st["w"], st["w_scale"] = _lay_out(w)
    st["wt"], st["wt_scale"] = _lay_out(w.transpose(1, 2).contiguous()) if case["train"] else (None, None)
    if op == "linear":
        for k in ("w", "w_scale", "wt", "wt_scale"):
            st[k] = None if st[k] is None else st[k][0]
    del w
    f8, u8 = torch.float8_e4m3fn, torch.uint8
    st["xq"], st["xs"] = _empty((M, _ld(C)), f8), _empty((M, _sld(C)), u8)
    st["y"] = _empty((M, N), torch.bfloat16)
    if case["train"]:
        st["dy"] = (_randn(g, M, N) * live).to(torch.bfloat16)
        st["dyq"], st["dys"] = _empty((M, _ld(N)), f8), _empty((M, _sld(N)), u8)
        st["dyt"], st["dyts"] = _empty((N, _ld(M)), f8), _empty((N, _sld(M)), u8)
        st["xt"], st["xts"] = _empty((C, _ld(M)), f8), _empty((C, _sld(M)), u8)
        st["dx"] = _empty((M, C), torch.bfloat16)
        st["dw"] = _empty((N, C) if op == "linear" else (G, N, C), torch.float32)
    return st


def _lay_out(w):
    """A weight stack [G, N, C] as a program holds it: e4m3 [G, N, ld(C)] and the
    exponents (plus 127) of its 128 x 128 blocks, uint8 [G, blocks of N, sld(C)]."""
    G, N, C = w.shape
    full = torch.nn.functional.pad(w, (0, _ld(C) - C, 0, _ld(N) - N))
    t = full.view(G, -1, BLOCK, _ld(C) // BLOCK, BLOCK)
    e = _exponent(t.abs().amax(dim=(2, 4), keepdim=True))
    q = (t * _two_to(-e)).view(G, _ld(N), _ld(C))[:, :N].to(torch.float8_e4m3fn).contiguous()
    scale = torch.nn.functional.pad((e + 127).to(torch.uint8).view(G, -1, _ld(C) // BLOCK),
                                    (0, _sld(C) - _ld(C) // BLOCK))
    return q, scale.contiguous()


# --------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------

def _exponent(amax):
    """The least whole e >= -126 with amax <= 448 * 2^e."""
    m, x = torch.frexp(amax)
    return torch.where(m <= 0.875, x - 9, x - 8).clamp(min=-126).to(torch.int32)


def _two_to(e):
    return ((e + 127) << 23).view(torch.float32)


def _stand_for(x):
    """x [rows, n] rounded to 8 bits along n, as the float32 values it then stands for."""
    t = torch.nn.functional.pad(x.float(), (0, _ld(x.shape[1]) - x.shape[1])).reshape(x.shape[0], -1, BLOCK)
    e = _exponent(t.abs().amax(dim=2, keepdim=True))
    return ((t * _two_to(-e)).to(torch.float8_e4m3fn).float() * _two_to(e)).reshape(x.shape[0], -1)[:, :x.shape[1]]


def _weight_values(q, scale, C):
    """The float32 values of a laid out weight [.., N, ld(C)], as [.., N, C]."""
    N, ld = q.shape[-2:]
    f = _two_to(scale[..., :ld // BLOCK].to(torch.int32) - 127)
    f = f.repeat_interleave(BLOCK, -2)[..., :N, :].repeat_interleave(BLOCK, -1)
    return (q.float() * f)[..., :C]


def _plain_linear(st):
    x, C = st["x"], st["x"].shape[1]
    w = _weight_values(st["w"], st["w_scale"], C)
    y = torch.mm(_stand_for(x), w.t()).to(torch.bfloat16)
    if not st["case"]["train"]:
        return dict(y=y)
    dy = st["dy"]
    wt = _weight_values(st["wt"], st["wt_scale"], dy.shape[1])
    dx = torch.mm(_stand_for(dy), wt.t()).to(torch.bfloat16)
    dw = torch.mm(_stand_for(dy.t()), _stand_for(x.t()).t())
    return dict(y=y, dx=dx, dw=dw)


def _plain_experts(st):
    x, off = st["x"], st["off"].long()
    M, C = x.shape
    G, most = off.numel() - 1, st["largest"]
    at = torch.arange(M, device=x.device)
    owner = torch.searchsorted(off[1:], at, right=True)
    at = owner * most + at - off[owner]

    def spread(t):
        """Rows [M, n] as one padded block of rows for each expert, [G, most, n]."""
        full = torch.zeros((G * most, t.shape[1]), dtype=t.dtype, device=t.device)
        return full.index_copy_(0, at, t).view(G, most, -1)

    def product(t, w):
        return torch.bmm(spread(t), w.transpose(1, 2).contiguous()).view(G * most, -1)[at].to(torch.bfloat16)

    y = product(_stand_for(x), _weight_values(st["w"], st["w_scale"], C))
    if not st["case"]["train"]:
        return dict(y=y)
    dy = st["dy"]
    N = dy.shape[1]
    dx = product(_stand_for(dy), _weight_values(st["wt"], st["wt_scale"], N))
    # along the rows: every expert's rows begin at a multiple of 128, so no block spans two experts
    dyt = spread(_stand_for(dy.t()).t().contiguous()).transpose(1, 2).contiguous()
    dw = torch.bmm(dyt, spread(_stand_for(x.t()).t().contiguous()))
    return dict(y=y, dx=dx, dw=dw)


def _plain_route(st):
    s, b, case = st["s"], st["b"], st["case"]
    N, E = s.shape
    K = case["K"]
    order = torch.sort(s + b, dim=1, descending=True, stable=True).indices[:, :K]
    chosen = torch.gather(s, 1, order)
    total = chosen.sum(1, keepdim=True)
    per = torch.where(total > 0, 1 / total, torch.zeros_like(total))
    gate = chosen * per
    if not case["train"]:
        return dict(topk=order.to(torch.int32), gate=gate)
    off, B = st["seq_off"].long(), case["seqs"]
    seq = torch.searchsorted(off[1:], torch.arange(N, device=s.device), right=True)
    live = seq < B
    if st["valid"] is not None:
        live = live & (st["valid"] != 0)
    seq = seq.clamp(max=B - 1)
    lv = live.unsqueeze(1)
    topk = torch.where(lv, order, torch.full_like(order, -1)).to(torch.int32)
    gate = torch.where(lv, gate, torch.zeros_like(gate))
    # counts and summed probabilities of each sequence: products with its tokens' indicator, in 64 bits
    of = ((torch.arange(B, device=s.device).unsqueeze(1) == seq) & live).double()
    hit = torch.zeros((N, E), dtype=torch.float64, device=s.device).scatter_(1, order, 1.0)
    count = torch.mm(of, hit)
    del hit
    z = s.sum(1, keepdim=True)
    inv = torch.where(lv & (z > 0), 1 / z, torch.zeros_like(z))
    p = s * inv
    psum = torch.mm(of, p.double())
    del of
    T = count.sum(1, keepdim=True) / K
    filled = (T > 0).sum().clamp(min=1)
    share = torch.where(T > 0, 1 / T, torch.zeros_like(T))
    f = count * share * (E / K)
    loss = (st["coef"] / filled * (f * psum * share).sum()).float().reshape(1)
    # the gradient: a shift of f common to a row changes nothing, and f - 1 keeps what 32 bits would lose
    weight = (st["coef"] / filled * (f - 1) * share).float() * st["dloss"]
    wr = weight[seq]
    ds = (wr - (wr * p).sum(1, keepdim=True)) * inv
    dg = torch.where(lv, st["dgate"], torch.zeros_like(st["dgate"]))
    ds.scatter_add_(1, order, (dg - (dg * gate).sum(1, keepdim=True)) * per)
    return dict(topk=topk, gate=gate, count=count.to(torch.int32), loss=loss, dlogits=ds * (s * (1 - s)))


def _plain_exchange(st):
    case, topk, gate, rows = st["case"], st["topk"], st["gate"], st["rows"]
    N, K = topk.shape
    E, a = case["E"], case["align"]
    R, H = rows.shape
    dev = topk.device
    key = topk.reshape(-1).long()
    key = torch.where((key >= 0) & (key < E), key, torch.full_like(key, E))
    key, order = torch.sort(key, stable=True)
    first = torch.searchsorted(key, torch.arange(E + 1, device=dev))
    off = torch.zeros(E + 1, dtype=torch.int64, device=dev)
    off[1:] = torch.cumsum((first[1:] - first[:-1] + a - 1) // a * a, 0)
    routed = key < E
    row = off[key.clamp(max=E - 1)] + torch.arange(N * K, device=dev) - first[key.clamp(max=E - 1)]
    pos = torch.full((N * K,), -1, dtype=torch.int64, device=dev)
    pos[order] = torch.where(routed, row, torch.full_like(row, -1))
    row_src = torch.full((R + 1,), -1, dtype=torch.int64, device=dev)
    row_src[torch.where(routed, row, torch.full_like(row, R))] = order // K
    row_src = row_src[:R]
    pos = pos.view(N, K)
    live = (pos >= 0).unsqueeze(2)
    picked = torch.where(live, rows[pos.clamp(min=0)].float(), torch.zeros((), device=dev))
    out = (picked * gate.unsqueeze(2)).sum(1).to(torch.bfloat16)
    found = dict(off=off.to(torch.int32), row_src=row_src.to(torch.int32), pos=pos.to(torch.int32), out=out)
    if not case["train"]:
        return found
    dout = st["dout"].float()
    found["dgate"] = (picked * dout.unsqueeze(1)).sum(2)
    del picked
    of_row = torch.zeros(R + 1, device=dev)
    of_row[torch.where(pos >= 0, pos, torch.full_like(pos, R))] = gate
    drows = dout[row_src.clamp(min=0)] * of_row[:R].unsqueeze(1)
    found["drows"] = torch.where((row_src >= 0).unsqueeze(1), drows, torch.zeros((), device=dev)).to(torch.bfloat16)
    return found


# --------------------------------------------------------------------------
# the library's calls
# --------------------------------------------------------------------------

def _own_route(st):
    from exact_quantile_selection_amd import qb

    K = st["case"]["K"]
    if not st["case"]["train"]:
        qb.qb_balance_forward(st["s"], st["b"], K, st["topk"], gate=st["gate"])
        return dict(topk=st["topk"], gate=st["gate"])
    qb.qb_balance_forward(st["s"], st["b"], K, st["topk"], gate=st["gate"], count=st["count"], weight=st["weight"],
                          loss=st["loss"], ws=st["ws"], coef=st["coef"], seq_off=st["seq_off"], valid=st["valid"])
    qb.qb_balance_backward(st["s"], st["topk"], weight=st["weight"], dloss=st["dloss"], dgate=st["dgate"],
                           dlogits=st["dlogits"], seq_off=st["seq_off"], valid=st["valid"])
    return {k: st[k] for k in ("topk", "gate", "count", "loss", "dlogits")}


def _own_product(st):
    from exact_quantile_selection_amd import qb

    off = st.get("off")
    qb.qb_fp8_quantize(st["x"], st["xq"], st["xs"])
    qb.qb_fp8_product(st["xq"], st["xs"], st["w"], st["w_scale"], st["y"], off=off)
    if not st["case"]["train"]:
        return dict(y=st["y"])
    qb.qb_fp8_quantize(st["dy"], st["dyq"], st["dys"])
    qb.qb_fp8_product(st["dyq"], st["dys"], st["wt"], st["wt_scale"], st["dx"], off=off)
    qb.qb_fp8_quantize_cols(st["x"], st["xt"], st["xts"])
    qb.qb_fp8_quantize_cols(st["dy"], st["dyt"], st["dyts"])
    qb.qb_fp8_weight_grad(st["dyt"], st["dyts"], st["xt"], st["xts"], st["dw"], off=off)
    return dict(y=st["y"], dx=st["dx"], dw=st["dw"])


def _own_exchange(st):
    from exact_quantile_selection_amd import qb

    case = st["case"]
    qb.qb_dispatch(st["topk"], case["E"], case["align"], st["off"], st["row_src"], st["pos"], st["ws"])
    qb.qb_combine(st["rows"], st["pos"], st["out"], gate=st["gate"])
    found = {k: st[k] for k in ("off", "row_src", "pos", "out")}
    if case["train"]:
        qb.qb_combine_backward(st["dout"], st["rows"], st["pos"], st["row_src"], st["drows"], gate=st["gate"],
                               dgate=st["dgate"])
        found["dgate"], found["drows"] = st["dgate"], st["drows"]
    return found


def run(state):
    op = state["case"]["op"]
    if own:
        return {"route": _own_route, "exchange": _own_exchange}.get(op, _own_product)(state)
    return {"route": _plain_route, "linear": _plain_linear, "experts": _plain_experts,
            "exchange": _plain_exchange}[op](state)


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def _pow2(e):
    """2^e for whole e, in 64 bits, exactly."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _eighth(x, dim):
    """x in 64 bits, rounded along `dim` to e4m3 values times a power of two for
    each 128 of them, from the types' definition: the least power that keeps the
    block within 448, and 3 fraction bits above the least normal exponent -6."""
    x = x.double().movedim(dim, -1)
    n = x.shape[-1]
    t = torch.cat([x, x.new_zeros(x.shape[:-1] + (-n % BLOCK,))], -1).unflatten(-1, (-1, BLOCK))
    top = t.abs().max(-1, keepdim=True).values
    low = torch.floor(torch.log2(top.clamp(min=2.0 ** -300))) - 8
    e = torch.where(top > TOP * _pow2(low), low + 1, low).clamp(min=-126)
    v = t / _pow2(e)
    step = _pow2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -60))).clamp(min=-6) - 3)
    return (torch.round(v / step) * step * _pow2(e)).flatten(-2)[..., :n].movedim(-1, dim)


def _held(q, scale, C):
    """The 64-bit values of a laid out weight stack, [.., N, C]."""
    row = torch.arange(q.shape[-2], device=q.device) // BLOCK
    col = torch.arange(C, device=q.device) // BLOCK
    return q[..., :C].float().double() * _pow2(scale[..., row, :][..., col].double() - 127)


def _exact_product(st):
    train, x = st["case"]["train"], st["x"]
    C, N = x.shape[1], st["y"].shape[1]
    xr, w = _eighth(x, 1), _held(st["w"], st["w_scale"], C)
    if "off" not in st:
        found = dict(y=xr @ w.T)
        if train:
            found["dx"] = _eighth(st["dy"], 1) @ _held(st["wt"], st["wt_scale"], N).T
            found["dw"] = _eighth(st["dy"], 0).T @ _eighth(x, 0)
        return found
    bounds = st["off"].tolist()
    found = dict(y=torch.zeros((x.shape[0], N), dtype=torch.float64, device=x.device))
    if train:
        dr, wt = _eighth(st["dy"], 1), _held(st["wt"], st["wt_scale"], N)
        xc, dc = _eighth(x, 0), _eighth(st["dy"], 0)
        found["dx"] = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
        found["dw"] = torch.zeros(w.shape, dtype=torch.float64, device=x.device)
    for e, (i, j) in enumerate(zip(bounds, bounds[1:])):
        if i < j:
            found["y"][i:j] = xr[i:j] @ w[e].T
            if train:
                found["dx"][i:j] = dr[i:j] @ wt[e].T
                found["dw"][e] = dc[i:j].T @ xc[i:j]
    return found


def _exact_route(st):
    case, s = st["case"], st["s"]
    N, E = s.shape
    K, train = case["K"], case["train"]
    left = s + st["b"]           # the order is that of the 32-bit sums
    number = torch.arange(E, device=s.device)
    picks = []
    for _ in range(K):           # the largest one left, the lower index of equal ones
        best = torch.where(left == left.max(1, keepdim=True).values, number, E).min(1, keepdim=True).values
        picks.append(best)
        left = left.scatter(1, best, -math.inf)
    order = torch.cat(picks, 1)
    s = s.double()
    mine = torch.gather(s, 1, order)
    total = mine.sum(1, keepdim=True)
    gate = torch.where(total > 0, mine / total, 0.0)
    if not train:
        return dict(topk=order.to(torch.int32), gate=gate)
    on = torch.zeros(N, dtype=torch.bool, device=s.device)
    bounds = st["seq_off"].tolist()
    on[bounds[0]:bounds[-1]] = True
    if st["valid"] is not None:
        on &= st["valid"].bool()
    on = on.unsqueeze(1)
    member = torch.zeros((N, E), dtype=torch.float64, device=s.device).scatter(1, order, 1.0) * on
    z = s.sum(1, keepdim=True)
    p = torch.where(on & (z > 0), s / z, 0.0)
    gate = torch.where(on, gate, 0.0)
    counts, loss, ds = [], 0.0, torch.zeros_like(s)
    spans = list(zip(bounds, bounds[1:]))
    filled = max(1, sum(bool(on[i:j].any()) for i, j in spans))
    for i, j in spans:
        c, T = member[i:j].sum(0), int(on[i:j].sum())
        counts.append(c)
        if T:
            f = c * E / (K * T)
            loss = loss + st["coef"] / filled * (f * p[i:j].sum(0) / T).sum()
            back = st["dloss"].double() * st["coef"] / (filled * T)
            ds[i:j] = torch.where(on[i:j] & (z[i:j] > 0), back * (f - (p[i:j] @ f).unsqueeze(1)) / z[i:j], 0.0)
    dg = st["dgate"].double()
    inner = (dg * gate).sum(1, keepdim=True)
    ds = ds + torch.zeros_like(s).scatter(1, order, torch.where(on & (total > 0), (dg - inner) / total, 0.0))
    return dict(topk=torch.where(on, order, -1).to(torch.int32), gate=gate, count=torch.stack(counts).to(torch.int32),
                loss=torch.as_tensor(loss, dtype=torch.float64, device=s.device).reshape(1), dlogits=ds * s * (1 - s))


def _exact_exchange(st):
    case = st["case"]
    ids, rows, R = st["topk"].cpu().tolist(), st["rows"], st["rows"].shape[0]
    N, K, E, a = case["N"], case["K"], case["E"], case["align"]
    lists = [[] for _ in range(E)]
    for t, mine in enumerate(ids):
        for k, e in enumerate(mine):
            if 0 <= e < E:
                lists[e].append(t * K + k)
    off, source, place = [0], [-1] * R, [-1] * (N * K)
    for mine in lists:
        for i, pair in enumerate(mine):
            source[off[-1] + i], place[pair] = pair // K, off[-1] + i
        off.append(off[-1] + -(-len(mine) // a) * a)
    whole = dict(dtype=torch.int32, device=rows.device)
    src, pos = torch.tensor(source, **whole), torch.tensor(place, **whole).view(N, K)
    gate, out = st["gate"].double(), torch.zeros((N, rows.shape[1]), dtype=torch.float64, device=rows.device)
    found = dict(off=torch.tensor(off, **whole), row_src=src, pos=pos, out=out)
    if case["train"]:
        found["dgate"] = torch.zeros((N, K), dtype=torch.float64, device=rows.device)
        found["drows"] = torch.zeros(rows.shape, dtype=torch.float64, device=rows.device)
        dout = st["dout"].double()
    for k in range(K):
        t = torch.nonzero(pos[:, k] >= 0).flatten()
        r = pos[t, k].long()
        mine = rows[r].double()
        out[t] += gate[t, k].unsqueeze(1) * mine
        if case["train"]:
            found["dgate"][t, k] = (mine * dout[t]).sum(1)
            found["drows"][r] = gate[t, k].unsqueeze(1) * dout[t]
    return found


def exact(case, seed):
    st = prepare(case, seed)
    return {"route": _exact_route, "exchange": _exact_exchange}.get(case["op"], _exact_product)(st)
