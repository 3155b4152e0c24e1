"""The measured operators of a training step around the MoE layer share: routing by scores (softmax or sigmoid, with
a balance bias and groups of experts), its backward, and AdamW over many tensors with states in 32 or 8 bits.

Each case names an operator (`op`) and its sizes. With `own` false `run` computes the operator in its plain form,
elementary torch operations in FP32 (FP64 where an order or a long sum hangs on the last bits); with `own` true it
makes the library's calls on the same state.
"""
import math

import torch

own = False

_SIZES = {
    # Routing: scores, choice of groups and experts, gates, counts and the permutation.
    # one token of a decode step, grouped sigmoid routing: launch latency decides
    "route_1": dict(op="route", T=1, E=256, El=32, k=8, n=1, score="sigmoid", G=8, tg=4, top=2, bias=True, renorm=True,
                    train=False),
    # a small batch of odd size on a width that is no power of two
    "route_333": dict(op="route", T=333, E=60, El=15, k=6, n=1, score="softmax", G=4, tg=2, top=1, bias=False,
                      renorm=False, train=False),
    # the 16K-token one-GPU share in two chunks, with the bias update of a training step
    "route_16k": dict(op="route", T=16384, E=128, El=16, k=8, n=2, score="sigmoid", G=1, tg=1, top=1, bias=True,
                      renorm=True, train=True),
    # a long-context batch with a wide grouped router: streams the logits from HBM
    "route_128k": dict(op="route", T=131072, E=256, El=32, k=8, n=2, score="sigmoid", G=8, tg=4, top=2, bias=True,
                       renorm=True, train=False),
    # Backward of the routing: logits gradient and, where `dwr`, the router weight gradient.
    # a small BF16 layer with softmax scores that are not renormalised (every logit gets a gradient)
    "route_bwd_1000": dict(op="route_bwd", T=1000, H=256, E=32, k=4, score="softmax", renorm=False, dwr=True),
    # the 16K-token one-GPU share
    "route_bwd_16k": dict(op="route_bwd", T=16384, H=2048, E=128, k=8, score="sigmoid", renorm=True, dwr=True),
    # the logits gradient alone of a long-context batch: streams it to HBM
    "route_bwd_128k": dict(op="route_bwd", T=131072, H=64, E=256, k=8, score="softmax", renorm=False, dwr=False),
    # AdamW: the three tensors of a layer (W1, W2, W_r), or ragged ones.
    # the tiny FP32 configuration's weights
    "adamw_tiny": dict(op="adamw", count=3, total=8 * 3 * 256 * 128 + 8 * 128, seed=0, w="f32", bits=32, clip=False),
    # the one-GPU share's weights (16 local experts): BF16 with FP32 masters, gradient clipping
    "adamw_layer": dict(op="adamw", count=3, total=16 * 3 * 768 * 2048 + 128 * 2048, seed=0, w="master", bits=32,
                        clip=True),
    # the same with 8-bit states
    "adamw_layer_8bit": dict(op="adamw", count=3, total=16 * 3 * 768 * 2048 + 128 * 2048, seed=0, w="master", bits=8,
                             clip=True),
    # many tensors of odd sizes, BF16 weights without masters, 8-bit states
    "adamw_many_8bit": dict(op="adamw", count=201, total=4000000, seed=3, w="bf16", bits=8, clip=True),
    # many tensors of odd sizes, FP32 weights and states
    "adamw_many": dict(op="adamw", count=97, total=1000000, seed=5, w="f32", bits=32, clip=True),
}


def listed():
    return [dict(v, name=k) for k, v in _SIZES.items()]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "route_bwd", "adamw"])
    score, renorm = rng.choice(["sigmoid", "softmax"]), rng.random() < 0.6
    if op == "route":
        G = rng.choice([1, 1, 2, 4, 8])
        E = G * 4 * rng.randint(1, 64 // G)
        tg = rng.randint(1, G)
        k = rng.randint(1, min(8, tg * (E // G)))
        return dict(op=op, T=_log(rng, 1, 100000), E=E, El=rng.randint(1, E), k=k, n=rng.randint(1, 3), score=score, G=G,
                    tg=tg, top=rng.randint(1, 2), bias=rng.random() < 0.7, renorm=renorm, train=False)
    if op == "route_bwd":
        E = 4 * rng.randint(2, 64)
        dwr = rng.random() < 0.6
        # one renormalised gate is constant: no gradient to look at
        return dict(op=op, T=_log(rng, 1, 16000 if dwr else 100000), H=64 * rng.randint(1, 32), E=E,
                    k=rng.randint(1 + renorm, 8), score=score, renorm=renorm, dwr=dwr)
    total = _log(rng, 1000, 60000000)
    return dict(op=op, count=rng.randint(1, min(250, max(1, total // 500))), total=total, seed=rng.randint(1, 1000000),
                w=rng.choice(["f32", "master", "bf16"]), bits=rng.choice([32, 8]), clip=rng.random() < 0.6)


# ---------------------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


BLOCK = 256          # elements of one scale of an 8-bit state
SCALE = 2.5          # gate multiplier
RATE = 0.001         # bias update
LR, BETA1, BETA2, EPS, STEP, SEED, MAX_NORM = 3e-4, 0.9, 0.95, 1e-8, 120, 12345, 1.0


def tensor_sizes(case):
    """Elements of each tensor: a layer's three shapes, or ragged ones that add up to `total` about."""
    total, count = case["total"], case["count"]
    if case["seed"] == 0:  # W1 : W2 = 2 : 1, and W_r
        wr = {8 * 3 * 256 * 128 + 8 * 128: 8 * 128}.get(total, 128 * 2048)
        return [(total - wr) // 3 * 2, (total - wr) // 3, wr]
    cuts = [math.exp(2.0 * math.sin(case["seed"] + 1.7 * i)) for i in range(count)]
    return [max(1, int(total * c / sum(cuts))) for c in cuts]


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    op = case["op"]
    f32, i32, dev, bf16 = torch.float32, torch.int32, "cuda", torch.bfloat16
    if op == "route":
        T, E, El, k, n = (case[x] for x in ("T", "E", "El", "k", "n"))
        # logits with an uneven popularity of the experts, as a router has them
        st["logits"] = _randn(g, T, E) + 0.5 * _randn(g, 1, E)
        st["bias_t"] = 0.1 * _randn(g, E) if case["bias"] else None
        P_c = (-(-T // n) * min(k, El) + 3) // 4 * 4
        st.update(P_c=P_c, topk_idx=torch.empty(T, k, dtype=i32, device=dev), gates=torch.empty(T, k, device=dev),
                  counts=torch.empty(n, E, dtype=i32, device=dev), offsets=torch.empty(n, El + 1, dtype=i32, device=dev),
                  row_of=torch.empty(T, k, dtype=i32, device=dev),
                  src_token=torch.empty(n * P_c, dtype=i32, device=dev))
    elif op == "route_bwd":
        T, H, E, k = (case[x] for x in ("T", "H", "E", "k"))
        st["logits"] = _randn(g, T, E) + 0.5 * _randn(g, 1, E)
        # chosen with a balance bias: not simply the largest logits
        st["idx"] = torch.topk(st["logits"] + 0.3 * _randn(g, 1, E), k, dim=1).indices.to(i32).contiguous()
        st["dgates"] = _randn(g, T, k)
        st["x"] = _randn(g, T, H).to(bf16) if case["dwr"] else None
        st.update(dlogits=torch.empty(T, E, device=dev), acc=torch.empty(E, H, device=dev),
                  dwr_t=torch.empty(E, H, dtype=bf16, device=dev))
    else:
        sizes = tensor_sizes(case)
        at, starts = 0, []
        for s in sizes:  # one flat buffer, each tensor from a multiple of a block on
            starts.append(at)
            at += -(-s // BLOCK) * BLOCK
        live = torch.zeros(at, device=dev)
        decay = torch.zeros(at, device=dev)
        for i, (s, a) in enumerate(zip(sizes, starts)):
            live[a:a + s] = 1.0
            decay[a:a + s] = 0.1 if i % 3 != 2 else 0.0  # the router (and biases) without weight decay
        st["decay"] = decay
        wdt = f32 if case["w"] == "f32" else bf16
        # weights N(0, 0.02), gradients of uneven size from tensor row to tensor row, states of a run under way
        spread = torch.exp(_randn(g, at // 64 + 1)).repeat_interleave(64)[:at]
        st["grad"] = (_randn(g, at) * spread * 1e-3 * live).to(wdt)
        full = _randn(g, at) * 0.02 * live
        st["w_t"] = full.to(wdt)
        st["master"] = full if case["w"] == "master" else None
        m = (_randn(g, at) * spread * 3e-4 * live)
        v = (_randn(g, at) * spread * 1e-3).square() * live
        if case["bits"] == 8:
            st["mc"], st["ms"] = _encode_m(m, None)
            st["vc"], st["vs"] = _encode_v(v, None)
            st["m"], st["v"] = torch.empty(at, device=dev), torch.empty(at, device=dev)
        else:
            st["m"], st["v"] = m, v
        st["norm"] = torch.empty(2, device=dev)
    if own:
        import combine_moe_route_02_amd as mh
        if op == "adamw":
            at8 = case["bits"] == 8
            es, gs = st["w_t"].element_size(), st["grad"].element_size()
            parts = []
            for i, (s, a) in enumerate(zip(sizes, starts)):
                parts.append(dict(
                    w=st["w_t"][a:a + s], grad=st["grad"][a:a + s],
                    master=None if st["master"] is None else st["master"][a:a + s],
                    m=(st["mc"] if at8 else st["m"])[a:a + s], v=(st["vc"] if at8 else st["v"])[a:a + s],
                    m_scale=st["ms"][a // BLOCK:] if at8 else None, v_scale=st["vs"][a // BLOCK:] if at8 else None,
                    weight_decay=0.1 if i % 3 != 2 else 0.0))
            st["tensors"] = mh.make_adamw_tensors(parts)
            st["options"] = mh.make_adamw_options(lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS, step=STEP,
                                                  state_bits=case["bits"], seed=SEED,
                                                  grad_scale=st["norm"][1:] if case["clip"] else None)
            st["ws"] = torch.empty(mh.moe_grad_norm_bytes(), dtype=torch.uint8, device=dev)
        else:
            T, E, k = case["T"], case["E"], case["k"]
            st["desc"] = mh.make_desc(T=T, H=case.get("H", 64), I=64, E=E, E_local=case.get("El", 1), k=k,
                                      n_chunks=case.get("n", 1), dtype="bf16")
            st["how"] = mh.make_router_scores(score=case["score"], n_groups=case.get("G", 1),
                                              topk_groups=case.get("tg", 1), group_top=case.get("top", 1),
                                              renormalize=case["renorm"], scale=SCALE)
            st["ws"] = torch.zeros(mh.workspace_bytes(st["desc"])["workspace"], dtype=torch.uint8, device=dev)
    return st


# ---------------------------------------------------------------------------------------------- plain forms

def _scores(logits, score):
    """Scores in FP64: their order decides which experts are chosen."""
    lg = logits.double()
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-lg))
    ex = torch.exp(lg - lg.amax(1, keepdim=True))
    return ex / ex.sum(1, keepdim=True)


def _best(values, k):
    """Places of the k largest per row, ties to the lower index."""
    return torch.sort(values, dim=1, descending=True, stable=True).indices[:, :k]


def _plain_route(st):
    T, E, El, k, n, G, tg, P_c = (st[x] for x in ("T", "E", "El", "k", "n", "G", "tg", "P_c"))
    i32, dev = torch.int32, "cuda"
    s = _scores(st["logits"], st["score"])
    c = s.float() if st["bias_t"] is None else (s + st["bias_t"].double()).float()
    if G > 1:
        per = c.reshape(T, G, E // G)
        top = torch.sort(per, dim=2, descending=True).values[:, :, :min(st["top"], E // G)]
        keep = torch.zeros(T, G, device=dev).scatter_(1, _best(top.sum(2), tg), 1.0)
        c = torch.where(keep.unsqueeze(2) > 0, per, torch.full_like(per, -math.inf)).reshape(T, E)
    idx = _best(c, k)
    w = s.gather(1, idx)
    gates = (w / w.sum(1, keepdim=True) if st["renorm"] else w) * SCALE
    # the permutation: local slots in order of chunk, expert, token
    tc = -(-T // n)
    chunk = (torch.arange(T, device=dev) // tc).unsqueeze(1).expand(T, k)
    ones = torch.ones(T * k, dtype=torch.int64, device=dev)
    counts = torch.zeros(n * E, dtype=torch.int64, device=dev).scatter_add_(0, (chunk * E + idx).reshape(-1), ones)
    counts = counts.reshape(n, E)
    local = counts[:, :El]
    off = torch.cat([torch.zeros(n, 1, dtype=local.dtype, device=dev), torch.cumsum(local, 1)], 1)
    key = torch.where(idx < El, chunk * El + idx, torch.full_like(idx, n * El)).reshape(-1)
    order = torch.sort(key, stable=True).indices
    place = torch.empty_like(order).scatter_(0, order, torch.arange(T * k, device=dev))
    before = torch.cumsum(off[:, El], 0) - off[:, El]  # local slots of the chunks before
    flat = chunk.reshape(-1)
    row = flat * P_c + place - before[flat]
    is_local = key < n * El
    row = torch.where(is_local, row, torch.full_like(row, -1))
    src = torch.full((n * P_c + 1,), -1, dtype=torch.int64, device=dev)
    src.scatter_(0, torch.where(is_local, row, torch.full_like(row, n * P_c)), torch.arange(T * k, device=dev) // k)
    out = dict(topk_idx=idx.to(i32), gates=gates.float(), counts=counts.to(i32), offsets=off.to(i32),
               row_of=row.reshape(T, k).to(i32), src_token=src[:n * P_c].to(i32))
    if st["train"]:
        load = counts.sum(0)
        st["bias_t"] += RATE * torch.sign(load.sum() - E * load).float()
        out["bias"] = st["bias_t"]
    return out


def _plain_route_bwd(st):
    T, E = st["T"], st["E"]
    idx, dg, lg = st["idx"].long(), st["dgates"], st["logits"]
    z = lg.gather(1, idx)
    if st["score"] == "sigmoid":
        s, rest = 1.0 / (1.0 + torch.exp(-z)), 1.0 / (1.0 + torch.exp(z))
    else:
        ex = torch.exp(lg - lg.amax(1, keepdim=True))
        p = ex / ex.sum(1, keepdim=True)
        s, rest = p.gather(1, idx), 1.0
    if st["renorm"]:
        gh = s / s.sum(1, keepdim=True)
        dz = SCALE * gh * (dg - (gh * dg).sum(1, keepdim=True)) * rest
        dl = torch.zeros(T, E, device="cuda").scatter_(1, idx, dz)
    elif st["score"] == "sigmoid":
        dl = torch.zeros(T, E, device="cuda").scatter_(1, idx, SCALE * dg * s * rest)
    else:
        chosen = torch.zeros(T, E, device="cuda").scatter_(1, idx, dg)
        dl = SCALE * p * (chosen - (s * dg).sum(1, keepdim=True))
    if not st["dwr"]:
        return dict(dlogits=dl)
    return dict(dlogits=dl, dwr=(dl.t() @ st["x"].float()).to(torch.bfloat16))


def _levels(top, power):
    """The values that codes 0..top stand for, in units of the block's scale; every product rounded once."""
    t = torch.arange(top + 1, device="cuda").float() * (1.0 / top)
    t = t * t
    return t * t if power == 4 else t


def _encode(a, top, power, u):
    """Codes of a in [0, 1]: the level below, or the one above with the chance of how near it is (u: 16 random bits)."""
    level = _levels(top, power)
    c = (torch.searchsorted(level, a, right=True) - 1).clamp(0, top - 1)
    lo, hi = level[c], level[c + 1]
    r = 0.5 if u is None else u.float() * 2.0 ** -16
    return c + (a - lo > r * (hi - lo))


def _shares(x):
    """Magnitudes in units of their block's largest, and that one (blocks under 2^-120 count as zeros)."""
    per = x.abs().reshape(-1, BLOCK)
    big = per.amax(1, keepdim=True)
    big = torch.where(big < 2.0 ** -120, torch.zeros_like(big), big)
    inv = torch.where(big > 0, torch.ones_like(big) / big, torch.zeros_like(big))
    return (per * inv).clamp(max=1.0).reshape(-1), big.reshape(-1)


def _encode_m(m, u):
    a, big = _shares(m)
    return (_encode(a, 127, 2, u) * torch.sign(m)).to(torch.int8), big


def _encode_v(v, u):
    a, big = _shares(v)
    c = torch.where(a > 0, _encode(a, 255, 4, u).clamp(min=1), torch.zeros((), dtype=torch.int64, device="cuda"))
    return c.to(torch.uint8), big


def _decode_m(code, scale):
    level = _levels(127, 2)[code.long().abs()] * torch.sign(code.float())
    return (level.reshape(-1, BLOCK) * scale.unsqueeze(1)).reshape(-1)


def _decode_v(code, scale):
    return (_levels(255, 4)[code.long()].reshape(-1, BLOCK) * scale.unsqueeze(1)).reshape(-1)


_M32 = 0xffffffff


def _random(n):
    """A 32-bit hash of each element's place, of the step and of the seed, and a second one from it."""
    key = (STEP * 0x243F6A89 + SEED) & _M32
    key ^= key >> 16
    key = (key * 0xB7E15163) & _M32
    key ^= key >> 15
    x = (torch.arange(n, device="cuda") * 0x9E3779B9 + key) & _M32
    x = ((x ^ (x >> 16)) * 0xB7E15163) & _M32
    x = x ^ (x >> 15)
    return x, (x * 0x243F6A89) & _M32


def _plain_adamw(st):
    n = st["grad"].numel()
    g = st["grad"].float()
    out = {}
    if st["clip"]:
        norm = st["grad"].double().square().sum().sqrt()
        factor = torch.where(norm > MAX_NORM, MAX_NORM / norm, torch.ones_like(norm)).float()
        out["norm"] = torch.stack([norm.float(), factor])
        g = g * factor
    if st["bits"] == 8:
        x, y = _random(n)
        m, v = _decode_m(st["mc"], st["ms"]), _decode_v(st["vc"], st["vs"])
    elif st["w"] == "bf16":
        y = _random(n)[1]
        m, v = st["m"], st["v"]
    else:
        m, v = st["m"], st["v"]
    # each product and sum on its own: states in 8 bits hang on the last bit of these
    m = m * BETA1 + g * (1.0 - BETA1)
    v = v * BETA2 + (g * g) * (1.0 - BETA2)
    old = st["master"] if st["w"] == "master" else st["w_t"].float()
    denom = torch.sqrt(v) * (1.0 / math.sqrt(1.0 - BETA2 ** STEP)) + EPS
    new = old * (1.0 - LR * st["decay"]) - (LR / (1.0 - BETA1 ** STEP)) * m / denom
    if st["w"] == "master":
        st["master"].copy_(new)
        out["master"] = st["master"]
    if st["w"] == "bf16":  # rounded up with the chance of how near the value above is
        bits = new.view(torch.int32).long() & _M32
        bits = ((bits + (y >> 16)) >> 16) << 16
        new = torch.where(bits >= 2 ** 31, bits - 2 ** 32, bits).to(torch.int32).view(torch.float32)
    st["w_t"].copy_(new)
    if st["bits"] == 8:
        st["mc"], st["ms"] = _encode_m(m, x & 0xffff)
        st["vc"], st["vs"] = _encode_v(v, x >> 16)
        m, v = _decode_m(st["mc"], st["ms"]), _decode_v(st["vc"], st["vs"])
    else:
        st["m"].copy_(m)
        st["v"].copy_(v)
    return dict(out, w=st["w_t"], m=m, v=v)


# ---------------------------------------------------------------------------------------------- the library's calls

def _own_route(st, mh):
    mh.moe_route_scores(st["desc"], -1, st["how"], st["logits"], st["bias_t"], st["topk_idx"], st["gates"], st["counts"],
                        st["offsets"], st["row_of"], st["src_token"], st["ws"])
    out = {x: st[x] for x in ("topk_idx", "gates", "counts", "offsets", "row_of", "src_token")}
    if st["train"]:
        mh.moe_router_bias_update(st["E"], st["n"], st["counts"], RATE, st["bias_t"])
        out["bias"] = st["bias_t"]
    return out


def _own_route_bwd(st, mh):
    more = (st["acc"], st["dwr_t"], st["ws"]) if st["dwr"] else (None, None, None)
    mh.moe_route_scores_bwd(st["desc"], -1, st["how"], st["logits"], st["dgates"], st["idx"], st["x"], st["dlogits"], *more)
    return dict(dlogits=st["dlogits"], dwr=st["dwr_t"]) if st["dwr"] else dict(dlogits=st["dlogits"])


def _own_adamw(st, mh):
    out = {}
    if st["clip"]:
        mh.moe_grad_norm(st["tensors"], MAX_NORM, st["norm"], st["ws"])
        out["norm"] = st["norm"]
    mh.moe_adamw_step(st["options"], st["tensors"])
    if st["bits"] == 8:
        mh.moe_adamw_unpack(st["m"].numel(), st["mc"], st["ms"], st["vc"], st["vs"], st["m"], st["v"])
    if st["w"] == "master":
        out["master"] = st["master"]
    return dict(out, w=st["w_t"], m=st["m"], v=st["v"])


def run(state):
    op = state["op"]
    if own:
        import combine_moe_route_02_amd as mh
        return {"route": _own_route, "route_bwd": _own_route_bwd, "adamw": _own_adamw}[op](state, mh)
    return {"route": _plain_route, "route_bwd": _plain_route_bwd, "adamw": _plain_adamw}[op](state)


# ---------------------------------------------------------------------------------------------- work and exact values

def work(case):
    op = case["op"]
    if op == "route":
        T, E, El, k, n = (case[x] for x in ("T", "E", "El", "k", "n"))
        P = n * ((-(-T // n) * min(k, El) + 3) // 4 * 4)
        # logits read; indices, gates, rows, the rows' tokens and the tables written
        return dict(bytes=4 * T * E + 4 * E * case["bias"] + 12 * T * k + 4 * P + 4 * n * (E + El + 1), flops=8 * T * E)
    if op == "route_bwd":
        T, H, E, k = (case[x] for x in ("T", "H", "E", "k"))
        whole = case["score"] == "softmax" and not case["renorm"]
        b = 4 * T * E + 8 * T * k + 4 * T * (E if whole else k)
        if case["dwr"]:
            return dict(bytes=b + 2 * T * H + 2 * E * H, flops=2 * T * E * H)
        return dict(bytes=b, flops=8 * T * (E if whole else k))
    n = sum(tensor_sizes(case))
    ws = {"f32": 4 + 4 + 4, "master": 2 + 4 + 4 + 2, "bf16": 2 + 2 + 2}[case["w"]]  # gradient, weight in and out
    # states in and out; 8-bit ones are also handed back as values
    return dict(bytes=n * (ws + (16 if case["bits"] == 32 else 4 + 8)), flops=16 * n)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op == "route":
        T, E, k, G = case["T"], case["E"], case["k"], case["G"]
        lg = st["logits"].to(f64)
        s = torch.sigmoid(lg) if case["score"] == "sigmoid" else torch.softmax(lg, 1)
        b = torch.zeros(E, dtype=f64, device="cuda") if st["bias_t"] is None else st["bias_t"].to(f64)
        # the choice is made on sums rounded once to FP32: part of the definition
        c = (s + b).to(torch.float32).to(f64)
        size = E // G
        if G > 1:
            blocks = c.split(size, 1)
            rank = torch.stack([x.topk(min(case["top"], size), 1).values.sum(1).to(torch.float32) for x in blocks], 1)
            # a lower group wins a tie: beaten by those that are larger, or equal and in front
            beaten = torch.zeros(T, G, dtype=torch.int64, device="cuda")
            for a in range(G):
                for o in range(G):
                    if o != a:
                        beaten[:, a] += (rank[:, o] >= rank[:, a]) if o < a else (rank[:, o] > rank[:, a])
            for a in range(G):
                c[:, a * size:(a + 1) * size][beaten[:, a] >= case["tg"]] = -math.inf
        rows = torch.arange(T, device="cuda")
        picks = []
        for _ in range(k):
            at = (c == c.max(1, keepdim=True).values).to(torch.int8).argmax(1)  # the first of the largest
            picks.append(s[rows, at])
            c[rows, at] = -math.inf
        w = torch.stack(picks, 1)
        gates = SCALE * (w / w.sum(1, keepdim=True) if case["renorm"] else w)
        out = dict(topk_idx=None, gates=gates, counts=None, offsets=None, row_of=None, src_token=None)
        if case["train"]:
            out["bias"] = None
        return out
    if op == "route_bwd":
        lg = st["logits"].to(f64).requires_grad_(True)
        s = torch.sigmoid(lg) if case["score"] == "sigmoid" else torch.softmax(lg, 1)
        w = torch.gather(s, 1, st["idx"].long())
        gates = SCALE * (w / w.sum(1, keepdim=True) if case["renorm"] else w)
        (dl,) = torch.autograd.grad((gates * st["dgates"].to(f64)).sum(), lg)
        if not case["dwr"]:
            return dict(dlogits=dl)
        return dict(dlogits=dl, dwr=torch.matmul(dl.t().contiguous(), st["x"].to(f64)))
    bits, out = case["bits"], {}
    g = st["grad"].to(f64)
    if case["clip"]:
        norm = torch.linalg.vector_norm(g)
        factor = float(min(1.0, MAX_NORM / max(float(norm), 1e-300)))
        out["norm"] = torch.tensor([float(norm), factor], dtype=f64)
        g = g * factor
    if bits == 8:
        step = torch.repeat_interleave(st["ms"].to(f64), BLOCK)
        q = st["mc"].to(f64) / 127.0
        m = step * q * q.abs()
        v = torch.repeat_interleave(st["vs"].to(f64), BLOCK) * (st["vc"].to(f64) / 255.0) ** 4
    else:
        m, v = st["m"].to(f64), st["v"].to(f64)
    m = BETA1 * m + (1.0 - BETA1) * g
    v = BETA2 * v + (1.0 - BETA2) * g ** 2
    w = (st["w_t"] if st["master"] is None else st["master"]).to(f64)
    m_hat, v_hat = m / (1.0 - BETA1 ** STEP), v / (1.0 - BETA2 ** STEP)
    w = w - LR * st["decay"].to(f64) * w - LR * m_hat / (torch.sqrt(v_hat) + EPS)
    if case["w"] == "master":
        out["master"] = w
    # weights and states that are rounded by chance have no value of their own in 64 bits
    by_chance = bits == 8
    return dict(out, w=None if case["w"] == "bf16" else w, m=None if by_chance else m, v=None if by_chance else v)
