"""The measured operators of the MoE layer share: the router's loss with its gradient, the dense router
gradient of dispatch backward, and the 8-bit integer expert products for serving.

Each case names an operator (`op`) and its sizes. With `own` false `run` computes the operator in its plain form,
elementary torch operations in FP32; with `own` true it makes the library's calls on the same state.
"""
import math

import torch

own = False

_SIZES = {
    # Router loss (balance + z) and its gradient, one training step's call.
    # a short batch of one sequence: launch latency decides
    "loss_512": dict(op="loss", T=512, E=128, k=8, S=1, masked=False),
    # the 16K-token one-GPU share, 16 packed sequences of ragged length with padding tokens masked out
    "loss_16k_packed": dict(op="loss", T=16384, E=128, k=8, S=16, masked=True),
    # a long-context batch with a wide router: streams the logits from HBM
    "loss_128k": dict(op="loss", T=131072, E=256, k=8, S=1, masked=False),
    # Dispatch backward with the router loss's dense logits gradient.
    # the tiny FP32 configuration
    "dx_f32_256": dict(op="dx", T=256, H=128, E=8, El=8, k=2, dtype="f32"),
    # a small ragged BF16 layer
    "dx_bf16_1000": dict(op="dx", T=1000, H=256, E=32, El=8, k=4, dtype="bf16"),
    # the 16K-token one-GPU share (16 of 128 experts local)
    "dx_bf16_16k": dict(op="dx", T=16384, H=2048, E=128, El=16, k=8, dtype="bf16"),
    # 8-bit integer product with a scale per token and channel, activations quantised on the way.
    # one token of a decode step through a square projection
    "linear_1": dict(op="linear", rows=1, N=2048, K=2048),
    # a decode batch of odd size into a wide hidden state
    "linear_77": dict(op="linear", rows=77, N=7168, K=2048),
    # a prefill batch: matrix-core bound
    "linear_8k": dict(op="linear", rows=8192, N=4096, K=7168),
    # 8-bit integer experts: dispatch, SwiGLU experts, combine.
    # one token of a decode step, every expert on this GPU
    "experts_1": dict(op="experts", T=1, H=2048, I=768, E=128, El=128, k=8),
    # a decode batch of odd size that touches most experts
    "experts_33": dict(op="experts", T=33, H=2048, I=768, E=128, El=128, k=8),
    # the 16K-token one-GPU share
    "experts_16k": dict(op="experts", T=16384, H=2048, I=768, E=128, El=16, k=8),
}


def listed():
    return [dict(v, name=k) for k, v in _SIZES.items()]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["loss", "dx", "linear", "experts"])
    if op == "loss":
        T, E = _log(rng, 1, 100000), 4 * rng.randint(2, 64)
        return dict(op=op, T=T, E=E, k=rng.randint(1, min(8, E)), S=_log(rng, 1, 64), masked=rng.random() < 0.5)
    if op == "dx":
        E = 4 * rng.randint(2, 40)
        return dict(op=op, T=_log(rng, 1, 16000), H=64 * rng.randint(1, 32), E=E, El=rng.randint(1, E),
                    k=rng.randint(1, 8), dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]))
    if op == "linear":
        return dict(op=op, rows=_log(rng, 1, 8000), N=8 * rng.randint(8, 512), K=64 * rng.randint(2, 112))
    E = 8 * rng.randint(2, 16)
    El = rng.choice([E, max(1, E // 8)])
    return dict(op=op, T=_log(rng, 1, 2000 if El == E else 16000), H=64 * rng.randint(2, 32), I=64 * rng.randint(1, 16),
                E=E, El=El, k=rng.randint(1, 8))


# ---------------------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _routing(g, T, E, El, k):
    """Top-k routing of N(0,1) logits and the stable permutation of the local slots (experts 0..El-1): what the
    routing call hands on. `slot` is each (token, j)'s place in a [El, cap] table of the experts' rows."""
    logits = _randn(g, T, E)
    val, idx = torch.topk(logits, k, dim=1)
    gates = torch.softmax(val, dim=1)
    flat = idx.reshape(-1)
    local = flat < El
    key = torch.where(local, flat, torch.full_like(flat, El))
    order = torch.argsort(key, stable=True)
    counts = torch.bincount(key, minlength=El + 1)[:El]
    offsets = torch.zeros(El + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0)
    n = int(offsets[-1])
    row = torch.full_like(flat, -1)
    row[order[:n]] = torch.arange(n, device="cuda")
    cap = max(1, int(counts.max()))
    rank = row - offsets[key.clamp(max=El - 1)]
    slot = torch.where(local, key * cap + rank, torch.full_like(flat, -1)).reshape(T, k)
    P = (T * min(k, El) + 3) // 4 * 4
    src = torch.full((P,), -1, dtype=torch.int64, device="cuda")
    src[:n] = order[:n] // k
    i32 = torch.int32
    return dict(idx=idx.to(i32).contiguous(), gates=gates.contiguous(), offsets=offsets.to(i32), counts=counts, P=P, n=n,
                row_of=row.reshape(T, k).to(i32).contiguous(), src=src.to(i32), cap=cap, slot=slot)


def _i8_weights(g, groups, rows, cols):
    """Weights N(0, 0.02) as a program keeps them: int8 codes and one FP32 scale per output channel."""
    w = (_randn(g, groups, rows, cols) * 0.02).to(torch.bfloat16).float()
    amax = w.abs().amax(-1, keepdim=True)
    return torch.round(w * (127.0 / amax)).to(torch.int8), (amax / 127.0).squeeze(-1).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    op = case["op"]
    f32, i32, dev = torch.float32, torch.int32, "cuda"
    if op == "loss":
        T, E, k, S = case["T"], case["E"], case["k"], case["S"]
        # logits with an uneven popularity of the experts, as a router has them
        st["logits"] = _randn(g, T, E) + 0.5 * _randn(g, 1, E)
        st["idx"] = torch.topk(st["logits"], k, dim=1).indices.to(i32).contiguous()
        cuts = torch.randint(0, T + 1, (S - 1,), generator=g, device=dev).sort().values
        ends = torch.tensor([0, T], device=dev)
        st["seg"] = torch.cat([ends[:1], cuts, ends[1:]]).to(i32)
        st["mask"] = None
        if case["masked"]:
            st["mask"] = (torch.rand(T, generator=g, device=dev) < 0.9).to(torch.uint8)
            st["logits"][st["mask"] == 0] = float("nan")  # padding rows hold no values
        st.update(lse=torch.empty(T, device=dev), counts=torch.empty(S, E, dtype=i32, device=dev),
                  tokens=torch.empty(S + 2, dtype=i32, device=dev), probs=torch.empty(S, E, device=dev),
                  loss=torch.empty(3, device=dev), dloss=torch.rand(1, generator=g, device=dev) + 0.5,
                  dlogits=torch.empty(T, E, device=dev))
        if own:
            import combine_moe_route_02_amd as mh
            st["desc"] = mh.make_desc(T=T, H=64, I=64, E=E, E_local=1, k=k, n_chunks=1, dtype="bf16")
            st["ws"] = torch.zeros(mh.moe_router_loss_bytes(st["desc"], S), dtype=torch.uint8, device=dev)
    elif op == "dx":
        T, H, E, El, k = (case[n] for n in ("T", "H", "E", "El", "k"))
        dt = f32 if case["dtype"] == "f32" else torch.bfloat16
        st.update(_routing(g, T, E, El, k))
        st["dxd"] = _randn(g, st["P"], H).to(dt)
        st["w_r"] = (_randn(g, E, H) * 0.02).to(dt)
        st["dlogits"] = _randn(g, T, E) * 0.1
        st["dx"] = torch.empty(T, H, dtype=dt, device=dev)
        if own:
            import combine_moe_route_02_amd as mh
            st["desc"] = mh.make_desc(T=T, H=H, I=64, E=E, E_local=El, k=k, n_chunks=1, dtype=case["dtype"],
                                      flags=mh.FLAG_ROUTER_LOSS)
    elif op == "linear":
        R, N, K = case["rows"], case["N"], case["K"]
        st["x"] = _randn(g, R, K).to(torch.bfloat16)
        w, ws = _i8_weights(g, 1, N, K)
        st.update(w=w[0], ws=ws[0], xq=torch.empty(R, K, dtype=torch.int8, device=dev),
                  xs=torch.empty(R, device=dev), y=torch.empty(R, N, dtype=torch.bfloat16, device=dev))
    else:
        T, H, I, E, El, k = (case[n] for n in ("T", "H", "I", "E", "El", "k"))
        st.update(_routing(g, T, E, El, k))
        st["x"] = _randn(g, T, H).to(torch.bfloat16)
        st["w1"], st["w1s"] = _i8_weights(g, El, 2 * I, H)
        st["w2"], st["w2s"] = _i8_weights(g, El, H, I)
        P = st["P"]
        # the plain form's plan: experts with rows, and the token of each of their rows (padded)
        st["active"] = torch.nonzero(st["counts"]).reshape(-1)
        tok = torch.zeros(El * st["cap"], dtype=torch.int64, device=dev)
        t_of = torch.arange(T, device=dev).unsqueeze(1).expand(T, k)
        tok[st["slot"][st["slot"] >= 0]] = t_of[st["slot"] >= 0]
        st["tok"] = tok.reshape(El, st["cap"])[st["active"]]
        st["place"] = torch.zeros(El, dtype=torch.int64, device=dev)
        st["place"][st["active"]] = torch.arange(len(st["active"]), device=dev)
        st.update(xd=torch.empty(P, H, dtype=torch.int8, device=dev), xds=torch.empty(P, device=dev),
                  hs=torch.empty(P, device=dev), h=torch.empty(5 * P * I, dtype=torch.uint8, device=dev),
                  yd=torch.empty(P, H, dtype=torch.bfloat16, device=dev),
                  out=torch.empty((T * k + 3) // 4 * 4, H, dtype=torch.bfloat16, device=dev))
        if own:
            import combine_moe_route_02_amd as mh
            st["desc"] = mh.make_desc(T=T, H=H, I=I, E=E, E_local=El, k=k, n_chunks=1, dtype="int8")
    return st


# ---------------------------------------------------------------------------------------------- plain forms

BALANCE, Z = 0.01, 0.001  # loss coefficients
_BLOCK = 512


def _plain_loss(st):
    T, E, k, S = st["T"], st["E"], st["k"], st["S"]
    f64, zero = torch.float64, torch.zeros((), device="cuda")
    seg = torch.searchsorted(st["seg"][1:-1].contiguous(), torch.arange(T, device="cuda", dtype=torch.int32), right=True)
    keep = torch.ones(T, dtype=torch.bool, device="cuda") if st["mask"] is None else st["mask"] != 0
    member = ((torch.arange(S, device="cuda").unsqueeze(1) == seg) & keep).to(f64)  # [S, T]
    lg = torch.where(keep.unsqueeze(1), st["logits"], zero)
    m = lg.amax(1, keepdim=True)
    ex = torch.exp(lg - m)
    den = ex.sum(1, keepdim=True)
    p = ex / den
    lse = torch.where(keep, (m + torch.log(den)).squeeze(1), zero)
    # sums over the tokens of a segment, long ones: in 64 bits, blocks of tokens first
    B = -(-T // _BLOCK)
    parts = torch.nn.functional.pad(member, (0, B * _BLOCK - T)).reshape(S, B, _BLOCK).transpose(0, 1).contiguous()

    def over_tokens(v):
        v = torch.nn.functional.pad(v.to(f64), (0, 0, 0, B * _BLOCK - T)).reshape(B, _BLOCK, E)
        return torch.bmm(parts, v).sum(0)

    probs = over_tokens(p)
    counts = over_tokens(torch.zeros(T, E, device="cuda").scatter_(1, st["idx"].long(), 1.0))
    tokens = member.sum(1, keepdim=True)
    full, n, nd = (tokens > 0).sum(), tokens.sum(), tokens.clamp(min=1)
    bal = E * (counts / (nd * k) * (probs / nd)).sum() / full.clamp(min=1)
    z = (lse.to(f64) ** 2).sum() / n.clamp(min=1)
    # centred: the difference below keeps its digits when the load is nearly even
    w = (BALANCE / (full.clamp(min=1) * nd) * (counts * (E / k) / nd - 1.0)).float()[seg]
    dl = p * (w - (w * p).sum(1, keepdim=True)) + p * (2.0 * Z / n.clamp(min=1) * lse.to(f64)).float().unsqueeze(1)
    dl = torch.where(keep.unsqueeze(1), dl * st["dloss"], zero)
    return dict(loss=torch.stack([BALANCE * bal + Z * z, bal, z]).float(), lse=lse, counts=counts.int(),
                tokens=torch.cat([tokens.reshape(-1), n.reshape(1), full.reshape(1)]).int(), probs=probs.float(),
                dlogits=dl)


def _plain_dx(st):
    row = st["row_of"].long()
    part = st["dxd"][row.clamp(min=0)].float()
    part = (part * (row >= 0).unsqueeze(2)).sum(1)
    return (part + st["dlogits"] @ st["w_r"].float()).to(st["dxd"].dtype)


def _quantize(x):
    """Codes (as FP32) and scale of each row: 127 steps to the row's largest magnitude."""
    amax = x.abs().amax(-1, keepdim=True)
    full = amax > 0
    # tensor by tensor: a division by a scalar, or of one, would go through a rounded reciprocal
    top = torch.full_like(amax, 127.0)
    inv = torch.where(full, top / amax, torch.zeros_like(amax))
    return torch.round(x * inv).clamp(-127.0, 127.0), torch.where(full, amax / top, torch.ones_like(amax))


def _plain_linear(st):
    xq, xs = _quantize(st["x"].float())
    return ((xq @ st["w"].float().t()) * xs * st["ws"]).to(torch.bfloat16)


def _plain_experts(st):
    I, H, act = st["I"], st["H"], st["active"]
    T, k, cap = st["T"], st["k"], st["cap"]
    if len(act) == 0:
        return torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    xq, xs = _quantize(st["x"].float())
    a, s = xq[st["tok"]], xs[st["tok"]]
    gu = torch.bmm(a, st["w1"][act].float().transpose(1, 2)) * s * st["w1s"][act].unsqueeze(1)
    h = gu[..., :I] * torch.sigmoid(gu[..., :I]) * gu[..., I:]
    hq, hs = _quantize(h)
    y = torch.bmm(hq, st["w2"][act].float().transpose(1, 2)) * hs * st["w2s"][act].unsqueeze(1)
    slot = st["slot"].clamp(min=0)
    y = y.reshape(-1, H)[st["place"][slot // cap] * cap + slot % cap]
    gate = torch.where(st["slot"] >= 0, st["gates"], torch.zeros((), device="cuda"))
    return (y * gate.unsqueeze(2)).sum(1).to(torch.bfloat16)


# ---------------------------------------------------------------------------------------------- the library's calls

def _own_loss(st, mh):
    d, S = st["desc"], st["S"]
    mh.moe_router_loss(d, S, BALANCE, Z, st["logits"], st["idx"], st["seg"], st["mask"], st["lse"], st["counts"],
                       st["tokens"], st["probs"], st["loss"], st["ws"])
    mh.moe_router_loss_bwd(d, S, BALANCE, Z, st["logits"], st["lse"], st["seg"], st["mask"], st["counts"],
                           st["tokens"], st["dloss"], st["dlogits"])
    return {n: st[n] for n in ("loss", "lse", "counts", "tokens", "probs", "dlogits")}


def _own_dx(st, mh):
    mh.moe_dispatch_bwd(st["desc"], -1, st["dxd"], st["row_of"], st["idx"], st["dlogits"], st["w_r"], st["dx"])
    return st["dx"]


def _own_linear(st, mh):
    R, N, K = st["rows"], st["N"], st["K"]
    mh.moe_quantize_rows_i8(R, K, st["x"], st["xq"], st["xs"])
    mh.moe_expert_matmul_i8(1, R, N, K, st["xq"], st["xs"], st["w"], st["ws"], None, st["y"])
    return st["y"]


def _own_experts(st, mh):
    d = st["desc"]
    mh.moe_dispatch(d, -1, st["x"], st["row_of"], st["xd"], st["xds"], st["hs"])
    mh.moe_expert_ffn(d, -1, st["xd"], st["xds"], st["w1"], st["w1s"], st["w2"], st["w2s"], st["offsets"], None,
                      st["h"], st["hs"], st["yd"])
    mh.moe_combine(d, -1, st["yd"], st["gates"], st["row_of"], st["out"])
    return st["out"][:st["T"]]


def run(state):
    op = state["op"]
    if own:
        import combine_moe_route_02_amd as mh
        return {"loss": _own_loss, "dx": _own_dx, "linear": _own_linear, "experts": _own_experts}[op](state, mh)
    return {"loss": _plain_loss, "dx": _plain_dx, "linear": _plain_linear, "experts": _plain_experts}[op](state)


# ---------------------------------------------------------------------------------------------- work and exact values

def work(case):
    op = case["op"]
    if op == "loss":
        T, E, k, S = case["T"], case["E"], case["k"], case["S"]
        # logits read once, their gradient written once; indices, lse, mask, per-segment tables
        return dict(bytes=8 * T * E + 4 * T * k + 4 * T + T * case["masked"] + 12 * S * E, flops=14 * T * E)
    if op == "dx":
        T, H, E, El, k = (case[n] for n in ("T", "H", "E", "El", "k"))
        s = 4 if case["dtype"] == "f32" else 2
        n = T * k * El / E
        return dict(bytes=(n + T + E) * H * s + 4 * T * E + 4 * T * k, flops=2 * T * E * H + n * H)
    if op == "linear":
        R, N, K = case["rows"], case["N"], case["K"]
        return dict(bytes=2 * R * K + N * K + 4 * N + 2 * R * N, flops=2 * R * N * K)
    T, H, I, E, El, k = (case[n] for n in ("T", "H", "I", "E", "El", "k"))
    active = El * (1.0 - (1.0 - k / E) ** T)  # experts that get a row
    n = T * k * El / E
    return dict(bytes=active * (3 * H * I + 4 * (2 * I + H)) + 4 * T * H + 8 * T * k, flops=6 * n * H * I)


def _exact_quantize(x, given=True):
    # The codes of given values are fixed by two FP32 roundings, of 127 / amax and of its product with the value: with
    # BF16 values exact halves between two codes are common, and which way one falls is part of the definition.
    # Computed values (h) have no such halves and stay in 64 bits.
    big = x.abs().max(dim=-1, keepdim=True).values
    safe = torch.where(big == 0, torch.full_like(big, 127.0), big)
    kind = torch.float32 if given else torch.float64
    step = torch.div(torch.full_like(safe, 127.0).to(kind), safe.to(kind))
    return torch.clamp((x.to(kind) * step).round(), -127, 127).double(), safe / 127.0


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op == "loss":
        T, E, k, S = case["T"], case["E"], case["k"], case["S"]
        lg, idx, cuts = st["logits"].to(f64), st["idx"].long(), st["seg"].tolist()
        keep = [True] * T if st["mask"] is None else [bool(v) for v in st["mask"].tolist()]
        rows = [torch.tensor([t for t in range(cuts[s], cuts[s + 1]) if keep[t]], dtype=torch.int64, device="cuda")
                for s in range(S)]
        full, n = sum(len(r) > 0 for r in rows), sum(len(r) for r in rows)
        lse, dl = torch.zeros(T, dtype=f64, device="cuda"), torch.zeros(T, E, dtype=f64, device="cuda")
        probs, bal, g = torch.zeros(S, E, dtype=f64, device="cuda"), 0.0, float(st["dloss"].double())
        counts = torch.zeros(S, E, dtype=torch.int32, device="cuda")
        for s, r in enumerate(rows):
            if len(r) == 0:
                continue
            lse[r] = torch.logsumexp(lg[r], 1)
            p = torch.exp(lg[r] - lse[r].unsqueeze(1))
            c = torch.bincount(idx[r].reshape(-1), minlength=E)
            counts[s] = c.int()
            share = c.to(f64) / (len(r) * k)
            probs[s] = p.sum(0)
            bal += E * float((share * probs[s]).sum()) / len(r) / full
            dp = BALANCE * E * share / len(r) / full
            dl[r] = g * p * (dp - (p @ dp).unsqueeze(1) + 2.0 * Z / n * lse[r].unsqueeze(1))
        z = float((lse ** 2).sum()) / max(n, 1)
        loss = torch.tensor([BALANCE * bal + Z * z, bal, z], dtype=f64)
        tokens = torch.tensor([len(r) for r in rows] + [n, full], dtype=torch.int32)
        return dict(loss=loss, lse=lse, counts=counts, tokens=tokens, probs=probs, dlogits=dl)
    if op == "dx":
        out = st["dlogits"].to(f64) @ st["w_r"].to(f64)
        for j in range(case["k"]):
            r = st["row_of"][:, j].long()
            at = torch.nonzero(r >= 0).reshape(-1)
            out[at] += st["dxd"][r[at]].to(f64)
        return out
    if op == "linear":
        xq, xs = _exact_quantize(st["x"].to(f64))
        return torch.matmul(xq, st["w"].to(f64).t().contiguous()) * xs * st["ws"].to(f64)
    I, off, n = case["I"], st["offsets"].tolist(), st["n"]
    xq, xs = _exact_quantize(st["x"].to(f64))
    src = st["src"][:n].long()
    yd = torch.zeros(max(n, 1), case["H"], dtype=f64, device="cuda")
    for e in range(case["El"]):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        gu = torch.matmul(xq[src[a:b]], st["w1"][e].to(f64).t().contiguous()) * xs[src[a:b]] * st["w1s"][e].to(f64)
        h = gu[:, :I] / (1.0 + torch.exp(-gu[:, :I])) * gu[:, I:]
        hq, hs = _exact_quantize(h, given=False)
        yd[a:b] = torch.matmul(hq, st["w2"][e].to(f64).t().contiguous()) * hs * st["w2s"][e].to(f64)
    out = torch.zeros(case["T"], case["H"], dtype=f64, device="cuda")
    for j in range(case["k"]):
        r = st["row_of"][:, j].long()
        at = torch.nonzero(r >= 0).reshape(-1)
        out[at] += yd[r[at]] * st["gates"][at, j].to(f64).unsqueeze(1)
    return out
