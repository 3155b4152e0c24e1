"""GPU parity of routing by scores, its backward, the bias update and the layers that route by scores, against FP64.

Integers are equal: the choice is defined by sums rounded once to FP32. Gates: the exponent's argument is a difference
rounded once (2^-24 of it), the exponential, the sums of at most 8 (and, softmax without renormalising, the FP64 sum's one
rounding) and the division take 2^-24 or 2^-23 each, 24 of 2^-24 in all: GATE(arg) = (|arg| + 24) 2^-24 relative.
The gradient's factors carry the same error, its sum over slots or experts another 16 of 2^-24: TERM = GATE + 32 2^-24
of the terms. Arguments: |l| up to 32 here (differences up to 64) unless a test says otherwise."""
import numpy as np
import pytest

import oracle
from moe_inputs import MoeConfig
from oracle import router_loss as orl
from oracle import router_scores as ors

pytestmark = pytest.mark.gpu
harness = pytest.importorskip("harness")
F = 2.0 ** -24
GATE = (64 + 24) * F
TERM = GATE + 32 * F


def _gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import combine_moe_route_02_amd as mh
    mh.lib()
    return torch, mh


def _buffers(torch, mh, d):
    i32 = torch.int32
    P = d.n_chunks * d.P_c
    full = lambda shape, dt: torch.full(shape, -7, dtype=dt, device="cuda")  # noqa: E731
    return {"topk_idx": full((d.T, d.k), i32), "gates": full((d.T, d.k), torch.float32), "counts": full((d.n_chunks, d.E), i32),
            "offsets": full((d.n_chunks, d.E_local + 1), i32), "row_of": full((d.T, d.k), i32), "src_token": full((P,), i32),
            "workspace": torch.zeros(max(1, mh.workspace_bytes(d)["workspace"]), dtype=torch.uint8, device="cuda")}


NAMES = ("topk_idx", "gates", "counts", "offsets", "row_of", "src_token", "workspace")


def _forward(torch, mh, lg, bias, k, how, n=1, El=None, e0=0, dtype="f32", chunk=-1, b=None, stream=None):
    T, E = lg.shape
    d = mh.make_desc(T=T, H=64, I=64, E=E, E_local=E if El is None else El, e0=e0, k=k, n_chunks=n, dtype=dtype)
    b = _buffers(torch, mh, d) if b is None else b
    mh.moe_route_scores(d, chunk, mh.make_router_scores(**how), torch.from_numpy(lg).cuda(),
                        None if bias is None else torch.from_numpy(bias).cuda(), *[b[x] for x in NAMES], stream)
    torch.cuda.synchronize()
    return d, b


def _check(d, b, lg, bias, how, tol=GATE):
    want = ors.choose(ors.scores(lg, how["score"]), bias, d.k, how.get("n_groups", 1), how.get("topk_groups", 1), how.get("group_top", 1))
    got = {x: b[x].cpu().numpy() for x in NAMES[:-1]}
    np.testing.assert_array_equal(got["topk_idx"], want)
    for name, x in zip(("counts", "offsets", "row_of", "src_token"), oracle.layout(want, d.E, d.e0, d.E_local, d.n_chunks, d.P_c)):
        np.testing.assert_array_equal(got[name], x, err_msg=name)
    g = ors.gates(lg, want, how["score"], how.get("renormalize", True), how.get("scale", 1.0))
    bad = np.abs(got["gates"] - g) > tol * np.abs(g) + 2.0 ** -126  # (results below the normal range)
    assert not bad.any(), (np.argwhere(bad)[:3], got["gates"][bad][:3], g[bad][:3])


def _draw(T, E, seed, std=1.0, bias=0.2):
    rng = np.random.default_rng(seed)
    lg = np.clip(rng.standard_normal((T, E)) * std, -32, 32).astype(np.float32)
    return lg, (rng.standard_normal(E) * bias).astype(np.float32) if bias else None


# tokens around the 16-token tile and the 64-token block, E at every vector count, widths that are no multiple of 4 or 16
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,G,tg,top", [
    (1, 256, 8, 8, 4, 2), (1, 4, 1, 1, 1, 1), (15, 7, 7, 1, 1, 1), (17, 60, 6, 4, 2, 1), (64, 128, 8, 1, 1, 1), (65, 130, 3, 10, 3, 2),
    (130, 64, 8, 64, 8, 1), (40, 64, 8, 64, 33, 2), (33, 512, 8, 16, 2, 2), (50, 1024, 5, 32, 7, 2), (20, 1000, 8, 1, 1, 1), (300, 16, 2, 2, 1, 2),
    (70, 8, 4, 2, 1, 2), (21, 1, 1, 1, 1, 1), (35, 72, 8, 3, 1, 2), (90, 192, 8, 24, 9, 2), (48, 264, 8, 33, 20, 1)])
def test_choice_gates_and_rows(score, T, E, k, G, tg, top):
    torch, mh = _gpu()
    print(f"[route_scores] {score, T, E, k, G, tg, top}", flush=True)
    for renorm, with_bias in ((True, True), (False, True), (True, False)):
        lg, bias = _draw(T, E, T + E + k, std=3.0)
        how = dict(score=score, n_groups=G, topk_groups=tg, group_top=top, renormalize=renorm, scale=2.5)
        d, b = _forward(torch, mh, lg, bias if with_bias else None, k, how)
        _check(d, b, lg, bias if with_bias else None, how)


@pytest.mark.parametrize("T,E,El,e0,k,n,dtype", [(1000, 32, 8, 4, 4, 2, "bf16"), (777, 128, 16, 112, 8, 3, "fp8"), (5, 8, 4, 0, 2, 4, "f32"),
                                                 (333, 60, 0, 0, 6, 2, "int8"), (9000, 64, 64, 0, 8, 1, "bf16"), (20000, 256, 32, 32, 8, 2, "bf16")])
def test_chunks_and_local_experts(T, E, El, e0, k, n, dtype):
    torch, mh = _gpu()
    print(f"[route_scores] {T, E, El, e0, k, n, dtype}", flush=True)
    lg, bias = _draw(T, E, T)
    how = dict(score="sigmoid", n_groups=4, topk_groups=2, group_top=2)
    d, b = _forward(torch, mh, lg, bias, k, how, n, El, e0, dtype)
    _check(d, b, lg, bias, how)
    _, c = d, _buffers(torch, mh, d)
    for chunk in reversed(range(n)):  # chunk by chunk, in any order: the same
        _forward(torch, mh, lg, bias, k, how, n, El, e0, dtype, chunk, c)
    for x in NAMES[:-1]:
        assert torch.equal(b[x], c[x]), x


def test_many_chunks_without_local_experts():
    torch, mh = _gpu()
    lg, bias = _draw(131, 8, 1)
    how = dict(score="softmax", n_groups=2)
    d, b = _forward(torch, mh, lg, bias, 2, how, n=70000, El=0)  # more than the chunks of one launch
    _check(d, b, lg, bias, how)


def test_more_chunks_than_one_scan_takes():
    """Chunks past 65535 whose histograms are scanned first: moe_route with short ones, score routing with two workgroups each."""
    torch, mh = _gpu()
    T, E, k, n = 131, 128, 4, 70000
    lg, _ = _draw(T, E, 2)
    d = mh.make_desc(T=T, H=64, I=64, E=E, E_local=0, k=k, n_chunks=n, dtype="f32")
    b = _buffers(torch, mh, d)
    mh.moe_route(d, -1, torch.from_numpy(lg).cuda(), *[b[x] for x in NAMES])
    idx = oracle.route(lg, k)[0]
    np.testing.assert_array_equal(b["topk_idx"].cpu().numpy(), idx)
    want = np.zeros((n, E), np.int32)
    np.add.at(want, (np.arange(T)[:, None], idx), 1)
    np.testing.assert_array_equal(b["counts"].cpu().numpy(), want)
    assert not b["offsets"].any() and (b["row_of"] == -1).all()
    E, tc = 260, 17
    T = tc * n
    d = mh.make_desc(T=T, H=64, I=64, E=E, E_local=0, k=2, n_chunks=n, dtype="f32")
    b = _buffers(torch, mh, d)
    x = torch.zeros(T, E, device="cuda")
    first = torch.arange(n, device="cuda").repeat_interleave(tc) % E  # one expert per chunk in front, and the lowest other
    x.scatter_(1, first[:, None], 1.0)
    mh.moe_route_scores(d, -1, mh.make_router_scores(score="sigmoid"), x, None, *[b[i] for i in NAMES])
    assert torch.equal(b["topk_idx"], torch.stack([first, (first == 0).long()], 1).int())
    counts = torch.zeros(n, E, dtype=torch.int32, device="cuda")
    c = torch.arange(n, device="cuda")
    counts[c, c % E] = tc
    counts[c, (c % E == 0).long()] = tc
    assert torch.equal(b["counts"], counts) and not b["offsets"].any()


@pytest.mark.parametrize("E", [64, 256, 512])
def test_rows_off_their_alignment(E):
    torch, mh = _gpu()
    T, k = 70, 8
    lg, bias = _draw(T, E, E)
    how = dict(score="sigmoid", n_groups=8, topk_groups=4, group_top=2)
    d, want = _forward(torch, mh, lg, bias, k, how)
    off = lambda a: torch.from_numpy(np.append(np.float32(0), a.ravel())).cuda()[1:].view(a.shape)  # noqa: E731
    dg = np.ones((T, k), np.float32) + lg[:, :k]
    for shift_logits, shift_bias in ((True, False), (False, True), (True, True)):
        b = _buffers(torch, mh, d)
        x, bi = off(lg) if shift_logits else torch.from_numpy(lg).cuda(), off(bias) if shift_bias else torch.from_numpy(bias).cuda()
        assert x.data_ptr() % 16 == 4 * shift_logits and bi.data_ptr() % 16 == 4 * shift_bias
        mh.moe_route_scores(d, -1, mh.make_router_scores(**how), x, bi, *[b[n] for n in NAMES])
        torch.cuda.synchronize()
        _check(d, b, lg, bias, how)
    dl, off_dl = torch.zeros(T, E, device="cuda"), off(np.zeros((T, E), np.float32))
    r, g = mh.make_router_scores(**how), torch.from_numpy(dg).cuda()
    mh.moe_route_scores_bwd(d, -1, r, torch.from_numpy(lg).cuda(), g, want["topk_idx"], None, dl)
    mh.moe_route_scores_bwd(d, -1, r, off(lg), g, want["topk_idx"], None, off_dl)
    assert torch.equal(dl, off_dl) and float(dl.abs().max()) > 0


def test_offsets_past_32_bits():
    torch, mh = _gpu()
    T, E, k, n = 2 ** 21 + 77, 1024, 2, 64  # 2^31 + 78848 logits
    rng = np.random.default_rng(5)
    rows = [0, 1, 2 ** 20, 2 ** 21 - 1, 2 ** 21, 2 ** 21 + 1, T - 1]
    lg = rng.standard_normal((len(rows), E)).astype(np.float32)
    x = torch.zeros(T, E, device="cuda")
    x[rows] = torch.from_numpy(lg).cuda()
    d = mh.make_desc(T=T, H=64, I=64, E=E, E_local=1, e0=1, k=k, n_chunks=1, dtype="f32")
    b = _buffers(torch, mh, d)
    for score, renorm in (("sigmoid", True), ("softmax", False)):
        r = mh.make_router_scores(score=score, n_groups=n, topk_groups=3, renormalize=renorm)
        mh.moe_route_scores(d, -1, r, x, None, *[b[i] for i in NAMES])
        want = ors.choose(ors.scores(lg, score), None, k, n, 3, 1)
        np.testing.assert_array_equal(b["topk_idx"][rows].cpu().numpy(), want)
        plain = torch.ones(T, dtype=torch.bool, device="cuda")
        plain[rows] = False  # the others are ties: the first experts
        assert bool((b["topk_idx"][plain] == torch.arange(k, device="cuda")).all())
        assert int(b["counts"].sum()) == T * k
        dg = torch.ones(T, k, device="cuda")
        dg[:, 1] = 3.0
        dl = torch.full((T, E), 9.0, device="cuda")
        mh.moe_route_scores_bwd(d, -1, r, x, dg, b["topk_idx"], None, dl)
        ones = np.ones((len(rows), k), np.float32)
        ones[:, 1] = 3.0
        lim = TERM * ors.backward_bound(lg, want, ones, score, renorm, 1.0) + 2.0 ** -126
        assert np.all(np.abs(dl[rows].cpu().numpy() - ors.backward(lg, want, ones, score, renorm)) <= lim)
        assert float(dl.abs().max()) < 2.0
        del dl


def test_plain_routing_is_the_same_as_moe_route():
    torch, mh = _gpu()
    lg, _ = _draw(500, 64, 3)
    d, b = _forward(torch, mh, lg, None, 8, dict(score="softmax"))
    c = _buffers(torch, mh, d)
    mh.moe_route(d, -1, torch.from_numpy(lg).cuda(), *[c[x] for x in NAMES])
    torch.cuda.synchronize()
    for x in ("topk_idx", "counts", "offsets", "row_of", "src_token"):
        assert torch.equal(b[x], c[x]), x
    assert float((b["gates"] - c["gates"]).abs().max()) <= 2 * GATE


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("G,tg,top", [(1, 1, 1), (4, 2, 2), (8, 8, 1)])
def test_rows_that_are_not_ordinary(score, renorm, G, tg, top):
    torch, mh = _gpu()
    E, k = 32, 4
    rng = np.random.default_rng(8)
    lg, bias = _draw(200, E, 8)
    inf = np.inf
    lg[0] = -inf                                  # nothing to choose by
    lg[1] = np.nan
    lg[2, ::3] = np.nan
    lg[3, 5] = inf
    lg[4, [1, 9, 17, 25, 30]] = inf
    lg[5, 2:] = -inf                              # fewer values than slots
    lg[6] = 0.0                                   # ties everywhere
    lg[7] = np.float32(-0.0)
    lg[8] = np.round(lg[8])
    lg[9] = 20 + np.arange(E)                     # saturated sigmoids
    lg[10] = np.finfo(np.float32).min             # the type's lowest value as a mask
    lg[11, :16] = np.finfo(np.float32).min
    lg[12] = -200 + lg[12]                        # scores below FP32's range
    lg[13] = 88 + lg[13] * 4
    lg[20:60] = rng.integers(-2, 3, (40, E))      # many ties
    lg[60:100] = np.nextafter(lg[60:100, :1], np.float32(9)) * np.ones((1, E), dtype=np.float32)
    lg[60:100, rng.integers(0, E, 40)] += np.float32(2.0 ** -22)  # neighbours in the last bits
    odd = bias.copy()
    odd[3], odd[7], odd[11], odd[20] = -inf, np.nan, inf, -3e38
    how = dict(score=score, n_groups=G, topk_groups=tg, group_top=top, renormalize=renorm)
    for b_ in (None, bias, np.zeros(E, np.float32), odd, np.full(E, -inf, np.float32), np.full(E, np.float32(1e9))):
        d, b = _forward(torch, mh, lg, b_, k, how)
        _check(d, b, lg, b_, how, tol=(400 + 24) * F)  # arguments up to 400


def test_nearest_neighbours_are_ordered_by_their_exact_sums():
    """Sums that differ in the last bit of FP32, or not at all: rows whose scores lie a few FP32 steps apart."""
    torch, mh = _gpu()
    T, E, k = 4000, 64, 8
    rng = np.random.default_rng(11)
    lg = (rng.standard_normal((T, 1)) + rng.integers(-4, 5, (T, E)) * 2.0 ** -24 * rng.choice([1, 4, 16], (T, 1))).astype(np.float32)
    bias = (rng.integers(-3, 4, E) * 2.0 ** -25).astype(np.float32)
    for score in ("softmax", "sigmoid"):
        for G, tg in ((1, 1), (8, 4)):
            how = dict(score=score, n_groups=G, topk_groups=tg, group_top=2)
            d, b = _forward(torch, mh, lg, bias, k, how)
            _check(d, b, lg, bias, how)


def _close_rows(rng, T, E, score, above):
    """Rows whose FP32 sums lie around an edge where the low bits that a lane's list gives to an element's number run over:
    in every fourth row two to four experts within two FP32 steps of the edge, those with the highest and the lowest number
    among them, behind `above` clear ones (the other rows are clear: what one row of a wave's four needs settled, all
    get). Returns logits [T, E] and the bias [E]."""
    ne = 4
    while ne * 16 < E:
        ne *= 2
    e = np.arange(E)
    number = 4 * (e // 64) + e % 4 if E % 4 == 0 else e // 16
    sink, clear = E // 2, E // 2 + 1 + np.arange(above)
    rest = np.setdiff1d(e, np.append(clear, sink))
    low, high = rest[number[rest] == 0], rest[number[rest] == number[rest].max()]
    if score == "sigmoid":
        bias, span = rng.uniform(0.3, 0.4, E), 0.25
    else:
        bias, span = rng.uniform(0.78, 0.83, E), 0.04
        bias[sink] = -1.0
    bias[clear] = 1.5 + 0.01 * np.arange(above)
    bias = bias.astype(np.float32)
    want = np.full((T, E), 1e-7 if score == "softmax" else 0.007)  # the scores
    x = rng.uniform(1.0, 1.0 + span, T).astype(np.float32)
    x = (x.view(np.uint32) | np.uint32(ne - 1)).view(np.float32).astype(np.float64)  # the last value below an edge
    for t in range(T):
        more = rng.choice(rest, rng.integers(0, 4), replace=False)
        near = np.concatenate([[rng.choice(low)], [rng.choice(high)], np.setdiff1d(more, np.append(low, high))])
        near = near[:1 if t % 4 else 4 if score == "sigmoid" else 3].astype(int)
        want[t, near] = x[t] + rng.uniform(-0.7, 1.7, near.size) * 2.0 ** -23 - bias[near]
    if score == "sigmoid":
        return np.log(want / (1.0 - want)).astype(np.float32), bias
    want[:, sink] = 0.0
    want[:, sink] = 1.0 - want.sum(axis=1)
    assert want.min() > 0
    return np.log(want).astype(np.float32), bias


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,above,k,G,tg", [(9000, 256, 0, 1, 1, 1), (3000, 256, 6, 8, 1, 1), (60, 256, 0, 1, 1, 1), (3000, 512, 0, 1, 1, 1),
                                              (2000, 512, 3, 5, 1, 1), (2000, 1024, 0, 1, 1, 1), (2000, 1024, 2, 3, 1, 1), (2000, 250, 1, 2, 1, 1),
                                              (2000, 1000, 0, 2, 1, 1), (2000, 64, 0, 1, 1, 1), (2000, 128, 2, 4, 1, 1), (3000, 256, 0, 2, 8, 7),
                                              (2000, 1024, 0, 1, 4, 3)])
def test_sums_a_step_apart_whose_keys_lie_further(score, T, E, above, k, G, tg):
    torch, mh = _gpu()
    print(f"[route_scores] close {score, T, E, above, k, G, tg}", flush=True)
    lg, bias = _close_rows(np.random.default_rng(E + k), T, E, score, above)
    how = dict(score=score, n_groups=G, topk_groups=tg, group_top=1)
    want = ors.choose(ors.scores(lg, score), bias, k, G, tg, 1)
    d, b = _forward(torch, mh, lg, bias, k, how)
    bad = (b["topk_idx"].cpu().numpy() != want).any(axis=1)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3].ravel(), b["topk_idx"].cpu().numpy()[bad][:3], want[bad][:3])
    _check(d, b, lg, bias, how)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,G,tg", [(128, 1, 1), (256, 1, 1), (256, 8, 7), (252, 1, 1), (250, 1, 1), (1024, 1, 1)])
def test_equal_scores_in_rows_where_one_lane_has_most(score, E, G, tg):
    """Ties between experts of different lanes with the same number, and more of the largest in one lane than its list
    holds: the experts chosen are distinct and the definition's."""
    torch, mh = _gpu()
    print(f"[route_scores] ties {score, E, G, tg}", flush=True)
    T, k = 1200, 8
    rng = np.random.default_rng(E + G)
    e = np.arange(E)
    lane, number = ((e // 4) % 16, 4 * (e // 64) + e % 4) if E % 4 == 0 else (e % 16, e // 16)
    lg = rng.uniform(-2, -1, (T, E)).astype(np.float32)
    for t in range(0, T, 2):
        own = rng.permutation(e[lane == rng.integers(0, 16)])[:rng.integers(4, 9)]
        lg[t, own] = 1.0 + rng.permutation(own.size) / 16.0  # in any order with the ties
        for _ in range(rng.integers(1, 4)):
            same = rng.permutation(e[number == rng.integers(0, number.max())])
            lg[t, same[:rng.integers(2, 5)]] = rng.choice([0.5, 1.03125, 2.0])
    for bias in (None, np.full(E, np.float32(0.25))):
        how = dict(score=score, n_groups=G, topk_groups=tg, group_top=2)
        d, b = _forward(torch, mh, lg, bias, k, how)
        _check(d, b, lg, bias, how)


def test_no_tokens():
    torch, mh = _gpu()
    d, b = _forward(torch, mh, np.zeros((0, 16), np.float32), None, 2, dict(score="sigmoid"), n=2, El=4)
    assert not b["counts"].any() and not b["offsets"].any()
    dl = torch.zeros(0, 16, device="cuda")
    mh.moe_route_scores_bwd(d, -1, mh.make_router_scores(), dl, dl, b["topk_idx"], None, dl)


# ------------------------------------------------------------------ backward

CASES = [(score, renorm) for score in ("softmax", "sigmoid") for renorm in (True, False)]


@pytest.mark.parametrize("score,renorm", CASES)
@pytest.mark.parametrize("T,E,k,dtype,n", [(1, 8, 2, "f32", 1), (37, 33, 5, "f32", 2), (200, 4, 4, "bf16", 1), (130, 128, 8, "bf16", 2),
                                           (75, 132, 8, "bf16", 1), (66, 1000, 7, "f32", 1), (51, 1024, 8, "bf16", 3), (29, 1, 1, "f32", 1), (40, 256, 1, "bf16", 1)])
def test_backward(score, renorm, T, E, k, dtype, n):
    torch, mh = _gpu()
    print(f"[route_scores] backward {score, renorm, T, E, k, dtype, n}", flush=True)
    H = 128
    rng = np.random.default_rng(T + E)
    lg, bias = _draw(T, E, T + E, std=2.0)
    idx, _ = ors.route(lg, bias, k, score, renormalize=renorm)
    dg = (rng.standard_normal((T, k)) * 10.0 ** rng.uniform(-3, 2, (T, 1))).astype(np.float32)
    how = mh.make_router_scores(score=score, renormalize=renorm, scale=1.5)
    for flags in (0, mh.FLAG_ROUTER_LOSS):
        d = mh.make_desc(T=T, H=H, I=64, E=E, E_local=1, k=k, n_chunks=n, dtype=dtype, flags=flags)
        old = rng.standard_normal((T, E)).astype(np.float32) if flags else np.full((T, E), 5.0, np.float32)
        want = ors.backward(lg, idx, dg, score, renorm, 1.5) + (old if flags else 0)
        lim = TERM * ors.backward_bound(lg, idx, dg, score, renorm, 1.5) + 2.0 ** -126
        if flags:
            lim = lim + 2 * F * np.abs(want) + 2 * F * np.abs(old)
        x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).cuda().to(torch.float32 if dtype == "f32" else torch.bfloat16)
        ws = torch.zeros(mh.workspace_bytes(d)["workspace"], dtype=torch.uint8, device="cuda")
        dev = [torch.from_numpy(a).cuda() for a in (lg, dg, idx)]
        for with_x in (True, False):
            dl = torch.full((T + 1, E), 9.0, device="cuda")
            dl[:T] = torch.from_numpy(old).cuda()
            acc, dwr = torch.full((E, H), 3.0, device="cuda"), torch.full((E, H), 3.0, device="cuda", dtype=x.dtype)
            mh.moe_route_scores_bwd(d, -1, how, *dev, x if with_x else None, dl, *((acc, dwr, ws) if with_x else ()))
            torch.cuda.synchronize()
            bad = np.abs(dl[:T].cpu().numpy() - want) > lim
            assert not bad.any(), (np.argwhere(bad)[:3], dl[:T].cpu().numpy()[bad][:3], want[bad][:3])
            assert (dl[T] == 9.0).all()
            if with_x:
                ref = want.T @ x.double().cpu().numpy()
                # T terms in FP32 (BF16: of dlogits in two parts, 2^-17), and dwr's own rounding
                mag = (np.abs(want) + lim).T @ np.abs(x.double().cpu().numpy())
                err = (lim.T @ np.abs(x.double().cpu().numpy())) + (T * F + (0 if dtype == "f32" else 2.0 ** -16)) * mag
                assert np.all(np.abs(acc.double().cpu().numpy() - ref) <= err + 2.0 ** -120)
                assert np.all(np.abs(dwr.double().cpu().numpy() - ref) <= err + (F if dtype == "f32" else 2.0 ** -8) * (np.abs(ref) + err) + 2.0 ** -120)


@pytest.mark.parametrize("score,renorm", CASES)
def test_backward_matches_differences_of_the_forward(score, renorm):
    """Central differences of the kernel's own gates: FP32 gates are good to GATE, so a step of 1/64 leaves
    GATE / (2 / 64) of rounding and (1 / 64)^2 / 6 of the third derivative, below 1 for these scores, per slot."""
    torch, mh = _gpu()
    T, E, k = 24, 8, 3
    rng = np.random.default_rng(2)
    lg = rng.standard_normal((T, E)).astype(np.float32)
    lg = np.round(lg * 64) / 64 + np.arange(E, dtype=np.float32) / 8  # steps are exact, the choice does not change often
    dg = rng.standard_normal((T, k)).astype(np.float32)
    how = dict(score=score, renormalize=renorm, scale=1.0)
    d, b = _forward(torch, mh, lg, None, k, how)
    dl = torch.empty(T, E, device="cuda")
    mh.moe_route_scores_bwd(d, -1, mh.make_router_scores(**how), torch.from_numpy(lg).cuda(), torch.from_numpy(dg).cuda(), b["topk_idx"], None, dl)
    got, idx, h = dl.cpu().numpy(), b["topk_idx"].cpu().numpy(), np.float32(1 / 64)
    seen = 0
    for e in range(E):
        diff, same = np.zeros(T), np.ones(T, dtype=bool)
        for s in (1, -1):
            moved = lg.copy()
            moved[:, e] += s * h
            _, c = _forward(torch, mh, moved, None, k, how)
            ci, cg = c["topk_idx"].cpu().numpy(), c["gates"].cpu().numpy().astype(np.float64)
            order = np.argsort(ci, axis=1)
            mine = np.argsort(idx, axis=1)
            same &= np.all(np.take_along_axis(ci, order, 1) == np.take_along_axis(idx, mine, 1), axis=1)
            diff += s * (np.take_along_axis(cg, order, 1) * np.take_along_axis(dg, mine, 1)).sum(axis=1) / (2 * float(h))
        lim = (np.abs(dg).sum(axis=1)) * (GATE / (2 * float(h)) + float(h) ** 2 / 6 + TERM)
        assert np.all(np.abs(diff - got[:, e])[same] <= lim[same])
        seen += int(same.sum())
    assert seen > T * E // 2


def test_backward_of_rows_without_values():
    torch, mh = _gpu()
    lg = np.zeros((4, 8), np.float32)
    lg[0], lg[1], lg[2, 4:], lg[3, 0] = -np.inf, np.nan, -np.inf, np.inf
    dg = np.ones((4, 3), np.float32) * np.arange(1, 4, dtype=np.float32)
    for score, renorm in CASES:
        idx, _ = ors.route(lg, None, 3, score, renormalize=renorm)
        want = ors.backward(lg, idx, dg, score, renorm)
        d = mh.make_desc(T=4, H=64, I=64, E=8, E_local=1, k=3, n_chunks=1, dtype="f32")
        dl = torch.full((4, 8), 9.0, device="cuda")
        mh.moe_route_scores_bwd(d, -1, mh.make_router_scores(score=score, renormalize=renorm), torch.from_numpy(lg).cuda(),
                                torch.from_numpy(dg).cuda(), torch.from_numpy(idx).cuda(), None, dl)
        np.testing.assert_allclose(dl.cpu().numpy(), want, atol=16 * F, rtol=0)


# ------------------------------------------------------------------ bias update, streams, graphs

@pytest.mark.parametrize("E,rows", [(1, 1), (8, 2), (60, 3), (256, 1), (1000, 2), (1024, 7)])
def test_bias_update(E, rows):
    torch, mh = _gpu()
    rng = np.random.default_rng(E)
    counts = rng.integers(0, 5, (rows, E)).astype(np.int32)
    bias = rng.standard_normal(E).astype(np.float32)
    b = torch.from_numpy(np.append(bias, np.float32(4.0))).cuda()
    mh.moe_router_bias_update(E, rows, torch.from_numpy(counts).cuda(), 0.001, b)
    np.testing.assert_array_equal(b.cpu().numpy()[:E], ors.bias_update(bias, counts, 0.001))
    assert float(b[E]) == 4.0
    big = np.full((2, E), 2 ** 31 - 1, dtype=np.int32)  # sums past 32 bits
    big[0, 0] = 0
    c = torch.from_numpy(bias).cuda()
    mh.moe_router_bias_update(E, 2, torch.from_numpy(big).cuda(), 0.5, c)
    np.testing.assert_array_equal(c.cpu().numpy(), ors.bias_update(bias, big, 0.5))


def test_two_routings_at_once():
    torch, mh = _gpu()
    cases = [(20000, 256, dict(score="sigmoid", n_groups=8, topk_groups=4, group_top=2)), (3000, 128, dict(score="softmax"))]
    want = [_forward(torch, mh, *_draw(T, E, T), 8, how)[1] for T, E, how in cases]
    dev = []
    for T, E, how in cases:
        lg, bias = _draw(T, E, T)
        d = mh.make_desc(T=T, H=64, I=64, E=E, E_local=E, k=8, n_chunks=1, dtype="f32")
        dev.append((d, mh.make_router_scores(**how), torch.from_numpy(lg).cuda(), torch.from_numpy(bias).cuda(), _buffers(torch, mh, d), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(3):
        for d, r, lg, bias, b, stream in dev:
            mh.moe_route_scores(d, -1, r, lg, bias, *[b[x] for x in NAMES], stream)
    torch.cuda.synchronize()
    for (*_, b, _), ref in zip(dev, want):
        for x in NAMES[:-1]:
            assert torch.equal(b[x], ref[x]), x


def test_on_another_stream_and_in_a_graph():
    torch, mh = _gpu()
    lg, bias = _draw(700, 128, 5)
    how = dict(score="sigmoid", n_groups=8, topk_groups=4, group_top=2)
    d, ref = _forward(torch, mh, lg, bias, 8, how, n=2, El=16)
    r = mh.make_router_scores(**how)
    dev, bi = torch.from_numpy(lg).cuda(), torch.from_numpy(bias).cuda()
    dg, dl = torch.ones(700, 8, device="cuda"), torch.empty(700, 128, device="cuda")
    side, b = torch.cuda.Stream(), _buffers(torch, mh, d)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(1_000_000)
        mh.moe_route_scores(d, -1, r, dev, bi, *[b[x] for x in NAMES])
    torch.cuda.synchronize()
    for x in NAMES[:-1]:
        assert torch.equal(b[x], ref[x]), x
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        mh.moe_route_scores(d, -1, r, dev, bi, *[b[x] for x in NAMES])
        mh.moe_route_scores_bwd(d, -1, r, dev, dg, b["topk_idx"], None, dl)
        mh.moe_router_bias_update(128, 2, b["counts"], 0.01, bi)
    for i in range(4):
        lg2, _ = _draw(700, 128, 50 + i)
        before = bi.cpu().numpy().copy()
        dev.copy_(torch.from_numpy(lg2).cuda())
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        _check(d, b, lg2, before, how)
        got = dl.clone()
        np.testing.assert_array_equal(bi.cpu().numpy(), ors.bias_update(before, b["counts"].cpu().numpy(), 0.01))
        mh.moe_route_scores_bwd(d, -1, r, dev, dg, b["topk_idx"], None, dl)
        assert torch.equal(got, dl)


# ------------------------------------------------------------------ layers that route by scores

LAYERS = [MoeConfig("rs_f32", T=200, H=128, I=64, E=12, E_local=6, e0=3, k=3, n_chunks=3, dtype="f32", seed_base=1100, x_std=0.02, backward=True),
          MoeConfig("rs_bf16", T=1000, H=256, I=192, E=32, E_local=8, e0=4, k=4, n_chunks=2, dtype="bf16", seed_base=1110, backward=True)]
HOWS = [dict(score="sigmoid", n_groups=4, topk_groups=2, group_top=2, renormalize=True, scale=2.5),
        dict(score="softmax", renormalize=False, scale=3.0),
        dict(score="sigmoid", renormalize=False)]


def _layer_bufs(torch, mh, cfg, how, flags=0, backward=True):
    inp = harness.moe_inputs.make_inputs(cfg, with_backward=backward)
    d = mh.make_desc(T=cfg.T, H=cfg.H, I=cfg.I, E=cfg.E, E_local=cfg.E_local, k=cfg.k, n_chunks=cfg.n_chunks,
                     dtype=cfg.dtype, e0=cfg.e0, flags=mh.FLAG_ROUTER_SCORES | flags)
    b = mh.allocate(d, backward=backward, n_segments=1)
    wdt = "bf16" if cfg.dtype == "fp8" else cfg.dtype
    for name in ("x", "logits", "w1", "w2", "w_r") + (("dy",) if backward else ()):
        b[name] = harness.to_dev(inp, name, wdt)
    bias = (np.random.default_rng(cfg.seed_base).standard_normal(cfg.E) * 0.1).astype(np.float32)
    b["router_bias"], b["router_scores"] = torch.from_numpy(bias).cuda(), mh.make_router_scores(**how)
    b.update(balance_coef=0.02, z_coef=0.003)
    return d, b, inp, bias


def _layer_ref(cfg, inp, bias, how, P_c, loss):
    idx, gates = ors.route(inp["logits"], bias, cfg.k, **how)
    counts, offsets, row_of, src = oracle.layout(idx, cfg.E, cfg.e0, cfg.E_local, cfg.n_chunks, P_c)
    xd = oracle.dispatch(np.asarray(inp["x"], dtype=np.float64), src)
    gu, h, yd = oracle.expert_ffn(xd, offsets, P_c, inp["w1"], inp["w2"])
    ref = dict(idx=idx, gates=gates, counts=counts, offsets=offsets, row_of=row_of, src_token=src, out=oracle.combine(yd, gates, row_of))
    if not cfg.backward:
        return ref
    from oracle import ffn as of
    dyd, dgates = of.combine_bwd(inp["dy"], yd, gates, row_of, src.size)
    dl = ors.backward(inp["logits"], idx, dgates, how["score"], how.get("renormalize", True), how.get("scale", 1.0))
    if loss:
        dl = dl + orl.router_loss_bwd(orl.router_loss(inp["logits"], idx, cfg.k, 0.02, 0.003), cfg.k, 0.02, 0.003)
    _, dxd, dw1, dw2 = of.ffn_bwd(dyd, xd, gu, h, offsets, P_c, inp["w1"], inp["w2"])
    ref["bwd"] = dict(dgates=dgates, dlogits=dl, dx=of.dispatch_bwd(dxd, row_of, dl, inp["w_r"]), dw1=dw1, dw2=dw2,
                      dwr=dl.T @ np.asarray(inp["x"], dtype=np.float64))
    return ref


def _stages(mh, d, b, s):
    r = b["router_scores"]
    mh.moe_route_scores(d, -1, r, b["logits"], b["router_bias"], *[b[x] for x in NAMES], s)
    mh.moe_dispatch(d, -1, b["x"], b["row_of"], b["xd"], None, None, s)
    mh.moe_expert_ffn(d, -1, b["xd"], None, b["w1"], None, b["w2"], None, b["offsets"], b["gu"], b["h"], None, b["yd"], s)
    mh.moe_combine(d, -1, b["yd"], b["gates"], b["row_of"], b["out"], s)
    mh.moe_combine_bwd(d, -1, b["dy"], b["yd"], b["gates"], b["row_of"], b["dyd"], b["dgates"], s)
    mh.moe_route_scores_bwd(d, -1, r, b["logits"], b["dgates"], b["topk_idx"], b["x"], b["dlogits"], b["dwr_acc"], b["dwr"], b["workspace"], s)
    mh.moe_expert_ffn_bwd(d, -1, b["dyd"], b["xd"], b["gu"], b["h"], b["w1"], b["w2"], b["offsets"], b["dgu"], b["dxd"],
                          b["dw1"], b["dw2"], b["workspace"], s)
    mh.moe_dispatch_bwd(d, -1, b["dxd"], b["row_of"], b["topk_idx"], b["dlogits"], b["w_r"], b["dx"], s)


OUT = ("out", "topk_idx", "gates", "dgates", "dlogits", "dx", "dwr", "dw1", "dw2")


@pytest.mark.parametrize("loss", [False, True])
@pytest.mark.parametrize("how", HOWS, ids=["grouped", "softmax", "sigmoid"])
@pytest.mark.parametrize("cfg", LAYERS, ids=lambda c: c.name)
def test_layer(cfg, how, loss):
    torch, mh = _gpu()
    print(f"[route_scores] layer {cfg.name} {how} {loss}", flush=True)
    d, b, inp, bias = _layer_bufs(torch, mh, cfg, how, mh.FLAG_ROUTER_LOSS if loss else 0)
    cs, aux = torch.cuda.current_stream(), torch.cuda.Stream()
    mh.moe_layer_forward_backward(d, b, cs, aux)
    torch.cuda.synchronize()
    ref = _layer_ref(cfg, inp, bias, how, d.P_c, loss)
    run = harness.Run(cfg, d, b, inp)
    for name in ("topk_idx", "counts", "offsets", "row_of", "src_token"):
        np.testing.assert_array_equal(b[name].cpu().numpy(), ref["idx" if name == "topk_idx" else name], err_msg=name)
    np.testing.assert_allclose(b["gates"].cpu().numpy(), ref["gates"], rtol=GATE)
    harness.assert_close("out", harness.to_np(b["out"][:cfg.T]), ref["out"], cfg.dtype)
    harness.check_backward(run, ref)
    keep = {n: b[n].clone() for n in OUT}
    mh.moe_layer_forward(d, b, cs, aux)
    mh.moe_layer_backward(d, b, cs, aux)
    torch.cuda.synchronize()
    rows = lambda n, t: t[:cfg.T] if n == "out" else t  # noqa: E731
    for n in OUT:
        assert torch.equal(rows(n, keep[n]), rows(n, b[n])), n
    if loss:
        return
    # the stage calls, dispatch backward with the dense sum where the gradient is dense
    if how["score"] == "softmax":
        d2 = mh.MoeDesc.from_buffer_copy(d)
        d2.flags |= mh.FLAG_ROUTER_LOSS
        b["dlogits"].zero_()
    else:
        d2 = d
    for n in OUT:
        if n != "dlogits" or d2 is d:
            b[n].fill_(3)
    _stages(mh, d2, b, cs)
    torch.cuda.synchronize()
    for n in OUT:
        assert torch.equal(rows(n, keep[n]), rows(n, b[n])), n


@pytest.mark.parametrize("loss", [False, True])
@pytest.mark.parametrize("how", HOWS[:2], ids=["grouped", "softmax"])
def test_layer_from_x(how, loss):
    """Without logits: the layer on the logits that the projection left is the same, bit for bit."""
    torch, mh = _gpu()
    cfg = LAYERS[1]
    d, b, _, _ = _layer_bufs(torch, mh, cfg, how, mh.FLAG_ROUTER_LOSS if loss else 0)
    cs, aux = torch.cuda.current_stream(), torch.cuda.Stream()
    b["logits"] = None
    b["w_r"].mul_(8.0)
    b["router_logits"].fill_(float("nan"))
    mh.moe_layer_forward_backward(d, b, cs, aux)
    torch.cuda.synchronize()
    # FP32 sums of H exact products, in any order: H 2^-24 of the sum of magnitudes
    want = b["x"].double() @ b["w_r"].double().t().contiguous()
    mag = b["x"].double().abs() @ b["w_r"].double().abs().t().contiguous()
    assert ((b["router_logits"].double() - want).abs() <= cfg.H * F * mag).all()
    keep = {n: b[n].clone() for n in OUT}
    b["logits"] = b["router_logits"].clone()
    for n in OUT:
        b[n].fill_(3)
    mh.moe_layer_forward_backward(d, b, cs, aux)
    torch.cuda.synchronize()
    for n in OUT:
        assert torch.equal(keep[n][:cfg.T], b[n][:cfg.T]), n


@pytest.mark.parametrize("dtype", ["fp8", "int8"])
def test_serving_layer(dtype):
    """Forward-only payloads: the layer is dispatch, experts and combine behind the same routing."""
    torch, mh = _gpu()
    cfg = MoeConfig("rs_" + dtype, T=300, H=256, I=128, E=16, E_local=8, e0=2, k=2, n_chunks=2, dtype="bf16", seed_base=1120)
    d0, b, inp, bias = _layer_bufs(torch, mh, cfg, HOWS[0], backward=False)
    d = mh.make_desc(T=cfg.T, H=cfg.H, I=cfg.I, E=cfg.E, E_local=cfg.E_local, k=cfg.k, n_chunks=2, dtype=dtype, e0=cfg.e0, flags=mh.FLAG_ROUTER_SCORES)
    c = mh.allocate(d, backward=False)
    c.update({n: b[n] for n in ("x", "logits", "router_bias", "router_scores", "w_r")})
    for n, rows, cols in (("w1", 8 * 2 * cfg.I, cfg.H), ("w2", 8 * cfg.H, cfg.I)):
        c[n] = torch.empty(rows, cols, dtype=torch.uint8, device="cuda")
        c[n + "_scale"] = torch.empty(rows, device="cuda")
        (mh.moe_quantize_rows_fp8 if dtype == "fp8" else mh.moe_quantize_rows_i8)(rows, cols, b[n], c[n], c[n + "_scale"])
    mh.moe_layer_forward(d, c, torch.cuda.current_stream(), torch.cuda.Stream())
    torch.cuda.synchronize()
    ref = _layer_ref(cfg, inp, bias, HOWS[0], d.P_c, False)
    np.testing.assert_array_equal(c["topk_idx"].cpu().numpy(), ref["idx"])
    got = c["out"][:cfg.T].clone()
    mh.moe_dispatch(d, -1, c["x"], c["row_of"], c["xd"], c["xd_scale"], c["h_scale"])
    mh.moe_expert_ffn(d, -1, c["xd"], c["xd_scale"], c["w1"], c["w1_scale"], c["w2"], c["w2_scale"], c["offsets"], None, c["h"], c["h_scale"], c["yd"])
    mh.moe_combine(d, -1, c["yd"], c["gates"], c["row_of"], c["out"])
    torch.cuda.synchronize()
    assert torch.equal(got, c["out"][:cfg.T])
    rel = np.linalg.norm(harness.to_np(got) - ref["out"]) / np.linalg.norm(ref["out"])
    # An e4m3 code is off by at most 2^-4 of the value, in the root mean square by 2^-4 / sqrt(3) = 0.036. G and U are sums of
    # products of two such values: sqrt(2) 0.036 = 0.051 of their norm. h = silu(G) U with |G| about 0.3, where z silu'(z) /
    # silu(z) stays under 1.2: sqrt(1.2^2 + 1) 0.051 = 0.080; the codes of h and of W2 add 0.036 each:
    # sqrt(0.080^2 + 2 * 0.036^2) = 0.095. Int8 codes, 127 to a row's largest value (3 deviations), are five times finer.
    assert rel <= (0.095 if dtype == "fp8" else 0.06), rel


@pytest.mark.parametrize("dtype", ["fp8", "int8"])
def test_serving_layer_from_x(dtype):
    """Without logits: the layer on the logits that the projection left is the same, bit for bit."""
    torch, mh = _gpu()
    cfg = MoeConfig("rsx_" + dtype, T=300, H=256, I=128, E=32, E_local=8, e0=2, k=2, n_chunks=2, dtype="bf16", seed_base=1130)
    _, b, _, _ = _layer_bufs(torch, mh, cfg, HOWS[0], backward=False)
    d = mh.make_desc(T=cfg.T, H=cfg.H, I=cfg.I, E=cfg.E, E_local=cfg.E_local, k=cfg.k, n_chunks=2, dtype=dtype, e0=cfg.e0, flags=mh.FLAG_ROUTER_SCORES)
    c = mh.allocate(d, backward=False)
    c.update({n: b[n] for n in ("x", "router_bias", "router_scores", "w_r")})
    c["w_r"].mul_(8.0)
    for n, rows, cols in (("w1", 8 * 2 * cfg.I, cfg.H), ("w2", 8 * cfg.H, cfg.I)):
        c[n] = torch.empty(rows, cols, dtype=torch.uint8, device="cuda")
        c[n + "_scale"] = torch.empty(rows, device="cuda")
        (mh.moe_quantize_rows_fp8 if dtype == "fp8" else mh.moe_quantize_rows_i8)(rows, cols, b[n], c[n], c[n + "_scale"])
    got = {}
    for logits in (None, "router_logits"):
        c["logits"] = None if logits is None else c[logits].clone()
        c["out"].fill_(3)
        mh.moe_layer_forward(d, c, torch.cuda.current_stream(), torch.cuda.Stream())
        torch.cuda.synchronize()
        now = {n: c[n][:cfg.T].clone() for n in ("out", "topk_idx", "gates")}
        assert not got or all(torch.equal(got[n], now[n]) for n in now)
        got = now
    lg, bias = c["router_logits"].cpu().numpy(), c["router_bias"].cpu().numpy()
    np.testing.assert_array_equal(got["topk_idx"].cpu().numpy(), ors.route(lg, bias, cfg.k, **HOWS[0])[0])
    assert float(got["out"].float().abs().max()) > 0


@pytest.mark.parametrize("how", HOWS[:2], ids=["grouped", "softmax"])
def test_layer_replays_in_a_graph(how):
    torch, mh = _gpu()
    d, b, _, _ = _layer_bufs(torch, mh, LAYERS[1], how)
    main, aux = torch.cuda.Stream(), torch.cuda.Stream()
    mh.moe_layer_forward_backward(d, b, torch.cuda.current_stream(), aux)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=main):
        mh.moe_layer_forward_backward(d, b, torch.cuda.current_stream(), aux)
    l0 = b["logits"].clone()
    for i in range(3):
        b["logits"].copy_(l0 * (1 + i))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = {n: b[n].clone() for n in OUT}
        for n in OUT:
            b[n].fill_(3)
        mh.moe_layer_forward_backward(d, b, torch.cuda.current_stream(), aux)
        torch.cuda.synchronize()
        for n in OUT:
            assert torch.equal(got[n][:1000], b[n][:1000]), (i, n)
