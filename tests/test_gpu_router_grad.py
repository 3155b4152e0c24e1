"""GPU parity of the dense router gradient (MOE_FLAG_ROUTER_LOSS) and of the layer primitives that run the router loss.

Stage tolerances. BF16 dx: dlogits in two BF16 parts loses 2^-17 of each value, the FP32 sums of E + k terms round at
2^-24 of the terms each, and dx rounds once, 2^-8 of its value. FP32 dx: (E + k) 2^-24 of the terms, and the MFMA-free
sum. dlogits adds two FP32 values: 2^-24 of the sum, beside the error of the route backward's own three products
(6 * 2^-24 of their terms). The layer's outputs take the harness's bounds of their dtype; the loss adds only terms that
are linear in dlogits, so the reference is the layer's oracle plus the loss's dlogits, its product with W_r and with x."""
import numpy as np
import pytest

import moe_inputs
from moe_inputs import MoeConfig
from oracle import fp8 as ofp8
from oracle import router_loss as orl

pytestmark = pytest.mark.gpu
harness = pytest.importorskip("harness")
F = 2.0 ** -24


def _gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import combine_moe_route_02_amd as mh
    mh.lib()
    return torch, mh


def _dev(torch, a, dtype):
    if dtype == "f32":
        return torch.from_numpy(a).cuda(), a.astype(np.float64)
    bits = moe_inputs.f32_to_bf16_bits(a)
    return torch.from_numpy(bits.view(np.int16)).cuda().view(torch.bfloat16), moe_inputs.bf16_bits_to_f32(bits).astype(np.float64)


def _setup(torch, mh, T, H, E, El, k, n, dtype, seed, flags=0):
    rng = np.random.default_rng(seed)
    d = mh.make_desc(T=T, H=H, I=64, E=E, E_local=El, k=k, n_chunks=n, dtype=dtype, flags=mh.FLAG_ROUTER_LOSS | flags)
    P = n * d.P_c
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    row = np.full((T, k), -1, dtype=np.int32)
    local = idx < El
    row[local] = rng.permutation(P)[:local.sum()]
    dxd, dxd64 = _dev(torch, rng.standard_normal((max(P, 1), H)).astype(np.float32), dtype)
    w, w64 = _dev(torch, (rng.standard_normal((E, H)) * 0.1).astype(np.float32), dtype)
    dl = (rng.standard_normal((T, E)) * 10.0 ** rng.uniform(-3, 1, (T, 1))).astype(np.float32)
    return d, rng, idx, row, dxd, dxd64, w, w64, dl


def _ref(row, dxd64, dl, w64):
    ref, mag = dl.astype(np.float64) @ w64, np.abs(dl.astype(np.float64)) @ np.abs(w64)
    for j in range(row.shape[1]):
        m = row[:, j] >= 0
        ref[m] += dxd64[row[m, j]]
        mag[m] += np.abs(dxd64[row[m, j]])
    return ref, mag


# tokens around the 32-token tile, E at each fragment count and past it, H at each slice end
SHAPES = [(1, 64, 4, 4, 1, 1), (31, 192, 8, 3, 2, 1), (33, 320, 32, 32, 8, 1), (100, 256, 100, 20, 5, 3),
          (257, 128, 128, 16, 8, 2), (65, 576, 132, 60, 7, 1), (70, 64, 256, 10, 3, 1), (40, 448, 260, 260, 8, 1),
          (50, 192, 512, 5, 4, 2), (64, 256, 1024, 40, 8, 1), (1000, 2048, 128, 16, 8, 2), (20, 64, 16, 0, 2, 1)]


@pytest.mark.parametrize("T,H,E,El,k,n", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_dispatch_bwd(T, H, E, El, k, n, dtype):
    torch, mh = _gpu()
    print(f"[router_grad] {T, H, E, El, k, n, dtype}", flush=True)
    d, rng, idx, row, dxd, dxd64, w, w64, dl = _setup(torch, mh, T, H, E, El, k, n, dtype, T + H + E)
    dx = torch.full((T + 1, H), -5.0, dtype=dxd.dtype, device="cuda")
    args = (dxd if El else None, torch.from_numpy(row).cuda(), torch.from_numpy(idx).cuda(), torch.from_numpy(dl).cuda(), w)
    mh.moe_dispatch_bwd(d, -1, *args, dx)
    torch.cuda.synchronize()
    got = harness.to_np(dx)
    assert np.all(got[T] == -5.0)
    ref, mag = _ref(row, dxd64, dl, w64)
    lim = (E + k) * F * mag if dtype == "f32" else 2.0 ** -8 * np.abs(ref) + ((E + k) * F + 2.0 ** -17) * mag * (1 + 2.0 ** -8)
    assert np.all(np.abs(got[:T] - ref) <= lim), np.max(np.abs(got[:T] - ref) / np.maximum(lim, 1e-300))
    # chunk by chunk the same bits, and only the chunk's rows written
    tc = -(-T // n)
    again = torch.full_like(dx, -5.0)
    for c in range(n):
        mh.moe_dispatch_bwd(d, c, *args, again)
        torch.cuda.synchronize()
        assert torch.equal(again[:min(T, (c + 1) * tc)], dx[:min(T, (c + 1) * tc)])
        assert (again[min(T, (c + 1) * tc):] == -5.0).all()


# FP32 takes any number of experts: around the chunks of 64, odd ones, a single one
@pytest.mark.parametrize("T,H,E,El,k,n", [(33, 64, 1, 1, 1, 1), (5, 192, 3, 2, 2, 1), (64, 128, 63, 7, 8, 1), (65, 320, 65, 65, 8, 2),
                                          (97, 192, 131, 40, 5, 1), (300, 1088, 127, 30, 6, 3)])
def test_dispatch_bwd_f32_any_experts(T, H, E, El, k, n):
    test_dispatch_bwd(T, H, E, El, k, n, "f32")


@pytest.mark.parametrize("T,H,E,El,k,n", [SHAPES[2], SHAPES[3], SHAPES[5], SHAPES[8]])
def test_dispatch_bwd_fp8_rows(T, H, E, El, k, n):
    torch, mh = _gpu()
    d, rng, idx, row, _, _, w, w64, dl = _setup(torch, mh, T, H, E, El, k, n, "bf16", T * 3, mh.FLAG_FP8_DXD)
    P, nb = n * d.P_c, (H + 255) // 256
    codes = rng.integers(0, 127, (P, H)).astype(np.uint8) | (rng.integers(0, 2, (P, H)).astype(np.uint8) << 7)
    codes[(codes & 0x7f) == 0x7f] = 0
    sc = (rng.random((P, nb)) * 0.01 + 0.001).astype(np.float32)
    buf = torch.zeros(P * H * 2, dtype=torch.uint8, device="cuda")
    buf[:P * H] = torch.from_numpy(codes.reshape(-1)).cuda()
    buf[P * H:P * H + 4 * P * nb] = torch.from_numpy(sc.view(np.uint8).reshape(-1)).cuda()
    dx = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    mh.moe_dispatch_bwd(d, -1, buf, torch.from_numpy(row).cuda(), torch.from_numpy(idx).cuda(), torch.from_numpy(dl).cuda(), w, dx)
    torch.cuda.synchronize()
    ref, mag = _ref(row, ofp8.dequantize_row_blocks(codes, sc), dl, w64)
    # a dequantised value is one FP32 product: one more rounding of each term
    lim = 2.0 ** -8 * np.abs(ref) + ((E + 2 * k) * F + 2.0 ** -17) * mag * (1 + 2.0 ** -8)
    assert np.all(np.abs(harness.to_np(dx) - ref) <= lim)


@pytest.mark.parametrize("T,H,E,k,n,dtype", [(1, 64, 4, 1, 1, "bf16"), (50, 128, 32, 8, 3, "bf16"), (300, 192, 132, 5, 2, "bf16"),
                                             (90, 64, 7, 3, 2, "f32")])
def test_route_bwd_adds_to_dlogits(T, H, E, k, n, dtype):
    torch, mh = _gpu()
    rng = np.random.default_rng(T + E)
    kw = dict(T=T, H=H, I=64, E=E, E_local=1, k=k, n_chunks=n, dtype=dtype)
    d = mh.make_desc(flags=mh.FLAG_ROUTER_LOSS, **kw)
    b = mh.allocate(d)
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    gates = rng.random((T, k)).astype(np.float32)
    gates /= gates.sum(1, keepdims=True)
    dg, base = rng.standard_normal((T, k)).astype(np.float32), rng.standard_normal((T, E)).astype(np.float32)
    x, x64 = _dev(torch, rng.standard_normal((T, H)).astype(np.float32), dtype)
    args = [torch.from_numpy(a).cuda() for a in (dg, gates, idx)] + [x]
    b["dlogits"].copy_(torch.from_numpy(base))
    mh.moe_route_bwd(d, -1, *args, b["dlogits"], b["dwr_acc"], b["dwr"], b["workspace"])
    torch.cuda.synchronize()
    g64, dg64 = gates.astype(np.float64), dg.astype(np.float64)
    sel = g64 * (dg64 - (g64 * dg64).sum(1, keepdims=True))
    mag = g64 * (np.abs(dg64) + (g64 * np.abs(dg64)).sum(1, keepdims=True))
    want, terms = base.astype(np.float64), np.abs(base).astype(np.float64)
    add, addm = np.zeros((T, E)), np.zeros((T, E))
    np.put_along_axis(add, idx.astype(np.int64), sel, 1)
    np.put_along_axis(addm, idx.astype(np.int64), mag, 1)
    want, terms = want + add, addm
    got = b["dlogits"].cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - want) <= F * np.abs(want) + (k + 6) * F * terms)
    # the weight gradient is the product of the dense rows
    wr, wrm = got.T @ x64, np.abs(got).T @ np.abs(x64)
    eps = 2.0 ** -8 * np.abs(wr) + (T * F + 2.0 ** -16) * wrm if dtype == "bf16" else (T + 2) * F * wrm
    assert np.all(np.abs(harness.to_np(b["dwr"]) - wr) <= eps * (1 + 2.0 ** -8))


LAYERS = [
    MoeConfig("rl_n1", T=300, H=128, I=64, E=8, E_local=4, e0=2, k=2, n_chunks=1, dtype="bf16", seed_base=980, backward=True),
    MoeConfig("rl_n3", T=1000, H=256, I=192, E=32, E_local=8, e0=4, k=4, n_chunks=3, dtype="bf16", seed_base=985, backward=True),
    MoeConfig("rl_zipf", T=1500, H=320, I=128, E=64, E_local=8, k=8, n_chunks=2, dtype="bf16", seed_base=990, zipf_s=1.2,
              n_empty=2, backward=True),
    MoeConfig("rl_f32", T=256, H=128, I=256, E=8, E_local=8, k=2, n_chunks=1, dtype="f32", seed_base=0, x_std=0.02, backward=True),
    MoeConfig("rl_none_local", T=200, H=128, I=64, E=8, E_local=0, e0=8, k=2, n_chunks=2, dtype="bf16", seed_base=995, backward=True),
]
A, Z, G = 60.0, 2.0, 0.75  # the loss's part of dx shows against the experts' (checked below)


def _layer(torch, mh, cfg, flags, how, two=True):
    inp = moe_inputs.make_inputs(cfg, with_backward=True)
    d = mh.make_desc(T=cfg.T, H=cfg.H, I=cfg.I, E=cfg.E, E_local=cfg.E_local, k=cfg.k, n_chunks=cfg.n_chunks,
                     dtype=cfg.dtype, e0=cfg.e0, flags=flags | mh.FLAG_ROUTER_LOSS)
    off = [0, cfg.T // 3, cfg.T // 3, cfg.T - 5]
    mask = (np.random.default_rng(1).random(cfg.T) < 0.9).astype(np.uint8)
    b = mh.allocate(d, n_segments=3)
    for name in ("x", "logits", "w1", "w2", "w_r", "dy"):
        b[name] = harness.to_dev(inp, name, cfg.dtype)
    b.update(seg_offsets=torch.tensor(off, dtype=torch.int32, device="cuda"), token_mask=torch.from_numpy(mask).cuda(),
             dloss=torch.full((1,), G, device="cuda"), balance_coef=A, z_coef=Z)
    if flags & mh.FLAG_FP8_DGRAD:
        mh.moe_quantize_cols_fp8(cfg.E_local, 2 * cfg.I, cfg.H, b["w1"], b["w1t"], b["w1t_scale"])
        mh.moe_quantize_cols_fp8(cfg.E_local, cfg.H, cfg.I, b["w2"], b["w2t"], b["w2t_scale"])
    if how == "from_x":
        b["logits"] = None
    cs = torch.cuda.current_stream()
    aux = torch.cuda.Stream() if two else cs
    if how == "apart":
        mh.moe_layer_forward(d, b, cs, aux)
        mh.moe_layer_backward(d, b, cs, aux)
    else:
        mh.moe_layer_forward_backward(d, b, cs, aux)
    torch.cuda.synchronize()
    if how == "from_x":
        inp["logits"] = b["router_logits"].cpu().numpy()
    return harness.Run(cfg, d, b, inp), off, mask


def _check(run, off, mask, mh):
    cfg, b = run.cfg, run.bufs
    f = orl.router_loss(run.inp["logits"], b["topk_idx"].cpu().numpy(), cfg.k, A, Z, off, mask)
    np.testing.assert_array_equal(b["seg_counts"].cpu().numpy(), f["seg_counts"])
    np.testing.assert_allclose(b["router_loss"].cpu().numpy(), f["loss"], rtol=6e-5)
    dl = orl.router_loss_bwd(f, cfg.k, A, Z, G)
    run.desc.flags &= ~mh.FLAG_ROUTER_LOSS
    ref = harness.run_oracle(run)
    w_r, x = run.inp["w_r"].astype(np.float64), run.inp["x"].astype(np.float64)
    bw = ref["bwd"]
    part = np.linalg.norm(dl @ w_r) / np.linalg.norm(bw["dx"] + dl @ w_r)
    # without the loss's term, or with it twice, dx would be off by this share: twice the BF16 bound at least (the FP8
    # bounds of dx are wider; there dlogits and dwr, at the BF16 bound, show it)
    assert part > 2 * harness.TOL["bf16"][0], part
    bw["dlogits"], bw["dx"], bw["dwr"] = bw["dlogits"] + dl, bw["dx"] + dl @ w_r, bw["dwr"] + dl.T @ x
    harness.check_forward(run, ref)
    harness.check_backward(run, ref)


@pytest.mark.parametrize("how", ["fused", "apart", "from_x"])
@pytest.mark.parametrize("cfg", LAYERS, ids=[c.name for c in LAYERS])
def test_layer(cfg, how):
    torch, mh = _gpu()
    if how == "from_x" and (cfg.E % 32 or cfg.dtype != "bf16"):
        how = "apart"
    print(f"[router_grad] {cfg} {how}", flush=True)
    _check(*_layer(torch, mh, cfg, 0, how), mh)


@pytest.mark.parametrize("flags", [1, 2, 4, 7])
def test_layer_with_fp8_backward(flags):
    torch, mh = _gpu()
    _check(*_layer(torch, mh, LAYERS[1], flags, "fused"), mh)


def test_layer_without_tokens():
    torch, mh = _gpu()
    d = mh.make_desc(T=0, H=128, I=64, E=8, E_local=4, k=2, n_chunks=2, flags=mh.FLAG_ROUTER_LOSS)
    b = mh.allocate(d, n_segments=2)
    for name, shape in (("w1", (4, 128, 128)), ("w2", (4, 128, 64)), ("w_r", (8, 128))):
        b[name] = torch.ones(shape, dtype=torch.bfloat16, device="cuda")
    for name in ("x", "dy"):
        b[name] = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    b.update(logits=torch.empty(0, 8, device="cuda"), seg_offsets=torch.zeros(3, dtype=torch.int32, device="cuda"), balance_coef=A, z_coef=Z)
    b["router_loss"].fill_(9.0)
    mh.moe_layer_forward_backward(d, b, torch.cuda.current_stream(), torch.cuda.Stream())
    torch.cuda.synchronize()
    for name in ("router_loss", "seg_tokens", "seg_counts", "seg_probs", "dwr", "dw1", "dw2"):
        assert not b[name].float().any().item(), name


def test_layer_is_the_same_on_one_stream_and_as_stages():
    torch, mh = _gpu()
    cfg = LAYERS[1]
    names = ("router_loss", "seg_probs", "router_lse", "dlogits", "dx", "dwr", "dw1")
    run, _, _ = _layer(torch, mh, cfg, 0, "fused")
    one, _, _ = _layer(torch, mh, cfg, 0, "fused", two=False)
    apart, _, _ = _layer(torch, mh, cfg, 0, "apart")
    stages, _, _ = _layer(torch, mh, cfg, 0, "fused")
    b, d = stages.bufs, stages.desc
    for n in names:
        b[n].zero_()
    s = torch.cuda.current_stream()
    mh.moe_router_loss(d, 3, A, Z, b["logits"], b["topk_idx"], b["seg_offsets"], b["token_mask"], b["router_lse"],
                       b["seg_counts"], b["seg_tokens"], b["seg_probs"], b["router_loss"], b["loss_workspace"], s)
    mh.moe_router_loss_bwd(d, 3, A, Z, b["logits"], b["router_lse"], b["seg_offsets"], b["token_mask"], b["seg_counts"],
                           b["seg_tokens"], b["dloss"], b["dlogits"], s)
    mh.moe_combine_bwd(d, -1, b["dy"], b["yd"], b["gates"], b["row_of"], b["dyd"], b["dgates"], s)
    mh.moe_route_bwd(d, -1, b["dgates"], b["gates"], b["topk_idx"], b["x"], b["dlogits"], b["dwr_acc"], b["dwr"], b["workspace"], s)
    mh.moe_expert_ffn_bwd(d, -1, b["dyd"], b["xd"], b["gu"], b["h"], b["w1"], b["w2"], b["offsets"], b["dgu"], b["dxd"],
                          b["dw1"], b["dw2"], b["workspace"], s)
    mh.moe_dispatch_bwd(d, -1, b["dxd"], b["row_of"], b["topk_idx"], b["dlogits"], b["w_r"], b["dx"], s)
    torch.cuda.synchronize()
    for other in (one, apart, stages):
        for n in names:
            assert torch.equal(run.bufs[n], other.bufs[n]), n


def test_layer_replays_in_a_graph():
    torch, mh = _gpu()
    run, _, _ = _layer(torch, mh, LAYERS[1], 0, "fused")
    b, d = run.bufs, run.desc
    names = ("router_loss", "dlogits", "dx", "dwr", "dw1", "out")
    main, aux = torch.cuda.Stream(), torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=main):
        mh.moe_layer_forward_backward(d, b, torch.cuda.current_stream(), aux)
    x0 = b["x"].clone()
    for i in range(3):
        b["x"].copy_(x0 * (1 + i))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = {n: b[n].clone() for n in names}
        for n in names:
            b[n].fill_(3.0)
        mh.moe_layer_forward_backward(d, b, torch.cuda.current_stream(), aux)
        torch.cuda.synchronize()
        for n in names:
            assert torch.equal(got[n][:run.cfg.T] if n == "out" else got[n], b[n][:run.cfg.T] if n == "out" else b[n]), (i, n)


# Workgroups that walk many tiles (the slots' rows go round three buffers, rows and dlogits load a tile ahead), at each
# number of expert fragments, with tokens that hold more local slots than are loaded ahead; FP8 rows; FP32
@pytest.mark.parametrize("T,H,E,El,k,kind", [(16390, 2048, 128, 100, 8, "bf16"), (9001, 2112, 32, 9, 4, "bf16"), (9001, 2048, 64, 64, 8, "fp8"),
                                             (7003, 2304, 200, 150, 7, "bf16"), (5000, 2048, 260, 40, 8, "fp8"), (5005, 2048, 1000, 900, 8, "bf16"),
                                             (16390, 1088, 128, 16, 8, "f32"), (5003, 2048, 157, 157, 8, "f32")])
def test_dispatch_bwd_of_many_tiles(T, H, E, El, k, kind):
    torch, mh = _gpu()
    print(f"[router_grad] many tiles {T, H, E, El, k, kind}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(T + H + E)
    f32, f64 = torch.float32, torch.float64
    dt = f32 if kind == "f32" else torch.bfloat16
    d = mh.make_desc(T=T, H=H, I=64, E=E, E_local=El, k=k, n_chunks=1, dtype="f32" if kind == "f32" else "bf16",
                     flags=mh.FLAG_ROUTER_LOSS | (mh.FLAG_FP8_DXD if kind == "fp8" else 0))
    P, nb = d.P_c, (H + 255) // 256
    idx = torch.rand(T, E, generator=g, device="cuda").topk(k, 1).indices.to(torch.int32)
    local = idx < El
    row = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    row[local] = torch.randperm(P, generator=g, device="cuda")[:int(local.sum())].to(torch.int32)
    w = (torch.randn(E, H, generator=g, device="cuda") * 0.1).to(dt)
    dl = torch.randn(T, E, generator=g, device="cuda") * 10.0 ** (4 * torch.rand(T, 1, generator=g, device="cuda") - 3)
    val = torch.randn(P, H, generator=g, device="cuda").to(dt)
    dxd = val
    if kind == "fp8":
        codes = torch.randint(0, 127, (P, H), generator=g, device="cuda", dtype=torch.uint8)
        codes |= torch.randint(0, 2, (P, H), generator=g, device="cuda", dtype=torch.uint8) << 7
        sc = torch.rand(P, nb, generator=g, device="cuda") * 0.01 + 0.001
        val = codes.view(torch.float8_e4m3fn).to(f32) * sc.repeat_interleave(256, 1)[:, :H]
        dxd = torch.zeros(P * H * 2, dtype=torch.uint8, device="cuda")
        dxd[:P * H] = codes.reshape(-1)
        dxd[P * H:P * H + 4 * P * nb] = sc.view(torch.uint8).reshape(-1)
    dx = torch.full((T + 1, H), -5.0, dtype=dt, device="cuda")
    mh.moe_dispatch_bwd(d, -1, dxd, row, idx, dl, w, dx)
    torch.cuda.synchronize()
    want, mag = dl.to(f64) @ w.to(f64), dl.to(f64).abs() @ w.to(f64).abs()
    for j in range(k):
        part = val[row[:, j].clamp(min=0).long()].to(f64) * (row[:, j:j + 1] >= 0)
        want += part
        mag += part.abs()
    # (FP8 rows: the values above are the FP32 products that the kernel forms; one more rounding covers another order)
    lim = (E + k) * F * mag if kind == "f32" else 2.0 ** -8 * want.abs() + ((E + 2 * k) * F + 2.0 ** -17) * mag * (1 + 2.0 ** -8)
    bad = (dx[:T].to(f64) - want).abs() > lim
    assert not bad.any(), torch.nonzero(bad)[:4].tolist()
    assert (dx[T] == -5.0).all()


# FP32 in several chunks, chunks without a token, every expert local and chosen by every token
@pytest.mark.parametrize("how", ["fused", "apart"])
@pytest.mark.parametrize("cfg", [
    MoeConfig("rl_f32_n3", T=200, H=128, I=64, E=12, E_local=6, e0=3, k=3, n_chunks=3, dtype="f32", seed_base=1000, x_std=0.02, backward=True),
    MoeConfig("rl_empty_chunks", T=7, H=128, I=64, E=8, E_local=8, k=2, n_chunks=5, dtype="bf16", seed_base=1005, backward=True),
    MoeConfig("rl_all_chosen", T=260, H=192, I=128, E=8, E_local=8, k=8, n_chunks=2, dtype="bf16", seed_base=1010, backward=True),
], ids=lambda c: c.name)
def test_layer_at_the_edges(cfg, how):
    torch, mh = _gpu()
    print(f"[router_grad] {cfg} {how}", flush=True)
    _check(*_layer(torch, mh, cfg, 0, how), mh)


@pytest.mark.parametrize("delayed", ["compute", "aux"])
@pytest.mark.parametrize("flags", [0, 1 | 2 | 4])
@pytest.mark.parametrize("how", ["fused", "apart", "from_x"])
def test_layer_with_a_delay_on_one_stream(how, flags, delayed):
    """Work queued on one of the two streams in front of the call: the loss and its gradient run on either of them and
    must see every chunk's routing, and every reader of dlogits the loss's gradient."""
    torch, mh = _gpu()
    cfg = LAYERS[1]
    names = ("router_loss", "seg_counts", "seg_probs", "router_lse", "dlogits", "dx", "dwr", "dw1", "dw2")
    run, _, _ = _layer(torch, mh, cfg, flags, how)
    b, d = run.bufs, run.desc
    ref = {n: b[n].clone() for n in names}
    cs, aux = torch.cuda.current_stream(), torch.cuda.Stream()

    def delay():
        with torch.cuda.stream(cs if delayed == "compute" else aux):
            torch.cuda._sleep(2_000_000)
    for n in names + ("topk_idx", "router_logits"):
        b[n].zero_()
    torch.cuda.synchronize()
    delay()
    if how == "apart":
        mh.moe_layer_forward(d, b, cs, aux)
        delay()
        mh.moe_layer_backward(d, b, cs, aux)
    else:
        mh.moe_layer_forward_backward(d, b, cs, aux)
    torch.cuda.synchronize()
    for n in names:
        assert torch.equal(ref[n], b[n]), n
