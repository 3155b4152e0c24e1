"""GPU parity of AdamW over many tensors, the gradients' norm, the 8-bit averages and the layer's update.

Averages in 32 bits and codes in 8 are defined bit by bit (every FP32 operation rounded once) and compared as such.
Weights: from the FP32 averages, sqrt, the product with the bias correction, the sum with eps and the quotient take at
most 2^-23 each, c1 and c2 one rounding each, so the update is good to UPD = 16 2^-24 of itself; w (1 - lr wd) rounds
twice, the difference once: 3 2^-24 of the weight. A BF16 weight is the rounding of its master, or (without one) one of
the two values next to the result."""
import numpy as np
import pytest

from oracle import adamw as oa

pytestmark = pytest.mark.gpu
F = 2.0 ** -24
UPD = 16 * F
LR, B1, B2, EPS = 1e-3, 0.9, 0.95, 1e-8


def _gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import combine_moe_route_02_amd as mh
    mh.lib()
    return torch, mh


def _np(t):
    return t.detach().float().cpu().numpy()


class _Set:
    """Tensors of given sizes with averages of a run under way, on the GPU and as FP32 values."""

    def __init__(self, torch, mh, sizes, kind, gdt, bits, seed=0, fresh=False):
        rng = np.random.default_rng(seed)
        self.torch, self.mh, self.sizes, self.kind, self.bits = torch, mh, sizes, kind, bits
        wdt = torch.float32 if kind == "f32" else torch.bfloat16
        g_dt = torch.float32 if gdt == "f32" else torch.bfloat16
        self.parts, self.m0, self.v0, self.guards = [], [], [], []
        for i, n in enumerate(sizes):
            spread = np.exp(rng.standard_normal(n))
            new = lambda a, dt: self._guarded(torch.from_numpy(a.astype(np.float32)).to(dt))  # noqa: E731
            w = (rng.standard_normal(n) * 0.02).astype(np.float32)
            p = dict(grad=new(rng.standard_normal(n) * spread * 0.01, g_dt), w=new(w, wdt),
                     lr_scale=(1.0, 0.5)[i % 2], weight_decay=(0.1, 0.0, 0.03)[i % 3])
            if kind == "master":
                p["master"] = new(w, torch.float32)
                p["w"].copy_(p["master"].to(wdt))
            zero = 0.0 if fresh else 1.0
            m = (rng.standard_normal(n) * spread * 0.003 * zero).astype(np.float32)
            v = (np.square(rng.standard_normal(n) * spread) * 1e-4 * zero).astype(np.float32)
            if bits == 8:
                (mc, ms), (vc, vs) = oa.encode(m, "m"), oa.encode(v, "v")
                m, v = oa.decode(mc, ms, "m"), oa.decode(vc, vs, "v")
                p.update(m=self._guarded(torch.from_numpy(mc)), v=self._guarded(torch.from_numpy(vc)),
                         m_scale=torch.from_numpy(ms).cuda(), v_scale=torch.from_numpy(vs).cuda())
            else:
                p.update(m=new(m, torch.float32), v=new(v, torch.float32))
            self.m0.append(m)
            self.v0.append(v)
            self.parts.append(p)
        self.w0 = [_np(p.get("master") if kind == "master" else p["w"]) for p in self.parts]
        self.g = [_np(p["grad"]) for p in self.parts]
        self.table = mh.make_adamw_tensors(self.parts)

    def _guarded(self, t):
        """A view of n elements with 16 more behind, which have to stay."""
        full = self.torch.zeros(t.numel() + 16, dtype=t.dtype, device="cuda")
        full[t.numel():] = 77
        full[:t.numel()] = t.cuda()
        self.guards.append((full, t.numel()))
        return full[:t.numel()]

    def check(self, step, seed=0, scale=1.0, lr=LR):
        self.torch.cuda.synchronize()
        for full, n in self.guards:
            assert (full[n:] == 77).all()
        at = oa.places(self.sizes)
        for i, p in enumerate(self.parts):
            if self.sizes[i] == 0:
                continue
            bits, more = oa.random_bits(at[i], seed, step)
            m, v = oa.averages(self.g[i], self.m0[i], self.v0[i], B1, B2, scale)
            if self.bits == 8:
                for x, which, r in ((m, "m", bits & np.uint64(0xffff)), (v, "v", bits >> np.uint64(16))):
                    c, s = oa.encode(x, which, r)
                    np.testing.assert_array_equal(p[which].cpu().numpy(), c, err_msg=f"{which} codes of tensor {i}")
                    np.testing.assert_array_equal(p[which + "_scale"].cpu().numpy(), s)
            else:
                np.testing.assert_array_equal(_np(p["m"]), m)
                np.testing.assert_array_equal(_np(p["v"]), v)
            mine = lr * p["lr_scale"]
            w, m, v = self.w0[i].astype(np.float64), m.astype(np.float64), v.astype(np.float64)
            upd = mine / (1 - B1 ** step) * m / (np.sqrt(v / (1 - B2 ** step)) + EPS)
            want = w * (1 - mine * p["weight_decay"]) - upd
            lim = 3 * F * (np.abs(w) + np.abs(upd)) + UPD * np.abs(upd) + 2.0 ** -126
            got = _np(p["w"]).astype(np.float64)
            if self.kind == "bf16":  # one of the two neighbours of a value within lim of `want`
                step_ = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(want) + lim, 2.0 ** -126))) - 7)
                assert np.all(np.abs(got - want) <= step_ + lim)
                continue
            if self.kind == "master":
                full = p["master"]
                assert self.torch.equal(p["w"], full.to(self.torch.bfloat16))
                got = _np(full).astype(np.float64)
            bad = np.abs(got - want) > lim
            assert not bad.any(), (i, np.argwhere(bad)[:3], got[bad][:3], want[bad][:3])


SIZES = [1, 7, 8, 255, 256, 257, 2047, 2048, 2049, 5000, 0, 33333]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("gdt", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["f32", "master", "bf16"])
def test_step(kind, gdt, bits):
    torch, mh = _gpu()
    print(f"[adamw] {kind, gdt, bits}", flush=True)
    s = _Set(torch, mh, SIZES, kind, gdt, bits, seed=1)
    mh.moe_adamw_step(mh.make_adamw_options(LR, B1, B2, EPS, step=17, state_bits=bits, seed=99), s.table)
    s.check(17, 99)


@pytest.mark.parametrize("bits", [32, 8])
def test_first_step_of_a_new_run(bits):
    torch, mh = _gpu()
    s = _Set(torch, mh, [3000, 10], "master", "bf16", bits, seed=2, fresh=True)
    state = mh.adamw_state(3000, bits)
    assert all(torch.equal(state[x], s.parts[0][x]) for x in state)
    mh.moe_adamw_step(mh.make_adamw_options(LR, B1, B2, EPS, step=1, state_bits=bits), s.table)
    s.check(1)


@pytest.mark.parametrize("bits", [32, 8])
def test_more_tensors_than_a_launch_holds(bits):
    torch, mh = _gpu()
    sizes = [int(x) for x in np.random.default_rng(3).integers(1, 900, 300)]
    s = _Set(torch, mh, sizes, "f32", "bf16", bits, seed=3)
    mh.moe_adamw_step(mh.make_adamw_options(LR, B1, B2, EPS, step=5, state_bits=bits, seed=4), s.table)
    s.check(5, 4)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("count", [40, 41, 256, 257, 600])  # around what the launches hold
def test_lists_of_every_length(count, bits):
    torch, mh = _gpu()
    sizes = [int(x) for x in np.random.default_rng(count).integers(0, 600, count)]
    s = _Set(torch, mh, sizes, "master", "bf16", bits, seed=count)
    mh.moe_adamw_step(mh.make_adamw_options(LR, B1, B2, EPS, step=3, state_bits=bits, seed=6), s.table)
    s.check(3, 6)


def test_offsets_past_32_bits():
    torch, mh = _gpu()
    n = 2 ** 31 + 2048 + 3
    rng = np.random.default_rng(12)
    at = [0, 4096, 2 ** 31 - 256, n - 3 - 256]  # places of 256 elements and, at the end, three
    small = rng.standard_normal((len(at), 256)).astype(np.float32)
    g = torch.zeros(n, device="cuda", dtype=torch.bfloat16)
    for a, x in zip(at, small):
        g[a:a + 256] = torch.from_numpy(x).cuda().bfloat16()
    g[n - 3:] = 2.0
    for bits in (32, 8):
        w = torch.full((n,), 0.5, device="cuda", dtype=torch.bfloat16)
        state = mh.adamw_state(n, bits)
        table = mh.make_adamw_tensors([dict(w=w, grad=g, weight_decay=0.0, **state)])
        mh.moe_adamw_step(mh.make_adamw_options(0.125, B1, B2, EPS, step=1, state_bits=bits, seed=1), table)
        # a first step moves every weight with a gradient by lr: 0.5 +- 0.125, a BF16 value (8 bits: the codes' chance
        # is the averages', not this step's weight); neighbours by the chance of the rounding, 2^-8
        torch.cuda.synchronize()
        for a, x in zip(at, small):
            want = 0.5 - 0.125 * np.sign(g[a:a + 256].float().cpu().numpy())
            assert np.all(np.abs(w[a:a + 256].float().cpu().numpy() - want) <= 2.0 ** -8)
        assert bool(((w[n - 3:].float() - 0.375).abs() <= 2.0 ** -8).all())
        assert int((w != 0.5).sum()) == int((g != 0).sum())
        if bits == 8:
            m = state["m"]
            assert int(m[n - 1]) == 127 and int((m != 0).sum()) <= int((g != 0).sum())
            fm, fv = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
            mh.moe_adamw_unpack(n, m, state["m_scale"], state["v"], state["v_scale"], fm, fv)
            mc, vc = torch.empty_like(m), torch.empty_like(state["v"])
            ms, vs = torch.empty_like(state["m_scale"]), torch.empty_like(state["v_scale"])
            mh.moe_adamw_pack(n, fm, fv, mc, ms, vc, vs)
            torch.cuda.synchronize()
            assert abs(float(fm[n - 1]) - 0.2) <= 2.0 ** -20  # (1 - beta1) 2, its block's largest
            assert torch.equal(mc, m) and torch.equal(vc, state["v"])
        else:
            assert abs(float(state["m"][n - 1]) - 0.2) <= 2.0 ** -20
        del w, state, table
    out, ws = torch.empty(2, device="cuda"), torch.empty(mh.moe_grad_norm_bytes(), dtype=torch.uint8, device="cuda")
    mh.moe_grad_norm(mh.make_adamw_tensors([dict(grad=g)]), 1.0, out, ws)
    parts = [g[a:a + 256].double() for a in at] + [g[n - 3:].double()]
    want = float(torch.cat(parts).norm())
    assert abs(float(out[0]) - want) <= 2 * F * want


def test_tensors_of_every_kind_in_one_call():
    """Places run through the whole list, whatever kinds its tensors are; the order of the weights does not matter."""
    torch, mh = _gpu()
    sets = [_Set(torch, mh, [300, 41], k, g, 8, seed=i) for i, (k, g) in enumerate((k, g) for k in ("f32", "master", "bf16") for g in ("f32", "bf16"))]
    parts = [p for s in reversed(sets) for p in s.parts]
    whole = sets[0]
    mh.moe_adamw_step(mh.make_adamw_options(LR, B1, B2, EPS, step=9, state_bits=8, seed=1), mh.make_adamw_tensors(parts))
    torch.cuda.synchronize()
    at = oa.places([p["grad"].numel() for p in parts])
    i = 0
    for s in reversed(sets):
        for j, p in enumerate(s.parts):
            bits, _ = oa.random_bits(at[i], 1, 9)
            m, v = oa.averages(s.g[j], s.m0[j], s.v0[j], B1, B2)
            np.testing.assert_array_equal(p["m"].cpu().numpy(), oa.encode(m, "m", bits & np.uint64(0xffff))[0])
            np.testing.assert_array_equal(p["v"].cpu().numpy(), oa.encode(v, "v", bits >> np.uint64(16))[0])
            i += 1
    assert whole.kind == "f32"


def test_bf16_weights_move_as_far_as_fp32_ones():
    """Updates far below a BF16 step: the mean over many equal weights is that of FP32 ones. Every weight moves up one
    step with the chance of its part; the mean of n has a deviation of at most half a step / sqrt(n); 6 of these."""
    torch, mh = _gpu()
    n = 1 << 18
    p = dict(grad=torch.full((n,), 1.0, device="cuda"), w=torch.full((n,), 0.75, dtype=torch.bfloat16, device="cuda"), **mh.adamw_state(n))
    t = mh.make_adamw_tensors([p])
    for step in range(1, 21):
        mh.moe_adamw_step(mh.make_adamw_options(1e-5, B1, B2, EPS, step=step, seed=3), t)
    mean = float(p["w"].double().mean())
    assert abs(mean - (0.75 - 20e-5)) <= 6 * 0.5 * 2.0 ** -8 * np.sqrt(20 / n) + 20 * 2.0 ** -24 + 20 * 2.0 ** -8 * 2.0 ** -16
    assert len(torch.unique(p["w"])) > 1


def test_8_bit_averages_follow_fp32_ones():
    """v of a constant gradient, from zero: 1 - b2^t of g^2 after t steps. One step's rounding has a deviation of at most half
    a gap of codes (gap <= 4 / 255 of the value at the top codes), kept with a factor b2 per step: sqrt(1 / (1 - b2^2)) = 3.2
    of it in the end, averaged over n elements."""
    torch, mh = _gpu()
    n = 1 << 16
    g = torch.full((n,), 0.5, device="cuda")
    g[::256] = 1.0
    p = dict(grad=g, w=torch.zeros(n, device="cuda"), **mh.adamw_state(n, 8))
    t = mh.make_adamw_tensors([p])
    for step in range(1, 41):
        mh.moe_adamw_step(mh.make_adamw_options(0.0, B1, B2, EPS, step=step, state_bits=8, seed=5), t)
    m, v = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    mh.moe_adamw_unpack(n, p["m"], p["m_scale"], p["v"], p["v_scale"], m, v)
    keep = torch.arange(n, device="cuda") % 256 != 0
    for x, beta, want in ((m, B1, 0.5 * (1 - B1 ** 40)), (v, B2, 0.25 * (1 - B2 ** 40))):
        got = float(x[keep].double().mean())
        assert abs(got - want) <= want * (6 * 0.5 * 4 / 127 * 3.2 / np.sqrt(n) + 40 * 2.0 ** -16 * 4 / 127 + 40 * 2.0 ** -22)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("kind", ["f32", "master", "bf16"])
def test_gradients_that_are_not_finite_stay_where_they_are(kind, bits):
    torch, mh = _gpu()
    s = _Set(torch, mh, [1000], kind, "f32", bits, seed=6)
    p = s.parts[0]
    p["grad"][5], p["grad"][300], p["grad"][999] = float("nan"), float("inf"), 3e38
    before = p["w"].clone()
    mh.moe_adamw_step(mh.make_adamw_options(LR, B1, B2, EPS, step=3, state_bits=bits), s.table)
    torch.cuda.synchronize()
    w = p["w"].float()
    assert torch.isnan(w[5]) and torch.isnan(w[300])
    others = torch.ones(1000, dtype=torch.bool, device="cuda")
    others[[5, 300, 999]] = False
    assert torch.isfinite(w[others]).all()
    assert (w[999] - before[999].float()).abs() <= 2.0 ** -7 * before[999].abs().float() + 1e-30 or kind != "bf16"
    if bits == 8:  # a block with NaN or infinity stays NaN as a whole, the others do not
        m, v = torch.empty(1000, device="cuda"), torch.empty(1000, device="cuda")
        mh.moe_adamw_unpack(1000, p["m"], p["m_scale"], p["v"], p["v_scale"], m, v)
        for x in (m, v):
            assert torch.isnan(x[:512]).all() and torch.isfinite(x[512:768]).all()
        assert torch.isnan(v[768:]).all()  # (3e38)^2


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("kind", ["f32", "master", "bf16"])
def test_a_square_past_fp32_moves_nothing_but_the_decay(kind, bits):
    """v' is infinite, the update 0: w (1 - lr wd) is left, two roundings of FP32, and in BF16 one of the two neighbours."""
    torch, mh = _gpu()
    s = _Set(torch, mh, [1000], kind, "f32", bits, seed=6)
    p = s.parts[0]
    p["grad"][999] = 3e38
    mh.moe_adamw_step(mh.make_adamw_options(LR, B1, B2, EPS, step=3, state_bits=bits), s.table)
    torch.cuda.synchronize()
    want = float(s.w0[0][999]) * (1 - LR * p["lr_scale"] * p["weight_decay"])
    got = float(_np(p["master"] if kind == "master" else p["w"])[999])
    assert abs(got - want) <= (2.0 ** -7 if kind == "bf16" else 2 * F) * abs(want)
    if kind == "master":
        assert torch.equal(p["w"], p["master"].to(torch.bfloat16))


def test_a_scale_that_is_not_finite_leaves_everything():
    torch, mh = _gpu()
    for bits in (32, 8):
        s = _Set(torch, mh, [1000, 300], "master", "bf16", bits, seed=7)
        before = [{k: v.clone() for k, v in p.items() if hasattr(v, "clone")} for p in s.parts]
        for bad in ("nan", "inf", "-inf"):
            f = torch.tensor([float(bad)], device="cuda")
            mh.moe_adamw_step(mh.make_adamw_options(LR, B1, B2, EPS, step=3, state_bits=bits, grad_scale=f), s.table)
            torch.cuda.synchronize()
            for p, q in zip(s.parts, before):
                assert all(torch.equal(p[k], q[k]) for k in q)


# ------------------------------------------------------------------ norm

@pytest.mark.parametrize("sizes,gdt", [([1], "f32"), (SIZES, "bf16"), ([300] * 100, "f32"), ([5_000_003, 17], "bf16"),
                                       ([300, 9000] * 150, "f32"), (list(range(1, 700)), "bf16")])
def test_norm(sizes, gdt):
    torch, mh = _gpu()
    print(f"[adamw] norm {len(sizes), gdt}", flush=True)
    rng = np.random.default_rng(9)
    dt = torch.float32 if gdt == "f32" else torch.bfloat16
    grads = [torch.from_numpy((rng.standard_normal(n) * 10.0 ** rng.uniform(-9, 3)).astype(np.float32)).cuda().to(dt) for n in sizes]
    t = mh.make_adamw_tensors([dict(grad=g) for g in grads])
    want = float(np.sqrt(sum(float((g.double() ** 2).sum()) for g in grads)))
    out, ws = torch.empty(3, device="cuda").fill_(5), torch.empty(mh.moe_grad_norm_bytes(), dtype=torch.uint8, device="cuda").fill_(0xff)
    for max_norm in (want * 0.25, want * 2, float("inf")):
        mh.moe_grad_norm(t, max_norm, out, ws)
        norm, factor, guard = out.cpu().tolist()
        assert abs(norm - want) <= 2 * F * want
        assert abs(factor - min(1.0, max_norm / want)) <= 2 * F and guard == 5.0
    first = out.clone()
    for _ in range(3):
        mh.moe_grad_norm(t, float("inf"), out, ws)
        assert torch.equal(first, out)


def test_norm_of_mixed_types_and_of_nothing():
    torch, mh = _gpu()
    out, ws = torch.empty(2, device="cuda"), torch.empty(mh.moe_grad_norm_bytes(), dtype=torch.uint8, device="cuda").fill_(0xff)
    a, b = torch.full((10,), 3.0, device="cuda"), torch.full((10,), 4.0, device="cuda", dtype=torch.bfloat16)
    mh.moe_grad_norm(mh.make_adamw_tensors([dict(grad=a), dict(grad=b), dict(grad=a)] * 40), 1.0, out, ws)
    want = np.sqrt(40 * (20 * 9.0 + 10 * 16.0))
    np.testing.assert_allclose(out.cpu().numpy(), [want, 1 / want], rtol=2 * F)
    mh.moe_grad_norm(mh.make_adamw_tensors([]), 1.0, out, ws)
    assert out.cpu().tolist() == [0.0, 1.0]
    mh.moe_grad_norm(mh.make_adamw_tensors([dict(grad=a[:0])]), 1.0, out, ws)
    assert out.cpu().tolist() == [0.0, 1.0]
    for bad, norm in ((float("nan"), np.nan), (float("inf"), np.inf)):
        a[3] = bad
        mh.moe_grad_norm(mh.make_adamw_tensors([dict(grad=a)]), 1.0, out, ws)
        got = out.cpu().numpy()
        assert np.isnan(got[1]) and np.array_equal(got[:1], [norm], equal_nan=True)
    big = torch.full((5,), 3e38, device="cuda")  # squares past FP32's range, a norm past it too
    mh.moe_grad_norm(mh.make_adamw_tensors([dict(grad=big)]), 1.0, out, ws)
    assert np.isinf(out.cpu().numpy()[0]) and np.isnan(out.cpu().numpy()[1])
    mh.moe_grad_norm(mh.make_adamw_tensors([dict(grad=big[:1])]), 1.0, out, ws)
    np.testing.assert_allclose(out.cpu().numpy(), [np.float32(3e38), 1 / np.float64(np.float32(3e38))], rtol=2 * F)


@pytest.mark.parametrize("gdt", ["f32", "bf16"])
@pytest.mark.parametrize("sizes,value", [([1], 3e38), ([1000], 1e25), ([5000, 3], 2e19), ([1000, 70], 1e-25), ([9], 2.0 ** -126), ([300] * 50, 3e-22)])
def test_norm_of_gradients_whose_squares_leave_fp32(sizes, value, gdt):
    """The sum is FP64 throughout: the norm is good to its own rounding, 2^-24, and the sums' far smaller ones."""
    torch, mh = _gpu()
    dt = torch.float32 if gdt == "f32" else torch.bfloat16
    grads = [torch.full((n,), value, device="cuda").to(dt) for n in sizes]
    want = float(grads[0][0]) * np.sqrt(sum(sizes))
    out, ws = torch.empty(2, device="cuda"), torch.empty(mh.moe_grad_norm_bytes(), dtype=torch.uint8, device="cuda")
    mh.moe_grad_norm(mh.make_adamw_tensors([dict(grad=g) for g in grads]), want * 0.25, out, ws)
    norm, factor = out.cpu().tolist()
    assert abs(norm - want) <= 2 * F * want and abs(factor - 0.25) <= 2 * F


@pytest.mark.parametrize("bits", [32, 8])
def test_clipped_step(bits):
    torch, mh = _gpu()
    s = _Set(torch, mh, [4000, 123], "master", "bf16", bits, seed=12)
    out, ws = torch.empty(2, device="cuda"), torch.empty(mh.moe_grad_norm_bytes(), dtype=torch.uint8, device="cuda")
    mh.moe_grad_norm(s.table, 0.01, out, ws)
    mh.moe_adamw_step(mh.make_adamw_options(LR, B1, B2, EPS, step=4, state_bits=bits, grad_scale=out[1:]), s.table)
    scale = float(out[1])
    assert scale < 0.5
    s.check(4, 0, scale)


# ------------------------------------------------------------------ pack and unpack

@pytest.mark.parametrize("n", [1, 255, 256, 257, 2048, 10_001])
def test_pack_and_unpack(n):
    torch, mh = _gpu()
    rng = np.random.default_rng(n)
    m = (rng.standard_normal(n) * np.exp(3 * rng.standard_normal(n))).astype(np.float32)
    v = (m * rng.standard_normal(n)).astype(np.float32) ** 2
    m[::5] = 0
    if n > 600:
        m[256:512], v[256:512] = 0, 2.0 ** -122
    mc, vc = torch.full((n + 3,), 55, dtype=torch.int8, device="cuda"), torch.full((n + 3,), 55, dtype=torch.uint8, device="cuda")
    ms, vs = torch.empty((n + 255) // 256, device="cuda"), torch.empty((n + 255) // 256, device="cuda")
    mh.moe_adamw_pack(n, torch.from_numpy(m).cuda(), torch.from_numpy(v).cuda(), mc, ms, vc, vs)
    for c, s, x, which in ((mc, ms, m, "m"), (vc, vs, v, "v")):
        want, ws = oa.encode(x, which)
        np.testing.assert_array_equal(c.cpu().numpy()[:n], want)
        np.testing.assert_array_equal(s.cpu().numpy(), ws)
        assert (c[n:] == 55).all()
    fm, fv = torch.full((n + 3,), 5.0, device="cuda"), torch.full((n + 3,), 5.0, device="cuda")
    mh.moe_adamw_unpack(n, mc, ms, vc, vs, fm, fv)
    np.testing.assert_array_equal(fm.cpu().numpy()[:n], oa.decode(mc.cpu().numpy()[:n], ms.cpu().numpy(), "m"))
    np.testing.assert_array_equal(fv.cpu().numpy()[:n], oa.decode(vc.cpu().numpy()[:n], vs.cpu().numpy(), "v"))
    assert (fm[n:] == 5.0).all() and (fv[n:] == 5.0).all()


def test_pack_of_negative_zeros():
    """A second average of -0 counts as 0, also beside its block's largest."""
    torch, mh = _gpu()
    n = 1000
    v = np.square(np.random.default_rng(3).standard_normal(n)).astype(np.float32)
    v[1::4] = -0.0
    v[[2, 258, 514, 770]] = 50.0
    mc, vc = torch.empty(n, dtype=torch.int8, device="cuda"), torch.empty(n, dtype=torch.uint8, device="cuda")
    ms, vs = torch.empty(4, device="cuda"), torch.empty(4, device="cuda")
    mh.moe_adamw_pack(n, torch.from_numpy(-v).cuda(), torch.from_numpy(v).cuda(), mc, ms, vc, vs)
    for c, s, x, which in ((mc, ms, -v, "m"), (vc, vs, v, "v")):
        want, ws = oa.encode(x, which)
        np.testing.assert_array_equal(s.cpu().numpy(), ws)
        np.testing.assert_array_equal(c.cpu().numpy(), want)


def test_every_code_stands_for_itself():
    """All levels, and values between them on both sides of each middle, as one block's shares of 1."""
    torch, mh = _gpu()
    for which in ("m", "v"):
        lev = oa.levels(which).astype(np.float64)
        x = [1.0]
        for lo, hi in zip(lev[:-1], lev[1:]):
            x += [lo, np.nextafter(np.float32(lo), np.float32(2)), 0.501 * lo + 0.499 * hi, 0.499 * lo + 0.501 * hi, np.nextafter(np.float32(hi), np.float32(0))]
        x = np.array(x, dtype=np.float32)
        blocks = -(-x.size // 255)
        full = np.zeros((blocks, 256), dtype=np.float32)
        full[:, 0] = 1.0
        full[:, 1:].reshape(-1)[:0]
        flat = np.zeros(blocks * 255, dtype=np.float32)
        flat[:x.size] = x
        full[:, 1:] = flat.reshape(blocks, 255)
        full = full.reshape(-1)
        n = full.size
        mc, vc = torch.empty(n, dtype=torch.int8, device="cuda"), torch.empty(n, dtype=torch.uint8, device="cuda")
        ms, vs = torch.empty(blocks, device="cuda"), torch.empty(blocks, device="cuda")
        dev = torch.from_numpy(full).cuda()
        mh.moe_adamw_pack(n, dev, dev, mc, ms, vc, vs)
        got = (mc if which == "m" else vc).cpu().numpy()
        np.testing.assert_array_equal(got, oa.encode(full, which)[0])
        mh.moe_adamw_pack(n, -dev, dev, mc, ms, vc, vs)
        np.testing.assert_array_equal(mc.cpu().numpy(), oa.encode(-full, "m")[0])


# ------------------------------------------------------------------ streams, graphs, the layer

@pytest.mark.parametrize("bits", [32, 8])
def test_long_lists_replay_from_a_graph(bits):
    """More tensors than the short argument list and than a launch holds, captured; the table is gone before the replays."""
    torch, mh = _gpu()
    sizes = [int(x) for x in np.random.default_rng(21).integers(0, 900, 300)]
    a, b = (_Set(torch, mh, sizes, "master", "bf16", bits, seed=22) for _ in range(2))
    step = torch.ones(1, dtype=torch.int64, device="cuda")
    norm, ws = torch.empty(2, device="cuda"), torch.empty(mh.moe_grad_norm_bytes(), dtype=torch.uint8, device="cuda")
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        table = mh.make_adamw_tensors(a.parts)
        mh.moe_grad_norm(table, 0.05, norm, ws)
        mh.moe_adamw_step(mh.make_adamw_options(LR, B1, B2, EPS, state_bits=bits, seed=2, step_dev=step, grad_scale=norm[1:]), table)
        for row in table.table:
            row.n = row.w = row.grad = 0
    norm2, ws2 = torch.empty(2, device="cuda"), torch.empty_like(ws)
    for i in range(1, 4):
        for p, q in zip(a.parts, b.parts):
            p["grad"].mul_(1.5)
            q["grad"].mul_(1.5)
        step.fill_(i)
        torch.cuda.synchronize()
        g.replay()
        mh.moe_grad_norm(b.table, 0.05, norm2, ws2)
        mh.moe_adamw_step(mh.make_adamw_options(LR, B1, B2, EPS, step=i, state_bits=bits, seed=2, grad_scale=norm2[1:]), b.table)
        torch.cuda.synchronize()
        assert torch.equal(norm, norm2)
        for p, q in zip(a.parts, b.parts):
            for name in ("w", "master", "m", "v") + (("m_scale", "v_scale") if bits == 8 else ()):
                assert torch.equal(p[name], q[name]), (i, name)


@pytest.mark.parametrize("bits", [32, 8])
def test_replayed_with_step_and_rate_on_the_device(bits):
    torch, mh = _gpu()
    a, b = (_Set(torch, mh, [5000, 77], "bf16", "bf16", bits, seed=13) for _ in range(2))
    step, lr = torch.ones(1, dtype=torch.int64, device="cuda"), torch.full((1,), LR, dtype=torch.float64, device="cuda")
    norm, ws = torch.empty(2, device="cuda"), torch.empty(mh.moe_grad_norm_bytes(), dtype=torch.uint8, device="cuda")
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        mh.moe_grad_norm(a.table, 0.05, norm, ws)
        mh.moe_adamw_step(mh.make_adamw_options(9.0, B1, B2, EPS, state_bits=bits, seed=2, step_dev=step, lr_dev=lr, grad_scale=norm[1:]), a.table)
    norm2, ws2 = torch.empty(2, device="cuda"), torch.empty_like(ws)
    for i in range(1, 5):
        for s in (a, b):
            for p in s.parts:
                p["grad"].copy_(torch.randn(p["grad"].shape, generator=torch.Generator("cuda").manual_seed(i), device="cuda") * i)
        step.fill_(i)
        lr.fill_(LR / i)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        mh.moe_grad_norm(b.table, 0.05, norm2, ws2)
        mh.moe_adamw_step(mh.make_adamw_options(LR / i, B1, B2, EPS, step=i, state_bits=bits, seed=2, grad_scale=norm2[1:]), b.table)
        torch.cuda.synchronize()
        assert torch.equal(norm, norm2)
        for p, q in zip(a.parts, b.parts):
            for k in ("m", "v") + (("m_scale", "v_scale") if bits == 8 else ()):
                assert torch.equal(p[k], q[k]), (i, k)
            # the bias corrections come from two libraries' logarithms: a last bit of c1 may move a rounding
            assert float((p["w"].float() - q["w"].float()).abs().max()) <= 2.0 ** -7 * float(q["w"].float().abs().max())
            p["w"].copy_(q["w"])


def test_on_another_stream():
    torch, mh = _gpu()
    s = _Set(torch, mh, [30000], "f32", "f32", 8, seed=14)
    g = s.parts[0]["grad"].clone()
    s.parts[0]["grad"].zero_()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(1_000_000)
        s.parts[0]["grad"].copy_(g)
        mh.moe_adamw_step(mh.make_adamw_options(LR, B1, B2, EPS, step=2, state_bits=8), s.table)
    s.check(2)


@pytest.mark.parametrize("bits,master,clip", [(32, True, True), (8, True, False), (8, False, True)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layer_update(dtype, bits, master, clip):
    """Forward, backward and update of a layer for three steps: the update is AdamW and the bias update on the layer's
    own buffers, and the next forward runs on what it wrote."""
    torch, mh = _gpu()
    from oracle import router_scores as ors
    print(f"[adamw] layer {dtype, bits, master, clip}", flush=True)
    T, H, I, E, El, k, n = 300, 128, 64, 16, 4, 2, 2
    d = mh.make_desc(T=T, H=H, I=I, E=E, E_local=El, k=k, n_chunks=n, dtype=dtype, flags=mh.FLAG_ROUTER_SCORES)
    b = mh.allocate(d)
    gen = torch.Generator("cuda").manual_seed(1)
    pay = torch.float32 if dtype == "f32" else torch.bfloat16
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    b.update(x=rand(T, H).to(pay), dy=rand(T, H).to(pay), w1=(rand(El, 2 * I, H) * 0.05).to(pay), w2=(rand(El, H, I) * 0.05).to(pay),
             w_r=(rand(E, H) * 0.05).to(pay), logits=rand(T, E), router_bias=torch.zeros(E, device="cuda"),
             router_scores=mh.make_router_scores("sigmoid", 4, 2, 2))
    o = mh.make_layer_optimizer(d, b, mh.make_adamw_options(LR, B1, B2, EPS, state_bits=bits, seed=6), master=master,
                                weight_decay=0.1, max_norm=0.5 if clip else None, bias_rate=0.01)
    twin = {f: b[f].clone() for f in ("w1", "w2", "w_r")}
    ref = mh.make_layer_optimizer(d, twin, mh.make_adamw_options(LR, B1, B2, EPS, state_bits=bits, seed=6), master=master,
                                  weight_decay=0.1, max_norm=0.5 if clip else None)
    cs, aux = torch.cuda.current_stream(), torch.cuda.Stream()
    for step in range(1, 4):
        b["logits"] = (b["x"].float() @ b["w_r"].float().t()).contiguous()
        mh.moe_layer_forward_backward(d, b, cs, aux)
        bias = b["router_bias"].cpu().numpy().copy()
        o.adamw.step = step
        mh.moe_layer_update(d, b, o)
        torch.cuda.synchronize()
        np.testing.assert_array_equal(b["router_bias"].cpu().numpy(), ors.bias_update(bias, b["counts"].cpu().numpy(), 0.01))
        parts = []
        for f, g in (("w1", "dw1"), ("w2", "dw2"), ("w_r", "dwr")):
            parts.append(dict(w=twin[f], grad=b[g], weight_decay=0.0 if f == "w_r" else 0.1, **ref.buffers[f]))
        t = mh.make_adamw_tensors(parts)
        opt = mh.make_adamw_options(LR, B1, B2, EPS, step=step, state_bits=bits, seed=6)
        if clip:
            mh.moe_grad_norm(t, 0.5, ref.buffers["norm"], ref.buffers["norm_workspace"])
            assert torch.equal(o.buffers["norm"], ref.buffers["norm"]) and float(o.buffers["norm"][1]) < 1
            opt = mh.make_adamw_options(LR, B1, B2, EPS, step=step, state_bits=bits, seed=6, grad_scale=ref.buffers["norm"][1:])
        before = {f: twin[f].clone() for f in twin}
        mh.moe_adamw_step(opt, t)
        torch.cuda.synchronize()
        for f in twin:
            assert torch.equal(b[f], twin[f]), f
            assert not torch.equal(before[f], twin[f]), f
            assert all(torch.equal(o.buffers[f][x], ref.buffers[f][x]) for x in o.buffers[f]), f


def _training_layer(torch, mh, bits, step):
    """A layer that routes from x by scores, with its optimizer; the step number on the device."""
    d = mh.make_desc(T=500, H=128, I=64, E=32, E_local=8, k=4, n_chunks=2, dtype="bf16", flags=mh.FLAG_ROUTER_SCORES)
    b = mh.allocate(d)
    gen = torch.Generator("cuda").manual_seed(3)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    b.update(x=rand(500, 128), dy=rand(500, 128), w1=rand(8, 128, 128) * 0.05, w2=rand(8, 128, 64) * 0.05, w_r=rand(32, 128) * 0.05,
             logits=None, router_bias=torch.zeros(32, device="cuda"), router_scores=mh.make_router_scores("sigmoid", 8, 4, 2))
    opt = mh.make_adamw_options(LR, B1, B2, EPS, state_bits=bits, seed=8, step_dev=step)
    return d, b, mh.make_layer_optimizer(d, b, opt, weight_decay=0.1, max_norm=0.5, bias_rate=0.01)


@pytest.mark.parametrize("bits", [32, 8])
def test_a_captured_training_step_replays(bits):
    torch, mh = _gpu()
    step, step2 = (torch.zeros(1, dtype=torch.int64, device="cuda") for _ in range(2))
    d, b, o = _training_layer(torch, mh, bits, step)
    _, b2, o2 = _training_layer(torch, mh, bits, step2)
    main, aux, aux2 = (torch.cuda.Stream() for _ in range(3))

    def run(bufs, optimizer, number, side):
        number.add_(1)
        mh.moe_layer_forward_backward(d, bufs, torch.cuda.current_stream(), side)
        mh.moe_layer_update(d, bufs, optimizer)

    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=main):
        run(b, o, step, aux)
    start = b["w1"].clone()
    for i in range(4):
        for bufs in (b, b2):
            bufs["x"].copy_(torch.randn(500, 128, generator=torch.Generator("cuda").manual_seed(i), device="cuda"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        run(b2, o2, step2, aux2)
        torch.cuda.synchronize()
        for f in ("w1", "w2", "w_r", "router_bias", "counts", "topk_idx"):
            assert torch.equal(b[f], b2[f]), (i, f)
        for f in ("w1", "w2", "w_r"):
            assert all(torch.equal(o.buffers[f][x], o2.buffers[f][x]) for x in o.buffers[f]), (i, f)
        assert torch.equal(o.buffers["norm"], o2.buffers["norm"])
    assert int(step) == 4 and not torch.equal(start, b["w1"])


def test_two_updates_at_once():
    torch, mh = _gpu()
    pair = [[_Set(torch, mh, [40_000, 999, 3], "master", "bf16", bits, seed=bits) for bits in (32, 8)] for _ in range(2)]
    norms = [torch.empty(2, device="cuda") for _ in range(4)]
    wss = [torch.empty(mh.moe_grad_norm_bytes(), dtype=torch.uint8, device="cuda") for _ in range(4)]

    def run(s, norm, ws):
        mh.moe_grad_norm(s.table, 0.5, norm, ws)
        mh.moe_adamw_step(mh.make_adamw_options(LR, B1, B2, EPS, step=2, state_bits=s.bits, seed=1, grad_scale=norm[1:]), s.table)

    for s, norm, ws in zip(pair[0], norms, wss):  # one after the other
        run(s, norm, ws)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for stream, s, norm, ws in zip(streams, pair[1], norms[2:], wss[2:]):  # side by side
        with torch.cuda.stream(stream):
            run(s, norm, ws)
    torch.cuda.synchronize()
    for a, b in zip(*pair):
        for p, q in zip(a.parts, b.parts):
            for f in p:
                if torch.is_tensor(p[f]):
                    assert torch.equal(p[f], q[f]), f
