"""GPU parity of the 8-bit integer path against the NumPy oracle.

Codes and scales are compared bit for bit (both sides take the same FP32 steps); so are products of the same codes
computed by different calls, since the sums are exact. A product's value is an exact integer, rounded once to FP32
(2^-24), times the rounded product of two scales (two more), rounded once to BF16: 2^-8 of the value plus 3 * 2^-24.
The layer's output differs from the oracle's by the rounding of yd (2^-9 / sqrt(3) rms at most) and the BF16 rounding of
out (2^-8 / sqrt(3)), together under the 2^-8 sqrt(2 / 3) of two BF16 roundings that the bound allows, and by codes of h that fall on the other side of a half because h carries FP32 rounding (a relative 1e-6 moves a share
2e-6 / step of the codes, under 1e-3 of the norm): 2^-8 * sqrt(2 / 3) + 1e-3 = 4.2e-3 of the norm."""
import numpy as np
import pytest

import moe_inputs
import oracle
from moe_inputs import MoeConfig
from oracle import int8 as oi8

pytestmark = pytest.mark.gpu
harness = pytest.importorskip("harness")
OUT_TOL = 4.2e-3
MM_TOL = 2.0 ** -8 + 3 * 2.0 ** -24


def _gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import combine_moe_route_02_amd as mh
    mh.lib()
    return torch, mh


def _bf16(torch, a):
    """FP32 values -> device BF16 tensor and the rounded values."""
    bits = moe_inputs.f32_to_bf16_bits(a)
    return torch.from_numpy(bits.view(np.int16)).cuda().view(torch.bfloat16), moe_inputs.bf16_bits_to_f32(bits)


@pytest.mark.parametrize("rows,cols", [(1, 8), (3, 64), (5, 520), (17, 1024), (64, 2048), (7, 4104), (9, 8192), (3, 8200), (2, 20000)])
def test_quantize_rows_bitwise(rows, cols):
    torch, mh = _gpu()
    rng = np.random.default_rng(rows * cols)
    a = rng.standard_normal((rows, cols)).astype(np.float32)
    if rows > 2:
        a[1] = 0.0
        a[2] *= 1e-39           # the multiplier overflows
    if rows > 6:
        a[3, 5], a[4, 6], a[5, 7] = np.nan, np.inf, -np.inf
        a[6] = 1.5              # all equal
    dev, val = _bf16(torch, a)
    codes = torch.full((rows, cols), 77, dtype=torch.int8, device="cuda")
    scale = torch.full((rows,), 7.0, device="cuda")
    mh.moe_quantize_rows_i8(rows, cols, dev, codes, scale)
    torch.cuda.synchronize()
    q, s = oi8.quantize_rows(val)
    np.testing.assert_array_equal(codes.cpu().numpy(), q)
    np.testing.assert_array_equal(scale.cpu().numpy(), s)


def _product(torch, mh, rows, N, K, G, off, seed, lo=-127):
    rng = np.random.default_rng(seed)
    x, w = rng.integers(lo, 128, (rows, K)).astype(np.int8), rng.integers(lo, 128, (G, N, K)).astype(np.int8)
    xs, ws = (rng.random(rows) + 0.1).astype(np.float32), (rng.random((G, N)) + 0.1).astype(np.float32)
    y = torch.full((rows, N), -3.0, dtype=torch.bfloat16, device="cuda")
    off_d = None if off is None else torch.tensor(off, dtype=torch.int32, device="cuda")
    mh.moe_expert_matmul_i8(G, rows, N, K, torch.from_numpy(x).cuda(), torch.from_numpy(xs).cuda(), torch.from_numpy(w).cuda(),
                            torch.from_numpy(ws).cuda(), off_d, y)
    torch.cuda.synchronize()
    return y.float().cpu().numpy().astype(np.float64), oi8.matmul(x, xs, w, ws, off)


def _assert_product(got, want):
    out = np.isnan(want)
    assert np.all(got[out] == -3.0), "a row outside every group was written"
    assert np.all(np.abs(got - want)[~out] <= MM_TOL * np.abs(want[~out]))


# rows around every row tile, columns and K that end inside a tile
@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 31, 33, 64, 65, 100, 129, 300])
@pytest.mark.parametrize("N,K", [(8, 64), (72, 192), (256, 128), (520, 1088), (128, 2048)])
def test_dense_product(rows, N, K):
    torch, mh = _gpu()
    _assert_product(*_product(torch, mh, rows, N, K, 1, None, rows + N + K))


@pytest.mark.parametrize("off", [
    [0, 0, 5, 5, 40], [3, 3, 3, 3, 3], [2, 19, 20, 36, 37],   # empty groups, rows in no group
    [0, 1, 2, 3, 4], [0, 300, 300, 301, 700], [-5, 10, 2000, 2000, 9999],
])
@pytest.mark.parametrize("N,K", [(64, 64), (200, 320)])
def test_grouped_product(off, N, K):
    torch, mh = _gpu()
    rows = 40 if max(off) <= 40 else 700
    _assert_product(*_product(torch, mh, rows, N, K, 4, off, len(off) + N))


# More tiles than CUs, so that workgroups run several tiles in a row: one, two, three and four stages of K, a last
# row tile of few rows and a last column tile of 8 columns
@pytest.mark.parametrize("rows,N,K", [(4400, 4616, 64), (4400, 4616, 128), (4500, 4616, 192), (4608, 4616, 256)])
def test_many_tiles_per_workgroup(rows, N, K):
    torch, mh = _gpu()
    _assert_product(*_product(torch, mh, rows, N, K, 1, None, K))


# Small tiles (128 x 128): rows past a few tiles, and tiles enough for two rounds with fewer stages than a tile's loads
# run ahead
@pytest.mark.parametrize("rows", [130, 200, 321, 513, 1025])
@pytest.mark.parametrize("N,K", [(8, 64), (520, 192), (1032, 1088), (264, 2112)])
def test_dense_product_of_many_rows(rows, N, K):
    torch, mh = _gpu()
    _assert_product(*_product(torch, mh, rows, N, K, 1, None, rows + N + K))


@pytest.mark.parametrize("K", [64, 128, 192, 256, 320, 384, 448, 576])
def test_small_tiles_in_a_row(K):
    torch, mh = _gpu()
    _assert_product(*_product(torch, mh, 2007, 2312, K, 1, None, K))


# Few rows per group: whole K per wave (128 groups on 256 columns), halves of it (on 128), quarters; more groups than a
# workgroup has threads, most of them empty; groups of more rows than a pass holds
@pytest.mark.parametrize("G,N,K,low,high", [(128, 256, 320, 0, 9), (128, 136, 192, 0, 9), (128, 256, 64, 3, 4), (64, 128, 448, 0, 33),
                                            (600, 72, 128, 0, 2), (16, 512, 320, 10, 40), (16, 512, 320, 20, 140),
                                            (4, 200, 192, 60, 130), (2, 520, 1088, 100, 128), (2, 520, 192, 60, 96),
                                            (300, 64, 576, 20, 60), (80, 56, 1088, 30, 70)])
def test_few_rows_of_many_groups(G, N, K, low, high):
    torch, mh = _gpu()
    rng = np.random.default_rng(G + N + K)
    lens = rng.integers(low, high, G)
    if G == 600:
        lens *= rng.integers(0, 12, G) == 0
    if G == 16:
        lens[5] = 300 if high > 100 else 200
    off = [3] + list(3 + np.cumsum(lens))
    _assert_product(*_product(torch, mh, int(off[-1]) + 5, N, K, G, off, 17))


def test_many_uneven_groups():
    """Sixty groups of 0 to 900 rows: large and small row tiles of many groups, several per workgroup."""
    torch, mh = _gpu()
    rng = np.random.default_rng(12)
    lens = rng.integers(0, 900, 60)
    lens[[3, 17, 59]] = 0
    lens[[4, 30]] = [256, 1]
    off = [7] + list(7 + np.cumsum(lens))
    _assert_product(*_product(torch, mh, int(off[-1]) + 9, 264, 192, 60, off, 13))


def test_product_of_the_extreme_codes():
    """-128 everywhere at a long K: the int32 sum is 2^14 K."""
    torch, mh = _gpu()
    for rows in (1, 40, 300):
        K, N = 65536, 16
        x = torch.full((rows, K), -128, dtype=torch.int8, device="cuda")
        w = torch.full((1, N, K), -128, dtype=torch.int8, device="cuda")
        y = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")
        one = torch.ones(max(rows, N), device="cuda")
        mh.moe_expert_matmul_i8(1, rows, N, K, x, one, w, one, None, y)
        torch.cuda.synchronize()
        assert (y == 2.0 ** 30).all()


def test_product_does_not_depend_on_the_other_rows():
    """A row's product is the same bits alone, among a few rows and among many: the sums are exact, so the kernels that
    serve few and many rows agree."""
    torch, mh = _gpu()
    g = torch.Generator(device="cuda").manual_seed(4)
    rows, N, K = 700, 320, 1024
    x = torch.randint(-127, 128, (rows, K), generator=g, device="cuda", dtype=torch.int8)
    w = torch.randint(-127, 128, (1, N, K), generator=g, device="cuda", dtype=torch.int8)
    xs, ws = torch.rand(rows, generator=g, device="cuda"), torch.rand(N, generator=g, device="cuda")
    full = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")
    mh.moe_expert_matmul_i8(1, rows, N, K, x, xs, w, ws, None, full)
    for n in (1, 3, 16, 20, 64, 130):
        y = torch.empty(n, N, dtype=torch.bfloat16, device="cuda")
        mh.moe_expert_matmul_i8(1, n, N, K, x, xs, w, ws, None, y)
        torch.cuda.synchronize()
        assert torch.equal(y, full[:n]), n


CASES = [
    MoeConfig("i8_t1", T=1, H=128, I=64, E=8, E_local=8, k=2, n_chunks=1, dtype="int8", seed_base=900),
    MoeConfig("i8_t1_remote", T=1, H=128, I=64, E=64, E_local=2, e0=60, k=1, n_chunks=1, dtype="int8", seed_base=905),
    MoeConfig("i8_t3", T=3, H=320, I=192, E=16, E_local=16, k=8, n_chunks=1, dtype="int8", seed_base=910),
    MoeConfig("i8_t33", T=33, H=256, I=128, E=8, E_local=8, k=4, n_chunks=1, dtype="int8", seed_base=920),
    MoeConfig("i8_t70_n3", T=70, H=512, I=320, E=32, E_local=12, e0=5, k=5, n_chunks=3, dtype="int8", seed_base=930),
    MoeConfig("i8_t200_few_experts", T=200, H=192, I=64, E=4, E_local=3, k=2, n_chunks=1, dtype="int8", seed_base=935),
    MoeConfig("i8_t1000", T=1000, H=256, I=192, E=32, E_local=8, e0=4, k=4, n_chunks=2, dtype="int8", seed_base=940),
    MoeConfig("i8_zipf", T=3000, H=512, I=256, E=32, E_local=8, k=8, n_chunks=2, dtype="int8", seed_base=950,
              zipf_s=1.2, n_empty=2),
    MoeConfig("i8_small_tiles", T=700, H=448, I=192, E=8, E_local=5, e0=3, k=4, n_chunks=2, dtype="int8", seed_base=980),
    MoeConfig("i8_large_tiles", T=4100, H=128, I=512, E=8, E_local=8, k=4, n_chunks=1, dtype="int8", seed_base=985),
    MoeConfig("i8_down_wide", T=64, H=1024, I=64, E=32, E_local=32, k=8, n_chunks=1, dtype="int8", seed_base=990),
    MoeConfig("i8_down_wide_rows", T=250, H=1088, I=64, E=32, E_local=32, k=8, n_chunks=1, dtype="int8", seed_base=995),
    MoeConfig("i8_down_32_columns", T=8, H=2048, I=64, E=32, E_local=32, k=8, n_chunks=1, dtype="int8", seed_base=1000),
    MoeConfig("i8_down_32_columns_rows", T=41, H=2112, I=128, E=32, E_local=32, k=8, n_chunks=1, dtype="int8", seed_base=1005),
    MoeConfig("i8_wide", T=20, H=9216, I=64, E=8, E_local=4, k=2, n_chunks=1, dtype="int8", seed_base=960),
]


def _layer(torch, mh, cfg, stages, two_streams=True):
    inp = moe_inputs.make_inputs(cfg, parts=("x", "logits", "w1", "w2"))
    d = mh.make_desc(T=cfg.T, H=cfg.H, I=cfg.I, E=cfg.E, E_local=cfg.E_local, k=cfg.k, n_chunks=cfg.n_chunks, dtype="int8",
                     e0=cfg.e0)
    b = mh.allocate(d)
    b["out"].fill_(-7.0)
    b["yd"].fill_(-9.0)
    for name in ("x", "logits"):
        b[name] = harness.to_dev(inp, name, "bf16")
    for name, rows, cols in (("w1", 2 * cfg.I, cfg.H), ("w2", cfg.H, cfg.I)):
        w = harness.to_dev(inp, name, "bf16")
        b[name] = torch.empty(w.shape, dtype=torch.int8, device="cuda")
        b[name + "_scale"] = torch.empty(w.shape[:-1], device="cuda")
        mh.moe_quantize_rows_i8(cfg.E_local * rows, cols, w, b[name], b[name + "_scale"])
    cs = torch.cuda.current_stream()
    if stages:
        harness.run_stages(mh, d, b, False, cs)
    else:
        mh.moe_layer_forward(d, b, cs, torch.cuda.Stream() if two_streams else cs)
    torch.cuda.synchronize()
    return inp, d, b


@pytest.mark.parametrize("cfg", CASES, ids=[c.name for c in CASES])
def test_layer_forward(cfg):
    torch, mh = _gpu()
    print(f"[int8] {cfg}", flush=True)
    inp, d, b = _layer(torch, mh, cfg, stages=False)
    w1q, w1s = oi8.quantize_rows(inp["w1"])
    w2q, w2s = oi8.quantize_rows(inp["w2"])
    np.testing.assert_array_equal(b["w1"].cpu().numpy(), w1q)
    ref = oi8.forward(inp["x"], inp["logits"], w1q, w1s, w2q, w2s, k=cfg.k, e0=cfg.e0, E_local=cfg.E_local,
                      n_chunks=cfg.n_chunks, P_c=d.P_c)
    for n in ("offsets", "row_of", "src_token"):
        np.testing.assert_array_equal(b[n].cpu().numpy(), ref[n])
    used = ref["src_token"] >= 0
    np.testing.assert_array_equal(b["xd"].cpu().numpy()[used], ref["xdq"][used])
    np.testing.assert_array_equal(b["xd_scale"].cpu().numpy()[used], ref["xds"][used])
    out = harness.to_np(b["out"])
    assert np.all(out[cfg.T:] == -7.0) and np.all(harness.to_np(b["yd"])[~used] == -9.0)
    err = np.linalg.norm(out[:cfg.T] - ref["out"])
    assert err <= OUT_TOL * np.linalg.norm(ref["out"]), err / np.linalg.norm(ref["out"])
    _, _, c = _layer(torch, mh, cfg, stages=True)
    _, _, e = _layer(torch, mh, cfg, stages=False, two_streams=False)
    for o in (c, e):
        assert torch.equal(b["out"], o["out"]) and torch.equal(b["yd"], o["yd"])


def test_layer_routes_from_x():
    torch, mh = _gpu()
    cfg = MoeConfig("i8_from_x", T=65, H=256, I=64, E=32, E_local=32, k=4, n_chunks=2, dtype="int8", seed_base=970)
    inp, d, b = _layer(torch, mh, cfg, stages=True)
    w_r = moe_inputs.make_inputs(cfg, parts=("w_r",))
    b["w_r"] = harness.to_dev(w_r, "w_r", "bf16")
    logits = torch.empty(cfg.T, cfg.E, device="cuda")
    mh.moe_route_x(d, -1, b["x"], b["w_r"], logits, b["topk_idx"], b["gates"], b["counts"], b["offsets"], b["row_of"],
                   b["src_token"], b["workspace"])
    b["logits"] = logits
    cs = torch.cuda.current_stream()
    mh.moe_layer_forward(d, b, cs, cs)
    torch.cuda.synchronize()
    want = b["out"][:cfg.T].clone()
    b["logits"] = None
    mh.moe_layer_forward(d, b, cs, torch.cuda.Stream())
    torch.cuda.synchronize()
    assert torch.equal(b["out"][:cfg.T], want)


def test_rows_region_wider_than_routing_needs():
    """A caller's P_c above the static worst case, and its own table of rows that fills it: more experts have rows than
    the descriptor's tokens could reach."""
    torch, mh = _gpu()
    T, H, I, El, k = 2, 128, 64, 24, 1
    d = mh.make_desc(T=T, H=H, I=I, E=El, E_local=El, k=k, n_chunks=1, dtype="int8", P_c=48, P_out=4)
    rng = np.random.default_rng(3)
    xq, xs = rng.integers(-127, 128, (48, H)).astype(np.int8), (rng.random(48) + 0.1).astype(np.float32) * 0.01
    w1, w2 = rng.integers(-127, 128, (El, 2 * I, H)).astype(np.int8), rng.integers(-127, 128, (El, H, I)).astype(np.int8)
    w1s, w2s = np.full((El, 2 * I), 0.01, np.float32), np.full((El, H), 0.01, np.float32)
    off = np.arange(0, 2 * El + 1, 2, dtype=np.int32)
    dev = [torch.from_numpy(a).cuda() for a in (xq, xs, w1, w1s, w2, w2s, off)]
    h, hs = torch.empty(5 * 48 * I, dtype=torch.uint8, device="cuda"), torch.empty(48, device="cuda")
    yd = torch.zeros(48, H, dtype=torch.bfloat16, device="cuda")
    mh.moe_expert_ffn(d, 0, dev[0], dev[1], dev[2], dev[3], dev[4], dev[5], dev[6], None, h, hs, yd)
    torch.cuda.synchronize()
    gu = oi8.matmul(xq, xs, w1, w1s, off)
    hq, hsc = oi8.quantize_rows((gu[:, :I] / (1 + np.exp(-gu[:, :I])) * gu[:, I:]).astype(np.float32))
    want = oi8.matmul(hq, hsc, w2, w2s, off)
    got = oi8.decode_yd(yd.view(torch.int16).cpu().numpy())
    assert np.linalg.norm(got - want) <= OUT_TOL * np.linalg.norm(want)


def _ffn(torch, mh, T, H, I, xq, xs, w1, w1s, w2, w2s):
    """yd codes of T rows through one expert: few rows, or with more the GEMM."""
    d = mh.make_desc(T=T, H=H, I=I, E=1, E_local=1, k=1, n_chunks=1, dtype="int8")
    dev = [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in (xq, xs, w1, w1s, w2, w2s)]
    off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    h, hs = torch.empty(5 * d.P_c * I, dtype=torch.uint8, device="cuda"), torch.empty(d.P_c, device="cuda")
    yd = torch.zeros(d.P_c, H, dtype=torch.int16, device="cuda")
    mh.moe_expert_ffn(d, 0, dev[0], dev[1], dev[2], dev[3], dev[4], dev[5], off, None, h, hs, yd)
    torch.cuda.synchronize()
    return yd.cpu().numpy()[:T]


def test_rows_between_the_experts_and_combine_are_the_same_from_either_kernel():
    torch, mh = _gpu()
    rng = np.random.default_rng(8)
    T, H, I = 700, 320, 192
    xq, xs = rng.integers(-127, 128, (T, H)).astype(np.int8), (rng.random(T) + 0.1).astype(np.float32) * 0.01
    w = [rng.integers(-127, 128, (1, 2 * I, H)).astype(np.int8), (rng.random((1, 2 * I)) * 0.01).astype(np.float32),
         rng.integers(-127, 128, (1, H, I)).astype(np.int8), (rng.random((1, H)) * 0.01).astype(np.float32)]
    many = _ffn(torch, mh, T, H, I, xq, xs, *w)
    for n in (1, 16, 30, 47, 130):
        np.testing.assert_array_equal(_ffn(torch, mh, n, H, I, xq[:n], xs[:n], *w), many[:n])


@pytest.mark.parametrize("T", [8, 400])
def test_rows_between_the_experts_and_combine_at_the_ends_of_their_range(T):
    """Every column of h is equal, so its codes are 127 and y = 127 sum(w2) (h / 127) w2_scale: column scales take y
    through subnormal, smallest, ordinary, largest and too large values, and NaN. 2^-9 is the rounding, 1e-5 covers h's
    sigmoid and scales; a subnormal is off by half a step, 2^-71, at most."""
    torch, mh = _gpu()
    H, I = 128, 64
    xq, xs = np.full((T, H), 100, np.int8), np.full(T, 1e-3, np.float32)
    w1, w1s = np.full((1, 2 * I, H), 20, np.int8), np.full((1, 2 * I), 1e-3, np.float32)
    w2 = np.ones((1, H, I), np.int8)
    w2[0, 1::2] = -1
    scale = np.array([1e-38, 1e-30, 1e-24, 1e-21, 1e-20, 1e-18, 1e-9, 1e-3, 1.0, 1e9, 1e16, 2e18, 5e18, 1e20, 1e36, 0.0],
                     np.float32)
    w2s = np.tile(scale, H // len(scale))[None].copy()
    w2s[0, 32], w2s[0, 34] = np.nan, np.inf
    w2s[0, 33:34].view(np.uint32)[:] = 0xffffffff   # a NaN whose every bit is set
    got = oi8.decode_yd(_ffn(torch, mh, T, H, I, xq, xs, w1, w1s, w2, w2s))
    g = 20.0 * 100 * H * 1e-6
    y = g / (1 + np.exp(-g)) * g * I * w2[0, :, 0] * w2s[0].astype(np.float64)
    big = ~(np.abs(y) < 2.0 ** 65 * (1 - 1.5 * 2.0 ** -9))
    near = np.abs(np.abs(y) / 2.0 ** 65 - 1) < 0.01    # (no column falls there: either side would do)
    assert not near.any() and big.any() and (np.abs(y[~big]) > 2.0 ** 63).any() and ((0 < np.abs(y)) & (np.abs(y) < 2.0 ** -63)).any()
    assert np.isnan(got[:, big]).all()
    assert np.all(np.abs(got - y)[:, ~big] <= (2.0 ** -9 + 1e-5) * np.abs(y[~big]) + 2.0 ** -71)


def test_combine_reads_every_code_of_the_rows():
    torch, mh = _gpu()
    T, H = 1024, 64
    codes = np.arange(T * H, dtype=np.int64).astype(np.uint16).reshape(T, H)
    d = mh.make_desc(T=T, H=H, I=64, E=1, E_local=1, k=1, n_chunks=1, dtype="int8")
    out = torch.empty(d.P_out, H, dtype=torch.bfloat16, device="cuda")
    row = torch.arange(T, dtype=torch.int32, device="cuda").reshape(T, 1)
    mh.moe_combine(d, 0, torch.from_numpy(codes.view(np.int16)).cuda(), torch.ones(T, 1, device="cuda"), row, out)
    torch.cuda.synchronize()
    val = oi8.decode_yd(codes.view(np.int16))
    nan = np.isnan(val)
    want = moe_inputs.bf16_bits_to_f32(moe_inputs.f32_to_bf16_bits(np.where(nan, 0, val).astype(np.float32)))
    got = harness.to_np(out[:T])
    assert np.isnan(got[nan]).all() and nan.sum() == 2
    np.testing.assert_array_equal(got[~nan], want[~nan])


def test_layer_without_tokens():
    torch, mh = _gpu()
    d = mh.make_desc(T=0, H=128, I=64, E=8, E_local=4, k=2, n_chunks=2, dtype="int8")
    b = mh.allocate(d)
    b["x"] = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    b["logits"] = torch.empty(0, 8, device="cuda")
    for name, shape in (("w1", (4, 128, 128)), ("w2", (4, 128, 64))):
        b[name], b[name + "_scale"] = torch.ones(shape, dtype=torch.int8, device="cuda"), torch.ones(shape[:2], device="cuda")
    mh.moe_layer_forward(d, b, torch.cuda.current_stream(), torch.cuda.Stream())
    torch.cuda.synchronize()
    assert not b["offsets"].any().item()


def test_products_side_by_side_on_two_streams():
    """Two calls at once, each on its own stream and of another kind, give what each gives alone."""
    torch, mh = _gpu()
    g = torch.Generator(device="cuda").manual_seed(4)
    shapes = [(1, 40, 1024, 2048), (1, 900, 1032, 1088), (1, 5000, 2056, 320)]
    data, want = [], []
    for G, rows, N, K in shapes:
        x = torch.randint(-127, 128, (rows, K), dtype=torch.int8, device="cuda", generator=g)
        w = torch.randint(-127, 128, (G, N, K), dtype=torch.int8, device="cuda", generator=g)
        xs, ws = torch.rand(rows, device="cuda", generator=g) + 0.1, torch.rand(G, N, device="cuda", generator=g) + 0.1
        data.append((G, rows, N, K, x, xs, w, ws, None))
        want.append(torch.empty(rows, N, dtype=torch.bfloat16, device="cuda"))
        mh.moe_expert_matmul_i8(*data[-1], want[-1])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in shapes]
    got = [[torch.empty_like(w) for w in want] for _ in range(4)]
    torch.cuda.synchronize()
    for ys in got:
        for a, y, s in zip(data, ys, streams):
            mh.moe_expert_matmul_i8(*a, y, s)
    torch.cuda.synchronize()
    for ys in got:
        for y, w in zip(ys, want):
            assert torch.equal(y, w)


def test_a_row_that_is_not_finite_stays_visible_and_alone():
    torch, mh = _gpu()
    cfg = CASES[3]
    inp, d, b = _layer(torch, mh, cfg, stages=True)
    want = b["out"].clone()
    b["x"][7, 3] = float("nan")
    harness.run_stages(mh, d, b, False, torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert torch.isnan(b["out"][7]).all()
    keep = [t for t in range(cfg.T) if t != 7]
    assert torch.equal(b["out"][keep], want[keep])


@pytest.mark.parametrize("cfg", [CASES[0], CASES[3], CASES[6], CASES[7], CASES[9]], ids=["t1", "t33", "t1000", "small_tiles", "large_tiles"])
def test_replays_of_a_graph(cfg):
    torch, mh = _gpu()
    inp, d, b = _layer(torch, mh, cfg, stages=True)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        harness.run_stages(mh, d, b, False, torch.cuda.current_stream())
    x0 = b["x"].clone()
    for i in range(3):
        b["x"].copy_(x0 * (i + 1.25))
        g.replay()
        torch.cuda.synchronize()
        got = b["out"].clone()
        b["out"].fill_(0.0)
        harness.run_stages(mh, d, b, False, torch.cuda.current_stream())
        torch.cuda.synchronize()
        assert torch.equal(got[:cfg.T], b["out"][:cfg.T]), i


@pytest.mark.parametrize("T", [8, 400])
def test_rows_between_the_experts_and_combine_of_long_sums_and_small_scales(T):
    """The row's and the column's scale are small and the integer sum is long, so that the product of the scales is far
    below y. Every column of h is equal (codes 127), so y = sum(w2) h w2_scale; 2^-9 is the rounding, 1e-5 covers h's sigmoid
    and the FP32 steps, 2^-71 is half a subnormal step."""
    torch, mh = _gpu()
    H, I = 128, 2048
    xq, xs = np.full((T, H), 100, np.int8), np.full(T, 1e-3, np.float32)
    w1, w1s = np.full((1, 2 * I, H), 20, np.int8), np.full((1, 2 * I), 1e-3, np.float32)
    w1s[0, I:] = 1e-3 * 2.0 ** -38
    w2 = np.full((1, H, I), 127, np.int8)
    w2[0, 1::2] = -127
    w2s = (np.float32(1.3) * 2.0 ** -(np.arange(H) % 32).astype(np.float32) * 2.0 ** -14)[None].astype(np.float32)
    got = oi8.decode_yd(_ffn(torch, mh, T, H, I, xq, xs, w1, w1s, w2, w2s))
    g, u = 256e3 * float(xs[0]) * float(w1s[0, 0]), 256e3 * float(xs[0]) * float(w1s[0, I])
    y = g / (1 + np.exp(-g)) * u * I * w2[0, :, 0].astype(np.float64) * w2s[0].astype(np.float64)
    assert np.abs(y).max() < 2.0 ** -35 and np.abs(y).min() > 2.0 ** -70 and np.abs(y).min() < 2.0 ** -60
    assert np.all(np.abs(got - y) <= (2.0 ** -9 + 1e-5) * np.abs(y) + 2.0 ** -71)


def test_quantize_the_most_rows():
    torch, mh = _gpu()
    rows, cols = 2 ** 26 - 4, 8
    src = torch.ones(rows, cols, dtype=torch.bfloat16, device="cuda")
    src[-1] = torch.arange(8, device="cuda").to(torch.bfloat16)
    codes, scale = torch.zeros(rows, cols, dtype=torch.int8, device="cuda"), torch.zeros(rows, device="cuda")
    mh.moe_quantize_rows_i8(rows, cols, src, codes, scale)
    torch.cuda.synchronize()
    q, s = oi8.quantize_rows(np.arange(8, dtype=np.float32)[None])
    assert codes[-1].tolist() == q[0].tolist() and scale[-1].item() == s[0]
    assert (codes[:-1] == 127).all() and (scale[:-1] == float(np.float32(1) / np.float32(127))).all()


# More than 2048 tokens: a wave per token, the row in 1, 2, 4, 8 or 16 vectors a lane, or read twice
@pytest.mark.parametrize("H", [64, 512, 576, 1024, 2048, 2112, 4096, 8192, 8256, 16384])
def test_dispatch_of_many_tokens_bitwise(H):
    torch, mh = _gpu()
    T, E, El, k = 2049, 8, 3, 2
    rng = np.random.default_rng(H)
    a = rng.standard_normal((T, H)).astype(np.float32) * 10.0 ** rng.uniform(-3, 3, (T, 1)).astype(np.float32)
    a[5], a[6, -1], a[7, 0] = 0.0, np.nan, -np.inf
    dev, val = _bf16(torch, a)
    d = mh.make_desc(T=T, H=H, I=64, E=E, E_local=El, k=k, n_chunks=1, dtype="int8")
    row = np.full((T, k), -1, np.int32)
    local = rng.random((T, k)) < El / E
    local[5:8] = True
    row[local] = rng.permutation(d.P_c)[:local.sum()]
    xd, xds = torch.full((d.P_c, H), 77, dtype=torch.int8, device="cuda"), torch.full((d.P_c,), 7.0, device="cuda")
    mh.moe_dispatch(d, -1, dev, torch.from_numpy(row).cuda(), xd, xds, None)
    torch.cuda.synchronize()
    q, s = oi8.quantize_rows(val)
    want, wants = np.full((d.P_c, H), 77, np.int8), np.full(d.P_c, 7.0, np.float32)
    for j in range(k):
        m = row[:, j] >= 0
        want[row[m, j]], wants[row[m, j]] = q[m], s[m]
    np.testing.assert_array_equal(xd.cpu().numpy(), want)
    np.testing.assert_array_equal(xds.cpu().numpy(), wants)


# The GEMM's path stage by stage, each against 64 bits from what the stage before it left: 256 x 256 tiles for both
# products (the first two: several tiles a workgroup, last row tiles of uneven experts, odd numbers of stages; the third
# takes them for gate/up), and every length of h's quantisation (1, 2, 4, 8 or 16 vectors a lane, or read twice)
@pytest.mark.parametrize("T,H,I,E,El,k", [(3000, 832, 448, 8, 8, 6), (8200, 2112, 832, 16, 8, 4), (5001, 576, 1344, 8, 5, 7),
                                          (300, 64, 256, 2, 2, 1), (301, 128, 512, 2, 2, 1), (302, 64, 1024, 2, 2, 2),
                                          (303, 128, 1088, 2, 2, 1), (304, 64, 2112, 2, 2, 1), (305, 64, 4096, 2, 1, 2),
                                          (306, 64, 4160, 2, 2, 1)])
def test_expert_stages_one_by_one(T, H, I, E, El, k):
    torch, mh = _gpu()
    print(f"[int8] stages {T, H, I, E, El, k}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(T + I)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    d = mh.make_desc(T=T, H=H, I=I, E=E, E_local=El, k=k, n_chunks=1, dtype="int8")
    b = mh.allocate(d)
    b["x"] = rn(T, H).to(torch.bfloat16)
    b["logits"] = rn(T, E) + 0.7 * rn(1, E)     # experts of uneven length
    for name, rows, cols in (("w1", 2 * I, H), ("w2", H, I)):
        b[name], b[name + "_scale"] = torch.empty(El, rows, cols, dtype=torch.int8, device="cuda"), torch.empty(El, rows, device="cuda")
        mh.moe_quantize_rows_i8(El * rows, cols, (rn(El, rows, cols) * 0.05).to(torch.bfloat16), b[name], b[name + "_scale"])
    b["yd"].view(torch.int16).fill_(0x1234)
    harness.run_stages(mh, d, b, False, torch.cuda.current_stream())
    torch.cuda.synchronize()
    off, P, f64 = b["offsets"][0].tolist(), d.P_c, torch.float64
    n = off[-1]
    h = b["h"][:4 * P * I].view(torch.float32).reshape(P, I)
    hq, hs = b["h"][4 * P * I:5 * P * I].view(torch.int8).reshape(P, I), b["h_scale"]
    yd = torch.from_numpy(oi8.decode_yd(b["yd"].view(torch.int16).cpu().numpy())).cuda()
    assert (b["yd"].view(torch.int16)[n:] == 0x1234).all()

    def product(rows, s, w, ws):
        return (rows.to(f64) @ w.to(f64).t().contiguous()) * s.to(f64).unsqueeze(1) * ws.to(f64)
    for e in range(El):
        r = slice(off[e], off[e + 1])
        gu = product(b["xd"][r], b["xd_scale"][r], b["w1"][e], b["w1_scale"][e])
        G, U = gu[:, :I], gu[:, I:]
        want = G / (1 + torch.exp(-G)) * U
        # G and U: three FP32 roundings each, of which the sigmoid feels |G| more; its exponential's argument |G| 2^-23, the
        # exponential and the reciprocal 2^-23 each, one sum and two products
        bad = (h[r].to(f64) - want).abs() > (16 + 6 * G.abs()) * 2.0 ** -24 * want.abs()
        assert not bad.any(), (e, torch.nonzero(bad)[:4].tolist())
        # a product is exact in int32, three FP32 roundings, and half a step of 8 mantissa bits
        want = product(hq[r], hs[r], b["w2"][e], b["w2_scale"][e])
        bad = (yd[r] - want).abs() > (2.0 ** -9 + 2.0 ** -20) * want.abs() + 2.0 ** -71
        assert not bad.any(), (e, torch.nonzero(bad)[:4].tolist())
    q, s = oi8.quantize_rows(h[:n].cpu().numpy())
    np.testing.assert_array_equal(hq[:n].cpu().numpy(), q)
    np.testing.assert_array_equal(hs[:n].cpu().numpy(), s)
    row = b["row_of"].long()
    part = yd[row.clamp(min=0)] * (b["gates"].to(f64) * (row >= 0)).unsqueeze(2)
    want, terms = part.sum(1), part.abs().sum(1)
    assert ((b["out"][:T].to(f64) - want).abs() <= 2.0 ** -8 * want.abs() + 2 * k * 2.0 ** -24 * terms).all()


# The error that the rows of yd add to the output's own rounding, as a root mean square in units of that rounding. A code's
# error is uniform over a step half as long as BF16's: sqrt(1 + 1/4) = 1.118 together, where the gates spread the values. With
# k = 1 the gate is 1: an even code is a BF16 value (only the code's own 1/4), an odd one a tie (half a step, 3 in these units,
# and the 1/4): the mean is 7/4, 1.323. The squares of 300 thousand errors or more average to 1% here (their own spread is
# of the size of their mean): 1% on the ratio is more than five deviations.
@pytest.mark.parametrize("k,El,factor", [(1, 8, 1.323), (2, 8, 1.118), (8, 8, 1.118), (4, 3, 1.118)])
def test_error_of_the_layer_in_units_of_the_outputs_rounding(k, El, factor):
    torch, mh = _gpu()
    T, H, I, E, f64 = 1500, 512, 256, 8, torch.float64
    g = torch.Generator(device="cuda").manual_seed(k)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    d = mh.make_desc(T=T, H=H, I=I, E=E, E_local=El, k=k, n_chunks=1, dtype="int8")
    b = mh.allocate(d)
    b["x"], b["logits"] = rn(T, H).to(torch.bfloat16), rn(T, E)
    for name, rows, cols in (("w1", 2 * I, H), ("w2", H, I)):
        b[name], b[name + "_scale"] = torch.empty(El, rows, cols, dtype=torch.int8, device="cuda"), torch.empty(El, rows, device="cuda")
        mh.moe_quantize_rows_i8(El * rows, cols, (rn(El, rows, cols) * 0.05).to(torch.bfloat16), b[name], b[name + "_scale"])
    mh.moe_layer_forward(d, b, torch.cuda.current_stream(), torch.cuda.Stream())
    torch.cuda.synchronize()
    P, off = d.P_c, b["offsets"][0].tolist()
    y = torch.zeros(P, H, dtype=f64, device="cuda")
    hq = b["h"][4 * P * I:5 * P * I].view(torch.int8).reshape(P, I)
    for e in range(El):
        r = slice(off[e], off[e + 1])
        y[r] = (hq[r].to(f64) @ b["w2"][e].to(f64).t().contiguous()) * b["h_scale"][r].to(f64).unsqueeze(1) * b["w2_scale"][e].to(f64)
    row = b["row_of"].long()
    want = (y[row.clamp(min=0)] * (b["gates"].to(f64) * (row >= 0)).unsqueeze(2)).sum(1)
    assert (want != 0).sum() >= 300000
    one = (want.to(torch.bfloat16).to(f64) - want).norm()
    both = (b["out"][:T].to(f64) - want).norm()
    print(f"[int8] k {k}: {both / one:.4f} of one rounding, {both / want.norm():.3e} of the norm", flush=True)
    assert both <= 1.01 * factor * one


# Chunks without a token, no local expert, one expert in all, every expert chosen by every token
@pytest.mark.parametrize("cfg", [
    MoeConfig("i8_empty_chunks", T=2, H=128, I=64, E=8, E_local=8, k=3, n_chunks=5, dtype="int8", seed_base=1010),
    MoeConfig("i8_one_expert", T=37, H=192, I=128, E=1, E_local=1, k=1, n_chunks=2, dtype="int8", seed_base=1020),
    MoeConfig("i8_all_chosen", T=400, H=256, I=128, E=8, E_local=5, e0=3, k=8, n_chunks=3, dtype="int8", seed_base=1030),
    MoeConfig("i8_top1", T=900, H=320, I=192, E=16, E_local=16, k=1, n_chunks=1, dtype="int8", seed_base=1040),
], ids=lambda c: c.name)
def test_layer_forward_at_the_edges(cfg):
    test_layer_forward(cfg)


def test_layer_without_a_local_expert():
    torch, mh = _gpu()
    for T in (3, 3000):
        d = mh.make_desc(T=T, H=128, I=64, E=8, E_local=0, e0=8, k=2, n_chunks=2, dtype="int8")
        b = mh.allocate(d)
        b["x"], b["logits"] = torch.randn(T, 128, device="cuda").to(torch.bfloat16), torch.randn(T, 8, device="cuda")
        b["out"].fill_(3.0)
        mh.moe_layer_forward(d, b, torch.cuda.current_stream(), torch.cuda.Stream())
        torch.cuda.synchronize()
        assert not b["out"][:T].any() and (b["out"][T:] == 3.0).all() and (b["row_of"] == -1).all()
