"""GPU parity of the router loss and its gradient against the FP64 oracle.

Tolerances. A probability exp(x - lse) carries the rounding of its exponent, |x - m| log2(e) 2^-23 relative for the
product and the subtraction (|x - m| <= 64 here: 1.1e-5), the hardware exponential and reciprocal (2^-22 each) and the
sum of E terms (under 1e-6 by pairs), so TOL = 2e-5 of the terms that are added covers p, the sums over tokens, the
losses and the gradient (whose terms oracle.router_loss.grad_bound gives). lse = m + log(s) rounds once at its own
size, and log(s) is off by at most the relative error of s."""
import numpy as np
import pytest

from oracle import router_loss as orl

pytestmark = pytest.mark.gpu
TOL = 2e-5


def _gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import combine_moe_route_02_amd as mh
    mh.lib()
    return torch, mh


def _desc(mh, T, E, k):
    return mh.make_desc(T=T, H=64, I=64, E=E, E_local=1, k=k, n_chunks=1, dtype="f32")


def _buffers(torch, mh, d, S):
    T, E = d.T, d.E
    return {"lse": torch.full((T,), 7.0, device="cuda"), "counts": torch.full((S, E), -7, dtype=torch.int32, device="cuda"),
            "tokens": torch.full((S + 2,), -7, dtype=torch.int32, device="cuda"),
            "probs": torch.full((S, E), 7.0, device="cuda"), "loss": torch.full((3,), 7.0, device="cuda"),
            "dlogits": torch.full((T, E), 7.0, device="cuda"),
            "ws": torch.zeros(mh.moe_router_loss_bytes(d, S), dtype=torch.uint8, device="cuda")}


def _call(mh, d, S, a, z, lg, idx, off, mask, dl, b, stream=None):
    mh.moe_router_loss(d, S, a, z, lg, idx, off, mask, b["lse"], b["counts"], b["tokens"], b["probs"], b["loss"], b["ws"],
                       stream)
    mh.moe_router_loss_bwd(d, S, a, z, lg, b["lse"], off, mask, b["counts"], b["tokens"], dl, b["dlogits"], stream)


def _draw(T, E, k, seed, std=1.0):
    rng = np.random.default_rng(seed)
    lg = (rng.standard_normal((T, E)) * std).astype(np.float32)
    idx = np.argsort(-lg, axis=1, kind="stable")[:, :k].astype(np.int32)
    return rng, lg, idx


def _check(b, f, k, a, z, g):
    got = {n: v.cpu().numpy() for n, v in b.items() if n != "ws"}
    np.testing.assert_array_equal(got["counts"], f["seg_counts"])
    np.testing.assert_array_equal(got["tokens"], f["seg_tokens"])
    assert np.all(np.abs(got["lse"] - f["lse"]) <= TOL + 2.0 ** -23 * np.abs(f["lse"]))
    assert np.all(np.abs(got["probs"] - f["seg_probs"]) <= TOL * f["seg_probs"] + 1e-30)
    scale = np.array([abs(a) * f["loss"][1] + abs(z) * f["loss"][2], f["loss"][1], f["loss"][2]])
    # the z-loss squares lse: its error is twice that of lse, absolute TOL at the size of lse
    rms = np.sqrt(f["loss"][2])
    assert np.all(np.abs(got["loss"] - f["loss"]) <= TOL * scale + 2 * TOL * rms * np.array([abs(z), 0.0, 1.0]))
    want = orl.router_loss_bwd(f, k, a, z, g)
    lim = TOL * orl.grad_bound(f, k, a, z, g)
    n = max(1, int(f["seg_tokens"][-2]))
    lim += abs(g) * f["p"] * 2 * abs(z) / n * TOL  # the absolute error of lse in the z term
    bad = np.abs(got["dlogits"] - want) > lim + 1e-37
    assert not bad.any(), (np.argwhere(bad)[:4], got["dlogits"][bad][:4], want[bad][:4])


# T around the tile (32 rows) and the passes of a block, E across every lane shape and the scalar one
@pytest.mark.parametrize("T", [1, 7, 32, 33, 500])
@pytest.mark.parametrize("E,k", [(4, 1), (64, 2), (100, 8), (128, 8), (132, 3), (256, 8), (512, 4), (1024, 8), (7, 7), (333, 5)])
def test_one_segment(T, E, k):
    torch, mh = _gpu()
    _, lg, idx = _draw(T, E, k, 10 * T + E)
    a, z, g = 0.02, 0.003, 1.7
    d, b = _desc(mh, T, E, k), None
    b = _buffers(torch, mh, d, 1)
    _call(mh, d, 1, a, z, torch.from_numpy(lg).cuda(), torch.from_numpy(idx).cuda(), None, None,
          torch.tensor([g], device="cuda"), b)
    torch.cuda.synchronize()
    _check(b, orl.router_loss(lg, idx, k, a, z), k, a, z, g)


@pytest.mark.parametrize("off,masked", [
    ([0, 10, 10, 700, 701, 1500], True),       # empty and one-token segments, all rows covered
    ([5, 400, 1400], False),                   # rows before the first and behind the last segment
    ([1500, 1500], False), ([0, 0, 0], True),  # nothing counted
    (list(range(0, 1500, 5)) + [1500], True),  # more segments than a block has threads
])
def test_segments_and_masks(off, masked):
    torch, mh = _gpu()
    T, E, k = 1500, 96, 6
    rng, lg, idx = _draw(T, E, k, len(off), std=3.0)
    mask = None
    if masked:
        mask = (rng.random(T) < 0.8).astype(np.uint8)
        lg[mask == 0] = [np.nan, np.inf, -np.inf][len(off) % 3]
    lg[400:410] = -np.inf                      # no finite logit: left out
    lg[20:30, ::2] = -np.inf                   # disabled experts
    a, z = 1.5, 0.25
    S = len(off) - 1
    d = _desc(mh, T, E, k)
    b = _buffers(torch, mh, d, S)
    _call(mh, d, S, a, z, torch.from_numpy(lg).cuda(), torch.from_numpy(idx).cuda(),
          torch.tensor(off, dtype=torch.int32, device="cuda"), None if mask is None else torch.from_numpy(mask).cuda(),
          None, b)
    torch.cuda.synchronize()
    _check(b, orl.router_loss(lg, idx, k, a, z, off, mask), k, a, z, 1.0)


# Few tiles in several segments (one block adds them), at each lane shape, and just past that
@pytest.mark.parametrize("T,E,k,S", [(12, 80, 3, 22), (1, 4, 1, 2), (40, 7, 2, 5), (65, 64, 8, 3), (300, 128, 8, 17), (200, 256, 4, 9),
                                     (90, 512, 2, 8), (64, 1024, 8, 3), (33, 333, 5, 6), (2000, 60, 6, 40), (1400, 160, 3, 2),
                                     (700, 512, 8, 30), (5, 136, 4, 58), (267, 212, 8, 57), (3000, 64, 4, 2), (4000, 100, 3, 40)])
def test_few_tiles_in_segments(T, E, k, S):
    torch, mh = _gpu()
    rng, lg, idx = _draw(T, E, k, T + E + S, std=2.0)
    mask = (rng.random(T) < 0.7).astype(np.uint8)
    lg[mask == 0] = np.nan
    off = np.sort(rng.integers(0, T + 1, S + 1)).astype(np.int32)
    a, z, g = 0.7, 0.01, -0.6
    d = _desc(mh, T, E, k)
    b = _buffers(torch, mh, d, S)
    _call(mh, d, S, a, z, torch.from_numpy(lg).cuda(), torch.from_numpy(idx).cuda(), torch.from_numpy(off).cuda(),
          torch.from_numpy(mask).cuda(), torch.tensor([g], device="cuda"), b)
    torch.cuda.synchronize()
    _check(b, orl.router_loss(lg, idx, k, a, z, off.tolist(), mask), k, a, z, g)


def test_rows_of_the_lowest_value():
    """A row that holds the type's lowest value everywhere is an even row; its lse squared passes FP32, so the z part
    is infinite and a loss that does not use it stays finite."""
    torch, mh = _gpu()
    T, E, k = 50, 64, 4
    _, lg, idx = _draw(T, E, k, 8)
    lg[30] = np.finfo(np.float32).min
    lg[31, :60] = np.finfo(np.float32).min
    d = _desc(mh, T, E, k)
    b = _buffers(torch, mh, d, 1)
    _call(mh, d, 1, 0.5, 0.0, torch.from_numpy(lg).cuda(), torch.from_numpy(idx).cuda(), None, None, None, b)
    torch.cuda.synchronize()
    assert torch.isinf(b["loss"][2]).item()
    f = orl.router_loss(lg, idx, k, 0.5, 0.0)
    b["loss"][2] = 0.0
    f["loss"][2] = 0.0
    _check(b, f, k, 0.5, 0.0, 1.0)


def test_nan_of_a_counted_token_stays_visible():
    torch, mh = _gpu()
    T, E, k = 70, 64, 2
    _, lg, idx = _draw(T, E, k, 3)
    lg[40, 3] = np.nan
    d = _desc(mh, T, E, k)
    b = _buffers(torch, mh, d, 1)
    _call(mh, d, 1, 1.0, 1.0, torch.from_numpy(lg).cuda(), torch.from_numpy(idx).cuda(), None, None, None, b)
    torch.cuda.synchronize()
    assert torch.isnan(b["loss"]).all() and torch.isnan(b["dlogits"][40]).all()
    assert torch.isfinite(b["dlogits"][:40]).all() and torch.isfinite(b["dlogits"][41:]).all()


def test_unaligned_rows_and_long_input():
    """A logits pointer off the 16-byte grid, and tiles of more than 32 rows (T > 32768)."""
    torch, mh = _gpu()
    for T, E, k, shift in ((200, 64, 4, 1), (70001, 8, 2, 0)):
        _, lg, idx = _draw(T, E, k, T)
        flat = torch.zeros(T * E + 4, device="cuda")
        view = flat[shift:shift + T * E]
        view.copy_(torch.from_numpy(lg).cuda().reshape(-1))
        d = _desc(mh, T, E, k)
        b = _buffers(torch, mh, d, 1)
        _call(mh, d, 1, 0.3, 0.1, view, torch.from_numpy(idx).cuda(), None, None, None, b)
        torch.cuda.synchronize()
        _check(b, orl.router_loss(lg, idx, k, 0.3, 0.1), k, 0.3, 0.1, 1.0)


def test_no_tokens():
    torch, mh = _gpu()
    d = _desc(mh, 0, 32, 4)
    b = _buffers(torch, mh, d, 2)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    _call(mh, d, 2, 1.0, 1.0, None, None, off, None, None, b)
    torch.cuda.synchronize()
    assert not b["loss"].any() and not b["tokens"].any() and not b["counts"].any() and not b["probs"].any()


def test_gradient_matches_differences_of_the_loss():
    """Central differences of the kernel's own loss. With step h the truncation is h^2/6 of a third derivative near the
    loss itself, and the FP32 loss rounds at 2^-24 of its size on both sides: both are far under the 2% asked of the
    directional derivative for h = 0.05."""
    torch, mh = _gpu()
    T, E, k, a, z, h = 48, 32, 4, 1.0, 0.1, 0.05
    rng, lg, idx = _draw(T, E, k, 5)
    v = rng.standard_normal((T, E)).astype(np.float32)
    d = _desc(mh, T, E, k)
    b = _buffers(torch, mh, d, 1)
    idx_d = torch.from_numpy(idx).cuda()

    def loss(x):
        _call(mh, d, 1, a, z, torch.from_numpy(x.astype(np.float32)).cuda(), idx_d, None, None, None, b)
        torch.cuda.synchronize()
        return b["loss"][0].item()

    diff = (loss(lg + h * v) - loss(lg - h * v)) / (2 * h)
    loss(lg)
    along = float((b["dlogits"].cpu().numpy().astype(np.float64) * v).sum())
    assert abs(diff - along) <= 0.02 * abs(along) + 2.0 ** -22 / h


def test_repeats_bit_for_bit_on_streams_and_in_a_graph():
    torch, mh = _gpu()
    T, E, k, S = 3000, 128, 8, 3
    _, lg, idx = _draw(T, E, k, 6)
    off = torch.tensor([0, 1000, 1001, 2990], dtype=torch.int32, device="cuda")
    lg_d, idx_d = torch.from_numpy(lg).cuda(), torch.from_numpy(idx).cuda()
    d = _desc(mh, T, E, k)
    ref = _buffers(torch, mh, d, S)
    _call(mh, d, S, 1.0, 0.1, lg_d, idx_d, off, None, None, ref)
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    b = _buffers(torch, mh, d, S)
    other.wait_stream(torch.cuda.current_stream())
    _call(mh, d, S, 1.0, 0.1, lg_d, idx_d, off, None, None, b, other)
    torch.cuda.synchronize()
    for n in ref:
        if n != "ws":
            assert torch.equal(ref[n], b[n]), n
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _call(mh, d, S, 1.0, 0.1, lg_d, idx_d, off, None, None, b)
    for i in range(3):
        lg2 = torch.from_numpy(np.roll(lg, i, axis=0)).cuda()
        idx2 = torch.from_numpy(np.roll(idx, i, axis=0)).cuda()
        lg_d.copy_(lg2)
        idx_d.copy_(idx2)
        g.replay()
        torch.cuda.synchronize()
        _call(mh, d, S, 1.0, 0.1, lg2, idx2, off, None, None, ref)  # eager work between the replays
        torch.cuda.synchronize()
        for n in ref:
            if n != "ws":
                assert torch.equal(ref[n], b[n]), (i, n)


@pytest.mark.parametrize("E", [64, 256, 100, 333])
@pytest.mark.parametrize("g", [np.inf, np.nan])
def test_tokens_left_out_have_zero_gradient_whatever_the_upstream_gradient_is(E, g):
    """A step whose upstream gradient has overflowed (a loss scaler sees that from the counted rows): masked tokens,
    tokens outside every segment and tokens without a finite logit still get rows of zeros."""
    torch, mh = _gpu()
    T, k = 90, 4
    _, lg, idx = _draw(T, E, k, 11)
    mask = np.ones(T, np.uint8)
    mask[10:20] = 0
    lg[30:40] = -np.inf
    off = torch.tensor([5, 50, 80], dtype=torch.int32, device="cuda")
    d = _desc(mh, T, E, k)
    b = _buffers(torch, mh, d, 2)
    _call(mh, d, 2, 0.5, 0.1, torch.from_numpy(lg).cuda(), torch.from_numpy(idx).cuda(), off, torch.from_numpy(mask).cuda(),
          torch.tensor([g], dtype=torch.float32, device="cuda"), b)
    torch.cuda.synchronize()
    got = b["dlogits"].cpu().numpy()
    out = np.zeros(T, bool)
    out[:5] = out[10:20] = out[30:40] = out[80:] = True
    assert np.all(got[out] == 0.0)
    assert not np.isfinite(got[~out]).any(axis=1).all()


# As many segments as the call takes, of a few tokens or of none; many experts with many segments
@pytest.mark.parametrize("T,E,k,S", [(70000, 8, 2, 65536), (500, 12, 3, 65536), (9000, 1024, 8, 3000), (40000, 33, 4, 20000)])
def test_very_many_segments(T, E, k, S):
    torch, mh = _gpu()
    print(f"[router_loss] {T, E, k, S}", flush=True)
    rng, lg, idx = _draw(T, E, k, S)
    mask = (rng.random(T) < 0.9).astype(np.uint8)
    lg[mask == 0] = np.nan
    off = np.sort(rng.integers(0, T + 1, S + 1)).astype(np.int32)
    a, z, g = 0.7, 0.01, -0.6
    d = _desc(mh, T, E, k)
    b = _buffers(torch, mh, d, S)
    args = (torch.from_numpy(lg).cuda(), torch.from_numpy(idx).cuda(), torch.from_numpy(off).cuda(), torch.from_numpy(mask).cuda(),
            torch.tensor([g], device="cuda"))
    for _ in range(2):  # (the second call finds the arrival counter as the first left it)
        _call(mh, d, S, a, z, *args, b)
    torch.cuda.synchronize()
    _check(b, orl.router_loss(lg, idx, k, a, z, off.tolist(), mask), k, a, z, g)
