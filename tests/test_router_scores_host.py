"""Refusals of routing by scores (no GPU: every check runs before a launch)."""
import os

import pytest

mh = pytest.importorskip("combine_moe_route_02_amd")


def _desc(**kw):
    if not os.path.exists(mh.LIB_PATH):
        pytest.skip("libmoe.so not built (run __graft_entry__.build())")
    base = dict(T=1000, H=64, I=64, E=32, E_local=8, k=4, n_chunks=2, dtype="bf16")
    base.update(kw)
    return mh.make_desc(**base)


def _status(fn, *a):
    try:
        fn(*a)
    except mh.MoeError as e:
        return e.status
    return 0


FWD = ("logits", "bias", "topk_idx", "gates", "counts", "offsets", "row_of", "src_token", "workspace")
BWD = ("logits", "dgates", "topk_idx", "x", "dlogits", "dwr_acc", "dwr", "workspace")


def _fwd(d, r, chunk=-1, **null):
    return _status(mh.moe_route_scores, d, chunk, r, *[null.get(n, 16) for n in FWD], 0)


def _bwd(d, r, chunk=-1, **null):
    return _status(mh.moe_route_scores_bwd, d, chunk, r, *[null.get(n, 16 + 16 * i) for i, n in enumerate(BWD)], 0)


@pytest.mark.parametrize("call", [_fwd, _bwd])
@pytest.mark.parametrize("kw,status", [
    (dict(score=2), -1), (dict(score=-1), -1), (dict(n_groups=0), -1), (dict(n_groups=3), -1), (dict(n_groups=-4), -1),
    (dict(n_groups=8, topk_groups=0), -1), (dict(n_groups=8, topk_groups=9), -1), (dict(group_top=0), -1),
    (dict(group_top=3), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1),
    (dict(n_groups=32, topk_groups=3), -1),  # three experts for four slots
])
def test_options_are_checked(call, kw, status):
    assert call(_desc(), mh.make_router_scores(**kw)) == status
    r = mh.make_router_scores()
    r.renormalize = 2
    assert call(_desc(), r) == -1


@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_options_descriptor_and_chunk(call):
    r = mh.make_router_scores()
    assert call(_desc(), None) == -1
    assert call(_desc(E=128), mh.make_router_scores(n_groups=128, topk_groups=128)) == -3
    assert call(_desc(), r, chunk=2) == -1 and call(_desc(), r, chunk=-2) == -1
    assert call(_desc(k=9), r) == -3


@pytest.mark.parametrize("name", [n for n in FWD if n != "bias"])
def test_forward_needs_its_buffers(name):
    assert _fwd(_desc(), mh.make_router_scores(), **{name: None}) == -1


@pytest.mark.parametrize("name", [n for n in BWD if n != "x"])
def test_backward_needs_its_buffers(name):
    assert _bwd(_desc(), mh.make_router_scores(), **{name: None}) == -1


def test_workspace_is_aligned():
    assert _fwd(_desc(), mh.make_router_scores(), workspace=24) == -1
    bufs = {f: 16 * (i + 1) for i, f in enumerate(mh.TENSOR_FIELDS)}
    bufs.update(router_scores=mh.make_router_scores(), workspace=24)
    for fn in (mh.moe_layer_forward, mh.moe_layer_backward, mh.moe_layer_forward_backward):
        assert _status(fn, _desc(flags=mh.FLAG_ROUTER_SCORES), bufs, 0, 0) == -1


def test_backward_types_and_alias():
    r = mh.make_router_scores()
    assert _bwd(_desc(dtype="fp8"), r) == -3 and _bwd(_desc(dtype="int8"), r) == -3
    assert _bwd(_desc(), r, dlogits=16) == -1  # the logits buffer
    assert _bwd(_desc(), r, dlogits=24) == -1 and _bwd(_desc(), r, logits=20) == -1  # not 16-byte aligned
    # without x nothing but dlogits is asked for; no tokens, no work
    assert _bwd(_desc(T=0), r, x=None, dwr_acc=None, dwr=None, workspace=None, logits=None, dgates=None, topk_idx=None, dlogits=None) == 0
    assert _bwd(_desc(), r, x=None, dwr_acc=None, dwr=None, workspace=None, dlogits=None) == -1


def test_bias_update_is_checked():
    f = mh.moe_router_bias_update
    assert _status(f, 0, 1, 16, 0.1, 16, 0) == -3 and _status(f, 1025, 1, 16, 0.1, 16, 0) == -3
    assert _status(f, 8, -1, 16, 0.1, 16, 0) == -1
    assert _status(f, 8, 1, None, 0.1, 16, 0) == -1 and _status(f, 8, 1, 16, 0.1, None, 0) == -1
    assert _status(f, 8, 1, 16, float("nan"), 16, 0) == -1
    assert _status(f, 8, 0, None, 0.1, None, 0) == 0


# ------------------------------------------------------------------ MOE_FLAG_ROUTER_SCORES

def test_flag_goes_with_every_dtype():
    for dt in ("f32", "bf16", "fp8", "int8"):
        assert _status(mh.workspace_bytes, _desc(dtype=dt, flags=mh.FLAG_ROUTER_SCORES)) == 0
    assert _status(mh.workspace_bytes, _desc(flags=mh.FLAG_ROUTER_SCORES | mh.FLAG_ROUTER_LOSS | mh.FLAG_FP8_DXD)) == 0
    assert _status(mh.workspace_bytes, _desc(flags=128)) == -1
    assert mh.workspace_bytes(_desc(flags=mh.FLAG_ROUTER_SCORES)) == mh.workspace_bytes(_desc())


def test_layer_checks_the_options():
    d = _desc(flags=mh.FLAG_ROUTER_SCORES)
    bufs = {f: 16 * (i + 1) for i, f in enumerate(mh.TENSOR_FIELDS)}
    bufs["router_scores"] = mh.make_router_scores(n_groups=3)
    for fn in (mh.moe_layer_forward, mh.moe_layer_backward, mh.moe_layer_forward_backward):
        assert _status(fn, d, bufs, 0, 0) == -1
        assert _status(fn, d, {**bufs, "router_scores": None}, 0, 0) == -1  # zeroed options: no group at all
        assert _status(fn, d, {**bufs, "router_scores": mh.make_router_scores(), "logits": None, "router_logits": None}, 0, 0) == -1
        # from x: the projection's descriptors only
        from_x = {**bufs, "router_scores": mh.make_router_scores(), "logits": None}
        assert _status(fn, _desc(flags=mh.FLAG_ROUTER_SCORES, E=36), from_x, 0, 0) == -3
        assert _status(fn, _desc(flags=mh.FLAG_ROUTER_SCORES, dtype="f32"), from_x, 0, 0) == -3
    assert _status(mh.moe_layer_backward, d, {**bufs, "router_scores": mh.make_router_scores(), "dlogits": bufs["logits"]}, 0, 0) == -1
