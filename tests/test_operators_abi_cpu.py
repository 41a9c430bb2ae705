"""Refusals of the operators around the routed experts: argument errors are
found before any launch, so no device memory is touched -- no GPU."""
import ctypes as C

import pytest

from streamed_quantized_expert_b200 import build, ops

P = 1 << 21  # an aligned address that nothing reads
INV, UNS = ops.MOE_ERR_INVALID, ops.MOE_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return ops.lib()


def refused(status, fn, *args):
    with pytest.raises(ops.MoeError) as ei:
        fn(*args)
    assert ei.value.status == status


def route(T=4, d=None, cfg=None, bias=P, L=0.0, table=P, ns=0, sw=None, logits=P, ids=P, w=P):
    d = d or ops.desc(64, 4, 64, 32, 32, 4)
    return (logits, T, d, cfg, bias, L, table, ns, sw, ids, w)


def test_struct_size():
    assert C.sizeof(ops.RouteConfig) == 24


@pytest.mark.parametrize("status,kw,cfg", [
    (INV, dict(), None),
    (INV, dict(T=-1), dict()),
    (INV, dict(logits=None), dict()),
    (INV, dict(ids=None), dict()),
    (INV, dict(w=None), dict()),
    (INV, dict(L=-0.5), dict()),
    (INV, dict(L=float("nan")), dict()),
    (INV, dict(L=0.5, table=None), dict()),
    (INV, dict(ns=9), dict()),
    (INV, dict(ns=-1), dict()),
    (INV, dict(), dict(score=2)),
    (INV, dict(), dict(n_groups=0)),
    (INV, dict(), dict(n_groups=7)),                             # 64 experts do not form 7 groups
    (INV, dict(), dict(n_groups=8, top_groups=0)),
    (INV, dict(), dict(n_groups=8, top_groups=9)),
    (INV, dict(), dict(n_groups=8, top_groups=4, group_top=3)),
    (INV, dict(), dict(n_groups=8, top_groups=4, group_top=0)),
    (UNS, dict(), dict(n_groups=64, top_groups=32, group_top=1)),  # more than 32 groups
    (INV, dict(), dict(n_groups=64, top_groups=32, group_top=2)),  # groups of one expert
    (INV, dict(d=ops.desc(64, 9, 64, 32, 32, 4)), dict(n_groups=8, top_groups=1)),  # k above the kept groups
    (INV, dict(), dict(scale=float("inf"))),
    (INV, dict(), dict(scale=float("nan"))),
    (INV, dict(d=ops.desc(64, 65, 64, 32, 32, 4)), dict()),
    (UNS, dict(d=ops.desc(2048, 4, 64, 32, 32, 4)), dict()),
    (UNS, dict(T=(1 << 22) + 1), dict()),
    (INV, dict(logits=P + 1), dict()), (INV, dict(bias=P + 2), dict()), (INV, dict(L=0.5, table=P + 2), dict()),
    (INV, dict(ns=1, sw=P + 3), dict()), (INV, dict(ids=P + 1), dict()), (INV, dict(w=P + 2), dict()),
])
def test_route_refusals(status, kw, cfg):
    c = None if cfg is None else ops.route_config(**cfg)
    refused(status, ops.moe_route_grouped, *route(cfg=c, **kw))


def test_no_tokens_is_no_work():
    cfg = ops.route_config()
    ops.moe_route_grouped(*route(T=0, cfg=cfg, logits=None, ids=None, w=None))
    ops.moe_add_norm_quant(None, 0, None, 0, None, 1e-6, 0, 64, None, None, None, None)
    ops.moe_quantize_channels(None, 0, 0, 64, None, None)
    ops.moe_swiglu_quant(None, 0, 0, 64, None, None)
    ops.moe_int_matmul(None, None, 0, None, None, 64, 64, None, None, None, 0, None)
    ops.moe_int_matmul(None, None, 4, None, None, 0, 64, None, None, None, 0, None)


def norm(h=P, ht=0, delta=P, dt=0, gamma=P, eps=1e-6, T=4, H=64, ho=P, x=P, q=P, qs=P):
    return (h, ht, delta, dt, gamma, eps, T, H, ho, x, q, qs)


@pytest.mark.parametrize("status,kw", [
    (INV, dict(h=None)), (INV, dict(gamma=None)), (INV, dict(x=None, q=None, qs=None)),
    (INV, dict(qs=None)), (INV, dict(q=None)), (INV, dict(ht=2)), (INV, dict(dt=-1)), (INV, dict(T=-1)),
    (INV, dict(H=0)), (INV, dict(H=63)), (INV, dict(H=12)), (UNS, dict(H=65544)),
    (INV, dict(eps=0.0)), (INV, dict(eps=-1.0)), (INV, dict(eps=float("nan"))), (INV, dict(eps=float("inf"))),
    (INV, dict(h=P + 8)), (INV, dict(delta=P + 4)), (INV, dict(gamma=P + 2)), (INV, dict(ho=P + 8)),
    (INV, dict(x=P + 8)), (INV, dict(q=P + 4)), (INV, dict(qs=P + 2)),
])
def test_norm_refusals(status, kw):
    refused(status, ops.moe_add_norm_quant, *norm(**kw))


@pytest.mark.parametrize("status,args", [
    (INV, (None, 0, 4, 64, P, P)), (INV, (P, 0, 4, 64, None, P)), (INV, (P, 0, 4, 64, P, None)),
    (INV, (P, 3, 4, 64, P, P)), (INV, (P, 0, -4, 64, P, P)), (INV, (P, 0, 4, 60, P, P)), (INV, (P, 0, 4, 0, P, P)),
    (UNS, (P, 0, 4, 65544, P, P)), (INV, (P + 8, 0, 4, 64, P, P)), (INV, (P, 0, 4, 64, P + 4, P)),
    (INV, (P, 0, 4, 64, P, P + 1)),
])
@pytest.mark.parametrize("fn", ["moe_quantize_channels", "moe_swiglu_quant"])
def test_row_quant_refusals(fn, status, args):
    refused(status, getattr(ops, fn), *args)


def mm(xq=P, xs=P, T=4, wq=P, ws=P, N=64, K=64, add=None, row_w=None, y=P, yt=0, err=P):
    return (xq, xs, T, wq, ws, N, K, add, row_w, y, yt, err)


@pytest.mark.parametrize("status,kw", [
    (INV, dict(xq=None)), (INV, dict(xs=None)), (INV, dict(wq=None)), (INV, dict(ws=None)), (INV, dict(y=None)),
    (INV, dict(T=-1)), (INV, dict(N=-1)), (INV, dict(K=0)), (INV, dict(K=24)), (UNS, dict(K=65552)),
    (UNS, dict(T=(1 << 20) + 1)), (UNS, dict(N=(1 << 20) + 1)), (INV, dict(yt=2)),
    (INV, dict(xq=P + 8)), (INV, dict(wq=P + 1)), (INV, dict(xs=P + 2)), (INV, dict(y=P + 1)),
    (INV, dict(yt=1, y=P + 2)), (INV, dict(add=P + 2)), (INV, dict(row_w=P + 1)),
    (INV, dict(err=P + 2)),
    (INV, dict(add=P, y=P, yt=0)),  # in place only where y is fp32
])
def test_int_matmul_refusals(status, kw):
    refused(status, ops.moe_int_matmul, *mm(**kw))
