"""What the microscaled 4-bit calls, the router and the layer refuse, checked on
the host before any HIP call (the addresses are never dereferenced)."""
import pytest

import block_quantized_gemv_kq_amd as kq

A = 0x10000   # aligned to everything
F32, F16, BF16 = kq.KQ_F32, kq.KQ_F16, kq.KQ_BF16
ARG, SHAPE, ALIGN = kq.KQ_ERR_ARG, kq.KQ_ERR_SHAPE, kq.KQ_ERR_ALIGN


def refuse(name, good, cases, empty=()):
    fn = getattr(kq.lib(), name)
    keys = list(good)
    for change, want in cases:
        args = {**good, **change}
        got = fn(*[args[k] for k in keys])
        assert got == want, (name, change, got, want)
        assert kq.last_error(), (name, change)
    for change in empty:
        args = {**good, **change}
        assert fn(*[args[k] for k in keys]) == kq.KQ_OK, (name, change)


def bad_k(key, most=kq.KQ_MAX_K):
    return [({key: k}, SHAPE) for k in (0, -32, 16, 33, most + 32)]


def test_quantize_refusals():
    refuse("kq_mx4_quantize", dict(type=F16, x=A, ldx=64, codes=A, scales=A, R=4, K=64, stream=None),
           bad_k("K") + [({"type": 3}, ARG), ({"type": -1}, ARG), ({"x": None}, ARG), ({"codes": None}, ARG),
                         ({"scales": None}, ARG), ({"R": -1}, ARG), ({"R": kq.KQ_MX4_MAX_ROWS + 1}, ARG),
                         ({"ldx": 63}, ARG), ({"ldx": 1 << 36}, ARG), ({"x": A + 1}, ALIGN),
                         ({"x": A + 2, "type": F32}, ALIGN), ({"codes": A + 8}, ALIGN), ({"scales": A + 2}, ALIGN),
                         ({"R": kq.KQ_MX4_MAX_ROWS, "ldx": 65}, ARG)],
           [{"R": 0}, {"R": 0, "x": None, "codes": None, "scales": None}])


def test_dequantize_refusals():
    refuse("kq_mx4_dequantize", dict(codes=A, scales=A, type=F32, out=A, ldo=64, R=4, K=64, stream=None),
           bad_k("K") + [({"type": 7}, ARG), ({"out": None}, ARG), ({"codes": None}, ARG), ({"scales": None}, ARG),
                         ({"R": -1}, ARG), ({"ldo": 32}, ARG), ({"out": A + 2}, ALIGN), ({"codes": A + 4}, ALIGN),
                         ({"scales": A + 1}, ALIGN)],
           [{"R": 0}])


def test_gemv_refusals():
    refuse("kq_mx4_gemv", dict(codes=A, scales=A, type=F16, x=A, y=A, N=48, K=64, M=2, stream=None),
           bad_k("K") + [({"type": 5}, ARG), ({"M": -1}, ARG), ({"M": kq.KQ_MAX_M + 1}, ARG), ({"N": -1}, ARG),
                         ({"N": kq.KQ_MX4_MAX_ROWS + 1}, ARG), ({"codes": None}, ARG), ({"scales": None}, ARG),
                         ({"x": None}, ARG), ({"y": None}, ARG), ({"codes": A + 8}, ALIGN), ({"scales": A + 2}, ALIGN),
                         ({"x": A + 8}, ALIGN), ({"y": A + 2}, ALIGN)],
           [{"M": 0}, {"N": 0}, {"N": 0, "codes": None}])


def test_gemm_refusals():
    refuse("kq_mx4_gemm", dict(ac=A, asc=A, wc=A, ws=A, type=BF16, y=A, M=2, N=48, K=64, stream=None),
           bad_k("K") + [({"type": -2}, ARG), ({"M": -1}, ARG), ({"N": -1}, ARG), ({"M": kq.KQ_MX4_MAX_ROWS + 1}, ARG),
                         ({"N": kq.KQ_MX4_MAX_ROWS + 1}, ARG), ({"ac": None}, ARG), ({"asc": None}, ARG),
                         ({"wc": None}, ARG), ({"ws": None}, ARG), ({"y": None}, ARG), ({"ac": A + 8}, ALIGN),
                         ({"wc": A + 8}, ALIGN), ({"asc": A + 2}, ALIGN), ({"ws": A + 1}, ALIGN), ({"y": A + 8}, ALIGN),
                         ({"M": kq.KQ_MX4_MAX_ROWS, "N": kq.KQ_MX4_MAX_ROWS}, ARG)],
           [{"M": 0}, {"N": 0}])


ROUTE = dict(xtype=F16, x=A, wtype=F32, W=A, M=2, K=64, E=8, top_k=2, renorm=1, ids=A, weights=A, ws=A, wsb=2 * 8 * 8,
             stream=None)
ROUTE_CASES = [({"xtype": 3}, ARG), ({"wtype": -1}, ARG), ({"M": -1}, ARG), ({"M": 65}, ARG), ({"E": 0}, ARG),
               ({"E": kq.KQ_MOE_MAX_EXPERTS + 1}, ARG), ({"top_k": 0}, ARG), ({"top_k": 9}, ARG),
               ({"top_k": 65, "E": 128}, ARG), ({"renorm": 2}, ARG), ({"x": None}, ARG), ({"W": None}, ARG),
               ({"ids": None}, ARG), ({"weights": None}, ARG), ({"ws": None}, ARG), ({"x": A + 8}, ALIGN),
               ({"W": A + 8}, ALIGN), ({"ids": A + 2}, ALIGN), ({"weights": A + 2}, ALIGN), ({"ws": A + 8}, ALIGN)]


def test_route_refusals():
    need = kq.kq_moe_route_workspace_bytes(2, 8)
    good = dict(ROUTE, wsb=need)
    refuse("kq_moe_route", good, bad_k("K") + ROUTE_CASES + [({"wsb": need - 1}, ARG), ({"wsb": -1}, ARG)], [{"M": 0}])
    refuse("kq_moe_route_workspace_bytes", dict(M=2, E=8),
           [({"M": 65}, ARG), ({"M": -1}, ARG), ({"E": 0}, ARG), ({"E": kq.KQ_MOE_MAX_EXPERTS + 1}, ARG)])


def test_layer_refusals():
    need = kq.kq_mx4_moe_layer_workspace_bytes(64, 96, 2, 2, 8)
    good = dict(xtype=BF16, x=A, wtype=F16, W=A, gc=A, gs=A, uc=A, us=A, dc=A, ds=A, y=A, ids=A, weights=A, hidden=64,
                inter=96, M=2, top_k=2, E=8, renorm=0, ws=A, wsb=need, stream=None)
    cases = bad_k("hidden", kq.KQ_MOE_MAX_DIM) + bad_k("inter", kq.KQ_MOE_MAX_DIM) + ROUTE_CASES
    cases += [({k: None}, ARG) for k in ("gc", "gs", "uc", "us", "dc", "ds", "y")]
    cases += [({k: A + 8}, ALIGN) for k in ("gc", "uc", "dc")] + [({k: A + 2}, ALIGN) for k in ("gs", "us", "ds", "y")]
    cases += [({"wsb": need - 1}, ARG)]
    refuse("kq_mx4_moe_layer", good, cases, [{"M": 0}])
    refuse("kq_mx4_moe_layer_workspace_bytes", dict(hidden=64, inter=96, M=2, top_k=2, E=8),
           [({"hidden": 48}, SHAPE), ({"inter": 0}, SHAPE), ({"M": 65}, ARG), ({"top_k": 9}, ARG), ({"E": 0}, ARG)])


def test_binding_names():
    assert kq.TYPES == {"f32": 0, "f16": 1, "bf16": 2}
    with pytest.raises(KeyError):
        kq.kq_mx4_quantize("f64", A, 64, A, A, 1, 64, stream=0)
    with pytest.raises(kq.KQError):
        kq.kq_mx4_gemv(A, A, "f16", A, A, 16, 33, 1, stream=0)
