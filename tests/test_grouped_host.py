"""Host-side checks of the int8 and grouped products and of the combine: the C ABI's
refusals (each call fails validation or has nothing to do, so no HIP call is made) and the
binding's checks of shapes, dtypes and devices."""
import pytest
import torch

nv = pytest.importorskip("nvfp4_quantized_moe_02_amd")
B = nv.binding

OK, EINVAL, EUNSUP, EWS = 0, -1, -2, -3
P = 0x10000  # 64 KiB-aligned non-null address; never dereferenced by a failing call
F32, BF16, F16 = 0, 1, 2


def linear_i8(x=P, sx=P, T=4, w=P, sw=P, N=64, K=64, out=P, od=F32):
    return B.load_library().nvfp4_linear_i8(x, sx, T, w, sw, N, K, out, od, None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), EINVAL), (dict(sx=None), EINVAL), (dict(w=None), EINVAL), (dict(sw=None), EINVAL),
    (dict(out=None), EINVAL), (dict(T=-1), EINVAL), (dict(N=0), EINVAL), (dict(K=0), EINVAL), (dict(od=3), EINVAL),
    (dict(od=-1), EINVAL), (dict(x=P + 8), EINVAL), (dict(w=P + 4), EINVAL), (dict(out=P + 2), EINVAL),
    (dict(sx=P + 2), EINVAL), (dict(K=24), EUNSUP), (dict(K=131072), EUNSUP), (dict(N=(1 << 20) + 1), EUNSUP),
    (dict(T=(1 << 30) + 1), EUNSUP), (dict(T=1 << 30, N=1 << 20), EUNSUP),
    (dict(T=0, x=None, sx=None, out=None), OK),
])
def test_linear_i8_refusals(kw, want):
    assert linear_i8(**kw) == want


def grouped(x=P, xr=8, w=P, dt=BF16, off=P, E=4, pairs=P, topk=2, rows=16, N=64, K=64, out=P, od=F32):
    return B.load_library().nvfp4_grouped_linear(x, xr, w, dt, off, E, pairs, topk, rows, N, K, out, od, None)


def grouped_i8(x=P, sx=P, xr=8, w=P, sw=P, off=P, E=4, pairs=P, topk=2, rows=16, N=64, K=64, out=P, od=F32):
    return B.load_library().nvfp4_grouped_linear_i8(x, sx, xr, w, sw, off, E, pairs, topk, rows, N, K, out, od, None)


def dx(dy=P, w=P, dt=BF16, off=P, E=4, rows=16, N=64, K=64, out=P, od=F32):
    return B.load_library().nvfp4_grouped_linear_dx(dy, w, dt, off, E, rows, N, K, out, od, None)


def dw(dy=P, x=P, xr=8, dt=BF16, off=P, E=4, pairs=P, topk=2, rows=16, N=64, K=64, out=P, od=F32):
    return B.load_library().nvfp4_grouped_linear_dw(dy, x, xr, dt, off, E, pairs, topk, rows, N, K, out, od, None)


COMMON = [
    (dict(off=None), EINVAL), (dict(E=0), EINVAL), (dict(rows=-1), EINVAL), (dict(N=0), EINVAL), (dict(K=0), EINVAL),
    (dict(out=None), EINVAL), (dict(od=3), EINVAL), (dict(out=P + 8), EINVAL), (dict(off=P + 2), EINVAL),
    (dict(E=8193), EUNSUP), (dict(N=(1 << 20) + 16), EUNSUP), (dict(K=(1 << 20) + 16), EUNSUP),
]
LISTED = [
    (dict(topk=0), EINVAL), (dict(topk=3), EINVAL), (dict(xr=-1), EINVAL), (dict(pairs=None), EINVAL),
    (dict(pairs=P + 1), EINVAL), (dict(xr=1 << 30, topk=2, rows=0), EINVAL),
]
SIXTEEN = [(dict(dt=F32), EUNSUP), (dict(dt=3), EINVAL), (dict(N=12), EUNSUP), (dict(K=12), EUNSUP)]


@pytest.mark.parametrize("fn,kw,want",
                         [(f, k, w) for f in (grouped, grouped_i8, dw) for k, w in COMMON + LISTED]
                         + [(dx, k, w) for k, w in COMMON]
                         + [(f, k, w) for f in (grouped, dx, dw) for k, w in SIXTEEN]
                         + [(f, k, EINVAL) for f in (grouped, dx) for k in (dict(w=None), dict(w=P + 8))]
                         + [(f, k, EINVAL) for f in (grouped, dw) for k in (dict(x=None), dict(x=P + 8))]
                         + [(f, k, EINVAL) for f in (dx, dw) for k in (dict(dy=None), dict(dy=P + 8))]
                         + [(grouped_i8, dict(K=24), EUNSUP), (grouped_i8, dict(K=131072), EUNSUP),
                            (grouped_i8, dict(sw=None), EINVAL), (grouped_i8, dict(sx=P + 1), EINVAL)])
def test_grouped_refusals(fn, kw, want):
    assert fn(**kw) == want


def test_grouped_without_rows_is_a_no_op():
    assert grouped(x=None, xr=0, rows=0, out=None, pairs=None) == OK
    assert grouped_i8(x=None, sx=None, xr=0, rows=0, out=None, pairs=None) == OK
    assert dx(dy=None, rows=0, out=None) == OK


def combine(y=P, yd=BF16, pairs=P, w=P, T=4, topk=2, H=64, out=P, od=F32, ws=P, wsb=1 << 20):
    return B.load_library().nvfp4_moe_combine(y, yd, pairs, w, T, topk, H, out, od, ws, wsb, None)


def combine_grad(dout=P, y=P, yd=BF16, pairs=P, w=P, T=4, topk=2, H=64, out=P, dwt=P, ws=P, wsb=1 << 20):
    return B.load_library().nvfp4_moe_combine_grad(dout, y, yd, pairs, w, T, topk, H, out, dwt, ws, wsb, None)


@pytest.mark.parametrize("fn", [combine, combine_grad])
@pytest.mark.parametrize("kw,want", [
    (dict(y=None), EINVAL), (dict(pairs=None), EINVAL), (dict(out=None), EINVAL), (dict(ws=None, T=1024), EINVAL),
    (dict(T=-1), EINVAL), (dict(topk=0), EINVAL), (dict(H=0), EINVAL), (dict(yd=3), EINVAL), (dict(y=P + 2), EINVAL),
    (dict(out=P + 2), EINVAL), (dict(ws=P + 4), EINVAL), (dict(w=P + 2), EINVAL), (dict(wsb=8191, T=1024), EWS),
    (dict(T=1 << 30, topk=2), EUNSUP), (dict(H=(1 << 20) + 1), EUNSUP), (dict(T=0, y=None, pairs=None, out=None), OK),
])
def test_combine_refusals(fn, kw, want):
    assert fn(**kw) == want


def test_combine_workspace():
    lib = B.load_library()
    assert lib.nvfp4_moe_combine_workspace_size(8192, 8) >= 8192 * 8 * 4
    assert lib.nvfp4_moe_combine_workspace_size(128, 8) == 0  # small lists need none
    assert lib.nvfp4_moe_combine_workspace_size(129, 8) >= 129 * 8 * 4
    assert lib.nvfp4_moe_combine_workspace_size(-1, 8) == 0
    assert lib.nvfp4_moe_combine_workspace_size(1, 0) == 0
    assert combine_grad(dout=None) == EINVAL
    assert combine(od=3) == EINVAL


def test_binding_checks():
    i8, f, i = torch.int8, torch.float32, torch.int32
    x, s = torch.zeros(4, 32, dtype=i8), torch.zeros(4)
    w, sw = torch.zeros(8, 32, dtype=i8), torch.zeros(8)
    h, we = torch.zeros(4, 32, dtype=torch.bfloat16), torch.zeros(2, 8, 32, dtype=torch.bfloat16)
    off, pr = torch.zeros(3, dtype=i), torch.zeros(8, dtype=i)
    bad = [
        lambda: nv.linear_i8(x, s, w[:, :16], sw),                       # K differs
        lambda: nv.linear_i8(x.float(), s, w, sw),                       # dtype
        lambda: nv.linear_i8(x, s[:3], w, sw),                           # scales
        lambda: nv.linear_i8(x, s, w, sw),                               # host tensors
        lambda: nv.linear_i8(x, s, w, sw, out=torch.zeros(4, 9)),        # out's shape
        lambda: nv.grouped_linear(h, we.half(), off),                    # dtypes differ
        lambda: nv.grouped_linear(h, we, off[:2]),                       # offsets
        lambda: nv.grouped_linear(h, we, off, pr, 3),                    # pairs
        lambda: nv.grouped_linear(h, we, off.long()),
        lambda: nv.grouped_linear(h, we, off),                           # host tensors
        lambda: nv.grouped_linear_dx(h, we, off),                        # N differs
        lambda: nv.grouped_linear_dw(h, h[:3], off),                     # rows differ
        lambda: nv.grouped_linear_i8(x, s, w[None], sw, off[:2]),        # w_scale not [E][N]
        lambda: nv.moe_combine(h, pr, 2),                                # list length
        lambda: nv.moe_combine(h, pr[:4], 3),
        lambda: nv.moe_combine(h, pr[:4], 2, torch.zeros(3, 2)),
        lambda: nv.moe_combine(h, pr[:4], 2, ws=torch.zeros(512, dtype=i)),
        lambda: nv.moe_combine_grad(h[:2], h.half(), pr[:4], torch.zeros(2, 2)),
        lambda: nv.moe_combine_grad(h[:2], h, pr, torch.zeros(2, 2)),
    ]
    for k, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {k} was accepted")
