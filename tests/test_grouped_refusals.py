"""What the grouped products and the MXFP4 conversions refuse, before anything is launched (no GPU needed), and what they
take as nothing to do."""
import ctypes

import pytest
import torch

import grouped_util as gu

P = 1 << 20  # an aligned address that nothing dereferences


@pytest.fixture(scope="module")
def mb():
    from mixture_experts_decode_moe_amd import binding
    return binding


@pytest.fixture(scope="module")
def lib(mb):
    return mb.raw_lib()


def call(lib, name, defaults, order, **kw):
    a = {**defaults, **kw}
    return getattr(lib, name)(*[a[k] for k in order], None)


Q = dict(x=P, x_type=1, x_ld=64, rows=4, cols=64, q=P, s=P)
D = dict(q=P, s=P, rows=4, cols=64, out=P, out_type=1, out_ld=64)


@pytest.mark.parametrize("kw,rc", [
    (dict(rows=0, x=None), 0), (dict(rows=-1), -1), (dict(cols=0), -1), (dict(x_type=0), -1), (dict(x_type=4), -1),
    (dict(x_ld=63), -1), (dict(x=None), -1), (dict(q=None), -1), (dict(s=None), -1), (dict(x=P + 1), -1),
    (dict(x=P + 2, x_type=3), -1), (dict(q=P + 8), -1), (dict(s=P + 8), -1),
    (dict(cols=2 ** 31 - 1, x_ld=2 ** 31), -2),
])
def test_mx_quantize_refusals(lib, kw, rc):
    assert call(lib, "moe_mx_quantize", Q, Q, **kw) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(rows=0, out=None), 0), (dict(rows=-1), -1), (dict(cols=0), -1), (dict(out_type=9), -1), (dict(out_ld=10), -1),
    (dict(out=None), -1), (dict(q=None), -1), (dict(s=P + 4), -1), (dict(out=P + 2, out_type=3), -1),
])
def test_mx_dequantize_refusals(lib, kw, rc):
    assert call(lib, "moe_mx_dequantize", D, D, **kw) == rc


def mx_args(mb):
    m = mb.MoeMxRows(P, P)
    return dict(x=ctypes.byref(m), T=4, n_rows=4, w=ctypes.byref(m), up=None, E=2, N=40, K=50, offsets=P, row_tok=None,
                row_w=None, out=P, out_type=3, out_ld=40)


def test_mx_grouped_gemm_refusals(mb, lib):
    base = mx_args(mb)
    half, odd = mb.MoeMxRows(P, None), mb.MoeMxRows(P + 8, P)
    for kw, rc in [
        (dict(n_rows=0, T=0), 0), (dict(n_rows=-1), -1), (dict(E=0), -1), (dict(N=0), -1), (dict(K=0), -1),
        (dict(offsets=None), -1), (dict(offsets=P + 2), -1), (dict(E=1025), -2), (dict(N=65537, out_ld=65537), -2),
        (dict(K=65537), -2), (dict(n_rows=2 ** 30 + 7), -2), (dict(out_type=0), -1), (dict(out_ld=39), -1),
        (dict(n_rows=5), -1), (dict(T=-1), -1), (dict(x=None), -1), (dict(w=None), -1), (dict(x=ctypes.byref(half)), -1),
        (dict(w=ctypes.byref(odd)), -1), (dict(up=ctypes.byref(half)), -1), (dict(out=None), -1), (dict(out=P + 2), -1),
        (dict(row_tok=P + 1), -1), (dict(row_w=P + 2), -1),
        # more items than 32 bits count
        (dict(n_rows=2 ** 29, T=2 ** 29, N=65536, out_ld=65536), -2),
    ]:
        assert call(lib, "moe_mx_grouped_gemm", base, base, **kw) == rc, kw


F = dict(x=P, x_ld=64, T=4, n_rows=4, w=P, type=1, E=2, N=40, K=64, offsets=P, row_tok=None, row_w=None, out=P, out_type=3,
         out_ld=40)
X = dict(dy=P, dy_ld=40, n_rows=4, w=P, type=2, E=2, N=40, K=64, offsets=P, dx=P, out_type=2, dx_ld=64)
W = dict(dy=P, dy_ld=40, x=P, x_ld=64, T=4, n_rows=4, type=1, E=2, N=40, K=64, offsets=P, row_tok=None, dw=P, out_type=1, ws=None,
         ws_bytes=0)


@pytest.mark.parametrize("name,base", [("moe_grouped_gemm", F), ("moe_grouped_gemm_dx", X), ("moe_grouped_gemm_dw", W)])
@pytest.mark.parametrize("kw,rc", [
    (dict(n_rows=-1), -1), (dict(E=0), -1), (dict(N=-8), -1), (dict(K=0), -1), (dict(offsets=None), -1), (dict(E=1025), -2),
    (dict(type=0), -1), (dict(type=3, out_type=3), -2), (dict(out_type=7), -1), (dict(N=36), -2), (dict(K=60), -2),
    (dict(n_rows=2 ** 31 - 1), -2),
])
def test_grouped_gemm_common_refusals(lib, name, base, kw, rc):
    assert call(lib, name, base, base, **kw) == rc


@pytest.mark.parametrize("name,base,kw,rc", [
    ("moe_grouped_gemm", F, dict(n_rows=0, T=0, x=None, out=None), 0),
    ("moe_grouped_gemm", F, dict(out_type=2), -2),  # float16 out of bfloat16 rows
    ("moe_grouped_gemm", F, dict(n_rows=5), -1),
    ("moe_grouped_gemm", F, dict(x=None), -1),
    ("moe_grouped_gemm", F, dict(w=P + 8), -1),
    ("moe_grouped_gemm", F, dict(x=P + 8), -1),
    ("moe_grouped_gemm", F, dict(x_ld=56), -1),
    ("moe_grouped_gemm", F, dict(x_ld=68), -2),
    ("moe_grouped_gemm", F, dict(x_ld=2 ** 24 + 8), -2),
    ("moe_grouped_gemm", F, dict(out=P + 4), -1),
    ("moe_grouped_gemm", F, dict(out_ld=44), -2),
    ("moe_grouped_gemm", F, dict(row_w=P + 1), -1),
    ("moe_grouped_gemm_dx", X, dict(n_rows=0, dy=None, dx=None), 0),
    ("moe_grouped_gemm_dx", X, dict(out_type=1), -2),
    ("moe_grouped_gemm_dx", X, dict(dy=None), -1),
    ("moe_grouped_gemm_dx", X, dict(dy_ld=32), -1),
    ("moe_grouped_gemm_dx", X, dict(dx=P + 2), -1),
    ("moe_grouped_gemm_dx", X, dict(dx_ld=72, w=None), -1),
    ("moe_grouped_gemm_dw", W, dict(dw=None), -1),
    ("moe_grouped_gemm_dw", W, dict(dw=P + 4), -1),
    ("moe_grouped_gemm_dw", W, dict(dy=None), -1),
    ("moe_grouped_gemm_dw", W, dict(x=None), -1),
    ("moe_grouped_gemm_dw", W, dict(T=3), -1),
    ("moe_grouped_gemm_dw", W, dict(x_ld=66), -2),
    ("moe_grouped_gemm_dw", W, dict(dy_ld=8), -1),
])
def test_grouped_gemm_refusals(lib, name, base, kw, rc):
    assert call(lib, name, base, base, **kw) == rc


def test_dw_workspace(lib):
    """A few matrices with many rows are summed in parts: the call wants room for them, others want none."""
    size = lib.moe_grouped_gemm_dw_workspace_bytes
    assert size(4096, 64, 512, 1024) == 0 and size(100, 1, 64, 64) == 0 and size(0, 1, 64, 64) == 0
    assert size(-1, 1, 64, 64) == 0 and size(4096, 0, 64, 64) == 0 and size(4096, 1, 65537, 64) == 0
    need = size(16384, 1, 512, 520)
    assert need >= 2 * 512 * 520 * 4
    big = dict(T=16384, n_rows=16384, E=1, N=512, K=520, x_ld=520, dy_ld=512)
    for kw in (dict(), dict(ws=P), dict(ws=P, ws_bytes=need - 1), dict(ws=P + 64, ws_bytes=need)):
        assert call(lib, "moe_grouped_gemm_dw", W, W, **big, **kw) == -3


def test_binding_refuses_host_tensors_and_wrong_kinds(mb):
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        mb.mx_quantize(x, x, x)
    with pytest.raises(TypeError):
        mb.mx_quantize(None, x, x)


def test_plain_mx_codes_round_trip():
    """The oracle's own properties: grid values times a power of two survive, ties go to the even code, the largest
    magnitudes saturate, blocks of zeros and of non-finite values."""
    x = torch.zeros(1, 64)
    x[0, :8] = gu.GRID.float() * 2 ** 5
    x[0, 8:15] = -gu.GRID[1:].float() * 2 ** 5
    q, s = gu.mx_encode(x)
    assert torch.equal(gu.mx_decode(q, s, 64), x.double()) and s[0].tolist() == [127 + 5, 0, 0, 0]
    t = torch.tensor([[0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.9] + [0.0] * 24])
    assert gu.mx_decode(*gu.mx_encode(t), 32)[0, :8].tolist() == [0, 1, 1, 2, 2, 4, 4, 6]
    t[0, 3] = float("inf")
    q, s = gu.mx_encode(t)
    assert int(s[0, 0]) == 255 and not q.any() and gu.mx_decode(q, s, 32).isnan().all()
