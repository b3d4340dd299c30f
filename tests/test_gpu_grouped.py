"""GPU: MXFP4 conversions bit for bit, grouped products (16-bit with both gradients, MXFP4) against 64-bit sums within
derived bounds, at the sizes, strides, groups and values where they can go wrong."""
import pytest
import torch

import grouped_util as gu

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def say(msg):
    print(f"[gpu] {msg}", flush=True)


@pytest.fixture(scope="module")
def mb():
    from mixture_experts_decode_moe_amd import binding
    return binding


def dev(t):
    return None if t is None else t.cuda()


def strided(t, pad, fill):
    """t on the GPU with `pad` more elements a row, all of them `fill`."""
    base = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=t.dtype, device="cuda")
    base[:, :t.shape[1]] = t
    return base[:, :t.shape[1]]


# ---- MXFP4 ------------------------------------------------------------------

def encode(mb, x, **kw):
    rows, cols = x.shape
    q = torch.full((rows, gu.padded(cols) // 2), 0xAB, dtype=torch.uint8, device="cuda")
    s = torch.full((rows, gu.padded(cols) // 32), 0xCD, dtype=torch.uint8, device="cuda")
    mb.mx_quantize(x, q, s, **kw)
    return q, s


def same_codes(got, want):
    assert torch.equal(got[1].cpu(), want[1])
    assert torch.equal(got[0].cpu(), want[0])


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (3, 31, 0), (5, 33, 3), (7, 128, 0), (17, 200, 8), (130, 2048, 0),
                                           (9, 1000, 24), (4100, 129, 0)])
def test_mx_quantize_bits(mb, dtype, rows, cols, pad):
    g = torch.Generator().manual_seed(rows * 1000 + cols)
    x = torch.randn(rows, cols, generator=g) * torch.exp(2 * torch.randn(rows, 1, generator=g))
    x = x.clamp(-6e4, 6e4).to(dtype)
    say(f"quantise {dtype} {rows}x{cols} pad {pad}")
    xd = strided(x, pad, float("nan"))
    got = encode(mb, xd)
    same_codes(got, gu.mx_encode(x.float()))
    for out_dtype in (F32, BF, HF):
        out = strided(torch.zeros(rows, cols, dtype=out_dtype), pad, 7.0)
        mb.mx_dequantize(*got, out)
        want = gu.mx_decode(got[0].cpu(), got[1].cpu(), cols).to(out_dtype)
        assert torch.equal(out.cpu(), want)
        if pad:  # between the rows nothing is written
            assert bool((out.as_strided((rows, pad), (cols + pad, 1), cols) == 7.0).all())


@pytest.mark.parametrize("dtype", [BF, HF, F32])
def test_mx_rows_at_any_element(mb, dtype):
    """Rows that begin at any element, of every length beside a unit's and a lane's end, in every phase of 16 bytes."""
    say(f"rows at any element {dtype}")
    g = torch.Generator().manual_seed(11)
    for cols in (1, 2, 5, 7, 8, 9, 15, 17, 31, 63, 65, 127, 129, 135, 137, 257):
        for first in (1, 2, 3):
            ld = cols + first
            x = torch.randn(6, cols, generator=g).to(dtype)
            base = torch.full((first + 6 * ld,), float("nan"), dtype=dtype, device="cuda")
            rows = base.as_strided((6, cols), (ld, 1), first)
            rows.copy_(x)
            got = encode(mb, rows)
            same_codes(got, gu.mx_encode(x.float()))
            base.fill_(7.0)
            mb.mx_dequantize(*got, rows)
            assert torch.equal(rows.cpu(), gu.mx_decode(got[0].cpu(), got[1].cpu(), cols).to(dtype))
            left = torch.ones(base.numel(), dtype=torch.bool)
            left.as_strided((6, cols), (ld, 1), first).fill_(False)
            assert bool((base.cpu()[left] == 7.0).all())


def test_mx_quantize_every_16_bit_value(mb):
    """Every finite bfloat16 and float16 value as a block's largest and beside larger ones, and the borders of the grid
    at both ends of fp32's range."""
    say("quantise: all 16-bit values")
    for dtype in (BF, HF):
        v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dtype)
        v = v[torch.isfinite(v)]
        x = torch.zeros(v.numel(), 64, dtype=dtype)
        x[:, 0] = v
        x[:, 32] = v
        x[:, 40] = torch.roll(v, 1)
        x[:, 63] = torch.roll(v, 77)
        same_codes(encode(mb, x.cuda()), gu.mx_encode(x.float()))
    border = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0])
    around = torch.cat([border, torch.nextafter(border, torch.zeros(9)), torch.nextafter(border, torch.full((9,), 9.0))])
    x = torch.zeros(250, 32)
    for i, e in enumerate(range(-126, 124)):
        x[i, :27] = torch.ldexp(around * torch.where(torch.arange(27) % 2 == 0, 1.0, -1.0), torch.tensor(e))
        x[i, 27] = torch.ldexp(torch.tensor(4.5), torch.tensor(e))
    same_codes(encode(mb, x.cuda()), gu.mx_encode(x))


def test_mx_quantize_non_finite_denormal_and_zero_blocks(mb):
    x = torch.randn(6, 160, generator=torch.Generator().manual_seed(1))
    x[0, 3] = float("inf")
    x[1, 40] = float("-inf")
    x[2, 159] = float("nan")
    x[3] = 0
    x[4, 5:9] = -0.0
    x[5] = torch.randint(-9, 9, (160,), generator=torch.Generator().manual_seed(2)) * 2.0 ** -149  # fp32's smallest steps
    say("quantise: non-finite, denormal, zero")
    got = encode(mb, x.cuda())
    same_codes(got, gu.mx_encode(x))
    out = torch.empty(6, 160, device="cuda")
    mb.mx_dequantize(*got, out)
    assert torch.equal(out.cpu().isnan(), gu.mx_decode(*gu.mx_encode(x), 160).isnan())


def test_mx_dequantize_every_code_and_scale(mb):
    """All 16 codes under all 256 scales, in the three types: exact but for the type's own rounding."""
    say("dequantise: every code and scale")
    q = torch.zeros(256, 64, dtype=torch.uint8)
    q[:, :8] = torch.arange(8, dtype=torch.uint8) * 2 + (torch.arange(8, dtype=torch.uint8) * 2 + 1) * 16
    s = torch.arange(256, dtype=torch.uint8)[:, None].expand(256, 4).contiguous()
    want = gu.mx_decode(q, s, 16)
    for dtype in (F32, BF, HF):
        out = torch.empty(256, 16, dtype=dtype, device="cuda")
        mb.mx_dequantize(q.cuda(), s.cuda(), out)
        assert torch.equal(torch.nan_to_num(out.cpu(), nan=77.0), torch.nan_to_num(want.to(dtype), nan=77.0))


# ---- grouped products -----------------------------------------------------------

def cases():
    """(label, E, offsets or None, n_rows): groups of length zero and one, beside and across tile borders, one large
    group among empty ones, rows before the first group and behind the last, more experts than rows."""
    def off(counts, first=0):
        return torch.tensor([first] + counts, dtype=torch.int32).cumsum(0).to(torch.int32)

    g = torch.Generator().manual_seed(5)
    many = torch.zeros(1024, dtype=torch.int64)
    many[torch.randperm(1024, generator=g)[:40]] = 1
    many[1023] = 3
    return [
        ("one expert, one row", 1, None, 1),
        ("one expert, no offsets", 1, None, 200),
        ("no rows in any group", 3, off([0, 0, 0]), 5),
        ("ragged", 7, off([130, 0, 127, 1, 64, 16, 300]), 638),
        ("rows outside the groups", 5, off([17, 0, 33, 2, 15], first=6), 90),
        ("decode", 64, off(torch.bincount(torch.randint(0, 64, (40,), generator=g), minlength=64).tolist()), 40),
        ("1024 experts", 1024, off(many.tolist()), int(many.sum())),
        ("many rows", 5, off([700, 0, 1301, 1, 897], first=9), 2920),
        ("many groups", 150, off(torch.bincount(torch.randint(0, 150, (2400,), generator=g) // 2 * 2, minlength=150)
                                 .tolist()), 2409),
    ]


CASES = {c[0]: c for c in cases()}


def tokens(n_rows, T, seed):
    """Source rows with repeats and some out of range (they read zeros)."""
    t = torch.randint(0, T, (n_rows,), generator=torch.Generator().manual_seed(seed), dtype=torch.int32)
    if n_rows > 8:
        t[1], t[5], t[7] = -1, T, t[6]
    return t


def check(out, ref, mag, used, dtype, length, step, label):
    """Rows in groups within the bound, the others as they were (7)."""
    got = out.cpu().double()
    assert bool((got[~used] == 7.0).all()), "rows outside the groups were written"
    limit = gu.rounded(ref, gu.sum_bound(mag, length, step), dtype)
    diff = (got - ref).abs()[used]
    worst = float((diff / limit[used]).max()) if diff.numel() else 0.0
    say(f"  {label}: at most {worst:.2f} of the bound")
    assert bool((diff <= limit[used]).all())


@pytest.mark.parametrize("label", list(CASES))
@pytest.mark.parametrize("N,K,dtype,out_dtype", [(8, 8, BF, F32), (136, 72, HF, HF), (264, 1000, BF, BF)])
def test_grouped_gemm(mb, label, N, K, dtype, out_dtype):
    _, E, offsets, n_rows = CASES[label]
    g = torch.Generator().manual_seed(N + n_rows)
    for gather in (False, True):
        say(f"grouped_gemm {label} N={N} K={K} {dtype} gather={gather}")
        T = n_rows if not gather else max(1, n_rows // 3)
        x = torch.randn(T, K, generator=g).to(dtype)
        w = (torch.randn(E, N, K, generator=g) / K ** 0.5).to(dtype)
        tok = tokens(n_rows, T, 3) if gather else None
        row_w = torch.rand(n_rows, generator=g) if gather else None
        out = strided(torch.full((n_rows, N), 7.0, dtype=out_dtype), 8, 7.0)
        mb.grouped_gemm(strided(x, 16, float("nan")), dev(w), dev(offsets), out, row_tok=dev(tok), row_w=dev(row_w))
        y, m = gu.product(gu.gathered(x, tok, n_rows), w.double(), offsets, n_rows)
        if row_w is not None:
            y, m = y * row_w[:, None].double(), m * row_w[:, None].double() * (1 + 2.0 ** -10)
        check(out, y, m, gu.in_groups(offsets, n_rows), out_dtype, K, 32, label)


@pytest.mark.parametrize("label", list(CASES))
@pytest.mark.parametrize("N,K,dtype,out_dtype", [(8, 8, HF, F32), (72, 136, BF, BF), (1000, 264, HF, HF)])
def test_grouped_gemm_dx(mb, label, N, K, dtype, out_dtype):
    _, E, offsets, n_rows = CASES[label]
    say(f"grouped_gemm_dx {label} N={N} K={K} {dtype}")
    g = torch.Generator().manual_seed(N + n_rows)
    dy = torch.randn(n_rows, N, generator=g).to(dtype)
    w = (torch.randn(E, N, K, generator=g) / N ** 0.5).to(dtype)
    out = strided(torch.full((n_rows, K), 7.0, dtype=out_dtype), 8, 7.0)
    mb.grouped_gemm_dx(strided(dy, 8, float("nan")), dev(w), dev(offsets), out)
    y, m = gu.product(dy.double(), w.double().transpose(1, 2).contiguous(), offsets, n_rows)
    check(out, y, m, gu.in_groups(offsets, n_rows), out_dtype, N, 32, label)


@pytest.mark.parametrize("label", list(CASES))
@pytest.mark.parametrize("N,K,dtype,out_dtype", [(8, 8, BF, BF), (136, 200, HF, F32)])
def test_grouped_gemm_dw(mb, label, N, K, dtype, out_dtype):
    _, E, offsets, n_rows = CASES[label]
    g = torch.Generator().manual_seed(N + n_rows)
    used = gu.in_groups(offsets, n_rows)
    for gather in (False, True):
        say(f"grouped_gemm_dw {label} N={N} K={K} {dtype} gather={gather}")
        T = n_rows if not gather else max(1, n_rows // 3)
        x = torch.randn(T, K, generator=g).to(dtype)
        dy = torch.randn(n_rows, N, generator=g).to(dtype)
        tok = tokens(n_rows, T, 4) if gather else None
        rows = gu.gathered(x, tok, n_rows)
        ref = torch.zeros(E, N, K, dtype=torch.float64)
        mag = torch.zeros_like(ref)
        most = 0
        for e, a, b in gu.groups(offsets, n_rows, E):
            ref[e] = dy[a:b].double().T @ rows[a:b]
            mag[e] = dy[a:b].double().abs().T @ rows[a:b].abs()
            most = max(most, b - a)
        dy = dy.clone()
        dy[~used] = float("nan")  # rows of no group reach no sum
        out = torch.full((E, N, K), 7.0, dtype=out_dtype, device="cuda")
        mb.grouped_gemm_dw(strided(dy, 8, float("nan")), strided(x, 8, float("nan")), dev(offsets), out, row_tok=dev(tok))
        limit = gu.rounded(ref, gu.sum_bound(mag, max(1, most), 32), out_dtype)
        diff = (out.cpu().double() - ref).abs()
        assert bool((diff <= limit).all())


@pytest.mark.parametrize("counts,N,K,dtype,out_dtype", [([5000], 136, 264, BF, BF), ([3001], 8, 8, HF, F32),
                                                        ([4000, 0, 17, 2300], 128, 200, HF, HF)])
def test_grouped_gemm_dw_in_parts(mb, counts, N, K, dtype, out_dtype):
    """Few small matrices with many rows: the rows are summed in parts; ragged, empty and short groups; a workspace of the
    caller's, and a graph."""
    rows, E = sum(counts), len(counts)
    say(f"dw in parts {counts} N={N} K={K}")
    need = mb.grouped_gemm_dw_workspace_bytes(rows, E, N, K)
    assert need > 0
    g = torch.Generator().manual_seed(rows)
    off = torch.tensor([0] + counts).cumsum(0).to(torch.int32)
    tok = tokens(rows, 700, 6)
    x, dy = torch.randn(700, K, generator=g).to(dtype), torch.randn(rows, N, generator=g).to(dtype)
    xr = gu.gathered(x, tok, rows)
    ref = torch.stack([dy[a:b].double().T @ xr[a:b] for _, a, b in gu.groups(off, rows, E)])
    mag = torch.stack([dy[a:b].double().abs().T @ xr[a:b].abs() for _, a, b in gu.groups(off, rows, E)])
    args = dev(dy), dev(x), dev(off)
    out = torch.full((E, N, K), 7.0, dtype=out_dtype, device="cuda")
    mb.grouped_gemm_dw(*args, out, row_tok=dev(tok))
    # a part is a shorter sum; the parts are at most 16 more additions
    limit = gu.rounded(ref, gu.sum_bound(mag, rows, 32) + 16 * 2.0 ** -24 * mag, out_dtype)
    assert bool(((out.cpu().double() - ref).abs() <= limit).all())
    first = out.clone()
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    t = dev(tok)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mb.grouped_gemm_dw(*args, out, row_tok=t, ws=ws)
    for _ in range(3):
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first) and bool((ws[need:] == 0xFF).all())


@pytest.mark.parametrize("E,N,K,dtype,out_dtype", [(12, 520, 1000, BF, BF), (33, 1032, 1800, HF, HF)])
@pytest.mark.parametrize("heavy", [0, -1])
def test_grouped_gemm_dw_uneven_groups(mb, E, N, K, dtype, out_dtype, heavy):
    """One group with most of the rows, first or last, empty ones and short ones: every tile is made, by one block."""
    counts = [0 if e % 3 == 1 else 5 + e for e in range(E)]
    counts[heavy] = 1500
    off = torch.tensor([3] + counts, dtype=torch.int32).cumsum(0).to(torch.int32)
    n_rows = int(off[-1]) + 2
    say(f"dw uneven E={E} N={N} K={K} {dtype} heavy={heavy}")
    g = torch.Generator().manual_seed(E + heavy)
    dy, x = torch.randn(n_rows, N, generator=g).to(dtype), torch.randn(n_rows, K, generator=g).to(dtype)
    out = torch.full((E, N, K), 7.0, dtype=out_dtype, device="cuda")
    mb.grouped_gemm_dw(dev(dy), dev(x), dev(off), out)
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        p, q = dy[a:b].double(), x[a:b].double()
        ref = p.T @ q
        limit = gu.rounded(ref, gu.sum_bound(p.abs().T @ q.abs(), max(1, b - a), 32), out_dtype)
        assert bool(((out[e].cpu().double() - ref).abs() <= limit).all()), e


def test_grouped_gemm_dw_without_rows_is_zero(mb):
    say("dw, n_rows = 0")
    out = torch.full((3, 16, 24), 7.0, device="cuda")
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    mb.grouped_gemm_dw(torch.empty(0, 16, dtype=BF, device="cuda"), torch.ones(5, 24, dtype=BF, device="cuda"), off, out)
    assert not bool(out.any())


@pytest.mark.parametrize("label", list(CASES))
@pytest.mark.parametrize("N,K,swiglu,out_dtype", [(1, 1, False, F32), (7, 33, True, BF), (130, 200, False, HF),
                                                  (129, 520, True, F32), (256, 512, False, BF)])
def test_mx_grouped_gemm(mb, label, N, K, swiglu, out_dtype):
    _, E, offsets, n_rows = CASES[label]
    if E == 1024:
        N = min(N, 40)
    g = torch.Generator().manual_seed(N + n_rows + K)
    for gather in (False, True):
        say(f"mx_grouped_gemm {label} N={N} K={K} swiglu={swiglu} gather={gather}")
        T = n_rows if not gather else max(1, n_rows // 3)

        def codes(rows, scale):
            return gu.mx_encode(torch.randn(rows, K, generator=g) * scale * torch.exp(torch.randn(rows, 1, generator=g)))

        x, w, up = codes(T, 1.0), codes(E * N, K ** -0.5), codes(E * N, K ** -0.5) if swiglu else None
        tok = tokens(n_rows, T, 5) if gather else None
        row_w = torch.rand(n_rows, generator=g) if gather else None
        out = strided(torch.full((n_rows, N), 7.0, dtype=out_dtype), 5 if N % 2 else 8, 7.0)
        mb.mx_grouped_gemm((dev(x[0]), dev(x[1])), (dev(w[0]), dev(w[1])), E, K, dev(offsets), out,
                           up=None if up is None else (dev(up[0]), dev(up[1])), row_tok=dev(tok), row_w=dev(row_w))
        rows = gu.gathered(gu.mx_decode(*x, K), tok, n_rows)
        y, m = gu.product(rows, gu.mx_decode(*w, K).reshape(E, N, K), offsets, n_rows)
        m = gu.sum_bound(m, K, 128)
        if swiglu:
            u, mu = gu.product(rows, gu.mx_decode(*up, K).reshape(E, N, K), offsets, n_rows)
            mu = gu.sum_bound(mu, K, 128)
            # |silu'| <= 1.1; the exponential, the quotient and the products round a few times (2^-20 in all)
            a = gu.silu(y)
            m = 1.1 * m * (u.abs() + mu) + (a.abs() + 1.1 * m) * mu + 2.0 ** -20 * (a * u).abs()
            y = a * u
        if row_w is not None:
            y, m = y * row_w[:, None].double(), (m + 2.0 ** -23 * y.abs()) * row_w[:, None].double()
        got = out.cpu().double()
        used = gu.in_groups(offsets, n_rows)
        assert bool((got[~used] == 7.0).all())
        limit = gu.rounded(y, m, out_dtype)
        assert bool(((got - y).abs()[used] <= limit[used]).all())
        pad = out.as_strided((n_rows, 5 if N % 2 else 8), (out.stride(0), 1), N)
        assert bool((pad == 7.0).all())


@pytest.mark.parametrize("K", [1016, 1024, 1032, 4096, 5000])
def test_long_reductions_of_few_rows(mb, K):
    """Reductions that several waves share, the last of them with a part, a whole share or none."""
    off = torch.tensor([0, 17, 17, 18, 40], dtype=torch.int32)
    g = torch.Generator().manual_seed(K)
    for dtype in (BF, HF):
        say(f"long reductions K={K} {dtype}")
        x, w = torch.randn(41, K, generator=g).to(dtype), (torch.randn(4, 40, K, generator=g) / K ** 0.5).to(dtype)
        out = torch.full((41, 40), 7.0, device="cuda")
        mb.grouped_gemm(strided(x, 8, float("nan")), dev(w), dev(off), out)
        y, m = gu.product(x.double(), w.double(), off, 41)
        check(out, y, m, gu.in_groups(off, 41), F32, K, 32, f"K={K}")
    for k in (4 * K, 4 * K + 33):  # as many bytes a row, and an odd end
        x, w = gu.mx_encode(torch.randn(41, k, generator=g)), gu.mx_encode(torch.randn(4 * 40, k, generator=g))
        out = torch.full((41, 40), 7.0, device="cuda")
        mb.mx_grouped_gemm((dev(x[0]), dev(x[1])), (dev(w[0]), dev(w[1])), 4, k, dev(off), out)
        y, m = gu.product(gu.mx_decode(*x, k), gu.mx_decode(*w, k).reshape(4, 40, k), off, 41)
        check(out, y, m, gu.in_groups(off, 41), F32, k, 128, f"MXFP4 K={k}")


@pytest.mark.parametrize("wide,odd", [(264, 257), (1096, 1090)])
def test_as_many_tiles_as_compute_units(mb, wide, odd):
    """Calls of up to one tile a compute unit, of 64 columns and of 128, with reductions of up to ten steps."""
    _, E, off, rows = CASES["many rows"]
    g = torch.Generator().manual_seed(wide)
    used = gu.in_groups(off, rows)
    for k in (72, 640):
        for dtype, out_dtype in ((BF, BF), (HF, F32)):
            say(f"one tile a unit {wide} k={k} {dtype}")
            x, w = torch.randn(rows, k, generator=g).to(dtype), torch.randn(E, wide, k, generator=g).to(dtype)
            out = torch.full((rows, wide), 7.0, dtype=out_dtype, device="cuda")
            mb.grouped_gemm(strided(x, 8, float("nan")), dev(w), dev(off), out)
            check(out, *gu.product(x.double(), w.double(), off, rows), used, out_dtype, k, 32, "fwd")
            wt = w.transpose(1, 2).contiguous()  # [E][k][wide]
            out.fill_(7.0)
            mb.grouped_gemm_dx(strided(x, 8, float("nan")), dev(wt), dev(off), out)
            check(out, *gu.product(x.double(), w.double(), off, rows), used, out_dtype, k, 32, "dx")
        kx = 4 * k + 5
        x, w = gu.mx_encode(torch.randn(rows, kx, generator=g)), gu.mx_encode(torch.randn(E * odd, kx, generator=g))
        out = torch.full((rows, odd), 7.0, dtype=BF, device="cuda")
        mb.mx_grouped_gemm((dev(x[0]), dev(x[1])), (dev(w[0]), dev(w[1])), E, kx, dev(off), out)
        x64, w64 = gu.mx_decode(*x, kx), gu.mx_decode(*w, kx).reshape(E, odd, kx)
        check(out, *gu.product(x64, w64, off, rows), used, BF, kx, 128, "MXFP4")
        # SwiGLU of a product with itself: silu(p) p, half of the columns
        half = odd // 2
        part = [t.reshape(E, odd, -1)[:, :half].contiguous() for t in w]
        out = torch.full((rows, half), 7.0, device="cuda")
        m = (dev(part[0]), dev(part[1]))
        mb.mx_grouped_gemm((dev(x[0]), dev(x[1])), m, E, kx, dev(off), out, up=m)
        y, mag = gu.product(x64, w64[:, :half], off, rows)
        err = gu.sum_bound(mag, kx, 128)
        a = gu.silu(y)
        # as in test_mx_grouped_gemm: |silu'| <= 1.1, both factors off by err
        limit = 1.1 * err * (y.abs() + err) + (a.abs() + 1.1 * err) * err + 2.0 ** -20 * (a * y).abs()
        got = out.cpu().double()
        assert bool((got[~used] == 7.0).all())
        assert bool(((got - a * y).abs()[used] <= gu.rounded(a * y, limit, F32)[used]).all())


@pytest.mark.parametrize("op", ["gemm", "gemm_dx", "gemm_dw"])
@pytest.mark.parametrize("dtype,out_dtype", [(BF, F32), (HF, HF)])
def test_many_tiles(mb, op, dtype, out_dtype):
    """Calls of more than four wide tiles a compute unit, and of more than 32 for a block; widths that end inside one."""
    say(f"many tiles {op} {dtype}")
    g = torch.Generator().manual_seed(31)
    for E, wide, other, rows in ((1024, 2312, 16, 1060), (40, 7048, 72, 900)):
        counts = torch.bincount(torch.randint(0, E, (rows,), generator=g), minlength=E)
        off = torch.cat([torch.zeros(1), counts.cumsum(0)]).to(torch.int32)
        N, K = (other, wide) if op == "gemm_dx" else (wide, other)
        x = torch.randn(rows, K, generator=g).to(dtype)
        dy = torch.randn(rows, N, generator=g).to(dtype)
        w = torch.randn(E, N, K, generator=g).to(dtype)
        if op == "gemm_dw":
            out = torch.full((E, N, K), 7.0, dtype=out_dtype, device="cuda")
            mb.grouped_gemm_dw(dev(dy), dev(x), dev(off), out)
            for e, a, b in gu.groups(off, rows, E):
                ref = dy[a:b].double().T @ x[a:b].double()
                mag = dy[a:b].double().abs().T @ x[a:b].double().abs()
                limit = gu.rounded(ref, gu.sum_bound(mag, max(1, b - a), 32), out_dtype)
                assert bool(((out[e].cpu().double() - ref).abs() <= limit).all())
            continue
        out = torch.full((rows, wide), 7.0, dtype=out_dtype, device="cuda")
        if op == "gemm":
            mb.grouped_gemm(dev(x), dev(w), dev(off), out)
            y, m = gu.product(x.double(), w.double(), off, rows)
        else:
            mb.grouped_gemm_dx(dev(dy), dev(w), dev(off), out)
            y, m = gu.product(dy.double(), w.double().transpose(1, 2), off, rows)
        check(out, y, m, gu.in_groups(off, rows), out_dtype, other, 32, f"E={E}")


def test_mx_many_tiles(mb):
    """More than 32 tiles a block; codes and scales drawn as bytes."""
    say("MXFP4, many tiles")
    g = torch.Generator().manual_seed(33)
    E, N, K, rows = 1024, 1092, 40, 1100
    off = torch.cat([torch.zeros(1), torch.bincount(torch.randint(0, E, (rows,), generator=g), minlength=E).cumsum(0)]).to(torch.int32)

    def draw(n):
        q = torch.randint(0, 256, (n, 64), generator=g, dtype=torch.uint8)
        q[:, K // 2:] = 0
        return q, torch.randint(120, 130, (n, 4), generator=g, dtype=torch.uint8)

    x, w, up = draw(rows), draw(E * N), draw(E * N)
    out = torch.full((rows, N), 7.0, device="cuda")
    mb.mx_grouped_gemm(tuple(map(dev, x)), tuple(map(dev, w)), E, K, dev(off), out, up=tuple(map(dev, up)))
    xr = gu.mx_decode(*x, K)
    y, m = gu.product(xr, gu.mx_decode(*w, K).reshape(E, N, K), off, rows)
    u, mu = gu.product(xr, gu.mx_decode(*up, K).reshape(E, N, K), off, rows)
    m, mu, a = gu.sum_bound(m, K, 128), gu.sum_bound(mu, K, 128), gu.silu(y)
    m = 1.1 * m * (u.abs() + mu) + (a.abs() + 1.1 * m) * mu + 2.0 ** -20 * (a * u).abs()
    # below -87 the exponential leaves fp32 and the result, at most 2^-118 of u, may become zero
    m = m + torch.where(y < -80, 2.0 ** -100 * u.abs(), 0.0)
    assert bool(((out.cpu().double() - a * u).abs() <= gu.rounded(a * u, m, F32)).all())


def test_places_past_32_bits(mb):
    """Rows and matrices that lie more than 2^32 bytes into their arrays."""
    say("places past 32 bits")
    g = torch.Generator().manual_seed(35)
    K, T = 2048, (1 << 20) + 64  # 4.3 GB of rows
    x = torch.empty(T, K, dtype=BF, device="cuda")
    at = torch.tensor([T - 1, 5, T - 64, 1 << 19], dtype=torch.int32)
    rows = torch.randn(4, K, generator=g).to(BF)
    x[at.long().cuda()] = dev(rows)
    E, N = 600, 2048  # 5 GB of matrices
    w = torch.empty(E, N, K, dtype=BF, device="cuda")
    used = torch.randn(2, N, K, generator=g).to(BF)
    w[3], w[E - 1] = dev(used[0]), dev(used[1])
    counts = torch.zeros(E, dtype=torch.int64)
    counts[3], counts[E - 1] = 1, 3
    off = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]).to(torch.int32)
    ref = torch.cat([rows[:1].double() @ used[0].double().T, rows[1:].double() @ used[1].double().T])
    mag = torch.cat([rows[:1].double().abs() @ used[0].double().abs().T, rows[1:].double().abs() @ used[1].double().abs().T])
    limit = gu.rounded(ref, gu.sum_bound(mag, K, 32), F32)
    for more in (0, 300):  # the few-row kernel, and the tiles (with rows of token 5 for company)
        tok = torch.cat([torch.full((more,), 5, dtype=torch.int32), at])
        offsets = off + more * (torch.arange(E + 1) > 0).to(torch.int32)
        out = torch.empty(4 + more, N, device="cuda")
        w[0] = 0
        mb.grouped_gemm(x, w, dev(offsets.to(torch.int32)), out, row_tok=dev(tok))
        assert bool(((out[more:].cpu().double() - ref).abs() <= limit).all())
    dy = torch.randn(4, N, generator=g).to(BF)
    dx = torch.empty(4, K, device="cuda")
    mb.grouped_gemm_dx(dev(dy), w, dev(off), dx)
    ref = torch.cat([dy[:1].double() @ used[0].double(), dy[1:].double() @ used[1].double()])
    mag = torch.cat([dy[:1].double().abs() @ used[0].double().abs(), dy[1:].double().abs() @ used[1].double().abs()])
    assert bool(((dx.cpu().double() - ref).abs() <= gu.rounded(ref, gu.sum_bound(mag, N, 32), F32)).all())
    del w
    dw = torch.full((E, N, K), 7.0, dtype=BF, device="cuda")
    mb.grouped_gemm_dw(dev(dy), x, dev(off), dw, row_tok=dev(at))
    ref = dy[1:].double().T @ rows[1:].double()
    mag = dy[1:].double().abs().T @ rows[1:].double().abs()
    assert bool(((dw[E - 1].cpu().double() - ref).abs() <= gu.rounded(ref, gu.sum_bound(mag, 3, 32), BF)).all())
    assert not bool(dw[E - 2].any())


@pytest.mark.parametrize("dtype", [BF, HF])
def test_small_and_large_values(mb, dtype):
    """Denormal 16-bit values count, infinities and NaN spread as the sums do."""
    say(f"denormals, infinities {dtype}")
    for rows in (4, 300):
        tiny = torch.finfo(dtype).smallest_normal / 4
        x = torch.full((rows, 64), tiny, dtype=dtype)
        w = torch.full((1, 16, 64), 1.0 if dtype == HF else 2.0 ** 20, dtype=dtype)
        out = torch.empty(rows, 16, device="cuda")
        mb.grouped_gemm(dev(x), dev(w), None, out)
        assert torch.equal(out.cpu().double(), x.double() @ w[0].double().T)
        x = torch.ones(rows, 64, dtype=dtype)
        x[1, 3], x[2, 5], x[3, 7], x[3, 8] = float("inf"), float("nan"), float("inf"), float("-inf")
        mb.grouped_gemm(dev(x), dev(w), None, out)
        got = out.cpu()
        assert bool((got[1] == float("inf")).all()) and bool(got[2:4].isnan().all()) and bool(got[0].isfinite().all())


def test_mx_nan_blocks_reach_only_their_sums(mb):
    """A NaN block of one row makes that row NaN, one of a weight row that column; infinities in 16 bits likewise."""
    say("NaN blocks")
    g = torch.Generator().manual_seed(9)
    x, w = torch.randn(40, 200, generator=g), torch.randn(70, 200, generator=g)
    x[3, 150] = float("inf")
    w[66, 10] = float("nan")
    out = torch.empty(40, 70, device="cuda")
    mb.mx_grouped_gemm(tuple(map(dev, gu.mx_encode(x))), tuple(map(dev, gu.mx_encode(w))), 1, 200, None, out)
    want = torch.zeros(40, 70, dtype=torch.bool)
    want[3], want[:, 66] = True, True
    assert torch.equal(out.isnan().cpu(), want)


def test_offsets_outside_the_rows_are_clamped(mb):
    """Offsets below zero, above n_rows or falling leave memory alone: groups are cut to the rows there are."""
    say("bad offsets")
    x = torch.randn(20, 64, generator=torch.Generator().manual_seed(2)).to(BF)
    w = torch.randn(4, 16, 64, generator=torch.Generator().manual_seed(3)).to(BF)
    off = torch.tensor([-7, 5, 3, 12, 4000], dtype=torch.int32)
    out = torch.full((24, 16), 7.0, device="cuda")
    mb.grouped_gemm(dev(x), dev(w), dev(off), out[:20])
    want = torch.tensor([0, 5, 5, 12, 20], dtype=torch.int32)  # rows 3..4 belong to experts 0 and 2
    y, m = gu.product(x.double(), w.double(), want, 20)
    sure = torch.ones(20, dtype=torch.bool)
    sure[3:5] = False
    diff = (out[:20].cpu().double() - y).abs()[sure]
    assert bool((diff <= gu.rounded(y, gu.sum_bound(m, 64, 32), F32)[sure]).all())
    assert bool((out[20:] == 7.0).all())


# ---- as they are used -----------------------------------------------------------

def route(mb, T, E, topk, seed):
    """A permutation by expert from moe_permute."""
    g = torch.Generator().manual_seed(seed)
    ids = torch.stack([torch.randperm(E, generator=g)[:topk] for _ in range(T)]).to(torch.int32).cuda()
    wts = torch.rand(T, topk, generator=g).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    out = {"counts": torch.empty(E, **i32), "offsets": torch.empty(E + 1, **i32), "row_tok": torch.empty(T * topk, **i32),
           "row_w": torch.empty(T * topk, device="cuda"), "inv_pos": torch.empty(T, topk, **i32),
           "active": torch.empty(E, **i32), "n_active": torch.empty(1, **i32)}
    ws = torch.empty(mb.permute_workspace_bytes(T, topk, E), dtype=torch.uint8, device="cuda")
    mb.permute(ids, wts, E, out, ws)
    return out


class MxLayer:
    """The routed experts on MXFP4: tokens quantised once, gate/up with SwiGLU, quantised again, down, combined."""

    def __init__(self, mb, T, E, topk, H, F, seed):
        g = torch.Generator().manual_seed(seed)
        self.mb, self.T, self.E, self.topk, self.H, self.F = mb, T, E, topk, H, F
        self.p = route(mb, T, E, topk, seed)
        self.x = torch.randn(T, H, generator=g).to(BF).cuda()
        self.w = {n: (torch.randn(E, r, c, generator=g) / c ** 0.5) for n, r, c in
                  (("gate", F, H), ("up", F, H), ("down", H, F))}
        self.q = {n: encode(mb, w.reshape(-1, w.shape[2]).cuda()) for n, w in self.w.items()}
        rows = T * topk
        u8 = dict(dtype=torch.uint8, device="cuda")
        self.xq = (torch.empty(T, gu.padded(H) // 2, **u8), torch.empty(T, gu.padded(H) // 32, **u8))
        self.aq = (torch.empty(rows, gu.padded(F) // 2, **u8), torch.empty(rows, gu.padded(F) // 32, **u8))
        self.act = torch.empty(rows, F, dtype=BF, device="cuda")
        self.rows = torch.empty(rows, H, device="cuda")
        self.y = torch.empty(T, H, device="cuda")

    def run(self, stream=None):
        mb, p = self.mb, self.p
        mb.mx_quantize(self.x, *self.xq, stream=stream)
        mb.mx_grouped_gemm(self.xq, self.q["gate"], self.E, self.H, p["offsets"], self.act, up=self.q["up"],
                           row_tok=p["row_tok"], stream=stream)
        mb.mx_quantize(self.act, *self.aq, stream=stream)
        mb.mx_grouped_gemm(self.aq, self.q["down"], self.E, self.F, p["offsets"], self.rows, row_w=p["row_w"], stream=stream)
        mb.combine(self.rows, p["inv_pos"], self.T, self.topk, self.H, None, self.y, stream=stream)
        return self.y


@pytest.mark.parametrize("T", [1, 16, 300])
def test_mx_layer(mb, T):
    """Each stage of the run against 64 bits on the stage's own inputs."""
    say(f"MXFP4 layer T={T}")
    L = MxLayer(mb, T, 32, 4, 512, 256, 40 + T)
    y = L.run().cpu().double()
    off, tok = L.p["offsets"].cpu(), L.p["row_tok"].cpu()
    n = T * 4
    same_codes(L.xq, gu.mx_encode(L.x.cpu().float()))
    same_codes(L.aq, gu.mx_encode(L.act.cpu().float()))
    dec = {k: gu.mx_decode(v[0].cpu(), v[1].cpu(), L.w[k].shape[2]).reshape(L.w[k].shape) for k, v in L.q.items()}
    xr = gu.gathered(gu.mx_decode(L.xq[0].cpu(), L.xq[1].cpu(), 512), tok, n)
    a, _ = gu.product(xr, dec["gate"], off, n)
    u, _ = gu.product(xr, dec["up"], off, n)
    act = gu.silu(a) * u
    assert float((L.act.cpu().double() - act).norm() / act.norm()) < 2.0 ** -8
    ar = gu.mx_decode(L.aq[0].cpu(), L.aq[1].cpu(), 256)
    d, m = gu.product(ar, dec["down"], off, n)
    rw = L.p["row_w"].cpu().double()[:, None]
    d, m = d * rw, (gu.sum_bound(m, 256, 128) + 2.0 ** -23 * d.abs()) * rw
    assert bool(((L.rows.cpu().double() - d).abs() <= gu.rounded(d, m, F32)).all())
    inv = L.p["inv_pos"].cpu().long()
    ref = L.rows.cpu().double()[inv].sum(1)
    assert bool(((y - ref).abs() <= 4 * 2.0 ** -24 * L.rows.cpu().double()[inv].abs().sum(1)).all())


def test_mx_layer_captured_and_on_another_stream(mb):
    """A captured run replayed between eager ones, and a run on a side stream, give the eager bits."""
    say("MXFP4 layer: graph and streams")
    L = MxLayer(mb, 24, 32, 4, 512, 256, 77)
    eager = L.run().clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    L.y.zero_()
    torch.cuda.synchronize()
    L.run(stream=side)
    side.synchronize()
    assert torch.equal(L.y, eager)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.run()
    other = MxLayer(mb, 24, 32, 4, 512, 256, 78)
    for _ in range(3):
        L.y.zero_()
        graph.replay()
        theirs = other.run().clone()
        torch.cuda.synchronize()
        assert torch.equal(L.y, eager)
        assert torch.equal(other.run(), theirs)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_expert_training_step(mb, dtype):
    """Forward and both gradients of the gate, up and down products of one step, against autograd in 64 bits on the same
    16-bit values; the gradient by the tokens is the combine's sum of dx rows."""
    say(f"training step {dtype}")
    T, E, topk, H, F = 50, 12, 3, 256, 128
    p = route(mb, T, E, topk, 91)
    n = T * topk
    off, tok = p["offsets"].cpu(), p["row_tok"].cpu()
    g = torch.Generator().manual_seed(92)
    x = torch.randn(T, H, generator=g).to(dtype)
    w = (torch.randn(E, F, H, generator=g) / H ** 0.5).to(dtype)
    dy = torch.randn(n, F, generator=g).to(dtype)
    out = torch.empty(n, F, device="cuda")
    mb.grouped_gemm(dev(x), dev(w), p["offsets"], out, row_tok=p["row_tok"])
    dx = torch.empty(n, H, device="cuda")
    mb.grouped_gemm_dx(dev(dy), dev(w), p["offsets"], dx)
    dw = torch.empty(E, F, H, device="cuda")
    mb.grouped_gemm_dw(dev(dy), dev(x), p["offsets"], dw, row_tok=p["row_tok"])
    dtok = torch.empty(T, H, device="cuda")
    mb.combine(dx, p["inv_pos"], T, topk, H, None, dtok)
    x64, w64 = x.double().requires_grad_(), w.double().requires_grad_()
    y = torch.cat([x64[tok[a:b].long()] @ w64[e].T for e, a, b in gu.groups(off, n, E)])
    (y * dy.double()).sum().backward()
    my = torch.cat([x.double().abs()[tok[a:b].long()] @ w.double().abs()[e].T for e, a, b in gu.groups(off, n, E)])
    assert bool(((out.cpu().double() - y).abs() <= gu.rounded(y, gu.sum_bound(my, H, 32), F32)).all())
    mw = torch.stack([dy[a:b].double().abs().T @ x.double().abs()[tok[a:b].long()] for _, a, b in gu.groups(off, n, E)])
    assert bool(((dw.cpu().double() - w64.grad).abs() <= gu.rounded(w64.grad, gu.sum_bound(mw, n, 32), F32)).all())
    mx = torch.zeros(T, H, dtype=torch.float64)
    rows = torch.cat([dy[a:b].double().abs() @ w[e].double().abs() for e, a, b in gu.groups(off, n, E)])
    mx.index_add_(0, tok.long(), rows)
    assert bool(((dtok.cpu().double() - x64.grad).abs() <= gu.sum_bound(mx, F, 32) + 4 * 2.0 ** -24 * mx).all())
    # and against differences of the forward product: it is linear in x, so one central difference is exact
    # up to rounding
    i, j = 7, 11
    step = 0.5
    f = []
    for d in (step, -step):
        xp = x.float().clone()
        xp[i, j] += d
        moved = xp.to(dtype)
        mb.grouped_gemm(dev(moved), dev(w), p["offsets"], out, row_tok=p["row_tok"])
        f.append((float(moved[i, j]), float((out.cpu().double() * dy.double()).sum())))
    slope = (f[0][1] - f[1][1]) / (f[0][0] - f[1][0])
    # each of the two sums is off by at most the bound of its elements times dy
    err = float((gu.sum_bound(my * 2, H, 32) * dy.double().abs()).sum()) * 2 / (f[0][0] - f[1][0])
    assert abs(slope - float(dtok[i, j])) <= err


def test_gradients_captured_and_on_two_streams(mb):
    """Forward, dx and a dw in parts (whose workspace the binding allocates) in one graph, replayed between eager calls,
    and at once on two streams: the eager bits each time."""
    say("gradients: graph and streams")
    g = torch.Generator().manual_seed(8)
    off = torch.tensor([0, 1500, 1500, 4000], dtype=torch.int32).cuda()
    sets = []
    for _ in range(2):
        x, dy = torch.randn(4000, 264, generator=g).to(BF).cuda(), torch.randn(4000, 136, generator=g).to(BF).cuda()
        w = torch.randn(3, 136, 264, generator=g).to(BF).cuda()
        sets.append((x, dy, w, torch.empty(4000, 136, device="cuda"), torch.empty(4000, 264, device="cuda"),
                     torch.empty(3, 136, 264, device="cuda")))
    assert mb.grouped_gemm_dw_workspace_bytes(4000, 3, 136, 264) > 0

    def step(k, stream=None):
        x, dy, w, y, dx, dw = sets[k]
        mb.grouped_gemm(x, w, off, y, stream=stream)
        mb.grouped_gemm_dx(dy, w, off, dx, stream=stream)
        mb.grouped_gemm_dw(dy, x, off, dw, stream=stream)

    def results(k):
        return [t.clone() for t in sets[k][3:]]

    eager = []
    for k in (0, 1):
        step(k)
        eager.append(results(k))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(0)
    for _ in range(3):
        for t in sets[0][3:]:
            t.zero_()
        graph.replay()
        step(1)
        torch.cuda.synchronize()
        for k in (0, 1):
            assert all(torch.equal(a, b) for a, b in zip(results(k), eager[k]))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for t in sets[0][3:] + sets[1][3:]:
        t.zero_()
    torch.cuda.synchronize()
    for _ in range(10):
        for k in (0, 1):
            step(k, streams[k])
    torch.cuda.synchronize()
    for k in (0, 1):
        assert all(torch.equal(a, b) for a, b in zip(results(k), eager[k]))


def test_two_calls_on_two_streams(mb):
    """Calls share nothing: two at once on two streams give what they give alone."""
    say("two streams at once")
    a, b = (MxLayer(mb, 64, 32, 4, 512, 256, 100 + i) for i in range(2))
    ya, yb = a.run().clone(), b.run().clone()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for layer, s in zip((a, b), streams):
            layer.run(stream=s)
    torch.cuda.synchronize()
    assert torch.equal(a.y, ya) and torch.equal(b.y, yb)
