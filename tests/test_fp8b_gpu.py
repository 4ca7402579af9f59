"""The block-scaled fp8 operators against their definitions in 64 bits.

Tolerances, derived before the first run:
  codes of given inputs   bit for bit: scale, reciprocal and product are single
                          IEEE fp32 operations, the code the nearest.
  products                a block's 128 exact products are summed on the tensor
                          cores (each addition off by at most 2^-23 of the sum
                          of magnitudes), then each block's sum takes three
                          fp32 roundings and the running sum one per block:
                          |y - ref| <= (128 * 2^-23 + (blocks + 3) * 2^-24) S,
                          S = the same product of magnitudes; bf16 outputs add
                          half a step, 2^-8 |ref|.
  SwiGLU                  errors of g and u as above through h = silu(g) u
                          (|silu'| <= 1.1), plus 2^-19 |h| for the exponential
                          and the divide.
  codes of computed values  half a step of E4M3: 2^-4 of the value, or 2^-10
                          of the scale among the subnormal codes.
  norm                    r: k + 1 fused adds, each 2^-24 of the magnitudes;
                          y: the mean of squares, root, divide and two products
                          together under 2^-18 relative.
"""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
B, FMAX = 128, 448.0
F8 = torch.float8_e4m3fn
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import expert_routed_ffn_selectedsoftmax_gb300 as pkg
    torch.cuda.set_device(0)
    return pkg


def rand(*shape, seed=0, sd=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed + 1000 * len(shape) + sum(shape))
    return torch.randn(*shape, generator=g, device=DEV) * sd


def blocks(n):
    return (n + B - 1) // B


def quant(x, block_rows):
    """The definition in fp32: codes, scales of [..., rows, cols]."""
    rows, cols = x.shape[-2:]
    nr, nc = -(-rows // block_rows), blocks(cols)
    pad = torch.zeros(*x.shape[:-2], nr * block_rows, nc * B, device=x.device)
    pad[..., :rows, :cols] = x.float()
    t = pad.view(*x.shape[:-2], nr, block_rows, nc, B)
    amax = t.abs().amax(dim=(-3, -1))        # (propagates NaN)
    # (a tensor divisor: torch divides by a Python number through its reciprocal)
    s = torch.where(torch.isfinite(amax), amax / torch.full_like(amax, FMAX), torch.nan)
    s = torch.where(s < 2.0 ** -126, torch.zeros_like(s), s)
    f = torch.where(s == 0, s, torch.ones_like(s) / s)[..., :, None, :, None]
    c = torch.where(f.isnan(), torch.nan, (t * f).clamp(-FMAX, FMAX)).reshape(pad.shape)
    return c[..., :rows, :cols].to(F8).contiguous(), s


def value(q, s, block_rows):
    """codes * scales in 64 bits."""
    rows, cols = q.shape[-2:]
    r = torch.arange(rows, device=q.device) // block_rows
    c = torch.arange(cols, device=q.device) // B
    return q.view(F8).double() * s.double()[..., r, :][..., c]


def bits(t):
    return t.view(torch.uint8) if t.element_size() == 1 else t.view(torch.int32)


def same_codes(got, want):
    """Equal codes; NaN codes may differ in sign."""
    a, b = got.view(F8).float(), want.view(F8).float()
    assert torch.equal(a.isnan(), b.isnan())
    assert torch.equal(a.nan_to_num(1.0), b.nan_to_num(1.0)), f"{int((a.nan_to_num(1.0) != b.nan_to_num(1.0)).sum())} codes differ"


def same_scales(got, want):
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(1.0), want.nan_to_num(1.0))


# ------------------------------------------------------------- quantisation

@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("batch,rows,cols,block_rows", [
    (None, 1, 16, 1), (None, 1, 128, 1), (None, 37, 2816, 1), (None, 5, 1040, 1), (3, 7, 144, 1), (None, 4099, 512, 1),
    (None, 1, 16, 128), (None, 128, 128, 128), (None, 129, 272, 128), (3, 200, 400, 128), (2, 1000, 2816, 128)])
def test_quant(moe, dt, batch, rows, cols, block_rows):
    shape = (rows, cols) if batch is None else (batch, rows, cols)
    x = (rand(*shape) * torch.exp(rand(*shape[:-1], 1, seed=1))).to(DT[dt])
    q, s = moe.moe_quant_fp8b(x, block_rows=block_rows)
    wq, ws = quant(x, block_rows)
    assert q.dtype == F8 and q.shape == x.shape and s.shape == ws.shape
    same_scales(s, ws)
    same_codes(q, wq)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quant_special_values(moe, block_rows):
    """Zero, tiny, huge, infinite and NaN blocks; -0; ties to the even code."""
    x = rand(9 * 128, 128)
    x[0:128] = 0
    x[128:256] = 1e-44                      # amax / 448 underflows to zero
    x[256:384] *= 1e-36                     # the scale is about the smallest normal number: some rows' are 0
    x[384:512] *= 3e37
    x[512:640, 5] = float("inf")
    x[640:768, 77] = float("nan")
    x[768:896, 3], x[768:896, 4] = float("-inf"), float("nan")
    ladder = torch.arange(128, device=DEV).float() / 8
    x[896:1024] = ladder                    # borders of two codes among them
    x[896:1024, 127] = FMAX
    x[1024:] = -0.0
    q, s = moe.moe_quant_fp8b(x, block_rows=block_rows)
    wq, ws = quant(x, block_rows)
    same_scales(s, ws)
    same_codes(q, wq)
    assert bool((s[: 256 // block_rows] == 0).all()) and bool(s[512 // block_rows : 896 // block_rows].isnan().all())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols,block_rows", [(4096, 1024, 1), (4096, 1024, 128), (999, 2000, 1), (300, 400, 128)])
def test_quant_against_the_quotient(moe, dt, rows, cols, block_rows):
    """Codes against the nearest-even ones of 448 x / max|x|, not by the kernel's own
    operations.  s, 1/s and the product are each off by 2^-24 at most, so a code may
    differ only where the quotient is within 3 x 2^-24 (and its square's share) of
    the border, and then by one step.  A border is (n + 1/2) steps, n < 16: 448 |x|
    and border * max|x| have at most 29 bits and are compared exactly in 64."""
    x = (rand(rows, cols, seed=3) * torch.exp(rand(rows, 1, seed=4, sd=0.5))).to(DT[dt])
    q, s = moe.moe_quant_fp8b(x, block_rows=block_rows)
    nr, nc = -(-rows // block_rows), blocks(cols)
    pad = torch.zeros(nr * block_rows, nc * B, dtype=torch.float64, device=DEV)
    pad[:rows, :cols] = x.double().abs()
    top = pad.view(nr, block_rows, nc, B).amax(dim=(1, 3))
    assert bool(((s.double() * FMAX - top).abs() <= 2.0 ** -24 * top).all())
    top = top.repeat_interleave(block_rows, 0)[:rows].repeat_interleave(B, 1)[:, :cols]
    x448, got = FMAX * x.double().abs(), q.double().abs()
    quo = x448 / top
    step = torch.exp2(torch.floor(torch.log2(quo.clamp(min=2.0 ** -30))).clamp(min=-6) - 3)
    low = torch.floor(quo / step)
    side = x448 - (low + 0.5) * step * top                    # sign: above or below the border, 0 on it
    even = low + (low % 2)
    want = torch.where(side > 0, low + 1, torch.where(side < 0, low, even)) * step
    near = side.abs() <= 3.01 * 2.0 ** -24 * x448
    assert torch.equal(got[~near], want[~near])
    assert bool(((got == low * step) | (got == (low + 1) * step)).all())
    assert bool(((q.double() >= 0) | (x.double() < 0)).all()) and bool(((q.double() <= 0) | (x.double() > 0)).all())


def test_quant_strided_and_given_outputs(moe):
    big = rand(2, 40, 512)
    x = big[..., :256]                      # rows 512 apart, batches 40 * 512 apart
    q = torch.full((2, 40, 256), 1.0, device=DEV).to(F8)
    s = torch.zeros(2, 40, 2, device=DEV)
    rq, rs = moe.moe_quant_fp8b(x, codes=q, scales=s)
    assert rq is q and rs is s
    wq, ws = quant(x, 1)
    same_codes(q, wq)
    same_scales(s, ws)
    empty = moe.moe_quant_fp8b(x[:, :0])
    assert empty[0].shape == (2, 0, 256) and empty[1].shape == (2, 0, 2)


# --------------------------------------------------------------------- norm

def norm_ref(x, weight, eps, delta=None, topk_w=None, inv=None):
    """(r, y, bound of r's error) in 64 bits."""
    r, mag, n = x.double(), x.double().abs(), 0
    if delta is not None and inv is None:
        r, mag, n = r + delta.double(), mag + delta.double().abs(), 1
    elif delta is not None:
        n = topk_w.shape[1]
        for j in range(n):
            at = inv.view(-1, n)[:, j].long()
            ok = (at >= 0) & (at < delta.shape[0])
            term = torch.where(ok[:, None], topk_w[:, j:j + 1].double() * delta.double()[at.clamp(0, delta.shape[0] - 1)], 0.0)
            r, mag = r + term, mag + term.abs()
    y = r / torch.sqrt((r * r).mean(1, keepdim=True) + eps) * weight.double()
    return r, y, (n + 1) * 2.0 ** -24 * mag


def check_codes(q, s, y, err):
    """Codes of computed values y known up to err, per row and 128 columns."""
    rows, cols = y.shape
    pad = torch.zeros(rows, blocks(cols) * B, dtype=torch.float64, device=y.device)
    pad[:, :cols] = y.abs()
    epad = torch.zeros_like(pad)
    epad[:, :cols] = err
    amax, emax = (t.view(rows, -1, B).amax(2) for t in (pad, epad))
    assert bool(((s.double() - amax / FMAX).abs() <= emax / FMAX + 2.0 ** -23 * amax / FMAX + 2.0 ** -149).all())
    got = value(q, s, 1)
    each = s.double().repeat_interleave(B, 1)[:, :cols]
    tol = err + (y.abs() + err) * (2.0 ** -4 + 2.0 ** -22) + each * 2.0 ** -10
    worst = ((got - y).abs() - tol).max()
    assert worst <= 0, f"codes off by {float(worst):.3e} more than half a step"


def check_norm(x, weight, eps, out, delta=None, topk_w=None, inv=None):
    resid, normed, q, s = out
    r, y, err = norm_ref(x, weight, eps, delta, topk_w, inv)
    step = torch.finfo(x.dtype).eps / 2
    assert resid.dtype == x.dtype
    if delta is None:
        assert resid is x
    else:
        assert bool(((resid.double() - r).abs() <= err + step * (r.abs() + err)).all())
    # y's error: r's, scaled, plus the relative error of the root and products
    rms = torch.sqrt((r * r).mean(1, keepdim=True) + eps)
    relerr = torch.sqrt((err * err).mean(1, keepdim=True)) / rms
    yerr = err / rms * weight.double().abs() + y.abs() * (relerr + 2.0 ** -18)
    if normed is not None:
        assert normed.dtype == torch.bfloat16
        assert bool(((normed.double() - y).abs() <= yerr + 2.0 ** -8 * (y.abs() + yerr)).all())
    check_codes(q, s, y, yerr)


@pytest.mark.parametrize("dt,ddt,wdt", [("f32", "bf16", "f32"), ("f32", "f32", "bf16"), ("bf16", "bf16", "bf16"), ("bf16", "f32", "f32")])
@pytest.mark.parametrize("T,d,k", [(1, 16, 0), (1, 2048, 0), (3, 144, 1), (37, 1024, 2), (5, 4112, 3), (33, 8192, 8), (2, 16384, 2)])
def test_norm(moe, dt, ddt, wdt, T, d, k):
    x, w = rand(T, d, sd=2.0).to(DT[dt]), (1 + rand(d, sd=0.2)).to(DT[wdt])
    delta = rand(T * max(k, 1), d, seed=1).to(DT[ddt])
    topk_w = inv = None
    if k:
        topk_w = torch.softmax(rand(T, k), 1)
        inv = torch.randperm(T * k, device=DEV).int()
    out = moe.moe_norm_fp8b(x, w, 1e-5, delta=delta, topk_w=topk_w, inv=inv)
    check_norm(x, w, 1e-5, out, delta, topk_w, inv)
    alone = moe.moe_norm_fp8b(x, w, 1e-5, want_normed=False)
    assert alone[1] is None
    check_norm(x, w, 1e-5, alone)


def test_norm_slots_without_rows(moe):
    """Slots outside [0, rows of delta) add nothing, NaN rows among delta that
    no slot names do not matter, an index may come twice; delta without rows."""
    T, d, k = 9, 256, 4
    x, w = rand(T, d), torch.ones(d, device=DEV)
    delta = rand(12, d, seed=2)
    delta[11] = float("nan")
    inv = torch.randint(0, 11, (T, k), device=DEV).int()
    inv[0] = -1
    inv[1, 2], inv[2, 0], inv[3] = 12, -2 ** 31, 5
    topk_w = torch.softmax(rand(T, k), 1)
    inv = inv.reshape(-1)
    out = moe.moe_norm_fp8b(x, w, 1e-5, delta=delta, topk_w=topk_w, inv=inv)
    check_norm(x, w, 1e-5, out, delta, topk_w, inv)
    assert torch.equal(out[0][0], x[0])
    none = moe.moe_norm_fp8b(x, w, 1e-5, delta=delta[:0], topk_w=topk_w, inv=inv)
    assert torch.equal(none[0], x)


def test_norm_zero_and_non_finite_rows(moe):
    x = rand(4, 256)
    x[0] = 0
    x[1, 3] = float("inf")
    x[2, 130] = float("nan")
    w = torch.ones(256, device=DEV)
    r, y, q, s = moe.moe_norm_fp8b(x, w, 0.0 + 1e-6)
    assert not y[0].any() and not s[0].any() and not q[0].float().any()
    assert bool(s[2].isnan().all()) and bool(q[2].float().isnan().all())
    # inf / inf is NaN in its block; the other block's values are 0
    assert bool(s[1, 0].isnan()) and float(s[1, 1]) == 0.0
    last = x[3:]
    one = moe.moe_norm_fp8b(last, w, 1e-6)
    check_norm(last, w, 1e-6, one)
    assert torch.equal(bits(one[2]), bits(q[3:])) and torch.equal(one[3], s[3:])


@pytest.mark.parametrize("size", [1e-42, 1e-38, 1e-37, 1e-30, 1e-20, 1e15])
def test_norm_of_small_and_large_rows(moe, size):
    """Values whose squares vanish beside eps, scales at the smallest normal
    number and below (those blocks are zeros), and large ones."""
    x, w = (rand(5, 384) * size), 1 + rand(384, sd=0.1)
    _, y, q, s = moe.moe_norm_fp8b(x, w, 1e-6)
    _, want, err = norm_ref(x, w, 1e-6)
    rms = torch.sqrt((x.double() ** 2).mean(1, keepdim=True) + 1e-6)
    yerr = err / rms * w.double().abs() + want.abs() * 2.0 ** -18 + 2.0 ** -149 * 1e3
    amax = want.abs().view(5, 3, B).amax(2)
    zero = (s == 0) & (amax / FMAX < 2.0 ** -126 * 1.001)      # counted as zeros
    assert bool(((s > 0) | zero).all())
    keep = (s > 0).repeat_interleave(B, 1)
    assert not q.float()[~keep].any()
    got = value(q, s, 1)
    tol = yerr + (want.abs() + yerr) * (2.0 ** -4 + 2.0 ** -22) + s.double().repeat_interleave(B, 1) * 2.0 ** -10
    assert bool((((got - want).abs() <= tol) | ~keep).all())


def test_norm_of_rows_whose_squares_overflow(moe):
    """Finite rows beyond the fp32 sum of squares give zeros, as the header says;
    the residual and the other rows are as without them."""
    x, w = rand(6, 384), torch.ones(384, device=DEV)
    want = moe.moe_norm_fp8b(x, w, 1e-6, delta=x)
    big = x.clone()
    big[2], big[4] = 1e20, -3e37
    resid, y, q, s = moe.moe_norm_fp8b(big, w, 1e-6, delta=big)
    assert torch.equal(resid, big + big)
    for r in (2, 4):
        assert not y[r].any() and not q[r].float().any() and not s[r].any()
    for a, b in zip((resid, y, q, s), want):
        keep = [0, 1, 3, 5]
        assert torch.equal(a[keep].float(), b[keep].float())


def test_norm_in_place_and_strided(moe):
    T, d = 21, 512
    wide, dwide = rand(T, 1024), rand(T, 768).bfloat16()
    x, delta, w = wide[:, 256:768], dwide[:, :d], torch.ones(d, device=DEV)
    check_norm(x, w, 1e-6, moe.moe_norm_fp8b(x, w, 1e-6, delta=delta), delta)
    x2 = x.clone()
    want = moe.moe_norm_fp8b(x2.clone(), w, 1e-6, delta=delta)
    got = moe.moe_norm_fp8b(x2, w, 1e-6, delta=delta, resid=x2)
    assert got[0] is x2
    for a, b in zip(got, want):
        assert torch.equal(a.float(), b.float())
    z = moe.moe_norm_fp8b(x[:0], w)
    assert z[2].shape == (0, d)


# ----------------------------------------------------------------- products

def pair(rows, K, seed=0, block_rows=1, lead=()):
    x = rand(*lead, rows, K, seed=seed) * torch.exp(rand(*lead, rows, 1, seed=seed + 1, sd=0.5))
    return quant(x, block_rows)


def product_bound(xv, wv, K):
    return (128 * 2.0 ** -23 + (blocks(K) + 3) * 2.0 ** -24) * (xv.abs() @ wv.abs().T)


def check_product(y, xv, wv, K):
    ref = xv @ wv.T
    tol = product_bound(xv, wv, K)
    if y.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (ref.abs() + tol)
    worst = ((y.double() - ref).abs() - tol).max() if ref.numel() else 0.0
    assert worst <= 0, f"off by {float(worst):.3e} more than the bound"


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("T,K,N", [(1, 16, 1), (1, 128, 256), (1, 2048, 2816), (2, 144, 7), (33, 272, 130), (127, 512, 257),
                                   (128, 1040, 1000), (129, 256, 96), (300, 2816, 384), (1111, 640, 2050), (2500, 512, 2304)])
def test_gemm(moe, out, T, K, N):
    xq, xs = pair(T, K)
    wq, ws = pair(N, K, seed=5, block_rows=128)
    y = moe.moe_gemm_fp8b(xq, xs, wq, ws, out_dtype=DT[out])
    assert y.shape == (T, N) and y.dtype == DT[out]
    check_product(y, value(xq, xs, 1), value(wq, ws, 128), K)
    assert torch.equal(y, moe.moe_gemm_fp8b(xq, xs, wq, ws, out_dtype=DT[out]))


@pytest.mark.parametrize("T", [1, 16])
@pytest.mark.parametrize("K", [896, 912, 1008, 1040, 1296])
def test_gemm_of_few_rows_whole_and_split(moe, T, K):
    """Reductions of 7 to 11 blocks, the last one ragged: on both sides of the
    length from which few tiles split it, also where the parts are unequal."""
    N = 1024
    xq, xs = pair(T, K)
    wq, ws = pair(N, K, seed=6, block_rows=128)
    y = moe.moe_gemm_fp8b(xq, xs, wq, ws, out_dtype=torch.float32)
    check_product(y, value(xq, xs, 1), value(wq, ws, 128), K)
    assert torch.equal(y, moe.moe_gemm_fp8b(xq, xs, wq, ws, out_dtype=torch.float32))


@pytest.mark.parametrize("T", [1, 16])
@pytest.mark.parametrize("d", [384, 400, 512, 656])
def test_gate_up_of_few_rows_whole_and_split(moe, T, d):
    """The same for gate/up, which splits from 4 blocks."""
    F = 400
    xq, xs = pair(T, d)
    (gq, gs), (uq, us) = (quant(rand(F, d, seed=s, sd=d ** -0.5), 128) for s in (1, 2))
    hq, hs = moe.moe_gate_up_fp8b(xq, xs, gq, gs, uq, us)
    h, err = swiglu_ref(value(xq, xs, 1), value(gq, gs, 128), value(uq, us, 128), d)
    check_codes(hq, hs, h, err)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("N", [129, 255, 1001, 1050])
@pytest.mark.parametrize("pad", [0, 3, 6, 7])
@pytest.mark.parametrize("T", [20, 4000])     # (few rows, and the tiled kernel)
def test_unaligned_output_rows(moe, out, N, pad, T):
    """Rows that begin or end inside 16 bytes: nothing beside them is written."""
    K = 272
    xq, xs = pair(T, K)
    wq, ws = pair(N, K, seed=3, block_rows=128)
    wide = torch.full((T + 2, N + pad), 3.0, dtype=DT[out], device=DEV)
    y = moe.moe_gemm_fp8b(xq, xs, wq, ws, out=wide[1:-1, :N])
    check_product(y, value(xq, xs, 1), value(wq, ws, 128), K)
    assert bool((wide[0] == 3).all()) and bool((wide[-1] == 3).all()) and bool((wide[:, N:] == 3).all())


def test_gemm_every_code(moe):
    """Every finite code of both signs on both sides, exact sums: one nonzero
    weight per output column."""
    codes = torch.tensor([c for c in range(256) if c & 0x7F != 0x7F], dtype=torch.uint8, device=DEV)   # 254
    K = 256
    xq = torch.zeros(254, K, dtype=torch.uint8, device=DEV)
    xq[:, 200] = codes
    wq = torch.zeros(254, K, dtype=torch.uint8, device=DEV)
    wq[:, 200] = codes
    xs, ws = torch.ones(254, 2, device=DEV), torch.ones(2, 2, device=DEV)
    y = moe.moe_gemm_fp8b(xq, xs, wq, ws, out_dtype=torch.float32)
    v = codes.view(F8).double()
    assert torch.equal(y.double(), v[:, None] * v[None, :])


def test_gemm_scales_act_on_their_own_block(moe):
    """Scales of very different size per block of K, of N and per row; a zero
    and a NaN scale stay in their rows and columns."""
    T, K, N = 70, 5 * 128, 3 * 128 + 16
    xq, xs = pair(T, K)
    wq, ws = pair(N, K, seed=3, block_rows=128)
    xs = xs * 4.0 ** torch.randint(-8, 8, xs.shape, device=DEV)
    ws = ws * 4.0 ** torch.randint(-8, 8, ws.shape, device=DEV)
    xs[7] = 0
    check_product(moe.moe_gemm_fp8b(xq, xs, wq, ws, out_dtype=torch.float32), value(xq, xs, 1), value(wq, ws, 128), K)
    xs[9, 2], ws[1, 3] = float("nan"), float("nan")
    bad = moe.moe_gemm_fp8b(xq, xs, wq, ws, out_dtype=torch.float32).isnan()
    want = torch.zeros_like(bad)
    want[9] = True
    want[:, 128:256] = True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("T", [45, 3007])
def test_gemm_strided(moe, T):
    """Rows further apart than their length, in and out, aligned and not."""
    K, N = 384, 1000
    wide = torch.zeros(T, 1024, device=DEV).to(F8)
    xq, xs = pair(T, K)
    wide[:, 512:512 + K] = xq
    wq, ws = pair(N, K, seed=2, block_rows=128)
    for dt in DT.values():
        for pad in (0, 8, 5):       # 5: rows whose 16-byte pieces are not aligned
            buf = torch.full((T, N + pad + (8 if pad == 8 else 3)), 7.0, dtype=dt, device=DEV)
            y = moe.moe_gemm_fp8b(wide[:, 512:512 + K], xs, wq, ws, out=buf[:, pad:pad + N])
            check_product(y, value(xq, xs, 1), value(wq, ws, 128), K)
            assert bool((buf[:, :pad] == 7).all()) and bool((buf[:, pad + N:] == 7).all())


def grouping(T, E, k, seed, skew=0.5):
    """(offsets, perm_tok, expert of each grouped row), k distinct experts per token."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    scores = torch.randn(T, E, generator=g, device=DEV) + skew * torch.randn(E, generator=g, device=DEV)
    slots = scores.topk(k, dim=1).indices.reshape(-1)
    order = torch.argsort(slots, stable=True)
    off = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), torch.bincount(slots, minlength=E).cumsum(0)]).int()
    return off, (order // k).int(), slots[order]


GROUPS = [  # T, E, k, K, N (F), skew
    (1, 1, 1, 128, 128, 0.0), (1, 64, 2, 1024, 512, 0.5), (3, 5, 2, 144, 80, 0.5), (64, 16, 1, 2816, 256, 0.5),
    (128, 64, 2, 256, 272, 0.5), (200, 256, 8, 128, 64, 0.5), (700, 3, 1, 272, 400, 2.0), (1500, 8, 2, 512, 768, 1.0),
    (40, 4, 1, 640, 128, 30.0), (2048, 16, 1, 256, 1040, 0.5)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("T,E,k,K,N,skew", GROUPS)
def test_grouped_gemm(moe, T, E, k, K, N, skew, gather, out):
    off, perm, expert = grouping(T, E, k, seed=T + E, skew=skew)
    rows = T * k
    xq, xs = pair(T if gather else rows, K)
    N = N + 3      # (an odd width: stores that are not whole pieces)
    wq, ws = pair(N, K, seed=7, block_rows=128, lead=(E,))
    y = moe.moe_grouped_gemm_fp8b(xq, xs, wq, ws, off, perm_tok=perm if gather else None, out_dtype=DT[out])
    assert y.shape == (rows, N)
    xv, wv = value(xq, xs, 1), value(wq, ws, 128)
    xv = xv[perm.long()] if gather else xv
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        check_product(y[a:b], xv[a:b], wv[e], K)


def swiglu_ref(xv, gv, uv, K):
    g, u = xv @ gv.T, xv @ uv.T
    dg, du = product_bound(xv, gv, K), product_bound(xv, uv, K)
    silu = g * torch.sigmoid(g)
    h = silu * u
    err = 1.1 * dg * (u.abs() + du) + (silu.abs() + 1.1 * dg) * du + 2.0 ** -19 * h.abs()
    return h, err


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("T,E,k,d,F,skew", GROUPS)
def test_gate_up(moe, T, E, k, d, F, skew, gather):
    off, perm, expert = grouping(T, E, k, seed=T + E + 1, skew=skew)
    rows = T * k
    xq, xs = pair(T if gather else rows, d)
    (gq, gs), (uq, us) = (quant(rand(E, F, d, seed=s, sd=d ** -0.5), 128) for s in (11, 12))
    hq, hs = moe.moe_gate_up_fp8b(xq, xs, gq, gs, uq, us, offsets=off, perm_tok=perm if gather else None)
    assert hq.shape == (rows, F) and hs.shape == (rows, blocks(F)) and hq.dtype == F8
    xv = value(xq, xs, 1)
    xv = xv[perm.long()] if gather else xv
    gv, uv = value(gq, gs, 128), value(uq, us, 128)
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        if a < b:
            h, err = swiglu_ref(xv[a:b], gv[e], uv[e], d)
            check_codes(hq[a:b], hs[a:b], h, err)
    again = moe.moe_gate_up_fp8b(xq, xs, gq, gs, uq, us, offsets=off, perm_tok=perm if gather else None)
    assert torch.equal(bits(hq), bits(again[0])) and torch.equal(hs, again[1])


@pytest.mark.parametrize("T", [1, 40, 300])
def test_gate_up_dense(moe, T):
    """No offsets, weights [F, d]: the dense layer's call."""
    d, F = 256, 400
    xq, xs = pair(T, d)
    (gq, gs), (uq, us) = (quant(rand(F, d, seed=s, sd=d ** -0.5), 128) for s in (1, 2))
    hq, hs = moe.moe_gate_up_fp8b(xq, xs, gq, gs, uq, us)
    h, err = swiglu_ref(value(xq, xs, 1), value(gq, gs, 128), value(uq, us, 128), d)
    check_codes(hq, hs, h, err)


# rows, d of the few-rows kernel, whole and split over a cluster, and of the tiled one
GATE_RANGE = [(201, 256), (201, 640), (5025, 256)]


def one_column(sx, d, F, su):
    """Operands whose sums are exact: x has +-1 in column 200 and |sx| as that
    block's scale, the gate's weights are 1 there, the up weights small codes times
    su: g = sx in every column, u = sx * code * su."""
    rows = sx.shape[0]
    xq = torch.zeros(rows, d, device=DEV)
    xq[:, 200] = torch.where(sx < 0, -1.0, 1.0)
    xs = torch.ones(rows, blocks(d), device=DEV)
    xs[:, 1] = sx.abs()
    gq, uq = torch.zeros(F, d, device=DEV), torch.zeros(F, d, device=DEV)
    gq[:, 200] = 1.0
    uq[:, 200] = 1 + (torch.arange(F, device=DEV) % 29).div(4, rounding_mode="floor") / 4
    one = torch.ones(blocks(F), blocks(d), device=DEV)
    return (xq.to(F8), xs, gq.to(F8), one, uq.to(F8), one * su), uq[:, 200].double() * su


@pytest.mark.parametrize("rows,d", GATE_RANGE)
def test_gate_up_over_the_gate_sums_range(moe, rows, d):
    """g from -100 to 100 on exact sums.  Off by __expf's 2 + 1.173 |g| units in
    the last place (2^-23), 2 of the divide and half a unit each of the sum and
    the product: (5 + 1.18 |g|) 2^-23 |h|; |silu| below |g| 2^-125 may count as 0.
    The up sums are large, so that h at g = -87 is far from the smallest numbers."""
    F, g = 272, torch.linspace(-100, 100, 201, device=DEV).repeat(rows // 201)
    args, up = one_column(g, d, F, 2.0 ** 40)
    hq, hs = moe.moe_gate_up_fp8b(*args)
    g = g.double()[:, None]
    u = g * up
    h = g * torch.sigmoid(g) * u
    check_codes(hq, hs, h, h.abs() * (5 + 1.18 * g.abs()) * 2.0 ** -23 + g.abs() * u.abs() * 2.0 ** -125)
    below = (g[:, 0] < -89) | (g[:, 0] == 0)
    assert not hs[below].any() and not hq[below].float().any() and bool((hs[(g[:, 0] > -87) & ~below] > 0).all())


@pytest.mark.parametrize("rows,d", GATE_RANGE)
def test_gate_up_of_non_finite_gate_sums(moe, rows, d):
    """Gate sums that are NaN, infinite or overflow: NaN codes with NaN scales in
    their rows, as the definition has it; the other rows keep theirs."""
    F = 272
    g = torch.linspace(-20, 20, 201, device=DEV).repeat(rows // 201)
    args, _ = one_column(g, d, F, 1.0)
    hq, hs = moe.moe_gate_up_fp8b(*args)
    bad = [0, 3, 40, 77, rows - 1]
    for r, v in zip(bad, (float("nan"), float("inf"), float("-inf"), 3e38, -3e38)):
        args[0][r, 200] = -2.0 if v < 0 else 2.0
        args[1][r, 1] = abs(v)
    bq, bs = moe.moe_gate_up_fp8b(*args)
    keep = torch.ones(rows, dtype=torch.bool, device=DEV)
    keep[bad] = False
    assert torch.equal(bits(bq)[keep], bits(hq)[keep]) and torch.equal(bs[keep], hs[keep])
    assert bool(bs[~keep].isnan().all()) and bool(bq[~keep].float().isnan().all())


@pytest.mark.parametrize("T,E", [(6, 4), (400, 4), (3000, 7)])
def test_padded_batch_leaves_the_rest(moe, T, E):
    """Groups that do not start at 0 and end before the last row: rows outside
    them keep what they held; bad offsets stay inside the buffers."""
    K, N = 256, 160
    xq, xs = pair(T, K)
    wq, ws = pair(N, K, seed=4, block_rows=128, lead=(E,))
    cuts = torch.linspace(2, T - 2, E + 1, device=DEV).int()
    out = torch.full((T, N), 3.0, device=DEV)
    hq, hs = torch.full((T, N), 5, dtype=torch.uint8, device=DEV), torch.full((T, 2), 9.0, device=DEV)
    moe.moe_grouped_gemm_fp8b(xq, xs, wq, ws, cuts, out=out)
    moe.moe_gate_up_fp8b(xq, xs, wq, ws, wq, ws, offsets=cuts, h_q=hq, h_s=hs)
    a, b = int(cuts[0]), int(cuts[-1])
    for t, v in ((out, 3.0), (hq, 5), (hs, 9.0)):
        assert bool((t[:a] == v).all()) and bool((t[b:] == v).all())
    xv, wv = value(xq, xs, 1), value(wq, ws, 128)
    for e in range(E):
        check_product(out[cuts[e]:cuts[e + 1]], xv[cuts[e]:cuts[e + 1]], wv[e], K)
    # descending, negative and too large offsets: clamped, nothing outside [0, rows) touched
    status = torch.zeros(64, dtype=torch.int32, device=DEV)
    for wild in ([-5, T + 77] * E + [2 ** 31 - 1], [0, T] * E + [T], [T, 0] * E + [0]):
        wild = torch.tensor(wild[:E + 1], dtype=torch.int32, device=DEV)
        pad = torch.full((T + 2, N), 3.0, device=DEV)
        moe.moe_grouped_gemm_fp8b(xq, xs, wq, ws, wild, out=pad[1:-1], status=status)
        assert moe.moe_check(status) == 0      # (groups that overlap: more tiles than the rows can hold)
        assert bool((pad[0] == 3).all()) and bool((pad[-1] == 3).all())


@pytest.mark.parametrize("T", [50, 5000])
def test_rows_out_of_range_stay_their_own(moe, T):
    """A perm_tok outside [0, x_rows) spoils its own row alone."""
    E, K, N = 3, 256, 128
    off, perm, _ = grouping(T, E, 1, seed=1)
    xq, xs = pair(T, K)
    wq, ws = pair(N, K, seed=4, block_rows=128, lead=(E,))
    want = moe.moe_grouped_gemm_fp8b(xq, xs, wq, ws, off, perm_tok=perm)
    bad = perm.clone()
    bad[4], bad[17], bad[49] = -1, T, 2 ** 31 - 1
    got = moe.moe_grouped_gemm_fp8b(xq, xs, wq, ws, off, perm_tok=bad)
    keep = torch.ones(T, dtype=torch.bool, device=DEV)
    keep[[4, 17, 49]] = False
    assert torch.equal(got[keep], want[keep])


def test_empty(moe):
    f = lambda *s: torch.zeros(*s, device=DEV)
    q = lambda *s: torch.zeros(*s, device=DEV).to(F8)
    off = torch.zeros(5, dtype=torch.int32, device=DEV)
    assert moe.moe_gemm_fp8b(q(0, 128), f(0, 1), q(8, 128), f(1, 1)).shape == (0, 8)
    assert moe.moe_grouped_gemm_fp8b(q(0, 128), f(0, 1), q(4, 8, 128), f(4, 1, 1), off).shape == (0, 8)
    # rows, but no expert holds any
    out = torch.full((6, 8), 2.0, device=DEV)
    moe.moe_grouped_gemm_fp8b(q(6, 128), f(6, 1), q(4, 8, 128), f(4, 1, 1), off, out=out)
    assert bool((out == 2).all())


def test_given_workspace(moe):
    """A workspace of the caller's, used again by the next call; one too small."""
    T, E, K, N = 2000, 4, 256, 512
    off, perm, _ = grouping(T, E, 2, seed=1)
    xq, xs = pair(T, K)
    wq, ws = pair(N, K, seed=4, block_rows=128, lead=(E,))
    work = torch.empty(moe.moe_fp8b_workspace_size(2 * T, K), dtype=torch.uint8, device=DEV)
    want = moe.moe_grouped_gemm_fp8b(xq, xs, wq, ws, off, perm_tok=perm)
    h_want = moe.moe_gate_up_fp8b(xq, xs, wq, ws, wq, ws, offsets=off, perm_tok=perm)
    for _ in range(2):
        got = moe.moe_grouped_gemm_fp8b(xq, xs, wq, ws, off, perm_tok=perm, workspace=work)
        h = moe.moe_gate_up_fp8b(xq, xs, wq, ws, wq, ws, offsets=off, perm_tok=perm, workspace=work)
    assert torch.equal(got, want) and torch.equal(bits(h[0]), bits(h_want[0])) and torch.equal(h[1], h_want[1])
    with pytest.raises(moe.MoeError) as e:
        moe.moe_grouped_gemm_fp8b(xq, xs, wq, ws, off, perm_tok=perm, workspace=work[:-1])
    assert e.value.status == 3      # MOE_ERR_WORKSPACE


def test_few_and_many_rows_agree(moe):
    """The same rows through the few-rows kernel (alone) and the tiled one (among
    many): the sums differ by their order at most."""
    K, N = 1024, 640
    xq, xs = pair(6000, K)
    wq, ws = pair(N, K, seed=4, block_rows=128)
    many = moe.moe_gemm_fp8b(xq, xs, wq, ws, out_dtype=torch.float32)
    few = moe.moe_gemm_fp8b(xq[:20], xs[:20], wq, ws, out_dtype=torch.float32)
    tol = product_bound(value(xq[:20], xs[:20], 1), value(wq, ws, 128), K)
    assert bool(((many[:20].double() - few.double()).abs() <= 2 * tol).all())


def test_status_word(moe):
    status = torch.zeros(64, dtype=torch.int32, device=DEV)
    xq, xs = pair(40, 256)
    wq, ws = pair(300, 256, block_rows=128)
    moe.moe_gemm_fp8b(xq, xs, wq, ws, status=status)
    assert moe.moe_check(status) == 0


@pytest.mark.parametrize("T,E,K,N", [(1, 1, 1024, 256), (40, 24, 640, 512), (3000, 3, 256, 1040)])
def test_expired_wait_is_reported_and_not_silent(moe, T, E, K, N):
    """A wait that gives up (1 ms, on a barrier nothing arrives on) in the split,
    the few-rows and the tiled kernel: every row of a group is NaN, the other
    rows keep what they held, the status word reports the timeout, and the next
    call is right."""
    import ctypes
    L = moe.load_library()
    xq, xs = pair(T, K)
    wq, ws = pair(N, K, seed=4, block_rows=128, lead=(E,))
    off = torch.linspace(0, T, E + 1, device=DEV).int()
    off[-1] = max(T - 1, 1)
    status = torch.zeros(64, dtype=torch.int32, device=DEV)
    out = torch.full((T, N), 3.0, device=DEV)
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    st = L.moe_grouped_gemm_fp8b_expire_wait(p(xq), p(xs), T, K, K, p(wq), p(ws), E, N, p(off), None, T, p(out), 0, N,
                                             None, 0, p(status), 1_000_000,
                                             ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert st == 0
    with pytest.raises(moe.MoeError) as e:
        moe.moe_check(status)
    assert e.value.status == 5      # MOE_ERR_TIMEOUT
    n = int(off[-1])
    assert bool(out[:n].isnan().all()) and bool((out[n:] == 3).all())
    status.zero_()
    y = moe.moe_grouped_gemm_fp8b(xq, xs, wq, ws, off, out_dtype=torch.float32, status=status)
    assert moe.moe_check(status) == 0
    xv, wv = value(xq, xs, 1), value(wq, ws, 128)
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        check_product(y[a:b], xv[a:b], wv[e], K)


# split over a cluster, few rows, tiled; one or two blocks of K for a CTA, so that
# its loads and products are all issued before the sums give up, and more
SUMS = [(1, 1, 1024, 256), (40, 24, 256, 512), (3000, 3, 256, 1040), (1, 1, 2816, 256), (40, 24, 1024, 512), (3000, 3, 1040, 1040)]


@pytest.mark.parametrize("T,E,K,N", SUMS)
def test_expired_sums_are_reported(moe, T, E, K, N):
    """The wait of the summing warps gives up while every load and product goes
    on: the status word reports it too, also where the other warps have left
    their loops by then; rows are NaN, the rest is left, the next call is right."""
    import ctypes
    L = moe.load_library()
    xq, xs = pair(T, K)
    wq, ws = pair(N, K, seed=4, block_rows=128, lead=(E,))
    off = torch.linspace(0, T, E + 1, device=DEV).int()
    off[-1] = max(T - 1, 1)
    status = torch.zeros(64, dtype=torch.int32, device=DEV)
    out = torch.full((T, N), 3.0, device=DEV)
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    st = L.moe_grouped_gemm_fp8b_expire_sums(p(xq), p(xs), T, K, K, p(wq), p(ws), E, N, p(off), None, T, p(out), 0, N,
                                             None, 0, p(status), 1_000_000,
                                             ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert st == 0
    with pytest.raises(moe.MoeError) as e:
        moe.moe_check(status)
    assert e.value.status == 5      # MOE_ERR_TIMEOUT
    n = int(off[-1])
    assert bool(out[:n].isnan().all()) and bool((out[n:] == 3).all())
    status.zero_()
    y = moe.moe_grouped_gemm_fp8b(xq, xs, wq, ws, off, out_dtype=torch.float32, status=status)
    assert moe.moe_check(status) == 0
    xv, wv = value(xq, xs, 1), value(wq, ws, 128)
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        check_product(y[a:b], xv[a:b], wv[e], K)


@pytest.mark.parametrize("who", ["wait", "sums"])
@pytest.mark.parametrize("T,E,d,F", [(1, 1, 512, 256), (40, 24, 256, 272), (3000, 3, 256, 400), (1, 1, 2816, 256),
                                     (40, 24, 1024, 400), (3000, 3, 1040, 400)])
def test_expired_gate_up(moe, T, E, d, F, who):
    """The same for gate/up (split over a cluster, few rows, tiled), for the loads'
    wait and the sums': NaN codes with NaN scales, reported, the rest as it was."""
    import ctypes
    L = moe.load_library()
    xq, xs = pair(T, d)
    (gq, gs), (uq, us) = (quant(rand(E, F, d, seed=s, sd=d ** -0.5), 128) for s in (1, 2))
    off = torch.linspace(0, T, E + 1, device=DEV).int()
    off[-1] = max(T - 1, 1)
    status = torch.zeros(64, dtype=torch.int32, device=DEV)
    hq = torch.full((T, F), 5, dtype=torch.uint8, device=DEV)
    hs = torch.full((T, blocks(F)), 9.0, device=DEV)
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    hook = getattr(L, f"moe_gate_up_fp8b_expire_{who}")
    assert hook(p(xq), p(xs), T, d, d, p(gq), p(gs), p(uq), p(us), E, F, p(off), None, T, p(hq), p(hs), None, 0,
                p(status), 1_000_000, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
    with pytest.raises(moe.MoeError) as e:
        moe.moe_check(status)
    assert e.value.status == 5      # MOE_ERR_TIMEOUT
    n = int(off[-1])
    assert bool((hq[:n] == 0x7F).all()) and bool(hs[:n].isnan().all())
    assert bool((hq[n:] == 5).all()) and bool((hs[n:] == 9).all())
    status.zero_()
    hq, hs = moe.moe_gate_up_fp8b(xq, xs, gq, gs, uq, us, offsets=off, status=status)
    assert moe.moe_check(status) == 0
    xv, gv, uv = value(xq, xs, 1), value(gq, gs, 128), value(uq, us, 128)
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        if a < b:
            h, err = swiglu_ref(xv[a:b], gv[e], uv[e], d)
            check_codes(hq[a:b], hs[a:b], h, err)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("N", [4, 8, 16, 40])
def test_narrow_outputs_of_many_rows(moe, N, out):
    """Outputs narrower than the stores' boxes, rows 16 bytes apart and more."""
    T, K = 6000, 144
    xq, xs = pair(T, K)
    wq, ws = pair(N, K, seed=3, block_rows=128)
    wide = torch.full((T + 2, N), 3.0, dtype=DT[out], device=DEV)
    y = moe.moe_gemm_fp8b(xq, xs, wq, ws, out=wide[1:-1])
    check_product(y, value(xq, xs, 1), value(wq, ws, 128), K)
    assert bool((wide[0] == 3).all()) and bool((wide[-1] == 3).all())


# ------------------------------------- which kernel, and the tiled one's values

class KernelNode(ctypes.Structure):          # CUDA_KERNEL_NODE_PARAMS_v2
    _fields_ = [("func", ctypes.c_void_p), ("dims", ctypes.c_uint * 7), ("params", ctypes.c_void_p),
                ("extra", ctypes.c_void_p), ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


def kernel_of(call):
    """"tiled", "few rows" or "split": the product kernel that `call` launches, by
    the names of the kernels in its captured graph."""
    call()                                   # (set-up of a kernel's first launch is not captured)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    cu, raw, n = ctypes.CDLL("libcuda.so.1"), ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.c_size_t(0)
    assert cu.cuGraphGetNodes(raw, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert cu.cuGraphGetNodes(raw, nodes, ctypes.byref(n)) == 0
    names = []
    for node in nodes:
        kind, p, name = ctypes.c_int(-1), KernelNode(), ctypes.c_char_p()
        assert cu.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0
        if kind.value != 0:                  # CU_GRAPH_NODE_TYPE_KERNEL
            continue
        assert cu.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(p)) == 0
        get = (cu.cuFuncGetName, p.func) if p.func else (cu.cuKernelGetName, p.kern)
        assert get[0](ctypes.byref(name), ctypes.c_void_p(get[1])) == 0
        names.append(name.value.decode())
    if any("product_kernel" in m for m in names):
        return "tiled"
    few = [m for m in names if "decode_kernel" in m]
    assert len(few) == 1, names
    return "split" if "decode_kernelILi0ELb1E" in few[0] or "decode_kernelILi1ELb1E" in few[0] else "few rows"


def by_rule(rows, E, N, K, gate_up):
    """The rule for the product's kernel (fp8b_decode.cu) on this device."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    experts = min(E, rows)
    tiles = ((rows - experts) // 32 + experts) * blocks(N)
    if rows > 16 * experts and tiles > sms:
        return "tiled"
    return "split" if 2 * tiles <= sms and blocks(K) >= (4 if gate_up else 8) else "few rows"


TILED_GEMM = [(2500, 2816, 384), (4000, 1040, 1000), (3000, 272, 130), (5000, 144, 7), (2600, 640, 2050)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("T,K,N", TILED_GEMM)
def test_gemm_tiled(moe, out, T, K, N):
    """Sizes above the few-rows rule: long reductions, ragged last blocks."""
    xq, xs = pair(T, K)
    wq, ws = pair(N, K, seed=5, block_rows=128)
    call = lambda: moe.moe_gemm_fp8b(xq, xs, wq, ws, out_dtype=DT[out])
    assert kernel_of(call) == "tiled" == by_rule(T, 1, N, K, False)
    y = call()
    check_product(y, value(xq, xs, 1), value(wq, ws, 128), K)
    assert torch.equal(y, call())


@pytest.mark.parametrize("T", [254 * 20, 254 * 33 + 5])
def test_gemm_tiled_every_code(moe, T):
    """Every finite code of both signs on both sides through the tiled kernel."""
    codes = torch.tensor([c for c in range(256) if c & 0x7F != 0x7F], dtype=torch.uint8, device=DEV)   # 254
    K = 256
    left = codes.repeat(-(-T // 254))[:T]
    xq, wq = torch.zeros(T, K, dtype=torch.uint8, device=DEV), torch.zeros(254, K, dtype=torch.uint8, device=DEV)
    xq[:, 200], wq[:, 200] = left, codes
    xs, ws = torch.ones(T, 2, device=DEV), torch.ones(2, 2, device=DEV)
    call = lambda: moe.moe_gemm_fp8b(xq, xs, wq, ws, out_dtype=torch.float32)
    assert kernel_of(call) == "tiled" == by_rule(T, 1, 254, K, False)
    assert torch.equal(call().double(), left.view(F8).double()[:, None] * codes.view(F8).double()[None, :])


@pytest.mark.parametrize("T", [5000, 8191])
def test_gemm_tiled_scales_act_on_their_own_block(moe, T):
    """Scales of very different size per block of K, of N and per row; a zero and a
    NaN scale stay in their rows and columns, in the tiled kernel."""
    K, N = 5 * 128, 3 * 128 + 16
    xq, xs = pair(T, K)
    wq, ws = pair(N, K, seed=3, block_rows=128)
    xs = xs * 4.0 ** torch.randint(-8, 8, xs.shape, device=DEV)
    ws = ws * 4.0 ** torch.randint(-8, 8, ws.shape, device=DEV)
    xs[7] = 0
    call = lambda: moe.moe_gemm_fp8b(xq, xs, wq, ws, out_dtype=torch.float32)
    assert kernel_of(call) == "tiled" == by_rule(T, 1, N, K, False)
    check_product(call(), value(xq, xs, 1), value(wq, ws, 128), K)
    xs[9, 2], xs[T - 1, 4], ws[1, 3] = float("nan"), float("nan"), float("nan")
    bad = call().isnan()
    want = torch.zeros_like(bad)
    want[9] = want[T - 1] = True
    want[:, 128:256] = True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("T,d,F", [(3000, 272, 400), (3000, 1040, 384), (2700, 2816, 272), (6000, 144, 16)])
def test_gate_up_dense_tiled(moe, T, d, F):
    """The dense layer's call (no offsets) above the few-rows rule, with ragged last
    blocks of d and of F."""
    xq, xs = pair(T, d)
    (gq, gs), (uq, us) = (quant(rand(F, d, seed=s, sd=d ** -0.5), 128) for s in (1, 2))
    call = lambda: moe.moe_gate_up_fp8b(xq, xs, gq, gs, uq, us)
    assert kernel_of(call) == "tiled" == by_rule(T, 1, F, d, True)
    hq, hs = call()
    h, err = swiglu_ref(value(xq, xs, 1), value(gq, gs, 128), value(uq, us, 128), d)
    check_codes(hq, hs, h, err)


TILED_GROUPS = [(3000, 3, 1, 272, 400, 2.0), (2600, 8, 2, 400, 272, 1.0), (5000, 16, 1, 640, 384, 0.5), (4000, 64, 4, 144, 80, 1.0)]


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("T,E,k,K,N,skew", TILED_GROUPS)
def test_grouped_tiled(moe, T, E, k, K, N, skew, gather):
    """The grouped products and gate/up above the few-rows rule, ragged last blocks."""
    off, perm, _ = grouping(T, E, k, seed=T + E, skew=skew)
    rows = T * k
    xq, xs = pair(T if gather else rows, K)
    (gq, gs), (uq, us) = (quant(rand(E, N, K, seed=s, sd=K ** -0.5), 128) for s in (11, 12))
    p = perm if gather else None
    product = lambda: moe.moe_grouped_gemm_fp8b(xq, xs, gq, gs, off, perm_tok=p, out_dtype=torch.float32)
    gate_up = lambda: moe.moe_gate_up_fp8b(xq, xs, gq, gs, uq, us, offsets=off, perm_tok=p)
    assert kernel_of(product) == kernel_of(gate_up) == "tiled" == by_rule(rows, E, N, K, False)
    y, (hq, hs) = product(), gate_up()
    xv = value(xq, xs, 1)
    xv = xv[perm.long()] if gather else xv
    gv, uv = value(gq, gs, 128), value(uq, us, 128)
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        if a < b:
            check_product(y[a:b], xv[a:b], gv[e], K)
            h, err = swiglu_ref(xv[a:b], gv[e], uv[e], K)
            check_codes(hq[a:b], hs[a:b], h, err)


@pytest.mark.parametrize("T,E,K,N,gate_up,kind", [
    (1, 1, 1024, 256, False, "split"), (16, 1, 912, 1024, False, "split"), (16, 1, 896, 1024, False, "few rows"),
    (40, 24, 640, 512, False, "few rows"), (300, 1, 2816, 384, False, "split"), (2500, 1, 2816, 384, False, "tiled"),
    (1, 1, 512, 256, True, "split"), (16, 1, 384, 400, True, "few rows"), (300, 1, 256, 400, True, "few rows"),
    (3000, 1, 256, 400, True, "tiled")])
def test_which_kernel(moe, T, E, K, N, gate_up, kind):
    """The kernel that cases of these tests are meant for, by the rule and as launched."""
    off = torch.linspace(0, T, E + 1, device=DEV).int()
    xq, xs = pair(T, K)
    wq, ws = pair(N, K, seed=4, block_rows=128, lead=(E,))
    if gate_up:
        call = lambda: moe.moe_gate_up_fp8b(xq, xs, wq, ws, wq, ws, offsets=off)
    else:
        call = lambda: moe.moe_grouped_gemm_fp8b(xq, xs, wq, ws, off)
    assert kernel_of(call) == kind == by_rule(T, E, N, K, gate_up)


# --------------------------------------------------- streams, graphs, chains

def layer(E, d, F, seed):
    w = {n: quant(rand(E, *s, seed=seed + i, sd=s[1] ** -0.5), 128)
         for i, (n, s) in enumerate((("g", (F, d)), ("u", (F, d)), ("d", (d, F))))}
    return w | {"router": rand(E, d, seed=seed + 9, sd=d ** -0.5).bfloat16(), "bias": rand(E, seed=seed, sd=0.5),
                "norm": 1 + rand(d, seed=seed, sd=0.1)}


def run_layers(moe, x, layers, k, keep=None):
    """Layers of norm, route, permute, gate/up, down; each norm takes the
    combine of the layer before; a last norm ends the stack."""
    delta = topk_w = inv = None
    for w in layers:
        resid, normed, q, s = moe.moe_norm_fp8b(x, w["norm"], 1e-6, delta=delta, topk_w=topk_w, inv=inv)
        idx, topk_w = moe.moe_route(normed, w["router"], w["bias"], k)
        _, off, perm, inv = moe.moe_permute(idx, w["router"].shape[0])
        hq, hs = moe.moe_gate_up_fp8b(q, s, *w["g"], *w["u"], offsets=off, perm_tok=perm)
        y = moe.moe_grouped_gemm_fp8b(hq, hs, *w["d"], off)
        if keep is not None:
            keep.append(dict(x=x, delta=delta, resid=resid, normed=normed, q=q, s=s, idx=idx, topk_w=topk_w, off=off,
                             perm=perm, inv=inv, hq=hq, hs=hs, y=y))
        x, delta = resid, y
    return moe.moe_norm_fp8b(x, layers[0]["norm"], 1e-6, delta=delta, topk_w=topk_w, inv=inv)


@pytest.mark.parametrize("T,E,k,d,F", [(1, 8, 2, 256, 128), (96, 16, 2, 512, 256), (700, 8, 1, 256, 400), (64, 16, 4, 256, 256)])
def test_layers_in_a_row(moe, T, E, k, d, F):
    """Two expert layers as a serving loop runs them: every step against the
    definition on what the step was given, the end against the same stack of
    layers on unquantised values."""
    layers = [layer(E, d, F, seed=20 + i) for i in range(2)]
    x = rand(T, d, sd=2.0)
    keep = []
    resid, normed, q, s = run_layers(moe, x, layers, k, keep)
    prev = None
    for w, m in zip(layers, keep):
        check_norm(m["x"], w["norm"], 1e-6, (m["resid"] if prev else m["x"], m["normed"], m["q"], m["s"]), m["delta"],
                   prev and prev["topk_w"], prev and prev["inv"])
        slots = m["idx"].reshape(-1).long()
        assert torch.equal(m["perm"].long(), torch.argsort(slots, stable=True) // k)
        xv = value(m["q"], m["s"], 1)[m["perm"].long()]
        hv = value(m["hq"], m["hs"], 1)
        for e in range(E):
            a, b = int(m["off"][e]), int(m["off"][e + 1])
            if a < b:
                h, err = swiglu_ref(xv[a:b], value(*(t[e] for t in w["g"]), 128), value(*(t[e] for t in w["u"]), 128), d)
                check_codes(m["hq"][a:b], m["hs"][a:b], h, err)
                check_product(m["y"][a:b], hv[a:b], value(*(t[e] for t in w["d"]), 128), F)
        prev = m
    check_norm(prev["resid"], layers[0]["norm"], 1e-6, (resid, normed, q, s), prev["y"], prev["topk_w"], prev["inv"])


def test_layers_of_many_rows(moe):
    """Two layers whose products all take the tiled kernel, rows gathered."""
    test_layers_in_a_row(moe, 3000, 8, 2, 272, 400)


@pytest.mark.parametrize("T", [48, 1500])     # (the second gathers into a workspace)
def test_streams_and_captured_graphs(moe, T):
    """The stack of layers on a side stream, and captured and replayed with new
    inputs, gives what it gives eagerly, bit for bit; two captured graphs
    replayed side by side do not disturb each other."""
    E, k, d, F = 16, 2, 512, 256
    layers = [layer(E, d, F, seed=40 + i) for i in range(2)]
    xs = [rand(T, d, seed=i, sd=2.0) for i in range(4)]
    want = [run_layers(moe, x, layers, k) for x in xs]
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    with torch.cuda.stream(side[0]):
        got = run_layers(moe, xs[0], layers, k)
    side[0].synchronize()
    for a, b in zip(got, want[0]):
        assert torch.equal(a.float(), b.float())
    graphs = []
    for i in range(2):
        buf = xs[i].clone()
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            out = run_layers(moe, buf, layers, k)
        graphs.append((g, buf, out))
    for turn in range(2):
        for i, (g, buf, out) in enumerate(graphs):
            with torch.cuda.stream(side[i]):
                buf.copy_(xs[2 * turn + i])
                g.replay()
        torch.cuda.synchronize()
        for i, (g, buf, out) in enumerate(graphs):
            for a, b in zip(out, want[2 * turn + i]):
                assert torch.equal(a.float(), b.float())


def test_long_offsets(moe):
    """Rows whose byte and element offsets pass 2^31: the last rows of a tall
    output and of a tall input."""
    T, K, N = 1_200_000, 16, 2048          # out: 2.4e9 elements
    xq, xs = quant(rand(128, K), 1)
    xq = xq.view(torch.uint8).repeat(T // 128, 1)
    xs = xs.repeat(T // 128, 1)
    wq, ws = pair(N, K, seed=3, block_rows=128)
    y = moe.moe_gemm_fp8b(xq, xs, wq, ws)
    ref = moe.moe_gemm_fp8b(xq[:128], xs[:128], wq, ws)
    for at in (0, T // 2 // 128 * 128, T - 128):
        assert torch.equal(y[at:at + 128], ref)
    del xq, xs
    q, s = moe.moe_quant_fp8b(y)           # 2.4e9 codes
    rq, rs = quant(ref, 1)
    same_codes(q[-128:], rq)
    same_scales(s[-128:], rs)
