"""The 8-bit integer operators against their definitions in 64 bits.

Tolerances, derived before the first run:
  quantisation  code for code: the whole number nearest to the exact quotient; the scale is
             one fp32 divide.
  products   A = sum |x_q| |w_q|.  Below 2^24 every sum of codes' products is a whole number
             that fp32 holds: exact.  Otherwise each of the K additions is off by at most
             2^-23 of A.  The two scales are two fp32 products: y = sum * sx * sw is within
             (2 * 2^-24 + 2^-47) |y|, plus K 2^-23 A sx sw where A reaches 2^24.  A bf16
             output adds finfo.eps / 2 = 2^-8 |y|.
  gate/up    g and u as above; h = silu(g) u moves by |silu'| <= 1.1 times g's error, and
             silu itself is off by (5 + 1.18 |g|) 2^-23 (bf16 output: the fast exponential)
             or 2^-20 (fp32); where |g| > 87 it may be 0 for |g| 2^-126.  bf16 rounds once
             more, 2^-8.
  Results near the smallest normal number may lose 2^-149 (fp32) or 2^-133 (bf16) more.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import expert_routed_ffn_selectedsoftmax_gb300 as pkg
    torch.cuda.set_device(0)
    return pkg


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def rand(*shape, seed=0, sd=1.0):
    return torch.randn(*shape, generator=gen(seed + 1000 * len(shape) + sum(shape)), device=DEV) * sd


def codes(*shape, seed=0):
    """int8 codes of every size, and fp32 scales of a few magnitudes per row."""
    g = gen(seed + sum(shape))
    q = (torch.randn(*shape, generator=g, device=DEV) * 32).round().clamp(-127, 127).to(torch.int8)
    s = torch.exp(torch.randn(*shape[:-1], generator=g, device=DEV)) * 0.01
    return q, s


# ------------------------------------------------------------- quantisation

def check_quant(x, q, s):
    """Codes and scales of rows, exactly: 127 |x| and (n + 1/2) max|x| have at most 32 bits
    and are compared in 64."""
    assert q.dtype == torch.int8 and s.dtype == torch.float32 and q.shape == x.shape and s.shape == x.shape[:-1]
    v = x.double()
    top = v.abs().amax(-1)
    bad = ~torch.isfinite(top)
    assert torch.equal(s.isnan(), bad)
    want = (top.float() / torch.full_like(s, 127.0))       # (a tensor divisor: a true divide)
    want = torch.where(want < 2.0 ** -126, torch.zeros_like(want), want)
    assert torch.equal(s[~bad], want[~bad])
    zero = bad | (want == 0)
    assert not q[zero].any()
    v, top, q = v[~zero], top[~zero][:, None], q[~zero].double()
    left = 127.0 * v.abs()
    low = torch.floor(left / top)
    low = torch.where(low * top > left, low - 1, low)       # (a quotient that rounded up to a whole number)
    side = left - (low + 0.5) * top
    n = torch.where(side > 0, low + 1, torch.where(side < 0, low, low + low % 2))
    assert torch.equal(q.abs(), n)
    assert bool(((q == 0) | (q.sign() == v.sign())).all())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 2048), (3, 48), (37, 2816), (5, 1040), (4099, 512), (2500, 4096), (2433, 8192),
                                       (7, 8208), (2, 40000), (2600, 16400), (3000, 16), (2500, 2000)])
def test_quant(moe, dt, rows, cols):
    x = (rand(rows, cols) * torch.exp(rand(rows, 1, seed=1))).to(DT[dt])
    check_quant(x, *moe.moe_quant_i8(x))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_quant_on_borders(moe, dt):
    """Rows whose quotients are ties, one unit beside a tie, and beside whole numbers."""
    n = torch.arange(0, 127, device=DEV, dtype=torch.float64)
    rows = []
    for top in (127.0, 254.0, 127.0 * 2 ** -100, 127.0 * 2.0 ** 90, 1.0, 3.0, 0.7):
        tie = (n + 0.5) * top / 127
        for shift in (-2.0 ** -22, -2.0 ** -23, 0.0, 2.0 ** -23, 2.0 ** -22, 2.0 ** -8, -2.0 ** -8):
            for sign in (1, -1):
                rows.append(torch.cat([sign * tie * (1 + shift), torch.tensor([top], device=DEV, dtype=torch.float64)]))
    x = torch.stack(rows).to(DT[dt])
    check_quant(x, *moe.moe_quant_i8(x))
    many = x.repeat(30, 1)
    check_quant(many, *moe.moe_quant_i8(many))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [1, 3000])
def test_quant_special_rows(moe, dt, rows):
    x = rand(9, 160).repeat(rows, 1).view(rows, 9, 160).clone()
    x[:, 0] = 0
    x[:, 1] = 1e-44
    x[:, 2] *= 1e-36
    x[:, 3] *= 3e37
    x[:, 4, 5] = float("inf")
    x[:, 5, 77] = float("nan")
    x[:, 6, 3], x[:, 6, 4] = float("-inf"), float("nan")
    x[:, 7] = -0.0
    x = x.view(-1, 160).to(DT[dt])
    q, s = moe.moe_quant_i8(x)
    check_quant(x, q, s)
    assert bool(s.view(rows, 9)[:, 4:7].isnan().all())


def test_quant_strides_batches_and_given_outputs(moe):
    big = rand(2, 40, 512)
    x = big[..., 128:384]
    q, s = torch.ones(2, 40, 256, device=DEV, dtype=torch.int8), torch.zeros(2, 40, device=DEV)
    got = moe.moe_quant_i8(x, codes=q, scales=s)
    assert got[0] is q and got[1] is s
    check_quant(x, q, s)
    one = rand(5, 1, 64)                                   # batches of one row
    check_quant(one, *moe.moe_quant_i8(one))
    apart = rand(5, 3, 64)[:, :1]                          # ... that lie apart
    check_quant(apart, *moe.moe_quant_i8(apart))
    empty = moe.moe_quant_i8(x[:, :0])
    assert empty[0].shape == (2, 0, 256) and empty[1].shape == (2, 0)
    with pytest.raises(ValueError):
        moe.moe_quant_i8(big[:, ::2, :256][:, :3])
    with pytest.raises(moe.MoeError):
        moe.moe_quant_i8(rand(4, 24))


# ----------------------------------------------------------------- products

def product_ref(x, w, sx, sw):
    """(values, bound of their error) of one group, 64 bits; x [r, K], w [N, K] codes."""
    xd, wd = x.double(), w.double()
    scale = sx.double()[:, None] * sw.double()[None, :]
    y, a = xd @ wd.T, xd.abs() @ wd.abs().T
    extra = torch.where(a < 2.0 ** 24, 0.0, x.shape[1] * 2.0 ** -23 * a)
    ref = y * scale
    return ref, (2 * 2.0 ** -24 + 2.0 ** -47) * ref.abs() + extra * scale


def close(got, ref, bound):
    least = 2.0 ** -149 if got.dtype == torch.float32 else 2.0 ** -133
    half = torch.finfo(got.dtype).eps / 2 if got.dtype != torch.float32 else 0.0
    tol = bound + half * (ref.abs() + bound) + least
    assert bool((got.double().isnan() == ref.isnan()).all())
    worst = ((got.double() - ref).abs() - tol).nan_to_num(-1.0).max() if ref.numel() else torch.tensor(0.0)
    assert not worst > 0, f"off by {float(worst):.3e} more than the bound"


def swiglu_ref(g, eg, u, eu, f32):
    sig = torch.sigmoid(g)
    h = g * sig * u
    silu = (2.0 ** -20 if f32 else (5 + 1.18 * g.abs()) * 2.0 ** -23) * (h.abs() + 1.1 * eg * u.abs())
    silu = silu + torch.where(g.abs() > 87, g.abs() * 2.0 ** -126 * u.abs(), 0.0)
    return h, 1.1 * eg * (u.abs() + eu) + (g * sig).abs() * eu + silu


def groups(T, E, k, seed=0, skew=0.5):
    """offsets, perm_tok of k distinct experts per token."""
    scores = rand(T, E, seed=seed) + skew * rand(E, seed=seed + 1)
    slots = scores.topk(k, dim=1).indices.reshape(-1)
    order = torch.argsort(slots, stable=True)
    counts = torch.bincount(slots, minlength=E)
    off = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
    return off, (order // k).int()


def check_grouped(out, xq, xs, mats, off, tok):
    """`mats`: [(w_q, w_s)] for a product, two of them for gate/up."""
    off = off.tolist()
    for e in range(len(off) - 1):
        if off[e] == off[e + 1]:
            continue
        rows = tok[off[e]:off[e + 1]].long() if tok is not None else slice(off[e], off[e + 1])
        each = [product_ref(xq[rows], wq[e], xs[rows], ws[e]) for wq, ws in mats]
        if len(each) == 2:
            each = [swiglu_ref(*each[0], *each[1], out.dtype == torch.float32)]
        close(out[off[e]:off[e + 1]], *each[0])


DENSE = [(1, 16, 1), (1, 2048, 5632), (3, 48, 7), (8, 128, 128), (9, 1040, 333), (31, 512, 1024), (33, 2816, 200), (64, 64, 4096),
         (100, 4096, 131), (128, 256, 256), (129, 272, 257), (200, 1024, 2048), (300, 3600, 100), (513, 80, 640), (1000, 1536, 777),
         (2050, 2048, 640), (5000, 144, 1000)]


@pytest.mark.parametrize("odt", ["f32", "bf16"])
@pytest.mark.parametrize("T,K,N", DENSE)
def test_gemm(moe, odt, T, K, N):
    (xq, xs), (wq, ws) = codes(T, K), codes(N, K, seed=1)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = moe.moe_gemm_i8(xq, xs, wq, ws, out_dtype=DT[odt], status=st)
    assert out.shape == (T, N) and out.dtype == DT[odt] and int(st) == 0
    close(out, *product_ref(xq, wq, xs, ws))


@pytest.mark.parametrize("odt", ["f32", "bf16"])
@pytest.mark.parametrize("T,d,F", DENSE)
def test_gate_up_dense(moe, odt, T, d, F):
    (xq, xs), (gq, gs), (uq, us) = codes(T, d), codes(F, d, seed=1), codes(F, d, seed=2)
    out = moe.moe_gate_up_i8(xq, xs, gq, gs, uq, us, h_dtype=DT[odt])
    assert out.shape == (T, F) and out.dtype == DT[odt]
    g, u = product_ref(xq, gq, xs, gs), product_ref(xq, uq, xs, us)
    close(out, *swiglu_ref(*g, *u, odt == "f32"))


GROUPED = [(1, 4, 1, 64, 100), (1, 64, 2, 1024, 512), (64, 16, 1, 2816, 256), (128, 64, 2, 1024, 512), (7, 8, 8, 272, 130),
           (300, 3, 2, 512, 700), (2000, 5, 2, 400, 513), (1024, 64, 2, 512, 384), (4096, 16, 1, 256, 320), (3, 256, 4, 128, 64),
           (900, 2, 1, 2064, 129)]


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("T,E,k,K,N", GROUPED)
def test_grouped_gemm(moe, gather, T, E, k, K, N):
    off, tok = groups(T, E, k)
    (xq, xs), (wq, ws) = codes(T if gather else T * k, K), codes(E, N, K, seed=1)
    for odt in (torch.bfloat16, torch.float32):
        out = moe.moe_grouped_gemm_i8(xq, xs, wq, ws, off, perm_tok=tok if gather else None, out_dtype=odt)
        check_grouped(out, xq, xs, [(wq, ws)], off, tok if gather else None)


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("T,E,k,d,F", GROUPED)
def test_gate_up_grouped(moe, gather, T, E, k, d, F):
    off, tok = groups(T, E, k)
    (xq, xs), (gq, gs), (uq, us) = codes(T if gather else T * k, d), codes(E, F, d, seed=1), codes(E, F, d, seed=2)
    for odt in (torch.bfloat16, torch.float32):
        out = moe.moe_gate_up_i8(xq, xs, gq, gs, uq, us, offsets=off, perm_tok=tok if gather else None, h_dtype=odt)
        check_grouped(out, xq, xs, [(gq, gs), (uq, us)], off, tok if gather else None)


@pytest.mark.parametrize("T,K,N", [(1, 1024, 40), (5, 1024, 40), (20, 1024, 200), (300, 1024, 200), (700, 1024, 300)])
def test_largest_codes_add_up_exactly(moe, T, K, N):
    """Rows of -128 and 127 at K = 1024, the largest sums that are exact: 2^24 itself (a power
    of two) and whole numbers below, for any order of the sums."""
    xq = torch.full((T, K), -128, dtype=torch.int8, device=DEV)
    wq = torch.full((N, K), -128, dtype=torch.int8, device=DEV)
    xq[1::3], wq[1::3] = 127, 127
    xq[2::3, ::2], wq[2::3, 1::3] = 127, 1
    one = lambda n: torch.ones(n, device=DEV)
    out = moe.moe_gemm_i8(xq, one(T), wq, one(N), out_dtype=torch.float32)
    assert torch.equal(out.double(), xq.double() @ wq.double().T)


@pytest.mark.parametrize("T", [2, 40, 300])
def test_long_reductions_of_large_codes(moe, T):
    """Sums beyond 2^24."""
    K, N = 16384, 140
    xq = torch.randint(100, 128, (T, K), generator=gen(1), device=DEV).to(torch.int8)
    wq = torch.randint(100, 128, (N, K), generator=gen(2), device=DEV).to(torch.int8)
    xs, ws = torch.full((T,), 0.01, device=DEV), torch.full((N,), 0.02, device=DEV)
    close(moe.moe_gemm_i8(xq, xs, wq, ws, out_dtype=torch.float32), *product_ref(xq, wq, xs, ws))


@pytest.mark.parametrize("rows", [3, 40, 600])
def test_scales_of_every_kind(moe, rows):
    """Zero, NaN, infinite, tiny and large scales: a row's reach that row, a channel's that
    channel."""
    K, N = 256, 150
    (xq, xs), (wq, ws) = codes(rows, K), codes(N, K, seed=1)
    xs, ws = xs.clone(), ws.clone()
    xs[0], xs[1], xs[2] = 0.0, float("nan"), 1e30
    ws[0], ws[1], ws[2], ws[3] = 0.0, float("nan"), 1e-30, 2.0 ** -126
    out = moe.moe_gemm_i8(xq, xs, wq, ws, out_dtype=torch.float32)
    ref, bound = product_ref(xq, wq, xs, ws)
    close(out, ref, bound)
    assert bool(out[1].isnan().all()) and bool(out[:, 1].isnan().all())
    h = moe.moe_gate_up_i8(xq, xs, wq, ws, wq, ws, h_dtype=torch.float32)
    assert bool(h[1].isnan().all()) and bool(h[:, 1].isnan().all())
    assert not h[0, 2:].any()


@pytest.mark.parametrize("odt", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [3, 40, 600])
def test_gate_sums_from_minus_200_to_200(moe, odt, rows):
    """SwiGLU where the exponential overflows and vanishes."""
    K, N = 128, 160
    (xq, _), (gq, _), (uq, us) = codes(rows, K), codes(N, K, seed=1), codes(N, K, seed=2)
    sums = xq.double() @ gq.double().T
    xs = (torch.rand(rows, generator=gen(4), device=DEV) * 200 / sums.abs().amax(1)).float()
    gs = torch.ones(N, device=DEV)
    h = moe.moe_gate_up_i8(xq, xs, gq, gs, uq, us, h_dtype=DT[odt])
    g, u = product_ref(xq, gq, xs, gs), product_ref(xq, uq, xs, us)
    assert float(g[0].max()) > 100 and float(g[0].min()) < -100
    close(h, *swiglu_ref(*g, *u, odt == "f32"))


@pytest.mark.parametrize("gate_up", [False, True])
@pytest.mark.parametrize("rows", [6, 70, 400])
def test_groups_of_every_kind(moe, rows, gate_up):
    """Empty groups, one with everything, groups that end before the last row (a padded
    batch: those rows stay), offsets out of range and in disorder, bad token indices."""
    K, N, E = 144, 72, 5
    (xq, xs), (wq, ws), (uq, us) = codes(rows, K), codes(E, N, K, seed=1), codes(E, N, K, seed=2)
    mats = [(wq, ws), (uq, us)] if gate_up else [(wq, ws)]

    def call(off, tok=None, out=None):
        if gate_up:
            return moe.moe_gate_up_i8(xq, xs, wq, ws, uq, us, offsets=off, perm_tok=tok, h=out)
        return moe.moe_grouped_gemm_i8(xq, xs, wq, ws, off, perm_tok=tok, out=out)
    half = rows // 2
    for cut in ([0, 0, 0, 0, 0, 0], [0, 0, rows, rows, rows, rows], [0, 1, 1, 2, half, half], [0, half, half, half, half, rows]):
        off = torch.tensor(cut, dtype=torch.int32, device=DEV)
        out = torch.full((rows, N), 7.0, device=DEV, dtype=torch.bfloat16)
        assert call(off, out=out) is out
        check_grouped(out, xq, xs, mats, off, None)
        assert bool((out[cut[-1]:] == 7).all())
    for cut in ([-5, 2, 2, half, half, 10 ** 9], [0, half, 1, rows, rows, rows]):   # clamped; a group that ends before it begins is empty
        off = torch.tensor(cut, dtype=torch.int32, device=DEV)
        assert call(off).shape == (rows, N)
    tok = torch.arange(rows, device=DEV).int().flip(0).contiguous()
    bad = tok.clone()
    bad[1], bad[4] = -7, rows
    off = torch.tensor([0, 1, half, half, rows, rows], dtype=torch.int32, device=DEV)
    a, b = call(off, tok), call(off, bad)
    keep = torch.ones(rows, dtype=torch.bool, device=DEV)
    keep[1] = keep[4] = False
    check_grouped(a, xq, xs, mats, off, tok)
    assert torch.equal(a[keep], b[keep])


def test_groups_that_overlap(moe):
    """Offsets in disorder can put more tiles on the groups than there are rows: the call
    ends, and rows that one group alone holds are right."""
    rows, K, N, E = 64, 256, 130, 8
    (xq, xs), (wq, ws) = codes(rows, K), codes(E, N, K, seed=1)
    off = torch.tensor([0, 64, 0, 64, 0, 64, 0, 64, 0], dtype=torch.int32, device=DEV)
    assert moe.moe_grouped_gemm_i8(xq, xs, wq, ws, off).shape == (rows, N)
    torch.cuda.synchronize()


@pytest.mark.parametrize("odt", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 9, 40, 300, 900])
@pytest.mark.parametrize("off,N,wide", [(0, 64, 80), (1, 129, 140), (8, 200, 224), (3, 61, 70), (0, 260, 260)])
def test_rows_apart_and_unaligned_outputs(moe, odt, T, off, N, wide):
    """x rows and output rows further apart than their length, outputs on any boundary of
    their type; what lies beside the output stays."""
    K = 192
    big, xs = codes(T, 256)
    xq = big[:, 32:32 + K]
    wq, ws = codes(N, K, seed=1)
    base = torch.full((T, wide), 7.0, device=DEV, dtype=DT[odt])
    out = base[:, off:off + N]
    moe.moe_gemm_i8(xq, xs, wq, ws, out=out)
    close(out, *product_ref(xq, wq, xs, ws))
    assert bool((base[:, :off] == 7).all()) and bool((base[:, off + N:] == 7).all())
    base.fill_(7.0)
    moe.moe_gate_up_i8(xq, xs, wq, ws, wq, ws, h=out)
    g = product_ref(xq, wq, xs, ws)
    close(out, *swiglu_ref(*g, *g, odt == "f32"))
    assert bool((base[:, :off] == 7).all()) and bool((base[:, off + N:] == 7).all())


def test_empty_calls_and_device_refusals(moe):
    (xq, xs), (wq, ws) = codes(4, 64), codes(2, 32, 64, seed=1)
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    assert moe.moe_gemm_i8(xq[:0], xs[:0], wq[0], ws[0]).shape == (0, 32)
    assert moe.moe_grouped_gemm_i8(xq, xs, wq, ws, off, perm_tok=off[:0]).shape == (0, 32)
    assert moe.moe_gate_up_i8(xq[:0], xs[:0], wq, ws, wq, ws, offsets=off).shape == (0, 32)
    with pytest.raises(ValueError):
        moe.moe_gemm_i8(xq, xs.cpu(), wq[0], ws[0])
    with pytest.raises(moe.MoeError):
        moe.moe_gemm_i8(codes(4, 24)[0], xs, codes(5, 24)[0], torch.ones(5, device=DEV))
    with pytest.raises(moe.MoeError):                      # rows that do not begin on 16 bytes
        moe.moe_gemm_i8(codes(4, 80)[0][:, 8:72], xs, wq[0], ws[0])


def test_codes_beyond_32_bits(moe):
    """Weights whose codes lie past 2^31, and output rows past 2^31 elements."""
    E, N, K = 256, 2100, 4096                              # 2.2e9 codes
    wq = torch.zeros(E, N, K, dtype=torch.int8, device=DEV)
    ws = torch.zeros(E, N, device=DEV)
    tail, ts = codes(2, N, K, seed=3)
    wq[-2:], ws[-2:] = tail, ts
    for rows in (4, 6000):
        xq, xs = codes(rows, K)
        off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
        off[-2], off[-1] = rows // 2, rows
        out = moe.moe_grouped_gemm_i8(xq, xs, wq, ws, off, out_dtype=torch.float32)
        pick = torch.tensor([0, rows // 2 - 1, rows // 2, rows - 1], device=DEV)
        for i, r in enumerate(pick.tolist()):
            close(out[r:r + 1], *product_ref(xq[r:r + 1], tail[i // 2], xs[r:r + 1], ts[i // 2]))


# ----------------------------------------------------------- an expert layer

def layer(moe, x, wr, bias, k, g, u, dn, E):
    idx, w = moe.moe_route(x, wr, bias, k)
    _, off, tok, inv = moe.moe_permute(idx, E)
    xq, xs = moe.moe_quant_i8(x)
    h = moe.moe_gate_up_i8(xq, xs, *g, *u, offsets=off, perm_tok=tok)
    hq, hs = moe.moe_quant_i8(h)
    y = moe.moe_grouped_gemm_i8(hq, hs, *dn, off)
    return moe.moe_combine(y, w, inv), (idx, w, off, tok, inv, xq, xs, h, hq, hs, y)


@pytest.mark.parametrize("T,d,E,k,F", [(1, 256, 8, 2, 128), (64, 512, 16, 1, 304), (300, 256, 8, 2, 208), (2000, 384, 4, 2, 512)])
def test_an_expert_layer(moe, T, d, E, k, F):
    """route, permute, quant, gate/up, quant, down, combine: every step against 64 bits on the
    step before's own outputs; on a side stream and replayed from a graph the same bits; and
    the same rows through dispatch."""
    x = rand(T, d).bfloat16()
    wr, bias = rand(E, d, sd=d ** -0.5).bfloat16(), rand(E, sd=0.3)
    g, u, dn = (moe.moe_quant_i8(rand(*s, sd=s[2] ** -0.5, seed=i)) for i, s in enumerate(((E, F, d), (E, F, d), (E, d, F))))
    args = (moe, x, wr, bias, k, g, u, dn, E)
    out, (idx, w, off, tok, inv, xq, xs, h, hq, hs, y) = layer(*args)
    check_quant(x, xq, xs)
    check_grouped(h, xq, xs, [g, u], off, tok)
    check_quant(h, hq, hs)
    check_grouped(y, hq, hs, [dn], off, None)
    rows = y.double()[inv.view(T, k).long()] * w.double()[..., None]
    close(out, rows.sum(1), k * 2.0 ** -24 * rows.abs().sum(1) * (1 + 1e-6))
    # rows sent to their experts first: the same products
    grouped = moe.moe_dispatch(x, inv, k)
    gq, gs = moe.moe_quant_i8(grouped)
    assert torch.equal(gq, xq[tok.long()]) and torch.equal(gs, xs[tok.long()])
    assert torch.equal(moe.moe_gate_up_i8(gq, gs, *g, *u, offsets=off), h)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        there = layer(*args)[0]
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(there, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = layer(*args)[0]
    for seed in (5, 6):
        x.copy_(rand(T, d, seed=seed).bfloat16())
        graph.replay()
        assert torch.equal(held, layer(*args)[0])


@pytest.mark.parametrize("role", [0, 1, 2])
@pytest.mark.parametrize("gate_up", [False, True])
@pytest.mark.parametrize("T,K,N,E", [(20, 2048, 300, 1), (300, 256, 200, 6), (3000, 2048, 520, 3)])   # split, few rows, tiled
def test_a_wait_that_expires(moe, T, K, N, E, gate_up, role):
    """The first wait of the loads, the converters or the sums gives up after 1 ms in every
    CTA (nothing arrives on its barrier): NaN rows, the status word, rows outside the groups as
    they were, and the next call right."""
    import ctypes
    L = moe.load_library()
    (xq, xs), (wq, ws), (uq, us) = codes(T, K), codes(E, N, K, seed=1), codes(E, N, K, seed=2)
    cut = [T * e // (E + 1) for e in range(E + 1)]         # (rows behind the last group)
    off = torch.tensor(cut, dtype=torch.int32, device=DEV)
    out = torch.full((T, N), 7.0, device=DEV)
    scratch = torch.empty(max(moe.moe_i8_workspace_size(T, K), 256), dtype=torch.uint8, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    tail = (E, N, p(off), None, T, p(out), 0, N, p(scratch), scratch.numel(), p(st), role, 1_000_000,
            ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    if gate_up:
        assert L.moe_gate_up_i8_expire_wait(p(xq), p(xs), T, K, K, p(wq), p(ws), p(uq), p(us), *tail) == 0
    else:
        assert L.moe_grouped_gemm_i8_expire_wait(p(xq), p(xs), T, K, K, p(wq), p(ws), *tail) == 0
    torch.cuda.synchronize()
    assert bool(out[:cut[-1]].isnan().all()) and bool((out[cut[-1]:] == 7).all()) and int(st) & 1
    with pytest.raises(moe.MoeError):
        moe.moe_check(st)
    st.zero_()
    if gate_up:
        moe.moe_gate_up_i8(xq, xs, wq, ws, uq, us, offsets=off, h=out, workspace=scratch, status=st)
    else:
        moe.moe_grouped_gemm_i8(xq, xs, wq, ws, off, out=out, workspace=scratch, status=st)
    check_grouped(out, xq, xs, [(wq, ws), (uq, us)] if gate_up else [(wq, ws)], off, None)
    assert bool((out[cut[-1]:] == 7).all()) and moe.moe_check(st) == 0


@pytest.mark.parametrize("T,E,d,F", [(512, 16, 2048, 2816), (128, 16, 2048, 2816), (20, 1, 8192, 2048), (6, 2, 8192, 4096), (1500, 16, 2048, 2816)])
def test_weights_that_come_late(moe, T, E, d, F):
    """Weights from HBM, larger than the L2 together, whose blocks may land out of order: the
    converters of a block wait for that block.  Every call's outputs are the same, and those of
    one call right."""
    off, tok = groups(T, E, 1)
    xq, xs = codes(T, d)
    sets = [(codes(E, F, d, seed=i), codes(E, F, d, seed=i + 7)) for i in range(3)]
    first = [None] * 3
    for turn in range(30):
        (gq, gs), (uq, us) = sets[turn % 3]
        h = moe.moe_gate_up_i8(xq, xs, gq, gs, uq, us, offsets=off, perm_tok=tok)
        y = moe.moe_grouped_gemm_i8(xq, xs, uq, us, off, perm_tok=tok)
        if first[turn % 3] is None:
            first[turn % 3] = (h, y)
        assert torch.equal(h, first[turn % 3][0]) and torch.equal(y, first[turn % 3][1])
    g, u = sets[0]
    check_grouped(first[0][0], xq, xs, [g, u], off, tok)
    check_grouped(first[0][1], xq, xs, [u], off, tok)


@pytest.mark.parametrize("T,K,N", [(64, 2048, 5632), (700, 4096, 1024), (1000, 1536, 777), (2050, 2048, 640), (24, 4096, 2048),
                                   (3000, 2048, 2048), (8, 8192, 1024)])
def test_repeated_calls(moe, T, K, N):
    """Calls back to back on fresh codes, each against 64 bits: a block that is read while the
    next one lands, or before it has, shows in some of many."""
    for turn in range(40):
        (xq, xs), (wq, ws) = codes(T, K, seed=turn), codes(N, K, seed=turn + 1)
        outs = [moe.moe_gemm_i8(xq, xs, wq, ws, out_dtype=torch.float32) for _ in range(4)]
        ref, bound = product_ref(xq, wq, xs, ws)
        for out in outs:
            close(out, ref, bound)


def test_two_calls_at_once(moe):
    """Two streams with calls of their own workspaces; one workspace shared by calls in order."""
    T, K, N = 700, 512, 640
    (xq, xs), (wq, ws) = codes(T, K), codes(N, K, seed=1)
    want = moe.moe_gemm_i8(xq, xs, wq, ws)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(moe.moe_gemm_i8(xq, xs, wq, ws))
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(o, want) for each in outs for o in each)
    shared = torch.empty(max(moe.moe_i8_workspace_size(T, K), 256), dtype=torch.uint8, device=DEV)
    other, os_ = codes(T, K, seed=9)
    a = moe.moe_gemm_i8(xq, xs, wq, ws, workspace=shared)
    b = moe.moe_gemm_i8(other, os_, wq, ws, workspace=shared)
    assert torch.equal(a, want) and torch.equal(b, moe.moe_gemm_i8(other, os_, wq, ws))


def tiled_scratch(moe, rows, K):
    """A workspace whose bytes tell whether a call wrote it: the 128-token tiles' kernel does."""
    return torch.full((moe.moe_i8_workspace_size(rows, K),), 0xA5, dtype=torch.uint8, device=DEV)


@pytest.mark.parametrize("odt", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1057, 1100, 1169])          # last tiles of 33, 76 and 17 tokens
@pytest.mark.parametrize("off,N,wide", [(0, 640, 640), (0, 600, 648), (8, 584, 616), (1, 577, 700), (3, 517, 540)])
def test_tiled_outputs(moe, odt, T, off, N, wide):
    """128-token tiles: output rows that go out whole, that end inside a tile, and that lie on
    any boundary of their type; x rows apart; what lies beside the output stays."""
    K = 3088
    big, xs = codes(T, 3200)
    xq = big[:, 48:48 + K]
    (wq, ws), (uq, us) = codes(N, K, seed=1), codes(N, K, seed=2)
    base = torch.full((T, wide), 7.0, device=DEV, dtype=DT[odt])
    out = base[:, off:off + N]
    y, u = product_ref(xq, wq, xs, ws), product_ref(xq, uq, xs, us)
    for gate_up in (False, True):
        base.fill_(7.0)
        scratch = tiled_scratch(moe, T, K)
        if gate_up:
            moe.moe_gate_up_i8(xq, xs, wq, ws, uq, us, h=out, workspace=scratch)
            close(out, *swiglu_ref(*y, *u, odt == "f32"))
        else:
            moe.moe_gemm_i8(xq, xs, wq, ws, out=out, workspace=scratch)
            close(out, *y)
        assert bool((base[:, :off] == 7).all()) and bool((base[:, off + N:] == 7).all())
        assert not bool((scratch == 0xA5).all())


@pytest.mark.parametrize("odt", ["f32", "bf16"])
@pytest.mark.parametrize("gate_up", [False, True])
@pytest.mark.parametrize("sizes,N", [([700, 0, 1, 129, 128, 17, 400], 777), ([0, 0, 1500], 777), ([33, 1000, 5, 6], 1000)])
def test_tiled_groups(moe, odt, gate_up, sizes, N):
    """128-token tiles of ragged groups, gathered from tokens named more than once; grouped rows
    behind the last group stay."""
    K, x_rows, E = 2064, 500, len(sizes)
    (xq, xs), (wq, ws), (uq, us) = codes(x_rows, K), codes(E, N, K, seed=1), codes(E, N, K, seed=2)
    off = torch.tensor([0] + sizes, device=DEV).cumsum(0).int()
    used = sum(sizes)
    rows = used + 50
    tok = torch.randint(0, x_rows, (rows,), device=DEV, dtype=torch.int32)
    out = torch.full((rows, N), 7.0, device=DEV, dtype=DT[odt])
    scratch = tiled_scratch(moe, rows, K)
    if gate_up:
        moe.moe_gate_up_i8(xq, xs, wq, ws, uq, us, offsets=off, perm_tok=tok, h=out, workspace=scratch)
    else:
        moe.moe_grouped_gemm_i8(xq, xs, wq, ws, off, perm_tok=tok, out=out, workspace=scratch)
    check_grouped(out, xq, xs, [(wq, ws), (uq, us)] if gate_up else [(wq, ws)], off, tok)
    assert bool((out[used:] == 7).all()) and not bool((scratch == 0xA5).all())


def test_two_tiled_calls_at_once(moe):
    """128-token tiles on two streams and as two captured graphs replayed side by side, each
    call with a workspace of its own."""
    T, K, N = 700, 4096, 1024
    sets = [(codes(T, K, seed=i), codes(N, K, seed=i + 1)) for i in range(2)]
    scratch = [tiled_scratch(moe, T, K) for _ in sets]
    want = [moe.moe_gemm_i8(*x, *w) for x, w in sets]
    outs = [torch.empty_like(v) for v in want]
    calls = [lambda i=i: moe.moe_gemm_i8(*sets[i][0], *sets[i][1], out=outs[i], workspace=scratch[i]) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in sets]
    graphs = []
    for call in calls:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            for _ in range(4):
                call()
    for run in (calls, [g.replay for g in graphs]):
        for o in outs:
            o.zero_()
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        for _ in range(6):
            for i, s in enumerate(streams):
                with torch.cuda.stream(s):
                    run[i]()
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        assert all(torch.equal(o, v) for o, v in zip(outs, want))
    assert all(not bool((s == 0xA5).all()) for s in scratch)


# (tokens, columns, channels): the reduction of a 128-token tile is split over clusters of 2, 4 and 8
SPLIT_TILES = [(1000, 4096, 1001), (300, 8192, 1000), (107, 16384, 899), (401, 8208, 640)]


@pytest.mark.parametrize("odt", ["f32", "bf16"])
@pytest.mark.parametrize("T,K,N", SPLIT_TILES)
def test_tiles_split_over_clusters(moe, odt, T, K, N):
    (xq, xs), (wq, ws), (uq, us) = codes(T, K), codes(N, K, seed=1), codes(N, K, seed=2)
    y, u = product_ref(xq, wq, xs, ws), product_ref(xq, uq, xs, us)
    base = torch.full((T, N + 5), 7.0, device=DEV, dtype=DT[odt])
    for gate_up in (False, True):
        scratch, out = tiled_scratch(moe, T, K), base[:, 3:3 + N]
        for _ in range(3):
            base.fill_(7.0)
            if gate_up:
                moe.moe_gate_up_i8(xq, xs, wq, ws, uq, us, h=out, workspace=scratch)
                close(out, *swiglu_ref(*y, *u, odt == "f32"))
            else:
                moe.moe_gemm_i8(xq, xs, wq, ws, out=out, workspace=scratch)
                close(out, *y)
            assert bool((base[:, :3] == 7).all()) and bool((base[:, 3 + N:] == 7).all())
        assert not bool((scratch == 0xA5).all())


@pytest.mark.parametrize("gate_up", [False, True])
@pytest.mark.parametrize("sizes,N", [([333], 640), ([0, 200, 133], 640), ([129, 0, 1, 70], 512)])
def test_groups_of_split_tiles(moe, gate_up, sizes, N):
    """Fewer tiles than the grid has clusters for, rows behind the last group."""
    K, E = 8192, len(sizes)
    off = torch.tensor([0] + sizes, device=DEV).cumsum(0).int()
    used = sum(sizes)
    (xq, xs), (wq, ws), (uq, us) = codes(used + 40, K), codes(E, N, K, seed=1), codes(E, N, K, seed=2)
    for odt in (torch.float32, torch.bfloat16):
        out = torch.full((used + 40, N), 7.0, device=DEV, dtype=odt)
        if gate_up:
            moe.moe_gate_up_i8(xq, xs, wq, ws, uq, us, offsets=off, h=out)
        else:
            moe.moe_grouped_gemm_i8(xq, xs, wq, ws, off, out=out)
        check_grouped(out, xq, xs, [(wq, ws), (uq, us)] if gate_up else [(wq, ws)], off, None)
        assert bool((out[used:] == 7).all())


@pytest.mark.parametrize("role", [0, 1, 2])
@pytest.mark.parametrize("gate_up", [False, True])
def test_a_wait_that_expires_in_a_split_tile(moe, gate_up, role):
    test_a_wait_that_expires(moe, 400, 8192, 640, 1, gate_up, role)


def test_split_tiles_side_by_side(moe):
    """Clusters of two calls on two streams, more than run at the same time, and captured."""
    T, K, N = 512, 8192, 1024
    sets = [(codes(T, K, seed=i), codes(N, K, seed=i + 1)) for i in range(2)]
    want = [moe.moe_gemm_i8(*x, *w) for x, w in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    outs = [[], []]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(moe.moe_gemm_i8(*sets[i][0], *sets[i][1]))
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(o, v) for each, v in zip(outs, want) for o in each)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = [moe.moe_gemm_i8(*x, *w) for x, w in sets]
    for _ in range(5):
        graph.replay()
    assert all(torch.equal(o, v) for o, v in zip(held, want))


def test_the_first_call_of_a_process_is_captured():
    """Kernel attributes and the number of clusters that run at once are asked for inside a
    capture: of the split tiles, the whole ones, the few-rows and the CUDA-core kernel."""
    import subprocess
    import sys
    code = """
import torch
import expert_routed_ffn_selectedsoftmax_gb300 as moe
moe.load_library()
c = lambda *s: (torch.randint(-127, 128, s, dtype=torch.int8, device="cuda"), torch.rand(*s[:-1], device="cuda"))
sizes = [(512, 8192, 1024), (3000, 512, 2048), (64, 512, 512), (1, 512, 512)]
sets = [(c(T, K), c(N, K)) for T, K, N in sizes]
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    held = [moe.moe_gemm_i8(*x, *w) for x, w in sets]
for _ in range(2):
    graph.replay()
assert all(torch.equal(o, moe.moe_gemm_i8(*x, *w)) for o, (x, w) in zip(held, sets))
for o, ((x, xs), (w, ws)) in zip(held, sets):
    ref = (x.double() @ w.double().T) * xs.double()[:, None] * ws.double()
    a = (x.double().abs() @ w.double().abs().T) * xs.double()[:, None] * ws.double()
    assert bool(((o.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + x.shape[1] * 2.0 ** -23 * a).all())
print("right")
"""
    done = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and "right" in done.stdout, done.stderr[-2000:]


@pytest.mark.parametrize("odt", ["f32", "bf16"])
@pytest.mark.parametrize("rows,K,N", [(2, 128, 700), (40, 128, 400), (600, 128, 160), (1100, 3088, 600), (300, 8192, 1000)])
def test_far_negative_gates(moe, odt, rows, K, N):
    """Gate sums down to -110 beside factors of 1e30: silu(g) there is small, not 0.  In the
    CUDA-core, the few-rows and the tiled kernel, whole and split.
    Bounds: silu as in the header, (5 + 1.18 |g|) 2^-23 or 5 2^-23 of itself and, below the normal
    numbers, (|g| + 2) 2^-149; g is two products of fp32 (2^-23 |g| at most), which silu's slope
    |1 + g| exp(g) carries on (1.01 for its change on the way); u three roundings, 2^-22."""
    (xq, _), (gq, _), (uq, _) = codes(rows, K), codes(N, K, seed=1), codes(N, K, seed=2)
    sums = xq.double() @ gq.double().T
    xs = (110.0 / -sums.amin(1)).float()
    gs, us = torch.ones(N, device=DEV), torch.full((N,), 1e30, device=DEV)
    scratch = tiled_scratch(moe, rows, K) if K > 128 else None
    h = moe.moe_gate_up_i8(xq, xs, gq, gs, uq, us, h_dtype=DT[odt], workspace=scratch)
    assert scratch is None or not bool((scratch == 0xA5).all())
    g = sums * xs.double()[:, None]
    u = (xq.double() @ uq.double().T) * xs.double()[:, None] * us.double()
    ref = g * torch.sigmoid(g) * u
    rel = 5 * 2.0 ** -23 if odt == "f32" else (5 + 1.18 * g.abs()) * 2.0 ** -23
    bound = rel * ref.abs() + 1.01 * (1 + g).abs() * torch.exp(torch.minimum(g, -g)) * 2.0 ** -23 * g.abs() * u.abs()
    bound = torch.where(g > -2, 1.1 * 2.0 ** -23 * g.abs() * u.abs() + rel * ref.abs(), bound) + 2.0 ** -22 * ref.abs()
    bound = bound + torch.where(g < -87.3, (g.abs() + 2) * 2.0 ** -149 * u.abs(), 0.0)
    close(h, ref, bound)
    far = (g < -88) & (g > -102) & (u != 0)
    assert int(far.sum()) > 0 and bool((h[far] != 0).all())


# Sizes that the 128-token tiles take, whole and with a reduction split over clusters (a test that
# uses them holds the scratch to it, so that another rule does not move it elsewhere).
TILED = [(1100, 3088, 600), (300, 8192, 1000)]


def tiled_gemm(moe, xq, xs, wq, ws, **kw):
    scratch = tiled_scratch(moe, *xq.shape)
    out = moe.moe_gemm_i8(xq, xs, wq, ws, workspace=scratch, **kw)
    assert not bool((scratch == 0xA5).all())
    return out


def tiled_gate_up(moe, xq, xs, gq, gs, uq, us, **kw):
    scratch = tiled_scratch(moe, *xq.shape)
    out = moe.moe_gate_up_i8(xq, xs, gq, gs, uq, us, workspace=scratch, **kw)
    assert not bool((scratch == 0xA5).all())
    return out


@pytest.mark.parametrize("T,K,N", [(2200, 1024, 1030), (300, 8192, 1000), (107, 16384, 899)])
def test_tiled_largest_codes_add_up_exactly(moe, T, K, N):
    """Rows of -128 and 127 in 1024 columns spread over K, zeros in the others: the largest
    sums that are exact, 2^24 itself among them."""
    xq, wq = torch.zeros(T, K, dtype=torch.int8, device=DEV), torch.zeros(N, K, dtype=torch.int8, device=DEV)
    at = torch.arange(0, K, K // 1024, device=DEV)
    a, b = xq[:, at], wq[:, at]
    a[:], b[:] = -128, -128
    a[1::3], b[1::3] = 127, 127
    a[2::3, ::2], b[2::3, 1::3] = 127, 1
    xq[:, at], wq[:, at] = a, b
    one = lambda n: torch.ones(n, device=DEV)
    out = tiled_gemm(moe, xq, one(T), wq, one(N), out_dtype=torch.float32)
    assert torch.equal(out.double(), xq.double() @ wq.double().T)


@pytest.mark.parametrize("T,K,N", [(2, 16384, 140), (40, 16384, 140), (3, 32768, 1000), (300, 4096, 64), (107, 16384, 899), (2100, 16384, 640)])
def test_long_reductions_that_cancel_add_up_exactly(moe, T, K, N):
    """Magnitudes whose sum passes 2^24 many times, products that cancel in pairs of columns but
    for a few: every partial sum, of any 16 columns and of any share of the reduction, is a whole
    number below 2^24, so the result is exact, and a column that is lost or read twice
    shows.  In the CUDA-core, the few-rows and the tiled kernel, whole and split."""
    xq = torch.randint(-127, 128, (T, K), generator=gen(1), device=DEV).to(torch.int8)
    wq = torch.randint(100, 128, (N, K), generator=gen(2), device=DEV).to(torch.int8)
    xq[:, 1::2], wq[:, 1::2] = -xq[:, ::2], wq[:, ::2]
    odd = torch.randint(0, K // 2, (K // 64,), generator=gen(3), device=DEV).unique() * 2 + 1
    wq[:, odd] -= torch.randint(1, 90, (N, len(odd)), generator=gen(4), device=DEV).to(torch.int8)
    exact = xq.double() @ wq.double().T
    assert float((xq.double().abs() @ wq.double().abs().T).max()) > 2 ** 24 and float(exact.abs().max()) < 2 ** 23
    one = lambda n: torch.ones(n, device=DEV)
    out = moe.moe_gemm_i8(xq, one(T), wq, one(N), out_dtype=torch.float32)
    assert bool((exact != 0).any()) and torch.equal(out.double(), exact)


@pytest.mark.parametrize("T,K,N", TILED)
def test_tiled_scales_of_every_kind(moe, T, K, N):
    (xq, xs), (wq, ws) = codes(T, K), codes(N, K, seed=1)
    xs, ws = xs.clone(), ws.clone()
    inf, nan = float("inf"), float("nan")
    for at in (0, T - 4):
        xs[at:at + 4] = torch.tensor([0.0, nan, 1e30, inf], device=DEV)
    for at in (0, N - 6):
        ws[at:at + 6] = torch.tensor([0.0, nan, 1e-30, 2.0 ** -126, inf, -1.0], device=DEV)
    for odt in (torch.float32, torch.bfloat16):
        out = tiled_gemm(moe, xq, xs, wq, ws, out_dtype=odt)
        # in the call's order: the sum times the token's scale, times the channel's
        y = (xq.double() @ wq.double().T).float() * xs[:, None] * ws[None, :]
        plain = y.isfinite()
        assert torch.equal(out.isnan(), y.isnan()) and torch.equal(out[~plain & ~y.isnan()].float(), y[~plain & ~y.isnan()])
        ref, bound = product_ref(xq, wq, xs, ws)
        close(torch.where(plain, out, 0.0), torch.where(plain, ref, 0.0), torch.where(plain, bound, 0.0))
        h = tiled_gate_up(moe, xq, xs, wq, ws, wq, ws, h_dtype=odt)
        assert bool(h[1].isnan().all()) and bool(h[:, 1].isnan().all()) and bool(h[T - 3].isnan().all())
        assert not h[0, 2:4].any() and not h[T - 4, 2:4].any()


@pytest.mark.parametrize("odt", ["f32", "bf16"])
@pytest.mark.parametrize("T,K,N", TILED)
def test_tiled_gate_sums_from_minus_200_to_200(moe, odt, T, K, N):
    (xq, _), (gq, _), (uq, us) = codes(T, K), codes(N, K, seed=1), codes(N, K, seed=2)
    sums = xq.double() @ gq.double().T
    xs = (torch.rand(T, generator=gen(4), device=DEV) * 200 / sums.abs().amax(1)).float()
    gs = torch.ones(N, device=DEV)
    h = tiled_gate_up(moe, xq, xs, gq, gs, uq, us, h_dtype=DT[odt])
    g, u = product_ref(xq, gq, xs, gs), product_ref(xq, uq, xs, us)
    assert float(g[0].max()) > 100 and float(g[0].min()) < -100
    close(h, *swiglu_ref(*g, *u, odt == "f32"))


def ragged_call(moe, gate_up, xq, xs, mats, off, tok=None, out=None, tiled=False):
    rows = len(tok) if tok is not None else xq.shape[0]
    scratch = tiled_scratch(moe, rows, xq.shape[1]) if tiled else None
    if gate_up:
        (wq, ws), (uq, us) = mats
        out = moe.moe_gate_up_i8(xq, xs, wq, ws, uq, us, offsets=off, perm_tok=tok, h=out, workspace=scratch)
    else:
        out = moe.moe_grouped_gemm_i8(xq, xs, *mats[0], off, perm_tok=tok, out=out, workspace=scratch)
    assert not tiled or not bool((scratch == 0xA5).all())
    return out


RAGGED = [(2, 144, 72, False), (6, 144, 72, False), (70, 144, 72, False), (400, 144, 72, False), (1500, 2064, 777, True), (410, 8192, 320, True)]


@pytest.mark.parametrize("gate_up", [False, True])
@pytest.mark.parametrize("rows,K,N,tiled", RAGGED)
def test_offsets_of_every_kind(moe, rows, K, N, tiled, gate_up):
    """Groups in every kernel (CUDA cores, few rows, tiles whole and split): empty ones, one with
    everything, a padded batch's rows behind them as they were; offsets out of range count as
    the nearest row; a group that ends before it begins is empty, and rows that one group
    alone holds are right where others overlap; bad token indices spoil their own row only."""
    E, half = 5, rows // 2
    (xq, xs), (wq, ws), (uq, us) = codes(rows, K), codes(E, N, K, seed=1), codes(E, N, K, seed=2)
    mats = [(wq, ws), (uq, us)] if gate_up else [(wq, ws)]
    third = rows // 3
    cuts = [[0, 0, rows, rows, rows, rows], [0, 1, 1, 1, half, half], [0, half, half, half, half, rows],
            [-5, 1, 1, half, half, 10 ** 9], [-2 ** 31, 0, third, third, 2 ** 31 - 1, 2 ** 31 - 1]]
    for cut in cuts:
        off = torch.tensor(cut, dtype=torch.int32, device=DEV)
        out = torch.full((rows, N), 7.0, device=DEV, dtype=torch.bfloat16)
        ragged_call(moe, gate_up, xq, xs, mats, off, out=out, tiled=tiled)
        kept = off.clamp(0, rows)
        check_grouped(out, xq, xs, mats, kept, None)
        assert bool((out[int(kept[-1]):] == 7).all())
    # 0 .. 2/3, none, 1/3 .. all, none, none: the first and the last third are one group's alone
    off = torch.tensor([0, 2 * third, third, rows, rows, rows], dtype=torch.int32, device=DEV)
    out = ragged_call(moe, gate_up, xq, xs, mats, off, tiled=tiled)
    alone = torch.tensor([0, third, third, third, third, third], dtype=torch.int32)
    if third:
        check_grouped(out, xq, xs, mats, alone, None)
        check_grouped(out[2 * third:], xq[2 * third:], xs[2 * third:], mats,
                      torch.tensor([0, 0, 0, rows - 2 * third, rows - 2 * third, rows - 2 * third]), None)
    tok = torch.arange(rows, device=DEV).int().flip(0).contiguous()
    bad = tok.clone()
    at = sorted({1, rows // 2, rows - 1})
    bad[at] = torch.tensor([-7, rows, 2 ** 31 - 1], dtype=torch.int32, device=DEV)[:len(at)]
    off = torch.tensor([0, 1, half, half, rows, rows], dtype=torch.int32, device=DEV)
    a, b = (ragged_call(moe, gate_up, xq, xs, mats, off, tok=t, tiled=tiled) for t in (tok, bad))
    keep = torch.ones(rows, dtype=torch.bool, device=DEV)
    keep[at] = False
    check_grouped(a, xq, xs, mats, off, tok)
    assert torch.equal(a[keep], b[keep])


@pytest.mark.parametrize("gate_up", [False, True])
@pytest.mark.parametrize("T,K,N", TILED)
def test_one_workspace_by_calls_in_order(moe, T, K, N, gate_up):
    """Calls on other tokens that hold the same workspace, back to back on a stream and in one
    graph: the next call's fp16 rows are written when the product before has read its own."""
    sets = [codes(T, K, seed=20 + i) for i in range(4)]
    (wq, ws), (uq, us) = codes(N, K, seed=1), codes(N, K, seed=2)
    scratch = tiled_scratch(moe, T, K)
    outs = [torch.empty(T, N, device=DEV) for _ in range(12)]
    want = []
    for xq, xs in sets:
        y = product_ref(xq, wq, xs, ws)
        want.append(swiglu_ref(*y, *product_ref(xq, uq, xs, us), True) if gate_up else y)

    def chain():
        for i, out in enumerate(outs):
            xq, xs = sets[i % 4]
            if gate_up:
                moe.moe_gate_up_i8(xq, xs, wq, ws, uq, us, h=out, workspace=scratch)
            else:
                moe.moe_gemm_i8(xq, xs, wq, ws, out=out, workspace=scratch)
    chain()
    assert not bool((scratch == 0xA5).all())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    for run in (chain, graph.replay, graph.replay):
        for out in outs:
            out.zero_()
        run()
        for i, out in enumerate(outs):
            close(out, *want[i % 4])


@pytest.mark.parametrize("gate_up", [False, True])
@pytest.mark.parametrize("T,K,N", [(2, 512, 200), (40, 512, 200), (40, 512, 201), (1100, 3088, 600), (1100, 3088, 601)])
def test_rows_past_32_bits(moe, T, K, N, gate_up):
    """Token rows whose codes, and output rows whose elements, lie past 2^31, in the CUDA-core, the
    few-rows and the tiled kernel, stored in 16-byte pieces and element by element."""
    apart = (2 ** 31 // (T - 1) + 64) // 16 * 16
    xq, xs = codes(T, K)
    far = torch.zeros((T - 1) * apart + K, dtype=torch.int8, device=DEV).as_strided((T, K), (apart, 1))
    far.copy_(xq)
    (wq, ws), (uq, us) = codes(N, K, seed=1), codes(N, K, seed=2)
    out = torch.zeros((T - 1) * apart + N, dtype=torch.bfloat16, device=DEV).as_strided((T, N), (apart, 1))
    assert (T - 1) * apart > 2 ** 31
    y = product_ref(xq, wq, xs, ws)
    if gate_up:
        moe.moe_gate_up_i8(far, xs, wq, ws, uq, us, h=out)
        y = swiglu_ref(*y, *product_ref(xq, uq, xs, us), False)
    else:
        moe.moe_gemm_i8(far, xs, wq, ws, out=out)
    close(out.contiguous(), *y)


@pytest.mark.parametrize("T,K,N", [(2, 16384, 140), (40, 16384, 140), (64, 4096, 4096), (300, 16384, 140), (107, 16384, 899),
                                   (2100, 16384, 640), (2100, 4096, 640)])
def test_sums_beyond_2_to_24(moe, T, K, N):
    """Large codes of one sign, the worst for sums that are cut off.  On the CUDA cores the sum is
    a whole number, rounded once.  On the tensor cores each of the K / 16 steps may cut a unit
    in the last place off the sum so far, at most 2^-23 of A, and a split reduction's up
    to 7 additions round once each."""
    xq = torch.randint(100, 128, (T, K), generator=gen(1), device=DEV).to(torch.int8)
    wq = torch.randint(100, 128, (N, K), generator=gen(2), device=DEV).to(torch.int8)
    one = lambda n: torch.ones(n, device=DEV)
    out = moe.moe_gemm_i8(xq, one(T), wq, one(N), out_dtype=torch.float32)
    exact = xq.double() @ wq.double().T
    assert float(exact.min()) > 2 ** 24
    if T <= 2:
        assert torch.equal(out, exact.float())
    assert bool(((out.double() - exact).abs() <= (K / 16 + 7) * 2.0 ** -23 * exact).all())
