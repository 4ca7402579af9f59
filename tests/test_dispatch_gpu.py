"""Dispatch, combine and their backward passes against their definitions in 64 bits.

Tolerances, derived before the first run:
  dispatch   bit for bit.
  its gradient, combine   k terms added in fp32 (combine: fused multiply-adds): each
             step is off by at most 2^-24 of the running sum of magnitudes M, so
             k 2^-24 M (1 + k 2^-24); the output's rounding adds finfo.eps / 2 of the
             value (bf16 2^-8; fp32 has had its own).
  dy         one fp32 product, 2^-24, and the rounding to y's type.
  dw         d fused multiply-adds in some order: d 2^-24 M at most.
  Results below the smallest normal number may lose 2^-149 (fp32) or 2^-133 (bf16) more.
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


def rand(*shape, seed=0, sd=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed + 1000 * len(shape) + sum(shape))
    return torch.randn(*shape, generator=g, device=DEV) * sd


def perm(n, seed=0):
    return torch.randperm(n, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV).int()


def rounding(t):
    return torch.finfo(t).eps / 2 if t != torch.float32 else 0.0


def close(got, ref, bound):
    """|got - ref| <= bound + the output's rounding."""
    least = 2.0 ** -149 if got.dtype == torch.float32 else 2.0 ** -133
    tol = bound + rounding(got.dtype) * (ref.abs() + bound) + least
    worst = ((got.double() - ref).abs() - tol).max() if ref.numel() else torch.tensor(0.0)
    assert not worst > 0 and not got.isnan().any(), f"off by {float(worst):.3e} more than the bound"


def slots(inv, T, k, rows):
    at = inv.view(T, k).long()
    return at, (at >= 0) & (at < rows)


def gather_ref(y, inv, T, k, w=None):
    """(sum over the slots, sum of magnitudes) in 64 bits."""
    at, ok = slots(inv, T, k, y.shape[0])
    s = torch.zeros(T, y.shape[1], dtype=torch.float64, device=DEV)
    m = torch.zeros_like(s)
    for j in range(k):
        hit = ok[:, j].nonzero()[:, 0]
        term = y[at[hit, j]].double() * (w[hit, j:j + 1].double() if w is not None else 1.0)
        s[hit] += term
        m[hit] += term.abs()
    return s, m


def check_combine(got, y, w, inv, T, k):
    ref, m = gather_ref(y, inv, T, k, w)
    close(got, ref, k * 2.0 ** -24 * m * (1 + 1e-6))


def check_combine_backward(dy, dw, g, y, w, inv, before=None):
    """`before`: what dy held (rows that no slot names keep it)."""
    T, k = w.shape
    d = y.shape[1]
    at, ok = slots(inv, T, k, y.shape[0])
    ref = torch.zeros(y.shape, dtype=torch.float64, device=DEV)
    named = torch.zeros(y.shape[0], dtype=torch.bool, device=DEV)
    ref_w = torch.zeros(T, k, dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(ref_w)
    for j in range(k):
        hit = ok[:, j].nonzero()[:, 0]
        rows = at[hit, j]
        ref[rows] = w[hit, j:j + 1].double() * g[hit].double()
        named[rows] = True
        prod = g[hit].double() * y[rows].double()
        ref_w[hit, j], mag[hit, j] = prod.sum(1), prod.abs().sum(1)
    if dy is not None:
        close(dy[named], ref[named], 2.0 ** -24 * ref[named].abs())
        if before is not None:
            assert torch.equal(dy[~named], before[~named])
    if dw is not None:
        assert dw.dtype == torch.float32
        close(dw, ref_w, d * 2.0 ** -24 * mag * (1 + 1e-3))


SIZES = [(1, 1, 1), (1, 8, 16), (3, 2, 7), (5, 3, 4112), (37, 2, 1024), (128, 2, 1024), (999, 3, 1001), (257, 8, 130), (2, 4, 16392),
         (4000, 1, 72), (2500, 5, 264)]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,k,d", SIZES)
def test_dispatch_and_its_gradient(moe, dt, T, k, d):
    x, inv = rand(T, d).to(DT[dt]), perm(T * k)
    out = moe.moe_dispatch(x, inv, k)
    want = torch.empty_like(out)
    want[inv.long()] = x.repeat_interleave(k, 0)
    assert out.dtype == x.dtype and torch.equal(out, want)
    g = rand(T * k, d, seed=1).to(DT[dt])
    dx = moe.moe_dispatch_backward(g, inv, k)
    assert dx.dtype == g.dtype and dx.shape == (T, d)
    ref, m = gather_ref(g, inv, T, k)
    close(dx, ref, k * 2.0 ** -24 * m * (1 + 1e-6))


@pytest.mark.parametrize("dt,odt", [("f32", "f32"), ("f32", "bf16"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("T,k,d", SIZES)
def test_combine_and_its_gradients(moe, dt, odt, T, k, d):
    y, inv = rand(T * k, d).to(DT[dt]), perm(T * k)
    w = torch.softmax(rand(T, k), 1)
    out = moe.moe_combine(y, w, inv, out_dtype=DT[odt])
    assert out.dtype == DT[odt] and out.shape == (T, d)
    check_combine(out, y, w, inv, T, k)
    g = rand(T, d, seed=1).to(DT[odt])
    dy, dw = moe.moe_combine_backward(g, y, w, inv)
    assert dy.dtype == y.dtype and dy.shape == y.shape and dw.shape == w.shape
    check_combine_backward(dy, dw, g, y, w, inv)
    only = moe.moe_combine_backward(g, y, w, inv, want_dw=False)
    assert only[1] is None and torch.equal(only[0], dy)
    only = moe.moe_combine_backward(g, y, w, inv, want_dy=False)
    assert only[0] is None and torch.equal(only[1], dw)


@pytest.mark.parametrize("d", [5, 256])
def test_slots_without_rows(moe, d):
    """Dropped slots (indices out of range on either side), rows that no slot names
    (a padded batch), NaN and infinities in those rows and in the dropped slots' weights."""
    T, k, rows = 50, 4, 230
    inv = perm(rows)[:T * k].clone()
    inv[::7] = torch.tensor([-1, rows, 2 ** 31 - 1, -2 ** 31, -5, rows + 1, 10 ** 9] * 5, device=DEV, dtype=torch.int32)[:len(inv[::7])]
    inv[:k] = -1                                    # a token without any row
    at, ok = slots(inv, T, k, rows)
    named = torch.zeros(rows, dtype=torch.bool, device=DEV)
    named[at[ok]] = True
    y = rand(rows, d)
    y[~named] = float("nan")
    y[(~named).nonzero()[0]] = float("inf")
    w = torch.softmax(rand(T, k), 1)
    w[~ok] = float("nan")
    out = moe.moe_combine(y, w, inv)
    check_combine(out, y, w, inv, T, k)
    assert not out[0].any()
    g = rand(T, d, seed=2)
    before = rand(rows, d, seed=3)
    dy = before.clone()
    got = moe.moe_combine_backward(g, y, w, inv, dy=dy)
    assert got[0] is dy
    check_combine_backward(dy, got[1], g, y, w, inv, before)
    assert not got[1][~ok].any()
    x = rand(T, d, seed=4)
    sent = before.clone()
    moe.moe_dispatch(x, inv, k, out=sent)
    assert torch.equal(sent[~named], before[~named])
    want = before.clone()
    want[at[ok]] = x[ok.nonzero()[:, 0]]
    assert torch.equal(sent, want)
    dx = moe.moe_dispatch_backward(y, inv, k)
    ref, m = gather_ref(y, inv, T, k)
    close(dx, ref, k * 2.0 ** -24 * m * (1 + 1e-6))
    # no grouped rows at all
    assert not moe.moe_combine(y[:0], w, inv).any()
    assert not moe.moe_dispatch_backward(y[:0], inv, k).any()
    assert moe.moe_dispatch(x, inv, k, out=sent[:0]).shape == (0, d)


def test_a_row_read_twice(moe):
    """Where rows are only read, two slots may name the same one."""
    T, k, d = 20, 2, 64
    y, w = rand(7, d), rand(T, k)
    inv = torch.randint(0, 7, (T * k,), device=DEV).int()
    inv[:2] = 3
    check_combine(moe.moe_combine(y, w, inv), y, w, inv, T, k)
    dw = moe.moe_combine_backward(rand(T, d, seed=1), y, w, inv, want_dy=False)[1]
    check_combine_backward(None, dw, rand(T, d, seed=1), y, w, inv)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("off,d,wide", [(0, 64, 80), (8, 64, 96), (1, 64, 97), (3, 61, 70), (4, 64, 76)])
def test_strides_and_alignments(moe, dt, off, d, wide):
    """Column slices: rows further apart than their length, on any boundary of the type;
    what lies beside the outputs stays."""
    T, k = 33, 3
    t = DT[dt]
    cut = lambda m: m[:, off:off + d]
    inv, w = perm(T * k), torch.softmax(rand(T, k), 1)
    y, x = cut(rand(T * k, wide).to(t)), cut(rand(T, wide, seed=5).to(t))
    base = torch.full((T * k, wide), 7.0, device=DEV, dtype=t)

    def beside(m):
        return torch.cat([m[:, :off], m[:, off + d:]], 1)
    o = base[:T].clone()
    moe.moe_combine(y, w, inv, out=cut(o))
    check_combine(cut(o), y, w, inv, T, k)
    assert bool((beside(o) == 7).all())
    o = base.clone()
    dw = moe.moe_combine_backward(x, y, w, inv, dy=cut(o))[1]
    check_combine_backward(cut(o), dw, x, y, w, inv)
    assert bool((beside(o) == 7).all())
    o = base.clone()
    moe.moe_dispatch(x, inv, k, out=cut(o))
    assert torch.equal(cut(o)[inv.long()], x.repeat_interleave(k, 0)) and bool((beside(o) == 7).all())
    o = base[:T].clone()
    moe.moe_dispatch_backward(y, inv, k, out=cut(o))
    ref, m = gather_ref(y, inv, T, k)
    close(cut(o), ref, k * 2.0 ** -24 * m * (1 + 1e-6))
    assert bool((beside(o) == 7).all())


def test_no_tokens(moe):
    x, inv = rand(0, 16), torch.zeros(0, dtype=torch.int32, device=DEV)
    w = torch.zeros(0, 2, device=DEV)
    assert moe.moe_dispatch(x, inv, 2).shape == (0, 16)
    assert moe.moe_dispatch_backward(x, inv, 2).shape == (0, 16)
    assert moe.moe_combine(x, w, inv).shape == (0, 16)
    keep = rand(3, 16)
    dy, dw = moe.moe_combine_backward(x, keep, w, inv, dy=keep.clone())
    assert torch.equal(dy, keep) and dw.shape == (0, 2)


@pytest.mark.parametrize("value", [float("inf"), float("nan"), 3e38, 1e-42])
def test_special_values(moe, value):
    """They reach their own token's output and gradients, and no other's."""
    T, k, d = 12, 2, 40
    y, w, inv = rand(T * k, d), torch.full((T, k), 0.5, device=DEV), perm(T * k)
    clean = moe.moe_combine(y, w, inv)
    hit = int(inv[2 * k])                         # token 2's first row
    y2 = y.clone()
    y2[hit, 3] = value
    out = moe.moe_combine(y2, w, inv)
    want = y2[hit, 3] * 0.5 + y2[int(inv[2 * k + 1]), 3] * 0.5
    assert bool((out[2, 3] == want) | (out[2, 3].isnan() & want.isnan()))
    out[2, 3] = clean[2, 3]
    assert torch.equal(out, clean)
    g = torch.ones(T, d, device=DEV)
    dw = moe.moe_combine_backward(g, y2, w, inv)[1]
    base = moe.moe_combine_backward(g, y, w, inv)[1]
    same = torch.ones(T, k, dtype=torch.bool, device=DEV)
    same[2, 0] = False
    assert torch.equal(dw[same], base[same])
    want = y2[hit].double().sum().float()
    assert bool(dw[2, 0].isnan() == want.isnan()) and bool(dw[2, 0].isinf() == want.isinf())


class Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, moe, x, inv, k):
        ctx.moe, ctx.k = moe, k
        ctx.save_for_backward(inv)
        return moe.moe_dispatch(x, inv, k)

    @staticmethod
    def backward(ctx, g):
        return None, ctx.moe.moe_dispatch_backward(g.contiguous(), ctx.saved_tensors[0], ctx.k), None, None


class Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, moe, y, w, inv):
        ctx.moe = moe
        ctx.save_for_backward(y, w, inv)
        return moe.moe_combine(y, w, inv)

    @staticmethod
    def backward(ctx, g):
        y, w, inv = ctx.saved_tensors
        return None, *ctx.moe.moe_combine_backward(g.contiguous(), y, w, inv), None


def test_an_expert_layer_trains_through_them(moe):
    """route -> permute -> dispatch -> the experts' own products -> combine in fp32: the
    gradients against autograd in 64 bits.  Every step is a product or sum of fp32; the
    chain is 2 products of up to 48 terms and their backward: 1e-4 of the largest value
    covers 48 * 4 * 2^-24 = 1.1e-5 of the magnitudes' sums several times."""
    T, d, E, k, F = 64, 48, 4, 2, 40
    x, wr = rand(T, d), rand(E, d, sd=d ** -0.5)
    idx, w = moe.moe_route(x, wr, None, k)
    _, offsets, perm_tok, inv = moe.moe_permute(idx, E)
    up, down = rand(E, F, d, sd=d ** -0.5), rand(E, d, F, sd=F ** -0.5)
    g = rand(T, d, seed=9)

    def grads(dtype, dispatch, combine):
        p = [t.to(dtype).clone().requires_grad_() for t in (x, w, up, down)]
        rows, off = dispatch(p[0]), offsets.tolist()
        y = torch.cat([torch.relu(rows[off[e]:off[e + 1]] @ p[2][e].T) @ p[3][e].T for e in range(E)])
        combine(y, p[1]).backward(g.to(dtype))
        return [t.grad.double() for t in p]
    at = inv.view(T, k).long()
    want = grads(torch.float64, lambda t: t[perm_tok.long()], lambda y, ww: (ww[..., None] * y[at]).sum(1))
    got = grads(torch.float32, lambda t: Dispatch.apply(moe, t, inv, k), lambda y, ww: Combine.apply(moe, y, ww, inv))
    for a, b in zip(got, want):
        assert float((a - b).abs().max()) <= 1e-4 * float(b.abs().max())


def test_gradients_against_differences(moe):
    """combine is linear in y and in w: a step of 2 in one direction changes <g, out> by
    exactly twice the gradient's product with it.  Both sides are sums of fp32 results, each
    within its bound above."""
    T, k, d = 9, 3, 30
    y, w, inv, g = rand(T * k, d), rand(T, k), perm(T * k), rand(T, d, seed=1)
    dy, dw = moe.moe_combine_backward(g, y, w, inv)
    f = lambda a, b: float((g.double() * moe.moe_combine(a, b, inv).double()).sum())
    ey, ew = rand(T * k, d, seed=2), rand(T, k, seed=3)
    size = float((g.abs().double().sum(1) * (w.abs() + ew.abs()).double().sum(1)).sum() * (y.abs().max() + ey.abs().max()))
    tol = (d + 8) * 2.0 ** -24 * 4 * size
    assert abs(f(y + ey, w) - f(y - ey, w) - 2 * float((dy.double() * ey.double()).sum())) <= tol
    assert abs(f(y, w + ew) - f(y, w - ew) - 2 * float((dw.double() * ew.double()).sum())) <= tol
    x, e = rand(T, d, seed=4), rand(T, d, seed=5)
    gg = rand(T * k, d, seed=6)
    dx = moe.moe_dispatch_backward(gg, inv, k)
    h = lambda a: float((gg.double() * moe.moe_dispatch(a, inv, k).double()).sum())
    size = float(gg.abs().double().sum() * (x.abs().max() + e.abs().max()))
    assert abs(h(x + e) - h(x - e) - 2 * float((dx.double() * e.double()).sum())) <= (k + 4) * 2.0 ** -24 * 4 * size


def test_rows_beyond_32_bits(moe):
    """Grouped rows whose elements lie past 2^31."""
    d, rows = 1032, 2 ** 21 + 9                    # 2.16e9 elements of bf16
    y = torch.zeros(rows, d, device=DEV, dtype=torch.bfloat16)
    T, k = 3, 2
    inv = torch.tensor([rows - 1, 5, rows - 2, rows - 9, 0, 2 ** 21 - 1], dtype=torch.int32, device=DEV)
    x = rand(T, d).bfloat16()
    moe.moe_dispatch(x, inv, k, out=y)
    assert torch.equal(y[inv.long()], x.repeat_interleave(k, 0))
    assert int((y != 0).any(1).sum()) == T * k
    w = torch.softmax(rand(T, k), 1)
    check_combine(moe.moe_combine(y, w, inv), y, w, inv, T, k)
    dw = moe.moe_combine_backward(x, y, w, inv, want_dy=False)[1]
    check_combine_backward(None, dw, x, y, w, inv)


def test_streams_and_graphs(moe):
    """A side stream, and a captured chain replayed on other inputs; run to run the same bits."""
    T, k, d = 200, 2, 512
    x, y, w, inv, g = rand(T, d), rand(T * k, d), torch.softmax(rand(T, k), 1), perm(T * k), rand(T, d, seed=1)

    def chain():
        return (moe.moe_dispatch(x, inv, k), moe.moe_combine(y, w, inv), moe.moe_dispatch_backward(y, inv, k),
                *moe.moe_combine_backward(g, y, w, inv))
    first = chain()
    assert all(torch.equal(a, b) for a, b in zip(first, chain()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        there = chain()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(first, there))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = chain()
    for seed in (11, 12):
        for t in (x, y, g):
            t.copy_(rand(*t.shape, seed=seed))
        inv.copy_(perm(T * k, seed=seed))
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(held, chain()))


def test_device_refusals(moe):
    x, inv = rand(4, 16), perm(8)
    with pytest.raises(ValueError):
        moe.moe_dispatch(x, inv.cpu(), 2)
    with pytest.raises(ValueError):
        moe.moe_combine(rand(8, 16), torch.ones(4, 2), inv)
    with pytest.raises(moe.MoeError):
        moe.moe_dispatch(rand(1, 16), perm(9), 9)


@pytest.mark.parametrize("dt,odt", [("f32", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("T,k,d", [(1601, 2, 1000), (1600, 3, 1003), (1555, 1, 8200), (1530, 1, 8197), (304, 2, 2312), (305, 2, 2309),
                                   (300, 8, 520), (16, 2, 513)])
def test_combine_by_threads_of_a_token(moe, dt, odt, T, k, d):
    """Many and few tokens, narrow and wide: one warp, two, four or sixteen to a token."""
    test_combine_and_its_gradients(moe, dt, odt, T, k, d)


def poisoned(moe, call):
    """`call`'s new outputs out of memory that held NaN: blocks of every size it allocates are
    filled and given back first."""
    shapes = [t.shape for t in call() if t is not None]
    dtypes = [t.dtype for t in call() if t is not None]
    for _ in range(2):
        held = [torch.full(s, float("nan"), dtype=t, device=DEV) for s, t in zip(shapes, dtypes) for _ in range(3)]
        del held
    return call()


def padded_slots(T, k, rows, drop, seed=0):
    """inv of T*k slots over `rows` rows, some of them dropped, and which rows are named."""
    inv = perm(max(rows, T * k), seed=seed)[:T * k].clone()      # (beyond rows: dropped, where rows < T*k)
    if drop:
        values = torch.tensor([-1, rows, 2 ** 31 - 1, -2 ** 31, -5, rows + 1], dtype=torch.int32, device=DEV)
        at = torch.arange(0, T * k, drop, device=DEV)
        inv[at] = values[torch.arange(len(at), device=DEV) % 6]
    named = torch.zeros(rows, dtype=torch.bool, device=DEV)
    named[inv[(inv >= 0) & (inv < rows)].long()] = True
    return inv, named


FILL = [(1, 1, 5, 1, 0), (0, 2, 40, 16, 0), (7, 3, 21, 33, 2), (50, 4, 230, 5, 7), (600, 2, 1200, 264, 5), (600, 2, 70000, 24, 5),
        (1700, 2, 3400, 520, 9), (1700, 8, 13600, 48, 1), (1700, 3, 5000, 1001, 11), (40, 2, 80, 4100, 3), (5000, 8, 41000, 3, 4),
        (300, 2, 500, 64, 0)]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,k,rows,d,drop", FILL)
def test_rows_without_slots_are_zeros_in_new_outputs(moe, dt, T, k, rows, d, drop):
    """Padded batches and dropped slots: a new output's other rows hold zeros, whatever the
    memory held; the named ones are the same bits as in an output that is given."""
    inv, named = padded_slots(T, k, rows, drop)
    y, w, g = rand(rows, d).to(DT[dt]), rand(T, k), rand(T, d, seed=1).to(DT[dt])
    dy, dw = poisoned(moe, lambda: moe.moe_combine_backward(g, y, w, inv))
    given = torch.full_like(y, 7.0)
    dw2 = moe.moe_combine_backward(g, y, w, inv, dy=given)[1]
    assert torch.equal(dy[named], given[named]) and torch.equal(dw, dw2)
    assert not dy[~named].any() and bool((given[~named] == 7).all())
    check_combine_backward(dy, dw, g, y, w, inv)
    if rows <= T * k:                                      # a dispatch's own rows: T*k
        inv, named = padded_slots(T, k, T * k, drop)
        sent, = poisoned(moe, lambda: (moe.moe_dispatch(g, inv, k),))
        given = torch.full_like(sent, 7.0)
        moe.moe_dispatch(g, inv, k, out=given)
        assert torch.equal(sent[named], given[named]) and not sent[~named].any() and bool((given[~named] == 7).all())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("off,d,wide", [(0, 64, 80), (1, 61, 97), (3, 5, 70), (4, 64, 76)])
def test_filled_rows_apart(moe, dt, off, d, wide):
    """The C calls' filled forms into column slices: zeros inside them only; inv off 16-byte
    boundaries; replayed from a graph on other slots."""
    import ctypes
    L, t = moe.load_library(), DT[dt]
    T, k, rows = 200, 3, 700
    both = torch.zeros(T * k + 3, dtype=torch.int32, device=DEV)
    inv = both[off % 4:off % 4 + T * k]
    base = torch.full((rows, wide), 7.0, device=DEV, dtype=t)
    out, x = base[:, off:off + d], rand(T, d).to(t)
    w, y, dw = rand(T, k), rand(rows, d, seed=2).to(t), torch.empty(T, k, device=DEV)
    p = lambda v: ctypes.c_void_p(v.data_ptr())
    stream = lambda: ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    e = 0 if dt == "f32" else 1

    def sent():
        assert L.moe_dispatch_filled(p(x), e, T, d, d, p(inv), k, p(out), rows, wide, stream()) == 0

    def back():
        assert L.moe_combine_backward_filled(p(x), e, T, d, d, p(y), e, rows, d, p(w), p(inv), k, p(out), wide, p(dw), stream()) == 0
    inv.copy_(padded_slots(T, k, rows, 5)[0])
    sent(), back()
    graphs = []
    for call in (sent, back):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call()
    for seed, drop in ((1, 0), (2, 4), (3, 1)):
        new, named = padded_slots(T, k, rows, drop, seed=seed)
        inv.copy_(new)
        slot = ((new >= 0) & (new < rows)).nonzero()[:, 0]
        for i, graph in enumerate(graphs):
            base.fill_(7.0)
            graph.replay()
            assert not out[~named].any() and bool((base[:, :off] == 7).all()) and bool((base[:, off + d:] == 7).all())
            if i == 0:
                assert torch.equal(out[new[slot].long()], x[slot // k])
            else:
                check_combine_backward(out, dw, x, y, w, new)


def test_filled_beyond_the_marked_slots(moe):
    """More slots than are marked bit by bit (2^21): every row is zeroed ahead."""
    T, k, d = 300_000, 8, 3
    rows = T * k
    inv, named = padded_slots(T, k, rows, 3)
    x = rand(T, d).bfloat16()
    sent, = poisoned(moe, lambda: (moe.moe_dispatch(x, inv, k),))
    slot = ((inv >= 0) & (inv < rows)).nonzero()[:, 0]
    assert torch.equal(sent[inv[slot].long()], x[slot // k]) and not sent[~named].any()
    y, w = rand(rows, d).bfloat16(), rand(T, k)
    dy, dw = poisoned(moe, lambda: moe.moe_combine_backward(x, y, w, inv))
    assert not dy[~named].any()
    check_combine_backward(dy, dw, x, y, w, inv)


def test_calls_are_recorded(moe):
    """Inputs that require grad: the outputs carry their graph, and the gradients are the backward
    calls' own bits (bf16 and fp32, a padded batch, dropped slots, one input alone, a gradient
    that is one value seen everywhere, one whose rows lie apart)."""
    T, k, d, rows = 60, 3, 40, 200
    for dt, odt in ((torch.float32, torch.float32), (torch.bfloat16, torch.float32), (torch.bfloat16, torch.bfloat16)):
        inv, named = padded_slots(T, k, rows, 7)
        y, w = rand(rows, d).to(dt).requires_grad_(), rand(T, k).requires_grad_()
        g = rand(T, d, seed=3).to(odt)
        out = moe.moe_combine(y, w, inv, out_dtype=odt)
        assert out.requires_grad and torch.equal(out, moe.moe_combine(y.detach(), w.detach(), inv, out_dtype=odt))
        out.backward(g)
        dy, dw = moe.moe_combine_backward(g, y.detach(), w.detach(), inv)
        assert torch.equal(y.grad, dy) and torch.equal(w.grad, dw) and not y.grad[~named].any()
        for a, b, want in ((y, w.detach(), dy), (y.detach(), w, dw)):
            got, = torch.autograd.grad(moe.moe_combine(a, b, inv, out_dtype=odt), a if a.requires_grad else b, g)
            assert torch.equal(got, want)
        one = moe.moe_combine(y, w, inv, out_dtype=odt)
        got = torch.autograd.grad(one.sum(), (y, w))
        want = moe.moe_combine_backward(torch.ones_like(one).detach(), y.detach(), w.detach(), inv)
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        x = rand(T, d, seed=4).to(dt).requires_grad_()
        inv, named = padded_slots(T, k, T * k, 5)
        wide = rand(T * k, 2 * d, seed=5).to(dt)
        sent = moe.moe_dispatch(x, inv, k)
        assert sent.requires_grad and torch.equal(sent, moe.moe_dispatch(x.detach(), inv, k))
        got, = torch.autograd.grad(sent, x, wide[:, :d])
        assert torch.equal(got, moe.moe_dispatch_backward(wide[:, :d], inv, k))
        with torch.no_grad():
            assert not moe.moe_dispatch(x, inv, k).requires_grad
            moe.moe_dispatch(x, inv, k, out=torch.zeros_like(sent))
        assert not moe.moe_dispatch(x.detach(), inv, k).requires_grad


def test_recorded_twice(moe):
    """Gradients of the gradients against autograd's of the plain form in 64 bits.  Every value
    is a sum of at most d = 40 products of two factors, in fp32 and in some order: (d + 8) 2^-24
    of the sum of their magnitudes, which the plain form gives for inputs without signs."""
    T, k, d, rows = 30, 3, 40, 100
    inv, _ = padded_slots(T, k, rows, 7)
    at = inv.view(T, k).long()
    ok = ((at >= 0) & (at < rows))[..., None]
    at = torch.where(ok[..., 0], at, 0)
    y, w, g, x = rand(rows, d), rand(T, k), rand(T, d, seed=1), rand(T, d, seed=2)
    u, v = rand(rows, d, seed=3), rand(T, k, seed=4)

    def plain(sign):
        p = [sign(t.double()).clone().requires_grad_() for t in (y, w, g)]
        out = (p[1][..., None] * torch.where(ok, p[0][at], 0.0)).sum(1)
        dy, dw = torch.autograd.grad(out, p[:2], p[2], create_graph=True)
        return torch.autograd.grad((dy * sign(u.double())).sum() + (dw * sign(v.double())).sum(), p)

    def ours():
        p = [t.clone().requires_grad_() for t in (y, w, g)]
        dy, dw = torch.autograd.grad(moe.moe_combine(*p[:2], inv), p[:2], p[2], create_graph=True)
        return torch.autograd.grad((dy * u).sum() + (dw * v).sum(), p)
    for a, b, m in zip(ours(), plain(lambda t: t), plain(torch.abs)):
        assert bool(((a.double() - b).abs() <= (d + 8) * 2.0 ** -24 * m).all())
    # by hand, one output alone
    p = [t.clone().requires_grad_() for t in (g, y, w)]
    dy, none = moe.moe_combine_backward(*p, inv, want_dw=False)
    assert none is None
    got = torch.autograd.grad(dy, p, u, allow_unused=True)
    assert torch.equal(got[0], moe.moe_combine(u, w, inv)) and got[1] is None
    assert torch.equal(got[2], moe.moe_combine_backward(g, u, w, inv, want_dy=False)[1])
    # dispatch is linear: the gradient of its gradient is itself (rows beyond the slots: zeros)
    q = u.clone().requires_grad_()
    got, = torch.autograd.grad(moe.moe_dispatch_backward(q, inv, k), q, x)
    want = torch.zeros_like(u)
    moe.moe_dispatch(x, inv, k, out=want)
    assert torch.equal(got, want)


def test_given_outputs_keep_no_graph(moe):
    """An input requires grad and an output is given: the call runs, without a graph, and warns."""
    x, inv = rand(4, 16).requires_grad_(), perm(8)
    y, w = rand(8, 16).requires_grad_(), torch.rand(4, 2, device=DEV, requires_grad=True)
    calls = ((lambda o: moe.moe_dispatch(x, inv, 2, out=o), (8, 16)), (lambda o: moe.moe_combine(y, w, inv, out=o), (4, 16)),
             (lambda o: moe.moe_dispatch_backward(y, inv, 2, out=o), (4, 16)),
             (lambda o: moe.moe_combine_backward(x, y, w, inv, dy=o)[0], (8, 16)))
    for call, shape in calls:
        out = torch.empty(*shape, device=DEV)
        with pytest.warns(UserWarning, match="given"):
            assert call(out) is out
        assert not out.requires_grad
        with torch.no_grad():
            again = call(None)
        assert torch.equal(out, again)


def test_a_recorded_step_is_captured(moe):
    """Forward and backward of a layer in one graph (warmed up on a side stream), replayed on
    other inputs."""
    T, k, d = 64, 2, 48
    x, w, inv, g = rand(T, d).requires_grad_(), torch.softmax(rand(T, k), 1).requires_grad_(), perm(T * k), rand(T, d, seed=9)
    up, down = rand(d).requires_grad_(), rand(d, seed=1).requires_grad_()
    leaves = (x, w, up, down)

    def step():
        y = torch.relu(moe.moe_dispatch(x, inv, k) * up) * down
        return torch.autograd.grad(moe.moe_combine(y, w, inv), leaves, g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in (11, 12):
        with torch.no_grad():
            x.copy_(rand(T, d, seed=seed))
            inv.copy_(perm(T * k, seed=seed))
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(held, step()))


def test_gradients_beyond_32_bits(moe):
    """dy's rows and a gradient's grouped rows whose elements lie past 2^31, given and new."""
    d, rows = 1032, 2 ** 21 + 9                    # 2.16e9 elements of bf16
    T, k = 3, 2
    inv = torch.tensor([rows - 1, 5, rows - 2, rows - 9, 0, 2 ** 21 - 1], dtype=torch.int32, device=DEV)
    x, w = rand(T, d).bfloat16(), torch.softmax(rand(T, k), 1)
    y = torch.zeros(rows, d, device=DEV, dtype=torch.bfloat16)
    y[inv.long()] = rand(T * k, d, seed=1).bfloat16()
    ref, m = gather_ref(y, inv, T, k)
    close(moe.moe_dispatch_backward(y, inv, k), ref, k * 2.0 ** -24 * m * (1 + 1e-6))
    at = inv.long()
    want = (w.view(-1, 1) * x.float().repeat_interleave(k, 0))
    named = torch.zeros(rows, dtype=torch.bool, device=DEV)
    named[at] = True
    dy = torch.full_like(y, 7.0)
    moe.moe_combine_backward(x, y, w, inv, want_dw=False, dy=dy)
    close(dy[at], want.double(), 2.0 ** -24 * want.abs().double())
    assert int((dy != 7).any(1).sum()) == T * k
    del dy
    new = moe.moe_combine_backward(x, y, w, inv, want_dw=False)[0]
    close(new[at], want.double(), 2.0 ** -24 * want.abs().double())
    assert int((new != 0).any(1).sum()) == T * k
