"""Host-side checks of the 8-bit integer operators and of dispatch and combine: every
refused argument comes back before any CUDA call, from the library and from the binding."""
import ctypes
import os
import re

import pytest

torch = pytest.importorskip("torch")

I, U, W, OK = 1, 2, 3, 0     # MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_OK
F32, BF16, Q8_0 = 0, 1, 2
vp = ctypes.c_void_p
FAKE, ODD8, ODD2, ODD1 = vp(0x10000), vp(0x10008), vp(0x10002), vp(0x10001)   # never dereferenced


@pytest.fixture(scope="module")
def lib():
    from expert_routed_ffn_selectedsoftmax_gb300 import build, binding
    build.build()
    return binding.load_library()


def test_quant_arguments(lib):
    def call(**kw):
        a = dict(dict(x=FAKE, dt=BF16, rows=4, cols=256, ldx=256, q=FAKE, s=FAKE), **kw)
        return lib.moe_quant_i8(*a.values(), None)
    for bad in (dict(dt=Q8_0), dict(dt=9), dict(cols=0), dict(cols=24), dict(cols=-16), dict(ldx=240), dict(ldx=260),
                dict(rows=-1), dict(x=None), dict(q=None), dict(s=None), dict(x=ODD8), dict(q=ODD8), dict(s=ODD2)):
        assert call(**bad) == I, bad
    assert call(rows=0, x=None, q=None, s=None) == OK


def test_product_arguments(lib):
    base = dict(xq=FAKE, xs=FAKE, xr=8, K=256, ldx=256, wq=FAKE, ws=FAKE, E=4, N=64, off=FAKE, perm=None, rows=8, out=FAKE,
                odt=BF16, ldo=64, ws_=FAKE, wsb=1 << 20, st=None)
    gu = dict(xq=FAKE, xs=FAKE, xr=8, K=256, ldx=256, wq=FAKE, ws=FAKE, uq=FAKE, us=FAKE, E=4, N=64, off=FAKE, perm=None, rows=8,
              out=FAKE, odt=BF16, ldo=64, ws_=FAKE, wsb=1 << 20, st=None)
    grouped = lambda **kw: lib.moe_grouped_gemm_i8(*dict(base, **kw).values(), None)
    gate_up = lambda **kw: lib.moe_gate_up_i8(*dict(gu, **kw).values(), None)
    for bad in (dict(xr=-1), dict(K=0), dict(K=24, ldx=32), dict(ldx=240), dict(ldx=264), dict(E=0), dict(N=0), dict(rows=-1),
                dict(off=None), dict(rows=9), dict(xr=0, perm=FAKE), dict(xq=None), dict(xs=None), dict(wq=None), dict(ws=None),
                dict(xq=ODD8), dict(wq=ODD8), dict(xs=ODD2), dict(ws=ODD2), dict(off=ODD2), dict(perm=ODD2), dict(st=ODD2),
                dict(out=None), dict(odt=Q8_0), dict(ldo=63), dict(out=ODD1), dict(odt=F32, out=ODD2)):
        assert grouped(**bad) == I, bad
        assert gate_up(**bad) == I, bad
    for bad in (dict(uq=None), dict(us=None), dict(uq=ODD8), dict(us=ODD2)):
        assert gate_up(**bad) == I, bad
    assert grouped(E=257) == U and gate_up(E=257) == U
    assert grouped(rows=2 ** 30 + 1, xr=2 ** 30 + 1) == U
    assert grouped(rows=0, xr=0, xq=None, out=None) == OK and gate_up(rows=0, xr=0, xq=None, out=None) == OK
    # scratch of widened rows, 2 bytes a code, to 256 bytes; none up to 32 rows
    for rows, K in ((-1, 256), (80, 250), (80, 0), (32, 256)):
        assert lib.moe_i8_workspace_size(rows, K) == 0
    assert lib.moe_i8_workspace_size(33, 48) == 3328
    for call in (grouped, gate_up):
        for bad in (dict(rows=33, xr=33, ws_=None), dict(rows=33, xr=33, ws_=vp(0x10080))):
            assert call(**bad) == I, bad
        assert call(rows=33, xr=33, wsb=33 * 512 - 1) == W
    for role, ns in ((-1, 1000), (3, 1000), (0, 0), (1, 100_000_001)):
        assert lib.moe_grouped_gemm_i8_expire_wait(*base.values(), role, ns, None) == I
        assert lib.moe_gate_up_i8_expire_wait(*gu.values(), role, ns, None) == I
    dense = dict(xq=FAKE, xs=FAKE, T=4, K=256, ldx=256, wq=FAKE, ws=FAKE, N=64, out=FAKE, odt=BF16, ldo=64, ws_=FAKE,
                 wsb=1 << 20, st=None)
    gemm = lambda **kw: lib.moe_gemm_i8(*dict(dense, **kw).values(), None)
    for bad in (dict(T=-1), dict(K=250), dict(ldx=128), dict(N=0), dict(odt=5), dict(ldo=32), dict(xq=None), dict(out=None)):
        assert gemm(**bad) == I, bad
    assert gemm(T=0, xq=None, out=None) == OK


def test_dispatch_and_combine_arguments(lib):
    send = lambda **kw: lib.moe_dispatch(*dict(dict(x=FAKE, dt=F32, T=4, d=5, ldx=5, inv=FAKE, k=2, out=FAKE, rows=8, ldo=5),
                                               **kw).values(), None)
    back = lambda **kw: lib.moe_dispatch_backward(*dict(dict(g=FAKE, dt=F32, rows=8, d=5, ldg=5, inv=FAKE, T=4, k=2, dx=FAKE,
                                                             ldx=5), **kw).values(), None)
    comb = lambda **kw: lib.moe_combine(*dict(dict(y=FAKE, dt=F32, rows=8, d=5, ldy=5, w=FAKE, inv=FAKE, T=4, k=2, out=FAKE,
                                                   odt=F32, ldo=5), **kw).values(), None)
    cback = lambda **kw: lib.moe_combine_backward(*dict(dict(g=FAKE, gdt=F32, T=4, d=5, ldg=5, y=FAKE, dt=F32, rows=8, ldy=5,
                                                             w=FAKE, inv=FAKE, k=2, dy=FAKE, lddy=5, dw=FAKE), **kw).values(), None)
    for call in (send, back, comb, cback):
        for bad in (dict(T=-1), dict(k=0), dict(k=-1), dict(rows=-1), dict(d=0), dict(inv=None), dict(inv=ODD2), dict(dt=Q8_0),
                    dict(dt=7)):
            assert call(**bad) == I, bad
        assert call(k=9) == U and call(T=2 ** 31 - 1) == U
    for bad in (dict(x=None), dict(out=None), dict(ldx=4), dict(ldo=4), dict(x=ODD2), dict(out=ODD1)):
        assert send(**bad) == I, bad
    for bad in (dict(g=None), dict(dx=None), dict(ldg=4), dict(ldx=4), dict(g=ODD2), dict(dx=ODD1)):
        assert back(**bad) == I, bad
    for bad in (dict(y=None), dict(out=None), dict(w=None), dict(ldy=4), dict(ldo=4), dict(odt=3), dict(w=ODD2), dict(y=ODD2)):
        assert comb(**bad) == I, bad
    for bad in (dict(g=None), dict(y=None), dict(w=None), dict(ldg=4), dict(ldy=4), dict(lddy=4), dict(gdt=3), dict(w=ODD2),
                dict(dw=ODD2), dict(dy=ODD1), dict(g=ODD1)):
        assert cback(**bad) == I, bad
    assert send(T=0, x=None, out=None, inv=None) == OK and send(rows=0, out=None) == OK
    assert back(T=0, g=None, dx=None, inv=None) == OK
    assert comb(T=0, y=None, out=None, w=None, inv=None) == OK
    assert cback(T=0, g=None, y=None, w=None, inv=None) == OK
    assert cback(dy=None, dw=None, y=None) == OK


def test_binding_refuses_wrong_pairs():
    """Shapes, types, devices and strides are checked before the library is called (CPU
    tensors: a call that passes every check ends at the device's)."""
    import expert_routed_ffn_selectedsoftmax_gb300 as moe
    i8 = torch.int8
    xq, xs = torch.zeros(4, 256, dtype=i8), torch.zeros(4)
    wq, ws = torch.zeros(3, 200, 256, dtype=i8), torch.zeros(3, 200)
    off, perm = torch.zeros(4, dtype=torch.int32), torch.zeros(8, dtype=torch.int32)
    good = dict(x_q=xq, x_s=xs, w_q=wq, w_s=ws, offsets=off, perm_tok=perm)
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_grouped_gemm_i8(**good)
    for bad, err in ((dict(x_s=torch.zeros(4, 1)), ValueError), (dict(x_s=torch.zeros(5)), ValueError),
                     (dict(w_s=torch.zeros(3, 1)), ValueError), (dict(offsets=off[:3]), ValueError),
                     (dict(offsets=off.long()), TypeError), (dict(perm_tok=perm.long()), TypeError),
                     (dict(perm_tok=torch.zeros(16, dtype=torch.int32)[::2]), ValueError),
                     (dict(x_q=xq.to(torch.uint8)), TypeError), (dict(x_q=torch.zeros(4, 512, dtype=i8)[:, ::2]), ValueError),
                     (dict(w_q=wq.transpose(1, 2)), ValueError), (dict(out_dtype=torch.float16), TypeError),
                     (dict(out_dtype="bf16"), TypeError), (dict(out=torch.zeros(4, 200)), ValueError),
                     (dict(offsets=None), ValueError), (dict(status=torch.zeros(1)), TypeError)):
        with pytest.raises(err):
            moe.moe_grouped_gemm_i8(**dict(good, **bad))
    for bad in (dict(w_q=torch.zeros(200, 128, dtype=i8)), dict(w_q=wq), dict(w_s=torch.zeros(2)), dict(out=torch.zeros(4, 100))):
        with pytest.raises(ValueError):
            moe.moe_gemm_i8(**dict(dict(x_q=xq, x_s=xs, w_q=wq[0], w_s=ws[0]), **bad))
    gu = dict(x_q=xq, x_s=xs, wg_q=wq, wg_s=ws, wu_q=wq, wu_s=ws, offsets=off, perm_tok=perm)
    for bad in (dict(wu_q=wq[:2]), dict(wu_s=ws[:2]), dict(h=torch.zeros(4, 200))):
        with pytest.raises(ValueError):
            moe.moe_gate_up_i8(**dict(gu, **bad))
    with pytest.raises(TypeError):
        moe.moe_gate_up_i8(**dict(gu, h_dtype=torch.int8))
    x = torch.zeros(4, 256)
    for bad, err in ((dict(x=torch.zeros(256)), ValueError), (dict(x=torch.zeros(4, 4, dtype=torch.int32)), TypeError),
                     (dict(x=x.t()), ValueError), (dict(x=torch.zeros(2, 4, 512)[:, :3]), ValueError), (dict(x=[1.0]), TypeError),
                     (dict(scales=torch.zeros(4, 2)), ValueError), (dict(codes=torch.zeros(4, 256)), TypeError), (dict(), ValueError)):
        with pytest.raises(err):
            moe.moe_quant_i8(**dict(dict(x=x), **bad))


def test_binding_refuses_wrong_slots():
    import expert_routed_ffn_selectedsoftmax_gb300 as moe
    x, y, w, inv = torch.zeros(4, 10), torch.zeros(8, 10), torch.zeros(4, 2), torch.zeros(8, dtype=torch.int32)
    for call in (lambda: moe.moe_dispatch(x, inv, 2), lambda: moe.moe_dispatch_backward(y, inv, 2),
                 lambda: moe.moe_combine(y, w, inv), lambda: moe.moe_combine_backward(x, y, w, inv)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    for args, err in (((x, inv[:7], 2), ValueError), ((x, inv, 4), ValueError), ((x, inv, 0), ValueError), ((x, inv, -2), ValueError),
                      ((x, inv, None), TypeError), ((x, inv.long(), 2), TypeError), ((x.half(), inv, 2), TypeError),
                      ((x[0], inv, 2), ValueError), ((x.t(), inv, 2), ValueError), ((x, inv, 2, torch.zeros(8, 9)), ValueError),
                      ((x, inv, 2, y.bfloat16()), TypeError)):
        with pytest.raises(err):
            moe.moe_dispatch(*args)
    for args, err in (((y, inv, 3), ValueError), ((y, inv, 2, torch.zeros(5, 10)), ValueError), ((y, inv.float(), 2), TypeError)):
        with pytest.raises(err):
            moe.moe_dispatch_backward(*args)
    for kw, err in ((dict(topk_w=w[:3]), ValueError), (dict(topk_w=w.double()), TypeError), (dict(topk_w=w.view(-1)), ValueError),
                    (dict(inv=inv[:6]), ValueError), (dict(out=torch.zeros(4, 9)), ValueError), (dict(out_dtype=torch.float64), TypeError),
                    (dict(y=y.view(2, 4, 10)), ValueError)):
        with pytest.raises(err):
            moe.moe_combine(**dict(dict(y=y, topk_w=w, inv=inv), **kw))
    for kw, err in ((dict(grad=torch.zeros(4, 9)), ValueError), (dict(grad=torch.zeros(5, 10)), ValueError),
                    (dict(dy=torch.zeros(7, 10)), ValueError), (dict(dy=y.bfloat16()), TypeError), (dict(dw=torch.zeros(8)), ValueError),
                    (dict(dy=y, want_dy=False), ValueError), (dict(dw=w, want_dw=False), ValueError)):
        with pytest.raises(err):
            moe.moe_combine_backward(**dict(dict(grad=x, y=y, topk_w=w, inv=inv), **kw))
    with pytest.raises(RuntimeError, match="ambiguous"):
        moe.moe_combine_backward(x, y, w, inv, want_dy=torch.ones(2))


def source(name):
    """A kernel's source without its comments."""
    text = open(os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "expert_routed_ffn_selectedsoftmax_gb300", "csrc",
                             name)).read()
    return re.sub(r"//[^\n]*", "", text)


def warp_waits(name):
    """The statements of a kernel's source that wait on a barrier as part of a role (not the ones
    that let copies and MMAs in flight end, which nothing follows)."""
    found = [s for s in re.split(r"[;{}]", source(name)) if re.search(r"\b(bar_wait|mbar_wait_slow)\(&", s)]
    return [" ".join(s.split()) for s in found if "no_abort" not in s]


@pytest.mark.parametrize("name", ["i8_tc.cu"])
def test_a_warp_gives_up_as_a_whole(name):
    """A bounded wait's answer is each lane's own (its lanes poll one after the other): a role
    that a whole warp runs takes the warp's vote, or lanes that give up would leave the
    others at a barrier of the full warp."""
    waits = warp_waits(name)
    assert len(waits) >= 4
    for statement in waits:
        # (the multiplying warps vote once behind both of theirs)
        assert "__all_sync(0xffffffffu" in statement or re.match(r"(bool )?mine_ok = ", statement), statement
    role = source(name)
    role = role[role.index("bool mine_ok"):]
    assert "__all_sync(0xffffffffu, mine_ok)" in role[:role.index("issued = it")]


@pytest.mark.parametrize("name", ["fp8b_decode.cu", "fp8b_gemm.cu"])
def test_an_unvoted_role_ends_as_a_whole(name):
    """The multiplying warps of the block-scaled fp8 products wait lane by lane and hold no
    barrier of the warp in their loop; how much they have issued, which decides whether the
    whole warp waits for it after a wait that gave up, is taken over all lanes."""
    text = source(name)
    role = text[text.index("const bool leader = elect_one()"):]
    role = role[:role.index("} else {")]
    assert role.count("bar_wait(&") == 2 and "__syncwarp" not in role and "__all_sync" not in role
    assert "issued = __reduce_max_sync(0xffffffffu, it)" in role and "issued = it" not in role


def test_widths_near_the_end_of_32_bits_are_refused(lib):
    """A tile's, or a thread's, columns may end behind the matrix's last one and are counted in
    32 bits: widths within 256 of 2^31 are not taken."""
    most = 2 ** 31 - 1
    for d in (most, most - 255):
        for dt in (F32, BF16):
            assert lib.moe_dispatch(FAKE, dt, 1, d, d, FAKE, 1, FAKE, 1, d, None) == U
            assert lib.moe_dispatch_backward(FAKE, dt, 1, d, d, FAKE, 1, 1, FAKE, d, None) == U
            assert lib.moe_combine(FAKE, dt, 1, d, d, FAKE, FAKE, 1, 1, FAKE, dt, d, None) == U
            assert lib.moe_combine_backward(FAKE, dt, 1, d, d, FAKE, dt, 1, d, FAKE, FAKE, 1, FAKE, d, FAKE, None) == U
    for K, N in ((16, most), (16, most - 255), (most - 15, 16), (most - 255, 16)):
        K -= K % 16
        wide = 1 << 40
        assert lib.moe_gemm_i8(FAKE, FAKE, 1, K, K, FAKE, FAKE, N, FAKE, BF16, N, FAKE, wide, None, None) == U
        assert lib.moe_grouped_gemm_i8(FAKE, FAKE, 1, K, K, FAKE, FAKE, 1, N, None, None, 1, FAKE, F32, N, FAKE, wide, None, None) == U
        assert lib.moe_gate_up_i8(FAKE, FAKE, 1, K, K, FAKE, FAKE, FAKE, FAKE, 1, N, None, None, 1, FAKE, F32, N, FAKE, wide, None,
                                  None) == U
        assert lib.moe_gemm_fp8b(FAKE, FAKE, 1, K, K, FAKE, FAKE, N, FAKE, F32, N, None, None) == U
        assert lib.moe_gate_up_fp8b(FAKE, FAKE, 1, K, K, FAKE, FAKE, FAKE, FAKE, 1, N - N % 16, None, None, 1, FAKE, FAKE, FAKE, wide,
                                    None, None) == U


def test_filled_forms_check_what_the_plain_ones_do(lib):
    send = lambda **kw: lib.moe_dispatch_filled(*dict(dict(x=FAKE, dt=F32, T=4, d=5, ldx=5, inv=FAKE, k=2, out=FAKE, rows=8, ldo=5),
                                                      **kw).values(), None)
    back = lambda **kw: lib.moe_combine_backward_filled(*dict(
        dict(g=FAKE, gdt=F32, T=4, d=5, ldg=5, y=FAKE, dt=F32, rows=8, ldy=5, w=FAKE, inv=FAKE, k=2, dy=FAKE, lddy=5, dw=FAKE),
        **kw).values(), None)
    for call in (send, back):
        for bad in (dict(T=-1), dict(k=0), dict(rows=-1), dict(d=0), dict(inv=None), dict(inv=ODD2), dict(dt=Q8_0)):
            assert call(**bad) == I, bad
        assert call(k=9) == U and call(T=2 ** 31 - 1) == U
    for bad in (dict(x=None), dict(out=None), dict(ldo=4), dict(out=ODD1), dict(T=0, out=None)):
        assert send(**bad) == I, bad
    for bad in (dict(g=None), dict(y=None), dict(w=None), dict(lddy=4), dict(dw=ODD2), dict(dy=ODD1)):
        assert back(**bad) == I, bad
    assert send(rows=0, out=None) == OK and send(T=0, rows=0, x=None, out=None, inv=None) == OK
    assert back(T=0, rows=0, g=None, y=None, w=None, inv=None) == OK and back(T=0, dy=None, g=None, y=None, w=None, inv=None) == OK
    assert back(dy=None, dw=None, y=None) == OK
