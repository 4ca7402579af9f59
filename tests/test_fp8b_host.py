"""Host-side checks of the block-scaled fp8 operators: every refused argument
comes back before any CUDA call, from the library and from the binding."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

I, U, OK = 1, 2, 0     # MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_OK
F32, BF16, Q8_0 = 0, 1, 2
vp = ctypes.c_void_p
FAKE, ODD = vp(0x10000), vp(0x10004)    # never dereferenced: every call here fails validation (or is empty)
ODD2 = vp(0x10001)


@pytest.fixture(scope="module")
def lib():
    from expert_routed_ffn_selectedsoftmax_gb300 import build, binding
    build.build()
    return binding.load_library()


def test_quant_arguments(lib):
    base = dict(x=FAKE, dt=BF16, batch=2, rows=4, cols=256, ldx=256, br=1, q=FAKE, s=FAKE)

    def call(**kw):
        a = dict(base, **kw)
        return lib.moe_quant_fp8b(a["x"], a["dt"], a["batch"], a["rows"], a["cols"], a["ldx"], a["br"], a["q"],
                                  a["s"], None)
    for bad in (dict(dt=Q8_0), dict(dt=9), dict(cols=0), dict(cols=24), dict(cols=-16), dict(ldx=240),
                dict(ldx=260), dict(br=0), dict(br=64), dict(rows=-1), dict(batch=-1), dict(x=None), dict(q=None),
                dict(s=None), dict(x=ODD), dict(q=ODD), dict(s=ODD2)):
        assert call(**bad) == I, bad
    assert call(rows=0, x=None, q=None, s=None) == OK
    assert call(batch=0, x=None, q=None, s=None) == OK


def test_norm_arguments(lib):
    base = dict(x=FAKE, dt=F32, T=4, d=256, ldx=256, delta=FAKE, ddt=BF16, n=8, ldd=256, w=FAKE, inv=FAKE, k=2,
                g=FAKE, gdt=F32, eps=1e-6, r=FAKE, y=FAKE, q=FAKE, s=FAKE)

    def call(**kw):
        a = dict(base, **kw)
        return lib.moe_norm_fp8b(a["x"], a["dt"], a["T"], a["d"], a["ldx"], a["delta"], a["ddt"], a["n"], a["ldd"],
                                 a["w"], a["inv"], a["k"], a["g"], a["gdt"], a["eps"], a["r"], a["y"], a["q"],
                                 a["s"], None)
    for bad in (dict(dt=Q8_0), dict(ddt=Q8_0), dict(gdt=6), dict(T=-1), dict(d=0), dict(d=40), dict(ldx=248),
                dict(ldx=260), dict(ldd=128), dict(ldd=257), dict(k=-1), dict(eps=-1.0), dict(eps=float("nan")),
                dict(x=None), dict(g=None), dict(q=None), dict(s=None), dict(r=None), dict(delta=None),
                dict(w=None), dict(inv=None), dict(n=-1), dict(k=0, n=3), dict(x=ODD), dict(delta=ODD),
                dict(g=ODD), dict(r=ODD), dict(y=ODD), dict(q=ODD), dict(s=ODD2), dict(w=ODD2), dict(inv=ODD2)):
        assert call(**bad) == I, bad
    assert call(k=9) == U
    assert call(d=16400, ldx=16400, ldd=16400) == U
    assert call(T=0, x=None, g=None, q=None, s=None) == OK


def test_product_arguments(lib):
    base = dict(xq=FAKE, xs=FAKE, xr=8, K=256, ldx=256, wq=FAKE, ws=FAKE, E=4, N=64, off=FAKE, perm=None, rows=8,
                out=FAKE, odt=BF16, ldo=64, ws_=FAKE, wsb=1 << 20, st=None)

    def grouped(**kw):
        a = dict(base, **kw)
        return lib.moe_grouped_gemm_fp8b(a["xq"], a["xs"], a["xr"], a["K"], a["ldx"], a["wq"], a["ws"], a["E"],
                                         a["N"], a["off"], a["perm"], a["rows"], a["out"], a["odt"], a["ldo"],
                                         a["ws_"], a["wsb"], a["st"], None)

    def gate_up(**kw):
        a = dict(dict(base, uq=FAKE, us=FAKE, hq=FAKE, hs=FAKE), **kw)
        return lib.moe_gate_up_fp8b(a["xq"], a["xs"], a["xr"], a["K"], a["ldx"], a["wq"], a["ws"], a["uq"],
                                    a["us"], a["E"], a["N"], a["off"], a["perm"], a["rows"], a["hq"], a["hs"],
                                    a["ws_"], a["wsb"], a["st"], None)
    both = (dict(xr=-1), dict(K=0), dict(K=24, ldx=32), dict(ldx=240), dict(ldx=264), dict(E=0), dict(N=0),
            dict(rows=-1), dict(off=None), dict(rows=9), dict(xr=0, perm=FAKE), dict(xq=None), dict(xs=None),
            dict(wq=None), dict(ws=None), dict(xq=ODD), dict(wq=ODD), dict(xs=ODD2), dict(ws=ODD2),
            dict(off=ODD2), dict(perm=ODD2), dict(st=ODD2), dict(perm=FAKE, ws_=None), dict(perm=FAKE, ws_=vp(0x10080)))
    for bad in both:
        assert grouped(**bad) == I, bad
        assert gate_up(**bad) == I, bad
    for bad in (dict(out=None), dict(odt=Q8_0), dict(ldo=63), dict(out=ODD2)):
        assert grouped(**bad) == I, bad
    for bad in (dict(N=72), dict(uq=None), dict(us=None), dict(hq=None), dict(hs=None), dict(uq=ODD), dict(hq=ODD),
                dict(us=ODD2), dict(hs=ODD2)):
        assert gate_up(**bad) == I, bad
    # scratch of gathered rows: 8 x 256 codes and 8 x 2 scales, each to 256 bytes
    assert lib.moe_fp8b_workspace_size(8, 256) == 2048 + 256
    assert lib.moe_fp8b_workspace_size(8, 250) == 0 and lib.moe_fp8b_workspace_size(-1, 256) == 0
    assert grouped(perm=FAKE, wsb=2303) == 3 and gate_up(perm=FAKE, wsb=2303) == 3      # MOE_ERR_WORKSPACE
    assert grouped(E=257) == U and gate_up(E=257) == U
    assert grouped(rows=0, xr=0, xq=None, out=None) == OK and gate_up(rows=0, xr=0, xq=None, hq=None) == OK
    for ns in (0, 100_000_001):
        assert lib.moe_grouped_gemm_fp8b_expire_wait(FAKE, FAKE, 8, 256, 256, FAKE, FAKE, 4, 64, FAKE, None, 8, FAKE, F32,
                                                     64, None, 0, None, ns, None) == I
    g = lambda **kw: lib.moe_gemm_fp8b(*dict(dict(a=FAKE, b=FAKE, T=4, K=256, l=256, c=FAKE, d=FAKE, N=64, o=FAKE,
                                                  t=BF16, m=64, s=None, z=None), **kw).values())
    for bad in (dict(T=-1), dict(K=250), dict(l=128), dict(N=0), dict(t=5), dict(m=32), dict(a=None), dict(o=None)):
        assert g(**bad) == I, bad
    assert g(T=0, a=None, o=None) == OK


def test_hook_arguments(lib):
    """The wait's limit of the hooks: 1 ns to 100 ms."""
    for ns in (0, 100_000_001):
        assert lib.moe_grouped_gemm_fp8b_expire_sums(FAKE, FAKE, 8, 256, 256, FAKE, FAKE, 4, 64, FAKE, None, 8, FAKE, F32,
                                                     64, None, 0, None, ns, None) == I
        for hook in (lib.moe_gate_up_fp8b_expire_wait, lib.moe_gate_up_fp8b_expire_sums):
            assert hook(FAKE, FAKE, 8, 256, 256, FAKE, FAKE, FAKE, FAKE, 4, 64, FAKE, None, 8, FAKE, FAKE, None, 0, None,
                        ns, None) == I


def test_binding_refuses_wrong_pairs():
    """Shapes, types, devices and strides are checked before the library is
    called (CPU tensors: a call that passes every check ends at the device's)."""
    import expert_routed_ffn_selectedsoftmax_gb300 as moe
    f8 = torch.float8_e4m3fn
    xq, xs = torch.zeros(4, 256).to(f8), torch.zeros(4, 2)
    wq, ws = torch.zeros(3, 200, 256).to(f8), torch.zeros(3, 2, 2)
    off, perm = torch.zeros(4, dtype=torch.int32), torch.zeros(8, dtype=torch.int32)
    good = dict(x_q=xq, x_s=xs, w_q=wq, w_s=ws, offsets=off, perm_tok=perm)
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_grouped_gemm_fp8b(**good)
    for bad, err in ((dict(x_s=torch.zeros(4, 3)), ValueError), (dict(w_s=torch.zeros(3, 1, 2)), ValueError),
                     (dict(offsets=off[:3]), ValueError), (dict(offsets=off.long()), TypeError),
                     (dict(perm_tok=perm.long()), TypeError), (dict(perm_tok=torch.zeros(16, dtype=torch.int32)[::2]), ValueError),
                     (dict(x_q=torch.zeros(4, 256)), TypeError), (dict(x_q=torch.zeros(4, 512).to(f8)[:, ::2]), ValueError),
                     (dict(w_q=wq.transpose(1, 2)), ValueError), (dict(out_dtype=torch.float16), TypeError),
                     (dict(out=torch.zeros(4, 200)), ValueError), (dict(offsets=None), ValueError),
                     (dict(status=torch.zeros(1)), TypeError)):
        with pytest.raises(err):
            moe.moe_grouped_gemm_fp8b(**dict(good, **bad))
    for bad in (dict(w_q=torch.zeros(200, 128).to(f8)), dict(w_s=torch.zeros(2, 3)), dict(out=torch.zeros(4, 100))):
        with pytest.raises(ValueError):
            moe.moe_gemm_fp8b(**dict(dict(x_q=xq, x_s=xs, w_q=wq[0], w_s=ws[0]), **bad))
    gu = dict(x_q=xq, x_s=xs, wg_q=wq, wg_s=ws, wu_q=wq, wu_s=ws, offsets=off, perm_tok=perm)
    for bad in (dict(wu_q=wq[:2]), dict(wu_s=ws[:2]), dict(h_q=torch.zeros(4, 200).to(f8)), dict(h_s=torch.zeros(8, 1))):
        with pytest.raises(ValueError):
            moe.moe_gate_up_fp8b(**dict(gu, **bad))
    x = torch.zeros(4, 256)
    nm = dict(x=x, weight=torch.ones(256), delta=torch.zeros(8, 256), topk_w=torch.zeros(4, 2), inv=perm)
    for bad, err in ((dict(weight=torch.ones(128)), ValueError), (dict(inv=perm[:7]), ValueError),
                     (dict(inv=None), ValueError), (dict(delta=None), ValueError),
                     (dict(delta=torch.zeros(4, 128)), ValueError), (dict(x=x.half()), TypeError),
                     (dict(resid=torch.zeros(4, 256).bfloat16()), TypeError), (dict(topk_w=nm["topk_w"].double()), TypeError),
                     (dict(delta=torch.zeros(3, 256), topk_w=None, inv=None), ValueError)):
        with pytest.raises(err):
            moe.moe_norm_fp8b(**dict(nm, **bad))
    for bad, err in ((dict(x=torch.zeros(256)), ValueError), (dict(block_rows=64), ValueError),
                     (dict(x=torch.zeros(4, 4, dtype=torch.int32)), TypeError), (dict(x=x.t()), ValueError),
                     (dict(x=torch.zeros(2, 4, 512)[:, :3]), ValueError), (dict(x=[1.0]), TypeError), (dict(scales=torch.zeros(4, 3)), ValueError)):
        with pytest.raises(err):
            moe.moe_quant_fp8b(**dict(dict(x=x), **bad))


def test_binding_passes_on_python_errors():
    """An argument whose conversion raises gives that error, not a later one's."""
    import expert_routed_ffn_selectedsoftmax_gb300 as moe
    x, w = torch.zeros(4, 256), torch.ones(256)
    with pytest.raises(RuntimeError, match="ambiguous"):
        moe.moe_norm_fp8b(x, w, want_normed=torch.ones(2))
    with pytest.raises(TypeError):
        moe.moe_norm_fp8b(x, w, eps="small")
    with pytest.raises(TypeError):
        moe.moe_quant_fp8b(x, block_rows=None)
